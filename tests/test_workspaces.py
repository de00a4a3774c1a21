"""Workspaces that the binding takes from torch's allocator: on which stream, and for how long."""
import contextlib
import weakref

import pytest
import torch

from gaussian_mixture_sequence_gb300 import gma

DEV = "cuda:0"


def test_a_workspace_is_allocated_on_the_stream_of_the_call(monkeypatch):
    current, taken = ["default"], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", lambda n, **kw: taken.append((n, current[-1])))
    gma._alloc(100, DEV, None)
    gma._alloc(0, DEV, "side")
    assert taken == [(100, "default"), (16, "side")] and current == ["default"]


class _Held:
    """A library whose calls record whether the workspace that was handed out is still held."""

    def __init__(self, block):
        self.block, self.held = block, []

    def __getattr__(self, name):
        if name.endswith("_size"):
            return lambda *a: 64

        def call(*a):
            self.held.append(self.block() is not None)
            return 0
        return call


@pytest.mark.parametrize("name", ["responsibilities", "stats", "causal", "bidir", "cross", "backward", "decode", "beam",
                                  "balance", "balance_backward"])
def test_a_workspace_is_held_until_the_launches_are_queued(monkeypatch, name):
    """On host tensors, with the library and the checks of pointers replaced."""
    block = [lambda: None]

    def alloc(need, dev, stream):
        t = torch.empty(max(need, 16), dtype=torch.uint8)
        block[0] = weakref.ref(t)
        return t

    lib = _Held(lambda: block[0]())
    monkeypatch.setattr(gma, "_alloc", alloc)
    monkeypatch.setattr(gma, "_lib", lib)
    monkeypatch.setattr(gma, "load", lambda: lib)
    monkeypatch.setattr(gma, "_ptr", lambda *a, **k: 16)
    monkeypatch.setattr(gma, "_p", lambda *a, **k: 16)
    monkeypatch.setattr(gma, "_device_index", lambda *a: 0)
    monkeypatch.setattr(gma, "_current_device", lambda: 0)
    monkeypatch.setattr(gma, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(gma, "_stream", lambda dev, stream: None)
    _calls("cpu", small=True)[name][1](None)
    assert lib.held == [True] and block[0]() is None


def _calls(dev=DEV, small=False):
    """name -> (workspace bytes, call(stream)) of every kind of entry point that takes a workspace."""
    g = torch.Generator(device=dev).manual_seed(3)
    mk = lambda *s: torch.randn(*s, device=dev, generator=g)
    B, H, N, D, K = 2, 2, 3 if small else 300, 64, 128
    s = gma.Shape.make(B, H, N, D, 64, K)
    prm = (mk(H, K, D), mk(H, K, D), mk(H, K))
    q, k, v, out = mk(B, H, N, D), mk(B, H, N, D), mk(B, H, N, 64), mk(B, H, N, 64)
    gamma, rows = mk(B, H, N, K), [mk(B, H, N, D) for _ in range(3)]
    loss, prob, usage, ent = mk(H), mk(H, K), mk(H, K), mk(H, 2)
    counts = torch.zeros(H, K, dtype=torch.int64, device=dev)
    grads = [mk(*p.shape) for p in prm]
    state, tok, tout = mk(B, H, K * 64 + K), mk(B, H, 64), mk(B, H, 64)
    V = 40 if small else 40000
    bs = gma.BeamShape.make(16, 8, V)
    logits, score, sco = mk(16, 8, V), mk(16, 8), mk(16, 8)
    par, ids = (torch.zeros(16, 8, dtype=torch.int32, device=dev) for _ in range(2))
    size = lambda op: gma.gma_workspace_size(s, op)
    return {
        "responsibilities": (size(gma.OP_RESPONSIBILITIES),
                             lambda st: gma.gma_responsibilities(s, *prm, q, gamma, stream=st)),
        "stats": (size(gma.OP_USAGE),
                  lambda st: gma.gma_responsibility_stats(s, *prm, q, usage, counts, ent, stream=st)),
        "causal": (size(gma.OP_CAUSAL), lambda st: gma.gma_forward_causal(s, *prm, q, k, v, out, stream=st)),
        "bidir": (size(gma.OP_BIDIR), lambda st: gma.gma_forward_bidir(s, *prm, q, k, v, out, stream=st)),
        "cross": (gma.gma_cross_workspace_size(s, N),
                  lambda st: gma.gma_forward_cross(s, *prm, q, k, v, out, stream=st)),
        "backward": (size(gma.OP_BACKWARD),
                     lambda st: gma.gma_backward(s, *prm, q, k, v, out, *rows, *grads, stream=st)),
        "decode": (size(gma.OP_DECODE), lambda st: gma.gma_decode_step(s, *prm, tok, tok, tok, state, tout, stream=st)),
        "beam": (gma.gma_beam_workspace_size(bs),
                 lambda st: gma.gma_beam_select(bs, logits, score, sco, par, ids, stream=st)),
        "balance": (gma.gma_balance_workspace_size(s),
                    lambda st: gma.gma_balance_loss(s, *prm, q, gamma, loss, counts, prob, stream=st)),
        "balance_backward": (gma.gma_balance_workspace_size(s),
                             lambda st: gma.gma_balance_backward(s, *prm, q, gamma, counts, loss, rows[0], *grads,
                                                                 stream=st)),
    }


@pytest.mark.gpu
def test_a_call_on_another_stream_leaves_blocks_with_pending_work_alone():
    """A block is freed while a copy from it is still queued on the current stream; a call on another
    stream that takes a workspace of its size must not get it."""
    side = torch.cuda.Stream()
    for name, (need, call) in _calls().items():
        assert need > 0, name
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        block = torch.full((need,), 0x5A, dtype=torch.uint8, device=DEV)
        copy = torch.zeros_like(block)
        torch.cuda._sleep(100_000_000)   # some 50 ms
        copy.copy_(block)
        del block
        call(side)
        torch.cuda.synchronize()
        assert (copy == 0x5A).all(), name
