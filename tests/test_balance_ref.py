"""The balance loss's 64-bit formulas against central differences (the counts held, as they pass no
gradient), and the refusals of the entry points (host-side: nothing is launched)."""
import ctypes

import numpy as np
import pytest

import op_refs
from gaussian_mixture_sequence_gb300 import build as gbuild
from gaussian_mixture_sequence_gb300 import gma


@pytest.mark.parametrize("lengths", [None, [4, 0], [1, 6]])
def test_gradient_formulas_against_differences(lengths):
    rng = np.random.default_rng(5)
    B, H, N, D, K = 2, 2, 6, 3, 4
    x, mu = rng.standard_normal((B, H, N, D)), rng.standard_normal((H, K, D))
    r, lp = rng.standard_normal((H, K, D)), rng.standard_normal((H, K))
    w = rng.standard_normal(H)
    gamma, _, counts, _ = op_refs.balance(x, mu, r, lp, lengths)
    T = max(1, op_refs.lengths_of(lengths, B, N).sum())

    def loss(*a):
        return (w * K * (counts / T * op_refs.balance(*a, lengths)[3]).sum(1)).sum()

    got = op_refs.balance_grad(x, mu, r, lp, gamma, counts, w, lengths)
    args = [x, mu, r, lp]
    for i, name in enumerate(("dx", "dmu", "dvar_raw", "dlogit_pi")):
        num = np.zeros_like(args[i])
        for at in np.ndindex(num.shape):
            v = [a.copy() for a in args]
            v[i][at] += 1e-5
            up = loss(*v)
            v[i][at] -= 2e-5
            num[at] = (up - loss(*v)) / 2e-5
        # differences at step 1e-5: truncation and rounding both below 1e-8 here
        assert np.abs(num - got[name][0]).max() < 1e-8, name


def test_loss_of_uniform_and_of_collapsed_use():
    K, D = 4, 2
    mu = np.stack([np.array([[10.0 * k, 0.0] for k in range(K)])])
    r, lp = np.ones((1, K, D)), np.zeros((1, K))
    even = np.repeat(mu[0], 3, 0)[None, None]
    _, loss, counts, prob = op_refs.balance(even, mu, r, lp)
    assert counts.tolist() == [[3, 3, 3, 3]] and np.allclose(loss, 1.0) and np.allclose(prob, 0.25)
    _, loss, counts, _ = op_refs.balance(np.repeat(mu[0, :1], 12, 0)[None, None], mu, r, lp)
    assert counts.tolist() == [[12, 0, 0, 0]] and np.allclose(loss, 4.0)


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gma.load()


PRM = ("mu", "var_raw", "logit_pi")
FWD = ("x", "lengths", "gamma", "loss", "counts", "prob", "ws")
BWD = ("x", "lengths", "gamma", "counts", "dloss", "dx", "dmu", "dvar_raw", "dlogit_pi", "ws")


def _at(n):
    return (1 << 30) + (PRM + FWD + BWD).index(n) * (1 << 28)


def _call(lib, names, shape, wn=1 << 40, accumulate=0, **kw):
    p = {**{n: _at(n) for n in PRM + names}, **kw}
    prm = gma._Params(*(p[n] for n in PRM))
    ref = ctypes.byref(shape) if shape is not None else None
    if names is FWD:
        return lib.gma_balance_loss(ref, prm, *(p[n] for n in FWD), wn, None)
    return lib.gma_balance_backward(ref, prm, *(p[n] for n in BWD[:-1]), accumulate, p["ws"], wn, None)


def _shape(**kw):
    return gma.Shape.make(**{**dict(B=2, H=3, N=100, d_route=64, d_v=64, K=128), **kw})


@pytest.mark.parametrize("kw,status", [(dict(d_route=48), 2), (dict(K=513), 2), (dict(B=0), 1), (dict(N=-1), 1),
                                       (dict(K=0), 1), (dict(B=300, H=300), 2)])
def test_rejects_bad_shapes(lib, kw, status):
    s = _shape(**kw)
    assert gma.gma_balance_workspace_size(s) == 0
    for names in (FWD, BWD):
        assert _call(lib, names, s) == status
        assert _call(lib, names, None) == 1


def test_rejects_bad_buffers(lib):
    s = _shape()
    need = gma.gma_balance_workspace_size(s)
    assert need > gma.gma_workspace_size(s, gma.OP_RESPONSIBILITIES)
    for names in (FWD, BWD):
        for n in PRM + names:
            if n == "ws":
                assert _call(lib, names, s, ws=None) == 4 and _call(lib, names, s, wn=need - 1) == 4
            elif n != "lengths":
                assert _call(lib, names, s, **{n: None}) == 1, n
            assert _call(lib, names, s, **{n: _at(n) + 4}) == 3, n
    for a, b in (("gamma", "x"), ("loss", "prob"), ("counts", "mu"), ("ws", "gamma"), ("prob", "lengths")):
        assert _call(lib, FWD, s, **{a: _at(b)}) == 1, (a, b)
    for a, b in (("dx", "x"), ("dx", "gamma"), ("dmu", "dvar_raw"), ("dlogit_pi", "logit_pi"), ("dmu", "mu"),
                 ("ws", "dx"), ("dvar_raw", "counts"), ("dlogit_pi", "dloss")):
        assert _call(lib, BWD, s, **{a: _at(b)}) == 1, (a, b)
    assert _call(lib, BWD, s, accumulate=2) == 1


def test_empty_sequences_leave_accumulated_gradients(lib):
    # no rows and nothing to overwrite: nothing is launched
    s = _shape(N=0)
    assert _call(lib, BWD, s, accumulate=1, x=None, gamma=None, dx=None) == 0


def test_binding_refuses_host_tensors():
    import torch
    s = _shape(B=1, H=1, N=4, d_route=16, K=2)
    z = torch.zeros
    p = (z(1, 2, 16), z(1, 2, 16), z(1, 2))
    with pytest.raises(TypeError, match="CUDA tensor"):
        gma.gma_balance_loss(s, *p, z(1, 1, 4, 16), z(1, 1, 4, 2), z(1), z(1, 2), z(1, 2))
    with pytest.raises(TypeError, match="CUDA tensor"):
        gma.gma_balance_backward(s, *p, z(1, 1, 4, 16), z(1, 1, 4, 2), z(1, 2), z(1), *p, z(1))


@pytest.mark.parametrize("N", [(1 << 30) + 1, (1 << 31) - 200, (1 << 31) - 1])
def test_rejects_sequences_whose_positions_would_pass_31_bits(lib, N):
    s = _shape(B=1, H=1, N=N, d_route=16, d_v=16, K=2)
    assert gma.gma_balance_workspace_size(s) == 0
    for names in (FWD, BWD):
        assert _call(lib, names, s) == 2
    s.N = 1 << 30   # passes the shape's checks (the parameter's alignment is what fails)
    assert gma.gma_balance_workspace_size(s) > 0
    for names in (FWD, BWD):
        assert _call(lib, names, s, mu=_at("mu") + 4) == 3
