"""The gated recurrence's 64-bit formulas against central differences, and the refusals of its
entry points (host-side: nothing is launched)."""
import ctypes

import numpy as np
import pytest

import op_refs
from gaussian_mixture_sequence_gb300 import build as gbuild
from gaussian_mixture_sequence_gb300 import gma


@pytest.mark.parametrize("mean", [False, True])
@pytest.mark.parametrize("lengths", [None, [5, 0]])
def test_gradient_formulas_against_differences(mean, lengths):
    rng = np.random.default_rng(3)
    B, H, N, D = 2, 1, 5, 3
    x, g, w = (rng.standard_normal((B, H, N, D)) for _ in range(3))
    h0, ws = rng.standard_normal((B, H, D)), rng.standard_normal((B, H, D))

    def loss(x, g, h0):
        out, st, _, _ = op_refs.scan(x, g, mean, lengths, h0)
        return np.nansum(out * w) + (st * ws).sum()

    out = np.nan_to_num(op_refs.scan(x, g, mean, lengths, h0)[0])
    got = op_refs.scan_grad(x, g, out, w, mean, lengths, h0, ws)
    for name, arr, k in (("dx", x, 0), ("dgate", g, 1), ("dstate_in", h0, 2)):
        num = np.zeros_like(arr)
        for i in np.ndindex(arr.shape):
            args = [x.copy(), g.copy(), h0.copy()]
            args[k][i] += 1e-5
            up = loss(*args)
            args[k][i] -= 2e-5
            num[i] = (up - loss(*args)) / 2e-5
        # central differences at step 1e-5: truncation and rounding both below 1e-8 here
        assert np.abs(num - got[name][0]).max() < 1e-8, name


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gma.load()


BASE = 1 << 30
STEP = 1 << 26   # the fake buffers do not overlap


def _bufs(names):
    return {n: BASE + i * STEP for i, n in enumerate(names)}


FWD = ("x", "gate", "lengths", "state_in", "state_out", "out")
BWD = ("x", "gate", "out", "dout", "lengths", "state_in", "dstate_out", "dx", "dgate", "dstate_in")
ONE = ("x", "gate", "state", "out")


def _call(fn, names, shape, **kw):
    p = {**_bufs(names), **kw}
    return fn(ctypes.byref(shape) if shape is not None else None, *(p[n] for n in names), None)


def _entries(lib):
    return ((lib.gma_gated_scan, FWD), (lib.gma_gated_scan_backward, BWD), (lib.gma_gated_step, ONE))


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(H=0), 1), (dict(D=0), 1), (dict(D=65537), 2), (dict(B=300, H=300), 2),
])
def test_rejects_bad_shapes(lib, kw, status):
    s = gma.ScanShape.make(**{**dict(B=2, H=3, N=100, D=64), **kw})
    for fn, names in _entries(lib):
        assert _call(fn, names, s) == status


def test_rejects_bad_lengths_and_enums(lib):
    for fn, names in _entries(lib)[:2]:
        assert _call(fn, names, gma.ScanShape.make(2, 3, -1, 64)) == 1
        assert _call(fn, names, gma.ScanShape.make(2000, 32, 1 << 20, 64)) == 2
    for field in ("form", "dtype"):
        s = gma.ScanShape.make(2, 3, 100, 64)
        setattr(s, field, 2)
        for fn, names in _entries(lib):
            assert _call(fn, names, s) == 1
    for fn, names in _entries(lib):
        assert _call(fn, names, None) == 1


def test_rejects_null_misaligned_and_overlapping_buffers(lib):
    s = gma.ScanShape.make(2, 3, 100, 64, form="mean")
    optional = {"lengths", "state_in", "state_out", "dstate_out", "dstate_in"}
    for fn, names in _entries(lib):
        b = _bufs(names)
        for n in names:
            if n not in optional:
                assert _call(fn, names, s, **{n: None}) == 1, n
            assert _call(fn, names, s, **{n: b[n] + 4}) == 3, n
        if names is not BWD:
            assert _call(fn, names, s, out=b["x"]) == 1
    b = _bufs(FWD)
    assert _call(lib.gma_gated_scan, FWD, s, state_out=b["out"] + 64) == 1
    assert _call(lib.gma_gated_scan, FWD, s, state_out=b["state_in"] + 16) == 1   # overlaps without being it
    b = _bufs(BWD)
    assert _call(lib.gma_gated_scan_backward, BWD, s, dx=b["dout"]) == 1
    assert _call(lib.gma_gated_scan_backward, BWD, s, dgate=b["out"] + 16 * 100) == 1
    assert _call(lib.gma_gated_scan_backward, BWD, s, dstate_in=b["state_in"]) == 1


def test_empty_sequences_without_states_do_nothing(lib):
    s = gma.ScanShape.make(2, 3, 0, 64)
    assert _call(lib.gma_gated_scan, FWD, s, **{n: None for n in FWD}) == 0
    assert _call(lib.gma_gated_scan_backward, BWD, s, **{n: None for n in BWD}) == 0


def test_binding_refuses_wrong_tensors():
    import torch
    s = gma.ScanShape.make(1, 1, 8, 16)
    x = torch.zeros(1, 1, 8, 16)
    for call in (lambda: gma.gma_gated_scan(s, x, x, x), lambda: gma.gma_gated_step(s, x, x, x, x),
                 lambda: gma.gma_gated_scan_backward(s, None, x, x, x, x, x)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()
    with pytest.raises(KeyError):
        gma.ScanShape.make(1, 1, 8, 16, form="product")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 64])
def test_rejects_sequences_whose_positions_would_pass_31_bits(lib, D, dtype):
    for fn, names in _entries(lib)[:2]:
        for N in ((1 << 30) + 1, (1 << 31) - 20000, (1 << 31) - 1):
            assert _call(fn, names, gma.ScanShape.make(1, 1, N, D, dtype=dtype)) == 2
        # 2^30 itself passes the shape's checks (the first pointer's alignment is what fails)
        assert _call(fn, names, gma.ScanShape.make(1, 1, 1 << 30, 1, dtype=dtype), x=BASE + 4) == 3
    one = gma.ScanShape.make(1, 1, (1 << 31) - 1, D, dtype=dtype)   # (not looked at by the step)
    assert _call(lib.gma_gated_step, ONE, one, x=BASE + 4) == 3
