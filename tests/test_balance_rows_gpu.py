"""The balance loss and its gradients where every warp takes several rows and every CTA several batches of
rows, as in training: steps of the walk over whole and over many short sequences, the rows fetched ahead, the
two buffers of the parameter sums.

The reference is op_refs.balance and op_refs.balance_grad, many rows at a time on tensors of 64 bits (held against
the row-by-row form below, on the host), with the same bounds."""
import numpy as np
import pytest
import torch

import op_refs
from gaussian_mixture_sequence_gb300 import gma

DEV = "cuda:0"
EPS = op_refs.EPS
NAMES = ("dx", "dmu", "dvar_raw", "dlogit_pi")


def _f64(*t):
    return tuple(v.double() for v in t)


def _rows(n, N, device):
    """Of one head: which of the [B, N] rows take part."""
    return torch.arange(N, device=device) < torch.tensor([int(v) for v in n], device=device).view(-1, 1)


def _spans(rows, K, D):
    step = max(1, (1 << 24) // (K * D))
    return [slice(i, min(rows, i + step)) for i in range(0, rows, step)]


def _posteriors(x, mu, r, lp, n):
    """gamma [B,H,N,K], counts [H,K]."""
    x, mu, r, lp = _f64(x, mu, r, lp)
    B, H, N, _ = x.shape
    K = mu.shape[1]
    gamma = torch.zeros(B, H, N, K, dtype=torch.float64, device=x.device)
    counts = torch.zeros(H, K, dtype=torch.int64, device=x.device)
    var = torch.logaddexp(r, torch.zeros_like(r))
    live = _rows(n, N, x.device)
    for h in range(H):
        xs = x[:, h][live]
        p = torch.zeros(len(xs), K, dtype=torch.float64, device=x.device)
        for at in _spans(len(xs), K, x.shape[3]):
            z = xs[at, None] - mu[h]
            ell = lp[h] - 0.5 * (z * z / var[h] + var[h].log()).sum(2)
            p[at] = torch.softmax(ell, 1)
            counts[h] += torch.bincount(ell.argmax(1), minlength=K)
        gamma[:, h][live] = p
    return gamma, counts


def _gradients(x, mu, r, lp, gamma, counts, dl, n):
    """{name: (value, bound)} of op_refs.balance_grad."""
    x, mu, r, lp, gamma, dl, cnt = _f64(x, mu, r, lp, gamma, dl, counts)
    B, H, N, D = x.shape
    K, T = mu.shape[1], max(1, int(sum(n)))
    a = 1.0 / torch.logaddexp(r, torch.zeros_like(r))
    many = (N * B + 64) * EPS
    dx, bx = torch.zeros_like(x), torch.zeros_like(x)
    s1, s2, e1, e2 = (torch.zeros_like(mu) for _ in range(4))
    s0, e0 = torch.zeros_like(lp), torch.zeros_like(lp)
    live = _rows(n, N, x.device)
    for h in range(H):
        g = dl[h] * K * cnt[h] / T / T
        xs, ps = x[:, h][live], gamma[:, h][live]
        o, bo = torch.zeros_like(xs), torch.zeros_like(xs)
        for at in _spans(len(xs), K, D):
            p = ps[at]
            u = g - g[p.argmax(1)].unsqueeze(1)
            d = p * (u - (p * u).sum(1, keepdim=True))
            ed = 40 * EPS * p * (u.abs() + (p * u.abs()).sum(1, keepdim=True)) + EPS * d.abs().amax(1, keepdim=True)
            y = xs[at, None] - mu[h]
            w = d.unsqueeze(2) * y
            ew = (ed + 16 * EPS * d.abs()).unsqueeze(2) * y.abs()
            o[at] = -(w * a[h]).sum(1)
            bo[at] = ((ew + (K + 8) * EPS * w.abs()) * a[h]).sum(1)
            e = ew + many * w.abs()
            s1[h] += w.sum(0)
            s2[h] += (w * y).sum(0)
            s0[h] += d.sum(0)
            e1[h] += e.sum(0)
            e2[h] += (e * y.abs()).sum(0)
            e0[h] += (ed + many * d.abs()).sum(0)
        dx[:, h][live], bx[:, h][live] = o, bo
    sig, t0 = torch.sigmoid(r), s0.unsqueeze(2)
    pi = torch.softmax(lp, 1)
    return {"dx": (dx, bx), "dmu": (a * s1, a * (e1 + 16 * EPS * s1.abs())),
            "dvar_raw": (0.5 * a * (a * s2 - t0) * sig,
                         0.5 * a * sig * (a * (e2 + 32 * EPS * s2.abs()) + e0.unsqueeze(2) + 16 * EPS * t0.abs())),
            "dlogit_pi": (s0 - pi * s0.sum(1, keepdim=True),
                          e0 + pi * (e0.sum(1, keepdim=True) + (K + 16) * EPS * s0.abs().sum(1, keepdim=True)))}


@pytest.mark.parametrize("lengths", [None, [9, 0, 5]])
def test_the_reference_is_the_row_by_row_one(lengths):
    g = torch.Generator().manual_seed(1)
    mk = lambda *s: torch.randn(*s, generator=g)
    B, H, N, D, K = 3, 2, 9, 16, 5
    x, mu, r, lp, dl = mk(B, H, N, D), mk(H, K, D), mk(H, K, D), mk(H, K), mk(H)
    n = op_refs.lengths_of(lengths, B, N)
    gamma, counts = _posteriors(x, mu, r, lp, n)
    host = [v.double().numpy() for v in (x, mu, r, lp)]
    wg, _, wc, _ = op_refs.balance(*host, lengths)
    assert np.array_equal(counts.numpy(), wc) and np.abs(gamma.numpy() - wg).max() < 1e-14
    want = op_refs.balance_grad(*host, wg, wc, dl.double().numpy(), lengths)
    got = _gradients(x, mu, r, lp, gamma, counts, dl, n)
    for name in NAMES:
        for p, q in zip(got[name], want[name]):
            assert np.abs(p.numpy() - q).max() <= 1e-12 * np.abs(q).max(), name


def _inputs(B, H, N, D, K, dtype, kind, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    mk = lambda *s: torch.randn(*s, device=DEV, generator=g)
    mu, r, lp, x = mk(H, K, D), 0.5 * mk(H, K, D), mk(H, K), mk(B, H, N, D)
    if kind == "clustered":
        c = torch.randint(0, K, (B, H, N), device=DEV, generator=g)
        x = mu[torch.arange(H, device=DEV).view(1, H, 1), c] + 0.8 * x
    elif kind == "flat":
        mu, r = 0.05 * mu, r + 3.0
    return (mu, r, lp), x.to(torch.bfloat16 if dtype == "bf16" else torch.float32), mk(H)


def _run(prm, x, dl, lengths, base=None):
    B, H, N, D = x.shape
    K = prm[0].shape[1]
    s = gma.Shape.make(B, H, N, D, 64, K, x_dtype=x.dtype)
    ln = torch.tensor([int(v) for v in lengths], dtype=torch.int32, device=DEV)
    gamma, loss, prob = torch.full((B, H, N, K), 7.0, device=DEV), torch.empty(H, device=DEV), torch.empty(H, K,
                                                                                                         device=DEV)
    counts = torch.empty(H, K, dtype=torch.int64, device=DEV)
    gma.gma_balance_loss(s, *prm, x, gamma, loss, counts, prob, lengths=ln)
    grads = [torch.full(t.shape, 7.0, device=DEV) if base is None else b.clone()
             for t, b in zip((x, *prm), base or (None,) * 4)]
    gma.gma_balance_backward(s, *prm, x, gamma, counts, dl, *grads, lengths=ln, accumulate=base is not None)
    return gamma, loss, counts, prob, *grads


# steps of the walk (rows): 1216 / H parts of 8 in the refinement, 152 / H of 32 in dx, of 64 (32) in the sums
CASES = [  # B, H, N, D, K, lengths, kind
    (3, 8, 1500, 64, 128, [1500, 0, 777], "normal"), (3, 8, 1500, 64, 128, [1, 1500, 1499], "flat"),
    (3, 8, 1500, 64, 256, [640, 1500, 33], "clustered"), (3, 8, 1500, 16, 5, [1500, 1100, 0], "normal"),
    (2, 8, 1500, 128, 300, [1500, 200], "normal"), (3, 8, 1500, 32, 40, [700, 0, 1500], "clustered"),
    (4, 40, 97, 64, 128, [97, 96, 0, 50], "normal"), (4, 40, 97, 128, 24, [97, 1, 97, 97], "flat"),
    (3, 40, 131, 64, 500, [131, 7, 100], "clustered"), (2, 152, 200, 16, 8, [200, 150], "normal"),
    (2, 200, 150, 64, 20, [149, 150], "clustered"),
    # a step passes over whole sequences
    (500, 8, 3, 64, 128, "any", "normal"), (2000, 16, 1, 32, 33, "any", "flat"), (700, 8, 7, 64, 256, "any", "clustered"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,N,D,K,lengths,kind", CASES)
def test_several_rows_a_warp_and_batches_a_cta(B, H, N, D, K, lengths, kind, dtype):
    prm, x, dl = _inputs(B, H, N, D, K, dtype, kind, 300 + N + K)
    n = np.random.default_rng(7).integers(0, N + 1, B) if lengths == "any" else lengths
    first = _run(prm, x, dl, n)
    gamma, loss, counts, prob, *grads = first
    wg, wc = _posteriors(x, *prm, n)
    assert torch.equal(counts, wc)
    assert ((gamma.double() - wg).abs() <= 24 * EPS * wg + 2.0 ** -23).all()
    behind = ~_rows(n, N, x.device).view(B, 1, N).expand(B, H, N)
    assert (gamma[behind] == 0).all() and (grads[0][behind] == 0).all()
    T = int(sum(n))
    wp = wg.sum((0, 2)) / T
    # (a warp's fp32 sums of its rows, at most a unit a row)
    assert ((prob.double() - wp).abs() <= (48 + B * N / 8) * EPS * wp + 2.0 ** -23).all()
    wl = K * (wc / T * wp).sum(1)
    assert ((loss.double() - wl).abs() <= (50 + B * N / 8) * EPS * wl + K * 2.0 ** -23).all()
    ref = _gradients(x, *prm, gamma, counts, dl, n)
    full = _gradients(x, *prm, wg, wc, dl, n)
    for name, got in zip(NAMES, grads):
        want, bound = ref[name]
        off = (got.double() - want).abs() - bound - 1e-37
        assert (off <= 0).all(), (name, off.max().item())
        want = full[name][0]
        if want.norm() > 1e-3 * dl.abs().max() / T:   # (as in test_balance_gpu: 24 units each, joined by differences)
            rel = ((got.double() - want).norm() / want.norm()).item()
            print(f"{name}: {rel:.2e} of the norm off the 64-bit gradient")
            assert rel <= 2e-5, (name, rel)
    again = _run(prm, x, dl, n)
    assert all(torch.equal(p, q) for p, q in zip(first, again))
    g = torch.Generator(device=DEV).manual_seed(8)
    base = [torch.randn(t.shape, device=DEV, generator=g) for t in grads]
    for b, p, q in zip(base, grads, _run(prm, x, dl, n, base)[4:]):
        assert torch.equal(q, b + p)
