"""Sliding-window attention on fp16 tensors where weights or gradients are far from
1: fp16 has a narrow range, normal from 2^-14 to 2^16, and what the kernels round to
it for a product is brought into it by powers of two.

Tolerances as in test_gpu_window.py, but for the relative error of a weight, which
is taken for the head size: err = (d 2^-23 + 2^-21) (1 + L).  What falls below
fp16's normal range is rounded to steps of 2^-24, so by 2^-25 of
  the weights of O, which are 2^7 at a row's maximum (as it was when it last moved): 2^-32;
  P in dV's product, 2^14 P: 2^-39;
  dS, whose power of two is the largest with 2 |dO| |v| 2^e <= 2^14, with the largest
    norms of a row of dO (dQ: of that row) and of v; within a factor of 4 for whole
    exponents: 2^-25 2 |dO| |v| 4 / 2^14 = 2^-36 |dO| |v|.
Nothing else is added for the types' range but half a step of the fp16 results, 2^-25."""
import math

import pytest
import torch

import test_gpu_window as base
from test_gpu_window import F16, _backward, _forward, _logits, _near, _seen

pytestmark = pytest.mark.gpu
pkg = base.pkg
U = torch.finfo(F16).eps / 2
STEP = 2.0 ** -25


def _err(q, k, seen, scale):
    """Relative error of a weight, by rows."""
    rep = k.repeat_interleave(q.shape[1] // k.shape[1], 1)
    big = (abs(scale) * (q.abs() @ rep.abs().mT)).masked_fill(~seen, 0).amax(-1, keepdim=True)
    return (q.shape[-1] * 2.0 ** -23 + 2.0 ** -21) * (1 + big)


def _check_forward(pkg, q, k, v, window, sinks, scale):
    o, lse = pkg.attn_fwd_window(q, k, v, window, sinks, scale=scale)
    assert pkg.sync_status() == 0
    q, k, v = q.double(), k.double(), v.double()
    ro, rl = _forward(q, k, v, window, sinks, scale)
    seen = _seen(q.shape[2], k.shape[2], window, sinks, q.device)
    err, n = _err(q, k, seen, scale), seen.sum(-1).max().item() * 2.0 ** -24
    p = torch.softmax(_logits(q, k, scale).masked_fill(~seen, -math.inf), -1)
    vv = v.abs().repeat_interleave(q.shape[1] // k.shape[1], 1)
    _near("o", o, ro, U * ro.abs() + ((2 * U + 2 * err + n) * p + 2.0 ** -32 * seen) @ vv + STEP)
    _near("lse", lse, rl, err[..., 0] + 2.0 ** -22 * rl.abs())
    return o, lse


def _check_backward(pkg, q, k, v, do, window, sinks, scale):
    o, lse = pkg.attn_fwd_window(q, k, v, window, sinks, scale=scale)
    got = pkg.attn_bwd_window(q, k, v, o, do, lse, window, sinks, scale=scale)
    assert pkg.sync_status() == 0
    q, k, v, o, do, lse = (x.double() for x in (q, k, v, o, do, lse))
    want = _backward(q, k, v, o, do, lse, window, sinks, scale)
    B, Hq, nq, d = q.shape
    hk, g = k.shape[1], q.shape[1] // k.shape[1]
    rep = lambda x: x.repeat_interleave(g, 1)  # noqa: E731
    group = lambda x: x.view(B, hk, g, *x.shape[2:]).sum(2)  # noqa: E731
    seen = _seen(nq, k.shape[2], window, sinks, q.device)
    err = _err(q, k, seen, scale)
    n_keys, n_rows = seen.sum(-1).max().item() * 2.0 ** -24, g * seen.sum(0).max().item() * 2.0 ** -24
    p = torch.where(seen, torch.exp(_logits(q, k, scale) - lse[..., None]), 0.0)
    ds = (p * (do @ rep(v).mT - (do * o).sum(-1, keepdim=True))).abs()
    mag = p * (do.abs() @ rep(v).abs().mT + (do * o).abs().sum(-1, keepdim=True))
    row = do.norm(dim=-1, keepdim=True)
    most = rep(v.norm(dim=-1).amax(-1))[..., None, None]
    low = lambda r: 2.0 ** -36 * r * most * seen  # noqa: E731
    all_rows = rep(row.view(B, hk, -1).amax(-1))[..., None, None]
    tol = (U * want[0].abs() + abs(scale) * ((U * ds + (2 * err + n_keys) * mag + low(row)) @ rep(k).abs()) + STEP,
           U * want[1].abs() + abs(scale) * group((U * ds + (2 * err + n_rows) * mag + low(all_rows)).mT @ q.abs()) + STEP,
           U * want[2].abs() + group(((U + 2 * err + n_rows) * p + 2.0 ** -39 * seen).mT @ do.abs()) + STEP)
    for name, x, w, t in zip(("dq", "dk", "dv"), got, want, tol):
        past = w.abs() - t > 65519  # rounds to infinity (one element of the large gradients: dk of 69690 at d = 32)
        assert (x[past] == w[past].sign() * math.inf).all()
        _near(name, x.masked_fill(past, 0), w.masked_fill(past, 0), t)


def _randn(seed, *shapes):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(s, generator=g) for s in shapes]


def _half(*x):
    return [t.to(F16).cuda() for t in x]


def _problem(d, seed, n=1100, B=1, Hq=4, Hk=2, nk=None):
    """Logits of order 1 from small q and k and a large scale, so that dQ and dK of a small dO are in fp16's range."""
    q, k, v, do = _randn(seed, (B, Hq, n, d), (B, Hk, nk or n, d), (B, Hk, nk or n, d), (B, Hq, n, d))
    return q / 64, k / 64, v, do, 4096 / math.sqrt(d)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("size", [1.0, 1e-2, 1e-3, 3e-5, 3e-6])
def test_small_gradients(pkg, d, size):
    """dS = P (dP - D) of P = 1 / 1000 is below fp16's range from dO of 1e-3 on."""
    q, k, v, do, scale = _problem(d, d)
    _check_backward(pkg, *_half(q, k, v, do * size), 1024, 4, scale)


@pytest.mark.parametrize("d", [32, 64, 128])
def test_large_gradients(pkg, d):
    """dS past fp16's largest value, of which dQ and dK are within it."""
    q, k, v, do = _randn(d, (2, 3, 300, d), (2, 3, 300, d), (2, 3, 300, d), (2, 3, 300, d))
    _check_backward(pkg, *_half(q, k, v * 20, do * 500 * math.sqrt(128 / d)), 100, 2, 1 / math.sqrt(d))


@pytest.mark.parametrize("d", [32, 64, 128])
def test_rows_of_very_different_size(pkg, d):
    """A row's dQ keeps its bits beside rows with gradients ten thousand times as large, another head's dK beside such heads."""
    q, k, v, do, scale = _problem(d, d + 1, n=700, B=2, nk=900)
    do *= torch.tensor([1.0, 1e-4]).repeat(350)[:, None]
    do[1, :2] *= 1e-3
    _check_backward(pkg, *_half(q, k, v, do), 400, 130, scale)


@pytest.mark.parametrize("n,nk,window", [(1, 1, 1), (1, 300, 300), (129, 129, 40), (513, 700, 200)])
def test_nothing_to_scale_by(pkg, n, nk, window):
    """Rows, heads and whole calls without a gradient, and values of zero."""
    q, k, v, do, scale = _problem(64, n, n=n, nk=nk)
    do[:, :2] = 0
    do[:, :, n // 2:] *= 1e-3
    _check_backward(pkg, *_half(q, k, v, do), window, 2, scale)
    _check_backward(pkg, *_half(q, k, v, do * 0), window, 2, scale)
    _check_backward(pkg, *_half(q, k, v * 0, do), window, 2, scale)


@pytest.mark.parametrize("heads,n,d", [(1, 5000, 64), (40, 300, 128), (700, 130, 32)])
def test_the_largest_row_anywhere(pkg, heads, n, d):
    """One row of dO or of v a million times the others', in the last head: read by one block or by one of many."""
    q, k, v, do, scale = _problem(d, heads, n=n, Hq=heads, Hk=heads)
    for at in (0, n // 2 + 3, n - 1):
        for x in (do, v):
            parts = [q, k, v * 1e-3, do * 1e-3]
            parts[3 if x is do else 2][:, -1, at] = x[:, -1, at] * 1e3
            _check_backward(pkg, *_half(*parts), 64, 0, scale)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("sinks", [0, 3, 200])
def test_hidden_keys_leave_no_trace(pkg, d, sinks):
    """Other finite values in keys that no query sees change no bit, not by the power of two either."""
    q, k, v, do, scale = _problem(d, d, n=130, nk=900)
    q, k, v, do = _half(q, k, v, do * 1e-3)
    window, hidden = 200, slice(sinks, 900 - 130 - 200 + 1)
    o, lse = pkg.attn_fwd_window(q, k, v, window, sinks, scale=scale)
    grads = pkg.attn_bwd_window(q, k, v, o, do, lse, window, sinks, scale=scale)
    k[:, :, hidden], v[:, :, hidden] = 1e4, -3e4
    again = pkg.attn_fwd_window(q, k, v, window, sinks, scale=scale)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    for x, y in zip(grads, pkg.attn_bwd_window(q, k, v, o, do, lse, window, sinks, scale=scale)):
        assert torch.equal(x, y)
    assert (grads[1][:, :, hidden] == 0).all() and (grads[2][:, :, hidden] == 0).all()
    assert pkg.sync_status() == 0


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("gap", [8.0, 13.0, 15.25, 17.5, 21.0])
@pytest.mark.parametrize("nq,nk,window,sinks", [(700, 700, 200, 1), (4, 3000, 2500, 1), (300, 300, 300, 0)])
def test_a_sink_that_holds_the_weight(pkg, d, gap, nq, nk, window, sinks):
    """A first key with nearly all of the weight and a value of zero, as models make of sinks: O is what the other keys' small weights make of it."""
    q, k, v = _randn(nq + d, (1, 4, nq, d), (1, 2, nk, d), (1, 2, nk, d))
    q, k, v = q * 0.05, k * 0.5, v * 4000
    q[..., 0], k[..., 0], k[:, :, 0] = 1.0, 0.0, 0.0
    k[:, :, 0, 0], v[:, :, 0] = gap, 0.0
    _check_forward(pkg, *_half(q, k, v.clamp(-6e4, 6e4)), window, sinks, 1.0)
