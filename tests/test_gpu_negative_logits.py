"""Rows whose logits are all far below 0 (keys that point away from the queries): the
softmax does not depend on where they lie, and no weight may vanish.

With q of a + 0.1 n and k of -a + 0.1 n (n normal), a^2 d = `depth`, all logits are
about -depth.  Tolerances: S errs by d 2^-23 of sum |q k| in fp32, so a weight by
err = (d 2^-23 + 2^-21) (1 + L) with L the largest sum |q k| of the row, LSE by that
and 2^-22 |LSE|; weights that multiply V are rounded to the type (u) and normalised
by their own sum (u), O is rounded once (u |O|); n 2^-24 for sums of n.  fp16
weights and results below the normal range: half a step of 2^-24."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from io_aware_exact_12_gb300 import build as b
    b.build()
    import io_aware_exact_12_gb300 as p
    p.lib()
    return p


def _inputs(B, H, N, d, depth, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn((B, H, N, d), generator=g) for _ in range(3))
    a = math.sqrt(depth / d)
    return [x.to(dtype).cuda() for x in (q * 0.1 + a, k * 0.1 - a, v)]


def _reference(q, k, v, seen):
    q, k, v = q.double(), k.double(), v.double()
    s = (q @ k.mT).masked_fill(~seen, -math.inf)
    assert s.amax() < -5
    big = (q.abs() @ k.abs().mT).masked_fill(~seen, 0).amax(-1, keepdim=True)
    err = (q.shape[-1] * 2.0 ** -23 + 2.0 ** -21) * (1 + big)
    w = torch.softmax(s, -1)
    return w @ v, torch.logsumexp(s, -1), err, w, v


def _check(o, lse, ref, seen, u):
    ro, rl, err, w, v = ref
    assert torch.isfinite(lse).all() and torch.isfinite(o.float()).all()
    assert ((lse.double() - rl).abs() <= err[..., 0] + 2.0 ** -22 * rl.abs()).all()
    if u is None:
        return
    n = seen.sum(-1).max().item() * 2.0 ** -24
    step = 2.0 ** -25 if u == 2.0 ** -11 else 0.0
    tol = u * ro.abs() + ((2 * u + 2 * err + n) * w + step * seen) @ v.abs() + step
    e = (o.double() - ro).abs()
    assert (e <= tol).all(), "off by %g of its tolerance" % (e / tol).max()


@pytest.mark.parametrize("depth", [12.0, 40.0, 150.0, 1000.0])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("N,causal", [(1, False), (100, False), (128, True), (300, False), (300, True), (1030, True)])
def test_dense_forwards(pkg, N, causal, d, dtype, depth):
    q, k, v = _inputs(2, 2, N, d, depth, dtype, N + d)
    seen = torch.ones((N, N), dtype=torch.bool, device="cuda")
    seen = seen.tril() if causal else seen
    ref, u, nb = _reference(q, k, v, seen), torch.finfo(dtype).eps / 2, -(-N // 128)
    mask = torch.ones((1, nb, nb), dtype=torch.uint8, device="cuda")
    _check(*pkg.attn_fwd(q, k, v, scale=1.0, causal=causal), ref, seen, u)
    _check(*pkg.attn_fwd_blocksparse(q, k, v, mask, scale=1.0, causal=causal), ref, seen, u)
    # dropped weights: LSE is of all of them, and O is no larger than the kept ones can make it
    for o, lse in (pkg.attn_fwd_dropout(q, k, v, 0.25, 5, scale=1.0, causal=causal), pkg.attn_fwd_blocksparse_dropout(q, k, v, mask, 0.25, 5, scale=1.0, causal=causal)):
        _check(o, lse, ref, seen, None)
        assert (o.double().abs() <= 1.02 / 0.75 * v.double().abs().amax()).all()
        assert N < 100 or o.double().abs().amax() > 0.01
    if causal:
        _check(*pkg.attn_fwd_window(q, k, v, N, scale=1.0), ref, seen, u)
    assert pkg.sync_status() == 0


@pytest.mark.parametrize("depth", [40.0, 150.0])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_the_gradients_of_such_rows(pkg, dtype, depth):
    """Through attention(): finite, and dV's columns add up to dO's, as each row's weights add up to 1."""
    q, k, v = (x.requires_grad_() for x in _inputs(1, 2, 400, 64, depth, dtype, 3))
    do = torch.randn(q.shape, generator=torch.Generator().manual_seed(4)).to(dtype).cuda()
    pkg.attention(q, k, v, scale=1.0, causal=True).backward(do)
    assert all(torch.isfinite(x.grad).all() for x in (q, k, v))
    u = torch.finfo(dtype).eps / 2
    err = 2 * (64 * 2.0 ** -23 + 2.0 ** -21) * (1 + 1.5 * depth)
    total, want = v.grad.double().sum(2), do.double().sum(2)
    tol = u * v.grad.double().abs().sum(2) + (u + err + 400 * 2.0 ** -24) * do.double().abs().sum(2) + 400 * (400 * 2.0 ** -25 if dtype == F16 else 0)
    assert ((total - want).abs() <= tol).all()
    assert pkg.sync_status() == 0


@pytest.mark.parametrize("depth", [12.0, 40.0, 150.0])
@pytest.mark.parametrize("N,causal", [(100, False), (128, True), (300, False), (1030, True)])
def test_fp8_forward(pkg, N, causal, depth, d=128):
    """Weights rounded to e4m3 with at most 2^-4, normalised by their sum: 0.134 of sum P |V - O|, and 2^-9 of the largest weight for those below its normal range."""
    q, k, v = _inputs(1, 2, N, d, depth, torch.float8_e4m3fn, N + d)
    seen = torch.ones((N, N), dtype=torch.bool, device="cuda")
    seen = seen.tril() if causal else seen
    o, lse = pkg.attn_fwd_fp8(q, k, v, 1.0, 1.0, 1.0, scale=1.0, causal=causal)
    assert pkg.sync_status() == 0
    ro, rl, err, w, vv = ref = _reference(q.float(), k.float(), v.float(), seen)
    _check(o, lse, ref, seen, None)
    spread = (w[..., None] * (vv[:, :, None] - ro[:, :, :, None]).abs()).sum(3) if N <= 300 else 2 * (w @ vv.abs())
    low = (2.0 ** -9 * w.amax(-1, keepdim=True) * seen) @ vv.abs()
    assert ((o.double() - ro).abs() <= (0.134 + 2 * err) * spread + 2.0 ** -8 * ro.abs() + low + 2e-3).all()


@pytest.mark.parametrize("depth", [12.0, 150.0])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_decode(pkg, d, depth):
    q, k, v = _inputs(2, 2, 1000, d, depth, BF16, d)
    seen = torch.ones((1, 1000), dtype=torch.bool, device="cuda")
    ref = _reference(q[:, :, -1:], k, v, seen)
    o, lse = pkg.attn_decode(q[:, :, -1].contiguous(), k, v, scale=1.0)
    _check(o[:, :, None], lse[:, :, None], ref, seen, 2.0 ** -8)
    assert pkg.sync_status() == 0
