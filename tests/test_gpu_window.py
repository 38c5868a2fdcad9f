"""Sliding-window attention with sinks on the GPU, both passes, against plain
float64 forms; the same forms against differences on the CPU.

Tolerances come from the arithmetic.  u = finfo(t).eps / 2 is the most that a
rounding to type t errs by, relative to the value.
  S is an fp32 sum of d <= 128 exact products, at most 128 2^-23 (twice the bound
    for rounding, as the tensor cores truncate) of sum |q k|, and its product with
    the scale and the subtraction of the maximum or of LSE err by 2^-22 of what is
    about as large: with L = max |scale| sum |q k| over a row a weight errs by
    2^-15 (1 + L) relative, exp2 and the sums included.
  O: weights multiply V rounded to t and are normalised by the sum of the rounded
    ones, so by u on either side: 2 u sum P |v|; one rounding of the result, u |O|.
  LSE: 2^-15 (1 + L).
  dV: u sum P |dO| for the rounded weights and one rounding.
  dS = P o (dP - D) in fp32, rounded to t: u sum |dS| |k| (dK: |q|), 2^-15 (1 + L) of
    P (sum |dO v| + sum |dO o|) for its fp32 parts, one rounding.
  Sums over n rows or keys in fp32, in any order: n 2^-24 of the sum of magnitudes.
  fp16 results below the normal range: half a step of 2^-24.
The backward's reference takes the kernel's O and LSE as they are, as the call does.
"""
import math

import pytest
import torch

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


def _seen(nq, nk, window, sinks, device="cpu"):
    p = torch.arange(nq, device=device)[:, None] + nk - nq
    j = torch.arange(nk, device=device)
    return (j <= p) & ((j > p - window) | (j < sinks))


def _logits(q, k, scale):
    g = q.shape[1] // k.shape[1]
    return scale * (q @ k.repeat_interleave(g, 1).mT)


def _forward(q, k, v, window, sinks, scale):
    """O and LSE from the definition."""
    g = q.shape[1] // k.shape[1]
    s = _logits(q, k, scale).masked_fill(~_seen(q.shape[2], k.shape[2], window, sinks, q.device), -math.inf)
    return torch.softmax(s, -1) @ v.repeat_interleave(g, 1), torch.logsumexp(s, -1)


def _backward(q, k, v, o, do, lse, window, sinks, scale):
    """dQ, dK, dV from the formulas."""
    B, Hq, nq, d = q.shape
    hk, g = k.shape[1], q.shape[1] // k.shape[1]
    seen = _seen(nq, k.shape[2], window, sinks, q.device)
    p = torch.where(seen, torch.exp(_logits(q, k, scale) - lse[..., None]), 0.0)
    ds = p * (do @ v.repeat_interleave(g, 1).mT - (do * o).sum(-1, keepdim=True))
    group = lambda x: x.view(B, hk, g, *x.shape[2:]).sum(2)  # noqa: E731
    return scale * (ds @ k.repeat_interleave(g, 1)), scale * group(ds.mT @ q), group(p.mT @ do)


def _bounds(q, k, v, o, do, lse, window, sinks, scale, u):
    """Tolerances of (o, lse, dq, dk, dv) about the references of the same inputs."""
    B, Hq, nq, d = q.shape
    hk, g, nk = k.shape[1], q.shape[1] // k.shape[1], k.shape[2]
    seen = _seen(nq, nk, window, sinks, q.device)
    rep = lambda x: x.repeat_interleave(g, 1)  # noqa: E731
    group = lambda x: x.view(B, hk, g, *x.shape[2:]).sum(2)  # noqa: E731
    a = abs(scale)
    s = _logits(q, k, scale).masked_fill(~seen, -math.inf)
    big = (a * (q.abs() @ rep(k).abs().mT)).masked_fill(~seen, 0).amax(-1, keepdim=True)
    err = 2.0 ** -15 * (1 + big)
    p = torch.softmax(s, -1)
    n_keys, n_rows = seen.sum(-1).max().item() * 2.0 ** -24, g * seen.sum(0).max().item() * 2.0 ** -24
    floor = 2.0 ** -25 if u == torch.finfo(F16).eps / 2 else 0.0
    spread = p @ rep(v).abs()
    out = [u * (p @ rep(v)).abs() + (2 * u + 2 * err + n_keys) * spread + floor, err[..., 0]]
    if do is not None:
        mag = do.abs() @ rep(v).abs().mT + (do.abs() * o.abs()).sum(-1, keepdim=True)
        pp = torch.where(seen, torch.exp(s - lse[..., None]), 0.0)
        ds = (pp * (do @ rep(v).mT - (do * o).sum(-1, keepdim=True))).abs()
        part = lambda n: u * ds + (2 * err + n) * pp * mag  # noqa: E731
        dq, dk, dv = _backward(q, k, v, o, do, lse, window, sinks, scale)
        f = floor * 4
        # P, in the weights' product, is rounded to fp16 with steps of 2^-24 below its normal range
        small = (floor * seen) if floor else 0.0 * pp
        out += [u * dq.abs() + a * (part(n_keys) + small) @ rep(k).abs() + f,
                u * dk.abs() + a * group((part(n_rows) + small).mT @ q.abs()) + f,
                u * dv.abs() + group(((u + 2 * err + n_rows) * pp + small).mT @ do.abs()) + f]
    return out


def _inputs(B, Hq, Hk, nq, nk, d, dtype, layout, seed, spread=1.0):
    """q, k, v, do on the GPU: [B, H, N, d] in memory, [B, N, H, d], or slices of one projection's output."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: (torch.randn(s, generator=g) * spread).to(dtype).cuda()  # noqa: E731
    if layout == "heads":
        return r(B, Hq, nq, d), r(B, Hk, nk, d), r(B, Hk, nk, d), r(B, Hq, nq, d) / spread
    t = lambda x: x.transpose(1, 2)  # noqa: E731
    if layout == "tokens":
        return t(r(B, nq, Hq, d)), t(r(B, nk, Hk, d)), t(r(B, nk, Hk, d)), t(r(B, nq, Hq, d) / spread)
    qkv = r(B, nk, Hq + 2 * Hk, d)
    q, k, v = qkv.split([Hq, Hk, Hk], 2)
    return t(q[:, nk - nq:]), t(k), t(v), t(r(B, nq, Hq + 1, d)[:, :, 1:] / spread)


def _near(name, got, want, tol):
    assert torch.isfinite(got.float()).all(), name
    err = (got.double() - want).abs()
    worst = (err / tol.clamp_min(1e-300)).max()
    assert (err <= tol).all(), "%s off by %g of its tolerance (%g)" % (name, worst, err.max())


def _check(pkg, q, k, v, do, window, sinks, scale=None, **kw):
    scale = 1 / math.sqrt(q.shape[-1]) if scale is None else scale
    f = lambda x: x.double()  # noqa: E731
    u = torch.finfo(q.dtype).eps / 2
    o, lse = pkg.attn_fwd_window(q, k, v, window, sinks, scale=scale)
    assert pkg.sync_status() == 0
    assert pkg.last_launch_count() == 1
    ro, rl = _forward(f(q), f(k), f(v), window, sinks, scale)
    to, tl = _bounds(f(q), f(k), f(v), None, None, None, window, sinks, scale, u)
    _near("lse", lse, rl, tl)
    _near("o", o, ro, to)
    if do is None:
        return o, lse
    grads = pkg.attn_bwd_window(q, k, v, o, do, lse, window, sinks, scale=scale, **kw)
    assert pkg.sync_status() == 0
    want = _backward(f(q), f(k), f(v), f(o), f(do), f(lse), window, sinks, scale)
    tol = _bounds(f(q), f(k), f(v), f(o), f(do), f(lse), window, sinks, scale, u)[2:]
    for name, x, y, t in zip(("dq", "dk", "dv"), grads, want, tol):
        assert x.shape == y.shape
        _near(name, x, y, t)
    return (o, lse) + tuple(grads)


# ------------------------------------------------------------------ formulas

@pytest.mark.parametrize("nq,nk,window,sinks", [(5, 5, 2, 1), (4, 7, 3, 2), (6, 6, 6, 0), (1, 3, 1, 3)])
def test_the_formulas_are_the_derivative(nq, nk, window, sinks):
    """Central differences of <O, dO> in every element of q, k and v, float64; two query heads to a key/value head."""
    g = torch.Generator().manual_seed(nq)
    q, k, v, do = (torch.randn((1, h, n, 3), generator=g, dtype=torch.float64) for h, n in ((2, nq), (1, nk), (1, nk), (2, nq)))
    o, lse = _forward(q, k, v, window, sinks, 0.7)
    grads = _backward(q, k, v, o, do, lse, window, sinks, 0.7)
    for x, got in zip((q, k, v), grads):
        for i in range(x.numel()):
            was, e = x.view(-1)[i].item(), 1e-5
            ends = []
            for step in (e, -e):
                x.view(-1)[i] = was + step
                ends.append((_forward(q, k, v, window, sinks, 0.7)[0] * do).sum().item())
            x.view(-1)[i] = was
            # truncation e^2 / 6 of a third derivative of order 10, cancellation 2^-52 / e of sums of order 10
            assert abs((ends[0] - ends[1]) / (2 * e) - got.view(-1)[i].item()) <= 1e-8


# ------------------------------------------------------------------ both passes

gpu = pytest.mark.gpu

SHAPES = [
    # B, Hq, Hk, nq, nk, window, sinks
    (1, 1, 1, 1, 1, 1, 0),
    (2, 2, 1, 2, 2, 1, 0),
    (1, 2, 2, 1, 300, 40, 3),
    (1, 4, 2, 127, 127, 1, 1),
    (2, 2, 2, 128, 128, 128, 0),
    (1, 3, 1, 129, 129, 128, 1),
    (1, 2, 1, 200, 200, 7, 4),
    (1, 2, 2, 257, 600, 100, 130),
    (2, 3, 3, 383, 383, 129, 0),
    (1, 8, 1, 500, 500, 64, 64),
    (1, 2, 2, 513, 1024, 127, 256),
    (1, 4, 4, 640, 1000, 1000, 0),
    (1, 2, 1, 640, 641, 5000, 7),
    (1, 2, 2, 300, 300, 1, 1000),
    (1, 2, 2, 1030, 1030, 256, 4),
    (1, 1, 1, 2000, 2100, 300, 300),
]


@gpu
@pytest.mark.parametrize("d,dtype,layout", [(32, BF16, "tokens"), (32, F16, "heads"), (64, BF16, "heads"), (64, F16, "slices"), (128, BF16, "slices"), (128, F16, "tokens")])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_both_passes(pkg, shape, d, dtype, layout):
    B, Hq, Hk, nq, nk, window, sinks = shape
    _check(pkg, *_inputs(B, Hq, Hk, nq, nk, d, dtype, layout, nq + d), window, sinks)


@gpu
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("scale", [0.0, -0.3, 0.6])
def test_scales(pkg, d, scale):
    _check(pkg, *_inputs(1, 2, 1, 300, 300, d, F16, "heads", 1), 70, 5, scale=scale)


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_large_logits(pkg, d):
    """Logits of a hundred: the running maximum moves by more than exp2's range between tiles."""
    _check(pkg, *_inputs(1, 2, 2, 700, 700, d, BF16, "heads", 2, spread=4.0), 400, 9)


@gpu
@pytest.mark.parametrize("Hq,Hk", [(12, 1), (16, 2), (9, 3), (5, 5)])
def test_groups_of_heads(pkg, Hq, Hk):
    _check(pkg, *_inputs(2, Hq, Hk, 260, 390, 64, BF16, "slices", Hq), 90, 2)
    _check(pkg, *_inputs(1, Hq, Hk, 200, 200, 128, BF16, "tokens", Hq), 200, 0)


@gpu
@pytest.mark.parametrize("seed", range(24))
def test_drawn_shapes(pkg, seed):
    import random
    r = random.Random(seed)
    hk = r.choice([1, 2, 3])
    nk = int(2 ** r.uniform(0, 11))
    nq = nk if r.random() < 0.5 else r.randint(1, nk)
    args = (r.choice([1, 2, 3]), hk * r.choice([1, 2, 4, 5]), hk, nq, nk, r.choice([32, 64, 128]), r.choice([BF16, F16]), r.choice(["heads", "tokens", "slices"]), seed)
    _check(pkg, *_inputs(*args), int(2 ** r.uniform(0, 11)), r.choice([0, 1, 4, 127, 128, 129, 500]))


FEW = [
    # several blocks to an item: eight, four, two; items shorter than the blocks are many (the causal masks)
    (1, 8, 2, 1, 9000, 9000, 0),
    (1, 4, 4, 16, 3000, 2500, 130),
    (1, 2, 1, 130, 2500, 1100, 4),
    (2, 1, 1, 1500, 1500, 1500, 0),
    (1, 4, 1, 100, 700, 256, 4),
    (1, 64, 8, 128, 1500, 1300, 4),
    (1, 100, 4, 100, 2600, 2500, 1),
]


@gpu
@pytest.mark.parametrize("d,dtype,layout", [(32, BF16, "tokens"), (64, F16, "slices"), (128, BF16, "heads"), (128, F16, "tokens")])
@pytest.mark.parametrize("shape", FEW, ids=lambda s: "x".join(map(str, s)))
def test_few_rows_over_many_keys(pkg, shape, d, dtype, layout):
    B, Hq, Hk, nq, nk, window, sinks = shape
    q, k, v, _ = _inputs(B, Hq, Hk, nq, nk, d, dtype, layout, nk + d)
    o, lse = _check(pkg, q, k, v, None, window, sinks)
    again = pkg.attn_fwd_window(q, k, v, window, sinks)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@gpu
@pytest.mark.parametrize("d", [32, 64, 128])
def test_parts_of_very_different_weight(pkg, d):
    """Logits of a hundred, and a part that holds nearly all of a row's weight."""
    q, k, v, do = _inputs(1, 2, 1, 40, 4000, d, BF16, "tokens", 8, spread=4.0)
    _check(pkg, q, k, v, do, 3500, 9)
    k[:, :, 1000:1128] *= 2
    _check(pkg, q, k, v, None, 3500, 9, scale=-0.2)


@gpu
def test_captured_parts_replay(pkg):
    q, k, v, _ = _inputs(1, 4, 2, 8, 5000, 64, F16, "heads", 9)
    pkg.attn_fwd_window(q, k, v, 4096, 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = pkg.attn_fwd_window(q, k, v, 4096, 4)
    for seed in (10, 11):
        fresh = _inputs(1, 4, 2, 8, 5000, 64, F16, "heads", seed)
        for x, y in zip((q, k, v), fresh):
            x.copy_(y)
        graph.replay()
        want = pkg.attn_fwd_window(q, k, v, 4096, 4)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert pkg.sync_status() == 0


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_long_sequence(pkg, d):
    """Many tiles between the sinks and the window, and the sinks' gradients over all of them."""
    q, k, v, do = _inputs(1, 2, 1, 6000, 6000, d, BF16, "tokens", 3)
    _check(pkg, q, k, v, do, 500, 4)


@gpu
def test_a_window_of_all_is_the_causal_mask(pkg):
    q, k, v, do = _inputs(2, 3, 3, 700, 700, 64, F16, "heads", 4)
    o, lse = pkg.attn_fwd_window(q, k, v, 700)
    ro, rl = pkg.attn_fwd(q, k, v, causal=True)
    u = torch.finfo(F16).eps / 2
    f = lambda x: x.double()  # noqa: E731
    to, tl = _bounds(f(q), f(k), f(v), None, None, None, 700, 0, 0.125, u)
    _near("o", o, f(ro), 2 * to)
    _near("lse", lse, f(rl), 2 * tl)


@gpu
@pytest.mark.parametrize("d", [32, 64, 128])
def test_hidden_keys_leave_no_trace(pkg, d):
    """Other finite values in keys that no query sees change no bit; those keys have no gradient."""
    q, k, v, do = _inputs(1, 4, 2, 130, 900, d, BF16, "heads", 5)
    window, sinks = 200, 3
    o, lse = pkg.attn_fwd_window(q, k, v, window, sinks)
    dq, dk, dv = pkg.attn_bwd_window(q, k, v, o, do, lse, window, sinks)
    hidden = slice(sinks, 900 - 130 - window + 1)
    k2, v2 = k.clone(), v.clone()
    k2[:, :, hidden] = 1e4
    v2[:, :, hidden] = -1e4
    o2, lse2 = pkg.attn_fwd_window(q, k2, v2, window, sinks)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    dq2, dk2, dv2 = pkg.attn_bwd_window(q, k2, v2, o, do, lse, window, sinks)
    assert torch.equal(dk, dk2) and torch.equal(dv, dv2)
    assert (dk[:, :, hidden] == 0).all() and (dv[:, :, hidden] == 0).all()
    assert pkg.sync_status() == 0


@gpu
def test_what_repeats_bit_for_bit(pkg):
    """O, LSE, dK and dV; dQ's sums have no fixed order."""
    q, k, v, do = _inputs(1, 8, 2, 3000, 3000, 128, BF16, "tokens", 6)
    first = pkg.attn_fwd_window(q, k, v, 300, 4)
    grads = pkg.attn_bwd_window(q, k, v, first[0], do, first[1], 300, 4)
    for _ in range(5):
        again = pkg.attn_fwd_window(q, k, v, 300, 4)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
        more = pkg.attn_bwd_window(q, k, v, first[0], do, first[1], 300, 4)
        assert torch.equal(more[1], grads[1]) and torch.equal(more[2], grads[2])


@gpu
def test_writes_what_it_is_given(pkg):
    """Outputs as slices of wider buffers, whose other elements stay; dq, dk and dv beside one another in one buffer."""
    B, Hq, Hk, n, d = 2, 4, 2, 333, 64
    q, k, v, do = _inputs(B, Hq, Hk, n, n, d, BF16, "slices", 7)
    want = _check(pkg, q, k, v, do, 100, 4)
    wide = torch.full((B, n, Hq + 2, d), 7.0, dtype=BF16, device="cuda")
    lse = torch.zeros((B, Hq, n), device="cuda")
    o = wide[:, :, 1:1 + Hq].transpose(1, 2)
    got = pkg.attn_fwd_window(q, k, v, 100, 4, o=o, lse=lse)
    assert got[0] is o and got[1] is lse
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and (wide[:, :, 0] == 7).all() and (wide[:, :, -1] == 7).all()
    grads = torch.full((B, n, Hq + 2 * Hk, d), 7.0, dtype=BF16, device="cuda")
    dq, dk, dv = (x.transpose(1, 2) for x in grads.split([Hq, Hk, Hk], 2))
    pkg.attn_bwd_window(q, k, v, o, do, lse, 100, 4, dq=dq, dk=dk, dv=dv)
    assert torch.equal(dk, want[3]) and torch.equal(dv, want[4])
    tol = _bounds(*(x.double() for x in (q, k, v, o, do, lse)), 100, 4, 0.125, torch.finfo(BF16).eps / 2)[2]
    _near("dq", dq, want[2].double(), 2 * tol)
    assert pkg.sync_status() == 0


@gpu
def test_outputs_follow_the_inputs_order(pkg):
    q, k, v, do = _inputs(1, 4, 2, 50, 60, 64, BF16, "tokens", 8)
    o, lse = pkg.attn_fwd_window(q, k, v, 10)
    assert o.transpose(1, 2).is_contiguous()
    dq, dk, dv = pkg.attn_bwd_window(q, k, v, o, do, lse, 10)
    assert dq.transpose(1, 2).is_contiguous() and dk.transpose(1, 2).is_contiguous()
    q, k, v, do = _inputs(1, 4, 2, 50, 60, 64, BF16, "heads", 8)
    assert pkg.attn_fwd_window(q, k, v, 10)[0].is_contiguous()


@gpu
def test_autograd(pkg):
    """attention(..., window=...) with shared heads, an expanded gradient, and inputs whose strides the call does not take."""
    q, k, v, do = _inputs(2, 4, 2, 200, 200, 64, F16, "tokens", 9)
    odd = torch.zeros((2, 4, 200, 65), dtype=F16, device="cuda")[..., 1:]
    odd.copy_(q)
    leaves = [x.detach().clone().requires_grad_() for x in (q, k, v)]
    o = pkg.attention(*leaves, window=50, sinks=3)
    o.backward(do)
    want = _check(pkg, q, k, v, do, 50, 3)
    tol = _bounds(*(x.double() for x in (q, k, v, want[0], do, want[1])), 50, 3, 0.125, torch.finfo(F16).eps / 2)[2:]
    for leaf, w, t in zip(leaves, want[2:], tol):
        _near("grad", leaf.grad, w.double(), 2 * t)
    x = odd.detach().requires_grad_()
    o2 = pkg.attention(x, k, v, window=50, sinks=3)
    assert torch.equal(o2, o)
    o2.sum().backward()
    ones = torch.ones_like(o)
    f = [t.double() for t in (q, k, v, want[0], ones, want[1])]
    _near("grad", x.grad, _backward(*f, 50, 3, 0.125)[0], _bounds(*f, 50, 3, 0.125, torch.finfo(F16).eps / 2)[2])
    # one key/value head, broadcast to all queries' heads
    one = k[:, :1].detach().clone().requires_grad_()
    pkg.attention(q, one.expand(2, 4, 200, 64), v.repeat_interleave(2, 1), window=50).backward(do)
    shared = k[:, :1].detach().clone().requires_grad_()
    pkg.attention(q, shared, v[:, :1], window=50)
    assert one.grad.shape == (2, 1, 200, 64) and torch.isfinite(one.grad).all()
    with pytest.raises(ValueError):
        pkg.attention(q, k, v, window=50, dropout_p=0.1)
    with pytest.raises(ValueError):
        pkg.attention(q, k, v, sinks=2)


@gpu
def test_captured_step_replays(pkg):
    q, k, v, do = _inputs(1, 4, 2, 700, 700, 128, BF16, "tokens", 10)
    want = _check(pkg, q, k, v, do, 300, 4)
    bufs = [torch.zeros_like(x) for x in (q, k, v, do)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # first calls of a kernel are not made in a capture
        o, lse = pkg.attn_fwd_window(*bufs[:3], 300, 4)
        pkg.attn_bwd_window(*bufs[:3], o, bufs[3], lse, 300, 4)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = pkg.attn_fwd_window(*bufs[:3], 300, 4)
        dq, dk, dv = pkg.attn_bwd_window(*bufs[:3], o, bufs[3], lse, 300, 4)
    for to, x in zip(bufs, (q, k, v, do)):
        to.copy_(x)
    for _ in range(3):
        graph.replay()
    assert pkg.sync_status() == 0
    for got, w in zip((o, lse, dk, dv), want[:2] + want[3:]):
        assert torch.equal(got, w)
    tol = _bounds(*(x.double() for x in (q, k, v, want[0], do, want[1])), 300, 4, 128 ** -0.5, torch.finfo(BF16).eps / 2)[2]
    _near("dq", dq, want[2].double(), 2 * tol)


@gpu
def test_two_graphs_of_one_pool(pkg):
    """Two captured steps that share a memory pool, their workspaces among it, replayed in turns."""
    sets = [_inputs(1, 4, 2, n, n, 64, BF16, "tokens", n) for n in (500, 900)]
    want = [_check(pkg, *x, 200, 4) for x in sets]
    pool, graphs, outs = torch.cuda.graph_pool_handle(), [], []
    for q, k, v, do in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            o, lse = pkg.attn_fwd_window(q, k, v, 200, 4)
            outs.append((o, lse) + pkg.attn_bwd_window(q, k, v, o, do, lse, 200, 4))
        graphs.append(graph)
    for i in (0, 1, 1, 0, 1):
        graphs[i].replay()
        got = [x.clone() for x in outs[i]]
        torch.cuda.synchronize()
        for x, w in zip(got, want[i]):
            assert torch.equal(x, w)
    assert pkg.sync_status() == 0


@gpu
def test_a_padded_batch(pkg):
    """Sequences padded at their end: what stands there changes nothing before it, and without a gradient adds none."""
    q, k, v, do = _inputs(2, 4, 2, 300, 300, 64, F16, "tokens", 15)
    real = 211
    do[1, :, real:] = 0
    a = pkg.attn_fwd_window(q, k, v, 70, 3)
    ga = pkg.attn_bwd_window(q, k, v, a[0], do, a[1], 70, 3)
    q2, k2, v2 = q.clone(), k.clone(), v.clone()
    for x in (q2, k2, v2):
        x[1, :, real:] = 55.0
    b = pkg.attn_fwd_window(q2, k2, v2, 70, 3)
    gb = pkg.attn_bwd_window(q2, k2, v2, b[0], do, b[1], 70, 3)
    assert torch.equal(a[0][1, :, :real], b[0][1, :, :real]) and torch.equal(a[1][1, :, :real], b[1][1, :, :real])
    for x, y in zip(ga, gb):
        assert torch.equal(x[1, :, :real], y[1, :, :real]) and torch.equal(x[0], y[0])
        assert (x[1, :, real:] == 0).all() and (y[1, :, real:] == 0).all()


@gpu
def test_past_32_bit_offsets(pkg):
    """Tensors of more than 2^31 elements; the last head's last rows and keys, and the sinks' gradients of a short run of rows."""
    B, Hq, Hk, n, d, window, sinks = 1, 72, 2, 262144, 128, 100, 4
    g = torch.Generator(device="cuda").manual_seed(16)
    r = lambda h: torch.randn((B, n, h, d), generator=g, device="cuda", dtype=BF16).transpose(1, 2)  # noqa: E731
    q, k, v, do = r(Hq), r(Hk), r(Hk), r(Hq)
    assert q.numel() > 2 ** 31
    do[:, :, :-600] = 0  # gradients of the last rows only, so that a float64 form of them is small
    o, lse = pkg.attn_fwd_window(q, k, v, window, sinks)
    dq, dk, dv = pkg.attn_bwd_window(q, k, v, o, do, lse, window, sinks)
    assert pkg.sync_status() == 0
    h, G, first = Hq - 1, Hq // Hk, n - 600
    keys = torch.cat([torch.arange(sinks), torch.arange(first - window, n)]).cuda()  # all that the last rows see
    rows = slice(first, n)
    f = lambda x: x.double()  # noqa: E731
    group = slice(Hq - G, Hq)
    kk, vv, qq, oo, dd, ll = f(k[:, 1:, keys]), f(v[:, 1:, keys]), f(q[:, group, rows]), f(o[:, group, rows]), f(do[:, group, rows]), f(lse[:, group, rows])
    # as a problem of its own: keys 0 .. are the sinks and those before the rows, in their order; the mask of positions is the same
    u, scale = torch.finfo(BF16).eps / 2, d ** -0.5
    pos = torch.arange(first, n, device="cuda")[:, None]
    seen = (keys <= pos) & ((keys > pos - window) | (keys < sinks))
    s = (scale * (qq @ kk.mT)).masked_fill(~seen, -math.inf)
    p = torch.softmax(s, -1)
    big = (scale * (qq.abs() @ kk.abs().mT)).masked_fill(~seen, 0).amax(-1, keepdim=True)
    err = 2.0 ** -15 * (1 + big)
    _near("o", o[:, group, rows], p @ vv, u * (p @ vv).abs() + (2 * u + 2 * err) * (p @ vv.abs()))
    _near("lse", lse[:, group, rows], torch.logsumexp(s, -1), err[..., 0])
    pp = torch.where(seen, torch.exp(s - ll[..., None]), 0.0)
    ds = pp * (dd @ vv.mT - (dd * oo).sum(-1, keepdim=True))
    mag = pp * (dd.abs() @ vv.abs().mT + (dd.abs() * oo.abs()).sum(-1, keepdim=True))
    n_rows = G * 600 * 2.0 ** -24
    want = scale * (ds @ kk)
    _near("dq", dq[:, group, rows], want, u * want.abs() + scale * ((u * ds.abs() + 2 * err * mag) @ kk.abs()))
    want = scale * (ds.mT @ qq).sum(1)
    _near("dk", dk[:, 1, keys], want, u * want.abs() + scale * ((u * ds.abs() + (2 * err + n_rows) * mag).mT @ qq.abs()).sum(1))
    want = (pp.mT @ dd).sum(1)
    _near("dv", dv[:, 1, keys], want, u * want.abs() + (((u + 2 * err + n_rows) * pp).mT @ dd.abs()).sum(1))
    assert (dq[:, :, :first] == 0).all()
    assert (dk[:, :, sinks:first - window - 128] == 0).all() and (dv[:, :, sinks:first - window - 128] == 0).all()


@gpu
def test_two_streams_at_once(pkg):
    sets = [_inputs(1, 4, 2, 900, 900, 64, BF16, "tokens", s) for s in (11, 12)]
    want = [_check(pkg, *x, 200, 4) for x in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for x, s in zip(sets, streams):
        o, lse = pkg.attn_fwd_window(*x[:3], 200, 4, stream=s)
        got.append((o, lse) + pkg.attn_bwd_window(*x[:3], o, x[3], lse, 200, 4, stream=s))
    torch.cuda.synchronize()
    assert pkg.sync_status() == 0
    for g, w in zip(got, want):
        for i in (0, 1, 3, 4):
            assert torch.equal(g[i], w[i])


@gpu
def test_first_call_of_a_thread(pkg):
    """A thread that has made no CUDA call yet has no current context."""
    import threading
    q, k, v, do = _inputs(1, 4, 2, 300, 300, 64, BF16, "tokens", 14)
    want = _check(pkg, q, k, v, do, 100, 4)
    outs = [torch.empty_like(x) for x in want]
    dense = [do.contiguous() for _ in range(4)]
    row = torch.empty_like(want[1])
    torch.cuda.synchronize()
    failed = []

    def work(call):
        try:
            call()
        except Exception as e:
            failed.append(e)

    for call in (lambda: pkg.attn_fwd_window(q, k, v, 100, 4, o=outs[0], lse=outs[1]),
                 lambda: pkg.attn_bwd_window(q, k, v, want[0], do, want[1], 100, 4, dq=outs[2], dk=outs[3], dv=outs[4]),
                 lambda: pkg.attn_fwd(*dense[:3], o=dense[3], lse=row)):
        t = threading.Thread(target=work, args=(call,))
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    assert pkg.sync_status() == 0
    for i in (0, 1, 3, 4):
        assert torch.equal(outs[i], want[i])


@gpu
def test_the_binding_refuses(pkg):
    q, k, v, do = _inputs(1, 4, 2, 50, 60, 64, BF16, "tokens", 13)
    o, lse = pkg.attn_fwd_window(q, k, v, 10)
    bad = [
        (ValueError, lambda: pkg.attn_fwd_window(q, k, v, 0)),
        (ValueError, lambda: pkg.attn_fwd_window(q, k, v, 10, -1)),
        (TypeError, lambda: pkg.attn_fwd_window(q, k, v, 1.5)),
        (ValueError, lambda: pkg.attn_fwd_window(k, q, q, 10)),                       # heads do not divide
        (ValueError, lambda: pkg.attn_fwd_window(q, k[:, :, :40], v[:, :, :40], 10)),  # fewer keys than queries
        (ValueError, lambda: pkg.attn_fwd_window(q, k, v[:, :, :40], 10)),
        (TypeError, lambda: pkg.attn_fwd_window(q, k.half(), v, 10)),
        (TypeError, lambda: pkg.attn_fwd_window(q.float(), k, v, 10)),
        (TypeError, lambda: pkg.attn_fwd_window(q.cpu(), k, v, 10)),
        (ValueError, lambda: pkg.attn_fwd_window(q[0], k, v, 10)),
        (ValueError, lambda: pkg.attn_fwd_window(q.transpose(2, 3), k, v, 10)),
        (ValueError, lambda: pkg.attn_fwd_window(q, k, v, 10, o=o[:, :, :3])),
        (ValueError, lambda: pkg.attn_fwd_window(q, k, v, 10, lse=lse.half())),
        (ValueError, lambda: pkg.attn_bwd_window(q, k, v, o[:, :, :3], do, lse, 10)),
        (ValueError, lambda: pkg.attn_bwd_window(q, k, v, o, do, lse[:, :3], 10)),
        (pkg.AttnError, lambda: pkg.attn_fwd_window(q, k, v, 10, scale=math.nan)),
        (pkg.AttnError, lambda: pkg.attn_fwd_window(q, k, v, 10, o=q)),
        (pkg.AttnError, lambda: pkg.attn_fwd_window(q, k[:1].expand(1, 2, 60, 64)[:, :1].expand(1, 2, 60, 64), v, 10)),
        (pkg.AttnError, lambda: pkg.attn_bwd_window(q, k, v, o, do, lse, 10, dq=do)),
        (pkg.AttnError, lambda: pkg.attn_fwd_window(q[..., :48], k[..., :48], v[..., :48], 10)),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()
    assert pkg.sync_status() == 0
    # a window or a number of sinks past any length is one of all keys
    a = pkg.attn_fwd_window(q, k, v, 1 << 70, 1 << 70)
    assert torch.equal(a[0], pkg.attn_fwd_window(q, k, v, 60)[0])
