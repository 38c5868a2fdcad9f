"""Sliding-window attention where blocks take over the work of blocks that have not
started (more items than the GPU holds blocks), against the float64 forms and
tolerances of test_gpu_window.py; and what a call repeats bit for bit: all of its
outputs, dQ among them, on whatever stream or thread, eager or replayed."""
import math
import threading

import pytest
import torch

import test_gpu_window as base
from test_gpu_window import BF16, F16, _backward, _bounds, _check, _inputs, _near

pytestmark = pytest.mark.gpu
pkg = base.pkg


def _both(pkg, q, k, v, do, window, sinks, **kw):
    o, lse = pkg.attn_fwd_window(q, k, v, window, sinks, **kw)
    return (o, lse) + tuple(pkg.attn_bwd_window(q, k, v, o, do, lse, window, sinks, **kw))


def _same(got, want):
    for name, x, y in zip(("o", "lse", "dq", "dk", "dv"), got, want):
        assert torch.equal(x, y), name


# Items: row tiles x query heads for the forward (304 blocks at once) and dQ (152), key tiles x key/value heads for dK and dV (152).
MANY = [
    # B, Hq, Hk, nq, nk, window, sinks
    (8, 24, 24, 513, 513, 100, 0),      # 960 and 960; last tiles of one row, of one key
    (8, 24, 24, 513, 700, 100, 4),      # 960 and 1152, every third tile of keys without a visit but the sinks'
    (8, 24, 24, 400, 900, 128, 130),    # two tiles of sinks
    (4, 48, 12, 640, 640, 300, 1),      # shared heads
    (5, 24, 3, 1500, 1500, 100, 4),     # whole tiles, cut ones and runs of sinks in one grid
    (40, 8, 8, 300, 1300, 7, 0),        # most key tiles without a visit
    (60, 12, 4, 129, 129, 1000, 0),     # two row tiles, the second of one row
]


@pytest.mark.parametrize("d,dtype,layout", [(32, BF16, "tokens"), (32, F16, "heads"), (64, BF16, "heads"), (64, F16, "slices"), (128, BF16, "slices"), (128, F16, "heads"),
                                            (128, BF16, "tokens")])
@pytest.mark.parametrize("shape", MANY, ids=lambda s: "x".join(map(str, s)))
def test_many_items(pkg, shape, d, dtype, layout):
    B, Hq, Hk, nq, nk, window, sinks = shape
    x = _inputs(B, Hq, Hk, nq, nk, d, dtype, layout, nk + d)
    first = _check(pkg, *x, window, sinks)
    for _ in range(3):
        _same(_both(pkg, *x, window, sinks, scale=1 / math.sqrt(d)), first)
    assert pkg.sync_status() == 0


def test_whole_tiles_cut_tiles_and_runs_of_sinks(pkg):
    """That the fifth shape above has all three: 15 heads of 11 tiles without sinks, of which 13 are past the 152 that run at once."""
    need = pkg.lib().attn_bwd_window_workspace(5, 24, 3, 1500, 1500, 64, 100, 4)
    partial = (need - 2 * 5 * 24 * 1536 * 4) // (2 * 128 * 64 * 4)
    assert partial > 13 * 8 and (partial - 13 * 8) % 15 == 0


@pytest.mark.parametrize("d,dtype", [(32, F16), (64, BF16), (64, F16), (128, BF16)])
@pytest.mark.parametrize("B,H,n", [(300, 12, 100), (200, 12, 129), (400, 8, 1)])
def test_items_of_one_tile(pkg, B, H, n, d, dtype):
    """Items that see one tile of keys follow one another in a block: each hands its stages on while the next has begun."""
    x = _inputs(B, H, H, n, n, d, dtype, "heads", n)
    first = _check(pkg, *x, 1000, 0)
    for _ in range(40):
        _same(_both(pkg, *x, 1000, 0, scale=1 / math.sqrt(d)), first)
    assert pkg.sync_status() == 0


@pytest.mark.parametrize("B,Hq,Hk,nq,nk,d,dtype,window,sinks", [
    (1, 8, 2, 5000, 5000, 128, BF16, 300, 4),
    (1, 8, 2, 5000, 5000, 64, F16, 300, 4),
    (2, 4, 4, 2000, 4001, 32, BF16, 1, 1000),
    (1, 16, 16, 900, 900, 64, BF16, 900, 0),
    (2, 24, 1, 1111, 1111, 128, F16, 77, 200),
    (1, 2, 1, 100, 5000, 128, BF16, 4000, 4),
])
def test_all_repeats_bit_for_bit(pkg, B, Hq, Hk, nq, nk, d, dtype, window, sinks):
    x = _inputs(B, Hq, Hk, nq, nk, d, dtype, "tokens", nq)
    first = _both(pkg, *x, window, sinks)
    for _ in range(20):
        _same(_both(pkg, *x, window, sinks), first)
    assert pkg.sync_status() == 0


@pytest.mark.parametrize("d,dtype", [(32, F16), (64, BF16), (128, BF16), (128, F16)])
def test_streams_threads_and_replays(pkg, d, dtype):
    """The same bits on two streams at once, from a new thread, into given tensors and by a graph."""
    x = _inputs(1, 8, 2, 1500, 1500, d, dtype, "tokens", d)
    want = _both(pkg, *x, 200, 4)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[_both(pkg, *x, 200, 4, stream=s) for s in streams] for _ in range(5)]
    torch.cuda.synchronize()
    for pair in got:
        for one in pair:
            _same(one, want)

    outs = [torch.full_like(t, 7.0) for t in want]
    failed = []

    def work():
        try:
            pkg.attn_fwd_window(*x[:3], 200, 4, o=outs[0], lse=outs[1])
            pkg.attn_bwd_window(*x[:3], outs[0], x[3], outs[1], 200, 4, dq=outs[2], dk=outs[3], dv=outs[4])
        except Exception as e:
            failed.append(e)

    torch.cuda.synchronize()
    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    _same(outs, want)

    bufs = [torch.zeros_like(t) for t in x]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = _both(pkg, *bufs, 200, 4)
    for to, t in zip(bufs, x):
        to.copy_(t)
    for _ in range(3):
        graph.replay()
    _same(captured, want)
    assert pkg.sync_status() == 0


def test_a_threads_dense_call(pkg):
    """The dense forward as a thread's first call gives what it gives elsewhere."""
    q, k, v, _ = (t.contiguous() for t in _inputs(1, 4, 4, 300, 300, 64, BF16, "tokens", 14))
    want = pkg.attn_fwd(q, k, v, causal=True)
    o, lse = torch.full_like(q, 7.0), torch.full_like(want[1], 7.0)
    torch.cuda.synchronize()
    t = threading.Thread(target=lambda: pkg.attn_fwd(q, k, v, causal=True, o=o, lse=lse))
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and pkg.sync_status() == 0


@pytest.mark.parametrize("d", [32, 64, 128])
def test_hidden_keys_do_not_reach_dq(pkg, d):
    q, k, v, do = _inputs(1, 4, 2, 130, 900, d, BF16, "heads", 5)
    window, sinks = 200, 3
    want = _both(pkg, q, k, v, do, window, sinks)
    hidden = slice(sinks, 900 - 130 - window + 1)
    k, v = k.clone(), v.clone()
    k[:, :, hidden], v[:, :, hidden] = 1e4, -1e4
    _same(_both(pkg, q, k, v, do, window, sinks), want)


def test_slices_of_one_buffer(pkg):
    """dq, dk and dv side by side in one buffer: the bits of dense ones."""
    x = _inputs(2, 4, 2, 333, 333, 64, BF16, "slices", 7)
    want = _both(pkg, *x, 100, 4)
    grads = torch.full((2, 333, 8, 64), 7.0, dtype=BF16, device="cuda")
    dq, dk, dv = (t.transpose(1, 2) for t in grads.split([4, 2, 2], 2))
    pkg.attn_bwd_window(*x[:3], want[0], x[3], want[1], 100, 4, dq=dq, dk=dk, dv=dv)
    _same((dq, dk, dv), want[2:])


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_autograd_of_shared_and_broadcast_heads(pkg, dtype):
    """Gradients through attention() are the call's, bit for bit; those of one key/value head are the sums over the query heads, whether
    the call shares the head or the caller has broadcast it."""
    n, d, u = 200, 64, torch.finfo(dtype).eps / 2
    q, k, v, do = _inputs(2, 4, 1, n, n, d, dtype, "tokens", 9)
    want = _both(pkg, q, k, v, do, 50, 3)
    leaves = [t.detach().clone().requires_grad_() for t in (q, k, v)]
    o = pkg.attention(*leaves, window=50, sinks=3)
    o.backward(do)
    _same((o, want[1]) + tuple(t.grad for t in leaves), want)
    f = lambda *t: [x.double() for x in t]  # noqa: E731
    args = f(q, k, v, want[0], do, want[1])
    ref = _backward(*args, 50, 3, d ** -0.5)
    for x, r, t in zip(leaves, ref, _bounds(*args, 50, 3, d ** -0.5, u)[2:]):
        _near("shared", x.grad, r, t)
    # broadcast: a gradient of each query head, rounded, then their sum, rounded
    leaves = [t.detach().clone().requires_grad_() for t in (q, k, v)]
    o = pkg.attention(leaves[0], leaves[1].expand(2, 4, n, d), leaves[2].expand(2, 4, n, d), window=50, sinks=3)
    assert torch.equal(o, want[0])
    o.backward(do)
    kk, vv = (t.expand(2, 4, n, d) for t in (args[1], args[2]))
    ref = _backward(args[0], kk, vv, *args[3:], 50, 3, d ** -0.5)
    tol = _bounds(args[0], kk, vv, *args[3:], 50, 3, d ** -0.5, u)[2:]
    _near("dq", leaves[0].grad, ref[0], tol[0])
    for x, r, t in zip(leaves[1:], ref[1:], tol[1:]):
        total = r.sum(1, keepdim=True)
        # the four may be added in their own type: three more roundings of partial sums
        more = u * (total.abs() + 3 * r.abs().sum(1, keepdim=True))
        _near("broadcast", x.grad, total, (t.sum(1, keepdim=True) + more) * (1 + 4 * u))
