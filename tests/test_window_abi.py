"""Refusals of the windowed entry points and of the step's bookkeeping: every bad
argument is answered before any CUDA call, so fake pointers serve and no GPU is needed."""
import ctypes

import pytest

from io_aware_exact_12_gb300 import build as build_mod

MB = 1 << 20
Q, K, V, O, DO, LSE, DQ, DK, DV, TABLE, LENS, NEW, OLD, RING, STATE, STATE2, START, SLOTS, WS = (0x100000000 + i * 64 * MB for i in range(19))


@pytest.fixture(scope="module")
def pkg():
    build_mod.build()
    import io_aware_exact_12_gb300 as p
    p.lib()
    return p


def _t(pkg, p, heads, n, d=64, batch=None, head=None, row=None):
    return ctypes.byref(pkg._BhndStruct(p, heads * n * d if batch is None else batch, n * d if head is None else head, d if row is None else row))


def _fwd(pkg, q=None, k=None, v=None, o=None, lse=LSE, B=2, Hq=4, Hk=2, nq=16, nk=32, d=64, window=8, sinks=1, scale=0.1, type=0):
    return pkg.lib().attn_fwd_window(q or _t(pkg, Q, 4, 16), k or _t(pkg, K, 2, 32), v or _t(pkg, V, 2, 32), o or _t(pkg, O, 4, 16), lse, B, Hq, Hk, nq, nk, d, window,
                                     sinks, scale, type, None)


def _bwd(pkg, o=None, do=None, lse=LSE, dq=None, dk=None, dv=None, window=8, ws=WS):
    return pkg.lib().attn_bwd_window(_t(pkg, Q, 4, 16), _t(pkg, K, 2, 32), _t(pkg, V, 2, 32), o or _t(pkg, O, 4, 16), do or _t(pkg, DO, 4, 16), lse,
                                     dq or _t(pkg, DQ, 4, 16), dk or _t(pkg, DK, 2, 32), dv or _t(pkg, DV, 2, 32), 2, 4, 2, 16, 32, 64, window, 1, 0.1, 0, ws, None)


def _past_checks(rc):
    return rc in (3, 5)  # no device here, or not the right one


@pytest.fixture(autouse=True)
def _no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("the pointers are not memory")


def test_valid_arguments_reach_the_device_check(pkg):
    assert _past_checks(_fwd(pkg)) and _past_checks(_bwd(pkg)) and _past_checks(_assign(pkg)) and _past_checks(_decode(pkg))


def test_sizes(pkg):
    for kw in (dict(B=0), dict(Hq=0), dict(Hk=0), dict(Hk=3), dict(nq=0), dict(nk=8), dict(window=0), dict(window=-5), dict(sinks=-1), dict(type=2), dict(type=-1),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38), dict(lse=None), dict(lse=LSE + 2)):
        assert _fwd(pkg, **kw) == 1, kw
    for kw in (dict(d=48), dict(d=256), dict(B=20000), dict(nk=(1 << 24) + 1)):
        assert _fwd(pkg, **kw) == 2, kw


def test_backward_workspace(pkg):
    need = pkg.lib().attn_bwd_window_workspace
    good = (2, 4, 2, 16, 32, 64, 8, 1)
    assert need(*good) >= 2 * 2 * 4 * 128 * 4
    for at, bad in ((0, 0), (1, 3), (2, 0), (3, 0), (4, 8), (5, 48), (6, 0), (7, -1), (0, 20000)):
        assert need(*(bad if i == at else x for i, x in enumerate(good))) == 0, (at, bad)
    # two row vectors, runs of sinks (8 to an SM) and of cut tiles (16 to each of fewer than 152) at most, however long the sequence
    assert need(1, 1, 1, 1 << 24, 1 << 24, 128, 128, 4) <= 2 * (1 << 24) * 4 + (8 * 152 + 1 + 16 * 152) * 2 * 128 * 128 * 4


def test_tensors(pkg):
    for name, heads, n in (("q", 4, 16), ("k", 2, 32), ("v", 2, 32), ("o", 4, 16)):
        p = {"q": Q, "k": K, "v": V, "o": O}[name]
        for bad in (_t(pkg, None, heads, n), _t(pkg, p + 8, heads, n), _t(pkg, p, heads, n, row=-64), _t(pkg, p, heads, n, row=63), _t(pkg, p, heads, n, row=60),
                    _t(pkg, p, heads, n, row=0), _t(pkg, p, heads, n, head=0), _t(pkg, p, heads, n, batch=64), _t(pkg, p, heads, n, batch=1 << 39)):
            assert _fwd(pkg, **{name: bad}) == 1, name
    # token-major tensors, and any stride along an extent of 1
    assert _past_checks(_fwd(pkg, q=_t(pkg, Q, 4, 16, head=64, row=256)))
    assert _past_checks(_fwd(pkg, q=_t(pkg, Q, 4, 1, head=64, row=12345), o=_t(pkg, O, 4, 1), nq=1))


def test_overlaps(pkg):
    assert _fwd(pkg, o=_t(pkg, Q, 4, 16)) == 1
    assert _fwd(pkg, o=_t(pkg, K, 4, 16)) == 1
    assert _fwd(pkg, lse=Q) == 1
    assert _fwd(pkg, lse=O + 64) == 1
    assert _bwd(pkg, dq=_t(pkg, DK, 4, 16)) == 1
    assert _bwd(pkg, dk=_t(pkg, DV, 2, 32)) == 1
    assert _bwd(pkg, dv=_t(pkg, DO, 2, 32)) == 1
    assert _bwd(pkg, dq=_t(pkg, LSE, 4, 16)) == 1
    for ws in (None, WS + 8, Q, LSE, DK, DO):
        assert _bwd(pkg, ws=ws) == 1, ws
    # slices of one buffer side by side are apart, unless they reach into one another
    row = 10 * 64
    s = lambda at, heads, n=32: _t(pkg, TABLE + at * 128, heads, n, batch=n * row, head=64, row=row)  # noqa: E731
    assert _past_checks(_bwd(pkg, dk=s(0, 2), dv=s(2, 2)))
    assert _past_checks(_bwd(pkg, dk=s(8, 2), dv=s(0, 2)))
    assert _bwd(pkg, dk=s(0, 2), dv=s(1, 2)) == 1
    assert _bwd(pkg, dk=s(0, 2), dv=s(9, 2)) == 1


def _kv(pkg, **kw):
    H, page, d = 2, 16, 64
    f = dict(k_pages=K, v_pages=V, k_min=None, k_max=None, block_table=TABLE, seq_lens=LENS, table_stride=8, num_pages=32, page_size=page, kv_heads=H, head_dim=d,
             max_pages=8, B=3, type=0, k_scale=1.0, v_scale=1.0)
    f.update(kw)
    three = ctypes.c_longlong * 3
    return ctypes.byref(pkg._PagedKvStruct(k_strides=three(H * page * d, page * d, d), v_strides=three(H * page * d, page * d, d), **f))


def _decode(pkg, window=8, sinks=2, scale=0.1, ws=WS, heads=4, o=O, **kw):
    q = ctypes.byref(pkg._RowsStruct(Q, heads * 64, 64))
    return pkg.lib().attn_paged_decode_window(_kv(pkg, **kw), q, heads, o, LSE, window, sinks, scale, 0, ws, None)


def _assign(pkg, n_new=NEW, lens=OLD, ring=RING, cap=40, state=STATE, out=STATE2, start=START, slots=SLOTS, rows=64, window=20, sinks=4, ws=WS, **kw):
    return pkg.lib().attn_paged_assign(_kv(pkg, **kw), n_new, lens, ring, cap, state, out, start, slots, rows, window, sinks, ws, None)


def test_decode_window(pkg):
    for kw in (dict(window=0), dict(window=-1), dict(sinks=-1), dict(scale=float("nan")), dict(ws=None), dict(ws=WS + 8), dict(heads=3), dict(o=O + 8), dict(block_table=None)):
        assert _decode(pkg, **kw) == 1, kw
    for kw in (dict(window=(1 << 30) + 1), dict(sinks=(1 << 30) + 1), dict(page_size=12)):
        assert _decode(pkg, **kw) == 2, kw
    L, P = pkg.lib(), 1 << 30
    assert L.attn_paged_decode_window_workspace(_kv(pkg), 4, 8, 2) > 0
    for bad in ((3, 8, 2), (4, 0, 2), (4, 8, -1), (4, P + 1, 0), (4, 8, P + 1)):
        assert L.attn_paged_decode_window_workspace(_kv(pkg), *bad) == 0
    # never more than over all pages, and no more for a wider window than for a table
    most = L.attn_paged_decode_workspace(_kv(pkg), 4, 0)
    assert L.attn_paged_decode_window_workspace(_kv(pkg), 4, 8, 2) <= most == L.attn_paged_decode_window_workspace(_kv(pkg), 4, P, P)


def test_assign(pkg):
    for kw in (dict(n_new=None), dict(ring=None), dict(state=None), dict(start=None), dict(ws=None), dict(cap=0), dict(rows=-1), dict(window=-1), dict(sinks=-1),
               dict(n_new=NEW + 2), dict(lens=OLD + 1), dict(ring=RING + 2), dict(state=STATE + 1), dict(out=STATE2 + 2), dict(start=START + 2), dict(slots=SLOTS + 4),
               dict(ws=WS + 4), dict(block_table=None), dict(seq_lens=None)):
        assert _assign(pkg, **kw) == 1, kw
    for kw in (dict(window=(1 << 30) + 1), dict(sinks=(1 << 30) + 1), dict(rows=(1 << 30) + 1), dict(cap=(1 << 30) + 1)):
        assert _assign(pkg, **kw) == 2, kw
    # overlaps: what is written with what is read, or with what else is written
    for kw in (dict(n_new=LENS), dict(n_new=TABLE), dict(lens=LENS + 4), dict(ring=NEW), dict(ring=OLD), dict(out=STATE + 4), dict(out=NEW), dict(start=NEW), dict(slots=START),
               dict(ws=SLOTS), dict(ring=TABLE), dict(state=RING, out=None), dict(ring=K), dict(ws=V)):
        assert _assign(pkg, **kw) == 1, kw
    # in place, and without what is not wanted
    for kw in (dict(lens=None), dict(lens=LENS), dict(out=None), dict(out=STATE), dict(slots=None), dict(rows=0), dict(window=0, sinks=0)):
        assert _past_checks(_assign(pkg, **kw)), kw
    assert pkg.lib().attn_paged_assign_workspace(_kv(pkg)) > 0
    assert pkg.lib().attn_paged_assign_workspace(_kv(pkg, B=0)) == 0
