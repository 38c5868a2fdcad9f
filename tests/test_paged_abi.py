"""Refusals of the paged-cache entry points: every bad argument is answered
before any CUDA call, so fake pointers serve and no GPU is needed."""
import copy
import ctypes

import pytest
import torch

from io_aware_exact_12_gb300 import build as build_mod

MB = 1 << 20
K, V, Q, O, LSE, LIST, TABLE, LENS, KMIN, KMAX, WS, NEWK, NEWV, QOUT, START, COS, SIN = (
    0x100000000 + i * 64 * MB for i in range(17))


@pytest.fixture(scope="module")
def pkg():
    build_mod.build()
    import io_aware_exact_12_gb300 as p
    p.lib()
    return p


def _kv(pkg, **kw):
    P, H, page, d = kw.pop("P", 32), kw.pop("H", 2), kw.pop("page", 16), kw.pop("d", 64)
    f = dict(k_pages=K, v_pages=V, k_min=KMIN, k_max=KMAX, block_table=TABLE, seq_lens=LENS, table_stride=8,
             num_pages=P, page_size=page, kv_heads=H, head_dim=d, max_pages=8, B=3, type=0, k_scale=1.0, v_scale=1.0)
    ks = kw.pop("k_strides", (H * page * d, page * d, d))
    vs = kw.pop("v_strides", (H * page * d, page * d, d))
    f.update(kw)
    three = ctypes.c_longlong * 3
    return pkg._PagedKvStruct(k_strides=three(*ks), v_strides=three(*vs), **f)


def _rows(pkg, p, heads=2, d=64, row=None, head=None):
    return ctypes.byref(pkg._RowsStruct(p, heads * d if row is None else row, d if head is None else head))


def _append(pkg, kv=None, k=None, v=None, q=None, q_out=None, heads=4, rows=3, start=None, cos=COS, sin=SIN,
            table_rows=128, rot=64, x=0, no_q=False, **kw):
    kv = _kv(pkg, **kw) if kv is None else kv
    q = None if no_q else (q or _rows(pkg, Q, heads))
    q_out = None if no_q else (q_out or _rows(pkg, QOUT, heads))
    return pkg.lib().attn_paged_append(ctypes.byref(kv), k or _rows(pkg, NEWK), v or _rows(pkg, NEWV), q, q_out,
                                       heads, rows, start, cos, sin, table_rows, rot, 0, x, None)


def _decode(pkg, q=None, heads=4, o=O, lse=LSE, pages=None, n=0, scale=0.125, x=0, ws=WS, **kw):
    kv = _kv(pkg, **kw)
    return pkg.lib().attn_paged_decode(ctypes.byref(kv), q or _rows(pkg, Q, heads), heads, o, lse, pages, n, scale, x,
                                       ws, None)


def _select(pkg, q=None, heads=4, pages=LIST, n=4, first=1, last=1, x=0, ws=WS, **kw):
    kv = _kv(pkg, **kw)
    return pkg.lib().attn_paged_select(ctypes.byref(kv), q or _rows(pkg, Q, heads), heads, pages, n, first, last, x,
                                       ws, None)


def test_valid_arguments_reach_the_device_check(pkg):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: fake pointers would launch")
    assert _append(pkg) in (3, 5)
    assert _append(pkg, no_q=True, heads=0) in (3, 5)
    assert _append(pkg, start=START, rows=100) in (3, 5)
    assert _append(pkg, q_out=_rows(pkg, Q, 4)) in (3, 5)  # in place
    assert _decode(pkg) in (3, 5)
    assert _decode(pkg, pages=LIST, n=4) in (3, 5)
    assert _select(pkg) in (3, 5)
    # pages stored as [page_size, kv_heads, d]; K and V in turns in one array
    assert _decode(pkg, k_strides=(2048, 64, 128), v_strides=(2048, 64, 128)) in (3, 5)
    assert _decode(pkg, v_pages=K + 4096, k_strides=(4096, 1024, 64), v_strides=(4096, 1024, 64)) in (3, 5)


CACHE = [
    (dict(k_pages=None), 1), (dict(v_pages=None), 1), (dict(block_table=None), 1), (dict(seq_lens=None), 1),
    (dict(k_pages=K + 8), 1), (dict(v_pages=V + 2), 1), (dict(block_table=TABLE + 2), 1), (dict(seq_lens=LENS + 1), 1),
    (dict(B=0), 1), (dict(P=0), 1), (dict(H=0, k_strides=(2048, 1024, 64), v_strides=(2048, 1024, 64)), 1),
    (dict(max_pages=0), 1), (dict(type=3), 1), (dict(type=1), 1),  # an fp16 cache takes no bf16 rows
    (dict(k_scale=0.5), 1), (dict(v_scale=2.0), 1),                # scales are e4m3's
    (dict(type=2, k_scale=0.0), 1), (dict(type=2, v_scale=float("inf")), 1), (dict(type=2, k_scale=float("nan")), 1),
    (dict(d=96), 2), (dict(d=256), 2), (dict(page=12), 2), (dict(page=2048), 2), (dict(B=40000), 2),
    (dict(max_pages=1 << 27, table_stride=1 << 27), 2), (dict(table_stride=7), 1), (dict(table_stride=-1), 1),
    (dict(k_max=None), 1), (dict(k_min=KMAX), 1), (dict(k_min=K + 64), 1),
    (dict(v_pages=K), 1),
    (dict(k_strides=(2048, 1024, 60)), 1),    # not a multiple of 16 bytes
    (dict(k_strides=(2048, 1024, 0)), 1),     # rows overlap
    (dict(v_strides=(2048, 512, 64)), 1),
    (dict(v_strides=(1024, 1024, 64)), 1),
    (dict(k_strides=(-2048, 1024, 64)), 1),
    (dict(k_strides=(1 << 41, 1024, 64)), 1),
]


@pytest.mark.parametrize("kw,code", CACHE, ids=[str(c[0]) for c in CACHE])
def test_bad_caches_are_refused_by_every_call(pkg, kw, code):
    assert _append(pkg, **kw) == code
    assert _decode(pkg, **kw) == code
    assert _select(pkg, **kw) == code


def test_append_refusals(pkg):
    assert _append(pkg, k=_rows(pkg, None)) == 1
    assert _append(pkg, v=_rows(pkg, NEWV + 8)) == 1
    assert _append(pkg, k=_rows(pkg, NEWK, row=100)) == 1       # row stride not a multiple of 8 elements
    assert _append(pkg, k=_rows(pkg, NEWK, head=-64)) == 1
    assert _append(pkg, rows=4) == 1                             # one row per sequence without token_start
    assert _append(pkg, rows=-1, start=START) == 1
    assert _append(pkg, start=START + 2, rows=10) == 1
    assert _append(pkg, q_out=_rows(pkg, Q + 128, 4)) == 1       # overlaps q but is not q
    assert _append(pkg, q_out=_rows(pkg, NEWK, 4)) == 1
    assert _append(pkg, q_out=_rows(pkg, QOUT, 4, row=0)) == 1   # an output's rows share bytes
    assert _append(pkg, k=_rows(pkg, K)) == 1                    # new rows inside the cache
    assert _append(pkg, rot=8) == 2
    assert _append(pkg, rot=128) == 2
    assert _append(pkg, cos=None) == 1
    assert _append(pkg, sin=SIN + 4) == 1
    assert _append(pkg, table_rows=0) == 1
    assert _append(pkg, cos=K) == 1                              # the cache would overwrite the table
    assert _append(pkg, x=2) == 1                                # rows are bf16 or fp16
    assert _append(pkg, heads=0) == 1                            # q given without heads
    assert _append(pkg, rows=0, start=START) == 0                # nothing to do


def test_decode_refusals(pkg):
    assert _decode(pkg, o=None) == 1
    assert _decode(pkg, lse=None) == 1
    assert _decode(pkg, o=O + 8) == 1
    assert _decode(pkg, lse=LSE + 2) == 1
    assert _decode(pkg, o=Q) == 1
    assert _decode(pkg, o=K + 4096) == 1
    assert _decode(pkg, lse=O) == 1
    assert _decode(pkg, scale=float("nan")) == 1
    assert _decode(pkg, heads=3) == 1                            # not a multiple of the KV heads
    assert _decode(pkg, heads=0) == 1
    assert _decode(pkg, heads=40000) == 2
    assert _decode(pkg, pages=LIST, n=0) == 1
    assert _decode(pkg, pages=LIST + 1, n=4) == 1
    assert _decode(pkg, pages=LIST, n=1 << 27) == 2
    assert _decode(pkg, o=LIST, pages=LIST, n=4) == 1
    assert _decode(pkg, q=_rows(pkg, Q, 4, head=20)) == 1
    assert _decode(pkg, x=2) == 1
    kv = _kv(pkg)
    if pkg.lib().attn_paged_decode_workspace(ctypes.byref(kv), 4, 0):
        assert _decode(pkg, ws=None) == 1
        assert _decode(pkg, ws=Q) == 1


def test_select_refusals(pkg):
    assert _select(pkg, pages=None) == 1
    assert _select(pkg, pages=LIST + 2) == 1
    assert _select(pkg, n=0) == 1
    assert _select(pkg, n=3, first=2, last=2) == 1
    assert _select(pkg, first=-1) == 1
    assert _select(pkg, last=-1) == 1
    assert _select(pkg, heads=5) == 1
    assert _select(pkg, k_min=None, k_max=None) == 1
    assert _select(pkg, pages=KMIN) == 1
    assert _select(pkg, n=1 << 27) == 2
    kv = _kv(pkg)
    if pkg.lib().attn_paged_select_workspace(ctypes.byref(kv)):
        assert _select(pkg, ws=None) == 1
        assert _select(pkg, ws=LIST) == 1


def test_workspace_sizes_of_bad_arguments_are_zero(pkg):
    L = pkg.lib()
    assert L.attn_paged_decode_workspace(None, 4, 0) == 0
    assert L.attn_paged_decode_workspace(ctypes.byref(_kv(pkg)), 3, 0) == 0
    assert L.attn_paged_decode_workspace(ctypes.byref(_kv(pkg, B=0)), 4, 0) == 0
    assert L.attn_paged_select_workspace(None) == 0


def test_the_binding_refuses_what_is_no_cache(pkg):
    t = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(TypeError):
        pkg.PagedKV(t, t, i, i[0])                               # not on a GPU
    for f in (pkg.attn_paged_append, pkg.attn_paged_decode, pkg.attn_paged_select):
        with pytest.raises(TypeError):
            f(t, t, 1)


def test_a_cache_description_cannot_be_changed(pkg):
    """The calls go by the structure that was built at first: an assignment would be passed over in silence, and the
    tensor it replaced freed while the kernels still read it."""
    kv = object.__new__(pkg.PagedKV)
    for name in pkg.PagedKV.__slots__ + ("other",):
        with pytest.raises(AttributeError, match="cannot be changed"):
            setattr(kv, name, 1)
        with pytest.raises(AttributeError, match="cannot be changed"):
            delattr(kv, name)
    assert copy.copy(kv) is kv


def test_many_sequences_of_many_heads_are_taken(pkg):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: fake pointers would launch")
    for B, H, heads in ((512, 8, 128), (1024, 8, 64), (256, 16, 384), (4000, 16, 64)):
        kw = dict(B=B, H=H, heads=heads, table_stride=8, P=4)
        assert _decode(pkg, **kw) in (3, 5), kw
        assert _select(pkg, **kw) in (3, 5), kw
    assert _decode(pkg, B=1, H=1, heads=65535, P=4) in (3, 5)
    assert _decode(pkg, B=1, H=1, heads=65536, P=4) == 2
    assert _decode(pkg, B=2, H=1, heads=40000, P=4) == 2


def test_workspace_sizes_of_refused_sizes_are_zero(pkg):
    """A caller allocates what these say before the call can refuse the sizes."""
    L, by = pkg.lib(), ctypes.byref
    for kw in (dict(d=96), dict(d=256), dict(page=12), dict(page=2048), dict(B=40000), dict(H=70000, k_strides=(0, 0, 0), v_strides=(0, 0, 0)),
               dict(max_pages=1 << 27, table_stride=1 << 27), dict(max_pages=2147483647, table_stride=1 << 31), dict(P=0), dict(max_pages=0)):
        assert L.attn_paged_decode_workspace(by(_kv(pkg, **kw)), 4 * (35000 if "H" in kw else 1), 0) == 0, kw
        assert L.attn_paged_select_workspace(by(_kv(pkg, **kw))) == 0, kw
    assert L.attn_paged_decode_workspace(by(_kv(pkg)), 65538, 0) == 0
    assert L.attn_paged_decode_workspace(by(_kv(pkg)), 40000, 0) == 0
    assert L.attn_paged_decode_workspace(by(_kv(pkg)), 4, 1 << 27) == 0
    assert L.attn_paged_decode_workspace(by(_kv(pkg)), 4, 0) > 0 and L.attn_paged_select_workspace(by(_kv(pkg))) > 0


def test_decode_refuses_scales_whose_product_overflows(pkg):
    assert _decode(pkg, scale=3e38) == 1
    assert _decode(pkg, scale=-3e38) == 1
    assert _decode(pkg, type=2, scale=1e10, k_scale=1e30) == 1
    if not torch.cuda.is_available():
        assert _decode(pkg, scale=2e38) in (3, 5)
        assert _decode(pkg, type=2, scale=1e-10, k_scale=1e30) in (3, 5)


def test_many_sequences_of_many_key_value_heads_are_taken(pkg):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: fake pointers would launch")
    for B, H in ((1024, 64), (8192, 128), (4096, 20)):
        kw = dict(B=B, H=H, P=4, d=32)
        rows = [_rows(pkg, p, H, 32) for p in (NEWK, NEWV, Q, QOUT)]
        assert _decode(pkg, q=rows[2], heads=H, **kw) in (3, 5), kw
        assert _select(pkg, q=rows[2], heads=H, n=3, **kw) in (3, 5), kw
        assert _append(pkg, k=rows[0], v=rows[1], no_q=True, heads=0, rows=B, rot=32, **kw) in (3, 5), kw
    for B, H in ((8192, 129), (8193, 8), (20000, 4)):
        assert _decode(pkg, heads=H, B=B, H=H, P=4) == 2
        assert pkg.lib().attn_paged_select_workspace(ctypes.byref(_kv(pkg, B=B, H=H))) == 0
