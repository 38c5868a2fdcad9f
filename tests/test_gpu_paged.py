"""The paged cache on the GPU against plain float64 forms: appending rotated
rows, decoding over all pages or over selected ones, selecting pages, and the
three together as a server runs them.

Tolerances come from the arithmetic.  A rounding to a type errs by at most half
a step, finfo(t).eps / 2 of the value.
  append: fp32 rotation of exact inputs errs by at most 3 roundings, 2^-22 of
    |x1| + |x2|, then one rounding to the stored type (e4m3: after a
    multiplication by 1 / scale, 2 more fp32 roundings; below 2^-6 its step is
    2^-9 whatever the value).
  decode: logits are fp32 sums of d products with the weights' argument rounded
    once more, off by dt <= (d + 8) 2^-24 sum |q k| |scale| each; a weight then
    by 2 dt + 2^-20 relative (exp2 and the sums); P is rounded to 16 bits with
    the same rounded weights in the denominator, so by the 16-bit type's eps / 2
    about a mean of w |v|.  O then has one rounding of its own.
    (The kernel keeps more of P, two 16-bit words and an fp32 sum, so that this
    part is an upper bound; test_decode_weights_keep_more_than_16_bits has its own.)
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F16, E4M3 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
NAN_BYTE = 0x7F


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from io_aware_exact_12_gb300 import build as b
    b.build()
    import io_aware_exact_12_gb300 as p
    p.lib()
    return p


def _raw(t):
    return t.view(torch.uint8) if t.dtype == E4M3 else t


def _storage(P, H, page, d, dtype, layout):
    """Two [P, H, page, d] views in the given memory order, every element NaN."""
    def nans(shape):
        if dtype == E4M3:
            return torch.full(shape, NAN_BYTE, dtype=torch.uint8, device="cuda").view(E4M3)
        return torch.full(shape, math.nan, dtype=dtype, device="cuda")
    if layout == "heads":       # [P, H, page, d]
        return nans((P, H, page, d)), nans((P, H, page, d))
    if layout == "tokens":      # [P, page, H, d]
        return nans((P, page, H, d)).permute(0, 2, 1, 3), nans((P, page, H, d)).permute(0, 2, 1, 3)
    both = nans((P, 2, H, page, d))  # K and V of a page in turns
    return both[:, 0], both[:, 1]


class Case:
    """A cache of sequences `lens`: random pages, NaN in every slot that no token fills, table entries behind a
    sequence's pages that no kernel may follow."""

    def __init__(self, pkg, lens, H=2, page=16, d=64, dtype=BF16, layout="heads", seed=0, scales=(1.0, 1.0), width=None,
                 summaries=False, fill=True, spare=3):
        g = torch.Generator().manual_seed(seed)
        self.g, self.lens_list, self.H, self.page, self.d, self.dtype = g, list(lens), H, page, d, dtype
        need = [-(-n // page) for n in lens]
        width = max(need + [1]) + 1 if width is None else width
        P = sum(need) + spare
        ids = torch.randperm(P, generator=g).tolist()
        self.table = torch.full((len(lens), width), 0x7FFFFFF0, dtype=torch.int32)
        for b, n in enumerate(need):
            for j in range(n):
                self.table[b, j] = ids.pop()
        self.free = ids
        self.k, self.v = _storage(P, H, page, d, dtype, layout)
        self.scales = scales if dtype == E4M3 else (1.0, 1.0)
        self.k_ref = torch.zeros(len(lens), H, max(need + [1]) * page, d, dtype=torch.float64)  # as values
        self.v_ref = self.k_ref.clone()
        for b, n in enumerate(lens if fill else []):
            for ref, to, s in ((self.k_ref, self.k, self.scales[0]), (self.v_ref, self.v, self.scales[1])):
                x = torch.randn((H, n, d), generator=g) / s
                x = x.clamp(-448, 448).to(dtype)
                ref[b, :, :n] = x.double() * s
                for j in range(need[b]):
                    m = min(page, n - j * page)
                    _raw(to)[int(self.table[b, j]), :, :m] = _raw(x[:, j * page:j * page + m].contiguous()).cuda()
        self.k_min = self.k_max = None
        if summaries:
            self.k_min = torch.zeros(P, H, d, dtype=dtype, device="cuda")
            self.k_max = torch.zeros(P, H, d, dtype=dtype, device="cuda")
            for b, n in enumerate(lens if fill else []):
                for j in range(need[b]):
                    x = self.k_ref[b, :, j * page:min(n, (j + 1) * page)] / self.scales[0]
                    _raw(self.k_min)[int(self.table[b, j])] = _raw(x.amin(1).to(dtype)).cuda()
                    _raw(self.k_max)[int(self.table[b, j])] = _raw(x.amax(1).to(dtype)).cuda()
        self.block_table = self.table.cuda()
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.kv = pkg.PagedKV(self.k, self.v, self.block_table, self.seq_lens, k_scale=self.scales[0],
                              v_scale=self.scales[1], k_min=self.k_min, k_max=self.k_max)

    def randn(self, *shape, dtype=None):
        return torch.randn(shape, generator=self.g).to(dtype or (BF16 if self.dtype == E4M3 else self.dtype))


def _reference(c, q, scale, keys=None):
    """float64 attention of q [B, Hq, d] over the cached values; keys[b][h]: the visible positions (None: all).
    Also each output's tolerance."""
    B, Hq, d = q.shape
    G = Hq // c.H
    o, lse = torch.zeros(B, Hq, d, dtype=torch.float64), torch.full((B, Hq), -math.inf, dtype=torch.float64)
    tol_o, tol_l = torch.zeros(B, Hq, d, dtype=torch.float64), torch.zeros(B, Hq, dtype=torch.float64)
    eps = torch.finfo(q.dtype).eps / 2
    eps_p = eps if c.dtype != E4M3 else torch.finfo(F16).eps / 2  # an e4m3 cache is multiplied in fp16
    for b, n in enumerate(c.lens_list):
        for h in range(c.H):
            at = torch.arange(n) if keys is None else torch.as_tensor(keys[b][h], dtype=torch.long)
            if len(at) == 0:
                continue
            k, v = c.k_ref[b, h, at], c.v_ref[b, h, at]
            x = q[b, h * G:(h + 1) * G].double()
            t = scale * (x @ k.T)
            w = torch.softmax(t, -1)
            dt = ((d + 8) * 2.0 ** -24 * abs(scale) * (x.abs() @ k.abs().T)).amax(-1, keepdim=True)
            rows = slice(h * G, (h + 1) * G)
            o[b, rows], lse[b, rows] = w @ v, torch.logsumexp(t, -1)
            spread = w @ v.abs() + (w @ v).abs()
            tol_o[b, rows] = eps * (w @ v).abs() * (1 + 1e-3) + (eps_p + 2 * dt + 2.0 ** -20) * spread + 1e-30
            if q.dtype == F16:
                tol_o[b, rows] += 2.0 ** -25  # fp16 steps below its normal range
            tol_l[b, rows] = dt[:, 0] + 2.0 ** -20 + 2.0 ** -22 * lse[b, rows].abs()
    return o, lse, tol_o, tol_l


def _check_decode(pkg, c, q, scale=None, pages=None, keys=None, **kw):
    scale = 1 / math.sqrt(c.d) if scale is None else scale
    o, lse = pkg.attn_paged_decode(c.kv, q.cuda() if not q.is_cuda else q, pages=pages, scale=scale, **kw)
    assert pkg.sync_status() == 0
    ro, rl, to, tl = _reference(c, q.cpu(), scale, keys)
    err = (o.double().cpu() - ro).abs()
    assert torch.isfinite(o.float()).all()
    assert (err <= to).all(), "o off by %g of its tolerance" % (err / to).max()
    l = lse.double().cpu()
    none = rl == -math.inf
    assert torch.equal(l == -math.inf, none)
    lerr = (l[~none] - rl[~none]).abs()
    assert (lerr <= tl[~none]).all(), "lse off by %g of its tolerance" % (lerr / tl[~none]).max()
    assert (o.cpu()[none] == 0).all()
    return o, lse


TYPES = [(BF16, BF16, (1.0, 1.0)), (F16, F16, (1.0, 1.0)), (BF16, E4M3, (0.03, 0.011)), (F16, E4M3, (0.0625, 0.5))]


# ------------------------------------------------------------------ decode

@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("x,dtype,scales", TYPES)
def test_decode_lengths_around_the_borders(pkg, x, dtype, scales, d):
    lens = [0, 1, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 1000, 0]
    c = Case(pkg, lens, H=2, page=16, d=d, dtype=dtype, scales=scales, seed=d)
    _check_decode(pkg, c, c.randn(len(lens), 6, d, dtype=x))


@pytest.mark.parametrize("page", [8, 24, 32, 56, 64, 128, 1024])
@pytest.mark.parametrize("layout", ["heads", "tokens", "turns"])
def test_decode_pages_and_layouts(pkg, page, layout):
    lens = [700, 1, page, page + 1, 2 * page - 1]
    c = Case(pkg, lens, H=3, page=page, d=128, layout=layout, seed=page)
    _check_decode(pkg, c, c.randn(len(lens), 3, 128))
    c = Case(pkg, lens, H=1, page=page, d=64, dtype=E4M3, layout=layout, seed=page, scales=(0.02, 0.03))
    _check_decode(pkg, c, c.randn(len(lens), 4, 64, dtype=F16))


@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 9, 15, 16, 17, 24, 33, 71])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_decode_group_sizes(pkg, group, dtype):
    c = Case(pkg, [300, 41], H=2, d=64, dtype=dtype, seed=group, scales=(0.02, 0.03))
    _check_decode(pkg, c, c.randn(2, 2 * group, 64))


@pytest.mark.parametrize("scale", [0.0, -0.3, 0.5])
def test_decode_scales(pkg, scale):
    c = Case(pkg, [900, 3], d=128, seed=4)
    _check_decode(pkg, c, c.randn(2, 4, 128), scale=scale)


def test_decode_large_logits(pkg):
    """Logits of a few hundred: the running maximum moves by more than exp2's range between tiles."""
    c = Case(pkg, [2000, 77], d=128, dtype=F16, seed=5)
    _check_decode(pkg, c, c.randn(2, 8, 128) * 16, scale=1.0)


def test_decode_tiny_and_huge_queries_over_an_8_bit_cache(pkg):
    """bf16 queries outside fp16's range, with scales that bring the logits back."""
    for power in (-100, 90):
        c = Case(pkg, [500], H=1, d=64, dtype=E4M3, seed=6, scales=(2.0 ** -5, 0.1))
        q = (c.randn(1, 4, 64).float() * 2.0 ** power).to(BF16)
        _check_decode(pkg, c, q, scale=0.125 * 2.0 ** -power)


def test_decode_one_long_sequence(pkg):
    """Many splits of one (sequence, head)."""
    c = Case(pkg, [70001], H=1, page=64, d=64, seed=7)
    _check_decode(pkg, c, c.randn(1, 4, 64))


@pytest.mark.parametrize("B", [1, 7, 200])
def test_decode_ragged_batches(pkg, B):
    g = torch.Generator().manual_seed(B)
    lens = [int(x) for x in (torch.rand(B, generator=g) ** 3 * 1500)]
    c = Case(pkg, lens, H=2, d=32, seed=B, width=200)
    _check_decode(pkg, c, c.randn(B, 8, 32))


def test_decode_a_slice_of_a_projection(pkg):
    c = Case(pkg, [100, 200, 5], d=64, seed=8)
    qkv = c.randn(3, 4 + 2 + 2, 64).cuda()
    _check_decode(pkg, c, qkv[:, :4])
    _check_decode(pkg, c, qkv.transpose(0, 1).contiguous().transpose(0, 1)[:, 2:6])


def test_decode_writes_what_it_is_given(pkg):
    c = Case(pkg, [50, 0], d=64, seed=9)
    o = torch.full((4, 4, 64), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((4, 4), 7.0, device="cuda")
    r = pkg.attn_paged_decode(c.kv, c.randn(2, 4, 64).cuda(), o=o[:2], lse=lse[:2])
    assert pkg.sync_status() == 0
    assert r[0].data_ptr() == o.data_ptr() and r[1].data_ptr() == lse.data_ptr()
    assert (o[2:] == 7).all() and (lse[2:] == 7).all() and (o[1] == 0).all()


def test_decode_past_32_bit_offsets(pkg):
    """Pages more than 4 GB apart."""
    d, page, H = 128, 64, 4
    P = (5 << 30) // (H * page * d * 2)
    k = torch.zeros((P, H, page, d), dtype=BF16, device="cuda")
    v = torch.zeros((P, H, page, d), dtype=BF16, device="cuda")
    c = Case(pkg, [150, 20], H=H, page=page, d=d, seed=10, spare=0)
    far = torch.tensor([P - 1, 3, P - 2, P - 3])
    near = torch.cat([c.table[0, :3], c.table[1, :1]]).long()
    k[far.cuda()], v[far.cuda()] = c.k[near.cuda()], c.v[near.cuda()]
    c.block_table[0, :3] = far[:3].int().cuda()
    c.block_table[1, :1] = far[3:].int().cuda()
    c.kv = pkg.PagedKV(k, v, c.block_table, c.seq_lens)
    _check_decode(pkg, c, c.randn(2, 8, d))


def test_decode_is_reproducible(pkg):
    c = Case(pkg, [5000, 1, 1203], H=2, d=128, seed=11)
    q = c.randn(3, 8, 128).cuda()
    first = pkg.attn_paged_decode(c.kv, q)
    for _ in range(5):
        again = pkg.attn_paged_decode(c.kv, q)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert pkg.sync_status() == 0


def test_bad_page_numbers_and_lengths_are_left_out(pkg):
    c = Case(pkg, [100, 100], H=1, d=64, seed=12)
    q = c.randn(2, 2, 64)
    good = c.block_table.clone()
    for bad in (-1, c.k.shape[0], 0x7FFFFFFF):
        c.block_table.copy_(good)
        c.block_table[0, 2] = bad
        o, lse = pkg.attn_paged_decode(c.kv, q.cuda())
        assert pkg.sync_status() == 6
        ro, rl, to, tl = _reference(c, q, 0.125, [[[i for i in range(100) if i // 16 != 2]], [list(range(100))]])
        assert ((o.double().cpu() - ro).abs() <= to).all() and ((lse.double().cpu() - rl).abs() <= tl).all()
    c.block_table.copy_(good)
    assert pkg.sync_status() == 0
    c.seq_lens[1] = -5
    o, lse = pkg.attn_paged_decode(c.kv, q.cuda())
    assert pkg.sync_status() == 6
    assert (o[1] == 0).all() and (lse[1] == -math.inf).all()
    c.seq_lens[1] = 1 << 29  # more than the table row holds: cut to it, and the row's end holds no page
    pkg.attn_paged_decode(c.kv, q.cuda())
    assert pkg.sync_status() == 6
    # an unrelated call is not disturbed
    x = torch.randn(1, 2, 300, 64, dtype=BF16, device="cuda")
    pkg.attn_fwd(x, x, x)
    assert pkg.sync_status() == 0


# ------------------------------------------------------------------ append

def _rotated(x, pos, cos, sin, interleaved):
    y, mag = x.double().clone(), x.double().abs()
    if cos is None:
        return y, mag
    half = cos.shape[1]
    cs, sn = cos[pos].double()[:, None], sin[pos].double()[:, None]
    one, two = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved
                else (slice(0, half), slice(half, 2 * half)))
    a, b = x[..., one].double(), x[..., two].double()
    y[..., one], y[..., two] = a * cs - b * sn, b * cs + a * sn
    mag[..., one] = mag[..., two] = a.abs() + b.abs()
    return y, mag


def _near(got, want, mag, dtype, scale=1.0):
    """got, as stored, within one rounding of want / scale (and of the fp32 work before it)."""
    want, mag = want / scale, mag / scale
    tol = torch.finfo(dtype).eps / 2 * want.abs() * (1 + 1e-3) + 2.0 ** -21 * mag
    if dtype == E4M3:
        want = want.clamp(-448, 448)
        tol = torch.maximum(tol * (1 + 1e-3), torch.tensor(2.0 ** -10)) + 2.0 ** -21 * mag
    elif dtype == F16:
        tol = tol + 2.0 ** -25
    err = (got.double() - want).abs()
    assert (err <= tol).all(), "off by %g of the tolerance" % (err / tol).max()


def _check_append(pkg, c, new, x, Hq=4, rot=None, interleaved=False, pad=0, single=False, in_place=False, positions=None):
    """Appends the last new[b] tokens of each sequence and compares everything that the call may touch."""
    B, d, page = len(new), c.d, c.page
    rot = d if rot is None else rot
    T = sum(new) + pad
    qkv = c.randn(T, Hq + 2 * c.H, d, dtype=x).cuda()
    q, k, v = qkv.split([Hq, c.H, c.H], dim=1)
    cos, sin = pkg.rotation_tables(positions or max(c.lens_list), rot, device="cuda") if rot else (None, None)
    start = None if single else torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
    before = [_raw(t).clone() for t in (c.k, c.v)]
    sums = [_raw(t).clone() for t in (c.k_min, c.k_max)] if c.k_min is not None else None
    q_in, k_in, v_in = q.cpu(), k.cpu(), v.cpu()
    q_out = q if in_place else torch.full((T, Hq, d), 3.0, dtype=x, device="cuda")
    r = pkg.attn_paged_append(c.kv, k, v, q=q, q_out=q_out, token_start=start, cos=cos, sin=sin, interleaved=interleaved)
    assert r is q_out
    assert pkg.sync_status() == 0
    cos, sin = (cos.cpu(), sin.cpu()) if rot else (None, None)
    kc, vc = _raw(c.k).cpu(), _raw(c.v).cpu()
    touched = torch.zeros(c.k.shape[0], page, dtype=torch.bool)
    for b, n in enumerate(new):
        t, s = c.lens_list[b], sum(new[:b])
        if t == 0:
            assert torch.equal(q_out[s:s + n].cpu(), q_in[s:s + n] if in_place else torch.full_like(q_in[s:s + n], 3.0))
            continue
        pos = torch.arange(t - n, t)
        ids = c.table[b, pos // page].long()
        touched[ids, pos % page] = True
        y, mag = _rotated(q_in[s:s + n], pos, cos, sin, interleaved)
        _near(q_out[s:s + n].cpu(), y, mag, x)
        y, mag = _rotated(k_in[s:s + n], pos, cos, sin, interleaved)
        got = kc[ids, :, pos % page]
        _near(got.view(c.dtype), y, mag, c.dtype, c.scales[0])
        c.k_ref[b, :, pos] = got.view(c.dtype).double().transpose(0, 1) * c.scales[0]
        got = vc[ids, :, pos % page]
        _near(got.view(c.dtype), v_in[s:s + n].double(), v_in[s:s + n].double().abs(), c.dtype, c.scales[1])
        c.v_ref[b, :, pos] = got.view(c.dtype).double().transpose(0, 1) * c.scales[1]
    rest = ~touched[:, None, :, None].expand(c.k.shape)
    for got, old in ((kc, before[0].cpu()), (vc, before[1].cpu())):  # NaN included, bit for bit
        assert torch.equal(got.view(torch.uint8 if c.dtype == E4M3 else torch.int16)[rest],
                           old.view(torch.uint8 if c.dtype == E4M3 else torch.int16)[rest])
    tail = slice(sum(new), T)
    assert torch.equal(q_out[tail].cpu(), q_in[tail] if in_place else torch.full_like(q_in[tail], 3.0))
    if sums is not None:
        want = [t.cpu().view(c.dtype).float() for t in sums]
        for b, n in enumerate(new):
            t = c.lens_list[b]
            for j in range((t - n) // page, -(-t // page)) if t and n else ():
                id, first = int(c.table[b, j]), max(t - n, j * page)
                x_ = c.kv.k_pages[id].cpu().float()[:, first - j * page:min(page, t - j * page)]
                lo, hi = x_.amin(1), x_.amax(1)
                fresh = first == j * page
                want[0][id] = lo if fresh else torch.minimum(lo, want[0][id])
                want[1][id] = hi if fresh else torch.maximum(hi, want[1][id])
        assert torch.equal(c.k_min.cpu().float(), want[0]) and torch.equal(c.k_max.cpu().float(), want[1])


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("x,dtype,scales", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_prompts(pkg, x, dtype, scales, d, interleaved):
    new = [1, 33, 0, 16, 17, 100, 15, 2]
    lens = [1, 33, 50, 48, 30, 117, 47, 40]
    c = Case(pkg, lens, H=2, d=d, dtype=dtype, scales=scales, seed=d, summaries=True)
    _check_append(pkg, c, new, x, interleaved=interleaved, pad=5)


@pytest.mark.parametrize("x,dtype,scales", TYPES)
def test_append_single_tokens(pkg, x, dtype, scales):
    lens = [1, 0, 16, 17, 100, 0]
    for summaries in (False, True):
        c = Case(pkg, lens, H=3, d=64, dtype=dtype, scales=scales, seed=3, summaries=summaries)
        _check_append(pkg, c, [1] * 6, x, Hq=9, single=True)


@pytest.mark.parametrize("page", [8, 24, 64, 1024])
@pytest.mark.parametrize("layout", ["heads", "tokens", "turns"])
@pytest.mark.parametrize("summaries", [False, True])
def test_append_pages_and_layouts(pkg, page, layout, summaries):
    new = [page, page + 1, 1, 2 * page + 3]
    lens = [page, 2 * page + 2, page + 1, 3 * page + 2]
    c = Case(pkg, lens, H=1, page=page, d=32, layout=layout, seed=page, summaries=summaries)
    _check_append(pkg, c, new, BF16, Hq=2)


@pytest.mark.parametrize("rot", [0, 16, 48, 64])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_rotates_a_part_of_the_channels(pkg, rot, interleaved):
    c = Case(pkg, [40, 9], H=2, d=64, seed=rot)
    _check_append(pkg, c, [21, 9], BF16, rot=rot, interleaved=interleaved)


def test_append_in_place(pkg):
    c = Case(pkg, [40, 0, 9], H=2, d=64, seed=2)
    _check_append(pkg, c, [21, 0, 9], BF16, in_place=True, pad=3)


def test_append_many_sequences(pkg):
    g = torch.Generator().manual_seed(1)
    new = [int(x) for x in torch.randint(0, 20, (300,), generator=g)]
    lens = [n + int(x) if n else 0 for n, x in zip(new, torch.randint(0, 40, (300,), generator=g))]
    c = Case(pkg, lens, H=1, d=32, page=8, seed=1, summaries=True)
    _check_append(pkg, c, new, BF16, Hq=1)


def test_append_far_positions(pkg):
    """Angles of far positions come from the tables; only they limit the position."""
    c = Case(pkg, [100000], H=1, d=64, page=64, seed=1, fill=False)
    _check_append(pkg, c, [70], BF16)


def test_append_saturates_and_keeps_nan(pkg):
    c = Case(pkg, [4], H=1, d=32, dtype=E4M3, seed=1, scales=(0.5, 0.25), summaries=True)
    x = torch.zeros(4, 1, 32, dtype=BF16, device="cuda")
    x[0], x[1], x[2, :, ::2] = 1e4, -1e4, math.nan
    pkg.attn_paged_append(c.kv, x, x, token_start=torch.tensor([0, 4], dtype=torch.int32, device="cuda"))
    assert pkg.sync_status() == 0
    k = c.k[int(c.table[0, 0])].float().cpu()[0, :4]
    assert (k[0] == 448).all() and (k[1] == -448).all() and k[2, ::2].isnan().all() and (k[3] == 0).all()
    assert (c.k_max[int(c.table[0, 0])].float() == 448).all() and (c.k_min[int(c.table[0, 0])].float() == -448).all()


def test_append_bad_tables_write_nothing(pkg):
    c = Case(pkg, [20, 20], H=1, d=32, seed=1)
    k = torch.ones(2, 1, 32, dtype=BF16, device="cuda")
    before = (c.k.clone(), c.v.clone())
    same = lambda: all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip((c.k, c.v), before))  # noqa: E731
    c.block_table[:, 1] = torch.tensor([-3, c.k.shape[0]], dtype=torch.int32)
    pkg.attn_paged_append(c.kv, k, k)
    assert pkg.sync_status() == 6 and same()
    for bad in ([0, 2, 1], [-1, 0, 2], [0, 0, 3], [2, 2, 1]):
        pkg.attn_paged_append(c.kv, k, k, token_start=torch.tensor(bad, dtype=torch.int32, device="cuda"))
        assert pkg.sync_status() == 6 and same(), bad
    c.block_table.copy_(c.table)
    cos, sin = pkg.rotation_tables(19, 32, device="cuda")  # one position short
    pkg.attn_paged_append(c.kv, k, k, cos=cos, sin=sin)
    assert pkg.sync_status() == 6 and same()
    c.seq_lens.fill_(1 << 28)
    pkg.attn_paged_append(c.kv, k, k)
    assert pkg.sync_status() == 6 and same()


def test_append_of_nothing(pkg):
    c = Case(pkg, [20], H=1, d=32, seed=1)
    k = torch.empty(0, 1, 32, dtype=BF16, device="cuda")
    assert pkg.attn_paged_append(c.kv, k, k, token_start=torch.zeros(2, dtype=torch.int32, device="cuda")) is None
    assert pkg.last_launch_count() == 0 and pkg.sync_status() == 0


# ------------------------------------------------------------------ selection

def _chosen(c, q, n, first, last):
    """The definition in float64 on the CPU: [B][H] ascending page lists."""
    B, Hq, d = q.shape
    G, out = Hq // c.H, []
    lo, hi = c.k_min.cpu().double(), c.k_max.cpu().double()
    for b, t in enumerate(c.lens_list):
        used, rows = -(-t // c.page), []
        for h in range(c.H):
            ids = c.table[b, :used].long()
            x = q[b, h * G:(h + 1) * G].double()[:, None]
            s = torch.maximum(x * lo[ids, h], x * hi[ids, h]).sum(-1).amax(0) if used else torch.zeros(0)
            order = sorted(range(used), key=lambda j: (not (j < first or j >= used - last), -float(s[j]), j))
            rows.append(sorted(order[:n]))
        out.append(rows)
    return out


def _check_select(pkg, c, q, n, first=1, last=1):
    pages = pkg.attn_paged_select(c.kv, q.cuda(), n, keep_first=first, keep_last=last)
    assert pkg.sync_status() == 0
    want = _chosen(c, q, n, first, last)
    full = torch.full((len(c.lens_list), c.H, n), -1, dtype=torch.int32)
    for b, rows in enumerate(want):
        for h, row in enumerate(rows):
            full[b, h, :len(row)] = torch.tensor(row, dtype=torch.int32)
    assert torch.equal(pages.cpu(), full)
    return pages, want


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("x,dtype,scales", TYPES)
def test_select_and_decode(pkg, x, dtype, scales, d):
    lens = [0, 1, 16 * 12, 16 * 12 + 1, 16 * 13, 1003, 2500]
    c = Case(pkg, lens, H=2, d=d, dtype=dtype, scales=scales, seed=d + 1, summaries=True)
    q = c.randn(len(lens), 6, d, dtype=x)
    pages, want = _check_select(pkg, c, q, 12)
    keys = [[[p * 16 + i for p in row for i in range(16) if p * 16 + i < lens[b]] for row in rows]
            for b, rows in enumerate(want)]
    _check_decode(pkg, c, q, pages=pages, keys=keys)


@pytest.mark.parametrize("n,first,last", [(1, 0, 0), (1, 0, 1), (1, 1, 0), (2, 1, 1), (8, 4, 4), (31, 0, 0), (32, 0, 0),
                                          (100, 3, 1), (700, 1, 1), (5000, 0, 0)])
def test_select_counts(pkg, n, first, last):
    c = Case(pkg, [8 * 31 + 3, 8 * 2000, 5], H=1, page=8, d=32, seed=n, summaries=True)
    _check_select(pkg, c, c.randn(3, 5, 32), n, first, last)


@pytest.mark.parametrize("group", [1, 4, 8, 16, 17, 40])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_select_group_sizes(pkg, group, dtype):
    c = Case(pkg, [3000, 700], H=2, d=64, dtype=dtype, seed=group, summaries=True, scales=(0.02, 0.02))
    _check_select(pkg, c, c.randn(2, 2 * group, 64), 20)


def test_select_more_pages_than_a_block_has_threads(pkg):
    c = Case(pkg, [8 * 9001], H=1, page=8, d=32, seed=1, summaries=True)
    _check_select(pkg, c, c.randn(1, 4, 32), 333)


def test_select_ties_go_to_the_lowest_page(pkg):
    c = Case(pkg, [16 * 500], H=2, d=64, seed=1, summaries=True)
    q = c.randn(1, 4, 64)
    for t in (c.k_min, c.k_max):
        t.zero_()
    _check_select(pkg, c, q, 37)                 # every score is 0
    some = torch.randint(0, 4, (c.k.shape[0],), generator=c.g)
    kinds = torch.randn(4, 2, 64, generator=c.g).to(BF16)
    c.k_min.copy_(kinds[some])
    c.k_max.copy_(kinds[some])                   # four scores, each some hundred times
    for n in (3, 100, 250, 499):
        _check_select(pkg, c, q, n)


def test_select_orders_scores_that_fp32_cannot_tell_apart(pkg):
    """One large channel, the same on every page, and small ones that differ below its fp32 step."""
    d, n = 64, 400
    c = Case(pkg, [16 * n], H=1, d=d, seed=1, summaries=True)
    q = torch.ones(1, 2, d, dtype=BF16)
    lo = torch.zeros(c.k.shape[0], 1, d, dtype=BF16)
    lo[..., 0] = 2.0 ** 13
    lo[..., 1:] = (torch.randint(-8, 9, lo[..., 1:].shape, generator=c.g) * 2.0 ** -16).to(BF16)
    c.k_min.copy_(lo)
    c.k_max.copy_(lo)
    for m in (2, 50, 200, 399):
        _check_select(pkg, c, q, m)


def test_select_cancelling_sums(pkg):
    """Channels of opposite sign that cancel to a small score, in an order that a rounded sum would mistake."""
    c = Case(pkg, [16 * 600], H=1, d=128, seed=3, summaries=True)
    q = c.randn(1, 3, 128) * 8
    big = (torch.randn(c.k.shape[0], 1, 128, generator=c.g) * 100).to(BF16)
    c.k_min.copy_(big)
    c.k_max.copy_(big)
    for m in (2, 77, 300):
        _check_select(pkg, c, q, m)


def test_select_is_not_confused_by_bad_pages(pkg):
    c = Case(pkg, [16 * 40], H=1, d=32, seed=1, summaries=True)
    c.block_table[0, 7] = -1
    pages = pkg.attn_paged_select(c.kv, c.randn(1, 2, 32).cuda(), 10)
    assert pkg.sync_status() == 6
    p = pages.cpu()[0, 0].tolist()
    assert p == sorted(set(p)) and 0 <= p[0] and p[-1] < 40 and 7 not in p


def test_decode_any_list_of_pages(pkg):
    """Lists need not come from the selection: any order, gaps, indices behind the end."""
    c = Case(pkg, [16 * 20 + 5, 30], H=2, d=64, seed=1)
    q = c.randn(2, 4, 64)
    lists = torch.tensor([[[20, -1, 3, 7, 0, -1], [5, 21, 19, 1000, -7, 2]], [[-1] * 6, [1, 2, -1, -1, -1, -1]]],
                         dtype=torch.int32)
    keys = [[[p * 16 + i for p in row if p >= 0 for i in range(16) if p * 16 + i < c.lens_list[b]]
             for row in rows.tolist()] for b, rows in enumerate(lists)]
    _check_decode(pkg, c, q, pages=lists.cuda(), keys=keys)


@pytest.mark.parametrize("x,dtype,scales", TYPES)
@pytest.mark.parametrize("longest", [1, 60, 128, 256])
def test_many_short_sequences(pkg, x, dtype, scales, longest):
    """More items than warps, each a few tiles: a warp takes an item for itself."""
    g = torch.Generator().manual_seed(longest)
    lens = [int(v) for v in torch.randint(0, longest + 1, (230,), generator=g)]
    for d, heads, Hq in ((64, 16, 32), (128, 8, 96)):
        c = Case(pkg, lens, H=heads, d=d, dtype=dtype, scales=scales, seed=longest)
        _check_decode(pkg, c, c.randn(len(lens), Hq, d, dtype=x))


@pytest.mark.parametrize("per_sm", [1, 2, 3, 4])
@pytest.mark.parametrize("more", [-1, 0, 1, 30])
@pytest.mark.parametrize("longest", [100, 400])
def test_about_as_many_items_as_blocks(pkg, per_sm, more, longest):
    """Items a little fewer and more than the blocks that the GPU holds at one, two, three and four per SM, under a
    wide table, all with tokens and some without."""
    g = torch.Generator().manual_seed(per_sm)
    n = per_sm * torch.cuda.get_device_properties(0).multi_processor_count + more
    lens = [1 + int(v) for v in torch.randint(0, longest, (n,), generator=g)]
    c = Case(pkg, lens, H=1, page=64, d=128, seed=1, width=200)
    q = c.randn(n, 2, 128)
    _check_decode(pkg, c, q)
    for b in (0, n // 2, n - 1):
        c.lens_list[b] = 0
    c.seq_lens.copy_(torch.tensor(c.lens_list, dtype=torch.int32))
    _check_decode(pkg, c, q)


def test_many_short_sequences_through_lists(pkg):
    lens = [i % 40 for i in range(200)]
    c = Case(pkg, lens, H=16, page=8, d=32, dtype=F16, seed=1, summaries=True)
    q = c.randn(200, 32, 32)
    pages, want = _check_select(pkg, c, q, 3)
    keys = [[[p * 8 + i for p in row for i in range(8) if p * 8 + i < lens[b]] for row in rows] for b, rows in enumerate(want)]
    _check_decode(pkg, c, q, pages=pages, keys=keys)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("seed", range(24))
def test_drawn_calls_are_right_and_repeat_bit_for_bit(pkg, seed):
    g = torch.Generator().manual_seed(1000 + seed)

    def pick(*of):
        return of[int(torch.randint(0, len(of), (1,), generator=g))]

    x, dtype, scales = pick(*TYPES)
    B, H, G, n = pick(1, 5, 40, 200, 400), pick(1, 2, 8), pick(1, 4, 16, 20), pick(2, 7, 32)
    top = pick(20, 130, 600) if B * H < 1000 else pick(5, 30, 60)
    lens = [int(v) for v in torch.randint(0, top + 1, (B,), generator=g)]
    c = Case(pkg, lens, H=H, page=pick(8, 16, 64), d=pick(32, 64, 128), dtype=dtype, scales=scales, seed=seed,
             width=pick(None, 80), summaries=True, layout=pick("heads", "tokens", "turns"))
    q = c.randn(B, H * G, c.d, dtype=x).cuda()
    o, lse = _check_decode(pkg, c, q)
    pages = pkg.attn_paged_select(c.kv, q, n)
    first = pkg.attn_paged_decode(c.kv, q, pages=pages)
    for _ in range(10):
        again = pkg.attn_paged_decode(c.kv, q)
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)
        listed = pkg.attn_paged_select(c.kv, q, n)
        again = pkg.attn_paged_decode(c.kv, q, pages=listed)
        assert torch.equal(listed, pages) and torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    assert pkg.sync_status() == 0


def test_a_server_run(pkg):
    """Prompts appended, then steps of append, select and decode, with a sequence that starts late and one that ends;
    against float64 over what the cache holds, and the prompt's last token against the dense causal forward."""
    H, Hq, d, page, B = 2, 8, 64, 16, 3
    prompts, steps = [37, 0, 90], 6
    final = [n + steps if n else 2 for n in prompts]
    c = Case(pkg, final, H=H, d=d, page=page, seed=1, summaries=True, fill=False)
    cos, sin = pkg.rotation_tables(256, d, device="cuda")
    # prompts
    T = sum(prompts)
    q, k, v = (c.randn(T, h, d).cuda() for h in (Hq, H, H))
    start = torch.tensor([0, 37, 37, 127], dtype=torch.int32, device="cuda")
    c.seq_lens.copy_(torch.tensor(prompts, dtype=torch.int32))
    qr = pkg.attn_paged_append(c.kv, k, v, q=q, token_start=start, cos=cos, sin=sin)
    c.lens_list = list(prompts)

    def read_back():
        for b, t in enumerate(c.lens_list):
            pos = torch.arange(t)
            ids = c.table[b, pos // page].long()
            c.k_ref[b, :, :t] = c.k.cpu()[ids, :, pos % page].double().transpose(0, 1)
            c.v_ref[b, :, :t] = c.v.cpu()[ids, :, pos % page].double().transpose(0, 1)
    read_back()
    last = torch.stack([qr[36], qr[36], qr[126]])
    o, lse = _check_decode(pkg, c, last)
    dense_k = c.k_ref[2, :, :90].to(BF16).repeat_interleave(4, 0)[None].cuda()
    dense_v = c.v_ref[2, :, :90].to(BF16).repeat_interleave(4, 0)[None].cuda()
    of, lf = pkg.attn_fwd(qr[37:].transpose(0, 1).contiguous()[None], dense_k, dense_v, causal=True)
    assert (of[0, :, 89].float() - o[2].float()).abs().max() <= 2e-2
    assert (lf[0, :, 89] - lse[2]).abs().max() <= 1e-3
    # steps
    for s in range(steps):
        c.lens_list = [37 + s + 1, max(0, s - steps + 3), 90 + s + 1 if s < 4 else 0]
        c.seq_lens.copy_(torch.tensor(c.lens_list, dtype=torch.int32))
        q, k, v = (c.randn(B, h, d).cuda() for h in (Hq, H, H))
        qr = pkg.attn_paged_append(c.kv, k, v, q=q, cos=cos, sin=sin)
        qr[torch.tensor(c.lens_list) == 0] = 0
        pages = pkg.attn_paged_select(c.kv, qr, 3)
        assert pkg.sync_status() == 0
        read_back()
        want = _chosen(c, qr.cpu(), 3, 1, 1)
        assert [[[p for p in row if p >= 0] for row in rows] for rows in pages.tolist()] == want
        _check_decode(pkg, c, qr)
        keys = [[[p * page + i for p in row for i in range(page) if p * page + i < c.lens_list[b]] for row in rows]
                for b, rows in enumerate(want)]
        _check_decode(pkg, c, qr, pages=pages, keys=keys)


def _step(pkg, c, q, k, v, cos, sin, n):
    qr = pkg.attn_paged_append(c.kv, k, v, q=q, cos=cos, sin=sin)
    pages = pkg.attn_paged_select(c.kv, qr, n)
    return (qr, pages) + pkg.attn_paged_decode(c.kv, qr) + pkg.attn_paged_decode(c.kv, qr, pages=pages)


def test_captured_step_replays_with_other_lengths(pkg):
    lens = [200, 60, 333]
    c = Case(pkg, lens, H=2, d=64, seed=1, summaries=True, width=40)
    q, k, v = (c.randn(3, h, 64).cuda() for h in (4, 2, 2))
    cos, sin = pkg.rotation_tables(1024, 64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(pkg, c, q, k, v, cos, sin, 5)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):  # two graphs of the same step, replayed in turns
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(_step(pkg, c, q, k, v, cos, sin, 5))
        graphs.append(graph)
    for now in ([200, 60, 333], [16, 0, 170], [1, 64, 300]):
        c.seq_lens.copy_(torch.tensor(now, dtype=torch.int32))
        eager = [t.clone() for t in _step(pkg, c, q, k, v, cos, sin, 5)]
        for graph, out in zip(graphs, outs):
            out[2].fill_(5.0)
            graph.replay()
            torch.cuda.synchronize()
            live = [b for b, n in enumerate(now) if n]
            for got, want in zip(out, eager):  # bit for bit: 64 tokens reach slots that nothing filled, and are NaN
                bits = {2: torch.int16, 4: torch.int32}[got.element_size()]
                assert torch.equal(got[live].view(bits), want[live].view(bits))
    assert pkg.sync_status() == 0


def test_two_streams_at_once(pkg):
    cases = [Case(pkg, [900 + i, 33, 0, 2047], H=2, d=128, seed=i, summaries=True) for i in range(2)]
    qs = [c.randn(4, 8, 128).cuda() for c in cases]
    want = [(pkg.attn_paged_select(c.kv, q, 7),) + pkg.attn_paged_decode(c.kv, q) for c, q in zip(cases, qs)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (c, q, s) in enumerate(zip(cases, qs, streams)):
            got[i].append((pkg.attn_paged_select(c.kv, q, 7, stream=s),) + pkg.attn_paged_decode(c.kv, q, stream=s))
    torch.cuda.synchronize()
    assert pkg.sync_status() == 0
    for g, w in zip(got, want):
        for r in g:
            assert all(torch.equal(a, b) for a, b in zip(r, w))


@pytest.mark.parametrize("x,dtype,scales", TYPES)
def test_decode_many_turns_of_the_ring(pkg, x, dtype, scales):
    """Shares of some tens of tiles per CTA, cut items and lengths that end inside tiles and pages."""
    g = torch.Generator().manual_seed(5)
    lens = [2500] + [int(v) for v in torch.randint(0, 2500, (60,), generator=g)] + [0, 0, 0]
    c = Case(pkg, lens, H=8, d=128, dtype=dtype, scales=scales, seed=5)
    for _ in range(3):
        _check_decode(pkg, c, c.randn(len(lens), 16, 128, dtype=x))


# ------------------------------------------------------------------ the binding's own checks

def test_the_binding_refuses(pkg):
    c = Case(pkg, [20, 3], H=2, d=64, summaries=True, seed=1)
    q, k = c.randn(2, 4, 64).cuda(), c.randn(2, 2, 64).cuda()
    cos, sin = pkg.rotation_tables(64, 64, device="cuda")
    start = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    before = (c.k.clone(), c.v.clone())
    app, dec, sel = pkg.attn_paged_append, pkg.attn_paged_decode, pkg.attn_paged_select
    wrong = [
        (TypeError, lambda: dec(c.kv, q.cpu())), (TypeError, lambda: dec(c.kv, q.half())), (TypeError, lambda: dec(c.kv, q.float())),
        (TypeError, lambda: dec(c.kv, None)), (TypeError, lambda: dec(None, q)), (ValueError, lambda: dec(c.kv, q[:1])),
        (ValueError, lambda: dec(c.kv, q[..., :32])), (ValueError, lambda: dec(c.kv, q[:, 0])),
        (ValueError, lambda: dec(c.kv, q.transpose(1, 2).contiguous().transpose(1, 2))),
        (pkg.AttnError, lambda: dec(c.kv, q[:, :3])), (pkg.AttnError, lambda: dec(c.kv, q, scale=math.inf)),
        (TypeError, lambda: dec(c.kv, q, scale="x")), (ValueError, lambda: dec(c.kv, q, o=torch.empty(2, 4, 32, dtype=BF16, device="cuda"))),
        (TypeError, lambda: dec(c.kv, q, o=torch.empty(2, 4, 64, device="cuda"))), (pkg.AttnError, lambda: dec(c.kv, q, o=q)),
        (ValueError, lambda: dec(c.kv, q, lse=torch.empty(2, 3, device="cuda"))), (TypeError, lambda: dec(c.kv, q, lse=q)),
        (ValueError, lambda: dec(c.kv, q, pages=torch.zeros(2, 2, 0, dtype=torch.int32, device="cuda"))),
        (ValueError, lambda: dec(c.kv, q, pages=torch.zeros(2, 1, 3, dtype=torch.int32, device="cuda"))),
        (ValueError, lambda: dec(c.kv, q, pages=torch.zeros(2, 2, 3, dtype=torch.int64, device="cuda"))),
        (TypeError, lambda: dec(c.kv, q, pages=[0])),
        (ValueError, lambda: sel(c.kv, q, 0)), (ValueError, lambda: sel(c.kv, q, 1)), (ValueError, lambda: sel(c.kv, q, 4, keep_first=-1)),
        (ValueError, lambda: sel(c.kv, q, 4, pages=torch.zeros(2, 2, 3, dtype=torch.int32, device="cuda"))),
        (ValueError, lambda: sel(pkg.PagedKV(c.k, c.v, c.block_table, c.seq_lens), q, 4)), (TypeError, lambda: sel(c.kv, q, "x")),
        (TypeError, lambda: app(c.kv, k, k.half())), (TypeError, lambda: app(c.kv, k.half(), k.half())), (ValueError, lambda: app(c.kv, q, q)),
        (ValueError, lambda: app(c.kv, k[:1], k[:1])), (ValueError, lambda: app(c.kv, k, k, token_start=start[:2])),
        (ValueError, lambda: app(c.kv, k, k, token_start=start.long())), (ValueError, lambda: app(c.kv, k, k, cos=cos)),
        (TypeError, lambda: app(c.kv, k, k, cos=cos.half(), sin=sin.half())), (ValueError, lambda: app(c.kv, k, k, cos=cos, sin=sin[:3])),
        (pkg.AttnError, lambda: app(c.kv, k, k, cos=cos[:, :4].contiguous(), sin=sin[:, :4].contiguous())),
        (ValueError, lambda: app(c.kv, k, k, q_out=q)), (ValueError, lambda: app(c.kv, k, k, q=q[:1], token_start=start)),
        (pkg.AttnError, lambda: app(c.kv, k, k, q=q, q_out=torch.empty(8, 4, 64, dtype=BF16, device="cuda")[::1][:1].expand(2, 4, 64))),
    ]
    for i, (error, call) in enumerate(wrong):
        with pytest.raises(error):
            call()
            pytest.fail("call %d was taken" % i)
    assert pkg.sync_status() == 0
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip((c.k, c.v), before))


def test_calls_on_a_side_stream_allocate_there(pkg):
    """Outputs and workspace of a call with a stream come from that stream's pool, and the current stream stays."""
    c = Case(pkg, [500, 30], H=2, d=64, summaries=True, seed=2)
    q = c.randn(2, 4, 64).cuda()
    want = pkg.attn_paged_decode(c.kv, q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    here = torch.cuda.current_stream()
    got = pkg.attn_paged_decode(c.kv, q, stream=side)
    assert torch.cuda.current_stream() == here
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert pkg.sync_status() == 0


@pytest.mark.parametrize("x,dtype,scales", TYPES)
@pytest.mark.parametrize("B,longest,d", [(1, 1000, 128), (1, 500, 64), (3, 250, 128), (5, 120, 32), (16, 200, 128), (2, 30, 64)])
def test_short_items_in_clusters(pkg, x, dtype, scales, B, longest, d):
    """Tables as wide as the longest sequence: an item goes to 1, 2, 4 or 8 CTAs, some of them without a tile."""
    g = torch.Generator().manual_seed(B)
    lens = [longest] + [int(v) for v in torch.randint(0, longest + 1, (B - 1,), generator=g)]
    c = Case(pkg, lens, H=4, d=d, dtype=dtype, scales=scales, seed=B, width=-(-longest // 16))
    _check_decode(pkg, c, c.randn(B, 12, d, dtype=x))
    _check_decode(pkg, c, c.randn(B, 44, d, dtype=x))
    c.lens_list = [0] * B
    c.seq_lens.zero_()
    _check_decode(pkg, c, c.randn(B, 12, d, dtype=x))


# ------------------------------------------------------------------ what the documentation allows and is easily forgotten

def test_sequences_share_pages(pkg):
    """A common prefix stands in the cache once."""
    c = Case(pkg, [100, 90, 70], H=2, d=64, seed=1)
    for b, n in ((1, 4), (2, 3)):  # whole pages of sequence 0
        c.block_table[b, :n] = c.block_table[0, :n]
        c.k_ref[b, :, :n * 16], c.v_ref[b, :, :n * 16] = c.k_ref[0, :, :n * 16], c.v_ref[0, :, :n * 16]
    _check_decode(pkg, c, c.randn(3, 4, 64))


def test_thousands_of_sequences(pkg):
    g = torch.Generator().manual_seed(1)
    lens = [int(v) for v in torch.randint(0, 20, (3000,), generator=g)]
    c = Case(pkg, lens, H=1, page=8, d=32, seed=1, summaries=True)
    _check_decode(pkg, c, c.randn(3000, 2, 32))
    _check_select(pkg, c, c.randn(3000, 2, 32), 2)
    c = Case(pkg, lens, H=1, page=8, d=32, seed=1, summaries=True)
    _check_append(pkg, c, [1] * 3000, BF16, Hq=2, single=True)
    c = Case(pkg, lens, H=1, page=8, d=32, seed=1)
    _check_append(pkg, c, [n // 2 for n in lens], BF16, Hq=2)


def test_rows_before_the_first_sequence_are_padding(pkg):
    c = Case(pkg, [9, 30], H=1, d=32, seed=1, fill=False)
    k, v, q = c.randn(20, 1, 32).cuda(), c.randn(20, 1, 32).cuda(), c.randn(20, 2, 32).cuda()
    out = torch.full((20, 2, 32), 3.0, dtype=BF16, device="cuda")
    pkg.attn_paged_append(c.kv, k, v, q=q, q_out=out, token_start=torch.tensor([5, 7, 17], dtype=torch.int32, device="cuda"))
    assert pkg.sync_status() == 0
    assert (out[:5] == 3).all() and (out[17:] == 3).all() and torch.equal(out[5:17], q[5:17])
    for b, (rows, first) in enumerate(((range(5, 7), 7), (range(7, 17), 20))):
        for i, r in enumerate(rows):
            pos = first + i
            assert torch.equal(c.k[int(c.table[b, pos // 16]), :, pos % 16], k[r])
            assert torch.equal(c.v[int(c.table[b, pos // 16]), :, pos % 16], v[r])


def test_append_past_32_bit_offsets(pkg):
    d, page, H = 128, 64, 4
    P = (5 << 30) // (H * page * d * 2)
    k = torch.zeros((P, H, page, d), dtype=BF16, device="cuda")
    v = torch.zeros((P, H, page, d), dtype=BF16, device="cuda")
    table = torch.tensor([[P - 1, P - 2]], dtype=torch.int32, device="cuda")
    kv = pkg.PagedKV(k, v, table, torch.tensor([100], dtype=torch.int32, device="cuda"))
    x = torch.randn(100, 2 * H, d, device="cuda").to(BF16)
    pkg.attn_paged_append(kv, x[:, :H], x[:, H:], token_start=torch.tensor([0, 100], dtype=torch.int32, device="cuda"))
    assert pkg.sync_status() == 0
    for pages, new in ((k, x[:, :H]), (v, x[:, H:])):
        assert torch.equal(pages[P - 1].transpose(0, 1), new[:64]) and torch.equal(pages[P - 2, :, :36].transpose(0, 1), new[64:])
        assert (pages[P - 2, :, 36:] == 0).all() and (pages[:P - 2].view(torch.int16) != 0).sum() == 0


@pytest.mark.parametrize("pages", [3000, 9000])
def test_select_more_ties_than_shared_memory_holds(pkg, pages):
    c = Case(pkg, [8 * pages], H=1, page=8, d=32, seed=1, summaries=True)
    q = c.randn(1, 3, 32)
    c.k_min.zero_()
    c.k_max.zero_()
    _check_select(pkg, c, q, 37)
    kinds = torch.randn(2, 1, 32, generator=c.g).to(BF16)
    some = kinds[torch.randint(0, 2, (c.k.shape[0],), generator=c.g)]
    c.k_min.copy_(some)
    c.k_max.copy_(some)
    for n in (5, pages // 3, pages - 100):
        _check_select(pkg, c, q, n)


def test_select_scores_beyond_fp32(pkg):
    """Sums that overflow fp32, or vanish in it, are ordered all the same."""
    for power, scale in ((100, 100), (-100, -60)):
        c = Case(pkg, [16 * 1500], H=1, d=64, seed=2, summaries=True)
        q = (c.randn(1, 4, 64).float() * 2.0 ** power).to(BF16)
        for t in (c.k_min, c.k_max):
            t.copy_((t.float() * 2.0 ** scale).to(BF16))
        _check_select(pkg, c, q, 70)


def test_select_takes_nan_and_infinite_scores_first(pkg):
    c = Case(pkg, [16 * 300], H=1, d=32, seed=3, summaries=True)
    q = c.randn(1, 2, 32)
    ids = c.table[0].long()
    c.k_max[ids[50], 0, 4] = math.nan
    c.k_min[ids[50], 0, 4] = math.nan
    c.k_max[ids[70]] = math.inf
    c.k_min[ids[70]] = -math.inf
    got = pkg.attn_paged_select(c.kv, q.cuda(), 2, keep_first=0, keep_last=0)
    assert pkg.sync_status() == 0 and got[0, 0].tolist() == [50, 70]
    got = pkg.attn_paged_select(c.kv, q.cuda(), 12, keep_first=1, keep_last=1)[0, 0].tolist()
    assert pkg.sync_status() == 0 and {0, 50, 70, 299} <= set(got) and got == sorted(set(got))


def test_select_with_hardly_a_page_in_the_table(pkg):
    c = Case(pkg, [16 * 100], H=2, d=32, seed=4, summaries=True)
    good = [3, 60, 61]
    for j in range(100):
        if j not in good:
            c.block_table[0, j] = -1
    got = pkg.attn_paged_select(c.kv, c.randn(1, 4, 32).cuda(), 10)
    assert pkg.sync_status() == 6
    for row in got[0].tolist():
        assert row == sorted(set(row)) and row[0] == 0 and row[-1] == 99 and set(good) <= set(row)


def test_nan_queries_give_nan(pkg):
    """A NaN in a query is not an empty sequence."""
    for lens in ([100], [40000], [3] * 700):
        c = Case(pkg, lens, H=1, d=32, seed=5)
        q = c.randn(len(lens), 2, 32).cuda()
        q[:, 1, 7] = math.nan
        o, lse = pkg.attn_paged_decode(c.kv, q)
        assert pkg.sync_status() == 0
        assert o[:, 1].isnan().all() and lse[:, 1].isnan().all() and o[:, 0].isfinite().all() and lse[:, 0].isfinite().all()


def test_two_threads_at_once(pkg):
    import threading
    cases = [Case(pkg, [900 + i, 33, 2047], H=2, d=64, seed=i, summaries=True) for i in range(4)]
    qs = [c.randn(3, 8, 64).cuda() for c in cases]
    want = [(pkg.attn_paged_select(c.kv, q, 7),) + pkg.attn_paged_decode(c.kv, q) for c, q in zip(cases, qs)]
    torch.cuda.synchronize()
    wrong = []

    def work(c, q, w):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(30):
                got = (pkg.attn_paged_select(c.kv, q, 7),) + pkg.attn_paged_decode(c.kv, q)
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, w)):
                    wrong.append(c)
    threads = [threading.Thread(target=work, args=x) for x in zip(cases, qs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and pkg.sync_status() == 0


FIRST_CALL_IN_A_CAPTURE = """
import torch, sys
sys.path.insert(0, %r)
import io_aware_exact_12_gb300 as p
x = lambda *s: torch.randn(s, device="cuda").to(torch.bfloat16)
k, v, lo, hi, q, new = x(40, 2, 16, 64), x(40, 2, 16, 64), x(40, 2, 64) - 1, x(40, 2, 64) + 1, x(2, 4, 64), x(2, 2, 64)
kv = p.PagedKV(k, v, torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20), torch.tensor([300, 17], dtype=torch.int32, device="cuda"), k_min=lo, k_max=hi)
def step():
    p.attn_paged_append(kv, new, new)
    return p.attn_paged_decode(kv, q, pages=p.attn_paged_select(kv, q, 5)) + p.attn_paged_decode(kv, q)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = step()
g.replay()
torch.cuda.synchronize()
assert p.sync_status() == 0
assert all(torch.equal(a, b) for a, b in zip(out, step()))
print("ok")
"""


def test_first_call_of_a_process_in_a_capture(pkg):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_IN_A_CAPTURE % root], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr


@pytest.mark.parametrize("x,dtype,scales", TYPES)
@pytest.mark.parametrize("d", [32, 64, 128])
def test_one_item_in_hundreds_of_parts(pkg, x, dtype, scales, d):
    c = Case(pkg, [90001], H=1, page=64, d=d, dtype=dtype, scales=scales, seed=d)
    _check_decode(pkg, c, c.randn(1, 5, d, dtype=x))
    _check_decode(pkg, c, c.randn(1, 17, d, dtype=x))


# ------------------------------------------------------------------ lanes that part

@pytest.mark.parametrize("group,d", [(1, 32), (3, 32), (5, 32), (1, 64), (3, 64), (7, 128), (9, 32), (11, 64)])
@pytest.mark.parametrize("longest", [40, 250, 500])
def test_clusters_whose_warps_have_lanes_without_work(pkg, group, d, longest):
    """Rows that fill no warp in the join, CTAs without a tile, and a producer that waits for a stage: the barrier over the
    cluster comes behind all of them."""
    g = torch.Generator().manual_seed(group)
    lens = [longest, 0, 1] + [int(v) for v in torch.randint(0, longest + 1, (3,), generator=g)]
    c = Case(pkg, lens, H=2, d=d, seed=longest, width=-(-longest // 16))
    q = c.randn(len(lens), 2 * group, d).cuda()
    o, lse = _check_decode(pkg, c, q)
    for _ in range(20):
        again = pkg.attn_paged_decode(c.kv, q)
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    assert pkg.sync_status() == 0


# ------------------------------------------------------------------ small weights

@pytest.mark.parametrize("x,dtype,scales", [(BF16, BF16, (1.0, 1.0)), (F16, F16, (1.0, 1.0)), (BF16, E4M3, (1.0, 0.5)), (F16, E4M3, (1.0, 0.5))])
@pytest.mark.parametrize("above", [8.0, 12.0, 15.0, 16.5, 17.2, 17.5, 20.0])
@pytest.mark.parametrize("n,d", [(500, 64), (4000, 128), (70000, 64)])
def test_decode_one_key_far_above_the_others(pkg, x, dtype, scales, above, n, d):
    """A key that takes nearly all of the weight and whose value is 0 (an attention sink): O is what the others leave, so
    they must keep their bits, down to 2^-29 of the largest weight (20 in the exponent; fp16 weights with the largest at
    2^15 are normal numbers down to there)."""
    c = Case(pkg, [n], H=1, page=16, d=d, dtype=dtype, scales=scales, seed=1)
    q = c.randn(1, 4, d, dtype=x) * 0.03
    q[..., 0] = 1.0
    at = 77
    c.k_ref[0, 0, :n, 0] = 0.0
    c.k_ref[0, 0, at] = 0.0
    c.k_ref[0, 0, at, 0] = (torch.tensor(above * math.sqrt(d)).to(dtype)).double()
    c.v_ref[0, 0, at] = 0.0
    ids = c.table[0, :-(-n // 16)].long().cuda()
    slots = torch.arange(len(ids) * 16, device="cuda")
    live = slots < n
    for to, ref, s in ((c.k, c.k_ref, scales[0]), (c.v, c.v_ref, scales[1])):
        rows = (ref[0, 0, :n] / s).to(dtype).cuda()
        _raw(to)[ids[slots[live] // 16], 0, slots[live] % 16] = _raw(rows)
    assert (q[0].double() @ c.k_ref[0, 0, :n].T / math.sqrt(d)).sort(-1).values[:, -2].max() < 1.0
    _check_decode(pkg, c, q)


@pytest.mark.parametrize("dtype", [F16, E4M3])
@pytest.mark.parametrize("power", [3, 8, 12])
def test_decode_logits_far_from_zero(pkg, dtype, power):
    """All logits near +-2^power (and beyond 2^20 with fp16), where a shift of the exponent is a rounding of its own."""
    for sign in (1, -1):
        c = Case(pkg, [900], H=1, d=64, dtype=dtype, seed=power, scales=(1.0, 1.0))
        q = c.randn(1, 4, 64, dtype=F16) * 0.05
        q[..., 0] = 16.0
        kx = torch.tensor(sign * 2.0 ** min(power, 8))
        c.k_ref[0, 0, :900, 0] = kx.double()
        slots = torch.arange(900)
        _raw(c.k)[c.table[0, slots // 16].long().cuda(), 0, (slots % 16).cuda(), 0] = _raw(kx.to(dtype).reshape(1)).cuda()
        _check_decode(pkg, c, q, scale=2.0 ** (power - 4 - min(power, 8)))
        if dtype == F16:
            _check_decode(pkg, c, q, scale=2.0 ** (21 - 4 - min(power, 8)))


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("x,dtype,scales", TYPES)
@pytest.mark.parametrize("group", [2, 12])
def test_decode_weights_keep_more_than_16_bits(pkg, x, dtype, scales, d, group):
    """Values of alternating sign: O is a small difference, and a weight's error shows in it undivided.  With h the half step
    of a 16-bit word, a weight's first word is its rounding of p (1 - 2 h), off by h p at most, so the second has 3 h p at
    most and errs by 3 h^2 p; the rest of the tolerance is _reference's."""
    lens = [2, 4, 16, 64, 300, 3000]
    c = Case(pkg, lens, H=1, d=d, dtype=dtype, scales=scales, seed=d + group)
    for b, n in enumerate(lens):
        pos = torch.arange(n)
        sign = (1.0 - 2.0 * (pos % 2)).to(dtype)
        c.v_ref[b, 0, :n] = sign.double()[:, None] * scales[1]
        _raw(c.v)[c.table[b, pos // 16].long().cuda(), 0, (pos % 16).cuda()] = _raw(sign[:, None].expand(n, d).contiguous()).cuda()
    q = c.randn(len(lens), group, d, dtype=x)
    scale = 1 / math.sqrt(d)
    o, lse = _check_decode(pkg, c, q)
    eps, word = torch.finfo(x).eps / 2, torch.finfo(F16 if dtype == E4M3 else dtype).eps / 2
    for b, n in enumerate(lens):
        k, v, y = c.k_ref[b, 0, :n], c.v_ref[b, 0, :n], q[b].double()
        w = torch.softmax(scale * (y @ k.T), -1)
        dt = ((d + 8) * 2.0 ** -24 * scale * (y.abs() @ k.abs().T)).amax(-1, keepdim=True)
        want = w @ v
        tol = eps * want.abs() * (1 + 1e-3) + (3 * word ** 2 + 2 * dt + 2.0 ** -20) * (w @ v.abs() + want.abs())
        err = (o[b].double().cpu() - want).abs()
        assert (err <= tol).all(), "sequence of %d: off by %g of its tolerance" % (n, (err / tol).max())


# ------------------------------------------------------------------ 8-bit scales

@pytest.mark.parametrize("x", [BF16, F16])
@pytest.mark.parametrize("scale", [math.exp(0.37 * i - 3) for i in range(12)] + [448.0 / 3 * 2.0 ** -i for i in (9, 30)] + [1.9999 * 2.0 ** -83, 1e-25, 1e25,
                                   1.0, 2.0 ** -6, 7.0, 0.21875, 0.4375, 0.03, 448.0 / 3, 2.0 ** -126, 2.0 ** -127, 2.0 ** -140, 1.5 * 2.0 ** -133,
                                   2.0 ** 127, 3e38])
def test_append_stores_the_quotient_bit_for_bit(pkg, x, scale):
    """Every 16-bit value through each scale, against fp32 division."""
    d, n = 128, 512
    c = Case(pkg, [n], H=1, page=32, d=d, dtype=E4M3, scales=(scale, scale * 0.75), seed=1, fill=False)
    every = torch.arange(-32768, 32768).to(torch.int16).view(x).reshape(n, 1, d)
    back = every.flip(0).contiguous()
    pkg.attn_paged_append(c.kv, every.cuda(), back.cuda(), token_start=torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    assert pkg.sync_status() == 0
    pos = torch.arange(n)
    for cache, rows, s in ((c.k, every, scale), (c.v, back, scale * 0.75)):
        got = _raw(cache).cpu()[c.table[0, pos // 32].long(), :, pos % 32].view(E4M3)
        want = (rows.float() / torch.tensor(s, dtype=torch.float32)).clamp(-448, 448).to(E4M3)
        nan = want.float().isnan()
        assert torch.equal(got.float().isnan(), nan)
        assert torch.equal(_raw(got)[~nan], _raw(want)[~nan])


# ------------------------------------------------------------------ lists longer than their sequences

@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("page", [8, 16, 64])
def test_list_entries_past_the_number_of_pages_are_not_read(pkg, d, dtype, page):
    """As many entries count as the sequence has pages, whatever the tile that they lie in."""
    lens = [2 * page, 2 * page - 3, 1, 3 * page + 1, 0]
    c = Case(pkg, lens, H=1, page=page, d=d, dtype=dtype, seed=page, scales=(0.02, 0.03))
    lists = torch.tensor([[1, -1, 0, 0, 1, 1, 0, 0], [0, 1, 0, 1, 0, 1, 0, 1], [0, 0, 0, 0, 0, 0, 0, 0], [3, 0, 2, -1, 1, 1, 1, 1],
                          [0, 0, 0, 0, 0, 0, 0, 0]], dtype=torch.int32)[:, None]
    keys = []
    for n, row in zip(lens, lists[:, 0].tolist()):
        row = [p for p in row[:-(-n // page)] if p >= 0]
        keys.append([[p * page + i for p in row for i in range(page) if p * page + i < n]])
    _check_decode(pkg, c, c.randn(len(lens), 4, d), pages=lists.cuda(), keys=keys)


# ------------------------------------------------------------------ scores that differ in their last bits

@pytest.mark.parametrize("x,dtype,scales", TYPES)
@pytest.mark.parametrize("n,group", [(600, 1), (600, 6), (1500, 3)])
def test_select_equal_and_nearly_equal_sums_of_other_terms(pkg, x, dtype, scales, n, group):
    """Pages whose summaries are permutations of one set of values under queries of one value in all channels: equal scores
    from other running sums.  On some pages the smallest term is a step of its own larger or smaller, 2^-40 to 2^-52 of the
    terms' magnitude.  All sums fit 53 bits, so float64 has them exactly, in any order."""
    d, t = 128, torch
    g = t.Generator().manual_seed(n + group)
    # large, middling and small values: what the running sums round off spans more than 24 bits
    top, mid, step = {BF16: (2.0 ** 10, 2.0 ** -4, 2.0 ** -27), F16: (2.0 ** 10, 2.0 ** -2, 2.0 ** -24), E4M3: (2.0 ** 7, 2.0 ** -2, 2.0 ** -9)}[dtype]
    bits = {BF16: 128, F16: 1024, E4M3: 8}[dtype]
    large, middle = ((1 + t.randint(0, bits, (k,), generator=g).double() / bits) * v for k, v in ((40, top), (48, mid)))
    small = t.randint(2, 8, (40,), generator=g).double() * step
    large, middle = large.to(dtype).double(), middle.to(dtype).double()
    sign = 1.0 - 2.0 * t.randint(0, 2, (d,), generator=g)
    values = t.cat([large, middle, small]) * sign
    c = Case(pkg, [16 * n], H=1, d=d, dtype=dtype, scales=scales, seed=1, summaries=True, fill=False)
    pages = t.stack([values[t.randperm(d, generator=g)] for _ in range(c.k.shape[0])])
    odd = t.randint(0, c.k.shape[0], (n // 10,), generator=g)
    at = pages[odd].abs().argmin(1)
    pages[odd, at] += step * (1.0 - 2.0 * t.randint(0, 2, (len(odd),), generator=g))
    assert t.equal(pages.to(dtype).double(), pages)
    for s in (c.k_min, c.k_max):
        _raw(s).copy_(_raw(pages.to(dtype))[:, None].cuda())
    q = t.full((1, group, d), 1.0 + 2.0 ** -7 * 37, dtype=x)
    q[0, group // 2:] *= -1  # the other half of the heads ranks the other way round
    for m in (2, n // 15, n // 2, n - 7):
        _check_select(pkg, c, q, m)


@pytest.mark.parametrize("x,dtype,scales", TYPES)
def test_select_takes_pages_of_nan_keys_first(pkg, x, dtype, scales):
    """Append passes NaN over in the summaries, so a page of nothing else keeps what a summary starts with; its logits are
    NaN, and so it ranks first.  The same for an infinite bound under a query of 0."""
    n = 100
    c = Case(pkg, [16 * n], H=1, d=32, dtype=dtype, scales=scales, seed=3, summaries=True, fill=False)
    rows = c.randn(16 * n, 1, 32, dtype=x)
    rows[16 * 41:16 * 42] = math.nan
    rows[16 * 60:16 * 61, :, 5] = math.nan  # one channel of a page
    pkg.attn_paged_append(c.kv, rows.cuda(), rows.cuda(), token_start=torch.tensor([0, 16 * n], dtype=torch.int32, device="cuda"))
    for sign in (1, -1):
        q = sign * (c.randn(1, 3, 32, dtype=x).abs() + 0.1)
        got = pkg.attn_paged_select(c.kv, q.cuda(), 2, keep_first=0, keep_last=0)
        assert pkg.sync_status() == 0 and got[0, 0].tolist() == [41, 60]
    if dtype == E4M3:
        return  # has no infinities
    c.k_min[int(c.table[0, 70]), 0, 9] = -math.inf
    q = c.randn(1, 3, 32, dtype=x).abs() + 0.1
    q[..., 9] = 0
    got = pkg.attn_paged_select(c.kv, q.cuda(), 3, keep_first=0, keep_last=0)
    assert pkg.sync_status() == 0 and got[0, 0].tolist() == [41, 60, 70]


def test_a_cache_keeps_what_it_was_built_with(pkg):
    c = Case(pkg, [100, 20], H=2, d=64, seed=1)
    q = c.randn(2, 4, 64)
    _check_decode(pkg, c, q)
    with pytest.raises(AttributeError):
        c.kv.seq_lens = torch.tensor([5, 5], dtype=torch.int32, device="cuda")
    assert c.kv.seq_lens is c.seq_lens and c.kv.block_table is c.block_table and c.kv.k_pages is c.k and c.kv.device == c.k.device
    assert (c.kv.B, c.kv.kv_heads, c.kv.page_size, c.kv.head_dim, c.kv.dtype) == (2, 2, 16, 64, BF16)
    c.lens_list = [5, 5]
    c.seq_lens.fill_(5)
    _check_decode(pkg, c, q)


@pytest.mark.parametrize("B,H,Hq", [(520, 8, 128), (260, 16, 384), (1500, 2, 90)])
def test_more_query_heads_in_all_than_a_grid_has_rows(pkg, B, H, Hq):
    """B * query heads past 65535."""
    g = torch.Generator().manual_seed(B)
    lens = [int(v) for v in torch.randint(0, 60, (B,), generator=g)]
    c = Case(pkg, lens, H=H, d=32, page=8, seed=B, summaries=True)
    q = c.randn(B, Hq, 32)
    o, lse = _check_decode(pkg, c, q)
    pages, want = _check_select(pkg, c, q, 3)
    keys = [[[p * 8 + i for p in row for i in range(8) if p * 8 + i < lens[b]] for row in rows] for b, rows in enumerate(want)]
    _check_decode(pkg, c, q, pages=pages, keys=keys)


def test_refused_sizes_take_no_memory(pkg):
    """A table that is too wide is refused before a workspace for it is allocated."""
    H, page = 512, 16
    k = torch.zeros((2, H, page, 32), dtype=BF16, device="cuda")
    lo = torch.zeros((2, H, 32), dtype=BF16, device="cuda")
    table = torch.zeros((1, (1 << 26) + 1), dtype=torch.int32, device="cuda")
    kv = pkg.PagedKV(k, k.clone(), table, torch.tensor([3], dtype=torch.int32, device="cuda"), k_min=lo, k_max=lo.clone())
    q = torch.zeros((1, H, 32), dtype=BF16, device="cuda")
    for call in (lambda: pkg.attn_paged_select(kv, q, 4), lambda: pkg.attn_paged_decode(kv, q)):
        torch.cuda.reset_peak_memory_stats()
        now = torch.cuda.memory_allocated()
        with pytest.raises(pkg.AttnError) as e:
            call()
        assert e.value.code == 2 and torch.cuda.max_memory_allocated() - now < 1 << 20


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("n", [40, 700, 9000])
def test_decode_logits_about_the_end_of_the_shift(pkg, sign, n):
    """Integer logits on either side of +-2^20 (in units of log2), where the weights' origin goes from 15 below the maximum to
    the maximum itself: tiles, warps and blocks with either are joined.  The products are exact, so only the weights' words
    and the sums err."""
    d = 64
    c = Case(pkg, [n], H=1, d=d, dtype=F16, seed=n)
    k = torch.zeros(n, d, dtype=torch.float64)
    k[:, 0] = 1024
    k[:, 1] = torch.randint(-14, 15, (n,), generator=c.g).double()
    k[::97, 1] += torch.randint(-1000, 5, (len(k[::97]),), generator=c.g)
    pos = torch.arange(n)
    _raw(c.k)[c.table[0, pos // 16].long().cuda(), 0, (pos % 16).cuda()] = k.to(F16).cuda()
    q = torch.zeros(1, 2, d, dtype=F16)
    q[0, :, 0], q[0, :, 1] = sign * 1024, torch.tensor([1.0, -1.0])
    scale = math.log(2.0)
    assert float(torch.tensor(scale) * torch.tensor(1.4426950408889634)) == 1.0  # fp32: the factor is exact too
    o, lse = pkg.attn_paged_decode(c.kv, q.cuda(), scale=scale)
    assert pkg.sync_status() == 0
    s = q[0].double() @ k.T
    w = torch.softmax((s - s.amax(-1, keepdim=True)) * math.log(2.0), -1)
    v = c.v_ref[0, 0, :n]
    want = w @ v
    tol = 2.0 ** -11 * want.abs() * (1 + 1e-3) + (3 * 2.0 ** -22 + 2.0 ** -19) * (w @ v.abs() + want.abs()) + 2.0 ** -25
    err = (o[0].double().cpu() - want).abs()
    assert (err <= tol).all(), "off by %g of its tolerance" % (err / tol).max()
    l = torch.logsumexp(s * math.log(2.0), -1)
    assert ((lse[0].double().cpu() - l).abs() <= 2.0 ** -22 * l.abs()).all()


@pytest.mark.parametrize("B,live", [(4096, 2), (60000, 3)])
def test_long_runs_of_slots_without_a_sequence(pkg, B, live):
    """Slots between two sequences that hold none."""
    at = [0] + sorted(int(v) for v in torch.randint(1, B - 1, (live - 2,), generator=torch.Generator().manual_seed(B))) + [B - 1]
    c = Case(pkg, [4000 - 7 * i for i in range(live)], H=1, d=64, seed=1, summaries=True)
    q = c.randn(live, 2, 64).cuda()
    want = pkg.attn_paged_decode(c.kv, q)
    table = torch.full((B, c.table.shape[1]), 0x7FFFFFF0, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    table[at], lens[at] = c.block_table, c.seq_lens
    wide = torch.full((B, 2, 64), math.nan, dtype=BF16, device="cuda")
    wide[at] = q
    kv = pkg.PagedKV(c.k, c.v, table, lens, k_min=c.k_min, k_max=c.k_max)
    o, lse = pkg.attn_paged_decode(kv, wide)
    assert pkg.sync_status() == 0
    ro, rl, to, tl = _reference(c, q.cpu(), 1 / 8)
    assert ((o[at].double().cpu() - ro).abs() <= to).all() and ((lse[at].double().cpu() - rl).abs() <= tl).all()
    assert ((want[0].double().cpu() - ro).abs() <= to).all()
    empty = torch.ones(B, dtype=torch.bool, device="cuda")
    empty[at] = False
    assert (o[empty] == 0).all() and (lse[empty] == -math.inf).all()
    pages = pkg.attn_paged_select(kv, wide, 7)
    assert pkg.sync_status() == 0
    assert torch.equal(pages[at], pkg.attn_paged_select(c.kv, q, 7)) and (pages[empty] == -1).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n", [3, 100, 5000, 40000])
def test_infinite_values_stay_infinite(pkg, dtype, n):
    """A visible V of inf under a positive weight makes that channel inf, with its sign, and no other channel."""
    c = Case(pkg, [n, n], H=1, d=64, dtype=dtype, seed=n)
    q = c.randn(2, 12, 64).cuda()
    for at, ch, x in ((1, 5, math.inf), (n - 1, 20, -math.inf), (n // 2, 63, math.inf)):
        c.v[int(c.table[0, at // 16]), 0, at % 16, ch] = x
    o, lse = pkg.attn_paged_decode(c.kv, q)
    assert pkg.sync_status() == 0
    want = {5: math.inf, 20: -math.inf, 63: math.inf}
    for ch in range(64):
        if ch in want:
            assert (o[0, :, ch] == want[ch]).all(), ch
        else:
            assert o[0, :, ch].isfinite().all(), ch
    assert o[1].isfinite().all() and lse.isfinite().all()


def test_more_key_value_heads_in_all_than_a_grid_has_rows(pkg):
    """B * kv_heads past 65535: a thousand slots of 64 heads, forty of them with a sequence."""
    g = torch.Generator().manual_seed(1)
    B, H = 1100, 64
    lens = [0] * B
    for b in [0, B - 1, 1023, 1024] + torch.randint(0, B, (36,), generator=g).tolist():
        lens[b] = int(torch.randint(1, 70, (1,), generator=g))
    c = Case(pkg, lens, H=H, d=32, page=8, seed=2, summaries=True)
    q = c.randn(B, H, 32)
    _check_decode(pkg, c, q)
    _check_select(pkg, c, q, 3)
    _check_append(pkg, c, [1] * B, BF16, Hq=H, single=True)
