"""The paged cache of a model with a sliding window: decode over the window and
the sinks against plain float64 forms (tolerances: test_gpu_paged.py), the step's
bookkeeping against a list-by-list statement of it, and both with the append as a
server runs them."""
import math
import random

import pytest
import torch

import test_gpu_paged as paged
from test_gpu_paged import BF16, E4M3, F16, TYPES, Case, _reference

pytestmark = pytest.mark.gpu
pkg = paged.pkg


def _keys(n, window, sinks):
    return [j for j in range(n) if j >= n - window or j < sinks]


def _check_window(pkg, c, q, window, sinks, scale=None, **kw):
    scale = 1 / math.sqrt(c.d) if scale is None else scale
    keys = [[_keys(n, window, sinks)] * c.H for n in c.lens_list]
    o, lse = pkg.attn_paged_decode_window(c.kv, q.cuda(), window, sinks, scale=scale, **kw)
    assert pkg.sync_status() == 0
    ro, rl, to, tl = _reference(c, q.cpu(), scale, keys)
    assert torch.isfinite(o.float()).all()
    err = (o.double().cpu() - ro).abs()
    assert (err <= to).all(), "o off by %g of its tolerance" % (err / to).max()
    none = rl == -math.inf
    assert torch.equal(lse.double().cpu() == -math.inf, none) and (o.cpu()[none] == 0).all()
    lerr = (lse.double().cpu()[~none] - rl[~none]).abs()
    assert (lerr <= tl[~none]).all(), "lse off by %g of its tolerance" % (lerr / tl[~none]).max()
    return o, lse


def _forget(c, window, sinks):
    """Table entries and slots of hidden tokens: pages with nothing to see are not the sequence's any more, slots hold NaN."""
    for b, n in enumerate(c.lens_list):
        seen = set(_keys(n, window, sinks))
        for j in range(-(-n // c.page)):
            tokens = range(j * c.page, min(n, (j + 1) * c.page))
            p = int(c.table[b, j])
            for t in tokens:
                if t not in seen:
                    for x in (c.k, c.v):
                        row = paged._raw(x)[p, :, t - j * c.page]
                        row.fill_(paged.NAN_BYTE if c.dtype == E4M3 else math.nan)
            if not any(t in seen for t in tokens):
                c.block_table[b, j] = random.Random(j).choice([-1, 0x7FFFFFF0])


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 193, 500, 1000, 0]


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("x,dtype,scales", TYPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (63, 4), (64, 64), (65, 130), (128, 1), (300, 7), (2000, 5)])
def test_lengths_around_the_borders(pkg, x, dtype, scales, d, window, sinks):
    c = Case(pkg, LENS, H=2, page=16, d=d, dtype=dtype, scales=scales, seed=d + window)
    _forget(c, window, sinks)
    _check_window(pkg, c, c.randn(len(LENS), 6, d, dtype=x), window, sinks)


@pytest.mark.parametrize("page", [8, 24, 32, 56, 64, 128, 1024])
@pytest.mark.parametrize("layout", ["heads", "tokens", "turns"])
def test_pages_and_layouts(pkg, page, layout):
    lens = [700, 1, page, page + 1, 2 * page - 1, 3 * page + 5]
    c = Case(pkg, lens, H=3, page=page, d=128, layout=layout, seed=page)
    _forget(c, 100, 30)
    _check_window(pkg, c, c.randn(len(lens), 3, 128), 100, 30)
    c = Case(pkg, lens, H=1, page=page, d=64, dtype=E4M3, layout=layout, seed=page, scales=(0.02, 0.03))
    _forget(c, 33, 1)
    _check_window(pkg, c, c.randn(len(lens), 4, 64, dtype=F16), 33, 1)


@pytest.mark.parametrize("group", [1, 3, 8, 9, 16, 17, 33])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_group_sizes(pkg, group, dtype):
    c = Case(pkg, [900, 41], H=2, d=64, dtype=dtype, seed=group, scales=(0.02, 0.03))
    _check_window(pkg, c, c.randn(2, 2 * group, 64), 200, 5)


@pytest.mark.parametrize("B", [1, 7, 200, 1500])
@pytest.mark.parametrize("window,sinks", [(20, 0), (400, 4), (90, 300)])
def test_ragged_batches(pkg, B, window, sinks):
    """Few items in clusters, shares of many, whole short items to a warp."""
    g = torch.Generator().manual_seed(B)
    lens = [int(x) for x in (torch.rand(B, generator=g) ** 3 * 1500)]
    c = Case(pkg, lens, H=2, d=32, seed=B, width=200)
    _check_window(pkg, c, c.randn(B, 8, 32), window, sinks)


@pytest.mark.parametrize("window,sinks", [(60000, 100), (5000, 0)])
def test_one_long_sequence(pkg, window, sinks):
    c = Case(pkg, [70001], H=1, page=64, d=64, seed=7)
    _check_window(pkg, c, c.randn(1, 4, 64), window, sinks)


def test_a_window_of_all_is_the_whole_cache(pkg):
    c = Case(pkg, [700, 64, 0, 1], H=2, d=64, seed=8)
    q = c.randn(4, 4, 64).cuda()
    a, b = pkg.attn_paged_decode_window(c.kv, q, 700), pkg.attn_paged_decode(c.kv, q)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for big in (1 << 30, 1 << 80):
        a = pkg.attn_paged_decode_window(c.kv, q, big, big)
        assert torch.equal(a[0], b[0])


def test_many_streams_and_repeats(pkg):
    c = Case(pkg, [3000, 50, 700] * 20, H=4, d=128, seed=9)
    q = c.randn(60, 8, 128).cuda()
    first = _check_window(pkg, c, q, 500, 4)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        more = [pkg.attn_paged_decode_window(c.kv, q, 500, 4, stream=s) for s in streams]
        torch.cuda.synchronize()
        for o, lse in more:
            assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


def test_bad_pages_in_sight_are_left_out(pkg):
    c = Case(pkg, [400], H=1, d=64, seed=10)
    q = c.randn(1, 2, 64)
    c.block_table[0, 24] = -7  # tokens 384 .. 399, in the window
    o, lse = pkg.attn_paged_decode_window(c.kv, q.cuda(), 100, 4)
    assert pkg.status_string(pkg.sync_status()) == "device-side check failed"
    keys = [[[j for j in _keys(400, 100, 4) if j < 384]]]
    ro, rl, to, tl = _reference(c, q, 0.125, keys)
    assert ((o.double().cpu() - ro).abs() <= to).all() and ((lse.double().cpu() - rl).abs() <= tl).all()


def test_captured_decode_replays_with_other_lengths(pkg):
    c = Case(pkg, [900, 300, 1200], H=2, d=64, seed=11)
    q = c.randn(3, 4, 64).cuda()
    pkg.attn_paged_decode_window(c.kv, q, 256, 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = pkg.attn_paged_decode_window(c.kv, q, 256, 4)
    for lens in ([900, 300, 1200], [1, 0, 257], [260, 261, 4]):
        c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        assert pkg.sync_status() == 0
        c.lens_list = lens
        ro, rl, to, tl = _reference(c, q.cpu(), 0.125, [[_keys(n, 256, 4)] * 2 for n in lens])
        assert ((o.double().cpu() - ro).abs() <= to).all()


# ------------------------------------------------------------------ bookkeeping

class Books:
    """What attn_paged_assign does, list by list."""

    def __init__(self, table, lens, ring, state, page, window, sinks):
        self.table, self.lens, self.ring, self.state = [list(r) for r in table], list(lens), list(ring), list(state)
        self.page, self.first = page, -(-sinks // page) if window else 0
        self.turns = -(-(window - 1) // page) + 1 if window else None

    def step(self, new, rows=None):
        page, cap = self.page, len(self.ring)
        own = lambda n: -(-n // page) if self.turns is None else min(-(-n // page), self.first + self.turns)  # noqa: E731
        head, count = self.state
        take = sum(own(n + m) - own(n) for n, m in zip(self.lens, new) if m > 0)
        back = sum(own(n) for n, m in zip(self.lens, new) if m < 0)
        total = sum(max(m, 0) for m in new)
        assert take <= count and count + back <= cap and (rows is None or total <= rows)
        start, slots, end = [0], [], (head + count) % cap
        for b, m in enumerate(new):
            n, row = self.lens[b], self.table[b]
            if m < 0:
                for j in range(own(n)):
                    self.ring[end] = row[j]
                    end = (end + 1) % cap
                self.lens[b] = 0
            else:
                for j in range(-(-n // page), -(-(n + m) // page)):
                    if self.turns is None or j < self.first + self.turns:
                        row[j] = self.ring[head]
                        head = (head + 1) % cap
                    else:
                        row[j] = row[j - self.turns]
                slots += [row[p // page] * page + p % page for p in range(n, n + m)]
                self.lens[b] = n + m
            start.append(start[-1] + max(m, 0))
        self.state = [head, count - take + back]
        return start, slots + [-1] * ((rows or 0) - total)


class Server:
    """A cache without a token, and its books; the ring starts at `at`."""

    def __init__(self, pkg, B, page=16, pages=64, width=16, window=0, sinks=0, at=5, H=1, d=32, cap=None, seed=0):
        g = torch.Generator().manual_seed(seed)
        cap = cap or pages
        ring = [-9] * cap
        for i, p in enumerate(torch.randperm(pages, generator=g).tolist()):
            ring[(at + i) % cap] = p
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.ring, self.state = i32(ring), i32([at % cap, pages])
        self.table, self.lens = torch.full((B, width), -5, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
        self.k, self.v = (torch.full((pages, H, page, d), math.nan, dtype=BF16, device="cuda") for _ in range(2))
        self.kv = pkg.PagedKV(self.k, self.v, self.table, self.lens)
        self.books = Books(self.table.tolist(), [0] * B, ring, [at % cap, pages], page, window, sinks)
        self.pkg, self.window, self.sinks, self.i32 = pkg, window, sinks, i32

    def same(self):
        assert self.table.tolist() == self.books.table
        assert self.lens.tolist() == self.books.lens
        assert self.ring.tolist() == self.books.ring
        assert self.state.tolist() == self.books.state

    def step(self, new, extra=0):
        rows = sum(max(0, m) for m in new) + extra
        slots = torch.full((rows,), 77, dtype=torch.int64, device="cuda") if rows else None
        start = self.pkg.attn_paged_assign(self.kv, self.i32(new), self.ring, self.state, slots=slots, rows=rows, window=self.window, sinks=self.sinks)
        assert self.pkg.sync_status() == 0
        want, places = self.books.step(new, rows)
        assert start.tolist() == want
        assert slots is None or slots.tolist() == places
        self.same()
        return start


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (16, 0), (40, 5), (33, 33), (17, 100)])
@pytest.mark.parametrize("page", [8, 16, 24])
def test_steps_in_place(pkg, page, window, sinks):
    r = random.Random(page + window + sinks)
    s = Server(pkg, 5, page=page, pages=200, width=40, window=window, sinks=sinks, at=190)
    most = s.books.turns * page if window else 100
    for i in range(40):
        new = []
        for n in s.books.lens:
            m = r.choice([0, 1, 1, 1, -1 if n else 0, r.randint(1, min(most, 60))])
            new.append(m if n + m <= 40 * page else -1)
        s.step(new, extra=r.choice([0, 0, 7]))
    s.step([-1] * 5)
    assert s.books.state[1] == 200 and sorted(s.books.ring) == list(range(200))  # every page has come back


@pytest.mark.parametrize("B,longest,page", [(1, 1, 8), (1, 9000, 16), (33, 500, 32), (1024, 20, 8), (1025, 3, 8), (3000, 40, 16), (7, 40000, 64)])
def test_sizes(pkg, B, longest, page):
    """One block, or two kernels: many sequences, many tokens."""
    r = random.Random(B)
    width = 2 * -(-longest // page) + 1
    s = Server(pkg, B, page=page, pages=B * width, width=width, cap=B * width + 13, at=B)
    s.step([r.choice([0, 1, longest, r.randint(1, longest)]) for _ in range(B)], extra=5)
    s.step([r.choice([-1, 0, 1, r.randint(1, longest)]) for _ in range(B)])
    s.step([r.choice([-1, 1]) for _ in range(B)])


def test_apart_from_its_inputs_a_step_can_be_taken_again(pkg):
    s = Server(pkg, 4, pages=40, width=8, window=40, sinks=4)
    s.step([30, 10, 0, 40])
    old, state = s.lens.clone(), s.state.clone()
    out, start, slots = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(5, dtype=torch.int32, device="cuda"), torch.zeros(64, dtype=torch.int64, device="cuda")
    want = None
    for new in ([3, -1, 7, 20], [1, 1, 1, 1], [3, -1, 7, 20]):
        got = pkg.attn_paged_assign(s.kv, s.i32(new), s.ring, state, lens=old, free_out=out, token_start=start, slots=slots, window=40, sinks=4)
        assert got is start
        result = (s.lens.tolist(), out.tolist(), start.tolist(), slots.tolist())
        want = want or result
    assert result == want and state.tolist() == s.books.state and pkg.sync_status() == 0
    places = s.books.step([3, -1, 7, 20], 64)
    assert result == (s.books.lens, s.books.state, places[0], places[1])


@pytest.mark.parametrize("B", [3, 1500])
def test_a_step_that_cannot_be_done_is_not_done(pkg, B):
    s = Server(pkg, B, pages=B * 2, width=4, window=40, sinks=4)
    s.step([16] * B)
    taken = [1] * (B - 3)
    before = [x.clone() for x in (s.table, s.lens, s.ring, s.state)]
    cases = [
        ([17, 17, 0] + [17] * (B - 3), None),   # more pages than there are
        ([1, -2, 1] + taken, None),             # not a count
        ([1, 49, 1] + taken, None),             # past the table's end
        ([1, 1, 1] + taken, B - 1),             # more than rows
        ([1, 1, 0x7FFFFFFF] + taken, None),
    ]
    for new, rows in cases:
        slots = torch.zeros(4 * B if rows is None else rows, dtype=torch.int64, device="cuda")
        out = torch.zeros(2, dtype=torch.int32, device="cuda")
        start = pkg.attn_paged_assign(s.kv, s.i32(new), s.ring, s.state, free_out=out, slots=slots, window=40, sinks=4)
        assert pkg.status_string(pkg.sync_status()) == "device-side check failed", new[:3]
        assert (start == 0).all() and (slots == -1).all()
        assert all(torch.equal(a, b) for a, b in zip((s.table, s.lens, s.ring, s.state), before))
        assert torch.equal(out, s.state)
    for lens, state in (([16, -1, 16], None), ([16, 65, 16], None), (None, [-1, 3]), (None, [B * 2, 3]), (None, [0, -1]), (None, [0, 2 * B + 1])):
        old = s.lens.clone()
        if lens:
            old[:3] = s.i32(lens)
        st, out = s.i32(state) if state else s.state.clone(), torch.zeros(2, dtype=torch.int32, device="cuda")
        start = pkg.attn_paged_assign(s.kv, s.i32([1] * B), s.ring, st, lens=old, free_out=out, window=40, sinks=4)
        assert pkg.sync_status() == 6 and (start == 0).all() and torch.equal(out, st) and torch.equal(s.lens, old)
        s.lens.copy_(before[1])
        assert torch.equal(s.table, before[0]) and torch.equal(s.ring, before[2])
    # a windowed sequence's new tokens would share slots: turns = 4 pages
    t = Server(pkg, 1, pages=20, width=16, window=40, sinks=4)
    slots = torch.zeros(80, dtype=torch.int64, device="cuda")
    pkg.attn_paged_assign(t.kv, t.i32([65]), t.ring, t.state, slots=slots, window=40, sinks=4)
    assert pkg.sync_status() == 6
    t.same()
    t.step([64])
    # the ring has no room for what comes back
    full = Server(pkg, 2, pages=6, width=4)
    full.step([16, 16])
    full.state.copy_(full.i32([0, 6]))
    pkg.attn_paged_assign(full.kv, full.i32([-1, 0]), full.ring, full.state)
    assert pkg.sync_status() == 6 and full.lens.tolist() == [16, 16] and full.state.tolist() == [0, 6]


def test_bad_page_numbers_are_handed_on_as_none(pkg):
    s = Server(pkg, 2, pages=8, width=4, at=0)
    s.ring[1] = 1000
    slots = torch.zeros(40, dtype=torch.int64, device="cuda")
    pkg.attn_paged_assign(s.kv, s.i32([16, 17]), s.ring, s.state, slots=slots)
    assert pkg.sync_status() == 6
    assert s.table[1, 0].item() == -1 and (slots[16:32] == -1).all() and s.table[0, 0].item() == s.ring[0].item() and slots[32].item() == s.ring[2].item() * 16
    s.table[0, 0] = 99
    pkg.attn_paged_assign(s.kv, s.i32([-1, 0]), s.ring, s.state)
    assert pkg.sync_status() == 6 and s.ring[0].item() == -1 and s.state.tolist() == [3, 6]


def test_assign_refuses(pkg):
    s = Server(pkg, 3, pages=12)
    n = s.i32([1, 1, 1])
    bad = [
        (TypeError, lambda: pkg.attn_paged_assign(None, n, s.ring, s.state)),
        (ValueError, lambda: pkg.attn_paged_assign(s.kv, n[:2], s.ring, s.state)),
        (ValueError, lambda: pkg.attn_paged_assign(s.kv, n.long(), s.ring, s.state)),
        (TypeError, lambda: pkg.attn_paged_assign(s.kv, n.cpu(), s.ring, s.state)),
        (ValueError, lambda: pkg.attn_paged_assign(s.kv, n, s.ring[::2], s.state)),
        (ValueError, lambda: pkg.attn_paged_assign(s.kv, n, s.ring[:0], s.state)),
        (ValueError, lambda: pkg.attn_paged_assign(s.kv, n, s.ring, s.state[:1])),
        (ValueError, lambda: pkg.attn_paged_assign(s.kv, n, s.ring, s.state, lens=n[:2])),
        (ValueError, lambda: pkg.attn_paged_assign(s.kv, n, s.ring, s.state, slots=n)),
        (ValueError, lambda: pkg.attn_paged_assign(s.kv, n, s.ring, s.state, slots=torch.zeros(4, dtype=torch.int64, device="cuda"), rows=5)),
        (ValueError, lambda: pkg.attn_paged_assign(s.kv, n, s.ring, s.state, window=-1)),
        (pkg.AttnError, lambda: pkg.attn_paged_assign(s.kv, n, n, s.state)),
        (ValueError, lambda: pkg.attn_paged_decode_window(s.kv, torch.zeros(3, 2, 32, dtype=BF16, device="cuda"), 0)),
        (TypeError, lambda: pkg.attn_paged_decode_window(s.kv, torch.zeros(3, 2, 32, dtype=F16, device="cuda"), 4)),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()
    assert pkg.sync_status() == 0
    s.same()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("window,sinks,page", [(40, 5, 8), (64, 0, 16), (100, 20, 16)])
def test_a_windowed_server_run(pkg, window, sinks, page, graph):
    """Prompts by attn_fwd_window, their keys and values into the cache in chunks, then tokens one by one through assign,
    append and decode, a sequence ending and another one taking its slot; a sequence's rows agree with attn_fwd_window over
    all of its tokens to both calls' tolerances, although the cache keeps only a few pages of it."""
    B, H, Hq, d, steps = 3, 2, 4, 64, 60
    g = torch.Generator().manual_seed(window)
    s = Server(pkg, B, page=page, pages=B * (-(-sinks // page) + -(-(window - 1) // page) + 1), width=-(-400 // page), window=window, sinks=sinks, H=H, d=d)
    chunk = s.books.turns * page
    hist = [None] * B  # (q, k, v) of each sequence, [heads, n, d]
    new_rows = lambda n: tuple(torch.randn((n, h, d), generator=g).to(BF16).cuda() for h in (Hq, H, H))  # noqa: E731

    def prompt(b, n):
        q, k, v = new_rows(n)
        for at in range(0, n, chunk):
            m = min(chunk, n - at)
            start = s.step([m if x == b else 0 for x in range(B)])
            pkg.attn_paged_append(s.kv, k[at:at + m], v[at:at + m], token_start=start)
        hist[b] = [x.transpose(0, 1) for x in (q, k, v)]

    for b, n in enumerate((150, 7, 64)):
        prompt(b, n)
    n_new = s.i32([1] * B)
    bufs = new_rows(B)

    def call():
        start = pkg.attn_paged_assign(s.kv, n_new, s.ring, s.state, window=window, sinks=sinks)
        pkg.attn_paged_append(s.kv, bufs[1], bufs[2], token_start=start)
        return pkg.attn_paged_decode_window(s.kv, bufs[0], window, sinks)

    captured = None
    if graph:
        keep = [x.clone() for x in (s.table, s.lens, s.ring, s.state, s.k, s.v)]
        call()
        for x, y in zip((s.table, s.lens, s.ring, s.state, s.k, s.v), keep):
            x.copy_(y)
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            outs = call()
    for i in range(steps):
        if i == 30:
            s.step([0, 0, -1])
            prompt(2, 90)
        rows = new_rows(B)
        for to, x in zip(bufs, rows):
            to.copy_(x)
        if captured:
            captured.replay()
            o, lse = outs
        else:
            o, lse = call()
        s.books.step([1] * B)
        s.same()
        for b in range(B):
            hist[b] = [torch.cat([x, y[b][:, None]], 1) for x, y in zip(hist[b], rows)]
        if i % 7 == 0 or i == steps - 1:
            for b in range(B):
                q, k, v = (x[None] for x in hist[b])
                ro, rl = pkg.attn_fwd_window(q[:, :, -1:].contiguous(), k.contiguous(), v.contiguous(), window, sinks)
                # either side within u |O| + 2 u P|v| and 2^-15 (1 + L) of the value: weights of one, rounded to bf16 at worst
                n = k.shape[2]
                at = torch.tensor(_keys(n, window, sinks), device="cuda")
                kk, vv, qq = k[0, :, at].double().repeat_interleave(Hq // H, 0), v[0, :, at].double().repeat_interleave(Hq // H, 0), q[0, :, -1].double()
                t = (kk @ qq[:, :, None])[..., 0] / math.sqrt(d)
                big = ((kk.abs() @ qq.abs()[:, :, None])[..., 0] / math.sqrt(d)).amax(-1, keepdim=True)
                w = torch.softmax(t, -1)[:, None]
                tol = 2.0 ** -8 * (w @ vv)[:, 0].abs() + (2 * 2.0 ** -8 + 2 * 2.0 ** -15 * (1 + big)) * (w @ vv.abs())[:, 0]
                assert ((o[b].double() - ro[0, :, 0].double()).abs() <= 2 * tol).all()
                assert ((o[b].double() - (w @ vv)[:, 0]).abs() <= tol).all()
                assert ((lse[b].double() - rl[0, :, 0].double()).abs() <= 2 * 2.0 ** -15 * (1 + big[:, 0])).all()
    assert pkg.sync_status() == 0
