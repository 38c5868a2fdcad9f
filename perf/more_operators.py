"""Cases for attention with a sliding window and sinks (the first tokens, which
stay visible): prompts, training steps, single tokens over a paged cache; and
for the bookkeeping of that cache, which turns request lengths into block
tables and slots.

Each case is one pass with the shapes, head groups, strides and element types
of use; run() computes it either in plain torch operations or, with `own` set,
through the package's entry points, and exact() states the definition in
float64.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "e4m3": 1}
E4M3_MAX = 448.0
BLOCK = 512  # query rows that the plain form takes together


def listed():
    dense = {"x": "bf16", "D": 128, "token_major": True, "sinks": 4}
    paged = {"op": "decode", "x": "bf16", "cache": "bf16", "D": 128, "page": 16, "sinks": 4, "ragged": 0, "empty": 0}
    plan = {"op": "assign", "page": 16, "ragged": 1, "prompts": 0, "ended": 0, "idle": 0, "window": 0, "sinks": 0}
    return [
        # a short request of one user, small heads: latency alone
        {**dense, "op": "fwd", "name": "fwd_short", "B": 1, "Hq": 8, "Hkv": 2, "Nq": 200, "Nk": 200, "D": 64, "window": 64},
        # a prompt with shared heads, tensors as a projection leaves them
        {**dense, "op": "fwd", "name": "fwd_prompt", "B": 1, "Hq": 32, "Hkv": 8, "Nq": 8192, "Nk": 8192, "window": 1024},
        # the last part of a long prompt against all keys so far, odd sizes, a head of its own for every query head
        {**dense, "op": "fwd", "name": "fwd_chunk", "B": 1, "Hq": 16, "Hkv": 16, "Nq": 2001, "Nk": 20011, "D": 64, "window": 511, "sinks": 130, "x": "f16", "token_major": False},
        # a long document, wide window
        {**dense, "op": "fwd", "name": "fwd_long", "B": 1, "Hq": 32, "Hkv": 8, "Nq": 32768, "Nk": 32768, "window": 4096},
        # a small model's training step, ragged length, narrow heads
        {**dense, "op": "train", "name": "train_small", "B": 2, "Hq": 8, "Hkv": 8, "Nq": 500, "Nk": 500, "D": 32, "window": 100, "sinks": 1, "x": "f16", "token_major": False},
        # many short sequences, no sinks
        {**dense, "op": "train", "name": "train_short", "B": 8, "Hq": 12, "Hkv": 12, "Nq": 1024, "Nk": 1024, "D": 64, "window": 256, "sinks": 0, "token_major": False},
        # long sequences with shared heads, window and sinks
        {**dense, "op": "train", "name": "train_long", "B": 2, "Hq": 16, "Hkv": 4, "Nq": 8192, "Nk": 8192, "window": 1024},
        # a chat of one user: latency alone
        {**paged, "name": "decode_one", "B": 1, "Hq": 32, "Hkv": 8, "L": 5000, "window": 512},
        # a busy server: sequences of any length, many within the window, some slots empty, 8-bit cache
        {**paged, "name": "decode_ragged_e4m3", "B": 128, "Hq": 32, "Hkv": 8, "L": 16384, "window": 1024, "cache": "e4m3", "page": 32, "ragged": 7, "empty": 3},
        # long contexts, wide window, a large batch
        {**paged, "name": "decode_long", "B": 64, "Hq": 64, "Hkv": 8, "L": 131071, "window": 4096, "x": "f16", "cache": "f16", "page": 64, "ragged": 5},
        # one step of a server with windowed sequences: a token each, a few slots idle
        {**plan, "name": "assign_step", "B": 64, "L": 16384, "window": 1024, "sinks": 4, "idle": 5},
        # a scheduler's large step: prompts beside running sequences, ended ones hand back their pages
        {**plan, "name": "assign_prompts", "B": 4096, "L": 4096, "prompts": 512, "ended": 200, "idle": 100},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "train", "decode", "assign"])
    page = rng.choice([8, 16, 16, 24, 32, 64])
    if op == "assign":
        c = {"op": op, "page": page, "B": _spread(rng, 1, 4096), "L": _spread(rng, 64, 16384), "ragged": rng.randrange(1, 1000), "sinks": rng.choice([0, 1, 4, 100])}
        c["window"] = 0 if rng.random() < 0.5 else _spread(rng, 1, 4096)
        c["prompts"] = min(c["B"], _spread(rng, 1, 512)) if rng.random() < 0.6 else 0
        c["ended"], c["idle"] = rng.randrange(0, 1 + c["B"] // 8), rng.randrange(0, 1 + c["B"] // 8)
        c["L"] = min(c["L"], (1 << 24) // c["B"], (1 << 21) // max(1, c["prompts"]))
        return c
    x = rng.choice(["bf16", "f16"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    c = {"op": op, "x": x, "D": rng.choice([32, 64, 128, 128]), "Hkv": hkv, "Hq": hkv * rng.choice([1, 1, 2, 3, 4, 8]), "sinks": rng.choice([0, 1, 4, 4, 17, 128, 200]),
         "window": _spread(rng, 1, 4096)}
    if op == "decode":
        c |= {"cache": rng.choice([x, x, "e4m3"]), "page": page, "B": _spread(rng, 1, 64), "L": _spread(rng, 1, 131072), "ragged": rng.choice([0, rng.randrange(1, 1000)]), "empty": 0}
        c["empty"] = rng.randrange(0, 1 + c["B"] // 8)
        return c
    c["token_major"] = rng.random() < 0.5
    least = 1 if op == "fwd" else 2  # a row that sees one key has no gradient but in v
    c["Nq"], c["window"] = _spread(rng, least, 16384 if op == "fwd" else 4096), max(least, c["window"])
    c["Nk"] = c["Nq"] + (0 if rng.random() < 0.6 else _spread(rng, 1, 16384 if op == "fwd" else 4096))
    # no more work than the largest listed case of its kind
    most, wide = (4e9 if op == "fwd" else 2.5e8) / c["Hq"], c["window"] + c["sinks"]
    c["Nq"], c["Nk"] = min(c["Nq"], int(most / wide)), c["Nk"] - c["Nq"] + min(c["Nq"], int(most / wide))
    c["B"] = _spread(rng, 1, max(1, min(8, int(most / wide / c["Nq"]))))
    return c


def _randn(shape, dtype, g, scale=1.0):
    """Normal values in `dtype`, made in pieces so that no fp32 copy of a whole cache exists."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for part in out.view(torch.uint8 if dtype.itemsize == 1 else dtype).reshape(-1).split(1 << 28):
        v = torch.randn(part.numel(), generator=g, device="cuda", dtype=torch.float32 if dtype.itemsize == 1 else dtype)
        part.copy_(((v * scale).clamp_(-E4M3_MAX, E4M3_MAX).to(dtype).view(torch.uint8)) if dtype.itemsize == 1 else v)
    return out


def _rolling(c):
    """Pages of the sinks and pages in turns of a windowed sequence; without a window nothing turns."""
    if not c["window"]:
        return 0, 1 << 30
    return -(-c["sinks"] // c["page"]), -(-(c["window"] - 1) // c["page"]) + 1


def _lens(c):
    """Cached tokens of each sequence; slots without one stand at the end."""
    rng = random.Random(c["ragged"])
    lens = [c["L"] if b == 0 or not c["ragged"] else max(1, int(c["L"] * rng.random())) for b in range(c["B"])]
    return [0 if b >= c["B"] - c["empty"] else n for b, n in enumerate(lens)]


def _step(c):
    """(tokens held, new tokens or -1 for an ended sequence) of a scheduler's step."""
    rng = random.Random(c["ragged"])
    most = 1 << 30 if not c["window"] else _rolling(c)[1] * c["page"]  # new tokens of a windowed sequence in one step
    old, new = [], []
    for b in range(c["B"]):
        n = max(1, int(c["L"] * rng.random()))
        old.append(n if b >= c["prompts"] or rng.random() < 0.5 else 0)
        new.append(min(most, max(1, int(c["L"] * rng.random()))) if b < c["prompts"] else 1)
    kind = rng.sample(range(c["B"]), c["ended"] + c["idle"])
    for i, b in enumerate(kind):
        new[b] = -1 if i < c["ended"] else 0
    return old, new


def _prepare_assign(c, g):
    old, new = _step(c)
    page, (first, turns) = c["page"], _rolling(c)
    width = max(-(-(n + max(m, 0)) // page) for n, m in zip(old, new))
    old_t, new_t = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (old, new))
    col = torch.arange(width, device="cuda")
    held = (old_t[:, None].long() + page - 1) // page
    real = (col < held) & (col < first + turns)  # pages of their own; later ones turn
    rank = (real.flatten().cumsum(0) - 1).view_as(real)
    used = int(real.sum())
    need = sum(max(0, min(-(-(n + m) // page), first + turns) - min(-(-n // page), first + turns)) for n, m in zip(old, new) if m > 0)
    pages = used + need + 1 + need // 4
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.where(real, order[rank.clamp(0, pages - 1)], -1)
    if c["window"]:
        table = torch.where(col < held, table.gather(1, torch.where(col < first + turns, col, first + (col - first) % turns).expand_as(real)), -1)
    # the ring of free pages starts anywhere
    at = int(torch.randint(pages, (1,), generator=g, device="cuda"))
    ring = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    free = order[used:]
    ring[(at + torch.arange(free.numel(), device="cuda")) % pages] = free
    rows = sum(max(0, m) for m in new)
    s = {"case": c, "lens": old_t, "n_new": new_t, "table": table.contiguous(), "new_lens": torch.zeros_like(old_t), "ring": ring, "pages": pages,
         "free": torch.tensor([at, free.numel()], dtype=torch.int32, device="cuda"), "free_out": torch.zeros(2, dtype=torch.int32, device="cuda"),
         "start": torch.zeros(c["B"] + 1, dtype=torch.int32, device="cuda"), "slots": torch.zeros(rows, dtype=torch.int64, device="cuda"), "kv": None}
    # the cache that the step is for: rows of a token are small here, the bookkeeping does not look at them
    s["cache"] = [torch.zeros((pages, 1, page, 32), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    return s


def _prepare_decode(c, g):
    lens, page, (first, turns) = _lens(c), c["page"], _rolling(c)
    width = max(1, max(-(-n // page) for n in lens))
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    col = torch.arange(width, device="cuda")
    held = (lens_t[:, None].long() + page - 1) // page
    real = (col < held) & (col < first + turns)
    pages = int(real.sum()) + 1
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.where(real, order[(real.flatten().cumsum(0) - 1).view_as(real).clamp(0, pages - 1)], 0)
    table = table.gather(1, torch.where(col < first + turns, col, first + (col - first) % turns).expand_as(real)).contiguous()
    cache, scale = TYPES[c["cache"]], (1.0 / 64, 1.0 / 32) if c["cache"] == "e4m3" else (1.0, 1.0)
    shape = (pages, c["Hkv"], page, c["D"])
    return {"case": c, "table": table, "lens": lens_t, "k_scale": scale[0], "v_scale": scale[1], "kv": None,
            "k_pages": _randn(shape, cache, g, 1 / scale[0]), "v_pages": _randn(shape, cache, g, 1 / scale[1]), "q": _randn((c["B"], c["Hq"], c["D"]), TYPES[c["x"]], g)}


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda")
    g.manual_seed(seed)
    if c["op"] == "assign":
        return _prepare_assign(c, g)
    if c["op"] == "decode":
        return _prepare_decode(c, g)
    x, s = TYPES[c["x"]], {"case": c}
    if c["token_major"]:  # [B, N, heads, D] seen as [B, heads, N, D]; k and v are slices of one projection's output
        s["q"] = _randn((c["B"], c["Nq"], c["Hq"], c["D"]), x, g).transpose(1, 2)
        k, v = _randn((c["B"], c["Nk"], 2 * c["Hkv"], c["D"]), x, g).split(c["Hkv"], dim=2)
        s["k"], s["v"] = k.transpose(1, 2), v.transpose(1, 2)
        s["do"] = _randn((c["B"], c["Nq"], c["Hq"], c["D"]), x, g).transpose(1, 2) if c["op"] == "train" else None
    else:
        s["q"] = _randn((c["B"], c["Hq"], c["Nq"], c["D"]), x, g)
        s["k"], s["v"] = _randn((c["B"], c["Hkv"], c["Nk"], c["D"]), x, g), _randn((c["B"], c["Hkv"], c["Nk"], c["D"]), x, g)
        s["do"] = _randn((c["B"], c["Hq"], c["Nq"], c["D"]), x, g) if c["op"] == "train" else None
    return s


def _blocks(c):
    """The plain form's view: blocks of query rows, the keys that any row of a block can see, and who sees which."""
    nq, nk, w, sinks = c["Nq"], c["Nk"], min(c["window"], c["Nk"]), min(c["sinks"], c["Nk"])
    t = min(BLOCK, nq)
    n = -(-nq // t)
    pos = torch.arange(n * t, device="cuda").view(n, t) + nk - nq
    near = pos[:, :1] - w + 1 + torch.arange(w + t - 1, device="cuda")
    key = torch.cat([torch.arange(sinks, device="cuda").expand(n, sinks), near], 1)
    p, j = pos[:, :, None], key[:, None, :]
    first = torch.arange(key.shape[1], device="cuda") < sinks
    seen = torch.where(first, j <= p - w, (j > p - w) & (j <= p) & (j >= 0)) & (j <= p) & (p < nk)
    return n, t, key.clamp(0, nk - 1), seen


def _plain_fwd(c, q, k, v):
    n, t, key, seen = _blocks(c)
    b, hk, g, d, m = c["B"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"], key.shape[1]
    pad = n * t - c["Nq"]
    qb = torch.nn.functional.pad(q.float(), (0, 0, 0, pad)).view(b, hk, g, n, t, d).permute(0, 1, 3, 2, 4, 5).reshape(b, hk, n, g * t, d)
    kb, vb = (u.float()[:, :, key.flatten()].view(b, hk, n, m, d) for u in (k, v))
    s = (qb @ kb.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).view(b, hk, n, g, t, m).masked_fill_(~seen[:, None], float("-inf"))
    top = s.amax(-1, keepdim=True).clamp_min_(-3e38)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    total = total.masked_fill(total == 0, 1)  # rows of padding
    o = (p.view(b, hk, n, g * t, m) @ vb).view(b, hk, n, g, t, d) / total
    lse = (top + total.log()).squeeze(-1)
    rows = lambda u: u.permute(0, 1, 3, 2, 4, *range(5, u.dim())).reshape(b, c["Hq"], n * t, *u.shape[5:])[:, :, :c["Nq"]]  # noqa: E731
    return rows(o).to(q.dtype), rows(lse), (p.div_(total).view(b, hk, n, g * t, m), qb, kb, vb, key, rows)


def _plain_train(c, q, k, v, do):
    o, lse, (p, qb, kb, vb, key, rows) = _plain_fwd(c, q, k, v)
    n, t, d, b, hk, g = key.shape[0], qb.shape[3] // (c["Hq"] // c["Hkv"]), c["D"], c["B"], c["Hkv"], c["Hq"] // c["Hkv"]
    pad = n * t - c["Nq"]
    block = lambda u: torch.nn.functional.pad(u.float(), (0, 0, 0, pad)).view(b, hk, g, n, t, d).permute(0, 1, 3, 2, 4, 5).reshape(b, hk, n, g * t, d)  # noqa: E731
    dob = block(do)
    dvb = p.transpose(-1, -2) @ dob
    ds = (dob @ vb.transpose(-1, -2)).sub_((dob * block(o)).sum(-1, keepdim=True)).mul_(p).mul_(1.0 / math.sqrt(d))
    dq = rows((ds @ kb).view(b, hk, n, g, t, d)).to(q.dtype)
    dkb = ds.transpose(-1, -2) @ qb
    dk, dv = (torch.zeros((b, hk, c["Nk"], d), device="cuda").index_add_(2, key.flatten(), u.reshape(b, hk, -1, d)).to(q.dtype) for u in (dkb, dvb))
    return o, lse, dq, dk, dv


def _plain_decode(s):
    c, d = s["case"], s["case"]["D"]
    w, sinks, page = min(c["window"], c["L"]), min(c["sinks"], c["L"]), c["page"]
    ln = s["lens"].long()[:, None]
    pos = torch.cat([torch.arange(sinks, device="cuda").expand(c["B"], sinks), ln - w + torch.arange(w, device="cuda")], 1)
    first = torch.arange(sinks + w, device="cuda") < sinks
    seen = torch.where(first, pos < ln - w, pos >= 0)
    pos = pos.clamp(0, s["table"].shape[1] * page - 1)
    at = s["table"].long().gather(1, pos // page), pos % page
    g = c["Hq"] // c["Hkv"]
    kk, vv = (u.transpose(1, 2)[at].float() for u in (s["k_pages"], s["v_pages"]))  # [B, M, Hkv, D]
    q = s["q"].float().view(c["B"], c["Hkv"], g, d)
    lg = (q @ kk.permute(0, 2, 3, 1)) * (s["k_scale"] / math.sqrt(d))
    lg = lg.masked_fill(~seen[:, None, None], float("-inf"))
    top = lg.amax(-1, keepdim=True).clamp_min(-3e38)
    p = (lg - top).exp()
    total = p.sum(-1, keepdim=True)
    o = (p @ vv.permute(0, 2, 1, 3)) * (s["v_scale"] / total.masked_fill(total == 0, 1))
    return o.reshape(c["B"], c["Hq"], d).to(s["q"].dtype), (top + total.log()).reshape(c["B"], c["Hq"])


def _plain_assign(s):
    c, page, (first, turns) = s["case"], s["case"]["page"], _rolling(s["case"])
    old, n = s["lens"].long(), s["n_new"].long()
    more = n.clamp_min(0)
    new = torch.where(n < 0, 0, old + more)
    had, have = (old + page - 1) // page, (new + page - 1) // page
    take = torch.where(n < 0, 0, have.clamp_max(first + turns) - had.clamp_max(first + turns))
    start = torch.cat([more.new_zeros(1), more.cumsum(0)])
    base = take.cumsum(0) - take
    ring, cap = s["ring"], s["pages"]
    head, count = s["free"][0].long(), s["free"][1].long()
    # new table entries: pages of the ring, or the page that turns
    col = torch.arange(s["table"].shape[1], device="cuda")
    root = torch.where(col < first + turns, col, first + (col - first) % turns)
    fresh = ring[(head + base[:, None] + root - had.clamp_max(first + turns)[:, None]) % cap]
    value = torch.where(root >= had[:, None], fresh, s["table"].gather(1, root.expand(c["B"], -1)))
    fill = (n > 0)[:, None] & (col >= had[:, None]) & (col < have[:, None])
    s["table"].copy_(torch.where(fill, value, s["table"]))
    # slots of the new tokens
    row = torch.arange(s["slots"].numel(), device="cuda")
    seq = torch.searchsorted(start, row, right=True) - 1
    pos = old[seq] + row - start[seq]
    s["slots"].copy_(s["table"][seq, pos // page].long() * page + pos % page)
    # pages of ended sequences, behind the free ones
    back = (n < 0)[:, None] & (col < had.clamp_max(first + turns)[:, None])
    rank = back.flatten().cumsum(0) - 1
    to = torch.where(back.flatten(), (head + count + rank) % cap, cap)
    s["ring"].copy_(torch.cat([ring, ring.new_zeros(1)]).scatter_(0, to, torch.where(back, s["table"], 0).flatten())[:cap])
    s["start"].copy_(start)
    s["new_lens"].copy_(new)
    used = take.sum()
    s["free_out"].copy_(torch.stack([(head + used) % cap, count - used + back.sum()]))


def _kv(s):
    """The cache's handle, which a program makes once."""
    if s["kv"] is None:
        from io_aware_exact_12_gb300 import PagedKV
        if s["case"]["op"] == "assign":
            s["kv"] = PagedKV(*s["cache"], s["table"], s["new_lens"])
        else:
            s["kv"] = PagedKV(s["k_pages"], s["v_pages"], s["table"], s["lens"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return s["kv"]


def run(state):
    s, c = state, state["case"]
    w, sinks = c["window"], c["sinks"]
    if own:
        import io_aware_exact_12_gb300 as attn
        if c["op"] == "fwd":
            o, lse = attn.attn_fwd_window(s["q"], s["k"], s["v"], w, sinks)
        elif c["op"] == "train":
            o, lse = attn.attn_fwd_window(s["q"], s["k"], s["v"], w, sinks)
            dq, dk, dv = attn.attn_bwd_window(s["q"], s["k"], s["v"], o, s["do"], lse, w, sinks)
        elif c["op"] == "decode":
            o, lse = attn.attn_paged_decode_window(_kv(s), s["q"], w, sinks)
        else:
            attn.attn_paged_assign(_kv(s), s["n_new"], s["ring"], s["free"], lens=s["lens"], free_out=s["free_out"], token_start=s["start"], slots=s["slots"], window=w, sinks=sinks)
    elif c["op"] == "fwd":
        o, lse, _ = _plain_fwd(c, s["q"], s["k"], s["v"])
    elif c["op"] == "train":
        o, lse, dq, dk, dv = _plain_train(c, s["q"], s["k"], s["v"], s["do"])
    elif c["op"] == "decode":
        o, lse = _plain_decode(s)
    else:
        _plain_assign(s)
    if c["op"] == "assign":
        return {"table": s["table"], "lens": s["new_lens"], "start": s["start"], "slots": s["slots"], "ring": s["ring"], "free": s["free_out"]}
    if c["op"] == "train":
        return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    return {"o": o, "lse": lse}


def _pairs(nq, nk, window, sinks):
    """Visible (query, key) pairs of one head."""
    total = 0
    for p in range(nk - nq, nk):
        near = min(window, p + 1)
        total += near + min(sinks, p + 1 - near)
    return total


def work(case):
    c = case
    if c["op"] == "assign":
        old, new = _step(c)
        first, turns = _rolling(c)
        rows = sum(max(0, m) for m in new)
        pages = sum(-(-(n + m) // c["page"]) - -(-n // c["page"]) for n, m in zip(old, new) if m > 0)
        back = sum(min(-(-n // c["page"]), first + turns) for n, m in zip(old, new) if m < 0)
        return {"bytes": c["B"] * 16 + rows * 8 + (pages + back) * 8, "flops": 2 * rows}
    if c["op"] == "decode":
        keys = sum(min(n, c["window"]) + min(c["sinks"], max(0, n - c["window"])) for n in _lens(c))
        io = c["B"] * c["Hq"] * (2 * c["D"] * SIZE[c["x"]] + 4) + c["B"] * 4
        return {"bytes": 2 * keys * c["Hkv"] * c["D"] * SIZE[c["cache"]] + io, "flops": 4 * keys * c["Hq"] * c["D"]}
    pairs = c["B"] * c["Hq"] * _pairs(c["Nq"], c["Nk"], c["window"], c["sinks"])
    near = min(c["Nk"], c["Nq"] + c["window"] - 1)
    seen = near + min(c["sinks"], c["Nk"] - near)  # keys that some query sees
    q, k, row = c["B"] * c["Hq"] * c["Nq"] * c["D"] * 2, c["B"] * c["Hkv"] * seen * c["D"] * 2, c["B"] * c["Hkv"] * c["Nk"] * c["D"] * 2
    lse = c["B"] * c["Hq"] * c["Nq"] * 4
    if c["op"] == "fwd":
        return {"bytes": 2 * q + 2 * k + lse, "flops": 4 * c["D"] * pairs}
    return {"bytes": 4 * q + 2 * k + 2 * row + lse, "flops": 14 * c["D"] * pairs}


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "assign":
        return None  # whole numbers
    f, d = torch.float64, c["D"]
    g = c["Hq"] // c["Hkv"]
    if c["op"] == "decode":
        o, lse = torch.zeros((c["B"], c["Hq"], d), dtype=f, device="cuda"), torch.full((c["B"], c["Hq"]), float("-inf"), dtype=f, device="cuda")
        for b, n in enumerate(s["lens"].tolist()):
            if not n:
                continue
            at = [j for j in range(n) if j < c["sinks"]] if n > c["window"] else []
            at = torch.tensor([j for j in at if j < n - c["window"]] + list(range(max(0, n - c["window"]), n)), device="cuda")
            ids = s["table"][b][at // c["page"]].long()
            k, v = (u[ids, :, at % c["page"]].to(torch.float32).to(f) * r for u, r in ((s["k_pages"], s["k_scale"]), (s["v_pages"], s["v_scale"])))
            for h in range(c["Hkv"]):
                lg = s["q"][b, h * g:(h + 1) * g].to(f) @ k[:, h].T / math.sqrt(d)
                lse[b, h * g:(h + 1) * g] = torch.logsumexp(lg, -1)
                o[b, h * g:(h + 1) * g] = torch.softmax(lg, -1) @ v[:, h]
        return {"o": o, "lse": lse}
    train = c["op"] == "train"
    q, k, v = (s[n].to(f) for n in ("q", "k", "v"))
    off = c["Nk"] - c["Nq"]
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], dtype=f, device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for r in range(0, c["Nq"], 256):
        e = min(c["Nq"], r + 256)
        i = torch.arange(r + off, e + off, device="cuda")[:, None]
        lo = max(0, r + off - c["window"] + 1)
        j = torch.cat([torch.arange(min(c["sinks"], lo), device="cuda"), torch.arange(lo, e + off, device="cuda")])
        hidden = (j > i) | ((i - j >= c["window"]) & (j >= c["sinks"]))
        for h in range(c["Hq"]):
            kh, vh, qh = k[:, h // g, j], v[:, h // g, j], q[:, h, r:e]
            lg = torch.where(hidden, float("-inf"), qh @ kh.mT / math.sqrt(d))
            lse[:, h, r:e] = torch.logsumexp(lg, -1)
            p = torch.softmax(lg, -1)
            o[:, h, r:e] = p @ vh
            if train:
                do = s["do"][:, h, r:e].to(f)
                dp = do @ vh.mT
                ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(d)
                dq[:, h, r:e] = ds @ kh
                dk[:, h // g].index_add_(1, j, ds.mT @ qh)
                dv[:, h // g].index_add_(1, j, p.mT @ do)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv} if train else {"o": o, "lse": lse}
