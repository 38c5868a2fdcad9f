"""Cases for the paged-cache operators: appending rotated keys and values,
attention of one new token over the cache, and the same attention over the
pages that a cheap score selects.

Each case is one pass of one operator with the shapes, ragged lengths, page
tables and element types of serving; run() computes it either in plain torch
operations or, with `own` set, through the package's entry points, and
exact() states the definition in float64.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "e4m3": 1}
E4M3_MAX = 448.0


def listed():
    base = {"D": 128, "x": "bf16", "cache": "bf16", "page": 16, "ragged": 0, "empty": 0}
    step = {"op": "append", "new": 1, "pad": 0, "rot": 128, "interleaved": False, "summary": False}
    sparse = {"op": "sparse", "first": 1, "last": 1}
    return [
        # a chat of one user: the new token's key and value, latency alone
        {**base, **step, "name": "append_step_one", "B": 1, "Hq": 32, "Hkv": 8, "L": 1000},
        # one step of a busy server with graph slots that hold no sequence, small heads, summaries for the sparse reads
        {**base, **step, "name": "append_step_batch", "B": 256, "Hq": 16, "Hkv": 2, "D": 64, "rot": 64, "L": 8192, "x": "f16", "cache": "f16", "page": 64,
         "ragged": 3, "empty": 13, "interleaved": True, "summary": True},
        # a batch of prompts of unlike lengths, some behind a cached prefix
        {**base, **step, "name": "append_prompts", "B": 16, "Hq": 32, "Hkv": 8, "L": 4096, "new": 3001, "ragged": 5, "summary": True},
        # one long document into an 8-bit cache, rows of padding behind it, half of the channels rotated
        {**base, **step, "name": "append_document_e4m3", "B": 1, "Hq": 16, "Hkv": 4, "L": 65537, "new": 65537, "cache": "e4m3", "page": 32, "rot": 64, "pad": 63},
        # a chat of one user, short cache: latency alone
        {**base, "op": "decode", "name": "decode_one", "B": 1, "Hq": 32, "Hkv": 8, "L": 1000},
        # a busy server: sequences of any length up to 8192, some slots empty
        {**base, "op": "decode", "name": "decode_ragged", "B": 64, "Hq": 32, "Hkv": 8, "L": 8192, "ragged": 7, "empty": 3},
        # two long documents
        {**base, "op": "decode", "name": "decode_long", "B": 2, "Hq": 64, "Hkv": 8, "L": 131071, "x": "f16", "cache": "f16", "page": 64},
        # heads of their own for every query head, small heads, 8-bit cache
        {**base, "op": "decode", "name": "decode_heads_e4m3", "B": 128, "Hq": 16, "Hkv": 16, "D": 64, "L": 4096, "cache": "e4m3", "page": 32, "ragged": 11},
        # one user's long context, an eighth of it read
        {**base, **sparse, "name": "sparse_one", "B": 1, "Hq": 32, "Hkv": 8, "L": 16001, "select": 128},
        # a server's batch of unlike contexts, short ones read whole
        {**base, **sparse, "name": "sparse_batch", "B": 32, "Hq": 16, "Hkv": 4, "L": 32768, "x": "f16", "cache": "f16", "page": 32, "ragged": 13, "empty": 1, "select": 64, "last": 2},
        # very long contexts in large pages
        {**base, **sparse, "name": "sparse_long", "B": 8, "Hq": 32, "Hkv": 8, "L": 262143, "page": 64, "select": 256},
        # small pages in an 8-bit cache: many summaries for each token that is read
        {**base, **sparse, "name": "sparse_e4m3", "B": 4, "Hq": 40, "Hkv": 8, "L": 131072, "cache": "e4m3", "ragged": 17, "select": 128},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "sparse"])
    x = rng.choice(["bf16", "f16"])
    hkv = rng.choice([1, 2, 3, 4, 8, 16])
    c = {
        "op": op, "x": x, "cache": rng.choice([x, x, "e4m3"]), "D": rng.choice([32, 64, 128, 128]), "Hkv": hkv,
        "Hq": hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16, 24]), "page": rng.choice([8, 16, 16, 24, 32, 64, 128]),
        "B": _spread(rng, 1, 256), "ragged": rng.choice([0, rng.randrange(1, 1000)]), "empty": 0,
    }
    c["empty"] = rng.randrange(0, 1 + c["B"] // 8)
    token = hkv * c["D"] * 2 * SIZE[c["cache"]]  # bytes of one cached token
    if op == "append":
        single = rng.random() < 0.5
        wide = (2 * hkv + c["Hq"]) * c["D"] * 4
        c["new"] = 1 if single else _spread(rng, 2, max(3, min(60000, int(6e8 / wide / c["B"]))))
        c["L"] = c["new"] + _spread(rng, 1, max(2, min(16384, int(2e9 / token / c["B"]))))
        c["pad"] = 0 if single else rng.choice([0, 0, rng.randrange(1, 128)])
        c["rot"] = rng.choice([0, c["D"], c["D"], c["D"] // 2 if c["D"] > 32 else 16])
        c["interleaved"] = rng.random() < 0.3
        c["summary"] = rng.random() < 0.5
    else:
        c["L"] = _spread(rng, 1, max(64, min(200000, int(1e9 / token / c["B"]))))
        if op == "sparse":
            c["first"], c["last"] = rng.choice([0, 1, 1, 2]), rng.choice([1, 1, 4])
            c["select"] = max(c["first"] + c["last"], _spread(rng, 4, max(8, min(512, 1 + c["L"] // c["page"] // 2))))
    return c


def _lens(c):
    """(new tokens, cached tokens after them) of each sequence."""
    rng, new, lens = random.Random(c["ragged"]), [], []
    for b in range(c["B"]):
        u, w = (1.0, 1.0) if b == 0 or not c["ragged"] else (rng.random(), rng.random())
        n = max(1, int(c.get("new", 1) * u))
        new.append(n)
        lens.append(max(n, int(c["L"] * max(u, w) if c["op"] == "append" else c["L"] * u), 1))
    for b in range(c["B"] - c["empty"], c["B"]):  # slots without a sequence stand at the end
        new[b], lens[b] = (1, 0) if c.get("new", 1) == 1 else (0, 0)
    return new, lens


def _randn(shape, dtype, g, scale=1.0):
    """Normal values in `dtype`, made in pieces so that no fp32 copy of a whole cache exists."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for part in out.view(torch.uint8 if dtype.itemsize == 1 else dtype).reshape(-1).split(1 << 28):
        v = torch.randn(part.numel(), generator=g, device="cuda", dtype=torch.float32 if dtype.itemsize == 1 else dtype)
        part.copy_(((v * scale).clamp_(-E4M3_MAX, E4M3_MAX).to(dtype).view(torch.uint8)) if dtype.itemsize == 1 else v)
    return out


def _tables(rows, rot):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * inv
    return angle.cos().float(), angle.sin().float()


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda")
    g.manual_seed(seed)
    new, lens = _lens(c)
    x, cache = TYPES[c["x"]], TYPES[c["cache"]]
    need = [-(-n // c["page"]) for n in lens]
    width = max(max(need), 1)
    pages = sum(need) + 1
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((c["B"], width), dtype=torch.int32)
    take = torch.arange(pages, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = take[at:at + n]
        at += n
    table = order[table.to("cuda").long()].contiguous()
    shape = (pages, c["Hkv"], c["page"], c["D"])
    scale = (1.0 / 64, 1.0 / 32) if c["cache"] == "e4m3" else (1.0, 1.0)
    s = {"case": c, "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"), "k_scale": scale[0], "v_scale": scale[1],
         "k_pages": _randn(shape, cache, g, 1 / scale[0]), "v_pages": _randn(shape, cache, g, 1 / scale[1]), "k_min": None, "k_max": None}
    if c["op"] == "append":
        rows = sum(new)
        single = c["new"] == 1
        # keys, values and queries are slices of one projection's output, as a model has them
        qkv = _randn((rows + c["pad"], c["Hq"] + 2 * c["Hkv"], c["D"]), x, g)
        s["q"], s["k"], s["v"] = qkv.split([c["Hq"], c["Hkv"], c["Hkv"]], dim=1)
        s["q_out"] = torch.zeros((rows + c["pad"], c["Hq"], c["D"]), dtype=x, device="cuda")
        s["start"] = None if single else torch.tensor([sum(new[:b]) for b in range(c["B"] + 1)], dtype=torch.int32, device="cuda")
        s["cos"], s["sin"] = _tables(max(lens), c["rot"]) if c["rot"] else (None, None)
    else:
        s["q"] = _randn((c["B"], c["Hq"], c["D"]), x, g)
    if c["op"] == "sparse" or c.get("summary"):
        k = s["k_pages"]
        lo, hi = [], []
        for part in k.split(max(1, (1 << 28) // k[0].numel())):  # whole pages: the unused slots of a last page only loosen its bound
            part = part.to(torch.float16) if k.dtype.itemsize == 1 else part
            lo.append(part.amin(2).to(k.dtype))
            hi.append(part.amax(2).to(k.dtype))
        s["k_min"], s["k_max"] = torch.cat(lo), torch.cat(hi)
    if own:
        import io_aware_exact_12_gb300 as attn
        s["kv"] = attn.PagedKV(s["k_pages"], s["v_pages"], s["table"], s["lens"], k_scale=scale[0], v_scale=scale[1], k_min=s["k_min"], k_max=s["k_max"])
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        import io_aware_exact_12_gb300 as attn
        c = state["case"]
        if op == "append":
            attn.attn_paged_append(state["kv"], state["k"], state["v"], q=state["q"], q_out=state["q_out"], token_start=state["start"], cos=state["cos"], sin=state["sin"],
                                   interleaved=c["interleaved"])
            return _appended(state)
        if op == "decode":
            o, lse = attn.attn_paged_decode(state["kv"], state["q"])
            return {"o": o, "lse": lse}
        pages = attn.attn_paged_select(state["kv"], state["q"], c["select"], keep_first=c["first"], keep_last=c["last"])
        o, lse = attn.attn_paged_decode(state["kv"], state["q"], pages=pages)
        return {"pages": pages, "o": o, "lse": lse}
    if op == "append":
        return _append(state)
    if op == "decode":
        return _decode(state)
    return _sparse(state)


def _appended(s):
    out = {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if s["k_min"] is not None:
        out["k_min"], out["k_max"] = s["k_min"], s["k_max"]
    return out


def _rotate(x, cos, sin, interleaved):
    """fp32 x [rows, heads, d], cos and sin [rows, rot / 2]."""
    half = cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    y = x.clone()
    one, two = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    y[..., one] = x[..., one] * cos - x[..., two] * sin
    y[..., two] = x[..., two] * cos + x[..., one] * sin
    return y


def _stored(x, dtype, scale):
    return (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(dtype) if dtype.itemsize == 1 else x.to(dtype)


def _append(s):
    c, lens, table = s["case"], s["lens"].long(), s["table"]
    rows, page, pages = s["k"].shape[0], c["page"], s["k_pages"].shape[0]
    r = torch.arange(rows, device="cuda")
    if s["start"] is None:
        b, pos = r, lens - 1
        live = lens > 0
    else:
        start = s["start"].long()
        b = (torch.searchsorted(start, r, right=True) - 1).clamp(max=c["B"] - 1)
        pos = lens[b] - start[b + 1] + r
        live = r < start[-1]
    pos = torch.where(live, pos, 0)
    at, slot = table[b, pos // page].long(), pos % page
    k, v, q = s["k"].float(), s["v"].float(), s["q"].float()
    if s["cos"] is not None:
        cos, sin = s["cos"][pos], s["sin"][pos]
        k, q = _rotate(k, cos, sin, c["interleaved"]), _rotate(q, cos, sin, c["interleaved"])
    s["q_out"].copy_(torch.where(live[:, None, None], q.to(s["q_out"].dtype), s["q_out"]))
    dtype = s["k_pages"].dtype
    k, v = _stored(k, dtype, s["k_scale"]), _stored(v, dtype, s["v_scale"])
    raw = torch.uint8 if dtype.itemsize == 1 else dtype
    keep = live.nonzero()[:, 0]
    s["k_pages"].view(raw)[at[keep], :, slot[keep]] = k.view(raw)[keep]
    s["v_pages"].view(raw)[at[keep], :, slot[keep]] = v.view(raw)[keep]
    if s["k_min"] is not None:
        to = torch.where(live, at, pages)
        fresh = torch.zeros(pages + 1, device="cuda").scatter_reduce_(0, to, (slot == 0).float(), "amax")[:pages, None, None] > 0
        to = to[:, None, None].expand(k.shape)
        for name, how, none in (("k_min", "amin", math.inf), ("k_max", "amax", -math.inf)):
            old = torch.where(fresh, none, s[name].float())
            new = torch.cat([old, old[:1]]).scatter_reduce_(0, to, k.float(), how)[:pages]
            s[name].copy_(new.to(dtype))
    return _appended(s)


def _gathered(pages, table):
    """Pages [P, H, page, d] through a table [B, H or 1, n] as fp32 [B, H, n * page, d]."""
    raw = pages.view(torch.uint8) if pages.dtype.itemsize == 1 else pages
    heads = torch.arange(pages.shape[1], device="cuda")[None, :, None]
    x = raw[table.long(), heads]
    return x.view(pages.dtype).float().flatten(2, 3)


def _attend(s, table, seen):
    """Attention of q over the pages of `table` [B, H or 1, n], keys where `seen` [B, H or 1, n * page]."""
    c = s["case"]
    q = s["q"].float().unflatten(1, (c["Hkv"], c["Hq"] // c["Hkv"]))
    k, v = _gathered(s["k_pages"], table), _gathered(s["v_pages"], table)
    t = (q @ k.transpose(2, 3)) * (s["k_scale"] / math.sqrt(c["D"]))
    t = t.masked_fill(~seen[:, :, None], -math.inf)
    m = t.amax(-1, keepdim=True)
    p = torch.exp(t - m.masked_fill(m == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    o = (p @ v) * s["v_scale"] / total.masked_fill(total == 0, 1.0)
    lse = (m + total.log())[..., 0]
    return {"o": o.flatten(1, 2).to(s["q"].dtype), "lse": lse.flatten(1, 2)}


def _decode(s):
    n = s["table"].shape[1] * s["case"]["page"]
    seen = torch.arange(n, device="cuda")[None, None] < s["lens"][:, None, None]
    return _attend(s, s["table"][:, None], seen)


def _sparse(s):
    c, width = s["case"], s["table"].shape[1]
    used = (s["lens"][:, None, None] + c["page"] - 1) // c["page"]  # pages of each sequence
    j = torch.arange(width, device="cuda")[None, None]
    lo, hi = (s[name][s["table"].long()] if c["cache"] != "e4m3" else s[name].view(torch.uint8)[s["table"].long()].view(s[name].dtype) for name in ("k_min", "k_max"))
    lo, hi = lo.double().permute(0, 2, 3, 1), hi.double().permute(0, 2, 3, 1)  # [B, Hkv, d, width]
    q = s["q"].double().unflatten(1, (c["Hkv"], c["Hq"] // c["Hkv"]))
    # scores in 64 bits: two pages next to the border must not change places
    score = (q.clamp(min=0) @ hi + q.clamp(max=0) @ lo).amax(2)
    score = torch.where((j < c["first"]) | (j >= used - c["last"]), math.inf, score)
    score = torch.where(j < used, score, -math.inf)
    best = score.sort(dim=-1, descending=True, stable=True).indices[..., :c["select"]]
    if best.shape[-1] < c["select"]:
        best = torch.nn.functional.pad(best, (0, c["select"] - best.shape[-1]), value=width)
    best = torch.where(best < used, best, width).sort(dim=-1).values
    there = best < width
    table = s["table"][:, None].expand(-1, c["Hkv"], -1).gather(2, best.clamp(max=width - 1))
    key = best[..., None] * c["page"] + torch.arange(c["page"], device="cuda")
    seen = (there[..., None] & (key < s["lens"][:, None, None, None])).flatten(2)
    return {"pages": torch.where(there, best, -1).to(torch.int32), **_attend(s, table, seen)}


def work(case):
    c = case
    new, lens = _lens(c)
    e, d = SIZE[c["cache"]], c["D"]
    if c["op"] == "append":
        live = [(n, t) for n, t in zip(new, lens) if t]
        rows = sum(n for n, _ in live)
        size = rows * d * (2 * c["Hkv"] * (2 + e) + c["Hq"] * 4)
        spans, rotated = sorted((t - n, t) for n, t in live), 0
        end = 0
        for lo, hi in spans:  # positions that some row stands at: their table rows are read once
            rotated += max(0, hi - max(lo, end))
            end = max(end, hi)
        size += rotated * c["rot"] * 4 + c["B"] * 8 + sum(-(-t // c["page"]) - (t - n) // c["page"] for n, t in live) * 4
        if c["summary"]:
            size += sum(-(-t // c["page"]) - (t - n) // c["page"] + (1 if (t - n) % c["page"] else 0) for n, t in live) * 2 * c["Hkv"] * d * e
        return {"bytes": size, "flops": 3 * rows * c["rot"] * (c["Hq"] + c["Hkv"])}
    pages = [-(-t // c["page"]) for t in lens]
    flops = 0
    size = c["B"] * (c["Hq"] * (4 * d + 4) + 4)
    if c["op"] == "sparse":
        read = [t if p <= c["select"] else (c["select"] - 1) * c["page"] + (t - 1) % c["page"] + 1 for t, p in zip(lens, pages)]
        size += sum(p for p in pages if p > c["select"]) * c["Hkv"] * 2 * d * e + c["B"] * c["Hkv"] * c["select"] * 4
        flops += 4 * sum(p for p in pages if p > c["select"]) * c["Hq"] * d
    else:
        read = lens
    size += sum(read) * c["Hkv"] * 2 * d * e + sum(pages) * 4
    return {"bytes": size, "flops": flops + 4 * sum(read) * c["Hq"] * d}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    new, lens = _lens(c)
    table = s["table"].tolist() if sum(lens) < 3e6 else None
    if table is None:
        return None
    if c["op"] == "append":
        return _exact_append(c, s, new, lens, table)
    group, o, lse, chosen = c["Hq"] // c["Hkv"], [], [], []
    for b, n in enumerate(lens):
        if not n:
            o.append(torch.zeros(c["Hq"], c["D"], dtype=torch.float64, device="cuda"))
            lse.append(torch.full((c["Hq"],), -math.inf, dtype=torch.float64, device="cuda"))
            chosen.append(torch.full((c["Hkv"], c.get("select", 1)), -1, dtype=torch.int32, device="cuda"))
            continue
        used = -(-n // c["page"])
        ids = torch.tensor(table[b][:used], device="cuda")
        q = s["q"][b].double().reshape(c["Hkv"], group, c["D"])
        pick = torch.arange(used, device="cuda").expand(c["Hkv"], used)
        if c["op"] == "sparse":
            if used > c["select"]:
                lo, hi = (_take(s[name], ids).double().transpose(0, 1) for name in ("k_min", "k_max"))
                sums = torch.zeros(c["Hkv"], used, group, dtype=torch.float64, device="cuda")
                for i in range(group):
                    sums[..., i] = torch.maximum(q[:, None, i] * lo, q[:, None, i] * hi).sum(-1)
                rank = sums.max(-1).values
                rank[:, :c["first"]] = math.inf
                rank[:, max(0, used - c["last"]):] = math.inf
                pick = torch.argsort(rank, dim=1, descending=True, stable=True)[:, :c["select"]].sort(1).values
            row = torch.full((c["Hkv"], c["select"]), -1, dtype=torch.int32, device="cuda")
            row[:, :pick.shape[1]] = pick.to(torch.int32)
            chosen.append(row)
        heads = []
        for h in range(c["Hkv"]):
            at = ids[pick[h]]
            k = _take(s["k_pages"][:, h], at).double().reshape(-1, c["D"]) * s["k_scale"]
            v = _take(s["v_pages"][:, h], at).double().reshape(-1, c["D"]) * s["v_scale"]
            inside = (pick[h][:, None] * c["page"] + torch.arange(c["page"], device="cuda")).reshape(-1) < n
            logits = (q[h] @ k[inside].T) / math.sqrt(c["D"])
            heads.append((torch.softmax(logits, -1) @ v[inside], torch.logsumexp(logits, -1)))
        o.append(torch.cat([x[0] for x in heads]))
        lse.append(torch.cat([x[1] for x in heads]))
    out = {"o": torch.stack(o), "lse": torch.stack(lse)}
    if c["op"] == "sparse":
        out["pages"] = torch.stack(chosen)
    return out


def _take(x, at):
    return x.view(torch.uint8)[at].view(x.dtype) if x.dtype.itemsize == 1 else x[at]


def _exact_append(c, s, new, lens, table):
    k_out, v_out, q_out = s["k_pages"].double(), s["v_pages"].double(), s["q_out"].double()
    at = 0
    for b, (n, t) in enumerate(zip(new, lens)):
        rows, at = slice(at, at + n), at + n
        if not t:
            continue
        pos = torch.arange(t - n, t, device="cuda")
        ids = torch.tensor(table[b], device="cuda")[pos // c["page"]]
        turned = []
        for x in (s["k"][rows].double(), s["q"][rows].double()):
            r = c["rot"]
            if r:
                cos, sin = s["cos"][t - n:t].double()[:, None], s["sin"][t - n:t].double()[:, None]
                z = x[..., :r].unflatten(-1, (r // 2, 2)).movedim(-1, 0) if c["interleaved"] else x[..., :r].unflatten(-1, (2, r // 2)).movedim(-2, 0)
                z = torch.stack([z[0] * cos - z[1] * sin, z[1] * cos + z[0] * sin])
                z = z.movedim(0, -1).flatten(-2) if c["interleaved"] else z.movedim(0, -2).flatten(-2)
                x = torch.cat([z, x[..., r:]], -1)
            turned.append(x)
        k_out[ids, :, pos % c["page"]] = turned[0] / s["k_scale"]
        v_out[ids, :, pos % c["page"]] = s["v"][rows].double() / s["v_scale"]
        q_out[rows] = turned[1]
    out = {"q": q_out, "k_pages": k_out, "v_pages": v_out}
    if s["k_min"] is not None:  # of what is stored, and an exact minimum of it: no rounding of its own
        out["k_min"], out["k_max"] = s["k_min"].double(), s["k_max"].double()
        for n, t, ids in zip(new, lens, table):
            for j in range((t - n) // c["page"], -(-t // c["page"])) if t else ():
                k = k_out[ids[j], :, max(0, t - n - j * c["page"]):min(c["page"], t - j * c["page"])]
                whole = t - n <= j * c["page"]
                out["k_min"][ids[j]] = k.amin(1) if whole else torch.minimum(k.amin(1), out["k_min"][ids[j]])
                out["k_max"][ids[j]] = k.amax(1) if whole else torch.maximum(k.amax(1), out["k_max"][ids[j]])
    return out
