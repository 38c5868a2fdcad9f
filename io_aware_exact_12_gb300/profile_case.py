"""Runs one attention op a fixed number of times on synthetic inputs, for
capturing it under a profiler (ncu).  Warm-up launches come first, so a
capture can skip them with ``-s``.

  python -m io_aware_exact_12_gb300.profile_case --op fwd --B 2 --H 16 --N 8192 --d 128 --launches 2
  python -m io_aware_exact_12_gb300.profile_case --op bwd ...   (one attn_bwd = 3 launches)
  python -m io_aware_exact_12_gb300.profile_case --op naive ... (materialising 3-step
      torch comparator: S = QK^T, P = softmax(S), O = PV, to measure its DRAM bytes)
  --op fwd_dropout / bwd_dropout: the dropout entries with p = 0.1
  --op decode: one query token per head against an N-token cache (B, H, N, d)
  --op fwd_blocksparse / bwd_blocksparse: a seeded random 25 %-dense per-head
      block mask (diagonal on), as in bench.py
  --op fwd_fp8: the e4m3 forward (d = 128) on per-tensor-quantised inputs
  --op paged_append / paged_decode / paged_select: B sequences of N tokens in pages
      of 16, H key/value heads and 4 H query heads; append writes all N tokens with
      rotation and summaries, select takes an eighth of the pages; --dtype e4m3 for
      an 8-bit cache
  --op window_fwd / window_bwd: sliding window (--window, --sinks), H query heads and
      H / 4 key/value heads, token-major tensors (one window_bwd = 2 or 3 launches)
  --op paged_window: paged_decode with the window and the sinks
  --op paged_assign: the bookkeeping of N new tokens for each of B sequences
"""
from __future__ import annotations

import argparse
import math

import torch


def paged(attn, a):
    """The paged-cache ops on a cache whose pages lie in random order."""
    g = torch.Generator(device="cuda").manual_seed(4)
    page, pages = 16, (a.N + 15) // 16
    x = torch.bfloat16 if a.dtype == "e4m3" else {"bf16": torch.bfloat16, "f16": torch.float16}[a.dtype]
    cache = torch.float8_e4m3fn if a.dtype == "e4m3" else x
    randn = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=x)  # noqa: E731
    k, v = (randn(a.B * pages, a.H, page, a.d).to(cache) for _ in range(2))
    lo, hi = (f(k.to(x), 2).to(cache) for f in (torch.amin, torch.amax))
    table = torch.randperm(a.B * pages, generator=g, device="cuda").to(torch.int32).view(a.B, pages)
    kv = attn.PagedKV(k, v, table, torch.full((a.B,), a.N, dtype=torch.int32, device="cuda"), k_min=lo, k_max=hi)
    q = randn(a.B, 4 * a.H, a.d)
    if a.op == "paged_append":
        rows = randn(a.B * a.N, 6 * a.H, a.d)
        cos, sin = attn.rotation_tables(a.N, a.d, device="cuda")
        start = torch.arange(0, a.B * a.N + 1, a.N, dtype=torch.int32, device="cuda")
        out = torch.empty(a.B * a.N, 4 * a.H, a.d, dtype=x, device="cuda")
        run = lambda: attn.attn_paged_append(kv, rows[:, :a.H], rows[:, a.H:2 * a.H], q=rows[:, 2 * a.H:], q_out=out,  # noqa: E731
                                             token_start=start, cos=cos, sin=sin)
    elif a.op == "paged_decode":
        run = lambda: attn.attn_paged_decode(kv, q)  # noqa: E731
    elif a.op == "paged_window":
        run = lambda: attn.attn_paged_decode_window(kv, q, a.window, a.sinks)  # noqa: E731
    elif a.op == "paged_assign":
        i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        new, none, ring = kv.seq_lens.clone(), torch.zeros_like(kv.seq_lens), table.flatten().clone()
        free, after, slots = i32(0, ring.numel()), i32(0, 0), torch.zeros(a.B * a.N, dtype=torch.int64, device="cuda")
        run = lambda: attn.attn_paged_assign(kv, new, ring, free, lens=none, free_out=after, slots=slots)  # noqa: E731
    else:
        run = lambda: attn.attn_paged_select(kv, q, max(2, pages // 8))  # noqa: E731
    for _ in range(a.warmup + a.launches):
        run()
    torch.cuda.synchronize()
    st = attn.sync_status()
    print("done op=%s status=%d" % (a.op, st))
    return 1 if st else 0


def window(attn, a):
    """Both passes under a sliding window."""
    g = torch.Generator(device="cuda").manual_seed(4)
    x = {"bf16": torch.bfloat16, "f16": torch.float16}[a.dtype]
    q, k, v, do = (torch.randn((a.B, a.N, h, a.d), generator=g, device="cuda", dtype=x).transpose(1, 2)
                   for h in (a.H, max(1, a.H // 4), max(1, a.H // 4), a.H))
    o, lse = attn.attn_fwd_window(q, k, v, a.window, a.sinks)
    for _ in range(a.warmup + a.launches):
        if a.op == "window_fwd":
            attn.attn_fwd_window(q, k, v, a.window, a.sinks, o=o, lse=lse)
        else:
            attn.attn_bwd_window(q, k, v, o, do, lse, a.window, a.sinks)
    torch.cuda.synchronize()
    st = attn.sync_status()
    print("done op=%s status=%d" % (a.op, st))
    return 1 if st else 0


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--op", choices=["fwd", "bwd", "naive", "fwd_dropout", "bwd_dropout", "decode",
                                     "fwd_blocksparse", "bwd_blocksparse", "fwd_fp8", "paged_append",
                                     "paged_decode", "paged_select", "paged_window", "paged_assign", "window_fwd",
                                     "window_bwd"], default="fwd")
    ap.add_argument("--B", type=int, default=2)
    ap.add_argument("--H", type=int, default=16)
    ap.add_argument("--N", type=int, default=8192)
    ap.add_argument("--d", type=int, default=128)
    ap.add_argument("--causal", action="store_true")
    ap.add_argument("--window", type=int, default=1024)
    ap.add_argument("--sinks", type=int, default=4)
    ap.add_argument("--dtype", default="bf16")
    ap.add_argument("--warmup", type=int, default=2)
    ap.add_argument("--launches", type=int, default=2)
    a = ap.parse_args(argv)

    import io_aware_exact_12_gb300 as attn
    if a.op.startswith("paged"):
        return paged(attn, a)
    if a.op.startswith("window"):
        return window(attn, a)
    from io_aware_exact_12_gb300.synth import AttnShape, make_inputs
    x = make_inputs(AttnShape(a.B, a.H, a.N, a.d), a.dtype, seed=4, device="cuda")
    q, k, v, do = x["q"], x["k"], x["v"], x["do"]
    scale = 1.0 / math.sqrt(a.d)
    o, lse = attn.attn_fwd(q, k, v, scale=scale, causal=a.causal)
    if a.op.endswith("dropout"):
        o, lse = attn.attn_fwd_dropout(q, k, v, 0.1, 1234, 0, scale=scale, causal=a.causal)
    q1 = q[:, :, 0].contiguous()
    if a.op == "fwd_fp8":
        from io_aware_exact_12_gb300.synth import make_inputs_fp8
        x8 = make_inputs_fp8(AttnShape(a.B, a.H, a.N, a.d), seed=4)
        q8, k8, v8 = (x8[n][0].cuda() for n in ("q", "k", "v"))
        sq, sk, sv = x8["q"][1], x8["k"][1], x8["v"][1]
    if a.op.endswith("blocksparse"):
        nb = (a.N + 127) // 128
        g = torch.Generator().manual_seed(3)
        mask = (torch.rand((a.H, nb, nb), generator=g) < 0.25).to(torch.uint8)
        mask[:, torch.arange(nb), torch.arange(nb)] = 1
        mask = mask.cuda()
        o, lse = attn.attn_fwd_blocksparse(q, k, v, mask, scale=scale, causal=a.causal)

    def run():
        if a.op == "fwd_fp8":
            attn.attn_fwd_fp8(q8, k8, v8, sq, sk, sv, causal=a.causal, o=o, lse=lse)
        elif a.op == "fwd_blocksparse":
            attn.attn_fwd_blocksparse(q, k, v, mask, scale=scale, causal=a.causal, o=o, lse=lse)
        elif a.op == "bwd_blocksparse":
            attn.attn_bwd_blocksparse(q, k, v, o, do, lse, mask, scale=scale, causal=a.causal)
        elif a.op == "fwd_dropout":
            attn.attn_fwd_dropout(q, k, v, 0.1, 1234, 0, scale=scale, causal=a.causal, o=o, lse=lse)
        elif a.op == "bwd_dropout":
            attn.attn_bwd_dropout(q, k, v, o, do, lse, 0.1, 1234, 0, scale=scale, causal=a.causal)
        elif a.op == "decode":
            attn.attn_decode(q1, k, v, scale=scale)
        elif a.op == "fwd":
            attn.attn_fwd(q, k, v, scale=scale, causal=a.causal, o=o, lse=lse)
        elif a.op == "bwd":
            attn.attn_bwd(q, k, v, o, do, lse, scale=scale, causal=a.causal)
        else:
            s = torch.matmul(q, k.transpose(-2, -1)) * scale
            if a.causal:
                s = s.masked_fill(torch.ones(a.N, a.N, dtype=torch.bool, device=q.device).triu(1),
                                  float("-inf"))
            torch.matmul(torch.softmax(s, dim=-1), v)

    for _ in range(a.warmup):
        run()
    torch.cuda.synchronize()
    for _ in range(a.launches):
        run()
    torch.cuda.synchronize()
    st = attn.sync_status()
    print("done op=%s status=%d" % (a.op, st))
    return 1 if st else 0


if __name__ == "__main__":
    raise SystemExit(main())
