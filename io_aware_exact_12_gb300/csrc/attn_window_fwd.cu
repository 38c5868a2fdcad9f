// attn_window_fwd.cu -- causal attention with a sliding window and sinks,
// forward: O_i = sum_j softmax_j(scale q_i . k_j) v_j over the keys j <= p_i with
// j > p_i - window or j < sinks, query i standing at p_i = i + Nk - Nq.
//
// The online softmax of FlashAttention (PKM page), "三招" 1 and 2, over the key
// tiles that any row of a 128-row query tile sees: the tiles of sinks, then those
// from the first row's window to the last row's position.  No other tile is
// loaded or multiplied, and only the tiles at either edge of the window and those
// that end the sinks are masked, key by key.
//
// A tile's chain bounds it: S, the softmax of its rows, P, P V, each behind the one
// before, in two CTAs to an SM that cover one another in part.  A tile of 128 keys at
// d = 128 is 16 products of 128 x 128 x 16, 64 cycles each; where the list is long it
// goes by in 2000 cycles, the tensor pipe active 50 % of them (32768 queries, 32 / 8
// heads, window 4096: 1.81 ms, 1140 TFLOP/s of visible pairs).  At window 1024 it takes
// 2280 (42 %): edge tiles, half of which is hidden, and an item's start and end (8192
// queries: 152 us, 850).  At d = 128 the row threads spill 72 to 76 bytes, the clusters'
// form 40 to 56 at every d.  GB300 mapping:
//   * an item is 128 query rows of a head; two CTAs to an SM, so that one's softmax
//     meets the other's matrix products.  Blocks take over the items of blocks that
//     have not started (cluster launch control) and load the next item's first tiles
//     while this one's output is written: at window 1024 an item is ten tiles, and
//     starting a CTA, its first loads and its output took as long as three (8192
//     queries, 32 / 8 heads of 128: 165 -> 152 us).
//   * one warp loads (TMA, 4-D maps, so any strides of batch, head and row), one
//     thread issues the tcgen05.mma, S = Q K^T from shared memory, O += P V with P
//     from TMEM; a warpgroup does the softmax, a thread to a row.  (Two threads to a
//     row, who exchange its maximum, gained nothing at d = 64, where the products pace
//     it too, and do not have the registers at d = 128.)
//   * few items with long lists of tiles (a chunk of a prompt, a handful of tokens): a
//     cluster to an item (SPLIT), its positions in equal runs, joined in the order of
//     the runs through the cluster's shared memory (16 queries of 32 heads over window
//     4096: 58 -> 19 us; one over 32768 keys: 419 -> 72).
//   * few sinks (kNarrow at most in their last tile): that tile's S is formed for 32
//     keys and its P V summed over 32 (4 sinks, window 1024: 157 -> 151 us; 16384
//     queries, 16 / 4 heads, window 256: 93 -> 79).
//   * scale log2(e) is folded into exp2; the reference maximum moves only when it
//     grows by more than 2^8, and O is rescaled in TMEM then.  l is summed twice:
//     in fp32 of the weights as they are, for LSE, and of the weights rounded to the
//     input type that multiply V, to normalise O.  (Weights of 16 bits are what a
//     16-bit product takes; O is off by 2.2e-3 in norm with bf16, where fp32 weights
//     and O's own rounding make 1.6e-3; a second product with the remainders would
//     double P V.)
#include <cfloat>
#include <type_traits>

#include "attn_internal.h"
#include "attn_window_tiles.cuh"

namespace attn {
namespace {

constexpr float kRescaleLog2 = 8.0f;
constexpr int kNarrow = 32;  // keys of a tile with a few sinks
constexpr int kParts = 8;     // blocks to an item, at most
// Weights are 2^kShift at the maximum.  fp16 ends at 2^16 and is normal from 2^-14 on:
// with 2^7 under a maximum that may lie 2^8 behind, weights keep their bits down to
// 2^-21 of the largest, as those beside a sink are that holds nearly all of it, where
// 2^0 keeps them to 2^-14.  bf16 has fp32's range.
template <bool BF16>
constexpr float kShift = BF16 ? 0.f : 7.f;
template <bool BF16>
constexpr float kUnshift = BF16 ? 1.f : 1.f / 128;  // 2^-kShift

template <int D>
struct WfCfg : TileLayout<D> {
  using T = TileLayout<D>;
  static constexpr int NST = D == 128 ? 1 : 2;  // K and V stages
  static constexpr int OFF_K = T::TILE;
  static constexpr int OFF_V = OFF_K + NST * T::TILE;
  static constexpr int OFF_BAR = OFF_V + NST * T::TILE;
  static constexpr int B_Q = 0;
  static constexpr int B_QEMPTY = 1;
  static constexpr int B_KFULL = 2;
  static constexpr int B_KEMPTY = B_KFULL + NST;
  static constexpr int B_VFULL = B_KEMPTY + NST;
  static constexpr int B_VEMPTY = B_VFULL + NST;
  static constexpr int B_S = B_VEMPTY + NST;  // S is in TMEM
  static constexpr int B_P = B_S + 1;         // P is in TMEM
  static constexpr int B_O = B_P + 1;         // P V is complete
  static constexpr int B_TAKEN = B_O + 1;     // S is in registers (P apart)
  static constexpr int B_NEXT = B_TAKEN + 1;   // the next item is known
  static constexpr int B_READ = B_NEXT + 2;    // and read by all
  static constexpr int B_DONE = B_READ + 2;
  static constexpr int NBAR = B_DONE + 1;
  static constexpr int OFF_NEXT = (OFF_BAR + NBAR * 8 + 15) & ~15;  // two answers
  static constexpr int OFF_SLOT = OFF_NEXT + 32;
  static constexpr int OFF_ABORT = OFF_SLOT + 4;
  // Staging of the output at d = 128: half a row for each of a warp's 32.
  static constexpr bool STAGE = D == 128;
  static constexpr int OFF_STAGE = (OFF_ABORT + 4 + 15) & ~15;
  static constexpr int SMEM = OFF_STAGE + (STAGE ? 4 * 32 * 128 : 0);
  static constexpr int THREADS = 256;
  static constexpr int W_LOAD = 4, W_MMA = 5;  // warps
  static constexpr int CTAS = 2;                // per SM
  static constexpr int REGS = (65536 / (THREADS * CTAS)) & ~7;
  static constexpr int REGS_ROW = D == 128 ? 200 : 208, REGS_CTRL = D == 128 ? 56 : 48;
  static_assert(128 * REGS_ROW + 128 * REGS_CTRL <= THREADS * REGS, "register split");
  static constexpr uint32_t COLS = 256;
  // P has TMEM columns of its own at d <= 64: the next S can then be formed while
  // P V is pending.  At d = 128 the columns are full and P lies over half of S.
  static constexpr bool APART = D <= 64;
  static constexpr uint32_t T_O = 128;
  static constexpr uint32_t T_P = APART ? 128 + D : 0;
  static_assert(128 + D + (APART ? 64 : 0) <= COLS, "TMEM");
  static_assert(CTAS * (SMEM + 1024) <= 233472, "shared memory");
};

// Byte offset of 16-byte unit u of a row of 128 bytes in the output's staging
// copy, swizzled so that rows by threads and units by threads meet no bank twice.
__device__ __forceinline__ uint32_t staged(int row, int u) { return static_cast<uint32_t>(row * 128 + ((u ^ (row & 7)) << 4)); }

// SPLIT: a cluster of `parts` blocks to an item, each with its share of the positions.
template <int D, bool BF16, bool SPLIT>
__global__ void __launch_bounds__(WfCfg<D>::THREADS, WfCfg<D>::CTAS)
    attn_window_fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                           const __grid_constant__ CUtensorMap mv, const WindowArgs a, int nrows, int group, int parts) {
  using C = WfCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sbase = smem_addr(smem);
  if (sbase & 1023u) {  // the swizzle's atoms; never expected
    if (threadIdx.x == 0) atomicExch(a.status, kStatusDeviceCheck);
    return;
  }
  auto bar = [&](int i) -> uint32_t { return sbase + C::OFF_BAR + 8u * static_cast<uint32_t>(i); };
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + C::OFF_SLOT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
  const uint32_t sK = sbase + C::OFF_K, sV = sbase + C::OFF_V;
  if (warp == C::W_LOAD && lane == 0) {
    for (int x = 0; x < C::NBAR; ++x) mbar_init(bar(x), 1);
    mbar_init(bar(C::B_P), 128);
    mbar_init(bar(C::B_TAKEN), 128);
    for (int x = 0; x < 2; ++x) mbar_init(bar(C::B_READ + x), 5);  // the softmax warps and the issuer
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&mq);
    prefetch_tensormap(&mk);
    prefetch_tensormap(&mv);
  }
  if (warp == C::W_MMA) {
    tmem_alloc(smem_addr(slot), C::COLS);
    tmem_relinquish();
  }
  griddep_wait();  // launched overlapped (launch_serialized): what is above reads no tensor
  griddep_launch_dependents();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *slot;
  const Items items = {sbase + C::OFF_NEXT, bar(C::B_NEXT), bar(C::B_READ), abort_flag, a.status};
  const int first_item = SPLIT ? blockIdx.x / parts : blockIdx.x, part = SPLIT ? blockIdx.x % parts : 0;
  auto from = [&](const RowItem& it) { return SPLIT ? it.npos * part / parts : 0; };
  auto upto = [&](const RowItem& it) { return SPLIT ? it.npos * (part + 1) / parts : it.npos; };
  // `n` counts positions over all items and gives stages and phases.
  // The last tile of sinks may have few of them: then kNarrow of its keys are enough.
  auto narrow = [&](const RowItem& it, int p) { return p == it.ns - 1 && a.sinks - p * 128 <= kNarrow; };

  if (warp >= C::W_LOAD) {
    regs_decrease<C::REGS_CTRL>();
    if (warp == C::W_LOAD && lane == 0) {
      // ------------------------------------------------------------ loads
      auto load = [&](uint32_t dst, const CUtensorMap* map, uint32_t full, int row, int head, int b) {
#pragma unroll
        for (int c = 0; c < C::NCH; ++c) tma_load_4d(dst + c * C::CHUNK, map, full, c * C::CH, row, head, b);
      };
      int nk = 0, nv = 0, nq = 0;  // issued
      bool ok = true;
      int asked = 0;
      for (int i = first_item; ok && i >= 0;) {
        if (!SPLIT) {
          if (!(ok = items.ask(asked))) break;
          ++asked;
        }
        const RowItem it(a, i, nrows, group);
        const int p0 = from(it), p1 = upto(it);
        for (int p = p0; p < p1; ++p) {
          const int s = nk % C::NST, turn = (nk / C::NST - 1) & 1;
          if (nk >= C::NST && !(ok = mbar_wait(bar(C::B_KEMPTY + s), turn, abort_flag, a.status))) break;
          mbar_arrive_expect_tx(bar(C::B_KFULL + s), C::TILE);
          load(sK + s * C::TILE, &mk, bar(C::B_KFULL + s), it.key0(p), it.hk, it.b);
          ++nk;
          if (p == p0) {
            if (nq > 0 && !(ok = mbar_wait(bar(C::B_QEMPTY), (nq - 1) & 1, abort_flag, a.status))) break;
            mbar_arrive_expect_tx(bar(C::B_Q), C::TILE);
            load(sbase, &mq, bar(C::B_Q), it.row0, it.h, it.b);
            ++nq;
          }
          if (nv >= C::NST && !(ok = mbar_wait(bar(C::B_VEMPTY + s), turn, abort_flag, a.status))) break;
          mbar_arrive_expect_tx(bar(C::B_VFULL + s), C::TILE);
          load(sV + s * C::TILE, &mv, bar(C::B_VFULL + s), it.key0(p), it.hk, it.b);
          ++nv;
        }
        i = SPLIT ? -1 : items.after(asked - 1, ok);
      }
      if (*abort_flag) {  // what is in flight lands before the shared memory goes
        items.drain_last(asked);
        if (nq) drain(bar(C::B_Q), (nq - 1) & 1);
        for (int s = 0; s < C::NST; ++s) {
          if (nk > s) drain(bar(C::B_KFULL + s), ((nk - 1 - s) / C::NST) & 1);
          if (nv > s) drain(bar(C::B_VFULL + s), ((nv - 1 - s) / C::NST) & 1);
        }
      }
    } else if (warp == C::W_MMA && lane == 0) {
      // ----------------------------------------------- matrix instructions
      // A chain S, P V, S, P V, ...; whichever next step is ready goes out.  At d = 128
      // S(p + 1) overwrites the P that P V(p) reads, so it waits for that to complete:
      // MMAs run in the order of issue where they have one accumulator, no others are
      // promised to.  (The wait costs nothing that shows with bf16, 0.7 % with fp16.)  K
      // and V stages and Q are handed back by the softmax, whose waits tell when the MMAs that read
      // them are complete.  An item's first P V overwrites the O of the one before,
      // which the threads that wrote this P have read.
      constexpr uint32_t HI = smem_desc_hi(C::SBO, C::SWZ);
      const uint32_t id_s = instr_desc_f16(128, 128, BF16, false, false, a.negate != 0);
      const uint32_t id_sn = instr_desc_f16(128, kNarrow, BF16, false, false, a.negate != 0);
      const uint32_t id_o = instr_desc_f16(128, D, BF16, false, true);
      bool ok = true;
      int n0 = 0;  // positions of the items before
      IdleWatch watch;
      for (int i = first_item, k = 0; ok && i >= 0; ++k) {
        const RowItem it(a, i, nrows, group);
        const int p0 = from(it), end = n0 + upto(it) - p0, thin = it.ns > 0 && narrow(it, it.ns - 1) ? n0 + it.ns - 1 - p0 : -1;
        if (!SPLIT || n0 < end) ok = mbar_wait(bar(C::B_Q), k & 1, abort_flag, a.status);
        int js = n0, jp = n0;          // next S and P V
        int k_seen = n0, v_seen = n0;  // positions whose loads have been seen to land
        const uint32_t q_lo = smem_desc_lo(sbase, 16);
        while (ok && jp < end) {
          bool progress = false;
          const int sv = jp % C::NST;
          if (jp < js && mbar_probe(bar(C::B_P), jp & 1) && (jp < v_seen || mbar_probe(bar(C::B_VFULL + sv), (jp / C::NST) & 1))) {
            v_seen = max(v_seen, jp + 1);
            tc_fence_after_sync();
            const uint32_t v_lo = smem_desc_lo(sV + sv * C::TILE, C::CHUNK);
#pragma unroll
            for (int kk = 0; kk < kNarrow / 16; ++kk)
              mma_ts_w(tmem + C::T_O, tmem + C::T_P + kk * 8, v_lo + mn_step<D>(kk), HI, id_o, (jp > n0 || kk > 0) ? 1u : 0u);
            if (jp != thin) {
#pragma unroll
              for (int kk = kNarrow / 16; kk < 8; ++kk) mma_ts_w(tmem + C::T_O, tmem + C::T_P + kk * 8, v_lo + mn_step<D>(kk), HI, id_o, 1u);
            }
            tc_commit(bar(C::B_O));
            ++jp;
            progress = true;
          }
          const int sk = js % C::NST;
          if (js < end && (js == 0 || (C::APART ? mbar_probe(bar(C::B_TAKEN), (js - 1) & 1) : js == jp && mbar_probe(bar(C::B_O), (js - 1) & 1))) &&
              (js < k_seen || mbar_probe(bar(C::B_KFULL + sk), (js / C::NST) & 1))) {
            k_seen = max(k_seen, js + 1);
            tc_fence_after_sync();
            const uint32_t k_lo = smem_desc_lo(sK + sk * C::TILE, 16), id = js == thin ? id_sn : id_s;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) mma_ss_w(tmem, q_lo + k_step<D>(kk), HI, k_lo + k_step<D>(kk), HI, id, kk > 0 ? 1u : 0u);
            tc_commit(bar(C::B_S));
            ++js;
            progress = true;
          }
          if (progress) watch.progress();
          else ok = watch.idle(abort_flag, a.status, kWaitLimitNs);
        }
        n0 = end;
        if (SPLIT) break;
        i = items.after(k, ok);
        items.read(k);
      }
      tc_commit(bar(C::B_DONE));  // before TMEM is released
      drain(bar(C::B_DONE), 0);
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------------- softmax
    regs_increase<C::REGS_ROW>();
    const int r = threadIdx.x;
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tS = tmem + lanes, tO = tmem + lanes + C::T_O, tP = tmem + lanes + C::T_P;
    const float sl2 = fmaxf(a.sl2, FLT_MIN);  // a scale of 0: hidden keys are -inf, and that times 0 is NaN
    const float2 sl2x2 = make_float2(sl2, sl2);
    const int off = a.Nk - a.Nq, wnd = a.window, nsk = a.sinks;
    auto release = [&](int first, int n) {
      if (r == 0) mbar_arrive(bar(first + n % C::NST));
    };
    bool ok = true;
    int n = 0;
    for (int i = first_item, k = 0; ok && i >= 0; ++k) {
      const RowItem it(a, i, nrows, group);
      const int p0 = from(it), p1 = upto(it), row = it.row0 + r;
      float m = -INFINITY, l_exact = 0.f, l_round = 0.f;
      // A position with W of its tile's keys.
      auto step = [&](int p, auto width) {
        constexpr int W = decltype(width)::value;
        // (a warp's lanes go on or stop together: they vote below)
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_S), n & 1, abort_flag, a.status)))) return;
        tc_fence_after_sync();
        if (r == 0) {
          mbar_arrive(bar(C::B_KEMPTY + n % C::NST));
          if (!C::APART && p > p0) mbar_arrive(bar(C::B_VEMPTY + (n - 1) % C::NST));
          if (p == p1 - 1) mbar_arrive(bar(C::B_QEMPTY));
        }
        float sv[W];
        if constexpr (W == 128) {
          uint32_t u[64];
          tmem_ld64(tS, u);
#pragma unroll
          for (int c = 0; c < 64; ++c) sv[c] = __uint_as_float(u[c]);
          tmem_ld64(tS + 64, u);
#pragma unroll
          for (int c = 0; c < 64; ++c) sv[64 + c] = __uint_as_float(u[c]);
        } else {
          uint32_t u[32];
          tmem_ld32(tS, u);
#pragma unroll
          for (int c = 0; c < 32; ++c) sv[c] = __uint_as_float(u[c]);
        }
        if constexpr (C::APART) {
          tc_fence_before_sync();
          mbar_arrive(bar(C::B_TAKEN));
        }
        // Key kv0 + c is visible iff c <= at and (c >= first or c < sinks).
        const int kv0 = it.key0(p);
        const int at = row + off - kv0;
        const bool right = kv0 + 127 > it.row0 + off;
        const bool left = kv0 < it.row0 + 127 + off - wnd + 1 && kv0 + W > nsk;
        if (right) {
#pragma unroll
          for (int c = 0; c < W; ++c)
            if (c > at) sv[c] = -INFINITY;
        }
        if (left) {
          const int first = at - wnd + 1, sinks = nsk - kv0;
#pragma unroll
          for (int c = 0; c < W; ++c)
            if (c < first && c >= sinks) sv[c] = -INFINITY;
        }
        float mx;
        {
          float a0 = sv[0], a1 = sv[1], a2 = sv[2], a3 = sv[3];
#pragma unroll
          for (int c = 4; c + 8 <= W; c += 8) {
            a0 = max3f(a0, sv[c], sv[c + 1]);
            a1 = max3f(a1, sv[c + 2], sv[c + 3]);
            a2 = max3f(a2, sv[c + 4], sv[c + 5]);
            a3 = max3f(a3, sv[c + 6], sv[c + 7]);
          }
          a0 = max3f(a0, sv[W - 4], sv[W - 3]);
          a1 = max3f(a1, sv[W - 2], sv[W - 1]);
          mx = fmaxf(fmaxf(a0, a1), fmaxf(a2, a3));
        }
        const float m_new = fmaxf(m, mx * sl2);
        float alpha = 1.f;
        if (m_new > m + kRescaleLog2) {  // also with the row's first visible key (m = -inf)
          alpha = ex2_approx(m - m_new);
          m = m_new;
        }
        const float neg_m = m == -INFINITY ? 0.f : BF16 ? -m : kShift<BF16> - m;
        const float2 nm2 = make_float2(neg_m, neg_m);
#pragma unroll
        for (int c = 0; c < W; c += 2) {
          const float2 t = fma2(make_float2(sv[c], sv[c + 1]), sl2x2, nm2);
          sv[c] = ex2_approx(t.x);
          sv[c + 1] = ex2_approx(t.y);
        }
        if (C::APART && p > p0) {  // P V(n - 1) is complete: P may be written, O is what it will be
          ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_O), (n - 1) & 1, abort_flag, a.status));
          if (!ok) return;
          tc_fence_after_sync();
          release(C::B_VEMPTY, n - 1);
        }
        if (p > p0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
          for (int c0 = 0; c0 < D / 32; ++c0) {
            uint32_t ov[32];
            tmem_ld32(tO + c0 * 32, ov);
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
            tmem_st32(tO + c0 * 32, ov);
          }
        }
        // P goes out first, the sums follow while P V runs.
        uint32_t pk[W / 64 + 1][32];
#pragma unroll
        for (int x = 0; x < (W + 63) / 64; ++x) {
#pragma unroll
          for (int e = 0; e < 32; ++e) pk[x][e] = x * 64 + 2 * e < W ? pack2<BF16>(sv[(x * 64 + 2 * e) % W], sv[(x * 64 + 2 * e + 1) % W]) : 0u;
          tmem_st32(tP + x * 32, pk[x]);
        }
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(bar(C::B_P));
        float2 e0 = make_float2(0.f, 0.f), e1 = e0;
        float r0 = 0.f, r1 = 0.f, r2 = 0.f, r3 = 0.f;
#pragma unroll
        for (int c = 0; c < W; c += 4) {
          e0 = add2(e0, make_float2(sv[c], sv[c + 1]));
          e1 = add2(e1, make_float2(sv[c + 2], sv[c + 3]));
        }
#pragma unroll
        for (int e = 0; e < W / 4; e += 2) {
          r0 = add_halves<BF16>(r0, pk[0][e]);
          r1 = add_halves<BF16>(r1, pk[0][e + 1]);
          r2 = add_halves<BF16>(r2, W == 128 ? pk[W / 128][e] : pk[0][W / 4 + e]);
          r3 = add_halves<BF16>(r3, W == 128 ? pk[W / 128][e + 1] : pk[0][W / 4 + e + 1]);
        }
        l_exact = l_exact * alpha + ((e0.x + e0.y) + (e1.x + e1.y));
        l_round = l_round * alpha + ((r0 + r1) + (r2 + r3));
        ++n;
      };
      for (int p = p0; ok && p < p1; ++p) {
        if (narrow(it, p)) step(p, std::integral_constant<int, kNarrow>{});
        else step(p, std::integral_constant<int, 128>{});
      }
      if constexpr (SPLIT) {
        // O as it is, in fp32, m and l, where Q, K and V were, whose loads and products are
        // complete; 16 bytes of a warp's rows side by side.
        if (p1 > p0 && ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_O), (n - 1) & 1, abort_flag, a.status));
        tc_fence_after_sync();
        float* mine = reinterpret_cast<float*>(smem);
        if (p1 > p0 && ok) {
#pragma unroll
          for (int c0 = 0; c0 < D / 32; ++c0) {
            uint32_t ov[32];
            tmem_ld32(tO + c0 * 32, ov);
#pragma unroll
            for (int e = 0; e < 8; ++e) reinterpret_cast<uint4*>(mine)[(c0 * 8 + e) * 128 + r] = make_uint4(ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]);
          }
        }
        mine[128 * D + r] = ok ? m : -INFINITY, mine[128 * D + 128 + r] = l_exact, mine[128 * D + 256 + r] = l_round;
        break;
      }
      // -------------------------------------------------------------- output
      ok = __all_sync(0xffffffffu, ok && mbar_wait(bar(C::B_O), (n - 1) & 1, abort_flag, a.status));
      if (!ok) break;
      tc_fence_after_sync();
      release(C::B_VEMPTY, n - 1);
      const float inv = 1.0f / l_round;
      uint8_t* stage = smem + C::OFF_STAGE + warp * 32 * 128;
      uint8_t* out = a.o.p + it.b * a.o.b + it.h * a.o.h;
#pragma unroll
      for (int c0 = 0; c0 < D / 32; ++c0) {
        uint32_t ov[32], pk[16];
        tmem_ld32(tO + c0 * 32, ov);
#pragma unroll
        for (int e = 0; e < 16; ++e) pk[e] = pack2<BF16>(__uint_as_float(ov[2 * e]) * inv, __uint_as_float(ov[2 * e + 1]) * inv);
        if (C::STAGE || row < a.Nq) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4*>(C::STAGE ? stage + staged(lane, (c0 & 1) * 4 + e) : out + row * a.o.n + c0 * 64 + e * 16) =
                make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
        }
        if (C::STAGE && (c0 & 1)) {  // half a row of each of the warp's: whole 128-byte lines
          __syncwarp();
          const int row_w = it.row0 + (r & ~31);
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const int rr = x * 4 + (lane >> 3), u = lane & 7;
            const uint4 val = *reinterpret_cast<const uint4*>(stage + staged(rr, u));
            if (row_w + rr < a.Nq) *reinterpret_cast<uint4*>(out + (row_w + rr) * a.o.n + (c0 >> 1) * 128 + u * 16) = val;
          }
          __syncwarp();
        }
      }
      if (row < a.Nq) a.lse[(static_cast<int64_t>(it.b) * a.Hq + it.h) * a.Nq + row] = (m + log2f(l_exact * kUnshift<BF16>)) * 0.69314718055994531f;
      tc_fence_before_sync();  // O is read before this thread's next P lets it be overwritten
      i = items.after(k, ok);
      items.read_by_warp(k, lane, ok);
    }
  }
  if constexpr (SPLIT) {
    static_assert(128 * D * 4 + 3 * 512 <= C::OFF_BAR, "a part's results");
    cluster_sync();
    if (warp < C::W_LOAD) {
      // A block has 128 / parts of the rows, a thread D / parts channels of one; parts in order.
      const RowItem it(a, first_item, nrows, group);
      const int rows = 128 / parts, rr = part * rows + threadIdx.x % rows, row = it.row0 + rr;  // (parts is a power of two)
      const int c0 = threadIdx.x / rows * (D / 4 / parts), c1 = c0 + D / 4 / parts;              // in fours
      if (row < a.Nq) {
        float f[kParts], e[kParts], l[kParts], m = -INFINITY, l_exact = 0.f, l_round = 0.f;
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
          const uint32_t at = in_block(sbase, k < parts ? k : 0) + (128 * D + rr) * 4;
          f[k] = load_cluster4(at), e[k] = load_cluster4(at + 512), l[k] = load_cluster4(at + 1024);
          if (k >= parts) f[k] = -INFINITY;
        }
#pragma unroll
        for (int k = 0; k < kParts; ++k) m = fmaxf(m, f[k]);
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
          f[k] = f[k] == -INFINITY ? 0.f : ex2_approx(f[k] - m);  // 0: sees none of this row's keys
          l_exact += f[k] * e[k], l_round += f[k] * l[k];
        }
        const float inv = 1.0f / l_round;
        uint8_t* out = a.o.p + it.b * a.o.b + it.h * a.o.h + row * a.o.n;
        for (int c = c0; c < c1; c += 2) {  // (an odd one out at the end goes alone)
          float o[8] = {};
#pragma unroll
          for (int k = 0; k < kParts; ++k) {
            if (f[k] == 0.f) continue;  // also where there is no O
            const uint32_t at = in_block(sbase, k) + rr * 16;
            const float4 u = load_cluster16(at + c * 2048), v = load_cluster16(at + min(c + 1, c1 - 1) * 2048);
            o[0] += f[k] * u.x, o[1] += f[k] * u.y, o[2] += f[k] * u.z, o[3] += f[k] * u.w;
            o[4] += f[k] * v.x, o[5] += f[k] * v.y, o[6] += f[k] * v.z, o[7] += f[k] * v.w;
          }
          *reinterpret_cast<uint2*>(out + c * 8) = make_uint2(pack2<BF16>(o[0] * inv, o[1] * inv), pack2<BF16>(o[2] * inv, o[3] * inv));
          if (c + 1 < c1)
            *reinterpret_cast<uint2*>(out + c * 8 + 8) = make_uint2(pack2<BF16>(o[4] * inv, o[5] * inv), pack2<BF16>(o[6] * inv, o[7] * inv));
        }
        if (c0 == 0) a.lse[(static_cast<int64_t>(it.b) * a.Hq + it.h) * a.Nq + row] = (m + log2f(l_exact * kUnshift<BF16>)) * 0.69314718055994531f;
      }
    }
    cluster_sync();  // nobody's shared memory goes before it is read
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == C::W_MMA) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::COLS);
  }
}

// Blocks to an item, a power of two: as many as the GPU holds, two to an SM, if that
// takes enough positions out of the longest item's chain.  A position in one CTA takes
// 0.9 (d = 32) to 1.2 us (128), the join 2 to 3 us, more with two CTAs to every SM and most
// with two parts, who have the most rows each to join.  128 queries, d = 128, one block
// and several: 8 heads, window 256 14.0 and 12.4 us, 1024 23.2 and 12.2, 4096 58.2 and
// 16.5; 64 heads, window 256 14.1 and 16.9, 512 17.2 and 17.8, 768 20.4 and 18.7; 120
// heads, window 1024 24.0 and 26.1, 2048 36.4 and 33.6.
int parts_of(const WindowArgs& a, int64_t items) {
  const int64_t most = std::min<int64_t>((a.Nk + 127) / 128, (a.window + 254) / 128 + 1 + (a.sinks + 127) / 128);  // positions
  const int64_t sms = device_sm_count();
  int parts = 1;
  while (parts < kParts && items * parts * 2 <= 2 * sms && most >= 2 * parts) parts *= 2;
  const int least = items * parts <= sms ? 3 : parts > 2 ? 6 : 8;
  return most - (most + parts - 1) / parts >= least ? parts : 1;
}

template <int D, bool BF16>
int launch_t(const WindowArgs& a) {
  using C = WfCfg<D>;
  CUtensorMap mq, mk, mv;
  if (!encode_strided_map(&mq, a.q, a.B, a.Hq, a.Nq, D, C::CH, BF16) || !encode_strided_map(&mk, a.k, a.B, a.Hk, a.Nk, D, C::CH, BF16) ||
      !encode_strided_map(&mv, a.v, a.B, a.Hk, a.Nk, D, C::CH, BF16))
    return kStatusCuda;
  const int nrows = (a.Nq + 127) / 128, heads = a.B * a.Hq;
  const int64_t items = static_cast<int64_t>(nrows) * heads;
  if (items > 0x7fffffff) return kStatusUnsupported;
  const int parts = parts_of(a, items);
  auto kern = parts > 1 ? attn_window_fwd_kernel<D, BF16, true> : attn_window_fwd_kernel<D, BF16, false>;
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kern), C::SMEM)) return kStatusCuda;
  if (!check_launch_regs(reinterpret_cast<const void*>(kern), C::REGS)) return kStatusDeviceCheck;  // the split's sum
  const int group = order_head_group(heads, int64_t{4} * a.Nk * D, int64_t{128} << 20);
  return launch_clusters(parts, kern, static_cast<unsigned>(items * parts), C::THREADS, C::SMEM, a.stream, mq, mk, mv, a, nrows, group, parts) ==
                 cudaSuccess
             ? kStatusOk
             : kStatusCuda;
}

template <int D>
int launch_d(const WindowArgs& a) {
  return a.bf16 ? launch_t<D, true>(a) : launch_t<D, false>(a);
}

}  // namespace

int launch_window_fwd(const WindowArgs& a, int* launches) {
  *launches = 1;
  return a.d == 32 ? launch_d<32>(a) : a.d == 64 ? launch_d<64>(a) : launch_d<128>(a);
}

}  // namespace attn
