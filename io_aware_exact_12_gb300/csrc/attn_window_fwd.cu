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
// The tensor cores bound it (4 d flops a pair against 4 d bytes a key for 128
// rows).  GB300 mapping:
//   * a CTA takes NQ tiles of 128 query rows: one, with two CTAs to an SM, or the
//     same rows of two query heads that share a key/value head, which then share
//     every tile that is loaded.  Their tile lists are the same, so neither walks
//     tiles that only the other needs (two tiles of neighbouring rows would).
//   * one warp loads (TMA, 4-D maps, so any strides of batch, head and row), one
//     thread issues the tcgen05.mma, S = Q K^T from shared memory, O += P V with P
//     from TMEM; a warpgroup to each query tile does its softmax, a thread to a row.
//   * scale log2(e) is folded into exp2; the reference maximum moves only when it
//     grows by more than 2^8, and O is rescaled in TMEM then.  l is summed twice:
//     in fp32 of the weights as they are, for LSE, and of the weights rounded to the
//     input type that multiply V, to normalise O.
#include "attn_internal.h"
#include "attn_window.h"
#include "tc_sm103.cuh"

namespace attn {
namespace {

constexpr float kRescaleLog2 = 8.0f;

template <int D, int NQ>
struct WfCfg {
  static constexpr int ROWB = D >= 64 ? 128 : 64;  // bytes of a swizzled row
  static constexpr int CH = ROWB / 2;              // elements of it
  static constexpr int NCH = D / CH;               // column chunks of a tile
  static constexpr uint32_t SWZ = ROWB == 128 ? kSwizzle128B : kSwizzle64B;
  static constexpr int SBO = 8 * ROWB;
  static constexpr int CHUNK = 128 * ROWB;         // bytes of a chunk of 128 rows
  static constexpr int TILE = 128 * D * 2;
  static constexpr int NST = NQ == 1 && D == 128 ? 1 : 2;  // K and V stages
  static constexpr int OFF_K = NQ * TILE;
  static constexpr int OFF_V = OFF_K + NST * TILE;
  static constexpr int OFF_BAR = OFF_V + NST * TILE;
  static constexpr int B_Q = 0;
  static constexpr int B_KFULL = 1;
  static constexpr int B_KEMPTY = B_KFULL + NST;
  static constexpr int B_VFULL = B_KEMPTY + NST;
  static constexpr int B_VEMPTY = B_VFULL + NST;
  static constexpr int B_S = B_VEMPTY + NST;  // S_q is in TMEM
  static constexpr int B_P = B_S + 2;         // P_q is in TMEM
  static constexpr int B_O = B_P + 2;         // P_q V is complete
  static constexpr int B_TAKEN = B_O + 2;     // S_q is in registers (P apart)
  static constexpr int B_DONE = B_TAKEN + 2;
  static constexpr int NBAR = B_DONE + 1;
  static constexpr int OFF_SLOT = OFF_BAR + NBAR * 8;
  static constexpr int OFF_ABORT = OFF_SLOT + 4;
  static constexpr int SMEM = OFF_ABORT + 4;
  static constexpr int THREADS = 128 * NQ + 128;
  static constexpr int W_LOAD = 4 * NQ, W_MMA = 4 * NQ + 1;  // warps
  static constexpr int CTAS = 3 - NQ;                        // per SM
  static constexpr int REGS = (65536 / (THREADS * CTAS)) & ~7;
  static constexpr int REGS_ROW = NQ == 2 ? 224 : 208, REGS_CTRL = NQ == 2 ? 56 : 48;
  static_assert(NQ * 128 * REGS_ROW + 128 * REGS_CTRL <= THREADS * REGS, "register split");
  static constexpr uint32_t COLS = NQ == 2 ? 512 : 256;
  // P has TMEM columns of its own at d <= 64: the next S can then be formed while
  // P V is pending.  At d = 128 the columns are full and P lies over half of S.
  static constexpr bool APART = D <= 64;
  static constexpr uint32_t T_O = NQ * 128;                        // + D q
  static constexpr uint32_t T_P = APART ? NQ * 128 + NQ * D : 0;   // + T_PSTEP q
  static constexpr uint32_t T_PSTEP = APART ? 64 : 128;
  static_assert(NQ * 128 + NQ * D + (APART ? NQ * 64 : 0) <= COLS, "TMEM");
  static_assert(CTAS * (SMEM + 1024) <= 233472, "shared memory");
};

// Descriptor steps (16-byte units) of the 16-deep slice kk: of a K-major tile
// (rows of D channels) and of an MN-major one (16 rows on).
template <int D>
__host__ __device__ constexpr uint32_t k_step(int kk) {
  using C = WfCfg<D, 1>;
  return static_cast<uint32_t>(((kk * 16) / C::CH * C::CHUNK + (kk * 16) % C::CH * 2) >> 4);
}
template <int D>
__host__ __device__ constexpr uint32_t mn_step(int kk) {
  return static_cast<uint32_t>((kk * 16 * WfCfg<D, 1>::ROWB) >> 4);
}

// Byte offset of 16-byte unit u of a row of 256 bytes in the output's staging
// copy, swizzled so that rows by threads and units by threads meet no bank twice.
__device__ __forceinline__ uint32_t staged(int row, int u) { return static_cast<uint32_t>(row * 256 + ((u ^ (row & 7)) << 4)); }

// A wait for work that has been issued, also after an abort.
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_test(bar, parity))
    if (global_timer_ns() - t0 > kWaitLimitNs) return;
}

template <int D, bool BF16, int NQ>
__global__ void __launch_bounds__(WfCfg<D, NQ>::THREADS, WfCfg<D, NQ>::CTAS)
    attn_window_fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                           const __grid_constant__ CUtensorMap mv, const WindowArgs a, int head_group, int overlap) {
  using C = WfCfg<D, NQ>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (overlap) {  // launched overlapped (launch_serialized)
    griddep_wait();
    griddep_launch_dependents();
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Later rows, which under a wide window have more tiles, first.
  int rank, hb;
  grouped_rank_order(blockIdx.x + blockIdx.y * gridDim.x, gridDim.x, gridDim.y, head_group, rank, hb);
  const int row0 = (gridDim.x - 1 - rank) * 128;
  const int b = hb * NQ / a.Hq, h0 = hb * NQ - b * a.Hq, hk = h0 / (a.Hq / a.Hk);
  const int off = a.Nk - a.Nq;
  // Positions 0 .. npos - 1 of the CTA's list of key tiles.
  const int w0 = max(0, row0 + off - a.window + 1) >> 7;
  const int ns = min(w0, (a.sinks + 127) >> 7);
  const int npos = ns + ((min(row0 + 127, a.Nq - 1) + off) >> 7) - w0 + 1;
  auto key0 = [&](int p) { return (p < ns ? p : w0 + p - ns) * 128; };

  const uint32_t sbase = smem_addr(smem);
  if (sbase & 1023u) {  // the swizzle's atoms; never expected
    if (threadIdx.x == 0) atomicExch(a.status, kStatusDeviceCheck);
    return;
  }
  auto bar = [&](int i) -> uint32_t { return sbase + C::OFF_BAR + 8u * static_cast<uint32_t>(i); };
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + C::OFF_SLOT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
  const uint32_t sK = sbase + C::OFF_K, sV = sbase + C::OFF_V;
  auto load = [&](uint32_t dst, const CUtensorMap* map, int full, int row, int head) {
#pragma unroll
    for (int c = 0; c < C::NCH; ++c) tma_load_4d(dst + c * C::CHUNK, map, bar(full), c * C::CH, row, head, b);
  };
  auto load_k = [&](int p) {
    const int s = p % C::NST;
    mbar_arrive_expect_tx(bar(C::B_KFULL + s), C::TILE);
    load(sK + s * C::TILE, &mk, C::B_KFULL + s, key0(p), hk);
  };
  auto load_v = [&](int p) {
    const int s = p % C::NST;
    mbar_arrive_expect_tx(bar(C::B_VFULL + s), C::TILE);
    load(sV + s * C::TILE, &mv, C::B_VFULL + s, key0(p), hk);
  };
  // The first loads travel while TMEM is allocated.
  const int pre = min(npos, C::NST);
  if (warp == C::W_LOAD && lane == 0) {
    mbar_init(bar(C::B_Q), 1);
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(bar(C::B_KFULL + s), 1);
      mbar_init(bar(C::B_VFULL + s), 1);
      mbar_init(bar(C::B_KEMPTY + s), NQ);  // a thread of each query tile
      mbar_init(bar(C::B_VEMPTY + s), NQ);
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(bar(C::B_S + q), 1);
      mbar_init(bar(C::B_P + q), 128);
      mbar_init(bar(C::B_O + q), 1);
      mbar_init(bar(C::B_TAKEN + q), 128);
    }
    mbar_init(bar(C::B_DONE), 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&mq);
    prefetch_tensormap(&mk);
    prefetch_tensormap(&mv);
    mbar_arrive_expect_tx(bar(C::B_Q), NQ * C::TILE);
    for (int q = 0; q < NQ; ++q) load(sbase + q * C::TILE, &mq, C::B_Q, row0, h0 + q);
    for (int p = 0; p < pre; ++p) {
      load_k(p);
      load_v(p);
    }
  }
  if (warp == C::W_MMA) {
    tmem_alloc(smem_addr(slot), C::COLS);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *slot;

  if (warp >= C::W_LOAD) {
    regs_decrease<C::REGS_CTRL>();
    if (warp == C::W_LOAD && lane == 0) {
      // ------------------------------------------------------------ loads
      int nk = pre, nv = pre;  // issued
      for (int p = pre; p < npos; ++p) {
        const int s = p % C::NST, turn = (p / C::NST - 1) & 1;
        if (!mbar_wait(bar(C::B_KEMPTY + s), turn, abort_flag, a.status)) break;
        load_k(p);
        ++nk;
        if (!mbar_wait(bar(C::B_VEMPTY + s), turn, abort_flag, a.status)) break;
        load_v(p);
        ++nv;
      }
      if (*abort_flag) {  // copies in flight land before the shared memory goes
        drain(bar(C::B_Q), 0);
        for (int s = 0; s < C::NST; ++s) {
          if (nk > s) drain(bar(C::B_KFULL + s), ((nk - 1 - s) / C::NST) & 1);
          if (nv > s) drain(bar(C::B_VFULL + s), ((nv - 1 - s) / C::NST) & 1);
        }
      }
    } else if (warp == C::W_MMA && lane == 0) {
      // ----------------------------------------------- matrix instructions
      // A chain S, P V, S, P V, ... for each query tile; whichever next step is
      // ready goes out.  At d = 128 S(p + 1) is issued right behind the P V(p)
      // whose P it overwrites: one thread's MMAs run in the order of issue.  K and
      // V stages are handed back by the softmax, whose waits tell when the MMAs
      // that read them are complete.
      constexpr uint32_t HI = smem_desc_hi(C::SBO, C::SWZ);
      const uint32_t id_s = instr_desc_f16(128, 128, BF16, false, false, a.negate != 0);
      const uint32_t id_o = instr_desc_f16(128, D, BF16, false, true);
      bool ok = mbar_wait(bar(C::B_Q), 0, abort_flag, a.status);
      tc_fence_after_sync();
      int js[2] = {0, 0}, jp[2] = {0, 0};  // next S and P V of each tile
      int k_seen = 0, v_seen = 0;          // positions whose loads have been seen to land
      IdleWatch watch;
      while (ok && (jp[0] < npos || (NQ > 1 && jp[1] < npos))) {
        bool progress = false;
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          const int jv = jp[q];
          if (jv < js[q] && mbar_probe(bar(C::B_P + q), jv & 1) &&
              (jv < v_seen || mbar_probe(bar(C::B_VFULL + jv % C::NST), (jv / C::NST) & 1))) {
            v_seen = max(v_seen, jv + 1);
            tc_fence_after_sync();
            const uint32_t d_o = tmem + C::T_O + q * D, a_p = tmem + C::T_P + q * C::T_PSTEP;
            const uint32_t v_lo = smem_desc_lo(sV + (jv % C::NST) * C::TILE, C::CHUNK);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) mma_ts_w(d_o, a_p + kk * 8, v_lo + mn_step<D>(kk), HI, id_o, (jv > 0 || kk > 0) ? 1u : 0u);
            tc_commit(bar(C::B_O + q));
            jp[q] = jv + 1;
            progress = true;
          }
          const int jk = js[q];
          if (jk < npos && (C::APART ? jk == 0 || mbar_probe(bar(C::B_TAKEN + q), (jk - 1) & 1) : jk == jp[q]) &&
              (jk < k_seen || mbar_probe(bar(C::B_KFULL + jk % C::NST), (jk / C::NST) & 1))) {
            k_seen = max(k_seen, jk + 1);
            tc_fence_after_sync();
            const uint32_t d_s = tmem + q * 128, q_lo = smem_desc_lo(sbase + q * C::TILE, 16);
            const uint32_t k_lo = smem_desc_lo(sK + (jk % C::NST) * C::TILE, 16);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) mma_ss_w(d_s, q_lo + k_step<D>(kk), HI, k_lo + k_step<D>(kk), HI, id_s, kk > 0 ? 1u : 0u);
            tc_commit(bar(C::B_S + q));
            js[q] = jk + 1;
            progress = true;
          }
        }
        if (progress) watch.progress();
        else ok = watch.idle(abort_flag, a.status, kWaitLimitNs);
      }
      tc_commit(bar(C::B_DONE));  // before TMEM is released
      drain(bar(C::B_DONE), 0);
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------------- softmax
    regs_increase<C::REGS_ROW>();
    const int q = warp >> 2, r = threadIdx.x & 127, row = row0 + r;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + q * 128, tO = tmem + lanes + C::T_O + q * D, tP = tmem + lanes + C::T_P + q * C::T_PSTEP;
    const float sl2 = a.sl2;
    const float2 sl2x2 = make_float2(sl2, sl2);
    float m = -INFINITY, l_exact = 0.f, l_round = 0.f;
    bool ok = true;
    auto release = [&](int first, int p) {
      if (r == 0) mbar_arrive(bar(first + p % C::NST));
    };
    for (int p = 0; p < npos; ++p) {
      // (a warp's lanes go on or stop together: they vote below)
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_S + q), p & 1, abort_flag, a.status)))) break;
      tc_fence_after_sync();
      release(C::B_KEMPTY, p);
      if (!C::APART && p > 0) release(C::B_VEMPTY, p - 1);  // S(p)'s commit covers P V(p - 1)
      float sv[128];
      {
        uint32_t u[64];
        tmem_ld64(tS, u);
#pragma unroll
        for (int c = 0; c < 64; ++c) sv[c] = __uint_as_float(u[c]);
        tmem_ld64(tS + 64, u);
#pragma unroll
        for (int c = 0; c < 64; ++c) sv[64 + c] = __uint_as_float(u[c]);
      }
      if constexpr (C::APART) {
        tc_fence_before_sync();
        mbar_arrive(bar(C::B_TAKEN + q));
      }
      // Key kv0 + c is visible iff c <= last and (c >= first or c < sinks).
      const int kv0 = key0(p);
      const int at = row + off - kv0;
      const bool right = kv0 + 127 > row0 + off;
      const bool left = kv0 < row0 + 127 + off - a.window + 1 && kv0 + 128 > a.sinks;
      if (right) {
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c > at) sv[c] = -INFINITY;
      }
      if (left) {
        const int first = at - a.window + 1, sinks = a.sinks - kv0;
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c < first && c >= sinks) sv[c] = -INFINITY;
      }
      float mx;
      {
        float a0 = sv[0], a1 = sv[1], a2 = sv[2], a3 = sv[3];
#pragma unroll
        for (int c = 4; c < 128; c += 8) {
          a0 = max3f(a0, sv[c], sv[c + 1]);
          a1 = max3f(a1, sv[c + 2], sv[c + 3]);
          a2 = max3f(a2, sv[c + 4], sv[c + 5]);
          a3 = max3f(a3, sv[c + 6], sv[c + 7]);
        }
        mx = fmaxf(fmaxf(a0, a1), fmaxf(a2, a3));
      }
      const float m_new = fmaxf(m, mx * sl2);
      float alpha = 1.f;
      if (m_new > m + kRescaleLog2) {  // also with the row's first visible key (m = -inf)
        alpha = ex2_approx(m - m_new);
        m = m_new;
      }
      const float neg_m = m == -INFINITY ? 0.f : -m;
      const float2 nm2 = make_float2(neg_m, neg_m);
#pragma unroll
      for (int c = 0; c < 128; c += 2) {
        const float2 t = fma2(make_float2(sv[c], sv[c + 1]), sl2x2, nm2);
        sv[c] = ex2_approx(t.x);
        sv[c + 1] = ex2_approx(t.y);
      }
      if (sl2 == 0.f && (left || right)) {  // -inf times 0 is NaN: hidden keys once more
        const int first = at - a.window + 1, sinks = a.sinks - kv0;
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c > at || (c < first && c >= sinks)) sv[c] = 0.f;
      }
      if (C::APART && p > 0) {  // P V(p - 1) is complete: P may be written, O is what it will be
        ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_O + q), (p - 1) & 1, abort_flag, a.status));
        if (!ok) break;
        tc_fence_after_sync();
        release(C::B_VEMPTY, p - 1);
      }
      if (p > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
        for (int c0 = 0; c0 < D / 32; ++c0) {
          uint32_t ov[32];
          tmem_ld32(tO + c0 * 32, ov);
#pragma unroll
          for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
          tmem_st32(tO + c0 * 32, ov);
        }
      }
      // P goes out first, the sums follow while P V runs.
      uint32_t pk0[32], pk1[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) pk0[i] = pack2<BF16>(sv[2 * i], sv[2 * i + 1]);
      tmem_st32(tP, pk0);
#pragma unroll
      for (int i = 0; i < 32; ++i) pk1[i] = pack2<BF16>(sv[64 + 2 * i], sv[64 + 2 * i + 1]);
      tmem_st32(tP + 32, pk1);
      tmem_st_wait();
      tc_fence_before_sync();
      mbar_arrive(bar(C::B_P + q));
      float2 e0 = make_float2(0.f, 0.f), e1 = e0;
      float r0 = 0.f, r1 = 0.f, r2 = 0.f, r3 = 0.f;
#pragma unroll
      for (int c = 0; c < 128; c += 4) {
        e0 = add2(e0, make_float2(sv[c], sv[c + 1]));
        e1 = add2(e1, make_float2(sv[c + 2], sv[c + 3]));
      }
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        r0 = add_halves<BF16>(r0, pk0[i]);
        r1 = add_halves<BF16>(r1, pk0[i + 1]);
        r2 = add_halves<BF16>(r2, pk1[i]);
        r3 = add_halves<BF16>(r3, pk1[i + 1]);
      }
      l_exact = l_exact * alpha + ((e0.x + e0.y) + (e1.x + e1.y));
      l_round = l_round * alpha + ((r0 + r1) + (r2 + r3));
    }
    // ---------------------------------------------------------------- output
    // At d = 128 through the tile's Q in shared memory, which no MMA reads any
    // more, so that a warp stores whole rows.
    constexpr bool STAGE = D == 128;
    if (__all_sync(0xffffffffu, ok && mbar_wait(bar(C::B_O + q), (npos - 1) & 1, abort_flag, a.status))) {
      tc_fence_after_sync();
      const float inv = 1.0f / l_round;
      uint8_t* stage = smem + q * C::TILE;
      uint8_t* out = a.o.p + b * a.o.b + (h0 + q) * a.o.h;
#pragma unroll
      for (int c0 = 0; c0 < D / 32; ++c0) {
        uint32_t ov[32], pk[16];
        tmem_ld32(tO + c0 * 32, ov);
#pragma unroll
        for (int i = 0; i < 16; ++i) pk[i] = pack2<BF16>(__uint_as_float(ov[2 * i]) * inv, __uint_as_float(ov[2 * i + 1]) * inv);
        if (STAGE || row < a.Nq) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(STAGE ? stage + staged(r, c0 * 4 + i) : out + row * a.o.n + c0 * 64 + i * 16) =
                make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
        }
      }
      if constexpr (STAGE) {
        __syncwarp();
#pragma unroll
        for (int it = 0; it < 16; ++it) {
          const int rr = (r & ~31) + it * 2 + (lane >> 4), u = lane & 15;
          const uint4 val = *reinterpret_cast<const uint4*>(stage + staged(rr, u));
          if (row0 + rr < a.Nq) *reinterpret_cast<uint4*>(out + (row0 + rr) * a.o.n + u * 16) = val;
        }
      }
      if (row < a.Nq) a.lse[(static_cast<int64_t>(b) * a.Hq + h0 + q) * a.Nq + row] = (m + log2f(l_exact)) * 0.69314718055994531f;
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == C::W_MMA) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::COLS);
  }
}

template <int D, bool BF16, int NQ>
int launch_t(const WindowArgs& a) {
  using C = WfCfg<D, NQ>;
  CUtensorMap mq, mk, mv;
  if (!encode_strided_map(&mq, a.q, a.B, a.Hq, a.Nq, D, C::CH, BF16) || !encode_strided_map(&mk, a.k, a.B, a.Hk, a.Nk, D, C::CH, BF16) ||
      !encode_strided_map(&mv, a.v, a.B, a.Hk, a.Nk, D, C::CH, BF16))
    return kStatusCuda;
  auto kern = attn_window_fwd_kernel<D, BF16, NQ>;
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kern), C::SMEM)) return kStatusCuda;
  if (!check_launch_regs(reinterpret_cast<const void*>(kern), C::REGS)) return kStatusDeviceCheck;  // the split's sum
  const dim3 grid((a.Nq + 127) / 128, a.B * a.Hq / NQ);
  const bool overlap = overlap_launches(static_cast<int64_t>(grid.x) * grid.y, C::CTAS);
  const int group = order_head_group(grid.y, int64_t{4} * a.Nk * D, int64_t{128} << 20);
  return launch_serialized(overlap, kern, grid, dim3(C::THREADS), C::SMEM, a.stream, mq, mk, mv, a, group, overlap ? 1 : 0) == cudaSuccess
             ? kStatusOk
             : kStatusCuda;
}

template <int D>
int launch_d(const WindowArgs& a) {
  return a.bf16 ? launch_t<D, true, 1>(a) : launch_t<D, false, 1>(a);
}

}  // namespace

int launch_window_fwd(const WindowArgs& a, int* launches) {
  *launches = 1;
  return a.d == 32 ? launch_d<32>(a) : a.d == 64 ? launch_d<64>(a) : launch_d<128>(a);
}

}  // namespace attn
