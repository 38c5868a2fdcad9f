// attn_window_bwd.cu -- causal attention with a sliding window and sinks,
// backward: with P = exp(s - LSE) on the visible pairs and D_i = dO_i . O_i,
//   dV_j = sum_i P_ij dO_i,  dS = P o (dO V^T - D),
//   dQ = scale dS K,  dK = scale sum_i dS^T Q,
// the sums also over the query heads that share the key/value head
// (FlashAttention (PKM page), "三招" 3 Recomputation; FlashAttention深度攻略 §6).
//
// Key tile j (128 keys) is seen by the query tiles from its own position on to
// `window` behind its last key, or by all later ones where it holds sinks; for
// each of the key/value head's query heads.  These visits are a CTA's loop; K_j
// and V_j stay in shared memory, dK and dV accumulate in TMEM.  Where a tile has
// many more visits than others (sinks) or there are few tiles, its visits are cut
// into runs of CTAs that leave fp32 partial tiles.
//   attn_window_pre_kernel : -D_i and -LSE log2(e) by rows, padded to whole tiles
//       (-inf there, so that P is 0), zeros in the fp32 dQ accumulator.
//   attn_window_bwd_kernel : five products a visit on tcgen05, as below.
//   attn_window_out_kernel : dQ to its type; the runs' partial dK, dV, added in
//       the order of the runs.
//
// attn_window_bwd_kernel: 16 warps, one CTA to an SM.
//   warp 12: TMA loads; K_j, V_j once, Q_i, dO_i and the two row vectors in a ring.
//   warp 13: one thread issues S^T = K Q^T, dP^T = V dO^T, dV += P^T dO (P^T from
//       TMEM), dK += dS^T Q, dQ_i = dS K (at d = 128 as dQ_i^T = K^T dS^T).
//   warps 0-7: P^T and dS^T, two threads to a key row, 64 queries each; at the end
//       dK (warps 0-3) and dV (4-7).
//   warps 8-11: dQ_i out of TMEM and into the accumulator by reductions of whole
//       128-byte lines: a thread to a channel at d = 128, else groups of 8 lanes
//       exchange 16-byte pieces of their rows first.
//   TMEM: S^T / P^T [0, 128), dP^T / dQ [128, 256), dK, dV.
#include "attn_internal.h"
#include "attn_window.h"
#include "tc_sm103.cuh"

namespace attn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// The grid's items: runs of visits of key tiles.  Tiles with sinks come first.
struct WbPlan {
  int tiles, sink_tiles;       // of a key/value head
  int sink_runs, runs;         // CTAs to a tile with and without sinks
  int sink_items, group;       // items of tiles with sinks; heads in flight together
  int npad;                    // rows of a head's row vectors
  float *lse2, *dvec, *dq;     // scratch
  float* part;                 // [split item][dK, dV][128][d]
};

template <int D>
struct WbCfg {
  static constexpr int ROWB = D >= 64 ? 128 : 64;
  static constexpr int CH = ROWB / 2;
  static constexpr int NCH = D / CH;
  static constexpr uint32_t SWZ = ROWB == 128 ? kSwizzle128B : kSwizzle64B;
  static constexpr int SBO = 8 * ROWB;
  static constexpr int CHUNK = 128 * ROWB;
  static constexpr int TILE = 128 * D * 2;
  static constexpr int DS_CHUNK = 128 * 128;  // 64 queries x 128 keys
  static constexpr int NST = 2;               // Q, dO stages
  static constexpr int VEC = 128 * 4;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = TILE;
  static constexpr int OFF_Q = 2 * TILE;
  static constexpr int OFF_DO = OFF_Q + NST * TILE;
  static constexpr int OFF_DS = OFF_DO + NST * TILE;
  static constexpr int OFF_LSE = OFF_DS + 2 * DS_CHUNK;
  static constexpr int OFF_D = OFF_LSE + NST * VEC;
  static constexpr int OFF_BAR = OFF_D + NST * VEC;
  static constexpr int B_KV = 0;
  static constexpr int B_QFULL = 1;
  static constexpr int B_QEMPTY = B_QFULL + NST;
  static constexpr int B_S = B_QEMPTY + NST;
  static constexpr int B_DP = B_S + 1;
  static constexpr int B_P = B_DP + 1;
  static constexpr int B_DS = B_P + 1;
  static constexpr int B_DQ = B_DS + 1;       // dK(i) and dQ(i) are complete
  static constexpr int B_DQFREE = B_DQ + 1;   // dQ's columns are read
  static constexpr int B_DONE = B_DQFREE + 1;
  static constexpr int NBAR = B_DONE + 1;
  static constexpr int OFF_SLOT = OFF_BAR + NBAR * 8;
  static constexpr int OFF_ABORT = OFF_SLOT + 4;
  static constexpr int SMEM = OFF_ABORT + 4;
  static constexpr int THREADS = 512;
  static constexpr int REGS = 128, REGS_ROW = 152, REGS_DQ = 144, REGS_CTRL = 64;
  static_assert(128 * (2 * REGS_ROW + REGS_DQ + REGS_CTRL) <= THREADS * REGS, "register split");
  static constexpr uint32_t T_S = 0, T_DP = 128, T_DK = 256, T_DV = 256 + D;
  static constexpr bool DQ_T = D == 128;  // lanes of dQ are channels
  static_assert(SMEM <= 232448, "shared memory");
};

// Descriptor steps (16-byte units) of the 16-deep slice kk: of a K-major tile with
// rows of D channels, of an MN-major one, and of the dS^T tile (128 keys x 128
// queries) as dS^T (K-major) and as dS (MN-major).
template <int D>
__host__ __device__ constexpr uint32_t k_step(int kk) {
  using C = WbCfg<D>;
  return static_cast<uint32_t>(((kk * 16) / C::CH * C::CHUNK + (kk * 16) % C::CH * 2) >> 4);
}
template <int D>
__host__ __device__ constexpr uint32_t mn_step(int kk) {
  return static_cast<uint32_t>((kk * 16 * WbCfg<D>::ROWB) >> 4);
}
__host__ __device__ constexpr uint32_t ds_k_step(int kk) { return static_cast<uint32_t>(((kk * 16) / 64 * (128 * 128) + (kk * 16) % 64 * 2) >> 4); }
__host__ __device__ constexpr uint32_t ds_mn_step(int kk) { return static_cast<uint32_t>((kk * 16 * 128) >> 4); }

// Byte offset of 16-byte unit u of a row of 256 bytes in the staging copy of dK or
// dV, swizzled so that rows by threads and units by threads meet no bank twice.
__device__ __forceinline__ uint32_t staged(int row, int u) { return static_cast<uint32_t>(row * 256 + ((u ^ (row & 7)) << 4)); }

// A wait for work that has been issued, also after an abort.
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_test(bar, parity))
    if (global_timer_ns() - t0 > kWaitLimitNs) return;
}

// ---------------------------------------------------------------- row vectors
// Eight lanes to a row; HBM bounds it (2 tensors in, 4 d bytes of zeros out).
template <int D, bool BF16>
__global__ void __launch_bounds__(256) attn_window_pre_kernel(const WindowArgs a, const WbPlan p) {
  griddep_wait();  // (launch_serialized)
  griddep_launch_dependents();
  const int64_t rid = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 3;  // of [B * Hq][npad]
  const int sub = threadIdx.x & 7;
  const int64_t bh = rid / p.npad;
  const int i = static_cast<int>(rid - bh * p.npad);
  const bool inside = bh < static_cast<int64_t>(a.B) * a.Hq, real = inside && i < a.Nq;
  float acc = 0.f;
  if (real) {
    const int b = static_cast<int>(bh / a.Hq), h = static_cast<int>(bh - static_cast<int64_t>(b) * a.Hq);
    const uint8_t *o = a.o.p + b * a.o.b + h * a.o.h + i * a.o.n, *dO = a.dO.p + b * a.dO.b + h * a.dO.h + i * a.dO.n;
#pragma unroll
    for (int k = sub; k < D / 8; k += 8) {  // 16-byte pieces
      const uint4 x = *reinterpret_cast<const uint4*>(o + k * 16), y = *reinterpret_cast<const uint4*>(dO + k * 16);
      const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 u = unpack2<BF16>(xw[e]), w = unpack2<BF16>(yw[e]);
        acc = fmaf(u.x, w.x, acc);
        acc = fmaf(u.y, w.y, acc);
      }
    }
    float4* z = reinterpret_cast<float4*>(p.dq + (bh * a.Nq + i) * D);
#pragma unroll
    for (int k = 0; k < D / 32; ++k) z[sub + 8 * k] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  acc += __shfl_xor_sync(0xffffffffu, acc, 4);
  acc += __shfl_xor_sync(0xffffffffu, acc, 2);
  acc += __shfl_xor_sync(0xffffffffu, acc, 1);
  if (inside && sub == 0) {
    p.dvec[rid] = real ? -acc : 0.f;
    p.lse2[rid] = real ? -a.lse[bh * a.Nq + i] * kLog2e : -INFINITY;
  }
}

// ------------------------------------------------------------------- outputs
// Eight channels at a time: dQ from its accumulator, then the split tiles' dK and dV.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) attn_window_out_kernel(const WindowArgs a, const WbPlan p) {
  griddep_wait();  // (launch_serialized)
  griddep_launch_dependents();
  constexpr int G = D / 8;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256, from = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  auto packed = [](const float (&x)[8]) {
    return make_uint4(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]), pack2<BF16>(x[4], x[5]), pack2<BF16>(x[6], x[7]));
  };
  auto add = [](float (&x)[8], const float* f) {
    const float4 u = reinterpret_cast<const float4*>(f)[0], w = reinterpret_cast<const float4*>(f)[1];
    x[0] += u.x, x[1] += u.y, x[2] += u.z, x[3] += u.w, x[4] += w.x, x[5] += w.y, x[6] += w.z, x[7] += w.w;
  };
  const int64_t rows = static_cast<int64_t>(a.B) * a.Hq * a.Nq;
  for (int64_t t = from; t < rows * G; t += step) {
    const int64_t row = t / G, bh = row / a.Nq;
    const int c = static_cast<int>(t % G), i = static_cast<int>(row - bh * a.Nq);
    const int b = static_cast<int>(bh / a.Hq), h = static_cast<int>(bh - static_cast<int64_t>(b) * a.Hq);
    float x[8] = {};
    add(x, p.dq + t * 8);
    *reinterpret_cast<uint4*>(a.dq.p + b * a.dq.b + h * a.dq.h + i * a.dq.n + c * 16) = packed(x);
  }
  // Split tiles: those with sinks, then the others; each one's runs are in a row.
  const int64_t heads = static_cast<int64_t>(a.B) * a.Hk;
  const int64_t s_tiles = p.sink_runs > 1 ? heads * p.sink_tiles : 0;
  const int64_t w_tiles = p.runs > 1 ? heads * (p.tiles - p.sink_tiles) : 0;
  for (int64_t t = from; t < (s_tiles + w_tiles) * 2 * 128 * G; t += step) {
    const int c = static_cast<int>(t % G), r = static_cast<int>(t / G % 128), out = static_cast<int>(t / (G * 128) % 2);
    int64_t tile = t / (G * 256), slot;
    int n, jt, hb;
    if (tile < s_tiles) {
      n = p.sink_runs, slot = tile * n;
      hb = static_cast<int>(tile / p.sink_tiles), jt = static_cast<int>(tile % p.sink_tiles);
    } else {
      tile -= s_tiles;
      n = p.runs, slot = (p.sink_runs > 1 ? p.sink_items : 0) + tile * n;
      const int per = p.tiles - p.sink_tiles;
      hb = static_cast<int>(tile / per), jt = p.sink_tiles + static_cast<int>(tile % per);
    }
    const int j = jt * 128 + r;
    if (j >= a.Nk) continue;
    float x[8] = {};
    for (int k = 0; k < n; ++k) add(x, p.part + (((slot + k) * 2 + out) * 128 + r) * D + c * 8);
    const Bhnd& d = out ? a.dv : a.dk;
    *reinterpret_cast<uint4*>(d.p + hb / a.Hk * d.b + hb % a.Hk * d.h + j * d.n + c * 16) = packed(x);
  }
}

// ------------------------------------------------------------------ main pass
template <int D, bool BF16>
__global__ void __launch_bounds__(WbCfg<D>::THREADS, 1)
    attn_window_bwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                           const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mdo, const WindowArgs a,
                           const WbPlan p) {
  using C = WbCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.Hq / a.Hk, off = a.Nk - a.Nq, heads = a.B * a.Hk;
  // The item: key tile jt of head hb, run `run` of n_runs, and its place among the partial tiles.
  int jt, hb, run, n_runs;
  int64_t slot = 0;
  {
    const int item = blockIdx.x;
    if (item < p.sink_items) {
      n_runs = p.sink_runs;
      const int tile = item / n_runs;
      run = item - tile * n_runs;
      hb = tile / p.sink_tiles, jt = tile - hb * p.sink_tiles;
      slot = item;
    } else {
      n_runs = p.runs;
      const int tile = (item - p.sink_items) / n_runs, per = p.tiles - p.sink_tiles;
      run = item - p.sink_items - tile * n_runs;
      grouped_rank_order(tile, per, heads, p.group, jt, hb);
      slot = (p.sink_runs > 1 ? p.sink_items : 0) + (static_cast<int64_t>(hb) * per + jt) * n_runs + run;
      jt += p.sink_tiles;
    }
  }
  const int b = hb / a.Hk, hk = hb - b * a.Hk, kv0 = jt * 128;
  // Query tiles [q_lo, q_lo + nt) see the tile; its visits are those of each query head.
  const int q_lo = max(0, kv0 - off) >> 7;
  const int last = kv0 < a.sinks ? a.Nq - 1 : min(a.Nq - 1, kv0 + 126 + a.window - off);
  const int nt = kv0 - off >= a.Nq || last < 0 ? 0 : (last >> 7) + 1 - q_lo;
  const int64_t all = static_cast<int64_t>(nt) * G;
  const int v0 = static_cast<int>(all * run / n_runs), nv = static_cast<int>(all * (run + 1) / n_runs) - v0;
  struct Visit {
    int g, qt;  // query head within the group, query tile
  };
  const Visit first = {nt ? v0 / nt : 0, nt ? q_lo + v0 % nt : 0};
  auto advance = [&](Visit& v) {
    if (++v.qt == q_lo + nt) v.qt = q_lo, ++v.g;
  };

  const uint32_t sbase = smem_addr(smem);
  if (sbase & 1023u) {  // the swizzle's atoms; never expected
    if (threadIdx.x == 0) atomicExch(a.status, kStatusDeviceCheck);
    return;
  }
  auto bar = [&](int i) -> uint32_t { return sbase + C::OFF_BAR + 8u * static_cast<uint32_t>(i); };
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + C::OFF_SLOT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
  const uint32_t sK = sbase + C::OFF_K, sV = sbase + C::OFF_V, sQ = sbase + C::OFF_Q, sDO = sbase + C::OFF_DO, sDS = sbase + C::OFF_DS;
  auto load_stage = [&](int s, const Visit& v) {
    const uint32_t full = bar(C::B_QFULL + s);
    const int q0 = v.qt * 128, h = hk * G + v.g;
    mbar_arrive_expect_tx(full, 2 * C::TILE + 2 * C::VEC);
    for (int c = 0; c < C::NCH; ++c) {
      tma_load_4d(sQ + s * C::TILE + c * C::CHUNK, &mq, full, c * C::CH, q0, h, b);
      tma_load_4d(sDO + s * C::TILE + c * C::CHUNK, &mdo, full, c * C::CH, q0, h, b);
    }
    const int64_t at = (static_cast<int64_t>(b) * a.Hq + h) * p.npad + q0;
    bulk_load(sbase + C::OFF_LSE + s * C::VEC, p.lse2 + at, C::VEC, full);
    bulk_load(sbase + C::OFF_D + s * C::VEC, p.dvec + at, C::VEC, full);
  };
  const int pre = min(nv, C::NST);  // the first loads travel while TMEM is allocated
  Visit ahead = first;
  if (warp == 12 && lane == 0) {
    mbar_init(bar(C::B_KV), 1);
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(bar(C::B_QFULL + s), 1);
      mbar_init(bar(C::B_QEMPTY + s), 1);
    }
    mbar_init(bar(C::B_S), 1);
    mbar_init(bar(C::B_DP), 1);
    mbar_init(bar(C::B_P), 256);
    mbar_init(bar(C::B_DS), 256);
    mbar_init(bar(C::B_DQ), 1);
    mbar_init(bar(C::B_DQFREE), 128);
    mbar_init(bar(C::B_DONE), 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&mq);
    prefetch_tensormap(&mk);
    prefetch_tensormap(&mv);
    prefetch_tensormap(&mdo);
    if (nv > 0) {  // a run without visits loads nothing
      mbar_arrive_expect_tx(bar(C::B_KV), 2 * C::TILE);
      for (int c = 0; c < C::NCH; ++c) {
        tma_load_4d(sK + c * C::CHUNK, &mk, bar(C::B_KV), c * C::CH, kv0, hk, b);
        tma_load_4d(sV + c * C::CHUNK, &mv, bar(C::B_KV), c * C::CH, kv0, hk, b);
      }
    }
    for (int it = 0; it < pre; ++it) {
      load_stage(it, ahead);
      advance(ahead);
    }
  }
  if (warp == 13) {
    tmem_alloc(smem_addr(tslot), 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tslot;

  if (warp >= 12) {
    regs_decrease<C::REGS_CTRL>();
    if (warp == 12 && lane == 0) {
      // -------------------------------------------------------------- loads
      int issued = pre;
      for (int it = pre; it < nv; ++it) {
        const int s = it % C::NST;
        if (!mbar_wait(bar(C::B_QEMPTY + s), (it / C::NST - 1) & 1, abort_flag, a.status)) break;
        load_stage(s, ahead);
        advance(ahead);
        issued = it + 1;
      }
      if (*abort_flag && nv > 0) {  // copies in flight land before the shared memory goes
        drain(bar(C::B_KV), 0);
        for (int s = 0; s < C::NST; ++s)
          if (issued > s) drain(bar(C::B_QFULL + s), ((issued - 1 - s) / C::NST) & 1);
      }
    } else if (warp == 13 && lane == 0) {
      // ------------------------------------------------- matrix instructions
      // Four chains over the visits, each step issued as soon as it is ready:
      //   S(i)        needs Q_i, and dV(i - 1) issued, whose P^T it overwrites (one
      //               thread's MMAs run in the order of issue)
      //   dP(i)       needs dO_i, and dQ(i - 1) read, whose columns it overwrites
      //   dV(i)       needs P^T(i)
      //   dK(i), dQ(i) need dS^T(i)
      const uint32_t id_st = instr_desc_f16(128, 128, BF16, false, false, a.negate != 0);
      const uint32_t id_dpt = instr_desc_f16(128, 128, BF16, false, false);
      const uint32_t id_kv = instr_desc_f16(128, D, BF16, false, true);
      const uint32_t id_dq = instr_desc_f16(128, C::DQ_T ? 128 : D, BF16, true, true);
      constexpr uint32_t HT = smem_desc_hi(C::SBO, C::SWZ), HDS = smem_desc_hi(1024, kSwizzle128B);
      const uint32_t k_klo = smem_desc_lo(sK, 16), v_klo = smem_desc_lo(sV, 16), k_mnlo = smem_desc_lo(sK, C::CHUNK);
      const uint32_t ds_klo = smem_desc_lo(sDS, 16), ds_mnlo = smem_desc_lo(sDS, C::DS_CHUNK);
      bool ok = nv == 0 || mbar_wait(bar(C::B_KV), 0, abort_flag, a.status);
      tc_fence_after_sync();
      int is = 0, ip = 0, iv = 0, ik = 0;
      IdleWatch watch;
      while (ok && ik < nv) {
        bool progress = false;
        if (is < nv && is == iv && mbar_probe(bar(C::B_QFULL + is % C::NST), (is / C::NST) & 1)) {
          tc_fence_after_sync();
          const uint32_t q_lo = smem_desc_lo(sQ + (is % C::NST) * C::TILE, 16);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss_w(tmem + C::T_S, k_klo + k_step<D>(kk), HT, q_lo + k_step<D>(kk), HT, id_st, kk > 0 ? 1u : 0u);
          tc_commit(bar(C::B_S));
          ++is;
          progress = true;
        }
        if (ip < nv && ip == ik && (ip == 0 || mbar_probe(bar(C::B_DQFREE), (ip - 1) & 1)) &&
            mbar_probe(bar(C::B_QFULL + ip % C::NST), (ip / C::NST) & 1)) {
          tc_fence_after_sync();
          const uint32_t do_lo = smem_desc_lo(sDO + (ip % C::NST) * C::TILE, 16);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss_w(tmem + C::T_DP, v_klo + k_step<D>(kk), HT, do_lo + k_step<D>(kk), HT, id_dpt, kk > 0 ? 1u : 0u);
          tc_commit(bar(C::B_DP));
          ++ip;
          progress = true;
        }
        if (iv < is && mbar_probe(bar(C::B_P), iv & 1)) {
          tc_fence_after_sync();
          const uint32_t do_lo = smem_desc_lo(sDO + (iv % C::NST) * C::TILE, C::CHUNK);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts_w(tmem + C::T_DV, tmem + C::T_S + (kk >> 2) * 64 + (kk & 3) * 8, do_lo + mn_step<D>(kk), HT, id_kv,
                     (iv > 0 || kk > 0) ? 1u : 0u);
          ++iv;
          progress = true;
        }
        if (ik < iv && ik < ip && mbar_probe(bar(C::B_DS), ik & 1)) {
          tc_fence_after_sync();
          const uint32_t q_mnlo = smem_desc_lo(sQ + (ik % C::NST) * C::TILE, C::CHUNK);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ss_w(tmem + C::T_DK, ds_klo + ds_k_step(kk), HDS, q_mnlo + mn_step<D>(kk), HT, id_kv, (ik > 0 || kk > 0) ? 1u : 0u);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            if constexpr (C::DQ_T)
              mma_ss_w(tmem + C::T_DP, k_mnlo + mn_step<D>(kk), HT, ds_mnlo + ds_mn_step(kk), HDS, id_dq, kk > 0 ? 1u : 0u);
            else
              mma_ss_w(tmem + C::T_DP, ds_mnlo + ds_mn_step(kk), HDS, k_mnlo + mn_step<D>(kk), HT, id_dq, kk > 0 ? 1u : 0u);
          }
          tc_commit(bar(C::B_DQ));  // dQ_i is there, the dS^T tile and the Q, dO stage are free
          ++ik;
          progress = true;
        }
        if (progress) watch.progress();
        else ok = watch.idle(abort_flag, a.status, kWaitLimitNs);
      }
      tc_commit(bar(C::B_DONE));  // before TMEM is released
      drain(bar(C::B_DONE), 0);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------- P^T and dS^T
    regs_increase<C::REGS_ROW>();
    const int half = warp >> 2, t = threadIdx.x & 127, j = kv0 + t;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float* s_lse = reinterpret_cast<const float*>(smem + C::OFF_LSE);
    const float* s_d = reinterpret_cast<const float*>(smem + C::OFF_D);
    uint8_t* ds_row = smem + C::OFF_DS + half * C::DS_CHUNK + t * 128;
    const float2 sl2x2 = make_float2(a.sl2, a.sl2);
    // Row i sees this key iff from <= i < to.
    const int from = j < a.Nk ? j - off : a.Nq, to = j < a.sinks ? a.Nq : j - off + a.window;
    bool ok = true;
    Visit v = first;
    for (int it = 0; it < nv; ++it, advance(v)) {
      const int s = it % C::NST, q0 = v.qt * 128 + half * 64;
      // (a warp's lanes go on or stop together: what follows wants all of them)
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_S), it & 1, abort_flag, a.status)))) break;
      tc_fence_after_sync();
      float pr[64];
      {
        uint32_t u[64];
        tmem_ld64(tmem + lanes + C::T_S + half * 64, u);
#pragma unroll
        for (int c = 0; c < 64; ++c) pr[c] = __uint_as_float(u[c]);
      }
      const float2* nlse = reinterpret_cast<const float2*>(s_lse + s * 128 + half * 64);
#pragma unroll
      for (int c = 0; c < 64; c += 2) {
        const float2 e = fma2(make_float2(pr[c], pr[c + 1]), sl2x2, nlse[c / 2]);
        pr[c] = ex2_approx(e.x);
        pr[c + 1] = ex2_approx(e.y);
      }
      if (from > q0) {
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (c < from - q0) pr[c] = 0.f;
      }
      if (to < q0 + 64) {
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (c >= to - q0) pr[c] = 0.f;
      }
      {
        uint32_t pk[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) pk[i] = pack2<BF16>(pr[2 * i], pr[2 * i + 1]);
        tmem_st32(tmem + lanes + C::T_S + half * 64, pk);
      }
      tmem_st_wait();
      tc_fence_before_sync();
      mbar_arrive(bar(C::B_P));
      ok = mbar_wait(bar(C::B_DP), it & 1, abort_flag, a.status) && (it == 0 || mbar_wait(bar(C::B_DQ), (it - 1) & 1, abort_flag, a.status));
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      if (C::DQ_T && it > 0 && threadIdx.x == 0) mbar_arrive(bar(C::B_QEMPTY + (it - 1) % C::NST));
      tc_fence_after_sync();
      const float2* nd = reinterpret_cast<const float2*>(s_d + s * 128 + half * 64);
#pragma unroll
      for (int c0 = 0; c0 < 2; ++c0) {
        uint32_t dp[32], pk[16];
        tmem_ld32(tmem + lanes + C::T_DP + half * 64 + c0 * 32, dp);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int c = c0 * 32 + 2 * i;
          const float2 gd = add2(make_float2(__uint_as_float(dp[2 * i]), __uint_as_float(dp[2 * i + 1])), nd[c / 2]);
          const float2 ds = mul2(make_float2(pr[c], pr[c + 1]), gd);
          pk[i] = pack2<BF16>(ds.x, ds.y);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
          *reinterpret_cast<uint4*>(ds_row + (((c0 * 4 + u) ^ (t & 7)) * 16)) = make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
      }
      fence_proxy_async_smem();
      tc_fence_before_sync();
      mbar_arrive(bar(C::B_DS));
    }
    // dK (warps 0-3, times scale) or dV.  At d = 128 16-bit rows go through the K or V
    // tile in shared memory, which no MMA reads any more.
    const Bhnd& dst = half ? a.dv : a.dk;
    uint8_t* out = dst.p + b * dst.b + hk * dst.h;
    float4* partial = reinterpret_cast<float4*>(p.part + ((slot * 2 + half) * 128 + t) * D);
    const bool ep = __all_sync(0xffffffffu, ok && nv > 0 && mbar_wait(bar(C::B_DQ), (nv - 1) & 1, abort_flag, a.status));
    const float mul = half ? 1.f : a.scale;
    const uint32_t col = tmem + lanes + (half ? C::T_DV : C::T_DK);
    constexpr bool STAGE = D == 128;
    if (ep) {
      tc_fence_after_sync();
      uint8_t* stage = smem + (half ? C::OFF_V : C::OFF_K);
#pragma unroll
      for (int c0 = 0; c0 < D / 32; ++c0) {
        uint32_t x[32];
        tmem_ld32(col + c0 * 32, x);
        if (n_runs > 1) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            partial[c0 * 8 + i] = make_float4(__uint_as_float(x[4 * i]) * mul, __uint_as_float(x[4 * i + 1]) * mul,
                                              __uint_as_float(x[4 * i + 2]) * mul, __uint_as_float(x[4 * i + 3]) * mul);
          continue;
        }
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) pk[i] = pack2<BF16>(__uint_as_float(x[2 * i]) * mul, __uint_as_float(x[2 * i + 1]) * mul);
        if (STAGE || j < a.Nk) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(STAGE ? stage + staged(t, c0 * 4 + i) : out + j * dst.n + c0 * 64 + i * 16) =
                make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
        }
      }
      if (STAGE && n_runs == 1) {
        __syncwarp();
#pragma unroll
        for (int it = 0; it < 16; ++it) {
          const int rr = (t & ~31) + it * 2 + (lane >> 4), u = lane & 15;
          const uint4 val = *reinterpret_cast<const uint4*>(stage + staged(rr, u));
          if (kv0 + rr < a.Nk) *reinterpret_cast<uint4*>(out + (kv0 + rr) * dst.n + u * 16) = val;
        }
      }
    } else if (ok && nv == 0) {  // nothing sees these keys
      if (n_runs > 1) {
        for (int i = 0; i < D / 4; ++i) partial[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      } else if (j < a.Nk) {
        for (int i = 0; i < D / 8; ++i) *reinterpret_cast<uint4*>(out + j * dst.n + i * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  } else {
    // ----------------------------------------------------------------- dQ
    regs_increase<C::REGS_DQ>();
    const int t = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    constexpr int NCOL = C::DQ_T ? 128 : D;
    Visit v = first;
    for (int it = 0; it < nv; ++it, advance(v)) {
      const int q0 = v.qt * 128;
      if (!__all_sync(0xffffffffu, mbar_wait(bar(C::B_DQ), it & 1, abort_flag, a.status))) break;
      if (!C::DQ_T && t == 0) mbar_arrive(bar(C::B_QEMPTY + it % C::NST));  // (at d = 128 these warps are the later ones)
      tc_fence_after_sync();
      uint32_t x[NCOL];
#pragma unroll
      for (int c0 = 0; c0 < NCOL / 32; ++c0) {
        uint32_t w[32];
        tmem_ld32(tmem + lanes + C::T_DP + c0 * 32, w);
#pragma unroll
        for (int i = 0; i < 32; ++i) x[c0 * 32 + i] = w[i];
      }
      tc_fence_before_sync();
      mbar_arrive(bar(C::B_DQFREE));
      float* acc = p.dq + (static_cast<int64_t>(b) * a.Hq + hk * G + v.g) * a.Nq * D;
      if constexpr (C::DQ_T) {
        float* dst = acc + static_cast<int64_t>(q0) * D + t;
        const int rows = min(128, a.Nq - q0);
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c < rows) red_add_f32(dst + c * D, __uint_as_float(x[c]) * a.scale);
      } else {
        // Lanes l and l ^ m swap the pieces whose index differs from the lane's in
        // bit m, for m = 1, 2, 4: piece k of lane l becomes piece l of lane k.
        const int l8 = t & 7, row0 = q0 + (t & ~7);
#pragma unroll
        for (int g = 0; g < D / 32; ++g) {
          float w[8][4];
#pragma unroll
          for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) w[k][e] = __uint_as_float(x[32 * g + 4 * k + e]);
#pragma unroll
          for (int m = 1; m < 8; m <<= 1) {
            const bool hi = (l8 & m) != 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              if (k & m) continue;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float got = __shfl_xor_sync(0xffffffffu, hi ? w[k][e] : w[k | m][e], m);
                if (hi) w[k][e] = got;
                else w[k | m][e] = got;
              }
            }
          }
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (row0 + k < a.Nq)
              red_add_v4(acc + static_cast<int64_t>(row0 + k) * D + 32 * g + 4 * l8, w[k][0] * a.scale, w[k][1] * a.scale, w[k][2] * a.scale,
                         w[k][3] * a.scale);
        }
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 13) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// Runs to a tile with and without sinks.
void plan_runs(const WindowArgs& a, int sms, WbPlan* p) {
  const int64_t G = a.Hq / a.Hk, heads = static_cast<int64_t>(a.B) * a.Hk, ntq = (a.Nq + 127) / 128;
  const int64_t near = std::min<int64_t>(ntq, (static_cast<int64_t>(a.window) + 126) / 128 + 1);
  const int64_t vs = G * ntq, vw = G * near;  // visits of a tile, at most
  p->tiles = (a.Nk + 127) / 128;
  p->sink_tiles = std::min(p->tiles, (a.sinks + 127) / 128);
  const int64_t w_tiles = heads * (p->tiles - p->sink_tiles), s_tiles = heads * p->sink_tiles;
  const int64_t total = s_tiles * vs + w_tiles * vw;
  // Few tiles: runs of two visits or more until the SMs have one each.
  int64_t runs = 1;
  if (w_tiles + s_tiles < sms) runs = std::max<int64_t>(1, std::min((vw + 1) / 2, sms / std::max<int64_t>(1, w_tiles + s_tiles)));
  const int64_t len = std::max({(vw + runs - 1) / runs, total / (8 * static_cast<int64_t>(sms)), int64_t{2}});
  p->runs = static_cast<int>(runs);
  p->sink_runs = p->sink_tiles ? static_cast<int>((vs + len - 1) / len) : 1;
  p->sink_items = static_cast<int>(s_tiles * p->sink_runs);
}

template <int D, bool BF16>
int launch_t(const WindowArgs& a, int* launches) {
  using C = WbCfg<D>;
  CUtensorMap mq, mk, mv, mdo;
  if (!encode_strided_map(&mq, a.q, a.B, a.Hq, a.Nq, D, C::CH, BF16) || !encode_strided_map(&mk, a.k, a.B, a.Hk, a.Nk, D, C::CH, BF16) ||
      !encode_strided_map(&mv, a.v, a.B, a.Hk, a.Nk, D, C::CH, BF16) || !encode_strided_map(&mdo, a.dO, a.B, a.Hq, a.Nq, D, C::CH, BF16))
    return kStatusCuda;
  auto kern = attn_window_bwd_kernel<D, BF16>;
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kern), C::SMEM)) return kStatusCuda;
  if (!check_launch_regs(reinterpret_cast<const void*>(kern), C::REGS)) return kStatusDeviceCheck;  // the split's sum
  const int sms = device_sm_count();
  if (sms < 1) return kStatusCuda;
  WbPlan p = {};
  plan_runs(a, sms, &p);
  const int64_t heads = static_cast<int64_t>(a.B) * a.Hk, w_items = heads * (p.tiles - p.sink_tiles) * p.runs;
  const int64_t items = p.sink_items + w_items;
  if (items > 0x7fffffff) return kStatusUnsupported;
  p.npad = (a.Nq + 127) / 128 * 128;
  p.group = order_head_group(static_cast<int>(heads), int64_t{8} * a.Nq * D * (a.Hq / a.Hk), int64_t{32} << 20);
  const int64_t bh = static_cast<int64_t>(a.B) * a.Hq, rows = bh * p.npad;
  const int64_t split = (p.sink_runs > 1 ? p.sink_items : 0) + (p.runs > 1 ? w_items : 0);
  auto up = [](int64_t x) { return (x + 255) & ~int64_t{255}; };
  const int64_t dq_bytes = up(bh * a.Nq * D * 4), vec_bytes = up(rows * 4);
  void* ws = nullptr;
  if (cudaMallocAsync(&ws, dq_bytes + 2 * vec_bytes + split * 2 * 128 * D * 4, a.stream) != cudaSuccess) return kStatusCuda;
  uint8_t* at = static_cast<uint8_t*>(ws);
  p.dq = reinterpret_cast<float*>(at);
  p.lse2 = reinterpret_cast<float*>(at + dq_bytes);
  p.dvec = reinterpret_cast<float*>(at + dq_bytes + vec_bytes);
  p.part = reinterpret_cast<float*>(at + dq_bytes + 2 * vec_bytes);
  *launches = 3;
  const bool overlap = overlap_launches(items, 1);
  bool ok = launch_serialized(overlap, attn_window_pre_kernel<D, BF16>, dim3(static_cast<unsigned>((rows * 8 + 255) / 256)), dim3(256), 0,
                              a.stream, a, p) == cudaSuccess;
  ok = ok && launch_serialized(false, kern, dim3(static_cast<unsigned>(items)), dim3(C::THREADS), C::SMEM, a.stream, mq, mk, mv, mdo, a, p) ==
                 cudaSuccess;
  const int64_t work = std::max(bh * a.Nq, split * 256) * (D / 8);
  ok = ok && launch_serialized(overlap, attn_window_out_kernel<D, BF16>, dim3(static_cast<unsigned>(std::min<int64_t>((work + 255) / 256, 16 * sms))),
                               dim3(256), 0, a.stream, a, p) == cudaSuccess;
  ok = cudaFreeAsync(ws, a.stream) == cudaSuccess && ok;
  return ok && cudaGetLastError() == cudaSuccess ? kStatusOk : kStatusCuda;
}

template <int D>
int launch_d(const WindowArgs& a, int* launches) {
  return a.bf16 ? launch_t<D, true>(a, launches) : launch_t<D, false>(a, launches);
}

}  // namespace

int launch_window_bwd(const WindowArgs& a, int* launches) {
  return a.d == 32 ? launch_d<32>(a, launches) : a.d == 64 ? launch_d<64>(a, launches) : launch_d<128>(a, launches);
}

}  // namespace attn
