// attn_window_bwd.cu -- causal attention with a sliding window and sinks,
// backward: with P = exp(s - LSE) on the visible pairs and D_i = dO_i . O_i,
//   dV_j = sum_i P_ij dO_i,  dS = P o (dO V^T - D),
//   dQ = scale dS K,  dK = scale sum_i dS^T Q,
// the sums also over the query heads that share the key/value head
// (FlashAttention (PKM page), "三招" 3 Recomputation; FlashAttention深度攻略 §6).
//
//   attn_window_range_kernel : fp16 only: the largest rows of dO and v, from which come
//       the powers of two that keep dS in fp16's range (F16Range).
//   attn_window_dq_kernel  : an item is 128 query rows of a head, which walk the key
//       tiles they see as the forward does: S = Q K^T, dP = dO V^T, dQ += dS K.  It
//       also leaves -D and -LSE log2(e) of its rows for the next kernel.
//   attn_window_dkv_kernel : an item is 128 keys and the query tiles that see them, of
//       all query heads that share them ("visits"): S^T = K Q^T, dP^T = V dO^T,
//       dV += P^T dO, dK += dS^T Q.  Where a tile has many more visits than others
//       (sinks) or there are few tiles, its visits are cut into runs that leave fp32
//       partial tiles.
//   attn_window_sum_kernel : those, added in the order of the runs.
//
// Seven products a tile instead of the five of one pass that adds dQ up in memory:
// there the additions (64 KB of fp32 a visit at d = 128) paced everything, 7000
// cycles a visit against 4000 of the five products, although the L2 alone takes such
// a tile from every SM in 3000, and the accumulator's zeros and its conversion cost
// another tenth.  Two sequences of 8192, 16 / 4 heads of 128, window 1024, 4 sinks:
// 624 us that way, 504 so (dQ 232, dK and dV 266, sums 13); eight of 1024, 12 heads of
// 64, window 256: 88 and 77.  No sum depends on the order of CTAs, so a call repeats
// bit for bit.
//
// What bounds both loops is a tile's chain, S and dP, the rows' P and dS, the products
// that take those: with one CTA to an SM the tensor pipe waits for the rows and they
// for it.  The products, 128 x 128 x 16 in 64 cycles each at d = 128, are 1536 cycles of
// the 3450 that a tile of dQ takes (pipe active 44 %), 2048 of 3800 for dK and dV (54 %).
//
// P and dS are fp32 until they become operands of 16-bit products, rounded to the
// inputs' type (fp16: times powers of two); everything is summed in fp32.  (Gradients
// are off by 2.4e-3 in norm with bf16, where fp32 operands and the results' own rounding
// make 1.7e-3; fp16 3.0e-4 and 2.2e-4.)
//
// Both loops run on tcgen05, one CTA to an SM: warps 0-7 work on rows, two threads to
// each, 64 columns a thread; warp 8 loads by TMA; one thread of warp 9 issues the
// products.  dS (and P^T, dS^T) goes to TMEM over the half of S (dP) that the thread
// has read and is an operand from there.  A product that overwrites such an operand
// waits for the one that reads it to complete: MMAs run in the order of issue where
// they have one accumulator, no others are promised to.  (Issued right behind, with the
// same bits in 100 forward and 50 backward runs of 54 cases, the long backward above
// takes 487 us, the short one 76.5, two of 500, 8 heads of 32, 18.6 instead of 19.1.)
#include "attn_internal.h"
#include "attn_window_tiles.cuh"

namespace attn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// The dK, dV grid's items: tiles without sinks, the last of them cut into runs of
// their visits, then the runs of the tiles with sinks.
struct WbPlan {
  int tiles, sink_tiles;       // of a key/value head
  int whole, cut;              // tiles without sinks, of all heads: whole and cut
  int runs, sink_runs;         // CTAs to a cut tile and to one with sinks
  int group;                   // heads in flight together
  int npad;                    // rows of a head's row vectors
  float *lse2, *dvec;          // row vectors, padded to whole tiles (-inf, 0), as F16Range has them
  float* part;                 // [item in runs][dK, dV][128][d]
  int blocks;                  // of the range kernel to a key/value head (fp16)
  float2* most;                // [B * Hk][blocks] largest |dO row|^2 and |v|^2
};

// What brings P and dS into fp16's range, normal from 2^-14 to 2^16, where they are
// operands: P = 1 / 1000 of a window times a dO of 1 / 1000 is below it, and a dO of
// 1000 times v of 20 past it.  P is at most 1 and goes as 2^kP P.  O is a mean of rows
// of v, so |dP - D| <= 2 |dO| |v| with the rows' norms, and dS goes as 2^e dS with the
// largest whole e for which that is at most 2^kP (a factor of 4 is left for
// roundings).  The norms are a row's own and v's largest for dQ; for dK, which sums over
// rows, the largest of all rows of the query heads that share the key.  Powers of two
// round nothing, and 2^14 above fp16's last normal number leaves 2^28 for rows and
// weights below the largest.  bf16 has fp32's range.
struct F16Range {
  static constexpr float kP = 14.f;
  static constexpr float kInvP = 1.f / 16384;
  float in, out;  // 2^(e - kP), which makes 2^e dS of 2^kP P, and 2^-e
  // From squared norms, of finite fp16 rows (their product is in fp32's range).
  __device__ __forceinline__ F16Range(float rows, float values) {
    const float m = rows * values;
    const int e = m > 0.f && m < INFINITY ? 12 - (((__float_as_int(m) >> 23) - 127) >> 1) : 0;  // |dO| |v| < 2^(13 - e)
    in = __int_as_float((e - 14 + 127) << 23);
    out = __int_as_float((127 - e) << 23);
  }
};

// Maximum of the warp's values, none below 0: as whole numbers, their bits have the same order.
__device__ __forceinline__ float warp_max(float x) { return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x))); }

// The largest squared norms that the range kernel's blocks found for a key/value head; by a whole warp.
__device__ __forceinline__ float2 most_of(const WbPlan& p, int64_t head, int lane) {
  float2 m = make_float2(0.f, 0.f);
  for (int x = lane; x < p.blocks; x += 32) {
    const float2 y = p.most[head * p.blocks + x];
    m = make_float2(fmaxf(m.x, y.x), fmaxf(m.y, y.y));
  }
  return make_float2(warp_max(m.x), warp_max(m.y));
}

// What both kernels share.
template <int D>
struct Tile : TileLayout<D> {
  static constexpr int THREADS = 384;
  static constexpr int REGS = 168, REGS_ROW = 184, REGS_CTRL = 136;
  static_assert(256 * REGS_ROW + 128 * REGS_CTRL <= THREADS * REGS, "register split");
  static constexpr int W_LOAD = 8, W_MMA = 9;
  static constexpr bool STAGE = D == 128;  // outputs leave through shared memory, whole lines at a time
};

// dQ: Q and dO of an item, rings of K and V tiles.  The item's O, of which only D is
// wanted, passes through the K ring before the keys.
template <int D>
struct DqCfg : Tile<D> {
  using T = Tile<D>;
  static constexpr int NK = 3, NV = 2;  // a K tile is held until its dQ step is complete
  static constexpr int OFF_DO = T::TILE;
  static constexpr int OFF_K = 2 * T::TILE;
  static constexpr int OFF_V = OFF_K + NK * T::TILE;
  static constexpr int OFF_ROWS = OFF_V + NV * T::TILE;  // [2][2][128] fp32: halves of D, of two items
  static constexpr int OFF_NORMS = OFF_ROWS + 4 * 512;   // [2][2][128] bytes: exponents of halves of |dO|^2 (fp16)
  static constexpr int OFF_BAR = OFF_NORMS + 512;
  static constexpr int B_Q = 0;
  static constexpr int B_QEMPTY = 1;
  static constexpr int B_KFULL = 2;
  static constexpr int B_KEMPTY = B_KFULL + NK;
  static constexpr int B_VFULL = B_KEMPTY + NK;
  static constexpr int B_VEMPTY = B_VFULL + NV;
  static constexpr int B_S = B_VEMPTY + NV;   // S(n) is in buffer n & 1
  static constexpr int B_DP = B_S + 2;
  static constexpr int B_TAKEN = B_DP + 1;     // dP is in registers
  static constexpr int B_DS = B_TAKEN + 1;     // dS(n) is in buffer n & 1
  static constexpr int B_READ_DS = B_DS + 2;   // dQ(n), which reads buffer n & 1, is complete
  static constexpr int B_OUT = B_READ_DS + 2;  // the item's dQ is complete
  static constexpr int B_ROWS = B_OUT + 1;     // both halves of the rows' D are in shared memory
  static constexpr int B_NEXT = B_ROWS + 1;
  static constexpr int B_READ = B_NEXT + 2;
  static constexpr int B_DONE = B_READ + 2;
  static constexpr int NBAR = B_DONE + 1;
  static constexpr int OFF_NEXT = (OFF_BAR + NBAR * 8 + 15) & ~15;
  static constexpr int OFF_SLOT = OFF_NEXT + 32;
  static constexpr int OFF_ABORT = OFF_SLOT + 4;
  static constexpr int SMEM = OFF_ABORT + 4;
  static constexpr uint32_t T_S = 0, T_DP = 256, T_DQ = 384;  // S: two buffers of 128
  static_assert(SMEM <= 232448, "shared memory");
};

// dK, dV: K and V of an item, a ring of Q, dO tiles with their rows' vectors.
template <int D>
struct DkvCfg : Tile<D> {
  using T = Tile<D>;
  static constexpr int NST = 2;
  static constexpr int VEC = 128 * 4;
  static constexpr int OFF_V = T::TILE;
  static constexpr int OFF_Q = 2 * T::TILE;
  static constexpr int OFF_DO = OFF_Q + NST * T::TILE;
  static constexpr int OFF_LSE = OFF_DO + NST * T::TILE;
  static constexpr int OFF_D = OFF_LSE + NST * VEC;
  static constexpr int OFF_STAGE = OFF_D + NST * VEC;
  static constexpr int OFF_BAR = OFF_STAGE + (T::STAGE ? 8 * 4096 : 0);
  static constexpr int B_K = 0;
  static constexpr int B_V = 1;
  static constexpr int B_KEMPTY = 2;
  static constexpr int B_VEMPTY = 3;
  static constexpr int B_QFULL = 4;
  static constexpr int B_QEMPTY = B_QFULL + NST;
  static constexpr int B_S = B_QEMPTY + NST;
  static constexpr int B_DP = B_S + 1;
  static constexpr int B_P = B_DP + 1;
  static constexpr int B_DS = B_P + 1;
  static constexpr int B_DV = B_DS + 1;        // dV(n) is complete
  static constexpr int B_OUT = B_DV + 1;       // the item's dK and dV are complete
  static constexpr int B_NEXT = B_OUT + 1;
  static constexpr int B_READ = B_NEXT + 2;
  static constexpr int B_DONE = B_READ + 2;
  static constexpr int NBAR = B_DONE + 1;
  static constexpr int OFF_NEXT = (OFF_BAR + NBAR * 8 + 15) & ~15;
  static constexpr int OFF_SLOT = OFF_NEXT + 32;
  static constexpr int OFF_ABORT = OFF_SLOT + 4;
  static constexpr int SMEM = OFF_ABORT + 4;
  static constexpr uint32_t T_S = 0, T_DP = 128, T_DK = 256, T_DV = 256 + D;
  static_assert(SMEM <= 232448, "shared memory");
};

// TMEM columns of the 16-deep slice kk of an operand whose halves lie 64 columns apart.
__host__ __device__ constexpr uint32_t half_step(int kk) { return static_cast<uint32_t>((kk >> 2) * 64 + (kk & 3) * 8); }

// Byte offset of 16-byte unit u of a row in a tile, as TMA has laid it.
template <int D>
__device__ __forceinline__ uint32_t tile_unit(int row, int u) {
  if constexpr (D >= 64) return static_cast<uint32_t>((u >> 3) * Tile<D>::CHUNK + row * 128 + (((u & 7) ^ (row & 7)) << 4));
  else return static_cast<uint32_t>(row * 64 + ((u ^ ((row >> 1) & 3)) << 4));
}

// Byte offset of 16-byte unit u of a row of 128 bytes in a warp's staging copy,
// swizzled so that rows by threads and units by threads meet no bank twice.
__device__ __forceinline__ uint32_t staged(int row, int u) { return static_cast<uint32_t>(row * 128 + ((u ^ (row & 7)) << 4)); }

// A warp's 32 rows of 64 channels, 16 packed words of 32 channels in `lo` and `hi`, to
// out + row * stride: through shared memory, 128 contiguous bytes a row.
__device__ __forceinline__ void store_rows(uint8_t* stage, int lane, const uint32_t (&w)[32], uint8_t* out, int64_t stride, int rows) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    *reinterpret_cast<uint4*>(stage + staged(lane, e)) = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
  __syncwarp();
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    const int r = x * 4 + (lane >> 3), u = lane & 7;
    const uint4 val = *reinterpret_cast<const uint4*>(stage + staged(r, u));
    if (r < rows) *reinterpret_cast<uint4*>(out + r * stride + u * 16) = val;
  }
  __syncwarp();
}

template <bool BF16>
__device__ __forceinline__ float scaled(uint32_t x, float unmul, float scale) {
  return (BF16 ? __uint_as_float(x) : __uint_as_float(x) * unmul) * scale;
}

// Sum of squares of eight fp16 values.
__device__ __forceinline__ float square_of(const uint4& v) {
  const float2 a = unpack2<false>(v.x), b = unpack2<false>(v.y), c = unpack2<false>(v.z), d = unpack2<false>(v.w);
  return ((a.x * a.x + a.y * a.y) + (b.x * b.x + b.y * b.y)) + ((c.x * c.x + c.y * c.y) + (d.x * d.x + d.y * d.y));
}

// ---------------------------------------------------------------------- range
// Largest squared norms of the rows of dO and of the v that are seen, a block's share of a key/value
// head's; the row kernels join the blocks' (most_of).  16 bytes a thread, D / 8 threads
// to a row.  Bytes bound it where it is more than a launch: 84 MB of two sequences of
// 8192, 16 / 4 heads of 128, in 20 us, of 12.4 at the copy's rate.  With it and what
// the row kernels do with it, fp16's backward takes 528 us there where bf16's takes 487,
// 86 against 77 for eight of 1024, 12 heads of 64, 21.6 against 18.6 for two of 500, 8 heads of 32.
constexpr int kRangeThreads = 256;

template <int D>
__global__ void __launch_bounds__(kRangeThreads) attn_window_range_kernel(const WindowArgs a, const WbPlan p) {
  griddep_wait();  // launched overlapped (launch_serialized)
  griddep_launch_dependents();
  constexpr int U = D / 8, ROWS = kRangeThreads / U, AHEAD = 4;
  const int part = blockIdx.x, hb = blockIdx.y, b = hb / a.Hk, hk = hb - b * a.Hk, G = a.Hq / a.Hk;
  const int u = threadIdx.x % U, in_warp = threadIdx.x % 32 / U, step = p.blocks * ROWS;
  const int first = part * ROWS + static_cast<int>(threadIdx.x) / 32 * (32 / U);  // of the warp's rows
  auto most = [&](const uint8_t* base, int64_t stride, int from, int n) {
    float m = 0.f;
    for (int w0 = from + first; w0 < n; w0 += AHEAD * step) {
      const int r0 = w0 + in_warp;
      uint4 v[AHEAD];
#pragma unroll
      for (int x = 0; x < AHEAD; ++x)
        v[x] = r0 + x * step < n ? *reinterpret_cast<const uint4*>(base + (r0 + x * step) * stride + u * 16) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int x = 0; x < AHEAD; ++x) {
        float s = square_of(v[x]);
#pragma unroll
        for (int y = 1; y < U; y <<= 1) s += __shfl_xor_sync(0xffffffffu, s, y);
        m = fmaxf(m, s);
      }
    }
    return m;
  };
  // Keys that some query sees: the sinks, and from the first query's window on.
  const uint8_t* v = a.v.p + b * a.v.b + hk * a.v.h;
  const int near = max(0, a.Nk - a.Nq - a.window + 1);
  float2 m = make_float2(0.f, fmaxf(most(v, a.v.n, 0, min(a.sinks, near)), most(v, a.v.n, near, a.Nk)));
  for (int g = 0; g < G; ++g) m.x = fmaxf(m.x, most(a.dO.p + b * a.dO.b + (hk * G + g) * a.dO.h, a.dO.n, 0, a.Nq));
  __shared__ float2 warps[kRangeThreads / 32];
  m = make_float2(warp_max(m.x), warp_max(m.y));
  if (threadIdx.x % 32 == 0) warps[threadIdx.x / 32] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (const float2& w : warps) m = make_float2(fmaxf(m.x, w.x), fmaxf(m.y, w.y));
    p.most[static_cast<int64_t>(hb) * p.blocks + part] = m;
  }
}

// ------------------------------------------------------------------------- dQ
template <int D, bool BF16>
__global__ void __launch_bounds__(DqCfg<D>::THREADS, 1)
    attn_window_dq_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                          const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mdo,
                          const __grid_constant__ CUtensorMap mo, const WindowArgs a, const WbPlan pl, int nrows, int group) {
  using C = DqCfg<D>;
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
  const uint32_t sDO = sbase + C::OFF_DO, sK = sbase + C::OFF_K, sV = sbase + C::OFF_V;
  if (warp == C::W_LOAD && lane == 0) {
    for (int x = 0; x < C::NBAR; ++x) mbar_init(bar(x), 1);
    for (int x : {C::B_TAKEN, C::B_DS, C::B_DS + 1, C::B_ROWS}) mbar_init(bar(x), 256);
    for (int x = 0; x < 2; ++x) mbar_init(bar(C::B_READ + x), 9);  // 8 warps and the issuer
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&mq);
    prefetch_tensormap(&mk);
    prefetch_tensormap(&mv);
    prefetch_tensormap(&mdo);
    prefetch_tensormap(&mo);
  }
  if (warp == C::W_MMA) {
    tmem_alloc(smem_addr(slot), 512);
    tmem_relinquish();
  }
  griddep_wait();  // launched overlapped (launch_serialized): what is above reads no tensor
  griddep_launch_dependents();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *slot;
  const Items items = {sbase + C::OFF_NEXT, bar(C::B_NEXT), bar(C::B_READ), abort_flag, a.status};
  // `n` counts positions over all items and gives buffers, V stages and phases; the K
  // ring has item k's O at n + k, its first key tile behind it.

  if (warp >= C::W_LOAD) {
    regs_decrease<C::REGS_CTRL>();
    if (warp == C::W_LOAD && lane == 0) {
      // -------------------------------------------------------------- loads
      auto load = [&](uint32_t dst, const CUtensorMap* map, uint32_t full, int row, int head, int b) {
#pragma unroll
        for (int c = 0; c < C::NCH; ++c) tma_load_4d(dst + c * C::CHUNK, map, full, c * C::CH, row, head, b);
      };
      int asked = 0, nk = 0, nv = 0, nq = 0;
      bool ok = true;
      for (int i = blockIdx.x; ok && i >= 0;) {
        if (!(ok = items.ask(asked))) break;
        ++asked;
        const RowItem it(a, i, nrows, group);
        auto load_k = [&](const CUtensorMap* map, int row, int head) {
          const int s = nk % C::NK;
          if (nk >= C::NK && !(ok = mbar_wait(bar(C::B_KEMPTY + s), (nk / C::NK - 1) & 1, abort_flag, a.status))) return;
          mbar_arrive_expect_tx(bar(C::B_KFULL + s), C::TILE);
          load(sK + s * C::TILE, map, bar(C::B_KFULL + s), row, head, it.b);
          ++nk;
        };
        load_k(&mo, it.row0, it.h);
        for (int p = 0; ok && p < it.npos; ++p) {
          const int sv = nv % C::NV;
          load_k(&mk, it.key0(p), it.hk);
          if (!ok) break;
          if (p == 0) {
            if (nq > 0 && !(ok = mbar_wait(bar(C::B_QEMPTY), (nq - 1) & 1, abort_flag, a.status))) break;
            mbar_arrive_expect_tx(bar(C::B_Q), 2 * C::TILE);
            load(sbase, &mq, bar(C::B_Q), it.row0, it.h, it.b);
            load(sDO, &mdo, bar(C::B_Q), it.row0, it.h, it.b);
            ++nq;
          }
          if (nv >= C::NV && !(ok = mbar_wait(bar(C::B_VEMPTY + sv), (nv / C::NV - 1) & 1, abort_flag, a.status))) break;
          mbar_arrive_expect_tx(bar(C::B_VFULL + sv), C::TILE);
          load(sV + sv * C::TILE, &mv, bar(C::B_VFULL + sv), it.key0(p), it.hk, it.b);
          ++nv;
        }
        i = items.after(asked - 1, ok);
      }
      if (*abort_flag) {  // what is in flight lands before the shared memory goes
        items.drain_last(asked);
        if (nq) drain(bar(C::B_Q), (nq - 1) & 1);
        for (int s = 0; s < C::NK; ++s)
          if (nk > s) drain(bar(C::B_KFULL + s), ((nk - 1 - s) / C::NK) & 1);
        for (int s = 0; s < C::NV; ++s)
          if (nv > s) drain(bar(C::B_VFULL + s), ((nv - 1 - s) / C::NV) & 1);
      }
    } else if (warp == C::W_MMA && lane == 0) {
      // ------------------------------------------------- matrix instructions
      // Three chains over an item's positions, each step issued as soon as it is ready:
      //   S(n)  needs K(n), and dQ(n - 2) complete, whose dS it overwrites
      //   dP(n) needs V(n), and dP(n - 1) in registers
      //   dQ(n) needs dS(n); the item's first overwrites a dQ that has been read
      constexpr uint32_t HI = smem_desc_hi(C::SBO, C::SWZ);
      const uint32_t id_s = instr_desc_f16(128, 128, BF16, false, false, a.negate != 0);
      const uint32_t id_dp = instr_desc_f16(128, 128, BF16, false, false);
      const uint32_t id_dq = instr_desc_f16(128, D, BF16, false, true);
      const uint32_t q_lo = smem_desc_lo(sbase, 16), do_lo = smem_desc_lo(sDO, 16);
      bool ok = true;
      int n0 = 0;
      IdleWatch watch;
      for (int i = blockIdx.x, k = 0; ok && i >= 0; ++k) {
        const int end = n0 + RowItem(a, i, nrows, group).npos;
        ok = mbar_wait(bar(C::B_Q), k & 1, abort_flag, a.status);
        int is = n0, ip = n0, iq = n0;
        const int ahead = k + 1;  // O tiles in the K ring so far
        while (ok && iq < end) {
          bool progress = false;
          if (ip < end && (ip == 0 || mbar_probe(bar(C::B_TAKEN), (ip - 1) & 1)) &&
              mbar_probe(bar(C::B_VFULL + ip % C::NV), (ip / C::NV) & 1)) {
            tc_fence_after_sync();
            const uint32_t v_lo = smem_desc_lo(sV + (ip % C::NV) * C::TILE, 16);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ss_w(tmem + C::T_DP, do_lo + k_step<D>(kk), HI, v_lo + k_step<D>(kk), HI, id_dp, kk > 0 ? 1u : 0u);
            tc_commit(bar(C::B_DP));
            ++ip;
            progress = true;
          }
          if (is < end && is <= iq + 1 && (is < 2 || mbar_probe(bar(C::B_READ_DS + (is & 1)), (is / 2 - 1) & 1)) &&
              mbar_probe(bar(C::B_KFULL + (is + ahead) % C::NK), ((is + ahead) / C::NK) & 1)) {
            tc_fence_after_sync();
            const uint32_t k_lo = smem_desc_lo(sK + ((is + ahead) % C::NK) * C::TILE, 16);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ss_w(tmem + C::T_S + (is & 1) * 128, q_lo + k_step<D>(kk), HI, k_lo + k_step<D>(kk), HI, id_s, kk > 0 ? 1u : 0u);
            tc_commit(bar(C::B_S + (is & 1)));
            ++is;
            progress = true;
          }
          if (iq < ip && mbar_probe(bar(C::B_DS + (iq & 1)), (iq >> 1) & 1)) {
            tc_fence_after_sync();
            const uint32_t k_lo = smem_desc_lo(sK + ((iq + ahead) % C::NK) * C::TILE, C::CHUNK);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_ts_w(tmem + C::T_DQ, tmem + C::T_S + (iq & 1) * 128 + half_step(kk), k_lo + mn_step<D>(kk), HI, id_dq,
                       (iq > n0 || kk > 0) ? 1u : 0u);
            tc_commit(bar(C::B_KEMPTY + (iq + ahead) % C::NK));
            tc_commit(bar(C::B_READ_DS + (iq & 1)));
            if (++iq == end) tc_commit(bar(C::B_OUT));
            progress = true;
          }
          if (progress) watch.progress();
          else ok = watch.idle(abort_flag, a.status, kWaitLimitNs);
        }
        n0 = end;
        i = items.after(k, ok);
        items.read(k);
      }
      tc_commit(bar(C::B_DONE));  // before TMEM is released
      drain(bar(C::B_DONE), 0);
    }
    __syncwarp();
  } else {
    // ----------------------------------------------------------------- dS
    regs_increase<C::REGS_ROW>();
    const int half = warp >> 2, r = threadIdx.x & 127, off = a.Nk - a.Nq;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float2 sl2x2 = make_float2(a.sl2, a.sl2);
    bool ok = true;
    int n = 0;
    for (int i = blockIdx.x, k = 0; ok && i >= 0; ++k) {
      const RowItem it(a, i, nrows, group);
      const int row = it.row0 + r;
      const int64_t bh = static_cast<int64_t>(it.b) * a.Hq + it.h;
      const float lse2 = row < a.Nq ? -a.lse[bh * a.Nq + row] * kLog2e + (BF16 ? 0.f : F16Range::kP) : -INFINITY;
      float2 most = make_float2(0.f, 0.f);
      if constexpr (!BF16) most = most_of(pl, static_cast<int64_t>(it.b) * a.Hk + it.hk, lane);
      // D, half a row a thread, while the first products run.
      ok = mbar_wait(bar(C::B_KFULL + (n + k) % C::NK), ((n + k) / C::NK) & 1, abort_flag, a.status) &&
           mbar_wait(bar(C::B_Q), k & 1, abort_flag, a.status);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      float d = 0.f, norm = 0.f;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        const uint32_t at = tile_unit<D>(r, half * (D / 16) + c);
        const uint4 x = *reinterpret_cast<const uint4*>(smem + C::OFF_K + (n + k) % C::NK * C::TILE + at);
        const uint4 y = *reinterpret_cast<const uint4*>(smem + C::OFF_DO + at);
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = unpack2<BF16>(xw[e]), g = unpack2<BF16>(yw[e]);
          d = fmaf(f.x, g.x, fmaf(f.y, g.y, d));
          if (!BF16) norm = fmaf(g.x, g.x, fmaf(g.y, g.y, norm));
        }
      }
      float* sum = reinterpret_cast<float*>(smem + C::OFF_ROWS) + (k & 1) * 256 + r;  // (who writes here again has waited for the item between)
      uint8_t* norms = smem + C::OFF_NORMS + (k & 1) * 256 + r;
      sum[half * 128] = d;
      if (!BF16) norms[half * 128] = static_cast<uint8_t>(__float_as_uint(norm) >> 23);
      mbar_arrive(bar(C::B_ROWS));
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_ROWS), k & 1, abort_flag, a.status)))) break;
      if (threadIdx.x == 0) {
        fence_proxy_async_smem();  // O is read before its stage is loaded again
        mbar_arrive(bar(C::B_KEMPTY + (n + k) % C::NK));
      }
      float nd = -(sum[0] + sum[128]), mul = 1.f, unmul = 1.f;
      if (half == 0) {
        pl.lse2[bh * pl.npad + row] = lse2;
        pl.dvec[bh * pl.npad + row] = BF16 ? nd : nd * F16Range(most.x, most.y).in;
      }
      if constexpr (!BF16) {
        const int up = max(norms[0], norms[128]);  // |dO|^2 < 2^(up - 125)
        const F16Range range(up ? __int_as_float((up + 2) << 23) : 0.f, most.y);
        mul = range.in, unmul = range.out, nd *= mul;
      }
      const float2 l2 = make_float2(lse2, lse2), nd2 = make_float2(nd, nd), mul2x2 = make_float2(mul, mul);
      for (int p = 0; p < it.npos; ++p, ++n) {
        // (a warp's lanes go on or stop together: what follows wants all of them)
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_S + (n & 1)), (n >> 1) & 1, abort_flag, a.status)))) break;
        tc_fence_after_sync();
        const uint32_t tS = tmem + lanes + C::T_S + (n & 1) * 128 + half * 64;
        float pr[64];
        {
          uint32_t u[64];
          tmem_ld64(tS, u);
#pragma unroll
          for (int c = 0; c < 64; ++c) pr[c] = __uint_as_float(u[c]);
        }
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          const float2 e = fma2(make_float2(pr[c], pr[c + 1]), sl2x2, l2);
          pr[c] = ex2_approx(e.x);
          pr[c + 1] = ex2_approx(e.y);
        }
        // Key kv0 + c is visible iff c <= at and (c >= first or c < sinks).
        const int kv0 = it.key0(p) + half * 64, at = row + off - kv0;
        if (kv0 + 63 > it.row0 + off) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c > at) pr[c] = 0.f;
        }
        if (kv0 < it.row0 + 127 + off - a.window + 1 && kv0 + 64 > a.sinks) {
          const int first = at - a.window + 1, sinks = a.sinks - kv0;
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c < first && c >= sinks) pr[c] = 0.f;
        }
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_DP), n & 1, abort_flag, a.status)))) break;
        tc_fence_after_sync();
        if (threadIdx.x == 0) {
          mbar_arrive(bar(C::B_VEMPTY + n % C::NV));
          if (p == it.npos - 1) mbar_arrive(bar(C::B_QEMPTY));  // (S of this position is complete too)
        }
        uint32_t dp[64], pk[32];
        tmem_ld64(tmem + lanes + C::T_DP + half * 64, dp);
        tc_fence_before_sync();
        mbar_arrive(bar(C::B_TAKEN));
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float2 x = make_float2(__uint_as_float(dp[2 * e]), __uint_as_float(dp[2 * e + 1])), gd = BF16 ? add2(x, nd2) : fma2(x, mul2x2, nd2);
          const float2 ds = mul2(make_float2(pr[2 * e], pr[2 * e + 1]), gd);
          pk[e] = pack2<BF16>(ds.x, ds.y);
        }
        tmem_st32(tS, pk);
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(bar(C::B_DS + (n & 1)));
      }
      // ------------------------------------------------------------ output
      if (!(ok = __all_sync(0xffffffffu, ok && mbar_wait(bar(C::B_OUT), k & 1, abort_flag, a.status)))) break;
      tc_fence_after_sync();
      uint8_t* out = a.dq.p + it.b * a.dq.b + it.h * a.dq.h;
      // A thread's channels: 64 at d = 128, else 32 (a line or half of one).
#pragma unroll
      for (int c0 = 0; c0 < (D == 128 ? 2 : 1); ++c0) {
        const int c = half * (D == 128 ? 64 : 32) + c0 * 32;
        if (c >= D) break;
        uint32_t x[32];
        tmem_ld32(tmem + lanes + C::T_DQ + c, x);
        if (row < a.Nq) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int f = 0; f < 4; ++f)
              w[f] = pack2<BF16>(scaled<BF16>(x[8 * e + 2 * f], unmul, a.scale), scaled<BF16>(x[8 * e + 2 * f + 1], unmul, a.scale));
            *reinterpret_cast<uint4*>(out + row * a.dq.n + c * 2 + e * 16) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      tc_fence_before_sync();  // dQ is read before this thread's next dS lets it be overwritten
      i = items.after(k, ok);
      items.read_by_warp(k, lane, ok);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == C::W_MMA) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// --------------------------------------------------------------------- dK, dV
struct Visit {
  int g, qt;  // query head within the group, query tile
};

// Key tile jt of head hb, and a run of its visits.
struct DkvItem {
  int b, hk, kv0;    // sequence, key/value head, first key
  int q_lo, nt, nv;  // first query tile that sees the keys, how many do; visits of the run
  int n_runs;
  Visit first;
  int64_t slot;      // among the partial tiles
  __device__ __forceinline__ DkvItem(const WindowArgs& a, const WbPlan& p, int item) {
    const int heads = a.B * a.Hk, G = a.Hq / a.Hk, off = a.Nk - a.Nq, cut_items = p.cut * p.runs;
    int at = item - p.whole, tile = item, run = 0, jt, hb;  // at: among the items in runs
    slot = 0, n_runs = 1;
    if (at >= cut_items) {
      slot = at - (p.runs > 1 ? 0 : cut_items);
      at -= cut_items;
      n_runs = p.sink_runs, tile = at / n_runs, run = at - tile * n_runs;
      hb = tile / p.sink_tiles, jt = tile - hb * p.sink_tiles;
    } else {
      if (at >= 0) slot = at, n_runs = p.runs, tile = at / n_runs, run = at - tile * n_runs, tile += p.whole;
      grouped_rank_order(tile, p.tiles - p.sink_tiles, heads, p.group, jt, hb);
      jt += p.sink_tiles;
    }
    b = hb / a.Hk, hk = hb - b * a.Hk, kv0 = jt * 128;
    q_lo = max(0, kv0 - off) >> 7;
    const int last = kv0 < a.sinks ? a.Nq - 1 : min(a.Nq - 1, kv0 + 126 + a.window - off);
    nt = kv0 - off >= a.Nq || last < 0 ? 0 : (last >> 7) + 1 - q_lo;
    const int64_t all = static_cast<int64_t>(nt) * G;
    const int v0 = static_cast<int>(all * run / n_runs);
    nv = static_cast<int>(all * (run + 1) / n_runs) - v0;
    first = {nt ? v0 / nt : 0, nt ? q_lo + v0 % nt : 0};
  }
  __device__ __forceinline__ void advance(Visit& v) const {
    if (++v.qt == q_lo + nt) v.qt = q_lo, ++v.g;
  }
};

template <int D, bool BF16>
__global__ void __launch_bounds__(DkvCfg<D>::THREADS, 1)
    attn_window_dkv_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                           const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mdo, const WindowArgs a,
                           const WbPlan p) {
  using C = DkvCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.Hq / a.Hk, off = a.Nk - a.Nq;
  const uint32_t sbase = smem_addr(smem);
  if (sbase & 1023u) {  // the swizzle's atoms; never expected
    if (threadIdx.x == 0) atomicExch(a.status, kStatusDeviceCheck);
    return;
  }
  auto bar = [&](int i) -> uint32_t { return sbase + C::OFF_BAR + 8u * static_cast<uint32_t>(i); };
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + C::OFF_SLOT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
  const uint32_t sV = sbase + C::OFF_V, sQ = sbase + C::OFF_Q, sDO = sbase + C::OFF_DO;
  if (warp == C::W_LOAD && lane == 0) {
    for (int x = 0; x < C::NBAR; ++x) {
      const bool rows = x == C::B_P || x == C::B_DS;
      mbar_init(bar(x), rows ? 256 : x == C::B_READ || x == C::B_READ + 1 ? 9 : 1);  // (read by 8 warps and the issuer)
    }
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&mq);
    prefetch_tensormap(&mk);
    prefetch_tensormap(&mv);
    prefetch_tensormap(&mdo);
  }
  if (warp == C::W_MMA) {
    tmem_alloc(smem_addr(slot), 512);
    tmem_relinquish();
  }
  griddep_wait();  // launched overlapped (launch_serialized): what is above reads no tensor
  griddep_launch_dependents();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *slot;
  const Items items = {sbase + C::OFF_NEXT, bar(C::B_NEXT), bar(C::B_READ), abort_flag, a.status};
  // `n` counts visits over all items and gives stages and phases.

  if (warp >= C::W_LOAD) {
    regs_decrease<C::REGS_CTRL>();
    if (warp == C::W_LOAD && lane == 0) {
      // -------------------------------------------------------------- loads
      int asked = 0, nk = 0, nv = 0, n = 0;
      bool ok = true;
      for (int i = blockIdx.x; ok && i >= 0;) {
        if (!(ok = items.ask(asked))) break;
        ++asked;
        const DkvItem w(a, p, i);
        Visit v = w.first;
        auto load_keys = [&](uint32_t dst, const CUtensorMap* map, int full, int empty, int& count) {
          if (count > 0 && !(ok = mbar_wait(bar(empty), (count - 1) & 1, abort_flag, a.status))) return;
          mbar_arrive_expect_tx(bar(full), C::TILE);
          for (int c = 0; c < C::NCH; ++c) tma_load_4d(dst + c * C::CHUNK, map, bar(full), c * C::CH, w.kv0, w.hk, w.b);
          ++count;
        };
        if (w.nv > 0) load_keys(sbase, &mk, C::B_K, C::B_KEMPTY, nk);
        for (int it = 0; ok && it < w.nv; ++it, ++n, w.advance(v)) {
          const int s = n % C::NST;
          if (n >= C::NST && !(ok = mbar_wait(bar(C::B_QEMPTY + s), (n / C::NST - 1) & 1, abort_flag, a.status))) break;
          const uint32_t full = bar(C::B_QFULL + s);
          const int q0 = v.qt * 128, h = w.hk * G + v.g;
          mbar_arrive_expect_tx(full, 2 * C::TILE + 2 * C::VEC);
          for (int c = 0; c < C::NCH; ++c) tma_load_4d(sQ + s * C::TILE + c * C::CHUNK, &mq, full, c * C::CH, q0, h, w.b);
          for (int c = 0; c < C::NCH; ++c) tma_load_4d(sDO + s * C::TILE + c * C::CHUNK, &mdo, full, c * C::CH, q0, h, w.b);
          const int64_t at = (static_cast<int64_t>(w.b) * a.Hq + h) * p.npad + q0;
          bulk_load(sbase + C::OFF_LSE + s * C::VEC, p.lse2 + at, C::VEC, full);
          bulk_load(sbase + C::OFF_D + s * C::VEC, p.dvec + at, C::VEC, full);
          if (it == 0) load_keys(sV, &mv, C::B_V, C::B_VEMPTY, nv);
        }
        i = items.after(asked - 1, ok);
      }
      if (*abort_flag) {  // what is in flight lands before the shared memory goes
        items.drain_last(asked);
        if (nk) drain(bar(C::B_K), (nk - 1) & 1);
        if (nv) drain(bar(C::B_V), (nv - 1) & 1);
        for (int s = 0; s < C::NST; ++s)
          if (n > s) drain(bar(C::B_QFULL + s), ((n - 1 - s) / C::NST) & 1);
      }
    } else if (warp == C::W_MMA && lane == 0) {
      // ------------------------------------------------- matrix instructions
      // Four chains over an item's visits, each step issued as soon as it is ready:
      //   S(n)  needs Q_n, and dV(n - 1) complete, whose P^T it overwrites
      //   dP(n) needs dO_n, and dK(n - 1) complete, whose dS^T it overwrites
      //   dV(n) needs P^T(n), dK(n) needs dS^T(n); the item's first overwrite a dV, dK
      //         that have been read
      // S(n + 1) does not wait for dK(n), so that P^T(n + 1) is worked on while dK(n) and
      // dP(n + 1) run.
      constexpr uint32_t HI = smem_desc_hi(C::SBO, C::SWZ);
      const uint32_t id_s = instr_desc_f16(128, 128, BF16, false, false, a.negate != 0);
      const uint32_t id_dp = instr_desc_f16(128, 128, BF16, false, false);
      const uint32_t id_out = instr_desc_f16(128, D, BF16, false, true);
      const uint32_t k_lo = smem_desc_lo(sbase, 16), v_lo = smem_desc_lo(sV, 16);
      bool ok = true;
      int n0 = 0, keys = 0;  // visits and key tiles of the items before
      IdleWatch watch;
      for (int i = blockIdx.x, k = 0; ok && i >= 0; ++k) {
        const int end = n0 + DkvItem(a, p, i).nv;
        if (end > n0) {
          ok = mbar_wait(bar(C::B_K), keys & 1, abort_flag, a.status) && mbar_wait(bar(C::B_V), keys & 1, abort_flag, a.status);
          ++keys;
          tc_fence_after_sync();
        }
        int is = n0, ip = n0, iv = n0, ik = n0;
        while (ok && ik < end) {
          bool progress = false;
          if (iv < is && mbar_probe(bar(C::B_P), iv & 1)) {
            tc_fence_after_sync();
            const uint32_t do_lo = smem_desc_lo(sDO + (iv % C::NST) * C::TILE, C::CHUNK);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_ts_w(tmem + C::T_DV, tmem + C::T_S + half_step(kk), do_lo + mn_step<D>(kk), HI, id_out, (iv > n0 || kk > 0) ? 1u : 0u);
            tc_commit(bar(C::B_DV));
            ++iv;
            progress = true;
          }
          if (is < end && is == iv && (is == 0 || mbar_probe(bar(C::B_DV), (is - 1) & 1)) && mbar_probe(bar(C::B_QFULL + is % C::NST), (is / C::NST) & 1)) {
            tc_fence_after_sync();
            const uint32_t q_lo = smem_desc_lo(sQ + (is % C::NST) * C::TILE, 16);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ss_w(tmem + C::T_S, k_lo + k_step<D>(kk), HI, q_lo + k_step<D>(kk), HI, id_s, kk > 0 ? 1u : 0u);
            tc_commit(bar(C::B_S));
            ++is;
            progress = true;
          }
          if (ik < iv && ik < ip && mbar_probe(bar(C::B_DS), ik & 1)) {
            tc_fence_after_sync();
            const uint32_t q_lo = smem_desc_lo(sQ + (ik % C::NST) * C::TILE, C::CHUNK);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_ts_w(tmem + C::T_DK, tmem + C::T_DP + half_step(kk), q_lo + mn_step<D>(kk), HI, id_out, (ik > n0 || kk > 0) ? 1u : 0u);
            tc_commit(bar(C::B_QEMPTY + ik % C::NST));
            if (++ik == end) tc_commit(bar(C::B_OUT));
            progress = true;
          }
          if (ip < is && ip == ik && (ip == 0 || mbar_probe(bar(C::B_QEMPTY + (ip - 1) % C::NST), ((ip - 1) / C::NST) & 1))) {  // (Q_n and dO_n land together)
            tc_fence_after_sync();
            const uint32_t do_lo = smem_desc_lo(sDO + (ip % C::NST) * C::TILE, 16);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ss_w(tmem + C::T_DP, v_lo + k_step<D>(kk), HI, do_lo + k_step<D>(kk), HI, id_dp, kk > 0 ? 1u : 0u);
            tc_commit(bar(C::B_DP));
            ++ip;
            progress = true;
          }
          if (progress) watch.progress();
          else ok = watch.idle(abort_flag, a.status, kWaitLimitNs);
        }
        n0 = end;
        i = items.after(k, ok);
        items.read(k);
      }
      tc_commit(bar(C::B_DONE));  // before TMEM is released
      drain(bar(C::B_DONE), 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------- P^T and dS^T
    regs_increase<C::REGS_ROW>();
    const int half = warp >> 2, t = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + C::T_S + half * 64, tDP = tmem + lanes + C::T_DP + half * 64;
    const float* s_lse = reinterpret_cast<const float*>(smem + C::OFF_LSE);
    const float* s_d = reinterpret_cast<const float*>(smem + C::OFF_D);
    const float2 sl2x2 = make_float2(a.sl2, a.sl2);
    bool ok = true;
    int n = 0, outs = 0;
    for (int i = blockIdx.x, k = 0; ok && i >= 0; ++k) {
      const DkvItem w(a, p, i);
      const int j = w.kv0 + t;
      // Row i sees this key iff from <= i < to.
      const int from = j < a.Nk ? j - off : a.Nq, to = j < a.sinks ? a.Nq : j - off + a.window;
      Visit v = w.first;
      float2 mul2x2 = make_float2(1.f, 1.f);
      float unmul = 1.f;
      if (!BF16 && w.nv > 0) {  // (D's vector has `in` already)
        const float2 most = most_of(p, static_cast<int64_t>(w.b) * a.Hk + w.hk, lane);
        const F16Range range(most.x, most.y);
        mul2x2 = make_float2(range.in, range.in), unmul = half ? F16Range::kInvP : range.out;
      }
      for (int it = 0; it < w.nv; ++it, ++n, w.advance(v)) {
        const int s = n % C::NST, q0 = v.qt * 128 + half * 64;
        // (a warp's lanes go on or stop together: what follows wants all of them)
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_S), n & 1, abort_flag, a.status)))) break;
        tc_fence_after_sync();
        if (threadIdx.x == 0 && it == w.nv - 1) mbar_arrive(bar(C::B_KEMPTY));
        float pr[64];
        {
          uint32_t u[64];
          tmem_ld64(tS, u);
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
        uint32_t pk[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) pk[e] = pack2<BF16>(pr[2 * e], pr[2 * e + 1]);
        tmem_st32(tS, pk);
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(bar(C::B_P));
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_DP), n & 1, abort_flag, a.status)))) break;
        tc_fence_after_sync();
        if (threadIdx.x == 0 && it == w.nv - 1) mbar_arrive(bar(C::B_VEMPTY));
        const float2* nd = reinterpret_cast<const float2*>(s_d + s * 128 + half * 64);
        uint32_t dp[64];
        tmem_ld64(tDP, dp);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float2 x = make_float2(__uint_as_float(dp[2 * e]), __uint_as_float(dp[2 * e + 1])), gd = BF16 ? add2(x, nd[e]) : fma2(x, mul2x2, nd[e]);
          const float2 ds = mul2(make_float2(pr[2 * e], pr[2 * e + 1]), gd);
          pk[e] = pack2<BF16>(ds.x, ds.y);
        }
        tmem_st32(tDP, pk);
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(bar(C::B_DS));
      }
      if (!ok) break;
      // dK (warps 0-3, times scale) or dV.
      const Bhnd& dst = half ? a.dv : a.dk;
      uint8_t* out = dst.p + w.b * dst.b + w.hk * dst.h;
      float4* partial = reinterpret_cast<float4*>(p.part + ((w.slot * 2 + half) * 128 + t) * D);
      const float mul = half ? 1.f : a.scale;
      if (w.nv > 0) {
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_OUT), outs & 1, abort_flag, a.status)))) break;
        ++outs;
        tc_fence_after_sync();
        const uint32_t col = tmem + lanes + (half ? C::T_DV : C::T_DK);
        if (w.n_runs > 1) {
#pragma unroll
          for (int c0 = 0; c0 < D / 32; ++c0) {
            uint32_t x[32];
            tmem_ld32(col + c0 * 32, x);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              partial[c0 * 8 + e] = make_float4(scaled<BF16>(x[4 * e], unmul, mul), scaled<BF16>(x[4 * e + 1], unmul, mul),
                                                scaled<BF16>(x[4 * e + 2], unmul, mul), scaled<BF16>(x[4 * e + 3], unmul, mul));
          }
        } else if constexpr (C::STAGE) {
          const int row_w = w.kv0 + (warp & 3) * 32;
#pragma unroll
          for (int c0 = 0; c0 < 2; ++c0) {
            uint32_t x[64], y[32];
            tmem_ld64(col + c0 * 64, x);
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = pack2<BF16>(scaled<BF16>(x[2 * e], unmul, mul), scaled<BF16>(x[2 * e + 1], unmul, mul));
            store_rows(smem + C::OFF_STAGE + warp * 4096, lane, y, out + row_w * dst.n + c0 * 128, dst.n, a.Nk - row_w);
          }
        } else {
#pragma unroll
          for (int c0 = 0; c0 < D / 32; ++c0) {
            uint32_t x[32];
            tmem_ld32(col + c0 * 32, x);
            if (j < a.Nk) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t y[4];
#pragma unroll
                for (int f = 0; f < 4; ++f)
                  y[f] = pack2<BF16>(scaled<BF16>(x[8 * e + 2 * f], unmul, mul), scaled<BF16>(x[8 * e + 2 * f + 1], unmul, mul));
                *reinterpret_cast<uint4*>(out + j * dst.n + c0 * 64 + e * 16) = make_uint4(y[0], y[1], y[2], y[3]);
              }
            }
          }
        }
        tc_fence_before_sync();  // dK, dV are read before this thread's next P^T, dS^T let them be overwritten
      } else if (w.n_runs > 1) {  // nothing sees these keys
        for (int e = 0; e < D / 4; ++e) partial[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      } else if (j < a.Nk) {
        for (int e = 0; e < D / 8; ++e) *reinterpret_cast<uint4*>(out + j * dst.n + e * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      i = items.after(k, ok);
      items.read_by_warp(k, lane, ok);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == C::W_MMA) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------- partial tiles
// dK and dV of the tiles in runs, eight channels a thread: the cut tiles, then those
// with sinks.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) attn_window_sum_kernel(const WindowArgs a, const WbPlan p) {
  griddep_wait();  // (launch_serialized)
  griddep_launch_dependents();
  constexpr int G = D / 8;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256, from = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int heads = a.B * a.Hk;
  const int64_t w_tiles = p.runs > 1 ? p.cut : 0, s_tiles = p.sink_runs > 1 ? static_cast<int64_t>(heads) * p.sink_tiles : 0;
  for (int64_t t = from; t < (s_tiles + w_tiles) * 2 * 128 * G; t += step) {
    const int c = static_cast<int>(t % G), r = static_cast<int>(t / G % 128), out = static_cast<int>(t / (G * 128) % 2);
    int64_t tile = t / (G * 256), slot;
    int n, jt, hb;
    if (tile < w_tiles) {
      n = p.runs, slot = tile * n;
      grouped_rank_order(p.whole + static_cast<int>(tile), p.tiles - p.sink_tiles, heads, p.group, jt, hb);
      jt += p.sink_tiles;
    } else {
      tile -= w_tiles;
      n = p.sink_runs, slot = w_tiles * p.runs + tile * n;
      hb = static_cast<int>(tile / p.sink_tiles), jt = static_cast<int>(tile - static_cast<int64_t>(hb) * p.sink_tiles);
    }
    const int j = jt * 128 + r;
    if (j >= a.Nk) continue;
    float x[8] = {};
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const float4* f = reinterpret_cast<const float4*>(p.part + (((slot + k) * 2 + out) * 128 + r) * D + c * 8);
      const float4 u = f[0], w = f[1];
      x[0] += u.x, x[1] += u.y, x[2] += u.z, x[3] += u.w, x[4] += w.x, x[5] += w.y, x[6] += w.z, x[7] += w.w;
    }
    const Bhnd& d = out ? a.dv : a.dk;
    *reinterpret_cast<uint4*>(d.p + hb / a.Hk * d.b + hb % a.Hk * d.h + j * d.n + c * 16) =
        make_uint4(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]), pack2<BF16>(x[4], x[5]), pack2<BF16>(x[6], x[7]));
  }
}

// Which tiles are cut, and into how many runs.  One CTA to an SM and tiles of about
// equal length: the last round of whole tiles, which would leave SMs without one, goes
// out in runs instead, and the tiles with sinks, longer by the ratio of sequence to
// window, come last in runs about as long.  A run costs its partial tiles and as much
// time as two visits, and with the first of them the sum kernel costs as much as four:
// below a gain of kCutGain visits tiles stay whole.
constexpr int kCutGain = 8;

void plan_runs(const WindowArgs& a, WbPlan* p) {
  const int64_t sms = 152;  // of the GPU this is for; with others the plan is as good as right
  const int64_t G = a.Hq / a.Hk, heads = static_cast<int64_t>(a.B) * a.Hk, ntq = (a.Nq + 127) / 128;
  // Query tiles that see a tile of keys: window + 127 rows, the first of them row
  // -(Nk - Nq) modulo 128 of its tile.
  const int64_t in_tile = (128 - (a.Nk - a.Nq) % 128) % 128;
  const int64_t near = std::min<int64_t>(ntq, (in_tile + a.window + 126) / 128 + 1);
  const int64_t vs = G * ntq, vw = G * near;  // visits of a tile, at most
  p->tiles = (a.Nk + 127) / 128;
  p->sink_tiles = std::min(p->tiles, (a.sinks + 127) / 128);
  const int64_t w_tiles = heads * (p->tiles - p->sink_tiles), s_tiles = heads * p->sink_tiles;
  int64_t cut = w_tiles % sms, runs = 1;
  if (cut) runs = std::min({sms / cut, (vw + 1) / 2, int64_t{16}});
  if (vw - (vw + runs - 1) / runs < kCutGain || w_tiles >= int64_t{16} * sms) cut = 0, runs = 1;
  p->whole = static_cast<int>(w_tiles - cut);
  p->cut = static_cast<int>(cut);
  p->runs = static_cast<int>(runs);
  // (no more than about 8 runs of sinks to an SM)
  const int64_t len = std::max({(vw + 2) / 3, s_tiles * vs / (8 * sms), int64_t{kCutGain} / 2});
  p->sink_runs = p->sink_tiles && vs - vw >= kCutGain ? static_cast<int>((vs + len - 1) / len) : 1;
}

// The plan but for its pointers; returns the number of partial tiles.
int64_t plan(const WindowArgs& a, WbPlan* p) {
  plan_runs(a, p);
  p->npad = (a.Nq + 127) / 128 * 128;
  // Blocks of the range kernel to a head: four rounds of loads each, about eight to an SM in all.
  const int64_t heads = static_cast<int64_t>(a.B) * a.Hk, rows = std::min<int64_t>(a.Nk, static_cast<int64_t>(a.Nq) + a.window), round = 4 * kRangeThreads * 8 / a.d;
  p->blocks = static_cast<int>(std::max<int64_t>(1, std::min({(rows + round - 1) / round, 8 * 152 / heads, int64_t{128}})));
  return (p->runs > 1 ? static_cast<int64_t>(p->cut) * p->runs : 0) +
         (p->sink_runs > 1 ? static_cast<int64_t>(a.B) * a.Hk * p->sink_tiles * p->sink_runs : 0);
}

template <int D, bool BF16>
int launch_t(const WindowArgs& a, int* launches) {
  using Q = DqCfg<D>;
  using K = DkvCfg<D>;
  CUtensorMap mq, mk, mv, mdo, mo;
  if (!encode_strided_map(&mq, a.q, a.B, a.Hq, a.Nq, D, Q::CH, BF16) || !encode_strided_map(&mk, a.k, a.B, a.Hk, a.Nk, D, Q::CH, BF16) ||
      !encode_strided_map(&mv, a.v, a.B, a.Hk, a.Nk, D, Q::CH, BF16) || !encode_strided_map(&mdo, a.dO, a.B, a.Hq, a.Nq, D, Q::CH, BF16) ||
      !encode_strided_map(&mo, a.o, a.B, a.Hq, a.Nq, D, Q::CH, BF16))
    return kStatusCuda;
  auto kq = attn_window_dq_kernel<D, BF16>;
  auto kk = attn_window_dkv_kernel<D, BF16>;
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kq), Q::SMEM) || !ensure_smem_attr(reinterpret_cast<const void*>(kk), K::SMEM))
    return kStatusCuda;
  if (!check_launch_regs(reinterpret_cast<const void*>(kq), Q::REGS) || !check_launch_regs(reinterpret_cast<const void*>(kk), K::REGS))
    return kStatusDeviceCheck;  // the splits' sums
  WbPlan p = {};
  const int64_t split = plan(a, &p);
  const int nrows = p.npad / 128;
  const int64_t heads = static_cast<int64_t>(a.B) * a.Hk, bh = static_cast<int64_t>(a.B) * a.Hq;
  const int64_t items = p.whole + static_cast<int64_t>(p.cut) * p.runs + heads * p.sink_tiles * p.sink_runs;
  if (items > 0x7fffffff || bh * nrows > 0x7fffffff) return kStatusUnsupported;
  p.group = order_head_group(static_cast<int>(heads), int64_t{4} * a.Nq * D * (a.Hq / a.Hk), int64_t{64} << 20);
  p.lse2 = reinterpret_cast<float*>(a.ws);
  p.dvec = p.lse2 + bh * p.npad;
  p.part = p.dvec + bh * p.npad;
  p.most = reinterpret_cast<float2*>(p.part + split * 2 * 128 * D);
  *launches = (split ? 3 : 2) + (BF16 ? 0 : 1);
  const int group = order_head_group(static_cast<int>(bh), int64_t{4} * a.Nk * D, int64_t{128} << 20);
  bool ok = BF16 || launch_serialized(true, attn_window_range_kernel<D>, dim3(static_cast<unsigned>(p.blocks), static_cast<unsigned>(heads)),
                                      dim3(kRangeThreads), 0, a.stream, a, p) == cudaSuccess;
  ok = ok && launch_serialized(true, kq, dim3(static_cast<unsigned>(bh * nrows)), dim3(Q::THREADS), Q::SMEM, a.stream, mq, mk, mv, mdo, mo, a, p,
                               nrows, group) == cudaSuccess;
  ok = ok && launch_serialized(true, kk, dim3(static_cast<unsigned>(items)), dim3(K::THREADS), K::SMEM, a.stream, mq, mk, mv, mdo, a, p) ==
                 cudaSuccess;
  if (split) {
    const int64_t tiles = (p.runs > 1 ? p.cut : 0) + (p.sink_runs > 1 ? heads * p.sink_tiles : 0);
    ok = ok && launch_serialized(true, attn_window_sum_kernel<D, BF16>, dim3(static_cast<unsigned>(std::min<int64_t>(tiles * D / 8, 16 * 152))),
                                 dim3(256), 0, a.stream, a, p) == cudaSuccess;
  }
  return ok && cudaGetLastError() == cudaSuccess ? kStatusOk : kStatusCuda;
}

template <int D>
int launch_d(const WindowArgs& a, int* launches) {
  return a.bf16 ? launch_t<D, true>(a, launches) : launch_t<D, false>(a, launches);
}

}  // namespace

int64_t window_bwd_workspace(const WindowArgs& a) {
  WbPlan p = {};
  const int64_t split = plan(a, &p);
  return 2 * static_cast<int64_t>(a.B) * a.Hq * p.npad * 4 + split * 2 * 128 * a.d * 4 + static_cast<int64_t>(a.B) * a.Hk * p.blocks * 8;
}

int launch_window_bwd(const WindowArgs& a, int* launches) {
  return a.d == 32 ? launch_d<32>(a, launches) : a.d == 64 ? launch_d<64>(a, launches) : launch_d<128>(a, launches);
}

}  // namespace attn
