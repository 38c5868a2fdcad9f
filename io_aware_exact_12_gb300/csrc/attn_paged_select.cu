// attn_paged_select.cu -- for each sequence and key/value head the pages whose
// keys can have the largest logit with the new token's queries.
//
//   score(p) = max over the head's queries g of
//              sum_c max(q_gc kmin_pc, q_gc kmax_pc)
//            = max_g (q_g^+ . kmax_p + q_g^- . kmin_p),
//
// the least upper bound of q_g . k over the box that the page's summary spans.
// The first and last pages of a sequence are always taken; the rest go by the
// score, equal ones by the lower index.  Two pages next to the border must not
// change places by an fp32 sum's rounding; but multiplying every summary in 64
// bits would cost many times what HBM needs to deliver it.  Hence two kernels:
//
//   attn_paged_score_kernel : every page's score as a matrix product of 2 d
//       channels with fp32 sums (m16n8k16, the queries as rows; e4m3 summaries
//       widened to fp16).  Reads 2 d elements per page and head once for up to 16
//       query heads to a key/value head (once per 16 beyond): HBM bound.
//   attn_paged_pick_kernel : one CTA per (sequence, KV head).  A score s errs by
//       at most eps = 2.125 d 2^-23 max_g |q_g|_1 max |k|, if each of the 2 d / 16
//       steps cuts 17 aligned terms at 2^-23 of the largest or less (a model of the
//       matrix unit that the tests bear out; nothing documents it).  A histogram
//       brackets the border to [L, H) with H - L <= 4 eps; pages at H + 2 eps or
//       above are in, those below L - 2 eps out, and only those between (a few)
//       are scored again, to 53 bits or more.  With eps = inf (a sum that overflowed or is
//       NaN) that is all of them, in fp64.
//
// Measured (GB300; the copy's rate is 6.8 TB/s), both kernels: 8 sequences of 4096
// pages, 32 / 8 heads of 128, bf16, 134 MB of summaries: 36 us, scores 26 and pick
// 11; 4 of up to 8192 pages, 40 / 8 heads, e4m3, 55 MB: 27 us; one of 1001 pages:
// 10 us (GPU time in a replayed graph).  The pick runs on one SM per head and is bound
// by its own 7 to 11 us of barriers and cold instructions.
#include <atomic>
#include <cmath>

#include "attn_paged.h"
#include "tc_sm103.cuh"

namespace attn {
namespace {

constexpr int kScoreWarps = 2;
constexpr int kScoreThreads = 32 * kScoreWarps;
constexpr int kScoreDepth = 4;                  // groups of 8 pages in flight per warp
constexpr int kScoreStep = 8 * kScoreWarps;     // pages of a CTA's turn
constexpr int kScoreChunk = 4 * kScoreStep;     // pages of a CTA, at least
constexpr int kPickBins = 1024;  // of the histogram
constexpr int kPickCap = 1024;  // candidates kept in shared memory
constexpr int kPickHeld = 4;    // scores that a thread keeps in registers (1, 2, 4, 8 of them: 22.2, 22.5,
                                // 22.5, 23.5 us for one of 16001; 42.6, 42.5, 41.7, 41.7 for 4 of 131072)

struct SelectScratch {  // per (sequence, head)
  float* score;         // [max_pages]
  float* eps;           // [chunks] error of a score CTA's scores
  uint64_t* key;        // [max_pages] exact scores, used beyond kPickCap candidates
};

__host__ __device__ inline int64_t up16(int64_t x) { return (x + 15) & ~int64_t{15}; }

__host__ __device__ inline int score_chunks(int max_pages) { return (max_pages + kScoreChunk - 1) / kScoreChunk; }
__host__ __device__ inline int64_t select_scratch_bytes(int max_pages) {
  return up16(int64_t{4} * max_pages) + up16(int64_t{4} * score_chunks(max_pages)) + int64_t{8} * max_pages + (max_pages & 1) * 8;
}
__device__ __forceinline__ SelectScratch scratch_of(uint8_t* ws, int64_t bh, int max_pages) {
  uint8_t* p = ws + bh * select_scratch_bytes(max_pages);
  SelectScratch s;
  s.score = reinterpret_cast<float*>(p);
  s.eps = reinterpret_cast<float*>(p + up16(int64_t{4} * max_pages));
  s.key = reinterpret_cast<uint64_t*>(p + up16(int64_t{4} * max_pages) + up16(int64_t{4} * score_chunks(max_pages)));
  return s;
}

// ------------------------------------------------------------------- scores

// Sign mask of two 16-bit floats: all ones in the halves that are negative.
__device__ __forceinline__ uint32_t negative_halves(uint32_t x) { return ((x >> 15) & 0x00010001u) * 0xffffu; }

// The larger magnitudes of two pairs, with some sign; a NaN gives way.
template <bool BF16>
__device__ __forceinline__ uint32_t max_magnitude(uint32_t m, uint32_t x) {
  uint32_t r;
  if constexpr (BF16) asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(x));
  else asm("max.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(x));
  return r;
}
template <bool BF16>
__device__ __forceinline__ float magnitude(uint32_t m) {
  const float2 f = unpack2<BF16>(m);
  return fmaxf(fabsf(f.x), fabsf(f.y));
}

// Copies the first `size` bytes and fills the rest with zeros.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, uint32_t size) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}
// The larger one, or NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// A warp scores 8 pages at a time.  The sum over channels may run in any order,
// so a thread takes whole 16-byte pieces of its page's summaries and the queries
// are laid out to match: piece v of thread t4 holds bytes (4 v + t4) VB and on.
// The pieces of the next groups travel as asynchronous copies into slots of
// shared memory that only their thread reads.
template <int X, int C, int D, bool WIDE>  // WIDE: more than 8 query heads
__global__ void __launch_bounds__(kScoreThreads) attn_paged_score_kernel(const PagedSelectArgs a, int chunk) {
  griddep_wait();  // launched overlapped (launch_serialized)
  griddep_launch_dependents();
  constexpr bool E8 = C == kTypeE4m3;
  constexpr bool BF = C == kTypeBf16;
  constexpr int ROW = D * (E8 ? 1 : 2);
  constexpr int VB = ROW / 4 < 16 ? ROW / 4 : 16;  // bytes of a piece
  constexpr int NV = ROW / (4 * VB);
  constexpr int WPV = VB / 4;                      // words of a piece
  constexpr int NS = D / 16;                       // steps of 16 channels
  constexpr int SLOT = 2 * NV * kScoreThreads * 16;
  __shared__ __align__(16) uint8_t ring[kScoreDepth * SLOT];
  const PagedKv& kv = a.kv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  // Heads in turn, so that a page's summaries, side by side in memory, are read
  // at about the same time.
  const int b = blockIdx.y, h = blockIdx.x % kv.H, part = blockIdx.x / kv.H, G = a.Hq / kv.H;
  const int used = (checked_len(kv, b) + kv.page - 1) / kv.page;
  const int p0 = part * chunk + warp * 8;           // the warp's first page
  const int p1 = min(used, (part + 1) * chunk);
  if (used <= a.n_select || part * chunk >= used) return;
  const SelectScratch sc = scratch_of(a.ws, static_cast<int64_t>(b) * kv.H + h, kv.max_pages);
  const int groups = p1 > p0 ? (p1 - p0 + 8 * kScoreWarps - 1) / (8 * kScoreWarps) : 0;
  const uint32_t slots = smem_addr(ring) + threadIdx.x * 16;

  // Page numbers of four groups in one load: lane (g, t4) has page g of group i + t4.
  static_assert(kScoreDepth == 4, "a batch of page numbers is as long as the ring");
  auto look_up = [&](int i) {
    const int j = p0 + (i + t4) * 8 * kScoreWarps + g;
    return j < p1 ? checked_page(kv, b, j) : -1;
  };
  const int64_t page_bytes = static_cast<int64_t>(kv.H) * ROW;
  const uint8_t *kmin = kv.kmin + h * ROW + t4 * VB, *kmax = kv.kmax + h * ROW + t4 * VB;
  uint32_t big = 0;
  float qmost = 0.f;  // largest |q|_1
  for (int r0 = 0; r0 < G; r0 += WIDE ? 16 : 8) {
    int ids = look_up(0), more = look_up(4);
    uint32_t found = 0;  // bit i % 32: the page of group i exists
    auto fetch = [&](int i) {
      const int id = __shfl_sync(0xffffffffu, ids, (lane & ~3) | (i & 3));
      const int64_t at = static_cast<int64_t>(max(id, 0)) * page_bytes;
      const uint32_t to = slots + (i % kScoreDepth) * SLOT, size = id >= 0 ? VB : 0;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        copy_async<VB>(to + v * (kScoreThreads * 16), kmin + at + v * 4 * VB, size);
        copy_async<VB>(to + (NV + v) * (kScoreThreads * 16), kmax + at + v * 4 * VB, size);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      found = (found & ~(1u << (i & 31))) | ((id >= 0 ? 1u : 0u) << (i & 31));
      if ((i & 3) == 3) {
        ids = more;
        more = look_up(i + 5);
      }
    };
#pragma unroll 1
    for (int i = 0; i < kScoreDepth; ++i) fetch(i);
    // q^+ and q^- of rows g and g + 8 as A fragments.
    uint32_t qp[NS][WIDE ? 4 : 2], qn[NS][WIDE ? 4 : 2];
    float mul[2] = {1.f, 1.f};
    constexpr int NR = WIDE ? 2 : 1;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const bool live = r0 + g + 8 * r < G;
      const uint8_t* q = a.q.p + b * a.q.row + (static_cast<int64_t>(h) * G + r0 + g + 8 * r) * a.q.head;
      uint32_t w[NS][2];
      if constexpr (E8) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int i = 0; i < WPV; ++i) {
            const uint2 x = live ? *reinterpret_cast<const uint2*>(q + 2 * ((v * 4 + t4) * VB + i * 4)) : make_uint2(0u, 0u);
            w[v * WPV + i][0] = x.x, w[v * WPV + i][1] = x.y;
          }
        if constexpr (X == kTypeBf16) {  // into fp16's range by a power of two
          float m = 0.f;
#pragma unroll
          for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float2 f = unpack2<true>(w[s][i]);
              m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          const int e = max(20, static_cast<int>(__float_as_uint(m) >> 23));
          const float fac = e == 255 ? 1.f : __uint_as_float(static_cast<uint32_t>(262 - e) << 23);
          mul[r] = e == 255 ? 1.f : __uint_as_float(static_cast<uint32_t>(e - 8) << 23);
#pragma unroll
          for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float2 f = unpack2<true>(w[s][i]);
              w[s][i] = pack2<false>(f.x * fac, f.y * fac);
            }
        }
      } else {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int i = 0; i < WPV; ++i)
            w[(v * WPV + i) / 2][(v * WPV + i) % 2] =
                live ? *reinterpret_cast<const uint32_t*>(q + (v * 4 + t4) * VB + i * 4) : 0u;
      }
      float sum = 0.f;
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 f = unpack2<BF>(w[s][i]);
          sum += fabsf(f.x) + fabsf(f.y);
          const uint32_t neg = negative_halves(w[s][i]);
          qp[s][i * NR + r] = w[s][i] & ~neg;
          qn[s][i * NR + r] = w[s][i] & neg;
        }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      sum *= mul[r];
      qmost = sum <= qmost ? qmost : sum;  // a NaN stays
    }
#pragma unroll 1
    for (int i = 0; i < groups; ++i) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kScoreDepth - 1) : "memory");
      const bool there = (found >> (i & 31)) & 1;
      uint32_t lo[NV * WPV], hi[NV * WPV];
      const uint32_t at = slots + (i % kScoreDepth) * SLOT;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if constexpr (VB == 16) {
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(lo[4 * v]), "=r"(lo[4 * v + 1]), "=r"(lo[4 * v + 2]),
                       "=r"(lo[4 * v + 3]) : "r"(at + v * (kScoreThreads * 16)) : "memory");
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(hi[4 * v]), "=r"(hi[4 * v + 1]), "=r"(hi[4 * v + 2]),
                       "=r"(hi[4 * v + 3]) : "r"(at + (NV + v) * (kScoreThreads * 16)) : "memory");
        } else {
          asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(lo[2 * v]), "=r"(lo[2 * v + 1])
                       : "r"(at + v * (kScoreThreads * 16)) : "memory");
          asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(hi[2 * v]), "=r"(hi[2 * v + 1])
                       : "r"(at + (NV + v) * (kScoreThreads * 16)) : "memory");
        }
      }
      __syncwarp();  // look-ups part the lanes, the matrix steps want them together
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        uint32_t l0, l1, h0, h1;
        if constexpr (E8) {
          l0 = e4m3_pair(lo[s]), l1 = e4m3_pair_hi(lo[s]), h0 = e4m3_pair(hi[s]), h1 = e4m3_pair_hi(hi[s]);
        } else {
          l0 = lo[2 * s], l1 = lo[2 * s + 1], h0 = hi[2 * s], h1 = hi[2 * s + 1];
        }
        big = max_magnitude<BF>(max_magnitude<BF>(max_magnitude<BF>(max_magnitude<BF>(big, l0), l1), h0), h1);
        if constexpr (WIDE) {
          mma16<BF>(acc, qp[s][0], qp[s][1], qp[s][2], qp[s][3], h0, h1);
          mma16<BF>(acc, qn[s][0], qn[s][1], qn[s][2], qn[s][3], l0, l1);
        } else {
          mma16<BF>(acc, qp[s][0], 0u, qp[s][1], 0u, h0, h1);
          mma16<BF>(acc, qn[s][0], 0u, qn[s][1], 0u, l0, l1);
        }
      }
      const uint32_t have = __ballot_sync(0xffffffffu, there);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float best = -INFINITY;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          float s = acc[2 * r + x];
          if constexpr (E8 && X == kTypeBf16) s *= mul[r];
          if (r0 + g + 8 * r < G) best = max_nan(best, s);
        }
#pragma unroll
        for (int y = 4; y < 32; y <<= 1) best = max_nan(best, __shfl_xor_sync(0xffffffffu, best, y));
        const int j = p0 + i * 8 * kScoreWarps + 2 * t4 + x;
        if (g == 0 && j < p1) {
          if (!(fabsf(best) <= 3.402823466e38f)) best = INFINITY;                // NaN too: the pick scores all anew
          if (!((have >> ((2 * t4 + x) * 4)) & 1)) best = -3.402823466e38f;     // no page there: last
          sc.score[j] = r0 ? fmaxf(sc.score[j], best) : best;
        }
      }
      fetch(i + kScoreDepth);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  float m = magnitude<BF>(big);
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  const bool odd = __any_sync(0xffffffffu, isnan(qmost));
#pragma unroll
  for (int x = 4; x < 32; x <<= 1) qmost = fmaxf(qmost, __shfl_xor_sync(0xffffffffu, qmost, x));
  __shared__ float sm[kScoreWarps];
  if (lane == 0) sm[warp] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    const float eps = D * 2.6e-7f * qmost * fmaxf(sm[0], sm[1]);  // 2.125 d 2^-23, and the rounding of sum and product
    sc.eps[part] = odd || !(eps <= 1e37f) ? INFINITY : eps;
  }
}

// --------------------------------------------------------------------- pick

// Order-preserving maps of scores to unsigned keys; NaN ranks first.
__device__ __forceinline__ uint64_t key64(double x) {
  if (isnan(x)) return ~0ull;
  x = x == 0.0 ? 0.0 : x;  // -0 equals +0
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x));
  return (u >> 63) ? ~u : u | (1ull << 63);
}
__device__ __forceinline__ uint32_t key32(float x) {
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_key32(uint32_t k) { return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k); }

// N consecutive elements as fp32, 4 to 32 bytes.
template <int TYPE, int N>
__device__ __forceinline__ void load_channels(const uint8_t* p, float (&f)[N]) {
  constexpr int W = N * (TYPE == kTypeE4m3 ? 1 : 2) / 4;  // words
  uint32_t w[W];
  if constexpr (W >= 4) {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p + 4 * i);
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
  } else if constexpr (W == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    float2 x;
    if constexpr (TYPE == kTypeE4m3) x = unpack2<false>((i & 1) ? e4m3_pair_hi(w[i / 2]) : e4m3_pair(w[i / 2]));
    else x = unpack2<TYPE == kTypeBf16>(w[i]);
    f[2 * i] = x.x, f[2 * i + 1] = x.y;
  }
}

struct PickShared {
  int count[2][32];
  float f[3][32];
  int hist[kPickBins];
  int list[kPickCap];
  uint64_t key[kPickCap];
  int m, bin;
};

// Sum over the block, for every thread; `turn` alternates so that one barrier
// per sum is enough.
template <int T>
__device__ __forceinline__ int block_sum(int v, PickShared& sm, int turn) {
  const int lane = threadIdx.x & 31;
  v = __reduce_add_sync(0xffffffffu, v);
  if (lane == 0) sm.count[turn][threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, lane < T / 32 ? sm.count[turn][lane] : 0);
}

// A sum in three fp32 words: the running sum, the sum of what its additions round off
// (exact, by Knuth's error-free sum) and the sum of what those round off.  Only the last
// one's own roundings are lost, 2^-59 of the terms' magnitude for d = 128.  The fp64 units
// have a sixtieth of the fp32 rate: some tens of candidates took 20 us there.
struct Sum3 {
  float hi, mid, lo;
};
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Sum3 add(const Sum3& s, float x) {
  const Two h = two_sum(s.hi, x), m = two_sum(s.mid, h.lo);
  return {h.hi, m.hi, __fadd_rn(s.lo, m.lo)};
}
__device__ __forceinline__ Sum3 add(const Sum3& a, const Sum3& b) {  // the same for (b, a)
  const Two h = two_sum(a.hi, b.hi), m = two_sum(a.mid, b.mid), n = two_sum(m.hi, h.lo);
  return {h.hi, n.hi, __fadd_rn(__fadd_rn(a.lo, b.lo), __fadd_rn(m.lo, n.lo))};
}
// Order-preserving key of a finite sum: the leading word's, 2^32 to a step of it, and the
// rest in such units: 56 bits.
__device__ __forceinline__ uint64_t key_of(const Sum3& s) {
  const Two v = two_sum(s.mid, s.lo), w = two_sum(s.hi, v.hi), x = two_sum(w.lo, v.lo);
  const float top = __fadd_rn(w.hi, x.hi), low = __fsub_rn(x.hi, __fsub_rn(top, w.hi));  // exact: w.hi is 0 or the larger
  const int e = max(static_cast<int>((__float_as_uint(top) >> 23) & 255u), 60);  // below 2^-67 the rest counts for less
  const float unit = __uint_as_float(static_cast<uint32_t>(309 - e) << 23);      // 2^32 steps of `top`
  const long long rest = static_cast<long long>(__float2int_rn(low * unit)) + __float2int_rn(x.lo * unit);
  return (static_cast<uint64_t>(key32(top)) << 32) + static_cast<uint64_t>(rest);
}

// The definition, by one warp; every lane gets it.  Eight lanes take a head,
// four heads at a time.  Products of two 16-bit floats are exact in fp32
// (WORDS: none of them near the ends of its range).
template <int X, int C, int D, bool WORDS>
__device__ __forceinline__ uint64_t exact_key(const PagedSelectArgs& a, int b, int h, int G, int j) {
  constexpr int CB = C == kTypeE4m3 ? 1 : 2;
  const int lane = threadIdx.x & 31, c0 = (lane & 7) * (D / 8);
  const int id = checked_page(a.kv, b, j);
  if (id < 0) return 0;
  const int64_t at = ((static_cast<int64_t>(id) * a.kv.H + h) * D + c0) * CB;
  float lo[D / 8], hi[D / 8];
  load_channels<C>(a.kv.kmin + at, lo);
  load_channels<C>(a.kv.kmax + at, hi);
  double best = -INFINITY;
  uint64_t top = 0;
  for (int g0 = 0; g0 < G; g0 += 4) {
    const int g = min(g0 + (lane >> 3), G - 1);  // the last head again where there is none
    const uint8_t* q = a.q.p + b * a.q.row + (static_cast<int64_t>(h) * G + g) * a.q.head;
    Sum3 s = {0.f, 0.f, 0.f};
    double d = 0.0;
    float qf[D / 8];
    load_channels<X>(q + c0 * 2, qf);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const float x = qf[i];
      if constexpr (WORDS) {
        s = add(s, __fmul_rn(x, x >= 0.f ? hi[i] : lo[i]));
      } else {
        // Both products, as the definition has it: where every key of a page was NaN, append
        // leaves kmin = inf and kmax = -inf, and 0 times an infinite one is NaN.
        const double u = static_cast<double>(x) * lo[i], v = static_cast<double>(x) * hi[i];
        d += isnan(u) || isnan(v) ? NAN : fmax(u, v);
      }
    }
#pragma unroll
    for (int x = 1; x < 8; x <<= 1) {
      if constexpr (WORDS)
        s = add(s, Sum3{__shfl_xor_sync(0xffffffffu, s.hi, x), __shfl_xor_sync(0xffffffffu, s.mid, x),
                        __shfl_xor_sync(0xffffffffu, s.lo, x)});
      else
        d += __shfl_xor_sync(0xffffffffu, d, x);
    }
    if constexpr (WORDS) {
      top = max(top, key_of(s));
    } else {
      best = isnan(d) || isnan(best) ? NAN : fmax(best, d);
    }
  }
#pragma unroll
  for (int x = 8; x < 32; x <<= 1) {
    if constexpr (WORDS) {
      top = max(top, static_cast<uint64_t>(__shfl_xor_sync(0xffffffffu, static_cast<unsigned long long>(top), x)));
    } else {
      const double d = __shfl_xor_sync(0xffffffffu, best, x);
      best = isnan(d) || isnan(best) ? NAN : fmax(best, d);
    }
  }
  if constexpr (WORDS) return top;
  return key64(best);
}

template <int X, int C, int D, int T>  // T threads
__global__ void __launch_bounds__(T) attn_paged_pick_kernel(const PagedSelectArgs a, int chunk) {
  griddep_wait();  // launched overlapped (launch_serialized)
  griddep_launch_dependents();
  __shared__ PickShared sm;
  const PagedKv& kv = a.kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / kv.H, h = blockIdx.x % kv.H, G = a.Hq / kv.H;
  // The first scores of each thread, before it is known how many there are; the
  // scratch behind them is there, and what it holds is not looked at.
  const SelectScratch sc = scratch_of(a.ws, blockIdx.x, kv.max_pages);
  float* score = sc.score;
  float held[kPickHeld];
#pragma unroll
  for (int i = 0; i < kPickHeld; ++i) {
    const int j = i * T + tid;
    held[i] = j < kv.max_pages ? score[j] : 0.f;
  }
  const int used = (checked_len(kv, b) + kv.page - 1) / kv.page;
  int* out = a.pages + static_cast<int64_t>(blockIdx.x) * a.n_select;
  if (used <= a.n_select) {
    for (int i = tid; i < a.n_select; i += T) out[i] = i < used ? i : -1;
    return;
  }
  const int first = a.keep_first, end = used - a.keep_last;  // the pages that go by their score
  const int want = a.n_select - a.keep_first - a.keep_last;
  // All scored pages of this thread, as they came.
  auto each = [&](auto&& body) {
#pragma unroll
    for (int i = 0; i < kPickHeld; ++i) {
      const int j = i * T + tid;
      if (j >= first && j < end) body(j, held[i]);
    }
    for (int j = kPickHeld * T + tid; j < end; j += T)
      if (j >= first) body(j, score[j]);
  };
  int turn = 0;
  float sure = INFINITY;  // pages with this score or more are in
  if (want > 0) {
    // Range of the scores and their error.  Pages that the table does not have
    // count for nothing here: they are out, or the last resort.
    constexpr float kNone = -3.402823466e38f;
    float least = INFINITY, most = -INFINITY, eps = 0.f;
    int none = 0;
    each([&](int, float s) {
      none += s <= kNone;
      least = fminf(least, s <= kNone ? INFINITY : s), most = fmaxf(most, s);
    });
    for (int i = tid; i < (used + chunk - 1) / chunk; i += T) eps = fmaxf(eps, sc.eps[i]);
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      least = fminf(least, __shfl_xor_sync(0xffffffffu, least, x));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, x));
      eps = fmaxf(eps, __shfl_xor_sync(0xffffffffu, eps, x));
    }
    if (lane == 0) sm.f[0][warp] = least, sm.f[1][warp] = most, sm.f[2][warp] = eps;
    if (tid == 0) sm.m = 0;
    for (int i = tid; i < kPickBins; i += T) sm.hist[i] = 0;
    none = block_sum<T>(none, sm, turn);
    const int from_warp = min(lane, T / 32 - 1);
    least = sm.f[0][from_warp], most = sm.f[1][from_warp], eps = sm.f[2][from_warp];
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      least = fminf(least, __shfl_xor_sync(0xffffffffu, least, x));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, x));
      eps = fmaxf(eps, __shfl_xor_sync(0xffffffffu, eps, x));
    }
    if (!(most - least <= 1e37f) || end - first - none < want) eps = INFINITY;
    // Sums in fp32 words where no product overflows (the terms' magnitude is at most
    // eps / (d 2.6e-7)), nor the last bits vanish below fp32's range.
    const bool words = eps < 1e32f && eps > 1e-24f;
    float from = -INFINITY;  // candidates: from <= score < sure
    if (eps < INFINITY) {
      // The border lies in [lo, hi]: less than `want` scores are above, at least
      // `want` reach lo.  A turn cuts that to a bin of 1024 and a rounding.
      float lo = least, hi = most;
      for (int n = 0; n < 64; ++n) {
        const float width = hi - lo, scale = kPickBins / width;
        if (width <= 4.f * eps || !(scale <= 1e37f)) break;
        int above = 0;
        each([&](int, float s) {
          above += s > hi;
          if (s >= lo && s <= hi) atomicAdd(&sm.hist[min(kPickBins - 1, static_cast<int>((s - lo) * scale))], 1);
        });
        turn ^= 1;
        above = block_sum<T>(above, sm, turn);  // its barrier completes the histogram
        constexpr int kEach = kPickBins / T;
        int bins[kEach], mine = 0;  // thread 0 has the highest ones
#pragma unroll
        for (int i = 0; i < kEach; ++i) mine += bins[i] = sm.hist[kPickBins - 1 - tid * kEach - i];
        int upto = mine;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, upto, x);
          if (lane >= x) upto += y;
        }
        turn ^= 1;
        if (lane == 31) sm.count[turn][warp] = upto;
        __syncthreads();
        upto += above + __reduce_add_sync(0xffffffffu, lane < warp ? sm.count[turn][lane] : 0);
        int upper = upto - mine;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const int bin = kPickBins - 1 - tid * kEach - i;
          if (upper < want && want <= upper + bins[i]) sm.bin = bin;
          upper += bins[i];
          sm.hist[bin] = 0;  // for the next turn
        }
        __syncthreads();
        const float l = lo + sm.bin * (width / kPickBins), h = lo + (sm.bin + 1) * (width / kPickBins);
        const float slack = 4e-7f * (fabsf(lo) + fabsf(hi));  // of these sums and of the bins' rounding
        const float nl = fmaxf(lo, l - slack), nh = fminf(hi, h + slack);
        if (nh - nl > 0.5f * width) break;  // as narrow as fp32 can tell
        lo = nl, hi = nh;
      }
      from = lo - 2.f * eps;
      sure = hi + 2.f * eps;
      // Rounding of the two sums; and more than hi, whatever eps.
      from -= fabsf(from) * 1e-6f;
      sure += fabsf(sure) * 1e-6f + 2e-38f;
    }
    // Pages that are in, and candidates.
    int in_all = 0;
    each([&](int j, float s) {
      const bool in = eps < INFINITY && s >= sure;
      in_all += in;
      if (!in && s >= from) {
        const int at = atomicAdd(&sm.m, 1);
        if (at < kPickCap) sm.list[at] = j;
      }
    });
    turn ^= 1;
    const int r = want - block_sum<T>(in_all, sm, turn), m = sm.m;  // r of the m candidates are in
    const bool few = m <= kPickCap;
    if (m > r) {
      if (few) {
        for (int i = warp; i < m; i += T / 32) {
          const int j = sm.list[i];
          const uint64_t k = words ? exact_key<X, C, D, true>(a, b, h, G, j) : exact_key<X, C, D, false>(a, b, h, G, j);
          if (lane == 0) sm.key[i] = k;
        }
        __syncthreads();
        for (int i = warp; i < m; i += T / 32) {
          const uint64_t k = sm.key[i];
          const int j = sm.list[i];
          int ahead = 0;
          for (int y0 = 0; y0 < m; y0 += 32) {
            const int y = y0 + lane;
            ahead += __popc(__ballot_sync(0xffffffffu, y < m && (sm.key[y] > k || (sm.key[y] == k && sm.list[y] < j))));
          }
          if (lane == 0) score[j] = ahead < r ? INFINITY : -INFINITY;
        }
      } else {
        for (int j = first + warp; j < end; j += T / 32) {
          const float s = score[j];
          if (s >= from && !(eps < INFINITY && s >= sure)) {
            const uint64_t k = words ? exact_key<X, C, D, true>(a, b, h, G, j) : exact_key<X, C, D, false>(a, b, h, G, j);
            if (lane == 0) sc.key[j] = k;
          }
        }
        __syncthreads();
        // The r-th largest key bit by bit, then equal keys by the r-th lowest page.
        auto cand = [&](int j) {
          const float s = score[j];
          return s >= from && !(eps < INFINITY && s >= sure);
        };
        uint64_t border = 0;
        for (int bit = 63; bit >= 0; --bit) {
          turn ^= 1;
          const uint64_t t = border | (1ull << bit);
          int c = 0;
          for (int j = first + tid; j < end; j += T) c += cand(j) && sc.key[j] >= t;
          if (block_sum<T>(c, sm, turn) >= r) border = t;
        }
        turn ^= 1;
        int c = 0;
        for (int j = first + tid; j < end; j += T) c += cand(j) && sc.key[j] > border;
        const int equal = r - block_sum<T>(c, sm, turn);
        int lo = first, hi = end;  // least j with `equal` pages at the border below it
        while (lo < hi) {
          turn ^= 1;
          const int mid = lo + (hi - lo) / 2;
          int e = 0;
          for (int j = first + tid; j < mid; j += T) e += cand(j) && sc.key[j] == border;
          if (block_sum<T>(e, sm, turn) >= equal) hi = mid;
          else lo = mid + 1;
        }
        for (int j = first + tid; j < end; j += T)
          if (cand(j)) score[j] = sc.key[j] > border || (sc.key[j] == border && j < lo) ? INFINITY : -INFINITY;
      }
    } else {
      for (int j = first + tid; j < end; j += T) {
        const float s = score[j];
        if (s >= from) score[j] = INFINITY;
      }
    }
    __syncthreads();
  }
  // Ascending output: a run of pages per warp, places by a scan over the warps.
  const int per = (used + T - 1) / T * 32;
  const int j0 = min(used, warp * per), j1 = min(used, j0 + per);
  auto taken = [&](int j) { return j < j1 && (j < first || j >= end || (want > 0 && score[j] >= sure)); };
  int mine = 0;
#pragma unroll 4
  for (int j = j0; j < j1; j += 32) mine += taken(j + lane);
  mine = __reduce_add_sync(0xffffffffu, mine);
  turn ^= 1;
  if (lane == 0) sm.count[turn][warp] = mine;
  __syncthreads();
  int at = __reduce_add_sync(0xffffffffu, lane < warp ? sm.count[turn][lane] : 0);
#pragma unroll 4
  for (int j = j0; j < j1; j += 32) {
    const uint32_t who = __ballot_sync(0xffffffffu, taken(j + lane));
    if ((who >> lane) & 1) out[at + __popc(who & ((1u << lane) - 1))] = j + lane;
    at += __popc(who);
  }
}

template <int X, int C, int D>
int launch_t(const PagedSelectArgs& a) {
  // A CTA takes 4 us to its first result and 0.6 us a turn from there, so the
  // walks are as long as it takes for all CTAs to be resident at once, and not
  // shorter than four turns (against runs of 128 pages: selection and decode of 8
  // sequences of 4096 pages 131 -> 129 us, 4 of 8192 in e4m3 46 -> 44).
  auto score = a.Hq / a.kv.H > 8 ? attn_paged_score_kernel<X, C, D, true> : attn_paged_score_kernel<X, C, D, false>;
  static std::atomic<int> per_sm[2];
  int fit = per_sm[a.Hq / a.kv.H > 8].load();
  if (fit < 1) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, score, kScoreThreads, 0) != cudaSuccess || fit < 1)
      return kStatusCuda;
    per_sm[a.Hq / a.kv.H > 8].store(fit);
  }
  const int64_t heads = static_cast<int64_t>(a.kv.B) * a.kv.H;
  const int64_t each = std::max<int64_t>(1, static_cast<int64_t>(fit) * std::max(1, device_sm_count()) / heads);  // CTAs of a head
  const int64_t steps = (a.kv.max_pages + kScoreStep - 1) / kScoreStep;
  const int chunk = static_cast<int>(std::max<int64_t>(kScoreChunk, (steps + each - 1) / each * kScoreStep));
  const dim3 grid((a.kv.max_pages + chunk - 1) / chunk * a.kv.H, a.kv.B);
  if (launch_serialized(true, score, grid, dim3(kScoreThreads), 0, a.stream, a, chunk) != cudaSuccess) return kStatusCuda;
  // Fewer warps cost less to bring together, more walk a long list faster (one
  // sequence of 188 pages 16.8 against 18.7 us, of 8192 45.2 against 41.8).
  auto pick = a.kv.max_pages <= 2048 ? attn_paged_pick_kernel<X, C, D, 512> : attn_paged_pick_kernel<X, C, D, 1024>;
  return launch_serialized(true, pick, dim3(a.kv.B * a.kv.H), dim3(a.kv.max_pages <= 2048 ? 512 : 1024), 0, a.stream, a,
                           chunk) == cudaSuccess
             ? kStatusOk
             : kStatusCuda;
}

template <int X, int C>
int launch_d(const PagedSelectArgs& a) {
  switch (a.kv.d) {
    case 32: return launch_t<X, C, 32>(a);
    case 64: return launch_t<X, C, 64>(a);
    default: return launch_t<X, C, 128>(a);
  }
}

}  // namespace

int64_t paged_select_workspace(int B, int H, int max_pages) {
  return static_cast<int64_t>(B) * H * select_scratch_bytes(max_pages);
}

int launch_paged_select(const PagedSelectArgs& a, int* launches) {
  *launches = 2;
  if (a.x_type == kTypeBf16)
    return a.kv.type == kTypeE4m3 ? launch_d<kTypeBf16, kTypeE4m3>(a) : launch_d<kTypeBf16, kTypeBf16>(a);
  return a.kv.type == kTypeE4m3 ? launch_d<kTypeF16, kTypeE4m3>(a) : launch_d<kTypeF16, kTypeF16>(a);
}

}  // namespace attn
