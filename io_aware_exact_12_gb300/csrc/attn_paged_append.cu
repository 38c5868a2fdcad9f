// attn_paged_append.cu -- new tokens' keys and values into a paged cache, with
// the position rotation (of the queries too) and the cast to the cache's type
// applied on the way, and the pages' key summaries kept up to date.
//
//   (x1, x2) -> (x1 cos - x2 sin, x2 cos + x1 sin), fp32, one rounding at the
//   store; summaries: channelwise min and max of the keys as stored, so a
//   summary is exact in the cache's type.
//
// Nothing is computed to speak of: 3 flops per rotated element against 4 bytes
// moved, so HBM bounds prompts and the launch bounds single tokens.  Work is
// cut into units: the tokens of one sequence inside one aligned span of
// positions (a page with summaries, else 8 to 32 tokens, which a page boundary
// never cuts).  A thread owns sixteen channels of one head (an item: the two
// 8-element chunks that the rotation couples) and walks the unit's tokens, so
// the minima and maxima stay in its registers and need no exchange.  Its next
// kAppendDepth tokens are in flight as asynchronous copies into a slot of
// shared memory that only it reads: no barrier, and no registers held while
// they travel.  (TMA would bring whole rows, but a thread wants two chunks that lie
// half a head apart, from strides that are the caller's.)
//
// Measured (GB300; the copy's rate is 6.8 TB/s): 16 ragged prompts, 26.6 k tokens,
// 32 / 8 heads of 128, bf16, with summaries, 652 MB: 101 us (6.5 TB/s); a document of
// 65537 tokens, 16 / 4 heads of 128, half of the channels rotated, e4m3, 755 MB:
// 120 us (6.3 TB/s); single tokens of 1 or 256 sequences: 2 to 3 us.
#include <cmath>

#include "attn_paged.h"
#include "tc_sm103.cuh"

namespace attn {
namespace {

constexpr int kAppendThreads = 128;
constexpr int kAppendSpan = 32;  // tokens of a unit without summaries, at most
constexpr int kAppendDepth = 4;  // tokens in flight per thread

__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 load_shared16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// Minima and maxima of pairs in the 16-bit type that holds the stored values
// exactly (fp16 for e4m3); a NaN gives way to the other operand.
template <int C>
__device__ __forceinline__ uint32_t min_pair(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (C == kTypeBf16) asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <int C>
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (C == kTypeBf16) asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Stored elements to pairs of that 16-bit type and back (exact).
template <int C>
__device__ __forceinline__ void load_pairs(const uint8_t* p, uint32_t (&w)[4]) {
  if constexpr (C == kTypeE4m3) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = e4m3_pair(v.x), w[1] = e4m3_pair_hi(v.x), w[2] = e4m3_pair(v.y), w[3] = e4m3_pair_hi(v.y);
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
}
template <int C>
__device__ __forceinline__ void store_pairs(uint8_t* p, const uint32_t (&w)[4]) {
  if constexpr (C == kTypeE4m3) {
    uint32_t v[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // Infinite where every key was NaN; e4m3 has no infinity, and 448 would pass for a key.
      float2 f = unpack2<false>(w[i]);
      if (isinf(f.x)) f.x = NAN;
      if (isinf(f.y)) f.y = NAN;
      v[i >> 1] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3)) << ((i & 1) * 16);
    }
    *reinterpret_cast<uint2*>(p) = make_uint2(v[0], v[1]);
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
// Rounds to the stored type (nearest even; e4m3 saturates at +-448 and keeps
// NaN) and stores; w becomes the stored values as pairs.
template <int C>
__device__ __forceinline__ void round_store(uint8_t* p, const float (&f)[8], uint32_t (&w)[4]) {
  if constexpr (C == kTypeE4m3) {
    uint32_t v[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i >> 1] |= static_cast<uint32_t>(
                       __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i], f[2 * i + 1]), __NV_SATFINITE, __NV_E4M3))
                   << ((i & 1) * 16);
    *reinterpret_cast<uint2*>(p) = make_uint2(v[0], v[1]);
    w[0] = e4m3_pair(v[0]), w[1] = e4m3_pair_hi(v[0]), w[2] = e4m3_pair(v[1]), w[3] = e4m3_pair_hi(v[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack2<C == kTypeBf16>(f[2 * i], f[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
template <int X>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack2<X == kTypeBf16>(w[i]);
    f[2 * i] = x.x, f[2 * i + 1] = x.y;
  }
}

// How x / scale is computed for the conversion to e4m3.
enum : int {
  kProduct,    // by 1 / scale, which is exact: normal powers of two
  kCorrected,  // the product and one correction by its exact remainder
  kDivision,   // scales for which remainders may leave fp32's normal range
};
int quotient_of(float scale) {
  int e = 0;
  if (scale >= 1.17549435e-38f && std::frexp(scale, &e) == 0.5f) return kProduct;
  return scale > 1e-25f && scale < 1e25f ? kCorrected : kDivision;
}

// The product alone errs by up to 3 units of the last place against the rounded quotient
// and so takes ties of e4m3 to the wrong neighbour.  Corrected (Markstein, IBM J. Res.
// Dev. 34, 1990) it is 2^-46 off before its last rounding; zeros and values that saturate
// stay as they are.  65537 tokens, 16 / 4 heads of 128: product 120 us, corrected 122,
// division 150.
template <int S>
__device__ __forceinline__ float quotient(float x, float unit, float inv) {
  if constexpr (S == kDivision) return __fdiv_rn(x, unit);
  const float q = x * inv;
  if constexpr (S == kProduct) return q;
  const float c = fmaf(fmaf(-q, unit, x), inv, q);
  return fabsf(q) < 1024.f && q != 0.f ? c : q;
}

template <int X, int C, int S>
__global__ void __launch_bounds__(kAppendThreads) attn_paged_append_kernel(const PagedAppendArgs a, int span) {
  griddep_wait();  // launched overlapped (launch_serialized)
  griddep_launch_dependents();
  const PagedKv& kv = a.kv;
  const int per_head = kv.d / 16;
  const int k_items = kv.H * per_head;
  const int item = blockIdx.y * kAppendThreads + threadIdx.x;

  // The unit: rows [r0, r0 + n) at positions [p0, p0 + n).
  int b, n, p0, r0;
  if (!a.token_start) {
    b = blockIdx.x;
    const int len = checked_len(kv, b);
    if (len == 0) return;
    n = 1, p0 = len - 1, r0 = b;
  } else {
    // Sequence b's units start at token_start[b] / span + 2 b: n tokens touch
    // at most n / span + 2 spans, so the ranges of two sequences are disjoint.
    const int u = blockIdx.x;
    int lo = 0, hi = kv.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.token_start[mid] / span + 2 * mid <= u) lo = mid;
      else hi = mid - 1;
    }
    b = lo;
    const int s = a.token_start[b], e = a.token_start[b + 1];
    const int len = checked_len(kv, b);
    if (e == s || len == 0) return;
    if (s < 0 || e < s || e > a.rows || len < e - s) {
      record_check(kv.check);
      return;
    }
    const int first = len - (e - s);
    const int j = u - (s / span + 2 * b);
    if (j < 0) return;
    const int64_t from = (static_cast<int64_t>(first / span) + j) * span;
    if (from >= len) return;
    p0 = max(first, static_cast<int>(from));
    n = min(len, static_cast<int>(min(from + span, static_cast<int64_t>(len)))) - p0;
    r0 = s + (p0 - first);
  }
  if (a.rot && p0 + n > a.table_rows) {
    record_check(kv.check);
    n = a.table_rows - p0;
    if (n <= 0) return;
  }
  const int id = checked_page(kv, b, p0 / kv.page);
  if (id < 0) return;
  const int slot0 = p0 % kv.page;

  // The item: K, V or Q, its head and its pair of chunks.
  int kind, h, i;
  if (item < k_items) kind = 0, h = item / per_head, i = item % per_head;
  else if (item < 2 * k_items) kind = 1, h = (item - k_items) / per_head, i = item % per_head;
  else if (item < 2 * k_items + a.Hq * per_head) kind = 2, h = (item - 2 * k_items) / per_head, i = item % per_head;
  else kind = 3, h = 0, i = 0;  // only helps its warp to fetch the angles
  const bool turn = (kind == 0 || kind == 2) && i < a.rot / 16;
  // First channels of the two chunks: halves of the rotated channels, or of the
  // others, apart, so that neighbouring threads' chunks are neighbours in memory.
  const int base = kind == 1 || turn ? 0 : a.rot, range = kind == 1 ? kv.d : turn ? a.rot : kv.d - a.rot;
  const int c0 = base + 8 * (i - base / 16), c1 = c0 + range / 2;

  const PagedRows& in = kind == 0 ? a.k : kind == 1 ? a.v : a.q;
  const uint8_t* src = in.p + r0 * in.row + h * in.head;
  uint8_t* dst;
  int64_t step;
  if (kind == 2) {
    dst = a.q_out.p + r0 * a.q_out.row + h * a.q_out.head;
    step = a.q_out.row;
  } else {
    step = kind ? kv.v_tok : kv.k_tok;
    dst = kind ? kv.v + id * kv.v_page + h * kv.v_head : kv.k + id * kv.k_page + h * kv.k_head;
    dst += slot0 * step;
  }
  constexpr int CB = C == kTypeE4m3 ? 1 : 2;
  const float unit = kind ? kv.v_scale : kv.k_scale, inv = 1.f / unit;

  // Slot of token t: two 16-byte pieces per thread, a warp's pieces side by
  // side, and the token's rows of cos and sin once per warp (its heads share them).
  constexpr int kWarps = kAppendThreads / 32, kTable = 512;  // bytes of two table rows at most
  __shared__ __align__(16) uint8_t ring[kAppendDepth * (2 * kAppendThreads * 16 + kWarps * kTable)];
  const int lane = threadIdx.x & 31;
  const uint32_t slots = smem_addr(ring) + threadIdx.x * 16;
  const uint32_t tables = smem_addr(ring) + kAppendDepth * 2 * kAppendThreads * 16 + (threadIdx.x >> 5) * kTable;
  const int half = a.rot / 2;
  // Lane l < rot / 4 fetches 16 bytes of a token's angles, cos before sin.
  const float* angle = lane < half / 4 ? a.cos + lane * 4 : a.sin + (lane * 4 - half);
  angle += static_cast<int64_t>(p0) * half;
  auto fetch = [&](int t) {
    if (t < n) {
      const uint32_t at = slots + (t % kAppendDepth) * (2 * kAppendThreads * 16);
      if (kind < 3) {
        copy16_async(at, src + t * in.row + c0 * 2);
        copy16_async(at + kAppendThreads * 16, src + t * in.row + c1 * 2);
      }
      if (lane < a.rot / 4)
        copy16_async(tables + (t % kAppendDepth) * (kWarps * kTable) + lane * 16, angle + static_cast<int64_t>(t) * half);
    }
    copies_commit();
  };
#pragma unroll
  for (int t = 0; t < kAppendDepth; ++t) fetch(t);
  const bool track = kind == 0 && kv.kmin != nullptr;
  const bool plain = !turn && !track && (kind == 2 || C == X);
  constexpr uint32_t kInf = C == kTypeBf16 ? 0x7f807f80u : 0x7c007c00u;
  uint32_t lo[2][4], hi[2][4];
#pragma unroll
  for (int e = 0; e < 4; ++e) lo[0][e] = lo[1][e] = kInf, hi[0][e] = hi[1][e] = kInf | 0x80008000u;

  for (int t = 0; t < n; ++t) {
    copies_wait<kAppendDepth - 1>();
    __syncwarp();  // the other lanes' angles too
    const uint32_t at = slots + (t % kAppendDepth) * (2 * kAppendThreads * 16);
    uint8_t* to = dst + t * step;
    const uint4 xw = load_shared16(at), yw = load_shared16(at + kAppendThreads * 16);
    float cs[8], sn[8];
    if (turn) {
      // Eight angles: of channels c0 .. c0 + 7, or of four pairs in either chunk.
      const uint32_t tb = tables + (t % kAppendDepth) * (kWarps * kTable);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t from = tb + (a.interleaved ? (e ? c1 : c0) * 2 : c0 * 4 + 16 * e);
        const uint4 u = load_shared16(from), v = load_shared16(from + half * 4);
        cs[4 * e] = __uint_as_float(u.x), cs[4 * e + 1] = __uint_as_float(u.y);
        cs[4 * e + 2] = __uint_as_float(u.z), cs[4 * e + 3] = __uint_as_float(u.w);
        sn[4 * e] = __uint_as_float(v.x), sn[4 * e + 1] = __uint_as_float(v.y);
        sn[4 * e + 2] = __uint_as_float(v.z), sn[4 * e + 3] = __uint_as_float(v.w);
      }
    }
    __syncwarp();  // every lane has its angles before the slot is fetched into again
    fetch(t + kAppendDepth);
    if (kind == 3) continue;
    if (plain) {  // as it is
      *reinterpret_cast<uint4*>(to + c0 * 2) = xw;
      *reinterpret_cast<uint4*>(to + c1 * 2) = yw;
      continue;
    }
    float x[8], y[8];
    unpack8<X>(xw, x);
    unpack8<X>(yw, y);
    if (turn) {
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float* z = e < 4 ? x + 2 * e : y + 2 * (e - 4);
          const float u = z[0], w = z[1];
          z[0] = u * cs[e] - w * sn[e];
          z[1] = w * cs[e] + u * sn[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float u = x[e], w = y[e];
          x[e] = u * cs[e] - w * sn[e];
          y[e] = w * cs[e] + u * sn[e];
        }
      }
    }
    uint32_t w0[4], w1[4];
    if (kind == 2) {
      round_store<X>(to + c0 * 2, x, w0);
      round_store<X>(to + c1 * 2, y, w1);
    } else {
      if constexpr (C == kTypeE4m3) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = quotient<S>(x[e], unit, inv), y[e] = quotient<S>(y[e], unit, inv);
      }
      round_store<C>(to + c0 * CB, x, w0);
      round_store<C>(to + c1 * CB, y, w1);
      if (track) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          lo[0][e] = min_pair<C>(lo[0][e], w0[e]), hi[0][e] = max_pair<C>(hi[0][e], w0[e]);
          lo[1][e] = min_pair<C>(lo[1][e], w1[e]), hi[1][e] = max_pair<C>(hi[1][e], w1[e]);
        }
      }
    }
  }
  if (track) {
    const int64_t at = (static_cast<int64_t>(id) * kv.H + h) * kv.d;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint8_t *mn = kv.kmin + (at + (x ? c1 : c0)) * CB, *mx = kv.kmax + (at + (x ? c1 : c0)) * CB;
      if (slot0 != 0) {  // earlier tokens of the page
        uint32_t w[4];
        load_pairs<C>(mn, w);
#pragma unroll
        for (int e = 0; e < 4; ++e) lo[x][e] = min_pair<C>(lo[x][e], w[e]);
        load_pairs<C>(mx, w);
#pragma unroll
        for (int e = 0; e < 4; ++e) hi[x][e] = max_pair<C>(hi[x][e], w[e]);
      }
      store_pairs<C>(mn, lo[x]);
      store_pairs<C>(mx, hi[x]);
    }
  }
}

template <int X, int C, int S = kProduct>
int launch_append_t(const PagedAppendArgs& a) {
  const int items = (2 * a.kv.H + a.Hq) * (a.kv.d / 16);
  const int slices = (items + kAppendThreads - 1) / kAppendThreads;
  int span = a.kv.page;
  if (!a.kv.kmin) {  // longer walks amortise a unit's start, as long as they leave eight CTAs to an SM
    span = 8;
    while (span < kAppendSpan && a.kv.page % (2 * span) == 0 &&
           static_cast<int64_t>(a.rows / (2 * span)) * slices >= 8 * std::max(1, device_sm_count()))
      span *= 2;
  }
  const int64_t units = a.token_start ? a.rows / span + 2 * static_cast<int64_t>(a.kv.B) : a.kv.B;
  const dim3 grid(static_cast<unsigned>(units), slices);
  return launch_serialized(true, attn_paged_append_kernel<X, C, S>, grid, dim3(kAppendThreads), 0, a.stream, a, span) ==
                 cudaSuccess
             ? kStatusOk
             : kStatusCuda;
}

}  // namespace

int launch_paged_append(const PagedAppendArgs& a, int* launches) {
  *launches = 1;
  const bool bf = a.x_type == kTypeBf16;
  if (a.kv.type != kTypeE4m3) return bf ? launch_append_t<kTypeBf16, kTypeBf16>(a) : launch_append_t<kTypeF16, kTypeF16>(a);
  switch (std::max(quotient_of(a.kv.k_scale), quotient_of(a.kv.v_scale))) {  // the more general one serves both
    case kProduct: return bf ? launch_append_t<kTypeBf16, kTypeE4m3>(a) : launch_append_t<kTypeF16, kTypeE4m3>(a);
    case kCorrected:
      return bf ? launch_append_t<kTypeBf16, kTypeE4m3, kCorrected>(a) : launch_append_t<kTypeF16, kTypeE4m3, kCorrected>(a);
    default:
      return bf ? launch_append_t<kTypeBf16, kTypeE4m3, kDivision>(a) : launch_append_t<kTypeF16, kTypeE4m3, kDivision>(a);
  }
}

}  // namespace attn
