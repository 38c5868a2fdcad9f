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
// positions (a page with summaries, else 8 tokens, which a page boundary never
// cuts).  A thread owns sixteen channels of one head (an item: the two
// 8-element chunks that the rotation couples) and walks the unit's tokens, so
// the minima and maxima stay in its registers and need no exchange.
#include <cmath>

#include "attn_paged.h"
#include "tc_sm103.cuh"

namespace attn {
namespace {

constexpr int kAppendThreads = 128;
constexpr int kAppendSpan = 8;   // tokens of a unit without summaries
constexpr int kAppendBatch = 4;  // tokens in flight per thread

template <int X, int C>
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
  else return;
  const bool turn = kind != 1 && i < a.rot / 16;
  int c0 = 16 * i, c1 = 16 * i + 8;  // first channels of the two chunks
  if (turn && !a.interleaved) c0 = 8 * i, c1 = a.rot / 2 + 8 * i;

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
  const float inv = 1.f / (kind ? kv.v_scale : kv.k_scale);

  float lo0[8], lo1[8], hi0[8], hi1[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) lo0[e] = lo1[e] = INFINITY, hi0[e] = hi1[e] = -INFINITY;

  for (int t0 = 0; t0 < n; t0 += kAppendBatch) {
    float x[kAppendBatch][8], y[kAppendBatch][8];
#pragma unroll
    for (int t = 0; t < kAppendBatch; ++t)
      if (t0 + t < n) {
        load8<X>(src + (t0 + t) * in.row + c0 * 2, x[t]);
        load8<X>(src + (t0 + t) * in.row + c1 * 2, y[t]);
      }
#pragma unroll
    for (int t = 0; t < kAppendBatch; ++t) {
      if (t0 + t >= n) break;
      if (turn) {
        const int64_t at = static_cast<int64_t>(p0 + t0 + t) * (a.rot / 2) + 8 * i;
        float cs[8], sn[8];
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          *reinterpret_cast<float4*>(cs + e) = __ldg(reinterpret_cast<const float4*>(a.cos + at + e));
          *reinterpret_cast<float4*>(sn + e) = __ldg(reinterpret_cast<const float4*>(a.sin + at + e));
        }
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float* z = e < 4 ? x[t] + 2 * e : y[t] + 2 * (e - 4);
            const float u = z[0], w = z[1];
            z[0] = u * cs[e] - w * sn[e];
            z[1] = w * cs[e] + u * sn[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float u = x[t][e], w = y[t][e];
            x[t][e] = u * cs[e] - w * sn[e];
            y[t][e] = w * cs[e] + u * sn[e];
          }
        }
      }
      uint8_t* to = dst + (t0 + t) * step;
      if (kind == 2) {
        store8<X>(to + c0 * 2, x[t]);
        store8<X>(to + c1 * 2, y[t]);
      } else {
        if constexpr (C == kTypeE4m3) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[t][e] *= inv, y[t][e] *= inv;
        }
        store8<C>(to + c0 * CB, x[t]);
        store8<C>(to + c1 * CB, y[t]);
        if (kv.kmin && kind == 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {  // fminf / fmaxf pass over a NaN
            lo0[e] = fminf(lo0[e], x[t][e]), hi0[e] = fmaxf(hi0[e], x[t][e]);
            lo1[e] = fminf(lo1[e], y[t][e]), hi1[e] = fmaxf(hi1[e], y[t][e]);
          }
        }
      }
    }
  }
  if (kv.kmin && kind == 0) {
    const int64_t at = (static_cast<int64_t>(id) * kv.H + h) * kv.d;
    uint8_t *mn = kv.kmin + at * CB, *mx = kv.kmax + at * CB;
    if (slot0 != 0) {  // earlier tokens of the page
      float w[8];
#define ATTN_JOIN(acc, ptr, c, op)         \
  load8<C>(ptr + (c) * CB, w);             \
  _Pragma("unroll") for (int e = 0; e < 8; ++e) acc[e] = op(acc[e], w[e]);
      ATTN_JOIN(lo0, mn, c0, fminf)
      ATTN_JOIN(lo1, mn, c1, fminf)
      ATTN_JOIN(hi0, mx, c0, fmaxf)
      ATTN_JOIN(hi1, mx, c1, fmaxf)
#undef ATTN_JOIN
    }
    store8<C>(mn + c0 * CB, lo0);
    store8<C>(mn + c1 * CB, lo1);
    store8<C>(mx + c0 * CB, hi0);
    store8<C>(mx + c1 * CB, hi1);
  }
}

template <int X, int C>
int launch_append_t(const PagedAppendArgs& a) {
  const int span = a.kv.kmin ? a.kv.page : kAppendSpan;
  const int64_t units = a.token_start ? a.rows / span + 2 * static_cast<int64_t>(a.kv.B) : a.kv.B;
  const int items = (2 * a.kv.H + a.Hq) * (a.kv.d / 16);
  const dim3 grid(static_cast<unsigned>(units), (items + kAppendThreads - 1) / kAppendThreads);
  return launch_serialized(true, attn_paged_append_kernel<X, C>, grid, dim3(kAppendThreads), 0, a.stream, a, span) ==
                 cudaSuccess
             ? kStatusOk
             : kStatusCuda;
}

}  // namespace

int launch_paged_append(const PagedAppendArgs& a, int* launches) {
  *launches = 1;
  if (a.x_type == kTypeBf16)
    return a.kv.type == kTypeE4m3 ? launch_append_t<kTypeBf16, kTypeE4m3>(a) : launch_append_t<kTypeBf16, kTypeBf16>(a);
  return a.kv.type == kTypeE4m3 ? launch_append_t<kTypeF16, kTypeE4m3>(a) : launch_append_t<kTypeF16, kTypeF16>(a);
}

}  // namespace attn
