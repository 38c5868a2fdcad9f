// attn_paged_decode.cu -- attention of one new token per sequence over a paged
// cache: ragged lengths, query heads that share a key/value head, all pages or
// a list of selected ones.
//
// FlashAttention (PKM page), "注意" section: decode has no N x N matrix, its
// cost is reading the cache, and the variant for it splits the keys; the join
// is exact by the online softmax of "三招" 2.
#include <cmath>

#include "attn_paged.h"
#include "tc_sm103.cuh"

namespace attn {
namespace {

constexpr int kPdThreads = 128;

// Keys of one split of one query head; partial (m, l, O) to scratch.
template <int X, int C, int D>
__global__ void __launch_bounds__(kPdThreads) attn_paged_split_kernel(const PagedDecodeArgs a, float* part, int keys) {
  griddep_wait();  // launched overlapped (launch_serialized)
  griddep_launch_dependents();
  const PagedKv& kv = a.kv;
  constexpr int LPK = D / 8;  // lanes of a key
  constexpr int GROUPS = kPdThreads / LPK;
  constexpr int CB = C == kTypeE4m3 ? 1 : 2;
  const int s = blockIdx.x, S = gridDim.x, b = blockIdx.y / a.Hq, hq = blockIdx.y % a.Hq;
  const int h = hq / (a.Hq / kv.H);
  const int g = threadIdx.x / LPK, c = (threadIdx.x % LPK) * 8;
  const int len = checked_len(kv, b);
  const int64_t entries = a.pages ? a.n_pages : (len + kv.page - 1) / kv.page;
  const int64_t k0 = static_cast<int64_t>(s) * keys, k1 = min(entries * kv.page, k0 + keys);

  float q[8];
  load8<X>(a.q.p + b * a.q.row + hq * a.q.head + c * 2, q);
  float m = -INFINITY, l = 0.f, acc[8] = {};
  for (int64_t kk = k0; kk < k1; kk += GROUPS) {
    const int64_t key = kk + g;
    bool seen = key < k1;
    float kf[8] = {}, vf[8] = {};
    if (seen) {
      const int e = static_cast<int>(key / kv.page), slot = static_cast<int>(key % kv.page);
      const int j = a.pages ? a.pages[(static_cast<int64_t>(b) * kv.H + h) * a.n_pages + e] : e;
      seen = j >= 0 && static_cast<int64_t>(j) * kv.page + slot < len;
      if (seen) {
        const int id = checked_page(kv, b, j);
        seen = id >= 0;
        if (seen) {
          load8<C>(kv.k + id * kv.k_page + h * kv.k_head + slot * kv.k_tok + c * CB, kf);
          load8<C>(kv.v + id * kv.v_page + h * kv.v_head + slot * kv.v_tok + c * CB, vf);
        }
      }
    }
    float t = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) t = fmaf(q[e], kf[e], t);
#pragma unroll
    for (int x = LPK / 2; x; x >>= 1) t += __shfl_xor_sync(0xffffffffu, t, x);
    if (!seen) continue;
    t *= a.sl2;
    const float mn = fmaxf(m, t);
    if (mn == -INFINITY) continue;
    const float alpha = exp2f(m - mn), p = exp2f(t - mn);
    m = mn;
    l = l * alpha + p;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = acc[e] * alpha + p * vf[e];
  }
  __shared__ float sm_m[GROUPS], sm_l[GROUPS], sm_o[GROUPS][D];
  if (c == 0) sm_m[g] = m, sm_l[g] = l;
#pragma unroll
  for (int e = 0; e < 8; ++e) sm_o[g][c + e] = acc[e];
  __syncthreads();
  float mm = -INFINITY;
  for (int i = 0; i < GROUPS; ++i) mm = fmaxf(mm, sm_m[i]);
  float* out = part + (static_cast<int64_t>(blockIdx.y) * S + s) * (D + 2);
  for (int x = threadIdx.x; x < D + 1; x += kPdThreads) {
    float sum = 0.f;
    for (int i = 0; i < GROUPS; ++i)
      if (sm_m[i] != -INFINITY) sum += exp2f(sm_m[i] - mm) * (x < D ? sm_o[i][x] : sm_l[i]);
    out[x < D ? 2 + x : 1] = sum;
  }
  if (threadIdx.x == 0) out[0] = mm;
}

template <int X, int D>
__global__ void __launch_bounds__(128) attn_paged_merge_kernel(const PagedDecodeArgs a, const float* part, int S) {
  griddep_wait();  // launched overlapped (launch_serialized)
  griddep_launch_dependents();
  const float* p = part + static_cast<int64_t>(blockIdx.x) * S * (D + 2);
  float mm = -INFINITY;
  for (int s = 0; s < S; ++s) mm = fmaxf(mm, p[s * (D + 2)]);
  float l = 0.f;
  for (int s = 0; s < S; ++s)
    if (p[s * (D + 2)] != -INFINITY) l += exp2f(p[s * (D + 2)] - mm) * p[s * (D + 2) + 1];
  const int c = threadIdx.x;
  if (c < D) {
    float o = 0.f;
    for (int s = 0; s < S; ++s)
      if (p[s * (D + 2)] != -INFINITY) o += exp2f(p[s * (D + 2)] - mm) * p[s * (D + 2) + 2 + c];
    o = l > 0.f ? o / l * a.kv.v_scale : l;  // no key: 0 (NaN stays NaN)
    const int64_t at = static_cast<int64_t>(blockIdx.x) * D + c;
    if constexpr (X == kTypeBf16) reinterpret_cast<__nv_bfloat16*>(a.o)[at] = __float2bfloat16_rn(o);
    else reinterpret_cast<__half*>(a.o)[at] = __float2half_rn(o);
  }
  if (c == 0) a.lse[blockIdx.x] = l == 0.f ? -INFINITY : (mm + log2f(l)) * 0.69314718055994531f;
}

int split_count(int B, int Hq, int64_t keys) {
  const int64_t want = (152 * 8 + static_cast<int64_t>(B) * Hq - 1) / (static_cast<int64_t>(B) * Hq);
  return static_cast<int>(std::max<int64_t>(1, std::min(std::min<int64_t>(want, (keys + 255) / 256), int64_t{256})));
}

template <int X, int C, int D>
int launch_t(const PagedDecodeArgs& a) {
  const int64_t keys = static_cast<int64_t>(a.pages ? a.n_pages : a.kv.max_pages) * a.kv.page;
  const int S = split_count(a.kv.B, a.Hq, keys);
  float* part = reinterpret_cast<float*>(a.ws);
  if (launch_serialized(true, attn_paged_split_kernel<X, C, D>, dim3(S, a.kv.B * a.Hq), dim3(kPdThreads), 0, a.stream,
                        a, part, static_cast<int>((keys + S - 1) / S)) != cudaSuccess)
    return kStatusCuda;
  return launch_serialized(true, attn_paged_merge_kernel<X, D>, dim3(a.kv.B * a.Hq), dim3(128), 0, a.stream, a, part,
                           S) == cudaSuccess
             ? kStatusOk
             : kStatusCuda;
}

template <int X, int C>
int launch_d(const PagedDecodeArgs& a) {
  switch (a.kv.d) {
    case 32: return launch_t<X, C, 32>(a);
    case 64: return launch_t<X, C, 64>(a);
    default: return launch_t<X, C, 128>(a);
  }
}

}  // namespace

int64_t paged_decode_workspace(int B, int Hq, int H, int d, int page, int n_pages) {
  const int64_t keys = static_cast<int64_t>(n_pages) * page;
  return static_cast<int64_t>(B) * Hq * split_count(B, Hq, keys) * (d + 2) * 4;
}

int launch_paged_decode(const PagedDecodeArgs& a, int* launches) {
  *launches = 2;
  if (a.x_type == kTypeBf16)
    return a.kv.type == kTypeE4m3 ? launch_d<kTypeBf16, kTypeE4m3>(a) : launch_d<kTypeBf16, kTypeBf16>(a);
  return a.kv.type == kTypeE4m3 ? launch_d<kTypeF16, kTypeE4m3>(a) : launch_d<kTypeF16, kTypeF16>(a);
}

}  // namespace attn
