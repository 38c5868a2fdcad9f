// attn_paged_select.cu -- for each sequence and key/value head the pages whose
// keys can have the largest logit with the new token's queries.
//
//   score(p) = max over the head's queries g of
//              sum_c max(q_gc kmin_pc, q_gc kmax_pc),
//
// the least upper bound of q_g . k over the box that the page's summary spans.
// The first and last pages of a sequence are always taken; the rest go by the
// score, equal ones by the lower index.  Two pages next to the border must not
// change places by rounding, so the order is that of scores in 64 bits.
#include <cmath>

#include "attn_paged.h"
#include "tc_sm103.cuh"

namespace attn {
namespace {

constexpr int kSelThreads = 512;

// Order-preserving map of a score to an unsigned key; NaN ranks first.
__device__ __forceinline__ uint64_t key64(double x) {
  if (isnan(x)) return ~0ull;
  x = x == 0.0 ? 0.0 : x;  // -0 equals +0
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x));
  return (u >> 63) ? ~u : u | (1ull << 63);
}

template <int X>
__device__ __forceinline__ double load1(const uint8_t* p, int i) {
  if constexpr (X == kTypeBf16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
  else if constexpr (X == kTypeF16) return __half2float(reinterpret_cast<const __half*>(p)[i]);
  else return __half2float(__half(__nv_cvt_fp8_to_halfraw(p[i], __NV_E4M3)));
}

// Sum of one value per thread over the block, given to every thread.
__device__ __forceinline__ int block_sum(int v, int* sm) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();  // sm is free again
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  int s = 0;
  for (int i = 0; i < kSelThreads / 32; ++i) s += sm[i];
  return s;
}

template <int X, int C>
__global__ void __launch_bounds__(kSelThreads) attn_paged_select_kernel(const PagedSelectArgs a) {
  griddep_wait();  // launched overlapped (launch_serialized)
  griddep_launch_dependents();
  const PagedKv& kv = a.kv;
  constexpr int CB = C == kTypeE4m3 ? 1 : 2;
  __shared__ int sm[kSelThreads / 32];
  const int b = blockIdx.x / kv.H, h = blockIdx.x % kv.H, G = a.Hq / kv.H;
  const int used = (checked_len(kv, b) + kv.page - 1) / kv.page;
  int* out = a.pages + static_cast<int64_t>(blockIdx.x) * a.n_select;
  if (used <= a.n_select) {
    for (int i = threadIdx.x; i < a.n_select; i += kSelThreads) out[i] = i < used ? i : -1;
    return;
  }
  uint64_t* key = reinterpret_cast<uint64_t*>(a.ws) + static_cast<int64_t>(blockIdx.x) * kv.max_pages;
  for (int j = threadIdx.x; j < used; j += kSelThreads) {
    uint64_t k = ~0ull;
    if (j >= a.keep_first && j < used - a.keep_last) {
      const int id = checked_page(kv, b, j);
      k = 0;
      if (id >= 0) {
        const int64_t at = (static_cast<int64_t>(id) * kv.H + h) * kv.d * CB;
        double best = -INFINITY;
        for (int g = 0; g < G; ++g) {
          const uint8_t* q = a.q.p + b * a.q.row + (h * G + g) * a.q.head;
          double s = 0.0;
          for (int c = 0; c < kv.d; ++c) {
            const double x = load1<X>(q, c);
            s = fma(x, x >= 0.0 ? load1<C>(kv.kmax + at, c) : load1<C>(kv.kmin + at, c), s);
          }
          best = isnan(s) || isnan(best) ? NAN : fmax(best, s);
        }
        k = key64(best);
      }
    }
    key[j] = k;
  }
  __syncthreads();
  // The n-th largest key, bit by bit from the top.
  uint64_t border = 0;
  for (int bit = 63; bit >= 0; --bit) {
    const uint64_t t = border | (1ull << bit);
    int n = 0;
    for (int j = threadIdx.x; j < used; j += kSelThreads) n += key[j] >= t;
    if (block_sum(n, sm) >= a.n_select) border = t;
  }
  int above = 0;
  for (int j = threadIdx.x; j < used; j += kSelThreads) above += key[j] > border;
  int equal = a.n_select - block_sum(above, sm);  // so many of those at the border, lowest first
  // Ascending output: pages in chunks of the block, ranks by a scan.
  int base = 0;
  for (int j0 = 0; j0 < used; j0 += kSelThreads) {
    const int j = j0 + threadIdx.x;
    const uint64_t k = j < used ? key[j] : 0;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const bool eq = j < used && k == border;
    const uint32_t be = __ballot_sync(0xffffffffu, eq);
    __syncthreads();
    if (lane == 0) sm[w] = __popc(be);
    __syncthreads();
    int before = 0, total = 0;
    for (int i = 0; i < kSelThreads / 32; ++i) before += i < w ? sm[i] : 0, total += sm[i];
    const bool take = j < used && (k > border || (eq && before + __popc(be & ((1u << lane) - 1)) < equal));
    equal = max(0, equal - total);
    const uint32_t bt = __ballot_sync(0xffffffffu, take);
    __syncthreads();
    if (lane == 0) sm[w] = __popc(bt);
    __syncthreads();
    int rank = base;
    for (int i = 0; i < kSelThreads / 32; ++i) rank += i < w ? sm[i] : 0, base += sm[i];
    if (take) out[rank + __popc(bt & ((1u << lane) - 1))] = j;
  }
}

template <int X, int C>
int launch_t(const PagedSelectArgs& a) {
  return launch_serialized(true, attn_paged_select_kernel<X, C>, dim3(a.kv.B * a.kv.H), dim3(kSelThreads), 0, a.stream,
                           a) == cudaSuccess
             ? kStatusOk
             : kStatusCuda;
}

}  // namespace

int64_t paged_select_workspace(int B, int H, int max_pages) { return static_cast<int64_t>(B) * H * max_pages * 8; }

int launch_paged_select(const PagedSelectArgs& a, int* launches) {
  *launches = 1;
  if (a.x_type == kTypeBf16)
    return a.kv.type == kTypeE4m3 ? launch_t<kTypeBf16, kTypeE4m3>(a) : launch_t<kTypeBf16, kTypeBf16>(a);
  return a.kv.type == kTypeE4m3 ? launch_t<kTypeF16, kTypeE4m3>(a) : launch_t<kTypeF16, kTypeF16>(a);
}

}  // namespace attn
