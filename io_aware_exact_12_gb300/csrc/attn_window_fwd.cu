// attn_window_fwd.cu -- sliding-window attention with sinks, forward.
//
// First form: a warp to a query row, a lane to a key for the logits and to
// D / 32 channels for the output; online softmax over 32 keys at a time.
#include "attn_window.h"
#include "tc_sm103.cuh"

namespace attn {
namespace {

template <int D, bool BF16>
__device__ __forceinline__ float dot_rows(const uint8_t* a, const uint8_t* b) {
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < D; c += 8) {
    const uint4 x = *reinterpret_cast<const uint4*>(a + c * 2), y = *reinterpret_cast<const uint4*>(b + c * 2);
    const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 u = unpack2<BF16>(xw[e]), w = unpack2<BF16>(yw[e]);
      s = fmaf(u.x, w.x, fmaf(u.y, w.y, s));
    }
  }
  return s;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(128) attn_window_fwd_kernel(const WindowArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(a.B) * a.Hq * a.Nq) return;
  const int i = static_cast<int>(row % a.Nq), h = static_cast<int>(row / a.Nq % a.Hq), b = static_cast<int>(row / a.Nq / a.Hq);
  const uint8_t* q = a.q.p + b * a.q.b + h * a.q.h + i * a.q.n;
  const int hk = h / (a.Hq / a.Hk);
  const uint8_t *k = a.k.p + b * a.k.b + hk * a.k.h, *v = a.v.p + b * a.v.b + hk * a.v.h;
  const int p = i + a.Nk - a.Nq, lo = max(0, p - a.window + 1), sinks = min(a.sinks, lo);
  const float mul = a.negate ? -a.sl2 : a.sl2;
  float m = -INFINITY, l = 0.f, acc[D / 32] = {};
  for (int at = 0; at < sinks + p + 1 - lo; at += 32) {
    const int t = at + lane, j = t < sinks ? t : lo + t - sinks;
    const bool seen = j <= p;
    const float s = seen ? dot_rows<D, BF16>(q, k + j * a.k.n) * mul : -INFINITY;
    float top = s;
    for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float mn = fmaxf(m, top), f = m == -INFINITY ? 0.f : exp2f(m - mn);
    const float w = seen && mn > -INFINITY ? exp2f(s - mn) : 0.f;
    m = mn;
    l = l * f + w;
    for (int c = 0; c < D / 32; ++c) acc[c] *= f;
    for (int x = 0; x < 32; ++x) {
      const float wx = __shfl_sync(0xffffffffu, w, x);
      const int jx = __shfl_sync(0xffffffffu, j, x);
      if (jx > p) break;
      const uint16_t* vr = reinterpret_cast<const uint16_t*>(v + jx * a.v.n);
      for (int c = 0; c < D / 32; ++c) acc[c] = fmaf(wx, unpack2<BF16>(vr[c * 32 + lane]).x, acc[c]);
    }
  }
  for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  uint16_t* o = reinterpret_cast<uint16_t*>(a.o.p + b * a.o.b + h * a.o.h + i * a.o.n);
  for (int c = 0; c < D / 32; ++c) o[c * 32 + lane] = static_cast<uint16_t>(pack2<BF16>(acc[c] / l, 0.f) & 0xffffu);
  if (lane == 0) a.lse[row] = (m + log2f(l)) * 0.69314718055994531f;
}

template <int D>
int launch_d(const WindowArgs& a) {
  const int64_t rows = static_cast<int64_t>(a.B) * a.Hq * a.Nq;
  const dim3 grid(static_cast<unsigned>((rows + 3) / 4));
  if (a.bf16) attn_window_fwd_kernel<D, true><<<grid, 128, 0, a.stream>>>(a);
  else attn_window_fwd_kernel<D, false><<<grid, 128, 0, a.stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? kStatusOk : kStatusCuda;
}

}  // namespace

int launch_window_fwd(const WindowArgs& a, int* launches) {
  *launches = 1;
  return a.d == 32 ? launch_d<32>(a) : a.d == 64 ? launch_d<64>(a) : launch_d<128>(a);
}

}  // namespace attn
