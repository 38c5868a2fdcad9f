// attn_window_bwd.cu -- sliding-window attention with sinks, backward:
//   P = exp(s - LSE), D_i = dO_i . O_i, dS = P o (dO V^T - D),
//   dQ = scale dS K, dK = scale sum dS^T Q, dV = sum P^T dO,
// the sums over the query heads that share a key/value head.
//
// First form: a warp to a query row for dQ, a warp to a key for dK and dV.
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

template <bool BF16>
__device__ __forceinline__ float element(const uint8_t* row, int c) {
  return unpack2<BF16>(reinterpret_cast<const uint16_t*>(row)[c]).x;
}

// P and dS of one (query, key) pair.
template <int D, bool BF16>
__device__ __forceinline__ void pair(const WindowArgs& a, int b, int h, int i, const uint8_t* k, const uint8_t* v, float& p, float& ds) {
  const uint8_t *q = a.q.p + b * a.q.b + h * a.q.h + i * a.q.n, *dO = a.dO.p + b * a.dO.b + h * a.dO.h + i * a.dO.n;
  const uint8_t* o = a.o.p + b * a.o.b + h * a.o.h + i * a.o.n;
  const float s = dot_rows<D, BF16>(q, k) * (a.negate ? -a.sl2 : a.sl2);
  p = exp2f(s - a.lse[(static_cast<int64_t>(b) * a.Hq + h) * a.Nq + i] * 1.4426950408889634f);
  ds = p * (dot_rows<D, BF16>(dO, v) - dot_rows<D, BF16>(dO, o));
}

template <int D, bool BF16>
__global__ void __launch_bounds__(128) attn_window_dq_kernel(const WindowArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(a.B) * a.Hq * a.Nq) return;
  const int i = static_cast<int>(row % a.Nq), h = static_cast<int>(row / a.Nq % a.Hq), b = static_cast<int>(row / a.Nq / a.Hq);
  const int hk = h / (a.Hq / a.Hk);
  const uint8_t *k = a.k.p + b * a.k.b + hk * a.k.h, *v = a.v.p + b * a.v.b + hk * a.v.h;
  const int p = i + a.Nk - a.Nq, lo = max(0, p - a.window + 1), sinks = min(a.sinks, lo);
  float acc[D / 32] = {};
  for (int at = 0; at < sinks + p + 1 - lo; at += 32) {
    const int t = at + lane, j = t < sinks ? t : lo + t - sinks;
    float w = 0.f, ds = 0.f;
    if (j <= p) pair<D, BF16>(a, b, h, i, k + j * a.k.n, v + j * a.v.n, w, ds);
    for (int x = 0; x < 32; ++x) {
      const float g = __shfl_sync(0xffffffffu, ds, x);
      const int jx = __shfl_sync(0xffffffffu, j, x);
      if (jx > p) break;
      for (int c = 0; c < D / 32; ++c) acc[c] = fmaf(g, element<BF16>(k + jx * a.k.n, c * 32 + lane), acc[c]);
    }
  }
  uint16_t* out = reinterpret_cast<uint16_t*>(a.dq.p + b * a.dq.b + h * a.dq.h + i * a.dq.n);
  for (int c = 0; c < D / 32; ++c) out[c * 32 + lane] = static_cast<uint16_t>(pack2<BF16>(acc[c] * a.scale, 0.f) & 0xffffu);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(128) attn_window_dkv_kernel(const WindowArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(a.B) * a.Hk * a.Nk) return;
  const int j = static_cast<int>(row % a.Nk), hk = static_cast<int>(row / a.Nk % a.Hk), b = static_cast<int>(row / a.Nk / a.Hk);
  const uint8_t *k = a.k.p + b * a.k.b + hk * a.k.h + j * a.k.n, *v = a.v.p + b * a.v.b + hk * a.v.h + j * a.v.n;
  const int G = a.Hq / a.Hk, off = a.Nk - a.Nq;
  const int i0 = max(0, j - off), i1 = j < a.sinks ? a.Nq : static_cast<int>(min(static_cast<int64_t>(a.Nq), static_cast<int64_t>(j) - off + a.window));
  float gk[D / 32] = {}, gv[D / 32] = {};
  for (int h = hk * G; h < (hk + 1) * G; ++h)
    for (int at = i0; at < i1; at += 32) {
      float w = 0.f, ds = 0.f;
      if (at + lane < i1) pair<D, BF16>(a, b, h, at + lane, k, v, w, ds);
      for (int x = 0; x < 32 && at + x < i1; ++x) {
        const float wx = __shfl_sync(0xffffffffu, w, x), sx = __shfl_sync(0xffffffffu, ds, x);
        const uint8_t *q = a.q.p + b * a.q.b + h * a.q.h + (at + x) * a.q.n, *dO = a.dO.p + b * a.dO.b + h * a.dO.h + (at + x) * a.dO.n;
        for (int c = 0; c < D / 32; ++c) {
          gk[c] = fmaf(sx, element<BF16>(q, c * 32 + lane), gk[c]);
          gv[c] = fmaf(wx, element<BF16>(dO, c * 32 + lane), gv[c]);
        }
      }
    }
  uint16_t* dk = reinterpret_cast<uint16_t*>(a.dk.p + b * a.dk.b + hk * a.dk.h + j * a.dk.n);
  uint16_t* dv = reinterpret_cast<uint16_t*>(a.dv.p + b * a.dv.b + hk * a.dv.h + j * a.dv.n);
  for (int c = 0; c < D / 32; ++c) {
    dk[c * 32 + lane] = static_cast<uint16_t>(pack2<BF16>(gk[c] * a.scale, 0.f) & 0xffffu);
    dv[c * 32 + lane] = static_cast<uint16_t>(pack2<BF16>(gv[c], 0.f) & 0xffffu);
  }
}

template <int D, bool BF16>
int launch_t(const WindowArgs& a) {
  const int64_t rows = static_cast<int64_t>(a.B) * a.Hq * a.Nq, keys = static_cast<int64_t>(a.B) * a.Hk * a.Nk;
  attn_window_dq_kernel<D, BF16><<<static_cast<unsigned>((rows + 3) / 4), 128, 0, a.stream>>>(a);
  attn_window_dkv_kernel<D, BF16><<<static_cast<unsigned>((keys + 3) / 4), 128, 0, a.stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? kStatusOk : kStatusCuda;
}

template <int D>
int launch_d(const WindowArgs& a) { return a.bf16 ? launch_t<D, true>(a) : launch_t<D, false>(a); }

}  // namespace

int launch_window_bwd(const WindowArgs& a, int* launches) {
  *launches = 2;
  return a.d == 32 ? launch_d<32>(a) : a.d == 64 ? launch_d<64>(a) : launch_d<128>(a);
}

}  // namespace attn
