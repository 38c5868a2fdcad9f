// attn_paged.h -- what the paged-cache kernels share: the argument bundles the
// C ABI fills, element loads and the device-side check.  Not part of the ABI.
//
// A paged cache holds key and value rows in pages of `page` tokens; sequence
// b's token at position p lies in page block_table[b][p / page], slot p % page.
// Lengths and tables live on the device and change from step to step, so the
// host sees sizes only and every kernel checks the page numbers and lengths it
// reads: a bad one is skipped (never dereferenced) and recorded.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn_internal.h"

namespace attn {

// Element types of the C ABI (attn_type_t).
constexpr int kTypeBf16 = 0;
constexpr int kTypeF16 = 1;
constexpr int kTypeE4m3 = 2;

inline int type_bytes(int type) { return type == kTypeE4m3 ? 1 : 2; }

// Strides are in bytes.
struct PagedKv {
  uint8_t *k, *v;
  int64_t k_page, k_head, k_tok, v_page, v_head, v_tok;
  uint8_t *kmin, *kmax;  // [num_pages][H][d], or null
  const int* table;
  int64_t table_stride;  // ints
  const int* lens;
  int num_pages, page, H, d, max_pages, B;
  int type;
  float k_scale, v_scale;
  int* check;  // sticky word of device-side checks
};

struct PagedRows {  // [rows][heads][d], strides in bytes
  uint8_t* p;
  int64_t row, head;
};

struct PagedAppendArgs {
  PagedKv kv;
  PagedRows k, v, q, q_out;
  int Hq;                  // 0: no q
  int rows;
  const int* token_start;  // null: row b belongs to sequence b
  const float *cos, *sin;  // [table_rows][rot / 2]
  int table_rows, rot;
  int interleaved;
  int x_type;
  cudaStream_t stream;
};

struct PagedDecodeArgs {
  PagedKv kv;
  PagedRows q;
  int Hq;
  uint8_t* o;  // [B][Hq][d]
  float* lse;  // [B][Hq]
  const int* pages;  // [B][H][n_pages] page indices of the sequence, or null: all pages
  int n_pages;
  float sl2;  // scale * k_scale * log2(e), signed
  int x_type;
  cudaStream_t stream;
  uint8_t* ws;
  int* status;  // sticky word of bounded waits
};

struct PagedSelectArgs {
  PagedKv kv;
  PagedRows q;
  int Hq;
  int* pages;  // [B][H][n_select]
  int n_select, keep_first, keep_last;
  int x_type;
  cudaStream_t stream;
  uint8_t* ws;
};

// Each returns a status code; the launch counts go to *launches.
int launch_paged_append(const PagedAppendArgs& a, int* launches);
int launch_paged_decode(const PagedDecodeArgs& a, int* launches);
int launch_paged_select(const PagedSelectArgs& a, int* launches);

// Scratch bytes; they depend on sizes alone.
int64_t paged_decode_workspace(int B, int Hq, int H, int d, int page, int n_pages);
int64_t paged_select_workspace(int B, int H, int max_pages);

#ifdef __CUDACC__

__device__ __forceinline__ void record_check(int* word) { atomicExch(word, kStatusDeviceCheck); }

// Length of sequence b, cut to what its table row can hold.
__device__ __forceinline__ int checked_len(const PagedKv& kv, int b) {
  const int n = kv.lens[b];
  const int64_t most = static_cast<int64_t>(kv.max_pages) * kv.page;
  if (n < 0 || n > most) {
    record_check(kv.check);
    return n < 0 ? 0 : static_cast<int>(most);
  }
  return n;
}

// Physical page of the sequence's page j, or -1 (recorded) where the table has none.
__device__ __forceinline__ int checked_page(const PagedKv& kv, int b, int j) {
  const int id = kv.table[b * kv.table_stride + j];
  if (id < 0 || id >= kv.num_pages) {
    record_check(kv.check);
    return -1;
  }
  return id;
}

// Eight consecutive elements as fp32.
template <int TYPE>
__device__ __forceinline__ void load8(const uint8_t* p, float (&f)[8]) {
  if constexpr (TYPE == kTypeE4m3) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    const uint32_t u[2] = {w.x, w.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2_raw h =
          __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(u[i >> 1] >> ((i & 1) * 16)), __NV_E4M3);
      const float2 x = __half22float2(__half2(h));
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    }
  } else {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 x;
      if constexpr (TYPE == kTypeBf16)
        x = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
      else
        x = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    }
  }
}

// Rounds eight fp32 values to the element type (to nearest even; e4m3
// saturates at +-448 and keeps NaN) and stores them.  f becomes the values
// as stored.
template <int TYPE>
__device__ __forceinline__ void store8(uint8_t* p, float (&f)[8]) {
  if constexpr (TYPE == kTypeE4m3) {
    uint32_t u[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_fp8x2_storage_t s =
          __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i], f[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
      u[i >> 1] |= static_cast<uint32_t>(s) << ((i & 1) * 16);
      const float2 x = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(s, __NV_E4M3)));
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    }
    *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
  } else {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 x;
      if constexpr (TYPE == kTypeBf16) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&b);
        x = __bfloat1622float2(b);
      } else {
        const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&h);
        x = __half22float2(h);
      }
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

// D += A B of m16n8k16: rows are lane / 4 (a0, a2) and that + 8 (a1, a3), fp32 sums.
template <bool BF16>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  if constexpr (BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two e4m3 bytes (low half of the word) as two fp16 values; exact.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(two));
  return r;
}

#endif  // __CUDACC__

}  // namespace attn
