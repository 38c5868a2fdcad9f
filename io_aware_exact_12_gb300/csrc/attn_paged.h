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
  int window = 0, sinks = 0;  // window > 0: the last `window` tokens and the first `sinks` ones (pages is null)
  int box_shift = 0;          // log2 of the keys of a box; the launcher's
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

struct PagedAssignArgs {
  PagedKv kv;
  int* table;       // kv.table and kv.lens, which this call writes
  int* lens_out;
  const int* lens;  // tokens before the step; may be lens_out
  const int* n_new;
  int* free_pages;  // ring of free_cap page numbers
  int free_cap;
  const int* free_state;  // first free page's position, number of free pages
  int* free_out;          // may be free_state
  int* token_start;       // [B + 1]
  int64_t* slots;         // [rows], or null
  int rows;
  int first, turns;  // pages of sinks, pages in turns behind them (0: no window)
  uint32_t page_mul, page_shift;  // division by the page size; the launcher's
  cudaStream_t stream;
  uint8_t* ws;
};

// Each returns a status code; the launch counts go to *launches.
int launch_paged_append(const PagedAppendArgs& a, int* launches);
int launch_paged_decode(const PagedDecodeArgs& a, int* launches);
int launch_paged_select(const PagedSelectArgs& a, int* launches);
int launch_paged_assign(const PagedAssignArgs& a, int* launches);

// Scratch bytes; they depend on sizes alone.
int64_t paged_decode_workspace(int B, int Hq, int H, int d, int64_t keys);
int64_t paged_window_keys(int window, int sinks, int64_t most);  // keys of a windowed call, for the workspace
int64_t paged_select_workspace(int B, int H, int max_pages);
int64_t paged_assign_workspace(int B);

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

// Two e4m3 bytes (the low or high half of a word) as two fp16 values; exact.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t four) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(four));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_pair_hi(uint32_t four) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(four));
  return r;
}

#endif  // __CUDACC__

}  // namespace attn
