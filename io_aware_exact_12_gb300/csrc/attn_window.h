// attn_window.h -- argument bundle of the sliding-window kernels
// (attn_window_fwd.cu, attn_window_bwd.cu).  Not part of the ABI.
//
// Query i of Nq stands at position p = i + Nk - Nq; key j is visible to it iff
// j <= p and (j > p - window or j < sinks).  Query head h reads key/value head
// h / (Hq / Hk).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "attn_internal.h"

namespace attn {

struct Bhnd {  // [B][heads][N][d] with contiguous channels, strides in bytes
  uint8_t* p;
  int64_t b, h, n;
};

struct WindowArgs {
  Bhnd q, k, v, o;
  Bhnd dO, dq, dk, dv;  // backward only
  float* lse;           // [B][Hq][Nq]; the backward reads it
  int B, Hq, Hk, Nq, Nk, d;
  int window, sinks;    // at most Nk each
  float sl2;            // |scale| * log2(e)
  float scale;
  int negate;           // scale < 0
  bool bf16;
  cudaStream_t stream;
  int* status;
  uint8_t* ws;          // backward only: window_bwd_workspace() bytes
};

// 4-D tiled map of a [B][heads][N][d] tensor: dims (d, N, heads, B), box
// (box_inner, 128, 1, 1), swizzled over the box's rows, zero fill.
bool encode_strided_map(CUtensorMap* map, const Bhnd& t, int B, int heads, int N, int d, int box_inner, bool bf16);

int launch_window_fwd(const WindowArgs& a, int* launches);
int launch_window_bwd(const WindowArgs& a, int* launches);
int64_t window_bwd_workspace(const WindowArgs& a);  // from the sizes alone

}  // namespace attn
