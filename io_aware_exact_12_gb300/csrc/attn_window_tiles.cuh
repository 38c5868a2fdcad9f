// attn_window_tiles.cuh -- what the sliding-window kernels share on the device:
// tiles and their descriptors, the list of key tiles that 128 query rows see, and
// the loop in which a block takes over the work of blocks that have not started.
#pragma once

#include "attn_window.h"
#include "tc_sm103.cuh"

namespace attn {

// 4-D tiled bulk tensor load global -> shared (tma_load_3d with one dimension more).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// Tiles of 128 rows of D channels in shared memory, swizzled by TMA.
template <int D>
struct TileLayout {
  static constexpr int ROWB = D >= 64 ? 128 : 64;  // bytes of a swizzled row
  static constexpr int CH = ROWB / 2;              // elements of it
  static constexpr int NCH = D / CH;               // column chunks of a tile
  static constexpr uint32_t SWZ = ROWB == 128 ? kSwizzle128B : kSwizzle64B;
  static constexpr int SBO = 8 * ROWB;
  static constexpr int CHUNK = 128 * ROWB;         // bytes of a chunk of 128 rows
  static constexpr int TILE = 128 * D * 2;
};

// Descriptor steps (16-byte units) of the 16-deep slice kk: of a K-major tile (rows
// of D channels) and of an MN-major one (16 rows on).
template <int D>
__host__ __device__ constexpr uint32_t k_step(int kk) {
  using C = TileLayout<D>;
  return static_cast<uint32_t>(((kk * 16) / C::CH * C::CHUNK + (kk * 16) % C::CH * 2) >> 4);
}
template <int D>
__host__ __device__ constexpr uint32_t mn_step(int kk) {
  return static_cast<uint32_t>((kk * 16 * TileLayout<D>::ROWB) >> 4);
}

// A wait for work that has been issued, also after an abort.
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_test(bar, parity))
    if (global_timer_ns() - t0 > kWaitLimitNs) return;
}

// ------------------------------------------------------------------- clusters
// A barrier over the cluster's threads; what they wrote before it, also to shared
// memory, is visible to all behind it.  (`.aligned` wants a warp's lanes together.)
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of another block's shared memory in the cluster.
__device__ __forceinline__ uint32_t in_block(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 load_cluster16(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float load_cluster4(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// launch_serialized, overlapped, of blocks in clusters of `cluster`.
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(int cluster, void (*kern)(KArgs...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

// ------------------------------------------------- work of blocks not started
// Asks for the index of a block of this grid that has not started, which then
// never will: a running block takes its work (16 bytes at `addr`, signalled as
// transaction bytes on `bar`).  Once refused, a block must not ask again.
__device__ __forceinline__ void block_request(uint32_t addr, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(addr), "r"(bar)
               : "memory");
}
// The answer: blockIdx.x, or -1.
__device__ __forceinline__ int block_answer(uint32_t addr) {
  int x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\t"
      "ld.shared.b128 h, [%1];\n\t"
      "mov.b32 %0, -1;\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, h;\n\t}"
      : "=r"(x)
      : "r"(addr)
      : "memory");
  return x;
}

// The loop over items that every role runs: the first is the block's own; while it
// runs the loader asks for that of a block that has not started, and so on.
struct Items {
  uint32_t answers, b_next, b_read;  // two answers, their barriers
  volatile int* abort_flag;
  int* status;
  // The item after the k-th, or -1.
  __device__ __forceinline__ int after(int k, bool& ok) const {
    ok = ok && mbar_wait(b_next + (k & 1) * 8, (k >> 1) & 1, abort_flag, status);
    return ok ? block_answer(answers + (k & 1) * 16) : -1;
  }
  // By each other role once it has it: the issuer's thread, or a whole warp, which
  // goes on or stops together.
  __device__ __forceinline__ void read(int k) const {
    fence_proxy_async_smem();  // the answer is read before the next one is written
    mbar_arrive(b_read + (k & 1) * 8);
  }
  __device__ __forceinline__ void read_by_warp(int k, int lane, bool& ok) const {
    ok = __all_sync(0xffffffffu, ok);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(b_read + (k & 1) * 8);
  }
  // The loader's k-th question.
  __device__ __forceinline__ bool ask(int k) const {
    if (k >= 2 && !mbar_wait(b_read + (k & 1) * 8, ((k >> 1) - 1) & 1, abort_flag, status)) return false;
    mbar_arrive_expect_tx(b_next + (k & 1) * 8, 16);
    block_request(answers + (k & 1) * 16, b_next + (k & 1) * 8);
    return true;
  }
  __device__ __forceinline__ void drain_last(int asked) const {
    if (asked) drain(b_next + ((asked - 1) & 1) * 8, ((asked - 1) >> 1) & 1);
  }
};

// 128 query rows of a head, and the list of key tiles they see.
struct RowItem {
  int row0, b, h, hk;
  int ns, skip, npos;  // tiles of sinks, tiles left out behind them, tiles in all
  __device__ __forceinline__ RowItem(const WindowArgs& a, int item, int nrows, int group) {
    int rank, bh;
    grouped_rank_order(item, nrows, a.B * a.Hq, group, rank, bh);
    row0 = (nrows - 1 - rank) * 128;  // later rows, which under a wide window have more tiles, first
    b = bh / a.Hq, h = bh - b * a.Hq, hk = h / (a.Hq / a.Hk);
    const int off = a.Nk - a.Nq;
    const int w0 = max(0, row0 + off - a.window + 1) >> 7;
    ns = min(w0, (a.sinks + 127) >> 7);
    skip = w0 - ns;
    npos = ((min(row0 + 127, a.Nq - 1) + off) >> 7) - skip + 1;
  }
  __device__ __forceinline__ int key0(int p) const { return (p < ns ? p : p + skip) * 128; }
};

}  // namespace attn
