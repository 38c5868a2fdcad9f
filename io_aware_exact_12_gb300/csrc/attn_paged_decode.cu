// attn_paged_decode.cu -- attention of one new token per sequence over a paged
// cache: ragged lengths, query heads that share a key/value head, all pages or
// a list of selected ones.
//
// FlashAttention (PKM page), "注意" section: decode has no N x N matrix, its
// cost is reading the cache, and the variant for it splits the keys; the join
// is exact by the online softmax of "三招" 2: with m = max_s m_s,
//     l = sum_s e^{m_s - m} l_s,   O = sum_s e^{m_s - m} O_s / l.
//
// Every cached byte is read once for up to 16 query heads to a key/value head (once
// per 16 beyond), so HBM bounds it: G = Hq / Hkv query heads make 2 G flops per
// element, beyond the fp32 units' rate from G = 4 or so.  The products run as
// m16n8k16 matrix instructions, 16 rows of the cache times 8 or 16 query heads.  At
// 6 TB/s and G = 4 they keep the tensor pipe 13 % busy (e4m3, widened to fp16 in
// registers: 24 %), so tcgen05, whose operands would have to lie in shared memory as
// 64 rows at least and widened, has nothing to gain there.
//
//   attn_paged_decode_kernel : two or three CTAs per SM, each with a share of all
//       tiles of keys (tile lists of the items (b, KV head, group of up to 16
//       query heads) laid end to end; the lengths are on the device, so every
//       CTA sums them and finds its own share).  One producer warp walks the
//       page tables and keeps a ring of TMA loads in flight, boxes of rows that
//       never cross a page; four consumer warps take tiles in turn, each with an
//       online softmax of its own, and are merged in shared memory where an
//       item ends.  Short items go whole to clusters of CTAs instead, which join
//       their results through shared memory.
//   The weights multiply V as two 16-bit words (one and its remainder), so O keeps
//   what fp32 weights give up to 3 2^-16 and l is the fp32 sum of the weights as they are.
//   attn_paged_merge_kernel : joins the items that were cut by a CTA border.
//
// Measured (GB300, GPU time in a replayed graph; calls one by one take 1 to 3 us
// more; the copy's rate is 6.8 TB/s): two sequences of 131071 tokens, 64 / 8 heads of
// 128, fp16, 1074 MB: 157 us (6.8 TB/s); 61 sequences of up to 8192, 32 / 8 heads of
// 128, bf16, 965 MB: 152 us (6.3 TB/s); 128 of up to 4096, 16 / 16 heads of 64, e4m3,
// 511 MB: 94 us (5.4 TB/s; its items are short, an item's start and end cost as much
// as four tiles); 16 of 8192, 64 / 4 heads of 128, bf16, 268 MB: 55 us (4.9 TB/s; two
// groups of 8 heads share a tile's fragments, and the e4m3 form of 128 channels spills
// 60 to 100 bytes of registers); one of 1000 tokens: 8.9 us, of which 4 us pass until
// the first tile has come (length, page table and tile are three trips to memory, one
// after the other).
#include <atomic>
#include <cmath>

#include "attn_paged.h"
#include "tc_sm103.cuh"

namespace attn {
namespace {

constexpr int kPdWarps = 4;  // consumers
constexpr int kPdThreads = 32 * (kPdWarps + 1);
constexpr int kPdRows = 16;  // query heads of an item, at most
// An item's start and end are worth kPdExtra tiles in the shares, where items are
// more than half the CTAs (64 sequences of 8 heads of up to 500 keys 34.3 -> 21.1 us,
// 32 of up to 300 16.8 -> 13.0; with fewer items they cost one sequence of 2000 10.5
// -> 11.0) or shares have kPdShare tiles or more. Up to kPdSolo tiles
// and with more items than CTAs a warp takes a whole item: 128 sequences of up to
// 100 24.3 -> 19.3 us; with 6 tiles instead of 4, 250 of up to 180 33.5 -> 45.5.
constexpr int kPdExtra = 4;
constexpr int kPdShare = 16;
constexpr int kPdSolo = 4;

template <int C, int D, int NT>  // NT: groups of 8 query heads
struct PdCfg {
  static constexpr int ROWS = 8 * NT;
  static constexpr int CB = C == kTypeE4m3 ? 1 : 2;
  static constexpr int ROW = D * CB;                   // bytes of a cached row
  static constexpr int RBX = ROW < 128 ? ROW : 128;    // bytes of a row in one box (the swizzle's span)
  static constexpr int NH = ROW / RBX;
  static constexpr int MINB = NT == 1 && ROW <= 64 ? 3 : 2;  // CTAs per SM
  static constexpr int TK = ROW >= 256 ? 32 : 64;      // keys of a tile
  static constexpr int HALF = TK * ROW;                // K (or V) bytes of a stage
  static constexpr int OTHER = kPdWarps * ROWS * D * 4 + kPdWarps * 2 * ROWS * 4 + 1024;
  static constexpr int RING = 227 * 1024 / MINB - 1024 - OTHER;
  // A multiple of the warps, so that a stage always serves the same warp: loads
  // land out of order, and a warp that looked at a stage whose previous tile,
  // another warp's, had not landed yet would take the phase before for its own.
  static constexpr int STAGES = (RING / (2 * HALF) < 16 ? RING / (2 * HALF) : 16) / kPdWarps * kPdWarps;
  static_assert(STAGES >= kPdWarps && STAGES % kPdWarps == 0, "stages belong to warps");
  static constexpr int SPW = STAGES / kPdWarps;        // stages of a warp
  static constexpr int OFF_O = STAGES * 2 * HALF;      // [warps][ROWS][D] fp32
  static constexpr int OFF_ML = OFF_O + kPdWarps * ROWS * D * 4;  // [warps][2][ROWS]
  static constexpr int OFF_BAR = OFF_ML + kPdWarps * 2 * ROWS * 4;
  static constexpr int OFF_MASK = OFF_BAR + 2 * STAGES * 8;  // visible keys of a stage
  static constexpr int OFF_SCHED = OFF_MASK + STAGES * 8;
  static constexpr int SMEM = OFF_SCHED + 192;
  static_assert(MINB * (SMEM + 1024) <= 228 * 1024, "MINB CTAs fit an SM");
};

struct Part {  // an item that CTA `first` begins and CTA `last` ends
  int b, hr, first, last;
};

// Floats of one partial result: O [rows][D], then m and l [rows] each.
__host__ __device__ constexpr int part_floats(int d, int rows) { return rows * (d + 2); }

// The reference point of the weights 2^(s - m) for a maximum x.  Weights that multiply
// V as fp16 have the largest at 2^15, not 1: then those down to 2^-29 of it are normal
// numbers (10 and more bits) and those down to 2^-40 not nothing.  With the largest at
// 1, keys 2^-25 of it and less were dropped, and with a sink whose value is 0 they are all
// that O consists of.  The factor cancels in O and is part of m in lse.  From 2^20 on m
// stays the maximum itself: there the shift would be rounded, up to an overflow.
template <bool FP16>
__device__ __forceinline__ float weight_origin(float x) {
  if constexpr (FP16) return fabsf(x) < 1048576.f ? x - 15.f : x;
  else return x;
}

// ln of the sum of 2^s for weights that add to l.  The shift is taken out of both
// sides first: log2 of a sum about 1, not 2^15, has the smaller step.
__device__ __forceinline__ float log_sum(float m, float l, bool fp16) {
  if (l == 0.f) return -INFINITY;
  return (fp16 ? (m + 15.f) + log2f(l * 0x1p-15f) : m + log2f(l)) * 0.69314718055994531f;
}

// Weight of a part with maximum m in a join with maximum mm.  Without a maximum
// the part's sums are 0 (no visible key) or NaN (nothing but NaN logits), and
// either goes into the join as it is.
__device__ __forceinline__ float part_weight(float m, float mm) { return m == -INFINITY ? 1.f : ex2_approx(m - mm); }

struct Sched {
  long long w0, total, bound_tile[2];  // share's start and the whole, in weights; tiles before the share's bounds
  int b, hr, tile;  // first tile of the CTA
  int n_act, extra, solo, abort_flag;
  int up[2];  // tiles from a bound of the share to the next item's start
  long long warp_sum[kPdThreads / 32];
  int warp_most[kPdThreads / 32], warp_live[kPdThreads / 32];
};
static_assert(sizeof(Sched) <= 192, "OFF_SCHED");

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Transposes an 8 x 8 matrix of 16-bit elements, two of a row per lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// Barrier over the cluster's threads; what they wrote before it, also to shared
// memory, is visible to all behind it.  `.aligned` wants a warp's lanes together,
// and callers come out of loops and spins that lanes leave apart.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of another CTA's shared memory in the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, int rank) {
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
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ void consumer_sync() {
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kPdWarps) : "memory");
}

template <int TK>
__device__ __forceinline__ int tiles_of(const PagedDecodeArgs& a, int len) {
  if (len <= 0) return 0;
  // A list without repetitions has no more entries than the sequence has pages.
  return ((a.pages ? min(a.n_pages, (len + a.kv.page - 1) / a.kv.page) * a.kv.page : len) + TK - 1) / TK;
}

__device__ __forceinline__ long long divide(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// Finds the CTA's share of the tiles.  All threads; B numbers are read once.
// An item costs its tiles and a start and an end (queries, merge): `extra` tiles'
// worth, laid before its tiles, so that a share of many short items gets fewer.
// Where every item is short and there are many, items are not cut ("solo"): a
// CTA has those that begin in its share, and a warp takes each for itself.
template <int TK>
__device__ __forceinline__ void find_share(const PagedDecodeArgs& a, int HR, Sched& s) {
  const int tid = threadIdx.x, lane = tid & 31, B = a.kv.B;
  const int per = (B + kPdThreads - 1) / kPdThreads;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  long long mine = 0;
  int most = 0, alive = 0;  // longest item, sequences with tokens
  for (int b = b0; b < b1; ++b) {
    const int t = tiles_of<TK>(a, checked_len(a.kv, b));
    mine += t, most = max(most, t), alive += t > 0;
  }
  mine *= HR;
  long long upto = mine;
  int before = alive;  // up to and with this thread's
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, upto, x);
    const int z = __shfl_up_sync(0xffffffffu, before, x);
    if (lane >= x) upto += y, before += z;
    most = max(most, __shfl_xor_sync(0xffffffffu, most, x));
  }
  if (lane == 31) s.warp_sum[tid >> 5] = upto, s.warp_most[tid >> 5] = most, s.warp_live[tid >> 5] = before;
  if (tid == 0) s.b = s.hr = s.tile = 0, s.w0 = 0, s.bound_tile[0] = s.bound_tile[1] = 0, s.up[0] = s.up[1] = 0;
  __syncthreads();
  long long total = 0;
  int live = 0;
  most = 0;
#pragma unroll
  for (int i = 0; i < kPdThreads / 32; ++i) {
    if (i < (tid >> 5)) upto += s.warp_sum[i], before += s.warp_live[i];
    total += s.warp_sum[i];
    most = max(most, s.warp_most[i]), live += s.warp_live[i];
  }
  // Few tiles: a tile per consumer warp, in as many CTAs to every item.
  const long long items = static_cast<long long>(live) * HR;
  const long long want = items ? items * divide(total + items * kPdWarps - 1, items * kPdWarps) : 0;
  const int n_act = static_cast<int>(min(static_cast<long long>(gridDim.x), want));
  const bool solo = most <= kPdSolo && items > gridDim.x;
  const int extra = total >= kPdShare * static_cast<long long>(n_act) || (!solo && 2 * items > gridDim.x) ? kPdExtra : 0;
  total += items * extra;
  mine += static_cast<long long>(alive) * HR * extra;
  upto += static_cast<long long>(before) * HR * extra;
  const int c = blockIdx.x;
  if (tid == 0) s.total = total, s.n_act = n_act, s.extra = extra, s.solo = solo;
  if (c < n_act) {
    const long long bound[2] = {divide(total * c, n_act), divide(total * (c + 1), n_act)};
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const long long w = bound[x];
      if (x == 1 && w == total) {  // the last share ends with all
        if (tid == 0) s.bound_tile[1] = total - items * extra;
        continue;
      }
      if (!(upto - mine <= w && w < upto)) continue;
      long long at = upto - mine, tiles = at - static_cast<long long>(before - alive) * HR * extra;
      for (int b = b0; b < b1; ++b) {
        const int t = tiles_of<TK>(a, checked_len(a.kv, b));
        if (t == 0) continue;
        if (w < at + static_cast<long long>(t + extra) * HR) {
          const int hr = static_cast<int>(divide(w - at, t + extra));
          const int tile = max(0, static_cast<int>(w - at - static_cast<long long>(hr) * (t + extra)) - extra);
          s.up[x] = tile ? t - tile : 0;
          s.bound_tile[x] = tiles + static_cast<long long>(hr) * t + tile;
          if (x == 0) s.b = b, s.hr = hr, s.tile = tile, s.w0 = at + static_cast<long long>(hr) * (t + extra);
          break;
        }
        at += static_cast<long long>(t + extra) * HR;
        tiles += static_cast<long long>(t) * HR;
      }
    }
  }
  __syncthreads();
}

// Position in the list of items.
struct Item {
  int b, hr, tiles, len;
};
template <int TK>
__device__ __forceinline__ void next_item(const PagedDecodeArgs& a, int HR, Item& it) {
  if (++it.hr < HR) return;
  it.hr = 0;
  do {
    if (++it.b >= a.kv.B) {
      it.tiles = 0;
      return;
    }
    it.len = checked_len(a.kv, it.b);
    it.tiles = tiles_of<TK>(a, it.len);
  } while (it.tiles == 0);
}

template <int X>
__device__ __forceinline__ void store_out4(uint8_t* p, const float (&o)[4]) {
  *reinterpret_cast<uint2*>(p) =
      make_uint2(pack2<X == kTypeBf16>(o[0], o[1]), pack2<X == kTypeBf16>(o[2], o[3]));
}

template <int X, int C, int D, int NT>
__global__ void __launch_bounds__(kPdThreads, (PdCfg<C, D, NT>::MINB))
    attn_paged_decode_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                             const PagedDecodeArgs a, int RT, int box_rows, int cluster, int by_item, Part* parts,
                             float* part) {
  using F = PdCfg<C, D, NT>;
  constexpr int TK = F::TK, ROWS = F::ROWS;
  constexpr bool BF = C == kTypeBf16;
  constexpr bool E8 = C == kTypeE4m3;
  extern __shared__ __align__(1024) uint8_t smem[];
  const PagedKv& kv = a.kv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int HR = kv.H * RT, G = a.Hq / kv.H;
  Sched& s = *reinterpret_cast<Sched*>(smem + F::OFF_SCHED);
  const uint32_t sbase = smem_addr(smem);
  const uint32_t full = sbase + F::OFF_BAR, empty = full + F::STAGES * 8;
  uint64_t* masks = reinterpret_cast<uint64_t*>(smem + F::OFF_MASK);
  if (threadIdx.x == 0) {
    for (int i = 0; i < F::STAGES; ++i) {
      mbar_init(full + i * 8, 1);
      mbar_init(empty + i * 8, 1);
    }
    s.abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&mk);
    prefetch_tensormap(&mv);
  }
  griddep_wait();  // launched overlapped (launch_serialized)
  griddep_launch_dependents();
  if (cluster) {
    // An item to each cluster, its tiles in equal runs to the CTAs.
    if (threadIdx.x == 0) {
      const int item = blockIdx.x / cluster, rank = blockIdx.x % cluster;
      s.b = item / HR, s.hr = item % HR;
      const long long t = tiles_of<TK>(a, checked_len(kv, s.b));
      s.bound_tile[0] = s.tile = static_cast<int>(t * rank / cluster), s.bound_tile[1] = t * (rank + 1) / cluster;
      s.w0 = 0, s.total = 1, s.n_act = 1, s.extra = 0, s.solo = 0, s.up[0] = s.up[1] = 0;
    }
    __syncthreads();
  } else {
    find_share<TK>(a, HR, s);
  }
  const bool solo = s.solo;
  // Solo: from the first item that begins here to the end of the last one.
  const int share = static_cast<int>(s.bound_tile[1] - s.bound_tile[0]);
  const int n = solo ? share - s.up[0] + s.up[1] : share;
  const int c = blockIdx.x;

  volatile int* abort_flag = &s.abort_flag;
  Item it = {s.b, s.hr, 0, 0};  // sequence 0 where there is no tile
  it.len = checked_len(kv, it.b);
  it.tiles = tiles_of<TK>(a, it.len);
  int tile = s.tile;
  if (solo && tile) {
    next_item<TK>(a, HR, it);
    tile = 0;
  }

  if (warp == kPdWarps) {  // ---------------------------------- producer warp
    // Each lane looks up one box (box_rows keys of one page) of the next
    // tiles, so one round trip through list and table serves 32 boxes.
    const int nb = TK / box_rows, batch = 32 / nb;  // boxes of a tile, tiles of a batch
    const int box = lane % nb;
    bool ok = true;
    // Tile i goes to warp i % 4, or (solo) the j-th item to warp j % 4; `taken`
    // counts each warp's tiles.
    int w = kPdWarps - 1, taken[kPdWarps] = {};
    for (int i0 = 0; ok && i0 < n; i0 += batch) {
      Item mine = it;
      int t = tile + lane / nb;
      const bool live = i0 + lane / nb < n;
      while (live && mine.tiles > 0 && t >= mine.tiles) {
        t -= mine.tiles;
        next_item<TK>(a, HR, mine);
      }
      int id = -1, h = 0, row = 0, seen = 0;
      if (live) {
        const int key = t * TK + box * box_rows;
        const int e = key / kv.page;
        row = key - e * kv.page;
        h = mine.hr / RT;
        int j = e;
        // Of a list only as many entries as the sequence has pages (tiles_of), also inside the last tile.
        if (a.pages)
          j = e < min(a.n_pages, (mine.len + kv.page - 1) / kv.page)
                  ? a.pages[(static_cast<int64_t>(mine.b) * kv.H + h) * a.n_pages + e]
                  : -1;
        const int64_t left = static_cast<int64_t>(mine.len) - (static_cast<int64_t>(j) * kv.page + row);
        if (j >= 0 && left > 0) {
          seen = static_cast<int>(min(left, static_cast<int64_t>(box_rows)));
          id = checked_page(kv, mine.b, j);
          if (id < 0) seen = 0;
        }
      }
      // A box without a visible key is not loaded: its scores are masked and its
      // V rows zeroed, whatever the stage held before.
      int vis = id >= 0 ? 1 : 0;
      uint64_t mask = (seen == 64 ? ~0ull : ((1ull << seen) - 1)) << (box * box_rows);
      for (int x = 1; x < nb; x <<= 1) {
        mask |= __shfl_xor_sync(0xffffffffu, mask, x);
        vis += __shfl_xor_sync(0xffffffffu, vis, x);
      }
      const uint32_t begin = __ballot_sync(0xffffffffu, t == 0);
      for (int k = 0; k < batch && i0 + k < n; ++k) {
        if (!solo || ((begin >> (k * nb)) & 1)) w = (w + 1) % kPdWarps;
        int turn = 0;  // the warp's tiles so far
#pragma unroll
        for (int x = 0; x < kPdWarps; ++x)
          if (x == w) turn = taken[x]++;
        const int st = w + kPdWarps * (turn % F::SPW);
        if (turn >= F::SPW) ok = mbar_wait(empty + st * 8, (turn / F::SPW - 1) & 1, abort_flag, a.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
#pragma unroll
          for (int x = 0; x < kPdWarps; ++x)
            if (x == w) --taken[x];  // not issued
          break;
        }
        if (lane == k * nb) {
          masks[st] = mask;
          mbar_arrive_expect_tx(full + st * 8, vis * box_rows * F::ROW * 2);
        }
        __syncwarp();
        if (lane / nb == k && id >= 0) {
          const uint32_t dst = sbase + st * 2 * F::HALF + box * box_rows * F::RBX;
#pragma unroll
          for (int hf = 0; hf < F::NH; ++hf) {
            tma_load_4d(dst + hf * TK * F::RBX, &mk, full + st * 8, hf * F::RBX, row, h, id);
            tma_load_4d(dst + F::HALF + hf * TK * F::RBX, &mv, full + st * 8, hf * F::RBX, row, h, id);
          }
        }
      }
      // The batch's end, for all lanes alike.
      tile += batch;
      while (it.tiles > 0 && tile >= it.tiles && i0 + batch < n) {
        tile -= it.tiles;
        next_item<TK>(a, HR, it);
      }
    }
    // No copy may be in flight when the CTA ends, also where the consumers gave
    // up: wait for the last ones here.
#pragma unroll
    for (int x = 0; x < kPdWarps; ++x)
      for (int k = max(0, taken[x] - F::SPW); k < taken[x]; ++k) {
        const uint64_t since = global_timer_ns();
        while (!mbar_test(full + (x + kPdWarps * (k % F::SPW)) * 8, (k / F::SPW) & 1) &&
               global_timer_ns() - since < kWaitLimitNs) {
        }
      }
    if (cluster) {
      cluster_sync();
      cluster_sync();
    }
    return;
  }

  // ------------------------------------------------------------ consumer warps
  // Sequences without tokens: o = 0, lse = -inf; while the first loads travel.
  for (int b = c; b < kv.B && !cluster; b += gridDim.x) {
    if (tiles_of<TK>(a, checked_len(kv, b))) continue;
    for (int i = threadIdx.x; i < a.Hq * D / 8; i += 32 * kPdWarps)
      reinterpret_cast<uint4*>(a.o + static_cast<int64_t>(b) * a.Hq * D * 2)[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int i = threadIdx.x; i < a.Hq; i += 32 * kPdWarps) a.lse[static_cast<int64_t>(b) * a.Hq + i] = -INFINITY;
    if (by_item)
      for (int i = threadIdx.x; i < HR; i += 32 * kPdWarps) parts[b * HR + i] = Part{0, 0, 0, -1};
  }
  if (!by_item && !cluster && threadIdx.x == 0) parts[c] = Part{0, 0, 0, -1};  // the last item may set it below

  // Both products have the cache as the 16-row operand and the query heads as
  // the 8 (NT = 2: 16) columns, so that few heads waste little:
  //   S^T [keys, heads] = K Q^T,  O^T [channels, heads] += V^T P^T.
  // In fragments: key or channel by g = lane / 4, heads 2 t4 and 2 t4 + 1.
  float* so = reinterpret_cast<float*>(smem + F::OFF_O);
  float* sml = reinterpret_cast<float*>(smem + F::OFF_ML);
  const int g = lane >> 2, t4 = lane & 3, l8 = lane & 7, mi = lane >> 3;
  const int swz = F::RBX == 128 ? l8 : F::RBX == 64 ? l8 >> 1 : l8 >> 2;
  constexpr int CPB = F::RBX / 16;  // 16-byte chunks of a box row
  // A weight's first word is rounded from this much of it, so that no rounding reaches
  // the weight itself.
  constexpr float kFirstWord = BF ? 1.f - 0x1p-7f : 1.f - 0x1p-10f;
  bool ok = true;
  int cur = 0, turn = 0;       // tiles of the CTA that are done, and of this warp
  long long w0 = s.w0;         // start of the item, in weights
  for (int item = 0; cur < n && it.tiles > tile; ++item) {
    const int end = min(n, cur + it.tiles - tile);
    // This warp's tiles of the item.
    int tiles = (end - warp + kPdWarps - 1) / kPdWarps - (cur - warp + kPdWarps - 1) / kPdWarps;
    if (solo) {
      tiles = end - cur;
      if (item % kPdWarps != warp) {
        cur = end;
        if (cur < n) next_item<TK>(a, HR, it);
        continue;
      }
    }
    const int h = it.hr / RT, r0 = (it.hr % RT) * ROWS;
    const int rows = min(ROWS, G - r0);
    const int64_t head0 = static_cast<int64_t>(h) * G + r0;
    // The queries as B fragments, head 8 nt + g.  An e4m3 cache is multiplied in
    // fp16: its channels are taken in the order in which four bytes lie in a
    // register, and bf16 queries are scaled by a power of two per head so that
    // the largest lies in [2^8, 2^9) (what then falls below fp16's normal range
    // is 2^-22 of it).
    uint32_t qf[NT][D / 16][2];
    float mul[NT][2];  // of heads 2 t4 and 2 t4 + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint8_t* q = a.q.p + it.b * a.q.row + (head0 + nt * 8 + g) * a.q.head;
      const bool live = nt * 8 + g < rows;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        if constexpr (E8) {
          const uint2 x = live ? *reinterpret_cast<const uint2*>(q + ks * 32 + t4 * 8) : make_uint2(0u, 0u);
          qf[nt][ks][0] = x.x, qf[nt][ks][1] = x.y;
        } else {
          qf[nt][ks][0] = live ? *reinterpret_cast<const uint32_t*>(q + ks * 32 + t4 * 4) : 0u;
          qf[nt][ks][1] = live ? *reinterpret_cast<const uint32_t*>(q + ks * 32 + 16 + t4 * 4) : 0u;
        }
      }
      mul[nt][0] = mul[nt][1] = a.sl2;
      if constexpr (E8 && X == kTypeBf16) {
        float big = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float2 f = unpack2<true>(qf[nt][ks][x]);
            big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        // 2^(8 - e) for a largest value of exponent e, within the normal range; 1 for an infinite one
        const int e = max(20, static_cast<int>(__float_as_uint(big) >> 23));
        const float fac = e == 255 ? 1.f : __uint_as_float(static_cast<uint32_t>(262 - e) << 23);
        const float back = a.sl2 * (e == 255 ? 1.f : __uint_as_float(static_cast<uint32_t>(e - 8) << 23));
        mul[nt][0] = __shfl_sync(0xffffffffu, back, t4 * 8);
        mul[nt][1] = __shfl_sync(0xffffffffu, back, t4 * 8 + 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float2 f = unpack2<true>(qf[nt][ks][x]);
            qf[nt][ks][x] = pack2<false>(f.x * fac, f.y * fac);
          }
      }
    }

    float m[NT][2], l[NT][2];  // maximum (weight_origin of it) and this thread's share of the sum
    float o[NT][D / 16][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY, l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
#pragma unroll
        for (int x = 0; x < D / 16; ++x) o[nt][x][y] = 0.f;
      }
    }

    for (; tiles > 0; --tiles, ++turn) {
      const int st = warp + kPdWarps * (turn % F::SPW);
      if (ok) ok = mbar_wait(full + st * 8, (turn / F::SPW) & 1, abort_flag, a.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) continue;
      const uint64_t mask = masks[st];
      if (mask == 0) {  // nothing to see, nothing was loaded
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + st * 8);
        continue;
      }
      const uint32_t kb = sbase + st * 2 * F::HALF, vb = kb + F::HALF;
      const bool whole = mask == (TK == 64 ? ~0ull : (1ull << (TK & 63)) - 1);
      if (!whole) {
        // Slots behind the sequence's end may hold NaN: their V rows become 0.
        for (int r = lane; r < TK; r += 32)
          if (!((mask >> r) & 1))
            for (int x = 0; x < F::NH; ++x)
#pragma unroll
              for (int y = 0; y < F::RBX; y += 16)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vb + (x * TK + r) * F::RBX + y), "r"(0)
                             : "memory");
        fence_proxy_async_smem();  // before the stage's next load
      }
      __syncwarp();  // the zeros are there, and the lanes together for the matrix steps
      // S^T = K Q^T
      float sc[NT][TK / 16][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < TK / 16; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) sc[nt][x][y] = 0.f;
#pragma unroll
      for (int x = 0; x < TK / 16; ++x) {
        const uint32_t at = kb + (x * 16 + (mi & 1) * 8 + l8) * F::RBX;
        if constexpr (E8) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ks += 2) {
            uint32_t r[4];
            ldsm4(at + (((ks + (mi >> 1)) ^ swz) << 4), r);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t a0 = e4m3_pair(r[2 * y]), a2 = e4m3_pair_hi(r[2 * y]);
              const uint32_t a1 = e4m3_pair(r[2 * y + 1]), a3 = e4m3_pair_hi(r[2 * y + 1]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16<false>(sc[nt][x], a0, a1, a2, a3, qf[nt][ks + y][0], qf[nt][ks + y][1]);
            }
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const int chunk = ks * 2 + (mi >> 1);
            uint32_t r[4];
            ldsm4(at + (chunk / CPB) * TK * F::RBX + (((chunk % CPB) ^ swz) << 4), r);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16<BF>(sc[nt][x], r[0], r[1], r[2], r[3], qf[nt][ks][0], qf[nt][ks][1]);
          }
        }
      }
      // Online softmax, in units of log2.
      uint32_t pf[NT][TK / 16][2], pr[NT][TK / 16][2];  // weights, remainders
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
        for (int x = 0; x < TK / 16; ++x) {
          float(&v)[4] = sc[nt][x];
          v[0] *= mul[nt][0], v[1] *= mul[nt][1], v[2] *= mul[nt][0], v[3] *= mul[nt][1];
          if (!whole) {
            const uint32_t two = static_cast<uint32_t>(mask >> (x * 16 + g));
            if (!(two & 1)) v[0] = v[1] = -INFINITY;
            if (!(two & 256)) v[2] = v[3] = -INFINITY;
          }
          x0 = max3f(x0, v[0], v[2]);
          x1 = max3f(x1, v[1], v[3]);
        }
#pragma unroll
        for (int y = 4; y < 32; y <<= 1) {
          x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, y));
          x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, y));
        }
        const float n0 = fmaxf(m[nt][0], weight_origin<!BF>(x0)), n1 = fmaxf(m[nt][1], weight_origin<!BF>(x1));
        if (__any_sync(0xffffffffu, n0 > m[nt][0] || n1 > m[nt][1])) {  // rare once some tiles are seen
          const float a0 = m[nt][0] == -INFINITY ? 0.f : ex2_approx(m[nt][0] - n0);
          const float a1 = m[nt][1] == -INFINITY ? 0.f : ex2_approx(m[nt][1] - n1);
          m[nt][0] = n0, m[nt][1] = n1;
          l[nt][0] *= a0, l[nt][1] *= a1;
#pragma unroll
          for (int x = 0; x < D / 16; ++x) o[nt][x][0] *= a0, o[nt][x][1] *= a1, o[nt][x][2] *= a0, o[nt][x][3] *= a1;
        }
        // No key yet: weights 0.
        const float z0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], z1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
        for (int x = 0; x < TK / 16; ++x) {
          const float(&v)[4] = sc[nt][x];
          const float p0 = ex2_approx(v[0] - z0), p1 = ex2_approx(v[1] - z1);
          const float p2 = ex2_approx(v[2] - z0), p3 = ex2_approx(v[3] - z1);
          l[nt][0] += p0 + p2;
          l[nt][1] += p1 + p3;
          const uint32_t u = pack2<BF>(p0 * kFirstWord, p1 * kFirstWord), w = pack2<BF>(p2 * kFirstWord, p3 * kFirstWord);
          const float2 uf = unpack2<BF>(u), wf = unpack2<BF>(w);
          pf[nt][x][0] = transpose8(u);
          pf[nt][x][1] = transpose8(w);
          pr[nt][x][0] = transpose8(pack2<BF>(p0 - uf.x, p1 - uf.y));
          pr[nt][x][1] = transpose8(pack2<BF>(p2 - wf.x, p3 - wf.y));
        }
      }
      // O^T += V^T P^T, with every weight as two 16-bit words, a first one a little below
      // it and the remainder: 3 2^-16 (fp16: 3 2^-22) of it is lost at most, against 2^-8
      // (2^-11) in one word, which was an O with up to 1.3 times the error of fp32 weights.
      // Both words are positive where the weight is, or a value of inf would become NaN.
      // The matrix pipe has room for the second product (two sequences of 131071 tokens
      // 155.3 -> 155.2 us, 16 of 16384 in e4m3 94.3 -> 95.3, one of 1000 8.84 -> 8.97).
#pragma unroll
      for (int kk = 0; kk < TK / 16; ++kk) {
        if constexpr (E8) {
          const uint32_t at = vb + (kk * 16 + (mi & 1) * 8 + l8) * F::RBX;
#pragma unroll
          for (int x = 0; x < D / 16; x += 2) {
            uint32_t r[4];
            ldsm4_t(at + (((x + (mi >> 1)) ^ swz) << 4), r);
#pragma unroll
            for (int y = 0; y < 2; ++y) {  // two channels of two keys each: rows g and g + 8 are channels 2 g and 2 g + 1
              const uint32_t lo = __byte_perm(r[2 * y], 0, 0x3120), hi = __byte_perm(r[2 * y + 1], 0, 0x3120);
              const uint32_t a0 = e4m3_pair(lo), a1 = e4m3_pair_hi(lo), a2 = e4m3_pair(hi), a3 = e4m3_pair_hi(hi);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma16<false>(o[nt][x + y], a0, a1, a2, a3, pf[nt][kk][0], pf[nt][kk][1]);
                mma16<false>(o[nt][x + y], a0, a1, a2, a3, pr[nt][kk][0], pr[nt][kk][1]);
              }
            }
          }
        } else {
          const uint32_t at = vb + (kk * 16 + (mi >> 1) * 8 + l8) * F::RBX;
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            const int chunk = 2 * x + (mi & 1);
            uint32_t r[4];
            ldsm4_t(at + (chunk / CPB) * TK * F::RBX + (((chunk % CPB) ^ swz) << 4), r);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16<BF>(o[nt][x], r[0], r[1], r[2], r[3], pf[nt][kk][0], pf[nt][kk][1]);
              mma16<BF>(o[nt][x], r[0], r[1], r[2], r[3], pr[nt][kk][0], pr[nt][kk][1]);
            }
          }
        }
      }
      // The next load writes where these lanes have just read, by another path: only
      // the fence orders it behind the reads.  Without it the last fragments of V were
      // now and then the next tile's (one item of 600 in every fifth call); it costs
      // nothing that can be measured.
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + st * 8);
    }

    // The item's end in this CTA: the four warps are merged (solo: one is all).
    // Columns are swizzled by the head, so that the fragments' stores meet no bank
    // twice.
    float* ml = sml + warp * 2 * ROWS;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int y = 4; y < 32; y <<= 1) {
        l[nt][0] += __shfl_xor_sync(0xffffffffu, l[nt][0], y);
        l[nt][1] += __shfl_xor_sync(0xffffffffu, l[nt][1], y);
      }
      if (g < 2) {
        const int r = nt * 8 + 2 * t4 + g;
        ml[r] = m[nt][g], ml[ROWS + r] = l[nt][g];
      }
      float* w0 = so + (warp * ROWS + nt * 8 + 2 * t4) * D;  // heads 2 t4 and 2 t4 + 1
      const int sw = t4 << 3;
#pragma unroll
      for (int x = 0; x < D / 16; ++x) {
        const float(&v)[4] = o[nt][x];
        if constexpr (E8) {
          const int col = (x * 16 + 2 * g) ^ sw;
          *reinterpret_cast<float2*>(w0 + col) = make_float2(v[0], v[2]);
          *reinterpret_cast<float2*>(w0 + D + col) = make_float2(v[1], v[3]);
        } else {
          const int c0 = (x * 16 + g) ^ sw, c1 = (x * 16 + 8 + g) ^ sw;
          w0[c0] = v[0], w0[D + c0] = v[1], w0[c1] = v[2], w0[D + c1] = v[3];
        }
      }
    }
    if (solo) __syncwarp();
    else consumer_sync();
    const bool begins = tile == 0, ends = end - cur == it.tiles - tile;
    const bool direct = begins && ends && !cluster;
    // In a cluster the partial result stays in shared memory, where the ring was.
    float* out = cluster ? reinterpret_cast<float*>(smem)
                         : part + (static_cast<int64_t>(c) * 2 + (begins ? 1 : 0)) * part_floats(D, ROWS);
    for (int x = solo ? lane : threadIdx.x; x < rows * (D / 4); x += solo ? 32 : 32 * kPdWarps) {
      const int r = x / (D / 4), col = (x % (D / 4)) * 4;
      float mw[kPdWarps], mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kPdWarps; ++w) mm = fmaxf(mm, mw[w] = sml[(solo ? warp : w) * 2 * ROWS + r]);
      float ll = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int x = 0; x < kPdWarps; ++x) {
        if (solo && x) break;
        const int w = solo ? warp : x;
        const float f = part_weight(mw[x], mm);
        ll += f * sml[w * 2 * ROWS + ROWS + r];
        const float4 v = *reinterpret_cast<const float4*>(so + (w * ROWS + r) * D + (col ^ (((r >> 1) & 3) << 3)));
        acc[0] += f * v.x, acc[1] += f * v.y, acc[2] += f * v.z, acc[3] += f * v.w;
      }
      if (direct) {
        const float inv = ll == 0.f ? 0.f : kv.v_scale / ll;
#pragma unroll
        for (int y = 0; y < 4; ++y) acc[y] *= inv;
        const int64_t at = static_cast<int64_t>(it.b) * a.Hq + head0 + r;
        store_out4<X>(a.o + (at * D + col) * 2, acc);
        if (col == 0) a.lse[at] = log_sum(mm, ll, !BF);
      } else {
        *reinterpret_cast<float4*>(out + r * D + col) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        if (col == 0) {
          out[ROWS * D + r] = mm;
          out[ROWS * (D + 1) + r] = ll;
        }
      }
    }
    if (!cluster && !solo && begins && threadIdx.x == 0 && (by_item || !ends)) {
      const long long e = w0 + s.extra + it.tiles;  // CTA c starts at total * c / n_act
      const int last = static_cast<int>(divide(e * s.n_act + s.total - 1, s.total) - 1);
      parts[by_item ? it.b * HR + it.hr : c] = Part{it.b, it.hr, c, ends ? -1 : last};
    }
    if (solo) __syncwarp();  // the area is free for the next item
    else consumer_sync();
    w0 += s.extra + it.tiles;
    cur = end;
    tile = 0;
    if (cur < n) next_item<TK>(a, HR, it);
  }
  if (cluster) {
    // Join of the cluster's partial results, in the order of the CTAs.
    const float* mine = reinterpret_cast<const float*>(smem);
    if (n == 0 && threadIdx.x < ROWS) const_cast<float*>(mine)[ROWS * (D + 1) + threadIdx.x] = 0.f;  // l: nothing seen
    cluster_sync();
    const int h = s.hr / RT, r0 = (s.hr % RT) * ROWS, rows = min(ROWS, G - r0), rank = blockIdx.x % cluster;
    for (int x = rank * 32 * kPdWarps + threadIdx.x; x < rows * (D / 4); x += cluster * 32 * kPdWarps) {
      const int r = x / (D / 4), col = (x % (D / 4)) * 4;
      const uint32_t at = smem_addr(mine);
      float mm = -INFINITY;
      for (int k = 0; k < cluster; ++k) {
        const uint32_t p = in_cta(at, k);
        if (load_cluster4(p + (ROWS * (D + 1) + r) * 4) != 0.f) mm = fmaxf(mm, load_cluster4(p + (ROWS * D + r) * 4));
      }
      float ll = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
      for (int k = 0; k < cluster; ++k) {
        const uint32_t p = in_cta(at, k);
        const float l = load_cluster4(p + (ROWS * (D + 1) + r) * 4);
        if (l == 0.f) continue;
        const float f = part_weight(load_cluster4(p + (ROWS * D + r) * 4), mm);
        const float4 v = load_cluster16(p + (r * D + col) * 4);
        ll += f * l;
        acc[0] += f * v.x, acc[1] += f * v.y, acc[2] += f * v.z, acc[3] += f * v.w;
      }
      const float inv = ll == 0.f ? 0.f : kv.v_scale / ll;
#pragma unroll
      for (int y = 0; y < 4; ++y) acc[y] *= inv;
      const int64_t to = static_cast<int64_t>(s.b) * a.Hq + static_cast<int64_t>(h) * G + r0 + r;
      store_out4<X>(a.o + (to * D + col) * 2, acc);
      if (col == 0) a.lse[to] = log_sum(mm, ll, !BF);
    }
    cluster_sync();  // nobody's shared memory goes before it is read
  }
}

// One block per (cut item, query head): joins the parts in the order of the
// CTAs, so the result does not depend on which finished first.  Every warp
// works out the weights for itself; groups of D / 4 lanes take parts in turn.
constexpr int kMergeThreads = 128;

template <int X, int D>
__global__ void __launch_bounds__(kMergeThreads)
    attn_paged_merge_kernel(const PagedDecodeArgs a, int RT, int ROWS, const Part* parts, const float* part) {
  griddep_wait();  // launched overlapped (launch_serialized)
  griddep_launch_dependents();
  const Part p = parts[blockIdx.x];
  if (p.last < 0) return;
  const int G = a.Hq / a.kv.H, r = blockIdx.y;
  const int r0 = (p.hr % RT) * ROWS;
  if (r >= min(ROWS, G - r0)) return;
  const int n = p.last - p.first + 1, lane = threadIdx.x & 31;
  // CTA `first` has the item's beginning in its slot 1, the others theirs in slot 0.
  const float* base = part + static_cast<int64_t>(p.first) * 2 * part_floats(D, ROWS);
  auto at = [&](int i) { return base + (i ? 2 * i : 1) * part_floats(D, ROWS); };
  float m = -INFINITY;
  for (int i = lane; i < n; i += 32) m = fmaxf(m, at(i)[ROWS * D + r]);
#pragma unroll
  for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  float l = 0.f;
  for (int i = lane; i < n; i += 32) {
    const float* s = at(i) + r;
    const float f = part_weight(s[ROWS * D], m);
    l += f * s[ROWS * (D + 1)];
  }
#pragma unroll
  for (int x = 16; x; x >>= 1) {
    l += __shfl_xor_sync(0xffffffffu, l, x);
  }
  constexpr int LPR = D / 4, GROUPS = kMergeThreads / LPR;
  const int grp = threadIdx.x / LPR, c4 = threadIdx.x % LPR;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = grp; i < n; i += GROUPS) {
    const float4 v = *reinterpret_cast<const float4*>(at(i) + r * D + c4 * 4);
    const float f = part_weight(at(i)[ROWS * D + r], m);
    o.x += f * v.x, o.y += f * v.y, o.z += f * v.z, o.w += f * v.w;
  }
  __shared__ float4 sm[GROUPS][LPR];
  sm[grp][c4] = o;
  __syncthreads();
  const int64_t out = static_cast<int64_t>(p.b) * a.Hq + static_cast<int64_t>(p.hr / RT) * G + r0 + r;
  if (grp == 0) {
#pragma unroll
    for (int i = 1; i < GROUPS; ++i) {
      const float4 v = sm[i][c4];
      o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
    }
    const float inv = l == 0.f ? 0.f : a.kv.v_scale / l;
    const float w[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
    store_out4<X>(a.o + (out * D + c4 * 4) * 2, w);
  }
  if (threadIdx.x == 0) a.lse[out] = log_sum(m, l, a.kv.type != kTypeBf16);
}

// The same for items cut into many parts: a block to every 32 columns, whose
// threads share the parts' statistics.
constexpr int kManyThreads = 512;
constexpr int kMergeParts = 1024;  // at most, one to a CTA

template <int X, int D>
__global__ void __launch_bounds__(kManyThreads)
    attn_paged_merge_many_kernel(const PagedDecodeArgs a, int RT, int ROWS, const Part* parts, const float* part) {
  griddep_wait();  // launched overlapped (launch_serialized)
  griddep_launch_dependents();
  const Part p = parts[blockIdx.x];
  if (p.last < 0) return;
  const int G = a.Hq / a.kv.H, r = blockIdx.y;
  const int r0 = (p.hr % RT) * ROWS;
  if (r >= min(ROWS, G - r0)) return;
  constexpr int T = kManyThreads, warps = T / 32;
  const int n = p.last - p.first + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // CTA `first` has the item's beginning in its slot 1, the others theirs in slot 0.
  const float* base = part + static_cast<int64_t>(p.first) * 2 * part_floats(D, ROWS);
  auto at = [&](int i) { return base + (i ? 2 * i : 1) * part_floats(D, ROWS); };
  __shared__ float weight[kMergeParts], sums[2][kManyThreads / 32];
  __shared__ float4 sm[kManyThreads];
  float m = -INFINITY;
  for (int i = threadIdx.x; i < n; i += T) m = fmaxf(m, at(i)[ROWS * D + r]);
#pragma unroll
  for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  if (lane == 0) sums[0][warp] = m;
  __syncthreads();
  for (int i = 0; i < warps; ++i) m = fmaxf(m, sums[0][i]);
  float l = 0.f;
  for (int i = threadIdx.x; i < n; i += T) {
    const float* s = at(i) + r;
    const float f = part_weight(s[ROWS * D], m);
    weight[i] = f;
    l += f * s[ROWS * (D + 1)];
  }
#pragma unroll
  for (int x = 16; x; x >>= 1) {
    l += __shfl_xor_sync(0xffffffffu, l, x);
  }
  if (lane == 0) sums[1][warp] = l;
  __syncthreads();
  l = 0.f;
  for (int i = 0; i < warps; ++i) l += sums[1][i];
  constexpr int LPR = 8, GROUPS = T / LPR;  // eight lanes take a part's 32 columns
  const int grp = threadIdx.x / LPR, c = blockIdx.z * 32 + (threadIdx.x % LPR) * 4;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = grp; i < n; i += GROUPS) {
    const float4 v = *reinterpret_cast<const float4*>(at(i) + r * D + c);
    const float f = weight[i];
    o.x += f * v.x, o.y += f * v.y, o.z += f * v.z, o.w += f * v.w;
  }
  sm[threadIdx.x] = o;
  __syncthreads();
  const int64_t out = static_cast<int64_t>(p.b) * a.Hq + static_cast<int64_t>(p.hr / RT) * G + r0 + r;
  if (grp == 0) {
    for (int i = 1; i < min(GROUPS, n); ++i) {
      const float4 v = sm[threadIdx.x + i * LPR];
      o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
    }
    const float inv = l == 0.f ? 0.f : a.kv.v_scale / l;
    const float w[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
    store_out4<X>(a.o + (out * D + c) * 2, w);
  }
  if (threadIdx.x == 0 && blockIdx.z == 0) a.lse[out] = log_sum(m, l, a.kv.type != kTypeBf16);
}

constexpr int kMaxCtas = kMergeParts;  // of the decode kernel

// CTAs that find a tile for each of their warps, if every sequence fills its table.
int64_t most_ctas(int64_t items, int64_t keys, int tk) { return items * (((keys + tk - 1) / tk + kPdWarps - 1) / kPdWarps); }

int row_tiles(int Hq, int H) { return (Hq / H + kPdRows - 1) / kPdRows; }

// CTAs of a cluster for short items, or 0: the join through shared memory saves
// the partial results' way through L2 and the merge kernel (one sequence of 1000
// 10.2 -> 8.7 us, 16 of up to 200 16.4 -> 8.4).  A warp has one tile, or two where
// the clusters have more CTAs than the GPU has SMs (else cutting the items finer is
// faster: one sequence of 2000 10.5 against 10.3 us).  The clusters may be twice
// what is resident at once (64 sequences of up to 100 13.6 against 16.6 us; four
// times: 32 of up to 300 25.6 against 13.0), unless most warps would have nothing
// to do (64 of up to 20 12.6 against 10.9).
int cluster_size(int64_t items, int64_t tiles, int sms) {
  for (int k = 1; k <= 8; k *= 2)
    if (k * kPdWarps >= tiles || (k == 8 && 2 * k * kPdWarps >= tiles && items * k > sms))
      return items * k <= (2 * tiles > kPdWarps ? 4 : 2) * sms ? k : 0;
  return 0;
}

template <typename Kernel>
cudaError_t launch_clusters(Kernel kern, int ctas, int cluster, size_t smem, cudaStream_t stream, const CUtensorMap& mk,
                            const CUtensorMap& mv, const PagedDecodeArgs& a, int RT, int box, int size) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kPdThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, mk, mv, a, RT, box, size, 0, static_cast<Part*>(nullptr), static_cast<float*>(nullptr));
}

template <int X, int C, int D, int NT>
int launch_t(const PagedDecodeArgs& a, int* launches) {
  using F = PdCfg<C, D, NT>;
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is raised
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return kStatusCuda;
  auto kern = attn_paged_decode_kernel<X, C, D, NT>;
  if (!((ready.load() >> dev) & 1)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, F::SMEM) != cudaSuccess) return kStatusCuda;
    ready.fetch_or(1ull << dev);
  }
  const int RT = row_tiles(a.Hq, a.kv.H);
  int box = 8;
  while (box < F::TK && a.kv.page % (2 * box) == 0) box *= 2;
  CUtensorMap mk, mv;
  if (!encode_pages_map(&mk, a.kv.k, F::ROW, a.kv.page, a.kv.H, a.kv.num_pages, a.kv.k_tok, a.kv.k_head, a.kv.k_page, F::RBX,
                        box) ||
      !encode_pages_map(&mv, a.kv.v, F::ROW, a.kv.page, a.kv.H, a.kv.num_pages, a.kv.v_tok, a.kv.v_head, a.kv.v_page, F::RBX,
                        box))
    return kStatusCuda;
  const int sms = device_sm_count();
  if (sms < 1) return kStatusCuda;
  const int64_t keys = static_cast<int64_t>(a.pages ? a.n_pages : a.kv.max_pages) * a.kv.page;
  const int64_t items = static_cast<int64_t>(a.kv.B) * a.kv.H * RT;
  const int cluster = cluster_size(items, (keys + F::TK - 1) / F::TK, sms);
  if (cluster) {
    *launches = 1;
    return launch_clusters(kern, static_cast<int>(items) * cluster, cluster, F::SMEM, a.stream, mk, mv, a, RT, box, cluster) ==
                   cudaSuccess
               ? kStatusOk
               : kStatusCuda;
  }
  const int ctas = static_cast<int>(std::min<int64_t>(std::min(F::MINB * sms, kMaxCtas), most_ctas(items, keys, F::TK)));
  const int by_item = items <= ctas;
  Part* parts = reinterpret_cast<Part*>(a.ws);
  float* part = reinterpret_cast<float*>(a.ws + kMaxCtas * sizeof(Part));
  // Overlapped with the kernel before where every CTA finds room beside that
  // one's last blocks: two per SM.  Of three per SM some did not, and started not
  // when those blocks ended but when a CTA of their own kernel did (e4m3 heads 119
  // against 97 us); for the others it saves up to 1 us.
  if (launch_serialized(ctas <= 2 * sms, kern, dim3(ctas), dim3(kPdThreads), F::SMEM, a.stream, mk, mv, a, RT, box, 0, by_item, parts,
                        part) != cudaSuccess)
    return kStatusCuda;
  // The wide form is faster from about 32 parts on (one sequence of 131071 and one KV
  // head, 304 parts: 36 -> 22 us; eight heads of 16000, 38 parts: 22.0 -> 20.1; of
  // 2000, 16 parts: 10.5 -> 11.0).
  const bool many = items * 32 <= ctas;
  const dim3 grid(by_item ? static_cast<int>(items) : ctas, std::min(F::ROWS, a.Hq / a.kv.H), many ? D / 32 : 1);
  return launch_serialized(true, many ? attn_paged_merge_many_kernel<X, D> : attn_paged_merge_kernel<X, D>, grid,
                           dim3(many ? kManyThreads : kMergeThreads), 0, a.stream, a, RT, F::ROWS, parts, part) == cudaSuccess
             ? kStatusOk
             : kStatusCuda;
}

template <int X, int C>
int launch_d(const PagedDecodeArgs& a, int* launches) {
  const bool wide = a.Hq / a.kv.H > 8;
  switch (a.kv.d) {
    case 32: return wide ? launch_t<X, C, 32, 2>(a, launches) : launch_t<X, C, 32, 1>(a, launches);
    case 64: return wide ? launch_t<X, C, 64, 2>(a, launches) : launch_t<X, C, 64, 1>(a, launches);
    default: return wide ? launch_t<X, C, 128, 2>(a, launches) : launch_t<X, C, 128, 1>(a, launches);
  }
}

}  // namespace

int64_t paged_decode_workspace(int B, int Hq, int H, int d, int page, int n_pages) {
  // Two partial results for each CTA, as many as the largest GPU of the family
  // could hold; a bound by the tiles keeps it small for small problems.
  const int64_t items = static_cast<int64_t>(B) * H * row_tiles(Hq, H);
  const int64_t ctas = std::min<int64_t>(kMaxCtas, most_ctas(items, static_cast<int64_t>(n_pages) * page, 32));
  return kMaxCtas * static_cast<int64_t>(sizeof(Part)) + ctas * 2 * part_floats(d, kPdRows) * 4;
}

int launch_paged_decode(const PagedDecodeArgs& a, int* launches) {
  *launches = 2;
  if (a.x_type == kTypeBf16)
    return a.kv.type == kTypeE4m3 ? launch_d<kTypeBf16, kTypeE4m3>(a, launches) : launch_d<kTypeBf16, kTypeBf16>(a, launches);
  return a.kv.type == kTypeE4m3 ? launch_d<kTypeF16, kTypeE4m3>(a, launches) : launch_d<kTypeF16, kTypeF16>(a, launches);
}

}  // namespace attn
