// attn_paged_assign.cu -- a serving step's bookkeeping on the device: from the
// new tokens of each sequence the pages that they need, the block table's new
// entries, the lengths, the packed rows' starts and a slot for every new token.
//
// With L_b tokens held, n_b new ones and pages of P slots, sequence b needs the
// pages ceil(L_b / P) .. ceil((L_b + n_b) / P) - 1.  Page j of a windowed
// sequence from j = first + turns on is page j - turns again (`first` pages of
// sinks, `turns` that the window needs): its keys have left the window.  The
// other new pages come from a ring of free ones in the order of the sequences,
// so a prefix sum over the counts says which; sequences that have ended put
// theirs behind the ring's last.  The step is done whole or not at all, so the
// sums are taken before anything is written.
//
//   attn_paged_plan_kernel : one block; checks, the three prefix sums (tokens,
//       pages taken, pages handed back), lengths and starts.  With ALL, for a step of
//       few tokens, it does the second kernel's work too, its sums in shared memory.
//   attn_paged_fill_kernel : a warp to 128 rows of new tokens, four to a thread: the
//       token's sequence, searched for between those of the warp's first and last
//       row, its slot, and the table entry where it is a page's first; then the pages
//       of ended sequences.
//
// Few bytes and no arithmetic to speak of.  A step of 64 sequences, 4.6 us a call, is a
// launch and a handful of dependent loads in the one block.  One of 4096 with 962000 new
// tokens takes 20.5 (plan 10, fill 12; its 8.4 MB would take 1.3): the sums are one
// block's, in four rounds, and the fill searches, looks up and stores for each token (issue
// active 56 %).  What counted (33 -> 20.5): one round of sums, taken back if a check
// fails, instead of one round of checks and another of sums; a thread's rows in
// flight together; divisions by the page size as products.
#include "attn_paged.h"
#include "tc_sm103.cuh"

namespace attn {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kRows = 4;  // rows of a thread of the fill, 32 apart

// What the plan leaves for the fill: a header, then an item per sequence.
struct Plan {
  int head, behind;  // ring positions: the first free page, and the one behind the last
  int tokens;        // new rows
  int done;          // 0: the step was refused
};
struct PlanItem {
  int old, n, take, back;  // tokens held, new ones (-1: ended); pages taken and handed back before this sequence
};

// floor(x / page) for 0 <= x < 2^31 (Granlund, Montgomery, "Division by Invariant
// Integers using Multiplication", 1994: with l = ceil(log2 d) and m = floor(2^32
// (2^l - d) / d) + 1 the quotient is (hi(m x) + x) >> l).
__device__ __forceinline__ int page_of(const PagedAssignArgs& a, int x) {
  return static_cast<int>((__umulhi(a.page_mul, static_cast<uint32_t>(x)) + static_cast<uint32_t>(x)) >> a.page_shift);
}
__device__ __forceinline__ int pages_for(const PagedAssignArgs& a, int tokens) { return page_of(a, tokens + a.kv.page - 1); }

// Pages of its own that a sequence of `pages` pages holds.
__device__ __forceinline__ int held_pages(const PagedAssignArgs& a, int pages) {
  return a.turns ? min(pages, a.first + a.turns) : pages;
}

// Position i < 2 free_cap of the ring.
__device__ __forceinline__ int ring_at(const PagedAssignArgs& a, int64_t i) { return static_cast<int>(i < a.free_cap ? i : i - a.free_cap); }

// The sequence of row r < start[B], by a whole warp: 32 probes at a time.
__device__ __forceinline__ int sequence_of(const int* start, int B, int r, int lane) {
  int lo = 0, n = B;  // start[lo] <= r < start[lo + n]
  while (n > 1) {
    const int step = (n + 31) >> 5, at = lo + lane * step;
    const bool below = lane * step < n && start[at] <= r;
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, below));  // lane 0's holds
    const int left = n - last * step;
    lo += last * step;
    n = min(step, left);
  }
  return lo;
}

// The work of warp `w` of `warps`: runs of rows, and sequences that are over.
template <int ROWS>
__device__ __forceinline__ void fill(const PagedAssignArgs& a, const Plan& p, const PlanItem* items, const int* start, int w, int warps, int lane) {
  const int page = a.kv.page, B = a.kv.B;
  for (int r0 = w * 32 * ROWS; r0 < a.rows; r0 += warps * 32 * ROWS) {
    int first = 0, last = 0;
    if (r0 < p.tokens) {
      first = sequence_of(start, B, r0, lane);
      last = sequence_of(start, B, min(r0 + 32 * ROWS, p.tokens) - 1, lane);
    }
    // Each step for all of the thread's rows before the next: their loads travel together.
    int lo[ROWS], hi[ROWS], id[ROWS];  // start[lo] <= r < start[hi]
#pragma unroll
    for (int x = 0; x < ROWS; ++x) lo[x] = first, hi[x] = last + 1;
    for (int n = last - first; n > 0; n >>= 1)
#pragma unroll
      for (int x = 0; x < ROWS; ++x) {
        const int mid = (lo[x] + hi[x]) >> 1;
        if (mid == lo[x]) continue;
        if (start[mid] <= r0 + x * 32 + lane) lo[x] = mid;
        else hi[x] = mid;
      }
    int page_no[ROWS], slot[ROWS];
#pragma unroll
    for (int x = 0; x < ROWS; ++x) {
      const int r = r0 + x * 32 + lane;
      id[x] = -1, page_no[x] = 0, slot[x] = 1;
      if (r >= p.tokens) continue;
      const PlanItem it = items[lo[x]];
      const int pos = it.old + r - start[lo[x]];
      const int j = page_of(a, pos);
      page_no[x] = j, slot[x] = pos - j * page;
      if (slot[x] && !a.slots) continue;
      const int root = a.turns && j >= a.first + a.turns ? a.first + (j - a.first) % a.turns : j;
      const int had = pages_for(a, it.old);
      id[x] = root >= had ? a.free_pages[ring_at(a, static_cast<int64_t>(p.head) + it.take + root - had)] : a.table[lo[x] * a.kv.table_stride + root];
    }
#pragma unroll
    for (int x = 0; x < ROWS; ++x) {
      const int r = r0 + x * 32 + lane;
      if (r >= a.rows) break;
      if (r < p.tokens && (a.slots || slot[x] == 0)) {
        if (id[x] < 0 || id[x] >= a.kv.num_pages) {
          record_check(a.kv.check);
          id[x] = -1;
        }
        if (slot[x] == 0) a.table[lo[x] * a.kv.table_stride + page_no[x]] = id[x];
      }
      if (a.slots) a.slots[r] = id[x] < 0 ? -1 : static_cast<int64_t>(id[x]) * page + slot[x];
    }
  }
  if (!p.done) return;
  for (int b = w; b < B; b += warps) {
    const PlanItem it = items[b];
    if (it.n >= 0) continue;
    const int n = held_pages(a, pages_for(a, it.old));
    const int* row = a.table + b * a.kv.table_stride;
    for (int i = lane; i < n; i += 32) {
      int id = row[i];
      if (id < 0 || id >= a.kv.num_pages) {
        record_check(a.kv.check);
        id = -1;
      }
      a.free_pages[ring_at(a, static_cast<int64_t>(p.behind) + it.back + i)] = id;
    }
  }
}

// Sums stop at kMany, which is more than any sum that a step may have: exact below
// it, and a step with one that is not is refused, so that 32 bits do.
constexpr uint32_t kMany = (1u << 30) + 1;
__device__ __forceinline__ uint32_t plus(uint32_t x, uint32_t y) { return min(x + y, kMany); }
struct Counts {
  uint32_t tokens, take, back;
  __device__ __forceinline__ Counts operator+(const Counts& o) const { return {plus(tokens, o.tokens), plus(take, o.take), plus(back, o.back)}; }
};

// Sum over the warp's lanes up to this one.
__device__ __forceinline__ Counts lanes_upto(Counts c, int lane) {
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const Counts y = {__shfl_up_sync(0xffffffffu, c.tokens, x), __shfl_up_sync(0xffffffffu, c.take, x), __shfl_up_sync(0xffffffffu, c.back, x)};
    if (lane >= x) c = c + y;
  }
  return c;
}
__device__ __forceinline__ Counts of_lane(const Counts& c, int lane) {
  return {__shfl_sync(0xffffffffu, c.tokens, lane), __shfl_sync(0xffffffffu, c.take, lane), __shfl_sync(0xffffffffu, c.back, lane)};
}

// What a sequence adds to the sums.
__device__ __forceinline__ Counts counts_of(const PagedAssignArgs& a, int old, int n) {
  const uint32_t had = held_pages(a, pages_for(a, old));
  return {static_cast<uint32_t>(max(n, 0)), n > 0 ? held_pages(a, pages_for(a, old + n)) - had : 0u, n < 0 ? had : 0u};
}

template <bool ALL>
__global__ void __launch_bounds__(kPlanThreads) attn_paged_plan_kernel(const PagedAssignArgs a) {
  griddep_wait();  // launched overlapped (launch_serialized)
  griddep_launch_dependents();
  constexpr int kWarps = kPlanThreads / 32;
  __shared__ Counts sums[2][kWarps];
  __shared__ int bad;
  __shared__ PlanItem s_items[ALL ? kPlanThreads : 1];
  __shared__ int s_start[ALL ? kPlanThreads + 1 : 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5, B = a.kv.B;
  const int64_t most = static_cast<int64_t>(a.kv.max_pages) * a.kv.page, most_new = a.turns ? static_cast<int64_t>(a.turns) * a.kv.page : most;
  if (tid == 0) bad = 0;
  const int head = a.free_state[0], count = a.free_state[1];
  bool wrong = head < 0 || head >= a.free_cap || count < 0 || count > a.free_cap;
  // A sequence to a thread, in rounds.  What is written holds if the step is done; if
  // not, it is taken back below.
  PlanItem* items = ALL ? s_items : reinterpret_cast<PlanItem*>(a.ws + sizeof(Plan));
  Counts total = {0, 0, 0};
  for (int b0 = 0, turn = 0; b0 < B; b0 += blockDim.x, turn ^= 1) {
    const int b = b0 + tid, old = b < B ? a.lens[b] : 0, n = b < B ? a.n_new[b] : 0;
    const bool fits = old >= 0 && old <= most && n >= -1 && static_cast<int64_t>(old) + n <= most && n <= most_new;
    if (!fits) wrong = true;
    const Counts mine = fits ? counts_of(a, old, n) : Counts{0, 0, 0};
    const Counts upto = lanes_upto(mine, lane);
    if (lane == 31) sums[turn][warp] = upto;
    __syncthreads();
    const Counts of_warps = lanes_upto(lane < warps ? sums[turn][lane] : Counts{0, 0, 0}, lane);
    Counts at = total + Counts{upto.tokens - mine.tokens, upto.take - mine.take, upto.back - mine.back};  // exact if the whole is
    if (warp > 0) at = at + of_lane(of_warps, warp - 1);
    if (b < B) {
      items[b] = PlanItem{old, n, static_cast<int>(at.take), static_cast<int>(at.back)};
      a.token_start[b] = at.tokens;
      a.lens_out[b] = n < 0 || !fits ? 0 : old + n;
      if (ALL) s_start[b] = at.tokens;
    }
    total = total + of_lane(of_warps, 31);
  }
  if (wrong) bad = 1;
  __syncthreads();
  // Pages that come back must not come to lie on free ones that this step takes.
  const bool ok = !bad && total.tokens <= static_cast<uint32_t>(a.rows) && total.take <= static_cast<uint32_t>(count) &&
                  count + total.back <= static_cast<uint32_t>(a.free_cap);
  if (!ok)
    for (int b = tid; b < B; b += blockDim.x) {
      a.token_start[b] = 0;
      a.lens_out[b] = items[b].old;
    }
  const Plan plan = {head, ok ? ring_at(a, static_cast<int64_t>(head) + count) : 0, ok ? static_cast<int>(total.tokens) : 0, ok};
  if (tid == 0) {
    a.token_start[B] = plan.tokens;
    a.free_out[0] = ok ? ring_at(a, static_cast<int64_t>(head) + total.take) : head;
    a.free_out[1] = ok ? static_cast<int>(count - total.take + total.back) : count;
    if (!ALL) *reinterpret_cast<Plan*>(a.ws) = plan;
    if (!ok) record_check(a.kv.check);
  }
  if constexpr (ALL) {
    __syncthreads();
    fill<1>(a, plan, s_items, s_start, warp, warps, lane);
  }
}

__global__ void __launch_bounds__(kFillThreads) attn_paged_fill_kernel(const PagedAssignArgs a) {
  griddep_wait();  // launched overlapped (launch_serialized)
  griddep_launch_dependents();
  const Plan plan = *reinterpret_cast<const Plan*>(a.ws);
  fill<kRows>(a, plan, reinterpret_cast<const PlanItem*>(a.ws + sizeof(Plan)), a.token_start, (blockIdx.x * kFillThreads + threadIdx.x) >> 5,
       gridDim.x * (kFillThreads / 32), threadIdx.x & 31);
}

}  // namespace

int64_t paged_assign_workspace(int B) { return static_cast<int64_t>(sizeof(Plan)) + static_cast<int64_t>(B) * sizeof(PlanItem); }

int launch_paged_assign(const PagedAssignArgs& args, int* launches) {
  PagedAssignArgs a = args;
  a.page_shift = 0;
  while ((1 << a.page_shift) < a.kv.page) ++a.page_shift;
  a.page_mul = static_cast<uint32_t>((((uint64_t{1} << 32) * ((uint64_t{1} << a.page_shift) - a.kv.page)) / a.kv.page) + 1);
  // One block does all where a second kernel would have little to do.
  const bool all = a.kv.B <= kPlanThreads && a.rows <= 4 * kPlanThreads;
  *launches = all ? 1 : 2;
  const int64_t need = all ? std::max(a.kv.B, a.rows) : a.kv.B;
  const int threads = static_cast<int>(std::min<int64_t>(kPlanThreads, (std::max<int64_t>(need, 128) + 31) / 32 * 32));
  if (launch_serialized(true, all ? attn_paged_plan_kernel<true> : attn_paged_plan_kernel<false>, dim3(1), dim3(threads), 0, a.stream, a) !=
      cudaSuccess)
    return kStatusCuda;
  if (all) return kStatusOk;
  const int sms = device_sm_count();
  if (sms < 1) return kStatusCuda;
  const int64_t warps = std::max((a.rows + 32 * kRows - 1) / (32 * kRows), a.kv.B);
  const int blocks = static_cast<int>(std::min<int64_t>((warps * 32 + kFillThreads - 1) / kFillThreads, 16 * sms));
  return launch_serialized(true, attn_paged_fill_kernel, dim3(blocks), dim3(kFillThreads), 0, a.stream, a) == cudaSuccess ? kStatusOk
                                                                                                                      : kStatusCuda;
}

}  // namespace attn
