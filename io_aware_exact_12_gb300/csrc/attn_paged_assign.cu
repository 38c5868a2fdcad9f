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
// theirs behind the ring's last.  The step is done whole or not at all.
//
//   attn_paged_plan_kernel : one block; checks, the three prefix sums (tokens,
//       pages taken, pages handed back), lengths and starts.  With `all` it does
//       the second kernel's work too.
//   attn_paged_fill_kernel : a thread to every new token: its sequence by
//       bisection of the starts, its slot, and the table entry where it is a
//       page's first; then the pages of ended sequences.
#include "attn_paged.h"
#include "tc_sm103.cuh"

namespace attn {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kFillThreads = 256;

// What the plan leaves for the fill: a header, then one word per sequence.
struct Plan {
  int head, behind;  // ring positions: the first free page, and the one behind the last
  int tokens;        // new rows
  int done;          // 0: the step was refused
};
struct PlanItem {
  int old, n, take, back;  // tokens held, new ones (-1: ended); pages taken and handed back before this sequence
};

__device__ __forceinline__ int pages_for(int tokens, int page) { return static_cast<int>((static_cast<int64_t>(tokens) + page - 1) / page); }

// Pages of its own that a sequence of `pages` pages holds.
__device__ __forceinline__ int held_pages(const PagedAssignArgs& a, int pages) {
  return a.turns ? min(pages, a.first + a.turns) : pages;
}

__device__ __forceinline__ int ring_at(const PagedAssignArgs& a, int64_t i) { return static_cast<int>(i % a.free_cap); }

// Rows `from`, from + step, ..., and the sequences likewise.
__device__ void fill(const PagedAssignArgs& a, int from, int step) {
  const Plan p = *reinterpret_cast<const Plan*>(a.ws);
  const PlanItem* items = reinterpret_cast<const PlanItem*>(a.ws + sizeof(Plan));
  const int page = a.kv.page, B = a.kv.B;
  for (int64_t r = from; r < a.rows; r += step) {
    if (r >= p.tokens) {
      if (a.slots) a.slots[r] = -1;
      continue;
    }
    int lo = 0, hi = B;  // start[lo] <= r < start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.token_start[mid] <= r) lo = mid;
      else hi = mid;
    }
    const PlanItem it = items[lo];
    const int pos = it.old + static_cast<int>(r - a.token_start[lo]);
    const int j = pos / page, slot = pos - j * page;
    const bool opens = slot == 0;
    if (!opens && !a.slots) continue;
    const int root = a.turns && j >= a.first + a.turns ? a.first + (j - a.first) % a.turns : j;
    const int had = pages_for(it.old, page);
    int* row = a.table + lo * a.kv.table_stride;
    int id = root >= had ? a.free_pages[ring_at(a, static_cast<int64_t>(p.head) + it.take + root - had)] : row[root];
    if (id < 0 || id >= a.kv.num_pages) {
      record_check(a.kv.check);
      id = -1;
    }
    if (opens) row[j] = id;
    if (a.slots) a.slots[r] = id < 0 ? -1 : static_cast<int64_t>(id) * page + slot;
  }
  if (!p.done) return;
  for (int b = from >> 5; b < B; b += step >> 5) {  // a warp to a sequence
    const PlanItem it = items[b];
    if (it.n >= 0) continue;
    const int n = held_pages(a, pages_for(it.old, page));
    const int* row = a.table + b * a.kv.table_stride;
    for (int i = threadIdx.x & 31; i < n; i += 32) {
      int id = row[i];
      if (id < 0 || id >= a.kv.num_pages) {
        record_check(a.kv.check);
        id = -1;
      }
      a.free_pages[ring_at(a, static_cast<int64_t>(p.behind) + it.back + i)] = id;
    }
  }
}

__global__ void __launch_bounds__(kPlanThreads) attn_paged_plan_kernel(const PagedAssignArgs a, int all) {
  griddep_wait();  // launched overlapped (launch_serialized)
  griddep_launch_dependents();
  __shared__ long long sums[3][kPlanThreads / 32];
  __shared__ int bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = a.kv.B, page = a.kv.page;
  const int64_t most = static_cast<int64_t>(a.kv.max_pages) * page;
  const int per = (B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  if (tid == 0) bad = 0;
  __syncthreads();
  const int head = a.free_state[0], count = a.free_state[1];
  long long mine[3] = {0, 0, 0};  // tokens, pages taken, pages handed back
  bool wrong = head < 0 || head >= a.free_cap || count < 0 || count > a.free_cap;
  // What a sequence adds to the three sums.
  auto adds = [&](int old, int n, int& take, int& back) {
    const int had = held_pages(a, pages_for(old, page));
    take = n > 0 ? held_pages(a, pages_for(old + n, page)) - had : 0;
    back = n < 0 ? had : 0;
  };
  for (int b = b0; b < b1; ++b) {
    const int old = a.lens[b], n = a.n_new[b];
    if (old < 0 || old > most || n < -1 || static_cast<int64_t>(old) + n > most || (a.turns && n > static_cast<int64_t>(a.turns) * page)) {
      wrong = true;
      break;
    }
    int take, back;
    adds(old, n, take, back);
    mine[0] += max(n, 0), mine[1] += take, mine[2] += back;
  }
  if (wrong) bad = 1;
  long long upto[3] = {mine[0], mine[1], mine[2]};
#pragma unroll
  for (int x = 1; x < 32; x <<= 1)
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const long long y = __shfl_up_sync(0xffffffffu, upto[k], x);
      if (lane >= x) upto[k] += y;
    }
  if (lane == 31)
    for (int k = 0; k < 3; ++k) sums[k][warp] = upto[k];
  __syncthreads();
  long long total[3] = {0, 0, 0};
  for (int i = 0; i < kPlanThreads / 32; ++i)
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if (i < warp) upto[k] += sums[k][i];
      total[k] += sums[k][i];
    }
  // Handed back pages must not come to lie on free ones that this step takes.
  const bool ok = !bad && total[0] <= a.rows && total[1] <= count && count + total[2] <= a.free_cap;
  PlanItem* items = reinterpret_cast<PlanItem*>(a.ws + sizeof(Plan));
  int start = static_cast<int>(ok ? upto[0] - mine[0] : 0), take0 = static_cast<int>(upto[1] - mine[1]), back0 = static_cast<int>(upto[2] - mine[2]);
  for (int b = b0; b < b1; ++b) {
    const int old = a.lens[b], n = ok ? a.n_new[b] : 0;
    items[b] = PlanItem{old, n, take0, back0};
    a.token_start[b] = start;
    a.lens_out[b] = n < 0 ? 0 : old + n;
    if (!ok) continue;
    int take, back;
    adds(old, n, take, back);
    start += max(n, 0), take0 += take, back0 += back;
  }
  if (tid == 0) {
    a.token_start[B] = ok ? static_cast<int>(total[0]) : 0;
    *reinterpret_cast<Plan*>(a.ws) = Plan{ok ? head : 0, ok ? ring_at(a, static_cast<int64_t>(head) + count) : 0, ok ? static_cast<int>(total[0]) : 0, ok};
    a.free_out[0] = ok ? ring_at(a, head + total[1]) : head;
    a.free_out[1] = ok ? static_cast<int>(count - total[1] + total[2]) : count;
    if (!ok) record_check(a.kv.check);
  }
  if (!all) return;
  __syncthreads();
  fill(a, tid, kPlanThreads);
}

__global__ void __launch_bounds__(kFillThreads) attn_paged_fill_kernel(const PagedAssignArgs a) {
  griddep_wait();  // launched overlapped (launch_serialized)
  griddep_launch_dependents();
  fill(a, blockIdx.x * kFillThreads + threadIdx.x, gridDim.x * kFillThreads);
}

}  // namespace

int64_t paged_assign_workspace(int B) { return static_cast<int64_t>(sizeof(Plan)) + static_cast<int64_t>(B) * sizeof(PlanItem); }

int launch_paged_assign(const PagedAssignArgs& a, int* launches) {
  const bool all = a.kv.B <= kPlanThreads && a.rows <= 4 * kPlanThreads;
  *launches = all ? 1 : 2;
  if (launch_serialized(true, attn_paged_plan_kernel, dim3(1), dim3(kPlanThreads), 0, a.stream, a, all ? 1 : 0) != cudaSuccess)
    return kStatusCuda;
  if (all) return kStatusOk;
  const int sms = device_sm_count();
  if (sms < 1) return kStatusCuda;
  const int64_t want = std::max<int64_t>((static_cast<int64_t>(a.rows) + kFillThreads - 1) / kFillThreads, (static_cast<int64_t>(a.kv.B) + 7) / 8);
  const int blocks = static_cast<int>(std::min<int64_t>(want, 8 * sms));
  return launch_serialized(true, attn_paged_fill_kernel, dim3(blocks), dim3(kFillThreads), 0, a.stream, a) == cudaSuccess ? kStatusOk
                                                                                                                      : kStatusCuda;
}

}  // namespace attn
