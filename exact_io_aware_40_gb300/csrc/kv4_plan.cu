// kv4_plan.cu -- block tables, slot maps and the free list of a step, from the
// requests' lengths, in one launch.
//
// With n_b new tokens and need_b new pages per request, everything follows from
// three prefix sums over the requests (tokens, pages taken, pages returned).
// Requests are served while the inclusive sums fit, so the served ones are a
// prefix of the list.  Every CTA computes the sums for itself (they are small
// beside a launch's latency, and a second launch or a grid-wide wait would cost
// more) and then takes its share of the outputs: a slot or a page finds its
// request by a binary search in the sums, which gives even shares whatever the
// lengths.  A new token's page is read from the free list, not from the table
// entry that another CTA may just be writing.
// Bound: a launch and three dependent phases; 3.3 us for 16 requests, 8.2 us for
// 1024 with prompts.
#include "fa.h"
#include "kv4.h"

namespace fa {
namespace {

constexpr int kPlanThreads = 512;

struct Sums {
  long long tokens, pages, back;
};

__device__ __forceinline__ Sums operator+(Sums a, Sums b) {
  return {a.tokens + b.tokens, a.pages + b.pages, a.back + b.back};
}

__device__ __forceinline__ Sums shfl_up(Sums v, int d) {
  return {__shfl_up_sync(0xffffffffu, v.tokens, d), __shfl_up_sync(0xffffffffu, v.pages, d),
          __shfl_up_sync(0xffffffffu, v.back, d)};
}

// What request b asks for.  A request with invalid lengths asks for more pages
// than there can be.
__device__ __forceinline__ Sums asked(const Kv4PlanArgs& a, int b, int* past_out, int* held_out) {
  const int past = a.past[b], n = a.fresh[b];
  const int page = 1 << a.page_shift;
  const long long room = static_cast<long long>(a.max_pages) << a.page_shift;
  const long long after = static_cast<long long>(past) + (n > 0 ? n : 0);
  *past_out = past;
  *held_out = 0;
  if (past < 0 || n < -1 || after > room) return {0, 1ll << 40, 0};
  const long long held = (past + static_cast<long long>(page) - 1) >> a.page_shift;
  *held_out = static_cast<int>(held);
  if (n < 0) return {0, 0, held};
  return {n, ((after + page - 1) >> a.page_shift) - held, 0};
}

// The last i in [0, n) with at[i] <= x (at[0] <= x).
__device__ __forceinline__ int last_at_most(const int* at, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) kv4_plan_kernel(const Kv4PlanArgs a) {
  extern __shared__ int sums[];
  int* cu = sums;                // [B + 1] tokens before request b
  int* pg = cu + a.B + 1;        // [B + 1] pages taken before it
  int* bk = pg + a.B + 1;        // [B + 1] pages returned before it
  __shared__ Sums warp_sum[kPlanThreads / 32];
  __shared__ int served;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int F = a.num_pages;
  int head = a.ring_state[0], count = a.ring_state[1];
  if (head < 0 || head >= F || count < 0 || count > F) {
    if (blockIdx.x == 0 && tid == 0) atomicCAS(a.input_err, 0, FA_ERR_INVALID_ARG);
    head = 0;
    count = 0;
  }
  if (tid == 0) served = 0;

  const int per = (a.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  Sums mine{0, 0, 0};
  int past, held;
  for (int b = b0; b < b1; ++b) mine = mine + asked(a, b, &past, &held);
  Sums run = mine;  // inclusive over the warp
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Sums o = shfl_up(run, d);
    if (lane >= d) run = run + o;
  }
  if (lane == 31) warp_sum[warp] = run;
  __syncthreads();
  Sums before{run.tokens - mine.tokens, run.pages - mine.pages, run.back - mine.back};
  for (int w = 0; w < warp; ++w) before = before + warp_sum[w];

  constexpr long long kCap = 0x7fffffff;
  int fit = 0;
  for (int b = b0; b < b1; ++b) {
    cu[b] = static_cast<int>(min(before.tokens, kCap));
    pg[b] = static_cast<int>(min(before.pages, kCap));
    bk[b] = static_cast<int>(min(before.back, kCap));
    before = before + asked(a, b, &past, &held);
    if (before.tokens <= a.max_tokens && before.pages <= count) ++fit;
  }
  if (b1 == a.B && b0 < b1) {
    cu[a.B] = static_cast<int>(min(before.tokens, kCap));
    pg[a.B] = static_cast<int>(min(before.pages, kCap));
    bk[a.B] = static_cast<int>(min(before.back, kCap));
  }
  if (fit) atomicAdd(&served, fit);
  __syncthreads();
  const int S = served;  // requests 0 .. S - 1 are served
  const int tokens = cu[S], pages = pg[S];
  int back = bk[a.B];
  if (back > F - count) {  // more pages come back than were ever taken
    if (blockIdx.x == 0 && tid == 0) atomicCAS(a.input_err, 0, FA_ERR_INVALID_ARG);
    back = F - count;
  }

  const int gt = blockIdx.x * kPlanThreads + tid, gn = gridDim.x * kPlanThreads;
  for (int b = gt; b < a.B; b += gn) {
    const int n = a.fresh[b], p = a.past[b];
    a.kv_len[b] = n == -1 ? 0 : (b < S ? p + n : p);
  }
  for (int b = gt; b <= a.B; b += gn) a.cu_q[b] = cu[min(b, S)];
  if (gt == 0) {
    int h = head + pages;
    a.state_out[0] = h >= F ? h - F : h;
    a.state_out[1] = count - pages + back;
    a.state_out[2] = tokens;
    a.state_out[3] = S;
  }
  // Page j of the pages taken: entry j of the ring, from its front.
  for (int j = gt; j < pages; j += gn) {
    const int b = last_at_most(pg, S, j);
    asked(a, b, &past, &held);
    int at = head + j;
    at = at >= F ? at - F : at;
    a.table[static_cast<long long>(b) * a.max_pages + held + (j - pg[b])] = a.ring[at];
  }
  // Page j of the pages returned, behind the ring's last entry (never one of
  // the entries read above: count + back <= num_pages).
  for (int j = gt; j < back; j += gn) {
    const int b = last_at_most(bk, a.B, j);
    long long at = static_cast<long long>(head) + count + j;
    at = at % F;
    a.ring[at] = a.table[static_cast<long long>(b) * a.max_pages + (j - bk[b])];
  }
  bool bad = false;
  for (int t = gt; t < a.max_tokens; t += gn) {
    int slot = -1;
    if (t < tokens) {
      const int b = last_at_most(cu, S, t);
      asked(a, b, &past, &held);
      const int pos = past + (t - cu[b]);
      const int idx = pos >> a.page_shift;
      int page;
      if (idx >= held) {
        int at = head + pg[b] + (idx - held);
        at = at >= F ? at - F : at;
        page = a.ring[at];
      } else {
        page = a.table[static_cast<long long>(b) * a.max_pages + idx];
      }
      if (page >= 0 && page < a.num_pages)
        slot = (page << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
      else
        bad = true;
    }
    a.slots[t] = slot;
  }
  if (bad) atomicCAS(a.input_err, 0, FA_ERR_INVALID_ARG);
}

}  // namespace

cudaError_t launch_kv4_plan(const Kv4PlanArgs& a, cudaStream_t stream) {
  const size_t smem = 3 * sizeof(int) * (static_cast<size_t>(a.B) + 1);
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kv4_plan_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  // One CTA up to some thousand slots (a decode step): more would only repeat
  // the sums.
  long long ctas = (static_cast<long long>(a.max_tokens) + 4 * kPlanThreads - 1) / (4 * kPlanThreads);
  ctas = ctas < 1 ? 1 : ctas > 128 ? 128 : ctas;
  kv4_plan_kernel<<<static_cast<unsigned>(ctas), kPlanThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace fa
