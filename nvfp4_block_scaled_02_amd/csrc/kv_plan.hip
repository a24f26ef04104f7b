// kv_plan.hip -- pages, slots and positions of a step's new tokens from the
// requests' lengths.
#include "kv.hpp"

namespace nvfp4 {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;

// Inclusive sum over the workgroup, in thread order, of two values at once
// (both below 2^62); `total` gets the workgroup's sums.
struct Pair64 {
  int64_t a, b;
};
__device__ __forceinline__ Pair64 block_scan(Pair64 v, Pair64* wave_sums, Pair64& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t a = __shfl_up((long long)v.a, d), b = __shfl_up((long long)v.b, d);
    if (lane >= d) {
      v.a += a;
      v.b += b;
    }
  }
  __syncthreads();  // wave_sums may still be read from the last chunk
  if (lane == 63) wave_sums[wave] = v;
  __syncthreads();
  total = Pair64{0, 0};
#pragma unroll
  for (int i = 0; i < kPlanWaves; ++i) {
    const Pair64 s = wave_sums[i];
    if (i < wave) {
      v.a += s.a;
      v.b += s.b;
    }
    total.a += s.a;
    total.b += s.b;
  }
  return v;
}

struct Request {
  int64_t first;  // first of its new tokens
  int64_t page0;  // pages that the requests before it take
  int32_t ctx, have;
  int32_t ok, pad;
};

// Every workgroup scans all requests in chunks of 1024 (8 bytes a request,
// from the caches) and writes its 1024 tokens: no workgroup waits for
// another, and one launch does it.  Workgroup 0 writes the per-request
// outputs.  The first token of each new page writes its table entry.  Bound by
// the latency of a launch and four dependent reads (lengths, free count, free
// page, table): 5.4 us for 32 requests of one token, 6.8 us for 1024 requests
// with some 65 thousand.
__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(nvfp4_kv_plan_args a, int shift) {
  __shared__ Pair64 wave_sums[kPlanWaves];
  __shared__ Request req[kPlanThreads];
  __shared__ int refused_here;
  const int page_size = 1 << shift;
  int64_t free_count = *a.free_count;
  free_count = free_count < 0 ? 0 : free_count > a.num_pages ? a.num_pages : free_count;
  const int64_t t = (int64_t)blockIdx.x * kPlanThreads + threadIdx.x;
  const int64_t block_t0 = (int64_t)blockIdx.x * kPlanThreads;
  int64_t tok0 = 0, page0 = 0, taken = 0;
  bool mine = t < a.tokens;  // still to be written
  if (threadIdx.x == 0) refused_here = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) a.cu_new[0] = 0;
  for (int64_t b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
    const int64_t b = b0 + threadIdx.x;
    int64_t ctx = 0, fresh = 0;
    if (b < a.batch) {
      ctx = a.ctx_lens[b];
      fresh = a.new_lens[b];
      ctx = ctx < 0 ? 0 : ctx;
      fresh = fresh < 0 ? 0 : fresh;
    }
    const int64_t have = (ctx + page_size - 1) >> shift;
    const int64_t need = (ctx + fresh + page_size - 1) >> shift;
    // lengths and positions are 32-bit numbers, whatever the table has room for
    const bool fits = need <= a.table_width && ctx + fresh <= INT32_MAX;
    const int64_t more = fits ? need - have : 0;
    Pair64 total;
    const Pair64 sum = block_scan(Pair64{fresh, more}, wave_sums, total);
    // new tokens that the step has no room for: their ends ascend, so no
    // request behind such a one is admitted to a page either
    const bool room = fresh == 0 || tok0 + sum.a <= a.tokens;
    const bool ok = fits && room && (more == 0 || page0 + sum.b <= free_count);
    req[threadIdx.x] = Request{tok0 + sum.a - fresh, page0 + sum.b - more, (int32_t)ctx, (int32_t)have, ok, 0};
    if (blockIdx.x == 0 && b < a.batch) {
      a.cu_new[b + 1] = (int32_t)(tok0 + sum.a < INT32_MAX ? tok0 + sum.a : INT32_MAX);
      a.seq_lens[b] = (int32_t)(ok ? ctx + fresh : ctx);
      if (!ok) atomicAdd(&refused_here, 1);
    }
    // pages taken: the running total of the last admitted request (totals
    // ascend, so those within the free count and the tokens are a prefix)
    __syncthreads();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      const auto within = [&](int64_t tokens, int64_t pages) { return tokens <= a.tokens && pages <= free_count; };
      if (within(tok0 + total.a, page0 + total.b)) taken = page0 + total.b;
      else if (within(tok0, page0)) {
        int lo = 0, hi = kPlanThreads - 1;  // first request past either: at the latest the chunk's last
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (within(req[mid + 1].first, req[mid + 1].page0)) lo = mid + 1;
          else hi = mid;
        }
        taken = req[lo].page0;
      }
    }
    const int64_t end = tok0 + total.a;
    if (mine && t < end && t >= tok0) {
      int lo = 0, hi = kPlanThreads - 1;  // last request that begins at or before t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (req[mid].first <= t) lo = mid;
        else hi = mid - 1;
      }
      const Request r = req[lo];
      const int64_t pos = r.ctx + (t - r.first);
      const int64_t page_at = pos >> shift;
      int64_t slot = -1;
      if (r.ok) {
        int64_t page;
        int32_t* entry = a.block_table + (b0 + lo) * a.table_width + page_at;
        if (page_at < r.have) {
          page = *entry;
        } else {
          page = a.free_pages[free_count - 1 - (r.page0 + page_at - r.have)];
          if ((pos & (page_size - 1)) == 0) *entry = (int32_t)page;
        }
        if (page >= 0 && page < a.num_pages) slot = (page << shift) + (pos & (page_size - 1));
      }
      a.positions[t] = (int32_t)pos;
      a.slots[t] = slot;
      mine = false;
    }
    tok0 = end;
    page0 += total.b;
    // a workgroup whose tokens are all written needs no further requests
    if (blockIdx.x != 0 && tok0 >= block_t0 + kPlanThreads) return;
    __syncthreads();
  }
  if (mine) {
    a.positions[t] = 0;
    a.slots[t] = -1;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *a.free_count_out = (int32_t)(free_count - taken);
    *a.refused = refused_here;
  }
}

hipError_t launch_kv_plan(const nvfp4_kv_plan_args& a, hipStream_t s) {
  const int64_t g = (a.tokens + kPlanThreads - 1) / kPlanThreads;
  hipLaunchKernelGGL(kv_plan_kernel, dim3((unsigned)(g < 1 ? 1 : g)), dim3(kPlanThreads), 0, s, a,
                     __builtin_ctz((unsigned)a.page_size));
  return hipGetLastError();
}

}  // namespace nvfp4
