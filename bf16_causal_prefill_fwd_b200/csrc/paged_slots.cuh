// Bookkeeping of a serving step over a paged cache, on the device: from the
// requests' lengths (ctx cached, nw new tokens) the kernel writes
//   cu[b]     = sum of nw before b,          kv[b] = ctx[b] + nw[b]
//   pos[t]    = ctx[b] + (t - cu[b])          for the new token t of request b
//   slot[t]   = page * page_size + pos % page_size, page = table[b][pos / page_size]
// and, given a free list, first enters the pages a request lacks,
//   table[b][j] = free[head + fresh(0..b-1) + j - held(b)],  held = ceil(ctx / ps)
// with fresh(b) = ceil(kv / ps) - ceil(ctx / ps), in request order.
//
// It reads a few integers per request and writes eight bytes per token, so what
// bounds it is latency: one launch, no pass over global memory between its
// steps. Every block of one cluster scans all requests for itself (two prefix
// sums, kept in shared memory), then takes its share of the tokens, finding a
// token's request by bisection. A new token's page is computed from the scan,
// not read back from the table. The free list's head may be updated in place:
// the cluster barrier stands between the last read and the one write. A decoding
// step of 13 requests takes 4.8-5.0 us a call in a loop, 512 requests with 16 thousand
// new tokens 7.5 us; of either the launch is about 3, what an append of as few tokens
// takes (2.7), and the rest the scan's steps and their barriers.
//
// Anything that does not fit (a negative length, one past 32 bits, more tokens than
// `total`, more pages than a table row holds or than are free) is found before any table
// entry or the head is written: the step is then empty (cu and kv zero, every
// slot -1) and the status word says why.
#pragma once

#include "paged_common.cuh"

namespace b200p {

constexpr int kSlotsThreads = 1024;
constexpr int kSlotsCluster = 8;
constexpr int kSlotsMaxBatch = 16384;  // three arrays in shared memory

struct PagedSlots {
  int* table;
  int64_t table_stride;
  int width;
  const int* ctx;
  const int* nw;
  int B, total, page_size;
  const int* free_pages;  // NULL: the table is complete
  int free_count;
  const int* head_in;
  int* head_out;
  int* cu;
  int* kv;
  int* pos;
  int* slot;
};

// Index of the last entry of s[0..n] that is <= x (s non-decreasing, s[0] <= x < s[n]).
__device__ __forceinline__ int last_not_above(const int* s, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Pages of c rows; c + ps may pass 2^31.
__device__ __forceinline__ int pages_of(int c, int ps) {
  return static_cast<int>((static_cast<uint32_t>(c) + ps - 1) / static_cast<uint32_t>(ps));
}

__global__ void __launch_bounds__(kSlotsThreads) paged_slots_kernel(const PagedSlots p) {
  extern __shared__ int sm[];
  int* s_cu = sm;               // [B + 1]
  int* s_fr = sm + (p.B + 1);   // [B + 1]
  int* s_ctx = s_fr + (p.B + 1);  // [B]
  __shared__ int2 warp_sum[kSlotsThreads / 32];
  __shared__ int s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x, blocks = gridDim.x;
  const int ps = p.page_size;
  const bool alloc = p.free_pages != nullptr;
  if (tid == 0) s_bad = 0;
  pdl_launch_dependents();
  pdl_wait();
  __syncthreads();

  const int head = alloc ? *p.head_in : 0;
  // prefix sums over the requests, kSlotsThreads at a time
  int2 run = make_int2(0, 0);
  int bad = 0;
  for (int b0 = 0; b0 < p.B; b0 += kSlotsThreads) {
    const int b = b0 + tid;
    int n = 0, fresh = 0;
    if (b < p.B) {
      const int c = __ldg(p.ctx + b);
      s_ctx[b] = c;
      n = __ldg(p.nw + b);
      const int64_t rows = static_cast<int64_t>(c) + n, want = (rows + ps - 1) / ps;
      if (c < 0 || n < 0 || n > p.total || want > p.width || rows > 0x7fffffff) {
        bad = -kPagedInvalid;
        n = 0;
      } else if (alloc) {
        fresh = static_cast<int>(want) - pages_of(c, ps);
      }
    }
    // n <= total < 2^30 and at most kSlotsThreads of them: saturate so that no sum overflows
    int2 x = make_int2(n, fresh);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int ux = __shfl_up_sync(0xffffffffu, x.x, o), uy = __shfl_up_sync(0xffffffffu, x.y, o);
      if (lane >= o) {
        x.x = min(x.x + ux, p.total + 1);
        x.y += uy;
      }
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int2 before = run;
    for (int w = 0; w < warp; ++w) {
      before.x = min(before.x + warp_sum[w].x, p.total + 1);
      before.y += warp_sum[w].y;
    }
    if (b < p.B) {
      s_cu[b + 1] = min(before.x + x.x, p.total + 1);
      s_fr[b + 1] = before.y + x.y;
    }
    for (int w = 0; w < kSlotsThreads / 32; ++w) {
      run.x = min(run.x + warp_sum[w].x, p.total + 1);
      run.y += warp_sum[w].y;
    }
    __syncthreads();
  }
  if (tid == 0) s_cu[0] = s_fr[0] = 0;
  if (run.x > p.total) bad = max(bad, -kPagedInvalid);
  if (alloc && (head < 0 || run.y > p.free_count - head)) bad = max(bad, -kPagedNoPages);
  if (bad) atomicMax(&s_bad, bad);
  __syncthreads();
  bad = s_bad;
  if (bad && rank == 0 && tid == 0) paged_report(-bad);
  // what every block has read may now be written: the head in place, new table entries
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");

  const int step = blocks * kSlotsThreads, at = rank * kSlotsThreads + tid;
  const int used = bad ? 0 : run.x;
  for (int b = at; b <= p.B; b += step) {
    p.cu[b] = bad ? 0 : s_cu[b];
    if (b < p.B) p.kv[b] = bad ? 0 : s_ctx[b] + s_cu[b + 1] - s_cu[b];
  }
  if (alloc && !bad) {
    for (int j = at; j < run.y; j += step) {
      const int b = last_not_above(s_fr, p.B, j);
      const int held = pages_of(s_ctx[b], ps);
      p.table[b * p.table_stride + held + (j - s_fr[b])] = __ldg(p.free_pages + head + j);
    }
  }
  if (alloc && rank == 0 && tid == 0) *p.head_out = head + (bad ? 0 : run.y);
#pragma unroll 2
  for (int t = at; t < p.total; t += step) {
    int pos = 0, slot = -1;
    if (t < used) {
      const int b = last_not_above(s_cu, p.B, t);
      const int c = s_ctx[b];
      pos = c + t - s_cu[b];
      const int idx = pos / ps, held = pages_of(c, ps);
      const int page = alloc && idx >= held ? __ldg(p.free_pages + head + s_fr[b] + idx - held)
                                            : p.table[b * p.table_stride + idx];
      const int64_t at_slot = static_cast<int64_t>(page) * ps + (pos - idx * ps);
      if (page < 0 || at_slot > 0x7fffffff)
        paged_report(kPagedInvalid);  // a table entry that is no page: the token keeps slot -1
      else
        slot = static_cast<int>(at_slot);
    }
    p.pos[t] = pos;
    p.slot[t] = slot;
  }
}

}  // namespace b200p
