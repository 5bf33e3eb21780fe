// Shared pieces of the paged-cache kernels: the device status word, bounded
// waits, the PTX they use beyond sm100_ptx.cuh, and the split of a batch's
// attention work into equal runs of key tiles.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sm100_ptx.cuh"

namespace b200p {

using namespace b200;  // the PTX wrappers

constexpr uint64_t kPagedWaitLimitNs = 2000000000ull;  // bounded waits: 2 s
constexpr int kPagedTimeout = -4;                      // B200ATTN_ERR_TIMEOUT
constexpr int kPagedInvalid = -1;                      // B200ATTN_ERR_INVALID
constexpr int kPagedNoPages = -6;                      // B200ATTN_ERR_PAGES
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Probabilities in fp16 (e4m3 caches) are held as 2^x times their value, so that the
// largest of a row is near 2^15 and uses the type's range: rounding takes at most
// 2^-25 off any of them, so that a row of n keys, its small probabilities under the
// smallest subnormal among them, loses at most n 2^-40 of its largest. The factor is
// in the row sum, too; the m that is kept with it is less by x.
constexpr float kHalfExp = 15.0f;

// Status word of these kernels; b200attn_check reads it with the other one.
__device__ int g_paged_status;

__device__ __forceinline__ void paged_report(int code) { atomicCAS(&g_paged_status, 0, code); }

// Bounded mbarrier wait, as the prefill kernels have it: false if it gave up
// after two seconds or another role of the block already had.
__device__ __forceinline__ bool paged_wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  const uint64_t t0 = global_timer_ns();
  while (true) {
    if (mbar_try_wait_suspend(bar, parity, 1000000u)) return true;
    if (*abort_flag) return false;
    if (global_timer_ns() - t0 > kPagedWaitLimitNs) {
      *abort_flag = 1;
      paged_report(kPagedTimeout);
      return false;
    }
  }
}

__device__ __forceinline__ bool paged_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  return paged_wait_slow(bar, parity, abort_flag);
}

// Programmatic dependent launch: let the next kernel of the stream start its
// blocks / wait until the kernels this one depends on have finished and their
// writes can be seen.
__device__ __forceinline__ void pdl_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Transpose of an 8x8 matrix of 16-bit values held one row per four lanes.
__device__ __forceinline__ uint32_t movm_t(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// D += A B, 16 x 8 x 16, fp32 accumulators; HALF: fp16 operands, else bf16.
template <bool HALF>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (HALF) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

// Two e4m3 codes (low 16 bits of c) -> f16x2, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(c)));
  return r;
}

// Two fp32 -> f16x2, lo in bits [0,16), held at +-65504; NaN stays NaN.
__device__ __forceinline__ uint32_t pack_f16x2_sat(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// n / d for 0 <= n < 2^31 by a multiplication: with l = ceil(log2 d) and m =
// ceil(2^(31 + l) / d), n m / 2^(31 + l) exceeds n / d by less than 1 / d, so the
// floors agree (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994).
struct FastDiv {
  uint32_t d, m, s;
};
inline FastDiv fast_div(uint32_t d) {
  uint32_t l = 0;
  while ((uint64_t(1) << l) < d) ++l;
  if (l == 0) return {1, 0, 0};  // d = 1: taken apart in the division
  return {d, static_cast<uint32_t>(((uint64_t(1) << (31 + l)) + d - 1) / d), l - 1};
}
__device__ __forceinline__ uint32_t operator/(uint32_t n, const FastDiv& f) {
  return f.m == 0 ? n : __umulhi(n, f.m) >> f.s;
}

// What the attention kernels are given. Strides are in elements.
struct PagedAttn {
  const __nv_bfloat16* q;  // [T, Hq, d_qk], rows of one token contiguous
  int64_t q_stride;        // between tokens
  const int* table;        // [B, width] page numbers
  int table_stride;
  int width;
  const int* cu;       // [B + 1] first new token of each request
  const int* kv_lens;  // [B] keys of each request, new ones included
  int B, T, Hq, Hkv, G;
  FastDiv group;  // G
  FastDiv pair;   // tokens of a pair of row tiles (chunks)
  int num_pages, page_size;
  FastDiv rows;  // page_size
  int box;       // rows of a page one TMA copy takes: gcd(page_size, key tile)
  int max_q;     // bound on the new tokens of one request
  int causal;
  float scale_log2;      // softmax scale * log2(e)
  const float* k_scale;  // [Hkv], e4m3 caches
  const float* v_scale;
  __nv_bfloat16* o;  // [T, Hq, d_v]
  float* lse;        // [Hq, T] or NULL
  int* desc;         // workspace: one PartDesc per block
  float* part_ml;    // workspace: (m, l) per slot and row
  float* part_o;     // workspace: O per slot and row
  int slot_rows;     // rows of a slot
};

// One request as the kernels see it; tiles == 0: nothing is computed for it.
struct Request {
  int t0, nq, kv;
};

// Reads request b. Lengths that do not fit the tensors are reported and give
// an empty request, so that no later index can leave them.
__device__ __forceinline__ Request paged_request(const PagedAttn& p, int b, bool report) {
  Request r;
  r.t0 = __ldg(p.cu + b);
  const int t1 = __ldg(p.cu + b + 1);
  r.nq = t1 - r.t0;
  r.kv = __ldg(p.kv_lens + b);
  const bool bad = r.t0 < 0 || t1 > p.T || r.nq < 0 || r.nq > p.max_q || r.kv < 0 ||
                   r.kv > static_cast<int64_t>(p.width) * p.page_size;
  if (bad) {
    if (report) paged_report(kPagedInvalid);
    r.t0 = r.nq = r.kv = 0;
  }
  return r;
}

// Page of key `key` of request b, or num_pages (out of the tensor map's range:
// the copy reads zeros) behind the last key and for a page number that is none.
__device__ __forceinline__ int paged_page(const PagedAttn& p, int b, int key, int kv) {
  if (key >= kv) return p.num_pages;
  const int page = __ldg(p.table + static_cast<int64_t>(b) * p.table_stride + static_cast<uint32_t>(key) / p.rows);
  if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.num_pages)) {
    paged_report(kPagedInvalid);
    return p.num_pages;
  }
  return page;
}

// Row of its page that key `key` has.
__device__ __forceinline__ int paged_row(const PagedAttn& p, int key) {
  return key - static_cast<int>(static_cast<uint32_t>(key) / p.rows) * p.page_size;
}

// A block's run of a line of work that all requests form in order, request b
// taking cost(b) * Hkv of it: runs are `per` long, this one starts at `first`,
// `off` into request b (`req`, of cost `cost` per head), and is `count` long.
struct Run {
  int b, off, count, first, per, cost;
  Request req;
};

// By one whole warp, 32 requests at a time (the next ones' lengths, the only
// memory it waits for, are read ahead): the sum of the costs in 64 bits --
// requests whose rows overlap could make the line longer than the host's bound,
// which is then refused -- and the request the run starts in by a scan over the
// lanes. No other warp waits meanwhile.
//
// No run is shorter than the root of a third of the longest unit (`longest` of each
// request): a unit's parts are joined one after another, and a part costs the join
// about a third of what a piece of work costs. One request of 4 tokens and 13k keys,
// one head of 102 key blocks: 60 us in runs of one, 23 in runs of 5; over 64k keys
// 72 us in runs of 4, 43 in runs of 12.
template <typename Cost, typename Longest>
__device__ __forceinline__ Run plan_run(const PagedAttn& p, Cost cost, Longest longest) {
  const int lane = threadIdx.x & 31;
  const bool report = blockIdx.x == 0;
  Request ahead = {0, 0, 0};
  if (lane < p.B) ahead = paged_request(p, lane, report);
  int c = 0, most = 0;
  long long sum = 0;
  Request x = {0, 0, 0};
#pragma unroll 1
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    x = ahead;
    ahead.nq = 0;
    if (b0 + 32 + lane < p.B) ahead = paged_request(p, b0 + 32 + lane, report);
    c = b0 + lane < p.B ? cost(x) : 0;
    sum += c;
    if (b0 + lane < p.B) most = max(most, longest(x));
  }
  most = __reduce_max_sync(0xffffffffu, most);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  Run r = {0, 0, 0, 0, 1, 1, {0, 0, 0}};
  if (sum * p.Hkv >= (1ll << 31)) {
    if (report && lane == 0) paged_report(kPagedInvalid);
    return r;
  }
  const int total = static_cast<int>(sum) * p.Hkv;
  r.per = max(static_cast<int>(sqrtf(most * (1.0f / 3.0f))),
              static_cast<int>((total + gridDim.x - 1) / static_cast<int>(gridDim.x)));
  r.first = blockIdx.x * r.per;
  r.count = max(0, min(r.per, total - r.first));
  if (r.count == 0) return r;
  int before = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    if (p.B > 32) {  // else both are there still
      c = 0;
      if (b0 + lane < p.B) {
        x = paged_request(p, b0 + lane, false);
        c = cost(x);
      }
    }
    const int y = c * p.Hkv;
    int inc = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, r.first < before + inc);
    if (past != 0) {
      const int at = __ffs(past) - 1;
      r.b = b0 + at;
      r.off = __shfl_sync(0xffffffffu, r.first - (before + inc - y), at);
      r.cost = __shfl_sync(0xffffffffu, c, at);
      r.req.t0 = __shfl_sync(0xffffffffu, x.t0, at);
      r.req.nq = __shfl_sync(0xffffffffu, x.nq, at);
      r.req.kv = __shfl_sync(0xffffffffu, x.kv, at);
      return r;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  r.count = 0;  // lengths that changed while being read
  return r;
}

// The part of a split unit that begins in a block, for the merge: its rows, and
// the last block that holds a part of it (-1: the block begins no split unit).
struct PartDesc {
  int last, t0, row0, nrows, hkv, pad[3];
};

}  // namespace b200p
