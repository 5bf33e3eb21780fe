// Joining the parts of the units that several blocks have worked on: block c of
// the grid takes the unit that begins, but does not end, in block c; its rows
// are spread over gridDim.y. O = sum_b 2^(m_b - M) O_b / sum_b 2^(m_b - M) l_b,
// the running way, in block order, so results do not depend on timing. All it
// waits for is memory (2 to 5 us behind the attention kernel, most of it the
// launch), so (m, l) and O of several parts are asked for at once, neither
// depending on the other.
#pragma once

#include "paged_common.cuh"

namespace b200p {

struct JoinRow {
  float m = -INFINITY, l = 0.0f;
  // Factors of what has been added so far and of the part (x.x, x.y) = (m, l). A
  // part with l = 0 saw none of the row's keys and may have left O unwritten.
  __device__ __forceinline__ void add(float2 x, float& keep, float& take) {
    keep = 1.0f;
    take = 0.0f;
    if (x.y == 0.0f) return;
    const float mn = fmaxf(m, x.x);
    keep = m == -INFINITY ? 0.0f : ex2_approx(m - mn);
    take = ex2_approx(x.x - mn);
    m = mn;
    l = fmaf(l, keep, x.y * take);
  }
  __device__ __forceinline__ float lse() const { return l == 0.0f ? -INFINITY : (m + fast_log2(l)) * kLn2; }
};

__device__ __forceinline__ void join_add(float4& acc, const float4& o, float keep, float take) {
  if (take == 0.0f) return;  // (a NaN factor is not 0)
  acc.x = fmaf(acc.x, keep, o.x * take);
  acc.y = fmaf(acc.y, keep, o.y * take);
  acc.z = fmaf(acc.z, keep, o.z * take);
  acc.w = fmaf(acc.w, keep, o.w * take);
}

// Slot of part i of the unit that begins in block c: the block's tail slot, then
// the head slots of the blocks after it.
__device__ __forceinline__ int64_t join_slot(const PagedAttn& p, int c, int i) {
  return static_cast<int64_t>(2 * (c + i) + (i == 0 ? 1 : 0)) * p.slot_rows;
}

__device__ __forceinline__ void join_place(const PagedAttn& p, const PartDesc& e, int r, int& tok, int& hq) {
  const uint32_t row = e.row0 + r, t = row / p.group;
  hq = e.hkv * p.G + row - t * p.G;
  tok = e.t0 + t;
}

// Few rows (decoding): part_o is [slot][row][DV]. A row may have hundreds of parts
// (one long request over the whole GPU): a block takes a row, each of its warps
// every fourth part, and the four results meet in shared memory.
template <int DV>
__global__ void __launch_bounds__(128) paged_join_few_kernel(const PagedAttn p) {
  static_assert(DV == 128, "32 lanes x 4 columns");
  __shared__ float s_o[4][DV], s_ml[4][2];
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PartDesc e = reinterpret_cast<const PartDesc*>(p.desc)[c];
  if (e.last < 0) return;
  const int parts = e.last - c + 1;
  const float v_scale = p.v_scale != nullptr ? __ldg(p.v_scale + e.hkv) : 1.0f;
  for (int r = blockIdx.y; r < e.nrows; r += gridDim.y) {
    JoinRow j;
    float4 acc = {};
    for (int i0 = warp; i0 < parts; i0 += 16) {  // four parts' loads under way before the first is used
      float2 x[4];
      float4 o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t at = join_slot(p, c, min(i0 + 4 * k, parts - 1)) + r;
        x[k] = *reinterpret_cast<const float2*>(p.part_ml + 2 * at);
        o[k] = *reinterpret_cast<const float4*>(p.part_o + at * DV + 4 * lane);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (i0 + 4 * k >= parts) break;
        float keep, take;
        j.add(x[k], keep, take);
        join_add(acc, o[k], keep, take);
      }
    }
    *reinterpret_cast<float4*>(&s_o[warp][4 * lane]) = acc;
    if (lane == 0) {
      s_ml[warp][0] = j.m;
      s_ml[warp][1] = j.l;
    }
    __syncthreads();
    const int td = threadIdx.x;
    JoinRow all;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      float keep, take;
      all.add(make_float2(s_ml[w][0], s_ml[w][1]), keep, take);
      if (take != 0.0f) sum = fmaf(sum, keep, s_o[w][td] * take);
    }
    int tok, hq;
    join_place(p, e, r, tok, hq);
    p.o[(static_cast<int64_t>(tok) * p.Hq + hq) * DV + td] =
        __float2bfloat16(all.l == 0.0f ? 0.0f : sum * (1.0f / all.l) * v_scale);
    if (p.lse != nullptr && td == 0) p.lse[static_cast<int64_t>(hq) * p.T + tok] = all.lse();
    __syncthreads();  // s_o is written again
  }
}

// Many rows (chunks): part_o is [slot][DV / 4][row][4], as the threads that hold
// a row each write it in whole lines. A block takes 16 rows at a time, eight
// threads to a row, 16 columns each; the bf16 rows leave through shared memory.
template <int DV>
__global__ void __launch_bounds__(128) paged_join_rows_kernel(const PagedAttn p) {
  static_assert(DV == 128, "8 threads x 4 x 4 columns");
  __shared__ __align__(16) uint32_t s_o[16][DV / 2 + 4];
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x, lr = threadIdx.x & 15, l8 = threadIdx.x >> 4;
  const PartDesc e = reinterpret_cast<const PartDesc*>(p.desc)[c];
  if (e.last < 0) return;
  const int parts = e.last - c + 1;
  const float v_scale = p.v_scale != nullptr ? __ldg(p.v_scale + e.hkv) : 1.0f;
  for (int r0 = 16 * blockIdx.y; r0 < e.nrows; r0 += 16 * gridDim.y) {
    const int r = min(r0 + lr, e.nrows - 1);
    JoinRow j;
    float4 acc[4] = {};
#pragma unroll 2
    for (int i = 0; i < parts; ++i) {
      const int64_t at = join_slot(p, c, i);
      const float2 x = *reinterpret_cast<const float2*>(p.part_ml + 2 * (at + r));
      float4 o[4];
#pragma unroll
      for (int n = 0; n < 4; ++n)
        o[n] = *reinterpret_cast<const float4*>(p.part_o + at * DV + (static_cast<int64_t>(l8 + 8 * n) * p.slot_rows + r) * 4);
      float keep, take;
      j.add(x, keep, take);
#pragma unroll
      for (int n = 0; n < 4; ++n) join_add(acc[n], o[n], keep, take);
    }
    const float inv = j.l == 0.0f ? 0.0f : 1.0f / j.l, vs = j.l == 0.0f ? 0.0f : v_scale;
#pragma unroll
    for (int n = 0; n < 4; ++n)
      *reinterpret_cast<uint2*>(&s_o[lr][2 * (l8 + 8 * n)]) =
          make_uint2(pack_bf16x2(acc[n].x * inv * vs, acc[n].y * inv * vs),
                     pack_bf16x2(acc[n].z * inv * vs, acc[n].w * inv * vs));
    int tok, hq;
    if (p.lse != nullptr && l8 == 0 && r0 + lr < e.nrows) {
      join_place(p, e, r, tok, hq);
      p.lse[static_cast<int64_t>(hq) * p.T + tok] = j.lse();
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < 2; ++n) {  // 16 threads to a row of 256 bytes
      const int row = 8 * n + (threadIdx.x >> 4);
      if (r0 + row < e.nrows) {
        join_place(p, e, r0 + row, tok, hq);
        reinterpret_cast<uint4*>(p.o + (static_cast<int64_t>(tok) * p.Hq + hq) * DV)[lr] =
            *reinterpret_cast<const uint4*>(&s_o[row][4 * lr]);
      }
    }
    __syncthreads();  // s_o is written again
  }
}

}  // namespace b200p
