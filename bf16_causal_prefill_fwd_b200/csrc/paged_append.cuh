// Writes the K and V rows of new tokens to their cache slots: for token t and
// slot s = slots[t], page s / page_size, row s % page_size,
//   bf16 cache:  cache = x
//   e4m3 cache:  cache = e4m3(x / scale[h]), round to nearest even, held at +-448
// (the division is IEEE fp32, so a code is the one the definition gives).
//
// Bound by memory: 2 (d_qk + d_v) bytes read per token and head, the same or
// half of that written. A thread moves units of 16 elements (two 16-byte loads,
// one or two 16-byte stores) of K and V alike; consecutive threads take
// consecutive units of a token's row, so loads and stores are whole lines
// whatever the order of the slots.
#pragma once

#include "paged_common.cuh"

namespace b200p {

constexpr int kAppendThreads = 256;
constexpr int kAppendUnit = 16;  // elements per thread and step

struct PagedAppend {
  const __nv_bfloat16* x[2];  // K, V: [T, H, d], rows of one token contiguous
  int64_t x_stride[2];        // between tokens, in elements
  void* cache[2];
  int64_t page_stride[2], token_stride[2], head_stride[2];
  const float* scale[2];
  const int* slots;
  int T, H, d[2];
  int num_pages, page_size;
};

__device__ __forceinline__ uint32_t e4m3x4_of(uint32_t b01, uint32_t b23, float s) {
  const float f0 = __fdiv_rn(__uint_as_float(b01 << 16), s), f1 = __fdiv_rn(__uint_as_float(b01 & 0xffff0000u), s);
  const float f2 = __fdiv_rn(__uint_as_float(b23 << 16), s), f3 = __fdiv_rn(__uint_as_float(b23 & 0xffff0000u), s);
  return static_cast<uint32_t>(pack_e4m3x2(f0, f1)) | (static_cast<uint32_t>(pack_e4m3x2(f2, f3)) << 16);
}

template <bool FP8>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const PagedAppend p) {
  const int uk = p.d[0] / kAppendUnit, uv = p.d[1] / kAppendUnit;
  const int k_units = p.H * uk;
  const uint32_t per_token = p.H * (uk + uv);
  const uint32_t n = static_cast<uint32_t>(p.T) * per_token;  // < 2^31 (the host checks)
  for (uint32_t i = blockIdx.x * kAppendThreads + threadIdx.x; i < n; i += gridDim.x * kAppendThreads) {
    const int t = i / per_token;
    int u = i - t * per_token;
    const int which = u >= k_units;  // 0: K, 1: V
    if (which) u -= k_units;
    const int upr = which ? uv : uk;
    const int h = u / upr, e = (u - h * upr) * kAppendUnit;
    const uint4* src = reinterpret_cast<const uint4*>(p.x[which] + t * p.x_stride[which] +
                                                      static_cast<int64_t>(h) * p.d[which] + e);
    const int slot = __ldg(p.slots + t);
    const uint4 a = __ldg(src), b = __ldg(src + 1);
    if (slot < 0) continue;  // a padded row
    const int page = slot / p.page_size;
    if (page >= p.num_pages) {
      paged_report(kPagedInvalid);
      continue;
    }
    const int64_t off = page * p.page_stride[which] + (slot - page * p.page_size) * p.token_stride[which] +
                        h * p.head_stride[which] + e;
    if constexpr (FP8) {
      const float s = __ldg(p.scale[which] + h);
      uint4 c;
      c.x = e4m3x4_of(a.x, a.y, s);
      c.y = e4m3x4_of(a.z, a.w, s);
      c.z = e4m3x4_of(b.x, b.y, s);
      c.w = e4m3x4_of(b.z, b.w, s);
      *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.cache[which]) + off) = c;
    } else {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.cache[which]) + off);
      dst[0] = a;
      dst[1] = b;
    }
  }
}

}  // namespace b200p
