// Writes the K and V rows of new tokens to their cache slots: for token t and
// slot s = slots[t], page s / page_size, row s % page_size,
//   bf16 cache:  cache = x
//   e4m3 cache:  cache = e4m3(x / scale[h]), round to nearest even, held at +-448
// (the quotient is the correctly rounded one, so a code is the one the
// definition gives).
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
  int T, H;
  int num_pages;
  FastDiv page_size, per_token;  // per_token: units of one token, H (d_qk + d_v) / 16
};

// x / s rounded to nearest even, by Markstein's correction: with r = 1 / s
// rounded and q = x r within an ulp of the quotient, q + (x - q s) r rounds to
// the quotient itself ("Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990). 3 FMAs instead of a called division, which
// bounded the kernel. x is first held at +-512 s (any code from 464 s on is
// 448), so that an infinite or overflowing quotient never meets the correction;
// NaN stays NaN. Scales whose reciprocal or 512-fold is not a plain normal
// number take the division.
struct CodeScale {
  float s, r, lim;
  bool plain;
  __device__ __forceinline__ explicit CodeScale(float scale)
      : s(scale), r(1.0f / scale), lim(512.0f * scale), plain(scale > 1e-30f && scale < 1e30f) {}
  __device__ __forceinline__ float quotient(float x) const {
    if (!plain) return __fdiv_rn(x, s);
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(lim));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(-lim));
    const float q = x * r;
    return fmaf(fmaf(-q, s, x), r, q);
  }
  __device__ __forceinline__ uint32_t codes(uint32_t b01, uint32_t b23) const {
    const float f0 = quotient(__uint_as_float(b01 << 16)), f1 = quotient(__uint_as_float(b01 & 0xffff0000u));
    const float f2 = quotient(__uint_as_float(b23 << 16)), f3 = quotient(__uint_as_float(b23 & 0xffff0000u));
    return static_cast<uint32_t>(pack_e4m3x2(f0, f1)) | (static_cast<uint32_t>(pack_e4m3x2(f2, f3)) << 16);
  }
};

template <int DQK, int DV, bool FP8>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const PagedAppend p) {
  constexpr int UK = DQK / kAppendUnit, UV = DV / kAppendUnit;
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t k_units = p.H * UK;
  const uint32_t n = p.T * p.per_token.d;  // < 2^31 (the host checks)
  for (uint32_t i = blockIdx.x * kAppendThreads + threadIdx.x; i < n; i += gridDim.x * kAppendThreads) {
    const uint32_t t = i / p.per_token;
    uint32_t u = i - t * p.per_token.d;
    const bool v = u >= k_units;
    uint32_t h, e;
    if (v) {
      u -= k_units;
      h = u / UV;
      e = (u - h * UV) * kAppendUnit;
    } else {
      h = u / UK;
      e = (u - h * UK) * kAppendUnit;
    }
    const uint4* src = reinterpret_cast<const uint4*>(p.x[v] + t * p.x_stride[v] + h * (v ? DV : DQK) + e);
    const int slot = __ldg(p.slots + t);
    const uint4 a = __ldg(src), b = __ldg(src + 1);
    if (slot < 0) continue;  // a padded row
    const uint32_t page = static_cast<uint32_t>(slot) / p.page_size;
    if (page >= static_cast<uint32_t>(p.num_pages)) {
      paged_report(kPagedInvalid);
      continue;
    }
    const int64_t off = page * p.page_stride[v] + (slot - page * p.page_size.d) * p.token_stride[v] +
                        h * p.head_stride[v] + e;
    if constexpr (FP8) {
      const CodeScale cs(__ldg(p.scale[v] + h));
      uint4 c;
      c.x = cs.codes(a.x, a.y);
      c.y = cs.codes(a.z, a.w);
      c.z = cs.codes(b.x, b.y);
      c.w = cs.codes(b.z, b.w);
      *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.cache[v]) + off) = c;
    } else {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.cache[v]) + off);
      dst[0] = a;
      dst[1] = b;
    }
  }
}

}  // namespace b200p
