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
// whatever the order of the slots. 16384 tokens of 8 heads of 128: bf16 20.7-22.4 us
// (6.0-6.5 TB/s), e4m3 18.4-18.9 us (5.3 TB/s; the conversion's instructions take 78% of
// the issue slots with one element at a time, 21.2 us, which is why it works on pairs).
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
// System/6000 processor", 1990), on fp32 pairs: 3 instructions for two elements
// instead of called divisions, which bounded the kernel. All three terms carry
// the opposite sign (t = -q), so that x = -0 keeps its sign, and the codes' sign
// bits are turned round at the end. x is first held at +-512 s rounded up to
// bf16 (any code from 464 s on is 448), so that an infinite or overflowing
// quotient never meets the correction; NaN stays NaN. Scales so small or large that
// a bound or the last bits of a residual leave the normal numbers take the division.
struct CodeScale {
  float s, r;
  uint32_t lim;  // bf16x2
  bool plain;
  __device__ __forceinline__ explicit CodeScale(float scale)
      : s(scale), r(1.0f / scale), plain(scale > 1e-26f && scale < 1e30f) {
    const uint32_t b = __bfloat16_as_ushort(__float2bfloat16_ru(512.0f * scale));
    lim = b | b << 16;
  }
  // Codes of minus the quotients of two elements.
  __device__ __forceinline__ uint32_t pair(uint32_t x) const {
    asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(x) : "r"(lim));
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(x) : "r"(lim ^ 0x80008000u));
    const float x0 = __uint_as_float(x << 16), x1 = __uint_as_float(x & 0xffff0000u);
    float t0, t1, e0, e1;
    ffma2(x0, x1, -r, -r, -0.0f, -0.0f, t0, t1);
    ffma2(t0, t1, s, s, x0, x1, e0, e1);
    ffma2(e0, e1, -r, -r, t0, t1, t0, t1);
    return pack_e4m3x2(t0, t1);
  }
  __device__ __noinline__ static uint32_t divided(uint32_t x, float s) {
    return pack_e4m3x2(__fdiv_rn(__uint_as_float(x << 16), s), __fdiv_rn(__uint_as_float(x & 0xffff0000u), s));
  }
  __device__ __forceinline__ uint32_t codes(uint32_t b01, uint32_t b23) const {
    if (!plain) return divided(b01, s) | divided(b23, s) << 16;
    return (pair(b01) | pair(b23) << 16) ^ 0x80808080u;
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
