// Attention of few query rows per request over a paged cache (decoding, and
// checking a handful of drafted tokens): G query heads of a key/value head
// times nq new tokens give at most 8 * NT rows.
//
//   O[r] = sum_j p_rj V_j / sum_j p_rj,   p_rj = 2^(c S_rj - m_r),  S = Q K^T
//
// with one pass over the keys, the running maximum m and sum l of each row in
// registers. Every key and value is read once and used for a few rows, so the
// kernel is bound by HBM; what it has to do is keep loads in flight on every
// SM, whatever the lengths.
//
// Split. The keys of every (request, key/value head) are cut into tiles (dec_keys),
// the tiles of the whole batch form one line, and each of the resident blocks
// takes an equal run of it: a long context is spread over many blocks and short
// ones share a block. A unit whose tiles lie in several blocks leaves (m, l, O)
// per block in the workspace, and a second kernel joins them in block order,
// so results do not depend on timing. Blocks find their run from the lengths in
// device memory.
//
// Block: one warp copies pages to a ring of stages in shared memory (TMA, one
// box per page piece and 128-byte column block, 128-byte swizzle; what lies
// behind the last page is read as zeros through an out-of-range page number);
// four warps take a quarter of each stage's keys each. S^T = K Q^T (16 keys x 8 rows)
// puts the keys on the M side of mma.sync.m16n8k16, so that 4 to 8 rows fill the
// N side of 8 instead of wasting half of M = 16; P^T goes from accumulator to B
// operand with movmatrix; O^T = V^T P^T. The tensor cores' own rate is of no
// concern here: 16 products per 8 KB of cache.
//
// Measured (G = 4, Hkv = 8, d = 128): 64 requests of up to 16k keys, bf16, 1.88 GB
// of cache: 278-290 us, 6.5-6.75 TB/s, what a plain copy reaches; 24 requests of 9-32k
// keys, e4m3, 1.0 GB: 168-176 us, 5.65-5.95 TB/s, held back by the conversions (31% of the
// issue slots in bursts between the products); one request of 4096 keys: 9.1 us, of
// which two launches and the join are about 6. 16 heads of 192/128, 32 requests of
// 1-16k keys: bf16 462-474 us (6.8-7.0 TB/s), e4m3 282-298 us (5.4-5.7 TB/s). 12 rows of
// 24 requests, e4m3: 182-187 us.
//
// e4m3 caches: codes become fp16 exactly (cvt.rn.f16x2.e4m3x2), Q is brought to
// fp16 by a power of two per row (its largest element in [1/2, 1): every bf16
// above 2^-16 of it keeps all its bits), P is fp16; the scales of K and V go
// into the softmax factor and the output. The probabilities are rounded to 16 bits
// for the second product (bf16, or fp16 as kHalfExp says) and summed as they were:
// the product's operands have one type, and a second part of P would double it. A
// row's largest is exactly 1 here, so the result is hardly further from 64 bits (0.0018
// of its size rms, bf16) than its own rounding (0.0017).
#pragma once

#include "paged_common.cuh"

namespace b200p {

constexpr int kDecWarps = 4;     // consumer warps
// Keys per tile (one stage of the ring): 16 per warp, of an e4m3 cache 32, whose
// two groups' conversions and products fill each other's gaps (24 requests of 9-32k
// keys 182 -> 170 us). At 192 two stages of that size would not fit two blocks an SM.
__host__ __device__ constexpr int dec_keys(bool fp8, int d_qk) { return fp8 && d_qk == 128 ? 128 : 64; }
constexpr int kDecThreads = 32 * (kDecWarps + 1);
constexpr int kDecMaxBlocks = 480;  // workspace slots are sized for this many blocks
constexpr int kDecMaxRows = 16;

template <int DQK, int DV, bool FP8, int NT>
struct DecCfg {
  static constexpr int ESZ = FP8 ? 1 : 2;
  static constexpr int KC = (DQK * ESZ + 127) / 128;  // 128-byte column blocks of a K row
  static constexpr int VC = (DV * ESZ + 127) / 128;
  static constexpr int KEYS = dec_keys(FP8, DQK), KG = KEYS / (16 * kDecWarps);  // groups of 16 keys per warp and tile
  static constexpr int CHUNK = KEYS * 128;  // one column block of a tile
  static constexpr int K_BYTES = KC * CHUNK, V_BYTES = VC * CHUNK;
  static constexpr int STAGE = K_BYTES + V_BYTES;
  static constexpr int MROW = DV + 4;                           // floats per row there (bank offset of 8 for two rows)
  static constexpr int MERGE = kDecWarps * 8 * MROW * 4;  // O of the four warps, eight rows at a time
  static constexpr int ML = kDecWarps * 8 * 2 * 4;      // their (m, l)
  static constexpr int FIXED = MERGE + ML + 512 /*barriers, plan*/ + 1024 /*alignment*/;
  // Blocks per SM. Two are enough to stream bf16 pages; with e4m3 a tile is half
  // the bytes for more instructions, and where a warp has 16 keys of it (192/128) a
  // third block's warps fill the gaps: 32 requests of 1-16k keys 283 us for 284.6 with
  // two, 4 of 1-8k 20.8 for 21.4, 24 of 4-16k with 32/8 heads 112.0 for 113.5.
  static constexpr int BLOCKS = FP8 && NT == 1 && KG == 1 ? 3 : 2;
  static constexpr int BUDGET = 227 * 1024 / BLOCKS / 1024 * 1024 - (BLOCKS == 2 ? 0 : 1024);
  static constexpr int FIT = (BUDGET - FIXED) / STAGE;
  static constexpr int STAGES = FIT > 6 ? 6 : FIT;
  static constexpr int SMEM = STAGES * STAGE + FIXED;
  static_assert(STAGES >= 2 && SMEM <= BUDGET, "shared memory");
};

// Tiles of one key/value head of a request: none without new tokens; a request
// without keys still has one, which masks everything.
template <int KEYS>
__device__ __forceinline__ int dec_tiles(const Request& r) {
  return r.nq == 0 ? 0 : max(1, (r.kv + KEYS - 1) / KEYS);
}

// A block's place in the line of tiles: request, head and tile to start at.
struct DecStart {
  int b, h, tile, count, first, total, per;
};

// Every thread of the block; `sm`: kDecThreads + 8 ints of shared memory.
template <int KEYS>
__device__ __forceinline__ DecStart dec_start(const PagedAttn& p, int* sm) {
  const int tid = threadIdx.x;
  // thread t sums requests [t * seg, (t + 1) * seg)
  const int seg = (p.B + kDecThreads - 1) / kDecThreads;
  const int b0 = min(tid * seg, p.B), b1 = min(b0 + seg, p.B);
  int sum = 0;
  for (int b = b0; b < b1; ++b) sum += dec_tiles<KEYS>(paged_request(p, b, blockIdx.x == 0));
  sm[tid] = sum;
  if (tid < 3) sm[kDecThreads + 1 + tid] = 0;
  __syncthreads();
  if (tid < 32) {
    constexpr int per_lane = kDecThreads / 32;
    int v[per_lane], s = 0;
#pragma unroll
    for (int i = 0; i < per_lane; ++i) {
      v[i] = s;
      s += sm[tid * per_lane + i];
    }
    int inc = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (tid >= o) inc += u;
    }
#pragma unroll
    for (int i = 0; i < per_lane; ++i) sm[tid * per_lane + i] = inc - s + v[i];
    if (tid == 31) sm[kDecThreads] = inc;
  }
  __syncthreads();
  DecStart d;
  d.total = sm[kDecThreads] * p.Hkv;
  d.per = (d.total + gridDim.x - 1) / static_cast<int>(gridDim.x);
  d.first = blockIdx.x * d.per;
  d.count = max(0, min(d.per, d.total - d.first));
  if (d.count > 0) {
    const int mine = sm[tid] * p.Hkv;
    if (mine <= d.first && d.first < mine + sum * p.Hkv) {
      int acc = mine;
      for (int b = b0; b < b1; ++b) {
        const int n = dec_tiles<KEYS>(paged_request(p, b, false));
        if (d.first < acc + n * p.Hkv) {
          sm[kDecThreads + 1] = b;
          sm[kDecThreads + 2] = (d.first - acc) / n;
          sm[kDecThreads + 3] = (d.first - acc) % n;
          break;
        }
        acc += n * p.Hkv;
      }
    }
  }
  __syncthreads();
  d.b = sm[kDecThreads + 1];
  d.h = sm[kDecThreads + 2];
  d.tile = sm[kDecThreads + 3];
  return d;
}

// Walks the units of a block's run in order.
template <int KEYS>
struct DecWalk {
  const PagedAttn& p;
  Request r;
  int b, h, k0, n, left, at;  // unit (b, h): tiles [k0, k0 + n) of its `tiles`; `left` after it; `at` its place in the line
  int tiles;
  __device__ DecWalk(const PagedAttn& params, const DecStart& d) : p(params) {
    b = d.b;
    h = d.h;
    k0 = d.tile;
    left = d.count;
    at = d.first;
    n = 0;
    if (left > 0) {
      r = paged_request(p, b, false);
      tiles = dec_tiles<KEYS>(r);
      n = min(left, tiles - k0);
      left -= n;
    }
  }
  __device__ bool valid() const { return n > 0; }
  __device__ void next() {
    at += n;
    if (left == 0) {
      n = 0;
      return;
    }
    k0 = 0;
    if (++h == p.Hkv) {
      h = 0;
      do {  // more tiles are left, so a request with tiles follows
        if (++b >= p.B) {
          n = left = 0;
          return;
        }
        r = paged_request(p, b, false);
        tiles = dec_tiles<KEYS>(r);
      } while (tiles == 0);
    }
    n = min(left, tiles);
    left -= n;
  }
};

template <int DQK, int DV, bool FP8, int NT>
__global__ void __launch_bounds__(kDecThreads, DecCfg<DQK, DV, FP8, NT>::BLOCKS)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const PagedAttn p) {
  using C = DecCfg<DQK, DV, FP8, NT>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* gen = smem_raw + (base - raw);
  float* s_merge = reinterpret_cast<float*>(gen + C::STAGES * C::STAGE);  // [warp][row][DV]
  float* s_ml = s_merge + C::MERGE / 4;                                  // [warp][row][2]
  const uint32_t s_bar = base + C::STAGES * C::STAGE + C::MERGE + C::ML;
  uint8_t* bar_gen = gen + C::STAGES * C::STAGE + C::MERGE + C::ML;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bar_gen + 16 * C::STAGES);
  int* s_plan = reinterpret_cast<int*>(s_merge);  // before the first merge
  const uint32_t bFull = s_bar, bEmpty = s_bar + 8 * C::STAGES;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(bFull + 8 * s, 1);
      mbar_init(bEmpty + 8 * s, kDecWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  pdl_wait();
  const DecStart d = dec_start<C::KEYS>(p, s_plan);  // its barriers order the set-up above too
  __syncthreads();
  if (threadIdx.x == 0) reinterpret_cast<PartDesc*>(p.desc)[blockIdx.x].last = -1;

  if (warp == kDecWarps) {
    // ------------------------------------------------------------ copies
    const int boxes = C::KEYS / p.box;  // per tile
    const int issues = boxes * (C::KC + C::VC);
    const int ahead = 32 / boxes;        // tiles whose page numbers one load of the warp covers: a power of two
    uint32_t it = 0;
    bool ok = true;
    for (DecWalk<C::KEYS> w(p, d); ok && w.valid(); w.next()) {
      int page = 0;
      for (int k = 0; k < w.n; ++k, ++it) {
        const int kt = w.k0 + k, a = k & (ahead - 1);
        if (a == 0) page = lane < ahead * boxes ? paged_page(p, w.b, kt * C::KEYS + lane * p.box, w.r.kv) : 0;
        const uint32_t s = it % C::STAGES;
        if (it >= C::STAGES) {
          ok = paged_wait(bEmpty + 8 * s, ((it / C::STAGES) - 1) & 1, abort_flag);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
        }
        if (lane == 0) mbar_arrive_expect_tx(bFull + 8 * s, C::STAGE);
        __syncwarp();
        const int box = lane / (C::KC + C::VC), c = lane % (C::KC + C::VC);
        const int pg = __shfl_sync(0xffffffffu, page, a * boxes + (lane < issues ? box : 0));
        if (lane < issues) {
          const int row = paged_row(p, kt * C::KEYS + box * p.box);
          const uint32_t dst = base + s * C::STAGE + c * C::CHUNK + box * p.box * 128;
          if (c < C::KC)
            tma_load_4d(dst, &tmK, bFull + 8 * s, c * (128 / C::ESZ), w.h, row, pg);
          else
            tma_load_4d(dst, &tmV, bFull + 8 * s, (c - C::KC) * (128 / C::ESZ), w.h, row, pg);
        }
      }
    }
    if (!ok) __nanosleep(200000);  // copies in flight land before the block ends
  } else {
    // ------------------------------------------------------------ products
    uint32_t it = 0;
    bool ok = true;
    const int key0 = 16 * C::KG * warp;  // this warp's keys of a tile
    const int mrow = (lane & 15), mhalf = lane >> 4;
    for (DecWalk<C::KEYS> w(p, d); w.valid(); w.next()) {
      const int nrows = w.r.nq * p.G;
      // Q^T as B operand: row n = lane / 4 of each group of eight
      constexpr int KS = DQK / 16;
      uint32_t qf[NT][KS][2];
      float cs[NT][2];  // softmax factor of the rows this lane holds scores of
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int r = 8 * j + (lane >> 2);
        const bool has = r < nrows;
        const int tok = has ? r / p.G : 0;
        const __nv_bfloat16* q = p.q + (w.r.t0 + tok) * p.q_stride +
                                 static_cast<int64_t>(w.h * p.G + (has ? r - tok * p.G : 0)) * DQK;
        float row_c = p.scale_log2;
        if constexpr (!FP8) {
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const uint32_t* s = reinterpret_cast<const uint32_t*>(q + 16 * k + 2 * (lane & 3));
            qf[j][k][0] = has ? __ldg(s) : 0u;
            qf[j][k][1] = has ? __ldg(s + 4) : 0u;
          }
        } else {
          // codes 4c .. 4c + 3 of a unit of 16 are what one lane gets of K: the
          // contraction runs over d in that order
          float amax = 0.0f;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const uint2 v = has ? __ldg(reinterpret_cast<const uint2*>(q + 16 * k + 4 * (lane & 3))) : make_uint2(0, 0);
            qf[j][k][0] = v.x;
            qf[j][k][1] = v.y;
            amax = fmaxf(amax, fmaxf(fmaxf(fabsf(__uint_as_float(v.x << 16)), fabsf(__uint_as_float(v.x & 0xffff0000u))),
                                     fmaxf(fabsf(__uint_as_float(v.y << 16)), fabsf(__uint_as_float(v.y & 0xffff0000u)))));
          }
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
          int e = 0;
          if (amax > 0.0f && amax < INFINITY) e = max(-126, min(126, static_cast<int>(__float_as_uint(amax) >> 23) - 126));
          const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
          const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              qf[j][k][i] = pack_f16x2(__uint_as_float(qf[j][k][i] << 16) * down,
                                       __uint_as_float(qf[j][k][i] & 0xffff0000u) * down);
          row_c *= up * __ldg(p.k_scale + w.h);
        }
        cs[j][0] = __shfl_sync(0xffffffffu, row_c, 8 * (lane & 3));
        cs[j][1] = __shfl_sync(0xffffffffu, row_c, 8 * (lane & 3) + 4);
      }
      // last key each of this lane's rows sees
      int see[NT][2];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = 8 * j + 2 * (lane & 3) + i;
          see[j][i] = p.causal ? min(w.r.kv - w.r.nq + r / p.G, w.r.kv - 1) : w.r.kv - 1;
        }
      const int all_see = p.causal ? w.r.kv - w.r.nq : w.r.kv - 1;  // keys up to here are visible to every row

      float m[NT][2], l[NT][2];
      float o[DV / 16][NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j) m[j][0] = m[j][1] = -INFINITY, l[j][0] = l[j][1] = 0.0f;
#pragma unroll
      for (int t = 0; t < DV / 16; ++t)
#pragma unroll
        for (int j = 0; j < NT; ++j) o[t][j][0] = o[t][j][1] = o[t][j][2] = o[t][j][3] = 0.0f;

      for (int k = 0; k < w.n; ++k, ++it) {
        const uint32_t s = it % C::STAGES;
        // After a wait that ran out the warp goes on without waiting, so that it
        // meets the others at their barriers; the status word voids the result.
        if (ok) ok = paged_wait(bFull + 8 * s, (it / C::STAGES) & 1, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        const uint32_t sk = base + s * C::STAGE, sv = sk + C::K_BYTES;
        const int kv0 = (w.k0 + k) * C::KEYS + key0;  // first key of this warp
        if (kv0 + 16 * C::KG > w.r.kv) {
          // Rows behind the last key may hold anything; a probability of zero
          // does not silence a NaN, so their values are cleared.
          const int from = max(0, w.r.kv - kv0);
          for (int i = lane; i < (16 * C::KG - from) * C::VC * 8; i += 32) {
            const int row = key0 + from + i / (C::VC * 8), c = (i / 8) % C::VC;
            st_shared_v4(sv + c * C::CHUNK + row * 128 + 16 * (i & 7), 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        // S^T = K Q^T; the products of even and odd steps in accumulators of their own
        float sc[C::KG][NT][4], sd[C::KG][NT][4];
#pragma unroll
        for (int gi = 0; gi < C::KG; ++gi)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[gi][j][i] = sd[gi][j][i] = 0.0f;
        if constexpr (!FP8) {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            const int u = 2 * ks + mhalf, row = key0 + mrow;
            uint32_t a[4];
            ldsm_x4(sk + (u >> 3) * C::CHUNK + row * 128 + (((u & 7) ^ (row & 7)) << 4), a);
#pragma unroll
            for (int j = 0; j < NT; ++j)
              mma16816<false>((ks & 1) ? sd[0][j] : sc[0][j], a, qf[j][ks][0], qf[j][ks][1]);
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < KS; ks += 2) {
#pragma unroll
            for (int gi = 0; gi < C::KG; ++gi) {
              const int u = ks + mhalf, row = key0 + 16 * gi + mrow;
              uint32_t c[4];  // (keys 0-7, 8-15) of unit ks, then of unit ks + 1
              ldsm_x4(sk + (u >> 3) * C::CHUNK + row * 128 + (((u & 7) ^ (row & 7)) << 4), c);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t a[4] = {e4m3x2_f16x2(c[2 * i]), e4m3x2_f16x2(c[2 * i + 1]),
                                       e4m3x2_f16x2(c[2 * i] >> 16), e4m3x2_f16x2(c[2 * i + 1] >> 16)};
#pragma unroll
                for (int j = 0; j < NT; ++j)
                  mma16816<true>(i ? sd[gi][j] : sc[gi][j], a, qf[j][ks + i][0], qf[j][ks + i][1]);
              }
            }
          }
        }
        uint32_t pb[C::KG][NT][2];
        float alpha[NT][2];
        bool moved = false;
        const bool edge = kv0 + 16 * C::KG - 1 > all_see;
        const int kl = kv0 + (lane >> 2);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          float x[C::KG][4];
#pragma unroll
          for (int gi = 0; gi < C::KG; ++gi)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[gi][i] = (sc[gi][j][i] + sd[gi][j][i]) * cs[j][i & 1];
              if (edge && kl + 16 * gi + 8 * (i >> 1) > see[j][i & 1]) x[gi][i] = -INFINITY;
            }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float mx = fmaxf(x[0][i], x[0][i + 2]);
#pragma unroll
            for (int gi = 1; gi < C::KG; ++gi) mx = fmaxf(mx, fmaxf(x[gi][i], x[gi][i + 2]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            if constexpr (FP8) mx -= kHalfExp;
            const float mn = fmaxf(m[j][i], mx);
            alpha[j][i] = mn > m[j][i] ? ex2_approx(m[j][i] - mn) : 1.0f;
            moved |= mn > m[j][i];
            m[j][i] = mn;
            const float ref = mn == -INFINITY ? 0.0f : mn;  // nothing seen yet: every probability is 0
            float sum = 0.0f;
#pragma unroll
            for (int gi = 0; gi < C::KG; ++gi) {
              x[gi][i] = ex2_approx(x[gi][i] - ref);
              x[gi][i + 2] = ex2_approx(x[gi][i + 2] - ref);
              sum += x[gi][i] + x[gi][i + 2];
            }
            l[j][i] = fmaf(l[j][i], alpha[j][i], sum);
          }
#pragma unroll
          for (int gi = 0; gi < C::KG; ++gi) {
            // (held at fp16's largest: where scores above 2^24 are rounded, m - 15 may be m - 16)
            pb[gi][j][0] = movm_t(FP8 ? pack_f16x2_sat(x[gi][0], x[gi][1]) : pack_bf16x2(x[gi][0], x[gi][1]));
            pb[gi][j][1] = movm_t(FP8 ? pack_f16x2_sat(x[gi][2], x[gi][3]) : pack_bf16x2(x[gi][2], x[gi][3]));
          }
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int t = 0; t < DV / 16; ++t)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[t][j][i] *= alpha[j][i & 1];
        }
        // O^T += V^T P^T
        if constexpr (!FP8) {
#pragma unroll
          for (int t = 0; t < DV / 16; ++t) {
            // matrices (keys 0-7, d 0-7), (keys 0-7, d 8-15), (keys 8-15, d 0-7), (keys 8-15, d 8-15)
            const int row = key0 + ((lane >> 4) << 3) + (lane & 7), u = 2 * t + ((lane >> 3) & 1);
            uint32_t a[4];
            ldsm_x4_t(sv + (u >> 3) * C::CHUNK + row * 128 + (((u & 7) ^ (row & 7)) << 4), a);
#pragma unroll
            for (int j = 0; j < NT; ++j) mma16816<false>(o[t][j], a, pb[0][j][0], pb[0][j][1]);
          }
        } else {
#pragma unroll
          for (int t = 0; t < DV / 16; t += 2) {
#pragma unroll
            for (int gi = 0; gi < C::KG; ++gi) {
              // (keys 0-7, 8-15) of unit t, then of unit t + 1; a transposed pair of
              // codes is (d = 2g, 2g + 1): even d on rows 0-7 of M, odd on 8-15
              const int row = key0 + 16 * gi + (lane & 15), u = t + mhalf;
              uint32_t c[4];
              ldsm_x4_t(sv + row * 128 + ((u ^ (row & 7)) << 4), c);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t lo = c[2 * i], hi = c[2 * i + 1];
                const uint32_t a[4] = {e4m3x2_f16x2(prmt(lo, 0u, 0x4420u)), e4m3x2_f16x2(prmt(lo, 0u, 0x4431u)),
                                       e4m3x2_f16x2(prmt(hi, 0u, 0x4420u)), e4m3x2_f16x2(prmt(hi, 0u, 0x4431u))};
#pragma unroll
                for (int j = 0; j < NT; ++j) mma16816<true>(o[t + i][j], a, pb[gi][j][0], pb[gi][j][1]);
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bEmpty + 8 * s);
      }

      // ---------------------------------------------------------- the unit's end: join the four warps
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          l[j][i] += __shfl_xor_sync(0xffffffffu, l[j][i], 4);
          l[j][i] += __shfl_xor_sync(0xffffffffu, l[j][i], 8);
          l[j][i] += __shfl_xor_sync(0xffffffffu, l[j][i], 16);
        }
      const bool whole = w.n == w.tiles;
      const bool head = w.k0 > 0;  // the unit began in an earlier block
      const int slot = 2 * blockIdx.x + (head ? 0 : 1);
      const int td = threadIdx.x;  // one output column per thread
      static_assert(DV == 32 * kDecWarps, "one column per thread");
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (8 * j >= nrows) break;
        named_bar_sync(1, 32 * kDecWarps);  // the buffer's last readers are done
        if (lane < 4) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            s_ml[(warp * 8 + 2 * lane + i) * 2] = m[j][i];
            s_ml[(warp * 8 + 2 * lane + i) * 2 + 1] = l[j][i];
          }
        }
#pragma unroll
        for (int t = 0; t < DV / 16; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 2 * (lane & 3) + (i & 1);
            const int dd = 16 * t + (FP8 ? 2 * (lane >> 2) + (i >> 1) : (lane >> 2) + 8 * (i >> 1));
            s_merge[(warp * 8 + r) * C::MROW + dd] = o[t][j][i];
          }
        named_bar_sync(1, 32 * kDecWarps);
        for (int r8 = 0; r8 < 8 && 8 * j + r8 < nrows; ++r8) {
          const int r = 8 * j + r8;
          float mm = -INFINITY;
#pragma unroll
          for (int v = 0; v < kDecWarps; ++v) mm = fmaxf(mm, s_ml[(v * 8 + r8) * 2]);
          const float ref = mm == -INFINITY ? 0.0f : mm;
          float ll = 0.0f, acc = 0.0f;
#pragma unroll
          for (int v = 0; v < kDecWarps; ++v) {
            const float f = ex2_approx(s_ml[(v * 8 + r8) * 2] - ref);
            ll = fmaf(s_ml[(v * 8 + r8) * 2 + 1], f, ll);
            acc = fmaf(s_merge[(v * 8 + r8) * C::MROW + td], f, acc);
          }
          if (whole) {
            const int tok = r / p.G, hq = w.h * p.G + r - tok * p.G;
            const float x = ll == 0.0f ? 0.0f : acc * (1.0f / ll) * (FP8 ? __ldg(p.v_scale + w.h) : 1.0f);
            p.o[(static_cast<int64_t>(w.r.t0 + tok) * p.Hq + hq) * DV + td] = __float2bfloat16(x);
            if (p.lse != nullptr && td == 0)
              p.lse[static_cast<int64_t>(hq) * p.T + w.r.t0 + tok] =
                  ll == 0.0f ? -INFINITY : (mm + fast_log2(ll)) * kLn2;
          } else {
            p.part_o[(static_cast<int64_t>(slot) * p.slot_rows + r) * DV + td] = acc;
            if (td < 2) p.part_ml[(slot * p.slot_rows + r) * 2 + td] = td == 0 ? mm : ll;
          }
        }
      }
      if (!whole && !head && td == 0) {
        PartDesc e;
        e.last = (w.at + w.tiles - 1) / d.per;  // the block that has the unit's last tile
        e.t0 = w.r.t0;
        e.row0 = 0;
        e.nrows = nrows;
        e.hkv = w.h;
        e.pad[0] = e.pad[1] = e.pad[2] = 0;
        reinterpret_cast<PartDesc*>(p.desc)[blockIdx.x] = e;
      }
    }
  }
}

}  // namespace b200p
