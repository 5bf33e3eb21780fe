// Attention of a chunk of new tokens over a paged cache: the many-rows half of
// b200attn_paged_fwd (prompts read in pieces, drafted tokens, mixed steps).
//
//   O[r] = sum_j p_rj V_j / sum_j p_rj,  p_rj = 2^(c S_rj - m_r),  S = Q K^T
//
// on tcgen05, by the scheme of the prefill kernel: 128 x 128 score tiles into
// tensor memory, one thread per row for the softmax, P back to tensor memory,
// O accumulated there, two row tiles per block sharing each key block.
//
// Rows. The G query heads of a key/value head see the same keys, so a tile's
// rows are (token, head) pairs: floor(128 / G) tokens times G heads. A chunk of
// a few tokens then fills G times more rows of the tensor core's M = 128 than a
// tile per head, and each key block is read once for all G heads. One TMA box
// {64 columns, G heads, tokens} lays the rows out so.
//
// Split. A unit is (request, key/value head, pair of row tiles) and runs over
// its key blocks of 128. The blocks of all units (and a fixed cost per unit) form
// one line that is cut into equal runs, one per SM: a step of few units still uses every SM, and no SM
// waits for a longer unit. A unit cut by a run's end leaves (m, l, O) per part,
// joined in block order (paged_join.cuh). Every block finds its run from the
// lengths in device memory.
//
// Keys and values. One warp copies K, one V, page piece by page piece (TMA,
// 128-byte swizzle; pages behind the last are read as zeros through an
// out-of-range page number). The rows behind the last key inside its page may
// hold anything, and 0 * NaN is NaN, so the V warp clears them in shared memory
// before the tensor core reads them; scores are replaced by select.
//
// e4m3 caches. S = Q K^T stays in e4m3 on the K side without losing Q: after a
// power of two per row (its largest element in [2^7, 2^8)), a bf16 number is the
// sum of two e4m3 numbers -- the one nearest to it (4 bits) and the rest (4
// bits) -- exactly for elements within 2^-10 of the row's largest, to 2^-18 of it
// below. Both halves are products of kind::f8f6f4 into one accumulator, at twice
// the rate of 16 bits each, so K's codes go to the tensor core as they are. P
// would need the same split in the softmax, the busiest warps here; instead V's
// codes become fp16 (exactly) in shared memory, by the two copying warps, and P
// is fp16. Converting K as well, with four more warps, took 503 us where this
// took 395 then (4 requests of 500-1300 new tokens, 2-12k keys).
//
// P is rounded to 16 bits for the second product (bf16, or fp16 as ch_p_exp says) and
// summed in fp32 as it was: both operands of a product have one type, and a second
// part of P would be half as many products again. With bf16 the result is 0.0023 of its
// size (rms) off the one in 64 bits, its own rounding alone 0.0017, each the same half
// step; with fp16 0.0017.
//
// Bound by the tensor core (2 x 2 x 128^3 products per key block and pair) and,
// for chunks of a few tokens, by reading the cache. Measured, a call: 4096 tokens over
// 32k keys (32/8 heads of 128, bf16) 1.65-1.72 ms, 1200-1250 TFLOP/s under the power cap,
// tensor pipe 79% busy, MUFU 80%; ragged chunks of 1-1500 tokens 183-188 us (53%: each
// SM's run begins with an empty pipeline and ends with a part to write and join); the
// same kind over an e4m3 cache 344-353 us (52%); 192/128 heads 246-250 us (57%), e4m3
// 215-221 us; 32 requests of 3-9 drafted tokens 128-134 us, 4.8-5.0 TB/s of cache.
#pragma once

#include "paged_common.cuh"

namespace b200p {

constexpr int kChM = 128;  // rows per tile
constexpr int kChN = 128;  // keys per block
constexpr int kChRows = 2 * kChM;
// What a unit costs beyond its key blocks (its Q, the pipeline's filling, its
// output), in key blocks: counted in when the line is cut, so that a run of many
// short units is not longer than one of few long ones. Measured on ragged chunks
// of 1-1500 tokens and on one 2048-token prompt: 2 blocks 185 and 50.8 us, 3 186
// and 49.9, 4 188 and 50.4, 5 189 and 50.3; a first form of the kernel, slower at
// a unit's ends, took 228 and 88 us with 1 for 200 and 74 with 3.
constexpr int kChUnitCost = 3;
constexpr int kChMaxBlocks = 160;  // workspace slots are sized for this many blocks

constexpr int kChUnits = 8;  // units the K warp may be ahead by; more than the blocks its ring holds

template <int DQK, int DV, bool FP8>
struct ChCfg {
  static constexpr int THREADS = 384, REGS_LAUNCH = 168;
  // Register split by warpgroup: copies and issue, softmax; the sum stays within
  // what the block was launched with. The warps that convert V need more, for the
  // copies' places at 192 most (e4m3 chunks of 128 and 192/128: 88 and 208 registers
  // 352 and 258 us, 104 and 200 360 and 250, 120 and 192 372 and 252).
  static constexpr int REGS_CTRL = FP8 ? (DQK == 128 ? 88 : 104) : 72, REGS_SOFT = FP8 && DQK != 128 ? 200 : 208;
  static_assert(128 * REGS_CTRL + 256 * REGS_SOFT <= THREADS * REGS_LAUNCH, "registers");
  static constexpr int CHUNK = kChM * 128;  // 128 rows x 128 bytes, swizzled
  static constexpr int KSZ = FP8 ? 1 : 2;
  static constexpr int Q_CHUNKS = 2 * DQK / 128;  // bf16, or two halves of codes side by side
  static constexpr int K_CHUNKS = (DQK * KSZ + 127) / 128, V_CHUNKS = DV / 64;
  static constexpr int Q_BYTES = Q_CHUNKS * CHUNK, K_BYTES = K_CHUNKS * CHUNK, V_BYTES = V_CHUNKS * CHUNK;
  static constexpr int STAGES = FP8 ? (DQK == 128 ? 3 : 2) : 0, VC_BYTES = kChN * DV;  // staged codes of V
  static constexpr int AVAIL = 227 * 1024 - 2048 - 2 * Q_BYTES - STAGES * VC_BYTES;
  static constexpr int PAIRS = AVAIL / (K_BYTES + V_BYTES);
  static constexpr int SV = PAIRS >= 2 ? 2 : 1;
  static constexpr int SK_FIT = (AVAIL - SV * V_BYTES) / K_BYTES, SK = SK_FIT > 4 ? 4 : SK_FIT;
  static constexpr int BARS = 2 + 2 + 2 * SK + 2 * SV + 1 + 6 + 2 + 1 + 2 + 2 + 2 + 2 + 2 + 2 * kChUnits;
  static constexpr int SMEM = 2 * Q_BYTES + SK * K_BYTES + SV * V_BYTES + STAGES * VC_BYTES + 1024 + 1024;
  static_assert(8 * BARS + 8 <= 512 && 512 + kChUnits * 64 <= 1024 && SMEM <= 227 * 1024 && SK >= 2, "shared memory");
  // Tensor memory: S [0, 128) for both tiles in turn, O_t at 128 + 128 t, P_t
  // (16-bit, 64 columns) at 384 + 64 t.
  static constexpr int TM_O = 128, TM_P = 384;
  // Instruction descriptors: kind::f16 with bf16 (format 1), or kind::f8f6f4 with
  // e4m3 (0) for S and kind::f16 with fp16 (0) for O.
  static constexpr uint32_t FMT = FP8 ? 0u : 1u;
  static constexpr uint32_t IDESC_QK = idesc_dense(FMT, FMT, kChM, kChN, false);
  static constexpr uint32_t IDESC_PV = idesc_dense(FMT, FMT, kChM, DV, true);
  static constexpr float P_MAX = FP8 ? kHalfExp : 16.0f;  // probabilities reach 2^P_MAX
};

// Exponent that the largest probability of a row gets when its reference is moved;
// it may then grow to P_MAX, by 16 (bf16), 8 or 2 binades, before O is rescaled. The
// fp16 P of up to kChLongKeys keys lose at most n 2^-32 of a row's largest by rounding
// (2^-12), those of more n 2^-38 (2^-8 at 2^30 keys). Room of 8, 4, 2 and 0 binades takes
// 348, 353, 361 and 371 us for e4m3 chunks over 2-12k keys, of 16, 8, 4 and 0 1678, 1682,
// 1704 and 1788 us for the long bf16 chunk; over many keys the maximum hardly moves.
constexpr int kChLongKeys = 1 << 20;
template <bool FP8>
__device__ __forceinline__ float ch_p_exp(int kv) {
  return !FP8 ? 0.0f : (kv <= kChLongKeys ? kHalfExp - 8.0f : kHalfExp - 2.0f);
}

// Key blocks of row tile `tile` of a request: 0 if the tile has no token; one
// that masks everything for tokens that see no key.
__device__ __forceinline__ int ch_blocks(const Request& r, int tile, int tpt, int causal) {
  const int first = tile * tpt;
  if (first >= r.nq) return 0;
  const int seen = causal ? r.kv - r.nq + min(r.nq, first + tpt) : r.kv;
  return max(1, (min(seen, r.kv) + kChN - 1) / kChN);
}

// Key blocks of pair `p`: its last tile that exists has most.
__device__ __forceinline__ int ch_pair_blocks(const Request& r, int p, int tpt, int causal) {
  return max(ch_blocks(r, 2 * p, tpt, causal), ch_blocks(r, 2 * p + 1, tpt, causal));
}

// sum of floor(i / 2^k) over i = 0 .. x - 1
__device__ __forceinline__ int shift_sum(int x, int k) {
  const int t = x >> k;
  return (static_cast<int>(static_cast<int64_t>(t) * (t - 1) / 2) << k) + t * (x - (t << k));
}

// sum of floor((a i + b) / m) over i = 0 .. n - 1 (a, b >= 0; m = kChN, a power of
// two): in closed form if a is one too, else by exchanging the roles of a and m as
// in Euclid's algorithm: a few steps, whatever n (such sums and their reciprocity:
// Graham, Knuth and Patashnik, "Concrete Mathematics", 1989, section 3.5).
__device__ __forceinline__ int floor_sum(int n, int m, int a, int b) {
  int s = 0;
  if ((a & (a - 1)) == 0) {
    if (a >= m) return static_cast<int>(static_cast<int64_t>(n) * (n - 1) / 2) * (a / kChN) + n * (b / kChN);
    const int la = __ffs(a) - 1, u = (b & (kChN - 1)) >> la;
    return n * (b / kChN) + shift_sum(n + u, __ffs(kChN) - 1 - la) - shift_sum(u, __ffs(kChN) - 1 - la);
  }
  while (true) {
    if (a >= m) {
      const int q = a / m;
      s += static_cast<int>(static_cast<int64_t>(n) * (n - 1) / 2) * q;
      a -= q * m;
    }
    if (b >= m) {
      const int q = b / m;
      s += n * q;
      b -= q * m;
    }
    const int64_t y = static_cast<int64_t>(a) * n + b;  // < 2^31 where it goes on: it counts keys
    if (y < m) return s;
    n = static_cast<uint32_t>(y) / static_cast<uint32_t>(m);
    b = static_cast<int>(y) - n * m;
    const int t = m;
    m = a;
    a = t;
  }
}

__device__ __forceinline__ int ch_pairs(const PagedAttn& p, const Request& r, int tpt) {
  return static_cast<uint32_t>(r.nq + 2 * tpt - 1) / p.pair;
}

// Length in the line of the units of one key/value head of a request.
__device__ __forceinline__ int ch_head_cost(const PagedAttn& p, const Request& r, int tpt) {
  const int n = ch_pairs(p, r, tpt);
  if (n == 0) return 0;
  if (!p.causal) return n * (ch_pair_blocks(r, 0, tpt, 0) + kChUnitCost);
  int s = n * kChUnitCost;
  if (n > 4 && r.kv >= r.nq) {
    // every pair but the last sees kv - nq + 2 tpt (i + 1) keys, the last one all
    s += floor_sum(n - 1, kChN, 2 * tpt, r.kv - r.nq + 2 * tpt + kChN - 1) + (r.kv + kChN - 1) / kChN;
  } else {
    for (int i = 0; i < n; ++i) s += ch_pair_blocks(r, i, tpt, 1);
  }
  return s;
}

__device__ __forceinline__ void ld_shared_v4(uint32_t addr, int& a, int& b, int& c, int& d) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr) : "memory");
}

// A block's run: it starts `skip` into unit (b, h, pair), is `count` long, and
// `first` is its place in the line; runs are `per` long.
struct ChStart {
  int b, h, pair, skip, count, first, per;
  Request r;
};

// By one warp of the block.
__device__ __forceinline__ ChStart ch_start(const PagedAttn& p, int tpt) {
  const int lane = threadIdx.x & 31;
  const Run run = plan_run(
      p, [&](const Request& x) { return ch_head_cost(p, x, tpt); },
      [](const Request& x) { return x.nq > 0 ? (x.kv + kChN - 1) / kChN : 0; });
  ChStart d = {run.b, 0, 0, 0, run.count, run.first, run.per, run.req};
  if (run.count == 0) return d;
  const Request r = run.req;
  const int n = max(1, run.cost), pairs = ch_pairs(p, r, tpt);
  d.h = run.off / n;
  int off = run.off - d.h * n;
  for (int i0 = 0; i0 < pairs; i0 += 32) {  // the pair that `off` lies in, 32 at a time
    const int x = i0 + lane < pairs ? ch_pair_blocks(r, i0 + lane, tpt, p.causal) + kChUnitCost : 0;
    int inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, off < inc);
    if (past != 0) {
      const int at = __ffs(past) - 1;
      d.pair = i0 + at;
      d.skip = __shfl_sync(0xffffffffu, off - (inc - x), at);
      return d;
    }
    off -= __shfl_sync(0xffffffffu, inc, 31);
  }
  d.count = 0;  // lengths that changed while being read
  return d;
}

// Walks the pieces of a block's run: key blocks [kb, ke) of unit (b, h, pair).
// A unit takes kChUnitCost + (its key blocks) of the line, the cost first.
// The piece that begins inside a unit comes last, so that every block starts a
// unit at key 0 at the same time: blocks of one key/value head then go over its
// keys together and share them in L2 (one chunk of 4096 tokens over 28k keys read
// 2.7 GB from HBM with the pieces in order, 0.66 GB so).
// Only the K warp walks; the other roles read what it finds (ChUnit).
struct ChWalk {
  const PagedAttn& p;
  const ChStart start;
  bool later;            // the first piece is still to come
  Request r;
  int b, h, pair, tpt;
  int kb, ke, n0, n1;  // this piece; key blocks of the unit's tiles
  int left, at;        // what is left of the run after this piece; the unit's place in the line
  __device__ ChWalk(const PagedAttn& params, const ChStart& s, int tokens)
      : p(params), start(s), later(false), tpt(tokens) {
    kb = ke = 0;
    if (s.count > 0) {
      begin();
      later = kb > 0;
      if (later || !valid()) next();
    }
  }
  __device__ void begin() {
    b = start.b;
    h = start.h;
    pair = start.pair;
    left = start.count;
    at = start.first - start.skip;
    r = start.r;
    take(start.skip);
  }
  __device__ void take(int skip) {
    n0 = ch_blocks(r, 2 * pair, tpt, p.causal);
    n1 = ch_blocks(r, 2 * pair + 1, tpt, p.causal);
    const int n = min(left, max(n0, n1) + kChUnitCost - skip);
    kb = max(0, skip - kChUnitCost);
    ke = max(0, skip + n - kChUnitCost);
    left -= n;
  }
  __device__ bool valid() const { return ke > kb; }
  __device__ bool whole() const { return kb == 0 && ke == max(n0, n1); }
  __device__ int last() const { return at + kChUnitCost + max(n0, n1) - 1; }  // place of the unit's last key block
  __device__ void next() {
    do {
      at += max(n0, n1) + kChUnitCost;
      kb = ke = 0;
      if (left == 0) {
        if (later) {
          begin();
          left = 0;
          later = false;
        }
        return;
      }
      if (++pair == ch_pairs(p, r, tpt)) {
        pair = 0;
        if (++h == p.Hkv) {
          h = 0;
          do {  // more is left, so a request with tokens follows
            if (++b >= p.B) {
              left = later = 0;
              return;
            }
            r = paged_request(p, b, false);
          } while (r.nq == 0);
        }
      }
      take(0);
    } while (!valid());  // the run's end may hold no more than a unit's cost
  }
};

// A piece of work as every role of the block sees it, in a ring of shared memory.
// The K warp fills it as it walks, units ahead of the others: no other role
// computes or keeps the walk (the softmax warps hold a whole score row each), and
// none waits for a request's lengths. kb == ke: the end.
struct ChUnit {
  int b, h, t0, nq;    // request, key/value head, the request's first row of Q, its new tokens
  int kv, tok0, kb, ke;  // its keys; first token of tile 0; key blocks [kb, ke)
  int n0, n1;          // key blocks of the unit's tiles
  int whole;           // the unit is not split
  int last;            // the block that has its last piece
  __device__ int end(int t) const { return min(ke, t ? n1 : n0); }  // tile t runs blocks [kb, end(t))
  __device__ bool has(int t) const { return end(t) > kb; }
  __device__ bool valid() const { return ke > kb; }
  __device__ void put(uint32_t at) const {
    st_shared_v4(at, b, h, t0, nq);
    st_shared_v4(at + 16, kv, tok0, kb, ke);
    st_shared_v4(at + 32, n0, n1, whole, last);
  }
  __device__ void get(uint32_t at) {
    ld_shared_v4(at, b, h, t0, nq);
    ld_shared_v4(at + 16, kv, tok0, kb, ke);
    ld_shared_v4(at + 32, n0, n1, whole, last);
  }
};

__device__ __forceinline__ void st_shared_v2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

__device__ __forceinline__ __half2 bits_half2(uint32_t x) {
  __half2 h;
  memcpy(&h, &x, 4);
  return h;
}

// Largest of two or three; NaN if one of them is.
__device__ __forceinline__ float max2_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// 32 bytes, a whole sector, of one row: with 16 a thread, ragged chunks took 1.5%
// longer.
__device__ __forceinline__ void st_global_32b(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Rows [64 half, 64 half + 64) of a staged 128 x 128 block of V's codes -> the
// fp16 tile, by one warp; rows from `keys` on as zeros. 16 lanes take a row, eight
// codes each: eight lanes' stores are one row of a column block, all 32 banks.
__device__ __forceinline__ void ch_convert_v(const uint2* staged, uint32_t dst, int half, int lane, int keys) {
  const int u = lane & 7;
  const uint32_t col = dst + ((lane >> 3) & 1) * (kChN * 128);
#pragma unroll 1
  for (int g = 0; g < 8; ++g) {
    uint2 c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = staged[(64 * half + 8 * g) * 16 + 32 * i + lane];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 64 * half + 8 * g + 2 * i + (lane >> 4);
      st_shared_v4(col + row * 128 + ((u ^ (row & 7)) << 4), e4m3x2_f16x2(c[i].x), e4m3x2_f16x2(c[i].x >> 16),
                   e4m3x2_f16x2(c[i].y), e4m3x2_f16x2(c[i].y >> 16));
    }
  }
  if (keys < 64 * half + 64) {  // whatever they were converted from
    __syncwarp();
    for (int row = max(keys, 64 * half) + (lane >> 4); row < 64 * half + 64; row += 2)
      st_shared_v4(col + row * 128 + ((u ^ (row & 7)) << 4), 0u, 0u, 0u, 0u);
  }
}

template <int DQK, int DV, bool FP8>
__global__ void __launch_bounds__(ChCfg<DQK, DV, FP8>::THREADS, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const PagedAttn p) {
  using C = ChCfg<DQK, DV, FP8>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* gen = smem_raw + (base - raw);
  const uint32_t sQ = base, sK = sQ + 2 * C::Q_BYTES, sV = sK + C::SK * C::K_BYTES;
  const uint32_t sVc = sV + C::SV * C::V_BYTES, sBar = sVc + C::STAGES * C::VC_BYTES;
  uint8_t* bar_gen = gen + (sBar - base);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_gen + 8 * C::BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bar_gen + 8 * C::BARS + 4);

  const uint32_t bQFull = sBar;                  // [2] Q tile there (TMA, or 128 softmax threads)
  const uint32_t bQEmpty = bQFull + 16;          // [2] the tile's last QK^T has read it
  const uint32_t bKFull = bQEmpty + 16;          // [SK]
  const uint32_t bKEmpty = bKFull + 8 * C::SK;   // [SK]
  const uint32_t bVFull = bKEmpty + 8 * C::SK;   // [SV]
  const uint32_t bVEmpty = bVFull + 8 * C::SV;   // [SV]
  const uint32_t bVTail = bVEmpty + 8 * C::SV;   // a V block whose last rows must be cleared
  const uint32_t bCFull = bVTail + 8;            // [STAGES] staged codes of V (e4m3)
  const uint32_t bCEmpty = bCFull + 24;          // [STAGES] converted
  const uint32_t bSFull = bCEmpty + 24;          // [2]
  const uint32_t bSFree = bSFull + 16;           // [1] the S buffer has been copied out
  const uint32_t bPFull = bSFree + 8;            // [2]
  const uint32_t bPDone = bPFull + 16;           // [2]
  const uint32_t bOFull = bPDone + 16;           // [2]
  const uint32_t bOEmpty = bOFull + 16;          // [2]
  const uint32_t bDrain = bOEmpty + 16;          // [2]
  const uint32_t bUFull = bDrain + 16;           // [kChUnits] a unit is in the ring
  const uint32_t bUEmpty = bUFull + 8 * kChUnits;  // [kChUnits] every role is done with it
  const uint32_t sUnit = sBar + 512;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tpt = kChM / p.G;  // tokens per tile

  pdl_launch_dependents();
  if (warp == 0) {
    if (lane == 0) {
      for (int t = 0; t < 2; ++t) {
        mbar_init(bQFull + 8 * t, FP8 ? 128 : 1);
        mbar_init(bQEmpty + 8 * t, 1);
        mbar_init(bSFull + 8 * t, 1);
        mbar_init(bPFull + 8 * t, 128);
        mbar_init(bPDone + 8 * t, 1);
        mbar_init(bOFull + 8 * t, 1);
        mbar_init(bOEmpty + 8 * t, 128);
        mbar_init(bDrain + 8 * t, 1);
        
      }
      for (int i = 0; i < kChUnits; ++i) {
        mbar_init(bUFull + 8 * i, 1);
        mbar_init(bUEmpty + 8 * i, FP8 ? 12 : 11);  // the warps that read units
      }
      for (int i = 0; i < C::STAGES; ++i) {
        mbar_init(bCFull + 8 * i, 1);
        mbar_init(bCEmpty + 8 * i, 64);
      }
      mbar_init(bSFree, 128);
      mbar_init(bVTail, 1);
      for (int s = 0; s < C::SK; ++s) {
        mbar_init(bKFull + 8 * s, 1);
        mbar_init(bKEmpty + 8 * s, 1);
      }
      for (int s = 0; s < C::SV; ++s) {
        mbar_init(bVFull + 8 * s, FP8 ? 64 : 1);
        mbar_init(bVEmpty + 8 * s, 1);
      }
      *abort_flag = 0;
      fence_mbar_init();
      if constexpr (!FP8) prefetch_tmap(&tmQ);
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
    }
  }
  pdl_wait();
  if (warp == 2) {  // not before: the kernel that is waited for may still need tensor memory
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) reinterpret_cast<PartDesc*>(p.desc)[blockIdx.x].last = -1;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // The m-th unit of the block (a whole warp or one thread); the warp says when it
  // is done with it.
  auto unit_get = [&](uint32_t m, ChUnit& u) -> bool {
    const bool got = paged_wait(bUFull + 8 * (m % kChUnits), (m / kChUnits) & 1, abort_flag);
    u.get(sUnit + 64 * (m % kChUnits));
    return got;
  };
  auto unit_done = [&](uint32_t m) { mbar_arrive(bUEmpty + 8 * (m % kChUnits)); };

  if (warp < 4) {
    setmaxnreg_dec<C::REGS_CTRL>();
    if (warp == 0 || warp == 3) {
      // ---------------------------------------------------------- copies: warp 0 K, warp 3 V
      const bool is_k = warp == 0;
      const bool staged = FP8 && !is_k;
      const uint32_t nslot = staged ? C::STAGES : (is_k ? C::SK : C::SV);
      const uint32_t ring = staged ? sVc : (is_k ? sK : sV);
      const uint32_t slot_bytes = staged ? C::VC_BYTES : (is_k ? C::K_BYTES : C::V_BYTES);
      const uint32_t bFull = staged ? bCFull : (is_k ? bKFull : bVFull);
      const uint32_t bEmpty = staged ? bCEmpty : (is_k ? bKEmpty : bVEmpty);
      const CUtensorMap* tm = is_k ? &tmK : &tmV;
      // one copy takes `box` rows of a page, 128 bytes of each (staged codes of V: a row)
      const int chunks = staged ? 1 : (is_k ? C::K_CHUNKS : C::V_CHUNKS);
      const int boxes = kChN / p.box, issues = boxes * chunks, ahead = 32 / boxes;
      const int box = lane / chunks, c = lane - box * chunks;
      int page = 0;
      bool ok = true;
      // Block j of request b's head h into slot s; `bar` counts its bytes. `kb`: the piece's first block.
      auto copy_block = [&](int b, int h, int kv, int kb, int j, uint32_t s, uint32_t bar) {
        const int a = (j - kb) & (ahead - 1);  // 32 / boxes is a power of two
        if (a == 0) page = lane < ahead * boxes ? paged_page(p, b, j * kChN + lane * p.box, kv) : 0;
        if (lane == 0) mbar_arrive_expect_tx(bar, slot_bytes);
        __syncwarp();
        const int pg = __shfl_sync(0xffffffffu, page, a * boxes + (lane < issues ? box : 0));
        if (lane < issues)
          tma_load_4d(ring + s * slot_bytes + c * C::CHUNK + box * p.box * 128, tm, bar, c * (128 / C::KSZ), h,
                      paged_row(p, j * kChN + box * p.box), pg);
      };
      // The ring's next slot, once the block before in it has been used.
      uint32_t slot = nslot - 1, turns = ~0u;  // turns of the ring before this one
      auto next_slot = [&]() -> uint32_t {
        if (++slot == nslot) {
          slot = 0;
          ++turns;
        }
        if (turns > 0) ok = __all_sync(0xffffffffu, paged_wait(bEmpty + 8 * slot, (turns - 1) & 1, abort_flag));
        return slot;
      };
      // Tells the other roles the m-th unit (K warp).
      auto publish = [&](const ChWalk& w, uint32_t m) {
        if (m >= kChUnits)
          ok = __all_sync(0xffffffffu, paged_wait(bUEmpty + 8 * (m % kChUnits), ((m / kChUnits) - 1) & 1, abort_flag));
        if (lane == 0) {
          ChUnit u;
          u.b = w.b, u.h = w.h, u.t0 = w.r.t0, u.nq = w.r.nq;
          u.kv = w.r.kv, u.tok0 = 2 * w.pair * tpt, u.kb = w.kb, u.ke = w.ke;
          u.n0 = w.n0, u.n1 = w.n1, u.whole = w.whole(), u.last = w.valid() ? w.last() / w.start.per : 0;
          u.put(sUnit + 64 * (m % kChUnits));
          mbar_arrive(bUFull + 8 * (m % kChUnits));
        }
      };
      if constexpr (!FP8) {
        uint32_t m = 0;
        if (is_k) {
          ChWalk w(p, ch_start(p, tpt), tpt);
          for (;; w.next(), ++m) {
            publish(w, m);
            if (!ok || !w.valid()) break;
            for (int j = w.kb; j < w.ke && ok; ++j) {
              const uint32_t s = next_slot();
              if (ok) copy_block(w.b, w.h, w.r.kv, w.kb, j, s, bFull + 8 * s);
            }
          }
        } else {
          uint32_t tails = 0;
          ChUnit w;
          for (; ok; ++m) {
            ok = __all_sync(0xffffffffu, unit_get(m, w));
            if (!ok || !w.valid()) break;
            for (int j = w.kb; j < w.ke && ok; ++j) {
              const uint32_t s = next_slot();
              if (!ok) break;
              const bool tail = (j + 1) * kChN > w.kv;
              copy_block(w.b, w.h, w.kv, w.kb, j, s, tail ? bVTail : bFull + 8 * s);
              if (tail) {
                ok = __all_sync(0xffffffffu, paged_wait(bVTail, tails & 1, abort_flag));
                ++tails;
                const int from = max(0, w.kv - j * kChN);
                for (int i = lane; i < (kChN - from) * C::V_CHUNKS * 8; i += 32) {
                  const int row = from + i / (C::V_CHUNKS * 8), cc = (i / 8) % C::V_CHUNKS;
                  st_shared_v4(ring + s * slot_bytes + cc * C::CHUNK + row * 128 + 16 * (i & 7), 0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bFull + 8 * s);
              }
            }
            __syncwarp();
            if (lane == 0) unit_done(m);
          }
        }
      } else {
        // Each warp keeps its ring full (K, or staged codes of V) and, block by
        // block, converts its half of V. The copies run ahead, with a place in
        // the units of their own; block i's slot is free once block i - nslot
        // has been used, which no later block's V is needed for.
        ChWalk walk(p, is_k ? ch_start(p, tpt) : ChStart{}, tpt);  // K warp
        ChUnit ld, w;
        uint32_t issued = 0, it = 0, lm = 0, m = 0;
        int lj = 0;
        bool more = true;
        auto ld_unit = [&]() {  // the next unit to copy
          if (is_k) {
            if (lm > 0) walk.next();
            publish(walk, lm);
            __syncwarp();
          }
          ok = ok && __all_sync(0xffffffffu, unit_get(lm, ld));
          ++lm;
          more = ok && ld.valid();
          lj = ld.kb;
        };
        ld_unit();
        for (; ok; ++m) {
          ok = __all_sync(0xffffffffu, unit_get(m, w));
          if (!ok || !w.valid()) break;
          for (int j = w.kb; j < w.ke && ok; ++j, ++it) {
            for (; more && issued < it + nslot; ++issued) {
              const uint32_t s = next_slot();
              if (!ok) break;
              copy_block(ld.b, ld.h, ld.kv, ld.kb, lj, s, bFull + 8 * s);
              if (++lj >= ld.ke) ld_unit();
            }
            if (!ok) break;
            const uint32_t cs = it % C::STAGES, s = it % C::SV;
            ok = paged_wait(bCFull + 8 * cs, (it / C::STAGES) & 1, abort_flag);
            if (ok && it >= C::SV) ok = paged_wait(bVEmpty + 8 * s, ((it / C::SV) - 1) & 1, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ch_convert_v(reinterpret_cast<const uint2*>(gen + (sVc - base) + cs * C::VC_BYTES), sV + s * C::V_BYTES,
                         is_k ? 0 : 1, lane, w.kv - j * kChN);
            fence_proxy_async_smem();
            mbar_arrive(bCEmpty + 8 * cs);
            mbar_arrive(bVFull + 8 * s);
          }
          __syncwarp();
          if (lane == 0) unit_done(m);
        }
      }
      if (!ok) __nanosleep(200000);  // copies in flight land before the block ends
      __syncwarp();
    } else {
      // ---------------------------------------------------------- MMA issuers: warp 1 S = Q K^T, warp 2 O += P V
      if (lane == 0) {
        const uint32_t q_lo0 = sdesc_lo(sQ, 16), k_lo0 = sdesc_lo(sK, 16), v_lo0 = sdesc_lo(sV, C::CHUNK);
        uint32_t it = 0, ns = 0, cnt[2] = {0, 0}, g[2] = {0, 0};
        bool ok = true;
        ChUnit w;
        for (uint32_t m = 0; ok; ++m) {
          if (!(ok = unit_get(m, w)) || !w.valid()) break;
          if (warp == 1) {
            if constexpr (!FP8) {
              // Q, once the tile's last products with the one before are done (this thread issued them)
              for (int t = 0; t < 2; ++t) {
                if (!w.has(t)) continue;
                if (cnt[t] > 0 && !(ok = paged_wait(bQEmpty + 8 * t, (cnt[t] - 1) & 1, abort_flag))) break;
                mbar_arrive_expect_tx(bQFull + 8 * t, C::Q_CHUNKS * 128 * tpt * p.G);
                for (int i = 0; i < C::Q_CHUNKS; ++i)
                  tma_load_3d(sQ + t * C::Q_BYTES + i * C::CHUNK, &tmQ, bQFull + 8 * t, i * 64, w.h * p.G,
                              w.t0 + w.tok0 + t * tpt);
              }
              if (!ok) break;
            }
            for (int j = w.kb; j < w.ke && ok; ++j, ++it) {
              const uint32_t s = it % C::SK;
              if (!(ok = paged_wait(bKFull + 8 * s, (it / C::SK) & 1, abort_flag))) break;
              for (int t = 0; t < 2; ++t) {
                const int e = w.end(t);
                if (j >= e) continue;
                if (j == w.kb && !(ok = paged_wait(bQFull + 8 * t, cnt[t]++ & 1, abort_flag))) break;
                if (ns > 0 && !(ok = paged_wait(bSFree, (ns - 1) & 1, abort_flag))) break;
                ++ns;
                tc_fence_after();
                const uint32_t a_lo = q_lo0 + t * (C::Q_BYTES >> 4), b_lo = k_lo0 + s * (C::K_BYTES >> 4);
                // 32 bytes of each row per step: 16 bf16, or 32 codes (Q's first and second halves
                // against the same K)
#pragma unroll
                for (int kk = 0; kk < 2 * DQK / 32; ++kk) {
                  const int kb = FP8 ? kk % (DQK / 32) : kk;
                  mma_ss_lo<FP8>(tmem, a_lo + (((kk / 4) * C::CHUNK + (kk % 4) * 32) >> 4),
                                 b_lo + (((kb / 4) * C::CHUNK + (kb % 4) * 32) >> 4), C::IDESC_QK, kk > 0 ? 1u : 0u);
                }
                tc_commit(bSFull + 8 * t);
                if (j == e - 1) tc_commit(bQEmpty + 8 * t);
              }
              if (!ok) break;
              tc_commit(bKEmpty + 8 * s);
            }
          } else {
            for (int j = w.kb; j < w.ke && ok; ++j, ++it) {
              const uint32_t s = it % C::SV;
              if (!(ok = paged_wait(bVFull + 8 * s, (it / C::SV) & 1, abort_flag))) break;
              for (int t = 0; t < 2; ++t) {
                const int e = w.end(t);
                if (j >= e) continue;
                if (!(ok = paged_wait(bPFull + 8 * t, g[t]++ & 1, abort_flag))) break;
                if (j == w.kb) {
                  if (cnt[t] > 0 && !(ok = paged_wait(bOEmpty + 8 * t, (cnt[t] - 1) & 1, abort_flag))) break;
                  ++cnt[t];
                }
                tc_fence_after();
                const uint32_t o = tmem + C::TM_O + 128 * t, a = tmem + C::TM_P + 64 * t;
                const uint32_t b_lo = v_lo0 + s * (C::V_BYTES >> 4);
#pragma unroll
                for (int kk = 0; kk < kChN / 16; ++kk)
                  mma_ts_lo<false>(o, a + 8 * kk, b_lo + ((kk * 16 * 128) >> 4), C::IDESC_PV,
                                   kk > 0 || j > w.kb ? 1u : 0u);
                tc_commit(bPDone + 8 * t);
                if (j == e - 1) tc_commit(bOFull + 8 * t);
              }
              if (!ok) break;
              tc_commit(bVEmpty + 8 * s);
            }
          }
          if (ok) unit_done(m);
        }
        // every MMA this thread issued has completed before the block frees its tensor memory
        const uint32_t drain = bDrain + 8 * (warp - 1);
        tc_commit(drain);
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(drain, 0) && global_timer_ns() - t0 < kPagedWaitLimitNs) {
        }
        if (!FP8 && warp == 1 && !ok) __nanosleep(200000);  // copies of Q in flight land before the block ends
      }
      __syncwarp();
    }
  } else {
    setmaxnreg_inc<C::REGS_SOFT>();
    // ------------------------------------------------------------ softmax and epilogue, one thread per row
    const int t = (warp - 4) >> 2;
    const int r = threadIdx.x - 128 - 128 * t;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t tS = tmem + lanes, tO = tmem + lanes + C::TM_O + 128 * t, tP = tmem + lanes + C::TM_P + 64 * t;
    uint32_t g = 0, units = 0;  // key blocks and pieces this tile has done
    bool ok = true;
    ChUnit w;
    for (uint32_t m = 0; ok; ++m) {
      ok = __all_sync(0xffffffffu, unit_get(m, w));
      if (!ok || !w.valid()) break;
      float c_log2 = p.scale_log2;
      int see, see_all, end;
      {
      const int rtok = static_cast<uint32_t>(r) / p.group;
      const int tok = w.tok0 + t * tpt + rtok;
      const bool real = rtok < tpt && tok < w.nq;
      const bool whole = w.whole != 0, head = w.kb > 0;
      if (t == 0 && r == 0 && !whole && !head) {
        PartDesc e;
        e.last = w.last;
        e.t0 = w.t0;
        e.row0 = w.tok0 * p.G;
        e.nrows = min(2 * tpt, w.nq - w.tok0) * p.G;
        e.hkv = w.h;
        e.pad[0] = e.pad[1] = e.pad[2] = 0;
        reinterpret_cast<PartDesc*>(p.desc)[blockIdx.x] = e;
      }
      if (!w.has(t)) {  // none of this tile's blocks are in this piece
        if (real && !whole) {
          const int64_t part =
              static_cast<int64_t>(2 * blockIdx.x + (head ? 0 : 1)) * p.slot_rows + t * tpt * p.G + r;
          p.part_ml[2 * part] = -INFINITY;
          p.part_ml[2 * part + 1] = 0.0f;
        }
        __syncwarp();
        if (lane == 0) unit_done(m);
        continue;
      }
      if constexpr (FP8) {
        // Q as two e4m3 numbers per element, side by side: codes [0, d) nearest,
        // [d, 2 d) the rest. Eight lanes take a row, so that loads are whole lines;
        // a row's factor then goes to the thread that has its scores.
        if (units > 0) ok = paged_wait(bQEmpty + 8 * t, (units - 1) & 1, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        constexpr int NU = DQK / 64;  // 16-byte pieces of a row per lane
        const int l8 = lane & 7;
        float mine = 1.0f;
        uint4 rows[8][NU];  // every load under way before the first is used
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const int rr = 32 * (warp & 3) + 4 * s + (lane >> 3);
          const int rt = static_cast<uint32_t>(rr) / p.group, tk = w.tok0 + t * tpt + rt;
          const bool has = rt < tpt && tk < w.nq;
          const uint4* src = reinterpret_cast<const uint4*>(
              p.q + (w.t0 + (has ? tk : 0)) * p.q_stride +
              static_cast<int64_t>(w.h * p.G + (has ? rr - rt * p.G : 0)) * DQK) + l8;
#pragma unroll
          for (int n = 0; n < NU; ++n) rows[s][n] = has ? __ldg(src + 8 * n) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const int rr = 32 * (warp & 3) + 4 * s + (lane >> 3);
          const uint4(&x)[NU] = rows[s];
          float amax = 0.0f;
          auto absmax2 = [](uint32_t v) {
            return fmaxf(fabsf(__uint_as_float(v << 16)), fabsf(__uint_as_float(v & 0xffff0000u)));
          };
#pragma unroll
          for (int n = 0; n < NU; ++n)
            amax = fmaxf(amax, fmaxf(fmaxf(absmax2(x[n].x), absmax2(x[n].y)), fmaxf(absmax2(x[n].z), absmax2(x[n].w))));
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          int e = 0;
          if (amax > 0.0f && amax < INFINITY)
            e = max(-118, min(126, static_cast<int>(__float_as_uint(amax) >> 23) - 134));
          float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
          if (amax == INFINITY) down = __uint_as_float(0x7fffffffu);  // an infinite element: NaN scores
          const float up = __shfl_sync(0xffffffffu, __uint_as_float(static_cast<uint32_t>(127 + e) << 23), 8 * (lane & 3));
          if ((lane >> 2) == s) mine = up;
          const uint32_t row = sQ + t * C::Q_BYTES + rr * 128;
#pragma unroll
          for (int n = 0; n < NU; ++n) {
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t a = k ? x[n].z : x[n].x, b = k ? x[n].w : x[n].y;
              const float f0 = __uint_as_float(a << 16) * down, f1 = __uint_as_float(a & 0xffff0000u) * down;
              const float f2 = __uint_as_float(b << 16) * down, f3 = __uint_as_float(b & 0xffff0000u) * down;
              const uint32_t h01 = pack_e4m3x2(f0, f1), h23 = pack_e4m3x2(f2, f3);
              const float2 g01 = __half22float2(bits_half2(e4m3x2_f16x2(h01)));
              const float2 g23 = __half22float2(bits_half2(e4m3x2_f16x2(h23)));
              hi[k] = h01 | (h23 << 16);
              lo[k] = static_cast<uint32_t>(pack_e4m3x2(f0 - g01.x, f1 - g01.y)) |
                      (static_cast<uint32_t>(pack_e4m3x2(f2 - g23.x, f3 - g23.y)) << 16);
            }
            const int uh = 4 * n + (l8 >> 1), ul = DQK / 16 + uh;  // 16-byte units of the row
            st_shared_v2(row + (uh >> 3) * C::CHUNK + (((uh & 7) ^ (rr & 7)) << 4) + 8 * (l8 & 1), hi[0], hi[1]);
            st_shared_v2(row + (ul >> 3) * C::CHUNK + (((ul & 7) ^ (rr & 7)) << 4) + 8 * (l8 & 1), lo[0], lo[1]);
          }
        }
        c_log2 *= mine * __ldg(p.k_scale + w.h);
        fence_proxy_async_smem();
        mbar_arrive(bQFull + 8 * t);
      }
      ++units;
      // keys this row sees: j <= see; the tile's first row sees fewest
      const int off = p.causal ? w.kv - w.nq : w.kv - 1;
      see = p.causal ? min(off + tok, w.kv - 1) : off;
      see_all = p.causal ? min(off + w.tok0 + t * tpt, w.kv - 1) : off;
      // a zero scale behaves as a tiny one; a NaN stays, but for a row that sees no key
      if (c_log2 < 1e-30f || see < 0) c_log2 = 1e-30f;

      end = w.end(t);
      }

      const float p_exp = ch_p_exp<FP8>(w.kv);
      float m_ref = -INFINITY, l_run = 0.0f;  // probabilities are 2^(score - m_ref), at most 2^P_MAX
      const int kb = w.kb;
      for (int j = kb; j < end; ++j, ++g) {
        ok = __all_sync(0xffffffffu, paged_wait(bSFull + 8 * t, g & 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
        uint32_t sr[128];
        tmem_ld32(tS + 0, sr);
        tmem_ld32(tS + 32, sr + 32);
        tmem_ld32(tS + 64, sr + 64);
        tmem_ld32(tS + 96, sr + 96);
        tmem_ld_wait32(sr);
        reg_fence32(sr + 32);
        reg_fence32(sr + 64);
        reg_fence32(sr + 96);
        tc_fence_before();
        mbar_arrive(bSFree);  // S may take the next product now

        const int kv0 = j * kChN;
        if (kv0 + kChN - 1 > see_all) {
          const int lim = see - kv0;
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c > lim) sr[c] = __float_as_uint(-INFINITY);
        }
        // row maximum; a NaN score stays one
        float x0 = __uint_as_float(sr[0]), x1 = __uint_as_float(sr[1]);
        float x2 = __uint_as_float(sr[2]), x3 = __uint_as_float(sr[3]);
#pragma unroll
        for (int c = 4; c < 124; c += 8) {
          x0 = max3_nan(x0, __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
          x1 = max3_nan(x1, __uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3]));
          x2 = max3_nan(x2, __uint_as_float(sr[c + 4]), __uint_as_float(sr[c + 5]));
          x3 = max3_nan(x3, __uint_as_float(sr[c + 6]), __uint_as_float(sr[c + 7]));
        }
        x0 = max3_nan(x0, __uint_as_float(sr[124]), __uint_as_float(sr[125]));
        x1 = max3_nan(x1, __uint_as_float(sr[126]), __uint_as_float(sr[127]));
        x0 = max3_nan(x0, x1, x2);
        const float m_new = max2_nan(x0 * c_log2, x3 * c_log2);
        // fp16: large scores, whose rounding is more than a fraction of a binade, leave that much less room (the
        // reference itself never moves down)
        const float room = FP8 ? fmaxf(fmaf(fabsf(m_ref), -0x1p-22f, C::P_MAX), p_exp) : C::P_MAX;
        const bool need = !(m_new <= m_ref + room);  // true for NaN too
        float alpha = 1.0f;
        if (need) {
          const float to = m_new - p_exp;
          alpha = ex2_approx(m_ref - to);
          m_ref = to;
        }
        l_run *= alpha;

        // probabilities, packed in place; a row that has seen nothing yet has m = -inf and only masked scores.
        // All on the MUFU unit: what these warps lack is issue slots (and, under the power cap, energy), and a
        // polynomial for one score in four on the FMA pipe took long chunks 1765 us for 1690, e4m3 chunks 403 for
        // 362; for one in eight 1727 and 393.
        const float nm = m_ref == -INFINITY ? 0.0f : -m_ref;
        float sa = 0.f, sb = 0.f, sc = 0.f, sd = 0.f;
#pragma unroll
        for (int c = 0; c < 128; c += 4) {
          float y0, y1, y2, y3;
          ffma2_bcast(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1]), c_log2, nm, y0, y1);
          ffma2_bcast(__uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3]), c_log2, nm, y2, y3);
          const float p0 = ex2_approx(y0), p1 = ex2_approx(y1), p2 = ex2_approx(y2), p3 = ex2_approx(y3);
          fadd2(sa, sb, p0, p1);
          fadd2(sc, sd, p2, p3);
          sr[c >> 1] = FP8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
          sr[(c >> 1) + 1] = FP8 ? pack_f16x2(p2, p3) : pack_bf16x2(p2, p3);
        }
        l_run += (sa + sb) + (sc + sd);

        // P and O are free once PV of the tile's block before has completed
        bool w_ok = g == 0 || paged_wait(bPDone + 8 * t, (g - 1) & 1, abort_flag);
        const bool resc = j > kb && __any_sync(0xffffffffu, need);
        ok = __all_sync(0xffffffffu, w_ok);
        if (!ok) break;
        tc_fence_after();
        if (resc) {
#pragma unroll 1
          for (int cc = 0; cc < DV; cc += 32) {
            uint32_t orr[32];
            tmem_ld32(tO + cc, orr);
            tmem_ld_wait32(orr);
#pragma unroll
            for (int i = 0; i < 32; ++i) orr[i] = __float_as_uint(__uint_as_float(orr[i]) * alpha);
            tmem_st32(tO + cc, orr);
          }
        }
        tmem_st32(tP, sr);
        tmem_st32(tP + 32, sr + 32);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bPFull + 8 * t);
      }
      if (!ok) break;

      ok = __all_sync(0xffffffffu, paged_wait(bOFull + 8 * t, (units - 1) & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      w.get(sUnit + 64 * (m % kChUnits));  // not kept in registers over the keys
      const int rtok = static_cast<uint32_t>(r) / p.group, rhead = r - rtok * p.G;
      const int tok = w.tok0 + t * tpt + rtok;
      const bool real = rtok < tpt && tok < w.nq;
      const bool whole = w.whole != 0;
      const int64_t part =
          static_cast<int64_t>(2 * blockIdx.x + (w.kb > 0 ? 0 : 1)) * p.slot_rows + t * tpt * p.G + r;
      const float inv = l_run == 0.0f ? 0.0f : 1.0f / l_run;
      const float v_mult = !FP8 ? 1.0f : (l_run == 0.0f ? 0.0f : __ldg(p.v_scale + w.h));
      const int hq = w.h * p.G + rhead;
      __nv_bfloat16* orow = p.o + (static_cast<int64_t>(w.t0 + (real ? tok : 0)) * p.Hq + (real ? hq : 0)) * DV;
      // parts: [slot][DV / 4][row][4], whole lines for a warp's 32 rows
      float* prow = p.part_o + static_cast<int64_t>(2 * blockIdx.x + (w.kb > 0 ? 0 : 1)) * p.slot_rows * DV +
                    (real ? t * tpt * p.G + r : 0) * 4;
#pragma unroll 1
      for (int cc = 0; cc < DV; cc += 32) {
        uint32_t orr[32];
        tmem_ld32(tO + cc, orr);
        tmem_ld_wait32(orr);
        if (real && whole) {
          uint32_t y[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            y[i] = pack_bf16x2(__uint_as_float(orr[2 * i]) * inv * v_mult, __uint_as_float(orr[2 * i + 1]) * inv * v_mult);
          st_global_32b(orow + cc, y);
          st_global_32b(orow + cc + 16, y + 8);
        } else if (real) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(prow + static_cast<int64_t>(cc / 4 + i) * p.slot_rows * 4) =
                make_uint4(orr[4 * i], orr[4 * i + 1], orr[4 * i + 2], orr[4 * i + 3]);
        }
      }
      if (real && !whole) {
        p.part_ml[2 * part] = m_ref;
        p.part_ml[2 * part + 1] = l_run;
      } else if (real && p.lse != nullptr) {
        p.lse[static_cast<int64_t>(hq) * p.T + w.t0 + tok] =
            l_run == 0.0f ? -INFINITY : (m_ref + fast_log2(l_run)) * kLn2;
      }
      tc_fence_before();
      mbar_arrive(bOEmpty + 8 * t);
      __syncwarp();
      if (lane == 0) unit_done(m);
    }
  }

  // -------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace b200p
