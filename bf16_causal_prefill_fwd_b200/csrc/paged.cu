// C-ABI entry points of the paged-cache operators (declared in
// include/b200attn.h): argument validation, tensor-map encoding, kernel
// selection and launch. What they compute runs in the paged_*.cuh kernels.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/b200attn.h"
#include "paged_append.cuh"
#include "paged_chunk.cuh"
#include "paged_common.cuh"
#include "paged_decode.cuh"
#include "paged_join.cuh"
#include "paged_slots.cuh"
#include "paged_status.h"

namespace {

using b200p::PagedAttn;

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int gcd(int a, int b) {
  while (b != 0) {
    const int r = a % b;
    a = b;
    b = r;
  }
  return a;
}

constexpr int kDevices = 64;

// Compute capability 10.0; *sm_count: SMs of the current device (looked up once
// per device), *device: its number.
int device_ok(int* sm_count, int* device) {
  static std::atomic<int> sms[kDevices];  // 0: not looked up yet, -1: not supported
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return B200ATTN_ERR_CUDA;
  int n = sms[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return B200ATTN_ERR_CUDA;
    if (major != 10 || minor != 0) n = -1;
    sms[dev].store(n, std::memory_order_relaxed);
  }
  if (n < 0) return B200ATTN_ERR_UNSUPPORTED;
  *sm_count = n;
  *device = dev;
  return B200ATTN_OK;
}

// Lets `kern` use `bytes` of dynamic shared memory, once per kernel and device
// (`done` is the kernel's own). With `regs`, the kernel must have been built with
// that many registers per thread: a role split (setmaxnreg) of another launch
// allocation would wait for registers that do not exist.
int prepare_kernel(const void* kern, int bytes, int regs, int device, std::atomic<uint64_t>& done) {
  const uint64_t bit = uint64_t(1) << device;
  if (done.load(std::memory_order_acquire) & bit) return B200ATTN_OK;
  cudaFuncAttributes a;
  if (cudaFuncGetAttributes(&a, kern) != cudaSuccess ||
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return B200ATTN_ERR_CUDA;
  if (regs != 0 && a.numRegs != regs) return B200ATTN_ERR_UNSUPPORTED;
  done.fetch_or(bit, std::memory_order_release);
  return B200ATTN_OK;
}

// A stride the kernels may use: a multiple of 16 bytes, not negative.
bool stride_ok(int64_t elems, int esz) { return elems >= 0 && elems < (int64_t(1) << 38) && elems * esz % 16 == 0; }

// The distance of tokens of `heads` contiguous heads: they do not overlap.
bool rows_ok(size_t stride, int tokens, int heads, int d) {
  return tokens == 1 || (stride_ok(static_cast<int64_t>(stride), 2) && static_cast<int64_t>(stride) >= int64_t(heads) * d);
}

// Argument checks that every entry point taking a cache shares.
int check_cache(const b200attn_paged_cache* c) {
  if (!c || !c->k || !c->v) return B200ATTN_ERR_INVALID;
  if (c->num_pages < 1 || c->page_size < 1 || c->Hkv < 1 || c->d_qk < 1 || c->d_v < 1) return B200ATTN_ERR_INVALID;
  if (c->dtype != B200ATTN_BF16 && c->dtype != B200ATTN_FP8_E4M3) return B200ATTN_ERR_UNSUPPORTED;
  if (!(c->d_v == 128 && (c->d_qk == 128 || c->d_qk == 192))) return B200ATTN_ERR_UNSUPPORTED;
  if (c->page_size % 16 != 0) return B200ATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(c->num_pages) * c->page_size >= (int64_t(1) << 31)) return B200ATTN_ERR_UNSUPPORTED;
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return B200ATTN_ERR_INVALID;
  const int esz = c->dtype == B200ATTN_BF16 ? 2 : 1;
  const int64_t s[6] = {c->k_page_stride, c->k_token_stride, c->k_head_stride,
                        c->v_page_stride, c->v_token_stride, c->v_head_stride};
  const int size[3] = {c->num_pages, c->page_size, c->Hkv};
  for (int i = 0; i < 6; ++i)  // the stride of a dimension of one is not used
    if (size[i % 3] > 1 && (s[i] == 0 || !stride_ok(s[i], esz))) return B200ATTN_ERR_INVALID;
  if (c->dtype == B200ATTN_FP8_E4M3 &&
      (!c->k_scale || !c->v_scale || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)))
    return B200ATTN_ERR_INVALID;
  return B200ATTN_OK;
}

// A cache tensor as a 4-D map {d, head, row of the page, page} with a box of one
// head of `rows` rows, 128 bytes of each, with the 128-byte swizzle or (swizzle
// false) as they are; out of range reads zero.
bool page_map(CUtensorMap* m, const void* ptr, bool fp8, int d, int H, int ps, int pages, int64_t head, int64_t token,
              int64_t page, int rows, bool swizzle) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t esz = fp8 ? 1 : 2;
  // a dimension of one element may come with any stride
  const cuuint64_t sh = H > 1 ? head * esz : d * esz, st = ps > 1 ? token * esz : d * esz,
                   sp = pages > 1 ? page * esz : d * esz;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)ps, (cuuint64_t)pages};
  const cuuint64_t strides[3] = {sh, st, sp};
  const cuuint32_t box[4] = {(cuuint32_t)(128 / esz), 1, (cuuint32_t)rows, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return enc(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr),
             dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
             // no more than a row: the bytes behind it are another head's (256 bytes at a time read 1.4 times
             // an e4m3 cache's 128-byte rows from HBM)
             fp8 ? (d % 128 == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_64B)
                 : (d % 128 == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B),
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool page_maps(CUtensorMap* tk, CUtensorMap* tv, const b200attn_paged_cache* c, int rows, bool swizzle_v) {
  const bool fp8 = c->dtype == B200ATTN_FP8_E4M3;
  return page_map(tk, c->k, fp8, c->d_qk, c->Hkv, c->page_size, c->num_pages, c->k_head_stride, c->k_token_stride,
                  c->k_page_stride, rows, true) &&
         page_map(tv, c->v, fp8, c->d_v, c->Hkv, c->page_size, c->num_pages, c->v_head_stride, c->v_token_stride,
                  c->v_page_stride, rows, swizzle_v);
}

// Launch whose blocks may be scheduled while the kernel before it in the stream
// drains. Every kernel of this file first waits for that kernel and its writes
// (griddepcontrol.wait), so only the launch itself and the block's set-up
// overlap; each lets its successor do the same once all its blocks run.
template <typename... Args>
int launch(void (*kern)(Args...), dim3 grid, int threads, int smem, int cluster, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? B200ATTN_OK : B200ATTN_ERR_CUDA;
}

size_t round_up(size_t n) { return (n + 255) / 256 * 256; }

// Workspace of the attention kernels: descriptors, (m, l), O of 2 * blocks slots.
struct Parts {
  size_t ml, o, bytes;
};
Parts parts_of(int blocks, int rows) {
  Parts w;
  w.ml = round_up(sizeof(b200p::PartDesc) * blocks);
  w.o = w.ml + round_up(sizeof(float) * 2 * 2 * blocks * rows);
  w.bytes = w.o + round_up(sizeof(float) * 128 * 2 * blocks * rows);
  return w;
}

// The few-rows kernel serves up to 16 query rows per key/value head; the choice
// is by the bound on a request's new tokens alone, which the host knows. At 16 rows
// (4 tokens, 4 heads a group) 64 requests over up to 16k bf16 keys take 313-354 us with
// it and 314-369 with the other, one over 4096 17-23 and 20-27; 24 requests of 12 rows
// over 9-32k e4m3 keys 187 and 307. Above, its rows would no longer fit the registers.
bool few_rows(int max_q, int G) { return static_cast<int64_t>(max_q) * G <= b200p::kDecMaxRows; }

template <int DQK, bool FP8, int NT>
int launch_decode(const b200attn_paged_cache* c, PagedAttn p, int sm_count, int device, cudaStream_t st) {
  using C = b200p::DecCfg<DQK, 128, FP8, NT>;
  p.box = gcd(p.page_size, C::KEYS);
  p.slot_rows = b200p::kDecMaxRows;
  CUtensorMap tk, tv;
  if (!page_maps(&tk, &tv, c, p.box, true)) return B200ATTN_ERR_CUDA;
  auto kern = b200p::paged_decode_kernel<DQK, 128, FP8, NT>;
  static std::atomic<uint64_t> done{0};
  const int rc = prepare_kernel(reinterpret_cast<const void*>(kern), C::SMEM, 0, device, done);
  if (rc != B200ATTN_OK) return rc;
  int blocks = C::BLOCKS * sm_count;
  if (blocks > b200p::kDecMaxBlocks) blocks = b200p::kDecMaxBlocks;
  const int lrc = launch(kern, dim3(blocks, 1, 1), b200p::kDecThreads, C::SMEM, 1, st, static_cast<const CUtensorMap>(tk),
                         static_cast<const CUtensorMap>(tv), static_cast<const PagedAttn>(p));
  if (lrc != B200ATTN_OK) return lrc;
  return launch(b200p::paged_join_few_kernel<128>, dim3(blocks, 4, 1), 128, 0, 1, st, static_cast<const PagedAttn>(p));
}

template <int DQK, bool FP8>
int launch_few(const b200attn_paged_cache* c, const PagedAttn& p, int sm_count, int device, cudaStream_t st) {
  if (p.max_q * p.G <= 8) return launch_decode<DQK, FP8, 1>(c, p, sm_count, device, st);
  return launch_decode<DQK, FP8, 2>(c, p, sm_count, device, st);
}

// Rows of a workspace slot of the many-rows kernel.
int chunk_rows(int total, int G) {
  const int64_t rows = static_cast<int64_t>(total) * G;
  return rows < b200p::kChRows ? static_cast<int>(rows) : b200p::kChRows;
}

template <int DQK, bool FP8>
int launch_chunk(const b200attn_paged_cache* c, PagedAttn p, int sm_count, int device, cudaStream_t st) {
  using C = b200p::ChCfg<DQK, 128, FP8>;
  p.box = gcd(p.page_size, b200p::kChN);
  p.slot_rows = chunk_rows(p.T, p.G);
  p.pair = b200p::fast_div(2 * (b200p::kChM / p.G));
  CUtensorMap tq = {}, tk = {}, tv = {};
  if (!FP8) {
    // {d, head, token} with a box of 64 columns, the G heads of a group and a tile's tokens
    const cuuint64_t dims[3] = {DQK, (cuuint64_t)p.Hq, (cuuint64_t)p.T};
    const cuuint64_t strides[2] = {DQK * 2, (cuuint64_t)(p.T > 1 ? p.q_stride : static_cast<int64_t>(p.Hq) * DQK) * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)(b200p::kChM / p.G)};
    const cuuint32_t one[3] = {1, 1, 1};
    EncodeTiledFn enc = encode_fn();
    if (!enc || enc(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(p.q), dims, strides, box, one,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return B200ATTN_ERR_CUDA;
  }
  if (!page_maps(&tk, &tv, c, p.box, !FP8)) return B200ATTN_ERR_CUDA;
  auto kern = b200p::paged_chunk_kernel<DQK, 128, FP8>;
  static std::atomic<uint64_t> done{0};
  const int rc = prepare_kernel(reinterpret_cast<const void*>(kern), C::SMEM, C::REGS_LAUNCH, device, done);
  if (rc != B200ATTN_OK) return rc;
  const int blocks = sm_count < b200p::kChMaxBlocks ? sm_count : b200p::kChMaxBlocks;
  const int lrc = launch(kern, dim3(blocks, 1, 1), C::THREADS, C::SMEM, 1, st, static_cast<const CUtensorMap>(tq),
                         static_cast<const CUtensorMap>(tk), static_cast<const CUtensorMap>(tv),
                         static_cast<const PagedAttn>(p));
  if (lrc != B200ATTN_OK) return lrc;
  return launch(b200p::paged_join_rows_kernel<128>, dim3(blocks, (p.slot_rows + 15) / 16, 1), 128, 0, 1, st,
                static_cast<const PagedAttn>(p));
}

}  // namespace

int b200_paged_take_status() {
  int status = 0;
  const int zero = 0;
  if (cudaMemcpyFromSymbol(&status, b200p::g_paged_status, sizeof(int)) != cudaSuccess) return B200ATTN_ERR_CUDA;
  if (status != 0 && cudaMemcpyToSymbol(b200p::g_paged_status, &zero, sizeof(int)) != cudaSuccess)
    return B200ATTN_ERR_CUDA;
  return status;
}

extern "C" {

int b200attn_paged_slots(int* block_table, size_t table_stride, int table_width, const int* context_lens,
                         const int* new_lens, int batch, int total, int page_size, const int* free_pages,
                         int free_count, const int* free_head, int* free_head_out, int* cu_seqlens, int* kv_lens,
                         int* positions, int* slots, void* stream) {
  if (batch < 1 || total < 0 || table_width < 1 || page_size < 1 || free_count < 0)
    return B200ATTN_ERR_INVALID;
  if (!block_table || !context_lens || !new_lens || !cu_seqlens || !kv_lens) return B200ATTN_ERR_INVALID;
  if (total > 0 && (!positions || !slots)) return B200ATTN_ERR_INVALID;
  if (free_pages && (!free_head || !free_head_out)) return B200ATTN_ERR_INVALID;
  const void* ptrs[10] = {block_table, context_lens,  new_lens,   cu_seqlens, kv_lens,
                          positions,   free_head_out, free_pages, free_head,  slots};
  for (const void* p : ptrs)
    if (!aligned(p, 4)) return B200ATTN_ERR_INVALID;
  if (batch > b200p::kSlotsMaxBatch || total >= (1 << 30) || table_stride > 0x7fffffff) return B200ATTN_ERR_UNSUPPORTED;
  int sm_count = 0, device = 0;
  const int rc = device_ok(&sm_count, &device);
  if (rc != B200ATTN_OK) return rc;

  b200p::PagedSlots p = {};
  p.table = block_table;
  p.table_stride = table_stride;
  p.width = table_width;
  p.ctx = context_lens;
  p.nw = new_lens;
  p.B = batch;
  p.total = total;
  p.page_size = page_size;
  p.free_pages = free_pages;
  p.free_count = free_count;
  p.head_in = free_head;
  p.head_out = free_head_out;
  p.cu = cu_seqlens;
  p.kv = kv_lens;
  p.pos = positions;
  p.slot = slots;
  const int smem = (3 * batch + 2) * static_cast<int>(sizeof(int));
  static std::atomic<uint64_t> done{0};
  const int prc = prepare_kernel(reinterpret_cast<const void*>(b200p::paged_slots_kernel),
                                 (3 * b200p::kSlotsMaxBatch + 2) * static_cast<int>(sizeof(int)), 0, device, done);
  if (prc != B200ATTN_OK) return prc;
  // One cluster: its barrier stands between reading the free list's head and
  // writing it. A step that one block covers in a pass or two takes one block.
  const int blocks = total <= b200p::kSlotsThreads ? 1 : b200p::kSlotsCluster;
  return launch(b200p::paged_slots_kernel, dim3(blocks, 1, 1), b200p::kSlotsThreads, smem, blocks,
                static_cast<cudaStream_t>(stream), static_cast<const b200p::PagedSlots>(p));
}

int b200attn_paged_append(const void* k, const void* v, size_t k_stride, size_t v_stride, int total,
                          const b200attn_paged_cache* cache, const int* slots, void* stream) {
  const int cc = check_cache(cache);
  if (cc != B200ATTN_OK) return cc;
  if (total < 0) return B200ATTN_ERR_INVALID;
  if (total == 0) return B200ATTN_OK;
  if (!k || !v || !slots || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4)) return B200ATTN_ERR_INVALID;
  if (!rows_ok(k_stride, total, cache->Hkv, cache->d_qk) || !rows_ok(v_stride, total, cache->Hkv, cache->d_v))
    return B200ATTN_ERR_INVALID;
  const int64_t units =
      static_cast<int64_t>(total) * cache->Hkv * ((cache->d_qk + cache->d_v) / b200p::kAppendUnit);
  if (units >= (int64_t(1) << 31)) return B200ATTN_ERR_UNSUPPORTED;
  int sm_count = 0, device = 0;
  const int rc = device_ok(&sm_count, &device);
  if (rc != B200ATTN_OK) return rc;

  b200p::PagedAppend p = {};
  p.x[0] = static_cast<const __nv_bfloat16*>(k);
  p.x[1] = static_cast<const __nv_bfloat16*>(v);
  p.x_stride[0] = k_stride;
  p.x_stride[1] = v_stride;
  p.cache[0] = cache->k;
  p.cache[1] = cache->v;
  p.page_stride[0] = cache->k_page_stride;
  p.page_stride[1] = cache->v_page_stride;
  p.token_stride[0] = cache->k_token_stride;
  p.token_stride[1] = cache->v_token_stride;
  p.head_stride[0] = cache->k_head_stride;
  p.head_stride[1] = cache->v_head_stride;
  p.scale[0] = cache->k_scale;
  p.scale[1] = cache->v_scale;
  p.slots = slots;
  p.T = total;
  p.H = cache->Hkv;
  p.num_pages = cache->num_pages;
  p.page_size = b200p::fast_div(cache->page_size);
  p.per_token = b200p::fast_div(cache->Hkv * ((cache->d_qk + cache->d_v) / b200p::kAppendUnit));
  const int64_t want = (units + b200p::kAppendThreads - 1) / b200p::kAppendThreads;
  // One unit per thread while the grid is below 64 blocks per SM: measured side by side on 16k tokens, 8 blocks per SM
  // looping took 23.6 us (bf16) and 20.7 us (e4m3), 64 20.7 and 19.4; two or four units in flight per thread were slower.
  const int blocks = static_cast<int>(want < 64 * sm_count ? want : 64 * sm_count);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto kern = cache->dtype == B200ATTN_BF16
                  ? (cache->d_qk == 128 ? b200p::paged_append_kernel<128, 128, false> : b200p::paged_append_kernel<192, 128, false>)
                  : (cache->d_qk == 128 ? b200p::paged_append_kernel<128, 128, true> : b200p::paged_append_kernel<192, 128, true>);
  return launch(kern, dim3(blocks, 1, 1), b200p::kAppendThreads, 0, 1, st, static_cast<const b200p::PagedAppend>(p));
}

size_t b200attn_paged_fwd_workspace_bytes(int total, int max_seqlen_q, int Hq, int Hkv) {
  if (total < 1 || max_seqlen_q < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return 0;
  // never less than for fewer tokens, whichever kernel takes those
  const size_t few = parts_of(b200p::kDecMaxBlocks, b200p::kDecMaxRows).bytes;
  if (few_rows(max_seqlen_q < total ? max_seqlen_q : total, Hq / Hkv)) return few;
  const size_t many = parts_of(b200p::kChMaxBlocks, chunk_rows(total, Hq / Hkv)).bytes;
  return many > few ? many : few;
}

int b200attn_paged_fwd(const void* q, size_t q_stride, const b200attn_paged_cache* cache, const int* block_table,
                       size_t table_stride, int table_width, const int* cu_seqlens, const int* kv_lens, int batch,
                       int total, int max_seqlen_q, int Hq, int causal, float softmax_scale, void* o, float* lse,
                       void* workspace, size_t workspace_bytes, void* stream) {
  const int cc = check_cache(cache);
  if (cc != B200ATTN_OK) return cc;
  if (batch < 1 || total < 0 || Hq < 1 || max_seqlen_q < 1 || table_width < 1)
    return B200ATTN_ERR_INVALID;
  if (Hq % cache->Hkv != 0 || (causal != 0 && causal != 1) || !std::isfinite(softmax_scale)) return B200ATTN_ERR_INVALID;
  if (total == 0) return B200ATTN_OK;  // no new tokens
  if (max_seqlen_q > total) max_seqlen_q = total;
  if (!q || !o || !block_table || !cu_seqlens || !kv_lens) return B200ATTN_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(o, 32) || !aligned(block_table, 4) || !aligned(cu_seqlens, 4) ||
      !aligned(kv_lens, 4) || !aligned(lse, 4) || !rows_ok(q_stride, total, Hq, cache->d_qk))
    return B200ATTN_ERR_INVALID;
  const int G = Hq / cache->Hkv;
  if (G > 128) return B200ATTN_ERR_UNSUPPORTED;
  // the kernels count query rows and the line of key tiles in 32 bits
  constexpr int64_t limit = int64_t(1) << 31;
  const int64_t keys = static_cast<int64_t>(table_width) * cache->page_size;
  const int64_t lines = static_cast<int64_t>(batch) * cache->Hkv;
  if (keys >= limit / 2 || table_stride > 0x7fffffff || static_cast<int64_t>(total) * Hq >= limit || lines >= limit)
    return B200ATTN_ERR_UNSUPPORTED;
  if (few_rows(max_seqlen_q, G)) {
    if (lines * (keys / 64 /* the smallest tile */ + 1) >= limit) return B200ATTN_ERR_UNSUPPORTED;
  } else {  // pairs of row tiles, by the bound on new tokens or by the rows there are
    const int64_t per = 2 * (b200p::kChM / G), most = max_seqlen_q;
    const int64_t each = batch * ((most + per - 1) / per), packed = total / per + batch;
    const int64_t units = (each < packed ? each : packed) * cache->Hkv;
    if (units >= limit || units * (keys / b200p::kChN + 1 + b200p::kChUnitCost) >= limit) return B200ATTN_ERR_UNSUPPORTED;
  }
  const size_t need = b200attn_paged_fwd_workspace_bytes(total, max_seqlen_q, Hq, cache->Hkv);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return B200ATTN_ERR_WORKSPACE;
  int sm_count = 0, device = 0;
  const int rc = device_ok(&sm_count, &device);
  if (rc != B200ATTN_OK) return rc;

  const bool fp8 = cache->dtype == B200ATTN_FP8_E4M3;
  PagedAttn p = {};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride = q_stride;
  p.table = block_table;
  p.table_stride = static_cast<int>(table_stride);
  p.width = table_width;
  p.cu = cu_seqlens;
  p.kv_lens = kv_lens;
  p.B = batch;
  p.T = total;
  p.Hq = Hq;
  p.Hkv = cache->Hkv;
  p.G = G;
  p.group = b200p::fast_div(G);
  p.num_pages = cache->num_pages;
  p.page_size = cache->page_size;
  p.rows = b200p::fast_div(cache->page_size);
  p.max_q = max_seqlen_q;
  p.causal = causal;
  const double s = softmax_scale > 0.0f ? static_cast<double>(softmax_scale)
                                        : 1.0 / std::sqrt(static_cast<double>(cache->d_qk));
  p.scale_log2 = static_cast<float>(s * 1.4426950408889634);
  p.k_scale = fp8 ? cache->k_scale : nullptr;
  p.v_scale = fp8 ? cache->v_scale : nullptr;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const bool few = few_rows(max_seqlen_q, G);
  const Parts w = few ? parts_of(b200p::kDecMaxBlocks, b200p::kDecMaxRows)
                      : parts_of(b200p::kChMaxBlocks, chunk_rows(total, G));
  p.desc = reinterpret_cast<int*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + w.ml);
  p.part_o = reinterpret_cast<float*>(ws + w.o);
  if (few) {
    if (cache->d_qk == 128)
      return fp8 ? launch_few<128, true>(cache, p, sm_count, device, st) : launch_few<128, false>(cache, p, sm_count, device, st);
    return fp8 ? launch_few<192, true>(cache, p, sm_count, device, st) : launch_few<192, false>(cache, p, sm_count, device, st);
  }
  if (cache->d_qk == 128)
    return fp8 ? launch_chunk<128, true>(cache, p, sm_count, device, st) : launch_chunk<128, false>(cache, p, sm_count, device, st);
  return fp8 ? launch_chunk<192, true>(cache, p, sm_count, device, st) : launch_chunk<192, false>(cache, p, sm_count, device, st);
}

}  // extern "C"
