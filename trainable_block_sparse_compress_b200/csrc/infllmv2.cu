// infllmv2.cu -- C ABI of the InfLLM v2 block-sparse attention library (sm_100a).
//
// Host side of every entry point declared in include/infllmv2.h: argument checks
// before any launch, TMA tensor-map encoding (driver entry point fetched through the
// runtime, so the library needs no -lcuda), workspace carving and kernel launches on
// the caller's stream.  All device code lives in the included .cuh files.
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>
#include <cstring>
#include <initializer_list>
#include <map>
#include <mutex>
#include <tuple>
#include <utility>

#include "../../include/infllmv2.h"
#include "append.cuh"
#include "attn.cuh"
#include "attn_bwd.cuh"
#include "attn_bwd_tc.cuh"
#include "attn_dec.cuh"
#include "attn_tc.cuh"
#include "common.cuh"
#include "compress.cuh"
#include "decode_step.cuh"
#include "norm_rope.cuh"
#include "select_decode.cuh"
#include "select_prefill.cuh"
#include "select_prefill_tc.cuh"
#include "topk.cuh"
#include "window.cuh"
#include "window_bwd_tc.cuh"
#include "window_decode.cuh"
#include "window_tc.cuh"

using namespace infllmv2;

namespace {

constexpr int kVersion = 300;  // 0.3.0

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_params(const infllmv2_params* p) {
  if (p == nullptr) return INFLLMV2_ERR_INVALID_ARG;
  if (p->batch < 1 || p->num_kv_heads < 1 || p->num_q_heads < 1 || p->head_dim < 1) return INFLLMV2_ERR_INVALID_ARG;
  if (p->num_q_heads % p->num_kv_heads != 0) return INFLLMV2_ERR_INVALID_ARG;
  if (p->block_size < 1 || p->kernel_size < 1 || p->kernel_stride < 1) return INFLLMV2_ERR_INVALID_ARG;
  if (p->topk < 1 || p->n_init < 0 || p->n_local < 0) return INFLLMV2_ERR_INVALID_ARG;
  if (static_cast<long long>(p->n_init) + p->n_local > p->topk) return INFLLMV2_ERR_INVALID_ARG;
  if (!(p->softmax_scale <= 0.f || std::isfinite(p->softmax_scale))) return INFLLMV2_ERR_INVALID_ARG;
  if ((p->score_mode != INFLLMV2_SCORE_SOFTMAX_SUM && p->score_mode != INFLLMV2_SCORE_LOGIT_SUM) ||
      (p->pool_mode != INFLLMV2_POOL_OVERLAP && p->pool_mode != INFLLMV2_POOL_INSIDE))
    return INFLLMV2_ERR_INVALID_ARG;
  const int G = p->num_q_heads / p->num_kv_heads;
  if (p->head_dim != kHeadDim || p->block_size != kBlock || p->kernel_size != kKernel ||
      p->kernel_stride != kStride)
    return INFLLMV2_ERR_UNSUPPORTED;
  if (!(G == 1 || G == 2 || G == 4 || G == 8 || G == 16)) return INFLLMV2_ERR_UNSUPPORTED;
  if (p->topk > kMaxTopk) return INFLLMV2_ERR_UNSUPPORTED;
  if (static_cast<long long>(p->batch) * p->num_q_heads > (1LL << 24)) return INFLLMV2_ERR_UNSUPPORTED;
  return INFLLMV2_OK;
}

int check_len(int32_t L) { return (L >= 1 && L <= INFLLMV2_MAX_SEQ_LEN) ? INFLLMV2_OK : INFLLMV2_ERR_INVALID_ARG; }

int64_t num_kernels(int64_t n) { return n >= kKernel ? (n - kKernel) / kStride + 1 : 0; }
int64_t num_blocks(int64_t n) { return (n + kBlock - 1) / kBlock; }
int round32(int64_t x) { return static_cast<int>((x + 31) / 32 * 32); }

float scale_log2(const infllmv2_params* p) {
  const float s = p->softmax_scale > 0.f ? p->softmax_scale : 1.f / std::sqrt(static_cast<float>(p->head_dim));
  return s * 1.4426950408889634f;
}

// ------------------------------------------------------------ tensor maps

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

bool get_encoder() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode != nullptr;
}

// 2-D view [rows, 128] of a bf16 tensor, box {64 columns, box_rows}, 128-byte swizzle,
// zero fill outside the tensor.
bool make_map(CUtensorMap* m, const void* ptr, uint64_t rows, uint32_t box_rows) {
  if (!get_encoder()) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(kHeadDim), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(kHeadDim) * 2};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// 3-D view [tokens, heads, 128] of the prefill queries, box {64 columns, G heads, 128 / G
// tokens}: the 128 (token, head) rows of one selection tile.
bool make_q_map_3d(CUtensorMap* m, const void* q, uint64_t tokens, uint64_t heads, int G) {
  if (!get_encoder()) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(kHeadDim), static_cast<cuuint64_t>(heads),
                        static_cast<cuuint64_t>(tokens)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(kHeadDim) * 2, static_cast<cuuint64_t>(heads * kHeadDim * 2)};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(128 / G)};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// 3-D view [sequence x kv-head, tokens, 128] of keys or values, box {64 columns, 64 tokens, 1};
// rows at or past `rows` (of Lmax) read as zeros.
bool make_kv_map_3d(CUtensorMap* m, const void* ptr, uint64_t items, uint64_t rows, uint64_t Lmax) {
  if (!get_encoder()) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(kHeadDim), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(items)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(kHeadDim) * 2, static_cast<cuuint64_t>(Lmax * kHeadDim * 2)};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(kWfSeg), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// 4-D view [sequence, token, head, 128] of query rows, box {64 columns, G heads, 128 / G tokens,
// 1}: the rows of a tile past a sequence's Lq tokens read as zeros.
bool make_q_map_4d(CUtensorMap* m, const void* q, uint64_t B, uint64_t Lq, uint64_t heads, int G) {
  if (!get_encoder()) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(kHeadDim), static_cast<cuuint64_t>(heads),
                        static_cast<cuuint64_t>(Lq), static_cast<cuuint64_t>(B)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(kHeadDim) * 2, static_cast<cuuint64_t>(heads * kHeadDim * 2),
                           static_cast<cuuint64_t>(Lq * heads * kHeadDim * 2)};
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(128 / G), 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(q), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

constexpr size_t kMaxSmem = 227 * 1024;

int launch_status() { return cudaGetLastError() == cudaSuccess ? INFLLMV2_OK : INFLLMV2_ERR_CUDA; }

// The status of a runtime call that failed: reported here, not by the next call's launch_status().
int cuda_failed() {
  (void)cudaGetLastError();
  return INFLLMV2_ERR_CUDA;
}

constexpr int kMaxCachedDevices = 64;

// Multiprocessors of the current device (looked up once per device).
int num_sms() {
  static std::atomic<int> cache[kMaxCachedDevices];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (dev < kMaxCachedDevices && (n = cache[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
  if (dev < kMaxCachedDevices) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

int set_smem(const void* fn, size_t bytes) {
  return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) ==
                 cudaSuccess
             ? INFLLMV2_OK
             : cuda_failed();
}

// Clusters of C CTAs of `kern` that the device holds at once (cached per kernel, size, threads,
// shared memory and device), or -1 when a runtime call fails.
template <typename... Params>
int max_active_clusters(void (*kern)(Params...), int C, int threads, size_t smem) {
  static std::mutex mu;
  static std::map<std::tuple<const void*, int, int, size_t, int>, int> cache;
  const void* fn = reinterpret_cast<const void*>(kern);
  int dev = 0, active = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cuda_failed(), -1;
  std::lock_guard<std::mutex> lock(mu);
  const auto key = std::make_tuple(fn, C, threads, smem, dev);
  auto it = cache.find(key);
  if (it != cache.end()) return it->second;
  if (set_smem(fn, smem) != INFLLMV2_OK) return -1;
  if (C > 8 && cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return cuda_failed(), -1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(C));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(C);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaOccupancyMaxActiveClusters(&active, kern, &cfg);
  if (e != cudaSuccess) {
    (void)cuda_failed();
    if (e != cudaErrorInvalidClusterSize) return -1;
    active = 0;  // a size that the device cannot hold
  }
  cache.emplace(key, active);
  return active;
}

// Launches `kern` on a 1-D grid in clusters of C CTAs.  Sizes above 8 need the
// non-portable opt-in.  With `pdl` the kernel may start while the previous kernel on the
// stream finishes (it must call grid_dependency_wait() before reading any input).  A cluster
// shape that the device cannot co-schedule is reported as unsupported before any launch.
template <typename... Params, typename... Args>
int launch_cluster(void (*kern)(Params...), unsigned grid, int C, int threads, size_t smem, cudaStream_t s,
                   bool pdl, Args&&... args) {
  const int fits = max_active_clusters(kern, C, threads, smem);
  if (fits < 0) return INFLLMV2_ERR_CUDA;
  if (fits < 1) return INFLLMV2_ERR_UNSUPPORTED;
  const void* fn = reinterpret_cast<const void*>(kern);
  int st = set_smem(fn, smem);
  if (st != INFLLMV2_OK) return st;
  if (C > 8 && cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return cuda_failed();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(C);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...) == cudaSuccess ? INFLLMV2_OK : cuda_failed();
}

// Launches `kern` so that it may start while the previous kernel on the stream finishes (it
// calls grid_dependency_wait() before it reads anything that kernel wrote).
template <typename... Params, typename... Args>
int launch_pdl(void (*kern)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...) == cudaSuccess ? INFLLMV2_OK : cuda_failed();
}

// Decode work layout.  Each (sequence, kv-head) item's selected blocks are split over
// CTAs.  Normally a cluster of C CTAs (a power of two up to 16, as large as keeps all
// CTAs resident at two per SM) merges its partials in distributed shared memory.  When
// even 16 CTAs per item leave most SMs idle (fewer items than SMs / 16), the blocks are
// split further, two or more per CTA, and the partials meet in the workspace.
struct DecodePlan {
  int cluster;   // CTAs per cluster (cluster path), 0 for the workspace path
  int n_splits;  // workspace path: splits per item
  int per_split;
};

DecodePlan decode_plan(const infllmv2_params* p) {
  const long long items = static_cast<long long>(p->batch) * p->num_kv_heads;
  const long long target = 2LL * num_sms();
  DecodePlan d{0, 1, p->topk};
  if (items * kAdMaxCluster >= num_sms()) {
    int c = 1;
    while (c < kAdMaxCluster && items * c * 2 <= target) c *= 2;
    d.cluster = c;
    return d;
  }
  int s = static_cast<int>(std::min<long long>((target + items - 1) / items, (p->topk + 1) / 2));
  s = std::max(1, std::min(s, kMaxDecodeSplits));
  d.per_split = (p->topk + s - 1) / s;
  d.n_splits = (p->topk + d.per_split - 1) / d.per_split;
  return d;
}

// Selection cluster size: enough CTAs for the longest sequence's kernels (at most
// kSdMaxChunk per CTA), and as many as keep all CTAs resident at two per SM.
int select_cluster(const infllmv2_params* p, int64_t nk) {
  const long long items = static_cast<long long>(p->batch) * p->num_kv_heads;
  const long long target = 2LL * num_sms();
  int c = 1;
  while (c < kSdMaxCluster && (static_cast<int64_t>(c) * kSdMaxChunk < nk || items * c * 2 <= target)) c *= 2;
  return c;
}

// Decode-step cluster size: enough CTAs for the longest sequence's kernels (at most
// kSdMaxChunk per CTA), then doubled while all CTAs stay at two per SM and every item's
// cluster is resident at once (a cluster left for a second wave costs a whole step).
int decode_step_cluster(const infllmv2_params* p, int64_t nk) {
  const long long items = static_cast<long long>(p->batch) * p->num_kv_heads;
  const long long target = 2LL * num_sms();
  int c = 1;
  while (c < kSdMaxCluster && static_cast<int64_t>(c) * kSdMaxChunk < nk) c *= 2;
  while (c < kSdMaxCluster && items * c * 2 <= target &&
         items <= max_active_clusters(decode_step_kernel, 2 * c, kSdThreads, decode_step_smem_bytes()))
    c *= 2;
  return c;
}

// Workspace of the backward pass, in order (each part 256-byte aligned): D [B, Hq, L]
// fp32; cnt, cursor, off [n] and segoff [n + 1] int32 (n = B * Hkv * blocks); the row
// lists [B * Hkv * L * topk] int32; dK and dV accumulators [B, Hkv, L, d] fp32.
struct BwdLayout {
  size_t delta, cnt, cursor, off, segoff, list, dk, dv, total;
  long long n;
};
BwdLayout bwd_layout(const infllmv2_params* p, int32_t L) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  BwdLayout w;
  const size_t B = p->batch, Hq = p->num_q_heads, Hkv = p->num_kv_heads;
  w.n = static_cast<long long>(B * Hkv * num_blocks(L));
  w.delta = 0;
  w.cnt = up(w.delta + B * Hq * L * 4);
  w.cursor = up(w.cnt + w.n * 4);
  w.off = up(w.cursor + w.n * 4);
  w.segoff = up(w.off + w.n * 4);
  w.list = up(w.segoff + (w.n + 1) * 4);
  w.dk = up(w.list + B * Hkv * static_cast<size_t>(L) * p->topk * 4);
  w.dv = up(w.dk + B * Hkv * static_cast<size_t>(L) * kHeadDim * 4);
  w.total = up(w.dv + B * Hkv * static_cast<size_t>(L) * kHeadDim * 4);
  return w;
}

// Row tiles and key splits of the window attention's forward.  A CTA has 256 rows while such tiles
// keep every SM busy, else 128 rows with the keys shared between its two warpgroups; when even
// those leave more than half of the SMs idle, the keys of each are split over up to 32 CTAs and
// joined through the workspace, but not below four key tiles (of `key_tiles`) a CTA: the join
// costs more than that.
struct WindowPlan {
  int rows, row_tiles;
  long long items;  // row_tiles * B * Hkv
  int n_splits;
};
WindowPlan window_plan(const infllmv2_params* p, int32_t Lq, long long key_tiles) {
  WindowPlan d;
  const int G = p->num_q_heads / p->num_kv_heads;
  const long long bg = static_cast<long long>(p->batch) * p->num_kv_heads;
  d.rows = (Lq + 256 / G - 1) / (256 / G) * bg >= num_sms() ? 256 : 128;
  d.row_tiles = (Lq + d.rows / G - 1) / (d.rows / G);
  d.items = d.row_tiles * bg;
  d.n_splits = static_cast<int>(
      std::max<long long>(1, std::min(std::min<long long>(32, key_tiles / 4), num_sms() / d.items)));
  return d;
}

// Chunks of the window decode.  Up to 8 segments are one chunk: the join costs as much as the
// segments (8.2 us either way at 8 segments, 10.3 against 8.2 with 64 items, and 2 us more host
// time).  Beyond that, while every (sequence, kv-head)'s segments make no more than 8 per CTA slot
// (two CTAs an SM), one wave takes them, at least two a chunk; beyond that about six waves of chunks
// even out ragged lengths.  Chunks that a cluster of 16 could take with at most half as many again
// are one, while the device holds every item's cluster at once.  Counted for full caches of Lmax
// tokens.
struct WindowDecodePlan {
  int per_chunk, chunks;
  bool cluster;
};
WindowDecodePlan window_decode_plan(const infllmv2_params* p, int32_t Lmax, int32_t window, int32_t n_sink) {
  const long long items = static_cast<long long>(p->batch) * p->num_kv_heads, slots = 2LL * num_sms();
  const long long win = (std::min<long long>(window, Lmax) + kWfSeg - 1) / kWfSeg;
  // two runs of keys may make one segment more than one run of the whole cache
  const long long segs = std::min<long long>(num_blocks(Lmax) + 1, win + (std::min<long long>(n_sink, Lmax) + kWfSeg - 1) / kWfSeg);
  if (segs <= 8) return {8, 1, false};
  const long long each = (items * segs + slots - 1) / slots;
  const long long per = each <= 8 ? std::max<long long>(2, each) : std::max<long long>(8, (each + 5) / 6);
  const long long per_c = std::max(per, (segs + kWdMaxCluster - 1) / kWdMaxCluster);
  if (2 * per_c <= 3 * per) {
    const int chunks = static_cast<int>((segs + per_c - 1) / per_c);
    if (items <= max_active_clusters(window_decode_kernel<true>, chunks, kWdThreads, window_decode_smem_bytes()))
      return {static_cast<int>(per_c), chunks, true};
  }
  return {static_cast<int>(per), static_cast<int>((segs + per - 1) / per), false};
}

// Backward of the window attention: cuts of the key tiles' query ranges (counted for sequences
// of L tokens).  The aim is two CTAs of equal work an SM, at least 16 query tiles each (a partial
// costs a write and a read of 128 KB): a kind of key tile whose range is n such shares, rounded,
// is cut into n chunks, unless that needs more than kWbMaxParts partials (then the shares grow).
constexpr int kWbMaxParts = 512;
constexpr size_t kWbPartBytes = 2 * kWbKeys * kHeadDim * sizeof(float);
struct WindowBwdPlan {
  int key_tiles, sink_tiles, chunks_s, chunks_w, q_tiles_s, q_tiles_w;
  long long parts;  // partials of all (sequence, kv-head)s
  size_t lse2, delta, part, total;
};
WindowBwdPlan window_bwd_plan(const infllmv2_params* p, int32_t L, int32_t window, int32_t n_sink) {
  WindowBwdPlan d;
  const long long G = p->num_q_heads / p->num_kv_heads, items = static_cast<long long>(p->batch) * p->num_kv_heads;
  d.key_tiles = (L + kWbKeys - 1) / kWbKeys;
  d.sink_tiles = static_cast<int>(std::min<long long>(d.key_tiles, (static_cast<long long>(n_sink) + kWbKeys - 1) / kWbKeys));
  long long visits = 0, longest[2] = {0, 0};
  for (int i = 0; i < d.key_tiles; ++i) {
    const bool sink = i < d.sink_tiles;
    const long long u0 = static_cast<long long>(i) * kWbKeys;
    const long long end = sink ? L : std::min<long long>(L, u0 + kWbKeys - 1 + window);
    const long long n = ((end - u0) * G + 127) / 128;
    visits += n;
    longest[sink] = std::max(longest[sink], n);
  }
  long long q = std::max<long long>(16, visits * items / (2 * num_sms()) + 1);
  for (;; q += q / 4) {
    d.chunks_s = static_cast<int>(std::max<long long>(1, (longest[1] + q / 2) / q));
    d.chunks_w = static_cast<int>(std::max<long long>(1, (longest[0] + q / 2) / q));
    d.parts = items * ((d.chunks_s > 1 ? static_cast<long long>(d.sink_tiles) * d.chunks_s : 0) +
                       (d.chunks_w > 1 ? static_cast<long long>(d.key_tiles - d.sink_tiles) * d.chunks_w : 0));
    if (d.parts <= kWbMaxParts) break;
  }
  d.q_tiles_s = static_cast<int>(std::max<long long>(1, (longest[1] + d.chunks_s - 1) / d.chunks_s));
  d.q_tiles_w = static_cast<int>(std::max<long long>(1, (longest[0] + d.chunks_w - 1) / d.chunks_w));
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t stats = up(static_cast<size_t>(p->batch) * p->num_q_heads * d.key_tiles * kWbKeys * sizeof(float));
  d.lse2 = 0;
  d.delta = stats;
  d.part = 2 * stats;
  d.total = d.part + static_cast<size_t>(d.parts) * kWbPartBytes;
  return d;
}

unsigned norm_rope_bwd_grid(const infllmv2_params* p, int32_t Lq, NormRopeParams* a);
// CTAs per SM of the norm-and-rotation kernels, and waves of the forward.
constexpr int kNrCtas = 4, kNrWaves = 32;

size_t ws_size(const infllmv2_params* p, int op, int32_t L) {
  if (check_params(p) != INFLLMV2_OK || check_len(L) != INFLLMV2_OK) return static_cast<size_t>(-1);
  switch (op) {
    case INFLLMV2_OP_COMPRESS:
    case INFLLMV2_OP_SELECT_PREFILL:
    case INFLLMV2_OP_ATTN_PREFILL:
      return 0;
    case INFLLMV2_OP_SELECT_DECODE:
      return 0;
    case INFLLMV2_OP_ATTN_BACKWARD:
      return bwd_layout(p, L).total;
    case INFLLMV2_OP_ATTN_DECODE: {
      const DecodePlan d = decode_plan(p);
      if (d.cluster > 0) return 0;
      const size_t rows = static_cast<size_t>(p->batch) * p->num_kv_heads * d.n_splits * kGroupRows;
      return rows * kHeadDim * sizeof(float) + rows * sizeof(float);
    }
    case INFLLMV2_OP_QK_NORM_ROPE_BACKWARD: {
      NormRopeParams a;
      return static_cast<size_t>(norm_rope_bwd_grid(p, L, &a)) * kHeadDim * sizeof(float);
    }
    case INFLLMV2_OP_WINDOW_ATTN: {
      const WindowPlan d = window_plan(p, L, 1 << 30);  // for every window
      return d.n_splits == 1 ? 0 : static_cast<size_t>(d.items) * d.n_splits * d.rows * (kHeadDim + 1) * sizeof(float);
    }
    case INFLLMV2_OP_WINDOW_DECODE: {  // for every window and n_sink: window_decode_plan's chunks at most
      const size_t items = static_cast<size_t>(p->batch) * p->num_kv_heads, segs = num_blocks(L) + 1;
      if (segs <= 2) return 0;
      const size_t most = std::min<size_t>(12 * static_cast<size_t>(num_sms()) + items, items * ((segs + 1) / 2));
      return most * (p->num_q_heads / p->num_kv_heads) * (kHeadDim + 1) * sizeof(float);
    }
    case INFLLMV2_OP_WINDOW_BACKWARD: {  // for every window and n_sink
      const WindowBwdPlan d = window_bwd_plan(p, L, L, 0);
      const long long most = static_cast<long long>(p->batch) * p->num_kv_heads * d.key_tiles *
                             ((static_cast<long long>(L) * (p->num_q_heads / p->num_kv_heads) + 2047) / 2048 + 1);
      return d.part + static_cast<size_t>(std::min<long long>(kWbMaxParts, most)) * kWbPartBytes;
    }
    default:
      return static_cast<size_t>(-1);
  }
}

int check_chunk(int32_t Lq, const int32_t* q_lens, const int32_t* kv_lens, int32_t Lmax);

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Shared checks and parameters of the norm-and-rotation calls.
int norm_rope_args(const infllmv2_params* p, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                   int32_t Lq, const void* qw, const void* kw, int32_t weights_fp32, float eps, const float* table,
                   int32_t table_rows, int32_t rot, int32_t interleaved, const int32_t* starts,
                   const int32_t* q_lens, NormRopeParams& a) {
  int st = check_params(p);
  if (st != INFLLMV2_OK) return st;
  if ((st = check_len(Lq)) != INFLLMV2_OK || (st = check_len(table_rows)) != INFLLMV2_OK) return st;
  if (!q || !k || !table || !aligned16(q) || !aligned16(k) || !aligned16(table) || !aligned16(qw) || !aligned16(kw) ||
      !aligned4(starts) || !aligned4(q_lens))
    return INFLLMV2_ERR_INVALID_ARG;
  const int64_t qn = static_cast<int64_t>(p->num_q_heads) * kHeadDim, kn = static_cast<int64_t>(p->num_kv_heads) * kHeadDim;
  if (q_stride < qn || k_stride < kn || q_stride % 8 != 0 || k_stride % 8 != 0) return INFLLMV2_ERR_INVALID_ARG;
  if (static_cast<uint64_t>(p->batch) * Lq > 0x7fffffffULL) return INFLLMV2_ERR_UNSUPPORTED;  // 32-bit token numbers
  if (!(eps > 0.f) || !std::isfinite(eps)) return INFLLMV2_ERR_INVALID_ARG;
  if (rot < 16 || rot > kHeadDim || rot % 16 != 0) return INFLLMV2_ERR_INVALID_ARG;
  if ((interleaved != 0 && interleaved != 1) || (weights_fp32 != 0 && weights_fp32 != 1)) return INFLLMV2_ERR_INVALID_ARG;
  a = {};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.qw = qw;
  a.kw = kw;
  a.table = table;
  a.starts = starts;
  a.q_lens = q_lens;
  a.B = p->batch;
  a.Lq = Lq;
  a.Hq = p->num_q_heads;
  a.Hkv = p->num_kv_heads;
  a.weights_fp32 = weights_fp32;
  a.table_rows = table_rows;
  a.rot = rot;
  a.eps = eps;
  return INFLLMV2_OK;
}

// Heads of one chunk: up to 8 heads a half-warp (the table row and the weights are loaded once for
// them), fewer while the launch would leave half of the GPU's warps (ctas_per_sm CTAs an SM)
// without work.  Returns the token pairs.
long long norm_rope_chunks(const infllmv2_params* p, int32_t Lq, int ctas_per_sm, NormRopeParams* a) {
  const long long pairs = (static_cast<long long>(p->batch) * Lq + 1) / 2;
  const long long room = static_cast<long long>(ctas_per_sm) * num_sms();
  const int Hq = p->num_q_heads, H2 = 2 * p->num_kv_heads;
  int heads = 8;
  for (; heads > 1; heads = (heads + 1) / 2)
    if (pairs * ((Hq + heads - 1) / heads + (H2 + heads - 1) / heads) * 2 > room * kNrWarps) break;
  const int qc = (Hq + heads - 1) / heads;  // evened out over the query chunks
  a->heads = heads == 1 ? 1 : std::max((Hq + qc - 1) / qc, std::min(heads, H2));
  a->q_chunks = (Hq + a->heads - 1) / a->heads;
  a->kv_chunks = (H2 + a->heads - 1) / a->heads;
  return pairs;
}

// Grid of the forward (0: too large): as many CTAs for every chunk, at most kNrWaves waves.
unsigned norm_rope_grid(const infllmv2_params* p, int32_t Lq, NormRopeParams* a) {
  const long long pairs = norm_rope_chunks(p, Lq, kNrCtas, a), chunks = a->q_chunks + a->kv_chunks;
  const long long room = static_cast<long long>(kNrWaves) * kNrCtas * num_sms();
  const long long x = std::min<long long>((pairs + kNrWarps - 1) / kNrWarps, std::max<long long>(1, room / chunks));
  a->q_ctas = a->kv_ctas = static_cast<int>(x);
  return x * chunks > 0x7fffffffLL ? 0u : static_cast<unsigned>(x * chunks);
}

// Grid of the backward (0: too large): one wave, dealt to the chunks by the rows that they move for a
// token (three a query or key head, two a value head).
unsigned norm_rope_bwd_grid(const infllmv2_params* p, int32_t Lq, NormRopeParams* a) {
  const long long most = (norm_rope_chunks(p, Lq, kNrBwdCtas, a) + kNrWarps - 1) / kNrWarps;
  const long long room = static_cast<long long>(kNrBwdCtas) * num_sms(), qc = a->q_chunks, kc = a->kv_chunks;
  const long long wq = 3 * a->heads, wkv = 5 * ((p->num_kv_heads + kc - 1) / kc);
  const long long xq = std::max<long long>(1, room * wq / (qc * wq + kc * wkv));
  const long long xkv = std::max<long long>(1, (room - qc * xq) / kc);
  a->q_ctas = static_cast<int>(std::min(most, xq));
  a->kv_ctas = static_cast<int>(std::min(most, xkv));
  const long long grid = qc * a->q_ctas + kc * a->kv_ctas;
  return grid > 0x7fffffffLL ? 0u : static_cast<unsigned>(grid);
}

// Shared checks and parameters of the window attention calls.
int window_args(const infllmv2_params* p, const void* q, int32_t Lq, const void* k, const void* v,
                const int32_t* q_lens, const int32_t* kv_lens, int32_t Lmax, int32_t window, int32_t n_sink,
                WinParams& a) {
  int st = check_params(p);
  if (st != INFLLMV2_OK) return st;
  if ((st = check_chunk(Lq, q_lens, kv_lens, Lmax)) != INFLLMV2_OK) return st;
  if (!q || !k || !v || !aligned16(q) || !aligned16(k) || !aligned16(v)) return INFLLMV2_ERR_INVALID_ARG;
  if (window < 1 || n_sink < 0) return INFLLMV2_ERR_INVALID_ARG;
  if (static_cast<uint64_t>(p->batch) * Lq * p->num_q_heads > 0x7fffffffULL ||
      static_cast<uint64_t>(p->batch) * p->num_kv_heads * Lmax > 0x7fffffffULL)
    return INFLLMV2_ERR_UNSUPPORTED;  // 32-bit row numbers
  a = {};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.q_lens = q_lens;
  a.kv_lens = kv_lens;
  a.B = p->batch;
  a.Hq = p->num_q_heads;
  a.Hkv = p->num_kv_heads;
  a.G = p->num_q_heads / p->num_kv_heads;
  a.Lq = Lq;
  a.Lmax = Lmax;
  a.window = window;
  a.n_sink = n_sink;
  a.scale_log2 = scale_log2(p);
  a.scale = a.scale_log2 / 1.4426950408889634f;
  return INFLLMV2_OK;
}

// Chunk arguments: Lq and Lmax in [1, INFLLMV2_MAX_SEQ_LEN], Lq <= Lmax, length arrays
// 4-byte aligned (their values are read and clamped on the GPU).
int check_chunk(int32_t Lq, const int32_t* q_lens, const int32_t* kv_lens, int32_t Lmax) {
  if (check_len(Lq) != INFLLMV2_OK || check_len(Lmax) != INFLLMV2_OK || Lq > Lmax) return INFLLMV2_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(q_lens) & 3u) || (reinterpret_cast<uintptr_t>(kv_lens) & 3u))
    return INFLLMV2_ERR_INVALID_ARG;
  return INFLLMV2_OK;
}

// Prefill selection for Lq query rows per sequence against caches of Lmax tokens: a fresh
// prefill (q_lens = kv_lens = NULL, Lq = Lmax = L) or a chunk of the last q_lens[b] of
// kv_lens[b] cached tokens.
int select_prefill(const infllmv2_params* p, const void* q, int32_t Lq, const void* kc, const int32_t* q_lens,
                   const int32_t* kv_lens, int32_t Lmax, int32_t* block_idx, cudaStream_t s) {
  if (q == nullptr || block_idx == nullptr || !aligned16(q) || !aligned16(block_idx)) return INFLLMV2_ERR_INVALID_ARG;
  const int64_t nk = num_kernels(Lmax);
  if (nk > 0 && (kc == nullptr || !aligned16(kc))) return INFLLMV2_ERR_INVALID_ARG;
  if (static_cast<uint64_t>(p->batch) * p->num_kv_heads * static_cast<uint64_t>(nk) > 0x7fffffffULL ||
      static_cast<uint64_t>(p->batch) * Lq > 0x7fffffffULL)
    return INFLLMV2_ERR_UNSUPPORTED;  // TMA coordinates are 32-bit
  const int G = p->num_q_heads / p->num_kv_heads;
  const int nblk_cap = round32(num_blocks(Lmax));
  CUtensorMap tm_kc;
  std::memset(&tm_kc, 0, sizeof tm_kc);
  if (nk > 0) {
    if (!make_map(&tm_kc, kc, static_cast<uint64_t>(p->batch) * p->num_kv_heads * nk, kKcTile))
      return INFLLMV2_ERR_CUDA;
  } else {
    // no complete kernel: every row keeps only its forced blocks; the kernel path runs
    // with an empty score loop (no tile is loaded, so the map is never dereferenced)
    if (!make_map(&tm_kc, q, kKcTile, kKcTile)) return INFLLMV2_ERR_CUDA;
  }
  SelPrefillParams a;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.idx = block_idx;
  a.q_lens = q_lens;
  a.kv_lens = kv_lens;
  a.B = p->batch;
  a.Lq = Lq;
  a.Lmax = Lmax;
  a.Hq = p->num_q_heads;
  a.Hkv = p->num_kv_heads;
  a.G = G;
  a.NKmax = static_cast<int>(nk);
  a.topk = p->topk;
  a.n_init = p->n_init;
  a.n_local = p->n_local;
  a.score_mode = p->score_mode;
  a.pool_mode = p->pool_mode;
  a.nblk_cap = nblk_cap;
  a.scale_log2 = scale_log2(p);
  int st;
  // tensor-core path: 128 / G tokens x G heads per 128-row UMMA tile, with a 3-slot Kc
  // ring, or 2 slots when the block keys of long sequences need the room
  a.stages = sel_tc_smem_bytes(nblk_cap, G, 3) <= kMaxSmem ? 3 : 2;
  if (nk > 0 && sel_tc_smem_bytes(nblk_cap, G, a.stages) <= kMaxSmem) {
    const int tt = sel_tc_tokens(G);
    a.tiles_per_bg = (Lq + tt - 1) / tt;
    const long long grid = static_cast<long long>(a.tiles_per_bg) * p->batch * p->num_kv_heads;
    if (grid > 0x7fffffffLL) return INFLLMV2_ERR_UNSUPPORTED;
    CUtensorMap tm_q3, tm_kca, tm_kcb;
    const uint64_t kc_rows = static_cast<uint64_t>(p->batch) * p->num_kv_heads * nk;
    if (!make_q_map_3d(&tm_q3, q, static_cast<uint64_t>(p->batch) * Lq, p->num_q_heads, G) ||
        !make_map(&tm_kca, kc, kc_rows, kTcN) || !make_map(&tm_kcb, kc, kc_rows, kTcNB))
      return INFLLMV2_ERR_CUDA;
    const size_t smem = sel_tc_smem_bytes(nblk_cap, G, a.stages);
    auto run = [&](auto kern) -> int {
      int r = set_smem(reinterpret_cast<const void*>(kern), smem);
      if (r != INFLLMV2_OK) return r;
      kern<<<static_cast<unsigned>(grid), kTcThreads, smem, s>>>(tm_q3, tm_kca, tm_kcb, a);
      return launch_status();
    };
    switch (G) {
      case 16: return run(select_prefill_tc_kernel<16>);
      case 8: return run(select_prefill_tc_kernel<8>);
      case 4: return run(select_prefill_tc_kernel<4>);
      case 2: return run(select_prefill_tc_kernel<2>);
      default: return run(select_prefill_tc_kernel<1>);
    }
  }
  // m16n8k16 path: 8 tokens per CTA, one warp per token
  a.tiles_per_bg = (Lq + kSelWarps - 1) / kSelWarps;
  const long long grid = static_cast<long long>(a.tiles_per_bg) * p->batch * p->num_kv_heads;
  if (grid > 0x7fffffffLL) return INFLLMV2_ERR_UNSUPPORTED;
  const size_t smem = sel_prefill_smem_bytes(nblk_cap);
  if ((st = set_smem(reinterpret_cast<const void*>(select_prefill_kernel), smem)) != INFLLMV2_OK) return st;
  select_prefill_kernel<<<static_cast<unsigned>(grid), kSelThreads, smem, s>>>(tm_kc, a);
  return launch_status();
}

// Maps over the sinks alone (rows past them read as zeros); without sinks no segment uses them.
bool sink_maps(const WinParams& w, const CUtensorMap& tk, const CUtensorMap& tv, CUtensorMap* tks, CUtensorMap* tvs) {
  if (w.n_sink == 0) {
    *tks = tk;
    *tvs = tv;
    return true;
  }
  const uint64_t items = static_cast<uint64_t>(w.B) * w.Hkv, sinks = static_cast<uint64_t>(std::min(w.n_sink, w.Lmax));
  return make_kv_map_3d(tks, w.k, items, sinks, w.Lmax) && make_kv_map_3d(tvs, w.v, items, sinks, w.Lmax);
}

// Forward of the window attention on the tensor cores.
int launch_window(const infllmv2_params* p, const WinParams& w, void* ws, cudaStream_t s) {
  const long long tokens = std::min<long long>(w.Lq, 256 / w.G);  // of a CTA
  const long long keys = std::min<long long>(w.Lmax, std::min<long long>(w.Lmax, static_cast<long long>(w.window) + tokens) +
                                                         std::min<long long>(w.Lmax, w.n_sink));
  const WindowPlan d = window_plan(p, w.Lq, (keys + 127) / 128);
  WinTcParams a;
  a.rows = d.rows;
  a.w = w;
  a.g_log2 = 0;
  while ((1 << a.g_log2) < w.G) ++a.g_log2;
  a.row_tiles = d.row_tiles;
  a.n_splits = d.n_splits;
  a.part_o = static_cast<float*>(ws);
  a.part_lse = d.n_splits > 1 ? a.part_o + static_cast<size_t>(d.items) * d.n_splits * d.rows * kHeadDim : nullptr;
  const uint64_t items = static_cast<uint64_t>(w.B) * w.Hkv;
  CUtensorMap tq, tk, tv, tks, tvs;
  if (!make_q_map_3d(&tq, w.q, static_cast<uint64_t>(w.B) * w.Lq, w.Hq, w.G) ||
      !make_kv_map_3d(&tk, w.k, items, w.Lmax, w.Lmax) || !make_kv_map_3d(&tv, w.v, items, w.Lmax, w.Lmax) ||
      !sink_maps(w, tk, tv, &tks, &tvs))
    return INFLLMV2_ERR_CUDA;
  const size_t smem = window_tc_smem_bytes();
  auto run = [&](auto kern) {
    const int st = set_smem(reinterpret_cast<const void*>(kern), smem);
    if (st != INFLLMV2_OK) return st;
    return launch_pdl(kern, dim3(static_cast<unsigned>(d.items * d.n_splits)), kWfThreads, smem, s, tq, tk, tv, tks, tvs, a);
  };
  const int st = d.rows == 128 ? run(window_tc_kernel<true>) : run(window_tc_kernel<false>);
  if (st != INFLLMV2_OK || d.n_splits == 1) return st;
  const long long rows = static_cast<long long>(w.B) * w.Lq * w.Hq;
  return launch_pdl(window_merge_kernel, dim3(static_cast<unsigned>((rows + 7) / 8)), 256, 0, s, a);
}

int launch_window_decode(const infllmv2_params* p, const WinParams& w, void* ws, cudaStream_t s) {
  const WindowDecodePlan d = window_decode_plan(p, w.Lmax, w.window, w.n_sink);
  WinDecodeParams a;
  a.w = w;
  a.g_log2 = 0;
  while ((1 << a.g_log2) < w.G) ++a.g_log2;
  a.per_chunk = d.per_chunk;
  a.chunks = d.chunks;
  a.part_o = static_cast<float*>(ws);
  const size_t rows = static_cast<size_t>(w.B) * w.Hq * d.chunks;
  a.part_lse = a.part_o + (d.chunks > 1 ? rows * kHeadDim : 0);
  const uint64_t items = static_cast<uint64_t>(w.B) * w.Hkv;
  if (items * d.chunks > 0x7fffffffULL) return INFLLMV2_ERR_UNSUPPORTED;
  CUtensorMap tk, tv, tks, tvs;
  if (!make_kv_map_3d(&tk, w.k, items, w.Lmax, w.Lmax) || !make_kv_map_3d(&tv, w.v, items, w.Lmax, w.Lmax) ||
      !sink_maps(w, tk, tv, &tks, &tvs))
    return INFLLMV2_ERR_CUDA;
  const size_t smem = window_decode_smem_bytes();
  const unsigned grid = static_cast<unsigned>(items * d.chunks);
  if (d.cluster)
    return launch_cluster(window_decode_kernel<true>, grid, d.chunks, kWdThreads, smem, s, true, tk, tv, tks, tvs, a);
  int st = set_smem(reinterpret_cast<const void*>(window_decode_kernel<false>), smem);
  if (st != INFLLMV2_OK) return st;
  st = launch_pdl(window_decode_kernel<false>, grid, kWdThreads, smem, s, tk, tv, tks, tvs, a);
  if (st != INFLLMV2_OK || d.chunks == 1) return st;
  return launch_pdl(window_decode_merge_kernel, static_cast<unsigned>(w.B * w.Hq), 128, 0, s, a);
}

// Backward of the window attention (the workspace has window_bwd_plan's layout).
int launch_window_backward(const infllmv2_params* p, const WinParams& w, void* ws, cudaStream_t s) {
  const WindowBwdPlan d = window_bwd_plan(p, w.Lq, w.window, w.n_sink);
  unsigned char* wb = static_cast<unsigned char*>(ws);
  WinBwdParams a;
  a.w = w;
  a.g_log2 = 0;
  while ((1 << a.g_log2) < w.G) ++a.g_log2;
  a.Lp = d.key_tiles * kWbKeys;
  a.lse2 = reinterpret_cast<float*>(wb + d.lse2);
  a.delta = reinterpret_cast<float*>(wb + d.delta);
  a.part = reinterpret_cast<float*>(wb + d.part);
  a.key_tiles = d.key_tiles;
  a.sink_tiles = d.sink_tiles;
  a.chunks_s = d.chunks_s;
  a.chunks_w = d.chunks_w;
  a.q_tiles_s = d.q_tiles_s;
  a.q_tiles_w = d.q_tiles_w;
  a.row_tiles = (w.Lq * w.G + 127) / 128;
  const uint64_t items = static_cast<uint64_t>(w.B) * w.Hkv;
  CUtensorMap tq, tdo, tk, tv, tks, tvs;
  if (!make_q_map_4d(&tq, w.q, w.B, w.Lq, w.Hq, w.G) || !make_q_map_4d(&tdo, w.d_o, w.B, w.Lq, w.Hq, w.G) ||
      !make_kv_map_3d(&tk, w.k, items, w.Lmax, w.Lmax) || !make_kv_map_3d(&tv, w.v, items, w.Lmax, w.Lmax) ||
      !sink_maps(w, tk, tv, &tks, &tvs))
    return INFLLMV2_ERR_CUDA;
  const size_t smem = window_bwd_smem_bytes();
  int st;
  if ((st = set_smem(reinterpret_cast<const void*>(window_bwd_tc_kernel), smem)) != INFLLMV2_OK) return st;
  const long long delta_items = static_cast<long long>(w.B) * a.Lp * ((w.Hq + 3) / 4);
  const long long ctas = static_cast<long long>(items) * (static_cast<long long>(d.sink_tiles) * d.chunks_s +
                                                          static_cast<long long>(d.key_tiles - d.sink_tiles) * d.chunks_w);
  const long long dq_ctas = static_cast<long long>(items) * a.row_tiles;
  if (delta_items > 0x7fffffffLL || ctas + dq_ctas > 0x7fffffffLL || items > 65535) return INFLLMV2_ERR_UNSUPPORTED;
  a.kv_items = static_cast<int>(ctas);
  const dim3 delta_grid(static_cast<unsigned>(std::min<long long>((delta_items + 15) / 16, 64LL * num_sms())));
  if ((st = launch_pdl(window_delta_kernel, delta_grid, 256, 0, s, a)) != INFLLMV2_OK) return st;
  st = launch_pdl(window_bwd_tc_kernel, dim3(static_cast<unsigned>(ctas + dq_ctas)), kWbThreads, smem, s, tq, tdo, tk, tv,
                  tks, tvs, a);
  if (st != INFLLMV2_OK) return st;
  const int first = d.chunks_s > 1 ? 0 : d.sink_tiles;
  const int split = d.chunks_w > 1 ? d.key_tiles - first : (d.chunks_s > 1 ? d.sink_tiles : 0);
  if (split > 0) {
    const dim3 grid(static_cast<unsigned>(split) * (2 * kWbKeys / 8), static_cast<unsigned>(items));
    return launch_pdl(window_dkdv_merge_kernel, grid, 256, 0, s, a, first, split);
  }
  return INFLLMV2_OK;
}

int launch_attn(const infllmv2_params* p, const void* q, uint64_t q_rows, const void* k, const void* v,
                uint64_t kv_rows, AttnParams& a, cudaStream_t s);

// Prefill attention for Lq query rows per sequence against caches of Lmax tokens (a fresh
// prefill or a chunk, as for select_prefill).
int attn_prefill(const infllmv2_params* p, const void* q, int32_t Lq, const void* k, const void* v,
                 const int32_t* q_lens, const int32_t* kv_lens, int32_t Lmax, const int32_t* block_idx, void* o,
                 float* lse, cudaStream_t s) {
  if (!q || !k || !v || !block_idx || !o) return INFLLMV2_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(block_idx) || !aligned16(o))
    return INFLLMV2_ERR_INVALID_ARG;
  if (lse != nullptr && (reinterpret_cast<uintptr_t>(lse) & 3u)) return INFLLMV2_ERR_INVALID_ARG;
  const uint64_t q_rows = static_cast<uint64_t>(p->batch) * Lq * p->num_q_heads;
  const uint64_t kv_rows = static_cast<uint64_t>(p->batch) * p->num_kv_heads * Lmax;
  if (q_rows > 0x7fffffffULL || kv_rows > 0x7fffffffULL) return INFLLMV2_ERR_UNSUPPORTED;  // 32-bit TMA rows
  AttnParams a;
  a.idx = block_idx;
  a.lens = nullptr;
  a.q_lens = q_lens;
  a.kv_lens = kv_lens;
  a.B = p->batch;
  a.Hq = p->num_q_heads;
  a.Hkv = p->num_kv_heads;
  a.G = p->num_q_heads / p->num_kv_heads;
  a.Lq = Lq;
  a.Lmax = Lmax;
  a.topk = p->topk;
  a.n_splits = 1;
  a.blocks_per_split = p->topk;
  a.scale_log2 = scale_log2(p);
  a.num_items = static_cast<long long>(p->batch) * p->num_kv_heads * Lq;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.part_o = nullptr;
  a.part_lse = nullptr;
  {
    // tensor-core path: per item, K/V block pairs against 16 query rows from the group's
    // first head (for G < 16 the rows past the group are other heads' queries: their
    // columns of S, P and O are computed and never written; rows past the end of q are
    // zero-filled by the copy)
    CUtensorMap tq, tk, tv;
    if (!make_map(&tq, q, q_rows, kGroupRows) || !make_map(&tk, k, kv_rows, kBlock) ||
        !make_map(&tv, v, kv_rows, kBlock))
      return INFLLMV2_ERR_CUDA;
    const size_t smem = attn_tc_smem_bytes();
    int st = set_smem(reinterpret_cast<const void*>(attn_tc_kernel), smem);
    if (st != INFLLMV2_OK) return st;
    const long long grid = std::min<long long>(a.num_items, num_sms());
    if (grid <= 0) return INFLLMV2_OK;
    attn_tc_kernel<<<static_cast<unsigned>(grid), kAtThreads, smem, s>>>(tq, tk, tv, a);
    return launch_status();
  }
}

int launch_attn(const infllmv2_params* p, const void* q, uint64_t q_rows, const void* k, const void* v,
                       uint64_t kv_rows, AttnParams& a, cudaStream_t s) {
  CUtensorMap tq, tk, tv;
  if (!make_map(&tq, q, q_rows, kGroupRows) || !make_map(&tk, k, kv_rows, kBlock) ||
      !make_map(&tv, v, kv_rows, kBlock))
    return INFLLMV2_ERR_CUDA;
  const size_t smem = attn_smem_bytes();
  int st = set_smem(reinterpret_cast<const void*>(attn_kernel), smem);
  if (st != INFLLMV2_OK) return st;
  const long long grid = std::min<long long>(a.num_items, num_sms());
  if (grid <= 0) return INFLLMV2_OK;
  attn_kernel<<<static_cast<unsigned>(grid), kAttnThreads, smem, s>>>(tq, tk, tv, a);
  return launch_status();
}

}  // namespace

extern "C" {

int64_t infllmv2_num_kernels(const infllmv2_params* p, int64_t n) {
  if (p == nullptr || p->kernel_size < 1 || p->kernel_stride < 1 || n < p->kernel_size) return 0;
  return (n - p->kernel_size) / p->kernel_stride + 1;
}

int infllmv2_check_params(const infllmv2_params* p) { return check_params(p); }

int infllmv2_version(void) { return kVersion; }

const char* infllmv2_status_string(int status) {
  switch (status) {
    case INFLLMV2_OK:
      return "ok";
    case INFLLMV2_ERR_INVALID_ARG:
      return "invalid argument";
    case INFLLMV2_ERR_UNSUPPORTED:
      return "unsupported configuration";
    case INFLLMV2_ERR_WORKSPACE:
      return "workspace missing or too small";
    case INFLLMV2_ERR_CUDA:
      return "CUDA error";
    default:
      return "unknown status";
  }
}

size_t infllmv2_workspace_size(const infllmv2_params* p, int op, int32_t L_or_Lmax) {
  return ws_size(p, op, L_or_Lmax);
}

int infllmv2_device_error(int clear) {
  unsigned int v = 0;
  if (cudaDeviceSynchronize() != cudaSuccess) return INFLLMV2_ERR_CUDA;
  if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof v) != cudaSuccess) return INFLLMV2_ERR_CUDA;
  if (clear) {
    unsigned int z = 0;
    if (cudaMemcpyToSymbol(g_device_error, &z, sizeof z) != cudaSuccess) return INFLLMV2_ERR_CUDA;
  }
  return static_cast<int>(v);
}

int infllmv2_compress_keys(const infllmv2_params* p, const void* k, const int32_t* lens, int32_t Lmax, void* kc,
                           infllmv2_stream_t stream) {
  int st = check_params(p);
  if (st != INFLLMV2_OK) return st;
  if ((st = check_len(Lmax)) != INFLLMV2_OK) return st;
  if (k == nullptr || !aligned16(k)) return INFLLMV2_ERR_INVALID_ARG;
  if (lens != nullptr && (reinterpret_cast<uintptr_t>(lens) & 3u)) return INFLLMV2_ERR_INVALID_ARG;
  const int nk = static_cast<int>(num_kernels(Lmax));
  if (nk == 0) return INFLLMV2_OK;  // kc has no rows (and may be NULL)
  if (kc == nullptr || !aligned16(kc)) return INFLLMV2_ERR_INVALID_ARG;
  const long long grid =
      static_cast<long long>(p->batch) * p->num_kv_heads * ((nk + kCompressKPC - 1) / kCompressKPC);
  if (grid > 0x7fffffffLL) return INFLLMV2_ERR_UNSUPPORTED;
  compress_kernel<<<static_cast<unsigned>(grid), kCompressThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      static_cast<const __nv_bfloat16*>(k), lens, Lmax, nk, p->num_kv_heads, static_cast<__nv_bfloat16*>(kc));
  return launch_status();
}

int infllmv2_append_kv(const infllmv2_params* p, const void* k_new, const void* v_new, void* k_cache,
                       void* v_cache, int32_t* lens, int32_t Lmax, void* kc, infllmv2_stream_t stream) {
  int st = check_params(p);
  if (st != INFLLMV2_OK) return st;
  if ((st = check_len(Lmax)) != INFLLMV2_OK) return st;
  if (!k_new || !v_new || !k_cache || !v_cache || !lens) return INFLLMV2_ERR_INVALID_ARG;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(lens) & 3u))
    return INFLLMV2_ERR_INVALID_ARG;
  const int64_t nk = num_kernels(Lmax);
  if (nk > 0 && (kc == nullptr || !aligned16(kc))) return INFLLMV2_ERR_INVALID_ARG;
  append_kv_kernel<<<static_cast<unsigned>(p->batch), kHeadDim, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      static_cast<const __nv_bfloat16*>(k_new), static_cast<const __nv_bfloat16*>(v_new),
      static_cast<__nv_bfloat16*>(k_cache), static_cast<__nv_bfloat16*>(v_cache), lens, Lmax,
      static_cast<int>(nk), p->num_kv_heads, static_cast<__nv_bfloat16*>(kc));
  return launch_status();
}

int infllmv2_select_blocks(const infllmv2_params* p, int mode, const void* q, const void* kc,
                           const int32_t* lens, int32_t L, int32_t* block_idx, void* ws, size_t ws_bytes,
                           infllmv2_stream_t stream) {
  int st = check_params(p);
  if (st != INFLLMV2_OK) return st;
  if ((st = check_len(L)) != INFLLMV2_OK) return st;
  if (mode == INFLLMV2_MODE_PREFILL) {
    if (lens != nullptr) return INFLLMV2_ERR_INVALID_ARG;
    return select_prefill(p, q, L, kc, nullptr, nullptr, L, block_idx, reinterpret_cast<cudaStream_t>(stream));
  }
  if (mode != INFLLMV2_MODE_DECODE) return INFLLMV2_ERR_INVALID_ARG;
  (void)ws;  // decode selection needs no workspace
  (void)ws_bytes;
  if (q == nullptr || block_idx == nullptr || !aligned16(q) || !aligned16(block_idx)) return INFLLMV2_ERR_INVALID_ARG;
  if (lens == nullptr || (reinterpret_cast<uintptr_t>(lens) & 3u)) return INFLLMV2_ERR_INVALID_ARG;
  const int64_t nk = num_kernels(L);
  if (nk > 0 && (kc == nullptr || !aligned16(kc))) return INFLLMV2_ERR_INVALID_ARG;
  if (static_cast<uint64_t>(p->batch) * p->num_kv_heads * static_cast<uint64_t>(nk) > 0x7fffffffULL)
    return INFLLMV2_ERR_UNSUPPORTED;  // TMA row coordinates are 32-bit
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int G = p->num_q_heads / p->num_kv_heads;
  CUtensorMap tm_kc;
  std::memset(&tm_kc, 0, sizeof tm_kc);
  // a map over a 1-row dummy extent is never dereferenced when there are no kernels
  if (nk > 0 && !make_map(&tm_kc, kc, static_cast<uint64_t>(p->batch) * p->num_kv_heads * nk, kKcTile))
    return INFLLMV2_ERR_CUDA;
  SelDecodeParams a;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.lens = lens;
  a.idx = block_idx;
  a.B = p->batch;
  a.Hq = p->num_q_heads;
  a.Hkv = p->num_kv_heads;
  a.G = G;
  a.Lmax = L;
  a.NKmax = static_cast<int>(nk);
  a.topk = p->topk;
  a.n_init = p->n_init;
  a.n_local = p->n_local;
  a.score_mode = p->score_mode;
  a.pool_mode = p->pool_mode;
  a.scale_log2 = scale_log2(p);
  if (nk == 0 && !make_map(&tm_kc, q, kKcTile, kKcTile)) return INFLLMV2_ERR_CUDA;  // never read: no tiles
  const int C = select_cluster(p, nk);
  const long long grid = static_cast<long long>(C) * p->batch * p->num_kv_heads;
  if (grid > 0x7fffffffLL) return INFLLMV2_ERR_UNSUPPORTED;
  const size_t smem = sel_decode_smem_bytes();
  return launch_cluster(select_decode_kernel, static_cast<unsigned>(grid), C, kSdThreads, smem, s, true, tm_kc,
                        a);
}

int infllmv2_select_blocks_chunk(const infllmv2_params* p, const void* q, int32_t Lq, const void* kc,
                                 const int32_t* q_lens, const int32_t* kv_lens, int32_t Lmax, int32_t* block_idx,
                                 void* ws, size_t ws_bytes, infllmv2_stream_t stream) {
  (void)ws;  // no workspace needed
  (void)ws_bytes;
  int st = check_params(p);
  if (st != INFLLMV2_OK) return st;
  if ((st = check_chunk(Lq, q_lens, kv_lens, Lmax)) != INFLLMV2_OK) return st;
  return select_prefill(p, q, Lq, kc, q_lens, kv_lens, Lmax, block_idx, reinterpret_cast<cudaStream_t>(stream));
}

int infllmv2_sparse_attn_prefill(const infllmv2_params* p, const void* q, const void* k, const void* v,
                                 const int32_t* block_idx, int32_t L, void* o, float* lse, void* ws,
                                 size_t ws_bytes, infllmv2_stream_t stream) {
  (void)ws;
  (void)ws_bytes;
  int st = check_params(p);
  if (st != INFLLMV2_OK) return st;
  if ((st = check_len(L)) != INFLLMV2_OK) return st;
  return attn_prefill(p, q, L, k, v, nullptr, nullptr, L, block_idx, o, lse, reinterpret_cast<cudaStream_t>(stream));
}

int infllmv2_sparse_attn_chunk(const infllmv2_params* p, const void* q, int32_t Lq, const void* k, const void* v,
                               const int32_t* q_lens, const int32_t* kv_lens, int32_t Lmax,
                               const int32_t* block_idx, void* o, float* lse, void* ws, size_t ws_bytes,
                               infllmv2_stream_t stream) {
  (void)ws;  // no workspace needed
  (void)ws_bytes;
  int st = check_params(p);
  if (st != INFLLMV2_OK) return st;
  if ((st = check_chunk(Lq, q_lens, kv_lens, Lmax)) != INFLLMV2_OK) return st;
  return attn_prefill(p, q, Lq, k, v, q_lens, kv_lens, Lmax, block_idx, o, lse,
                      reinterpret_cast<cudaStream_t>(stream));
}

int infllmv2_sparse_attn_backward(const infllmv2_params* p, const void* q, const void* k, const void* v,
                                  const void* o, const float* lse, const void* d_o, const int32_t* block_idx, int32_t L,
                                  void* dq, void* dk, void* dv, void* ws, size_t ws_bytes, infllmv2_stream_t stream) {
  int st = check_params(p);
  if (st != INFLLMV2_OK) return st;
  if ((st = check_len(L)) != INFLLMV2_OK) return st;
  if (!q || !k || !v || !o || !lse || !d_o || !block_idx || !dq || !dk || !dv) return INFLLMV2_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(d_o) || !aligned16(block_idx) ||
      !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return INFLLMV2_ERR_INVALID_ARG;
  const BwdLayout w = bwd_layout(p, L);
  if (ws == nullptr || ws_bytes < w.total || !aligned16(ws)) return INFLLMV2_ERR_WORKSPACE;
  const long long rows = static_cast<long long>(p->batch) * p->num_kv_heads * L;
  const uint64_t q_rows = static_cast<uint64_t>(p->batch) * L * p->num_q_heads;
  if (rows * p->topk > 0x7fffffffLL || q_rows > 0x7fffffffULL || w.n + 1 > 0x7fffffffLL)
    return INFLLMV2_ERR_UNSUPPORTED;  // 32-bit row lists and TMA rows
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  unsigned char* wb = static_cast<unsigned char*>(ws);
  BwdParams a;
  a.idx = block_idx;
  a.lse = lse;
  a.delta = reinterpret_cast<float*>(wb + w.delta);
  a.cnt = reinterpret_cast<int32_t*>(wb + w.cnt);
  a.off = reinterpret_cast<int32_t*>(wb + w.off);
  a.segoff = reinterpret_cast<int32_t*>(wb + w.segoff);
  a.list = reinterpret_cast<int32_t*>(wb + w.list);
  a.B = p->batch;
  a.Hq = p->num_q_heads;
  a.Hkv = p->num_kv_heads;
  a.G = p->num_q_heads / p->num_kv_heads;
  a.L = L;
  a.topk = p->topk;
  a.nblk = static_cast<int>(num_blocks(L));
  a.scale_log2 = scale_log2(p);
  a.scale = a.scale_log2 / 1.4426950408889634f;
  a.num_items = rows;
  a.dq = static_cast<__nv_bfloat16*>(dq);
  a.dk32 = reinterpret_cast<float*>(wb + w.dk);
  a.dv32 = reinterpret_cast<float*>(wb + w.dv);
  CUtensorMap tq, tdo, tk, tv;
  if (!make_map(&tq, q, q_rows, kGroupRows) || !make_map(&tdo, d_o, q_rows, kGroupRows) ||
      !make_map(&tk, k, static_cast<uint64_t>(rows), kBlock) || !make_map(&tv, v, static_cast<uint64_t>(rows), kBlock))
    return INFLLMV2_ERR_CUDA;
  // counters and the fp32 accumulators start at zero
  if (cudaMemsetAsync(wb + w.cnt, 0, w.off - w.cnt, s) != cudaSuccess ||
      cudaMemsetAsync(wb + w.dk, 0, w.total - w.dk, s) != cudaSuccess)
    return INFLLMV2_ERR_CUDA;
  const int n = static_cast<int>(w.n);
  bwd_delta_kernel<<<static_cast<unsigned>((q_rows + 7) / 8), 256, 0, s>>>(
      static_cast<const __nv_bfloat16*>(d_o), static_cast<const __nv_bfloat16*>(o), p->batch, L, p->num_q_heads,
      const_cast<float*>(a.delta));
  const unsigned rgrid = static_cast<unsigned>((rows + 255) / 256);
  bwd_count_kernel<<<rgrid, 256, 0, s>>>(block_idx, static_cast<int>(rows), L, p->topk, a.nblk,
                                         const_cast<int32_t*>(a.cnt));
  bwd_scan_kernel<<<1, 1024, 0, s>>>(a.cnt, n, const_cast<int32_t*>(a.off), const_cast<int32_t*>(a.segoff));
  bwd_fill_kernel<<<rgrid, 256, 0, s>>>(block_idx, static_cast<int>(rows), L, p->topk, a.nblk, a.off,
                                        reinterpret_cast<int32_t*>(wb + w.cursor), const_cast<int32_t*>(a.list));
  if ((st = launch_status()) != INFLLMV2_OK) return st;
  const size_t smem_q = bwd_dq_smem_bytes(), smem_kv = bwd_dkdv_tc_smem_bytes();
  if ((st = set_smem(reinterpret_cast<const void*>(bwd_dq_kernel), smem_q)) != INFLLMV2_OK) return st;
  if ((st = set_smem(reinterpret_cast<const void*>(bwd_dkdv_tc_kernel), smem_kv)) != INFLLMV2_OK) return st;
  bwd_dq_kernel<<<static_cast<unsigned>(std::min<long long>(rows, num_sms())), kBwdThreads, smem_q, s>>>(tq, tdo, tk,
                                                                                                        tv, a);
  bwd_dkdv_tc_kernel<<<static_cast<unsigned>(num_sms()), kBtThreads, smem_kv, s>>>(tq, tdo, tk, tv, a);
  const long long n4 = rows * kHeadDim / 4;
  bwd_cast_kernel<<<static_cast<unsigned>(std::min<long long>((n4 + 255) / 256, 8LL * num_sms())), 256, 0, s>>>(
      reinterpret_cast<const float4*>(a.dk32), reinterpret_cast<const float4*>(a.dv32), n4, static_cast<uint2*>(dk),
      static_cast<uint2*>(dv));
  return launch_status();
}

int infllmv2_sparse_attn_decode(const infllmv2_params* p, const void* q, const void* k_cache, const void* v_cache,
                                const int32_t* lens, int32_t Lmax, const int32_t* block_idx, void* o, float* lse,
                                void* ws, size_t ws_bytes, infllmv2_stream_t stream) {
  int st = check_params(p);
  if (st != INFLLMV2_OK) return st;
  if ((st = check_len(Lmax)) != INFLLMV2_OK) return st;
  if (!q || !k_cache || !v_cache || !lens || !block_idx || !o) return INFLLMV2_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(block_idx) || !aligned16(o) ||
      (reinterpret_cast<uintptr_t>(lens) & 3u))
    return INFLLMV2_ERR_INVALID_ARG;
  if (lse != nullptr && (reinterpret_cast<uintptr_t>(lse) & 3u)) return INFLLMV2_ERR_INVALID_ARG;
  const size_t need = ws_size(p, INFLLMV2_OP_ATTN_DECODE, Lmax);
  if (need > 0 && (ws == nullptr || ws_bytes < need || !aligned16(ws))) return INFLLMV2_ERR_WORKSPACE;
  const uint64_t kv_rows = static_cast<uint64_t>(p->batch) * p->num_kv_heads * Lmax;
  if (kv_rows > 0x7fffffffULL) return INFLLMV2_ERR_UNSUPPORTED;  // TMA row coordinates are 32-bit
  const DecodePlan d = decode_plan(p);
  AttnParams a;
  a.idx = block_idx;
  a.lens = lens;
  a.q_lens = nullptr;
  a.kv_lens = nullptr;
  a.B = p->batch;
  a.Hq = p->num_q_heads;
  a.Hkv = p->num_kv_heads;
  a.G = p->num_q_heads / p->num_kv_heads;
  a.Lq = 1;
  a.Lmax = Lmax;
  a.topk = p->topk;
  a.n_splits = d.n_splits;
  a.blocks_per_split = d.per_split;
  a.scale_log2 = scale_log2(p);
  a.num_items = static_cast<long long>(p->batch) * p->num_kv_heads * d.n_splits;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.part_o = nullptr;
  a.part_lse = nullptr;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const uint64_t q_rows = static_cast<uint64_t>(p->batch) * p->num_q_heads;
  if (d.cluster > 0) {
    CUtensorMap tq, tk, tv;
    if (!make_map(&tq, q, q_rows, kGroupRows) || !make_map(&tk, k_cache, kv_rows, kBlock) ||
        !make_map(&tv, v_cache, kv_rows, kBlock))
      return INFLLMV2_ERR_CUDA;
    const long long grid = static_cast<long long>(d.cluster) * p->batch * p->num_kv_heads;
    if (grid > 0x7fffffffLL) return INFLLMV2_ERR_UNSUPPORTED;
    return launch_cluster(attn_decode_cluster_kernel, static_cast<unsigned>(grid), d.cluster, kAdThreads,
                          attn_dec_smem_bytes(), s, true, tq, tk, tv, a);
  }
  const size_t rows = static_cast<size_t>(p->batch) * p->num_kv_heads * d.n_splits * kGroupRows;
  a.part_o = static_cast<float*>(ws);
  a.part_lse = a.part_o + rows * kHeadDim;
  st = launch_attn(p, q, q_rows, k_cache, v_cache, kv_rows, a, s);
  if (st != INFLLMV2_OK) return st;
  attn_merge_kernel<<<static_cast<unsigned>(static_cast<long long>(p->batch) * p->num_kv_heads * a.G), 128, 0, s>>>(
      a.part_o, a.part_lse, d.n_splits, p->num_q_heads, p->num_kv_heads, a.G, static_cast<__nv_bfloat16*>(o), lse);
  return launch_status();
}

int infllmv2_decode_step(const infllmv2_params* p, const void* q, const void* k_new, const void* v_new, void* k_cache,
                         void* v_cache, void* kc, const int32_t* lens, int32_t* lens_out, int32_t Lmax,
                         int32_t* block_idx, void* o, float* lse, infllmv2_stream_t stream) {
  int st = check_params(p);
  if (st != INFLLMV2_OK) return st;
  if ((st = check_len(Lmax)) != INFLLMV2_OK) return st;
  if (!q || !k_cache || !v_cache || !lens || !block_idx || !o) return INFLLMV2_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(block_idx) || !aligned16(o) ||
      (reinterpret_cast<uintptr_t>(lens) & 3u))
    return INFLLMV2_ERR_INVALID_ARG;
  if ((k_new == nullptr) != (v_new == nullptr)) return INFLLMV2_ERR_INVALID_ARG;
  if (k_new != nullptr) {  // append: the new rows, and a separate array for the new lengths
    if (!aligned16(k_new) || !aligned16(v_new) || lens_out == nullptr || lens_out == lens ||
        (reinterpret_cast<uintptr_t>(lens_out) & 3u) || kc == nullptr)
      return INFLLMV2_ERR_INVALID_ARG;
  }
  if (lse != nullptr && (reinterpret_cast<uintptr_t>(lse) & 3u)) return INFLLMV2_ERR_INVALID_ARG;
  const int64_t nk = num_kernels(Lmax);
  if (nk > 0 && (kc == nullptr || !aligned16(kc))) return INFLLMV2_ERR_INVALID_ARG;
  const uint64_t kv_rows = static_cast<uint64_t>(p->batch) * p->num_kv_heads * Lmax;
  if (kv_rows > 0x7fffffffULL ||
      static_cast<uint64_t>(p->batch) * p->num_kv_heads * static_cast<uint64_t>(nk) > 0x7fffffffULL)
    return INFLLMV2_ERR_UNSUPPORTED;  // TMA row coordinates are 32-bit
  const int G = p->num_q_heads / p->num_kv_heads;
  DecodeStepParams P;
  SelDecodeParams& a = P.sel;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.lens = lens;
  a.idx = block_idx;
  a.B = p->batch;
  a.Hq = p->num_q_heads;
  a.Hkv = p->num_kv_heads;
  a.G = G;
  a.Lmax = Lmax;
  a.NKmax = static_cast<int>(nk);
  a.topk = p->topk;
  a.n_init = p->n_init;
  a.n_local = p->n_local;
  a.score_mode = p->score_mode;
  a.pool_mode = p->pool_mode;
  a.scale_log2 = scale_log2(p);
  AttnParams& t = P.attn;
  t.idx = block_idx;
  t.lens = lens;
  t.q_lens = nullptr;
  t.kv_lens = nullptr;
  t.B = p->batch;
  t.Hq = p->num_q_heads;
  t.Hkv = p->num_kv_heads;
  t.G = G;
  t.Lq = 1;
  t.Lmax = Lmax;
  t.topk = p->topk;
  t.n_splits = 1;
  t.blocks_per_split = p->topk;
  t.scale_log2 = a.scale_log2;
  t.num_items = static_cast<long long>(p->batch) * p->num_kv_heads;
  t.o = static_cast<__nv_bfloat16*>(o);
  t.lse = lse;
  t.part_o = nullptr;
  t.part_lse = nullptr;
  P.k_new = static_cast<const __nv_bfloat16*>(k_new);
  P.v_new = static_cast<const __nv_bfloat16*>(v_new);
  P.k_cache = static_cast<__nv_bfloat16*>(k_cache);
  P.v_cache = static_cast<__nv_bfloat16*>(v_cache);
  P.kc = static_cast<__nv_bfloat16*>(kc);
  P.lens_out = lens_out;
  CUtensorMap tm_kc, tq, tk, tv;
  std::memset(&tm_kc, 0, sizeof tm_kc);
  const uint64_t q_rows = static_cast<uint64_t>(p->batch) * p->num_q_heads;
  // with no complete kernel a map over a dummy extent is never dereferenced
  if (!(nk > 0 ? make_map(&tm_kc, kc, static_cast<uint64_t>(p->batch) * p->num_kv_heads * nk, kKcTile)
               : make_map(&tm_kc, q, kKcTile, kKcTile)) ||
      !make_map(&tq, q, q_rows, kGroupRows) || !make_map(&tk, k_cache, kv_rows, kBlock) ||
      !make_map(&tv, v_cache, kv_rows, kBlock))
    return INFLLMV2_ERR_CUDA;
  const int C = decode_step_cluster(p, nk);
  const long long grid = static_cast<long long>(C) * p->batch * p->num_kv_heads;
  if (grid > 0x7fffffffLL) return INFLLMV2_ERR_UNSUPPORTED;
  return launch_cluster(decode_step_kernel, static_cast<unsigned>(grid), C, kSdThreads, decode_step_smem_bytes(),
                        reinterpret_cast<cudaStream_t>(stream), true, tm_kc, tq, tk, tv, P);
}

int infllmv2_rope_table(const infllmv2_params* p, const float* inv_freq, int32_t rot, int32_t n, float scale,
                        float* table, infllmv2_stream_t stream) {
  int st = check_params(p);
  if (st != INFLLMV2_OK) return st;
  if ((st = check_len(n)) != INFLLMV2_OK) return st;
  if (!inv_freq || !table || !aligned4(inv_freq) || !aligned16(table)) return INFLLMV2_ERR_INVALID_ARG;
  if (rot < 16 || rot > kHeadDim || rot % 16 != 0 || !std::isfinite(scale)) return INFLLMV2_ERR_INVALID_ARG;
  const long long ctas = (static_cast<long long>(n) * (rot / 2) + 255) / 256;
  rope_table_kernel<<<static_cast<unsigned>(std::min<long long>(ctas, 8LL * num_sms())), 256, 0,
                      reinterpret_cast<cudaStream_t>(stream)>>>(inv_freq, rot, n, scale, table);
  return launch_status();
}

int infllmv2_qk_norm_rope(const infllmv2_params* p, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                          const void* v, int64_t v_stride, int32_t Lq, const void* q_weight, const void* k_weight,
                          int32_t weights_fp32, float eps, const float* table, int32_t table_rows, int32_t rot,
                          int32_t interleaved, const int32_t* starts, const int32_t* q_lens, void* q_out, void* k_out,
                          void* v_out, int32_t Lout, int32_t at_position, int32_t* lens_out,
                          infllmv2_stream_t stream) {
  NormRopeParams a;
  int st = norm_rope_args(p, q, q_stride, k, k_stride, Lq, q_weight, k_weight, weights_fp32, eps, table, table_rows,
                          rot, interleaved, starts, q_lens, a);
  if (st != INFLLMV2_OK) return st;
  if ((st = check_len(Lout)) != INFLLMV2_OK) return st;
  if (!v || !q_out || !k_out || !v_out || !aligned16(v) || !aligned16(q_out) || !aligned16(k_out) ||
      !aligned16(v_out) || !aligned4(lens_out) || (lens_out != nullptr && (lens_out == starts || lens_out == q_lens)))
    return INFLLMV2_ERR_INVALID_ARG;
  if (v_stride < static_cast<int64_t>(p->num_kv_heads) * kHeadDim || v_stride % 8 != 0) return INFLLMV2_ERR_INVALID_ARG;
  if ((at_position != 0 && at_position != 1) || (at_position == 0 && Lout < Lq)) return INFLLMV2_ERR_INVALID_ARG;
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.v_stride = v_stride;
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  a.v_out = static_cast<__nv_bfloat16*>(v_out);
  a.Lout = Lout;
  a.at_position = at_position;
  a.lens_out = lens_out;
  const unsigned grid = norm_rope_grid(p, Lq, &a);
  if (grid == 0) return INFLLMV2_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return interleaved ? launch_pdl(qk_norm_rope_kernel<true>, grid, kNrThreads, 0, s, a)
                     : launch_pdl(qk_norm_rope_kernel<false>, grid, kNrThreads, 0, s, a);
}

int infllmv2_qk_norm_rope_backward(const infllmv2_params* p, const void* q, int64_t q_stride, const void* k,
                                   int64_t k_stride, const void* d_q, const void* d_k, const void* d_v, int32_t Lq,
                                   const void* q_weight, const void* k_weight, int32_t weights_fp32, float eps,
                                   const float* table, int32_t table_rows, int32_t rot, int32_t interleaved,
                                   const int32_t* starts, const int32_t* q_lens, void* dq_in, int64_t dq_stride,
                                   void* dk_in, int64_t dk_stride, void* dv_in, int64_t dv_stride, float* d_qw,
                                   float* d_kw, void* ws, size_t ws_bytes, infllmv2_stream_t stream) {
  NormRopeParams a;
  int st = norm_rope_args(p, q, q_stride, k, k_stride, Lq, q_weight, k_weight, weights_fp32, eps, table, table_rows,
                          rot, interleaved, starts, q_lens, a);
  if (st != INFLLMV2_OK) return st;
  if (!d_q || !d_k || !d_v || !dq_in || !dk_in || !dv_in || !aligned16(d_q) || !aligned16(d_k) || !aligned16(d_v) ||
      !aligned16(dq_in) || !aligned16(dk_in) || !aligned16(dv_in) || !aligned4(d_qw) || !aligned4(d_kw))
    return INFLLMV2_ERR_INVALID_ARG;
  const int64_t kn = static_cast<int64_t>(p->num_kv_heads) * kHeadDim;
  if (dq_stride < static_cast<int64_t>(p->num_q_heads) * kHeadDim || dk_stride < kn || dv_stride < kn ||
      dq_stride % 8 != 0 || dk_stride % 8 != 0 || dv_stride % 8 != 0)
    return INFLLMV2_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned16(ws) || ws_bytes < ws_size(p, INFLLMV2_OP_QK_NORM_ROPE_BACKWARD, Lq))
    return INFLLMV2_ERR_WORKSPACE;
  a.dq = static_cast<const __nv_bfloat16*>(d_q);
  a.dk = static_cast<const __nv_bfloat16*>(d_k);
  a.dv = static_cast<const __nv_bfloat16*>(d_v);
  a.q_out = static_cast<__nv_bfloat16*>(dq_in);
  a.k_out = static_cast<__nv_bfloat16*>(dk_in);
  a.v_out = static_cast<__nv_bfloat16*>(dv_in);
  a.dq_stride = dq_stride;
  a.dk_stride = dk_stride;
  a.dv_stride = dv_stride;
  a.part = static_cast<float*>(ws);
  const unsigned grid = norm_rope_bwd_grid(p, Lq, &a);
  if (grid == 0) return INFLLMV2_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto kernel = interleaved ? qk_norm_rope_bwd_kernel<true> : qk_norm_rope_bwd_kernel<false>;
  if ((st = set_smem(reinterpret_cast<const void*>(kernel), kNrBwdSmem)) != INFLLMV2_OK) return st;
  kernel<<<grid, kNrThreads, kNrBwdSmem, s>>>(a);
  if ((st = launch_status()) != INFLLMV2_OK || (!d_qw && !d_kw)) return st;
  return launch_pdl(qk_norm_rope_bwd_weights_kernel, dim3(8), 1024, 0, s, a.part, a.q_chunks * a.q_ctas,
                    a.kv_chunks * a.kv_ctas, d_qw, d_kw);
}

int infllmv2_window_attn(const infllmv2_params* p, const void* q, int32_t Lq, const void* k, const void* v,
                         const int32_t* q_lens, const int32_t* kv_lens, int32_t Lmax, int32_t window, int32_t n_sink,
                         void* o, float* lse, void* ws, size_t ws_bytes, infllmv2_stream_t stream) {
  WinParams a;
  int st = window_args(p, q, Lq, k, v, q_lens, kv_lens, Lmax, window, n_sink, a);
  if (st != INFLLMV2_OK) return st;
  if (!o || !aligned16(o) || !aligned4(lse)) return INFLLMV2_ERR_INVALID_ARG;
  const size_t need = ws_size(p, INFLLMV2_OP_WINDOW_ATTN, Lq);
  if (need > 0 && (ws == nullptr || ws_bytes < need || !aligned16(ws))) return INFLLMV2_ERR_WORKSPACE;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  return launch_window(p, a, ws, reinterpret_cast<cudaStream_t>(stream));
}

int infllmv2_window_attn_decode(const infllmv2_params* p, const void* q, const void* k_cache, const void* v_cache,
                                const int32_t* lens, int32_t Lmax, int32_t window, int32_t n_sink, void* o, float* lse,
                                void* ws, size_t ws_bytes, infllmv2_stream_t stream) {
  WinParams a;
  int st = window_args(p, q, 1, k_cache, v_cache, nullptr, lens, Lmax, window, n_sink, a);
  if (st != INFLLMV2_OK) return st;
  if (!lens || !o || !aligned16(o) || !aligned4(lse)) return INFLLMV2_ERR_INVALID_ARG;
  const size_t need = ws_size(p, INFLLMV2_OP_WINDOW_DECODE, Lmax);
  if (need > 0 && (ws == nullptr || ws_bytes < need || !aligned16(ws))) return INFLLMV2_ERR_WORKSPACE;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  return launch_window_decode(p, a, ws, reinterpret_cast<cudaStream_t>(stream));
}

int infllmv2_window_attn_backward(const infllmv2_params* p, const void* q, const void* k, const void* v, const void* o,
                                  const float* lse, const void* d_o, const int32_t* lens, int32_t L, int32_t window,
                                  int32_t n_sink, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                                  infllmv2_stream_t stream) {
  WinParams a;
  int st = window_args(p, q, L, k, v, lens, lens, L, window, n_sink, a);
  if (st != INFLLMV2_OK) return st;
  if (!o || !lse || !d_o || !dq || !dk || !dv || !aligned16(o) || !aligned16(d_o) || !aligned16(dq) ||
      !aligned16(dk) || !aligned16(dv) || !aligned4(lse))
    return INFLLMV2_ERR_INVALID_ARG;
  const size_t need = ws_size(p, INFLLMV2_OP_WINDOW_BACKWARD, L);
  if (need > 0 && (ws == nullptr || ws_bytes < need || !aligned16(ws))) return INFLLMV2_ERR_WORKSPACE;
  // dq and dk / dv are written while other CTAs still read these
  const size_t row = static_cast<size_t>(p->batch) * L * kHeadDim * sizeof(__nv_bfloat16);
  const size_t qn = row * p->num_q_heads, kn = row * p->num_kv_heads;
  for (const void* x : {q, d_o})
    if (overlap(dq, qn, x, qn) || overlap(dk, kn, x, qn) || overlap(dv, kn, x, qn)) return INFLLMV2_ERR_INVALID_ARG;
  for (const void* x : {k, v})
    if (overlap(dq, qn, x, kn) || overlap(dk, kn, x, kn) || overlap(dv, kn, x, kn)) return INFLLMV2_ERR_INVALID_ARG;
  if (overlap(dq, qn, dk, kn) || overlap(dq, qn, dv, kn) || overlap(dk, kn, dv, kn)) return INFLLMV2_ERR_INVALID_ARG;
  a.o_in = static_cast<const __nv_bfloat16*>(o);
  a.lse = const_cast<float*>(lse);
  a.d_o = static_cast<const __nv_bfloat16*>(d_o);
  a.dq = static_cast<__nv_bfloat16*>(dq);
  a.dk = static_cast<__nv_bfloat16*>(dk);
  a.dv = static_cast<__nv_bfloat16*>(dv);
  return launch_window_backward(p, a, ws, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"

// ------------------------------------------------ decode attention without allocation
// The split partials of infllmv2_sparse_attn_decode_noalloc live in this file-scope
// device array instead of a caller workspace.  Host code only ever sees the symbol's
// host-side stand-in, so the device address is looked up once per device.
static __device__ __align__(256) unsigned char g_noalloc_scratch[INFLLMV2_NOALLOC_SCRATCH_BYTES];

namespace {
constexpr int kMaxDevices = 64;
std::mutex g_noalloc_mu;
void* g_noalloc_ptr[kMaxDevices] = {};

int noalloc_scratch(void** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return INFLLMV2_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return INFLLMV2_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_noalloc_mu);
  if (g_noalloc_ptr[dev] == nullptr) {
    void* ptr = nullptr;
    if (cudaGetSymbolAddress(&ptr, g_noalloc_scratch) != cudaSuccess || ptr == nullptr) return INFLLMV2_ERR_CUDA;
    g_noalloc_ptr[dev] = ptr;
  }
  *out = g_noalloc_ptr[dev];
  return INFLLMV2_OK;
}
}  // namespace

extern "C" int infllmv2_sparse_attn_decode_noalloc(const infllmv2_params* p, const void* q, const void* k_cache,
                                                   const void* v_cache, const int32_t* lens, int32_t Lmax,
                                                   const int32_t* block_idx, void* o, float* lse,
                                                   infllmv2_stream_t stream) {
  const int st = check_params(p);
  if (st != INFLLMV2_OK) return st;
  const size_t need = ws_size(p, INFLLMV2_OP_ATTN_DECODE, Lmax);
  if (need == static_cast<size_t>(-1)) return INFLLMV2_ERR_INVALID_ARG;
  if (need > INFLLMV2_NOALLOC_SCRATCH_BYTES) return INFLLMV2_ERR_WORKSPACE;
  void* scratch = nullptr;
  const int sst = noalloc_scratch(&scratch);
  if (sst != INFLLMV2_OK) return sst;
  return infllmv2_sparse_attn_decode(p, q, k_cache, v_cache, lens, Lmax, block_idx, o, lse, scratch,
                                     INFLLMV2_NOALLOC_SCRATCH_BYTES, stream);
}
