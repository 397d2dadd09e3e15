// window_decode.cuh -- sliding-window attention of one decode token per sequence
// (csrc/window.cuh states it).
//
// Bound by HBM: 512 bytes of K and V per visible key and kv-head, read once for the group's G
// <= 16 heads.  The visible keys are the sinks and the window, two runs cut into segments of 64
// keys that start at the run's first key; a CTA takes `per_chunk` consecutive segments of one
// (sequence, kv-head).  Warp 4 streams them with TMA into a ring of 32 KB stages (three, so two
// CTAs share an SM and keep 192 KB in flight); warps 0-3 take 16 keys of each segment: 16 heads
// x 16 keys of scores with m16n8k16 MMAs (a tcgen05 tile would need 64 rows), an online softmax
// with its own reference per warp, and P V, with no synchronisation between the warps until the
// chunk ends.  A (sequence, kv-head) that is one chunk writes its output directly; up to 16 chunks
// are a thread-block cluster and joined through distributed shared memory (one launch, no round
// trip through HBM); more are joined by window_decode_merge_kernel through the workspace.
// Measured: 32 ragged 128K sequences, 32 / 2 heads, every key: 465 us a call, 6.9 TB/s (452 repeated);
// 8 sequences, W 4096, on the GPU: 12.3 us in one cluster launch, 13.1 us with the join through the
// workspace (cold L2: 20.5, 21.5); 15.7 us a call.
#pragma once
#include <cooperative_groups.h>

#include "common.cuh"
#include "tcgen05.cuh"
#include "window_tc.cuh"

namespace infllmv2 {

constexpr int kWdWarps = 4;
constexpr int kWdThreads = 32 * (kWdWarps + 1);
constexpr int kWdStages = 3;
constexpr int kWdHalf = kWfSeg * 128;          // 8 KB: 64 columns of 64 rows
constexpr int kWdStageBytes = 4 * kWdHalf;     // K halves, then V halves

struct WdSmem {
  uint64_t full[kWdStages], empty[kWdStages];
  float m[kWdWarps][kGroupRows], l[kWdWarps][kGroupRows];
  float lse[kGroupRows];  // cluster: this CTA's base-2 log-sum-exps
  volatile int abort;
};
constexpr size_t window_decode_smem_bytes() {
  return 1024 + static_cast<size_t>(kWdStages) * kWdStageBytes + sizeof(WdSmem);
}
constexpr int kWdPartFloats = kWdWarps * kGroupRows * kHeadDim;  // the warps' partial outputs, then the CTA's
static_assert(kWdStages * kWdStageBytes >= (kWdPartFloats + kGroupRows * kHeadDim) * 4, "partial outputs in the ring");
constexpr int kWdMaxCluster = 16;

struct WinDecodeParams {
  WinParams w;
  int g_log2, per_chunk, chunks;  // segments of a chunk; chunks per (sequence, kv-head)
  float* part_o;                  // [B * Hkv, chunks, G, 128] normalised
  float* part_lse;                // [B * Hkv, chunks, G] base 2
};

// grid = B * Hkv * chunks.  A CTA past its sequence's keys ends at once, or (kCluster: the chunks of
// a (sequence, kv-head) are one cluster) only takes part in the join.
template <bool kCluster>
__global__ void __launch_bounds__(kWdThreads, 2)
    window_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ CUtensorMap tm_ks, const __grid_constant__ CUtensorMap tm_vs,
                         const WinDecodeParams p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* ring = align_smem(smem_raw, 1024);
  WdSmem& S = *reinterpret_cast<WdSmem*>(ring + kWdStages * kWdStageBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WinParams& w = p.w;
  const int chunk = blockIdx.x % p.chunks, bg = blockIdx.x / p.chunks;
  const int b = bg / w.Hkv, g = bg - b * w.Hkv;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kWdStages; ++s) {
      mbar_init(&S.full[s], 1);
      mbar_init(&S.empty[s], kWdWarps);
    }
    S.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  allow_dependent_launch();
  grid_dependency_wait();
  const int len = min(w.kv_lens[b], w.Lmax);
  if (len <= 0) {  // no query: zeros and -inf
    if (chunk == 0)
      for (int i = threadIdx.x; i < w.G * kHeadDim; i += kWdThreads) {
        const size_t row = static_cast<size_t>(b) * w.Hq + (g << p.g_log2) + i / kHeadDim;
        w.o[row * kHeadDim + i % kHeadDim] = __float2bfloat16(0.f);
        if (w.lse && i % kHeadDim == 0) w.lse[row] = -INFINITY;
      }
    return;
  }
  const int t = len - 1;
  const WinRuns runs(t, t, w.window, w.n_sink);
  const int segs = runs.ns + runs.nw;
  const int s0 = chunk * p.per_chunk, s1 = min(segs, s0 + p.per_chunk);
  if (!kCluster && s0 >= s1) return;
  const int n = max(s1 - s0, 0);

  if (warp == kWdWarps) {
    if (lane == 0) {
      int i = 0;
      for (; i < n; ++i) {
        const int st = i % kWdStages, seg = s0 + i;
        if (i >= kWdStages) mbar_wait_short(&S.empty[st], static_cast<uint32_t>(i / kWdStages - 1) & 1u, &S.abort);
        if (S.abort) break;
        unsigned char* dst = ring + st * kWdStageBytes;
        const bool sink = runs.is_sink(seg);
        const int key = runs.first_key(seg);
        mbar_arrive_expect_tx(&S.full[st], kWdStageBytes);
        for (int h = 0; h < 2; ++h) {
          tma_load_3d(dst + h * kWdHalf, sink ? &tm_ks : &tm_k, &S.full[st], 64 * h, key, bg);
          tma_load_3d(dst + (2 + h) * kWdHalf, sink ? &tm_vs : &tm_v, &S.full[st], 64 * h, key, bg);
        }
      }
      drain_ring(S.full, i);  // every copy lands before the ring is used for the joins and the CTA ends
    }
    __syncwarp();
  }

  // consumers: A fragments of the 16 query rows (rows past the group are zero)
  uint32_t qa[8][4];
  float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  const int r = lane >> 2, c2 = (lane & 3) * 2;
  if (warp < kWdWarps) {
    const __nv_bfloat16* q = w.q + (static_cast<size_t>(b) * w.Hq + (g << p.g_log2)) * kHeadDim;
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = r + 8 * (i & 1), col = 16 * k + 8 * (i >> 1) + c2;
        qa[k][i] = row < w.G ? *reinterpret_cast<const uint32_t*>(q + row * kHeadDim + col) : 0u;
      }
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
    const int key_w = 16 * warp;  // this warp's keys of a segment
    for (int i = 0; i < n; ++i) {
      const int st = i % kWdStages, seg = s0 + i;
      mbar_wait_short(&S.full[st], static_cast<uint32_t>(i / kWdStages) & 1u, &S.abort);
      unsigned char* kt = ring + st * kWdStageBytes;
      unsigned char* vt = kt + 2 * kWdHalf;
      // keys of this warp that the query sees: a prefix of the segment's, in either run
      const int limit = (runs.is_sink(seg) ? w.n_sink : len) - runs.first_key(seg) - key_w;
      const bool dead = limit <= 0;
      if (!dead) {
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        const int krow = key_w + (lane & 7) + ((lane >> 4) << 3), kch = (lane >> 3) & 1;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t b0, b1, b2, b3;
          ldsm_x4(smem_u32(kt + (k >> 2) * kWdHalf + sw128(krow, 2 * (k & 3) + kch)), b0, b1, b2, b3);
          mma_bf16(s[0], qa[k], b0, b1);
          mma_bf16(s[1], qa[k], b2, b3);
        }
        if (limit < 16) {
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (8 * nt + c2 + (c & 1) >= limit) s[nt][c] = -INFINITY;
          // rows of V past the last key may hold anything (0 x NaN is not 0)
          for (int e = lane; e < (16 - limit) * 16; e += 32)
            *reinterpret_cast<uint4*>(vt + (e & 8 ? kWdHalf : 0) + (key_w + limit + (e >> 4)) * 128 + (e & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
        }
        float mx[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mx[h] = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2)) * w.scale_log2;
        }
        // the reference moves only when a row's maximum rose by more than 2^8
        if (__any_sync(0xffffffffu, mx[0] > m[0] + 8.f || mx[1] > m[1] + 8.f)) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float mn = fmaxf(m[h], mx[h]), f = ex2(m[h] - mn);
            m[h] = mn;
            l[h] *= f;
#pragma unroll
            for (int d = 0; d < 16; ++d) o[d][2 * h] *= f, o[d][2 * h + 1] *= f;
          }
        }
        float e[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            e[nt][c] = ex2(fmaf(s[nt][c], w.scale_log2, -m[c >> 1]));
            l[c >> 1] += e[nt][c];
          }
        const uint32_t pa[4] = {pack_bf16(e[0][0], e[0][1]), pack_bf16(e[0][2], e[0][3]), pack_bf16(e[1][0], e[1][1]),
                                pack_bf16(e[1][2], e[1][3])};
        const int vrow = key_w + (lane & 15), vch = lane >> 4;
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          uint32_t b0, b1, b2, b3;
          ldsm_x4_t(smem_u32(vt + (d >> 2) * kWdHalf + sw128(vrow, 2 * (d & 3) + vch)), b0, b1, b2, b3);
          mma_bf16(o[2 * d], pa, b0, b1);
          mma_bf16(o[2 * d + 1], pa, b2, b3);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.empty[st]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if ((lane & 3) == 0) {
        S.m[warp][r + 8 * h] = m[h];
        S.l[warp][r + 8 * h] = l[h];
      }
    }
  }
  __syncthreads();  // the ring is free: every stage has been read
  float* part = reinterpret_cast<float*>(ring);  // [warp][row][128]
  if (warp < kWdWarps)
#pragma unroll
    for (int d = 0; d < 16; ++d)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (r + 8 * h < w.G)
          *reinterpret_cast<float2*>(part + (warp * kGroupRows + r + 8 * h) * kHeadDim + 8 * d + c2) =
              make_float2(o[d][2 * h], o[d][2 * h + 1]);
  __syncthreads();
  // join the warps: a thread takes 4 columns of rows threadIdx / 32, + 4, ...
  float* joint = part + kWdPartFloats;  // cluster: [row][128]
  if (warp < kWdWarps)
    for (int row = warp; row < w.G; row += kWdWarps) {
      if (kCluster && n == 0) {
        if (lane == 0) S.lse[row] = -INFINITY;
        continue;
      }
      float mm = -INFINITY;
#pragma unroll
      for (int v = 0; v < kWdWarps; ++v) mm = fmaxf(mm, S.m[v][row]);
      float acc[4] = {0.f, 0.f, 0.f, 0.f}, z = 0.f;
#pragma unroll
      for (int v = 0; v < kWdWarps; ++v) {
        const float f = ex2(S.m[v][row] - mm);  // 0 for a warp that saw no key
        z = fmaf(f, S.l[v][row], z);
        const float4 x = *(reinterpret_cast<const float4*>(part + (v * kGroupRows + row) * kHeadDim) + lane);
        acc[0] = fmaf(f, x.x, acc[0]), acc[1] = fmaf(f, x.y, acc[1]);
        acc[2] = fmaf(f, x.z, acc[2]), acc[3] = fmaf(f, x.w, acc[3]);
      }
      const float inv = 1.f / z, lse2 = mm + lg2(z);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] *= inv;
      const size_t head = static_cast<size_t>(b) * w.Hq + (g << p.g_log2) + row;
      if (kCluster) {
        *(reinterpret_cast<float4*>(joint + row * kHeadDim) + lane) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        if (lane == 0) S.lse[row] = lse2;
      } else if (p.chunks == 1) {
        store4(w.o + head * kHeadDim, lane, acc);
        if (w.lse && lane == 0) w.lse[head] = lse2 * 0.6931471805599453f;
      } else {
        const size_t pr = static_cast<size_t>(blockIdx.x) * w.G + row;
        *(reinterpret_cast<float4*>(p.part_o + pr * kHeadDim) + lane) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        if (lane == 0) p.part_lse[pr] = lse2;
      }
    }
  if (kCluster) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();  // every CTA's rows are final
    if (warp < kWdWarps)
      for (int row = chunk * kWdWarps + warp; row < w.G; row += p.chunks * kWdWarps) {
        // lane = chunk (at most 16): every weight is known before the first row is read
        const float l = lane < p.chunks ? cluster.map_shared_rank(S.lse, lane)[row] : -INFINITY;
        float mx = l;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float e = ex2(l - mx);  // 0 for a chunk without keys: its row is not read
        float z = e;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int c = 0; c < p.chunks; ++c) {
          const float ec = __shfl_sync(0xffffffffu, e, c);
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          if (ec > 0.f) x = *(reinterpret_cast<const float4*>(cluster.map_shared_rank(joint, c) + row * kHeadDim) + lane);
          acc[0] = fmaf(ec, x.x, acc[0]), acc[1] = fmaf(ec, x.y, acc[1]);
          acc[2] = fmaf(ec, x.z, acc[2]), acc[3] = fmaf(ec, x.w, acc[3]);
        }
        const float inv = 1.f / z;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] *= inv;
        const size_t head = static_cast<size_t>(b) * w.Hq + (g << p.g_log2) + row;
        store4(w.o + head * kHeadDim, lane, acc);
        if (w.lse && lane == 0) w.lse[head] = (mx + lg2(z)) * 0.6931471805599453f;
      }
    cluster.sync();  // the others' shared memory stays until every row has been read
  }
}

// Joins the chunks: a CTA per (sequence, q-head), its four warps taking every fourth chunk.
__global__ void __launch_bounds__(128) window_decode_merge_kernel(const WinDecodeParams p) {
  __shared__ float red[4][kHeadDim], zs[4];
  const WinParams& w = p.w;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / w.Hq, h = blockIdx.x - b * w.Hq;
  grid_dependency_wait();
  const int len = min(w.kv_lens[b], w.Lmax);
  if (len <= 0) return;  // written by the first kernel
  const WinRuns runs(len - 1, len - 1, w.window, w.n_sink);
  const int live = (runs.ns + runs.nw + p.per_chunk - 1) / p.per_chunk;
  const size_t row0 = static_cast<size_t>(b * w.Hkv + (h >> p.g_log2)) * p.chunks * w.G + (h & (w.G - 1));
  // this warp's first rows are on their way while the maximum is found
  float4 x[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (warp + 4 * u < live)
      x[u] = *(reinterpret_cast<const float4*>(p.part_o + (row0 + static_cast<size_t>(warp + 4 * u) * w.G) * kHeadDim) + lane);
  }
  float mx = -INFINITY;
  for (int c = lane; c < live; c += 32) mx = fmaxf(mx, p.part_lse[row0 + static_cast<size_t>(c) * w.G]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
  float acc[4] = {0.f, 0.f, 0.f, 0.f}, z = 0.f;
  for (int c0 = warp; c0 < live; c0 += 16) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = c0 + 4 * u;
      if (c < live) {
        const float e = ex2(p.part_lse[row0 + static_cast<size_t>(c) * w.G] - mx);
        z += e;
        acc[0] = fmaf(e, x[u].x, acc[0]), acc[1] = fmaf(e, x[u].y, acc[1]);
        acc[2] = fmaf(e, x[u].z, acc[2]), acc[3] = fmaf(e, x[u].w, acc[3]);
      }
      if (c + 16 < live)
        x[u] = *(reinterpret_cast<const float4*>(p.part_o + (row0 + static_cast<size_t>(c + 16) * w.G) * kHeadDim) + lane);
    }
  }
  *(reinterpret_cast<float4*>(red[warp]) + lane) = make_float4(acc[0], acc[1], acc[2], acc[3]);
  if (lane == 0) zs[warp] = z;
  __syncthreads();
  const float zt = (zs[0] + zs[1]) + (zs[2] + zs[3]);
  const int d = threadIdx.x;
  const size_t head = blockIdx.x;
  w.o[head * kHeadDim + d] = __float2bfloat16(((red[0][d] + red[1][d]) + (red[2][d] + red[3][d])) / zt);
  if (w.lse && d == 0) w.lse[head] = (mx + lg2(zt)) * 0.6931471805599453f;
}

}  // namespace infllmv2
