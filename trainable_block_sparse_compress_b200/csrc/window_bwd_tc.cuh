// window_bwd_tc.cuh -- backward of the sliding-window attention (csrc/window.cuh states it) on
// the 5th-generation tensor cores.
//
// Rows are (token, head of the group) as in the forward: 128 / G tokens x G heads a tile.
//   window_delta_kernel  D = dO . O and lse in base 2, negated, one value per row, laid out row by
//           row ([B, Hkv, token, head of the group], tokens padded to 128) so that a tile's 128
//           values are contiguous; rows past a sequence's end get -lse = -inf (P = 0) and D = 0.
//   window_bwd_tc_kernel, dK / dV items: per 128 keys of a (sequence, kv-head), over the query tiles
//           that see one of them: S^T = K Q^T and dP^T = V dO^T (keys x rows), P^T = exp2(S^T - lse),
//           dS^T = P^T (dP^T - D), then dV += P^T dO and dK += dS^T Q with P^T and dS^T as A
//           operands in TMEM (bf16, written over S^T and dP^T): nothing but the Q / dO tiles
//           passes through shared memory, and the group's heads are summed in the accumulator.
//   window_bwd_tc_kernel, dq items: per 128 rows, over the keys that they see: S = Q K^T, dP = dO V^T,
//           dQ += dS K with dS as the A operand in TMEM.
// S and dP are computed in both (7 products instead of 5): that keeps dq out of fp32 atomics
// (its order of sums is fixed) and of a 4-byte accumulator in HBM.
// A tile of keys that holds sinks is seen by every later query: its query range (and any
// other, when there are few tiles of keys) is cut into chunks of query tiles whose
// partial sums meet in the workspace; window_dkdv_merge_kernel adds them in order.
// P and dS are rounded to bf16 as operands, dq, dK and dV once at the end; all else is fp32.
//
// Bound by the tensor pipe (70 % busy) and, in long runs, the power cap.  Measured, 32768 tokens,
// 32 / 2 heads, W 4096, 64 sinks: 5.6 ms (0.94 PFLOP/s of the algorithmic 5 products, 1.3 of the 7),
// 6.4 to 6.5 ms a call back to back.  Two elementwise warpgroups of 64 columns each instead of four: 10 ms.
#pragma once
#include "common.cuh"
#include "tcgen05.cuh"
#include "window_tc.cuh"

namespace infllmv2 {

constexpr int kWbGroups = 4;                 // elementwise warpgroups, 32 columns of a tile each
constexpr int kWbEltWarps = 4 * kWbGroups;
constexpr int kWbThreads = 32 * (kWbEltWarps + 2);
constexpr int kWbTmaWarp = kWbEltWarps, kWbMmaWarp = kWbEltWarps + 1;
constexpr int kWbSlots = 5;
constexpr int kWbKeys = 128;  // keys of a dK / dV tile

struct WbSmem {
  uint64_t res_full, full[kWbSlots], s_full, dp_full, p_full, ds_full, free_[2], done, mma_done, tail[2];
  uint64_t st_full[2], st_empty[2];
  alignas(16) float stats[2][2][128];  // dK / dV: lse and D of a query tile's rows
  uint32_t tmem_base;
  volatile int abort;
};

constexpr size_t window_bwd_smem_bytes() {
  return static_cast<size_t>(2 + kWbSlots) * kWfTileBytes + sizeof(WbSmem);
}
static_assert(window_bwd_smem_bytes() <= 227 * 1024, "shared memory of one CTA");

struct WinBwdParams {
  WinParams w;
  int g_log2, Lp;       // Lp: tokens padded to a multiple of 128
  float *lse2, *delta;  // [B, Hkv, Lp, G]: -lse in base 2 and -D
  // dK / dV: key tiles 0 .. sink_tiles-1 have chunks_s chunks of q_tiles_s query tiles, the others
  // chunks_w of q_tiles_w; a kind with more than one chunk goes through the partials
  int key_tiles, sink_tiles, chunks_s, chunks_w, q_tiles_s, q_tiles_w, row_tiles;
  int kv_items;         // CTAs of the dK / dV part
  float* part;          // [chunk slot][dV, dK][128 keys][128]
};

// One half-warp per four heads of a token, four rows of O and dO in flight: bound by HBM.
// grid-stride over B * Lp * ceil(Hq / 4) items, two to a warp.
__global__ void __launch_bounds__(256) window_delta_kernel(const WinBwdParams p) {
  const WinParams& w = p.w;
  const int l = threadIdx.x & 15;
  allow_dependent_launch();
  grid_dependency_wait();
  const unsigned groups = (static_cast<unsigned>(w.Hq) + 3) / 4, items = static_cast<unsigned>(w.B) * p.Lp * groups;
  for (unsigned base = blockIdx.x * 16 + (threadIdx.x >> 5) * 2; base < items; base += gridDim.x * 16) {
    const unsigned it = min(base + ((threadIdx.x >> 4) & 1), items - 1);  // an odd count: the last twice
    const unsigned tok = it / groups, b = tok / static_cast<unsigned>(p.Lp);
    const int h0 = static_cast<int>(it - tok * groups) * 4, t = static_cast<int>(tok - b * p.Lp);
    const bool in = t < chunk_lens(w.q_lens, w.kv_lens, static_cast<int>(b), w.Lq, w.Lmax).q_len;
    const size_t o = ((static_cast<size_t>(b) * w.Lq + t) * w.Hq + h0) * kHeadDim;
    const bool mine = l < 4 && h0 + l < w.Hq;  // lane l: head h0 + l
    float lse = INFINITY, dl = 0.f;
    if (in && mine) lse = w.lse[(static_cast<size_t>(b) * w.Hq + h0 + l) * w.Lq + t] * 1.4426950408889634f;
    uint4 x[4], y[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      x[u] = y[u] = make_uint4(0, 0, 0, 0);
      if (in && h0 + u < w.Hq) {
        x[u] = *(reinterpret_cast<const uint4*>(w.o_in + o + u * kHeadDim) + l);
        y[u] = *(reinterpret_cast<const uint4*>(w.d_o + o + u * kHeadDim) + l);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t xa[4] = {x[u].x, x[u].y, x[u].z, x[u].w}, xb[4] = {y[u].x, y[u].y, y[u].z, y[u].w};
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s = fmaf(__uint_as_float(xa[i] << 16), __uint_as_float(xb[i] << 16), s);
        s = fmaf(__uint_as_float(xa[i] & 0xffff0000u), __uint_as_float(xb[i] & 0xffff0000u), s);
      }
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d, 16);
      if (l == u) dl = s;
    }
    if (mine) {
      const int h = h0 + l;
      const size_t i = ((static_cast<size_t>(b) * w.Hkv + (h >> p.g_log2)) * p.Lp + t) * w.G + (h & (w.G - 1));
      p.lse2[i] = -lse;
      p.delta[i] = -dl;
    }
  }
}

// Zeroes rows r0 .. 127 of a 128-row tile (both halves), by one warp.
__device__ __forceinline__ void zero_tile_rows(unsigned char* tile, int r0, int lane) {
  for (int i = max(r0, 0) * 8 + lane; i < 128 * 8; i += 32) {
    *reinterpret_cast<uint4*>(tile + i * 16) = make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(tile + kWfHalf + i * 16) = make_uint4(0, 0, 0, 0);
  }
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z,
                                            int u) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(u)
      : "memory");
}

// Query tokens that see a key of tile `i`: from its first key to t_end(i) (exclusive).
__device__ __forceinline__ int window_t_end(const WinParams& w, int i, int len) {
  if (i * kWbKeys < w.n_sink) return len;
  return static_cast<int>(min(static_cast<long long>(len), static_cast<long long>(i) * kWbKeys + kWbKeys - 1 + w.window));
}

// Zeroes the values of 16 pairs whose bit (0..31) is not set.
__device__ __forceinline__ void mask_pairs(uint64_t (&v)[16], uint32_t bits) {
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    float a, b;
    unf2(v[q], a, b);
    v[q] = f2((bits >> (2 * q)) & 1u ? a : 0.f, (bits >> (2 * q + 1)) & 1u ? b : 0.f);
  }
}

// D[tmem] += A[tmem] * B: A holds 32 values of K in the first 16 columns of each of its four
// 32-column quarters (a warpgroup writes its quarter over what it has read), B's 128 rows are
// the K axis.
__device__ __forceinline__ void umma_acc(uint32_t d, uint32_t a, uint64_t b, bool first) {
  constexpr uint32_t id = idesc_bf16_f32(128, 128, false, true);
#pragma unroll
  for (int k = 0; k < 8; ++k)
    umma_bf16_ta(d, a + 32u * (k >> 1) + 8u * (k & 1), b + static_cast<uint64_t>(k * (2048 >> 4)), id,
                 (!first || k > 0) ? 1u : 0u);
}

// The ring as its reader sees it: items in order, their slots counted (a division by the number
// of slots would be on the issuing thread's path, which bounds the tensor pipe).
struct WbRing {
  int slot = 0;
  uint32_t phase = 0;
  // has the next item landed?  Asked a batch of products ahead of take(), which costs ~120 cycles
  // when it has to look.
  __device__ __forceinline__ bool probe(WbSmem& S) const { return mbar_test(&S.full[slot], phase); }
  // waits for the next item; its slot's offset in descriptor units, or -1 after a timeout
  __device__ __forceinline__ int take(WbSmem& S, bool seen = false) {
    const bool ok = seen || mbar_wait_short(&S.full[slot], phase, &S.abort);
    tc_fence_after();
    const int off = ok ? slot * (kWfTileBytes >> 4) : -1;
    if (++slot == kWbSlots) {
      slot = 0;
      phase ^= 1u;
    }
    return off;
  }
};

// One dK / dV item: `cta` of B * Hkv * (sink_tiles * chunks_s + (key_tiles - sink_tiles) *
// chunks_w).  TMEM: S^T 0, dP^T 128, dV 256, dK 384.
__device__ __forceinline__ void window_dkdv(const CUtensorMap& tm_q, const CUtensorMap& tm_do, const CUtensorMap& tm_k,
                                            const CUtensorMap& tm_v, const WinBwdParams& p, unsigned char* base,
                                            int cta) {
  unsigned char* kv = base;                        // K tile, V tile
  unsigned char* ring = base + 2 * kWfTileBytes;   // Q / dO slots: Q0 dO0 Q1 dO1 ...
  WbSmem& S = *reinterpret_cast<WbSmem*>(ring + kWbSlots * kWfTileBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WinParams& w = p.w;

  const int bg = cta % (w.B * w.Hkv), e = cta / (w.B * w.Hkv);
  const bool sink_kind = e < p.sink_tiles * p.chunks_s;
  const int chunks = sink_kind ? p.chunks_s : p.chunks_w;
  const int e2 = sink_kind ? e : e - p.sink_tiles * p.chunks_s;
  const int tile = (sink_kind ? 0 : p.sink_tiles) + e2 / chunks, chunk = e2 % chunks;
  const int b = bg / w.Hkv, g = bg - b * w.Hkv;
  const int tt = 128 >> p.g_log2;
  const int len = chunk_lens(w.q_lens, w.kv_lens, b, w.Lq, w.Lmax).q_len;
  const int u0 = tile * kWbKeys;
  if (u0 >= len) return;
  const int t_end = window_t_end(w, tile, len);
  const int n_all = (t_end - u0 + tt - 1) / tt;
  const int q_tiles = sink_kind ? p.q_tiles_s : p.q_tiles_w;
  const int i0 = chunk * q_tiles, i1 = chunks == 1 ? n_all : min(n_all, i0 + q_tiles);
  if (i0 >= i1) return;
  const int n = i1 - i0;
  const int ta = u0 + i0 * tt;  // first token
  // The query tiles are taken from the first multiple of n on, round: CTAs that start together then
  // read the same tokens at the same time although their ranges start a key tile apart, and L2
  // serves them (16K tokens, W 4096: 6.4 GB from HBM when each starts at its own first token).
  const int turn = (n - (ta / tt) % n) % n;
  auto tile_at = [&](int i) { return i + turn < n ? i + turn : i + turn - n; };

  if (threadIdx.x == 0) {
    mbar_init(&S.res_full, 1);
    for (int s = 0; s < kWbSlots; ++s) mbar_init(&S.full[s], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&S.tail[s], 1);
      mbar_init(&S.st_full[s], 1);
      mbar_init(&S.st_empty[s], kWbEltWarps);
    }
    mbar_init(&S.s_full, 1);
    mbar_init(&S.p_full, kWbEltWarps);
    mbar_init(&S.ds_full, kWbEltWarps);
    mbar_init(&S.dp_full, 1);
    mbar_init(&S.done, 1);
    mbar_init(&S.mma_done, 1);
    S.abort = 0;
    fence_mbar_init();
  }
  if (warp == kWbMmaWarp) {
    tmem_alloc(&S.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;

  if (warp == kWbTmaWarp) {
    if (lane == 0) {
      mbar_arrive_expect_tx(&S.res_full, 2 * kWfTileBytes);
      for (int h = 0; h < 2; ++h)
        for (int s = 0; s < 2; ++s) {
          tma_load_3d(kv + h * kWfHalf + s * (kWfSeg * 128), &tm_k, &S.res_full, 64 * h, u0 + 64 * s, bg);
          tma_load_3d(kv + kWfTileBytes + h * kWfHalf + s * (kWfSeg * 128), &tm_v, &S.res_full, 64 * h, u0 + 64 * s,
                      bg);
        }
    }
    const size_t stat0 = (static_cast<size_t>(bg) * p.Lp + ta) << p.g_log2;
    int slot = 0, issued = 0;
    int stats = 0;
    uint32_t tails = 0;
    bool stop = false;
    for (int i = 0; i < n && !stop; ++i) {
      const int o = tile_at(i), t0 = ta + o * tt;
      const bool any = w.q_lens != nullptr && t0 + tt > len;  // rows past the end may hold anything
      for (int kd = 0; kd < 2; ++kd) {
        // Items 2t + 5 and 2t + 6 take the slots of Q and dO of tile t, which have been read once dP
        // of tile t + 1 is complete (dV and dK of tile t were issued before it).  Its barrier is
        // never two phases on: dP of tile t + 2 waits for item 2t + 5, and dP of tile 0, whose phase
        // must be over before the next is asked for, is waited for before dP of tile 1 can start.
        if (issued == 3) mbar_wait_short(&S.dp_full, 0, &S.abort);
        if (issued >= kWbSlots && issued % 2 == 1)
          mbar_wait_short(&S.dp_full, static_cast<uint32_t>((issued - kWbSlots) / 2 + 1) & 1u, &S.abort);
        if (kd == 0 && i >= 2) mbar_wait_short(&S.st_empty[i & 1], static_cast<uint32_t>((i >> 1) - 1) & 1u, &S.abort);
        stop = __any_sync(0xffffffffu, S.abort != 0);
        if (stop) break;
        unsigned char* dst = ring + slot * kWfTileBytes;
        if (lane == 0) {
          uint64_t* bar = any ? &S.tail[kd] : &S.full[slot];
          mbar_arrive_expect_tx(bar, kWfTileBytes);
          for (int h = 0; h < 2; ++h)
            tma_load_4d(dst + h * kWfHalf, kd ? &tm_do : &tm_q, bar, 64 * h, g << p.g_log2, t0, b);
          if (kd == 0) {
            mbar_arrive_expect_tx(&S.st_full[i & 1], 1024);
            for (int s = 0; s < 2; ++s)
              asm volatile(
                  "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], 512, [%2];" ::"r"(
                      smem_u32(S.stats[i & 1][s])),
                  "l"((s ? p.delta : p.lse2) + stat0 + static_cast<size_t>(o) * 128), "r"(smem_u32(&S.st_full[i & 1]))
                  : "memory");
          }
        }
        if (kd == 0) ++stats;
        ++issued;
        if (any) {
          tails |= 1u << kd;
          if (mbar_wait_short(&S.tail[kd], 0, &S.abort)) zero_tile_rows(dst, (len - t0) << p.g_log2, lane);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.full[slot]);
        }
        __syncwarp();
        if (++slot == kWbSlots) slot = 0;
      }
    }
    if (lane == 0) {  // every copy this thread issued lands before the CTA ends
      mbar_wait_drain(&S.res_full, 0);
      for (int kd = 0; kd < 2; ++kd)
        if ((tails >> kd) & 1u) mbar_wait_drain(&S.tail[kd], 0);
      drain_ring(S.full, issued);
      drain_ring(S.st_full, stats);
    }
    return;
  }

  if (warp == kWbMmaWarp) {
    // The warp stays converged: with the operands in uniform registers a product takes few issue
    // slots, for which this warp competes with the elementwise warps of its scheduler.
    const bool lead = elect_one();
    const uint64_t kd = desc_k_sw128(smem_u32(kv)), vd = kd + (kWfTileBytes >> 4);
    const uint64_t rk = desc_k_sw128(smem_u32(ring)), rm = desc_mn_sw128(smem_u32(ring), kWfHalf, 1024);
    // Order: S(0) dP(0) | dV(i) S(i+1) | dK(i) dP(i+1).  dV(i) and S(i+1) run while dS(i) is
    // formed, dK(i) and dP(i+1) while the exponentials of tile i+1 are.
    WbRing items;
    int q = -1, o = -1;  // offsets of tile i's Q and dO
    bool ok = mbar_wait_short(&S.res_full, 0, &S.abort) && (q = items.take(S)) >= 0;
    if (ok) {
      if (lead) {
        umma_rows(tmem, kd, rk + q);
        umma_commit(&S.s_full);
      }
      ok = (o = items.take(S)) >= 0;
    }
    if (ok && lead) {
      umma_rows(tmem + 128, vd, rk + o);
      umma_commit(&S.dp_full);
    }
    for (int i = 0; i < n && ok; ++i) {
      const bool more = i + 1 < n;
      int qn = 0, on = 0;
      if (!mbar_wait_short(&S.p_full, i & 1u, &S.abort)) break;
      bool seen = more && items.probe(S);
      tc_fence_after();
      if (lead) umma_acc(tmem + 256, tmem, rm + o, i == 0);
      if (more) {
        if ((qn = items.take(S, seen)) < 0) break;
        if (lead) {
          umma_rows(tmem, kd, rk + qn);
          umma_commit(&S.s_full);
        }
      }
      if (!mbar_wait_short(&S.ds_full, i & 1u, &S.abort)) break;
      seen = more && items.probe(S);
      tc_fence_after();
      if (lead) umma_acc(tmem + 384, tmem + 128, rm + q, i == 0);
      if (more) {
        if ((on = items.take(S, seen)) < 0) break;
        if (lead) {
          umma_rows(tmem + 128, vd, rk + on);
          umma_commit(&S.dp_full);
        }
      }
      q = qn;
      o = on;
    }
    if (lead) {
      umma_commit(&S.done);
      umma_commit(&S.mma_done);
    }
    __syncwarp();
    named_bar_sync(1, 32 * (kWbEltWarps + 1));
    if (lane == 0) mbar_wait_drain(&S.mma_done, 0);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
    return;
  }

  // ------------------------------- elementwise: thread = key, a warpgroup 32 of the tile's rows
  const int wg = warp >> 2;
  const int key = threadIdx.x & 127, u = u0 + key;
  const uint32_t tl = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + 32u * wg;
  const uint64_t sl2 = f2(w.scale_log2, w.scale_log2);
  // rows (of this warpgroup's 32) whose queries see the key: tokens u .. hi - 1
  const int hi = u < w.n_sink ? len : static_cast<int>(min(static_cast<long long>(len), static_cast<long long>(u) + w.window));
  for (int i = 0; i < n; ++i) {
    const int t0 = ta + tile_at(i) * tt;
    // every key of the tile is seen by every row: no masks
    const bool all = t0 >= u0 + kWbKeys - 1 && t0 + tt <= len &&
                     (static_cast<long long>(t0) + tt <= static_cast<long long>(u0) + w.window || u0 + kWbKeys <= w.n_sink);
    const float4* st = reinterpret_cast<const float4*>(S.stats[i & 1][0] + 32 * wg);
    const float4* sd = reinterpret_cast<const float4*>(S.stats[i & 1][1] + 32 * wg);
    mbar_wait_short(&S.st_full[i & 1], static_cast<uint32_t>(i >> 1) & 1u, &S.abort);
    mbar_wait_short(&S.s_full, i & 1u, &S.abort);
    tc_fence_after();
    uint32_t v[32];
    tmem_ld32_nowait(tl, v);
    uint64_t pr[16];  // P^T, in pairs
    tmem_wait_ld_tied(v);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float4 ls = st[q];  // negated lse
      pr[2 * q] = fma2(f2(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1])), sl2, f2(ls.x, ls.y));
      pr[2 * q + 1] = fma2(f2(__uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3])), sl2, f2(ls.z, ls.w));
    }
#pragma unroll
    for (int q = 0; q < 16; ++q) pr[q] = ex2_pair(pr[q]);
    uint32_t mk = 0xffffffffu;
    if (!all) {
      mk = static_cast<uint32_t>(low_bits(static_cast<long long>(hi - t0) * w.G - 32 * wg) &
                                 ~low_bits(static_cast<long long>(u - t0) * w.G - 32 * wg));
      mask_pairs(pr, mk);
    }
    uint32_t pk[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) pk[q] = pack_pair(pr[q]);
    tmem_st16_nowait(tl, pk);
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.p_full);
    mbar_wait_short(&S.dp_full, i & 1u, &S.abort);
    tc_fence_after();
    tmem_ld32_nowait(tl + 128, v);
    tmem_wait_ld_tied(v);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float4 dl = sd[q];  // negated D
      pr[2 * q] = mul2(pr[2 * q], add2(f2(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1])), f2(dl.x, dl.y)));
      pr[2 * q + 1] =
          mul2(pr[2 * q + 1], add2(f2(__uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3])), f2(dl.z, dl.w)));
    }
    if (!all) mask_pairs(pr, mk);  // dP of a masked place may be anything
#pragma unroll
    for (int q = 0; q < 16; ++q) pk[q] = pack_pair(pr[q]);
    tmem_st16_nowait(tl + 128, pk);
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&S.ds_full);
      mbar_arrive(&S.st_empty[i & 1]);
    }
  }
  mbar_wait_short(&S.done, 0, &S.abort);
  tc_fence_after();
  // warpgroups 0, 1 write dV, 2, 3 dK: thread = key, half of its 128 values
  const uint32_t acc = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + 256u + 64u * wg;
  const int which = wg >> 1, c0 = 64 * (wg & 1);
  const float f = which ? w.scale : 1.f;
  // slot of the partials: the CTA's place among those of split kinds
  const int slot = (sink_kind ? 0 : (p.chunks_s > 1 ? p.sink_tiles * p.chunks_s : 0)) + e2;
  const size_t item = static_cast<size_t>(slot) * (w.B * w.Hkv) + bg;
#pragma unroll 1
  for (int q = 0; q < 2; ++q) {
    uint32_t v[32];
    __syncwarp();
    tmem_ld32(acc + 32 * q, v);
    if (chunks > 1) {
      float4* dst = reinterpret_cast<float4*>(p.part + ((item * 2 + which) * kWbKeys + key) * kHeadDim + c0 + 32 * q);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        dst[i] = make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]), __uint_as_float(v[4 * i + 2]),
                             __uint_as_float(v[4 * i + 3]));
    } else if (u < len) {
      uint4* dst = reinterpret_cast<uint4*>((which ? w.dk : w.dv) + (static_cast<size_t>(bg) * w.Lmax + u) * kHeadDim + c0 + 32 * q);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t x[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          x[c] = pack_bf16(__uint_as_float(v[8 * i + 2 * c]) * f, __uint_as_float(v[8 * i + 2 * c + 1]) * f);
        dst[i] = make_uint4(x[0], x[1], x[2], x[3]);
      }
    }
  }
  tc_fence_before();
  named_bar_sync(1, 32 * (kWbEltWarps + 1));  // TMEM may be freed
}

// Adds the chunks of the split key tiles in order: a warp per (key, dV or dK) row.
// grid.x covers the split tiles of one (sequence, kv-head) x 128 keys x 2 / 8, grid.y = B * Hkv.
__global__ void __launch_bounds__(256) window_dkdv_merge_kernel(const WinBwdParams p, int first_tile, int tiles) {
  const WinParams& w = p.w;
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int ti = row / (2 * kWbKeys), which = row / kWbKeys & 1, key = row & (kWbKeys - 1);
  grid_dependency_wait();
  if (ti >= tiles) return;
  const int tile = first_tile + ti, bg = blockIdx.y, b = bg / w.Hkv;
  const int len = chunk_lens(w.q_lens, w.kv_lens, b, w.Lq, w.Lmax).q_len;
  const int u = tile * kWbKeys + key;
  if (u >= len) return;
  const bool sink = tile < p.sink_tiles;
  const int chunks = sink ? p.chunks_s : p.chunks_w;
  const int slot0 = sink ? tile * chunks : (p.chunks_s > 1 ? p.sink_tiles * p.chunks_s : 0) + (tile - p.sink_tiles) * chunks;
  const int tt = 128 >> p.g_log2;
  const int n_all = (window_t_end(w, tile, len) - tile * kWbKeys + tt - 1) / tt;
  const int q_tiles = sink ? p.q_tiles_s : p.q_tiles_w;
  const int live = min(chunks, (n_all + q_tiles - 1) / q_tiles);
  float a[4] = {0.f, 0.f, 0.f, 0.f};
  for (int c = 0; c < live; ++c) {
    const size_t item = static_cast<size_t>(slot0 + c) * (w.B * w.Hkv) + bg;
    const float4 x = *(reinterpret_cast<const float4*>(p.part + ((item * 2 + which) * kWbKeys + key) * kHeadDim) + lane);
    a[0] += x.x, a[1] += x.y, a[2] += x.z, a[3] += x.w;
  }
  if (which)
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] *= w.scale;
  store4((which ? w.dk : w.dv) + (static_cast<size_t>(bg) * w.Lmax + u) * kHeadDim, lane, a);
}

// One dq item: `cta` of row_tiles * B * Hkv, the last row tiles first.  TMEM: S 0, dP 128 (dS
// over it), dQ 384.
__device__ __forceinline__ void window_dq(const CUtensorMap& tm_q, const CUtensorMap& tm_do, const CUtensorMap& tm_k,
                                          const CUtensorMap& tm_v, const CUtensorMap& tm_ks, const CUtensorMap& tm_vs,
                                          const WinBwdParams& p, unsigned char* base, int cta) {
  unsigned char* qd = base;                        // Q tile, dO tile
  unsigned char* ring = base + 2 * kWfTileBytes;   // K / V slots: K0 V0 K1 V1 ...
  WbSmem& S = *reinterpret_cast<WbSmem*>(ring + kWbSlots * kWfTileBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WinParams& w = p.w;

  const int bg = cta % (w.B * w.Hkv);
  const int tile = p.row_tiles - 1 - cta / (w.B * w.Hkv);
  const int b = bg / w.Hkv, g = bg - b * w.Hkv;
  const int tt = 128 >> p.g_log2;
  const int r0 = tile * tt;
  const int len = chunk_lens(w.q_lens, w.kv_lens, b, w.Lq, w.Lmax).q_len;
  if (r0 >= len) return;
  const int t_last = min(r0 + tt, len) - 1;
  const WinRuns runs(r0, t_last, w.window, w.n_sink);
  const int n = runs.tiles();

  if (threadIdx.x == 0) {
    mbar_init(&S.res_full, 1);
    for (int s = 0; s < kWbSlots; ++s) mbar_init(&S.full[s], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&S.tail[s], 1);
      mbar_init(&S.free_[s], 1);
    }
    mbar_init(&S.s_full, 1);
    mbar_init(&S.p_full, kWbEltWarps);
    mbar_init(&S.ds_full, kWbEltWarps);
    mbar_init(&S.dp_full, 1);
    mbar_init(&S.done, 1);
    mbar_init(&S.mma_done, 1);
    S.abort = 0;
    fence_mbar_init();
  }
  if (warp == kWbMmaWarp) {
    tmem_alloc(&S.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;

  if (warp == kWbTmaWarp) {
    if (lane == 0) {
      mbar_arrive_expect_tx(&S.res_full, 2 * kWfTileBytes);
      for (int h = 0; h < 2; ++h) {
        tma_load_4d(qd + h * kWfHalf, &tm_q, &S.res_full, 64 * h, g << p.g_log2, r0, b);
        tma_load_4d(qd + kWfTileBytes + h * kWfHalf, &tm_do, &S.res_full, 64 * h, g << p.g_log2, r0, b);
      }
    }
    int slot = 0, issued = 0;
    bool tail_used = false, stop = false;
    for (int j = 0; j < n && !stop; ++j)
      for (int kv = 0; kv < 2; ++kv) {
        // Items 2t + 5 and 2t + 6 take the slots of K and V of tile t, which have been read once dQ
        // of tile t is complete.  dQ of tile t + 2 waits for item 2t + 5, so the barrier of tile t
        // (one of two) is never a phase further.
        if (issued >= kWbSlots && issued % 2 == 1) {
          const int t = (issued - kWbSlots) / 2;
          mbar_wait_short(&S.free_[t & 1], static_cast<uint32_t>(t >> 1) & 1u, &S.abort);
        }
        stop = __any_sync(0xffffffffu, S.abort != 0);
        if (stop) break;
        unsigned char* dst = ring + slot * kWfTileBytes;
        // rows of K past the sequence's end may hold anything (dS there is 0, but 0 x NaN is not)
        int clean[2];
        bool any = false;
        for (int s = 0; s < 2; ++s) {
          const int seg = 2 * j + s;
          clean[s] = seg < runs.ns + runs.nw && !runs.is_sink(seg) ? len - runs.first_key(seg) : kWfSeg;
          any |= kv == 0 && w.kv_lens != nullptr && clean[s] < kWfSeg;
        }
        if (lane == 0) {
          uint64_t* bar = any ? &S.tail[0] : &S.full[slot];
          mbar_arrive_expect_tx(bar, kWfTileBytes);
          for (int s = 0; s < 2; ++s) {
            const int seg = 2 * j + s;
            const bool pad = seg >= runs.ns + runs.nw;
            const CUtensorMap* m = runs.is_sink(seg) ? (kv ? &tm_vs : &tm_ks) : (kv ? &tm_v : &tm_k);
            const int k0 = pad ? w.Lmax : runs.first_key(seg);
            for (int h = 0; h < 2; ++h)
              tma_load_3d(dst + h * kWfHalf + s * (kWfSeg * 128), m, bar, 64 * h, k0, bg);
          }
        }
        ++issued;
        if (any) {
          tail_used = true;
          if (mbar_wait_short(&S.tail[0], 0, &S.abort))
            for (int s = 0; s < 2; ++s)
              for (int i = max(clean[s], 0) * 8 + lane; i < kWfSeg * 8; i += 32)
                for (int h = 0; h < 2; ++h)
                  *reinterpret_cast<uint4*>(dst + h * kWfHalf + s * (kWfSeg * 128) + i * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.full[slot]);
        }
        __syncwarp();
        if (++slot == kWbSlots) slot = 0;
      }
    if (lane == 0) {  // every copy this thread issued lands before the CTA ends
      mbar_wait_drain(&S.res_full, 0);
      if (tail_used) mbar_wait_drain(&S.tail[0], 0);
      drain_ring(S.full, issued);
    }
    return;
  }

  if (warp == kWbMmaWarp) {
    const bool lead = elect_one();  // as for dK / dV
    const uint64_t qdesc = desc_k_sw128(smem_u32(qd)), ddesc = qdesc + (kWfTileBytes >> 4);
    const uint64_t rk = desc_k_sw128(smem_u32(ring)), rm = desc_mn_sw128(smem_u32(ring), kWfHalf, 1024);
    // Order: S(0) dP(0) | S(j+1) | dQ(j) dP(j+1).  S(j+1) starts once the scores of tile j are in
    // registers and is there when their dS is done; dP(j+1) runs under the exponentials.
    WbRing items;
    int k0 = -1, k1 = -1;  // offsets of K of tiles j and j + 1
    auto issue_s = [&](int& k, bool seen) {
      if ((k = items.take(S, seen)) < 0) return false;
      if (lead) {
        umma_rows(tmem, qdesc, rk + k);
        umma_commit(&S.s_full);
      }
      return true;
    };
    auto issue_dp = [&](bool seen) {
      const int v = items.take(S, seen);
      if (v < 0) return false;
      if (lead) {
        umma_rows(tmem + 128, ddesc, rk + v);
        umma_commit(&S.dp_full);
      }
      return true;
    };
    bool ok = mbar_wait_short(&S.res_full, 0, &S.abort) && issue_s(k0, false) && issue_dp(false);
    for (int j = 0; j < n && ok; ++j) {
      const bool more = j + 1 < n;
      bool seen = more && items.probe(S);
      if (!mbar_wait_short(&S.p_full, j & 1u, &S.abort)) break;  // the scores have been read
      tc_fence_after();
      if (more && !issue_s(k1, seen)) break;
      if (!mbar_wait_short(&S.ds_full, j & 1u, &S.abort)) break;
      seen = more && items.probe(S);
      tc_fence_after();
      if (lead) {
        umma_acc(tmem + 384, tmem + 128, rm + k0, j == 0);
        umma_commit(&S.free_[j & 1]);
      }
      k0 = k1;
      if (more && !issue_dp(seen)) break;
    }
    if (lead) {
      umma_commit(&S.done);
      umma_commit(&S.mma_done);
    }
    __syncwarp();
    named_bar_sync(1, 32 * (kWbEltWarps + 1));
    if (lane == 0) mbar_wait_drain(&S.mma_done, 0);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
    return;
  }

  // -------------------------- elementwise: thread = row, a warpgroup 32 keys (half a segment)
  const int wg = warp >> 2;
  const int row = threadIdx.x & 127;
  const int t = r0 + (row >> p.g_log2);
  const bool valid = t < len;
  const size_t si = ((static_cast<size_t>(bg) * p.Lp + r0) << p.g_log2) + row;
  const float nl = p.lse2[si], nd = p.delta[si];  // negated
  const uint64_t lse2 = f2(nl, nl), dl = f2(nd, nd), sl2 = f2(w.scale_log2, w.scale_log2);
  const uint32_t lane0 = static_cast<uint32_t>(32 * (warp & 3)) << 16;
  for (int j = 0; j < n; ++j) {
    const int seg = 2 * j + (wg >> 1), u0 = runs.first_key(seg);
    const bool all = u0 + kWfSeg - 1 <= r0 && t_last == r0 + tt - 1 &&
                     (runs.is_sink(seg) ? u0 + kWfSeg <= w.n_sink
                                        : (u0 > t_last - w.window || u0 + kWfSeg <= w.n_sink));
    const uint32_t ts = tmem + lane0 + 32u * wg, td = ts + 128u;
    mbar_wait_short(&S.s_full, j & 1u, &S.abort);
    tc_fence_after();
    uint32_t v[32];
    tmem_ld32_nowait(ts, v);
    uint64_t pr[16];
    tmem_wait_ld_tied(v);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.p_full);  // S may be overwritten
#pragma unroll
    for (int q = 0; q < 16; ++q)
      pr[q] = ex2_pair(fma2(f2(__uint_as_float(v[2 * q]), __uint_as_float(v[2 * q + 1])), sl2, lse2));
    mbar_wait_short(&S.dp_full, j & 1u, &S.abort);
    tc_fence_after();
    tmem_ld32_nowait(td, v);
    tmem_wait_ld_tied(v);
#pragma unroll
    for (int q = 0; q < 16; ++q)
      pr[q] = mul2(pr[q], add2(f2(__uint_as_float(v[2 * q]), __uint_as_float(v[2 * q + 1])), dl));
    if (!all) mask_pairs(pr, valid ? static_cast<uint32_t>(runs.mask(seg, t, w.window) >> (32 * (wg & 1))) : 0u);
    uint32_t pk[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) pk[q] = pack_pair(pr[q]);
    tmem_st16_nowait(td, pk);
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.ds_full);
  }
  mbar_wait_short(&S.done, 0, &S.abort);
  tc_fence_after();
  // a warpgroup writes 32 of the row's 128 values
  const int h = (g << p.g_log2) + (row & (w.G - 1));
  {
    uint32_t v[32];
    __syncwarp();
    tmem_ld32(tmem + lane0 + 384u + 32u * wg, v);
    if (valid) {
      uint4* dst = reinterpret_cast<uint4*>(w.dq + ((static_cast<size_t>(b) * w.Lq + t) * w.Hq + h) * kHeadDim + 32 * wg);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t x[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          x[c] = pack_bf16(__uint_as_float(v[8 * i + 2 * c]) * w.scale, __uint_as_float(v[8 * i + 2 * c + 1]) * w.scale);
        dst[i] = make_uint4(x[0], x[1], x[2], x[3]);
      }
    }
  }
  tc_fence_before();
  named_bar_sync(1, 32 * (kWbEltWarps + 1));  // TMEM may be freed
}

// grid = the dK / dV items (long), then the dq items, which fill the SMs that the last of the
// former leave idle.
__global__ void __launch_bounds__(kWbThreads, 1)
    window_bwd_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                         const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ CUtensorMap tm_ks, const __grid_constant__ CUtensorMap tm_vs,
                         const WinBwdParams p) {
  extern __shared__ __align__(1024) unsigned char smem_1k[];
  const int cta = static_cast<int>(blockIdx.x);
  allow_dependent_launch();
  grid_dependency_wait();
  if (cta < p.kv_items)
    window_dkdv(tm_q, tm_do, tm_k, tm_v, p, smem_1k, cta);
  else
    window_dq(tm_q, tm_do, tm_k, tm_v, tm_ks, tm_vs, p, smem_1k, cta - p.kv_items);
}

}  // namespace infllmv2
