// window_tc.cuh -- forward of the sliding-window attention (csrc/window.cuh states it) on the
// 5th-generation tensor cores (tcgen05 + TMEM).
//
// A CTA takes two 128-row query tiles of one (sequence, kv-head): row = (token, head of the
// group), 128 / G tokens x G heads, so the group's heads share every K/V tile and a short
// window wastes few masked keys (the union of 256 / G tokens' windows).  The keys that any of
// the CTA's queries sees form at most two runs, the sinks and the window; they are cut into
// segments of 64 keys that start exactly at the run's first key, and two segments make a
// 128-key tile, so a few sinks cost half a tile.
//   warp 8  (one thread, TMA) streams Q once and K / V tiles through one ring of 32 KB slots
//           (order K0 V0 K1 V1 ..., also the order in which they are released);
//   warp 9  issues S_x = Q_x K^T (M128 N128 K16 x 8) and O_x += P_x V (A = P from TMEM, V through an
//           MN-major descriptor) for the two query tiles x in turn, so one tile's products run under
//           the other tile's softmax (an issuing warp for each x measured slower: the two streams
//           interleave and both tiles wait for both);
//   warps 0-3 / 4-7: one softmax warpgroup per query tile, thread = row: no shuffles.  The
//           reference maximum follows the running maximum lazily: only when a warp holds a row
//           whose maximum rose by more than 2^8 is O rescaled (in TMEM); P <= 2^8 keeps bf16's
//           relative precision.
// Sums and the maximum are fp32; P is rounded to bf16 (an operand of the second product), O once at
// the end.  P overwrites S in TMEM: 64 of its 128 columns, written in two halves so the first four
// K-steps of P V start before the second half's exponentials.  TMEM: S0 S1 O0 O1, all 512 columns.
//
// Bound by the chain of a tile: scores, softmax (~2100 cycles), P V and the next scores (~1100);
// the tensor pipe is busy 55 % of the time.  Measured: 128K prompt, 32 / 2 heads, W 4096: 1.17 PFLOP/s
// (7.5 ms; 8.7 ms a call back to back, under the power cap); 2 x 8191 tokens, 32 / 8 heads, causal:
// 0.94 ms (1.1 ms a call).
// 64-key tiles with two score buffers (no chain, but a 64-wide product takes 59 of a 128-wide one's
// 64 cycles) 11.2 ms; two threads a row 8.7.
#pragma once
#include "common.cuh"
#include "tcgen05.cuh"
#include "window.cuh"

namespace infllmv2 {

constexpr int kWfTileBytes = 128 * 128 * 2;  // 32 KB: 128 rows of Q, K or V (two 64-column halves)
constexpr int kWfHalf = kWfTileBytes / 2;
constexpr int kWfSeg = 64;                   // keys of a segment
constexpr int kWfSlots = 5;
constexpr int kWfThreads = 32 * 12;  // warps 10 and 11 only give their registers away
// Registers a thread: 168 at launch (65,536 over 12 warps), then 208 for the softmax warpgroups
// (a row's 128 scores stay in registers) and 72 for the third: 2 x 208 + 72 <= 3 x 168.
constexpr int kWfSoftRegs = 208, kWfOtherRegs = 72;
constexpr int kWfTmaWarp = 8, kWfMmaWarp = 9;
constexpr uint32_t kWfColO = 256;

struct WfSmem {
  uint64_t q_full[2], full[kWfSlots], step[2], s_full[2], p_full[2][2], mma_done, tail;
  uint32_t tmem_base;
  volatile int abort;
};

constexpr size_t window_tc_smem_bytes() {
  return 1024 + static_cast<size_t>(2 + kWfSlots) * kWfTileBytes + sizeof(WfSmem);
}
static_assert(window_tc_smem_bytes() <= 227 * 1024, "shared memory of one CTA");

// D[tmem] (+)= A[tmem] * B[smem]: A holds bf16 pairs, 8 columns for 16 values of K.
__device__ __forceinline__ void umma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %6, %7, %8}, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(0u), "r"(0u), "r"(0u), "r"(0u)
      : "memory");
}

// Products over 128 head dimensions: D[tmem] = A[128 rows] * B[128 rows]^T, both tiles K-major
// (descriptors of their first bytes).
__device__ __forceinline__ void umma_rows(uint32_t d, uint64_t a, uint64_t b) {
  constexpr uint32_t id = idesc_bf16_f32(128, 128, false, false);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint64_t o = static_cast<uint64_t>(((k >> 2) * kWfHalf + (k & 3) * 32) >> 4);
    umma_bf16(d, a + o, b + o, id, k > 0 ? 1u : 0u);
  }
}
// D[tmem] (+)= A[tmem] * B: 64 values of K, A in 32 columns, B's 64 rows (of 128 values).
__device__ __forceinline__ void umma_pv_half(uint32_t d, uint32_t a, uint64_t b, bool accumulate) {
  constexpr uint32_t id = idesc_bf16_f32(128, 128, false, true);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    umma_bf16_ta(d, a + 8u * k, b + static_cast<uint64_t>(k * (2048 >> 4)), id, (accumulate || k > 0) ? 1u : 0u);
}

// 32 columns of this thread's TMEM lane into v[0..31], without the wait (tmem_wait_ld follows).
__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
        "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
        "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}

// Waits for every load of this thread and ties the registers to the wait, so no use of them is
// scheduled before it.
template <int N>
__device__ __forceinline__ void tmem_wait_ld_tied(uint32_t (&v)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(v[i]));
}

// 16 columns of this thread's TMEM lane, without the wait (tmem_wait_st follows).
__device__ __forceinline__ void tmem_st16_nowait(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Bits 0 .. n-1 of a 64-bit mask (none for n <= 0, all for n >= 64).
__device__ __forceinline__ uint64_t low_bits(long long n) {
  return n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1ull);
}

// The keys of a CTA's queries, as segments of 64: `ns` segments of sinks from key 0, then `nw`
// segments from key `lo`.  When the sinks reach the window there is one run, from key 0.
struct WinRuns {
  int ns, nw, lo, n_sink, t_max;
  __device__ WinRuns(int t_min, int t_max_, int window, int n_sink_) : n_sink(n_sink_), t_max(t_max_) {
    const int a = max(0, t_min - window + 1);
    const bool one = n_sink_ >= a;
    lo = one ? 0 : a;
    ns = one ? 0 : (n_sink_ + kWfSeg - 1) / kWfSeg;
    nw = (t_max_ - lo + kWfSeg) / kWfSeg;
  }
  __device__ int tiles() const { return (ns + nw + 1) / 2; }
  __device__ bool is_sink(int seg) const { return seg < ns; }
  __device__ int first_key(int seg) const { return seg < ns ? seg * kWfSeg : lo + (seg - ns) * kWfSeg; }
  // keys of segment `seg` that the query at t sees
  __device__ uint64_t mask(int seg, int t, int window) const {
    const int u0 = first_key(seg);
    const uint64_t past = low_bits(static_cast<long long>(t) - u0 + 1);
    const uint64_t sink = low_bits(static_cast<long long>(n_sink) - u0);
    if (is_sink(seg)) return past & sink;
    return past & (sink | ~low_bits(static_cast<long long>(t) - window - u0 + 1));
  }
};

struct WinTcParams {
  WinParams w;
  int g_log2;          // log2 of the group size
  int rows;            // rows of a CTA: 256, or 128 (paired)
  int row_tiles;       // tiles of that many rows per (sequence, kv-head)
  int n_splits;        // key splits of a row tile (1: O and lse are written directly)
  float* part_o;       // splits: [CTA][rows][128] normalised partial outputs
  float* part_lse;     // [CTA][rows] base-2 log-sum-exps (-inf: no key)
};

// grid = row_tiles * B * Hkv * n_splits (the last row tiles, which see the most keys, first).
// kPaired, for calls of few rows: the CTA has one 128-row query tile, and x is not a query tile
// but every other key tile; the two states are joined through shared memory at the end.
template <bool kPaired>
__global__ void __launch_bounds__(kWfThreads, 1)
    window_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_ks,
                     const __grid_constant__ CUtensorMap tm_vs, const WinTcParams p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* base = align_smem(smem_raw, 1024);
  unsigned char* qs = base;                        // two query tiles
  unsigned char* ring = base + 2 * kWfTileBytes;   // K / V slots
  WfSmem& S = *reinterpret_cast<WfSmem*>(ring + kWfSlots * kWfTileBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WinParams& w = p.w;

  int bid = blockIdx.x;
  const int split = bid % p.n_splits;
  bid /= p.n_splits;
  const int bg = bid % (w.B * w.Hkv);
  const int tile = p.row_tiles - 1 - bid / (w.B * w.Hkv);
  const int b = bg / w.Hkv, g = bg - b * w.Hkv;
  const int tt = 128 >> p.g_log2;  // tokens of a 128-row tile
  const int ct = kPaired ? tt : 2 * tt;  // tokens of the CTA
  const int r0 = tile * ct;
  grid_dependency_wait();
  allow_dependent_launch();
  const ChunkLens c = chunk_lens(w.q_lens, w.kv_lens, b, w.Lq, w.Lmax);
  if (r0 >= c.q_len) return;
  const int pos0 = c.kv_len - c.q_len;
  const WinRuns runs(pos0 + r0, pos0 + min(r0 + ct, c.q_len) - 1, w.window, w.n_sink);
  // key tiles of this split, and of each query tile within them
  const int all = runs.tiles(), per = (all + p.n_splits - 1) / p.n_splits;
  const int j0 = min(split * per, all), j1 = min(j0 + per, all);
  int jb[2], je[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int ra = r0 + x * tt, rb = min(ra + tt, c.q_len) - 1;  // first and last row
    const int skip = runs.ns == 0 && w.n_sink == 0 ? max(0, pos0 + ra - w.window + 1 - runs.lo) / 128 : 0;
    const int end = (runs.ns + (pos0 + rb - runs.lo) / kWfSeg) / 2 + 1;
    jb[x] = max(j0, skip);
    je[x] = ra < c.q_len ? min(j1, end) : 0;
    if (kPaired) {
      jb[x] = j0 + x;
      je[x] = j1;
    }
    if (je[x] <= jb[x]) jb[x] = je[x] = 0;
  }
  constexpr int kStep = kPaired ? 2 : 1;  // x takes the key tiles jb[x], jb[x] + kStep, ... < je[x]
  auto takes = [&](int x, int j) { return j >= jb[x] && j < je[x] && (!kPaired || ((j - jb[x]) & 1) == 0); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kWfSlots; ++s) mbar_init(&S.full[s], 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&S.step[x], 1);
      mbar_init(&S.q_full[x], 1);
      mbar_init(&S.s_full[x], 1);
      mbar_init(&S.p_full[x][0], 4);
      mbar_init(&S.p_full[x][1], 4);
    }
    mbar_init(&S.mma_done, 1);
    mbar_init(&S.tail, 1);
    S.abort = 0;
    fence_mbar_init();
  }
  if (warp == kWfMmaWarp) {
    tmem_alloc(&S.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;

  if (warp >= kWfTmaWarp) {  // the third warpgroup, one instruction for its four warps
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWfOtherRegs));
  if (warp > kWfMmaWarp) return;
  if (warp == kWfTmaWarp) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      for (int x = 0; x < (kPaired ? 1 : 2); ++x)
        if (je[x] > jb[x]) {
          mbar_arrive_expect_tx(&S.q_full[x], kWfTileBytes);
          for (int h = 0; h < 2; ++h)
            tma_load_3d(qs + x * kWfTileBytes + h * kWfHalf, &tm_q, &S.q_full[x], 64 * h, g << p.g_log2,
                        b * w.Lq + r0 + x * tt);
        }
    }
    int slot = 0, issued = 0;
    bool tail_used = false, stop = false;
    for (int j = j0; j < j1 && !stop; ++j)
      for (int kv = 0; kv < 2; ++kv) {
        // Step s (counted from the one before the first tile) reads items 2s - 1 and 2s, whose slots
        // items 2s + 4 and 2s + 5 take.  Step s + 2 waits for item 2s + 4, so the barrier of step s
        // (one of two) is never a phase further.
        if (issued >= 4 && issued % 2 == 0) {
          const int s = (issued - 4) / 2;
          mbar_wait_short(&S.step[s & 1], static_cast<uint32_t>(s >> 1) & 1u, &S.abort);
        }
        stop = __any_sync(0xffffffffu, S.abort != 0);
        if (stop) break;
        unsigned char* dst = ring + slot * kWfTileBytes;
        // rows of V past the cache's end may hold anything (0 x NaN is not 0): such a tile lands on
        // a barrier of its own and is cleaned before it is handed on
        int clean[2];
        bool any = false;
        for (int s = 0; s < 2; ++s) {
          const int seg = 2 * j + s;
          clean[s] = seg < runs.ns + runs.nw && !runs.is_sink(seg) ? c.kv_len - runs.first_key(seg) : kWfSeg;
          any |= kv == 1 && w.kv_lens != nullptr && clean[s] < kWfSeg;
        }
        if (lane == 0) {
          uint64_t* bar = any ? &S.tail : &S.full[slot];
          mbar_arrive_expect_tx(bar, kWfTileBytes);
          for (int s = 0; s < 2; ++s) {
            const int seg = 2 * j + s;
            const bool pad = seg >= runs.ns + runs.nw;  // an odd count: rows past the tensor, zero-filled
            const CUtensorMap* m = runs.is_sink(seg) ? (kv ? &tm_vs : &tm_ks) : (kv ? &tm_v : &tm_k);
            const int key = pad ? w.Lmax : runs.first_key(seg);
            for (int h = 0; h < 2; ++h)
              tma_load_3d(dst + h * kWfHalf + s * (kWfSeg * 128), m, bar, 64 * h, key, bg);
          }
        }
        ++issued;
        if (any) {
          tail_used = true;
          if (mbar_wait_short(&S.tail, 0, &S.abort))
            for (int s = 0; s < 2; ++s)
              for (int i = max(clean[s], 0) * 8 + lane; i < kWfSeg * 8; i += 32)
                for (int h = 0; h < 2; ++h)
                  *reinterpret_cast<uint4*>(dst + h * kWfHalf + s * (kWfSeg * 128) + i * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.full[slot]);
        }
        __syncwarp();
        if (++slot == kWfSlots) slot = 0;
      }
    if (lane == 0) {  // every copy this thread issued lands before the CTA ends
      for (int x = 0; x < (kPaired ? 1 : 2); ++x)
        if (je[x] > jb[x]) mbar_wait_drain(&S.q_full[x], 0);
      if (tail_used) mbar_wait_drain(&S.tail, 0);
      drain_ring(S.full, issued);
    }
    return;
  }

  {
    // -------------------------------------------------------------------- MMA issuer
    // The tensor pipe holds about four products (256 cycles) beyond the one it runs, a completed
    // barrier takes this warp ~120 cycles to see, and a wait for an operand that is there already
    // must not let the pipe run empty: each barrier is probed (without blocking) before the batch
    // of products that precedes its use.
    const bool lead = elect_one();
    const uint64_t qd = desc_k_sw128(smem_u32(qs)), kd = desc_k_sw128(smem_u32(ring));
    const uint64_t vd = desc_mn_sw128(smem_u32(ring), kWfHalf, 1024);
    bool ok = true;
    auto need = [&](bool seen, uint64_t* bar, uint32_t parity) {
      if (ok && !seen) ok = mbar_wait_short(bar, parity, &S.abort);
    };
    for (int x = 0; x < (kPaired ? 1 : 2); ++x)
      if (je[x] > jb[x]) need(false, &S.q_full[x], 0);
    int slot = 0;               // ring position of the next item (K of a tile, then its V)
    uint32_t phase = 0;
    auto advance = [&] {
      if (++slot == kWfSlots) {
        slot = 0;
        phase ^= 1u;
      }
    };
    uint32_t np0 = 0, np1 = 0;  // probability tiles consumed
    // O_x += P_x V (with P number np of x) and S_x = Q_x K of the next tile.
    auto run_tile = [&](int x, uint32_t& np, bool pv, bool qk, bool p_seen, uint64_t v, uint64_t k, uint64_t* kbar,
                        uint32_t kphase, bool k_known) {
      bool k_seen = k_known;
      if (pv) {
        need(p_seen, &S.p_full[x][0], np & 1u);
        const bool h1 = mbar_test(&S.p_full[x][1], np & 1u);
        tc_fence_after();
        if (ok && lead) umma_pv_half(tmem + kWfColO + 128u * x, tmem + 128u * x, v, np > 0);
        need(h1, &S.p_full[x][1], np & 1u);
        if (qk && !k_known) k_seen = mbar_test(kbar, kphase);
        tc_fence_after();
        if (ok && lead) umma_pv_half(tmem + kWfColO + 128u * x, tmem + 128u * x + 32u, v + 512u, true);
        ++np;
      }
      if (qk) {
        need(k_seen, kbar, kphase);
        if (ok && lead) {
          umma_rows(tmem + 128u * x, qd + (kPaired ? 0 : x) * (kWfTileBytes >> 4), k);
          umma_commit(&S.s_full[x]);
        }
      }
    };
    for (int j = j0 - 1; j < j1 && ok; ++j) {
      const bool pv0 = takes(0, j), qk0 = takes(0, j + 1), pv1 = takes(1, j), qk1 = takes(1, j + 1);
      const bool p0 = !kPaired && pv0 && mbar_test(&S.p_full[0][0], np0 & 1u);
      uint64_t v = vd, k = kd;
      if (j >= j0) {
        need(false, &S.full[slot], phase);  // V came with the K read a step ago: seen at once
        v += static_cast<uint32_t>(slot) * (kWfTileBytes >> 4);
        advance();
      }
      uint64_t* const kbar = &S.full[slot];
      const uint32_t kphase = phase;
      const bool has_k = j + 1 < j1;
      if (has_k) {
        k += static_cast<uint32_t>(slot) * (kWfTileBytes >> 4);
        advance();
      }
      if (kPaired) {  // the next tile's scores first: they go to the other buffer
        if (qk0) run_tile(0, np0, false, true, false, v, k, kbar, kphase, false);
        if (qk1) run_tile(1, np1, false, true, false, v, k, kbar, kphase, false);
        if (pv0) run_tile(0, np0, true, false, false, v, k, kbar, kphase, true);
        if (pv1) run_tile(1, np1, true, false, false, v, k, kbar, kphase, true);
      } else {
        run_tile(0, np0, pv0, qk0, p0, v, k, kbar, kphase, false);
        const bool p1 = pv1 && mbar_test(&S.p_full[1][0], np1 & 1u);
        run_tile(1, np1, pv1, qk1, p1, v, k, kbar, kphase, qk0);
      }
      if (ok && has_k && !qk0 && !qk1) need(false, kbar, kphase);  // its slot is released below all the same
      if (ok && lead) umma_commit(&S.step[(j + 1 - j0) & 1]);  // V of tile j and K of tile j + 1 have been read
      __syncwarp();
    }
    if (lead) umma_commit(&S.mma_done);
    __syncwarp();
    named_bar_sync(1, 32 * 9);  // the softmax warps have used TMEM for the last time
    if (lane == 0) mbar_wait_drain(&S.mma_done, 0);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
    return;
  }
  }

  // ------------------------------------------------------------------- softmax warpgroups
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWfSoftRegs));
  const int x = warp >> 2;
  const int row = threadIdx.x & 127;
  const int rx = kPaired ? r0 : r0 + x * tt;  // first token of the warpgroup's rows
  const int r = rx + (row >> p.g_log2);
  const bool valid = r < c.q_len;
  const bool warp_live = __any_sync(0xffffffffu, valid);
  const int t = pos0 + min(r, c.q_len - 1);
  const int tx_min = pos0 + rx, tx_max = pos0 + min(rx + tt, c.q_len) - 1;
  const uint32_t tl = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
  const uint32_t ts = tl + 128u * x, to = tl + kWfColO + 128u * x;
  const float sl2 = w.scale_log2;
  float m2 = -INFINITY, sum = 0.f;  // reference maximum (scaled, base 2) and sum of the row
  uint32_t n = 0;
  for (int j = jb[x]; j < je[x]; j += kStep, ++n) {
    mbar_wait_short(&S.s_full[x], n & 1u, &S.abort);  // after a timeout the loop runs on: its loads are collective
    tc_fence_after();
    if (warp_live) {
      uint32_t v[128];
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_ld32_nowait(ts + 32 * q, v + 32 * q);
      tmem_wait_ld_tied(v);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int seg = 2 * j + s, u0 = runs.first_key(seg);
        const bool full = u0 + kWfSeg - 1 <= tx_min &&
                          (runs.is_sink(seg) ? u0 + kWfSeg <= w.n_sink
                                             : (u0 > tx_max - w.window || u0 + kWfSeg <= w.n_sink));
        if (!full) {
          const uint64_t mk = runs.mask(seg, t, w.window);
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (!((mk >> i) & 1ull)) v[64 * s + i] = 0xff800000u;  // -inf
        }
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < 128; i += 4)
#pragma unroll
        for (int q = 0; q < 4; ++q) mx[q] = fmaxf(mx[q], __uint_as_float(v[i + q]));
      const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
      // the row's reference moves when its maximum is 2^8 above it (from -inf: always)
      if (__any_sync(0xffffffffu, mt > m2 + 8.f)) {
        const float mn = fmaxf(m2, mt);
        const float f = mn == -INFINITY ? 1.f : ex2(m2 - mn);
        m2 = mn;
        sum *= f;
        if (n > 0) {  // the last product into O came before this S: both are complete
#pragma unroll 1
          for (int q = 0; q < 8; ++q) {
            uint32_t o16[16];
            tmem_ld16(to + 16 * q, o16);
#pragma unroll
            for (int i = 0; i < 16; ++i) o16[i] = __float_as_uint(__uint_as_float(o16[i]) * f);
            tmem_st16(to + 16 * q, o16);
          }
        }
      }
      const float mr = m2 == -INFINITY ? 0.f : -m2;  // nothing visible yet: every exponential is 0
      const uint64_t sl2p = f2(sl2, sl2), mr2 = f2(mr, mr);
      uint64_t sm[2] = {0, 0};
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint64_t e = ex2_pair(
              fma2(f2(__uint_as_float(v[32 * h + 2 * i]), __uint_as_float(v[32 * h + 2 * i + 1])), sl2p, mr2));
          sm[i & 1] = add2(sm[i & 1], e);
          pk[i] = pack_pair(e);
        }
        tmem_st16_nowait(ts + 16 * h, pk);
        if (h & 1) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.p_full[x][h >> 1]);
        }
      }
      float s0, s1;
      unf2(add2(sm[0], sm[1]), s0, s1);
      sum += s0 + s1;
    } else {  // no row of this warp exists: its lanes of P and O are never read
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&S.p_full[x][0]);
        mbar_arrive(&S.p_full[x][1]);
      }
    }
  }
  mbar_wait_short(&S.mma_done, 0, &S.abort);
  tc_fence_after();
  // paired: the second warpgroup leaves its state in the ring (every product has read it), as
  // [16-byte column][row] so that a warp's accesses are consecutive
  float4* joint = reinterpret_cast<float4*>(ring);
  float2* joint_ms = reinterpret_cast<float2*>(joint + 32 * 128);
  float f_own = 1.f, f_other = 0.f;
  if (kPaired) {
    if (x == 1) {
      joint_ms[row] = make_float2(n > 0 ? m2 : -INFINITY, sum);
      if (warp_live && n > 0)
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          uint32_t v[32];
          tmem_ld32(to + 32 * q, v);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            joint[(8 * q + i) * 128 + row] = make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                                         __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]));
        }
    }
    named_bar_sync(2, 256);
    if (x == 0) {
      const float2 o = joint_ms[row];
      const float mn = fmaxf(m2, o.x);
      f_own = m2 == -INFINITY ? 0.f : ex2(m2 - mn);
      f_other = o.x == -INFINITY ? 0.f : ex2(o.x - mn);  // 0 also where that state has no tile
      sum = sum * f_own + (f_other > 0.f ? o.y * f_other : 0.f);
      m2 = mn;
    }
  }
  if (warp_live && (!kPaired || x == 0)) {
    const int h = (g << p.g_log2) + (row & ((1 << p.g_log2) - 1));
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    const float lse2 = sum > 0.f ? m2 + lg2(sum) : -INFINITY;
    const size_t orow = (static_cast<size_t>(b) * w.Lq + r) * w.Hq + h;
    const size_t prow = static_cast<size_t>(blockIdx.x) * p.rows + x * 128 + row;
    if (valid) {
      if (p.n_splits > 1)
        p.part_lse[prow] = lse2;
      else if (w.lse)
        w.lse[(static_cast<size_t>(b) * w.Hq + h) * w.Lq + r] = lse2 * 0.6931471805599453f;
    }
    const float inv_own = inv * f_own, inv_other = inv * f_other;
    if (n > 0)
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        uint32_t v[32];
        tmem_ld32(to + 32 * q, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * inv_own);
        if (kPaired && inv_other > 0.f)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 o = joint[(8 * q + i) * 128 + row];
            v[4 * i] = __float_as_uint(fmaf(o.x, inv_other, __uint_as_float(v[4 * i])));
            v[4 * i + 1] = __float_as_uint(fmaf(o.y, inv_other, __uint_as_float(v[4 * i + 1])));
            v[4 * i + 2] = __float_as_uint(fmaf(o.z, inv_other, __uint_as_float(v[4 * i + 2])));
            v[4 * i + 3] = __float_as_uint(fmaf(o.w, inv_other, __uint_as_float(v[4 * i + 3])));
          }
        if (valid && p.n_splits > 1) {
          uint4* dst = reinterpret_cast<uint4*>(p.part_o + prow * kHeadDim + 32 * q);
#pragma unroll
          for (int i = 0; i < 8; ++i) dst[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        } else if (valid) {
          uint4* dst = reinterpret_cast<uint4*>(w.o + orow * kHeadDim + 32 * q);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              u[e] = pack_bf16(__uint_as_float(v[8 * i + 2 * e]), __uint_as_float(v[8 * i + 2 * e + 1]));
            dst[i] = make_uint4(u[0], u[1], u[2], u[3]);
          }
        }
        __syncwarp();
      }
  }
  tc_fence_before();
  named_bar_sync(1, 32 * 9);  // TMEM may be freed
}

// Joins the key splits of a row: one warp per (sequence, query row, q-head).  The weights are
// 2^(lse_s - lse); splits without a visible key (lse -inf) are not read.
__global__ void __launch_bounds__(256) window_merge_kernel(const WinTcParams p) {
  const WinParams& w = p.w;
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  grid_dependency_wait();
  if (row >= static_cast<long long>(w.B) * w.Lq * w.Hq) return;
  const int h = static_cast<int>(row % w.Hq), r = static_cast<int>(row / w.Hq % w.Lq);
  const int b = static_cast<int>(row / w.Hq / w.Lq);
  const ChunkLens c = chunk_lens(w.q_lens, w.kv_lens, b, w.Lq, w.Lmax);
  if (r >= c.q_len) return;
  const int ct = p.rows >> p.g_log2, tile = r / ct;
  const int bg = b * w.Hkv + (h >> p.g_log2);
  const size_t cta = (static_cast<size_t>(p.row_tiles - 1 - tile) * w.B * w.Hkv + bg) * p.n_splits;
  const size_t in = static_cast<size_t>(r - tile * ct) * w.G + (h & (w.G - 1));  // row of the CTA
  // lane = split (at most 32): every weight is known before the first row is read, so the reads
  // do not wait for one another
  const float l = lane < p.n_splits ? p.part_lse[(cta + lane) * p.rows + in] : -INFINITY;
  float mx = l;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
  const float e = ex2(l - mx);  // 0 for a split without a visible key: its row is not read
  float z = e;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int s = 0; s < p.n_splits; ++s) {
    const float es = __shfl_sync(0xffffffffu, e, s);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (es > 0.f) o = *(reinterpret_cast<const float4*>(p.part_o + ((cta + s) * p.rows + in) * kHeadDim) + lane);
    acc[0] = fmaf(es, o.x, acc[0]), acc[1] = fmaf(es, o.y, acc[1]);
    acc[2] = fmaf(es, o.z, acc[2]), acc[3] = fmaf(es, o.w, acc[3]);
  }
  const float inv = 1.f / z;
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] *= inv;
  store4(w.o + row * kHeadDim, lane, acc);
  if (w.lse && lane == 0) w.lse[(static_cast<size_t>(b) * w.Hq + h) * w.Lq + r] = (mx + lg2(z)) * 0.6931471805599453f;
}

}  // namespace infllmv2
