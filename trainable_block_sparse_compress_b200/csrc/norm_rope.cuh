// norm_rope.cuh -- per-head RMS norm of queries and keys with the position rotation in the
// same pass, from the projection's token rows to the attention's layouts, and its backward.
//
// For a head row x (128 values) of q or k at position t, with weights w:
//   r = 1 / sqrt(mean(x^2) + eps),  y = x r w,
//   (y_a, y_b) <- (y_a c_i - y_b s_i, y_a s_i + y_b c_i) for the pairs of the first rot dims.
// Backward, with g = R(-t) dy (the rotation is orthogonal up to the table's scale, and its
// transpose is the rotation by -t with the same scale):
//   d_w = sum over rows of g x r,   dx = r (g w) - x r^3 mean(g w x)
// (formed as r (g w - (x r) r mean(g w x)): r^3 leaves fp32's range before dx does).
// Everything is fp32 in registers, rounded once to bf16 on the way out.
//
// Both passes are bound by HBM: each head row is read once and written once (256 bytes each
// way).  A half-warp holds a row, a lane two runs of 4 values that are each other's rotation
// partners (rot / 2 apart, or adjacent for interleaved pairs), so a rotation needs no shuffle
// and 4 cosines and sines a lane; the norm is four shuffles.  A half-warp takes several heads
// of one token (all queries, or keys and values), so the token's row of the table and one
// weight vector stay in registers, with kNrRows rows in flight; the arithmetic is packed in
// pairs (f32x2), since with one value an instruction the issue slots, not HBM, would bound it.
// Measured on a 128K prompt, 32 / 2 heads, 2.48 GB: 453 us a call on changing inputs (0.83 of the
// measured copy bandwidth), 412 us (0.92) repeated on one; against that, 12 heads an item 442, six
// rows in flight at two CTAs an SM 526, one wave of CTAs (the short key and value items then leave
// their SMs early) 477 to 806.
// The backward copies a lane's values into its own slots of shared memory, kNrBwdRows rows ahead
// of the ones it works on: rows in flight cost no registers.  One wave of CTAs, dealt to the query
// and to the key and value heads by their bytes.  Measured, 2 x 8191 tokens, 453 MB: 94 us a call (0.73; 0.85
// at 65536 tokens); rows loaded into registers 112, as many CTAs for each chunk of heads 103, two
// rows ahead 100, eight rows with 12 warps an SM 120, one row's dependent chain at a time 94.
#pragma once
#include <type_traits>

#include "append.cuh"
#include "common.cuh"

namespace infllmv2 {

constexpr int kNrThreads = 256;
constexpr int kNrWarps = kNrThreads / 32;
constexpr int kNrRows = 4;       // head rows in flight per half-warp, forward
constexpr int kNrBwdRows = 4;    // backward: rows of a batch
constexpr int kNrBwdCtas = 2;    // CTAs an SM

struct NormRopeParams {
  const __nv_bfloat16 *q, *k, *v;        // token rows
  long long q_stride, k_stride, v_stride;  // elements between token rows
  const void *qw, *kw;                   // [128] or NULL
  const float* table;                    // [table_rows, rot]
  const int32_t *starts, *q_lens;
  __nv_bfloat16 *q_out, *k_out, *v_out;  // forward outputs / backward: input gradients (token rows)
  int32_t* lens_out;
  const __nv_bfloat16 *dq, *dk, *dv;     // backward: gradients in the attention's layouts
  long long dq_stride, dk_stride, dv_stride;
  float* part;                           // backward: [CTA][128] partial d_w
  int B, Lq, Hq, Hkv, Lout, at_position, weights_fp32, table_rows, rot;
  int heads, q_chunks, kv_chunks;        // heads of one chunk, chunks of a token
  int q_ctas, kv_ctas;                   // CTAs of a query chunk, of a key and value chunk
  float eps;
};

__device__ __forceinline__ uint64_t swap2(uint64_t v) {
  float a, b;
  unf2(v, a, b);
  return f2(b, a);
}

// A lane's 8 values of a row: pairs 0, 1 are its first run of 4, pairs 2, 3 the second.
struct Row8 {
  uint64_t v[4];
};
struct Raw8 {
  uint2 a, b;
};

__device__ __forceinline__ uint64_t unpack_pair(uint32_t u) {
  return f2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ Row8 unpack8(const Raw8& r) {
  return {{unpack_pair(r.a.x), unpack_pair(r.a.y), unpack_pair(r.b.x), unpack_pair(r.b.y)}};
}
__device__ __forceinline__ Raw8 pack8(const Row8& y) {
  return {make_uint2(pack_pair(y.v[0]), pack_pair(y.v[1])), make_uint2(pack_pair(y.v[2]), pack_pair(y.v[3]))};
}

// First elements of the lane's two runs.
template <bool kInterleaved>
__device__ __forceinline__ void lane_runs(int rot, int l, int& a, int& b) {
  if (kInterleaved) {
    a = 8 * l, b = 8 * l + 4;
  } else if (l < rot / 8) {
    a = 4 * l, b = rot / 2 + 4 * l;
  } else {  // past the rotated dimensions
    a = 8 * l, b = 8 * l + 4;
  }
}

__device__ __forceinline__ Raw8 load_row(const __nv_bfloat16* row, int a, int b) {
  return {*reinterpret_cast<const uint2*>(row + a), *reinterpret_cast<const uint2*>(row + b)};
}
__device__ __forceinline__ void store_row(__nv_bfloat16* row, int a, int b, const Raw8& r) {
  *reinterpret_cast<uint2*>(row + a) = r.a;
  *reinterpret_cast<uint2*>(row + b) = r.b;
}

__device__ __forceinline__ Row8 load_weights(const void* w, int fp32, int a, int b) {
  if (w == nullptr) {
    const uint64_t one = f2(1.f, 1.f);
    return {{one, one, one, one}};
  }
  if (!fp32) return unpack8(load_row(static_cast<const __nv_bfloat16*>(w), a, b));
  const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + a);
  const float4 y = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + b);
  return {{f2(x.x, x.y), f2(x.z, x.w), f2(y.x, y.y), f2(y.z, y.w)}};
}

// Cosines and sines of the lane's four rotation pairs at table row t (1 and 0 past rot).
__device__ __forceinline__ void load_angles(const float* table, int rot, int t, int l, float (&c)[4], float (&s)[4]) {
  if (8 * l >= rot) return;
  const float* row = table + static_cast<size_t>(t) * rot + 4 * l;
  const float4 x = *reinterpret_cast<const float4*>(row), y = *reinterpret_cast<const float4*>(row + rot / 2);
  c[0] = x.x, c[1] = x.y, c[2] = x.z, c[3] = x.w;
  s[0] = y.x, s[1] = y.y, s[2] = y.z, s[3] = y.w;
}

// Rotation by the lane's angles, in packed pairs.  Pairs rot / 2 apart: (a, b) = (a c - b s,
// a s + b c) run by run.  Interleaved: (x0, x1) = (x0, x1) (c, c) + (x1, x0) (-s, s).
template <bool kInterleaved>
struct Turn {
  uint64_t c[kInterleaved ? 4 : 2], s[kInterleaved ? 4 : 2];
  __device__ __forceinline__ void set(const float (&cs)[4], const float (&sn)[4], float sign) {
    if (kInterleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = f2(cs[i], cs[i]), s[i] = f2(-sign * sn[i], sign * sn[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        c[i] = f2(cs[2 * i], cs[2 * i + 1]), s[i] = f2(sign * sn[2 * i], sign * sn[2 * i + 1]);
    }
  }
  __device__ __forceinline__ void apply(Row8& y) const {
    if (kInterleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y.v[i] = fma2(y.v[i], c[i], mul2(swap2(y.v[i]), s[i]));
    } else {
      const uint64_t neg = f2(-1.f, -1.f);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint64_t a = y.v[i], b = y.v[i + 2];
        y.v[i] = fma2(a, c[i], mul2(mul2(b, s[i]), neg));
        y.v[i + 2] = fma2(a, s[i], mul2(b, c[i]));
      }
    }
  }
};

__device__ __forceinline__ float half_sum(float x) {
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d, 16);
  return x;
}
__device__ __forceinline__ float dot8(const Row8& x, const Row8& y) {
  float a, b;
  unf2(fma2(x.v[0], y.v[0], mul2(x.v[1], y.v[1])), a, b);
  float c, d;
  unf2(fma2(x.v[2], y.v[2], mul2(x.v[3], y.v[3])), c, d);
  return (a + b) + (c + d);
}

// A half-warp's token: sequence b, row r of it, first position t0; live unless the row is
// padding or its sequence leaves the table or the caches (then all its rows are left alone).
struct NormRopeToken {
  unsigned tok;
  int b, r, t0, n;
  bool in, fits, live;
  __device__ __forceinline__ NormRopeToken(const NormRopeParams& p, unsigned token, unsigned tokens) {
    in = token < tokens;
    tok = in ? token : 0;
    b = static_cast<int>(tok / static_cast<unsigned>(p.Lq));
    r = static_cast<int>(tok - static_cast<unsigned>(b) * static_cast<unsigned>(p.Lq));
    t0 = p.starts ? p.starts[b] : 0;
    n = p.q_lens ? min(max(p.q_lens[b], 0), p.Lq) : p.Lq;
    const long long end = static_cast<long long>(t0) + n;
    fits = t0 >= 0 && end <= p.table_rows && (!p.at_position || end <= p.Lout);
    live = in && fits && r < n;
  }
};

// A CTA's chunk of heads (p.heads query heads, or p.heads of the Hkv key and then Hkv value heads)
// and its place among the chunk's CTAs.  kEven: as many CTAs for every chunk, the chunks of a
// token side by side; else the query chunks' CTAs come first.
template <bool kEven>
struct NormRopeChunk {
  int chunk, h0, h1;
  unsigned x, ctas;
  bool isq;
  __device__ __forceinline__ explicit NormRopeChunk(const NormRopeParams& p) {
    if (kEven) {
      const unsigned n = p.q_chunks + p.kv_chunks;
      chunk = static_cast<int>(blockIdx.x % n);
      x = blockIdx.x / n;
      ctas = gridDim.x / n;
      isq = chunk < p.q_chunks;
    } else {
      const unsigned i = blockIdx.x, q = p.q_chunks * p.q_ctas, kc = p.kv_chunks, qc = p.q_chunks;
      isq = i < q;
      chunk = static_cast<int>(isq ? i % qc : qc + (i - q) % kc);
      x = isq ? i / qc : (i - q) / kc;
      ctas = isq ? p.q_ctas : p.kv_ctas;
    }
    h0 = (isq ? chunk : chunk - p.q_chunks) * p.heads;
    h1 = min(h0 + p.heads, isq ? p.Hq : 2 * p.Hkv);
  }
  // the CTA's row of the partial weight gradients: the query chunks', then the key and value chunks'
  __device__ __forceinline__ int part(const NormRopeParams& p) const {
    return static_cast<int>((isq ? chunk * ctas : p.q_chunks * p.q_ctas + (chunk - p.q_chunks) * ctas) + x);
  }
};

// A warp per two tokens, grid-stride over the chunk's CTAs.
template <bool kInterleaved>
__global__ void __launch_bounds__(kNrThreads, 4) qk_norm_rope_kernel(const NormRopeParams p) {
  grid_dependency_wait();
  const int l = threadIdx.x & 15;
  const unsigned tokens = static_cast<unsigned>(p.B) * static_cast<unsigned>(p.Lq);
  const NormRopeChunk<true> ch(p);
  const bool isq = ch.isq;
  const int h0 = ch.h0, h1 = ch.h1;
  int ra, rb;
  lane_runs<kInterleaved>(p.rot, l, ra, rb);
  const Row8 w = load_weights(isq ? p.qw : p.kw, p.weights_fp32, ra, rb);
  for (unsigned pair = ch.x * kNrWarps + (threadIdx.x >> 5); pair < (tokens + 1) / 2; pair += ch.ctas * kNrWarps) {
    const NormRopeToken k(p, 2 * pair + ((threadIdx.x >> 4) & 1), tokens);
    if (k.in && k.r == 0 && ch.chunk == 0 && l == 0) {
      if (!k.fits) atomicOr(&g_device_error, kDevErrCacheFull);
      if (p.lens_out) p.lens_out[k.b] = k.fits ? k.t0 + k.n : k.t0;
    }
    float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
    if (k.live) load_angles(p.table, p.rot, k.t0 + k.r, l, c, s);
    const __nv_bfloat16* q = p.q + k.tok * p.q_stride;
    const __nv_bfloat16* ks = p.k + k.tok * p.k_stride;
    const __nv_bfloat16* vs = p.v + k.tok * p.v_stride - p.Hkv * kHeadDim;
    __nv_bfloat16* qo = p.q_out + static_cast<size_t>(k.tok) * p.Hq * kHeadDim;
    const size_t head = static_cast<size_t>(p.Lout) * kHeadDim;
    const size_t ko = static_cast<size_t>(k.b) * p.Hkv * head + static_cast<size_t>(p.at_position ? k.t0 + k.r : k.r) * kHeadDim;
    for (int hb = h0; hb < h1; hb += kNrRows) {
      Raw8 raw[kNrRows];
#pragma unroll
      for (int u = 0; u < kNrRows; ++u) {
        const int h = hb + u;
        raw[u] = {make_uint2(0, 0), make_uint2(0, 0)};
        if (k.live && h < h1) raw[u] = load_row((isq ? q : h < p.Hkv ? ks : vs) + h * kHeadDim, ra, rb);
      }
      Turn<kInterleaved> turn;
      turn.set(c, s, 1.f);
#pragma unroll
      for (int u = 0; u < kNrRows; ++u) {
        const int h = hb + u;
        if (h >= h1) break;  // the same for the whole CTA
        Row8 y = unpack8(raw[u]);
        const float rs = rsqrtf(half_sum(dot8(y, y)) * (1.f / kHeadDim) + p.eps);
        const uint64_t r2 = f2(rs, rs);
#pragma unroll
        for (int i = 0; i < 4; ++i) y.v[i] = mul2(mul2(y.v[i], r2), w.v[i]);
        turn.apply(y);
        if (!k.live) continue;
        if (isq)
          store_row(qo + h * kHeadDim, ra, rb, pack8(y));
        else if (h < p.Hkv)
          store_row(p.k_out + ko + h * head, ra, rb, pack8(y));
        else
          store_row(p.v_out + ko + (h - p.Hkv) * head, ra, rb, raw[u]);
      }
    }
  }
}

// Asynchronous copy of a lane's N bytes into its own slot of shared memory; zeros unless `live`.
template <int N>
__device__ __forceinline__ void copy_async(void* dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(src), "n"(N), "r"(live ? N : 0)
               : "memory");
}

// A warp's buffers of the backward: the rows of two batches of heads and the angles of
// two tokens, a lane's values in the lane's own slots (no conflicts, nothing to synchronise).
struct NrBwdWarp {
  uint2 x[2][kNrBwdRows][2][32], g[2][kNrBwdRows][2][32];
  float4 cs[2][2][32];
};
constexpr size_t kNrBwdSmem = kNrWarps * sizeof(NrBwdWarp);
static_assert(sizeof(NrBwdWarp) >= 2 * kHeadDim * sizeof(float), "the half-warps' weight gradients");

// The backward over the same chunks: input gradients, and one row of partial weight gradients
// per CTA (its half-warps' sums added in a fixed order).  The next batch of heads (or the next
// token's first) is copied into shared memory while one is worked on.
template <bool kInterleaved>
__global__ void __launch_bounds__(kNrThreads, kNrBwdCtas) qk_norm_rope_bwd_kernel(const NormRopeParams p) {
  extern __shared__ __align__(16) unsigned char nr_smem[];
  const int l = threadIdx.x & 15, lane = threadIdx.x & 31;
  NrBwdWarp& S = reinterpret_cast<NrBwdWarp*>(nr_smem)[threadIdx.x >> 5];
  const unsigned tokens = static_cast<unsigned>(p.B) * static_cast<unsigned>(p.Lq), pairs = (tokens + 1) / 2;
  const NormRopeChunk<false> ch(p);
  const bool isq = ch.isq;
  // the key and value heads are dealt to their chunks in turn: each chunk has its share of both
  const int hs = isq ? 1 : p.kv_chunks, h0 = isq ? ch.h0 : ch.chunk - p.q_chunks, h1 = isq ? ch.h1 : 2 * p.Hkv;
  const int hn = isq ? h1 : p.Hkv;  // heads with a norm
  int ra, rb;
  lane_runs<kInterleaved>(p.rot, l, ra, rb);
  const Row8 w = load_weights(isq ? p.qw : p.kw, p.weights_fp32, ra, rb);
  const size_t head = static_cast<size_t>(p.Lq) * kHeadDim;
  Row8 acc = {{0, 0, 0, 0}};

  auto fetch_rows = [&](const NormRopeToken& k, int hb, int st) {
    const __nv_bfloat16* x0 = isq ? p.q + k.tok * p.q_stride : p.k + k.tok * p.k_stride;
    const __nv_bfloat16* gq = p.dq + static_cast<size_t>(k.tok) * p.Hq * kHeadDim;
    const size_t go = static_cast<size_t>(k.b) * p.Hkv * head + static_cast<size_t>(k.r) * kHeadDim;
#pragma unroll
    for (int u = 0; u < kNrBwdRows; ++u) {
      const int h = hb + u * hs;
      if (h >= h1) break;  // the same for the whole CTA
      if (isq || h < p.Hkv) {
        const __nv_bfloat16* x = x0 + h * kHeadDim;
        copy_async<8>(&S.x[st][u][0][lane], x + ra, k.live);
        copy_async<8>(&S.x[st][u][1][lane], x + rb, k.live);
      }
      const __nv_bfloat16* g = isq ? gq + h * kHeadDim : h < p.Hkv ? p.dk + go + h * head : p.dv + go + (h - p.Hkv) * head;
      copy_async<8>(&S.g[st][u][0][lane], g + ra, k.live);
      copy_async<8>(&S.g[st][u][1][lane], g + rb, k.live);
    }
  };
  auto fetch_token = [&](unsigned pair, int slot, int st) {
    const NormRopeToken k(p, 2 * pair + ((threadIdx.x >> 4) & 1), tokens);
    if (k.in && !k.fits && k.r == 0 && ch.chunk == 0 && l == 0) atomicOr(&g_device_error, kDevErrCacheFull);
    if (8 * l < p.rot) {
      const float* row = p.table + static_cast<size_t>(k.live ? k.t0 + k.r : 0) * p.rot + 4 * l;
      copy_async<16>(&S.cs[slot][0][lane], row, k.live);
      copy_async<16>(&S.cs[slot][1][lane], row + p.rot / 2, k.live);
    }
    fetch_rows(k, h0, st);
    return k;
  };

  // N rows at once: a row's chain of dependent instructions is longer than its share of the memory's time
  auto work = [&](auto rows, const NormRopeToken& k, const Turn<kInterleaved>& back, int h, int st, int u) {
    constexpr int N = decltype(rows)::value;
    Row8 x[N], g[N], gw[N];
    float ss[N], dot[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      x[j] = unpack8({S.x[st][u + j][0][lane], S.x[st][u + j][1][lane]});
      g[j] = unpack8({S.g[st][u + j][0][lane], S.g[st][u + j][1][lane]});
      back.apply(g[j]);
#pragma unroll
      for (int i = 0; i < 4; ++i) gw[j].v[i] = mul2(g[j].v[i], w.v[i]);
      ss[j] = dot8(x[j], x[j]), dot[j] = dot8(gw[j], x[j]);
    }
#pragma unroll
    for (int d = 8; d > 0; d >>= 1)
#pragma unroll
      for (int j = 0; j < N; ++j) {
        ss[j] += __shfl_xor_sync(0xffffffffu, ss[j], d, 16);
        dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], d, 16);
      }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float rs = rsqrtf(ss[j] * (1.f / kHeadDim) + p.eps);
      // dx = r (g w - (x r) r mean(g w x)): no power of r, which for a tiny row and eps leaves fp32's range
      const float t = -rs * dot[j] * (1.f / kHeadDim);
      const uint64_t r2 = f2(rs, rs), t2 = f2(t, t);
      Row8 dx;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t xr = mul2(x[j].v[i], r2);
        acc.v[i] = fma2(g[j].v[i], xr, acc.v[i]);  // rows that are not live are zeros
        dx.v[i] = mul2(fma2(xr, t2, gw[j].v[i]), r2);
      }
      const int hj = h + j * hs;
      if (k.live)
        store_row(isq ? p.q_out + k.tok * p.dq_stride + hj * kHeadDim : p.k_out + k.tok * p.dk_stride + hj * kHeadDim,
                  ra, rb, pack8(dx));
    }
  };

  unsigned pair = ch.x * kNrWarps + (threadIdx.x >> 5);
  const unsigned step = ch.ctas * kNrWarps;
  if (pair < pairs) {
    int slot = 0, st = 0;
    NormRopeToken k = fetch_token(pair, 0, 0);
    asm volatile("cp.async.commit_group;" ::: "memory");
    for (; pair < pairs; pair += step, slot ^= 1) {
      NormRopeToken next = k;
      Turn<kInterleaved> back;
      for (int hb = h0; hb < h1; hb += kNrBwdRows * hs, st ^= 1) {
        if (hb + kNrBwdRows * hs < h1)
          fetch_rows(k, hb + kNrBwdRows * hs, st ^ 1);
        else if (pairs - pair > step)
          next = fetch_token(pair + step, slot ^ 1, st ^ 1);
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        if (hb == h0) {
          float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
          if (8 * l < p.rot) {
            const float4 a = S.cs[slot][0][lane], b = S.cs[slot][1][lane];
            c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w;
            s[0] = b.x, s[1] = b.y, s[2] = b.z, s[3] = b.w;
          }
          back.set(c, s, -1.f);
        }
        // the branches are the same for the whole CTA
        for (int u = 0; u < kNrBwdRows;) {
          const int h = hb + u * hs;
          if (h >= h1) break;
          if (!isq && h >= p.Hkv) {
            if (k.live)
              store_row(p.v_out + k.tok * p.dv_stride + (h - p.Hkv) * kHeadDim, ra, rb,
                        {S.g[st][u][0][lane], S.g[st][u][1][lane]});
            ++u;
          } else if (u + 1 < kNrBwdRows && h + hs < hn) {
            work(std::integral_constant<int, 2>{}, k, back, h, st, u);
            u += 2;
          } else {
            work(std::integral_constant<int, 1>{}, k, back, h, st, u);
            ++u;
          }
        }
      }
      k = next;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  __syncthreads();
  float(*red)[kHeadDim] = reinterpret_cast<float(*)[kHeadDim]>(nr_smem);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int d = (i < 2 ? ra : rb) + 2 * (i & 1);
    unf2(acc.v[i], red[threadIdx.x >> 4][d], red[threadIdx.x >> 4][d + 1]);
  }
  __syncthreads();
  if (threadIdx.x < kHeadDim) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 2 * kNrWarps; ++i) a += red[i][threadIdx.x];
    p.part[static_cast<size_t>(ch.part(p)) * kHeadDim + threadIdx.x] = a;
  }
}

// d_qw (from the first q_parts rows of partials) and d_kw (from the other k_parts): grid 8, a
// CTA sums 32 of the 256 columns, 32 threads of a column over every 32nd row, then over the
// threads, in fp64 in a fixed order.
__global__ void __launch_bounds__(1024)
    qk_norm_rope_bwd_weights_kernel(const float* __restrict__ part, int q_parts, int k_parts,
                                    float* __restrict__ d_qw, float* __restrict__ d_kw) {
  __shared__ double red[32][33];
  grid_dependency_wait();
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, col = (blockIdx.x & 3) * 32 + x;
  const bool isq = blockIdx.x < 4;
  if (!isq) part += static_cast<size_t>(q_parts) * kHeadDim;
  const int parts = isq ? q_parts : k_parts;
  double a = 0.0;
  for (int i = y; i < parts; i += 32) a += part[static_cast<size_t>(i) * kHeadDim + col];
  red[y][x] = a;
  __syncthreads();
  if (y == 0) {
    for (int i = 1; i < 32; ++i) a += red[i][x];
    float* out = isq ? d_qw : d_kw;
    if (out) out[col] = static_cast<float>(a);
  }
}

// Table row t: scale cos(t f_i), scale sin(t f_i); the angle is formed and reduced in fp64.
__global__ void __launch_bounds__(256)
    rope_table_kernel(const float* __restrict__ inv_freq, int rot, int n, float scale, float* __restrict__ table) {
  const int h = rot / 2;
  const long long total = static_cast<long long>(n) * h;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const long long t = i / h;
    const int j = static_cast<int>(i - t * h);
    double sn, cs;
    sincos(static_cast<double>(t) * static_cast<double>(inv_freq[j]), &sn, &cs);
    table[t * rot + j] = static_cast<float>(cs * scale);
    table[t * rot + h + j] = static_cast<float>(sn * scale);
  }
}

}  // namespace infllmv2
