// norm_rope.cuh -- per-head RMS norm of queries and keys with the position rotation in the
// same pass, from the projection's token rows to the attention's layouts, and its backward.
//
// For a head row x (128 values) of q or k at position t, with weights w:
//   r = 1 / sqrt(mean(x^2) + eps),  y = x r w,
//   (y_a, y_b) <- (y_a c_i - y_b s_i, y_a s_i + y_b c_i) for the pairs of the first rot dims.
// Backward, with g = R(-t) dy (the rotation is orthogonal up to the table's scale, and its
// transpose is the rotation by -t with the same scale):
//   d_w = sum over rows of g x r,   dx = r (g w) - x r^3 mean(g w x).
// Everything is fp32 in registers, rounded once to bf16 on the way out.
//
// Both passes are bound by HBM: each head row is read once and written once (256 bytes each
// way).  A half-warp holds a row (a lane 8 values: one 16-byte load), so the norm is four
// shuffles and a rotation's partner is in the same lane (interleaved pairs) or one shuffle
// away (pairs rot / 2 apart; rot is a multiple of 16, so partners sit in the same place of
// two lanes).  A half-warp takes several heads of one token, so the token's row of the table
// and the weights are in registers for all of them, with four rows in flight.
#pragma once
#include "append.cuh"
#include "common.cuh"

namespace infllmv2 {

constexpr int kNrThreads = 256;
constexpr int kNrHalves = kNrThreads / 16;  // half-warps of a CTA
constexpr int kNrUnroll = 4;                // head rows in flight per half-warp
constexpr int kNrMaxParts = 1024;           // CTAs of the backward at most (rows of d_w partials)

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
  float* part;                           // backward: [grid][2][128] partial d_w
  int B, Lq, Hq, Hkv, Lout, at_position, weights_fp32, table_rows, rot;
  int heads_per_item, chunks;            // heads of one item, items of one token
  float eps;
};

struct Row8 {
  float v[8];
};

__device__ __forceinline__ Row8 unpack8(const uint4& u) {
  Row8 r;
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = __uint_as_float(w[i] << 16);
    r.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  return r;
}
__device__ __forceinline__ uint4 pack8(const Row8& r) {
  return make_uint4(pack_bf16(r.v[0], r.v[1]), pack_bf16(r.v[2], r.v[3]), pack_bf16(r.v[4], r.v[5]),
                    pack_bf16(r.v[6], r.v[7]));
}

__device__ __forceinline__ Row8 load_weights(const void* w, int fp32, int l) {
  Row8 r;
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = 1.f;
  } else if (fp32) {
    const float4 a = __ldg(static_cast<const float4*>(w) + 2 * l), b = __ldg(static_cast<const float4*>(w) + 2 * l + 1);
    r.v[0] = a.x, r.v[1] = a.y, r.v[2] = a.z, r.v[3] = a.w;
    r.v[4] = b.x, r.v[5] = b.y, r.v[6] = b.z, r.v[7] = b.w;
  } else {
    r = unpack8(__ldg(static_cast<const uint4*>(w) + l));
  }
  return r;
}

// This lane's cosines and sines of table row `t`: of its 8 dimensions (pairs rot / 2 apart)
// or of its 4 pairs (interleaved; the first four entries).
template <bool kInterleaved>
__device__ __forceinline__ void load_angles(const float* table, int rot, int t, int l, Row8& c, Row8& s) {
  const float* row = table + static_cast<size_t>(t) * rot;
  if (8 * l >= rot) return;
  if (kInterleaved) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(row + 4 * l));
    const float4 b = __ldg(reinterpret_cast<const float4*>(row + rot / 2 + 4 * l));
    c.v[0] = a.x, c.v[1] = a.y, c.v[2] = a.z, c.v[3] = a.w;
    s.v[0] = b.x, s.v[1] = b.y, s.v[2] = b.z, s.v[3] = b.w;
  } else {
    const int m = rot / 16, i = 8 * (l < m ? l : l - m);
    const float sg = l < m ? -1.f : 1.f;  // y_a takes -s y_b, y_b takes +s y_a
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(row + i + 4 * h));
      const float4 b = __ldg(reinterpret_cast<const float4*>(row + rot / 2 + i + 4 * h));
      c.v[4 * h] = a.x, c.v[4 * h + 1] = a.y, c.v[4 * h + 2] = a.z, c.v[4 * h + 3] = a.w;
      s.v[4 * h] = sg * b.x, s.v[4 * h + 1] = sg * b.y, s.v[4 * h + 2] = sg * b.z, s.v[4 * h + 3] = sg * b.w;
    }
  }
}

// Rotates this lane's 8 values by the angles (kBack: by their negatives).  Called by whole
// half-warps.
template <bool kInterleaved, bool kBack>
__device__ __forceinline__ void rotate(Row8& y, const Row8& c, const Row8& s, int rot, int l) {
  if (kInterleaved) {
    if (8 * l < rot) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = y.v[2 * i], b = y.v[2 * i + 1], sn = kBack ? -s.v[i] : s.v[i];
        y.v[2 * i] = fmaf(a, c.v[i], -b * sn);
        y.v[2 * i + 1] = fmaf(a, sn, b * c.v[i]);
      }
    }
  } else {
    const int m = rot / 16;
    const int src = l < m ? l + m : (l < 2 * m ? l - m : l);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float o = __shfl_sync(0xffffffffu, y.v[i], src, 16);
      if (l < 2 * m) y.v[i] = fmaf(y.v[i], c.v[i], o * (kBack ? -s.v[i] : s.v[i]));
    }
  }
}

__device__ __forceinline__ float half_sum(float x) {
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d, 16);
  return x;
}

// The item's sequence: its rows and first position; false (all its rows are left alone) when
// the rows leave the table or the caches.
__device__ __forceinline__ bool norm_rope_seq(const NormRopeParams& p, int b, int& n, int& t0) {
  t0 = p.starts ? p.starts[b] : 0;
  n = p.q_lens ? min(max(p.q_lens[b], 0), p.Lq) : p.Lq;
  const long long end = static_cast<long long>(t0) + n;
  return t0 >= 0 && end <= p.table_rows && (!p.at_position || end <= p.Lout);
}

// Grid-stride over (token, chunk of heads) items, one per half-warp; head h < Hq is a query
// head, then Hkv key heads, then Hkv value heads.
template <bool kInterleaved>
__global__ void __launch_bounds__(kNrThreads) qk_norm_rope_kernel(const NormRopeParams p) {
  grid_dependency_wait();
  const int l = threadIdx.x & 15;
  const long long items = static_cast<long long>(p.B) * p.Lq * p.chunks;
  const Row8 wq = load_weights(p.qw, p.weights_fp32, l), wk = load_weights(p.kw, p.weights_fp32, l);
  const int H = p.Hq + 2 * p.Hkv;
  const long long stride = static_cast<long long>(gridDim.x) * kNrHalves;
  // both halves of a warp run the same number of rounds: shuffles name the whole warp
  const long long first = static_cast<long long>(blockIdx.x) * kNrHalves + (threadIdx.x >> 5) * 2;
  for (long long base = first; base < items; base += stride) {
    const long long it = base + ((threadIdx.x >> 4) & 1);
    const bool in = it < items;
    const long long tok = in ? it / p.chunks : 0;
    const int b = static_cast<int>(tok / p.Lq), r = static_cast<int>(tok - static_cast<long long>(b) * p.Lq);
    const int h0 = in ? static_cast<int>(it - tok * p.chunks) * p.heads_per_item : 0;
    int n, t0;
    const bool fits = norm_rope_seq(p, b, n, t0);
    if (in && r == 0 && h0 == 0 && l == 0) {
      if (!fits) atomicOr(&g_device_error, kDevErrCacheFull);
      if (p.lens_out) p.lens_out[b] = fits ? t0 + n : t0;
    }
    const bool live = in && fits && r < n;
    Row8 c, s;
#pragma unroll
    for (int i = 0; i < 8; ++i) c.v[i] = 1.f, s.v[i] = 0.f;
    if (live) load_angles<kInterleaved>(p.table, p.rot, t0 + r, l, c, s);
    const int orow = p.at_position ? t0 + r : r;
    for (int hb = 0; hb < p.heads_per_item; hb += kNrUnroll) {
      uint4 raw[kNrUnroll];
#pragma unroll
      for (int u = 0; u < kNrUnroll; ++u) {
        const int h = h0 + hb + u;
        raw[u] = make_uint4(0, 0, 0, 0);
        if (live && hb + u < p.heads_per_item && h < H) {
          const __nv_bfloat16* src = h < p.Hq ? p.q + tok * p.q_stride + h * kHeadDim
                                     : h < p.Hq + p.Hkv
                                         ? p.k + tok * p.k_stride + (h - p.Hq) * kHeadDim
                                         : p.v + tok * p.v_stride + (h - p.Hq - p.Hkv) * kHeadDim;
          raw[u] = *(reinterpret_cast<const uint4*>(src) + l);
        }
      }
#pragma unroll
      for (int u = 0; u < kNrUnroll; ++u) {
        const int h = h0 + hb + u;
        Row8 y = unpack8(raw[u]);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(y.v[i], y.v[i], ss);
        const float rs = rsqrtf(half_sum(ss) * (1.f / kHeadDim) + p.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) y.v[i] = y.v[i] * rs * (h < p.Hq ? wq.v[i] : wk.v[i]);
        rotate<kInterleaved, false>(y, c, s, p.rot, l);
        if (live && hb + u < p.heads_per_item && h < H) {
          if (h < p.Hq) {
            *(reinterpret_cast<uint4*>(p.q_out + (tok * p.Hq + h) * kHeadDim) + l) = pack8(y);
          } else {
            const bool isk = h < p.Hq + p.Hkv;
            const int g = h - p.Hq - (isk ? 0 : p.Hkv);
            const size_t o = ((static_cast<size_t>(b) * p.Hkv + g) * p.Lout + orow) * kHeadDim;
            *(reinterpret_cast<uint4*>((isk ? p.k_out : p.v_out) + o) + l) = isk ? pack8(y) : raw[u];
          }
        }
      }
    }
  }
}

// The backward over the same items: input gradients, and one row of partial weight gradients
// per CTA (its half-warps' sums added in a fixed order).
template <bool kInterleaved>
__global__ void __launch_bounds__(kNrThreads) qk_norm_rope_bwd_kernel(const NormRopeParams p) {
  const int l = threadIdx.x & 15;
  const long long items = static_cast<long long>(p.B) * p.Lq * p.chunks;
  const Row8 wq = load_weights(p.qw, p.weights_fp32, l), wk = load_weights(p.kw, p.weights_fp32, l);
  const int H = p.Hq + 2 * p.Hkv;
  const long long stride = static_cast<long long>(gridDim.x) * kNrHalves;
  const long long first = static_cast<long long>(blockIdx.x) * kNrHalves + (threadIdx.x >> 5) * 2;
  Row8 aq, ak;
#pragma unroll
  for (int i = 0; i < 8; ++i) aq.v[i] = ak.v[i] = 0.f;
  for (long long base = first; base < items; base += stride) {
    const long long it = base + ((threadIdx.x >> 4) & 1);
    const bool in = it < items;
    const long long tok = in ? it / p.chunks : 0;
    const int b = static_cast<int>(tok / p.Lq), r = static_cast<int>(tok - static_cast<long long>(b) * p.Lq);
    const int h0 = in ? static_cast<int>(it - tok * p.chunks) * p.heads_per_item : 0;
    int n, t0;
    const bool fits = norm_rope_seq(p, b, n, t0);
    if (in && !fits && r == 0 && h0 == 0 && l == 0) atomicOr(&g_device_error, kDevErrCacheFull);
    const bool live = in && fits && r < n;
    Row8 c, s;
#pragma unroll
    for (int i = 0; i < 8; ++i) c.v[i] = 1.f, s.v[i] = 0.f;
    if (live) load_angles<kInterleaved>(p.table, p.rot, t0 + r, l, c, s);
    for (int hb = 0; hb < p.heads_per_item; hb += 2) {
      uint4 rx[2], rg[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int h = h0 + hb + u;
        rx[u] = rg[u] = make_uint4(0, 0, 0, 0);
        if (live && hb + u < p.heads_per_item && h < H) {
          if (h < p.Hq) {
            rx[u] = *(reinterpret_cast<const uint4*>(p.q + tok * p.q_stride + h * kHeadDim) + l);
            rg[u] = *(reinterpret_cast<const uint4*>(p.dq + (tok * p.Hq + h) * kHeadDim) + l);
          } else {
            const bool isk = h < p.Hq + p.Hkv;
            const int g = h - p.Hq - (isk ? 0 : p.Hkv);
            const size_t o = ((static_cast<size_t>(b) * p.Hkv + g) * p.Lq + r) * kHeadDim;
            if (isk) rx[u] = *(reinterpret_cast<const uint4*>(p.k + tok * p.k_stride + g * kHeadDim) + l);
            rg[u] = *(reinterpret_cast<const uint4*>((isk ? p.dk : p.dv) + o) + l);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int h = h0 + hb + u;
        const bool isq = h < p.Hq, isk = !isq && h < p.Hq + p.Hkv;
        const Row8 x = unpack8(rx[u]);
        Row8 g = unpack8(rg[u]);
        rotate<kInterleaved, true>(g, c, s, p.rot, l);
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = fmaf(x.v[i], x.v[i], ss);
          dot = fmaf(g.v[i] * (isq ? wq.v[i] : wk.v[i]), x.v[i], dot);
        }
        ss = half_sum(ss);
        dot = half_sum(dot);
        const float rs = rsqrtf(ss * (1.f / kHeadDim) + p.eps);
        const float k3 = rs * rs * rs * dot * (1.f / kHeadDim);
        if (live && hb + u < p.heads_per_item && h < H) {
          Row8 dx;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float w = isq ? wq.v[i] : wk.v[i];
            const float dw = g.v[i] * x.v[i] * rs;
            if (isq) aq.v[i] += dw;
            if (isk) ak.v[i] += dw;
            dx.v[i] = fmaf(rs * g.v[i], w, -x.v[i] * k3);
          }
          __nv_bfloat16* dst = isq   ? p.q_out + tok * p.dq_stride + h * kHeadDim
                               : isk ? p.k_out + tok * p.dk_stride + (h - p.Hq) * kHeadDim
                                     : p.v_out + tok * p.dv_stride + (h - p.Hq - p.Hkv) * kHeadDim;
          *(reinterpret_cast<uint4*>(dst) + l) = isq || isk ? pack8(dx) : rg[u];
        }
      }
    }
  }
  __shared__ float red[kNrHalves][2][kHeadDim];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    red[threadIdx.x >> 4][0][8 * l + i] = aq.v[i];
    red[threadIdx.x >> 4][1][8 * l + i] = ak.v[i];
  }
  __syncthreads();
  float a = 0.f;
#pragma unroll
  for (int w = 0; w < kNrHalves; ++w) a += red[w][threadIdx.x >> 7][threadIdx.x & 127];
  p.part[static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x] = a;
}

// d_qw and d_kw from the CTAs' partials: grid 8, a CTA sums 32 of the 256 columns, 32 threads
// of a column over every 32nd part, then over the threads, in fp64 in a fixed order.
__global__ void __launch_bounds__(1024)
    qk_norm_rope_bwd_weights_kernel(const float* __restrict__ part, int parts, float* __restrict__ d_qw,
                                    float* __restrict__ d_kw) {
  __shared__ double red[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, col = blockIdx.x * 32 + x;
  double a = 0.0;
  for (int i = y; i < parts; i += 32) a += part[static_cast<size_t>(i) * 256 + col];
  red[y][x] = a;
  __syncthreads();
  if (y == 0) {
    for (int i = 1; i < 32; ++i) a += red[i][x];
    float* out = col < kHeadDim ? d_qw : d_kw;
    if (out) out[col & (kHeadDim - 1)] = static_cast<float>(a);
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
