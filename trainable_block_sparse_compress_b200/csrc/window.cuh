// window.cuh -- sliding-window attention with a few first tokens that stay visible (sinks).
//
// The query at position t sees the keys u <= t with u > t - window or u < n_sink:
//   O = softmax(scale q K^T) V over them; lse = log of the softmax's normaliser.
// Backward, with P = exp(scale q K^T - lse), D = dO . O:
//   dS = P (dO V^T - D), dq = scale dS K, dK = scale dS^T q, dV = P^T dO.
#pragma once
#include "common.cuh"

namespace infllmv2 {

struct WinParams {
  const __nv_bfloat16 *q, *k, *v;
  const int32_t *q_lens, *kv_lens;
  int B, Hq, Hkv, G, Lq, Lmax, window, n_sink;
  float scale, scale_log2;
  __nv_bfloat16* o;
  float* lse;                      // forward: output; backward: input
  const __nv_bfloat16 *o_in, *d_o;
  __nv_bfloat16 *dq, *dk, *dv;
};

__device__ __forceinline__ void load4(const __nv_bfloat16* p, int lane, float (&x)[4]) {
  const uint2 u = *(reinterpret_cast<const uint2*>(p) + lane);
  x[0] = __uint_as_float(u.x << 16), x[1] = __uint_as_float(u.x & 0xffff0000u);
  x[2] = __uint_as_float(u.y << 16), x[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, int lane, const float (&x)[4]) {
  *(reinterpret_cast<uint2*>(p) + lane) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
}
__device__ __forceinline__ float warp_dot4(const float (&a)[4], const float (&b)[4]) {
  float s = fmaf(a[0], b[0], fmaf(a[1], b[1], fmaf(a[2], b[2], a[3] * b[3])));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  return s;
}

// One warp per (sequence, query row, q-head), a lane four of the 128 dimensions.
__global__ void __launch_bounds__(128) window_rows_kernel(const WinParams p, int decode) {
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= static_cast<long long>(p.B) * p.Lq * p.Hq) return;
  const int h = static_cast<int>(row % p.Hq), r = static_cast<int>(row / p.Hq % p.Lq);
  const int b = static_cast<int>(row / p.Hq / p.Lq);
  const ChunkLens c = chunk_lens(p.q_lens, p.kv_lens, b, p.Lq, p.Lmax);
  const size_t li = (static_cast<size_t>(b) * p.Hq + h) * p.Lq + r;
  float acc[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, z = 0.f;
  if (r >= c.q_len) {
    if (!decode) return;
    store4(p.o + row * kHeadDim, lane, acc);
    if (p.lse && lane == 0) p.lse[li] = -INFINITY;
    return;
  }
  const int t = c.kv_len - c.q_len + r;
  float q[4];
  load4(p.q + row * kHeadDim, lane, q);
  const size_t base = (static_cast<size_t>(b) * p.Hkv + h / p.G) * p.Lmax * kHeadDim;
  const int lo = max(0, t - p.window + 1);
  for (int u = min(p.n_sink, lo) > 0 ? 0 : lo; u <= t; ++u) {
    if (u == p.n_sink && u < lo) u = lo;
    float kk[4], vv[4];
    load4(p.k + base + static_cast<size_t>(u) * kHeadDim, lane, kk);
    load4(p.v + base + static_cast<size_t>(u) * kHeadDim, lane, vv);
    const float x = warp_dot4(q, kk) * p.scale_log2;
    const float mn = fmaxf(m, x), f = ex2(m - mn), e = ex2(x - mn);
    m = mn;
    z = fmaf(z, f, e);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(acc[i], f, e * vv[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] /= z;
  store4(p.o + row * kHeadDim, lane, acc);
  if (p.lse && lane == 0) p.lse[li] = (m + lg2(z)) * 0.6931471805599453f;
}

}  // namespace infllmv2
