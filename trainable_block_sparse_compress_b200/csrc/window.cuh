// window.cuh -- sliding-window attention with a few first tokens that stay visible (sinks).
//
// The query at position t sees the keys u <= t with u > t - window or u < n_sink:
//   O = softmax(scale q K^T) V over them; lse = log of the softmax's normaliser.
// Kernels: csrc/window_tc.cuh (prefill and chunks), csrc/window_decode.cuh (one token per
// sequence), csrc/window_bwd_tc.cuh (backward).
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

// Four consecutive values of a row per lane, rounded to bf16.
__device__ __forceinline__ void store4(__nv_bfloat16* p, int lane, const float (&x)[4]) {
  *(reinterpret_cast<uint2*>(p) + lane) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
}

}  // namespace infllmv2
