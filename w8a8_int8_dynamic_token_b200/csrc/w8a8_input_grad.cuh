// w8a8_input_grad.cuh -- the rows of the W8A8 layer's input gradient.
//
// For y = x^ W^T + bias with W^[n,k] = Wq[n,k] * s_w[n] (the dequantized
// weight; the rounding of x to int8 passes the gradient straight through),
//   dx[m,k] = sum_n dy[m,n] * s_w[n] * Wq[n,k].
// The channel scales lie along the contraction, so they cannot leave the sum;
// they are taken into the rows first, and the rows are quantized per token:
//   g[m,n]  = dy[m,n] * s_w[n]                          (fp32, rounded once)
//   s_g[m]  = max_n |g[m,n]| / 127                      (fp32, IEEE)
//   c[m,n]  = clamp(rint(g[m,n] / s_g[m]), -127, 127)   (0 in a row of zeros)
//   dx[m,k] = bf16_rne((float)(sum_n c[m,n] * Wq[n,k]) * s_g[m])
// The product is exact in int32 and runs in the layer's own tensor-core
// kernels, which read Wq as it is stored (its columns contiguous: MN-major
// operands, see B_MN / A_MN there), so no transposed copy is kept.
//
// g is bounded by memory: 2 M N bytes of dy in, M N bytes of codes out.
#pragma once

#include <cstdint>

#include "w8a8_ptx.cuh"
#include "w8a8_quant.cuh"

namespace w8a8 {

// g = dy * s_w for one vector of 8.
__device__ __forceinline__ void scale_vec8(uint4 v, const float *sw, float (&g)[8]) {
  unpack8(v, g);
  const float4 a = __ldg(reinterpret_cast<const float4 *>(sw));
  const float4 b = __ldg(reinterpret_cast<const float4 *>(sw) + 1);
  g[0] = __fmul_rn(g[0], a.x); g[1] = __fmul_rn(g[1], a.y);
  g[2] = __fmul_rn(g[2], a.z); g[3] = __fmul_rn(g[3], a.w);
  g[4] = __fmul_rn(g[4], b.x); g[5] = __fmul_rn(g[5], b.y);
  g[6] = __fmul_rn(g[6], b.z); g[7] = __fmul_rn(g[7], b.w);
}

__device__ __forceinline__ uint2 grad_codes8(const float (&g)[8], float s, float y, bool fast) {
  uint32_t c[8];
  if (fast) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = quant_fast(g[i], s, y);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = quant_exact(g[i], s);
  }
  return pack_codes(c);
}

// One block of 256 threads per row; V > 0: the row's vectors stay in
// registers (up to V per thread), V == 0: rows of any length in two passes.
// The codes' rows are ldc bytes apart.
template <int V>
__global__ void __launch_bounds__(256)
    quant_grad_rows_kernel(const uint16_t *__restrict__ dy, int N, int64_t lddy,
                           const float *__restrict__ s_w, int8_t *__restrict__ codes, int64_t ldc,
                           float *__restrict__ s_g) {
  __shared__ uint32_t red[8];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  const int nvec = N >> 3;
  const uint4 *src = reinterpret_cast<const uint4 *>(dy + row * lddy);
  // the product that follows reads only Wq before its own dependency wait
  grid_dependents_launch();
  grid_dependency_wait();
  uint4 v[V > 0 ? V : 1];
  float m = 0.0f;
  if constexpr (V > 0) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int vi = tid + 256 * j;
      v[j] = vi < nvec ? __ldcs(src + vi) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int vi = tid + 256 * j;
      if (vi < nvec) {
        float g[8];
        scale_vec8(v[j], s_w + 8 * vi, g);
        m = absmax8(g, m);
      }
    }
  } else {
    for (int vi = tid; vi < nvec; vi += 256) {
      float g[8];
      scale_vec8(__ldg(src + vi), s_w + 8 * vi, g);
      m = absmax8(g, m);
    }
  }
  uint32_t mb = warp_max_u32(__float_as_uint(m), 32);
  if ((tid & 31) == 0) red[tid >> 5] = mb;
  __syncthreads();
  mb = 0u;
#pragma unroll
  for (int w = 0; w < 8; ++w) mb = max(mb, red[w]);
  const float amax = __uint_as_float(mb);
  const float sc = (amax == 0.0f) ? 0.0f : __fdiv_rn(amax, 127.0f);
  const bool fast = quant_fast_ok(sc);
  const float rc = fast ? __frcp_rn(sc) : 0.0f;
  if (tid == 0) s_g[row] = sc;
  uint2 *dst = reinterpret_cast<uint2 *>(codes + row * ldc);
  if constexpr (V > 0) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int vi = tid + 256 * j;
      if (vi < nvec) {
        float g[8];
        scale_vec8(v[j], s_w + 8 * vi, g);
        dst[vi] = sc == 0.0f ? make_uint2(0u, 0u) : grad_codes8(g, sc, rc, fast);
      }
    }
  } else {
    for (int vi = tid; vi < nvec; vi += 256) {
      float g[8];
      scale_vec8(__ldcs(src + vi), s_w + 8 * vi, g);
      dst[vi] = sc == 0.0f ? make_uint2(0u, 0u) : grad_codes8(g, sc, rc, fast);
    }
  }
}

}  // namespace w8a8
