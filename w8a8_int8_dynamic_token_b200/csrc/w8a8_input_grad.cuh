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
// A NaN in a row makes the row's scale and with it its whole dx NaN, an infinity
// makes them infinite or NaN, so that a training loop sees both.
//
// The rows are bound by memory: 2 M N bytes of dy in, M N bytes of codes out.
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

// The first block clears the arrival counters of the product that follows (its
// epilogue reads them behind its own dependency wait): one launch less than a
// memset ahead of this kernel, 3 us on its way.
__device__ __forceinline__ void clear_split_counters(unsigned long long *counters, int n) {
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < n; i += blockDim.x) counters[i] = 0ull;
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

constexpr int kGradThreads = 512;
constexpr int kGradWarps = kGradThreads / 32;
// A block per row (up to several rows per SM, or very long ones); V > 0: the row's products stay
// in registers (up to V vectors per thread), V == 0: rows of any length in two
// passes.
// The codes' rows are ldc bytes apart.
template <int V>
__global__ void __launch_bounds__(kGradThreads)
    quant_grad_rows_kernel(const uint16_t *__restrict__ dy, int N, int64_t lddy,
                           const float *__restrict__ s_w, int8_t *__restrict__ codes, int64_t ldc,
                           float *__restrict__ s_g, unsigned long long *counters, int n_counters) {
  __shared__ uint32_t red[kGradWarps];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  const int nvec = N >> 3;
  const uint4 *src = reinterpret_cast<const uint4 *>(dy + row * lddy);
  // the product that follows reads only Wq before its own dependency wait
  grid_dependents_launch();
  grid_dependency_wait();
  clear_split_counters(counters, n_counters);
  float g[V > 0 ? V : 1][8];
  float m = 0.0f;
  if constexpr (V > 0) {
    uint4 v[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int vi = tid + kGradThreads * j;
      v[j] = vi < nvec ? __ldcs(src + vi) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int vi = tid + kGradThreads * j;
      scale_vec8(v[j], s_w + 8 * (vi < nvec ? vi : 0), g[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) m = absmax_nan(m, g[j][i]);
    }
  } else {
    for (int vi = tid; vi < nvec; vi += kGradThreads) {
      scale_vec8(__ldg(src + vi), s_w + 8 * vi, g[0]);
#pragma unroll
      for (int i = 0; i < 8; ++i) m = absmax_nan(m, g[0][i]);
    }
  }
  uint32_t mb = warp_max_u32(__float_as_uint(m), 32);
  if ((tid & 31) == 0) red[tid >> 5] = mb;
  __syncthreads();
  mb = 0u;
#pragma unroll
  for (int w = 0; w < kGradWarps; ++w) mb = max(mb, red[w]);
  const float amax = __uint_as_float(mb);
  const float sc = (amax == 0.0f) ? 0.0f : __fdiv_rn(amax, 127.0f);
  const bool fast = quant_fast_ok(sc);
  const float rc = fast ? __frcp_rn(sc) : 0.0f;
  if (tid == 0) s_g[row] = sc;
  uint2 *dst = reinterpret_cast<uint2 *>(codes + row * ldc);
  if constexpr (V > 0) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int vi = tid + kGradThreads * j;
      if (vi < nvec) dst[vi] = sc == 0.0f ? make_uint2(0u, 0u) : grad_codes8(g[j], sc, rc, fast);
    }
  } else {
    for (int vi = tid; vi < nvec; vi += kGradThreads) {
      scale_vec8(__ldcs(src + vi), s_w + 8 * vi, g[0]);
      dst[vi] = sc == 0.0f ? make_uint2(0u, 0u) : grad_codes8(g[0], sc, rc, fast);
    }
  }
}

// The same rows for many of them: one block of 16 warps per SM, persistent, in
// groups of G warps (1, 2 or 4, as in quant_rows_bulk_kernel), each on a row
// of its own, so that the groups' phases fill one another's latencies.  The
// channel scales lie in shared memory, as two arrays of the even and odd
// 16-byte halves of a vector's eight (32-byte steps between lanes would
// conflict in pairs); rows come through one ring of bulk copies that all
// groups share.  A row is multiplied twice, for its maximum and for its codes.
// A slot's rows belong to different groups where the slots are no multiple of
// the groups (7 and 4 at 12288 values), and nothing else keeps the groups in
// step, so a group can reach its row while the slot's copy two or more before
// it is still under way; the barrier's parity alone would then let it through.
// It therefore waits until the row's own copy has been asked for (`issued`),
// which happens once the copy before it has landed, and only then for its phase.
// 4352 x 12288 takes 41 us in a capture (160 MB of traffic: 28.7 as a bare stream
// of the same reads and writes), bound by shared memory: 12 bytes an element, 18
// us of it; the count of copies is 2% (8704 x 8192, whole calls: 74.3 and 72.9).
// With the scales in registers instead (whole block on two rows at a time, one
// barrier per two rows) it took 38 where this took 37, with two such teams 46.
constexpr int kGradBulkWarps = 16;
constexpr int kGradMaxSlots = 16;

// Until `count` copies have been asked for in a slot (bounded as every wait).
__device__ __forceinline__ bool issued_wait(volatile int *issued, int count, volatile int *abort_flag) {
  if (*issued >= count) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t i = 1;; ++i) {
    if (*issued >= count) return true;
    if ((i & 31u) == 0u) {
      if (*abort_flag) return false;
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        atomicOr(&g_device_error, W8A8_DEVERR_TIMEOUT);
        return false;
      }
    }
  }
}

__global__ void __launch_bounds__(kGradBulkWarps * 32, 1)
    quant_grad_bulk_kernel(const uint16_t *__restrict__ dy, int M, int N, int64_t lddy,
                           const float *__restrict__ s_w, int8_t *__restrict__ codes, int64_t ldc,
                           float *__restrict__ s_g, int group_warps, int slots,
                           unsigned long long *counters, int n_counters) {
  extern __shared__ __align__(128) uint8_t grad_smem[];
  __shared__ uint64_t bars[kGradMaxSlots];
  __shared__ uint32_t red[kGradBulkWarps];
  __shared__ int okf[kGradBulkWarps];
  __shared__ volatile int issued[kGradMaxSlots];  // copies asked for so far
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = group_warps, groups = kGradBulkWarps / G;
  const int group = warp / G, gw = warp - group * G;
  const int gthreads = G * 32, t = gw * 32 + lane;
  const int nvec = N >> 3;
  const uint32_t row_bytes = static_cast<uint32_t>(N) * 2u;
  float4 *const sw_even = reinterpret_cast<float4 *>(grad_smem), *const sw_odd = sw_even + nvec;
  uint8_t *const ring = grad_smem + static_cast<size_t>(N) * 4;
  const int stride = static_cast<int>(gridDim.x);
  const int mine = (M - static_cast<int>(blockIdx.x) + stride - 1) / stride;  // rows of this block
  if (threadIdx.x == 0) {
    for (int s = 0; s < slots; ++s) {
      mbar_init(&bars[s], 1);
      issued[s] = 0;
    }
    abort_flag = 0;
    fence_mbarrier_init();
  }
  // the product that follows reads only Wq before its own dependency wait
  grid_dependents_launch();
  grid_dependency_wait();
  auto fill = [&](int i, int s) {  // one thread: this block's i-th row
    const int64_t row = static_cast<int64_t>(blockIdx.x) + static_cast<int64_t>(i) * stride;
    mbar_arrive_expect_tx(&bars[s], row_bytes);
    bulk_load_g2s(ring + s * row_bytes, dy + row * lddy, row_bytes, &bars[s]);
    issued[s] = i / slots + 1;
  };
  if (threadIdx.x == 0)
    for (int i = 0; i < slots && i < mine; ++i) fill(i, i);
  for (int v = threadIdx.x; v < nvec; v += kGradBulkWarps * 32) {
    sw_even[v] = __ldg(reinterpret_cast<const float4 *>(s_w) + 2 * v);
    sw_odd[v] = __ldg(reinterpret_cast<const float4 *>(s_w) + 2 * v + 1);
  }
  clear_split_counters(counters, n_counters);
  __syncthreads();
  // the products of vector v of a row
  auto products = [&](const uint4 *xs, int v, float2 (&g)[4]) {
    const uint4 x = xs[v];
    const float4 a = sw_even[v], b = sw_odd[v];
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    const float2 s[4] = {make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)};
#pragma unroll
    for (int h = 0; h < 4; ++h)
      g[h] = mul2_rn(make_float2(__uint_as_float(w[h] << 16), __uint_as_float(w[h] & 0xFFFF0000u)), s[h]);
  };
  int i = group;
  bool ok = true;
  for (; i < mine; i += groups) {
    const int slot = i % slots, phase = i / slots;
    ok = issued_wait(&issued[slot], phase + 1, &abort_flag) &&
         mbar_wait(&bars[slot], static_cast<uint32_t>(phase) & 1u, &abort_flag);
    ok = __all_sync(0xFFFFFFFFu, ok);
    if (G > 1) {  // the group's warps leave together or not at all
      if (lane == 0) okf[warp] = ok ? 1 : 0;
      named_barrier_sync(1 + group, gthreads);
      for (int w = 0; w < G; ++w) ok = ok && okf[group * G + w] != 0;
    }
    if (!ok) break;
    const int64_t row = static_cast<int64_t>(blockIdx.x) + static_cast<int64_t>(i) * stride;
    const uint4 *xs = reinterpret_cast<const uint4 *>(ring + slot * row_bytes);
    float m0 = 0.0f, m1 = 0.0f;
#pragma unroll 4
    for (int v = t; v < nvec; v += gthreads) {
      float2 g[4];
      products(xs, v, g);
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        m0 = absmax_nan(m0, g[h].x);
        m1 = absmax_nan(m1, g[h].y);
      }
    }
    uint32_t mb = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(absmax_nan(m0, m1)));
    if (G > 1) {  // across the group's warps
      if (lane == 0) red[warp] = mb;
      named_barrier_sync(1 + group, gthreads);
      mb = 0u;
      for (int w = 0; w < G; ++w) mb = max(mb, red[group * G + w]);
    }
    const float amax = __uint_as_float(mb);
    const float sc = (amax == 0.0f) ? 0.0f : __fdiv_rn(amax, 127.0f);
    const bool fast = quant_fast_ok(sc);
    const float rc = fast ? __frcp_rn(sc) : 0.0f;
    if (t == 0) s_g[row] = sc;
    uint2 *dst = reinterpret_cast<uint2 *>(codes + row * ldc);
    if (fast) {
      const float2 neg_s = make_float2(-sc, -sc), y = make_float2(rc, rc);
#pragma unroll 2
      for (int v = t; v < nvec; v += gthreads) {
        float2 g[4];
        products(xs, v, g);
        uint32_t c[8];
#pragma unroll
        for (int h = 0; h < 4; ++h) {  // quant_fast on two values at once
          const float2 q0 = mul2_rn_q(g[h], y);
          const float2 e = fma2_rn(q0, neg_s, g[h]);
          const float2 r = add2_rn_q(fma2_rn(e, y, q0), make_float2(kRintMagic, kRintMagic));
          c[2 * h] = __float_as_uint(r.x);
          c[2 * h + 1] = __float_as_uint(r.y);
        }
        dst[v] = pack_codes(c);
      }
    } else {
      for (int v = t; v < nvec; v += gthreads) {
        float2 g[4];
        products(xs, v, g);
        uint32_t c[8];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          c[2 * h] = sc == 0.0f ? 0u : quant_exact(g[h].x, sc);
          c[2 * h + 1] = sc == 0.0f ? 0u : quant_exact(g[h].y, sc);
        }
        dst[v] = pack_codes(c);
      }
    }
    // every thread of the group is done with the slot (and with red[]) before
    // the slot takes the row that is `slots` rows on, whichever group's it is
    if (G > 1) named_barrier_sync(1 + group, gthreads); else __syncwarp();
    if (t == 0 && i + slots < mine) fill(i + slots, slot);
  }
  __syncthreads();  // nothing more is asked for
  if (threadIdx.x == 0 && abort_flag != 0) {
    // gave up: the copies in flight land before the block leaves
    volatile int never = 0;
    for (int s = 0; s < slots; ++s)
      if (issued[s] > 0) mbar_wait(&bars[s], static_cast<uint32_t>(issued[s] - 1) & 1u, &never);
  }
}

}  // namespace w8a8
