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
constexpr int kGradMaxV = 3;      // vectors of a row per thread in the streaming kernel: 12288 columns
constexpr int kGradRows = 2;      // rows of a chunk per thread
// Blocks per SM of the streaming kernel.
template <int V>
constexpr int kGradBlocks = V == 1 ? 2 : 1;
constexpr int kGradMaxSlots = 6;

// A block per row (few rows, or very long ones); V > 0: the row's vectors stay
// in registers (up to V per thread), V == 0: rows of any length in two passes.
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
  uint4 v[V > 0 ? V : 1];
  float m = 0.0f;
  if constexpr (V > 0) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int vi = tid + kGradThreads * j;
      v[j] = vi < nvec ? __ldcs(src + vi) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int vi = tid + kGradThreads * j;
      if (vi < nvec) {
        float g[8];
        scale_vec8(v[j], s_w + 8 * vi, g);
        m = absmax8(g, m);
      }
    }
  } else {
    for (int vi = tid; vi < nvec; vi += kGradThreads) {
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
      if (vi < nvec) {
        float g[8];
        scale_vec8(v[j], s_w + 8 * vi, g);
        dst[vi] = sc == 0.0f ? make_uint2(0u, 0u) : grad_codes8(g, sc, rc, fast);
      }
    }
  } else {
    for (int vi = tid; vi < nvec; vi += kGradThreads) {
      float g[8];
      scale_vec8(__ldcs(src + vi), s_w + 8 * vi, g);
      dst[vi] = sc == 0.0f ? make_uint2(0u, 0u) : grad_codes8(g, sc, rc, fast);
    }
  }
}

// RN(amax / 127) with the constant's reciprocal and one correction step (see
// quant_fast), an IEEE division where the step could leave the normal range.
__device__ __forceinline__ float scale_of(float amax) {
  if (!(amax >= 1e-28f && amax <= 1e36f)) return __fdiv_rn(amax, 127.0f);
  constexpr float kInv = 1.0f / 127.0f;
  const float q0 = __fmul_rn(amax, kInv);
  return __fmaf_rn(__fmaf_rn(-127.0f, q0, amax), kInv, q0);
}

// The same rows for many of them: persistent blocks, one per SM, or two where a
// row takes one vector per thread.  A thread keeps V vectors of columns (tpr
// threads a row, rpi rows at once), so their channel scales stay in registers;
// chunks of kGradRows * rpi rows come through a ring of bulk copies, and the
// rows' maxima meet at one barrier per chunk.  The products stay in registers
// between maximum and codes (V > 1: 4352 x 12288 in 38 us, 49 when they are
// formed twice in two blocks per SM), or are formed again (V == 1, where two
// blocks fill each other's barriers: 512 x 4096 in 6.4 us, 8.5 with one).
template <int V>
__global__ void __launch_bounds__(kGradThreads, kGradBlocks<V>)
    quant_grad_stream_kernel(const uint16_t *__restrict__ dy, int M, int N, int64_t lddy,
                             const float *__restrict__ s_w, int8_t *__restrict__ codes, int64_t ldc,
                             float *__restrict__ s_g, int tpr, int rpi, int slots,
                             unsigned long long *counters, int n_counters) {
  extern __shared__ __align__(128) uint8_t grad_smem[];
  __shared__ uint64_t full[kGradMaxSlots], empty[kGradMaxSlots];
  __shared__ int abort_flag;
  constexpr int K = kGradRows;
  constexpr bool KEEP = kGradBlocks<V> == 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int chunk_rows = rpi * K;
  const uint32_t row_bytes = static_cast<uint32_t>(N) * 2u;
  const uint32_t slot_bytes = chunk_rows * row_bytes;
  uint32_t *row_max = reinterpret_cast<uint32_t *>(grad_smem + slots * slot_bytes);  // [3][chunk_rows]
  const int chunks = (M + chunk_rows - 1) / chunk_rows;
  const int row = tid / tpr, vec = tid - row * tpr, nvec = N >> 3;
  const bool live = row < rpi;
  if (tid == 0) {
    for (int s = 0; s < slots; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kGradWarps);
    }
    abort_flag = 0;
    fence_mbarrier_init();
  }
  for (int i = tid; i < 3 * chunk_rows; i += kGradThreads) row_max[i] = 0u;
  __syncthreads();
  // the product that follows reads only Wq before its own dependency wait
  grid_dependents_launch();
  grid_dependency_wait();
  clear_split_counters(counters, n_counters);
  float2 sw[V][4];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int vi = vec + tpr * j;
    if (live && vi < nvec) {
      const float4 a = __ldg(reinterpret_cast<const float4 *>(s_w + 8 * vi));
      const float4 b = __ldg(reinterpret_cast<const float4 *>(s_w + 8 * vi) + 1);
      sw[j][0] = make_float2(a.x, a.y);
      sw[j][1] = make_float2(a.z, a.w);
      sw[j][2] = make_float2(b.x, b.y);
      sw[j][3] = make_float2(b.z, b.w);
    }
  }
  auto fill = [&](int i, int s) {  // the first warp: this block's i-th chunk
    const int r0 = (static_cast<int>(blockIdx.x) + i * static_cast<int>(gridDim.x)) * chunk_rows;
    const int rows = M - r0 < chunk_rows ? M - r0 : chunk_rows;
    if (lane == 0) mbar_arrive_expect_tx(&full[s], rows * row_bytes);
    __syncwarp();
    const uint16_t *src = dy + static_cast<int64_t>(r0) * lddy;
    uint8_t *dst = grad_smem + s * slot_bytes;
    if (lddy == N) {
      if (lane == 0) bulk_load_g2s(dst, src, rows * row_bytes, &full[s]);
    } else {
      for (int r = lane; r < rows; r += 32) bulk_load_g2s(dst + r * row_bytes, src + r * lddy, row_bytes, &full[s]);
    }
  };
  const int mine = (chunks - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
  int asked = 0;
  if (warp == 0)
    for (; asked < slots && asked < mine; ++asked) fill(asked, asked);
  const bool one_row = (tpr & 31) == 0;  // a warp's threads share a row
  const int first = __shfl_sync(0xFFFFFFFFu, row, 0);
  int slot = 0, turn = 0;
  uint32_t par = 0;      // parity of the fill being read
  bool ok = true;        // after a wait gave up the flow goes on, but stores nothing
  auto refill = [&](int s, uint32_t parity) {  // the first warp
    if (ok) ok = mbar_wait(&empty[s], parity, &abort_flag);
    ok = __all_sync(0xFFFFFFFFu, ok);
    if (ok) fill(asked++, s);
  };
  for (int i = 0; i < mine; ++i) {
    const int r0 = (static_cast<int>(blockIdx.x) + i * static_cast<int>(gridDim.x)) * chunk_rows;
    if (ok) ok = mbar_wait(&full[slot], par, &abort_flag);
    const uint8_t *src = grad_smem + slot * slot_bytes + row * row_bytes + vec * 16u;
    // the products of vector j of this thread's k-th row
    auto products = [&](int k, int j, float2 (&g)[4]) {
      const uint4 v = *reinterpret_cast<const uint4 *>(src + static_cast<uint32_t>(k * rpi) * row_bytes + j * tpr * 16u);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int h = 0; h < 4; ++h)
        g[h] = mul2_rn(make_float2(__uint_as_float(w[h] << 16), __uint_as_float(w[h] & 0xFFFF0000u)), sw[j][h]);
    };
    float2 kept[KEEP ? K : 1][KEEP ? V : 1][4];
    uint32_t mb[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float m = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (live && vec + tpr * j < nvec) {  // rows past M: what the slot held, never stored
          float2(&g)[4] = kept[KEEP ? k : 0][KEEP ? j : 0];
          products(k, j, g);
#pragma unroll
          for (int h = 0; h < 4; ++h) m = fmaxf(m, fmaxf(fabsf(g[h].x), fabsf(g[h].y)));
        }
      }
      mb[k] = __float_as_uint(m);
    }
    if constexpr (KEEP) {  // the rows are in registers
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[slot]);
    }
    // one maximum per warp and row (a warp holds one or two rows, or several
    // narrow ones) goes to shared memory
    uint32_t *mx = row_max + turn * chunk_rows;
    if (one_row) {
#pragma unroll
      for (int k = 0; k < K; ++k) mb[k] = __reduce_max_sync(0xFFFFFFFFu, mb[k]);
      if (lane == 0 && live) {
#pragma unroll
        for (int k = 0; k < K; ++k) atomicMax(mx + row + k * rpi, mb[k]);
      }
    } else if (tpr > 32) {
      uint32_t m1[K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        m1[k] = __reduce_max_sync(0xFFFFFFFFu, row == first ? 0u : mb[k]);
        mb[k] = __reduce_max_sync(0xFFFFFFFFu, row == first ? mb[k] : 0u);
      }
      if (lane == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (first < rpi) atomicMax(mx + first + k * rpi, mb[k]);
          if (first + 1 < rpi) atomicMax(mx + first + 1 + k * rpi, m1[k]);
        }
      }
    } else if (live) {
#pragma unroll
      for (int k = 0; k < K; ++k) atomicMax(mx + row + k * rpi, mb[k]);
    }
    __syncthreads();
    if (KEEP && warp == 0 && asked < mine) refill(slot, par);  // released before the barrier
    // the maxima of two chunks ago are no longer read: cleared for the chunk
    // after the next
    uint32_t *old = row_max + (turn == 0 ? 2 : turn - 1) * chunk_rows;
    for (int r = tid; r < chunk_rows; r += kGradThreads) old[r] = 0u;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t m = static_cast<int64_t>(r0) + row + k * rpi;
      if (live && m < M && ok) {
        const float amax = __uint_as_float(mx[row + k * rpi]);
        const float sc = amax == 0.0f ? 0.0f : scale_of(amax);
        const bool fast = quant_fast_ok(sc);
        const float rc = fast ? __frcp_rn(sc) : 0.0f;
        if (vec == 0) s_g[m] = sc;
        int8_t *dst = codes + m * ldc;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (vec + tpr * j < nvec) {
            float2(&g)[4] = kept[KEEP ? k : 0][KEEP ? j : 0];
            if constexpr (!KEEP) products(k, j, g);
            uint32_t c[8];
            if (fast) {
#pragma unroll
              for (int h = 0; h < 4; ++h) {  // quant_fast on two values at once
                const float2 x = g[h], y = make_float2(rc, rc);
                const float2 q0 = mul2_rn_q(x, y);
                const float2 e = fma2_rn(q0, make_float2(-sc, -sc), x);
                const float2 r = add2_rn_q(fma2_rn(e, y, q0), make_float2(kRintMagic, kRintMagic));
                c[2 * h] = __float_as_uint(r.x);
                c[2 * h + 1] = __float_as_uint(r.y);
              }
            } else {
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                c[2 * h] = sc == 0.0f ? 0u : quant_exact(g[h].x, sc);
                c[2 * h + 1] = sc == 0.0f ? 0u : quant_exact(g[h].y, sc);
              }
            }
            *reinterpret_cast<uint2 *>(dst + 8 * (vec + tpr * j)) = pack_codes(c);
          }
        }
      }
    }
    if constexpr (!KEEP) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[slot]);
      // the chunk before this one is by now done in every warp, so its slot
      // is filled again
      const int before = slot == 0 ? slots - 1 : slot - 1;
      if (warp == 0 && i > 0 && asked < mine) refill(before, slot == 0 ? par ^ 1u : par);
    }
    turn = turn == 2 ? 0 : turn + 1;
    if (++slot == slots) {
      slot = 0;
      par ^= 1u;
    }
  }
  if (warp == 0 && !ok) {  // copies still in flight land before the block leaves
    for (int i = asked - slots < 0 ? 0 : asked - slots; i < asked; ++i) {
      volatile int never = 0;
      mbar_wait(&full[i % slots], static_cast<uint32_t>(i / slots) & 1u, &never);
    }
  }
}

}  // namespace w8a8
