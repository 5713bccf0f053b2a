// w8a8_norm.cuh -- group normalization of channels-last tensors, with SiLU.
//
// x [B, S, C] (S pixels of C channels, channels adjacent), G groups of
// c = C / G adjacent channels.  Over the S * c values of a sample's group:
//   mean = E x,  rstd = 1 / sqrt(E (x - mean)^2 + eps)
//   z = (x - mean) * rstd * w + b,  y = z or z * sigmoid(z)
// The int8 form quantizes each pixel's row of y (fp32, not rounded to bf16
// first) for the W8A8 layer that follows: s = max|y| / 127, q = rint(y / s).
// Backward, with xh = (x - mean) * rstd, n = S * c and dz = dy * y'(z):
//   dw = sum dz * xh,  db = sum dz   (over samples and pixels)
//   dx = rstd * (w dz - (1/n) sum w dz - xh * (1/n) sum w dz xh)
//
// Work is cut into (sample, run of pixels) slabs.  A thread keeps one 16-byte
// vector of channels and walks over pixels, so a block reads whole rows.
// Statistics: batches of 8 pixels per channel are reduced in two passes over
// registers (mean, then squared deviations) and joined by the pairwise update
// of Chan, Golub and LeVeque (1979); no difference of large squares appears,
// so a mean far from zero costs no precision.  All joins run in a fixed order
// (no atomics on sums): results do not depend on scheduling.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "w8a8_ptx.cuh"
#include "w8a8_quant.cuh"
#include "w8a8_rotary.cuh"

namespace w8a8 {

constexpr int kNormThreads = 512;  // at most; whole warps, rpi rows of tpr threads
constexpr int kNormMaxVecs = 512;  // 16-byte vectors of a pixel: 4096 channels, 2048 in fp32
constexpr int kNormBatch = 8;  // pixels per statistics batch
constexpr int kNormRows = 4;   // pixels in flight per thread elsewhere

struct NormParams {
  const void *x, *dy;
  void *y;                       // y, or dx
  int64_t xb, xs, dyb, dys, yb, ys;  // strides of a sample and a pixel, elements
  int32_t B, S, C, G;
  int32_t slabs;                 // per sample
  int32_t tpr, rpi;              // threads per row, rows per block iteration
  const void *weight, *bias;     // [C] in x's type or fp32, or nullptr
  int32_t param_f32;
  float eps;
  int32_t silu;
  float2 *part;                  // [B][slabs][G]: (mean, M2), or the group sums
  float2 *chan;                  // [B][slabs][C]: channel sums (backward)
  float *mean_out, *rstd_out;    // [B, G] or nullptr
  const float *mean_in, *rstd_in;
  int8_t *q;
  float *s_q;
  float *dweight, *dbias;        // [C] or nullptr
};

// Pixels [lo, hi) of slab j: an even share, the first slabs one more.
__device__ __forceinline__ void slab_range(int S, int slabs, int j, int &lo, int &hi) {
  const int per = S / slabs, extra = S % slabs;
  lo = j * per + (j < extra ? j : extra);
  hi = lo + per + (j < extra ? 1 : 0);
}

__device__ __forceinline__ float norm_param(const void *p, int f32, int c, float none,
                                            const __nv_bfloat16 *) {
  if (p == nullptr) return none;
  return f32 ? static_cast<const float *>(p)[c] : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[c]);
}
__device__ __forceinline__ float norm_param(const void *p, int f32, int c, float none,
                                            const __half *) {
  if (p == nullptr) return none;
  return f32 ? static_cast<const float *>(p)[c] : __half2float(static_cast<const __half *>(p)[c]);
}
__device__ __forceinline__ float norm_param(const void *p, int, int c, float none, const float *) {
  return p == nullptr ? none : static_cast<const float *>(p)[c];
}

template <typename T>
constexpr int kNormVec = 16 / static_cast<int>(sizeof(T));

__device__ __forceinline__ float silu(float z) { return __fdividef(z, 1.0f + __expf(-z)); }

// Sum over the warp in a fixed order.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Statistics of one slab: (mean, M2) of each group into part[b][slab][g].
// Shared memory: float2 [rpi][C], then the row counts are arithmetic.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_stats_kernel(const NormParams p) {
  constexpr int V = kNormVec<T>;
  extern __shared__ float2 chan_stat[];  // [rpi][C]
  const int b = blockIdx.x / p.slabs, slab = blockIdx.x - b * p.slabs;
  int lo, hi;
  slab_range(p.S, p.slabs, slab, lo, hi);
  const int row = threadIdx.x / p.tpr, vec = threadIdx.x - row * p.tpr;
  const T *x = static_cast<const T *>(p.x) + b * p.xb + vec * V;
  float mean[V], m2[V];
#pragma unroll
  for (int i = 0; i < V; ++i) mean[i] = m2[i] = 0.0f;
  int n = 0;
  if (row < p.rpi) {
    for (int s0 = lo + row; s0 < hi; s0 += kNormBatch * p.rpi) {
      T v[kNormBatch][V];
#pragma unroll
      for (int j = 0; j < kNormBatch; ++j) {
        const int s = s0 + j * p.rpi;
        if (s < hi) VecIO<T, V, true>::load(x + s * p.xs, v[j]);
      }
      const int left = (hi - s0 + p.rpi - 1) / p.rpi;
      const int nb = left < kNormBatch ? left : kNormBatch;
      const float inv = 1.0f / nb;
      const float share = static_cast<float>(nb) / static_cast<float>(n + nb);
      const float cross = share * n;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < kNormBatch; ++j)
          if (j < nb) sum += to_f32<T>(v[j][i]);
        const float mb = sum * inv;
        float sq = 0.0f;
#pragma unroll
        for (int j = 0; j < kNormBatch; ++j) {
          if (j < nb) {
            const float d = to_f32<T>(v[j][i]) - mb;
            sq += d * d;
          }
        }
        const float delta = mb - mean[i];
        mean[i] += delta * share;
        m2[i] += sq + delta * delta * cross;
      }
      n += nb;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) chan_stat[row * p.C + vec * V + i] = make_float2(mean[i], m2[i]);
  }
  __syncthreads();
  // a warp per group joins its rpi x c entries: entries of row r stand for
  // n_r pixels
  const int c = p.C / p.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int pixels = hi - lo;
  const float inv_n = 1.0f / (static_cast<float>(pixels) * c);
  for (int g = warp; g < p.G; g += warps) {
    float sum = 0.0f;
    for (int e = lane; e < p.rpi * c; e += 32) {
      const int r = e / c, ch = g * c + (e - r * c);
      const int nr = r < pixels ? (pixels - r + p.rpi - 1) / p.rpi : 0;
      sum += nr * chan_stat[r * p.C + ch].x;
    }
    const float gm = warp_sum(sum) * inv_n;
    float sq = 0.0f;
    for (int e = lane; e < p.rpi * c; e += 32) {
      const int r = e / c, ch = g * c + (e - r * c);
      const int nr = r < pixels ? (pixels - r + p.rpi - 1) / p.rpi : 0;
      const float2 st = chan_stat[r * p.C + ch];
      const float d = st.x - gm;
      sq += st.y + nr * d * d;
    }
    sq = warp_sum(sq);
    if (lane == 0) p.part[(static_cast<int64_t>(b) * p.slabs + slab) * p.G + g] = make_float2(gm, sq);
  }
}

// Joins a sample's slab statistics: (mean, rstd) of each group into out[G]
// (shared memory).  All threads of the block call it; synchronizes at the end.
__device__ __forceinline__ void norm_join(const NormParams &p, int b, float2 *out) {
  const int c = p.C / p.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const float inv_s = 1.0f / p.S;
  {
    for (int g = warp; g < p.G; g += warps) {
      const float2 *part = p.part + static_cast<int64_t>(b) * p.slabs * p.G + g;
      float sum = 0.0f;
      for (int j = lane; j < p.slabs; j += 32) {
        int lo, hi;
        slab_range(p.S, p.slabs, j, lo, hi);
        sum += (hi - lo) * inv_s * part[static_cast<int64_t>(j) * p.G].x;
      }
      const float mean = warp_sum(sum);
      float sq = 0.0f;
      for (int j = lane; j < p.slabs; j += 32) {
        int lo, hi;
        slab_range(p.S, p.slabs, j, lo, hi);
        const float2 st = part[static_cast<int64_t>(j) * p.G];
        const float d = st.x - mean;
        sq += st.y + static_cast<float>(hi - lo) * c * d * d;
      }
      const float var = warp_sum(sq) / (static_cast<float>(p.S) * c);
      if (lane == 0) out[g] = make_float2(mean, 1.0f / sqrtf(var + p.eps));
    }
  }
  __syncthreads();
}

// Normalizes one slab (see norm_stats_kernel for the mapping).  QUANT: int8
// rows and their scales instead of y.
template <typename T, bool QUANT>
__global__ void __launch_bounds__(kNormThreads) norm_apply_kernel(const NormParams p) {
  constexpr int V = kNormVec<T>;
  constexpr int R = kNormRows;
  extern __shared__ float2 group_stat[];  // [G]; QUANT: then uint [R * rpi] row maxima
  const int b = blockIdx.x / p.slabs, slab = blockIdx.x - b * p.slabs;
  int lo, hi;
  slab_range(p.S, p.slabs, slab, lo, hi);
  norm_join(p, b, group_stat);
  const int c = p.C / p.G;
  if (slab == 0 && p.mean_out != nullptr) {
    for (int g = threadIdx.x; g < p.G; g += blockDim.x) {
      p.mean_out[static_cast<int64_t>(b) * p.G + g] = group_stat[g].x;
      p.rstd_out[static_cast<int64_t>(b) * p.G + g] = group_stat[g].y;
    }
  }
  const int row = threadIdx.x / p.tpr, vec = threadIdx.x - row * p.tpr;
  const bool live = row < p.rpi;
  float scale[V], shift[V], mean[V];
  if (live) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int ch = vec * V + i;
      const float2 st = group_stat[ch / c];
      mean[i] = st.x;
      scale[i] = st.y * norm_param(p.weight, p.param_f32, ch, 1.0f, static_cast<const T *>(nullptr));
      shift[i] = norm_param(p.bias, p.param_f32, ch, 0.0f, static_cast<const T *>(nullptr));
    }
  }
  const T *x = static_cast<const T *>(p.x) + b * p.xb + vec * V;
  if constexpr (!QUANT) {
    if (!live) return;
    T *y = static_cast<T *>(p.y) + b * p.yb + vec * V;
    for (int s0 = lo + row; s0 < hi; s0 += R * p.rpi) {
      T v[R][V];
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int s = s0 + j * p.rpi;
        if (s < hi) VecIO<T, V, true>::load(x + s * p.xs, v[j]);
      }
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int s = s0 + j * p.rpi;
        if (s >= hi) break;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float z = __fmaf_rn(to_f32<T>(v[j][i]) - mean[i], scale[i], shift[i]);
          v[j][i] = from_f32<T>(p.silu ? silu(z) : z);
        }
        VecIO<T, V, true>::store(y + s * p.ys, v[j]);
      }
    }
  } else {
    uint32_t *row_max = reinterpret_cast<uint32_t *>(group_stat + p.G);  // [R * rpi]
    for (int base = lo; base < hi; base += R * p.rpi) {  // block-uniform
      for (int i = threadIdx.x; i < R * p.rpi; i += blockDim.x) row_max[i] = 0u;
      __syncthreads();
      float z[R][V];
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int s = base + row + j * p.rpi;
        if (!live || s >= hi) continue;
        T v[V];
        VecIO<T, V, true>::load(x + s * p.xs, v);
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float zz = __fmaf_rn(to_f32<T>(v[i]) - mean[i], scale[i], shift[i]);
          z[j][i] = p.silu ? silu(zz) : zz;
          m = fmaxf(m, fabsf(z[j][i]));
        }
        atomicMax(&row_max[row + j * p.rpi], __float_as_uint(m));  // order-independent
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int s = base + row + j * p.rpi;
        if (!live || s >= hi) continue;
        const float amax = __uint_as_float(row_max[row + j * p.rpi]);
        const float sc = (amax == 0.0f) ? 0.0f : __fdiv_rn(amax, 127.0f);
        const bool fast = quant_fast_ok(sc);
        const float rc = fast ? __frcp_rn(sc) : 0.0f;
        static_assert(V == 8, "int8 rows are made of bf16 activations");
        uint32_t code[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
          code[i] = fast ? quant_fast(z[j][i], sc, rc) : quant_exact(z[j][i], sc);
        const int64_t pix = static_cast<int64_t>(b) * p.S + s;
        *reinterpret_cast<uint2 *>(p.q + pix * p.C + vec * V) =
            sc == 0.0f ? make_uint2(0u, 0u) : pack_codes(code);
        if (vec == 0) p.s_q[pix] = sc;
      }
      __syncthreads();
    }
  }
}

// y'(z) for SiLU: sigma + z sigma (1 - sigma).
__device__ __forceinline__ float silu_grad(float z) {
  const float sig = __fdividef(1.0f, 1.0f + __expf(-z));
  return sig * (1.0f + z * (1.0f - sig));
}

// Backward sums of one slab: per channel (sum dz, sum dz xh) into chan, per
// group (sum w dz, sum w dz xh) into part.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_grad_sums_kernel(const NormParams p) {
  constexpr int V = kNormVec<T>;
  constexpr int R = 4;
  extern __shared__ float2 chan_sum[];  // [rpi][C]
  const int b = blockIdx.x / p.slabs, slab = blockIdx.x - b * p.slabs;
  int lo, hi;
  slab_range(p.S, p.slabs, slab, lo, hi);
  const int c = p.C / p.G;
  const int row = threadIdx.x / p.tpr, vec = threadIdx.x - row * p.tpr;
  if (row < p.rpi) {
    float mean[V], rstd[V], w[V], bias[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int ch = vec * V + i;
      mean[i] = p.mean_in[static_cast<int64_t>(b) * p.G + ch / c];
      rstd[i] = p.rstd_in[static_cast<int64_t>(b) * p.G + ch / c];
      w[i] = norm_param(p.weight, p.param_f32, ch, 1.0f, static_cast<const T *>(nullptr));
      bias[i] = norm_param(p.bias, p.param_f32, ch, 0.0f, static_cast<const T *>(nullptr));
    }
    const T *x = static_cast<const T *>(p.x) + b * p.xb + vec * V;
    const T *dy = static_cast<const T *>(p.dy) + b * p.dyb + vec * V;
    float s1[V], s2[V];
#pragma unroll
    for (int i = 0; i < V; ++i) s1[i] = s2[i] = 0.0f;
    for (int s0 = lo + row; s0 < hi; s0 += R * p.rpi) {
      T xv[R][V], gv[R][V];
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int s = s0 + j * p.rpi;
        if (s < hi) {
          VecIO<T, V, true>::load(x + s * p.xs, xv[j]);
          VecIO<T, V, true>::load(dy + s * p.dys, gv[j]);
        }
      }
      float t1[V], t2[V];  // sums of the batch join the running ones once
#pragma unroll
      for (int i = 0; i < V; ++i) t1[i] = t2[i] = 0.0f;
#pragma unroll
      for (int j = 0; j < R; ++j) {
        if (s0 + j * p.rpi >= hi) break;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float xh = (to_f32<T>(xv[j][i]) - mean[i]) * rstd[i];
          float dz = to_f32<T>(gv[j][i]);
          if (p.silu) dz *= silu_grad(__fmaf_rn(xh, w[i], bias[i]));
          t1[i] += dz;
          t2[i] = __fmaf_rn(dz, xh, t2[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s1[i] += t1[i];
        s2[i] += t2[i];
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) chan_sum[row * p.C + vec * V + i] = make_float2(s1[i], s2[i]);
  }
  __syncthreads();
  const int64_t slot = static_cast<int64_t>(b) * p.slabs + slab;
  for (int ch = threadIdx.x; ch < p.C; ch += blockDim.x) {
    float2 t = chan_sum[ch];
    for (int r = 1; r < p.rpi; ++r) {
      t.x += chan_sum[r * p.C + ch].x;
      t.y += chan_sum[r * p.C + ch].y;
    }
    p.chan[slot * p.C + ch] = t;
    const float w = norm_param(p.weight, p.param_f32, ch, 1.0f, static_cast<const T *>(nullptr));
    chan_sum[ch] = make_float2(w * t.x, w * t.y);  // this thread's own entries
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  for (int g = warp; g < p.G; g += warps) {
    float a = 0.0f, d = 0.0f;
    for (int i = lane; i < c; i += 32) {
      a += chan_sum[g * c + i].x;
      d += chan_sum[g * c + i].y;
    }
    a = warp_sum(a);
    d = warp_sum(d);
    if (lane == 0) p.part[slot * p.G + g] = make_float2(a, d);
  }
}

// dw and db: one warp per channel adds the slabs' sums in a fixed order.
__global__ void __launch_bounds__(256) norm_grad_params_kernel(const NormParams p) {
  const int ch = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (ch >= p.C) return;
  float a = 0.0f, d = 0.0f;
  const int64_t slots = static_cast<int64_t>(p.B) * p.slabs;
  for (int64_t j = lane; j < slots; j += 32) {
    const float2 t = p.chan[j * p.C + ch];
    a += t.x;
    d += t.y;
  }
  a = warp_sum(a);
  d = warp_sum(d);
  if (lane == 0) {
    if (p.dbias != nullptr) p.dbias[ch] = a;
    if (p.dweight != nullptr) p.dweight[ch] = d;
  }
}

// dx of one slab.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_grad_apply_kernel(const NormParams p) {
  constexpr int V = kNormVec<T>;
  constexpr int R = 4;
  extern __shared__ float2 group_sum[];  // [G]: (1/n) sum w dz, (1/n) sum w dz xh
  const int b = blockIdx.x / p.slabs, slab = blockIdx.x - b * p.slabs;
  int lo, hi;
  slab_range(p.S, p.slabs, slab, lo, hi);
  const int c = p.C / p.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  {
    const float inv_n = 1.0f / (static_cast<float>(p.S) * c);
    for (int g = warp; g < p.G; g += warps) {
      float a = 0.0f, d = 0.0f;
      for (int j = lane; j < p.slabs; j += 32) {
        const float2 t = p.part[(static_cast<int64_t>(b) * p.slabs + j) * p.G + g];
        a += t.x;
        d += t.y;
      }
      a = warp_sum(a);
      d = warp_sum(d);
      if (lane == 0) group_sum[g] = make_float2(a * inv_n, d * inv_n);
    }
  }
  __syncthreads();
  const int row = threadIdx.x / p.tpr, vec = threadIdx.x - row * p.tpr;
  if (row >= p.rpi) return;
  float mean[V], rstd[V], w[V], bias[V], c1[V], c2[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int ch = vec * V + i;
    mean[i] = p.mean_in[static_cast<int64_t>(b) * p.G + ch / c];
    rstd[i] = p.rstd_in[static_cast<int64_t>(b) * p.G + ch / c];
    w[i] = norm_param(p.weight, p.param_f32, ch, 1.0f, static_cast<const T *>(nullptr));
    bias[i] = norm_param(p.bias, p.param_f32, ch, 0.0f, static_cast<const T *>(nullptr));
    c1[i] = group_sum[ch / c].x;
    c2[i] = group_sum[ch / c].y;
  }
  const T *x = static_cast<const T *>(p.x) + b * p.xb + vec * V;
  const T *dy = static_cast<const T *>(p.dy) + b * p.dyb + vec * V;
  T *dx = static_cast<T *>(p.y) + b * p.yb + vec * V;
  for (int s0 = lo + row; s0 < hi; s0 += R * p.rpi) {
    T xv[R][V], gv[R][V];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int s = s0 + j * p.rpi;
      if (s < hi) {
        VecIO<T, V, true>::load(x + s * p.xs, xv[j]);
        VecIO<T, V, true>::load(dy + s * p.dys, gv[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int s = s0 + j * p.rpi;
      if (s >= hi) break;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float xh = (to_f32<T>(xv[j][i]) - mean[i]) * rstd[i];
        float dz = to_f32<T>(gv[j][i]);
        if (p.silu) dz *= silu_grad(__fmaf_rn(xh, w[i], bias[i]));
        gv[j][i] = from_f32<T>(rstd[i] * (__fmaf_rn(w[i], dz, -c1[i]) - xh * c2[i]));
      }
      VecIO<T, V, true>::store(dx + s * p.ys, gv[j]);
    }
  }
}

}  // namespace w8a8
