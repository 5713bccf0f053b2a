// w8a8_norm.cuh -- group normalization of channels-last tensors, with SiLU.
//
// x [B, S, C] (S pixels of C channels, channels adjacent), G groups of
// c = C / G adjacent channels.  Over the S * c values of a sample's group:
//   mean = E x,  rstd = 1 / sqrt(E (x - mean)^2 + eps)
//   z = (x - mean) * rstd * w + b,  y = z or z * sigmoid(z)
// The int8 form quantizes each pixel's row of y (fp32, not rounded to bf16
// first) for the W8A8 layer that follows: s = max|y| / 127, q = rint(y (127 / max|y|));
// a NaN in a row makes its scale NaN.
// Backward, with xh = (x - mean) * rstd, n = S * c and dz = dy * y'(z):
//   dw = sum dz * xh,  db = sum dz   (over samples and pixels)
//   dx = rstd * (w dz - (1/n) sum w dz - xh * (1/n) sum w dz xh)
//
// Every form needs a sum over a whole sample before it can write its first
// value, and is bound by memory: one read of the inputs, one write.  One
// launch does both passes.  A sample's pixels are cut into slabs, one per
// block, one block per SM, all resident at once (a cooperative launch).  The
// first warp streams the slab through a ring of shared memory with bulk
// copies; all warps reduce each chunk as it lands.  The last chunks
// of the first pass stay in the ring, so a slab of up to 192 KB (28 MB over
// the GPU) is read once; of longer ones the second pass, which runs backwards,
// reads the rest again, the most recently read chunks first.
//
// Measured in a graph: 1048576 x 128 in bf16 with SiLU 150 us (537 MB once; 776
// with what is read twice, 5.2 TB/s), twice as many pixels 285 (5.7 TB/s, the
// same without SiLU: memory); 2 x 4096 x 1280 to int8 rows 23; gradient of 4 x
// 4096 x 512 26.5.  Below the ring's size latency is what is left: 9 us for 2 x 64
// x 1280 (launch, first loads, one exchange).
//
// Statistics: a thread keeps one 16-byte vector of channels; batches of rows
// are reduced in two passes over registers (mean, then squared deviations)
// and joined by the pairwise update of Chan, Golub and LeVeque (1979), which
// takes no difference of large squares.  The mean itself, of a thread and of the
// group, is one fp32 value, off by some 2^-24 of its size per join, and x - mean
// is off by as much: a group whose mean is m standard deviations from zero
// loses about log2(m) bits (of rstd, too, where it has few values; over many
// the joins' errors cancel).  All joins run in a fixed order (no atomics on
// sums): equal inputs give equal bits.
//
// The blocks of a sample exchange (mean, squared deviations) or the gradient's
// two sums per group through 16-byte entries that carry their launch's tag and
// are read and written as one 128-bit access, so an entry is valid exactly
// when its tag is: one round trip, no barrier and nothing to clear beforehand.
// Each block marks (tagged too) that it has read them; the sample's first block
// waits for the marks beside its second pass and takes all tags back, so a
// replayed graph, whose launches carry the same tag, finds none of its own.
// The channels' sums of dw and db go the same way, one warp per channel reading
// (and clearing) every block's entry beside the second pass (4 x 4096 x 512:
// 26.8 us; 27.7 after the second pass, 28.4 in a launch of their own).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <type_traits>

#include "w8a8_gemm.cuh"
#include "w8a8_ptx.cuh"
#include "w8a8_quant.cuh"
#include "w8a8_rotary.cuh"

namespace w8a8 {

constexpr int kNormThreads = 512;  // rpi rows of tpr threads, the rest idle
constexpr int kNormWarps = kNormThreads / 32;
constexpr int kNormMaxVecs = 512;  // 16-byte vectors of a pixel: 4096 channels, 2048 in fp32
constexpr int kNormMaxSlots = 8;

// What a launch computes.
constexpr int kNormForward = 0, kNormQuant = 1, kNormBackward = 2;
// Rows of a chunk per thread.
template <int MODE>
constexpr int kNormRows = MODE == kNormBackward ? 2 : 4;

struct NormParams {
  const void *x, *dy;
  void *y;                           // y, or dx
  int64_t xb, xs, dyb, dys, yb, ys;  // strides of a sample and a pixel, elements
  int32_t B, S, C, G;
  int32_t tpr, rpi;                  // threads per row, rows per block iteration
  int32_t group_channels;            // C / G
  int32_t slab_part, slab_extra;     // S over slabs: quotient and remainder
  int32_t chunks, chunks_longer;     // of a slab of slab_part pixels, and of one more
  int32_t many, many_longer;         // its pixels over rpi
  int32_t row_entries;               // (C / G) / run
  int32_t run;                       // channels of a vector that surely share a group
  int32_t group_shift;               // 2^group_shift threads join a group: 32, fewer where groups are many
  int32_t slabs;                     // blocks sharing a sample
  int32_t teams;                     // samples in flight: gridDim.y
  int32_t slots, chunk_bytes;        // of one tensor
  const void *weight, *bias;         // [C] in x's type or fp32, 16-byte aligned, or nullptr
  int32_t param_f32;
  float eps;
  uint4 *entries;                    // [B][G][slabs] (slabs > 1)
  unsigned long long *readers;       // [B][slabs] (slabs > 1)
  unsigned long long tag;
  uint4 *chan;                       // [blocks][C]: entries of the channels' sums (backward)
  float2 *chan_run;                  // [blocks][C]: the same over a block's samples so far (B > teams)
  float *mean_out, *rstd_out;        // [B, G] or nullptr
  const float *mean_in, *rstd_in;
  int8_t *q;
  float *s_q;
  float *dweight, *dbias;            // [C] or nullptr
};

template <typename T>
constexpr int kNormVec = 16 / static_cast<int>(sizeof(T));

// A 16-byte vector as pairs of fp32 values, and back (rounded to nearest).
template <typename T>
struct Pairs;
template <>
struct Pairs<__nv_bfloat16> {
  __device__ static __forceinline__ void get(uint4 v, float2 (&f)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
  __device__ static __forceinline__ uint4 put(const float2 (&f)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[i].x, f[i].y);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Pairs<__half> {
  __device__ static __forceinline__ void get(uint4 v, float2 (&f)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
  }
  __device__ static __forceinline__ uint4 put(const float2 (&f)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[i].x, f[i].y);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Pairs<float> {
  __device__ static __forceinline__ void get(uint4 v, float2 (&f)[2]) {
    f[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  __device__ static __forceinline__ uint4 put(const float2 (&f)[2]) {
    return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                      __float_as_uint(f[1].y));
  }
};

// The parameters of V adjacent channels from ch on (`none` where there are
// none): one or two 16-byte loads, no load behind a branch on another's value.
template <typename T>
__device__ __forceinline__ void norm_param(const void *p, int f32, int ch, float none,
                                           float2 (&out)[kNormVec<T> / 2]) {
  constexpr int V = kNormVec<T>;
  if (p == nullptr) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) out[i] = make_float2(none, none);
  } else if (f32) {
    const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + ch);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const float4 v = __ldg(q + i);
      out[2 * i] = make_float2(v.x, v.y);
      out[2 * i + 1] = make_float2(v.z, v.w);
    }
  } else {
    Pairs<T>::get(__ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(p) + ch)), out);
  }
}

// f(i, its group) for V adjacent channels, the first of them channel `in` of
// group g, c a group.
template <int V, typename F>
__device__ __forceinline__ void each_group(int g, int in, int c, F f) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    f(i, g);
    if (++in == c) {
      in = 0;
      ++g;
    }
  }
}

// Component i of an array of pairs.
template <int H>
__device__ __forceinline__ float &at(float2 (&v)[H], int i) {
  return (i & 1) ? v[i >> 1].y : v[i >> 1].x;
}

// sigmoid of two values: 1 / (1 + 2^(-z log2 e)).  The power may overflow: the
// gate is then 0, as it is from z = -87.3 on, where it leaves fp32's normal
// numbers (z * sigmoid(z) is off by less than 2^-119 there).  A reciprocal each:
// one for both, 1 / a = b / (a b), takes a quarter less of the special-function unit
// (16 a clock and SM), but needs its powers held below 2^63, which stops the gate
// at 2^-63, or formed from |z|, whose selections cost more than they save
// (1048576 x 128 forward: 150.2 us; 148.4 stopped, 155.6 from |z|; gradient of
// 4 x 4096 x 512: 26.4, 26.6, 27.5).
__device__ __forceinline__ float2 sigmoid2(float2 z) {
  const float2 t = mul2_rn(z, make_float2(-1.4426950408889634f, -1.4426950408889634f));
  float2 e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  const float2 d = add2_rn(e, make_float2(1.0f, 1.0f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
  return r;
}

// Sum over the warp in a fixed order.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

__device__ __forceinline__ void entry_store(uint4 *p, float2 v, unsigned long long tag) {
  const unsigned long long lo = (static_cast<unsigned long long>(__float_as_uint(v.y)) << 32) |
                                __float_as_uint(v.x);
  asm volatile("{\n\t.reg .b128 q;\n\tmov.b128 q, {%1, %2};\n\tst.relaxed.gpu.global.b128 [%0], q;\n\t}" ::"l"(p),
               "l"(lo), "l"(tag)
               : "memory");
}

__device__ __forceinline__ unsigned long long entry_load(const uint4 *p, float2 &v) {
  unsigned long long lo, tag;
  asm volatile("{\n\t.reg .b128 q;\n\tld.relaxed.gpu.global.b128 q, [%2];\n\tmov.b128 {%0, %1}, q;\n\t}"
               : "=l"(lo), "=l"(tag)
               : "l"(p)
               : "memory");
  v = make_float2(__uint_as_float(static_cast<uint32_t>(lo)), __uint_as_float(static_cast<uint32_t>(lo >> 32)));
  return tag;
}

// The entry at p once it carries `tag` (bounded like every other wait).
__device__ __forceinline__ bool entry_wait(const uint4 *p, unsigned long long tag, float2 &v,
                                           volatile int *abort_flag) {
  if (entry_load(p, v) == tag) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t i = 1;; ++i) {
    if (entry_load(p, v) == tag) return true;
    if ((i & 15u) == 0u) {
      if (*abort_flag) return false;
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        atomicOr(&g_device_error, W8A8_DEVERR_TIMEOUT);
        return false;
      }
    }
  }
}

// One warp's loads of a chunk: `rows` rows of `row_bytes` bytes, `step` bytes
// apart, into dst (adjacent rows in one copy).
__device__ __forceinline__ void norm_load_rows(uint8_t *dst, const uint8_t *src, int rows,
                                               uint32_t row_bytes, int64_t step, uint64_t *bar,
                                               int lane) {
  if (step == static_cast<int64_t>(row_bytes)) {
    if (lane == 0) bulk_load_g2s(dst, src, rows * row_bytes, bar);
  } else {
    for (int r = lane; r < rows; r += 32)
      bulk_load_g2s(dst + r * row_bytes, src + r * step, row_bytes, bar);
  }
}

template <typename T, int MODE, bool SILU>
__global__ void __launch_bounds__(kNormThreads, 1) norm_kernel(const __grid_constant__ NormParams p) {
  constexpr int V = kNormVec<T>, H = V / 2;  // values and pairs of a vector
  constexpr int K = kNormRows<MODE>;
  constexpr bool BWD = MODE == kNormBackward;
  extern __shared__ __align__(128) uint8_t norm_smem[];
  __shared__ uint64_t full[kNormMaxSlots], empty[kNormMaxSlots];
  __shared__ int abort_flag;
  const int NS = p.slots;
  const int slot_bytes = p.chunk_bytes * (BWD ? 2 : 1);
  // [slots][x rows, dy rows] | the statistics' region | [slots] row maxima (int8 form)
  float2 *region = reinterpret_cast<float2 *>(norm_smem + NS * slot_bytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int chunk_rows = p.rpi * K;
  const uint32_t row_bytes = static_cast<uint32_t>(p.C) * sizeof(T);
  // pixels [lo, lo + pixels) of the samples team, team + teams, ...: the first
  // slabs one more
  const int slab = blockIdx.x;
  const bool longer = slab < p.slab_extra;
  const int lo = slab * p.slab_part + (longer ? slab : p.slab_extra);
  const int pixels = p.slab_part + (longer ? 1 : 0);
  const int chunks = longer ? p.chunks_longer : p.chunks;

  // ---- loads, issued by the first warp.  A slot is filled again once all
  // warps have released it; the refill is asked for a chunk later, when the
  // others have caught up.
  uint32_t used = 0, empty_par = 0, fill_par = 0;  // bit s: slot s (first warp)
  uint32_t full_par = 0;
  bool ok = true;  // after a wait gave up the flow goes on, but stores nothing
  auto fill = [&](int b, int chunk, int s) {
    const uint32_t bit = 1u << s;
    if (used & bit) {
      if (ok) ok = mbar_wait(&empty[s], (empty_par & bit) ? 1u : 0u, &abort_flag);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) return;
      empty_par ^= bit;
      fill_par ^= bit;
    }
    used |= bit;
    const int r0 = lo + chunk * chunk_rows;
    const int rows = lo + pixels - r0 < chunk_rows ? lo + pixels - r0 : chunk_rows;
    if (lane == 0) mbar_arrive_expect_tx(&full[s], rows * row_bytes * (BWD ? 2u : 1u));
    __syncwarp();
    uint8_t *dst = norm_smem + s * slot_bytes;
    norm_load_rows(dst, static_cast<const uint8_t *>(p.x) + (b * p.xb + r0 * p.xs) * static_cast<int64_t>(sizeof(T)),
                   rows, row_bytes, p.xs * static_cast<int64_t>(sizeof(T)), &full[s], lane);
    if constexpr (BWD)
      norm_load_rows(dst + p.chunk_bytes,
                     static_cast<const uint8_t *>(p.dy) + (b * p.dyb + r0 * p.dys) * static_cast<int64_t>(sizeof(T)),
                     rows, row_bytes, p.dys * static_cast<int64_t>(sizeof(T)), &full[s], lane);
  };
  const int row = tid / p.tpr, vec = tid - row * p.tpr;
  const bool live = row < p.rpi;
  const bool parameters = BWD && (p.dweight != nullptr || p.dbias != nullptr);
  const int c = p.group_channels;
  const int group0 = vec * V / c, in0 = vec * V - group0 * c;  // the vector's first channel
  // Gradient: per channel rstd, -mean, weight and bias.  Loaded before the
  // first copies are asked for: a whole ring per block (28 MB over the GPU)
  // would be ahead of these few values (measured: 5.5 us of wait, 3.0 before).
  float2 rs[H], nm[H], wt[H], bs[H];
  auto load_params = [&](int b) {
    if (BWD && live) {
      norm_param<T>(p.weight, p.param_f32, vec * V, 1.0f, wt);
      norm_param<T>(p.bias, p.param_f32, vec * V, 0.0f, bs);
      const int64_t at0 = static_cast<int64_t>(b) * p.G;
      each_group<V>(group0, in0, c, [&](int i, int g) {
        at(nm, i) = -__ldg(p.mean_in + at0 + g);
        at(rs, i) = __ldg(p.rstd_in + at0 + g);
      });
    }
  };
  load_params(blockIdx.y);
  if constexpr (BWD) __syncthreads();
  if (warp == 0) {
    if (lane == 0) {
      for (int s = 0; s < NS; ++s) {
        mbar_init(&full[s], 1);
        mbar_init(&empty[s], kNormWarps);
      }
      abort_flag = 0;
      fence_mbarrier_init();
    }
    __syncwarp();
    for (int i = 0; i < NS && i < chunks; ++i) fill(blockIdx.y, i, i);
  }
  const uint32_t offset = static_cast<uint32_t>(row) * row_bytes + vec * 16u;
  const uint32_t row_step = static_cast<uint32_t>(p.rpi) * row_bytes;
  // this thread's rows of the last chunk
  int last_nb = 0;
#pragma unroll
  for (int k = 0; k < K; ++k)
    last_nb += live && (chunks - 1) * chunk_rows + row + k * p.rpi < pixels ? 1 : 0;
  __syncthreads();

  auto arrive_full = [&](int s) {
    if (ok) ok = mbar_wait(&full[s], (full_par >> s) & 1u, &abort_flag);
    full_par ^= 1u << s;
  };
  auto release = [&](int s) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);
  };

  for (int b = blockIdx.y; b < p.B; b += p.teams) {
    if (b != static_cast<int>(blockIdx.y)) {
      load_params(b);
      if (warp == 0)
        for (int i = 0; i < NS && i < chunks; ++i) fill(b, i, i);
    }
    // xh and dz of a vector (gradient)
    auto grad_vec = [&](uint4 xv, uint4 gv, float2 (&xh)[H], float2 (&dz)[H]) {
      Pairs<T>::get(xv, xh);
      Pairs<T>::get(gv, dz);
#pragma unroll
      for (int i = 0; i < H; ++i) {
        xh[i] = mul2_rn(add2_rn(xh[i], nm[i]), rs[i]);
        if constexpr (SILU) {  // y'(z) = s + z s (1 - s)
          const float2 z = fma2_rn(xh[i], wt[i], bs[i]);
          const float2 s = sigmoid2(z);
          const float2 zs = mul2_rn(z, s);
          const float2 d = add2_rn(s, fma2_rn(make_float2(-zs.x, -zs.y), s, zs));
          dz[i] = mul2_rn(dz[i], d);
        }
      }
    };

    // ---- first pass: per channel (mean, squared deviations), or the two sums
    float2 s1[H], s2[H];
#pragma unroll
    for (int i = 0; i < H; ++i) s1[i] = s2[i] = make_float2(0.0f, 0.0f);
    // One chunk's rows of this thread joined to the running values; `all`: K of
    // them (every chunk but the last), else nb.
    int n = 0;
    auto reduce = [&](const uint8_t *src, int nb, auto all) {
      constexpr bool ALL = decltype(all)::value;
      if constexpr (BWD) {
        float2 t1[H], t2[H];  // the chunk's sums join the running ones once
#pragma unroll
        for (int h = 0; h < H; ++h) t1[h] = t2[h] = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (ALL || k < nb) {
            float2 xh[H], dz[H];
            grad_vec(*reinterpret_cast<const uint4 *>(src + k * row_step),
                     *reinterpret_cast<const uint4 *>(src + p.chunk_bytes + k * row_step), xh, dz);
#pragma unroll
            for (int h = 0; h < H; ++h) {
              t1[h] = add2_rn(t1[h], dz[h]);
              t2[h] = fma2_rn(dz[h], xh[h], t2[h]);
            }
          }
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
          s1[h] = add2_rn(s1[h], t1[h]);
          s2[h] = add2_rn(s2[h], t2[h]);
        }
      } else {
        float2 v[K][H];
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (ALL || k < nb) Pairs<T>::get(*reinterpret_cast<const uint4 *>(src + k * row_step), v[k]);
        }
        const float inv = ALL ? 1.0f / K : 1.0f / nb;
        const float share = __fdividef(static_cast<float>(ALL ? K : nb), static_cast<float>(n + (ALL ? K : nb)));
        const float cross = share * n;
#pragma unroll
        for (int h = 0; h < H; ++h) {
          float2 sum = v[0][h];
#pragma unroll
          for (int k = 1; k < K; ++k)
            if (ALL || k < nb) sum = add2_rn(sum, v[k][h]);
          const float2 mb = mul2_rn(sum, make_float2(inv, inv));
          const float2 back = make_float2(-mb.x, -mb.y);
          float2 sq = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int k = 0; k < K; ++k) {
            if (ALL || k < nb) {
              const float2 d = add2_rn(v[k][h], back);
              sq = fma2_rn(d, d, sq);
            }
          }
          if (n == 0) {
            s1[h] = mb;
            s2[h] = sq;
          } else {
            const float2 delta = add2_rn(mb, make_float2(-s1[h].x, -s1[h].y));
            s1[h] = fma2_rn(delta, make_float2(share, share), s1[h]);
            sq = fma2_rn(mul2_rn(delta, delta), make_float2(cross, cross), sq);
            s2[h] = add2_rn(s2[h], sq);
          }
        }
      }
      n += ALL ? K : nb;
    };
    int slot = 0;
    for (int i = 0; i < chunks - 1; ++i) {
      arrive_full(slot);
      if (live) reduce(norm_smem + slot * slot_bytes + offset, K, std::true_type{});
      if (i + NS < chunks) release(slot);  // the last chunks stay for the second pass
      const int before = slot == 0 ? NS - 1 : slot - 1;
      if (warp == 0 && i > 0 && i - 1 + NS < chunks) fill(b, i - 1 + NS, before);
      slot = slot + 1 == NS ? 0 : slot + 1;
    }
    arrive_full(slot);
    if (last_nb == K)
      reduce(norm_smem + slot * slot_bytes + offset, K, std::true_type{});
    else if (last_nb > 0)
      reduce(norm_smem + slot * slot_bytes + offset, last_nb, std::false_type{});

    // ---- the slab's groups.  A thread first joins runs of `run` channels of
    // its vector that share a group; region[row][vec * (V / run) + i].
    const int run = p.run;                  // 1, 2, 4 or 8 channels
    const int width = p.row_entries * p.G;  // entries of a row
    const int cpg = p.row_entries;          // entries of a group in a row
    __syncthreads();  // the region is free again
    if (live) {
      float a[V], d[V];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        a[2 * h] = s1[h].x; a[2 * h + 1] = s1[h].y;
        d[2 * h] = s2[h].x; d[2 * h + 1] = s2[h].y;
      }
      if constexpr (BWD) {
        // the rows' sums: region [rpi][C]
#pragma unroll
        for (int i = 0; i < V; ++i) region[row * p.C + vec * V + i] = make_float2(a[i], d[i]);
      } else {
#pragma unroll
        for (int w = 1; w < V; w *= 2) {     // equal counts: mean of means
          if (w < run) {
            const float nw = 0.5f * n * w;
#pragma unroll
            for (int i = 0; i < V; i += 2 * w) {
              const float delta = a[i + w] - a[i];
              a[i] += 0.5f * delta;
              d[i] += d[i + w] + delta * delta * nw;
            }
          }
        }
        if (run == 1) {
#pragma unroll
          for (int i = 0; i < V; ++i) region[row * width + vec * V + i] = make_float2(a[i], d[i]);
        } else if (run == 2) {
#pragma unroll
          for (int i = 0; i < V / 2; ++i) region[row * width + vec * (V / 2) + i] = make_float2(a[2 * i], d[2 * i]);
        } else if (run == 4) {
#pragma unroll
          for (int i = 0; i < V / 4; ++i) region[row * width + vec * (V / 4) + i] = make_float2(a[4 * i], d[4 * i]);
        } else {
          region[row * width + vec] = make_float2(a[0], d[0]);
        }
      }
    }
    __syncthreads();
    if constexpr (BWD) {
      // per channel over the rows, to global memory; weighted in place
      for (int ch = tid; ch < p.C; ch += kNormThreads) {
        float2 t = region[ch];
#pragma unroll 4
        for (int r = 1; r < p.rpi; ++r) {
          t.x += region[r * p.C + ch].x;
          t.y += region[r * p.C + ch].y;
        }
        if (ok && parameters) {
          float2 all = t;  // over this block's samples
          const int64_t at0 = static_cast<int64_t>(blockIdx.y * gridDim.x + slab) * p.C + ch;
          if (b != static_cast<int>(blockIdx.y)) {
            const float2 before = p.chan_run[at0];
            all = make_float2(before.x + t.x, before.y + t.y);
          }
          if (b + p.teams < p.B) p.chan_run[at0] = all;
          else entry_store(p.chan + at0, all, p.tag);
        }
        float w = 1.0f;
        if (p.weight != nullptr)
          w = p.param_f32 ? __ldg(static_cast<const float *>(p.weight) + ch)
                          : to_f32<T>(static_cast<const T *>(p.weight)[ch]);
        region[ch] = make_float2(w * t.x, w * t.y);
      }
      __syncthreads();
    }
    // `lanes` neighbouring threads per group join its entries, publish them
    // or (alone) finish the group.  All groups at once up to 512 of them.
    float2 *stat = region + (BWD ? p.C : p.rpi * width);
    const float count = static_cast<float>(p.S) * c;  // values of a group
    uint4 *const entries = p.entries + static_cast<int64_t>(b) * p.G * p.slabs;
    const int lanes = 1 << p.group_shift, sub = tid & (lanes - 1);
    auto group_sum = [&](float v) {
      for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      return v;
    };
    auto finish = [&](float2 t) {
      return BWD ? make_float2(t.x / count, t.y / count) : make_float2(t.x, rsqrtf(t.y / count + p.eps));
    };
    const int gstep = kNormThreads >> p.group_shift;
#pragma unroll 1
    for (int g0 = 0; g0 < p.G; g0 += gstep) {  // whole warps stay together
      const int g = g0 + (tid >> p.group_shift);
      float2 mine = make_float2(0.0f, 0.0f);
      if constexpr (BWD) {
        if (g < p.G) {
          for (int e = sub; e < c; e += lanes) {
            mine.x += region[g * c + e].x;
            mine.y += region[g * c + e].y;
          }
        }
        mine = make_float2(group_sum(mine.x), group_sum(mine.y));
      } else {
        // entry e: `run` channels of the group in row e / cpg, standing for
        // the row's pixels.  Rows below pixels % rpi have one pixel more.
        const int many = longer ? p.many_longer : p.many, more = pixels - many * p.rpi;
        const int total = p.rpi * cpg;
        const float2 *from = region + g * cpg;
        if (g < p.G) {
          int r = 0, col = sub;
          for (; col >= cpg; col -= cpg) ++r;
          for (int e = sub; e < total; e += lanes) {
            mine.x += static_cast<float>(many + (r < more ? 1 : 0)) * from[r * width + col].x;
            for (col += lanes; col >= cpg; col -= cpg) ++r;
          }
        }
        const float mean = group_sum(mine.x) / (static_cast<float>(pixels) * cpg);
        if (g < p.G) {
          int r = 0, col = sub;
          for (; col >= cpg; col -= cpg) ++r;
          for (int e = sub; e < total; e += lanes) {
            const float2 st = from[r * width + col];
            const float dd = st.x - mean;
            mine.y += st.y + static_cast<float>(many + (r < more ? 1 : 0)) * run * dd * dd;
            for (col += lanes; col >= cpg; col -= cpg) ++r;
          }
        }
        mine = make_float2(mean, group_sum(mine.y));
      }
      if (sub == 0 && g < p.G) {
        if (p.slabs == 1) stat[g] = finish(mine);
        else if (ok) entry_store(entries + static_cast<int64_t>(g) * p.slabs + slab, mine, p.tag);
      }
    }
    // what the second pass needs of the parameters, while the entries travel
    float2 wt2[H], bs2[H];
    if constexpr (!BWD) {
      if (live) {
        norm_param<T>(p.weight, p.param_f32, vec * V, 1.0f, wt2);
        norm_param<T>(p.bias, p.param_f32, vec * V, 0.0f, bs2);
      }
    }
    // ---- the sample's groups, from every block's entry
    if (p.slabs > 1) {
      constexpr int E = 5;  // entries a lane has under way at once
      const int part = p.slab_part, extra = p.slab_extra;
#pragma unroll 1
      for (int g0 = 0; g0 < p.G; g0 += gstep) {
        const int g = g0 + (tid >> p.group_shift);
        const uint4 *e = entries + static_cast<int64_t>(g) * p.slabs;
        float2 t = make_float2(0.0f, 0.0f);  // this lane's mean and deviations, or sums
        float have = 0.0f;                   // pixels they stand for
#pragma unroll 1
        for (int j0 = 0; j0 < p.slabs; j0 += E * lanes) {
          float2 v[E];
          unsigned long long tag[E];
#pragma unroll
          for (int u = 0; u < E; ++u) {
            const int j = j0 + sub + lanes * u;
            tag[u] = p.tag;
            v[u] = make_float2(0.0f, 0.0f);
            if (j < p.slabs && g < p.G) tag[u] = entry_load(e + j, v[u]);
          }
#pragma unroll
          for (int u = 0; u < E; ++u) {
            if (tag[u] != p.tag && ok) ok = entry_wait(e + j0 + sub + lanes * u, p.tag, v[u], &abort_flag);
          }
          if constexpr (BWD) {
#pragma unroll
            for (int u = 0; u < E; ++u) {
              t.x += v[u].x;
              t.y += v[u].y;
            }
          } else {
            float pix = 0.0f, mean = 0.0f, dev = 0.0f;
#pragma unroll
            for (int u = 0; u < E; ++u) {
              const int j = j0 + sub + lanes * u;
              const float n = j < p.slabs ? static_cast<float>(part + (j < extra ? 1 : 0)) : 0.0f;
              pix += n;
              mean += n * v[u].x;
            }
            if (pix > 0.0f) {
              mean /= pix;
#pragma unroll
              for (int u = 0; u < E; ++u) {
                const int j = j0 + sub + lanes * u;
                const float n = j < p.slabs ? static_cast<float>(part + (j < extra ? 1 : 0)) : 0.0f;
                const float dd = v[u].x - mean;
                dev += v[u].y + n * c * dd * dd;
              }
              const float delta = mean - t.x, share = pix / (have + pix);
              t.y += dev + delta * delta * share * have * c;
              t.x += delta * share;
              have += pix;
            }
          }
        }
        if constexpr (BWD) {
          t = make_float2(group_sum(t.x), group_sum(t.y));
        } else {
          const float mean = group_sum(have * t.x) / static_cast<float>(p.S);
          const float dd = t.x - mean;
          t = make_float2(mean, group_sum(t.y + have * c * dd * dd));
        }
        if (sub == 0 && g < p.G) stat[g] = finish(t);
      }
      ok = __all_sync(0xFFFFFFFFu, ok);
    }
    __syncthreads();
    // This block has read the sample's entries: the barrier puts its threads'
    // loads before this store, whose release pairs with the acquire of the block
    // that overwrites them.  A warp in the middle: the fence would keep the first
    // from its loads and the last from the channels' sums (2 x 64 x 1280: 8.7 us;
    // 8.9 from the first).
    if (p.slabs > 1 && tid == kNormThreads / 2 && ok)
      st_release_gpu_u64(p.readers + static_cast<int64_t>(b) * p.slabs + slab, p.tag);
    if constexpr (BWD) {
      // dw and db: a warp per channel (the last warps: the first one loads) adds
      // the blocks' sums in a fixed order, as the others start on the second
      // pass.  Each is read once, and its tag goes with that.
      const int blocks = gridDim.x * gridDim.y, block = blockIdx.y * gridDim.x + blockIdx.x;
      for (int ch = block + (kNormWarps - 1 - warp) * blocks; parameters && b + p.teams >= p.B && ch < p.C; ch += blocks * kNormWarps) {
        constexpr int E = 5;  // entries a lane has under way at once
        float a = 0.0f, d = 0.0f;
#pragma unroll 1
        for (int j0 = lane; j0 < blocks; j0 += 32 * E) {
          float2 v[E];
          unsigned long long tag[E];
#pragma unroll
          for (int u = 0; u < E; ++u) {
            const int j = j0 + 32 * u;
            tag[u] = p.tag;
            v[u] = make_float2(0.0f, 0.0f);
            if (j < blocks) tag[u] = entry_load(p.chan + static_cast<int64_t>(j) * p.C + ch, v[u]);
          }
#pragma unroll
          for (int u = 0; u < E; ++u) {
            uint4 *const e = p.chan + static_cast<int64_t>(j0 + 32 * u) * p.C + ch;
            if (tag[u] != p.tag && ok) ok = entry_wait(e, p.tag, v[u], &abort_flag);
            if (ok && j0 + 32 * u < blocks) entry_store(e, make_float2(0.0f, 0.0f), 0ull);
            a += v[u].x;
            d += v[u].y;
          }
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        a = warp_sum(a);
        d = warp_sum(d);
        if (lane == 0 && ok) {
          if (p.dbias != nullptr) p.dbias[ch] = a;
          if (p.dweight != nullptr) p.dweight[ch] = d;
        }
      }
    }
    if (!BWD && slab == 0 && p.mean_out != nullptr && ok) {
      for (int g = tid; g < p.G; g += kNormThreads) {
        p.mean_out[static_cast<int64_t>(b) * p.G + g] = stat[g].x;
        p.rstd_out[static_cast<int64_t>(b) * p.G + g] = stat[g].y;
      }
    }

    // ---- second pass, backwards
    // forward: y = act((x + k3) * k1 + k2); gradient: dx = dz * k1 + k2 + xh * k3
    float2 k1[H], k2[H], k3[H];
    if (live) {
      each_group<V>(group0, in0, c, [&](int i, int g) {
        const float2 st = stat[g];
        if constexpr (BWD) {
          const float r = at(rs, i);
          at(k1, i) = r * at(wt, i);
          at(k2, i) = -r * st.x;
          at(k3, i) = -r * st.y;
        } else {
          at(k1, i) = st.y * at(wt2, i);
          at(k2, i) = at(bs2, i);
          at(k3, i) = -st.x;
        }
      });
    }
    // K rows (`all`), or nb of them: no branch between rows where there are K,
    // so that their work interleaves.  y of this thread's rows of a chunk:
    auto values = [&](const uint8_t *src, int k, float2 (&z)[H]) __attribute__((always_inline)) {
      const uint4 xv = *reinterpret_cast<const uint4 *>(src + k * row_step);
      if constexpr (BWD) {
        float2 xh[H];
        grad_vec(xv, *reinterpret_cast<const uint4 *>(src + p.chunk_bytes + k * row_step), xh, z);
#pragma unroll
        for (int h = 0; h < H; ++h) z[h] = fma2_rn(z[h], k1[h], fma2_rn(xh[h], k3[h], k2[h]));
      } else {
        Pairs<T>::get(xv, z);
#pragma unroll
        for (int h = 0; h < H; ++h) {
          z[h] = fma2_rn(add2_rn(z[h], k3[h]), k1[h], k2[h]);
          if constexpr (SILU) z[h] = mul2_rn(z[h], sigmoid2(z[h]));
        }
      }
    };
    if constexpr (MODE == kNormQuant) {
      // int8 rows.  Windows of up to a ring of chunks: first every row's
      // maximum, then the scales, then the codes, with a barrier between (y is
      // formed twice: a barrier per chunk, with y kept, took 10 us where this
      // takes 6, at 2 x 4096 x 1280).  Rows of a chunk without branches between
      // them and one thread per row for its scale: 262144 x 512 takes 167 us
      // (202 with each thread dividing for its rows, and a branch per row);
      // windows of half a ring, to load one while the other is rounded, 171.
      uint32_t *row_max = reinterpret_cast<uint32_t *>(stat + p.G);  // [slots][chunk_rows]
      const bool one_row = (p.tpr & 31) == 0;  // a warp's threads share a row
      const bool two_rows = p.tpr > 32 || p.tpr == 16;  // or lie in at most two
      const int first = __shfl_sync(0xFFFFFFFFu, row, 0);
      // One maximum per warp and row goes to shared memory (a warp holds one or
      // two rows, or several narrow ones; maxima do not depend on the order).
      auto maxima = [&](const uint8_t *src, uint32_t *mx, int nb, auto all) {
        constexpr bool ALL = decltype(all)::value;
        uint32_t mb[K];
#pragma unroll
        for (int k = 0; k < K; ++k) mb[k] = 0u;
        if (live) {
#pragma unroll
          for (int k = 0; k < K; ++k) {
            if (ALL || k < nb) {
              float2 z[H];
              values(src, k, z);
              float m = 0.0f;
#pragma unroll
              for (int h = 0; h < H; ++h) m = absmax_nan(absmax_nan(m, z[h].x), z[h].y);
              mb[k] = __float_as_uint(m);
            }
          }
        }
        if (one_row) {
#pragma unroll
          for (int k = 0; k < K; ++k) mb[k] = __reduce_max_sync(0xFFFFFFFFu, mb[k]);
          if (lane == 0 && live) {
#pragma unroll
            for (int k = 0; k < K; ++k) atomicMax(mx + row + k * p.rpi, mb[k]);
          }
        } else if (two_rows) {
#pragma unroll
          for (int k = 0; k < K; ++k) {
            const uint32_t m1 = __reduce_max_sync(0xFFFFFFFFu, row == first ? 0u : mb[k]);
            const uint32_t m0 = __reduce_max_sync(0xFFFFFFFFu, row == first ? mb[k] : 0u);
            if (lane == 0) {
              if (first < p.rpi) atomicMax(mx + first + k * p.rpi, m0);
              if (first + 1 < p.rpi) atomicMax(mx + first + 1 + k * p.rpi, m1);
            }
          }
        } else if (live) {
#pragma unroll
          for (int k = 0; k < K; ++k) atomicMax(mx + row + k * p.rpi, mb[k]);
        }
      };
      auto codes = [&](const uint8_t *src, const uint32_t *mx, int nb, int64_t pix, auto all) {
        constexpr bool ALL = decltype(all)::value;
        static_assert(V == 8, "int8 rows are made of bf16 activations");
        float r[K];
        bool plain = true;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          r[k] = __uint_as_float(mx[row + k * p.rpi]);
          if (ALL || k < nb) plain = plain && r[k] != 0.0f;
        }
        if (!ok) return;
        uint2 *to = reinterpret_cast<uint2 *>(p.q + pix * p.C + vec * V);
        const int64_t to_row = static_cast<int64_t>(p.rpi) * p.C / static_cast<int64_t>(sizeof(uint2));
        if (plain) {
          // rint(y * f), f = 127 / amax rounded once: the exact product enters
          // the rounding in one fused step.  The quotient y / s of the layer's
          // own quantization, by quant_fast, would take two reads and three
          // packed operations more (262144 x 512: 182 us against 167) and moves
          // a code only where y / s is within 127 * 2^-23 of a tie.
#pragma unroll
          for (int k = 0; k < K; ++k) {
            if (ALL || k < nb) {
              float2 z[H];
              values(src, k, z);
              uint32_t code[V];
#pragma unroll
              for (int h = 0; h < H; ++h) {
                const float2 t = fma2_rn(z[h], make_float2(r[k], r[k]), make_float2(kRintMagic, kRintMagic));
                code[2 * h] = __float_as_uint(t.x);
                code[2 * h + 1] = __float_as_uint(t.y);
              }
              to[k * to_row] = pack_codes(code);
            }
          }
        } else {
#pragma unroll 1
          for (int k = 0; k < (ALL ? K : nb); ++k) {
            const float sc = p.s_q[pix + k * p.rpi];  // this block's own, behind a barrier
            float2 z[H];
            values(src, k, z);
            uint32_t code[V];
#pragma unroll
            for (int h = 0; h < H; ++h) {
              code[2 * h] = sc == 0.0f ? 0u : quant_exact(z[h].x, sc);
              code[2 * h + 1] = sc == 0.0f ? 0u : quant_exact(z[h].y, sc);
            }
            to[k * to_row] = pack_codes(code);
          }
        }
      };
      for (int top = chunks - 1; top >= 0; top -= NS) {
        const int low = top - NS + 1 < 0 ? 0 : top - NS + 1;
        __syncthreads();  // the window before is done with the maxima
        for (int i = tid; i < NS * chunk_rows; i += kNormThreads) row_max[i] = 0u;
        __syncthreads();
        int s = slot;
        for (int i = top; i >= low; --i) {
          if (i < chunks - NS) arrive_full(s);
          const uint8_t *src = norm_smem + s * slot_bytes + offset;
          if (i < chunks - 1)
            maxima(src, row_max + s * chunk_rows, K, std::true_type{});
          else
            maxima(src, row_max + s * chunk_rows, last_nb, std::false_type{});
          s = s == 0 ? NS - 1 : s - 1;
        }
        __syncthreads();
        // The rows' scales, and in place of a maximum the factor of its codes:
        // 127 / amax, or 0 (divide) for a row of zeros, next to the subnormals,
        // where the factor leaves fp32, and where it nears them itself.
        s = slot;
        for (int i = top; i >= low; --i) {
          const int r0 = i * chunk_rows;
          for (int j = tid; j < chunk_rows && r0 + j < pixels; j += kNormThreads) {
            const float amax = __uint_as_float(row_max[s * chunk_rows + j]);
            if (ok) p.s_q[static_cast<int64_t>(b) * p.S + lo + r0 + j] = __fdiv_rn(amax, 127.0f);
            row_max[s * chunk_rows + j] =
                __float_as_uint(amax >= 1e-30f && amax <= 1e37f ? __fdiv_rn(127.0f, amax) : 0.0f);
          }
          s = s == 0 ? NS - 1 : s - 1;
        }
        __syncthreads();
        for (int i = top; i >= low; --i) {
          if (warp == 0 && i < top && i + 1 >= NS) fill(b, i + 1 - NS, slot + 1 == NS ? 0 : slot + 1);
          const uint8_t *src = norm_smem + slot * slot_bytes + offset;
          const int64_t pix = static_cast<int64_t>(b) * p.S + lo + static_cast<int64_t>(i) * chunk_rows + row;
          if (i < chunks - 1) {
            if (live) codes(src, row_max + slot * chunk_rows, K, pix, std::true_type{});
          } else if (last_nb > 0) {
            codes(src, row_max + slot * chunk_rows, last_nb, pix, std::false_type{});
          }
          release(slot);
          slot = slot == 0 ? NS - 1 : slot - 1;
        }
        // the next window's maxima need all of its chunks, the one that takes
        // the slot released last among them
        if (warp == 0 && low >= NS) fill(b, low - NS, slot + 1 == NS ? 0 : slot + 1);
      }
    } else {
      // where this thread's first row of a chunk goes, from the last chunk down
      uint8_t *dst = static_cast<uint8_t *>(p.y) +
                     (b * p.yb + (lo + static_cast<int64_t>(chunks - 1) * chunk_rows + row) * p.ys + vec * V) *
                         static_cast<int64_t>(sizeof(T));
      const int64_t dst_row = p.rpi * p.ys * static_cast<int64_t>(sizeof(T));
      const int64_t dst_chunk = dst_row * K;
      auto apply = [&](const uint8_t *src, int nb, auto all) {
        constexpr bool ALL = decltype(all)::value;
        float2 z[K][H];
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (ALL || k < nb) values(src, k, z[k]);
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (ALL || k < nb) *reinterpret_cast<uint4 *>(dst + k * dst_row) = Pairs<T>::put(z[k]);
      };
      for (int i = chunks - 1; i >= 0; --i) {
        if (i < chunks - NS) arrive_full(slot);
        if (warp == 0 && i + 1 < chunks && i + 1 >= NS) fill(b, i + 1 - NS, slot + 1 == NS ? 0 : slot + 1);
        const uint8_t *src = norm_smem + slot * slot_bytes + offset;
        if (i < chunks - 1 ? live : last_nb == K) {
          if (ok) apply(src, K, std::true_type{});
        } else if (i == chunks - 1 && last_nb > 0) {
          if (ok) apply(src, last_nb, std::false_type{});
        }
        release(slot);
        slot = slot == 0 ? NS - 1 : slot - 1;
        dst -= dst_chunk;
      }
    }
    if (p.slabs > 1 && slab == 0) {
      // Once every block has read the sample's entries, their tags go.  A wait
      // may have given up in some threads only, so all of them come to the
      // barrier.
      for (int j = tid; j < p.slabs && ok; j += kNormThreads) {
        unsigned long long *r = p.readers + static_cast<int64_t>(b) * p.slabs + j;
        const uint64_t t0 = global_timer_ns();
        for (uint32_t i = 1; ok && ld_acquire_gpu_u64(r) != p.tag; ++i) {
          if ((i & 15u) == 0u && global_timer_ns() - t0 > kWaitLimitNs) {
            abort_flag = 1;
            atomicOr(&g_device_error, W8A8_DEVERR_TIMEOUT);
            ok = false;
          }
        }
        if (ok) *reinterpret_cast<volatile unsigned long long *>(r) = 0ull;
      }
      ok = __syncthreads_and(ok);
      if (ok) {
        uint4 *e = p.entries + static_cast<int64_t>(b) * p.G * p.slabs;
        for (int i = tid; i < p.G * p.slabs; i += kNormThreads) entry_store(e + i, make_float2(0.0f, 0.0f), 0ull);
      }
    }
  }
  if (warp == 0 && !ok) {  // copies still in flight land before the block leaves
    for (int s = 0; s < NS; ++s) {
      volatile int never = 0;
      if (used & (1u << s)) mbar_wait(&full[s], (fill_par >> s) & 1u, &never);
    }
  }
}

}  // namespace w8a8
