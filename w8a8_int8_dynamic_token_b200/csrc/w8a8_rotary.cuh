// w8a8_rotary.cuh -- rotary positions on the heads a projection wrote.
//
// A head's first `rot` values are pairs (a, b): values i and i + rot / 2 in
// the half layout, 2i and 2i + 1 in the interleaved one.  Pair i of the token
// at position pos (along the axis that pair follows) turns by t = pos * f_i:
//   a' = scale * (a cos t - b sin t),   b' = scale * (a sin t + b cos t);
// the values behind `rot` are copied.  The gradient is the transposed map
// (t -> -t, the same scale).
//
// Angles.  A 32-bit product pos * f loses the angle of far positions, so the
// frequencies are held as turns per position in 64-bit fixed point, rounded to the
// nearest (with 1 / (2 pi) in 192 bits, see turns_q64): pos * f modulo one turn is
// then one wrapping 64-bit integer product, off by at most |pos| * 2^-65 turns
// (1.2e-8 radians at 2^36).  Its top 32 bits are taken relative to the nearest
// quarter turn, which leaves sincospif an angle off by 2.4e-8 radians at most.
//
// Bound by memory: every value is read once and written once.  A block takes
// one or a few tokens.  Each thread keeps one place within the head and one
// token, asks for its first heads' values, and only then computes its share of
// the block's cosines and sines (one sincospif per pair and token instead of
// one per pair, token and head) into shared memory: the loads cover the
// latency of positions and sines, and the factors stay in registers over the
// heads.  Blocks are small (128 threads where a head has up to 32 units) and
// registers held to 64, so that blocks in different phases share an SM:
// 16384 x 40 heads of 128 in fp16 take 56 us (6.0 TB/s), in blocks of 256
// threads 60, of 512 68, and 78 without the register limit.  A programmatic
// dependent launch on both sides hides the ramp: calls one after another of
// 4352 x 64 heads 28.1 -> 26.9 us, of 3027 x 16 heads of 256 in fp32 22.5 -> 20.9.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "w8a8_ptx.cuh"

namespace w8a8 {

constexpr int kRotMaxDim = 512;
constexpr int kRotMaxPairs = kRotMaxDim / 2;
constexpr int kRotMaxAxes = 8;
constexpr int kRotThreads = 512;  // at most
constexpr int kRotMaxTokens = 16;  // tokens a block takes at most
constexpr int kRotUnroll = 4;      // heads in flight per thread

// The heads of one tensor; strides in elements.
struct RotHeads {
  const void *x;
  void *y;
  int32_t heads;
  int64_t xb, xt, xh, yb, yt, yh;
};

struct RotParams {
  RotHeads t[2];
  int32_t total_heads;    // of both tensors
  int32_t batch, tokens;  // batch * tokens < 2^31
  int32_t dim, rot;
  int32_t block_tokens;   // tokens a block takes: divides by
  int32_t units;          // a head's units of work: rotated ones, then copied ones
  int32_t rot_units;
  int32_t bx, by;         // threads along the units; along tokens and heads
  const void *pos;
  int32_t pos_is_64, axes;
  int64_t pos_b, pos_t;   // strides of pos in elements; its axes are adjacent
  float scale;
  int32_t backward;
  unsigned long long freq[kRotMaxPairs];  // turns per position * 2^64
  uint8_t axis[kRotMaxPairs];
};

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }

// VEC values at p: one 16-byte access, or single values where WIDE is false.
template <typename T, int VEC, bool WIDE>
struct VecIO {
  __device__ static __forceinline__ void load(const T *p, T (&v)[VEC]) {
    if constexpr (WIDE) {
      static_assert(sizeof(T) * VEC == 16, "one 16-byte access");
      *reinterpret_cast<uint4 *>(v) = *reinterpret_cast<const uint4 *>(p);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = p[i];
    }
  }
  __device__ static __forceinline__ void store(T *p, const T (&v)[VEC]) {
    if constexpr (WIDE) {
      *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(v);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) p[i] = v[i];
    }
  }
};

// VEC: values of one access.  A unit is one access (interleaved, or copied
// values) or the two accesses of the same pairs (half layout).
template <typename T, int VEC, bool HALF, bool WIDE>
__global__ void __launch_bounds__(kRotThreads, 2)
    rotary_kernel(const __grid_constant__ RotParams p) {
  extern __shared__ float2 turn[];  // [block_tokens][rot / 2]: scale * (cos, sin)
  using IO = VecIO<T, VEC, WIDE>;
  constexpr int NP = HALF ? VEC : VEC / 2;  // pairs of a rotated unit
  constexpr int U = kRotUnroll;
  // a dependent reads only weights before its own wait, which completes after
  // this kernel and, through this wait, the one before it
  grid_dependents_launch();
  grid_dependency_wait();  // x and the positions may come from the preceding kernel
  const int pairs = p.rot >> 1, nt = p.block_tokens;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * nt;
  const int64_t total = static_cast<int64_t>(p.batch) * p.tokens;

  // this thread: unit u of the heads h, h + rows, ... of token tt of the block
  const int ty = threadIdx.x / p.bx, u = threadIdx.x - ty * p.bx;
  const int rows = p.by / nt;
  const int h_first = ty / nt, tt = ty - h_first * nt;
  const bool active = h_first < rows && first + tt < total;
  const bool rotated = u < p.rot_units;
  const int v0 = rotated ? u * VEC : p.rot + (u - p.rot_units) * VEC;  // first value in the head
  const int at = static_cast<int>(first) + tt;
  const int b = at / p.tokens, tok = at - b * p.tokens;
  T va[U][VEC], vb[HALF ? U : 1][VEC];
  // heads h, h + rows, ... (U of them): their place in x or y
  auto place = [&](int h, bool to) -> int64_t {
    const RotHeads &t = p.t[h >= p.t[0].heads ? 1 : 0];
    const int hh = h >= p.t[0].heads ? h - p.t[0].heads : h;
    return (to ? b * t.yb + tok * t.yt + hh * t.yh : b * t.xb + tok * t.xt + hh * t.xh) + v0;
  };
  auto load = [&](int h0) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int h = h0 + j * rows;
      if (h < p.total_heads) {
        const T *src = static_cast<const T *>(p.t[h >= p.t[0].heads ? 1 : 0].x) + place(h, false);
        IO::load(src, va[j]);
        if constexpr (HALF) {
          if (rotated) IO::load(src + pairs, vb[j]);
        }
      }
    }
  };
  if (active) load(h_first);

  const int here = total - first < nt ? static_cast<int>(total - first) : nt;
  for (int i = threadIdx.x; i < here * pairs; i += blockDim.x) {
    const int it = i / pairs, pair = i - it * pairs;
    const int iat = static_cast<int>(first) + it;
    const int ib = iat / p.tokens, itok = iat - ib * p.tokens;
    const int64_t off = ib * p.pos_b + itok * p.pos_t + p.axis[pair];
    const long long pos = p.pos_is_64 ? static_cast<const long long *>(p.pos)[off]
                                      : static_cast<const int *>(p.pos)[off];
    const unsigned long long turns = static_cast<unsigned long long>(pos) * p.freq[pair];
    // the nearest quarter turn, and the rest in half turns (within a quarter of
    // one: four times as fine in fp32 as the whole angle)
    const uint32_t hi = static_cast<uint32_t>(turns >> 32);
    const uint32_t quarter = (hi + (1u << 29)) >> 30;
    const int rest = static_cast<int>(hi - (quarter << 30));
    float s, c;
    sincospif(static_cast<float>(rest) * 4.656612873077393e-10f, &s, &c);
    if (quarter & 1u) {
      const float t = c;
      c = -s;
      s = t;
    }
    const float turned = quarter & 2u ? -p.scale : p.scale;
    turn[i] = make_float2(c * turned, (p.backward ? -s : s) * turned);
  }
  __syncthreads();
  if (!active) return;

  float cs[NP], sn[NP];
  if (rotated) {
    const float2 *f = turn + tt * pairs + (HALF ? v0 : v0 >> 1);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const float2 v = f[i];
      cs[i] = v.x;
      sn[i] = v.y;
    }
  }
  for (int h0 = h_first;;) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int h = h0 + j * rows;
      if (h >= p.total_heads) break;
      T *dst = static_cast<T *>(p.t[h >= p.t[0].heads ? 1 : 0].y) + place(h, true);
      if (rotated) {
        if constexpr (HALF) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const float x0 = to_f32<T>(va[j][i]), x1 = to_f32<T>(vb[j][i]);
            va[j][i] = from_f32<T>(__fmaf_rn(x0, cs[i], -(x1 * sn[i])));
            vb[j][i] = from_f32<T>(__fmaf_rn(x0, sn[i], x1 * cs[i]));
          }
          IO::store(dst + pairs, vb[j]);
        } else {
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const float x0 = to_f32<T>(va[j][2 * i]), x1 = to_f32<T>(va[j][2 * i + 1]);
            va[j][2 * i] = from_f32<T>(__fmaf_rn(x0, cs[i], -(x1 * sn[i])));
            va[j][2 * i + 1] = from_f32<T>(__fmaf_rn(x0, sn[i], x1 * cs[i]));
          }
        }
      }
      IO::store(dst, va[j]);
    }
    h0 += U * rows;
    if (h0 >= p.total_heads) break;
    load(h0);
  }
}

}  // namespace w8a8
