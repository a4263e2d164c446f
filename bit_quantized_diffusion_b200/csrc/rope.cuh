// rope.cuh -- rotary positions: the rotation of the heads of a row, and the tables of
// its angles' cosines and sines.
//
//   angle(m, i) = positions[m, axis[i]] * freq[i],   c = scale cos(angle), s = scale sin(angle)
//   pair (a, b) -> (a c - b s, b c + a s)
//   pairs: (2i, 2i + 1) interleaved, (i, i + P) in the half layout; columns from 2P on are copied
//
// Far positions: a float32 product position * freq is off by half a unit in its last
// place, 0.03 radians at 10^6. The angle is formed in whole turns instead, freq / 2 pi
// as a 64-bit binary fraction: position times that fraction modulo 2^64 is the angle's
// fraction of a turn, the wrap of the integer product being the range reduction. Its
// top 32 bits, as a signed number of turns in [-1/2, 1/2), go to sincospi. The
// fraction carries freq's 53 bits down to 2^-64 of a turn: the angle is off by 2^-52 of
// itself and 2^-64 turns per position.
#pragma once

#include "sm100.cuh"

namespace svdq {

constexpr int kRopeMaxPairs = 512;

struct RopeParams {
  int M, A, P;
  const void* positions;  // [M, A] int32 or int64
  int pos64;
  const double* freq;     // [P] radians per position
  const int* axis;        // [P] or null (0)
  float scale;
  // rotation
  int heads, D;
  const void* X;
  size_t ldx, ldhx;       // row and head strides, in elements
  void* Y;
  size_t ldy, ldhy;
  // tables
  float* cos;
  float* sin;
};

// radians per position -> turns per position as a fraction of 2^64 (whole turns drop out)
__device__ __forceinline__ uint64_t rope_fraction(double freq) {
  const double turns = freq * 0.15915494309189535;  // 1 / (2 pi)
  const double part = turns - floor(turns);         // [0, 1)
  return __double2ull_rd(part * 18446744073709551616.0);
}

__device__ __forceinline__ float2 rope_cos_sin(long long pos, uint64_t fraction, float scale) {
  const uint64_t turn = static_cast<uint64_t>(pos) * fraction;
  const float half_turns = static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f;  // 2^-31
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * scale, s * scale);
}

__device__ __forceinline__ long long rope_position(const RopeParams& p, size_t m, int axis) {
  const size_t at = m * p.A + axis;
  return p.pos64 ? static_cast<const long long*>(p.positions)[at]
                 : static_cast<long long>(static_cast<const int*>(p.positions)[at]);
}

template <typename T, int V>
struct alignas(sizeof(T) * V) RopeVec {
  T e[V];
};
__device__ __forceinline__ float rope_f(float v) { return v; }
__device__ __forceinline__ float rope_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void rope_put(float& d, float v) { d = v; }
__device__ __forceinline__ void rope_put(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }

// One block per (row, share of the heads). Its angles first, one per thread, into shared
// memory; then units of V adjacent elements (half layout: V of the first and V of the
// second half) over all its heads.
template <typename T, int V, bool kInterleaved>
__global__ void __launch_bounds__(256) rope_kernel(const RopeParams p) {
  __shared__ float2 cs[kRopeMaxPairs];
  const size_t m = blockIdx.x;
  grid_dep_wait();
  grid_dep_launch();
  for (int i = threadIdx.x; i < p.P; i += blockDim.x) {
    const int a = p.axis != nullptr ? p.axis[i] : 0;
    // an axis that the positions do not have gives NaN, and no read
    cs[i] = a >= 0 && a < p.A ? rope_cos_sin(rope_position(p, m, a), rope_fraction(p.freq[i]), p.scale)
                              : make_float2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff));
  }
  __syncthreads();
  const T* x = static_cast<const T*>(p.X) + m * p.ldx;
  T* y = static_cast<T*>(p.Y) + m * p.ldy;
  const int R = 2 * p.P;
  using Vec = RopeVec<T, V>;
  // a head's units: interleaved, its V-element vectors; half layout, first those that hold
  // pairs, then the copied ones
  const int turned = p.P / V;
  const int units = kInterleaved ? p.D / V : turned + (p.D - R) / V;
  const int total = units * p.heads;
  for (int u = blockIdx.y * blockDim.x + threadIdx.x; u < total; u += blockDim.x * gridDim.y) {
    const int h = u / units, c = u % units;
    const T* xh = x + static_cast<size_t>(h) * p.ldhx;
    T* yh = y + static_cast<size_t>(h) * p.ldhy;
    if (kInterleaved) {
      Vec v = *reinterpret_cast<const Vec*>(xh + c * V);
#pragma unroll
      for (int j = 0; j < V; j += 2) {
        const int i = (c * V + j) / 2;
        if (i < p.P) {
          const float2 t = cs[i];
          const float a = rope_f(v.e[j]), b = rope_f(v.e[j + 1]);
          rope_put(v.e[j], fmaf(a, t.x, -b * t.y));
          rope_put(v.e[j + 1], fmaf(b, t.x, a * t.y));
        }
      }
      *reinterpret_cast<Vec*>(yh + c * V) = v;
    } else if (c < turned) {
      Vec v = *reinterpret_cast<const Vec*>(xh + c * V), w = *reinterpret_cast<const Vec*>(xh + p.P + c * V);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float2 t = cs[c * V + j];
        const float a = rope_f(v.e[j]), b = rope_f(w.e[j]);
        rope_put(v.e[j], fmaf(a, t.x, -b * t.y));
        rope_put(w.e[j], fmaf(b, t.x, a * t.y));
      }
      *reinterpret_cast<Vec*>(yh + c * V) = v;
      *reinterpret_cast<Vec*>(yh + p.P + c * V) = w;
    } else {
      const int at = R + (c - turned) * V;
      *reinterpret_cast<Vec*>(yh + at) = *reinterpret_cast<const Vec*>(xh + at);
    }
  }
}

// cos, sin as [M, P] (row-major) or [P, M] (angle-major): one angle per thread and step,
// neighbours in memory to neighbouring threads.
template <bool kAngleMajor>
__global__ void __launch_bounds__(256) rope_table_kernel(const RopeParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const size_t n = static_cast<size_t>(p.M) * p.P;
  for (size_t k = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x; k < n;
       k += static_cast<size_t>(gridDim.x) * blockDim.x) {
    const size_t m = kAngleMajor ? k % p.M : k / p.P;
    const int i = static_cast<int>(kAngleMajor ? k / p.M : k % p.P);
    const int a = p.axis != nullptr ? p.axis[i] : 0;
    const float2 t = a >= 0 && a < p.A ? rope_cos_sin(rope_position(p, m, a), rope_fraction(p.freq[i]), p.scale)
                                       : make_float2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff));
    p.cos[k] = t.x;
    p.sin[k] = t.y;
  }
}

}  // namespace svdq
