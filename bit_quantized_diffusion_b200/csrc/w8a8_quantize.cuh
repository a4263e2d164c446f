// w8a8_quantize.cuh -- rows to E4M3 codes with one float32 scale each, optionally
// behind the residual's addition and a root-mean-square norm, in one pass.
//
//   h = X + residual                          (float32; residual_out = RN(h))
//   y = h rsqrt(mean(h^2) + eps) weight       (norm; else y = h)
//   t = max(max_k |y|, 2^-100),  scale = t / 448,  codes = RN_e4m3(y (448 / t))
//
// The norm's factor is one number per row, so max |y| = rsqrt(...) max |h weight|:
// both reductions (the sum of squares, the maximum) run over the same registers and
// meet in one block-wide exchange; the row is read once and kept in registers. The
// floor 2^-100 keeps 448 / t finite, so an all-zero row has scale 2^-100 / 448 and
// codes 0 and no case of its own. The maximum is taken on the bits of |y|, where NaN
// is above infinity is above every number: a row that holds NaN has scale NaN.
#pragma once

#include "sm100.cuh"

namespace svdq {

struct W8QuantParams {
  int K;
  const void* X;
  size_t ldx;
  const void* residual;   // like X, or null
  size_t ldr;
  void* residual_out;     // like X
  size_t ldo;
  const __nv_bfloat16* weight;  // [K] or null (1)
  float eps;
  uint8_t* codes;         // [M, K]
  float* scale;           // [M]
};

// eight values as float32; kF32: float32 storage, else bf16
template <bool kF32>
struct W8Vec {
  uint4 v[kF32 ? 2 : 1];
};
template <bool kF32>
__device__ __forceinline__ W8Vec<kF32> w8_load(const void* base, size_t at) {
  W8Vec<kF32> r;
  if constexpr (kF32) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + at);
    r.v[0] = q[0];
    r.v[1] = q[1];
  } else {
    r.v[0] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at);
  }
  return r;
}
template <bool kF32>
__device__ __forceinline__ void w8_floats(const W8Vec<kF32>& r, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < (kF32 ? 2 : 1); ++i) {
    const uint32_t w[4] = {r.v[i].x, r.v[i].y, r.v[i].z, r.v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (kF32) {
        f[4 * i + j] = __uint_as_float(w[j]);
      } else {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    }
  }
}

// eight float32 -> eight E4M3 codes, element i in byte i
__device__ __forceinline__ uint2 e4m3x8(const float (&v)[8]) {
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
  return make_uint2(h[0] | (static_cast<uint32_t>(h[1]) << 16), h[2] | (static_cast<uint32_t>(h[3]) << 16));
}

// One block per row; thread i holds the row's 8-value vectors i, i + blockDim.x, ...
template <bool kNorm, bool kF32, int kVecs>
__global__ void __launch_bounds__(1024) w8a8_quantize_kernel(const W8QuantParams p) {
  const size_t row = blockIdx.x;
  const int nvec = p.K / 8, T = blockDim.x, tid = threadIdx.x;
  grid_dep_wait();
  grid_dep_launch();
  float h[kVecs][8];
  float ss = 0.0f;
  uint32_t top = 0;
  W8Vec<kF32> xv[kVecs], rv[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int v = tid + i * T;
    if (v < nvec) {
      xv[i] = w8_load<kF32>(p.X, row * p.ldx + static_cast<size_t>(v) * 8);
      if (kNorm && p.residual != nullptr) rv[i] = w8_load<kF32>(p.residual, row * p.ldr + static_cast<size_t>(v) * 8);
    }
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int v = tid + i * T;
    if (v < nvec) {
      w8_floats<kF32>(xv[i], h[i]);
      if (kNorm) {
        if (p.residual != nullptr) {
          float r[8];
          w8_floats<kF32>(rv[i], r);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i][j] += r[j];
          const size_t at = row * p.ldo + static_cast<size_t>(v) * 8;
          if constexpr (kF32) {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.residual_out) + at);
            o[0] = make_float4(h[i][0], h[i][1], h[i][2], h[i][3]);
            o[1] = make_float4(h[i][4], h[i][5], h[i][6], h[i][7]);
          } else {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(h[i][2 * j], h[i][2 * j + 1]);
              w[j] = *reinterpret_cast<const uint32_t*>(&b);
            }
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.residual_out) + at) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(h[i][j], h[i][j], ss);
        if (p.weight != nullptr) {
          float g[8];
          w8_floats<false>(w8_load<false>(p.weight, static_cast<size_t>(v) * 8), g);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i][j] *= g[j];
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(h[i][j]) & 0x7FFFFFFFu);
    }
  }
  // both reductions over the block
  __shared__ float s_ss[32];
  __shared__ uint32_t s_top[32];
  const int warps = T / 32, warp = tid / 32, lane = tid % 32;
  top = __reduce_max_sync(0xffffffffu, top);
  if (kNorm) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  }
  if (warps > 1) {
    if (lane == 0) {
      s_top[warp] = top;
      s_ss[warp] = ss;
    }
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, lane < warps ? s_top[lane] : 0u);
    if (kNorm) {
      ss = lane < warps ? s_ss[lane] : 0.0f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
  }
  float t = __uint_as_float(top);
  float rs = 1.0f;
  if (kNorm) {
    rs = 1.0f / sqrtf(ss / static_cast<float>(p.K) + p.eps);
    t *= rs;
  }
  if (t < 7.888609052210118e-31f) t = 7.888609052210118e-31f;  // 2^-100; NaN stays
  const float inv = 448.0f / t;
  if (tid == 0) p.scale[row] = t / 448.0f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int v = tid + i * T;
    if (v < nvec) {
      float q[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = (kNorm ? h[i][j] * rs : h[i][j]) * inv;
      *reinterpret_cast<uint2*>(p.codes + row * static_cast<size_t>(p.K) + static_cast<size_t>(v) * 8) = e4m3x8(q);
    }
  }
}

}  // namespace svdq
