// w8a8_quantize.cuh -- rows to E4M3 codes with one float32 scale each, optionally
// behind the residual's addition and a root-mean-square norm, in one pass.
//
//   h = X + residual                          (float32; residual_out = RN(h))
//   y = h rsqrt(mean(h^2) + eps) weight       (norm; else y = h)
//   t = max(max_k |y|, 2^-100),  scale = t / 448,  codes = RN_e4m3(y (448 / t))
//
// The norm's factor is one number per row, so max |y| = rsqrt(...) max |h weight|:
// both reductions (the sum of squares, the maximum) run over the same registers and
// meet in one block-wide exchange; the row is read once and kept in registers. Bound by
// HBM: 4608 rows of 3840 with residual and norm, bf16, 123.9 MB: 22.6 us, 5.5 TB/s; 4096 rows of
// 15360, codes alone, 188.8 MB: 30.3 us, 6.2 TB/s. Rows that only pass the norm (4608 of 3840, 53 MB: 13.9
// us, 3.8 TB/s, issue slots 55 % busy) are held by what every thread repeats for its 30 values: the
// wait, the exchange and its barrier, a square root and a division. The
// floor 2^-100 keeps 448 / t finite, so an all-zero row has scale 2^-100 / 448 and
// codes 0 and no case of its own. The maximum is taken on the bits of |y|, where NaN
// is above infinity is above every number: a row that holds NaN has scale NaN. Rows whose squares leave
// float32's range go through the reductions a second time, scaled by a power of two.
#pragma once

#include "sm100.cuh"

namespace svdq {

// what a row goes through: codes alone, the norm first, the residual's addition before that
enum W8Row : int { kW8Plain = 0, kW8Norm = 1, kW8ResidualNorm = 2 };

struct W8QuantParams {
  int K;
  const void* X;
  size_t ldx;
  const void* residual;   // like X, or null
  size_t ldr;
  void* residual_out;     // like X
  size_t ldo;
  const __nv_bfloat16* weight;  // [K] or null (1)
  float eps, inv_k;       // inv_k = 1 / K
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
__device__ __forceinline__ void w8_floats(const W8Vec<kF32>& r, float2 (&f)[4]) {
#pragma unroll
  for (int i = 0; i < (kF32 ? 2 : 1); ++i) {
    const uint32_t w[4] = {r.v[i].x, r.v[i].y, r.v[i].z, r.v[i].w};
    if constexpr (kF32) {
      f[2 * i] = make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
      f[2 * i + 1] = make_float2(__uint_as_float(w[2]), __uint_as_float(w[3]));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        f[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
    }
  }
}

// max(|a|, |b|, |c|), NaN if one of them is
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// eight float32 -> eight E4M3 codes, element i in byte i
__device__ __forceinline__ uint2 e4m3x8(const float2 (&v)[4]) {
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[i]) : "f"(v[i].y), "f"(v[i].x));
  return make_uint2(h[0] | (static_cast<uint32_t>(h[1]) << 16), h[2] | (static_cast<uint32_t>(h[3]) << 16));
}

// h = X + residual of one vector.
template <int kRow, bool kF32>
__device__ __forceinline__ void w8_sum(const W8Vec<kF32>& xv, const W8Vec<kF32>& rv, float2 (&h)[4]) {
  w8_floats<kF32>(xv, h);
  if (kRow == kW8ResidualNorm) {
    float2 r[4];
    w8_floats<kF32>(rv, r);
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = __fadd2_rn(h[j], r[j]);
  }
}

// h in X's type, and its way out
template <bool kF32>
__device__ __forceinline__ W8Vec<kF32> w8_round(const float2 (&h)[4]) {
  W8Vec<kF32> o;
  if constexpr (kF32) {
    o.v[0] = make_uint4(__float_as_uint(h[0].x), __float_as_uint(h[0].y), __float_as_uint(h[1].x), __float_as_uint(h[1].y));
    o.v[1] = make_uint4(__float_as_uint(h[2].x), __float_as_uint(h[2].y), __float_as_uint(h[3].x), __float_as_uint(h[3].y));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 b = __float22bfloat162_rn(h[j]);
      w[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    o.v[0] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return o;
}
template <bool kF32>
__device__ __forceinline__ void w8_sum_out(const W8QuantParams& p, size_t row, int v, const W8Vec<kF32>& o) {
  const size_t at = row * p.ldo + static_cast<size_t>(v) * 8;
  uint4* to = kF32 ? reinterpret_cast<uint4*>(static_cast<float*>(p.residual_out) + at)
                   : reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.residual_out) + at);
#pragma unroll
  for (int i = 0; i < (kF32 ? 2 : 1); ++i) to[i] = o.v[i];
}

// This thread's part of both reductions: the squares of h, and the maximum of h times its weight
// (as float32, or null: from memory), which h leaves as.
template <bool kNorm>
__device__ __forceinline__ void w8_measure(const W8QuantParams& p, int v, const float2* wv, float2 (&h)[4], float2& ss,
                                           float& top) {
  if (kNorm) {
#pragma unroll
    for (int j = 0; j < 4; ++j) ss = __ffma2_rn(h[j], h[j], ss);
    if (p.weight != nullptr) {
      float2 g[4];
      if (wv != nullptr) {
        const float4 a = reinterpret_cast<const float4*>(wv)[0], b = reinterpret_cast<const float4*>(wv)[1];
        g[0] = make_float2(a.x, a.y), g[1] = make_float2(a.z, a.w);
        g[2] = make_float2(b.x, b.y), g[3] = make_float2(b.z, b.w);
      } else {
        w8_floats<false>(w8_load<false>(p.weight, static_cast<size_t>(v) * 8), g);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = __fmul2_rn(h[j], g[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) top = max3_abs_nan(top, h[j].x, h[j].y);
}

// Both reductions over the block, through `part` [32] (zeros behind the last warp's), the
// partial sums in an order of their own; false in every thread if `ok` is false in one.
template <bool kNorm>
__device__ __forceinline__ bool w8_reduce(float2 ss2, float top1, float& ss, float& top, bool ok, float2* part) {
  const int warps = blockDim.x / 32;
  // no sign: the bits are ordered like the numbers, NaN above them
  top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top1)));
  ss = ss2.x + ss2.y;
  if (kNorm) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  }
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = make_float2(ss, top);
  ok = __syncthreads_and(ok);
  if (warps <= 8) {
    ss = top = 0.0f;
    for (int i = 0; i < warps; i += 2) {
      const float4 v = *reinterpret_cast<const float4*>(part + i);
      ss = ss + v.x + v.z;
      top = max3_abs_nan(top, v.y, v.w);
    }
  } else {
    const float2 v = part[threadIdx.x % 32];
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v.y)));
    ss = v.x;
    if (kNorm) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
  }
  return ok;
}

// The row's scale (or the mark of a row that comes once more: no scale is negative), and what turns its
// values into codes: one factor, or, where that would leave float32's range (an all but empty row), rs
// and then inv.
constexpr float kW8Again = -1.0f;
struct W8Factors {
  float one, rs, inv;
};
template <bool kNorm>
__device__ __forceinline__ W8Factors w8_scale(const W8QuantParams& p, size_t row, float ss, float top, float eps,
                                              bool again = false) {
  W8Factors f;
  float t = top;
  f.rs = 1.0f;
  if (kNorm) {
    f.rs = rsqrtf(fmaf(ss, p.inv_k, eps));
    t *= f.rs;
  }
  if (t < 7.888609052210118e-31f) t = 7.888609052210118e-31f;  // 2^-100; NaN stays
  f.inv = __fdiv_rn(448.0f, t);
  f.one = f.rs * f.inv;
  if (threadIdx.x == 0) p.scale[row] = again ? kW8Again : __fdiv_rn(t, 448.0f);
  return f;
}

template <bool kNorm, int kVecs>
__device__ __forceinline__ void w8_give(const W8QuantParams& p, size_t row, float2 (&h)[kVecs][4], const W8Factors& f, int first) {
  float mul = f.one;
  if (kNorm && !(f.one < 1e37f)) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) h[i][j] = __fmul2_rn(h[i][j], make_float2(f.rs, f.rs));
    mul = f.inv;
  }
  uint2* out = reinterpret_cast<uint2*>(p.codes + row * static_cast<size_t>(p.K)) + first;
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
    if (static_cast<int>(first + i * blockDim.x) < p.K / 8) {
      float2 q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) q[j] = __fmul2_rn(h[i][j], make_float2(mul, mul));
      out[i * blockDim.x] = e4m3x8(q);
    }
}

// Squares leave float32's range long before the values do. Where their sum overflowed, or is so small (and
// eps too) that squares were lost, the row goes through both reductions once more, times this power of
// two, and eps times its square: y is the same. 1 where neither holds; the same in every thread of
// the block. Up to K = 2^15 values the second sum keeps its range: below 2^15 (2^128 2^-100)^2 = 2^71, and
// below 2^15 2^-90 2^200 = 2^125. (A row that holds infinity comes here too; its scale stays not finite.)
__device__ __forceinline__ float w8_rescale(const W8QuantParams& p, float ss) {
  if (ss > 3.402823466e38f) return 7.888609052210118e-31f;                                   // 2^-100
  return fmaf(ss, p.inv_k, p.eps) < 8.077935669463161e-28f ? 1.2676506002282294e30f : 1.0f;  // 2^-90, 2^100
}

// Such a row from its beginning, out of memory: x and r (float32 sums: the sum, and no r), with its
// 16-bit sum's copy out. Out of line, its parameters by value, and called where nothing of the common
// way is live any more: inside the ring's loop, or with the address of the kernel's parameters, it cost
// every row 7 to 13 %. Each thread touches the vectors that it had before.
template <int kRow, bool kF32>
__device__ __noinline__ void w8_row_again(const W8QuantParams p, size_t row, const void* x, const void* r,
                                          float2 (*part)[32]) {
  float2 h[1][4], ss2;
  float ss, top, f = 1.0f;
  auto sum = [&](int v) {
    const W8Vec<kF32> xv = w8_load<kF32>(x, static_cast<size_t>(v) * 8);
    w8_sum<kRow, kF32>(xv, kRow == kW8ResidualNorm ? w8_load<kF32>(r, static_cast<size_t>(v) * 8) : xv, h[0]);
  };
  auto measure = [&](int v) {
#pragma unroll
    for (int j = 0; j < 4; ++j) h[0][j] = __fmul2_rn(h[0][j], make_float2(f, f));
    w8_measure<true>(p, v, nullptr, h[0], ss2, top);
  };
  for (int pass = 0; pass == 0 || (pass == 1 && f != 1.0f); ++pass) {
    ss2 = make_float2(0.0f, 0.0f);
    top = 0.0f;
#pragma unroll 1
    for (int v = threadIdx.x; v < p.K / 8; v += blockDim.x) {
      sum(v);
      measure(v);
    }
    w8_reduce<true>(ss2, top, ss, top, true, part[pass]);
    if (pass == 0) f = w8_rescale(p, ss);
  }
  const W8Factors g = w8_scale<true>(p, row, ss, top, p.eps * f * f);
#pragma unroll 1
  for (int v = threadIdx.x; v < p.K / 8; v += blockDim.x) {
    sum(v);
    if (kRow == kW8ResidualNorm) w8_sum_out<kF32>(p, row, v, w8_round<kF32>(h[0]));
    measure(v);
    w8_give<true, 1>(p, row, h, g, v);
  }
  __syncthreads();  // `part` is free
}
template <int kRow, bool kF32>
__device__ __forceinline__ void w8_again(const W8QuantParams& p, size_t row, float2 (*part)[32]) {
  constexpr size_t esz = kF32 ? 4 : 2;
  if constexpr (kRow == kW8ResidualNorm && kF32)
    w8_row_again<kW8Norm, kF32>(p, row, static_cast<const char*>(p.residual_out) + row * p.ldo * esz, nullptr, part);
  else
    w8_row_again<kRow, kF32>(p, row, static_cast<const char*>(p.X) + row * p.ldx * esz,
                             kRow == kW8ResidualNorm ? static_cast<const char*>(p.residual) + row * p.ldr * esz : nullptr, part);
}

// One block per row; thread i holds the row's 8-value vectors i, i + blockDim.x, ...
// For few rows, and for rows too long for the ring below.
template <int kRow, bool kF32>
__global__ void __launch_bounds__(1024) w8a8_quantize_kernel(const W8QuantParams p) {
  constexpr bool kNorm = kRow != kW8Plain;
  constexpr int kVecs = 4;
  __shared__ __align__(16) float2 part[kNorm ? 2 : 1][32];
  const size_t row = blockIdx.x;
  const int nvec = p.K / 8, T = blockDim.x, tid = threadIdx.x;
  if (tid < 32 && tid >= T / 32) part[0][tid] = part[kNorm][tid] = make_float2(0.0f, 0.0f);
  grid_dep_wait();
  grid_dep_launch();
  float2 h[kVecs][4], ss2 = make_float2(0.0f, 0.0f);
  float ss, top = 0.0f;
  W8Vec<kF32> xv[kVecs], rv[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int v = tid + i * T;
    if (v < nvec) {
      xv[i] = w8_load<kF32>(p.X, row * p.ldx + static_cast<size_t>(v) * 8);
      if (kRow == kW8ResidualNorm) rv[i] = w8_load<kF32>(p.residual, row * p.ldr + static_cast<size_t>(v) * 8);
    }
  }
  // A 16-bit sum leaves last: it may go where the residual or X is, which a row that goes through the
  // reductions again still has to read. (A float32 one goes at once and is read again itself. Before the
  // codes the 16-bit sum took one row of 3840 2.59 us, behind them it takes 2.51.)
  constexpr bool kKeep = kRow == kW8ResidualNorm && !kF32;
  W8Vec<kF32> sum[kKeep ? kVecs : 1];
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
    if (tid + i * T < nvec) {
      w8_sum<kRow, kF32>(xv[i], rv[i], h[i]);
      if constexpr (kKeep) sum[i] = w8_round<kF32>(h[i]);
      else if (kRow == kW8ResidualNorm) w8_sum_out<kF32>(p, row, tid + i * T, w8_round<kF32>(h[i]));
      w8_measure<kNorm>(p, tid + i * T, nullptr, h[i], ss2, top);
    }
  w8_reduce<kNorm>(ss2, top, ss, top, true, part[0]);
  if constexpr (kNorm) {
    if (w8_rescale(p, ss) != 1.0f) {
      __syncthreads();  // `part` has been read
      w8_again<kRow, kF32>(p, row, part);
      return;
    }
  }
  w8_give<kNorm, kVecs>(p, row, h, w8_scale<kNorm>(p, row, ss, top, p.eps), tid);
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (tid + i * T < nvec) w8_sum_out<kF32>(p, row, tid + i * T, sum[i]);
  }
}

// Many rows: persistent blocks, each with a ring of rows (X, then the residual) that bulk
// copies fill ahead, so that the loads go on through the reduction and the
// stores of the row before.
constexpr size_t kW8RingBytes = 227 * 1024;  // of an SM, for all its blocks' rings and weights
constexpr size_t kW8RingOwn = 2048;          // a block's barriers and exchange, and what the system keeps
constexpr int kW8RingStages = 2;
struct W8RingParams {
  int M;
  uint32_t* status;
};
template <int kRow, bool kF32>
__global__ void __launch_bounds__(1024) w8a8_quantize_ring_kernel(const W8QuantParams p,
                                                                  const W8RingParams q) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(16) float2 part[2][32];
  __shared__ uint64_t s_bars[kW8RingStages];
  constexpr bool kNorm = kRow != kW8Plain, has_r = kRow == kW8ResidualNorm;
  constexpr int kVecs = 4;
  const int nvec = p.K / 8, T = blockDim.x, tid = threadIdx.x;
  constexpr int NS = kW8RingStages;
  static_assert(NS == 2, "the other stage is s ^ 1");
  const uint32_t x_bytes = p.K * (kF32 ? 4 : 2);
  const uint32_t stage_bytes = has_r ? 2 * x_bytes : x_bytes;
  const uint32_t bars = smem_u32(s_bars), base = smem_u32(ring);
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) mbar_init(bars + 8 * s, 1);
    fence_barrier_init();
  }
  if (tid < 32 && tid >= T / 32) part[0][tid] = part[1][tid] = make_float2(0.0f, 0.0f);
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  auto fetch = [&](size_t row, int s) {
    constexpr size_t esz = kF32 ? 4 : 2;
    mbar_arrive_expect_tx(bars + 8 * s, stage_bytes);
    bulk_load(base + s * stage_bytes, static_cast<const char*>(p.X) + row * p.ldx * esz, x_bytes, bars + 8 * s);
    if (has_r)
      bulk_load(base + s * stage_bytes + x_bytes, static_cast<const char*>(p.residual) + row * p.ldr * esz, x_bytes,
                bars + 8 * s);
  };
  if (tid == 0)
    for (int s = 0; s < NS; ++s)
      if (blockIdx.x + static_cast<size_t>(s) * gridDim.x < q.M) fetch(blockIdx.x + static_cast<size_t>(s) * gridDim.x, s);
  // the weight behind the ring, as float32: each thread reads back what it wrote itself
  const bool has_w = kNorm && p.weight != nullptr;
  float2* weight = reinterpret_cast<float2*>(ring + NS * stage_bytes);
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
    if (has_w && tid + i * T < nvec) {
      float2 g[4];
      w8_floats<false>(w8_load<false>(p.weight, static_cast<size_t>(tid + i * T) * 8), g);
#pragma unroll
      for (int j = 0; j < 4; ++j) weight[(tid + i * T) * 4 + j] = g[j];
    }
  int s = 0, phase = 0, odd = 0;
  bool again = false;  // a row's squares left float32's range
  for (size_t row = blockIdx.x; row < q.M; row += gridDim.x) {
    bool ok = mbar_wait(bars + 8 * s, phase, q.status);
    float2 h[kVecs][4], ss2 = make_float2(0.0f, 0.0f);
    float ss, top = 0.0f;
    const uint8_t* st = ring + s * stage_bytes;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int v = tid + i * T;
      if (v < nvec) {
        const W8Vec<kF32> xv = w8_load<kF32>(st, static_cast<size_t>(v) * 8);
        W8Vec<kF32> rv = xv;
        if (has_r) rv = w8_load<kF32>(st + x_bytes, static_cast<size_t>(v) * 8);
        w8_sum<kRow, kF32>(xv, rv, h[i]);
        if (has_r) w8_sum_out<kF32>(p, row, v, w8_round<kF32>(h[i]));
        w8_measure<kNorm>(p, v, weight + v * 4, h[i], ss2, top);
      }
    }
    // the exchange's barrier also says that the stage has been read
    if (!w8_reduce<kNorm>(ss2, top, ss, top, ok, part[odd])) {
      // a wait has run out: the copies on their way land (or run out again) before the block ends
      if (tid == 0) {
        mbar_wait(bars + 8 * s, phase, q.status);
        if (row + gridDim.x < q.M) mbar_wait(bars + 8 * (s ^ 1), s == 0 ? phase : phase ^ 1, q.status);
      }
      break;
    }
    const bool rare = kNorm && w8_rescale(p, ss) != 1.0f;
    again |= rare;
    if constexpr (has_r && !kF32) {
      // a sum in place is taken back: the row is read once more
      if (rare && (p.residual_out == p.X || p.residual_out == p.residual)) {
        const uint8_t* was = p.residual_out == p.X ? st : st + x_bytes;
#pragma unroll 1
        for (int v = tid; v < nvec; v += T)
          w8_sum_out<kF32>(p, row, v, w8_load<kF32>(was, static_cast<size_t>(v) * 8));
        __syncthreads();
      }
    }
    const size_t next = row + static_cast<size_t>(NS) * gridDim.x;
    if (tid == 0 && next < q.M) fetch(next, s);
    w8_give<kNorm, kVecs>(p, row, h, w8_scale<kNorm>(p, row, ss, top, p.eps, rare), tid);
    odd ^= 1;
    if (++s == NS) s = 0, phase ^= 1;
  }
  if constexpr (kNorm) {
    if (again) {
      __syncthreads();  // `part` has been read, the marks are there
      for (size_t row = blockIdx.x; row < q.M; row += gridDim.x)
        if (p.scale[row] == kW8Again) w8_again<kRow, kF32>(p, row, part);
    }
  }
}

}  // namespace svdq
