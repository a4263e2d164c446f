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
// fraction of a turn, the wrap of the integer product being the range reduction. The
// fraction carries freq's 53 bits down to 2^-64 of a turn: the angle is off by 2^-52 of
// itself and 2^-64 turns per position. All 64 bits go on: the nearest quarter turn, which
// swaps and signs, and a signed rest of at most an eighth, made a float32 in two halves, so that
// a small rest keeps its bits and a small sine, or a cosine near a quarter turn, its relative precision
// (of the top 32 bits alone the sine of position 1 at frequency 1e-4 was off by 8e-6 of itself).
// The rest's sine and cosine are the first terms of their power series (x^9 and x^10; what is
// left out is below 2^-28 of the value). With U = 2^-24 the rest is off by 2.5 U of itself (conversion, 2 pi,
// sum), the series by 2 U more, the scale by one: cosine and sine are off by less than 2^-21 of themselves.
#pragma once

#include <type_traits>

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

// The position's angle under a pair's fraction, in 2^-64 of a turn.
__device__ __forceinline__ uint64_t rope_turn(long long pos, uint64_t fraction) {
  return static_cast<uint64_t>(pos) * fraction;
}

// Cosines and sines of two angles, each times its scale: c = (c0, c1), s = (s0, s1). Both
// angles go through the series together, as pairs of float32.
__device__ __forceinline__ void rope_cos_sin2(uint64_t turn0, uint64_t turn1, float2 scale, float2& c, float2& s) {
  // an eighth on, and half of 2^-32, which rounds the upper half: its bits 31, 30 are the nearest quarter turn,
  // its others the rest plus an eighth; the lower half, as a signed number, is what the rest has below
  constexpr uint64_t kOn = (1ull << 61) + (1ull << 31);
  const uint32_t t0 = static_cast<uint32_t>((turn0 + kOn) >> 32), t1 = static_cast<uint32_t>((turn1 + kOn) >> 32);
  auto upper = [](uint32_t t) { return static_cast<float>(static_cast<int>(t & 0x3FFFFFFFu) - 0x20000000); };
  auto lower = [](uint64_t turn) { return static_cast<float>(static_cast<int>(static_cast<uint32_t>(turn))); };
  auto k = [](float v) { return make_float2(v, v); };
  const float2 x = __ffma2_rn(make_float2(upper(t0), upper(t1)), k(1.4629180792671596e-9f),                // 2 pi 2^-32
                              __fmul2_rn(make_float2(lower(turn0), lower(turn1)), k(3.4061215800865545e-19f)));  // 2 pi 2^-64
  const float2 xx = __fmul2_rn(x, x);
  float2 a = __ffma2_rn(xx, k(2.7557319e-6f), k(-1.9841270e-4f));   // 1 / 9!, 1 / 7!
  a = __ffma2_rn(xx, a, k(8.3333333e-3f));                          // 1 / 5!
  a = __ffma2_rn(xx, a, k(-1.6666667e-1f));                         // 1 / 3!
  a = __ffma2_rn(__fmul2_rn(x, xx), a, x);
  float2 b = __ffma2_rn(xx, k(-2.7557319e-7f), k(2.4801587e-5f));   // 1 / 10!, 1 / 8!
  b = __ffma2_rn(xx, b, k(-1.3888889e-3f));                         // 1 / 6!
  b = __ffma2_rn(xx, b, k(4.1666667e-2f));                          // 1 / 4!
  b = __ffma2_rn(xx, b, k(-0.5f));
  b = __ffma2_rn(xx, b, k(1.0f));
  // each quarter turn on: (c, s) -> (-s, c)
  auto turned = [](uint32_t t, float cv, float sv, float& co, float& so) {
    const bool swap = t & 0x40000000u;
    co = __uint_as_float(__float_as_uint(swap ? sv : cv) ^ ((t + 0x40000000u) & 0x80000000u));
    so = __uint_as_float(__float_as_uint(swap ? cv : sv) ^ (t & 0x80000000u));
  };
  turned(t0, b.x, a.x, c.x, s.x);
  turned(t1, b.y, a.y, c.y, s.y);
  c = __fmul2_rn(c, scale);
  s = __fmul2_rn(s, scale);
}

// A row's position. (By ordinary loads, here and below, not the read-only path: what makes positions may
// still be writing them when this grid starts.)
__device__ __forceinline__ long long rope_position(const RopeParams& p, size_t m, int axis) {
  const size_t at = m * p.A + axis;
  return p.pos64 ? static_cast<const long long*>(p.positions)[at]
                 : static_cast<long long>(static_cast<const int*>(p.positions)[at]);
}

// The same, issued where it stands: the rotation's few heads wait for it (4608 rows of 2 heads of 128: 18.6
// us, 18.9 with the load that the compiler moves).
__device__ __forceinline__ long long rope_position_in_order(const RopeParams& p, size_t m, int axis) {
  const size_t at = m * p.A + axis;
  long long v;
  if (p.pos64) {
    asm volatile("ld.global.b64 %0, [%1];" : "=l"(v) : "l"(static_cast<const long long*>(p.positions) + at));
  } else {
    int w;
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(w) : "l"(static_cast<const int*>(p.positions) + at));
    v = w;
  }
  return v;
}

template <typename T, int V>
struct alignas(sizeof(T) * V) RopeVec {
  T e[V];
};
// V elements as float32 and back; bf16 two at a time
template <int V>
__device__ __forceinline__ void rope_unpack(const RopeVec<float, V>& v, float (&f)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) f[j] = v.e[j];
}
template <int V>
__device__ __forceinline__ void rope_unpack(const RopeVec<__nv_bfloat16, V>& v, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = __bfloat162float(v.e[0]);
  } else {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      const uint32_t w = reinterpret_cast<const uint32_t*>(&v)[j / 2];
      f[j] = __uint_as_float(w << 16);
      f[j + 1] = __uint_as_float(w & 0xFFFF0000u);
    }
  }
}
template <int V>
__device__ __forceinline__ void rope_pack(const float (&f)[V], RopeVec<float, V>& v) {
#pragma unroll
  for (int j = 0; j < V; ++j) v.e[j] = f[j];
}
template <int V>
__device__ __forceinline__ void rope_pack(const float (&f)[V], RopeVec<__nv_bfloat16, V>& v) {
  if constexpr (V == 1) {
    v.e[0] = __float2bfloat16_rn(f[0]);
  } else {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[j], f[j + 1]);
      reinterpret_cast<uint32_t*>(&v)[j / 2] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
}

// Pairs (a, b) turned, two at a time: (a c - b s, b c + a s).
template <int N>
__device__ __forceinline__ void rope_turn_pairs(float (&a)[N], float (&b)[N], const float (&c)[N], const float (&s)[N]) {
#pragma unroll
  for (int q = 0; q < N; q += 2) {
    if constexpr (N % 2 == 0) {
      const float2 av = make_float2(a[q], a[q + 1]), bv = make_float2(b[q], b[q + 1]);
      const float2 cv = make_float2(c[q], c[q + 1]), sv = make_float2(s[q], s[q + 1]);
      const float2 ra = __ffma2_rn(av, cv, __fmul2_rn(bv, make_float2(-sv.x, -sv.y)));
      const float2 rb = __ffma2_rn(bv, cv, __fmul2_rn(av, sv));
      a[q] = ra.x; a[q + 1] = ra.y;
      b[q] = rb.x; b[q + 1] = rb.y;
    } else {
      const float av = a[q], bv = b[q];
      a[q] = fmaf(av, c[q], -bv * s[q]);
      b[q] = fmaf(bv, c[q], av * s[q]);
    }
  }
}

// A pair's fraction, axis and scale. A frequency that is not finite, or an axis that the
// positions do not have: scale NaN, and axis 0 read for the latter.
struct RopePair {
  uint64_t fraction;
  int axis;
  float scale;
};
__device__ __forceinline__ RopePair rope_pair(const RopeParams& p, int i) {
  const int a = p.axis != nullptr ? p.axis[i] : 0;
  const bool there = a >= 0 && a < p.A;
  const double f = p.freq[i];
  return {rope_fraction(f), there ? a : 0, there && isfinite(f) ? p.scale : __int_as_float(0x7fffffff)};
}

// One block per (row, share of the heads). The row's angles go through shared memory once;
// then a thread keeps its V columns of a head (half layout: V of the first half and the V
// they pair with), their cosines and sines in registers, and walks over the heads, with the
// loads of kRopeHeads heads in flight, the first before the angles are made. Bound by HBM
// (4608 rows of 60 heads of 128, bf16, 141.6 MB: 25.0 us, 5.7 TB/s; 30.9 us with a head at a
// time and the angles read from shared memory for each).
constexpr int kRopeHeads = 4;
template <typename T, int V, bool kInterleaved>
__global__ void __launch_bounds__(256) rope_kernel(const RopeParams p) {
  __shared__ __align__(16) float cos_s[kRopeMaxPairs], sin_s[kRopeMaxPairs];
  const size_t m = blockIdx.x;
  const T* x = static_cast<const T*>(p.X) + m * p.ldx;
  T* y = static_cast<T*>(p.Y) + m * p.ldy;
  using Vec = RopeVec<T, V>;
  // a head's units: interleaved, its V-element vectors; half layout, first those that hold
  // pairs, then the copied ones
  const int turned = p.P / V;
  const int units = kInterleaved ? p.D / V : turned + (p.D - 2 * p.P) / V;
  const int per_head = min(units, 256), heads_at_once = 256 / per_head;
  const int group = threadIdx.x / per_head, step = heads_at_once * gridDim.y;
  const int h0 = group < heads_at_once ? static_cast<int>(blockIdx.y) * heads_at_once + group : p.heads;
  Vec v[kRopeHeads], w[kInterleaved ? 1 : kRopeHeads];
  auto column = [&](int c) { return kInterleaved || c < turned ? c * V : 2 * p.P + (c - turned) * V; };
  auto load = [&](int c, int h) {
    const T* at = x + static_cast<size_t>(h) * p.ldhx + column(c);
    const size_t next = static_cast<size_t>(step) * p.ldhx;
#pragma unroll
    for (int j = 0; j < kRopeHeads; ++j) {
      if (h + j * step < p.heads) {
        v[j] = *reinterpret_cast<const Vec*>(at);
        if constexpr (!kInterleaved) {
          if (c < turned) w[j] = *reinterpret_cast<const Vec*>(at + p.P);
        }
      }
      at += next;
    }
  };
  int c = threadIdx.x % per_head;
  grid_dep_wait();
  grid_dep_launch();
  load(c, h0);
  for (int i = 2 * threadIdx.x; i < p.P; i += 2 * blockDim.x) {
    const RopePair a = rope_pair(p, i), b = i + 1 < p.P ? rope_pair(p, i + 1) : a;
    float2 cc, ss;
    rope_cos_sin2(rope_turn(rope_position_in_order(p, m, a.axis), a.fraction), rope_turn(rope_position_in_order(p, m, b.axis), b.fraction),
                  make_float2(a.scale, b.scale), cc, ss);
    // (an odd last pair's neighbour is inside the arrays, and not read)
    *reinterpret_cast<float2*>(cos_s + i) = cc;
    *reinterpret_cast<float2*>(sin_s + i) = ss;
  }
  __syncthreads();
  for (; c < units; c += per_head) {
    constexpr int kPairs = kInterleaved ? V / 2 : V;
    const int pairs = min(kPairs, p.P - c * kPairs);  // an interleaved unit may reach past the last pair
    float ct[kPairs], st[kPairs];
#pragma unroll
    for (int q = 0; q < kPairs; ++q)
      if (q < pairs) {
        ct[q] = cos_s[c * kPairs + q];
        st[q] = sin_s[c * kPairs + q];
      }
    for (int h = h0; h < p.heads;) {
      T* at = y + static_cast<size_t>(h) * p.ldhy + column(c);
      const size_t next = static_cast<size_t>(step) * p.ldhy;
#pragma unroll
      for (int j = 0; j < kRopeHeads; ++j) {
        if (h + j * step < p.heads) {
          if constexpr (kInterleaved) {
            if (pairs > 0) {
              float f[V], a[kPairs], b[kPairs];
              rope_unpack<V>(v[j], f);
#pragma unroll
              for (int q = 0; q < kPairs; ++q) a[q] = f[2 * q], b[q] = f[2 * q + 1];
              rope_turn_pairs<kPairs>(a, b, ct, st);
#pragma unroll
              for (int q = 0; q < kPairs; ++q)
                if (q < pairs) f[2 * q] = a[q], f[2 * q + 1] = b[q];
              rope_pack<V>(f, v[j]);
            }
          } else if (pairs > 0 && c < turned) {
            float a[V], b[V];
            rope_unpack<V>(v[j], a);
            rope_unpack<V>(w[j], b);
            rope_turn_pairs<V>(a, b, ct, st);
            rope_pack<V>(a, v[j]);
            rope_pack<V>(b, w[j]);
            *reinterpret_cast<Vec*>(at + p.P) = w[j];
          }
          *reinterpret_cast<Vec*>(at) = v[j];
        }
        at += next;
      }
      h += kRopeHeads * step;
      if (h < p.heads) load(c, h);
    }
    if (c + per_head < units) load(c + per_head, h0);
  }
}

// cos, sin as [M, P]: a thread keeps V adjacent pairs, their fractions in registers, and
// walks down the rows, four at a time. Its pairs' positions: one per row where there is one
// axis, two where its pairs lie on two (so that no lane of a warp takes another way), else one
// per pair. 131072 rows of 64 pairs, 67.6 MB: 15.4 us, 4.4 TB/s (a plain fill: 3.7), issue
// slots 60 % busy, from int64 positions the same within 1 % (40.4 us with sincospif of a float32 half-turn).
template <int V, typename Pos>
__global__ void __launch_bounds__(256, 4) rope_table_kernel(const RopeParams p) {
  const int nq = p.P / V, per_row = min(nq, 256), rows = 256 / per_row;
  const int r = threadIdx.x / per_row;
  grid_dep_wait();
  grid_dep_launch();
  if (r >= rows) return;
  const Pos* positions = static_cast<const Pos*>(p.positions);
  for (int q = threadIdx.x % per_row; q < nq; q += per_row) {
    RopePair pair[V];
    bool two = true;
    uint32_t last = 0;  // bit j: pair j lies on the last pair's axis
#pragma unroll
    for (int j = 0; j < V; ++j) pair[j] = rope_pair(p, q * V + j);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (pair[j].axis == pair[V - 1].axis) last |= 1u << j;
      else two = two && pair[j].axis == pair[0].axis;
    }
    const size_t step = static_cast<size_t>(gridDim.x) * rows;
    auto put = [&](size_t m, const Pos (&pos)[V]) {
      RopeVec<float, V> c, s;
      if constexpr (V == 1) {
        float2 cc, ss;
        const uint64_t turn = rope_turn(pos[0], pair[0].fraction);
        rope_cos_sin2(turn, turn, make_float2(pair[0].scale, pair[0].scale), cc, ss);
        c.e[0] = cc.x;
        s.e[0] = ss.x;
      } else {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
          float2 cc, ss;
          rope_cos_sin2(rope_turn(pos[j], pair[j].fraction), rope_turn(pos[j + 1], pair[j + 1].fraction),
                        make_float2(pair[j].scale, pair[j + 1].scale), cc, ss);
          c.e[j] = cc.x, c.e[j + 1] = cc.y;
          s.e[j] = ss.x, s.e[j + 1] = ss.y;
        }
      }
      *reinterpret_cast<RopeVec<float, V>*>(p.cos + m * p.P + q * V) = c;
      *reinterpret_cast<RopeVec<float, V>*>(p.sin + m * p.P + q * V) = s;
    };
    size_t m = static_cast<size_t>(blockIdx.x) * rows + r;
    // kPos positions per row, of the first pair and of the last
    auto walk = [&](auto count) {
      constexpr int kPos = decltype(count)::value;
      for (; m < p.M; m += 4 * step) {
        Pos four[4][kPos];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (m + k * step < p.M) {
            four[k][0] = positions[(m + k * step) * p.A + pair[0].axis];
            if (kPos > 1) four[k][kPos - 1] = positions[(m + k * step) * p.A + pair[V - 1].axis];
          }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (m + k * step >= p.M) break;
          Pos pos[V];
#pragma unroll
          for (int j = 0; j < V; ++j) pos[j] = kPos > 1 && (last >> j & 1) ? four[k][kPos - 1] : four[k][0];
          put(m + k * step, pos);
        }
      }
    };
    if (p.A == 1 || V == 1) {
      walk(std::integral_constant<int, 1>());
    } else if (two) {
      walk(std::integral_constant<int, 2>());
    } else {
      for (; m < p.M; m += step) {
        Pos pos[V];
#pragma unroll
        for (int j = 0; j < V; ++j) pos[j] = positions[m * p.A + pair[j].axis];
        put(m, pos);
      }
    }
  }
}

// cos, sin as [P, M]: neighbouring threads take neighbouring rows, a block kRopeTablePairs
// pairs, whose fractions are made once, in shared memory (100000 rows of 64 pairs, 51.6 MB: 14.0 us).
constexpr int kRopeTablePairs = 8;
__global__ void __launch_bounds__(256) rope_table_angle_major_kernel(const RopeParams p) {
  __shared__ RopePair pairs[kRopeTablePairs];
  const int i0 = blockIdx.y * kRopeTablePairs, n = min(p.P - i0, kRopeTablePairs);
  grid_dep_wait();
  grid_dep_launch();
  if (threadIdx.x < kRopeTablePairs) pairs[threadIdx.x] = rope_pair(p, i0 + min(static_cast<int>(threadIdx.x), n - 1));
  __syncthreads();
  for (size_t m = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x; m < p.M; m += static_cast<size_t>(gridDim.x) * 256) {
#pragma unroll
    for (int j = 0; j < kRopeTablePairs; j += 2) {
      if (j >= n) break;
      const RopePair a = pairs[j], b = pairs[j + 1];
      float2 c, s;
      rope_cos_sin2(rope_turn(rope_position(p, m, a.axis), a.fraction), rope_turn(rope_position(p, m, b.axis), b.fraction),
                    make_float2(a.scale, b.scale), c, s);
      const size_t at = static_cast<size_t>(i0 + j) * p.M + m;
      p.cos[at] = c.x;
      p.sin[at] = s.x;
      if (j + 1 < n) {
        p.cos[at + p.M] = c.y;
        p.sin[at + p.M] = s.y;
      }
    }
  }
}

}  // namespace svdq
