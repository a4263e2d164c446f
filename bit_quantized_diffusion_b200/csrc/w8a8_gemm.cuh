// w8a8_gemm.cuh -- the 8-bit linear: E4M3 activations and weights with one float32
// scale per activation row and per weight row, on tcgen05 kind::f8f6f4, with bias,
// activation, residual or the gated product in the epilogue.
//
//   z[m,n] = (sum_k a[m,k] w[n,k]) sa[m] sw[n] + bias[n]
//   plain:  Y[m,n] = act(z[m,n]) + residual[m,n]
//   gated:  Y[m,n] = act(z[m,n]) z[m, F + n]             (w holds 2F rows: gate, then up)
//
// The scales leave the sum over k, so the tensor cores add plain E4M3 products in
// float32 and the epilogue applies both scales once per output; nothing but Y is
// rounded to 16 bits, once.
//
// w8a8_gemm_kernel: persistent, a cluster of two CTAs on two SMs per 256 x bn tile
// (cta_group::2): each CTA stages its own 128 rows of A and half of the tile's bn B rows
// (128 bytes of K per row and stage, 128-byte swizzle). A gated tile takes bn / 2 gate
// rows in the first CTA and the matching bn / 2 up rows in the second, so both halves
// of an output meet in one accumulator and the [M, 2F] product never reaches memory.
// K need not fill the last stage: TMA fills both operands with zeros there.
//
// Warp roles per CTA (10 warps):
//   warp 0     TMA producer
//   warp 1     tensor-memory owner; in the leader CTA also the MMA issuer (one thread)
//   warps 2-9  epilogue, two warps per tensor-memory lane quadrant: accumulator -> shared
//              memory -> scales, bias, activation, residual -> memory
// Bound by the tensor cores and, over many launches, by the power cap: gated, 4608 x 3840 x
// 10240, 725 GFLOP, takes 229 us alone (3.17 PFLOP/s at 1.9 GHz) and 277-286 us in a row
// (1.15-1.25 GHz at 990 W); 4096 x 15360 x 3840 168 us alone (2.87 PFLOP/s), 207-220 in a row.
// Few columns or a short K: by the epilogue and by what a tile costs to start. Up to some 1000 rows: by
// the way of the operands through L2, since narrow tiles, or few, read A again for each (256 x 3840 x 3840
// 9.1 us, 256 x 15360 x 3840 23.1, gated 256 x 3840 x 10240 27; the memory's time is 3.0, 10.2, 12.9).
// Tensor memory holds two accumulators of up to 256 columns, so a tile's epilogue runs under
// the next tile's MMAs.
#pragma once

#include <type_traits>

#include "sm100.cuh"

namespace svdq {

constexpr int kW8Threads = 320;
constexpr int kW8EpiWarps = 8;
constexpr int kW8BM = 128;                      // rows per CTA (a pair's tile: 256)
constexpr int kW8MaxBN = 256;                   // accumulator columns per tile, at most
constexpr int kW8KStage = 128;                  // values (bytes) of K per stage
constexpr int kW8AStage = kW8BM * kW8KStage;    // 16 KB
constexpr int kW8StageOut = 4096;               // epilogue staging bytes per warp
constexpr uint32_t kW8Ring = 5 * (kW8AStage + kW8MaxBN / 2 * kW8KStage);  // 160 KB of stages
constexpr int kW8MaxStages = 8;
constexpr uint32_t kW8Out = kW8Ring;
constexpr uint32_t kW8Vec = kW8Out + kW8EpiWarps * kW8StageOut;  // per warp: scales [128], bias [128]
constexpr uint32_t kW8Bars = kW8Vec + kW8EpiWarps * 256 * 4;
constexpr uint32_t kW8TmemSlot = kW8Bars + 8 * (2 * kW8MaxStages + 4);
constexpr size_t kW8SmemBytes = kW8TmemSlot + 16 + 1024;
static_assert(kW8SmemBytes <= 232448, "shared memory of one CTA");

enum W8Act : int { kW8ActNone = 0, kW8ActGelu = 1, kW8ActSilu = 2 };

struct W8Params {
  int M, N, K;                 // N: output columns (F when gated)
  int bn;                      // accumulator columns per tile: a multiple of 32, gated of 64
  int stages;                  // ring stages of bn's size
  int tiles_m, tiles;
  int band, band_tiles;        // tiles run through bands of this many row tiles, M fastest within
  int act;
  int out_f32;
  const float* a_scale;        // [M]
  const float* w_scale;        // [N] or, gated, [2 N]
  const __nv_bfloat16* bias;   // like w_scale, or null
  const void* residual;        // the output's type, row stride ldr, or null
  int ldr;
  void* Y;
  int ldy;
  uint32_t* status;
};

// D[tmem] (+)= A[smem] B[smem]^T over both CTAs of a pair, kind::f8f6f4.
__device__ __forceinline__ void mma_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor, kind::f8f6f4: E4M3 A and B (format 0), f32 accumulator, K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(uint32_t M, uint32_t N) {
  return (1u << 4)            // D format: f32
         | ((N >> 3) << 17)   // N / 8
         | ((M >> 4) << 24);  // M / 16
}

// GELU (tanh form) through 1 + tanh(u) = 2 / (1 + exp(-2u)), and SiLU: y over one plus
// an exponential. Where the exponential overflows the quotient is 0, the limit of both. The fast
// exponential and quotient (2 + 1.17 |e| and 2 units in the last place) take the relative error up as
// the exponential grows, on the negative side: 3e-6 of silu(-20), which is 4e-8. (A 16-bit output's own
// rounding is 4e-3.)
__device__ __forceinline__ float w8_act(float y, int act) {
  if (act == kW8ActNone) return y;
  const float e = act == kW8ActSilu ? -y : -1.5957691216057308f * fmaf(0.044715f * y, y * y, y);
  return __fdividef(y, 1.0f + __expf(e));
}

// Each thread reads 16 consecutive columns of its lane from either address.
__device__ __forceinline__ void tmem_ld16x2(uint32_t a, uint32_t b, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(a));
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(b));
}

__device__ __forceinline__ void tmem_ld16(uint32_t a, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(a));
}

template <bool kGated, bool kF32>
__global__ void __launch_bounds__(kW8Threads, 1)
    w8a8_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                     const W8Params p) {
  const int NS = p.stages, half_n = p.bn / 2;
  const int tile_n = kGated ? half_n : p.bn;  // output columns per tile
  const uint32_t stage_bytes = kW8AStage + static_cast<uint32_t>(half_n) * kW8KStage;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int ktiles = (p.K + kW8KStage - 1) / kW8KStage;
  const int unit = blockIdx.x / 2, units = gridDim.x / 2;
  const int my_tiles = p.tiles > unit ? (p.tiles - 1 - unit) / units + 1 : 0;
  auto tile_mn = [&](int i, int& m0, int& n0) {
    const int t = unit + i * units;
    const int band = t / p.band_tiles, r = t - band * p.band_tiles;
    const int rows = min(p.band, p.tiles_m - band * p.band);
    m0 = (band * p.band + r % rows) * (2 * kW8BM);
    n0 = r / rows * tile_n;
  };
  auto a_st = [&](int s) { return sbase + s * stage_bytes; };
  auto b_st = [&](int s) { return a_st(s) + kW8AStage; };
  auto bar_full = [&](int s) { return sbase + kW8Bars + 8 * s; };
  auto bar_empty = [&](int s) { return sbase + kW8Bars + 8 * (NS + s); };
  auto bar_acc_full = [&](int b) { return sbase + kW8Bars + 8 * (2 * NS + b); };
  auto bar_acc_free = [&](int b) { return sbase + kW8Bars + 8 * (2 * NS + 2 + b); };
  auto lead = [&](uint32_t a) { return map_peer_smem(a, 0); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kW8TmemSlot);

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(bar_full(s), 1);   // the leader's producer, whose bytes cover both CTAs' loads
      mbar_init(bar_empty(s), 1);  // MMA commit
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_acc_full(b), 1);
      mbar_init(bar_acc_free(b), 2 * kW8EpiWarps);
    }
    fence_barrier_init();
    prefetch_tmap(&tm_a);
    prefetch_tmap(&tm_b);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_converged();
  grid_dep_wait();
  grid_dep_launch();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (elect_one()) {
      bool ok = true;
      int s = 0, phase = 0;  // ring stage, and the parity of its use
      long long loads = 0;
      for (int i = 0; i < my_tiles && ok; ++i) {
        int m0, n0;
        tile_mn(i, m0, n0);
        const int mrow = m0 + kW8BM * static_cast<int>(rank);
        const int nrow = n0 + (leader ? 0 : (kGated ? p.N : half_n));
        for (int kt = 0; kt < ktiles; ++kt) {
          ok = mbar_wait(bar_empty(s), phase ^ 1, p.status);
          if (!ok) break;
          if (leader) mbar_arrive_expect_tx(bar_full(s), 2 * stage_bytes);
          const uint32_t fb = lead(bar_full(s));
          tma_load_2d_pair(a_st(s), &tm_a, fb, kt * kW8KStage, mrow);
          tma_load_2d_pair(b_st(s), &tm_b, fb, kt * kW8KStage, nrow);
          if (++s == NS) s = 0, phase ^= 1;
          ++loads;
        }
      }
      // No CTA of the pair leaves (they meet at the end) before the last loads have landed, also
      // after a wait has run out
      for (int back = 1; leader && back <= NS && back <= loads; ++back) {
        if (--s < 0) s = NS - 1, phase ^= 1;
        mbar_wait(bar_full(s), phase, p.status);
      }
    }
  } else if (warp == 1) {
    if (leader && elect_one()) {
      bool ok = true;
      const uint32_t id = idesc_e4m3_f32(2 * kW8BM, p.bn);
      const uint64_t a0 = smem_desc(a_st(0), 16, 1024, kSwizzle128B);
      const uint64_t b0 = smem_desc(b_st(0), 16, 1024, kSwizzle128B);
      const uint64_t step = static_cast<uint64_t>(stage_bytes >> 4);
      int s = 0, phase = 0;
      for (int i = 0; i < my_tiles && ok; ++i) {
        const uint32_t acc = tmem + (i & 1) * kW8MaxBN;
        if (i >= 2) {  // both CTAs' epilogues have read this accumulator
          ok = mbar_wait(bar_acc_free(i & 1), ((i >> 1) - 1) & 1, p.status);
          if (!ok) break;
        }
        tc_fence_after();
        for (int kt = 0; kt < ktiles; ++kt) {
          ok = mbar_wait(bar_full(s), phase, p.status);
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = a0 + step * static_cast<uint64_t>(s), bd = b0 + step * static_cast<uint64_t>(s);
#pragma unroll
          for (int k = 0; k < 4; ++k)  // 32 values of K per MMA, 32 bytes (2 units) further along the row
            mma_f8_pair(acc, ad + 2 * k, bd + 2 * k, id, (kt > 0 || k > 0) ? 1u : 0u);
          tc_commit_pair(bar_empty(s), 0x3);
          if (++s == NS) s = 0, phase ^= 1;
        }
        if (ok) tc_commit_pair(bar_acc_full(i & 1), 0x3);
      }
    }
  } else {
    const int quad = warp & 3;         // tensor-memory lanes 32 quad .. 32 quad + 31
    const int half = (warp - 2) >> 2;  // which of the quadrant's two warps: it takes every other sub-tile
    const int ew = warp - 2;
    // A sub-tile (kCols output columns; gated, 16 gate and the 16 up columns) goes through shared
    // memory as it is, one row per lane (float32, 128-byte rows, gated 64-byte rows of gate and
    // of up, 16-byte units swizzled), and comes out in pieces of kWide adjacent columns, a row's
    // pieces in adjacent lanes: whole sectors to and from memory, and a lane keeps its columns'
    // scales and bias through a sub-tile, its rows' scales through a tile.
    constexpr int kCols = kGated ? 16 : 32, kWide = kF32 ? 4 : 8, kPieces = kCols / kWide, kRows = 32 / kPieces;
    const uint32_t buf = sbase + kW8Out + ew * kW8StageOut;
    float* sw_s = reinterpret_cast<float*>(smem + kW8Vec) + ew * 256;  // [4 sub-tiles][32]
    float* bias_s = sw_s + 128;
    const int subs = tile_n / kCols;  // a tile's sub-tiles; this warp's: half, half + 2, ...
    const int lrow = lane * kWide / kCols, lcol = lane * kWide % kCols;
    using Out = std::conditional_t<kF32, float, __nv_bfloat16>;
    const Out* residual = static_cast<const Out*>(p.residual);
    Out* out = static_cast<Out*>(p.Y);
    const bool add = !kGated && p.residual != nullptr;
    auto first_row = [&](int m0) { return m0 + kW8BM * static_cast<int>(rank) + quad * 32; };
    auto unit = [&](int row, int c) {  // 16-byte unit c of a row, in this warp's buffer
      return kGated ? buf + row * 64 + ((c ^ ((row >> 1) & 3)) << 4) : buf + row * 128 + ((c ^ (row & 7)) << 4);
    };
    // scales and bias of this warp's columns, scales of the lane's rows: read a tile ahead
    float nsw[4], nbias[4], nsa[kPieces];
    auto read_scales = [&](int i) {
      int m0, n0;
      tile_mn(i, m0, n0);
      const int mrow = first_row(m0);
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int m = mrow + k * kRows + lrow;
        nsa[k] = m < p.M ? p.a_scale[m] : 0.0f;
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int oc = n0 + (2 * t + half) * kCols + lane % kCols;
        const int row = kGated && lane >= 16 ? p.N + oc : oc;
        const bool in = 2 * t + half < subs && oc < p.N;
        nsw[t] = in ? p.w_scale[row] : 0.0f;
        nbias[t] = in && p.bias != nullptr ? __bfloat162float(p.bias[row]) : 0.0f;
      }
      if (add && mrow + lane < p.M)
        for (int t = half; t < subs && n0 + t * 32 < p.N; t += 2)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(residual + static_cast<size_t>(mrow + lane) * p.ldr + n0 + t * 32));
    };
    uint4 res[kPieces];  // the residual of a sub-tile, read one sub-tile ahead
    auto read_residual = [&](int mrow, int n) {
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int m = mrow + k * kRows + lrow;
        if (m < p.M && n + lcol < p.N)
          res[k] = *reinterpret_cast<const uint4*>(residual + static_cast<size_t>(m) * p.ldr + n + lcol);
      }
    };
    bool ok = true;
    if (my_tiles > 0) {
      read_scales(0);
      int m0, n0;
      tile_mn(0, m0, n0);
      if (add && half < subs) read_residual(first_row(m0), n0 + half * kCols);
    }
    for (int i = 0; i < my_tiles && ok; ++i) {
      int m0, n0;
      tile_mn(i, m0, n0);
      const int mrow = first_row(m0);
      float sa[kPieces];
#pragma unroll
      for (int k = 0; k < kPieces; ++k) sa[k] = nsa[k];
      __syncwarp();
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        sw_s[t * 32 + lane] = nsw[t];
        bias_s[t * 32 + lane] = nbias[t];
      }
      if (i + 1 < my_tiles) read_scales(i + 1);
      ok = mbar_wait(bar_acc_full(i & 1), (i >> 1) & 1, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t t_row = tmem + (i & 1) * kW8MaxBN + (static_cast<uint32_t>(quad * 32) << 16);
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(lead(bar_acc_free(i & 1)));
      };
      if (half >= subs) release();
#pragma unroll 1
      for (int t = half; t < subs; t += 2) {
        uint32_t acc[32];
        if constexpr (kGated) tmem_ld16x2(t_row + t * 16, t_row + half_n + t * 16, acc);
        else tmem_ld32(t_row + t * 32, acc);
        tmem_ld_wait();
        if (t + 2 >= subs) release();
        __syncwarp();  // the sub-tile before has been read
#pragma unroll
        for (int c = 0; c < 8; ++c)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(kGated ? unit(lane, c & 3) + (c >> 2) * 2048 : unit(lane, c)),
                       "r"(acc[4 * c]), "r"(acc[4 * c + 1]), "r"(acc[4 * c + 2]), "r"(acc[4 * c + 3])
                       : "memory");
        __syncwarp();
        const int n = n0 + t * kCols;
        if (n < p.N && mrow < p.M) {  // warp-uniform
          const float* swp = sw_s + (t >> 1) * 32 + lcol;
          const float* bp = bias_s + (t >> 1) * 32 + lcol;
          float4 sw[kWide / 4], bias[kWide / 4], usw[kWide / 4], ubias[kWide / 4];
#pragma unroll
          for (int q = 0; q < kWide / 4; ++q) {
            sw[q] = reinterpret_cast<const float4*>(swp)[q];
            bias[q] = reinterpret_cast<const float4*>(bp)[q];
            if (kGated) {
              usw[q] = reinterpret_cast<const float4*>(swp + 16)[q];
              ubias[q] = reinterpret_cast<const float4*>(bp + 16)[q];
            }
          }
#pragma unroll
          for (int k = 0; k < kPieces; ++k) {
            const int row = k * kRows + lrow, m = mrow + row;
            const float2 s2 = make_float2(sa[k], sa[k]);
            float2 y[kWide / 2];
#pragma unroll
            for (int q = 0; q < kWide / 4; ++q) {
              const float4 v = lds_f4(unit(row, lcol / 4 + q));
              y[2 * q] = __ffma2_rn(__fmul2_rn(make_float2(v.x, v.y), s2), make_float2(sw[q].x, sw[q].y),
                                    make_float2(bias[q].x, bias[q].y));
              y[2 * q + 1] = __ffma2_rn(__fmul2_rn(make_float2(v.z, v.w), s2), make_float2(sw[q].z, sw[q].w),
                                        make_float2(bias[q].z, bias[q].w));
            }
            if (p.act != kW8ActNone) {
#pragma unroll
              for (int q = 0; q < kWide / 2; ++q) y[q] = make_float2(w8_act(y[q].x, p.act), w8_act(y[q].y, p.act));
            }
            if constexpr (kGated) {
#pragma unroll
              for (int q = 0; q < kWide / 4; ++q) {
                const float4 v = lds_f4(unit(row, lcol / 4 + q) + 2048);
                y[2 * q] = __fmul2_rn(y[2 * q], __ffma2_rn(__fmul2_rn(make_float2(v.x, v.y), s2), make_float2(usw[q].x, usw[q].y),
                                                           make_float2(ubias[q].x, ubias[q].y)));
                y[2 * q + 1] = __fmul2_rn(y[2 * q + 1], __ffma2_rn(__fmul2_rn(make_float2(v.z, v.w), s2), make_float2(usw[q].z, usw[q].w),
                                                                   make_float2(ubias[q].z, ubias[q].w)));
              }
            }
            uint32_t w[4];
            if constexpr (kF32) {
              if (add) {
                y[0] = __fadd2_rn(y[0], make_float2(__uint_as_float(res[k].x), __uint_as_float(res[k].y)));
                y[1] = __fadd2_rn(y[1], make_float2(__uint_as_float(res[k].z), __uint_as_float(res[k].w)));
              }
              w[0] = __float_as_uint(y[0].x); w[1] = __float_as_uint(y[0].y);
              w[2] = __float_as_uint(y[1].x); w[3] = __float_as_uint(y[1].y);
            } else {
              const uint32_t r4[4] = {res[k].x, res[k].y, res[k].z, res[k].w};
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                if (add)
                  y[q] = __fadd2_rn(y[q], make_float2(__uint_as_float(r4[q] << 16), __uint_as_float(r4[q] & 0xFFFF0000u)));
                const __nv_bfloat162 b2 = __float22bfloat162_rn(y[q]);
                w[q] = *reinterpret_cast<const uint32_t*>(&b2);
              }
            }
            if (m < p.M && n + lcol < p.N)
              *reinterpret_cast<uint4*>(out + static_cast<size_t>(m) * p.ldy + n + lcol) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        if (add) {
          if (t + 2 < subs) {
            read_residual(mrow, n + 2 * kCols);
          } else if (i + 1 < my_tiles) {
            int m1, n1;
            tile_mn(i + 1, m1, n1);
            read_residual(first_row(m1), n1 + half * kCols);
          }
        }
      }
    }
  }

  tc_fence_before();
  // the leader's MMAs write both CTAs' tensor memory: release it once every warp
  // of the pair is done
  cluster_sync_converged();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// w8a8_stream_kernel: up to 128 tokens (or tiles of as many, where a long K meets few
// columns), where the product is bound by reading the weight once. The operands change sides: 128
// weight rows are the MMA's M (tensor-memory lanes), the tokens, rounded up to 16, its N, so a
// handful of tokens costs no padding to 256 rows. One tile of 128 weight rows (gated: 64 gate rows and the 64 matching up
// rows) per cluster, whose CTAs split K and add their float32 partial sums through
// distributed shared memory, in rank order: weights narrower than a row tile per SM
// still keep every SM loading, without memory to add in and without atomics.
// Bound by HBM: gated, 4 x 3840 x 10240, 78.8 MB: 15.0 us, 5.2 TB/s; 77 x 3840 x 15360 with GELU,
// 61.7 MB: 14.9 us; 128 x 3840 x 15360 with a residual, 67.3 MB: 17.0 us. (Unsplit tiles too through
// shared memory [T][128] and 8-byte stores by all warps: 15.0, 15.5 and 19.5 us.)
//
//   warp 0     TMA producer: W [2 x 64 rows x 128 B] and X [T x 128 B] per stage
//   warp 1     tensor-memory owner and MMA issuer (one thread)
//   warps 2-9  the residual's lines into L2; then the accumulator, two warps per tensor-memory
//              lane quadrant. One CTA per tile: straight to the outputs, a lane per weight row,
//              whose scale, bias and residual it holds by then (gated, the gate's warps take half
//              of the tokens and the up rows' the other half, and each hands the other's over
//              through shared memory). A cluster: to shared memory [T][128]
//   all warps  of a cluster: the sum over it and the epilogue, four adjacent outputs per
//              thread and step, a thread's columns the same in every step
constexpr int kWsThreads = 320;
constexpr int kWsMaxT = 128;
constexpr int kWsMaxStages = 12;
constexpr size_t kWsWholeSm = 226 * 1024, kWsHalfSm = 113 * 1024;  // a CTA's shared memory, at most

struct WsParams {
  int M, N, K;                 // N: output columns (F when gated)
  int T, tb;                   // tokens per tile, a multiple of 16; tensor-memory columns (32, 64, 128)
  int splits, stages;          // cluster size; pipeline stages
  int shared;                  // more CTAs than SMs: two on one
  int act, out_f32;
  const float* a_scale;
  const float* w_scale;
  const __nv_bfloat16* bias;
  const void* residual;
  size_t ldr;
  void* Y;
  size_t ldy;
  uint32_t* status;
};

__host__ __device__ constexpr uint32_t ws_stage_bytes(int T) { return 128 * 128 + static_cast<uint32_t>(T) * 128; }
constexpr uint32_t kWsTail = 512 + 8 * (2 * kWsMaxStages + 1) + 24;  // token scales [128], barriers, tensor-memory slot
__host__ __device__ constexpr size_t ws_smem_bytes(int T, int stages) {
  return static_cast<size_t>(stages) * ws_stage_bytes(T) + kWsTail + 1024;
}

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ float4 lds_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

// four adjacent values of the output's type
__device__ __forceinline__ void w8_load4(const void* base, size_t at, int f32, float (&r)[4]) {
  if (f32) {
    const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(base) + at);
    r[0] = __uint_as_float(v.x << 16); r[1] = __uint_as_float(v.x & 0xFFFF0000u);
    r[2] = __uint_as_float(v.y << 16); r[3] = __uint_as_float(v.y & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void w8_store4(void* base, size_t at, int f32, const float (&y)[4]) {
  if (f32) {
    *reinterpret_cast<float4*>(static_cast<float*>(base) + at) = make_float4(y[0], y[1], y[2], y[3]);
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(y[0], y[1]), b = __floats2bfloat162_rn(y[2], y[3]);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(base) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
}

template <bool kGated, bool kSplit>
__global__ void __launch_bounds__(kWsThreads, 2)
    w8a8_stream_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                       const WsParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int NS = p.stages, T = p.T;
  const uint32_t SB = ws_stage_bytes(T);
  float* sa_s = reinterpret_cast<float*>(smem + NS * SB);
  const uint32_t bars = sbase + NS * SB + 512;
  auto bar_full = [&](int s) { return bars + 8 * s; };
  auto bar_empty = [&](int s) { return bars + 8 * (NS + s); };
  const uint32_t bar_acc = bars + 8 * 2 * NS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + NS * SB + 512 + 8 * (2 * NS + 1));
  const int splits = kSplit ? p.splits : 1;
  const int rank = kSplit ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = blockIdx.x / splits;
  constexpr int kCols = kGated ? 64 : 128;      // output columns per tile
  const int n0 = tile * kCols;
  // this tile's tokens; more than one tile only where K is split
  const int m0 = kSplit ? blockIdx.y * T : 0, rows = kSplit ? min(T, p.M - m0) : p.M;
  const int ktiles = (p.K + kW8KStage - 1) / kW8KStage;
  const int k0 = rank * ktiles / splits, k1 = (rank + 1) * ktiles / splits;

  auto load = [&](int kt, int s) {
    const uint32_t st = sbase + s * SB;
    mbar_arrive_expect_tx(bar_full(s), SB);
    tma_load_2d(st, &tm_w, bar_full(s), kt * kW8KStage, n0);
    tma_load_2d(st + 64 * 128, &tm_w, bar_full(s), kt * kW8KStage, kGated ? p.N + n0 : n0 + 64);
    tma_load_2d(st + 128 * 128, &tm_x, bar_full(s), kt * kW8KStage, m0);
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 1);
    }
    mbar_init(bar_acc, 1);
    fence_barrier_init();
    // the first loads, which wait for no one else's set-up
    grid_dep_wait();
    for (int g = 0; g < NS && k0 + g < k1; ++g) load(k0 + g, g);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), p.tb);
    tmem_relinquish();
  }
  tc_fence_before();
  cta_sync_converged();
  // The next grid's set-up under this one's work; but where this grid's blocks share SMs, only
  // at its end: the next one's blocks would take the second places (gated, 4 x 3840 x 10240, calls
  // in a row: 18.8 us, and 15.2 at the end).
  grid_dep_wait();
  if (!p.shared) grid_dep_launch();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // a CTA's share of its cluster's outputs: items of four adjacent columns, e .. e1 in
  // steps of the block, which keep a thread at the same columns; their scales and bias now
  constexpr int kQuads = kCols / 4;
  static_assert(kWsThreads % kQuads == 0, "a thread keeps its columns");
  const int items = rows * kQuads;
  const int e1 = (rank + 1) * items / splits;
  int e = rank * items / splits + static_cast<int>(threadIdx.x);
  const int c = 4 * (e % kQuads), n = n0 + c;
  float sw[kGated ? 8 : 4], bias[kGated ? 8 : 4];
#pragma unroll
  for (int q = 0; kSplit && q < (kGated ? 8 : 4); ++q) {
    const int row = (q < 4 ? n : p.N + n) + (q & 3);
    sw[q] = n < p.N ? p.w_scale[row] : 0.0f;
    bias[q] = n < p.N && p.bias != nullptr ? __bfloat162float(p.bias[row]) : 0.0f;
  }
  // a step's residual, the first now, each other one a step ahead
  float r[4];
  auto residual = [&](int from) {
    if (p.residual != nullptr && n < p.N && from < e1)
      w8_load4(p.residual, static_cast<size_t>(m0 + from / kQuads) * p.ldr + n, p.out_f32, r);
  };
  if (kSplit) residual(e);
  // the cluster's four sums of row m from accumulator column col, in rank order
  auto sum4 = [&](int m, int col) {
    const uint32_t at = sbase + (m * 128 + col) * 4;
    float4 v = lds_cluster_f4(map_peer_smem(at, 0));
#pragma unroll 4
    for (int r = 1; r < splits; ++r) {
      const float4 o = lds_cluster_f4(map_peer_smem(at, r));
      v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
    }
    return v;
  };

  if (warp == 0) {
    if (lane == 0) {
      int last = min(NS, k1 - k0) - 1;
      for (int g = NS; k0 + g < k1; ++g) {
        const int s = g % NS;
        if (!mbar_wait(bar_empty(s), ((g / NS) & 1) ^ 1, p.status)) break;
        load(k0 + g, s);
        last = g;
      }
      // the last loads have landed before the block ends, also after a wait has run out
      for (int g = max(0, last - NS + 1); g <= last; ++g) mbar_wait(bar_full(g % NS), (g / NS) & 1, p.status);
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t id = idesc_e4m3_f32(128, T);
      bool ok = true;
      for (int kt = k0; kt < k1; ++kt) {
        const int g = kt - k0, s = g % NS;
        ok = mbar_wait(bar_full(s), (g / NS) & 1, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t st = sbase + s * SB;
        const uint64_t wd = smem_desc(st, 16, 1024, kSwizzle128B);
        const uint64_t xd = smem_desc(st + 128 * 128, 16, 1024, kSwizzle128B);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_f8(tmem, wd + 2 * k, xd + 2 * k, id, (g > 0 || k > 0) ? 1u : 0u);
        tc_commit(bar_empty(s));
      }
      if (ok) tc_commit(bar_acc);
    }
  } else {
    const int quad = warp & 3;
    for (int i = threadIdx.x - 64; i < rows; i += kWsThreads - 64) sa_s[i] = p.a_scale[m0 + i];
    if (p.residual != nullptr) {
      // the residual in whole lines: what is read at the end would add a latency per step, and a lane's
      // two bytes of many rows, unsplit, reach memory slower (100 x 512 x 15360: 8.6 us, without 9.4)
      const int esz = p.out_f32 ? 4 : 2, lines = kCols * esz / 128;
      for (int i = threadIdx.x - 64; i < rows * lines; i += kWsThreads - 64) {
        const int col = n0 + (i % lines) * (128 / esz);
        if (col < p.N)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(p.residual) +
                                                        (static_cast<size_t>(m0 + i / lines) * p.ldr + col) * esz));
      }
    }
    const uint32_t t_row = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const int half = (warp - 2) / 4;
    if constexpr (kSplit) {
      // the stages' memory is free once the last MMA is done
      bool ok = mbar_wait(bar_acc, 0, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) {
        tc_fence_after();
        float* part = reinterpret_cast<float*>(smem);  // [T][128]
        for (int c = half * 32; c < T; c += 64) {
          uint32_t acc[32];
          tmem_ld32(t_row + c, acc);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < 32; ++q)
            if (c + q < T) part[(c + q) * 128 + quad * 32 + lane] = __uint_as_float(acc[q]);
        }
        tc_fence_before();
      }
    } else {
      // every other 16 tokens of the quadrant's rows; gated, eight of each 16 per warp
      constexpr int kKeep = kGated ? 8 : 16;
      const bool up = kGated && quad >= 2;
      const int col = (kGated ? quad & 1 : quad) * 32 + lane, n = n0 + col, first = up ? 8 : 0;
      const bool in = n < p.N;
      const float sw = in ? p.w_scale[n] : 0.0f, usw = kGated && in ? p.w_scale[p.N + n] : 0.0f;
      const float bias = in && p.bias != nullptr ? __bfloat162float(p.bias[n]) : 0.0f;
      const float ubias = kGated && in && p.bias != nullptr ? __bfloat162float(p.bias[p.N + n]) : 0.0f;
      // the residual of the warp's 16 tokens k: all of it now in bf16, two values to a register; in
      // float32 two k ahead
      uint32_t res[kGated ? 1 : 32];
      const bool add = !kGated && p.residual != nullptr && in;
      auto read_residual = [&](int k) {
        const int from = half * 16 + 32 * k;
        if (add && from < rows) {
          // (behind the last row: that one again, so that no branch parts the loads)
          auto at = [&](int q) { return static_cast<size_t>(min(from + q, rows - 1)) * p.ldr + n; };
          if (p.out_f32) {
#pragma unroll
            for (int q = 0; q < 16; ++q)
              res[k % 2 * 16 + q] = __float_as_uint(static_cast<const float*>(p.residual)[at(q)]);
          } else {
            uint32_t v[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) v[q] = static_cast<const uint16_t*>(p.residual)[at(q)];
#pragma unroll
            for (int q = 0; q < 8; ++q) res[k * 8 + q] = v[2 * q] | v[2 * q + 1] << 16;
          }
        }
      };
      if constexpr (!kGated) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k < 2 || !p.out_f32) read_residual(k);
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");  // the tokens' scales
      bool ok = mbar_wait(bar_acc, 0, p.status);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      if (p.shared) grid_dep_launch();
      float* other = reinterpret_cast<float*>(smem) + col;  // [T][64], in the stages' memory, free now
      uint32_t acc[16];
      if (kGated) {
        for (int c = half * 16; ok && c < T; c += 32) {
          tmem_ld16(t_row + c, acc);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < 8; ++q) other[(c + 8 - first + q) * 64] = __uint_as_float(up ? acc[q] : acc[8 + q]);
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");  // (also after a wait has run out)
      }
#pragma unroll
      for (int k = 0; k < kWsMaxT / 32; ++k) {
        const int c = half * 16 + 32 * k;
        if (!ok || c >= T) break;
        tmem_ld16(t_row + c, acc);
        tmem_ld_wait();
        float2 y[kKeep / 2];  // of tokens 2 q, 2 q + 1 (behind the last row: the scale of none, not stored)
#pragma unroll
        for (int q = 0; q < kKeep / 2; ++q) {
          const int m = c + first + 2 * q;
          const float2 sa = *reinterpret_cast<const float2*>(sa_s + m);
          const float2 v = __fmul2_rn(up ? make_float2(__uint_as_float(acc[(2 * q + 8) % 16]), __uint_as_float(acc[(2 * q + 9) % 16]))
                                         : make_float2(__uint_as_float(acc[2 * q]), __uint_as_float(acc[2 * q + 1])), sa);
          if constexpr (kGated) {
            const float2 o = __fmul2_rn(make_float2(other[m * 64], other[(m + 1) * 64]), sa);
            const float2 gate = __ffma2_rn(up ? o : v, make_float2(sw, sw), make_float2(bias, bias));
            const float2 through = __ffma2_rn(up ? v : o, make_float2(usw, usw), make_float2(ubias, ubias));
            y[q] = __fmul2_rn(make_float2(w8_act(gate.x, p.act), w8_act(gate.y, p.act)), through);
          } else {
            const float2 z = __ffma2_rn(v, make_float2(sw, sw), make_float2(bias, bias));
            y[q] = make_float2(w8_act(z.x, p.act), w8_act(z.y, p.act));
          }
        }
        if constexpr (!kGated) {
          if (add) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const uint32_t two = res[k * 8 + q], a = res[k % 2 * 16 + 2 * q], b = res[k % 2 * 16 + 2 * q + 1];
              y[q] = __fadd2_rn(y[q], make_float2(__uint_as_float(p.out_f32 ? a : two << 16),
                                                  __uint_as_float(p.out_f32 ? b : two & 0xFFFF0000u)));
            }
          }
          if (k < 2 && p.out_f32) read_residual(k + 2);
        }
        if (p.out_f32) {
          float* at = static_cast<float*>(p.Y) + static_cast<size_t>(c + first) * p.ldy + n;
#pragma unroll
          for (int q = 0; q < kKeep; ++q) {
            if (in && c + first + q < rows) *at = q % 2 ? y[q / 2].y : y[q / 2].x;
            at += p.ldy;
          }
        } else {
          // neighbouring lanes trade a token each: a lane stores two columns of every other token
          const bool odd = lane & 1;
          __nv_bfloat16* at = static_cast<__nv_bfloat16*>(p.Y) + static_cast<size_t>(c + first + odd) * p.ldy + (n - odd);
#pragma unroll
          for (int q = 0; q < kKeep / 2; ++q) {
            const float got = __shfl_xor_sync(0xffffffffu, odd ? y[q].x : y[q].y, 1);
            const __nv_bfloat162 two = odd ? __floats2bfloat162_rn(got, y[q].y) : __floats2bfloat162_rn(y[q].x, got);
            if (in && c + first + odd + 2 * q < rows) *reinterpret_cast<__nv_bfloat162*>(at) = two;
            at += 2 * p.ldy;
          }
        }
      }
      tc_fence_before();
    }
  }
  if (kSplit) cluster_sync_converged(); else cta_sync_converged();
  if (kSplit && p.shared) grid_dep_launch();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tb);
  }
  if (kSplit && n < p.N) {
    for (; e < e1; e += kWsThreads) {
      const int m = e / kQuads;
      const float sa = sa_s[m];
      const float4 v = sum4(m, c);
      float y[4];
      y[0] = fmaf(v.x * sa, sw[0], bias[0]);
      y[1] = fmaf(v.y * sa, sw[1], bias[1]);
      y[2] = fmaf(v.z * sa, sw[2], bias[2]);
      y[3] = fmaf(v.w * sa, sw[3], bias[3]);
#pragma unroll
      for (int q = 0; q < 4; ++q) y[q] = w8_act(y[q], p.act);
      if (kGated) {
        const float4 w = sum4(m, 64 + c);
        y[0] *= fmaf(w.x * sa, sw[4], bias[4]);
        y[1] *= fmaf(w.y * sa, sw[5], bias[5]);
        y[2] *= fmaf(w.z * sa, sw[6], bias[6]);
        y[3] *= fmaf(w.w * sa, sw[7], bias[7]);
      }
      if (p.residual != nullptr) {
#pragma unroll
        for (int q = 0; q < 4; ++q) y[q] += r[q];
      }
      residual(e + kWsThreads);
      w8_store4(p.Y, static_cast<size_t>(m0 + m) * p.ldy + n, p.out_f32, y);
    }
  }
  // peers read this CTA's sums until here
  if (kSplit) cluster_sync_converged();
}

// w8a8_gemv_kernel: up to 16 tokens of a small weight. There the tensor-memory kernels' set-up (tensor maps,
// barriers, tensor memory, the first copy's way) is as long as reading the weight, so a
// block of 16 weight rows (gated: 8 gate rows and the 8 matching up rows) reads it straight
// into the fragments of the warp-level MMA, m16n8k32 on E4M3. The sum over k may run in any
// order, so a lane's 16 bytes of a row are the fragments of two MMAs as they lie there, and
// its 16 bytes of a token match them: neither operand passes through shared memory. Warps
// take every other 64 bytes of K; their partial sums meet in shared memory in a fixed order.
// One token, K = N = 3840, 14.8 MB: 5.7 us, of which an empty launch is 2.2; 240 blocks leave some SMs
// two of them and others one.
constexpr int kWvMaxM = 16;
constexpr int kWvUnroll = 4;  // 64-byte steps whose loads are on their way together

// (Not the read-only path, here and for the tokens: the grid before, which may have made either operand, can
// still be writing when this one starts.)
__device__ __forceinline__ uint4 ldg_stream(const uint8_t* at) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(at));
  return v;
}

__device__ __forceinline__ void mma_e4m3_16832(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
      " {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct WvParams {
  int M, N, K;                 // N: output columns (F when gated)
  const uint8_t* a;            // [M, K]
  const uint8_t* w;            // [N, K] or, gated, [2 N, K]
  int act, out_f32;
  const float* a_scale;
  const float* w_scale;
  const __nv_bfloat16* bias;
  const void* residual;
  size_t ldr;
  void* Y;
  size_t ldy;
};

template <bool kGated, int kTokens8>  // kTokens8: groups of 8 tokens
__global__ void __launch_bounds__(512) w8a8_gemv_kernel(const WvParams p) {
  __shared__ float part[16][16 * 8 * kTokens8];  // [warp][weight row][token]
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t = lane % 4;
  constexpr int kCols = kGated ? 8 : 16;
  const int n0 = blockIdx.x * kCols;
  const size_t K = p.K;
  const uint8_t* w0 = p.w + (static_cast<size_t>(n0) + g) * K + 16 * t;
  const uint8_t* w1 = p.w + (static_cast<size_t>(kGated ? p.N + n0 : n0 + 8) + g) * K + 16 * t;
  grid_dep_wait();
  grid_dep_launch();
  float acc[kTokens8][4] = {};
  for (int k0 = 64 * warp; k0 < p.K; k0 += 64 * warps * kWvUnroll) {
    uint4 a[kWvUnroll][2], b[kWvUnroll][kTokens8];
#pragma unroll
    for (int u = 0; u < kWvUnroll; ++u) {
      const int k = k0 + 64 * warps * u;
      const bool in = k + 16 * t < p.K;
      a[u][0] = in ? ldg_stream(w0 + k) : make_uint4(0, 0, 0, 0);
      a[u][1] = in ? ldg_stream(w1 + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < kTokens8; ++j)
        b[u][j] = in && 8 * j + g < p.M
                      ? *reinterpret_cast<const uint4*>(p.a + (8 * j + g) * K + k + 16 * t)
                      : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kWvUnroll; ++u)
#pragma unroll
      for (int j = 0; j < kTokens8; ++j) {
        mma_e4m3_16832(acc[j], a[u][0].x, a[u][1].x, a[u][0].y, a[u][1].y, b[u][j].x, b[u][j].y);
        mma_e4m3_16832(acc[j], a[u][0].z, a[u][1].z, a[u][0].w, a[u][1].w, b[u][j].z, b[u][j].w);
      }
  }
  // (row g, tokens 2t, 2t + 1) and (row g + 8, the same tokens) of each group of tokens
#pragma unroll
  for (int j = 0; j < kTokens8; ++j) {
    part[warp][(8 * j + 2 * t) * 16 + g] = acc[j][0];
    part[warp][(8 * j + 2 * t + 1) * 16 + g] = acc[j][1];
    part[warp][(8 * j + 2 * t) * 16 + g + 8] = acc[j][2];
    part[warp][(8 * j + 2 * t + 1) * 16 + g + 8] = acc[j][3];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.M * kCols; e += blockDim.x) {
    const int m = e / kCols, c = e % kCols, n = n0 + c;
    auto z = [&](int row16, int row) {
      float s = part[0][m * 16 + row16];
      for (int i = 1; i < warps; ++i) s += part[i][m * 16 + row16];
      return fmaf(s * p.a_scale[m], p.w_scale[row], p.bias != nullptr ? __bfloat162float(p.bias[row]) : 0.0f);
    };
    float y = w8_act(z(c, n), p.act);
    if (kGated) y *= z(c + 8, p.N + n);
    const size_t at = static_cast<size_t>(m) * p.ldy + n, ar = static_cast<size_t>(m) * p.ldr + n;
    if (p.out_f32) {
      if (p.residual != nullptr) y += static_cast<const float*>(p.residual)[ar];
      static_cast<float*>(p.Y)[at] = y;
    } else {
      if (p.residual != nullptr) y += __bfloat162float(static_cast<const __nv_bfloat16*>(p.residual)[ar]);
      static_cast<__nv_bfloat16*>(p.Y)[at] = __float2bfloat16_rn(y);
    }
  }
}

}  // namespace svdq
