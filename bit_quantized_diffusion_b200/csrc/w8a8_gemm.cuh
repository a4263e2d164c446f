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
// w8a8_gemm_kernel: persistent, a cluster of two CTAs on two SMs per 256 x 256 tile
// (cta_group::2): each CTA stages its own 128 rows of A and 128 of the tile's B rows
// (128 bytes of K per row and stage, 128-byte swizzle). A gated tile takes 128 gate
// rows in the first CTA and the matching 128 up rows in the second, so both halves
// of an output meet in one accumulator and the [M, 2F] product never reaches memory.
// K need not fill the last stage: TMA fills both operands with zeros there.
//
// Warp roles per CTA (10 warps):
//   warp 0     TMA producer
//   warp 1     tensor-memory owner; in the leader CTA also the MMA issuer (one thread)
//   warps 2-9  epilogue, two warps per tensor-memory lane quadrant
// Tensor memory holds two 256-column accumulators, so a tile's epilogue runs under
// the next tile's MMAs.
#pragma once

#include "sm100.cuh"

namespace svdq {

constexpr int kW8Threads = 320;
constexpr int kW8EpiWarps = 8;
constexpr int kW8BM = 128;                      // rows per CTA (a pair's tile: 256)
constexpr int kW8BN = 256;                      // accumulator columns per tile
constexpr int kW8KStage = 128;                  // values (bytes) of K per stage
constexpr int kW8Stages = 5;
constexpr int kW8AStage = kW8BM * kW8KStage;    // 16 KB
constexpr int kW8BStage = (kW8BN / 2) * kW8KStage;
constexpr int kW8StageBytes = kW8AStage + kW8BStage;
constexpr int kW8StageOut = 4096;               // epilogue staging bytes per warp
constexpr uint32_t kW8Out = kW8Stages * kW8StageBytes;
constexpr uint32_t kW8Vec = kW8Out + kW8EpiWarps * kW8StageOut;  // per warp: scales [128], bias [128]
constexpr uint32_t kW8Bars = kW8Vec + kW8EpiWarps * 256 * 4;
constexpr uint32_t kW8TmemSlot = kW8Bars + 8 * (2 * kW8Stages + 4);
constexpr size_t kW8SmemBytes = kW8TmemSlot + 16 + 1024;
static_assert(kW8SmemBytes <= 232448, "shared memory of one CTA");

enum W8Act : int { kW8ActNone = 0, kW8ActGelu = 1, kW8ActSilu = 2 };

struct W8Params {
  int M, N, K;                 // N: output columns (F when gated)
  int tiles_m, tiles;
  int act;
  int out_f32;
  const float* a_scale;        // [M]
  const float* w_scale;        // [N] or, gated, [2 N]
  const __nv_bfloat16* bias;   // like w_scale, or null
  const void* residual;        // the output's type, row stride ldr, or null
  int ldr;
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
// an exponential. Where the exponential overflows the quotient is 0, the limit of both.
__device__ __forceinline__ float w8_act(float y, int act) {
  if (act == kW8ActNone) return y;
  const float e = act == kW8ActSilu ? -y : -1.5957691216057308f * fmaf(0.044715f * y, y * y, y);
  return __fdividef(y, 1.0f + __expf(e));
}

template <bool kGated>
__global__ void __launch_bounds__(kW8Threads, 1)
    w8a8_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                     const __grid_constant__ CUtensorMap tm_y, const W8Params p) {
  constexpr int NS = kW8Stages;
  constexpr int kTileN = kGated ? kW8BN / 2 : kW8BN;  // output columns per tile
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
    m0 = (t % p.tiles_m) * (2 * kW8BM);
    n0 = (t / p.tiles_m) * kTileN;
  };
  auto a_st = [&](int s) { return sbase + s * kW8StageBytes; };
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
    prefetch_tmap(&tm_y);
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
      int g = 0;
      for (int i = 0; i < my_tiles && ok; ++i) {
        int m0, n0;
        tile_mn(i, m0, n0);
        const int mrow = m0 + kW8BM * static_cast<int>(rank);
        const int nrow = kGated ? n0 + (leader ? 0 : p.N) : n0 + kW8BN / 2 * static_cast<int>(rank);
        for (int kt = 0; kt < ktiles; ++kt, ++g) {
          const int s = g % NS;
          ok = mbar_wait(bar_empty(s), ((g / NS) & 1) ^ 1, p.status);
          if (!ok) break;
          if (leader) mbar_arrive_expect_tx(bar_full(s), 2 * kW8StageBytes);
          const uint32_t fb = lead(bar_full(s));
          tma_load_2d_pair(a_st(s), &tm_a, fb, kt * kW8KStage, mrow);
          tma_load_2d_pair(b_st(s), &tm_b, fb, kt * kW8KStage, nrow);
        }
      }
    }
  } else if (warp == 1) {
    if (leader && elect_one()) {
      bool ok = true;
      constexpr uint32_t id = idesc_e4m3_f32(2 * kW8BM, kW8BN);
      const uint64_t a0 = smem_desc(a_st(0), 16, 1024, kSwizzle128B);
      const uint64_t b0 = smem_desc(b_st(0), 16, 1024, kSwizzle128B);
      constexpr uint64_t kStep = static_cast<uint64_t>(kW8StageBytes >> 4);
      int g = 0;
      for (int i = 0; i < my_tiles && ok; ++i) {
        const uint32_t acc = tmem + (i & 1) * kW8BN;
        if (i >= 2) {  // both CTAs' epilogues have read this accumulator
          ok = mbar_wait(bar_acc_free(i & 1), ((i >> 1) - 1) & 1, p.status);
          if (!ok) break;
        }
        tc_fence_after();
        for (int kt = 0; kt < ktiles; ++kt, ++g) {
          const int s = g % NS;
          ok = mbar_wait(bar_full(s), (g / NS) & 1, p.status);
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = a0 + kStep * static_cast<uint64_t>(s), bd = b0 + kStep * static_cast<uint64_t>(s);
#pragma unroll
          for (int k = 0; k < 4; ++k)  // 32 values of K per MMA, 32 bytes (2 units) further along the row
            mma_f8_pair(acc, ad + 2 * k, bd + 2 * k, id, (kt > 0 || k > 0) ? 1u : 0u);
          tc_commit_pair(bar_empty(s), 0x3);
        }
        if (ok) tc_commit_pair(bar_acc_full(i & 1), 0x3);
      }
    }
  } else {
    const int quad = warp & 3;         // tensor-memory lanes 32 quad .. 32 quad + 31
    const int half = (warp - 2) >> 2;  // which of the quadrant's two warps
    const int ew = warp - 2;
    const uint32_t out_buf = sbase + kW8Out + ew * kW8StageOut;
    float* sw_s = reinterpret_cast<float*>(smem + kW8Vec) + ew * 256;  // [4 sub-tiles][32]
    float* bias_s = sw_s + 128;
    int stores = 0;
    bool ok = true;
    for (int i = 0; i < my_tiles && ok; ++i) {
      int m0, n0;
      tile_mn(i, m0, n0);
      const int mrow = m0 + kW8BM * static_cast<int>(rank) + quad * 32;
      const int m = mrow + lane;
      const float sa = m < p.M ? p.a_scale[m] : 0.0f;
      // this warp's accumulator columns: sub-tile t starts at col(t); output column n0 + ocol(t)
      auto col = [&](int t) { return kGated ? (t & 1) * 128 + (half * 2 + (t >> 1)) * 32 : half * 128 + t * 32; };
      __syncwarp();
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        // the weight row of this column
        const int oc = n0 + (kGated ? (col(t) & 127) : col(t)) + lane;
        const bool in = oc < p.N;
        const int row = kGated && (t & 1) ? p.N + oc : oc;
        sw_s[t * 32 + lane] = in ? p.w_scale[row] : 0.0f;
        bias_s[t * 32 + lane] = in && p.bias != nullptr ? __bfloat162float(p.bias[row]) : 0.0f;
      }
      __syncwarp();
      ok = mbar_wait(bar_acc_full(i & 1), (i >> 1) & 1, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t t_row = tmem + (i & 1) * kW8BN + (static_cast<uint32_t>(quad * 32) << 16);
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(lead(bar_acc_free(i & 1)));
      };
      auto finish = [&](const uint32_t (&acc)[32], int t, float (&z)[32]) {
        const float4* sv = reinterpret_cast<const float4*>(sw_s + t * 32);
        const float4* bv = reinterpret_cast<const float4*>(bias_s + t * 32);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float4 s4 = sv[q], b4 = bv[q];
          z[4 * q + 0] = fmaf(__uint_as_float(acc[4 * q + 0]) * sa, s4.x, b4.x);
          z[4 * q + 1] = fmaf(__uint_as_float(acc[4 * q + 1]) * sa, s4.y, b4.y);
          z[4 * q + 2] = fmaf(__uint_as_float(acc[4 * q + 2]) * sa, s4.z, b4.z);
          z[4 * q + 3] = fmaf(__uint_as_float(acc[4 * q + 3]) * sa, s4.w, b4.w);
        }
      };
      auto store_sub = [&](float (&y)[32], int n) {
        if (p.residual != nullptr && m < p.M) {
          if (p.out_f32) {
            const float* r = static_cast<const float*>(p.residual) + static_cast<size_t>(m) * p.ldr + n;
#pragma unroll
            for (int c = 0; c < 8; ++c)
              if (n + 4 * c < p.N) {
                const float4 v = *reinterpret_cast<const float4*>(r + 4 * c);
                y[4 * c] += v.x; y[4 * c + 1] += v.y; y[4 * c + 2] += v.z; y[4 * c + 3] += v.w;
              }
          } else {
            const __nv_bfloat16* r = static_cast<const __nv_bfloat16*>(p.residual) + static_cast<size_t>(m) * p.ldr + n;
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (n + 8 * c < p.N) {
                const uint4 v = *reinterpret_cast<const uint4*>(r + 8 * c);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  y[8 * c + 2 * j] += __uint_as_float(w[j] << 16);
                  y[8 * c + 2 * j + 1] += __uint_as_float(w[j] & 0xFFFF0000u);
                }
              }
          }
        }
        uint32_t buf;
        if (p.out_f32) {
          buf = out_buf;  // one 4 KB buffer, rows of 128 B, 128-byte swizzle
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
#pragma unroll
          for (int c = 0; c < 8; ++c)
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                             buf + lane * 128 + ((c ^ (lane & 7)) << 4)),
                         "f"(y[4 * c]), "f"(y[4 * c + 1]), "f"(y[4 * c + 2]), "f"(y[4 * c + 3])
                         : "memory");
        } else {
          buf = out_buf + (stores & 1) * 2048;  // two 2 KB buffers, rows of 64 B, 64-byte swizzle
          if (lane == 0) bulk_wait_read<1>();
          __syncwarp();
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * j], y[2 * j + 1]);
            pk[j] = *reinterpret_cast<const uint32_t*>(&b);
          }
#pragma unroll
          for (int c = 0; c < 4; ++c)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             buf + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)),
                         "r"(pk[4 * c]), "r"(pk[4 * c + 1]), "r"(pk[4 * c + 2]), "r"(pk[4 * c + 3])
                         : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&tm_y, buf, n, mrow);
          bulk_commit();
        }
        ++stores;
      };
      if constexpr (kGated) {
#pragma unroll 1
        for (int t = 0; t < 4; t += 2) {
          uint32_t ga[32], ua[32];
          tmem_ld32(t_row + col(t), ga);
          tmem_ld32(t_row + col(t + 1), ua);
          tmem_ld_wait();
          if (t == 2) release();
          const int n = n0 + col(t);
          if (n >= p.N || mrow >= p.M) continue;  // warp-uniform
          float y[32], u[32];
          finish(ga, t, y);
          finish(ua, t + 1, u);
#pragma unroll
          for (int q = 0; q < 32; ++q) y[q] = w8_act(y[q], p.act) * u[q];
          store_sub(y, n);
        }
      } else {
#pragma unroll 1
        for (int t = 0; t < 4; ++t) {
          uint32_t acc[32];
          tmem_ld32(t_row + col(t), acc);
          tmem_ld_wait();
          if (t == 3) release();
          const int n = n0 + col(t);
          if (n >= p.N || mrow >= p.M) continue;  // warp-uniform
          float y[32];
          finish(acc, t, y);
          if (p.act != kW8ActNone) {
#pragma unroll
            for (int q = 0; q < 32; ++q) y[q] = w8_act(y[q], p.act);
          }
          store_sub(y, n);
        }
      }
    }
    if (lane == 0) bulk_wait_all();
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

}  // namespace svdq
