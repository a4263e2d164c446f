// svdq.cu -- the C ABI of include/svdq.h: argument checks, tensor-map
// construction, launch configuration and the device status word.
// All kernels live in this one translation unit.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <utility>

#include "../../include/svdq.h"
#include "awq.cuh"
#include "awq_gemm.cuh"
#include "int4_gemm.cuh"
#include "mlp_fc1.cuh"
#include "pack.cuh"
#include "prep.cuh"
#include "quantize_act.cuh"
#include "rope.cuh"
#include "w4a4_gemm.cuh"
#include "w8a8_gemm.cuh"
#include "w8a8_quantize.cuh"

namespace {

using namespace svdq;

__device__ uint32_t g_svdq_status;

// Working space of svdq_quantize_act_noalloc: the partial down-projections of
// K splits 1 .. S-1, (S - 1) * M * r floats at most kXl1ScratchFloats (8 MiB).
// Nothing in it needs to start at zero (each call writes every element it
// reads); two such calls in flight at the same time race on it.
constexpr size_t kXl1ScratchFloats = size_t(1) << 21;
static __device__ __align__(256) float g_xl1_scratch[kXl1ScratchFloats];

constexpr int kMaxDevices = 64;

struct DeviceInfo {
  bool ready = false;
  int num_sms = 0;
  int gemm_pairs = 0;  // co-resident clusters of the CTA-pair NVFP4 GEMM
  int int4_pairs = 0;  // the same for the INT4 GEMM
  int mlp_pairs = 0;   // the same for the fused MLP's fc1
  int w8_pairs = 0;    // the same for the 8-bit GEMM
  int w8_clusters[3] = {};  // co-resident clusters of 2, 4, 8 of the streaming 8-bit kernel, an SM to each CTA
  int gemm_pair_mode = -1;  // -1: by shape; SVDQ_GEMM_PAIR=0/1 forces single-CTA / CTA-pair tiles
  uint32_t* status = nullptr;
  float* xl1_scratch = nullptr;  // device address of g_xl1_scratch
  bool pdl = true;  // programmatic dependent launch of the hot-path kernels (SVDQ_PDL=0: off)
};

std::mutex g_mu;
DeviceInfo g_dev[kMaxDevices];

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encode = nullptr;

// Launch a hot-path kernel. With programmatic dependent launch the grid may be
// scheduled while the previous grid in the stream is finishing: every such
// kernel runs grid_dep_wait before its first global access, so stream order
// holds, and only its launch and prologue overlap the previous grid's tail.
// cluster_x > 1 launches clusters of that many CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_kernel(const DeviceInfo* d, void (*kern)(KArgs...), dim3 grid, dim3 block,
                          size_t smem, cudaStream_t stream, int cluster_x, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (cluster_x > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster_x;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (d->pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// the ring quantizer's shared memory, for every variant
template <int kRow, bool kF32>
cudaError_t ring_attributes() {
  const auto f = w8a8_quantize_ring_kernel<kRow, kF32>;
  const cudaError_t e =
      cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kW8RingBytes - kW8RingOwn));
  return e != cudaSuccess ? e
                          : cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout,
                                                 cudaSharedmemCarveoutMaxShared);
}
cudaError_t w8a8_quantize_attributes() {
  for (const cudaError_t e : {ring_attributes<kW8Plain, true>(), ring_attributes<kW8Plain, false>(),
                              ring_attributes<kW8Norm, true>(), ring_attributes<kW8Norm, false>(),
                              ring_attributes<kW8ResidualNorm, true>(), ring_attributes<kW8ResidualNorm, false>()})
    if (e != cudaSuccess) return e;
  return cudaSuccess;
}

// Per-device set-up (status word address, SM count, kernel attributes), done
// once per device with that device current.
svdq_status device_setup(DeviceInfo** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SVDQ_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceInfo& d = g_dev[dev];
  if (!d.ready) {
    if (g_encode == nullptr) {
      cudaDriverEntryPointQueryResult q;
      void* fn = nullptr;
      if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) !=
              cudaSuccess ||
          q != cudaDriverEntryPointSuccess || fn == nullptr)
        return SVDQ_ERR_CUDA;
      g_encode = reinterpret_cast<EncodeTiledFn>(fn);
    }
    void* st = nullptr;
    if (cudaGetSymbolAddress(&st, g_svdq_status) != cudaSuccess) return SVDQ_ERR_CUDA;
    void* scratch = nullptr;  // this device's copy (the device is current here)
    if (cudaGetSymbolAddress(&scratch, g_xl1_scratch) != cudaSuccess) return SVDQ_ERR_CUDA;
    if (cudaDeviceGetAttribute(&d.num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return SVDQ_ERR_CUDA;
    const int max_smem = 232448;
    if (cudaFuncSetAttribute(quantize_act_kernel<0>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             max_smem) != cudaSuccess ||
        cudaFuncSetAttribute(quantize_act_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             max_smem) != cudaSuccess ||
        cudaFuncSetAttribute(w4a4_nvfp4_gemm_kernel<false>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(GmCfg<false>::kSmemBytes)) != cudaSuccess ||
        cudaFuncSetAttribute(w4a4_nvfp4_gemm_kernel<true>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(GmCfg<true>::kSmemBytes)) != cudaSuccess ||
        cudaFuncSetAttribute(w4a4_nvfp4_gemm_kernel<false, true>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(GmCfg<false, true>::kSmemBytes)) != cudaSuccess ||
        cudaFuncSetAttribute(w4a4_nvfp4_gemm_kernel<true, true>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(GmCfg<true, true>::kSmemBytes)) != cudaSuccess)
      return SVDQ_ERR_CUDA;
    if (cudaFuncSetAttribute(w4a4_int4_gemm_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kI4SmemBytes)) != cudaSuccess ||
        cudaFuncSetAttribute(w4a4_mlp_fc1_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kMlSmemBytes)) != cudaSuccess ||
        w8a8_quantize_attributes() != cudaSuccess ||
        cudaFuncSetAttribute(w8a8_gemm_kernel<false, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kW8SmemBytes)) != cudaSuccess ||
        cudaFuncSetAttribute(w8a8_gemm_kernel<false, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kW8SmemBytes)) != cudaSuccess ||
        cudaFuncSetAttribute(w8a8_gemm_kernel<true, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kW8SmemBytes)) != cudaSuccess ||
        cudaFuncSetAttribute(w8a8_gemm_kernel<true, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kW8SmemBytes)) != cudaSuccess ||
        cudaFuncSetAttribute(w8a8_stream_kernel<false, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem) !=
            cudaSuccess ||
        cudaFuncSetAttribute(w8a8_stream_kernel<false, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem) !=
            cudaSuccess ||
        cudaFuncSetAttribute(w8a8_stream_kernel<true, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem) !=
            cudaSuccess ||
        cudaFuncSetAttribute(w8a8_stream_kernel<true, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem) !=
            cudaSuccess)
      return SVDQ_ERR_CUDA;
    // all of the SM's unified L1/shared storage as shared memory, so that the
    // occupancy the host code plans for (e.g. two quantizer CTAs per SM) is real
    for (const void* f : {reinterpret_cast<const void*>(quantize_act_kernel<0>),
                          reinterpret_cast<const void*>(quantize_act_kernel<1>),
                          reinterpret_cast<const void*>(w4a4_nvfp4_gemm_kernel<false>),
                          reinterpret_cast<const void*>(w4a4_nvfp4_gemm_kernel<true>),
                          reinterpret_cast<const void*>(w4a4_nvfp4_gemm_kernel<false, true>),
                          reinterpret_cast<const void*>(w4a4_nvfp4_gemm_kernel<true, true>),
                          reinterpret_cast<const void*>(w4a4_int4_gemm_kernel<true>),
                          reinterpret_cast<const void*>(awq_gemm_kernel),
                          reinterpret_cast<const void*>(w4a4_mlp_fc1_kernel),
                          reinterpret_cast<const void*>(w8a8_gemm_kernel<false, false>),
                          reinterpret_cast<const void*>(w8a8_gemm_kernel<false, true>),
                          reinterpret_cast<const void*>(w8a8_gemm_kernel<true, false>),
                          reinterpret_cast<const void*>(w8a8_gemm_kernel<true, true>),
                          reinterpret_cast<const void*>(w8a8_stream_kernel<false, false>),
                          reinterpret_cast<const void*>(w8a8_stream_kernel<false, true>),
                          reinterpret_cast<const void*>(w8a8_stream_kernel<true, false>),
                          reinterpret_cast<const void*>(w8a8_stream_kernel<true, true>),
                          reinterpret_cast<const void*>(awq_gemv_kernel<1>),
                          reinterpret_cast<const void*>(awq_gemv_kernel<2>)})
      if (cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared) != cudaSuccess)
        return SVDQ_ERR_CUDA;
    if (cudaFuncSetAttribute(awq_gemm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             max_smem) != cudaSuccess ||
        cudaFuncSetAttribute(awq_gemv_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             max_smem) != cudaSuccess ||
        cudaFuncSetAttribute(awq_gemv_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             max_smem) != cudaSuccess)
      return SVDQ_ERR_CUDA;
    {
      // how many 2-CTA clusters of the pair GEMM can be resident at once (a
      // persistent grid larger than that would run its last clusters late)
      auto clusters_of = [&](auto kern, int threads, size_t smem, int size, int most) {
        cudaLaunchConfig_t q = {};
        q.gridDim = dim3(size * most, 1, 1);
        q.blockDim = dim3(threads, 1, 1);
        q.dynamicSmemBytes = smem;
        cudaLaunchAttribute a[1];
        a[0].id = cudaLaunchAttributeClusterDimension;
        a[0].val.clusterDim.x = size;
        a[0].val.clusterDim.y = 1;
        a[0].val.clusterDim.z = 1;
        q.attrs = a;
        q.numAttrs = 1;
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, kern, &q) != cudaSuccess || clusters <= 0) {
          (void)cudaGetLastError();
          clusters = most;
        }
        return clusters < most ? clusters : most;
      };
      auto pairs = [&](auto kern, int threads, size_t smem) {
        return clusters_of(kern, threads, smem, 2, d.num_sms / 2);
      };
      d.gemm_pairs = pairs(w4a4_nvfp4_gemm_kernel<true>, kGmThreads, GmCfg<true>::kSmemBytes);
      d.int4_pairs = pairs(w4a4_int4_gemm_kernel<true>, kI4Threads, kI4SmemBytes);
      d.mlp_pairs = pairs(w4a4_mlp_fc1_kernel, kMlThreads, kMlSmemBytes);
      d.w8_pairs = pairs(w8a8_gemm_kernel<false, false>, kW8Threads, kW8SmemBytes);
      for (int i = 0; i < 3; ++i)
        d.w8_clusters[i] = clusters_of(w8a8_stream_kernel<false, true>, kWsThreads, kWsWholeSm, 2 << i, d.num_sms / (2 << i));
      if (std::getenv("SVDQ_DEBUG") != nullptr)
        std::fprintf(stderr, "svdq: %d SMs, %d / %d co-resident NVFP4 / INT4 GEMM CTA pairs\n",
                     d.num_sms, d.gemm_pairs, d.int4_pairs);
    }
    if (const char* e = std::getenv("SVDQ_GEMM_PAIR")) d.gemm_pair_mode = std::atoi(e) != 0;
    if (const char* e = std::getenv("SVDQ_PDL")) d.pdl = std::atoi(e) != 0;
    d.status = static_cast<uint32_t*>(st);
    d.xl1_scratch = static_cast<float*>(scratch);
    d.ready = true;
  }
  *out = &d;
  return SVDQ_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool debug_on() { return std::getenv("SVDQ_DEBUG") != nullptr; }

svdq_status launch_status() {
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess && debug_on()) std::fprintf(stderr, "svdq: launch failed: %s\n", cudaGetErrorString(e));
  return e == cudaSuccess ? SVDQ_OK : SVDQ_ERR_CUDA;
}

bool make_tmap_2d(CUtensorMap* m, CUtensorMapDataType dt, const void* ptr, uint64_t inner,
                  uint64_t outer, uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer,
                  CUtensorMapSwizzle swz) {
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {row_bytes};
  const cuuint32_t box[2] = {box_inner, box_outer};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = g_encode(m, dt, 2, const_cast<void*>(ptr), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS && debug_on())
    std::fprintf(stderr, "svdq: tensor map (dims %llu x %llu, box %u x %u) failed: %d\n",
                 static_cast<unsigned long long>(inner), static_cast<unsigned long long>(outer),
                 box_inner, box_outer, static_cast<int>(r));
  return r == CUDA_SUCCESS;
}

// A 3-D map over [outer][mid][inner] 8-byte elements, rows contiguous, for
// unswizzled boxes {inner, box_mid, box_outer} (the inner dimension whole).
bool make_tmap_3d_u64(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t mid, uint64_t outer,
                      uint32_t box_mid, uint32_t box_outer) {
  const cuuint64_t dims[3] = {inner, mid, outer};
  const cuuint64_t strides[2] = {inner * 8, inner * 8 * mid};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(inner), box_mid, box_outer};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT64, 3, const_cast<void*>(ptr), dims,
                              strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS && debug_on())
    std::fprintf(stderr, "svdq: 3-d tensor map (%llu x %llu x %llu) failed: %d\n",
                 static_cast<unsigned long long>(inner), static_cast<unsigned long long>(mid),
                 static_cast<unsigned long long>(outer), static_cast<int>(r));
  return r == CUDA_SUCCESS;
}

bool rank_ok(int r) { return r == 0 || (r % 16 == 0 && r >= 16 && r <= 256); }

size_t pad128(int rows) { return (static_cast<size_t>(rows) + 127) / 128 * 128; }

unsigned grid_for(size_t n, unsigned threads) {
  size_t b = (n + threads - 1) / threads;
  if (b < 1) b = 1;
  if (b > 65535u * 8u) b = 65535u * 8u;
  return static_cast<unsigned>(b);
}

// INT4 W4A4 GEMM (w4a4_int4_gemm_kernel): packed codes [rows, K/2] as one-group
// boxes [128 rows x 32 B], group-major FP16 scales [K/64][rows padded to 128]
// as one-group boxes [128], Y as 32 x 32 TMA-store boxes. Always CTA pairs, at
// any M: each CTA's converters fill 128 of a tile's 256 weight rows, so one CTA
// alone would leave half of the tile's B operand unfilled. Rows of a pair's tile
// past M read as zeros (TMA fill) and are clipped by the TMA store.
svdq_status launch_int4_gemm(const DeviceInfo* d, int M, int N, int K, int r, const void* a_codes,
                             const void* a_scales, const float* xl1, const void* w_codes,
                             const void* w_scales, const void* L2, const void* bias, void* Y,
                             int ldy, svdq_out out, cudaStream_t stream) {
  const int ctas = 2;
  CUtensorMap tm_a, tm_b, tm_sa, tm_sw, tm_l2, tm_y;
  const uint64_t G = static_cast<uint64_t>(K / 64);
  if (!make_tmap_2d(&tm_a, CU_TENSOR_MAP_DATA_TYPE_UINT8, a_codes, K / 2, M, K / 2, 32, kI4BM,
                    CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !make_tmap_2d(&tm_b, CU_TENSOR_MAP_DATA_TYPE_UINT8, w_codes, K / 2, N, K / 2, 32, kI4BM,
                    CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !make_tmap_2d(&tm_sa, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a_scales, pad128(M), G, pad128(M) * 2,
                    128, 1, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !make_tmap_2d(&tm_sw, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, w_scales, pad128(N), G, pad128(N) * 2,
                    128, 1, CU_TENSOR_MAP_SWIZZLE_NONE))
    return SVDQ_ERR_CUDA;
  if (r > 0) {
    if (!make_tmap_2d(&tm_l2, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, L2, N, r,
                      static_cast<uint64_t>(N) * 2, 64, kI4LrK, CU_TENSOR_MAP_SWIZZLE_128B))
      return SVDQ_ERR_CUDA;
  } else {
    tm_l2 = tm_a;
  }
  // output: 32 x 32 boxes, bf16 rows of 64 B (64-byte swizzle) or f32 rows of 128 B
  const bool f32 = out == SVDQ_OUT_F32;
  const int esz = f32 ? 4 : 2;
  if (!make_tmap_2d(&tm_y, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                    Y, N, M, static_cast<uint64_t>(ldy) * esz, 32, 32,
                    f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
    return SVDQ_ERR_CUDA;
  I4Params p;
  p.M = M;
  p.N = N;
  p.K = K;
  p.r = r;
  p.xl1 = xl1;
  p.bias = static_cast<const __nv_bfloat16*>(bias);
  p.out_f32 = f32;
  p.status = d->status;
  p.tiles_m = (M + kI4BM * ctas - 1) / (kI4BM * ctas);
  p.tiles = p.tiles_m * ((N + kI4BN - 1) / kI4BN);
  const int units = p.tiles < d->int4_pairs ? p.tiles : d->int4_pairs;
  const cudaError_t e = launch_kernel(d, w4a4_int4_gemm_kernel<true>, dim3(units * 2), dim3(kI4Threads),
                                      kI4SmemBytes, stream, 2, tm_a, tm_b, tm_sa, tm_sw, tm_l2, tm_y, p);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return SVDQ_ERR_CUDA;
  }
  return launch_status();
}

// AWQ W4A16 on the tensor cores (awq_gemm_kernel): token tiles of T = M rounded
// up to 16 (at most 128), 128 weight rows per tile, one persistent CTA per SM;
// weights and (s, z) in the fragment order of svdq_pack(AWQ).
svdq_status launch_awq_gemm(const DeviceInfo* d, int M, int N, int K, const void* X,
                            const void* qweight, const void* sz, const void* bias, void* Y,
                            cudaStream_t stream) {
  const int T = M >= kAgMaxT ? kAgMaxT : (M + 15) / 16 * 16;
  const int tb = T <= 32 ? 32 : (T <= 64 ? 64 : 128);
  int stages = kAgMaxStages;
  while (stages > 2 && ag_smem_bytes(T, stages) > 232448) --stages;
  const int G = K / 64, nblocks = (N + 15) / 16;
  CUtensorMap tm_q, tm_sz, tm_x;
  if (!make_tmap_3d_u64(&tm_q, qweight, 64, G, nblocks, 1, 8) ||
      !make_tmap_3d_u64(&tm_sz, sz, 8, G, nblocks, 1, 8) ||
      !make_tmap_2d(&tm_x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, X, K, M, static_cast<uint64_t>(K) * 2, 64,
                    T, CU_TENSOR_MAP_SWIZZLE_128B))
    return SVDQ_ERR_CUDA;
  AgParams p;
  p.M = M;
  p.N = N;
  p.K = K;
  p.T = T;
  p.tb = tb;
  p.nbuf = 512 / tb;
  p.stages = stages;
  p.tiles_m = (M + kAgMaxT - 1) / kAgMaxT;
  p.tiles = p.tiles_m * ((N + kAgRows - 1) / kAgRows);
  p.sz = static_cast<const uint32_t*>(sz);
  p.bias = static_cast<const __nv_bfloat16*>(bias);
  p.Y = static_cast<__nv_bfloat16*>(Y);
  p.status = d->status;
  const int grid = p.tiles < d->num_sms ? p.tiles : d->num_sms;
  if (debug_on())
    std::fprintf(stderr, "awq_w4a16_linear (tensor cores): M=%d N=%d K=%d T=%d stages=%d tiles=%d grid=%d\n",
                 M, N, K, T, stages, p.tiles, grid);
  if (launch_kernel(d, awq_gemm_kernel, dim3(grid), dim3(kAgThreads), ag_smem_bytes(T, stages), stream, 1,
                    tm_q, tm_sz, tm_x, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return SVDQ_ERR_CUDA;
  }
  return launch_status();
}

svdq_status quantize_act_impl(svdq_format format, int M, int K, int r, const void* X, int ldx,
                              const float* smooth_inv, const void* L1s, void* codes, void* scales,
                              float* xl1, bool static_rest, svdq_stream_t stream,
                              const float* tensor_scale = nullptr) {
  if (format != SVDQ_NVFP4_G16 && format != SVDQ_INT4_G64) return SVDQ_ERR_INVALID_ARG;
  if (tensor_scale != nullptr && format != SVDQ_NVFP4_G16) return SVDQ_ERR_INVALID_ARG;
  if (tensor_scale != nullptr && (reinterpret_cast<uintptr_t>(tensor_scale) & 7u))
    return SVDQ_ERR_ALIGNMENT;
  if (M < 1 || K < 64 || K % 64 || !rank_ok(r) || ldx < K) return SVDQ_ERR_INVALID_ARG;
  if (X == nullptr || codes == nullptr || scales == nullptr) return SVDQ_ERR_INVALID_ARG;
  if ((r > 0) != (L1s != nullptr) || (r > 0) != (xl1 != nullptr)) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(codes) || !aligned16(scales) || ldx % 8 ||
      (smooth_inv && !aligned16(smooth_inv)) || (L1s && !aligned16(L1s)) ||
      (xl1 && !aligned16(xl1)))
    return SVDQ_ERR_ALIGNMENT;
  DeviceInfo* d = nullptr;
  if (svdq_status st = device_setup(&d); st != SVDQ_OK) return st;

  CUtensorMap tm_x, tm_l1;
  if (!make_tmap_2d(&tm_x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, X, K, M, static_cast<uint64_t>(ldx) * 2,
                    64, 128, CU_TENSOR_MAP_SWIZZLE_128B))
    return SVDQ_ERR_CUDA;
  if (r > 0) {
    if (!make_tmap_2d(&tm_l1, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, L1s, K, 2 * r,
                      static_cast<uint64_t>(K) * 2, 64, r, CU_TENSOR_MAP_SWIZZLE_128B))
      return SVDQ_ERR_CUDA;
  } else {
    tm_l1 = tm_x;  // unused
  }

  const int row_blocks = (M + 127) / 128;
  // One CTA per SM (the kernel allocates tensor memory), K split into
  // qa_splits(M, K) ranges; ring stages of two 64-column sub-chunks where at
  // least two such stages fit, else of one.
  const int ksplit = qa_splits(M, K);
  const size_t budget = 227 * 1024;
  int spc = 0, stages = 0;
  for (int c = 2; c >= 1 && stages == 0; --c)
    for (int st = 8; st >= 2 && stages == 0; --st)
      if (qa_smem_bytes(r, st, c) <= budget) {
        spc = c;
        stages = st;
      }
  if (stages == 0) return SVDQ_ERR_UNSUPPORTED;
  const size_t smem_bytes = qa_smem_bytes(r, stages, spc);
  auto kern = format == SVDQ_NVFP4_G16 ? quantize_act_kernel<0> : quantize_act_kernel<1>;
  if (debug_on())
    std::fprintf(stderr,
                 "svdq_quantize_act: M=%d K=%d r=%d stages=%d x %d sub-chunks ksplit=%d grid=%d "
                 "smem=%zu\n",
                 M, K, r, stages, spc, ksplit, ksplit * row_blocks, smem_bytes);

  QuantActParams p;
  p.M = M;
  p.K = K;
  p.r = r;
  p.ksplit = ksplit;
  p.stages = stages;
  p.spc = spc;
  p.m_pad = static_cast<int>(pad128(M));
  p.smooth_inv = smooth_inv;
  p.tensor_scale = tensor_scale;
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = static_cast<uint8_t*>(scales);
  // splits 1 .. S-1: the rest of the caller's buffer, or the library's static
  // working space (svdq_quantize_act_noalloc)
  const size_t rest_floats = static_cast<size_t>(ksplit - 1) * M * r;
  if (static_rest && r > 0 && rest_floats > kXl1ScratchFloats) {
    if (debug_on())
      std::fprintf(stderr,
                   "svdq_quantize_act_noalloc: needs %zu floats of working space, the static "
                   "array holds %zu\n",
                   rest_floats, kXl1ScratchFloats);
    return SVDQ_ERR_UNSUPPORTED;
  }
  p.xl1 = xl1;
  p.xl1_rest = r > 0 ? (static_rest ? d->xl1_scratch : xl1 + static_cast<size_t>(M) * r) : nullptr;
  p.status = d->status;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (launch_kernel(d, kern, dim3(ksplit, row_blocks, 1), dim3(kQaThreads), smem_bytes, cs, 1, tm_x,
                    tm_l1, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return SVDQ_ERR_CUDA;
  }
  if (r > 0 && ksplit > 1) {
    // xl1[0] += xl1[1] + ... + xl1[S-1], in order
    const size_t n4 = static_cast<size_t>(M) * r / 4;
    if (launch_kernel(d, xl1_reduce_kernel, dim3(grid_for(n4, 256)), dim3(256), 0, cs, 1,
                      reinterpret_cast<float4*>(xl1), reinterpret_cast<const float4*>(p.xl1_rest),
                      ksplit, n4) != cudaSuccess) {
      (void)cudaGetLastError();
      return SVDQ_ERR_CUDA;
    }
  }
  return launch_status();
}

}  // namespace

extern "C" {

const char* svdq_status_str(svdq_status s) {
  switch (s) {
    case SVDQ_OK: return "ok";
    case SVDQ_ERR_INVALID_ARG: return "invalid argument";
    case SVDQ_ERR_ALIGNMENT: return "pointer or leading dimension not 16-byte aligned";
    case SVDQ_ERR_UNSUPPORTED: return "unsupported by this build";
    case SVDQ_ERR_CUDA: return "CUDA error";
    case SVDQ_ERR_TIMEOUT: return "a kernel's bounded wait ran out";
  }
  return "unknown status";
}

int svdq_version(void) { return 100; }

size_t svdq_codes_bytes(svdq_format f, int rows, int K) {
  if ((f != SVDQ_NVFP4_G16 && f != SVDQ_INT4_G64) || rows < 1 || K < 64 || K % 64) return 0;
  return static_cast<size_t>(rows) * (K / 2);
}

size_t svdq_scales_bytes(svdq_format f, int rows, int K) {
  if (rows < 1 || K < 64 || K % 64) return 0;
  if (f == SVDQ_NVFP4_G16) return pad128(rows) * (K / 16);
  if (f == SVDQ_INT4_G64) return pad128(rows) * (K / 64) * 2;
  return 0;
}

size_t awq_qweight_bytes(int N, int K) {
  if (N < 1 || K < 64 || K % 64) return 0;
  return (static_cast<size_t>(N) + 15) / 16 * 16 * (K / 2);
}

size_t awq_sz_bytes(int N, int K) {
  if (N < 1 || K < 64 || K % 64) return 0;
  return (static_cast<size_t>(N) + 15) / 16 * 16 * (K / 64) * 4;
}

int svdq_xl1_splits(int M, int K, int r) {
  if (M < 1 || K < 64 || K % 64 || !rank_ok(r)) return 0;
  return r == 0 ? 1 : qa_splits(M, K);
}

svdq_status svdq_quantize_act(svdq_format format, int M, int K, int r, const void* X, int ldx,
                              const float* smooth_inv, const void* L1s, void* codes,
                              void* scales, float* xl1, svdq_stream_t stream) {
  return quantize_act_impl(format, M, K, r, X, ldx, smooth_inv, L1s, codes, scales, xl1, false,
                           stream);
}

svdq_status svdq_quantize_act_noalloc(svdq_format format, int M, int K, int r, const void* X,
                                      int ldx, const float* smooth_inv, const void* L1s,
                                      void* codes, void* scales, float* xl1,
                                      svdq_stream_t stream) {
  return quantize_act_impl(format, M, K, r, X, ldx, smooth_inv, L1s, codes, scales, xl1, true,
                           stream);
}

}  // extern "C"

namespace {

// the fused QKV epilogue's arguments (svdq_w4a4_linear_qkv_norm_rope)
struct QkNormArgs {
  int q_heads;
  float eps;
  const void* norm_q;
  const void* norm_k;
  const float* rope_cos;
  const float* rope_sin;
};

svdq_status w4a4_linear_impl(svdq_format format, int M, int N, int K, int r, const void* a_codes,
                             const void* a_scales, const float* xl1, const void* w_codes,
                             const void* w_scales, const void* L2, const void* bias, void* Y,
                             int ldy, svdq_out out, svdq_stream_t stream, const float* a_tscale,
                             const float* w_tscale, const QkNormArgs* qk = nullptr) {
  if (format != SVDQ_NVFP4_G16 && format != SVDQ_INT4_G64) return SVDQ_ERR_INVALID_ARG;
  if ((a_tscale != nullptr) != (w_tscale != nullptr)) return SVDQ_ERR_INVALID_ARG;
  if (a_tscale != nullptr && format != SVDQ_NVFP4_G16) return SVDQ_ERR_INVALID_ARG;
  if (a_tscale != nullptr && ((reinterpret_cast<uintptr_t>(a_tscale) & 3u) ||
                              (reinterpret_cast<uintptr_t>(w_tscale) & 3u)))
    return SVDQ_ERR_ALIGNMENT;
  if (out != SVDQ_OUT_BF16 && out != SVDQ_OUT_F32) return SVDQ_ERR_INVALID_ARG;
  if (M < 1 || N < 16 || N % 16 || K < 64 || K % 64 || !rank_ok(r) || ldy < N)
    return SVDQ_ERR_INVALID_ARG;
  if (!a_codes || !a_scales || !w_codes || !w_scales || !Y) return SVDQ_ERR_INVALID_ARG;
  if ((r > 0) != (xl1 != nullptr) || (r > 0) != (L2 != nullptr)) return SVDQ_ERR_INVALID_ARG;
  const int esz = out == SVDQ_OUT_F32 ? 4 : 2;
  if (!aligned16(a_codes) || !aligned16(a_scales) || !aligned16(w_codes) || !aligned16(w_scales) ||
      !aligned16(Y) || (xl1 && !aligned16(xl1)) || (L2 && !aligned16(L2)) ||
      (bias && !aligned16(bias)) || (static_cast<size_t>(ldy) * esz) % 16)
    return SVDQ_ERR_ALIGNMENT;
  if (qk != nullptr && format != SVDQ_NVFP4_G16) return SVDQ_ERR_UNSUPPORTED;
  DeviceInfo* d = nullptr;
  if (svdq_status st = device_setup(&d); st != SVDQ_OK) return st;
  if (format == SVDQ_INT4_G64)
    return launch_int4_gemm(d, M, N, K, r, a_codes, a_scales, xl1, w_codes, w_scales, L2, bias, Y,
                            ldy, out, static_cast<cudaStream_t>(stream));

  // CTA pairs (cta_group::2, 256-row tiles): each CTA stages half of B, so a
  // pair moves a third less operand data per MMA than two single CTAs; measured
  // on B200 they are faster at every shape once the pair's cross-CTA arrivals
  // use CTA-scope release (QKV 70.3 vs 75.0 us, fc1 r=128 115.8 vs 122.1 us).
  const bool pair_auto = true;
  const bool pair = (d->gemm_pair_mode < 0 ? pair_auto : d->gemm_pair_mode != 0) && M > kGmBM;
  const int ctas = pair ? 2 : 1;
  const int b_rows = kGmBN / ctas;
  CUtensorMap tm_a, tm_b, tm_sfa, tm_sfb, tm_l2, tm_xl1, tm_y;
  const uint64_t kb = static_cast<uint64_t>(K / 64);
  if (!make_tmap_2d(&tm_a, CU_TENSOR_MAP_DATA_TYPE_UINT8, a_codes, K / 2, M, K / 2, kGmBKBytes,
                    kGmBM, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_2d(&tm_b, CU_TENSOR_MAP_DATA_TYPE_UINT8, w_codes, K / 2, N, K / 2, kGmBKBytes,
                    b_rows, CU_TENSOR_MAP_SWIZZLE_128B) ||
      // scale atoms as rows of 256 B (two rows per 512-byte atom), 8 rows = 4 atoms per box
      !make_tmap_2d(&tm_sfa, CU_TENSOR_MAP_DATA_TYPE_UINT8, a_scales, 256, pad128(M) / 128 * kb * 2,
                    256, 256, 8, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !make_tmap_2d(&tm_sfb, CU_TENSOR_MAP_DATA_TYPE_UINT8, w_scales, 256, pad128(N) / 128 * kb * 2,
                    256, 256, 8, CU_TENSOR_MAP_SWIZZLE_NONE))
    return SVDQ_ERR_CUDA;
  if (r > 0) {
    // xl1 [M, r] float32 in chunks of 32 columns x 128 rows, 128-byte swizzle
    if (!make_tmap_2d(&tm_l2, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, L2, N, r,
                      static_cast<uint64_t>(N) * 2, 64, kGmLrK, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_tmap_2d(&tm_xl1, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, xl1, r, M,
                      static_cast<uint64_t>(r) * 4, kGmLrK, kGmBM, CU_TENSOR_MAP_SWIZZLE_128B))
      return SVDQ_ERR_CUDA;
  } else {
    tm_l2 = tm_a;
    tm_xl1 = tm_a;
  }
  // output: 32 x 32 boxes, bf16 rows of 64 B (64-byte swizzle) or f32 rows of 128 B
  const bool f32 = out == SVDQ_OUT_F32;
  if (!make_tmap_2d(&tm_y, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                    Y, N, M, static_cast<uint64_t>(ldy) * esz, 32, 32,
                    f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
    return SVDQ_ERR_CUDA;
  GemmParams p;
  p.M = M;
  p.N = N;
  p.K = K;
  p.r = r;
  p.bias = static_cast<const __nv_bfloat16*>(bias);
  p.a_tscale = a_tscale;
  p.w_tscale = w_tscale;
  p.out_f32 = f32;
  p.status = d->status;
  p.q_heads = qk != nullptr ? qk->q_heads : 0;
  p.eps = qk != nullptr ? qk->eps : 0.0f;
  p.norm_q = qk != nullptr ? static_cast<const __nv_bfloat16*>(qk->norm_q) : nullptr;
  p.norm_k = qk != nullptr ? static_cast<const __nv_bfloat16*>(qk->norm_k) : nullptr;
  p.rope_cos = qk != nullptr ? qk->rope_cos : nullptr;
  p.rope_sin = qk != nullptr ? qk->rope_sin : nullptr;
  p.tiles_m = (M + kGmBM * ctas - 1) / (kGmBM * ctas);
  p.tiles = p.tiles_m * ((N + kGmBN - 1) / kGmBN);
  const int max_units = pair ? d->gemm_pairs : d->num_sms;
  const int units = p.tiles < max_units ? p.tiles : max_units;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (qk != nullptr)
    e = pair ? launch_kernel(d, w4a4_nvfp4_gemm_kernel<true, true>, dim3(units * 2), dim3(kGmThreads),
                             GmCfg<true, true>::kSmemBytes, cs, 2, tm_a, tm_b, tm_sfa, tm_sfb, tm_l2,
                             tm_xl1, tm_y, p)
             : launch_kernel(d, w4a4_nvfp4_gemm_kernel<false, true>, dim3(units), dim3(kGmThreads),
                             GmCfg<false, true>::kSmemBytes, cs, 1, tm_a, tm_b, tm_sfa, tm_sfb, tm_l2,
                             tm_xl1, tm_y, p);
  else
    e = pair ? launch_kernel(d, w4a4_nvfp4_gemm_kernel<true>, dim3(units * 2), dim3(kGmThreads),
                             GmCfg<true>::kSmemBytes, cs, 2, tm_a, tm_b, tm_sfa, tm_sfb, tm_l2, tm_xl1,
                             tm_y, p)
             : launch_kernel(d, w4a4_nvfp4_gemm_kernel<false>, dim3(units), dim3(kGmThreads),
                             GmCfg<false>::kSmemBytes, cs, 1, tm_a, tm_b, tm_sfa, tm_sfb, tm_l2, tm_xl1,
                             tm_y, p);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return SVDQ_ERR_CUDA;
  }
  return launch_status();
}

}  // namespace

extern "C" {

svdq_status svdq_w4a4_linear(svdq_format format, int M, int N, int K, int r, const void* a_codes,
                             const void* a_scales, const float* xl1, const void* w_codes,
                             const void* w_scales, const void* L2, const void* bias, void* Y,
                             int ldy, svdq_out out, svdq_stream_t stream) {
  return w4a4_linear_impl(format, M, N, K, r, a_codes, a_scales, xl1, w_codes, w_scales, L2, bias,
                          Y, ldy, out, stream, nullptr, nullptr);
}

svdq_status svdq_w4a4_linear_two_level(int M, int N, int K, int r, const void* a_codes,
                                       const void* a_scales, const float* a_tensor_scale,
                                       const float* xl1, const void* w_codes, const void* w_scales,
                                       const float* w_tensor_scale, const void* L2, const void* bias,
                                       void* Y, int ldy, svdq_out out, svdq_stream_t stream) {
  if (a_tensor_scale == nullptr || w_tensor_scale == nullptr) return SVDQ_ERR_INVALID_ARG;
  return w4a4_linear_impl(SVDQ_NVFP4_G16, M, N, K, r, a_codes, a_scales, xl1, w_codes, w_scales,
                          L2, bias, Y, ldy, out, stream, a_tensor_scale, w_tensor_scale);
}

svdq_status svdq_w4a4_linear_qkv_norm_rope(int M, int N, int K, int r, const void* a_codes,
                                           const void* a_scales, const float* xl1,
                                           const void* w_codes, const void* w_scales, const void* L2,
                                           const void* bias, const void* norm_q, const void* norm_k,
                                           float eps, const float* rope_cos, const float* rope_sin,
                                           void* Y, int ldy, svdq_out out, svdq_stream_t stream) {
  if (N < 384 || N % 384 || !(eps >= 0.0f) || eps > 3.0e38f) return SVDQ_ERR_INVALID_ARG;
  if ((rope_cos != nullptr) != (rope_sin != nullptr)) return SVDQ_ERR_INVALID_ARG;
  if ((rope_cos && (!aligned4(rope_cos) || !aligned4(rope_sin))) ||
      (reinterpret_cast<uintptr_t>(norm_q) & 1u) || (reinterpret_cast<uintptr_t>(norm_k) & 1u))
    return SVDQ_ERR_ALIGNMENT;
  const QkNormArgs qk{N / 384, eps, norm_q, norm_k, rope_cos, rope_sin};
  return w4a4_linear_impl(SVDQ_NVFP4_G16, M, N, K, r, a_codes, a_scales, xl1, w_codes, w_scales,
                          L2, bias, Y, ldy, out, stream, nullptr, nullptr, &qk);
}

int svdq_mlp_splits(int M, int N1) {
  if (M < 1 || N1 < kMlBN || N1 % kMlBN) return 0;
  DeviceInfo* d = nullptr;
  if (device_setup(&d) != SVDQ_OK) return 0;
  const int row_blocks = (M + 2 * kMlBM - 1) / (2 * kMlBM), ntn = N1 / kMlBN;
  int nsplit = d->mlp_pairs / row_blocks;
  if (nsplit < 1) nsplit = 1;
  if (nsplit > 8) nsplit = 8;
  if (nsplit > ntn) nsplit = ntn;
  const int tps = (ntn + nsplit - 1) / nsplit;
  return (ntn + tps - 1) / tps;
}

svdq_status svdq_mlp_fc1(int M, int N1, int K1, int r1, int r2, const void* a_codes, const void* a_scales,
                         const float* xl1_1, const void* w_codes, const void* w_scales, const void* L2_1,
                         const void* bias1, const float* smooth_inv2, const void* L1t_2, void* codes2,
                         void* scales2, float* xl1_2, float* hhat, svdq_stream_t stream) {
  if (M < 1 || N1 < kMlBN || N1 % kMlBN || K1 < 64 || K1 % 64 || !rank_ok(r1)) return SVDQ_ERR_INVALID_ARG;
  if (r2 < 0 || r2 > kMlR2Max || r2 % 32) return SVDQ_ERR_INVALID_ARG;
  if (!a_codes || !a_scales || !w_codes || !w_scales || !codes2 || !scales2) return SVDQ_ERR_INVALID_ARG;
  if ((r1 > 0) != (xl1_1 != nullptr) || (r1 > 0) != (L2_1 != nullptr)) return SVDQ_ERR_INVALID_ARG;
  if ((r2 > 0) != (L1t_2 != nullptr) || (r2 > 0) != (xl1_2 != nullptr)) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(a_codes) || !aligned16(a_scales) || !aligned16(w_codes) || !aligned16(w_scales) ||
      !aligned16(codes2) || !aligned16(scales2) || (xl1_1 && !aligned16(xl1_1)) || (L2_1 && !aligned16(L2_1)) ||
      (L1t_2 && !aligned16(L1t_2)) || (xl1_2 && !aligned16(xl1_2)) || (hhat && !aligned16(hhat)) ||
      (smooth_inv2 && (reinterpret_cast<uintptr_t>(smooth_inv2) & 3u)) ||
      (bias1 && (reinterpret_cast<uintptr_t>(bias1) & 1u)))
    return SVDQ_ERR_ALIGNMENT;
  DeviceInfo* d = nullptr;
  if (svdq_status st = device_setup(&d); st != SVDQ_OK) return st;
  const uint64_t kb = static_cast<uint64_t>(K1 / 64);
  CUtensorMap tm_a, tm_b, tm_sfa, tm_sfb, tm_l2, tm_xl1, tm_l1t;
  if (!make_tmap_2d(&tm_a, CU_TENSOR_MAP_DATA_TYPE_UINT8, a_codes, K1 / 2, M, K1 / 2, 128, kMlBM,
                    CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_2d(&tm_b, CU_TENSOR_MAP_DATA_TYPE_UINT8, w_codes, K1 / 2, N1, K1 / 2, 128, kMlBRows,
                    CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_2d(&tm_sfa, CU_TENSOR_MAP_DATA_TYPE_UINT8, a_scales, 256, pad128(M) / 128 * kb * 2, 256, 256,
                    8, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !make_tmap_2d(&tm_sfb, CU_TENSOR_MAP_DATA_TYPE_UINT8, w_scales, 256, pad128(N1) / 128 * kb * 2, 256,
                    256, 8, CU_TENSOR_MAP_SWIZZLE_NONE))
    return SVDQ_ERR_CUDA;
  if (r1 > 0) {
    if (!make_tmap_2d(&tm_l2, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, L2_1, N1, r1, static_cast<uint64_t>(N1) * 2,
                      64, kMlLrK, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_tmap_2d(&tm_xl1, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, xl1_1, r1, M, static_cast<uint64_t>(r1) * 4,
                      kMlLrK, kMlBM, CU_TENSOR_MAP_SWIZZLE_128B))
      return SVDQ_ERR_CUDA;
  } else {
    tm_l2 = tm_a;
    tm_xl1 = tm_a;
  }
  if (r2 > 0) {
    // L1_2^T [r2, N1] bf16: 64-column boxes of this CTA's r2 / 2 ranks
    if (!make_tmap_2d(&tm_l1t, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, L1t_2, N1, r2, static_cast<uint64_t>(N1) * 2,
                      64, r2 / 2, CU_TENSOR_MAP_SWIZZLE_128B))
      return SVDQ_ERR_CUDA;
  } else {
    tm_l1t = tm_a;
  }
  MlpParams p;
  p.M = M;
  p.N1 = N1;
  p.K1 = K1;
  p.r1 = r1;
  p.r2 = r2;
  p.row_blocks = (M + 2 * kMlBM - 1) / (2 * kMlBM);
  p.ntn = N1 / kMlBN;
  p.nsplit = svdq_mlp_splits(M, N1);
  p.tps = (p.ntn + p.nsplit - 1) / p.nsplit;
  p.units = p.row_blocks * p.nsplit;
  p.bias1 = static_cast<const __nv_bfloat16*>(bias1);
  p.smooth_inv2 = smooth_inv2;
  p.codes2 = static_cast<uint8_t*>(codes2);
  p.scales2 = static_cast<uint8_t*>(scales2);
  p.xl1_part = xl1_2;
  p.hhat = hhat;
  p.status = d->status;
  const int pairs = p.units < d->mlp_pairs ? p.units : d->mlp_pairs;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (debug_on())
    std::fprintf(stderr, "svdq_mlp_fc1: M=%d N1=%d K1=%d r1=%d r2=%d units=%d (splits %d, %d tiles each) pairs=%d\n",
                 M, N1, K1, r1, r2, p.units, p.nsplit, p.tps, pairs);
  if (launch_kernel(d, w4a4_mlp_fc1_kernel, dim3(2 * pairs), dim3(kMlThreads), kMlSmemBytes, cs, 2, tm_a, tm_b,
                    tm_sfa, tm_sfb, tm_l2, tm_xl1, tm_l1t, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return SVDQ_ERR_CUDA;
  }
  if (r2 > 0 && p.nsplit > 1) {
    // xl1_2[0] += xl1_2[1] + ... in order
    const size_t n4 = static_cast<size_t>(M) * r2 / 4;
    if (launch_kernel(d, xl1_reduce_kernel, dim3(grid_for(n4, 256)), dim3(256), 0, cs, 1,
                      reinterpret_cast<float4*>(xl1_2), reinterpret_cast<const float4*>(xl1_2 + static_cast<size_t>(M) * r2),
                      p.nsplit, n4) != cudaSuccess) {
      (void)cudaGetLastError();
      return SVDQ_ERR_CUDA;
    }
  }
  return launch_status();
}

svdq_status svdq_tensor_scale(int M, int K, const void* X, int ldx, const float* smooth_inv,
                              float* scale, svdq_stream_t stream) {
  if (M < 1 || K < 64 || K % 64 || ldx < K || ldx % 8 || !X || !scale) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(X) || (reinterpret_cast<uintptr_t>(scale) & 7u) ||
      (smooth_inv && !aligned16(smooth_inv)))
    return SVDQ_ERR_ALIGNMENT;
  DeviceInfo* d = nullptr;
  if (svdq_status st = device_setup(&d); st != SVDQ_OK) return st;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(scale, 0, sizeof(float), cs) != cudaSuccess) {
    (void)cudaGetLastError();
    return SVDQ_ERR_CUDA;
  }
  const size_t units = static_cast<size_t>(M) * (K / 8);
  unsigned grid = grid_for(units, 256);
  if (grid > static_cast<unsigned>(4 * d->num_sms)) grid = 4 * d->num_sms;
  if (launch_kernel(d, tensor_absmax_kernel, dim3(grid), dim3(256), 0, cs, 1,
                    static_cast<const __nv_bfloat16*>(X), ldx, smooth_inv, M, K,
                    reinterpret_cast<uint32_t*>(scale)) != cudaSuccess ||
      launch_kernel(d, tensor_scale_finalize_kernel, dim3(1), dim3(1), 0, cs, 1, scale) !=
          cudaSuccess) {
    (void)cudaGetLastError();
    return SVDQ_ERR_CUDA;
  }
  return launch_status();
}

svdq_status svdq_quantize_act_two_level(int M, int K, int r, const void* X, int ldx,
                                        const float* smooth_inv, const float* tensor_scale,
                                        const void* L1s, void* codes, void* scales, float* xl1,
                                        svdq_stream_t stream) {
  if (tensor_scale == nullptr) return SVDQ_ERR_INVALID_ARG;
  return quantize_act_impl(SVDQ_NVFP4_G16, M, K, r, X, ldx, smooth_inv, L1s, codes, scales, xl1,
                           false, stream, tensor_scale);
}

svdq_status awq_w4a16_linear(int M, int N, int K, int group, const void* X, const void* qweight,
                             const void* sz, const void* bias, void* Y, svdq_stream_t stream) {
  if (group != 64 || M < 1 || N < 1 || K < 64 || K % 64) return SVDQ_ERR_INVALID_ARG;
  if (!X || !qweight || !sz || !Y) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(qweight) || !aligned16(sz) || !aligned16(Y) ||
      (bias && (reinterpret_cast<uintptr_t>(bias) & 1)))
    return SVDQ_ERR_ALIGNMENT;
  DeviceInfo* d = nullptr;
  if (svdq_status st = device_setup(&d); st != SVDQ_OK) return st;
  // the path by M; SVDQ_AWQ_PATH=0 / 1 forces the GEMV / the tensor-core GEMM (read per call)
  const char* force = std::getenv("SVDQ_AWQ_PATH");
  const bool gemm = force != nullptr ? std::atoi(force) != 0 : M > kAwqMaxM;
  if (gemm) return launch_awq_gemm(d, M, N, K, X, qweight, sz, bias, Y, static_cast<cudaStream_t>(stream));
  if (M > kAwqMaxM) return SVDQ_ERR_UNSUPPORTED;  // the GEMV was forced
  // tokens per launch: at most 16 (two 8-token MMA blocks), and as many X rows
  // as fit in shared memory beside a weight ring of at least two stages
  const size_t smem_cap = 232448;
  auto fits = [&](int mc, int stages) {
    return awq_smem_bytes(mc, K, mc > 8 ? 2 : 1, stages) <= smem_cap;
  };
  int mc = M < 16 ? M : 16;
  while (mc > 1 && !fits(mc, 2)) --mc;
  if (!fits(mc, 2)) return SVDQ_ERR_UNSUPPORTED;
  const int nblocks = (N + 15) / 16;
  // one persistent CTA per SM, each streaming a contiguous run of 16-row blocks,
  // taken bpr at a time: the smallest power of two (<= 8) covering its blocks
  const int grid = nblocks < d->num_sms ? nblocks : d->num_sms;
  const int per_cta = (nblocks + grid - 1) / grid;
  int bpr = 1;
  while (bpr < per_cta && bpr < 8) bpr *= 2;
  // the stage boxes: weights [blocks][groups][64 x 8 B], (s, z) [blocks][groups][8 x 8 B]
  const int G = K / 64, wpb = kAwqConsumers / bpr, gsk = kAwqWarpGroups * wpb;
  CUtensorMap tm_q, tm_sz;
  if (!make_tmap_3d_u64(&tm_q, qweight, 64, G, nblocks, gsk, bpr) ||
      !make_tmap_3d_u64(&tm_sz, sz, 8, G, nblocks, gsk, bpr))
    return SVDQ_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  for (int m0 = 0; m0 < M; m0 += mc) {
    const int mm = M - m0 < mc ? M - m0 : mc;
    const int kmb = mm > 8 ? 2 : 1;
    int stages = kAwqMaxStages;
    while (stages > 2 && awq_smem_bytes(mm, K, kmb, stages) > smem_cap) --stages;
    AwqParams p;
    p.M = mm;
    p.N = N;
    p.K = K;
    p.stages = stages;
    p.bpr = bpr;
    p.X = static_cast<const __nv_bfloat16*>(X) + static_cast<size_t>(m0) * K;
    p.qweight = static_cast<const uint4*>(qweight);
    p.sz = static_cast<const uint32_t*>(sz);
    p.bias = static_cast<const __nv_bfloat16*>(bias);
    p.Y = static_cast<__nv_bfloat16*>(Y) + static_cast<size_t>(m0) * N;
    p.status = d->status;
    const size_t smem = awq_smem_bytes(mm, K, kmb, stages);
    const cudaError_t e =
        kmb == 1 ? launch_kernel(d, awq_gemv_kernel<1>, dim3(grid), dim3(kAwqThreads), smem, s, 1,
                                 tm_q, tm_sz, p)
                 : launch_kernel(d, awq_gemv_kernel<2>, dim3(grid), dim3(kAwqThreads), smem, s, 1,
                                 tm_q, tm_sz, p);
    if (e != cudaSuccess) {
      (void)cudaGetLastError();
      return SVDQ_ERR_CUDA;
    }
  }
  return launch_status();
}

svdq_status svdq_pack(svdq_pack_kind kind, svdq_format format, int rows, int K,
                      const void* plain_codes, const void* plain_scales, const void* plain_zeros,
                      void* tiled_codes, void* tiled_scales, svdq_stream_t stream) {
  if (rows < 1 || K < 64 || K % 64) return SVDQ_ERR_INVALID_ARG;
  if (!plain_codes || !plain_scales || !tiled_codes || !tiled_scales) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(plain_codes) || !aligned16(tiled_codes) || !aligned16(tiled_scales) ||
      (reinterpret_cast<uintptr_t>(plain_scales) & 1))
    return SVDQ_ERR_ALIGNMENT;
  if (kind != SVDQ_PACK_ACT && kind != SVDQ_PACK_WEIGHT && kind != SVDQ_PACK_AWQ)
    return SVDQ_ERR_INVALID_ARG;
  if (kind == SVDQ_PACK_AWQ) {
    if (plain_zeros == nullptr || (reinterpret_cast<uintptr_t>(plain_zeros) & 1)) return SVDQ_ERR_INVALID_ARG;
  } else if (plain_zeros != nullptr || (format != SVDQ_NVFP4_G16 && format != SVDQ_INT4_G64)) {
    return SVDQ_ERR_INVALID_ARG;
  }
  DeviceInfo* d = nullptr;
  if (svdq_status st = device_setup(&d); st != SVDQ_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned T = 256;
  if (kind == SVDQ_PACK_ACT || kind == SVDQ_PACK_WEIGHT) {
    if (plain_zeros != nullptr) return SVDQ_ERR_INVALID_ARG;
    if (format != SVDQ_NVFP4_G16 && format != SVDQ_INT4_G64) return SVDQ_ERR_INVALID_ARG;
    const size_t n16 = static_cast<size_t>(rows) * (K / 2) / 16;
    // the tiled codes of both formats are the plain bytes
    copy_bytes_kernel<<<grid_for(n16, T), T, 0, s>>>(static_cast<const uint4*>(plain_codes),
                                                     static_cast<uint4*>(tiled_codes), n16);
    if (format == SVDQ_NVFP4_G16) {
      const size_t n = pad128(rows) * (K / 16);
      pack_nvfp4_scales_kernel<<<grid_for(n, T), T, 0, s>>>(
          static_cast<const uint8_t*>(plain_scales), static_cast<uint8_t*>(tiled_scales), rows, K);
    } else {
      const size_t n = pad128(rows) * (K / 64);
      pack_int4_scales_kernel<<<grid_for(n, T), T, 0, s>>>(
          static_cast<const uint16_t*>(plain_scales), static_cast<uint16_t*>(tiled_scales), rows,
          K);
    }
    return launch_status();
  }
  if (kind == SVDQ_PACK_AWQ) {
    if (plain_zeros == nullptr || (reinterpret_cast<uintptr_t>(plain_zeros) & 1))
      return SVDQ_ERR_INVALID_ARG;
    const size_t nw = (static_cast<size_t>(rows) + 15) / 16 * (K / 64) * 128;
    pack_awq_qweight_kernel<<<grid_for(nw, T), T, 0, s>>>(
        static_cast<const uint8_t*>(plain_codes), static_cast<uint32_t*>(tiled_codes), rows, K);
    const size_t ns = (static_cast<size_t>(rows) + 15) / 16 * (K / 64) * 16;
    pack_awq_sz_kernel<<<grid_for(ns, T), T, 0, s>>>(
        static_cast<const uint16_t*>(plain_scales), static_cast<const uint16_t*>(plain_zeros),
        static_cast<uint32_t*>(tiled_scales), rows, K);
    return launch_status();
  }
  return SVDQ_ERR_INVALID_ARG;
}

svdq_status svdq_unpack(svdq_pack_kind kind, svdq_format format, int rows, int K,
                        const void* tiled_codes, const void* tiled_scales, void* plain_codes,
                        void* plain_scales, void* plain_zeros, svdq_stream_t stream) {
  if (rows < 1 || K < 64 || K % 64) return SVDQ_ERR_INVALID_ARG;
  if (!plain_codes || !plain_scales || !tiled_codes || !tiled_scales) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(plain_codes) || !aligned16(tiled_codes) || !aligned16(tiled_scales) ||
      (reinterpret_cast<uintptr_t>(plain_scales) & 1))
    return SVDQ_ERR_ALIGNMENT;
  if (kind != SVDQ_PACK_ACT && kind != SVDQ_PACK_WEIGHT && kind != SVDQ_PACK_AWQ)
    return SVDQ_ERR_INVALID_ARG;
  if (kind == SVDQ_PACK_AWQ) {
    if (plain_zeros == nullptr || (reinterpret_cast<uintptr_t>(plain_zeros) & 1)) return SVDQ_ERR_INVALID_ARG;
  } else if (plain_zeros != nullptr || (format != SVDQ_NVFP4_G16 && format != SVDQ_INT4_G64)) {
    return SVDQ_ERR_INVALID_ARG;
  }
  DeviceInfo* d = nullptr;
  if (svdq_status st = device_setup(&d); st != SVDQ_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned T = 256;
  if (kind == SVDQ_PACK_ACT || kind == SVDQ_PACK_WEIGHT) {
    if (plain_zeros != nullptr) return SVDQ_ERR_INVALID_ARG;
    if (format != SVDQ_NVFP4_G16 && format != SVDQ_INT4_G64) return SVDQ_ERR_INVALID_ARG;
    const size_t n16 = static_cast<size_t>(rows) * (K / 2) / 16;
    copy_bytes_kernel<<<grid_for(n16, T), T, 0, s>>>(static_cast<const uint4*>(tiled_codes),
                                                     static_cast<uint4*>(plain_codes), n16);
    if (format == SVDQ_NVFP4_G16) {
      const size_t n = static_cast<size_t>(rows) * (K / 16);
      unpack_nvfp4_scales_kernel<<<grid_for(n, T), T, 0, s>>>(
          static_cast<const uint8_t*>(tiled_scales), static_cast<uint8_t*>(plain_scales), rows, K);
    } else {
      const size_t n = static_cast<size_t>(rows) * (K / 64);
      unpack_int4_scales_kernel<<<grid_for(n, T), T, 0, s>>>(
          static_cast<const uint16_t*>(tiled_scales), static_cast<uint16_t*>(plain_scales), rows,
          K);
    }
    return launch_status();
  }
  if (kind == SVDQ_PACK_AWQ) {
    if (plain_zeros == nullptr || (reinterpret_cast<uintptr_t>(plain_zeros) & 1))
      return SVDQ_ERR_INVALID_ARG;
    const size_t nb = static_cast<size_t>(rows) * (K / 2);
    unpack_awq_qweight_kernel<<<grid_for(nb, T), T, 0, s>>>(
        static_cast<const uint32_t*>(tiled_codes), static_cast<uint8_t*>(plain_codes), rows, K);
    const size_t ns = static_cast<size_t>(rows) * (K / 64);
    unpack_awq_sz_kernel<<<grid_for(ns, T), T, 0, s>>>(
        static_cast<const uint32_t*>(tiled_scales), static_cast<uint16_t*>(plain_scales),
        static_cast<uint16_t*>(plain_zeros), rows, K);
    return launch_status();
  }
  return SVDQ_ERR_INVALID_ARG;
}

svdq_status svdq_pack_lowrank(int K, int r, const void* L1, const float* smooth_inv, void* L1s,
                              svdq_stream_t stream) {
  if (K < 64 || K % 64 || r < 16 || r > 256 || r % 16 || !L1 || !L1s) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(L1) || !aligned16(L1s) || (smooth_inv && !aligned16(smooth_inv)))
    return SVDQ_ERR_ALIGNMENT;
  DeviceInfo* d = nullptr;
  if (svdq_status st = device_setup(&d); st != SVDQ_OK) return st;
  const size_t n = static_cast<size_t>(K) * r;
  pack_lowrank_kernel<<<grid_for(n, 256), 256, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const __nv_bfloat16*>(L1), smooth_inv, static_cast<__nv_bfloat16*>(L1s), K, r);
  return launch_status();
}

svdq_status svdq_column_absmax(int rows, int K, const void* A, int lda, float* absmax,
                               svdq_stream_t stream) {
  if (rows < 1 || K < 8 || K % 8 || lda < K || lda % 8 || !A || !absmax) return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(A) || (reinterpret_cast<uintptr_t>(absmax) & 3u)) return SVDQ_ERR_ALIGNMENT;
  DeviceInfo* d = nullptr;
  if (svdq_status st = device_setup(&d); st != SVDQ_OK) return st;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(absmax, 0, static_cast<size_t>(K) * sizeof(float), cs) != cudaSuccess) {
    (void)cudaGetLastError();
    return SVDQ_ERR_CUDA;
  }
  // at least one thread per 8 columns; the rows are split among the rest
  const size_t units = static_cast<size_t>(K / 8);
  unsigned grid = grid_for(units * static_cast<size_t>(rows), 256);
  if (grid > static_cast<unsigned>(4 * d->num_sms)) grid = 4 * d->num_sms;
  const unsigned min_grid = static_cast<unsigned>((units + 255) / 256);
  if (grid < min_grid) grid = min_grid;
  column_absmax_kernel<<<grid, 256, 0, cs>>>(static_cast<const uint16_t*>(A), rows, K, lda,
                                             reinterpret_cast<uint32_t*>(absmax));
  return launch_status();
}

svdq_status svdq_smoothing(int N, int K, const float* x_absmax, const void* W, float* smooth_inv,
                           svdq_stream_t stream) {
  if (N < 1 || K < 8 || K % 8 || !x_absmax || !W || !smooth_inv) return SVDQ_ERR_INVALID_ARG;
  if (svdq_status st = svdq_column_absmax(N, K, W, K, smooth_inv, stream); st != SVDQ_OK) return st;
  smoothing_kernel<<<(K + 255) / 256, 256, 0, static_cast<cudaStream_t>(stream)>>>(x_absmax, smooth_inv, K);
  return launch_status();
}

svdq_status svdq_lowrank_factors(int N, int K, int r, const double* U, int ldu, const double* S,
                                 const double* Vh, int ldvh, void* L1, void* L2, svdq_stream_t stream) {
  if (N < 1 || K < 1 || r < 1 || r > N || r > K || ldu < r || ldvh < K) return SVDQ_ERR_INVALID_ARG;
  if (!U || !S || !Vh || !L1 || !L2) return SVDQ_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(U) & 7u) || (reinterpret_cast<uintptr_t>(S) & 7u) ||
      (reinterpret_cast<uintptr_t>(Vh) & 7u) || (reinterpret_cast<uintptr_t>(L1) & 1u) ||
      (reinterpret_cast<uintptr_t>(L2) & 1u))
    return SVDQ_ERR_ALIGNMENT;
  DeviceInfo* d = nullptr;
  if (svdq_status st = device_setup(&d); st != SVDQ_OK) return st;
  const size_t total = static_cast<size_t>(K) * r + static_cast<size_t>(r) * N;
  lowrank_factors_kernel<<<grid_for(total, 256), 256, 0, static_cast<cudaStream_t>(stream)>>>(
      U, ldu, S, Vh, ldvh, static_cast<uint16_t*>(L1), static_cast<uint16_t*>(L2), N, K, r);
  return launch_status();
}

svdq_status svdq_residual(int N, int K, int r, const void* W, const float* smooth_inv, const void* L1,
                          const void* L2, void* R, svdq_stream_t stream) {
  if (N < 1 || K < 1 || r < 0 || r > 4096 || !W || !smooth_inv || !R) return SVDQ_ERR_INVALID_ARG;
  if ((r > 0) != (L1 != nullptr) || (r > 0) != (L2 != nullptr)) return SVDQ_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(W) & 1u) || (reinterpret_cast<uintptr_t>(R) & 1u) ||
      (reinterpret_cast<uintptr_t>(smooth_inv) & 3u) || (reinterpret_cast<uintptr_t>(L1) & 1u) ||
      (reinterpret_cast<uintptr_t>(L2) & 1u))
    return SVDQ_ERR_ALIGNMENT;
  DeviceInfo* d = nullptr;
  if (svdq_status st = device_setup(&d); st != SVDQ_OK) return st;
  const dim3 grid((K + kResTile - 1) / kResTile, (N + kResTile - 1) / kResTile);
  residual_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint16_t*>(W), smooth_inv, static_cast<const uint16_t*>(L1),
      static_cast<const uint16_t*>(L2), static_cast<uint16_t*>(R), N, K, r);
  return launch_status();
}

svdq_status awq_quantize_weight(int N, int K, const void* W, void* qweight, void* sz,
                                svdq_stream_t stream) {
  if (N < 1 || K < 64 || K % 64 || !W || !qweight || !sz) return SVDQ_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(W) & 1u) || !aligned16(qweight) || !aligned16(sz))
    return SVDQ_ERR_ALIGNMENT;
  DeviceInfo* d = nullptr;
  if (svdq_status st = device_setup(&d); st != SVDQ_OK) return st;
  const size_t blocks = static_cast<size_t>((N + 15) / 16) * (K / 64);
  if (blocks > 0x7FFFFFFFull) return SVDQ_ERR_UNSUPPORTED;
  awq_quantize_kernel<<<static_cast<unsigned>(blocks), 128, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint16_t*>(W), N, K, static_cast<uint32_t*>(qweight), static_cast<uint32_t*>(sz));
  return launch_status();
}

}  // extern "C"

namespace {

// The 8-bit linear of at most kWvMaxM tokens and a small weight: a block per 16 weight rows.
svdq_status launch_w8a8_gemv(const DeviceInfo* d, bool gated, const W8Params& q, const void* a_codes,
                             const void* w_codes, void* Y, int ldy, svdq_stream_t stream) {
  WvParams p;
  p.M = q.M;
  p.N = q.N;
  p.K = q.K;
  p.a = static_cast<const uint8_t*>(a_codes);
  p.w = static_cast<const uint8_t*>(w_codes);
  p.act = q.act;
  p.out_f32 = q.out_f32;
  p.a_scale = q.a_scale;
  p.w_scale = q.w_scale;
  p.bias = q.bias;
  p.residual = q.residual;
  p.ldr = q.ldr;
  p.Y = Y;
  p.ldy = ldy;
  const int blocks = q.N / (gated ? 8 : 16);
  const int warps = q.K > 2048 ? 16 : 8;  // at most four 64-byte steps of K each
  auto kern = gated ? (q.M > 8 ? w8a8_gemv_kernel<true, 2> : w8a8_gemv_kernel<true, 1>)
                    : (q.M > 8 ? w8a8_gemv_kernel<false, 2> : w8a8_gemv_kernel<false, 1>);
  if (launch_kernel(d, kern, dim3(blocks), dim3(32 * warps), 0, static_cast<cudaStream_t>(stream), 1, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return SVDQ_ERR_CUDA;
  }
  return launch_status();
}

// How the streaming kernel takes a product: token tiles of T, and a cluster of `splits` CTAs
// (at most 8, at most half the K tiles) per tile of 128 weight rows.
struct StreamPlan {
  long long tiles;             // of weight rows
  int token_tiles, T, ktiles, splits;
};
// More clusters than can run with an SM to each CTA (33 of four, 15 of eight: they leave some SMs
// out): two CTAs to an SM. 64 x 5120 x 4736 in clusters of four, 37 of them: 16.8 us as two waves.
bool stream_shares(const DeviceInfo* d, const StreamPlan& s, int splits) {
  const int most = splits == 1 ? d->num_sms : d->w8_clusters[splits == 8 ? 2 : splits / 4];
  return s.tiles * s.token_tiles > most;
}
// One token tile, in ns: the sum over a cluster and its set-up against the stages of K that it
// saves, both growing with T; a stage's way in, longer in wider clusters, or all SMs' share of
// the memory; CTAs that share an SM end one after the other. Fitted to 222 shapes (up to 104 row
// tiles, K 512 to 15360, 4 to 128 tokens) timed with every count: the choice is 0.3 % slower than the
// fastest on average, 9 % at worst; on 61 shapes beyond them (106 to 148 row tiles, K 4096 to
// 15360) that it splits, 1.7 % slower than the faster of split and whole on average, 7 % at worst. 64
// tokens, (K, N): (1024, 5760) takes 5.0, 5.8, 6.5 us with 1, 2, 4; (3840, 3840) 10.3, 9.3, 8.4, 9.5 with
// 1, 2, 4, 8; (12288, 1024) 28.4, 18.1, 11.4, 8.9.
long long stream_cost(const DeviceInfo* d, const StreamPlan& s, int splits) {
  long long stage = 280;
  for (int i = splits; i > 1; i /= 2) stage += 40;
  const long long own = (s.ktiles + splits - 1) / splits * stage, all = s.tiles * s.ktiles * 16 / 10;
  long long cost = (own > all ? own : all) + (splits == 1 ? 2200 + 18ll * s.T : 4500 + 23ll * s.T);
  if (splits > 1 && stream_shares(d, s, splits)) cost += 350 + 45ll * s.T;
  return cost;
}
StreamPlan stream_plan(const DeviceInfo* d, bool gated, int M, int N, int K) {
  StreamPlan s;
  const int tile_n = gated ? 64 : 128;
  s.tiles = (static_cast<long long>(N) + tile_n - 1) / tile_n;
  s.token_tiles = (M + kWsMaxT - 1) / kWsMaxT;
  s.T = ((M + s.token_tiles - 1) / s.token_tiles + 15) / 16 * 16;
  s.ktiles = (K + kW8KStage - 1) / kW8KStage;
  s.splits = 1;
  if (s.token_tiles == 1) {
    for (int n = 2, i = 0; n <= 8 && 2 * n <= s.ktiles && s.tiles <= 2 * d->w8_clusters[i]; n *= 2, ++i)
      if (stream_cost(d, s, n) < stream_cost(d, s, s.splits)) s.splits = n;
  } else {  // where token tiles are chosen at all: the smallest that gives four in five SMs a CTA
    while (s.splits < 8 && 2 * s.splits <= s.ktiles && 5 * s.tiles * s.token_tiles * s.splits < 4ll * d->num_sms)
      s.splits *= 2;
  }
  return s;
}

svdq_status launch_w8a8_stream(const DeviceInfo* d, bool gated, const W8Params& q, const StreamPlan& plan,
                               const void* a_codes, const void* w_codes, void* Y, int ldy, svdq_stream_t stream) {
  WsParams p;
  p.M = q.M;
  p.N = q.N;
  p.K = q.K;
  p.T = plan.T;
  p.tb = p.T <= 32 ? 32 : (p.T <= 64 ? 64 : 128);
  const int splits = plan.splits, ktiles = plan.ktiles;
  if (plan.tiles > INT32_MAX / 8 || plan.token_tiles > 65535) return SVDQ_ERR_UNSUPPORTED;
  const int tiles = static_cast<int>(plan.tiles);
  p.splits = splits;
  p.shared = stream_shares(d, plan, splits);
  // two CTAs to an SM also for the widest clusters: few of eight whole SMs each find room at once
  const size_t budget = p.shared || splits == 8 ? kWsHalfSm : kWsWholeSm;
  const int per_cta = (ktiles + splits - 1) / splits;
  int stages = kWsMaxStages;
  while (stages > 2 && (ws_smem_bytes(p.T, stages) > budget || stages > per_cta)) --stages;
  p.stages = stages;
  p.act = q.act;
  p.out_f32 = q.out_f32;
  p.a_scale = q.a_scale;
  p.w_scale = q.w_scale;
  p.bias = q.bias;
  p.residual = q.residual;
  p.ldr = q.ldr;
  p.Y = Y;
  p.ldy = ldy;
  p.status = q.status;
  CUtensorMap tm_w, tm_x;
  if (!make_tmap_2d(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, w_codes, q.K, gated ? 2ull * q.N : q.N, q.K, kW8KStage, 64,
                    CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_2d(&tm_x, CU_TENSOR_MAP_DATA_TYPE_UINT8, a_codes, q.K, q.M, q.K, kW8KStage, p.T,
                    CU_TENSOR_MAP_SWIZZLE_128B))
    return SVDQ_ERR_CUDA;
  auto kern = gated ? (splits > 1 ? w8a8_stream_kernel<true, true> : w8a8_stream_kernel<true, false>)
                    : (splits > 1 ? w8a8_stream_kernel<false, true> : w8a8_stream_kernel<false, false>);
  if (launch_kernel(d, kern, dim3(tiles * splits, plan.token_tiles), dim3(kWsThreads), ws_smem_bytes(p.T, stages),
                    static_cast<cudaStream_t>(stream), splits, tm_w, tm_x, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return SVDQ_ERR_CUDA;
  }
  return launch_status();
}

// the 8-bit linear and its gated form (N: output columns; gated, the weight has 2 N rows)
svdq_status w8a8_linear_impl(bool gated, int M, int N, int K, const void* a_codes, const float* a_scale,
                             const void* w_codes, const float* w_scale, const void* bias, svdq_act act,
                             const void* residual, int ldr, void* Y, int ldy, svdq_out out,
                             svdq_stream_t stream) {
  if (act != SVDQ_ACT_NONE && act != SVDQ_ACT_GELU && act != SVDQ_ACT_SILU) return SVDQ_ERR_INVALID_ARG;
  if (out != SVDQ_OUT_BF16 && out != SVDQ_OUT_F32) return SVDQ_ERR_INVALID_ARG;
  if (M < 1 || N < 16 || N % 16 || K < 16 || K % 16 || ldy < N || (gated && N > INT32_MAX / 2))
    return SVDQ_ERR_INVALID_ARG;
  if (!a_codes || !a_scale || !w_codes || !w_scale || !Y || (residual && ldr < N)) return SVDQ_ERR_INVALID_ARG;
  if (M > (1 << 30) || N > (1 << 30) || K > (1 << 30)) return SVDQ_ERR_UNSUPPORTED;  // tile corners stay in an int
  const size_t esz = out == SVDQ_OUT_F32 ? 4 : 2;
  if (!aligned16(a_codes) || !aligned16(w_codes) || !aligned16(Y) || (ldy * esz) % 16 || !aligned4(a_scale) ||
      !aligned4(w_scale) || (bias && (reinterpret_cast<uintptr_t>(bias) & 1u)) ||
      (residual && (!aligned16(residual) || (ldr * esz) % 16)))
    return SVDQ_ERR_ALIGNMENT;
  DeviceInfo* d = nullptr;
  if (svdq_status st = device_setup(&d); st != SVDQ_OK) return st;
  W8Params p;
  p.M = M;
  p.N = N;
  p.K = K;
  p.act = act == SVDQ_ACT_GELU ? kW8ActGelu : (act == SVDQ_ACT_SILU ? kW8ActSilu : kW8ActNone);
  p.out_f32 = out == SVDQ_OUT_F32;
  p.a_scale = a_scale;
  p.w_scale = w_scale;
  p.bias = static_cast<const __nv_bfloat16*>(bias);
  p.residual = residual;
  p.ldr = ldr;
  p.Y = Y;
  p.ldy = ldy;
  p.status = d->status;
  // One to sixteen tokens of a small weight: no set-up (one token: K = N = 1024 2.5 us against 3.7
  // streamed, K = N = 3840 5.9 against 7.1; sixteen: K = N = 1024 2.9 against 4.0). Where a warp would go
  // round more than once, or the SMs get more than two blocks each, the copies of the streaming
  // kernel keep more bytes on their way (one token: K = 15360, N = 3840 15.8 against 13.6, K = 3840,
  // N = 15360 19.0 against 12.2; sixteen: K = N = 3840 10.9 against 7.4).
  if (M <= kWvMaxM && K <= (M <= 8 ? 4096 : 2048) && N / (gated ? 8 : 16) <= 2 * d->num_sms)
    return launch_w8a8_gemv(d, gated, p, a_codes, w_codes, Y, ldy, stream);
  // Few tokens stream the weight (64 tokens, streamed / in CTA pairs: K = N = 1024 4.8 / 4.7 us,
  // K = 1024, N = 15360 7.4 / 10.4). Above 64 only where the row tiles reach three in five SMs: the
  // epilogue of a tile grows with the tokens (128 tokens: K = N = 1024 6.1 / 4.6, K = 3840, N = 3840 9.7 / 9.0,
  // N = 10240 14.0 / 12.4, N = 12800 14.0 / 13.9, N = 15360 14.0 / 15.8; K = 1040, N = 15360 9.9 / 11.2), or
  // by what the split of a long K saves (below).
  const StreamPlan plan = stream_plan(d, gated, M, N, K);
  if (M <= 64 || (M <= kWsMaxT && 5 * plan.tiles >= 3ll * d->num_sms))
    return launch_w8a8_stream(d, gated, p, plan, a_codes, w_codes, Y, ldy, stream);
  // The tile's width: the one whose waves of tiles over the CTA pairs take least, a stage
  // of K costing its operands' way in, 256 + bn rows per pair (at 256 columns that equals its
  // MMA time). K = 3840: M = 256, N = 3840 takes 10.7 us at 64 columns and 18.4 at 256, M = 4608
  // 101 and 65; of 28 shapes measured at every width the choice was the fastest each time.
  const long long tiles_m = (static_cast<long long>(M) + 2 * kW8BM - 1) / (2 * kW8BM);
  long long best = -1;
  for (int bn = kW8MaxBN; bn >= 64; bn -= gated ? 64 : 32) {
    const int tile_n = gated ? bn / 2 : bn;
    const long long tiles = tiles_m * ((static_cast<long long>(N) + tile_n - 1) / tile_n);
    const long long waves = (tiles + d->w8_pairs - 1) / d->w8_pairs;
    const long long cost = waves * (bn + 256);
    if (tiles <= INT32_MAX / 2 && (best < 0 || cost < best)) {
      best = cost;
      p.bn = bn;
      p.tiles = static_cast<int>(tiles);
    }
  }
  if (best < 0) return SVDQ_ERR_UNSUPPORTED;
  // A long K over few tiles leaves most pairs idle, while clusters that split K reach every SM. Both
  // sides in clocks: the operands' way in, and, for the clusters, the sum over them and, past eight
  // of the widest, their waiting for whole groups of SMs. Set on 399 shapes timed both ways (65 to 1024
  // tokens, K 2048 to 15360, N 64 to 10240): 0.4 % slower than the faster one on average, 18 % at worst (72,
  // 2048, 272). (M, K, N), streamed / in pairs: (128, 5120, 3840) 10.2 / 10.6 and (128, 5120, 5120) 13.7 /
  // 11.7; (340, 4096, 512) 8.1 / 8.8, 1024 12.6 / 9.0; (768, 4096, 1024) 12.6 / 9.4; (768, 12512, 144) 11.1 / 19.5.
  const long long clusters = plan.tiles * plan.token_tiles;
  const long long split_cost = (plan.ktiles + plan.splits - 1) / plan.splits * (128ll + plan.T) * 3 + 4500 +
                               (plan.splits == 8 && clusters > 8 ? 5000 : 0);
  if (plan.splits > 1 && split_cost < best * plan.ktiles)
    return launch_w8a8_stream(d, gated, p, plan, a_codes, w_codes, Y, ldy, stream);
  p.tiles_m = static_cast<int>(tiles_m);
  // Row tiles in bands whose rows of A stay in a part of L2 while the weight passes by:
  // the weight is read once per band, A once. (M, K, N) = (4096, 15360, 3840), A 63 MB: two
  // bands 211 us, one 219; (4608, 3840, 2 x 10240), A 18 MB: one band 280 us, two 287.
  long long band = (40ll << 20) / (2ll * kW8BM * K);
  if (band < 1) band = 1;
  const long long bands = (tiles_m + band - 1) / band;
  p.band = static_cast<int>((tiles_m + bands - 1) / bands);
  p.band_tiles = p.band * (p.tiles / p.tiles_m);
  p.stages = static_cast<int>(kW8Ring / (kW8AStage + p.bn / 2 * kW8KStage));
  if (p.stages > kW8MaxStages) p.stages = kW8MaxStages;
  CUtensorMap tm_a, tm_b;
  if (!make_tmap_2d(&tm_a, CU_TENSOR_MAP_DATA_TYPE_UINT8, a_codes, K, M, K, kW8KStage, kW8BM,
                    CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_2d(&tm_b, CU_TENSOR_MAP_DATA_TYPE_UINT8, w_codes, K, gated ? 2ull * N : N, K, kW8KStage,
                    p.bn / 2, CU_TENSOR_MAP_SWIZZLE_128B))
    return SVDQ_ERR_CUDA;
  const int units = p.tiles < d->w8_pairs ? p.tiles : d->w8_pairs;
  const bool f32 = out == SVDQ_OUT_F32;
  auto kern = gated ? (f32 ? w8a8_gemm_kernel<true, true> : w8a8_gemm_kernel<true, false>)
                    : (f32 ? w8a8_gemm_kernel<false, true> : w8a8_gemm_kernel<false, false>);
  if (launch_kernel(d, kern, dim3(units * 2), dim3(kW8Threads), kW8SmemBytes, static_cast<cudaStream_t>(stream), 2,
                    tm_a, tm_b, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return SVDQ_ERR_CUDA;
  }
  return launch_status();
}

svdq_status w8a8_quantize_impl(bool norm, int M, int K, const void* X, int ldx, const void* residual, int ldr,
                               const void* weight, float eps, void* residual_out, int ldo, svdq_out dtype,
                               void* codes, float* scale, svdq_stream_t stream) {
  if (dtype != SVDQ_OUT_BF16 && dtype != SVDQ_OUT_F32) return SVDQ_ERR_INVALID_ARG;
  if (M < 1 || K < 16 || K % 16 || K > 32768 || ldx < K) return SVDQ_ERR_INVALID_ARG;
  if (!X || !codes || !scale || (residual != nullptr) != (residual_out != nullptr)) return SVDQ_ERR_INVALID_ARG;
  if (residual && (ldr < K || ldo < K)) return SVDQ_ERR_INVALID_ARG;
  if (norm && (!(eps >= 0.0f) || !std::isfinite(eps))) return SVDQ_ERR_INVALID_ARG;
  const int unit = dtype == SVDQ_OUT_F32 ? 4 : 8;  // elements of 16 bytes
  if (!aligned16(X) || ldx % unit || !aligned16(codes) || !aligned4(scale) || (weight && !aligned16(weight)) ||
      (residual && (!aligned16(residual) || !aligned16(residual_out) || ldr % unit || ldo % unit)))
    return SVDQ_ERR_ALIGNMENT;
  DeviceInfo* d = nullptr;
  if (svdq_status st = device_setup(&d); st != SVDQ_OK) return st;
  W8QuantParams p;
  p.K = K;
  p.X = X;
  p.ldx = ldx;
  p.residual = residual;
  p.ldr = ldr;
  p.residual_out = residual_out;
  p.ldo = ldo;
  p.weight = static_cast<const __nv_bfloat16*>(weight);
  p.eps = eps;
  p.inv_k = 1.0f / static_cast<float>(K);
  p.codes = static_cast<uint8_t*>(codes);
  p.scale = scale;
  const bool f32 = dtype == SVDQ_OUT_F32;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  // four 8-value vectors per thread
  const int nvec = K / 8, threads = (nvec + 127) / 128 * 32;
  // The ring, where every SM gets rows enough: as many blocks as keep two rows and the weight
  // in shared memory, up to 1024 threads an SM. 4608 rows of 3840: bf16 with residual 22.4 us
  // against 22.7 without the ring, float32 38.1 against 44.0; 4096 of 15360, codes alone, 30.3
  // against 35.0 (with more rows ahead 32.2). 9999 rows of 64 in place 6.4 against 11.2; but 20000 of 2048 in
  // place, bf16, 53.0 against 45.9.
  const size_t weight_bytes = weight ? static_cast<size_t>(K) * 4 : 0;
  const size_t row_bytes = static_cast<size_t>(K) * (f32 ? 4 : 2) * (residual ? 2 : 1);
  size_t blocks = kW8RingBytes / (kW8RingStages * row_bytes + weight_bytes + kW8RingOwn);
  if (blocks > 1024u / threads) blocks = 1024u / threads;
  cudaError_t e;
  if (blocks > 0 && static_cast<size_t>(M) >= 2 * d->num_sms * blocks) {
    W8RingParams q;
    q.M = M;
    q.status = d->status;
    auto kern = !norm      ? (f32 ? w8a8_quantize_ring_kernel<kW8Plain, true> : w8a8_quantize_ring_kernel<kW8Plain, false>)
                : residual ? (f32 ? w8a8_quantize_ring_kernel<kW8ResidualNorm, true>
                                  : w8a8_quantize_ring_kernel<kW8ResidualNorm, false>)
                           : (f32 ? w8a8_quantize_ring_kernel<kW8Norm, true> : w8a8_quantize_ring_kernel<kW8Norm, false>);
    e = launch_kernel(d, kern, dim3(static_cast<unsigned>(d->num_sms * blocks)), dim3(threads),
                      kW8RingStages * row_bytes + weight_bytes, cs, 1, p, q);
  } else {
    auto kern = !norm      ? (f32 ? w8a8_quantize_kernel<kW8Plain, true> : w8a8_quantize_kernel<kW8Plain, false>)
                : residual ? (f32 ? w8a8_quantize_kernel<kW8ResidualNorm, true> : w8a8_quantize_kernel<kW8ResidualNorm, false>)
                           : (f32 ? w8a8_quantize_kernel<kW8Norm, true> : w8a8_quantize_kernel<kW8Norm, false>);
    e = launch_kernel(d, kern, dim3(M), dim3(threads), 0, cs, 1, p);
  }
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return SVDQ_ERR_CUDA;
  }
  return launch_status();
}

// the arguments that the rotation and its tables share
svdq_status rope_params(RopeParams* p, int M, int axes, int pairs, const void* positions, int position_bytes,
                        const double* freq, const int* axis, float scale) {
  if (M < 1 || axes < 1 || pairs < 1 || pairs > kRopeMaxPairs || !positions || !freq) return SVDQ_ERR_INVALID_ARG;
  if ((position_bytes != 4 && position_bytes != 8) || !std::isfinite(scale)) return SVDQ_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(positions) & (position_bytes - 1)) || (reinterpret_cast<uintptr_t>(freq) & 7u) ||
      (axis && !aligned4(axis)))
    return SVDQ_ERR_ALIGNMENT;
  *p = RopeParams{};
  p->M = M;
  p->A = axes;
  p->P = pairs;
  p->positions = positions;
  p->pos64 = position_bytes == 8;
  p->freq = freq;
  p->axis = axis;
  p->scale = scale;
  return SVDQ_OK;
}

template <typename T, int V>
auto rope_kernel_of(bool interleaved) {
  if constexpr (V > 1) {
    if (interleaved) return rope_kernel<T, V, true>;
  }
  return rope_kernel<T, V, false>;
}

}  // namespace

extern "C" {

svdq_status w8a8_quantize_act(int M, int K, const void* X, int ldx, svdq_out dtype, void* codes, float* scale,
                              svdq_stream_t stream) {
  return w8a8_quantize_impl(false, M, K, X, ldx, nullptr, 0, nullptr, 0.0f, nullptr, 0, dtype, codes, scale, stream);
}

svdq_status w8a8_rmsnorm_quantize(int M, int K, const void* X, int ldx, const void* residual, int ldr,
                                  const void* weight, float eps, void* residual_out, int ldo, svdq_out dtype,
                                  void* codes, float* scale, svdq_stream_t stream) {
  return w8a8_quantize_impl(true, M, K, X, ldx, residual, ldr, weight, eps, residual_out, ldo, dtype, codes, scale,
                            stream);
}

svdq_status w8a8_linear(int M, int N, int K, const void* a_codes, const float* a_scale, const void* w_codes,
                        const float* w_scale, const void* bias, svdq_act act, const void* residual, int ldr,
                        void* Y, int ldy, svdq_out out, svdq_stream_t stream) {
  return w8a8_linear_impl(false, M, N, K, a_codes, a_scale, w_codes, w_scale, bias, act, residual, ldr, Y, ldy, out,
                          stream);
}

svdq_status w8a8_gated_linear(int M, int F, int K, const void* a_codes, const float* a_scale, const void* w_codes,
                              const float* w_scale, const void* bias, svdq_act act, void* Y, int ldy, svdq_out out,
                              svdq_stream_t stream) {
  return w8a8_linear_impl(true, M, F, K, a_codes, a_scale, w_codes, w_scale, bias, act, nullptr, 0, Y, ldy, out,
                          stream);
}

svdq_status svdq_rope(int M, int heads, int head_dim, int pairs, int axes, const void* positions, int position_bytes,
                      const double* freq, const int* axis, float scale, int interleaved, svdq_out dtype,
                      const void* X, int ldx, int ldhx, void* Y, int ldy, int ldhy, svdq_stream_t stream) {
  RopeParams p;
  if (svdq_status st = rope_params(&p, M, axes, pairs, positions, position_bytes, freq, axis, scale); st != SVDQ_OK)
    return st;
  if (dtype != SVDQ_OUT_BF16 && dtype != SVDQ_OUT_F32) return SVDQ_ERR_INVALID_ARG;
  if (heads < 1 || head_dim < 2 || head_dim % 2 || 2 * pairs > head_dim || !X || !Y) return SVDQ_ERR_INVALID_ARG;
  if (static_cast<long long>(heads) * head_dim > (1 << 30)) return SVDQ_ERR_UNSUPPORTED;
  if (ldx < 0 || ldhx < 0 || ldx % 2 || ldhx % 2 || ldy % 2 || ldhy % 2) return SVDQ_ERR_INVALID_ARG;
  // rows and heads of Y do not meet, in whichever order they lie
  const long long row_span = (heads - 1ll) * ldhy + head_dim, head_span = (M - 1ll) * ldy + head_dim;
  if (ldy < head_dim || ldhy < head_dim || (ldy < row_span && M > 1 && ldhy < head_span && heads > 1))
    return SVDQ_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(Y)) return SVDQ_ERR_ALIGNMENT;
  DeviceInfo* d = nullptr;
  if (svdq_status st = device_setup(&d); st != SVDQ_OK) return st;
  p.heads = heads;
  p.D = head_dim;
  p.X = X;
  p.ldx = ldx;
  p.ldhx = ldhx;
  p.Y = Y;
  p.ldy = ldy;
  p.ldhy = ldhy;
  // the widest vector (16 bytes at most) that every row, head and half starts on
  const int all = ldx | ldhx | ldy | ldhy | head_dim | (interleaved ? 0 : pairs);
  const bool f32 = dtype == SVDQ_OUT_F32;
  int V = f32 ? 4 : 8;
  while (all % V) V /= 2;
  auto kern = f32 ? (V == 4 ? rope_kernel_of<float, 4>(interleaved)
                            : (V == 2 ? rope_kernel_of<float, 2>(interleaved) : rope_kernel_of<float, 1>(interleaved)))
                  : (V == 8   ? rope_kernel_of<__nv_bfloat16, 8>(interleaved)
                     : V == 4 ? rope_kernel_of<__nv_bfloat16, 4>(interleaved)
                     : V == 2 ? rope_kernel_of<__nv_bfloat16, 2>(interleaved)
                              : rope_kernel_of<__nv_bfloat16, 1>(interleaved));
  // few rows: a row's heads are shared by blocks until the SMs are taken
  const int units = interleaved ? head_dim / V : pairs / V + (head_dim - 2 * pairs) / V;
  const int at_once = units < 256 ? 256 / units : 1;
  const long long per_row = (heads + at_once - 1) / at_once, wanted = (4ll * d->num_sms + M - 1) / M;
  const unsigned shares = static_cast<unsigned>(per_row < wanted ? per_row : wanted);
  if (launch_kernel(d, kern, dim3(M, shares), dim3(256), 0, static_cast<cudaStream_t>(stream), 1, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return SVDQ_ERR_CUDA;
  }
  return launch_status();
}

svdq_status svdq_rope_table(int M, int pairs, int axes, const void* positions, int position_bytes, const double* freq,
                            const int* axis, float scale, int angle_major, float* cos, float* sin,
                            svdq_stream_t stream) {
  RopeParams p;
  if (svdq_status st = rope_params(&p, M, axes, pairs, positions, position_bytes, freq, axis, scale); st != SVDQ_OK)
    return st;
  if (!cos || !sin) return SVDQ_ERR_INVALID_ARG;
  if (!aligned4(cos) || !aligned4(sin)) return SVDQ_ERR_ALIGNMENT;
  DeviceInfo* d = nullptr;
  if (svdq_status st = device_setup(&d); st != SVDQ_OK) return st;
  p.cos = cos;
  p.sin = sin;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (angle_major) {
    const int across = (pairs + kRopeTablePairs - 1) / kRopeTablePairs, wanted = (8 * d->num_sms + across - 1) / across;
    const int down = (M - 1) / 256 + 1;
    e = launch_kernel(d, rope_table_angle_major_kernel, dim3(down < wanted ? down : wanted, across), dim3(256), 0, cs, 1, p);
  } else {
    // four pairs per thread and 16-byte stores where rows keep that alignment
    const bool wide = pairs % 4 == 0 && aligned16(cos) && aligned16(sin);
    const int per_row = wide ? pairs / 4 : pairs, rows = per_row < 256 ? 256 / per_row : 1;
    int grid = (M - 1) / rows + 1;
    if (grid > 8 * d->num_sms) grid = 8 * d->num_sms;
    auto kern = position_bytes == 8 ? (wide ? rope_table_kernel<4, long long> : rope_table_kernel<1, long long>)
                                    : (wide ? rope_table_kernel<4, int> : rope_table_kernel<1, int>);
    e = launch_kernel(d, kern, dim3(grid), dim3(256), 0, cs, 1, p);
  }
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return SVDQ_ERR_CUDA;
  }
  return launch_status();
}

svdq_status svdq_check_device_status(svdq_stream_t stream) {
  DeviceInfo* d = nullptr;
  if (svdq_status st = device_setup(&d); st != SVDQ_OK) return st;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) {
    (void)cudaGetLastError();
    return SVDQ_ERR_CUDA;
  }
  uint32_t v = 0;
  if (cudaMemcpyFromSymbol(&v, g_svdq_status, sizeof(v)) != cudaSuccess) return SVDQ_ERR_CUDA;
  if (v != 0) {
    const uint32_t zero = 0;
    if (cudaMemcpyToSymbol(g_svdq_status, &zero, sizeof(zero)) != cudaSuccess)
      return SVDQ_ERR_CUDA;
  }
  return (v & kStatusTimeout) ? SVDQ_ERR_TIMEOUT : SVDQ_OK;
}

svdq_status svdq_debug_wait_timeout(int limit_us, svdq_stream_t stream) {
  if (limit_us < 1 || limit_us > 1000000) return SVDQ_ERR_INVALID_ARG;
  DeviceInfo* d = nullptr;
  if (svdq_status st = device_setup(&d); st != SVDQ_OK) return st;
  debug_wait_timeout_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(
      d->status, static_cast<uint64_t>(limit_us) * 1000ull);
  return launch_status();
}

}  // extern "C"
