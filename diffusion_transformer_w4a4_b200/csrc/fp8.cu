// FP8 (E4M3) linear layer with one binary32 scale for each block of 128:
//
//   s_x[m,j] = fl32(max(max|x[m, block j]|, 2^-100) / 448),  qx = E4M3(clamp(fl32(x fl32(1/s_x)))),
//   Y[m,n]   = bf16( sum_j s_x[m,j] s_w[n/128,j] sum_{k in block j} qx[m,k] qw[n,k] + b[n] ).
//
// The floor 2^-100 keeps s and 1/s normal numbers, so a block of zeros (or of subnormals) needs no branch.
// Two kernels per forward:
//   k_fp8_quantize: 16 lanes to a block of 128, the maximum by shuffles; bound by memory (2 + 1 bytes an element).
//   k_gemm_fp8: tcgen05.mma kind::f8f6f4 over one block of 128 inputs at a time into a tensor-memory accumulator
//     of its own; the scales differ from block to block, so eight warps fold each finished block into sums in
//     registers, acc += (s_x s_w) d, while the tensor cores work on the next blocks.  The weight scale is one
//     number for a warp's columns (a tile's column half lies inside one block of 128 rows of W) and the
//     activation scale one number for a thread's row, so a fold is one fused multiply-add an element.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>
#include <new>

#include "sm100.cuh"
#include "svdq_internal.h"

struct svdq_fp8_layer {
  int64_t N, K;
  int device;
  const float* bias;     // [N]
  const float* wscales;  // [NB, KB]
  const uint8_t* wcodes;  // [N, K]
  CUtensorMap map_w[3];  // boxes of 96, 128 and 64 rows
};

namespace svdq {
namespace {

constexpr int kBlk = 128;
constexpr float kFp8Max = 448.f;
constexpr float kAmaxMin = 0x1p-100f;
constexpr int kQuantThreads = 256;

struct F8Blob {
  size_t bias, wscales, wcodes, total;
};
F8Blob f8_blob_layout(int64_t N, int64_t K) {
  const int64_t nb = (N + kBlk - 1) / kBlk, kb = (K + kBlk - 1) / kBlk;
  F8Blob b{};
  b.bias = 0;
  b.wscales = align_up((size_t)N * 4, kAlign);
  b.wcodes = align_up(b.wscales + (size_t)(nb * kb) * 4, kAlign);
  b.total = align_up(b.wcodes + (size_t)N * K, kAlign);
  return b;
}
struct F8Ws {
  size_t codes, scales, status, total;
  int64_t ld;  // columns of the scales
};
F8Ws f8_ws_layout(int64_t M, int64_t K) {
  F8Ws w{};
  w.ld = (M + kBlk - 1) / kBlk * kBlk;
  w.codes = 0;
  w.scales = align_up((size_t)M * K, kAlign);
  w.status = align_up(w.scales + (size_t)((K + kBlk - 1) / kBlk) * w.ld * 4, kAlign);
  w.total = w.status + 16;
  return w;
}
bool f8_shape_ok(int64_t N, int64_t K) {
  return N >= 8 && N % 8 == 0 && N <= (1 << 24) && K >= 16 && K % 16 == 0 && K <= (1 << 20);
}

// ------------------------------------------------------------------ quantizer
// One block of 128 inputs of one token to 16 lanes.
__global__ void __launch_bounds__(kQuantThreads) k_fp8_quantize(const uint16_t* __restrict__ x, int64_t M, int K, int KB,
                                                              uint8_t* __restrict__ codes, float* __restrict__ scales,
                                                              int64_t ld, int* __restrict__ status) {
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;  // the GEMM that follows records errors here
  const int sub = threadIdx.x & 15;
  const int64_t blocks = M * KB;
  // whole warps take a round together (two blocks): the shuffles need every lane
  for (int64_t i0 = ((int64_t)blockIdx.x * kQuantThreads + (threadIdx.x & ~31)) >> 4; i0 < blocks;
       i0 += (int64_t)gridDim.x * kQuantThreads >> 4) {
    const int64_t i = i0 + ((threadIdx.x >> 4) & 1);
    const int64_t m = i / KB;
    const int j = (int)(i - m * KB);
    const int k = j * kBlk + 8 * sub;
    const bool on = i < blocks && k < K;
    const int64_t at = m * K + k;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (on && SVDQ_INB(status, 2 * at, 16, 2 * M * K)) u = __ldcs((const uint4*)(x + at));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    float v[8], mx = kAmaxMin;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(w[e] << 16);
      v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
      mx = fmaxf(mx, fmaxf(fabsf(v[2 * e]), fabsf(v[2 * e + 1])));  // a NaN stays out here and gives a NaN code
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float s = __fdiv_rn(mx, kFp8Max), inv = __fdiv_rn(1.f, s);
    if (on) {
      uint32_t q[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * h] * inv, v[4 * h + 1] * inv), __NV_SATFINITE,
                                                     __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * h + 2] * inv, v[4 * h + 3] * inv),
                                                     __NV_SATFINITE, __NV_E4M3);
        q[h] = lo | (hi << 16);
      }
      if (SVDQ_INB(status, at, 8, M * K)) *(uint2*)(codes + at) = make_uint2(q[0], q[1]);
      if (sub == 0 && SVDQ_INB(status, 4 * (j * ld + m), 4, 4 * (int64_t)KB * ld)) scales[j * ld + m] = s;
    }
  }
}

// ------------------------------------------------------------------ GEMM
// PAIR: two CTAs on a 256 x 192 tile (each 128 rows of X and 96 of W a stage, 128 x 192 of the sums).  One CTA
// alone on 128 x 192 would read 40 KiB for 384 clocks of products, 104 bytes a clock, which the L2 does not give to
// 148 SMs at once; a pair reads 28 KiB a CTA.
// A fold costs a warp about three times a tensor-memory latency whatever its width, so a tile's columns go to
// warpgroups of 64 columns each: 64 sums and 64 loaded columns a thread, three warps to each scheduler at 192.
template <int BN, bool PAIR>
struct Tile {
  static constexpr int kRowsB = PAIR ? BN / 2 : BN;  // rows of W in this CTA's stage
  static constexpr int kStageA = 128 * kBlk, kStageB = kRowsB * kBlk, kStage = kStageA + kStageB;
  static constexpr int kStages = BN == 192 ? 7 : (BN == 128 ? 6 : 8);
  static constexpr int kBufs = BN == 192 ? 2 : 4;  // tensor-memory accumulators in flight
  static constexpr uint32_t kCols = BN == 192 ? 512 : BN * kBufs;
  static constexpr int kTileM = PAIR ? 256 : 128;
  static constexpr int kFoldWarps = BN / 16;  // warps 0.. fold (a warpgroup for 64 columns)
  static constexpr int kLoadWarp = kFoldWarps, kMmaWarp = kFoldWarps + 1;
  static constexpr int kThreads = 32 * kFoldWarps + 128;
  static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + 512;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
};

struct F8Params {
  int M, N, KB, NB, m_tiles, num_tiles;
  const float* sx;  // [KB, ld]
  long long ld;
  const float* sw;  // [NB, KB]
  const float* bias;
  uint16_t* Y;
  int* status;
  unsigned long long limit;
};
struct F8Maps {
  CUtensorMap a, b;
};

template <int BN, bool PAIR>
__global__ void __launch_bounds__((Tile<BN, PAIR>::kThreads), 1) k_gemm_fp8(const __grid_constant__ F8Maps maps,
                                                             const __grid_constant__ F8Params p) {
  using T = Tile<BN, PAIR>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* stages = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);  // [kStages][A | B]
  uint64_t* full = (uint64_t*)(stages + T::kStages * T::kStage);
  uint64_t* empty = full + T::kStages;
  uint64_t* acc_full = empty + T::kStages;   // [kBufs]
  uint64_t* acc_empty = acc_full + T::kBufs;  // [kBufs]
  uint64_t* mma_done = acc_empty + T::kBufs;
  uint32_t* tmem_slot = (uint32_t*)(mma_done + 1);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  WaitCtl wc{abort_flag, p.status, p.limit};
  const uint32_t rank = PAIR ? cluster_ctarank() : 0;  // the CTA of rank 0 issues the pair's products
  const int tile0 = PAIR ? blockIdx.x >> 1 : blockIdx.x, tile_step = PAIR ? gridDim.x >> 1 : gridDim.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < T::kStages; ++s) {
      mbar_init(&full[s], PAIR && rank == 0 ? 2 : 1);  // rank 0 also waits for the other CTA's stage
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < T::kBufs; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], (PAIR ? 2 : 1) * T::kFoldWarps);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // The quantizer's codes and scales; and an earlier kernel that let this one start may still need tensor
  // memory on this SM, so the allocation comes behind it too.
  pdl_wait();
  if (warp == T::kMmaWarp) {
    if constexpr (PAIR) {
      tmem_alloc_pair(tmem_slot, T::kCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, T::kCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // both CTAs' barriers and tensor memory are there
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= T::kFoldWarps) {
    if (warp == T::kLoadWarp && lane == 0) {
      // ---------------------------------------------------------- TMA producer
      prefetch_tmap(&maps.a);
      prefetch_tmap(&maps.b);
      int it = 0;
      bool ok = true;
      for (int tile = tile0; tile < p.num_tiles && ok; tile += tile_step) {
        const int mt = tile % p.m_tiles, nt = tile / p.m_tiles;
        for (int j = 0; j < p.KB; ++j, ++it) {
          const int s = it % T::kStages;
          if (!timed_wait(&empty[s], ((it / T::kStages) & 1) ^ 1, wc)) {
            ok = false;
            break;
          }
          uint8_t* st = stages + s * T::kStage;
          mbar_arrive_expect_tx(&full[s], T::kStage);
          tma_load_2d(&maps.a, &full[s], st, j * kBlk, mt * T::kTileM + (int)rank * 128);
          tma_load_2d(&maps.b, &full[s], st + T::kStageA, j * kBlk, nt * BN + (int)rank * T::kRowsB);
        }
      }
      // No block leaves with copies in flight, whoever gave up on them.
      for (int j = (it > T::kStages ? it - T::kStages : 0); j < it; ++j)
        mbar_wait_drain(&full[j % T::kStages], (j / T::kStages) & 1, drain_limit(p.limit));
    } else if (PAIR && rank == 1 && warp == T::kMmaWarp) {
      // ---------------------------------------------------------- the pair's other CTA: pass on that a stage is loaded
      if (lane == 0) {
        int it = 0;
        bool ok = true;
        for (int tile = tile0; tile < p.num_tiles && ok; tile += tile_step)
          for (int j = 0; j < p.KB && ok; ++j, ++it) {
            const int s = it % T::kStages;
            ok = timed_wait(&full[s], (it / T::kStages) & 1, wc);
            if (ok) mbar_arrive_cluster(dsmem_addr(smem_u32(&full[s]), 0));
          }
      }
    } else if (warp == T::kMmaWarp) {
      // ---------------------------------------------------------- MMA issuer: one accumulator per block of 128
      // The whole warp walks the loop (its values then live in uniform registers, where the instruction wants
      // them) and one lane issues.
      constexpr uint64_t kDesc = sdesc_const(16, 1024, LAYOUT_SW128);
      constexpr uint32_t idesc = idesc_e4m3_f32(PAIR ? 256 : 128, BN);
      const uint32_t first = sdesc_addr(stages);
      int s = 0, b = 0;
      uint32_t s_par = 0, b_par = 1;
      bool ok = true;
      for (int tile = tile0; tile < p.num_tiles && ok; tile += tile_step) {
        for (int j = 0; j < p.KB; ++j) {
          ok = warp_timed_wait(&acc_empty[b], b_par, wc) && warp_timed_wait(&full[s], s_par, wc);
          if (!ok) break;
          tc_fence_after();
          const uint64_t da = kDesc + first + (uint32_t)(s * (T::kStage >> 4)), db = da + (T::kStageA >> 4);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kBlk / 32; ++kk) {  // K = 32 codes (bytes) per instruction
              if constexpr (PAIR)
                mma_f8f6f4_pair(tmem + b * BN, da + 2 * kk, db + 2 * kk, idesc, kk != 0 ? 1u : 0u);
              else
                mma_f8f6f4(tmem + b * BN, da + 2 * kk, db + 2 * kk, idesc, kk != 0 ? 1u : 0u);
            }
            if constexpr (PAIR) {
              umma_commit_both(&empty[s]);
              umma_commit_both(&acc_full[b]);
            } else {
              umma_commit(&empty[s]);
              umma_commit(&acc_full[b]);
            }
          }
          __syncwarp();
          if (++s == T::kStages) {
            s = 0;
            s_par ^= 1;
          }
          if (++b == T::kBufs) {
            b = 0;
            b_par ^= 1;
          }
        }
      }
      if (elect_one()) {
        if constexpr (PAIR)
          umma_commit_pair(mma_done);
        else
          umma_commit(mma_done);
        mbar_wait_drain(mma_done, 0, drain_limit(p.limit));
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ fold and epilogue
    const int q = warp & 3;   // tensor-memory lane quarter
    const int h = warp >> 2;  // columns 64 h.. of the tile: inside one block of 128 rows of W
    int it = 0;
    bool ok = true;
    for (int tile = tile0; tile < p.num_tiles && ok; tile += tile_step) {
      const int mt = tile % p.m_tiles, nt = tile / p.m_tiles;
      const int m = mt * T::kTileM + (int)rank * 128 + 32 * q + lane;
      const int n0 = nt * BN + 64 * h;
      const int nb = min(n0 / kBlk, p.NB - 1);  // columns past N are not stored
      const float* sw = p.sw + (long long)nb * p.KB;
      const bool row = m < p.ld;  // the second CTA's rows can lie past the scales' last column
      const float* sx = p.sx + m;
      uint64_t acc[32];  // pairs of columns; the sums start from the bias
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int n = n0 + 4 * i;
        float4 b4 = make_float4(0.f, 0.f, 0.f, 0.f);
        if (n < p.N && SVDQ_INB(p.status, 4ll * n, 16, 4ll * p.N)) b4 = __ldg((const float4*)(p.bias + n));
        acc[2 * i] = pack2(b4.x, b4.y);
        acc[2 * i + 1] = pack2(b4.z, b4.w);
      }
      // The scales of two blocks ahead: a load is used two folds after it is issued.
      [[maybe_unused]] const long long sx_extent = 4ll * p.KB * p.ld, sw_extent = 4ll * p.NB * p.KB;  // debug build
      float xs[2], ws[2];
      auto fetch = [&](int j, int u) {
        xs[u] = ws[u] = 0.f;
        if (row && j < p.KB && SVDQ_INB(p.status, 4 * (j * p.ld + m), 4, sx_extent) &&
            SVDQ_INB(p.status, 4 * ((long long)nb * p.KB + j), 4, sw_extent)) {
          xs[u] = sx[j * p.ld];
          ws[u] = __ldg(sw + j);
        }
      };
#pragma unroll
      for (int u = 0; u < 2; ++u) fetch(u, u);
      for (int j0 = 0; j0 < p.KB && ok; j0 += 2) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (j0 + u >= p.KB) break;
          const int b = it % T::kBufs;
          ok = warp_timed_wait(&acc_full[b], (it / T::kBufs) & 1, wc);
          if (!ok) break;
          ++it;
          tc_fence_after();
          const float s = xs[u] * ws[u];
          const uint64_t s2 = pack2(s, s);
          fetch(j0 + u + 2, u);
          const uint32_t taddr = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(b * BN + 64 * h);
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            uint32_t r[32];
            tmem_ld_32x32b_x32(taddr + c, r);
            tmem_ld_wait_regs(r);
            if (c == 32) {  // every column of this accumulator is in registers
              tc_fence_before();
              __syncwarp();
              if (lane == 0) {
                if (PAIR)
                  mbar_arrive_cluster(dsmem_addr(smem_u32(&acc_empty[b]), 0));
                else
                  mbar_arrive(&acc_empty[b]);
              }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[c / 2 + i] = fma2(pack2(r[2 * i], r[2 * i + 1]), s2, acc[c / 2 + i]);
          }
        }
      }
      if (!ok) break;
      if (m < p.M) {
        const bool wide = (p.N & 15) == 0 && ((uintptr_t)p.Y & 31) == 0;  // rows of whole 32-byte sectors
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int n = n0 + 16 * v;
          if (n >= p.N) break;
          uint32_t o[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 y0 = unpack2(acc[8 * v + 2 * e]), y1 = unpack2(acc[8 * v + 2 * e + 1]);
            __nv_bfloat162 h0 = __floats2bfloat162_rn(y0.x, y0.y), h1 = __floats2bfloat162_rn(y1.x, y1.y);
            o[2 * e] = *(uint32_t*)&h0;
            o[2 * e + 1] = *(uint32_t*)&h1;
          }
          const long long at = (long long)m * p.N + n;
          if (wide) {
            if (SVDQ_INB(p.status, 2 * at, 32, 2ll * p.M * p.N)) st_global_32b(p.Y + at, o);
          } else {
            if (SVDQ_INB(p.status, 2 * at, 16, 2ll * p.M * p.N))
              *(uint4*)(p.Y + at) = make_uint4(o[0], o[1], o[2], o[3]);
            if (n + 8 < p.N && SVDQ_INB(p.status, 2 * at + 16, 16, 2ll * p.M * p.N))
              *(uint4*)(p.Y + at + 8) = make_uint4(o[4], o[5], o[6], o[7]);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // neither CTA is needed by the other's products, loads or barriers any more
  if (warp == T::kMmaWarp) {
    tc_fence_after();
    if constexpr (PAIR)
      tmem_dealloc_pair(tmem, T::kCols);
    else
      tmem_dealloc(tmem, T::kCols);
  }
}

int launch_f8_quantize(const svdq_fp8_layer* L, const void* X, int64_t M, uint8_t* ws, cudaStream_t stream) {
  const F8Ws w = f8_ws_layout(M, L->K);
  const int KB = (int)((L->K + kBlk - 1) / kBlk);
  int64_t grid = (M * KB + kQuantThreads / 16 - 1) / (kQuantThreads / 16);
  const int64_t cap = 16 * (int64_t)device_sm_count(L->device);
  if (grid > cap) grid = cap;
  return launch_pdl(k_fp8_quantize, dim3((unsigned)grid), dim3(kQuantThreads), 0, stream, (const uint16_t*)X, M,
                    (int)L->K, KB, ws + w.codes, (float*)(ws + w.scales), w.ld, (int*)(ws + w.status)) == cudaSuccess
             ? SVDQ_OK
             : SVDQ_ERR_CUDA;
}

template <int BN, bool PAIR>
int launch_f8_tile(const svdq_fp8_layer* L, const F8Maps& maps, F8Params& p, cudaStream_t stream) {
  using T = Tile<BN, PAIR>;
  {  // the shared-memory attribute belongs to the kernel on each device: set it once per device
    static std::mutex mu;
    static bool attr_set[64] = {};
    if (L->device < 0 || L->device >= 64) return SVDQ_ERR_CUDA;
    std::lock_guard<std::mutex> lock(mu);
    if (!attr_set[L->device]) {
      if (cudaFuncSetAttribute(k_gemm_fp8<BN, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)T::kSmem) !=
          cudaSuccess)
        return SVDQ_ERR_CUDA;
      attr_set[L->device] = true;
    }
  }
  p.m_tiles = (p.M + T::kTileM - 1) / T::kTileM;
  p.num_tiles = p.m_tiles * ((p.N + BN - 1) / BN);
  const int slots = device_sm_count(L->device) / (PAIR ? 2 : 1);
  const int grid = (p.num_tiles < slots ? p.num_tiles : slots) * (PAIR ? 2 : 1);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(T::kThreads);
  cfg.dynamicSmemBytes = T::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_gemm_fp8<BN, PAIR>, maps, p) == cudaSuccess ? SVDQ_OK : SVDQ_ERR_CUDA;
}

int launch_f8_gemm(const svdq_fp8_layer* L, int64_t M, void* Y, uint8_t* ws, cudaStream_t stream) {
  const F8Ws w = f8_ws_layout(M, L->K);
  F8Maps maps;
  std::memset(&maps, 0, sizeof(maps));
  int st = encode_tmap_2d(&maps.a, CU_TENSOR_MAP_DATA_TYPE_UINT8, ws + w.codes, (uint64_t)L->K, (uint64_t)M,
                          (uint64_t)L->K, kBlk, 128, CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != SVDQ_OK) return st;
  F8Params p{};
  p.M = (int)M;
  p.N = (int)L->N;
  p.KB = (int)((L->K + kBlk - 1) / kBlk);
  p.NB = (int)((L->N + kBlk - 1) / kBlk);
  p.sx = (const float*)(ws + w.scales);
  p.ld = w.ld;
  p.sw = L->wscales;
  p.bias = L->bias;
  p.Y = (uint16_t*)Y;
  p.status = (int*)(ws + w.status);
  p.limit = wait_limit_cycles();
  // Rounds of tiles over the SMs times the time of a tile's block: pairs on 256 x 192 where they fill the SMs,
  // narrower tiles of one CTA where there are too few (a tile's fixed part counts as about 64 columns).
  const int64_t sms = device_sm_count(L->device);
  auto rounds = [&](int64_t tm, int64_t tn, int64_t slots) {
    return ((M + tm - 1) / tm * ((L->N + tn - 1) / tn) + slots - 1) / slots;
  };
  const int64_t cost[3] = {rounds(256, 192, sms / 2) * (192 + 64), rounds(128, 128, sms) * (128 + 64),
                           rounds(128, 64, sms) * (64 + 64)};
  const int best = cost[0] <= cost[1] && cost[0] <= cost[2] ? 0 : (cost[1] <= cost[2] ? 1 : 2);
  maps.b = L->map_w[best];
  return best == 0 ? launch_f8_tile<192, true>(L, maps, p, stream)
                   : best == 1 ? launch_f8_tile<128, false>(L, maps, p, stream)
                               : launch_f8_tile<64, false>(L, maps, p, stream);
}

}  // namespace
}  // namespace svdq

using namespace svdq;

extern "C" {

svdq_status svdq_fp8_prepare(const uint16_t* W, int64_t N, int64_t K, uint8_t* wcodes, float* wscales) {
  if (!W || !wcodes || !wscales || !f8_shape_ok(N, K)) return SVDQ_ERR_INVALID_ARG;
  const int64_t nb = (N + kBlk - 1) / kBlk, kb = (K + kBlk - 1) / kBlk;
  for (int64_t i = 0; i < nb; ++i) {
    const int64_t n1 = std::min(N, (i + 1) * kBlk);
    for (int64_t j = 0; j < kb; ++j) {
      const int64_t k1 = std::min(K, (j + 1) * kBlk);
      float amax = kAmaxMin;
      for (int64_t n = i * kBlk; n < n1; ++n)
        for (int64_t k = j * kBlk; k < k1; ++k) {
          const float v = host::bf16_to_f32(W[n * K + k]);
          if (!std::isfinite(v)) return SVDQ_ERR_NUMERIC;
          amax = std::max(amax, std::fabs(v));
        }
      const float s = amax / kFp8Max;  // binary32 division
      const float inv = 1.f / s;
      wscales[i * kb + j] = s;
      for (int64_t n = i * kBlk; n < n1; ++n)
        for (int64_t k = j * kBlk; k < k1; ++k) {
          const float prod = host::bf16_to_f32(W[n * K + k]) * inv;  // binary32 product
          wcodes[n * K + k] = host::f32_to_e4m3_sat(prod);
        }
    }
  }
  return SVDQ_OK;
}

svdq_status svdq_fp8_packed_size(int64_t N, int64_t K, size_t* bytes) {
  if (!bytes || !f8_shape_ok(N, K)) return SVDQ_ERR_INVALID_ARG;
  *bytes = f8_blob_layout(N, K).total;
  return SVDQ_OK;
}

svdq_status svdq_fp8_pack(int64_t N, int64_t K, const uint8_t* wcodes, const float* wscales, const uint16_t* bias,
                          void* blob_v, size_t blob_bytes) {
  if (!wcodes || !wscales || !blob_v || !f8_shape_ok(N, K)) return SVDQ_ERR_INVALID_ARG;
  const F8Blob b = f8_blob_layout(N, K);
  if (blob_bytes < b.total) return SVDQ_ERR_INVALID_ARG;
  const int64_t ns = ((N + kBlk - 1) / kBlk) * ((K + kBlk - 1) / kBlk);
  for (int64_t i = 0; i < ns; ++i)
    if (!(wscales[i] >= 0.f) || !std::isfinite(wscales[i])) return SVDQ_ERR_INVALID_ARG;
  for (int64_t i = 0; i < N * K; ++i)
    if ((wcodes[i] & 0x7F) == 0x7F) return SVDQ_ERR_INVALID_ARG;  // E4M3 NaN
  uint8_t* blob = (uint8_t*)blob_v;
  std::memset(blob, 0, b.total);
  float* bf = (float*)(blob + b.bias);
  for (int64_t n = 0; n < N; ++n) bf[n] = bias ? host::bf16_to_f32(bias[n]) : 0.f;
  std::memcpy(blob + b.wscales, wscales, (size_t)ns * 4);
  std::memcpy(blob + b.wcodes, wcodes, (size_t)N * K);
  return SVDQ_OK;
}

svdq_status svdq_fp8_layer_create(const void* dev_blob, size_t blob_bytes, int64_t N, int64_t K,
                                  svdq_fp8_layer** out) {
  if (!out) return SVDQ_ERR_INVALID_ARG;
  *out = nullptr;
  if (!dev_blob || !f8_shape_ok(N, K) || ((uintptr_t)dev_blob & 255)) return SVDQ_ERR_INVALID_ARG;
  const F8Blob b = f8_blob_layout(N, K);
  if (blob_bytes < b.total) return SVDQ_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return SVDQ_ERR_UNSUPPORTED_DEVICE;
  }
  svdq_status st = svdq_device_check(dev);
  if (st != SVDQ_OK) return st;
  st = (svdq_status)check_blob_pointer(dev_blob, dev);
  if (st != SVDQ_OK) return st;
  svdq_fp8_layer* L = new (std::nothrow) svdq_fp8_layer();
  if (!L) return SVDQ_ERR_OOM;
  const uint8_t* base = (const uint8_t*)dev_blob;
  L->N = N;
  L->K = K;
  L->device = dev;
  L->bias = (const float*)(base + b.bias);
  L->wscales = (const float*)(base + b.wscales);
  L->wcodes = base + b.wcodes;
  const uint32_t rows[3] = {96, 128, 64};
  for (int i = 0; i < 3; ++i) {
    if (encode_tmap_2d(&L->map_w[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, L->wcodes, (uint64_t)K, (uint64_t)N, (uint64_t)K,
                       kBlk, rows[i], CU_TENSOR_MAP_SWIZZLE_128B) != SVDQ_OK) {
      delete L;
      return SVDQ_ERR_CUDA;
    }
  }
  *out = L;
  return SVDQ_OK;
}

void svdq_fp8_layer_destroy(svdq_fp8_layer* layer) { delete layer; }

svdq_status svdq_fp8_workspace_size(const svdq_fp8_layer* L, int64_t M, size_t* bytes) {
  if (!L || !bytes || M < 0 || M > (1 << 30)) return SVDQ_ERR_INVALID_ARG;
  *bytes = f8_ws_layout(M, L->K).total;
  return SVDQ_OK;
}

static svdq_status f8_check(const svdq_fp8_layer* L, int64_t M, const void* ws, size_t ws_bytes) {
  if (!L || M < 0 || M > (1 << 30) || !ws || ((uintptr_t)ws & 255)) return SVDQ_ERR_INVALID_ARG;
  if (ws_bytes < f8_ws_layout(M, L->K).total) return SVDQ_ERR_INVALID_ARG;
  return SVDQ_OK;
}

svdq_status svdq_fp8_quantize_act(const svdq_fp8_layer* L, const void* X, int64_t M, void* ws, size_t ws_bytes,
                                  void* stream) {
  svdq_status st = f8_check(L, M, ws, ws_bytes);
  if (st != SVDQ_OK) return st;
  if (M == 0) return SVDQ_OK;
  if (!X || ((uintptr_t)X & 15)) return SVDQ_ERR_INVALID_ARG;
  st = (svdq_status)require_current_device(L->device);
  if (st != SVDQ_OK) return st;
  NvtxRange range("svdq/fp8_quantize");
  return (svdq_status)launch_f8_quantize(L, X, M, (uint8_t*)ws, (cudaStream_t)stream);
}

svdq_status svdq_fp8_gemm(const svdq_fp8_layer* L, int64_t M, void* Y, void* ws, size_t ws_bytes, void* stream) {
  svdq_status st = f8_check(L, M, ws, ws_bytes);
  if (st != SVDQ_OK) return st;
  if (M == 0) return SVDQ_OK;
  if (!Y || ((uintptr_t)Y & 15)) return SVDQ_ERR_INVALID_ARG;
  st = (svdq_status)require_current_device(L->device);
  if (st != SVDQ_OK) return st;
  NvtxRange range("svdq/fp8_gemm");
  return (svdq_status)launch_f8_gemm(L, M, Y, (uint8_t*)ws, (cudaStream_t)stream);
}

svdq_status svdq_fp8_forward(const svdq_fp8_layer* L, const void* X, int64_t M, void* Y, void* ws, size_t ws_bytes,
                             void* stream) {
  if (M > 0 && (!Y || ((uintptr_t)Y & 15))) return SVDQ_ERR_INVALID_ARG;  // before anything is enqueued
  svdq_status st = svdq_fp8_quantize_act(L, X, M, ws, ws_bytes, stream);
  if (st != SVDQ_OK) return st;
  return svdq_fp8_gemm(L, M, Y, ws, ws_bytes, stream);
}

svdq_status svdq_fp8_read_status(const svdq_fp8_layer* L, int64_t M, const void* ws, size_t ws_bytes,
                                 int* device_status) {
  svdq_status st = f8_check(L, M, ws, ws_bytes);
  if (st != SVDQ_OK) return st;
  if (!device_status) return SVDQ_ERR_INVALID_ARG;
  int v = 0;
  if (cudaMemcpy(&v, (const uint8_t*)ws + f8_ws_layout(M, L->K).status, 4, cudaMemcpyDeviceToHost) != cudaSuccess)
    return SVDQ_ERR_CUDA;
  *device_status = v;
  return SVDQ_OK;
}

}  // extern "C"
