// FP8 (E4M3) linear layer with one binary32 scale for each block of 128:
//
//   s_x[m,j] = fl32(max(max|x[m, block j]|, 2^-100) / 448),  qx = E4M3(clamp(fl32(x fl32(1/s_x)))),
//   Y[m,n]   = bf16( sum_j s_x[m,j] s_w[n/128,j] sum_{k in block j} qx[m,k] qw[n,k] + b[n] ).
//
// The floor 2^-100 keeps s and 1/s normal numbers, so a block of zeros (or of subnormals) needs no branch.
// Two kernels per forward:
//   k_fp8_quantize  16 lanes to a block of 128, the maximum by shuffles; bound by memory (2 + 1 bytes an element:
//                   4608 x 3072 8.8 us, 4.8 TB/s; 4608 x 12288 35 us, 4.9 TB/s).
//   the product     tcgen05.mma kind::f8f6f4 over one block of 128 inputs at a time into a tensor-memory accumulator of its
//                   own; the scales differ from block to block, so warps fold each finished block into sums in registers,
//                   acc += (s_x s_w) d, while the tensor cores work on the next.  The weight scale is one number for a
//                   warp's columns (they lie inside one block of 128 rows of W) and the activation scale one number for a
//                   thread's row, so a fold is one fused multiply-add an element.
//     k_gemm_fp8      tiles of 128 tokens by 256, 128 or 64 outputs, persistent; or, with fewer tiles than SMs and many
//                     inputs, a tile to a cluster whose CTAs split the inputs.  4608 x 3072 x 12288: 160 us
//                     (2.2 PFLOP/s); bound by the fold, which shares tensor memory with the products: a block takes about
//                     980 clocks against 512 of products (tensor pipe 52 % busy).  Loading 64 columns at a time is what
//                     made it fast (when that took 166 us: 32 at a time, the next under way meanwhile, 177; accumulators
//                     freed by halves 174).
//     k_gemm_fp8_few  up to 64 tokens: bound by the weight (2 x 3072 x 18432: 13.1 us with the quantizer, 4.3 TB/s).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>
#include <new>
#include <type_traits>

#include "sm100.cuh"
#include "svdq_internal.h"

struct svdq_fp8_layer {
  int64_t N, K;
  int device;
  const float* bias;     // [N]
  const float* wscales;  // [NB, KB]
  const uint8_t* wcodes;  // [N, K]
  const int* far;         // a scale above kFarScale is among them
  CUtensorMap map_w[3];  // boxes of 256, 128 and 64 rows
};

namespace svdq {
namespace {

constexpr int kBlk = 128;
constexpr float kFp8Max = 448.f;
constexpr float kAmaxMin = 0x1p-100f;
// Weight scales above this may take the product of the scales past binary32; below it none does, as s_x is at most the
// largest bf16 / 448 (or infinite, with a NaN among the codes).
constexpr float kFarScale = 448.f;
constexpr int kQuantThreads = 256;

// Scales of a row (of X, or of a block of 128 rows of W): one per block of 128 inputs, padded to whole 16 bytes.
int64_t f8_scale_ld(int64_t K) { return ((K + kBlk - 1) / kBlk + 3) / 4 * 4; }
struct F8Blob {
  size_t bias, wscales, wcodes, far, total;
};
F8Blob f8_blob_layout(int64_t N, int64_t K) {
  const int64_t nb = (N + kBlk - 1) / kBlk, kb = f8_scale_ld(K);
  F8Blob b{};
  b.bias = 0;
  b.wscales = align_up((size_t)N * 4, kAlign);
  b.wcodes = align_up(b.wscales + (size_t)(nb * kb) * 4, kAlign);
  b.far = align_up(b.wcodes + (size_t)N * K, kAlign);
  b.total = b.far + kAlign;
  return b;
}
struct F8Ws {
  size_t codes, scales, status, total;
};
F8Ws f8_ws_layout(int64_t M, int64_t K) {
  F8Ws w{};
  w.codes = 0;
  w.scales = align_up((size_t)M * K, kAlign);
  w.status = align_up(w.scales + (size_t)M * f8_scale_ld(K) * 4, kAlign);
  w.total = w.status + 16;
  return w;
}
bool f8_shape_ok(int64_t N, int64_t K) {
  return N >= 8 && N % 8 == 0 && N <= (1 << 24) && K >= 16 && K % 16 == 0 && K <= (1 << 20);
}

// ------------------------------------------------------------------ quantizer
// 16 lanes to a block of 128 inputs of one token, R blocks at a time, all asked for before the first is used: four where
// there are enough to fill the SMs (4608 x 12288: 35 us; one at a time 44), one where there are few (the latency of one block).
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2(*(const __nv_bfloat162*)&a, *(const __nv_bfloat162*)&b);
  return *(const uint32_t*)&m;
}
template <int R>
__global__ void __launch_bounds__(kQuantThreads) k_fp8_quantize(const uint16_t* __restrict__ x, int64_t M, int K, int KB,
                                                              uint8_t* __restrict__ codes, float* __restrict__ scales,
                                                              int ld, int* __restrict__ status) {
  pdl_wait();
  pdl_launch_dependents();  // the GEMM's CTAs may set up and ask for their weights
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;  // the GEMM that follows records errors here
  const int sub = threadIdx.x & 15, step = kQuantThreads / 16;
  const int64_t i = (int64_t)blockIdx.x * (R * step) + (threadIdx.x >> 4);
  int64_t m = M <= (1 << 17) ? (int64_t)((uint32_t)i / (uint32_t)KB) : i / KB;  // M KB < 2^31 there
  int j = (int)(i - m * KB);
  uint4 u[R];
  int64_t at[R], sc[R];
  bool on[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int k = j * kBlk + 8 * sub;
    on[r] = m < M && k < K;
    at[r] = m * K + k;
    sc[r] = m * ld + j;
    u[r] = make_uint4(0, 0, 0, 0);
    if (on[r] && SVDQ_INB(status, 2 * at[r], 16, 2 * M * K)) u[r] = __ldcs((const uint4*)(x + at[r]));
    j += step;
    while (j >= KB) {
      j -= KB;
      ++m;
    }
  }
  // The largest magnitude of each block, two elements at a time; a NaN stays out here and gives a NaN code.
  float mx = 0.f;  // of block r in the lanes sub = r (mod R)
#pragma unroll
  for (int r = 0; r < R; ++r) {
    uint32_t m = max_bf16x2(max_bf16x2(u[r].x & 0x7FFF7FFFu, u[r].y & 0x7FFF7FFFu),
                            max_bf16x2(u[r].z & 0x7FFF7FFFu, u[r].w & 0x7FFF7FFFu));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float f = fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    mx = (sub & (R - 1)) == r ? f : mx;
  }
  // One division for the R blocks, each in lanes of its own.
  const float s_mine = __fdiv_rn(fmaxf(mx, kAmaxMin), kFp8Max), inv_mine = __fdiv_rn(1.f, s_mine);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float s = __shfl_sync(0xffffffffu, s_mine, r, 16), inv = __shfl_sync(0xffffffffu, inv_mine, r, 16);
    if (on[r]) {
      const uint64_t inv2 = pack2(inv, inv);
      const uint32_t w[4] = {u[r].x, u[r].y, u[r].z, u[r].w};
      uint32_t q[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        q[e] = __nv_cvt_float2_to_fp8x2(unpack2(mul2(pack2(w[e] << 16, w[e] & 0xFFFF0000u), inv2)), __NV_SATFINITE,
                                        __NV_E4M3);
      if (SVDQ_INB(status, at[r], 8, M * K)) *(uint2*)(codes + at[r]) = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
      if (sub == 0 && SVDQ_INB(status, 4 * sc[r], 4, 4 * M * ld)) scales[sc[r]] = s;
    }
  }
}

// ------------------------------------------------------------------ GEMM
// A tile is 128 rows of X by BN of W; warps 0-7 fold (four to a half of the columns, which lies inside one block of 128
// rows of W), warp 8 loads, warp 9 issues the products (10 and 11 only round the warpgroup out).
template <int BN>
struct Tile {
  static constexpr int kStageA = 128 * kBlk, kStageB = BN * kBlk, kStage = kStageA + kStageB;
  static constexpr int kStages = BN == 256 ? 4 : (BN == 128 ? 6 : 8);
  static constexpr int kBufs = BN == 256 ? 2 : 4;  // tensor-memory accumulators in flight
  static constexpr uint32_t kCols = BN * kBufs;
  static constexpr int kFoldWarps = 8, kLoadWarp = 8, kMmaWarp = 9;
  static constexpr int kFoldCols = BN / 2;
  static constexpr int kOutCols = kFoldCols < 64 ? kFoldCols : 64;  // columns that go out together
  static constexpr int kOut = 32 * kOutCols * 2;                   // their bytes for the 32 rows of a warp
  static constexpr int kPartLd = BN + 4;                           // floats between the rows of partial sums
  static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + kFoldWarps * kOut + 512;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(128 * kPartLd * 4 <= kStages * kStage, "partial sums fit the stages");
};
constexpr int kGemmThreads = 384;
constexpr int kMaxSplit = 8;  // CTAs of a cluster
// Of a tile's outputs, four columns each, those that one CTA of a cluster joins: neighbours, in whole lines of 128 bytes
// (taken in turn instead, a warp's loads from the others' shared memory lie c times as far apart, and cost about that).
__device__ __forceinline__ int join_share(int units, int splits) { return ((units + splits - 1) / splits + 7) & ~7; }
// A block of 384 threads starts with 168 registers a thread.  At 256 columns a folding thread holds 128 sums and 64
// columns on their way, so the folding warps take 224 and leave the others 56: 128 * (2 * 224 + 56) = 384 * 168.
constexpr int kFoldRegs = 224, kOtherRegs = 56;
static_assert(128 * (2 * kFoldRegs + kOtherRegs) <= 384 * 168, "the split stays within the launch's registers");

struct F8Params {
  int M, N, KB, NB, m_tiles, num_tiles, splits, per;  // per: blocks of 128 inputs of a CTA
  const float* sx;  // [M, ld]
  const float* sw;  // [NB, ld]
  const int* far;
  int ld;
  const float* bias;
  uint16_t* Y;
  int* status;
  unsigned long long limit;
};
struct F8Maps {
  CUtensorMap a, b, y;  // y: 64 columns of 32 rows
};

// a += s * (32 or 64 columns of tensor memory from `t`) in one statement: the columns come with one latency, and the
// registers they pass through stay inside it.
__device__ __forceinline__ void fold32(uint32_t t, float s, float* a) {
  asm volatile(
      "{\n\t.reg .b32 t<32>;\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {t0,t1,t2,t3,t4,t5,t6,t7,t8,t9,t10,t11,t12,t13,t14,t15,"
      "t16,t17,t18,t19,t20,t21,t22,t23,t24,t25,t26,t27,t28,t29,t30,t31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n\t"
      "fma.rn.f32 %0, t0, %33, %0;\n\t"
      "fma.rn.f32 %1, t1, %33, %1;\n\t"
      "fma.rn.f32 %2, t2, %33, %2;\n\t"
      "fma.rn.f32 %3, t3, %33, %3;\n\t"
      "fma.rn.f32 %4, t4, %33, %4;\n\t"
      "fma.rn.f32 %5, t5, %33, %5;\n\t"
      "fma.rn.f32 %6, t6, %33, %6;\n\t"
      "fma.rn.f32 %7, t7, %33, %7;\n\t"
      "fma.rn.f32 %8, t8, %33, %8;\n\t"
      "fma.rn.f32 %9, t9, %33, %9;\n\t"
      "fma.rn.f32 %10, t10, %33, %10;\n\t"
      "fma.rn.f32 %11, t11, %33, %11;\n\t"
      "fma.rn.f32 %12, t12, %33, %12;\n\t"
      "fma.rn.f32 %13, t13, %33, %13;\n\t"
      "fma.rn.f32 %14, t14, %33, %14;\n\t"
      "fma.rn.f32 %15, t15, %33, %15;\n\t"
      "fma.rn.f32 %16, t16, %33, %16;\n\t"
      "fma.rn.f32 %17, t17, %33, %17;\n\t"
      "fma.rn.f32 %18, t18, %33, %18;\n\t"
      "fma.rn.f32 %19, t19, %33, %19;\n\t"
      "fma.rn.f32 %20, t20, %33, %20;\n\t"
      "fma.rn.f32 %21, t21, %33, %21;\n\t"
      "fma.rn.f32 %22, t22, %33, %22;\n\t"
      "fma.rn.f32 %23, t23, %33, %23;\n\t"
      "fma.rn.f32 %24, t24, %33, %24;\n\t"
      "fma.rn.f32 %25, t25, %33, %25;\n\t"
      "fma.rn.f32 %26, t26, %33, %26;\n\t"
      "fma.rn.f32 %27, t27, %33, %27;\n\t"
      "fma.rn.f32 %28, t28, %33, %28;\n\t"
      "fma.rn.f32 %29, t29, %33, %29;\n\t"
      "fma.rn.f32 %30, t30, %33, %30;\n\t"
      "fma.rn.f32 %31, t31, %33, %31;\n\t"
      "}"
      : "+f"(a[0]), "+f"(a[1]), "+f"(a[2]), "+f"(a[3]), "+f"(a[4]), "+f"(a[5]), "+f"(a[6]), "+f"(a[7]),
        "+f"(a[8]), "+f"(a[9]), "+f"(a[10]), "+f"(a[11]), "+f"(a[12]), "+f"(a[13]), "+f"(a[14]), "+f"(a[15]),
        "+f"(a[16]), "+f"(a[17]), "+f"(a[18]), "+f"(a[19]), "+f"(a[20]), "+f"(a[21]), "+f"(a[22]), "+f"(a[23]),
        "+f"(a[24]), "+f"(a[25]), "+f"(a[26]), "+f"(a[27]), "+f"(a[28]), "+f"(a[29]), "+f"(a[30]), "+f"(a[31])
      : "r"(t), "f"(s)
      : "memory");
}
__device__ __forceinline__ void fold64(uint32_t t, float s, float* a) {
  asm volatile(
      "{\n\t.reg .b32 t<64>;\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {t0,t1,t2,t3,t4,t5,t6,t7,t8,t9,t10,t11,t12,t13,t14,t15,"
      "t16,t17,t18,t19,t20,t21,t22,t23,t24,t25,t26,t27,t28,t29,t30,t31,"
      "t32,t33,t34,t35,t36,t37,t38,t39,t40,t41,t42,t43,t44,t45,t46,t47,"
      "t48,t49,t50,t51,t52,t53,t54,t55,t56,t57,t58,t59,t60,t61,t62,t63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n\t"
      "fma.rn.f32 %0, t0, %65, %0;\n\t"
      "fma.rn.f32 %1, t1, %65, %1;\n\t"
      "fma.rn.f32 %2, t2, %65, %2;\n\t"
      "fma.rn.f32 %3, t3, %65, %3;\n\t"
      "fma.rn.f32 %4, t4, %65, %4;\n\t"
      "fma.rn.f32 %5, t5, %65, %5;\n\t"
      "fma.rn.f32 %6, t6, %65, %6;\n\t"
      "fma.rn.f32 %7, t7, %65, %7;\n\t"
      "fma.rn.f32 %8, t8, %65, %8;\n\t"
      "fma.rn.f32 %9, t9, %65, %9;\n\t"
      "fma.rn.f32 %10, t10, %65, %10;\n\t"
      "fma.rn.f32 %11, t11, %65, %11;\n\t"
      "fma.rn.f32 %12, t12, %65, %12;\n\t"
      "fma.rn.f32 %13, t13, %65, %13;\n\t"
      "fma.rn.f32 %14, t14, %65, %14;\n\t"
      "fma.rn.f32 %15, t15, %65, %15;\n\t"
      "fma.rn.f32 %16, t16, %65, %16;\n\t"
      "fma.rn.f32 %17, t17, %65, %17;\n\t"
      "fma.rn.f32 %18, t18, %65, %18;\n\t"
      "fma.rn.f32 %19, t19, %65, %19;\n\t"
      "fma.rn.f32 %20, t20, %65, %20;\n\t"
      "fma.rn.f32 %21, t21, %65, %21;\n\t"
      "fma.rn.f32 %22, t22, %65, %22;\n\t"
      "fma.rn.f32 %23, t23, %65, %23;\n\t"
      "fma.rn.f32 %24, t24, %65, %24;\n\t"
      "fma.rn.f32 %25, t25, %65, %25;\n\t"
      "fma.rn.f32 %26, t26, %65, %26;\n\t"
      "fma.rn.f32 %27, t27, %65, %27;\n\t"
      "fma.rn.f32 %28, t28, %65, %28;\n\t"
      "fma.rn.f32 %29, t29, %65, %29;\n\t"
      "fma.rn.f32 %30, t30, %65, %30;\n\t"
      "fma.rn.f32 %31, t31, %65, %31;\n\t"
      "fma.rn.f32 %32, t32, %65, %32;\n\t"
      "fma.rn.f32 %33, t33, %65, %33;\n\t"
      "fma.rn.f32 %34, t34, %65, %34;\n\t"
      "fma.rn.f32 %35, t35, %65, %35;\n\t"
      "fma.rn.f32 %36, t36, %65, %36;\n\t"
      "fma.rn.f32 %37, t37, %65, %37;\n\t"
      "fma.rn.f32 %38, t38, %65, %38;\n\t"
      "fma.rn.f32 %39, t39, %65, %39;\n\t"
      "fma.rn.f32 %40, t40, %65, %40;\n\t"
      "fma.rn.f32 %41, t41, %65, %41;\n\t"
      "fma.rn.f32 %42, t42, %65, %42;\n\t"
      "fma.rn.f32 %43, t43, %65, %43;\n\t"
      "fma.rn.f32 %44, t44, %65, %44;\n\t"
      "fma.rn.f32 %45, t45, %65, %45;\n\t"
      "fma.rn.f32 %46, t46, %65, %46;\n\t"
      "fma.rn.f32 %47, t47, %65, %47;\n\t"
      "fma.rn.f32 %48, t48, %65, %48;\n\t"
      "fma.rn.f32 %49, t49, %65, %49;\n\t"
      "fma.rn.f32 %50, t50, %65, %50;\n\t"
      "fma.rn.f32 %51, t51, %65, %51;\n\t"
      "fma.rn.f32 %52, t52, %65, %52;\n\t"
      "fma.rn.f32 %53, t53, %65, %53;\n\t"
      "fma.rn.f32 %54, t54, %65, %54;\n\t"
      "fma.rn.f32 %55, t55, %65, %55;\n\t"
      "fma.rn.f32 %56, t56, %65, %56;\n\t"
      "fma.rn.f32 %57, t57, %65, %57;\n\t"
      "fma.rn.f32 %58, t58, %65, %58;\n\t"
      "fma.rn.f32 %59, t59, %65, %59;\n\t"
      "fma.rn.f32 %60, t60, %65, %60;\n\t"
      "fma.rn.f32 %61, t61, %65, %61;\n\t"
      "fma.rn.f32 %62, t62, %65, %62;\n\t"
      "fma.rn.f32 %63, t63, %65, %63;\n\t"
      "}"
      : "+f"(a[0]), "+f"(a[1]), "+f"(a[2]), "+f"(a[3]), "+f"(a[4]), "+f"(a[5]), "+f"(a[6]), "+f"(a[7]),
        "+f"(a[8]), "+f"(a[9]), "+f"(a[10]), "+f"(a[11]), "+f"(a[12]), "+f"(a[13]), "+f"(a[14]), "+f"(a[15]),
        "+f"(a[16]), "+f"(a[17]), "+f"(a[18]), "+f"(a[19]), "+f"(a[20]), "+f"(a[21]), "+f"(a[22]), "+f"(a[23]),
        "+f"(a[24]), "+f"(a[25]), "+f"(a[26]), "+f"(a[27]), "+f"(a[28]), "+f"(a[29]), "+f"(a[30]), "+f"(a[31]),
        "+f"(a[32]), "+f"(a[33]), "+f"(a[34]), "+f"(a[35]), "+f"(a[36]), "+f"(a[37]), "+f"(a[38]), "+f"(a[39]),
        "+f"(a[40]), "+f"(a[41]), "+f"(a[42]), "+f"(a[43]), "+f"(a[44]), "+f"(a[45]), "+f"(a[46]), "+f"(a[47]),
        "+f"(a[48]), "+f"(a[49]), "+f"(a[50]), "+f"(a[51]), "+f"(a[52]), "+f"(a[53]), "+f"(a[54]), "+f"(a[55]),
        "+f"(a[56]), "+f"(a[57]), "+f"(a[58]), "+f"(a[59]), "+f"(a[60]), "+f"(a[61]), "+f"(a[62]), "+f"(a[63])
      : "r"(t), "f"(s)
      : "memory");
}

// Where s_x s_w is past binary32 although the block's sum d may be small or 0: d is multiplied by the smaller scale in
// tensor memory first, and the fold takes the larger.  (Both are at least 1 there, or the input holds an infinity.)  Tiles
// have a loop of their own for layers that can come to this: the test in the common one, once for four blocks, cost
// 4608 x 3072 x 12288 5 us.
__device__ __forceinline__ bool past_f32(float s) { return !(s <= 3.402823466e38f); }
template <class Factor>  // factor(column)
__device__ __forceinline__ void scale_columns(uint32_t t, int cols, Factor&& factor) {
#pragma unroll 1
  for (int c = 0; c < cols; c += 16) {
    uint32_t d[16];
    tmem_ld_32x32b_x16(t + c, d);
    tmem_ld_wait_regs(d);
#pragma unroll
    for (int i = 0; i < 16; ++i) d[i] = __float_as_uint(__uint_as_float(d[i]) * factor(c + i));
    tmem_st_32x32b_x16(t + c, d);
  }
  tmem_st_wait();
}

template <int BN, bool SPLIT>
__global__ void __launch_bounds__(kGemmThreads, 1) k_gemm_fp8(const __grid_constant__ F8Maps maps,
                                                             const __grid_constant__ F8Params p) {
  using T = Tile<BN>;
  constexpr int FC = T::kFoldCols, OC = T::kOutCols;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* stages = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);  // [kStages][A | B]
  uint8_t* sm_out = stages + T::kStages * T::kStage;  // [kFoldWarps][kOut]
  uint64_t* full = (uint64_t*)(sm_out + T::kFoldWarps * T::kOut);
  uint64_t* empty = full + T::kStages;
  uint64_t* acc_full = empty + T::kStages;   // [kBufs]
  uint64_t* acc_empty = acc_full + T::kBufs;  // [kBufs]
  uint64_t* mma_done = acc_empty + T::kBufs;
  uint32_t* tmem_slot = (uint32_t*)(mma_done + 1);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  WaitCtl wc{abort_flag, p.status, p.limit};
  // SPLIT: a tile to a cluster, whose CTAs take `per` blocks of 128 inputs each (a multiple of 4).
  const int rank = SPLIT ? (int)cluster_ctarank() : 0;
  const int tile0 = SPLIT ? (int)blockIdx.x / p.splits : (int)blockIdx.x, step = SPLIT ? p.num_tiles : (int)gridDim.x;
  const int j_first = SPLIT ? rank * p.per : 0, KB = SPLIT ? min(p.per, p.KB - j_first) : p.KB;
  if (threadIdx.x == 0) {
    for (int s = 0; s < T::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < T::kBufs; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], T::kFoldWarps);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // The quantizer's codes and scales; and an earlier kernel that let this one start may still need tensor
  // memory on this SM, so the allocation comes behind it too.
  pdl_wait();
  if (warp == T::kMmaWarp) {
    tmem_alloc(tmem_slot, T::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= T::kFoldWarps) {
    if constexpr (BN == 256) reg_shrink<kOtherRegs>();
    if (warp == T::kLoadWarp && lane == 0) {
      // ---------------------------------------------------------- TMA producer
      prefetch_tmap(&maps.a);
      prefetch_tmap(&maps.b);
      int it = 0;
      bool ok = true;
      for (int tile = tile0; tile < p.num_tiles && ok; tile += step) {
        const int mt = tile % p.m_tiles, nt = tile / p.m_tiles;
        for (int j = 0; j < KB; ++j, ++it) {
          const int s = it % T::kStages;
          if (!timed_wait(&empty[s], ((it / T::kStages) & 1) ^ 1, wc)) {
            ok = false;
            break;
          }
          uint8_t* st = stages + s * T::kStage;
          mbar_arrive_expect_tx(&full[s], T::kStage);
          tma_load_2d(&maps.a, &full[s], st, (j_first + j) * kBlk, mt * 128);
          tma_load_2d(&maps.b, &full[s], st + T::kStageA, (j_first + j) * kBlk, nt * BN);
        }
      }
      // No block leaves with copies in flight, whoever gave up on them.
      for (int j = (it > T::kStages ? it - T::kStages : 0); j < it; ++j)
        mbar_wait_drain(&full[j % T::kStages], (j / T::kStages) & 1, drain_limit(p.limit));
    } else if (warp == T::kMmaWarp) {
      // ---------------------------------------------------------- MMA issuer: one accumulator per block of 128
      if (elect_one()) {
        constexpr uint64_t kDesc = sdesc_const(16, 1024, LAYOUT_SW128);
        constexpr uint32_t idesc = idesc_e4m3_f32(128, BN);
        const uint64_t first = kDesc + sdesc_addr(stages);
        int s = 0, b = 0;
        uint32_t s_par = 0, b_par = 1;
        bool ok = true;
        for (int tile = tile0; tile < p.num_tiles && ok; tile += step) {
          for (int j = 0; j < KB; ++j) {
            ok = timed_wait(&acc_empty[b], b_par, wc) && timed_wait(&full[s], s_par, wc);
            if (!ok) break;
            tc_fence_after();
            const uint64_t da = first + (uint32_t)(s * (T::kStage >> 4)), db = da + (T::kStageA >> 4);
#pragma unroll
            for (int kk = 0; kk < kBlk / 32; ++kk)  // K = 32 codes (bytes) per instruction
              mma_f8f6f4(tmem + b * BN, da + 2 * kk, db + 2 * kk, idesc, kk != 0 ? 1u : 0u);
            umma_commit(&empty[s]);
            umma_commit(&acc_full[b]);
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
        umma_commit(mma_done);
        mbar_wait_drain(mma_done, 0, drain_limit(p.limit));
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ fold and epilogue
    if constexpr (BN == 256) reg_grow<kFoldRegs>();
    const int q = warp & 3;   // tensor-memory lane quarter
    const int h = warp >> 2;  // column half
    const uint32_t taddr = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(FC * h);
    // Scales of this thread's row and this warp's columns in a tile; four blocks of 128 to a load.
    const float4 *px = nullptr, *pw = nullptr;
    auto scales_of = [&](int mt, int nt) {
      const int m = min(mt * 128 + 32 * q + lane, p.M - 1);  // rows past the last are not stored
      const int nb = min((nt * BN + FC * h) / kBlk, p.NB - 1);  // nor are columns past N
      px = (const float4*)(p.sx + (long long)m * p.ld + j_first);
      pw = (const float4*)(p.sw + (long long)nb * p.ld + j_first);
    };
    auto fetch = [&](float4& x, float4& w) {
      if (SVDQ_INB(p.status, (const char*)px - (const char*)p.sx, 16, 4ll * p.M * p.ld)) x = __ldg(px);
      if (SVDQ_INB(p.status, (const char*)pw - (const char*)p.sw, 16, 4ll * p.NB * p.ld)) w = __ldg(pw);
      ++px;
      ++pw;
    };
    int mt = tile0 % p.m_tiles, nt = tile0 / p.m_tiles, mt_next = 0, nt_next = 0;
    scales_of(mt, nt);
    int b = 0;
    uint32_t b_par = 0;
    bool ok = true;
    float4 xn = make_float4(0.f, 0.f, 0.f, 0.f), wn = xn;  // the next four blocks' scales, asked for four folds ahead
    fetch(xn, wn);
    // far: a product of scales may be past binary32.
    auto tiles = [&](auto far) {
      for (int tile = tile0; tile < p.num_tiles && ok; tile += step) {
        const int m0 = mt * 128 + 32 * q;
        const int n0 = nt * BN + FC * h;
        // The bias is added at the end; bring it near now.
        if (8 * lane < FC && n0 + 8 * lane < p.N)
          asm volatile("prefetch.global.L1 [%0];" ::"l"(p.bias + n0 + 8 * lane));
        float acc[FC];
#pragma unroll
        for (int i = 0; i < FC; ++i) acc[i] = 0.f;
        auto block = [&](float s, auto&& before) {  // the next accumulator's part of the sums
          ok = timed_wait(&acc_full[b], b_par, wc) && ok;
          __syncwarp();
          tc_fence_after();
          const uint32_t t = taddr + (uint32_t)(b * BN);
          before(t);
          if constexpr (FC == 128) {
            fold64(t, s, acc);
            fold64(t + 64, s, acc + 64);
          } else if constexpr (FC == 64) {
            fold64(t, s, acc);
          } else {
            fold32(t, s, acc);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[b]);
          if (++b == T::kBufs) {
            b = 0;
            b_par ^= 1;
          }
        };
        if constexpr (far.value) {
          for (int j = 0; j < KB && ok; ++j) {
            const long long ax = (long long)min(m0 + lane, p.M - 1) * p.ld + j_first + j;
            const long long aw = (long long)min(n0 / kBlk, p.NB - 1) * p.ld + j_first + j;
            float x = 0.f, w = 0.f;
            if (SVDQ_INB(p.status, 4 * ax, 4, 4ll * p.M * p.ld) && SVDQ_INB(p.status, 4 * aw, 4, 4ll * p.NB * p.ld)) {
              x = p.sx[ax];
              w = __ldg(p.sw + aw);
            }
            const bool past = past_f32(x * w);
            block(past ? fmaxf(x, w) : x * w, [&](uint32_t t) {
              if (__any_sync(0xffffffffu, past)) scale_columns(t, FC, [&](int) { return past ? fminf(x, w) : 1.f; });
            });
            ok = __all_sync(0xffffffffu, ok);
          }
          mt_next = (tile + step) % p.m_tiles;
          nt_next = (tile + step) / p.m_tiles;
        } else {
          for (int j0 = 0; j0 < KB; j0 += 4) {
            const float sc[4] = {xn.x * wn.x, xn.y * wn.y, xn.z * wn.z, xn.w * wn.w};
            if (j0 + 4 >= KB) {  // the next tile's (past the last tile: any place inside)
              const int next = min(tile + step, p.num_tiles - 1);
              mt_next = next % p.m_tiles;
              nt_next = next / p.m_tiles;
              scales_of(mt_next, nt_next);
            }
            fetch(xn, wn);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              if (j0 + u >= KB) break;
              block(sc[u], [](uint32_t) {});
            }
            ok = __all_sync(0xffffffffu, ok);  // an expired wait: its sums are not stored
            if (!ok) break;
          }
        }
        if (!ok) break;
        if constexpr (SPLIT) {  // every load and product of this CTA is complete: the sums go where the stages were
          float* part = (float*)stages + (32 * q + lane) * T::kPartLd + FC * h;
#pragma unroll
          for (int i = 0; i < FC; i += 4) *(float4*)(part + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
          break;
        }
        // A thread has a row, and rows lie far apart in memory: OC columns of the warp's 32 rows go through shared memory
        // (16-byte pieces, swizzled by the row).  64 columns leave by a bulk tensor store, which the next tile's folds need
        // not wait for; 32 columns by neighbouring lanes that write a row's neighbouring pieces.
        constexpr int PIECES = OC / 8;  // of a row
        uint8_t* mine = sm_out + warp * T::kOut;
#pragma unroll
        for (int c = 0; c < FC; c += OC) {
          if (OC == 64 && lane == 0) bulk_wait_read<0>();  // the store before has read its source
          __syncwarp();
#pragma unroll
          for (int v = 0; v < PIECES; ++v) {
            float4 b0 = make_float4(0.f, 0.f, 0.f, 0.f), b1 = b0;
            if (n0 + c + 8 * v < p.N && SVDQ_INB(p.status, 4ll * (n0 + c + 8 * v), 32, 4ll * p.N)) {
              b0 = __ldg((const float4*)(p.bias + n0 + c + 8 * v));
              b1 = __ldg((const float4*)(p.bias + n0 + c + 8 * v) + 1);
            }
            const float bb[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              __nv_bfloat162 hv = __floats2bfloat162_rn(acc[c + 8 * v + 2 * e] + bb[2 * e],
                                                        acc[c + 8 * v + 2 * e + 1] + bb[2 * e + 1]);
              o[e] = *(uint32_t*)&hv;
            }
            *(uint4*)(mine + lane * (OC * 2) + ((v ^ lane) & (PIECES - 1)) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
          }
          if constexpr (OC == 64) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && m0 < p.M && n0 + c < p.N) {  // rows and columns past the last are clipped
              tma_store_2d(&maps.y, mine, n0 + c, m0);
              bulk_commit();
            }
          } else {
            __syncwarp();
            const int piece = lane & (PIECES - 1), n = n0 + c + 8 * piece;
            constexpr int ROWS = 32 / PIECES;  // rows to an instruction
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
              const int r = ROWS * i + lane / PIECES;
              const uint4 y = *(const uint4*)(mine + r * (OC * 2) + ((piece ^ r) & (PIECES - 1)) * 16);
              const long long at = (long long)(m0 + r) * p.N + n;
              if (m0 + r < p.M && n < p.N && SVDQ_INB(p.status, 2 * at, 16, 2ll * p.M * p.N)) *(uint4*)(p.Y + at) = y;
            }
            __syncwarp();
          }
        }
        mt = mt_next;
        nt = nt_next;
      }
    };
    if (__ldg(p.far) != 0) {
      tiles(std::true_type{});
    } else {
      tiles(std::false_type{});
    }
    if (!SPLIT && OC == 64 && lane == 0) bulk_wait<0>();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == T::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, T::kCols);
  }
  if constexpr (SPLIT) {  // join: four columns of a row to a thread, U of them at once
    constexpr int U = 4;
    const int m0 = tile0 % p.m_tiles * 128, n0 = tile0 / p.m_tiles * BN;
    const int units = min(128, p.M - m0) * (BN / 4), share = join_share(units, p.splits);
    const int first = rank * share, total = min(share, units - first);  // this CTA's (none, if negative)
    const bool good = *abort_flag == 0;
    if (!good) {  // an expired wait: the others' sums become NaN
      for (int i = threadIdx.x; i < 128 * T::kPartLd; i += kGemmThreads) ((float*)stages)[i] = __int_as_float(0x7FC00000);
    }
    cluster_sync();
    if (good) {
      const uint32_t base = smem_u32(stages);
      for (int u0 = threadIdx.x; u0 < total; u0 += U * kGemmThreads) {
        int row[U], n[U];
        uint32_t from[U];
        float4 y[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const int u = first + min(u0 + j * kGemmThreads, total - 1);
          const int c = 4 * (u % (BN / 4));
          row[j] = u / (BN / 4);
          n[j] = n0 + c;
          from[j] = base + (uint32_t)(row[j] * T::kPartLd + c) * 4;
          y[j] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (n[j] < p.N && SVDQ_INB(p.status, 4ll * n[j], 16, 4ll * p.N)) y[j] = __ldg((const float4*)(p.bias + n[j]));
        }
#pragma unroll 2
        for (int r = 0; r < p.splits; ++r) {
          float4 x[U];
#pragma unroll
          for (int j = 0; j < U; ++j) x[j] = dsmem_ld_f32x4(dsmem_addr(from[j], r));
#pragma unroll
          for (int j = 0; j < U; ++j) {
            y[j].x += x[j].x;
            y[j].y += x[j].y;
            y[j].z += x[j].z;
            y[j].w += x[j].w;
          }
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const long long at = (long long)(m0 + row[j]) * p.N + n[j];
          if (u0 + j * kGemmThreads < total && n[j] < p.N && SVDQ_INB(p.status, 2 * at, 8, 2ll * p.M * p.N)) {
            __nv_bfloat162 lo = __floats2bfloat162_rn(y[j].x, y[j].y), hi = __floats2bfloat162_rn(y[j].z, y[j].w);
            *(uint2*)(p.Y + at) = make_uint2(*(uint32_t*)&lo, *(uint32_t*)&hi);
          }
        }
      }
    }
    cluster_sync();  // a CTA's shared memory stays until every other has read it
  }
}

// ------------------------------------------------------------------ GEMM, few tokens
// Up to 64 tokens: bound by the weight, which is read once.  The operands change places, so that a tile is 128 rows of W
// (one block of the weight scales) by BT tokens and no tensor-core row goes to a token that is not there; one thread
// holds a row's sums for all tokens.  A cluster's CTAs split the inputs where there are fewer tiles than SMs, and join
// through distributed shared memory in the order of their ranks.  Two CTAs share an SM.  The loads of W do not wait for
// the quantizer.
template <int BT>
struct Few {
  static constexpr int kStageW = 128 * kBlk, kStage = kStageW + BT * kBlk;
  static constexpr int kStages = BT == 16 ? 5 : (BT == 32 ? 4 : 3);
  static constexpr int kBufs = BT == 64 ? 4 : 8;
  static constexpr uint32_t kCols = BT * kBufs;
  static constexpr int kTable = BT == 64 ? 24576 : 16384;  // bytes of scales: [block][token]
  static constexpr int kMaxBlocks = kTable / (4 * BT);
  static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + kTable + 512;
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs on an SM");
  static_assert(BT * 128 * 4 <= kStages * kStage, "partial sums fit the stages");
};
constexpr int kFewThreads = 192;  // warps 0-3 fold, 4 loads, 5 issues the products

template <int BT>
__global__ void __launch_bounds__(kFewThreads, 2) k_gemm_fp8_few(const __grid_constant__ F8Maps maps,
                                                               const __grid_constant__ F8Params p) {
  using T = Few<BT>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* stages = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);  // [kStages][W | X]
  float* table = (float*)(stages + T::kStages * T::kStage);                        // [blocks of this CTA][BT]
  uint64_t* full = (uint64_t*)((uint8_t*)table + T::kTable);
  uint64_t* empty = full + T::kStages;
  uint64_t* acc_full = empty + T::kStages;    // [kBufs]
  uint64_t* acc_empty = acc_full + T::kBufs;  // [kBufs]
  uint64_t* mma_done = acc_empty + T::kBufs;
  uint32_t* tmem_slot = (uint32_t*)(mma_done + 1);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  volatile int* wide_flag = abort_flag + 1;  // a product of scales of this CTA is past binary32
  const int warp = warp_index(), lane = threadIdx.x & 31;
  WaitCtl wc{abort_flag, p.status, p.limit};
  const int rank = p.splits > 1 ? (int)cluster_ctarank() : 0;
  const int nt = blockIdx.x / p.splits;
  const int per = (p.KB + p.splits - 1) / p.splits;
  const int j_first = min(rank * per, p.KB), blocks = min(per, p.KB - j_first);

  if (threadIdx.x == 0) {
    for (int s = 0; s < T::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < T::kBufs; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 4);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    *wide_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  if (warp == 4 && lane == 0) {  // the first stages' weights
    for (int j = 0; j < min(blocks, T::kStages); ++j) {
      mbar_arrive_expect_tx(&full[j], T::kStage);
      tma_load_2d(&maps.b, &full[j], stages + j * T::kStage, (j_first + j) * kBlk, nt * 128);
    }
  }
  pdl_wait();  // the quantizer's codes and scales; tensor memory that an earlier kernel may still need on this SM
  if (warp == 5) {
    tmem_alloc(tmem_slot, T::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  float acc[BT];
#pragma unroll
  for (int i = 0; i < BT; ++i) acc[i] = 0.f;

  if (warp == 4) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int j = 0;
      for (; j < blocks; ++j) {
        const int s = j % T::kStages;
        uint8_t* st = stages + s * T::kStage;
        if (j >= T::kStages) {
          if (!timed_wait(&empty[s], ((j / T::kStages) & 1) ^ 1, wc)) break;
          mbar_arrive_expect_tx(&full[s], T::kStage);
          tma_load_2d(&maps.b, &full[s], st, (j_first + j) * kBlk, nt * 128);
        }
        tma_load_2d(&maps.a, &full[s], st + T::kStageW, (j_first + j) * kBlk, 0);
      }
      // No block leaves with copies in flight, whoever gave up on them.
      for (int k = (j > T::kStages ? j - T::kStages : 0); k < j; ++k)
        mbar_wait_drain(&full[k % T::kStages], (k / T::kStages) & 1, drain_limit(p.limit));
    }
  } else if (warp == 5) {
    // ------------------------------------------------------------ MMA issuer: one accumulator per block of 128
    if (elect_one()) {
      constexpr uint64_t kDesc = sdesc_const(16, 1024, LAYOUT_SW128);
      constexpr uint32_t idesc = idesc_e4m3_f32(128, BT);
      const uint64_t first = kDesc + sdesc_addr(stages);
      for (int j = 0; j < blocks; ++j) {
        const int s = j % T::kStages, b = j % T::kBufs;
        if (!timed_wait(&acc_empty[b], ((j / T::kBufs) & 1) ^ 1, wc) ||
            !timed_wait(&full[s], (j / T::kStages) & 1, wc))
          break;
        tc_fence_after();
        const uint64_t dw = first + (uint32_t)(s * (T::kStage >> 4)), dx = dw + (T::kStageW >> 4);
#pragma unroll
        for (int kk = 0; kk < kBlk / 32; ++kk)  // K = 32 codes (bytes) per instruction
          mma_f8f6f4(tmem + b * BT, dw + 2 * kk, dx + 2 * kk, idesc, kk != 0 ? 1u : 0u);
        umma_commit(&empty[s]);
        umma_commit(&acc_full[b]);
      }
      umma_commit(mma_done);
      mbar_wait_drain(mma_done, 0, drain_limit(p.limit));
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ fold
    for (int i = threadIdx.x; i < blocks * BT; i += 128) {  // s_w s_x of this CTA's blocks
      const int t = i / blocks, j = i - t * blocks;
      const long long ax = (long long)t * p.ld + j_first + j, aw = (long long)nt * p.ld + j_first + j;
      float v = 0.f;
      if (t < p.M && SVDQ_INB(p.status, 4 * ax, 4, 4ll * p.M * p.ld) &&
          SVDQ_INB(p.status, 4 * aw, 4, 4ll * p.NB * p.ld)) {
        const float x = p.sx[ax], w = __ldg(p.sw + aw);
        v = x * w;
        if (past_f32(v)) {  // the larger, and the smaller comes to the sums
          v = fmaxf(x, w);
          *wide_flag = 1;
        }
      }
      table[j * BT + t] = v;
    }
    named_bar_sync(1, 128);
    const bool wide = *wide_flag != 0;
    const uint32_t taddr = tmem + ((uint32_t)(32 * warp) << 16);
    for (int j = 0; j < blocks; ++j) {
      const int b = j % T::kBufs;
      if (!warp_timed_wait(&acc_full[b], (j / T::kBufs) & 1, wc)) break;
      tc_fence_after();
      if (wide) {
        scale_columns(taddr + (uint32_t)(b * BT), BT, [&](int t) {
          const long long ax = (long long)t * p.ld + j_first + j, aw = (long long)nt * p.ld + j_first + j;
          if (t >= p.M || !SVDQ_INB(p.status, 4 * ax, 4, 4ll * p.M * p.ld) ||
              !SVDQ_INB(p.status, 4 * aw, 4, 4ll * p.NB * p.ld))
            return 1.f;
          const float x = p.sx[ax], w = __ldg(p.sw + aw);
          return past_f32(x * w) ? fminf(x, w) : 1.f;
        });
      }
      uint32_t r[BT];
      tmem_ld_cols(taddr + (uint32_t)(b * BT), r);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[b]);
#pragma unroll
      for (int i = 0; i < BT; i += 4) {
        const float4 sc = *(const float4*)(table + j * BT + i);
        acc[i] = fmaf(__uint_as_float(r[i]), sc.x, acc[i]);
        acc[i + 1] = fmaf(__uint_as_float(r[i + 1]), sc.y, acc[i + 1]);
        acc[i + 2] = fmaf(__uint_as_float(r[i + 2]), sc.z, acc[i + 2]);
        acc[i + 3] = fmaf(__uint_as_float(r[i + 3]), sc.w, acc[i + 3]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, T::kCols);
  }
  const bool good = *abort_flag == 0;  // after an expired wait this CTA stores nothing, and the others' sums become NaN
  if (p.splits == 1) {
    const int n = nt * 128 + threadIdx.x;
    if (good && warp < 4 && n < p.N && SVDQ_INB(p.status, 4ll * n, 4, 4ll * p.N)) {
      const float bias = __ldg(p.bias + n);
#pragma unroll
      for (int t = 0; t < BT; ++t) {
        const long long at = (long long)t * p.N + n;
        if (t < p.M && SVDQ_INB(p.status, 2 * at, 2, 2ll * p.M * p.N))
          p.Y[at] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[t] + bias));
      }
    }
    return;
  }
  float* part = (float*)stages;  // [BT][128]: every load and product is complete
  if (warp < 4) {
#pragma unroll
    for (int t = 0; t < BT; ++t) part[t * 128 + threadIdx.x] = good ? acc[t] : __int_as_float(0x7FC00000);
  }
  cluster_sync();
  if (good) {
    const uint32_t base = smem_u32(part);
    const int share = join_share(p.M * 32, p.splits), end = min(p.M * 32, (rank + 1) * share);
    for (int u = rank * share + threadIdx.x; u < end; u += kFewThreads) {
      const int t = u >> 5, c = 4 * (u & 31), n = nt * 128 + c;
      float4 x[kMaxSplit];
#pragma unroll
      for (int r = 0; r < kMaxSplit; ++r)  // all asked for before the first is used
        x[r] = r < p.splits ? dsmem_ld_f32x4(dsmem_addr(base + (uint32_t)(t * 128 + c) * 4, r))
                            : make_float4(0.f, 0.f, 0.f, 0.f);
      const long long at = (long long)t * p.N + n;
      if (n < p.N && SVDQ_INB(p.status, 4ll * n, 16, 4ll * p.N) && SVDQ_INB(p.status, 2 * at, 8, 2ll * p.M * p.N)) {
        float4 y = __ldg((const float4*)(p.bias + n));
#pragma unroll
        for (int r = 0; r < kMaxSplit; ++r) {
          y.x += x[r].x;
          y.y += x[r].y;
          y.z += x[r].z;
          y.w += x[r].w;
        }
        __nv_bfloat162 lo = __floats2bfloat162_rn(y.x, y.y), hi = __floats2bfloat162_rn(y.z, y.w);
        *(uint2*)(p.Y + at) = make_uint2(*(uint32_t*)&lo, *(uint32_t*)&hi);
      }
    }
  }
  cluster_sync();  // a CTA's shared memory stays until every other has read it
}

int launch_f8_quantize(const svdq_fp8_layer* L, const void* X, int64_t M, uint8_t* ws, cudaStream_t stream) {
  const F8Ws w = f8_ws_layout(M, L->K);
  const int KB = (int)((L->K + kBlk - 1) / kBlk);
  const int64_t rounds = (M * KB + kQuantThreads / 16 - 1) / (kQuantThreads / 16);
  const bool many = rounds >= 8 * (int64_t)device_sm_count(L->device);
  const dim3 grid((unsigned)(many ? (rounds + 3) / 4 : rounds));
  return launch_pdl(many ? k_fp8_quantize<4> : k_fp8_quantize<1>, grid, dim3(kQuantThreads), 0, stream,
                    (const uint16_t*)X, M, (int)L->K, KB, ws + w.codes, (float*)(ws + w.scales), (int)f8_scale_ld(L->K),
                    (int*)(ws + w.status)) == cudaSuccess
             ? SVDQ_OK
             : SVDQ_ERR_CUDA;
}

// Once per device and kernel: the shared-memory attribute, and how many clusters of each size are resident at once.
struct Fit {
  bool set = false;
  int clusters[kMaxSplit + 1] = {};
};
cudaLaunchConfig_t cluster_config(int grid, int threads, size_t smem, int splits, cudaLaunchAttribute (&attr)[2]) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}
template <auto kernel>
const Fit* fit_of(int dev, int threads, size_t smem, bool clusters) {
  static std::mutex mu;
  static Fit fits[64];
  if (dev < 0 || dev >= 64) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  Fit& f = fits[dev];
  if (!f.set) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
      return nullptr;
    for (int c = 2; clusters && c <= kMaxSplit; ++c) {
      cudaLaunchAttribute attr[2];
      cudaLaunchConfig_t cfg = cluster_config(296 * c, threads, smem, c, attr);
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&f.clusters[c], kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        f.clusters[c] = 0;
      }
    }
    f.set = true;
  }
  return &f;
}
template <int BN, bool SPLIT>
const Fit* tile_fit(int dev) {
  return fit_of<k_gemm_fp8<BN, SPLIT>>(dev, kGemmThreads, Tile<BN>::kSmem, SPLIT);
}
template <int BN, bool SPLIT>
int launch_f8_tile(const F8Maps& maps, const F8Params& p, int grid, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = cluster_config(grid, kGemmThreads, Tile<BN>::kSmem, p.splits, attr);
  if (!SPLIT) {
    cfg.attrs = attr + 1;
    cfg.numAttrs = 1;
  }
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, k_gemm_fp8<BN, SPLIT>, maps, p) == cudaSuccess ? SVDQ_OK : SVDQ_ERR_CUDA;
}

template <int BT>
int launch_f8_few(const svdq_fp8_layer* L, const F8Maps& maps, F8Params& p, cudaStream_t stream) {
  using T = Few<BT>;
  const Fit* f = fit_of<k_gemm_fp8_few<BT>>(L->device, kFewThreads, T::kSmem, true);
  if (!f) return SVDQ_ERR_CUDA;
  const int tiles = p.NB;
  // The largest cluster of which one for each tile is resident at once, two blocks of 128 to a CTA at least; up to four
  // blocks are faster than a join (2 tokens, 512 -> 1024: 4.0 us, two CTAs 4.6;  1024 -> 1024: four 4.6, two 5.3).
  p.splits = 1;
  for (int c = 2; c <= kMaxSplit && 2 * c <= p.KB && p.KB > 4; ++c)
    if (tiles <= f->clusters[c]) p.splits = c;
  while ((p.KB + p.splits - 1) / p.splits > T::kMaxBlocks) {
    if (p.splits == kMaxSplit) return -1;  // more inputs than the table of scales holds: the tiles above take them
    ++p.splits;
  }
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = cluster_config(tiles * p.splits, kFewThreads, T::kSmem, p.splits, attr);
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, k_gemm_fp8_few<BT>, maps, p) == cudaSuccess ? SVDQ_OK : SVDQ_ERR_CUDA;
}

// Tile width and cluster size: the least estimate of the time, in nanoseconds beyond the launch, as fitted to measurements
// with 30 to 2048 tokens, 320 to 9216 outputs and 512 to 9728 inputs of every width and cluster size.  Measured, us:
//   128 tokens, 9728 -> 1024: 64 columns over clusters of 5 11.9, of 2 16.5, unsplit 24.4; 128 columns over 7 13.5
//   512 tokens, 9728 -> 1024: 128 columns over 4 17.1; 64 over 2 19.2; unsplit 27.1
//   512 tokens, 3072 -> 3072: 128 columns 12.9; 256 16.8; 64 17.9 (two rounds over the SMs)
//   1024 tokens, 3072 -> 9216: 256 columns 30.6; 128 36.5; 64 58.7
struct F8Plan {
  int width, splits, per;  // width: 0, 1, 2 for 256, 128, 64 columns
};
int f8_plan(F8Plan* plan, int64_t M, int64_t N, int64_t KB, int dev) {
  const Fit* fits[3] = {tile_fit<256, false>(dev), tile_fit<128, true>(dev), tile_fit<64, true>(dev)};
  if (!fits[0] || !fits[1] || !fits[2] || !tile_fit<128, false>(dev) || !tile_fit<64, false>(dev)) return SVDQ_ERR_CUDA;
  const int64_t sms = device_sm_count(dev), rows = std::min<int64_t>(M, 128);
  static const int kBlock[3] = {480, 290, 250}, kTile[3] = {700, 500, 500};       // a block of 128 inputs, a tile
  static const int kJoin[3] = {0, 400, 0}, kJoinCta[3] = {0, 400, 250};           // of 128 rows: once, and for each CTA
  int64_t best = INT64_MAX;
  for (int w = 0; w < 3; ++w) {
    const int64_t tiles = (M + 127) / 128 * ((N + (256 >> w) - 1) / (256 >> w));
    for (int c = 1; c <= (w ? kMaxSplit : 1); ++c) {
      const int64_t per = c == 1 ? KB : (KB + 4 * c - 1) / (4 * c) * 4;  // scales are read four blocks at a time
      // (as many clusters as fit at once took a second round on some devices)
      if (c > 1 && (tiles >= fits[w]->clusters[c] || (KB + per - 1) / per != c)) continue;
      const int64_t rounds = c > 1 ? 1 : (tiles + sms - 1) / sms;
      const int64_t cost =
          rounds * (per * kBlock[w] + kTile[w]) + (c > 1 ? 1500 + (kJoin[w] + c * kJoinCta[w]) * rows / 128 : 0);
      if (cost < best) {
        best = cost;
        *plan = {w, c, (int)per};
      }
    }
  }
  return SVDQ_OK;
}

int launch_f8_gemm(const svdq_fp8_layer* L, int64_t M, void* Y, uint8_t* ws, cudaStream_t stream) {
  const F8Ws w = f8_ws_layout(M, L->K);
  F8Maps maps;
  std::memset(&maps, 0, sizeof(maps));
  F8Params p{};
  p.M = (int)M;
  p.N = (int)L->N;
  p.KB = (int)((L->K + kBlk - 1) / kBlk);
  p.NB = (int)((L->N + kBlk - 1) / kBlk);
  p.sx = (const float*)(ws + w.scales);
  p.ld = (int)f8_scale_ld(L->K);
  p.sw = L->wscales;
  p.far = L->far;
  p.bias = L->bias;
  p.Y = (uint16_t*)Y;
  p.status = (int*)(ws + w.status);
  p.limit = wait_limit_cycles();
  // From 33 tokens only while clusters of four and more fit beside one another, and for 9 to 64 blocks of 128 inputs:
  // 60 tokens, 3072 -> 3072 7.9 us against 9.0 with the tiles below, but 3072 -> 9216 11.4 against 10.0, 512 -> 3072 6.9
  // against 5.4 and 12288 -> 600 11.2 against 10.1.  (30 tokens, 3072 -> 9216: 8.9 against 12.2.)
  const bool narrow = 4 * ((L->N + kBlk - 1) / kBlk) <= device_sm_count(L->device) && p.KB > 8 && p.KB <= 64;
  const int few = M <= 16 ? 16 : (M <= 32 ? 32 : (M <= 64 && narrow ? 64 : 0));
  int st = encode_tmap_2d(&maps.a, CU_TENSOR_MAP_DATA_TYPE_UINT8, ws + w.codes, (uint64_t)L->K, (uint64_t)M,
                          (uint64_t)L->K, kBlk, few ? (uint32_t)few : 128, CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != SVDQ_OK) return st;
  if (few) {
    maps.b = L->map_w[1];
    st = few == 16   ? launch_f8_few<16>(L, maps, p, stream)
         : few == 32 ? launch_f8_few<32>(L, maps, p, stream)
                     : launch_f8_few<64>(L, maps, p, stream);
    if (st != -1) return st;
    st = encode_tmap_2d(&maps.a, CU_TENSOR_MAP_DATA_TYPE_UINT8, ws + w.codes, (uint64_t)L->K, (uint64_t)M,
                        (uint64_t)L->K, kBlk, 128, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != SVDQ_OK) return st;
  }
  F8Plan plan{};
  st = f8_plan(&plan, M, L->N, p.KB, L->device);
  if (st != SVDQ_OK) return st;
  p.splits = plan.splits;
  p.per = plan.per;
  p.m_tiles = (p.M + 127) / 128;
  p.num_tiles = p.m_tiles * (int)((L->N + (256 >> plan.width) - 1) / (256 >> plan.width));
  maps.b = L->map_w[plan.width];
  if (plan.splits > 1) {
    const int grid = p.num_tiles * plan.splits;
    return plan.width == 1 ? launch_f8_tile<128, true>(maps, p, grid, stream)
                           : launch_f8_tile<64, true>(maps, p, grid, stream);
  }
  st = encode_tmap_2d(&maps.y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, Y, (uint64_t)L->N, (uint64_t)M, (uint64_t)L->N * 2, 64, 32,
                      CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != SVDQ_OK) return st;
  const int sms = device_sm_count(L->device), grid = p.num_tiles < sms ? p.num_tiles : sms;
  return plan.width == 0   ? launch_f8_tile<256, false>(maps, p, grid, stream)
         : plan.width == 1 ? launch_f8_tile<128, false>(maps, p, grid, stream)
                           : launch_f8_tile<64, false>(maps, p, grid, stream);
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
  for (int64_t i = 0; i < N * K;) {  // E4M3 NaN; a stretch at a time, which the compiler turns into vectors
    const int64_t end = std::min(N * K, i + 4096);
    int bad = 0;
    for (; i < end; ++i) bad |= (wcodes[i] & 0x7F) == 0x7F;
    if (bad) return SVDQ_ERR_INVALID_ARG;
  }
  uint8_t* blob = (uint8_t*)blob_v;
  std::memset(blob, 0, b.wcodes);
  std::memset(blob + b.wcodes + (size_t)N * K, 0, b.total - b.wcodes - (size_t)N * K);
  const int far = *std::max_element(wscales, wscales + ns) > kFarScale;
  std::memcpy(blob + b.far, &far, sizeof(far));
  float* bf = (float*)(blob + b.bias);
  for (int64_t n = 0; n < N; ++n) bf[n] = bias ? host::bf16_to_f32(bias[n]) : 0.f;
  const int64_t kb = (K + kBlk - 1) / kBlk, ld = f8_scale_ld(K);
  for (int64_t i = 0; i < (N + kBlk - 1) / kBlk; ++i)
    std::memcpy(blob + b.wscales + (size_t)(i * ld) * 4, wscales + i * kb, (size_t)kb * 4);
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
  L->far = (const int*)(base + b.far);
  const uint32_t rows[3] = {256, 128, 64};
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
  // tiles and quantizer CTAs are counted in 31 bits
  if ((M + 127) / 128 * ((L->N + 63) / 64) > (1 << 30) || M * ((L->K + kBlk - 1) / kBlk) > ((int64_t)1 << 36))
    return SVDQ_ERR_INVALID_ARG;
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
