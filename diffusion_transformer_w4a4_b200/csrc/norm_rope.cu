// RMS norm of the query and key heads and the position rotation, in one pass:
//
//   y = rot( w * x / sqrt(mean x^2 + eps) ),  rot: (a, c) -> (a cos - c sin, a sin + c cos).
//
// Bound by memory: every element is read once and written once, 16 bytes (8 elements) to a lane.  A
// head's row of dim elements lies in LG lanes (the power of two >= dim / 8), so the mean is a sum over
// shuffles and no shared memory is needed.  A CTA takes one token at a time: its lanes keep the token's
// cosines and sines and the weight in registers and walk the token's heads with them.
#include <cuda_bf16.h>

#include <cmath>

#include "sm100.cuh"
#include "svdq_internal.h"

namespace svdq {
namespace {

constexpr int kThreads = 128;

struct Side {
  const uint16_t* x;
  uint16_t* y;
  long long x_sb, x_st, x_sh, y_sb, y_st, y_sh;  // elements
  int batch, tokens, heads;
  const uint16_t* weight;
  const float* rope;
  long long rope_rows;
  const int32_t* positions;
  long long x_extent, y_extent;  // bytes
};
struct NormParams {
  Side side[2];
  int dim, rot, pairs;
  float eps;
  int* status;
};

__device__ __forceinline__ void unpack(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// UNROLL heads of one token at a time; PAIRS: 0 adjacent, 1 halves.
template <int LG, int PAIRS>
__device__ __forceinline__ void do_side(const NormParams& p, const Side& sd, long long token) {
  constexpr int ROWS = kThreads / LG, UNROLL = 4;
  const int sub = threadIdx.x % LG, first = threadIdx.x / LG;
  const int e0 = 8 * sub;
  const bool on = e0 < p.dim;
  const int b = (int)(token / sd.tokens), s = (int)(token - (long long)b * sd.tokens);
  float w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.f;
  if (sd.weight && on && SVDQ_INB(p.status, 2 * e0, 16, 2 * p.dim)) unpack(__ldg((const uint4*)(sd.weight + e0)), w);
  // cosine and sine of this lane's pairs (adjacent: 4; halves: one for each element)
  constexpr int NP = PAIRS == 0 ? 4 : 8;
  float cs[NP], sn[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
  }
  const int half = p.rot >> 1;
  bool bad = false;
  if (sd.rope && p.rot > 0) {
    long long row = s;
    if (sd.positions) {
      row = SVDQ_INB(p.status, 4 * token, 4, 4ll * sd.batch * sd.tokens) ? (long long)__ldg(sd.positions + token) : -1;
      bad = row < 0 || row >= sd.rope_rows;
      if (bad) row = 0;
    }
    const float* r = sd.rope + row * p.rot;
#pragma unroll
    for (int g = 0; g < 2; ++g) {  // four elements: two adjacent pairs, or four halves' pairs
      const int e = e0 + 4 * g;
      if (e >= p.rot) continue;
      const int at = PAIRS == 0 ? e : 2 * (e < half ? e : e - half);  // floats from the row's start
      if (!SVDQ_INB(p.status, 4 * (row * p.rot + at), PAIRS == 0 ? 16 : 32, 4 * sd.rope_rows * p.rot)) continue;
#pragma unroll
      for (int v = 0; v < (PAIRS == 0 ? 1 : 2); ++v) {
        const float4 t = __ldg((const float4*)(r + at) + v);
        const int i = PAIRS == 0 ? 2 * g : 4 * g + 2 * v;
        cs[i] = t.x;
        sn[i] = t.y;
        cs[i + 1] = t.z;
        sn[i + 1] = t.w;
      }
      if (PAIRS == 1 && e < half) {  // the first of a pair subtracts
#pragma unroll
        for (int i = 0; i < 4; ++i) sn[4 * g + i] = -sn[4 * g + i];
      }
    }
  }
  if (bad && p.status && threadIdx.x == 0) atomicCAS(p.status, 0, SVDQ_ERR_INVALID_ARG);
  const long long xb = b * sd.x_sb + s * sd.x_st, yb = b * sd.y_sb + s * sd.y_st;
  // every lane takes every round (the shuffles need whole warps); heads past the last read nothing
  for (int h0 = 0; h0 < sd.heads; h0 += ROWS * UNROLL) {
    uint4 u[UNROLL];
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      const int h = h0 + k * ROWS + first;
      u[k] = make_uint4(0, 0, 0, 0);
      const long long off = xb + (long long)h * sd.x_sh + e0;
      if (on && h < sd.heads && SVDQ_INB(p.status, 2 * off, 16, sd.x_extent)) u[k] = *(const uint4*)(sd.x + off);
    }
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      if (h0 + k * ROWS >= sd.heads) break;
      const int h = h0 + k * ROWS + first;
      float v[8];
      unpack(u[k], v);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
#pragma unroll
      for (int o = LG / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      float r = rsqrtf(ss / (float)p.dim + p.eps);
      if (bad) r = __int_as_float(0x7FC00000);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= r * w[i];
      float y[8];
      if (PAIRS == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[2 * i] = v[2 * i] * cs[i] - v[2 * i + 1] * sn[i];
          y[2 * i + 1] = v[2 * i] * sn[i] + v[2 * i + 1] * cs[i];
        }
      } else {
        // the partner of element e is e +- rot/2; its place among a lane's eight is i or (rot/2 = 4 mod 8) i ^ 4
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = e0 + i;
          const int pe = e < half ? e + half : (e < p.rot ? e - half : e);
          const float send = (half & 4) ? v[i ^ 4] : v[i];
          float partner = __shfl_sync(0xffffffffu, send, pe >> 3, LG);
          y[i] = e < p.rot ? v[i] * cs[i] + partner * sn[i] : v[i];
        }
      }
      const long long off = yb + (long long)h * sd.y_sh + e0;
      if (on && h < sd.heads && SVDQ_INB(p.status, 2 * off, 16, sd.y_extent)) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          __nv_bfloat162 hv = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
          o[i] = *(uint32_t*)&hv;
        }
        *(uint4*)(sd.y + off) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

template <int LG, int PAIRS>
__global__ void __launch_bounds__(kThreads) k_qk_norm_rope(const __grid_constant__ NormParams p) {
  pdl_wait();
  const long long n0 = (long long)p.side[0].batch * p.side[0].tokens, n1 = (long long)p.side[1].batch * p.side[1].tokens;
  const long long n = n0 > n1 ? n0 : n1;
  for (long long token = blockIdx.x; token < n; token += gridDim.x) {
    if (token < n0) do_side<LG, PAIRS>(p, p.side[0], token);
    if (token < n1) do_side<LG, PAIRS>(p, p.side[1], token);
  }
}

template <int LG>
cudaError_t launch(const NormParams& p, unsigned grid, cudaStream_t stream) {
  return p.pairs == SVDQ_PAIRS_HALVES
             ? launch_pdl(k_qk_norm_rope<LG, 1>, dim3(grid), dim3(kThreads), 0, stream, p)
             : launch_pdl(k_qk_norm_rope<LG, 0>, dim3(grid), dim3(kThreads), 0, stream, p);
}

}  // namespace
}  // namespace svdq

using namespace svdq;

extern "C" svdq_status svdq_qk_norm_rope(const svdq_norm_rope_args* q, const svdq_norm_rope_args* k, int64_t dim,
                                         int64_t rot_dim, int pairs, float eps, int32_t* status, void* stream) {
  const int64_t lim = (int64_t)1 << 30;
  if (!q && !k) return SVDQ_ERR_INVALID_ARG;
  if (dim < 8 || dim > 256 || dim % 8 != 0 || rot_dim < 0 || rot_dim > dim || rot_dim % 8 != 0)
    return SVDQ_ERR_INVALID_ARG;
  if (pairs != SVDQ_PAIRS_INTERLEAVED && pairs != SVDQ_PAIRS_HALVES) return SVDQ_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps) || ((uintptr_t)status & 3)) return SVDQ_ERR_INVALID_ARG;
  const svdq_norm_rope_args* in[2] = {q, k};
  NormParams p{};
  int64_t tokens = 0;
  for (int i = 0; i < 2; ++i) {
    const svdq_norm_rope_args* a = in[i];
    Side& sd = p.side[i];
    sd.tokens = 1;  // an absent side has no batch
    if (!a) continue;
    if (a->batch < 0 || a->tokens < 0 || a->heads < 0 || a->batch > lim || a->tokens > lim || a->heads > lim)
      return SVDQ_ERR_INVALID_ARG;
    if (a->batch == 0 || a->tokens == 0 || a->heads == 0) continue;
    if (a->batch * a->tokens > lim) return SVDQ_ERR_INVALID_ARG;
    int st = check_heads(a->y, a->batch, a->tokens, a->heads, dim, true);
    if (st == SVDQ_OK) st = check_heads(a->x, a->batch, a->tokens, a->heads, dim, false);
    if (st != SVDQ_OK) return (svdq_status)st;
    if (((uintptr_t)a->weight & 15) || ((uintptr_t)a->rope & 15) || ((uintptr_t)a->positions & 3))
      return SVDQ_ERR_INVALID_ARG;
    const bool rotates = a->rope && rot_dim > 0;
    if (rotates && (a->rope_rows < 1 || a->rope_rows > lim || (!a->positions && a->rope_rows < a->tokens)))
      return SVDQ_ERR_INVALID_ARG;
    sd.x = (const uint16_t*)a->x.data;
    sd.y = (uint16_t*)a->y.data;
    sd.x_sb = a->x.stride_batch;
    sd.x_st = a->x.stride_token;
    sd.x_sh = a->x.stride_head;
    sd.y_sb = a->y.stride_batch;
    sd.y_st = a->y.stride_token;
    sd.y_sh = a->y.stride_head;
    sd.batch = (int)a->batch;
    sd.tokens = (int)a->tokens;
    sd.heads = (int)a->heads;
    sd.weight = (const uint16_t*)a->weight;
    sd.rope = rotates ? a->rope : nullptr;
    sd.rope_rows = a->rope_rows;
    sd.positions = rotates ? a->positions : nullptr;
    sd.x_extent = heads_extent(a->x, a->batch, a->tokens, a->heads, dim);
    sd.y_extent = heads_extent(a->y, a->batch, a->tokens, a->heads, dim);
    if (a->batch * a->tokens > tokens) tokens = a->batch * a->tokens;
  }
  if (tokens == 0) return SVDQ_OK;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return SVDQ_ERR_UNSUPPORTED_DEVICE;
  }
  const svdq_status sd = svdq_device_check(dev);
  if (sd != SVDQ_OK) return sd;
  if (status && check_blob_pointer(status, dev) != SVDQ_OK) return SVDQ_ERR_INVALID_ARG;
  for (const Side& s : p.side) {
    const void* ptrs[5] = {s.x, s.y, s.weight, s.rope, s.positions};
    for (const void* ptr : ptrs)
      if (ptr && check_blob_pointer(ptr, dev) != SVDQ_OK) return SVDQ_ERR_INVALID_ARG;
  }
  p.dim = (int)dim;
  p.rot = (int)rot_dim;
  p.pairs = pairs;
  p.eps = eps;
  p.status = status;
  NvtxRange range("svdq/qk_norm_rope");
  const unsigned grid = (unsigned)(tokens < (1 << 20) ? tokens : (1 << 20));
  const cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  if (dim <= 8) e = launch<1>(p, grid, s);
  else if (dim <= 16) e = launch<2>(p, grid, s);
  else if (dim <= 32) e = launch<4>(p, grid, s);
  else if (dim <= 64) e = launch<8>(p, grid, s);
  else if (dim <= 128) e = launch<16>(p, grid, s);
  else e = launch<32>(p, grid, s);
  return e == cudaSuccess ? SVDQ_OK : SVDQ_ERR_CUDA;
}
