// RMS norm of the query and key heads and the position rotation, in one pass:
//
//   y = rot( w * x / sqrt(mean x^2 + eps) ),  rot: (a, c) -> (a cos - c sin, a sin + c cos).
//
// Bound by memory: every element is read once and written once, 16 bytes (8 elements) to a lane (9216 tokens of 24 + 24
// heads of 128: 44.4 us, 5.1 TB/s; half-split pairs, whose elements come in two pieces of 8 bytes, 47.2).  A head's row of
// dim elements lies in LG lanes (the power of two >= dim / 8), so the mean is a sum over shuffles and no shared memory
// is needed.  A CTA takes one token at a time: its lanes keep the token's cosines and sines and the weight in registers
// and walk the token's heads with them.
#include <cuda_bf16.h>

#include <cmath>

#include "sm100.cuh"
#include "svdq_internal.h"

namespace svdq {
namespace {

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

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *(const uint32_t*)&v;
}

// One token of one side.  PAIRS: 0 adjacent, 1 halves.  The weight is multiplied into the cosines and sines once, so
// that an output costs a product with 1/rms, a product and a fused multiply-add (two outputs to an instruction); the
// kernel issues about as long as it moves data, so instructions count.
// `u` holds the first heads' elements, asked for before anything else of the token.
constexpr int kUnroll = 3;  // heads of a lane in flight for each side
constexpr float kLeast = 0x1p-100f;  // least mean square that is taken as it comes: what its squares lose is below 2^-141
struct Place {
  int b, s;
};
__device__ __forceinline__ Place place_of(const Side& sd, long long token) {
  const unsigned t = (unsigned)token, n = (unsigned)sd.tokens;  // batch * tokens <= 2^30
  return {(int)(t / n), (int)(t % n)};
}
// The first elements of a lane's two groups of four: adjacent pairs, eight neighbours; halves, four elements and their four
// partners rot/2 further on, and past rot eight neighbours again, so that no lane needs another's elements.
struct Groups {
  int a, b;
  bool turned;  // rotated (adjacent pairs: the first group; a row's rotated part may end between the two)
};
template <int LG, int PAIRS>
__device__ __forceinline__ Groups groups_of(const NormParams& p, const Side& sd) {
  const int sub = threadIdx.x % LG, rot = sd.rope ? p.rot : 0;
  if (PAIRS == 1 && 8 * sub < rot) return {4 * sub, 4 * sub + rot / 2, true};
  return {8 * sub, 8 * sub + 4, 8 * sub < rot};
}
template <int T, int LG, int PAIRS>
__device__ __forceinline__ void load_heads(const NormParams& p, const Side& sd, const Place& at, int h0,
                                           uint4 (&u)[kUnroll]) {
  constexpr int ROWS = T / LG;
  const Groups e = groups_of<LG, PAIRS>(p, sd);
  const bool on = 8 * (int)(threadIdx.x % LG) < p.dim;
  const long long xb = at.b * sd.x_sb + at.s * sd.x_st;
#pragma unroll
  for (int k = 0; k < kUnroll; ++k) {
    const int h = h0 + k * ROWS + (int)threadIdx.x / LG;
    u[k] = make_uint4(0, 0, 0, 0);
    if (!on || h >= sd.heads) continue;
    const long long off = xb + (long long)h * sd.x_sh + e.a;
    if constexpr (PAIRS == 0) {
      if (SVDQ_INB(p.status, 2 * off, 16, sd.x_extent)) u[k] = *(const uint4*)(sd.x + off);
    } else {
      const long long off_b = off - e.a + e.b;
      if (SVDQ_INB(p.status, 2 * off, 8, sd.x_extent) && SVDQ_INB(p.status, 2 * off_b, 8, sd.x_extent)) {
        const uint2 lo = *(const uint2*)(sd.x + off), hi = *(const uint2*)(sd.x + off_b);
        u[k] = make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
    }
  }
}
template <int T, int LG, int PAIRS>
__device__ __forceinline__ void do_side(const NormParams& p, const Side& sd, long long token, const Place& place,
                                        uint4 (&u)[kUnroll]) {
  constexpr int ROWS = T / LG, UNROLL = kUnroll;
  const int first = threadIdx.x / LG;
  const Groups e = groups_of<LG, PAIRS>(p, sd);
  const bool on = 8 * (int)(threadIdx.x % LG) < p.dim;
  const int b = place.b, s = place.s;
  const float* r = nullptr;  // the token's row of cosines and sines
  [[maybe_unused]] long long row = s;
  bool bad = false;
  if (sd.rope) {
    if (sd.positions) {
      row = SVDQ_INB(p.status, 4 * token, 4, 4ll * sd.batch * sd.tokens) ? (long long)__ldg(sd.positions + token) : -1;
      bad = row < 0 || row >= sd.rope_rows;
      if (bad) row = 0;
    }
    r = sd.rope + row * p.rot;
  }
  if (bad && p.status && threadIdx.x == 0) atomicCAS(p.status, 0, SVDQ_ERR_INVALID_ARG);
  float w[8];  // of the first group, of the second
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.f;
  if (sd.weight && on && SVDQ_INB(p.status, 2 * e.a, 8, 2 * p.dim) && SVDQ_INB(p.status, 2 * e.b, 8, 2 * p.dim)) {
    const uint2 lo = __ldg((const uint2*)(sd.weight + e.a)), hi = __ldg((const uint2*)(sd.weight + e.b));
    unpack(make_uint4(lo.x, lo.y, hi.x, hi.y), w);
  }
  // Coefficients of a lane's four pairs, two pairs (g) to a register: ca multiplies the element, cb its partner;
  // [g][0] for the firsts of the pairs, [g][1] for the seconds.
  uint64_t ca2[2][2], cb2[2][2];
  bool turned[2];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    // adjacent: pairs 2g, 2g + 1 are the lane's group g; halves: elements 2g, 2g + 1 of the first group, and of the second
    const int f0 = PAIRS == 0 ? 4 * g : 2 * g, f1 = PAIRS == 0 ? 4 * g + 2 : 2 * g + 1;        // firsts, among w
    const int s0 = PAIRS == 0 ? 4 * g + 1 : 4 + 2 * g, s1 = PAIRS == 0 ? 4 * g + 3 : 5 + 2 * g;  // seconds
    turned[g] = PAIRS == 0 ? r != nullptr && e.a + 4 * g < p.rot : e.turned;
    float4 t = make_float4(1.f, 0.f, 1.f, 0.f);
    const int at = PAIRS == 0 ? e.a + 4 * g : 2 * e.a + 4 * g;  // in the table's row
    if (turned[g] && SVDQ_INB(p.status, 4 * (row * p.rot + at), 16, 4 * sd.rope_rows * p.rot))
      t = __ldg((const float4*)(r + at));
    ca2[g][0] = pack2(w[f0] * t.x, w[f1] * t.z);
    cb2[g][0] = pack2(-w[s0] * t.y, -w[s1] * t.w);
    ca2[g][1] = pack2(w[s0] * t.x, w[s1] * t.z);
    cb2[g][1] = pack2(w[f0] * t.y, w[f1] * t.w);
  }
  const long long yb = b * sd.y_sb + s * sd.y_st;
  const float inv_dim = 1.f / (float)p.dim;
  // every lane takes every round (the shuffles need whole warps); heads past the last read nothing
  for (int h0 = 0; h0 < sd.heads; h0 += ROWS * UNROLL) {
    if (h0 > 0) load_heads<T, LG, PAIRS>(p, sd, place, h0, u);
#pragma unroll
    for (int k = 0; k < UNROLL; ++k) {
      if (h0 + k * ROWS >= sd.heads) break;
      const int h = h0 + k * ROWS + first;
      const uint32_t in[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
      uint64_t lo[2], hi[2], ss2 = 0;  // the firsts of the pairs, the seconds
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if constexpr (PAIRS == 0) {
          lo[g] = pack2(in[2 * g] << 16, in[2 * g + 1] << 16);
          hi[g] = pack2(in[2 * g] & 0xFFFF0000u, in[2 * g + 1] & 0xFFFF0000u);
        } else {
          lo[g] = pack2(in[g] << 16, in[g] & 0xFFFF0000u);
          hi[g] = pack2(in[2 + g] << 16, in[2 + g] & 0xFFFF0000u);
        }
        ss2 = fma2(lo[g], lo[g], ss2);
        ss2 = fma2(hi[g], hi[g], ss2);
      }
      const float2 sp = unpack2(ss2);
      float ss = sp.x + sp.y;
#pragma unroll
      for (int o = LG / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float t = fmaf(ss, inv_dim, p.eps);
      float inv = rsqrtf(t);
      if (__any_sync(0xffffffffu, !(t >= kLeast && t < INFINITY))) {
        // Past binary32, or so small that squares lost their bits: the same on 2^-96 x or 2^96 x.  On 2^96 x, which is exact,
        // the head goes on; 2^-96 goes to the root instead, as the smaller elements would lose bits.  (The vote costs
        // 0.3 us of the 44 for a block of 9216 tokens; a branch for each head without it 2, the heads done again after the
        // round 1.)
        const float by = t < kLeast ? 0x1p96f : (t < INFINITY ? 1.f : 0x1p-96f);
        const uint64_t by2 = pack2(by, by);
        uint64_t q2 = 0;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const uint64_t a = mul2(lo[g], by2), c = mul2(hi[g], by2);
          q2 = fma2(a, a, q2);
          q2 = fma2(c, c, q2);
          if (by > 1.f) {
            lo[g] = a;
            hi[g] = c;
          }
        }
        const float2 qp = unpack2(q2);
        float qs = qp.x + qp.y;
#pragma unroll
        for (int o = LG / 2; o > 0; o >>= 1) qs += __shfl_xor_sync(0xffffffffu, qs, o);
        inv = rsqrtf(fmaf(qs, inv_dim, p.eps * by * by)) * (by < 1.f ? by : 1.f);
      }
      if (bad) inv = __int_as_float(0x7FC00000);
      const uint64_t inv2 = pack2(inv, inv);
      float2 y[2][2];  // [g][0] of the firsts of two pairs, [g][1] of the seconds
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        lo[g] = mul2(lo[g], inv2);
        hi[g] = mul2(hi[g], inv2);
        uint64_t a = mul2(lo[g], ca2[g][0]), c = mul2(hi[g], ca2[g][1]);
        if (turned[g]) {
          a = fma2(hi[g], cb2[g][0], a);
          c = fma2(lo[g], cb2[g][1], c);
        }
        y[g][0] = unpack2(a);
        y[g][1] = unpack2(c);
      }
      const long long off = yb + (long long)h * sd.y_sh + e.a;
      if (!on || h >= sd.heads) continue;
      if constexpr (PAIRS == 0) {
        if (SVDQ_INB(p.status, 2 * off, 16, sd.y_extent))
          *(uint4*)(sd.y + off) = make_uint4(bf16x2(y[0][0].x, y[0][1].x), bf16x2(y[0][0].y, y[0][1].y),
                                             bf16x2(y[1][0].x, y[1][1].x), bf16x2(y[1][0].y, y[1][1].y));
      } else {
        const long long off_b = off - e.a + e.b;
        if (SVDQ_INB(p.status, 2 * off, 8, sd.y_extent) && SVDQ_INB(p.status, 2 * off_b, 8, sd.y_extent)) {
          *(uint2*)(sd.y + off) = make_uint2(bf16x2(y[0][0].x, y[0][0].y), bf16x2(y[1][0].x, y[1][0].y));
          *(uint2*)(sd.y + off_b) = make_uint2(bf16x2(y[0][1].x, y[0][1].y), bf16x2(y[1][1].x, y[1][1].y));
        }
      }
    }
  }
}

template <int T, int LG, int PAIRS>
__global__ void __launch_bounds__(T, 768 / T) k_qk_norm_rope(const __grid_constant__ NormParams p) {
  pdl_wait();
  const long long n0 = (long long)p.side[0].batch * p.side[0].tokens, n1 = (long long)p.side[1].batch * p.side[1].tokens;
  const long long n = n0 > n1 ? n0 : n1;
  for (long long token = blockIdx.x; token < n; token += gridDim.x) {
    uint4 u0[kUnroll], u1[kUnroll];
    const Place at0 = place_of(p.side[0], token), at1 = place_of(p.side[1], token);
    if (token < n0) load_heads<T, LG, PAIRS>(p, p.side[0], at0, 0, u0);
    if (token < n1) load_heads<T, LG, PAIRS>(p, p.side[1], at1, 0, u1);
    if (token < n0) do_side<T, LG, PAIRS>(p, p.side[0], token, at0, u0);
    if (token < n1) do_side<T, LG, PAIRS>(p, p.side[1], token, at1, u1);
  }
}

template <int T, int LG>
cudaError_t launch(const NormParams& p, unsigned grid, cudaStream_t stream) {
  return p.pairs == SVDQ_PAIRS_HALVES
             ? launch_pdl(k_qk_norm_rope<T, LG, 1>, dim3(grid), dim3(T), 0, stream, p)
             : launch_pdl(k_qk_norm_rope<T, LG, 0>, dim3(grid), dim3(T), 0, stream, p);
}
// Threads to a token.  Few tokens: four warps, for the latency (one token of 24 + 24 heads of 128: 2.7 us, with one warp
// 6.9).  With more, the SMs are filled by tokens, and fewer threads to each leave fewer of them without a head and load
// the token's coefficients less often: 999 tokens of 16 + 4 heads of 72 5.0 us with four warps, 4.0 with two, 4.7 with
// one; 18000 of 16 + 4 of 96 58, 44 and 37; 9216 of 24 + 24 of 128 44.3, 43.7 and 44.5.
template <int LG>
cudaError_t launch(const NormParams& p, int64_t tokens, int dev, cudaStream_t stream) {
  const unsigned grid = (unsigned)(tokens < (1 << 20) ? tokens : (1 << 20));
  const int64_t sms = device_sm_count(dev);
  if (tokens <= 2 * sms) return launch<128, LG>(p, grid, stream);
  const int lanes = (p.side[0].heads + p.side[1].heads) * LG;
  return tokens >= 12 * sms && lanes <= 512 ? launch<32, LG>(p, grid, stream) : launch<64, LG>(p, grid, stream);
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
  const cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  if (dim <= 8) e = launch<1>(p, tokens, dev, s);
  else if (dim <= 16) e = launch<2>(p, tokens, dev, s);
  else if (dim <= 32) e = launch<4>(p, tokens, dev, s);
  else if (dim <= 64) e = launch<8>(p, tokens, dev, s);
  else if (dim <= 128) e = launch<16>(p, tokens, dev, s);
  else e = launch<32>(p, tokens, dev, s);
  return e == cudaSuccess ? SVDQ_OK : SVDQ_ERR_CUDA;
}
