// Attention of queries over another sequence's keys and values (cross attention),
//
//   O[b,s,h,:] = sum_t p_t V[b,t,g,:] / sum_t p_t,   p_t = exp(scale Q[b,s,h,:] . K[b,t,g,:]),
//
// t over the keys that sample b keeps (t < kv_len[b], kv_mask[b,t] != 0), g = h / (heads / kv_heads).
//
// One pass over the keys with a running maximum m and sum l per row:
//   m' = max(m, max_t s_t),  l' = l 2^(c (m - m')) + sum_t 2^(c (s_t - m')),  O' = O 2^(c (m - m')) + P V,
// with c = scale log2(e).  The rescaling of O is left out while m' exceeds the maximum in use by
// less than 2^kLazy in p (sums and O are binary32, so p up to 2^8 costs no precision).
//
// Tiles: 128 rows x 128 keys.  S = Q K^T (tcgen05.mma kind::f16, binary32 in tensor memory); one thread
// per row reads its S row twice (maximum, exponentials), writes P as bf16 over it, and P V reads P from tensor memory.
// P is rounded to bf16 because the product takes 16-bit operands; its sum l uses the unrounded values.  Two streams
// of 128 rows run in turn, so that one's products overlap the other's exponentials:
//   kPairs       the streams are two query tiles that share the key tiles (each key tile is read once for 256 rows);
//                persistent, one CTA per SM.
//   kSplitPairs  the same for fewer rows, the keys split over a cluster of up to 8 CTAs that join through distributed
//                shared memory, in a fixed order (one launch, no workspace, no atomics).
//   kSingle      the streams are the even and odd key tiles of one query tile, joined at the end; and a cluster splits
//                the keys further.
//   kQuarter     kSingle with 32 rows at most, as in decoding: the rows lie in all four lane quarters of the tile, and a
//                quarter's warp takes only its quarter of the keys, so that no warp idles and a tile's exponentials
//                take a quarter of the time; the other quarters' P is zero there, and the quarters are joined too.
// What bounds it: with many rows the chain S -> exponentials -> P -> product, about 3200 clocks for a key tile of both
// streams against 2048 of products (heads of 128: 24 x 4096 x 4608 in 200 us, 1.16 PFLOP/s); with few rows latency
// (2 x 24 heads of one token over 4096 keys: 13.2 us, 34 MB of keys and values at 2.5 TB/s).  A quarter of the
// exponentials are computed by a polynomial, as the special-function unit is the busiest: 24 x 4096 x 4608 in 195-200 us
// against 217 with none of them, 223 with an eighth and 218 with a half.
// Rows of a tile are (token, query head of the group) pairs, so heads that share keys share their tiles.
//
// Masked keys: scores become -inf by selection, and the masked rows of V are zeroed in shared memory
// before the product (0 x NaN would poison it).  Rows without a key give 0.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>

#include "sm100.cuh"
#include "svdq_internal.h"

namespace svdq {
namespace {

constexpr int kRows = 128, kKeys = 128;
constexpr int kChunkBytes = 128 * 128;  // 128 rows of 64 bf16
constexpr int kThreads = 384;           // warps 0-3, 4-7 softmax; 8 loads; 9 products; 10 masked rows of V
constexpr float kLazy = 8.f;
constexpr int kMaxSplit = 8;
constexpr float kLog2E = 1.4426950408889634f;

template <int DC>
struct Geo {  // DC: 64-wide chunks of the head dimension
  static constexpr int kSlots = DC == 2 ? 4 : 8;
  static constexpr int kTile = DC * kChunkBytes;
  static constexpr int kPartLd = 64 * DC + 4;
  static constexpr int kStage = 8 * 32 * 128;  // kPairs: 64 columns of 32 rows a softmax warp; else m, l and weights
  static constexpr size_t kSmem = 1024 + (size_t)(2 + kSlots) * kTile + kStage + 512;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(256 * kPartLd * 4 <= (2 + kSlots) * kTile, "partial results fit the query tiles and the ring");
};

// How the work is spread (see the top): pairs of query tiles, the same with their keys split over a cluster, one query
// tile with its keys split over the streams and a cluster, and that with a quarter of a tile's keys to a warp.
enum Mode { kPairs, kSplitPairs, kSingle, kQuarter };

struct AttnParams {
  int sq, sk, hq, hk, d;
  int group;       // query heads packed into the rows of a tile
  int tok_tile;    // tokens per 128-row tile: 128 / group
  int row_tiles;   // work items per (sample, item head): tiles (or pairs of tiles) of tokens
  int heads_it;    // item heads: hq / group
  int items;
  int step, step_rt, step_h, step_b;  // CTAs (clusters) between a CTA's items, and the same divided as an item is
  int ksteps;      // ceil(d / 16)
  int npv;         // d rounded up to 16
  int splits;
  int q_bm, q_hm, k_bm, k_hm, v_bm, v_hm;  // 0 where that dimension is broadcast (or of size one)
  float c;                                 // scale * log2(e)
  const int* kv_len;
  const uint8_t* kv_mask;
  long long mask_ld, mask_extent;
  int o_tma;  // a warp's 32 rows are whole tokens: written by bulk tensor stores
  uint16_t* out;
  long long o_sb, o_st, o_sh, out_extent;  // elements; extent in bytes
  int batch;
  int* status;
  unsigned long long limit;
};
struct AttnMaps {
  CUtensorMap q, k, v, o;  // o (PAIR, o_tma): 64 columns of the 32 rows of a softmax warp
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^x of two x <= 126 without the special-function unit, which at 16 results a clock bounds the softmax:
// x = n + f, n the nearest integer (found by adding 1.5 * 2^23), 2^f by the polynomial of degree 4 with the least
// relative error on [-1/2, 1/2] (2.7e-6 in binary32, from a Remez exchange), n added to the exponent.  Below -125,
// where the result would be subnormal or the sum of exponents wrap, it is 0 (a score of -inf has no share at all).
__device__ __forceinline__ float2 ex2_poly(float2 x) {
  const uint64_t v = pack2(x.x, x.y);
  const uint64_t magic = pack2(12582912.f, 12582912.f), unmagic = pack2(-12582912.f, -12582912.f);
  const uint64_t t = add2(v, magic);
  const uint64_t f = fma2(add2(t, unmagic), pack2(-1.f, -1.f), v);
  uint64_t y = fma2(pack2(0.009570102207362652f, 0.009570102207362652f), f,
                    pack2(0.05591785907745361f, 0.05591785907745361f));
  y = fma2(y, f, pack2(0.240247443318367f, 0.240247443318367f));
  y = fma2(y, f, pack2(0.6931217908859253f, 0.6931217908859253f));
  y = fma2(y, f, pack2(0.9999992847442627f, 0.9999992847442627f));
  const float2 yy = unpack2(y), tt = unpack2(t);
  const float a = __uint_as_float(__float_as_uint(yy.x) + (__float_as_uint(tt.x) << 23));
  const float b = __uint_as_float(__float_as_uint(yy.y) + (__float_as_uint(tt.y) << 23));
  return make_float2(x.x < -125.f ? 0.f : a, x.y < -125.f ? 0.f : b);
}
// Largest of three; NaN if one is NaN.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// c m, which the exponents subtract: 0 for a row without a score above -inf (its exponentials are all 0), and NaN where
// it is infinite (an infinite or NaN score, or scale times a score past binary32), so that the whole row becomes NaN.
__device__ __forceinline__ float offset_of(float m, float c) {
  const float x = m * c;
  return m == -INFINITY ? 0.f : x + (x - x);
}

// One tile of one row (a thread each): the row of scores at tensor-memory address t_s becomes P there, m and l and, where
// the maximum has risen, the row of O at t_o follow.  masked: keys whose bit in w is 0 do not count.  Arrives on `part`
// when three quarters of P are written (its product starts while the last quarter is computed).
// A row that is not valid (past the tile's last, where shared memory holds anything) has no say in when the warp rescales:
// equal calls round alike.
// The scores are read twice, for the maximum and for the exponentials: a row of 128 in registers leaves too few of
// the 168 a thread has for the rest, and what then goes through local memory costs more than the second read.
__device__ __forceinline__ void softmax_tile(uint32_t t_s, uint32_t t_o, bool masked, const uint32_t (&w)[4], float c,
                                             int npv, bool first, bool valid, float& m, float& l, uint64_t* part,
                                             int lane) {
  float m4[4] = {m, m, m, m};  // four chains
  if (masked) {  // -inf replaces the scores that do not count, here and for the second read
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t r[32];
      tmem_ld_cols(t_s + 32 * k, r);
#pragma unroll
      for (int j = 0; j < 32; ++j) r[j] = (w[k] >> j) & 1u ? r[j] : 0xFF800000u;
      tmem_st_32x32b_x32(t_s + 32 * k, r);
#pragma unroll
      for (int j = 0; j < 32; j += 2)
        m4[(j >> 1) & 3] = max3(m4[(j >> 1) & 3], __uint_as_float(r[j]), __uint_as_float(r[j + 1]));
    }
    tmem_st_wait();
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t r0[32], r1[32];
      tmem_ld_32x32b_x32(t_s + 64 * h, r0);
      tmem_ld_32x32b_x32(t_s + 64 * h + 32, r1);
      tmem_ld_wait_regs(r0);
      reg_order(r1);
#pragma unroll
      for (int j = 0; j < 32; ++j) m4[j & 3] = max3(m4[j & 3], __uint_as_float(r0[j]), __uint_as_float(r1[j]));
    }
  }
  const float mx = max3(m4[0], m4[1], max3(m4[2], m4[3], m4[3]));
  uint32_t sr[2][32];
  tmem_ld_32x32b_x32(t_s, sr[0]);
  if (first) {
    m = mx;
  } else if (__any_sync(0xffffffffu, valid && !((mx - m) * c <= kLazy))) {  // risen, or NaN
    const float f = mx == -INFINITY ? 1.f : ex2((m - mx) * c);
    m = mx;
    l *= f;
    // every product of the previous tile is complete: S of this tile was issued after it
    for (int cc = 0; cc < npv; cc += 16) {
      uint32_t o[16];
      tmem_ld_32x32b_x16(t_o + cc, o);
      tmem_ld_wait_regs(o);
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
      tmem_st_32x32b_x16(t_o + cc, o);
    }
  }
  const float mc = offset_of(m, c);
  const uint64_t c2 = pack2(c, c), nmc2 = pack2(-mc, -mc);
  uint64_t l2[4] = {0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t(&r)[32] = sr[k & 1];
    tmem_ld_wait_regs(r);
    if (k < 3) tmem_ld_32x32b_x32(t_s + 32 * (k + 1), sr[(k + 1) & 1]);  // ahead of this quarter's exponentials
    uint32_t pr[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float2 x = unpack2(fma2(pack2(r[2 * j], r[2 * j + 1]), c2, nmc2));
      const float2 e = (j & 3) == 3 ? ex2_poly(x) : make_float2(ex2(x.x), ex2(x.y));
      l2[j & 3] = add2(l2[j & 3], pack2(e.x, e.y));
      __nv_bfloat162 hv = __floats2bfloat162_rn(e.x, e.y);
      pr[j] = *(uint32_t*)&hv;
    }
    tmem_st_32x32b_x16(t_s + 16 * k, pr);  // over scores that are in registers by now
    if (k == 2) {
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(part);
    }
  }
  const float2 ls = unpack2(add2(add2(l2[0], l2[1]), add2(l2[2], l2[3])));
  l += ls.x + ls.y;
  tmem_st_wait();
}

__device__ __forceinline__ int raw_len(const AttnParams& p, int b) {
  if (!p.kv_len || !SVDQ_INB(p.status, 4ll * b, 4, 4ll * p.batch)) return p.sk;
  return __ldg(p.kv_len + b);
}

// Bits of the 128 keys of tile t that count (the same in every lane).
__device__ __forceinline__ void key_words(const AttnParams& p, int b, int t, int nkeys, int lane, uint32_t (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int key = t * kKeys + 32 * i + lane;
    bool on = key < nkeys;
    if (on && p.kv_mask) {
      const long long at = (long long)b * p.mask_ld + key;
      on = SVDQ_INB(p.status, at, 1, p.mask_extent) && p.kv_mask[at] != 0;
    }
    w[i] = __ballot_sync(0xffffffffu, on);
  }
}

// One work item: sample, item head, first token of stream 0, key tiles.
struct Item {
  int b, h, tok0, nkeys, t0, t1;
  bool second;  // PAIR: the second query tile has rows
};
// Walks a CTA's items without divisions (the step comes divided from the host), and with the length of the next item's
// sample already asked for: both would otherwise stand between two items' work.
struct Walk {
  int item, b, h, rt, len;
  __device__ __forceinline__ Walk(const AttnParams& p, int first) : item(first) {
    rt = first % p.row_tiles;
    const int bh = first / p.row_tiles;
    h = bh % p.heads_it;
    b = bh / p.heads_it;
    len = item < p.items ? raw_len(p, b) : 0;
  }
  __device__ __forceinline__ bool more(const AttnParams& p) const { return item < p.items; }
  template <int MODE>
  __device__ __forceinline__ Item get(const AttnParams& p, int split) const {
    constexpr bool PAIR = MODE == kPairs || MODE == kSplitPairs;
    Item it;
    it.b = b;
    it.h = h;
    it.tok0 = rt * p.tok_tile * (PAIR ? 2 : 1);
    it.nkeys = max(0, min(len, p.sk));
    const int n = (it.nkeys + kKeys - 1) / kKeys;
    if (MODE == kPairs) {
      it.t0 = 0;
      it.t1 = n;
    } else {
      const int per = (n + p.splits - 1) / p.splits;
      it.t0 = min(split * per, n);
      it.t1 = min(it.t0 + per, n);
    }
    it.second = PAIR && it.tok0 + p.tok_tile < p.sq;
    return it;
  }
  __device__ __forceinline__ void step(const AttnParams& p) {
    item += p.step;
    rt += p.step_rt;
    int c = rt >= p.row_tiles;
    rt -= c ? p.row_tiles : 0;
    h += p.step_h + c;
    c = h >= p.heads_it;
    h -= c ? p.heads_it : 0;
    b += p.step_b + c;
    if (item < p.items) len = raw_len(p, b);
  }
};

// Ring position (relative to the item's first) of stream s's tile in iteration i.
template <bool PAIR>
__device__ __forceinline__ int ring_pos(int i, int s, bool is_v, int n) {
  if (PAIR) return 2 * i + (is_v ? 1 : 0);
  const bool both = 2 * i + 1 < n;  // this iteration has a tile for each stream
  return 4 * i + (is_v ? (both ? 2 : 1) : 0) + s;
}

// softmax_tile for QUART: of the tile's keys only those of this warp's lane quarter.
__device__ __forceinline__ void softmax_quarter(uint32_t t_s, uint32_t t_o, int quarter, uint32_t w, float c, int npv,
                                                bool first, bool valid, float& m, float& l) {
  uint32_t r[32];
  tmem_ld_cols(t_s + 32 * quarter, r);
  float m4[4] = {m, m, m, m};
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    r[j] = (w >> j) & 1u ? r[j] : 0xFF800000u;
    m4[j & 3] = max3(m4[j & 3], m4[j & 3], __uint_as_float(r[j]));
  }
  const float mx = max3(m4[0], m4[1], max3(m4[2], m4[3], m4[3]));
  if (first) {
    m = mx;
  } else if (__any_sync(0xffffffffu, valid && !((mx - m) * c <= kLazy))) {  // risen, or NaN
    const float f = mx == -INFINITY ? 1.f : ex2((m - mx) * c);
    m = mx;
    l *= f;
    for (int cc = 0; cc < npv; cc += 16) {
      uint32_t o[16];
      tmem_ld_32x32b_x16(t_o + cc, o);
      tmem_ld_wait_regs(o);
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
      tmem_st_32x32b_x16(t_o + cc, o);
    }
  }
  const float mc = offset_of(m, c);
  uint32_t pr[16];
  float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float e0 = ex2(fmaf(__uint_as_float(r[2 * j]), c, -mc)), e1 = ex2(fmaf(__uint_as_float(r[2 * j + 1]), c, -mc));
    l4[j & 3] += e0 + e1;
    __nv_bfloat162 hv = __floats2bfloat162_rn(e0, e1);
    pr[j] = *(uint32_t*)&hv;
  }
  l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t z[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) z[j] = k == quarter ? pr[j] : 0u;
    tmem_st_32x32b_x16(t_s + 16 * k, z);
  }
  tmem_st_wait();
}

template <int MODE, int DC>
__global__ void __launch_bounds__(kThreads, 1) k_attn(const __grid_constant__ AttnMaps maps,
                                                      const __grid_constant__ AttnParams p) {
  using G = Geo<DC>;
  constexpr bool PAIR = MODE == kPairs || MODE == kSplitPairs, QUART = MODE == kQuarter;
  constexpr bool JOIN = MODE != kPairs;  // results of several CTAs or streams are joined at the end
  // Query tiles; key and value tiles in flight.  Where there is one query tile the ring has the other's place (2 x 24 heads
  // of one token over 4096 keys: 13.9 -> 13.2 us).
  constexpr int QT = PAIR ? 2 : 1, SLOTS = G::kSlots + 2 - QT;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sm_q = smem;                    // [QT][tile]
  uint8_t* sm_kv = smem + QT * G::kTile;   // [SLOTS][tile]
  uint8_t* sm_stage = sm_kv + SLOTS * G::kTile;      // [8][4 KiB]
  float* sm_m = (float*)sm_stage;                    // [2][128]
  float* sm_l = sm_m + 256;                          // [2][128]
  uint64_t* q_full = (uint64_t*)(sm_stage + G::kStage);  // [2]
  uint64_t* q_empty = q_full + 2;                    // [2]
  uint64_t* kv_full = q_empty + 2;                   // [SLOTS]
  uint64_t* kv_empty = kv_full + SLOTS;              // [SLOTS]
  uint64_t* v_fixed = kv_empty + SLOTS;              // [SLOTS]
  uint64_t* s_full = v_fixed + SLOTS;                // [2]
  uint64_t* p_full = s_full + 2;                     // [2]
  uint64_t* p_part = p_full + 2;                     // [2] three quarters of P are there
  uint64_t* o_full = p_part + 2;                     // [2]
  uint64_t* mma_done = o_full + 2;
  uint32_t* tmem_slot = (uint32_t*)(mma_done + 1);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  WaitCtl wc{abort_flag, p.status, p.limit};

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 4);  // one arrival per softmax warp of the stream
      mbar_init(&p_part[s], 4);
      mbar_init(&o_full[s], 1);
    }
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
      mbar_init(&v_fixed[s], 1);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // An earlier kernel that let this one start may still need tensor memory on this SM: allocate behind it.
  pdl_wait();
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;  // S0/P0 | S1/P1 | O0 | O1, 128 columns each

  const bool fixing = p.kv_len != nullptr || p.kv_mask != nullptr;
  const int split = JOIN && p.splits > 1 ? (int)cluster_ctarank() : 0;
  const int item0 = JOIN ? (int)blockIdx.x / p.splits : (int)blockIdx.x;
  const Walk only(p, item0);  // (JOIN) the CTA's item

  if (warp == 8) {
    // ------------------------------------------------------------ loads
    if (lane == 0) {
      prefetch_tmap(&maps.q);
      prefetch_tmap(&maps.k);
      prefetch_tmap(&maps.v);
      int pos = 0;       // ring position of the next tile
      int nq[2] = {0, 0};  // query tiles loaded per stream
      bool ok = true;
      auto load_kv = [&](const CUtensorMap* map, int head, int bat, int t) {
        const int s = pos % SLOTS;
        if (!timed_wait(&kv_empty[s], ((pos / SLOTS) & 1) ^ 1, wc)) return false;
        mbar_arrive_expect_tx(&kv_full[s], G::kTile);
#pragma unroll
        for (int ch = 0; ch < DC; ++ch)
          tma_load_4d(map, &kv_full[s], sm_kv + s * G::kTile + ch * kChunkBytes, 64 * ch, head, t * kKeys, bat);
        ++pos;
        return true;
      };
      constexpr int kCopies = QUART ? 4 : 1;
      const uint32_t q_bytes = (uint32_t)(kCopies * DC * 128 * p.group * p.tok_tile);
      for (Walk walk(p, item0); walk.more(p) && ok; walk.step(p)) {
        const Item it = walk.get<MODE>(p, split);
        const int n = it.t1 - it.t0;
        if (n == 0) continue;
        const int kvh = (int)((long long)it.h * p.group * p.hk / p.hq);
        for (int s = 0; s < (it.second ? 2 : 1) && ok; ++s) {
          if (!timed_wait(&q_empty[s], (nq[s] & 1) ^ 1, wc)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&q_full[s], q_bytes);
#pragma unroll
          for (int ch = 0; ch < DC; ++ch)
#pragma unroll
            for (int cp = 0; cp < kCopies; ++cp)
              tma_load_4d(&maps.q, &q_full[s], sm_q + s * G::kTile + ch * kChunkBytes + cp * 4096, 64 * ch,
                          it.h * p.group * p.q_hm, it.tok0 + s * p.tok_tile, it.b * p.q_bm);
          ++nq[s];
        }
        if (PAIR) {
          for (int t = it.t0; t < it.t1 && ok; ++t)
            ok = load_kv(&maps.k, kvh * p.k_hm, it.b * p.k_bm, t) && load_kv(&maps.v, kvh * p.v_hm, it.b * p.v_bm, t);
        } else {
          for (int t = it.t0; t < it.t1 && ok; t += 2) {
            const int two = t + 1 < it.t1 ? 2 : 1;
            for (int s = 0; s < two && ok; ++s) ok = load_kv(&maps.k, kvh * p.k_hm, it.b * p.k_bm, t + s);
            for (int s = 0; s < two && ok; ++s) ok = load_kv(&maps.v, kvh * p.v_hm, it.b * p.v_bm, t + s);
          }
        }
      }
      // No block leaves with copies in flight, whoever gave up on them.
      for (int j = (pos > SLOTS ? pos - SLOTS : 0); j < pos; ++j)
        mbar_wait_drain(&kv_full[j % SLOTS], (j / SLOTS) & 1, drain_limit(p.limit));
      for (int s = 0; s < 2; ++s)
        if (nq[s]) mbar_wait_drain(&q_full[s], (nq[s] - 1) & 1, drain_limit(p.limit));
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------ products
    if (elect_one()) {
      // An instruction keeps the tensor cores busy for 64 clocks, so issuing one has to cost less: descriptors are
      // one addition each.
      constexpr uint64_t kDescK = sdesc_const(16, 1024, LAYOUT_SW128), kDescV = sdesc_const(kChunkBytes, 1024, LAYOUT_SW128);
      const uint64_t q_desc = kDescK + sdesc_addr(sm_q), k_desc = kDescK + sdesc_addr(sm_kv);
      const uint64_t v_desc = kDescV + sdesc_addr(sm_kv);
      const uint32_t idesc_s = idesc_bf16_f32(kRows, kKeys);
      const uint32_t idesc_o = idesc_bf16_f32(kRows, p.npv) | (1u << 16);  // B (= V) has the head dimension contiguous
      int base = 0, fixes = 0;
      int nq[2] = {0, 0}, np[2] = {0, 0};
      bool ok = true;
      auto slot_wait = [&](int pos) {
        if (!timed_wait(&kv_full[pos % SLOTS], (pos / SLOTS) & 1, wc)) return false;
        tc_fence_after();
        return true;
      };
      auto issue_s = [&](int s, int pos) {
        const uint64_t qd = q_desc + (uint32_t)((PAIR ? s : 0) * (G::kTile >> 4));
        const uint64_t kd = k_desc + (uint32_t)((pos % SLOTS) * (G::kTile >> 4));
        const uint32_t d = tmem + s * 128;
#pragma unroll
        for (int kk = 0; kk < 4 * DC; ++kk) {
          if (kk >= p.ksteps) break;
          const uint32_t off = (uint32_t)(((kk >> 2) * kChunkBytes + (kk & 3) * 32) >> 4);
          mma_bf16(d, qd + off, kd + off, idesc_s, kk != 0 ? 1u : 0u);
        }
        umma_commit(&s_full[s]);
      };
      auto issue_o = [&](int s, int pos, int k0, int k1, bool first) {
        const uint64_t vd = v_desc + (uint32_t)((pos % SLOTS) * (G::kTile >> 4));
        const uint32_t d = tmem + 256 + s * 128, pa = tmem + s * 128;
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          if (kk >= k0 && kk < k1) mma_bf16_ts(d, pa + 8 * kk, vd + 128 * kk, idesc_o, first && kk == 0 ? 0u : 1u);
      };
      for (Walk walk(p, item0); walk.more(p) && ok; walk.step(p)) {
        const Item it = walk.get<MODE>(p, split);
        const int n = it.t1 - it.t0;
        if (n == 0) continue;
        const int iters = PAIR ? n : (n + 1) / 2;
        auto has = [&](int i, int s) { return PAIR ? (s == 0 || it.second) && i < n : 2 * i + s < n; };
        for (int s = 0; s < 2 && ok; ++s) {
          if (!has(0, s)) continue;
          if (PAIR || s == 0) {
            ok = timed_wait(&q_full[s], nq[s] & 1, wc);
            ++nq[s];
          }
          const int kp = base + ring_pos<PAIR>(0, s, false, n);
          ok = ok && slot_wait(kp);
          if (!ok) break;
          issue_s(s, kp);
          if (!PAIR || s == 1 || !it.second) umma_commit(&kv_empty[kp % SLOTS]);
          if (PAIR && n == 1) umma_commit(&q_empty[s]);
        }
        for (int i = 0; i < iters && ok; ++i) {
          for (int s = 0; s < 2 && ok; ++s) {
            if (!has(i, s)) continue;
            const int vp = base + ring_pos<PAIR>(i, s, true, n);
            const int kp = base + ring_pos<PAIR>(i + 1, s, false, n);
            const bool last_user = !PAIR || s == 1 || !it.second;
            if (!PAIR || s == 0) {
              ok = slot_wait(vp) && (!has(i + 1, s) || slot_wait(kp));
              if (ok && fixing) {
                ok = timed_wait(&v_fixed[fixes % SLOTS], (fixes / SLOTS) & 1, wc);
                ++fixes;
              }
            }
            ok = ok && timed_wait(&p_part[s], np[s] & 1, wc);
            if (!ok) break;
            tc_fence_after();
            issue_o(s, vp, 0, 6, i == 0);
            ok = timed_wait(&p_full[s], np[s] & 1, wc);
            if (!ok) break;
            ++np[s];
            tc_fence_after();
            issue_o(s, vp, 6, 8, false);
            if (has(i + 1, s)) {
              issue_s(s, kp);
              if (last_user) umma_commit(&kv_empty[kp % SLOTS]);
              if (PAIR && i + 2 == n) umma_commit(&q_empty[s]);
            } else {
              umma_commit(&o_full[s]);
            }
            if (last_user) umma_commit(&kv_empty[vp % SLOTS]);
          }
        }
        base += 2 * n;
      }
      umma_commit(mma_done);
      mbar_wait_drain(mma_done, 0, drain_limit(p.limit));
    }
  } else if (warp == 10) {
    // ------------------------------------------------------------ zero the masked rows of V
    // Where keys can be masked, every V tile passes through here, so that this warp neither runs ahead
    // of the ring nor falls behind it; rows past the last key of all are zeros already (the loads fill them).
    int base = 0, fixes = 0;
    bool ok = true;
    for (Walk walk(p, item0); walk.more(p) && ok && fixing; walk.step(p)) {
      const Item it = walk.get<MODE>(p, split);
      const int n = it.t1 - it.t0;
      for (int j = 0; j < n && ok; ++j) {
        const int t = it.t0 + j;
        uint32_t w[4];
        key_words(p, it.b, t, it.nkeys, lane, w);
        const int pos = base + (PAIR ? ring_pos<PAIR>(j, 0, true, n) : ring_pos<PAIR>(j >> 1, j & 1, true, n));
        ok = warp_timed_wait(&kv_full[pos % SLOTS], (pos / SLOTS) & 1, wc);
        if (!ok) break;
        uint8_t* tile = sm_kv + (pos % SLOTS) * G::kTile + lane * 16;
        if ((w[0] & w[1] & w[2] & w[3]) != 0xffffffffu) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t mine = w[i] >> (lane >> 3);  // four rows at a time, eight lanes to a row's 128 bytes
#pragma unroll
            for (int r = 0; r < 32; r += 4) {
              if (!((mine >> r) & 1u)) {
#pragma unroll
                for (int ch = 0; ch < DC; ++ch)
                  *(uint4*)(tile + ch * kChunkBytes + (32 * i + r) * 128) = make_uint4(0, 0, 0, 0);
              }
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_fixed[fixes % SLOTS]);
        ++fixes;
      }
      base += 2 * n;
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax and output
    const int st = warp >> 2, quarter = warp & 3;
    const int row = 32 * quarter + lane;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const uint32_t t_s = tmem + lanes + st * 128, t_o = tmem + lanes + 256 + st * 128;
    const int r_tok = (QUART ? lane : row) / p.group, r_head = (QUART ? lane : row) - r_tok * p.group;
    int ns = 0, no = 0;
    bool ok = true;
    for (Walk walk(p, item0); walk.more(p) && ok;) {
      const Item it = walk.get<MODE>(p, split);
      walk.step(p);
      const int n = it.t1 - it.t0;
      if (PAIR && st == 1 && !it.second) continue;
      const int tok = it.tok0 + (PAIR ? st * p.tok_tile : 0) + r_tok;
      const bool valid = r_tok < p.tok_tile && tok < p.sq;
      const bool warp_valid = __any_sync(0xffffffffu, valid);
      const int my = PAIR ? n : (n - st + 1) / 2;  // tiles of this stream
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < my && ok; ++i) {
        const int t = it.t0 + (PAIR ? i : 2 * i + st);
        const bool masked = p.kv_mask || it.nkeys < (t + 1) * kKeys;
        uint32_t w[4] = {0, 0, 0, 0};
        if (masked) key_words(p, it.b, t, it.nkeys, lane, w);
        ok = warp_timed_wait(&s_full[st], ns & 1, wc);
        if (!ok) break;
        ++ns;
        tc_fence_after();
        if (warp_valid) {
          if constexpr (QUART) {
            const uint32_t wq = masked ? (quarter & 2 ? (quarter & 1 ? w[3] : w[2]) : (quarter & 1 ? w[1] : w[0])) : ~0u;
            softmax_quarter(t_s, t_o, quarter, wq, p.c, p.npv, i == 0, valid, m, l);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_part[st]);
          } else {
            softmax_tile(t_s, t_o, masked, w, p.c, p.npv, i == 0, valid, m, l, &p_part[st], lane);
          }
        } else {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_part[st]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[st]);
      }
      if (!JOIN) {
        if (!ok) break;
        if (n > 0) {
          ok = warp_timed_wait(&o_full[st], no & 1, wc);
          if (!ok) break;
          ++no;
          tc_fence_after();
        }
        if (warp_valid) {
          const float inv = l == 0.f ? 0.f : __fdividef(1.f, l);  // a row without a key: 0
          uint8_t* mine = sm_stage + warp * 4096;
          // A thread has a row, but rows lie far apart in memory: 64 columns of the warp's 32 rows go through shared
          // memory (16-byte pieces, swizzled by the row) and from there as whole 128-byte lines.
          const bool empty = __any_sync(0xffffffffu, l == 0.f);
          for (int cc = 0; cc < p.npv; cc += 64) {
            if (p.o_tma && lane == 0) bulk_wait_read<0>();  // the store before has read its source
            __syncwarp();
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              uint32_t o[32];
              if (n > 0) tmem_ld_cols(t_o + cc + 32 * hh, o);
              if (empty) {  // whatever O holds there
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = l == 0.f ? 0u : o[j];
              }
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                uint32_t y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  __nv_bfloat162 hv = __floats2bfloat162_rn(__uint_as_float(o[8 * v + 2 * j]) * inv,
                                                            __uint_as_float(o[8 * v + 2 * j + 1]) * inv);
                  y[j] = *(uint32_t*)&hv;
                }
                *(uint4*)(mine + lane * 128 + ((4 * hh + v) ^ (lane & 7)) * 16) = make_uint4(y[0], y[1], y[2], y[3]);
              }
            }
            if (p.o_tma) {
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {  // rows past the last token and columns past dim are clipped
                tma_store_4d(&maps.o, mine, cc, it.h * p.group, tok, it.b);
                bulk_commit();
              }
            } else {
              __syncwarp();
              const long long off = (long long)it.b * p.o_sb + (long long)tok * p.o_st +
                                    (long long)(it.h * p.group + r_head) * p.o_sh;
              const uint32_t rows_on = __ballot_sync(0xffffffffu, valid);
              const int col = cc + 8 * (lane & 7);
              for (int i = 0; i < 8; ++i) {
                const int r = 4 * i + (lane >> 3);
                const long long at = __shfl_sync(0xffffffffu, off, r) + col;
                const uint4 y = *(const uint4*)(mine + r * 128 + ((lane & 7) ^ (r & 7)) * 16);
                if (col < p.d && (rows_on >> r) & 1u && SVDQ_INB(p.status, 2 * at, 16, p.out_extent))
                  *(uint4*)(p.out + at) = y;
              }
              __syncwarp();
            }
          }
          tc_fence_before();  // these loads come before the products that the next P lets start
        }
      } else {
        // Parts to be joined: rows of O, not normalised, with m and l, in the place of the query and key tiles (every
        // product of both streams is complete).
        for (int s = 0; s < 2 && ok; ++s)
          if (PAIR ? n > 0 && (s == 0 || it.second) : s < n) ok = warp_timed_wait(&o_full[s], 0, wc);
        if (!ok) break;
        tc_fence_after();
        if (warp_valid) {
          const int pr = QUART ? (st * 4 + quarter) * 32 + lane : st * 128 + row;
          float* part = (float*)smem + pr * G::kPartLd;
          if (valid) {
            sm_m[pr] = m;
            sm_l[pr] = l;
          }
          for (int cc = 0; cc < p.npv; cc += 32) {
            uint32_t o[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = 0;
            if (my > 0) tmem_ld_cols(t_o + cc, o);
            if (valid) {
#pragma unroll
              for (int v = 0; v < 8; ++v)
                *(uint4*)(part + cc + 4 * v) = make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
            }
          }
        }
      }
    }
  }

  if (!JOIN && p.o_tma && warp < 8 && lane == 0) bulk_wait<0>();
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (JOIN) {
    // Join of the CTA's parts, four columns of a row to a thread, then of the cluster's CTAs, which share the rows out.
    // (Pairs of tiles: a part for each row, and only the second step.)
    constexpr int NP = QUART ? 8 : 2, RP = QUART ? 32 : 128;
    const bool good = *abort_flag == 0;
    const int tok0 = only.rt * p.tok_tile * (PAIR ? 2 : 1);
    const int per_row = p.d / 4, tile_rows = p.tok_tile * p.group;
    const int total = min(p.tok_tile * (PAIR ? 2 : 1), p.sq - tok0) * p.group * per_row;
    float* part = (float*)smem;
    float* fm = PAIR ? sm_m : (float*)(sm_stage + 2048);  // [128] of the CTA (PAIR: [256])
    float* fl = PAIR ? sm_l : fm + 128;
    auto store = [&](int row, int col, const float (&o)[4], float ll) {
      const float inv = 1.f / ll;
      uint32_t y[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        __nv_bfloat162 hv = __floats2bfloat162_rn(o[2 * j] * inv, o[2 * j + 1] * inv);
        y[j] = ll == 0.f ? 0u : *(uint32_t*)&hv;
      }
      const int tok = tok0 + row / p.group, head = only.h * p.group + row % p.group;
      const long long off = (long long)only.b * p.o_sb + (long long)tok * p.o_st + (long long)head * p.o_sh + col;
      if (SVDQ_INB(p.status, 2 * off, 8, p.out_extent)) *(uint2*)(p.out + off) = make_uint2(y[0], y[1]);
    };
    if (!PAIR && good) {
      for (int u = threadIdx.x; u < total; u += kThreads) {
        const int row = u / per_row, col = (u - row * per_row) * 4;
        float f[NP], mm = -INFINITY, ll = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          f[k] = sm_m[k * RP + row];
          mm = fmaxf(mm, f[k]);
        }
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          const float4 x = *(const float4*)(part + (k * RP + row) * G::kPartLd + col);
          f[k] = f[k] == -INFINITY ? 0.f : ex2((f[k] - mm) * p.c);
          ll = fmaf(sm_l[k * RP + row], f[k], ll);
          o[0] = fmaf(x.x, f[k], o[0]);
          o[1] = fmaf(x.y, f[k], o[1]);
          o[2] = fmaf(x.z, f[k], o[2]);
          o[3] = fmaf(x.w, f[k], o[3]);
        }
        if (p.splits == 1) {
          store(row, col, o, ll);
        } else {  // over the first part, whose place no other thread reads
          *(float4*)(part + row * G::kPartLd + col) = make_float4(o[0], o[1], o[2], o[3]);
          if (col == 0) {
            fm[row] = mm;
            fl[row] = ll;
          }
        }
      }
    }
    if (p.splits > 1) {
      // Rows split, split + splits, ... are this CTA's: first the weights of their parts (2^(c (m_r - m)) / l, so that
      // the sums need one load an element and part), then the sums, four elements to a thread at once.
      float* weight = (float*)(sm_stage + 4096);  // [row of this CTA][kMaxSplit]; the first is -1 for a row without a key
      const int rows = total / per_row, mine = (rows - split + p.splits - 1) / p.splits;
      const uint32_t a_part = smem_u32(part), a_m = smem_u32(fm), a_l = smem_u32(fl);
      auto place = [&](int row) { return PAIR && row >= tile_rows ? row - tile_rows + 128 : row; };  // of a row's part
      if (!good) {  // an expired wait: this CTA stores nothing, and the others' rows become NaN
        for (int i = threadIdx.x; i < (PAIR ? 256 : 128); i += kThreads) fm[i] = fl[i] = __int_as_float(0x7FC00000);
      }
      cluster_sync();
      if (good) {
        for (int i = threadIdx.x; i < mine; i += kThreads) {
          const int at = place(i * p.splits + split);
          float fr[kMaxSplit], lr[kMaxSplit], mm = -INFINITY, ll = 0.f;
#pragma unroll
          for (int r = 0; r < kMaxSplit; ++r) {  // all asked for before the first is used
            fr[r] = r < p.splits ? dsmem_ld_f32(dsmem_addr(a_m + 4 * at, r)) : -INFINITY;
            lr[r] = r < p.splits ? dsmem_ld_f32(dsmem_addr(a_l + 4 * at, r)) : 0.f;
          }
#pragma unroll
          for (int r = 0; r < kMaxSplit; ++r) mm = fmaxf(mm, fr[r]);
#pragma unroll
          for (int r = 0; r < kMaxSplit; ++r) {
            fr[r] = fr[r] == -INFINITY ? 0.f : ex2((fr[r] - mm) * p.c);
            ll = fmaf(lr[r], fr[r], ll);
          }
          const float inv = 1.f / ll;
#pragma unroll
          for (int r = 0; r < kMaxSplit; ++r) weight[i * kMaxSplit + r] = ll == 0.f ? -1.f : fr[r] * inv;
        }
      }
      __syncthreads();
      if (good) {
        constexpr int U = QUART ? 1 : 4, B = QUART ? kMaxSplit : 2;  // elements, and parts of each, asked for at once
        for (int u0 = threadIdx.x; u0 < mine * per_row; u0 += U * kThreads) {
          int row[U], col[U], i[U];
          uint32_t from[U];
          float4 o[U];
#pragma unroll
          for (int j = 0; j < U; ++j) {
            const int u = min(u0 + j * kThreads, mine * per_row - 1);
            i[j] = u / per_row;
            col[j] = (u - i[j] * per_row) * 4;
            row[j] = i[j] * p.splits + split;
            from[j] = a_part + (uint32_t)(place(row[j]) * G::kPartLd + col[j]) * 4;
            o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
          }
          for (int r0 = 0; r0 < p.splits; r0 += B) {
            float4 x[B][U];
#pragma unroll
            for (int r = 0; r < B; ++r)
#pragma unroll
              for (int j = 0; j < U; ++j)
                if (r0 + r < p.splits) x[r][j] = dsmem_ld_f32x4(dsmem_addr(from[j], r0 + r));
#pragma unroll
            for (int r = 0; r < B; ++r) {
              if (r0 + r >= p.splits) break;
#pragma unroll
              for (int j = 0; j < U; ++j) {
                const float f = weight[i[j] * kMaxSplit + r0 + r];
                o[j].x = fmaf(x[r][j].x, f, o[j].x);
                o[j].y = fmaf(x[r][j].y, f, o[j].y);
                o[j].z = fmaf(x[r][j].z, f, o[j].z);
                o[j].w = fmaf(x[r][j].w, f, o[j].w);
              }
            }
          }
#pragma unroll
          for (int j = 0; j < U; ++j) {
            const float y[4] = {o[j].x, o[j].y, o[j].z, o[j].w};
            if (u0 + j * kThreads < mine * per_row)
              store(row[j], col[j], y, weight[i[j] * kMaxSplit] < 0.f ? 0.f : 1.f);
          }
        }
      }
      cluster_sync();  // a CTA's shared memory stays until every other has read it
    }
  }
}

// Once per device: the shared-memory attribute (it belongs to the kernel on each device), and how many clusters of each
// size are resident at once (a cluster lies inside one GPC, so that 148 SMs hold 15 clusters of 8, not 18).
struct DeviceFit {
  bool set = false;
  int clusters[kMaxSplit + 1] = {};
};
template <int MODE, int DC>
const DeviceFit* device_fit(int dev) {
  static std::mutex mu;
  static DeviceFit fits[64];
  if (dev < 0 || dev >= 64) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  DeviceFit& f = fits[dev];
  if (!f.set) {
    const auto kern = k_attn<MODE, DC>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Geo<DC>::kSmem) != cudaSuccess)
      return nullptr;
    for (int c = 2; MODE != kPairs && c <= kMaxSplit; ++c) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)(148 * c));
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = Geo<DC>::kSmem;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = (unsigned)c;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&f.clusters[c], kern, &cfg) != cudaSuccess) {
        cudaGetLastError();
        f.clusters[c] = 0;
      }
    }
    f.set = true;
  }
  return &f;
}

template <int MODE, int DC>
int launch(const AttnMaps& maps, const AttnParams& p, cudaStream_t stream) {
  const int grid = MODE == kPairs ? p.step : p.items * p.splits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Geo<DC>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_attn<MODE, DC>, maps, p) == cudaSuccess ? SVDQ_OK : SVDQ_ERR_CUDA;
}

template <int DC>
const DeviceFit* device_fit(int mode, int dev) {
  return mode == kPairs        ? device_fit<kPairs, DC>(dev)
         : mode == kSplitPairs ? device_fit<kSplitPairs, DC>(dev)
         : mode == kSingle     ? device_fit<kSingle, DC>(dev)
                               : device_fit<kQuarter, DC>(dev);
}
template <int DC>
int launch(int mode, const AttnMaps& maps, const AttnParams& p, cudaStream_t stream) {
  return mode == kPairs        ? launch<kPairs, DC>(maps, p, stream)
         : mode == kSplitPairs ? launch<kSplitPairs, DC>(maps, p, stream)
         : mode == kSingle     ? launch<kSingle, DC>(maps, p, stream)
                               : launch<kQuarter, DC>(maps, p, stream);
}

// Mode and cluster size for so many tiles of query rows (over all samples and heads), pairs of them, and key tiles: the
// least of the modes' times, in tenths of a microsecond, as fitted to measurements with heads of 64 and 128, 24 to 1900
// tiles and 1 to 36 key tiles.  Measured, heads of 128 (one mode against the next best):
//   24 heads of 1000 tokens over 1024 keys (96 pairs, 192 tiles): pairs 19, single tiles 35 us
//   24 heads of 512 over 300 (48, 96): pairs 11, single 13;  over 4608: split pairs 43, single 51, pairs 65
//   24 heads of 128 over 4608 (24 tiles): single 22, pairs 58
struct Plan {
  int mode, splits;
};
int plan_of(Plan* plan, bool quart, bool wide, int64_t singles, int64_t pairs, int ktiles, int dev) {
  auto fit_of = [&](int mode) { return wide ? device_fit<2>(mode, dev) : device_fit<1>(mode, dev); };
  const int64_t sms = device_sm_count(dev);
  int64_t best = INT64_MAX;
  auto consider = [&](int mode, int splits, int64_t cost) {
    if (cost >= best) return;
    best = cost;
    *plan = {mode, splits};
  };
  auto fold = [](int64_t n, int64_t by) { return (n + by - 1) / by; };
  if (!quart) {
    const DeviceFit* f = fit_of(kSplitPairs);
    if (!f || !fit_of(kPairs)) return SVDQ_ERR_CUDA;
    const int tile = singles > pairs ? 17 : (wide ? 15 : 12);  // of keys; a pair's only tile is faster
    consider(kPairs, 1, 40 + fold(pairs, sms) * (10 + tile * ktiles));
    for (int c = 2; c <= kMaxSplit && 2 * c <= ktiles; ++c)
      if (pairs <= f->clusters[c]) consider(kSplitPairs, c, 128 + tile * fold(ktiles, c));
  }
  const int mode = quart ? kQuarter : kSingle;
  const DeviceFit* f = fit_of(mode);
  if (!f) return SVDQ_ERR_CUDA;
  const int fixed = wide ? 88 : 65, round = wide ? 23 : 15;  // round: two key tiles, one to a stream
  consider(mode, 1, fold(singles, sms) * (fixed + round * fold(ktiles, 2)));
  for (int c = 2; c <= kMaxSplit && 2 * c <= ktiles; ++c)
    if (singles <= f->clusters[c]) consider(mode, c, fixed + (quart ? 0 : 30) + round * fold(ktiles, 2 * c));
  return SVDQ_OK;
}

// Tensor map of a [batch, tokens, heads, dim] view.  A dimension of size one, or one with
// stride 0 (broadcast), becomes a dimension of size one whose coordinate is always 0.
int heads_map(CUtensorMap* map, const svdq_heads& h, int64_t batch, int64_t tokens, int64_t heads, int64_t dim,
              uint32_t box_heads, uint32_t box_tokens, int* batch_mul, int* head_mul) {
  *batch_mul = batch > 1 && h.stride_batch != 0;
  *head_mul = heads > 1 && h.stride_head != 0;
  const uint64_t any = (uint64_t)((dim * 2 + 15) / 16 * 16);
  const uint64_t dims[4] = {(uint64_t)dim, *head_mul ? (uint64_t)heads : 1, (uint64_t)tokens,
                            *batch_mul ? (uint64_t)batch : 1};
  const uint64_t strides[3] = {*head_mul ? (uint64_t)h.stride_head * 2 : any,
                               tokens > 1 ? (uint64_t)h.stride_token * 2 : any,
                               *batch_mul ? (uint64_t)h.stride_batch * 2 : any};
  const uint32_t box[4] = {64, box_heads, box_tokens, 1};
  return encode_tmap_4d_bf16(map, h.data, dims, strides, box);
}

}  // namespace

int check_heads(const svdq_heads& h, int64_t batch, int64_t tokens, int64_t heads, int64_t dim, bool out) {
  if (!h.data || ((uintptr_t)h.data & 15)) return SVDQ_ERR_INVALID_ARG;
  const int64_t size[3] = {batch, tokens, heads};
  const int64_t stride[3] = {h.stride_batch, h.stride_token, h.stride_head};
  int64_t span = dim;
  for (int i = 0; i < 3; ++i) {
    if (size[i] <= 1) continue;
    if (stride[i] < 0 || stride[i] % 8 != 0 || stride[i] > ((int64_t)1 << 38)) return SVDQ_ERR_INVALID_ARG;
    if (stride[i] == 0 && (out || i == 1)) return SVDQ_ERR_INVALID_ARG;
    if (stride[i] != 0 && stride[i] < dim) return SVDQ_ERR_INVALID_ARG;  // elements of two places overlap
    span += (size[i] - 1) * stride[i];
    if (span > ((int64_t)1 << 40)) return SVDQ_ERR_INVALID_ARG;
  }
  // No two places of an output are the same memory: in the order of the strides, each steps over all the ones below it.
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int i, int j) { return stride[i] < stride[j]; });
  int64_t below = dim;
  for (int i : order) {
    if (!out || size[i] <= 1) continue;
    if (stride[i] < below) return SVDQ_ERR_INVALID_ARG;
    below += (size[i] - 1) * stride[i];
  }
  return SVDQ_OK;
}
int64_t heads_extent(const svdq_heads& h, int64_t batch, int64_t tokens, int64_t heads, int64_t dim) {
  int64_t span = dim;
  if (batch > 1) span += (batch - 1) * h.stride_batch;
  if (tokens > 1) span += (tokens - 1) * h.stride_token;
  if (heads > 1) span += (heads - 1) * h.stride_head;
  return 2 * span;
}

}  // namespace svdq

using namespace svdq;

extern "C" svdq_status svdq_cross_attn(const svdq_attn_args* a, int32_t* status, void* stream) {
  if (!a || !status || ((uintptr_t)status & 3)) return SVDQ_ERR_INVALID_ARG;
  const int64_t lim = (int64_t)1 << 30;
  if (a->batch < 0 || a->q_tokens < 0 || a->kv_tokens < 0 || a->batch > lim || a->q_tokens > lim || a->kv_tokens > lim)
    return SVDQ_ERR_INVALID_ARG;
  if (a->heads < 1 || a->kv_heads < 1 || a->heads > 4096 || a->heads % a->kv_heads != 0) return SVDQ_ERR_INVALID_ARG;
  if (a->dim < 8 || a->dim > 128 || a->dim % 8 != 0) return SVDQ_ERR_INVALID_ARG;
  if (!(a->scale > 0.f) || !std::isfinite(a->scale * kLog2E)) return SVDQ_ERR_INVALID_ARG;
  if (a->batch == 0 || a->q_tokens == 0) return SVDQ_OK;
  int st = check_heads(a->o, a->batch, a->q_tokens, a->heads, a->dim, true);
  if (st == SVDQ_OK) st = check_heads(a->q, a->batch, a->q_tokens, a->heads, a->dim, false);
  if (st != SVDQ_OK) return (svdq_status)st;
  // without a key there is nothing to read, and the maps below need a valid tensor: stand in the queries
  const svdq_heads& kh = a->kv_tokens > 0 ? a->k : a->q;
  const svdq_heads& vh = a->kv_tokens > 0 ? a->v : a->q;
  if (a->kv_tokens > 0) {
    st = check_heads(a->k, a->batch, a->kv_tokens, a->kv_heads, a->dim, false);
    if (st == SVDQ_OK) st = check_heads(a->v, a->batch, a->kv_tokens, a->kv_heads, a->dim, false);
    if (st != SVDQ_OK) return (svdq_status)st;
  }
  if (a->o.data == a->q.data || (a->kv_tokens > 0 && (a->o.data == a->k.data || a->o.data == a->v.data)))
    return SVDQ_ERR_INVALID_ARG;
  if (a->kv_mask && a->batch > 1 && a->mask_stride < 0) return SVDQ_ERR_INVALID_ARG;
  if (((uintptr_t)a->kv_len & 3)) return SVDQ_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return SVDQ_ERR_UNSUPPORTED_DEVICE;
  }
  svdq_status sd = svdq_device_check(dev);
  if (sd != SVDQ_OK) return sd;
  const void* ptrs[7] = {a->q.data, kh.data, vh.data, a->o.data, a->kv_len, a->kv_mask, status};
  for (const void* ptr : ptrs)
    if (ptr && check_blob_pointer(ptr, dev) != SVDQ_OK) return SVDQ_ERR_INVALID_ARG;

  AttnParams p{};
  p.sq = (int)a->q_tokens;
  p.sk = (int)a->kv_tokens;
  p.hq = (int)a->heads;
  p.hk = (int)a->kv_heads;
  p.d = (int)a->dim;
  p.batch = (int)a->batch;
  const int share = p.hq / p.hk;
  // Query heads of one key head go into the rows of one tile; a broadcast query head, or more
  // of them than a tile has rows, is taken head by head.
  p.group = share <= kRows && (share == 1 || a->q.stride_head != 0) ? share : 1;
  // Few rows: one tile, held by each of its lane quarters.
  const bool quart = p.group <= 32 && (int64_t)p.sq * p.group <= 32;
  p.tok_tile = (quart ? 32 : kRows) / p.group;
  p.heads_it = p.hq / p.group;
  p.ksteps = (p.d + 15) / 16;
  p.npv = p.ksteps * 16;
  p.c = a->scale * kLog2E;
  p.kv_len = a->kv_len;
  p.kv_mask = a->kv_mask;
  p.mask_ld = a->batch > 1 ? a->mask_stride : 0;
  p.mask_extent = (a->batch - 1) * p.mask_ld + a->kv_tokens;
  p.out = (uint16_t*)a->o.data;
  p.o_sb = a->o.stride_batch;
  p.o_st = a->o.stride_token;
  p.o_sh = a->o.stride_head;
  p.out_extent = heads_extent(a->o, a->batch, a->q_tokens, a->heads, a->dim);
  p.status = status;
  p.limit = wait_limit_cycles();

  const int sms = device_sm_count(dev);
  const int64_t bh = (int64_t)p.batch * p.heads_it;
  const int64_t tiles = ((int64_t)p.sq + p.tok_tile - 1) / p.tok_tile;
  const int64_t pairs = (tiles + 1) / 2;
  if (bh * tiles > ((int64_t)1 << 30)) return SVDQ_ERR_INVALID_ARG;
  const bool wide = p.d > 64;
  Plan plan{};
  if (int e = plan_of(&plan, quart, wide, bh * tiles, bh * pairs, (p.sk + kKeys - 1) / kKeys, dev)) return (svdq_status)e;
  const bool pair = plan.mode == kPairs || plan.mode == kSplitPairs;
  p.splits = plan.splits;
  p.row_tiles = (int)(pair ? pairs : tiles);
  p.items = (int)(bh * p.row_tiles);
  p.step = plan.mode == kPairs && p.items > sms ? sms : p.items;  // kPairs: persistent CTAs; else one item to a cluster
  p.step_rt = p.step % p.row_tiles;
  p.step_h = p.step / p.row_tiles % p.heads_it;
  p.step_b = p.step / p.row_tiles / p.heads_it;

  AttnMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  int st_q = heads_map(&maps.q, a->q, a->batch, a->q_tokens, a->heads, a->dim, (uint32_t)p.group,
                       (uint32_t)p.tok_tile, &p.q_bm, &p.q_hm);
  const int64_t kt = a->kv_tokens > 0 ? a->kv_tokens : 1;
  int st_k = heads_map(&maps.k, kh, a->batch, kt, a->kv_heads, a->dim, 1, kKeys, &p.k_bm, &p.k_hm);
  if (plan.mode == kPairs && 32 % p.group == 0) {
    int bm = 0, hm = 0;
    p.o_tma = 1;
    if (heads_map(&maps.o, a->o, a->batch, a->q_tokens, a->heads, a->dim, (uint32_t)p.group, (uint32_t)(32 / p.group), &bm,
                  &hm) != SVDQ_OK)
      return SVDQ_ERR_CUDA;
  }
  int st_v = heads_map(&maps.v, vh, a->batch, kt, a->kv_heads, a->dim, 1, kKeys, &p.v_bm, &p.v_hm);
  if (st_q != SVDQ_OK || st_k != SVDQ_OK || st_v != SVDQ_OK) return SVDQ_ERR_CUDA;

  NvtxRange range("svdq/cross_attn");
  const cudaStream_t s = (cudaStream_t)stream;
  return (svdq_status)(wide ? launch<2>(plan.mode, maps, p, s) : launch<1>(plan.mode, maps, p, s));
}
