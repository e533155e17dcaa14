// The softmax of the tensor-core attention kernels: one query row per thread, its 128 logits
// of a block in TMEM, probabilities written over them as pairs of bf16 (the prompts' kernel)
// or of f16 (the 4-bit cache's, whose references are its own).
//
// In the prompts' kernel the reference m of a row is the maximum of some of its first logits and stays
// while the row's sum is below kBig: a common factor of P, O and the sum costs no precision (bf16
// and fp32 have the same exponents) and the final division removes it.  So a block has no
// maximum to find before its exponentials.  A block that passes the bound is done over with
// its maximum as the reference, O and the sum rescaled; S is still there, since P replaces it
// only after that test.
#pragma once

#include <cuda_fp16.h>

#include "tcgen.cuh"

namespace chunkkv {
namespace tcgen {

constexpr int kTile = 128;                        // query rows of a tile, keys of a block
constexpr float kBig = 16777216.f;                // bound of a row's sum under its reference
constexpr float kHuge = 4194304.f;                // references (in base-2 exponents) up to which one rounding will do

// What a row runs once per item or less is kept out of the loop over the blocks, in small
// loops of its own: at one pass an item, straight-line code costs its instruction fetches
// (an unrolled write of the output rows took 6000 cycles an item).

// -inf into the columns of S that the row does not see (those after `seen`), whatever
// they hold.  lo: what the warp's first row sees; columns up to there are left alone.
static __device__ __noinline__ void hide(uint32_t tS, int seen, int lo) {
#pragma unroll 1
  for (int c = max(lo + 1, 0) & ~31; c < kTile; c += 32) {
    float s[32];
    tmem_ld32(tS + c, s);
    tmem_wait(s);
#pragma unroll
    for (int i = 0; i < 32; ++i) s[i] = c + i <= seen ? s[i] : -INFINITY;
    tmem_st32(tS + c, s);
  }
  tmem_st_wait();
}
// Row maximum of S.
__device__ __forceinline__ float row_max(uint32_t tS) {
  float m = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < kTile; c += 32) {
    float s[32];
    tmem_ld32(tS + c, s);
    tmem_wait(s);
#pragma unroll
    for (int i = 0; i < 32; i += 2) m = fmaxf(m, fmaxf(s[i], s[i + 1]));
  }
  return m;
}
// A first reference: the maximum over the last 32 columns that all of the warp's rows
// reach into (any of a row's finite logits would do), or over all where a row has none
// there.
static __device__ __noinline__ float first_reference(uint32_t tS, int lo) {
  float m = -INFINITY;
  if (lo >= 0) {
    float s[32];
    tmem_ld32(tS + min(lo >> 5, 3) * 32, s);
    tmem_wait(s);
#pragma unroll
    for (int i = 0; i < 32; i += 2) m = fmaxf(m, fmaxf(s[i], s[i + 1]));
  }
  if (__any_sync(0xffffffffu, m == -INFINITY)) {
    const float all = row_max(tS);
    m = m == -INFINITY ? all : m;                             // a row's reference hangs on its own logits alone
  }
  return m;
}

// A pair of probabilities as it is written: bf16, or f16 (HALF).
template <bool HALF>
__device__ __forceinline__ uint32_t pack_p(float2 w) {
  if constexpr (HALF) {
    const __half2 h = __floats2half2_rn(w.x, w.y);
    return *(const uint32_t*)&h;
  } else {
    const __nv_bfloat162 b = __floats2bfloat162_rn(w.x, w.y);
    return *(const uint32_t*)&b;
  }
}

// 32 columns of P from 32 of S: pairs by one packed FMA, two exponentials, a packed sum
// and a packed conversion.
template <int C, bool HALF>
__device__ __forceinline__ void chunk_exp(const float (&s)[32], float2 a2, float2 n2, float2 (&sum)[2], uint32_t (&p)[64]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 e = __ffma2_rn(make_float2(s[2 * i], s[2 * i + 1]), a2, n2);
    const float2 w = make_float2(ex2(e.x), ex2(e.y));
    sum[i & 1] = __fadd2_rn(sum[i & 1], w);
    p[16 * C + i] = pack_p<HALF>(w);
  }
}
// A row's P under the reference -neg, and its sum.  Straight-line code: a branch per
// chunk cost 400 cycles of a block's 1000.
template <bool HALF = false>
__device__ __forceinline__ float row_exp(uint32_t tS, float alpha, float neg, uint32_t (&p)[64]) {
  float ra[32], rb[32];
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  const float2 a2 = make_float2(alpha, alpha), n2 = make_float2(neg, neg);
  tmem_ld32(tS, ra);
  tmem_wait(ra);
  tmem_ld32(tS + 32, rb);
  chunk_exp<0, HALF>(ra, a2, n2, sum, p);
  tmem_wait(rb);
  tmem_ld32(tS + 64, ra);
  chunk_exp<1, HALF>(rb, a2, n2, sum, p);
  tmem_wait(ra);
  tmem_ld32(tS + 96, rb);
  chunk_exp<2, HALF>(ra, a2, n2, sum, p);
  tmem_wait(rb);
  chunk_exp<3, HALF>(rb, a2, n2, sum, p);
  return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

// The same of (S - base) alpha + neg, with P written: its 16 columns of 32 logits lie among the columns read by then.
// The terms are added in row_exp's order: a row that is here only because another of its warp is keeps its bits.
template <bool HALF = false>
__device__ __forceinline__ float write_exp_from(uint32_t tS, float base, float alpha, float neg) {
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    float s[32];
    tmem_ld32(tS + 32 * c, s);
    tmem_wait(s);
    uint32_t p[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 w = make_float2(ex2(fmaf(s[2 * i] - base, alpha, neg)), ex2(fmaf(s[2 * i + 1] - base, alpha, neg)));
      sum[i & 1] = __fadd2_rn(sum[i & 1], w);
      p[i] = pack_p<HALF>(w);
    }
    tmem_st16(tS + 16 * c, p);
  }
  return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

// -m alpha, as row_exp takes it; NaN for a huge reference, so that the sums of its blocks are and block_again does them.
__device__ __forceinline__ float offset_of(float m, float alpha) {
  const float neg = -m * alpha;
  return fabsf(neg) <= kHuge ? neg : NAN;
}
// What the rounding of -m alpha took from a row's reference: its terms are 2^(S alpha - (m alpha - residual)).  Terms
// under two references are comparable only with it (near kHuge -m alpha is rounded to multiples of 1/4).
__device__ __forceinline__ float residual(float m, float alpha) {
  const float neg = offset_of(m, alpha);
  return neg == neg ? fmaf(m, alpha, neg) : 0.f;
}

// A block whose sum passed the bound, or whose reference is huge, done over: rows that are `over` move their
// reference to the block's maximum, and what O (at tO, unless it is still empty) and l
// hold goes with it.  Under a huge reference S alpha - m alpha in one rounding is off by
// more than an exponential bears (half a unit of m alpha in its last place), so there the
// difference comes first.  Returns (m, -m alpha, l); P is written.
template <int D>
static __device__ __noinline__ float3 block_again(uint32_t tS, uint32_t tO, float alpha, float m, float l, bool over) {
  const float bm = row_max(tS);
  const float mn = fmaxf(m, bm);
  float f = 1.f;
  if (over) {
    f = m == -INFINITY ? 0.f : ex2((m - mn) * alpha - residual(m, alpha) + residual(mn, alpha));
    m = mn;
  }
  const float neg = m == -INFINITY ? 0.f : offset_of(m, alpha);
  if (tO != 0xFFFFFFFFu) {
    // the blocks before are done: their products were issued before this S
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      float o[32];
      tmem_ld32(tO + 32 * c, o);
      tmem_wait(o);
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] *= f;
      tmem_st32(tO + 32 * c, o);
    }
  }
  const bool huge = neg != neg;
  const float sum = write_exp_from(tS, huge ? m : 0.f, alpha, huge ? 0.f : neg);
  return make_float3(m, neg, l * f + sum);
}

// Eight output columns as they are written, to a 16-byte piece.
__device__ __forceinline__ void put8(uint8_t* piece, const float* o) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(o[2 * e], o[2 * e + 1]);
    w[e] = *(const uint32_t*)&b;
  }
  *(uint4*)piece = make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace tcgen
}  // namespace chunkkv
