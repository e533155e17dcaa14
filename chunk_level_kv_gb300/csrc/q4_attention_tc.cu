// Attention of many query rows over the 4-bit paged cache on the tensor cores (tcgen05 + TMA +
// TMEM): bf16, head dimension up to 128.
//
//   O_i = sum_{j < n - m + 1 + i} softmax_j(scale q_i . k_j) v_j,   k_j and v_j = s c + m
//
// for the m query tokens at the end of a cache row of n tokens.  The products, the tiles and the
// order of work are those of the attention over packed prompts (prefill_tc.cu): two tiles of 128
// query rows (the gp query heads of a KV head at 128 / gp consecutive positions) against blocks of
// 128 keys from the last one down, S and O in TMEM, one thread per row.  What differs:
//
// - Operands are f16 (11 bits; in bf16 the rounding of the keys, the values and the weights made
//   the output's error 3 times that of its own rounding).  f16's range is kept by powers of two: a
//   query row is scaled by its largest element, a block's keys and its values by theirs (2^EK
//   and 2^EV; one warp looks them up in the pages' steps), so what a block holds below 2^-29 of its
//   largest value loses bits, and below 2^-40 is lost.  The scales leave again through the
//   exponent: a weight is P = 2^(S alpha 2^EK + EV - Z) with the row's reference Z, so O gathers
//   2^-Z V with every block's V at its own scale, and a block whose values are huge under
//   negligible weights costs the others nothing.
// - A block whose tokens' largest values lie more than 2^8 apart gets an exponent for each token, or
//   a large token that a row does not see, or weighs by nothing, would take the others' bits.  The row's
//   threads then weigh it column by column, in code of its own (block_apart: three times the time of a block).  So they do where EV
//   falls far below an earlier block's: weights that vanish beside Z still count in l.
// - A block's keys and values arrive as pages of codes (18 KB for 128 columns, bulk copies) and
//   eight converting warps expand them into the tensor cores' operands.  A word of 8 codes is 8
//   consecutive columns of a key, or 8 consecutive tokens of a value's column, which are 16
//   consecutive bytes of a K-major operand: V is stored as V^T, and both products take both
//   operands K-major.  1024 + c is an f16 number with c as its last bits; less 1024 it is c, and
//   one packed FMA makes s c + m of it, rounded once: 13 instructions for 8 codes.
// - The lengths are in device memory.  Work is counted in (two tiles, block) pairs; every CTA
//   takes an equal run of them (plan_run of decode.cuh), so that few rows against many keys
//   keep every SM busy.  Of query tiles whose keys are cut, the CTAs write parts (Z, l, O), and a
//   second launch joins them in order, 32 columns of 128 rows per CTA.
// - What a row must not see: S is set to -inf as for prompts.  A value can only be non-finite
//   as a group's m = NaN; where some row of the item does not see it, the converting warps
//   replace it by zero and note the first such token of each group of columns, and a row that
//   sees that token gets NaN there.
//
// A row's reference Z is a whole number near its first logits (plus EV, less kLift) and stays while
// a block's sum of weights is below kMost, which f16 holds; a block that passes it is done over
// from its own maximum.  The lift keeps weights down to 2^-18 of the reference's at full precision.
//
// What bounds it: no unit alone.  A block pair takes 2048 cycles of products and 3.8 thousand in all; issue slots are 55 % used
// and the tensor pipe 50 %.  Next to the exponentials of 256 rows the converting warps issue 3 thousand instructions for its
// 32768 codes, and a tile's softmax, 950 cycles alone, takes 1.9 thousand beside them; the twelve roles' loops share
// instruction caches (with 200 instructions more between them a block took 15 % longer).  Measured at 128 columns: 4001 queries
// on 16 to 17 thousand tokens of 28 / 4 heads 0.70 ms, 1.2 PFLOP/s of the visible pairs (2.3 ms if every block is
// block_apart's); 300 to 700 queries of two sequences on 4.9 to 9.7 thousand tokens of 32 / 8 heads 0.10 ms; 5 queries of
// eight sequences on 6.5 thousand 63 us.  At 128 columns the kernel spills 172 bytes a thread at its launch's 96 registers.
//
// Warp roles: 0-3 and 4-7 softmax of tile 0 and 1, 8 copies, 9 and 10 MMA issuers of tile 0 and 1,
// 11 scales, 12-19 conversion.  Every wait is bounded (tcgen.cuh); a CTA that gives up drains and exits.
#include <algorithm>

#include "decode.cuh"
#include "q4.cuh"
#include "tc_softmax.cuh"
#include "tensor_map.cuh"

namespace chunkkv {

int prefill_tc_heads(int G);                      // prefill_tc.cu

namespace {

using namespace tcgen;
using decode::Run;

constexpr int kStages = 4;                        // expanded K and V blocks (with three, the keys' conversion held the products up)
// Pages of codes, keys or values: what the rest leaves room for.  QT: tiles of a unit that hold queries; where few query
// tokens make one tile, the other's place holds more pages, and short turns wait less for their copies (26 thousand tokens
// of 64 rows: 199 -> 173 us).
template <int QT> constexpr int packed_pages() { return QT == 1 ? 14 : 7; }
constexpr int kItemRing = 2;
constexpr int kConvert = 8;                       // converting warps
constexpr int kThreads = 384 + 32 * kConvert;     // five warpgroups
constexpr int kLaunchRegs = 96, kSoftmaxRegs = 176, kOtherRegs = 40;
static_assert(256 * kSoftmaxRegs + (kThreads - 256) * kOtherRegs <= kThreads * kLaunchRegs, "register shares within the launch's");
constexpr int kNever = 0x7FFFFFFF;
// Blocks of a CTA's run at least: a block takes 2 us, a part half a microsecond of its unit's join.
constexpr int kLeastRun = 4;
constexpr int kScaleRing = 8;                     // blocks whose scales are known: the warps are at most 5 blocks apart
constexpr int kScaledRing = 4;                    // of them, those that the conversion may still wait for
// Exponents of 2 by which the largest values of a block's tokens may differ under one scale: more, and every token has its own.
constexpr int kNear = 8;
constexpr int kApartMost = 9;                     // block_apart's largest weight is 2^kApartMost: 128 of them stay in f16
// A block whose values' exponent is this much below an earlier one's of the item is weighed by block_apart: its weights may
// be 2^-126 and less beside the reference, and yet count in the row's sum.
constexpr int kFar = 80;
constexpr int kKeyFloor = -100, kValueFloor = -60;        // scales' least exponents: l has room for 2^(kSumExp + 60)
constexpr float kMost = 65000.f;                  // bound of a block's sum of weights: f16 ends at 65504
constexpr float kStay = 8.f;                      // largest weight of a block under a huge Z that stays, as an exponent (kMost: 2^9)
constexpr float kLift = 4.f;                      // a row's first weight is about 2^4
constexpr int kTopExp = 14;                       // the largest element of an operand is in [2^14, 2^15)
constexpr float kBack = 262144.f;                 // 2^(kSumExp - kTopExp): O over l back to its size
constexpr int kSumExp = 32;                       // l gathers 2^(kSumExp - Z) times the weights: far from both ends of fp32

template <int ND> constexpr int block_bytes() { return kTile * 64 * ND * 2; }
static_assert(q4_page_bytes(1) == 2 * q4_v(1), "keys and values take the same room");
constexpr int kControl = 1024;
constexpr int kTokenExps = kScaleRing * 2 * kTile;        // bytes: the exponents of a block's keys, and of its values
template <int ND, int QT> constexpr int smem_bytes() {
  return (QT + kStages) * block_bytes<ND>() + packed_pages<QT>() * q4_v(ND) + kControl + kTokenExps;
}
static_assert(smem_bytes<2, 1>() <= 227 * 1024 && smem_bytes<2, 2>() <= 227 * 1024, "an SM's shared memory");
// A tile's part: O as [4 warps][D columns][32 lanes], then the rows' Z and l.
template <int D> constexpr int part_floats() { return kTile * (D + 2); }
template <int N> constexpr uint32_t idesc() {     // fp32 D, f16 A and B, M = 128
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// tcgen's waits, with what follows a first try that fails out of the way: twelve roles' loops share the instruction caches,
// and with the waits' own loops among them a block took 15 % longer.
__device__ __forceinline__ bool wait_long(int32_t* err, volatile int* abort, long long timeout, uint32_t bar, uint32_t parity,
                                          int code) {
  const Ctl ctl{err, abort, timeout};
  return wait_bar(ctl, bar, parity, code);
}
__device__ __forceinline__ bool await(const Ctl& ctl, uint32_t bar, uint32_t parity, int code) {
  if (__builtin_expect(mbar_try_wait(bar, parity), 1)) return true;
  return wait_long(ctl.err, ctl.abort, ctl.timeout, bar, parity, code);
}
__device__ __forceinline__ bool await_warp(const Ctl& ctl, uint32_t bar, uint32_t parity, int code) {
  if (__builtin_expect(__all_sync(0xffffffffu, mbar_try_wait(bar, parity)), 1)) return true;
  return __all_sync(0xffffffffu, wait_long(ctl.err, ctl.abort, ctl.timeout, bar, parity, code));
}

struct Q4TcGeom {
  Q4Geom c;
  int32_t G, n_q;
  int32_t gp, inv_gp, pos;                        // query heads and positions of a tile; ceil(65536 / gp)
  int32_t per_kv;                                 // head groups of gp per KV head
  int32_t upr, units;                             // units (two tiles) of a row's head group, and of the call
  float alpha;
  int64_t o_sb;
  int32_t o_st, o_sh;
  long long timeout;
  const int32_t* q_lens;
  const uint8_t* pages;
  const int32_t* table;
  const int32_t* lens;
  __nv_bfloat16* out;
  int2* cut;                                      // [CTAs]: the unit that is cut and begins in the CTA's run (-1: none), its last CTA
  float* part;                                    // [2 CTAs][2 tiles][part_floats]
};

// A unit: two tiles of query rows of one head group of a cache row.
struct Unit {
  int b, hk, h, row;                              // sequence, KV head, first query head, cache row
  int q0, rows;                                   // first position, and how many exist
  int limit;                                      // last key that the first position sees (may be negative)
  int nb0, nb1, nb;                               // key blocks of the two tiles, and of both
  int tk;                                         // keys
};
__device__ __forceinline__ Unit unit_of(const Q4TcGeom& g, int i) {
  Unit u;
  const int hg = i / g.upr;
  u.row = hg / g.per_kv;
  u.b = u.row / g.c.Hkv;
  u.hk = u.row - u.b * g.c.Hkv;
  u.h = u.hk * g.G + (hg - u.row * g.per_kv) * g.gp;
  u.tk = safe_len(g.lens[u.row], g.c.max_pages);
  const int nq = g.q_lens ? min(max(g.q_lens[u.b], 0), g.n_q) : g.n_q;
  u.q0 = (i - hg * g.upr) * 2 * g.pos;
  u.rows = min(2 * g.pos, nq - u.q0);             // none or fewer: nothing to do
  u.limit = u.q0 + u.tk - nq;
  const int last0 = u.limit + min(u.rows, g.pos) - 1, last1 = u.limit + u.rows - 1;
  u.nb0 = u.rows <= 0 || last0 < 0 ? 0 : last0 / kTile + 1;
  u.nb1 = u.rows <= g.pos || last1 < 0 ? 0 : last1 / kTile + 1;
  u.nb = max(u.nb0, u.nb1);
  return u;
}

// A unit's part in one CTA, its keys counted from the part's first; the copying thread hands it to the other roles.
struct Item {
  int unit;                                       // -1: no more
  int b, h, q0, rows, limit, tk;
  int nb0, nb1, nb;
  int low;                                        // blocks low .. nb - 1 hold keys hidden to some row
  int part;                                       // where its part goes; -1: it is whole
};

__device__ __forceinline__ void put_row(const Q4TcGeom& g, __nv_bfloat16* out, int pos, int head, int c, uint4 w) {
  *(uint4*)(out + pos * g.o_st + head * g.o_sh + c) = w;
}

// A row of the output, by its thread.  tO: 0xFFFFFFFF for rows without any key; nan: a bit per group of 64 columns that is
// NaN.
template <int D>
__device__ __noinline__ void write_row(__nv_bfloat16* out, bool mine, int d, uint32_t tO, float inv, uint32_t nan) {
#pragma unroll 1
  for (int c = 0; c < D && c < d; c += 16) {
    float o[16];
    if (tO != 0xFFFFFFFFu) tmem_get16(tO + c, o);
    const bool bad = nan >> (c >> 6) & 1;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = bad ? NAN : tO != 0xFFFFFFFFu ? o[i] * inv : 0.f;
    if (mine) {
      put8((uint8_t*)(out + c), o);
      if (c + 8 < d) put8((uint8_t*)(out + c + 8), o + 8);
    }
  }
}

// A warp's rows of a tile's part to the workspace, a lane per row: whole lines per column.  tO: 0xFFFFFFFF where the part
// holds no key of the tile (Z = -inf and l = 0 say so).
template <int D>
__device__ __noinline__ void store_part(float* part, uint32_t tO, float Z, float l, int row, uint32_t nan) {
  float* po = part + (row >> 5) * (D * 32) + (row & 31);
  if (tO != 0xFFFFFFFFu) {
#pragma unroll 1
    for (int c = 0; c < D; c += 16) {
      float o[16];
      tmem_get16(tO + c, o);
      const bool bad = nan >> (c >> 6) & 1;
#pragma unroll
      for (int i = 0; i < 16; ++i) __stcg(po + (c + i) * 32, bad ? NAN : o[i]);
    }
  }
  __stcg(part + kTile * D + row, Z);
  __stcg(part + kTile * D + kTile + row, l);
}

__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
__device__ __forceinline__ uint32_t pack_half2(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *(const uint32_t*)&h;
}
// A group's m and s (two bf16 in a word), scaled, as two f16.
__device__ __forceinline__ uint32_t scaled(uint32_t w, float by) { return pack_half2(q4_m(w) * by, q4_s(w) * by); }

// Eight codes of a word (items 0 .. 7 in order) to eight f16, s c + m each; s and m of items 2 k, 2 k + 1 in pairs (of odd
// k, s / 16: those codes are taken 4 bits higher).
__device__ __forceinline__ uint4 expand(uint32_t w, const uint32_t (&s)[4], const uint32_t (&m)[4]) {
  const __half2 big = __halves2half2(__ushort_as_half(0x6400), __ushort_as_half(0x6400));
  const uint32_t u = w >> 8;
  const uint32_t a[4] = {(w & 0x000F000Fu) | 0x64006400u, (w & 0x00F000F0u) | 0x64006400u, (u & 0x000F000Fu) | 0x64006400u,
                         (u & 0x00F000F0u) | 0x64006400u};
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __half2 x = __hfma2(__hsub2(*(const __half2*)&a[k], big), *(const __half2*)&s[k], *(const __half2*)&m[k]);
    o[k] = *(const uint32_t*)&x;
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ uint32_t sixteenth(uint32_t s) {
  const __half2 x = __hmul2(*(const __half2*)&s, __halves2half2(__ushort_as_half(0x2C00), __ushort_as_half(0x2C00)));
  return *(const uint32_t*)&x;
}

// The largest magnitude that codes of a group can stand for (NaN: 0).
__device__ __forceinline__ float reach(uint32_t w) {
  const float m = q4_m(w);
  return fmaxf(0.f, fmaxf(fabsf(m), fabsf(fmaf(15.f, q4_s(w), m))));
}
__device__ __forceinline__ int exponent_of(uint32_t reach, int floor) { return min(127, max(floor, (int)(reach >> 23) - 127)); }
// Of the steps and smallest values (words [ND][64] of two pages) a lane's i-th share: where it lies, and its first token.
template <int ND>
__device__ __forceinline__ uint4* steps_at(uint8_t* half0, uint8_t* half1, int i, int lane, int& token) {
  const int v = i * 32 + lane, page = v / (16 * ND), at = v % (16 * ND) * 4;
  token = page * kPage + (at & (kPage - 1));
  return (uint4*)((page ? half1 : half0) + 2048 * ND + at * 4);
}
// What four tokens of a group reach, those from `left` on nothing.
__device__ __forceinline__ uint4 reach_four(const uint4& w, int token, int left) {
  auto of = [&](uint32_t x, int e) { return token + e < left ? __float_as_uint(reach(x)) : 0u; };
  return make_uint4(of(w.x, 0), of(w.y, 1), of(w.z, 2), of(w.w, 3));
}
// Scaled, as two f16.  pairs: the m of two tokens, and then their s (of odd pairs s / 16, see expand).
__device__ __forceinline__ uint4 scale_four(const uint4& w, const float4& by, bool pairs) {
  const uint4 x = make_uint4(scaled(w.x, by.x), scaled(w.y, by.y), scaled(w.z, by.z), scaled(w.w, by.w));
  return pairs ? make_uint4(__byte_perm(x.x, x.y, 0x5410), __byte_perm(x.x, x.y, 0x7632), __byte_perm(x.z, x.w, 0x5410),
                            sixteenth(__byte_perm(x.z, x.w, 0x7632)))
               : x;
}
// The keys' or the values' two pages of a block scaled in place, by one exponent, or token by token where their largest
// values lie too far apart; the tokens' exponents go to exps[token].  Returns the largest.
template <int ND>
__device__ __forceinline__ int scale_half(uint8_t* half0, uint8_t* half1, int left, int floor, bool pairs, int lane, int8_t* exps,
                                          bool& apart) {
  int token;
  uint32_t most = 0, least = 0xFFFFFFFFu;         // least: less one, so that zeros have no say
#pragma unroll 1
  for (int i = 0; i < ND; ++i) {
    const uint4 r = reach_four(*steps_at<ND>(half0, half1, i, lane, token), token, left);
    most = max(max(most, max(r.x, r.y)), max(r.z, r.w));
    least = min(min(least, min(r.x - 1, r.y - 1)), min(r.z - 1, r.w - 1));
  }
  most = __reduce_max_sync(0xffffffffu, most);
  least = __reduce_min_sync(0xffffffffu, least);
  const int top = exponent_of(most, floor);
  // by groups, which may lie further apart than tokens: exponents of their own are right for any tokens
  const bool own = most != 0 && top - exponent_of(least + 1, floor) > kNear;
  apart |= own;
  const float all = power_of_two(kTopExp - top);
  *(uint32_t*)(exps + 4 * lane) = 0x01010101u * (uint8_t)top;
  __syncwarp();
#pragma unroll 1
  for (int i = 0; i < ND; ++i) {
    uint4* to = steps_at<ND>(half0, half1, i, lane, token);
    const uint4 w = *to;
    float4 by = make_float4(all, all, all, all);
    if (__builtin_expect(own, 0)) {
      uint4 r = reach_four(w, token, left);
      if (ND == 2) {                              // the token's other group
        r.x = max(r.x, __shfl_xor_sync(0xffffffffu, r.x, 16));
        r.y = max(r.y, __shfl_xor_sync(0xffffffffu, r.y, 16));
        r.z = max(r.z, __shfl_xor_sync(0xffffffffu, r.z, 16));
        r.w = max(r.w, __shfl_xor_sync(0xffffffffu, r.w, 16));
      }
      const int4 e = make_int4(exponent_of(r.x, floor), exponent_of(r.y, floor), exponent_of(r.z, floor), exponent_of(r.w, floor));
      by = make_float4(power_of_two(kTopExp - e.x), power_of_two(kTopExp - e.y), power_of_two(kTopExp - e.z),
                       power_of_two(kTopExp - e.w));
      *(char4*)(exps + token) = make_char4(e.x, e.y, e.z, e.w);
    }
    *to = scale_four(w, by, pairs);
  }
  return top;
}
// A block's scales: what takes back that its keys and values were multiplied by 2^(kTopExp - EK), 2^(kTopExp - EV).
struct Scales {
  float k_up;                                     // 2^(EK - kTopExp); negative: the block is block_apart's
  float ev, sum_up;                               // EV, and 2^(kSumExp - EV)
};

// A query row in shared memory (ND panels of 64 columns, 16-byte pieces swizzled) from bf16 to f16, its largest element in
// [2^kTopExp, 2^(kTopExp + 1)); returns the exponent that takes it back.
template <int ND>
__device__ __noinline__ int narrow_row(uint8_t* tile, int row) {
  uint32_t top = 0;
#pragma unroll 4
  for (int i = 0; i < 8 * ND; ++i) {
    const uint4 w = *(const uint4*)(tile + (i >> 3) * (kTile * 128) + row * 128 + ((i ^ row) & 7) * 16);
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) top = max(top, max(x[e] << 16 & 0x7FFF0000u, x[e] & 0x7FFF0000u));
  }
  const int e2 = min(127, max(-110, (int)(top >> 23) - 127));
  const float down = power_of_two(kTopExp - e2);
#pragma unroll 4
  for (int i = 0; i < 8 * ND; ++i) {
    uint4* p = (uint4*)(tile + (i >> 3) * (kTile * 128) + row * 128 + ((i ^ row) & 7) * 16);
    const uint4 w = *p;
    *p = make_uint4(scaled(w.x, down), scaled(w.y, down), scaled(w.z, down), scaled(w.w, down));
  }
  return e2 - kTopExp;
}

// 2^d, d <= 0, in two factors: Z holds EV, so from one block to the next it may move by more than ex2's 2^-126, while what l
// has gathered still counts.
struct Fall {
  float a, b;
  __device__ __forceinline__ explicit Fall(float d) {
    const float first = fmaxf(d, -120.f);
    a = ex2(first);
    b = ex2(fmaxf(d - first, -120.f));
  }
  __device__ __forceinline__ float of(float x) const { return x * a * b; }
};
// A row of O times f; a whole warp's rows.  The blocks before are done: their products were issued before this S.
template <int D>
__device__ __forceinline__ void scale_row(uint32_t tO, const Fall& f) {
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    float o[32];
    tmem_ld32(tO + 32 * c, o);
    tmem_wait(o);
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = f.of(o[i]);
    tmem_st32(tO + 32 * c, o);
  }
}

// The exponentials of a block whose sum passed kMost, or whose Z is huge, done over: rows that are `over` move Z to the
// block's maximum, and what O (at tO, unless it is still empty) and l hold goes with it; a huge Z that is not passed stays.
// Their differences to the maximum are taken before they are scaled: under a huge Z one rounding of S alpha + EV - Z is off
// by more than an exponential bears (Z itself is: from 2^25 on no float lies within 1 of a row's first exponent).  The
// other rows' weights are what they were, and are added in row_exp's order.  Returns (Z, l).
template <int D>
__device__ __noinline__ float2 block_over(uint32_t tS, uint32_t tO, float alpha, float ev, float sum_up, float Z, float l, bool over) {
  const float top = row_max(tS);
  float base = 0.f, neg = ev - (Z == -INFINITY ? ev : Z);
  Fall f(0.f);
  if (over) {
    neg = fmaf(top, alpha, ev - Z);               // top's weight as an exponent
    base = top;
    if (top == -INFINITY) {
      base = neg = 0.f;                           // no logit but -inf (and NaN)
    } else if (Z == -INFINITY || l == 0.f || !(neg <= kStay)) {
      const float zn = rintf(fmaf(top, alpha, ev)) - kLift;
      if (l != 0.f) f = Fall(fminf(Z - zn, 0.f));             // else O is zero too, and Z this block's own first reference
      Z = zn;
      // top's own exponent, kLift and what Z was rounded by: a later block's terms stand beside these under one Z
      neg = fminf(fmaxf(fmaf(top, alpha, ev - zn), kLift - 1.f), kLift + 1.f);
    }
  }
  if (tO != 0xFFFFFFFFu) scale_row<D>(tO, f);
  return make_float2(Z, fmaf(write_exp_from<true>(tS, base, alpha, neg), sum_up, f.of(l)));
}

// A block whose tokens have exponents of their own: keys in exps[0 .. 127], values in exps[128 .. 255].  A row's weight of
// token c is 2^(S 2^EK_c alpha + EV_c - Z) as ever, but Z goes by the tokens that the row sees, and l takes each weight at
// its own scale.  Two passes over S: the largest exponent, then P, in write_exp_from's places.  Returns (Z, l).
template <int D>
__device__ __noinline__ float2 block_apart(uint32_t tS, uint32_t tO, float row_alpha, const volatile int8_t* exps, float Z, float l) {
  auto alpha_of = [&](int c) { return fminf(fmaxf(row_alpha * power_of_two((int)exps[c] - kTopExp), 1.2e-38f), 3.4e38f); };
  float top = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < kTile; c += 32) {
    float s[32];
    tmem_ld32(tS + c, s);
    tmem_wait(s);
#pragma unroll
    for (int i = 0; i < 32; ++i) top = fmaxf(top, fmaf(s[i], alpha_of(c + i), (float)exps[kTile + c + i]));
  }
  Fall f(0.f);
  float largest = top - Z;                        // the largest weight's exponent
  if (top != -INFINITY && !(largest <= (float)kApartMost)) {
    const float zn = rintf(top) - kLift;
    f = Fall(Z - zn);
    Z = zn;
    largest = kLift;
  }
  l = f.of(l);
  if (tO != 0xFFFFFFFFu) scale_row<D>(tO, f);
  const float ref = Z == -INFINITY ? 0.f : Z;
  const bool huge = fabsf(ref) > kHuge && top != -INFINITY;   // as in block_over: differences first
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    float s[32];
    tmem_ld32(tS + 32 * c, s);
    tmem_wait(s);
    uint32_t p[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float2 w;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int at = 32 * c + 2 * i + k;
        const float ev = (float)exps[kTile + at], u = fmaf(s[2 * i + k], alpha_of(at), huge ? ev : ev - ref);
        const float e = huge ? u - top + largest : u;
        (k ? w.y : w.x) = ex2(e);
        l += ex2(e - ev + (float)kSumExp);
      }
      p[i] = pack_p<true>(w);
    }
    tmem_st16(tS + 16 * c, p);
  }
  return make_float2(Z, l);
}

// A page's tokens or columns are dealt to kParts warps.
constexpr int kParts = kConvert / 2;
template <int ND> constexpr int kTiles = 4 * ND / kParts;
template <int ND> __device__ __forceinline__ int group_of(int w) { return (w >> 1) * kTiles<ND> / 4; }

// Keys of one page, a warp's share of its tokens (from `first` on; their steps already scaled f16), into rows of 64 columns
// (128 bytes, 16-byte pieces swizzled).
template <int ND>
__device__ __forceinline__ void expand_keys(const uint8_t* page, uint8_t* tile, int page_row, int first, int lane) {
#pragma unroll 1
  for (int i = 0; i < kPage / kParts / 8; ++i) {
    const int token = first + 8 * i + (lane >> 2), t4 = lane & 3, row = page_row + token;
    uint32_t w[2 * ND];
    if constexpr (ND == 2) {
      const uint4 v = *(const uint4*)(page + (token * 4 + t4) * 16);
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
      const uint2 v = *(const uint2*)(page + (token * 4 + t4) * 8);
      w[0] = v.x; w[1] = v.y;
    }
    uint8_t* dst = tile + row * 128;
    const int a = ((2 * t4) ^ (row & 7)) * 16, b = ((2 * t4 + 1) ^ (row & 7)) * 16;
#pragma unroll
    for (int p = 0; p < ND; ++p) {
      const uint32_t ms = *(const uint32_t*)(page + q4_k_ms(ND) + (p * kPage + token) * 4);
      const uint32_t s1 = __byte_perm(ms, ms, 0x3232), m1 = __byte_perm(ms, ms, 0x1010), s16 = sixteenth(s1);
      const uint32_t s[4] = {s1, s16, s1, s16}, m[4] = {m1, m1, m1, m1};
      *(uint4*)(dst + p * (kTile * 128) + a) = expand(w[2 * p], s, m);
      *(uint4*)(dst + p * (kTile * 128) + b) = expand(w[2 * p + 1], s, m);
    }
  }
}

// Values of one page, kTiles tiles of 16 columns from `first` on (all of one group), into rows of 64 tokens.
// MASKED: tokens from `left` on are zeros, and a NaN is replaced by zero; returns the first token that had one.
template <int ND, bool MASKED>
__device__ __forceinline__ int expand_values(const uint8_t* half, uint8_t* tile, int first, int left, int lane) {
  const int t4 = lane & 3, gid = lane >> 2, group = first >> 2;
  uint32_t s[2][4], m[2][4];
  int bad = kNever;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const uint4 v = *(const uint4*)(half + 2048 * ND + (group * kPage + 16 * t4 + 4 * x) * 4);
    uint32_t w[4] = {v.x, v.y, v.z, v.w};         // m, s, m, s of two tokens each
    if (MASKED) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int token = 16 * t4 + 4 * x + e, shift = 16 * (e & 1);
        const bool gone = token >= left, nan = (w[e & 2] >> shift & 0x7C00u) == 0x7C00u;
        if (!gone && nan) bad = min(bad, token);
        if (gone || nan) {
          w[e & 2] &= 0xFFFF0000u >> shift;
          w[(e & 2) + 1] &= 0xFFFF0000u >> shift;
        }
      }
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      m[x >> 1][2 * (x & 1) + y] = w[2 * y];
      s[x >> 1][2 * (x & 1) + y] = w[2 * y + 1];
    }
  }
#pragma unroll 1
  for (int i = 0; i < kTiles<ND>; ++i) {
    const uint4 w = *(const uint4*)(half + (first + i) * 512 + gid * 64 + t4 * 16);
    uint8_t* dst = tile + (16 * (first + i) + gid) * 128;     // columns 16 i + gid and 8 further: gid is the row in the swizzle
    const int a = ((2 * t4) ^ gid) * 16, b = ((2 * t4 + 1) ^ gid) * 16;
    *(uint4*)(dst + a) = expand(w.x, s[0], m[0]);
    *(uint4*)(dst + b) = expand(w.y, s[1], m[1]);
    *(uint4*)(dst + 1024 + a) = expand(w.z, s[0], m[0]);
    *(uint4*)(dst + 1024 + b) = expand(w.w, s[1], m[1]);
  }
  return bad;
}

template <int ND, int QT>
__global__ void __launch_bounds__(kThreads, 1)
q4_attention_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ Q4TcGeom g, int32_t* __restrict__ err) {
  constexpr int D = 64 * ND;
  constexpr int kBlock = block_bytes<ND>(), kHalf = q4_v(ND), kPacked = packed_pages<QT>();
  constexpr int kKPanel = kTile * 128, kVPanel = D * 128;     // 64 columns of 128 keys; 64 keys of D columns
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {                   // the swizzle pattern needs 1024-byte alignment
    if (threadIdx.x == 0) {
      atomicCAS(err, 0, (int)kDevMisalignedSmem);
      g.cut[blockIdx.x] = make_int2(-1, 0);
    }
    return;
  }
  uint8_t* sQ = smem;                             // QT tiles
  uint8_t* sKV = smem + QT * kBlock;              // kStages blocks: K, V, K, V ... of descending blocks
  uint8_t* sP = sKV + kStages * kBlock;           // kPacked pages: of a block, the keys' two and then the values'
  uint64_t* bars = (uint64_t*)(sP + kPacked * kHalf);
  const uint32_t q_full = smem_u32(bars), q_empty = q_full + 8, drained = q_full + 16;      // drained: [2]
  const uint32_t turn = q_full + 32, s_full = q_full + 48, p_full = s_full + 16, o_full = p_full + 16;        // [2] each
  const uint32_t kv_full = o_full + 16, kv_empty = kv_full + 8 * kStages;
  const uint32_t packed_full = kv_empty + 8 * kStages, packed_empty = packed_full + 8 * kPacked;
  const uint32_t item_full = packed_empty + 8 * kPacked, item_empty = item_full + 8 * kItemRing;
  const uint32_t q_ready = item_empty + 8 * kItemRing, scaled_full = q_ready + 16;         // [2], [kScaledRing]
  constexpr int kBars = 6 + 6 + 2 * kStages + 2 * kPacked + 2 * kItemRing + 2 + kScaledRing;
  uint32_t* tmem_slot = (uint32_t*)(bars + kBars);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  volatile Item* s_items = (volatile Item*)(abort_flag + 1);                               // [kItemRing]
  volatile int* s_bad = (volatile int*)(s_items + kItemRing);      // [kItemRing][kConvert]: first NaN token of a warp's group
  volatile Scales* s_scales = (volatile Scales*)(s_bad + kConvert * kItemRing);                  // [kScaleRing]
  using RunOf = decode::RunShared<kThreads / 32>;
  RunOf& run = *(RunOf*)((uint8_t*)bars + kControl - sizeof(RunOf));
  int8_t* s_exps = (int8_t*)bars + kControl;                  // [kScaleRing][keys, values][kTile]
  static_assert(8 * kBars + 8 + (sizeof(Item) + 4 * kConvert) * kItemRing + sizeof(Scales) * kScaleRing + sizeof(RunOf) <= kControl &&
                    sizeof(RunOf) % 8 == 0, "control block");

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1); mbar_init(q_empty, 2); mbar_init(drained, 1); mbar_init(drained + 8, 1);
    mbar_init(turn, 1); mbar_init(turn + 8, 1);
    for (int t = 0; t < 2; ++t) { mbar_init(s_full + 8 * t, 1); mbar_init(p_full + 8 * t, 128); mbar_init(o_full + 8 * t, 1); }
    for (int i = 0; i < kStages; ++i) { mbar_init(kv_full + 8 * i, kConvert); mbar_init(kv_empty + 8 * i, 2); }
    for (int i = 0; i < kPacked; ++i) { mbar_init(packed_full + 8 * i, 1); mbar_init(packed_empty + 8 * i, kConvert / 2 + 1); }
    // an item's slot is released by the MMA issuers, the scaling, the converting and the softmax warps
    for (int i = 0; i < kItemRing; ++i) { mbar_init(item_full + 8 * i, 1); mbar_init(item_empty + 8 * i, 11 + kConvert); }
    for (int t = 0; t < 2; ++t) mbar_init(q_ready + 8 * t, 128);
    for (int i = 0; i < kScaledRing; ++i) mbar_init(scaled_full + 8 * i, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&qmap) : "memory");
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  // units whose rows see no key: zeros
  for (int i = blockIdx.x; i < g.units; i += gridDim.x) {
    const Unit u = unit_of(g, i);
    if (u.nb > 0) continue;
    const int pieces = g.c.d / 8;
    __nv_bfloat16* out = g.out + u.b * g.o_sb + (int64_t)u.q0 * g.o_st + (int64_t)u.h * g.o_sh;
    for (int x = threadIdx.x; x < u.rows * g.gp * pieces; x += kThreads) {
      const int row = x / pieces;
      put_row(g, out, row / g.gp, row % g.gp, x % pieces * 8, make_uint4(0, 0, 0, 0));
    }
  }
  const Run plan = decode::plan_run<kThreads / 32>(g.units, [&](int i) { return unit_of(g, i).nb; }, run, decode::kWholeRow, kLeastRun);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const Ctl ctl{err, abort_flag, g.timeout};
  const int64_t x0 = run.cut[0], x1 = run.cut[1];
  uint32_t loaded = 0, q_loaded = 0;              // copies that the copying thread armed (for the teardown)

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ------------------------------------------------ softmax: one query row per thread
    const int t = warp >> 2, row = threadIdx.x & 127;
    // positions of this row and of the warp's first row
    const int my_pos = (row * g.inv_gp) >> 16, pos_lo = ((row - lane) * g.inv_gp) >> 16;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = lanes + t * kTile, tO = lanes + 256 + t * kTile;
    uint32_t sc = 0, oc = 0, qc = 0;              // phases of s_full, o_full and q_full
    uint32_t before = 0;                          // blocks of the items before
    for (uint32_t n = 0; __all_sync(0xffffffffu, !*abort_flag); ++n) {
      const int slot = n % kItemRing;
      if (!await_warp(ctl, item_full + 8 * slot, (n / kItemRing) & 1, kDevTimeoutEpilogue)) break;
      const volatile Item& it = s_items[slot];                // read where it is used: registers are short
      if (it.unit < 0) break;
      const int nb = t ? it.nb1 : it.nb0;
      const int limit = it.limit + t * g.pos + my_pos;        // last key that this row sees
      const bool live = my_pos < g.pos && t * g.pos + my_pos < it.rows;
      // ---- the queries as f16
      if (!await_warp(ctl, q_full, qc & 1, kDevTimeoutEpilogue)) break;
      ++qc;
      float row_alpha = 0.f;
      if (nb > 0) row_alpha = g.alpha * power_of_two(max(-126, narrow_row<ND>(sQ + t * kBlock, row)));
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(q_ready + 8 * t);
      // the row's reference and its sum; rows of the tile that do not exist never look for one
      float Z = live ? -INFINITY : 0.f, l = 0.f;
      bool ok = true;
      const uint32_t first = before + it.nb - 1;              // of block 0
      before += it.nb;
      for (int j = nb - 1; j >= 0; --j) {
        if (!await_warp(ctl, s_full + 8 * t, sc & 1, kDevTimeoutEpilogue)) { ok = false; break; }
        ++sc;
        fence_after();
        const volatile Scales& scales = s_scales[(first - j) % kScaleRing];
        // never 0 (0 x -inf) nor infinite
        const int seen = limit - j * kTile, lo = seen - (my_pos - pos_lo);       // columns 0 .. seen; the warp's first row's
        if (__builtin_expect(kTile - 1 > lo, 0)) hide(tS, seen, lo);          // a hidden key in the warp
        const float k_up = scales.k_up;
        if (__builtin_expect(k_up < 0.f, 0)) {
          const float2 r = block_apart<D>(tS, j < nb - 1 ? tO : 0xFFFFFFFFu, row_alpha,
                                          s_exps + (first - j) % kScaleRing * (2 * kTile), Z, l);
          Z = r.x;
          l = r.y;
          tmem_st_wait();
          fence_before();
          mbar_arrive(p_full + 8 * t);
          continue;
        }
        const float alpha = fminf(fmaxf(row_alpha * k_up, 1.2e-38f), 3.4e38f), ev = scales.ev;
        if (__builtin_expect(__any_sync(0xffffffffu, Z == -INFINITY), 0)) {
          const float bm = first_reference(tS, lo);
          if (Z == -INFINITY && bm != -INFINITY) Z = rintf(fmaf(bm, alpha, ev)) - kLift;     // P and O of the row are zero so far
        }
        uint32_t p[64];
        // exact up to kHuge; NaN for a larger Z, so that block_over does its blocks
        const float neg = fabsf(Z) <= kHuge ? ev - Z : Z == -INFINITY ? 0.f : NAN;
        const float sum = row_exp<true>(tS, alpha, neg, p);
        const bool over = live && !(sum <= kMost);            // a NaN too
        if (__builtin_expect(!__any_sync(0xffffffffu, over), 1)) {
          l = fmaf(sum, scales.sum_up, l);
          tmem_st32<0>(tS, p);
          tmem_st32<32>(tS + 32, p);
        } else {
          const float2 r = block_over<D>(tS, j < nb - 1 ? tO : 0xFFFFFFFFu, alpha, ev, scales.sum_up, Z, l, over);
          Z = r.x;
          l = r.y;
        }
        tmem_st_wait();
        fence_before();
        mbar_arrive(p_full + 8 * t);
      }
      if (!ok) break;
      // ---- the item's rows
      if (nb > 0) {
        if (!await_warp(ctl, o_full + 8 * t, oc & 1, kDevTimeoutEpilogue)) break;
        ++oc;
        fence_after();
      }
      uint32_t nan = 0;                                       // groups of columns whose NaN was taken out of the products
      if (nb > 0 && live)
        for (int i = 0; i < kConvert; ++i)
          if (s_bad[kConvert * slot + i] <= limit) nan |= 1u << group_of<ND>(i);
      const uint32_t src = nb > 0 ? tO : 0xFFFFFFFFu;
      if (pos_lo < g.pos && t * g.pos + pos_lo < it.rows) {   // a row of the warp exists
        if (it.part >= 0) {
          store_part<D>(g.part + ((int64_t)it.part * 2 + t) * part_floats<D>(), src, nb > 0 ? Z : -INFINITY, l, row, nan);
        } else {
          // no visible key: zeros; logits that are all -inf: NaN
          const float inv = l != 0.f ? kBack / l : limit < 0 ? 0.f : NAN;
          write_row<D>(g.out + it.b * g.o_sb + (int64_t)(it.q0 + t * g.pos + my_pos) * g.o_st + (int64_t)(it.h + row - my_pos * g.gp) * g.o_sh,
                       live, g.c.d, src, inv, nan);
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(item_empty + 8 * slot);
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8 && lane == 0) {
      // ------------------------------------------------ copies: pages of codes, queries
      bool ok = true;
      int2 cut = make_int2(-1, 0);
      int i = run.row[0];
      int64_t xr = x0 < x1 ? run.start[0] : x1;
      uint32_t n = 0;
      for (; ok && !*abort_flag; ++n) {
        const int slot = n % kItemRing;
        if (!await(ctl, item_empty + 8 * slot, ((n / kItemRing) & 1) ^ 1, kDevTimeoutTmaProducer)) break;
        Unit u;
        int64_t sa = 0, sb = 0;
        while (xr < x1) {                         // the next unit with work in this run
          u = unit_of(g, i);
          sa = xr > x0 ? xr : x0;
          sb = xr + u.nb < x1 ? xr + u.nb : x1;
          if (sa < sb) break;
          xr += u.nb;
          ++i;
        }
        if (xr >= x1) {
          s_items[slot].unit = -1;
          mbar_arrive(item_full + 8 * slot);
          break;
        }
        const int b0 = (int)(sa - xr), nb = (int)(sb - sa);
        const bool whole = nb == u.nb;
        Item it;
        it.unit = i;
        it.b = u.b;
        it.h = u.h;
        it.q0 = u.q0;
        it.rows = u.rows;
        it.limit = u.limit - b0 * kTile;
        it.tk = u.tk - b0 * kTile;
        it.nb0 = min(max(u.nb0 - b0, 0), nb);
        it.nb1 = min(max(u.nb1 - b0, 0), nb);
        it.nb = nb;
        it.low = max(it.limit + 1, 0) / kTile;
        it.part = whole ? -1 : 2 * (int)blockIdx.x + (b0 > 0 ? 0 : 1);
        if (!whole && b0 == 0) cut = make_int2(i, decode::last_of(plan, xr, u.nb));
        const int* from = (const int*)&it;
        volatile int* to = (volatile int*)&s_items[slot];
#pragma unroll
        for (int k = 0; k < (int)(sizeof(Item) / 4); ++k) to[k] = from[k];
        mbar_arrive(item_full + 8 * slot);
        auto load_q = [&]() {
          const int tiles = it.rows > g.pos ? 2 : 1;
          mbar_expect_tx(q_full, tiles * ND * g.gp * g.pos * 128);
          for (int x = 0; x < tiles * ND; ++x)
            tma_load_4d(smem_u32(sQ) + x * kKPanel, &qmap, q_full, 64 * (x % ND), it.h, it.q0 + x / ND * g.pos, it.b);
          ++q_loaded;
        };
        const int pages_held = decode::pages_of(u.tk);
        const int32_t* row_table = g.table + (int64_t)u.row * g.c.max_pages;
        int64_t page[2] = {0, 0};
        int pages = 0;
        for (int b = 0; b < 2 * nb && ok; ++b) {
          if (b == 2) {
            // the queries after the first K and V blocks: the last item's products still read the old ones
            ok = await(ctl, q_empty, (q_loaded & 1) ^ 1, kDevTimeoutTmaProducer);
            if (!ok) break;
            load_q();
          }
          if ((b & 1) == 0) {
            const int j = 2 * (b0 + nb - 1 - (b >> 1));       // the block's first page in the row
            pages = min(2, pages_held - j);
            for (int k = 0; k < pages; ++k) page[k] = safe_page(row_table[j + k], g.c.n_pages);
          }
          for (int k = 0; k < 2 && ok; ++k) {
            const int st = loaded % kPacked;
            ok = await(ctl, packed_empty + 8 * st, ((loaded / kPacked) & 1) ^ 1, kDevTimeoutTmaProducer);
            if (!ok) break;
            if (k < pages) {
              mbar_expect_tx(packed_full + 8 * st, kHalf);
              bulk_load(smem_u32(sP) + st * kHalf, g.pages + page[k] * q4_page_bytes(ND) + (b & 1) * kHalf, kHalf, packed_full + 8 * st);
            } else {
              mbar_arrive(packed_full + 8 * st);  // a row's last block may be of one page
            }
            ++loaded;
          }
        }
        if (ok && nb == 1) {                      // an item of one block: its queries come last
          ok = await(ctl, q_empty, (q_loaded & 1) ^ 1, kDevTimeoutTmaProducer);
          if (!ok) break;
          load_q();
        }
        xr += u.nb;
        ++i;
      }
      g.cut[blockIdx.x] = cut;
    } else if (warp == 9 || warp == 10) {
      // ------------------------------------------------ MMA issuer of one tile (the whole warp, one elected lane at an issue)
      const int t = warp - 9;
      uint32_t qc = 0, pc = 0, tc = 0;            // query loads, P tiles, turns
      int st = 0;                                 // stage in turn and its parity
      uint32_t ph = 0;
      const uint32_t tS = tmem + t * kTile, tO = tmem + 256 + t * kTile;
      const uint64_t qdesc = sw128_desc(smem_u32(sQ) + t * kBlock, 16, 1024);
      const uint64_t kvdesc = sw128_desc(smem_u32(sKV), 16, 1024);
      // S = Q K^T for the K block in stage sk, O += P V for the V block in stage sv; the stages are released
      // with the products that read them
      auto scores = [&](int sk, bool pass) {
        const uint64_t kd = kvdesc + sk * (kBlock >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kKPanel + (kk & 3) * 32) >> 4;
          mma_ss(tS, qdesc + off, kd + off, idesc<kTile>(), kk > 0);
          if (kk == D / 16 - 3 && pass) mbar_arrive(turn + 8 * (t ^ 1));
        }
        commit(s_full + 8 * t);
        commit(kv_empty + 8 * sk);
      };
      auto values = [&](int sv, bool add) {
        const uint64_t vd = kvdesc + sv * (kBlock >> 4);
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          mma_ts(tO, tS + 8 * kk, vd + (((kk >> 2) * kVPanel + (kk & 3) * 32) >> 4), idesc<D>(), add || kk > 0);
        commit(kv_empty + 8 * sv);
      };
      // a block that this tile does not need: released only once it is there, so that the
      // release counts for this use of the stage
      auto skip = [&](int sx) { if (lane == 0) mbar_arrive(kv_empty + 8 * sx); };
      auto next = [&]() { if (++st == kStages) { st = 0; ph ^= 1; } };
      for (uint32_t n = 0; __all_sync(0xffffffffu, !*abort_flag); ++n) {
        const int slot = n % kItemRing;
        if (!await_warp(ctl, item_full + 8 * slot, (n / kItemRing) & 1, kDevTimeoutMma)) break;
        struct { int unit, nb, nb0, nb1; } it;
        it.unit = __shfl_sync(0xffffffffu, s_items[slot].unit, 0);
        it.nb = __shfl_sync(0xffffffffu, s_items[slot].nb, 0);
        it.nb0 = __shfl_sync(0xffffffffu, s_items[slot].nb0, 0);
        it.nb1 = __shfl_sync(0xffffffffu, s_items[slot].nb1, 0);
        __syncwarp();
        if (lane == 0) mbar_arrive(item_empty + 8 * slot);
        if (it.unit < 0) break;
        const int nb = t ? it.nb1 : it.nb0;
        bool ok = await_warp(ctl, kv_full + 8 * st, ph, kDevTimeoutMma) && await_warp(ctl, q_ready + 8 * t, qc & 1, kDevTimeoutMma);
        if (!ok) break;
        ++qc;
        fence_after();
        if (it.nb - 1 < nb) {
          if (elect_one()) {
            scores(st, false);
            if (it.nb == 1) commit(q_empty);
          }
        } else {
          skip(st);
        }
        __syncwarp();
        next();
        for (int j = it.nb - 1; j >= 0; --j) {
          // V of this block and K of the one below it, and then P: nothing is waited for between the products
          const int sv = st;
          ok = await_warp(ctl, kv_full + 8 * sv, ph, kDevTimeoutMma);
          next();
          const int sk = st;
          if (ok && j >= 1) {
            ok = await_warp(ctl, kv_full + 8 * sk, ph, kDevTimeoutMma);
            next();
          }
          if (!ok) break;
          if (j < nb) {
            // the two tiles take turns, tile 0 first
            const bool both = j < min(it.nb0, it.nb1);
            if (both) {
              ok = await_warp(ctl, turn + 8 * t, (tc & 1) ^ (t ^ 1), kDevTimeoutMma);
              ++tc;
            }
            ok = ok && await_warp(ctl, p_full + 8 * t, pc & 1, kDevTimeoutMma);
            if (!ok) break;
            ++pc;
            fence_after();
            if (elect_one()) {
              values(sv, j < nb - 1);
              if (j >= 1) {
                scores(sk, both);
              } else {
                if (both) mbar_arrive(turn + 8 * (t ^ 1));
                commit(o_full + 8 * t);
              }
              if (j == 1) commit(q_empty);        // the queries have been read
            }
          } else {
            skip(sv);
            if (j >= 1 && j - 1 < nb) {
              fence_after();
              if (elect_one()) {
                scores(sk, false);
                if (j == 1) commit(q_empty);
              }
            } else if (j >= 1) {
              skip(sk);
            }
          }
          __syncwarp();
        }
        if (!ok) break;
        if (nb == 0 && lane == 0) mbar_arrive(q_empty);
        __syncwarp();
      }
    } else if (warp == 11) {
      // ------------------------------------------------ a block's scales, from the steps and smallest values of its groups
      uint32_t bc = 0;                            // blocks so far
      int st = 0;                                 // page of codes in turn and its parity
      uint32_t ph = 0;
      for (uint32_t n = 0; __all_sync(0xffffffffu, !*abort_flag); ++n) {
        const int slot = n % kItemRing;
        if (!await_warp(ctl, item_full + 8 * slot, (n / kItemRing) & 1, kDevTimeoutEpilogue)) break;
        const int unit = __shfl_sync(0xffffffffu, s_items[slot].unit, 0);
        if (unit < 0) break;
        const int nb = s_items[slot].nb, tk = s_items[slot].tk;
        int ev_top = kValueFloor;                 // of the item's blocks so far
        bool ok = true;
        for (int j = nb - 1; j >= 0 && ok; --j, ++bc) {
          int8_t* exps = s_exps + bc % kScaleRing * (2 * kTile);
          bool apart = false;
          int ek = 0, ev = 0;
          // in loops: what runs once a block costs most by its instructions' fetches
#pragma unroll 1
          for (int which = 0; which < 2 && ok; ++which) {
            int at[2];
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
              ok = ok && await_warp(ctl, packed_full + 8 * st, ph, kDevTimeoutEpilogue);
              at[0] = i ? at[0] : st;
              at[1] = st;
              if (++st == kPacked) { st = 0; ph ^= 1; }
            }
            if (!ok) break;
            ek = ev;
            // stale tokens past the row's end have no say
            ev = scale_half<ND>(sP + at[0] * kHalf, sP + at[1] * kHalf, tk - j * kTile, which ? kValueFloor : kKeyFloor, which, lane,
                                exps + which * kTile, apart);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");      // the next copy writes here
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(packed_empty + 8 * at[0]);
              mbar_arrive(packed_empty + 8 * at[1]);
            }
          }
          if (!ok) break;
          if (lane == 0) {
            volatile Scales& out = s_scales[bc % kScaleRing];
            out.k_up = apart || ev_top - ev > kFar ? -1.f : power_of_two(ek - kTopExp);
            out.ev = (float)ev;
            out.sum_up = power_of_two(kSumExp - ev);
            mbar_arrive(scaled_full + 8 * (bc % kScaledRing));
          }
          ev_top = max(ev_top, ev);
          __syncwarp();
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(item_empty + 8 * slot);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    // ------------------------------------------------ conversion: warp w takes page w & 1 of a block, and a quarter of its
    // tokens (keys) or of its columns (values)
    const int w = warp - 12, page = w & 1, part = w >> 1;
    uint32_t pc = 0;                              // halves of blocks so far
    int st = 0, ps = page;                        // stage and page of codes in turn
    uint32_t ph = 0;
    for (uint32_t n = 0; __all_sync(0xffffffffu, !*abort_flag); ++n) {
      const int slot = n % kItemRing;
      if (!await_warp(ctl, item_full + 8 * slot, (n / kItemRing) & 1, kDevTimeoutEpilogue)) break;
      const int unit = __shfl_sync(0xffffffffu, s_items[slot].unit, 0);
      if (unit < 0) break;
      const int nb = s_items[slot].nb, low = s_items[slot].low, tk = s_items[slot].tk;
      int bad = kNever;
      bool ok = true;
      for (int b = 0; b < 2 * nb && ok; ++b) {
        const int j = nb - 1 - (b >> 1);
        const uint32_t bc = pc >> 1;
        // the copies have landed once the scales are there
        ok = ((b & 1) != 0 || await_warp(ctl, scaled_full + 8 * (bc % kScaledRing), (bc / kScaledRing) & 1, kDevTimeoutEpilogue)) &&
             await_warp(ctl, kv_empty + 8 * st, ph ^ 1, kDevTimeoutEpilogue);
        if (!ok) break;
        const uint8_t* src = sP + ps * kHalf;
        uint8_t* dst = sKV + st * kBlock;
        if ((b & 1) == 0) {
          expand_keys<ND>(src, dst, page * kPage, kPage / kParts * part, lane);
        } else if (j < low) {
          expand_values<ND, false>(src, dst + page * kVPanel, kTiles<ND> * part, 0, lane);
        } else {
          // a later block's tokens come first: the smallest is kept
          const int at = j * kTile + page * kPage;
          const int x = expand_values<ND, true>(src, dst + page * kVPanel, kTiles<ND> * part, tk - at, lane);
          if (x != kNever) bad = min(bad, at + x);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");          // the products read it next
        if (b == 2 * nb - 1) {
          bad = __reduce_min_sync(0xffffffffu, bad);
          if (lane == 0) s_bad[kConvert * slot + w] = bad;
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(kv_full + 8 * st);
          mbar_arrive(packed_empty + 8 * ps);
        }
        ++pc;
        ps = ps + 2 >= kPacked ? ps + 2 - kPacked : ps + 2;
        if (++st == kStages) { st = 0; ph ^= 1; }
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(item_empty + 8 * slot);
    }
  }

  // ------------------------------------------------ teardown
  __syncwarp();
  pdl_trigger();
  fence_before();
  __syncthreads();
  fence_after();
  if (*abort_flag) {
    bool landed = true;
    if (warp == 8 && lane == 0) {
      for (uint32_t i = loaded > (uint32_t)kPacked ? loaded - kPacked : 0; i < loaded; ++i)
        landed &= drain_phase(packed_full + 8 * (i % kPacked), (i / kPacked) & 1);
      if (q_loaded > 0) landed &= drain_phase(q_full, (q_loaded - 1) & 1);
    }
    if (warp == 9 || warp == 10) {
      const uint32_t bar = drained + 8 * (warp - 9);
      if (elect_one()) commit(bar);
      __syncwarp();
      landed &= drain_phase(bar, 0);
    }
    if (!landed) {
      const long long t0 = clock64();
      while (clock64() - t0 < kDrainCycles) {
      }
    }
    fence_before();
    __syncthreads();
    fence_after();
  }
  if (warp == 9)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// The parts of a cut unit's tile together: 32 columns of its 128 rows per CTA, two warps for 32 rows
// (16 columns each), a lane per row; the parts are added in order.
template <int ND>
__global__ void __launch_bounds__(256)
q4_join_kernel(const __grid_constant__ Q4TcGeom g) {
  constexpr int D = 64 * ND;
  __shared__ __align__(16) uint8_t rows[kTile * 80];          // 64 bytes a row, 80 apart
  pdl_wait();
  const int2 cut = g.cut[blockIdx.x];
  const int t = blockIdx.y & 1, c0 = (blockIdx.y >> 1) * 32;
  if (cut.x >= 0 && c0 < g.c.d) {
    const Unit u = unit_of(g, cut.x);
    const int left = min(g.pos, u.rows - t * g.pos);          // positions of the tile that exist
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = (warp & 3) * 32 + lane, c = c0 + (warp >> 2) * 16;
    const int pos_lo = (((warp & 3) * 32) * g.inv_gp) >> 16;
    if (left > 0 && pos_lo < left) {                          // the warp has a row that exists
      auto part = [&](int k) { return g.part + ((int64_t)(2 * k + (k == (int)blockIdx.x)) * 2 + t) * part_floats<D>(); };
      float M = -INFINITY, L = 0.f, o[16];
#pragma unroll 8
      for (int k = blockIdx.x; k <= cut.y; ++k) M = fmaxf(M, __ldcg(part(k) + kTile * D + row));
      const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] = 0.f;
#pragma unroll 1                                              // it runs once, and its instructions' fetches count
      for (int k = blockIdx.x; k <= cut.y; ++k) {
        const float* p = part(k);
        const float Z = __ldcg(p + kTile * D + row), l = __ldcg(p + kTile * D + kTile + row);
        if (Z == -INFINITY && l == 0.f) continue;             // no key of the row: its O may not be there
        const Fall f(Z - ref);
        p += (warp & 3) * (D * 32) + c * 32 + lane;
        L = fmaf(l * f.a, f.b, L);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = fmaf(__ldcg(p + 32 * i) * f.a, f.b, o[i]);
      }
      // no visible key: zeros; logits that are all -inf: NaN
      const float inv = L != 0.f ? kBack / L : u.limit + t * g.pos + ((row * g.inv_gp) >> 16) < 0 ? 0.f : NAN;
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] *= inv;
      put8(rows + row * 80 + (warp >> 2) * 32, o);
      put8(rows + row * 80 + (warp >> 2) * 32 + 16, o + 8);
    }
    __syncthreads();
    __nv_bfloat16* out = g.out + u.b * g.o_sb + (int64_t)(u.q0 + t * g.pos) * g.o_st + (int64_t)u.h * g.o_sh;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = i * 64 + (threadIdx.x >> 2), k = threadIdx.x & 3, pos = (r * g.inv_gp) >> 16;
      if (pos < left && c0 + k * 8 < g.c.d) put_row(g, out, pos, r - pos * g.gp, c0 + k * 8, *(const uint4*)(rows + r * 80 + k * 16));
    }
  }
  pdl_trigger();
}

// ---------------------------------------------------------------- host side
template <int ND, int QT>
cudaError_t launch(const CUtensorMap& map, const Q4TcGeom& g, int32_t* err, int sms, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = raise_smem(q4_attention_tc_kernel<ND, QT>, smem_bytes<ND, QT>(), done);
  if (e != cudaSuccess) return e;
  const cudaError_t run =
      launch_pdl(q4_attention_tc_kernel<ND, QT>, dim3(sms), dim3(kThreads), (size_t)smem_bytes<ND, QT>(), s, map, g, err);
  if (run != cudaSuccess) return run;
  return launch_pdl(q4_join_kernel<ND>, dim3(sms, 4 * ND), dim3(256), 0, s, g);
}

constexpr size_t kCutBytes = 4096;                // [CTAs] int2
constexpr int kMaxCtas = kCutBytes / sizeof(int2);

}  // namespace

// Units of a call.
int64_t q4_tc_units(const Q4Geom& g, int G, int n_q) {
  const int gp = prefill_tc_heads(G), positions = 2 * (kTile / gp);
  return (int64_t)g.rows * (G / gp) * (((int64_t)n_q + positions - 1) / positions);
}

// [serving header | cut units | parts].
size_t q4_tc_workspace_bytes(const Q4Geom& g, int sms) {
  sms = std::min(sms, kMaxCtas);
  return kServeHeader + kCutBytes + (size_t)sms * 4 * (g.d64 == 64 ? part_floats<64>() : part_floats<128>()) * sizeof(float);
}

cudaError_t launch_q4_attention_tc(const Q4Geom& c, int G, int n_q, float alpha, const int32_t* q_lens, const void* q,
                                   int64_t q_sb, int64_t q_st, int64_t q_sh, void* out, int64_t o_sb, int64_t o_st,
                                   int64_t o_sh, const uint8_t* pages, const int32_t* table, const int32_t* lens, void* ws,
                                   int sms, cudaStream_t s) {
  const EncodeFn enc = encode_fn();
  if (enc == nullptr) return cudaErrorNotSupported;
  const int gp = prefill_tc_heads(G), B = c.rows / c.Hkv, pos = kTile / gp;
  // [B][n_q][Hq][d] in boxes of 64 columns of a tile's heads and positions; columns past d and positions past the end
  // read as zeros.  The stride of an axis of extent 1 is unused.
  CUtensorMap map;
  cuuint64_t dims[4] = {(cuuint64_t)c.d, (cuuint64_t)c.Hkv * G, (cuuint64_t)n_q, (cuuint64_t)B};
  cuuint64_t strides[3] = {(int64_t)c.Hkv * G == 1 ? 16 : (cuuint64_t)q_sh * 2, n_q == 1 ? 16 : (cuuint64_t)q_st * 2, B == 1 ? 16 : (cuuint64_t)q_sb * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)gp, (cuuint32_t)pos, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  if (enc(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(q), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  char* w = (char*)ws;
  Q4TcGeom g = {};
  g.c = c;
  g.G = G;
  g.n_q = n_q;
  g.gp = gp;
  g.inv_gp = (65536 + gp - 1) / gp;
  g.pos = pos;
  g.per_kv = G / gp;
  g.upr = (n_q + 2 * pos - 1) / (2 * pos);
  g.units = (int32_t)q4_tc_units(c, G, n_q);
  g.alpha = alpha;
  g.o_sb = o_sb;
  g.o_st = (int32_t)o_st;
  g.o_sh = (int32_t)o_sh;
  g.timeout = 4000000000LL;
  g.q_lens = q_lens;
  g.pages = pages;
  g.table = table;
  g.lens = lens;
  g.out = (__nv_bfloat16*)out;
  g.cut = (int2*)(w + kServeHeader);
  g.part = (float*)(w + kServeHeader + kCutBytes);
  sms = std::min(sms, kMaxCtas);
  int32_t* err = (int32_t*)w;
  if (n_q <= pos) return c.d64 == 64 ? launch<1, 1>(map, g, err, sms, s) : launch<2, 1>(map, g, err, sms, s);
  return c.d64 == 64 ? launch<1, 2>(map, g, err, sms, s) : launch<2, 2>(map, g, err, sms, s);
}

}  // namespace chunkkv
