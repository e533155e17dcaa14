// Attention over packed prompts on the tensor cores (tcgen05 + TMA + TMEM): bf16, head
// dimension up to 128.
//
//   O_i = sum_{j <= i + Tk - Tq} softmax_j(scale q_i . k_j) v_j
//
// A work item is two tiles of 128 query rows of one sequence.  A tile's rows are the gp
// query heads of a KV head (or of a part of its group) at 128 / gp consecutive positions,
// row = position * gp + head, so that short prompts fill their tiles and a block of keys
// and values serves every head of its group.  Where whole items would leave SMs idle
// (few query rows against many keys), an item takes a part of the keys, kb blocks: the
// parts' (m, l, O) go to the workspace, and a second launch adds them in order.
// The CTA (one per SM, claiming items from a counter in the workspace, the longest
// first) walks the keys in blocks of 128 and keeps for both tiles S = Q K^T (fp32, 128
// columns) and O (fp32, D columns) in TMEM: 512 columns.  Per block and tile:
//   S = Q K^T                  8 products of K = 16, operands in shared memory
//   P = 2^(S alpha - m)        one thread per row: the exponentials and their sum, P rounded
//                              to bf16 into the columns of S that it replaces
//   O += P V                   A operand P in TMEM, V as it lies ([keys][d], outer-major)
// While the threads of one tile work on its S, the tensor cores do the other tile's two
// products: 2 x 512 cycles at full rate, in which 128 threads have 128 x 128
// exponentials (512 cycles of the exponential unit) and about 200 other instructions
// each to do.  So the tensor cores bound it as long as the softmax keeps up.  What is left
// is the chain of one tile: P ready, products (1024), S ready, softmax (950), with about
// 200 cycles of barrier latency on each side, 2500 cycles a block pair for 2048 of products.
//
// Measured (one layer, 128 columns; the power limit decides within the ranges): 16384
// tokens of 28 / 4 heads 1.10 to 1.25 ms, 1.54 to 1.75 PFLOP/s of the visible pairs; 8192
// tokens of 32 / 8 heads 0.31 to 0.35 ms, 1.57 to 1.76 PFLOP/s; 16 prompts of 100 to 2000
// tokens packed 0.19 ms, 1.07 PFLOP/s (an item there has 6 block pairs, and its begin and
// end cost as much as three more); 420 and 455 new tokens on 5.3 and 7.7 thousand cached
// ones 0.09 ms; 64 new tokens on 9000 28 us.
//
// The reference m of a row is the maximum of some of its first logits and stays while
// the row's sum is below 2^24: a common factor of P, O and the sum costs no precision
// (bf16 and fp32 have the same exponents) and the final division removes it.
// So a block has no maximum to find before its exponentials, and they need no more
// than 64 logits in registers at a time.  A block that passes the bound is done over
// with its maximum as the reference, O and the sum rescaled; S is still there, since
// P replaces it only after that test.
//
// The blocks are taken from the last one down: the masked ones come first.  P is zero
// where a key is hidden, but 0 x inf is NaN, and the values of hidden keys (later
// positions, the next sequence's rows) may hold anything.  So a checking warp looks
// through the V of the masked blocks before the product and replaces non-finite
// elements by zero; rows that do see such a key get the element added at the end.
//
// Warp roles: 0-3 and 4-7 softmax of tile 0 and 1, 8 TMA producer, 9 and 10 MMA
// issuers of tile 0 and 1 (with one issuer for both, its waits for one tile kept the
// other's products back: a block pair took 3250 cycles), 11 V check, which holds every V
// block until it has seen it there.
// Every wait is bounded (tcgen.cuh); a CTA that gives up drains and exits.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "tcgen.cuh"

namespace chunkkv {
namespace {

using namespace tcgen;

constexpr int kTile = 128;                        // query rows of a tile, keys of a block
constexpr int kStages = 4;                        // K and V blocks in shared memory (five were no faster)
static_assert(kStages % 2 == 0, "K blocks lie in even stages, V blocks in odd ones");
constexpr int kItemRing = 2;
constexpr int kThreads = 384;                     // 12 warps, three warpgroups
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * 168, "register shares within the launch's");
constexpr int kMaxChecked = 4;                    // masked blocks of an item: 256 rows' limits span at most three
constexpr float kBig = 16777216.f;                // bound of a row's sum under its reference
constexpr float kHuge = 4194304.f;                // references (in base-2 exponents) up to which one rounding will do

template <int D> constexpr int block_bytes() { return kTile * D * 2; }
constexpr int kPanel = kTile * 128;               // 128 rows x 64 elements
constexpr int kStageOut = 32 * 128;               // a softmax warp's 32 rows x 64 output columns
template <int D> constexpr int smem_bytes() { return (2 + kStages) * block_bytes<D>() + 1024 + 8 * kStageOut; }
// A tile's part: O as [4 warps][D columns][32 lanes], then the rows' m and l.
template <int D> constexpr int part_floats() { return kTile * (D + 2); }
template <int N> constexpr uint32_t idesc() {     // fp32 D, bf16 A and B, M = 128
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
constexpr uint32_t kOuterMajorB = 1u << 16;

struct TcGeom {
  int32_t groups;                                 // head groups of gp query heads
  int32_t per_kv;                                 // of them per KV head
  int32_t gp, inv_gp;                             // inv_gp: ceil(65536 / gp), to divide a row by gp
  int32_t pos;                                    // positions of a tile, 128 / gp
  int32_t d;
  int32_t kb;                                     // key blocks of an item at most (0: items are whole)
  int32_t n_items;
  float alpha;
  int64_t v_st, v_sh, o_st, o_sh;                 // element strides of v and out
  long long timeout;
  float* part;                                    // [n_items][2][part_floats<D>()]
};
struct TcMaps { CUtensorMap q, k, v; };

// The producer decodes an item once and hands it to the other roles in shared memory.
struct Item {
  int item;                                       // -1: no more
  int h, hk;                                      // its first query head, its KV head
  int q0, k0, tk;                                 // packed rows where the item's queries and the sequence's keys begin
  int rows;                                       // positions that exist
  int limit;                                      // last key that the item's first position sees (may be negative)
  int nb0, nb1;                                   // key blocks of the two tiles
  int nb;                                         // blocks walked
  int low;                                        // blocks low .. nb - 1 hold keys hidden to some row
  int s, parts0, parts1;                          // the item's part, and how many each tile has (SPLIT)
};

template <bool SPLIT, int MAXB>
__device__ __forceinline__ Item decode_item(const TcGeom& g, const PrefillTable<MAXB>& tab, int item) {
  Item it;
  it.item = item;
  const int u = item / g.groups, hg = item - u * g.groups;
  it.h = hg * g.gp;
  it.hk = hg / g.per_kv;
  const int i = find_seq(tab, u);
  const PrefillSeq sq = tab.seq[i];
  const int unit = tab.uoff[i + 1] - 1 - u, ns = SPLIT ? sq.ns : 1;
  const int r0 = unit / ns * 2 * g.pos;           // later positions see more keys: they come first
  it.s = SPLIT ? ns - 1 - unit % ns : 0;          // item - s groups is the tile's first part
  it.q0 = sq.q0 + r0;
  it.rows = min(2 * g.pos, sq.tq - r0);
  it.k0 = sq.k0;
  it.tk = sq.tk;
  it.limit = r0 + sq.tk - sq.tq;                  // last key that the first row sees
  const int last0 = it.limit + min(it.rows, g.pos) - 1, last1 = it.limit + it.rows - 1;
  it.nb0 = last0 < 0 ? 0 : last0 / kTile + 1;
  it.nb1 = it.rows <= g.pos || last1 < 0 ? 0 : last1 / kTile + 1;
  it.parts0 = it.parts1 = 1;
  if (SPLIT) {
    it.parts0 = (it.nb0 + g.kb - 1) / g.kb;
    it.parts1 = (it.nb1 + g.kb - 1) / g.kb;
    // from here on counted from the part's first key
    const int b0 = it.s * g.kb;
    it.k0 += b0 * kTile;
    it.tk -= b0 * kTile;
    it.limit -= b0 * kTile;
    it.nb0 = min(max(it.nb0 - b0, 0), g.kb);
    it.nb1 = min(max(it.nb1 - b0, 0), g.kb);
  }
  it.nb = max(it.nb0, it.nb1);
  it.low = max(it.limit + 1, 0) / kTile;
  return it;
}

// What a row runs once per item or less is kept out of the loop over the blocks, in small
// loops of its own: at one pass an item, straight-line code costs its instruction fetches
// (an unrolled write of the output rows took 6000 cycles an item).

// -inf into the columns of S that the row does not see (those after `seen`), whatever
// they hold.  lo: what the warp's first row sees; columns up to there are left alone.
__device__ __noinline__ void hide(uint32_t tS, int seen, int lo) {
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
__device__ __noinline__ float first_reference(uint32_t tS, int lo) {
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

// 32 columns of P from 32 of S: pairs by one packed FMA, two exponentials, a packed sum
// and a packed conversion.
template <int C>
__device__ __forceinline__ void chunk_exp(const float (&s)[32], float2 a2, float2 n2, float2 (&sum)[2], uint32_t (&p)[64]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 e = __ffma2_rn(make_float2(s[2 * i], s[2 * i + 1]), a2, n2);
    const float2 w = make_float2(ex2(e.x), ex2(e.y));
    sum[i & 1] = __fadd2_rn(sum[i & 1], w);
    const __nv_bfloat162 b = __floats2bfloat162_rn(w.x, w.y);
    p[16 * C + i] = *(const uint32_t*)&b;
  }
}
// A row's P under the reference -neg, and its sum.  Straight-line code: a branch per
// chunk cost 400 cycles of a block's 1000.
__device__ __forceinline__ float row_exp(uint32_t tS, float alpha, float neg, uint32_t (&p)[64]) {
  float ra[32], rb[32];
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  const float2 a2 = make_float2(alpha, alpha), n2 = make_float2(neg, neg);
  tmem_ld32(tS, ra);
  tmem_wait(ra);
  tmem_ld32(tS + 32, rb);
  chunk_exp<0>(ra, a2, n2, sum, p);
  tmem_wait(rb);
  tmem_ld32(tS + 64, ra);
  chunk_exp<1>(rb, a2, n2, sum, p);
  tmem_wait(ra);
  tmem_ld32(tS + 96, rb);
  chunk_exp<2>(ra, a2, n2, sum, p);
  tmem_wait(rb);
  chunk_exp<3>(rb, a2, n2, sum, p);
  return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

// The same of (S - base) alpha + neg, with P written: its 16 columns of 32 logits lie among the columns read by then.
// The terms are added in row_exp's order: a row that is here only because another of its warp is keeps its bits.
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
      const __nv_bfloat162 b = __floats2bfloat162_rn(w.x, w.y);
      p[i] = *(const uint32_t*)&b;
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
__device__ __noinline__ float3 block_again(uint32_t tS, uint32_t tO, float alpha, float m, float l, bool over) {
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

// The keys with non-finite values that a row sees: a bit per key (null: none), their
// number, and the values of the first.
struct Bad {
  const uint32_t* keys;
  int n;
  const __nv_bfloat16* v;
};
// Calls add(column, value) for each such value in columns c0 .. c1 - 1.
template <typename F>
__device__ __forceinline__ void each_bad(const Bad& bad, int64_t v_st, int c0, int c1, F add) {
  for (int k = 0; k < bad.n; ++k) {
    if (!(bad.keys[k >> 5] >> (k & 31) & 1)) continue;
    for (int i = c0; i < c1; ++i) {
      const __nv_bfloat16 y = bad.v[k * v_st + i];
      if ((__bfloat16_as_ushort(y) & 0x7F80u) == 0x7F80u) add(i, __bfloat162float(y));
    }
  }
}

// A warp's rows of the output, 64 columns at a time through the warp's own staging rows,
// so that the stores are whole lines of a row: 16-byte piece k of row r lies at k ^ (r & 7).
// out: the tile's first position and head; left: positions of it that exist; tO:
// 0xFFFFFFFF for rows without any key.
template <int D>
__device__ __noinline__ void write_rows(const TcGeom& g, __nv_bfloat16* out, int left, uint32_t tO, float inv, uint8_t* stage,
                                        int row, Bad bad) {
  const int lane = row & 31;
  uint8_t* mine = stage + lane * 128;
  out += (lane & 7) * 8;
  // of the rows that this lane writes pieces of, -1: none (the plan keeps a tile's rows within 2^31 elements)
  int where[8];
  const int o_st = (int)g.o_st, o_sh = (int)g.o_sh;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int tr = row - lane + 4 * i + (lane >> 3), pos = (tr * g.inv_gp) >> 16;
    where[i] = pos < left ? pos * o_st + (tr - pos * g.gp) * o_sh : -1;
  }
#pragma unroll 1
  for (int c = 0; c < D && c < g.d; c += 64) {
#pragma unroll 2
    for (int k = 0; k < 4; ++k) {
      float o[16];
      if (tO != 0xFFFFFFFFu) tmem_get16(tO + c + 16 * k, o);
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] = tO != 0xFFFFFFFFu ? o[i] * inv : 0.f;
      put8(mine + ((2 * k) ^ (lane & 7)) * 16, o);
      put8(mine + ((2 * k + 1) ^ (lane & 7)) * 16, o + 8);
    }
    if (bad.keys)
      each_bad(bad, g.v_st, c, min(c + 64, g.d), [&](int i, float y) {
        __nv_bfloat16* o = (__nv_bfloat16*)(mine + (((i >> 3) & 7) ^ (lane & 7)) * 16) + (i & 7);
        *o = __float2bfloat16_rn(__bfloat162float(*o) + y);
      });
    __syncwarp();
    const bool inside = c + (lane & 7) * 8 < g.d;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3);
      const uint4 w = *(const uint4*)(stage + r * 128 + ((lane & 7) ^ (r & 7)) * 16);
      if (inside && where[i] >= 0) *(uint4*)(out + where[i] + c) = w;
    }
    __syncwarp();
  }
}

// A warp's rows of a tile's part to the workspace, a lane per row: whole lines per column.
template <int D>
__device__ __noinline__ void store_part(const TcGeom& g, float* part, uint32_t tO, float m, float l, int row, Bad bad) {
  float* po = part + (row >> 5) * (D * 32) + (row & 31);
#pragma unroll 1
  for (int c = 0; c < D; c += 16) {
    float o[16];
    tmem_get16(tO + c, o);
#pragma unroll
    for (int i = 0; i < 16; ++i) __stcg(po + (c + i) * 32, o[i]);
  }
  if (bad.keys) each_bad(bad, g.v_st, 0, g.d, [&](int i, float y) { po[32 * i] += y; });
  __stcg(part + kTile * D + row, m);
  __stcg(part + kTile * D + kTile + row, l);
}

template <int D, bool SPLIT, int MAXB>
__global__ void __launch_bounds__(kThreads, 1)
prefill_tc_kernel(const __grid_constant__ TcMaps maps, const __grid_constant__ TcGeom g,
                  const __grid_constant__ PrefillTable<MAXB> tab, const __nv_bfloat16* __restrict__ v,
                  __nv_bfloat16* __restrict__ out, int32_t* __restrict__ err, int32_t* __restrict__ sched) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int kBlock = block_bytes<D>(), kPanels = D / 64;
  if (smem_u32(smem) & 1023u) {                   // the swizzle pattern needs 1024-byte alignment
    if (threadIdx.x == 0) atomicCAS(err, 0, (int)kDevMisalignedSmem);
    return;
  }
  uint8_t* sQ = smem;                             // two tiles
  uint8_t* sKV = smem + 2 * kBlock;               // kStages blocks: K, V, K, V ... of descending blocks
  uint64_t* bars = (uint64_t*)(sKV + kStages * kBlock);
  const uint32_t q_full = smem_u32(bars), q_empty = q_full + 8, drained = q_full + 16;      // drained: [2]
  const uint32_t turn = q_full + 32, s_full = q_full + 48, p_full = s_full + 16, o_full = p_full + 16;        // [2] each
  const uint32_t kv_full = o_full + 16, kv_empty = kv_full + 8 * kStages, v_ok = kv_empty + 8 * kStages;
  const uint32_t item_full = v_ok + 8 * kStages, item_empty = item_full + 8 * kItemRing;
  const uint32_t checked = item_empty + 8 * kItemRing;                                     // [kItemRing]
  constexpr int kBars = 6 + 6 + 3 * kStages + 3 * kItemRing;
  uint32_t* tmem_slot = (uint32_t*)(bars + kBars);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  volatile Item* s_items = (volatile Item*)(abort_flag + 1);                               // [kItemRing]
  uint32_t* s_bad = (uint32_t*)(s_items + kItemRing);     // [kItemRing][kMaxChecked][4] keys, a bit each
  static_assert(8 * kBars + 8 + (sizeof(Item) + 4) * kItemRing + 16 * kItemRing * kMaxChecked <= 1024, "control block");

  volatile int* s_any = (volatile int*)(s_bad + kItemRing * kMaxChecked * 4);              // [kItemRing] any of them
  uint8_t* sOut = (uint8_t*)bars + 1024;           // [8][kStageOut]
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1); mbar_init(q_empty, 2); mbar_init(drained, 1); mbar_init(drained + 8, 1);
    mbar_init(turn, 1); mbar_init(turn + 8, 1);
    for (int t = 0; t < 2; ++t) { mbar_init(s_full + 8 * t, 1); mbar_init(p_full + 8 * t, 128); mbar_init(o_full + 8 * t, 1); }
    // a stage is released by the MMA issuers, one that holds V by the checking warp too
    for (int i = 0; i < kStages; ++i) { mbar_init(kv_full + 8 * i, 1); mbar_init(kv_empty + 8 * i, 2 + (i & 1)); mbar_init(v_ok + 8 * i, 1); }
    // an item's slot is released by the MMA issuers, the checking warp and each softmax warp
    for (int i = 0; i < kItemRing; ++i) {
      mbar_init(item_full + 8 * i, 1); mbar_init(item_empty + 8 * i, 11); mbar_init(checked + 8 * i, 1);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&maps.q) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&maps.k) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&maps.v) : "memory");
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const Ctl ctl{err, abort_flag, g.timeout};
  uint32_t loaded = 0, q_loaded = 0;              // copies that the producer armed (for the teardown)

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ------------------------------------------------ softmax: one query row per thread
    const int t = warp >> 2, row = threadIdx.x & 127;
    // positions of this row and of the warp's first row
    const int my_pos = (row * g.inv_gp) >> 16, pos_lo = ((row - lane) * g.inv_gp) >> 16;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = lanes + t * kTile, tO = lanes + 256 + t * kTile;
    uint32_t sc = 0, oc = 0, cc = 0;              // phases of s_full, o_full and (a bit per slot) checked
    pdl_wait();
    for (uint32_t n = 0; __all_sync(0xffffffffu, !*abort_flag); ++n) {
      const int slot = n % kItemRing;
      if (!wait_warp(ctl, item_full + 8 * slot, (n / kItemRing) & 1, kDevTimeoutEpilogue)) break;
      const volatile Item& it = s_items[slot];                // read where it is used: registers are short
      if (it.item < 0) break;
      const int nb = t ? it.nb1 : it.nb0;
      const int limit = it.limit + t * g.pos + my_pos;        // last key that this row sees
      const bool live = my_pos < g.pos && t * g.pos + my_pos < it.rows;
      // the row's reference, -m alpha, and its sum; rows of the tile that do not exist never look for one
      float m = live ? -INFINITY : 0.f, neg = 0.f, l = 0.f;
      bool ok = true;
      for (int j = nb - 1; j >= 0; --j) {
        if (!wait_warp(ctl, s_full + 8 * t, sc & 1, kDevTimeoutEpilogue)) { ok = false; break; }
        ++sc;
        fence_after();
        const int seen = limit - j * kTile, lo = seen - (my_pos - pos_lo);       // columns 0 .. seen; the warp's first row's
        if (kTile - 1 > lo) hide(tS, seen, lo);               // a hidden key in the warp
        if (__any_sync(0xffffffffu, m == -INFINITY)) {
          const float bm = first_reference(tS, lo);
          if (m == -INFINITY && bm != -INFINITY) {            // P and O of the row are zero so far
            m = bm;
            neg = offset_of(m, g.alpha);
          }
        }
        uint32_t p[64];
        const float sum = row_exp(tS, g.alpha, neg, p);
        const bool over = live && !(l + sum <= kBig);         // a NaN too, as under a huge reference
        if (!__any_sync(0xffffffffu, over)) {
          l += sum;
          tmem_st32<0>(tS, p);
          tmem_st32<32>(tS + 32, p);
        } else {
          const float3 r = block_again<D>(tS, j < nb - 1 ? tO : 0xFFFFFFFFu, g.alpha, m, l, over);
          m = r.x;
          neg = r.y;
          l = r.z;
        }
        tmem_st_wait();
        fence_before();
        mbar_arrive(p_full + 8 * t);
      }
      if (!ok) break;
      // ---- the item's rows
      // no visible key: zeros; logits that are all -inf: NaN (else l is 1 or more, from its reference)
      const float inv = l != 0.f ? __fdividef(1.f, l) : limit < 0 ? 0.f : NAN;
      bool flagged = false;
      if (it.nb > 0 && t * g.pos < it.rows) {
        if (!wait_warp(ctl, checked + 8 * slot, (cc >> slot) & 1, kDevTimeoutEpilogue)) break;
        flagged = s_any[slot] != 0;
      }
      if (it.nb > 0) cc ^= 1u << slot;
      if (nb > 0) {
        if (!wait_warp(ctl, o_full + 8 * t, oc & 1, kDevTimeoutEpilogue)) break;
        ++oc;
        fence_after();
      }
      // non-finite values that the check took out of the products (if any) for the rows that see them
      const Bad bad = {flagged && live ? s_bad + slot * kMaxChecked * 4 : nullptr,
                       min(min(it.nb - it.low, kMaxChecked) * kTile, min(limit + 1, it.tk) - it.low * kTile),
                       v + (int64_t)(it.k0 + it.low * kTile) * g.v_st + it.hk * g.v_sh};
      if (SPLIT) {
        // the part's (m, l, O) to the workspace; join_kernel adds a tile's parts
        if (nb > 0) store_part<D>(g, g.part + ((int64_t)it.item * 2 + t) * part_floats<D>(), tO, m, l, row, bad);
      } else if (pos_lo < g.pos && t * g.pos + pos_lo < it.rows) {
        write_rows<D>(g, out + (int64_t)(it.q0 + t * g.pos) * g.o_st + it.h * g.o_sh, min(g.pos, it.rows - t * g.pos),
                      nb > 0 ? tO : 0xFFFFFFFFu, inv, sOut + warp * kStageOut, row, bad);
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(item_empty + 8 * slot);      // the flags of this slot have been read
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8 && lane == 0) {
      // ------------------------------------------------ TMA producer
      pdl_wait();
      // a tile's rows: gp heads at each of its positions (rows past the box keep what they held)
      auto load_q = [&](const Item& it) {
        const int tiles = it.rows > g.pos ? 2 : 1;
        mbar_expect_tx(q_full, tiles * kPanels * g.gp * g.pos * 128);
        for (int x = 0; x < tiles * kPanels; ++x)
          tma_load_3d(smem_u32(sQ) + x * kPanel, &maps.q, q_full, 64 * (x % kPanels), it.h, it.q0 + x / kPanels * g.pos);
        ++q_loaded;
      };
      bool ok = true;
      for (uint32_t n = 0; ok && !*abort_flag; ++n) {
        const int slot = n % kItemRing;
        if (!wait_bar(ctl, item_empty + 8 * slot, ((n / kItemRing) & 1) ^ 1, kDevTimeoutTmaProducer)) break;
        const int item = atomicAdd(&sched[0], 1);
        if (item >= g.n_items) {
          s_items[slot].item = -1;
          mbar_arrive(item_full + 8 * slot);
          break;
        }
        const Item it = decode_item<SPLIT>(g, tab, item);
        const int* from = (const int*)&it;
        volatile int* to = (volatile int*)&s_items[slot];
#pragma unroll
        for (int i = 0; i < (int)(sizeof(Item) / 4); ++i) to[i] = from[i];
        mbar_arrive(item_full + 8 * slot);
        for (int b = 0; b < 2 * it.nb && ok; ++b) {
          if (b == 2) {
            // the queries after the first K and V blocks: the last item's products still read the old ones
            ok = wait_bar(ctl, q_empty, (q_loaded & 1) ^ 1, kDevTimeoutTmaProducer);
            if (!ok) break;
            load_q(it);
          }
          const int st = loaded % kStages;
          ok = wait_bar(ctl, kv_empty + 8 * st, ((loaded / kStages) & 1) ^ 1, kDevTimeoutTmaProducer);
          if (!ok) break;
          mbar_expect_tx(kv_full + 8 * st, kBlock);
          const CUtensorMap* map = (b & 1) ? &maps.v : &maps.k;
          const int tok = it.k0 + (it.nb - 1 - (b >> 1)) * kTile;
          for (int x = 0; x < kPanels; ++x)
            tma_load_3d(smem_u32(sKV) + st * kBlock + x * kPanel, map, kv_full + 8 * st, 64 * x, it.hk, tok);
          ++loaded;
        }
        if (ok && it.nb == 1) {                   // an item of one block: its queries come last
          ok = wait_bar(ctl, q_empty, (q_loaded & 1) ^ 1, kDevTimeoutTmaProducer);
          if (!ok) break;
          load_q(it);
        }
      }
    } else if (warp == 9 || warp == 10) {
      // ------------------------------------------------ MMA issuer of one tile (the whole warp, one elected lane at an issue)
      const int t = warp - 9;
      uint32_t qc = 0, pc = 0, tc = 0, okc = 0;   // query loads, P tiles, turns, and the parity of v_ok (a bit per stage)
      int st = 0;                                 // stage in turn and its parity
      uint32_t ph = 0;
      const uint32_t tS = tmem + t * kTile, tO = tmem + 256 + t * kTile;
      const uint64_t qdesc = sw128_desc(smem_u32(sQ) + t * kBlock, 16, 1024);
      const uint64_t kdesc = sw128_desc(smem_u32(sKV), 16, 1024), vdesc = sw128_desc(smem_u32(sKV), kPanel, 1024);
      // S = Q K^T for the K block in stage sk, O += P V for the V block in stage sv; the stages are released
      // with the products that read them
      auto scores = [&](int sk, bool pass) {
        const uint64_t kd = kdesc + sk * (kBlock >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kPanel + (kk & 3) * 32) >> 4;
          mma_ss(tS, qdesc + off, kd + off, idesc<kTile>(), kk > 0);
          if (kk == D / 16 - 3 && pass) mbar_arrive(turn + 8 * (t ^ 1));
        }
        commit(s_full + 8 * t);
        commit(kv_empty + 8 * sk);
      };
      auto values = [&](int sv, bool add) {
        const uint64_t vd = vdesc + sv * (kBlock >> 4);
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          mma_ts(tO, tS + 8 * kk, vd + ((kk * 2048) >> 4), idesc<D>() | kOuterMajorB, add || kk > 0);
        commit(kv_empty + 8 * sv);
      };
      // a block that this tile does not need: released only once it is there, so that the
      // release counts for this use of the stage
      auto skip = [&](int sx) { if (lane == 0) mbar_arrive(kv_empty + 8 * sx); };
      auto next = [&]() { if (++st == kStages) { st = 0; ph ^= 1; } };
      for (uint32_t n = 0; __all_sync(0xffffffffu, !*abort_flag); ++n) {
        const int slot = n % kItemRing;
        if (!wait_warp(ctl, item_full + 8 * slot, (n / kItemRing) & 1, kDevTimeoutMma)) break;
        struct { int item, nb, nb0, nb1, low; } it;
        it.item = __shfl_sync(0xffffffffu, s_items[slot].item, 0);
        it.nb = __shfl_sync(0xffffffffu, s_items[slot].nb, 0);
        it.nb0 = __shfl_sync(0xffffffffu, s_items[slot].nb0, 0);
        it.nb1 = __shfl_sync(0xffffffffu, s_items[slot].nb1, 0);
        it.low = __shfl_sync(0xffffffffu, s_items[slot].low, 0);
        if (lane == 0) mbar_arrive(item_empty + 8 * slot);
        if (it.item < 0) break;
        if (it.nb == 0) continue;
        const int nb = t ? it.nb1 : it.nb0;
        bool ok = wait_warp(ctl, kv_full + 8 * st, ph, kDevTimeoutMma) && wait_warp(ctl, q_full, qc & 1, kDevTimeoutMma);
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
          ok = wait_warp(ctl, kv_full + 8 * sv, ph, kDevTimeoutMma);
          if (ok && j < nb && j >= it.low) ok = wait_warp(ctl, v_ok + 8 * sv, (okc >> sv) & 1, kDevTimeoutMma);
          if (j >= it.low) okc ^= 1u << sv;
          next();
          const int sk = st;
          if (ok && j >= 1) {
            ok = wait_warp(ctl, kv_full + 8 * sk, ph, kDevTimeoutMma);
            next();
          }
          if (!ok) break;
          if (j < nb) {
            // the two tiles take turns, tile 0 first
            const bool both = j < min(it.nb0, it.nb1);
            if (both) {
              ok = wait_warp(ctl, turn + 8 * t, (tc & 1) ^ (t ^ 1), kDevTimeoutMma);
              ++tc;
            }
            ok = ok && wait_warp(ctl, p_full + 8 * t, pc & 1, kDevTimeoutMma);
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
      // ------------------------------------------------ check of the values that some row must not see
      uint32_t kv = 0;
      for (uint32_t n = 0; __all_sync(0xffffffffu, !*abort_flag); ++n) {
        const int slot = n % kItemRing;
        if (!wait_warp(ctl, item_full + 8 * slot, (n / kItemRing) & 1, kDevTimeoutEpilogue)) break;
        struct { int nb, low; } it;
        if (s_items[slot].item < 0) break;
        it.nb = s_items[slot].nb;
        it.low = s_items[slot].low;
        uint32_t* bad_keys = s_bad + slot * kMaxChecked * 4;
        for (int i = lane; i < kMaxChecked * 4; i += 32) bad_keys[i] = 0;
        __syncwarp();
        bool ok = true, any = false;
        // Every V block is waited for and released, checked or not: a phase that was left out could still be open
        // when a later one of its stage is waited for by parity, and one that this warp did not hold could be two
        // phases gone.
        for (int j = it.nb - 1; j >= 0 && ok; --j) {
          const uint32_t use = kv + 2 * (it.nb - 1 - j) + 1;
          const int st = use % kStages;
          ok = wait_warp(ctl, kv_full + 8 * st, (use / kStages) & 1, kDevTimeoutEpilogue);
          if (!ok) break;
          if (j < it.low) {
            if (lane == 0) mbar_arrive(kv_empty + 8 * st);
            continue;
          }
          uint4* blk = (uint4*)(sKV + st * kBlock);
          // 0 x + sum stays zero as long as every x is finite
          const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
          __nv_bfloat162 sum[4] = {zero, zero, zero, zero};
#pragma unroll 8
          for (int i = lane; i < kBlock / 16; i += 32) {
            const uint4 w = blk[i];
            sum[0] = __hfma2(*(const __nv_bfloat162*)&w.x, zero, sum[0]);
            sum[1] = __hfma2(*(const __nv_bfloat162*)&w.y, zero, sum[1]);
            sum[2] = __hfma2(*(const __nv_bfloat162*)&w.z, zero, sum[2]);
            sum[3] = __hfma2(*(const __nv_bfloat162*)&w.w, zero, sum[3]);
          }
          const __nv_bfloat162 all = __hadd2(__hadd2(sum[0], sum[1]), __hadd2(sum[2], sum[3]));
          const bool bad = (*(const uint32_t*)&all & 0x7FFF7FFFu) != 0;
          if (__any_sync(0xffffffffu, bad)) {
            any = true;
            for (int i = lane; i < kBlock / 16; i += 32) {
              uint4 w = blk[i];
              uint32_t* x = (uint32_t*)&w;
              bool hit = false;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if ((x[e] & 0x7F80u) == 0x7F80u) { x[e] &= 0xFFFF0000u; hit = true; }
                if ((x[e] & 0x7F800000u) == 0x7F800000u) { x[e] &= 0xFFFFu; hit = true; }
              }
              if (hit) {
                blk[i] = w;
                const int r = (i / 8) & (kTile - 1);          // rows of 128 bytes, whatever the swizzle
                atomicOr(&bad_keys[(j - it.low) * 4 + (r >> 5)], 1u << (r & 31));
              }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the products read it next
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(v_ok + 8 * st);
            mbar_arrive(kv_empty + 8 * st);
          }
        }
        if (!ok) break;
        kv += 2 * it.nb;
        __syncwarp();
        if (lane == 0) {
          s_any[slot] = any;
          if (it.nb > 0) mbar_arrive(checked + 8 * slot);
          mbar_arrive(item_empty + 8 * slot);
        }
      }
    }
  }

  // ------------------------------------------------ teardown
  __syncwarp();
  pdl_trigger();
  fence_before();
  __syncthreads();
  fence_after();
  if (threadIdx.x == 0) {
    // every producer of the launch has stopped claiming when the last CTA gets here
    __threadfence();
    if (atomicAdd(&sched[1], 1) == (int)gridDim.x - 1) {
      atomicExch(&sched[0], 0);
      atomicExch(&sched[1], 0);
    }
  }
  if (*abort_flag) {
    bool landed = true;
    if (warp == 8 && lane == 0) {
      for (uint32_t i = loaded > kStages ? loaded - kStages : 0; i < loaded; ++i)
        landed &= drain_phase(kv_full + 8 * (i % kStages), (i / kStages) & 1);
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

// The parts of a tile together: 32 columns of its 128 rows per CTA, two warps for 32 rows
// (16 columns each), a lane per row; the parts are added in order.
template <int D, int MAXB>
__global__ void __launch_bounds__(256)
join_kernel(const __grid_constant__ TcGeom g, const __grid_constant__ PrefillTable<MAXB> tab,
            __nv_bfloat16* __restrict__ out) {
  __shared__ __align__(16) uint8_t rows[kTile * 80];          // 64 bytes a row, 80 apart
  const int item = blockIdx.x >> 1, t = blockIdx.x & 1, c0 = blockIdx.y * 32;
  const Item it = decode_item<true>(g, tab, item);
  pdl_wait();
  if (it.s == 0 && t * g.pos < it.rows) {
    const int parts = t ? it.parts1 : it.parts0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = (warp & 3) * 32 + lane, c = c0 + (warp >> 2) * 16;
    const int64_t next = (int64_t)g.groups * 2 * part_floats<D>();
    const float* p0 = g.part + ((int64_t)item * 2 + t) * part_floats<D>();
    const float* ml = p0 + kTile * D + row;
    float M = -INFINITY, L = 0.f, o[16];
#pragma unroll 8
    for (int k = 0; k < parts; ++k) M = fmaxf(M, __ldcg(ml + k * next));
    const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = 0.f;
#pragma unroll 2
    for (int k = 0; k < parts; ++k) {
      const float m = __ldcg(ml + k * next), f = ex2((m - ref) * g.alpha - residual(m, g.alpha));
      const float* p = p0 + k * next + (warp & 3) * (D * 32) + c * 32 + lane;
      L = fmaf(__ldcg(ml + k * next + kTile), f, L);
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] = fmaf(__ldcg(p + 32 * i), f, o[i]);
    }
    // no visible key: zeros; logits that are all -inf: NaN
    const float inv = L != 0.f ? 1.f / L : it.limit + t * g.pos + ((row * g.inv_gp) >> 16) < 0 ? 0.f : NAN;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] *= inv;
    put8(rows + row * 80 + (warp >> 2) * 32, o);
    put8(rows + row * 80 + (warp >> 2) * 32 + 16, o + 8);
    __syncthreads();
    const int left = min(g.pos, it.rows - t * g.pos);         // positions of the tile that exist
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = i * 64 + (threadIdx.x >> 2), k = threadIdx.x & 3, pos = (r * g.inv_gp) >> 16;
      if (pos < left && c0 + k * 8 < g.d)
        *(uint4*)(out + (int64_t)(it.q0 + t * g.pos + pos) * g.o_st + (it.h + r - pos * g.gp) * g.o_sh + c0 + k * 8) =
            *(const uint4*)(rows + r * 80 + k * 16);
    }
  }
  pdl_trigger();
}

// ---------------------------------------------------------------- host side
using EncodeFn = PFN_cuTensorMapEncodeTiled_v12000;
EncodeFn encode_fn() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &qr) == cudaSuccess &&
        qr == cudaDriverEntryPointSuccess)
      fn = (EncodeFn)p;
  });
  return fn;
}

// [rows][heads][d] bf16 in boxes of 64 columns of some heads and rows; columns past d
// and rows past the end read as zeros.  The stride of an axis of extent 1 is unused.
bool encode(EncodeFn enc, CUtensorMap* map, const void* base, int d, int heads, int rows, int64_t st, int64_t sh,
            int box_heads, int box_rows) {
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {heads == 1 ? 16 : (cuuint64_t)sh * 2, rows == 1 ? 16 : (cuuint64_t)st * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool SPLIT, int MAXB>
cudaError_t launch(const TcMaps& maps, const TcGeom& g, const PrefillTable<MAXB>& tab, const void* v, void* out,
                   int32_t* err, int sms, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = raise_smem(prefill_tc_kernel<D, SPLIT, MAXB>, smem_bytes<D>(), done);
  if (e != cudaSuccess) return e;
  const cudaError_t run = launch_pdl(prefill_tc_kernel<D, SPLIT, MAXB>, dim3(std::min(g.n_items, sms)), dim3(kThreads),
                                     (size_t)smem_bytes<D>(), s, maps, g, tab, (const __nv_bfloat16*)v,
                                     (__nv_bfloat16*)out, err, err + kSchedWord);
  if (!SPLIT || run != cudaSuccess) return run;
  return launch_pdl(join_kernel<D, MAXB>, dim3(g.n_items * 2, (g.d + 31) / 32), dim3(256), 0, s, g, tab, (__nv_bfloat16*)out);
}

}  // namespace

// Query heads that share a tile, of the G of a KV head: the divisor of G that leaves the
// fewest of the tile's 128 rows empty, the largest one of those.
int prefill_tc_heads(int G) {
  int best = 1;
  for (int gp = 2; gp <= std::min(G, kTile); ++gp)
    if (G % gp == 0 && kTile / gp * gp >= kTile / best * best) best = gp;
  // a few empty rows are worth the sharing of keys and values
  for (int gp = best + 1; gp <= std::min(G, kTile); ++gp)
    if (G % gp == 0 && kTile / gp * gp >= 120) best = gp;
  return best;
}
// Positions of a work item (two tiles) and keys of a block.
int prefill_tc_rows(int G) { return 2 * (kTile / prefill_tc_heads(G)); }
int prefill_tc_block() { return kTile; }

// The workspace that split items need.
size_t prefill_tc_part_bytes(int64_t n_items, int d) {
  return (size_t)n_items * 2 * (d <= 64 ? part_floats<64>() : part_floats<128>()) * sizeof(float);
}

template <int MAXB>
cudaError_t launch_prefill_tc(const PrefillTable<MAXB>& tab, const PrefillGeom& p, int kb, int q_total, int k_total,
                              const void* q, const void* k, const void* v, void* out, int32_t* err, float* part,
                              int sms, cudaStream_t s) {
  const EncodeFn enc = encode_fn();
  if (enc == nullptr) return cudaErrorNotSupported;
  const int gp = prefill_tc_heads(p.G);
  static thread_local TcMaps maps;
  if (!encode(enc, &maps.q, q, p.d, p.Hq, q_total, p.q_st, p.q_sh, gp, kTile / gp) ||
      !encode(enc, &maps.k, k, p.d, p.Hkv, k_total, p.kv_st, p.kv_sh, 1, kTile) ||
      !encode(enc, &maps.v, v, p.d, p.Hkv, k_total, p.kv_st, p.kv_sh, 1, kTile))
    return cudaErrorInvalidValue;
  TcGeom g = {p.Hq / gp, p.G / gp, gp, (65536 + gp - 1) / gp, kTile / gp, p.d, kb, tab.uoff[tab.B] * (p.Hq / gp), p.alpha, p.kv_st, p.kv_sh, p.o_st, p.o_sh, 4000000000LL,
              part};
  if (kb > 0)
    return p.d <= 64 ? launch<64, true>(maps, g, tab, v, out, err, sms, s) : launch<128, true>(maps, g, tab, v, out, err, sms, s);
  return p.d <= 64 ? launch<64, false>(maps, g, tab, v, out, err, sms, s) : launch<128, false>(maps, g, tab, v, out, err, sms, s);
}
template cudaError_t launch_prefill_tc<kSmallBatch>(const PrefillTable<kSmallBatch>&, const PrefillGeom&, int, int, int,
                                                    const void*, const void*, const void*, void*, int32_t*,
                                                    float*, int, cudaStream_t);
template cudaError_t launch_prefill_tc<CHUNKKV_MAX_BATCH>(const PrefillTable<CHUNKKV_MAX_BATCH>&, const PrefillGeom&,
                                                          int, int, int, const void*, const void*, const void*, void*,
                                                          int32_t*, float*, int, cudaStream_t);

}  // namespace chunkkv
