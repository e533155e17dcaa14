// Attention over packed prompts on the tensor cores (tcgen05 + TMA + TMEM): bf16, head
// dimension up to 128.
//
//   O_i = sum_{j <= i + Tk - Tq} softmax_j(scale q_i . k_j) v_j
//
// A work item is one head's run of 256 query rows (two tiles of 128) of one sequence.
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
// each to do.  So the tensor cores bound it as long as the softmax keeps up.
//
// The reference m of a row is the maximum of the first block in which it sees a key, and
// stays while the row's sum is below 2^24: a common factor of P, O and the sum costs no
// precision (bf16 and fp32 have the same exponents) and the final division removes it.
// So a block has no maximum to find before its exponentials, and they need no more
// than 64 logits in registers at a time.  A block that passes the bound is done over
// with its maximum as the reference, O and the sum rescaled; S is still there, since
// P replaces it only after that test.
//
// The blocks are taken from the last one down: the masked ones come first.  P is zero
// where a key is hidden, but 0 x inf is NaN, and the values of hidden keys (later
// positions, the next sequence's rows) may hold anything.  So two checking warps look
// through the V of the masked blocks before the product and replace non-finite
// elements by zero; rows that do see such a key get the element added at the end.
//
// Warp roles: 0-3 and 4-7 softmax of tile 0 and 1, 8 TMA producer, 9 MMA issuer, 10 and
// 11 V check.  Every wait is bounded (tcgen.cuh); a CTA that gives up drains and exits.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "tcgen.cuh"

namespace chunkkv {
namespace {

using namespace tcgen;

constexpr int kTile = 128;                        // query rows of a tile, keys of a block
constexpr int kStages = 5;                        // K and V blocks in shared memory
constexpr int kItemRing = 2;
constexpr int kThreads = 384;                     // 12 warps, three warpgroups
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * 168, "register shares within the launch's");
constexpr int kMaxChecked = 4;                    // masked blocks of an item: 256 rows' limits span at most three
constexpr float kBig = 16777216.f;                // bound of a row's sum under its reference

template <int D> constexpr int block_bytes() { return kTile * D * 2; }
constexpr int kPanel = kTile * 128;               // 128 rows x 64 elements
template <int D> constexpr int smem_bytes() { return (2 + kStages) * block_bytes<D>() + 1024; }
template <int N> constexpr uint32_t idesc() {     // fp32 D, bf16 A and B, M = 128
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
constexpr uint32_t kOuterMajorB = 1u << 16;

struct TcGeom {
  int32_t Hq, G, d;
  int32_t rows;                                   // query rows of an item: 256, or 128 for few items
  int32_t n_items;
  float alpha;
  int64_t v_st, v_sh, o_st, o_sh;                 // element strides of v and out
  int32_t wide;                                   // out's rows are 32-byte aligned and d a multiple of 32
  long long timeout;
};
struct TcMaps { CUtensorMap q, k, v; };

struct Item {
  int h, hk;
  int q0, k0, tk;                                 // packed rows where the item's queries and the sequence's keys begin
  int rows;                                       // query rows that exist
  int limit;                                      // last key that the item's first row sees (may be negative)
  int nb0, nb1;                                   // key blocks of the two tiles
  int nb;                                         // blocks walked
  int low;                                        // blocks low .. nb - 1 hold keys hidden to some row
};

template <int MAXB>
__device__ __forceinline__ Item decode_item(const TcGeom& g, const PrefillTable<MAXB>& tab, int item) {
  Item it;
  const int u = item / g.Hq;
  it.h = item - u * g.Hq;
  it.hk = it.h / g.G;
  const int i = find_seq(tab, u);
  const PrefillSeq sq = tab.seq[i];
  const int r0 = (tab.uoff[i + 1] - 1 - u) * g.rows;        // later rows see more keys: they come first
  it.q0 = sq.q0 + r0;
  it.k0 = sq.k0;
  it.tk = sq.tk;
  it.rows = min(g.rows, sq.tq - r0);
  it.limit = r0 + sq.tk - sq.tq;
  const int last0 = it.limit + min(it.rows, kTile) - 1, last1 = it.limit + it.rows - 1;
  it.nb0 = last0 < 0 ? 0 : last0 / kTile + 1;
  it.nb1 = it.rows <= kTile || last1 < 0 ? 0 : last1 / kTile + 1;
  it.nb = max(it.nb0, it.nb1);
  it.low = max(it.limit + 1, 0) / kTile;
  return it;
}

// The first of the row's 32 columns at `first` that are hidden, and those after it.
template <bool MASK>
__device__ __forceinline__ float chunk_max(const float (&s)[32], int first, int seen, float m) {
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float a = !MASK || first + i <= seen ? s[i] : -INFINITY, b = !MASK || first + i + 1 <= seen ? s[i + 1] : -INFINITY;
    m = fmaxf(m, fmaxf(a, b));
  }
  return m;
}
// Row maximum over the columns 0 .. seen of S.
template <bool MASK>
__device__ __forceinline__ float row_max(uint32_t tS, int seen) {
  float ra[32], rb[32], m = -INFINITY;
  tmem_ld32(tS, ra);
  tmem_wait(ra);
  tmem_ld32(tS + 32, rb);
  m = chunk_max<MASK>(ra, 0, seen, m);
  tmem_wait(rb);
  tmem_ld32(tS + 64, ra);
  m = chunk_max<MASK>(rb, 32, seen, m);
  tmem_wait(ra);
  tmem_ld32(tS + 96, rb);
  m = chunk_max<MASK>(ra, 64, seen, m);
  tmem_wait(rb);
  return chunk_max<MASK>(rb, 96, seen, m);
}

// 32 columns of P from 32 of S: pairs by one packed FMA, two exponentials, a packed sum
// and a packed conversion.
template <bool MASK, int C>
__device__ __forceinline__ void chunk_exp(const float (&s)[32], float2 a2, float2 n2, int seen, float2 (&sum)[2],
                                          uint32_t (&p)[64]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 e = __ffma2_rn(make_float2(s[2 * i], s[2 * i + 1]), a2, n2);
    float2 w = make_float2(ex2(e.x), ex2(e.y));
    if (MASK) {                                               // whatever a hidden logit is
      w.x = 32 * C + 2 * i <= seen ? w.x : 0.f;
      w.y = 32 * C + 2 * i + 1 <= seen ? w.y : 0.f;
    }
    sum[i & 1] = __fadd2_rn(sum[i & 1], w);
    const __nv_bfloat162 b = __floats2bfloat162_rn(w.x, w.y);
    p[16 * C + i] = *(const uint32_t*)&b;
  }
}
// A row's P under the reference -neg, and its sum.
template <bool MASK>
__device__ __forceinline__ float row_exp(uint32_t tS, float alpha, float neg, int seen, uint32_t (&p)[64]) {
  float ra[32], rb[32];
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  const float2 a2 = make_float2(alpha, alpha), n2 = make_float2(neg, neg);
  tmem_ld32(tS, ra);
  tmem_wait(ra);
  tmem_ld32(tS + 32, rb);
  chunk_exp<MASK, 0>(ra, a2, n2, seen, sum, p);
  tmem_wait(rb);
  tmem_ld32(tS + 64, ra);
  chunk_exp<MASK, 1>(rb, a2, n2, seen, sum, p);
  tmem_wait(ra);
  tmem_ld32(tS + 96, rb);
  chunk_exp<MASK, 2>(ra, a2, n2, seen, sum, p);
  tmem_wait(rb);
  chunk_exp<MASK, 3>(rb, a2, n2, seen, sum, p);
  return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

template <int D, int MAXB>
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
  const uint32_t q_full = smem_u32(bars), q_empty = q_full + 8, drained = q_full + 16;
  const uint32_t s_full = q_full + 24, p_full = s_full + 16, o_full = p_full + 16;        // [2] each
  const uint32_t kv_full = o_full + 16, kv_empty = kv_full + 8 * kStages, v_ok = kv_empty + 8 * kStages;
  const uint32_t item_full = v_ok + 8 * kStages, item_empty = item_full + 8 * kItemRing;
  const uint32_t checked = item_empty + 8 * kItemRing;                                     // [kItemRing]
  constexpr int kBars = 3 + 6 + 3 * kStages + 3 * kItemRing;
  uint32_t* tmem_slot = (uint32_t*)(bars + kBars);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  volatile int* s_items = abort_flag + 1;                                                  // [kItemRing]
  uint32_t* s_bad = (uint32_t*)(s_items + kItemRing);     // [kItemRing][two warps][kMaxChecked][4] keys, a bit each
  static_assert(8 * kBars + 8 + 4 * kItemRing + 32 * kItemRing * kMaxChecked <= 1024, "control block");

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1); mbar_init(q_empty, 1); mbar_init(drained, 1);
    for (int t = 0; t < 2; ++t) { mbar_init(s_full + 8 * t, 1); mbar_init(p_full + 8 * t, 128); mbar_init(o_full + 8 * t, 1); }
    for (int i = 0; i < kStages; ++i) { mbar_init(kv_full + 8 * i, 1); mbar_init(kv_empty + 8 * i, 1); mbar_init(v_ok + 8 * i, 2); }
    // an item's slot is released by the MMA issuer, the checking warps and each softmax warp
    for (int i = 0; i < kItemRing; ++i) {
      mbar_init(item_full + 8 * i, 1); mbar_init(item_empty + 8 * i, 11); mbar_init(checked + 8 * i, 2);
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
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = lanes + t * kTile, tO = lanes + 256 + t * kTile;
    uint32_t sc = 0, oc = 0, cc = 0;              // phases of s_full, o_full and (a bit per slot) checked
    pdl_wait();
    for (uint32_t n = 0; __all_sync(0xffffffffu, !*abort_flag); ++n) {
      const int slot = n % kItemRing;
      if (!wait_warp(ctl, item_full + 8 * slot, (n / kItemRing) & 1, kDevTimeoutEpilogue)) break;
      const int item = s_items[slot];
      if (item < 0) break;
      const Item it = decode_item(g, tab, item);
      const int nb = t ? it.nb1 : it.nb0;
      const int limit = it.limit + t * kTile + row;           // last key that this row sees
      float m = -INFINITY, neg = 0.f, l = 0.f;                // the row's reference, -m alpha, and its sum
      bool ok = true;
      for (int j = nb - 1; j >= 0; --j) {
        if (!wait_warp(ctl, s_full + 8 * t, sc & 1, kDevTimeoutEpilogue)) { ok = false; break; }
        ++sc;
        fence_after();
        const int seen = limit - j * kTile;                   // columns 0 .. seen
        const bool masked = kTile - 1 > seen - lane;          // some key is hidden to the warp's first row
        if (__any_sync(0xffffffffu, m == -INFINITY)) {
          const float bm = masked ? row_max<true>(tS, seen) : row_max<false>(tS, seen);
          if (m == -INFINITY && bm != -INFINITY) {            // P and O of the row are zero so far
            m = bm;
            neg = -m * g.alpha;
          }
        }
        uint32_t p[64];
        float sum = masked ? row_exp<true>(tS, g.alpha, neg, seen, p) : row_exp<false>(tS, g.alpha, neg, seen, p);
        const bool over = !(l + sum <= kBig);                 // a NaN too
        if (__any_sync(0xffffffffu, over)) {
          const float bm = masked ? row_max<true>(tS, seen) : row_max<false>(tS, seen);
          const float mn = fmaxf(m, bm);
          const float f = over ? ex2((m - mn) * g.alpha) : 1.f;
          if (over) {
            m = mn;
            neg = -m * g.alpha;
          }
          l *= f;
          if (j < nb - 1) {
            // O holds the blocks before, all of them done: their products were issued before this S
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
          sum = masked ? row_exp<true>(tS, g.alpha, neg, seen, p) : row_exp<false>(tS, g.alpha, neg, seen, p);
        }
        l += sum;
        tmem_st32<0>(tS, p);
        tmem_st32<32>(tS + 32, p);
        tmem_st_wait();
        fence_before();
        mbar_arrive(p_full + 8 * t);
      }
      if (!ok) break;
      // ---- the item's rows
      const float inv = l == 0.f ? 0.f : 1.f / l;             // no visible key: zeros
      const bool live = t * kTile + row < it.rows;
      __nv_bfloat16* po = out + (int64_t)(it.q0 + t * kTile + row) * g.o_st + it.h * g.o_sh;
      bool flagged = false;
      if (it.nb > 0 && t * kTile < it.rows) {
        if (!wait_warp(ctl, checked + 8 * slot, (cc >> slot) & 1, kDevTimeoutEpilogue)) break;
        for (int c = 0; c < kMaxChecked * 8; ++c) flagged |= s_bad[slot * kMaxChecked * 8 + c] != 0;
      }
      if (it.nb > 0) cc ^= 1u << slot;
      if (nb > 0) {
        if (!wait_warp(ctl, o_full + 8 * t, oc & 1, kDevTimeoutEpilogue)) break;
        ++oc;
        fence_after();
      }
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        if (t * kTile >= it.rows || 32 * c >= g.d) break;     // the same for the whole warp
        float o[32];
        if (nb > 0) {
          tmem_ld32(tO + 32 * c, o);
          tmem_wait(o);
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = nb > 0 ? o[i] * inv : 0.f;
        if (flagged && live) {
          // non-finite values of visible keys, which the check took out of the products
          for (int k = 0; k < min(it.nb - it.low, kMaxChecked); ++k)
            for (int r = 0; r < kTile; ++r) {
              const int key = (it.low + k) * kTile + r;
              const uint32_t* bad = s_bad + slot * kMaxChecked * 8 + k * 4 + (r >> 5);
              if (key > limit || key >= it.tk || !((bad[0] | bad[kMaxChecked * 4]) >> (r & 31) & 1)) continue;
              const __nv_bfloat16* pv = v + (int64_t)(it.k0 + key) * g.v_st + it.hk * g.v_sh + 32 * c;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float x = 32 * c + i < g.d ? __bfloat162float(pv[i]) : 0.f;
                if ((__float_as_uint(x) & 0x7F800000u) == 0x7F800000u) o[i] += x;
              }
            }
        }
        if (live) {
#pragma unroll
          for (int i = 0; i < 32; i += 16) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(o[i + 2 * e], o[i + 2 * e + 1]);
              w[e] = *(const uint32_t*)&b;
            }
            // a lane per row: whole 32-byte sectors where the rows' alignment allows it
            if (g.wide) {
              asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(po + 32 * c + i), "r"(w[0]), "r"(w[1]),
                           "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
            } else {
              if (32 * c + i < g.d) *(uint4*)(po + 32 * c + i) = make_uint4(w[0], w[1], w[2], w[3]);
              if (32 * c + i + 8 < g.d) *(uint4*)(po + 32 * c + i + 8) = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        }
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
      bool ok = true;
      for (uint32_t n = 0; ok && !*abort_flag; ++n) {
        const int slot = n % kItemRing;
        if (!wait_bar(ctl, item_empty + 8 * slot, ((n / kItemRing) & 1) ^ 1, kDevTimeoutTmaProducer)) break;
        int item = atomicAdd(&sched[0], 1);
        if (item >= g.n_items) item = -1;
        s_items[slot] = item;
        mbar_arrive(item_full + 8 * slot);
        if (item < 0) break;
        const Item it = decode_item(g, tab, item);
        for (int b = 0; b < 2 * it.nb && ok; ++b) {
          if (b == 2) {
            // the queries after the first K and V blocks: the last item's products still read the old ones
            ok = wait_bar(ctl, q_empty, (q_loaded & 1) ^ 1, kDevTimeoutTmaProducer);
            if (!ok) break;
            const int tiles = it.rows > kTile ? 2 : 1;
            mbar_expect_tx(q_full, tiles * kBlock);
            for (int x = 0; x < tiles * kPanels; ++x)
              tma_load_3d(smem_u32(sQ) + x * kPanel, &maps.q, q_full, 64 * (x % kPanels), it.h,
                          it.q0 + x / kPanels * kTile);
            ++q_loaded;
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
          const int tiles = it.rows > kTile ? 2 : 1;
          mbar_expect_tx(q_full, tiles * kBlock);
          for (int x = 0; x < tiles * kPanels; ++x)
            tma_load_3d(smem_u32(sQ) + x * kPanel, &maps.q, q_full, 64 * (x % kPanels), it.h, it.q0 + x / kPanels * kTile);
          ++q_loaded;
        }
      }
    } else if (warp == 9) {
      // ------------------------------------------------ MMA issuer (the whole warp, one elected lane at each issue)
      uint32_t kv = 0, qc = 0, okc = 0, pc = 0;   // stages used, query loads; parities of v_ok (a bit per stage) and p_full
      const uint64_t qdesc = sw128_desc(smem_u32(sQ), 16, 1024);
      const uint64_t kdesc = sw128_desc(smem_u32(sKV), 16, 1024), vdesc = sw128_desc(smem_u32(sKV), kPanel, 1024);
      // S of tile t for the K block in stage st
      auto scores = [&](int t, int st) {
        if (elect_one()) {
          const uint64_t kd = kdesc + st * (kBlock >> 4), qd = qdesc + t * (kBlock >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * kPanel + (kk & 3) * 32) >> 4;
            mma_ss(tmem + t * kTile, qd + off, kd + off, idesc<kTile>(), kk > 0);
          }
          commit(s_full + 8 * t);
        }
        __syncwarp();
      };
      // O of tile t += P of the tile times the V block in stage st
      auto values = [&](int t, int st, bool add, bool last) {
        if (elect_one()) {
          const uint64_t vd = vdesc + st * (kBlock >> 4);
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            mma_ts(tmem + 256 + t * kTile, tmem + t * kTile + 8 * kk, vd + ((kk * 2048) >> 4), idesc<D>() | kOuterMajorB,
                   add || kk > 0);
          if (last) commit(o_full + 8 * t);
        }
        __syncwarp();
      };
      auto release = [&](uint32_t bar) {
        if (elect_one()) commit(bar);
        __syncwarp();
      };
      for (uint32_t n = 0; __all_sync(0xffffffffu, !*abort_flag); ++n) {
        const int slot = n % kItemRing;
        if (!wait_warp(ctl, item_full + 8 * slot, (n / kItemRing) & 1, kDevTimeoutMma)) break;
        const int item = __shfl_sync(0xffffffffu, s_items[slot], 0);
        if (lane == 0) mbar_arrive(item_empty + 8 * slot);
        if (item < 0) break;
        const Item it = decode_item(g, tab, item);
        if (it.nb == 0) continue;
        if (!wait_warp(ctl, q_full, qc & 1, kDevTimeoutMma)) break;
        ++qc;
        int st = kv % kStages;
        if (!wait_warp(ctl, kv_full + 8 * st, (kv / kStages) & 1, kDevTimeoutMma)) break;
        fence_after();
        if (it.nb - 1 < it.nb0) scores(0, st);
        if (it.nb - 1 < it.nb1) scores(1, st);
        release(kv_empty + 8 * st);
        ++kv;
        if (it.nb == 1) release(q_empty);
        bool ok = true;
        for (int j = it.nb - 1; j >= 0; --j) {
          const int sv = kv % kStages, sk = (kv + 1) % kStages;
          ok = wait_warp(ctl, kv_full + 8 * sv, (kv / kStages) & 1, kDevTimeoutMma);
          if (ok && j >= it.low) {
            ok = wait_warp(ctl, v_ok + 8 * sv, (okc >> sv) & 1, kDevTimeoutMma);
            okc ^= 1u << sv;
          }
          if (ok && j >= 1) ok = wait_warp(ctl, kv_full + 8 * sk, ((kv + 1) / kStages) & 1, kDevTimeoutMma);
          if (!ok) break;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int nb = t ? it.nb1 : it.nb0;
            if (j < nb) {
              ok = wait_warp(ctl, p_full + 8 * t, (pc >> t) & 1, kDevTimeoutMma);
              if (!ok) break;
              pc ^= 1u << t;
              fence_after();
              values(t, sv, j < nb - 1, j == 0);
            }
            if (j >= 1 && j - 1 < nb) {
              fence_after();
              scores(t, sk);
            }
          }
          if (!ok) break;
          release(kv_empty + 8 * sv);
          ++kv;
          if (j >= 1) {
            release(kv_empty + 8 * sk);
            ++kv;
            if (j == 1) release(q_empty);
          }
        }
        if (!ok) break;
      }
    } else if (warp >= 10) {
      // ------------------------------------------------ check of the values that some row must not see
      uint32_t kv = 0;
      for (uint32_t n = 0; __all_sync(0xffffffffu, !*abort_flag); ++n) {
        const int slot = n % kItemRing;
        if (!wait_warp(ctl, item_full + 8 * slot, (n / kItemRing) & 1, kDevTimeoutEpilogue)) break;
        const int item = s_items[slot];
        if (item < 0) break;
        const Item it = decode_item(g, tab, item);
        uint32_t* bad_keys = s_bad + (slot * 2 + warp - 10) * kMaxChecked * 4;
        for (int i = lane; i < kMaxChecked * 4; i += 32) bad_keys[i] = 0;
        __syncwarp();
        bool ok = true;
        for (int j = it.nb - 1; j >= it.low && ok; --j) {
          const uint32_t use = kv + 2 * (it.nb - 1 - j) + 1;
          const int st = use % kStages;
          ok = wait_warp(ctl, kv_full + 8 * st, (use / kStages) & 1, kDevTimeoutEpilogue);
          if (!ok) break;
          uint4* blk = (uint4*)(sKV + st * kBlock);           // a half for each of the two warps
          const int i0 = (warp - 10) * (kBlock / 32) + lane, i1 = (warp - 9) * (kBlock / 32);
          uint32_t top = 0;
#pragma unroll 8
          for (int i = i0; i < i1; i += 32) {
            const uint4 w = blk[i];
            top = __vmaxu2(top, __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                         __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu)));
          }
          const bool bad = (top & 0xFFFFu) >= 0x7F80u || (top >> 16) >= 0x7F80u;
          if (__any_sync(0xffffffffu, bad)) {
            for (int i = i0; i < i1; i += 32) {
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
          if (lane == 0) mbar_arrive(v_ok + 8 * st);
        }
        if (!ok) break;
        kv += 2 * it.nb;
        __syncwarp();
        if (lane == 0) {
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
    if (warp == 9) {
      if (elect_one()) commit(drained);
      __syncwarp();
      landed &= drain_phase(drained, 0);
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

// [rows][heads][d] bf16 in boxes of 128 rows x 64 columns of one head; columns past d
// and rows past the end read as zeros.  The stride of an axis of extent 1 is unused.
bool encode(EncodeFn enc, CUtensorMap* map, const void* base, int d, int heads, int rows, int64_t st, int64_t sh) {
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {heads == 1 ? 16 : (cuuint64_t)sh * 2, rows == 1 ? 16 : (cuuint64_t)st * 2};
  cuuint32_t box[3] = {64, 1, kTile};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int MAXB>
cudaError_t launch(const TcMaps& maps, const TcGeom& g, const PrefillTable<MAXB>& tab, const void* v, void* out,
                   int32_t* err, int sms, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = raise_smem(prefill_tc_kernel<D, MAXB>, smem_bytes<D>(), done);
  if (e != cudaSuccess) return e;
  return launch_pdl(prefill_tc_kernel<D, MAXB>, dim3(std::min(g.n_items, sms)), dim3(kThreads), (size_t)smem_bytes<D>(), s,
                    maps, g, tab, (const __nv_bfloat16*)v, (__nv_bfloat16*)out, err, err + kSchedWord);
}

}  // namespace

// Query rows of a work item.
int prefill_tc_rows() { return 2 * kTile; }

template <int MAXB>
cudaError_t launch_prefill_tc(const PrefillTable<MAXB>& tab, const PrefillGeom& p, int rows, int q_total, int k_total,
                              const void* q, const void* k, const void* v, void* out, int32_t* err, int sms,
                              cudaStream_t s) {
  const EncodeFn enc = encode_fn();
  if (enc == nullptr) return cudaErrorNotSupported;
  static thread_local TcMaps maps;
  if (!encode(enc, &maps.q, q, p.d, p.Hq, q_total, p.q_st, p.q_sh) ||
      !encode(enc, &maps.k, k, p.d, p.Hkv, k_total, p.kv_st, p.kv_sh) ||
      !encode(enc, &maps.v, v, p.d, p.Hkv, k_total, p.kv_st, p.kv_sh))
    return cudaErrorInvalidValue;
  TcGeom g = {p.Hq, p.G, p.d, rows, tab.uoff[tab.B] * p.Hq, p.alpha, p.kv_st, p.kv_sh, p.o_st, p.o_sh,
              p.d % 32 == 0 && p.o_st % 16 == 0 && p.o_sh % 16 == 0 && (uintptr_t)out % 32 == 0, 4000000000LL};
  if (p.d <= 64) return launch<64, MAXB>(maps, g, tab, v, out, err, sms, s);
  return launch<128, MAXB>(maps, g, tab, v, out, err, sms, s);
}
template cudaError_t launch_prefill_tc<kSmallBatch>(const PrefillTable<kSmallBatch>&, const PrefillGeom&, int, int, int,
                                                    const void*, const void*, const void*, void*, int32_t*, int,
                                                    cudaStream_t);
template cudaError_t launch_prefill_tc<CHUNKKV_MAX_BATCH>(const PrefillTable<CHUNKKV_MAX_BATCH>&, const PrefillGeom&,
                                                          int, int, int, const void*, const void*, const void*, void*,
                                                          int32_t*, int, cudaStream_t);

}  // namespace chunkkv
