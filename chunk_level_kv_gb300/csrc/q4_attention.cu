// Attention of a few query tokens over the 4-bit paged cache.
//
//   O = sum_j p_j V_j / sum_j p_j,   p_j = 2^(t_j - max t),   t_j = scale log2(e) (q . K_j)
//
// over the tokens j of one cache row that a query sees, with K_j = s c + m for each group of
// 64 columns (c: its codes 0 .. 15; s, m: its step and smallest value), and V_j alike.  So
//   q . K_j = sum over groups of s (q . c) + m sum(q),   O = sum_j (p_j s) c + sum_j p_j m
// and only the codes meet the tensor cores.
//
// What bounds it: every page is read once (9 bits for each key-value pair of elements), HBM.
// The arithmetic must keep out of the way: at 6.8 TB/s an SM receives 40 codes a clock, three
// instruction slots for each.  A code c as the low bits of a 16-bit word is the f16 number
// c 2^-24, exactly (a subnormal), and 4 bits higher c 2^-20: so a mask turns a 32-bit word's
// nibbles into f16 pairs, 5 instructions for 8 codes, and the other operand's elements that
// meet the higher ones are divided by 16 beforehand.  The products are m16n8k16 in f16 with
// fp32 sums; tcgen05 would want the codes expanded in shared memory, 4 times their bytes.
//   S^T = K Q^T and O^T = V^T P^T: the codes are the operand of 16 rows both times, 8 query rows
//   the one of 8 columns, so no product is spent on rows that do not exist.  A lane's logits are
//   2 query rows of 8 tokens; the weights p s change lanes for the second product as 8 x 8 f16
//   matrices transposed by the warp.  (With the query as the operand of 16 rows, half of them
//   zeros, the first product and its registers cost 300 of 1200 instructions a page.)
//   bf16: 8 query rows, or 16 as two sets of columns.  A query in f16, scaled by a power of two,
//         loses only what is below 2^-25 of its largest element; the weights p s are rounded to
//         f16, 2^-11 each, where the output's rounding is 2^-8.  Sums of products with subnormals
//         are good to about 2^-17 of their largest term (the unit aligns them by the exponent that
//         a subnormal is stored with).
//   fp32: 8 query rows; queries and weights as two f16 each (22 bits), in two products.  The codes
//         are made whole numbers c - 8 (m becomes m + 8 s), 11 instructions for 8 codes; with
//         subnormals the output was off by 60e-6.  The second product's sums are a page's, and added up in fp32.
//
// A weight p s is held as a multiple of the largest p s of its row so far (2^d times 2^max t), so
// that f16 holds it however far apart the steps of a row lie.
//
// Work split and join of a row's parts: as for the 8-bit cache (decode.cuh, q8_attention.cu).  A
// warp holds one page, whose keys and values are copied again as soon as each has been read.
//
// Measured: 64 sequences x 4 KV heads of 12 to 13 thousand tokens, 7 heads each (0.47 GB) 96 us,
// 4.9 TB/s, 72 % of a copy's rate (1050 instructions a page; issue slots 57 %, integer pipe 56 %,
// tensor pipe 26 %: with three warps a scheduler, latency); one sequence of 8 KV heads x 6.5 thousand
// tokens 12.6 us, 16 sequences of 256 to 300 tokens 8.1 us (latency).  Cold: 64 rows of 6.5 thousand
// tokens 35 us for 8 query rows, 48 us for 16; 256 rows of 6.5 thousand, 7 heads, 95 us at 192 columns
// (3.8 TB/s), 117 us at 256 (4.1), 103 us in fp32 at 128 (2.3).
#include <algorithm>
#include <type_traits>

#include "decode.cuh"
#include "q4.cuh"

namespace chunkkv {
namespace {

using namespace decode;

constexpr int kMaxGrid = 224;                    // CTAs of a pass (one per SM): a count for each in the header
constexpr int kMaxGroups = 16;                   // passes in one launch
constexpr int kCountByte = 32;                   // the counts of parts that have arrived, as decode attention's (q8_attention.cu)
static_assert(kCountByte + kMaxGrid * kMaxGroups <= (int)kServeHeader, "the counts lie in the serving header");
constexpr float kWeightExp = 12.f, kSlack = 3.f;  // the largest weight is 2^12 when O's unit is set, and 2^15 at most (f16 ends at 2^16)
// Rows that take the warps up to this many rounds are not cut: joining parts costs a call about 4 us, a round 1.
// (128 rows of 12 pages 10.6 us, cut from 8 pages on 20 us; 512 rows of 24 to 30 pages 47 and 52 us.)
constexpr int kWholeRounds = 3;
static_assert(kWholeRounds * 8 > 2 * kNearEnd, "a row's two ends do not meet");
constexpr int kQueryExp = 14;                    // the largest query element is in [2^14, 2^15)

struct Q4AttnArgs {
  const void* q;
  void* out;
  int64_t q_sb, q_st, q_sh, o_sb, o_st, o_sh;
  float alpha;                                   // scale * log2(e)
  int32_t G, n_q, p0;                            // query heads per KV head, query tokens, the first row of this launch
  const int32_t* q_lens;                         // query tokens of each sequence, or null: n_q
  int32_t* err;                                  // the workspace header: error word, counts of arrived parts
  float* part;                                   // [passes][2 CTAs][rows][64 ND + 4]: O, m, l
};

// Warps of a CTA, a page each in shared memory.  For 8 query rows of up to 128 columns twelve, of 168 registers a thread and
// 40 bytes spilled (256 rows of 12.8 thousand tokens, cold: 107 us; sixteen of 128 spill more, 121 us; eight 119 us); more
// rows or columns take the registers of eight (16 rows of 128 columns spill 60 bytes there, 256 columns 36, in fp32 28).
template <int ND, typename T, int RS>
constexpr int warps_of() { return sizeof(T) == 2 && RS == 1 && ND <= 2 ? 12 : 8; }
template <int ND>
constexpr int pitch() { return 64 * ND + 4; }    // O, m, l: in 16-byte rows
template <int ND>
constexpr bool q_in_regs() { return ND <= 2; }   // wider heads keep their query fragments in shared memory
template <int ND, typename T, int RS>
constexpr size_t smem_bytes() {
  return (size_t)warps_of<ND, T, RS>() * (q4_page_bytes(ND) + 8 * RS * pitch<ND>() * 4) + (q_in_regs<ND>() ? 0 : 2 * ND * 4 * 32 * 8);
}
// The halves of a page, each with its steps: two copies, and two barriers.
constexpr int half_bytes(int nd) { return q4_v(nd); }
static_assert(2 * half_bytes(1) == q4_page_bytes(1), "keys and values take the same room");

// Four codes of a word, of its items 4 h .. 4 h + 3, as two f16 pairs.
template <bool kExact>
__device__ __forceinline__ void codes_to_f16(uint32_t w, int h, uint32_t& lo, uint32_t& hi) {
  if constexpr (kExact) {                        // c - 8: a code below 1024's last bits, less 1032
    const uint32_t a = (w >> (8 * h) & 0x000F000Fu) | 0x64006400u, b = (w >> (8 * h + 4) & 0x000F000Fu) | 0x64006400u;
    const __half2 k = __halves2half2(__ushort_as_half(0x6408), __ushort_as_half(0x6408));
    const __half2 x = __hsub2(*(const __half2*)&a, k), y = __hsub2(*(const __half2*)&b, k);
    lo = *(const uint32_t*)&x;
    hi = *(const uint32_t*)&y;
  } else {                                       // c 2^-24 and c 2^-20
    w >>= 8 * h;
    lo = w & 0x000F000Fu;
    hi = w & 0x00F000F0u;
  }
}
// What code 0 (or code 8, kExact) stands for.
template <bool kExact>
__device__ __forceinline__ float base_of(uint32_t ms) {
  return kExact ? fmaf(q4_s(ms), 8.f, q4_m(ms)) : q4_m(ms);
}
// An 8 x 8 matrix of f16 transposed: lane (gid, t) held row gid, columns 2 t and 2 t + 1, and gets column gid, rows 2 t, 2 t + 1.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// D = A B (decode.cuh: D += A B).
__device__ __forceinline__ void mma16816_first(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The sequence's query tokens, kept inside what the query tensor holds.
__device__ __forceinline__ int queries_of(const Q4AttnArgs& a, int b) {
  return a.q_lens ? min(max(a.q_lens[b], 0), a.n_q) : a.n_q;
}

template <int ND, typename T, int RS>
__global__ void __launch_bounds__(32 * warps_of<ND, T, RS>(), 1)
q4_attention_kernel(Q4Geom g, Q4AttnArgs a, const uint8_t* __restrict__ pages, const int32_t* __restrict__ table,
                    const int32_t* __restrict__ lens) {
  constexpr int W = warps_of<ND, T, RS>(), kThreads = 32 * W, kBytes = q4_page_bytes(ND), kHalf = half_bytes(ND);
  constexpr int kPitch = pitch<ND>(), PR = 8 * RS;
  constexpr bool kSplit = sizeof(T) == 4;        // queries and weights in two parts
  static_assert(!kSplit || RS == 1, "two parts take the place of two sets of rows");
  constexpr int NB = kSplit ? 2 : RS;            // operands of 8 columns
  constexpr int kCodeExp = kSplit ? 0 : 24;      // a code is c 2^-kCodeExp, or c - 8
  constexpr float kSecond = kSplit ? 1.f : 0.0625f;            // of what meets the second pair of codes
  constexpr int KS = 4 * ND;                     // k steps of a logit, 16 columns each
  constexpr int MT = 4 * ND;                     // 16-column tiles of the output
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[2 * W];
  __shared__ RunShared<W> run;
  __shared__ int s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, t4 = lane & 3;
  const int my_token = 16 * (gid >> 1) + (gid & 1);
  uint8_t* pg = smem + warp * kBytes;
  float* sM = (float*)(smem + W * kBytes);       // [W][PR][kPitch]
  uint2* sQ = (uint2*)(sM + W * PR * kPitch);    // [NB][KS][32], one for all warps: they work on one cache row at a time
  const uint32_t kbar = smem_u32(&bars[2 * warp]), vbar = kbar + 8;
  if (lane == 0) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(kbar) : "memory");
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(vbar) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  pdl_wait();

  const Run plan = plan_run<W>(g, lens, run, kWholeRounds * W);
  const int64_t nc = plan.nc;
  const int p0 = a.p0 + blockIdx.y * PR, gn = min(PR, a.n_q * a.G - p0);
  auto out_at = [&](int b, int h, int row) {     // where row `row` of the pass is written
    const int i = (p0 + row) / a.G;
    return (T*)a.out + b * a.o_sb + i * a.o_st + (int64_t)(h * a.G + p0 + row - i * a.G) * a.o_sh;
  };
  // cache rows without a token
  for (int r = blockIdx.x; r < g.rows; r += gridDim.x)
    if (lens[r] <= 0) {
      const int live = min(gn, queries_of(a, r / g.Hkv) * a.G - p0);
      for (int i = tid; i < live * g.d; i += kThreads) store1(out_at(r / g.Hkv, r % g.Hkv, i / g.d) + i % g.d, 0.f);
    }
  __syncthreads();
  const int64_t x0 = run.cut[0], x1 = run.cut[1];
  if (x0 >= x1) {
    pdl_trigger();
    return;
  }

  // ---- this warp's pages are x0 + warp + W i
  Cursor cur;
  cur.base = run.row[0];
  cur.start = run.start[0];
  cur.load(g, lens, lane);
  auto page_at = [&](int64_t x) {
    int row, j, n;
    cur.locate(g, lens, lane, x, row, j, n);
    return safe_page(table[(int64_t)row * g.max_pages + j], g.n_pages);
  };
  int64_t x = x0 + warp;
  bool dead = false;
  uint32_t phase = 0;
  if (x < x1) {
    const uint8_t* src = pages + page_at(x) * kBytes;
    if (lane == 0) {
      copy_page(smem_u32(pg), src, kHalf, kbar);
      copy_page(smem_u32(pg) + kHalf, src + kHalf, kHalf, vbar);
    }
  }

  int r = run.row[0];                            // segment by segment: the CTA's part of cache row r
  int64_t xr = run.start[0];
  while (true) {
    const int len = safe_len(lens[r], g.max_pages), np = pages_of(len);
    const int64_t sa = xr > x0 ? xr : x0, sb = xr + np < x1 ? xr + np : x1;
    const int b = r / g.Hkv, h = r % g.Hkv, nq = queries_of(a, b);
    if (sa < sb) {
      // the query's fragments: columns 64 p + 16 t + 4 kk .. + 3 meet the items 4 (kk & 1) .. + 3 of the words that lane
      // t reads
      // its rows are gid (+ 8); what the logits need of them goes to the lanes that hold rows 2 t, 2 t + 1
      float ca[RS][2], cb[RS][2][ND];            // t = ca sum_g s acc + sum_g cb base
      int seen[RS][2];                           // tokens that the row's query sees
      uint2 qf[NB][q_in_regs<ND>() ? KS : 1];
      int seen_min = len;
#pragma unroll
      for (int rs = 0; rs < RS; ++rs) {
        const int row = gid + 8 * rs, i = (p0 + row) / a.G;
        const bool live = row < gn && i < nq;
        const int sees = live ? len - nq + 1 + i : len;
        seen_min = min(seen_min, sees);
        const T* q = (const T*)a.q + b * a.q_sb + i * a.q_st + (int64_t)(h * a.G + p0 + row - i * a.G) * a.q_sh;
        float qv[KS][4];
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const int c = (s >> 2) * 64 + t4 * 16 + (s & 3) * 4;
          qv[s][0] = qv[s][1] = qv[s][2] = qv[s][3] = 0.f;
          if (live && c < g.d) load4f(q + c, qv[s]);
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(qv[s][e]) & 0x7FFFFFFFu);
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // scaled by a power of two into f16's range, whatever the query's size
        const int e2 = min(127, max(-110, (int)(top >> 23) - 127));
        const float down = power_of_two(kQueryExp - e2);
        constexpr float kUp = kSplit ? 1.f / (1 << kQueryExp) : 1 << (24 - kQueryExp);
        const float c0 = fminf(a.alpha * power_of_two(e2) * kUp, 3.4e38f);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          ca[rs][e] = __shfl_sync(0xffffffffu, c0, 8 * t4 + 4 * e);
          seen[rs][e] = __shfl_sync(0xffffffffu, sees, 8 * t4 + 4 * e);
        }
#pragma unroll
        for (int p = 0; p < ND; ++p) {
          float sum = 0.f;
#pragma unroll
          for (int s = 4 * p; s < 4 * p + 4; ++s) sum += (qv[s][0] + qv[s][1]) + (qv[s][2] + qv[s][3]);
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          sum *= a.alpha;
#pragma unroll
          for (int e = 0; e < 2; ++e) cb[rs][e][p] = __shfl_sync(0xffffffffu, sum, 8 * t4 + 4 * e);
        }
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const float x0 = qv[s][0] * down, x1 = qv[s][1] * down, x2 = qv[s][2] * down * kSecond, x3 = qv[s][3] * down * kSecond;
          uint2 f[2];
          if constexpr (kSplit) {
            split_half2(x0, x1, 1.f, f[0].x, f[1].x);
            split_half2(x2, x3, 1.f, f[0].y, f[1].y);
          } else {
            f[0] = make_uint2(pack_half2(x0, x1), pack_half2(x2, x3));
          }
#pragma unroll
          for (int k = 0; k < (kSplit ? 2 : 1); ++k) {
            if constexpr (q_in_regs<ND>()) qf[rs + k][s] = f[k]; else sQ[((rs + k) * KS + s) * 32 + lane] = f[k];
          }
        }
      }
      __syncwarp();
      seen_min = __reduce_min_sync(0xffffffffu, seen_min);
      // of rows 2 t, 2 t + 1: reference, sum, O's unit as an exponent of 2 above the reference, sum of p base (sums: this lane's)
      float m[RS][2], l[RS][2], dl[RS][2], z[RS][2][ND];
#pragma unroll
      for (int rs = 0; rs < RS; ++rs)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m[rs][e] = dl[rs][e] = -INFINITY;
          l[rs][e] = 0.f;
#pragma unroll
          for (int p = 0; p < ND; ++p) z[rs][e][p] = 0.f;
        }
      float o[RS][MT][4];                        // O^T: columns 16 i + gid (+ 8: elements 2, 3) of rows 2 t, 2 t + 1
#pragma unroll
      for (int rs = 0; rs < RS; ++rs)
#pragma unroll
        for (int i = 0; i < MT; ++i) o[rs][i][0] = o[rs][i][1] = o[rs][i][2] = o[rs][i][3] = 0.f;

      while (x < sb) {
        const int64_t nx = x + W;
        const bool more = nx < x1;
        // the page to come: mostly of this row
        const int64_t next = nx < sb ? safe_page(table[(int64_t)r * g.max_pages + (nx - xr)], g.n_pages) : more ? page_at(nx) : 0;
        wait_copy(kbar, phase, dead, a.err);
        // ---- t.  Rows gid and gid + 8 of tile i are tokens 4 i + 16 (gid / 2) + gid % 2 and the second after it: transposed
        // by eights, lane t then holds tokens 16 t + 2 j + e, as its pieces of V
        float t[RS][8][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float acc[NB][ND][4];
          uint32_t kw[2][2 * ND];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint8_t* src = pg + (my_token + 4 * i + 2 * y) * (32 * ND) + t4 * (8 * ND);
            if constexpr (ND % 2 == 0) {
#pragma unroll
              for (int p = 0; p < ND / 2; ++p) {
                const uint4 w = *(const uint4*)(src + 16 * p);
                kw[y][4 * p] = w.x; kw[y][4 * p + 1] = w.y; kw[y][4 * p + 2] = w.z; kw[y][4 * p + 3] = w.w;
              }
            } else {
#pragma unroll
              for (int p = 0; p < ND; ++p) {
                const uint2 w = *(const uint2*)(src + 8 * p);
                kw[y][2 * p] = w.x; kw[y][2 * p + 1] = w.y;
              }
            }
          }
#pragma unroll
          for (int p = 0; p < ND; ++p)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              uint4 c;
              codes_to_f16<kSplit>(kw[0][2 * p + (s >> 1)], s & 1, c.x, c.z);
              codes_to_f16<kSplit>(kw[1][2 * p + (s >> 1)], s & 1, c.y, c.w);
#pragma unroll
              for (int k = 0; k < NB; ++k) {
                uint2 f;
                if constexpr (q_in_regs<ND>()) f = qf[k][4 * p + s]; else f = sQ[(k * KS + 4 * p + s) * 32 + lane];
                float (&d)[4] = acc[kSplit ? 0 : k][p];
                if (s == 0 && (!kSplit || k == 0)) mma16816_first(d, c, f.x, f.y); else mma16816(d, c, f.x, f.y);
              }
            }
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float sum[RS][2], off[RS][2];
#pragma unroll
            for (int p = 0; p < ND; ++p) {
              const uint32_t ms = *(const uint32_t*)(pg + q4_k_ms(ND) + (p * kPage + my_token + 4 * i + 2 * y) * 4);
              const float st = q4_s(ms), base = base_of<kSplit>(ms);
#pragma unroll
              for (int rs = 0; rs < RS; ++rs)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  sum[rs][e] = p == 0 ? acc[rs][p][2 * y + e] * st : fmaf(acc[rs][p][2 * y + e], st, sum[rs][e]);
                  off[rs][e] = p == 0 ? cb[rs][e][p] * base : fmaf(cb[rs][e][p], base, off[rs][e]);
                }
            }
#pragma unroll
            for (int rs = 0; rs < RS; ++rs)
#pragma unroll
              for (int e = 0; e < 2; ++e) t[rs][2 * i + y][e] = fmaf(sum[rs][e], ca[rs][e], off[rs][e]);
          }
        }
        __syncwarp();                            // every lane has read the keys
        if (more && lane == 0 && !dead) copy_page(smem_u32(pg), pages + next * kBytes, kHalf, kbar);
        wait_copy(vbar, phase, dead, a.err);
        // ---- weights p s and their largest, the reference, O's unit; the second product's operands
        uint32_t pb[NB][ND][8];
        auto weigh = [&](auto masked_c) {
          constexpr bool kMasked = decltype(masked_c)::value;
          const int at = (int)(x - xr) * kPage + my_token;    // the row's token that this lane holds first
          uint32_t vms[ND][8];
#pragma unroll
          for (int p = 0; p < ND; ++p)
#pragma unroll
            for (int j = 0; j < 8; ++j) vms[p][j] = *(const uint32_t*)(pg + q4_v_ms(ND) + (p * kPage + my_token + 2 * j) * 4);
#pragma unroll
          for (int rs = 0; rs < RS; ++rs) {
            float f[2], u[2] = {0.f, 0.f}, had[2], fl[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int left = seen[rs][e] - at;
              float top = -INFINITY;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                if (kMasked && 2 * j >= left) t[rs][j][e] = -INFINITY;
                top = fmaxf(top, t[rs][j][e]);
              }
#pragma unroll
              for (int x4 = 4; x4 < 32; x4 <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x4));
              const float mn = fmaxf(m[rs][e], top), ref = mn == -INFINITY ? 0.f : mn;
              const float drop = m[rs][e] == -INFINITY ? 0.f : mn - m[rs][e];
              fl[e] = ex2(-drop);
              had[e] = dl[rs][e] - drop;
              m[rs][e] = mn;
              float sum = 0.f;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                t[rs][j][e] = ex2(t[rs][j][e] - ref);
                sum += t[rs][j][e];
              }
              l[rs][e] = fmaf(l[rs][e], fl[e], sum);
              // the largest p s, of which hidden tokens have none whatever their steps are
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                float st = q4_s(vms[0][j]);
#pragma unroll
                for (int p = 1; p < ND; ++p) st = fmaxf(st, q4_s(vms[p][j]));
                u[e] = fmaxf(u[e], kMasked && 2 * j >= left ? 0.f : t[rs][j][e] * st);
              }
#pragma unroll
              for (int p = 0; p < ND; ++p) {
                float off = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) off = fmaf(t[rs][j][e], kMasked && 2 * j >= left ? 0.f : base_of<kSplit>(vms[p][j]), off);
                z[rs][e][p] = fmaf(z[rs][e][p], fl[e], off);
              }
            }
#pragma unroll
            for (int x4 = 4; x4 < 32; x4 <<= 1) {
              u[0] = fmaxf(u[0], __shfl_xor_sync(0xffffffffu, u[0], x4));
              u[1] = fmaxf(u[1], __shfl_xor_sync(0xffffffffu, u[1], x4));
            }
            // O's unit, 2^dl of the reference's: never smaller than it was, and set anew once the largest weight asks for
            // more than kSlack above it
            bool moved = false;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float need = u[e] > 0.f ? fmaxf(lg2(u[e]), -112.f) : -INFINITY;
              dl[rs][e] = need > had[e] + kSlack ? need : had[e];
              moved |= dl[rs][e] != had[e];
              f[e] = ex2(fminf(kWeightExp - dl[rs][e], 126.f));
            }
            if (__any_sync(0xffffffffu, moved)) {
              const float fa = had[0] == -INFINITY ? 0.f : ex2(had[0] - dl[rs][0]), fb = had[1] == -INFINITY ? 0.f : ex2(had[1] - dl[rs][1]);
#pragma unroll
              for (int i = 0; i < MT; ++i) {
                o[rs][i][0] *= fa;
                o[rs][i][1] *= fb;
                o[rs][i][2] *= fa;
                o[rs][i][3] *= fb;
              }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float second = j & 1 ? kSecond : 1.f;
              const float pa = t[rs][j][0] * (f[0] * second), pc = t[rs][j][1] * (f[1] * second);
#pragma unroll
              for (int p = 0; p < ND; ++p) {
                const float st = q4_s(vms[p][j]);
                float wa = pa * st, wb = pc * st;
                if (kMasked && 2 * j >= seen[rs][0] - at) wa = 0.f;
                if (kMasked && 2 * j >= seen[rs][1] - at) wb = 0.f;
                if constexpr (kSplit) {
                  uint32_t hi, lo;
                  split_half2(wa, wb, 1.f, hi, lo);
                  pb[0][p][j] = transpose8(hi);
                  pb[1][p][j] = transpose8(lo);
                } else {
                  pb[rs][p][j] = transpose8(pack_half2(wa, wb));
                }
              }
            }
          }
        };
        if ((int)(x - xr) * kPage + kPage > seen_min) weigh(std::true_type{}); else weigh(std::false_type{});
        // ---- O^T += c^T (p s)^T
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const uint4 w = *(const uint4*)(pg + q4_v(ND) + i * 512 + gid * 64 + t4 * 16);
          const uint32_t vw[2][2] = {{w.x, w.y}, {w.z, w.w}};
          // fp32: the unit cuts its sums off where an addition rounds, so a page has a sum of its own (128 rows of 8 thousand
          // tokens: error 4.5e-6 -> 1.0e-6, in no more time)
          float page[4];
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            uint4 c;
            codes_to_f16<kSplit>(vw[0][s >> 1], s & 1, c.x, c.z);
            codes_to_f16<kSplit>(vw[1][s >> 1], s & 1, c.y, c.w);
#pragma unroll
            for (int k = 0; k < NB; ++k) {
              const uint32_t b0 = pb[k][i / 4][2 * s], b1 = pb[k][i / 4][2 * s + 1];
              if constexpr (kSplit) {
                if (s == 0 && k == 0) mma16816_first(page, c, b0, b1); else mma16816(page, c, b0, b1);
              } else {
                mma16816(o[k][i], c, b0, b1);
              }
            }
          }
          if constexpr (kSplit) {
#pragma unroll
            for (int e = 0; e < 4; ++e) o[0][i][e] += page[e];
          }
        }
        __syncwarp();                            // every lane has read the values
        if (more && lane == 0 && !dead) copy_page(smem_u32(pg) + kHalf, pages + next * kBytes + kHalf, kHalf, vbar);
        phase ^= 1;
        x = nx;
      }

      // ---- the warps' parts of the segment together, in the reference's unit
#pragma unroll
      for (int rs = 0; rs < RS; ++rs)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float* mw = sM + (warp * PR + 8 * rs + 2 * t4 + e) * kPitch;
          // squared: 2^dl alone may be subnormal
          const float up = dl[rs][e] == -INFINITY ? 0.f : ex2(dl[rs][e] * 0.5f + 0.5f * (kCodeExp - kWeightExp));
#pragma unroll
          for (int p = 0; p < ND; ++p) {
            float zp = z[rs][e][p];
#pragma unroll
            for (int x4 = 4; x4 < 32; x4 <<= 1) zp += __shfl_xor_sync(0xffffffffu, zp, x4);
#pragma unroll
            for (int i = 4 * p; i < 4 * p + 4; ++i) {
              mw[16 * i + gid] = fmaf(o[rs][i][e] * up, up, zp);
              mw[16 * i + 8 + gid] = fmaf(o[rs][i][2 + e] * up, up, zp);
            }
          }
          float sum = l[rs][e];
#pragma unroll
          for (int x4 = 4; x4 < 32; x4 <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x4);
          if (gid == 0) {
            mw[64 * ND] = m[rs][e];
            mw[64 * ND + 1] = sum;
          }
        }
      __syncthreads();
      const bool whole = sa == xr && sb == xr + np;
      const int64_t first = first_of(plan, xr), last = last_of(plan, xr, np);
      float* part = a.part + (int64_t)blockIdx.y * 2 * nc * PR * kPitch;
      // a row that sees no token is zeros; logits that are all -inf give 0 / 0
      auto sees_none = [&](int q) { return len - nq + 1 + (p0 + q) / a.G <= 0; };
      const int live = min(gn, nq * a.G - p0);
      for (int i = tid; i < live * 64 * ND; i += kThreads) {
        const int q = i / (64 * ND), c = i % (64 * ND);
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, sM[(w * PR + q) * kPitch + 64 * ND]);
        const float ref = M == -INFINITY ? 0.f : M;
        float L = 0.f, acc = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float* src = sM + (w * PR + q) * kPitch;
          const float f = ex2(src[64 * ND] - ref);             // a warp without a page of this row holds zeros and -inf
          L = fmaf(src[64 * ND + 1], f, L);
          acc = fmaf(src[c], f, acc);
        }
        if (whole) {
          if (c < g.d) store1(out_at(b, h, q) + c, sees_none(q) ? 0.f : acc / L);
        } else {
          float* dst = part + ((2 * blockIdx.x + (sa > xr ? 0 : 1)) * PR + q) * kPitch;
          dst[c] = acc;
          if (c == 0) {
            dst[64 * ND] = M;
            dst[64 * ND + 1] = L;
          }
        }
      }
      if (!whole) {
        __threadfence();
        __syncthreads();
        if (tid == 0) {
          // a CTA is the first of one cut row at most: its byte counts that row's parts
          const int at = kCountByte + blockIdx.y * kMaxGrid + (int)first, shift = 8 * (at & 3);
          uint32_t* count = (uint32_t*)a.err + (at >> 2);
          s_last = (int)(atomicAdd(count, 1u << shift) >> shift & 0xFFu) == (int)(last - first);
          if (s_last) atomicSub(count, (uint32_t)(last - first + 1) << shift);   // as the next call expects it
          __threadfence();
        }
        __syncthreads();
        if (s_last) {
          // factors of the parts' O and the sums, then O: 16 bytes of a part per thread and step, the
          // parts dealt to as many groups of threads as there are, the groups' sums added in order
          const int np2 = (int)(last - first) + 1, ne = live * (16 * ND);
          float* sF = sM;                        // [np2][PR]
          float4* sA = (float4*)(sM + (size_t)W * PR * kPitch - 4 * kThreads);   // [groups][ne]
          static_assert(W * PR * kPitch - 4 * kThreads >= PR * kMaxGrid, "a factor for every part");
          auto src = [&](int k, int q) { return part + ((2 * (first + k) + (k == 0)) * PR + q) * kPitch; };
          __shared__ float s_sum[PR];
          for (int q = warp; q < live; q += W) {
            float M = -INFINITY;
            for (int k = lane; k < np2; k += 32) M = fmaxf(M, __ldcg(src(k, q) + 64 * ND));
#pragma unroll
            for (int o2 = 16; o2; o2 >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o2));
            const float ref = M == -INFINITY ? 0.f : M;
            float L = 0.f;
            for (int k = lane; k < np2; k += 32) {
              const float f = ex2(__ldcg(src(k, q) + 64 * ND) - ref);
              sF[k * PR + q] = f;
              L = fmaf(__ldcg(src(k, q) + 64 * ND + 1), f, L);
            }
#pragma unroll
            for (int o2 = 16; o2; o2 >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o2);
            if (lane == 0) s_sum[q] = L;
          }
          __syncthreads();
          auto finish = [&](float4 v, int q, int c) {
            const float L = s_sum[q];
            const bool none = sees_none(q);
            if (c < g.d)
              store4(out_at(b, h, q) + c, none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(v.x / L, v.y / L, v.z / L, v.w / L));
          };
          const int ng = max(1, kThreads / max(1, ne));
          for (int i = tid; i < ne * ng; i += kThreads) {
            const int e = i % ne, grp = i / ne, q = e / (16 * ND), c = (e % (16 * ND)) * 4;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int k = grp; k < np2; k += ng) {
              const float4 v = __ldcg((const float4*)(src(k, q) + c));
              const float f = sF[k * PR + q];
              acc.x = fmaf(v.x, f, acc.x);
              acc.y = fmaf(v.y, f, acc.y);
              acc.z = fmaf(v.z, f, acc.z);
              acc.w = fmaf(v.w, f, acc.w);
            }
            if (ng > 1) sA[i] = acc; else finish(acc, q, c);
          }
          if (ng > 1) {
            __syncthreads();
            if (tid < ne) {
              float4 acc = sA[tid];
              for (int grp = 1; grp < ng; ++grp) {
                const float4 v = sA[grp * ne + tid];
                acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
              }
              finish(acc, tid / (16 * ND), (tid % (16 * ND)) * 4);
            }
          }
        }
      }
      __syncthreads();                           // before the merge buffer is written again
    }
    xr += np;
    if (xr >= x1) break;
    ++r;
  }
  if (dead) {                                    // copies still under way land before the CTA's memory is released
    bool gave_up = false;
    wait_copy(kbar, phase, gave_up, a.err);
    wait_copy(vbar, phase, gave_up, a.err);
  }
  pdl_trigger();
}

template <int ND, typename T, int RS>
cudaError_t launch(const Q4Geom& g, const Q4AttnArgs& a, const uint8_t* pages, const int32_t* table, const int32_t* lens,
                   int grid, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = raise_smem(q4_attention_kernel<ND, T, RS>, (int)smem_bytes<ND, T, RS>(), done);
  if (e != cudaSuccess) return e;
  const int passes = min((int64_t)kMaxGroups, ((int64_t)a.n_q * a.G - a.p0 + 8 * RS - 1) / (8 * RS));
  return launch_pdl(q4_attention_kernel<ND, T, RS>, dim3(grid, passes), dim3(32 * warps_of<ND, T, RS>()), smem_bytes<ND, T, RS>(), s,
                    g, a, pages, table, lens);
}

template <typename T, int RS>
cudaError_t launch_nd(const Q4Geom& g, const Q4AttnArgs& a, const uint8_t* pages, const int32_t* table,
                      const int32_t* lens, int grid, cudaStream_t s) {
  switch (g.d64 / 64) {
    case 1: return launch<1, T, RS>(g, a, pages, table, lens, grid, s);
    case 2: return launch<2, T, RS>(g, a, pages, table, lens, grid, s);
    case 3: return launch<3, T, 1>(g, a, pages, table, lens, grid, s);
    default: return launch<4, T, 1>(g, a, pages, table, lens, grid, s);
  }
}

// Rows of a pass: 16 where the operand's other half is free and there are more than 8.
int rows_of_pass(const Q4Geom& g, bool bf16, int64_t rows) { return bf16 && g.d64 <= 128 && rows > 8 ? 16 : 8; }

}  // namespace

// [serving header | partials], for a grid of one CTA per SM.
size_t q4_workspace_bytes(const Q4Geom& g, bool bf16, int G, int n_q, int sms) {
  const int64_t rows = (int64_t)G * n_q;
  const int pr = rows_of_pass(g, bf16, rows);
  const int64_t passes = std::min<int64_t>(kMaxGroups, (rows + pr - 1) / pr);
  return kServeHeader + (size_t)passes * 2 * std::min(sms, kMaxGrid) * pr * (g.d64 + 4) * 4;
}

cudaError_t launch_q4_attention(const Q4Geom& g, bool bf16, int G, int n_q, float alpha, const int32_t* q_lens, const void* q,
                                int64_t q_sb, int64_t q_st, int64_t q_sh, void* out, int64_t o_sb, int64_t o_st,
                                int64_t o_sh, const uint8_t* pages, const int32_t* table, const int32_t* lens, void* ws,
                                int sms, cudaStream_t s) {
  char* w = (char*)ws;
  sms = std::min(sms, kMaxGrid);
  const int pr = rows_of_pass(g, bf16, (int64_t)G * n_q);
  // launches of more passes than there are counts for share them
  for (int64_t p0 = 0; p0 < (int64_t)G * n_q; p0 += pr * kMaxGroups) {
    Q4AttnArgs a = {q, out, q_sb, q_st, q_sh, o_sb, o_st, o_sh, alpha, G, n_q, (int32_t)p0, q_lens, (int32_t*)w,
                    (float*)(w + kServeHeader)};
    const cudaError_t e = !bf16     ? launch_nd<float, 1>(g, a, pages, table, lens, sms, s)
                          : pr == 8 ? launch_nd<__nv_bfloat16, 1>(g, a, pages, table, lens, sms, s)
                                    : launch_nd<__nv_bfloat16, 2>(g, a, pages, table, lens, sms, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace chunkkv
