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
//   S = Q K^T takes the query as the 16-row operand and gives a lane two tokens of one query
//   row; that is how O^T = V^T P^T wants its 8-column operand, so the weights go from one to
//   the other in registers, and V's codes fill all 16 rows (half the products and half the
//   sums' registers of O = P V).
//   bf16: up to 8 query rows, or 16 as two columns' worth of the second product.  A query in
//         f16, scaled by a power of two, loses only what is below 2^-25 of its largest element;
//         the weights p s are rounded to f16, 2^-11 each, where the output's rounding is 2^-8.
//         Sums of products with subnormals are good to about 2^-17 of their largest term (the
//         unit aligns them by the exponent that a subnormal is stored with).
//   fp32: 8 query rows, and rows 8-15 carry what f16 cut off (22 bits of each); the weights in
//         two products.  The codes are made whole numbers c - 8 (m becomes m + 8 s), 11 instructions
//         for 8 codes; with subnormals the output was off by 60e-6.
//
// A weight p s is held as a multiple of the largest p s of its row so far (2^d times 2^max t), so
// that f16 holds it however far apart the steps of a row lie.
//
// Work split, join of a row's parts and pages under way: as for the 8-bit cache (decode.cuh,
// q8_attention.cu); a page with its steps is one copy.
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
constexpr float kWeightExp = 14.f;               // the largest weight is 2^14 (f16 ends at 2^16)
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

// Warps of a CTA, a page each in shared memory.  Sixteen hide the products' latency best, and 8
// query rows of up to 128 columns fit their 128 registers a thread.
template <int ND, typename T, int RS>
constexpr int warps_of() { return sizeof(T) == 2 && RS == 1 && ND <= 2 ? 16 : 8; }
template <int ND>
constexpr int pitch() { return 64 * ND + 4; }    // O, m, l: in 16-byte rows
template <int ND>
constexpr bool q_in_regs() { return ND <= 2; }   // wider heads keep their query fragments in shared memory
template <int ND, typename T, int RS>
constexpr size_t smem_bytes() {
  return (size_t)warps_of<ND, T, RS>() * (q4_page_bytes(ND) + 8 * RS * pitch<ND>() * 4) + (q_in_regs<ND>() ? 0 : ND * 4 * 32 * 16);
}
// The halves of a page, each with its steps: two copies, and two barriers.
constexpr int half_bytes(int nd) { return q4_v(nd); }
static_assert(2 * half_bytes(1) == q4_page_bytes(1), "keys and values take the same room");

__device__ __forceinline__ float2 f2(float x, float y) { return make_float2(x, y); }
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
// What code 0 (or code 8, kExact) stands for, of two tokens.
template <bool kExact>
__device__ __forceinline__ float2 base_of(uint32_t a, uint32_t b, float2 s) {
  const float2 m = f2(q4_m(a), q4_m(b));
  return kExact ? __ffma2_rn(s, f2(8.f, 8.f), m) : m;
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
  constexpr bool kSplit = sizeof(T) == 4;        // the query's rows 8-15 carry the low parts of rows 0-7
  static_assert(!kSplit || RS == 1, "an operand has 16 rows");
  constexpr int kCodeExp = kSplit ? 0 : 24;      // a code is c 2^-kCodeExp, or c - 8
  constexpr float kSecond = kSplit ? 1.f : 0.0625f;            // of what meets the second pair of codes
  constexpr int KS = 4 * ND;                     // k steps of a logit, 16 columns each
  constexpr int MT = 4 * ND;                     // 16-column tiles of the output
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[2 * W];
  __shared__ RunShared<W> run;
  __shared__ int s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, t4 = lane & 3;
  uint8_t* pg = smem + warp * kBytes;
  float* sM = (float*)(smem + W * kBytes);       // [W][PR][kPitch]
  uint4* sQ = (uint4*)(sM + W * PR * kPitch);    // one for all warps: they work on one cache row at a time
  const uint32_t kbar = smem_u32(&bars[2 * warp]), vbar = kbar + 8;
  if (lane == 0) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(kbar) : "memory");
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(vbar) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  pdl_wait();

  const Run plan = plan_run<W>(g, lens, run);
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
      float ca[RS], cb[RS][ND];                  // t = ca 2^(kCodeExp - kQueryExp) sum_g s acc + sum_g cb base
      int seen[RS];                              // tokens that the row's query sees
      uint4 qf[q_in_regs<ND>() ? KS : 1];
      int seen_min = len;
#pragma unroll
      for (int rs = 0; rs < RS; ++rs) {
        const int row = gid + 8 * rs, i = (p0 + row) / a.G;
        const bool live = row < gn && i < nq;
        seen[rs] = live ? len - nq + 1 + i : len;
        seen_min = min(seen_min, seen[rs]);
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
#pragma unroll
        for (int p = 0; p < ND; ++p) {
          float sum = 0.f;
#pragma unroll
          for (int s = 4 * p; s < 4 * p + 4; ++s) sum += (qv[s][0] + qv[s][1]) + (qv[s][2] + qv[s][3]);
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          cb[rs][p] = sum * a.alpha;
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // scaled by a power of two into f16's range, whatever the query's size
        const int e2 = min(127, max(-110, (int)(top >> 23) - 127));
        const float down = power_of_two(kQueryExp - e2);
        ca[rs] = a.alpha * power_of_two(e2);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const float c0 = qv[s][0] * down, c1 = qv[s][1] * down, c2 = qv[s][2] * down * kSecond, c3 = qv[s][3] * down * kSecond;
          uint4 f = make_uint4(0, 0, 0, 0);
          if (rs > 0) {
            if constexpr (q_in_regs<ND>()) f = qf[s]; else f = sQ[s * 32 + lane];
          }
          if constexpr (kSplit) {
            split_half2(c0, c1, 1.f, f.x, f.y);
            split_half2(c2, c3, 1.f, f.z, f.w);
          } else if (rs == 0) {
            f.x = pack_half2(c0, c1);
            f.z = pack_half2(c2, c3);
          } else {
            f.y = pack_half2(c0, c1);
            f.w = pack_half2(c2, c3);
          }
          if constexpr (q_in_regs<ND>()) qf[s] = f; else sQ[s * 32 + lane] = f;
        }
      }
      seen_min = __reduce_min_sync(0xffffffffu, seen_min);
      float m[RS], l[RS], dl[RS], z[RS][ND];     // reference, sum, O's unit as an exponent of 2 above the reference, sum of p m
#pragma unroll
      for (int rs = 0; rs < RS; ++rs) {
        m[rs] = dl[rs] = -INFINITY;
        l[rs] = 0.f;
#pragma unroll
        for (int p = 0; p < ND; ++p) z[rs][p] = 0.f;
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
        // ---- t.  Column 2 t + e of tile i is token 16 t + 2 i + e of the page: the tokens that lane t's pieces of V hold
        float2 t[RS][8];
#pragma unroll
        for (int x4 = 0; x4 < 4; ++x4) {
          uint32_t ms[ND][4];
#pragma unroll
          for (int p = 0; p < ND; ++p) {
            const uint4 w = *(const uint4*)(pg + q4_k_ms(ND) + (p * kPage + 16 * t4 + 4 * x4) * 4);
            ms[p][0] = w.x; ms[p][1] = w.y; ms[p][2] = w.z; ms[p][3] = w.w;
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int i = 2 * x4 + y, token = 16 * (gid >> 1) + 2 * i + (gid & 1);
            const uint8_t* src = pg + token * (32 * ND) + t4 * (8 * ND);
            uint32_t kw[2 * ND];
            if constexpr (ND % 2 == 0) {
#pragma unroll
              for (int p = 0; p < ND / 2; ++p) {
                const uint4 w = *(const uint4*)(src + 16 * p);
                kw[4 * p] = w.x; kw[4 * p + 1] = w.y; kw[4 * p + 2] = w.z; kw[4 * p + 3] = w.w;
              }
            } else {
#pragma unroll
              for (int p = 0; p < ND; ++p) {
                const uint2 w = *(const uint2*)(src + 8 * p);
                kw[2 * p] = w.x; kw[2 * p + 1] = w.y;
              }
            }
            float2 sum[RS], off[RS];
#pragma unroll
            for (int p = 0; p < ND; ++p) {
              float acc[4];
#pragma unroll
              for (int s = 0; s < 4; ++s) {
                uint32_t b0, b1;
                codes_to_f16<kSplit>(kw[2 * p + (s >> 1)], s & 1, b0, b1);
                uint4 f;
                if constexpr (q_in_regs<ND>()) f = qf[4 * p + s]; else f = sQ[(4 * p + s) * 32 + lane];
                if (s == 0) mma16816_first(acc, f, b0, b1); else mma16816(acc, f, b0, b1);
              }
              const float2 s2 = f2(q4_s(ms[p][2 * y]), q4_s(ms[p][2 * y + 1])), m2 = base_of<kSplit>(ms[p][2 * y], ms[p][2 * y + 1], s2);
#pragma unroll
              for (int rs = 0; rs < RS; ++rs) {
                const float2 v = kSplit ? f2(acc[0] + acc[2], acc[1] + acc[3]) : f2(acc[2 * rs], acc[2 * rs + 1]);
                const float2 c2 = f2(cb[rs][p], cb[rs][p]);
                sum[rs] = p == 0 ? __fmul2_rn(v, s2) : __ffma2_rn(v, s2, sum[rs]);
                off[rs] = p == 0 ? __fmul2_rn(c2, m2) : __ffma2_rn(c2, m2, off[rs]);
              }
            }
#pragma unroll
            for (int rs = 0; rs < RS; ++rs) {
              constexpr float kUp = kSplit ? 1.f / (1 << kQueryExp) : 1 << (24 - kQueryExp);
              t[rs][i] = __ffma2_rn(__fmul2_rn(sum[rs], f2(kUp, kUp)), f2(ca[rs], ca[rs]), off[rs]);
            }
          }
        }
        __syncwarp();                            // every lane has read the keys
        if (more && lane == 0 && !dead) copy_page(smem_u32(pg), pages + next * kBytes, kHalf, kbar);
        wait_copy(vbar, phase, dead, a.err);
        // ---- weights p s and their largest, the reference, O's unit; the second product's operands
        uint32_t pb[RS * (kSplit ? 2 : 1)][ND][4][2];
        auto weigh = [&](auto masked_c) {
          constexpr bool kMasked = decltype(masked_c)::value;
          const int at = (int)(x - xr) * kPage + 16 * t4;     // the row's token that this lane holds first
#pragma unroll
          for (int rs = 0; rs < RS; ++rs) {
            const int left = seen[rs] - at;
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (kMasked) {
                if (2 * i >= left) t[rs][i].x = -INFINITY;
                if (2 * i + 1 >= left) t[rs][i].y = -INFINITY;
              }
              top = fmaxf(top, fmaxf(t[rs][i].x, t[rs][i].y));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float mn = fmaxf(m[rs], top), ref = mn == -INFINITY ? 0.f : mn;
            const float drop = m[rs] == -INFINITY ? 0.f : mn - m[rs], fl = ex2(-drop);
            m[rs] = mn;
            float2 sum = f2(0.f, 0.f), off[ND];
#pragma unroll
            for (int p = 0; p < ND; ++p) off[p] = f2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              t[rs][i] = f2(ex2(t[rs][i].x - ref), ex2(t[rs][i].y - ref));
              sum = __fadd2_rn(sum, t[rs][i]);
            }
            l[rs] = fmaf(l[rs], fl, sum.x + sum.y);
            // p s, of which hidden tokens have none whatever their steps are
            float u = 0.f;
            float2 w[ND][8];
#pragma unroll
            for (int p = 0; p < ND; ++p)
#pragma unroll
              for (int x4 = 0; x4 < 4; ++x4) {
                const uint4 v = *(const uint4*)(pg + q4_v_ms(ND) + (p * kPage + 16 * t4 + 4 * x4) * 4);
                uint32_t ms[4] = {v.x, v.y, v.z, v.w};
                if (kMasked) {
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    if (4 * x4 + e >= left) ms[e] = 0;
                }
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const float2 pr = t[rs][2 * x4 + y];
                  const float2 s2 = f2(q4_s(ms[2 * y]), q4_s(ms[2 * y + 1]));
                  w[p][2 * x4 + y] = __fmul2_rn(pr, s2);
                  off[p] = __ffma2_rn(pr, base_of<kSplit>(ms[2 * y], ms[2 * y + 1], s2), off[p]);
                  u = fmaxf(u, fmaxf(w[p][2 * x4 + y].x, w[p][2 * x4 + y].y));
                }
              }
#pragma unroll
            for (int p = 0; p < ND; ++p) z[rs][p] = fmaf(z[rs][p], fl, off[p].x + off[p].y);
            u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, 1));
            u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, 2));
            // O's unit, 2^dl of the reference's: as large as the largest weight asks, and never smaller than it was
            const float had = dl[rs] - drop, need = u > 0.f ? fmaxf(lg2(u), -112.f) : -INFINITY, now = fmaxf(had, need);
            if (__any_sync(0xffffffffu, now != had)) {
              const float fo = had == -INFINITY ? 0.f : ex2(had - now);
              const float fa = __shfl_sync(0xffffffffu, fo, 8 * t4), fb = __shfl_sync(0xffffffffu, fo, 8 * t4 + 4);
#pragma unroll
              for (int i = 0; i < MT; ++i) {
                o[rs][i][0] *= fa;
                o[rs][i][1] *= fb;
                o[rs][i][2] *= fa;
                o[rs][i][3] *= fb;
              }
            }
            dl[rs] = now;
            const float f = ex2(fminf(kWeightExp - now, 126.f)), fs = f * kSecond;
#pragma unroll
            for (int p = 0; p < ND; ++p)
#pragma unroll
              for (int s = 0; s < 4; ++s) {
                const float2 a0 = __fmul2_rn(w[p][2 * s], f2(f, f)), a1 = __fmul2_rn(w[p][2 * s + 1], f2(fs, fs));
                if constexpr (kSplit) {
                  split_half2(a0.x, a0.y, 1.f, pb[0][p][s][0], pb[1][p][s][0]);
                  split_half2(a1.x, a1.y, 1.f, pb[0][p][s][1], pb[1][p][s][1]);
                } else {
                  pb[rs][p][s][0] = pack_half2(a0.x, a0.y);
                  pb[rs][p][s][1] = pack_half2(a1.x, a1.y);
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
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            uint4 c;
            codes_to_f16<kSplit>(vw[0][s >> 1], s & 1, c.x, c.z);
            codes_to_f16<kSplit>(vw[1][s >> 1], s & 1, c.y, c.w);
#pragma unroll
            for (int k = 0; k < RS * (kSplit ? 2 : 1); ++k)
              mma16816(o[kSplit ? 0 : k][i], c, pb[k][i / 4][s][0], pb[k][i / 4][s][1]);
          }
        }
        __syncwarp();                            // every lane has read the values
        if (more && lane == 0 && !dead) copy_page(smem_u32(pg) + kHalf, pages + next * kBytes + kHalf, kHalf, vbar);
        phase ^= 1;
        x = nx;
      }

      // ---- the warps' parts of the segment together, in the reference's unit
#pragma unroll
      for (int rs = 0; rs < RS; ++rs) {
        l[rs] += __shfl_xor_sync(0xffffffffu, l[rs], 1);
        l[rs] += __shfl_xor_sync(0xffffffffu, l[rs], 2);
        float* mw = sM + (warp * PR + 8 * rs) * kPitch;
        // squared: 2^dl alone may be subnormal
        const float up = dl[rs] == -INFINITY ? 0.f : ex2(dl[rs] * 0.5f + 0.5f * (kCodeExp - kWeightExp));
        const float ua = __shfl_sync(0xffffffffu, up, 8 * t4), ub = __shfl_sync(0xffffffffu, up, 8 * t4 + 4);
#pragma unroll
        for (int p = 0; p < ND; ++p) {
          z[rs][p] += __shfl_xor_sync(0xffffffffu, z[rs][p], 1);
          z[rs][p] += __shfl_xor_sync(0xffffffffu, z[rs][p], 2);
          const float za = __shfl_sync(0xffffffffu, z[rs][p], 8 * t4), zb = __shfl_sync(0xffffffffu, z[rs][p], 8 * t4 + 4);
#pragma unroll
          for (int i = 4 * p; i < 4 * p + 4; ++i) {
            float* dst = mw + 2 * t4 * kPitch + 16 * i + gid;
            dst[0] = fmaf(o[rs][i][0] * ua, ua, za);
            dst[8] = fmaf(o[rs][i][2] * ua, ua, za);
            dst[kPitch] = fmaf(o[rs][i][1] * ub, ub, zb);
            dst[kPitch + 8] = fmaf(o[rs][i][3] * ub, ub, zb);
          }
        }
        if (t4 == 0) {
          mw[gid * kPitch + 64 * ND] = m[rs];
          mw[gid * kPitch + 64 * ND + 1] = l[rs];
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
