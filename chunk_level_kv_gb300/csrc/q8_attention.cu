// Single-token attention over the 8-bit paged cache.
//
//   O_g = sum_j 2^(t_j) s_v V_j / sum_j 2^(t_j),   t_j = scale log2(e) s_k (q_g . K_j)
//
// over the tokens j of one cache row, K and V int8 codes, s_k and s_v the scales of
// the token's page; one pass over the pages with a running maximum of t and sum.
//
// What bounds it: every page is read once (2 d bytes a token), HBM.  The arithmetic
// must keep out of the way: at 6.76 TB/s an SM receives 23 codes a clock, which leaves
// 5 instruction slots a code.  So both products run on the tensor cores in f16, in
// which an int8 code is exact (a byte permute and a packed subtraction turn four codes
// into two operand registers, 1.25 instructions a code), with the G <= 8 query heads of
// a KV head as the 16-row operand's rows 0-7.  Rows 8-15 carry what f16 cut off: the
// query is split into two f16 parts (22 bits) and so are the weights, so the products
// are as good as fp32 ones (down to 2^-38 of the largest weight times value scale, where
// f16 ends) and cost nothing more than the 16 rows that the instruction computes anyway.
// mma.sync and not tcgen05: the operands come from registers after the conversion, and an
// m128 tile would be 1/16 full.
//
// Work split: the pages of all rows in order are cut into one contiguous run per CTA
// (one CTA per SM), whatever the rows' lengths, which only the device knows: every CTA
// finds its run by a scan over the lengths.  Inside a CTA the pages go to the warps in
// turn; each warp has a K and a V slot that bulk copies fill while it works on the
// other, so about 100 KB per SM are under way.  A row that lies in one CTA is
// written at once; the CTAs that share a row write partials (O, l, references), and the last one to
// arrive adds them in CTA order, so that the result does not depend on the order of
// arrival.
//
// Measured: 64 sequences x 4 KV heads of 12 to 13 thousand tokens (0.83 GB) 137 us,
// 6.0 TB/s, 89 % of a copy's rate, and its DRAM reads are the pages' bytes; one sequence
// of 8 KV heads x 6.5 thousand tokens 12.3 us, 16 sequences of 256 to 300 tokens 7.4 us
// (latency: lengths, page index, page, products and join one after another).
#include <cuda_fp16.h>

#include "serve.cuh"

namespace chunkkv {
namespace {

constexpr int kMaxG = 8;                         // query heads per pass
constexpr int kMaxGrid = 224;                    // CTAs of a pass (one per SM): a count for each in the header
constexpr float kWeightScale = 14.f;             // weights are times 2^14: f16 keeps them to 2^-38 of the largest
constexpr float kMostScale = 8.5e37f;            // about 2^126
constexpr int kMaxGroups = 16;                   // passes of kMaxG heads in one launch
// Parts of a cut row that have arrived, 8 bits for each CTA (the row's first) and pass, zero between calls.  They lie
// at a place that no shape moves and that no serving call writes otherwise; the first pass's in the header proper.
constexpr int kCountByte = 32;
static_assert(kCountByte > 4 * (kSchedWord + 1) && kCountByte % 4 == 0 && kMaxGrid % 4 == 0, "behind the other words");
static_assert(kCountByte + kMaxGrid <= 256 && kMaxGrid < 256, "the first pass's counts lie in the header proper");
static_assert(kCountByte + kMaxGrid * kMaxGroups <= kServeHeader, "the counts lie in the serving header");

struct Q8AttnArgs {
  const void* q;
  void* out;
  int64_t q_sb, q_sh, o_sb, o_sh;
  float alpha;                                   // scale * log2(e)
  int32_t G, g0;                                 // query heads per KV head, and the first of this launch
  int32_t* err;                                  // the workspace header: error word, counts of arrived parts
  float* part;                                   // [passes][2 CTAs][8][d64 + 4]: O, m, l, O's reference
};

// Rows of up to this many pages are not cut: a row in two pieces costs the CTAs that
// share it about 4 us (partials, a counter, the join), a page about 0.4 us of a CTA's
// share of the bandwidth, and the eight warps take eight pages at once.
// A cut within kNearEnd pages of a long row's begin or end moves there, so that a CTA
// seldom has a second row for a few pages.
constexpr int kWholeRow = 8;
constexpr int kNearEnd = 3;
static_assert(kWholeRow > 2 * kNearEnd, "a row's two ends do not meet");

template <int ND>
constexpr int warps_of() { return ND <= 2 ? 8 : 4; }
template <int ND>
constexpr int page_bytes() { return ND * 64 * kPage; }
template <int ND>
constexpr int merge_pitch() { return 64 * ND + 3; }         // O, then m, l and O's reference
template <int ND>
constexpr int part_pitch() { return 64 * ND + 4; }          // the same in the workspace, in 16-byte rows
template <int ND>
constexpr bool q_in_regs() { return ND <= 2; }              // wider heads keep their query fragments in shared memory
template <int ND>
constexpr size_t smem_bytes() {
  return (size_t)warps_of<ND>() * (2 * page_bytes<ND>() + kMaxG * merge_pitch<ND>() * 4 +
                                   (q_in_regs<ND>() ? 0 : ND * 4 * 32 * 16));
}

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// D (16 x 8, fp32) += A (16 x 16, f16) B (16 x 8, f16)
__device__ __forceinline__ void mma16816(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
// Four int8 codes as two f16 pairs: a code plus 128 in the low byte of 0x64.. is
// 1024 + 128 + code, exactly.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  w ^= 0x80808080u;
  uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
  const __half2 k = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
  const __half2 x = __hsub2(*(__half2*)&a, k), y = __hsub2(*(__half2*)&b, k);
  lo = *(const uint32_t*)&x;
  hi = *(const uint32_t*)&y;
}
__device__ __forceinline__ uint32_t pack_half2(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *(const uint32_t*)&h;
}
// x = hi + lo in two f16 pairs (lo times up).
__device__ __forceinline__ void split_half2(float x, float y, float up, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  hi = *(const uint32_t*)&h;
  lo = pack_half2((x - f.x) * up, (y - f.y) * up);
}

__device__ __forceinline__ void load4f(const float* p, float (&x)[4]) {
  const float4 v = *(const float4*)p;
  x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void load4f(const __nv_bfloat16* p, float (&x)[4]) {
  const uint2 v = *(const uint2*)p;
  x[0] = __uint_as_float(v.x << 16);
  x[1] = __uint_as_float(v.x & 0xFFFF0000u);
  x[2] = __uint_as_float(v.y << 16);
  x[3] = __uint_as_float(v.y & 0xFFFF0000u);
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ void store4(float* p, float4 v) { *(float4*)p = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
  *(uint2*)p = make_uint2(*(const uint32_t*)&x, *(const uint32_t*)&y);
}

// O over the sum, from O's reference to the sum's.
__device__ __forceinline__ float4 finish(float4 o, float sum, float up) {
  return make_float4(o.x / sum * up, o.y / sum * up, o.z / sum * up, o.w / sum * up);
}

__device__ __forceinline__ int pages_of(int n) { return (n + kPage - 1) / kPage; }

// A bounded wait for one phase of a copy that this warp started.  Nothing but the
// copy itself completes it, so the limit (seconds) is never met in a healthy run; a
// warp that meets it records an error, waits no more and lets the kernel end.
__device__ __forceinline__ void wait_copy(uint32_t bar, uint32_t parity, bool& dead, int32_t* err) {
  if (dead) return;
  for (int i = 0; i < 4096; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok) : "r"(bar), "r"(parity), "r"(1000000u) : "memory");
    if (ok) return;
  }
  atomicCAS(err, 0, (int)kDevTimeoutTmaProducer);
  dead = true;
}
__device__ __forceinline__ void copy_page(uint32_t dst, const int8_t* src, uint32_t bytes, uint32_t bar) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(dst), "l"((uint64_t)src), "r"(bytes), "r"(bar) : "memory");
}

// Where global page x lies: rows are looked up 32 at a time, a lane each.
struct Cursor {
  int base;                 // row of lane 0
  int64_t start;            // pages before it
  int len;                  // this lane's row's length
  int64_t end;              // pages up to and with this lane's row

  __device__ void load(const Q8Geom& g, const int32_t* lens, int lane) {
    const int r = base + lane;
    len = r < g.rows ? safe_len(lens[r], g.max_pages) : 0;
    int n = pages_of(len);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += y;
    }
    end = start + n;
  }
  // Row, page inside the row and length of the row of page x (below the total, not
  // before an earlier call's).
  __device__ void locate(const Q8Geom& g, const int32_t* lens, int lane, int64_t x, int& row, int& j, int& n) {
    while (true) {
      const uint32_t above = __ballot_sync(0xffffffffu, end > x);
      if (above || base + 32 >= g.rows) {
        const int at = above ? __ffs(above) - 1 : 31;
        row = min(base + at, g.rows - 1);
        n = __shfl_sync(0xffffffffu, len, at);
        j = (int)(x - (__shfl_sync(0xffffffffu, end, at) - pages_of(n)));
        return;
      }
      start = __shfl_sync(0xffffffffu, end, 31);
      base += 32;
      load(g, lens, lane);
    }
  }
};

template <int ND, typename T>
__global__ void __launch_bounds__(32 * warps_of<ND>(), 1)
q8_attention_kernel(Q8Geom g, Q8AttnArgs a, const int8_t* __restrict__ k_pages, const int8_t* __restrict__ v_pages,
                    const float2* __restrict__ scales, const int32_t* __restrict__ table,
                    const int32_t* __restrict__ lens) {
  constexpr int W = warps_of<ND>(), kThreads = 32 * W, kBytes = page_bytes<ND>(), kPitch = merge_pitch<ND>();
  constexpr int kPart = part_pitch<ND>();
  constexpr int KS = 4 * ND;                     // k steps of a logit, 16 columns each
  constexpr int NT = 8 * ND;                     // 8-column tiles of the output
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[2 * W];
  __shared__ long long s_scan[W];
  __shared__ int64_t s_cut[2], s_start[2];       // the run's ends, and the pages before the rows that they lie in
  __shared__ int s_row[2], s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, t4 = lane & 3;
  uint8_t* sK = smem + warp * 2 * kBytes;
  uint8_t* sV = sK + kBytes;
  float* sM = (float*)(smem + W * 2 * kBytes);   // [W][8][kPitch]
  uint4* sQ = (uint4*)(sM + W * kMaxG * kPitch) + warp * KS * 32;
  const uint32_t kbar = smem_u32(&bars[2 * warp]), vbar = smem_u32(&bars[2 * warp + 1]);
  if (lane == 0) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(kbar) : "memory");
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(vbar) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();

  // ---- this CTA's run [x0, x1) of the pages of all rows, and the row in which it begins
  const int chunk = (g.rows + kThreads - 1) / kThreads;
  const int c0 = min(g.rows, tid * chunk), c1 = min(g.rows, c0 + chunk);
  long long mine = 0;
  for (int r = c0; r < c1; ++r) mine += pages_of(safe_len(lens[r], g.max_pages));
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  long long total = 0, before = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if (i == warp) before = total;
    total += s_scan[i];
  }
  before += incl - mine;                         // pages before this thread's rows
  // no more runs than pages: every CTA that shares a row has a part of it
  const int64_t nc = total < gridDim.x ? total : gridDim.x;
  const bool busy = blockIdx.x < nc;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t cut = busy ? total * (blockIdx.x + k) / nc : total;
    if (cut == total) {
      if (tid == 0) s_cut[k] = total;
    } else if (cut >= before && cut < before + mine) {
      int64_t x = before;
      int r = c0, n = 0;
      for (; r < c1; ++r) {
        n = pages_of(safe_len(lens[r], g.max_pages));
        if (x + n > cut) break;
        x += n;
      }
      // short rows stay in one piece, and a long one's end is no place to cut either
      s_cut[k] = n <= kWholeRow || cut - x <= kNearEnd ? x : x + n - cut <= kNearEnd ? x + n : cut;
      s_row[k] = r;
      s_start[k] = x;
    }
  }
  const int g0 = a.g0 + blockIdx.y * kMaxG, gn = min(kMaxG, a.G - g0);
  // rows without a token
  for (int r = blockIdx.x; r < g.rows; r += gridDim.x)
    if (lens[r] <= 0)
      for (int i = tid; i < gn * g.d; i += kThreads)
        store1((T*)a.out + (r / g.Hkv) * a.o_sb + ((r % g.Hkv) * a.G + g0 + i / g.d) * a.o_sh + i % g.d, 0.f);
  __syncthreads();
  const int64_t x0 = s_cut[0], x1 = s_cut[1];
  if (x0 >= x1) {
    pdl_trigger();
    return;
  }

  // ---- pages under way: [x] in the slots, [x + W] known by its index and scales, [x + 2 W] by its index
  Cursor cur;
  cur.base = s_row[0];
  cur.start = s_start[0];
  cur.load(g, lens, lane);
  int64_t x = x0 + warp;
  int j0 = 0, n0 = 0, j1 = 0, n1 = 0, row = 0;
  int64_t page1 = 0;
  float2 sc0 = make_float2(0.f, 0.f), sc1 = sc0;
  bool dead = false;
  uint32_t phase = 0;
  if (x < x1) {
    cur.locate(g, lens, lane, x, row, j0, n0);
    const int64_t page = safe_page(table[(int64_t)row * g.max_pages + j0], g.n_pages);
    if (lane == 0) {
      copy_page(smem_u32(sK), k_pages + page * kBytes, kBytes, kbar);
      copy_page(smem_u32(sV), v_pages + page * kBytes, kBytes, vbar);
    }
    sc0 = scales[page];
  }
  if (x + W < x1) {
    cur.locate(g, lens, lane, x + W, row, j1, n1);
    page1 = safe_page(table[(int64_t)row * g.max_pages + j1], g.n_pages);
  }

  int r = s_row[0];                              // segment by segment: the CTA's part of row r
  int64_t xr = s_start[0];
  while (true) {
    const int len = safe_len(lens[r], g.max_pages), np = pages_of(len);
    const int64_t sa = xr > x0 ? xr : x0, sb = xr + np < x1 ? xr + np : x1;
    const int b = r / g.Hkv, hq = (r % g.Hkv) * a.G + g0;
    if (sa < sb) {
      // the query's fragments: columns 64 p + 16 t + 4 kk .. + 3 are the 16-byte piece of a key that lane t reads
      float qs = 0.f;
      uint4 qf[q_in_regs<ND>() ? KS : 1];
      if (x < sb) {
        float qv[KS][4];
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const int c = (s >> 2) * 64 + t4 * 16 + (s & 3) * 4;
          qv[s][0] = qv[s][1] = qv[s][2] = qv[s][3] = 0.f;
          if (gid < gn && c < g.d) load4f((const T*)a.q + b * a.q_sb + (hq + gid) * a.q_sh + c, qv[s]);
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(qv[s][e]) & 0x7FFFFFFFu);
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // scaled by a power of two into f16's best range, whatever the query's size
        const int e2 = min(126, max(-126, (int)(top >> 23) - 127));
        const float down = __uint_as_float((uint32_t)(127 - e2) << 23);
        qs = a.alpha * __uint_as_float((uint32_t)(127 + e2) << 23);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          uint4 f;
          split_half2(qv[s][0] * down, qv[s][1] * down, 2048.f, f.x, f.y);
          split_half2(qv[s][2] * down, qv[s][3] * down, 2048.f, f.z, f.w);
          if constexpr (q_in_regs<ND>()) qf[s] = f; else sQ[s * 32 + lane] = f;
        }
      }
      float m = -INFINITY, l = 0.f, mo = -INFINITY;
      float o[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

      while (x < sb) {
        // indexes and scales of the pages to come
        const bool more = x + W < x1, more2 = x + 2 * W < x1;
        if (more) sc1 = scales[page1];
        int j2 = 0, n2 = 0;
        int64_t page2 = 0;
        if (more2) {
          cur.locate(g, lens, lane, x + 2 * W, row, j2, n2);
          page2 = safe_page(table[(int64_t)row * g.max_pages + j2], g.n_pages);
        }
        wait_copy(kbar, phase, dead, a.err);
        // S = Q K^T.  Column 2t + e of tile i is token 16 t + 2 i + e of the page: the tokens that lane t's
        // 16-byte pieces of V hold
        float s[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
          const int token = 16 * (gid >> 1) + 2 * i + (gid & 1);
#pragma unroll
          for (int p = 0; p < ND; ++p) {
            const uint4 w = *(const uint4*)(sK + p * (kPage * 64) + token * 64 + t4 * 16);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              uint32_t b0, b1;
              codes_to_f16(ww[kk], b0, b1);
              uint4 f;
              if constexpr (q_in_regs<ND>()) f = qf[4 * p + kk]; else f = sQ[(4 * p + kk) * 32 + lane];
              mma16816(s[i], f, b0, b1);
            }
          }
        }
        __syncwarp();                            // every lane has read the slot
        if (more && lane == 0 && !dead) copy_page(smem_u32(sK), k_pages + page1 * kBytes, kBytes, kbar);
        // t = (high + low 2^-11) s_k scale; the running maximum; weights 2^(t - m + 14)
        const float ts = sc0.x * qs;
        const int left = n0 - j0 * kPage - 16 * t4;          // tokens of the row from this lane's first on
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            s[i][e] = 2 * i + e < left ? fmaf(s[i][2 + e], 1.f / 2048.f, s[i][e]) * ts : -INFINITY;
            top = fmaxf(top, s[i][e]);
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float mn = fmaxf(m, top);
        const float ref = mn == -INFINITY ? 0.f : mn;
        if (m != -INFINITY) l *= ex2(m - mn);
        m = mn;
        // O has a reference of its own, the maximum of t + log2 s_v: how large a page's values are counts only with
        // the weight that they have, and f16 keeps every weight times s_v to 2^-38 of the largest
        const float on = fmaxf(mo, top + lg2(fabsf(sc0.y)));
        if (__any_sync(0xffffffffu, on != mo)) {
          const float fo = mo == -INFINITY ? 0.f : ex2(mo - on);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            o[i][0] *= fo;
            o[i][1] *= fo;
            o[i][2] *= fo;
            o[i][3] *= fo;
          }
        }
        mo = on;
        // 2^(t - ref) vr = 2^(t - on) s_v.  The power in two halves, since it alone may pass fp32's range, and the
        // product bounded, since 0 x inf is NaN (the bound meets weights below 2^-112 of the largest)
        const float half = ex2(0.5f * (ref - (on == -INFINITY ? 0.f : on)));
        float vr = sc0.y == 0.f ? 0.f : sc0.y * half * half;
        vr = vr > kMostScale ? kMostScale : vr;
        uint4 pf[4];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = ex2((s[2 * kk + (e >> 1)][e & 1] - ref) + kWeightScale);
            l += p;
            w[e] = p * vr;
          }
          split_half2(w[0], w[1], 1.f, pf[kk].x, pf[kk].y);
          split_half2(w[2], w[3], 1.f, pf[kk].z, pf[kk].w);
        }
        wait_copy(vbar, phase, dead, a.err);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const uint4 w = *(const uint4*)(sV + (8 * i + gid) * kPage + t4 * 16);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            uint32_t b0, b1;
            codes_to_f16(ww[kk], b0, b1);
            mma16816(o[i], pf[kk], b0, b1);
          }
        }
        __syncwarp();
        if (more && lane == 0 && !dead) copy_page(smem_u32(sV), v_pages + page1 * kBytes, kBytes, vbar);
        phase ^= 1;
        x += W;
        j0 = j1; n0 = n1; sc0 = sc1;
        j1 = j2; n1 = n2; page1 = page2;
      }

      // ---- the warps' parts of the segment together
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      float* mw = sM + (warp * kMaxG + gid) * kPitch;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        mw[8 * i + 2 * t4] = o[i][0] + o[i][2];
        mw[8 * i + 2 * t4 + 1] = o[i][1] + o[i][3];
      }
      if (t4 == 0) {
        mw[64 * ND] = m;
        mw[64 * ND + 1] = l;
        mw[64 * ND + 2] = mo;
      }
      __syncthreads();
      const bool whole = sa == xr && sb == xr + np;
      // the CTAs of a row that is cut: from the last one whose cut is at its begin or moves there, to the last
      // one whose cut does not move to its end
      const int64_t first = ((xr + kNearEnd + 1) * nc - 1) / total, last = ((xr + np - kNearEnd) * nc - 1) / total;
      float* part = a.part + (int64_t)blockIdx.y * 2 * nc * kMaxG * kPart;
      for (int i = tid; i < gn * 64 * ND; i += kThreads) {
        const int q = i / (64 * ND), c = i % (64 * ND);
        float M = -INFINITY, MO = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          M = fmaxf(M, sM[(w * kMaxG + q) * kPitch + 64 * ND]);
          MO = fmaxf(MO, sM[(w * kMaxG + q) * kPitch + 64 * ND + 2]);
        }
        const float ref = M == -INFINITY ? 0.f : M, oref = MO == -INFINITY ? 0.f : MO;
        float L = 0.f, acc = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float* src = sM + (w * kMaxG + q) * kPitch;
          // a warp without a page of this row holds zeros and -inf
          L += src[64 * ND + 1] * ex2(src[64 * ND] - ref);
          acc += src[c] * ex2(src[64 * ND + 2] - oref);
        }
        if (whole) {
          if (c < g.d) store1((T*)a.out + b * a.o_sb + (hq + q) * a.o_sh + c, acc / L * ex2(MO - M));
        } else {
          float* dst = part + ((2 * blockIdx.x + (sa > xr ? 0 : 1)) * kMaxG + q) * kPart;
          dst[c] = acc;
          if (c == 0) {
            dst[64 * ND] = M;
            dst[64 * ND + 1] = L;
            dst[64 * ND + 2] = MO;
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
          const int np2 = (int)(last - first) + 1, ne = gn * (16 * ND);
          float* sF = sM;                        // [np2][kMaxG]
          float4* sA = (float4*)(sM + (size_t)W * kMaxG * kPitch - 4 * kThreads);   // [groups][ne]
          static_assert(W * kMaxG * kPitch - 4 * kThreads >= kMaxG * kMaxGrid, "a factor for every part");
          auto src = [&](int k, int q) { return part + ((2 * (first + k) + (k == 0)) * kMaxG + q) * kPart; };
          __shared__ float s_sum[kMaxG], s_up[kMaxG];
          for (int q = warp; q < gn; q += W) {
            float M = -INFINITY, MO = -INFINITY;
            for (int k = lane; k < np2; k += 32) {
              M = fmaxf(M, __ldcg(src(k, q) + 64 * ND));
              MO = fmaxf(MO, __ldcg(src(k, q) + 64 * ND + 2));
            }
#pragma unroll
            for (int o2 = 16; o2; o2 >>= 1) {
              M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o2));
              MO = fmaxf(MO, __shfl_xor_sync(0xffffffffu, MO, o2));
            }
            const float ref = M == -INFINITY ? 0.f : M, oref = MO == -INFINITY ? 0.f : MO;
            float L = 0.f;
            for (int k = lane; k < np2; k += 32) {
              sF[k * kMaxG + q] = ex2(__ldcg(src(k, q) + 64 * ND + 2) - oref);
              L = fmaf(__ldcg(src(k, q) + 64 * ND + 1), ex2(__ldcg(src(k, q) + 64 * ND) - ref), L);
            }
#pragma unroll
            for (int o2 = 16; o2; o2 >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o2);
            if (lane == 0) {
              s_sum[q] = L;
              s_up[q] = ex2(MO - M);
            }
          }
          __syncthreads();
          const int ng = max(1, kThreads / ne);
          for (int i = tid; i < ne * ng; i += kThreads) {
            const int e = i % ne, grp = i / ne, q = e / (16 * ND), c = (e % (16 * ND)) * 4;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int k = grp; k < np2; k += ng) {
              const float4 v = __ldcg((const float4*)(src(k, q) + c));
              const float f = sF[k * kMaxG + q];
              acc.x = fmaf(v.x, f, acc.x);
              acc.y = fmaf(v.y, f, acc.y);
              acc.z = fmaf(v.z, f, acc.z);
              acc.w = fmaf(v.w, f, acc.w);
            }
            if (ng > 1) {
              sA[i] = acc;
            } else {
              T* dst = (T*)a.out + b * a.o_sb + (hq + q) * a.o_sh + c;
              if (c < g.d) store4(dst, finish(acc, s_sum[q], s_up[q]));
            }
          }
          if (ng > 1) {
            __syncthreads();
            if (tid < ne) {
              float4 acc = sA[tid];
              for (int grp = 1; grp < ng; ++grp) {
                const float4 v = sA[grp * ne + tid];
                acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
              }
              const int q = tid / (16 * ND), c = (tid % (16 * ND)) * 4;
              if (c < g.d) store4((T*)a.out + b * a.o_sb + (hq + q) * a.o_sh + c, finish(acc, s_sum[q], s_up[q]));
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

template <int ND, typename T>
cudaError_t launch(const Q8Geom& g, const Q8AttnArgs& a, const int8_t* k_pages, const int8_t* v_pages,
                   const float* scales, const int32_t* table, const int32_t* lens, int grid, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = raise_smem(q8_attention_kernel<ND, T>, (int)smem_bytes<ND>(), done);
  if (e != cudaSuccess) return e;
  const int passes = min(kMaxGroups, (a.G - a.g0 + kMaxG - 1) / kMaxG);
  return launch_pdl(q8_attention_kernel<ND, T>, dim3(grid, passes), dim3(32 * warps_of<ND>()), smem_bytes<ND>(), s, g,
                    a, k_pages, v_pages, (const float2*)scales, table, lens);
}

template <typename T>
cudaError_t launch_nd(const Q8Geom& g, const Q8AttnArgs& a, const int8_t* k_pages, const int8_t* v_pages,
                      const float* scales, const int32_t* table, const int32_t* lens, int grid, cudaStream_t s) {
  switch (g.d64 / 64) {
    case 1: return launch<1, T>(g, a, k_pages, v_pages, scales, table, lens, grid, s);
    case 2: return launch<2, T>(g, a, k_pages, v_pages, scales, table, lens, grid, s);
    case 3: return launch<3, T>(g, a, k_pages, v_pages, scales, table, lens, grid, s);
    default: return launch<4, T>(g, a, k_pages, v_pages, scales, table, lens, grid, s);
  }
}

}  // namespace

// [serving header | partials], for a grid of one CTA per SM.
size_t q8_workspace_bytes(const Q8Geom& g, int G, int sms) {
  const int groups = min(kMaxGroups, (G + kMaxG - 1) / kMaxG);
  return kServeHeader + (size_t)groups * 2 * (sms < kMaxGrid ? sms : kMaxGrid) * kMaxG * (g.d64 + 4) * 4;
}

cudaError_t launch_q8_attention(const Q8Geom& g, bool bf16, int G, float alpha, const void* q, int64_t q_sb,
                                int64_t q_sh, void* out, int64_t o_sb, int64_t o_sh, const int8_t* k_pages,
                                const int8_t* v_pages, const float* scales, const int32_t* table, const int32_t* lens,
                                void* ws, int sms, cudaStream_t s) {
  char* w = (char*)ws;
  sms = sms < kMaxGrid ? sms : kMaxGrid;
  // a pass for every 8 query heads of a KV head; launches of more passes than there are counts for share them
  for (int g0 = 0; g0 < G; g0 += kMaxG * kMaxGroups) {
    Q8AttnArgs a = {q, out, q_sb, q_sh, o_sb, o_sh, alpha, G, g0, (int32_t*)w, (float*)(w + kServeHeader)};
    const cudaError_t e = bf16 ? launch_nd<__nv_bfloat16>(g, a, k_pages, v_pages, scales, table, lens, sms, s)
                               : launch_nd<float>(g, a, k_pages, v_pages, scales, table, lens, sms, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace chunkkv
