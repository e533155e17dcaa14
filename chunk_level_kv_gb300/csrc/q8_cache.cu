// The 8-bit paged cache: page tables and slot maps from lengths, writing rows,
// reading rows back.
//
// A cache row is one (sequence, KV head): chunk compression keeps another number of
// tokens for every head, so every head has a length, pages and scales of its own.
// A page holds 64 tokens of one row, in the order in which the attention kernel's
// fragments read it:
//   keys    [d64 / 64][64 tokens][64 columns]  int8     (d64: d rounded up to 64)
//   values  [d64][64 tokens]                   int8     (transposed)
//   scales  [2]                                fp32     keys, values
#include "serve.cuh"

namespace chunkkv {
namespace {

// ------------------------------------------------------------ tables and slot maps

constexpr int kResizeThreads = 512;
constexpr int kSlotRun = 256;                   // tokens of a row that a warp maps: 5 pages at most, a lane each

__device__ __forceinline__ int pages_of(int n) { return n > 0 ? (n - 1) / kPage + 1 : 0; }

// A ring position below 3 n (head < n, at most n free before the call and after it).
__device__ __forceinline__ int wrap(long long x, int n) {
  if (x >= n) x -= n;
  if (x >= n) x -= n;
  return (int)x;
}

// Exclusive scan of (a, b) over the block; totals in ta, tb.
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long& ta, long long& tb) {
  __shared__ long long s[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long xa = a, xb = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long ya = __shfl_up_sync(0xffffffffu, xa, o), yb = __shfl_up_sync(0xffffffffu, xb, o);
    if (lane >= o) { xa += ya; xb += yb; }
  }
  if (lane == 31) { s[0][warp] = xa; s[1][warp] = xb; }
  __syncthreads();
  if (warp == 0) {
    const int nw = blockDim.x >> 5;
    long long wa = lane < nw ? s[0][lane] : 0, wb = lane < nw ? s[1][lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long ya = __shfl_up_sync(0xffffffffu, wa, o), yb = __shfl_up_sync(0xffffffffu, wb, o);
      if (lane >= o) { wa += ya; wb += yb; }
    }
    s[0][lane] = wa;
    s[1][lane] = wb;
  }
  __syncthreads();
  const long long pa = warp ? s[0][warp - 1] : 0, pb = warp ? s[1][warp - 1] : 0;
  ta = s[0][31];
  tb = s[1][31];
  a = pa + xa - a;
  b = pb + xb - b;
}

// Every CTA scans all rows' page counts (a few KB from L2) and then serves its own
// run of rows: pages that a row gains come from the ring's head in row order, pages
// that it gives back go behind the ring's free part, and the slots of its new tokens
// follow from both.  The entries read (free before the call) and those written (not
// free before it) never meet, so the CTAs need no order among them; the last one to
// arrive writes the lengths and the ring's state.  A CTA arrives once it has read them
// (its own rows' lengths go to shared memory), before it writes anything: a release
// with nothing to wait for, behind which the writes run.
// Latency bounds it (four dependent trips to L2): 6.5 us for 2048 rows with a 288-token
// slot map (4.7 MB), 6.2 us for 128 rows that gain 6.5 thousand tokens each (6.7 MB).
__global__ void __launch_bounds__(kResizeThreads)
resize_kernel(Q8Geom g, const int32_t* __restrict__ new_lens, int32_t* __restrict__ lens, int32_t* __restrict__ table,
              int32_t* __restrict__ ring, int32_t* state, int64_t* __restrict__ slots, int n_cap, int rows_per_cta) {
  extern __shared__ long long s_off[];                      // [2][rows_per_cta] pages gained / given before the row
  int* s_len = (int*)(s_off + 2 * rows_per_cta);            // [2][rows_per_cta] its length, and the new one
  __shared__ bool s_last;
  pdl_wait();
  const int tid = threadIdx.x;
  const int r0 = blockIdx.x * rows_per_cta, r1 = min(g.rows, r0 + rows_per_cta);
  const int chunk = (g.rows + kResizeThreads - 1) / kResizeThreads;
  const int c0 = min(g.rows, tid * chunk), c1 = min(g.rows, c0 + chunk);
  const int head = ((volatile int32_t*)state)[kRingHead], n_free = ((volatile int32_t*)state)[kRingFree];
  long long grow = 0, give = 0;
  bool bad = false;
#pragma unroll 4
  for (int r = c0; r < c1; ++r) {
    const int n = lens[r], m = new_lens[r];
    bad |= n < 0 || m < 0 || pages_of(m) > g.max_pages || pages_of(n) > g.max_pages || (slots && m - n > n_cap);
    const int d = pages_of(m) - pages_of(n);
    grow += max(d, 0);
    give += max(-d, 0);
  }
  long long grown, given;
  bad = __syncthreads_or(bad) || head < 0 || head >= g.n_pages || n_free < 0 || n_free > g.n_pages;
  block_scan2(grow, give, grown, given);
  const bool ok = !bad && grown <= n_free && n_free - grown + given <= g.n_pages;
  for (int r = c0; r < c1; ++r) {
    const int n = lens[r], m = new_lens[r];
    if (r >= r0 && r < r1) {
      s_off[r - r0] = grow;
      s_off[rows_per_cta + r - r0] = give;
      s_len[r - r0] = n;
      s_len[rows_per_cta + r - r0] = m;
    }
    const int d = pages_of(m) - pages_of(n);
    grow += max(d, 0);
    give += max(-d, 0);
  }
  __syncthreads();
  if (tid == 0) {
    int before;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(before) : "l"(&state[kRingTicket]) : "memory");
    s_last = before == (int)gridDim.x - 1;
  }
  if (ok) {
    // table entries: a warp per row
    for (int r = r0 + (tid >> 5); r < r1; r += kResizeThreads / 32) {
      const int have = pages_of(s_len[r - r0]), need = pages_of(s_len[rows_per_cta + r - r0]);
      int32_t* row = table + (int64_t)r * g.max_pages;
      for (int j = have + (tid & 31); j < need; j += 32)
        row[j] = ring[wrap(head + s_off[r - r0] + (j - have), g.n_pages)];
      for (int j = need + (tid & 31); j < have; j += 32) {
        ring[wrap(head + n_free + s_off[rows_per_cta + r - r0] + (j - need), g.n_pages)] = row[j];
        row[j] = -1;
      }
    }
  }
  // slots: a warp per run of kSlotRun tokens of a row.  Its lanes hold the run's pages (those that the row had
  // from the table, the others straight from the ring), and every step writes 64 slots.
  if (slots) {
    const int runs = (n_cap + kSlotRun - 1) / kSlotRun, lane = tid & 31;
    for (int w = tid >> 5; w < (r1 - r0) * runs; w += kResizeThreads / 32) {
      const int r = r0 + w / runs, i0 = w % runs * kSlotRun, i1 = min(n_cap, i0 + kSlotRun);
      const int n = s_len[r - r0], m = s_len[rows_per_cta + r - r0], have = pages_of(n);
      const int added = ok ? m - n : 0;
      int64_t* row_slots = slots + (int64_t)r * n_cap;
      int32_t page = -1;
      const int first = (n + i0) / kPage, j = first + lane;     // i0 < added makes these positions of the row
      if (i0 < added && j < pages_of(m))
        page = j < have ? table[(int64_t)r * g.max_pages + j] : ring[wrap(head + s_off[r - r0] + (j - have), g.n_pages)];
#pragma unroll 2
      for (int i = i0 + lane; i - lane < i1; i += 32) {
        const int pos = n + i;
        const int32_t p = __shfl_sync(0xffffffffu, page, i < added ? pos / kPage - first : 0);
        if (i < i1) row_slots[i] = i < added ? (int64_t)p * kPage + pos % kPage : -1;
      }
    }
  }
  __syncthreads();
  if (s_last) {
    if (ok)
      for (int r = tid; r < g.rows; r += kResizeThreads) lens[r] = new_lens[r];
    if (tid == 0) {
      if (ok) {
        state[kRingHead] = (int32_t)((head + grown) % g.n_pages);
        state[kRingFree] = (int32_t)(n_free - grown + given);
      }
      state[kRingStatus] = ok ? 0 : bad ? 2 : 1;
      state[kRingTicket] = 0;
    }
  }
  pdl_trigger();
}

// ------------------------------------------------------------ writing

constexpr int kIoThreads = 256;
constexpr float kInv127 = 1.0f / 127.0f;
constexpr float kSmallest = 7.888609052210118e-31f;          // 2^-100: below it a block counts as zero

// Eight elements of a row as they lie in memory, and one of them as fp32.
template <typename T>
struct Vec8;
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ void load(const float* p) { a = ((const float4*)p)[0]; b = ((const float4*)p)[1]; }
  __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};
template <>
struct Vec8<__nv_bfloat16> {
  uint4 v;
  __device__ void load(const __nv_bfloat16* p) { v = *(const uint4*)p; }
  __device__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  *(float4*)p = make_float4(x[0], x[1], x[2], x[3]);
  *(float4*)(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *(const uint32_t*)&b;
  }
  *(uint4*)p = make_uint4(w[0], w[1], w[2], w[3]);
}

// The 4 x 4 bytes of four words transposed: byte b of word i goes to byte i of word b.
__device__ __forceinline__ void transpose4(uint32_t (&w)[4]) {
  const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[2], w[3], 0x5140);
  const uint32_t c = __byte_perm(w[0], w[1], 0x7362), d = __byte_perm(w[2], w[3], 0x7362);
  w[0] = __byte_perm(a, b, 0x5410);
  w[1] = __byte_perm(a, b, 0x7632);
  w[2] = __byte_perm(c, d, 0x5410);
  w[3] = __byte_perm(c, d, 0x7632);
}

// Rounded to the nearest code, ties to even; NaN (0 x inf of a block with an
// infinity, whose scale is not finite either) becomes 0.
__device__ __forceinline__ int code_of(float x) { return max(-127, min(127, __float2int_rn(x))); }

// The codes of a 32-bit word times ratio, rounded again.
__device__ __forceinline__ uint32_t recode(uint32_t w, float ratio) {
  uint32_t o = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o |= ((uint32_t)code_of((float)(int8_t)(w >> (8 * i)) * ratio) & 0xFFu) << (8 * i);
  return o;
}

struct AppendArgs {
  const void* x[2];                // keys, values [B, Hkv, n_cap, d]
  int8_t* pages[2];
  int64_t st_b, st_h, st_t;
  int32_t n_cap;
};

// One CTA writes the part of one page that a row's new tokens fill, of the keys
// (blockIdx.z 0) or of the values (1).  Its threads hold the tokens in registers while
// the largest magnitude, and from it the page's scale, is found; a page that already
// holds tokens keeps its scale unless the new ones are larger, else its codes are
// rounded again for the new one.  Keys are written as they were read, 8 bytes a
// vector; values go through shared memory as codes and leave in 16-token pieces of a
// column, the bytes transposed 4 x 4 in registers.
// HBM bounds it: 8 x 6582 bf16 tokens of 128 columns (40 MB) are written and then read
// back (load_kernel, the same bytes the other way) in 19.8 us, 3.8 TB/s with both
// launches (16.7 us, 10.4 and 6.3, while the L2 holds them); with the tokens in shared
// memory as fp32 it was 27 us there.
template <int ND, typename T>
__global__ void __launch_bounds__(kIoThreads)
append_kernel(Q8Geom g, AppendArgs a, const int32_t* __restrict__ counts, const int64_t* __restrict__ slots,
              float* __restrict__ scales) {
  constexpr int kV8 = 8 * ND, kVecs = kPage * kV8 / kIoThreads;      // vectors of a row, and of a thread
  constexpr int kPitch = 64 * ND + 4;                                // bytes of a token's codes in shared memory
  __shared__ uint32_t s_top[kIoThreads / 32];
  __shared__ __align__(16) uint8_t s_code[kPage * kPitch];
  pdl_wait();
  const int r = blockIdx.y, which = blockIdx.z, tid = threadIdx.x;
  const int64_t* row_slots = slots + (int64_t)r * a.n_cap;
  const int n = min(max(counts[r], 0), a.n_cap);
  const int off0 = (int)(row_slots[0] & (kPage - 1));
  const int i0 = max(0, (int)blockIdx.x * kPage - off0), i1 = min(n, ((int)blockIdx.x + 1) * kPage - off0);
  if (i0 < i1) {                                                     // the same for the whole CTA
    const int64_t slot = row_slots[i0];
    const T* x = (const T*)(which ? a.x[1] : a.x[0]) + (r / g.Hkv) * a.st_b + (r % g.Hkv) * a.st_h + i0 * a.st_t;
    const int t0 = (int)(slot & (kPage - 1)), nt = min(i1 - i0, kPage - t0);
    const int64_t page = slot >> 6;
    Vec8<T> raw[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int t = (i * kIoThreads + tid) / kV8, c = (i * kIoThreads + tid) % kV8 * 8;
      if (t < nt && c < g.d) raw[i].load(x + t * a.st_t + c); else raw[i].zero();
    }
    const bool inside = slot >= 0 && page < g.n_pages;
    const float before = t0 == 0 || !inside ? 0.f : scales[page * 2 + which];
    // magnitudes compared as bit patterns: a NaN is above infinity and ends in the scale
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      float w[8];
      raw[i].get(w);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(w[e]) & 0x7FFFFFFFu);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if ((tid & 31) == 0) s_top[tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kIoThreads / 32; ++i) top = max(top, s_top[i]);
    const float amax = __uint_as_float(top);
    const float grown = amax < kSmallest ? 0.f : amax * kInv127;
    const float scale = grown > before || grown != grown ? grown : before;   // a NaN scale stays one
    const float ratio = scale != before ? __fdiv_rn(before, scale) : 1.f;
    const float inv = scale > 0.f ? __frcp_rn(scale) : 0.f;
    const bool again = t0 > 0 && ratio != 1.f;                       // older codes of the page to be rounded again
    int8_t* pg = (which ? a.pages[1] : a.pages[0]) + page * (int64_t)(64 * ND * kPage);
    if (inside) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        const int t = (i * kIoThreads + tid) / kV8, c = (i * kIoThreads + tid) % kV8 * 8;
        float w[8];
        raw[i].get(w);
        uint32_t q[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e >> 2] |= ((uint32_t)code_of(w[e] * inv) & 0xFFu) << (8 * (e & 3));
        if (which == 0) {
          if (t < nt) *(uint2*)(pg + (c >> 6) * (kPage * 64) + (t0 + t) * 64 + (c & 63)) = make_uint2(q[0], q[1]);
        } else if (t < nt) {
          uint32_t* dst = (uint32_t*)(s_code + (t0 + t) * kPitch + c);
          dst[0] = q[0];
          dst[1] = q[1];
        }
      }
      if (which == 0 && again)
        for (int i = tid; i < t0 * (4 * ND); i += kIoThreads) {
          const int t = i % t0, c = i / t0;                          // 16 columns of an older token
          uint4* p = (uint4*)(pg + (c / 4) * (kPage * 64) + t * 64 + (c % 4) * 16);
          uint4 w = *p;
          w.x = recode(w.x, ratio); w.y = recode(w.y, ratio); w.z = recode(w.z, ratio); w.w = recode(w.w, ratio);
          *p = w;
        }
      if (tid == 0 && (scale != before || t0 == 0)) scales[page * 2 + which] = scale;
    }
    if (which == 1) {
      __syncthreads();
      for (int i = tid; inside && i < 16 * ND * 4; i += kIoThreads) {
        const int c = (i >> 2) * 4, base = (i & 3) * 16;             // 4 columns, 16 tokens
        const bool touched = base < t0 + nt && base + 16 > t0;
        if (!touched && !(again && base < t0)) continue;
        const bool part = base < t0 || base + 16 > t0 + nt;          // other tokens' bytes are kept
        uint32_t w[4][4];                                            // [4 tokens each][word: 4 columns, then 4 tokens]
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
          for (int b = 0; b < 4; ++b) w[e][b] = *(const uint32_t*)(s_code + (base + 4 * e + b) * kPitch + c);
          transpose4(w[e]);
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          uint4* p = (uint4*)(pg + (c + b) * kPage + base);
          uint32_t o[4] = {w[0][b], w[1][b], w[2][b], w[3][b]};
          if (part) {
            const uint4 old4 = *p;
            uint32_t old[4] = {old4.x, old4.y, old4.z, old4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (again) old[e] = recode(old[e], ratio);
              uint32_t keep = 0;
#pragma unroll
              for (int z = 0; z < 4; ++z)
                if (base + 4 * e + z < t0 || base + 4 * e + z >= t0 + nt) keep |= 0xFFu << (8 * z);
              o[e] = (o[e] & ~keep) | (old[e] & keep);
            }
          }
          *p = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
  }
  pdl_trigger();
}

// ------------------------------------------------------------ reading back

struct LoadArgs {
  const int8_t* pages[2];
  void* out[2];
  int64_t st_t, n_rows;            // rows of the outputs: what lies past them is not written
  int32_t n_cap;
};

// One CTA reads one page of a row: codes times the page's scale, rounded once to the
// output's type (values: 4 x 4 bytes transposed in registers).  Timed with append_kernel.
template <typename T>
__global__ void __launch_bounds__(kIoThreads)
load_kernel(Q8Geom g, LoadArgs a, const int32_t* __restrict__ table, const int32_t* __restrict__ lens,
            const float* __restrict__ scales, const int64_t* __restrict__ start) {
  constexpr int kPitch = kPage + 4;                           // bytes of a column in shared memory
  extern __shared__ __align__(16) uint8_t bytes[];            // values: [d64][kPitch]
  pdl_wait();
  const int r = blockIdx.y, which = blockIdx.z, tid = threadIdx.x, j = blockIdx.x;
  const int n = min(safe_len(lens[r], g.max_pages), a.n_cap);
  int nt = min(kPage, n - j * kPage);
  const int64_t at = start[r];
  if (nt > 0 && at >= 0) {
    const int64_t page = safe_page(table[(int64_t)r * g.max_pages + j], g.n_pages);
    const float scale = scales[page * 2 + which];
    nt = (int)min((int64_t)nt, max(a.n_rows - at - j * kPage, (int64_t)0));
    const int8_t* pg = (which ? a.pages[1] : a.pages[0]) + page * (int64_t)(g.d64 * kPage);
    T* out = (T*)(which ? a.out[1] : a.out[0]) + (at + j * kPage) * a.st_t;
    const int v8 = g.d / 8;
    if (which == 0) {
#pragma unroll 4
      for (int i = tid; i < nt * v8; i += kIoThreads) {
        const int t = i / v8, c = (i % v8) * 8;
        const uint2 w = *(const uint2*)(pg + (c >> 6) * (kPage * 64) + t * 64 + (c & 63));
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (float)(int8_t)((e < 4 ? w.x : w.y) >> (8 * (e & 3))) * scale;
        store8(out + t * a.st_t + c, x);
      }
    } else {
#pragma unroll 2
      for (int i = tid; i < g.d64 * 4; i += kIoThreads) {
        const uint4 w = *(const uint4*)(pg + i * 16);
        uint32_t* dst = (uint32_t*)(bytes + (i >> 2) * kPitch + (i & 3) * 16);
        dst[0] = w.x; dst[1] = w.y; dst[2] = w.z; dst[3] = w.w;
      }
      __syncthreads();
      for (int i = tid; i < v8 * 16; i += kIoThreads) {
        const int c = i % v8 * 8, t = i / v8 * 4;             // 8 columns, 4 tokens
        if (t >= nt) continue;
        uint32_t w[2][4];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e >> 2][e & 3] = *(const uint32_t*)(bytes + (c + e) * kPitch + t);
        transpose4(w[0]);
        transpose4(w[1]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (t + k >= nt) break;
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = (float)(int8_t)(w[e >> 2][k] >> (8 * (e & 3))) * scale;
          store8(out + (t + k) * a.st_t + c, x);
        }
      }
    }
  }
  pdl_trigger();
}

template <typename T>
cudaError_t launch_append(const Q8Geom& g, const AppendArgs& a, const int32_t* counts, const int64_t* slots,
                          float* scales, cudaStream_t s) {
  // n_cap tokens that begin anywhere in a page touch this many pages
  const dim3 grid((a.n_cap + 2 * (kPage - 1)) / kPage, g.rows, 2);
  switch (g.d64 / 64) {
    case 1: return launch_pdl(append_kernel<1, T>, grid, dim3(kIoThreads), 0, s, g, a, counts, slots, scales);
    case 2: return launch_pdl(append_kernel<2, T>, grid, dim3(kIoThreads), 0, s, g, a, counts, slots, scales);
    case 3: return launch_pdl(append_kernel<3, T>, grid, dim3(kIoThreads), 0, s, g, a, counts, slots, scales);
    default: return launch_pdl(append_kernel<4, T>, grid, dim3(kIoThreads), 0, s, g, a, counts, slots, scales);
  }
}

}  // namespace

cudaError_t launch_q8_resize(const Q8Geom& g, const int32_t* new_lens, int32_t* lens, int32_t* table, int32_t* ring,
                             int32_t* state, int64_t* slots, int n_cap, int sms, cudaStream_t s) {
  const int grid = max(1, min(g.rows, sms));
  const int per = (g.rows + grid - 1) / grid;
  return launch_pdl(resize_kernel, dim3((g.rows + per - 1) / per), dim3(kResizeThreads),
                    (size_t)per * 2 * (sizeof(long long) + sizeof(int)), s, g, new_lens, lens, table, ring, state, slots, n_cap, per);
}

cudaError_t launch_q8_append(const Q8Geom& g, bool bf16, const void* k, const void* v, int64_t st_b, int64_t st_h,
                             int64_t st_t, const int32_t* counts, const int64_t* slots, int n_cap, int8_t* k_pages,
                             int8_t* v_pages, float* scales, cudaStream_t s) {
  AppendArgs a = {{k, v}, {k_pages, v_pages}, st_b, st_h, st_t, n_cap};
  return bf16 ? launch_append<__nv_bfloat16>(g, a, counts, slots, scales, s)
              : launch_append<float>(g, a, counts, slots, scales, s);
}

cudaError_t launch_q8_load(const Q8Geom& g, bool bf16, const int32_t* table, const int32_t* lens, const int8_t* k_pages,
                           const int8_t* v_pages, const float* scales, const int64_t* start, int n_cap, int64_t n_rows,
                           void* k_out, void* v_out, int64_t st_t, cudaStream_t s) {
  LoadArgs a = {{k_pages, v_pages}, {k_out, v_out}, st_t, n_rows, n_cap};
  const size_t smem = (size_t)g.d64 * (kPage + 4);
  const dim3 grid((n_cap + kPage - 1) / kPage, g.rows, 2);
  auto fn = bf16 ? load_kernel<__nv_bfloat16> : load_kernel<float>;
  return launch_pdl(fn, grid, dim3(kIoThreads), smem, s, g, a, table, lens, scales, start);
}

}  // namespace chunkkv
