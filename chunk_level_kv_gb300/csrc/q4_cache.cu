// The 4-bit paged cache: writing rows, reading rows back (its tables are the 8-bit cache's,
// resize_kernel of q8_cache.cu).
//
// A token's groups of 64 columns are quantised by themselves, so a token is final when it is
// written: nothing of a page changes when further tokens join it.  For a group whose values
// lie in [lo, hi],
//   m = lo rounded down to bf16,  s = (hi - m) / 15 rounded up to bf16,  c = round((x - m) / s)
// and a code stands for s c + m.  Rounding outwards keeps every value within half a step of
// a code; bf16 keeps fp32's range, and m is exact where the inputs are bf16.  Only where
// 15 s + m would be infinite is s the next lower bf16: values still are within half a step.
#include "q4.cuh"

namespace chunkkv {
namespace {

constexpr int kIoThreads = 256;
constexpr float kInv15 = 1.0f / 15.0f;
constexpr float kRound = 12582912.f;                         // 1.5 2^23
constexpr float kSmallest = 7.888609052210118e-31f;          // 2^-100: a group that spans less has step 0

// Smallest and largest, NaN if either is.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The step of a group near the end of the range: s, rounded up, is lowered to the next bf16 as long as 15 s + m would be
// infinite, in bf16 if hi itself is finite there.  Twice at most: 15 s + m then is below hi by more than roundings raise it.
constexpr float kHighEnd = 1.7e38f;                          // 2^127: 15 s + m passes hi by 2^-7 of it at most
constexpr float kBf16End = 339617752923046005526922703901628039168.f;      // (2 - 2^-8) 2^127, which rounds to infinity in bf16
__device__ __noinline__ float s_below_end(float m, float s, float hi) {
  const float end = hi < kBf16End ? kBf16End : INFINITY;
#pragma unroll 1
  for (int i = 0; i < 2; ++i)
    if (s > 0.f && !(fmaf(15.f, s, m) < end)) s = __uint_as_float(__float_as_uint(s) - 0x10000u);
  return s;
}

// Eight elements of a row as they lie in memory, and as fp32.
template <typename T>
struct Vec8;
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) { a = ((const float4*)p)[0]; b = ((const float4*)p)[1]; }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  // smallest and largest element (NaN if one is)
  __device__ __forceinline__ void range(float& lo, float& hi) const {
    float x[8];
    get(x);
    lo = min_nan(min_nan(min_nan(x[0], x[1]), min_nan(x[2], x[3])), min_nan(min_nan(x[4], x[5]), min_nan(x[6], x[7])));
    hi = max_nan(max_nan(max_nan(x[0], x[1]), max_nan(x[2], x[3])), max_nan(max_nan(x[4], x[5]), max_nan(x[6], x[7])));
  }
};
template <>
struct Vec8<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *(const uint4*)p; }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  // in pairs: bf16 comparisons are exact
  __device__ __forceinline__ void range(float& lo, float& hi) const {
    const __nv_bfloat162* x = (const __nv_bfloat162*)&v;
    const __nv_bfloat162 l = __hmin2_nan(__hmin2_nan(x[0], x[1]), __hmin2_nan(x[2], x[3]));
    const __nv_bfloat162 h = __hmax2_nan(__hmax2_nan(x[0], x[1]), __hmax2_nan(x[2], x[3]));
    lo = min_nan(__low2float(l), __high2float(l));
    hi = max_nan(__low2float(h), __high2float(h));
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

// ------------------------------------------------------------ writing

struct Q4AppendArgs {
  const void* x[2];                // keys, values [B, Hkv, n_cap, d]
  int64_t st_b, st_h, st_t;
  int32_t n_cap;
};

// One CTA writes the part of one page that a row's new tokens fill, of the keys
// (blockIdx.z 0) or of the values (1).  Four lanes hold a group of a token, 16 columns
// each, and find its smallest and largest value by shuffles (with eight lanes, what a group
// costs once was two thirds of the instructions).  A lane's codes are two words of the keys'
// part; values go through shared memory, a byte a code, and leave as words of eight tokens of a
// column (bytes paired into nibbles and transposed 4 x 4 in registers), merged with the older
// tokens' codes where a word is shared.
// Instructions bound it (630 a warp, issue slots 83 %): 32 rows of 13164 tokens of 128 columns in bf16
// (276 MB) 74 us, 3.7 TB/s; in fp32 (492 MB) 95 us, 5.2 TB/s.
template <int ND, typename T>
__global__ void __launch_bounds__(kIoThreads)
q4_append_kernel(Q4Geom g, Q4AppendArgs a, const int32_t* __restrict__ counts, const int64_t* __restrict__ slots,
                 uint8_t* __restrict__ pages) {
  constexpr int kV16 = 4 * ND, kVecs = ND;                           // 16-column pieces of a token, and of a thread
  static_assert(kPage * kV16 == kVecs * kIoThreads, "a page's pieces");
  constexpr int kPitch = 64 * ND + 4;                                // bytes of a token's codes in shared memory
  __shared__ __align__(16) uint8_t s_code[kPage * kPitch];
  pdl_wait();
  const int r = blockIdx.y, which = blockIdx.z, tid = threadIdx.x;
  const int64_t* row_slots = slots + (int64_t)r * a.n_cap;
  const int n = min(max(counts[r], 0), a.n_cap);
  const int off0 = (int)(row_slots[0] & (kPage - 1));
  const int i0 = max(0, (int)blockIdx.x * kPage - off0), i1 = min(n, ((int)blockIdx.x + 1) * kPage - off0);
  if (i0 < i1) {                                                     // the same for the whole CTA
    const int64_t slot = row_slots[i0];
    const int64_t page = slot >> 6;
    const int t0 = (int)(slot & (kPage - 1)), nt = min(i1 - i0, kPage - t0);
    const T* x = (const T*)(which ? a.x[1] : a.x[0]) + (r / g.Hkv) * a.st_b + (r % g.Hkv) * a.st_h + i0 * a.st_t;
    const bool inside = slot >= 0 && page < g.n_pages;
    uint8_t* pg = pages + page * q4_page_bytes(ND);
    uint32_t* k_words = (uint32_t*)pg;
    uint32_t* ms_words = (uint32_t*)(pg + (which ? q4_v_ms(ND) : q4_k_ms(ND)));
    if (inside) {
      Vec8<T> raw[kVecs][2];
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {                              // every load is under way before the first is used
        const int v = i * kIoThreads + tid, t = v / kV16, c = v % kV16 * 16;
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (t < nt && c + 8 * k < g.d) raw[i][k].load(x + t * a.st_t + c + 8 * k);
      }
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        const int v = i * kIoThreads + tid, t = v / kV16, c = v % kV16 * 16;
        if ((i * kIoThreads + (tid & ~31)) / kV16 >= nt) break;      // the whole warp is past the tokens
        float lo = INFINITY, hi = -INFINITY;
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (t < nt && c + 8 * k < g.d) {
            float l, h;
            raw[i][k].range(l, h);
            lo = min_nan(lo, l);
            hi = max_nan(hi, h);
          }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
          hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        // m downwards, s upwards: towards larger magnitudes is up by 0xFFFF and cut off
        const uint32_t lb = __float_as_uint(lo);
        float m = __uint_as_float((lb + ((int)lb < 0 ? 0xFFFFu : 0u)) & 0xFFFF0000u);
        const float span = hi - m;
        float s = span >= kSmallest ? __uint_as_float((__float_as_uint(span * kInv15) + 0xFFFFu) & 0xFFFF0000u) : 0.f;
        const bool bad = !(span <= 3.402823466e38f);                 // NaN, infinities, or further apart than fp32 holds
        if (bad) {
          m = __uint_as_float(0x7FC00000u);
          s = 0.f;
        }
        if (hi > kHighEnd) s = s_below_end(m, s, hi);
        const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
        if (t < nt) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            // The codes as whole numbers in fp32, 0 to 15: 15 s is not below hi - m (by a fiftieth, if s was lowered), so
            // (x - m) / s rounds to 15 at most.
            // Adding and taking off 1.5 2^23 rounds to the nearest, ties to even.
            const bool zero = bad || c + 8 * k >= g.d;               // codes of no value, or of columns past the end
            float w[8];
            raw[i][k].get(w);
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = __fadd_rn(__fmul_rn(w[e] - m, inv), kRound) - kRound;
            if (which == 0) {
              // nibbles 0 .. 3 are items 0, 2, 4, 6: four codes are a whole number below 2^16
              const float even = fmaf(fmaf(fmaf(w[6], 16.f, w[4]), 16.f, w[2]), 16.f, w[0]);
              const float odd = fmaf(fmaf(fmaf(w[7], 16.f, w[5]), 16.f, w[3]), 16.f, w[1]);
              const uint32_t word = __byte_perm(__float_as_uint(even + kRound), __float_as_uint(odd + kRound), 0x5410);
              k_words[q4_k_word(ND, t0 + t, c + 8 * k)] = zero ? 0 : word;
            } else {
              uint32_t* dst = (uint32_t*)(s_code + (t0 + t) * kPitch + c + 8 * k);       // a byte a code, in the columns' order
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t four = __byte_perm(__float_as_uint(fmaf(w[4 * e + 1], 256.f, w[4 * e]) + kRound),
                                                  __float_as_uint(fmaf(w[4 * e + 3], 256.f, w[4 * e + 2]) + kRound), 0x5410);
                dst[e] = zero ? 0 : four;
              }
            }
          }
          if ((c & 63) == 0) ms_words[(c >> 6) * kPage + t0 + t] = (__float_as_uint(m) >> 16) | (__float_as_uint(s) & 0xFFFF0000u);
        }
      }
    }
    if (which == 1) {
      __syncthreads();
      uint32_t* v_words = (uint32_t*)(pg + q4_v(ND));
      for (int i = tid; inside && i < 64 * ND * 2; i += kIoThreads) {
        // columns c .. c + 3, tokens t .. t + 7; the words of a warp lie in runs of 16
        const int c = (i >> 5) * 16 + ((i >> 1) & 1) * 8 + ((i >> 4) & 1) * 4, t = ((i >> 2) & 3) * 16 + (i & 1) * 8;
        if (t >= t0 + nt || t + 8 <= t0) continue;
        uint32_t b[8], keep = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool fresh = t + e >= t0 && t + e < t0 + nt;
          b[e] = fresh ? *(const uint32_t*)(s_code + (t + e) * kPitch + c) : 0;
          if (!fresh) keep |= 15u << (4 * q4_nibble(e));
        }
        // byte k of a column's word holds nibbles 2 k and 2 k + 1: items 0 and 2, 4 and 6, 1 and 3, 5 and 7
        uint32_t w[4] = {b[0] | b[2] << 4, b[4] | b[6] << 4, b[1] | b[3] << 4, b[5] | b[7] << 4};
        transpose4(w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t* p = v_words + q4_v_word(c + j, t);
          *p = keep ? w[j] | (*p & keep) : w[j];
        }
      }
    }
  }
  pdl_trigger();
}

// ------------------------------------------------------------ reading back

struct Q4LoadArgs {
  void* out[2];
  int64_t st_t, n_rows;            // rows of the outputs: what lies past them is not written
  int32_t n_cap;
};

// One CTA reads one page of a row: s c + m, rounded once to the output's type.  The values'
// codes come through shared memory (blocks of 16 columns 528 bytes apart: their words of
// the same tokens lie in different banks).  Latency bounds it (a CTA's length, start, table entry, steps
// and codes come one after another; writing the same bytes alone takes 33 us): the rows of
// q4_append_kernel's figure 56 us, 4.9 TB/s; in fp32 99 us, 5.0 TB/s.
template <int ND, typename T>
__global__ void __launch_bounds__(kIoThreads)
q4_load_kernel(Q4Geom g, Q4LoadArgs a, const int32_t* __restrict__ table, const int32_t* __restrict__ lens,
               const uint8_t* __restrict__ pages, const int64_t* __restrict__ start) {
  constexpr int kV8 = 8 * ND, kBlock = 132;                   // words of 16 columns, padded
  __shared__ __align__(16) uint32_t s_words[4 * ND * kBlock];
  __shared__ uint32_t s_ms[ND * kPage];
  pdl_wait();
  const int r = blockIdx.y, which = blockIdx.z, tid = threadIdx.x, j = blockIdx.x;
  const int n = min(safe_len(lens[r], g.max_pages), a.n_cap);
  int nt = min(kPage, n - j * kPage);
  const int64_t at = start[r];
  if (nt > 0 && at >= 0) {
    const int64_t page = safe_page(table[(int64_t)r * g.max_pages + j], g.n_pages);
    nt = (int)min((int64_t)nt, max(a.n_rows - at - j * kPage, (int64_t)0));
    const uint8_t* pg = pages + page * q4_page_bytes(ND);
    T* out = (T*)(which ? a.out[1] : a.out[0]) + (at + j * kPage) * a.st_t;
    const uint32_t* ms = (const uint32_t*)(pg + (which ? q4_v_ms(ND) : q4_k_ms(ND)));
    for (int i = tid; i < ND * kPage; i += kIoThreads) s_ms[i] = ms[i];
    if (which) {
      const uint4* src = (const uint4*)(pg + q4_v(ND));
      for (int i = tid; i < 128 * ND; i += kIoThreads) *(uint4*)(s_words + (i >> 5) * kBlock + (i & 31) * 4) = src[i];
    }
    __syncthreads();
    if (which == 0) {
      const uint32_t* words = (const uint32_t*)pg;
#pragma unroll 4
      for (int i = tid; i < nt * kV8; i += kIoThreads) {
        const int t = i / kV8, c = i % kV8 * 8;
        if (c >= g.d) continue;
        const uint32_t w = words[q4_k_word(ND, t, c)], p = s_ms[(c >> 6) * kPage + t];
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fmaf((float)(w >> (4 * q4_nibble(e)) & 15u), q4_s(p), q4_m(p));
        store8(out + t * a.st_t + c, x);
      }
    } else {
      for (int i = tid; i < kV8 * 16; i += kIoThreads) {
        const int c = i % kV8 * 8, t = i / kV8 * 4;           // 8 columns, 4 tokens
        if (t >= nt || c >= g.d) continue;
        const uint32_t* src = s_words + (c >> 4) * kBlock + (q4_v_word(c & 15, t) & 127);
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = src[16 * e] >> (t & 4 ? 8 : 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (t + k >= nt) break;
          const uint32_t p = s_ms[(c >> 6) * kPage + t + k];
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = fmaf((float)(w[e] >> (4 * q4_nibble(k)) & 15u), q4_s(p), q4_m(p));
          store8(out + (t + k) * a.st_t + c, x);
        }
      }
    }
  }
  pdl_trigger();
}

template <int ND, typename T>
cudaError_t append_nd(const Q4Geom& g, const Q4AppendArgs& a, const int32_t* counts, const int64_t* slots, uint8_t* pages,
                      cudaStream_t s) {
  // n_cap tokens that begin anywhere in a page touch this many pages
  const dim3 grid((a.n_cap + 2 * (kPage - 1)) / kPage, g.rows, 2);
  return launch_pdl(q4_append_kernel<ND, T>, grid, dim3(kIoThreads), 0, s, g, a, counts, slots, pages);
}
template <int ND, typename T>
cudaError_t load_nd(const Q4Geom& g, const Q4LoadArgs& a, const int32_t* table, const int32_t* lens, const uint8_t* pages,
                    const int64_t* start, cudaStream_t s) {
  const dim3 grid((a.n_cap + kPage - 1) / kPage, g.rows, 2);
  return launch_pdl(q4_load_kernel<ND, T>, grid, dim3(kIoThreads), 0, s, g, a, table, lens, pages, start);
}

template <typename T>
cudaError_t append_t(const Q4Geom& g, const Q4AppendArgs& a, const int32_t* counts, const int64_t* slots, uint8_t* pages,
                     cudaStream_t s) {
  switch (g.d64 / 64) {
    case 1: return append_nd<1, T>(g, a, counts, slots, pages, s);
    case 2: return append_nd<2, T>(g, a, counts, slots, pages, s);
    case 3: return append_nd<3, T>(g, a, counts, slots, pages, s);
    default: return append_nd<4, T>(g, a, counts, slots, pages, s);
  }
}
template <typename T>
cudaError_t load_t(const Q4Geom& g, const Q4LoadArgs& a, const int32_t* table, const int32_t* lens, const uint8_t* pages,
                   const int64_t* start, cudaStream_t s) {
  switch (g.d64 / 64) {
    case 1: return load_nd<1, T>(g, a, table, lens, pages, start, s);
    case 2: return load_nd<2, T>(g, a, table, lens, pages, start, s);
    case 3: return load_nd<3, T>(g, a, table, lens, pages, start, s);
    default: return load_nd<4, T>(g, a, table, lens, pages, start, s);
  }
}

}  // namespace

cudaError_t launch_q4_append(const Q4Geom& g, bool bf16, const void* k, const void* v, int64_t st_b, int64_t st_h,
                             int64_t st_t, const int32_t* counts, const int64_t* slots, int n_cap, uint8_t* pages,
                             cudaStream_t s) {
  const Q4AppendArgs a = {{k, v}, st_b, st_h, st_t, n_cap};
  return bf16 ? append_t<__nv_bfloat16>(g, a, counts, slots, pages, s) : append_t<float>(g, a, counts, slots, pages, s);
}

cudaError_t launch_q4_load(const Q4Geom& g, bool bf16, const int32_t* table, const int32_t* lens, const uint8_t* pages,
                           const int64_t* start, int n_cap, int64_t n_rows, void* k_out, void* v_out, int64_t st_t,
                           cudaStream_t s) {
  const Q4LoadArgs a = {{k_out, v_out}, st_t, n_rows, n_cap};
  return bf16 ? load_t<__nv_bfloat16>(g, a, table, lens, pages, start, s) : load_t<float>(g, a, table, lens, pages, start, s);
}

}  // namespace chunkkv
