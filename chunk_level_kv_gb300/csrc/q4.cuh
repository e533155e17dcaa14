// The 4-bit paged cache: where a page's parts lie (chunkkv.h states the layout).
#pragma once

#include "serve.cuh"

namespace chunkkv {

using Q4Geom = Q8Geom;                           // the same tables and pages of 64 tokens

// nd: 64-column groups of a token.  A page's parts, in bytes from its begin; a token's or a column's codes come in
// pieces of 8 bytes that hold 16 of them.
constexpr int q4_page_bytes(int nd) { return 4608 * nd; }
constexpr int q4_k_ms(int nd) { return 2048 * nd; }          // the keys' (m, s), behind their codes
constexpr int q4_v(int nd) { return 2304 * nd; }             // the values' codes
constexpr int q4_v_ms(int nd) { return 4352 * nd; }          // the values' (m, s)

// The nibble of item 0 .. 7 in its 32-bit word: pairs of items lie 16 bits apart, so that one mask yields two f16.
__host__ __device__ constexpr int q4_nibble(int i) { return (i >> 1) + 4 * (i & 1); }

// Words (of 8 codes) from the part's begin: columns c .. c + 7 of a token, tokens t .. t + 7 of a column.
__device__ __forceinline__ int q4_k_word(int nd, int token, int c) {
  return (token * 4 + ((c >> 4) & 3)) * (2 * nd) + (c >> 6) * 2 + ((c >> 3) & 1);
}
__device__ __forceinline__ int q4_v_word(int c, int token) {
  return (c >> 4) * 128 + (c & 7) * 16 + (token >> 4) * 4 + ((c >> 3) & 1) * 2 + ((token >> 3) & 1);
}

// A group's m and s as they are held: two bf16 in a word.
__device__ __forceinline__ float q4_m(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float q4_s(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

}  // namespace chunkkv
