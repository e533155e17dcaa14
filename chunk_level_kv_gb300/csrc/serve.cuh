// Shared definitions of the serving operators: attention over packed prompts and
// the 8-bit paged cache (page tables, writing, reading back, decode attention).
#pragma once

#include "common.cuh"

namespace chunkkv {

// The start of a serving workspace: the header that all calls share (common.cuh), and behind it decode attention's
// counts (q8_attention.cu), which partial results of any call leave alone.
constexpr size_t kHeader = 256, kServeHeader = 3840;

// ------------------------------------------------------------ prefill attention

// Sequences of a packed batch in the order in which their work is taken (longest
// first, so that the last items to start are short), with the q tile offsets.
struct PrefillSeq {
  int32_t q0, tq, k0, tk;          // first packed row and length of its queries and of its keys
  int32_t ns;                      // parts into which the keys of its q tiles are split (1: whole)
};
template <int MAXB>
struct PrefillTable {
  int32_t B;
  int32_t uoff[MAXB + 1];          // units (q tiles x parts) before sequence i
  PrefillSeq seq[MAXB];
};
// Two sizes of the table, which travels as a kernel argument: 0.8 KB for batches of
// up to 32 sequences and 24 KB above (a launch copies its arguments).
constexpr int kSmallBatch = 32;

struct PrefillGeom {
  int32_t Hq, Hkv, G, d;
  float alpha;                     // scale * log2(e): logits are handled as base-2 exponents
  int64_t q_st, q_sh, kv_st, kv_sh, o_st, o_sh;   // element strides (token, head)
};

// Sequence index of unit u.
template <int MAXB>
__device__ __forceinline__ int find_seq(const PrefillTable<MAXB>& t, int u) {
  int lo = 0, hi = t.B;            // uoff[lo] <= u < uoff[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.uoff[mid] <= u) lo = mid; else hi = mid;
  }
  return lo;
}

// ------------------------------------------------------------ 8-bit cache

constexpr int kPage = CHUNKKV_Q8_PAGE;          // tokens per page
static_assert(kPage == 64, "the page layout and the kernels take 64 tokens a page");

struct Q8Geom {
  int32_t rows, Hkv, d, d64;       // d64: d rounded up to 64 (columns of a page)
  int32_t n_pages, max_pages;
};

// A page index read from the table, kept inside the pool whatever the table holds.
__device__ __forceinline__ int64_t safe_page(int32_t p, int n_pages) {
  return (uint32_t)p < (uint32_t)n_pages ? p : 0;
}
// A row's length, kept inside what its table row can hold.
__device__ __forceinline__ int safe_len(int32_t n, int max_pages) {
  return (int)min((int64_t)max(n, 0), (int64_t)max_pages * kPage);
}

// The ring's state words (chunkkv_q8_cache.state).
enum { kRingHead = 0, kRingFree = 1, kRingStatus = 2, kRingTicket = 3 };

// Raises a kernel's dynamic shared-memory limit once per device (`done`: a bit per
// device, one word per kernel instance).
template <typename F>
cudaError_t raise_smem(F* kernel, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace chunkkv
