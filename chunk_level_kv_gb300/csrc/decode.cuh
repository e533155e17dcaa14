// What the single-token attention kernels over paged caches share: bounded waits for
// bulk copies, the lookup of pages, and the m16n8k16 product.
#pragma once

#include <cuda_fp16.h>

#include "serve.cuh"

namespace chunkkv {
namespace decode {

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
__device__ __forceinline__ void copy_page(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
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

  __device__ __forceinline__ void load(const Q8Geom& g, const int32_t* lens, int lane) {
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
  __device__ __forceinline__ void locate(const Q8Geom& g, const int32_t* lens, int lane, int64_t x, int& row, int& j, int& n) {
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

// The pages of all rows in order (or what else work is counted in: size(i) of item i) are cut
// into one contiguous run [x0, x1) per CTA, whatever the rows' lengths, which only the device
// knows: every CTA finds its run by a scan over the lengths.  Rows of up to kWholeRow pages are
// not cut (each kernel has its own number): a row in two pieces costs the CTAs that share it
// about 4 us (partials, a counter, the join), a page about 0.4 us of a CTA's share of the
// bandwidth, and the eight warps take eight pages at once.  A cut within kNearEnd pages
// of a long row's begin or end moves there, so that a CTA seldom has a second row for a few
// pages.
constexpr int kWholeRow = 8;
constexpr int kNearEnd = 3;
static_assert(kWholeRow > 2 * kNearEnd, "a row's two ends do not meet");

template <int W>
struct RunShared {
  long long scan[W];
  int64_t cut[2], start[2];                      // the run's ends, and the pages before the rows that they lie in
  int row[2];
};
struct Run {
  int64_t total, nc;                             // pages of all rows, and CTAs that have a run
};
// Ends in shared memory; to be read after a __syncthreads.
// whole: items of up to this size are not cut; least: a CTA's run is not shorter (but for the last ones).
template <int W, typename F>
__device__ __forceinline__ Run plan_run(int count, F size, RunShared<W>& sh, int whole = kWholeRow, int least = 1) {
  constexpr int kThreads = 32 * W;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int chunk = (count + kThreads - 1) / kThreads;
  const int c0 = min(count, tid * chunk), c1 = min(count, c0 + chunk);
  long long mine = 0;
  for (int r = c0; r < c1; ++r) mine += size(r);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sh.scan[warp] = incl;
  __syncthreads();
  long long total = 0, before = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if (i == warp) before = total;
    total += sh.scan[i];
  }
  before += incl - mine;                         // pages before this thread's rows
  // no more runs than pages: every CTA that shares a row has a part of it
  const int64_t most = (total + least - 1) / least, nc = most < gridDim.x ? most : gridDim.x;
  const bool busy = blockIdx.x < nc;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t cut = busy ? total * (blockIdx.x + k) / nc : total;
    if (cut == total) {
      if (tid == 0) sh.cut[k] = total;
    } else if (cut >= before && cut < before + mine) {
      int64_t x = before;
      int r = c0, n = 0;
      for (; r < c1; ++r) {
        n = size(r);
        if (x + n > cut) break;
        x += n;
      }
      // short rows stay in one piece, and a long one's end is no place to cut either
      sh.cut[k] = n <= whole || cut - x <= kNearEnd ? x : x + n - cut <= kNearEnd ? x + n : cut;
      sh.row[k] = r;
      sh.start[k] = x;
    }
  }
  return {total, nc};
}
template <int W>
__device__ __forceinline__ Run plan_run(const Q8Geom& g, const int32_t* __restrict__ lens, RunShared<W>& sh, int whole = kWholeRow) {
  return plan_run<W>(g.rows, [&](int r) { return pages_of(safe_len(lens[r], g.max_pages)); }, sh, whole);
}
// The CTAs that share an item whose n units begin at unit x and that is cut: from the last one whose cut is at its
// begin or moves there, to the last one whose cut does not move to its end.
__device__ __forceinline__ int first_of(const Run& run, int64_t x) { return (int)(((x + kNearEnd + 1) * run.nc - 1) / run.total); }
__device__ __forceinline__ int last_of(const Run& run, int64_t x, int n) {
  return (int)(((x + n - kNearEnd) * run.nc - 1) / run.total);
}

}  // namespace decode
}  // namespace chunkkv
