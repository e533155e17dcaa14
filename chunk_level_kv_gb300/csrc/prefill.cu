// Attention over packed prompts on the FMA pipes: any head dimension up to 256, fp32
// or bf16.
//
//   O_i = sum_{j <= i + Tk - Tq} softmax_j(scale q_i . k_j) v_j    per query head
//
// in one pass over the keys with a running row maximum m and sum l (base-2
// exponents, fp32): a new tile with maximum m' rescales what is held by 2^(m - m').
// A CTA owns 16 RM query rows of one head and walks the keys in tiles of 64; each of
// its 256 threads holds RM x 4 logits and RM rows x d/16 columns of the output in
// registers, and Q, K, V and the tile's probabilities lie in shared memory in fp32.
// RM = 4 where its CTAs fill the GPU; RM = 1 where they do not (four times as many CTAs,
// each of which reads more shared memory per product).
// A query row without any key (Tq > Tk) gives zeros.
//
// What bounds it: the FMA pipes and the shared-memory reads that feed them.  4 d products
// a visible pair on 152 x 128 lanes would take 2 us for 512 tokens, 4 query heads of 64
// columns; there its CTAs' latency decides, tile after tile: 26 us (16-row CTAs and the
// next tile read ahead; 54 us with 64-row CTAs).  8192 bf16 tokens of 32 heads take it
// 16.9 ms (33 TFLOP/s), against 0.31 ms on the tensor cores.
#include "serve.cuh"

namespace chunkkv {
namespace {

constexpr int kTile = 64;                                // keys of a tile
constexpr int kThreads = 256;

template <int ND>
constexpr int row_pitch() { return 64 * ND + 4; }        // floats; 4 more than a multiple of 32: no bank conflicts
template <int RM, int ND>
constexpr size_t smem_bytes() {
  return (size_t)((16 * RM + kTile) * row_pitch<ND>() + kTile * 64 * ND + 16 * RM * (kTile + 1)) * sizeof(float);
}

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) { return *(const float4*)p; }
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 v = *(const uint2*)p;
  return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                     __uint_as_float(v.y & 0xFFFF0000u));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *(float4*)p = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *(uint2*)p = make_uint2(*(uint32_t*)&a, *(uint32_t*)&b);
}

// `rows` rows of d elements, `pitch` floats apart in shared memory, columns up to
// 64 ND and rows at or beyond `rows` zero.
template <int ROWS, int ND, typename T>
__device__ __forceinline__ void load_tile(float* s, int pitch, const T* g, int64_t stride, int rows, int d) {
#pragma unroll 4
  for (int i = threadIdx.x; i < ROWS * 16 * ND; i += kThreads) {
    const int r = i / (16 * ND), c = (i % (16 * ND)) * 4;
    *(float4*)(s + r * pitch + c) = r < rows && c < d ? load4(g + r * stride + c) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

// O += P V over one tile.  SELECT: a hidden key adds nothing even where its value is
// an infinity or NaN (0 x inf would be NaN).
template <int RM, int ND, bool SELECT>
__device__ __forceinline__ void add_pv(float (&o)[RM][4 * ND], const float* sP, const float* sV, int ty, int tx,
                                       int first_last, int j0) {
  for (int j = 0; j < kTile; ++j) {
    float p[RM];
#pragma unroll
    for (int r = 0; r < RM; ++r) p[r] = sP[(ty * RM + r) * (kTile + 1) + j];
#pragma unroll
    for (int c = 0; c < ND; ++c) {
      const float4 v = *(const float4*)(sV + j * 64 * ND + c * 64 + tx * 4);
#pragma unroll
      for (int r = 0; r < RM; ++r) {
        if (SELECT && j0 + j > first_last + r) continue;
        o[r][4 * c] = fmaf(p[r], v.x, o[r][4 * c]);
        o[r][4 * c + 1] = fmaf(p[r], v.y, o[r][4 * c + 1]);
        o[r][4 * c + 2] = fmaf(p[r], v.z, o[r][4 * c + 2]);
        o[r][4 * c + 3] = fmaf(p[r], v.w, o[r][4 * c + 3]);
      }
    }
  }
}

template <int RM, int ND, typename T, int MAXB>
__global__ void __launch_bounds__(kThreads)
prefill_simt_kernel(const __grid_constant__ PrefillTable<MAXB> tab, PrefillGeom g, const T* __restrict__ q,
                    const T* __restrict__ k, const T* __restrict__ v, T* __restrict__ out) {
  extern __shared__ __align__(16) float smem[];
  constexpr int kPitch = row_pitch<ND>();
  float* sQ = smem;
  float* sK = sQ + 16 * RM * kPitch;
  float* sV = sK + kTile * kPitch;
  float* sP = sV + kTile * 64 * ND;
  const int i = find_seq(tab, blockIdx.x);
  const PrefillSeq sq = tab.seq[i];
  // later q tiles of a sequence see more keys: they start first
  const int r0 = (tab.uoff[i + 1] - 1 - (int)blockIdx.x) * (16 * RM);
  const int h = blockIdx.y, hk = h / g.G;
  const int rows = min(16 * RM, sq.tq - r0);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int last0 = r0 + ty * RM + (sq.tk - sq.tq);          // last key that this thread's first row sees
  const int n_keys = min(sq.tk, r0 + rows + (sq.tk - sq.tq));  // keys that the last row sees (may be <= 0)
  pdl_wait();
  load_tile<16 * RM, ND>(sQ, kPitch, q + (int64_t)(sq.q0 + r0) * g.q_st + h * g.q_sh, g.q_st, rows, g.d);
  float m[RM], l[RM], o[RM][4 * ND];
#pragma unroll
  for (int r = 0; r < RM; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int c = 0; c < 4 * ND; ++c) o[r][c] = 0.f;
  }
  // heads of up to 128 columns: a tile's keys and values are read into registers while the one before is in use
  constexpr bool kAhead = ND <= 2;
  constexpr int kVecs = kAhead ? kTile * 16 * ND / kThreads : 1;
  float4 rk[kVecs], rv[kVecs];
  auto read_ahead = [&](int j0) {
    const int64_t koff = (int64_t)(sq.k0 + j0) * g.kv_st + hk * g.kv_sh;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int x = i * kThreads + threadIdx.x, r = x / (16 * ND), c = (x % (16 * ND)) * 4;
      const bool in = r < sq.tk - j0 && c < g.d;
      rk[i] = in ? load4(k + koff + r * g.kv_st + c) : make_float4(0.f, 0.f, 0.f, 0.f);
      rv[i] = in ? load4(v + koff + r * g.kv_st + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  if (kAhead && n_keys > 0) read_ahead(0);
  for (int j0 = 0; j0 < n_keys; j0 += kTile) {
    __syncthreads();                                         // the previous tile's readers are done
    const int nk = min(kTile, sq.tk - j0);
    if constexpr (kAhead) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        const int x = i * kThreads + threadIdx.x, r = x / (16 * ND), c = (x % (16 * ND)) * 4;
        *(float4*)(sK + r * kPitch + c) = rk[i];
        *(float4*)(sV + r * 64 * ND + c) = rv[i];
      }
    } else {
      const int64_t koff = (int64_t)(sq.k0 + j0) * g.kv_st + hk * g.kv_sh;
      load_tile<kTile, ND>(sK, kPitch, k + koff, g.kv_st, nk, g.d);
      load_tile<kTile, ND>(sV, 64 * ND, v + koff, g.kv_st, nk, g.d);
    }
    __syncthreads();
    if (kAhead && j0 + kTile < n_keys) read_ahead(j0 + kTile);
    float s[RM][4];
#pragma unroll
    for (int r = 0; r < RM; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) s[r][c] = 0.f;
    for (int e = 0; e < g.d; e += 4) {
      float4 a[RM], b[4];
#pragma unroll
      for (int r = 0; r < RM; ++r) a[r] = *(const float4*)(sQ + (ty * RM + r) * kPitch + e);
#pragma unroll
      for (int c = 0; c < 4; ++c) b[c] = *(const float4*)(sK + (tx + 16 * c) * kPitch + e);
#pragma unroll
      for (int r = 0; r < RM; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          s[r][c] = fmaf(a[r].w, b[c].w, fmaf(a[r].z, b[c].z, fmaf(a[r].y, b[c].y, fmaf(a[r].x, b[c].x, s[r][c]))));
    }
    const bool masked = j0 + kTile > r0 + (sq.tk - sq.tq) + 1 || nk < kTile;   // the same for the whole CTA
#pragma unroll
    for (int r = 0; r < RM; ++r) {
      const int limit = min(last0 + r, sq.tk - 1);
      float top = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        s[r][c] = j0 + tx + 16 * c <= limit ? s[r][c] * g.alpha : -INFINITY;
        top = fmaxf(top, s[r][c]);
      }
#pragma unroll
      for (int x = 1; x < 16; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float mn = fmaxf(m[r], top);
      const float ref = mn == -INFINITY ? 0.f : mn;          // no key so far: every term is 2^-inf = 0
      const float f = exp2f(m[r] - ref);
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float p = exp2f(s[r][c] - ref);
        sP[(ty * RM + r) * (kTile + 1) + tx + 16 * c] = p;
        sum += p;
      }
#pragma unroll
      for (int x = 1; x < 16; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      l[r] = l[r] * f + sum;
      m[r] = mn;
#pragma unroll
      for (int c = 0; c < 4 * ND; ++c) o[r][c] *= f;
    }
    __syncwarp();                                            // a row's probabilities come from its own half warp
    if (masked)
      add_pv<RM, ND, true>(o, sP, sV, ty, tx, last0, j0);
    else
      add_pv<RM, ND, false>(o, sP, sV, ty, tx, last0, j0);
  }
#pragma unroll
  for (int r = 0; r < RM; ++r) {
    const int row = ty * RM + r;
    if (row >= rows) continue;
    // no visible key: zeros; logits that are all -inf: NaN (else l is 1 or more, from the maximum)
    const float inv = l[r] != 0.f ? 1.f / l[r] : last0 + r < 0 ? 0.f : NAN;
    T* po = out + (int64_t)(sq.q0 + r0 + row) * g.o_st + h * g.o_sh;
#pragma unroll
    for (int c = 0; c < ND; ++c)
      if (c * 64 + tx * 4 < g.d)
        store4(po + c * 64 + tx * 4,
               make_float4(o[r][4 * c] * inv, o[r][4 * c + 1] * inv, o[r][4 * c + 2] * inv, o[r][4 * c + 3] * inv));
  }
  pdl_trigger();
}

template <int RM, int ND, typename T, int MAXB>
cudaError_t launch(const PrefillTable<MAXB>& tab, const PrefillGeom& g, const void* q, const void* k, const void* v,
                   void* out, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = raise_smem(prefill_simt_kernel<RM, ND, T, MAXB>, (int)smem_bytes<RM, ND>(), done);
  if (e != cudaSuccess) return e;
  return launch_pdl(prefill_simt_kernel<RM, ND, T, MAXB>, dim3(tab.uoff[tab.B], g.Hq), dim3(kThreads), smem_bytes<RM, ND>(), s,
                    tab, g, (const T*)q, (const T*)k, (const T*)v, (T*)out);
}

template <int RM, typename T, int MAXB>
cudaError_t launch_nd(const PrefillTable<MAXB>& tab, const PrefillGeom& g, const void* q, const void* k, const void* v,
                      void* out, cudaStream_t s) {
  switch ((g.d + 63) / 64) {
    case 1: return launch<RM, 1, T, MAXB>(tab, g, q, k, v, out, s);
    case 2: return launch<RM, 2, T, MAXB>(tab, g, q, k, v, out, s);
    case 3: return launch<RM, 3, T, MAXB>(tab, g, q, k, v, out, s);
    default: return launch<RM, 4, T, MAXB>(tab, g, q, k, v, out, s);
  }
}

}  // namespace

// Query rows of a CTA, for a call that makes `ctas` CTAs of 64 rows.
int prefill_simt_rows(int64_t ctas, int sms) { return ctas < sms ? 16 : 64; }

template <int MAXB>
cudaError_t launch_prefill_simt(bool bf16, const PrefillTable<MAXB>& tab, const PrefillGeom& g, int rows, const void* q,
                                const void* k, const void* v, void* out, cudaStream_t s) {
  if (rows == 16)
    return bf16 ? launch_nd<1, __nv_bfloat16, MAXB>(tab, g, q, k, v, out, s) : launch_nd<1, float, MAXB>(tab, g, q, k, v, out, s);
  return bf16 ? launch_nd<4, __nv_bfloat16, MAXB>(tab, g, q, k, v, out, s) : launch_nd<4, float, MAXB>(tab, g, q, k, v, out, s);
}
template cudaError_t launch_prefill_simt<kSmallBatch>(bool, const PrefillTable<kSmallBatch>&, const PrefillGeom&, int,
                                                      const void*, const void*, const void*, void*, cudaStream_t);
template cudaError_t launch_prefill_simt<CHUNKKV_MAX_BATCH>(bool, const PrefillTable<CHUNKKV_MAX_BATCH>&,
                                                            const PrefillGeom&, int, const void*, const void*,
                                                            const void*, void*, cudaStream_t);

}  // namespace chunkkv
