// Single-token attention over the 8-bit paged cache.
//
//   O_g = sum_j 2^(t_j) s_v V_j / sum_j 2^(t_j),   t_j = scale log2(e) s_k (q_g . K_j)
//
// over the tokens j of one cache row, K and V int8 codes, s_k and s_v the scales of
// the token's page.  One CTA takes one query head and walks its row's pages with a
// running maximum and sum.
#include "serve.cuh"

namespace chunkkv {
namespace {

constexpr int kThreads = 128;

struct Q8AttnArgs {
  const void* q;
  void* out;
  int64_t q_sb, q_sh, o_sb, o_sh;
  float alpha;
  int32_t G;
};

__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <typename T>
__global__ void __launch_bounds__(kThreads)
q8_attention_kernel(Q8Geom g, Q8AttnArgs a, const int8_t* __restrict__ k_pages, const int8_t* __restrict__ v_pages,
                    const float* __restrict__ scales, const int32_t* __restrict__ table,
                    const int32_t* __restrict__ lens) {
  __shared__ float s_q[kMaxD], s_t[kPage], s_half[2][kPage];
  pdl_wait();
  const int r = blockIdx.x, gq = blockIdx.y, tid = threadIdx.x;
  const int b = r / g.Hkv, hq = (r % g.Hkv) * a.G + gq;
  const T* q = (const T*)a.q + b * a.q_sb + hq * a.q_sh;
  for (int e = tid; e < g.d64; e += kThreads) s_q[e] = e < g.d ? to_float(q[e]) : 0.f;
  const int n = safe_len(lens[r], g.max_pages);
  float m = -INFINITY, l = 0.f, o[2] = {0.f, 0.f};
  for (int j = 0; j * kPage < n; ++j) {
    const int64_t page = safe_page(table[(int64_t)r * g.max_pages + j], g.n_pages);
    const float sk = scales[page * 2] * a.alpha, sv = scales[page * 2 + 1];
    const int8_t* kp = k_pages + page * (int64_t)(g.d64 * kPage);
    const int8_t* vp = v_pages + page * (int64_t)(g.d64 * kPage);
    __syncthreads();
    const int t = tid & 63, half = tid >> 6;
    float acc = 0.f;
    for (int c = half * g.d64 / 2; c < (half + 1) * g.d64 / 2; ++c)
      acc = fmaf(s_q[c], (float)kp[(c >> 6) * (kPage * 64) + t * 64 + (c & 63)], acc);
    s_half[half][t] = acc;
    __syncthreads();
    if (tid < kPage) s_t[tid] = j * kPage + tid < n ? (s_half[0][tid] + s_half[1][tid]) * sk : -INFINITY;
    __syncthreads();
    float top = m;
    for (int i = 0; i < kPage; ++i) top = fmaxf(top, s_t[i]);
    const float ref = top == -INFINITY ? 0.f : top;
    const float f = exp2f(m - ref);
    m = top;
    l *= f;
    for (int i = 0; i < kPage; ++i) l += exp2f(s_t[i] - ref);
    for (int c = tid, x = 0; c < g.d64; c += kThreads, ++x) {
      float acc2 = 0.f;
      for (int i = 0; i < min(kPage, n - j * kPage); ++i)
        acc2 = fmaf(exp2f(s_t[i] - ref), (float)vp[c * kPage + i], acc2);
      o[x] = o[x] * f + acc2 * sv;
    }
  }
  T* out = (T*)a.out + b * a.o_sb + hq * a.o_sh;
  for (int c = tid, x = 0; c < g.d; c += kThreads, ++x) store1(out + c, l == 0.f ? 0.f : o[x] / l);
  pdl_trigger();
}

}  // namespace

size_t q8_workspace_bytes(const Q8Geom& g, int G) { return 256; }

cudaError_t launch_q8_attention(const Q8Geom& g, bool bf16, int G, float alpha, const void* q, int64_t q_sb,
                                int64_t q_sh, void* out, int64_t o_sb, int64_t o_sh, const int8_t* k_pages,
                                const int8_t* v_pages, const float* scales, const int32_t* table, const int32_t* lens,
                                void* ws, int sms, cudaStream_t s) {
  Q8AttnArgs a = {q, out, q_sb, q_sh, o_sb, o_sh, alpha, G};
  auto fn = bf16 ? q8_attention_kernel<__nv_bfloat16> : q8_attention_kernel<float>;
  return launch_pdl(fn, dim3(g.rows, G), dim3(kThreads), 0, s, g, a, k_pages, v_pages, scales, table, lens);
}

}  // namespace chunkkv
