// C-ABI entry points of the serving operators: argument checks and launch plans.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "serve.cuh"

namespace chunkkv {

int prefill_simt_rows(int64_t ctas, int sms);                                          // prefill.cu
template <int MAXB>
cudaError_t launch_prefill_simt(bool bf16, const PrefillTable<MAXB>& tab, const PrefillGeom& g, int rows, const void* q,
                                const void* k, const void* v, void* out, cudaStream_t s);
int prefill_tc_heads(int G);                                                           // prefill_tc.cu
int prefill_tc_rows(int G);
int prefill_tc_block();
size_t prefill_tc_part_bytes(int64_t n_items, int d);
template <int MAXB>
cudaError_t launch_prefill_tc(const PrefillTable<MAXB>& tab, const PrefillGeom& p, int kb, int q_total, int k_total,
                              const void* q, const void* k, const void* v, void* out, int32_t* err, float* part,
                              int sms, cudaStream_t s);
cudaError_t launch_q8_resize(const Q8Geom& g, const int32_t* new_lens, int32_t* lens, int32_t* table, int32_t* ring,
                             int32_t* state, int64_t* slots, int n_cap, int sms, cudaStream_t s);   // q8_cache.cu
cudaError_t launch_q8_append(const Q8Geom& g, bool bf16, const void* k, const void* v, int64_t st_b, int64_t st_h,
                             int64_t st_t, const int32_t* counts, const int64_t* slots, int n_cap, int8_t* k_pages,
                             int8_t* v_pages, float* scales, cudaStream_t s);
cudaError_t launch_q8_load(const Q8Geom& g, bool bf16, const int32_t* table, const int32_t* lens, const int8_t* k_pages,
                           const int8_t* v_pages, const float* scales, const int64_t* start, int n_cap, int64_t n_rows,
                           void* k_out, void* v_out, int64_t st_t, cudaStream_t s);
size_t q8_workspace_bytes(const Q8Geom& g, int G, int sms);                                   // q8_attention.cu
cudaError_t launch_q8_attention(const Q8Geom& g, bool bf16, int G, float alpha, const void* q, int64_t q_sb,
                                int64_t q_sh, void* out, int64_t o_sb, int64_t o_sh, const int8_t* k_pages,
                                const int8_t* v_pages, const float* scales, const int32_t* table, const int32_t* lens,
                                void* ws, int sms, cudaStream_t s);

namespace {

constexpr double kLog2e = 1.4426950408889634;

bool aligned(const void* p, uintptr_t n = 16) { return p != nullptr && ((uintptr_t)p & (n - 1)) == 0; }
chunkkv_status cuda_result(cudaError_t e) { return e == cudaSuccess ? CHUNKKV_OK : CHUNKKV_ERR_CUDA; }

// SMs of the current device (152 where no device is visible, as for the compression's plans).
int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) == cudaSuccess && dev < 64 && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) {
    cudaGetLastError();
    return 152;
  }
  if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

bool valid_dtype(int dtype) { return dtype == CHUNKKV_F32 || dtype == CHUNKKV_BF16; }
int elt_size(int dtype) { return dtype == CHUNKKV_BF16 ? 2 : 4; }
bool stride_ok(int64_t s, int elt) { return s >= 0 && s < (INT64_MAX >> 32) && (s * elt) % 16 == 0; }
bool scale_ok(float s) { return s > 0.f && isfinite(s); }

chunkkv_status check_prefill(const chunkkv_prefill_params* p) {
  if (p == nullptr || p->B < 0 || p->Hq < 1 || p->Hkv < 1 || p->d < 1 || !valid_dtype(p->dtype) || !scale_ok(p->scale) ||
      p->Hq % p->Hkv != 0)
    return CHUNKKV_ERR_INVALID_ARG;
  if (p->B > CHUNKKV_MAX_BATCH || p->d > kMaxD || p->Hq > 65535) return CHUNKKV_ERR_UNSUPPORTED;
  const int elt = elt_size(p->dtype);
  if ((p->d * elt) % 16 != 0) return CHUNKKV_ERR_INVALID_ARG;
  const int64_t st[6] = {p->q_stride_t, p->q_stride_h, p->kv_stride_t, p->kv_stride_h, p->o_stride_t, p->o_stride_h};
  for (int64_t s : st)
    if (!stride_ok(s, elt)) return CHUNKKV_ERR_INVALID_ARG;
  if (p->B > 0) {
    if (!p->cu_q || !p->cu_k || p->cu_q[0] != 0 || p->cu_k[0] != 0) return CHUNKKV_ERR_INVALID_ARG;
    for (int b = 0; b < p->B; ++b)
      if (p->cu_q[b + 1] < p->cu_q[b] || p->cu_k[b + 1] < p->cu_k[b]) return CHUNKKV_ERR_INVALID_ARG;
    // work items (at most one per 2 query positions, plus one per sequence, of each head) are counted in 32 bits
    if (((int64_t)p->cu_q[p->B] / 2 + p->B) * p->Hq > INT32_MAX / 2) return CHUNKKV_ERR_UNSUPPORTED;
  }
  return CHUNKKV_OK;
}

// The sequences by descending number of keys (ties in order), with their units: q tiles of `tile` rows, times the
// parts of at most kb key blocks that the last tile's keys make (kb = 0: whole).
template <int MAXB>
void fill_table(const chunkkv_prefill_params* p, int tile, int kb, PrefillTable<MAXB>& t) {
  int32_t order[MAXB];
  t.B = 0;
  for (int b = 0; b < p->B; ++b)
    if (p->cu_q[b + 1] > p->cu_q[b]) order[t.B++] = b;
  const int32_t* ck = p->cu_k;
  std::sort(order, order + t.B, [ck](int32_t x, int32_t y) {
    const int32_t nx = ck[x + 1] - ck[x], ny = ck[y + 1] - ck[y];
    return nx != ny ? nx > ny : x < y;
  });
  int32_t u = 0;
  for (int i = 0; i < t.B; ++i) {
    const int b = order[i];
    const int32_t tq = p->cu_q[b + 1] - p->cu_q[b], tk = ck[b + 1] - ck[b];
    const int32_t blocks = (int32_t)(((int64_t)tk + prefill_tc_block() - 1) / prefill_tc_block());
    const int32_t ns = kb > 0 && blocks > kb ? (blocks - 1) / kb + 1 : 1;
    t.seq[i] = {p->cu_q[b], tq, ck[b], tk, ns};
    t.uoff[i] = u;
    u += ((tq - 1) / tile + 1) * ns;
  }
  t.uoff[t.B] = u;
}

// Key blocks of a work item at most (0: items are not split), and the number of items.
//
// Whole items keep partial results out of memory (128 KB a part, written and read again, against 64 KB of keys
// and values a block).  But where few query rows meet many keys, the longest item takes much longer than an even
// share of the work for every SM; then the keys are split into parts of about that share.
constexpr int64_t kMinPart = 8;                 // blocks of a part at least

void plan_items(const chunkkv_prefill_params* p, int sms, int* kb, int64_t* n_items) {
  const int G = p->Hq / p->Hkv, groups = p->Hq / prefill_tc_heads(G);
  const int64_t rows = prefill_tc_rows(G), block = prefill_tc_block();
  int64_t work = 0, longest = 0, units = 0;
  for (int b = 0; b < p->B; ++b) {
    const int64_t tq = p->cu_q[b + 1] - p->cu_q[b], tk = p->cu_k[b + 1] - p->cu_k[b];
    for (int64_t r = 0; r < tq; r += rows, ++units) {
      const int64_t last = std::min(r + rows, tq) - 1 + tk - tq, n = last < 0 ? 0 : last / block + 1;
      work += n;
      longest = std::max(longest, n);
    }
  }
  const int64_t share = work * groups / sms;
  *kb = 0;
  *n_items = units * groups;
  if (longest < 2 * share + kMinPart) return;
  // the shortest parts that still make one wave of items, where there are such
  for (int64_t n = std::max(kMinPart, share + 1);; n += std::max<int64_t>(1, n / 8)) {
    units = 0;
    for (int b = 0; b < p->B; ++b) {
      const int64_t tq = p->cu_q[b + 1] - p->cu_q[b], tk = p->cu_k[b + 1] - p->cu_k[b];
      units += (tq + rows - 1) / rows * std::max<int64_t>(1, ((tk + block - 1) / block + n - 1) / n);
    }
    if (units * groups > sms && n < longest) continue;
    if (n >= longest) return;
    *kb = (int)n;
    *n_items = units * groups;
    return;
  }
}

// The tensor-core kernel: bf16 rows of up to 128 columns that tensor maps can address (no axis
// longer than 1 with stride 0, strides below 2^40 bytes), a tile of the output within 2^31 elements,
// and a key to attend to.
bool prefill_on_tc(const chunkkv_prefill_params* p) {
  const int64_t most = (int64_t)1 << 39;
  auto axis = [most](int64_t stride, int64_t n) { return n <= 1 || (stride > 0 && stride < most); };
  return p->dtype == CHUNKKV_BF16 && p->d <= 128 && p->B > 0 && p->cu_k[p->B] > 0 &&
         axis(p->q_stride_t, p->cu_q[p->B]) && axis(p->q_stride_h, p->Hq) && axis(p->kv_stride_t, p->cu_k[p->B]) &&
         axis(p->kv_stride_h, p->Hkv) && p->o_stride_t < (1 << 22) && p->o_stride_h < (1 << 22);
}

// Tensor maps address device memory only.
bool device_pointer(const void* p) {
  cudaPointerAttributes a;
  if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return a.type == cudaMemoryTypeDevice;
}

template <int MAXB>
cudaError_t run_prefill(const chunkkv_prefill_params* p, const PrefillGeom& g, bool tc, int kb, const void* q, const void* k,
                        const void* v, void* out, char* ws, cudaStream_t s) {
  static thread_local PrefillTable<MAXB> tab;
  if (!tc) {
    fill_table(p, 64, 0, tab);
    const int rows = prefill_simt_rows((int64_t)tab.uoff[tab.B] * p->Hq, sm_count());
    if (rows != 64) fill_table(p, rows, 0, tab);
    return launch_prefill_simt(p->dtype == CHUNKKV_BF16, tab, g, rows, q, k, v, out, s);
  }
  fill_table(p, prefill_tc_rows(p->Hq / p->Hkv), kb, tab);
  return launch_prefill_tc(tab, g, kb, p->cu_q[p->B], p->cu_k[p->B], q, k, v, out, (int32_t*)ws,
                           (float*)(ws + kServeHeader), sm_count(), s);
}

// How a call runs: on the tensor cores, in items of kb blocks (0: whole), and its workspace.
chunkkv_status plan_prefill(const chunkkv_prefill_params* p, bool* tc, int* kb, int64_t* n_items, size_t* bytes) {
  *tc = prefill_on_tc(p);
  *kb = 0;
  *n_items = 0;
  *bytes = kHeader;
  if (!*tc) return CHUNKKV_OK;
  plan_items(p, sm_count(), kb, n_items);
  if (*n_items > INT32_MAX / 2) return CHUNKKV_ERR_UNSUPPORTED;
  if (*kb > 0) *bytes = kServeHeader + prefill_tc_part_bytes(*n_items, p->d);
  return CHUNKKV_OK;
}

// The part of a cache that every call uses; `pages`: the call reads or writes them.
chunkkv_status check_cache(const chunkkv_q8_cache* c, bool pages, Q8Geom* g) {
  if (c == nullptr || c->B < 0 || c->Hkv < 1 || c->d < 1 || c->n_pages < 1 || c->max_pages < 1)
    return CHUNKKV_ERR_INVALID_ARG;
  if ((int64_t)c->B * c->Hkv > CHUNKKV_Q8_MAX_ROWS || c->d > kMaxD || c->max_pages > INT32_MAX / kPage - 2)
    return CHUNKKV_ERR_UNSUPPORTED;
  if (c->d % 8 != 0 || !aligned(c->table, 4) || !aligned(c->lens, 4)) return CHUNKKV_ERR_INVALID_ARG;
  if (pages && (!aligned(c->k_pages) || !aligned(c->v_pages) || !aligned(c->scales, 8))) return CHUNKKV_ERR_INVALID_ARG;
  *g = {c->B * c->Hkv, c->Hkv, c->d, (c->d + 63) / 64 * 64, c->n_pages, c->max_pages};
  return CHUNKKV_OK;
}

}  // namespace
}  // namespace chunkkv

using namespace chunkkv;

extern "C" {

chunkkv_status chunkkv_prefill_workspace_size(const chunkkv_prefill_params* p, size_t* bytes) {
  if (bytes == nullptr) return CHUNKKV_ERR_INVALID_ARG;
  const chunkkv_status st = check_prefill(p);
  if (st != CHUNKKV_OK) return st;
  bool tc;
  int kb;
  int64_t n_items;
  return plan_prefill(p, &tc, &kb, &n_items, bytes);
}

int32_t chunkkv_prefill_path(const chunkkv_prefill_params* p) {
  if (check_prefill(p) != CHUNKKV_OK) return -1;
  return prefill_on_tc(p) ? 1 : 0;
}

chunkkv_status chunkkv_prefill_attention(const chunkkv_prefill_params* p, const void* q, const void* k, const void* v,
                                         void* out, void* ws, size_t ws_bytes, chunkkv_stream_t stream) {
  const chunkkv_status st = check_prefill(p);
  if (st != CHUNKKV_OK) return st;
  if (p->B == 0 || p->cu_q[p->B] == 0) return CHUNKKV_OK;
  // k and v may be NULL only where no sequence has a key
  const bool no_keys = p->cu_k[p->B] == 0;
  if (!aligned(q) || !aligned(out) || !aligned(ws) || (!no_keys && (!aligned(k) || !aligned(v))))
    return CHUNKKV_ERR_INVALID_ARG;
  bool tc;
  int kb;
  int64_t n_items;
  size_t need;
  const chunkkv_status plan = plan_prefill(p, &tc, &kb, &n_items, &need);
  if (plan != CHUNKKV_OK) return plan;
  if (ws_bytes < need) return CHUNKKV_ERR_WORKSPACE_TOO_SMALL;
  if (tc && !(device_pointer(q) && device_pointer(k) && device_pointer(v))) return CHUNKKV_ERR_INVALID_ARG;
  PrefillGeom g = {p->Hq, p->Hkv, p->Hq / p->Hkv, p->d, (float)(p->scale * kLog2e), p->q_stride_t, p->q_stride_h,
                   p->kv_stride_t, p->kv_stride_h, p->o_stride_t, p->o_stride_h};
  const cudaStream_t cs = (cudaStream_t)stream;
  return cuda_result(p->B <= kSmallBatch
                         ? run_prefill<kSmallBatch>(p, g, tc, kb, q, k, v, out, (char*)ws, cs)
                         : run_prefill<CHUNKKV_MAX_BATCH>(p, g, tc, kb, q, k, v, out, (char*)ws, cs));
}

chunkkv_status chunkkv_q8_resize(const chunkkv_q8_cache* c, const int32_t* new_lens, int64_t* slots, int32_t n_cap,
                                 chunkkv_stream_t stream) {
  Q8Geom g;
  const chunkkv_status st = check_cache(c, false, &g);
  if (st != CHUNKKV_OK) return st;
  if (n_cap < 0) return CHUNKKV_ERR_INVALID_ARG;
  if (n_cap > INT32_MAX - 4 * kPage) return CHUNKKV_ERR_UNSUPPORTED;
  if (g.rows == 0) return CHUNKKV_OK;
  if (!aligned(new_lens, 4) || !aligned(c->ring, 4) || !aligned(c->state, 4) || (slots && !aligned(slots, 8)) ||
      new_lens == c->lens)
    return CHUNKKV_ERR_INVALID_ARG;
  return cuda_result(launch_q8_resize(g, new_lens, c->lens, c->table, c->ring, c->state, slots, n_cap, sm_count(),
                                      (cudaStream_t)stream));
}

chunkkv_status chunkkv_q8_append(const chunkkv_q8_cache* c, int32_t dtype, const void* k, const void* v, int64_t st_b,
                                 int64_t st_h, int64_t st_t, const int32_t* counts, const int64_t* slots,
                                 int32_t n_cap, chunkkv_stream_t stream) {
  Q8Geom g;
  const chunkkv_status st = check_cache(c, true, &g);
  if (st != CHUNKKV_OK) return st;
  if (!valid_dtype(dtype) || n_cap < 0) return CHUNKKV_ERR_INVALID_ARG;
  const int elt = elt_size(dtype);
  if ((g.d * elt) % 16 != 0 || !stride_ok(st_b, elt) || !stride_ok(st_h, elt) || !stride_ok(st_t, elt))
    return CHUNKKV_ERR_INVALID_ARG;
  if (n_cap > INT32_MAX - 4 * kPage) return CHUNKKV_ERR_UNSUPPORTED;
  if (g.rows == 0 || n_cap == 0) return CHUNKKV_OK;
  if (!aligned(k) || !aligned(v) || !aligned(counts, 4) || !aligned(slots, 8)) return CHUNKKV_ERR_INVALID_ARG;
  return cuda_result(launch_q8_append(g, dtype == CHUNKKV_BF16, k, v, st_b, st_h, st_t, counts, slots, n_cap,
                                      c->k_pages, c->v_pages, c->scales, (cudaStream_t)stream));
}

chunkkv_status chunkkv_q8_load(const chunkkv_q8_cache* c, int32_t dtype, const int64_t* start, int32_t n_cap,
                               void* k_out, void* v_out, int64_t st_t, chunkkv_stream_t stream) {
  return chunkkv_q8_load_bounded(c, dtype, start, n_cap, INT64_MAX, k_out, v_out, st_t, stream);
}

chunkkv_status chunkkv_q8_load_bounded(const chunkkv_q8_cache* c, int32_t dtype, const int64_t* start, int32_t n_cap,
                                       int64_t n_rows, void* k_out, void* v_out, int64_t st_t,
                                       chunkkv_stream_t stream) {
  Q8Geom g;
  const chunkkv_status st = check_cache(c, true, &g);
  if (st != CHUNKKV_OK) return st;
  if (!valid_dtype(dtype) || n_cap < 0 || n_rows < 0) return CHUNKKV_ERR_INVALID_ARG;
  const int elt = elt_size(dtype);
  if ((g.d * elt) % 16 != 0 || !stride_ok(st_t, elt)) return CHUNKKV_ERR_INVALID_ARG;
  if (n_cap > INT32_MAX - 4 * kPage) return CHUNKKV_ERR_UNSUPPORTED;
  if (g.rows == 0 || n_cap == 0 || n_rows == 0) return CHUNKKV_OK;
  if (!aligned(start, 8) || !aligned(k_out) || !aligned(v_out)) return CHUNKKV_ERR_INVALID_ARG;
  return cuda_result(launch_q8_load(g, dtype == CHUNKKV_BF16, c->table, c->lens, c->k_pages, c->v_pages, c->scales,
                                    start, std::min(n_cap, c->max_pages * kPage), n_rows, k_out, v_out, st_t,
                                    (cudaStream_t)stream));
}

chunkkv_status chunkkv_q8_workspace_size(const chunkkv_q8_cache* c, int32_t G, size_t* bytes) {
  Q8Geom g;
  const chunkkv_status st = check_cache(c, false, &g);
  if (st != CHUNKKV_OK) return st;
  if (bytes == nullptr || G < 1) return CHUNKKV_ERR_INVALID_ARG;
  *bytes = q8_workspace_bytes(g, G, sm_count());
  return CHUNKKV_OK;
}

chunkkv_status chunkkv_q8_attention(const chunkkv_q8_cache* c, int32_t dtype, int32_t G, float scale, const void* q,
                                    int64_t q_stride_b, int64_t q_stride_h, void* out, int64_t o_stride_b,
                                    int64_t o_stride_h, void* ws, size_t ws_bytes, chunkkv_stream_t stream) {
  Q8Geom g;
  const chunkkv_status st = check_cache(c, true, &g);
  if (st != CHUNKKV_OK) return st;
  if (!valid_dtype(dtype) || G < 1 || !scale_ok(scale)) return CHUNKKV_ERR_INVALID_ARG;
  const int elt = elt_size(dtype);
  const int64_t strides[4] = {q_stride_b, q_stride_h, o_stride_b, o_stride_h};
  for (int64_t s : strides)
    if (!stride_ok(s, elt)) return CHUNKKV_ERR_INVALID_ARG;
  if ((g.d * elt) % 16 != 0) return CHUNKKV_ERR_INVALID_ARG;
  if (G > 65535) return CHUNKKV_ERR_UNSUPPORTED;
  if (g.rows == 0) return CHUNKKV_OK;
  if (!aligned(q) || !aligned(out) || !aligned(ws)) return CHUNKKV_ERR_INVALID_ARG;
  if (ws_bytes < q8_workspace_bytes(g, G, sm_count())) return CHUNKKV_ERR_WORKSPACE_TOO_SMALL;
  return cuda_result(launch_q8_attention(g, dtype == CHUNKKV_BF16, G, (float)(scale * kLog2e), q, q_stride_b,
                                         q_stride_h, out, o_stride_b, o_stride_h, c->k_pages, c->v_pages, c->scales,
                                         c->table, c->lens, ws, sm_count(), (cudaStream_t)stream));
}

}  // extern "C"
