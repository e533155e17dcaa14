/*
 * chunkkv.h - ChunkKV chunk-level KV-cache compression on one NVIDIA GB300 (sm_103a).
 *
 * The operation is the one of "ChunkKV: Semantic-Preserving KV Cache
 * Compression for Efficient Long-Context LLM Inference" (NeurIPS'25 notes):
 *   §4.1 Algorithm 1  - score every key against an observation window of the
 *                       last w queries, sum the scores per chunk of c tokens,
 *                       keep the top k = floor(L_max / c) chunks plus the last
 *                       w tokens, index_select K and V by the kept positions;
 *   §4.2 Algorithm 2  - layers with l mod N_reuse != 0 do not score; they
 *                       gather with the index list of layer
 *                       floor(l / N_reuse) * N_reuse.
 * The window scores are attention probabilities as in "Kara" §2 Eq. (1):
 * softmax over all T keys of (Q_w K^T / sqrt(d)) for each window-query row,
 * summed over the w window rows and over the G = Hq / Hkv query heads that
 * share a KV head (query head hq belongs to KV head hq / G).  By default no
 * causal mask applies inside the window (the algorithm as printed);
 * chunkkv_params.causal_window = 1 masks each window query to the keys at or
 * before its own position.  Top-k ties go to the lower chunk index.
 * The kept list is the ascending, duplicate-free union of the selected
 * chunks' tokens and the last w tokens.
 *
 * Conventions for every call
 *  - Device pointers point to GPU global memory owned by the caller; the
 *    library never allocates or frees device memory while it runs and keeps
 *    no per-call state between calls (its one fixed device array is the
 *    scratch of chunkkv_score_noalloc, described there).  Host arrays
 *    (cu_seqlens, pointer tables) are read during the call only.
 *  - "Addressable" pointers (the K/V data that only the gather and the
 *    portable scoring kernel touch, marked below) may also point to host
 *    memory that the GPU reads and writes directly: pinned (cudaHostAlloc,
 *    cudaHostRegister) or, on systems with coherent host access, any host
 *    memory.  The kernels then move only the kept rows across the host link
 *    (NVLink-C2C on Grace systems) instead of a staging copy of whole
 *    layers.  Keys read by the tensor-core scoring kernel go through a TMA
 *    tensor map and must be device memory (cudaMalloc or a stream-ordered
 *    pool; cudaPointerGetAttributes type cudaMemoryTypeDevice); a host or
 *    managed pointer there is rejected with CHUNKKV_ERR_INVALID_ARG before
 *    anything is launched.
 *  - Every call is asynchronous on the given stream (0 = legacy default).
 *  - Arguments are checked on the host before anything is launched; a bad
 *    argument returns an error code and launches nothing.  A failed launch
 *    returns CHUNKKV_ERR_CUDA.  Conditions the GPU detects (a pipeline wait
 *    that ran out of time) are recorded in the workspace and reported by
 *    chunkkv_status_check.
 *  - Layouts (elements; the head dimension d is always contiguous):
 *      q_win        [B, w, Hq, d]  at q_win[b*q_stride_b + i*q_stride_w + hq*q_stride_h + e]
 *      k, v         [T_total, Hkv, d] at x[t*kv_stride_t + h*kv_stride_h + e], sequence b
 *                   owning rows cu_seqlens[b] .. cu_seqlens[b+1]-1 (varlen, ragged)
 *      chunk_scores [B, Hkv, C_max] fp32, chunk i of sequence b at [b][h][i], i < C_b
 *      indices      [B, Hkv, n_cap_max] int32, positions local to the sequence
 *      counts       [B, Hkv] int32
 *      k_out, v_out [B, Hkv, n_cap_max, d] in the input dtype
 *    Rows at or beyond counts[b][h] of indices / k_out / v_out, and chunk
 *    scores at or beyond C_b, are left unwritten.
 *  - Alignment: q_win, k, v, k_out and v_out start on 16-byte boundaries, and
 *    kv_stride_t, kv_stride_h, q_stride_* and d are multiples of 16 bytes.
 */
#ifndef CHUNKKV_H_
#define CHUNKKV_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* chunkkv_stream_t;   /* the same type as cudaStream_t */

typedef enum chunkkv_status {
  CHUNKKV_OK = 0,
  CHUNKKV_ERR_INVALID_ARG = 1,         /* a size, pointer, stride or alignment is invalid   */
  CHUNKKV_ERR_UNSUPPORTED = 2,         /* valid, but outside what this build implements    */
  CHUNKKV_ERR_WORKSPACE_TOO_SMALL = 3, /* ws_bytes < chunkkv_workspace_size(...)            */
  CHUNKKV_ERR_CUDA = 4,                /* a CUDA runtime call or kernel launch failed        */
  CHUNKKV_ERR_TIMEOUT = 5              /* a device-side wait gave up (chunkkv_status_check) */
} chunkkv_status;

typedef enum chunkkv_dtype { CHUNKKV_F32 = 0, CHUNKKV_BF16 = 1 } chunkkv_dtype;

/* Largest batch one call accepts (the sequence table travels as a launch argument). */
#define CHUNKKV_MAX_BATCH 1024
/* Largest number of layers one chunkkv_gather call moves. */
#define CHUNKKV_MAX_GATHER_LAYERS 64

typedef struct chunkkv_params {
  int32_t B;        /* sequences, 0 <= B <= CHUNKKV_MAX_BATCH                                  */
  int32_t Hq;       /* query heads; Hq % Hkv == 0                                               */
  int32_t Hkv;      /* key/value heads, >= 1                                                    */
  int32_t d;        /* head dimension, 1..256                                                   */
  int32_t w;        /* observation window = number of window queries = recent tokens kept, >= 0 */
  int32_t c;        /* chunk size, >= 1                                                         */
  int32_t L_max;    /* compressed budget; k = min(L_max / c, C_b) chunks per (b, head), >= 0     */
  int32_t dtype;    /* chunkkv_dtype of q_win, k, v, k_out, v_out                                */
  const int32_t* cu_seqlens;  /* HOST array [B+1]: cu[0] = 0, non-decreasing; T_b = cu[b+1]-cu[b] */
  int64_t q_stride_b, q_stride_w, q_stride_h;   /* element strides of q_win                     */
  int64_t kv_stride_t, kv_stride_h;             /* element strides of k and v (and their layers) */
  int32_t causal_window;  /* 0: every window query sees all T_b keys (the algorithm as printed);
                             1: window query q (0 <= q < w) sits at position T_b - w + q and sees
                             keys 0 .. T_b - w + q only (a query at a negative position adds nothing) */
} chunkkv_params;

/*
 * Output capacities: n_cap_max = max_b min(T_b, k_b*c + min(w, T_b)) is the row
 * capacity per (b, head) of indices/k_out/v_out; C_max = max_b ceil(T_b / c) is
 * the chunk capacity of chunk_scores.  Either output pointer may be NULL.
 */
chunkkv_status chunkkv_out_capacity(const chunkkv_params* p, int32_t* n_cap_max, int32_t* C_max);

/*
 * Bytes of device workspace chunkkv_score / chunkkv_compress_layers need for
 * these shapes (n_layers, n_reuse as passed to chunkkv_compress_layers; use
 * 1, 1 for chunkkv_score).  The workspace must be zero-filled before its first
 * use (cudaMemset / torch.zeros); afterwards the library keeps it consistent.
 * Its first 256 bytes hold the device error word (chunkkv_status_check) and the
 * counter from which the CTAs of a tensor-core scoring launch claim their work
 * items; the launch leaves the counter at zero when it ends.
 * One workspace must not be used by two calls that can run at the same time.
 */
chunkkv_status chunkkv_workspace_size(const chunkkv_params* p, int32_t n_layers, int32_t n_reuse,
                                      size_t* bytes);

/*
 * Window scores per chunk for one layer (ChunkKV §4.1 Algorithm 1 steps 1-3,
 * with the probabilities of Kara §2 Eq. (1)):
 *   A[b][h][i] = sum over g < G, q < w, j in chunk i of softmax_j(Q_w[b,q,h*G+g,:] . K[b,j,h,:] / sqrt(d))
 * q_win: addressable (on the tensor-core path device Q_w is read through a
 * tensor map when w divides 128, host Q_w is first packed with plain loads);
 * k: device when chunkkv_score_path(p) is 1 (tensor cores), else addressable;
 * layouts above.  chunk_scores: device, written for
 * i < C_b.  ws: device workspace of ws_bytes >= chunkkv_workspace_size(p, 1, 1).
 */
chunkkv_status chunkkv_score(const chunkkv_params* p, const void* q_win, const void* k,
                             float* chunk_scores, void* ws, size_t ws_bytes, chunkkv_stream_t stream);

/*
 * Top-k chunk selection and kept-index construction (ChunkKV §4.1 Algorithm 1
 * steps 4-6): for each (b, h) keep the k_b = min(L_max / c, C_b) chunks of
 * largest chunk_scores (ties to the lower chunk index; -0.0 equals +0.0; the
 * scores must not be NaN), and write the ascending union of their tokens and
 * of the last w tokens to indices[b][h][0 .. counts[b][h]).
 * chunk_scores: device [B, Hkv, C_max]; indices, counts: device outputs.
 */
chunkkv_status chunkkv_select(const chunkkv_params* p, const float* chunk_scores, int32_t* indices,
                              int32_t* counts, chunkkv_stream_t stream);

/*
 * index_select of K and V by a kept-index list (ChunkKV §4.1 Algorithm 1 step
 * 6), for n_layers layers that share one list (ChunkKV §4.2 Algorithm 2):
 *   k_out[l][b][h][r][:] = k[l][cu_seqlens[b] + indices[b][h][r]][h][:]  for r < counts[b][h]
 * and the same for v.  k, v, k_out, v_out: HOST arrays of n_layers
 * addressable pointers (1 <= n_layers <= CHUNKKV_MAX_GATHER_LAYERS); indices,
 * counts: device.
 * Indices must lie in [0, T_b); the copy is bit-exact.
 */
chunkkv_status chunkkv_gather(const chunkkv_params* p, int32_t n_layers, const int32_t* indices,
                              const int32_t* counts, const void* const* k, const void* const* v,
                              void* const* k_out, void* const* v_out, chunkkv_stream_t stream);

/*
 * The whole path over n_layers layers (ChunkKV §4.2 Algorithm 2 around §4.1
 * Algorithm 1): layers with l % n_reuse == 0 run score + select into index
 * group g = l / n_reuse; every layer l gathers its own K, V with group
 * l / n_reuse.
 *   q_win: HOST array of n_layers addressable pointers (entries of layers
 *          with l % n_reuse != 0 are not read and may be NULL; as for
 *          chunkkv_score, host Q_w costs one packing launch);
 *   k, v, k_out, v_out: HOST arrays of n_layers addressable pointers, except
 *          that k[l] of a scoring layer (l % n_reuse == 0) is device memory
 *          when chunkkv_score_path(p) is 1;
 *   indices: device [ceil(n_layers / n_reuse), B, Hkv, n_cap_max];
 *   counts:  device [ceil(n_layers / n_reuse), B, Hkv];
 *   chunk_scores: NULL, or device [ceil(n_layers / n_reuse), B, Hkv, C_max];
 *   ws: device workspace of ws_bytes >= chunkkv_workspace_size(p, n_layers, n_reuse).
 */
chunkkv_status chunkkv_compress_layers(const chunkkv_params* p, int32_t n_layers, int32_t n_reuse,
                                       const void* const* q_win, const void* const* k,
                                       const void* const* v, void* const* k_out, void* const* v_out,
                                       int32_t* indices, int32_t* counts, float* chunk_scores,
                                       void* ws, size_t ws_bytes, chunkkv_stream_t stream);

/*
 * Incremental compression during decoding (the notes keep the compressed cache
 * through decoding, ChunkKV §5.6; Kara §2 Eqs. (2)-(3) compress again once the
 * cache reaches its threshold), over n_layers layers with the index reuse of
 * ChunkKV §4.2 Algorithm 2.  Sequence b of p is the current cache of one
 * sequence: its first n_prev[b] positions were kept by earlier passes, the
 * rest are the n_new = T_b - n_prev[b] tokens decoded since.  A scoring layer
 * (l % n_reuse == 0) re-scores the new tail only (ChunkKV §4.1 Algorithm 1 on
 * the tail), with every window row normalised over all T_b keys of the cache:
 *   A[g][b][h][i] = sum over g', q and tail tokens j in chunk i of softmax over all T_b keys,
 * chunk i being tail tokens [i*c, min(i*c + c, n_new)); it keeps the
 * min(L_max / c, ceil(n_new / c)) best tail chunks (ties to the lower index)
 * plus the last w tail tokens into index group g = l / n_reuse, and every
 * layer l gathers its own rows with group l / n_reuse:
 *   indices[g][b][h][r]: ascending TAIL positions (0 = the first token after
 *                        the kept prefix), r < counts[g][b][h];
 *   k_out[l][b][h][r][:] = k[l][cu_seqlens[b] + n_prev[b] + indices[l / n_reuse][b][h][r]][h][:],
 *                        same for v,
 * which the caller appends after the n_prev[b] rows it keeps.  L_max is the
 * budget for the tail of this pass; n_prev is the same for every layer (the
 * layers' caches grow together).  The prefix positions are never selected or
 * moved.  Caches of different KV heads usually differ in length after a pass:
 * pass each head's cache as a sequence of its own (Hkv = 1, its G query heads)
 * when they do.
 *   n_prev: HOST [B], 0 <= n_prev[b] <= T_b;
 *   q_win, k, v, k_out, v_out: HOST arrays of n_layers pointers as for
 *          chunkkv_compress_layers; k_out[l], v_out[l] [B, Hkv, n_cap_max, d] with
 *          n_cap_max from chunkkv_tail_sizes;
 *   indices: device [ceil(n_layers / n_reuse), B, Hkv, n_cap_max];
 *   counts:  device [ceil(n_layers / n_reuse), B, Hkv];
 *   chunk_scores: NULL, or device [ceil(n_layers / n_reuse), B, Hkv, C_max] (tail
 *          chunks; entries >= C_b unspecified);
 *   ws: device workspace of ws_bytes >= chunkkv_tail_sizes' ws_bytes for the same
 *       n_layers and n_reuse (zero-filled before its first use, like
 *       chunkkv_workspace_size's).
 * B may be at most CHUNKKV_MAX_BATCH / 2 (the prefix and the tail of each cache
 * are scored as two sequences); causal_window must be 0 (CHUNKKV_ERR_UNSUPPORTED).
 */
chunkkv_status chunkkv_tail_sizes(const chunkkv_params* p, const int32_t* n_prev, int32_t n_layers, int32_t n_reuse,
                                  int32_t* n_cap_max, int32_t* C_max, size_t* ws_bytes);
chunkkv_status chunkkv_compress_tail(const chunkkv_params* p, const int32_t* n_prev, int32_t n_layers, int32_t n_reuse,
                                     const void* const* q_win, const void* const* k, const void* const* v,
                                     void* const* k_out, void* const* v_out, int32_t* indices, int32_t* counts,
                                     float* chunk_scores, void* ws, size_t ws_bytes, chunkkv_stream_t stream);

/*
 * Window scores for callers that cannot allocate device memory.  The ChunkKV
 * notes have no counterpart for this call; it exists for code that must not
 * call cudaMalloc when it scores (code running inside a memory pool or arena
 * that owns all device memory, allocator callbacks, runtimes with a memory
 * budget fixed at start-up) and has no workspace to lend.
 * It computes exactly what chunkkv_score computes, with the portable scoring
 * kernel, and takes no workspace: its scratch is one device array of
 * CHUNKKV_NOALLOC_SCRATCH_BYTES inside the library, which every GPU that loads
 * the library holds until the process exits.  It allocates nothing.
 *  - Shapes whose scratch would exceed that array return
 *    CHUNKKV_ERR_WORKSPACE_TOO_SMALL before anything is launched (about
 *    4 * w * G * Hkv * sum_b T_b / c bytes are needed; e.g. T = 32768 tokens with
 *    w*G = 128 rows and 8 KV heads fits).
 *  - All calls share the array and it keeps the last call's contents; a call
 *    reads only what it wrote itself, so nothing has to be cleared.  Calls whose
 *    kernels can overlap on the GPU (other streams, other threads) race on it.
 *  - The first call on each device looks up the array's device address with
 *    that device current; make it before any stream capture begins.
 */
#define CHUNKKV_NOALLOC_SCRATCH_BYTES (16u << 20)
chunkkv_status chunkkv_score_noalloc(const chunkkv_params* p, const void* q_win, const void* k,
                                     float* chunk_scores, chunkkv_stream_t stream);

/*
 * Synchronises the stream, then reads and clears the device-side error word of
 * the workspace.  Returns CHUNKKV_ERR_TIMEOUT if a kernel gave up waiting since
 * the last check (device_code, if not NULL, receives the raw code: the site
 * that gave up), CHUNKKV_ERR_CUDA if the stream reported an error, else CHUNKKV_OK.
 */
chunkkv_status chunkkv_status_check(void* ws, chunkkv_stream_t stream, int32_t* device_code);

/*
 * Adjacent-layer overlap of kept index lists: the Jaccard similarity of
 * consecutive layers' selections that ChunkKV §4.2 reports as the observation
 * behind Algorithm 2 (layer-wise index reuse), as exact counts.  Run on lists
 * scored independently per layer (chunkkv_compress_layers with n_reuse = 1) it
 * measures how much a reuse depth N_reuse would change the kept tokens.
 *   indices: device [n_lists, B, Hkv, n_cap_max] int32, each list ascending and
 *            duplicate-free in [0, T_b) for its first counts[...] entries
 *            (the layout chunkkv_compress_layers writes);
 *   counts:  device [n_lists, B, Hkv] int32;
 *   inter, uni: device [n_lists - 1, B, Hkv] int32, written with
 *            |I_l ∩ I_{l+1}| and |I_l ∪ I_{l+1}| for l = 0 .. n_lists - 2
 *            (Jaccard = inter / uni; two empty lists give 0 / 0).
 * Positions outside [0, T_b) are ignored.  n_lists == 1 or an empty batch
 * writes nothing.  Returns CHUNKKV_ERR_UNSUPPORTED when a sequence is longer
 * than the kernel's shared-memory bitmap holds (about 1.86 M tokens).
 */
chunkkv_status chunkkv_layer_overlap(const chunkkv_params* p, int32_t n_lists, const int32_t* indices,
                                     const int32_t* counts, int32_t* inter, int32_t* uni, chunkkv_stream_t stream);

/*
 * Self test of the failure path (a test aid; no counterpart in the pages).
 * Launches one thread that first starts an asynchronous bulk copy of ws bytes
 * 128..191 into shared memory, then waits, through the same bounded wait as the
 * tensor-core scoring kernel, on a barrier that nothing completes.  The wait
 * gives up after about a millisecond and records device code 0x1FF in the error
 * word of ws; the thread then drains its copy as the scoring kernel's teardown
 * does after a give-up (a bounded wait on the copy's own barrier phase, never a
 * fixed pause) and writes the 64 bytes that landed to ws bytes 64..127.  The
 * kernel returns and leaves the context usable; a following
 * chunkkv_status_check(ws, ...) returns CHUNKKV_ERR_TIMEOUT with that code.
 *   ws: device workspace of at least 256 bytes (bytes 0..3 and 64..127 are written).
 * Returns CHUNKKV_ERR_INVALID_ARG for a NULL, misaligned or too small ws.
 */
chunkkv_status chunkkv_selftest_wait_timeout(void* ws, size_t ws_bytes, chunkkv_stream_t stream);

/*
 * Throughput probe of the exponential unit (a measurement aid; no counterpart in
 * the pages).  The scoring kernels evaluate one base-2 exponential
 * (ex2.approx.ftz.f32) per window logit; this call launches `blocks` CTAs of
 * CHUNKKV_PROBE_THREADS threads, each thread evaluating `iters` rounds of
 * CHUNKKV_PROBE_CHAINS independent exponentials of that instruction, i.e.
 * blocks * CHUNKKV_PROBE_THREADS * CHUNKKV_PROBE_CHAINS * iters of them in all.
 * Timing the call (events on `stream`) gives the exponential rate that bounds
 * the scoring phase.
 *   sink: device, blocks * CHUNKKV_PROBE_THREADS floats (one result per thread).
 * Returns CHUNKKV_ERR_INVALID_ARG for a NULL sink or a non-positive count.
 */
#define CHUNKKV_PROBE_THREADS 256
#define CHUNKKV_PROBE_CHAINS 16
chunkkv_status chunkkv_probe_ex2(float* sink, int32_t blocks, int32_t iters, chunkkv_stream_t stream);

/* ------------------------------------------------------------------------
 * Serving around the compression: attention over the prompt before it, and the
 * compressed cache held in 8 bits after it (ChunkKV §5.6 keeps the compressed
 * cache through decoding).
 * ------------------------------------------------------------------------ */

/*
 * Causal attention over packed prompts with grouped heads:
 *   out[i][hq] = sum over j <= i + Tk - Tq of softmax_j(scale * q[i][hq] . k[j][hq / G]) * v[j][hq / G]
 * per sequence (i, j local to it): the last query sits at the last key, so Tq < Tk
 * continues a sequence whose first Tk - Tq keys are cached, and Tq > Tk leaves the
 * first Tq - Tk queries without a key; their rows are zeros (logits that are all
 * -inf give NaN, as the formula does).  A key that a query
 * does not see adds nothing to it, whatever k and v hold there (infinities and NaN
 * included).
 *   q, out [Tq_total, Hq, d], k, v [Tk_total, Hkv, d]: device memory, dtype's type
 *   (q, k, v and out start on 16-byte boundaries; every stride is a multiple of 16
 *   bytes; d is contiguous).  out may not overlap an input.
 * Sums and softmax statistics are fp32.  For bf16 the products run on the tensor
 * cores when chunkkv_prefill_path says 1 (probabilities are then rounded to bf16
 * before they weigh the values), else, and for fp32, in fp32 throughout.
 */
typedef struct chunkkv_prefill_params {
  int32_t B, Hq, Hkv, d;      /* as in chunkkv_params                                       */
  int32_t dtype;              /* chunkkv_dtype                                               */
  float scale;                /* > 0 and finite; usually 1 / sqrt(d)                         */
  const int32_t* cu_q;        /* HOST [B + 1], as chunkkv_params.cu_seqlens, of the queries  */
  const int32_t* cu_k;        /* HOST [B + 1], of the keys                                   */
  int64_t q_stride_t, q_stride_h;     /* element strides of q                               */
  int64_t kv_stride_t, kv_stride_h;   /* element strides of k and of v                      */
  int64_t o_stride_t, o_stride_h;     /* element strides of out                             */
} chunkkv_prefill_params;

/* Bytes of device workspace (zero-filled before its first use, like chunkkv_workspace_size's; its first
 * word is read by chunkkv_status_check).  One workspace must not serve two calls that can overlap. */
chunkkv_status chunkkv_prefill_workspace_size(const chunkkv_prefill_params* p, size_t* bytes);
/* Which kernel these shapes take: 0 = fp32 arithmetic, 1 = tensor cores, -1 = invalid parameters. */
int32_t chunkkv_prefill_path(const chunkkv_prefill_params* p);
chunkkv_status chunkkv_prefill_attention(const chunkkv_prefill_params* p, const void* q, const void* k, const void* v,
                                         void* out, void* ws, size_t ws_bytes, chunkkv_stream_t stream);

/*
 * The compressed cache in 8 bits.  A cache row r = b * Hkv + h is one (sequence, KV
 * head): chunk compression keeps another number of tokens for every head, so each
 * has a length, pages and scales of its own.  A page holds CHUNKKV_Q8_PAGE tokens of
 * one row as int8 codes with one fp32 scale for its keys and one for its values
 * (value = code * scale).  d64 is d rounded up to a multiple of 64.
 *   k_pages [n_pages][d64 / 64][CHUNKKV_Q8_PAGE][64], v_pages [n_pages][d64][CHUNKKV_Q8_PAGE]
 *           int8, device, 16-byte aligned, zero-filled before their first use;
 *   scales  [n_pages][2] fp32, device (keys, values), zero-filled before its first use;
 *   table   [B * Hkv][max_pages] int32, device: the page of tokens 64 j .. 64 j + 63;
 *   lens    [B * Hkv] int32, device: tokens held;
 *   ring    [n_pages] int32, device: the free pages, state[1] of them from position
 *           state[0] on, cyclically; at first a permutation of 0 .. n_pages - 1;
 *   state   [4] int32, device: head, number free, status of the last resize, 0.
 * table, lens, ring and state belong to one set of lengths; layers whose lengths
 * agree (one reuse group of ChunkKV §4.2) share them, each layer with its own
 * k_pages, v_pages and scales.  Calls that use one cache are ordered by their stream.
 */
#define CHUNKKV_Q8_PAGE 64
/* Largest number of cache rows (B * Hkv). */
#define CHUNKKV_Q8_MAX_ROWS 65535
typedef struct chunkkv_q8_cache {
  int32_t B, Hkv, d;
  int32_t n_pages, max_pages;
  int8_t* k_pages;
  int8_t* v_pages;
  float* scales;
  int32_t* table;
  int32_t* lens;
  int32_t* ring;
  int32_t* state;
} chunkkv_q8_cache;

/*
 * Block tables and slot maps on the GPU: sets every row's length to new_lens[r]
 * (device [B * Hkv] int32).  Rows that need more pages take them from the ring's
 * head, in row order; pages that a shorter row no longer needs go behind the ring's
 * free part, in row order, and their table entries become -1.  slots (NULL, or
 * device [B * Hkv][n_cap] int64) receives the slots page * CHUNKKV_Q8_PAGE + offset of
 * tokens lens[r] .. new_lens[r] - 1 and -1 beyond them.
 * All or nothing: state[2] is 0 when it was done; 1 when the ring has too few pages
 * and 2 when a length is negative, needs more than max_pages pages, or (with slots)
 * grows by more than n_cap: then nothing but state[2] and slots (all -1) is written.
 * Reads and writes table, lens, ring and state only (k_pages, v_pages and scales
 * may be NULL).
 */
chunkkv_status chunkkv_q8_resize(const chunkkv_q8_cache* c, const int32_t* new_lens, int64_t* slots, int32_t n_cap,
                                 chunkkv_stream_t stream);

/*
 * Writes new rows into one layer's pages: for r = b * Hkv + h the first
 * counts[b][h] (device int32) of the n_cap tokens k[b][h][i][:], v[b][h][i][:] (device,
 * element strides st_b, st_h, st_t; d contiguous) go to slots[r][i], as
 * chunkkv_q8_resize wrote them for these rows.  A page's scale becomes
 *   s = max(s_old, m / 127)    m: largest magnitude among its new tokens (zero if below 2^-100)
 * (s_old = 0 if the new tokens begin the page), its older codes round(code * (s_old / s))
 * if it grew, and the new codes round(x * (1 / s)), ties to even, in fp32.  A NaN or an
 * infinity makes the scale of its page NaN or infinite: the page then reads as NaN.
 */
chunkkv_status chunkkv_q8_append(const chunkkv_q8_cache* c, int32_t dtype, const void* k, const void* v, int64_t st_b,
                                 int64_t st_h, int64_t st_t, const int32_t* counts, const int64_t* slots,
                                 int32_t n_cap, chunkkv_stream_t stream);

/*
 * Reads rows back: token i < min(lens[r], n_cap) of row r goes to k_out and
 * v_out[(start[r] + i) * st_t + e] (device, dtype's type; start: device [B * Hkv]
 * int64, a negative entry skips the row), e.g. as the packed keys of a further
 * chunkkv_compress_layers or chunkkv_compress_tail call.  Where they end is in device
 * memory: chunkkv_q8_load trusts start, chunkkv_q8_load_bounded writes none of the rows
 * at or past n_rows of k_out and v_out.
 */
chunkkv_status chunkkv_q8_load(const chunkkv_q8_cache* c, int32_t dtype, const int64_t* start, int32_t n_cap,
                               void* k_out, void* v_out, int64_t st_t, chunkkv_stream_t stream);
chunkkv_status chunkkv_q8_load_bounded(const chunkkv_q8_cache* c, int32_t dtype, const int64_t* start, int32_t n_cap,
                                       int64_t n_rows, void* k_out, void* v_out, int64_t st_t,
                                       chunkkv_stream_t stream);

/*
 * Single-token attention over one layer's cache, G query heads per KV head:
 *   out[b][h * G + g] = sum_j softmax_j(scale * q[b][h * G + g] . K_j) V_j
 * over the lens[r] tokens of row r = b * Hkv + h; an empty row gives zeros.
 *   q, out: device [B, Hkv * G, d] with element strides (b, head), multiples of 16 bytes;
 *   scale > 0 and finite; sums and softmax statistics in fp32;
 *   ws: device workspace of chunkkv_q8_workspace_size bytes, zero-filled before its
 *       first use; not shared by calls that can overlap.  One workspace may serve
 *       caches and G of any kind and chunkkv_prefill_attention in turn; while G <= 8, the
 *       compression's calls too (for G > 8 they would write over counts that have to be
 *       zero).
 */
chunkkv_status chunkkv_q8_workspace_size(const chunkkv_q8_cache* c, int32_t G, size_t* bytes);
chunkkv_status chunkkv_q8_attention(const chunkkv_q8_cache* c, int32_t dtype, int32_t G, float scale, const void* q,
                                    int64_t q_stride_b, int64_t q_stride_h, void* out, int64_t o_stride_b,
                                    int64_t o_stride_h, void* ws, size_t ws_bytes, chunkkv_stream_t stream);

/*
 * The compressed cache in 4 bits: rows, tables, lengths and the ring as in
 * chunkkv_q8_cache, with one pool of pages a layer.  Every token's groups of 64
 * columns (ND = ceil(d / 64) of them, the last one maybe shorter) are quantised by
 * themselves, in fp32: for a group whose values lie in [lo, hi]
 *   m = lo rounded down to bf16
 *   s = (hi - m) * (1 / 15) rounded up to bf16; 0 if hi - m is below 2^-100
 *       (lowered to the next bf16, twice at most, while 15 s + m is infinite in fp32, or in
 *       bf16 where hi is finite in bf16: then 15 s may be below hi - m, by 2 % at most)
 *   c = round((x - m) * (1 / s)) in 0 .. 15, ties to even; 0 where s is 0
 * and a code stands for s * c + m, within half a step of x.  A group with a NaN or an infinity, or
 * whose m or hi - m is infinite (values below bf16's lowest, or further apart than fp32 can say),
 * has m = NaN and s = 0: it reads as NaN.
 * A page holds CHUNKKV_Q8_PAGE (64) tokens of one row in CHUNKKV_Q4_PAGE_BYTES(d) bytes:
 *   keys            [64 tokens][4][ND][8 bytes]     bytes (t, g) of a token: columns 64 g + 16 t .. + 15
 *   their (m, s)    [ND][64 tokens][2] bf16
 *   values          [4 ND][8][4][2][8 bytes]        bytes (p, c, t, h): tokens 16 t .. + 15 of column 16 p + 8 h + c
 *   their (m, s)    [ND][64 tokens][2] bf16
 * Of 16 codes in 8 bytes, code 8 w + 2 p + e (w, e: 0 .. 1, p: 0 .. 3) is nibble p + 4 e of the
 * w-th 32-bit word (little endian, nibble 0 the lowest).
 *   pages   [n_pages][CHUNKKV_Q4_PAGE_BYTES(d)], device, 16-byte aligned
 * d is a multiple of 8, at most 256.
 */
#define CHUNKKV_Q4_PAGE_BYTES(d) (4608 * (((d) + 63) / 64))
typedef struct chunkkv_q4_cache {
  int32_t B, Hkv, d;
  int32_t n_pages, max_pages;
  uint8_t* pages;
  int32_t* table;
  int32_t* lens;
  int32_t* ring;
  int32_t* state;
} chunkkv_q4_cache;

/* chunkkv_q8_resize for a 4-bit cache (pages may be NULL). */
chunkkv_status chunkkv_q4_resize(const chunkkv_q4_cache* c, const int32_t* new_lens, int64_t* slots, int32_t n_cap,
                                 chunkkv_stream_t stream);

/*
 * Writes new rows into one layer's pages; arguments as chunkkv_q8_append's.  A token is
 * final when it is written: no other token's codes change.
 */
chunkkv_status chunkkv_q4_append(const chunkkv_q4_cache* c, int32_t dtype, const void* k, const void* v, int64_t st_b,
                                 int64_t st_h, int64_t st_t, const int32_t* counts, const int64_t* slots,
                                 int32_t n_cap, chunkkv_stream_t stream);

/* Reads rows back, s * c + m rounded once to dtype's type; arguments as chunkkv_q8_load_bounded's. */
chunkkv_status chunkkv_q4_load(const chunkkv_q4_cache* c, int32_t dtype, const int64_t* start, int32_t n_cap,
                               int64_t n_rows, void* k_out, void* v_out, int64_t st_t, chunkkv_stream_t stream);

/*
 * Attention of n_q >= 1 query tokens a sequence over one layer's cache, G query heads per
 * KV head.  The m = q_lens[b] query tokens of sequence b (q_lens: device [B] int32, values
 * outside 0 .. n_q are taken as the nearer of the two; NULL: n_q each) are the last m of
 * every row's tokens, whose keys and values the cache holds already:
 *   out[b][i][h * G + g] = sum_j softmax_j(scale * q[b][i][h * G + g] . K_j) V_j
 * over the tokens j < lens[r] - m + 1 + i of row r = b * Hkv + h, for i < m: with n_q = 1 the
 * single-token attention over all of a row.  A query that sees no token gives zeros; logits
 * that are all -inf give NaN.  What a query does not see adds nothing, whatever it holds.
 * out[b][i] of i >= m is not written.
 *   q, out: device [B, n_q, Hkv * G, d] with element strides (b, token, head), multiples of
 *   16 bytes; out overlaps no input;
 *   scale > 0 and finite, scale * |q| below 2^116;
 *   sums and softmax statistics in fp32 (a row's tokens times its largest value must stay within it).
 *   For bf16 the weights are rounded to f16 (2^-11 each) before they weigh the values, as
 *   multiples of the row's largest product of a weight and its token's step (many query rows: its
 *   token's largest value): what lies below 2^-18 of it loses bits, below 2^-29 it is lost.
 *   q . c is good to about 2^-17 of its largest term.  With many query rows (chunkkv_q4_path 1)
 *   keys and values are rounded to f16 too, as multiples of the largest of their token, or of 2^-100
 *   (keys) and 2^-60 (values) if that is less: what lies below 2^-20 of it loses bits, below 2^-31
 *   it is lost (tokens whose largest are within 2^8 of each other may share one multiple);
 *   ws: device workspace of chunkkv_q4_workspace_size bytes, under chunkkv_q8_attention's
 *   terms: zero-filled before its first use, not shared by calls that can overlap; it may
 *   serve any of the attention calls in turn.
 */
chunkkv_status chunkkv_q4_workspace_size(const chunkkv_q4_cache* c, int32_t dtype, int32_t G, int32_t n_q, size_t* bytes);
/*
 * Which kernel such a call takes: 0 = one for few query rows, 1 = one for many, -1 = invalid
 * arguments.  A call that gets 1 takes 0 all the same where no tensor map can address q (an axis of
 * more than one element with a stride of 0, or q outside device memory) or where out's token or
 * head stride is 2^22 elements or more.
 */
int32_t chunkkv_q4_path(const chunkkv_q4_cache* c, int32_t dtype, int32_t G, int32_t n_q);
chunkkv_status chunkkv_q4_attention(const chunkkv_q4_cache* c, int32_t dtype, int32_t G, int32_t n_q,
                                    const int32_t* q_lens, float scale, const void* q, int64_t q_stride_b,
                                    int64_t q_stride_t, int64_t q_stride_h, void* out, int64_t o_stride_b,
                                    int64_t o_stride_t, int64_t o_stride_h, void* ws, size_t ws_bytes,
                                    chunkkv_stream_t stream);

/* Static description of a status code. */
const char* chunkkv_status_string(chunkkv_status s);

/* Which scoring kernel chunkkv_score would use for these shapes: 0 = SIMT, 1 = tensor-core. */
int32_t chunkkv_score_path(const chunkkv_params* p);

/*
 * Number of CUDA kernels this process has launched through the library so far
 * (every entry point, every device and host thread; a relaxed atomic counter
 * that only grows).  The difference of two readings around a region counts the
 * library's kernel launches in it.  Never fails.
 */
uint64_t chunkkv_launch_count(void);

/*
 * Phase timing of chunkkv_compress_layers and chunkkv_compress_tail (a
 * measurement aid).
 *   events: HOST array of CHUNKKV_PHASE_EVENTS cudaEvent_t handles (as void*)
 *           that the caller created and keeps alive; NULL with n_events = 0
 *           switches recording off.
 * While set, each chunkkv_compress_layers or chunkkv_compress_tail call made
 * by the same host thread records events[i] on its stream at phase boundary i:
 * 0 before the window-row packing (a phase without a launch when the scoring
 * kernel reads the window rows from q_win itself: w divides 128), 1 before
 * scoring, 2 before the log-sum-exp, 3 before the finalisation (for token-level
 * chunks in two passes: the second pass and the sum of its partial arrays), 4
 * before the top-k selection, 5 before the gather, 6 after the gather.  When
 * one kernel takes the log-sum-exp, the finalisation and the selection (calls
 * with enough (group, sequence, head) triples to fill the GPU), boundaries 2
 * and 3 come before it and 4 after it, so its time shows as the
 * finalisation's.  A record between two launches ends the
 * programmatic-dependent-launch overlap there, so recorded calls run a little
 * slower than unrecorded ones.
 * Returns CHUNKKV_ERR_INVALID_ARG if n_events is neither 0 nor
 * CHUNKKV_PHASE_EVENTS or a handle is NULL (the previous setting then stays).
 */
#define CHUNKKV_PHASE_EVENTS 7
chunkkv_status chunkkv_set_phase_events(void* const* events, int32_t n_events);

#ifdef __cplusplus
}
#endif

#endif /* CHUNKKV_H_ */
