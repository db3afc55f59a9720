/*
 * nt.h -- C ABI of the batch-1 quantized Llama decode step for NVIDIA GB300 (sm_103a).
 *
 * What it computes.  The decode step of the layer-streaming Llama engine that
 * the "ntransformer" pages describe (de.news.hada.io, "Überblick über
 * NTransformer" and "Hauptfunktionen": GGUF-style Q4_0 / Q8_0 / Q4_K / Q6_K
 * weights; Llama with RoPE, GQA, SwiGLU, RMSNorm and a KV cache; section
 * "Architektur und Codestruktur": GEMV, RMSNorm, RoPE, SwiGLU and softmax
 * kernels; "3-stufiges adaptives Caching" and "SLEP-Streaming": VRAM-resident
 * layers plus pinned-RAM layers copied host-to-device with double buffering;
 * blog.hotdry.top, "gpu-nvme-direct的实现架构": two staging buffers whose copy
 * and compute overlap on CUDA streams).  The pages plan but never show a
 * public C API ("Phase 5 ... öffentliche C-API (geplant)"), so the entry
 * points below are this library's own.
 *
 * Conventions for every function:
 *  - Returns nt_status; NT_OK on success.  On failure the output parameters
 *    are left untouched and nt_last_error() returns a message (thread-local).
 *    No C++ exception crosses this boundary.
 *  - "dev" pointers are CUDA device pointers owned by the caller; "host"
 *    pointers are ordinary host memory owned by the caller.  Objects created
 *    by *_create are owned by the library until the matching *_destroy.
 *  - "stream" is a cudaStream_t passed as void*; NULL means the legacy
 *    default stream.  Functions that take a stream are asynchronous on it;
 *    the others synchronise before they return.
 *  - One model is used by one host thread at a time.
 */
#ifndef NT_H
#define NT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  NT_OK = 0,
  NT_E_INVAL = 1,        /* invalid argument: shape, token, position, pointer, size */
  NT_E_NOMEM = 2,        /* device or pinned-host allocation failed                 */
  NT_E_CUDA = 3,         /* a CUDA runtime call failed (message has the CUDA error)  */
  NT_E_TIMEOUT = 4,      /* the host watchdog gave up waiting for the device         */
  NT_E_UNSUPPORTED = 5,  /* valid request this build does not implement              */
  NT_E_STATE = 6         /* call not valid in the object's current state             */
} nt_status;

/* Weight formats ("Quantisierungsformate Q4_0, Q8_0, Q4_K_M, Q5_K, Q6_K, F16
 * und F32", hada "Überblick").  F16 and F32 weights are not implemented
 * (NT_E_UNSUPPORTED); F16 is used only for the KV cache.
 * Canonical block bytes (little-endian), the export format:
 *   Q8_0  32 weights, 34 B:  f16 d | int8 q[32]                  w = d*q
 *   Q4_0  32 weights, 18 B:  f16 d | u8 qs[16]                   w = d*(q-8)
 *         (element k in byte k/2, low nibble for even k)
 *   Q4_K  256 weights, 144 B: f16 d | f16 dmin | 12 B of sixteen 6-bit fields
 *         (sc_0..7 then m_0..7, least-significant bit first) | u8 qs[128]
 *                                                               w = d*sc_j*q - dmin*m_j
 *   Q6_K  256 weights, 210 B: u8 ql[128] (low 4 bits, as Q4_0) | u8 qh[64]
 *         (high 2 bits of element k in byte k/4 at bits 2*(k%4)) | int8 sc[16] | f16 d
 *                                                               w = d*sc_j*(q-32)
 *   Q5_K  256 weights, 176 B: f16 d | f16 dmin | 12 B of 6-bit fields as Q4_K |
 *         u8 qh[32] (fifth bit of element k in byte k/8 at bit k%8) | u8 qs[128]
 *         (low 4 bits, as Q4_0), q in 0..31              w = d*sc_j*q - dmin*m_j
 * On the device each tensor is held as separate 16-byte-aligned streams
 * (codes, scales) with the same byte count. */
typedef enum { NT_F32 = 0, NT_F16 = 1, NT_Q8_0 = 2, NT_Q4_0 = 3, NT_Q4_K = 4, NT_Q6_K = 5, NT_Q5_K = 6 } nt_qtype;

/* Tensor roles inside a layer, and the two model-level matrices. */
enum {
  NT_ROLE_Q = 0, NT_ROLE_K = 1, NT_ROLE_V = 2, NT_ROLE_O = 3,
  NT_ROLE_GATE = 4, NT_ROLE_UP = 5, NT_ROLE_DOWN = 6,
  NT_ROLE_EMBD = 16,    /* [vocab x hidden], layer argument ignored */
  NT_ROLE_OUTPUT = 17   /* [vocab x hidden], layer argument ignored */
};

typedef struct nt_model nt_model;
typedef struct nt_qtensor nt_qtensor;

/* Model description.  Llama architecture with untied embeddings and unit norm
 * gains.  Weights are drawn from N(0, init_std^2) by the counter-based
 * generator keyed by (seed, tensor uid, element index) and quantized on the
 * device into the per-role formats. */
typedef struct {
  int32_t n_layers, hidden, n_heads, n_kv_heads, head_dim, ffn_dim, vocab, max_ctx;
  float rms_eps;      /* RMSNorm epsilon, e.g. 1e-5                  */
  float rope_theta;   /* RoPE base, e.g. 500000                      */
  float init_std;     /* weight standard deviation, e.g. 0.02        */
  nt_qtype t_embd, t_q, t_k, t_v, t_o, t_gate, t_up, t_down, t_out;
  uint64_t seed;
} nt_config;

/* Counters of the last steps (nt_get_stats). */
typedef struct {
  int64_t steps;           /* decode steps since create or reset                     */
  int32_t pos;             /* current position (number of cached tokens)            */
  int32_t n_resident;      /* layers resident in device memory                      */
  double last_step_ms;     /* wall time of the last nt_decode_step, device events    */
  double h2d_bytes;        /* bytes copied host-to-device in the last step          */
  double h2d_ms;           /* summed duration of those copies (copy-stream events)  */
  double compute_ms;       /* summed duration of the layer computations             */
  double overlap;          /* (h2d_ms + compute_ms - last_step_ms) / min(...), in [0,1] */
  int64_t weight_bytes;    /* quantized weight bytes read per step                  */
  int64_t kv_bytes_per_pos;/* KV cache bytes read per cached position per step      */
  double verify_weight_bytes; /* layer weight bytes the verification pass of the last
                              nt_speculative_step read (each multi-token launch reads
                              its weights once)                                      */
  double h2d_layer_min_GBs;   /* slowest and fastest single layer copy of the last   */
  double h2d_layer_max_GBs;   /* step, GB/s (0 when no layer was copied)             */
  int32_t h2d_layer_min_idx;  /* the layer whose copy was slowest (-1: none)         */
} nt_stats;

/* Per-kernel-class device times of profiled steps (nt_profile_steps). */
enum { NT_KC_GEMV = 0, NT_KC_ATTN = 1, NT_KC_OTHER = 2, NT_KC_COUNT = 3 };
typedef struct {
  int64_t launches[NT_KC_COUNT];
  double ms[NT_KC_COUNT];          /* summed event-to-event time of the launches */
  double bytes[NT_KC_COUNT];       /* summed algorithmic bytes of the launches   */
  double step_ms;                  /* mean wall time of a profiled step          */
  int64_t kernel_launches;         /* kernels launched over the profiled steps   */
} nt_kernel_times;

/* Message of the last failure on this thread ("" if none).  Never NULL. */
const char* nt_last_error(void);

/* ------------------------------------------------------------------ model -- */

/* Allocates device memory for all weights, the f16 KV cache ([layer][K|V]
 * [kv_head][max_ctx][head_dim]) and the activations, then generates and
 * quantizes every weight on the device.  Position starts at 0.
 * NT_E_INVAL: non-positive sizes, n_heads not a multiple of n_kv_heads,
 * head_dim odd, a column count not a multiple of the role format's block,
 * unsupported format.  NT_E_NOMEM: device allocation failed, or the model's
 * device allocations would pass the byte cap in the environment variable
 * NT_DEVICE_BYTES_LIMIT (decimal bytes; unset: no cap), a host-side stand-in
 * for running out of device memory. */
nt_status nt_model_create(const nt_config* cfg, nt_model** out);
void nt_model_destroy(nt_model* m);

/* Sets the position to 0 (cache contents are kept but no longer attended). */
nt_status nt_kv_reset(nt_model* m);

/* Fills cache positions [0, n_ctx) of every layer with N(0,1) draws rounded to
 * f16 (element (t, kv_head, d) of layer l uses counter index
 * (t*n_kv_heads + kv_head)*head_dim + d), treated as already-rotated keys, and
 * sets the position to n_ctx.  NT_E_INVAL if n_ctx > max_ctx. */
nt_status nt_kv_prefill(nt_model* m, int32_t n_ctx, uint64_t seed);

/* One decode step at the current position p (the pages' per-token loop:
 * embedding, n_layers x [RMSNorm, Q/K/V GEMV, RoPE, KV append, GQA attention,
 * O GEMV + residual, RMSNorm, gate/up GEMV, SwiGLU, down GEMV + residual],
 * final RMSNorm, output GEMV, greedy argmax with ties to the lowest id).
 * token: input id in [0, vocab).  next_token (host, required): the argmax.
 * logits_host (nullable): vocab floats.  top2_margin (nullable): top-1 minus
 * top-2 logit.  Synchronous.  Position becomes p+1.
 * A resident model runs the step as a CUDA graph of per-kernel launches.
 * NT_E_INVAL: token out of range or p == max_ctx.  NT_E_TIMEOUT: the host
 * watchdog (NT_WATCHDOG_MS, default 120 s) expired before the step finished. */
nt_status nt_decode_step(nt_model* m, int32_t token, int32_t* next_token, float* logits_host,
                         float* top2_margin);

/* n_steps greedy steps that feed each argmax back as the next input on the
 * device, starting from token; asynchronous on stream (the model's own
 * stream waits for it).  The produced ids are kept on the device
 * (nt_get_tokens).  Layer-streamed models are not supported here (NT_E_STATE);
 * use nt_decode_step. */
nt_status nt_decode_run(nt_model* m, int32_t token, int32_t n_steps, void* stream);

/* Copies the ids produced at positions [t0, t0+n) into host_out (n int32). */
nt_status nt_get_tokens(nt_model* m, int32_t t0, int32_t n, int32_t* host_out);

/* Reads n f16 cache values of (layer, kv: 0=K 1=V, kv_head) at positions
 * [t0, t0+n), head_dim values each, into host_out (n*head_dim uint16). */
nt_status nt_kv_export(nt_model* m, int32_t layer, int32_t kv, int32_t kv_head, int32_t t0, int32_t n,
                       uint16_t* host_out);

/* Layer streaming ("3-stufiges adaptives Caching": VRAM-resident layers plus
 * pinned-RAM layers copied host-to-device; "SLEP-Streaming ... Double
 * Buffering").  Layers [n_resident, n_layers) move to page-locked host memory
 * and their device copies are freed.  Every later nt_decode_step copies each
 * of them into one of n_staging device buffers on a copy stream while the
 * previous layer computes.  n_staging must be 2.  Results are bitwise
 * identical to the resident model.  Calling it again with n_resident =
 * n_layers brings every layer back to the device. */
nt_status nt_stream_layers(nt_model* m, int32_t n_resident, int32_t n_staging);

/* Tier placement ("Tier A" VRAM-resident layers, the rest streamed from pinned
 * RAM): how many layers of a model with configuration cfg fit in budget_bytes of
 * device memory next to everything else the model keeps there -- the token
 * embedding and output tensors, the K/V cache for max_ctx positions, the
 * activations and partials, and two staging buffers of one layer each when any
 * layer streams.  All layers have the same size, so the resident ones are the
 * first n.  Pure host arithmetic on the configuration (no device work).
 * n_resident (required) receives n in [0, n_layers]; device_bytes (nullable)
 * the device bytes of that placement; layer_bytes (nullable) the bytes of one
 * layer.  NT_E_INVAL: invalid configuration or negative budget.
 * NT_E_NOMEM: not even the non-layer allocations fit (n_resident is set to 0). */
nt_status nt_plan_residency(const nt_config* cfg, int64_t budget_bytes, int32_t* n_resident, int64_t* device_bytes,
                            int64_t* layer_bytes);

/* nt_stream_layers with the placement nt_plan_residency gives for the device
 * memory this model could use now: the driver's free memory plus what the
 * model already holds, minus margin_bytes.  n_resident_out (nullable) receives
 * the placement. */
nt_status nt_auto_residency(nt_model* m, int64_t margin_bytes, int32_t* n_resident_out);

/* ---- layer skip (hada "Leistung und Caching-Struktur": layer skip by cosine similarity;
 * hotdry "性能数据与瓶颈分析": the similarity between layer outputs is
 * computed beforehand and layers at or above the threshold, 0.98 there, are
 * skipped at inference) ----
 *
 * nt_layer_similarity runs one decode step exactly like nt_decode_step (same
 * result, position advanced by one, every layer evaluated whatever the skip
 * mask) and also writes cos_out[l], l < n_layers: the cosine similarity
 * between the residual stream entering layer l and leaving it, accumulated in
 * fp64 from the fp32 activations.  cos_out is host memory owned by the caller;
 * next_token as in nt_decode_step.  Works for resident and streamed models. */
nt_status nt_layer_similarity(nt_model* m, int32_t token, int32_t* next_token, double* cos_out);

/* Sets the layers later steps skip: mask[l] != 0 (n_layers bytes of host
 * memory, copied) skips layer l -- its weights are neither read nor copied from
 * the host tier, its K/V row is not written, and the residual stream passes
 * through unchanged.  mask = NULL evaluates every layer again.  Applies to
 * nt_decode_step, nt_decode_run and nt_profile_steps. */
nt_status nt_set_layer_skip(nt_model* m, const uint8_t* mask);

/* Host arithmetic: mask_out[l] = 1 for every layer with cos[l] >= threshold;
 * when max_skip > 0 and more qualify, only the max_skip most similar ones
 * (ties: lower layer first).  n_skipped (nullable) receives the count.
 * NT_E_INVAL on NULL arrays or n_layers < 0. */
nt_status nt_plan_layer_skip(const double* cos, int32_t n_layers, double threshold, int32_t max_skip,
                             uint8_t* mask_out, int32_t* n_skipped);

/* ---- self-speculative decoding (hada "Hauptfunktionen": the
 * VRAM-resident layers serve as the draft model, no extra model) ----
 *
 * One cycle from the current position p with input token `token`:
 *   draft   k greedy steps (1 <= k <= 8) of the model restricted to layers
 *           [0, n_draft) and the output head: d_1..d_k;
 *   verify  layers [n_draft, n_layers) and the head for token, d_1..d_{k-1} at
 *           positions p..p+k-1, layer by layer, so a host-tier layer is copied
 *           once per cycle rather than once per token; y_i is the full model's
 *           greedy token after position p+i;
 *   accept  j = the longest prefix with y_i == d_{i+1}; the emitted tokens are
 *           d_1..d_j, then y_j when j < k.
 * The emitted tokens are those nt_decode_step would produce from the same state,
 * bit for bit (every token gets the same arithmetic on the same inputs; layers
 * below n_draft are not recomputed, their K/V rows from the draft are the full
 * model's).  The verification runs each layer's GEMVs for several tokens per
 * launch (as nt_gemv_q_batch), so a resident layer's weights are read fewer than
 * k times; nt_stats.verify_weight_bytes reports the bytes read.  For a model
 * with every layer resident the cycle's device work is captured once as a CUDA
 * graph per (n_draft, k, skip mask) and replayed (nt_stream_layers and
 * nt_set_layer_skip discard it).  out_tokens (host, >= k entries) receives them, *n_out their count
 * (j + 1, or k when all are accepted), *n_accepted (nullable) j; the position
 * advances by *n_out.  Layers the skip mask names are skipped in both passes.
 * NT_E_INVAL: bad token, k or n_draft, or p + k > max_ctx. */
nt_status nt_speculative_step(nt_model* m, int32_t token, int32_t n_draft, int32_t k, int32_t* out_tokens,
                              int32_t* n_out, int32_t* n_accepted);

nt_status nt_get_stats(const nt_model* m, nt_stats* out);

/* Runs n_steps decode steps (from token, feeding back argmax) and returns
 * per-class device times: a CUDA event pair around every launch (not
 * graph-captured, no programmatic dependent launch).  For measurement only. */
nt_status nt_profile_steps(nt_model* m, int32_t token, int32_t n_steps, nt_kernel_times* out);

/* Times the step's GEMV launches on their own: one CUDA graph of a step's GEMV
 * launches (per layer QKV, O, gate/up, down, then the output head) as the step
 * issues them (programmatic dependent launches back to back), replayed n_reps
 * times between CUDA events on the model's stream.  Returns the mean device
 * time per GEMV launch, the mean algorithmic bytes per launch and the launches
 * per step.  The GEMVs read and overwrite the model's activations and the K/V
 * row at the current position: prefill or reset the cache afterwards.
 * Resident models only (NT_E_STATE otherwise).  For measurement only. */
nt_status nt_profile_gemvs(nt_model* m, int32_t n_reps, double* ms_per_launch, double* bytes_per_launch,
                           int32_t* launches_per_step);

/* Pointer to a weight tensor of the model (owned by the model).  For a
 * streamed layer the tensor refers to host memory: nt_qtensor_export works,
 * nt_gemv_q and nt_dequant return NT_E_STATE. */
nt_status nt_model_tensor(const nt_model* m, int32_t layer, int32_t role, const nt_qtensor** out);

/* -------------------------------------------------- quantized tensors -- */

/* A rows x cols quantized matrix (row-major, blocks along the columns)
 * generated on the device: element (r, c) is N(0, std^2) from (seed, uid,
 * r*cols + c), quantized by the format's rule.  NT_E_INVAL if cols is not a
 * multiple of the block (32 for Q8_0/Q4_0, 256 for Q4_K/Q6_K). */
nt_status nt_qtensor_create(nt_qtype type, int64_t rows, int64_t cols, uint64_t seed, uint32_t uid, float std,
                            nt_qtensor** out);
void nt_qtensor_destroy(nt_qtensor* t);

/* Format, shape and device bytes (the sum of the streams = rows*cols*bpw). */
nt_status nt_qtensor_info(const nt_qtensor* t, nt_qtype* type, int64_t* rows, int64_t* cols,
                          size_t* device_bytes);

/* Canonical block bytes of rows [row0, row0+nrows) into host_blocks;
 * nbytes must be at least nrows * (cols / block) * block_bytes. */
nt_status nt_qtensor_export(const nt_qtensor* t, int64_t row0, int64_t nrows, void* host_blocks, size_t nbytes);

/* Dequantized fp32 weights of rows [row0, row0+nrows) into dev_out
 * (nrows*cols floats, row-major), bit-exact under the formats' fp32
 * formulas (Q4_K as one fused multiply-add: fma(d*sc, q, -(dmin*m))). */
nt_status nt_dequant(const nt_qtensor* t, int64_t row0, int64_t nrows, float* dev_out, void* stream);

/* y = W x (hada "cuda/: GEMV-...-Kernel"): dev_x fp32[cols], dev_y fp32[rows].
 * Codes are multiplied exactly in integers against x carried as 16-bit fixed
 * point per 32-column block (error at most 2^-16 of the block's largest |x|);
 * per-block results are scaled and accumulated in fp32.  Asynchronous on
 * stream; launched with programmatic dependent launch, so it may start (and
 * read W) before the previous kernel on the stream ends, but reads x and
 * writes y only after it.  dev_x and dev_y must not overlap and must be
 * 16-byte aligned.  Matrices wider than 32768 columns (a multiple of 1024;
 * NT_E_UNSUPPORTED otherwise) run as launches over column windows of at most
 * 32768, each adding its window's products to y in window order. */
nt_status nt_gemv_q(const nt_qtensor* t, const float* dev_x, float* dev_y, void* stream);

/* y_i = W x_i for k vectors (1 <= k <= 8) in as few launches as fit: the
 * verification GEMV of self-speculative decoding (hada "Hauptfunktionen"), where
 * k draft tokens go through the same weights.  Each launch stages the x of up to
 * four tokens beside its weight ring and multiplies every weight tile it copies
 * by each of them, so the weights are read once per launch instead of once per
 * vector; where fewer than two x fit, one launch per vector.  Every y_i is bit for
 * bit what nt_gemv_q(t, dev_x[i], dev_y[i]) writes.  dev_x and dev_y are host
 * arrays of k device pointers (16-byte aligned; no y may overlap an x or another
 * y).  launches (nullable, host) receives the number of launches.  Asynchronous
 * on stream.  NT_E_INVAL: k outside [1, 8], NULL or misaligned vectors, overlaps. */
nt_status nt_gemv_q_batch(const nt_qtensor* t, const float* const* dev_x, float* const* dev_y, int32_t k,
                          int32_t* launches, void* stream);

/* ------------------------------------------------------------ attention -- */

/* GQA decode attention over an f16 cache, the step the decode step runs once
 * per layer (hada "Überblick": Llama with GQA and a KV cache; "Architektur und
 * Codestruktur": the softmax kernel).  For every query head j, with kv head
 * g = j / (n_heads / n_kv_heads):
 *   s_t = (q_j . K[g][t]) / sqrt(head_dim)  for t in [0, n_ctx),
 *   out_j = sum_t softmax(s)_t V[g][t]      (softmax with the maximum subtracted).
 * dev_q: fp32 [n_heads][head_dim], already rotated.  dev_k, dev_v: f16
 * [n_kv_heads][max_ctx][head_dim] (one layer of a model's cache); only
 * positions [0, n_ctx) are read.  dev_out: fp32 [n_heads][head_dim].
 * It runs the kernel the decode step launches, split into the same items as a
 * model with this max_ctx: chunks of C positions, C = max(32, 16 ceil(max_ctx/128))
 * up to max_ctx 2560 and min(320, 16 ceil(max_ctx/256)) beyond, ceil(max_ctx / C)
 * items per kv head, of which the first ceil(n_ctx / per) take
 * per = max(32, ceil(n_ctx / items)) positions each (the last the rest).  The
 * item partials are merged in a fixed order, so results do not depend on
 * timing; where the GPU can hold one thread-block cluster of a kv head's items
 * for every kv head at once the merge reads them across the cluster, otherwise
 * through the workspace, with the same arithmetic and bit-identical results.
 * dev_workspace: nt_attention_workspace_bytes() bytes of device memory or more,
 * owned by the caller; its contents on entry do not matter.  Calls that share a
 * workspace must not overlap on the GPU.  All device pointers 16-byte aligned;
 * dev_out and the workspace overlap no other buffer.
 * Asynchronous on stream: a one-CTA setup kernel, then the attention kernel.
 * NT_E_INVAL: n_ctx outside [1, max_ctx], non-positive sizes, n_heads not a
 * multiple of n_kv_heads, NULL, misaligned or overlapping pointers, a workspace
 * too small.  NT_E_UNSUPPORTED: head_dim other than 64 or 128, or n_heads /
 * n_kv_heads other than 1, 2, 4, 8 or 16. */
nt_status nt_attention_workspace_bytes(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t max_ctx,
                                       size_t* bytes);
nt_status nt_attention(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t max_ctx, int32_t n_ctx,
                       const float* dev_q, const void* dev_k, const void* dev_v, float* dev_out, void* dev_workspace,
                       size_t workspace_bytes, void* stream);

/* --------------------------------------------------- paged 4-bit K/V cache -- */

/* A K/V cache of several sequences at 4.5 bits per value, cut into pages that
 * sequences can share (the branches of a speculative draft, several samples of
 * one prompt), with the attention that reads it and the operators on its pages.
 * It stands beside the model's own f16 cache; the pages have no counterpart.
 *
 * Values.  Every 32 consecutive dimensions of a position and kv head are a Q4_0
 * block, value d (q - 8), whose scale has six mantissa bits:
 *   A = max |x|, h = the bits of f16(A r), r = 1 / 7 in fp32 (all roundings to nearest),
 *   d = the f16 of bits (h + 8) & 0xfff0,
 *   q = min(max(round(x / d) + 8, 0), 15), halves away from zero; 8 where d = 0.
 * A block that holds a NaN or an infinity, or whose d is above 896, is stored as
 * d = NaN and reads as NaN.
 * Six mantissa bits make every value, and the products the attention forms on
 * the way to it, exact in f16.
 *
 * Pages.  A page holds page_len positions of one layer: for each kv head its
 * page_len / 16 chunks of 16 positions, 18 head_dim bytes each.  With NG =
 * head_dim / 32, a chunk is
 *   K codes  [i 2][n 8][tg 4][j NG] words: position 8i + n, dimensions 32j + 8tg + 0..7
 *   V codes  [r 2][gi 8][tg 4][j NG] words: low half position 8r + 2tg, high half
 *            the next one, each of dimensions 32j + 4gi + 0..3
 *   K scales [position 16][j NG] f16
 *   V scales [r 2][tg 4][j NG][2] f16: positions 8r + 2tg and the next one
 * with the lowest dimension in the lowest bits of a word or half.
 *
 * The caller owns every buffer.  page p of layer l starts at pool +
 * (l * n_pages + p) * page bytes.  table[s][j] is the page of positions
 * [j page_len, (j + 1) page_len) of sequence s in every layer, for j <
 * ceil(len[s] / page_len), and -1 beyond; refs[p] counts the table entries that
 * name page p (0: free).  A new cache has table -1, len 0, refs 0, error 0.
 *
 * What the device finds wrong (lists, tables and lengths live there) is ORed
 * into *error as NT_KV4_* bits and never cleared by the library; each function
 * says what it leaves undone.  No such value makes a kernel read or write out of
 * the cache's bounds.  Calls on one cache, and calls that share a workspace,
 * must not overlap on the GPU, but for reads (nt_kv4_read, nt_attention_kv4 with
 * a workspace each).  All calls are asynchronous on stream, allocate nothing, can
 * be captured into a graph, and give the same result in every run.
 * Host checks, NT_E_INVAL: NULL or misaligned pointers (pool, workspaces, k, v, q
 * and out 16 bytes; all int32 arrays 4), sizes outside the ranges below, a
 * workspace too small, buffers that overlap.  NT_E_UNSUPPORTED: head_dim other
 * than 64 or 128. */
typedef struct {
  int32_t n_layers;     /* 1..65535                                                      */
  int32_t n_kv_heads;   /* 1..65535                                                      */
  int32_t head_dim;     /* 64 or 128                                                     */
  int32_t page_len;     /* positions per page: a multiple of 16, 16..256                 */
  int32_t n_pages;      /* pages of each layer, at least 1                               */
  int32_t max_seqs;     /* rows of the table, 1..65536                                   */
  int32_t max_pages;    /* columns of the table; max_pages * page_len at most 2^31 - 256 */
  void* pool;           /* dev: nt_kv4_pool_bytes() bytes                                */
  int32_t* table;       /* dev [max_seqs][max_pages]                                     */
  int32_t* len;         /* dev [max_seqs]: positions held                                */
  int32_t* refs;        /* dev [n_pages]                                                 */
  uint32_t* error;      /* dev [1]: NT_KV4_* bits                                        */
} nt_kv4_cache;

enum {
  NT_KV4_BAD_SEQ = 1,   /* a sequence out of range, listed twice, or not empty where it has to be */
  NT_KV4_BAD_LEN = 2,   /* a length, count or row range that does not fit                */
  NT_KV4_BAD_PAGE = 4,  /* a page index out of range, or a reference count that contradicts the call */
  NT_KV4_NO_PAGE = 8,   /* too few free pages                                            */
  NT_KV4_TIMEOUT = 16   /* a kernel gave up waiting for its own copies                   */
};

/* Bytes of one page of one layer, and of the whole pool (either nullable). */
nt_status nt_kv4_pool_bytes(const nt_kv4_cache* c, size_t* page_bytes, size_t* pool_bytes);

/* Bytes of a workspace that serves every call below on this cache with at most n
 * listed sequences, and nt_attention_kv4 with n_heads query heads.  Its contents
 * on entry do not matter. */
nt_status nt_kv4_workspace_bytes(const nt_kv4_cache* c, int32_t n_heads, int32_t n, size_t* bytes);

/* Room for dev_count[i] >= 0 more positions of each listed sequence dev_seq[i], i < n
 * (n <= max_seqs; dev_seq NULL: sequences 0..n-1): len grows by the count, and the
 * pages that it needs beyond those held are the lowest free ones, in list order.
 * Where the last page held is partly filled and shared (refs > 1), the sequence
 * gets a copy of it in a page of its own.  The new positions' contents are
 * whatever the pages held: nt_kv4_append writes them.  If any entry is invalid or
 * the free pages do not suffice, the call changes nothing but *error. */
nt_status nt_kv4_extend(const nt_kv4_cache* c, int32_t n, const int32_t* dev_seq, const int32_t* dev_count,
                        void* dev_workspace, size_t workspace_bytes, void* stream);

/* Sequence dev_dst[i], empty before, becomes the first dev_keep[i] positions of
 * dev_src[i] (dev_keep NULL: all of them): the full pages are shared, a partly
 * filled last one is copied into the lowest free page.  A source may be listed
 * several times, a destination once; a destination may be no source.  If any entry
 * is invalid, a page of a source's kept positions is out of range or held by nobody
 * (refs below 1), or the free pages do not suffice, the call changes nothing but
 * *error. */
nt_status nt_kv4_fork(const nt_kv4_cache* c, int32_t n, const int32_t* dev_src, const int32_t* dev_dst,
                      const int32_t* dev_keep, void* dev_workspace, size_t workspace_bytes, void* stream);

/* Listed sequences (dev_seq NULL: 0..n-1) keep their first dev_keep[i] positions (dev_keep NULL: none): the
 * pages behind are given back (refs one lower, the table entry -1).  An invalid
 * entry (keep outside [0, len], a sequence listed before) is passed over. */
nt_status nt_kv4_free(const nt_kv4_cache* c, int32_t n, const int32_t* dev_seq, const int32_t* dev_keep, void* stream);

/* Page dev_dst[i] becomes a copy of page dev_src[i] in every layer (n <= n_pages and 2^20);
 * tables and counts stay.  A pair is passed over (NT_KV4_BAD_PAGE) where a page is out of
 * range, its destination is one of an earlier pair, or its source is the
 * destination of another. */
nt_status nt_kv4_copy_pages(const nt_kv4_cache* c, int32_t n, const int32_t* dev_src, const int32_t* dev_dst,
                            void* stream);

/* Moves the pages in use (refs > 0), L of them, below page L, so that the pages
 * from L on are free: the k-th free page below L takes the k-th page in use from
 * L on, in every layer.  dev_table_out [max_seqs][max_pages] and dev_refs_out
 * [n_pages] receive the table and counts that go with it; each is either the
 * cache's own array or one that does not overlap it (the cache then still
 * describes the state before: moved pages keep their old bytes until they are
 * taken).  dev_live: L.  Table entries other than -1 that are out of range are copied
 * as they are, those that name a free page become -1; both set NT_KV4_BAD_PAGE. */
nt_status nt_kv4_compact(const nt_kv4_cache* c, int32_t* dev_table_out, int32_t* dev_refs_out, int32_t* dev_live,
                         void* dev_workspace, size_t workspace_bytes, void* stream);

/* Quantizes rows of keys (already rotated) and values into layer `layer`: rows
 * [dev_begin[i], dev_begin[i+1]) belong to the listed sequence dev_seq[i] (NULL:
 * sequence i) and become its last positions, the last row position len - 1.
 * dev_begin [n + 1] int32, ascending; NULL: one row each.  n_rows: rows of k and v;
 * those outside [dev_begin[0], dev_begin[n]) are not read.  Row r of kv head g
 * starts at element r * row_stride + g * head_stride of dev_k and of dev_v (f32 or f16 by
 * `type`: NT_F32, NT_F16; both strides multiples of 16 bytes), head_dim elements
 * each: a projection's [row][kv head][dim] as well as an f16 cache's [kv
 * head][position][dim].  n_rows / 16 + 2 n is at most 2^26, and n_kv_heads times
 * one more than that 2^32 - 2^17.  An entry is passed over where its sequence is out
 * of range, it has more rows than the sequence positions or rows outside [0, n_rows)
 * (dev_begin NULL: entry i's row is row i), or its range runs backwards (rows of other
 * entries may be passed over then too); rows are where their page is out of range or
 * not held by this sequence alone (refs other than 1).  With n_rows = 0 the lists are
 * not looked at.
 * A sequence listed twice is flagged; which of its rows are stored is not defined. */
nt_status nt_kv4_append(const nt_kv4_cache* c, int32_t layer, int32_t n, const int32_t* dev_seq,
                        const int32_t* dev_begin, int32_t n_rows, nt_qtype type, const void* dev_k, const void* dev_v,
                        int64_t row_stride, int64_t head_stride, void* stream);

/* The inverse: the last positions of the listed sequences, as nt_kv4_append would
 * write them, dequantized into dev_k and dev_v (f32 exactly; f16 rounded to nearest,
 * which is exact).  A sequence may be listed several times, and its pages shared.  Rows passed over, and
 * rows outside [dev_begin[0], dev_begin[n]), are left as they were. */
nt_status nt_kv4_read(const nt_kv4_cache* c, int32_t layer, int32_t n, const int32_t* dev_seq,
                      const int32_t* dev_begin, int32_t n_rows, nt_qtype type, void* dev_k, void* dev_v,
                      int64_t row_stride, int64_t head_stride, void* stream);

/* nt_attention over the paged cache: for the listed sequences (dev_seq NULL: 0..n-1;
 * a sequence may be listed several times) and every query head j, kv head g = j /
 * (n_heads / n_kv_heads),
 *   out_ij = sum_t softmax_t(q_ij . K[g][t] / sqrt(head_dim)) V[g][t],  t in [0, len),
 * and zeros where len = 0.  dev_q and dev_out: fp32, sequence i at element i * q_stride
 * and i * out_stride (multiples of 4, at least n_heads * head_dim), [n_heads][head_dim] each.
 * The statistics and sums are fp32; K and V enter exactly, q and the softmax
 * weights with about 22 bits (a weight of less than 2^-9 of the head's largest to
 * 2^-31 of that: an f16 pair ends there).  Scores may be of any size below 2^126.
 * A sequence out of range, a length that the table
 * cannot hold and a page index out of range give NaN in that sequence's outputs.
 * n at most 65536, n_kv_heads * max_pages * page_len at most 2^34 and a layer of the pool
 * at most 2^31 - 1 chunks.
 * NT_E_UNSUPPORTED: n_heads / n_kv_heads other than 1, 2, 4, 8 or 16. */
nt_status nt_attention_kv4(const nt_kv4_cache* c, int32_t layer, int32_t n_heads, int32_t n, const int32_t* dev_seq,
                           const float* dev_q, int64_t q_stride, float* dev_out, int64_t out_stride,
                           void* dev_workspace, size_t workspace_bytes, void* stream);

/* --------------------------------------------------- paged 8-bit K/V cache -- */

/* The paged cache at 8 bits per value: between the 4-bit one, whose pages, tables
 * and page operators it shares, and the f16 one; with the position rotation on the
 * way in, and attention to all positions or to the pages that a cheap score selects.
 * The pages have no counterpart.
 *
 * Values.  A page (page_len positions of one layer) has, for each kv head, one
 * exponent for its keys and one for its values; a value is an e4m3 code (1 sign, 4
 * exponent and 3 mantissa bits, bias 7, no infinity) times 2^exponent.  With A the
 * largest magnitude among the finite values up to 448 2^100,
 *   e(A) = the smallest integer from -100 on with A <= 448 2^e(A),
 *   code = x 2^-e rounded to nearest, ties to even.
 * NaN, infinities and magnitudes above 448 2^100 are stored as the code NaN, and
 * attention to such a position gives NaN.  The exponent of a page is e(A) of the rows
 * that began it; rows added later raise it to theirs where that is larger, and the
 * codes held are then rounded again for the larger one (an exact step but for codes
 * that lose bits at the lower end).  It falls when the page is begun anew: rows that
 * start at its first position.
 * Bounds.  Each page and kv head also has lo[d] and hi[d], whole numbers in units of
 * 2^(key exponent + 2): floor of the least and ceiling of the largest key code value
 * / 4 among the rows since the page was begun (-127 and 127 where one was NaN); when
 * the exponent rises, they are halved as often, rounded outwards.
 *
 * Pages.  page p of layer l starts at pool + (l * n_pages + p) * page bytes:
 *   for each kv head  K codes [page_len / 8][head_dim / 16][8][16]: (t / 8, d / 16, t % 8, d % 16)
 *                     V codes [page_len / 16][head_dim][16]:        (t / 16, d, t % 16)
 *   for each kv head  int8 K exponent, int8 V exponent, 14 bytes unused, int8 lo [head_dim], hi [head_dim]
 * The layouts are those in which the tensor cores read 8-bit operands from shared
 * memory, so a page's codes are copied there and multiplied as they are.
 *
 * Ownership, tables, lengths, counts, error bits, overlap of calls, host checks: as
 * for nt_kv4_cache, with NT_KV4_* bits.  NT_E_UNSUPPORTED: head_dim other than 64 or
 * 128, page_len other than 16, 32, 64 or 128. */
typedef struct {
  int32_t n_layers;     /* 1..65535                                                      */
  int32_t n_kv_heads;   /* 1..65535                                                      */
  int32_t head_dim;     /* 64 or 128                                                     */
  int32_t page_len;     /* positions per page: 16, 32, 64 or 128                         */
  int32_t n_pages;      /* pages of each layer, at least 1                               */
  int32_t max_seqs;     /* rows of the table, 1..65536                                   */
  int32_t max_pages;    /* columns of the table; max_pages * page_len at most 2^31 - 256 */
  void* pool;           /* dev: nt_kv8_pool_bytes() bytes                                */
  int32_t* table;       /* dev [max_seqs][max_pages]                                     */
  int32_t* len;         /* dev [max_seqs]: positions held                                */
  int32_t* refs;        /* dev [n_pages]                                                 */
  uint32_t* error;      /* dev [1]: NT_KV4_* bits                                        */
} nt_kv8_cache;

/* Bytes of one page of one layer, and of the whole pool (either nullable). */
nt_status nt_kv8_pool_bytes(const nt_kv8_cache* c, size_t* page_bytes, size_t* pool_bytes);

/* Bytes of a workspace that serves every call below on this cache with at most n
 * listed sequences (65536 for any larger n: no call takes more), and nt_kv8_select and
 * nt_attention_kv8 with n_heads query heads.  Its contents on entry do not matter. */
nt_status nt_kv8_workspace_bytes(const nt_kv8_cache* c, int32_t n_heads, int32_t n, size_t* bytes);

/* The page operators, as nt_kv4_extend, nt_kv4_fork, nt_kv4_free, nt_kv4_copy_pages
 * and nt_kv4_compact.  A copied page keeps its exponents and bounds, also where fewer
 * positions of it are kept: the bounds still hold. */
nt_status nt_kv8_extend(const nt_kv8_cache* c, int32_t n, const int32_t* dev_seq, const int32_t* dev_count,
                        void* dev_workspace, size_t workspace_bytes, void* stream);
nt_status nt_kv8_fork(const nt_kv8_cache* c, int32_t n, const int32_t* dev_src, const int32_t* dev_dst,
                      const int32_t* dev_keep, void* dev_workspace, size_t workspace_bytes, void* stream);
nt_status nt_kv8_free(const nt_kv8_cache* c, int32_t n, const int32_t* dev_seq, const int32_t* dev_keep, void* stream);
nt_status nt_kv8_copy_pages(const nt_kv8_cache* c, int32_t n, const int32_t* dev_src, const int32_t* dev_dst,
                            void* stream);
nt_status nt_kv8_compact(const nt_kv8_cache* c, int32_t* dev_table_out, int32_t* dev_refs_out, int32_t* dev_live,
                         void* dev_workspace, size_t workspace_bytes, void* stream);

/* Rows of keys and values into the last positions of the listed sequences, as
 * nt_kv4_append takes them (lists, row ranges, strides, types, limits with page_len in the
 * place of 16, what is passed over and flagged).
 * freq (host, head_dim / 2 doubles, read before the call returns; NULL: the keys
 * are rotated already): pair (2i, 2i + 1) of a key at position p is rotated by the
 * angle p freq[i], in radians (RoPE with base theta: freq[i] = theta^(-2i / head_dim)),
 *   (a, b) -> (a cos - b sin, a sin + b cos), rounded to fp32 once: products and sums carry about 45 bits,
 * the angle is exact to 2^-33 of a turn at any position.
 * dev_q (nullable; needs freq): queries of the same rows and type, row r at element
 * r * q_stride, [n_heads][head_dim]; dev_q_out (fp32, row r at element r *
 * q_out_stride) receives them rotated by their rows' positions.  Both strides are
 * multiples of 16 bytes and at least n_heads * head_dim.  In place (dev_q_out ==
 * dev_q) with NT_F32 and equal strides, else apart from every other buffer.  Rows of
 * entries that are passed over are left as they were in dev_q_out.
 * NT_E_INVAL: a frequency that is not finite or above 2^20 in magnitude. */
nt_status nt_kv8_append(const nt_kv8_cache* c, int32_t layer, int32_t n, const int32_t* dev_seq,
                        const int32_t* dev_begin, int32_t n_rows, nt_qtype type, const void* dev_k, const void* dev_v,
                        int64_t row_stride, int64_t head_stride, const double* freq, int32_t n_heads, const void* dev_q,
                        int64_t q_stride, float* dev_q_out, int64_t q_out_stride, void* stream);

/* The last positions of the listed sequences out of the cache, as nt_kv4_read (f32:
 * exactly; f16: rounded to nearest). */
nt_status nt_kv8_read(const nt_kv8_cache* c, int32_t layer, int32_t n, const int32_t* dev_seq,
                      const int32_t* dev_begin, int32_t n_rows, nt_qtype type, void* dev_k, void* dev_v,
                      int64_t row_stride, int64_t head_stride, void* stream);

/* Which pages each listed sequence's query should attend to, by an upper bound of its
 * scores on each page.  For entry i and kv head g, with q_h the query heads of g,
 * f the smallest integer such that the largest finite |q_hd| is at most 63 2^f (0
 * where all are zero),
 *   w_hd = q_hd 2^-f rounded to nearest, ties to even (infinities +-63, NaN 0),
 *   score(j) = 2^e_j sum_h sum_d max(w_hd lo_jd, w_hd hi_jd),   e_j page j's key exponent,
 * a sum of whole numbers below 2^24, so the choice does not depend on any order of
 * additions.  Of the m pages that hold the first ctx positions (dev_ctx[i]; NULL: all
 * of len), the first n_first and the last n_last are chosen and, up to n_select in
 * all, those of the highest scores, the lower page where scores are equal; all of them
 * where m <= n_select.  dev_pages [n][n_kv_heads][n_select] receives their places in
 * the sequence's table row, ascending, -1 behind.
 * An entry whose sequence or length is out of range gets -1 and sets its error bit; a page index
 * out of range counts as a page without bounds (score 0) and sets NT_KV4_BAD_PAGE.
 * NT_E_INVAL: n_select outside [1, 65536], n_first or n_last negative, n_first + n_last above n_select, or
 * n * n_kv_heads above 2^24.
 * NT_E_UNSUPPORTED: more than 16 query heads per kv head. */
nt_status nt_kv8_select(const nt_kv8_cache* c, int32_t layer, int32_t n_heads, int32_t n, const int32_t* dev_seq,
                        const int32_t* dev_ctx, const float* dev_q, int64_t q_stride, int32_t n_select, int32_t n_first,
                        int32_t n_last, int32_t* dev_pages, void* dev_workspace, size_t workspace_bytes, void* stream);

/* nt_attention over the 8-bit cache, as nt_attention_kv4 (lists, strides, empty and
 * unreadable sequences, limits).  dev_ctx (nullable): entry i attends to the first dev_ctx[i]
 * positions of its sequence, 0 <= dev_ctx[i] <= len, so that drafted tokens, listed
 * with their sequence once each, see the positions up to their own.
 * n_select = 0: all positions.  n_select > 0: those in the pages dev_pages
 * [n][n_kv_heads][n_select] names (nt_kv8_select): places in the table row, ascending,
 * each once, negative ones only behind them.  Where m pages hold the ctx positions, the
 * first min(m, n_select) places are looked at (no more can be right); one of them that is m or more,
 * not above the one before it, or behind a negative one, gives NaN in that entry's and kv
 * head's outputs and sets NT_KV4_BAD_PAGE.  No place at all, or no position, gives zeros.
 * Statistics and sums are fp32; codes enter exactly, q with about 24 bits.  A softmax weight is
 * held to 2^-28 of its head's largest where the values of its tile (128 positions) have one
 * exponent, to 2^-21 where their exponents lie up to 7 apart.  Where they lie further apart, or
 * the largest is more than 4 above that of a tile before, it is held to that share of the largest
 * weight of the tile that goes with values of like size (and the tile takes about three times as
 * long for two sizes, longer for more).  Below that a weight is kept or dropped by turns, so that
 * the sum of many holds: n of them are off by about sqrt(n) 2^-29, not by n.  Any 1 to 16 query
 * heads per kv head
 * (NT_E_UNSUPPORTED beyond). */
nt_status nt_attention_kv8(const nt_kv8_cache* c, int32_t layer, int32_t n_heads, int32_t n, const int32_t* dev_seq,
                           const int32_t* dev_ctx, int32_t n_select, const int32_t* dev_pages, const float* dev_q,
                           int64_t q_stride, float* dev_out, int64_t out_stride, void* dev_workspace,
                           size_t workspace_bytes, void* stream);

/* ------------------------------------------------ allocation-free variant -- */

/* y = W x as nt_gemv_q, then the index of the largest y (ties to the lowest
 * row; NaN values are never selected) into dev_index and the gap between the
 * largest and second-largest y into dev_margin (both device pointers, 4-byte
 * aligned).  dev_index is -1 only when every y is NaN; dev_margin is +inf when
 * a single y is not NaN, and NaN when the two largest are both +inf.  The pages have no counterpart: this entry point exists for
 * callers that cannot allocate device memory on this path, such as embedders
 * whose device memory is all reserved by their own allocator, or latency-bound
 * loops that cannot afford the implicit synchronisation of cudaMalloc/cudaFree.
 * It allocates nothing: the per-CTA partial results of the selection live in a
 * file-scope device array of 1024 x 16 bytes (16 KiB) that every GPU loading
 * this library holds until the process exits.  The first call on a device, with
 * that device current, looks up the array's device address
 * (cudaGetSymbolAddress) and keeps it for the life of the process; make that
 * first call before any stream capture, and make no call on a device after a
 * cudaDeviceReset of it (the reset unloads the array and the kept address goes
 * stale).
 * Every call shares the array and overwrites what it reads, so nothing needs
 * clearing, but calls that overlap on the GPU (for example on two streams at
 * once) race on it: serialise them.  Asynchronous on stream.
 * The GEMV launch is capped at 1024 CTAs, one summary slot each.
 * Errors: nt_gemv_q's argument rules; NT_E_INVAL for more than 2^31 - 2 rows;
 * NT_E_UNSUPPORTED for more than 28672 columns. */
nt_status nt_gemv_argmax_noalloc(const nt_qtensor* t, const float* dev_x, float* dev_y, int32_t* dev_index,
                                 float* dev_margin, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* NT_H */
