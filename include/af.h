/*
 * af.h — C ABI of the GB300 (sm_103a) forward pass of a GGUF-quantized
 * Llama-style decoder.
 *
 * What it computes (page title, section):
 *  - Airframe "GPU_PIPELINE.md" (Shimmy docs), per-layer operation diagram:
 *    RMS norm -> Q/K/V projections with inline dequantization -> RoPE with
 *    theta(t, i) = (t / yarn_scale) / base^(2i / head_dim) and
 *    yarn_scale = max_ctx / native_ctx when max_ctx > native_ctx -> K, V written
 *    to the KV cache at position t -> softmax(Q K^T / sqrt(head_dim)) V ->
 *    O projection + residual -> RMS norm -> gate, up -> gate*sigmoid(gate)*up
 *    -> down + residual.  "Prefill": prompts run in chunks of up to 512 tokens
 *    that fill KV slots start_pos..start_pos+n-1; only the last chunk's logits
 *    are used.  "Decode": one token at position t attends to slots 0..t.
 *    "Output head": LM head on the last position.  "KV cache": layout
 *    [n_layers][n_kv_heads][max_ctx][head_dim], K and V separate.
 *  - "Shimmy v2.0 Architecture", "Quantization": GGUF Q4_0 and Q8_0
 *    32-element blocks; "Extended Context (YaRN)": the theta scale applies to
 *    all positions.
 *  - "GPU Inference — dotLLM", "Forward Pass" (final RmsNorm on the last token,
 *    LM head, one host sync per step) and "Attention on GPU" (causal, GQA with
 *    group = n_heads / n_kv_heads).
 *
 * Conventions.
 *  - Every call returns an af_status.  Arguments are validated on the host
 *    before anything is launched; a call that fails validation changes nothing.
 *    af_last_error() returns a thread-local message for the last failure.
 *  - "_dev" pointers are device pointers on the current CUDA device; "_host"
 *    pointers are ordinary host memory.  `stream` is a cudaStream_t (NULL =
 *    legacy default stream).  Unless stated otherwise a call only enqueues
 *    work on the model's (or the given) stream and returns.
 *  - The caller owns every pointer it passes.  af_model_create and
 *    af_qweight_create copy (repack) the weights into memory they own, so the
 *    caller may free its blobs once the call has returned and the stream has
 *    been synchronised.
 *  - Weights: GGUF blocks, little-endian.
 *      Q8_0 (34 B): fp16 d, int8 q[32];             w_j = d * q_j
 *      Q4_0 (18 B): fp16 d, uint8 qs[16];            w_j = d * (n_j - 8),
 *                   n_j = qs[j] & 15 (j < 16), qs[j - 16] >> 4 (j >= 16)
 *      Q4_K (144 B per 256 weights): fp16 d, fp16 dmin, uint8 scales[12],
 *                   uint8 qs[128]; 6-bit scale s_j and min m_j of sub-block
 *                   j = e / 32 (j < 4: scales[j] & 63, scales[j + 4] & 63;
 *                   j >= 4: (scales[j + 4] & 15) | (scales[j - 4] >> 6) << 4,
 *                   (scales[j + 4] >> 4) | (scales[j] >> 6) << 4); code n_e in
 *                   the low (e % 64 < 32) or high nibble of qs[32 (e / 64) + e % 32];
 *                   w_e = d s_j n_e - dmin m_j
 *      Q5_K (176 B per 256 weights): fp16 d, fp16 dmin, uint8 scales[12] (as
 *                   Q4_K), uint8 qh[32], uint8 qs[128] (nibbles placed as Q4_K's);
 *                   the 5-bit code q_e = nibble + 16 * (bit 2 (e / 64) + (e % 64 >= 32)
 *                   of qh[e % 32]); w_e = d s_j q_e - dmin m_j
 *      Q6_K (210 B per 256 weights): uint8 ql[128], uint8 qh[64], int8
 *                   scales[16], fp16 d; with h = e / 128, k = (e % 128) / 32,
 *                   l = e % 32 the code q_e has its low 4 bits in the low (k < 2)
 *                   or high nibble of ql[64 h + 32 (k & 1) + l] and its high 2 bits
 *                   at bits 2k of qh[32 h + l]; w_e = d scales[e / 16] (q_e - 32)
 *    (Shimmy v2.0 Architecture, "Quantization": the K-quant super-blocks; their
 *    byte layout is GGUF's.)  A matrix [N, K] is N rows of K / 32 blocks each
 *    (K / 256 super-blocks for Q4_K, Q5_K and Q6_K; K must be a whole number of blocks).
 */
#ifndef AF_H
#define AF_H
#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum af_status {
    AF_OK = 0,
    AF_EINVAL = 1,   /* bad argument: null pointer, unsupported shape or type */
    AF_ERANGE = 2,   /* position / token id / size out of range */
    AF_ENOMEM = 3,   /* device or host allocation failed (nothing leaked) */
    AF_ECUDA = 4,    /* a CUDA runtime call failed; see af_last_error() */
    AF_ETIMEOUT = 5, /* a bounded device-side wait gave up */
    AF_ENOTIMPL = 6  /* valid request this build does not implement */
} af_status;

typedef enum af_wtype { AF_Q4_0 = 2, AF_Q8_0 = 8, AF_Q4_K = 12, AF_Q5_K = 13, AF_Q6_K = 14 } af_wtype; /* GGUF's type numbers */
/* KV cache element types.  AF_KV_Q8_0 / AF_KV_Q4_0: a quantized cache with an fp16 window (dotLLM, "CUDA
 * components": "Q8_0/Q4_0 + FP16 window"): a slot is written in fp16; once it lies more than kv_window
 * positions behind a step's last position it is replaced by the Q8_0 / Q4_0 quantization of its fp16 values,
 * per 32 values along head_dim (Q8_0: d = fp16(max|v| / 127), q = clamp(round-half-away(v / d), -127, 127);
 * Q4_0: d = fp16(m / -8) with m the value of largest magnitude, n = clamp(floor(v / d + 8.5), 0, 15),
 * q = n - 8; decisions in fp32 on the fp16 values), and reads of the slot see d * q.  Decode attention reads
 * retired slots from the quantized store; prefill attention reads the fp16 copy, where a retired slot holds
 * fp16(d * q). */
typedef enum af_dtype { AF_F32 = 0, AF_F16 = 1, AF_KV_Q8_0 = 2, AF_KV_Q4_0 = 3 } af_dtype;

typedef struct af_config {
    int32_t n_layers, n_embd, n_heads, n_kv_heads, head_dim, n_ff, n_vocab;
    int32_t wtype;      /* af_wtype of every matrix and of token_embd */
    int32_t kv_dtype;   /* af_dtype of the KV cache */
    int32_t max_ctx;    /* KV slots */
    int32_t native_ctx; /* yarn_scale = max_ctx / native_ctx if max_ctx > native_ctx, else 1 */
    int32_t max_chunk;  /* largest n accepted by af_prefill (0 = 512) */
    float rms_eps;      /* RMSNorm epsilon */
    float rope_base;    /* RoPE base */
    int32_t out_wtype;  /* af_wtype of the LM head (output.weight); 0 = wtype (a Q4_K_M model: Q4_K layers and
                           embedding with a Q6_K head) */
    int32_t kv_window;  /* quantized caches: slots kept in fp16 behind a step's last position; at least max_chunk, so
                           a step is never longer than the window (ignored for AF_F32 / AF_F16) */
} af_config;

/*
 * Layer blob (Airframe "GPU_PIPELINE.md", bindless layer buffer): one device
 * buffer per layer holding, in this order, each section at a 256-byte aligned
 * offset (see af_layer_offsets):
 *   attn_norm f32[E] | attn_q [H*D, E] | attn_k [KVH*D, E] | attn_v [KVH*D, E] |
 *   attn_o [E, H*D] | ffn_norm f32[E] | ffn_gate [F, E] | ffn_up [F, E] | ffn_down [E, F]
 * Matrices are [out, in] in GGUF blocks along `in`.
 */
typedef struct af_weights {
    const void* const* layer_blob; /* host array of n_layers device pointers */
    const void* token_embd;        /* device, [n_vocab, n_embd] blocks */
    const float* output_norm;      /* device, f32 [n_embd] */
    const void* output;            /* device, [n_vocab, n_embd] blocks of out_wtype (LM head, not tied) */
} af_weights;

typedef struct af_model af_model;
typedef struct af_qweight af_qweight;

/* Section offsets of a layer blob: off[0..8] in the order above, off[9] = blob bytes. */
int af_layer_offsets(const af_config* cfg, uint64_t off[10]);

/* KV cache bytes, n_layers * n_kv_heads * max_ctx * head_dim * elem * 2
 * (Airframe "GPU_PIPELINE.md", "KV cache" size formula).  A quantized cache holds every slot twice, in fp16
 * and in the quantized store: n_layers * n_kv_heads * 2 * max_ctx * (head_dim * 2 + head_dim / 32 * B),
 * B = 34 (Q8_0) or 18 (Q4_0) bytes per 32 values.  0 on a bad config. */
uint64_t af_kv_bytes(const af_config* cfg);

/*
 * Create a model on the current device.  Repacks every matrix into the
 * model's own layout, allocates the KV cache (zeroed) and the step scratch,
 * and builds the RoPE table.  Synchronises `stream` before returning.  With
 * stream == NULL the model creates (and later destroys) a blocking stream of
 * its own, which is ordered with the legacy default stream.
 * Supported: head_dim in {64, 128}, n_heads % n_kv_heads == 0 with
 * n_heads / n_kv_heads in {1, 2, 4, 8}, n_embd, n_ff, n_heads*head_dim
 * multiples of 64, even n_vocab; quantized caches: kv_window >= max_chunk and
 * max_ctx a multiple of 4.  Errors: AF_EINVAL, AF_ENOMEM, AF_ECUDA,
 * AF_ENOTIMPL (valid but unsupported shape).  *out is NULL on failure.
 */
int af_model_create(const af_config* cfg, const af_weights* w, void* stream, af_model** out);

/*
 * Prefill n tokens (1 <= n <= max_chunk) at absolute positions
 * start_pos..start_pos+n-1 (start_pos + n <= max_ctx).  Writes those KV slots;
 * row r attends to slots 0..start_pos+r.  The caller runs longer prompts as
 * consecutive chunks with increasing start_pos.  If logits_dev is not NULL it
 * receives the n_vocab fp32 logits of the last row.  tokens_host is copied
 * into the model's page-locked staging buffer before the call returns, so the
 * caller may reuse it at once (pageable or page-locked alike); the call first
 * waits for the previous af_prefill's copy out of that buffer.  Not for stream
 * capture (use af_prefill_dev there).  Errors: AF_EINVAL, AF_ERANGE (token id
 * outside [0, n_vocab) or positions past max_ctx), AF_ECUDA.
 */
int af_prefill(af_model* m, const int32_t* tokens_host, int32_t n, int32_t start_pos, float* logits_dev);

/* As af_prefill with the token ids already in device memory.  They are not
 * validated on the host; an id outside [0, n_vocab) reads embedding row 0. */
int af_prefill_dev(af_model* m, const int32_t* tokens_dev, int32_t n, int32_t start_pos, float* logits_dev);

/*
 * One decode step: the token at position pos (0 <= pos < max_ctx) attends to
 * slots 0..pos.  token = -1 feeds the previous step's greedy token (from the
 * device, no host round trip).  logits_dev (nullable) receives the fp32
 * logits.  If next_token_host is not NULL the call synchronises the model's
 * stream once and stores the greedy token there (argmax, lowest index on
 * ties); otherwise it only enqueues.
 */
int af_decode_step(af_model* m, int32_t token, int32_t pos, float* logits_dev, int32_t* next_token_host);

/* Synchronise the model's stream.  Returns AF_ETIMEOUT if a bounded device-side
 * wait of an earlier call gave up, else AF_OK; if next_token_host is not NULL it
 * receives the greedy token of the last call that produced logits.  A reported
 * timeout is cleared (af_decode_step with next_token_host reports and clears the
 * same way), so a later call reports only what happened after it.  The outputs
 * of the calls that timed out are not valid. */
int af_model_sync(af_model* m, int32_t* next_token_host);

/* Greedy token of the last af_decode_step / af_prefill with logits (device int32, valid after the stream). */
const int32_t* af_model_next_token_dev(const af_model* m);

/* Device pointers of the model's KV cache: K and V each [n_layers][n_kv_heads][max_ctx][head_dim]
 * in kv_dtype, fp16 for a quantized cache (Airframe "GPU_PIPELINE.md", "KV cache" layout).  Owned by the
 * model. */
int af_model_kv_cache(const af_model* m, void** k_dev, void** v_dev);

/* The quantized store of a quantized cache (AF_EINVAL otherwise): per slot of [n_layers][n_kv_heads][max_ctx],
 * the codes (Q8_0: head_dim int8 values q in element order; Q4_0: head_dim / 2 bytes, byte j holding
 * n = q + 8 of element 2j in its low and of element 2j + 1 in its high nibble) in *codes, and head_dim / 32 fp16
 * scales d in *scales; k_ for K, v_ for V.  Valid for slots that have retired.  Owned by the model. */
int af_model_kv_store(const af_model* m, void** k_codes, void** k_scales, void** v_codes, void** v_scales);

/* Zero the KV cache (the service is stateless between requests) and the error word.  Steps after it start
 * again at position 0; with a quantized cache, each step must start where the previous one ended (the
 * slots that leave the window are retired by the step that passes them). */
int af_reset(af_model* m);

/* Model's stream (as given to af_model_create). */
void* af_model_stream(const af_model* m);

/* Capture the residual stream after the embedding and after every layer of the
 * next af_prefill / af_decode_step into hidden_dev [n_layers+1][n][n_embd] fp32
 * (n = that call's token count).  One-shot; test instrumentation. */
int af_debug_capture(af_model* m, float* hidden_dev);

/*
 * How af_decode_step runs (both are this library's CUDA kernels):
 *   AF_DECODE_KERNELS (default): one launch per matrix / attention, chained
 *     with programmatic dependent launch and replayed as a CUDA graph (see
 *     af_set_decode_graph).
 *   AF_DECODE_PERSISTENT: one cooperative launch per token, one CTA per SM,
 *     phases (each matrix, attention) separated by bounded grid barriers; each
 *     warp's shared-memory slot streams its next stage of weights or cache
 *     tiles whatever phase it belongs to, so copies run ahead through the
 *     barriers (Q4_0 or Q8_0 for every matrix including the LM head, an fp32 or
 *     fp16 cache, head_dim 64 or 128, group 2, 4 or 8; AF_ENOTIMPL otherwise or
 *     where it cannot be resident).  Measured slower than the default.
 */
enum { AF_DECODE_PERSISTENT = 0, AF_DECODE_KERNELS = 1 };
int af_set_decode_mode(af_model* m, int mode);
int af_get_decode_mode(const af_model* m);

/* In AF_DECODE_KERNELS mode, use (1) or stop using (0) a CUDA graph (default 1). */
int af_set_decode_graph(af_model* m, int enable);

/* Trace the next persistent af_decode_step: trace_dev (device, uint64 [5 n_layers + 3])
 * receives the GPU global timer (ns) at kernel start, after the embedding, after each
 * of the 5 phases of every layer, and at the end.  One-shot; profiling aid. */
int af_debug_trace(af_model* m, uint64_t* trace_dev);

void af_model_destroy(af_model* m);

/* Test instrumentation of the error path: with polls != 0 the first wait of every decode GEMV launched
 * afterwards polls an mbarrier that nothing arrives on `polls` times, then takes its timeout path (error
 * word set, its bulk copies drained, early return) as a real timeout would; 0 turns it off.  Synchronises
 * the model's stream.  Lets a test see AF_ETIMEOUT without a fault or a hang. */
int af_debug_stall(af_model* m, uint32_t polls);

/*
 * Standalone quantized matmuls.
 * af_qweight_create repacks a [N, K] block matrix (N even, K a whole number
 * of blocks: K % 32 == 0, K % 256 == 0 for Q4_K / Q5_K / Q6_K; K <= 32768, or
 * <= 16384 for Q8_0, else AF_ENOTIMPL) into its own device memory (and
 * scratch for the GEMV); synchronises `stream`.
 *   af_qgemv: y[i]    = sum_j W[i][j] x[j]        x_dev fp32 [K], y_dev fp32 [N]
 *   af_qgemm: Y[m][i] = sum_j X[m][j] W[i][j]     X_dev fp32 [M, K] row-major,
 *                                                 Y_dev fp32 [M, N], M >= 1
 * Calls that share one af_qweight must be ordered on one stream (they share
 * its scratch).  af_qgemv accumulates exact integer products of the weight
 * codes with x held in 16-bit fixed point per 32-element block (K-quant
 * sub-block scales and mins applied per 32 or 16 elements in fp32); af_qgemm
 * runs on the tensor cores with X and W each split into fp16 hi + lo parts
 * (three fp16 products accumulated in fp32, relative error ~1e-6 per product;
 * K-quant weights are formed in fp32 before their split).
 * af_qgemm keeps the split X in buffers of the af_qweight: the first call
 * with a larger M than before synchronises `stream` and grows them.
 */
int af_qweight_create(int32_t wtype, const void* blocks_dev, int32_t N, int32_t K, void* stream, af_qweight** out);
int af_qgemv(const af_qweight* w, const float* x_dev, float* y_dev, void* stream);
int af_qgemm(const af_qweight* w, const float* X_dev, int32_t M, float* Y_dev, void* stream);
void af_qweight_destroy(af_qweight* w);

/* Synchronise `stream` and report w's error word: AF_ETIMEOUT if a bounded device-side wait of an af_qgemv /
 * af_qgemm on w gave up since the last report (the word is then cleared; those outputs are not valid), else
 * AF_OK. */
int af_qweight_status(const af_qweight* w, void* stream);

/* Test instrumentation: as af_debug_stall, for the af_qgemv calls on w (synchronises `stream`). */
int af_qweight_debug_stall(af_qweight* w, uint32_t polls, void* stream);

/*
 * Standalone causal GQA attention for one query row at position pos over a
 * caller's cache (Airframe per-layer ops: softmax(q K^T / sqrt(D)) V over
 * slots 0..pos; dotLLM "Attention on GPU": GQA group = H / KVH).
 *   q_dev   fp32 [H*D] (already rotated)
 *   k_dev, v_dev  [KVH][ctx][D] in kv_dtype
 *   out_dev fp32 [H*D]
 * Scratch (split partials) is allocated per call and freed after the stream
 * completes (the call synchronises `stream`).  AF_ETIMEOUT if a bounded
 * device-side wait gave up.
 */
int af_attention_decode(const float* q_dev, const void* k_dev, const void* v_dev, int32_t kv_dtype, int32_t n_heads,
                        int32_t n_kv_heads, int32_t head_dim, int32_t ctx, int32_t pos, float* out_dev, void* stream);

/*
 * af_attention_decode without any device allocation (no counterpart on the
 * pages: an interface for callers that cannot allocate mid-step, e.g. a
 * serving loop that cannot take the device-wide synchronisation of cudaFree,
 * or one whose memory is all handed to its own pool).  Same arguments, same
 * kernel and same result as af_attention_decode, but stream-ordered: it does
 * not synchronise `stream`.  Slots before pos are read ahead of the end of the
 * kernel before it: what af_kv_write, af_kv_read, af_rope, af_lora and
 * af_attention_paged have written into the cache is seen; a result of another
 * call of this header that lies in those slots may not be.
 * Scratch: one file-scope device array of this library (4 MiB of split
 * partials + 1024 arrival counters + an error word), used only when ctx >
 * 2048 (shorter caches take the cluster path, which merges in distributed
 * shared memory, where the device can schedule 8-CTA clusters).
 * On that path, calls with n_kv_heads > 1024 or whose partials need more than
 * 2^20 floats (n_heads * splits * (head_dim + 4), splits = max(1, 2 * SMs /
 * n_kv_heads)) return AF_ERANGE before launching.
 * Errors on the device: the call does not wait for the kernel, so it cannot
 * report AF_ETIMEOUT; if a bounded device-side wait gives up, every output
 * value of the affected kv heads is NaN instead.
 * The counters must start at zero: they are zero when the library is loaded
 * and every launch leaves them zero, a timed-out one included (each CTA
 * still arrives, and the last one resets the counter).  All calls on a device
 * share the one array, so calls that may overlap in time (different streams
 * without ordering between them) race and give wrong results: order them on
 * one stream.  The first call on each device looks up the array's address
 * (cudaGetSymbolAddress, with that device current) and loads the kernels; make
 * that first call before any stream capture.
 */
int af_attention_decode_static(const float* q_dev, const void* k_dev, const void* v_dev, int32_t kv_dtype,
                               int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t ctx, int32_t pos,
                               float* out_dev, void* stream);

/*
 * Standalone causal prefill attention (the tensor-core kernel af_prefill runs;
 * Airframe per-layer ops: softmax(q K^T / sqrt(D)) V, causal; dotLLM
 * "Attention on GPU": GQA group = H / KVH) for n query rows at positions
 * start_pos..start_pos+n-1 over a caller's cache.  Test entry point.
 *   q_dev   fp32 [n][H*D] (already rotated), row r at position start_pos + r
 *   k_dev, v_dev  [KVH][ctx][D] in kv_dtype (16-byte aligned); row r attends
 *           to slots 0..start_pos+r
 *   out_dev fp32 [n][H*D]: the fp16 hi + lo output planes of the kernel, summed
 * 1 <= n <= 512, start_pos + n <= ctx (AF_ERANGE).  The output planes are
 * allocated per call; the call synchronises `stream`.  AF_ETIMEOUT if a
 * bounded device-side wait gave up.
 */
int af_attention_prefill(const float* q_dev, const void* k_dev, const void* v_dev, int32_t kv_dtype, int32_t n_heads,
                         int32_t n_kv_heads, int32_t head_dim, int32_t ctx, int32_t start_pos, int32_t n,
                         float* out_dev, void* stream);

/*
 * Sampler chain on the device (Airframe GPU pipeline, sampler: "repetition
 * penalty -> temperature -> softmax -> top-p -> sample"): one kernel launch
 * of one 8-CTA thread-block cluster that keeps the logits in shared memory; no
 * device scratch and no allocation, so calls on different streams are
 * independent.  Asynchronous on `stream`:
 *   logits_dev  fp32 [n_vocab] (not modified), n_vocab <= 262144
 *   recent_dev  int32 [n_recent] recent token ids (device; NULL when n_recent = 0);
 *               each distinct id in [0, n_vocab) has its logit divided by
 *               repeat_penalty once (only when repeat_penalty > 1)
 *   temperature 0 -> greedy (argmax, lowest index on ties); > 0 divides the logits
 *   top_p       nucleus: the shortest prefix of the tokens sorted by
 *               (probability descending, index ascending) whose mass reaches
 *               top_p, plus every token tied with its last one; >= 1 keeps all
 *   u           the caller's uniform draw in [0, 1): the token returned is the
 *               first of that order whose cumulative mass reaches u times the
 *               nucleus mass
 *   token_dev   int32 [1] result
 * AF_EINVAL / AF_ERANGE for bad arguments (checked on the host).
 */
int af_sample(const float* logits_dev, int32_t n_vocab, const int32_t* recent_dev, int32_t n_recent,
              float repeat_penalty, float temperature, float top_p, float u, int32_t* token_dev, void* stream);

/*
 * The sampler chain (as af_sample) over a model's logits, on the model's stream:
 * the token drawn replaces the model's next-token word (af_model_next_token_dev),
 * so a following af_decode_step(m, -1, ...) feeds it.  A decode loop that
 * alternates af_decode_step(m, -1, pos, NULL, NULL) and af_model_sample(...)
 * samples on the device with no logits read back.
 *   logits_dev  the logits to sample (n_vocab fp32); NULL = the model's own
 *               buffer, which steps called with logits_dev = NULL write
 *   recent_dev, n_recent, repeat_penalty, temperature, top_p, u: as af_sample
 *   token_host  if not NULL: synchronises the model's stream once and stores
 *               the token drawn; otherwise the call only enqueues
 * AF_EINVAL / AF_ERANGE for bad arguments (checked on the host).
 */
int af_model_sample(af_model* m, const float* logits_dev, const int32_t* recent_dev, int32_t n_recent,
                    float repeat_penalty, float temperature, float top_p, float u, int32_t* token_host);

/*
 * Rotary positions on rows of heads, for queries and keys that are rotated outside af_model (drafted tokens at the
 * position of their depth, cached keys that move).  Pairs (a, b) of a head's first rot_dim values,
 *   y_a = m (x_a cos t - x_b sin t),  y_b = m (x_a sin t + x_b cos t),  t = pos * f_i,  i = 0 .. rot_dim / 2 - 1,
 * (a, b) = (2i, 2i + 1) (AF_ROPE_INTERLEAVED, as in af_model) or (i, i + rot_dim / 2) (AF_ROPE_HALF); the values from
 * rot_dim on are copied unchanged.  f_i = base^(-2i / rot_dim), for a context `factor` times native_ctx:
 *   AF_ROPE_LINEAR  f_i / factor (af_model's yarn_scale, Shimmy v2.0 Architecture, "Extended Context")
 *   AF_ROPE_NTK     the base becomes base * factor^(rot_dim / (rot_dim - 2)) (rot_dim >= 4)
 *   AF_ROPE_YARN    by parts: with r = native_ctx f_i / 2 pi turns over the native context and
 *                   w = clamp((r - turns_low) / (turns_high - turns_low), 0, 1), f_i (w + (1 - w) / factor)
 */
typedef enum af_rope_layout { AF_ROPE_INTERLEAVED = 0, AF_ROPE_HALF = 1 } af_rope_layout;
typedef enum af_rope_scaling { AF_ROPE_NONE = 0, AF_ROPE_LINEAR = 1, AF_ROPE_NTK = 2, AF_ROPE_YARN = 3 } af_rope_scaling;
typedef struct af_rope_config {
    int32_t head_dim;   /* even, <= 256 */
    int32_t rot_dim;    /* even, 2 .. head_dim */
    int32_t layout;     /* af_rope_layout */
    int32_t scaling;    /* af_rope_scaling */
    int32_t native_ctx; /* AF_ROPE_YARN */
    double base;        /* > 1; in 64 bits, as what the angles of far positions depend on */
    double factor;      /* > 0 (ignored by AF_ROPE_NONE) */
    double turns_low;   /* AF_ROPE_YARN: 0 <= turns_low < turns_high (1 and 32 in the method's paper) */
    double turns_high;
    double magnitude;   /* m; 0 = 1 (AF_ROPE_YARN's paper: 0.1 ln(factor) + 1) */
} af_rope_config;

/*
 *   x_dev   [n] rows of n_heads * head_dim values of dtype (AF_F32, or AF_F16 computed in fp32 and rounded once),
 *           consecutive rows ldx values apart (ldx >= n_heads * head_dim: the q and k heads of a fused projection
 *           are one call; the heads of a cache are one row each with n_heads = 1)
 *   y_dev   the result, rows ldy values apart; may be x_dev itself with ldy == ldx, and overlaps it in no other way
 *   pos_dev int32 [n], any value (a negative one rotates back); NULL: row r is at pos0 + r (pos0 + n - 1 < 2^31)
 * The angle is exact modulo a turn to 2^-33 of a turn at a million positions (2^-22 at 2^31; with a factor below 1, that
 * divided by the factor).  Asynchronous on `stream`, allocates nothing, can be captured.  Vectors of 16 bytes are moved
 * where rows, rot_dim and pointers allow it.  n = 0 does nothing.  Errors: AF_EINVAL, AF_ERANGE, AF_ENOTIMPL (head_dim > 256), AF_ECUDA.
 */
int af_rope(const af_rope_config* cfg, const void* x_dev, int64_t ldx, void* y_dev, int64_t ldy, int32_t dtype,
            int32_t n, int32_t n_heads, const int32_t* pos_dev, int32_t pos0, void* stream);

/*
 * Rows of keys and values into a caller's cache of any type, quantized as they are written, and slots of it back
 * as fp32 rows.  The cache of one layer, K and V each:
 *   AF_F32, AF_F16          [n_kv_heads][ctx][head_dim] values; k_scales = v_scales = NULL
 *   AF_KV_Q8_0, AF_KV_Q4_0  codes [n_kv_heads][ctx][head_dim or head_dim / 2 bytes] and fp16 scales
 *                           [n_kv_heads][ctx][head_dim / 32], as af_model_kv_store's: every slot is quantized at
 *                           once from the fp32 values given here (no fp16 window; a model's own store holds only
 *                           the slots that have left its window, so it is not a whole cache for these calls)
 * The decisions of the quantizers are those of exact arithmetic on the fp32 values.  A block of 32 that holds a NaN,
 * or whose scale overflows fp16, reads back as NaN.  What af_kv_write has written and af_kv_read returned gives the same
 * values when it is written again (scales below fp16's normal range excepted), so a read and a write move slots.
 *   k_dev, v_dev  fp32 rows [n] of n_kv_heads * head_dim values, ld apart (16-byte aligned, ld a multiple of 4)
 *   slots_dev     int32 [n]: the slot of each row; a row whose slot is outside [0, ctx) is skipped (af_kv_read
 *                 leaves its output row as it was).  Of rows with the same slot the last is written.  NULL: row r
 *                 is slot slot0 + r, inside the cache (AF_ERANGE)
 * head_dim: a multiple of 32 up to 256.  All device pointers but slots_dev are 16-byte aligned.  Asynchronous on
 * `stream`, allocate nothing, can be captured.  n = 0 does nothing.
 * Errors: AF_EINVAL, AF_ERANGE, AF_ENOTIMPL (head_dim), AF_ECUDA.
 */
int af_kv_write(const float* k_dev, const float* v_dev, int64_t ld, int32_t n, const int32_t* slots_dev, int32_t slot0,
                void* k_cache, void* k_scales, void* v_cache, void* v_scales, int32_t kv_dtype, int32_t n_kv_heads,
                int32_t head_dim, int32_t ctx, void* stream);
int af_kv_read(const void* k_cache, const void* k_scales, const void* v_cache, const void* v_scales, int32_t kv_dtype,
               int32_t n_kv_heads, int32_t head_dim, int32_t ctx, int32_t n, const int32_t* slots_dev, int32_t slot0,
               float* k_dev, float* v_dev, int64_t ld, void* stream);

/*
 * The mask and the positions of a tree of n drafted tokens (1 <= n <= 1024), once per tree for all layers:
 *   parent_dev  int32 [n]: the node a node follows, an earlier one, or -1 for the last accepted token (a value that
 *               is not an earlier node counts as -1)
 *   mask_dev    uint32 [n][(n + 31) / 32]: bit j % 32 of word j / 32 of row i is set where j is i or an ancestor
 *   pos_dev     int32 [n] (nullable): pos0 + the node's depth (0 for a child of the last accepted token)
 * Asynchronous on `stream`, allocates nothing, can be captured.  Errors: AF_EINVAL, AF_ERANGE, AF_ECUDA.
 */
int af_tree_mask(const int32_t* parent_dev, int32_t n, int32_t pos0, uint32_t* mask_dev, int32_t* pos_dev,
                 void* stream);

/*
 * Attention for a tree of drafted tokens over a caller's cache: every node sees slots 0..n_past-1, and of the slots
 * n_past..n_past+n-1, where node j's key and value are (af_kv_write with slot0 = n_past), those whose bit its mask
 * row has set; softmax(q K^T / sqrt(head_dim)) V over what it sees, GQA group = n_heads / n_kv_heads.
 *   q_dev     fp32 [n] rows of n_heads * head_dim values (rotated), ldq apart
 *   cache     as af_kv_write's; slots from n_past + n on are not read
 *   mask_dev  uint32 [n][(n + 31) / 32] as af_tree_mask writes it, or any other: a row that sees nothing (n_past = 0
 *             and no bit set) gives zeros, and what a hidden slot holds (NaN, infinities, numbers of any size) reaches
 *             no row it is hidden from
 *   ws_dev    scratch of at least af_attention_tree_workspace bytes (NULL where that is 0), 256-byte aligned, of any
 *             contents; calls that may overlap in time need scratch of their own.  A call of fewer nodes or slots may
 *             need more than a larger one (it has more splits); none needs more than
 *             512 * (the device's SMs) * (head_dim + 2) bytes, 10.1 MB with head_dim 128 on 152 SMs
 *   out_dev   fp32 [n] rows, ldo apart
 * Results keep fp32's precision: a slot's score 2^-20 of the sum of |q| times the slot's largest |k|, over sqrt(head_dim),
 * and a row's result 2^-20 of the largest weight times |v| that it sees (fp32 values above 2^110 may give infinities).
 * The bits do not change from call to call.  A row that sees a NaN or an infinity, or whose scores are all -infinity, gets
 * what the formula gives or NaN in its place, in any of its values.  The kernels' waits are bounded: rows of a block whose
 * wait gave up (copies that never arrive) are NaN.
 * 1 <= n <= 1024, 0 <= n_past <= 2^31 - 2049, n_past + n <= ctx, n_kv_heads * ctx < 2^31; head_dim 64 or 128, any whole
 * group up to 64.  Pointers are 16-byte aligned (mask_dev: 4), ldq and ldo multiples of 4.  Asynchronous on `stream`,
 * allocates nothing, can be captured (the first call on a device loads the kernels: make it before a capture).
 * Errors: AF_EINVAL, AF_ERANGE, AF_ENOTIMPL, AF_ECUDA.
 */
uint64_t af_attention_tree_workspace(int32_t kv_dtype, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                                     int32_t n_past, int32_t n);
int af_attention_tree(const float* q_dev, int64_t ldq, const void* k_cache, const void* k_scales, const void* v_cache,
                      const void* v_scales, int32_t kv_dtype, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                      int32_t ctx, int32_t n_past, int32_t n, const uint32_t* mask_dev, void* ws_dev, uint64_t ws_bytes,
                      float* out_dev, int64_t ldo, void* stream);

/*
 * A paged cache of many requests: a cache as af_kv_write's with ctx = n_pages * page_size slots, in which page p is the
 * slots p * page_size .. + page_size - 1 (of every kv head) and a request's tokens lie in the pages that its row of the
 * block table names, in order: the token at position t in slot table[t / page_size] * page_size + t % page_size.
 * af_kv_write and af_kv_read move its rows by those slots.
 *
 * af_kv_pages: one step of the loop that serves the requests, on the device, so that a captured step needs no host: slots
 * for the new tokens of all requests, pages for them from the free ones, and the pages of ended requests back.
 *   len_dev     int32 [n_seqs]: tokens that each request has in the cache
 *   new_dev     int32 [n_seqs]: tokens that the step adds to it; negative: the request has ended
 *   pool_dev    int32 [4]: head and count of the ring of free pages (two more are ignored)
 *   free_dev    int32 [n_pages]: the ring: free page i is free_dev[(head + i) % n_pages].  Pages are taken at the head, in
 *               the requests' order, and returned behind the last one
 *   table_dev   int32 [n_seqs][table_width]: the entries of pages taken are written, all others stay
 *   len_out_dev  int32 [n_seqs]: tokens after the step (ended: 0); may be len_dev
 *   pool_out_dev int32 [4]: the ring after the step, the number of requests refused, and the rows that the step wants; may
 *               be pool_dev
 *   start_dev   int32 [n_seqs + 1]: the batch's first row of each request, and the number of rows (2^31 - 1 for more)
 *   slots_dev, pos_dev, seq_dev  int32 [max_rows]: of each row (a request's new tokens in order, the requests in theirs)
 *               its slot, its position and its request; -1 in all three for the rows behind the last one and those of
 *               refused requests, which af_kv_write skips and af_attention_paged answers with zeros.  (A slot alone is -1
 *               where the table or the ring names no page of the cache.)
 * A request is refused, and stays as it is, if its length is negative or more than its table row holds, if the step would
 * make it so, if its rows do not end within max_rows, if it needs more pages than the requests before it (refused ones for
 * want of pages among them) have left, or if the ring has no room for the pages that it and those before it return.
 * A page belongs to one request; the ring never holds more than n_pages.  No entry of a page outside [0, n_pages) leads to
 * memory outside the cache, here or in af_attention_paged.
 *   ws_dev      scratch of af_kv_pages_workspace(n_seqs) bytes, 16-byte aligned, of any contents
 * 1 <= n_seqs <= 65536, 0 <= max_rows, page_size and table_width at least 1, n_pages * page_size and table_width *
 * page_size below 2^31 - 64.  Apart from the two pairs named, no two buffers overlap.  Asynchronous on `stream`, allocates
 * nothing, can be captured.  Errors: AF_EINVAL, AF_ERANGE, AF_ECUDA.
 */
uint64_t af_kv_pages_workspace(int32_t n_seqs);
int af_kv_pages(const int32_t* len_dev, const int32_t* new_dev, int32_t n_seqs, int32_t page_size, int32_t n_pages,
                const int32_t* pool_dev, int32_t* free_dev, int32_t* table_dev, int32_t table_width, int32_t* len_out_dev,
                int32_t* pool_out_dev, int32_t* start_dev, int32_t* slots_dev, int32_t* pos_dev, int32_t* seq_dev,
                int32_t max_rows, void* ws_dev, uint64_t ws_bytes, void* stream);

/*
 * Attention of single tokens over a paged cache (a decode step of many requests): row r of n attends to the positions
 * 0..pos_dev[r] of request seq_dev[r], its own among them (so its key and value are written first);
 * softmax(q K^T / sqrt(head_dim)) V, GQA group = n_heads / n_kv_heads.
 *   q_dev     fp32 [n] rows of n_heads * head_dim values (rotated), ldq apart
 *   cache     as af_kv_write's, with n_pages * page_size slots
 *   table_dev int32 [n_seqs][table_width], as af_kv_pages writes it
 *   seq_dev   int32 [n]: the table's row of each batch row, any order, the same one more than once if need be (several new
 *             tokens of a request are rows with positions of their own); NULL: row r is request r (n <= n_seqs)
 *   pos_dev   int32 [n].  A row with a negative position or a request outside [0, n_seqs) gives zeros; a position behind
 *             the table's last slot sees the slots that the table has.  Slots of pages outside [0, n_pages) are hidden: they
 *             are not read, and a row that sees no other slot gives zeros
 *   ws_dev    scratch of at least af_attention_paged_workspace bytes, 256-byte aligned, of any contents (6.4 MB with
 *             head_dim 128 on 152 SMs, whatever the rows); calls that may overlap in time need scratch of their own
 *   out_dev   fp32 [n] rows, ldo apart
 * The work is split by the slots that the rows see, found on the device: lengths may differ as they like, and a captured
 * call serves any lengths.  Precision, bits from call to call, and rows that see a NaN or an infinity: as
 * af_attention_tree's.  What slots hold that a row does not see reaches nothing.
 * 1 <= n <= 2048, 1 <= n_seqs <= 65536; head_dim 64 or 128, any whole group up to 64; n_kv_heads * n_pages * page_size below
 * 2^31, page_size and table_width at least 1, table_width * page_size below 2^31 - 64.  Pointers are 16-byte aligned
 * (table_dev, seq_dev, pos_dev: 4), ldq and ldo multiples of 4.  Asynchronous on `stream`, allocates nothing, can be captured
 * (the first call on a device loads the kernels: make it before a capture).  Errors: AF_EINVAL, AF_ERANGE, AF_ENOTIMPL, AF_ECUDA.
 */
uint64_t af_attention_paged_workspace(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim);
int af_attention_paged(const float* q_dev, int64_t ldq, const void* k_cache, const void* k_scales, const void* v_cache,
                       const void* v_scales, int32_t kv_dtype, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                       int32_t page_size, int32_t n_pages, const int32_t* table_dev, int32_t table_width, int32_t n_seqs,
                       const int32_t* seq_dev, const int32_t* pos_dev, int32_t n, void* ws_dev, uint64_t ws_bytes,
                       float* out_dev, int64_t ldo, void* stream);

/*
 * Low-rank adapters of many requests beside a shared projection (af_qgemm, af_qgemv): for row i of a batch, whose adapter
 * is a = ids_dev[i],   y_i = base_i + scale_a B_a (A_a x_i).
 * af_lora_plan puts the rows in the order of their adapters, once a step for all layers and projections:
 *   ids_dev   int32 [n]; a value outside [0, n_adapters) is a row without an adapter
 *   plan_dev  af_lora_plan_bytes(n, n_adapters) bytes, 16-byte aligned
 * af_lora, with the n and n_adapters of its plan (a plan of others, in a buffer of this call's size, gives rows of NaN):
 *   x_dev     fp32 [n] rows of K values, ldx apart
 *   a_dev     [n_adapters][rank][K], b_dev [n_adapters][N][rank] of dtype AF_F16 or AF_F32
 *   scale_dev fp32 [n_adapters]; NULL: 1
 *   rank_dev  int32 [n_adapters]: ranks of adapters that have fewer than `rank` (taken into [0, rank]); what lies behind
 *             them in a_dev and b_dev reaches nothing.  NULL: all have `rank`
 *   base_dev  fp32 [n] rows of N values, ldb apart: the projection's; may be y_dev with ldb == ldy, and overlaps it in no
 *             other way; NULL: zeros
 *   y_dev     fp32 [n] rows, ldy apart.  Rows without an adapter are the base's.  (May overlap x_dev, which is read first)
 *   ws_dev    scratch of af_lora_workspace(n, n_adapters, rank, K, N) bytes, 256-byte aligned, of any contents; calls that
 *             may overlap in time need scratch of their own
 * Precision: x, fp32 weights and A x keep 2^-22 of each value, or 2^-38 of the largest of 32 neighbours along K or the rank (of
 * a row of A x; 2^-150 where that is more still); sums are fp32's.  Where a value of the formula is not finite (a NaN or an infinity in a
 * row of x, in A for all rows of its adapter, in a row of B for their values of that column), or a sum leaves fp32's range, the
 * result is NaN or an infinity; no other row or value is touched.  A row's result depends on the other rows only through the
 * order in which K's sums are joined; its bits do not change from call to call with the same plan.
 * 1 <= n <= 65536, 1 <= n_adapters <= 4096; rank a multiple of 8 up to 128 (pad with rank_dev); K a multiple of 32, N any,
 * both up to 2^24.
 * x_dev, a_dev, b_dev are 16-byte aligned and ldx a multiple of 4; base_dev and y_dev 4-byte aligned (vectors of 16 bytes
 * are moved where they, N, ldb and ldy allow it).  Asynchronous on `stream`, allocate nothing, can be captured (the first
 * call on a device loads the kernels: make it before a capture).  Errors: AF_EINVAL, AF_ERANGE, AF_ENOTIMPL, AF_ECUDA.
 */
uint64_t af_lora_plan_bytes(int32_t n, int32_t n_adapters);
int af_lora_plan(const int32_t* ids_dev, int32_t n, int32_t n_adapters, void* plan_dev, uint64_t plan_bytes, void* stream);
uint64_t af_lora_workspace(int32_t n, int32_t n_adapters, int32_t rank, int32_t K, int32_t N);
int af_lora(const float* x_dev, int64_t ldx, int32_t n, const void* plan_dev, const void* a_dev, const void* b_dev,
            int32_t dtype, const float* scale_dev, const int32_t* rank_dev, int32_t n_adapters, int32_t rank, int32_t K,
            int32_t N, const float* base_dev, int64_t ldb, float* y_dev, int64_t ldy, void* ws_dev, uint64_t ws_bytes,
            void* stream);

/* Thread-local message for the last failed call on this thread ("" if none). */
const char* af_last_error(void);

#ifdef __cplusplus
}
#endif
#endif
