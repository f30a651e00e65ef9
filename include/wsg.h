/*
 * wsg.h - C ABI of the weight-streaming decode library (GB300, sm_103a).
 *
 * The library computes the batch-1 token-to-logits forward of a
 * Qwen3-shaped decoder and the standalone matrix-vector products that
 * dominate it. All arithmetic runs in this library's CUDA kernels.
 *
 * Sources (page title, section):
 *   "Megakernels", "What runs in the DSL": the forward pass
 *       token ID -> embedding; per layer RMSNorm -> Q/K/V projections ->
 *       per-head Q/K RMSNorm -> RoPE -> grouped-query attention + KV update
 *       -> output projection -> residual add -> RMSNorm -> gate/up
 *       projections -> SwiGLU -> down projection -> residual add; then final
 *       RMSNorm -> tied vocabulary projection -> logits.
 *   "Megakernels", "GPU-wide end-to-end generation": greedy argmax on the
 *       GPU with ties broken by lowest token ID; the host reads the ID;
 *       prompt tokens processed one at a time skip only the final norm and
 *       vocabulary projection; the first output comes from the final prompt
 *       row.
 *   "Megakernels", "Chunked prefill for long prompts": a chunk is a run of
 *       consecutive positions of the single request; every row attends to
 *       its whole causal prefix; only the final valid row reaches the
 *       vocabulary projection.
 *   "Our Kernel Benchmark Was Measuring the System Cache", "Summary": the
 *       4-bit matrix-vector product and its two-token variant.
 *
 * Conventions for every call:
 *   - Pointers named d_* are device pointers, h_* host pointers. All device
 *     memory belongs to the caller; the library never frees it.
 *   - `stream` is a cudaStream_t passed as void*; NULL means the legacy
 *     default stream. Calls are asynchronous on that stream unless stated.
 *   - Every call returns a dec_status. On failure nothing has been enqueued
 *     and dec_last_error() describes the cause. No call aborts the process.
 *   - Device-side problems that can only be seen while kernels run (a token
 *     ID outside the vocabulary, an all-NaN logit vector, a bounded wait
 *     that gave up) set bits of a device error word, read with
 *     dec_device_errors() or gemv_device_errors().
 */
#ifndef WSG_H
#define WSG_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  DEC_OK = 0,
  DEC_EINVAL = 1,     /* bad argument: NULL, size, alignment, dtype */
  DEC_ESTATE = 2,     /* call out of order (e.g. step before weights) */
  DEC_ECAPACITY = 3,  /* position or chunk beyond the configured capacity */
  DEC_ENOMEM = 4,     /* workspace too small, or a host allocation failed */
  DEC_ECUDA = 5,      /* a CUDA runtime call failed (message has the name) */
  DEC_EDEVICE = 6     /* device is not an sm_103 GPU */
} dec_status;

typedef enum { DEC_F32 = 0, DEC_BF16 = 1, DEC_Q4G64 = 2 } dec_dtype;

/* Device error bits (dec_device_errors / gemv_device_errors). */
#define DEC_DEVERR_WAIT_TIMEOUT 0x1u /* a bounded mbarrier wait gave up */
#define DEC_DEVERR_ARGMAX_NAN 0x2u   /* all logits NaN; token 0 was returned */
#define DEC_DEVERR_BAD_TOKEN 0x4u    /* a token ID outside [0, vocab) was read as 0 */
#define DEC_DEVERR_BAD_POSITION 0x8u /* a position reached the KV capacity; the step did nothing */
#define DEC_DEVERR_EXCHANGE_TIMEOUT 0x10u /* persistent engine: a wait for another CTA's words gave up */
#define DEC_DEVERR_GEMM_TIMEOUT 0x20u     /* chunked prefill, attn_shared_prefix, attn_tree_paged: a tensor-core pipeline wait gave up */
#define DEC_DEVERR_BARRIER_TIMEOUT 0x40u  /* persistent 4-bit engine: a grid barrier gave up (dec_reset clears it) */
#define DEC_DEVERR_BAD_PAGE 0x80u         /* a sequence, page or parent index of the paged calls was out of range */
#define DEC_DEVERR_BAD_TREE 0x100u        /* a drafted row's parent is not an earlier row of its request, or a tree has more rows than its mask */

/* dec_config.engine */
#define DEC_ENGINE_PERSISTENT 0 /* one cooperative launch runs whole forwards (default) */
#define DEC_ENGINE_STAGED 1     /* five kernels per layer, replayed as a CUDA graph */

/* dec_step flags */
#define DEC_SKIP_LOGITS 0x1u /* body only: no final norm, vocabulary projection or argmax */

/* Decoder geometry and storage ("Megakernels", "What runs in the DSL").
 * Requirements: layers, hidden, inter, n_q, n_kv, head_dim, vocab > 0;
 * n_q % n_kv == 0; head_dim a multiple of 8 and <= 128; hidden, inter and
 * n_q*head_dim multiples of 8; wdtype DEC_F32, DEC_BF16 or DEC_Q4G64 (the
 * 4-bit configuration: chunk_cap 0, hidden, inter and n_q*head_dim
 * multiples of 512 up to 16384; its persistent engine separates stages
 * with grid barriers, and its staged engine is the faster of the two);
 * kvdtype DEC_F32
 * or DEC_BF16; max_seq >= 1 is the KV capacity in positions; chunk_cap is
 * the largest row count of one dec_prefill_chunk call that runs batched
 * (0: prompts are processed one token at a time). engine selects the
 * execution of decode steps: DEC_ENGINE_PERSISTENT runs each call's forwards
 * inside one persistent kernel (one CTA per SM, a producer warp streaming
 * weights through shared memory ahead of the consumers, grid barriers
 * between dependent stages); DEC_ENGINE_STAGED launches the per-stage
 * kernels as a CUDA graph. Both compute the same forward. Decode attention
 * at position p splits the p + 1 cached keys of each key/value head into
 * nsplit = min(ceil((p + 1) / 64), min(64, SMs / n_kv)) key-parallel ranges
 * of ceil((p + 1) / nsplit) keys (the last one shorter), whose partial
 * softmax sums are merged in split order. */
typedef struct {
  int32_t layers, hidden, inter, n_q, n_kv, head_dim, vocab;
  float eps;        /* RMSNorm epsilon, e.g. 1e-6 */
  float rope_theta; /* RoPE base, e.g. 1e6 */
  int32_t wdtype;   /* dec_dtype of projections and the tied embedding */
  int32_t kvdtype;  /* dec_dtype of the KV cache */
  int32_t max_seq;
  int32_t chunk_cap;
  int32_t engine;   /* DEC_ENGINE_*: how steps are executed */
} dec_config;

/* One layer's tensors, device pointers, row-major [out][in] in wdtype.
 * With DEC_Q4G64 each matrix pointer (and embed) points at one buffer
 * holding the codes [out][in/8] uint32 (code j of word w at bits
 * [4j, 4j+4), column 8w+j), then the scales and then the biases
 * [out][in/64] fp16: w = s * q + b per 64-column group.
 * w_q [n_q*head_dim][hidden], w_k and w_v [n_kv*head_dim][hidden],
 * w_o [hidden][n_q*head_dim], w_gate and w_up [inter][hidden],
 * w_down [hidden][inter]; gains are float32: g_in and g_post [hidden],
 * g_q and g_k [head_dim] (one per layer, shared by all heads). Every
 * pointer must be 16-byte aligned. */
typedef struct {
  const void *w_q, *w_k, *w_v, *w_o, *w_gate, *w_up, *w_down;
  const float *g_in, *g_post, *g_q, *g_k;
} dec_layer_weights;

/* embed: [vocab][hidden] in wdtype, also the vocabulary head (tied).
 * layers: HOST array of cfg.layers entries (copied by dec_load_weights). */
typedef struct {
  const void* embed;
  const float* g_final;
  const dec_layer_weights* layers;
} dec_weights;

typedef struct dec_ctx dec_ctx;

/* Bytes of device workspace dec_create needs for cfg (KV cache, rotary
 * table, activations, argmax and attention partials, prefill scratch).
 * The cache holds keys and values in the selected dtype ("Megakernels",
 * "What runs in the DSL"), sized for max_seq positions, i.e. the P + N - 1
 * entries a generation leaves ("GPU-wide end-to-end generation").
 * Returns 0 if cfg is invalid. */
size_t dec_workspace_bytes(const dec_config* cfg);

/* Creates a decoder on the current CUDA device ("Megakernels", "What runs
 * in the DSL": the host precomputes the rotary constants once, before any
 * forward). d_workspace (>= 256-byte aligned, at least
 * dec_workspace_bytes(cfg) bytes) must stay allocated until dec_destroy.
 * Builds the rotary table and clears the cache; returns after that work has
 * finished. stream: the stream later calls run on.
 * Errors: DEC_EINVAL (cfg, NULL, alignment), DEC_ENOMEM (workspace too
 * small), DEC_EDEVICE (not sm_103), DEC_ECUDA. */
dec_status dec_create(const dec_config* cfg, void* d_workspace, size_t workspace_bytes, void* stream,
                      dec_ctx** out);

/* Registers the caller's weight tensors ("Megakernels", "What runs in the
 * DSL": the projections, norm gains and the tied embedding of the forward;
 * no copy: they must outlive the context). Errors: DEC_EINVAL on a NULL or
 * misaligned pointer, DEC_ECUDA. */
dec_status dec_load_weights(dec_ctx* ctx, const dec_weights* w);

/* Position back to 0 and every cache entry invalidated (the cache is
 * zeroed). Timed by the pages' protocol ("Benchmark methodology",
 * "Long-document chunked prefill": timing starts before cache reset). */
dec_status dec_reset(dec_ctx* ctx);

/* Moves the position back to pos (0 <= pos <= current position): cache
 * entries 0..pos-1 stay valid, the next forward runs at position pos and
 * overwrites slot pos. This is how a fixed-context timing trial repeats one
 * token at a fixed cache slot ("Megakernels", "Fixed-context methodology").
 * Asynchronous on the context's stream. Errors: DEC_EINVAL (NULL, pos
 * outside [0, position]), DEC_ECUDA. */
dec_status dec_rewind(dec_ctx* ctx, int32_t pos);

/* One forward of `token` at the current position p ("Megakernels", "What
 * runs in the DSL" for the forward; "GPU-wide end-to-end generation" for the
 * greedy argmax with lowest-ID ties and the host reading the token ID);
 * writes K/V at p and advances the position to p+1.
 * Without DEC_SKIP_LOGITS: final RMSNorm, tied vocabulary projection and
 * argmax (lowest ID on ties) run too. d_logits (nullable, float32[vocab])
 * receives the logits; h_next (nullable) receives the greedy token, and
 * then the call synchronizes the stream to read it. On the persistent engine
 * the token is passed with the launch and the greedy token is written by the
 * kernel into mapped page-locked host memory (no copy calls per step).
 * With DEC_SKIP_LOGITS: only the body runs; d_logits and h_next must be NULL.
 * Errors: DEC_ESTATE (no weights), DEC_ECAPACITY (p == max_seq),
 * DEC_EINVAL (token outside [0, vocab), bad flags). */
dec_status dec_step(dec_ctx* ctx, int32_t token, uint32_t flags, float* d_logits, int32_t* h_next);

/* Two-token verify step of the 4-bit configuration (cfg.wdtype ==
 * DEC_Q4G64): one forward of h_tokens[0] at position p and h_tokens[1] at
 * p+1, where row 1 attends to row 0's cache entry, both through the final
 * norm, the vocabulary projection and the argmax; every projection runs the
 * two-token 4-bit matrix-vector product ("Our Kernel Benchmark Was Measuring
 * the System Cache", Summary: the 4-bit matvec and its two-token variant,
 * the shape of checking a drafted token). d_logits (nullable) receives
 * float32[2][vocab]; h_next (nullable) receives int32[2], the greedy token
 * after each row, and then the call synchronizes the stream to read them.
 * Writes cache entries p and p+1 and advances the position to p+2; the
 * token stream holds h_next[1] at p+2. A caller whose draft h_tokens[1]
 * differs from h_next[0] rewinds to p+1 (dec_rewind) and continues from
 * h_next[0].
 * Errors: DEC_EINVAL (NULL, token outside [0, vocab), not the 4-bit
 * configuration), DEC_ESTATE (no weights), DEC_ECAPACITY (p + 2 > max_seq). */
dec_status dec_verify2(dec_ctx* ctx, const int32_t* h_tokens, float* d_logits, int32_t* h_next);

/* Prompt rows h_tokens[0..n) at positions p..p+n-1 ("Chunked prefill for
 * long prompts"). If cfg.chunk_cap > 0 and n <= chunk_cap the rows run
 * batched (tensor-core projections, causal attention over cache + chunk);
 * otherwise, or with chunk_cap == 0, one token at a time.
 * is_last != 0: the final row also runs the final norm, the vocabulary
 * projection and the argmax; d_logits / h_next as in dec_step (h_next
 * synchronizes). is_last == 0: d_logits and h_next must be NULL.
 * Errors: DEC_EINVAL (n < 1, token out of range), DEC_ECAPACITY
 * (p + n > max_seq), DEC_ESTATE. */
dec_status dec_prefill_chunk(dec_ctx* ctx, const int32_t* h_tokens, int32_t n, int32_t is_last, float* d_logits,
                             int32_t* h_next);

/* n greedy forwards without host involvement ("Megakernels", "GPU-wide
 * end-to-end generation": token IDs in, generated IDs out, the cache
 * advancing by one entry per forward and the next token chosen on the GPU
 * by the lowest-ID argmax; there the host reads each ID before the next
 * forward, here the ID stays on the device): the first input is `token` at
 * the current position, each later input is the previous output. Writes
 * the n outputs to d_tokens_out (device int32[n]). Asynchronous.
 * Errors: DEC_ECAPACITY (p + n > max_seq), DEC_EINVAL, DEC_ESTATE. */
dec_status dec_generate(dec_ctx* ctx, int32_t token, int32_t n, int32_t* d_tokens_out);

/* Read access to one layer's cache ("Benchmark methodology", "Long-document
 * chunked prefill": validation checks every valid K/V entry of every layer):
 * device pointers to K and V, each laid out [n_kv][max_seq][head_dim] in
 * kvdtype, and the number of valid positions. Keys are stored after Q/K-norm
 * and RoPE, values raw. Errors: DEC_EINVAL (NULL, layer out of range). */
dec_status dec_get_kv(const dec_ctx* ctx, int32_t layer, const void** d_k, const void** d_v, int32_t* n_valid);

/* Current position (number of valid cache entries; after a P-token prompt
 * and N outputs it is P + N - 1, the count "Megakernels", "GPU-wide
 * end-to-end generation" validates). -1 if ctx is NULL. */
int32_t dec_position(const dec_ctx* ctx);

/* Stage tracing of the persistent engines. The pages give no tracing API;
 * "Our Kernel Benchmark Was Measuring the System Cache", "Key takeaways",
 * warns that a synchronizing profiler only bounds a kernel's time from
 * below, so the engines stamp their own stages on the device instead.
 * dec_trace_bytes: size of the trace buffer (0 for the staged engine). dec_set_trace: with a non-NULL
 * device buffer of at least that size, every later persistent launch writes,
 * for its first forward, one %globaltimer stamp (nanoseconds) per
 * [cta][layer 0..layers][stage 0..4][event 0..3] as uint64. Stages 0-4 of a
 * layer are QKV, attention, O, gate/up, down; the extra layer index `layers`
 * holds the head (stage 0: vocabulary GEMV, stage 1 event 0: argmax done).
 * Float engine events: 0 stage entry, 1 inputs received and staged (includes
 * waiting for the producing stage), 2 outputs published, 3 every warp done
 * with the stage's weight boxes (attention: key loop done). 4-bit engine
 * events: 0 stage entry, 1 input vector staged in fixed point, 2 products
 * (attention: the attention body) done, 3 the grid barrier after the stage
 * passed; its head has events 0-2 of stage 0 only. After that block, [8][512][4] uint64 for each consumer warp of
 * CTA 0 and the first 512 weight boxes it consumes in the launch: SM clock
 * stamps (clock64) when the box's wait begins, when its data is ready and
 * when its dot products are issued, then the %globaltimer stamp of the wait's
 * beginning. NULL turns tracing off. */
size_t dec_trace_bytes(const dec_ctx* ctx);
dec_status dec_set_trace(dec_ctx* ctx, uint64_t* d_trace, size_t bytes);

/* Limit, in nanoseconds, of every wait of the persistent engines on another
 * CTA's results (exchange words, appended-row counts, grid barriers); 0
 * restores the default of 2 s. The pages give no API for this: the forward
 * runs as ordered stages with no host waits between them ("Megakernels",
 * "GPU-wide end-to-end generation"), so such waits are where a broken
 * launch would otherwise stall. A wait that runs out makes the launch give
 * up: the kernel sets DEC_DEVERR_EXCHANGE_TIMEOUT (float engine) or
 * DEC_DEVERR_BARRIER_TIMEOUT (4-bit engine), waits for its own copies in
 * flight (those waits keep a fixed 2 s limit) and returns; that call's
 * outputs, tokens and cache entries are then undefined, and dec_reset
 * restores a usable state. A limit of a few microseconds makes ordinary
 * forwards give up, which is how the tests exercise that path. The staged
 * engine has no such waits. Takes effect at the next launch.
 * Errors: DEC_EINVAL (NULL). */
dec_status dec_set_wait_limit(dec_ctx* ctx, uint64_t ns);

/* Synchronizes the context's stream and returns (and, if clear != 0,
 * clears) the device error bits DEC_DEVERR_* listed above, among them an
 * all-NaN logit vector at the argmax (the lowest-ID argmax of "Megakernels",
 * "GPU-wide end-to-end generation" has no answer there) and waits that gave
 * up. A set bit marks the affected call's outputs as invalid, as a failed check
 * invalidates a run in "Benchmark methodology", "Long-document chunked
 * prefill". Errors: DEC_EINVAL (NULL), DEC_ECUDA. */
dec_status dec_device_errors(dec_ctx* ctx, int32_t clear, uint32_t* bits);

/* Frees host-side state and CUDA graphs. The workspace stays the caller's
 * (the pages give no API; this is the counterpart of dec_create, which
 * follows "Megakernels", "What runs in the DSL"). */
void dec_destroy(dec_ctx* ctx);

/* Message for the last failed call on ctx (ctx == NULL: last failure of a
 * context-free call on this thread). Never NULL. The pages give no API; the
 * calls above report every failure with a status and this message instead
 * of aborting or continuing silently ("Benchmark methodology", "Long-document
 * chunked prefill": a failed check discards the whole run rather than
 * leaving a partial result that looks successful). */
const char* dec_last_error(const dec_ctx* ctx);

/* y = W x ("Our Kernel Benchmark Was Measuring the System Cache":
 * the matrix-vector product of the decode step).
 * wdtype DEC_F32: W float32 [out][in], x float32 [in];
 * wdtype DEC_BF16: W bfloat16 [out][in], x bfloat16 [in].
 * y float32 [out]; products accumulated in float32, partial sums reduced
 * in a fixed order (bit-reproducible). out, in >= 0 (out == 0: no work;
 * in == 0: y = 0). Any alignment is accepted; 16-byte aligned W with
 * in*sizeof(elem) a multiple of 16 takes the bulk-copy streaming path.
 * Ordering: the call is a programmatic dependent of the previous kernel on
 * `stream` and starts streaming W before that kernel has finished (x and y
 * only after), so W, a weight matrix, must not be written by the kernel
 * enqueued immediately before the call; anything earlier is ordered.
 * Errors: DEC_EINVAL, DEC_ECUDA. */
dec_status gemv(int32_t wdtype, const void* d_W, const void* d_x, float* d_y, int32_t out, int32_t in, void* stream);

/* y[t] = W x[t] for a 4-bit groupwise-affine W ("Our Kernel Benchmark Was
 * Measuring the System Cache", Summary and "Why it mattered, concretely":
 * the one-token matvec and the two-token variant). Each group of 64
 * consecutive columns of a row has an fp16 scale s and bias b, and
 * w = s*q + b for the 4-bit code q.
 * d_codes: uint32 [out][in/8], code j of word w in bits [4j, 4j+4), column
 * 8w+j; d_scale, d_bias: fp16 bits [out][in/64]; d_x: bfloat16 [ntok][in];
 * d_y: float32 [ntok][out]. ntok is 1 or 2; in % 64 == 0; d_codes 16-byte
 * aligned. With in % 512 == 0 (in <= 16384) and 16-byte aligned scales,
 * biases and x, the bulk-copy kernel runs: integer dot products of the codes
 * with x in 16-bit fixed point per 32 columns (step a power of two, error at
 * most 2^-15 of the 32 columns' largest |x|), float32 sums per row, fixed
 * order. Otherwise a per-warp kernel dequantises to float32. Both are
 * bit-reproducible. Like gemv, the call may start reading the codes, scales
 * and biases before the previous kernel on `stream` has finished (x and y
 * only after it): they must not be written by the kernel enqueued
 * immediately before the call. Errors: DEC_EINVAL, DEC_ECUDA. */
dec_status gemv_q4(const uint32_t* d_codes, const uint16_t* d_scale, const uint16_t* d_bias, const uint16_t* d_x,
                   float* d_y, int32_t out, int32_t in, int32_t ntok, void* stream);

/* Rows of W each warp of gemv_q4 handles per pass (1, 2, 4 or 8), for the
 * given ntok ("Our Kernel Benchmark Was Measuring the System Cache", "Why it
 * mattered, concretely": tuned on the cold number). r > 0 sets it, r == -1
 * returns to the automatic choice (the default: 1 when out <= 8 x the SM
 * count, else 4), r == 0 only reads it. Returns the setting in effect (0:
 * automatic), or -1 for a bad argument. Process-wide. */
int32_t gemv_q4_rows_per_warp(int32_t ntok, int32_t r);

/* Lossless bfloat16 storage of float32 weights ("Megakernels", "Lossless
 * decode-weight storage"): d_dst[i] = high 16 bits of d_src[i] for n
 * elements (device pointers, any alignment), and *h_bad (host) = how many
 * elements that storage does not hold exactly (low 16 bits non-zero, or not
 * finite). With *h_bad == 0 the bfloat16 copy widens back to the same
 * float32 bits, so a decoder created with wdtype DEC_BF16 over such copies
 * computes the float32 model's forward on half the weight bytes. Runs on
 * `stream` and synchronizes it to read the count. Calls on one device must
 * not overlap (they share the count). Errors: DEC_EINVAL, DEC_ECUDA. */
dec_status pack_bf16_exact(const float* d_src, uint16_t* d_dst, int64_t n, void* stream, int64_t* h_bad);

/* Reads (and if clear != 0 clears) the device error bits of the
 * context-free calls (gemv, gemv_q4, gemm_bf16, greedy_head_noalloc) on the
 * current device; synchronizes the device. The bits mean what they mean for
 * dec_device_errors (the argmax rule of "Megakernels", "GPU-wide end-to-end
 * generation"; bounded waits that gave up). Errors: DEC_EINVAL (NULL),
 * DEC_ECUDA. */
dec_status gemv_device_errors(int32_t clear, uint32_t* bits);

/* Greedy head for callers that cannot allocate device memory. The operation
 * is the decode step's head: the final RMSNorm and tied vocabulary
 * projection of "Megakernels", "What runs in the DSL", then the lowest-ID
 * argmax of "GPU-wide end-to-end generation"; the pages have no entry point
 * that runs it alone without allocating. Some callers cannot call cudaMalloc: code
 * running inside a host framework that owns every device allocation, or a
 * generation loop that must not risk the device synchronisation an
 * allocation can cause. This call computes x = RMSNorm(h) * gain (eps as
 * given), logits = E x and the greedy token (lowest ID among equal maxima)
 * with the same kernel as the decoder's head, but keeps that kernel's
 * scratch (per-CTA argmax partials, a counter, a position word) in a
 * fixed 8448-byte device array inside the library instead of a workspace.
 * wdtype DEC_F32 or DEC_BF16: d_embed [vocab][hidden] in that dtype (16-byte
 * aligned, rows a multiple of 16 bytes); d_h and d_gain float32 [hidden];
 * d_logits float32 [vocab] or NULL; d_token receives the int32 token.
 * Limits: at most 1024 CTAs of argmax partials (vocab x hidden beyond that is
 * rejected with DEC_EINVAL) and hidden small enough for the shared-memory
 * staging (DEC_EINVAL beyond it). The array persists on every device that
 * loaded the library until exit and is shared by all calls: calls that
 * overlap on the GPU (other streams, other threads) race on it and must be
 * serialised by the caller. The first call on a device looks up the array's
 * address and sets the kernel's shared-memory limit (under a lock, so first
 * calls from several host threads are safe); make that first call before any
 * stream capture. Device-side errors of the call (an all-NaN logit vector,
 * which returns token 0; a bounded wait that gave up) set bits of the
 * context-free error word that gemv_device_errors reads and clears.
 * Allocates nothing (no cudaMalloc, cudaFree or allocating library routine).
 * Errors: DEC_EINVAL, DEC_EDEVICE, DEC_ECUDA. */
dec_status greedy_head_noalloc(int32_t wdtype, const void* d_embed, const float* d_h, const float* d_gain, float eps,
                               int32_t vocab, int32_t hidden, float* d_logits, int32_t* d_token, void* stream);

/* Chunked-prefill projection GEMM as a standalone call ("Megakernels",
 * "Chunked prefill for long prompts": a chunk of prompt rows turns each
 * projection into a dense matrix product, run on the tensor cores):
 * C[m][n] = sum_k A[m][k] * W[n][k] for m < M, n < N (accumulate != 0:
 * C[m][n] += that sum). A [M][K] and W [N][K] are bfloat16, row-major,
 * 16-byte aligned (W is a weight matrix in the decoder's [out][in] layout);
 * C is float32 with row stride ldc >= N. Products are exact in FP32 and
 * accumulated in FP32 (tcgen05 tensor cores; 128-row tiles 256, 128 or 64
 * columns wide, chosen per call by the operand bytes the busiest SM
 * streams). K must be a multiple of 8. Asynchronous on `stream`; like gemv
 * the call may start reading W before the previous kernel on `stream` has
 * finished (A and C only after it), so W must not be written by the kernel
 * enqueued immediately before it. Device errors (a bounded wait that gave
 * up) are reported by gemv_device_errors.
 * Errors: DEC_EINVAL (sizes, alignment), DEC_EDEVICE, DEC_ECUDA. */
dec_status gemm_bf16(const uint16_t* d_A, const uint16_t* d_W, float* d_C, int32_t M, int32_t N, int32_t K,
                     int32_t ldc, int32_t accumulate, void* stream);

/* ---- Branches of one prompt ------------------------------------------------
 *
 * The calls below decode several continuations of ONE prefilled prompt
 * together. The prompt's keys and values stay where dec_prefill_chunk put
 * them (dec_get_kv: [n_kv][max_seq][head_dim]) and are shared by every
 * branch; each branch keeps its own later tokens in pages. A step of all
 * branches: kv_append_paged (per-head Q/K norm and rotation, new keys and
 * values into the pages), attn_shared_prefix, and after the vocabulary
 * projection beam_select and beam_reorder_pages. qk_norm_rope is the norm and
 * rotation alone. The sources decode a single stream; these calls
 * extend "Megakernels", "What runs in the DSL" (per-head Q/K RMSNorm, RoPE,
 * grouped-query attention and KV update) and "GPU-wide end-to-end generation"
 * (lowest-ID selection on the GPU) to several.
 *
 * Pools and tables: k_pages and v_pages are [num_pages][n_kv][page_size]
 * [head_dim] in kvdtype, 16-byte aligned; page_size is a power of two up to
 * 1024. Row b of page_table ([.][table_stride] int32) lists the pages of
 * sequence b in order: its token i lies in page table[b][i / page_size], row
 * i % page_size. A table entry that a call needs and that is outside
 * [0, num_pages) sets DEC_DEVERR_BAD_PAGE in the context-free error word
 * (gemv_device_errors) and the rows behind it are left out (not stored, not
 * attended to); nothing outside the pools is read or written.
 *
 * All of them take their arguments in a struct, are asynchronous on `stream`
 * (the struct may be reused once the call returns; the buffers when the work
 * is done), allocate nothing and can be captured into a graph; the first call
 * of each kind on a device sets its kernels up and must come before any stream
 * capture. Calls that share a workspace or write the same buffers must be
 * ordered by the caller (one stream, or events); a workspace needs no
 * initialisation and holds nothing between calls. Every pointer must belong to
 * the current device. Each call is a programmatic dependent of the stream's
 * previous kernel and reads nothing before that kernel has finished.
 * Common errors: DEC_EINVAL (NULL struct, sizes, dtype, NULL or misaligned
 * pointers), DEC_EDEVICE, DEC_ECUDA. */

/* Frequencies of the position rotation, angle = position * inv_freq[i] for
 * pair i of rot_dim / 2, from inv_freq[i] = theta^(-2i / rot_dim):
 * ROPE_LINEAR divides all of them by `factor` (positions interpolated);
 * ROPE_BASE stretches the base, theta * factor^(rot_dim / (rot_dim - 2)), so
 * that the slowest pair is divided by factor and the fastest kept;
 * ROPE_RAMP keeps the pairs that turn at least beta_fast times in
 * orig_context positions, divides those that turn at most beta_slow times by
 * factor, blends linearly in the number of turns between them, and gives
 * cosine and sine the factor 0.1 ln(factor) + 1 (the published YaRN rule);
 * the other kinds give 1. */
enum { ROPE_PLAIN = 0, ROPE_LINEAR = 1, ROPE_BASE = 2, ROPE_RAMP = 3 };

typedef struct {
  int32_t rot_dim; /* even, 2..128 */
  int32_t kind;    /* ROPE_* */
  double theta;    /* > 0, e.g. 1e6 */
  double factor;   /* >= 1 (unused by ROPE_PLAIN) */
  double orig_context, beta_slow, beta_fast; /* ROPE_RAMP: > 0, beta_slow < beta_fast, e.g. 32768, 1, 32 */
} rope_scaling;

/* Fills h_inv_freq (HOST, rot_dim / 2 doubles) and *h_factor (HOST). Runs on
 * the host only ("Megakernels", "What runs in the DSL": the host precomputes
 * the rotary constants once). Errors: DEC_EINVAL. */
dec_status rope_frequencies(const rope_scaling* s, double* h_inv_freq, float* h_factor);

/* rows x (n_q + n_kv) heads of head_dim (a multiple of 8 up to 128); row r of
 * q starts at q + r * q_stride elements and holds n_q heads side by side, k
 * likewise with n_kv. Each head is RMS-normalised over head_dim (skipped where
 * its gain is NULL), y = x / sqrt(mean(x^2) + eps) * g, and its first rot_dim
 * elements are rotated: pairs (i, i + rot_dim / 2), or (2i, 2i + 1) with
 * interleaved != 0, by positions[r] * inv_freq[i], cosine and sine times
 * rope_factor. rot_dim 0: no rotation. The arithmetic is float32 (angles are
 * reduced exactly, so far positions lose nothing) and each output is rounded
 * once. positions[r] < 0 marks a padded row: its outputs are left as they
 * were. q_out may be q itself (same dtype and stride), k_out likewise; outputs
 * must not overlap inputs in any other way. */
typedef struct {
  int32_t rows, n_q, n_kv, head_dim; /* n_q or n_kv may be 0; each at most 16384 */
  int32_t xdtype, ydtype;            /* q, k; q_out, k_out: DEC_F32 or DEC_BF16 */
  const void *q, *k;
  void *q_out, *k_out;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;
  const float *g_q, *g_k; /* [head_dim] or NULL */
  const int32_t* positions;
  const double* inv_freq; /* device, [rot_dim / 2] */
  float eps, rope_factor;
  int32_t rot_dim, interleaved;
} qk_rope_args;

/* Per-head Q/K RMSNorm and RoPE of "Megakernels", "What runs in the DSL", as a
 * call of its own. */
dec_status qk_norm_rope(const qk_rope_args* a, void* stream);

/* qk_norm_rope whose keys, with the values v beside them, go to pages: row r
 * is the token at positions[r] of sequence seq[r], stored at index
 * positions[r] - base_pos of that sequence's pages (base_pos: the tokens of
 * the shared prefix, which are not in pages). Keys are stored normalised and
 * rotated, values as they are, both rounded once to kvdtype. seq NULL: row r
 * belongs to sequence r. A padded row (positions[r] < 0) stores nothing and
 * leaves its q_out as it was. A seq[r] outside [0, n_seq) or an index outside
 * the table's width counts as a bad page; the row's q_out is still written.
 * Two rows at the same index of one sequence leave a mixture of both there. */
typedef struct {
  int32_t rows, n_q, n_kv, head_dim; /* n_q may be 0 */
  int32_t xdtype, ydtype, kvdtype;   /* q, k, v; q_out; pages */
  const void *q, *k, *v;
  void* q_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  const float *g_q, *g_k;
  const int32_t* positions;
  const double* inv_freq;
  float eps, rope_factor;
  int32_t rot_dim, interleaved;
  void *k_pages, *v_pages;
  const int32_t* page_table;
  const int32_t* seq;
  int32_t n_seq, num_pages, page_size, table_stride, base_pos;
} kv_append_args;

/* "Megakernels", "What runs in the DSL": norm, RoPE and KV update, here into
 * pages. */
dec_status kv_append_paged(const kv_append_args* a, void* stream);

/* Grouped-query attention of one query token for each of `batch` branches over
 * the shared prefix followed by the branch's own paged tokens:
 * out[b][h] = softmax(scale * q[b][h] . [Kp; Ks]) [Vp; Vs], query head h on
 * key/value head h / (n_q / n_kv). The prefix is prefix_len keys and values a
 * head, head g at prefix_k + g * prefix_stride * head_dim elements (the layout
 * of dec_get_kv with prefix_stride = max_seq), kvdtype like the pages; rows
 * past prefix_len are never used, whatever they hold. It is read once for all
 * branches. seq_len[b] is the number of the branch's own tokens (more than
 * table_stride * page_size counts as a bad page); seq_len[b] < 0 marks an
 * unused slot, whose out and lse are left as they were. A branch with nothing
 * to attend to gets zeros (and lse -inf). lse (nullable, float32
 * [batch][n_q]) receives the natural log of the softmax's denominator.
 * n_q / n_kv <= 16, batch * n_q < 2^24, prefix_len + table_stride * page_size
 * <= 2^30. A key or value that is not finite and attended to makes its rows
 * not finite, except that a score of -inf may have weight 0. Scores, softmax
 * sums and outputs are accumulated in float32; with DEC_BF16 q and out the
 * result is rounded once to bfloat16. What enters the products: bfloat16 as it
 * is; float32 queries over a bfloat16 cache and their probabilities in 24 bits;
 * the probabilities of bfloat16 queries in 16 (2^-16 of each is lost, so a
 * result next to a border of bfloat16 may round the other way); over a float32
 * cache every operand as a tf32 value and remainder, three of the four products
 * (about 2^-21 of each is lost). Scores times 1.45 and sums of up to 2^8 times the
 * values have to stay inside float32's range, float32 operands below 2^127.
 * The result does not depend on timing (partial results join in a fixed order).
 * How the work is cut up goes by the table's width, table_stride * page_size
 * tokens a branch, since the lengths are known on the device only: a table much
 * wider than the branches are long is slower where they are few (16 branches of
 * 256 tokens after 4,096 shared ones 11 us with a table for up to 512, 27 for
 * 4,096).
 * out may be q itself (with its stride); outputs and workspace must not overlap
 * anything else.
 * A bounded wait that gave up (a broken launch) sets DEC_DEVERR_GEMM_TIMEOUT in
 * the context-free error word. d_workspace: attn_shared_prefix_workspace(a)
 * bytes for these sizes, 256-byte aligned. */
typedef struct {
  int32_t batch, n_q, n_kv, head_dim;
  int32_t qdtype, kvdtype; /* q and out; prefix and pages: DEC_F32 or DEC_BF16 */
  const void* q;
  void* out;
  float* lse;
  int64_t q_stride, out_stride; /* elements between branches */
  const void *prefix_k, *prefix_v;
  int32_t prefix_len;
  int64_t prefix_stride; /* rows between heads, >= prefix_len */
  const void *k_pages, *v_pages;
  const int32_t* page_table;
  const int32_t* seq_len;
  int32_t num_pages, page_size, table_stride;
  float scale;
  void* d_workspace;
  size_t workspace_bytes;
} attn_shared_args;

/* Bytes of workspace for a call with these sizes (the pointers are not looked
 * at); 0 if they are invalid or the device is not supported. */
size_t attn_shared_prefix_workspace(const attn_shared_args* a);

/* "Megakernels", "What runs in the DSL": grouped-query attention, here of
 * several branches. Additional error: DEC_ENOMEM (workspace too small). */
dec_status attn_shared_prefix(const attn_shared_args* a, void* stream);

/* Beam search's selection: the n_out best of the beams x vocab continuations
 * by scores[b] + log_softmax(logits[b])[v], best first; of equal ones the
 * lowest b * vocab + v comes first (candidates are compared in 48 bits, over a
 * float32 sum of exponentials). out_scores float32, out_parents (b) and out_tokens
 * (v) int32 [n_out]. A logit of -inf or NaN is never chosen (NaN counts as
 * masked, as in the greedy argmax); a beam whose score, or score less
 * log-sum, is not finite, whose logits hold +inf, or which has no finite logit
 * offers nothing. A sum below the lowest finite float32 counts as that value,
 * behind those that reach it. Slots that nothing fills get parent -1, token -1
 * and score -inf. out_scores may be scores itself; outputs must not overlap
 * anything else.
 * beams 1..1024, n_out 1..1024, beams * vocab < 2^31; logits float32,
 * row b at logits + b * logits_stride. d_workspace as for
 * attn_shared_prefix; it holds a list of 12 bytes a logit for each of up to n_out
 * parts of the rows (13 MB for 64 beams x 151,936 and 128 outputs, 805 for 1,024
 * beams and outputs). */
typedef struct {
  int32_t beams, vocab, n_out;
  const float* logits;
  int64_t logits_stride;
  const float* scores;
  float* out_scores;
  int32_t *out_parents, *out_tokens;
  void* d_workspace;
  size_t workspace_bytes;
} beam_select_args;

size_t beam_select_workspace(const beam_select_args* a);

/* "Megakernels", "GPU-wide end-to-end generation": the selection of the next
 * tokens on the GPU with lowest-ID ties, here over several beams. Additional
 * error: DEC_ENOMEM. */
dec_status beam_select(const beam_select_args* a, void* stream);

/* After a selection: beam i continues beam p = parents[i]. Its new table row
 * lists p's filled pages (shared from now on, they are not written again),
 * then spare[i], which receives a copy of the old_len[p] % page_size tokens of
 * p's last, partly filled page (nothing where that is 0), in every layer; the
 * entries behind are -1, and new_len[i] = old_len[p]. So each beam owns the
 * page its next token goes to. The spare pages must differ from each other and
 * from every page of the old tables; the new table and lengths must not
 * overlap each other nor any input. parents[i] < 0, or a parent that is itself
 * unused (old_len < 0), makes slot i unused: new_len -1 and a row of -1.
 * old_len[p] must leave room for the next token (< table_stride * page_size); a
 * longer one, a parent >= beams, or a page of its tokens or a spare page outside
 * the pool sets DEC_DEVERR_BAD_PAGE and makes the slot unused. Layer l's pools
 * start l * layer_stride elements after k_pages and v_pages; layers must not
 * overlap. */
typedef struct {
  int32_t beams, layers, n_kv, head_dim, kvdtype;
  void *k_pages, *v_pages;
  int64_t layer_stride;
  int32_t num_pages, page_size, table_stride;
  const int32_t *parents, *spare; /* [beams] */
  const int32_t *old_table, *old_len;
  int32_t *new_table, *new_len;
} beam_reorder_args;

/* Counterpart of "Megakernels", "GPU-wide end-to-end generation" (the cache
 * entries a generation leaves) for branches that share entries. */
dec_status beam_reorder_pages(const beam_reorder_args* a, void* stream);

/* ---- Drafted trees of several requests ---------------------------------------
 *
 * The calls below run a step that checks drafted tokens of several requests over
 * the paged cache above; pools, tables, streams, workspaces and errors are as
 * for the branches. Request s holds tokens in pages and brings rows row_start[s]
 * .. row_start[s + 1] - 1: row 0 is its last known token, which is not in the
 * cache yet, the others are drafted ones, each below an earlier row of the
 * request (parents: its number within the request; row 0 has none, -1). Without
 * parents a request's rows are a chain, each row's parent the row before: a draft
 * in one line, the single tokens of an ordinary step, or a prompt's rows. Row i
 * goes to index held + i of the request's pages, siblings to different indexes,
 * and its position is held + its depth. mask gives the rows that a row attends
 * to, bit j % 32 of word j / 32 for row j of the request; the ancestors and the row
 * itself as step_slots makes it. A step: step_slots; in every layer kv_append_slots
 * and attn_tree_paged; after the vocabulary projection logits_adjust, which also
 * picks the greedy token after each row; tree_accept_paged, whose new lengths are
 * the next step's. They extend "Megakernels", "What runs in the DSL" and
 * "GPU-wide end-to-end generation" (greedy tokens on the GPU, lowest ID on ties)
 * to several drafted tokens at a time, as dec_verify2 does for one. */

/* Tables and slots of a step. held[s]: tokens that request s holds in pages, -1
 * once it has ended; fresh[s]: rows that it brings (below 0 counts as 0; an ended
 * request brings none). row_start [requests + 1]: the sum of the rows before, at
 * most `rows`. A request needs ceil((held + fresh) / page_size) pages and owns the
 * first owned[s] entries of its table row (the pages of its tokens, others left from
 * rejected drafts). What it lacks comes from the free pages, a ring of num_pages
 * entries: free_state[1] of them from entry free_state[0] on, in the requests'
 * order. A request is served if it lacks nothing or the free pages cover what it
 * and all requests before it lack; one that needs more pages than table_stride, has
 * rows past `rows`, or with a mask more than 32 * mask_words rows, is not and
 * asks for no page. Ended requests' pages go behind the ring's last entry, in order,
 * and can be given out from the next step on.
 * new_table: owned entries, then the new pages, then -1 (ended requests: -1); it
 * may be page_table itself, then the entries behind a request's pages are left as
 * they were. new_owned, new_free_state: what the next step starts from. ctx_len[s]:
 * held[s], or -1 for an ended request or one that is not served.
 * For every row r < rows: seq[r] its request, positions[r] = base_pos + held +
 * depth (base_pos: tokens of a shared prefix, which are not in pages), slots[r] =
 * page * page_size + row in the page, mask; -1, -1, -1 and a mask of 0 for rows of
 * requests that are not served and behind the last row. A row whose parent is not
 * an earlier row of its request (row 0's is not looked at), and rows below it,
 * have -1 and 0 too and set DEC_DEVERR_BAD_TREE; so does a request with more rows
 * than its mask has bits, or with parents and no mask more than 256 (such a prompt
 * goes in a step of its own, without parents and mask). Tables too narrow, rows past
 * `rows`, an owned count outside the table, pages out of range, a ring state outside
 * the ring and more returned pages than the ring has room for set
 * DEC_DEVERR_BAD_PAGE; running out of pages sets nothing. seq, positions, slots, mask
 * and parents may be NULL (mask without parents is a chain's). Up to 4096 requests,
 * masks up to 8 words.
 * Outputs must not overlap inputs or each other otherwise. */
typedef struct {
  int32_t requests, rows;
  int32_t num_pages, page_size, table_stride, base_pos, mask_words;
  const int32_t *held, *fresh, *owned; /* [requests] */
  const int32_t* parents;              /* [rows] or NULL */
  const int32_t* page_table;           /* [requests][table_stride] */
  int32_t* free_ring;                  /* [num_pages], in and out */
  const int32_t* free_state;           /* [2] first entry, entries */
  int32_t *new_table, *new_owned, *new_free_state;
  int32_t *row_start, *ctx_len;
  int32_t *seq, *positions;
  int64_t* slots;
  uint32_t* mask; /* [rows][mask_words] */
} step_slots_args;

dec_status step_slots(const step_slots_args* a, void* stream);

/* kv_append_paged by a map of slots: row r's key and value go to slots[r] =
 * page * page_size + row in the page. A padded row (positions[r] < 0) stores
 * nothing and leaves its q_out as it was; a slot of -1 stores nothing; one outside
 * the pool counts as a bad page, and its q_out is written. Two rows of one slot
 * leave a mixture of both there. Outputs must not overlap inputs (q_out may be q
 * itself; columns of one buffer do not overlap) or each other. */
typedef struct {
  int32_t rows, n_q, n_kv, head_dim; /* n_q may be 0 */
  int32_t xdtype, ydtype, kvdtype;   /* q, k, v; q_out; pages */
  const void *q, *k, *v;
  void* q_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  const float *g_q, *g_k;
  const int32_t* positions;
  const double* inv_freq;
  float eps, rope_factor;
  int32_t rot_dim, interleaved;
  void *k_pages, *v_pages;
  const int64_t* slots;
  int32_t num_pages, page_size;
} kv_slots_args;

dec_status kv_append_slots(const kv_slots_args* a, void* stream);

/* Grouped-query attention of all rows of a step: row i of request s over the shared
 * prefix (prefix_len keys and values a head, as in attn_shared_prefix; 0: none), the
 * request's seq_len[s] tokens in pages, and those of its rows that mask says (their
 * keys and values at index seq_len[s] + j of its pages); mask NULL: rows 0 .. i;
 * rows past the mask's bits are not attended to. out and lse as in
 * attn_shared_prefix; a row with nothing to attend to gets zeros (and lse -inf).
 * seq_len[s] < 0 marks an unused request, whose rows are left as they were, as are
 * rows of no request. What a row does not attend to does not reach it, whatever is
 * there (not finite as well), and rows of pages behind a request's last are never
 * used. row_start must not fall and lie in 0 .. rows (it is taken as if it did).
 * An index beyond table_stride * page_size counts as a bad page; its keys are left
 * out. Sizes, precision, order of results and the other rules are those of
 * attn_shared_prefix, with rows * n_q < 2^24, batch <= 4096 and (rows * n_q / 16 +
 * min(batch, rows) * n_kv) * (table_stride * page_size / 128 + 2) < 2^37. Matrix
 * instructions cut sums off instead of rounding them: at most 256 of one sum in a
 * row (2,048 keys), then it is added to a total in float32, so what is lost does not
 * grow with the length. The work is cut up on the device by the requests' lengths,
 * equal shares of key tiles for all SMs; which kernel runs, and with it a result's
 * last bits, goes by sizes that the host knows, the table's width among them, not the
 * lengths: single tokens of many short requests take longer with wide tables (256 of
 * 500 tokens 173 us with tables for more than 1,024, 104 with narrower ones). */
typedef struct {
  int32_t batch, rows, n_q, n_kv, head_dim;
  int32_t qdtype, kvdtype;
  const void* q;
  void* out;
  float* lse; /* [rows][n_q] or NULL */
  int64_t q_stride, out_stride;
  const int32_t* row_start; /* [batch + 1] */
  const uint32_t* mask;     /* [rows][mask_words] or NULL */
  int32_t mask_words;
  const void *prefix_k, *prefix_v;
  int32_t prefix_len;
  int64_t prefix_stride;
  const void *k_pages, *v_pages;
  const int32_t* page_table;
  const int32_t* seq_len;
  int32_t num_pages, page_size, table_stride;
  float scale;
  void* d_workspace;
  size_t workspace_bytes;
} attn_tree_args;

size_t attn_tree_paged_workspace(const attn_tree_args* a);

/* Additional error: DEC_ENOMEM (workspace too small). */
dec_status attn_tree_paged(const attn_tree_args* a, void* stream);

/* Logits by the rules of their requests. Row r belongs to request seq[r] (NULL: r;
 * outside [0, requests): the row is left as it was). Its text is the request's
 * tokens[0 .. tokens_len + tokens_base) and behind them, with draft_tokens, the
 * drafted tokens of those rows of the request that mask says (NULL: up to r
 * itself), in the rows' order. The first prompt_len (NULL: 0) tokens of it all are
 * its prompt, rows that bring a prompt's tokens among them. With n(v) the times
 * that token v comes after the prompt, a logit x of v becomes
 *   x / repetition (x > 0) or x * repetition, if v is in the text at all;
 *   x - frequency * n(v);  x - presence, if n(v) > 0;
 *   x + bias, if v is in the request's list of bias_len entries (of equal ones the
 *   last counts);
 *   -inf, if bit v % 32 of word v / 32 of the row's mask of allowed tokens is 0:
 *   row allowed_row[r] of `allowed` (< 0: none; NULL: row r; outside [0,
 *   allowed_rows): none, and DEC_DEVERR_BAD_TOKEN is set).
 * Each step is rounded to float32, out once to ydtype. repetition, frequency and
 * presence are float32 [requests] or NULL; repetition > 0. Tokens outside [0,
 * vocab) count nowhere, rows of a request past the mask's bits neither. next
 * (nullable, int32 [rows]): the token of the greatest resulting float32 logit, the
 * lowest of equal ones; NaN counts as masked; -1 if no logit is above -inf. out is
 * nullable where next is given, and may be logits itself (same dtype, stride).
 * vocab up to 2^20, rows up to 2^19 - 8; up to 2^19 tokens a text, as many drafted
 * ones and 1023 biases a list (longer ones are cut). Outputs must not overlap
 * anything else. */
typedef struct {
  int32_t rows, vocab, requests;
  int32_t xdtype, ydtype; /* logits; out: DEC_F32 or DEC_BF16 */
  const void* logits;
  int64_t logits_stride;
  void* out;
  int64_t out_stride;
  int32_t* next;
  const int32_t* seq;
  const int32_t* tokens; /* [requests][tokens_stride] or NULL: no text */
  int64_t tokens_stride;
  const int32_t *tokens_len, *prompt_len;
  int32_t tokens_base;
  const int32_t* draft_tokens; /* [rows] or NULL */
  const int32_t* row_start;    /* [requests + 1], with draft_tokens */
  const uint32_t* mask;        /* [rows][mask_words] or NULL */
  int32_t mask_words;
  const float *repetition, *frequency, *presence;
  const int32_t* bias_tokens; /* [requests][bias_stride] or NULL */
  const float* bias;
  const int32_t* bias_len;
  int32_t bias_stride;
  const uint32_t* allowed; /* [allowed_rows][allowed_stride words] or NULL */
  int64_t allowed_stride;
  int32_t allowed_rows;
  const int32_t* allowed_row;
} logits_adjust_args;

dec_status logits_adjust(const logits_adjust_args* a, void* stream);

/* The part of each tree that the greedy tokens confirm. Row 0 of a request is
 * accepted; after an accepted row r comes the first of its children whose drafted
 * token is next[r], until there is none (or path_stride rows are accepted).
 * count[s]: accepted rows; path[s][d]: their numbers within the request, out_tokens
 * [s][d] = next of them (the last one is the next step's row 0), -1 behind;
 * new_len[s] = seq_len[s] + count[s]. The keys and values of the accepted rows move
 * from index seq_len + path[d] of the request's pages to seq_len + d in every layer
 * (layer l's pools start l * layer_stride elements after k_pages and v_pages);
 * nothing else in the pools is written. tokens
 * (nullable): draft_tokens of the accepted rows are written to tokens[s][seq_len +
 * tokens_base + d]. A request with seq_len < 0 is left alone (count 0, path and
 * out_tokens -1, new_len = held[s], or -1 without held: with step_slots' ctx_len as
 * seq_len and its held, a request that was not served keeps its tokens and waits), one
 * without rows too (new_len = seq_len). A page of an
 * accepted row outside the pool or the table sets DEC_DEVERR_BAD_PAGE and that row is
 * not moved; a place outside tokens_stride is not written and sets
 * DEC_DEVERR_BAD_POSITION. layers may be 0 (nothing moves; no pools). path_stride up
 * to 256. Outputs, the pools among them, must not overlap inputs (tokens apart) or
 * each other. */
typedef struct {
  int32_t batch, rows, path_stride;
  int32_t layers, n_kv, head_dim, kvdtype;
  const int32_t* row_start; /* [batch + 1] */
  const int32_t* parents;   /* [rows], or NULL: chains */
  const int32_t *draft_tokens, *next; /* [rows] */
  const int32_t* seq_len;   /* [batch] */
  const int32_t* held;      /* [batch] or NULL */
  void *k_pages, *v_pages;
  int64_t layer_stride;
  int32_t num_pages, page_size, table_stride;
  const int32_t* page_table;
  int32_t* tokens; /* [batch][tokens_stride] or NULL */
  int64_t tokens_stride;
  int32_t tokens_base;
  int32_t *count, *new_len;   /* [batch] */
  int32_t *path, *out_tokens; /* [batch][path_stride] */
} tree_accept_args;

dec_status tree_accept_paged(const tree_accept_args* a, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* WSG_H */
