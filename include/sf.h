/*
 * sf.h — C ABI of the GB300 greedy speculative-decoding engine.
 *
 * One speculative round (the hot path) has four parts:
 *   draft    — a small draft model decodes K tokens greedily over its own
 *              static KV cache (sf_draft), or prompt lookup proposes up to K
 *              tokens (sf_ngram_draft);
 *   verify   — the target model runs one causal pass over the pending token
 *              and the K guesses and returns its own greedy choice at every
 *              position (sf_verify);
 *   accept   — the longest prefix of guesses that agrees with the target's
 *              choices is accepted, and the target's choice after it (the
 *              bonus token) is committed as well;
 *   rollback — both KV caches are cut back, in place, to the last committed
 *              position (sf_accept_rollback).
 * sf_step runs all four as one CUDA graph replay.
 *
 * Sources (page title, then section):
 *   "I Got 28 TPS Out of Free Kaggle GPUs. Here's What It Took." —
 *     "Speculative Decoding: The Idea" (draft guesses K tokens, the target
 *     checks them in one pass, agreed tokens are committed);
 *     "CUDA Graphs: What They Are and Why They Helped" (the whole draft
 *     forward, LM head and argmax replayed as one driver call);
 *     "Why It Kept Breaking (and How I Fixed It)" (static preallocated KV
 *     cache, in-place intermediates, explicit position updates, in-place KV
 *     rewind on rejection).
 *   "Qwen3.5-397B on 20 GPUs, through a relay" (Sangama results) —
 *     "Speculative decoding: correct, but slower (for now)" (look-back
 *     guesses of up to 4 tokens from the last 2-4 tokens; the verifier returns
 *     its own choice at every position; output equals normal decoding).
 *
 * Conventions for every call:
 *   - Ownership: the caller allocates and owns every device buffer (weights,
 *     both KV caches, the workspace). They must stay valid until sf_destroy.
 *     The library never allocates device memory; it allocates a little
 *     pinned host memory and one CUDA stream in sf_create.
 *   - Streams: all device work is enqueued on the stream given to sf_create.
 *     Calls that return host results synchronise that stream.
 *   - Errors: every call returns an sf_status and never aborts. On
 *     SF_ERR_ARG, SF_ERR_CAPACITY or SF_ERR_STATE nothing was enqueued and
 *     the engine state is unchanged. sf_last_error() gives a message for the
 *     calling thread's last failure.
 *   - Batch: sequences are independent; per-sequence lengths and accept
 *     lengths are kept on the device.
 *   - Rows per forward (batch * (K + 1)) are limited to SF_MAX_ROWS. Every
 *     forward reads each weight from HBM once: up to 16 bf16 rows on the
 *     weight-streaming mma.sync GEMM (all rows in one pass per CTA), more
 *     rows and every NF4 forward on the tcgen05 GEMM (tensor-memory
 *     accumulators, all token rows as the MMA's N side).
 */
#ifndef SF_H_
#define SF_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define SF_API __attribute__((visibility("default")))
#else
#define SF_API
#endif

#define SF_MAX_ROWS 80

typedef struct sf_engine* sf_handle;

typedef enum {
  SF_OK = 0,
  SF_ERR_ARG = 1,          /* invalid argument, null or misaligned pointer */
  SF_ERR_CAPACITY = 2,     /* a round would write past s_max cache slots */
  SF_ERR_CUDA = 3,         /* a CUDA runtime call failed */
  SF_ERR_NONFINITE = 4,    /* a non-finite logit was produced */
  SF_ERR_STATE = 5,        /* call out of order (e.g. verify before draft) */
  SF_ERR_UNSUPPORTED = 6,  /* shape or mode not supported by this build */
  SF_ERR_DEVICE = 7        /* a kernel reported a bounded wait that expired */
} sf_status;

/* Weight types: bf16; NF4 for the 7 linear maps of every layer (embedding,
 * norms, biases and LM head stay bf16); or fp32 for every tensor (the
 * single-precision correctness workload; plain fp32 arithmetic, not a fast path). */
enum { SF_WDTYPE_BF16 = 0, SF_WDTYPE_NF4 = 1, SF_WDTYPE_F32 = 2 };
/* Drafters: the draft model, prompt lookup, none (each round then commits
 * only the target's own next token: plain greedy decoding, the baseline the
 * speculative rounds are measured against), or prompt lookup with several
 * guesses verified side by side in one target pass (sf_tree_draft). */
enum { SF_DRAFT_NEURAL = 0, SF_DRAFT_NGRAM = 1, SF_DRAFT_NONE = 2, SF_DRAFT_TREE = 3 };

/* Decoder shape (Qwen2-style: GQA attention with RoPE, RMSNorm, SwiGLU MLP). */
typedef struct {
  int32_t layers, hidden, n_heads, n_kv_heads, head_dim, ffn, vocab;
  int32_t tied;       /* 1: the LM head is the embedding matrix */
  int32_t qkv_bias;   /* 1: q, k, v projections carry biases */
  int32_t embed_ld;   /* row stride of the embedding in elements; 0 = hidden */
  float rope_theta;   /* RoPE base */
  float rms_eps;      /* RMSNorm epsilon */
  int32_t wdtype;     /* SF_WDTYPE_BF16, SF_WDTYPE_NF4 or SF_WDTYPE_F32 */
} sf_model_cfg;

/*
 * Weight pointers (device, row-major [out, in], bf16 unless stated; every
 * tensor fp32 with SF_WDTYPE_F32), in this
 * order: embed [vocab, hidden] (row stride embed_ld); per layer: ln1 [hidden],
 * wq [n_heads*head_dim, hidden], wk, wv [n_kv_heads*head_dim, hidden],
 * bq, bk, bv (NULL when qkv_bias == 0), wo [hidden, n_heads*head_dim],
 * ln2 [hidden], wg, wu [ffn, hidden], wd [hidden, ffn]; final norm [hidden];
 * lm_head [vocab, hidden] (omitted when tied).
 * With SF_WDTYPE_NF4 each of wq, wk, wv, wo, wg, wu, wd takes two consecutive
 * slots: packed codes (uint8 [out, in/2], element 2i in the low nibble) then
 * block scales (fp16 [out, ld_s], ld_s = 8 * ceil(in / 512): the in/64 scales
 * of a row padded to a 16-byte row stride), as sf_nf4_quantize writes them;
 * in must be a multiple of 64.
 * Every row must start on a 16-byte boundary.
 * Returns the number of slots, or -1 for an invalid cfg.
 */
SF_API int32_t sf_weight_count(const sf_model_cfg* cfg);

/* Bytes of one KV cache: layout [layers][2 (k, v)][batch][n_kv_heads][s_max][head_dim] bf16. */
SF_API size_t sf_kv_bytes(const sf_model_cfg* cfg, int32_t batch, int32_t s_max);

/* Bytes of device workspace sf_create needs (dft may be NULL: n-gram only);
 * 0 for an invalid configuration. The caller allocates it once: the pages'
 * fix for graph replays is a static, preallocated cache and in-place
 * intermediates ("Why It Kept Breaking (and How I Fixed It)", fixes 1-2). */
SF_API size_t sf_workspace_bytes(const sf_model_cfg* tgt, const sf_model_cfg* dft, int32_t batch,
                          int32_t K, int32_t s_max);

/*
 * Bind caller-owned buffers and build the engine ("Speculative Decoding: The
 * Idea": a small draft model beside the target; for an n-gram-only engine,
 * "Speculative decoding: correct, but slower (for now)" on the Sangama
 * page). kv_d may be NULL when dft
 * is NULL. workspace must hold sf_workspace_bytes(...) bytes, 256-byte
 * aligned. batch: 1..32 independent sequences. K: guesses per round (1..15,
 * batch*(K+1) <= SF_MAX_ROWS).
 * s_max: cache slots per sequence, a multiple of 64.
 * cuda_stream: a cudaStream_t (NULL = legacy default stream).
 * The engine starts with SF_DRAFT_NEURAL when dft is given, else
 * SF_DRAFT_NGRAM (max guess K, n from 4 down to 2).
 */
SF_API sf_status sf_create(const sf_model_cfg* tgt, const void* const* tgt_w,
                    const sf_model_cfg* dft, const void* const* dft_w,
                    int32_t batch, int32_t K, int32_t s_max,
                    void* kv_t, void* kv_d, void* workspace, void* cuda_stream,
                    sf_handle* out);

/*
 * The same engine with the target's cache in pages: kv_pool is a pool of
 * n_pages (1..2^24) pages of 64 slots, layout [layers][2 (k, v)][n_pages]
 * [n_kv_heads][64][head_dim] bf16, that the sequences share. Each holds the
 * pages of the tokens it has and of the round under way instead of s_max
 * slots: every target pass begins with a page plan (sf_page_plan below) on the
 * device that takes the pages its rows need and gives back those that the last
 * rewind left behind, and attends over the pages (sf_paged_attention below).
 * The draft model's cache stays s_max slots per sequence. s_max is the most
 * tokens of a sequence. Calls that need more pages than the pool has return
 * SF_ERR_CAPACITY like those that pass s_max. workspace:
 * sf_paged_engine_workspace_bytes(...) bytes. SF_PERSISTENT applies to the
 * draft model only, and the timeline (sf_trace) leaves the target's attention
 * out. sf_get_pages: pages held per sequence (host [batch]) and free pages
 * (host [1]), each may be NULL.
 */
SF_API size_t sf_kv_pool_bytes(const sf_model_cfg* cfg, int32_t n_pages);
SF_API size_t sf_paged_engine_workspace_bytes(const sf_model_cfg* tgt, const sf_model_cfg* dft, int32_t batch,
                                              int32_t K, int32_t s_max, int32_t n_pages);
SF_API sf_status sf_create_paged(const sf_model_cfg* tgt, const void* const* tgt_w,
                    const sf_model_cfg* dft, const void* const* dft_w,
                    int32_t batch, int32_t K, int32_t s_max, int32_t n_pages,
                    void* kv_pool, void* kv_d, void* workspace, void* cuda_stream,
                    sf_handle* out);
SF_API sf_status sf_get_pages(sf_handle h, int32_t* h_held, int32_t* h_free);

/*
 * Load prompts and fill both caches (the step before the speculative loop;
 * "Qwen3.5-397B on 20 GPUs", "What made it faster": prompts go through in
 * pieces). h_tokens: host [batch][stride] int32,
 * h_lens: host [batch] prompt lengths (each >= 2 and <= stride; they may
 * differ). After it, each cache holds its prompt except the last token,
 * which is pending. Prompts of one length are filled side by side in chunks
 * of up to SF_MAX_ROWS rows; otherwise each sequence is filled on its own.
 */
SF_API sf_status sf_prefill(sf_handle h, const int32_t* h_tokens, const int32_t* h_lens, int32_t stride);

/*
 * Neural draft ("Speculative Decoding: The Idea": the small model guesses K
 * tokens one at a time; "CUDA Graphs: What They Are and Why They Helped":
 * the K steps replay as one graph): K greedy decode steps of the draft model. Writes the guesses
 * to the engine's device state and, when not NULL, to d_draft (device
 * [batch][K] int32) and their logits to d_logits (device [batch][K][vocab]
 * fp32). The first step runs two rows (the last two committed tokens) so the
 * draft cache always catches up with the committed sequence. With both
 * outputs NULL the K steps replay as one captured CUDA graph.
 */
SF_API sf_status sf_draft(sf_handle h, int32_t* d_draft, float* d_logits);

/*
 * Prompt-lookup draft ("Speculative decoding: correct, but slower (for
 * now)", Sangama page: guess what followed the last 2-4 tokens the last time
 * they appeared): for n = max_n down to min_n, the rightmost earlier
 * occurrence of the last n committed tokens; up to max_guess tokens that
 * followed it are proposed (cut at the end of the context). Optional device
 * outputs: d_prop [batch][max_guess] (unused slots 0), d_count [batch].
 * max_guess must be <= K.
 */
SF_API sf_status sf_ngram_draft(sf_handle h, int32_t max_guess, int32_t min_n, int32_t max_n,
                         int32_t* d_prop, int32_t* d_count);

/*
 * Several prompt-lookup guesses per round (the Sangama page, "Next": better
 * guesses for the look-back drafter; here several earlier occurrences are
 * checked by the target together instead of only the most recent one). The
 * earlier occurrences of the last n committed tokens are taken in
 * sf_ngram_draft's order (n from max_n down to min_n, rightmost first); each
 * gives up to g = K / n_cand tokens that followed it (cut at the end of the
 * context); a guess equal to one already taken is skipped; at most n_cand
 * guesses. Guess c fills verify rows 1 + c*g .. c*g + g. sf_verify then runs
 * the rows of each guess at the positions after the pending token, each
 * seeing the committed sequence and its own guess only, and
 * sf_accept_rollback takes the guess with the longest accepted prefix (the
 * lowest c on ties), commits as for one guess and moves that guess's
 * target-cache entries down to the committed slots. Optional device outputs:
 * d_prop [batch][n_cand][g] (unused 0), d_len [batch][n_cand] (0: no guess).
 * 1 <= n_cand <= K; 1 <= min_n <= max_n <= 64.
 */
SF_API sf_status sf_tree_draft(sf_handle h, int32_t n_cand, int32_t min_n, int32_t max_n, int32_t* d_prop,
                               int32_t* d_len);

/*
 * Target verify ("Speculative Decoding: The Idea": the target checks all
 * guesses in one forward pass; the Sangama page: the model's own choice at
 * every position): one causal pass over [pending, d_1..d_K] per sequence,
 * appending K+1 entries to the target cache. Optional device outputs: the
 * target's argmax at every row (d_tgt_argmax [batch][K+1] int32) and the
 * logits (d_logits [batch][K+1][vocab] fp32). Ties go to the lowest index.
 * With both outputs NULL the pass replays as one captured CUDA graph.
 */
SF_API sf_status sf_verify(sf_handle h, int32_t* d_tgt_argmax, float* d_logits);

/*
 * Accept and roll back ("Speculative Decoding: The Idea": keep the agreed
 * tokens; "Why It Kept Breaking (and How I Fixed It)", fix 4: in-place KV
 * rewind on rejection), per sequence: n = longest prefix of guesses equal to
 * the target's choices (capped at the number of real guesses); d_1..d_n and
 * the target's choice t_n are committed; both caches are cut back in place
 * to the committed length minus one. Host outputs (may be NULL):
 * h_n_accepted [batch], h_committed [batch][K+1], h_n_committed [batch].
 */
SF_API sf_status sf_accept_rollback(sf_handle h, int32_t* h_n_accepted, int32_t* h_committed,
                             int32_t* h_n_committed);

/* One whole round ("CUDA Graphs: What They Are and Why They Helped": one
 * driver call instead of a launch per kernel): draft (neural or n-gram, per
 * sf_set_drafter) + verify + accept/rollback as one CUDA graph replay. Host
 * outputs as in sf_accept_rollback (may be NULL). */
SF_API sf_status sf_step(sf_handle h, int32_t* h_n_committed, int32_t* h_committed);

/*
 * Run rounds until every sequence has at least n_new new tokens since its
 * prompt. The rounds run on the device as one graph launch: a WHILE
 * conditional node repeats the round graph, and a control kernel at the end
 * of each round decides on the device whether another round is needed and
 * fits in s_max (the pages' single driver call for the draft, "CUDA Graphs:
 * What They Are and Why They Helped", taken to the whole generation); the
 * host synchronises once. With SF_HOST_LOOP=1 in the environment at
 * sf_create the host replays the round graph instead, synchronising only to
 * count (same tokens). h_out: host [batch][n_new] (the first n_new generated
 * tokens). h_rounds: rounds run (may be NULL). SF_ERR_CAPACITY when s_max
 * runs out first.
 */
SF_API sf_status sf_generate(sf_handle h, int32_t n_new, int32_t* h_out, int32_t* h_rounds);

/* Rewind every sequence to its prompt (prefix already in the caches). */
SF_API sf_status sf_reset(sf_handle h);

/* Select the drafter used by sf_step / sf_generate (SF_DRAFT_*; min_n and
 * max_n apply to SF_DRAFT_NGRAM and SF_DRAFT_TREE only). */
SF_API sf_status sf_set_drafter(sf_handle h, int32_t mode, int32_t min_n, int32_t max_n);

/* Guesses per round of SF_DRAFT_TREE in sf_step / sf_generate (1..K; the
 * default is 2, or 1 when K = 1). */
SF_API sf_status sf_set_tree_candidates(sf_handle h, int32_t n_cand);

/* The guess each sequence's last multi-candidate round took (host [batch]). */
SF_API sf_status sf_tree_winner(sf_handle h, int32_t* h_c);

/* Current cache lengths per sequence (host [batch] each, may be NULL): the
 * positions the in-place rewind left ("Why It Kept Breaking", fixes 3-4:
 * explicit position updates, in-place rewind). */
SF_API sf_status sf_get_lengths(sf_handle h, int32_t* h_len_t, int32_t* h_len_d);

/* Accept-length histogram since prefill: host [batch][K+1]. */
SF_API sf_status sf_get_accept_hist(sf_handle h, int32_t* h_hist);

/*
 * Launch timeline, for profiling. Only when the environment variable
 * SF_TRACE=1 was set at sf_create: every kernel of the forward passes
 * stamps the GPU global timer (ns) when it starts and when its wait on the
 * preceding kernel returns. sf_trace copies up to max_launches pairs
 * {start, wait_done} into h_out (host, 2 x uint64 each) for launch slots
 * 0.. (launch n uses slot n mod 8192; graph replays rewrite their slots) and
 * returns the count; with h_out NULL it returns the number of launches
 * enqueued so far; 0 when tracing is off. sf_trace_label(i) names slot i ("qkv",
 * "attention", "merge", "o_proj", "gate_up", "down", "lm_head", "embed").
 */
SF_API int32_t sf_trace(sf_handle h, uint64_t* h_out, int32_t max_launches);
SF_API const char* sf_trace_label(sf_handle h, int32_t i);

/* Kernel launches in one round of the current drafter (the node count of
 * its round graph; every node is a kernel; sf_generate's device loop adds one
 * control kernel per round), or 0 before a round graph has been built by
 * sf_step / sf_generate. */
SF_API int64_t sf_round_launches(sf_handle h);

/* Name of a status code; message of the calling thread's last failure. */
SF_API const char* sf_status_str(sf_status s);
SF_API const char* sf_last_error(void);
/* Release the engine's graphs, stream and pinned host memory (the caller's
 * device buffers stay the caller's). NULL is ignored. */
SF_API void sf_destroy(sf_handle h);

/*
 * One skinny linear map on its own: y[m][n] = sum_k x[m][k] * W[n][k] for
 * m < M (1..SF_MAX_ROWS), the weight-streaming GEMM every projection of the
 * forward pass uses. W: device bf16 [N, ld] row-major (ld >= K, K and ld
 * multiples of 8, 16-byte aligned rows); x: device fp32 [M, K]; y: device
 * fp32 [M, N]. d_workspace: device scratch of
 * sf_linear_workspace_bytes(N, K) bytes, 256-byte aligned, for split-K
 * partial tiles, arrival counters (zeroed by the call) and a bf16 hi/lo copy
 * of x in the GEMM's operand order. Enqueued on cuda_stream; returns without
 * synchronising. There is no device status word here: should a weight-tile
 * wait ever expire, the kernel returns normally and y is unspecified.
 */
SF_API size_t sf_linear_workspace_bytes(int32_t N, int32_t K);
SF_API sf_status sf_linear(const void* d_w, int32_t N, int32_t K, int32_t ld, const float* d_x, int32_t M,
                           float* d_y, void* d_workspace, void* cuda_stream);

/*
 * The two halves of sf_linear. Every projection reads its token rows in the
 * order its GEMM kernel consumes them.
 * Up to 16 rows ("fragment order", the mma.sync kernel): bf16 pairs (hi =
 * bf16(v), lo = bf16(v - hi), about 16 mantissa bits of the fp32 value) in
 * the order the MMA lanes read their B operand: with T = ceil(M / 4) token
 * tiles, the 16-byte unit ((j * T + t) * 2 + h) * 32 + l holds, for 64-feature
 * chunk j, tile t, half h and lane l = 4 * col + c, the 8 features
 * 64j + 16c + 8h + 0..7 of token 4t + col / 2, hi parts for even col and lo
 * parts for odd col.
 * More than 16 rows (the tcgen05 kernel; the threshold is 17 unless
 * SF_UMMA_MIN_ROWS says otherwise): bf16(v) in the tensor-core B tile with
 * 128-byte swizzle: with T8 = ceil(M / 8), the 1024-byte block at byte
 * (j * T8 + t) * 1024 holds tokens 8t .. 8t+7 of chunk j, one 128-byte row
 * per token (row m % 8), its 16-byte piece q (features 64j + 8q .. +7) at
 * position q ^ (m % 8) of the row.
 * Features past K and tokens past M are zero.
 *   sf_frag_bytes(K, M): size of the copy to allocate (0 if invalid).
 *   sf_to_frag: x (device fp32 [M, ld], features 0..K-1) -> d_frag (device,
 *     16-byte aligned, sf_frag_bytes(K, M) bytes), enqueued on cuda_stream.
 *   sf_linear_frag: sf_linear reading the copy instead of x (same W, y and
 *     workspace rules); reuse one copy for several matrices that share x.
 */
SF_API size_t sf_frag_bytes(int32_t K, int32_t M);
SF_API sf_status sf_to_frag(const float* d_x, int32_t M, int32_t K, int32_t ld, void* d_frag, void* cuda_stream);
SF_API sf_status sf_linear_frag(const void* d_w, int32_t N, int32_t K, int32_t ld, const void* d_frag, int32_t M,
                                float* d_y, void* d_workspace, void* cuda_stream);

/*
 * sf_linear without any caller-provided scratch, for callers that cannot
 * allocate device memory where they need the projection: plug-ins whose
 * host framework owns every device allocation through its own pool, and
 * latency-critical loops that cannot afford cudaMalloc's implicit device
 * synchronisation. Same arguments and result as sf_linear minus d_workspace.
 * (The pages have no counterpart of this call.)
 *
 * The scratch is a file-scope device array of about 38 MB inside the
 * library, enough for N up to 1,048,576 output rows, K up to 65,536 inputs
 * and M up to SF_MAX_ROWS token rows; every GPU that loads the library keeps
 * it until the process exits. The call allocates nothing: the first call on
 * each device looks up the array's device address (cudaGetSymbolAddress)
 * with that device current and keeps it for the life of the process, so a
 * context reset (cudaDeviceReset) after that first call is not supported.
 * All calls share the array: it keeps the last call's contents, the counters
 * that must start at zero are cleared by each call, and calls that overlap
 * on the GPU race with each other. N, K or M beyond the limits returns
 * SF_ERR_ARG with a message in sf_last_error().
 */
SF_API sf_status sf_linear_noalloc(const void* d_w, int32_t N, int32_t K, int32_t ld, const float* d_x,
                                   int32_t M, float* d_y, void* cuda_stream);

/*
 * Blockwise NF4 quantisation of a bf16 matrix on the device (a preparation
 * step for SF_WDTYPE_NF4 weights): w [rows, cols] with row stride ld
 * elements, cols a multiple of 64; writes packed codes [rows, cols/2] and fp16
 * block scales [rows, 8 * ceil(cols / 512)] (padding entries untouched).
 * Codebook: the NormalFloat construction of
 * Dettmers et al., "QLoRA" (2023), section 3 (format named in "The Numbers").
 */
SF_API sf_status sf_nf4_quantize(const void* d_w, int32_t rows, int32_t cols, int32_t ld,
                          void* d_packed, void* d_scales, void* cuda_stream);

/* ------------------------------------------------------------------------
 * A key-value cache in pages, for programs that serve sequences of different
 * lengths from one pool (the engine's own caches are s_max slots per
 * sequence, unless it is made with pages). Three operators run one after the
 * other in a pass: sf_page_plan (block tables, cache slots and positions
 * from the requests' lengths), sf_kv_append (RoPE and the new rows' keys and
 * values into their slots) and sf_paged_attention (the new rows over their
 * requests' pages). Everything they need to know about a pass lies in device
 * memory, so a pass is captured into a CUDA graph once and replayed with
 * other lengths. No call synchronises or allocates; all work is enqueued on
 * cuda_stream. A pass's token rows lie request after request: starts[b] ..
 * starts[b + 1] - 1 are the newest rows of request b, the last of them at
 * position lens[b] - 1.
 */

/* Element types of rows and caches. */
enum { SF_DT_F32 = 0, SF_DT_BF16 = 1, SF_DT_F16 = 2 };

/* One layer's cache: k and v are device tensors [n_pages][n_kv_heads][page]
 * [head_dim] with any strides (in elements, the last dimension contiguous):
 * pages whose keys and values alternate in one pool, or pages laid out
 * [page][n_kv_heads][head_dim], are views of this form. dtype SF_DT_BF16 or
 * SF_DT_F16; page 16, 32, 64, 128 or 256; head_dim 64 or 128. Pointers
 * 16-byte aligned, strides positive multiples of 8, the page stride the
 * largest, n_pages * page < 2^31. Slot s is slot s % page of page s / page. */
typedef struct {
  void* k;
  void* v;
  int32_t dtype, n_pages, n_kv_heads, page, head_dim, reserved;
  int64_t k_page, k_head, k_slot;   /* strides of k */
  int64_t v_page, v_head, v_slot;   /* strides of v */
} sf_paged_cache;

/* n token rows of n_heads heads each: element (i, h, d) at
 * data[i * row + h * head + d] (row and head strides in elements; rows that a
 * call writes may not overlap). */
typedef struct {
  void* data;
  int32_t dtype, n_heads;
  int64_t row, head;
} sf_rows;

/*
 * Block tables and slot maps from request lengths. Request b is to hold
 * lens[b] tokens after the pass, its rows among them (0: it has finished), so
 * ceil(lens[b] / page) pages: entries 0 .. held[b] - 1 of row b of tables
 * [batch][table_width] are the pages it holds on entry; free[0 .. *n_free - 1]
 * is a stack of the pages nobody holds (capacity: the size of free). First
 * every page that a request no longer needs goes onto the stack, in request
 * order and within a request in table order; then every page that a request
 * lacks is taken from the top, in request order. A request whose pages would
 * not all be there (counting those that the requests before it want) gets
 * none and keeps what it holds, and so does every later request that wants
 * pages. Outputs: tables and free in place; held_out and n_free_out (they may
 * be held and n_free themselves); status [batch]: 0 served, 1 not enough
 * pages, 2 refused (a negative length, more pages than table_width, more rows
 * than tokens, or held[b] outside 0..table_width), the last two leaving the
 * request's pages as they are; and for each of the n_rows rows its cache slot
 * (page number * page + offset) and position. Rows of requests whose status
 * is not 0 and rows behind the last request get slot -1, position 0.
 * With held_out and n_free_out apart from held and n_free a call can be
 * repeated: it reads nothing that it changes. All int32; starts [batch + 1].
 * batch 1..8192; page a power of two 16..256; n_rows may be 0 (slots and
 * positions may then be NULL).
 */
SF_API sf_status sf_page_plan(const int32_t* d_lens, const int32_t* d_starts, int32_t batch, int32_t page,
                              int32_t* d_tables, int32_t table_width, const int32_t* d_held, int32_t* d_free,
                              int32_t capacity, const int32_t* d_n_free, int32_t n_rows, int32_t* d_slots,
                              int32_t* d_positions, int32_t* d_held_out, int32_t* d_n_free_out, int32_t* d_status,
                              void* cuda_stream);

/* The RoPE table of the engine's models: fp32 [n_pos][head_dim / 2][2] =
 * (cos, sin) of pos * theta^(-2 i / head_dim), computed in double precision. */
SF_API sf_status sf_rope_table(float* d_table, int32_t n_pos, int32_t head_dim, float theta, void* cuda_stream);

/*
 * RoPE and cache append of n rows: row i's keys and values go, rounded once,
 * to slot slots[i] of every KV head; with d_rope (sf_rope_table's layout,
 * n_pos positions) the keys and queries are first rotated by the row's
 * position (element i is paired with i + head_dim / 2), in fp32. q may be
 * NULL (keys and values only); otherwise its rows go to q_out (the same heads;
 * q's or the cache's type; it may be q itself when the types are equal). Rows
 * whose slot lies outside the cache, or whose position lies outside the table,
 * are padding: nothing is written for them. The slots of a call are distinct
 * (of two rows with one slot, it is open whose elements stay), and the cache's
 * own slots may not overlap (refused by their strides). positions is
 * read only with d_rope. k and v have one type, F32, BF16 or F16, and q the
 * same. Data 16-byte aligned, strides multiples of 8 (of 4 for F32).
 */
SF_API sf_status sf_kv_append(const sf_paged_cache* cache, int32_t n, const sf_rows* k, const sf_rows* v,
                              const int32_t* d_slots, const sf_rows* q, const sf_rows* q_out,
                              const int32_t* d_positions, const float* d_rope, int32_t n_pos, void* cuda_stream);

/*
 * Attention of the requests' newest rows over their pages: out = softmax(q k^T
 * * scale) v over the slots that the row sees, query head h reading KV head
 * h / (n_heads / n_kv_heads). Row j of the n_b rows of request b sees the
 * lens[b] - n_b slots before the pass's rows, and of those rows: the first to
 * its own (row i of the pass lies in slot lens[b] - n_b + i); with d_mask
 * (uint64 [n], max_rows <= 64) instead those whose bit i is set, which is how
 * several guesses are verified side by side. A row that sees nothing gives out
 * 0 and lse -infinity; what masked slots and slots past lens[b] hold, NaN
 * included, changes nothing. lse (fp32 [n][n_heads], may be NULL): the natural
 * logarithm of the row's sum of exponentials. d_starts NULL: every request has
 * n / batch rows (n a multiple of batch). A request may have 0 rows, and at
 * most max_rows (1..SF_MAX_ROWS; further ones are not computed). Rows outside
 * every request are left as they were. lens[b] is cut to table_width * page,
 * and a table entry that is no page of the cache reads as zeros.
 * q and out have one type: the cache's, or F32 over a BF16 cache (exact in the
 * queries and probabilities: each is three bf16 terms). Probabilities of 16-bit
 * queries are rounded to that type, by half a step of each, or in fp16 by 2^-37
 * of the row's largest if that is more. n_heads a multiple of n_kv_heads. A key
 * or value that is no finite number may make the rows that see it NaN, also
 * where the formula gives an infinity or a weight of 0.
 * workspace: sf_paged_attention_workspace_bytes(...) bytes of device scratch,
 * 256-byte aligned, any contents; calls that may overlap on the GPU need one
 * each. Waits inside the kernels are bounded (seconds; what they wait for takes
 * microseconds): one that runs out leaves NaN in the rows concerned.
 * The queries' tiles follow from what the tables can hold (batch, table_width,
 * page), as the lengths lie on the device. In tables much wider than the lengths
 * a few short requests with more than 16 queries a KV head take up to 1.45 times
 * as long as in tight ones (measured: one of 2057 tokens, 63 fp32 queries, 15.6
 * us in a table of 32768 tokens, 10.9 in one of 2112); single rows do not. A
 * result depends on that and on the whole batch's lengths in its last bits (the
 * split over the cache's length follows them) and is the same in every run.
 */
SF_API size_t sf_paged_attention_workspace_bytes(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                                                 int32_t max_rows);
SF_API sf_status sf_paged_attention(const sf_paged_cache* cache, const sf_rows* q, const sf_rows* out, int32_t n,
                                    const int32_t* d_tables, int32_t table_width, const int32_t* d_lens,
                                    const int32_t* d_starts, int32_t batch, int32_t max_rows,
                                    const uint64_t* d_mask, float scale, float* d_lse, void* d_workspace,
                                    void* cuda_stream);

/*
 * Attention of a chunk of new tokens over the pages: a whole prompt, or a long
 * piece of one, behind what its request holds already. As sf_paged_attention
 * without a mask, for requests of up to max_rows rows, 1..2^20 (max_rows *
 * n_heads / n_kv_heads at most 2^30): row j of the n_b rows of request b sees
 * the slots 0 .. lens[b] - n_b + j, and writes out and lse by the same rules
 * (types, strides, rows that see nothing, rows outside every request, odd
 * values, waits, the workspace).
 * Which kernels run follows the types and what the tables can hold (batch,
 * table_width, page) with max_rows, of which no more than n count; in tables much
 * wider than the lengths little chunks take the kernels of large ones (97 rows,
 * 14 / 2 heads of 64: 9.4 us in tight tables, 11.5 in wide ones). So do a result's
 * last bits, which follow the whole batch's lengths as well; they are the same in
 * every run.
 */
SF_API size_t sf_chunk_attention_workspace_bytes(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                                                 int32_t max_rows);
SF_API sf_status sf_chunk_attention(const sf_paged_cache* cache, const sf_rows* q, const sf_rows* out, int32_t n,
                                    const int32_t* d_tables, int32_t table_width, const int32_t* d_lens,
                                    const int32_t* d_starts, int32_t batch, int32_t max_rows, float scale,
                                    float* d_lse, void* d_workspace, void* cuda_stream);

/*
 * Pages that several requests hold. shares[p] (int32 [n_pages]) counts page p's
 * holders beyond the first: 0 for a page that one request holds, or none. Only
 * whole pages are shared, and nobody writes into one: a request appends behind
 * them, into pages of its own. sf_page_plan knows nothing of shares: requests
 * that hold shared pages may grow by it, but are cut and ended by sf_page_free.
 * All arrays int32, updated in place unless said otherwise; entries of tables
 * that are no page (outside 0..n_pages - 1) are passed over, not counted. Arrays
 * that a call writes may lie over no other of its arrays (refused).
 */

/*
 * Cuts requests short or ends them: request requests[i] is to hold keep[i]
 * tokens (keep NULL: 0), so the first ceil(keep[i] / page) of its pages. Of the
 * pages that it gives up, those that nobody else holds any more go onto the
 * stack (in the order of the list, within a request in table order, each at its
 * first place there), and the others' shares go down. status [n]: 0, or 2
 * where the call leaves the request as it is: a number outside 0..batch - 1 or
 * named earlier in the list, a negative keep, more than it holds, or a cut that
 * would end inside a page that others hold on entry (what is appended next
 * would change it for them). n 0..8192; batch 1..8192; batch * table_width and
 * n * table_width below 2^30. The stack has room for every page.
 */
SF_API sf_status sf_page_free(const int32_t* d_requests, const int32_t* d_keep, int32_t n, int32_t batch, int32_t page,
                              int32_t* d_tables, int32_t table_width, int32_t* d_held, int32_t* d_shares,
                              int32_t n_pages, int32_t* d_free, int32_t capacity, int32_t* d_n_free,
                              int32_t* d_status, void* cuda_stream);

/*
 * Forks requests: dst[i], which holds nothing, becomes a second holder of the
 * first lens[src[i]] tokens of src[i]. The pages that these fill are shared; for
 * a partly filled last one dst[i] gets a page off the stack, in the order of the
 * list, and source[i], target[i] and slots[i] say what sf_page_copy has to copy
 * into it in every layer (page, page, filled slots; -1, -1, 0: nothing).
 * status [n]: 0 forked; 1 not enough pages (for this one and those before it);
 * 2 refused: a number outside 0..batch - 1, src = dst, a dst that holds pages
 * on entry or is named earlier in the list, a negative length, or more tokens
 * than src holds pages for. Where it is not 0 nothing is changed for that fork.
 * One request may be forked many times. lens [batch] is not changed. Sizes as
 * in sf_page_free.
 */
SF_API sf_status sf_page_fork(const int32_t* d_src, const int32_t* d_dst, int32_t n, const int32_t* d_lens,
                              int32_t batch, int32_t page, int32_t* d_tables, int32_t table_width, int32_t* d_held,
                              int32_t* d_shares, int32_t n_pages, const int32_t* d_free, int32_t capacity,
                              int32_t* d_n_free, int32_t* d_source, int32_t* d_target, int32_t* d_slots,
                              int32_t* d_status, void* cuda_stream);

/*
 * Moves the held pages to the lowest numbers. Of U pages that the tables hold
 * (each counted once), those numbered U and up move, in ascending order, to the
 * pages below U that nobody holds. tables_out and shares_out (they may be tables
 * and shares themselves) say the same with the new numbers; entries behind a
 * request's pages stay as they are, and pages that nobody holds have shares 0.
 * The stack is written anew: every page that no table holds, the lowest on
 * top. source and target [moves], moves at least n_pages / 2, list what
 * sf_page_copy has to copy in every layer, count [1] how many they are; entries
 * behind them are -1. No target is a source. With tables_out and shares_out
 * apart from tables and shares a call can be repeated. batch 1..8192, batch *
 * table_width below 2^30, n_pages up to 2^20, capacity at least n_pages.
 */
SF_API sf_status sf_page_compact(const int32_t* d_tables, int32_t batch, int32_t table_width, const int32_t* d_held,
                                 const int32_t* d_shares, int32_t n_pages, int32_t* d_tables_out,
                                 int32_t* d_shares_out, int32_t* d_free, int32_t capacity, int32_t* d_n_free,
                                 int32_t* d_source, int32_t* d_target, int32_t moves, int32_t* d_count,
                                 void* cuda_stream);

/*
 * Copies pages: the first slots[i] slots (NULL: all) of page source[i] into page
 * target[i], keys and values of every KV head, in each of `layers` layers;
 * cache describes the first, and layer l lies l * k_layer and l * v_layer
 * elements behind it (one after the other, or the layers of a page side by side
 * within it). The first *count of the n pairs count (NULL: all); a pair with a
 * number that is no page of the cache is passed over. A page is a target at most
 * once and no source of the same call (else it is open what it holds). layers *
 * n_kv_heads at most 2^24.
 */
SF_API sf_status sf_page_copy(const sf_paged_cache* cache, int32_t layers, int64_t k_layer, int64_t v_layer,
                              const int32_t* d_source, const int32_t* d_target, const int32_t* d_slots, int32_t n,
                              const int32_t* d_count, void* cuda_stream);

/*
 * Log probabilities of given tokens. Row i of logits (n rows of vocab elements,
 * fp32, bf16 or fp16, row_stride elements apart) and token tokens[i] give, in
 * fp32 throughout:
 *   logprob [n]        x_t - lse, lse = log sum_v e^x_v
 *   entropy [n]        -sum_v p_v log p_v, in nats
 *   rank [n]           how many tokens stand in front of the given one
 *   top_ids, top_logprobs [n][top]   the first `top` tokens, 0..32 and at most
 *                      vocab, and their log probabilities
 * in the order of larger logits first, of equal ones the lower token (a NaN
 * counts as -infinity there, and -0 is 0). Any output may be NULL. A logit of
 * -infinity is a token that cannot come; of a row that has no other, every log
 * probability is -infinity and the entropy 0. A row that holds a NaN or
 * +infinity gives NaN for log probabilities and entropy. Rows whose token lies
 * outside 0..vocab - 1 are padding: nothing is written for them. vocab 1..2^31 -
 * 65; logits aligned to their type, with any row stride from 0 to 2^38. Outputs
 * may lie over no other array (refused).
 */
SF_API sf_status sf_token_logprobs(const void* d_logits, int32_t dtype, int64_t row_stride, int32_t n, int32_t vocab,
                                   const int32_t* d_tokens, int32_t top, float* d_logprob, float* d_entropy,
                                   int32_t* d_rank, int32_t* d_top_ids, float* d_top_logprobs, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* SF_H_ */
