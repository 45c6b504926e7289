/*
 * dflash.h - C ABI of the GB300 (sm_103a) greedy block-diffusion speculative
 * decoding round: target prefill, block drafting with target-context KV
 * injection, one-pass target verification, greedy acceptance and rollback.
 *
 * The operations follow two public pages:
 *   [digest] "DFlash: Block Diffusion for Flash Speculative Decoding"
 *            (paper digest: Method / Inference §4.1, the greedy decoding-round
 *            and draft-layer pseudocode, "Paper vs code").
 *   [review] "DFlash: Why a Diffusion Drafter Can Accelerate an Autoregressive
 *            Model" (technical review: §2.3 eq. 2, §4.1, Algorithm 1,
 *            §5.1 eq. 9-10).
 * and, for the runtime block size only, the "DFlash" wiki page (Ablations).
 *
 * Conventions
 * -----------
 * - Matrices are row-major [out_features, in_features] (y = W x), element
 *   type given by dflash_config.dtype (fp32 or bf16).  Norm scales are fp32.
 * - Every call is ordered on the CUDA stream given to dflash_init.  A call
 *   whose outputs are host pointers returns after the results are on the host;
 *   a call whose outputs are device pointers returns without synchronising.
 * - Token arrays may be host or device memory; the library asks the CUDA
 *   runtime which one a pointer is.
 * - No call throws, aborts or traps.  Each returns a dflash_status; the text
 *   of the last failure is available from dflash_last_error.  A call that
 *   fails a precondition changes no state.
 * - Device-side checks (for example a token id outside [0, vocab) passed in
 *   device memory) never fault: they record an error word that the next
 *   synchronising call turns into DFLASH_E_DEVICE_CHECK.
 * - One session serves one host thread at a time (calls on a ctx must not
 *   overlap); separate sessions are independent and may be driven from
 *   different threads.  dflash_init's error text is kept per thread.
 */
#ifndef DFLASH_H
#define DFLASH_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    DFLASH_OK = 0,
    DFLASH_E_INVAL = 1,        /* bad argument or inconsistent configuration */
    DFLASH_E_NOMEM = 2,        /* a device allocation failed */
    DFLASH_E_CUDA = 3,         /* a CUDA runtime call failed */
    DFLASH_E_STATE = 4,        /* call out of order (verify before draft, draft before prefill, ...) */
    DFLASH_E_CAPACITY = 5,     /* a sequence would grow past max_seq_len, or the KV page pool is full */
    DFLASH_E_TIMEOUT = 6,      /* a bounded device-side wait ran out */
    DFLASH_E_DEVICE_CHECK = 7  /* a device-side argument check failed */
} dflash_status;

enum { DFLASH_DTYPE_F32 = 0, DFLASH_DTYPE_BF16 = 1 };

/* Flags (dflash_config.flags). */
enum {
    DFLASH_FLAG_KEEP_LOGITS = 1, /* keep fp32 logits of the last prefill / draft / verify for dflash_inspect */
    DFLASH_FLAG_PROFILE = 2,     /* time every kernel class with CUDA events (see DFLASH_INSPECT_PROFILE) */
    DFLASH_FLAG_NO_GRAPHS = 4    /* launch every kernel directly instead of replaying captured CUDA graphs */
};

/* Kernel classes reported by DFLASH_INSPECT_PROFILE. */
enum {
    DFLASH_K_GEMM_QKV = 0,     /* fused q/k/v projection (target and draft layers) */
    DFLASH_K_GEMM_O = 1,       /* attention output projection + residual */
    DFLASH_K_GEMM_GATE_UP = 2, /* SwiGLU gate/up projection */
    DFLASH_K_GEMM_DOWN = 3,    /* SwiGLU down projection + residual */
    DFLASH_K_GEMM_HEAD = 4,    /* shared LM head */
    DFLASH_K_GEMM_FC = 5,      /* context fusion W_c */
    DFLASH_K_GEMM_CTX_KV = 6,  /* context key/value projection of the draft layers */
    DFLASH_K_ATTENTION = 7,
    DFLASH_K_NORM = 8,
    DFLASH_K_ROPE_STORE = 9,
    DFLASH_K_SWIGLU = 10,
    DFLASH_K_ARGMAX = 11,
    DFLASH_K_OTHER = 12,
    DFLASH_K_SAMPLING = 13,    /* filtered laws, draws and acceptance of the sampled round */
    DFLASH_K_COUNT = 14
};

/* One kernel class in the profile: launches, summed device time (CUDA events
 * bracketing each launch on the session stream), and the algorithmic bytes
 * moved and flops performed by those launches. */
typedef struct {
    int64_t launches;
    double ms;
    double bytes;
    double flops;
} dflash_profile_entry;

enum { DFLASH_MAX_CTX_LAYERS = 16 };

/* Device allocator used for every library-owned buffer.  Returns NULL on
 * failure.  When both are NULL the library uses cudaMalloc / cudaFree. */
typedef void* (*dflash_alloc_fn)(size_t bytes, void* user);
typedef void (*dflash_free_fn)(void* ptr, void* user);

typedef struct {
    int32_t dtype;             /* DFLASH_DTYPE_F32 or DFLASH_DTYPE_BF16 */
    int32_t vocab;             /* V */
    int32_t d_model;           /* d; multiple of 64 */
    int32_t n_heads;           /* H query heads */
    int32_t n_kv_heads;        /* H_kv; H % H_kv == 0 */
    int32_t head_dim;          /* 64 or 128 */
    int32_t ffn;               /* SwiGLU hidden size F; multiple of 64 */
    int32_t target_layers;     /* L_t */
    int32_t target_qk_norm;    /* 1: per-head RMSNorm of q and k in target layers */
    int32_t draft_layers;      /* L_d (the drafter always normalises q and k per head) */
    int32_t block_size;        /* B: anchor + B-1 mask positions; 1 <= B <= 32 */
    int32_t n_ctx_layers;      /* k target layers whose hidden states form the context feature */
    int32_t ctx_layer_ids[DFLASH_MAX_CTX_LAYERS]; /* 0-based target layers, residual after the layer */
    int32_t mask_token;        /* id embedded at the B-1 mask positions */
    int32_t max_batch;         /* sequences per session */
    int32_t max_seq_len;       /* longest sequence: prompt + generated + B */
    int32_t flags;             /* DFLASH_FLAG_* */
    float rms_eps;             /* RMSNorm epsilon */
    double rope_theta;         /* RoPE base */
    dflash_alloc_fn alloc;     /* optional allocator (see above) */
    dflash_free_fn free;
    void* alloc_user;
    int64_t kv_pool_tokens;    /* KV cache capacity shared by the batch, in tokens (rounded up to
                                  64-token pages); 0 = max_batch * max_seq_len */
} dflash_config;

/* One decoder layer, device pointers.  wq, wk, wv, w_gate and w_up are read
 * only inside dflash_init, which packs them into library-owned matrices (one
 * [q; k; v] projection, and in bf16 gate and up interleaved in 64-row tiles
 * for the fused SwiGLU), so they may be freed afterwards.  wo and w_down are
 * borrowed: every call reads them in place, so they must stay allocated and
 * unchanged until dflash_destroy, and be 16-byte aligned.  Norm scales are
 * copied. */
typedef struct {
    const void* wq;            /* [H*hd, d] */
    const void* wk;            /* [H_kv*hd, d] */
    const void* wv;            /* [H_kv*hd, d] */
    const void* wo;            /* [d, H*hd] */
    const void* w_gate;        /* [F, d] */
    const void* w_up;          /* [F, d] */
    const void* w_down;        /* [d, F] */
    const float* attn_norm;    /* [d] */
    const float* mlp_norm;     /* [d] */
    const float* q_norm;       /* [hd]; NULL for target layers without QK-norm */
    const float* k_norm;       /* [hd]; NULL for target layers without QK-norm */
} dflash_layer_weights;

/* Target decoder plus drafter.  The drafter shares the target's embedding
 * table and LM head ([digest] Method, Training §4.2 step 6; Paper vs code
 * "Embedding and head").  embed, head and fc are borrowed like wo and w_down
 * (in place until dflash_destroy, 16-byte aligned). */
typedef struct {
    const void* embed;                     /* [V, d] */
    const void* head;                      /* [V, d] */
    const float* final_norm;               /* [d] */
    const dflash_layer_weights* target;    /* host array of target_layers entries */
    const void* fc;                        /* W_c [d, k*d] (context fusion, [review] §5.1 eq. 9) */
    const float* fc_norm;                  /* [d] */
    const dflash_layer_weights* draft;     /* host array of draft_layers entries */
    const float* draft_norm;               /* [d] drafter's final RMSNorm */
} dflash_weights;

typedef struct {
    int64_t rounds;            /* draft+verify rounds run by dflash_generate */
    int64_t tokens;            /* tokens emitted, first tokens included */
    int64_t accepted;          /* accepted drafts, summed over sequences and rounds */
    double prefill_ms;         /* device time, CUDA events on the session stream */
    double draft_ms;           /* summed over rounds */
    double verify_ms;          /* summed over rounds */
    int64_t kernel_launches;   /* kernels this session has launched */
} dflash_stats;

typedef struct dflash_ctx dflash_ctx; /* opaque; owned by the library */

/* Create a session: validate cfg, allocate the paged target KV cache and the
 * draft context cache (one pool of kv_pool_tokens / 64 pages of 64 tokens,
 * shared by the batch: a sequence takes pages from the pool as it grows, so
 * a ragged batch needs only the sum of its lengths, and every page returns to
 * the pool at the next prefill), all round buffers for max_batch sequences of
 * up to max_seq_len tokens (nothing is allocated later), and pack the q/k/v
 * and gate/up matrices into the library's layout.  Those packed copies are the session's only weight
 * memory: (H + 2 H_kv) hd d + 2 F d elements per layer, about 13 of the 19.7 GB
 * of a Qwen3-8B-shaped target with its 5-layer drafter; the caller's wq, wk, wv,
 * w_gate and w_up may be freed once this returns, and every other matrix is
 * used in place.  cuda_stream is a cudaStream_t (NULL = legacy default stream).
 * Errors: E_INVAL (cfg, a NULL or misaligned borrowed weight), E_NOMEM, E_CUDA.
 * *out is NULL on failure. */
dflash_status dflash_init(const dflash_config* cfg, const dflash_weights* w, void* cuda_stream,
                          dflash_ctx** out);

/* Target prefill of a new batch ([digest] greedy decoding-round pseudocode,
 * prefill and fuse steps; [review] §5.1): a causal forward over each prompt,
 * the first token = argmax of the last row, and the context feature
 * RMSNorm(W_c [h_l1; ...; h_lk]) of every prompt position injected as keys and
 * values into every draft layer.  Afterwards each sequence's committed length
 * n_i = prompt_lens[i] and its anchor is its first token.
 * prompt_lens: host [batch]; prompt_tokens: host, concatenated (sum of lens);
 * first_tokens: host [batch] output.
 * Errors: E_INVAL (batch outside [1, max_batch], a length < 1, a token outside
 * [0, V)), E_CAPACITY (length + block_size > max_seq_len, or the KV page pool
 * cannot hold every prompt + block_size), E_CUDA. */
dflash_status dflash_prefill(dflash_ctx* ctx, int32_t batch, const int32_t* prompt_lens,
                             const int32_t* prompt_tokens, int32_t* first_tokens);

/* Prefill of a batch whose prompts begin with the same prefix_len tokens (a
 * system prompt): dflash_prefill on prompts prefix + own tokens, with the
 * prefix computed and stored once.  The whole 64-token pages of the prefix are
 * shared by every sequence's page table (its remaining tokens are prefilled
 * with each prompt), the prompts' own tokens run in ragged batched passes, and
 * until the next prefill the rounds attend to the shared keys once for the
 * batch (dflash_shared_prefix_attention) where that pays: behind 1024 shared
 * keys or more.
 * prefix: host [prefix_len]; prompt_lens: host [batch], each >= 1, without the
 * prefix; prompt_tokens: host, concatenated; first_tokens: host [batch] output.
 * The first call allocates the attention's workspace (kept until
 * dflash_destroy).  Errors: as dflash_prefill, with lengths prefix_len +
 * prompt_lens[i]; E_INVAL (prefix_len < 0, a prefix token outside [0, V)),
 * E_NOMEM. */
dflash_status dflash_prefill_shared(dflash_ctx* ctx, int32_t batch, int32_t prefix_len, const int32_t* prefix,
                                    const int32_t* prompt_lens, const int32_t* prompt_tokens, int32_t* first_tokens);

/* Set the block size B of the following rounds to block_size, between 1 and
 * the configured block size (the drafter's training block).  A drafter trained
 * at one block size still drafts well at a smaller one, and a smaller block
 * is cheaper to verify when the target is compute-bound at large batch
 * ("DFlash" wiki, Ablations: block size; [digest] Pitfalls, on §5.5.4 and tab. 8).
 * Weights, caches and committed lengths are unchanged; a pending context
 * append keeps the block size of the verify that produced it.  The sizes of
 * every round array (draft_tokens [batch, B-1], the sampled calls' uniforms,
 * dflash_inspect's per-row items) follow the new B from the next draft on,
 * and dflash_inspect's kept rows of earlier rounds are read with the current B.
 * Allowed before a prefill and between a verify and the next draft.
 * Errors: E_INVAL (ctx NULL or block_size outside [1, configured B]),
 * E_STATE (a draft awaits its verify). */
dflash_status dflash_set_block_size(dflash_ctx* ctx, int32_t block_size);

/* The block size of the next round (-1 for a NULL ctx). */
int32_t dflash_block_size(const dflash_ctx* ctx);

/* One drafting pass ([digest] Inference steps 2-3 and the draft-layer
 * pseudocode; [review] §5.1 eq. 10).  First appends the context features of
 * the anchor and accepted drafts of the previous verify (a_i + 1 rows per
 * sequence), then runs the drafter once over [anchor, MASK x (B-1)] at
 * positions n_i .. n_i+B-1, with bidirectional attention over
 * [context K/V ; block K/V], and writes the argmax of the shared head on the
 * B-1 mask rows.  The stored context entries are not modified.
 * draft_tokens: [batch, B-1] int32, host or device.
 * Errors: E_STATE (no prefill, or a draft not yet verified), E_CAPACITY, E_CUDA. */
dflash_status dflash_draft_block(dflash_ctx* ctx, int32_t* draft_tokens);

/* Verify a proposal with one causal target pass over [anchor, d_1..d_{B-1}]
 * at positions n_i .. n_i+B-1 ([digest] Inference step 4; [review] §4.1,
 * Algorithm 1).  Accepts the longest prefix with d_j equal to the target's
 * argmax at the position before it (a_i drafts), sets bonus_i to the target's
 * argmax after that prefix, keeps target cache entries for the anchor and the
 * a_i accepted drafts only (n_i += a_i + 1), and makes bonus_i the next
 * anchor.  The proposal need not come from dflash_draft_block: any tokens in
 * [0, V) are verified exactly.
 * draft_tokens: [batch, B-1] int32 input; accepted, bonus: [batch] int32
 * outputs; each host or device.
 * Errors: E_STATE (no dflash_draft_block since the last verify), E_INVAL
 * (host token outside [0, V)), E_DEVICE_CHECK (device token outside [0, V),
 * reported at the next synchronising call), E_CUDA. */
dflash_status dflash_verify(dflash_ctx* ctx, const int32_t* draft_tokens, int32_t* accepted,
                            int32_t* bonus);

/* Temperature sampling (T > 0): speculative rejection sampling ([review] §4.2
 * eq. 6-8 and Algorithm 1 steps 2-3, 7-8 and 10; [digest] Paper vs code
 * "Sampling rule").  The method's random numbers are inputs: every draw is
 * the lowest token z whose cumulative weight exceeds u * total weight, for a
 * caller-supplied uniform u in [0, 1).  Every law, the drafter's and the
 * target's, is filtered by the setting of dflash_set_sampling_filter (off by
 * default).  The vocabulary must fit the sampling kernels (each of up to 8
 * CTAs of a row stages its share of the row in shared memory: about 390K
 * tokens), else E_INVAL.
 *
 * dflash_draft_block_sampled: as dflash_draft_block, then the proposal of
 * mask row j is drawn from q_j = softmax(draft logits_j / T), filtered, with
 * u_draft[s*(B-1) + j-1]; the laws q are kept for the next verify.
 * u_draft: [batch, B-1] float, host (each in [0, 1), else E_INVAL) or device
 * (clamped to [0, 1)); draft_tokens: [batch, B-1] int32 output, host or device.
 * Errors: as dflash_draft_block, plus E_INVAL (T not positive and finite).
 *
 * dflash_verify_sampled: one causal target pass as dflash_verify; with
 * p_j = softmax(verify logits_j / T), filtered, proposal j (block row j+1) is accepted
 * while u_verify[s*B + j] < min(1, p_j(y)/q_{j+1}(y)) (where q_{j+1}(y) = 0:
 * always if p_j(y) > 0, else never); at the first rejection
 * the emitted token is drawn from [p_a - q_{a+1}]_+ (normalised), else from
 * p_{B-1}, with u_verify[s*B + B-1].  Caches keep the anchor and the a_i
 * accepted rows (n_i += a_i + 1); the emitted token is the next anchor.
 * u_verify: [batch, B] float (host or device, as above); draft_tokens:
 * [batch, B-1] int32 input (the laws are those of the preceding sampled draft);
 * accepted, emitted: [batch] int32 outputs, host or device.
 * Errors: E_STATE (no dflash_draft_block_sampled since the last verify),
 * E_INVAL (T, NULL, host token or uniform out of range), E_DEVICE_CHECK
 * (device token outside [0, V): treated as a rejection), E_CUDA. */
/* Top-k / top-p filter of the sampled round's laws ([digest] Paper vs code
 * "Sampling rule": they apply to both the draft and the target
 * distributions).  After the temperature, tokens rank by logit, highest
 * first, equal logits in increasing id; top-k keeps the first top_k of them
 * (0: all); top-p then keeps each token whose mass ranked before it, under
 * the top-k law renormalised, is below top_p (1: all); the kept tokens'
 * probabilities are renormalised, and eq. 6-8 apply to the filtered laws.
 * The GPU takes each mass in fp32 and sums them exactly in 2^-32 fixed point
 * (relative to the row's largest probability), so a token whose preceding
 * mass is within about 1e-6 of top_p may fall on either side; the kept set
 * is the same on every run.  Applies from the next
 * sampled draft on; allowed whenever no draft awaits its verify.
 * Errors: E_INVAL (ctx NULL, top_k < 0, top_p outside (0, 1]), E_STATE
 * (between a draft and its verify), E_CUDA. */
dflash_status dflash_set_sampling_filter(dflash_ctx* ctx, int32_t top_k, float top_p);

/* Penalties and biases of the target's logits (the rule of
 * dflash_process_logits), per sequence slot: host arrays of max_batch values
 * (bias lists [max_batch][bias_width], id < 0: unused), copied.  NULL arrays
 * are 1 / 0 / 0 and no bias; rules NULL turns them off.  They apply from the
 * next prefill on: to the first token and to every verified row, greedy and
 * sampled, where row j of a block follows the committed tokens, the anchor and
 * the first j drafts; so the emitted stream is that of decoding token by token
 * under the same rules.  The drafter's laws are not changed (a proposal may
 * come from any law).  The temperature and the filter act on the result.
 * Logits kept for dflash_inspect are those before the rules.
 * Errors: E_INVAL (repetition outside [2^-126, 2^126], a value not finite (a
 * bias may be -inf), an id >= V, bias_width outside [0, 4096]), E_NOMEM. */
typedef struct {
    const float* repetition;
    const float* presence;
    const float* frequency;
    int32_t bias_width;
    const int32_t* bias_ids;
    const float* bias_values;
} dflash_logit_rules;
dflash_status dflash_set_logit_rules(dflash_ctx* ctx, const dflash_logit_rules* rules);

/* Token masks (grammar states) of the next target pass alone: between a draft
 * and its verify, of that verify (rows = batch * B, row j of a block masks the
 * token after its first j drafts; a prefill in the verify's place drops them);
 * otherwise of the next prefill's first tokens (rows = its batch; a draft drops
 * them).  masks: [n_masks][ceil(V / 32)] bit sets, host or device, copied (bit
 * v % 32 of word v / 32: token v is allowed); mask_index: [rows], host or
 * device, < 0: no mask, as is a device index >= n_masks (a host one is
 * refused).  n_masks 0 drops the masks; a refused call leaves those set before.
 * Host arrays are the caller's again when the call returns (from page-locked
 * memory it waits for the stream); device arrays must stay until the copy, on
 * the session's stream, has run.
 * A row that the masks and biases leave without a token is E_DEVICE_CHECK at
 * the next synchronising call.
 * Errors: E_INVAL (sizes, NULL, n_masks above max_batch * block_size, a host
 * index >= n_masks), E_NOMEM, E_CUDA. */
dflash_status dflash_set_token_masks(dflash_ctx* ctx, int32_t n_masks, const uint32_t* masks, int32_t rows,
                                     const int32_t* mask_index);

dflash_status dflash_draft_block_sampled(dflash_ctx* ctx, float temperature, const float* u_draft,
                                        int32_t* draft_tokens);
dflash_status dflash_verify_sampled(dflash_ctx* ctx, float temperature, const int32_t* draft_tokens,
                                    const float* u_verify, int32_t* accepted, int32_t* emitted);

/* The drafter's training forward, loss value only ([review] §6 eq. 12 and
 * Algorithm 2; [digest] Training §4.2).  The target runs once, causally, over
 * the clean sequence tokens[0..n_tokens); for each anchor a the block
 * [tokens[a], MASK x (B-1)] at positions a .. a+B-1 attends to the fused
 * target features of positions < a and to itself; the loss is the mean over
 * anchors of sum_{k=1}^{B-1} exp(-(k-1)/lambda) * -log q_k(tokens[a+k]).
 * All blocks run in one drafter pass: block i uses sequence slot i+1, whose
 * page table shares slot 0's context pages below its anchor's page.
 * tokens: host [n_tokens]; anchors: host [n_anchors], each in [1, n_tokens-B];
 * loss: host float.  Needs B >= 2, n_anchors + 1 <= max_batch and
 * n_tokens + B <= max_seq_len.  Leaves the session empty (prefill before the
 * next round).  Errors: E_INVAL (NULL, anchor range, lambda <= 0, B < 2),
 * E_CAPACITY, E_DEVICE_CHECK, E_CUDA. */
dflash_status dflash_train_forward(dflash_ctx* ctx, int32_t n_tokens, const int32_t* tokens, int32_t n_anchors,
                                   const int32_t* anchors, float lambda, float* loss);

/* Greedy speculative generation ([digest] greedy decoding-round pseudocode):
 * prefill, then rounds of draft_block + verify until every sequence has
 * max_new_tokens tokens (the first token counts); each sequence's output is
 * cut to max_new_tokens.  out_tokens: host [batch, max_new_tokens];
 * out_lens: host [batch] (always max_new_tokens); stats may be NULL. */
dflash_status dflash_generate(dflash_ctx* ctx, int32_t batch, const int32_t* prompt_lens,
                              const int32_t* prompt_tokens, int32_t max_new_tokens, int32_t* out_tokens,
                              int32_t* out_lens, dflash_stats* stats);

/* Inspection of session state (for tests and profiling).  Copies into host
 * memory; synchronises the stream.  *written receives the byte count.
 *   DFLASH_INSPECT_LENGTHS        int32 [batch]: committed length n_i
 *   DFLASH_INSPECT_ANCHORS        int32 [batch]
 *   DFLASH_INSPECT_POSTERIOR      int32 [batch, B]: target argmax of the last verify
 *   DFLASH_INSPECT_TARGET_K/V     dtype [n_seq, H_kv, hd] of (seq, layer), n_seq committed rows
 *   DFLASH_INSPECT_DRAFT_K/V      same for the draft context cache
 *   DFLASH_INSPECT_LOGITS_PREFILL fp32 [batch, V]   (needs DFLASH_FLAG_KEEP_LOGITS)
 *   DFLASH_INSPECT_LOGITS_DRAFT   fp32 [batch, B, V] (all B rows of the last draft)
 *   DFLASH_INSPECT_LOGITS_VERIFY  fp32 [batch, B, V]
 *   DFLASH_INSPECT_STATS          dflash_stats
 *   DFLASH_INSPECT_HIDDEN_VERIFY  fp32 [batch, B, d]: final residual of the last verify
 *   DFLASH_INSPECT_PROFILE        dflash_profile_entry [DFLASH_K_COUNT] accumulated since the last reset
 * Errors: E_INVAL (unknown item, seq/layer out of range, bytes too small). */
enum {
    DFLASH_INSPECT_LENGTHS = 1,
    DFLASH_INSPECT_ANCHORS = 2,
    DFLASH_INSPECT_POSTERIOR = 3,
    DFLASH_INSPECT_TARGET_K = 4,
    DFLASH_INSPECT_TARGET_V = 5,
    DFLASH_INSPECT_DRAFT_K = 6,
    DFLASH_INSPECT_DRAFT_V = 7,
    DFLASH_INSPECT_LOGITS_PREFILL = 8,
    DFLASH_INSPECT_LOGITS_DRAFT = 9,
    DFLASH_INSPECT_LOGITS_VERIFY = 10,
    DFLASH_INSPECT_STATS = 11,
    DFLASH_INSPECT_HIDDEN_VERIFY = 12,
    DFLASH_INSPECT_PROFILE = 13,       /* dflash_profile_entry [DFLASH_K_COUNT]; needs DFLASH_FLAG_PROFILE */
    DFLASH_INSPECT_PROFILE_RESET = 14  /* clears the profile; copies nothing */
};
dflash_status dflash_inspect(dflash_ctx* ctx, int32_t what, int32_t seq, int32_t layer, void* host_dst,
                             size_t bytes, size_t* written);

/* Turn kernel-class timing on (1) or off (0) for this session.  While on,
 * every kernel class launch is bracketed by CUDA events on the session stream
 * and its algorithmic bytes and flops are recorded; read the totals with
 * DFLASH_INSPECT_PROFILE.  Timing adds event records between launches, so
 * headline timings are taken with it off.  Errors: E_INVAL (ctx NULL), E_CUDA. */
dflash_status dflash_set_profiling(dflash_ctx* ctx, int32_t on);

/* Maximum scratch, in bytes, of dflash_head_argmax_noalloc. */
enum { DFLASH_NOALLOC_SCRATCH_BYTES = 16 << 20 };

/* Shared-head argmax for callers that cannot allocate device memory.
 *
 * The paper has no counterpart to this call; it exists for deployment.  Some
 * callers cannot call cudaMalloc or any allocator: code running inside
 * another framework's fixed memory pool, an embedded runtime whose allocator
 * is locked, or a process whose device memory budget is settled before this
 * library is loaded.  Such a caller cannot create a session (dflash_init
 * allocates), but can still pick tokens from final hidden states with this
 * call: out[r] = argmax_v ( RMSNorm(x[r]) * norm_w ) . head[v], ties to the
 * lowest id.  It queues three kernels - an RMSNorm of the rows into the
 * element type of head, the head GEMM (tensor cores for bf16), and a row
 * argmax - plus a check of its error word.  dflash_verify computes the same
 * quantity with the norm and the argmax fused into its head GEMM; in bf16 the
 * two can pick different tokens where the two largest logits lie within
 * bf16 rounding of each other.
 *
 * Arguments (all device pointers except cuda_stream):
 *   dtype   DFLASH_DTYPE_F32 or DFLASH_DTYPE_BF16: element type of head
 *   x       fp32 [rows, d_model] hidden states (not modified)
 *   norm_w  fp32 [d_model] RMSNorm scale;  eps: RMSNorm epsilon (> 0)
 *   head    [vocab, d_model] LM head
 *   out     int32 [rows] token ids (written)
 *   cuda_stream  cudaStream_t the kernels are queued on (NULL = legacy default)
 * x, norm_w and head must be 16-byte aligned.  The call queues its kernels and
 * returns without synchronising.
 *
 * Memory: it allocates nothing.  Its intermediates (the normalised rows and
 * the fp32 logits, rows * (d_model * elem + vocab * 4) bytes plus alignment)
 * and a device error word live in one fixed array of
 * DFLASH_NOALLOC_SCRATCH_BYTES (16 MiB) that every GPU which loads this
 * library holds until the process exits.  Larger requests are rejected with
 * DFLASH_E_INVAL before anything is queued (for example at vocab 151936 and
 * d_model 4096 in bf16, up to 27 rows fit).
 * The first call on each device looks up that array's device address with
 * the device current; make that first call before any CUDA stream capture.
 * All calls share the array and it keeps the last call's contents; each call
 * clears its error word first, and nothing else needs to start at zero.
 * Calls that overlap on the GPU (on different streams, or from different
 * threads) race on the array: order them.
 * Errors: E_INVAL (NULL or misaligned pointer, bad sizes, request above the
 * maximum), E_CUDA (a launch failed or a kernel could not be prepared); the
 * text is available from dflash_last_error(NULL).  Because the call does not
 * synchronise, a failure on the device is reported in the output instead: if
 * a bounded device-side wait inside the head GEMM ran out (it should never),
 * every out[r] is -1, which is not a token id. */
dflash_status dflash_head_argmax_noalloc(int32_t dtype, const float* x, const float* norm_w, float eps,
                                         const void* head, int32_t rows, int32_t d_model, int32_t vocab,
                                         int32_t* out, void* cuda_stream);

/* ======================================================= serving operators
 * Stateless operators next to the round, on the caller's device memory.  They
 * allocate nothing, keep nothing between calls and never synchronise: each is
 * queued on cuda_stream (NULL = legacy default stream; the stream's device
 * must be current) and may be captured into a CUDA graph.  Argument errors are
 * E_INVAL before anything is queued, with the text in dflash_last_error(NULL);
 * what only the device can see is reported in an output, as each call says.
 * KV pages hold 64 tokens: a cache is [pages][H_kv][64][hd] (one layer), page
 * p token t of KV head h at ((p * H_kv + h) * 64 + t) * hd.  Sequences per
 * call: at most DFLASH_OPS_MAX_BATCH. */
enum { DFLASH_OPS_MAX_BATCH = 2048 };

/* Page tables and slot maps of a batch from its request lengths.  Request s
 * has kv_lens[s] tokens cached and appends new_lens[s].  With
 * old = ceil(kv / 64) and need = ceil((kv + new) / 64):
 *   table_out[s][j]  = table[s][j] for j < old; the next page of free_pages
 *                      (requests in order, free_pages[*used] first) for
 *                      old <= j < need; scratch_page for need <= j < width
 *   q_start[s]       = sum of new_lens before s; q_start[batch] = the total T
 *   row r < T (token j of request s): row_seq = s, row_pos = base_pos + kv + j,
 *                      slot = 64 * page + token, page = table_out[s][(kv+j)/64]
 *   rows T <= r < rows: row_seq = row_pos = -1, slot = -1
 *   used_out         = *used + pages taken
 * free_pages NULL: the caller's table already holds every page; nothing is
 * taken and table_out may be NULL.
 * status (device): 0, or a sum of 1 (the pool has too few pages), 2 (a request
 * needs more than width pages), 4 (T > rows), 8 (a negative length or *used).
 * When it is not 0 nothing is taken: table_out is not written, used_out =
 * *used, q_start is all 0 and every row is -1.
 * table_out may be table and used_out may be used (in place); no other overlap.
 * Rows of table and table_out are ld_table / ld_out entries apart.
 * Errors: E_INVAL (sizes, NULL), E_CUDA. */
typedef struct {
    int32_t batch;             /* 1 .. DFLASH_OPS_MAX_BATCH */
    int32_t width;             /* table entries per request */
    int32_t rows;              /* entries of row_seq, row_pos and slots */
    int32_t n_free;            /* entries of free_pages */
    int32_t base_pos;          /* position of a request's token 0 (a shared prefix before it) */
    int32_t scratch_page;
    int64_t ld_table;
    int64_t ld_out;
    const int32_t* kv_lens;    /* [batch] */
    const int32_t* new_lens;   /* [batch] */
    const int32_t* table;      /* [batch][width] */
    const int32_t* free_pages; /* [n_free] or NULL */
    const int32_t* used;       /* [1]: pages of free_pages taken before; NULL when free_pages is */
    int32_t* table_out;        /* [batch][width] */
    int32_t* used_out;         /* [1] */
    int32_t* q_start;          /* [batch + 1] */
    int32_t* row_seq;          /* [rows] or NULL */
    int32_t* row_pos;          /* [rows] or NULL */
    int64_t* slots;            /* [rows] or NULL */
    int32_t* status;           /* [1] */
} dflash_kv_tables_args;
dflash_status dflash_kv_tables(const dflash_kv_tables_args* args, void* cuda_stream);

/* Attention of a batch whose sequences begin with the same prefix.  The
 * prefix's keys and values (prefix_len tokens in prefix_pages, any length) are
 * read once for the whole batch; each sequence's own keys (kv_lens[s] tokens
 * in table[s], the rows of this call included) follow it.  Rows
 * q_start[s] .. q_start[s+1]-1 of q belong to sequence s; row j of its m rows
 * sees the whole prefix and its own keys i < kv_lens[s] - m + j + 1 (causal)
 * or i < kv_lens[s].  out = softmax(scale q.k) v per query head h over KV head
 * h / (H / H_kv); lse (optional) = natural log of the sum of exp(scale q.k).
 * A row that sees no key gets out = 0 and lse = -inf.  Rows outside
 * [q_start[0], q_start[batch]) are left as they were.  The slots of a page
 * past the last valid token may hold anything; keys and values of valid
 * tokens must be finite.
 * Device-side checks: a sequence with kv_lens[s] outside [0, 64 * width] gets
 * NaN in its rows' out and lse, one with a page outside [0, n_pages) among its
 * keys in every row that sees the page (rows of the sequence before those may
 * get NaN or their result).  Every row of every sequence gets NaN behind a bad
 * prefix page or a bounded device wait that ran out, every row of q behind a
 * q_start that decreases or leaves [0, rows] or work beyond 2^31 tiles of 64
 * keys.  Nothing is read or written out of range.
 * dtype F32 or BF16 (q, caches and out); head_dim 64 or 128; H at most 1024 and
 * at most 64 times H_kv; q, the caches and out 16-byte aligned, ld_q and ld_out
 * multiples of 16 bytes.  out may be q (in place, with one row stride).
 * The scores, the softmax and the accumulation are fp32; in BF16 each softmax
 * weight is rounded to bf16 for the product with v, or with the flag
 * DFLASH_ATTENTION_WEIGHT_PAIRS held as a sum of two bf16 values (16 bits), as
 * the sessions hold it; F32 calls round none and ignore the flag.
 * workspace: 16-byte aligned device memory of at least
 * dflash_shared_prefix_workspace() bytes, used by this call only until it has
 * finished: calls that may overlap need workspaces of their own.
 * Errors: E_INVAL, E_CUDA. */
enum { DFLASH_ATTENTION_WEIGHT_PAIRS = 1 };
typedef struct {
    int32_t dtype;
    int32_t n_heads;
    int32_t n_kv_heads;
    int32_t head_dim;
    int32_t batch;             /* 1 .. DFLASH_OPS_MAX_BATCH */
    int32_t rows;              /* rows of q, out and lse */
    int32_t n_pages;           /* pages of each cache */
    int32_t prefix_len;        /* tokens; prefix_pages holds ceil(prefix_len / 64) entries */
    int32_t width;             /* table entries per sequence */
    int32_t causal;
    float scale;               /* > 0 */
    union {
        int32_t flags;         /* 0, or DFLASH_ATTENTION_WEIGHT_PAIRS */
        int32_t reserved;
    };
    int64_t ld_q;              /* elements between rows of q (H * hd when contiguous) */
    int64_t ld_out;            /* elements between rows of out */
    int64_t ld_table;
    const void* q;             /* [rows][H][hd] */
    const void* k_cache;       /* [n_pages][H_kv][64][hd] */
    const void* v_cache;
    const int32_t* prefix_pages;
    const int32_t* table;      /* [batch][width]: sequence s's own keys 64 j .. 64 j + 63 */
    const int32_t* kv_lens;    /* [batch] */
    const int32_t* q_start;    /* [batch + 1] */
    void* out;                 /* [rows][H][hd] */
    float* lse;                /* [rows][H] or NULL */
    void* workspace;
    size_t workspace_bytes;
} dflash_shared_prefix_args;
dflash_status dflash_shared_prefix_attention(const dflash_shared_prefix_args* args, void* cuda_stream);
/* Bytes of workspace for a call with these sizes (any lengths within them, and
 * any smaller batch or rows); 0 for sizes that the call refuses. */
size_t dflash_shared_prefix_workspace(int32_t dtype, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                                      int32_t batch, int32_t rows);

/* Penalties for repeated tokens, biases and grammar masks on logits.  Rows are
 * sequence-major, rows_per_seq of them each; row j of sequence s continues
 * history[s][0 .. hist_lens[s]) and the first j of its drafts.  For token v
 * with c = its count among the tokens after the prompt (drafts included), in
 * this order:
 *   x = logits[v]
 *   seen in the prompt or after it:  x = x > 0 ? x / repetition : x * repetition
 *   x = x - frequency * c;   c > 0:  x = x - presence
 *   x = x + bias_values of the last entry of bias_ids[s] that is v
 *   bit v of the row's mask is 0:    x = -inf
 * in fp32, rounded once to the logits' type; x / repetition is the product of x
 * and the penalty's reciprocal, each rounded to fp32, for penalties between
 * 2^-126 and 2^126 (beyond, the reciprocal overflows or loses bits).  A mask
 * that allows no token
 * leaves a row of -inf.  Ids outside [0, vocab) in history, drafts and
 * bias_ids are skipped (padding); a mask_index outside [0, n_masks) means no
 * mask; hist_lens is clamped to [0, hist_width], prompt_lens to [0, hist_lens].
 * Each of the three groups may be left out: history NULL (no penalties),
 * bias_ids NULL, masks NULL; repetition / presence / frequency NULL are 1 / 0
 * / 0.  out may be logits (in place: only the tokens that change are touched),
 * with no other overlap; rows are ld_logits / ld_out elements apart and what
 * lies behind vocab in a row is not touched.
 * Errors: E_INVAL, E_CUDA. */
typedef struct {
    int32_t dtype;             /* of logits and out: F32 or BF16 */
    int32_t batch;
    int32_t rows_per_seq;      /* 1 .. 32 */
    int32_t vocab;
    int32_t hist_width;        /* columns of history, at most 2^29 */
    int32_t bias_width;        /* columns of bias_ids and bias_values, at most 2^29 */
    int32_t n_masks;
    int32_t reserved;          /* 0 */
    int64_t ld_logits;
    int64_t ld_out;
    int64_t ld_hist;           /* elements between rows of history */
    int64_t ld_mask;           /* words between masks: at least ceil(vocab / 32) */
    const void* logits;        /* [batch * rows_per_seq][vocab] */
    void* out;
    const int32_t* history;    /* [batch][hist_width] or NULL */
    const int32_t* hist_lens;  /* [batch] */
    const int32_t* prompt_lens; /* [batch]: the first prompt_lens[s] history tokens are the prompt */
    const int32_t* drafts;     /* [batch][rows_per_seq - 1] or NULL (no drafts between the rows) */
    const float* repetition;   /* [batch] or NULL */
    const float* presence;     /* [batch] or NULL */
    const float* frequency;    /* [batch] or NULL */
    const int32_t* bias_ids;   /* [batch][bias_width] or NULL */
    const float* bias_values;  /* [batch][bias_width] */
    const uint32_t* masks;     /* [n_masks][ld_mask] or NULL: bit v % 32 of word v / 32 is 1 when v is allowed */
    const int32_t* mask_index; /* [batch * rows_per_seq] */
} dflash_logits_args;
dflash_status dflash_process_logits(const dflash_logits_args* args, void* cuda_stream);

/* ------------------------------------------------------ trees of drafted tokens
 * A sequence's rows q_start[s] .. q_start[s+1]-1 (m of them) are the nodes of
 * a tree in drafting order: node 0 is the root (the anchor, committed whatever
 * the target says), a node's parent comes before it.  kv_lens[s] counts the
 * sequence's own keys, those of the m nodes, its last, among them: node i is
 * own key kv_lens[s] - m + i.  At most DFLASH_TREE_MAX_NODES nodes a tree.
 * Outputs of these calls, of the page calls and of the log probabilities
 * overlap neither one another nor an input, but where a call says so. */
enum { DFLASH_TREE_MAX_NODES = 1024 };

/* Masks, depths and positions of trees from their nodes' parents.
 *   masks[r]   = bit i % 32 of word i / 32 set for node r itself and each of
 *                its ancestors i, `words` words; the others 0
 *   depth[r]   = links between node r and its root
 *   row_pos[r] = base_pos + kv_lens[s] - m + depth[r]
 * parents[r] is the parent's number in its tree or -1 (a root).  A kv_lens[s] below
 * m means that the first m - kv_lens[s] nodes lie before the sequence's first own key:
 * dflash_tree_attention takes such a length (they have no key), and here their positions are
 * below base_pos, which has to leave room for them.
 * status[s] (device): 0, or a sum of 1 (a parent that does not come before its
 * child, or below -1), 2 (more nodes than 32 * words or than
 * DFLASH_TREE_MAX_NODES), 4 (q_start decreases or leaves [0, rows]), 8 (with row_pos: a
 * negative kv_lens[s], base_pos + kv_lens[s] - m < 0 or base_pos + kv_lens[s] > 2^31).
 * With 1 or 2 the sequence's rows get masks 0, depth -1 and row_pos -1, with 8 alone
 * a row_pos of -1 beside their masks and depths, with 4 nothing
 * of it is written.  Rows of no sequence are left as they were.
 * Errors: E_INVAL (sizes, NULL), E_CUDA. */
typedef struct {
    int32_t batch;             /* 1 .. DFLASH_OPS_MAX_BATCH */
    int32_t rows;              /* rows of parents, masks, depth and row_pos, at most 2^20 */
    int32_t words;             /* words a mask, at least 1 */
    int32_t base_pos;          /* position of a sequence's first own key (a shared prefix before it) */
    int64_t ld_mask;           /* words between masks */
    const int32_t* parents;    /* [rows] */
    const int32_t* q_start;    /* [batch + 1] */
    const int32_t* kv_lens;    /* [batch]; NULL when row_pos is */
    uint32_t* masks;           /* [rows][ld_mask] */
    int32_t* depth;            /* [rows] or NULL */
    int32_t* row_pos;          /* [rows] or NULL */
    int32_t* status;           /* [batch] */
} dflash_tree_masks_args;
dflash_status dflash_tree_masks(const dflash_tree_masks_args* args, void* cuda_stream);

/* Attention of trees: dflash_shared_prefix_attention (all that it says holds,
 * workspace, flags and an empty prefix included; attn.causal is ignored), but
 * row r of sequence s sees, behind the prefix, its committed keys
 * i < kv_lens[s] - m and of the m nodes' keys those whose bit is set in
 * masks[r] (bit i % 32 of word i / 32 for node i; nodes behind the last word
 * are not seen).  Masks are any sets: dflash_tree_masks makes those of trees.  A
 * row that sees no key gets out = 0 and lse = -inf.  What a node's key and value
 * hold does not matter to a row if no row of its sequence sees the node; the
 * values of nodes that some row sees must be finite, like all valid tokens'.
 * Errors: E_INVAL, E_CUDA. */
typedef struct {
    dflash_shared_prefix_args attn;
    const uint32_t* masks;     /* [attn.rows][ld_mask] */
    int64_t ld_mask;           /* words between masks */
    int32_t words;             /* words a mask, 1 .. 2^20 */
    int32_t reserved;          /* 0 */
} dflash_tree_attention_args;
dflash_status dflash_tree_attention(const dflash_tree_attention_args* args, void* cuda_stream);

/* Greedy acceptance of a verified tree: from the root on, the child that holds
 * the target's choice, the lowest where several do, until none does.
 *   path[s][0 .. accepted[s]] = the nodes kept, root first; behind them -1
 *   accepted[s] = drafts accepted (nodes kept but the root), at most width - 1
 *   bonus[s]    = posterior of the last node kept: the next anchor
 * parents, tokens, posterior: per row, the parent's number in the tree (-1: a
 * root), the drafted token, the target's choice behind the row.  A sequence
 * without rows gets accepted = bonus = -1 and a path of -1.
 * status[s] (device): 1, 2 (more than DFLASH_TREE_MAX_NODES nodes) or 4, as
 * dflash_tree_masks; when not 0, accepted = bonus = -1, path -1.
 * Errors: E_INVAL (sizes, NULL), E_CUDA. */
typedef struct {
    int32_t batch;
    int32_t rows;
    int32_t width;             /* entries of a path, 1 .. DFLASH_TREE_MAX_NODES */
    int32_t reserved;          /* 0 */
    const int32_t* parents;    /* [rows] */
    const int32_t* tokens;     /* [rows] */
    const int32_t* posterior;  /* [rows] */
    const int32_t* q_start;    /* [batch + 1] */
    int32_t* path;             /* [batch][width] */
    int32_t* accepted;         /* [batch] */
    int32_t* bonus;            /* [batch] */
    int32_t* status;           /* [batch] */
} dflash_tree_accept_args;
dflash_status dflash_tree_accept(const dflash_tree_accept_args* args, void* cuda_stream);

/* Keeps the accepted nodes of a cache: in every layer, of keys and values
 * alike, the token of node path[s][j] moves to node j's place, j <=
 * accepted[s], and kv_out[s] = kv_lens[s] - m + accepted[s] + 1.  The places
 * behind hold what they held, to be overwritten.  path must rise strictly, as
 * dflash_tree_accept's does (any other rule of acceptance may fill it).
 * A layer's cache is [n_pages][H_kv][64][hd], layers are ld_layer elements apart.
 * status[s] (device): 0, or a sum of 1 (accepted outside [-1, width), or a path
 * that does not rise within [0, m)), 4 (q_start decreases or is negative), 8
 * (kv_lens outside [m, 64 * width_table]), 16 (a page of a moved token outside
 * [0, n_pages)).  When not 0, nothing of the sequence moves and kv_out =
 * kv_lens.  With accepted[s] = -1 none of the m nodes is kept, the root neither: kv_out =
 * kv_lens - m, with status 0.  That is what a tree gets that dflash_tree_accept refused (its
 * status says so): the whole step of that sequence is taken back, its anchor's key and value
 * are still to be made.  No two sequences may hold the same page among their nodes'.
 * kv_out may not be kv_lens, and the layers of v_cache share no memory with those of k_cache
 * (they may lie between each other).  Errors: E_INVAL (sizes, NULL, caches that overlap), E_CUDA. */
typedef struct {
    int32_t dtype;             /* F32 or BF16 */
    int32_t batch;
    int32_t layers;            /* 1 .. 1024 */
    int32_t n_pages;
    int32_t n_kv_heads;
    int32_t head_dim;          /* a row of a head is a multiple of 16 bytes */
    int32_t width;             /* entries of a path, 1 .. DFLASH_TREE_MAX_NODES */
    int32_t width_table;       /* table entries per sequence */
    int64_t ld_layer;          /* elements between layers (a multiple of 16 bytes) */
    int64_t ld_table;
    void* k_cache;             /* [layers][n_pages][H_kv][64][hd], 16-byte aligned */
    void* v_cache;
    const int32_t* table;      /* [batch][width_table] */
    const int32_t* kv_lens;    /* [batch] */
    const int32_t* q_start;    /* [batch + 1] */
    const int32_t* path;       /* [batch][width] */
    const int32_t* accepted;   /* [batch] */
    int32_t* kv_out;           /* [batch] */
    int32_t* status;           /* [batch] */
} dflash_kv_compact_args;
dflash_status dflash_kv_compact(const dflash_kv_compact_args* args, void* cuda_stream);

/* ------------------------------------------------------ pages held by several
 * refs[p] counts the holders of page p beyond its first: 0 for a free page and
 * for one that a single sequence holds, so pages that dflash_kv_tables hands
 * out need nothing.  The free list is dflash_kv_tables': entries 0 .. *used - 1
 * are taken.  The counts do not say whether a page is free: that the sequences named
 * hold their pages is the caller's to keep. */

/* Sequences that continue others.  Child c continues sequence parents[c] (any
 * number of children a parent) with n = kv_lens[parents[c]] tokens:
 *   table_out[c][j] = the parent's page for j < n / 64, shared (its refs rise
 *                     by one); for n % 64 > 0 entry n / 64 is the next page of
 *                     free_pages (children in order) with the parent's last
 *                     n % 64 tokens copied, keys and values of every layer;
 *                     scratch_page behind
 *   lens_out[c] = n, used_out = *used + pages taken
 * A shared page is full, so neither side writes to it again.
 * status (device): 0, or a sum of 1 (the pool has too few pages), 2 (a parent
 * holds more than width pages), 8 (a negative length or *used, or a parent
 * outside [0, batch)): nothing is taken, table_out, refs and the caches are as
 * they were, lens_out is 0 and used_out = *used; and 16 (a page outside
 * [0, n_pages)) alone: such an entry is copied as it is, counted and copied to
 * or from nowhere, and the rest is done.
 * used_out may be used; table_out may be rows of the same matrix behind table's.
 * No other overlap.  Errors: E_INVAL (sizes, NULL), E_CUDA. */
typedef struct {
    int32_t dtype;
    int32_t batch;             /* sequences of table and kv_lens: 1 .. DFLASH_OPS_MAX_BATCH */
    int32_t children;          /* 1 .. DFLASH_OPS_MAX_BATCH */
    int32_t width;             /* table entries per sequence, parents and children alike */
    int32_t n_free;
    int32_t scratch_page;
    int32_t layers;            /* 1 .. 1024 */
    int32_t n_pages;
    int32_t n_kv_heads;
    int32_t head_dim;
    int64_t ld_layer;
    int64_t ld_table;
    int64_t ld_out;
    void* k_cache;             /* as dflash_kv_compact, or both the same */
    void* v_cache;
    const int32_t* parents;    /* [children] */
    const int32_t* kv_lens;    /* [batch] */
    const int32_t* table;      /* [batch][width] */
    const int32_t* free_pages; /* [n_free] */
    const int32_t* used;       /* [1] */
    int32_t* refs;             /* [n_pages] */
    int32_t* table_out;        /* [children][width] */
    int32_t* lens_out;         /* [children] */
    int32_t* used_out;         /* [1] */
    int32_t* status;           /* [1] */
} dflash_kv_fork_args;
dflash_status dflash_kv_fork(const dflash_kv_fork_args* args, void* cuda_stream);

/* Gives back the pages of sequences that have ended: each of the
 * ceil(kv_lens[s] / 64) pages of the sequences seqs[0 .. n) loses a holder, and a
 * page without one returns to the free list.  Returned pages lie in
 * free_pages[used_out .. *used - 1] in the order of their first mention (seqs in
 * order, then table entries): a release right behind the call that took the pages
 * restores the list.  The tables and lengths of the sequences are the caller's to
 * forget: a sequence ends once.  Of the mentions of one call too many are reported (32),
 * but a later call that names an ended sequence again is taken at its word, and its pages,
 * free or another's by then, go into the list a second time (or, where fewer pages
 * are taken than it returns, status 1).
 * With keep_lens a sequence s lives on with its first keep_lens[s] tokens and
 * gives back the pages behind them, entries ceil(keep_lens[s] / 64) and on: after
 * a step whose tree grew past a page and was cut behind it, kv_lens are the
 * lengths with the tree and keep_lens dflash_kv_compact's kv_out (dflash_kv_tables
 * takes new pages behind ceil(kv / 64), whatever the table holds there).  The page that
 * a cut ends inside (keep_lens[s] below kv_lens[s] and not a multiple of 64) is written to
 * next: behind the call it may have no other holder.  A sequence whose cut meets a shared
 * page can fork itself at the shorter length (dflash_kv_fork copies the page) and end.
 * status (device): 0, or a sum of 1 (more pages return than were taken), 2 (a
 * length above 64 * width), 8 (a negative length, keep_lens outside [0, kv_lens], a
 * *used outside [0, n_free], or a
 * sequence outside [0, batch) or named twice), 16 (a page outside [0, n_pages)
 * or with negative refs), 32 (a page returned by more sequences of the call than hold it), 64 (a
 * cut ends inside a page that others hold).
 * When not 0, nothing changes and used_out = *used.
 * used_out may be used.  Errors: E_INVAL (sizes, NULL), E_CUDA. */
typedef struct {
    int32_t batch;             /* sequences of table and kv_lens: 1 .. DFLASH_OPS_MAX_BATCH */
    int32_t n;                 /* sequences that end: 1 .. DFLASH_OPS_MAX_BATCH */
    int32_t width;             /* table entries per sequence, at most 2^18 */
    int32_t n_free;
    int32_t n_pages;
    int32_t reserved;          /* 0 */
    int64_t ld_table;
    const int32_t* seqs;       /* [n] */
    const int32_t* kv_lens;    /* [batch] */
    const int32_t* table;      /* [batch][width] */
    int32_t* free_pages;       /* [n_free] */
    const int32_t* used;       /* [1] */
    int32_t* refs;             /* [n_pages] */
    int32_t* used_out;         /* [1] */
    int32_t* status;           /* [1] */
    const int32_t* keep_lens;  /* [batch], or NULL: 0 */
} dflash_kv_release_args;
dflash_status dflash_kv_release(const dflash_kv_release_args* args, void* cuda_stream);

/* ------------------------------------------------------ log probabilities
 * Of each row x of logits, with its largest logit m and
 * z_v = (x_v - m) * inv_temperature (fp32; the difference comes before the
 * product, so that rows far from 0 are as exact as others):
 *   lse_parts    = m and L = ln sum_v exp(z_v)
 *   lse          = m * inv_temperature + L, rounded once (infinite where that is
 *                  beyond fp32, while what follows is not)
 *   logprobs[i]  = z_t - L for the row's i-th token t; 0 for a t outside
 *                  [0, vocab) (padding)
 *   ranks[i]     = tokens ahead of t: of a larger logit, or an equal one and a
 *                  lower id; -1 for padding (the logits themselves are compared, without
 *                  the temperature)
 *   entropy      = -sum_v p_v ln p_v, ln p_v = z_v - L
 *   top_ids, top_logprobs = the k likeliest tokens by their logits, likeliest first,
 *                  the lower id first among equal ones
 * Tokens at -inf have probability 0; they are no alternatives: where fewer than k
 * tokens are left, the list ends in id -1 and -inf.  A row of -inf alone has lse =
 * lse_parts = logprobs = -inf and entropy 0.  A row that holds NaN or +inf gets NaN
 * everywhere (but padding's 0), ranks and top_ids -1.
 * Any of the outputs may be NULL.  Rows are ld_logits elements apart.
 * Errors: E_INVAL, E_CUDA. */
enum { DFLASH_LOGPROBS_MAX_TOKENS = 32, DFLASH_LOGPROBS_MAX_TOP = 32 };
typedef struct {
    int32_t dtype;             /* of logits: F32 or BF16 */
    int32_t rows;
    int32_t vocab;
    int32_t n;                 /* tokens a row, 0 .. DFLASH_LOGPROBS_MAX_TOKENS */
    int32_t k;                 /* alternatives a row, 0 .. DFLASH_LOGPROBS_MAX_TOP */
    float inv_temperature;     /* 2^-20 .. 2^20 */
    int64_t ld_logits;
    const void* logits;        /* [rows][vocab] */
    const int32_t* tokens;     /* [rows][n]; NULL when n is 0 */
    float* logprobs;           /* [rows][n] or NULL */
    int32_t* ranks;            /* [rows][n] or NULL */
    float* entropy;            /* [rows] or NULL */
    float* lse;                /* [rows] or NULL */
    int32_t* top_ids;          /* [rows][k] or NULL */
    float* top_logprobs;       /* [rows][k] or NULL */
    float* lse_parts;          /* [rows][2], 8-byte aligned, or NULL */
} dflash_logprobs_args;
dflash_status dflash_token_logprobs(const dflash_logprobs_args* args, void* cuda_stream);

/* Gradient of a loss of those log probabilities and entropies by the logits,
 * with p_v = exp(x_v * inv_temperature - lse), from lse_parts exp(z_v - L), g_i =
 * grad_logprobs[i] (0 for padding) and h = grad_entropy:
 *   out_v = inv_temperature * (sum_{i: t_i = v} g_i - p_v sum_i g_i
 *                              - h p_v (ln p_v + entropy))
 * in fp32, rounded once to the logits' type.  lse and entropy are what
 * dflash_token_logprobs gave (both entropy and grad_entropy, or neither).  p
 * comes from lse_parts where they are given, as exact for rows of any size;
 * from lse alone, p is off by the factor exp(+-2^-24 |lse|): a row all of the
 * type's lowest value, whose lse is that value or below fp32's range, or one whose lse
 * is beyond it above, needs lse_parts.  A row
 * whose g and h are all 0 gets zeros, whatever it holds; one of -inf alone the
 * g at its tokens.  out may be logits, with one row
 * stride; no other overlap.
 * Errors: E_INVAL, E_CUDA. */
typedef struct {
    int32_t dtype;             /* of logits and out */
    int32_t rows;
    int32_t vocab;
    int32_t n;                 /* 0 .. DFLASH_LOGPROBS_MAX_TOKENS */
    float inv_temperature;
    int32_t reserved;          /* 0 */
    int64_t ld_logits;
    int64_t ld_out;
    const void* logits;
    const int32_t* tokens;     /* [rows][n]; NULL when n is 0 */
    const float* lse;          /* [rows]; NULL with lse_parts */
    const float* grad_logprobs; /* [rows][n]; NULL when n is 0 */
    const float* entropy;      /* [rows] or NULL */
    const float* grad_entropy; /* [rows] or NULL */
    void* out;                 /* [rows][vocab] */
    const float* lse_parts;    /* [rows][2], 8-byte aligned, or NULL: lse is read */
} dflash_logprobs_grad_args;
dflash_status dflash_token_logprobs_grad(const dflash_logprobs_grad_args* args, void* cuda_stream);

/* Release every library-owned buffer.  NULL is a no-op. */
void dflash_destroy(dflash_ctx* ctx);

/* Text of the last failure on ctx (or of the last failed dflash_init when ctx
 * is NULL).  Valid until the next call on the same ctx. */
const char* dflash_last_error(const dflash_ctx* ctx);

#ifdef __cplusplus
}
#endif
#endif /* DFLASH_H */
