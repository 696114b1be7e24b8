/*
 * moe.h — C ABI of the B200 (sm_100a) Grok-1 MoE feed-forward sublayer.
 *
 * The operation (grok-field-guide "Grok-1 blueprint", section "MoE sublayer";
 * Grok-1 book ch. 10 "Comparison with other MoE", sections 10.3, 10.3.1, 10.4):
 *   for every token t (row of x):
 *     logits = x[t] . w_router (+ router_bias)           fp32, 8 experts
 *     p      = softmax(logits)                           fp32
 *     (e0,e1)= the two largest logits, descending; an exact tie goes to the
 *              lower expert index; gates g0 = p[e0], g1 = p[e1], NOT renormalised
 *     y_s    = ( GELU(x[t] . w_gate[e_s]) * (x[t] . w_up[e_s]) ) . w_down[e_s]
 *     out[t] = g0 * y_0 + g1 * y_1
 *   GELU is the tanh approximation unless MOE_ACT_GELU_ERF is asked for. Every
 *   routed (token, expert) pair is computed: no capacity limit, no token drop
 *   (Grok-1 book ch. 10, section 10.3.2, capacity-factor box).
 * Options (moe_options_t) add the variants the same pages compare against:
 *   renormalize = 1: gates divided by g0 + g1 (Mixtral, ch. 10 section 10.3.1);
 *   MOE_ACT_SILU: SiLU instead of GELU on the gate branch (SwiGLU, section 10.4);
 *   post_norm_weight / residual: out[t] = residual[t] + w * y / sqrt(mean(y^2) + eps)
 *   with y the gate-weighted sum above, the sublayer's post-RMSNorm and residual
 *   add (sandwich norm, section 10.3.1; the blueprint's "added back to the trunk").
 *
 * Pointers. Every array argument is a DEVICE pointer on the device that owns
 * `stream`; the caller owns all of them; the library never frees or retains
 * them and never synchronises the stream. All arrays are dense, row-major,
 * 16-byte aligned:
 *   x        [T, d]      fp32 (MOE_F32) or bf16 (MOE_BF16, MOE_BF16_INT8W)
 *   w_router [d, E]      fp32 (always)
 *   w_gate   [E, d, f]   fp32 / bf16 / int8 (by dtype)
 *   w_up     [E, d, f]   fp32 / bf16 / int8
 *   w_down   [E, f, d]   fp32 / bf16 / int8
 *   out      [T, d]      same dtype as x
 * int8 weights carry one bf16 scale per output channel (Grok-1 book ch. 1,
 * section 1.2, INT8 box): w = q * s, s_gate/s_up [E, f], s_down [E, d].
 *
 * Limits of this version: E == 8, k == 2; MOE_F32 needs d % 64 == 0 and
 * f % 64 == 0; MOE_BF16 and MOE_BF16_INT8W need d % 256 == 0 and f % 128 == 0;
 * 0 <= T <= 2^24. T == 0 returns MOE_OK and launches nothing.
 *
 * Errors. Arguments are checked on the host before anything is launched; a
 * failed check returns its status and launches nothing. A launch failure
 * returns MOE_ERR_CUDA. Faults of earlier asynchronous work surface at the
 * caller's next synchronisation, not here. Kernels never trap: they record
 * what went wrong as bits of the workspace status word, which
 * moe_device_status() reads back as MOE_ERR_DEVICE_CHECK with the code:
 *   0x01, 0x02, 0x04, 0x08  a GEMM wait (producer, MMA, epilogue, int8
 *                           converter) exceeded its time limit; the kernel
 *                           unwound and the output is incomplete
 *   0x10                    moe_selftest_bounded_wait's wait ran out (expected)
 *   0x20                    MOE_BF16_INT8W: an activation or GeGLU intermediate
 *                           left the fp16 range (|v| > 65504 became infinite);
 *                           the output is not valid
 *   0x40                    library built with MOE_DEBUG_BOUNDS: an index
 *                           outside its array was caught and the access skipped;
 *                           moe_int8_product in every build: counts that leave
 *                           [0, R] were cut off
 * Behaviour on non-finite inputs is unspecified.
 */
#ifndef MOE_B200_MOE_H
#define MOE_B200_MOE_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MOE_EXPORT __attribute__((visibility("default")))
#else
#define MOE_EXPORT
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1,   /* null pointer, negative or inconsistent size   */
  MOE_ERR_UNSUPPORTED = 2,   /* E != 8, k != 2, or d / f not a supported multiple */
  MOE_ERR_MISALIGNED = 3,    /* a pointer is not 16-byte aligned              */
  MOE_ERR_WORKSPACE = 4,     /* workspace missing or smaller than needed      */
  MOE_ERR_CUDA = 5,          /* a CUDA runtime / driver call failed           */
  MOE_ERR_DEVICE_CHECK = 6   /* a kernel recorded a device-side check failure */
} moe_status_t;

typedef enum {
  MOE_F32 = 0,         /* fp32 activations and weights, fp32 arithmetic        */
  MOE_BF16 = 1,        /* bf16 activations and weights, fp32 accumulation      */
  MOE_BF16_INT8W = 2,  /* bf16 activations, int8 weights + bf16 channel scales;
                          the expert GEMMs run on fp16 operands: int8 -> fp16 is
                          exact, bf16 activations -> fp16 is exact for normal
                          values below 65504 in magnitude, and the GeGLU
                          intermediate is kept in fp16 (range |h| < 65504)     */
  MOE_INT8 = 3         /* rows that are 8-bit integers already (moe_int8_product) */
} moe_dtype_t;

/* Activation on the gate branch of every expert. */
typedef enum {
  MOE_ACT_GELU_TANH = 0,  /* GELU, tanh approximation (default, Grok-1) */
  MOE_ACT_GELU_ERF = 1,   /* GELU, z * Phi(z)                           */
  MOE_ACT_SILU = 2        /* SiLU, z * sigmoid(z) (Mixtral)             */
} moe_activation_t;

/* Kernel family. AUTO picks WEIGHT_STREAM (tokens on the MMA N side, split-K
 * down projection) when the average tokens per expert is small (T <= 128 with
 * bf16 weights, T <= 256 with int8 weights; measured crossovers), else token
 * tiles (tokens on the MMA M side). For those small bf16 batches only the down
 * projection streams its weights that way; the gate/up GEMM runs 128-token
 * tiles on single CTAs (measured faster). Above them, with bf16 weights the gate/up
 * GEMM then runs 256-token tiles on single CTAs from T = 512 on; below that,
 * and for the down GEMM, the device chooses from the expert counts between
 * 128-token tiles on single CTAs and 256-token tiles on CTA pairs
 * (cta_group::2). int8 weights take 256-token tiles on single CTAs.
 * TOKEN_TILE forces the pair form, TOKEN_TILE_SINGLE the single-CTA form
 * (128-token tiles for bf16). All compute the same result within rounding;
 * each H element accumulates the same K steps in the same order in every
 * token-tile form. */
typedef enum {
  MOE_PATH_AUTO = 0,
  MOE_PATH_TOKEN_TILE = 1,
  MOE_PATH_WEIGHT_STREAM = 2,
  MOE_PATH_TOKEN_TILE_SINGLE = 3
} moe_path_t;

/* Per-output-channel scales of int8 weights (device pointers, bf16). */
typedef struct {
  const void* s_gate; /* [E, f] */
  const void* s_up;   /* [E, f] */
  const void* s_down; /* [E, d] */
} moe_scales_t;

/* cudaStream_t, passed as an opaque handle (NULL = the legacy default stream). */
typedef void* moe_stream_t;

/* All arguments of one forward call (see the file header for layouts). */
typedef struct {
  const void* x;
  const float* w_router;
  const void* w_gate;
  const void* w_up;
  const void* w_down;
  const moe_scales_t* w_scales; /* host struct of device pointers; NULL unless MOE_BF16_INT8W */
  void* out;
  int64_t T, d, f;
  int32_t E, k;
  moe_dtype_t dtype;
} moe_args_t;

/* Per-call options; a zero-initialised struct (or opts == NULL) is the plain
 * Grok-1 sublayer with automatic kernel choices. */
typedef struct {
  moe_activation_t activation; /* gate-branch activation, MOE_ACT_GELU_TANH default      */
  const float* router_bias;    /* [E] fp32 device pointer added to the logits, or NULL    */
  moe_path_t path;             /* kernel family; MOE_PATH_AUTO by default                */
  int32_t down_splits;         /* split-K factor for w_down (must divide f/64); 0 = auto  */
  void* const* stage_events;   /* NULL, or 6 cudaEvent_t (host array) recorded on the
                                  stream before router, dispatch, gate/up GEMM, down
                                  GEMM, combine, and after combine (stage timing)        */
  int32_t renormalize;         /* 0: gates are the softmax probabilities (Grok-1);
                                  1: gates divided by their sum (Mixtral)                */
  const void* residual;        /* [T, d] x-dtype device pointer added to the output, or NULL */
  const float* post_norm_weight; /* [d] fp32 RMSNorm weight applied to the sublayer
                                  output before the residual add, or NULL (no norm)      */
  float norm_eps;              /* RMSNorm epsilon (> 0) when post_norm_weight is set      */
  int32_t row_gather;          /* 0: token tiles read a permuted copy of x made by the
                                  dispatch stage (default); 1: they gather their gate/up
                                  operand rows from x with TMA row gathers (no copy; slower
                                  on B200, where four-row gathers cannot feed the MMA).
                                  The weight-stream form always reads the copy;
                                  MOE_BF16_INT8W returns MOE_ERR_UNSUPPORTED with 1.      */
  int32_t separate_combine;    /* 0: the down projection's epilogue sums each token's two
                                  expert rows (default; bf16 and int8 weights without the
                                  post-norm); 1: a separate combine kernel does it (same
                                  result bit for bit)                                     */
} moe_options_t;

/* Optional outputs for inspection; each is a device pointer or NULL.
 * Permuted order = token slots sorted stably by (expert, token). */
typedef struct {
  int32_t* idx;        /* [T, 2] chosen experts, slot 0 = larger logit      */
  float* gates;        /* [T, 2] their softmax probabilities                */
  int32_t* counts;     /* [E]    token slots per expert                     */
  int32_t* offsets;    /* [E+1]  exclusive prefix of counts                 */
  int32_t* perm_token; /* [2T]   token of each permuted row                 */
  int32_t* perm_slot;  /* [2T]   slot (0/1) of each permuted row            */
  void* h;             /* [2T, f] GELU(x.Wg)*(x.Wu) per permuted row: x-dtype,
                          but fp16 for MOE_BF16_INT8W; when set, the kernels
                          write the intermediate here                         */
} moe_debug_t;

/* Passage: grok-field-guide "Grok-1 blueprint", section "MoE sublayer" (router,
 * top-2, gated experts, gate-weighted sum); gates as in Grok-1 book ch. 10,
 * section 10.3.1 (not renormalised); experts as in section 10.4 (GeGLU).
 * Forward pass with a library-owned workspace: one cache per device, grown
 * with cudaMalloc when a call needs more (never shrunk), guarded by a mutex.
 * Calls on one device share that workspace, so calls that may overlap on the
 * GPU (different streams) must use moe_forward_ex with their own workspaces.
 * Returns MOE_OK or an error status (see the file header). */
MOE_EXPORT moe_status_t moe_forward(const void* x, const float* w_router, const void* w_gate,
                         const void* w_up, const void* w_down,
                         const moe_scales_t* w_scales, void* out,
                         int64_t T, int64_t d, int64_t f, int32_t E, int32_t k,
                         moe_dtype_t dtype, moe_stream_t stream);

/* Passage: Grok-1 book ch. 11, section 11.3.1 item 3 (the sparse reorder and
 * grouped GEMM that replace the dense one-hot evaluation need the permuted
 * rows and intermediates this workspace holds).
 * Bytes of device workspace moe_forward_ex needs for these sizes with the
 * automatic kernel choices (path MOE_PATH_AUTO, automatic split-K), 0 on bad
 * arguments or T == 0. 256-byte multiple. Host only: no CUDA call. */
MOE_EXPORT size_t moe_workspace_size(int64_t T, int64_t d, int64_t f, int32_t E, int32_t k,
                                     moe_dtype_t dtype);

/* The same for a call whose moe_options_t sets `path` and `down_splits`
 * (0 = automatic), which change the workspace layout: 0 also when the split
 * factor does not divide f / 64 or the path is unknown. */
MOE_EXPORT size_t moe_workspace_size_ex(int64_t T, int64_t d, int64_t f, int32_t E, int32_t k,
                                        moe_dtype_t dtype, moe_path_t path, int32_t down_splits);

/* ---- Expert parallelism ----------------------------------------------------
 * Passage: Grok-1 book ch. 1, section 1.6.3 (the MoE layer shards the expert
 * axis over the devices of a (1, 8) mesh with shard_map). Building blocks of
 * that form on W GPUs, one process each, GPU r owning n = 8 / W consecutive
 * experts: each GPU routes and dispatches its own tokens (moe_route_dispatch;
 * the permuted rows are then grouped by owning GPU, because the permutation is
 * expert-major), the caller's communication library sends every block of rows
 * to its owner, the owner makes the received rows expert-contiguous
 * (moe_gather_rows), runs its experts on them (moe_experts_forward, which
 * also applies each row's gate), the rows go back the same way, and each GPU
 * sums its tokens' two rows (moe_combine). With the same split-K factor the
 * result equals moe_forward_ex's bit for bit. Every pointer is a device
 * pointer; workspaces are 256-byte aligned device memory of at least the
 * stated size; each call records its status word at the start of its
 * workspace (moe_device_status reads it). */

/* Outputs of moe_route_dispatch (device arrays owned by the caller). */
typedef struct {
  int32_t* idx;        /* [T, 2] chosen experts, slot 0 = larger logit          */
  float* gates;        /* [T, 2] their gates                                     */
  int32_t* counts;     /* [8]    token slots per expert                          */
  int32_t* offsets;    /* [9]    exclusive prefix of counts                      */
  int32_t* perm_token; /* [2T]   token of each permuted row                      */
  int32_t* perm_slot;  /* [2T]   slot of each permuted row                       */
  int32_t* slot_pos;   /* [T, 2] permuted row of each (token, slot)              */
  float* gate_perm;    /* [2T]   gate of each permuted row                       */
  void* xp;            /* [2T, d] x rows in permuted order: x's dtype, but fp16
                          for MOE_BF16_INT8W (the int8-weight GEMMs' operand)    */
} moe_routed_t;

/* Workspace bytes of moe_route_dispatch (0 on bad sizes or T == 0). */
MOE_EXPORT size_t moe_route_workspace_size(int64_t T, int64_t d, moe_dtype_t dtype);

/* The router and dispatch stages of moe_forward on T tokens: logits, softmax,
 * top-2 (gates renormalised if renormalize == 1), counts, offsets, the stable
 * (expert, token) permutation and the permuted copy of x. Same size limits
 * and errors as moe_forward_ex. */
MOE_EXPORT moe_status_t moe_route_dispatch(const void* x, const float* w_router, const float* router_bias,
                                           int64_t T, int64_t d, moe_dtype_t dtype, int32_t renormalize,
                                           const moe_routed_t* routed, void* workspace, size_t ws_bytes,
                                           moe_stream_t stream);

/* Rows for n_experts experts held by this GPU (row block e belongs to local
 * expert e, in order). */
typedef struct {
  const void* xp;              /* [R, d] rows, expert-contiguous: bf16 (MOE_BF16), fp16
                                  (MOE_BF16_INT8W) or fp32 (MOE_F32)                  */
  const int32_t* counts;       /* [n_experts] rows of each local expert (device)      */
  const float* gate;           /* [R] gate of each row, or NULL for 1                 */
  const void* w_gate;          /* [n_experts, d, f]                                   */
  const void* w_up;            /* [n_experts, d, f]                                   */
  const void* w_down;          /* [n_experts, f, d]                                   */
  const moe_scales_t* w_scales;/* MOE_BF16_INT8W: [n_experts, f], [n_experts, f],
                                  [n_experts, d]; else NULL                           */
  float* y;                    /* [R, d] fp32: gate * FFN_e(row)                       */
  int64_t R, d, f;
  int32_t n_experts;           /* 1 .. 8 */
  moe_dtype_t dtype;
} moe_expert_rows_t;

/* Workspace bytes of moe_experts_forward (0 on bad sizes, R == 0 or a split
 * factor that does not divide f / 64). `path` and `down_splits` as in
 * moe_options_t. */
MOE_EXPORT size_t moe_experts_workspace_size(int64_t R, int64_t d, int64_t f, int32_t n_experts,
                                             moe_dtype_t dtype, moe_path_t path, int32_t down_splits);

/* The expert GEMMs of moe_forward on rows already grouped by expert:
 * y[r] = gate[r] * down(act(xp[r] . w_gate[e]) * (xp[r] . w_up[e])) for the
 * rows r of local expert e (section 10.4 of ch. 10; activation, path and
 * down_splits from opts, NULL = defaults). Token-tile rows run on single CTAs
 * unless opts->path is MOE_PATH_TOKEN_TILE (CTA pairs). */
MOE_EXPORT moe_status_t moe_experts_forward(const moe_expert_rows_t* rows, const moe_options_t* opts,
                                            void* workspace, size_t ws_bytes, moe_stream_t stream);

/* out[t] = y[slot_pos[t,0]] + y[slot_pos[t,1]] (fp32 sum, in that order, then
 * cast to the x dtype: fp32 for MOE_F32, else bf16), with the post-RMSNorm
 * and residual add of moe_options_t when post_norm_weight / residual are set
 * (the blueprint's gate-weighted sum; ch. 10, section 10.3.1 sandwich norm).
 * y is [2T, d] fp32 in permuted order. Workspace: at least 256 bytes. */
MOE_EXPORT moe_status_t moe_combine(const float* y, const int32_t* slot_pos, int64_t T, int64_t d,
                                    moe_dtype_t dtype, const void* residual, const float* post_norm_weight,
                                    float norm_eps, void* out, void* workspace, size_t ws_bytes,
                                    moe_stream_t stream);

/* No counterpart on the pages (data movement of the expert-parallel form):
 * dst row i = src row index[i] (int32, device), for i < n; rows of row_bytes
 * bytes, a multiple of 4 (src and dst 4-byte aligned) or of 16 (16-byte
 * aligned, copied in 16-byte vectors); src has src_rows rows. Workspace: at
 * least 256 bytes. */
MOE_EXPORT moe_status_t moe_gather_rows(const void* src, int64_t src_rows, const int32_t* index, int64_t n,
                                        int64_t row_bytes, void* dst, void* workspace, size_t ws_bytes,
                                        moe_stream_t stream);

/* ---- Routing, products and combine of any E and k ---------------------------
 * The sublayer above fixes E = 8, k = 2 and the softmax router. The calls below
 * make the same layer of other routers and of 8-bit arithmetic:
 *   moe_topk_route -> moe_int8_product (gate/up) -> moe_int8_product (down)
 *   -> moe_combine_topk
 * and give the router's gradient for training. They follow the file header's rules
 * (dense, row-major, 16-byte aligned device arrays; checks on the host; no
 * synchronisation; nothing kept between calls); calls that may overlap on the
 * GPU need distinct workspaces and outputs. Outputs overlap neither one another
 * nor an input, except where a call says so. */

typedef enum {
  MOE_SCORE_SOFTMAX = 0, /* s = softmax(logits) over the E experts */
  MOE_SCORE_SIGMOID = 1  /* s = 1 / (1 + exp(-logit)) per expert   */
} moe_score_t;

typedef enum {
  MOE_GROUP_MAX = 0,      /* a group's value: its largest rank value                  */
  MOE_GROUP_TOP2_SUM = 1  /* the sum of its two largest score + bias (of the one it has) */
} moe_group_rule_t;

/* Routing of T tokens from their router logits. Per token:
 *   a logit that is -inf or NaN masks its expert (score 0, never chosen); +inf
 *   counts as the largest fp32; s = the scores of the rest (moe_score_t);
 *   rank value c = s + bias, or the logit itself without a bias (same order);
 *   with n_groups > 1 the E experts form n_groups runs of E / n_groups, and only
 *   the topk_groups groups of the largest value stay (ties: the lower group);
 *   idx = the k largest c in descending order, ties to the lower expert;
 *   weights = scale * s[idx], divided by the sum of s[idx] if renormalize == 1.
 * The bias steers the choice only. The choice is that of the values in 64 bits:
 * where 32 bits cannot decide, the kernel decides in 64. A token with fewer than
 * k experts to choose from gets idx -1 and weight 0 in the slots left over.
 * Limits: 1 <= E <= 1024, 1 <= k <= min(E, 32), 1 <= topk_groups <= n_groups <= 32,
 * E % n_groups == 0, 0 <= T <= 2^24, scale finite. */
typedef struct {
  const void* logits;        /* [T, E] MOE_F32 or MOE_BF16                               */
  const float* bias;         /* [E] fp32 or NULL; an expert with a NaN bias is masked     */
  const int32_t* n_tokens;   /* one int32 on the device, or NULL for T: rows from it on are
                                padding (idx -1, weights and scores 0, not dispatched)    */
  int64_t T;
  int32_t E, k;
  moe_dtype_t dtype;         /* of the logits                                             */
  moe_score_t score;
  int32_t n_groups, topk_groups; /* 1, 1: no groups                                       */
  moe_group_rule_t group_rule;
  int32_t renormalize;       /* 0 or 1                                                    */
  float scale;
} moe_topk_args_t;

/* Outputs. The dispatch arrays (counts .. gate_perm) are all given or all NULL;
 * permuted order = chosen slots sorted by (expert, token), as moe_routed_t's. */
typedef struct {
  int32_t* idx;        /* [T, k] chosen experts, -1 = none                              */
  float* weights;      /* [T, k]                                                         */
  float* scores;       /* [T, E] scores of every expert, or NULL                         */
  int32_t* counts;     /* [E]    slots per expert                                        */
  int32_t* offsets;    /* [E+1]  exclusive prefix of counts                              */
  int32_t* perm_token; /* [T*k]  token of each permuted row, -1 behind the last one       */
  int32_t* perm_slot;  /* [T*k]  its slot, -1 behind the last one                         */
  int32_t* slot_pos;   /* [T, k] permuted row of each slot, -1 = none                    */
  float* gate_perm;    /* [T*k]  weight of each permuted row, 0 behind the last one       */
} moe_topk_routed_t;

/* Workspace bytes of moe_topk_route with the dispatch arrays: 0 when none is needed (up to
 * 256 tokens; a call without the arrays needs none either) and on bad sizes. */
MOE_EXPORT size_t moe_topk_workspace_size(int64_t T, int32_t E, int32_t k);

/* See moe_topk_args_t. `workspace` may be NULL when none is needed; one that is given all
 * the same (256-byte aligned, 4 bytes or more) gets its status word written. */
MOE_EXPORT moe_status_t moe_topk_route(const moe_topk_args_t* args, const moe_topk_routed_t* routed,
                                       void* workspace, size_t ws_bytes, moe_stream_t stream);

/* Gradient of moe_topk_route's weights, and optionally of its scores, with
 * respect to the logits, for the choice `idx` it made (the choice itself has no
 * gradient; the bias takes none). args as given to moe_topk_route; bias and the
 * group fields are not looked at. Entries of idx outside [0, E) contribute nothing;
 * masked logits and padded rows get 0. Sums in fp32, fixed order, no atomics. */
MOE_EXPORT moe_status_t moe_topk_route_backward(const moe_topk_args_t* args,
                                                const int32_t* idx,          /* [T, k]               */
                                                const float* grad_weights,   /* [T, k]               */
                                                const float* grad_scores,    /* [T, E] or NULL       */
                                                void* grad_logits,           /* [T, E], logits' type */
                                                moe_stream_t stream);

/* Product of rows and int8 weights in 8-bit integers, one scale per row and one
 * per output channel, rows grouped by expert (or one plain matrix):
 *   y[r, n] = gate[r] * a[r] * s[e, n] * sum_k q[r, k] * w[e, k, n]
 * the sum in 32-bit integers (exact). With w_up the call computes the gated pair
 * of an expert, y = gate * act(z_w) * z_w_up, in one kernel. x in 16 or 32 bits
 * is brought to 8 on the way: a[r] = max|x[r]| / 127, q = x / a rounded to nearest
 * (ties to even; decided exactly), a row of zeros staying zero and a row with an
 * infinity or NaN giving a row of NaN; `index` gathers its rows.
 * w, w_up [n_experts, K, N] int8 and s, s_up [n_experts, N] bf16 are laid out as the
 * weights and scales of MOE_BF16_INT8W.
 * Limits: 0 <= R <= 2^24, K and N multiples of 16, 16 <= K < 131072 (the sum stays
 * below 2^31), 16 <= N <= 2^20, 1 <= n_experts <= 1024. */
typedef struct {
  const void* x;          /* [x_rows, K] MOE_F32 / MOE_BF16, or [R, K] MOE_INT8             */
  const float* x_scale;   /* [R]: MOE_INT8 rows' scales; else NULL                          */
  const int32_t* index;   /* [R] row of x for each row, or NULL (x_rows == R); an entry outside
                             [0, x_rows) stands for a row of zeros; NULL with MOE_INT8       */
  const int32_t* counts;  /* [n_experts] rows of each expert, in order (device); NULL with
                             n_experts == 1: all R rows. Rows of out behind the last expert's
                             are left as they were                                          */
  const void* w;          /* [n_experts, K, N] int8                                         */
  const void* w_up;       /* the same, or NULL                                              */
  const void* s;          /* [n_experts, N] bf16                                            */
  const void* s_up;       /* the same with w_up, else NULL                                  */
  const float* gate;      /* [R] or NULL for 1                                              */
  void* out;              /* [R, N] MOE_F32 or MOE_BF16                                     */
  int64_t x_rows, R, K, N;
  int32_t n_experts;
  moe_dtype_t x_dtype, out_dtype;
  moe_activation_t activation; /* with w_up                                                  */
} moe_int8_args_t;

/* Workspace bytes of moe_int8_product, 0 on bad sizes or R == 0. 256-byte multiple. */
MOE_EXPORT size_t moe_int8_workspace_size(int64_t R, int64_t K, int64_t N, int32_t n_experts,
                                          moe_dtype_t x_dtype, int32_t with_up);

/* See moe_int8_args_t. The status word at the start of the workspace also gets bit
 * 0x40 (in every build) when counts hold a negative number or add up to more than R:
 * such rows are not computed. */
MOE_EXPORT moe_status_t moe_int8_product(const moe_int8_args_t* args, void* workspace, size_t ws_bytes,
                                         moe_stream_t stream);

/* out[t] = residual[t] + sum over the k slots of weights[t, s] * y[slot_pos[t, s]],
 * summed in fp32 in slot order and rounded once. y [R, d] and out [T, d] are MOE_F32
 * or MOE_BF16 (residual has out's type); weights [T, k] fp32 or NULL for 1; a slot_pos
 * outside [0, R) adds nothing; out may be residual. Limits: 0 <= T <= 2^24, 1 <= k <= 32,
 * d a multiple of 8 up to 2^20, T * ceil(d / 1024) < 2^31, 0 <= R <= 2^29. Generalises
 * moe_combine (k = 2, fp32 rows). */
MOE_EXPORT moe_status_t moe_combine_topk(const void* y, moe_dtype_t y_dtype, int64_t R, const int32_t* slot_pos,
                                         const float* weights, int64_t T, int32_t k, int64_t d,
                                         const void* residual, void* out, moe_dtype_t out_dtype,
                                         moe_stream_t stream);

/* Passage: as moe_forward; the options follow Grok-1 book ch. 10, section
 * 10.3.1 (Mixtral renormalisation, sandwich post-norm) and section 10.4 (SiLU).
 * Forward pass on a caller-provided device workspace of ws_bytes bytes
 * (256-byte aligned, at least moe_workspace_size(...)); allocates nothing.
 * `opts` and `dbg` may be NULL. Concurrent calls need distinct workspaces. */
MOE_EXPORT moe_status_t moe_forward_ex(const moe_args_t* args, const moe_options_t* opts,
                            const moe_debug_t* dbg, void* workspace, size_t ws_bytes,
                            moe_stream_t stream);

/* Forward pass that allocates nothing: its scratch is a fixed 32 MiB device
 * array owned by the library (one per device that loads it, held until the
 * process exits). For callers that must not call cudaMalloc at run time, such
 * as a framework that reserves all device memory in its own pool at start-up,
 * or a latency-critical loop where an allocation would stall the device. The
 * pages have no counterpart: this is a deployment variant of moe_forward_ex.
 * Same arguments and results as moe_forward_ex without workspace and debug
 * outputs. With opts->down_splits == 0 the split-K factor is lowered until the
 * scratch fits. Returns MOE_ERR_WORKSPACE when the problem needs more than the
 * 32 MiB maximum (e.g. T = 64 at d = 6144, f = 32768 fits; T = 4096 does not).
 * The first call on a device looks up the array's device address and should
 * come before any stream capture; a call with T == 0 does only that set-up and
 * launches nothing. All calls on a device share the array: calls that may
 * overlap on the GPU race and must be ordered by the caller. The kernels'
 * status word lives in the array; moe_device_status(NULL, ...) reads it. */
MOE_EXPORT moe_status_t moe_forward_noalloc(const moe_args_t* args, const moe_options_t* opts,
                                            moe_stream_t stream);

/* No counterpart on the pages: the library's own failure reporting.
 * Synchronises `stream` and reads the status word that the kernels of the last
 * call on `workspace` recorded. With workspace == NULL it reads the two
 * library-owned words of the current device, the moe_forward cache's and the
 * moe_forward_noalloc scratch's (each if it exists), and reports their OR.
 * Returns MOE_OK, MOE_ERR_DEVICE_CHECK (and the raw code in *code if
 * code != NULL) or MOE_ERR_CUDA. */
MOE_EXPORT moe_status_t moe_device_status(const void* workspace, moe_stream_t stream, uint32_t* code);

/* Check of the failure path, with no fault: launches one thread that waits,
 * with the same bounded mbarrier wait the GEMM pipelines use, on a barrier that
 * nothing arrives on, giving up after `limit_us` microseconds (1 .. 10^7). The
 * kernel then records bit 0x10 in the status word at the start of `workspace`
 * (device memory, 256-byte aligned, at least 256 bytes) and returns, so a
 * following moe_device_status(workspace, stream, &code) returns
 * MOE_ERR_DEVICE_CHECK with code 0x10 and the context stays usable. No
 * counterpart on the pages: it exercises the library's own time limits.
 * Returns MOE_OK once launched, MOE_ERR_WORKSPACE / MOE_ERR_INVALID_ARG on bad
 * arguments, MOE_ERR_CUDA if the launch fails. */
MOE_EXPORT moe_status_t moe_selftest_bounded_wait(void* workspace, uint32_t limit_us, moe_stream_t stream);

/* No counterpart on the pages. Static description of a status code (never NULL). */
MOE_EXPORT const char* moe_status_string(moe_status_t status);

/* No counterpart on the pages. Library ABI version, currently 2. */
MOE_EXPORT int32_t moe_abi_version(void);

/* No counterpart on the pages. Options the library was compiled with, as bits:
 * MOE_BUILD_DEBUG_BOUNDS = the MOE_DEBUG_BOUNDS build (every index that one
 * kernel of the sublayer or of its expert-parallel pieces computes and another
 * uses is checked before the access; a failed check sets status bit 0x40 and
 * skips the access; slower, for testing). The kernels of the calls of any E and
 * k hold no such checks; indices and counts that a caller gives them are bounded
 * in every build. */
#define MOE_BUILD_DEBUG_BOUNDS 1
MOE_EXPORT int32_t moe_build_flags(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_B200_MOE_H */
