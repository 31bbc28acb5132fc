/*
 * lq.h -- C ABI of liblq: per-window int8 recurrent-state decode for Gated
 * DeltaNet (GDN) and Kimi Delta Attention (KDA) layers on GB300 (sm_103a).
 *
 * The method: LeapQuant (paperlayer.ai summary of arXiv 2609.38166v1). Each
 * head-state S (d_v x d_k = 128 x 128; row i = value channel, column j = key
 * channel) is held as
 *   - 8-bit codes (or 6- or 4-bit, lq_config.code_bits) with one fp32 step per
 *     value row (sigma),
 *   - one fp32 smoothing scale per key channel (lambda; §3.4 Residual smoothing),
 *   - C fp32 Compensator Tokens, each one whole row or column of the state, or
 *     with lq_config.comp_fit a fitted rank-one factor pair (§3.3 Compensator
 *     Tokens),
 * fixed for a window of W tokens (§3.2 Per-window quantization), plus a buffer
 * of up to W fp32 records (k_m, u_m, alpha_m), one per token of the open window.
 * Per token, the append step reads the state from the fixed boundary plus the
 * records (App. B.2 window unrolling, App. B.3 readout with a smoothed
 * quantized residual), forms the delta-rule correction u, stores the record and
 * writes the output. When the window is full, the fold rebuilds the state in
 * original coordinates, selects (or fits) compensators, smooths, rounds once
 * and empties the buffer (fastpathlabs.ai research note 4, "What we built": an
 * append step and a fold). Tokens whose update takes two rank-one sub-steps
 * (DeltaProduct with two steps, RWKV7) leave two records (App. A).
 *
 * Conventions for every call below:
 *   - Ownership: the caller owns every buffer. The library allocates no memory
 *     and creates no streams or events.
 *   - Pointers: device pointers on the current CUDA device (device or managed
 *     memory). Token inputs and outputs are contiguous fp32 arrays, 16-byte
 *     aligned (the generation calls at the end say what they take); the state
 *     buffer is 256-byte aligned.
 *   - Layout of token inputs: [n_states][d] row-major, state index
 *     s = (request * layers + layer) * heads + head, or any order the caller
 *     keeps fixed.
 *   - Asynchrony: calls enqueue kernels on `stream` (a cudaStream_t; NULL is
 *     the legacy default stream) and return without synchronizing. The return
 *     value covers host-side validation and the launch. Conditions found on
 *     the device (a full window, a phase mismatch, a state buffer written with
 *     another configuration) set the state buffer's status word, which
 *     lq_get_status reads; the affected head-states are left unchanged.
 *   - Threads: no global mutable state except a thread-local error message,
 *     the thread-local test hook of lq_debug_set_wait, a thread-local record
 *     of the kernel attributes (shared-memory size) already set per kernel and
 *     device, and the device address of lq_decode_step_noalloc's fixed array,
 *     looked up once per device.
 *   - n_states = 0 is valid and does nothing.
 */
#ifndef LQ_H
#define LQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A cudaStream_t, passed as an opaque pointer so that this header needs no CUDA headers. */
typedef void* lq_stream_t;

typedef enum {
  LQ_OK = 0,
  LQ_ERR_INVALID_ARG = -1, /* null/misaligned pointer, bad size, pointer not on the current device */
  LQ_ERR_UNSUPPORTED = -2, /* a configuration this build does not run (see lq_config)            */
  LQ_ERR_WINDOW_FULL = -3, /* device: append on a head-state that already holds W records         */
  LQ_ERR_CUDA = -4,        /* a CUDA runtime call failed (message in lq_last_error)              */
  LQ_ERR_TIMEOUT = -5,     /* device: a bounded wait inside a kernel gave up                       */
  LQ_ERR_PHASE = -6,       /* device: a head-state's record count differs from the stated phase    */
  LQ_ERR_STATE = -7,       /* device: the state buffer was not initialised with this config/size  */
  LQ_ERR_PARENT = -8       /* device: a beam's parent lies outside its group                        */
} lq_status;

/* lq_decode_step's `phase` when head-states may sit at different window positions. */
#define LQ_PHASE_ANY (-1)

typedef struct {
  int32_t d_k, d_v;      /* key / value channels: 128 and 128 in this build                 */
  int32_t window;        /* W: tokens per window, 1..32 (default 16)                        */
  int32_t n_comp;        /* C: compensators per head-state, 0..8 (default 4)                */
  int32_t decay_per_key; /* 0: scalar alpha per token (GDN); 1: alpha in R^{d_k} (KDA)      */
  int32_t smooth;        /* 1: residual smoothing on (default); 0: lambda = 1               */
  float lambda_floor;    /* positive floor of the smoothing scales (default 1e-6)           */
  int32_t code_bits;     /* code width: 8 (default), 6 or 4 ([LQ] §4 also evaluates 6- and   */
                         /* 4-bit states); codes in [-q, q], q = 2^(bits-1) - 1              */
  int32_t comp_fit;      /* 0 (default): a compensator is an outlier line, kept exactly;     */
                         /* 1..32: a rank-one factor a b^T fitted to the residual by that   */
                         /* many power-iteration sweeps from the longest row ([LQ] §3.3,    */
                         /* App. B.3, new factors fitted at the boundary; [RN4] "Where the */
                         /* time goes")                                                      */
  int32_t comp_block;    /* with comp_fit > 0: 1 fits the C factors together as a block     */
                         /* (subspace iteration), each fold starting from the previous      */
                         /* window's factors ([RN4] "Redesign"); 0 (default) one at a time  */
} lq_config;

/*
 * Byte offsets of the planes inside one state buffer (all 256-byte aligned)
 * and the per-head-state stride of each plane, in elements. The buffer holds,
 * for head-state s:
 *   counts   int32   [s]                       records held (0..W)
 *   codes    int8    [s][d_v][d_k]             row-major (8-bit codes), or
 *            uint8   [s][d_v][d_k / 2]         4-bit codes: two per byte, code 2j in the
 *                                              low nibble, each stored as c + 8 (1..15)
 *            uint8   [s][d_v][3 d_k / 4]       6-bit codes, each stored as c + 32 (1..63):
 *                                              per row, 64 bytes of low nibbles laid out
 *                                              as a 4-bit row, then 32 bytes holding the
 *                                              top two bits: for element e of 16-code
 *                                              block j, bits 8b + 2g of 32-bit word j,
 *                                              g = 2(e/8) + (e mod 2), b = (e mod 8) / 2
 *   sigma    fp32    [s][d_v]                  quantization step of each value row
 *   lambda   fp32    [s][d_k]                  smoothing scale of each key channel
 *   comp_id  int32   [s][comp_id_stride]       id < d_v: row id; else column id - d_v
 *   comp_line fp32   [s][C][128]               the compensator line, or with comp_fit > 0
 *            fp32    [s][C][256]               the factor pair: a (d_v), then unit b (d_k)
 *   rec_k    fp32    [s][W][d_k]               record keys, slot m-1 holds record m
 *   rec_u    fp32    [s][W][d_v]               record corrections u_m
 *   rec_alpha fp32   [s][alpha_stride]         GDN: W scalars; KDA: [W][d_k]
 *   full_list int32  [n_states]                work list of a mixed-phase decode step:
 *                                              the head-states whose window it filled
 *                                              (empty between calls)
 * A 256-byte header at offset 0 carries a magic number, a hash of the config
 * and n_states, the device status word and the length of the work list.
 * The boundary (codes, sigma, lambda, comp_id, comp_line) takes
 * (16384 + 512 + 512 + 4C + 512C) bytes per head-state with 8-bit codes: 1.19
 * bytes per element at C = 4, the figure of the LeapQuant summary, §4.3
 * Efficiency results (8192 + ... with 4-bit codes: 0.69 bytes per element).
 */
typedef struct {
  size_t total_bytes;
  size_t header, counts, codes, sigma, lambda, comp_id, comp_line, rec_k, rec_u, rec_alpha, full_list;
  int64_t comp_id_stride; /* int32 elements per head-state (C rounded up to a multiple of 4, at least 4) */
  int64_t alpha_stride;   /* fp32 elements per head-state in rec_alpha                               */
  int64_t boundary_bytes_per_state; /* codes + sigma + lambda + 4C id bytes + comp lines                  */
} lq_layout_t;

/* Default configuration: d_k = d_v = 128, W = 16, C = 4, GDN, smoothing on, floor 1e-6, 8-bit codes. */
void lq_config_default(lq_config* cfg);

/*
 * Bytes the caller must allocate for n_states head-states (0 if cfg or n_states
 * is invalid): the boundary of each head-state (LeapQuant summary §3.2
 * Per-window quantization: codes with their row steps; §3.3 Compensator Tokens;
 * §3.4 Residual smoothing; §4.3 Efficiency results gives 1.19 bytes per element
 * for it) plus its window's record buffer (research note 4, "What we built":
 * each token's change is kept as a record until the fold). Host only.
 */
size_t lq_state_bytes(const lq_config* cfg, int64_t n_states);

/* Fill *out with the plane offsets for n_states head-states (the planes listed above:
 * LeapQuant summary §3.2-3.4 for the boundary, research note 4 "What we built" for the
 * records). Host only; never touches a GPU. Errors: LQ_ERR_INVALID_ARG (NULL out, bad
 * n_states), LQ_ERR_UNSUPPORTED (a configuration this build does not run). */
int lq_layout(const lq_config* cfg, int64_t n_states, lq_layout_t* out);

/*
 * Initialise a state buffer: write the header, set every record count to 0 and
 * init-fold S0 into the boundary. This is the fold with no records: compensator
 * selection (LeapQuant summary §3.3 Compensator Tokens), smoothing (§3.4
 * Residual smoothing) and one rounding per row step (§3.2 Per-window
 * quantization; research note 4, "Why rounding the state is difficult").
 * S0 is fp32 [n_states][d_v][d_k] (row i = value channel), or NULL for the
 * zero state; it is only read. Clears the status word. Errors:
 * LQ_ERR_INVALID_ARG for a NULL or misaligned pointer (state 256 bytes, S0 16
 * bytes), memory not on the current device, or bad n_states.
 */
int lq_state_init(const lq_config* cfg, void* state, int64_t n_states, const float* S0, lq_stream_t stream);

/*
 * Re-initialise head-states first .. first+count-1 of a buffer that
 * lq_state_init set up for n_states: init-fold S0 (fp32 [count][d_v][d_k], or
 * NULL for zero) into their boundaries and set their record counts to 0. The
 * other head-states, the header and the status word are untouched, so a
 * serving loop can admit a request into its slots while the rest keep their
 * windows; requests admitted at different tokens then sit at different window
 * phases. A buffer whose header does not match (cfg, n_states) is left
 * unchanged and gets LQ_ERR_STATE. Errors: LQ_ERR_INVALID_ARG when
 * first < 0, count < 0 or first + count > n_states.
 */
int lq_state_init_range(const lq_config* cfg, void* state, int64_t n_states, int64_t first, int64_t count,
                        const float* S0, lq_stream_t stream);

/*
 * Append one token to every head-state: read from the fixed boundary plus the
 * buffered records, u = beta (v - S_{n-1}(alpha . k)), store record n,
 * o = S_n q. No fold: a head-state that already holds W records is left
 * unchanged and the status word is set to LQ_ERR_WINDOW_FULL.
 *   q, k  fp32 [n_states][d_k];  v, o  fp32 [n_states][d_v]
 *   alpha fp32 [n_states] (GDN) or [n_states][d_k] (KDA);  beta fp32 [n_states]
 * o may not alias any input. o's summation order is free; its term for the
 * new record, u (k . q), uses a compensated dot, so it stays within a few
 * float roundings of exact even when k . q nearly cancels (after a zero
 * state it is the whole output).
 */
int lq_append(const lq_config* cfg, void* state, int64_t n_states, const float* q, const float* k, const float* v,
              const float* alpha, const float* beta, float* o, lq_stream_t stream);

/*
 * Fold every head-state with the records it holds (any count 0..W), then empty
 * the buffer: rebuild the state in original coordinates from the boundary and
 * the records (LeapQuant summary App. B.3: reconstructed before fitting new
 * factors), select the compensators (§3.3), smooth the residual (§3.4) and
 * round it once (§3.2); research note 4, "What we built", names this second
 * part of the kernel, which also empties the record buffer.
 * A head-state whose header or record count is invalid is left unchanged and
 * sets LQ_ERR_STATE in the status word.
 */
int lq_fold(const lq_config* cfg, void* state, int64_t n_states, lq_stream_t stream);

/*
 * One decode token for every head-state: append, and fold every head-state
 * whose window that fills (count == W).
 * `phase` is the record count every head-state holds before this call
 * (0..W-1). It lets the library launch the append-only kernel for the W-1
 * steps that cannot fold, and fuse the fold into the append kernel at phase
 * W-1 while the state is on chip; a head-state whose count differs is left
 * unchanged and sets LQ_ERR_PHASE.
 * LQ_PHASE_ANY accepts any count 0..W-1 (head-states at different window
 * phases, e.g. requests admitted at different tokens): the append kernel puts
 * the head-states whose window it fills on the buffer's work list, and a
 * second kernel folds them, spread over every SM. With phases spread evenly,
 * 1/W of the head-states fold per token and no token carries a whole fold.
 * Arguments otherwise as lq_append.
 */
int lq_decode_step(const lq_config* cfg, void* state, int64_t n_states, int32_t phase, const float* q,
                   const float* k, const float* v, const float* alpha, const float* beta, float* o,
                   lq_stream_t stream);

/*
 * lq_decode_step with phase LQ_PHASE_ANY, for callers that cannot allocate
 * device memory: an engine that owns all device memory and hands each part of
 * the model only fixed buffers, where a cudaMalloc on the decode path would
 * stall the device and can fail once memory is full. The mixed-phase step needs
 * scratch: a list of the head-states whose window the token fills, and two
 * counters. lq_decode_step keeps it in the state buffer's work-list plane and
 * header; this call keeps it instead in a fixed array inside the library's own
 * device image, 256 KB plus 256 bytes, which every GPU that loads the library
 * holds until the process exits. It allocates nothing and leaves the state
 * buffer's work-list plane and header counters untouched. The pages have no
 * counterpart to this call; it is a deployment variant.
 *   - The first call on a device looks up the array's device address (with
 *     that device current) and remembers it; make that first call before
 *     any stream capture.
 *   - Every call on a device shares the one array. Each call clears the two
 *     counters first; calls whose kernels may overlap on the GPU (other
 *     streams, other threads) race on it and must be ordered by the caller.
 *   - Limits: n_states <= 65536 (LQ_ERR_INVALID_ARG above that); 8-bit codes
 *     with line compensators (code_bits = 8, comp_fit = 0), else
 *     LQ_ERR_UNSUPPORTED.
 * Arguments, results and device-side errors as lq_decode_step.
 */
int lq_decode_step_noalloc(const lq_config* cfg, void* state, int64_t n_states, const float* q, const float* k,
                           const float* v, const float* alpha, const float* beta, float* o, lq_stream_t stream);

/*
 * One two-record token for every head-state: a token whose update is two
 * rank-one sub-steps, as LeapQuant App. A ("Instances of the general update")
 * represents a DeltaProduct token with two steps:
 *   u1 = beta1 (v1 - S_{n-1}(alpha . k1)),  S_n     = S_{n-1} Diag(alpha) + u1 k1^T,
 *   u2 = beta2 (v2 - S_n k2),               S_{n+1} = S_n + u2 k2^T,
 *   o  = S_{n+1} q.
 * It stores records n = (k1, u1, alpha) and n+1 = (k2, u2, 1): exactly what
 * lq_decode_step does for (k1, v1, beta1, alpha) and then for (k2, v2, beta2,
 * alpha = 1), but with one read of the boundary. When the second record fills
 * the window (count == W), the head-state is folded in the same call.
 * `phase` is the record count every head-state holds before the call (0..W-2),
 * or LQ_PHASE_ANY. A head-state without room for both records (count > W-2)
 * is left unchanged and sets LQ_ERR_WINDOW_FULL; with an even W and only
 * two-record tokens that cannot happen.
 *   q, k1, k2 fp32 [n_states][d_k];  v1, v2, o fp32 [n_states][d_v]
 *   alpha fp32 [n_states] (GDN) or [n_states][d_k] (KDA);  beta1, beta2 fp32 [n_states]
 * Errors: as lq_decode_step; LQ_ERR_UNSUPPORTED when W < 2.
 */
int lq_decode_step2(const lq_config* cfg, void* state, int64_t n_states, int32_t phase, const float* q,
                    const float* k1, const float* v1, const float* beta1, const float* k2, const float* v2,
                    const float* beta2, const float* alpha, float* o, lq_stream_t stream);

/*
 * One RWKV7 token for every head-state (per-key decay: cfg->decay_per_key = 1).
 * RWKV7's erase direction differs from its write key, so LeapQuant App. A
 * ("Instances of the general update") splits the token into an erase and a
 * pure-write sub-step, two records:
 *   S_t = S_{t-1} (Diag(w) - kh (a . kh)^T) + v k^T,   o = S_t r;
 *   record n   = (a . kh, -(S_{n-1} kh), w)   the erase reads the state as it stands;
 *   record n+1 = (k, v, 1)                     the pure write reads nothing.
 * kh is the (normalized) erase direction, a its per-key rate, w the per-key decay.
 * Phases, folding and errors as lq_decode_step2 (two records per token; phase
 * 0..W-2 or LQ_PHASE_ANY); LQ_ERR_UNSUPPORTED for scalar decay or W < 2.
 *   r, w, kh, a, k fp32 [n_states][d_k];  v, o fp32 [n_states][d_v]
 */
int lq_decode_step_rwkv7(const lq_config* cfg, void* state, int64_t n_states, int32_t phase, const float* r,
                         const float* w, const float* kh, const float* a, const float* k, const float* v, float* o,
                         lq_stream_t stream);

/*
 * Write the state each head-state stands for, S_n = boundary x Diag(A_n) plus
 * the buffered records, in original coordinates (the fold's reconstruction,
 * without rounding: LeapQuant summary App. B.2 window unrolling, App. B.3
 * reconstruction in original coordinates), to S_out fp32 [n_states][d_v][d_k],
 * caller-owned, 16-byte aligned, not overlapping the state buffer. The state
 * is unchanged.
 */
int lq_export_state(const lq_config* cfg, const void* state, int64_t n_states, float* S_out, lq_stream_t stream);

/*
 * The fp32-state baseline: one decode token of the plain delta rule on whole
 * fp32 states: the kind of fp32-state kernel that LeapQuant's kernel speedups
 * are measured against ([LQ] §4.3; the update is §3.1 and App. A):
 *   u = beta (v - S (alpha . k)),  S <- S Diag(alpha) + u k^T,  o = S q.
 * S: fp32 [n_states][d_v][d_k] on the device, read and written in place (it is
 * not an lq state buffer: no header, codes or records). Token arguments as
 * lq_append; only cfg->d_k, d_v and decay_per_key are used. The summation
 * order is not pinned: results are compared with a tolerance. Errors:
 * LQ_ERR_INVALID_ARG for bad pointers, sizes or overlaps; nothing is checked on
 * the device.
 */
int lq_fp32_decode_step(const lq_config* cfg, float* S, int64_t n_states, const float* q, const float* k,
                        const float* v, const float* alpha, const float* beta, float* o, lq_stream_t stream);

/* ------------------------------------------------------------------------------
 * Generation: prompts in, tokens out, several hypotheses.
 *
 * Linear attention with a decay for each head (no delta rule):
 *   S_t = alpha_t S_{t-1} + v_t k_t^T,   o_t = S_t q_t,
 * on fp32 states S [d_v][d_k] (row = value channel, as everywhere in this header),
 * over whole prompts (lq_la_prefill) and for single tokens (lq_la_decode_step);
 * the selection of beam search (lq_beam_select) and the states that follow the
 * chosen hypotheses (lq_state_reorder, lq_fp32_state_reorder).
 * ------------------------------------------------------------------------------ */

/* Element types of q, k, v, o and of beam search's logits. Decays, states and scores are fp32. */
typedef enum { LQ_F32 = 0, LQ_BF16 = 1, LQ_F16 = 2 } lq_dtype;

typedef struct {
  int32_t d_k, d_v;         /* 128 and 128 in this build                                           */
  int32_t heads, key_heads; /* heads of v, o, alpha and S; heads of q and k. Head h reads key head  */
                            /* h / (heads / key_heads); heads must be a multiple of key_heads       */
  int32_t dtype;            /* lq_dtype of q, k, v and o                                             */
  int32_t reserved;         /* 0                                                                     */
  int64_t q_stride, k_stride, v_stride, o_stride; /* elements from one token to the next: at least   */
                            /* heads x 128 (key_heads x 128 for q, k), a multiple of 16 bytes; the   */
                            /* heads of a token and their channels are dense, so rows of one fused   */
                            /* projection can be passed as they are                                  */
  int64_t alpha_stride;     /* fp32 elements between tokens' decays: at least heads, or 0 for a decay */
                            /* that is the same for every token                                      */
} lq_la_config;

/* Dense token arrays: strides heads x 128, key_heads x 128 and heads; d_k = d_v = 128. */
void lq_la_config_default(lq_la_config* cfg, int32_t heads, int32_t key_heads, int32_t dtype);

/*
 * Bytes of workspace that are enough for lq_la_prefill with up to n_seqs sequences and
 * n_tokens tokens in all, none longer than max_len (0: not known); 0 when no such call
 * needs any or when an argument is invalid. Host only. A call needs some where sequences
 * may be split: 64 KB per head and segment, and 64 KB per head and sequence. (A call with
 * fewer tokens may be split where one with more is not: ask for the largest sizes once.)
 */
size_t lq_la_workspace_bytes(const lq_la_config* cfg, int64_t n_seqs, int64_t n_tokens, int64_t max_len);

/*
 * Linear attention over prompts: sequence b is tokens cu_seqlens[b] ..
 * cu_seqlens[b+1]-1 of the packed arrays; it starts from S0[b] (zero if S0 is
 * NULL) and leaves its last state in S_out[b] (not written if S_out is NULL).
 * lq_la_decode_step continues the same recurrence from S_out, in the order
 * [n_seqs][heads], as it is. The layout is also what lq_state_init, lq_state_init_range
 * and lq_fp32_decode_step take, but their tokens are delta-rule tokens, another
 * recurrence: hand them S_out only where a model changes over at that point.
 *   cu_seqlens int32 [n_seqs + 1] on the device, or NULL for one sequence of
 *              n_tokens; a sequence may be empty (its S_out is then its S0). A
 *              sequence whose bounds are not 0 <= begin <= end <= n_tokens, or
 *              that is longer than a stated max_len, is treated as empty.
 *   q, k       [n_tokens][key_heads][128], v, o [n_tokens][heads][128], of cfg->dtype
 *   alpha      fp32 [n_tokens][heads]. Any value is taken as the recurrence takes
 *              it; 0 forgets the state.
 *   S0, S_out  fp32 [n_seqs][heads][128][128]; S_out may be S0 itself (in place)
 *   max_len    the longest sequence, or 0 if the caller does not know it
 *   workspace  256-byte aligned, lq_la_workspace_bytes(...) bytes for these sizes or
 *              larger ones (NULL if that is 0); its contents need not be kept.
 * States are kept in fp32 and their products are taken to fp32's accuracy whatever the
 * type of the tokens; o is rounded once to cfg->dtype (with 16-bit types, products
 * that only o needs are taken to that type's accuracy).
 * A token's value, however large, infinite or NaN, reaches its own and later tokens
 * of its sequence only. Tokens that belong to no sequence get no output. o must not
 * overlap an input. Sequences must not overlap one another. Errors:
 * LQ_ERR_INVALID_ARG, LQ_ERR_UNSUPPORTED; nothing is reported from the device, but
 * should a bounded wait inside the kernel for bf16 tokens give up (2 s; it never
 * should), the outputs of that head's sequence or segment and its last state are NaN.
 * A head of a sequence whose state or outputs are not finite takes a slow path, token by
 * token (of a split sequence the segment, or the whole where a state between segments is
 * not finite); with bf16 tokens so do decays outside 0..1 and outputs past 1e18.
 */
int lq_la_prefill(const lq_la_config* cfg, int64_t n_seqs, int64_t n_tokens, int64_t max_len,
                  const int32_t* cu_seqlens, const void* q, const void* k, const void* v, const float* alpha,
                  const float* S0, float* S_out, void* o, void* workspace, size_t workspace_bytes,
                  lq_stream_t stream);

/*
 * The recurrent form: one token for each of n_seqs sequences on fp32 states
 * S [n_seqs][heads][128][128], read and written in place. Token arrays as above with
 * one token per sequence (strides between sequences). Errors: as lq_la_prefill.
 */
int lq_la_decode_step(const lq_la_config* cfg, float* S, int64_t n_seqs, const void* q, const void* k, const void* v,
                      const float* alpha, void* o, lq_stream_t stream);

/* Bytes of workspace lq_beam_select needs (0 if an argument is invalid). Host only. */
size_t lq_beam_workspace_bytes(int64_t batch, int32_t beams, int64_t vocab, int32_t n_best);

/*
 * The selection of beam search: for each of `batch` requests the n_best
 * continuations of its `beams` hypotheses, by
 *   score(b, t) = scores[b] + logits[b][t] - log sum_t' exp(logits[b][t']),
 * best first; equal scores go to the lowest b * vocab + t.
 *   logits     [batch][beams][vocab] of dtype; row_stride elements from one
 *              hypothesis' row to the next (>= vocab; any alignment)
 *   scores     fp32 [batch][beams], the hypotheses' scores so far
 *   out_scores fp32 [batch][n_best]; out_parent, out_token int32 [batch][n_best]:
 *              the hypothesis continued (0..beams-1) and its token
 *   beams 1..32, n_best 1..64 and at most beams * vocab, vocab 1..2^31-1 / beams
 * A masked token (logit -inf) scores -inf. So does every token of a hypothesis
 * whose score or log-sum-exp is not finite (a dead hypothesis, a row that is all
 * -inf, a NaN or +inf logit): they are chosen only when the finite candidates run
 * out, in the order of their index. Scores are compared in 64 bits; wherever the
 * order of the n_best hangs on it, log-sum-exps are good to 1e-10 (out_scores: to a
 * few 1e-7). Requests in which two hypotheses' candidates lie closer than 5e-6 take
 * longer: about 50 us for each such hypothesis of 131,071 tokens.
 * workspace: 256-byte aligned, lq_beam_workspace_bytes(...) bytes; contents need
 * not be kept. Outputs must not overlap the inputs or each other.
 */
int lq_beam_select(int32_t dtype, int64_t batch, int32_t beams, int64_t vocab, int32_t n_best, const void* logits,
                   int64_t row_stride, const float* scores, float* out_scores, int32_t* out_parent,
                   int32_t* out_token, void* workspace, size_t workspace_bytes, lq_stream_t stream);

/*
 * Let the head-states of a state buffer follow the hypotheses chosen: afterwards
 * beam b of group g holds what beam parent[g * beams + b] held before, in place.
 * The buffer's head-states are ordered
 *   s = ((x * groups + g) * beams + b) * inner + i,  x < outer, i < inner,
 * e.g. outer 1, inner = layers * heads for [request][beam][layer][head], or
 * outer = layers, inner = heads for [layer][request][beam][head]; the parents
 * (int32 [groups][beams] on the device) hold for every x and i, and
 * n_states = outer * groups * beams * inner. A beam that keeps its place is not
 * touched; of the others the boundary and the records held move. parent = 0 for
 * every b forks a group's first beam. beams 1..32.
 * On the device: LQ_ERR_PARENT for a parent outside 0..beams-1, LQ_ERR_STATE for a
 * buffer or record count that is not valid; that group is left unchanged.
 */
int lq_state_reorder(const lq_config* cfg, void* state, int64_t n_states, int64_t outer, int64_t groups,
                     int32_t beams, int64_t inner, const int32_t* parent, lq_stream_t stream);

/* The same for fp32 states S [n_states][128][128]. A group with a parent outside
 * 0..beams-1 is left unchanged; there is no status word to say so. */
int lq_fp32_state_reorder(float* S, int64_t n_states, int64_t outer, int64_t groups, int32_t beams, int64_t inner,
                          const int32_t* parent, lq_stream_t stream);

/* ------------------------------------------------------------------------------
 * State space layers: the short causal convolution in front of a recurrence, and the
 * selective scan, over packed prompts (lq_conv_prefill, lq_ssm_prefill) and for single
 * tokens on their own states (lq_conv_decode_step, lq_ssm_decode_step); and what a
 * model's logits say about given tokens (lq_token_logprobs).
 *
 * Packed sequences are lq_la_prefill's: sequence b is tokens cu_seqlens[b] ..
 * cu_seqlens[b+1]-1 (int32 [n_seqs + 1] on the device; NULL: one sequence of n_tokens).
 * A sequence may be empty; one whose bounds are not 0 <= begin <= end <= n_tokens, or
 * that is longer than a stated max_len, is treated as empty: its last state is its first
 * one. Tokens that belong to no sequence get no output, and sequences must not overlap
 * one another. Outputs must not overlap inputs, except where a state may be in place.
 * Token arrays, weights and states of these calls need the alignment of their elements
 * only; 16-byte aligned arrays and strides are faster where the text says so.
 * Errors of these calls: LQ_ERR_INVALID_ARG, LQ_ERR_UNSUPPORTED, LQ_ERR_CUDA; nothing is
 * reported from the device.
 * ------------------------------------------------------------------------------ */

typedef struct {
  int32_t channels;           /* 1..2^20                                                              */
  int32_t width;              /* W: taps, 2..4                                                         */
  int32_t dtype;              /* lq_dtype of x, y and the states                                       */
  int32_t silu;               /* 1: y = s / (1 + e^-s) of the sum s; 0: the sum itself                 */
  int64_t x_stride, y_stride; /* elements from one token to the next, at least channels                */
} lq_conv_config;

/* Dense token arrays. */
void lq_conv_config_default(lq_conv_config* cfg, int32_t channels, int32_t width, int32_t dtype, int32_t silu);

/*
 * Causal convolution of every channel over packed prompts:
 *   y[t][c] = act(bias[c] + sum_j weight[c][j] x[t - (W-1) + j][c]),   j = 0..W-1,
 * where the inputs before a sequence are S0[b] (zero if NULL), its W-1 inputs before
 * the first, oldest first.
 *   x, y       [n_tokens][channels] of cfg->dtype (tokens may lie apart)
 *   weight     fp32 [channels][width];  bias fp32 [channels] or NULL
 *   S0, S_out  [n_seqs][W-1][channels] of cfg->dtype, or NULL; S_out gets the last W-1
 *              inputs of each sequence, S0's among them where it has fewer tokens; it may
 *              be S0 itself
 * n_tokens is at most 2^31 - 256. Sums are kept in fp32; y is rounded once. Faster where x, y, S0, S_out, weight and the
 * strides are multiples of 16 bytes and so is a row of channels.
 */
int lq_conv_prefill(const lq_conv_config* cfg, int64_t n_seqs, int64_t n_tokens, int64_t max_len,
                    const int32_t* cu_seqlens, const void* x, const float* weight, const float* bias, const void* S0,
                    void* S_out, void* y, lq_stream_t stream);

/*
 * One token for each of n_seqs sequences: x, y [n_seqs][channels]; S [n_seqs][W-1][channels]
 * holds each sequence's last inputs, oldest first, and takes x in place of the oldest.
 */
int lq_conv_decode_step(const lq_conv_config* cfg, void* S, int64_t n_seqs, const void* x, const float* weight,
                        const float* bias, void* y, lq_stream_t stream);

typedef struct {
  int32_t channels, n_state; /* 1..2^20 channels of 1..64 states                                          */
  int32_t groups;            /* B and C are shared by channels / groups channels in a row; a divisor        */
  int32_t dtype;             /* lq_dtype of x, dt, z, B, C and y                                             */
  int32_t softplus;          /* 1: d = log(1 + e^(dt + dt_bias)); 0: d = dt + dt_bias                         */
  int32_t reserved;          /* 0                                                                            */
  int64_t x_stride, dt_stride, z_stride, y_stride; /* elements from one token to the next: at least channels */
  int64_t b_stride, c_stride;                      /* at least groups x n_state                              */
} lq_ssm_config;

/* Dense token arrays. */
void lq_ssm_config_default(lq_ssm_config* cfg, int32_t channels, int32_t n_state, int32_t groups, int32_t dtype,
                           int32_t softplus);

/*
 * Bytes of workspace that are enough for lq_ssm_prefill with up to n_seqs sequences and
 * n_tokens tokens in all, that state a max_len of at most max_len (0: calls that state
 * none, or any); 0 when no such call needs any or when an argument is invalid. Host only.
 * (A call that leaves its max_len out counts as one of n_tokens, however short its
 * sequences are: ask with 0 for it.)
 */
size_t lq_ssm_workspace_bytes(const lq_ssm_config* cfg, int64_t n_seqs, int64_t n_tokens, int64_t max_len);

/*
 * Selective state space scan over packed prompts. For channel c of group g = c / (channels
 * / groups) and its states n, with d = softplus(dt[t][c] + dt_bias[c]) (or without it):
 *   h[n] <- exp(d A[c][n]) h[n] + d x[t][c] B[t][g][n],
 *   y[t][c] = (sum_n C[t][g][n] h[n] + D[c] x[t][c]) * z / (1 + e^-z),   z = z[t][c]
 * (the last factor only where z is given).
 *   x, dt, z, y  [n_tokens][channels] of cfg->dtype (tokens may lie apart); z may be NULL
 *   B, C         [n_tokens][groups][n_state] of cfg->dtype; a token's are dense
 *   A            fp32 [channels][n_state]; D, dt_bias fp32 [channels] or NULL (no such term)
 *   S0, S_out    fp32 [n_seqs][channels][n_state] or NULL (a zero first state, no last
 *                one); S_out may be S0 itself
 *   max_len      the longest sequence, or 0 if the caller does not know it: the call is
 *                then divided as if one sequence had all tokens, which costs it two more
 *                launches, and up to a quarter of its time where prompts are ragged
 *   workspace    256-byte aligned, lq_ssm_workspace_bytes(...) bytes for these sizes or
 *                larger ones (NULL if that is 0); its contents need not be kept, but calls
 *                that may run at the same time (streams, graphs) need one each
 * n_tokens is at most 2^31 - 256. States and sums are kept in fp32; y is rounded once. Any value is taken as the recurrence
 * takes it; a token's value reaches its own and later tokens of its sequence only. (Where
 * n_state is not 8, 16, 32 or 64, outputs that an infinite x, d or d x makes infinite may be NaN,
 * here and in lq_ssm_decode_step; states are as the recurrence has them.) Long
 * sequences are split into segments; channels with a positive A, a negative or infinite d,
 * or values past 1e30 pass from segment to segment token by token, which is slow.
 */
int lq_ssm_prefill(const lq_ssm_config* cfg, int64_t n_seqs, int64_t n_tokens, int64_t max_len,
                   const int32_t* cu_seqlens, const void* x, const void* dt, const float* A, const void* B,
                   const void* C, const float* D, const void* z, const float* dt_bias, const float* S0, float* S_out,
                   void* y, void* workspace, size_t workspace_bytes, lq_stream_t stream);

/*
 * The recurrent form: one token for each of n_seqs sequences on fp32 states
 * S [n_seqs][channels][n_state], in place. Token arrays as above with one token per
 * sequence (strides between sequences).
 */
int lq_ssm_decode_step(const lq_ssm_config* cfg, float* S, int64_t n_seqs, const void* x, const void* dt,
                       const float* A, const void* B, const void* C, const float* D, const void* z,
                       const float* dt_bias, void* y, lq_stream_t stream);

/*
 * What each row of logits says, with lse = log sum_t exp(logits[r][t]):
 *   logprob[r]   = logits[r][tokens[r]] - lse: 0 where tokens[r] is negative (no token
 *                  asked for), NaN where it is not below vocab
 *   entropy[r]   = -sum_t p_t log p_t, p_t = exp(logits[r][t] - lse), in nats
 *   top_token[r][i], top_logprob[r][i]: the n_top largest logits, largest first, equal
 *                  ones in the order of their index, and their log probabilities
 *   logits       [rows][vocab] of dtype; row_stride elements from one row to the next
 *                (>= vocab; any alignment)
 *   tokens       int32 [rows], or NULL with logprob NULL; entropy fp32 [rows] or NULL;
 *                top_logprob fp32 and top_token int32 [rows][n_top], NULL if n_top is 0
 *   vocab 1..2^31-1, n_top 0..32 and at most vocab
 * Masked tokens (-inf) have probability 0 and log probability -inf, and are among the
 * n_top only when the others run out. A row without a distribution (all -inf, a NaN or a
 * +inf among it) gets NaN for every number and -1 for its top tokens (0 still where no
 * token is asked for). Sums are kept in fp32. Rows whose largest logits are very many equal
 * ones, or come in rising order, take longer.
 */
int lq_token_logprobs(int32_t dtype, int64_t rows, int64_t vocab, int32_t n_top, const void* logits,
                      int64_t row_stride, const int32_t* tokens, float* logprob, float* entropy, float* top_logprob,
                      int32_t* top_token, lq_stream_t stream);

/*
 * Synchronize `stream`, then read the state buffer's status word: LQ_OK or the
 * first device-side error recorded since lq_state_init / lq_clear_status.
 * *bad_state (if non-NULL) receives the index of the head-state that set it.
 */
int lq_get_status(const void* state, int64_t* bad_state, lq_stream_t stream);

/* Reset the status word to LQ_OK (enqueued on `stream`). */
int lq_clear_status(void* state, lq_stream_t stream);

/* Thread-local description of the last host-side error of this thread ("" if none). */
const char* lq_last_error(void);

/* Library version: major * 10000 + minor * 100 + patch. */
int lq_version(void);

/*
 * Test hook for the kernels' failure path; not for production use. Every
 * wait inside a kernel (for the bulk copies that stage a head-state into
 * shared memory) is bounded; when the bound runs out the kernel records
 * LQ_ERR_TIMEOUT in the status word with the head-state's index, leaves that
 * head-state unchanged and returns, so the context stays usable. After
 * LQ_ERR_TIMEOUT treat every output of that call as untrusted (copies may
 * still have been landing in the shared memory of the CTA that gave up) and
 * re-initialise the state before going on.
 * This call sets, for later calls made by this thread only:
 *   wait_ns          the bound on each wait (1..1e9 ns; 0 restores the 1 s default);
 *   extra_tx_append  bytes the append kernels (lq_append, lq_decode_step below
 *                    the window's last token, the two-record and RWKV7 steps)
 *                    announce to their barrier beyond those they copy (0..1024),
 *                    and so does lq_la_prefill for each chunk of bf16 tokens;
 *   extra_tx_fold    the same for the kernels that stage the records (the fused
 *                    last token of a window, lq_fold, the list fold, lq_export_state).
 * With an extra byte count the copies all land and the barrier never completes,
 * so the wait runs out after wait_ns (lq_la_prefill: twice that, per wait). lq_state_init has no such wait (it reads
 * S0 with plain loads). The pages have no counterpart; the failure-detection
 * design is this library's. Errors: LQ_ERR_INVALID_ARG for values out of range.
 */
int lq_debug_set_wait(uint64_t wait_ns, int32_t extra_tx_append, int32_t extra_tx_fold);

#ifdef __cplusplus
}
#endif

#endif /* LQ_H */
