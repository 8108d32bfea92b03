/*
 * lar.h -- C ABI of the recurrent linear-attention decode library (GB300, sm_103a).
 *
 * One decode step of linear attention with a fixed-size recurrent state per
 * (sequence, value head), kept in a paged fp32 state pool.  Three forms:
 *
 *   gdn_decode  gated delta rule, scalar decay per (token, v-head)
 *   kda_decode  gated delta rule, decay per key channel
 *   la_decode   Lightning Attention: decay per head, no delta term
 *
 * with variants for per-token pool slots (gdn_decode_tokens, kda_decode_tokens),
 * token-major spans of any length per sequence (gdn_decode_varlen,
 * kda_decode_varlen, la_decode_varlen) and the chunked form of the latter for
 * long spans (gdn_prefill, kda_prefill, la_prefill).  Around them stand the short
 * causal convolution in front of such a layer (conv_*), a further recurrent form,
 * the selective state space scan (ssm_*), the verification of drafted tokens
 * that makes the accepted counts (spec_verify), the draw of the tokens themselves
 * (sample_tokens), and, for the softmax-attention layers of hybrid models, a paged
 * key/value cache (kv_append) and the attention over it (attn_decode).  The chunked calls also set their
 * kernel's shared-memory limit (a function attribute) on every call; capturing
 * them into a CUDA graph has not been tested (the other calls' capture and
 * replay are).
 *
 * The delta-rule recurrence is the one the ROCm/aiter PR #4584 "Fused Gluon KDA
 * decode path" advisory review states: per token
 *     S <- exp(g_t) S;   S <- S + beta_t k_t (x) (v_t - S^T k_t);   o_t = S^T q_t
 * with S a K x V matrix (for KDA exp(g_t) scales key channel k by exp(g_t[k])).
 * Lightning Attention: S <- lambda_h S + k_t (x) v_t;  o_t = S^T q_t.
 * Every output is multiplied by `scale`.
 *
 * Pool addressing (flashinfer "fp32 sibling of #3268" 4D-pool page; cuLA PR #75):
 *   the state of batch entry b and v-head hv is read from slot read_idx[b] and
 *   written to slot write_idx[b] (NULL write_idx: the read slot).  A negative
 *   read index means a zero initial state; a negative write index skips the
 *   writeback.  Every pool byte outside the written (slot, head) states is left
 *   bit-identical.  The pool is read and written in place through its strides.
 *
 * Layouts (all strides in ELEMENTS and non-negative; shape[] is logical):
 *   S is stored transposed: pool[slot][hv][v][k] = S[k][v], k fastest.
 *   pool   fp32 or bf16, rank 4 [P, HV, V, K] (any slot/head/row strides), or
 *          rank 3 [P*HV, V, K] (slot p, head hv at row p*HV + hv).  k stride
 *          must be 1; the data pointer 16-byte aligned; slot, head and row
 *          strides multiples of 16 bytes (rows move as 16-byte chunks).  The
 *          arithmetic is fp32 either way: a bf16 state is widened on load and
 *          rounded to nearest even once per store.
 *   q, k   [B, T, H, K]  (rank 3 [B, H, K] means T = 1); fp32 or bf16, any strides
 *          (so q/k/v may be head-dim slices of one fused buffer).
 *   v      [B, T, HV, V] (rank 3 [B, HV, V]); fp32 or bf16, any strides.
 *   out    [B, T, HV, V] (rank 3 [B, HV, V]); fp32 or bf16 (round to nearest even).
 *          With LAR_STATE_KV (gdn_decode / kda_decode only) the state is held
 *          untransposed, pool[slot][hv][k][v] = S[k][v] with v fastest (the
 *          "nontranspose" layout of the flashinfer GDN decode kernels): rank 4
 *          [P, HV, K, V] or rank 3 [P*HV, K, V], v stride 1, V a multiple of
 *          16 bytes of elements (4 fp32 or 8 bf16); inter is [B, T, HV, K, V].
 *   inter  NULL, or fp32 or bf16 [B, T, HV, V, K] (rank 4 [B, HV, V, K] when
 *          T = 1): the state after each token; same alignment rules as the
 *          pool; its type is independent of the pool's.
 *   read_idx, write_idx  rank 1 [B], int32 or int64, any stride.
 *   H divides HV; v-head hv reads q/k head hv / (HV / H).
 *   K must be 16, 32, 64 or 128; V from 1 to 2^24; T from 1 to 16;
 *   B and HV at most 65535.
 *
 * Ownership and execution: the caller owns every buffer (device memory).
 * Every pointer of a call (tensor data and dev_err) must be memory of the
 * CUDA device that is current on the calling thread, and `stream` a stream of
 * that device: the kernel is launched there and dereferences the pointers
 * as given (memory of another device is not checked here, and a kernel that
 * touches it without peer access faults).  The library allocates nothing, keeps no state between calls and never
 * synchronises: each call validates on the host and then enqueues one kernel
 * on `stream` (a cudaStream_t; NULL is the legacy default stream).  The kernel
 * is launched with programmatic dependent launch: it may be scheduled while
 * the previous kernel on the stream drains, but it reads no memory before that
 * kernel has completed, so stream order is kept.  Calls may be made from
 * several host threads at once (the only host-side state is a per-device cache
 * of occupancy figures, filled under a lock on a kernel's first call) and may
 * be captured into CUDA graphs; make one uncaptured call of a configuration
 * first so that the one-time setup does not fall inside the capture.
 *
 * Errors: a host-detectable problem returns a status other than LAR_OK BEFORE
 * anything is launched (nothing is written).  Slot indices >= P are caught on
 * the device: that entry's state is not read (zero state) / not written, and
 * the bits LAR_DEVERR_* are OR-ed into *dev_err when dev_err is not NULL (a
 * caller-owned device int32, 4-byte aligned (else LAR_ERR_ALIGN) and clear of
 * every tensor of the call (else LAR_ERR_ALIAS); never cleared by the
 * library).  No kernel traps or asserts.
 *
 * Aliasing: pool, out and inter must not overlap one another or any input
 * (checked on the host by address range).  Entries must not read a slot that
 * another entry writes, and write slots must be distinct; such calls are
 * undefined (the kernels run entries concurrently).  In-place update (write
 * slot == read slot of the same entry) is allowed.
 */
#ifndef LAR_H_
#define LAR_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    LAR_F32 = 0,
    LAR_BF16 = 1,
    LAR_I32 = 2,
    LAR_I64 = 3,
    LAR_E4M3 = 4   /* 8 bits, 4 of exponent and 3 of mantissa, no infinities: pages of kv_append and attn_decode */
} lar_dtype;

/* A strided view of device memory.  data points at element [0, ..., 0]. */
typedef struct {
    void* data;
    int32_t dtype;      /* lar_dtype */
    int32_t ndim;       /* 1..5 */
    int64_t shape[5];
    int64_t stride[5];  /* in elements */
} lar_tensor;

typedef enum {
    LAR_OK = 0,
    LAR_ERR_NULL = 1,        /* a required tensor or pointer is NULL */
    LAR_ERR_DTYPE = 2,       /* unsupported dtype for that argument */
    LAR_ERR_RANK = 3,        /* wrong ndim */
    LAR_ERR_SHAPE = 4,       /* shapes disagree, or a size outside the supported range */
    LAR_ERR_STRIDE = 5,      /* k stride of pool/inter not 1, or negative strides */
    LAR_ERR_ALIGN = 6,       /* pool/inter pointer or strides not multiples of 16 bytes, or dev_err
                                not 4-byte aligned */
    LAR_ERR_ARG = 7,         /* inconsistent flags/arguments (e.g. A_log without LAR_GATE_RAW) */
    LAR_ERR_ALIAS = 8,       /* an output (dev_err included) overlaps another output or an input */
    LAR_ERR_LAUNCH = 9       /* the CUDA launch itself failed */
} lar_status;

/* flags for gdn_decode / kda_decode */
enum {
    LAR_QK_L2NORM = 1u << 0, /* q, k <- x / sqrt(sum x^2 + 1e-6) over K, in kernel */
    LAR_GATE_RAW = 1u << 1,  /* g <- -exp(A_log[hv]) * softplus(g + dt_bias), in kernel */
    LAR_BETA_RAW = 1u << 2,  /* beta <- 1 / (1 + exp(-beta)), in kernel */
    LAR_STATE_KV = 1u << 3   /* pool and inter hold S as [k][v] (v fastest), see below */
};

/* flags for conv_* and ssm_* */
enum {
    LAR_SILU = 1u << 4,       /* conv_*: out <- y / (1 + exp(-y)), in kernel */
    LAR_DT_SOFTPLUS = 1u << 5 /* ssm_*: dt <- softplus(dt + dt_bias), in kernel */
};

/* flags for kv_append */
enum {
    LAR_ROPE_INTERLEAVED = 1u << 6 /* rotated pairs are dimensions (2i, 2i + 1), not (i, i + rot / 2) */
};

/* bits OR-ed into *dev_err */
enum {
    LAR_DEVERR_READ_SLOT = 1,  /* some read_idx[b] >= P (that entry started from zero) */
    LAR_DEVERR_WRITE_SLOT = 2, /* some write slot >= P (that writeback was skipped) */
    LAR_DEVERR_ACCEPTED = 4,   /* some num_accepted[b] outside [1, T] (that entry started from zero) */
    LAR_DEVERR_SEQLEN = 8,     /* varlen: some span cu_seqlens[n]..[n+1] reversed or past the token
                                  arrays (treated as empty: the read state goes to the write slot) */
    LAR_DEVERR_TIMEOUT = 16,   /* chunked prefill: a bounded wait for the tensor cores gave up; that
                                  (sequence, head) skipped the rest of its span and its writeback */
    LAR_DEVERR_DRAFT = 32,     /* spec_verify: some drafted token outside [0, V) (rejected), or some
                                  num_draft[b] outside [0, T - 1] (taken as the nearer end) */
    LAR_DEVERR_PROBS = 64,     /* spec_verify: some row to draw from has no positive finite weight,
                                  or a sum that fp32 does not hold (its token is -1); sample_tokens:
                                  some row has no logit above -infinity (its token is -1) */
    LAR_DEVERR_PAGE = 128      /* kv_append, attn_decode: some block_table entry >= P (not written, not seen) */
};

/*
 * Gated delta rule, scalar decay (GDN).  Interface of flashinfer's
 * `gated_delta_rule_mtp` (initial_state = pool, initial_state_indices =
 * read_idx, output_state_indices = write_idx, cache_intermediate_states =
 * inter), recurrence from the aiter review.
 *   g       [B, T, HV] (rank 2 [B, HV] when T = 1): log-decay, or the raw gate
 *           input when LAR_GATE_RAW; fp32 or bf16, any strides.
 *   beta    [B, T, HV] (rank 2 when T = 1): fp32 or bf16; a logit when LAR_BETA_RAW.
 *   A_log   fp32 [HV]; required with LAR_GATE_RAW, must be NULL without it.
 *   dt_bias fp32 [HV]; optional with LAR_GATE_RAW (zero), must be NULL without it.
 */
lar_status gdn_decode(const lar_tensor* q, const lar_tensor* k, const lar_tensor* v,
                      const lar_tensor* g, const lar_tensor* beta,
                      const lar_tensor* A_log, const lar_tensor* dt_bias,
                      const lar_tensor* pool,
                      const lar_tensor* read_idx, const lar_tensor* write_idx,
                      const lar_tensor* out, const lar_tensor* inter,
                      float scale, uint32_t flags, int32_t* dev_err, void* stream);

/*
 * Gated delta rule, per-key-channel decay (KDA, "Kimi Delta Attention" in the
 * aiter review; its wrapper consumes A_log, dt_bias and use_gate_in_kernel).
 * Same as gdn_decode except:
 *   g       [B, T, HV, K] (rank 3 [B, HV, K] when T = 1)
 *   dt_bias fp32 [HV * K], channel k of head hv at hv * K + k
 */
lar_status kda_decode(const lar_tensor* q, const lar_tensor* k, const lar_tensor* v,
                      const lar_tensor* g, const lar_tensor* beta,
                      const lar_tensor* A_log, const lar_tensor* dt_bias,
                      const lar_tensor* pool,
                      const lar_tensor* read_idx, const lar_tensor* write_idx,
                      const lar_tensor* out, const lar_tensor* inter,
                      float scale, uint32_t flags, int32_t* dev_err, void* stream);

/*
 * Lightning-Attention decode (cuLA PR #75): S <- lambda_h S + k (x) v, o = S^T q.
 * HV == H here: q, k [B, T, H, K], v and out [B, T, H, V] (rank 3 for T = 1).
 *   decay  fp32 [H]: lambda_h.
 *   pool   rank 3 [P*H, V, K] (the page's layout; the state of entry b, head h
 *          is row read_idx[b] * H + h), or rank 4 [P, H, V, K] whose slot
 *          stride equals H times its head stride.  The first dimension of a
 *          rank-3 pool must be a multiple of H.
 */
lar_status la_decode(const lar_tensor* q, const lar_tensor* k, const lar_tensor* v,
                     const lar_tensor* decay, const lar_tensor* pool,
                     const lar_tensor* read_idx, const lar_tensor* write_idx,
                     const lar_tensor* out, const lar_tensor* inter,
                     float scale, int32_t* dev_err, void* stream);

/*
 * Multi-token decode with per-token pool slots (speculative / MTP verify).
 * The aiter KDA review describes these paged per-token state slots and the
 * seed chosen by the number of accepted draft tokens, and lists the two ways
 * such a wrapper went wrong (a flat index table read with the wrong row
 * stride; an accepted count of 0 reading before its row); both are closed here.
 *
 *   state_idx     int32/int64 [B, T] (rank 2 only): the state after token t of
 *                 entry b is written to pool slot state_idx[b][t]; a negative
 *                 slot skips that store.  There is no other writeback.
 *   num_accepted  int32/int64 [B] or NULL: the seed state of entry b is read
 *                 from slot state_idx[b][num_accepted[b] - 1] (the state after
 *                 the last accepted token of the previous step, which stored
 *                 its token states in the same row).  A count outside [1, T]
 *                 starts that entry from a zero state and sets
 *                 LAR_DEVERR_ACCEPTED.
 *   read_idx      [B] or NULL: the seed slot when num_accepted is NULL.
 *                 Exactly one of read_idx and num_accepted must be given.
 * All other arguments as gdn_decode / kda_decode (no write_idx, no inter).
 * The seed of an entry may be one of its own per-token slots (each state row
 * is read before it is overwritten); across entries the aliasing rules of
 * gdn_decode apply.
 */
lar_status gdn_decode_tokens(const lar_tensor* q, const lar_tensor* k, const lar_tensor* v,
                             const lar_tensor* g, const lar_tensor* beta,
                             const lar_tensor* A_log, const lar_tensor* dt_bias,
                             const lar_tensor* pool, const lar_tensor* read_idx,
                             const lar_tensor* num_accepted, const lar_tensor* state_idx,
                             const lar_tensor* out, float scale, uint32_t flags,
                             int32_t* dev_err, void* stream);

lar_status kda_decode_tokens(const lar_tensor* q, const lar_tensor* k, const lar_tensor* v,
                             const lar_tensor* g, const lar_tensor* beta,
                             const lar_tensor* A_log, const lar_tensor* dt_bias,
                             const lar_tensor* pool, const lar_tensor* read_idx,
                             const lar_tensor* num_accepted, const lar_tensor* state_idx,
                             const lar_tensor* out, float scale, uint32_t flags,
                             int32_t* dev_err, void* stream);

/*
 * Variable-length spans (the "varlen" mode of the aiter KDA decode path): N
 * sequences whose tokens are packed token-major, sequence n owning tokens
 * cu_seqlens[n] .. cu_seqlens[n+1] - 1 (any length, 0 included; long spans are
 * a fused-recurrent prefill that leaves its final state in the pool).  Each
 * sequence starts from slot read_idx[n] (negative: zero state), runs the same
 * recurrence token by token, writes o for each of its tokens and its final
 * state to write_idx[n] (negative: skipped; an empty span copies the read
 * state there).  Tokens outside every span are not written.
 *   q, k        [Ntok, H, K];  v, out  [Ntok, HV, V];  any strides, fp32 or bf16
 *   g, beta     [Ntok, HV] (KDA g: [Ntok, HV, K])
 *   cu_seqlens  [N + 1], int32 or int64, non-decreasing from 0 to at most Ntok
 *               (a span that is reversed or runs past Ntok is treated as empty
 *               and sets LAR_DEVERR_SEQLEN in *dev_err; spans that overlap,
 *               which non-decreasing offsets rule out, write the shared output
 *               rows in an unspecified order)
 *   read_idx, write_idx  [N] (write_idx NULL: the read slot)
 *   inter       NULL, or [Ntok, HV, V, K] fp32 or bf16: the state after each token
 *   pool        as for gdn_decode, [v][k] layout only (LAR_STATE_KV is rejected)
 * Flags, A_log, dt_bias and decay as for the fixed-T calls.  N <= 65535,
 * Ntok < 2^31.
 * Without a state cache (inter NULL) and at K = V = 128, spans of 16 tokens or
 * more are computed in the chunked form of gdn_prefill / kda_prefill /
 * la_prefill below (equal to the recurrence up to rounding, and several times
 * cheaper per token on such spans) and the shorter ones token by token: two
 * kernels on `stream`, each choosing its spans on the device from cu_seqlens.
 * The chunked kernel's grid has a row per possible long span (at most
 * Ntok / 16 when the valid spans are disjoint) and is not launched when Ntok <
 * 16; if any span is reversed (then valid spans may overlap) every span runs
 * token by token.  With a state cache every span runs token by token.
 */
lar_status gdn_decode_varlen(const lar_tensor* q, const lar_tensor* k, const lar_tensor* v,
                             const lar_tensor* g, const lar_tensor* beta,
                             const lar_tensor* A_log, const lar_tensor* dt_bias,
                             const lar_tensor* pool, const lar_tensor* cu_seqlens,
                             const lar_tensor* read_idx, const lar_tensor* write_idx,
                             const lar_tensor* out, const lar_tensor* inter,
                             float scale, uint32_t flags, int32_t* dev_err, void* stream);

lar_status kda_decode_varlen(const lar_tensor* q, const lar_tensor* k, const lar_tensor* v,
                             const lar_tensor* g, const lar_tensor* beta,
                             const lar_tensor* A_log, const lar_tensor* dt_bias,
                             const lar_tensor* pool, const lar_tensor* cu_seqlens,
                             const lar_tensor* read_idx, const lar_tensor* write_idx,
                             const lar_tensor* out, const lar_tensor* inter,
                             float scale, uint32_t flags, int32_t* dev_err, void* stream);

lar_status la_decode_varlen(const lar_tensor* q, const lar_tensor* k, const lar_tensor* v,
                            const lar_tensor* decay, const lar_tensor* pool,
                            const lar_tensor* cu_seqlens, const lar_tensor* read_idx,
                            const lar_tensor* write_idx, const lar_tensor* out,
                            const lar_tensor* inter, float scale, int32_t* dev_err, void* stream);

/*
 * Chunked prefill over variable-length spans (the form of the recurrence for
 * long spans): the same operation and arguments as gdn_decode_varlen /
 * la_decode_varlen, computed 32 tokens at a time with the recurrence unrolled
 * over each chunk into matrix products and a unit lower-triangular solve (the
 * per-token recurrence of the aiter KDA review, rearranged; equal up to
 * rounding).  Every output row of a token inside a span and every written state
 * is produced; there is no per-token state cache (the chunked form never forms
 * the intermediate states).
 *   K = V = 128 only (other shapes: LAR_ERR_SHAPE; use *_decode_varlen).
 * One CTA per (sequence, v-head) pair keeps the state on chip (registers and
 * tensor memory) for the whole span and runs the chunk's products on the
 * tensor cores; the work of a sequence is spread over its heads, so a span
 * shorter than a chunk costs a whole chunk (the *_decode_varlen calls send
 * such spans token by token).
 *
 * kda_prefill: KDA's per-key-channel decay moves into the chunk's dot
 * products: with P[t][s][c] = exp(g_{s+1}[c]) ... exp(g_t[c]) (products of the
 * per-token factors, never exponentials of differences),
 *     A[t][s] = beta_t sum_c k_t[c] k_s[c] P[t][s][c]  (s < t),
 *     o_t = sum_c q_t[c] E_t[c] (S0 column) + sum_{s<=t} (sum_c q_t[c] k_s[c] P[t][s][c]) d_s,
 *     S   = diag(E_last) S0 + sum_s (P[last][s] o k_s) d_s^T,
 * E_t[c] = exp(g_0[c]) ... exp(g_t[c]); arguments as kda_decode_varlen
 * (g [Ntok, HV, K], dt_bias [HV * K]) without the state cache.
 */
lar_status gdn_prefill(const lar_tensor* q, const lar_tensor* k, const lar_tensor* v,
                       const lar_tensor* g, const lar_tensor* beta,
                       const lar_tensor* A_log, const lar_tensor* dt_bias,
                       const lar_tensor* pool, const lar_tensor* cu_seqlens,
                       const lar_tensor* read_idx, const lar_tensor* write_idx,
                       const lar_tensor* out, float scale, uint32_t flags, int32_t* dev_err,
                       void* stream);

lar_status kda_prefill(const lar_tensor* q, const lar_tensor* k, const lar_tensor* v,
                       const lar_tensor* g, const lar_tensor* beta,
                       const lar_tensor* A_log, const lar_tensor* dt_bias,
                       const lar_tensor* pool, const lar_tensor* cu_seqlens,
                       const lar_tensor* read_idx, const lar_tensor* write_idx,
                       const lar_tensor* out, float scale, uint32_t flags, int32_t* dev_err,
                       void* stream);

lar_status la_prefill(const lar_tensor* q, const lar_tensor* k, const lar_tensor* v,
                      const lar_tensor* decay, const lar_tensor* pool,
                      const lar_tensor* cu_seqlens, const lar_tensor* read_idx,
                      const lar_tensor* write_idx, const lar_tensor* out, float scale,
                      int32_t* dev_err, void* stream);

/*
 * Short causal convolution over the tokens of a sequence, one filter a channel,
 * as it stands in front of the recurrent layers' q, k and v:
 *     y[t][c] = bias[c] + sum_{j < W} weight[c][j] x[t - (W - 1) + j][c]
 * and out = y, or y / (1 + exp(-y)) with LAR_SILU.  A sequence's state is its last
 * W - 1 inputs; inputs before its first token come from the state it starts from.
 *   x, out   [B, T, C] (rank 2 [B, C] means T = 1), T from 1 to 16; fp32 or bf16,
 *            any strides (out and pool: no two elements at one address).
 *            conv_prefill: packed spans, [Ntok, C], Ntok to 2^30.
 *   weight   [C, W], W from 2 to 4; bias [C] or NULL; fp32 or bf16, any strides.
 *   pool     fp32 or bf16 [P, W - 1, C], channel stride 1, any slot and row
 *            strides: row j of a slot is the input W - 1 - j tokens before the
 *            next one.  Inputs enter the pool rounded to its type.
 *   read_idx, write_idx, num_accepted, state_idx, cu_seqlens   as in gdn_decode,
 *            gdn_decode_tokens and gdn_decode_varlen: negative read slots are a
 *            zero state, negative write slots skip the store, slots >= P and bad
 *            counts or spans are flagged in *dev_err; B and N <= 65535.
 *            conv_prefill with an empty span copies the read state.
 *   C        from 1 to 2^24.
 * Channels that are contiguous, a multiple of 8, with 16-byte aligned rows move in
 * 16-byte accesses; other layouts element by element, with the same results.  Every
 * pointer is aligned to its elements (else LAR_ERR_ALIGN).  conv_prefill and ssm_prefill
 * set their kernel's shared-memory limit (a function attribute) on every call; all calls
 * of this header from here on may be captured into CUDA graphs.
 * Ownership, streams, errors and aliasing as for the decode calls above: pool and
 * out overlap nothing else of the call, entries name distinct write slots and read
 * no slot that another entry writes; an entry may read a slot that it writes.
 */
lar_status conv_decode(const lar_tensor* x, const lar_tensor* weight, const lar_tensor* bias,
                       const lar_tensor* pool, const lar_tensor* read_idx, const lar_tensor* write_idx,
                       const lar_tensor* out, uint32_t flags, int32_t* dev_err, void* stream);

lar_status conv_decode_tokens(const lar_tensor* x, const lar_tensor* weight, const lar_tensor* bias,
                              const lar_tensor* pool, const lar_tensor* read_idx,
                              const lar_tensor* num_accepted, const lar_tensor* state_idx,
                              const lar_tensor* out, uint32_t flags, int32_t* dev_err, void* stream);

lar_status conv_prefill(const lar_tensor* x, const lar_tensor* weight, const lar_tensor* bias,
                        const lar_tensor* pool, const lar_tensor* cu_seqlens, const lar_tensor* read_idx,
                        const lar_tensor* write_idx, const lar_tensor* out, uint32_t flags,
                        int32_t* dev_err, void* stream);

/*
 * Selective state space scan: per channel d a state h of N numbers, with a decay
 * and an input row that every token sets anew.  Per token
 *     s      = softplus(dt[d] + dt_bias[d]) with LAR_DT_SOFTPLUS, else dt[d]
 *     h[n]  <- exp(s A[d][n]) h[n] + s x[d] B[g][n]
 *     y      = sum_n C[g][n] h[n] + D[d] x[d];   out = y z / (1 + exp(-z))
 * without z: out = y; without D (NULL): no skip term.  g = d / (Dch / G), Dch
 * channels in G groups (G divides Dch).
 *   x, dt, z, out   [B, T, Dch] (rank 2 for T = 1), T from 1 to 16; ssm_prefill:
 *            [Ntok, Dch], Ntok to 2^30.  fp32 or bf16, any strides (out: no two elements at one
 *            address); z may be NULL.
 *   A        fp32 [Dch, N], any strides (usually negative, -infinity included: a step
 *            above 0 then forgets); N 16, 32, 64 or 128.
 *   B, C     [B, T, G, N] (rank 3 [B, G, N] for T = 1; packed [Ntok, G, N]), fp32
 *            or bf16, any strides.
 *   D        fp32 [Dch] or NULL.
 *   dt_bias  fp32 [Dch] or NULL; must be NULL without LAR_DT_SOFTPLUS.
 *   pool     fp32 or bf16 [P, Dch, N], state stride 1, 16-byte aligned with slot
 *            and channel strides that are multiples of 16 bytes.  The arithmetic
 *            is fp32; a bf16 state is rounded to nearest even once per store.
 *   read_idx, write_idx, num_accepted, state_idx, cu_seqlens   as for conv_*.
 *   Dch      from 1 to 2^24; ssm_prefill refuses a call of 2^31 blocks or more
 *            (LAR_ERR_SHAPE; a block is at least 4 warps of 64 / (N / 8) channels).
 * Spans that are long beside the others, or few, are computed in parts that are joined
 * (equal up to rounding); how depends on the sizes and span lengths alone, so a call
 * repeated gives the same bits.  In a call of more than 64 spans, unless all their channels
 * fill less than the device, none is split: a prompt of thousands of tokens is then faster in
 * a call without the single tokens.  Fast are x, dt, z, B, C and out of one type with 16-byte
 * aligned rows (Dch / G a multiple of 8); mixed types take 4 to 6 times as long.
 */
lar_status ssm_decode(const lar_tensor* x, const lar_tensor* dt, const lar_tensor* A, const lar_tensor* B,
                      const lar_tensor* C, const lar_tensor* D, const lar_tensor* z,
                      const lar_tensor* dt_bias, const lar_tensor* pool, const lar_tensor* read_idx,
                      const lar_tensor* write_idx, const lar_tensor* out, uint32_t flags,
                      int32_t* dev_err, void* stream);

lar_status ssm_decode_tokens(const lar_tensor* x, const lar_tensor* dt, const lar_tensor* A,
                             const lar_tensor* B, const lar_tensor* C, const lar_tensor* D,
                             const lar_tensor* z, const lar_tensor* dt_bias, const lar_tensor* pool,
                             const lar_tensor* read_idx, const lar_tensor* num_accepted,
                             const lar_tensor* state_idx, const lar_tensor* out, uint32_t flags,
                             int32_t* dev_err, void* stream);

lar_status ssm_prefill(const lar_tensor* x, const lar_tensor* dt, const lar_tensor* A, const lar_tensor* B,
                       const lar_tensor* C, const lar_tensor* D, const lar_tensor* z,
                       const lar_tensor* dt_bias, const lar_tensor* pool, const lar_tensor* cu_seqlens,
                       const lar_tensor* read_idx, const lar_tensor* write_idx, const lar_tensor* out,
                       uint32_t flags, int32_t* dev_err, void* stream);

/*
 * Verification of drafted tokens against the target model's probabilities, from
 * given random numbers.  A step of T tokens holds the last token known and k
 * drafted ones d_0 .. d_{k-1}, drawn from q_0 .. q_{k-1}; p_t is the target's
 * distribution at the place of d_t, p_k the one behind all of them.
 *     d_t is accepted if every draft before it is and u_accept[t] q_t(d_t) < p_t(d_t)
 *     n drafts accepted;  w = max(p_n - q_n, 0) if n < k, p_k if n = k
 *     next token: the first i with w[0] + .. + w[i] > u_sample (w[0] + .. + w[V - 1])
 * An empty residual (w all zero) is replaced by p_n.
 *   draft_tokens  int32/int64 [B, T - 1]; a token outside [0, V) is rejected.
 *   draft_probs   fp32 or bf16 [B, T - 1, V], or NULL: each draft was its model's
 *                 choice (q_t is 1 at d_t, 0 elsewhere).
 *   target_probs  fp32 or bf16 [B, T, V]; T from 1 to 16, V from 1 to 2^24.
 *   u_accept, u_sample   fp32 [B, T - 1], [B], in [0, 1).
 *   num_draft     int32/int64 [B] or NULL: k of each sequence, 0 to T - 1 (NULL:
 *                 T - 1); drafts behind it are not looked at.
 *   num_accepted  out, int32 or int64 [B]: n + 1, the tokens of the step that stand
 *                 (what *_decode_tokens take as num_accepted in the next step).
 *   tokens        out, int32 or int64 [B, T]: the accepted drafts, the next token,
 *                 then -1.
 * Any strides.  A weight that is not a positive finite number counts as 0; sums are
 * held to about 2^-48 of their value (weights up to 2^64, whole sums of 2^-100 or more), so
 * that the index is the one that exact sums give.  Acceptance is by the exact product.
 */
lar_status spec_verify(const lar_tensor* draft_tokens, const lar_tensor* draft_probs,
                       const lar_tensor* target_probs, const lar_tensor* u_accept,
                       const lar_tensor* u_sample, const lar_tensor* num_draft,
                       const lar_tensor* num_accepted, const lar_tensor* tokens, int32_t* dev_err,
                       void* stream);

/*
 * A paged cache of keys and values, as the softmax-attention layers between the recurrent
 * ones keep it.  What the two calls below share:
 *   k_cache, v_cache   [P, page, H, D]: P pages of `page` tokens (a multiple of 16, to
 *            1024), H heads (to 1024), D 64, 128 or 256.  bf16 or e4m3, both of one type.
 *            Dimension stride 1, 16-byte aligned, all other strides multiples of 16
 *            bytes: views of [P, H, page, D] or of one buffer with both halves will do.
 *   k_scale, v_scale   fp32 [P, H], any strides, with e4m3 pages; NULL with bf16 ones.  A
 *            value is its code times the scale of its page and head.
 *   block_table   int32/int64 [B, M]: place t of sequence b is token t % page of page
 *            block_table[b][t / page]; M page to 2^30.  A negative entry is no page (not
 *            written, not seen), one >= P neither, and flagged (LAR_DEVERR_PAGE).
 *   seq_lens int32/int64 [B]: tokens that sequence b has BEFORE the step: the step's token t
 *            is at place seq_lens[b] + t, in both calls.  Negative: no sequence here.
 *            Places from M page on are not written, not seen, and flagged
 *            (LAR_DEVERR_SEQLEN; queries are rotated there too, past 2^30 as at 2^30).
 *
 * kv_append: the keys and values of a step's (or a prompt's) tokens enter the cache, the
 * keys rotated by their place; with q, the queries are rotated into q_out.
 *   k, v     [B, T, H, D] (rank 3 for T = 1), T from 1 to 16; with cu_seqlens (int32/int64
 *            [B + 1], ascending) packed spans, [Ntok, H, D], Ntok to 2^30.  fp32 or bf16,
 *            any strides.
 *   q, q_out [.., Hq, D] or both NULL; H divides Hq, to 65535; fp32 or bf16, any strides
 *            (q_out: no two elements at one address).  Rows of tokens outside every span,
 *            or of no sequence, are left as they were.
 *   inv_freq fp32 [rot / 2], rot to D: pair i of dimensions (x, y) of a token at place t
 *            becomes rope_scale (x cos a - y sin a, y cos a + x sin a), a = t inv_freq[i]
 *            (its whole turns are dropped before it is rounded, so far places are as exact
 *            as near ones; frequencies to 2^60).  Dimensions from rot on are copied.  NULL:
 *            no rotation (then no flags, rope_scale 1).
 * e4m3: the scale is a power of two, 2^-64 to 2^64: the least with |x| <= 448 scale for the
 * values that enter a (page, head) in this call, and no less than that of the tokens that
 * stand before them in the page; if those have a smaller one, their codes are rounded to the
 * new one (exact unless a code falls below the least normal one).  A code is value / scale
 * rounded to nearest even (a rotated key from fp32: next to a tie, to either neighbour);
 * magnitudes past 448 2^64 are held there.  What is not finite (in fp32, once it is rotated)
 * becomes a NaN and has no say in the scale.
 * Tokens behind the appended ones in a page count as not there.
 * Aliasing: caches and scales are in and out; they and q_out overlap nothing else of the call
 * (keys' and values' views may lie between one another).  No page is named by two sequences,
 * or twice, where tokens are appended; pages in front of those are not touched, and may be
 * shared.  Fastest are bf16 rows that 16-byte loads fit and, for prompts, pages of 4096 angles or
 * fewer (tokens times rot / 2): prompts take 1.4 times as long in larger ones, and fp32 rows
 * twice.  Offsets that do not ascend are flagged (LAR_DEVERR_SEQLEN; with no tokens at all nothing
 * is looked at); which of the spans around them are taken is not defined.
 */
lar_status kv_append(const lar_tensor* q, const lar_tensor* k, const lar_tensor* v, const lar_tensor* q_out,
                     const lar_tensor* k_cache, const lar_tensor* v_cache, const lar_tensor* k_scale,
                     const lar_tensor* v_scale, const lar_tensor* block_table, const lar_tensor* seq_lens,
                     const lar_tensor* cu_seqlens, const lar_tensor* inv_freq, float rope_scale, uint32_t flags,
                     int32_t* dev_err, void* stream);

/*
 * attn_decode: attention of a step's tokens over the cache, after kv_append of the same
 * step (the same seq_lens).  Token t of sequence b sees the places 0 .. seq_lens[b] + t, or,
 * with window > 0, the last `window` of them:
 *     out = sum_j softmax_j(scale q K_j) V_j,   lse = log sum_j exp(scale q K_j)
 *   q, out   [B, T, Hq, D] (rank 3 for T = 1), T from 1 to 16, H divides Hq, Hq / H to 256;
 *            q bf16, out bf16 or fp32, any strides (out: no two elements at one address).
 *            Query head i reads key/value head i / (Hq / H).
 *   lse      fp32 [B, T, Hq] or NULL.  A row that sees nothing has out 0 and lse -infinity.
 *   workspace   fp32, contiguous, 16-byte aligned, of attn_workspace(T, Hq, H, D) elements
 *            or more (-1: the call does not take such sizes); what it holds need not be kept
 *            between calls, and calls that may run at the same time need one each.
 * What stands at places that a row does not see has no say in it, whatever it is.  Scores,
 * maxima and sums are fp32.  The weights of the second product are rounded to 11 bits with e4m3
 * pages (fp16; below 2^-21 of the greatest, each times its values' scale, to 2^-32 of that), to 16
 * bits with bf16 pages.  16-bit values may be as large as their type goes: where a sum passes
 * 2^115 it is taken once more (in about twice the time), with weights 2^-60 of what they were,
 * and values below 2^-66 beside such ones may count as 0.  How the work is split depends on the
 * lengths and sizes alone, so a repeated call gives the same bits.  Scales are positive normal numbers,
 * those of one sequence's values within 2^100 of one another.
 * The pages of a key/value head are walked once for every 32 of its T Hq / H rows (16 at D = 256).
 * Two kernels on `stream`.
 */
int64_t attn_workspace(int32_t T, int32_t Hq, int32_t H, int32_t D);

lar_status attn_decode(const lar_tensor* q, const lar_tensor* k_cache, const lar_tensor* v_cache,
                       const lar_tensor* k_scale, const lar_tensor* v_scale, const lar_tensor* block_table,
                       const lar_tensor* seq_lens, const lar_tensor* out, const lar_tensor* lse,
                       const lar_tensor* workspace, float scale, int32_t window, int32_t* dev_err, void* stream);

/*
 * The draw of tokens from logits and given random numbers, one a row:
 *     w[i] = exp((x[i] - max x) / temperature)
 * Of the tokens in falling order of x (equal ones by index) the first ones are kept: top_k of
 * them, those with w >= min_p, and, measured on what top_k leaves, the fewest whose weights
 * sum to top_p of the whole or more; the shortest of the three, one at least.
 *     token: the first i (by index) with  sum_{kept j <= i} w[j] > u sum_{kept j} w[j]
 *     probs[i] = w[i] / sum_{kept j} w[j], or 0: what spec_verify takes as draft_probs and
 *     target_probs
 *   logits   fp32 or bf16 [B, T, V] (rank 2 [B, V] for T = 1), T from 1 to 16, V from 1 to
 *            2^24.  NaN counts as -infinity; if the greatest is +infinity, the tokens that
 *            have it weigh 1 and the others nothing.
 *   u        fp32 [B, T] (rank 1 for T = 1), in [0, 1).
 *   temperature   fp32 [B] or NULL (1); 0 or less (or NaN) means the greatest logit alone.
 *   top_k    int32/int64 [B] or NULL; 0 or less: all.
 *   top_p    fp32 [B] or NULL; 1 or more: all; 0 or less (or NaN): the first.
 *   min_p    fp32 [B] or NULL; 0 or less (or NaN): all.
 *   tokens   out, int32 or int64 [B, T] (rank 1 for T = 1).
 *   probs    out, fp32 [B, T, V] (rank 2) or NULL.
 * Any strides (outputs: no two elements at one address; rows whose logits lie side by side are
 * read in half the time).  Weights are held to 2^-30 of themselves (temperatures from 2^-100 on)
 * or V 2^-62 of the greatest, sums exactly: the token is the one that exact arithmetic gives
 * unless u or a threshold is as near as that to a border.  Fastest are top_k up to a thousand or
 * so, and temperatures alone; top_p without top_k takes about twice as long, and rows of few
 * different logits several times.
 */
lar_status sample_tokens(const lar_tensor* logits, const lar_tensor* u, const lar_tensor* temperature,
                         const lar_tensor* top_k, const lar_tensor* top_p, const lar_tensor* min_p,
                         const lar_tensor* tokens, const lar_tensor* probs, int32_t* dev_err, void* stream);

/* Static, human-readable name of a status code. */
const char* lar_status_string(lar_status status);

#ifdef __cplusplus
}
#endif

#endif /* LAR_H_ */
