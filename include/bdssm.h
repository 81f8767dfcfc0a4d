/*
 * bdssm.h - C ABI of the bidirectional block-diffusion Mamba state hot path on MI355X.
 *
 * The method ("Training Hybrid Block Diffusion Language Models with Partial
 * Bidirectionality", eqs. (9)-(13) and the cache discussion around them) factors each
 * Mamba layer into a timestep-free prefix operator, which folds the clean prefix into a
 * cached forward state, and an active-block continuation, which runs a forward scan
 * seeded from that state plus a reverse scan confined to the active block. The three
 * calls below are those three operations:
 *
 *   bdssm_prefix_scan  - eq. (10): s_k = F_fwd(c), the forward scan of a prefix,
 *                        returning the boundary state (and optionally y and the state
 *                        after every chunk of the scan).
 *   bdssm_block_step   - eqs. (11)-(13): y = F_fwd(b; s_k) + rev(F_rev(rev(b))) + D x,
 *                        for one denoising step of the active block. The cached state is
 *                        read, never written (the cache must not depend on the step).
 *   bdssm_commit       - the clean forward pass over a finalized block that extends the
 *                        cache: s_{k+1} = F_fwd(b*; s_k), in place.
 *
 * bdssm_decode_graph_* record the calls of one active block (its denoising steps, then its
 * commit) once into a HIP graph and replay it, removing per-call launch latency from a
 * decode loop with static shapes.
 *
 * The scan F is the selective state-space recurrence of eq. (1) in its Mamba-2 form,
 * with one negative scalar A[h] per head:
 *     alpha_t = exp(dt[t,h] * A[h])
 *     S_t     = alpha_t * S_{t-1} + dt[t,h] * B[t,g] x[t,h]^T        (S is N x P)
 *     y[t,h]  = C[t,g] . S_t   (+ D[h] * x[t,h] where stated)
 * with g = h / (H/G): each group of H/G consecutive heads shares B and C. The reverse
 * scan starts from a zero state at the block's right end and runs t = T-1 ... 0 over
 * inputs given in natural token order; its outputs are in natural order too.
 *
 * Layouts (row-major, contiguous, b = stream):
 *     x  [b][len][H][P]     dt [b][len][H]     B, C [b][len][G][N]
 *     state [b][H][N][P] (float32)     chunk states [b][ceil(len/chunk)][H][N][P]
 *     y  [b][len][H][P]     A, D [H] (float32)
 * dt is the final step size (already passed through softplus and any clamp).
 *
 * Conventions for every call:
 *  - Pointers are device pointers (hipMalloc'd, or torch CUDA tensors); the caller owns
 *    every buffer. Base pointers must be 16-byte aligned. The library allocates nothing
 *    (except the graph object of bdssm_decode_graph_create) and never synchronizes.
 *  - `stream` is a hipStream_t (NULL = the default stream). Work is enqueued
 *    asynchronously; the returned status covers argument validation and the launch.
 *    Faults during execution surface at the caller's next synchronization.
 *  - Errors are status codes; nothing is thrown across the ABI. Invalid arguments are
 *    rejected before anything is launched, with no buffer modified.
 *  - Supported shapes: ngroups divides nheads; (d_state, headdim) in {(16,16), (128,64)};
 *    chunk in {16, 32, 64, 128, 256}; block_len in [0, 256]. batch, len and block_len
 *    may be 0 (nothing to do: a prefix scan of zero tokens returns h_init, or zero).
 *  - Thread-safe and re-entrant. Calls on one stream run in order.
 */
#ifndef BDSSM_H
#define BDSSM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define BDSSM_ABI_VERSION 4

typedef enum {
    BDSSM_OK = 0,
    BDSSM_ERR_NULL = 1,        /* a required pointer is NULL */
    BDSSM_ERR_SHAPE = 2,       /* a size is negative or inconsistent (e.g. H % G != 0) */
    BDSSM_ERR_UNSUPPORTED = 3, /* a valid size or dtype with no compiled kernel */
    BDSSM_ERR_ALIGN = 4,       /* a base pointer is not 16-byte aligned */
    BDSSM_ERR_ALIAS = 5,       /* an output overlaps an input it must not overlap */
    BDSSM_ERR_WORKSPACE = 6,   /* workspace missing or smaller than the query returned */
    BDSSM_ERR_HIP = 7,         /* the HIP runtime reported an error at launch */
    BDSSM_ERR_SCRATCH = 8      /* bdssm_prefix_scan_static: more workspace needed than the
                                  static scratch buffer holds */
} bdssm_status;

typedef enum { BDSSM_F32 = 0, BDSSM_BF16 = 1 } bdssm_dtype;

typedef struct {
    int32_t batch;    /* independent streams b */
    int32_t nheads;   /* H */
    int32_t headdim;  /* P */
    int32_t d_state;  /* N */
    int32_t ngroups;  /* G */
    int32_t in_dtype; /* bdssm_dtype of x, dt, B, C */
    int32_t y_dtype;  /* bdssm_dtype of y (F32 for parity checks, BF16 as activations) */
} bdssm_dims;

/* One token segment's inputs (device pointers, layouts above). */
typedef struct {
    const void *x, *dt, *B, *C;
} bdssm_seq;

/* ABI version implemented by the library (BDSSM_ABI_VERSION at build time). */
int bdssm_abi_version(void);

/* Static, human-readable name of a status code; never NULL. */
const char *bdssm_status_str(int status);

/* Bytes of device workspace bdssm_prefix_scan needs for these arguments. with_y and
 * with_chunk_states say whether y and chunk_states will be passed non-NULL. Returns 0
 * when no workspace is needed, and SIZE_MAX for arguments bdssm_prefix_scan would
 * reject. */
size_t bdssm_prefix_scan_workspace(const bdssm_dims *dims, int64_t len, int32_t chunk,
                                   int32_t with_y, int32_t with_chunk_states);

/*
 * Prefix scan: eq. (10), s_k = F_fwd(c^(k)), the forward recurrence over `len` prefix
 * tokens of every stream, computed chunk by chunk (chunk = Q tokens; the last chunk may
 * be shorter).
 *   in            prefix inputs, len tokens
 *   A, D          [H] float32
 *   h_init        [b][H][N][P] float32 starting state, or NULL for zero
 *   y             [b][len][H][P] in dims->y_dtype, y_t = C_t . S_t + D x_t; NULL = state only
 *   chunk_states  [b][ceil(len/Q)][H][N][P] float32: the state after tokens Q-1, 2Q-1, ...
 *                 and after the last token (so the last entry equals h_out); NULL = none
 *   h_out         [b][H][N][P] float32 final state; required; may be the same pointer as
 *                 h_init (updated in place) but must not otherwise overlap anything
 *   workspace     device buffer of at least bdssm_prefix_scan_workspace(...) bytes
 * y and chunk_states must not overlap any input or each other.
 */
bdssm_status bdssm_prefix_scan(const bdssm_dims *dims, int64_t len, int32_t chunk,
                               const bdssm_seq *in, const float *A, const float *D,
                               const float *h_init, void *y, float *chunk_states,
                               float *h_out, void *workspace, size_t workspace_bytes,
                               void *stream);

/*
 * Prefix scan that allocates nothing and takes no workspace, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid allocation): bdssm_prefix_scan, bitwise, with the workspace it would need taken
 * from a scratch buffer the library keeps in device memory -- a static array of
 * BDSSM_STATIC_SCRATCH_BYTES (64 MiB) per GPU, held from the library's first use of that
 * GPU until the process ends. Every call on one GPU shares that GPU's buffer and it keeps
 * the last call's contents (each call writes all it reads), so calls that overlap in time
 * on one GPU -- on different streams, or from different threads -- race and give wrong
 * results; calls in order on one stream are safe. On the matrix-core path (bf16 inputs,
 * (d_state, headdim) = (128, 64), chunk >= 64) the largest plan needs about 32 MiB on a
 * 256-CU MI355X, whatever the sizes; other paths need bdssm_prefix_scan_workspace bytes.
 * Arguments, layouts, ownership and errors as bdssm_prefix_scan, plus:
 *   BDSSM_ERR_SCRATCH  the call would need more than BDSSM_STATIC_SCRATCH_BYTES of workspace
 *                      (rejected before anything is launched)
 *   BDSSM_ERR_HIP      the buffer's device address could not be obtained
 */
#define BDSSM_STATIC_SCRATCH_BYTES ((size_t)64 << 20)
bdssm_status bdssm_prefix_scan_static(const bdssm_dims *dims, int64_t len, int32_t chunk,
                                      const bdssm_seq *in, const float *A, const float *D,
                                      const float *h_init, void *y, float *chunk_states,
                                      float *h_out, void *stream);

/*
 * Block step: eqs. (11)-(13), one denoising step of the active block of T = block_len
 * tokens:
 *   y_t = C_t . S_t            (forward scan from h_prefix over fwd, eq. 11)
 *       + C'_t . R_t           (reverse scan over rev from R_T = 0, eq. 12)
 *       + D[h] * x_fwd[t]      (skip term of eq. 1, applied once)
 *   h_prefix  [b][H][N][P] float32 cached state; read only, never written
 *   fwd, rev  the two directions' inputs, T tokens each, natural token order
 *   y         [b][T][H][P] in dims->y_dtype; must not overlap any input
 */
bdssm_status bdssm_block_step(const bdssm_dims *dims, int32_t block_len,
                              const float *h_prefix, const bdssm_seq *fwd,
                              const bdssm_seq *rev, const float *A, const float *D, void *y,
                              void *stream);

/*
 * Block step with separate parameters for the reverse direction (eq. (12) gives the
 * reverse scan its own parameters): the reverse recurrence decays with A_rev[h] instead of
 * A[h], and each direction keeps its own skip term,
 *   y_t = C_t . S_t + C'_t . R_t + D[h] * x_fwd[t] + D_rev[h] * x_rev[t].
 *   A_rev  [H] float32, required (pass A for a shared decay)
 *   D_rev  [H] float32, or NULL for no reverse skip term
 * Everything else as bdssm_block_step, which equals this call with A_rev = A, D_rev = NULL.
 * y must not overlap A_rev or D_rev either.
 */
bdssm_status bdssm_block_step_ex(const bdssm_dims *dims, int32_t block_len,
                                 const float *h_prefix, const bdssm_seq *fwd,
                                 const bdssm_seq *rev, const float *A, const float *D,
                                 const float *A_rev, const float *D_rev, void *y, void *stream);

/*
 * Full-window bidirectional scan: the system the block-local method is compared against, a
 * fully bidirectional Mamba layer over the whole sequence ("DiffuApriel", Sec. 3.2, eqs.
 * (4)-(6): a forward and a backward scan, each with its own parameters, summed; the
 * full-sequence bidirectional baselines of "Training Hybrid Block Diffusion Language Models
 * with Partial Bidirectionality", whose directionality discussion explains why their reverse
 * states cannot be cached). Over one window of len tokens -- the prefix and the active block
 * together -- with nothing cached:
 *   y_t = C_t . S_t             (forward scan from a zero state at token 0, over fwd)
 *       + C'_t . R_t            (reverse scan from a zero state past token len-1, over rev,
 *                                decaying with A_rev)
 *       + D[h] * x_fwd[t] (+ D_rev[h] * x_rev[t] when D_rev is given)
 * for every token of the window. Since the reverse states of prefix tokens depend on the
 * active block, a full-window model recomputes all of this on every denoising step; on the
 * block's own tokens the result equals bdssm_block_step from the prefix's state.
 *   fwd, rev        the two directions' inputs, len tokens each, natural token order
 *   A, D            [H] float32; A_rev [H] float32, required (pass A for a shared decay);
 *                   D_rev [H] float32 or NULL
 *   y               [b][len][H][P] in dims->y_dtype, written (forward half) then added to
 *                   (reverse half, so bf16 y is rounded twice); must not overlap any input
 *   chunk, workspace  as in bdssm_prefix_scan (bdssm_full_window_workspace bytes; both
 *                   directions use the same workspace in turn)
 * Errors as bdssm_prefix_scan.
 */
size_t bdssm_full_window_workspace(const bdssm_dims *dims, int64_t len, int32_t chunk);
bdssm_status bdssm_full_window(const bdssm_dims *dims, int64_t len, int32_t chunk, const bdssm_seq *fwd,
                               const bdssm_seq *rev, const float *A, const float *D, const float *A_rev,
                               const float *D_rev, void *y, void *workspace, size_t workspace_bytes,
                               void *stream);

/*
 * Commit: the clean forward pass over a finalized block of T = block_len tokens that
 * extends the cache, S <- F_fwd(clean; S), in place on h.
 *   clean  the block's clean inputs; clean->C may be NULL when y is NULL
 *   h      [b][H][N][P] float32, read then overwritten with the advanced state
 *   y      NULL, or [b][T][H][P] in dims->y_dtype: y_t = C_t . S_t + D x_t of the pass
 */
bdssm_status bdssm_commit(const bdssm_dims *dims, int32_t block_len, const bdssm_seq *clean,
                          const float *A, const float *D, float *h, void *y, void *stream);

/*
 * Cached state in operand form. The cached state is read by every denoising step of a
 * block and changes only when a block is committed (eqs. (9)-(11): s_k is fixed while
 * block k is denoised), so the re-encoding the block step's matrix-core product needs can
 * be made once per cached state instead of once per step. The operand form of a float32
 * state S is the bf16 pair hi = bf16(S), lo = bf16(S - hi) (round to nearest even; together
 * about 16 significant bits, the same pair bdssm_block_step forms from S on every call), laid
 * out as
 *     ops [b][H][2 (hi, lo)][N/8][P][8] bf16,  ops[..][k][n/8][p][n%8] = k-part of S[n][p],
 * which has the size of the float32 state. Supported for (d_state, headdim) = (128, 64).
 *
 * bdssm_state_ops_bytes: bytes of ops for these dims; SIZE_MAX for invalid or unsupported
 * dims.
 * bdssm_state_ops: writes ops from h [b][H][N][P] float32 (read only); ops must not overlap
 * h. Errors: BDSSM_ERR_NULL, BDSSM_ERR_UNSUPPORTED (other d_state/headdim), BDSSM_ERR_ALIGN,
 * BDSSM_ERR_ALIAS.
 */
size_t bdssm_state_ops_bytes(const bdssm_dims *dims);
bdssm_status bdssm_state_ops(const bdssm_dims *dims, const float *h, void *ops, void *stream);

/*
 * Block step from the cached state in operand form: bdssm_block_step_ex with the state
 * given as h_ops, made by bdssm_state_ops from h_prefix. For block_len <= 32 and
 * batch * nheads < 512 it runs the small-batch kernel of bdssm_block_step_ex and its y is
 * bitwise that call's on h_prefix; otherwise (block_len <= 128) a kernel that copies the
 * operand-form state and x straight into LDS, whose y agrees with bdssm_block_step_ex up to
 * rounding (the same bounds against the exact result). Errors as bdssm_block_step_ex, with
 * BDSSM_ERR_UNSUPPORTED for inputs other than bf16, (d_state, headdim) other than
 * (128, 64), or block_len > 128; y must not overlap h_ops.
 */
bdssm_status bdssm_block_step_ops(const bdssm_dims *dims, int32_t block_len, const void *h_ops,
                                  const bdssm_seq *fwd, const bdssm_seq *rev, const float *A,
                                  const float *D, const float *A_rev, const float *D_rev, void *y,
                                  void *stream);

/*
 * bf16 cached state. The block step reads the whole cached state on every denoising step,
 * so its bytes bound the step at large batch; a bf16 copy halves them at the cost of
 * rounding the state once (relative error 2^-9 per element). The bf16 state of a float32
 * state S is bf16(S), rounded to nearest even -- the operand form's hi part -- laid out as
 *     [b][H][N/8][P][8] bf16,  element (n, p) of a head at index (n/8 * P + p) * 8 + n % 8,
 * made once per cached state (after the prefix scan or a commit, which keep the float32
 * state as the master copy). Supported for d_state a multiple of 8.
 * bdssm_state_bf16_bytes: bytes of the bf16 state; SIZE_MAX for invalid or unsupported dims.
 * bdssm_state_bf16: writes it from h [b][H][N][P] float32 (read only); out must not overlap
 * h. Errors: BDSSM_ERR_NULL, BDSSM_ERR_UNSUPPORTED, BDSSM_ERR_ALIGN, BDSSM_ERR_ALIAS.
 */
size_t bdssm_state_bf16_bytes(const bdssm_dims *dims);
bdssm_status bdssm_state_bf16(const bdssm_dims *dims, const float *h, void *out, void *stream);

/*
 * Block step with every variant of the layer's parameters and of the cached state's form.
 * The reverse scan of eq. (12) has its own parameters (theta_rev): its decay A_rev and its
 * own skip weight D_rev; the skip weights may also be one per channel of x ([H][P], the
 * Mamba-2 layer's per-channel option) instead of one per head:
 *   y_t = C_t . S_t + C'_t . R_t + D (.) x_fwd[t] (+ D_rev (.) x_rev[t])
 * with (.) the per-head scalar or the per-channel product.
 *   state       the cached state in the form state_form:
 *                 BDSSM_STATE_F32   float32 [b][H][N][P] (as bdssm_block_step)
 *                 BDSSM_STATE_OPS   operand form (bdssm_state_ops; bf16 inputs, (d_state,
 *                                   headdim) = (128, 64), block_len <= 128 only)
 *                 BDSSM_STATE_BF16  bf16 state (bdssm_state_bf16)
 *               read only, never written
 *   params      A [H] required; D [H] (or [H][P]) required; A_rev [H] or NULL (= A);
 *               D_rev [H] (or [H][P]) or NULL (none); skip_per_channel 0 or 1
 * With the float32 state and per-head weights this is bdssm_block_step_ex, bitwise; with
 * the operand form, bdssm_block_step_ops. Errors as bdssm_block_step_ex, plus
 * BDSSM_ERR_UNSUPPORTED for an unknown state form or skip layout, or the operand form outside
 * its shapes. y must not overlap the state or any parameter.
 */
enum { BDSSM_STATE_F32 = 0, BDSSM_STATE_OPS = 1, BDSSM_STATE_BF16 = 2 };
typedef struct {
    const float *A, *D, *A_rev, *D_rev;
    int32_t skip_per_channel;
} bdssm_step_params;
bdssm_status bdssm_block_step_variant(const bdssm_dims *dims, int32_t block_len, const void *state,
                                      int32_t state_form, const bdssm_seq *fwd, const bdssm_seq *rev,
                                      const bdssm_step_params *params, void *y, void *stream);

/*
 * Commit with the block step's copy of the state refreshed in the same pass: bdssm_commit,
 * then state_copy <- the advanced state in the form state_form (BDSSM_STATE_OPS: the operand
 * form of bdssm_state_ops; BDSSM_STATE_BF16: the bf16 state of bdssm_state_bf16), bitwise
 * those calls' results. The cached state changes only at a commit (eqs. (9)-(11)), so this
 * is the one place a decode loop needs to re-encode it; with bf16 inputs, (d_state,
 * headdim) = (128, 64) and y == NULL one launch does both (the state walk writes both from
 * its registers), else a commit and an encoding launch.
 *   state_copy  [b][H][2][N/8][P][8] or [b][H][N/8][P][8] bf16; must not overlap h, y or
 *               any input
 * With block_len = 0 the state is unchanged and only the copy is written. Errors as
 * bdssm_commit, plus BDSSM_ERR_UNSUPPORTED for a state form other than those two, or the
 * operand form outside its shape.
 */
bdssm_status bdssm_commit_refresh(const bdssm_dims *dims, int32_t block_len, const bdssm_seq *clean,
                                  const float *A, const float *D, float *h, void *state_copy,
                                  int32_t state_form, void *y, void *stream);

/*
 * Convolution state. A Mamba layer's cache holds convolution state as well as the SSM
 * state (the cache discussion of "Training Hybrid Block Diffusion Language Models with
 * Partial Bidirectionality"); the pages leave the convolution itself open, and these calls
 * take the Mamba-2 layer's: before the scan, each of the CH = H*P + 2*G*N channels of a
 * token (x [H][P], then B [G][N], then C [G][N]) is convolved with its own `width` taps,
 * a bias is added and an activation applied, and the result, rounded to the input dtype,
 * is what the scan reads. dt is not convolved.
 *   forward (causal):   out_t = bias + sum_{k<W} w[k] u_{t-(W-1)+k}, where u_t for t < 0
 *                       comes from the conv state, the W-1 raw (unconvolved) rows that
 *                       precede the segment;
 *   reverse (anti-causal, the block's reverse branch, which has no state, eq. (12)):
 *                       out_t = bias + sum_{k<W} w[k] u_{t+(W-1)-k}, with u_t = 0 past the
 *                       segment's end (the causal convolution of the reversed block).
 * The conv state after a forward segment is the last W-1 rows of the raw input extended by
 * the previous state. Conv state layout: [b][W-1][CH] in dims->in_dtype.
 */
typedef struct {
    int32_t width;       /* W, 1..4 */
    int32_t activation;  /* 0 identity, 1 SiLU (v / (1 + exp(-v))) */
    const float *weight; /* [CH][W] float32, taps w[c][k] */
    const float *bias;   /* [CH] float32, or NULL for none */
} bdssm_conv_params;

/* Bytes of one convolved copy of x, B and C for `len` tokens (each part 256-byte aligned in
 * the buffer): bdssm_block_step_conv needs two, bdssm_commit_conv one. SIZE_MAX for
 * invalid dims or len < 0. */
size_t bdssm_conv_workspace(const bdssm_dims *dims, int64_t len);

/*
 * The convolution of one segment of `len` tokens: out.{x,B,C} <- act(conv(raw.{x,B,C})).
 *   reverse    0 forward (causal), 1 reverse (anti-causal)
 *   state_in   forward: [b][W-1][CH] history before the segment, or NULL for zeros (the
 *              start of a sequence); must be NULL when reverse
 *   raw, out   x, B, C are used (dt is ignored and may be NULL); out must not overlap raw,
 *              the parameters or the states
 *   state_out  forward: [b][W-1][CH] receives the new history, or NULL; it may be the same
 *              pointer as state_in (updated in place) but must not otherwise overlap
 *              anything; must be NULL when reverse
 * A prefix is convolved with this call (forward, state_in NULL, state_out = the cache's
 * conv state) before bdssm_prefix_scan reads it.
 */
bdssm_status bdssm_conv(const bdssm_dims *dims, int64_t len, const bdssm_conv_params *conv,
                        int32_t reverse, const void *state_in, const bdssm_seq *raw,
                        const bdssm_seq *out, void *state_out, void *stream);

/*
 * Block step on unconvolved inputs: the forward branch's x, B, C are convolved causally from
 * the cached conv state (conv_fwd), the reverse branch's anti-causally inside the block
 * (conv_rev, its own parameters; pass conv_fwd's for shared ones), both in one launch into
 * the workspace, then bdssm_block_step_ex runs on the convolved inputs with the raw dt.
 *   conv_state  [b][W_fwd-1][CH] in in_dtype, read only (NULL when W_fwd = 1)
 *   A_rev       as in bdssm_block_step_ex; NULL means A
 *   workspace   at least 2 * bdssm_conv_workspace(dims, block_len) bytes; must not overlap
 *               anything else
 * Everything else as bdssm_block_step_ex.
 */
bdssm_status bdssm_block_step_conv(const bdssm_dims *dims, int32_t block_len,
                                   const bdssm_conv_params *conv_fwd,
                                   const bdssm_conv_params *conv_rev, const float *h_prefix,
                                   const void *conv_state, const bdssm_seq *fwd,
                                   const bdssm_seq *rev, const float *A, const float *D,
                                   const float *A_rev, const float *D_rev, void *y,
                                   void *workspace, size_t workspace_bytes, void *stream);

/*
 * Commit on unconvolved inputs: the clean block is convolved causally from the conv state
 * into the workspace, the conv state is advanced in place, then bdssm_commit advances h.
 *   conv_state  [b][W-1][CH] in in_dtype, read then overwritten (NULL when W = 1)
 *   workspace   at least bdssm_conv_workspace(dims, block_len) bytes
 * Everything else as bdssm_commit, except that clean->C is always required (its raw rows
 * enter the conv state).
 */
bdssm_status bdssm_commit_conv(const bdssm_dims *dims, int32_t block_len,
                               const bdssm_conv_params *conv, const bdssm_seq *clean,
                               const float *A, const float *D, float *h, void *conv_state,
                               void *y, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Decode loop of one active block as a HIP graph: `steps` calls of bdssm_block_step (step
 * k reads fwd[k], rev[k] and writes y[k], all from the cached state h), followed, when
 * clean is not NULL, by bdssm_commit(clean, h, y_commit). This is the static-shape block
 * buffer of block-diffusion decoding, whose inputs change from step to step in place.
 *   fwd, rev   host arrays of `steps` input descriptors (device pointers)
 *   y          host array of `steps` device output pointers, [b][T][H][P] in y_dtype
 *   h          [b][H][N][P] float32: read by every step, then advanced by the commit
 *   h_ops      NULL, or the cached state in operand form (bdssm_state_ops of h, made by the
 *              caller before the first replay): the steps then read it (bdssm_block_step_ops)
 *              and the commit is followed by bdssm_state_ops(h -> h_ops), so that it holds
 *              the advanced state for the next replay
 *   clean      the commit's inputs, or NULL for steps only; y_commit as in bdssm_commit
 *   stream     the stream the calls are recorded on; must not be NULL (the legacy default
 *              stream cannot be captured). Nothing runs during creation.
 *   out        receives the graph; NULL on error
 * Every call is validated as bdssm_block_step / bdssm_commit validate it; the first
 * failing status is returned and no graph is made. The device pointers are baked into
 * the graph: the buffers must stay allocated, at the same addresses, while it exists.
 * Errors: BDSSM_ERR_NULL (dims, out, fwd, rev, y or stream NULL; steps < 1 with no commit),
 * BDSSM_ERR_SHAPE (steps < 0), the statuses of the recorded calls, BDSSM_ERR_HIP
 * (capture or instantiation failed).
 */
typedef struct bdssm_decode_graph bdssm_decode_graph;
bdssm_status bdssm_decode_graph_create(const bdssm_dims *dims, int32_t block_len, int32_t steps,
                                       float *h, void *h_ops, const bdssm_seq *fwd,
                                       const bdssm_seq *rev,
                                       const float *A, const float *D, void *const *y,
                                       const bdssm_seq *clean, void *y_commit, void *stream,
                                       bdssm_decode_graph **out);

/* Enqueues one replay of the recorded calls on `stream` (NULL = default stream). Runs
 * asynchronously, like the calls it replaces; allocates nothing. */
bdssm_status bdssm_decode_graph_launch(const bdssm_decode_graph *graph, void *stream);

/* Frees the graph (NULL is ignored). Replays already enqueued are not affected. */
void bdssm_decode_graph_destroy(bdssm_decode_graph *graph);

/*
 * The norms around a layer of the hybrid, fused with the layer's gate and with the residual
 * update. Both calls read a row once and write each output once; sums are float32.
 *   norm(v) = v / sqrt(mean(v^2) + eps)                        (BDSSM_NORM_RMS)
 *   norm(v) = (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps)  (BDSSM_NORM_LAYER)
 * Rows are tokens, [rows][width] row-major. Unlike the scan's tensors, every pointer of these
 * two calls needs its element's alignment only, and width may be any number of channels (at
 * most 16384 normalized together).
 */
enum { BDSSM_NORM_RMS = 0, BDSSM_NORM_LAYER = 1 };
typedef struct {
    int64_t rows;            /* tokens of all streams; may be 0 */
    int32_t width;           /* channels of a row */
    int32_t groups;          /* channel groups normalized apart, dividing width (gated norm);
                                1 for bdssm_residual_norm */
    int32_t rows_per_stream; /* tokens of a stream, for gate, gain and shift (else ignored) */
    int32_t kind;            /* BDSSM_NORM_RMS, BDSSM_NORM_LAYER (residual norm only) */
    int32_t x_dtype;         /* bdssm_dtype of y / of x and x_out; F32 or the same as dtype */
    int32_t dtype;           /* bdssm_dtype of z and out / of o, u, gate, gain and shift */
    float eps;               /* > 0 */
} bdssm_norm_dims;

/*
 * The norm after a scan with the layer's gate z (a Mamba-2 layer's output norm, before its
 * output projection), over channel groups of width / groups:
 *   norm_first = 0   out = norm(y silu(z)) weight
 *   norm_first = 1   out = norm(y) weight silu(z),        silu(z) = z / (1 + exp(-z))
 *   y       [rows][width] in x_dtype (a scan's y with its heads and channels as one row)
 *   z       [rows] rows of width channels in dtype, z_stride elements apart (>= width): a
 *           slice of the input projection's rows
 *   weight  [width] float32, or NULL for ones
 *   out     [rows][width] in dtype; may be y itself when the types are the same, must not
 *           overlap anything else
 * Errors: BDSSM_ERR_NULL, BDSSM_ERR_SHAPE, BDSSM_ERR_UNSUPPORTED (dtypes, kind, eps, more than
 * 16384 channels in a group, rows that reach past 64-bit addresses), BDSSM_ERR_ALIGN,
 * BDSSM_ERR_ALIAS, BDSSM_ERR_HIP.
 */
bdssm_status bdssm_gated_norm(const bdssm_norm_dims *dims, const void *y, const void *z, int64_t z_stride,
                              const float *weight, int32_t norm_first, void *out, void *stream);

/*
 * The residual update between two blocks: the norm after the block that ends, its gate and
 * residual scale, the addition, and the norm before the block that begins, with the timestep's
 * gain and shift (AdaLN: gamma_t norm(x) + beta_t; "Breaking the Bottleneck with DiffuApriel",
 * Sec. 3.2, eqs. (7)-(9)):
 *   t = norm(o) post_w (o itself when post_w is NULL)
 *   r = x + res_scale * gate[s] t
 *   u = norm(r) pre_w gain[s] + shift[s]            s = row / rows_per_stream
 *   x          [rows][width] in x_dtype: the residual stream
 *   o          [rows][width] in dtype: the block's output, or NULL for r = x
 *   post_w, pre_w      [width] float32, or NULL (no post norm; ones)
 *   gate, gain, shift  per stream [width] in dtype, mod_stride elements from stream to stream
 *                      (slices of one projection of the timestep), each or NULL (1, 1, 0)
 *   x_out      [rows][width] in x_dtype: r; may be x itself; NULL = not wanted
 *   u          [rows][width] in dtype: the next block's input; NULL = not wanted (one of the
 *              two is required). u is taken from r before r is rounded to x_dtype.
 * Outputs must not overlap anything but x_out == x. Errors as bdssm_gated_norm.
 */
typedef struct {
    const void *x, *o;
    const float *post_w, *pre_w;
    const void *gate, *gain, *shift;
    int64_t mod_stride;
    float res_scale;
} bdssm_residual;
bdssm_status bdssm_residual_norm(const bdssm_norm_dims *dims, const bdssm_residual *r, void *x_out, void *u,
                                 void *stream);

/*
 * Attention layers of the hybrid. A block-diffusion hybrid puts an attention layer between
 * groups of Mamba layers; its cache is the keys and values K_{1:k-1}, V_{1:k-1} of the
 * committed blocks (eq. (6) of "Training Hybrid Block Diffusion Language Models with Partial
 * Bidirectionality"), and its step and commit are to that cache what bdssm_block_step and
 * bdssm_commit are to the state: the step reads the cache and never writes it, the commit
 * (bdssm_kv_append) appends the finished block's keys and values.
 *
 * Paged cache: keys and values live in two pools of pages
 *     [num_pages][kv_heads][page_size][headdim],
 * and stream b's cached token j is slot j % page_size of page table[b][j / page_size]. An entry
 * outside [0, num_pages) is a page the stream does not hold (one given back): its tokens are
 * not attended to, and appends to it are dropped. lens[b] tokens of stream b are cached; lens
 * below 0 or above max_len are taken as 0 and max_len. Slots past a stream's length are never
 * used, whatever they hold.
 *
 * Chunk: the new tokens of every stream, rows of [heads][headdim] a stride apart (slices of one
 * projection). With starts NULL, stream b has the block_len rows from b * block_len; else the
 * rows starts[b] .. starts[b+1]-1 (ascending, at most block_len of them, which may be 0; a
 * longer stream's rows past block_len, and rows past `tokens`, are not computed).
 *
 * Chunk token i of stream b is at position p = lens[b] + i, cached token j at position j. A
 * query at p attends to key j (cached or of the chunk itself) when
 *     block = 0   always               block > 0   j / block <= p / block   (1: causal;
 *                                      32: whole blocks of 32, causal between them)
 * and window = 0 or p - j < window or j < sinks (a sliding window that looks `window` tokens
 * back, its own among them, beside the first `sinks` tokens). The softmax is over scale * q.k,
 * its maximum, sum and the weighted sum of values in float32; with bf16 values each weight is
 * rounded to bf16 for the matrix product. No weight exceeds 1 before the division by their sum,
 * so that a result is finite where the sum of the values' magnitudes is. A query that attends to
 * nothing gets zeros. What keys
 * and values hold that a query does not attend to never reaches its row, infinities and NaN
 * included; but beside a row that does attend to one, sums may be taken in another order and
 * weights rounded from another reference, so a row's last bits may depend on it.
 */
typedef struct {
    int32_t batch;     /* streams */
    int32_t nheads;    /* query heads, at most 512, a multiple of kv_heads: head h reads KV
                          head h / (nheads / kv_heads) */
    int32_t kv_heads;
    int32_t headdim;   /* 64 or 128 */
    int32_t dtype;     /* bdssm_dtype of q, k, v, the pages and out */
    int32_t page_size; /* tokens per page: 16, 32, 64, 128 or 256 */
} bdssm_attn_dims;

typedef struct {
    void *k, *v;          /* pools of pages; written by bdssm_kv_append only */
    const int32_t *table; /* [batch][max_pages] device page numbers */
    const int32_t *lens;  /* [batch] device cached tokens */
    int32_t num_pages;    /* pages in each pool */
    int32_t max_pages;    /* entries of a table row */
    int32_t max_len;      /* upper bound of lens (known on the host; sizes the launch);
                             at most max_pages * page_size */
} bdssm_kv_cache;

typedef struct {
    const void *q, *k, *v;              /* first rows; q unused by bdssm_kv_append */
    int64_t q_stride, k_stride, v_stride; /* elements between rows, multiples of 16 bytes, at
                                             most 2^24 */
    int64_t tokens;                     /* rows of q, k, v and out (batch * block_len when
                                           starts is NULL) */
    const int32_t *starts;              /* [batch + 1] device row offsets, or NULL */
    int32_t block_len;                  /* tokens of a stream, or the most of any */
} bdssm_attn_chunk;

typedef struct {
    float scale;    /* of q.k, > 0: e.g. 1 / sqrt(headdim) */
    int32_t block;  /* 0: no order; else tokens of a block (>= 1) */
    int32_t window; /* 0: none; else >= 1 */
    int32_t sinks;  /* >= 0; first tokens outside the window that stay visible */
} bdssm_attn_mask;

/*
 * Attention of the chunk's tokens over the cache and the chunk itself (cache and chunk are
 * only read).
 *   chunk->k, chunk->v  both NULL: the chunk has no keys of its own, the queries attend to the
 *             cache alone (then a mask can leave a query nothing)
 *   out       [tokens][nheads][headdim] in dtype; must not overlap anything
 *   workspace at least bdssm_attn_step_workspace(...) bytes for block_len, max_len and mask:
 *             partial results of a long cache that is split over workgroups. What the query
 *             says for one max_len serves every smaller one too, so that a decoding loop
 *             allocates once, for its longest cache. Other dims, another block_len (a smaller one
 *             too) or mask may need more: ask for each
 * Errors: BDSSM_ERR_NULL, BDSSM_ERR_SHAPE, BDSSM_ERR_UNSUPPORTED (headdim, page_size, dtype),
 * BDSSM_ERR_ALIGN (base pointers and row strides to 16 bytes; table, lens and starts to 4),
 * BDSSM_ERR_ALIAS, BDSSM_ERR_WORKSPACE, BDSSM_ERR_HIP. The workspace query returns SIZE_MAX
 * for arguments the call would reject.
 */
size_t bdssm_attn_step_workspace(const bdssm_attn_dims *dims, int32_t block_len, int32_t max_len,
                                 const bdssm_attn_mask *mask);
bdssm_status bdssm_attn_step(const bdssm_attn_dims *dims, const bdssm_attn_chunk *chunk, const bdssm_kv_cache *cache,
                             const bdssm_attn_mask *mask, void *out, void *workspace, size_t workspace_bytes,
                             void *stream);

/*
 * The commit of an attention layer: the chunk's keys and values become cached tokens
 * lens[b] .. lens[b] + n_b - 1 of their stream (tokens past the table's last page are dropped).
 *   lens_out  [batch] int32: the new lengths, min(lens[b] + n_b, max_pages * page_size), or
 *             NULL; must not overlap lens, since every workgroup reads it (a caller swaps the
 *             two). max_len bounds the lengths before the append.
 * Errors as bdssm_attn_step.
 */
bdssm_status bdssm_kv_append(const bdssm_attn_dims *dims, const bdssm_attn_chunk *chunk, const bdssm_kv_cache *cache,
                             int32_t *lens_out, void *stream);

/*
 * Attention with shaped scores or ranges of each token's own: bdssm_attn_step (its layouts, mask,
 * sums and roundings) whose score of query head h at position p with key j becomes
 *     s = scale * q.k                                  (mask->scale)
 *     s = cap * tanh(s / cap)                          where cap > 0
 *     s = s - slopes[h] * |p - j|                      where slopes is given
 * and whose mask becomes
 *     order:   as bdssm_attn_step, or j < prefix[b]    (the first prefix[b] positions of stream b
 *              are visible to each of its queries: a prompt that sees itself whole)
 *     window:  as bdssm_attn_step (it limits a prefix too)
 *     range:   first[i] <= j < last[i] for chunk row i, sinks included (the borders of the
 *              token's document, as positions of its stream; first >= last: the token attends
 *              to nothing, and gets zeros)
 * Positions outside the stream's keys are taken as their nearest end. Distances are exact up to
 * 2^24 and count from the nearest position that the query's window, order and range leave.
 * Workgroups skip keys that the ranges of all their rows leave out, so that documents packed
 * into one chunk cost about what they cost as streams of their own.
 *   cap       0 (none) or > 0, finite
 *   slopes    [nheads] device float32, finite, or NULL. Scores with their bias are held up to 2^26 in
 *             magnitude: a slope beyond that counts as 2^26 and a bias below -2^26 as that (or as
 *             itself), so that a steep slope leaves the nearest key all of a row's weight
 *   prefix    [batch] device int32, or NULL
 *   first, last  [tokens] device int32 in the order of chunk rows, each or NULL (0, no end)
 * Errors as bdssm_attn_step; BDSSM_ERR_UNSUPPORTED also for a cap that is negative or not finite,
 * or for which scale / cap or cap itself is beyond 2^-126 to 2^126 or so, and for a scale outside
 * 2^-64 to 2^64 where slopes are given. out and workspace must not overlap these arrays.
 * bdssm_attn_step_ex_workspace says what the call needs as bdssm_attn_step_workspace does; of
 * scores it looks at cap and at whether first and last are given, not at what they hold: without
 * ranges it is the same.
 */
typedef struct {
    float cap;
    const float *slopes;
    const int32_t *prefix;
    const int32_t *first, *last;
} bdssm_attn_scores;
size_t bdssm_attn_step_ex_workspace(const bdssm_attn_dims *dims, int32_t block_len, int32_t max_len,
                                    const bdssm_attn_mask *mask, const bdssm_attn_scores *scores);
bdssm_status bdssm_attn_step_ex(const bdssm_attn_dims *dims, const bdssm_attn_chunk *chunk, const bdssm_kv_cache *cache,
                                const bdssm_attn_mask *mask, const bdssm_attn_scores *scores, void *out,
                                void *workspace, size_t workspace_bytes, void *stream);

/*
 * Rotary positions: in each head the channels of a pair (a, b) are turned by the angle t of the
 * token's position and the pair's frequency f_i (radians per position),
 *     a' = scale (a cos t - b sin t),  b' = scale (a sin t + b cos t),   t = position * f_i
 * for pairs i < dim / 2 of channels (i, i + dim / 2), or (2i, 2i + 1) where interleaved; channels
 * from dim on are taken over as they are. Frequencies come as turns per position in units of
 * 2^-64, so that a position's angle, whole turns left out, is one wrapping integer product: it is
 * off by |position| 2^-65 turns at most, at any position. Sines and cosines are float32 with an
 * error of a few 2^-24, and so are products and sums, rounded once to dtype.
 *
 * bdssm_rotary_turns fills such a table on the host (copied to the device once, by the caller):
 *     f_i = base^(-2i / dim)                                     BDSSM_ROTARY_PLAIN
 *     f_i / factor                                               BDSSM_ROTARY_LINEAR
 *     the same of base factor^(dim / (dim - 2))                  BDSSM_ROTARY_BASE  (dim > 2: the
 *         lowest frequency is divided by factor, the highest is kept)
 *     f_i (g + (1 - g) / factor)                                 BDSSM_ROTARY_PARTS
 *         g = (r - low) / (high - low) within 0 and 1, r = trained f_i / (2 pi): pairs that make
 *         more than `high` turns within the trained length are kept, those with fewer than `low`
 *         are divided by factor
 *   turns   [dim / 2] host, written
 * Errors: BDSSM_ERR_NULL, BDSSM_ERR_SHAPE (dim odd, below 2 or above 512), BDSSM_ERR_UNSUPPORTED
 * (kind; base < 1, factor <= 0 or not finite; BASE with dim 2; PARTS with trained < 1 or
 * low >= high).
 */
enum { BDSSM_ROTARY_PLAIN = 0, BDSSM_ROTARY_LINEAR = 1, BDSSM_ROTARY_BASE = 2, BDSSM_ROTARY_PARTS = 3 };
typedef struct {
    int32_t dim;     /* rotated channels of a head */
    int32_t kind;
    double base;     /* e.g. 10000 */
    double factor;   /* how much longer than trained (ignored by PLAIN) */
    int32_t trained; /* PARTS: tokens of the contexts trained on */
    double low, high; /* PARTS: turns */
} bdssm_rotary_freqs;
bdssm_status bdssm_rotary_turns(const bdssm_rotary_freqs *freqs, uint64_t *turns);

typedef struct {
    int32_t dim;              /* rotated channels: even, 2 .. headdim */
    int32_t interleaved;      /* 0 or 1 */
    float scale;              /* of the rotated channels: 1, or a long context's factor; finite */
    const uint64_t *turns;    /* [dim / 2] device, 8-byte aligned */
    const int32_t *positions; /* [tokens] device, one for each chunk row (any value, negative ones
                                 too), or NULL: chunk token i of stream b is at lens[b] + i */
} bdssm_rotary;

typedef struct {
    void *q, *k;                /* first rows of [nheads][headdim] and of [kv_heads][headdim] */
    int64_t q_stride, k_stride; /* elements between rows, as in bdssm_attn_chunk */
} bdssm_rotary_out;

/*
 * Turns the chunk's queries and keys (each may be NULL with its output, not both; the chunk's v
 * is not used).
 *   lens   [batch] device: cached tokens, or NULL for none; below 0 taken as 0 (not read when
 *          positions are given)
 *   out    rows out->q, out->k: the chunk's own rows in place (same address and stride), or rows
 *          that overlap nothing. Slices of the same projection rows do not overlap.
 * Errors: BDSSM_ERR_NULL, BDSSM_ERR_SHAPE, BDSSM_ERR_UNSUPPORTED (also a chunk whose streams may
 * have more than 2^24 tokens each), BDSSM_ERR_ALIGN, BDSSM_ERR_ALIAS, BDSSM_ERR_HIP, as
 * bdssm_attn_step.
 */
bdssm_status bdssm_rotary_step(const bdssm_attn_dims *dims, const bdssm_attn_chunk *chunk, const bdssm_rotary *rotary,
                               const int32_t *lens, const bdssm_rotary_out *out, void *stream);

/*
 * The same on the way into the cache: queries to out->q, keys turned into the pages (and to
 * out->k where it is given), values into the pages, in one launch: bdssm_rotary_step followed by
 * bdssm_kv_append of its keys. The positions of the turn are the cache's own (lens[b] + i, lens
 * taken within 0 and max_len) unless rotary->positions gives others; the slots are the append's.
 *   chunk->q with out->q   both NULL: keys alone
 *   out      may be NULL when there are no queries
 *   lens_out as in bdssm_kv_append
 */
bdssm_status bdssm_rotary_append(const bdssm_attn_dims *dims, const bdssm_attn_chunk *chunk, const bdssm_kv_cache *cache,
                                 const bdssm_rotary *rotary, const bdssm_rotary_out *out, int32_t *lens_out, void *stream);

/*
 * Upkeep of a paged cache on the device, without a host round trip, so that a decoding loop that
 * takes, shares and gives back pages can be recorded as a graph. What the attention layers of a
 * stack share is one table and one pool's bookkeeping:
 *   table  [batch][max_pages]  as in bdssm_kv_cache; entries outside [0, num_pages) hold nothing
 *   lens   [batch]             cached tokens, taken within 0 and max_pages * page_size
 *   uses   [num_pages]         table entries that name a page; 0 (or less): the page is free
 * Pages are given out lowest number first, to streams in order, and a page that a call gives back
 * is free from the next call on: results depend on the contents alone. Integer atomics count the
 * uses, in whose order nothing depends.
 *   table_out, uses_out   may be table and uses themselves (in place) except for the fork's
 *                         table_out; else must not overlap anything
 *   workspace             at least bdssm_pages_workspace(dims) bytes (the same for all calls),
 *                         16-byte aligned; two calls that may run at the same time need one each
 * A whole page may be shared: a stream's length is not to be lowered into one and written again.
 * No call reads a count that the host does not have: where pages run out, the entries that lack
 * one stay empty (-1) and lacking[0] says how many.
 * Errors: BDSSM_ERR_NULL, BDSSM_ERR_SHAPE, BDSSM_ERR_UNSUPPORTED (page_size, batch above 65535,
 * positions past 2^31, an advance that could need 2^31 pages), BDSSM_ERR_ALIGN (4 bytes; workspace
 * 16), BDSSM_ERR_ALIAS, BDSSM_ERR_WORKSPACE, BDSSM_ERR_HIP. The query returns SIZE_MAX for dims the
 * calls reject.
 */
typedef struct {
    int32_t batch;     /* streams */
    int32_t page_size; /* tokens per page: 16, 32, 64, 128 or 256 */
    int32_t num_pages; /* pages of the pool */
    int32_t max_pages; /* entries of a table row */
} bdssm_pages_dims;

typedef struct {
    const int32_t *table, *lens, *uses;
} bdssm_pages;

size_t bdssm_pages_workspace(const bdssm_pages_dims *dims);

/*
 * Before a block is decoded (or appended): afterwards every stream holds the pages of its tokens
 * [0, lens[b] + n_b), n_b its new tokens, that a later query can see, and no others. Pages wholly
 * behind the window (and past the sinks) and pages wholly past the new tokens are given back;
 * entries from the first page that starts at lens[b] or later are filled with free pages. An empty
 * entry among cached tokens stays empty.
 *   starts     [batch + 1] device, as in bdssm_attn_chunk, or NULL: block_len tokens each
 *   block_len  new tokens of a stream, or the most of any
 *   window, sinks  as in bdssm_attn_mask
 *   lacking    [1] device: entries that found no free page
 */
bdssm_status bdssm_pages_advance(const bdssm_pages_dims *dims, const bdssm_pages *pages, const int32_t *starts,
                                 int32_t block_len, int32_t window, int32_t sinks, int32_t *table_out,
                                 int32_t *uses_out, int32_t *lacking, void *workspace, size_t workspace_bytes,
                                 void *stream);

/*
 * Streams rearranged, forked and ended: row b becomes the stream of row parents[b] (itself, if it
 * goes on). Streams with one parent share its whole pages; the first of them keeps its last,
 * partly filled page and what is held past it, each other one takes a free page for a copy of the
 * partly filled one. So pages that are still written have one user. A parent outside [0, batch)
 * leaves the row empty, and a row that no one descends from gives its pages back.
 *   parents    [batch] device
 *   table_out  must not overlap table;  lens_out [batch], must not overlap lens
 *   copies     [batch][2] device, written: (source, destination) for row b, or (-1, -1): the page
 *              copies to be made, in every layer's pools, by bdssm_pages_copy
 *   lacking    [1] device: copies that found no free page (the entry stays empty)
 */
bdssm_status bdssm_pages_fork(const bdssm_pages_dims *dims, const bdssm_pages *pages, const int32_t *parents,
                              int32_t *table_out, int32_t *lens_out, int32_t *uses_out, int32_t *copies,
                              int32_t *lacking, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Moves the used pages to the front of the pool: of n used pages, those numbered n or above go to
 * the free pages below n, the highest to the lowest. Afterwards exactly pages 0 to n - 1 are used.
 *   copies  [num_pages / 2][2] device, written: (source, destination) of the moves, then (-1, -1)
 *   live    [1] device: n
 */
bdssm_status bdssm_pages_compact(const bdssm_pages_dims *dims, const bdssm_pages *pages, int32_t *table_out,
                                 int32_t *uses_out, int32_t *copies, int32_t *live, void *workspace,
                                 size_t workspace_bytes, void *stream);

/*
 * Copies pages within one layer's pools (keys and values), as a fork's or a compaction's list says:
 * to be called for every layer, before the pages are read or given out again.
 *   cache   k, v and num_pages are used
 *   copies  [n][2] device (source, destination). Entries with a page outside the pool, and copies
 *           of a page to itself, are left out. No destination may be another entry's source or
 *           destination (a list that a fork or a compaction wrote never has one): what such a page
 *           holds afterwards is not defined.
 * Errors as bdssm_kv_append.
 */
bdssm_status bdssm_pages_copy(const bdssm_attn_dims *dims, const bdssm_kv_cache *cache, const int32_t *copies, int32_t n,
                              void *stream);

/*
 * Launch-shape override, for tests and launch-shape sweeps only (not for the hot path).
 * Several kernels implement the block step, each one in full and each checked against the
 * same bounds; the library picks one per call from the shapes. This call pins that choice
 * for every later call in the process until it is called again (NULL or all zeros =
 * automatic). Values are read once per call; a change racing with calls on other threads
 * applies to each of them either entirely or not at all.
 *   block_kernel  0 automatic; 1 the small-batch kernel (used where it applies:
 *                 block_len <= 32, bf16 inputs, (d_state, headdim) = (128, 64));
 *                 2 the bandwidth kernels
 *   lat_waves     small-batch kernel: wavefronts per workgroup, 2 or 4 (0 automatic)
 *   bw_heads      bandwidth kernels: heads per workgroup; ignored unless it divides H/G
 *                 (0 automatic)
 *   bw_splits     bandwidth kernel from the float32 state: column splits, 1, 2 or 4
 *                 (0 automatic)
 * Errors: BDSSM_ERR_UNSUPPORTED for values outside these sets (nothing is changed).
 */
typedef struct {
    int32_t block_kernel;
    int32_t lat_waves;
    int32_t bw_heads;
    int32_t bw_splits;
} bdssm_launch_override;
bdssm_status bdssm_set_launch_override(const bdssm_launch_override *o);

#ifdef __cplusplus
}
#endif

#endif /* BDSSM_H */
