/*
 * dspark.h -- C ABI of the DSpark per-cycle hot path on one GB300 (sm_103a).
 *
 * The method is DSpark's semi-autoregressive draft + confidence-scheduled
 * verification, as described in
 *   [D] "DSpark: confidence-scheduled speculative decoding" (ai-papers-daily
 *       digest): eq. (4) causal block distribution, eq. (5) Markov head,
 *       eq. (6) RNN head, eq. (7) confidence head, Module D (sequential
 *       temperature scaling), Module E + Algorithm 1 (prefix scheduler),
 *       Appendix A, production section (async top-K, flattened batch);
 *   [E] "DSpark explained" (interactive explainer), section 06 (single-token
 *       rejection rule).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - All tensor pointers are DEVICE pointers owned by the caller; row-major,
 *   contiguous, with the shapes given per field.  The library allocates no
 *   device memory: scratch comes from the caller through `ws`, whose size the
 *   matching *_workspace_size() function returns (256-byte aligned pointer;
 *   one that is not even 16-byte aligned is refused).
 * - Every call only enqueues work on `stream` (a cudaStream_t) and returns
 *   without synchronising.  Calls on one stream run in order.
 * - dtype: DSPARK_F32 or DSPARK_BF16 applies to U, h, W1, W2t, W and T.
 *   Logits accumulate in fp32 whatever the storage type.
 * - Return value: DSPARK_OK, or an error code for a problem the host can see
 *   (bad shape, NULL pointer, unsupported size, CUDA launch failure); the
 *   message is in dspark_last_error() (thread-local).  Problems only the
 *   device can see (a token id >= V, malformed tags, a confidence outside
 *   [0, 1], non-finite logits) are written as the first non-zero error code
 *   into `*err` (a device int32 the caller zeroes; may be NULL to ignore) and
 *   the outputs of the affected rows are then unspecified.
 * - Sampling is deterministic given (seed, cycle): Philox-4x32-10 with
 *   key = (seed lo, seed hi) and counter = (w0, w1, request, cycle << 2 | stream);
 *   stream 0 the draft draw (w0 = b / 2 for vocabulary block b of 16 entries,
 *   w1 = step k; words 2 (b % 2) and 2 (b % 2) + 1 are block b's uniforms u_b
 *   and u'_b): the block is argmax_b ln S_b - ln(-ln u_b) (S_b the block's sum
 *   of exp(z), ties to the lowest b), the token the first entry of that block
 *   whose running sum of exp(z) exceeds u'_b S_b,
 *   stream 1 acceptance uniforms (w0 = 0, w1 = position j, word 0),
 *   stream 2 the residual / bonus draw (w0 = 0, w1 = position, word 0): one
 *   uniform u per request, the token the first v whose cumulative weight
 *   (fp32, vocabulary order) exceeds u times the total weight.
 *   A word w maps to u = ((w >> 9) + 1/2) 2^-23.  Only the low 30 bits of
 *   `cycle` enter the counter.
 */
#ifndef DSPARK_H
#define DSPARK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define DSPARK_API __attribute__((visibility("default")))
#else
#define DSPARK_API
#endif

typedef struct CUstream_st *dspark_stream_t; /* same type as cudaStream_t */

enum {
    DSPARK_OK = 0,
    DSPARK_ERR_INVAL = 1,       /* bad argument: NULL pointer, shape, mode     */
    DSPARK_ERR_RANGE = 2,       /* token id >= V, B outside the SPS table,     */
                                /* confidence outside [0, 1]                   */
    DSPARK_ERR_NONFINITE = 3,   /* NaN / Inf logits left no sample             */
    DSPARK_ERR_CUDA = 4,        /* a CUDA runtime call failed                  */
    DSPARK_ERR_TIMEOUT = 5,     /* a bounded device-side wait gave up          */
    DSPARK_ERR_UNSUPPORTED = 6  /* size beyond what this build handles         */
};

enum { DSPARK_F32 = 0, DSPARK_BF16 = 1 };
enum { DSPARK_SCHED_SYNC = 0, DSPARK_SCHED_ASYNC = 1 };

/* ------------------------------------------------------------------------ */
/* Draft, Markov head.  [D] eq. (5) B(x_{k-1}, .) = W_1[x_{k-1}] W_2 added to  */
/* the base logits U_k in eq. (4), sampled left to right for k = 1..gamma     */
/* from the anchor x_0; confidence c_k = sigma(w^T [h_k ; W_1[x_{k-1}]] / T_k) */
/* by eq. (7) with the Module D temperature T_k (1 when sts_T is NULL).       */
/* ------------------------------------------------------------------------ */
typedef struct {
    int32_t R;            /* requests                                           */
    int32_t gamma;        /* block length                                       */
    int32_t V;            /* vocabulary                                         */
    int32_t r;            /* rank of W_1 W_2                                    */
    int32_t d;            /* hidden size of h                                   */
    int32_t dtype;        /* DSPARK_F32 | DSPARK_BF16                           */
    const void *U;        /* [R, gamma, V] base logits U_k                      */
    const void *h;        /* [R, gamma, d] backbone hidden states h_k           */
    const void *W1;       /* [V, r] embedding table W_1                         */
    const void *W2t;      /* [V, r] W_2 transposed: row v is column v of W_2    */
    const float *w;       /* [d + r] confidence weights (hidden part first)     */
    const float *sts_T;   /* [gamma] temperatures T_k, or NULL for 1            */
    const int32_t *anchor;/* [R] anchor tokens x_0                              */
    uint64_t seed;        /* Philox key                                         */
    uint64_t cycle;       /* decoding-cycle counter (Philox counter word 3)     */
    int32_t *x;           /* out [R, gamma] drafted tokens x_1..x_gamma         */
    float *logq;          /* out [R, gamma] log q_k(x_k)                        */
    float *lse;           /* out [R, gamma] log sum_v exp(U_k(v) + B_k(v))      */
    float *c;             /* out [R, gamma] confidences c_k                     */
    int32_t *err;         /* device error word (see conventions), or NULL       */
    float *conf_logit;    /* out [R, gamma] w^T [h_k ; W_1[x_{k-1}]], the logit  */
                          /* before 1/T_k (the input of dspark_sts_fit), or NULL */
} dspark_draft_args;

DSPARK_API size_t dspark_draft_markov_workspace_size(const dspark_draft_args *a);
DSPARK_API int dspark_draft_markov(const dspark_draft_args *a, void *ws, dspark_stream_t stream);
/* Step k (1..gamma) of the same loop alone: reads x_{k-1} (the anchor for
 * k = 1, else column k-2 of a->x) and writes column k-1 of x, logq, lse, c.
 * dspark_draft_markov equals calls for k = 1..gamma in order on one stream
 * with one workspace; the split lets an engine interleave other work between
 * steps.  Step 1 (re)starts the per-draft step counters kept in the
 * workspace, so a step k > 1 must follow steps 1..k-1 of the same draft.
 * (dspark_draft_markov itself runs all gamma steps in one launch on the
 * tensor-core path.) */
DSPARK_API int dspark_draft_markov_step(const dspark_draft_args *a, int32_t k, void *ws,
                                        dspark_stream_t stream);

/* Markov-head draft that allocates nothing and takes no workspace.
 *
 * The paper has no counterpart to this call; it exists for callers that
 * cannot allocate device memory: a plugin living inside another runtime whose
 * caching allocator already owns the device's memory, a plain C host with no
 * allocator of its own, or a code path that must not call cudaMalloc because
 * that call can synchronise the device.  Such callers still pass every input
 * and output tensor; only the scratch (the per-slice partial results the
 * steps exchange) comes from a fixed array inside the library, which every
 * GPU that loads the library holds until the process exits.
 *
 * - Limit: the scratch is what dspark_draft_markov_workspace_size() returns
 *   for the same arguments -- 32 bytes per (request, vocabulary range), once
 *   per step on the tensor-core path, plus 8 bytes per (request, step) and
 *   256, each part rounded up to 256 bytes; the ranges are one per SM on the
 *   tensor-core path (bf16, r a multiple of 64 up to 256, V a multiple of 8:
 *   all the standard workloads, under 11 MiB) and ceil(V / 64) on the
 *   CUDA-core path --
 *   and the array holds
 *   DSPARK_NOALLOC_SCRATCH_BYTES (16 MiB).  Larger needs return
 *   DSPARK_ERR_UNSUPPORTED (message in dspark_last_error()) and launch nothing.
 * - The first call on each device looks up the array's device address (with
 *   that device current) and caches it with the id of the device's current
 *   context; a call in another context of the device (after cudaDeviceReset,
 *   for instance, which unloads the module) looks it up again.  Make the first
 *   call in each context before any stream capture on the device.
 * - Every call on a device shares the one array.  Each call first clears the
 *   part that must start at zero (completion counters, with an asynchronous
 *   memset on the stream) and every step overwrites the rest before reading
 *   it, but calls that overlap on the GPU (different streams, or different
 *   host threads) race: serialise them, e.g. by issuing them on one stream.
 * Results equal dspark_draft_markov's for the same arguments. */
#define DSPARK_NOALLOC_SCRATCH_BYTES (16u << 20)
DSPARK_API int dspark_draft_markov_noalloc(const dspark_draft_args *a, dspark_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Draft, RNN head.  [D] eq. (6): z_k = [s_{k-1}; W_1[x_{k-1}]; h_k],          */
/* s_k = sigma(W_g z_k) s_{k-1} + (1 - sigma(W_g z_k)) tanh(W_c z_k),          */
/* B_k = W_2^T tanh(W_o z_k); otherwise as the Markov head.                    */
/* ------------------------------------------------------------------------ */
typedef struct {
    dspark_draft_args base; /* fields as for the Markov head                    */
    const void *W;          /* [3r, 2r + d]: rows [0,r) W_g, [r,2r) W_c, [2r,3r) W_o */
    const float *s0;        /* [R, r] initial state, or NULL for s_0 = 0        */
    float *A;               /* out [R, gamma, r] A_k = tanh(W_o z_k), the vector */
                            /* whose product with W_2 is B_k (verify needs it)  */
    float *s_out;           /* out [R, r] final state s_gamma, or NULL          */
} dspark_rnn_args;

/* The h_k columns of W do not depend on the recurrence: W[:, 2r:] h_k is
 * formed for all (request, k) first, one bf16 GEMM on the tensor cores
 * (tcgen05; fp32, or shapes it does not take -- d or 2r + d not a multiple of
 * 8 -- go to a CUDA-core kernel).  The workspace holds the draft scratch, two
 * [R, r] state buffers, the [R gamma, 3r] fp32 projection and 128 KiB per
 * 128 requests for the bf16 operands the tensor-core steps prepare. */
DSPARK_API size_t dspark_draft_rnn_workspace_size(const dspark_rnn_args *a);
DSPARK_API int dspark_draft_rnn(const dspark_rnn_args *a, void *ws, dspark_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Hardware-aware prefix scheduler.  [D] Module E, Algorithm 1:               */
/* a_{r,j} = prod_{i<=j} c_{r,i}; pool E = {(r,j): a_{r,j} > 0} sorted by a    */
/* descending (ties: request, then position, ascending); scan with            */
/* B = R + #admitted, tau = R + sum admitted a, Theta = tau * SPS(B).         */
/*  - DSPARK_SCHED_SYNC: Algorithm 1 with the early-stop break.                */
/*  - DSPARK_SCHED_ASYNC (production section): admit the top min(K, |E|)      */
/*    entries of the current order, no break, with K read from *K_in (the     */
/*    capacity computed two cycles earlier); *K_in < 0 or K_in == NULL falls  */
/*    back to SYNC.  Both modes write *K_out = argmax_m Theta(m) over the     */
/*    current pool without break (smallest m on ties), for use at cycle t+2.  */
/* Number formats: a is an fp32 running product; tau is summed exactly as     */
/* integers in units of 2^-32 (each a rounded to nearest-even on that grid);  */
/* Theta = (tau units * 2^-32) * SPS(B) in fp64.  Results are bit-exact.      */
/* Limits: R * gamma <= 8192.  The table must cover B in [R, R (gamma + 1)]   */
/* (checked on the host: DSPARK_ERR_RANGE).                                   */
/* ------------------------------------------------------------------------ */
typedef struct {
    int32_t R, gamma;
    const float *c;        /* [R, gamma] confidences, each in [0, 1]            */
    const double *sps;     /* [B_count] SPS(B_min + i), steps per second         */
    int32_t B_min, B_count;
    int32_t mode;          /* DSPARK_SCHED_SYNC | DSPARK_SCHED_ASYNC             */
    const int32_t *K_in;   /* device scalar: async capacity, or NULL             */
    int32_t *ell;          /* out [R] verify lengths l_r in 0..gamma             */
    int32_t *K_out;        /* out device scalar: capacity for cycle t + 2        */
    double *theta_best;    /* out device scalar: Theta at the admitted point     */
    float *a;              /* out [R, gamma] survival products, or NULL          */
    int32_t *err;
} dspark_sched_args;

DSPARK_API size_t dspark_schedule_workspace_size(const dspark_sched_args *a);
DSPARK_API int dspark_schedule(const dspark_sched_args *a, void *ws, dspark_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Flattened batch layout ([D] production section, marker tensor): from     */
/* ell [R] write tags [N, 2] = (request, position) for positions 0..l_r of   */
/* each request in request order, and N = sum_r (1 + l_r) to *N_out (device).*/
/* tags must hold R (gamma + 1) rows.                                         */
/* ------------------------------------------------------------------------ */
DSPARK_API int dspark_build_tags(int32_t R, int32_t gamma, const int32_t *ell, int32_t *tags,
                                 int32_t *N_out, int32_t *err, dspark_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Lossless verification.  [E] section 06: accept x_{j+1} with probability    */
/* min(1, p_j(x_{j+1}) / q_{j+1}(x_{j+1})), test: log u < log p - log q with */
/* u from Philox stream 1; at the first rejection j* sample y from           */
/* norm(max(0, p_{j*} - q_{j*+1})) (q recomputed from U, the bias operand and */
/* W_2; p itself if the residual is empty); if all l_r tokens pass sample     */
/* the bonus y from p_{l_r}, both by inverse CDF (one stream-2 uniform per   */
/* request; the pages fix no sampler, any exact draw keeps the method        */
/* lossless).  Row i of T is the target's logits for position                */
/* tags[i] = (r, j), i.e. the distribution of x_{j+1} given x_0..x_j; rows    */
/* are grouped by request with positions 0..l_r ascending, every request      */
/* present (violations: DSPARK_ERR_INVAL in *err).                            */
/* Entries of -inf have probability 0.  A row of nothing else allows no token: */
/* the drafted token tested on it is rejected, and the request's y, which is  */
/* then drawn from it, is 0, a token that it does not allow either, with      */
/* DSPARK_ERR_NONFINITE in *err; the other requests are not touched by it.    */
/* ------------------------------------------------------------------------ */
typedef struct {
    int32_t R, gamma, V, r, dtype;
    int32_t N;              /* rows of T (the capacity when N_dev is given)     */
    const int32_t *N_dev;   /* device scalar: rows in use, or NULL for N        */
    const void *T;          /* [N, V] target logits, flattened                  */
    const int32_t *tags;    /* [N, 2] (request, position)                       */
    const int32_t *anchor;  /* [R] x_0                                          */
    const int32_t *x;       /* [R, gamma] drafted tokens                        */
    const float *logq;      /* [R, gamma] from the draft                        */
    const float *lse;       /* [R, gamma] from the draft                        */
    const void *U;          /* [R, gamma, V] base logits (residual recompute)   */
    const void *W1;         /* [V, r] (Markov bias operand W_1[x_j])            */
    const void *W2t;        /* [V, r]                                           */
    const float *A;         /* [R, gamma, r] RNN bias operands, or NULL (Markov)*/
    uint64_t seed, cycle;
    int32_t *n_accept;      /* out [R] accepted draft tokens n_r                */
    int32_t *out_tokens;    /* out [R, gamma + 1] x_1..x_{n_r}, y, then -1      */
    int32_t *next_anchor;   /* out [R] y, the next cycle's anchor               */
    float *lse_p;           /* out [N] log sum exp of each row, or NULL         */
    float *logp;            /* out [N] log p_j(x_{j+1}) (NaN on last rows), or NULL */
    int32_t *err;
} dspark_verify_args;

DSPARK_API size_t dspark_verify_workspace_size(const dspark_verify_args *a);
DSPARK_API int dspark_verify(const dspark_verify_args *a, void *ws, dspark_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Sequential temperature scaling.  [D] Module D: c_i is the probability     */
/* that position i passes given that the positions before it passed, so the  */
/* prefix of length k is accepted with probability                           */
/* P_k = prod_{i<=k} sigma(s_i / T_i).  For k = 1..gamma in order, T_k is    */
/* the grid temperature that minimises the expected calibration error of P_k */
/* against the held-out outcome 1[n >= k], with T_1..T_{k-1} held fixed.     */
/* ECE: n_bins equal-width bins of [0, 1], bin(P) = min(floor(P n_bins),      */
/* n_bins - 1), ECE = (1/M) sum_b |sum_{m in b} (P_m - y_m)|.  The bin sums  */
/* are exact integers (P rounded to units of 2^-16 / n_bins), so results    */
/* depend on the order of the additions; the rounding can move a P within  */
/* 2^-17 / n_bins below a bin edge into the next bin.  Ties go to the lowest */
/* grid index.                                                               */
/* The fitted T is the draft's sts_T.  Device-side errors: a grid point that */
/* is not a positive finite number is skipped (DSPARK_ERR_INVAL), a NaN logit */
/* counts as 0 (DSPARK_ERR_NONFINITE), n outside 0..gamma is clamped          */
/* (DSPARK_ERR_RANGE).                                                        */
/* ------------------------------------------------------------------------ */
#define DSPARK_STS_MAX_GAMMA 64
#define DSPARK_STS_MAX_BINS 64
typedef struct {
    int32_t M;               /* held-out draft blocks                            */
    int32_t gamma;           /* positions per block (<= DSPARK_STS_MAX_GAMMA)    */
    int32_t G;               /* grid points                                      */
    int32_t n_bins;          /* ECE bins (1..DSPARK_STS_MAX_BINS)                */
    const float *logit;      /* [M, gamma] confidence logits s_k (conf_logit of  */
                             /* the draft, taken with T = 1)                     */
    const int32_t *n_accept; /* [M] accepted prefix length of each block, with   */
                             /* all gamma positions verified                     */
    const float *grid;       /* [G] candidate temperatures                       */
    float *T;                /* out [gamma] fitted temperatures T_k              */
    double *ece;             /* out [gamma] ECE of P_k at the fitted T_k         */
    double *curve;           /* out [gamma, G] ECE at every grid point, or NULL  */
    int32_t *err;            /* device error word, or NULL                       */
} dspark_sts_args;

/* Scratch: the [gamma, G, n_bins] bin sums (8 bytes each), gamma counters and
 * two [M] fp32 prefix-product buffers.  One launch per position on the given
 * stream, after one memset. */
DSPARK_API size_t dspark_sts_fit_workspace_size(const dspark_sts_args *a);
DSPARK_API int dspark_sts_fit(const dspark_sts_args *a, void *ws, dspark_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Acceptance diagnostics ([D] analysis 1: the per-position conditional      */
/* acceptance rate, whose denominator counts only the instances whose       */
/* positions 1..k-1 were all accepted; [D] offline results: the acceptance  */
/* length tau = accepted drafted tokens + the target's own token).           */
/* For the R requests of one cycle -- n_accept from dspark_verify, ell the    */
/* verified lengths (the scheduler's ell; NULL means gamma for all; ell < 0:  */
/* not in this cycle's batch, counted nowhere) -- the call ADDS into caller-  */
/* owned device counters, so consecutive cycles accumulate:                   */
/*   reached [gamma]   position k (index k-1) verified with 1..k-1 accepted   */
/*                     (ell >= k and n >= k - 1);                             */
/*   accepted [gamma]  position k accepted (n >= k);                          */
/*   tau_hist [gamma + 1]  requests by n (= tau - 1);                          */
/*   ell_hist [gamma + 1]  requests by ell (may be NULL).                      */
/* The conditional acceptance at position k is accepted / reached.  A request */
/* with n outside 0..min(ell, gamma) is skipped and DSPARK_ERR_RANGE written  */
/* to *err.  gamma <= DSPARK_DIAG_MAX_GAMMA.  No workspace; one launch.        */
/* ------------------------------------------------------------------------ */
#define DSPARK_DIAG_MAX_GAMMA 1024
typedef struct {
    int32_t R, gamma;
    const int32_t *n_accept;      /* [R]                                      */
    const int32_t *ell;           /* [R] or NULL                              */
    unsigned long long *reached;  /* [gamma]      accumulated                 */
    unsigned long long *accepted; /* [gamma]      accumulated                 */
    unsigned long long *tau_hist; /* [gamma + 1]  accumulated                 */
    unsigned long long *ell_hist; /* [gamma + 1]  accumulated, or NULL        */
    int32_t *err;                 /* device error word, or NULL               */
} dspark_accept_stats_args;

DSPARK_API int dspark_accept_stats(const dspark_accept_stats_args *a, dspark_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Drafter training losses ([D] Module F, eqs. 8-12) over B blocks of gamma   */
/* positions, row i = b gamma + k - 1, with w_k = exp(-(k - 1) / gamma):      */
/*   p_d = softmax(zd_i), p_t = softmax(zt_i) over V;                          */
/*   ce_i = -log p_d(xs_i); tv_i = ||p_d - p_t||_1; c*_i = 1 - tv_i / 2 (eq. 8);*/
/*   bce_i = -[c* log c + (1 - c*) log(1 - c)], c = sigma(s_i), evaluated as   */
/*           softplus(s_i) - c*_i s_i;                                         */
/*   L_ce, L_tv, L_conf = (1/B) sum_i w_k (ce_i, tv_i, bce_i)  (eqs. 9-11);    */
/*   L = a_ce L_ce + a_tv L_tv + a_conf L_conf  (eq. 12; the pages' defaults   */
/*       are 0.1, 0.9, 1.0).                                                   */
/* Outputs: row [N, 6] f32 = (lse_d, lse_t, ce, tv, c*, bce) per row (may be  */
/* NULL); loss [4] f64 = (L_ce, L_tv, L_conf, L), overwritten; grad_z [N, V]  */
/* f32 = dL/dzd with c* held fixed as a label (may be NULL: forward only):    */
/* w_k / B [a_ce (p_d - onehot(xs)) + a_tv p_d (sgn(p_d - p_t) - sum_u p_d,u   */
/* sgn_u)], sgn(0) = 0; grad_s [N] f32 = dL/ds = a_conf w_k / B (c - c*) (may */
/* be NULL).  zd, zt: dtype f32 or bf16, 16-byte aligned rows (V a multiple  */
/* of 8 for bf16, of 4 for f32).  Row sums run in fp32, the loss totals in   */
/* fp64 (added in an unspecified order).  A token outside 0..V-1 writes       */
/* DSPARK_ERR_RANGE to *err and that row's terms are skipped.  No workspace.  */
/* One launch.  Each row is swept three times (twice without grad_z).  For  */
/* V <= ~226K (bf16) or ~113K (f32) a cluster of 8 CTAs holds the row pair   */
/* in shared memory, 1/8 each, and HBM sees it once; for larger V the second */
/* and third sweeps read the row back from L2.                               */
/* ------------------------------------------------------------------------ */
typedef struct {
    int32_t B, gamma, V, dtype;
    const void *zd;          /* [N, V] draft logits, N = B gamma                 */
    const void *zt;          /* [N, V] target logits                             */
    const int32_t *xs;       /* [N] target tokens                                */
    const float *s;          /* [N] confidence logits                            */
    float a_ce, a_tv, a_conf;
    float *row;              /* out [N, 6] or NULL                               */
    double *loss;            /* out [4]                                          */
    float *grad_z;           /* out [N, V] or NULL                               */
    float *grad_s;           /* out [N] or NULL                                  */
    int32_t *err;            /* device error word, or NULL                       */
} dspark_train_loss_args;

DSPARK_API int dspark_train_losses(const dspark_train_loss_args *a, dspark_stream_t stream);

/* ------------------------------------------------------------------------ */
/* The target's pass: operators between the draft and dspark_verify.  The    */
/* pages treat the target model as given; a server that runs it over a paged */
/* key-value cache needs these four next to dspark_build_tags.  Rows are the */
/* flattened batch of dspark_build_tags: the rows of request r are           */
/* row_start[r] .. row_start[r + 1] - 1, row j of a request drafted after    */
/* (some of) the rows before it.  A cache holds n_pages pages of `page`      */
/* tokens; slot s is token s % page of page s / page.  Token t of request r  */
/* sits in page table[r, t / page].  Neither call below synchronises; where  */
/* the device finds an input out of range it writes DSPARK_ERR_RANGE to *err. */
/* ------------------------------------------------------------------------ */

/* The batch map of one cycle.  Request r has len[r] tokens in the cache, gets
 * rows[r] new ones and holds held[r] pages.  With need_r = ceil((len_r +
 * rows_r) / page), pages beyond need_r go back to the stack of free pages
 * (free_list[0 .. *n_free), the top is taken first) and missing ones are taken
 * from it:
 *   given back: in request then page order, the first ends on top;
 *   taken:      in request then page order, from the top, after all returns.
 * A request that is done has len = rows = 0 and gives back all its pages.
 *   row_start [R + 1]  running sum of rows;
 *   slot [N]  where row j of r is stored: token len_r + j;
 *   pos [N]   its position: len_r + j, or with `parents` len_r + its depth;
 *   mask [N, W] 64-bit words, bit j set where row j of the request is the row
 *             itself or one of its ancestors (with `parents` only).
 * parents[i] is the parent's index within the request (< its own), negative
 * for none; any other value is reported and read as none.  Rows at or beyond
 * row_start[R] get slot -1, pos 0, mask 0.  All or nothing: too few free
 * pages, more than max_pages pages, N or n_parents rows or 64 W rows of a
 * request (with `parents`), or a negative size is reported, row_start becomes
 * 0, every slot -1, held_out = held, n_free_out = n_free, and the table and
 * the stack stay as they are.  A page number outside the cache, among a
 * request's held entries or on the stack, is reported by the call that stores
 * rows into it (their slots are -1), gives it back or takes it; it stays what it
 * is and moves like any other.  held_out and n_free_out must not be held and
 * n_free: what the call reads it leaves (but for the table entries and the
 * stack entries that it fills), so a call may be repeated.  R at most
 * DSPARK_MAP_MAX_R, n_pages * page below 2^31.  One launch, no workspace.
 * With trees the caller brings two things that are not here: a verification of
 * tree rows (dspark_verify takes the chains of dspark_build_tags), and the move
 * of the accepted branch's keys and values to the slots of tokens len_r, len_r
 * + 1, ..: a row's slot goes by its place in the batch, the next cycle reads by
 * position. */
#define DSPARK_MAP_MAX_R 8192
typedef struct {
    int32_t R;
    int32_t page;             /* tokens of a page                               */
    int32_t n_pages;          /* pages of the cache = capacity of free_list      */
    int32_t max_pages;        /* columns of the table                           */
    int32_t N;                /* rows that slot, pos and mask hold               */
    int32_t n_parents;        /* entries of parents                             */
    int32_t W;                /* words of a mask row                            */
    const int32_t *len;       /* [R]                                            */
    const int32_t *rows;      /* [R]                                            */
    const int32_t *parents;   /* [n_parents], or NULL for chains                 */
    const int32_t *held;      /* [R]                                            */
    const int32_t *n_free;    /* device scalar                                  */
    int32_t *table;           /* in/out [R, max_pages]                          */
    int32_t *free_list;       /* in/out [n_pages]                               */
    int32_t *held_out;        /* out [R]                                        */
    int32_t *n_free_out;      /* out device scalar                              */
    int32_t *row_start;       /* out [R + 1]                                    */
    int32_t *slot;            /* out [N]                                        */
    int32_t *pos;             /* out [N]                                        */
    uint64_t *mask;           /* out [N, W]: with parents, else NULL             */
    int32_t *err;
} dspark_page_map_args;

DSPARK_API int dspark_page_map(const dspark_page_map_args *a, dspark_stream_t stream);

/* Keys and values of the rows into their slots: k_cache[slot / page, :,
 * slot % page, :] = k[i], likewise v.  A negative slot is skipped, one beyond
 * the cache reported and skipped; of two rows with one slot either may stay.
 * k and v may be views of a fused projection: strides of rows and heads in
 * elements, the D elements of a head adjacent.  One launch, no workspace. */
typedef struct {
    int32_t N, H, D;          /* rows, key-value heads, head size               */
    int32_t page, n_pages, dtype;
    const void *k, *v;        /* [N, H, D]                                      */
    int64_t k_row, k_head, v_row, v_head;  /* strides in elements               */
    const int32_t *slot;      /* [N]                                            */
    void *k_cache, *v_cache;  /* [n_pages, H, page, D]                          */
    int32_t *err;
} dspark_cache_store_args;

DSPARK_API int dspark_cache_store(const dspark_cache_store_args *a, dspark_stream_t stream);

/* Queries, keys and values of the rows on their way into the attention: norms of the
 * queries and keys of each head, their rotation by position, and the append to the
 * cache, in one pass.  For each head x of q and of k, computed in fp32 and rounded once:
 *   with a weight w:  x_d <- x_d w_d / sqrt(mean_d x_d^2 + eps)
 *   rotation by pos[i] freq[j] of pair j < rot / 2, (a, b) = (x_j, x_{j + rot / 2}), or
 *   with `interleaved` (x_{2j}, x_{2j + 1}):  (a cos - b sin, b cos + a sin);
 * elements at and beyond rot stay as they are.  The angle is that of the exact product,
 * whole turns left out before it is rounded, so far positions lose nothing (freq finite
 * and below 2^16, radians per position; pos any 32-bit number).
 * With `slot` keys and values go into the cache as by dspark_cache_store, and a row
 * whose slot is negative, or beyond the cache (reported), is left out altogether: its
 * queries are not written either.  Without, keys go to k_out and v is not looked at.
 * q or k may be NULL (no queries, no keys).  q_out may be q with q's strides, k_out
 * may be k with k's; other overlaps of what is read and written are not allowed.
 * Weights are of the type of the rows.  D at most DSPARK_ATTN_MAX_D, rot even, at most D
 * (0: norms only).  One launch, no workspace. */
typedef struct {
    int32_t N, Hq, H, D;      /* rows, query and key-value heads, head size      */
    int32_t rot, interleaved;
    int32_t page, n_pages, dtype;
    float eps;                /* above 0 with a weight                          */
    const void *q, *k, *v;    /* [N, Hq, D], [N, H, D] twice, D adjacent; q or k may be NULL */
    int64_t q_row, q_head, k_row, k_head, v_row, v_head;  /* strides in elements */
    const int32_t *pos;       /* [N]                                            */
    const float *freq;        /* [rot / 2]                                      */
    const void *q_weight, *k_weight;  /* [D], or NULL: no norm                   */
    const int32_t *slot;      /* [N], or NULL: no cache                          */
    void *q_out;              /* out [N, Hq, D], strides below                   */
    int64_t q_out_row, q_out_head;
    void *k_out;              /* out [N, H, D], strides below, without slot       */
    int64_t k_out_row, k_out_head;
    void *k_cache, *v_cache;  /* [n_pages, H, page, D], with slot                */
    int32_t *err;
} dspark_rope_store_args;

DSPARK_API int dspark_rope_store(const dspark_rope_store_args *a, dspark_stream_t stream);

/* A cache in 4 bits: 4.5 bits per element instead of 16.  16 neighbouring elements of a
 * head share a scale, held as one byte b:
 *   s(b) = 2^(b / 8 - 16) (1 + b % 8 / 8) for b <= 254;  255: the 16 are NaN;
 * an element is n s, n a whole number of -8 .. 7 held as n + 8.  The write takes
 *   s = the s(b) nearest to max |x| / 7 of the 16 (halfway: the even b),
 *   n = x / s rounded to the nearest whole number (halfway: the even one), within -7 .. 7,
 * both exactly, so the bytes do not depend on how they are computed; 16 elements with
 * an infinity or a NaN among them are held as NaN.  Values are off by 1/13 of the largest of
 * their 16 at most, or by 2^-17 where those are all small; beyond 401408 they are held as that.
 * Values written back give the same bytes.  n s has at most 8 significant bits: bf16
 * holds it exactly.
 * A page of a head is one run of page * D * 9 / 16 bytes: the codes of its tokens, D / 2
 * bytes each, then their scales, D / 16 bytes each.  Eight elements e_0 .. e_7 are four
 * bytes, two elements each (low half first): e_0 e_2, e_4 e_6, e_1 e_3, e_5 e_7.
 * D is a multiple of 16 up to DSPARK_ATTN_MAX_D, page * D a multiple of 128, the caches
 * [n_pages, H, page * D * 9 / 16] bytes on a boundary of 16. */

/* Keys and values of the rows into their slots of such caches; slots, strides and the
 * rest as for dspark_cache_store, but that two rows with one slot may leave the codes of one
 * with scales of the other: slots are to differ.  k_out and v_out, given both or neither, get
 * the values that the cache then holds, in the type of the rows (skipped rows are not written).
 * One launch, no workspace. */
typedef struct {
    int32_t N, H, D;          /* rows, key-value heads, head size               */
    int32_t page, n_pages, dtype;  /* dtype of k, v, k_out and v_out             */
    const void *k, *v;        /* [N, H, D]                                      */
    int64_t k_row, k_head, v_row, v_head;  /* strides in elements               */
    const int32_t *slot;      /* [N]                                            */
    uint8_t *k_cache, *v_cache;    /* [n_pages, H, page * D * 9 / 16]            */
    void *k_out, *v_out;      /* out [N, H, D] contiguous, or NULL               */
    int32_t *err;
} dspark_cache_store4_args;

DSPARK_API int dspark_cache_store4(const dspark_cache_store4_args *a, dspark_stream_t stream);

/* Attention of the drafted rows over the cache.  Row j of request r (its own
 * keys and values already stored) sees the tokens t < len[r] and, among the
 * request's new rows, row j' where bit j' of its mask words is set (mask NULL:
 * j' <= j, a chain):
 *   s_t = scale q . k_t,  out = sum_t softmax(s)_t v_t,  lse = ln sum_t exp(s_t).
 * Query head g uses key-value head g / (Hq / H).  What a row does not see has
 * no influence on it, infinities and NaN included; a row that sees nothing
 * gives out = 0, lse = -inf.  Rows at or beyond row_start[R] are not written.
 * A request whose sizes are negative, whose rows pass N (or 64 W with a mask)
 * or whose tokens pass the table is reported and its rows are not written; a
 * page number outside the cache is reported and the rows that see it are then
 * unspecified.  A call in which each SM would walk more than about 2^34 tokens,
 * minutes of work, is reported as DSPARK_ERR_UNSUPPORTED and no row is written.
 * max_rows, the largest number of rows of a request as far as
 * the host knows, only chooses the tile shape.
 * Statistics and sums are fp32.  bf16 with D a multiple of 8 up to 128, pages
 * of a multiple of 8 tokens, a scale that is not negative, and q (its strides
 * too), the caches and out 16-byte aligned, runs on the tensor cores (the softmax
 * weights are rounded to bf16 for the second product: an error of 0.0023 of the
 * output's size where its own rounding makes 0.0017); everything else with D <=
 * DSPARK_ATTN_MAX_D on the CUDA cores in fp32.  With a mask a request
 * has at most DSPARK_ATTN_MAX_TREE rows (W <= 4).  Results do not depend on
 * timing (no atomics on results). */
#define DSPARK_ATTN_MAX_D 256
#define DSPARK_ATTN_MAX_TREE 256
typedef struct {
    int32_t R, N, Hq, H, D;   /* requests, rows of q, query and key-value heads  */
    int32_t page, n_pages, max_pages, dtype;
    int32_t W;                /* words of a mask row                            */
    int32_t max_rows;         /* hint, at least 1                               */
    float scale;
    const void *q;            /* [N, Hq, D], strides below, D adjacent           */
    int64_t q_row, q_head;
    const void *k_cache, *v_cache;  /* [n_pages, H, page, D]                    */
    const int32_t *table;     /* [R, max_pages]                                 */
    const int32_t *len;       /* [R]                                            */
    const int32_t *row_start; /* [R + 1]                                        */
    const uint64_t *mask;     /* [N, W] or NULL                                 */
    void *out;                /* out [N, Hq, D], contiguous                     */
    float *lse;               /* out [N, Hq] or NULL                            */
    int32_t *err;
} dspark_tree_attention_args;

DSPARK_API size_t dspark_tree_attention_workspace_size(const dspark_tree_attention_args *a);
DSPARK_API int dspark_tree_attention(const dspark_tree_attention_args *a, void *ws, dspark_stream_t stream);

/* The same attention over caches in 4 bits (above), k_cache and v_cache [n_pages, H,
 * page * D * 9 / 16] bytes; dtype is that of q and out.  What is said of
 * dspark_tree_attention holds: what a row sees, rows that see nothing, errors, sums in
 * fp32, the bits do not depend on timing.  bf16 with D up to 128, pages whose largest
 * power of two (128 counted at most) is at least 8 and times D a multiple of 256, a
 * scale that is not negative, Hq / H up to 128, and q (its strides too) and out
 * 16-byte aligned, runs on the tensor cores: keys are exact in bf16, values in fp16,
 * and the softmax weights are rounded to fp16 for the second product: by 2^-11 of a weight
 * that is 2^-21 of its row's largest or more, by 2^-32 of the largest below that.  (The
 * second part adds up to 2^-32 n max |v| at most over n tokens that are all so small: less than
 * the rounding of an output of that size up to 2^23 tokens.)  Everything else on
 * the CUDA cores in fp32.  max_rows chooses between kernels and tile shapes, and the
 * workspace's size depends on it: size it with the max_rows of the call. */
DSPARK_API size_t dspark_tree_attention4_workspace_size(const dspark_tree_attention_args *a);
DSPARK_API int dspark_tree_attention4(const dspark_tree_attention_args *a, void *ws, dspark_stream_t stream);

/* Rules on the target's logits before dspark_verify.  For row i, row j of
 * request r, and token v, with c the number of times v stands in the output
 * part of the request's text (hist[r, prompt_len .. hist_len)) and among the
 * tokens tok of the rows j' >= 1 that the row continues, itself included
 * (mask as above; row 0 is the text's last token, counted there already):
 *   z = T[i, v];  if v was said (c > 0, or it stands in hist[r, 0 .. prompt_len)):
 *       z = z > 0 ? z / rep[r] : z * rep[r];
 *   z -= freq[r] c + pres[r] [c > 0];  z += the bias entries of v;
 *   out[i, v] = allow bit v of row allow_row[i] clear ? -inf : z
 * (allow_row[i] < 0: everything allowed; one at or beyond n_allow is reported
 * and read as that).  A row that allows nothing comes out as -inf throughout,
 * which dspark_verify reports.  Computed in fp32, rounded once.
 * Any rule may be absent: hist, tok, rep, freq, pres, bias_start, allow NULL.
 * Several bias entries of one token add in their order.  out may be T.  Rows
 * at or beyond row_start[R] are not written.  Tokens outside the vocabulary
 * are reported and ignored; lengths outside their arrays are reported and cut;
 * a request whose rows pass N (or 64 W with a mask) is reported and skipped.
 * The text and tok of a request without penalties are not read.
 * One launch, no workspace. */
typedef struct {
    int32_t R, N, V, dtype;
    int32_t max_hist;         /* columns of hist                                */
    int32_t n_bias;           /* entries of bias_id and bias_val                */
    int32_t n_allow;          /* rows of allow                                  */
    int32_t W;                /* words of a mask row                            */
    const void *T;            /* [N, V]                                         */
    const int32_t *row_start; /* [R + 1]                                        */
    const int32_t *tok;       /* [N] the rows' tokens, or NULL                   */
    const uint64_t *mask;     /* [N, W] or NULL for chains                      */
    const int32_t *hist;      /* [R, max_hist] or NULL                          */
    const int32_t *hist_len;  /* [R]: with hist                                 */
    const int32_t *prompt_len;/* [R], or NULL: no prompt                        */
    const float *rep, *freq, *pres;  /* [R] or NULL                             */
    const int32_t *bias_start;/* [R + 1] or NULL                                */
    const int32_t *bias_id;   /* [n_bias]                                       */
    const float *bias_val;    /* [n_bias]                                       */
    const uint32_t *allow;    /* [n_allow, ceil(V / 32)] or NULL                */
    const int32_t *allow_row; /* [N]: with allow                                */
    void *out;                /* out [N, V]                                     */
    int32_t *err;
} dspark_logit_rules_args;

DSPARK_API int dspark_logit_rules(const dspark_logit_rules_args *a, dspark_stream_t stream);

/* ------------------------------------------------------------------------ */
/* Helpers                                                                    */
/* ------------------------------------------------------------------------ */
/* Message of the last failing call on this host thread ("" if none). */
DSPARK_API const char *dspark_last_error(void);
/* Library version as major * 10000 + minor * 100 + patch. */
DSPARK_API int dspark_version(void);
/* Self-check of the device-side failure detection (no counterpart in the
 * pages).  Every spin-wait in the tensor-core kernels -- a CTA waiting for the
 * other CTAs of its M-tile, a role waiting on an mbarrier -- gives up after a
 * wall-clock limit, writes DSPARK_ERR_TIMEOUT into the error word and returns.
 * This call runs the same two waits on a condition that nothing satisfies
 * unless the caller set it: mode 0 waits for *flag >= target (a device int32);
 * mode 1 waits on a fresh mbarrier that completes only when target <= 0.
 * limit_ns in (0, 2e9].  After the stream reaches it, *err holds
 * DSPARK_ERR_TIMEOUT if the wait ran out, else it is unchanged. */
DSPARK_API int dspark_wait_selfcheck(const int32_t *flag, int32_t target, int32_t mode, uint64_t limit_ns,
                                     int32_t *err, dspark_stream_t stream);

/* Philox-4x32-10 on the device: out[i][0..3] for counters ctr[i][0..3] and
 * key (seed lo, seed hi), i < n.  Exposes the sampler's generator for checks. */
DSPARK_API int dspark_philox(const uint32_t *ctr, uint64_t seed, int32_t n, uint32_t *out,
                             dspark_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* DSPARK_H */
