/*
 * pararnn.h — C ABI of libpararnn.so: the ParaRNN / DEER parallel-in-time
 * Newton solve of ParaGRU and ParaLSTM, and its adjoint, on MI355X (gfx950).
 *
 * The method ("Параллельность RNN?", forpes.ru, section 1; voguetech.ru
 * ParaRNN article, "Что именно сделали технически"):
 *   - the T hidden states s_1..s_T of a sequence are the unknowns of the
 *     residual r_t = s_t - f(s_{t-1}, x_t) = 0, whose unique zero is the
 *     ordinary sequential trajectory (§1.1);
 *   - Newton's method solves it: J(s) ds = -r(s), s <- s + ds (§1.2);
 *   - J is block-bidiagonal (identity blocks, -df/ds(s_{t-1}) below), so
 *     each Newton system is the linear recurrence
 *     ds_t = A_t ds_{t-1} - r_t, A_t = df/ds(s_{t-1}) (§1.3, level 1),
 *     which is associative and is solved by a parallel scan of affine maps
 *     (§1.3, level 2);
 *   - for ParaGRU the local Jacobian A_t is diagonal, for ParaLSTM 2x2
 *     block diagonal per channel (ParaRNN article, item 3), so every
 *     channel (b, d) is an independent 1- or 2-dimensional problem.
 * The per-step transition is compiled into the kernels (the fully fused
 * tier of the ParaRNN article, "Три уровня производительности", item 3):
 *   ParaGRU  z = sig(a_z h + u_z), r = sig(a_r h + u_r),
 *            c = tanh(a_c (r h) + u_c),  h' = (1 - z) h + z c
 *   ParaLSTM i, f, o = sig(a_* h + u_*), g = tanh(a_g h + u_g),
 *            c' = f c + i g,  h' = o tanh(c')
 * u_* are the precomputed input projections W x_t + b (one plane per gate),
 * a_* the diagonal recurrent weights.
 *
 * Conventions for every entry point
 *   - Memory: every array pointer is a DEVICE pointer (HBM), owned by the
 *     caller; the library never allocates, frees or synchronises.  All work
 *     is enqueued on `stream` (a hipStream_t, NULL = default stream) and the
 *     call returns before it completes.  Outputs must not alias inputs.
 *     A call enqueues kernel launches only (per-launch state is cleared by
 *     a kernel, not by a memset), so it can be captured into a HIP graph;
 *     a captured call keeps its workspace, and two replays that overlap in
 *     time must not share one.  A call may be several launches that meet in
 *     its workspace, so neither may calls on different streams, nor threads
 *     whose calls on one stream are not kept apart by a lock.
 *   - Layout: per-time-step planes are indexed (b, d, t); element offset of
 *     (b, d, t) = b*stride_b + d*stride_d + t*stride_t.  Planes of `u` (and
 *     of `du`) use u_stride_*; state, gradient and lambda planes use
 *     s_stride_*.  The fast layout is channel-major [B][D][T] (stride_t = 1):
 *     a lane's steps are contiguous and load as 16-byte vectors.  Any other
 *     layout whose elements do not overlap is accepted, e.g. time-major
 *     [B][T][D] (stride_t = D, stride_d = 1, as a [B][T][G*D] projection
 *     gives per gate with stride_t = G*D).  The solves, the adjoint and the
 *     scan stage such planes channel-major in the workspace when it is at
 *     least pararnn_workspace_bytes(...) / pararnn_scan_workspace_bytes(...)
 *     (which count that room), run there and copy the results back; with a
 *     smaller workspace (the channel-major size), and always in the
 *     sequential call, each step is gathered with its own 4-byte load
 *     instead.  Results are bitwise the same either way.
 *     pararnn_project writes channel-major planes directly.  Initial states are dense [B][D]; diagonal
 *     weights are dense [G][D] float32 in gate order (GRU: z, r, c;
 *     LSTM: i, f, g, o).  LSTM state order is (c, h).
 *   - Errors: arguments are checked on the host before any HIP call; a bad
 *     argument returns PARARNN_ERR_INVALID / _UNSUPPORTED / _WORKSPACE and
 *     enqueues nothing.  A HIP launch error returns PARARNN_ERR_HIP.
 *     Non-convergence is not an error: it is reported in pararnn_info_t.
 *   - Determinism: results are bitwise reproducible run to run (no
 *     floating-point atomics; reductions run in a fixed order).
 */
#ifndef PARARNN_H
#define PARARNN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    PARARNN_OK = 0,
    PARARNN_ERR_INVALID = 1,     /* null pointer, size < 0, bad stride      */
    PARARNN_ERR_UNSUPPORTED = 2, /* valid request this build does not serve */
    PARARNN_ERR_WORKSPACE = 3,   /* workspace NULL or smaller than needed   */
    PARARNN_ERR_HIP = 4,         /* the HIP runtime reported a launch error */
    PARARNN_ERR_SCRATCH = 5      /* needs more than the static scratch      */
} pararnn_status_t;

typedef enum { PARARNN_F32 = 0, PARARNN_BF16 = 1 } pararnn_dtype_t;
typedef enum { PARARNN_GRU = 0, PARARNN_LSTM = 1 } pararnn_cell_t;

typedef struct {
    int64_t B, T, D;                 /* batch rows, time steps, channels     */
    int64_t u_stride_b, u_stride_d;  /* elements, every u / du plane         */
    int64_t s_stride_b, s_stride_d;  /* elements, every state/grad plane     */
    int64_t u_stride_t, s_stride_t;  /* elements between steps (1: [B][D][T]) */
} pararnn_shape_t;

typedef struct {
    /* A channel (or, for long sequences, a time block of it) stops once the
     * largest |r_t| over its steps and state components is < tol and every
     * earlier time block of the channel has stopped; NaN never counts as
     * converged.  At most max_iters Newton updates are applied; the final
     * residual is always evaluated. */
    float tol;
    int32_t max_iters;        /* >= 0                                          */
    int32_t steps_per_lane;   /* K: 0 = automatic, else 1, 2, 4, 8, 16, or 32
                                 (ParaGRU forward solve with W = 1 or 2 only)  */
    int32_t waves_per_block;  /* W: 0 = automatic, else 1, 2, 4 or 8; one
                                 workgroup covers 64 * K * W time steps       */
    int32_t init_from_output; /* 1: Newton starts from the values already in
                                 the output planes; 0: from s = 0             */
} pararnn_newton_t;

/* Written on the device by the solve (pass a device pointer, or NULL): each
 * work unit stores its own final max|r| and update count in the workspace,
 * and a one-workgroup pass after the solve folds them into this record. */
typedef struct {
    int32_t iters;        /* max Newton updates applied, over channels       */
    int32_t converged;    /* 1 iff every channel stopped with max|r| < tol    */
    float max_abs_res;    /* max over channels of the final max|r_t|          */
    int32_t nan_seen;     /* 1 if any final residual was NaN                  */
    int64_t iters_sum;    /* sum over work units of updates applied           */
    int64_t units;        /* work units = channels x time blocks              */
} pararnn_info_t;

/* Bytes of device workspace pararnn_solve_* / pararnn_adjoint need for this
 * problem and tiling (0 is possible).  Returns 0 on a bad argument too; the
 * solve itself reports the error.  For the adjoint pass adjoint = 1.
 * For a solve the figure counts the time-block hand-off (several blocks per
 * channel that run side by side, i.e. fewer than 1024 channels; with more, a
 * channel's blocks are solved one after the other inside one workgroup and
 * need none), 8 bytes per work unit for the convergence records an info
 * record is folded from, and the staging room of planes that are not
 * time-contiguous; a solve without an info record, on time-contiguous
 * planes with one block per channel, runs with no workspace at all. */
size_t pararnn_workspace_bytes(pararnn_cell_t cell, const pararnn_shape_t *shape,
                               const pararnn_newton_t *opt, int adjoint);

/*
 * ParaGRU forward solve.
 *   u[3]   : gate planes (z, r, c), [B][D][T], dtype u_dtype (F32 or BF16)
 *   a      : [3][D] float32 diagonal recurrent weights
 *   h0     : [B][D] float32 initial state s_0 (given, not solved for)
 *   h      : [B][D][T] float32 output, the converged states s_1..s_T
 *            (also the Newton start if opt->init_from_output)
 *   info   : device pararnn_info_t or NULL
 *   ws     : device workspace of ws_bytes >= pararnn_workspace_bytes(...)
 * Residual, Jacobian, scan and convergence test run in one kernel; the
 * states stay on chip across Newton iterations.
 */
pararnn_status_t pararnn_solve_gru(const pararnn_shape_t *shape, const void *const u[3],
                                   pararnn_dtype_t u_dtype, const float *a,
                                   const float *h0, float *h,
                                   const pararnn_newton_t *opt, pararnn_info_t *info,
                                   void *ws, size_t ws_bytes, void *stream);

/*
 * ParaLSTM forward solve.  u[4] gate planes (i, f, g, o); a [4][D];
 * c0, h0 [B][D]; outputs c, h [B][D][T].  Jacobians are 2x2 per channel.
 */
pararnn_status_t pararnn_solve_lstm(const pararnn_shape_t *shape, const void *const u[4],
                                    pararnn_dtype_t u_dtype, const float *a,
                                    const float *c0, const float *h0, float *c, float *h,
                                    const pararnn_newton_t *opt, pararnn_info_t *info,
                                    void *ws, size_t ws_bytes, void *stream);

/*
 * Adjoint (backward pass) of a converged solve, for the loss
 * L = sum_t <dL/ds_t, s_t>.  The adjoint lam_t = dL/ds_t (total) solves the
 * transposed block-bidiagonal system of §1.3, i.e. the reverse-time linear
 * recurrence lam_t = g_t + A_{t+1}^T lam_{t+1}, lam_{T+1} = 0, with
 * A_{t+1} = df/ds at (s_t, u_{t+1}); it is computed by a reverse parallel
 * scan, then the gate gradients follow elementwise.
 *   cell   : PARARNN_GRU (S = 1 state, G = 3 gates) or PARARNN_LSTM (2, 4)
 *   u      : G gate planes as for the solve (dtype u_dtype)
 *   a      : [G][D]
 *   s0     : S pointers to [B][D] initial states (LSTM order c, h)
 *   s      : S pointers to [B][D][T] converged states s_1..s_T
 *   gs     : S pointers to [B][D][T] upstream gradients dL/ds_t; an entry
 *            may be NULL, meaning zero (e.g. dL/dc_t for an LSTM)
 *   gs_end : NULL, or S pointers to [B][D] (an entry may be NULL = zero):
 *            a gradient added to dL/ds_T at the last step — what a
 *            continuation of the sequence sends back, i.e. the ds0 of the
 *            adjoint of the next time chunk (A_{T+1}^T lam_{T+1} of the
 *            uncut recurrence), so a sequence cut into chunks is
 *            differentiated chunk by chunk, last chunk first
 *   du     : G pointers to [B][D][T] float32 outputs dL/du (u_stride_*)
 *   da     : [G][D] float32 output dL/da (summed over batch and time)
 *   da_accumulate : 0: da = the sum; 1: da += the sum (chunk by chunk)
 *   ds0    : S pointers to [B][D] float32 outputs dL/ds_0
 *   lam    : NULL, or S pointers to [B][D][T] float32 outputs lam_t
 *   opt    : only steps_per_lane / waves_per_block are read (may be NULL)
 *   ws     : workspace (per-block da partials and carries)
 */
pararnn_status_t pararnn_adjoint(pararnn_cell_t cell, const pararnn_shape_t *shape,
                                 const void *const *u, pararnn_dtype_t u_dtype,
                                 const float *a, const float *const *s0,
                                 const float *const *s, const float *const *gs,
                                 const float *const *gs_end, float *const *du, float *da,
                                 int32_t da_accumulate, float *const *ds0,
                                 float *const *lam, const pararnn_newton_t *opt,
                                 void *ws, size_t ws_bytes, void *stream);

/*
 * The linear recurrence of a Newton iteration on its own, for callers that
 * assemble (A_t, b_t) themselves: "Параллельность RNN?" (forpes.ru), §1.3,
 * level 1 (forward substitution) solved as in level 2 (associative scan of
 * affine maps); the "parallel reduction" tier of the voguetech.ru ParaRNN
 * article ("Три уровня производительности", item 2).  Per channel (b, d):
 *   reverse = 0:  x_t = A_t x_{t-1} + b_t,  t = 1..T,  x_0 given
 *   reverse = 1:  x_t = A_t x_{t+1} + b_t,  t = T..1,  x_{T+1} given
 *   state_size : 1 (A_t scalar) or 2 (A_t a 2x2 block)
 *   A          : state_size^2 planes [B][D][T] float32 (u_stride_*), 2x2 blocks
 *                row-major (a00, a01, a10, a11)
 *   b          : state_size planes [B][D][T] float32 (u_stride_*)
 *   x0         : NULL (boundary value zero) or state_size pointers to [B][D]
 *   x          : state_size planes [B][D][T] float32 out (s_stride_*)
 *   opt        : only steps_per_lane / waves_per_block are read (may be NULL)
 *   ws         : pararnn_scan_workspace_bytes(...) bytes (0 is possible)
 * Same conventions as above: device pointers, caller's stream, no
 * allocation, argument checks before any HIP call.
 */
size_t pararnn_scan_workspace_bytes(int32_t state_size, const pararnn_shape_t *shape,
                                    const pararnn_newton_t *opt);
pararnn_status_t pararnn_scan(int32_t state_size, const pararnn_shape_t *shape,
                              const float *const *A, const float *const *b,
                              const float *const *x0, float *const *x, int32_t reverse,
                              const pararnn_newton_t *opt, void *ws, size_t ws_bytes,
                              void *stream);

/*
 * Step-by-step application of the recurrence, one lane per channel:
 * s_t = f(s_{t-1}, u_t) for t = 1..T from the given s_0 — the sequential
 * evaluation whose result the Newton solve reaches ("Параллельность RNN?",
 * forpes.ru, §1.1: the trajectory is the unique zero of the residual) and
 * the baseline of the pages' parallel-vs-sequential speed-up (voguetech.ru
 * ParaRNN article, "Что именно сделали технически").  Its time is T times
 * one step's dependency-chain latency, nearly independent of the number of
 * channels until they fill the device, so for many channels and moderate T
 * it can beat the Newton solve; for few channels and long T it cannot.
 *   cell, shape, u, u_dtype, a : as for pararnn_solve_gru / _lstm
 *   s0 : S pointers to [B][D] initial states (LSTM order c, h)
 *   s  : S pointers to [B][D][T] float32 outputs (s_stride_*)
 * Same conventions: device pointers, caller's stream, no allocation, no
 * workspace, arguments checked before any HIP call.
 */
pararnn_status_t pararnn_sequential(pararnn_cell_t cell, const pararnn_shape_t *shape,
                                    const void *const *u, pararnn_dtype_t u_dtype,
                                    const float *a, const float *const *s0, float *const *s,
                                    void *stream);

/*
 * Input projection: u = W x + b for every time step, the dense product that
 * precedes the recurrence (the cells take u_t = W x_t + b as precomputed
 * projections: voguetech.ru ParaRNN article, "Что именно сделали
 * технически", item 3).  Per batch row b:
 *     u[b][m][t] = sum_k W[m][k] x[b][t][k] + bias[m],  m < M, t < T, k < I
 * Written channel-major with time contiguous, so for M = G*D the rows of
 * gate g form that gate's [B][D][T] plane for the solves (plane g starts at
 * u + g*D*u_stride_m; u_stride_b, u_stride_m are its strides).
 *   x    : bfloat16, x[b][t][k] at b*x_stride_b + t*x_stride_t + k
 *   w    : bfloat16, W[m][k] at m*w_stride_m + k
 *   bias : float32 [M], or NULL (no bias)
 *   u    : u_dtype (PARARNN_F32, or PARARNN_BF16 rounded to nearest even),
 *          u[b][m][t] at b*u_stride_b + m*u_stride_m + t
 * Products of bf16 values are exact in fp32 and accumulate in fp32 on the
 * matrix cores.  Device pointers, caller's stream, no allocation; arguments
 * checked before any HIP call (sizes >= 0, strides large enough that rows
 * do not overlap).
 */
typedef struct {
    int64_t B, T, I, M;
    int64_t x_stride_b, x_stride_t;
    int64_t w_stride_m;
    int64_t u_stride_b, u_stride_m;
} pararnn_proj_shape_t;

pararnn_status_t pararnn_project(const pararnn_proj_shape_t *shape, const void *x,
                                 const void *w, const float *bias, void *u,
                                 pararnn_dtype_t u_dtype, void *stream);

/*
 * pararnn_solve_gru without a workspace argument, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc).  Arguments, results and errors are those
 * of pararnn_solve_gru; the workspace (time-block hand-off, convergence
 * records of the info record, staging of planes that are not
 * time-contiguous when it fits) comes from an array inside the library of
 * PARARNN_STATIC_SCRATCH_BYTES per GPU, held from the first call on that GPU
 * until the process ends.  A problem that needs more returns
 * PARARNN_ERR_SCRATCH before any HIP call (planes that are not
 * time-contiguous and do not fit are read step by step instead of staged).
 * The call allocates nothing and frees nothing; the first call on a device
 * looks up the array's device address (the caller's stream must belong to
 * the current device, else PARARNN_ERR_INVALID).  Every call on one GPU
 * shares that GPU's array and leaves its contents behind (the solve clears
 * what must start at zero with a kernel): calls whose executions overlap on
 * one GPU (different streams, concurrent graph replays) race and must be
 * serialised by the caller.
 */
#define PARARNN_STATIC_SCRATCH_BYTES (32u << 20)
pararnn_status_t pararnn_solve_gru_noalloc(const pararnn_shape_t *shape, const void *const u[3],
                                           pararnn_dtype_t u_dtype, const float *a,
                                           const float *h0, float *h,
                                           const pararnn_newton_t *opt, pararnn_info_t *info,
                                           void *stream);

/*
 * Gated linear recurrence: the linear-time companion of the ParaGRU cell,
 * whose decay depends on the input but not on the state, so that one scan
 * solves it exactly.  Per channel (b, d), with gate planes u = (u_r, u_i, u_x):
 *     l_t = -power softplus(lam_d) sig(u_r),   a_t = exp(l_t)
 *     h_t = k_t a_t h_{t-1} + sqrt(1 - a_t^2) sig(u_i) u_x
 * k_t = 0 where resets[b][t] is non-zero (the first step of a new document in
 * a packed row: nothing of the state before it is kept, also if that state is
 * not finite, and no gradient of the document goes back past it), else 1.
 *   shape   : u strides for u and du, s strides for h and gh
 *   u       : 3 planes [B][D][T], dtype u_dtype (F32 or BF16)
 *   lam     : [D] float32;  power : > 0, finite
 *   h0      : [B][D] float32, or NULL (zero)
 *   resets  : [B][T] bytes, dense, or NULL (none)
 *   h       : [B][D][T] float32 out, the states h_1..h_T
 *   h_last  : [B][D] float32 out, h_T (h_0 when T = 0), or NULL
 *   ws      : pararnn_gated_workspace_bytes(shape, 0) bytes (0 is possible)
 * The same conventions as the solves: device pointers, caller's stream, no
 * allocation, argument checks before any HIP call, any plane layout whose
 * elements do not overlap.  Channel-major planes run with a lane's steps
 * side by side, any other layout with a lane per channel.
 */
size_t pararnn_gated_workspace_bytes(const pararnn_shape_t *shape, int adjoint);
pararnn_status_t pararnn_gated_scan(const pararnn_shape_t *shape, const void *const u[3],
                                    pararnn_dtype_t u_dtype, const float *lam, float power,
                                    const float *h0, const uint8_t *resets, float *h,
                                    float *h_last, void *ws, size_t ws_bytes, void *stream);
/*
 * Its backward pass, for L = sum_t <gh_t, h_t> + <gh_last, h_T>.
 *   h       : the states of the forward pass
 *   gh      : [B][D][T] float32 (s strides), or NULL (zero)
 *   gh_last : [B][D] float32, or NULL (zero)
 *   du      : 3 planes out, dtype u_dtype, u strides
 *   dlam    : [D] float32 out, summed over batch and time in a fixed order
 *   dh0     : [B][D] float32 out, or NULL
 *   ws      : pararnn_gated_workspace_bytes(shape, 1) bytes
 */
pararnn_status_t pararnn_gated_scan_adjoint(const pararnn_shape_t *shape, const void *const u[3],
                                            pararnn_dtype_t u_dtype, const float *lam, float power,
                                            const float *h0, const uint8_t *resets,
                                            const float *h, const float *gh,
                                            const float *gh_last, void *const du[3], float *dlam,
                                            float *dh0, void *ws, size_t ws_bytes, void *stream);
/*
 * One step of it for B requests, their states in a pool: for every row b
 * with 0 <= slots[b] < pool,
 *     states[slots[b]] = out[b] = a states[slots[b]] + sqrt(1 - a^2) sig(u_i) u_x
 * A row whose slot lies outside the pool (-1, say) is idle: its output is
 * zero and no state changes.  The slots of live rows must be distinct.
 *   u      : 3 row blocks [B][D], dtype u_dtype, rows u_stride_b elements apart
 *   slots  : [B] int32, or NULL (row b has slot b)
 *   states : [pool][D] float32, updated in place;  out : [B][D] float32
 */
pararnn_status_t pararnn_gated_step(int64_t B, int64_t D, const void *const u[3],
                                    pararnn_dtype_t u_dtype, int64_t u_stride_b, const float *lam,
                                    float power, const int32_t *slots, float *states, int64_t pool,
                                    float *out, void *stream);

/*
 * Block boundary: what stands between one recurrent block and the next.  Per
 * step (b, t), over its D channels,
 *     v = h silu(gate)                               (v = h without a gate)
 *     y = x + scale (v rstd_post) w_post,            rstd_post = 1/sqrt(mean v^2 + eps)
 *     z = (y rstd_pre) w_pre,                        rstd_pre  = 1/sqrt(mean y^2 + eps)
 * h and gate are [B][D][T]-indexed planes (channel-major from the solves and
 * the projection); x, y, z are time-major [B][T][D] with the channels
 * contiguous, as pararnn_project reads them, so the change of layout between
 * the two happens on the way.
 *   h      : float32, or NULL: y = x, and only the second norm is computed
 *            (the first norm of a model); gate and w_post are not read then
 *   gate   : gate_dtype, or NULL (no gate)
 *   x, y   : x_dtype (share their strides); y may be NULL if h is
 *   w_post, w_pre : [D] float32
 *   scale  : finite;  eps : > 0, finite
 *   z      : z_dtype
 *   rstd   : [2][B][T] float32 out (rstd_post, rstd_pre), or NULL; without h
 *            its first half is not written
 */
typedef struct {
    int64_t B, T, D;
    int64_t h_stride_b, h_stride_d, h_stride_t; /* h, dh                    */
    int64_t g_stride_b, g_stride_d, g_stride_t; /* gate, dgate              */
    int64_t x_stride_b, x_stride_t;             /* x, y, gy, dx             */
    int64_t z_stride_b, z_stride_t;             /* z, gz                    */
} pararnn_block_shape_t;

pararnn_status_t pararnn_block_norm(const pararnn_block_shape_t *shape, const float *h,
                                    const void *gate, pararnn_dtype_t gate_dtype, const void *x,
                                    pararnn_dtype_t x_dtype, const float *w_post,
                                    const float *w_pre, float scale, float eps, void *y, void *z,
                                    pararnn_dtype_t z_dtype, float *rstd, void *stream);
/*
 * Its backward pass from the gradients gy of y and gz of z (either may be
 * NULL, meaning zero) and the forward's rstd.
 *   dh, dgate : h's and gate's strides; dgate in gate_dtype, NULL without a
 *               gate; both NULL without h
 *   dx        : x_dtype, x's strides
 *   dw_post   : [D] float32 out, NULL without h;  dw_pre : [D] float32 out;
 *               both summed over batch and time in a fixed order
 *   ws        : pararnn_block_workspace_bytes(shape) bytes
 */
size_t pararnn_block_workspace_bytes(const pararnn_block_shape_t *shape);
pararnn_status_t pararnn_block_norm_adjoint(const pararnn_block_shape_t *shape, const float *h,
                                            const void *gate, pararnn_dtype_t gate_dtype,
                                            const void *x, pararnn_dtype_t x_dtype,
                                            const float *w_post, const float *w_pre, float scale,
                                            const float *rstd, const void *gy, const void *gz,
                                            pararnn_dtype_t z_dtype, float *dh, void *dgate,
                                            void *dx, float *dw_post, float *dw_pre, void *ws,
                                            size_t ws_bytes, void *stream);

/*
 * Scores of given tokens from logits: with p = softmax(scale logits[n]),
 *     logprob[n] = log p[tokens[n]],  lse[n] = log sum exp(scale logits[n]),
 *     entropy[n] = -sum p log p,
 * and the `top` most likely tokens with their log probabilities, most likely
 * first, the lower index first among equals.
 *   logits  : [N][V], dtype F32 or BF16, rows row_stride >= V elements apart
 *   tokens  : [N] int64.  A negative token is not scored: logprob 0.  One
 *             past the vocabulary scores NaN.
 *   top     : 0 .. PARARNN_TOP_MAX
 *   scale   : inverse temperature, > 0, finite
 *   logprob, entropy, lse : [N] float32 out (entropy, lse may be NULL)
 *   top_index, top_logprob : [N][top] int64 / float32 out
 * A logit of -inf is a masked token: probability 0, never an alternative.
 * Alternatives a row does not have are index -1 with log probability -inf.
 * A row whose tokens are all masked has lse -inf, entropy 0 and logprob -inf.
 * A NaN or +inf among a row's logits makes its log probabilities NaN; NaN
 * logits are no alternatives.
 *   ws      : pararnn_logprobs_workspace_bytes(...) bytes (0 is possible)
 */
#define PARARNN_TOP_MAX 64
size_t pararnn_logprobs_workspace_bytes(int64_t N, int64_t V, int32_t top);
pararnn_status_t pararnn_token_logprobs(int64_t N, int64_t V, const void *logits,
                                        pararnn_dtype_t dtype, int64_t row_stride,
                                        const int64_t *tokens, int32_t top, float scale,
                                        float *logprob, float *entropy, float *lse,
                                        int64_t *top_index, float *top_logprob, void *ws,
                                        size_t ws_bytes, void *stream);
/*
 * Its gradient for the logits,
 *     dlogits_j = scale (g_logprob ([j = token] - p_j) + g_lse p_j
 *                        - g_entropy p_j (log p_j + entropy)),
 * from the forward's lse and entropy; g_* are [N] float32 or NULL (zero).  A
 * token that is not scored takes no g_logprob; a masked logit's p_j is 0; the
 * gradient of a row whose tokens are all masked is zero.  p comes from lse, a
 * float32: it is within half an ulp of |lse| of itself, which for logits beyond
 * 1e5 is a percent and for a row of the type's lowest value all of it (give
 * such a row no gradient).  dlogits has the
 * dtype of the logits, rows d_stride elements apart, and may be the logits'
 * own memory (same stride).
 */
pararnn_status_t pararnn_token_logprobs_adjoint(int64_t N, int64_t V, const void *logits,
                                                pararnn_dtype_t dtype, int64_t row_stride,
                                                const int64_t *tokens, float scale,
                                                const float *lse, const float *entropy,
                                                const float *g_logprob, const float *g_entropy,
                                                const float *g_lse, void *dlogits,
                                                int64_t d_stride, void *stream);

/*
 * Gated delta rule: a recurrence whose state is a matrix for each head, which
 * stores values under keys.  Per row b and value head h (key head h Hk / Hv:
 * Hv is a multiple of Hk, neighbouring value heads share a key head),
 *     S <- a S,  w = beta (v - k^T S),  S <- S + k w^T,  o = scale q^T S
 * with S [dk][dv] and a = exp(log_decay).  The state keeps its size where
 * |k|^2 beta <= 2 and a <= 1: keys of unit length and beta in [0, 2], say.
 *   q, k    : [B][Hk][dk][T]-indexed, v [B][Hv][dv][T], dtype F32 or BF16
 *   beta, log_decay : [B][Hv][T]-indexed float32; log_decay NULL: no decay
 *   h0      : [B][Hv][dk][dv] float32, dense, or NULL (zero)
 *   resets  : [B][T] bytes, dense, or NULL: non-zero at the first step of a
 *             new document.  It keeps nothing of the state before it, also if
 *             that is not finite, and no gradient goes back past it.  A log
 *             decay below -104, whose exponential is 0 in float32, does the
 *             same in its head; the gradient for it is 0.
 *   o       : [B][Hv][dv][T]-indexed float32 out
 *   last    : [B][Hv][dk][dv] float32 out, the last state (h0 at T = 0), or NULL
 *   ws      : pararnn_delta_workspace_bytes(shape, dtype, 0) bytes
 * Strides are of (b, h, d, t), and of (b, h, t) for the gates; inputs may
 * repeat elements (stride 0), outputs not.  The fast layout has the steps side
 * by side (stride 1 along t).  With the channels side by side, as a linear
 * layer leaves them, a bfloat16 scan takes 1.5 times as long and its backward
 * pass 1.15 times, and where dk is no multiple of 8 2.5 and 1.55 times; float32
 * 1.0 to 1.15 times.  dk is at most PARARNN_DELTA_KEY_MAX.
 *
 * Numbers: with float32 inputs all products are float32's.  With bfloat16
 * inputs what is multiplied with them (states, what the steps write, the
 * gradients) is rounded to two bfloat16, 16 bits and more, so that float32
 * results are about 5e-6 off in norm, not 3e-7; pass float32 copies where that
 * matters.  A number that is not finite can make the steps before it NaN, too,
 * of its document in its chunk of 64 steps (float32: 32), not those of earlier
 * chunks or of other documents: padding whose content is undefined belongs into
 * a document of its own.
 *
 * Workspace: forward 12 KB (float32: 4 KB) for a head's chunk of 64 (32)
 * steps.  Backward twice that and the states before and behind each chunk, and
 * two numbers for each value: 8 bytes times (K + chunk) times dv, K being dk
 * rounded up to 64, 128 or 256 and dv to a multiple of 32.  That is 0.9 GB for
 * B = 8, T = 4096, 8 heads of 128 x 128 in bfloat16, and 22 GB for B = 4, T =
 * 16384, 32 heads of 256 x 256.  Rows of the batch do not meet: calls for some
 * of them need as much less.
 */
#define PARARNN_DELTA_KEY_MAX 256
typedef struct {
    int64_t B, T, Hk, Hv, dk, dv;
    int64_t q_stride[4], k_stride[4], v_stride[4];
    int64_t o_stride[4];    /* o, and its gradient */
    int64_t gate_stride[3]; /* beta and log_decay  */
} pararnn_delta_shape_t;

size_t pararnn_delta_workspace_bytes(const pararnn_delta_shape_t *shape, pararnn_dtype_t dtype,
                                     int adjoint);
pararnn_status_t pararnn_delta_scan(const pararnn_delta_shape_t *shape, const void *q,
                                    const void *k, const void *v, pararnn_dtype_t dtype,
                                    const float *beta, const float *log_decay, const float *h0,
                                    const uint8_t *resets, float scale, float *o, float *last,
                                    void *ws, size_t ws_bytes, void *stream);
/*
 * Its backward pass, for L = sum <go, o> + <g_last, last>.
 *   go      : at o_stride (elements may repeat), or NULL (zero)
 *   g_last  : dense, or NULL (zero)
 *   dq, dk, dv : dtype, their own strides; heads that share a key head are
 *             summed in a fixed order
 *   dbeta, dlog_decay : [B][Hv][T] float32, dense (dlog_decay NULL without one)
 *   dh0     : [B][Hv][dk][dv] float32, or NULL
 *   ws      : pararnn_delta_workspace_bytes(shape, dtype, 1) bytes
 */
typedef struct {
    void *dq, *dk, *dv;
    int64_t dq_stride[4], dk_stride[4], dv_stride[4];
    float *dbeta, *dlog_decay, *dh0;
} pararnn_delta_grads_t;

pararnn_status_t pararnn_delta_scan_adjoint(const pararnn_delta_shape_t *shape, const void *q,
                                            const void *k, const void *v, pararnn_dtype_t dtype,
                                            const float *beta, const float *log_decay,
                                            const float *h0, const uint8_t *resets, float scale,
                                            const float *go, const float *g_last,
                                            const pararnn_delta_grads_t *grads, void *ws,
                                            size_t ws_bytes, void *stream);
/*
 * One step of it for B requests, their states in a pool, updated in place
 * (shape->T is 1, its time strides are not read): as for the gated recurrence,
 * a row whose slot lies outside the pool is idle, its output zero, and the
 * slots of live rows must be distinct.
 *   slots  : [B] int32, or NULL (row b has slot b)
 *   states : [pool][Hv][dk][dv] float32;  o : [B][Hv][dv]-indexed float32 out
 */
pararnn_status_t pararnn_delta_step(const pararnn_delta_shape_t *shape, const void *q,
                                    const void *k, const void *v, pararnn_dtype_t dtype,
                                    const float *beta, const float *log_decay,
                                    const int32_t *slots, float *states, int64_t pool, float scale,
                                    float *o, void *stream);

/*
 * Distillation from a teacher's most likely tokens, as pararnn_token_logprobs
 * lists them.  Per row, with p_e = exp(top_logprob[e]) the teacher's
 * probability of the token top_index[e], P their sum, and q = softmax(scale
 * logits) the student's,
 *     loss = sum_e p_e (log p_e - log q[top_index[e]])
 *            + r (log r - log q_rest)                     where tail is not 0,
 * r = 1 - P (taken as 0 below 1e-6, what rounding can leave of a full list) and
 * q_rest the student's probability of all tokens that are not listed.
 *   logits  : [N][V], dtype F32 or BF16, rows row_stride >= V elements apart
 *   top_index, top_logprob : [N][top] int64 / float32, top at most
 *             PARARNN_DISTILL_MAX.  A negative index is no entry.  A token
 *             that is listed twice counts once in q_rest, each time in the
 *             sums over e.  An index past the vocabulary makes the loss NaN.
 *   scale   : inverse temperature, > 0, finite
 *   loss, lse, log_rest : [N] float32 out (lse of scale logits; log q_rest)
 * A row without an entry has loss 0 and gradient 0.  A listed token of p_e > 0
 * whose logit is -inf makes the loss inf, and so does an r > 0 where the
 * student allows no other token.
 *   ws      : pararnn_distill_workspace_bytes(N, V) bytes (0 is possible)
 */
#define PARARNN_DISTILL_MAX 1024
size_t pararnn_distill_workspace_bytes(int64_t N, int64_t V);
pararnn_status_t pararnn_distill_top(int64_t N, int64_t V, const void *logits,
                                     pararnn_dtype_t dtype, int64_t row_stride,
                                     const int64_t *top_index, const float *top_logprob,
                                     int32_t top, int tail, float scale, float *loss, float *lse,
                                     float *log_rest, void *ws, size_t ws_bytes, void *stream);
/*
 * Its gradient for the logits,
 *     g_loss scale (q_j (P + r) - p_j)            for listed tokens,
 *     g_loss scale q_j (P + r - r / q_rest)       for the others
 * (r = 0 without a tail), from the forward's lse and log_rest.  A row whose
 * logits are all -inf has gradient 0, one with an index past the vocabulary NaN.
 * dlogits has the dtype of the logits, rows d_stride elements apart, and may be
 * the logits' own memory (same stride).
 */
pararnn_status_t pararnn_distill_top_adjoint(int64_t N, int64_t V, const void *logits,
                                             pararnn_dtype_t dtype, int64_t row_stride,
                                             const int64_t *top_index, const float *top_logprob,
                                             int32_t top, int tail, float scale, const float *lse,
                                             const float *log_rest, const float *g_loss,
                                             void *dlogits, int64_t d_stride, void *stream);

/*
 * What is done to logits before a token is sampled from them.  Per row n and
 * token j, in this order, in float32 and rounded once:
 *   - j in the row's history (the first lengths[n] of its tokens): x / repetition
 *     where x > 0, else x repetition;
 *   - j there c > 0 times from place prompt[n] on: x - frequency c - presence;
 *   - j in the row's bias list: x + its value, the last one if it is listed twice;
 *   - bit j of the row's mask 0: -inf.
 *   logits, out : [N][V], dtype F32 or BF16; out may be the logits (same stride)
 *   tokens  : [N][length] int64, rows token_stride apart; tokens outside the
 *             vocabulary (negative ones, say) are passed over
 *   lengths, prompt : [N] int32 or NULL (length; 0)
 *   repetition, presence, frequency : [N] float32 or NULL (1; 0; 0)
 *   bias_index, bias_value : [N][biases] int64 / float32; indices outside the
 *             vocabulary are passed over
 *   allowed : [allowed_count][allowed_stride] words of 32 bits, token j the bit
 *             j % 32 of word j / 32, or NULL; allowed_rows [N] int32 the mask of
 *             each row (one that is not there: none), or NULL (row n has mask n)
 */
typedef struct {
    const int64_t *tokens;
    int64_t token_stride, length;
    const int32_t *lengths, *prompt;
    const float *repetition, *presence, *frequency;
    const int64_t *bias_index;
    const float *bias_value;
    int64_t biases;
    const int32_t *allowed;
    int64_t allowed_stride, allowed_count;
    const int32_t *allowed_rows;
} pararnn_adjust_t;

pararnn_status_t pararnn_adjust_logits(int64_t N, int64_t V, const void *logits,
                                       pararnn_dtype_t dtype, int64_t row_stride,
                                       const pararnn_adjust_t *how, void *out, int64_t out_stride,
                                       void *stream);

/* Static description of a status code. */
const char *pararnn_status_string(pararnn_status_t status);

/* Tiling the library would use for this problem: K steps per lane, W waves
 * per workgroup, and time blocks per channel (1 = whole channel in one
 * workgroup).  Returns PARARNN_OK or the same error a solve would return. */
pararnn_status_t pararnn_plan(pararnn_cell_t cell, const pararnn_shape_t *shape,
                              const pararnn_newton_t *opt, int adjoint,
                              int32_t *steps_per_lane, int32_t *waves_per_block,
                              int64_t *time_blocks);

#ifdef __cplusplus
}
#endif

#endif /* PARARNN_H */
