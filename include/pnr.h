/*
 * pnr.h -- C ABI of libpnr: parallel-in-time Newton evaluation of a nonlinear RNN
 * on one AMD MI355X (gfx950).
 *
 * The operation.  Given inputs x_1..x_T, an initial state s_0 = h0 and a cell f, the
 * library returns the states s_t = f(s_{t-1}, x_t), t = 1..T.  Instead of stepping
 * through time it unfolds the recurrence into one system of nonlinear equations, one
 * per step (ParaRNN overview page, "Core Idea"; DEER poses the states as the solution
 * of a fixed-point problem: "Towards Scalable and Stable Parallelization of Nonlinear
 * RNNs", abstract) and solves it with Newton iterations (ParaRNN overview, "Newton's
 * Iteration").  One iteration k:
 *   r_t   = f(s_{t-1}^(k), x_t) - s_t^(k)                       residual, every t at once
 *   J_t   = df/ds evaluated at s_{t-1}                          Jacobian (mode below)
 *   rho_k = max_{b,t,i} |r|   (NaN counts as +inf)              two-level reduction
 *           stop if rho_k <= tol or rho_k is not finite          (ParaRNN overview, "Parallel Reduction")
 *   d_t   = J_t d_{t-1} + r_t, d_0 = 0                          block lower-bidiagonal solve,
 *                                                                done as a parallel scan of
 *                                                                affine maps
 *   s^(k+1) = s^(k) + d
 * The converged states equal sequential evaluation ("Parallelizing non-linear
 * sequential models over the sequence length", abstract).  The initial guess is
 * s^(0) = 0.  The Newton loop runs on the device: no host synchronisation happens
 * between iterations; the call synchronises once at its end.
 *
 * Cells (the pages print no equations; these are the readings implemented):
 *   PNR_CELL_GRU        GRU, dense recurrent matrix U [3D, D], gate blocks (r, z, n),
 *                       "linear before reset": n = tanh(gx_n + r*(U_n h + b_hn)),
 *                       h' = (1-z) n + z h.  State size S = D.
 *   PNR_CELL_GRU_DIAG   the same GRU with elementwise recurrent weights u [3, D]
 *                       (diagonal recurrence, as in ParaRNN's GRU adaptation).  S = D.
 *   PNR_CELL_LSTM_DIAG  LSTM with elementwise recurrent weights u [4, D], gate blocks
 *                       (i, f, o, g); state (c, h), S = 2D, c first.
 *
 * Jacobian modes (jac_mode):
 *   PNR_JAC_FULL  exact Jacobian in the cell's own structure: dense D x D (GRU),
 *                 diagonal (GRU_DIAG), one 2x2 block per channel (LSTM_DIAG).
 *   PNR_JAC_DIAG  its diagonal: quasi-Newton ("quasi-DEER"; "Towards Scalable and
 *                 Stable Parallelization of Nonlinear RNNs", abstract).
 *   PNR_JAC_ZERO  no Jacobian: a fixed-point (Picard) sweep.  Test mode.
 * pnr_cell.jac_every = e >= 1 recomputes the Jacobian only on iterations k with
 * k % e == 0 and reuses it otherwise (ParaRNN overview, "Newton's Iteration": the
 * Jacobian recomputed only every few steps); the residual is always fresh.
 *
 * Memory and layout.  Every tensor argument is a DEVICE pointer, row-major, owned by
 * the caller and not retained after the call returns (x and h_out may be NULL when
 * T = 0):
 *   x      [B, T, D_in]            x_dtype
 *   h0     [B, S]                  state_dtype (may be NULL: zeros)
 *   h_out  [B, T, S]               state_dtype; h_out[b, t] = s_{t+1}; h0 excluded
 *   W      [G*D, D_in]             x_dtype     (G = 3 for GRU cells, 4 for LSTM)
 *   U      GRU: [3D, D]; GRU_DIAG: [3, D]; LSTM_DIAG: [4, D]     state_dtype
 *   b_x    [G*D] (NULL = 0)        state_dtype; added to W x
 *   b_h    [G*D] (NULL = 0)        state_dtype; added to the recurrent term (for
 *                                  the GRU candidate gate it sits inside r*(...))
 * The library allocates no device memory: all scratch comes from pnr_cell.workspace,
 * at least pnr_workspace_bytes() bytes, 256-byte aligned.  Work is enqueued on
 * pnr_cell.stream (a hipStream_t; NULL = the default stream).
 *
 * Supported combinations (others return PNR_E_UNSUPPORTED):
 *   GRU:        (x, state) in {(f64, f64), (f32, f32), (bf16, f32)}; D <= 32 with
 *               PNR_JAC_FULL, D <= 64 (fp32 state) or 32 (fp64 state) otherwise
 *   GRU_DIAG,
 *   LSTM_DIAG:  (x, state) in {(f32, f32), (bf16, f32)}
 *
 * Launches.  Each Newton loop is one persistent kernel whose workgroups wait on one
 * another, sized to the device's resident capacity and launched with
 * hipLaunchCooperativeKernel, which guarantees that they are all resident at once, also
 * next to other work on the device; calls with distinct workspaces may therefore run on
 * different streams at the same time.  Every device-side wait is bounded: one that runs
 * out is reported as PNR_E_HIP, never a hang.  Setting PNR_COOPERATIVE=0 in the
 * environment (read once per process) selects ordinary launches, slightly cheaper, for
 * callers that run nothing else on the device while a call is in flight.
 *
 * Errors.  Functions never abort and never print.  Negative return codes mean no
 * result was produced; the text of the last error of the calling thread is
 * available from pnr_last_error().  Argument validation happens before any HIP call.
 */
#ifndef PNR_H
#define PNR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum pnr_cell_kind { PNR_CELL_GRU = 0, PNR_CELL_GRU_DIAG = 1, PNR_CELL_LSTM_DIAG = 2 };
enum pnr_jac_mode { PNR_JAC_FULL = 0, PNR_JAC_DIAG = 1, PNR_JAC_ZERO = 2 };
enum pnr_dtype { PNR_F64 = 0, PNR_F32 = 1, PNR_BF16 = 2 };
enum pnr_status {
  PNR_OK = 0,             /* converged: rho <= tol                                   */
  PNR_NOT_CONVERGED = 1,  /* max_iters updates applied, rho > tol; h_out = last iterate */
  PNR_NONFINITE = 2,      /* a residual was NaN/Inf; h_out = the iterate that made it   */
  PNR_E_INVALID = -1,     /* bad pointer, size, enum or combination                   */
  PNR_E_UNSUPPORTED = -2, /* valid request outside the supported set above            */
  PNR_E_WORKSPACE = -3,   /* workspace NULL, misaligned or smaller than required      */
  PNR_E_HIP = -4          /* a HIP runtime call failed                                */
};

/* Problem description.  All sizes must be >= 1 (T may be 0: nothing to do). */
typedef struct pnr_cell {
  int32_t kind;          /* pnr_cell_kind                                   */
  int32_t D;             /* channels (hidden size)                          */
  int32_t D_in;          /* input features                                  */
  int32_t T;             /* sequence length                                 */
  int32_t B;             /* batch                                           */
  int32_t x_dtype;       /* pnr_dtype of x and W                            */
  int32_t state_dtype;   /* pnr_dtype of h0, h_out, U, b_x, b_h             */
  int32_t jac_every;     /* >= 1                                            */
  void* stream;          /* hipStream_t, NULL = default stream              */
  void* workspace;       /* device scratch, >= pnr_workspace_bytes(...)     */
  size_t workspace_bytes;
} pnr_cell;

typedef struct pnr_params {
  const void* W;    /* [G*D, D_in]        x_dtype                       */
  const void* U;    /* see the cell list   state_dtype                   */
  const void* b_x;  /* [G*D] or NULL       state_dtype                   */
  const void* b_h;  /* [G*D] or NULL       state_dtype                   */
} pnr_params;

/*
 * Scratch bytes pnr_eval needs for this problem and Jacobian mode (0 on invalid
 * input; the reason is in pnr_last_error()).  Pure host arithmetic; no HIP call.
 * The Jacobian itself is never stored: it is rebuilt inside the iteration kernel from
 * the stored states (and, for the dense GRU, from U), so the dense mode needs no
 * O(T D^2) buffer and both Jacobian modes use O(T D) workspace.
 */
size_t pnr_workspace_bytes(const pnr_cell* cell, int jac_mode);

/*
 * Evaluate the RNN by parallel Newton iterations (see the top of this file).
 *   max_iters  >= 0: at most this many Newton updates; 0 returns the initial guess.
 *   tol        stop when rho_k <= tol; tol < 0 never stops early (exactly max_iters
 *              updates are applied).
 * Returns a pnr_status.  On PNR_OK / PNR_NOT_CONVERGED / PNR_NONFINITE, h_out holds
 * the iterate s^(k) whose residual rho_k was checked last, and the call has
 * synchronised the stream.  Thread-safe for distinct workspaces.
 */
int pnr_eval(const pnr_cell* cell, const pnr_params* params, const void* x, const void* h0,
             void* h_out, int max_iters, double tol, int jac_mode);

/*
 * pnr_eval with an adaptive Jacobian refresh, for the diagonal-recurrence cells
 * (PNR_CELL_GRU_DIAG, PNR_CELL_LSTM_DIAG).  The ParaRNN overview ("Newton's Iteration")
 * names recomputing the Jacobian only every few steps among its approximate-Newton
 * strategies; here the residual decides when, by a rule of this library's own: iteration
 * k takes a new Jacobian (at its current iterate) when
 *     k == 0,  or  k - (last refresh) >= cell->jac_every,
 *     or  k >= 2 and rho_{k-1} > refresh_ratio * rho_{k-2},
 * i.e. also when the update before last shrank the max-norm residual by less than the
 * ratio.  The rule looks one update back because the fused pass that evaluates the
 * residual rho_k also takes the Jacobian, before rho_k is known.  refresh_ratio = +inf
 * is pnr_eval's fixed schedule; refresh_ratio = 0 refreshes at every k >= 2.  Arguments,
 * workspace (pnr_workspace_bytes) and results as pnr_eval.  refresh_ratio must be >= 0
 * (PNR_E_INVALID otherwise, NaN included); the dense-U GRU returns PNR_E_UNSUPPORTED.
 */
int pnr_eval_adaptive(const pnr_cell* cell, const pnr_params* params, const void* x, const void* h0,
                      void* h_out, int max_iters, double tol, int jac_mode, double refresh_ratio);

/*
 * pnr_eval without allocation, for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid hipMalloc).  Same
 * arguments, iteration, results and errors as pnr_eval, except that pnr_cell.workspace
 * and workspace_bytes are ignored: the scratch (control words, residual partials,
 * look-back slots, gate pre-activations and iterates) lives in a static device array of
 * PNR_STATIC_SCRATCH_BYTES, one per device, held from the library's first use on that
 * device until the process ends.  A problem whose pnr_workspace_bytes() exceeds that
 * size returns PNR_E_WORKSPACE before any device work (e.g. B=8, T=4096, D=64 fits; the
 * long diagonal workloads do not).  The call makes no hipMalloc/hipFree and no other
 * allocating call; it clears what must start at zero with a kernel on the caller's
 * stream.  Every call on one device shares that device's array: calls that overlap on
 * one device (other threads, other streams) race and must be serialised by the caller.
 * Measurement mode (pnr_profile_enable) does not apply to this entry point.
 */
#define PNR_STATIC_SCRATCH_BYTES ((size_t)64 << 20)
int pnr_eval_static(const pnr_cell* cell, const pnr_params* params, const void* x, const void* h0,
                    void* h_out, int max_iters, double tol, int jac_mode);

/*
 * pnr_eval with a bounded iteration, for the diagonal-recurrence cells (PNR_CELL_GRU_DIAG,
 * PNR_CELL_LSTM_DIAG).  Undamped Newton can diverge ("Towards Scalable and Stable
 * Parallelization of Nonlinear RNNs", summary page, "Problem"): from the zero guess the
 * linearised recurrence of a stiff cell can be so expansive that the step overflows.
 * Here each new iterate is projected onto the box every reachable state lies in -- a
 * safeguard of this library's own, not the pages' damping -- and a component the step
 * made NaN keeps its current value:
 *     GRU_DIAG:   |h_t| <= max(1, |h0|)      (h' is a convex combination of tanh(.) and h)
 *     LSTM_DIAG:  |h_t| <= 1,  |c_t| <= |c0| + t      (t = 1..T)
 * The true states lie inside the box, so the projection never moves them: every property
 * of pnr_eval's iteration that rests on them holds (after k updates the first k states
 * are exact; the fixed point is the sequential trajectory), and iterates that stay inside
 * are pnr_eval's, bit for bit.  Arguments, workspace (pnr_workspace_bytes), jac_mode,
 * jac_every and results as pnr_eval; the dense-U GRU returns PNR_E_UNSUPPORTED.
 */
int pnr_eval_bounded(const pnr_cell* cell, const pnr_params* params, const void* x, const void* h0,
                     void* h_out, int max_iters, double tol, int jac_mode);

/*
 * pnr_eval with a low-rank approximation of the Jacobian, for the GRU with a dense
 * recurrent matrix (PNR_CELL_GRU; D <= 32, the sizes its dense Jacobian supports).  The
 * ParaRNN overview page ("Technical Implementation / Newton's Iteration") names low-rank
 * approximations among the approximate-Newton strategies, with no form; this library's
 * reading keeps the exact Jacobian's structure
 *     J_t = diag(z) + diag(al) U_z + diag(be) U_r + diag(ga) U_n
 * and replaces, in the Jacobian only, each gate block U_g by its best rank-`rank`
 * approximation (truncated singular value decomposition; computed on the device, once
 * per call, from the Gram matrix U_g^T U_g by the cyclic Jacobi eigenvalue method), with
 * U_g's own diagonal restored so that the Jacobian's diagonal stays exact.  The gates and
 * residuals still use U.  rank = D is pnr_eval's dense Jacobian (Newton); rank = 0 its
 * diagonal (quasi-Newton).  rank must be in [0, D] (PNR_E_INVALID).  Other arguments and
 * results as pnr_eval with jac_mode = PNR_JAC_FULL (cell->jac_every honoured).
 * Workspace: pnr_workspace_bytes_lowrank() bytes (pnr_workspace_bytes(cell, FULL) plus the
 * approximated factors, 3 D^2 state elements); 0 = invalid or unsupported request.
 */
size_t pnr_workspace_bytes_lowrank(const pnr_cell* cell, int rank);
int pnr_eval_lowrank(const pnr_cell* cell, const pnr_params* params, const void* x, const void* h0,
                     void* h_out, int max_iters, double tol, int rank);

/* Newton updates applied by the calling thread's last pnr_eval (-1 if it failed before). */
int pnr_iters_used(void);

/* rho of the state returned by the calling thread's last pnr_eval (NaN if none). */
double pnr_last_residual(void);

/*
 * Copies the residual history rho_0..rho_iters of the last pnr_eval (at most max_n
 * values) into host memory `out`; returns how many values that history has.
 */
int pnr_last_residual_history(double* out, int max_n);

/* Text of the calling thread's last error ("" if none).  Valid until the next call. */
const char* pnr_last_error(void);

/*
 * Damped Newton evaluation: ELK / quasi-ELK ("Towards Scalable and Stable
 * Parallelization of Nonlinear RNNs", abstract; summary page, "Approach": a
 * Levenberg-Marquardt trust region whose linear-Gaussian MAP solve is a Kalman filter
 * and smoother; with the diagonal Jacobian, quasi-ELK; "Limitations": the trust-region
 * strength is a hyperparameter).  Same iteration, stopping test and results as
 * pnr_eval, except that the update d minimises
 *     sum_t |d_t - J_t d_{t-1} - r_t|^2 + damping * sum_t |d_t|^2      (d_0 = 0)
 * instead of solving d_t = J_t d_{t-1} + r_t (damping -> 0 gives pnr_eval's step).  With
 * a diagonal J_t this splits into one scalar problem per state component, solved by a
 * Kalman filter (forward scan) and RTS smoother (backward scan).  The step is always
 * taken (fixed damping, no adaptive trust region).
 * Supported, with jac_every = 1 and (x, state) as for pnr_eval:
 *   PNR_CELL_GRU_DIAG, jac_mode PNR_JAC_FULL or PNR_JAC_DIAG (its exact Jacobian is
 *     diagonal, so both are ELK);
 *   PNR_CELL_LSTM_DIAG, jac_mode PNR_JAC_DIAG (quasi-ELK: the diagonal of the 2x2 block,
 *     dc'/dc and dh'/dh, per channel; h_out holds (c, h) as for pnr_eval);
 *   PNR_CELL_GRU (dense U), fp32 state, D <= 64, jac_mode PNR_JAC_DIAG (quasi-ELK: the
 *     diagonal of the dense Jacobian).  Each iteration is a host-driven sequence of
 *     launches (the recurrent GEMM, the cell, one 4-byte read-back of max |r|, the filter
 *     and smoother scans).
 * Others return PNR_E_UNSUPPORTED.  damping must be finite and > 0 (else PNR_E_INVALID).
 * Workspace: pnr_workspace_bytes_damped() bytes (the smoother's per-step gain and
 * offset take 8 bytes per state element more than pnr_eval).
 */
size_t pnr_workspace_bytes_damped(const pnr_cell* cell, int jac_mode);
int pnr_eval_damped(const pnr_cell* cell, const pnr_params* params, const void* x, const void* h0,
                    void* h_out, int max_iters, double tol, int jac_mode, double damping);

/*
 * Chunked evaluation (ParaRNN overview page, "Experimental Results", on long sequences:
 * the memory that stored hidden states take during the Newton iteration is kept in check
 * by chunking, together with gradient checkpointing).  The sequence is cut into consecutive
 * chunks of chunk_len steps (the last may be shorter).  Chunk c is evaluated exactly as
 * pnr_eval (damping == 0) or pnr_eval_damped (damping > 0) evaluates a sequence of its
 * length, with the same max_iters, tol and jac_mode per chunk, and with initial state
 * h0 for the first chunk and, for the others, the returned state at the previous chunk's
 * last step (h_out[b, t0 - 1]).  At convergence the result is the sequential one within
 * the tolerance, as for pnr_eval; the workspace covers one chunk instead of the whole
 * sequence (plus, for B > 1 with more than one chunk, contiguous staging of the chunk's
 * x, boundary state and output, copied on the stream).
 * Arguments and layouts as for pnr_eval / pnr_eval_damped; chunk_len >= 1; damping
 * finite and >= 0.  Results: the worst status over chunks (NONFINITE > NOT_CONVERGED >
 * OK; after a NONFINITE chunk the later chunks are not evaluated and their h_out
 * entries are left as they were); pnr_iters_used() = the sum of the chunks' iterations;
 * pnr_last_residual() = the largest final rho; pnr_last_residual_history() = the chunks'
 * histories one after another; in measurement mode (pnr_profile_enable) the profile
 * record holds sums over the chunks (resid_only: the number of chunks whose last pass
 * only evaluated the residual).  Synchronises the stream before returning.
 * pnr_workspace_bytes_chunked returns 0 for an invalid or unsupported request.
 */
size_t pnr_workspace_bytes_chunked(const pnr_cell* cell, int jac_mode, double damping, int chunk_len);
int pnr_eval_chunked(const pnr_cell* cell, const pnr_params* params, const void* x, const void* h0,
                     void* h_out, int max_iters, double tol, int jac_mode, double damping, int chunk_len);

/*
 * Backward pass: gradients through an evaluated sequence, for training through the
 * parallel evaluation ("Parallelizing non-linear sequential models over the sequence
 * length", abstract; ParaRNN overview, "Newton's Iteration": the block lower-triangular
 * system is solved by backward as well as forward substitution).  Given the states h
 * (e.g. pnr_eval's h_out at convergence) and g = dL/dh, the explicit loss gradient at
 * every state, it computes the gradients of L through the recurrence
 * s_t = f(s_{t-1}, x_t), s_0 = h0, taking h as its solution:
 *     lam_t = g_t + J_{t+1}^T lam_{t+1}   (lam_T = g_T; J exact, not approximated)
 * is run backwards in time as a scan, and each step's lam_t is sent back through the
 * cell's gates to the pre-activations, the recurrent weights and biases, the inputs
 * (through W) and h0.
 * Supported: PNR_CELL_GRU_DIAG and PNR_CELL_LSTM_DIAG (the adjoint is one scan: status
 * PNR_OK, pnr_iters_used() = 0), and PNR_CELL_GRU with D <= 64, whose dense Jacobians
 * couple the channels: there the adjoint system is solved by quasi-Newton refinement
 * ("Towards Scalable and Stable Parallelization of Nonlinear RNNs", abstract: the
 * diagonal approximation, here as the preconditioner of a diagonal scan, with the dense
 * J^T lam of each residual on MFMA) from lam = 0 until max |residual| <= 2e-5 max |g|,
 * checked after every group of 4 iterations, at most 256.  Status PNR_OK,
 * PNR_NOT_CONVERGED (gradients of the last iterate) or PNR_NONFINITE;
 * pnr_iters_used() = refinement updates applied (up to 3 past the passing check),
 * pnr_last_residual_history() = the residuals up to the passing one.  x in {f32, bf16}, state f32; the
 * cell's jac_every is ignored.  Device pointers, caller-owned; each gradient output may
 * be NULL (not computed); all gradients are fp32 and overwritten (not accumulated):
 *   h, grad_h  [B, T, S]   fp32, inputs (S = D, or 2D for the LSTM's (c, h))
 *   grad_x     [B, T, D_in]     grad_W    [G*D, D_in]     grad_U   as U ([3D, D] or [G, D])
 *   grad_b_x   [G*D]            grad_b_h  [G*D]           grad_h0  [B, S]
 * x, h0, params as for pnr_eval (h0 may be NULL: zeros).  Workspace:
 * pnr_workspace_bytes_backward() bytes (0 = invalid or unsupported request).  For the
 * diagonal cells the work is enqueued on cell->stream and the call returns without
 * waiting for it; the dense GRU's refinement reads its residual back every iteration
 * and the call returns with the work still enqueued for the final gradients.  In
 * measurement mode the profile record holds: proj_ms the recomputed gate
 * pre-activations, newton_ms the adjoint (scan kernel, or the refinement loop with its
 * read-backs), out_ms the reductions and gradient GEMMs.
 */
size_t pnr_workspace_bytes_backward(const pnr_cell* cell);
int pnr_backward(const pnr_cell* cell, const pnr_params* params, const void* x, const void* h0,
                 const void* h, const void* grad_h, void* grad_x, void* grad_W, void* grad_U,
                 void* grad_b_x, void* grad_b_h, void* grad_h0);

/*
 * pnr_backward with a choice of Jacobian in the adjoint recursion.  jac_mode PNR_JAC_FULL is
 * pnr_backward (the exact gradients).  PNR_JAC_DIAG is the diagonal approximation in the
 * backward pass ("Towards Scalable and Stable Parallelization of Nonlinear RNNs", summary
 * page, "Measured effects": diagonal Jacobian approximations "including in the backward
 * pass"): the adjoint carries diag(J_{t+1}) lam_{t+1} instead of J_{t+1}^T lam_{t+1}
 * (grad_h0 = diag(J_1) lam_1 likewise), while every step still sends its lam_t back
 * through the cell's gates exactly; the gradients are those approximate adjoints' (exact
 * for PNR_CELL_GRU_DIAG, whose Jacobian is diagonal).  For the dense GRU it is one
 * diagonal scan instead of the refinement: pnr_iters_used() = 1, pnr_last_residual() = 0.
 * Other jac_mode values return PNR_E_INVALID.  Arguments, workspace
 * (pnr_workspace_bytes_backward) and results otherwise as pnr_backward.
 */
int pnr_backward_approx(const pnr_cell* cell, const pnr_params* params, const void* x, const void* h0,
                        const void* h, const void* grad_h, void* grad_x, void* grad_W, void* grad_U,
                        void* grad_b_x, void* grad_b_h, void* grad_h0, int jac_mode);

/*
 * Backward pass over chunks, the gradient-checkpointing half of chunked evaluation
 * (ParaRNN overview page, "Experimental Results": chunking together with gradient
 * checkpointing keeps the memory of long sequences in check).  The sequence is cut into
 * consecutive chunks of chunk_len steps (the last may be shorter), as pnr_eval_chunked
 * cuts it, and the chunks are processed last to first, each by pnr_backward on the
 * chunk's steps, with initial state h0 for the first chunk and h[b, t0 - 1] for the
 * others.  The adjoint crossing a boundary, J^T lam of the later chunk's first step
 * (that chunk's grad_h0), is added to grad_h at the earlier chunk's last step, so that
 * the result is pnr_backward's on the whole sequence up to rounding (and, for the dense
 * GRU, up to each chunk's refinement tolerance).  Weight and bias gradients are summed
 * over chunks; grad_x and the first chunk's grad_h0 are written per chunk.  Arguments,
 * layouts and NULL outputs as for pnr_backward; chunk_len >= 1.  Workspace:
 * pnr_workspace_bytes_backward_chunked() bytes (0 = invalid or unsupported request): one
 * chunk's pnr_backward workspace, the chunk's grad_h, two B x S boundary adjoints, one
 * set of weight-gradient partials and, for B > 1 with more than one chunk, contiguous
 * staging of the chunk's x, h and grad_x.  Results: the worst status over chunks
 * (NONFINITE > NOT_CONVERGED > OK; every chunk is processed); pnr_iters_used() = the
 * sum of the chunks' refinement iterations; pnr_last_residual() = the largest;
 * pnr_last_residual_history() = the chunks' histories, last chunk first; the profile
 * record holds sums over chunks.  Synchronises the stream before returning.
 */
size_t pnr_workspace_bytes_backward_chunked(const pnr_cell* cell, int chunk_len);
int pnr_backward_chunked(const pnr_cell* cell, const pnr_params* params, const void* x,
                         const void* h0, const void* h, const void* grad_h, void* grad_x,
                         void* grad_W, void* grad_U, void* grad_b_x, void* grad_b_h,
                         void* grad_h0, int chunk_len);

/*
 * Standalone linear solve used inside every Newton iteration, exposed for testing
 * the scan on its own: d_t = A_t d_{t-1} + b_t, d_0 = 0 along t, for R independent
 * rows (ParaRNN overview, "Newton's Iteration": forward substitution on the block
 * lower-triangular system).  fp32, device pointers:
 *   kind 1 (diagonal):  A, b, d are [R, T]
 *   kind 2 (2x2 block): A is [R, 4, T] (a00, a01, a10, a11 planes), b and d [R, 2, T]
 * tile_len (0 = library default) sets the per-block tile along T; smaller tiles mean
 * more blocks linked by the decoupled look-back.  workspace as for pnr_eval, size
 * from pnr_scan_workspace_bytes.  Synchronises the stream before returning.
 */
size_t pnr_scan_workspace_bytes(int kind, int R, int T, int tile_len);
int pnr_scan(int kind, int R, int T, const float* A, const float* b, float* d, int tile_len,
             void* workspace, size_t workspace_bytes, void* stream);

/*
 * Per-phase timing of the calling thread's pnr_eval calls, for measurement only.  When
 * enabled (pnr_profile_enable(1)), pnr_eval records a HIP event before and after each
 * of its kernel launches on the caller's stream and, after its final synchronisation,
 * fills the record below (milliseconds of GPU time between those events).  The whole
 * Newton loop is one launch; `passes` counts the fused passes it ran (one per
 * residual evaluated: iters + 1).  Disabled by default; enabling it adds one event pair
 * per launch.  pnr_last_profile returns 0, or -1 if no profiled call completed.
 */
typedef struct pnr_profile {
  double total_ms;       /* first launch to last launch of the call                    */
  double proj_ms;        /* input projection                                            */
  double newton_ms;      /* the persistent Newton-loop kernel                           */
  double out_ms;         /* conversion of the returned iterate to h_out                 */
  int32_t passes;        /* fused passes of the Newton kernel (iters + 1)               */
  int32_t resid_only;    /* 1 if the last pass only evaluated the residual (max_iters)  */
} pnr_profile;

int pnr_profile_enable(int on);
int pnr_last_profile(pnr_profile* out);

/*
 * ---- Sequence mixing next to the recurrent cells ------------------------------------------
 *
 * Linear attention with a decay for each head: the linear recurrence whose state is a
 * matrix, evaluated exactly (no Newton iteration), for each batch row and state head:
 *   S_t = exp(g_t) S_{t-1} + k_t v_t^T          S [D_k, D_v], S_0 = state_in or zeros
 *   o_t = scale * S_t^T q_t
 * H query heads share H_kv state heads in consecutive groups of H / H_kv: query head h reads
 * the state of head h / (H / H_kv); keys, values, decays and states belong to the state head.
 *
 * Layout (device pointers, owned by the caller; elements of `dtype` unless stated):
 *   q          [B, T, H, D_k]         k [B, T, H_kv, D_k]         v [B, T, H_kv, D_v]
 *              with element strides {batch, token, head} of their own in the descriptor (all
 *              >= 0; the last axis contiguous), so slices of one projection need no copy
 *   log_decay  fp32: [H_kv] (PNR_DECAY_HEAD) or [B, T, H_kv] (PNR_DECAY_TOKEN).  A decay
 *              exp(g) <= 1 is meant, g <= 0; g below -104, -inf included, forgets the state
 *              completely (exp(g) is 0 in fp32); g > 0 is taken as it is
 *   state_in, state_out   fp32 [B, H_kv, D_k, D_v]
 *   o          [B, T, H, D_v] contiguous
 *   lens       int32 [B] or NULL: row b has min(max(lens[b], 0), T) tokens.  What lies behind
 *              a row's end is not read (it may hold anything), its outputs and gradients are
 *              zeros, and the state is the one after the row's last token (an empty row hands
 *              state_in on)
 * Supported: dtype PNR_F32 and PNR_BF16, 1 <= D_k, D_v <= 128 (others PNR_E_UNSUPPORTED),
 * H <= 32768 and B H <= 8 million.  Products are accumulated, and states, decays and sums held,
 * in fp32.  With bf16 inputs, states and the decay's gradient are as exact as in fp32, and o and the
 * gradients of q, k and v are rounded once, at the end (inside, scores and the state are held
 * to 2^-17 of each value).
 *
 * A NaN or an infinity in a token reaches what the formulas compute from it, within its row and
 * head: q_t reaches o_t; k_t, v_t and log_decay_t reach o from t on and the state after; k_t, v_t,
 * log_decay_t reach dL/dq from t on, grad_o_t dL/dq_t; q_t and grad_o_t reach dL/dk and dL/dv up to
 * t, log_decay_t those before t, v_t dL/dk_t, k_t dL/dv_t; q_t, grad_o_t and log_decay_t reach the
 * entry state's gradient.  The decay's gradient is summed along the row, and any of them may reach
 * all of it in its row and head.  An infinity may come out as a NaN.
 *
 * Outputs do not overlap inputs, but for the states where it is said.
 *
 * None of these calls waits for the device or allocates: the work is enqueued on
 * desc->stream, so they may be recorded into a HIP graph.  Return PNR_OK or a negative
 * pnr_status.
 */
enum pnr_decay_kind { PNR_DECAY_HEAD = 0, PNR_DECAY_TOKEN = 1 };

typedef struct pnr_linattn {
  int32_t B, T;          /* batch >= 1, tokens >= 0                                    */
  int32_t H, H_kv;       /* query heads, state heads; H_kv divides H                   */
  int32_t D_k, D_v;      /* head sizes of keys and queries, of values and outputs      */
  int32_t dtype;         /* pnr_dtype of q, k, v, o and their gradients                */
  int32_t decay;         /* pnr_decay_kind                                             */
  double scale;
  int64_t q_stride[3], k_stride[3], v_stride[3];   /* elements: batch, token, head      */
  const int32_t* lens;   /* [B] or NULL                                                */
  void* stream;          /* hipStream_t, NULL = default stream                         */
  void* workspace;       /* device scratch, 256-byte aligned                           */
  size_t workspace_bytes;
} pnr_linattn;

/*
 * All tokens of a sequence at once (a prompt, or the forward pass of a layer), in chunks
 * along time.  state_in may be NULL (zeros), state_out NULL (not wanted); they may be the
 * same buffer.  Workspace: pnr_linattn_workspace_bytes() bytes (0: none needed, or an invalid
 * request, which pnr_linattn_forward then names; pure host arithmetic).  With T = 0 only
 * state_out is written.
 */
size_t pnr_linattn_workspace_bytes(const pnr_linattn* desc);
int pnr_linattn_forward(const pnr_linattn* desc, const void* q, const void* k, const void* v,
                        const float* log_decay, const float* state_in, void* o, float* state_out);

/*
 * One token for each of B running requests (T is not read; the token strides and lens are
 * not either): q [B, H, D_k], k [B, H_kv, D_k], v [B, H_kv, D_v], log_decay [H_kv] or
 * [B, H_kv], o [B, H, D_v] contiguous.  state_in and state_out are pools
 * [n_slots, H_kv, D_k, D_v]; request b's state is read from and written to slot slots[b]
 * (int32 [B]), or slot b when slots is NULL (n_slots >= B then).  A slot outside
 * [0, n_slots) marks an idle row: its o is zeros and no state is touched.  No two rows may
 * name the same slot.  state_in and state_out may be the same buffer (updated in place);
 * otherwise slots that no row names keep what they held in state_out.  No workspace.
 */
int pnr_linattn_step(const pnr_linattn* desc, const void* q, const void* k, const void* v,
                     const float* log_decay, const float* state_in, const int32_t* slots, int n_slots,
                     void* o, float* state_out);

/*
 * Gradients of a loss through pnr_linattn_forward, given grad_o = dL/do (contiguous, as o)
 * and grad_state_out = dL/dstate_out (NULL: zeros):
 *   grad_q, grad_k, grad_v   dtype, contiguous [B, T, heads, D]; keys' and values' gradients
 *                            are summed over the query heads that share them
 *   grad_log_decay           fp32, as log_decay ([H_kv]: summed over rows and tokens, in an
 *                            order that does not change from call to call)
 *   grad_state_in            fp32 [B, H_kv, D_k, D_v]
 * Every gradient output may be NULL (not wanted); all are overwritten.  The states are
 * recomputed from the inputs.  Workspace: pnr_linattn_workspace_bytes_backward() bytes
 * (0: invalid request).
 */
size_t pnr_linattn_workspace_bytes_backward(const pnr_linattn* desc);
int pnr_linattn_backward(const pnr_linattn* desc, const void* q, const void* k, const void* v,
                         const float* log_decay, const float* state_in, const void* grad_o,
                         const float* grad_state_out, void* grad_q, void* grad_k, void* grad_v,
                         float* grad_log_decay, float* grad_state_in);

/*
 * Group norm with an activation, channels last.  x [N, L, C] contiguous; C is split into
 * `groups` runs of C / groups channels, and each (row n, group) is normalised over its L
 * positions and its channels (biased variance):
 *   z = (x - mean) / sqrt(var + eps) * weight + bias
 *   y = act(z), or with a gate  y = z * act(gate)
 * L = 1 normalises every token by heads (the norm after linear attention, N = B T); L > 1
 * a whole map or sequence.  weight, bias fp32 [C], or both NULL; gate as x or NULL; lens int32
 * [N] or NULL: only the first min(max(lens[n], 0), L) positions of row n belong to it: the
 * others are not read, and y and the gradients are zeros there (a row with none has mean 0
 * and rstd 1 / sqrt(eps)).  L <= 2^30, C <= 2^26, N * groups <= 2e9, or 16 million where L > 1 or a
 * group has more than 512 channels.  mean, rstd: fp32 [N, groups] outputs, kept for the backward
 * pass (NULL: not wanted).  dtype PNR_F32 or PNR_BF16 (x, gate, y and their gradients).  The calls
 * wait for nothing and allocate nothing.  Workspace sizes: 0 means none needed, or an
 * invalid request, which the call then names.
 */
enum pnr_act { PNR_ACT_NONE = 0, PNR_ACT_SILU = 1, PNR_ACT_GELU = 2 /* tanh form */ };

typedef struct pnr_norm {
  int32_t N, L, C, groups;   /* N, C >= 1, L >= 0, groups divides C                    */
  int32_t dtype, act;        /* pnr_dtype, pnr_act                                     */
  double eps;                /* > 0                                                    */
  const int32_t* lens;       /* [N] or NULL                                            */
  void* stream;
  void* workspace;           /* device scratch, 256-byte aligned                       */
  size_t workspace_bytes;
} pnr_norm;

size_t pnr_groupnorm_workspace_bytes(const pnr_norm* desc);
int pnr_groupnorm(const pnr_norm* desc, const void* x, const float* weight, const float* bias,
                  const void* gate, void* y, float* mean, float* rstd);

/*
 * Gradients through pnr_groupnorm, given grad_y and the forward call's mean and rstd:
 * grad_x, grad_gate (dtype, as x), grad_weight, grad_bias (fp32 [C], summed over N and L in
 * an order that does not change from call to call).  Each may be NULL; grad_gate needs a
 * gate, grad_weight a weight.  eps is not read.  All are overwritten.
 */
size_t pnr_groupnorm_workspace_bytes_backward(const pnr_norm* desc);
int pnr_groupnorm_backward(const pnr_norm* desc, const void* x, const float* weight, const float* bias,
                           const void* gate, const void* grad_y, const float* mean, const float* rstd,
                           void* grad_x, float* grad_weight, float* grad_bias, void* grad_gate);

/*
 * Selective scan: the recurrence of a state space layer whose step width, input and read-out
 * depend on the token.  For each batch row, channel e of E and state n of N, with g = e / (E / G)
 * the channel's group:
 *   delta = softplus(dt + dt_bias), or dt + dt_bias
 *   h_t = exp(delta_t A) h_{t-1} + delta_t u_t B_t      h_0 = state_in or zeros
 *   y_t = (sum over n of C_t h_t) + D u_t               and  y_t silu(z_t)  with a gate z
 *
 * Layout (device pointers, owned by the caller; elements of `dtype` unless stated):
 *   u, dt, z    [B, T, E] with element strides {batch, token}; z may be NULL (no gate; its strides are
 *               checked all the same, zeros will do)
 *   B, C        [B, T, G, N] with element strides {batch, token, group}
 *               (strides >= 0, the last axis contiguous: slices of projections need no copy)
 *   A           fp32 [E, N], finite; a decay is meant (A <= 0, delta >= 0), others are taken as they are
 *               (the gradients of states that grow may be NaN, zero ones too, from a stretch of tokens
 *               on whose sum of delta A is beyond fp32's exponent)
 *   D, dt_bias  fp32 [E] or NULL (zeros)
 *   state_in, state_out   fp32 [B, E, N]
 *   y           [B, T, E] contiguous
 *   lens        int32 [B] or NULL: row b has min(max(lens[b], 0), T) tokens.  What lies behind a
 *               row's end is not read, its outputs and gradients are zeros, and the state is the one
 *               after the row's last token (an empty row hands state_in on)
 * Supported: dtype PNR_F32 and PNR_BF16, 1 <= N <= 64 (others PNR_E_UNSUPPORTED), G divides E,
 * E <= 2^20, T <= 2^30, G ceil(E / G / 64) <= 65536, B times that <= 4 million; token strides of u, dt and z up to 2^23
 * (others PNR_E_UNSUPPORTED).  Everything inside is fp32; outputs of `dtype` are rounded once, at the
 * end.
 *
 * A NaN or an infinity in a token reaches what the formulas compute from it, within its row: u, dt,
 * z and grad_y their channel, B and C the channels of their group; forwards in time for y and the
 * states, backwards too for the gradients; grad_B and grad_C at a token are sums over the group's
 * channels.  An infinity may come out as a NaN.
 *
 * Outputs do not overlap inputs, but for the states where it is said.  None of these calls waits
 * for the device or allocates: the work is enqueued on desc->stream, so they may be recorded into a
 * HIP graph.  Return PNR_OK or a negative pnr_status.
 */
typedef struct pnr_selscan {
  int32_t B, T;          /* batch >= 1, tokens >= 0                                    */
  int32_t E, N, G;       /* channels, states of a channel, groups of B and C            */
  int32_t dtype;         /* pnr_dtype of u, dt, z, B, C, y and their gradients         */
  int32_t softplus;      /* 1: delta = softplus(dt + dt_bias); 0: dt + dt_bias          */
  int64_t u_stride[2], dt_stride[2], z_stride[2];  /* elements: batch, token            */
  int64_t B_stride[3], C_stride[3];                /* elements: batch, token, group     */
  const int32_t* lens;   /* [B] or NULL                                                */
  void* stream;          /* hipStream_t, NULL = default stream                         */
  void* workspace;       /* device scratch, 256-byte aligned                           */
  size_t workspace_bytes;
} pnr_selscan;

/*
 * All tokens of a sequence at once.  state_in may be NULL (zeros), state_out NULL (not wanted);
 * they may be the same buffer.  Workspace: pnr_selscan_workspace_bytes() bytes for the same desc (whether
 * lens is given counts; 0: none needed, or
 * an invalid request, which pnr_selscan_forward then names; pure host arithmetic).  With T = 0
 * only state_out is written.
 */
size_t pnr_selscan_workspace_bytes(const pnr_selscan* desc);
int pnr_selscan_forward(const pnr_selscan* desc, const void* u, const void* dt, const float* A,
                        const void* Bt, const void* Ct, const float* D, const void* z,
                        const float* dt_bias, const float* state_in, void* y, float* state_out);

/*
 * One token for each of B running requests (T, the token strides and lens are not read): u, dt, z
 * [B, E], B and C [B, G, N], y [B, E] contiguous.  state_in and state_out are pools
 * [n_slots, E, N]; request b's state is read from and written to slot slots[b] (int32 [B]), or slot
 * b when slots is NULL (n_slots >= B then).  A slot outside [0, n_slots) marks an idle row: its y is
 * zeros and no state is touched.  No two rows may name the same slot.  state_in and state_out may
 * be the same buffer (updated in place); otherwise slots that no row names keep what they held in
 * state_out.  No workspace.
 */
int pnr_selscan_step(const pnr_selscan* desc, const void* u, const void* dt, const float* A,
                     const void* Bt, const void* Ct, const float* D, const void* z,
                     const float* dt_bias, const float* state_in, const int32_t* slots, int n_slots,
                     void* y, float* state_out);

/*
 * Gradients of a loss through pnr_selscan_forward, given grad_y (contiguous, as y) and
 * grad_state_out = dL/dstate_out (NULL: zeros):
 *   grad_u, grad_dt, grad_z   dtype, [B, T, E] contiguous
 *   grad_B, grad_C            dtype, [B, T, G, N] contiguous, summed over the group's channels
 *   grad_A                    fp32 [E, N]; grad_D, grad_dt_bias fp32 [E]; summed over rows and tokens
 *   grad_state_in             fp32 [B, E, N]
 * Every gradient output may be NULL (not wanted; grad_z needs a z); all are overwritten.  Sums
 * are taken in an order that does not change from call to call.  The states are recomputed.
 * Workspace: pnr_selscan_workspace_bytes_backward() bytes (0: invalid request).
 */
size_t pnr_selscan_workspace_bytes_backward(const pnr_selscan* desc);
int pnr_selscan_backward(const pnr_selscan* desc, const void* u, const void* dt, const float* A,
                         const void* Bt, const void* Ct, const float* D, const void* z,
                         const float* dt_bias, const float* state_in, const void* grad_y,
                         const float* grad_state_out, void* grad_u, void* grad_dt, float* grad_A,
                         void* grad_B, void* grad_C, float* grad_D, void* grad_z,
                         float* grad_dt_bias, float* grad_state_in);

/*
 * Activations kept in 8 bits until the backward pass reads them.  x [B, T, E] in `dtype` with
 * element strides {batch, token} >= 0; 32 consecutive channels (the last block of a token may be
 * shorter) share the least power of two 2^e, e >= -126, with |x| <= 127 * 2^e, and
 *   codes      int8 [B, T, E]                   x / 2^e rounded to nearest, ties to even (at e = 122
 *                                               at most 63: 2^128 is infinite)
 *   exponents  uint8 [B, T, ceil(E / 32)]       e + 127, or 255 where the block holds a NaN or
 *                                               an infinity: all of it reads back as NaN
 * pnr_checkpoint_unpack writes code * 2^e to x [B, T, E] contiguous (exact in bf16 and in fp32;
 * x_stride is not read).  E <= 2^20, T <= 2^30, B T ceil(E / 32) <= 2^40.  No workspace; the calls
 * wait for nothing and allocate nothing.
 */
typedef struct pnr_checkpoint {
  int32_t B, T, E;       /* B, E >= 1, T >= 0                                          */
  int32_t dtype;         /* PNR_F32 or PNR_BF16                                        */
  int64_t x_stride[2];   /* elements: batch, token                                     */
  void* stream;
} pnr_checkpoint;

int pnr_checkpoint_pack(const pnr_checkpoint* desc, const void* x, int8_t* codes, uint8_t* exponents);
int pnr_checkpoint_unpack(const pnr_checkpoint* desc, const int8_t* codes, const uint8_t* exponents, void* x);

/*
 * Causal convolution along time, each channel by itself, W taps:
 *   p_t = bias + sum over j < W of weight[e, j] x_{t - W + 1 + j},   y = act(p)
 * x [B, T, E] with element strides {batch, token} (>= 0, channels contiguous), or, with
 * `exponents`, the codes [B, T, E] that pnr_checkpoint_pack wrote (x_stride is not used then, only
 * checked to be >= 0).
 * weight fp32 [E, W], bias fp32 [E] or NULL (zeros).  state_in [B, W - 1, E] are the inputs before
 * the first (NULL: zeros), state_out [B, W - 1, E] the last W - 1 inputs of each row, state_in's
 * among them where the row is shorter (NULL: not wanted).  y, the states and the gradients that
 * are not fp32 are of `dtype` and contiguous.  lens int32 [B] or NULL: row b has
 * min(max(lens[b], 0), T) tokens; what lies behind is not read, y and gradients are zeros there.
 * dtype PNR_F32 or PNR_BF16, act PNR_ACT_NONE or PNR_ACT_SILU, 1 <= W <= 8 (others
 * PNR_E_UNSUPPORTED), E <= 2^20, T <= 2^30, B (E / 64 + 1) <= 4 million.  Sums are fp32, outputs
 * rounded once.  A NaN or an infinity reaches what the formulas compute from it, within its channel
 * and row; an infinity may come out as a NaN.  Outputs do not overlap inputs.  The calls wait for nothing and allocate nothing.
 */
typedef struct pnr_conv {
  int32_t B, T, E, W;    /* B, E, W >= 1, T >= 0                                       */
  int32_t dtype, act;    /* pnr_dtype, pnr_act                                         */
  int64_t x_stride[2];   /* elements: batch, token                                     */
  const int32_t* lens;   /* [B] or NULL                                                */
  void* stream;
  void* workspace;       /* device scratch, 256-byte aligned                           */
  size_t workspace_bytes;
} pnr_conv;

int pnr_conv_forward(const pnr_conv* desc, const void* x, const uint8_t* exponents, const float* weight,
                     const float* bias, const void* state_in, void* y, void* state_out);

/*
 * One token for each of B requests (T, the token stride and lens are not read): x and y [B, E],
 * state_in and state_out pools [n_slots, W - 1, E], slots and idle rows as in pnr_selscan_step;
 * the pools may be the same buffer, and NULL with a single tap, which has no state.
 */
int pnr_conv_step(const pnr_conv* desc, const void* x, const float* weight, const float* bias,
                  const void* state_in, const int32_t* slots, int n_slots, void* y, void* state_out);

/*
 * Gradients through pnr_conv_forward of these arguments, given grad_y [B, T, E] and grad_state_out
 * (NULL: zeros): grad_x [B, T, E] and grad_state_in in `dtype`; grad_weight fp32 [E, W] and
 * grad_bias fp32 [E], summed over rows and tokens in an order that does not change from call to
 * call.  Each may be NULL; all are overwritten.  Workspace:
 * pnr_conv_workspace_bytes_backward() bytes (0: invalid request).
 */
size_t pnr_conv_workspace_bytes_backward(const pnr_conv* desc);
int pnr_conv_backward(const pnr_conv* desc, const void* x, const uint8_t* exponents, const float* weight,
                      const float* bias, const void* state_in, const void* grad_y,
                      const void* grad_state_out, void* grad_x, float* grad_weight, float* grad_bias,
                      void* grad_state_in);

#ifdef __cplusplus
}
#endif

#endif /* PNR_H */
