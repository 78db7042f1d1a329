/*
 * ss2d.h -- C ABI of libss2d.so, the MI355X (gfx950) SS2D forward operator.
 *
 * The operator (VMamba's 2D selective scan, "SS2D"):
 *   1. Cross-scan: a (B, D, H, W) feature map is read along four routes, each a sequence of
 *      length L = H * W over every channel d:
 *        route 0  row-major              pi_0(t) = t
 *        route 1  row-major, reversed    pi_1(t) = L - 1 - t
 *        route 2  column-major           pi_2(t) = (t mod H) * W + floor(t / H)
 *        route 3  column-major, reversed pi_3(t) = pi_2(L - 1 - t)
 *      (pi_k(t) is the raster index h * W + w visited at step t.)  Sources: the "Vision
 *      Mamba" explainer (dileepadev), CrossScanModule listing and its prose; the Chinese
 *      VMamba article (mhpn.cn), section 1, cross_scan; the VMamba review (nubint.ai),
 *      "Proposed method" (Cross-Scan Module with four routes).
 *   2. Selective scan on every route k and channel d, from a zero state h (N values):
 *        delta_t = softplus(dt_raw[b,k,d,t] + dt_bias[k,d])
 *        A_n     = -exp(A_log[k,d,n])
 *        h_n     = exp(delta_t * A_n) * h_n + delta_t * Bs[b,k,n,t] * x[b,d,pi_k(t)]
 *        y_k,t   = sum_n Cs[b,k,n,t] * h_n + Ds[k,d] * x[b,d,pi_k(t)]
 *      Sources: the explainer's SelectiveSSM listing (softplus of the dt projection with
 *      its bias, A = -exp(A_log), the exp discretisation of A and delta * B for B, zero
 *      initial state, output after the update, D skip term); the Vim summary (aipaper.cc),
 *      section 4.1 (discrete recurrence); one independent parameter set per route (the
 *      explainer's four SSMs).
 *   3. Cross-merge: y[b,d,pi_k(t)] = sum over k of y_k,t, each route's permutation undone
 *      and the routes summed (the explainer's CrossScanModule: inverse flips and
 *      transposes, outputs summed).
 *   ss1d_bidir_forward is the K = 2 case over a 1D sequence: route 0 forward, route 1 over
 *   the reversed sequence, summed after undoing the reversal (Vim summary, section 4.3).
 *
 * Precision: x, dt_raw, Bs, Cs and y share one data type (fp32 or bfloat16); A_log, Ds and
 * dt_bias are always fp32.  delta, the state h and every sum are fp32; y is rounded once
 * (round to nearest even for bfloat16).  The state never leaves the chip.
 *
 * Layouts (contiguous, row-major, device pointers, caller-owned):
 *   x, y      (B, D, H, W)          [ss1d_bidir_forward: (B, D, L)]
 *   dt_raw    (B, K, D, L)          in the scan order of route k (index t = step t)
 *   Bs, Cs    (B, K, N, L)          in the scan order of route k
 *   A_log     (K, D, N)  fp32
 *   Ds        (K, D)     fp32
 *   dt_bias   (K, D)     fp32
 * with K = 4 for ss2d_forward and K = 2 for ss1d_bidir_forward.
 *
 * Conventions shared by every entry point:
 *   - Inputs are read only.  y is written in full (no pre-zeroing needed) and must not
 *     overlap any input (z included, for the entry points that take it).
 *   - All arguments are validated before anything is enqueued; on an error nothing is
 *     launched and y is untouched.  Nothing is printed and no exception crosses the ABI.
 *   - The call is asynchronous on `stream` (a hipStream_t; NULL is the default stream).
 *     Faults inside the kernels surface at the caller's next synchronisation.
 *   - Calls keep no data between them (the training pair below hands its state over in a
 *     caller-owned buffer).  Internal scratch (a transposed copy of x, per-route
 *     fp32 partial outputs, chunk carries) is allocated on `stream` from a stream-ordered
 *     memory pool of the library's own (one per device, created at the first call on that
 *     device, held until the process ends) and released on `stream` in the same call.  The
 *     pool keeps freed blocks for later calls (its release threshold is unlimited), so the
 *     device memory of the largest scratch used so far stays reserved by the library until
 *     ss2d_scratch_trim hands it back; the device's default pool and its attributes are not
 *     touched.  Under stream capture the
 *     scratch becomes an allocation node of the graph (no synchronisation, copy or memset
 *     is enqueued, so every entry point can be captured; verified for one live graph at a
 *     time).  The sequence operators take the caller's scratch there instead, see below.
 *   - Results are deterministic: identical inputs, shapes and device give bitwise identical
 *     y (no atomics; the routes are summed in the fixed order 0, 1, 2, 3).
 *   - B == 0 or D == 0 is a valid empty call: it returns SS2D_OK, launches nothing and reads
 *     no pointer.
 *   - Thread safety: calls from several host threads are safe; calls on different streams
 *     run independently.
 */
#ifndef SS2D_H
#define SS2D_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The ss1d_delta_*, ss2d_norm_*, ss1d_scan_*, ss1d_conv_* and ss2d_group_norm_* entry points came
 * within version 12: a client that may meet an older library of that version looks for them by name. */
#define SS2D_ABI_VERSION 12

/* Status codes returned by every entry point. */
#define SS2D_OK 0
#define SS2D_ERR_NULL 1        /* a required pointer is NULL                                */
#define SS2D_ERR_SHAPE 2       /* a negative dimension, H/W/L/N < 1, or a size beyond the
                                  kernels' index range (L >= 2^30, or any tensor with
                                  2^62 elements or more)                                   */
#define SS2D_ERR_UNSUPPORTED 3 /* N not in {1, 2, 4, 8, 16, 32}, an unknown dtype or flag, or
                                  a size an entry point documents as unsupported          */
#define SS2D_ERR_ALIGN 4       /* a pointer not aligned to its element size                 */
#define SS2D_ERR_HIP 5         /* a HIP runtime call failed (see ss2d_last_hip_error)       */
#define SS2D_ERR_ALIAS 6       /* an output overlaps an input (or another output)            */
#define SS2D_ERR_SCRATCH 7     /* ss2d_forward_noalloc: the call needs more scratch than
                                  SS2D_NOALLOC_SCRATCH_BYTES; _ws entry points: it needs more
                                  than is given, or none is given under stream capture     */

/* Data types of x, dt_raw, Bs, Cs and y. */
#define SS2D_F32 0
#define SS2D_BF16 1

/* Four-route SS2D forward.  x, y: (B, D, H, W); dt_raw: (B, 4, D, L); Bs, Cs: (B, 4, N, L);
 * A_log: (4, D, N); Ds, dt_bias: (4, D); L = H * W.  dtype is SS2D_F32 or SS2D_BF16.
 * Returns SS2D_OK or one of the SS2D_ERR_* codes above. */
int ss2d_forward(const void *x, const void *dt_raw, const float *A_log, const void *Bs,
                 const void *Cs, const float *Ds, const float *dt_bias, void *y, int64_t B,
                 int64_t D, int64_t H, int64_t W, int64_t N, int dtype, void *stream);

/* Bidirectional 1D selective scan forward (Vim block: forward route plus reversed route,
 * summed).  x, y: (B, D, L); dt_raw: (B, 2, D, L); Bs, Cs: (B, 2, N, L); A_log: (2, D, N);
 * Ds, dt_bias: (2, D).  Same dtypes, errors and conventions as ss2d_forward. */
int ss1d_bidir_forward(const void *x, const void *dt_raw, const float *A_log, const void *Bs,
                       const void *Cs, const float *Ds, const float *dt_bias, void *y,
                       int64_t B, int64_t D, int64_t L, int64_t N, int dtype, void *stream);

/* ---- options: gate and zero-order hold --------------------------------------------------
 * ss2d_forward_ex and ss1d_bidir_forward_ex take two more arguments than the plain entry
 * points (which equal them with z = NULL, flags = 0):
 *
 *   z      optional gate, NULL for none.  Same shape, layout and data type as x and y.
 *          Each route's output is multiplied by SiLU(z) = z / (1 + exp(-z)) at its image
 *          position before the routes are added (the Vim summary, section 4.3, "Gating and
 *          Merging": forward and backward outputs each gated by SiLU(z), then added; the
 *          explainer's MambaBlock multiplies the scan output by silu(z)).  As z is shared by
 *          the routes, the library applies SiLU(z) once to the fp32 sum, before the single
 *          rounding.  z must be aligned to its element size and must not overlap y.
 *   flags  0 or SS2D_FLAG_ZOH.  SS2D_FLAG_ZOH discretises B by zero-order hold as well:
 *          Bbar = (exp(delta A) - 1) / A * B in place of delta * B (the Vim summary,
 *          section 4.1: Bbar = (delta A)^-1 (exp(delta A) - I) delta B); A = 0 takes the
 *          limit delta * B.  Unknown bits give SS2D_ERR_UNSUPPORTED.
 *
 * Every other argument, error and convention is that of the plain entry point. */
#define SS2D_FLAG_ZOH 1

int ss2d_forward_ex(const void *x, const void *dt_raw, const float *A_log, const void *Bs,
                    const void *Cs, const float *Ds, const float *dt_bias, const void *z,
                    void *y, int64_t B, int64_t D, int64_t H, int64_t W, int64_t N, int dtype,
                    int flags, void *stream);

int ss1d_bidir_forward_ex(const void *x, const void *dt_raw, const float *A_log,
                          const void *Bs, const void *Cs, const float *Ds,
                          const float *dt_bias, const void *z, void *y, int64_t B, int64_t D,
                          int64_t L, int64_t N, int dtype, int flags, void *stream);

/* ---- the forward without allocation ----------------------------------------------------------
 * For callers that cannot allocate device memory during the call: code under HIP graph
 * capture that must not record allocation nodes, tight serving loops, harnesses that forbid
 * hipMalloc.  ss2d_forward_noalloc is ss2d_forward_ex (same arguments, same kernels, same
 * result bit for bit) except for its scratch (the transposed copy of x, the per-route fp32
 * outputs, chunk carries): instead of the stream-ordered pool it uses a fixed device array
 * of SS2D_NOALLOC_SCRATCH_BYTES that the library holds on every device it runs on until the
 * process ends.  The call allocates and frees nothing (no hipMalloc, hipFree or stream-
 * ordered allocation; the array's address is looked up once per device at its first call).
 *
 * Size limit: the scratch a call needs is about 2 bytes per element of x for the
 * transposed copy (4 for fp32 data) plus 16 bytes per element of x for the four routes'
 * fp32 outputs, plus chunk carries when the plan cuts long sequences (e.g. the fp32
 * VMamba-T stage-1 shape with B = 8, D = 192, 56 x 56, N = 16 needs ~103 MB); a call needing
 * more returns SS2D_ERR_SCRATCH before anything is enqueued.  Use ss2d_forward_ex for
 * larger calls.
 *
 * Every call on one device shares that device's array, which keeps the last call's
 * contents (nothing in it needs to start at zero): two calls that overlap in time on one
 * device (on different streams, or from different host threads) race on it and give
 * undefined results.  Calls on one stream are ordered and safe. */
#define SS2D_NOALLOC_SCRATCH_BYTES ((size_t)128 << 20)
int ss2d_forward_noalloc(const void *x, const void *dt_raw, const float *A_log, const void *Bs,
                         const void *Cs, const float *Ds, const float *dt_bias, const void *z,
                         void *y, int64_t B, int64_t D, int64_t H, int64_t W, int64_t N,
                         int dtype, int flags, void *stream);

/* ---- backward ---------------------------------------------------------------------------
 * Gradients of the scalar sum over (b, d, l) of dy[b, d, l] * y[b, d, l], y being the output
 * of ss2d_forward (ss1d_bidir_forward) on the same inputs, with respect to every input:
 *   dx (shape of x), ddt_raw (shape of dt_raw), dBs, dCs (shape of Bs, Cs): the data type
 *     of x (dtype), each rounded once from an fp32 sum;
 *   dA_log (K, D, N), dDs (K, D), ddt_bias (K, D): fp32.
 * dy has the shape and data type of x.  Every output is written in full (not accumulated
 * into) and must overlap neither an input nor another output.
 *
 * The gradients follow reverse-mode differentiation of the forward recurrence (the Vim
 * summary, section 4.4: the backward pass recomputes the intermediate states instead of
 * storing them): per route, the adjoint lambda_t = dy_t C_t + Abar_t+1 lambda_t+1 runs
 * backwards from the end of the sequence; dC_t += dy_t h_t and dB_t += lambda_t delta_t u_t
 * are summed over the channels that share Bs and Cs; delta's gradient passes softplus'
 * derivative sigmoid(dt_raw + dt_bias).  States are recomputed from checkpoints taken every
 * 32 steps (scratch, 4 B * B * K * D * ceil(L / 32) * N); sums over channels and images are
 * taken in a fixed order, so results are deterministic.
 *
 * Supported: the plain operator (no gate, delta * B; ss2d_backward_ex below takes the gate
 * and the zero-order hold) with N in {1, 2, 4, 8, 16, 32}, as the forward; other N give
 * SS2D_ERR_UNSUPPORTED.  The kernels split each channel's states over four lanes: N = 1
 * and 2 run as four states, the extra ones with zero B and C rows, which keep them exactly
 * zero (scratch: padded copies of Bs, Cs and A_log and of their gradients); N = 32 runs at
 * two waves per SIMD.  Otherwise the conventions of ss2d_forward apply. */
int ss2d_backward(const void *x, const void *dt_raw, const float *A_log, const void *Bs,
                  const void *Cs, const float *Ds, const float *dt_bias, const void *dy,
                  void *dx, void *ddt_raw, float *dA_log, void *dBs, void *dCs, float *dDs,
                  float *ddt_bias, int64_t B, int64_t D, int64_t H, int64_t W, int64_t N,
                  int dtype, void *stream);

int ss1d_bidir_backward(const void *x, const void *dt_raw, const float *A_log,
                        const void *Bs, const void *Cs, const float *Ds,
                        const float *dt_bias, const void *dy, void *dx, void *ddt_raw,
                        float *dA_log, void *dBs, void *dCs, float *dDs, float *ddt_bias,
                        int64_t B, int64_t D, int64_t L, int64_t N, int dtype, void *stream);

/* ---- backward of the gated and the zero-order-hold operator --------------------------------
 * Gradients of the scalar sum over (b, d, l) of dy[b, d, l] * y[b, d, l], y being the output
 * of ss2d_forward_ex (ss1d_bidir_forward_ex) with the same gate z and flags.  With z = NULL
 * and flags = 0 this is ss2d_backward (ss1d_bidir_backward).
 *
 * Gate (z not NULL): y = (sum over the routes of y_k) * SiLU(z) (the gate of the Vim block,
 * Vim summary section 4.3; the explainer's SelectiveSSM output multiplied by the activated
 * z branch).  By the product rule every route's output receives g = dy * SiLU(z), and
 *   dz = dy * ys * SiLU'(z),   SiLU'(z) = sigmoid(z) * (1 + z * (1 - sigmoid(z))),
 * with ys the ungated route sum; dz (the shape and data type of x) must then be given, is
 * written in full and must overlap neither an input nor another output (with z = NULL, dz
 * is not used).  The checkpoint pass also writes the per-route outputs (scratch, fp32, as
 * in the forward), and the merge kernel forms g and dz from them; g stays in fp32 (scratch,
 * 4 B * B * D * L, twice that for the four routes' transposed copy) whatever the data type,
 * so that bfloat16 data lose nothing to a rounding of the gated gradient.
 *
 * SS2D_FLAG_ZOH: the zero-order-hold operator (Vim summary section 4.1), whose update is
 * h = a h + bb B u with a = exp(delta A) and bb = (a - 1) / A.  The adjoint recurrence is
 * unchanged; with bb in place of delta, dBs sums lambda * bb * u and dx sums
 * lambda * bb * B; d bb / d delta = a, so ddelta takes sum_n lambda * a * B * u in place of
 * sum_n lambda * B * u; and dA_log gains A * lambda * B * u * d bb / dA with
 * d bb / dA = delta^2 * psi(delta A), psi(v) = (v e^v - (e^v - 1)) / v^2 (its power series
 * for |v| < 1/4).
 *
 * Everything else, supported shapes and errors included, is as in ss2d_backward; flags
 * other than SS2D_FLAG_ZOH give SS2D_ERR_UNSUPPORTED. */
int ss2d_backward_ex(const void *x, const void *dt_raw, const float *A_log, const void *Bs,
                     const void *Cs, const float *Ds, const float *dt_bias, const void *z,
                     const void *dy, void *dx, void *ddt_raw, float *dA_log, void *dBs,
                     void *dCs, float *dDs, float *ddt_bias, void *dz, int64_t B, int64_t D,
                     int64_t H, int64_t W, int64_t N, int dtype, int flags, void *stream);

int ss1d_bidir_backward_ex(const void *x, const void *dt_raw, const float *A_log,
                           const void *Bs, const void *Cs, const float *Ds,
                           const float *dt_bias, const void *z, const void *dy, void *dx,
                           void *ddt_raw, float *dA_log, void *dBs, void *dCs, float *dDs,
                           float *ddt_bias, void *dz, int64_t B, int64_t D, int64_t L,
                           int64_t N, int dtype, int flags, void *stream);

/* ---- training: a forward that keeps the backward's checkpoints ---------------------------
 * In training the forward and the backward run on the same inputs.  The backward restarts
 * every 8-step quarter of the scan from the state before it, which ss2d_backward_ex obtains
 * by running the forward scan once more (the Vim summary, section 4.4: states are
 * recomputed, not kept in HBM per step); ss2d_forward_save keeps those states while it
 * computes y, and ss2d_backward_saved starts from them, so that the pair does the scan's
 * forward work once.
 *
 * saved: caller-owned device memory of ss2d_saved_state_bytes(K, B, D, L, N, gated) bytes
 * (K = 4 with L = H * W for the image operators, K = 2 for the bidirectional one; gated:
 * whether z is given), 16-byte aligned.  Layout: the state before every 8-step quarter,
 * (B, K, D, ceil(L / 8), N) fp32 (the first quarter's, zero, is not written; 16 bytes per
 * element of x for N = 16), then with the
 * gate the ungated route sum ((y_0 + y_1) + y_2) + y_3, (B, D, L) fp32, from which the
 * gate's backward forms g and dz.  ss2d_saved_state_bytes returns -1 for sizes the
 * operator rejects and for N not a multiple of 4.
 *
 * ss2d_forward_save: y as ss2d_forward_ex with the same arguments (bit for bit when that
 * call runs in one pass, i.e. without the chunked plan it takes for batches too small to
 * fill the chip; the training forward always runs one pass), and `saved` filled.
 * ss2d_backward_saved: every gradient as ss2d_backward_ex, bit for bit, reading `saved`
 * instead of recomputing it.  The backward's inputs, z, flags and shapes must be those of
 * the forward that filled `saved`, and `saved` unchanged since; the library cannot check
 * this (the state lives on the device), and other contents give undefined gradients.
 * `saved` overlaps no other argument.  N must be a multiple of 4 (SS2D_ERR_UNSUPPORTED
 * otherwise); everything else is as in ss2d_forward_ex and ss2d_backward_ex. */
int64_t ss2d_saved_state_bytes(int K, int64_t B, int64_t D, int64_t L, int64_t N, int gated);

int ss2d_forward_save(const void *x, const void *dt_raw, const float *A_log, const void *Bs,
                      const void *Cs, const float *Ds, const float *dt_bias, const void *z,
                      void *y, float *saved, int64_t B, int64_t D, int64_t H, int64_t W,
                      int64_t N, int dtype, int flags, void *stream);

int ss1d_bidir_forward_save(const void *x, const void *dt_raw, const float *A_log,
                            const void *Bs, const void *Cs, const float *Ds,
                            const float *dt_bias, const void *z, void *y, float *saved,
                            int64_t B, int64_t D, int64_t L, int64_t N, int dtype, int flags,
                            void *stream);

int ss2d_backward_saved(const void *x, const void *dt_raw, const float *A_log, const void *Bs,
                        const void *Cs, const float *Ds, const float *dt_bias, const void *z,
                        const float *saved, const void *dy, void *dx, void *ddt_raw,
                        float *dA_log, void *dBs, void *dCs, float *dDs, float *ddt_bias,
                        void *dz, int64_t B, int64_t D, int64_t H, int64_t W, int64_t N,
                        int dtype, int flags, void *stream);

int ss1d_bidir_backward_saved(const void *x, const void *dt_raw, const float *A_log,
                              const void *Bs, const void *Cs, const float *Ds,
                              const float *dt_bias, const void *z, const float *saved,
                              const void *dy, void *dx, void *ddt_raw, float *dA_log, void *dBs,
                              void *dCs, float *dDs, float *ddt_bias, void *dz, int64_t B,
                              int64_t D, int64_t L, int64_t N, int dtype, int flags,
                              void *stream);

/* The same pair for the operator over per-route inputs (ss2d_forward_routes,
 * ss2d_backward_routes): u (B, K, D, L) in place of x, du in place of dx; the saved state's
 * size and layout are those above. */
int ss2d_forward_routes_save(const void *u, const void *dt_raw, const float *A_log,
                             const void *Bs, const void *Cs, const float *Ds,
                             const float *dt_bias, const void *z, void *y, float *saved,
                             int64_t B, int64_t D, int64_t H, int64_t W, int64_t N, int dtype,
                             int flags, void *stream);

int ss1d_bidir_forward_routes_save(const void *u, const void *dt_raw, const float *A_log,
                                   const void *Bs, const void *Cs, const float *Ds,
                                   const float *dt_bias, const void *z, void *y, float *saved,
                                   int64_t B, int64_t D, int64_t L, int64_t N, int dtype,
                                   int flags, void *stream);

int ss2d_backward_routes_saved(const void *u, const void *dt_raw, const float *A_log,
                               const void *Bs, const void *Cs, const float *Ds,
                               const float *dt_bias, const void *z, const float *saved,
                               const void *dy, void *du, void *ddt_raw, float *dA_log, void *dBs,
                               void *dCs, float *dDs, float *ddt_bias, void *dz, int64_t B,
                               int64_t D, int64_t H, int64_t W, int64_t N, int dtype, int flags,
                               void *stream);

int ss1d_bidir_backward_routes_saved(const void *u, const void *dt_raw, const float *A_log,
                                     const void *Bs, const void *Cs, const float *Ds,
                                     const float *dt_bias, const void *z, const float *saved,
                                     const void *dy, void *du, void *ddt_raw, float *dA_log,
                                     void *dBs, void *dCs, float *dDs, float *ddt_bias, void *dz,
                                     int64_t B, int64_t D, int64_t L, int64_t N, int dtype,
                                     int flags, void *stream);

/* ---- backward of the operator over per-route inputs ---------------------------------------
 * Gradients of the scalar sum over (b, d, l) of dy[b, d, l] * y[b, d, l], y being the output
 * of ss2d_forward_routes (ss1d_bidir_forward_routes) on the same inputs, gate z and flags:
 * the gradients of ss2d_backward_ex, but with each route's own input u (B, K, D, L, in scan
 * order, the data type) in place of x, and du of that shape (the gradient of route k's
 * input at step t; the routes share no input, so nothing is summed across them) in place of
 * dx.  This is the gradient that the per-route front end (ss2d_project) continues with.
 * Every other argument, error and convention is that of ss2d_backward_ex. */
int ss2d_backward_routes(const void *u, const void *dt_raw, const float *A_log, const void *Bs,
                         const void *Cs, const float *Ds, const float *dt_bias, const void *z,
                         const void *dy, void *du, void *ddt_raw, float *dA_log, void *dBs,
                         void *dCs, float *dDs, float *ddt_bias, void *dz, int64_t B,
                         int64_t D, int64_t H, int64_t W, int64_t N, int dtype, int flags,
                         void *stream);

int ss1d_bidir_backward_routes(const void *u, const void *dt_raw, const float *A_log,
                               const void *Bs, const void *Cs, const float *Ds,
                               const float *dt_bias, const void *z, const void *dy, void *du,
                               void *ddt_raw, float *dA_log, void *dBs, void *dCs, float *dDs,
                               float *ddt_bias, void *dz, int64_t B, int64_t D, int64_t L,
                               int64_t N, int dtype, int flags, void *stream);

/* ---- per-route front end and the operator over per-route inputs ---------------------------
 * In the pages' per-direction modules every scan direction carries its own input layers: the
 * explainer's CrossScanModule holds one SelectiveSSM per direction (a depthwise Conv1d with
 * kernel d_conv and padding d_conv - 1 cut to the first L outputs, a SiLU, x_proj to
 * [dt, B, C] and dt_proj), and in the Vim block (Vim summary, section 4.3) each path runs a
 * Conv1d and a SiLU on its own copy of the sequence and generates delta, B and C from the
 * activated output, which is also the input of that path's scan.
 *
 * ss2d_project computes, for every route k and image b, from the shared input x (B, D, H, W)
 * [ss1d_bidir_project: (B, D, L), routes forward and reversed], with s_t = x[b, d, pi_k(t)]
 * and s_t = 0 for t < 0:
 *   u[b,k,d,t]      = SiLU(conv_b[k,d] + sum_{j<KW} conv_w[k,d,j] * s_{t-KW+1+j})
 *   xd[m,t]         = sum_d x_proj_w[k,m,d] * u[b,k,d,t]        m < R + 2N (no bias)
 *   dt_raw[b,k,d,t] = sum_{r<R} dt_proj_w[k,d,r] * xd[r,t]      (dt_proj's bias is dt_bias,
 *                                                               added inside the softplus)
 *   Bs[b,k,n,t]     = xd[R+n,t],   Cs[b,k,n,t] = xd[R+N+n,t]
 * i.e. a causal conv along each route (route 1 is causal in reversed raster order, routes 2
 * and 3 along columns), x_proj's output split [dt (R) | B (N) | C (N)].  Outputs, in the
 * scan order of each route, are exactly the inputs of ss2d_forward_routes:
 *   u, dt_raw (B, K, D, L) and Bs, Cs (B, K, N, L) in dtype;
 *   weights conv_w (K, D, KW), conv_b (K, D), x_proj_w (K, R + 2N, D), dt_proj_w (K, D, R):
 *   fp32, read only.
 * Supported: 1 <= KW <= 8, R >= 1, R + 2N <= 96 (else SS2D_ERR_UNSUPPORTED).  Every output is
 * written in full and must overlap neither an input nor another output (SS2D_ERR_ALIAS).
 * The conv and dt_proj are computed in fp32; x_proj accumulates in fp32 on the matrix cores
 * from u as stored (for bf16, the stored bf16 u, with each fp32 weight split into two bf16
 * parts whose sum carries 16 significant bits).  Scratch: a transposed copy of x for the
 * column routes (stream-ordered, as in ss2d_forward).
 *
 * ss2d_forward_routes is ss2d_forward_ex with each route's own input u (B, K, D, L), in scan
 * order, in place of the gathered x: step t of route k reads u[b,k,d,t] for both the update
 * (delta * B * u) and the skip term (Ds * u); outputs are added at the visited positions in
 * route order, optionally gated by z (B, D, H, W), with flags as in ss2d_forward_ex.
 * Every other argument, error and convention is that of ss2d_forward_ex. */
int ss2d_project(const void *x, const float *conv_w, const float *conv_b,
                 const float *x_proj_w, const float *dt_proj_w, void *u, void *dt_raw, void *Bs,
                 void *Cs, int64_t B, int64_t D, int64_t H, int64_t W, int64_t N, int64_t R,
                 int64_t KW, int dtype, void *stream);

int ss1d_bidir_project(const void *x, const float *conv_w, const float *conv_b,
                       const float *x_proj_w, const float *dt_proj_w, void *u, void *dt_raw,
                       void *Bs, void *Cs, int64_t B, int64_t D, int64_t L, int64_t N,
                       int64_t R, int64_t KW, int dtype, void *stream);

int ss2d_forward_routes(const void *u, const void *dt_raw, const float *A_log, const void *Bs,
                        const void *Cs, const float *Ds, const float *dt_bias, const void *z,
                        void *y, int64_t B, int64_t D, int64_t H, int64_t W, int64_t N,
                        int dtype, int flags, void *stream);

int ss1d_bidir_forward_routes(const void *u, const void *dt_raw, const float *A_log,
                              const void *Bs, const void *Cs, const float *Ds,
                              const float *dt_bias, const void *z, void *y, int64_t B,
                              int64_t D, int64_t L, int64_t N, int dtype, int flags,
                              void *stream);

/* ---- the front end and the operator with dt_proj folded into the scan ---------------------
 * dt_proj is linear and has no bias of its own (its bias is dt_bias, added inside the
 * softplus), and the explainer's SelectiveSSM applies it to the R-row dt slice of x_proj's
 * output (dt_rank = ceil(d_model / 16), a low rank): step t's dt_raw[d] is
 * sum_{r<R} dt_proj_w[k,d,r] * xd[r,t].  Forming that sum inside the scan, from the R rows
 * instead of the D rows, leaves the operator unchanged and removes dt_raw (B, K, D, L) from
 * memory: the front end stores the R dt rows and the scan reads them back.
 *
 * ss2d_project_lr / ss1d_bidir_project_lr are ss2d_project / ss1d_bidir_project without
 * dt_proj: in place of dt_raw they write dt_lr[b,k,r,t] = xd[r,t] (B, K, R, L) in dtype, and
 * take no dt_proj_w.  Every other output, argument and error is as there.
 *
 * ss2d_forward_routes_lr / ss1d_bidir_forward_routes_lr are ss2d_forward_routes /
 * ss1d_bidir_forward_routes with dt_raw given as the product
 *   dt_raw[b,k,d,t] = sum_{r<R} dt_w[k,d,r] * dt_lr[b,k,r,t]
 * formed in fp32 at every step (dt_lr (B, K, R, L) in dtype, dt_w (K, D, R) fp32, both read
 * only).  Supported: 1 <= R <= 4 (else SS2D_ERR_UNSUPPORTED); y must overlap neither dt_lr
 * nor dt_w (SS2D_ERR_ALIAS); NULL dt_lr or dt_w gives SS2D_ERR_NULL.  Every other argument,
 * error and convention is that of ss2d_forward_routes. */
int ss2d_project_lr(const void *x, const float *conv_w, const float *conv_b,
                    const float *x_proj_w, void *u, void *dt_lr, void *Bs, void *Cs, int64_t B,
                    int64_t D, int64_t H, int64_t W, int64_t N, int64_t R, int64_t KW,
                    int dtype, void *stream);

int ss1d_bidir_project_lr(const void *x, const float *conv_w, const float *conv_b,
                          const float *x_proj_w, void *u, void *dt_lr, void *Bs, void *Cs,
                          int64_t B, int64_t D, int64_t L, int64_t N, int64_t R, int64_t KW,
                          int dtype, void *stream);

int ss2d_forward_routes_lr(const void *u, const void *dt_lr, const float *dt_w,
                           const float *A_log, const void *Bs, const void *Cs, const float *Ds,
                           const float *dt_bias, const void *z, void *y, int64_t B, int64_t D,
                           int64_t H, int64_t W, int64_t N, int64_t R, int dtype, int flags,
                           void *stream);

int ss1d_bidir_forward_routes_lr(const void *u, const void *dt_lr, const float *dt_w,
                                 const float *A_log, const void *Bs, const void *Cs,
                                 const float *Ds, const float *dt_bias, const void *z, void *y,
                                 int64_t B, int64_t D, int64_t L, int64_t N, int64_t R,
                                 int dtype, int flags, void *stream);

/* ---- gated delta rule ---------------------------------------------------------------------
 * A selective scan whose state is a matrix: per sequence and value head h, with key head
 * h / (H / HK), a state S (DK, DV) that starts at h0 (zero without one) and per token
 *   S  <- exp(g_t) S                      (decay, g_t <= 0 a log; -inf forgets everything)
 *   u_t = beta_t (v_t - S^T k_t),   S <- S + k_t u_t^T        (the delta rule)
 *   o_t = scale S^T q_t.
 * k is used as given: the rule is stable for |k_t|^2 beta_t <= 2, so callers normalise k.
 *
 *   q, k      (B, L, HK, DK)  dtype        g, beta  (B, L, H)          fp32
 *   v, o      (B, L, H, DV)   dtype        h0, ht   (S, H, DK, DV)     fp32
 * strides: 9 element strides, (batch, token, head) of q, of k and of v, whose last axis is
 * contiguous (views into one fused projection, for instance; none negative); NULL for
 * contiguous tensors.  Every other tensor is contiguous.  H is a multiple of HK,
 * 1 <= DK <= 128 (SS2D_ERR_UNSUPPORTED above), any DV >= 1; v's token stride, H * DV and HK * DK
 * are at most 2^24 (SS2D_ERR_UNSUPPORTED above).
 *
 * cu_seqlens: NULL, and the B rows are S = B sequences of L tokens; or S + 1 ascending
 * offsets (device memory) into the L tokens of B = 1: sequence n holds tokens
 * cu_seqlens[n] .. cu_seqlens[n + 1] - 1, none for equal offsets.  Tokens outside of every
 * sequence are neither read nor written.  The offsets are device data that no call checks
 * on the host; the kernels cut them to [0, L], so that others than ascending ones give
 * wrong values but touch no other memory.
 *
 * Arithmetic: S, the chunk's triangular solve and every sum are fp32 for both data types.
 * For bfloat16 data a product's fp32 operand runs on the bf16 matrix cores as the sum of 3
 * bfloat16 terms (24 bits), those of o, dq and dk as 2 (17 bits) before their single rounding;
 * fp32 data use the fp32 matrix instructions.  Few or long sequences are cut into segments that
 * run at once: each gives its end state from a zero start, Z, and its matrix M, and the states
 * between them follow from S <- M S + Z, on operands of 3 terms for either type.
 *
 * NaN and infinities: o, the end states and the gradients are NaN or infinite wherever the
 * definition makes them so (an infinity may come out as NaN).  In o and the end states nothing
 * else is: a value of token t reaches no token before t, no other sequence or
 * head and, if it is v's, no other column.  A gradient that the definition leaves finite may be
 * NaN where it shares its sequence, head (q, k: key head) and block of 64 tokens with the value.
 *
 * ss1d_delta_forward writes o and, if ht is not NULL, the end states; ht may be h0 itself
 * (in place).  saved (NULL, or ss1d_delta_saved_bytes bytes of device memory, aligned to 256)
 * keeps what ss1d_delta_backward starts from: the states before every 64 tokens and at the
 * end, and v_t - S^T k_t and o_t in fp32.
 *
 * ss1d_delta_backward: the gradients of sum(dout * o) + sum(dht * ht) (dht NULL: none) with
 * respect to q, k (summed over the value heads that share them) and v in dtype, g, beta and,
 * if dh0 is not NULL, h0 in fp32; all contiguous.  saved: what ss1d_delta_forward kept for the
 * same inputs (other contents give undefined gradients), or NULL to compute it again.  dout
 * is contiguous.  Rows outside of every sequence are left as they are.  The gradient of a g
 * below -1000, whose decay is 0, is 0; others are differences of sums, fp32, of dout.o and dv.v
 * over up to 64 tokens: their accuracy is absolute, also where strong decays leave little of them.
 *
 * ss1d_delta_step is the form for serving: T tokens (few) of each of B sequences, whose
 * states are updated in place: row b's state is state[slots[b]], or state[b] with slots
 * NULL.  A row whose slot is negative or >= S is padding: nothing of it is read or written,
 * its rows of o included.  Rows that name the same slot are successive tokens of one
 * sequence, in row order.
 *
 * The shared conventions hold, except that kernel timing does not cover these entry points, and
 * that under stream capture scratch has to be the caller's: the _ws forms take it (scratch: device
 * memory aligned to 256, of scratch_bytes >= ss1d_delta_scratch_bytes, SS2D_ERR_SCRATCH below; NULL:
 * the library's, and SS2D_ERR_SCRATCH under capture), the others use the library's.  A captured
 * graph then holds kernels only, and its scratch is its own for as long as the caller keeps it.
 * Scratch (the step has none): per token, the chunks' matrices, about 0.4 KB per value head and
 * 6 DK (fp32: 12 DK) bytes per key head, DK rounded up to 32, 64 or 128; per segment and head,
 * M, Z and a state; the backward's gradients of the states in fp32, one per 64 tokens and head,
 * for bfloat16 data dv in fp32, and partial sums. */
int ss1d_delta_forward(const void *q, const void *k, const void *v, const float *g,
                       const float *beta, const float *h0, const int32_t *cu_seqlens, void *o,
                       float *ht, void *saved, int64_t B, int64_t L, int64_t S, int64_t HK,
                       int64_t H, int64_t DK, int64_t DV, const int64_t *strides, float scale,
                       int dtype, void *stream);

int ss1d_delta_forward_ws(const void *q, const void *k, const void *v, const float *g,
                          const float *beta, const float *h0, const int32_t *cu_seqlens, void *o,
                          float *ht, void *saved, void *scratch, int64_t scratch_bytes, int64_t B,
                          int64_t L, int64_t S, int64_t HK, int64_t H, int64_t DK, int64_t DV,
                          const int64_t *strides, float scale, int dtype, void *stream);

/* Bytes of scratch (-1 for sizes that the operator rejects) of a forward (backward 0) or a backward
 * (1); kept: whether `saved` is given to it; packed: whether cu_seqlens is. */
int64_t ss1d_delta_scratch_bytes(int backward, int kept, int64_t B, int64_t L, int64_t S, int64_t HK,
                                 int64_t H, int64_t DK, int64_t DV, int dtype, int packed);

/* Bytes of `saved` (-1 for sizes that the operator rejects); packed: whether cu_seqlens is
 * given. */
int64_t ss1d_delta_saved_bytes(int64_t B, int64_t L, int64_t S, int64_t H, int64_t DK, int64_t DV,
                               int packed);

int ss1d_delta_backward(const void *q, const void *k, const void *v, const float *g,
                        const float *beta, const float *h0, const int32_t *cu_seqlens,
                        const void *saved, const void *dout, const float *dht, void *dq, void *dk,
                        void *dv, float *dg, float *dbeta, float *dh0, int64_t B, int64_t L,
                        int64_t S, int64_t HK, int64_t H, int64_t DK, int64_t DV,
                        const int64_t *strides, float scale, int dtype, void *stream);

int ss1d_delta_backward_ws(const void *q, const void *k, const void *v, const float *g,
                           const float *beta, const float *h0, const int32_t *cu_seqlens,
                           const void *saved, const void *dout, const float *dht, void *dq, void *dk,
                           void *dv, float *dg, float *dbeta, float *dh0, void *scratch,
                           int64_t scratch_bytes, int64_t B, int64_t L, int64_t S, int64_t HK,
                           int64_t H, int64_t DK, int64_t DV, const int64_t *strides, float scale,
                           int dtype, void *stream);

/* Testing and tuning, as ss2d_set_launch_plan: for later calls from this host thread, the
 * chunks of 32 tokens per segment (even; 0: whole sequences, -1: automatic) that the forward
 * and the backward cut sequences into.  A saved state belongs to the setting it was made
 * with.  Returns SS2D_OK or SS2D_ERR_SHAPE. */
int ss1d_delta_set_segment(int64_t chunks);

int ss1d_delta_step(const void *q, const void *k, const void *v, const float *g,
                    const float *beta, float *state, const int32_t *slots, void *o, int64_t B,
                    int64_t T, int64_t S, int64_t HK, int64_t H, int64_t DK, int64_t DV,
                    const int64_t *strides, float scale, int dtype, void *stream);

/* ---- block norm -----------------------------------------------------------------------------
 * The norms before and after a block fused with its gate, residual scale and residual
 * connection (the explainer's VMambaBlock, x + SS2D(norm x), with the gate y SiLU(z) of its
 * SelectiveSSM):
 *   p = Norm(h; w_post, b_post)        after the block (p = h with w_post NULL)
 *   p <- p SiLU(z)                     gate (z NULL: none)
 *   y = residual + res_scale p         residual NULL: y = res_scale p; res_scale NULL: 1
 *   n = Norm(y; w_pre, b_pre)          before the next block (none with w_pre NULL)
 * over D channels; layer 0: Norm(x) = x / sqrt(mean(x^2) + eps) w; layer 1: with x - mean(x) in
 * place of x, plus b (a bias may be given with either kind, NULL for none).
 *
 *   channels_first 0: rows of D, (B * L, D);  1: (B, D, L), the layout of ss2d_forward's maps
 *     with L = H * W (the norm over D at every position).
 *   h, z, n: dtype; residual, y: ytype, which is dtype or SS2D_F32 (a residual stream kept
 *     in fp32); the vectors fp32: w_*, b_* (D), res_scale (G, D): G runs of B * L / G
 *     successive rows (channels first: of B / G images) each use their own row; G = 0 without.
 * All contiguous.  D <= 8192, channels first D <= 1024 and L <= 2^24 (SS2D_ERR_UNSUPPORTED
 * above).  y may be
 * the residual (in place) and may be NULL if n is given.  Everything is computed in fp32 from
 * the inputs as stored; n from y before its rounding.
 *
 * ss2d_norm_backward: the gradients of sum(dy * y) + sum(dn * n), given y as it was stored (the
 * second norm is recomputed from it) and the other inputs: dh, dz (given with z) in dtype,
 * dresidual (NULL if there was none) in ytype, and in fp32 dres_scale (G, D), dw_post, db_post
 * (given with b_post), dw_pre, db_pre (optional).  dy NULL: no gradient arrives at y.  y and
 * dn are needed with w_pre.  The vectors' sums over rows run in a fixed order (no atomics);
 * without rows they are 0.
 *
 * The shared conventions hold; kernel timing does not cover these entry points, and the backward's
 * scratch is as the gated delta rule's (ss2d_norm_backward_ws, ss2d_norm_scratch_bytes). */
int ss2d_norm_forward(const void *h, const void *z, const void *residual, const float *res_scale,
                      const float *w_post, const float *b_post, const float *w_pre,
                      const float *b_pre, void *y, void *n, int64_t B, int64_t L, int64_t D,
                      int64_t G, int channels_first, int layer, float eps, int dtype, int ytype,
                      void *stream);

int ss2d_norm_backward(const void *h, const void *z, const float *res_scale, const float *w_post,
                       const float *b_post, const float *w_pre, const void *y, const void *dy,
                       const void *dn, void *dh, void *dz, void *dresidual, float *dres_scale,
                       float *dw_post, float *db_post, float *dw_pre, float *db_pre, int64_t B,
                       int64_t L, int64_t D, int64_t G, int channels_first, int layer, float eps,
                       int dtype, int ytype, void *stream);

int ss2d_norm_backward_ws(const void *h, const void *z, const float *res_scale, const float *w_post,
                          const float *b_post, const float *w_pre, const void *y, const void *dy,
                          const void *dn, void *dh, void *dz, void *dresidual, float *dres_scale,
                          float *dw_post, float *db_post, float *dw_pre, float *db_pre, void *scratch,
                          int64_t scratch_bytes, int64_t B, int64_t L, int64_t D, int64_t G,
                          int channels_first, int layer, float eps, int dtype, int ytype,
                          void *stream);

/* Bytes of ss2d_norm_backward_ws's scratch (-1 for sizes that it rejects). */
int64_t ss2d_norm_scratch_bytes(int64_t B, int64_t L, int64_t D, int64_t G, int channels_first);

/* ---- selective scan in token order -----------------------------------------------------------
 * The scan of one causal route over tokens, with states in and out: per sequence and channel d, a
 * state h of N values that starts at h0 (zero without one) and per token
 *   delta = softplus(dt_raw + dt_bias),   h_n <- exp(-exp(A_log_n) delta) h_n + delta B_n u,
 *   y = (sum_n C_n h_n + Ds u) SiLU(z)                        (z NULL: no gate)
 * (the explainer's SelectiveSSM, whose scan and gate these are).  Channels last:
 *   u, dt_raw, z, y (B, L, D)  dtype       A_log (D, N), Ds, dt_bias (D)   fp32
 *   Bs, Cs          (B, L, G, N) dtype     h0, ht                (S, D, N)  fp32
 * B and C are shared by the D / G channels of a group (channel d: group d / (D / G)).
 * strides: 12 element strides, (batch, token) of u, of dt_raw and of z, then (batch, token, group)
 * of Bs and of Cs, whose last axes are contiguous (views into one projection, for instance; none
 * negative, token and group strides of more than one token or group at most 2^24, SS2D_ERR_SHAPE above;
 * z's unused without z); NULL for contiguous tensors.  Every other tensor is contiguous.  1 <= N <= 32 (SS2D_ERR_UNSUPPORTED
 * above), D a multiple of G, at most 2^24.
 *
 * Calls with a launch past 2^32 threads are refused (SS2D_ERR_SHAPE): of more than 2^24 blocks, each 64
 * channels (16 in short calls of few channels) of a group and of a sequence or segment; cut into
 * segments with S D N at 2^32; backward with 2^28 tokens, every sequence's in whole sixteens, or with
 * D (N + 2) at 2^28.
 *
 * cu_seqlens: NULL, and the B rows are S = B sequences of L tokens; or S + 1 ascending offsets
 * (device memory) into the L tokens of B = 1, as for the gated delta rule: tokens outside of every
 * sequence are neither read nor written, and the kernels cut offsets to [0, L].
 *
 * Arithmetic: delta, the state, every sum and the gate are fp32; outputs are rounded once.  A rate
 * exp(A_log) log2(e) above the largest fp32 (A_log of 88.4 or more) is taken as that: the state is
 * forgotten at every token whose delta is not 0.  Few sequences are cut into segments that run at
 * once from a zero start and are joined by h <- exp(A sum delta) h + end.  NaN and infinities reach
 * what the definition says, and nothing before their token, of another sequence or, if they are u's,
 * dt_raw's or z's, another channel (an infinity may come out as NaN); dB and dC of their token and
 * group are sums over channels, and a channel's dA_log, dDs and ddt_bias, sums over tokens, may be
 * NaN with any of its states.
 *
 * ss1d_scan_forward writes y and, if ht is not NULL, the end states; ht may be h0 itself (in place).
 * saved (NULL, or ss1d_scan_saved_bytes bytes of device memory, aligned to 256) keeps what
 * ss1d_scan_backward starts from: the states before every 16 tokens (8 for N > 16).
 *
 * ss1d_scan_backward: the gradients of sum(dy * y) + sum(dht * ht) (dht NULL: none) with respect to
 * u, dt_raw, z (given with z), Bs and Cs in dtype, and in fp32 A_log, Ds, dt_bias and, if dh0 is not
 * NULL, h0; all contiguous, as dy.  saved: what ss1d_scan_forward kept for the same inputs (other
 * contents give undefined gradients), or NULL to compute it again.  Rows outside of every sequence are
 * left as they are.  Sums run in a fixed order (no atomics); those over no tokens or no channels are 0.
 *
 * ss1d_scan_step is the form for serving: T tokens (few) of each of B sequences, whose states are
 * updated in place: row b's state is state[slots[b]], or state[b] with slots NULL (then S = B).  A row
 * whose slot is negative or >= S is padding: nothing of it is read or written, its rows of y included.
 * Rows that name the same slot are successive tokens of one sequence, in row order.
 *
 * The shared conventions hold, except that kernel timing does not cover these entry points and that
 * under stream capture scratch has to be the caller's: scratch is device memory aligned to 256 of
 * scratch_bytes >= ss1d_scan_scratch_bytes (SS2D_ERR_SCRATCH below), or NULL for the library's
 * (SS2D_ERR_SCRATCH under capture where any is needed).  The step needs none; a forward 8 N + 4 bytes
 * per segment and channel; a backward fp32 sums of dB and dC for every 64 channels of a group, those of
 * the parameters for every segment, and without `saved` the same and an unused y. */
int ss1d_scan_forward(const void *u, const void *dt_raw, const float *A_log, const void *Bs,
                      const void *Cs, const float *Ds, const float *dt_bias, const void *z,
                      const float *h0, const int32_t *cu_seqlens, void *y, float *ht, void *saved,
                      void *scratch, int64_t scratch_bytes, int64_t B, int64_t L, int64_t S, int64_t D,
                      int64_t G, int64_t N, const int64_t *strides, int dtype, void *stream);

int ss1d_scan_backward(const void *u, const void *dt_raw, const float *A_log, const void *Bs,
                       const void *Cs, const float *Ds, const float *dt_bias, const void *z,
                       const float *h0, const int32_t *cu_seqlens, const void *saved, const void *dy,
                       const float *dht, void *du, void *ddt_raw, float *dA_log, void *dBs, void *dCs,
                       float *dDs, float *ddt_bias, void *dz, float *dh0, void *scratch,
                       int64_t scratch_bytes, int64_t B, int64_t L, int64_t S, int64_t D, int64_t G,
                       int64_t N, const int64_t *strides, int dtype, void *stream);

/* Bytes of scratch (-1 for sizes that the operator rejects) of a forward (backward 0) or a backward
 * (1); kept: whether `saved` is given to it; packed: whether cu_seqlens is. */
int64_t ss1d_scan_scratch_bytes(int backward, int kept, int64_t B, int64_t L, int64_t S, int64_t D,
                                int64_t G, int64_t N, int dtype, int packed);

/* Bytes of `saved` (-1 for sizes that the operator rejects). */
int64_t ss1d_scan_saved_bytes(int64_t B, int64_t L, int64_t S, int64_t D, int64_t N, int packed);

/* Testing and tuning, as ss2d_set_launch_plan: for later calls from this host thread, the lanes that
 * share a channel in a forward without `saved` (4 or 16; 0: automatic) and the tokens of a segment,
 * rounded up to the kernels' tile (0: whole sequences, -1: automatic).  Returns SS2D_OK,
 * SS2D_ERR_UNSUPPORTED for other lanes or SS2D_ERR_SHAPE. */
int ss1d_scan_set_plan(int lanes, int64_t tokens);

int ss1d_scan_step(const void *u, const void *dt_raw, const float *A_log, const void *Bs,
                   const void *Cs, const float *Ds, const float *dt_bias, const void *z, float *state,
                   const int32_t *slots, void *y, int64_t B, int64_t T, int64_t S, int64_t D, int64_t G,
                   int64_t N, const int64_t *strides, int dtype, void *stream);

/* ---- short causal convolution -------------------------------------------------------------------
 * The depthwise convolution before the scan (the explainer's Conv1d with padding d_conv - 1, cut to
 * the tokens, and its SiLU), with the inputs before a sequence carried from call to call:
 *   y_t = act(conv_b + sum_{j < KW} conv_w_j x_{t - KW + 1 + j}),   act = SiLU (silu 1) or none (0)
 * per channel; x before a sequence's first token is its initial state, zero without one.
 *   x, y (B, L, D) dtype      conv_w (D, KW), conv_b (D, or NULL) fp32
 *   h0, ht (S, KW - 1, D) dtype: the KW - 1 inputs before the next token, the oldest first.
 * strides: 2 element strides, (batch, token) of x, whose last axis is contiguous; NULL for a
 * contiguous tensor.  1 <= KW <= 8 (SS2D_ERR_UNSUPPORTED above).  cu_seqlens, S, packed rows, ht in
 * place, padding rows and repeated slots of the step, scratch: as for the scan above.  Sums are fp32,
 * y is rounded once.
 *
 * ss1d_conv_backward: the gradients of sum(dy * y) + sum(dht * ht) with respect to x and, if dh0 is
 * not NULL, h0 in dtype, conv_w and (given with conv_b) conv_b in fp32; contiguous, as dy and dht.
 * Scratch (ss1d_conv_scratch_bytes): partial sums of the taps' gradients, in a fixed order. */
int ss1d_conv_forward(const void *x, const float *conv_w, const float *conv_b, const void *h0,
                      const int32_t *cu_seqlens, void *y, void *ht, int64_t B, int64_t L, int64_t S,
                      int64_t D, int64_t KW, const int64_t *strides, int silu, int dtype, void *stream);

int ss1d_conv_backward(const void *x, const float *conv_w, const float *conv_b, const void *h0,
                       const int32_t *cu_seqlens, const void *dy, const void *dht, void *dx,
                       float *dconv_w, float *dconv_b, void *dh0, void *scratch, int64_t scratch_bytes,
                       int64_t B, int64_t L, int64_t S, int64_t D, int64_t KW, const int64_t *strides,
                       int silu, int dtype, void *stream);

/* Bytes of ss1d_conv_backward's scratch (-1 for sizes that it rejects). */
int64_t ss1d_conv_scratch_bytes(int64_t B, int64_t L, int64_t S, int64_t D, int64_t KW, int dtype,
                                int packed);

int ss1d_conv_step(const void *x, const float *conv_w, const float *conv_b, void *state,
                   const int32_t *slots, void *y, int64_t B, int64_t T, int64_t S, int64_t D, int64_t KW,
                   const int64_t *strides, int silu, int dtype, void *stream);

/* ---- group norm ---------------------------------------------------------------------------------
 * A norm of channels-last maps over positions and groups of channels, with its activation:
 *   y = act((x - mean) / sqrt(var + eps) * weight + bias),   act = SiLU (silu 1) or none (0)
 * with mean and var (of the values themselves, about their mean) over the L positions and C / G
 * channels of an image's group.
 *   x, y (B, L, C) dtype, channels last (L = H * W for maps);  weight, bias (C) fp32, NULL for 1 and 0
 *   stats (B, G, 2) fp32, or NULL: mean and 1 / sqrt(var + eps), written by the forward for the
 *     backward, which computes them again without (no positions: 0 and 1 / sqrt(eps)).
 * All contiguous.  C a multiple of G, at most 2^20; L below 2^31; B G at most 2^25, B C about 2^28
 * (SS2D_ERR_SHAPE above).  Statistics are fp32, by the mean first and then the squares about it.
 *
 * ss2d_group_norm_backward: the gradients of sum(dy * y): dx in dtype, dweight and dbias (given with
 * weight, with bias) in fp32, summed in a fixed order; without positions they are 0.
 * Scratch (ss2d_group_norm_scratch_bytes; kept: whether stats is given): as for the scan above. */
int ss2d_group_norm_forward(const void *x, const float *weight, const float *bias, void *y, float *stats,
                            void *scratch, int64_t scratch_bytes, int64_t B, int64_t L, int64_t C,
                            int64_t G, int silu, float eps, int dtype, void *stream);

int ss2d_group_norm_backward(const void *x, const float *weight, const float *bias, const float *stats,
                             const void *dy, void *dx, float *dweight, float *dbias, void *scratch,
                             int64_t scratch_bytes, int64_t B, int64_t L, int64_t C, int64_t G, int silu,
                             float eps, int dtype, void *stream);

int64_t ss2d_group_norm_scratch_bytes(int backward, int kept, int64_t B, int64_t L, int64_t C, int64_t G,
                                      int dtype);

/* ---- launch-plan override (testing and tuning, not part of the operator) ---------------
 * Sets, for calls made later from the calling host thread only, the lanes that share one
 * channel's states in the forward scan (split: 1, 2 or 4; 0 = automatic) and the chunk
 * length of the chunked scan (chunk_len: 0 = one pass, > 0 = chunks of that many steps
 * rounded up to a multiple of 32, -1 = automatic).  The override changes how the work is
 * cut, not what is computed: any setting gives the operator's result (to rounding, which
 * may differ with the cut).  A split that does not divide N, or split 2 with chunks, falls
 * back to what the kernels support.  Returns SS2D_OK, SS2D_ERR_UNSUPPORTED for another
 * split, or SS2D_ERR_SHAPE for chunk_len < -1 or >= 2^30.  The default on every thread is
 * automatic (0, -1); no environment variable is read. */
int ss2d_set_launch_plan(int split, int64_t chunk_len);

/* Static, human-readable text for a status code (never NULL). */
const char *ss2d_status_string(int status);

/* SS2D_ABI_VERSION of the loaded library. */
int ss2d_abi_version(void);

/* hipError_t value of the last failed HIP call made by this library on the calling thread
 * (0 if none). */
int ss2d_last_hip_error(void);

/* ---- scratch pool (memory management, not part of the operator) -----------------------
 * Hands the device memory that the library's scratch pool on the calling thread's current
 * device reserves beyond keep_bytes back to the driver (hipMemPoolTrimTo), for callers that
 * need it for other allocations between calls; later calls allocate it again.  Writes the
 * bytes the pool still reserves afterwards to *reserved (may be NULL).  Only memory that
 * no call uses is released: scratch of a call still running, or whose release is still
 * pending on its stream, stays reserved, so synchronise the streams of earlier calls first.
 * On a device where the library has made no call there is no pool: SS2D_OK with
 * *reserved = 0.  Returns SS2D_OK or SS2D_ERR_HIP. */
int ss2d_scratch_trim(size_t keep_bytes, size_t *reserved);

/* ---- kernel timing (measurement support, not part of the operator) -----------------------
 * While enabled on a host thread, every call from that thread brackets each kernel launch
 * with a pair of HIP events on the call's stream.  ss2d_timing_read waits for the recorded
 * events, adds each kernel's duration to its kind, writes per-kind totals (milliseconds)
 * and launch counts to ms[SS2D_KERNEL_KINDS] and launches[SS2D_KERNEL_KINDS] (either may be
 * NULL), and clears the record.  ss2d_timing_enable returns the previous setting. */
#define SS2D_KERNEL_TRANSPOSE 0 /* per-plane transpose of x for the column routes      */
#define SS2D_KERNEL_SCAN 1      /* selective scan producing per-route outputs          */
#define SS2D_KERNEL_CHUNK_AGG 2 /* chunked scan, first pass (chunk end states)         */
#define SS2D_KERNEL_CARRY 3     /* not launched: chunk start states are composed in the
                                   scan's second pass (the kind keeps its number)        */
#define SS2D_KERNEL_MERGE 4     /* cross-merge into y (backward: route gradients into dx) */
#define SS2D_KERNEL_CHECKPOINT 5 /* backward: forward pass storing states every 8 steps  */
#define SS2D_KERNEL_SCAN_BWD 6  /* backward: adjoint scan                               */
#define SS2D_KERNEL_REDUCE 7    /* backward: sums over channel blocks and images         */
#define SS2D_KERNEL_PROJECT 8   /* per-route front end: conv + SiLU, x_proj, dt_proj      */
#define SS2D_KERNEL_KINDS 9
int ss2d_timing_enable(int enable);
int ss2d_timing_read(double *ms, int64_t *launches);

/* ---- issue-rate probe (measurement support, not part of the operator) ------------------
 * Measures, on the current device and `stream`, the instruction rates that bound the scan
 * kernel (whose state update issues 2 multiplies, 2 fused multiply-adds and one v_exp_f32
 * per state and step): three probe kernels at full occupancy (8 waves per SIMD, 8
 * independent chains per lane), after ~0.1 s of warm-up load, best of 3 runs each.  Writes
 *   out[0]  fp32 fused multiply-adds per second (lane operations),
 *   out[1]  v_exp_f32 per second (lane operations),
 *   out[2]  groups of 4 fused multiply-adds and 1 v_exp_f32 per second (one update's mix:
 *           a multiply issues like a fused multiply-add),
 *   out[3]  the shader clock the chip sustained during the grouped probe (Hz), from the
 *           shader and the 100 MHz reference counters,
 *   out[4]  the device's compute units,
 * to out[SS2D_PROBE_OUTPUTS] (caller-owned host memory).  Synchronises `stream`; takes
 * ~0.2 s.  Returns SS2D_OK, SS2D_ERR_NULL, or SS2D_ERR_HIP. */
#define SS2D_PROBE_OUTPUTS 5
int ss2d_probe_issue_rates(double *out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SS2D_H */
