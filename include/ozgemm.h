/*
 * ozgemm -- FP64 matrix multiplication C = A B emulated with exact
 * INT8 x INT8 -> INT32 matrix products (Ozaki Scheme II), for AMD MI355X
 * (gfx950).
 *
 * Method: the web page "Ozaki Scheme II：用 CRT 把高精度 GEMM 映射成少量 INT8
 * GEMM" (chatdocs.ruinique.com/nla/ozaki-scheme-ii), cited below as
 * "Ozaki II notes §n".  Its §7 lists the pipeline this library runs:
 *   1. bit budget k from M = prod m_t and the inner dimension q (§5);
 *   2. power-of-two row/column scalings D, E and truncation to integer
 *      matrices A' = trunc(DA), B' = trunc(BE) (§3);
 *   3. for each of s pairwise-coprime moduli m_t <= 256: symmetric int8
 *      residues of A' and B', one exact int8 GEMM, product mod m_t (§4, §6);
 *   4-5. CRT accumulation and reduction to the symmetric representative (§4, §5);
 *   6. unscaling by D^-1 and E^-1 (§7).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Matrices are column-major (BLAS convention): A is m x q with leading
 *    dimension lda >= max(1, m); B is q x n, ldb >= max(1, q); C is m x n,
 *    ldc >= max(1, m).  No alpha/beta: C is overwritten.  A caller holding
 *    row-major data passes (B^T, A^T) and receives C^T.
 *  - Every pointer argument that names matrix data is DEVICE memory owned by
 *    the caller; the library never allocates, frees or retains it.
 *  - Work is enqueued on the configured HIP stream and the calls return
 *    without synchronising (like BLAS on a GPU).  The caller synchronises.
 *  - Return value: 0 on success.  -i means argument i (1-based) is invalid;
 *    positive values are the OZGEMM_* codes below.  Arguments are checked
 *    before anything is enqueued, so outputs are untouched on any error.
 *  - The library keeps one global configuration; it is not thread-safe and
 *    calls that overlap on one stream-set race on the workspace.
 *  - s, the number of moduli, is 1..OZGEMM_S_MAX; the moduli are the first s
 *    of the greedy pairwise-coprime sequence 256, 255, 253, 251, 247, 241,
 *    239, 233, 229, 227, 223, 217, 211, 199, 197, 193, 191, 181, 179, 173.
 *  - Every int8 dot product of length < 2^17 (|.| <= q * 2^14) is exact in
 *    int32 (Ozaki II notes §6).  For q >= 2^17 the GEMM splits K into parts
 *    of at most 2^16 and adds their products mod m_t (the notes' block
 *    products; see ozgemm_gemm_parts), so q may go up to OZGEMM_Q_MAX; s
 *    must leave k >= 1 bits (§5).  Otherwise OZGEMM_RANGE.
 *  - Numerics: the result equals X * 2^(e_i + f_j - 2k) rounded once to
 *    nearest-even, where X = (A'B')_ij exactly.  Rows of A / columns of B that
 *    hold Inf or NaN make the outputs they touch NaN; all-zero rows/columns
 *    give +0; results beyond the double range round to +-Inf.
 */
#ifndef OZGEMM_H
#define OZGEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define OZGEMM_OK                  0
#define OZGEMM_NOT_CONFIGURED      1  /* ozgemm_config has not succeeded */
#define OZGEMM_RANGE               2  /* q > OZGEMM_Q_MAX, k(s, q) < 1 (conservative budget), q >= OZGEMM_FAST_Q_LIMIT (OS II-fast), or size beyond the configured maximum */
#define OZGEMM_WORKSPACE_TOO_SMALL 3  /* workspace_bytes below ozgemm_workspace_bytes(...) */
#define OZGEMM_HIP_ERROR           4  /* a HIP call failed; ozgemm_strerror(4) names it */

#define OZGEMM_S_MAX 20               /* largest supported number of moduli */
#define OZGEMM_Q_LIMIT (1 << 17)      /* int8 dot products of length < this are exact in int32 (Ozaki II notes §6) */
#define OZGEMM_Q_MAX   (1 << 27)      /* largest supported inner dimension */
#define OZGEMM_FAST_Q_LIMIT (1 << 23) /* OS II-fast needs q below this: its row-norm sums of q terms of at most 2^40 stay exact in 64 bits */
#define OZGEMM_MAX_ROWS 2096896       /* largest m and n: 2^21 - 256, so that the rows padded to 256 form at most 65535 tiles of 32 */
#define OZGEMM_EXP_NONFINITE 0x7fffffff /* exponent of a row/column holding Inf/NaN */
#define OZGEMM_PANELS_MAX 16          /* most column panels of the pipeline (ozgemm_set_panels) */
#define OZGEMM_ONE_PASS_Q_MIN 4096    /* ozgemm_dgemm reads B once for Q_MIN <= q <= Q_MAX (conservative budget) */
#define OZGEMM_ONE_PASS_Q_MAX 8192

/* Bit budgets of Scheme II (ozgemm_set_bound) */
#define OZGEMM_BOUND_CONSERVATIVE 0 /* c_max <= q 2^(k_A + k_B), k_A = k_B = k (Ozaki II notes §5) */
#define OZGEMM_BOUND_FAST         1 /* Cauchy-Schwarz c_max bound, OS II-fast (Ozaki II notes §9) */
#define OZGEMM_BOUND_ACCU         2 /* c_max bound from an extra exact int8 product, OS II-accu (Ozaki II notes §9) */
#define OZGEMM_ACCU_Q_MAX   (1 << 16) /* OS II-accu needs q <= this: its bound products stay exact in int32 */

/* Scheme I variants (Ozaki I notes, optimized algorithm) */
#define OZGEMM_S1_RN      0  /* RN split, per-product FP64 accumulation (direction 1) */
#define OZGEMM_S1_HYBRID  1  /* Hybrid split, group-wise INT32 accumulation (directions 2, 3) */
#define OZGEMM_S1_K_MAX   16 /* largest number of slices */
#define OZGEMM_S1_MAX_OUT 136 /* k (k + 1) / 2 at k = OZGEMM_S1_K_MAX */

/* ---------------------------------------------------------------------- */
/* Configuration                                                          */
/* ---------------------------------------------------------------------- */

/* Bytes of device workspace needed for problems up to max_m x max_n x max_q
 * with up to s_max moduli (the per-modulus int8 residue planes of A and B,
 * the uint8 product residues -- at least 128 MiB of them when max_q >= 3969,
 * for the K parts of skinny products -- and small per-row/column arrays).
 * Returns 0 for invalid arguments.  Host only. */
size_t ozgemm_workspace_bytes(int max_m, int max_n, int max_q, int s_max);

/* Record the maximum problem size, the HIP stream (a hipStream_t, may be
 * NULL for the null stream) and a caller-owned device workspace of
 * workspace_bytes bytes.  Nothing is allocated or launched.  Replaces any
 * previous configuration.  Errors: -1..-4 bad sizes (max_m and max_n at most
 * OZGEMM_MAX_ROWS, max_q at most OZGEMM_Q_MAX), -6 NULL workspace,
 * OZGEMM_WORKSPACE_TOO_SMALL. */
int ozgemm_config(int s_max, int max_m, int max_n, int max_q,
                  void *hip_stream, void *workspace, size_t workspace_bytes);

/* Change the stream used by later calls. */
int ozgemm_set_stream(void *hip_stream);

/* Column-panel pipeline of ozgemm_dgemm (Ozaki II notes §8 and §11: the
 * CRT of one part of C overlaps the products of the next part).  C is cut
 * into P column panels of whole 256-column tiles; each panel's B residues
 * and product residues are contiguous, its product is one launch, and its
 * CRT runs on a second stream of the library (default priority, created at
 * the first pipelined call and released by ozgemm_free or ozgemm_config),
 * ordered by events, while the next panel's product runs.  The call's
 * stream waits for the last CRT, so the call stays one unit of work on that
 * stream (and can be captured into a graph like an unpipelined one).
 * Results are identical to the unpipelined path.
 *   panels = 0 or 1: no pipeline (the default);
 *   2 <= panels <= OZGEMM_PANELS_MAX: that many panels whenever the shape
 *     allows (q < 2^17, n_pad >= 512, one K part per panel product).
 * It is off by default because on MI355X the persistent product grid holds
 * every compute unit, so the CRT only fills gaps: measured 1.5-2% slower
 * than the plain call at 16384 x 16384 x 1024 and 8192^3.
 * The setting persists until changed; ozgemm_free resets it to 0.
 * Returns 0, or -1 for panels outside 0..OZGEMM_PANELS_MAX. */
int ozgemm_set_panels(int panels);

/* Forget the configuration (the workspace stays the caller's). */
int ozgemm_free(void);

/* Text for a status code; for OZGEMM_HIP_ERROR it includes the HIP error. */
const char *ozgemm_strerror(int status);

/* ---------------------------------------------------------------------- */
/* The hot path                                                           */
/* ---------------------------------------------------------------------- */

/* C <- A B by Ozaki Scheme II with s moduli (Ozaki II notes §7).
 * m, n, q >= 0; m = 0 or n = 0 does nothing; q = 0 writes C = 0.
 * C must not overlap A or B (-8).  Requires m <= max_m, n <= max_n,
 * q <= max_q, s <= s_max of the configuration (OZGEMM_RANGE otherwise).
 * Enqueues the scale, residue, int8 GEMM and CRT kernels on the stream.
 * Under the conservative budget with OZGEMM_ONE_PASS_Q_MIN <= q <=
 * OZGEMM_ONE_PASS_Q_MAX, B's column exponents are taken inside its residue
 * pass, so B is read once; A is read twice (its row maxima need every column
 * first).  Shorter columns keep two passes, whose first is cheap there.  The
 * results are the same as those of the stage entry points.
 * The first call after ozgemm_config also copies a 16 KB constant table
 * into the workspace (a blocking host-to-device copy) and queries the
 * device's compute-unit count; later calls only enqueue kernels, so they can
 * be captured into a HIP graph once one call has run outside capture. */
int ozgemm_dgemm(int m, int n, int q,
                 const double *A, int lda, const double *B, int ldb,
                 double *C, int ldc, int s);

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): C <- A B
 * exactly as ozgemm_dgemm computes it (same kernels, same bit budget as set
 * by ozgemm_set_bound, same results), with every intermediate in a fixed
 * device array of OZGEMM_NOALLOC_BYTES bytes that the library holds on each
 * GPU it runs on until the process ends.  Needs no ozgemm_config; work goes
 * on `hip_stream` (a hipStream_t, NULL for the null stream) and the call
 * returns without synchronising.  The caller passes device pointers A, B, C
 * as for ozgemm_dgemm.  Calls no hipMalloc, hipFree or other allocating
 * routine.  The first call on a device looks up the array's address and
 * copies a 16 KB constant table into it (a blocking host-to-device copy), so
 * make one call outside any graph capture first.
 * The array is shared by every call on that GPU and keeps the last call's
 * contents: calls that overlap on one GPU (other streams, other host
 * threads) race on it and give wrong results.  Products are not cut into K
 * parts here (q >= 2^17 walks sequential K blocks).
 * Errors: those of ozgemm_dgemm (argument numbers 1..10; no
 * OZGEMM_NOT_CONFIGURED), and OZGEMM_RANGE when the intermediates of this
 * shape need more than OZGEMM_NOALLOC_BYTES: s (m_pad + n_pad) q_pad bytes of
 * residue planes, s m_pad n_pad of product residues (under OS II-accu at
 * least the bound's planes, about 9.02 m_pad n_pad bytes), 2 KB per padded
 * row of A for partial row maxima, and small arrays (m_pad, n_pad: m, n
 * rounded up to 256; q_pad: q rounded up to 128).  ozgemm_workspace_bytes(m, n, q, s)
 * <= OZGEMM_NOALLOC_BYTES is enough; for example 2048 x 2048 x 1024 fits at
 * s = 14, and 1024^3 at every s. */
#define OZGEMM_NOALLOC_BYTES (128 << 20)
int ozgemm_dgemm_noalloc(int m, int n, int q,
                         const double *A, int lda, const double *B, int ldb,
                         double *C, int ldc, int s, void *hip_stream);

/* ---------------------------------------------------------------------- */
/* Host-only introspection (no device needed)                              */
/* ---------------------------------------------------------------------- */

/* Write the first s moduli to moduli_out[0..s-1].  Returns 0 or -1. */
int ozgemm_moduli(int s, int *moduli_out);

/* k = floor(1/2 log2((M/2 - 1)/q)) for the first s moduli, evaluated with
 * exact integers (Ozaki II notes §5), for 1 <= q <= OZGEMM_Q_MAX (long inner
 * dimensions run as K parts, see ozgemm_gemm_parts).  Returns k, which is
 * < 1 when s and q leave no bits (ozgemm_dgemm then returns OZGEMM_RANGE
 * under the conservative budget); -1 for s outside 1..OZGEMM_S_MAX or q < 1;
 * -2 for q > OZGEMM_Q_MAX. */
int ozgemm_kbits(int s, int q);

/* Padded dimensions of the stage buffers below: rows of the residue planes
 * are padded to *m_pad / *n_pad, the inner dimension to *q_pad. */
int ozgemm_plane_dims(int m, int n, int q, int *m_pad, int *n_pad, int *q_pad);

/* Bit budget of later Scheme II calls (ozgemm_dgemm and its stages); the
 * setting persists until changed (ozgemm_free resets it to conservative).
 *   OZGEMM_BOUND_CONSERVATIVE: k = floor(1/2 log2((M/2 - 1)/q)) bits per
 *     entry of every row of A and column of B (Ozaki II notes §5).
 *   OZGEMM_BOUND_FAST: OS II-fast (Ozaki II notes §9).  With
 *     kappa_A + kappa_B = floor(log2(M/2 - 1)) split evenly, row i of A is
 *     scaled by 2^d_i, d_i = kappa_A - c_i - e_i, where 4^c_i is the smallest
 *     power of four >= S_i 2^-40 and S_i = sum_l ceil(|a_il| 2^(20 - e_i))^2
 *     (an exact integer bound of ||a_i 2^-e_i||^2 in units of 2^-40); columns
 *     of B likewise with kappa_B.  Then ||A'_i|| ||B'_j|| <= 2^(kappa_A +
 *     kappa_B) < M/2 (Cauchy-Schwarz), so the CRT result is still the exact
 *     A'B', and entries keep more bits whenever a row's norm is well below
 *     sqrt(q) times its maximum.  The stage exponents become
 *     e'_i = kb - d_i with kb = max(kappa_A, kappa_B), so that the row shift
 *     is kb - e'_i and the unscaling exponent e'_i + f'_j - 2 kb.  Needs
 *     q < OZGEMM_FAST_Q_LIMIT.
 *   OZGEMM_BOUND_ACCU: OS II-accu (Ozaki II notes §9): c_max is bounded by
 *     an extra exact int8 product.  With x_il = |a_il| 2^-e_i in [0, 1)
 *     (e_i the frexp exponent of the row maximum; y_lj likewise for the
 *     columns of B), each x is rounded up into two int8 bands,
 *     x <= H/127 + Lo/(127 2^7): H = ceil(127 x) for x >= 2^-7, Lo =
 *     ceil(127 2^7 x) below.  Then sum_l x_il y_lj <= N_ij / (127^2 2^14)
 *     with N = 2^14 H_A H_B^T + 2^7 (H_A Lo_B^T + Lo_A H_B^T) +
 *     127 min(row sum of Lo_A, column sum of Lo_B), two int8 products run
 *     on the product kernel (length q and 2q).  Row bit counts a_i and
 *     column bit counts b_j satisfy 2^(a_i + b_j) N_ij / (127^2 2^14) <=
 *     M/2 - 1 for every (i, j), compared exactly (a_i + b_j + L_ij <= K2
 *     with K2 = floor(log2(M/2 - 1)) and L_ij = K2 - floor(log2((M/2 - 1)
 *     127^2 2^14 / N_ij))): columns first take half of what their largest
 *     L leaves, rows then the most their columns allow, columns then the
 *     most their rows allow, all at most 76.  Row i of A' is
 *     trunc(a_il 2^(a_i - e_i)), so (|A'||B'|)_ij < M/2 and the CRT result
 *     is exact (§5).  The stage exponents are
 *     e'_i = 76 - a_i + e_i (shift base 76).  Every quantity is an exact
 *     integer, so results are reproducible.  Needs q <= OZGEMM_ACCU_Q_MAX,
 *     s >= 2 and k(s, q) >= 1, and room in the workspace's product region
 *     for two int32 planes and one int8 plane of m_pad x n_pad (about 9.02
 *     m_pad n_pad bytes, which s_max >= 10 always gives; otherwise
 *     OZGEMM_WORKSPACE_TOO_SMALL).
 * Returns 0, or -1 for an unknown mode. */
int ozgemm_set_bound(int mode);

/* Bit budget for (s, q) under `mode`: (k, k) for the conservative bound
 * (OZGEMM_RANGE if k < 1), (kappa_A, kappa_B) for OS II-fast (OZGEMM_RANGE
 * if q >= OZGEMM_FAST_Q_LIMIT), (K2, 76) for OS II-accu: the budget
 * a_i + b_j + L_ij <= K2 = floor(log2(M/2 - 1)) that the row and column bit
 * counts share, and their cap (OZGEMM_RANGE if q > OZGEMM_ACCU_Q_MAX, s < 2
 * or k < 1). */
int ozgemm_bound_budget(int s, int q, int mode, int *kappa_a, int *kappa_b);

/* ---------------------------------------------------------------------- */
/* Stage entry points (the same kernels ozgemm_dgemm runs), for parity     */
/* checks of each integer stage.  All buffers are caller-owned device      */
/* memory; the configured workspace and stream are used.                   */
/* ---------------------------------------------------------------------- */

/* Exponents (Ozaki II notes §3, §5): e[i] for i < m with
 * 2^(e_i - 1) <= max_l |a_il| < 2^e_i (0 for an all-zero row,
 * OZGEMM_EXP_NONFINITE for a row holding Inf/NaN); f[j] likewise for the
 * columns of B.  e has m entries, f has n.  Under OZGEMM_BOUND_FAST the
 * values are the shift exponents e'_i, f'_j of that budget (see
 * ozgemm_set_bound), which depend on s. */
int ozgemm_stage_scale(int m, int n, int q, int s,
                       const double *A, int lda, const double *B, int ldb,
                       int32_t *e, int32_t *f);

/* Truncation and residues (Ozaki II notes §3, §4, §6), with k = kbits(s, q):
 *   A'_il = trunc(a_il 2^(k - e_i)),  B'_lj = trunc(b_lj 2^(k - f_j)),
 *   Ares[t][i][l] = smod(A'_il, m_t),  Bres[t][j][l] = smod(B'_lj, m_t),
 * smod(x, m) in [-floor(m/2), ceil(m/2) - 1].  Planes are int8, K-contiguous:
 * Ares at t*m_pad*q_pad + i*q_pad + l, Bres at t*n_pad*q_pad + j*q_pad + l,
 * zero in the padding.  Aprime (m x q, ld m) and Bprime (q x n, ld q) are
 * optional (NULL to skip) float64 copies of A' and B'. */
int ozgemm_stage_residue(int m, int n, int q, int s,
                         const double *A, int lda, const double *B, int ldb,
                         const int32_t *e, const int32_t *f,
                         int8_t *Ares, int8_t *Bres,
                         double *Aprime, double *Bprime);

/* Per-modulus products (Ozaki II notes §4, §6): C_t = A_t B_t^T over q_pad,
 * exact in int32.  Ct (optional, NULL to skip) receives int32 planes,
 * column-major with ld m_pad: Ct[t*m_pad*n_pad + j*m_pad + i].  rt
 * (optional) receives C_t mod m_t in [0, m_t) as uint8 in the same layout.
 * Without Ct, the product may run as K parts (ozgemm_gemm_parts) whose
 * planes use the workspace's product region; rt must not lie in the
 * workspace. */
int ozgemm_stage_gemm(int m, int n, int q, int s,
                      const int8_t *Ares, const int8_t *Bres,
                      int32_t *Ct, uint8_t *rt);

/* Number of K parts the residue-only product of an m x n x q call with s
 * moduli runs as (ozgemm_dgemm, and ozgemm_stage_gemm without Ct), written
 * to *parts.  When moduli x output tiles of 256 x 256 leave the compute
 * units idle, the inner dimension is cut into P parts, one block per (part,
 * modulus, tile); each part's product mod m_t goes to a plane of the
 * workspace, and a reduction adds the P residues mod m_t (the sum of the
 * parts is the whole product; a part of at most 2^16 K entries is exact in
 * int32, Ozaki II notes §6).  1 = one part; 0 = q >= 2^17 with no room for
 * parts, walked as sequential K blocks instead.  The choice depends on the
 * device's compute units (queried on the current device) and on the
 * configured workspace.  Errors: -1..-5, OZGEMM_NOT_CONFIGURED,
 * OZGEMM_RANGE, OZGEMM_HIP_ERROR. */
int ozgemm_gemm_parts(int m, int n, int q, int s, int *parts);

/* CRT reconstruction, range reduction and unscaling (Ozaki II notes §4, §5,
 * §7): from rt (layout of ozgemm_stage_gemm), e and f, write the m x n result
 * C (ld ldc). */
int ozgemm_stage_crt(int m, int n, int q, int s,
                     const uint8_t *rt, const int32_t *e, const int32_t *f,
                     double *C, int ldc);

/* ---------------------------------------------------------------------- */
/* Scheme I: FP64 GEMM from int8 slices (secondary path)                   */
/*                                                                        */
/* Method: the course page "Ozaki Scheme" (zsc0tt.pages.dev/courses/      */
/* hpc-summer/ozaki-scheme), cited as "Ozaki I notes": its optimized      */
/* algorithm after Uchino, Ozaki and Imamura.  Each row of A and column  */
/* of B is split into k signed slices of beta bits,                       */
/* beta = min(7, floor((31 - log2 q) / 2)); slice p of a row is the       */
/* row's remaining residual rounded to nearest-even on a power-of-two     */
/* grid 2^g (|slice / 2^g| <= 2^(beta-1)).  The products A_i B_j with     */
/* i + j <= k + 1 (k (k + 1) / 2 of them) are exact int8 GEMMs and are    */
/* added up in FP64 in a fixed order, so results are reproducible.        */
/*   OZGEMM_S1_RN:     grid of slice p from the max of the row's residual */
/*                     (RN split); each product converted and added,      */
/*                     i-major, j-minor.                                  */
/*   OZGEMM_S1_HYBRID: grid of slice p = g0 - beta (p - 1), g0 from the   */
/*                     original row max (Hybrid split); products with the */
/*                     same i + j summed in int32, at most                */
/*                     r = max(1, 2^(31 - 2 beta - ceil(log2 q))) at a    */
/*                     time, then added in increasing i + j.              */
/* Grid exponents: g = ceil(log2 max|row|) + 1 - beta; 0 for an all-zero  */
/* row; OZGEMM_EXP_NONFINITE (first grid row only) for a row holding      */
/* Inf/NaN, whose slices are zero and whose outputs are NaN.              */
/* These calls use the configured stream and workspace; the workspace     */
/* must hold ozgemm_scheme1_workspace_bytes(m, n, q, k, variant) bytes    */
/* (else OZGEMM_WORKSPACE_TOO_SMALL).  q may exceed 2^17 (beta shrinks);  */
/* beta < 1 (q > 2^29) gives OZGEMM_RANGE.                                */
/* ---------------------------------------------------------------------- */

/* Slice width beta for inner dimension q, or -1 when none fits. */
int ozgemm_scheme1_beta(int q);

/* Number of int32 product planes (outputs of the products stage):
 * k (k + 1) / 2 for RN; the number of runs for Hybrid.  <0 on bad input. */
int ozgemm_scheme1_outputs(int k, int variant, int q);

/* Workspace bytes needed by a Scheme I call of this shape (0 on bad input). */
size_t ozgemm_scheme1_workspace_bytes(int m, int n, int q, int k, int variant);

/* C <- A B by Scheme I with k slices (1 <= k <= OZGEMM_S1_K_MAX).
 * Arguments and conventions as ozgemm_dgemm, with k and variant in place
 * of s.  Phase timing slots: [scale: 0, split, products, accumulation]. */
int ozgemm_scheme1_dgemm(int m, int n, int q,
                         const double *A, int lda, const double *B, int ldb,
                         double *C, int ldc, int k, int variant);

/* Split stage (Ozaki I notes, RN split / Hybrid split algorithms).
 * Aslices[p][i][l] (p < k) at p*m_pad*q_pad + i*q_pad + l: slice integers of
 * row i of A; Bslices[p][j][l] at p*n_pad*q_pad + j*q_pad + l for column j of
 * B (int8, zero in the padding; m_pad, n_pad, q_pad from ozgemm_plane_dims).
 * gA[p][i] at p*m_pad + i and gB[p][j] at p*n_pad + j: grid exponents, k
 * rows for RN, one row (g0) for Hybrid. */
int ozgemm_scheme1_stage_split(int m, int n, int q, int k, int variant,
                               const double *A, int lda, const double *B, int ldb,
                               int8_t *Aslices, int8_t *Bslices,
                               int32_t *gA, int32_t *gB);

/* Products stage: P[o][j][i] at o*m_pad*n_pad + j*m_pad + i (int32) for
 * o < ozgemm_scheme1_outputs(k, variant, q), in accumulation order:
 * RN: o-th pair (i, j) of the triangle, P = A_i B_j^T;
 * Hybrid: o-th run of pairs (s, g - s), P = sum of their products. */
int ozgemm_scheme1_stage_products(int m, int n, int q, int k, int variant,
                                  const int8_t *Aslices, const int8_t *Bslices,
                                  int32_t *P);

/* Accumulation stage: C (m x n, ld ldc) = sum over o, in order, of
 * P[o] scaled by 2^(gA + gB) of its slices (Hybrid: 2^(g0A + g0B - beta (g - 2))),
 * each addition rounded in FP64. */
int ozgemm_scheme1_stage_accumulate(int m, int n, int q, int k, int variant,
                                    const int32_t *P, const int32_t *gA,
                                    const int32_t *gB, double *C, int ldc);

/* ---------------------------------------------------------------------- */
/* Phase timing                                                           */
/* ---------------------------------------------------------------------- */

/* enable != 0: every later ozgemm_dgemm records HIP events on the stream
 * around its four phases (up to 4096 calls).  ozgemm_phase_ms adds, over the
 * calls since timing was enabled, the milliseconds of [scale, residue, gemm,
 * crt] into ms_out[0..3] (synchronising on the events) and the number of
 * calls into *calls (for a pipelined call, see ozgemm_set_panels: residue =
 * A's residues, gemm = B's residues, the products and the overlapped CRTs,
 * crt = the last panel's CRT tail).  ozgemm_phase_calls writes the same four times of each
 * call, ms_out[4c + p] for call c < min(calls, max_calls), and the number of
 * recorded calls into *calls (either pointer may be NULL when max_calls is
 * 0).  Disabling discards the events. */
int ozgemm_timing(int enable);
int ozgemm_phase_ms(double *ms_out, int *calls);
int ozgemm_phase_calls(double *ms_out, int max_calls, int *calls);

/* Measurement aid: the rate the int8 matrix cores sustain on their own, the
 * practical ceiling of the product step (Ozaki II notes §6: one int8 GEMM
 * per modulus; §10 reports the method against the int8 rate).  `blocks`
 * workgroups of four wavefronts each run `steps` steps of 32
 * v_mfma_i32_16x16x64_i8 with operands in registers, in the product
 * kernel's issue order (2^20 int8 operations per wavefront and step), on
 * pseudo-random operands from `seed`.  Each wavefront writes the XOR of its
 * accumulator words to sink[4 * block + wavefront] (device memory,
 * 4 * blocks uint32, caller owned), which makes the result checkable.
 * Asynchronous on hip_stream (NULL: the null stream); time it with events
 * on that stream.  Needs no configuration.  Returns 0, -1 for blocks
 * outside 1..2^20, -2 for steps < 1, -4 for sink == NULL, or
 * OZGEMM_HIP_ERROR. */
int ozgemm_mfma_ceiling(int blocks, int steps, unsigned seed, unsigned *sink, void *hip_stream);

/* ---------------------------------------------------------------------- */
/* Products over ragged groups, and orthogonalisation by products          */
/* ---------------------------------------------------------------------- */
/* What the layers of a mixture of experts and the optimiser of their
 * matrices need next to C = A B.  Conventions that differ from the calls
 * above: these calls keep no state and need no ozgemm_config; each takes its
 * stream (a hipStream_t, NULL for the null stream) and its workspace, so
 * calls with different workspaces may overlap, from any streams and host
 * threads, and be captured into graphs.  They allocate nothing, never
 * synchronise and copy nothing from the host.  The workspace (device memory,
 * 256-byte aligned) is scratch: its contents do not matter before the call
 * and mean nothing after it; calls that share one must not overlap.  Device
 * pointers belong to the current device.
 *
 * Element types.  Products of OZGEMM_BF16 and OZGEMM_F16 operands are formed
 * on matrix cores with FP32 accumulators and rounded once, to nearest-even.
 * OZGEMM_F32 operands are cut into two half-precision slices per entry on
 * power-of-two grids by row (of the inner dimension); three slice products
 * accumulate in FP32.  An entry's error is that of an FP32 product in blocks:
 * the slices hold an entry to 2^-23 and the products drop at most 2^-22 of a
 * term (2^-39 of the row's largest entry where that is more), under the
 * rounding of the FP32 sums.  A row that holds Inf or NaN makes the outputs
 * it touches NaN, as in ozgemm_dgemm.  F32 products of few columns and small
 * ones are multiplied in FP32 as they lie instead: an entry is itself however
 * far below its row's largest, and Inf and NaN follow the usual rules.  Which
 * of the two a call takes depends on its sizes and on the alignment of its
 * operands alone; slices always need a workspace, so a call for which
 * ..._workspace_bytes gives 0 goes in FP32.
 * (BF16 and F16 follow the usual rules for Inf and NaN.)  Results do not
 * depend on the order in which blocks run. */
#define OZGEMM_F64  0
#define OZGEMM_F32  1
#define OZGEMM_BF16 2
#define OZGEMM_F16  3
#define OZGEMM_E4M3 4 /* 8-bit floating point, 1-4-3: up to 448, no infinities */
#define OZGEMM_E5M2 5 /* 1-5-2: up to 57344 */

#define OZGEMM_GROUPS_MAX 65536 /* most groups of one call */

/* Groups.  n columns, of which group e < groups owns those from offsets[e]
 * up to offsets[e + 1]; offsets is a DEVICE array of groups + 1 integers in
 * increasing order (equal neighbours make an empty group) within [0, n].
 * Columns before offsets[0] and from offsets[groups] on belong to no group.
 * Offsets out of order or out of range are read as the nearest ordered ones
 * (running maximum, cut to [0, n]): nothing outside the operands is touched
 * (but for the other half of an aligned 4-byte word that begins or ends with
 * an operand's first or last 16-bit entry, which is read and not used). */

/* C(:, j) = op(A_e) B(:, j) for the columns j of every group e: the product
 * of a layer of experts (columns are tokens, sorted by expert), and, with
 * transa turned over and m and q swapped, its gradient for B.
 *   type    OZGEMM_F32, OZGEMM_BF16 or OZGEMM_F16 (-1)
 *   op(A_e) m x q; with transa = 0 A_e is m x q (lda >= max(1, m)), with
 *           transa = 1 it is q x m (lda >= max(1, q)), e.g. the row-major
 *           [m][q] weight of a linear layer.  A_e begins at A + e stridea
 *   B       q x n, ldb >= max(1, q);  C  m x n, ldc >= max(1, m), type
 *           ctype: `type` itself or OZGEMM_F32
 * Columns of no group are left as they were.  q = 0 gives zeros.  C must not
 * overlap A, B or the offsets, each from its first entry to its last (rows
 * that interleave overlap).  Every array begins at a multiple of its entries' size.
 * Products of few columns and small ones read their operands as they lie.
 * Larger ones do so with 16-bit operands whose rows begin on 16-byte
 * boundaries, K-contiguous ones (A with transa = 1, B) with q a multiple of 8,
 * K-strided ones (A with transa = 0) with m a multiple of 8; others, and F32
 * operands, then pass through the workspace.  Results too small to fill the
 * card are summed in parts of a long inner dimension, in a fixed order, whose
 * sums take room in the workspace too.
 * Errors: -i for argument i; OZGEMM_RANGE for m, n or q above
 * OZGEMM_MAX_ROWS, groups above OZGEMM_GROUPS_MAX or a grid of more than
 * 2^31 tiles; OZGEMM_WORKSPACE_TOO_SMALL. */
int ozgemm_grouped_gemm(int type, int ctype, int groups, int m, int n, int q, int transa,
                        const void *A, int lda, long long stridea, const void *B, int ldb,
                        const int32_t *offsets, void *C, int ldc,
                        void *workspace, size_t workspace_bytes, void *hip_stream);

/* Bytes of workspace the call above needs for these operands (the pointers
 * are looked at for their alignment alone); 0 where it needs none or the
 * arguments are invalid.  Host only. */
size_t ozgemm_grouped_gemm_workspace_bytes(int type, int groups, int m, int n, int q, int transa,
                                           const void *A, int lda, long long stridea,
                                           const void *B, int ldb);

/* C_e = sum over the columns j of group e of A(:, j) B(:, j)^T: the gradient
 * of a layer of experts for its weights.  A is m x n (lda >= max(1, m)), B
 * q x n (ldb >= max(1, q)), C_e m x q (ldc >= max(1, m)), beginning at
 * C + e stridec (stridec >= ldc q where groups > 1).  An empty group gives
 * zeros.  Types, errors and workspace as above; larger products read 16-bit
 * operands in place where columns begin on 16-byte boundaries and m and q are
 * multiples of 8.  Operands that pass through the workspace (there each group begins at
 * a multiple of 64) need n + 63 min(groups, n) <= 2^21 (OZGEMM_RANGE).  Small
 * results of many columns are summed in parts, in a fixed order, whose sums
 * take room in the workspace too. */
int ozgemm_grouped_outer(int type, int ctype, int groups, int m, int q, int n,
                         const void *A, int lda, const void *B, int ldb,
                         const int32_t *offsets, void *C, int ldc, long long stridec,
                         void *workspace, size_t workspace_bytes, void *hip_stream);

size_t ozgemm_grouped_outer_workspace_bytes(int type, int groups, int m, int q, int n,
                                            const void *A, int lda, const void *B, int ldb);

/* O = the result of `steps` Newton-Schulz steps on every m x n matrix G of a
 * batch:  X = G / (|G|_F + eps), then with P = X X^T (X^T X where m > n)
 *         X <- a X + (b P + c P^2) X     (X <- a X + X (b P + c P^2)),
 * the polynomial that takes X's singular values towards 1 and leaves its
 * singular vectors: the orthogonalised update of the Muon optimiser, with
 * (a, b, c) = (3.4445, -4.7750, 2.0315) five times.
 *   type    OZGEMM_F64, F32, BF16 or F16: G's and O's
 *   G, O    batches of column-major m x n matrices strideg, strideo apart; a
 *           row-major [n][m] array is the same thing and is orthogonalised as
 *           such.  O may be G itself (with its ldg and strideg), and must not
 *           overlap it otherwise.  strideg may be 0
 *   coeffs  HOST array of 3 steps numbers a, b, c, read before the call
 *           returns; |.| < 1e6
 *   s       moduli of the Scheme II products of OZGEMM_F64 (conservative
 *           budget whatever ozgemm_set_bound says); not looked at otherwise.
 *           Small F64 matrices, for which those would be slower, go by the
 *           FP64 matrix cores (a rule on the sizes and s)
 * Between its products X is kept in two half-precision slices (F64: as it is)
 * on a power-of-two grid that follows each matrix's own |G|_F / (|G|_F + eps)
 * and the coefficients: an entry to 2^-22 of itself or 2^-38 of the bound on X's
 * singular values, whichever is more; P and Q = b P + c P^2 likewise.  Their
 * products are formed as the grouped products of F32 operands are, whatever the
 * type, and the result is rounded to it once.
 * The norm is a sum of squares in FP64 (F64 entries beyond 1e153 overflow it:
 * zeros; those below 1e-162 count as none).  steps = 0 gives the normalised G.
 * A matrix of zeros gives zeros where eps > 0 (NaN where it is 0); one that holds Inf
 * or NaN gives NaN throughout (steps > 0).
 * Errors: -i for argument i; OZGEMM_RANGE for m or n above OZGEMM_ORTHO_MAX,
 * batch above 65535, coefficients whose steps may leave 1e18, or an s that
 * leaves no bits; OZGEMM_WORKSPACE_TOO_SMALL. */
#define OZGEMM_ORTHO_MAX 65536
#define OZGEMM_ORTHO_STEPS_MAX 64
int ozgemm_orthogonalize(int type, int batch, int m, int n, const void *G, int ldg, long long strideg,
                         int steps, const double *coeffs, double eps, int s,
                         void *O, int ldo, long long strideo,
                         void *workspace, size_t workspace_bytes, void *hip_stream);

/* Bytes of workspace the call above needs; 0 for invalid or empty arguments.
 * Host only. */
size_t ozgemm_orthogonalize_workspace_bytes(int type, int batch, int m, int n, int s);

/* ---------------------------------------------------------------------- */
/* A layer in 8 bits, and the clipping of its gradients                    */
/* ---------------------------------------------------------------------- */
/* Conventions as for the products over ragged groups: no state, the stream as
 * an argument, nothing allocated, copied from the host or waited for, capturable.
 *
 * Blocks.  A matrix in 8 bits is a matrix of OZGEMM_E4M3 or OZGEMM_E5M2 values
 * and a float scale for every 128 entries of a row, of that row alone (rows = 1)
 * or of 128 rows (rows = 128): the scale of row i and entries 128 b .. 128 b + 127
 * is at S[(i / rows) * srow + b * sblock].
 * The scales that these calls make are powers of two: the least 2^e >= 2^-126
 * with |x| <= MAX 2^e for all finite x of the block (MAX = 448 for E4M3, 57344 for
 * E5M2), 1 for a block of zeros; every value is x 2^-e rounded once, to
 * nearest-even.  Inf and NaN become NaN.  The products take any scales, whose
 * product, of a row's and a column's block, is taken in FP32.
 *
 * Every array begins at a multiple of its entries' size. */

/* V, S = the n x q matrix X in blocks, and Vt, St = its transpose in blocks (of
 * `rows` x 128 of the transpose), either or both (V or Vt NULL: not that one).
 *   type   OZGEMM_F32, BF16 or F16: X's; qtype OZGEMM_E4M3 or E5M2
 *   rows   1 or 128
 *   X      n rows of q entries, ldx >= max(1, q) apart
 *   V      n rows of q bytes, ldv >= max(1, q) apart; Vt q rows of n, ldvt >= max(1, n)
 * No array that is written may overlap another, and no two scales may have one place.
 * Errors: -i for argument i; OZGEMM_RANGE for n or q above OZGEMM_MAX_ROWS or
 * 2^24 and more tiles of 128 x 128. */
int ozgemm_quantize_blocks(int type, int qtype, int rows, int n, int q, const void *X, int ldx,
                           void *V, int ldv, float *S, long long srow, long long sblock,
                           void *Vt, int ldvt, float *St, long long strow, long long stblock,
                           void *hip_stream);

/* C(i, j) = sum over blocks b of SA(i, b) SB(j, b) sum over k in b of A(k, i) B(k, j).
 *   A      q x m (lda >= max(1, q)): the row-major [m][q] weight of a linear layer,
 *          with a scale for every rows_a = 1 or 128 of its rows
 *   B      q x n (ldb >= max(1, q)): n rows of activations, with a scale for each
 *   C      m x n, ldc >= max(1, m), of ctype OZGEMM_F32, BF16 or F16
 * The gradients of a layer are the same call on transposes (ozgemm_quantize_blocks
 * makes them): dX from dY and W turned over, dW from dY and X turned over.
 *
 * Sums.  OZGEMM_F32 results: products are exact and everything is summed in
 * FP32.  BF16 and F16 results of more than 16 columns: the 128 products of a
 * block are summed by the 8-bit matrix cores, which keep of each term what lies
 * above 2^-13 of the largest of the 32 terms next to it; blocks are scaled and
 * added in FP32.  What goes so is measured by the terms, not by their sum: over
 * a matrix of results 1.5e-5 of its norm for gaussian entries, 4.6e-5 with one
 * column of B's in a hundred 21 times larger, 8.6e-5 with it 301 times larger (F16
 * rounds to 2.1e-4, BF16 to 1.7e-3), and without a bound relative to a result
 * whose terms cancel.  F32 results do not lose it.  16 columns and fewer: as F32,
 * so a column's results have other last bits in a call of 16 columns than of 17 (and by
 * the order of sums, which follows m, n and q, elsewhere too).  Results are rounded
 * once, to nearest-even, and the same call gives the same bits.
 * NaN anywhere in a row makes the outputs it touches NaN.
 *
 * Operands are read in place where they begin on 16-byte boundaries and their
 * leading dimension, unless they have one row, is a multiple of 16 up to 2^22 (then as whole aligned 16-byte
 * pieces, of which the last of a row may reach past q: read and not used);
 * others pass through the workspace, as do the scales of large products whose srow
 * is not 1.  Few tiles with a long inner dimension are
 * summed in parts, in a fixed order, whose sums take room there too.
 * q = 0 gives zeros.  C must not overlap the operands or their scales.
 * Errors: -i for argument i; OZGEMM_RANGE for m, n or q above OZGEMM_MAX_ROWS or
 * a grid beyond 2^32 threads; OZGEMM_WORKSPACE_TOO_SMALL. */
int ozgemm_scaled_gemm(int atype, int btype, int ctype, int m, int n, int q,
                       const void *A, int lda, const float *SA, int rows_a, long long sarow, long long sablock,
                       const void *B, int ldb, const float *SB, long long sbrow, long long sbblock,
                       void *C, int ldc, void *workspace, size_t workspace_bytes, void *hip_stream);

/* Bytes of workspace the call above needs (the pointers are looked at for their
 * alignment alone); 0 where it needs none or the arguments are invalid.  Host only. */
size_t ozgemm_scaled_gemm_workspace_bytes(int m, int n, int q,
                                          const void *A, int lda, int rows_a, long long sarow, long long sablock,
                                          const void *B, int ldb, long long sbrow, long long sbblock);

/* Y = H w / sqrt(mean over the row of H^2 + eps) for n rows of q entries, H = X + R.
 *   type   OZGEMM_F32, BF16 or F16: X's, R's and H's; wtype: w's, `type` or OZGEMM_F32
 *   ytype  `type` itself, or OZGEMM_E4M3 or E5M2: then Y is values in blocks (rows = 1)
 *          with scales S, no two of them in one place (not looked at otherwise)
 *   R      the residual; NULL: H = X.  H receives the sum, each entry added in FP32
 *          and rounded to its type, which is what the norm is taken of; not looked
 *          at without R
 * Sums of squares and Y are FP64 and rounded once.  H may be X or R itself (with
 * its leading dimension), and so may a Y of the same type; what is written must not overlap otherwise.
 * Errors: -i for argument i (8: R never is); OZGEMM_RANGE for n or q above OZGEMM_MAX_ROWS. */
int ozgemm_rms_norm(int type, int ytype, int wtype, int n, int q, const void *X, int ldx, const void *R, int ldr,
                    const void *w, double eps, void *H, int ldh, void *Y, int ldy,
                    float *S, long long srow, long long sblock, void *hip_stream);

/* Its gradients: with r = 1 / sqrt(mean H^2 + eps) and g = dY w,
 *   dX = r g - H r^3 mean(g H) + dH   (also the residual's),   dw = sum over the rows of dY H r.
 *   dH     the gradient that reaches H from elsewhere; NULL: none
 *   dX     may be dY, H or dH itself (with its leading dimension)
 *   dw     q entries of wtype; NULL: not wanted
 * Statistics of a row are FP64, entries FP32 and rounded once (rows below 3e-39, whose r with eps = 0 FP32
 * does not hold, give Inf or NaN); dw is summed in
 * FP32 over every row of a few thousand groups and in FP64 over those, in a fixed
 * order.  n = 0 gives dw = 0.  Errors as above. */
int ozgemm_rms_norm_grads(int type, int wtype, int n, int q, const void *dY, int lddy, const void *H, int ldh,
                          const void *w, const void *dH, int lddh, double eps, void *dX, int lddx, void *dw,
                          void *workspace, size_t workspace_bytes, void *hip_stream);

/* Bytes of workspace the call above needs (dw: whether it is wanted).  Host only. */
size_t ozgemm_rms_norm_grads_workspace_bytes(int n, int q, int dw);

#define OZGEMM_ARRAYS_MAX 65536      /* most arrays of one call */
#define OZGEMM_ARRAY_MAX  1099511627776 /* 2^40: most entries of one */

/* *norm = sqrt(sum of the squares of all entries of `count` arrays), in FP64.
 *   types, in, sizes   HOST arrays of `count` types (OZGEMM_F64, F32, BF16 or F16),
 *                      device addresses and numbers of entries, read before the
 *                      call returns
 *   norm               device memory, one double; none of the arrays
 * Inf or NaN in any entry makes it Inf or NaN (F64 entries beyond 1e153 overflow it).
 * Sums are taken in a fixed order.  count = 0 gives 0.  Needs a workspace always. */
int ozgemm_gradient_norm(int count, const int *types, const void *const *in, const long long *sizes, double *norm,
                         void *workspace, size_t workspace_bytes, void *hip_stream);

/* Host only. */
size_t ozgemm_gradient_norm_workspace_bytes(int count, const int *types, const long long *sizes);

/* out[k] = in[k] min(1, most / (*norm + eps)), most >= 0, eps >= 0: the factor is
 * FP64, rounded to 24 bits (also below FP32's range) for arrays other than OZGEMM_F64, whose entries are rounded
 * once.  A norm of NaN makes every entry NaN, as do 0 / 0 and Inf / Inf.
 * out[k] may be in[k] (then nothing is read or written where the
 * factor is 1), and must share no memory with any other array or the norm;
 * otherwise -5.  `norm` is device memory: the one of ozgemm_gradient_norm, or of
 * several of them brought together. */
int ozgemm_clip_gradients(int count, const int *types, const void *const *in, const long long *sizes,
                          void *const *out, const double *norm, double most, double eps, void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* OZGEMM_H */
