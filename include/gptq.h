/*
 * gptq.h -- C ABI of the MI355X (gfx950) GPTQ layer-quantization library.
 *
 * The library computes, for one linear layer with weight W [out, n] (stored as
 * a Linear weight: rows = output neurons, columns = input dimensions) and a
 * calibration matrix X [tokens, n], integer codes Q, per-group scales and zero
 * points minimising the layer-wise reconstruction error ||X (W - What)^T||_F^2
 * (GPTQ-intrinsic LoRA technical summary, "problem statement"; Lattice Geometry
 * of NN Quantization, technical overview section 2, where the problem splits
 * into one closest-vector problem per output row).
 *
 * Conventions for every entry point
 *   - Pointers are DEVICE pointers unless marked [host].  The caller owns every
 *     input and output buffer; the library never frees or keeps them.
 *   - Row-major throughout.  X holds bfloat16 values as their uint16 bit
 *     patterns.  Matrices of size [rows, cols] have leading dimension cols
 *     unless an ld argument is given.
 *   - A context owns its device workspace (grown on demand, kept until
 *     gptq_destroy) and the HIP stream it was created with.  Calls are
 *     asynchronous on that stream except those marked SYNC, which wait for the
 *     stream before returning.  The context also owns a second stream (default
 *     priority) on which the factor runs part of its trailing updates; every
 *     call joins it back into the context's stream by event before its last
 *     launch, so work later enqueued on the context's stream sees all results.
 *     A context is not thread-safe: one context per host thread/stream.
 *   - Every call returns a gptq_status.  Argument errors are detected on the
 *     host before anything is launched.  After GPTQ_ERR_HIP the HIP error text
 *     is available from gptq_last_error().
 *   - Results are deterministic: repeated calls on the same inputs give the
 *     same bytes (no floating-point atomics; every reduction has a fixed order).
 */
#ifndef GPTQ_MI355X_H
#define GPTQ_MI355X_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  GPTQ_OK = 0,
  GPTQ_ERR_INVALID_ARG = 1, /* null pointer, negative size, bad bits/group/block */
  GPTQ_ERR_NOT_PD = 2,      /* damped Hessian not positive definite (see info) */
  GPTQ_ERR_NONFINITE = 3,   /* non-finite entry in H */
  GPTQ_ERR_UNSUPPORTED = 4, /* valid but unsupported shape or alignment */
  GPTQ_ERR_HIP = 5,         /* HIP runtime error (text in gptq_last_error) */
  GPTQ_ERR_NO_MEMORY = 6,   /* workspace allocation failed */
  GPTQ_ERR_NOT_CONVERGED = 7 /* a subspace iteration stopped at its step cap; every
                                output is written, from its last iterate */
} gptq_status;

typedef struct gptq_ctx_s* gptq_ctx;

/* Create a context on HIP device `device`, issuing work on `stream` (a
 * hipStream_t; NULL = the device's null stream).  *ctx [host] receives the
 * handle.  Creates the context's second stream and two events; device
 * workspace is allocated by the first call that needs it. */
int gptq_create(gptq_ctx* ctx, int device, void* stream);

/* Wait for the context's streams, free its workspace and the context. */
int gptq_destroy(gptq_ctx ctx);

/* Static text for a status code. */
const char* gptq_strerror(int status);

/* Text of the last error recorded in ctx (empty string if none). */
const char* gptq_last_error(gptq_ctx ctx);

/* Calibration Hessian (GPTQ-2D technical summary section 1, Gram G = A^T A;
 * Lattice Geometry section 3.1, X^T X):
 *   H[n][n] (fp32, full symmetric) = (accumulate ? H : 0) + X^T X
 * X[tokens][ldx] bf16 bit patterns; only the first n columns are read.
 * The sum is unscaled.  bf16 products are exact in fp32; accumulation is fp32
 * in a fixed order (split over tokens, partials summed in a fixed order), and
 * H is exactly symmetric.  Requires ldx >= n; rows are read with 16-byte
 * loads when ldx % 8 == 0 and X is 16-byte aligned, element by element
 * otherwise.  tokens == 0 leaves H (accumulate) or zeroes it.
 * Asynchronous. */
int gptq_hessian(gptq_ctx ctx, const uint16_t* X, int64_t tokens, int32_t n, int64_t ldx,
                 float* H, int accumulate);

/* Damping and factor (Lattice Geometry section 3.1: X^T X + lam I; GPTQ-2D
 * sections 2 and 4: the feedback factors are the unit-triangular factors of
 * the inverse Gram matrix):
 *   lam = lam_abs + lam_rel * mean(diag H)
 *   U[n][n] fp32, upper triangular with positive diagonal, zero below it, with
 *   (H + lam I)^{-1} = U^T U.
 * Computed in fp64 by Cholesky of the index-reversed damped matrix and a
 * triangular inverse (U = P chol(P H_lam P)^{-1} P, P the reversal), so pivots
 * are eliminated from column n-1 down to 0.
 * SYNC.  *info [host] = 0 on success, else 1 + the column (in H's numbering)
 * of the first non-positive pivot met in that order, and GPTQ_ERR_NOT_PD is
 * returned (U is then undefined).  *lam_used [host] (may be NULL) = lam.
 * H is not modified.  Non-finite H -> GPTQ_ERR_NONFINITE. */
int gptq_factor(gptq_ctx ctx, const float* H, int32_t n, double lam_abs, double lam_rel,
                float* U, int32_t* info, double* lam_used);

/* Blocked column sweep (GPTQ encyclopedia entry, technical approach: quantise
 * a column, update the remaining weights in closed form, groups with their own
 * scale; GPTQ-2D sections 1-2: fixed order, triangular feedback, GPTQ's lazy
 * block update).  For every row, columns j = 0..n-1 in natural order:
 *   at a group start (or once per row when group == 0, on the original row)
 *     fit lo = min(min v, 0), hi = max(max v, 0), s = (hi-lo)/maxq (s = 1 if
 *     hi == lo), r = 1/s, z = rne(-lo*r) on the current weights v of the group;
 *   x = fl32(fl32(w_j*r) + z), q = clamp(rne(x), 0, maxq), what = s (q - z),
 *   E_j = (w_j - what)/U_jj, and w_k -= E_j U_jk for k > j
 * with the in-block part done per column and the rest, after each block of
 * `block` columns, as W[:, b1:] -= E[:, b0:b1] U[b0:b1, b1:].
 * Inputs: W[out][n] fp32 (not modified), U[n][n] from gptq_factor, lam (the
 * damping used for U, for the objective).  Outputs: codes[out][n] uint8 in
 * [0, 2^bits-1]; scales[out][ng] fp32 and zeros[out][ng] uint8 with
 * ng = group ? n/group : 1; err[out][n] fp32 the scaled errors E (may be NULL);
 * obj[2] [host] = {J, J_lam}: J_lam = sum E^2 = tr(D (H+lam I) D^T) and
 * J = J_lam - lam ||D||^2 = ||X D^T||^2 with D = W - What.
 * Requirements: 2 <= bits <= 8; group == 0 or (group % 8 == 0, n % group == 0,
 * and group % block == 0 or block % group == 0); block in {16,32,64,128}.
 * SYNC (objective read back). */
int gptq_quantize(gptq_ctx ctx, const float* W, int32_t out, int32_t n, const float* U,
                  int32_t bits, int32_t group, int32_t block, double lam,
                  uint8_t* codes, float* scales, uint8_t* zeros, float* err, double* obj);

/* GPTQ-intrinsic LoRA (GPTQ-intrinsic LoRA technical summary, method section 2):
 * X~ = [X, X V_r] with V_r the top-r eigenvectors of H = X^T X; the sweep runs
 * on W~ = [W, 0] against the factor of X~^T X~ + lam I (lam = lam_abs +
 * lam_rel * mean(diag H)), rounding only the first n columns; the r appended
 * columns absorb the error.  Outputs codes/scales/zeros as gptq_quantize (W^T
 * ~ Q + L R in the pages' convention, i.e. W ~ What + R^T L^T):
 *   L[n][r] fp32: an orthonormal basis of the top-r eigenspace of H (found by
 *                 subspace iteration in fp64 on min(128, n, max(r + 32, 64))
 *                 columns with a Rayleigh-Ritz check every 4 steps, stopping
 *                 when ||H L - L diag(theta)||_F <= 1e-11 ||theta||; any basis
 *                 gives the same Q and the same product L R);
 *   R[r][out] fp32;
 *   obj[2] [host] = {J, J_lam}, J = ||X (W - What - R^T L^T)^T||^2.
 * X as gptq_hessian; 1 <= r <= min(128, n); requirements on bits/group/block as
 * gptq_quantize.  SYNC.  *info semantics as gptq_factor (may be NULL).
 * GPTQ_ERR_NOT_CONVERGED: the iteration reached its cap of 600 steps (the
 * r-th and (r+1)-th eigenvalues too close for it); every output is written,
 * from the last Ritz vectors. */
int gptq_lora(gptq_ctx ctx, const float* W, int32_t out, int32_t n, const uint16_t* X,
              int64_t tokens, int64_t ldx, int32_t r, int32_t bits, int32_t group,
              int32_t block, double lam_abs, double lam_rel, uint8_t* codes, float* scales,
              uint8_t* zeros, float* L, float* R, double* obj, int32_t* info);

/* gptq_quantize for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * the same arguments, checks, kernels and results (codes, scales, zeros, err
 * and obj bit-identical to gptq_quantize on the same inputs), but every
 * intermediate lives in a fixed array of about 12.7 MB of device memory that
 * the library holds for the process's lifetime, one copy per device, and
 * the pinned host staging it uses is made when the context is created.  The
 * call performs no hipMalloc, hipFree, hipHostMalloc or event creation.
 * Limits: out <= 1024, n <= 4096, out * n <= 2^20; beyond them
 * GPTQ_ERR_UNSUPPORTED with a message.  All contexts on one device share its array, whose
 * contents persist from call to call (the parts that must start at zero are
 * cleared by the call's own kernels): calls that overlap on one device race
 * and give undefined results; serialise them.  Per-kernel timing is off for
 * this call.  SYNC (objective read back). */
int gptq_quantize_noalloc(gptq_ctx ctx, const float* W, int32_t out, int32_t n, const float* U,
                          int32_t bits, int32_t group, int32_t block, double lam,
                          uint8_t* codes, float* scales, uint8_t* zeros, float* err, double* obj);

/* Gram matrix accurate to float64 rounding, H = X^T X in fp64 (the products
 * of bf16 values are exact in fp64 and the sums run in fp64 on fp64 MFMA).  X
 * as gptq_hessian; H[n][n] fp64, device, caller-owned, fully written.  The
 * Hessian the refinement steps below take.  ASYNC on the context's stream. */
int gptq_hessian64(gptq_ctx ctx, const uint16_t* X, int64_t tokens, int32_t n, int64_t ldx, double* H);

/* Refinement after the intrinsic LoRA (GPTQ-intrinsic LoRA technical summary,
 * section 4, Bid-Up refinement: OLrC fits L, R for a fixed Q, Bid-Up moves Q
 * on its fixed grid for fixed L, R, the two alternate and the layer objective
 * never increases).  Objective: J = tr(D H D^T), D = W - What - R^T L^T,
 * What = s (q - z) per group (fp32 as stored), H from gptq_hessian64.
 *
 * gptq_olrc: for the given codes, the rank-r correction C minimising J is
 * C = P P^T E with E = W - What and P the top-r eigenvectors of E H E^T
 * (found by the checked subspace iteration gptq_lora uses for L, in
 * dimension out; GPTQ_ERR_NOT_CONVERGED, with every output written, when it
 * reaches its cap).  Writes L[n][r] = E^T P and R[r][out] = P^T (fp32, device) and
 * J (host, the objective with that correction).  codes/scales/zeros as
 * gptq_quantize's outputs (read only); bits is checked only.
 *
 * gptq_bid_up: one pass over the columns j = 0..n-1 of every row: with
 * g = D H (gradient of the row objective up to the factor -2), the code
 * moves to q* = clamp(rne(x)), x = fl32(fl32(t / s) + z) (t / s as
 * t * fl32(1/s)), t = fl32(what_j + g_j / H_jj), only when that is strictly
 * nearer, |x - q*| < |x - q_j|; the move updates g for the later columns.
 * codes [out][n] are read and rewritten in place (device); L, R as written by
 * gptq_olrc; J (host) = the objective after the pass (its value before plus
 * the summed change of the moves).  The moves run on fp32 with the sweep's
 * lazy block updates (block as gptq_quantize).
 *
 * Both: W[out][n] fp32 and H[n][n] fp64 device; 1 <= r <= min(128, out, n);
 * requirements on bits/group/block as gptq_quantize.  SYNC. */
int gptq_olrc(gptq_ctx ctx, const float* W, int32_t out, int32_t n, const double* H, int32_t r,
              int32_t bits, int32_t group, const uint8_t* codes, const float* scales,
              const uint8_t* zeros, float* L, float* R, double* J);
int gptq_bid_up(gptq_ctx ctx, const float* W, int32_t out, int32_t n, const double* H, int32_t r,
                const float* L, const float* R, int32_t bits, int32_t group, int32_t block,
                uint8_t* codes, const float* scales, const uint8_t* zeros, double* J);

/* gptq_lora followed by `rounds` >= 1 rounds of gptq_olrc then gptq_bid_up,
 * and a last gptq_olrc, all on the fp64 Hessian the LoRA computes (shared,
 * not recomputed).  Outputs codes/scales/zeros (the grid stays the sweep's),
 * L, R from the last OLrC, and trace[2 rounds + 2] (host): J after the
 * sweep, then after every step (non-increasing up to rounding).  Arguments
 * otherwise as gptq_lora (also r <= out).  SYNC. */
int gptq_lora_refine(gptq_ctx ctx, const float* W, int32_t out, int32_t n, const uint16_t* X,
                     int64_t tokens, int64_t ldx, int32_t r, int32_t bits, int32_t group,
                     int32_t block, double lam_abs, double lam_rel, int32_t rounds, uint8_t* codes,
                     float* scales, uint8_t* zeros, float* L, float* R, double* trace, int32_t* info);

/* Cross Gram G = X^T Y (sum over tokens of x_t^T y_t), fp32 [n][n] written in
 * full (not symmetric), on the same bf16 MFMA tiles as gptq_hessian.  X and
 * Y are [tokens][ldx] bf16 bits with the same tokens and pitch; rows 16-byte
 * aligned and n % 8 == 0 (else GPTQ_ERR_UNSUPPORTED).  tokens == 0 writes
 * zeros.  ASYNC on the context's stream. */
int gptq_cross_gram(gptq_ctx ctx, const uint16_t* X, const uint16_t* Y, int64_t tokens, int32_t n,
                    int64_t ldx, float* G);

/* GPTQ with the quantised-input target (Lattice Geometry of NN Quantization,
 * section 5.1: when the layer's inputs come from already-quantised layers,
 * Xq instead of X, only the target of the nearest-plane problem changes).
 * Every row minimises ||Xq q - X w||^2 + lam ||q - w||^2 (damping as a ridge
 * towards w), which is the GPTQ sweep of gptq_quantize on the target
 *   W* = W (G + lam I)^T Hq_lam^{-1},  G = Xq^T X,  Hq_lam = Xq^T Xq + lam I,
 * lam = lam_abs + lam_rel * mean(diag(Xq^T Xq)), with the factor of Hq_lam.
 * With Xq = X the target is W.  The Grams run as gptq_hessian (fp32, bf16
 * MFMA; G over all tiles), the three products forming W* in fp64.
 * Inputs: W[out][n] fp32; X, Xq [tokens][ldx] bf16 bits (device), the same
 * tokens and pitch, rows 16-byte aligned, n % 16 == 0.  Outputs as
 * gptq_quantize (codes, scales, zeros; the grid is fitted on W*'s
 * error-updated values), Wt[out][n] fp32 the target W* (may be NULL), obj[2]
 * [host] = {J, J_lam} of the sweep relative to W* and Hq (J = tr((W* - What)
 * Hq (W* - What)^T); ||Xq What^T - X W^T||^2 differs from it by a constant of
 * W).  *info as gptq_factor.  Requirements on bits/group/block as
 * gptq_quantize.  SYNC. */
int gptq_quantize_qronos(gptq_ctx ctx, const float* W, int32_t out, int32_t n, const uint16_t* X,
                         const uint16_t* Xq, int64_t tokens, int64_t ldx, int32_t bits, int32_t group,
                         int32_t block, double lam_abs, double lam_rel, uint8_t* codes, float* scales,
                         uint8_t* zeros, float* Wt, double* obj, int32_t* info);

/* Two-sided adaptive rounding, GPTQ-2D (GPTQ-2D technical summary): integers
 * Z minimising ||A (Z - X) B||_F^2 greedily, with exactly the trajectory of
 * the one-sided sweep over vec(X) (column-major) under the Gram H kron G,
 * G = A^T A, H = B B^T (section 1; Theorem 2: same result in any order that
 * respects the dependencies, here anti-diagonals).  Rounding entry (i, j)
 * with delta = w_ij - z_ij, z_ij = clamp(rne(fl32(w_ij)), qmin, qmax), feeds
 * -Lg[k][i] delta Uh[j][l] to the entries k >= i, l >= j, with the unit
 * factors Lg[k][i] = UG[i][k] / UG[i][i], Uh[j][l] = UH[j][l] / UH[j][j]
 * (section 2: Kronecker feedback, rank-1 updates, the lazy buffer C = L E).
 * Inputs (device, fp32, row-major): X[m][n] the real target; UG[m][m] and
 * UH[n][n] upper with G^{-1} = UG^T UG, H^{-1} = UH^T UH (gptq_factor of G
 * and of H, with or without damping).  Outputs: Z[m][n] int32 in [qmin,
 * qmax]; delta[m][n] fp32 the rounding residuals w - z (may be NULL);
 * J [host] = sum of (delta_ij / (UG_ii UH_jj))^2 = ||A (Z - X) B||_F^2 for
 * the G, H the factors belong to.  The rounding decisions are taken in fp32
 * and the feedback accumulates in fp32.  SYNC. */
int gptq_round_2d(gptq_ctx ctx, const float* X, int32_t m, int32_t n, const float* UG, const float* UH,
                  int32_t qmin, int32_t qmax, int32_t* Z, float* delta, double* J);

/* One layer of a batch.  X may be NULL: then H must already hold the layer's
 * Hessian (several layers may point at the same H and X == NULL to share it).
 * H and U are caller-provided [n][n] fp32 buffers (H is written when X != NULL).
 * obj and info are outputs written by the call. */
typedef struct {
  const uint16_t* X;
  int64_t tokens;
  int64_t ldx;
  const float* W;
  int32_t out, n;
  int32_t bits, group, block;
  int32_t pad0;
  double lam_abs, lam_rel;
  float* H;
  float* U;
  uint8_t* codes;
  float* scales;
  uint8_t* zeros;
  float* err;      /* may be NULL */
  double obj[2];   /* out: {J, J_lam} */
  int32_t info;    /* out: as gptq_factor */
  int32_t pad1;
} gptq_layer;

/* Quantise many independent layers at once (Hessians, factors, sweeps and
 * trailing updates each run as one grouped launch over all layers per step).
 * layers [host] array of nlayers descriptors; results equal those of calling
 * gptq_hessian, gptq_factor and gptq_quantize per layer.  SYNC.  Returns the
 * first error met; per-layer info/obj are filled in for every layer. */
int gptq_quantize_batched(gptq_ctx ctx, int32_t nlayers, gptq_layer* layers);

/* Deployable outputs (GPTQ encyclopedia entry, technical approach: the
 * quantised weights are used through GPU matrix kernels at inference;
 * performance and accuracy: 4-bit weights take a quarter of the fp32 memory;
 * GPTQ-intrinsic LoRA technical summary, results: L and R themselves at low
 * precision, 4 and 8 bits).  The pages fix no storage format; ours follows.
 * All ASYNC on the context's stream; device buffers, caller-owned.
 *
 * gptq_pack_codes: codes[rows][n] uint8 -> packed[rows][words], words =
 * ceil(n bits / 32) uint32: each row is a little-endian bitstream, code k at
 * stream bits [k bits, (k + 1) bits), stream bit b in word b / 32 at position
 * b % 32, zero bits up to the end of the last word (at 4 bits: code k is the
 * nibble 4 (k % 8) of word k / 8; at 8 bits: byte k).  Code bits above `bits`
 * are ignored.  1 <= bits <= 8.  gptq_unpack_codes is the inverse (codes
 * written in [0, 2^bits - 1]). */
int gptq_pack_codes(gptq_ctx ctx, const uint8_t* codes, int32_t rows, int32_t n, int32_t bits,
                    uint32_t* packed);
int gptq_unpack_codes(gptq_ctx ctx, const uint32_t* packed, int32_t rows, int32_t n, int32_t bits,
                      uint8_t* codes);

/* Round-to-nearest of the low-rank factors of gptq_lora / gptq_olrc (L[n][r],
 * R[r][out] fp32), L at bits_L and R at bits_R (each 2..8): every rank
 * component, a column of L and a row of R, gets its own grid fitted as in
 * gptq_quantize (lo = min(min v, 0), hi = max(max v, 0), s = (hi - lo)/maxq,
 * z = rne(-lo/s) in [0, maxq], maxq = 2^bits - 1 of its factor),
 * then q = clamp(rne(fl32(fl32(v * fl32(1/s)) + z))), vhat = fl32(s (q - z)).
 * Outputs: Lcodes[n][r], Lscales[r], Lzeros[r], Rcodes[r][out], Rscales[r],
 * Rzeros[r]; Lhat[n][r] and Rhat[r][out] the dequantised factors (each may
 * be NULL).  r == 0 writes nothing. */
int gptq_quantize_lowrank(gptq_ctx ctx, const float* L, const float* R, int32_t n, int32_t r, int32_t out,
                          int32_t bits_L, int32_t bits_R, uint8_t* Lcodes, float* Lscales, uint8_t* Lzeros,
                          float* Lhat, uint8_t* Rcodes, float* Rscales, uint8_t* Rzeros, float* Rhat);

/* W4A16 product Y = X What^T of a 4-bit layer: X[M][ldx] bf16 bits (16-byte
 * aligned rows), packed[N][K/8] from gptq_pack_codes at 4 bits, scales[N][G]
 * fp32 and zeros[N][G] uint8 as gptq_quantize writes them (G = K/group, or 1
 * for group 0), What = s (q - z) per group.  Every weight enters the bf16
 * matrix unit as bf16(fl32(s (q - z))) (nearest, ties to even); products are
 * exact and summed in fp32 (for M <= 128 a split-K kernel sums in another
 * order).  Y[M][ldy] fp32, fully written in its M x N part.
 * K == 0 writes zeros.  Requirements: K % 32 == 0; group 0, K, or a power of
 * two >= 8 dividing K; ldx % 8 == 0, X and packed 16-byte aligned (else
 * GPTQ_ERR_UNSUPPORTED). */
int gptq_gemm_w4a16(gptq_ctx ctx, const uint16_t* X, int64_t M, int64_t ldx, const uint32_t* packed,
                    const float* scales, const uint8_t* zeros, int32_t N, int32_t K, int32_t group, float* Y,
                    int64_t ldy);

/* The same product for the other widths the layers are quantised at (GPTQ
 * encyclopedia entry, technical approach and performance and accuracy: 2 to
 * 4 bits; GPTQ-intrinsic LoRA technical summary, results: 3-bit layers, L
 * and R at 4 and 8 bits): bits in {2, 3, 4, 8}, packed[N][K bits/32] from
 * gptq_pack_codes at that width (each row one bitstream, so 32 codes fill
 * `bits` whole words).  Everything else, rounding and requirements included,
 * as gptq_gemm_w4a16, which is this call with bits = 4.  Other widths:
 * GPTQ_ERR_UNSUPPORTED. */
int gptq_gemm_wqa16(gptq_ctx ctx, const uint16_t* X, int64_t M, int64_t ldx, const uint32_t* packed,
                    const float* scales, const uint8_t* zeros, int32_t N, int32_t K, int32_t group, int32_t bits,
                    float* Y, int64_t ldy);

/* Serving operators: what a layer runs between its quantised products when it
 * answers token by token.  (The pages stop at the quantised weights' matrix
 * products; these operators have no counterpart there.)  All ASYNC on the
 * context's stream; device buffers, caller-owned.  They may be captured into
 * a HIP graph: the attention needs workspace, which its first call of a size
 * allocates, so run a call once before it is captured (one that needs more
 * while the stream is captured is refused: GPTQ_ERR_UNSUPPORTED).  That workspace
 * is the context's, also in a graph's replays: calls of a context and replays
 * of graphs captured with it run one after the other, on one stream or ordered by
 * events.  What overlaps (another stream, a graph beside eager calls) needs a context
 * of its own, or results are wrong, later ones included.  Element types of x, y, K
 * and V: GPTQ_BF16 (bit patterns) or GPTQ_F32; their last dimension (the head)
 * is contiguous, the strides of tokens and heads are given in elements. */
#define GPTQ_BF16 0
#define GPTQ_F32 1
#define GPTQ_ROPE_HALF 0        /* pairs (i, i + rot/2) */
#define GPTQ_ROPE_INTERLEAVED 1 /* pairs (2i, 2i + 1) */
#define GPTQ_ROPE_PLAIN 0  /* frequencies base^(-2i/rot) */
#define GPTQ_ROPE_LINEAR 1 /* all divided by factor */
#define GPTQ_ROPE_BASE 2   /* base times factor^(rot/(rot-2)) */
#define GPTQ_ROPE_PARTS 3  /* by turns over `original` positions: below `low` turns divided by
                              factor, above `high` kept, in between mixed in proportion */

typedef struct {
  int32_t kind;     /* GPTQ_ROPE_PLAIN .. GPTQ_ROPE_PARTS */
  int32_t original; /* length the frequencies were made for (parts) */
  double factor, low, high;
  double magnitude; /* both halves of the table are multiplied by it */
} gptq_rope_scaling;

/* Rotary table[length][2][rot/2] fp32: magnitude * cos and magnitude * sin of
 * position * frequency, angles in fp64.  rot even, at most 256; scaling [host]
 * may be NULL (plain, magnitude 1). */
int gptq_rope_table(gptq_ctx ctx, int32_t length, int32_t rot, double base, const gptq_rope_scaling* scaling,
                    float* table);

/* Rotary positions: every pair (a, b) of the first rot of dim values of
 * x[tokens][heads][dim] becomes (a c - b s, b c + a s) with c, s from the
 * table's row positions[token]; the other values are copied.  inverse != 0
 * turns back (s negated), which is also the gradient.  fp32 arithmetic,
 * rounded once to y's type.  A position outside 0..length-1 gives NaN in the
 * rotated part.  y may be x itself (same type and strides), else they must
 * not overlap.  rot and dim even; rot == 0 copies. */
int gptq_rope(gptq_ctx ctx, const void* x, int32_t x_type, int64_t tokens, int32_t heads, int32_t dim,
              int64_t x_token, int64_t x_head, const int32_t* positions, const float* table, int32_t length,
              int32_t rot, int32_t layout, int32_t inverse, void* y, int32_t y_type, int64_t y_token,
              int64_t y_head);

/* A paged key/value cache on min-max grids of 4 or 8 bits.  A slot is
 * page_number * page + offset.  With rb = dim bits / 8:
 *   k_codes[pages][heads][page][rb]: a token's codes side by side (4 bits:
 *     code 2i in the low half of byte i, code 2i + 1 in the high half, as
 *     gptq_pack_codes packs a row);
 *   v_codes[pages][heads][rb][page]: the tokens of a page side by side (4
 *     bits: byte row j holds dimension j in the low half, j + dim/2 in the high);
 *   scales fp32 and zeros uint8 [pages][heads][page]: one grid for every
 *     (token, head) of K and of V, value = scale * (code - zero).
 * dim 64, 96, 128, 192 or 256; page a power of two from 16 to 256; pages * page
 * < 2^31; buffers 16-byte aligned. */
typedef struct {
  uint8_t* k_codes;
  float* k_scales;
  uint8_t* k_zeros;
  uint8_t* v_codes;
  float* v_scales;
  uint8_t* v_zeros;
  int32_t pages, heads, page, dim, bits;
  int32_t pad0;
} gptq_kv_cache;

/* Quantise K[tokens][heads][dim] and V into the cache: token t goes to
 * slots[t] (a slot outside the pool: the token is skipped; the same slot
 * twice in one call: undefined contents).  Per row v, in fp32 steps: lo = min(min v,
 * 0), hi = max(max v, 0), s = fl32(hi - lo) fl32(1/maxq), r = 1/s, z = clamp(rne(-lo
 * r)), q = clamp(rne(fl32(fl32(v r) + z))), as gptq_quantize_lowrank but for the
 * product with 1/maxq in place of its quotient (one rounding of s apart).
 * A range below 2^-100 is stored as zeros (s = 1); a row with a non-finite
 * value, or whose range overflows, reads back as NaN.  Rows aligned to four
 * values (else GPTQ_ERR_UNSUPPORTED). */
int gptq_kv_write(gptq_ctx ctx, const gptq_kv_cache* cache, const void* K, const void* V, int32_t type,
                  int64_t tokens, int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head,
                  const int32_t* slots);

/* Read back: K[t], V[t] = fl32(s (q - z)) of slots[t], rounded once to the
 * type; zeros for a slot outside the pool.  Alignment as gptq_kv_write. */
int gptq_kv_read(gptq_ctx ctx, const gptq_kv_cache* cache, const int32_t* slots, int64_t tokens, void* K,
                 void* V, int32_t type, int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head);

/* Attention of the drafted tokens of every sequence over its cache:
 *   O[b][t][hq] = sum_j softmax_j(scale Q[b][t][hq] . Khat[j]) Vhat[j]
 * over the positions j of sequence b that token t sees: all j < lengths[b]
 * (the tokens before the drafted ones), and of the drafted tokens, which lie
 * at positions lengths[b] .. lengths[b] + tokens - 1, those whose bit is set in
 * mask[b][t][words] (bit i in word i / 32; itself only if its own bit is set),
 * or the first t + 1 without a mask (a chain; tokens = 1: one next token).
 * Position j lies in page tables[b][j / page].  Positions past the table's
 * width and those whose page number is outside the pool are not seen; a row
 * that sees nothing is zero, as is every row of a sequence with lengths < 0.
 * Query head hq reads cache head hq / (heads / cache.heads).  Q and O bf16
 * bits; scores, softmax and sums in fp32 (see the kernel for its operands).
 * Any finite queries and scale; keys and values of at most 2^100 in magnitude (the
 * sums of larger ones may pass fp32's range), zero points at most 2^bits - 1.
 * Rows of Q 16-byte aligned, rows of O 8-byte aligned; width * page <= 2^29; at
 * most 2^26 rows (token, head) of a sequence and 2^23 .. 2^24 workgroups in all
 * (GPTQ_ERR_UNSUPPORTED). */
int gptq_tree_attention(gptq_ctx ctx, const gptq_kv_cache* cache, const uint16_t* Q, int32_t seqs, int32_t tokens,
                        int32_t heads, int64_t q_seq, int64_t q_token, int64_t q_head, const int32_t* tables,
                        int32_t width, const int32_t* lengths, const uint32_t* mask, int32_t words, float scale,
                        uint16_t* O, int64_t o_seq, int64_t o_token, int64_t o_head);

/* Many requests on one quantised layer, each with a low-rank adapter of its own
 * (or none):
 *   Y[m][.] = X[m][.] What^T + alpha[a] (X[m][.] down[a]^T) up[a]^T, a = ids[m]
 * with What as in gptq_gemm_wqa16 (the same operands and requirements), down
 * [count][rank][K] and up[count][N][rank] bf16 bits, alpha[count] fp32 (NULL: 1),
 * ids[M] int32 (outside 0..count-1: a row without an adapter).  fp32 sums; X down^T
 * enters the second product as three bf16 numbers, which hold all of it.  What a row's
 * adapter holds reaches no other row.  Rows in any order; those of an adapter side
 * by side are fastest.  rank a multiple of 8, at most 128 (0: the product alone);
 * N at most 2^26, and no launch of 2^32 threads (weights or a Y of some 256 GB);
 * 16-byte aligned rows of X, codes and adapters (GPTQ_ERR_UNSUPPORTED).
 * Needs workspace, as gptq_tree_attention: run once before a capture.  Above 128 rows that
 * is a bf16 copy of the whole layer, 2 N K bytes (1 GB for 128256 x 4096), and up to
 * 150 MB of sums where several workgroups have a tile; for fewer rows 2 M K; and 4 to 16 M
 * rank bytes (M at most 16384).  The context keeps the largest so far, or twice the one
 * before it, and what it has outgrown, until gptq_destroy. */
typedef struct {
  const uint16_t* down;
  const uint16_t* up;
  const float* alpha;
  int32_t count, rank;
} gptq_adapters;

int gptq_gemm_adapters(gptq_ctx ctx, const uint16_t* X, int64_t M, int64_t ldx, const uint32_t* packed,
                       const float* scales, const uint8_t* zeros, int32_t N, int32_t K, int32_t group, int32_t bits,
                       const gptq_adapters* adapters, const int32_t* ids, float* Y, int64_t ldy);

/* P[b][t][v] = softmax over v of logits[b][t][v] / temperature[b], fp32, from
 * bf16 or fp32 logits; temperature[seqs] fp32 (NULL: 1).  Temperature 0: 1 at the
 * first maximum, 0 elsewhere.  A row of -infinity alone is zero; a row with a NaN,
 * with +infinity (temperature above 0), or whose temperature is negative or not
 * finite is NaN.  Strides in elements, the vocabulary contiguous; P must not
 * overlap the logits, nor its rows each other (one stride at least vocab, the other past
 * all rows of the first: GPTQ_ERR_INVALID_ARG).  vocab at most 2^22. */
int gptq_probabilities(gptq_ctx ctx, const void* logits, int32_t type, int64_t seqs, int32_t tokens, int32_t vocab,
                       int64_t x_seq, int64_t x_token, const float* temperature, float* P, int64_t p_seq,
                       int64_t p_token);

/* Drafted tokens of every sequence against the target's probabilities, from
 * given random numbers.  Node 0 is the last token that is certain, node i > 0 the
 * drafted token draft[b][i] below node parents[b][i] (a smaller index; any other
 * number: the node is not there; parents NULL: a chain, i below i - 1); P[b][i] is
 * the target's distribution after node i, Q[b][i] the draft's, which the children
 * of i were drawn from independently (Q NULL: they were chosen, not drawn).
 * From node c = 0 on, with r = P[b][c] and R = 1, the children x of c in the order
 * of their indexes: x is accepted if uniforms[b][i] Q(x) R < r(x), and the walk goes
 * on from it; otherwise r = max(r - R Q, 0) and R = sum r (without Q the test is
 * uniforms[b][i] R < r(x), then R -= r(x), r(x) = 0).  Where no child is accepted,
 * next[b] is the first v at which the sum of r up to v passes uniforms[b][0] times
 * the whole (the last v with r > 0 if none does, as with a number from 1 on or NaN;
 * r = P[b][c] if nothing is left of it; -1 if that is empty).  path[b]: the nodes of
 * the walk from 0 on, then -1; counts[b]: how many.  64-bit sums.  Probabilities below
 * 0 or NaN count as 0; a drafted token outside the vocabulary is not there.  tokens at
 * most 1024, vocab at most 2^20 (GPTQ_ERR_UNSUPPORTED).  Needs workspace, as
 * gptq_tree_attention. */
int gptq_verify_draft(gptq_ctx ctx, const float* P, int64_t p_seq, int64_t p_token, const float* Q, int64_t q_seq,
                      int64_t q_token, int32_t seqs, int32_t tokens, int32_t vocab, const int32_t* draft,
                      const int32_t* parents, const float* uniforms, int32_t* path, int32_t* counts, int32_t* next);

/* The accepted tokens' keys and values brought together: of sequence b the token
 * at position lengths[b] + path[b][j] goes to position lengths[b] + j, j <
 * counts[b] (path and counts as gptq_verify_draft gives them).  path[b] rises; the
 * tokens from the first entry on that does not, or is outside 0..tokens-1, stay. So
 * does a token whose old or new position lies past the table or outside the pool.  A
 * page that two sequences hold must not be moved in (undefined contents). */
int gptq_kv_compact(gptq_ctx ctx, const gptq_kv_cache* cache, const int32_t* tables, int32_t seqs, int32_t width,
                    const int32_t* lengths, const int32_t* path, int32_t tokens, const int32_t* counts);

/* Whole pages copied, src[i] to dst[i]; a pair with a number outside the pool is
 * skipped.  A page twice in dst, or in dst and in src: undefined contents. */
int gptq_kv_copy(gptq_ctx ctx, const gptq_kv_cache* cache, const int32_t* src, const int32_t* dst, int64_t n);

/* Page tables over reference counts, shared by the caches of all layers:
 * tables[seqs][width] page numbers (outside 0..pages-1: none), refs[pages] how many
 * entries name a page; a page with refs <= 0 is free.  Counts that do not agree with
 * the tables give pages to two owners, but no access outside the buffers.
 *
 * gptq_pages_free: entries past the pages of the first lengths[b] tokens are given
 * back (lengths[b] <= 0: all) and become -1.
 * gptq_pages_fork: row dst[i] gives its pages back and takes those of the first
 * lengths[src[i]] tokens of row src[i], which both hold from then on.  A pair with a
 * row outside 0..seqs-1 is left out, and so is one whose dst is a source of the call
 * or the dst of an earlier pair.  At most 65536 pairs.
 * gptq_pages_extend: room for added[b] tokens past the first lengths[b] of every
 * sequence (added[b] <= 0 or lengths[b] < 0: none).  An entry of that range without
 * a page gets one; one whose page others hold too gets one in its place, except
 * the last of the page's holders, in the tables' order, where all of them are
 * in the call.  The new pages are the lowest free ones, in the order of the entries.  Where a
 * replaced page holds some of the first lengths[b] tokens, copies[0][b] and
 * copies[1][b] (int32 [2][seqs]) are its number and the new page's, for gptq_kv_copy
 * on every layer's cache; otherwise -1.  info[0]: pages taken; info[1]: pages
 * lacking (free ones, or entries of a table); if any are, nothing changes.  At most
 * 8192 sequences.  Needs workspace, as gptq_tree_attention.
 * page: tokens of a page, a power of two from 16 to 256; seqs * width <= 2^30. */
int gptq_pages_free(gptq_ctx ctx, int32_t* refs, int32_t pages, int32_t* tables, int32_t seqs, int32_t width,
                    const int32_t* lengths, int32_t page);
int gptq_pages_fork(gptq_ctx ctx, int32_t* refs, int32_t pages, int32_t* tables, int32_t seqs, int32_t width,
                    const int32_t* lengths, const int32_t* src, const int32_t* dst, int32_t n, int32_t page);
int gptq_pages_extend(gptq_ctx ctx, int32_t* refs, int32_t pages, int32_t* tables, int32_t seqs, int32_t width,
                      const int32_t* lengths, const int32_t* added, int32_t page, int32_t* copies, int32_t* info);

/* Measurement support (not part of the method).  gptq_timing(ctx, kernels)
 * clears the totals and from then on brackets each launch of the named
 * kernels with a pair of HIP events on the context's stream.  kernels [host]
 * is a comma-separated list of kernel names (e.g. "k_syrk,k_sweep"), "*" for
 * every kernel the context launches, or NULL to stop recording (totals are
 * kept until the next gptq_timing call).  Kernel names: k_xpose, k_syrk,
 * k_syrk_reduce, k_syrk64, k_syrk64_reduce, k_damp_lambda, k_damp_fill,
 * k_chol_panel, k_chol_panel2, k_gemm64, k_gemm_ring64, k_gemm_ring128,
 * k_make_u, k_init_work, k_rowfit, k_sweep, k_trail, k_objective, and for the
 * LoRA and refinement paths k_lora_lambda, k_start_block, k_dgemm, k_dsum,
 * k_gram_chol, k_apply, k_lora_assemble, k_lora_extract, k_ref_init, k_resid,
 * k_gfinal, k_sum_parts, k_f32_to_f64, k_f64_to_f32, k_olrc_out, and for the
 * two-sided rounding k_r2d_unit, k_r2d_fill, k_r2d_tile, k_r2d_push, k_r2d_obj,
 * and for the quantised-input target k_qr_prep, k_qr_out, and for the
 * deployable outputs k_pack, k_unpack, k_lr_quant, k_gemm_w4a16,
 * k_gemv_w4a16 (4-bit codes), k_gemm_wqa16, k_gemv_wqa16 (other widths), and
 * for the serving operators k_rope_table, k_rope, k_kv_write, k_kv_read,
 * k_tree_attn, k_tree_attn_wide, k_attn_join, k_adapt_down, k_adapt_rows, k_adapt_tile,
 * k_probs, k_verify, k_kv_compact, k_kv_copy, k_pages_free, k_pages_fork, k_pages_extend.
 * gptq_kernel_time
 * waits for the recorded events and returns the summed elapsed milliseconds
 * and the number of timed launches of kernel `name` (0 and 0 if none).  Each
 * timed launch costs two event records on the stream. */
int gptq_timing(gptq_ctx ctx, const char* kernels);
int gptq_kernel_time(gptq_ctx ctx, const char* name, double* total_ms, int64_t* launches);

#ifdef __cplusplus
}
#endif

#endif /* GPTQ_MI355X_H */
