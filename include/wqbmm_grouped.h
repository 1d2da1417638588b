/*
 * wqbmm_grouped.h -- C ABI of the operators whose weights depend on the row: the
 * choice of experts, the order of rows by group, products with MXFP4 weights
 * grouped by expert with ragged sizes, the weighted sum of a token's experts,
 * and low-rank adapters of many requests beside a shared projection.
 *
 * A plan says which rows belong to which of G groups (experts, adapters):
 *   offsets  int32 [G + 1], ascending; group g has the places offsets[g] ...
 *            offsets[g + 1] - 1
 *   rows     int32 [S]: the row of x that a place stands for
 * wqbmm_group_rows makes one on the device; nothing of it is read by the host, so
 * one launch serves any distribution of the rows.  A mixture of experts for any number of tokens:
 *   moe_route (logits -> ids, weights), group_rows (ids -> plan, slots),
 *   mxfp4_grouped_matmul (gated: gate and up), mxfp4_grouped_matmul (down),
 *   moe_combine.
 *
 * Conventions are those of wqbmm.h: device pointers owned by the caller, arguments
 * checked on the host in the order null pointer -> shape -> support before any
 * launch, all work asynchronous on `stream`, workspace per (device, stream) with
 * the same growth and capture rules, deterministic results, gfx950 only.  Further
 * rules here:
 *   - Groups G: 1 to 1024.  Places S and rows: at most 2^24.  S * N, T * H and M * N:
 *     at most 2^38.  No rows (T, S or M of 0) is a no-op (but for group_rows, whose
 *     offsets become 0), and arrays with that extent may then be NULL.
 *   - ld* is the distance between rows in elements: at least the row length and
 *     at most 2^36.  Matrices of 16-bit values are 16-byte aligned and their ld a
 *     multiple of 8 where nothing else is said; logits, index arrays and fp32
 *     arrays are aligned to their elements.
 *   - Contracted lengths K are positive multiples of 32, at most 2^20.
 *   - What a plan holds is not trusted with memory: a row outside its matrix is read
 *     nowhere and written nowhere (each call says what becomes of it), and offsets
 *     that descend or lie outside [0, S] make y's values unspecified, no more.
 *   - Infinities and NaN are followed where they are chosen; what is left out
 *     (masked logits, choices of no group, rows of no group) has no effect.  MXFP4
 *     weights of 2^128 and more are beyond the products with 16-bit x (wqbmm_mxfp4.h).
 *   - An output overlaps no input, but for a y that is base.
 */
#ifndef WQBMM_GROUPED_H
#define WQBMM_GROUPED_H

#include <stdint.h>

#include "wqbmm.h"
#include "wqbmm_mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Per token the k experts with the largest logits (ties to the lowest index, -0
 * equal to 0; a NaN counts as the largest) and their softmax probabilities over
 * all E experts, divided by the sum of the chosen ones if renormalize != 0.
 * An expert whose logit is -inf is not chosen: where fewer than k are left, the
 * rest of the token's ids are -1 and their weights 0 (all of them, if its logits
 * are all -inf).
 *   logits   [T][E] F16, BF16 or F32, rows ld apart (any ld >= E)
 *   ids      int32 [T][k], weights fp32 [T][k]: outputs, in descending order
 * 1 <= E <= 1024, 1 <= k <= min(E, 16).
 */
wqbmm_status wqbmm_moe_route(const void* logits, int dtype, int64_t ld, int64_t T, int64_t E, int64_t k,
                             int renormalize, int32_t* ids, float* weights, void* stream);

/*
 * The plan of choices ids [T][k], S = T*k: the choices ordered by group, those of a
 * group by token and choice.  An id outside [0, G) is a choice of no group.
 *   offsets  int32 [G + 1]   offsets[0] = 0; offsets[G]: choices with a group
 *   rows     int32 [S]       rows[place] = token; behind offsets[G] the tokens of
 *                            the choices of no group, in order
 *   slots    int32 [T][k]    the place of each choice, -1 if it has no group
 * k >= 1, T*k <= 2^24.
 */
wqbmm_status wqbmm_group_rows(const int32_t* ids, int64_t T, int64_t k, int64_t G, int32_t* offsets, int32_t* rows,
                              int32_t* slots, void* stream);

/*
 * For each place s of group g: y[s] = W_g . x[rows[s]], sums in fp32, rounded
 * once; gated != 0: y[s] = silu(gate) * up, where gate is the first half of W_g's
 * rows and up the second, both products in fp32.
 *   x        [R][K], F16 or BF16 (rows ldx apart); act as for wqbmm_mxfp4_matmul
 *   rows     int32 [S], or NULL: x's rows are the places (then R >= S)
 *   w_tiled  tiled weights of G * N rows of K (wqbmm_mxfp4_tile_weights); N % 16 ==
 *            0 (gated: 32), G * N <= 2^24
 *   y        [S][N] (gated: [S][N / 2]), x's type.  Places in no group keep
 *            what they held; a place whose row lies outside x gets zeros.
 */
wqbmm_status wqbmm_mxfp4_grouped_matmul(const void* x, int dtype, int64_t ldx, int64_t R, const int32_t* rows,
                                        const int32_t* offsets, int64_t G, int64_t S, int64_t K, int64_t N,
                                        const void* w_tiled, void* y, int act, int gated, void* stream);

/*
 * y[t] = base[t] + the sum over j, in order, of weights[t][j] * z[slots[t][j]], in
 * fp32, rounded once.  A slot outside [0, S) adds nothing; base NULL: 0.
 *   z  [S][H] (rows ldz apart), base and y [T][H] (rows ldb and ldy apart), F16
 *   or BF16; H a multiple of 8, at most 2^20; 1 <= k <= 1024.  y may be base.
 */
wqbmm_status wqbmm_moe_combine(const void* z, int dtype, int64_t ldz, int64_t S, int64_t H, const int32_t* slots,
                               const float* weights, int64_t T, int64_t k, const void* base, int64_t ldb, void* y,
                               int64_t ldy, void* stream);

/*
 * y[m] = base[m] + B_l . (scales[l] * (A_l . x[m])) for each row m of adapter l; rows
 * of none: y[m] = base[m].  Sums and scales[l] * (A_l . x) in fp32, y rounded once.  B
 * multiplies the latter's values with 24 bits (BF16; those below 2^-110 to within
 * 2^-133) or 22 (F16; those more than 2^16 below their row's largest to within 2^-38
 * of it).  scales NULL: 1; base NULL: 0.
 *   x        [M][K], F16 or BF16 (rows ldx apart)
 *   a        [L][r][K], b [L][N][r], x's type, contiguous; r a multiple of 8, at
 *            most 256 (smaller adapters are padded with zeros); L <= 1024
 *   offsets, rows   the plan of wqbmm_group_rows for M ids (k = 1) and L groups.
 *            Each row of x stands in it once; one outside [0, M) is left out.
 *   base, y  [M][N], x's type (rows ldb and ldy apart; any N <= 2^20 and any ld >= N).
 *            y may be base: then rows of no adapter are not touched.
 */
wqbmm_status wqbmm_lora_matmul(const void* x, int dtype, int64_t ldx, int64_t M, int64_t K, int64_t N, int64_t r,
                               int64_t L, const void* a, const void* b, const float* scales, const int32_t* offsets,
                               const int32_t* rows, const void* base, int64_t ldb, void* y, int64_t ldy, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* WQBMM_GROUPED_H */
