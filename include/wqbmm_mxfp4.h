/*
 * wqbmm_mxfp4.h -- C ABI of the microscaled 4-bit floating-point (MXFP4)
 * operators: quantising and reading back, the product with MXFP4 weights, and
 * a mixture-of-experts layer with MXFP4 experts for a few tokens.
 *
 * Format.  32 consecutive values along K (a block) share one scale byte s that
 * stands for 2^(s - 127); s = 255 makes the whole block NaN.  An element is 4
 * bits: sign, two exponent bits, one mantissa bit; its magnitude is one of
 * 0, 0.5, 1, 1.5, 2, 3, 4, 6 (codes 0..7), and bit 3 is the sign.  A matrix of
 * rows x K is
 *   codes   uint8 [rows][K/2]    element k in the low nibble of byte k/2 if k
 *                                is even, in the high nibble if it is odd
 *   scales  uint8 [rows][K/32]
 *
 * Conventions are those of wqbmm.h: device pointers owned by the caller,
 * arguments checked on the host in the order null pointer -> shape ->
 * support before any launch, all work asynchronous on `stream`, workspace per
 * (device, stream) with the same growth and capture rules, deterministic
 * results, gfx950 only.  Further rules here:
 *   - K (and every other contracted length) is a positive multiple of 32, at
 *     most 2^20; rows and columns are any number from 1 to 2^24 (rows of x: 0
 *     is a no-op, and the arrays with that extent may then be NULL).
 *   - dtype is a wqbmm_dtype; 16-bit inputs have outputs of the same type.
 *   - ld* is the distance between rows in elements: at least the row length
 *     and a multiple of 8; every pointer is 16-byte aligned.
 *   - Infinities and NaN are followed: they give what the formulas give.
 *   - Weights of 2^128 and more (4 and 6 at scale 253, 2 and more at 254: fp32
 *     does not hold them either, and wqbmm_mxfp4_quantize makes none) are
 *     beyond the products with 16-bit x and the expert layer: what they are
 *     multiplied into comes out infinite or NaN, as if they were infinite.
 */
#ifndef WQBMM_MXFP4_H
#define WQBMM_MXFP4_H

#include <stdint.h>

#include "wqbmm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum wqbmm_dtype {
  WQBMM_DTYPE_F16 = 0,
  WQBMM_DTYPE_BF16 = 1,
  WQBMM_DTYPE_F32 = 2        /* quantize and dequantize only */
} wqbmm_dtype;

/* How wqbmm_mxfp4_matmul takes its activations. */
typedef enum wqbmm_mxfp4_act {
  WQBMM_MXFP4_ACT_16BIT = 0, /* as they are                                       */
  WQBMM_MXFP4_ACT_MXFP4 = 1  /* quantised as wqbmm_mxfp4_quantize does, in the call */
} wqbmm_mxfp4_act;

/*
 * x [M][K] (rows ldx apart; F16, BF16 or F32) -> codes [M][K/2], scales
 * [M][K/32].  Per block: s - 127 = floor(log2(max|x|)) - 2, kept in
 * [-127, 127]; each value is divided by 2^(s - 127), rounded half to even to
 * the eight magnitudes and clipped at 6.  A block of zeros has s = 0; a block
 * that holds an infinity or a NaN has s = 255 and codes 0.
 */
wqbmm_status wqbmm_mxfp4_quantize(const void* x, int dtype, int64_t M, int64_t K, int64_t ldx,
                                  void* codes, void* scales, void* stream);

/* codes, scales -> y [M][K] (rows ldy apart; F16, BF16 or F32): the values
 * that they stand for, rounded once (half to even) where the type needs it. */
wqbmm_status wqbmm_mxfp4_dequantize(const void* codes, const void* scales, int64_t M, int64_t K,
                                    void* y, int dtype, int64_t ldy, void* stream);

/*
 * Weights W [N][K] (row n holds output column n's weights) in codes and
 * scales -> the tiled form that the products read, once per weight.  Its
 * layout is internal.  A stack of E expert matrices with N % 16 == 0 is tiled
 * as one matrix of E*N rows.  wqbmm_mxfp4_tiled_weight_bytes: its size, or -1
 * if K or N breaks the rules (host only).
 */
int64_t wqbmm_mxfp4_tiled_weight_bytes(int64_t K, int64_t N);
wqbmm_status wqbmm_mxfp4_tile_weights(const void* codes, const void* scales, int64_t K, int64_t N,
                                      void* w_tiled, void* stream);

/*
 * y [M][N] = x [M][K] . W^T, F16 or BF16, sums in fp32, rounded once.
 * act = WQBMM_MXFP4_ACT_16BIT: the products x*w are exact (|w| < 2^128).
 * act = WQBMM_MXFP4_ACT_MXFP4: x is first quantised to MXFP4.
 */
wqbmm_status wqbmm_mxfp4_matmul(const void* x, int dtype, int64_t ldx, const void* w_tiled,
                                int64_t M, int64_t K, int64_t N, void* y, int act, void* stream);

/*
 * A mixture-of-experts layer for T <= 64 tokens.
 *   x            [T][H], F16 or BF16 (rows ldx apart)
 *   router       [E][H], x's type, contiguous
 *   gate_up      tiled weights of E * 2I rows of H: per expert I gate rows,
 *                then I up rows
 *   down         tiled weights of E * H rows of I
 *   y            [T][H], x's type
 *   topk_ids     int32 [T][k], topk_weights fp32 [T][k]: outputs
 * Per token: logits = router . x (fp32); the k experts with the largest
 * logits (ties to the lowest index; a NaN counts as the largest); their
 * softmax probabilities over all E experts, divided by their sum if
 * renormalize != 0; y = sum over them of weight * down_e . (silu(gate_e . x)
 * * (up_e . x)).  Intermediate values keep fp32's 24 bits.
 * Rules: H, I multiples of 32; 1 <= E <= 256; 1 <= k <= min(E, 16);
 * E * 2I and E * H at most 2^24.  More tokens: WQBMM_ERR_INVALID.
 */
wqbmm_status wqbmm_mxfp4_moe(const void* x, int dtype, int64_t ldx, int64_t T, int64_t H, int64_t I,
                             int64_t E, int64_t k, int renormalize, const void* router,
                             const void* gate_up, const void* down, void* y, int32_t* topk_ids,
                             float* topk_weights, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* WQBMM_MXFP4_H */
