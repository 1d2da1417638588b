// mx_api.cpp -- host side of include/wqbmm_mxfp4.h: argument validation, the
// choice of kernels, workspace.  Checks come in the order null pointer ->
// shape -> support, before any device call; nothing throws.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <mutex>

#include "../../include/wqbmm_mxfp4.h"
#include "mx_launch.hpp"

namespace {

using namespace wqbmm;

constexpr int64_t kMaxRows = int64_t(1) << 24;
constexpr int64_t kMaxK = int64_t(1) << 20;

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool good_k(int64_t K) { return K > 0 && K <= kMaxK && K % kMxBlock == 0; }
bool good_rows(int64_t M) { return M >= 0 && M <= kMaxRows; }
// The largest row distance keeps every byte offset within 64 bits.
bool good_ld(int64_t ld, int64_t K) { return ld >= K && ld % 8 == 0 && ld <= (int64_t(1) << 36); }
bool is_dtype(int d) { return d == WQBMM_DTYPE_F16 || d == WQBMM_DTYPE_BF16 || d == WQBMM_DTYPE_F32; }
bool is_16bit(int d) { return d == WQBMM_DTYPE_F16 || d == WQBMM_DTYPE_BF16; }

wqbmm_status status_of(hipError_t e) { return e == hipSuccess ? WQBMM_OK : WQBMM_ERR_LAUNCH; }

}  // namespace

extern "C" {

wqbmm_status wqbmm_mxfp4_quantize(const void* x, int dtype, int64_t M, int64_t K, int64_t ldx, void* codes,
                                  void* scales, void* stream) {
  if (M != 0 && (!x || !codes || !scales)) return WQBMM_ERR_NULLPTR;
  if (!good_rows(M) || !good_k(K) || !good_ld(ldx, K)) return WQBMM_ERR_INVALID;
  if (!aligned(x) || !aligned(codes) || !aligned(scales)) return WQBMM_ERR_INVALID;
  if (!is_dtype(dtype)) return WQBMM_ERR_UNSUPPORTED;
  if (M == 0) return WQBMM_OK;
  int dev = -1;
  const wqbmm_status st = host_check_device(&dev);
  if (st != WQBMM_OK) return st;
  return status_of(launch_mx_quantize(x, dtype, M, K, ldx, codes, scales, static_cast<hipStream_t>(stream)));
}

wqbmm_status wqbmm_mxfp4_dequantize(const void* codes, const void* scales, int64_t M, int64_t K, void* y, int dtype,
                                    int64_t ldy, void* stream) {
  if (M != 0 && (!codes || !scales || !y)) return WQBMM_ERR_NULLPTR;
  if (!good_rows(M) || !good_k(K) || !good_ld(ldy, K)) return WQBMM_ERR_INVALID;
  if (!aligned(codes) || !aligned(scales) || !aligned(y)) return WQBMM_ERR_INVALID;
  if (!is_dtype(dtype)) return WQBMM_ERR_UNSUPPORTED;
  if (M == 0) return WQBMM_OK;
  int dev = -1;
  const wqbmm_status st = host_check_device(&dev);
  if (st != WQBMM_OK) return st;
  return status_of(launch_mx_dequantize(codes, scales, M, K, y, dtype, ldy, static_cast<hipStream_t>(stream)));
}

int64_t wqbmm_mxfp4_tiled_weight_bytes(int64_t K, int64_t N) {
  if (!good_k(K) || N < 1 || N > kMaxRows) return -1;
  return (int64_t)mx_tiled_bytes(K, N);
}

wqbmm_status wqbmm_mxfp4_tile_weights(const void* codes, const void* scales, int64_t K, int64_t N, void* w_tiled,
                                      void* stream) {
  if (!codes || !scales || !w_tiled) return WQBMM_ERR_NULLPTR;
  if (wqbmm_mxfp4_tiled_weight_bytes(K, N) < 0) return WQBMM_ERR_INVALID;
  if (!aligned(codes) || !aligned(scales) || !aligned(w_tiled)) return WQBMM_ERR_INVALID;
  int dev = -1;
  const wqbmm_status st = host_check_device(&dev);
  if (st != WQBMM_OK) return st;
  return status_of(launch_mx_tile(codes, scales, K, N, w_tiled, static_cast<hipStream_t>(stream)));
}

wqbmm_status wqbmm_mxfp4_matmul(const void* x, int dtype, int64_t ldx, const void* w_tiled, int64_t M, int64_t K,
                                int64_t N, void* y, int act, void* stream) {
  if ((M != 0 && (!x || !y)) || !w_tiled) return WQBMM_ERR_NULLPTR;
  if (!good_rows(M) || wqbmm_mxfp4_tiled_weight_bytes(K, N) < 0 || !good_ld(ldx, K)) return WQBMM_ERR_INVALID;
  if (!aligned(x) || !aligned(w_tiled) || !aligned(y)) return WQBMM_ERR_INVALID;
  if (act != WQBMM_MXFP4_ACT_16BIT && act != WQBMM_MXFP4_ACT_MXFP4) return WQBMM_ERR_INVALID;
  if (!is_16bit(dtype)) return WQBMM_ERR_UNSUPPORTED;
  if (M == 0) return WQBMM_OK;
  int dev = -1;
  wqbmm_status st = host_check_device(&dev);
  if (st != WQBMM_OK) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const MxTiled w = mx_view(w_tiled, K, N);
  if (mx_use_gemv(M, K, N)) return status_of(launch_mx_gemv(x, dtype, ldx, w, M, K, N, y, act, s));
  if (!act && ldx >= kMxGemmMaxLd) {     // the tiled product addresses a tile of x with 31 bits
    for (int64_t m = 0; m < M; m += kMxGemvMaxM) {
      const hipError_t e = launch_mx_gemv(static_cast<const char*>(x) + m * ldx * 2, dtype, ldx, w,
                                          M - m < kMxGemvMaxM ? M - m : kMxGemvMaxM, K, N,
                                          static_cast<char*>(y) + m * N * 2, act, s);
      if (e != hipSuccess) return status_of(e);
    }
    return WQBMM_OK;
  }
  const MxGemmPlan plan = act ? mx_gemm4_plan(M, K, N) : mx_gemm16_plan(M, K, N);
  uint8_t* ws = nullptr;
  std::unique_lock<std::mutex> held;
  st = host_workspace(dev, s, plan.x_bytes + plan.part_bytes, &ws, &held);
  if (st != WQBMM_OK) return st;
  return status_of(act ? launch_mx_gemm4(x, dtype, ldx, w, M, K, N, y, plan, ws, s)
                       : launch_mx_gemm16(x, dtype, ldx, w, M, K, N, y, plan, ws, s));
}

wqbmm_status wqbmm_mxfp4_moe(const void* x, int dtype, int64_t ldx, int64_t T, int64_t H, int64_t I, int64_t E,
                             int64_t k, int renormalize, const void* router, const void* gate_up, const void* down,
                             void* y, int32_t* topk_ids, float* topk_weights, void* stream) {
  if ((T != 0 && (!x || !y || !topk_ids || !topk_weights)) || !router || !gate_up || !down) return WQBMM_ERR_NULLPTR;
  if (T < 0 || T > kMoeMaxT || !good_k(H) || !good_k(I) || !good_ld(ldx, H)) return WQBMM_ERR_INVALID;
  if (E < 1 || E > kMoeMaxE || k < 1 || k > kMoeMaxK || k > E) return WQBMM_ERR_INVALID;
  if (E * 2 * I > kMaxRows || E * H > kMaxRows) return WQBMM_ERR_INVALID;
  if (!aligned(x) || !aligned(router) || !aligned(gate_up) || !aligned(down) || !aligned(y) || !aligned(topk_ids) ||
      !aligned(topk_weights))
    return WQBMM_ERR_INVALID;
  if (!is_16bit(dtype)) return WQBMM_ERR_UNSUPPORTED;
  if (T == 0) return WQBMM_OK;
  int dev = -1;
  wqbmm_status st = host_check_device(&dev);
  if (st != WQBMM_OK) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t* ws = nullptr;
  std::unique_lock<std::mutex> held;
  st = host_workspace(dev, s, mx_moe_workspace_bytes(T, H, I, k), &ws, &held);
  if (st != WQBMM_OK) return st;
  return status_of(launch_mx_moe(x, dtype, ldx, T, H, I, E, k, renormalize != 0, router, mx_view(gate_up, H, E * 2 * I),
                                 mx_view(down, I, E * H), y, topk_ids, topk_weights, ws, s));
}

}  // extern "C"
