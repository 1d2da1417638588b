// grp_api.cpp -- host side of include/wqbmm_grouped.h: argument validation, the
// choice of kernels, workspace.  Checks come in the order null pointer ->
// shape -> support, before any device call; nothing throws.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <mutex>

#include "../../include/wqbmm_grouped.h"
#include "grp_launch.hpp"

namespace {

using namespace wqbmm;

constexpr int64_t kMaxRows = int64_t(1) << 24;
constexpr int64_t kMaxK = int64_t(1) << 20;
constexpr int64_t kMaxLd = int64_t(1) << 36;       // byte offsets stay within 64 bits
constexpr int64_t kMaxResult = int64_t(1) << 38;   // values of a result: tiles are counted in 31 bits

bool aligned(const void* p, int to = 16) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(to - 1)) == 0; }
bool good_k(int64_t K) { return K > 0 && K <= kMaxK && K % kMxBlock == 0; }
bool good_rows(int64_t M) { return M >= 0 && M <= kMaxRows; }
bool good_groups(int64_t G) { return G >= 1 && G <= kMaxGroups; }
bool good_any_ld(int64_t ld, int64_t n) { return ld >= n && ld <= kMaxLd; }
bool good_ld(int64_t ld, int64_t n) { return good_any_ld(ld, n) && ld % 8 == 0; }
bool is_16bit(int d) { return d == WQBMM_DTYPE_F16 || d == WQBMM_DTYPE_BF16; }

wqbmm_status status_of(hipError_t e) { return e == hipSuccess ? WQBMM_OK : WQBMM_ERR_LAUNCH; }

}  // namespace

extern "C" {

wqbmm_status wqbmm_moe_route(const void* logits, int dtype, int64_t ld, int64_t T, int64_t E, int64_t k,
                             int renormalize, int32_t* ids, float* weights, void* stream) {
  if (T != 0 && (!logits || !ids || !weights)) return WQBMM_ERR_NULLPTR;
  if (!good_rows(T) || !good_groups(E) || k < 1 || k > E || k > kRouteMaxK || !good_any_ld(ld, E))
    return WQBMM_ERR_INVALID;
  if (!aligned(logits, dtype == WQBMM_DTYPE_F32 ? 4 : 2) || !aligned(ids, 4) || !aligned(weights, 4))
    return WQBMM_ERR_INVALID;
  if (!is_16bit(dtype) && dtype != WQBMM_DTYPE_F32) return WQBMM_ERR_UNSUPPORTED;
  if (T == 0) return WQBMM_OK;
  int dev = -1;
  const wqbmm_status st = host_check_device(&dev);
  if (st != WQBMM_OK) return st;
  return status_of(launch_route(logits, dtype, ld, T, E, k, renormalize != 0, ids, weights,
                                static_cast<hipStream_t>(stream)));
}

wqbmm_status wqbmm_group_rows(const int32_t* ids, int64_t T, int64_t k, int64_t G, int32_t* offsets, int32_t* rows,
                              int32_t* slots, void* stream) {
  if (!offsets || (T != 0 && (!ids || !rows || !slots))) return WQBMM_ERR_NULLPTR;
  if (!good_rows(T) || k < 1 || k > kMaxRows || T * k > kMaxRows || !good_groups(G)) return WQBMM_ERR_INVALID;
  if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(slots, 4)) return WQBMM_ERR_INVALID;
  int dev = -1;
  wqbmm_status st = host_check_device(&dev);
  if (st != WQBMM_OK) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  uint8_t* ws = nullptr;
  std::unique_lock<std::mutex> held;
  const size_t bytes = group_rows_workspace_bytes(T * k, G);
  if (bytes != 0) {
    st = host_workspace(dev, s, bytes, &ws, &held);
    if (st != WQBMM_OK) return st;
  }
  return status_of(launch_group_rows(ids, T, k, G, offsets, rows, slots, ws, s));
}

wqbmm_status wqbmm_mxfp4_grouped_matmul(const void* x, int dtype, int64_t ldx, int64_t R, const int32_t* rows,
                                        const int32_t* offsets, int64_t G, int64_t S, int64_t K, int64_t N,
                                        const void* w_tiled, void* y, int act, int gated, void* stream) {
  if (!offsets || !w_tiled || (S != 0 && (!x || !y))) return WQBMM_ERR_NULLPTR;
  const int64_t step = gated ? 2 * kMxPanel : kMxPanel;
  if (!good_rows(S) || !good_rows(R) || (S != 0 && R < (rows ? 1 : S)) || !good_k(K) || !good_ld(ldx, K))
    return WQBMM_ERR_INVALID;
  if (!good_groups(G) || N < step || N % step != 0 || N > kMaxRows || G * N > kMaxRows || S * N > kMaxResult)
    return WQBMM_ERR_INVALID;
  if (!aligned(x) || !aligned(w_tiled) || !aligned(y) || !aligned(rows, 4) || !aligned(offsets, 4))
    return WQBMM_ERR_INVALID;
  if (act != WQBMM_MXFP4_ACT_16BIT && act != WQBMM_MXFP4_ACT_MXFP4) return WQBMM_ERR_INVALID;
  if (!is_16bit(dtype)) return WQBMM_ERR_UNSUPPORTED;
  if (S == 0) return WQBMM_OK;
  int dev = -1;
  wqbmm_status st = host_check_device(&dev);
  if (st != WQBMM_OK) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  Grouped a;
  a.x = static_cast<const uint16_t*>(x);
  a.ldx = ldx;
  a.R = R;
  a.rows = rows;
  a.offsets = offsets;
  a.G = (int)G;
  a.S = (int)S;
  a.blocks = (int)(K / kMxBlock);
  a.panels = (int)(N / kMxPanel);
  a.w = mx_view(w_tiled, K, G * N);
  a.y = static_cast<uint16_t*>(y);
  a.n_out = (int)(gated ? N / 2 : N);
  if (!mx_use_grouped_tiles(a, act)) return status_of(launch_mx_grouped_few(a, dtype, act, gated != 0, s));
  if (!act) return status_of(launch_mx_grouped16(a, dtype, gated != 0, s));
  uint8_t* ws = nullptr;
  std::unique_lock<std::mutex> held;
  st = host_workspace(dev, s, mx_grouped4_workspace_bytes(a), &ws, &held);
  if (st != WQBMM_OK) return st;
  return status_of(launch_mx_grouped4(a, dtype, gated != 0, ws, s));
}

wqbmm_status wqbmm_moe_combine(const void* z, int dtype, int64_t ldz, int64_t S, int64_t H, const int32_t* slots,
                               const float* weights, int64_t T, int64_t k, const void* base, int64_t ldb, void* y,
                               int64_t ldy, void* stream) {
  if ((T != 0 && (!slots || !weights || !y)) || (T != 0 && S != 0 && !z)) return WQBMM_ERR_NULLPTR;
  if (!good_rows(T) || !good_rows(S) || k < 1 || k > kMaxGroups || H < 8 || H > kMaxK || H % 8 != 0)
    return WQBMM_ERR_INVALID;
  if (!good_ld(ldz, H) || !good_ld(ldy, H) || (base && !good_ld(ldb, H)) || (base == y && base && ldb != ldy))
    return WQBMM_ERR_INVALID;
  if (T * H > kMaxResult) return WQBMM_ERR_INVALID;
  if (!aligned(z) || !aligned(base) || !aligned(y) || !aligned(slots, 4) || !aligned(weights, 4))
    return WQBMM_ERR_INVALID;
  if (!is_16bit(dtype)) return WQBMM_ERR_UNSUPPORTED;
  if (T == 0) return WQBMM_OK;
  int dev = -1;
  const wqbmm_status st = host_check_device(&dev);
  if (st != WQBMM_OK) return st;
  return status_of(launch_combine(z, dtype, ldz, S, H, slots, weights, T, k, base, ldb, y, ldy,
                                  static_cast<hipStream_t>(stream)));
}

wqbmm_status wqbmm_lora_matmul(const void* x, int dtype, int64_t ldx, int64_t M, int64_t K, int64_t N, int64_t r,
                               int64_t L, const void* a, const void* b, const float* scales, const int32_t* offsets,
                               const int32_t* rows, const void* base, int64_t ldb, void* y, int64_t ldy,
                               void* stream) {
  if (!a || !b || !offsets || (M != 0 && (!x || !rows || !y))) return WQBMM_ERR_NULLPTR;
  if (!good_rows(M) || !good_k(K) || N < 1 || N > kMaxK || M * N > kMaxResult) return WQBMM_ERR_INVALID;
  if (r < 8 || r > kLoraMaxR || r % 8 != 0 || !good_groups(L)) return WQBMM_ERR_INVALID;
  if (!good_ld(ldx, K) || !good_any_ld(ldy, N) || (base && !good_any_ld(ldb, N)) || (base == y && base && ldb != ldy))
    return WQBMM_ERR_INVALID;
  if (!aligned(x) || !aligned(a) || !aligned(b) || !aligned(base) || !aligned(y) || !aligned(scales, 4) ||
      !aligned(offsets, 4) || !aligned(rows, 4))
    return WQBMM_ERR_INVALID;
  if (!is_16bit(dtype)) return WQBMM_ERR_UNSUPPORTED;
  if (M == 0) return WQBMM_OK;
  int dev = -1;
  wqbmm_status st = host_check_device(&dev);
  if (st != WQBMM_OK) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  Lora p;
  p.x = static_cast<const uint16_t*>(x);
  p.ldx = ldx;
  p.M = (int)M;
  p.K = (int)K;
  p.N = (int)N;
  p.r = (int)r;
  p.L = (int)L;
  p.a = static_cast<const uint16_t*>(a);
  p.b = static_cast<const uint16_t*>(b);
  p.scales = scales;
  p.offsets = offsets;
  p.rows = rows;
  p.base = static_cast<const uint16_t*>(base);
  p.ldb = base ? ldb : 0;
  p.y = static_cast<uint16_t*>(y);
  p.ldy = ldy;
  const LoraPlan plan = lora_plan(M, K, r, L);
  uint8_t* ws = nullptr;
  std::unique_lock<std::mutex> held;
  st = host_workspace(dev, s, plan.bytes, &ws, &held);
  if (st != WQBMM_OK) return st;
  return status_of(launch_lora(p, dtype, plan, reinterpret_cast<float*>(ws), s));
}

}  // extern "C"
