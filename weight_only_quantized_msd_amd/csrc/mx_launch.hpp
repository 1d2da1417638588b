// mx_launch.hpp -- internal launcher interface of the MXFP4 operators
// (include/wqbmm_mxfp4.h).  Not part of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <mutex>
#include <type_traits>

#include "../../include/wqbmm.h"

namespace wqbmm {

// ---- tiled MXFP4 matrices ------------------------------------------------------
// Rows go in panels of 16, K in tiles of 128 (4 blocks).  Of panel p and K-tile
// kt, lane l of a wave holds row 16p + l%16, block 4*kt + l/16: its 32 codes
// are the 16 bytes at codes + ((p*KT + kt)*64 + l)*16, exactly the lane's
// operand of v_mfma_scale_f32_16x16x128_f8f6f4.  Its scale is byte kt%4 of the
// dword at scales + ((p*KQ + kt/4)*64 + l)*4, so one dword per lane serves a
// quad of four K-tiles (the instruction picks the byte).  Rows past the end
// and blocks past K hold code 0 and scale 127.  A block of zeros has scale 127
// (which keeps its value), so that the panel's flag below is about values only.
// flags[p] bit 0: every value of the panel is exact in fp16, i.e. each block's
// scale lies in [104, 140] (0.5 * 2^-23 = 2^-24 ... 6 * 2^13 = 49152).
constexpr int kMxPanel = 16;
constexpr int kMxTile = 128;
constexpr int kMxBlock = 32;
constexpr uint32_t kMxFlagF16 = 1;

struct MxTiled {
  const uint8_t* codes;
  const uint8_t* scales;
  const uint32_t* flags;
  int panels, kt, kq;
};

inline int64_t mx_panels(int64_t rows) { return (rows + kMxPanel - 1) / kMxPanel; }
inline int64_t mx_ktiles(int64_t K) { return (K + kMxTile - 1) / kMxTile; }
inline int64_t mx_kquads(int64_t K) { return (mx_ktiles(K) + 3) / 4; }
inline size_t mx_codes_bytes(int64_t K, int64_t rows) { return (size_t)(mx_panels(rows) * mx_ktiles(K)) * 1024u; }
inline size_t mx_scales_bytes(int64_t K, int64_t rows) { return (size_t)(mx_panels(rows) * mx_kquads(K)) * 256u; }
inline size_t mx_flags_bytes(int64_t rows) { return (size_t)((mx_panels(rows) + 3) / 4) * 16u; }
inline size_t mx_tiled_bytes(int64_t K, int64_t rows) {
  return mx_codes_bytes(K, rows) + mx_scales_bytes(K, rows) + mx_flags_bytes(rows);
}
inline MxTiled mx_view(const void* tiled, int64_t K, int64_t rows) {
  const uint8_t* p = static_cast<const uint8_t*>(tiled);
  MxTiled v;
  v.codes = p;
  v.scales = p + mx_codes_bytes(K, rows);
  v.flags = reinterpret_cast<const uint32_t*>(v.scales + mx_scales_bytes(K, rows));
  v.panels = (int)mx_panels(rows);
  v.kt = (int)mx_ktiles(K);
  v.kq = (int)mx_kquads(K);
  return v;
}

// Launches `kernel` and returns this launch's own error (hipGetLastError would
// also hand over an error that an earlier call of the program left behind).
template <typename... P, typename... A>
inline hipError_t mx_launch(void (*kernel)(P...), dim3 grid, dim3 block, hipStream_t stream, A&&... args) {
  void* ptrs[] = {const_cast<void*>(static_cast<const void*>(&args))...};
  static_assert((std::is_same<P, std::remove_cv_t<std::remove_reference_t<A>>>::value && ...),
                "arguments are passed by address: their types are the parameters'");
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, ptrs, 0, stream);
}

hipError_t launch_mx_quantize(const void* x, int dtype, int64_t M, int64_t K, int64_t ldx, void* codes,
                              void* scales, hipStream_t stream);
hipError_t launch_mx_dequantize(const void* codes, const void* scales, int64_t M, int64_t K, void* y,
                                int dtype, int64_t ldy, hipStream_t stream);
hipError_t launch_mx_tile(const void* codes, const void* scales, int64_t K, int64_t N, void* w_tiled,
                          hipStream_t stream);

// Few rows (M <= kMxGemvMaxM): one weight-streaming kernel, x read as it is.
constexpr int64_t kMxGemvMaxM = 64;
bool mx_use_gemv(int64_t M, int64_t K, int64_t N);
hipError_t launch_mx_gemv(const void* x, int dtype, int64_t ldx, const MxTiled& w, int64_t M, int64_t K,
                          int64_t N, void* y, int act, hipStream_t stream);

// More rows: tiled MFMA products, of 16-bit x (mx_gemm16.hip) or of x quantised
// into a tiled matrix in the workspace first (mx_gemm4.hip).
struct MxGemmPlan {
  int variant;                // workgroup tile, an index into the product's MxTileCost
  int64_t mblocks, nblocks;
  int64_t splits, kq_per;     // K-splits (quads of K-tiles each); > 1: fp32 partial sums + a reduction
  size_t x_bytes, part_bytes; // workspace: tiled x, then the partial sums
};
// A workgroup tile and what it takes: us for one K-tile (128 k) of a tile with
// every CU busy, and `fixed` us per round of tiles (first copies, output).
struct MxTileCost {
  int bm, bn;
  double fixed, per_ktile;
};
// The tile and split with the least estimated time: `base` us, then rounds of
// 256 workgroups; a split adds a launch of 2 us and its partial sums' traffic.
MxGemmPlan mx_choose(const MxTileCost* tiles, int count, double base, int64_t M, int64_t K, int64_t N);
constexpr int64_t kMxGemmMaxLd = int64_t(1) << 22;   // rows of 16-bit x are less than this apart
MxGemmPlan mx_gemm16_plan(int64_t M, int64_t K, int64_t N);
MxGemmPlan mx_gemm4_plan(int64_t M, int64_t K, int64_t N);
hipError_t launch_mx_gemm16(const void* x, int dtype, int64_t ldx, const MxTiled& w, int64_t M, int64_t K, int64_t N,
                            void* y, const MxGemmPlan& plan, uint8_t* ws, hipStream_t stream);
hipError_t launch_mx_gemm4(const void* x, int dtype, int64_t ldx, const MxTiled& w, int64_t M, int64_t K, int64_t N,
                           void* y, const MxGemmPlan& plan, uint8_t* ws, hipStream_t stream);
hipError_t launch_mx_reduce(const float* part, int splits, int64_t M, int64_t N, void* y, int dtype,
                            hipStream_t stream);

// The mixture-of-experts layer: routing, gate/up products, down product.
constexpr int kMoeMaxT = 64;
constexpr int kMoeMaxE = 256;
constexpr int kMoeMaxK = 16;
size_t mx_moe_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t k);
hipError_t launch_mx_moe(const void* x, int dtype, int64_t ldx, int64_t T, int64_t H, int64_t I, int64_t E,
                         int64_t k, bool renormalize, const void* router, const MxTiled& gate_up,
                         const MxTiled& down, void* y, int32_t* ids, float* weights, uint8_t* ws,
                         hipStream_t stream);

// Host services of msd_api.cpp: the device check (*dev_out: the current
// device), and `bytes` of the stream's workspace (wqbmm.h's rules), the caller's
// until *held goes: it is kept until the call has made its last launch.  They throw
// nothing.
wqbmm_status host_check_device(int* dev_out) noexcept;
wqbmm_status host_workspace(int dev, hipStream_t stream, size_t bytes, uint8_t** ws,
                            std::unique_lock<std::mutex>* held) noexcept;

}  // namespace wqbmm
