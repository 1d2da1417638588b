// mx_gemv.hip -- the product with MXFP4 weights for few rows of x (M <= 64):
// y[m][n] = sum_k x[m][k] * w[n][k], the weights streamed once.
//
// A workgroup owns P panels of 16 output columns and all of K; its eight waves
// take the quads of K-tiles (512 k) in turn, each with its own fp32 MFMA
// accumulators, which are added over the waves in wave order through LDS.  A
// lane's 16-byte chunk of a tile is the block l/16 of row l%16, so
//   * 16-bit x: the chunk's four dwords convert to four operands of
//     v_mfma_f32_16x16x32 (8 consecutive k of each of four blocks per
//     instruction; both operands use the same k), the block's scale applied by
//     the conversion, which is exact in bf16 for every scale;
//   * MXFP4 x: the lane holds the whole block l/16 of x's row l%16 as well, so
//     it quantises it in registers (no preparation kernel), and the chunk is
//     the scaled MFMA's operand as it is.
// fp16 x: where every weight of the workgroup's panels is exact in fp16
// (flags, practically always) the products run in fp16; otherwise x is split
// into two exact bf16 parts, at twice the MFMAs.
#include <algorithm>

#include "mx_device.hpp"
#include "mx_launch.hpp"

namespace wqbmm {

namespace {
constexpr int GEMV_WAVES = 8;

enum class Mode { kDirect, kSplit, kMxfp4 };

__device__ __forceinline__ uint32_t dword_of(const uint4& v, int j) {
  return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
}
}  // namespace

template <int DT>
__device__ __forceinline__ void mx_store4(uint16_t* __restrict__ y, int64_t m, int64_t n, int64_t N, mx_f4 v) {
  uint16_t* p = y + m * N + n;
  if ((N & 3) == 0) {                       // then n + 3 < N, and the store is aligned
    const uint32_t lo = mx_round16<DT>(v[0]) | ((uint32_t)mx_round16<DT>(v[1]) << 16);
    const uint32_t hi = mx_round16<DT>(v[2]) | ((uint32_t)mx_round16<DT>(v[3]) << 16);
    *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) p[i] = mx_round16<DT>(v[i]);
  }
}

template <int DT, Mode MODE, int MT, int P>
__device__ __forceinline__ void gemv_quads(const uint16_t* __restrict__ x, int64_t ldx, const MxTiled& w, int p0,
                                           int M, int blocks, int wave, int lane, mx_f4 (&acc)[P][MT]) {
  const int r = lane & 15, g = lane >> 4;
  for (int q = wave; q < w.kq; q += GEMV_WAVES) {
    uint4 c[P][4];
    uint32_t sc[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int64_t pp = min(p0 + p, w.panels - 1);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c[p][i] = *reinterpret_cast<const uint4*>(
            w.codes + ((pp * w.kt + min(4 * q + i, w.kt - 1)) * 64 + lane) * 16);
      sc[p] = *reinterpret_cast<const uint32_t*>(w.scales + ((pp * w.kq + q) * 64 + lane) * 4);
    }
    auto tile = [&](auto ic) {
      constexpr int i = decltype(ic)::value;
      if (4 * q + i >= w.kt) return;                  // uniform: the last quad's missing tiles
      const int b = 4 * (4 * q + i) + g;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int m = mt * 16 + r;
        uint4 xv[4] = {};
        if (m < M && b < blocks) {
          const uint4* src = reinterpret_cast<const uint4*>(x + m * ldx + (int64_t)b * kMxBlock);
#pragma unroll
          for (int j = 0; j < 4; ++j) xv[j] = src[j];
        }
        if constexpr (MODE == Mode::kMxfp4) {
          uint32_t top = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) top = mx_max16(xv[j], top);
          const uint32_t s = mx_scale_byte(mx_top_bits<DT>(mx_max16_fold(top)));
          const float f = mx_scale(s);
          const uint4 e = make_uint4(mx_encode8<DT>(xv[0], f), mx_encode8<DT>(xv[1], f), mx_encode8<DT>(xv[2], f),
                                     mx_encode8<DT>(xv[3], f));
#pragma unroll
          for (int p = 0; p < P; ++p) acc[p][mt] = mx_mfma4<i, 0>(c[p][i], sc[p], e, s, acc[p][mt]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint4 hi, lo;
            if constexpr (MODE == Mode::kSplit) mx_split8(xv[j], hi, lo);
#pragma unroll
            for (int p = 0; p < P; ++p) {
              const float f = mx_scale((sc[p] >> (8 * i)) & 0xffu);
              if constexpr (MODE == Mode::kSplit) {
                const uint4 a = mx_decode8<MX_BF16>(dword_of(c[p][i], j), f);
                acc[p][mt] = mx_mfma16<MX_BF16>(a, hi, acc[p][mt]);
                acc[p][mt] = mx_mfma16<MX_BF16>(a, lo, acc[p][mt]);
              } else {
                acc[p][mt] = mx_mfma16<DT>(mx_decode8<DT>(dword_of(c[p][i], j), f), xv[j], acc[p][mt]);
              }
            }
          }
        }
      }
    };
    tile(std::integral_constant<int, 0>{});
    tile(std::integral_constant<int, 1>{});
    tile(std::integral_constant<int, 2>{});
    tile(std::integral_constant<int, 3>{});
  }
}

template <int DT, bool ACT4, int MT, int P>
__global__ __launch_bounds__(GEMV_WAVES * 64) void mx_gemv_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                                 MxTiled w, int M, int blocks, int64_t N,
                                                                 uint16_t* __restrict__ y) {
  __shared__ mx_f4 part[GEMV_WAVES][P * MT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int p0 = blockIdx.x * P;
  mx_f4 acc[P][MT];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[p][mt] = mx_f4{0.f, 0.f, 0.f, 0.f};
  if constexpr (ACT4) {
    gemv_quads<DT, Mode::kMxfp4, MT, P>(x, ldx, w, p0, M, blocks, wave, lane, acc);
  } else if constexpr (DT == MX_BF16) {
    gemv_quads<DT, Mode::kDirect, MT, P>(x, ldx, w, p0, M, blocks, wave, lane, acc);
  } else {
    uint32_t flags = kMxFlagF16;
#pragma unroll
    for (int p = 0; p < P; ++p) flags &= w.flags[min(p0 + p, w.panels - 1)];
    if (flags & kMxFlagF16) gemv_quads<DT, Mode::kDirect, MT, P>(x, ldx, w, p0, M, blocks, wave, lane, acc);
    else gemv_quads<DT, Mode::kSplit, MT, P>(x, ldx, w, p0, M, blocks, wave, lane, acc);
  }
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) part[wave][p * MT + mt][lane] = acc[p][mt];
  __syncthreads();
  for (int t = threadIdx.x; t < P * MT * 64; t += GEMV_WAVES * 64) {
    const int pm = t >> 6;
    mx_f4 v = part[0][pm][lane];
#pragma unroll
    for (int k = 1; k < GEMV_WAVES; ++k) v += part[k][pm][lane];
    const int m = (pm % MT) * 16 + (lane & 15);
    const int64_t n = (int64_t)(p0 + pm / MT) * kMxPanel + 4 * (lane >> 4);
    if (m < M && n < N) mx_store4<DT>(y, m, n, N, v);
  }
}

template <int DT, bool ACT4, int MT>
static hipError_t gemv_mt(const void* x, int64_t ldx, const MxTiled& w, int M, int blocks, int64_t N, void* y,
                          hipStream_t stream) {
  auto* xp = static_cast<const uint16_t*>(x);
  auto* yp = static_cast<uint16_t*>(y);
  return mx_launch(mx_gemv_kernel<DT, ACT4, MT, 1>, dim3((unsigned)w.panels), dim3(GEMV_WAVES * 64), stream, xp, ldx,
                   w, M, blocks, N, yp);
}

template <int DT, bool ACT4>
static hipError_t gemv_dt(const void* x, int64_t ldx, const MxTiled& w, int M, int blocks, int64_t N, void* y,
                          hipStream_t stream) {
  if (M <= 16) return gemv_mt<DT, ACT4, 1>(x, ldx, w, M, blocks, N, y, stream);
  if (M <= 32) return gemv_mt<DT, ACT4, 2>(x, ldx, w, M, blocks, N, y, stream);
  return gemv_mt<DT, ACT4, 4>(x, ldx, w, M, blocks, N, y, stream);
}

hipError_t launch_mx_gemv(const void* x, int dtype, int64_t ldx, const MxTiled& w, int64_t M, int64_t K,
                          int64_t N, void* y, int act, hipStream_t stream) {
  const int m = (int)M, blocks = (int)(K / kMxBlock);
  if (dtype == MX_F16)
    return act ? gemv_dt<MX_F16, true>(x, ldx, w, m, blocks, N, y, stream)
               : gemv_dt<MX_F16, false>(x, ldx, w, m, blocks, N, y, stream);
  return act ? gemv_dt<MX_BF16, true>(x, ldx, w, m, blocks, N, y, stream)
             : gemv_dt<MX_BF16, false>(x, ldx, w, m, blocks, N, y, stream);
}

}  // namespace wqbmm
