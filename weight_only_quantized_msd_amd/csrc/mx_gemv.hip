// mx_gemv.hip -- the product with MXFP4 weights for few rows of x (M <= 64):
// y[m][n] = sum_k x[m][k] * w[n][k], the weights streamed once.
//
// A workgroup owns P panels of 16 output columns and all of K; its eight waves
// take units of K-tiles in turn, each with its own fp32 MFMA accumulators, which
// are added over the waves in wave order through LDS.  A lane's 16-byte chunk of
// a tile is the block l/16 of row l%16, so
//   * 16-bit x: the chunk's four dwords convert to four operands of
//     v_mfma_f32_16x16x32 (8 consecutive k of each of four blocks per
//     instruction; both operands use the same k), the block's scale applied by
//     the conversion, which is exact in bf16 below 2^128 (beyond, at scales 253
//     and 254, it gives infinities);
//   * MXFP4 x: the lane holds the whole block l/16 of x's row l%16 as well, so
//     it quantises it in registers (no preparation kernel), and the chunk is
//     the scaled MFMA's operand as it is.
// fp16 x: where every weight of the workgroup's panels is exact in fp16
// (flags, practically always) the products run in fp16; otherwise x is split
// into two exact bf16 parts, at twice the MFMAs.
//
// Bound by the weights' bytes and one trip to memory: 1 x 4096 x 4096 (M, K, N)
// 3.4-3.8 us, 16 x 4096 x 11008 7.7 us (24 MB), 16 x 8192 x 28672 31 us (125 MB, 4.0 TB/s).
#include <algorithm>

#include "mx_tile.hpp"

namespace wqbmm {

namespace {
constexpr int GEMV_WAVES = 8;

enum class Mode { kDirect, kSplit, kMxfp4 };
}  // namespace

template <int DT>
__device__ __forceinline__ void mx_store4(uint16_t* __restrict__ y, int64_t m, int64_t n, int64_t N, mx_f4 v) {
  uint16_t* p = y + m * N + n;
  if ((N & 3) == 0) {                       // then n + 3 < N, and the store is aligned
    *reinterpret_cast<uint2*>(p) = mx_pack4<DT>(v);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) p[i] = mx_round16<DT>(v[i]);
  }
}

// xs: 16 KB of LDS of this wave's own.  A unit is U K-tiles; its MT * 16 rows of
// x, 256 * U bytes each, fill them.  A copy moves 1 KB of whole rows (loading
// the operands straight from x, 16 bytes a lane from rows far apart, bound this
// kernel: 64 cache lines an instruction).  The 16-byte chunks of a row are
// permuted (chunk ^ row % 16: the reads of sixteen rows at one k then touch all
// banks).
template <int DT, Mode MODE, int MT, int P>
__device__ __forceinline__ void gemv_units(const uint16_t* __restrict__ x, int64_t ldx, const MxTiled& w, int p0,
                                           int M, int blocks, int wave, int lane, uint8_t* xs,
                                           mx_f4 (&acc)[P][MT]) {
  constexpr int U = 4 / MT, LANES = 16 * U, ROWS = 64 / LANES;       // lanes a row, rows a copy
  const int r = lane & 15, g = lane >> 4;
  for (int kt = wave * U; kt < w.kt; kt += GEMV_WAVES * U) {
    mx_wait_lds();                                    // the last unit's reads, before its rows are overwritten
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i * ROWS >= M) break;                       // rows past M: their products are not stored
      const int row = i * ROWS + lane / LANES;
      const int chunk = kt * 16 + ((lane % LANES) ^ (row & 15));
      const uint16_t* from = x + min(row, M - 1) * ldx + (chunk < blocks * 4 ? chunk * 8 : 0);
      __builtin_amdgcn_global_load_lds(from, xs + i * 1024, 16, 0, 0);
    }
    uint4 c[P][U];
    uint32_t sc[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int64_t pp = min(p0 + p, w.panels - 1);
#pragma unroll
      for (int i = 0; i < U; ++i)
        c[p][i] = *reinterpret_cast<const uint4*>(w.codes + ((pp * w.kt + min(kt + i, w.kt - 1)) * 64 + lane) * 16);
      sc[p] = *reinterpret_cast<const uint32_t*>(w.scales + ((pp * w.kq + kt / 4) * 64 + lane) * 4) >> (8 * (kt & 3));
    }
    mx_wait_vm<0>();
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (kt + i >= w.kt) break;                      // uniform: the last unit's missing tiles
      const bool whole = 4 * (kt + i) + 4 <= blocks, in = 4 * (kt + i) + g < blocks;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        uint4 xv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          xv[j] = *reinterpret_cast<const uint4*>(xs + (mt * 16 + r) * (LANES * 16) + ((16 * i + 4 * g + j) ^ r) * 16);
        if (!whole) {
#pragma unroll
          for (int j = 0; j < 4; ++j) xv[j] = in ? xv[j] : make_uint4(0u, 0u, 0u, 0u);
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
          for (int p = 0; p < P; ++p)
            acc[p][mt] = i == 0   ? mx_mfma4<0, 0>(c[p][i], sc[p], e, s, acc[p][mt])
                         : i == 1 ? mx_mfma4<1, 0>(c[p][i], sc[p], e, s, acc[p][mt])
                         : i == 2 ? mx_mfma4<2, 0>(c[p][i], sc[p], e, s, acc[p][mt])
                                  : mx_mfma4<3, 0>(c[p][i], sc[p], e, s, acc[p][mt]);
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
    }
  }
}

template <int DT, bool ACT4, int MT, int P>
__global__ __launch_bounds__(GEMV_WAVES * 64) void mx_gemv_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                                 MxTiled w, int M, int blocks, int64_t N,
                                                                 uint16_t* __restrict__ y) {
  // the units of x, then the waves' sums
  __shared__ __attribute__((aligned(16))) uint8_t lds[GEMV_WAVES * 16 * 1024];
  static_assert(P * MT <= 16, "a wave's sums take its 16 KB at most");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int p0 = blockIdx.x * P;
  uint8_t* const xs = lds + wave * 16 * 1024;
  mx_f4 acc[P][MT];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[p][mt] = mx_f4{0.f, 0.f, 0.f, 0.f};
  if constexpr (ACT4) {
    gemv_units<DT, Mode::kMxfp4, MT, P>(x, ldx, w, p0, M, blocks, wave, lane, xs, acc);
  } else if constexpr (DT == MX_BF16) {
    gemv_units<DT, Mode::kDirect, MT, P>(x, ldx, w, p0, M, blocks, wave, lane, xs, acc);
  } else {
    uint32_t flags = kMxFlagF16;
#pragma unroll
    for (int p = 0; p < P; ++p) flags &= w.flags[min(p0 + p, w.panels - 1)];
    if (flags & kMxFlagF16) gemv_units<DT, Mode::kDirect, MT, P>(x, ldx, w, p0, M, blocks, wave, lane, xs, acc);
    else gemv_units<DT, Mode::kSplit, MT, P>(x, ldx, w, p0, M, blocks, wave, lane, xs, acc);
  }
  mx_f4* const part = reinterpret_cast<mx_f4*>(lds);          // [wave][P * MT][64]
  __syncthreads();
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) part[(wave * P * MT + p * MT + mt) * 64 + lane] = acc[p][mt];
  __syncthreads();
  for (int t = threadIdx.x; t < P * MT * 64; t += GEMV_WAVES * 64) {
    const int pm = t >> 6;
    mx_f4 v = part[t];
#pragma unroll
    for (int k = 1; k < GEMV_WAVES; ++k) v += part[k * P * MT * 64 + t];
    const int m = (pm % MT) * 16 + (lane & 15);
    const int64_t n = (int64_t)(p0 + pm / MT) * kMxPanel + 4 * (lane >> 4);
    if (m < M && n < N) mx_store4<DT>(y, m, n, N, v);
  }
}

// Panels for a workgroup: one round of the 256 CUs where four are enough (each
// reads x once; 16 x 4096 x 11008 with 1, 2, 3, 4: 11.3, 10.0, 7.8, 8.0 us).
static int64_t panels_per_group(int64_t panels) { return std::min<int64_t>(4, (panels + 255) / 256); }

template <int DT, bool ACT4, int MT>
static hipError_t gemv_mt(const void* x, int64_t ldx, const MxTiled& w, int M, int blocks, int64_t N, void* y,
                          hipStream_t stream) {
  auto* xp = static_cast<const uint16_t*>(x);
  auto* yp = static_cast<uint16_t*>(y);
  const int per = (int)panels_per_group(w.panels);
  auto go = [&](auto* kernel) {
    return mx_launch(kernel, dim3((unsigned)((w.panels + per - 1) / per)), dim3(GEMV_WAVES * 64), stream, xp, ldx, w,
                     M, blocks, N, yp);
  };
  switch (per) {
    case 1: return go(mx_gemv_kernel<DT, ACT4, MT, 1>);
    case 2: return go(mx_gemv_kernel<DT, ACT4, MT, 2>);
    case 3: return go(mx_gemv_kernel<DT, ACT4, MT, 3>);
    default: return go(mx_gemv_kernel<DT, ACT4, MT, 4>);
  }
}

template <int DT, bool ACT4>
static hipError_t gemv_dt(const void* x, int64_t ldx, const MxTiled& w, int M, int blocks, int64_t N, void* y,
                          hipStream_t stream) {
  if (M <= 16) return gemv_mt<DT, ACT4, 1>(x, ldx, w, M, blocks, N, y, stream);
  if (M <= 32) return gemv_mt<DT, ACT4, 2>(x, ldx, w, M, blocks, N, y, stream);
  return gemv_mt<DT, ACT4, 4>(x, ldx, w, M, blocks, N, y, stream);
}

// More than 32 rows of x are reloaded by every workgroup in units of one
// K-tile: past about four of them for each wave the tiled product is faster
// (64 rows, us: 4096 x 11008 13 here, 15 tiled; 11008 x 4096 21 and 15; 8192 x
// 28672 50 and 39).
bool mx_use_gemv(int64_t M, int64_t K, int64_t N) {
  if (M <= 32 || M > kMxGemvMaxM) return M <= 32;
  const int64_t panels = mx_panels(N), per = panels_per_group(panels);
  return mx_ktiles(K) * (((panels + per - 1) / per + 255) / 256) <= 40;
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
