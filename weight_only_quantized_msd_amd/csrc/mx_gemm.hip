// mx_gemm.hip -- the product with MXFP4 weights for many rows of x:
// y[M][N] = x . W^T on the matrix cores, workgroup tiles of BM x BN.
//
// 16-bit x: each K-tile's rows of x (256 bytes a row) and panels of W go to
// LDS; a wave converts its panels' codes to 16-bit operands with the block's
// scale applied and multiplies on v_mfma_f32_16x16x32.  x lies in LDS with the
// 16-byte chunks of a row permuted (chunk ^ row % 16): the operand reads of
// sixteen rows at one k then touch all banks once.
// MXFP4 x: a preparation kernel quantises x into the tiled layout, and the
// product runs on v_mfma_scale_f32_16x16x128_f8f6f4, both operands as they lie.
// Few tiles: K is split over workgroups, whose fp32 partial sums a second
// kernel adds in split order.
#include <algorithm>

#include "mx_device.hpp"
#include "mx_launch.hpp"

namespace wqbmm {

namespace {

constexpr int NXCD = 8;

// The workgroup's output tile and K range.  XCD x (= id % 8) runs a contiguous
// range of tiles, numbered in bands of four row blocks, column-major within a
// band, so that the tiles an XCD runs together share operands in its L2.
struct Place {
  int rb, cb, split;
};
__device__ __forceinline__ Place place_of(int id, int mblocks, int nblocks, int splits) {
  constexpr int BAND = 4;
  const int tiles = mblocks * nblocks, total = tiles * splits;
  int t = id;
  if (total % NXCD == 0) t = (id % NXCD) * (total / NXCD) + id / NXCD;
  Place p;
  p.split = t / tiles;
  t %= tiles;
  const int band = t / (BAND * nblocks), in_band = t % (BAND * nblocks);
  const int rows = min(BAND, mblocks - band * BAND);
  p.rb = band * BAND + in_band % rows;
  p.cb = in_band / rows;
  return p;
}

// fp32 partial sums of split s start at s * part_stride(M, N) (whole 16-byte units).
__host__ __device__ inline int64_t part_stride(int64_t M, int64_t N) { return (M * N + 3) / 4 * 4; }

template <int DT>
__device__ __forceinline__ void store_out(uint16_t* __restrict__ y, float* __restrict__ part, int64_t m, int64_t n,
                                          int64_t N, mx_f4 v) {
  if (part) {
    float* p = part + m * N + n;
    if ((N & 3) == 0) {
      *reinterpret_cast<mx_f4*>(p) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < N) p[i] = v[i];
    }
    return;
  }
  uint16_t* p = y + m * N + n;
  if ((N & 3) == 0) {
    const uint32_t lo = mx_round16<DT>(v[0]) | ((uint32_t)mx_round16<DT>(v[1]) << 16);
    const uint32_t hi = mx_round16<DT>(v[2]) | ((uint32_t)mx_round16<DT>(v[3]) << 16);
    *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) p[i] = mx_round16<DT>(v[i]);
  }
}

__device__ __forceinline__ uint32_t dword_of(const uint4& v, int j) {
  return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
}

}  // namespace

// ---------------------------------------------------------------- 16-bit x
template <int DT, int BM, int BN, int WVM, int WVN>
__global__ __launch_bounds__(64 * WVM * WVN) void mx_gemm16_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                                   MxTiled w, int M, int blocks, int64_t N,
                                                                   int mblocks, int nblocks, int splits, int kq_per,
                                                                   uint16_t* __restrict__ y,
                                                                   float* __restrict__ part) {
  constexpr int WAVES = WVM * WVN;
  constexpr int TM = BM / WVM / 16, TN = BN / WVN / 16;     // the wave's 16-row and 16-column tiles
  constexpr int XP = BM / 4, WP = BN / 16;                  // 1 KB pieces of x and W per K-tile
  static_assert(XP % WAVES == 0 && WP % WAVES == 0, "every wave copies as many pieces");
  __shared__ __attribute__((aligned(16))) uint8_t sx0[XP * 1024], sx1[XP * 1024], sw0[WP * 1024], sw1[WP * 1024];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WVN, wn = wave % WVN;
  const int r = lane & 15, g = lane >> 4;
  const Place at = place_of(blockIdx.x, mblocks, nblocks, splits);
  const int m0 = at.rb * BM, p0 = at.cb * (BN / 16);
  const int kt_lo = at.split * kq_per * 4, kt_hi = min(w.kt, kt_lo + kq_per * 4);

  auto stage = [&](int kt, uint8_t* sx, uint8_t* sw) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < XP / WAVES; ++c) {
      const int pc = wave * (XP / WAVES) + c;
      const int row = 4 * pc + g;
      const int chunk = r ^ (row & 15);
      const uint16_t* src = x + (int64_t)min(m0 + row, M - 1) * ldx + (int64_t)kt * kMxTile + chunk * 8;
      if (4 * kt + 4 <= blocks) {
        __builtin_amdgcn_global_load_lds(reinterpret_cast<const uint8_t*>(src), sx + pc * 1024, 16, 0, 0);
      } else {                              // the last K-tile ends early: zeros past K
        uint4 v = {};
        if (4 * kt + chunk / 4 < blocks) v = *reinterpret_cast<const uint4*>(src);
        *reinterpret_cast<uint4*>(sx + pc * 1024 + lane * 16) = v;
      }
    }
#pragma unroll
    for (int c = 0; c < WP / WAVES; ++c) {
      const int pc = wave * (WP / WAVES) + c;
      const int64_t p = min(p0 + pc, w.panels - 1);
      __builtin_amdgcn_global_load_lds(w.codes + ((p * w.kt + kt) * 64 + lane) * 16, sw + pc * 1024, 16, 0, 0);
    }
  };
  uint32_t sc[TN], sc_next[TN];
  auto load_scales = [&](int q, uint32_t (&s)[TN]) {
#pragma unroll
    for (int c = 0; c < TN; ++c) {
      const int64_t p = min(p0 + wn * TN + c, w.panels - 1);
      s[c] = *reinterpret_cast<const uint32_t*>(w.scales + ((p * w.kq + min(q, w.kq - 1)) * 64 + lane) * 4);
    }
  };

  mx_f4 acc[TN][TM];
#pragma unroll
  for (int c = 0; c < TN; ++c)
#pragma unroll
    for (int t = 0; t < TM; ++t) acc[c][t] = mx_f4{0.f, 0.f, 0.f, 0.f};

  auto compute = [&](auto split_c, int kt, const uint8_t* sx, const uint8_t* sw) __attribute__((always_inline)) {
    constexpr bool SPLIT = decltype(split_c)::value;
    uint4 codes[TN];
    float f[TN];
#pragma unroll
    for (int c = 0; c < TN; ++c) {
      codes[c] = *reinterpret_cast<const uint4*>(sw + (wn * TN + c) * 1024 + lane * 16);
      f[c] = mx_scale((sc[c] >> (8 * (kt & 3))) & 0xffu);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint4 xv[TM];
#pragma unroll
      for (int t = 0; t < TM; ++t)
        xv[t] = *reinterpret_cast<const uint4*>(sx + ((wm * TM + t) * 16 + r) * 256 + (((4 * g + j) ^ r) * 16));
      if constexpr (SPLIT) {
        uint4 hi[TM], lo[TM];
#pragma unroll
        for (int t = 0; t < TM; ++t) mx_split8(xv[t], hi[t], lo[t]);
#pragma unroll
        for (int c = 0; c < TN; ++c) {
          const uint4 a = mx_decode8<MX_BF16>(dword_of(codes[c], j), f[c]);
#pragma unroll
          for (int t = 0; t < TM; ++t) {
            acc[c][t] = mx_mfma16<MX_BF16>(a, hi[t], acc[c][t]);
            acc[c][t] = mx_mfma16<MX_BF16>(a, lo[t], acc[c][t]);
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < TN; ++c) {
          const uint4 a = mx_decode8<DT>(dword_of(codes[c], j), f[c]);
#pragma unroll
          for (int t = 0; t < TM; ++t) acc[c][t] = mx_mfma16<DT>(a, xv[t], acc[c][t]);
        }
      }
    }
  };

  // Two named buffers in turn: the next K-tile is copied into one while the
  // other is multiplied; each wave waits for its own copies, and the barrier
  // publishes all of them and frees the buffer just read.
  auto run = [&](auto split_c) __attribute__((always_inline)) {
    load_scales(kt_lo / 4, sc);
    load_scales(kt_lo / 4 + 1, sc_next);
    auto advance = [&](int kt) __attribute__((always_inline)) {            // after K-tile kt: the next quad's scales
      if ((kt & 3) == 3) {
#pragma unroll
        for (int c = 0; c < TN; ++c) sc[c] = sc_next[c];
        load_scales(kt / 4 + 2, sc_next);
      }
    };
    stage(kt_lo, sx0, sw0);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    for (int kt = kt_lo; kt < kt_hi; kt += 2) {
      if (kt + 1 < kt_hi) stage(kt + 1, sx1, sw1);
      compute(split_c, kt, sx0, sw0);
      advance(kt);
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
      if (kt + 1 >= kt_hi) break;
      if (kt + 2 < kt_hi) stage(kt + 2, sx0, sw0);
      compute(split_c, kt + 1, sx1, sw1);
      advance(kt + 1);
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
    }
  };
  if constexpr (DT == MX_BF16) {
    run(std::false_type{});
  } else {
    // fp16 operands where all of the tile's weights are exact in fp16 (the
    // rule of mx_launch.hpp); else both parts of x in bf16
    uint32_t flags = kMxFlagF16;
    for (int c = 0; c < BN / 16; ++c) flags &= w.flags[min(p0 + c, w.panels - 1)];
    if (flags & kMxFlagF16) run(std::false_type{});
    else run(std::true_type{});
  }

  float* const out = part ? part + at.split * part_stride(M, N) : nullptr;
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    const int m = m0 + (wm * TM + t) * 16 + r;
#pragma unroll
    for (int c = 0; c < TN; ++c) {
      const int64_t n = (int64_t)(p0 + wn * TN + c) * kMxPanel + 4 * g;
      if (m < M && n < N) store_out<DT>(y, out, m, n, N, acc[c][t]);
    }
  }
}

// ---------------------------------------------------------------- MXFP4 x
// x -> tiled MXFP4.  A wave takes a panel's quad of K-tiles; a lane holds whole
// blocks, so nothing crosses lanes.
template <int DT>
__global__ __launch_bounds__(256) void mx_prep_kernel(const uint16_t* __restrict__ x, int64_t ldx, int M, int blocks,
                                                      int kt, int kq, int64_t waves, uint8_t* __restrict__ codes,
                                                      uint32_t* __restrict__ scales) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (id >= waves) return;
  const int64_t p = id / kq;
  const int q = (int)(id % kq);
  const int64_t m = p * kMxPanel + r;
  uint4 v[4][4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = 4 * (4 * q + i) + g;
    if (m < M && b < blocks) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[i][j] = reinterpret_cast<const uint4*>(x + m * ldx + (int64_t)b * kMxBlock)[j];
    }
  }
  uint32_t dword = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (4 * q + i >= kt) break;
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) top = mx_max16(v[i][j], top);
    const uint32_t s = mx_scale_byte(mx_top_bits<DT>(mx_max16_fold(top)));
    const float f = mx_scale(s);
    dword |= s << (8 * i);
    *reinterpret_cast<uint4*>(codes + ((p * kt + 4 * q + i) * 64 + lane) * 16) = make_uint4(
        mx_encode8<DT>(v[i][0], f), mx_encode8<DT>(v[i][1], f), mx_encode8<DT>(v[i][2], f), mx_encode8<DT>(v[i][3], f));
  }
  scales[(p * kq + q) * 64 + lane] = dword;
}

template <int DT, int BM, int BN, int WVM, int WVN>
__global__ __launch_bounds__(64 * WVM * WVN) void mx_gemm4_kernel(MxTiled x, MxTiled w, int M, int64_t N,
                                                                  int mblocks, int nblocks, int splits, int kq_per,
                                                                  uint16_t* __restrict__ y,
                                                                  float* __restrict__ part) {
  constexpr int WAVES = WVM * WVN;
  constexpr int TM = BM / WVM / 16, TN = BN / WVN / 16;
  constexpr int KS = 2;                                     // K-tiles a step
  constexpr int XP = BM / 16 * KS, WP = BN / 16 * KS;       // 1 KB pieces a step
  static_assert(XP % WAVES == 0 && WP % WAVES == 0, "every wave copies as many pieces");
  __shared__ __attribute__((aligned(16))) uint8_t sx0[XP * 1024], sx1[XP * 1024], sw0[WP * 1024], sw1[WP * 1024];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WVN, wn = wave % WVN;
  const Place at = place_of(blockIdx.x, mblocks, nblocks, splits);
  const int x0 = at.rb * (BM / 16), p0 = at.cb * (BN / 16);
  const int q_lo = at.split * kq_per, q_hi = min(w.kq, q_lo + kq_per);

  auto copy = [&](const MxTiled& a, int first, int pieces, int kt, uint8_t* s) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < pieces / WAVES; ++c) {
      const int pc = wave * (pieces / WAVES) + c;
      const int64_t p = min(first + pc / KS, a.panels - 1);
      const int k = min(kt + pc % KS, a.kt - 1);            // a tile past the end is not multiplied
      __builtin_amdgcn_global_load_lds(a.codes + ((p * a.kt + k) * 64 + lane) * 16, s + pc * 1024, 16, 0, 0);
    }
  };
  auto stage = [&](int kt, uint8_t* sx, uint8_t* sw) __attribute__((always_inline)) {
    copy(x, x0, XP, kt, sx);
    copy(w, p0, WP, kt, sw);
  };
  auto load_scales = [&](int q, uint32_t (&sx)[TM], uint32_t (&sw)[TN]) {
    const int qq = min(q, w.kq - 1);
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      const int64_t p = min(x0 + wm * TM + t, x.panels - 1);
      sx[t] = *reinterpret_cast<const uint32_t*>(x.scales + ((p * x.kq + qq) * 64 + lane) * 4);
    }
#pragma unroll
    for (int c = 0; c < TN; ++c) {
      const int64_t p = min(p0 + wn * TN + c, w.panels - 1);
      sw[c] = *reinterpret_cast<const uint32_t*>(w.scales + ((p * w.kq + qq) * 64 + lane) * 4);
    }
  };

  mx_f4 acc[TN][TM];
#pragma unroll
  for (int c = 0; c < TN; ++c)
#pragma unroll
    for (int t = 0; t < TM; ++t) acc[c][t] = mx_f4{0.f, 0.f, 0.f, 0.f};
  uint32_t scx[TM], scw[TN], nx[TM], nw[TN];

  // The K-tiles 4q + 2h, 4q + 2h + 1 from one buffer; h picks the scale bytes.
  auto compute = [&](auto hc, int q, const uint8_t* sx, const uint8_t* sw) __attribute__((always_inline)) {
    constexpr int h = decltype(hc)::value;
    auto tile = [&](auto ic) __attribute__((always_inline)) {
      constexpr int i = decltype(ic)::value;
      if (4 * q + 2 * h + i >= w.kt) return;
      uint4 a[TN], b[TM];
#pragma unroll
      for (int c = 0; c < TN; ++c)
        a[c] = *reinterpret_cast<const uint4*>(sw + ((wn * TN + c) * KS + i) * 1024 + lane * 16);
#pragma unroll
      for (int t = 0; t < TM; ++t)
        b[t] = *reinterpret_cast<const uint4*>(sx + ((wm * TM + t) * KS + i) * 1024 + lane * 16);
#pragma unroll
      for (int c = 0; c < TN; ++c)
#pragma unroll
        for (int t = 0; t < TM; ++t)
          acc[c][t] = mx_mfma4<2 * h + i, 2 * h + i>(a[c], scw[c], b[t], scx[t], acc[c][t]);
    };
    tile(std::integral_constant<int, 0>{});
    tile(std::integral_constant<int, 1>{});
  };

  load_scales(q_lo, scx, scw);
  stage(4 * q_lo, sx0, sw0);
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  for (int q = q_lo; q < q_hi; ++q) {
    load_scales(q + 1, nx, nw);
    if (4 * q + 2 < w.kt) stage(4 * q + 2, sx1, sw1);
    compute(std::integral_constant<int, 0>{}, q, sx0, sw0);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (q + 1 < q_hi) stage(4 * q + 4, sx0, sw0);
    compute(std::integral_constant<int, 1>{}, q, sx1, sw1);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < TM; ++t) scx[t] = nx[t];
#pragma unroll
    for (int c = 0; c < TN; ++c) scw[c] = nw[c];
  }

  float* const out = part ? part + at.split * part_stride(M, N) : nullptr;
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    const int m = (x0 + wm * TM + t) * 16 + (lane & 15);
#pragma unroll
    for (int c = 0; c < TN; ++c) {
      const int64_t n = (int64_t)(p0 + wn * TN + c) * kMxPanel + 4 * (lane >> 4);
      if (m < M && n < N) store_out<DT>(y, out, m, n, N, acc[c][t]);
    }
  }
}

// ---------------------------------------------------------------- K-splits
template <int DT>
__global__ __launch_bounds__(256) void mx_reduce_kernel(const float* __restrict__ part, int64_t stride, int splits,
                                                        int64_t count, uint16_t* __restrict__ y) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= count) return;
  mx_f4 v = *reinterpret_cast<const mx_f4*>(part + i);
  for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const mx_f4*>(part + s * stride + i);
  if (i + 3 < count) {
    const uint32_t lo = mx_round16<DT>(v[0]) | ((uint32_t)mx_round16<DT>(v[1]) << 16);
    const uint32_t hi = mx_round16<DT>(v[2]) | ((uint32_t)mx_round16<DT>(v[3]) << 16);
    *reinterpret_cast<uint2*>(y + i) = make_uint2(lo, hi);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < count) y[i + j] = mx_round16<DT>(v[j]);
  }
}

constexpr int GEMM_BM = 128, GEMM_BN = 256;

MxGemmPlan mx_gemm_plan(int64_t M, int64_t K, int64_t N, int act) {
  MxGemmPlan p{};
  p.mblocks = (M + GEMM_BM - 1) / GEMM_BM;
  p.nblocks = (N + GEMM_BN - 1) / GEMM_BN;
  const int64_t tiles = p.mblocks * p.nblocks, kq = mx_kquads(K);
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(kq, 256 / tiles));
  p.kq_per = (kq + want - 1) / want;
  p.splits = (kq + p.kq_per - 1) / p.kq_per;
  p.x_bytes = act ? (mx_tiled_bytes(K, M) + 255) / 256 * 256 : 0;
  p.part_bytes = p.splits > 1 ? (size_t)(p.splits * part_stride(M, N)) * 4 : 0;
  return p;
}

template <int DT>
static hipError_t gemm_dt(const void* x, int64_t ldx, const MxTiled& w, int64_t M, int64_t K, int64_t N, void* y,
                          int act, const MxGemmPlan& plan, uint8_t* ws, hipStream_t stream) {
  const int m = (int)M, blocks = (int)(K / kMxBlock);
  const int mb = (int)plan.mblocks, nb = (int)plan.nblocks, sp = (int)plan.splits, kp = (int)plan.kq_per;
  auto* xp = static_cast<const uint16_t*>(x);
  auto* yp = static_cast<uint16_t*>(y);
  float* part = sp > 1 ? reinterpret_cast<float*>(ws + plan.x_bytes) : nullptr;
  const dim3 grid((unsigned)(plan.mblocks * plan.nblocks * plan.splits));
  hipError_t e;
  if (act) {
    const MxTiled xt = mx_view(ws, K, M);
    auto* codes = ws;
    auto* scales = reinterpret_cast<uint32_t*>(const_cast<uint8_t*>(xt.scales));
    const int64_t waves = (int64_t)xt.panels * xt.kq;
    e = mx_launch(mx_prep_kernel<DT>, dim3((unsigned)((waves + 3) / 4)), dim3(256), stream, xp, ldx, m, blocks, xt.kt,
                  xt.kq, waves, codes, scales);
    if (e != hipSuccess) return e;
    e = mx_launch(mx_gemm4_kernel<DT, GEMM_BM, GEMM_BN, 2, 4>, grid, dim3(512), stream, xt, w, m, N, mb, nb, sp, kp,
                  yp, part);
  } else {
    e = mx_launch(mx_gemm16_kernel<DT, GEMM_BM, GEMM_BN, 2, 4>, grid, dim3(512), stream, xp, ldx, w, m, blocks, N, mb,
                  nb, sp, kp, yp, part);
  }
  if (e != hipSuccess || sp == 1) return e;
  const int64_t count = M * N, stride = part_stride(M, N);
  return mx_launch(mx_reduce_kernel<DT>, dim3((unsigned)((count + 1023) / 1024)), dim3(256), stream,
                   (const float*)part, stride, sp, count, yp);
}

hipError_t launch_mx_gemm(const void* x, int dtype, int64_t ldx, const MxTiled& w, int64_t M, int64_t K,
                          int64_t N, void* y, int act, const MxGemmPlan& plan, uint8_t* ws, hipStream_t stream) {
  return dtype == MX_F16 ? gemm_dt<MX_F16>(x, ldx, w, M, K, N, y, act, plan, ws, stream)
                         : gemm_dt<MX_BF16>(x, ldx, w, M, K, N, y, act, plan, ws, stream);
}

}  // namespace wqbmm
