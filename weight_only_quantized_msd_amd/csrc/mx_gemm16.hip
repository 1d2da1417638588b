// mx_gemm16.hip -- the product of 16-bit activations with MXFP4 weights for many
// rows: y[M][N] = x . W^T on v_mfma_f32_16x16x32, the codes converted to 16-bit
// operands with the block's scale applied (exact) as they are multiplied.
// Few tiles: K is split over workgroups, whose fp32 partial sums a second
// kernel adds in split order.
//
// 2048 x 4096 x 4096 (M, K, N): 51 us, of which 1.3 us for each of the 32
// K-tiles, 1.65 PFLOP/s; the matrix cores alone, on random bf16 operands in
// registers, reached 1.84 (the card's power limit), and the rest are the first
// copies, the output and the launch.
#include <algorithm>
#include <cmath>

#include "mx_tile.hpp"

namespace wqbmm {

namespace {

template <int CT>
__device__ __forceinline__ void mfma16_into(mx_f4& c, uint4 a, uint4 b) {
  const mx_i4 av = __builtin_bit_cast(mx_i4, a), bv = __builtin_bit_cast(mx_i4, b);
  if constexpr (CT == MX_BF16) asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(av), "v"(bv));
  else asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(av), "v"(bv));
}

// Four waves side by side along N, each with TM x TN results of 16 x 16.  A
// K-tile (128 k) of x (256 bytes a row) and of W's codes is a stage; three
// stages in LDS form a ring.  A K-tile is multiplied in four slices: slice j
// takes dword j of each lane's 32 codes, i.e. eight k of each of four blocks,
// and the same k of x.  While slice j is multiplied, the operands of the next
// one are read (x) and converted (W) into the other set of registers.  Before
// slice 3 the waves wait for their copies of the next stage and meet: then the
// next stage is read, and stage kt's buffer, which all have read, takes copies
// of stage kt + 3.
template <int DT, bool SPLIT, int TM, int TN>
struct Gemm16 {
  static constexpr int WAVES = 4;
  static constexpr int BM = TM * 16, BN = TN * 16 * WAVES;
  static constexpr int XP = BM / 4, WP = TN * WAVES;        // 1 KB pieces of x and W in a stage
  static constexpr int PX = XP / WAVES, PW = WP / WAVES, P = PX + PW;
  static constexpr int STAGE = (XP + WP) * 1024;
  static constexpr int CT = SPLIT ? MX_BF16 : DT;           // the type of the products
};

template <int DT, bool SPLIT, int TM, int TN>
__device__ __forceinline__ void gemm16_loop(const uint16_t* __restrict__ x, int64_t ldx, const MxTiled& w, int M,
                                            int blocks, int m0, int p0, int kt_lo, int kt_hi, uint8_t* s0,
                                            uint8_t* s1, uint8_t* s2, mx_f4 (&acc)[TN][TM]) {
  using G = Gemm16<DT, SPLIT, TM, TN>;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4, lane16 = lane * 16;

  // x's rows of this tile, up to the last one's end.
  const int rows = min(G::BM, M - m0);
  const auto xb = mx_buffer(x + (int64_t)m0 * ldx, ((rows - 1) * ldx + (int64_t)blocks * kMxBlock) * 2);
  // A piece is four rows of 256 bytes, whose 16-byte chunks are permuted (chunk
  // ^ row % 16: the reads of sixteen rows at one k then touch all banks).
  // xlast: in the K-tile that ends past K (`tail`, if there is one).
  const int tail = blocks % 4 != 0 ? blocks / 4 : -1;
  int xoff[G::PX], xlast[G::PX];
#pragma unroll
  for (int c = 0; c < G::PX; ++c) {
    const int row = 4 * (wave * G::PX + c) + g, chunk = r ^ (row & 15);
    xoff[c] = mx_x_row(row, rows, ldx) + mx_x_chunk(chunk, 4);
    xlast[c] = mx_x_row(row, rows, ldx) + mx_x_chunk(chunk, blocks % 4);
  }
  const auto wb = mx_buffer(w.codes + (int64_t)p0 * w.kt * 1024, (int64_t)min(G::WP, w.panels - p0) * w.kt * 1024);
  const auto sb = mx_buffer(w.scales + (int64_t)p0 * w.kq * 256, (int64_t)min(G::WP, w.panels - p0) * w.kq * 256);
  int panel[TN];
#pragma unroll
  for (int c = 0; c < TN; ++c) panel[c] = min(wave * TN + c, w.panels - p0 - 1);

  // A wave copies a share of the rows of x and its own panels of W.
  auto copy_x = [&](int c, int kt, uint8_t* s) __attribute__((always_inline)) {
    uint8_t* const to = s + (wave * G::PX + c) * 1024;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(xb, (__attribute__((address_space(3))) void*)to, 16,
                                             kt == tail ? xlast[c] : xoff[c], kt * 256, 0, 0);
  };
  auto copy_w = [&](int c, int kt, uint8_t* s) __attribute__((always_inline)) {
    uint8_t* const to = s + (G::XP + wave * TN + c) * 1024;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(wb, (__attribute__((address_space(3))) void*)to, 16, lane16,
                                             (panel[c] * w.kt + kt) * 1024, 0, 0);
  };
  auto copy = [&](int c, int kt, uint8_t* s) __attribute__((always_inline)) {
    if (c < TN) copy_w(c, kt, s);
    else copy_x(c - TN, kt, s);
  };
  // Past the end of the range: a tile that exists, so that the waits' counts hold.
  auto within = [&](int kt) __attribute__((always_inline)) { return kt < kt_hi ? kt : kt_lo; };
  uint32_t sc[TN];                                          // the scales of the K-tile after the present one
  auto load_scales = [&](int kt, uint32_t (&s)[TN]) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < TN; ++c)
      s[c] = __builtin_amdgcn_raw_buffer_load_b32(sb, lane * 4, (panel[c] * w.kq + kt / 4) * 256, 0);
  };

  uint4 x0[TM], x1[TM], w0[TN], w1[TN], raw[TN];
  float f[TN];
  auto read_x = [&](const uint8_t* s, int j, int t) __attribute__((always_inline)) {
    return *reinterpret_cast<const uint4*>(s + (t * 16 + r) * 256 + (((4 * g + j) ^ r) * 16));
  };
  auto read_w = [&](const uint8_t* s, int c) __attribute__((always_inline)) {
    return *reinterpret_cast<const uint4*>(s + (G::XP + wave * TN + c) * 1024 + lane16);
  };
  // The products of a slice; between them stand `beside(i)`, i = 0 ... TM * TN - 1
  // (memory accesses keep their place: the products are volatile asm).
  auto multiply = [&](const uint4 (&xs)[TM], const uint4 (&ws)[TN], auto beside) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      uint4 hi, lo;
      if constexpr (SPLIT) mx_split8(xs[t], hi, lo);
#pragma unroll
      for (int c = 0; c < TN; ++c) {
        beside(t * TN + c);
        if constexpr (SPLIT) {
          acc[c][t] = mx_mfma16<G::CT>(ws[c], hi, acc[c][t]);
          acc[c][t] = mx_mfma16<G::CT>(ws[c], lo, acc[c][t]);
        } else {
          mfma16_into<G::CT>(acc[c][t], ws[c], xs[t]);
          __builtin_amdgcn_sched_barrier(0);                // conversions keep their place, too
        }
      }
    }
  };
  // Between slices: the operands read and converted beside the last one are
  // there.  In the range's last K-tiles, x past K (the next row's values, or
  // none) becomes zero.
  auto ready = [&](auto mask_c, int kt, uint4 (&xs)[TM]) __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
    mx_wait_lds();
    if constexpr (decltype(mask_c)::value) {
      const bool in = 4 * kt + g < blocks;
#pragma unroll
      for (int t = 0; t < TM; ++t) xs[t] = in ? xs[t] : make_uint4(0u, 0u, 0u, 0u);
      __builtin_amdgcn_sched_barrier(0);
      mx_settle();
    }
  };
  // Conversions lo ... hi - 1 of the slice's 4 * TN (two values a lane each).
  auto convert = [&](int j, uint4 (&ws)[TN], int lo, int hi) __attribute__((always_inline)) {
#pragma unroll
    for (int i = lo; i < hi; ++i) {
      const uint32_t v = mx_decode2<G::CT>(dword_of(raw[i / 4], j), i % 4, f[i / 4]);
      if (i % 4 == 0) ws[i / 4].x = v;
      if (i % 4 == 1) ws[i / 4].y = v;
      if (i % 4 == 2) ws[i / 4].z = v;
      if (i % 4 == 3) ws[i / 4].w = v;
    }
  };
  // The next slice's operands, beside the present one's products: the reads
  // early, the conversions spread evenly.
  auto prepare = [&](const uint8_t* s, int j, uint4 (&xs)[TM], uint4 (&ws)[TN], int i) __attribute__((always_inline)) {
    constexpr int RS = TN * 3 / 4 > 0 ? TN * 3 / 4 : 1;
    if (i % RS == 0 && i / RS < TM) xs[i / RS] = read_x(s, j, i / RS);
    convert(j, ws, i * 4 * TN / (TM * TN), (i + 1) * 4 * TN / (TM * TN));
  };
  // K-tile kt's stage is s, the next one's `next`.  BEFORE, SCALES: whether the
  // last K-tile and this one load scales (the waits count these loads, and ones
  // without a use would be taken out: the last two K-tiles load none).
  auto tile = [&](auto mask_c, auto before_c, auto scales_c, int kt, uint8_t* s, const uint8_t* next) __attribute__((always_inline)) {
    ready(mask_c, kt, x0);
    multiply(x0, w0, [&](int i) __attribute__((always_inline)) { prepare(s, 1, x1, w1, i); });
    ready(mask_c, kt, x1);
    multiply(x1, w1, [&](int i) __attribute__((always_inline)) { prepare(s, 2, x0, w0, i); });
    ready(mask_c, kt, x0);
    multiply(x0, w0, [&](int i) __attribute__((always_inline)) { prepare(s, 3, x1, w1, i); });
    __builtin_amdgcn_sched_barrier(0);
    mx_wait_vm_lds<(decltype(before_c)::value ? TN : 0) + G::P>();   // what the last K-tile issued stays in flight
    mx_barrier();
    ready(mask_c, kt, x1);
#pragma unroll
    for (int c = 0; c < TN; ++c) f[c] = mx_scale((sc[c] >> (8 * ((kt + 1) & 3))) & 0xffu);
    if constexpr (decltype(scales_c)::value) load_scales(within(kt + 2), sc);
    const int k3 = within(kt + 3);
    constexpr int PRODUCTS = TM * TN, AT_ONCE = (G::P + PRODUCTS - 1) / PRODUCTS, CS = PRODUCTS * AT_ONCE / G::P;
    multiply(x1, w1, [&](int i) __attribute__((always_inline)) {
      if (i < TN) raw[i] = read_w(next, i);
      if (i < TM) x0[i] = read_x(next, 0, i);
      if (i % CS == 0) {
#pragma unroll
        for (int c = i / CS * AT_ONCE; c < (i / CS + 1) * AT_ONCE; ++c)
          if (c < G::P) copy(c, k3, s);
      }
      // in the second half, when the codes have come
      if (i >= PRODUCTS / 2) convert(0, w0, (2 * i - PRODUCTS) * 4 * TN / PRODUCTS, (2 * i + 2 - PRODUCTS) * 4 * TN / PRODUCTS);
    });
  };

  uint32_t first[TN];
  load_scales(kt_lo, first);
#pragma unroll
  for (int c = 0; c < G::P; ++c) copy(c, kt_lo, s0);
#pragma unroll
  for (int c = 0; c < G::P; ++c) copy(c, within(kt_lo + 1), s1);
  load_scales(within(kt_lo + 1), sc);                       // before stage 2, as the first tile's wait counts
#pragma unroll
  for (int c = 0; c < G::P; ++c) copy(c, within(kt_lo + 2), s2);
  mx_wait_vm_lds<2 * G::P + TN>();
  mx_barrier();
#pragma unroll
  for (int t = 0; t < TM; ++t) x0[t] = read_x(s0, 0, t);
#pragma unroll
  for (int c = 0; c < TN; ++c) {
    f[c] = mx_scale(first[c] & 0xffu);                      // kt_lo is a multiple of 4
    raw[c] = read_w(s0, c);
    w0[c] = mx_decode8<G::CT>(raw[c].x, f[c]);
  }
  using Yes = std::true_type;
  using No = std::false_type;
  const int whole = min(kt_hi, blocks / 4);                 // K-tiles that end within K
  int kt = kt_lo;
  for (; kt + 3 <= whole; kt += 3) {
    tile(No{}, Yes{}, Yes{}, kt, s0, s1);
    tile(No{}, Yes{}, Yes{}, kt + 1, s1, s2);
    tile(No{}, Yes{}, Yes{}, kt + 2, s2, s0);
  }
  if (kt < kt_hi) tile(Yes{}, Yes{}, Yes{}, kt, s0, s1);
  if (kt + 1 < kt_hi) tile(Yes{}, Yes{}, No{}, kt + 1, s1, s2);
  if (kt + 2 < kt_hi) tile(Yes{}, No{}, No{}, kt + 2, s2, s0);
  mx_wait_vm_lds<0>();                                      // copies must not outlive the workgroup's LDS
  mx_wait_results();
}

template <int DT, int TM, int TN>
__device__ __forceinline__ void gemm16_tile(const uint16_t* __restrict__ x, int64_t ldx, const MxTiled& w, int M,
                                            int blocks, int64_t N, int mblocks, int nblocks, int splits, int kq_per,
                                            uint16_t* __restrict__ y, float* __restrict__ part) {
  using G = Gemm16<DT, false, TM, TN>;
  // three variables: the compiler tells copies into one from reads of another
  __shared__ __attribute__((aligned(16))) uint8_t s0[G::STAGE], s1[G::STAGE], s2[G::STAGE];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const MxPlace at = mx_place(blockIdx.x, mblocks, nblocks, splits);
  const int m0 = at.rb * G::BM, p0 = at.cb * G::WP;
  const int kt_lo = at.split * kq_per * 4, kt_hi = min(w.kt, kt_lo + kq_per * 4);
  mx_f4 acc[TN][TM];
#pragma unroll
  for (int c = 0; c < TN; ++c)
#pragma unroll
    for (int t = 0; t < TM; ++t) acc[c][t] = mx_f4{0.f, 0.f, 0.f, 0.f};
  if constexpr (DT == MX_BF16) {
    gemm16_loop<DT, false, TM, TN>(x, ldx, w, M, blocks, m0, p0, kt_lo, kt_hi, s0, s1, s2, acc);
  } else {
    // fp16 operands where all of the tile's weights are exact in fp16 (the
    // rule of mx_launch.hpp); else both parts of x in bf16
    uint32_t flags = kMxFlagF16;
    for (int c = 0; c < G::WP; ++c) flags &= w.flags[min(p0 + c, w.panels - 1)];
    if (flags & kMxFlagF16) gemm16_loop<DT, false, TM, TN>(x, ldx, w, M, blocks, m0, p0, kt_lo, kt_hi, s0, s1, s2, acc);
    else gemm16_loop<DT, true, TM, TN>(x, ldx, w, M, blocks, m0, p0, kt_lo, kt_hi, s0, s1, s2, acc);
  }
  if (!part && (N & 7) == 0) {
    mx_barrier();                                           // no wave reads the stages or copies into them any more
    static_assert(2 * mx_stage_bytes<TM, TN>() <= G::STAGE, "the rows of two waves fit a stage");
    uint8_t* const mine = (wave < 2 ? s0 : s1) + (wave & 1) * mx_stage_bytes<TM, TN>();
    mx_store_rows<DT, TM, TN>(y, M, N, m0, (int64_t)(p0 + wave * TN) * kMxPanel, lane, mine,
                              [&](int c, int t) __attribute__((always_inline)) {
                                mx_keep_in_place(acc[c][t]);  // read here, not all of them ahead of the first store
                                return acc[c][t];
                              });
    return;
  }
  mx_store_tile<DT>(y, part, at.split, M, N, [&](auto put) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
      for (int c = 0; c < TN; ++c) {
        mx_keep_in_place(acc[c][t]);
        put(m0 + t * 16 + (lane & 15), (int64_t)(p0 + wave * TN + c) * kMxPanel + 4 * (lane >> 4), acc[c][t]);
      }
  });
}

}  // namespace

template <int DT, int TM, int TN>
__global__ __launch_bounds__(256) void mx_gemm16_kernel(const uint16_t* __restrict__ x, int64_t ldx, MxTiled w, int M,
                                                        int blocks, int64_t N, int mblocks, int nblocks, int splits,
                                                        int kq_per, uint16_t* __restrict__ y,
                                                        float* __restrict__ part) {
  gemm16_tile<DT, TM, TN>(x, ldx, w, M, blocks, N, mblocks, nblocks, splits, kq_per, y, part);
}

// ---------------------------------------------------------------- K-splits
// y = the partial sums added in split order; a thread takes four columns.
template <int DT>
__global__ __launch_bounds__(256) void mx_reduce_kernel(const float* __restrict__ part, int splits, int64_t count,
                                                        uint32_t units, int64_t N, uint16_t* __restrict__ y) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;            // of count = M * units
  if (i >= count) return;
  mx_f4 v = reinterpret_cast<const mx_f4*>(part)[i];
  for (int s = 1; s < splits; ++s) v += reinterpret_cast<const mx_f4*>(part)[s * count + i];
  if ((N & 3) == 0) {
    reinterpret_cast<uint2*>(y)[i] = mx_pack4<DT>(v);
    return;
  }
  const int64_t m = i / units, n = (i - m * units) * 4;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (n + j < N) y[m * N + n + j] = mx_round16<DT>(v[j]);
}

hipError_t launch_mx_reduce(const float* part, int splits, int64_t M, int64_t N, void* y, int dtype,
                            hipStream_t stream) {
  const uint32_t units = (uint32_t)(mx_part_pitch(N) / 4);
  const int64_t count = M * units;
  auto* yp = static_cast<uint16_t*>(y);
  auto* kernel = dtype == MX_F16 ? mx_reduce_kernel<MX_F16> : mx_reduce_kernel<MX_BF16>;
  return mx_launch(kernel, dim3((unsigned)((count + 255) / 256)), dim3(256), stream, part, splits, count, units, N, yp);
}

// ---------------------------------------------------------------- launch
MxGemmPlan mx_choose(const MxTileCost* tiles, int count, double base, int64_t M, int64_t K, int64_t N) {
  constexpr double CUS = 256, BYTES_PER_US = 5e6;
  constexpr int64_t MAX_SPLITS = 16;
  const int64_t kt = mx_ktiles(K), kq = mx_kquads(K);
  MxGemmPlan best{};
  double least = 0;
  for (int v = 0; v < count; ++v) {
    const int64_t mb = (M + tiles[v].bm - 1) / tiles[v].bm, nb = (N + tiles[v].bn - 1) / tiles[v].bn;
    for (int64_t s = 1; s <= std::min(MAX_SPLITS, kq) && (s == 1 || mb * nb * s <= 512); ++s) {
      const int64_t per = (kq + s - 1) / s, splits = (kq + per - 1) / per;
      if (splits != s) continue;
      const double rounds = std::ceil((double)(mb * nb) * (double)s / CUS);
      double us = base + rounds * (tiles[v].fixed + tiles[v].per_ktile * (double)std::min(kt, 4 * per));
      if (s > 1) us += 2.0 + (double)s * (double)M * (double)N * 8.0 / BYTES_PER_US;
      if (best.splits == 0 || us < least) {
        least = us;
        best.variant = v;
        best.mblocks = mb;
        best.nblocks = nb;
        best.splits = s;
        best.kq_per = per;
      }
    }
  }
  if (best.splits > 1) best.part_bytes = (size_t)(best.splits * M * mx_part_pitch(N)) * 4;
  return best;
}

// Measured at 2048 x 4096 x 4096 (M, K, N): 52 us with the first tile, 62 with
// the others; at 512 rows 30, 27 and 19 us; at 130 x 4128 x 4099 24, 18 and 17.
constexpr MxTileCost kTiles[] = {{128, 256, 6.0, 1.30}, {64, 256, 1.0, 0.83}, {64, 128, 0.0, 0.45}};

MxGemmPlan mx_gemm16_plan(int64_t M, int64_t K, int64_t N) { return mx_choose(kTiles, 3, 4.0, M, K, N); }

template <int DT>
static hipError_t gemm16_dt(const void* x, int64_t ldx, const MxTiled& w, int64_t M, int64_t K, int64_t N, void* y,
                            const MxGemmPlan& plan, float* part, hipStream_t stream) {
  const int m = (int)M, blocks = (int)(K / kMxBlock);
  const int mb = (int)plan.mblocks, nb = (int)plan.nblocks, sp = (int)plan.splits, kp = (int)plan.kq_per;
  auto* xp = static_cast<const uint16_t*>(x);
  auto* yp = static_cast<uint16_t*>(y);
  const dim3 grid((unsigned)(plan.mblocks * plan.nblocks * plan.splits));
  auto go = [&](auto* kernel) {
    return mx_launch(kernel, grid, dim3(256), stream, xp, ldx, w, m, blocks, N, mb, nb, sp, kp, yp, part);
  };
  switch (plan.variant) {
    case 0: return go(mx_gemm16_kernel<DT, 8, 4>);
    case 1: return go(mx_gemm16_kernel<DT, 4, 4>);
    default: return go(mx_gemm16_kernel<DT, 4, 2>);
  }
}

hipError_t launch_mx_gemm16(const void* x, int dtype, int64_t ldx, const MxTiled& w, int64_t M, int64_t K, int64_t N,
                            void* y, const MxGemmPlan& plan, uint8_t* ws, hipStream_t stream) {
  float* part = plan.splits > 1 ? reinterpret_cast<float*>(ws) : nullptr;
  const hipError_t e = dtype == MX_F16 ? gemm16_dt<MX_F16>(x, ldx, w, M, K, N, y, plan, part, stream)
                                       : gemm16_dt<MX_BF16>(x, ldx, w, M, K, N, y, plan, part, stream);
  if (e != hipSuccess || !part) return e;
  return launch_mx_reduce(part, (int)plan.splits, M, N, y, dtype, stream);
}

}  // namespace wqbmm
