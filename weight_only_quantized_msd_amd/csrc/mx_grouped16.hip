// mx_grouped16.hip -- products of 16-bit activations with MXFP4 weights grouped by
// expert, many rows a group, on the tiles of mx_gemm16.hpp.  A workgroup takes a tile of
// places of one group and a block of W's rows (gated: half of them gate, half up, so
// that a wave has both of a result in its own accumulators); x's rows are copied
// from where the plan says.
//
// 2047 x 2048 x 2048 gated (T, K, N), 64 experts of uneven size, 8 chosen, fp16: 136 us, 1.01
// PFLOP/s on the rows there are, bound by the conversion of W's codes beside the
// products (64 rows of x share one) and by the rows that tiles leave empty.  96 tokens: 32
// us a call among others on other weights, whose 142 MB come at 4.5 TB/s.
#include "mx_gemm16.hpp"
#include "mx_grouped_tile.hpp"

namespace wqbmm {

namespace {

template <int DT, bool SPLIT, int TM, int TN, bool GATED>
__device__ __forceinline__ void grouped16_products(const Grouped& a, const GroupTile& t, int cb, uint8_t* s0,
                                                   uint8_t* s1, mx_f4 (&acc)[TN][TM]) {
  using G = Gemm16<DT, SPLIT, TM, TN>;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t x0 = a.rows ? 0 : t.first, x_rows = a.rows ? a.R : t.rows, p0 = (int64_t)t.group * a.panels;
  Gemm16Operands<DT, SPLIT, TM, TN> o;
  o.x = {a.x + x0 * a.ldx, ((x_rows - 1) * a.ldx + (int64_t)a.blocks * kMxBlock) * 2};
  gemm16_rows(o, a.blocks, wave, lane, [&](int row) __attribute__((always_inline)) {
    const int from = grouped_row(a, t, row);
    return from < 0 ? 0 : (int)((from - x0) * a.ldx) * 2;
  });
  o.codes = {a.w.codes + p0 * a.w.kt * 1024, (int64_t)a.panels * a.w.kt * 1024};
  o.scales = {a.w.scales + p0 * a.w.kq * 256, (int64_t)a.panels * a.w.kq * 256};
#pragma unroll
  for (int c = 0; c < TN; ++c) o.panel[c] = grouped_panel<TN, G::WP, GATED>(wave * TN + c, cb, a.panels);
  // The first two K-tiles' scales are the same dwords; the loop's waits count both loads of them.
  int kt_lo = 0;
  asm volatile("" : "+s"(kt_lo));
  gemm16_loop<2>(o, a.blocks, a.w.kt, a.w.kq, kt_lo, a.w.kt, s0, s1, s1, acc);
}

template <int DT, bool SPLIT, int TM, int TN, bool GATED>
__device__ __forceinline__ void grouped16_tile(const Grouped& a, const GroupTile& t, int cb, uint8_t* s0, uint8_t* s1) {
  using G = Gemm16<DT, SPLIT, TM, TN>;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint32_t there = 0;
#pragma unroll
  for (int m = 0; m < TM; ++m) there |= (grouped_row(a, t, m * 16 + (lane & 15)) >= 0 ? 1u : 0u) << m;
  mx_f4 acc[TN][TM];
#pragma unroll
  for (int c = 0; c < TN; ++c)
#pragma unroll
    for (int m = 0; m < TM; ++m) acc[c][m] = mx_f4{0.f, 0.f, 0.f, 0.f};
  grouped16_products<DT, SPLIT, TM, TN, GATED>(a, t, cb, s0, s1, acc);
  mx_barrier();                                             // no wave reads the stages or copies into them any more
  constexpr int Q = GATED ? TN / 2 : TN;
  static_assert(2 * mx_stage_bytes<TM, Q>() <= G::STAGE, "the rows of two waves fit a stage");
  uint8_t* const mine = (wave < 2 ? s0 : s1) + (wave & 1) * mx_stage_bytes<TM, Q>();
  grouped_store<DT, TM, TN, GATED>(a, t, 0, (cb * G::WAVES + wave) * Q * kMxPanel, lane, there, mine, acc);
}

}  // namespace

// Tiles of 16 * TM places and 256 of W's rows, two workgroups a CU on rings of two stages:
// one's copies, look-ups and results pass while the other multiplies.  A tile with fewer
// rows is worked as 64 or 32 of them.  fp16: where not all of the tile's weights are exact
// in fp16, x in two bf16 parts, 64 rows at a time.
template <int DT, int TM, bool GATED>
__global__ __launch_bounds__(256, 2) void mx_grouped16_kernel(Grouped a, int cblocks) {
  constexpr int TN = 4;
  using G = Gemm16<DT, false, TM, TN>;
  // two variables: the compiler tells copies into one from reads of another
  __shared__ __attribute__((aligned(16))) uint8_t s0[G::STAGE], s1[G::STAGE];
  const int item = xcd_item(blockIdx.x), cb = item % cblocks;
  const GroupTile t = group_tile(a.offsets, a.G, a.S, G::BM, item / cblocks, false);
  if (t.group < 0) return;
  if constexpr (DT == MX_F16) {
    uint32_t flags = kMxFlagF16;
    for (int c = 0; c < G::WP; ++c)
      flags &= a.w.flags[(int64_t)t.group * a.panels + grouped_panel<TN, G::WP, GATED>(c, cb, a.panels)];
    if (!(flags & kMxFlagF16)) {
      GroupTile part = t;
      for (int m = 0; m < t.rows; m += 64) {
        part.first = t.first + m;
        part.rows = min(64, t.rows - m);
        grouped16_tile<DT, true, 4, TN, GATED>(a, part, cb, s0, s1);
        mx_wait_lds();
        mx_barrier();                                       // the results are read before the next rows are copied
      }
      return;
    }
  }
  if (t.rows <= 32) grouped16_tile<DT, false, 2, TN, GATED>(a, t, cb, s0, s1);
  else if (TM == 4 || t.rows <= 64) grouped16_tile<DT, false, 4, TN, GATED>(a, t, cb, s0, s1);
  else grouped16_tile<DT, false, TM, TN, GATED>(a, t, cb, s0, s1);
}

// W is converted once for a tile's rows, which takes as long as the products of 64 of
// them; tiles of 96 rows are faster where groups are large, and leave more rows
// empty where not.  us, 64 and 96 rows (128 on a ring of three stages, one workgroup a CU):
// 2047 x 2048 x 2048 gated (T, K, N), 64 experts, 8 chosen 132, 137 (147); 2048 x 11008 x
// 4096, 8, 2: 308, 271 (338); 2048 x 4096 x 8192 gated, 8, 2: 237, 221 (256); 300 x 4096
// x 4096, 4, 1: 28, 38 (46).
template <int DT, bool GATED>
static hipError_t grouped16_dt(const Grouped& a, hipStream_t stream) {
  auto go = [&](auto* kernel, int bm) {
    const int cblocks = (a.panels * kMxPanel + 255) / 256;
    const int64_t grid = (group_tiles(a.S, a.G, bm) * cblocks + 255) / 256 * 256;
    return mx_launch(kernel, dim3((unsigned)grid), dim3(256), stream, a, cblocks);
  };
  if (a.S >= 384 * (int64_t)a.G) return go(mx_grouped16_kernel<DT, 6, GATED>, 96);
  return go(mx_grouped16_kernel<DT, 4, GATED>, 64);
}

hipError_t launch_mx_grouped16(const Grouped& a, int dtype, bool gated, hipStream_t stream) {
  if (dtype == MX_F16) return gated ? grouped16_dt<MX_F16, true>(a, stream) : grouped16_dt<MX_F16, false>(a, stream);
  return gated ? grouped16_dt<MX_BF16, true>(a, stream) : grouped16_dt<MX_BF16, false>(a, stream);
}

// Tiles of 64 rows where there are about enough to fill the chip, from eight rows a group
// on; else, and where x or an expert's weights pass 31 bits, the kernel of few rows, whose
// workgroups are smaller and load less for a row that is not there.  us on one set of inputs,
// which the memory-side cache holds, few rows and tiles (with how many there are, as counted
// here; from memory, 96 x 2048 x 2048 takes 41 and 35 with 16-bit x, 40 and 37 with MXFP4 x):
//   16-bit x: 96 x 2048 x 2048 gated (T, K, N), 64 experts, 8 chosen (352) 30.4, 26.0;
//   100 x 4096 x 22016 gated, 8, 2 (602) 103, 84; 700 x 1056 x 1472 gated, 12, 3 (228)
//   27.9, 14.9; 300 x 4096 x 4096, 4, 1 (96) 25.1, 28.4; 200 x 1024 x 2048 gated, 16, 2 (112)
//   9.7, 12.7; 30 x 4096 x 4096, 1, 1 (0) 8.8, 23.3; with four rows a group 16 x 4096 x
//   22016 gated, 8, 2 (344) 62, 83; 32 x 2048 x 2048 gated, 64, 8 (288) 27.0, 25.1.
//   MXFP4 x, whose tiles have 128 columns: 96 x 2048 x 2048 gated, 64, 8 (704) 31.0, 29.8;
//   100 x 11008 x 4096, 8, 2 (224) 46.8, 34.6; 60 x 4096 x 11008, 2, 1 (86) 18.5, 16.5; 400 x
//   2048 x 2048, 8, 1 (160) 10.9, 12.8; 300 x 11008 x 2048, 2, 1 (80) 52, 34; 30 x 4096 x
//   4096, 1, 1 (0) 10.6, 15.2.
bool mx_use_grouped_tiles(const Grouped& a, int act) {
  const int64_t weights = (int64_t)a.panels * a.w.kt * 1024;
  const int64_t pitch = act ? (int64_t)a.w.kt * 64 : a.ldx * 2;          // bytes from row to row
  const int64_t x = pitch * (a.rows ? a.R : 256);
  if (weights >= kGroupedMaxBytes || x >= kGroupedMaxBytes) return false;
  const int64_t bn = act ? 128 : 256, items = (a.S / 64 + a.G / 2) * ((a.panels * kMxPanel + bn - 1) / bn);
  return a.S >= 8 * (int64_t)a.G && items >= (act ? 80 : 192);
}

}  // namespace wqbmm
