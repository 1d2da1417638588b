// mx_grouped.hip -- products with MXFP4 weights grouped by expert, ragged sizes, few
// rows a group: a workgroup takes some panels of 16 columns and up to 32 places of
// one group, which it finds from the offsets, so that one launch serves any
// distribution of the rows.  The waves share K (mx_expert.hpp).
//
// Bound by the weights' bytes after three trips to memory (offsets, rows, operands): 48 x
// 2048 x 2048 gated (T, K, N), 64 experts, 8 chosen, weights from memory, 37 us (142 MB, 3.9
// TB/s); one token 7.4 us, 5.6 with weights from the memory-side cache.
#include "grp_device.hpp"
#include "grp_launch.hpp"
#include "mx_expert.hpp"

namespace wqbmm {

namespace {

constexpr int FEW_WAVES = 4;

// Tile qm of 16 x 16 results of the P * MT sums: as it is, or gate and up together.
template <int P, int MT, bool GATED>
__device__ __forceinline__ mx_f4 result(const mx_f4* sums, int qm, int lane) {
  const mx_f4 v = total<P, MT>(sums, qm, FEW_WAVES, lane);
  if constexpr (!GATED) return v;
  else return gated(v, total<P, MT>(sums, P / 2 * MT + qm, FEW_WAVES, lane), 1.0f);
}

}  // namespace

// `MT` * 16 places of a tile.  P panels; gated: P / 2 of the gate, then the same P / 2 of up.
template <int DT, bool ACT4, bool GATED, int MT, int P>
__device__ __forceinline__ void few_rows(const Grouped& a, const GroupTile& t, int pb, const int* list,
                                         uint64_t rows_there, int wave, int lane, uint8_t* lds) {
  constexpr int Q = GATED ? P / 2 : P;
  const int half = GATED ? a.panels / 2 : a.panels;
  int64_t panel[P];
  uint32_t f16 = kMxFlagF16;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    panel[p] = (int64_t)t.group * a.panels + (p / Q) * half + min(pb * Q + p % Q, half - 1);
    if (DT == MX_F16 && !ACT4) f16 &= a.w.flags[panel[p]];
  }
  mx_f4 acc[P][MT];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[p][mt] = mx_f4{0.f, 0.f, 0.f, 0.f};
  uint8_t* const xs = lds + wave * (2 * PART_BYTES);
  auto row_at = [&](int i) __attribute__((always_inline)) { return list[i] * a.ldx; };
  auto units = [&](auto mode) __attribute__((always_inline)) {
    expert_units<DT, decltype(mode)::value, MT, P, true>(a.x, 0, row_at, a.w, panel, t.rows, a.blocks, wave, FEW_WAVES,
                                                           lane, xs, acc);
  };
  if constexpr (ACT4) units(std::integral_constant<Rows, Rows::kQuantized>{});
  else if (DT == MX_BF16 || f16) units(std::integral_constant<Rows, Rows::kAsIs>{});
  else units(std::integral_constant<Rows, Rows::kSplit>{});
  mx_f4* const sums = reinterpret_cast<mx_f4*>(lds);
  share_sums<P, MT>(sums, acc, wave, lane);
  for (int qm = wave; qm < Q * MT; qm += FEW_WAVES) {
    const int i = qm % MT * 16 + (lane & 15), n = (pb * Q + qm / MT) * kMxPanel + 4 * (lane >> 4);
    if (i >= t.rows || n >= a.n_out) continue;
    mx_f4 v = result<P, MT, GATED>(sums, qm, lane);
    if (!((rows_there >> i) & 1)) v = mx_f4{0.f, 0.f, 0.f, 0.f};
    *reinterpret_cast<uint2*>(a.y + (int64_t)(t.first + i) * a.n_out + n) = mx_pack4<DT>(v);
  }
}

template <int DT, bool ACT4, bool GATED, int P>
__global__ __launch_bounds__(FEW_WAVES * 64) void mx_grouped_few_kernel(Grouped a, int pblocks, int first) {
  constexpr int MINE = 2 * PART_BYTES;
  static_assert(MINE >= P * 2 * 1024, "a wave's sums");
  __shared__ __attribute__((aligned(16))) uint8_t lds[FEW_WAVES * MINE];
  __shared__ int lists[FEW_WAVES][32];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int item = first + blockIdx.x, pb = item % pblocks;
  const GroupTile t = group_tile(a.offsets, a.G, a.S, 32, item / pblocks, false);
  if (t.group < 0) return;                      // all waves find the same
  // The places' rows, each wave a list of its own; one outside x is read as row 0 and not used.
  int* const list = lists[wave];
  int row = -1;
  if (lane < t.rows) row = a.rows ? a.rows[t.first + lane] : t.first + lane;
  const bool there = row >= 0 && row < a.R;
  if (lane < 32) list[lane] = there ? row : 0;
  const uint64_t rows_there = __ballot(there);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  // up to 16 places: units twice as long, half the trips to memory
  if (t.rows <= 16) few_rows<DT, ACT4, GATED, 1, P>(a, t, pb, list, rows_there, wave, lane, lds);
  else few_rows<DT, ACT4, GATED, 2, P>(a, t, pb, list, rows_there, wave, lane, lds);
}

// Four panels a workgroup share the loads of its rows; two where the workgroups would make
// two rounds of the CUs or fewer.  us, four and two, weights from memory: 1 x 2048 x 2048
// gated (T, K, N), 64 experts, 8 chosen 8.1 and 7.4; 33 x 1056 x 1472 gated, 12, 3: 8.4 and
// 8.9 (from the memory-side cache 7.2 and 6.7); 16 x 11008 x 4096, 8, 2: 40.2 and 41.0; 200 x
// 1024 x 2048 gated, 16, 2: 12.2 and 14.8; 48 x 2048 x 2048 gated, 64, 8: 37.2 and 44.3.  (With
// 96 tokens, which are the tiled kernels' now, from that cache, 31.3 and 39.1: rows loaded in
// place, not staged, 34.8; eight panels 37.0; tiles of 16 or fewer rows worked as 32 33.8.)
template <int DT, bool ACT4, bool GATED>
static hipError_t few_dt(const Grouped& a, hipStream_t stream) {
  const int64_t tiles = group_tiles(a.S, a.G, 32);
  auto go = [&](auto* kernel, int panels) {
    const int pblocks = (a.n_out / kMxPanel + panels - 1) / panels;
    return in_launches(pblocks * tiles, [&](int64_t from, dim3 grid) {      // up to 2^27: S * N <= 2^38
      const int first = (int)from;
      return mx_launch(kernel, grid, dim3(FEW_WAVES * 64), stream, a, pblocks, first);
    });
  };
  const int four = GATED ? 2 : 4;               // panels of results of four panels of weights
  if ((a.n_out / kMxPanel + four - 1) / four * tiles <= 512) return go(mx_grouped_few_kernel<DT, ACT4, GATED, 2>, four / 2);
  return go(mx_grouped_few_kernel<DT, ACT4, GATED, 4>, four);
}

hipError_t launch_mx_grouped_few(const Grouped& a, int dtype, int act, bool gated, hipStream_t stream) {
  if (dtype == MX_F16) {
    if (act) return gated ? few_dt<MX_F16, true, true>(a, stream) : few_dt<MX_F16, true, false>(a, stream);
    return gated ? few_dt<MX_F16, false, true>(a, stream) : few_dt<MX_F16, false, false>(a, stream);
  }
  if (act) return gated ? few_dt<MX_BF16, true, true>(a, stream) : few_dt<MX_BF16, true, false>(a, stream);
  return gated ? few_dt<MX_BF16, false, true>(a, stream) : few_dt<MX_BF16, false, false>(a, stream);
}

}  // namespace wqbmm
