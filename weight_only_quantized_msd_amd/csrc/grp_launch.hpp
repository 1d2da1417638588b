// grp_launch.hpp -- internal launcher interface of the operators whose weights
// depend on the row (include/wqbmm_grouped.h).  Not part of the C ABI.
#pragma once

#include "mx_launch.hpp"

namespace wqbmm {

constexpr int kMaxGroups = 1024;
constexpr int kRouteMaxK = 16;
constexpr int kLoraMaxR = 256;

// A plan's tiles of `most` places, at most.
inline int64_t group_tiles(int64_t S, int64_t G, int64_t most) { return S / most + (G < S ? G : S); }

// A grid holds fewer than 2^32 threads: workgroups of 256 go in as many launches as that
// takes, each told its first one's number.
template <typename Go>
hipError_t in_launches(int64_t workgroups, Go&& go) {
  constexpr int64_t kMost = int64_t(1) << 23;
  hipError_t e = hipSuccess;
  for (int64_t first = 0; first < workgroups && e == hipSuccess; first += kMost)
    e = go(first, dim3((unsigned)(workgroups - first < kMost ? workgroups - first : kMost)));
  return e;
}

hipError_t launch_route(const void* logits, int dtype, int64_t ld, int64_t T, int64_t E, int64_t k, bool renormalize,
                        int32_t* ids, float* weights, hipStream_t stream);

size_t group_rows_workspace_bytes(int64_t S, int64_t G);
hipError_t launch_group_rows(const int32_t* ids, int64_t T, int64_t k, int64_t G, int32_t* offsets, int32_t* rows,
                             int32_t* slots, uint8_t* ws, hipStream_t stream);

hipError_t launch_combine(const void* z, int dtype, int64_t ldz, int64_t S, int64_t H, const int32_t* slots,
                          const float* weights, int64_t T, int64_t k, const void* base, int64_t ldb, void* y,
                          int64_t ldy, hipStream_t stream);

// A grouped product's operands.
struct Grouped {
  const uint16_t* x;
  int64_t ldx, R;              // x's rows
  const int32_t* rows;         // NULL: x's rows are the places
  const int32_t* offsets;
  int G, S, blocks;            // blocks of 32 along K
  int panels;                  // a group's panels of 16 rows of W
  MxTiled w;
  uint16_t* y;
  int n_out;
};
hipError_t launch_mx_grouped_few(const Grouped& a, int dtype, int act, bool gated, hipStream_t stream);

// Tiled products address an expert's weights and x (or a tile of it) with 31 bits.
constexpr int64_t kGroupedMaxBytes = int64_t(1) << 31;
bool mx_use_grouped_tiles(const Grouped& a, int act);
hipError_t launch_mx_grouped16(const Grouped& a, int dtype, bool gated, hipStream_t stream);
size_t mx_grouped4_workspace_bytes(const Grouped& a);
hipError_t launch_mx_grouped4(const Grouped& a, int dtype, bool gated, uint8_t* ws, hipStream_t stream);

struct Lora {
  const uint16_t* x;
  int64_t ldx;
  int M, K, N, r, L;
  const uint16_t *a, *b;
  const float* scales;
  const int32_t *offsets, *rows;
  const uint16_t* base;
  int64_t ldb;
  uint16_t* y;
  int64_t ldy;
};
struct LoraPlan {
  int splits, kt_per;          // K-splits of the first product, K-tiles of 128 each
  size_t bytes;                // workspace: its partial sums
};
LoraPlan lora_plan(int64_t M, int64_t K, int64_t r, int64_t L);
hipError_t launch_lora(const Lora& a, int dtype, const LoraPlan& plan, float* part, hipStream_t stream);

}  // namespace wqbmm
