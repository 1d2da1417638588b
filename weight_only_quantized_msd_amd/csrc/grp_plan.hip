// grp_plan.hip -- the choice of experts, the order of rows by group, and the
// weighted sum of a token's experts.  Small calls take 3 to 4 us, a launch and two trips to
// memory; the figures of large ones stand at the kernels.
#include <algorithm>

#include "grp_device.hpp"
#include "grp_launch.hpp"
#include "mx_device.hpp"

namespace wqbmm {

namespace {

constexpr int ROUTE_WAVES = 4;

// Orders floats as unsigned integers, every NaN above +inf; -inf is 0, for "not there".
__device__ __forceinline__ uint32_t route_key(float f) {
  if (f != f) return 0xffffffffu;
  if (f == -__builtin_inff()) return 0u;
  const uint32_t u = __float_as_uint(f + 0.0f);       // -0 becomes +0: equal values tie
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  auto step = [&](uint32_t other) __attribute__((always_inline)) { v = max(v, other); };
  step(__builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));
  step(__builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));
  step(__builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));
  step(__builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));
  step(__builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));
  step(__builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));
  return __builtin_amdgcn_readlane(v, 63);
}

__device__ __forceinline__ float wave_total(float v) {
  auto step = [&](int other) __attribute__((always_inline)) { v += __int_as_float(other); };
  step(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x111, 0xf, 0xf, false));
  step(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x112, 0xf, 0xf, false));
  step(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x114, 0xf, 0xf, false));
  step(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x118, 0xf, 0xf, false));
  step(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x142, 0xa, 0xf, false));
  step(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x143, 0xc, 0xf, false));
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

template <int DT>
__device__ __forceinline__ float logit_at(const void* row, int e) {
  if constexpr (DT == MX_F32) return static_cast<const float*>(row)[e];
  else return mx_lo<DT>(static_cast<const uint16_t*>(row)[e]);
}

}  // namespace

// ---------------------------------------------------------------- choice of experts
// A wave per token: lane l holds the logits of experts 64 * r + l.  The largest
// key is taken k times; its first holder in order of index is the choice.  Bound by the
// instructions' issue: 8191 x 256 bf16 logits, 8 chosen, 7 us.  (Keys sorted in each lane
// first, so that only the lanes' first ones are compared: 8.0.  Sixteen lanes a token,
// four tokens a wave: a quarter of the instructions, but two waves a SIMD: 17.)
template <int DT, int R>
__global__ __launch_bounds__(ROUTE_WAVES * 64) void route_kernel(const void* __restrict__ logits, int64_t ld, int T,
                                                                 int E, int k, int renormalize,
                                                                 int32_t* __restrict__ ids,
                                                                 float* __restrict__ weights) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * ROUTE_WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= T) return;
  const char* const row = static_cast<const char*>(logits) + (int64_t)t * ld * (DT == MX_F32 ? 4 : 2);
  float f[R];
  uint32_t key[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const bool in = 64 * r + lane < E;
    f[r] = logit_at<DT>(row, in ? 64 * r + lane : 0);
    key[r] = in ? route_key(f[r]) : 0u;
  }
  int id = -1;
  uint32_t chosen = 0;                          // lane j: the key of choice j
  for (int j = 0; j < k; ++j) {
    uint32_t top = key[0];
#pragma unroll
    for (int r = 1; r < R; ++r) top = max(top, key[r]);
    top = wave_max(top);
    if (top == 0u) break;                       // nothing is left
    bool found = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint64_t same = __ballot(key[r] == top);
      if (!found && same != 0) {
        const int at = __ffsll((unsigned long long)same) - 1;
        found = true;
        if (lane == at) key[r] = 0u;
        if (lane == j) {
          id = 64 * r + at;
          chosen = top;
        }
      }
    }
  }
  // the key is a float's bits again (any NaN for a NaN)
  const float mine = __uint_as_float(chosen & 0x80000000u ? chosen == 0xffffffffu ? 0x7fc00000u : chosen & 0x7fffffffu
                                                          : ~chosen);
  const float top = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(mine), 0));
  const float p = id >= 0 ? expf(mine - top) : 0.0f;
  float sum = p;
  if (!renormalize) {                           // over all experts instead
    sum = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r)
      sum += 64 * r + lane < E && f[r] != -__builtin_inff() ? expf(f[r] - top) : 0.0f;
  }
  sum = wave_total(sum);
  if (lane < k) {
    ids[(int64_t)t * k + lane] = id;
    weights[(int64_t)t * k + lane] = id >= 0 ? p / sum : 0.0f;
  }
}

template <int DT>
static hipError_t route_dt(const void* logits, int64_t ld, int64_t T, int64_t E, int64_t k, int renormalize,
                           int32_t* ids, float* weights, hipStream_t stream) {
  const int t = (int)T, e = (int)E, kk = (int)k;
  auto go = [&](auto* kernel) {
    return mx_launch(kernel, dim3((unsigned)((T + ROUTE_WAVES - 1) / ROUTE_WAVES)), dim3(ROUTE_WAVES * 64), stream,
                     logits, ld, t, e, kk, renormalize, ids, weights);
  };
  if (E <= 64) return go(route_kernel<DT, 1>);
  if (E <= 128) return go(route_kernel<DT, 2>);
  if (E <= 256) return go(route_kernel<DT, 4>);
  if (E <= 512) return go(route_kernel<DT, 8>);
  return go(route_kernel<DT, 16>);
}

hipError_t launch_route(const void* logits, int dtype, int64_t ld, int64_t T, int64_t E, int64_t k, bool renormalize,
                        int32_t* ids, float* weights, hipStream_t stream) {
  auto* run = dtype == MX_F16 ? route_dt<MX_F16> : dtype == MX_BF16 ? route_dt<MX_BF16> : route_dt<MX_F32>;
  return run(logits, ld, T, E, k, renormalize ? 1 : 0, ids, weights, stream);
}

// ---------------------------------------------------------------- rows by group
// A stable counting sort.  Each wave of a workgroup takes a contiguous stretch of
// the choices, 64 at a time in order, and keeps a count for each group in LDS of its
// own: lanes with the same group find each other by comparing the group's bits
// (a ballot each), so a choice's rank is the count so far plus the lanes before
// it, and no atomics are needed whose order could change results.  The choices
// without a group are group G.
//   One workgroup does all of it for few choices.  More go to several workgroups,
// in two launches: each counts its stretch, then each adds up the counts of those
// before it and places its own.
//   us, one workgroup and several: 4096 choices of 64 groups 7.6, 10.1; 8192 11.4, 10.3.
// Several, with 1024, 2048 and 4096 choices each: 131072 of 128 groups 11.6, 12.4, 14.9; of
// 512 groups, whose counts weigh more, 22.5, 19.0, 21.2.
constexpr int64_t kSortOne = 6144;              // choices that one workgroup takes
constexpr int64_t kSortMaxBlocks = 128;

struct SortPlan {
  int waves;                                    // of a workgroup; its counts stay within 64 KB
  int64_t per_wave, blocks;                     // choices a wave, a multiple of 64
};
static SortPlan sort_plan(int64_t S, int64_t G) {
  SortPlan p;
  p.waves = G < 512 ? 16 : 8;
  const int64_t each = G <= 256 ? 1024 : 2048;
  const int64_t most = S <= kSortOne ? 1 : std::min(kSortMaxBlocks, (S + each - 1) / each);
  p.per_wave = std::max<int64_t>(64, ((S + most * p.waves - 1) / (most * p.waves) + 63) / 64 * 64);
  p.blocks = std::max<int64_t>(1, (S + p.per_wave * p.waves - 1) / (p.per_wave * p.waves));
  return p;
}
static size_t sort_lds(const SortPlan& p, int64_t G) { return (size_t)((p.waves + 2) * (G + 1) + p.waves) * 4; }

// The lanes whose key is this lane's.
__device__ __forceinline__ uint64_t same_key(int key, int bits) {
  uint64_t same = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const bool one = (key >> b) & 1;
    const uint64_t votes = __ballot(one);
    same &= one ? votes : ~votes;
  }
  return same;
}

// The key of choice i: its group, G for none, G + 1 past the end.
__device__ __forceinline__ int choice_key(const int32_t* __restrict__ ids, int i, int hi, int G) {
  if (i >= hi) return G + 1;
  const int id = ids[i];
  return id >= 0 && id < G ? id : G;
}
// The ranks of 64 choices among those with the same key, counted from what `counts`
// (LDS, a wave's own, G + 1) held, which they are added to.
__device__ __forceinline__ int rank_choices(int key, int G, int bits, int lane, int* counts) {
  const uint64_t same = same_key(key, bits), ahead = same & ((1ull << lane) - 1);
  const int so_far = key <= G ? counts[key] : 0;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (key <= G && ahead == 0) counts[key] = so_far + __popcll(same);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  return so_far + __popcll(ahead);
}

// PHASE 0: all of it, one workgroup.  1: a workgroup's counts to `block_counts`
// [block][G + 1].  2: with all blocks' counts, places.  A wave's choices, up to
// KEEP * 64, keep keys and ranks in registers; more are ranked a second time.
template <int PHASE, int WAVES, int KEEP>
__global__ __launch_bounds__(WAVES * 64) void group_rows_kernel(const int32_t* __restrict__ ids, int S, int k, int G,
                                                                int bits, int per_wave, int* __restrict__ block_counts,
                                                                int32_t* __restrict__ offsets,
                                                                int32_t* __restrict__ rows,
                                                                int32_t* __restrict__ slots) {
  extern __shared__ int lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int groups = G + 1;
  int* const mine = lds + wave * groups;        // [wave][G + 1]
  int* const totals = lds + WAVES * groups;     // [G + 1]: of all blocks, then the groups' first places
  int* const before = totals + groups;          // [G + 1]: of the blocks before this one
  int* const sums = before + groups;            // [waves]
  const int lo = min((int64_t)S, ((int64_t)blockIdx.x * WAVES + wave) * per_wave);
  const int hi = min((int64_t)S, (int64_t)lo + per_wave);
  for (int i = threadIdx.x; i < (WAVES + 2) * groups; i += WAVES * 64) lds[i] = 0;
  __syncthreads();
  int key[KEEP], rank[KEEP];
  if (per_wave <= KEEP * 64) {
#pragma unroll
    for (int j = 0; j < KEEP; ++j) key[j] = choice_key(ids, lo + j * 64 + lane, hi, G);
#pragma unroll
    for (int j = 0; j < KEEP; ++j)
      if (j * 64 < per_wave) rank[j] = rank_choices(key[j], G, bits, lane, mine);
  } else {
    for (int i0 = lo; i0 < hi; i0 += 64) rank_choices(choice_key(ids, i0 + lane, hi, G), G, bits, lane, mine);
  }
  if constexpr (PHASE == 2) {
    // a thread adds up a group's counts of every `parts`-th block, eight loads in flight
    // (one at a time, this kernel took 9.8 us for 131072 choices of 128 groups, 7.4 so);
    // then integers are added in LDS, in any order
    const int parts = max(1, WAVES * 64 / groups), blocks = gridDim.x;
    for (int i = threadIdx.x; i < parts * groups; i += WAVES * 64) {
      const int g = i % groups;
      int all = 0, ahead = 0;
      for (int b0 = i / groups; b0 < blocks; b0 += 8 * parts) {
        int n[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) n[j] = block_counts[min(b0 + j * parts, blocks - 1) * groups + g];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int b = b0 + j * parts;
          all += b < blocks ? n[j] : 0;
          ahead += b < (int)blockIdx.x ? n[j] : 0;
        }
      }
      atomicAdd(&totals[g], all);
      atomicAdd(&before[g], ahead);
    }
  }
  __syncthreads();
  for (int g = threadIdx.x; g < groups; g += WAVES * 64) {            // counts -> what the waves before have
    int n = PHASE == 2 ? before[g] : 0, c[WAVES];
#pragma unroll
    for (int w = 0; w < WAVES; ++w) c[w] = lds[w * groups + g];
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      lds[w * groups + g] = n;
      n += c[w];
    }
    if constexpr (PHASE == 1) block_counts[(int64_t)blockIdx.x * groups + g] = n;
    if constexpr (PHASE == 0) totals[g] = n;
  }
  if constexpr (PHASE == 1) return;
  __syncthreads();
  // totals -> first places
  int carry = 0;
  for (int g0 = 0; g0 < groups; g0 += WAVES * 64) {
    const int g = g0 + threadIdx.x, n = g < groups ? totals[g] : 0;
    const int upto = wave_prefix(n);
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    int ahead = carry, s[WAVES];
#pragma unroll
    for (int w = 0; w < WAVES; ++w) s[w] = sums[w];
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      if (w < wave) ahead += s[w];
      carry += s[w];
    }
    if (g < groups) {
      totals[g] = ahead + upto - n;
      if (blockIdx.x == 0) offsets[g] = ahead + upto - n;
    }
    __syncthreads();
  }
  auto place = [&](int i, int key, int at) __attribute__((always_inline)) {
    if (at >= S) return;                        // only if ids changed between the launches
    rows[at] = i / k;
    slots[i] = key < G ? at : -1;
  };
  if (per_wave <= KEEP * 64) {                  // `mine` now holds what is ahead of the wave's own
#pragma unroll
    for (int j = 0; j < KEEP; ++j)
      if (lo + j * 64 + lane < hi) place(lo + j * 64 + lane, key[j], totals[key[j]] + mine[key[j]] + rank[j]);
  } else {
    for (int i0 = lo; i0 < hi; i0 += 64) {
      const int k0 = choice_key(ids, i0 + lane, hi, G), r0 = rank_choices(k0, G, bits, lane, mine);
      if (i0 + lane < hi) place(i0 + lane, k0, totals[k0] + r0);
    }
  }
}

size_t group_rows_workspace_bytes(int64_t S, int64_t G) {
  return S <= kSortOne ? 0 : (size_t)(sort_plan(S, G).blocks * (G + 1)) * 4;
}

hipError_t launch_group_rows(const int32_t* ids, int64_t T, int64_t k, int64_t G, int32_t* offsets, int32_t* rows,
                             int32_t* slots, uint8_t* ws, hipStream_t stream) {
  const int64_t S = T * k;
  const SortPlan p = sort_plan(S, G);
  const int s = (int)S, kk = (int)k, g = (int)G, per = (int)p.per_wave;
  int bits = 0;
  while ((G + 1) >> bits) ++bits;               // keys up to G + 1
  int* counts = reinterpret_cast<int*>(ws);
  auto go = [&](auto* kernel) {
    return mx_launch_shared(kernel, dim3((unsigned)p.blocks), dim3(p.waves * 64), sort_lds(p, G), stream, ids, s, kk, g,
                            bits, per, counts, offsets, rows, slots);
  };
  auto all = [&](auto waves) {
    constexpr int WAVES = decltype(waves)::value, KEEP = 16;
    if (S <= kSortOne) return go(group_rows_kernel<0, WAVES, KEEP>);
    const hipError_t e = go(group_rows_kernel<1, WAVES, KEEP>);
    return e != hipSuccess ? e : go(group_rows_kernel<2, WAVES, KEEP>);
  };
  return p.waves == 16 ? all(std::integral_constant<int, 16>{}) : all(std::integral_constant<int, 8>{});
}

// ---------------------------------------------------------------- weighted sum
// A thread takes eight columns of a token, up to four of its choices in flight.  Bound by
// memory: 4095 tokens, 8 choices, 4096 columns, with a base: 65 us, 5.1 TB/s.
template <int DT>
__global__ __launch_bounds__(256) void combine_kernel(const uint16_t* __restrict__ z, int64_t ldz, int S,
                                                      const int32_t* __restrict__ slots,
                                                      const float* __restrict__ weights, int k, const uint16_t* base,
                                                      int64_t ldb, uint16_t* y, int64_t ldy, uint32_t units,
                                                      int64_t count, uint32_t first) {
  const int64_t i = (int64_t)(first + blockIdx.x) * 256 + threadIdx.x;  // of count = T * units
  if (i >= count) return;
  const int64_t t = i / units, c = (i - t * units) * 8;
  float v[8] = {};
  if (base) {
    const uint4 b = *reinterpret_cast<const uint4*>(base + t * ldb + c);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = mx_lo<DT>(dword_of(b, q));
      v[2 * q + 1] = mx_hi<DT>(dword_of(b, q));
    }
  }
#pragma unroll 4
  for (int j = 0; j < k; ++j) {
    const int slot = slots[t * k + j];
    if (slot < 0 || slot >= S) continue;
    const float w = weights[t * k + j];
    const uint4 a = *reinterpret_cast<const uint4*>(z + slot * ldz + c);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = __builtin_fmaf(w, mx_lo<DT>(dword_of(a, q)), v[2 * q]);
      v[2 * q + 1] = __builtin_fmaf(w, mx_hi<DT>(dword_of(a, q)), v[2 * q + 1]);
    }
  }
  uint32_t o[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) o[q] = mx_round16<DT>(v[2 * q]) | (uint32_t)mx_round16<DT>(v[2 * q + 1]) << 16;
  *reinterpret_cast<uint4*>(y + t * ldy + c) = make_uint4(o[0], o[1], o[2], o[3]);
}

hipError_t launch_combine(const void* z, int dtype, int64_t ldz, int64_t S, int64_t H, const int32_t* slots,
                          const float* weights, int64_t T, int64_t k, const void* base, int64_t ldb, void* y,
                          int64_t ldy, hipStream_t stream) {
  auto* zp = static_cast<const uint16_t*>(z);
  auto* bp = static_cast<const uint16_t*>(base);
  auto* yp = static_cast<uint16_t*>(y);
  const uint32_t units = (uint32_t)(H / 8);
  const int64_t count = T * units;
  const int s = (int)S, kk = (int)k;
  auto* kernel = dtype == MX_F16 ? combine_kernel<MX_F16> : combine_kernel<MX_BF16>;
  return in_launches((count + 255) / 256, [&](int64_t from, dim3 grid) {    // up to 2^27: T * H <= 2^38
    const uint32_t first = (uint32_t)from;
    return mx_launch(kernel, grid, dim3(256), stream, zp, ldz, s, slots, weights, kk, bp, ldb, yp, ldy, units, count,
                     first);
  });
}

}  // namespace wqbmm
