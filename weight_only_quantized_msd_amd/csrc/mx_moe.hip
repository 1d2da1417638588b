// mx_moe.hip -- a mixture-of-experts layer with MXFP4 experts for up to 64
// tokens, in four launches:
//   route: logits = router . x, softmax, the k largest per token;
//   up:    h = weight * silu(gate_e . x) * (up_e . x) for every (token, choice)
//          pair, a workgroup for a reached expert and one or two panels of 16
//          rows of I;
//   down:  down_e . h for every pair, a workgroup for a reached expert and four
//          panels of 16 columns of y;
//   sum:   y = the sum of a token's pairs.
// Each reached expert's weights are read by one workgroup a panel (once, or once
// for every 32 of its rows); every sum has a fixed order.  There is no hand-off
// between workgroups inside a launch: each workgroup finds its expert's pairs
// itself from the ids (at most 1024 of them).
//
// Bound by the weights: 16 tokens, H = 4096, I = 11008, 8 experts, 2 chosen: route
// 6 us, up 73 (383 MB, 5.2 TB/s), down 41 (191 MB, 4.7 TB/s), sum 4.  Small layers
// are bound by the chain of launches and trips to memory: 33 tokens, H = 1056, I =
// 736, 12 experts, 3 chosen: 4.6 + 7.9 + 5.8 + 2.5 us.
//
// One token, and few, are taken by themselves in three launches, at the end of
// this file: 1 token, H = 2048, I = 1024, 64 experts, 8 chosen: 2.8 + 8.1 + 5.1 us.
#include <algorithm>

#include "mx_tile.hpp"

namespace wqbmm {

namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// Orders floats as unsigned integers, every NaN above +inf.
__device__ __forceinline__ uint32_t order_key(float f) {
  if (f != f) return 0xffffffffu;
  const uint32_t u = __float_as_uint(f + 0.0f);       // -0 becomes +0: equal values tie
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

}  // namespace

// ---------------------------------------------------------------- routing
constexpr int ROUTE_WAVES = 16;

// A wave's logits of N experts, lanes along H, with up to 4 * N loads of the
// router in flight (one expert and one load at a time: 11.7 us for 1 token, 64
// experts, H = 2048; this way, four experts a wave, 6.8).
template <int DT, int N>
__device__ __forceinline__ void router_logits(const uint4* __restrict__ xr, const uint16_t* __restrict__ router, int H,
                                              int E, int e0, int lane, float (&s)[N]) {
  constexpr int CB = 4;                         // chunks of x at a time
  const int chunks = H / 8;
  const uint4* rr[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    rr[i] = reinterpret_cast<const uint4*>(router + (int64_t)min(e0 + i, E - 1) * H);
    s[i] = 0.0f;
  }
  for (int c0 = 0; c0 < chunks; c0 += 64 * CB) {
    uint4 a[CB], b[N][CB];
#pragma unroll
    for (int j = 0; j < CB; ++j) {
      const int c = c0 + j * 64 + lane;
      const bool in = c < chunks;
      a[j] = in ? xr[c] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int i = 0; i < N; ++i) b[i][j] = in ? rr[i][c] : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int j = 0; j < CB; ++j)
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          s[i] = __builtin_fmaf(mx_lo<DT>(dword_of(a[j], q)), mx_lo<DT>(dword_of(b[i][j], q)), s[i]);
          s[i] = __builtin_fmaf(mx_hi<DT>(dword_of(a[j], q)), mx_hi<DT>(dword_of(b[i][j], q)), s[i]);
        }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = wave_sum(s[i]);
}

// The choices of one token, by one wave: lane l holds the logits f[r] of experts
// 64 * r + l.  Lane j < k gets the j-th choice (larger logit first, then lower
// index), and `mine / wave_sum(sum)` is its softmax weight.
struct Choice {                                 // of the wave's own, in LDS
  int id[kMoeMaxK];
  float logit[kMoeMaxK];
};

// How many of the first n lanes are ahead of each lane.
__device__ __forceinline__ int lanes_ahead(uint32_t key, int n, int lane) {
  int ahead = 0;
  for (int j = 0; j < n; ++j) {
    const uint32_t other = (uint32_t)__builtin_amdgcn_readlane((int)key, j);
    ahead += other > key || (other == key && j < lane);
  }
  return ahead;
}

// Up to 32 experts are ranked as they are.  Of more, the k-th largest key is
// found bit by bit (a comparison and a count of lanes each); the experts above
// it, and as many of those equal to it as there is room for, lowest index first,
// are ranked.  (One token, us of the layer: H = 4096, I = 1024, 256 experts, 8
// chosen 35 ranked by all waves of a workgroup, 21 this way; 2048, 1024, 64, 8
// 16.9 ranked, 15.2 this way; 512, 256, 4, 1 10.0 this way, 9.0 ranked.)
template <int R, bool RANK>
__device__ __forceinline__ void choose_from(const float (&f)[R], Choice& c, int E, int k, bool renormalize, int lane,
                                            int& my_id, float& mine, float& sum) {
  uint32_t key[R];
#pragma unroll
  for (int r = 0; r < R; ++r) key[r] = 64 * r + lane < E ? order_key(f[r]) : 0u;    // no float has key 0
  int rank;
  float my_logit;
  if constexpr (RANK) {
    rank = lanes_ahead(key[0], E, lane);
    my_id = lane;
    my_logit = f[0];
  } else {
    uint32_t kth = 0;
#pragma unroll
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t at = kth | 1u << bit;
      int n = 0;
#pragma unroll
      for (int r = 0; r < R; ++r) n += __popcll(__ballot(key[r] >= at));
      if (n >= k) kth = at;
    }
    int room = k, n = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) room -= __popcll(__ballot(key[r] > kth));
    const uint64_t below = (1ull << lane) - 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint64_t same = __ballot(key[r] == kth);
      const bool in = key[r] > kth || (key[r] == kth && __popcll(same & below) < room);
      room -= min(room, __popcll(same));
      const uint64_t all = __ballot(in);
      if (in) {
        c.id[n + __popcll(all & below)] = 64 * r + lane;
        c.logit[n + __popcll(all & below)] = f[r];
      }
      n += __popcll(all);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    my_id = c.id[min(lane, k - 1)];
    my_logit = c.logit[min(lane, k - 1)];
    rank = lanes_ahead(order_key(my_logit), k, lane);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  if (lane < (RANK ? E : k) && rank < k) {
    c.id[rank] = my_id;
    c.logit[rank] = my_logit;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  my_id = lane < k ? c.id[lane] : 0;
  const float top = c.logit[0];
  mine = lane < k ? expf(c.logit[lane] - top) : 0.0f;
  sum = mine;
  if (!renormalize) {                           // over all experts instead
    sum = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) sum += 64 * r + lane < E ? expf(f[r] - top) : 0.0f;
  }
}
__device__ __forceinline__ void choose(const float* logits, Choice& c, int E, int k, bool renormalize, int lane,
                                       int& my_id, float& mine, float& sum) {
  auto from = [&](auto rc, auto rank) __attribute__((always_inline)) {
    constexpr int R = decltype(rc)::value;
    float f[R];
#pragma unroll
    for (int r = 0; r < R; ++r) f[r] = logits[min(64 * r + lane, E - 1)];
    choose_from<R, decltype(rank)::value>(f, c, E, k, renormalize, lane, my_id, mine, sum);
  };
  if (E <= 32) from(std::integral_constant<int, 1>{}, std::true_type{});
  else if (E <= 64) from(std::integral_constant<int, 1>{}, std::false_type{});
  else from(std::integral_constant<int, kMoeMaxE / 64>{}, std::false_type{});
}

// One workgroup per token, four experts a wave at a time.
template <int DT>
__global__ __launch_bounds__(ROUTE_WAVES * 64) void mx_route_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                                    const uint16_t* __restrict__ router, int H,
                                                                    int E, int k, int renormalize,
                                                                    int32_t* __restrict__ ids,
                                                                    float* __restrict__ weights) {
  __shared__ float logits[kMoeMaxE];
  __shared__ Choice c;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = blockIdx.x;
  constexpr int N = 4;
  for (int e0 = wave * N; e0 < E; e0 += ROUTE_WAVES * N) {
    float s[N];
    router_logits<DT, N>(reinterpret_cast<const uint4*>(x + t * ldx), router, H, E, e0, lane, s);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (lane == 0 && e0 + i < E) logits[e0 + i] = s[i];
  }
  __syncthreads();
  if (wave != 0) return;
  int id;
  float mine, sum;
  choose(logits, c, E, k, renormalize != 0, lane, id, mine, sum);
  sum = wave_sum(sum);
  if (lane < k) {
    ids[t * k + lane] = id;
    weights[t * k + lane] = mine / sum;
  }
}

// ---------------------------------------------------------------- an expert's pairs
// Which expert a slot stands for: where there are fewer pairs (token * k +
// choice) than experts, slot i is pair i's expert, if no pair before i has the
// same; else slot i is expert i.  `list` (LDS of this wave's own, T entries)
// gets the expert's pairs in ascending order, for all lanes.  Returns the expert,
// or -1 if the slot is empty.  Each wave does this by itself: no barrier stands
// between the ids and the first load of weights.
__device__ __forceinline__ int slot_pairs(const int32_t* __restrict__ ids, int pairs, int E, int slot, int lane,
                                          uint16_t* list, int& count) {
  const bool by_pair = pairs < E;
  const int expert = by_pair ? ids[slot] : slot;
  int n = 0;
  bool mine = true;
  for (int p0 = 0; p0 < pairs; p0 += 64) {
    const int p = p0 + lane;
    const bool hit = p < pairs && ids[p] == expert;
    const uint64_t votes = __ballot(hit);
    if (hit) list[n + __popcll(votes & ((1ull << lane) - 1))] = (uint16_t)p;
    if (by_pair && n == 0 && votes != 0) mine = p0 + __ffsll((unsigned long long)votes) - 1 == slot;
    n += __popcll(votes);
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");      // lanes read what others wrote
  count = n;
  return n > 0 && mine ? expert : -1;
}

// ---------------------------------------------------------------- products
// Both products of an expert are the same contraction: P panels of its weights
// with the rows of its pairs (tokens' x; h), the waves of a workgroup taking
// units of U K-tiles in turn.  The rows come in one of two ways:
//   staged: each wave copies a unit's rows to LDS of its own (8 to 24 KB), 1 KB of
//     whole rows a copy, the 16-byte chunks of a row permuted (chunk ^ row % 16);
//   direct: each lane loads its 16-byte operands, which touches a cache line a
//     lane, but needs no LDS, so more workgroups share a CU.
// moe_dt says which.
enum class Rows {
  kAsIs,       // 16-bit
  kSplit,      // fp16 as two bf16
  kParts,      // h's three parts, added in the accumulators
  kPartRows    // h's parts as rows of their own
};
constexpr int PART_BYTES = 8 * 1024;           // staged rows of a wave: two of these, three for kParts

// h goes from one product to the other in 24 bits, fp32's, as three bf16 parts,
// whose products with the weights are exact, at h, h + part and h + 2 * part.  (In
// two parts, 16 bits, the layer's outputs were 1.1e-4 of their norm away from sums
// in fp32 at 16 x 4096 x 11008, 8 experts, 2 chosen, and are 0.6e-4 now; the layer
// took 129 us.  h in fp32, cut by the down product, took 144.)
__device__ __forceinline__ void store_h(uint16_t* __restrict__ h, int64_t part, int64_t at, mx_f4 v) {
  uint2 o[3];
  mx_split24(v, o);
#pragma unroll
  for (int n = 0; n < 3; ++n) *reinterpret_cast<uint2*>(h + n * part + at) = o[n];
}

// share * silu(a) * b
__device__ __forceinline__ mx_f4 gated(mx_f4 a, mx_f4 b, float share) {
  mx_f4 h;
#pragma unroll
  for (int j = 0; j < 4; ++j) h[j] = a[j] / (1.0f + expf(-a[j])) * b[j] * share;
  return h;
}

// h's rows, one for each pair, hold whole K-tiles (what lies past I is not used).
__host__ __device__ inline int64_t h_pitch(int64_t I) { return (I + 127) / 128 * 128; }

// Where h's value i of a row stands.  Within a K-tile of 128 values the 16-byte
// chunks are ordered (slice j, block g) instead of (g, j): the four lanes that
// read a row's slice j then read 64 bytes in a row.
__device__ __forceinline__ int h_place(int i) {
  return (i & ~127) | ((i & 24) << 2) | ((i & 96) >> 2) | (i & 7);
}

// row_at(i): the first value of row i, as an offset into `src`; h's parts are
// `part` values apart.
template <int DT, Rows MODE, int MT, int P, bool STAGED, typename RowAt>
__device__ __forceinline__ void expert_units(const uint16_t* __restrict__ src, int64_t part, RowAt&& row_at,
                                             const MxTiled& w, const int64_t (&panel)[P], int rows, int blocks,
                                             int wave, int waves, int lane, uint8_t* xs, mx_f4 (&acc)[P][MT]) {
  constexpr bool H = MODE == Rows::kParts || MODE == Rows::kPartRows;
  constexpr int PARTS = MODE == Rows::kParts ? 3 : 1, TERMS = MODE == Rows::kSplit ? 2 : PARTS;
  constexpr int U = !H ? (STAGED ? 4 / MT : 4) : !STAGED ? 2 : PARTS > 1 ? 1 : 2 / MT;
  constexpr int LANES = 16 * U, ROWS = 64 / LANES;
  constexpr int CT = MODE == Rows::kAsIs ? DT : MX_BF16;
  const int r = lane & 15, g = lane >> 4;
  auto chunk_of = [&](int i, int j) __attribute__((always_inline)) { return H ? 16 * i + 4 * j + g : 16 * i + 4 * g + j; };
  for (int kt = wave * U; kt < w.kt; kt += waves * U) {
    if constexpr (STAGED) {
      mx_wait_lds();                              // the last unit's reads, before its rows are overwritten
#pragma unroll
      for (int i = 0; i < 16 * MT / ROWS; ++i) {
        if (i * ROWS >= rows) break;
        const int row = i * ROWS + lane / LANES;
        const int chunk = kt * 16 + ((lane % LANES) ^ (row & 15));
        const bool in = chunk < (H ? w.kt * 16 : blocks * 4);
        const uint16_t* const from = src + row_at(min(row, rows - 1)) + (in ? chunk * 8 : 0);
#pragma unroll
        for (int n = 0; n < PARTS; ++n)
          __builtin_amdgcn_global_load_lds(from + n * part, xs + n * PART_BYTES + i * 1024, 16, 0, 0);
      }
    }
    uint4 c[P][U];
    uint32_t sc[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
#pragma unroll
      for (int i = 0; i < U; ++i)
        c[p][i] = *reinterpret_cast<const uint4*>(w.codes + ((panel[p] * w.kt + min(kt + i, w.kt - 1)) * 64 + lane) * 16);
      sc[p] = *reinterpret_cast<const uint32_t*>(w.scales + ((panel[p] * w.kq + kt / 4) * 64 + lane) * 4) >> (8 * (kt & 3));
    }
    if constexpr (STAGED) mx_wait_vm<0>();
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (kt + i >= w.kt) break;                  // uniform: the last unit's missing tiles
      const bool whole = 4 * (kt + i) + 4 <= blocks, in = 4 * (kt + i) + g < blocks;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        uint4 v[4][TERMS];
        if constexpr (STAGED) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int n = 0; n < PARTS; ++n)
              v[j][n] = *reinterpret_cast<const uint4*>(xs + n * PART_BYTES + (mt * 16 + r) * (LANES * 16) +
                                                        (chunk_of(i, j) ^ r) * 16);
          if (!whole) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int n = 0; n < PARTS; ++n) v[j][n] = in ? v[j][n] : make_uint4(0u, 0u, 0u, 0u);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int n = 0; n < PARTS; ++n) v[j][n] = make_uint4(0u, 0u, 0u, 0u);
          if (mt * 16 + r < rows && in) {
            const uint16_t* const from = src + row_at(mt * 16 + r) + kt * kMxTile;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int n = 0; n < PARTS; ++n)
                v[j][n] = *reinterpret_cast<const uint4*>(from + n * part + chunk_of(i, j) * 8);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (MODE == Rows::kSplit) {
            const uint4 both = v[j][0];
            mx_split8(both, v[j][0], v[j][1]);
          }
#pragma unroll
          for (int p = 0; p < P; ++p) {
            const uint4 a = mx_decode8<CT>(dword_of(c[p][i], j), mx_scale((sc[p] >> (8 * i)) & 0xffu));
#pragma unroll
            for (int n = 0; n < TERMS; ++n) acc[p][mt] = mx_mfma16<CT>(a, v[j][n], acc[p][mt]);
          }
        }
      }
    }
  }
}

// The waves' sums -> part [wave][P * MT][64]; call with all waves, after which
// total(i) adds sum i of the P * MT over the waves, in wave order.
template <int P, int MT>
__device__ __forceinline__ void share_sums(mx_f4* part, const mx_f4 (&acc)[P][MT], int wave, int lane) {
  __syncthreads();                                // the staged rows lie in the same memory
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) part[(wave * P * MT + p * MT + mt) * 64 + lane] = acc[p][mt];
  __syncthreads();
}
template <int P, int MT>
__device__ __forceinline__ mx_f4 total(const mx_f4* part, int i, int waves, int lane) {
  mx_f4 v = part[i * 64 + lane];
  for (int s = 1; s < waves; ++s) v += part[(s * P * MT + i) * 64 + lane];
  return v;
}

// h of `rows` pairs from `first` on, for Q panels of 16 rows of I; UP_WAVES waves.
constexpr int UP_WAVES = 4;
template <int DT, int MT, int Q, bool STAGED, typename RowAt, typename PairOf, typename ShareOf>
__device__ __forceinline__ void up_rows(const uint16_t* __restrict__ x, RowAt&& row_at, PairOf&& pair_of,
                                        ShareOf&& share_of, const MxTiled& w, int expert, int rows, int blocks, int I,
                                        int wave, int lane, uint8_t* lds, uint16_t* __restrict__ h, int64_t part) {
  constexpr int P = 2 * Q;                        // gate panels, then up panels
  uint8_t* const xs = lds + wave * (2 * PART_BYTES);
  mx_f4* const sums = reinterpret_cast<mx_f4*>(lds);
  int64_t panel[P];
  uint32_t f16 = kMxFlagF16;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    panel[q] = (int64_t)expert * (2 * I / kMxPanel) + min((int)blockIdx.x * Q + q, I / kMxPanel - 1);
    panel[Q + q] = panel[q] + I / kMxPanel;
    if (DT == MX_F16) f16 &= w.flags[panel[q]] & w.flags[panel[Q + q]];
  }
  mx_f4 acc[P][MT];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[p][mt] = mx_f4{0.f, 0.f, 0.f, 0.f};
  if (DT == MX_BF16 || f16)
    expert_units<DT, Rows::kAsIs, MT, P, STAGED>(x, 0, row_at, w, panel, rows, blocks, wave, UP_WAVES, lane, xs, acc);
  else
    expert_units<DT, Rows::kSplit, MT, P, STAGED>(x, 0, row_at, w, panel, rows, blocks, wave, UP_WAVES, lane, xs, acc);
  share_sums<P, MT>(sums, acc, wave, lane);
  for (int qm = wave; qm < Q * MT; qm += UP_WAVES) {
    const int i = qm % MT * 16 + (lane & 15);
    const int at = (blockIdx.x * Q + qm / MT) * kMxPanel + 4 * (lane >> 4);
    if (i >= rows || at >= I) continue;
    const mx_f4 a = total<P, MT>(sums, qm, UP_WAVES, lane), b = total<P, MT>(sums, Q * MT + qm, UP_WAVES, lane);
    store_h(h, part, pair_of(i) * h_pitch(I) + h_place(at), gated(a, b, share_of(i)));
  }
}

// Workgroup (Q panels of 16 rows of I, slot): h for all pairs of the slot's expert.
// Direct: four waves a SIMD, i.e. at most 128 registers.
template <int DT, int Q, bool STAGED>
__global__ __launch_bounds__(UP_WAVES * 64, STAGED ? 1 : 4) void mx_moe_up_kernel(
    const uint16_t* __restrict__ x, int64_t ldx, MxTiled w, const int32_t* __restrict__ ids,
    const float* __restrict__ weights, int pairs, int E, int k, int blocks, int I, uint16_t* __restrict__ h,
    int64_t part) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[UP_WAVES * (STAGED ? 2 * PART_BYTES : 4 * Q * 1024)];
  __shared__ uint16_t lists[UP_WAVES][kMoeMaxT];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint16_t* const list = lists[wave];
  int count = 0;
  const int expert = __builtin_amdgcn_readfirstlane(slot_pairs(ids, pairs, E, blockIdx.y, lane, list, count));
  if (expert < 0) return;                         // all waves find the same
  count = __builtin_amdgcn_readfirstlane(count);
  auto rows_from = [&](auto mt_c, int first) __attribute__((always_inline)) {
    constexpr int MT = decltype(mt_c)::value;
    up_rows<DT, MT, Q, STAGED>(
        x, [&](int i) __attribute__((always_inline)) { return (int64_t)(list[first + i] / k) * ldx; },
        [&](int i) __attribute__((always_inline)) { return (int)list[first + i]; },
        [&](int i) __attribute__((always_inline)) { return weights[list[first + i]]; }, w, expert,
        min(count - first, MT * 16), blocks, I, wave, lane, lds, h, part);
  };
  int first = 0;
  for (; count - first > 16; first += 32) {
    rows_from(std::integral_constant<int, 2>{}, first);
    __syncthreads();                              // the sums are read before they are overwritten
  }
  if (first < count) rows_from(std::integral_constant<int, 1>{}, first);
}

// Workgroup (four panels of 16 columns of y, slot): the expert's share of y, fp32,
// for each of its pairs.  The parts of h are three products for a pair's column; or,
// for few pairs, three columns of one product, whose sixteen hold five pairs.
// (Two panels took longer everywhere, direct, us: 48 x 2048 x 1024, 16 experts, 8
// chosen 26.6 and 18.2; 33 x 1056 x 736, 12, 3: 6.8 and 6.6.)
constexpr int DOWN_PANELS = 4;
enum class Down { kDirect, kStaged, kFew };
constexpr int down_waves(Down kind) { return kind == Down::kDirect ? 4 : kind == Down::kStaged ? 6 : 8; }
template <Down KIND>
__global__ __launch_bounds__(down_waves(KIND) * 64) void mx_moe_down_kernel(const uint16_t* __restrict__ h,
                                                                           int64_t part, MxTiled w,
                                                                           const int32_t* __restrict__ ids, int pairs,
                                                                           int E, int I, int H,
                                                                           float* __restrict__ sums) {
  constexpr int P = DOWN_PANELS, WAVES = down_waves(KIND);
  constexpr int MOST = KIND == Down::kFew ? 10 : 32;                     // pairs at a time
  constexpr int MINE = KIND == Down::kDirect ? 2 * P * 1024 : (KIND == Down::kFew ? 1 : 3) * PART_BYTES;
  static_assert(MINE >= 2 * P * 1024, "a wave's sums");
  __shared__ __attribute__((aligned(16))) uint8_t lds[WAVES * MINE];
  __shared__ uint16_t lists[WAVES][kMoeMaxT];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint16_t* const list = lists[wave];
  mx_f4* const shared = reinterpret_cast<mx_f4*>(lds);
  int count = 0;
  const int expert = __builtin_amdgcn_readfirstlane(slot_pairs(ids, pairs, E, blockIdx.y, lane, list, count));
  if (expert < 0) return;
  count = __builtin_amdgcn_readfirstlane(count);
  int64_t panel[P];
#pragma unroll
  for (int p = 0; p < P; ++p)
    panel[p] = (int64_t)expert * (H / kMxPanel) + min((int)blockIdx.x * P + p, H / kMxPanel - 1);

  auto pairs_from = [&](auto mt_c, int first) __attribute__((always_inline)) {
    constexpr int MT = decltype(mt_c)::value;
    const int here = min(count - first, MOST / 2 * MT);
    mx_f4 acc[P][MT];
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) acc[p][mt] = mx_f4{0.f, 0.f, 0.f, 0.f};
    uint8_t* const mine = lds + wave * MINE;
    if constexpr (KIND == Down::kFew) {                                  // row 3 * i + n is part n of pair i
      auto row_at = [&](int row) __attribute__((always_inline)) {
        return list[first + row / 3] * h_pitch(I) + row % 3 * part;
      };
      expert_units<MX_BF16, Rows::kPartRows, MT, P, true>(h, 0, row_at, w, panel, 3 * here, I / kMxBlock, wave, WAVES,
                                                          lane, mine, acc);
    } else {
      auto row_at = [&](int i) __attribute__((always_inline)) { return list[first + i] * h_pitch(I); };
      expert_units<MX_BF16, Rows::kParts, MT, P, KIND == Down::kStaged>(h, part, row_at, w, panel, here, I / kMxBlock,
                                                                        wave, WAVES, lane, mine, acc);
    }
    share_sums<P, MT>(shared, acc, wave, lane);
    if constexpr (KIND == Down::kFew) {
      for (int t = threadIdx.x; t < 4 * P * here; t += WAVES * 64) {      // four columns of a pair
        const int i = t / (4 * P), p = t / 4 % P, g = t % 4;
        mx_f4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int row = 3 * i; row < 3 * i + 3; ++row)
          v += total<P, MT>(shared, p * MT + row / 16, WAVES, 16 * g + row % 16);
        const int n = (blockIdx.x * P + p) * kMxPanel + 4 * g;
        if (n < H) *reinterpret_cast<mx_f4*>(sums + (int64_t)list[first + i] * H + n) = v;
      }
    } else {
      for (int pm = wave; pm < P * MT; pm += WAVES) {
        const int i = pm % MT * 16 + (lane & 15);
        const int n = (blockIdx.x * P + pm / MT) * kMxPanel + 4 * (lane >> 4);
        const mx_f4 v = total<P, MT>(shared, pm, WAVES, lane);
        if (i < here && n < H) *reinterpret_cast<mx_f4*>(sums + (int64_t)list[first + i] * H + n) = v;
      }
    }
  };
  int first = 0;
  for (; count - first > MOST / 2; first += MOST) {
    pairs_from(std::integral_constant<int, 2>{}, first);
    __syncthreads();                              // the sums are read before they are overwritten
  }
  if (first < count) pairs_from(std::integral_constant<int, 1>{}, first);
}

// y[t] = the sum of token t's pairs, in order of choice; a thread takes four columns.
template <int DT>
__global__ __launch_bounds__(256) void mx_moe_sum_kernel(const float* __restrict__ sums, int k, uint32_t units,
                                                         int64_t count, uint16_t* __restrict__ y) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;            // of count = T * units
  if (i >= count) return;
  const int64_t t = i / units, c = i - t * units;
  const mx_f4* const from = reinterpret_cast<const mx_f4*>(sums) + t * k * units + c;
  mx_f4 v = from[0];
#pragma unroll 4
  for (int j = 1; j < k; ++j) v += from[j * (int64_t)units];
  reinterpret_cast<uint2*>(y)[i] = mx_pack4<DT>(v);
}

// ---------------------------------------------------------------- tokens by themselves
// One token, or few (by_token): its choices are the k slots, and nothing is shared
// between tokens.  The logits come from many workgroups (a single one reads the
// router at some 100 GB/s), each workgroup of the gate and up product then chooses
// by itself, and one workgroup adds all experts' shares of its columns of y.
constexpr int ONE_UP_WAVES = 4, ONE_DOWN_WAVES = 16;
template <int DT>
__global__ __launch_bounds__(256) void mx_one_logits_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                            const uint16_t* __restrict__ router, int H, int E,
                                                            float* __restrict__ logits) {
  const int lane = threadIdx.x & 63;
  const int e = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float s[1];
  router_logits<DT, 1>(reinterpret_cast<const uint4*>(x + blockIdx.y * ldx), router, H, E, e, lane, s);
  if (lane == 0 && e < E) logits[blockIdx.y * E + e] = s[0];
}

// A unit of a row, 512 values from 512 * q on: 16 bytes a lane (of each of h's
// three parts).  In h chunk lane % 16 of a K-tile belongs to block lane % 4
// (h_place), in x to block lane % 16 / 4.
template <int PARTS>
struct OneRow {
  uint4 v[PARTS];
};
template <int PARTS>
__device__ __forceinline__ OneRow<PARTS> one_row(const uint16_t* __restrict__ src, int64_t part, int64_t row, int q,
                                                 int blocks, int lane) {
  OneRow<PARTS> o;
#pragma unroll
  for (int n = 0; n < PARTS; ++n) o.v[n] = make_uint4(0u, 0u, 0u, 0u);
  if (4 * (4 * q + (lane >> 4)) + (PARTS > 1 ? lane & 3 : (lane >> 2) & 3) < blocks) {
    const uint16_t* const from = src + row + (int64_t)q * 4 * kMxTile + lane * 8;
#pragma unroll
    for (int n = 0; n < PARTS; ++n) o.v[n] = *reinterpret_cast<const uint4*>(from + n * part);
  }
  return o;
}

// P panels' products with one row (x), or the sum over slots of each slot's (h).
// A unit is a slot's quad of K-tiles, the waves take them in turn; the next
// unit's row and codes are loaded while the present one is multiplied, and the
// row goes by way of LDS of the wave's own (`mine`), so that all of a unit is one
// trip to memory (1 token, 64 experts, 8 chosen, H = 2048, I = 1024: operands read
// in place, tile by tile, the down product took 7.4 us instead of 4.5 with h in two
// parts, the up product 8.9 instead of 8.1).  Column n of the products is part n of h; the columns
// after the last part repeat it.  `v` is the first unit's row.  fp16 x: two bf16
// parts unless `exact`, i.e. all of the panels' weights are exact in fp16.
template <int DT, int PARTS, int P, int WAVES, typename RowAt, typename PanelAt>
__device__ __forceinline__ void one_units(const uint16_t* __restrict__ src, int64_t part, OneRow<PARTS> v,
                                          RowAt&& row_at, PanelAt&& panel_at, bool exact, int slots, const MxTiled& w,
                                          int blocks, int wave, int lane, uint4* mine, mx_f4 (&acc)[P][1]) {
  const int g = lane >> 4, column = min(lane & 15, PARTS - 1), units = slots * w.kq;
  uint4 c[P][4], next[P][4];
  uint32_t sc[P], sc_next[P];
  OneRow<PARTS> v_next = v;
  auto load = [&](int u, uint4 (&to)[P][4], uint32_t (&s)[P]) __attribute__((always_inline)) {
    const int q = u % w.kq;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int64_t panel = panel_at(u / w.kq, p);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        to[p][i] = *reinterpret_cast<const uint4*>(w.codes + ((panel * w.kt + min(4 * q + i, w.kt - 1)) * 64 + lane) * 16);
      s[p] = *reinterpret_cast<const uint32_t*>(w.scales + ((panel * w.kq + q) * 64 + lane) * 4);
    }
  };
  if (wave < units) load(wave, c, sc);
  for (int u = wave; u < units; u += WAVES) {
    const int q = u % w.kq, after = u + WAVES;
#pragma unroll
    for (int n = 0; n < PARTS; ++n) mine[64 * n + lane] = v.v[n];
    if (after < units) {
      v_next = one_row<PARTS>(src, part, row_at(after / w.kq), after % w.kq, blocks, lane);
      load(after, next, sc_next);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (4 * q + i >= w.kt) break;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = 16 * i + (PARTS > 1 ? 4 * j + g : 4 * g + j);
        uint4 a = mine[64 * column + at], b;
        auto tile = [&](auto ct, bool two) __attribute__((always_inline)) {
          constexpr int CT = decltype(ct)::value;
#pragma unroll
          for (int p = 0; p < P; ++p) {
            const uint4 d = mx_decode8<CT>(dword_of(c[p][i], j), mx_scale((sc[p] >> (8 * i)) & 0xffu));
            acc[p][0] = mx_mfma16<CT>(d, a, acc[p][0]);
            if (two) acc[p][0] = mx_mfma16<CT>(d, b, acc[p][0]);
          }
        };
        if (PARTS > 1 || DT == MX_BF16 || exact) tile(std::integral_constant<int, DT>{}, false);
        else {
          const uint4 both = a;
          mx_split8(both, a, b);
          tile(std::integral_constant<int, MX_BF16>{}, true);
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int p = 0; p < P; ++p) {
#pragma unroll
      for (int i = 0; i < 4; ++i) c[p][i] = next[p][i];
      sc[p] = sc_next[p];
    }
    v = v_next;
  }
}

// Workgroup: a panel of 16 rows of I, one choice of one token.
template <int DT>
__global__ __launch_bounds__(ONE_UP_WAVES * 64) void mx_one_up_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                                     MxTiled w, const float* __restrict__ logits, int E, int k,
                                                                     int renormalize, int blocks, int I,
                                                                     int32_t* __restrict__ ids,
                                                                     float* __restrict__ weights,
                                                                     uint16_t* __restrict__ h, int64_t part) {
  __shared__ mx_f4 sums[ONE_UP_WAVES * 2 * 64];
  __shared__ uint4 rows[ONE_UP_WAVES][64];
  __shared__ Choice choices[ONE_UP_WAVES];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = blockIdx.z;
  const OneRow<1> first = one_row<1>(x, 0, t * ldx, wave, blocks, lane);
  int id;
  float mine, sum;
  choose(logits + t * E, choices[wave], E, k, renormalize != 0, lane, id, mine, sum);
  const int slot = blockIdx.y, expert = __builtin_amdgcn_readlane(id, slot), half = I / kMxPanel;
  const int64_t panel = (int64_t)expert * (2 * half) + blockIdx.x;
  const bool exact = DT == MX_BF16 || (w.flags[panel] & w.flags[panel + half] & kMxFlagF16) != 0;
  mx_f4 acc[2][1] = {{mx_f4{0.f, 0.f, 0.f, 0.f}}, {mx_f4{0.f, 0.f, 0.f, 0.f}}};
  one_units<DT, 1, 2, ONE_UP_WAVES>(
      x, 0, first, [&](int) __attribute__((always_inline)) { return t * ldx; },
      [&](int, int p) __attribute__((always_inline)) { return panel + p * half; }, exact, 1, w, blocks, wave, lane,
      rows[wave], acc);
  share_sums<2, 1>(sums, acc, wave, lane);
  if (wave != 0) return;
  const float weight = mine / wave_sum(sum), share = __shfl(weight, slot);
  if (blockIdx.x == 0 && slot == 0 && lane < k) {
    ids[t * k + lane] = id;
    weights[t * k + lane] = weight;
  }
  if ((lane & 15) == 0) {
    const mx_f4 a = total<2, 1>(sums, 0, ONE_UP_WAVES, lane), b = total<2, 1>(sums, 1, ONE_UP_WAVES, lane);
    store_h(h, part, (t * k + slot) * h_pitch(I) + h_place(blockIdx.x * kMxPanel + 4 * (lane >> 4)), gated(a, b, share));
  }
}

// Workgroup: a panel of 16 columns of y, all choices of one token.
template <int DT>
__global__ __launch_bounds__(ONE_DOWN_WAVES * 64) void mx_one_down_kernel(const uint16_t* __restrict__ h,
                                                                         int64_t part, MxTiled w,
                                                                         const int32_t* __restrict__ ids, int k,
                                                                         int I, int H, uint16_t* __restrict__ y) {
  __shared__ mx_f4 sums[ONE_DOWN_WAVES * 64];
  __shared__ uint4 rows[ONE_DOWN_WAVES][3 * 64];
  const int lane = threadIdx.x & 63, blocks = I / kMxBlock;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = blockIdx.y;
  auto row_at = [&](int slot) __attribute__((always_inline)) { return (t * k + slot) * h_pitch(I); };
  const OneRow<3> first = wave < k * w.kq ? one_row<3>(h, part, row_at(wave / w.kq), wave % w.kq, blocks, lane)
                                          : OneRow<3>{};
  mx_f4 acc[1][1] = {{mx_f4{0.f, 0.f, 0.f, 0.f}}};
  one_units<MX_BF16, 3, 1, ONE_DOWN_WAVES>(
      h, part, first, row_at,
      [&](int slot, int) __attribute__((always_inline)) { return (int64_t)ids[t * k + slot] * (H / kMxPanel) + blockIdx.x; },
      true, k, w, blocks, wave, lane, rows[wave], acc);
  share_sums<1, 1>(sums, acc, wave, lane);
  if (wave != 0) return;
  const mx_f4 mine = total<1, 1>(sums, 0, ONE_DOWN_WAVES, lane);        // of part lane % 16
  mx_f4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = mine[i] + __shfl_down(mine[i], 1) + __shfl_down(mine[i], 2);
  if ((lane & 15) == 0)
    *reinterpret_cast<uint2*>(y + t * H + blockIdx.x * kMxPanel + 4 * (lane >> 4)) = mx_pack4<DT>(v);
}

// ---------------------------------------------------------------- launches
// Each token by itself, in three launches, or the experts' pairs together, in
// four.  By itself every pair reads its expert's weights, which pays while most
// pairs have experts of their own (T * k <= 3/4 E), or while all that reading is
// small and the workgroups are few.  us of the layer together and by token (T, H,
// I, E, k): 2 x 2048 x 1024, 64, 8 26.3 and 18.1; 6: 50.6 and 41.0; 12: 63.8 and
// 66.8; 16 x 4096 x 1024, 256, 8 207 and 177; 3 x 4096 x 4096, 16, 4 75.1 and 69.2,
// 4: 83.9 and 84.2; 6 x 1056 x 736, 12, 3 18.1 and 16.2, 8: 18.6 and 19.7; 24 x 512 x
// 256, 4, 1 14.0 and 12.8, 32: 14.2 and 14.1; 24 x 1024 x 256, 64, 1 17.6 and 18.5.
static bool by_token(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k) {
  if (T == 1) return true;
  return (T <= 16 && 4 * T * k <= 3 * E) || (T * H <= 12288 && T * k * H * I <= (int64_t)14 << 20);
}

static int64_t h_part(int64_t T, int64_t I, int64_t k) { return T * k * h_pitch(I); }

// h in three parts, then the pairs' shares of y or the tokens' logits (by_token).
size_t mx_moe_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t k) {
  return (size_t)h_part(T, I, k) * 6 + (size_t)(T * std::max<int64_t>(kMoeMaxE, k * H) * 4);
}

template <int DT>
static hipError_t moe_dt(const void* x, int64_t ldx, int64_t T, int64_t H, int64_t I, int64_t E, int64_t k, int renorm,
                         const void* router, const MxTiled& gate_up, const MxTiled& down, void* y, int32_t* ids,
                         float* weights, uint8_t* ws, hipStream_t stream) {
  const int hidden = (int)H, i = (int)I, e = (int)E, kk = (int)k, pairs = (int)(T * k), x_blocks = hidden / kMxBlock;
  const int64_t part = h_part(T, I, k);
  auto* xp = static_cast<const uint16_t*>(x);
  auto* rp = static_cast<const uint16_t*>(router);
  auto* yp = static_cast<uint16_t*>(y);
  auto* h = reinterpret_cast<uint16_t*>(ws);
  auto* sums = reinterpret_cast<float*>(h + 3 * part);
  auto* ch = static_cast<const uint16_t*>(h);
  auto* cids = static_cast<const int32_t*>(ids);
  auto* cweights = static_cast<const float*>(weights);
  auto* csums = static_cast<const float*>(sums);
  const unsigned rows = (unsigned)(I / kMxPanel), panels = (unsigned)(H / kMxPanel);
  hipError_t err;
  if (by_token(T, H, I, E, k)) {
    const unsigned t = (unsigned)T;
    err = mx_launch(mx_one_logits_kernel<DT>, dim3((unsigned)((E + 3) / 4), t), dim3(256), stream, xp, ldx, rp, hidden,
                    e, sums);
    if (err != hipSuccess) return err;
    err = mx_launch(mx_one_up_kernel<DT>, dim3(rows, (unsigned)k, t), dim3(ONE_UP_WAVES * 64), stream, xp, ldx, gate_up,
                    csums, e, kk, renorm, x_blocks, i, ids, weights, h, part);
    if (err != hipSuccess) return err;
    return mx_launch(mx_one_down_kernel<DT>, dim3(panels, t), dim3(ONE_DOWN_WAVES * 64), stream, ch, part, down, cids,
                     kk, i, hidden, yp);
  }
  err = mx_launch(mx_route_kernel<DT>, dim3((unsigned)T), dim3(ROUTE_WAVES * 64), stream, xp, ldx, rp, hidden, e, kk,
                  renorm, ids, weights);
  if (err != hipSuccess) return err;
  const unsigned slots = (unsigned)std::min<int64_t>(E, pairs);
  auto up = [&](auto* kernel, unsigned q) {
    return mx_launch(kernel, dim3((rows + q - 1) / q, slots), dim3(UP_WAVES * 64), stream, xp, ldx, gate_up, cids,
                     cweights, pairs, e, kk, x_blocks, i, h, part);
  };
  // Two pairs of panels share staged rows where each wave has a unit of four K-tiles
  // (H >= 2048), or where many rows make up for fewer; else direct rows, a pair.  us
  // of the layer, direct and staged: 16 x 4096 x 11008, 8 experts, 2 chosen 131.9 and
  // 126.2; 48 x 2048 x 1024, 16, 8: 47.0 and 40.4; 64 x 2048 x 1024, 64, 8: 93.9 and
  // 92.0; 64 x 1024 x 4096, 4, 2: 46.2 and 43.2; but 64 x 1056 x 736, 12, 3: 24.3 and
  // 24.9; 33 x 1056 x 736, 12, 3: 20.5 and 21.4; 64 x 256 x 256, 4, 2: 19.6 and 22.0.
  const bool staged_x = H >= 2048 || (H >= 512 && T * k >= 24 * E);
  err = staged_x ? up(mx_moe_up_kernel<DT, 2, true>, 2) : up(mx_moe_up_kernel<DT, 1, false>, 1);
  if (err != hipSuccess) return err;
  auto go = [&](auto* kernel, Down kind) {
    return mx_launch(kernel, dim3((panels + DOWN_PANELS - 1) / DOWN_PANELS, slots), dim3(down_waves(kind) * 64), stream, ch,
                     part, down, cids, pairs, e, i, hidden, sums);
  };
  // Four panels share the loads of h.  Staged rows pay where the waves have work
  // each, or where the workgroups make one round at most; parts as rows up to five
  // pairs an expert.  us of the product, direct, staged and few: 16 x 4096 x 11008,
  // 8 experts, 2 chosen 52, 52 and 41.5; 40 x 4096 x 4096, 8, 1: 23.1, 22.1 and 20.5;
  // 33 x 1056 x 736, 12, 3: 6.6, 5.8 and 9.7; 64 x 4096 x 4096, 4, 2: 38, 27.5 and 37;
  // 64 x 2048 x 1024, 64, 8: 36, 49 and 58.
  const bool staged_h = I >= 2048 || (panels + DOWN_PANELS - 1) / DOWN_PANELS * slots <= 256;
  err = !staged_h ? go(mx_moe_down_kernel<Down::kDirect>, Down::kDirect)
        : T * k <= 5 * E ? go(mx_moe_down_kernel<Down::kFew>, Down::kFew)
                         : go(mx_moe_down_kernel<Down::kStaged>, Down::kStaged);
  if (err != hipSuccess) return err;
  const uint32_t units = (uint32_t)(H / 4);
  const int64_t n = T * units;
  return mx_launch(mx_moe_sum_kernel<DT>, dim3((unsigned)((n + 255) / 256)), dim3(256), stream, csums, kk, units, n, yp);
}

hipError_t launch_mx_moe(const void* x, int dtype, int64_t ldx, int64_t T, int64_t H, int64_t I, int64_t E, int64_t k,
                         bool renormalize, const void* router, const MxTiled& gate_up, const MxTiled& down, void* y,
                         int32_t* ids, float* weights, uint8_t* ws, hipStream_t stream) {
  auto* run = dtype == MX_F16 ? moe_dt<MX_F16> : moe_dt<MX_BF16>;
  return run(x, ldx, T, H, I, E, k, renormalize ? 1 : 0, router, gate_up, down, y, ids, weights, ws, stream);
}

}  // namespace wqbmm
