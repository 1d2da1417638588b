// mx_moe.hip -- a mixture-of-experts layer with MXFP4 experts for up to 64
// tokens, in three launches:
//   route: logits = router . x, softmax, the k largest per token;
//   up:    h = weight * silu(gate_e . x) * (up_e . x) for every (token, choice)
//          pair, per reached expert and panel of 16 rows of I;
//   down:  y = sum over a token's pairs of down_e . h, per panel of 16 columns
//          of y, over all reached experts.
// Each reached expert's weights are read once, by the workgroups of its panels;
// every sum has a fixed order.  There is no hand-off between workgroups inside
// a launch: each workgroup of `up` and `down` finds its expert's pairs itself
// from the ids (at most 1024 of them).
#include <algorithm>

#include "mx_device.hpp"
#include "mx_launch.hpp"

namespace wqbmm {

namespace {

__device__ __forceinline__ uint32_t dword_of(const uint4& v, int j) {
  return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
}

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

// One workgroup per token.  A wave takes experts in turn, lanes along H; wave 0
// then picks the k largest (key, lowest index first) and forms the weights.
template <int DT>
__global__ __launch_bounds__(ROUTE_WAVES * 64) void mx_route_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                                    const uint16_t* __restrict__ router, int H,
                                                                    int E, int k, int renormalize,
                                                                    int32_t* __restrict__ ids,
                                                                    float* __restrict__ weights) {
  __shared__ float logits[kMoeMaxE];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = blockIdx.x;
  const uint4* xr = reinterpret_cast<const uint4*>(x + t * ldx);
  for (int e = wave; e < E; e += ROUTE_WAVES) {
    const uint4* rr = reinterpret_cast<const uint4*>(router + (int64_t)e * H);
    float s = 0.0f;
    for (int c = lane; c < H / 8; c += 64) {
      const uint4 a = xr[c], b = rr[c];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s = __builtin_fmaf(mx_lo<DT>(dword_of(a, j)), mx_lo<DT>(dword_of(b, j)), s);
        s = __builtin_fmaf(mx_hi<DT>(dword_of(a, j)), mx_hi<DT>(dword_of(b, j)), s);
      }
    }
    s = wave_sum(s);
    if (lane == 0) logits[e] = s;
  }
  __syncthreads();
  if (wave != 0) return;
  constexpr int PER = kMoeMaxE / 64;
  float v[PER];
  uint64_t key[PER];
  float top = 0.0f;
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    v[i] = e < E ? logits[e] : 0.0f;
    // larger logit first, then the lower index; 0 is below every candidate
    key[i] = e < E ? ((uint64_t)order_key(v[i]) << 32) | (uint32_t)(0xffffffffu - e) : 0;
  }
  float total = 0.0f, mine = 0.0f;      // sum of the chosen; lane j holds the j-th choice
  int my_id = 0;
  for (int j = 0; j < k; ++j) {
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) best = best > key[i] ? best : key[i];
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
      const uint64_t o = __shfl_xor((unsigned long long)best, d);
      best = best > o ? best : o;
    }
    const int e = (int)(0xffffffffu - (uint32_t)best);
    const float l = logits[e];
    if (j == 0) top = l;
    const float p = expf(l - top);
    total += p;
    if (lane == j) {
      mine = p;
      my_id = e;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (key[i] == best) key[i] = 0;
  }
  if (!renormalize) {                   // over all experts instead
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane + 64 * i < E) s += expf(v[i] - top);
    total = wave_sum(s);
  }
  if (lane < k) {
    ids[t * k + lane] = my_id;
    weights[t * k + lane] = mine / total;
  }
}

// ---------------------------------------------------------------- up
// The pairs (token * k + choice) of the slot-th reached expert, in ascending
// order; returns the expert, or -1 if fewer are reached.  Every thread of the
// workgroup calls it.  mask: 8 words, counts: one per wave, list: up to 64.
template <int WAVES>
__device__ __forceinline__ int pairs_of_slot(const int32_t* __restrict__ ids, int pairs, int slot, uint32_t* mask,
                                             int* counts, uint16_t* list, int& count) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int PER = kMoeMaxT * kMoeMaxK / (WAVES * 64) > 0 ? kMoeMaxT * kMoeMaxK / (WAVES * 64) : 1;
  if (tid < kMoeMaxE / 32) mask[tid] = 0;
  __syncthreads();
  int id[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int p = i * WAVES * 64 + tid;
    id[i] = p < pairs ? ids[p] : -1;
    if (id[i] >= 0) atomicOr(&mask[id[i] >> 5], 1u << (id[i] & 31));
  }
  __syncthreads();
  int expert = -1, left = slot;
  for (int w = 0; w < kMoeMaxE / 32; ++w) {
    uint32_t m = mask[w];
    const int n = __popc(m);
    if (left < n) {
      for (; left > 0; --left) m &= m - 1;
      expert = 32 * w + __ffs(m) - 1;
      break;
    }
    left -= n;
  }
  if (expert < 0) return -1;
  int base = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const bool hit = id[i] == expert;
    const uint64_t votes = __ballot(hit);
    if (lane == 0) counts[wave] = __popcll(votes);
    __syncthreads();
    int before = base;
    for (int w = 0; w < WAVES; ++w) {
      if (w < wave) before += counts[w];
      base += counts[w];
    }
    if (hit) list[before + __popcll(votes & ((1ull << lane) - 1))] = (uint16_t)(i * WAVES * 64 + tid);
    __syncthreads();
  }
  count = base;
  return expert;
}

constexpr int UP_WAVES = 4;

// 16 significant bits of h: two bf16 parts, whose products with the weights
// are exact, and which keep fp32's range (h in fp16 would overflow early, in
// bf16 alone it would cost as much as the output's own rounding).
__device__ __forceinline__ void store_h(uint16_t* __restrict__ hi, uint16_t* __restrict__ lo, int64_t at, mx_f4 v) {
  uint32_t h[2], l[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const mx_bf2 b = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
    h[i] = __builtin_bit_cast(uint32_t, b);
    const float h0 = mx_lo<MX_BF16>(h[i]), h1 = mx_hi<MX_BF16>(h[i]);
    const mx_bf2 r = {(__bf16)(__builtin_isfinite(h0) ? v[2 * i] - h0 : 0.0f),
                      (__bf16)(__builtin_isfinite(h1) ? v[2 * i + 1] - h1 : 0.0f)};
    l[i] = __builtin_bit_cast(uint32_t, r);
  }
  *reinterpret_cast<uint2*>(hi + at) = make_uint2(h[0], h[1]);
  *reinterpret_cast<uint2*>(lo + at) = make_uint2(l[0], l[1]);
}

template <int DT, bool SPLIT, int MT>
__device__ __forceinline__ void up_quads(const uint16_t* __restrict__ x, int64_t ldx, const MxTiled& w,
                                         int64_t gate_panel, int64_t up_panel, const uint16_t* list, int count, int k,
                                         int blocks, int wave, int lane, mx_f4 (&acc)[2][MT]) {
  const int r = lane & 15, g = lane >> 4;
  const int64_t panel[2] = {gate_panel, up_panel};
  int64_t row[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
    row[mt] = mt * 16 + r < count ? (int64_t)(list[mt * 16 + r] / k) * ldx : -1;
  for (int q = wave; q < w.kq; q += UP_WAVES) {
    uint4 c[2][4];
    uint32_t sc[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c[p][i] = *reinterpret_cast<const uint4*>(
            w.codes + ((panel[p] * w.kt + min(4 * q + i, w.kt - 1)) * 64 + lane) * 16);
      sc[p] = *reinterpret_cast<const uint32_t*>(w.scales + ((panel[p] * w.kq + q) * 64 + lane) * 4);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (4 * q + i >= w.kt) break;
      const int b = 4 * (4 * q + i) + g;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if (mt * 16 >= count) break;
        uint4 xv[4] = {};
        if (row[mt] >= 0 && b < blocks) {
          const uint4* src = reinterpret_cast<const uint4*>(x + row[mt] + (int64_t)b * kMxBlock);
#pragma unroll
          for (int j = 0; j < 4; ++j) xv[j] = src[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint4 hi, lo;
          if constexpr (SPLIT) mx_split8(xv[j], hi, lo);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const float f = mx_scale((sc[p] >> (8 * i)) & 0xffu);
            if constexpr (SPLIT) {
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

// Workgroup (panel of 16 rows of I, slot): the gate panel and the up panel of
// the slot's expert for all of its pairs; the waves split H.
template <int DT, int MT>
__global__ __launch_bounds__(UP_WAVES * 64) void mx_moe_up_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                                 MxTiled w, const int32_t* __restrict__ ids,
                                                                 const float* __restrict__ weights, int pairs, int k,
                                                                 int blocks, int I, uint16_t* __restrict__ h_hi,
                                                                 uint16_t* __restrict__ h_lo) {
  __shared__ uint32_t mask[kMoeMaxE / 32];
  __shared__ int counts[UP_WAVES];
  __shared__ uint16_t list[kMoeMaxT];
  __shared__ mx_f4 part[UP_WAVES][2 * MT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int count = 0;
  const int expert = __builtin_amdgcn_readfirstlane(
      pairs_of_slot<UP_WAVES>(ids, pairs, blockIdx.y, mask, counts, list, count));
  if (expert < 0) return;
  count = __builtin_amdgcn_readfirstlane(count);
  const int64_t gate = (int64_t)expert * (2 * I / kMxPanel) + blockIdx.x, up = gate + I / kMxPanel;
  mx_f4 acc[2][MT];
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[p][mt] = mx_f4{0.f, 0.f, 0.f, 0.f};
  if constexpr (DT == MX_BF16) {
    up_quads<DT, false, MT>(x, ldx, w, gate, up, list, count, k, blocks, wave, lane, acc);
  } else {
    if (w.flags[gate] & w.flags[up] & kMxFlagF16)
      up_quads<DT, false, MT>(x, ldx, w, gate, up, list, count, k, blocks, wave, lane, acc);
    else
      up_quads<DT, true, MT>(x, ldx, w, gate, up, list, count, k, blocks, wave, lane, acc);
  }
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) part[wave][p * MT + mt][lane] = acc[p][mt];
  __syncthreads();
  for (int mt = wave; mt < MT; mt += UP_WAVES) {
    const int i = mt * 16 + (lane & 15);
    if (i >= count) continue;
    mx_f4 a = part[0][mt][lane], b = part[0][MT + mt][lane];
#pragma unroll
    for (int s = 1; s < UP_WAVES; ++s) {
      a += part[s][mt][lane];
      b += part[s][MT + mt][lane];
    }
    const int pair = list[i];
    const float share = weights[pair];
    mx_f4 h;
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = a[j] / (1.0f + expf(-a[j])) * b[j] * share;
    store_h(h_hi, h_lo, (int64_t)pair * I + blockIdx.x * kMxPanel + 4 * (lane >> 4), h);
  }
}

// ---------------------------------------------------------------- down
constexpr int DOWN_WAVES = 8;

// Workgroup: one panel of 16 columns of y, all reached experts.  Pairs are
// sorted by expert in LDS; a wave takes (expert, K range) items in turn and adds
// each item's products to its own sums per token, which are added over the
// waves at the end.
template <int DT, int MT>
__global__ __launch_bounds__(DOWN_WAVES * 64) void mx_moe_down_kernel(const uint16_t* __restrict__ h_hi,
                                                                     const uint16_t* __restrict__ h_lo, MxTiled w,
                                                                     const int32_t* __restrict__ ids, int T, int k,
                                                                     int I, int H, uint16_t* __restrict__ y) {
  constexpr int TOKENS = MT * 16;
  __shared__ int start[kMoeMaxE + 1];             // first sorted pair of each expert
  __shared__ int fill[kMoeMaxE];
  __shared__ uint16_t sorted[kMoeMaxT * kMoeMaxK];
  __shared__ uint16_t reached[kMoeMaxE];          // the reached experts, ascending
  __shared__ int n_reached;
  __shared__ mx_f4 sums[DOWN_WAVES][TOKENS][4];   // [wave][token][16 columns]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int pairs = T * k;
  constexpr int THREADS = DOWN_WAVES * 64;
  constexpr int PER = kMoeMaxT * kMoeMaxK / THREADS;
  if (tid < kMoeMaxE) fill[tid] = 0;
  for (int i = tid; i < DOWN_WAVES * TOKENS * 4; i += THREADS) (&sums[0][0][0])[i] = mx_f4{0.f, 0.f, 0.f, 0.f};
  __syncthreads();
  int id[PER], rank[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int p = i * THREADS + tid;
    id[i] = p < pairs ? ids[p] : -1;
    if (id[i] >= 0) rank[i] = atomicAdd(&fill[id[i]], 1);
  }
  __syncthreads();
  if (wave == 0) {                                // prefix sums of counts and of "reached"
    int base = 0, seen = 0;
    for (int i = 0; i < kMoeMaxE / 64; ++i) {
      const int c = fill[64 * i + lane];
      int s = c;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(s, d);
        if (lane >= d) s += o;
      }
      start[64 * i + lane] = base + s - c;
      const uint64_t votes = __ballot(c > 0);
      if (c > 0) reached[seen + __popcll(votes & ((1ull << lane) - 1))] = (uint16_t)(64 * i + lane);
      seen += __popcll(votes);
      base += __shfl(s, 63);
    }
    if (lane == 0) {
      start[kMoeMaxE] = base;
      n_reached = seen;
    }
  }
  __syncthreads();
  // The order of an expert's pairs only places them in columns of the product;
  // each sum's order does not depend on it.
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (id[i] >= 0) sorted[start[id[i]] + rank[i]] = (uint16_t)(i * THREADS + tid);
  __syncthreads();

  const int slots = __builtin_amdgcn_readfirstlane(n_reached);
  const int parts = min(w.kq, max(1, (DOWN_WAVES + slots - 1) / slots));   // K ranges per expert
  const int per = (w.kq + parts - 1) / parts;
  const int r = lane & 15, g = lane >> 4, blocks = I / kMxBlock;
  for (int item = wave; item < slots * parts; item += DOWN_WAVES) {
    const int e = __builtin_amdgcn_readfirstlane(reached[item / parts]);
    const int q_lo = item % parts * per, q_hi = min(w.kq, q_lo + per);
    const int first = __builtin_amdgcn_readfirstlane(start[e]);
    const int count = __builtin_amdgcn_readfirstlane(start[e + 1]) - first;
    const int64_t panel = (int64_t)e * (H / kMxPanel) + blockIdx.x;
    int pair[MT];
    mx_f4 acc[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      pair[mt] = mt * 16 + r < count ? sorted[first + mt * 16 + r] : -1;
      acc[mt] = mx_f4{0.f, 0.f, 0.f, 0.f};
    }
    for (int q = q_lo; q < q_hi; ++q) {
      uint4 c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c[i] = *reinterpret_cast<const uint4*>(
            w.codes + ((panel * w.kt + min(4 * q + i, w.kt - 1)) * 64 + lane) * 16);
      const uint32_t sc = *reinterpret_cast<const uint32_t*>(w.scales + ((panel * w.kq + q) * 64 + lane) * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (4 * q + i >= w.kt) break;
        const int b = 4 * (4 * q + i) + g;
        const float f = mx_scale((sc >> (8 * i)) & 0xffu);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          if (mt * 16 >= count) break;
          uint4 hi[4] = {}, lo[4] = {};
          if (pair[mt] >= 0 && b < blocks) {
            const int64_t at = (int64_t)pair[mt] * I + (int64_t)b * kMxBlock;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              hi[j] = reinterpret_cast<const uint4*>(h_hi + at)[j];
              lo[j] = reinterpret_cast<const uint4*>(h_lo + at)[j];
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 a = mx_decode8<MX_BF16>(dword_of(c[i], j), f);
            acc[mt] = mx_mfma16<MX_BF16>(a, hi[j], acc[mt]);
            acc[mt] = mx_mfma16<MX_BF16>(a, lo[j], acc[mt]);
          }
        }
      }
    }
    // an expert's pairs belong to different tokens: no two lanes meet here; a
    // token's earlier items may have been other lanes' (one wave, LDS in order)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
      if (pair[mt] >= 0) sums[wave][pair[mt] / k][g] += acc[mt];
  }
  __syncthreads();
  for (int i = tid; i < T * 4; i += THREADS) {
    const int t = i >> 2, j = i & 3;
    mx_f4 v = sums[0][t][j];
#pragma unroll
    for (int s = 1; s < DOWN_WAVES; ++s) v += sums[s][t][j];
    const uint32_t lo = mx_round16<DT>(v[0]) | ((uint32_t)mx_round16<DT>(v[1]) << 16);
    const uint32_t hi = mx_round16<DT>(v[2]) | ((uint32_t)mx_round16<DT>(v[3]) << 16);
    *reinterpret_cast<uint2*>(y + (int64_t)t * H + blockIdx.x * kMxPanel + 4 * j) = make_uint2(lo, hi);
  }
}

// ---------------------------------------------------------------- launches
static size_t h_bytes(int64_t T, int64_t I, int64_t k) { return (size_t)(T * k * I * 2 + 255) / 256 * 256; }

size_t mx_moe_workspace_bytes(int64_t T, int64_t I, int64_t k) { return 2 * h_bytes(T, I, k); }

template <int DT, int MT>
static hipError_t moe_mt(const uint16_t* x, int64_t ldx, int64_t T, int64_t H, int64_t I, int64_t E, int64_t k,
                         int renorm, const uint16_t* router, const MxTiled& gate_up, const MxTiled& down, uint16_t* y,
                         int32_t* ids, float* weights, uint8_t* ws, hipStream_t stream) {
  const int h = (int)H, i = (int)I, e = (int)E, kk = (int)k, t = (int)T, pairs = t * kk;
  const int h_blocks = h / kMxBlock;
  auto* hi = reinterpret_cast<uint16_t*>(ws);
  auto* lo = reinterpret_cast<uint16_t*>(ws + h_bytes(T, I, k));
  auto* cids = static_cast<const int32_t*>(ids);
  auto* cweights = static_cast<const float*>(weights);
  auto* chi = static_cast<const uint16_t*>(hi);
  auto* clo = static_cast<const uint16_t*>(lo);
  hipError_t err = mx_launch(mx_route_kernel<DT>, dim3((unsigned)T), dim3(ROUTE_WAVES * 64), stream, x, ldx, router, h,
                             e, kk, renorm, ids, weights);
  if (err != hipSuccess) return err;
  const dim3 up_grid((unsigned)(I / kMxPanel), (unsigned)std::min<int64_t>(E, pairs));
  err = mx_launch(mx_moe_up_kernel<DT, MT>, up_grid, dim3(UP_WAVES * 64), stream, x, ldx, gate_up, cids, cweights,
                  pairs, kk, h_blocks, i, hi, lo);
  if (err != hipSuccess) return err;
  return mx_launch(mx_moe_down_kernel<DT, MT>, dim3((unsigned)(H / kMxPanel)), dim3(DOWN_WAVES * 64), stream, chi, clo,
                   down, cids, t, kk, i, h, y);
}

template <int DT>
static hipError_t moe_dt(const void* x, int64_t ldx, int64_t T, int64_t H, int64_t I, int64_t E, int64_t k, int renorm,
                         const void* router, const MxTiled& gate_up, const MxTiled& down, void* y, int32_t* ids,
                         float* weights, uint8_t* ws, hipStream_t stream) {
  auto* xp = static_cast<const uint16_t*>(x);
  auto* rp = static_cast<const uint16_t*>(router);
  auto* yp = static_cast<uint16_t*>(y);
  auto* run = T <= 16 ? moe_mt<DT, 1> : T <= 32 ? moe_mt<DT, 2> : moe_mt<DT, 4>;
  return run(xp, ldx, T, H, I, E, k, renorm, rp, gate_up, down, yp, ids, weights, ws, stream);
}

hipError_t launch_mx_moe(const void* x, int dtype, int64_t ldx, int64_t T, int64_t H, int64_t I, int64_t E, int64_t k,
                         bool renormalize, const void* router, const MxTiled& gate_up, const MxTiled& down, void* y,
                         int32_t* ids, float* weights, uint8_t* ws, hipStream_t stream) {
  auto* run = dtype == MX_F16 ? moe_dt<MX_F16> : moe_dt<MX_BF16>;
  return run(x, ldx, T, H, I, E, k, renormalize ? 1 : 0, router, gate_up, down, y, ids, weights, ws, stream);
}

}  // namespace wqbmm
