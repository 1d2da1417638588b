// grp_lora.hip -- low-rank adapters of many requests beside a shared projection:
// y[m] = base[m] + scale_l * B_l . (A_l . x[m]), rows ordered by adapter.
//
// Two launches: v = A . x (x and the reached adapters read once; K is split over
// the waves of a workgroup, and over workgroups where there are few tiles of
// rows), fp32 partial sums in the workspace; then B . v, a tile of rows and
// columns a workgroup, added to base in registers.  v keeps fp32's sums; for the
// 16-bit products with B it is taken apart: bf16, three parts of eight bits (exact down
// to 2^-110); fp16, two parts of eleven after a row's values are scaled by a power of two
// to below 2^14.  These hold 22 bits of a value, or 2^-38 of its row's largest where that is
// more: part 1 ends at fp16's 2^-24, half of which is 2^-38 of the largest, 2^13 at least.
// (bf16 parts would need B taken apart as well; a third fp16 part would take half as much
// LDS again for v and leave two workgroups a CU at ranks 72 to 128, not three.)
//
// 48 rows, 16 adapters, rank 16, 4096 x 4096: 3.8 and 4.9 us, two launches of three trips to
// memory each.  2048 rows, 5 adapters, rank 64, 4096 -> 11008: 11 us (x and A, 26 MB) and 28
// (base and y, 90 MB, 3.2 TB/s, beside 120 MB of v and B from L2).
#include <algorithm>

#include "grp_device.hpp"
#include "grp_launch.hpp"
#include "mx_tile.hpp"

namespace wqbmm {

namespace {

constexpr int LORA_WAVES = 4;

// Eight values of a row of `n` 16-bit values from `i` on, or zeros past it.
__device__ __forceinline__ uint4 load8(const uint16_t* __restrict__ row, int i, int n) {
  return i < n ? *reinterpret_cast<const uint4*>(row + i) : make_uint4(0u, 0u, 0u, 0u);
}

}  // namespace

// ---------------------------------------------------------------- v = A . x
// part [split][place][pitch]; columns from r on are not used.  A workgroup takes MT * 16
// rows and RT * 16 of A's, at most 64, of which there are `rblocks`.  (Rank 256 as one block
// of 16 rows of x, 4096 rows, 4096 -> 4096: 200 us, 140 so.)
template <int DT, int RT, int MT>
__global__ __launch_bounds__(LORA_WAVES * 64) void lora_down_kernel(Lora p, int splits, int kt_per, int rblocks, int pitch,
                                                                   float* __restrict__ part) {
  __shared__ __attribute__((aligned(16))) mx_f4 sums[LORA_WAVES][RT * MT][64];
  const int lane = threadIdx.x & 63, i16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = blockIdx.x % splits, j0 = blockIdx.x / splits % rblocks * (RT * 16);
  const GroupTile t = group_tile(p.offsets, p.L, p.M, MT * 16, blockIdx.x / splits / rblocks, false);
  if (t.group < 0) return;
  const uint16_t* xr[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = p.rows[t.first + min(m * 16 + i16, t.rows - 1)];
    xr[m] = p.x + (row >= 0 && row < p.M ? row : 0) * p.ldx;
  }
  const uint16_t* ar[RT];
#pragma unroll
  for (int c = 0; c < RT; ++c) ar[c] = p.a + ((int64_t)t.group * p.r + min(j0 + c * 16 + i16, p.r - 1)) * p.K;
  mx_f4 acc[RT][MT];
#pragma unroll
  for (int c = 0; c < RT; ++c)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[c][m] = mx_f4{0.f, 0.f, 0.f, 0.f};
  const int kts = (p.K + 127) / 128, hi = min(kts, (split + 1) * kt_per);
  for (int kt = split * kt_per + wave; kt < hi; kt += LORA_WAVES) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = kt * 128 + i * 32 + g * 8;
      uint4 xv[MT], av[RT];
#pragma unroll
      for (int m = 0; m < MT; ++m) xv[m] = load8(xr[m], k, p.K);
#pragma unroll
      for (int c = 0; c < RT; ++c) av[c] = load8(ar[c], k, p.K);
#pragma unroll
      for (int c = 0; c < RT; ++c)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[c][m] = mx_mfma16<DT>(av[c], xv[m], acc[c][m]);
    }
  }
#pragma unroll
  for (int c = 0; c < RT; ++c)
#pragma unroll
    for (int m = 0; m < MT; ++m) sums[wave][c * MT + m][lane] = acc[c][m];
  __syncthreads();
  for (int cm = wave; cm < RT * MT; cm += LORA_WAVES) {
    mx_f4 v = sums[0][cm][lane];
#pragma unroll
    for (int w = 1; w < LORA_WAVES; ++w) v += sums[w][cm][lane];
    const int row = cm % MT * 16 + i16, j = j0 + cm / MT * 16 + 4 * g;
    if (row < t.rows && j < p.r)
      *reinterpret_cast<mx_f4*>(part + ((int64_t)split * p.M + t.first + row) * pitch + j) = v;
  }
}

// ---------------------------------------------------------------- y = base + B . v
// RC chunks of 32 columns of v.  A workgroup takes v's operands of MT * 16 rows to
// LDS once and then `nblocks` blocks of 64 columns a wave.  A wave's products leave a
// lane with four columns of a row, 32 bytes of it a store; by way of LDS of the wave's
// own it loads base, ahead of the products, and stores y in 16 bytes a lane, 128 of a
// row (2048 rows, rank 64, 11008 columns: 48 us without, 29 with).  The stores go past
// the caches, which base and B need (29 -> 26 us; 28 with what B's infinities take).
template <int DT>
__device__ __forceinline__ void lora_operands(mx_f4 (&v)[2], int units, uint4 (&part)[3], int& e) {
  if constexpr (DT == MX_BF16) {
    uint2 lo[3], hi[3];
    mx_split24(v[0], lo);
    mx_split24(v[1], hi);
#pragma unroll
    for (int n = 0; n < 3; ++n) part[n] = make_uint4(lo[n].x, lo[n].y, hi[n].x, hi[n].y);
    e = 0;
  } else {
    float top = 0.0f;                             // of the row: `units` lanes
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = fabsf(v[i / 4][i % 4]);
      top = fmaxf(top, __builtin_isfinite(a) ? a : 0.0f);     // what is not finite stays so at any scale
    }
    for (int d = units / 2; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    e = top == 0.0f ? 0 : 14 - __builtin_amdgcn_frexp_expf(top);     // below 2^14
    uint32_t h[4], l[4];
    // part 0 is 0 for 0 alone: it rounds f and 2^-24 of its sign, which part 1 takes off again (B's infinities)
    auto first = [](float f) __attribute__((always_inline)) {
      return mx_round16<MX_F16>(f + fmaxf(fminf(f * 0x1p127f, 0x1p-24f), -0x1p-24f));
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = __builtin_ldexpf(v[i / 2][i % 2 * 2], e), b = __builtin_ldexpf(v[i / 2][i % 2 * 2 + 1], e);
      h[i] = first(a) | (uint32_t)first(b) << 16;
      const float ra = a - mx_lo<MX_F16>(h[i]), rb = b - mx_hi<MX_F16>(h[i]);
      l[i] = mx_round16<MX_F16>(__builtin_isfinite(a) ? ra : 0.0f) |
             (uint32_t)mx_round16<MX_F16>(__builtin_isfinite(b) ? rb : 0.0f) << 16;
    }
    part[0] = make_uint4(h[0], h[1], h[2], h[3]);
    part[1] = make_uint4(l[0], l[1], l[2], l[3]);
  }
}

// B for v's later parts where it holds infinities: the largest finite values instead.  Part 0
// makes the result infinite; a later one may be 0 or of the other sign, and 0 * inf or
// inf - inf is NaN.  That only happens to results that come out NaN without this, so that the
// products are made again where one does (this in every product: 37 -> 46 us for 2048 rows, rank
// 128, 4096 x 4096, fp16).  Positive values order as 16-bit integers do, negative ones as
// unsigned ones.
template <int DT>
__device__ __forceinline__ uint4 lora_finite(uint4 b) {
  constexpr int16_t MOST = DT == MX_BF16 ? 0x7f7f : 0x7bff;
  typedef int16_t i16x2 __attribute__((ext_vector_type(2)));
  auto two = [](uint32_t w) __attribute__((always_inline)) {
    const mx_u16x2 negative = {(uint16_t)(MOST | 0x8000), (uint16_t)(MOST | 0x8000)};
    const i16x2 positive = {MOST, MOST};
    const mx_u16x2 v = __builtin_elementwise_min(__builtin_bit_cast(mx_u16x2, w), negative);
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(i16x2, v), positive));
  };
  return make_uint4(two(b.x), two(b.y), two(b.z), two(b.w));
}

template <int DT, int RC, int MT>
__global__ __launch_bounds__(LORA_WAVES * 64) void lora_up_kernel(Lora p, int splits, int pitch, int cblocks, int nblocks,
                                                                 const float* __restrict__ part) {
  constexpr int PARTS = DT == MX_BF16 ? 3 : 2, ROWS = MT * 16, UNITS = RC * 4, LD = RC * 32 + 8, NT = 4, COLS = NT * 16;
  constexpr int OUT = COLS + 4;                   // floats from row to row of a wave's results
  __shared__ __attribute__((aligned(16))) uint16_t vs[PARTS][ROWS][LD];
  __shared__ __attribute__((aligned(16))) float results[LORA_WAVES][16 * OUT];
  __shared__ int list[ROWS], down[ROWS];          // y's rows; fp16: the power of two taken out of v
  const int lane = threadIdx.x & 63, i16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool in_place = p.y == p.base;
  const GroupTile t = group_tile(p.offsets, p.L, p.M, ROWS, blockIdx.x / cblocks, !in_place);
  if (t.group < 0) return;
  const bool adapted = t.group < p.L;             // else rows of none: y = base
  for (int i = threadIdx.x; i < ROWS; i += LORA_WAVES * 64) {
    const int row = i < t.rows ? p.rows[t.first + i] : -1;
    list[i] = row >= 0 && row < p.M ? row : -1;
  }
  if (adapted) {
    const float scale = p.scales ? p.scales[t.group] : 1.0f;
    for (int u = threadIdx.x; u < ROWS * UNITS; u += LORA_WAVES * 64) {   // eight columns of a row; UNITS lanes a row
      const int row = u / UNITS, j = u % UNITS * 8;
      mx_f4 v[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      if (row < t.rows && j < p.r) {
        const float* const from = part + ((int64_t)t.first + row) * pitch + j;
        constexpr int AT_ONCE = 8;                // splits in flight together; added in order
        for (int s0 = 0; s0 < splits; s0 += AT_ONCE) {
          mx_f4 w[AT_ONCE][2];
#pragma unroll
          for (int s = 0; s < AT_ONCE; ++s) {
            const float* const at = from + (int64_t)min(s0 + s, splits - 1) * p.M * pitch;
            w[s][0] = *reinterpret_cast<const mx_f4*>(at);
            w[s][1] = *reinterpret_cast<const mx_f4*>(at + 4);
          }
#pragma unroll
          for (int s = 0; s < AT_ONCE; ++s)
            if (s0 + s < splits) {
              v[0] += w[s][0];
              v[1] += w[s][1];
            }
        }
        v[0] *= scale;
        v[1] *= scale;
      }
      uint4 o[3];
      int e;
      lora_operands<DT>(v, UNITS, o, e);
#pragma unroll
      for (int n = 0; n < PARTS; ++n) *reinterpret_cast<uint4*>(&vs[n][row][j]) = o[n];
      if (DT == MX_F16 && j == 0) down[row] = -e;
    }
  }
  __syncthreads();
  const bool whole = ((p.N | p.ldy | p.ldb) & 7) == 0;      // rows in 16-byte pieces
  const int row8 = lane >> 3, c8 = lane & 7;                // a lane's piece: rows row8 and row8 + 8 of 16
  float* const mine = results[wave];
  for (int nb = 0; nb < nblocks; ++nb) {
    const int n0 = ((blockIdx.x % cblocks * nblocks + nb) * LORA_WAVES + wave) * COLS;
    if (n0 >= p.N) break;
    const int n = n0 + c8 * 8;
    uint4 base[MT][2];
    if (whole && p.base) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = list[m * 16 + h * 8 + row8];
          base[m][h] = make_uint4(0u, 0u, 0u, 0u);
          if (row >= 0 && n < p.N) base[m][h] = *reinterpret_cast<const uint4*>(p.base + row * p.ldb + n);
        }
    }
    mx_f4 acc[NT][MT];
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[c][m] = mx_f4{0.f, 0.f, 0.f, 0.f};
    if (adapted) {
      const uint16_t* br[NT];
#pragma unroll
      for (int c = 0; c < NT; ++c) br[c] = p.b + ((int64_t)t.group * p.N + min(n0 + c * 16 + i16, p.N - 1)) * p.r;
#pragma unroll
      for (int kc = 0; kc < RC; ++kc) {
        uint4 bv[NT];
#pragma unroll
        for (int c = 0; c < NT; ++c) bv[c] = load8(br[c], kc * 32 + g * 8, p.r);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < PARTS; ++i) {
            const uint4 v = *reinterpret_cast<const uint4*>(&vs[i][m * 16 + i16][kc * 32 + g * 8]);
#pragma unroll
            for (int c = 0; c < NT; ++c) acc[c][m] = mx_mfma16<DT>(bv[c], v, acc[c][m]);
          }
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      bool nan = false;
#pragma unroll
      for (int c = 0; c < NT; ++c)
        nan |= __builtin_isunordered(acc[c][m][0], acc[c][m][1]) || __builtin_isunordered(acc[c][m][2], acc[c][m][3]);
      if (__any(nan)) {                           // the same bits again, but where B is infinite
        int column = i16;
        asm volatile("" : "+v"(column));          // no address is kept for this
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          const uint16_t* const br = p.b + ((int64_t)t.group * p.N + min(n0 + c * 16 + column, p.N - 1)) * p.r;
          acc[c][m] = mx_f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
          for (int j = g * 8; j < RC * 32; j += 32) {
            const uint4 bv = load8(br, j, p.r), rest = lora_finite<DT>(bv);
#pragma unroll
            for (int i = 0; i < PARTS; ++i)
              acc[c][m] = mx_mfma16<DT>(i == 0 ? bv : rest, *reinterpret_cast<const uint4*>(&vs[i][m * 16 + i16][j]), acc[c][m]);
          }
        }
      }
#pragma unroll
      for (int c = 0; c < NT; ++c) *reinterpret_cast<mx_f4*>(mine + i16 * OUT + c * 16 + g * 4) = acc[c][m];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = m * 16 + h * 8 + row8, row = list[at];
        mx_f4 v[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          v[i] = *reinterpret_cast<const mx_f4*>(mine + (h * 8 + row8) * OUT + c8 * 8 + i * 4);
          if (DT == MX_F16 && adapted) {
#pragma unroll
            for (int q = 0; q < 4; ++q) v[i][q] = __builtin_ldexpf(v[i][q], down[at]);
          }
        }
        if (row < 0) continue;
        uint16_t* const to = p.y + row * p.ldy + n;
        if (whole) {
          if (n >= p.N) continue;
          if (p.base) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t b0 = dword_of(base[m][h], 2 * i), b1 = dword_of(base[m][h], 2 * i + 1);
              v[i] += mx_f4{mx_lo<DT>(b0), mx_hi<DT>(b0), mx_lo<DT>(b1), mx_hi<DT>(b1)};
            }
          }
          const uint2 lo = mx_pack4<DT>(v[0]), hi = mx_pack4<DT>(v[1]);
          __builtin_nontemporal_store(mx_u4{lo.x, lo.y, hi.x, hi.y}, reinterpret_cast<mx_u4*>(to));
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (n + i < p.N) {
              const float f = v[i / 4][i % 4];
              to[i] = mx_round16<DT>(p.base ? f + mx_lo<DT>(p.base[row * p.ldb + n + i]) : f);
            }
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
  }
}

// ---------------------------------------------------------------- launch
static int64_t lora_pitch(int64_t r) { return (r + 15) / 16 * 16; }       // of a row of v's partial sums
// Rows of a tile: 64 where there are many, and some 20 an adapter, else 16.  us, 64 and 16, 4096
// -> 4096: 2048 rows, 5 adapters, rank 128 41, 66; 1024, 32, 64: 22.5, 24.9; 1500, 64, 128: 51,
// 58; but 1000, 4, 64: 21.0, 19.1; 600, 4, 16: 12.3, 9.9; 64, 1, 16: 11.8, 8.3.
static bool lora_tall(int64_t M, int64_t L) { return M >= 1024 && M >= 20 * L; }

LoraPlan lora_plan(int64_t M, int64_t K, int64_t r, int64_t L) {
  LoraPlan p;
  const int64_t kts = (K + 127) / 128, tiles = group_tiles(M, L, lora_tall(M, L) ? 64 : 16) * ((r + 63) / 64);
  const int64_t want = std::max<int64_t>(1, 256 / tiles);   // a workgroup a CU: more splits cost B . v more reads
  p.kt_per = (int)std::max<int64_t>(LORA_WAVES, (kts + want - 1) / want);
  p.splits = (int)((kts + p.kt_per - 1) / p.kt_per);
  p.bytes = (size_t)(p.splits * M * lora_pitch(r)) * 4;
  return p;
}

template <int DT, int MT>
static hipError_t lora_both(const Lora& p, const LoraPlan& plan, float* part, hipStream_t stream) {
  const int pitch = (int)lora_pitch(p.r), rblocks = (p.r + 63) / 64;
  auto down = [&](auto* kernel) {
    return mx_launch(kernel, dim3((unsigned)(plan.splits * rblocks * group_tiles(p.M, p.L, MT * 16))),
                     dim3(LORA_WAVES * 64), stream, p, plan.splits, plan.kt_per, rblocks, pitch, part);
  };
  const hipError_t e = p.r <= 16   ? down(lora_down_kernel<DT, 1, MT>)
                       : p.r <= 32 ? down(lora_down_kernel<DT, 2, MT>)
                                   : down(lora_down_kernel<DT, 4, MT>);
  if (e != hipSuccess) return e;
  const int all = (p.N + LORA_WAVES * 64 - 1) / (LORA_WAVES * 64);
  const int64_t tiles = group_tiles(p.M, p.L + 1, MT * 16);
  // About three workgroups a CU, one round; more column blocks each read v's partial sums
  // less often (2048 rows, rank 64, 11008 columns; 1, 2, 3, 4 blocks: 34, 29, 33, 35 us).
  const int nblocks = (int)std::max<int64_t>(1, std::min<int64_t>(8, all * tiles / 768));
  const int cblocks = (all + nblocks - 1) / nblocks;
  const float* sums = part;
  auto up = [&](auto* kernel) {
    return mx_launch(kernel, dim3((unsigned)(cblocks * tiles)), dim3(LORA_WAVES * 64), stream, p, plan.splits, pitch,
                     cblocks, nblocks, sums);
  };
  return p.r <= 32    ? up(lora_up_kernel<DT, 1, MT>)
         : p.r <= 64  ? up(lora_up_kernel<DT, 2, MT>)
         : p.r <= 128 ? up(lora_up_kernel<DT, 4, MT>)
                      : up(lora_up_kernel<DT, 8, MT>);
}

template <int DT>
static hipError_t lora_dt(const Lora& p, const LoraPlan& plan, float* part, hipStream_t stream) {
  return lora_tall(p.M, p.L) ? lora_both<DT, 4>(p, plan, part, stream) : lora_both<DT, 1>(p, plan, part, stream);
}

hipError_t launch_lora(const Lora& p, int dtype, const LoraPlan& plan, float* part, hipStream_t stream) {
  return dtype == MX_F16 ? lora_dt<MX_F16>(p, plan, part, stream) : lora_dt<MX_BF16>(p, plan, part, stream);
}

}  // namespace wqbmm
