// mx_gemm4.hip -- the product of MXFP4 activations with MXFP4 weights for many
// rows: a preparation kernel quantises x into the tiled layout, and the product
// runs on v_mfma_scale_f32_16x16x128_f8f6f4, both operands as they lie.
//
// 2001 x 8192 x 28672 (M, K, N): 212-220 us and 8.8 of preparation, 4.3 PFLOP/s.
// The matrix cores alone, on random operands in registers, reached 6.8 (the
// card's power limit; 9.6 on zeros); with the barriers and waits 6.1, with the LDS
// reads 5.3, with the copies 4.6 at long K; the rest are the first copies and the
// output of each round of tiles.
#include "mx_tile.hpp"

namespace wqbmm {

// x -> tiled MXFP4.  A wave takes two of a panel's K-tiles; a lane holds whole
// blocks, so nothing crosses lanes.
constexpr int PREP_TILES = 2;
template <int DT>
__global__ __launch_bounds__(256) void mx_prep_kernel(const uint16_t* __restrict__ x, int64_t ldx, int M, int blocks,
                                                      int kt, int kq, int64_t waves, uint8_t* __restrict__ codes,
                                                      uint16_t* __restrict__ scales) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int64_t id = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (id >= waves) return;
  const int per = kq * 4 / PREP_TILES;
  const int64_t p = id / per;
  const int t0 = (int)(id % per) * PREP_TILES;
  const int64_t m = p * kMxPanel + r;
  uint4 v[PREP_TILES][4];
#pragma unroll
  for (int i = 0; i < PREP_TILES; ++i) {
    const int b = 4 * (t0 + i) + g;
    const bool in = m < M && b < blocks;
    const uint4* const from = reinterpret_cast<const uint4*>(x + min(m, (int64_t)M - 1) * ldx + (in ? (int64_t)b * kMxBlock : 0));
#pragma unroll
    for (int j = 0; j < 4; ++j) v[i][j] = from[j];
    if (!in) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  uint32_t both = 0;
#pragma unroll
  for (int i = 0; i < PREP_TILES; ++i) {
    if (t0 + i >= kt) break;
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) top = mx_max16(v[i][j], top);
    const uint32_t s = mx_scale_byte(mx_top_bits<DT>(mx_max16_fold(top)));
    const float f = mx_scale(s);
    both |= s << (8 * i);
    *reinterpret_cast<uint4*>(codes + ((p * kt + t0 + i) * 64 + lane) * 16) = make_uint4(
        mx_encode8<DT>(v[i][0], f), mx_encode8<DT>(v[i][1], f), mx_encode8<DT>(v[i][2], f), mx_encode8<DT>(v[i][3], f));
  }
  scales[((p * kq + t0 / 4) * 64 + lane) * 2 + (t0 / 2 & 1)] = (uint16_t)both;
}

// c += a . b in place (mx_tile.hpp).  SEL: the scale byte of both operands.
template <int SEL>
__device__ __forceinline__ void mfma4_into(mx_f4& c, uint4 a, uint32_t sa, uint4 b, uint32_t sb) {
  const mx_i4 av = __builtin_bit_cast(mx_i4, a), bv = __builtin_bit_cast(mx_i4, b);
  if constexpr (SEL == 0)
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[0,0,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4" : "+a"(c) : "v"(av), "v"(bv), "v"(sa), "v"(sb));
  else if constexpr (SEL == 1)
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4" : "+a"(c) : "v"(av), "v"(bv), "v"(sa), "v"(sb));
  else if constexpr (SEL == 2)
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[0,0,0] op_sel_hi:[1,1,0] cbsz:4 blgp:4" : "+a"(c) : "v"(av), "v"(bv), "v"(sa), "v"(sb));
  else
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[1,1,0] cbsz:4 blgp:4" : "+a"(c) : "v"(av), "v"(bv), "v"(sa), "v"(sb));
}

// Workgroup tile (16*TM*WVM) x (16*TN*WVN), one wave per SIMD; a wave's TM x TN
// results of 16 x 16 stay in the accumulators.  One K-tile (128 k) of both
// operands is a stage of 1 KB pieces, as the MFMA takes them; four stages in
// LDS form a ring.  In phase k (K-tile k's products, operands in registers) a
// wave
//   - waits for its own copies of stage k+1, which were issued three phases
//     before, and meets the others at a barrier;
//   - issues its copies of stage k+3 into the buffer of stage k-1, whose reads
//     every wave consumed before that barrier;
//   - reads stage k+1 into the other set of operand registers, between the
//     products of stage k.  (The wait for these reads is explicit: the compiler
//     inserted none before some of the products.)
// Copies past the end of the K range repeat a tile that exists, so the counts
// of the waits are the same in every phase.
template <int DT, int TM, int TN, int WVM, int WVN>
__device__ __forceinline__ void gemm4_tile(const MxTiled& x, const MxTiled& w, int M, int64_t N, int mblocks,
                                           int nblocks, int splits, int kq_per, uint16_t* __restrict__ y,
                                           float* __restrict__ part) {
  constexpr int WAVES = WVM * WVN;
  constexpr int XP = TM * WVM, WP = TN * WVN;               // 1 KB pieces of a stage
  constexpr int PX = XP / WAVES, PW = (WP + WAVES - 1) / WAVES, P = PX + PW;   // a wave's copies of a stage
  constexpr int S = TM + TN;                                // a wave's operands, and its scale loads of a quad
  // every wave copies as many pieces: where WP is no multiple of WAVES some copy the last one again
  static_assert(XP % WAVES == 0, "");
  // four variables: the compiler tells copies into one from reads of another
  __shared__ __attribute__((aligned(16))) uint8_t s0[(XP + WP) * 1024], s1[(XP + WP) * 1024], s2[(XP + WP) * 1024],
      s3[(XP + WP) * 1024];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WVN, wn = wave % WVN;
  const MxPlace at = mx_place(blockIdx.x, mblocks, nblocks, splits);
  const int x0 = at.rb * XP, p0 = at.cb * WP;
  const int q_lo = at.split * kq_per, q_hi = min(w.kq, q_lo + kq_per);

  // Pieces and scales are addressed as buffer + panel's offset + lane's offset.
  const auto xb = mx_buffer(x.codes + (int64_t)x0 * x.kt * 1024, (int64_t)min(XP, x.panels - x0) * x.kt * 1024);
  const auto wb = mx_buffer(w.codes + (int64_t)p0 * w.kt * 1024, (int64_t)min(WP, w.panels - p0) * w.kt * 1024);
  const auto xsb = mx_buffer(x.scales + (int64_t)x0 * x.kq * 256, (int64_t)min(XP, x.panels - x0) * x.kq * 256);
  const auto wsb = mx_buffer(w.scales + (int64_t)p0 * w.kq * 256, (int64_t)min(WP, w.panels - p0) * w.kq * 256);
  int piece[P], sx_panel[TM], sw_panel[TN];
#pragma unroll
  for (int c = 0; c < P; ++c)
    piece[c] = c < PX ? min(wave * PX + c, x.panels - x0 - 1) * x.kt * 1024
                      : min(min(wave * PW + c - PX, WP - 1), w.panels - p0 - 1) * w.kt * 1024;
#pragma unroll
  for (int t = 0; t < TM; ++t) sx_panel[t] = min(wm * TM + t, x.panels - x0 - 1) * x.kq * 256;
#pragma unroll
  for (int c = 0; c < TN; ++c) sw_panel[c] = min(wn * TN + c, w.panels - p0 - 1) * w.kq * 256;
  const int lane4 = lane * 4, lane16 = lane * 16;
  auto copy = [&](int c, int k, uint8_t* s) __attribute__((always_inline)) {
    uint8_t* const to = s + (c < PX ? wave * PX + c : XP + min(wave * PW + c - PX, WP - 1)) * 1024;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(c < PX ? xb : wb, (__attribute__((address_space(3))) void*)to, 16, lane16,
                                             piece[c] + k, 0, 0);
  };
  auto offset_of = [&](int kt) __attribute__((always_inline)) { return min(kt, w.kt - 1) * 1024; };   // K <= 2^20
  auto stage = [&](int kt, uint8_t* s) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < P; ++c) copy(c, offset_of(kt), s);
  };
  uint32_t scx[TM], scw[TN], nx[TM], nw[TN];
  auto load_scale = [&](int i, int q, uint32_t (&sx)[TM], uint32_t (&sw)[TN]) __attribute__((always_inline)) {
    const int at_q = min(q, w.kq - 1) * 256;
    if (i < TM) sx[i < TM ? i : 0] = __builtin_amdgcn_raw_buffer_load_b32(xsb, lane4, sx_panel[i < TM ? i : 0] + at_q, 0);
    else sw[i - TM] = __builtin_amdgcn_raw_buffer_load_b32(wsb, lane4, sw_panel[i - TM] + at_q, 0);
  };

  mx_f4 acc[TN][TM];
#pragma unroll
  for (int c = 0; c < TN; ++c)
#pragma unroll
    for (int t = 0; t < TM; ++t) acc[c][t] = mx_f4{0.f, 0.f, 0.f, 0.f};

  // Two sets of operands, x's TM tiles and then w's TN: one is multiplied, the other read.
  uint4 o0[S], o1[S];
  auto read = [&](const uint8_t* s, uint4 (&o)[S], int i) __attribute__((always_inline)) {
    const int tile = i < TM ? wm * TM + i : XP + wn * TN + i - TM;
    o[i] = *reinterpret_cast<const uint4*>(s + tile * 1024 + lane16);
  };
  // Products of the stage in registers.  The reads of the next stage, the
  // copies of a later one and, in a quad's first phase, the next quad's scales
  // stand between them, in this order (the compiler moves no memory access
  // across a volatile asm).  The reads are issued in the first three quarters
  // of the phase, so that the wait for them at its end finds them done.
  auto multiply = [&](auto ic, auto scales_c, const uint4 (&o)[S], const uint8_t* next, uint4 (&o_next)[S], int kt,
                      uint8_t* into, int q_next) __attribute__((always_inline)) {
    constexpr int i = decltype(ic)::value;
    constexpr bool SCALES = decltype(scales_c)::value;
    constexpr int RS = TM * TN * 3 / 4 / S, CS = TM * TN / P, SS = TM * TN / S;   // products from one to the next
    const int k = offset_of(kt);
#pragma unroll
    for (int at = 0; at < TM * TN; ++at) {
      const int c = at / TM, t = at % TM;
      if (at % RS == 0 && at / RS < S) read(next, o_next, at / RS);
      if (SCALES && at % SS == 0 && at / SS < S) load_scale(at / SS, q_next, nx, nw);
      mfma4_into<i>(acc[c][t], o[TM + c], scw[c], o[t], scx[t]);
      if (at % CS == 1 && at / CS < P) copy(at / CS, k, into);
    }
  };
  // The wait for the copies leaves later ones in flight; in phase 1 these are
  // phase 0's, whose scale loads are among them.  After the last whole quad no
  // scales follow: phase 0 then loads none (loads without a use would be taken
  // out, and phase 1 would count on them), and phase 1 waits like the others.
  auto meet = [&](auto nc) __attribute__((always_inline)) {
    mx_wait_vm_lds<decltype(nc)::value>();
    mx_barrier();
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using I3 = std::integral_constant<int, 3>;
  using WaitP = std::integral_constant<int, P>;
  using None = std::false_type;
  auto phase0 = [&](auto scales_c, int q) __attribute__((always_inline)) {
    meet(WaitP{});
    multiply(I0{}, scales_c, o0, s1, o1, 4 * q + 3, s3, q + 1);
  };
  auto phase1 = [&](auto scales_c, int q) __attribute__((always_inline)) {
    meet(std::integral_constant<int, decltype(scales_c)::value ? P + S : P>{});
    multiply(I1{}, None{}, o1, s2, o0, 4 * q + 4, s0, 0);
  };
  auto phase2 = [&](int q) __attribute__((always_inline)) {
    meet(WaitP{});
    multiply(I2{}, None{}, o0, s3, o1, 4 * q + 5, s1, 0);
  };
  auto phase3 = [&](int q) __attribute__((always_inline)) {
    meet(WaitP{});
    multiply(I3{}, None{}, o1, s0, o0, 4 * q + 6, s2, 0);
  };

#pragma unroll
  for (int i = 0; i < S; ++i) load_scale(i, q_lo, scx, scw);
  stage(4 * q_lo, s0);
  stage(4 * q_lo + 1, s1);
  stage(4 * q_lo + 2, s2);
  meet(std::integral_constant<int, 2 * P>{});
#pragma unroll
  for (int i = 0; i < S; ++i) read(s0, o0, i);
  const int whole = min(q_hi, w.kt / 4);
  int q = q_lo;
  for (; q < whole; ++q) {
    phase0(std::true_type{}, q);
    phase1(std::true_type{}, q);
    phase2(q);
    phase3(q);
#pragma unroll
    for (int t = 0; t < TM; ++t) scx[t] = nx[t];
#pragma unroll
    for (int c = 0; c < TN; ++c) scw[c] = nw[c];
  }
  if (q < q_hi) {                                           // the last quad ends early
    phase0(None{}, q);
    if (4 * q + 1 < w.kt) phase1(None{}, q);
    if (4 * q + 2 < w.kt) phase2(q);
  }
  mx_wait_vm<0>();                                          // copies must not outlive the workgroup's LDS
  mx_wait_results();
  if (!part && (N & 7) == 0) {
    mx_barrier();                                           // no wave reads the stages or copies into them any more
    static_assert(mx_stage_bytes<TM, TN>() <= (XP + WP) * 1024, "a wave's rows fit a stage");
    uint8_t* const mine = wave == 0 ? s0 : wave == 1 ? s1 : wave == 2 ? s2 : s3;
    mx_store_rows<DT, TM, TN>(y, M, N, (x0 + wm * TM) * 16, (int64_t)(p0 + wn * TN) * kMxPanel, lane, mine,
                              [&](int c, int t) __attribute__((always_inline)) {
                                mx_keep_in_place(acc[c][t]);   // read here, not all of them ahead of the first store
                                return acc[c][t];
                              });
    return;
  }

  mx_store_tile<DT>(y, part, at.split, M, N, [&](auto put) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
      for (int c = 0; c < TN; ++c) {
        mx_keep_in_place(acc[c][t]);                           // read here, not all of them ahead of the first store
        put((x0 + wm * TM + t) * 16 + (lane & 15), (int64_t)(p0 + wn * TN + c) * kMxPanel + 4 * (lane >> 4), acc[c][t]);
      }
  });
}

template <int DT, int TM, int TN, int WVM, int WVN>
__global__ __launch_bounds__(64 * WVM * WVN) void mx_gemm4_kernel(MxTiled x, MxTiled w, int M, int64_t N,
                                                                  int mblocks, int nblocks, int splits, int kq_per,
                                                                  uint16_t* __restrict__ y,
                                                                  float* __restrict__ part) {
  gemm4_tile<DT, TM, TN, WVM, WVN>(x, w, M, N, mblocks, nblocks, splits, kq_per, y, part);
}

// ---------------------------------------------------------------- launch
// Measured (with the preparation) at 2048 x 4096 x 4096: 36, 33, 27 and 32 us; at
// 2001 x 8192 x 28672: 240, 231, 273 and 371 us; at 256 x 4096 x 4096: 30, 28, 20
// and 15 us.
constexpr MxTileCost kTiles[] = {{256, 256, 6.0, 0.85}, {256, 224, 6.0, 0.78}, {128, 256, 4.0, 0.50}, {64, 128, 0.0, 0.20}};

MxGemmPlan mx_gemm4_plan(int64_t M, int64_t K, int64_t N) {
  MxGemmPlan p = mx_choose(kTiles, 4, 7.0, M, K, N);
  p.x_bytes = (mx_tiled_bytes(K, M) + 255) / 256 * 256;
  return p;
}

template <int DT>
static hipError_t gemm4_dt(const void* x, int64_t ldx, const MxTiled& w, int64_t M, int64_t K, int64_t N, void* y,
                           const MxGemmPlan& plan, uint8_t* ws, hipStream_t stream) {
  const int m = (int)M, blocks = (int)(K / kMxBlock);
  const int mb = (int)plan.mblocks, nb = (int)plan.nblocks, sp = (int)plan.splits, kp = (int)plan.kq_per;
  auto* xp = static_cast<const uint16_t*>(x);
  auto* yp = static_cast<uint16_t*>(y);
  const MxTiled xt = mx_view(ws, K, M);
  auto* codes = ws;
  auto* scales = reinterpret_cast<uint16_t*>(const_cast<uint8_t*>(xt.scales));
  float* part = sp > 1 ? reinterpret_cast<float*>(ws + plan.x_bytes) : nullptr;
  const int64_t waves = (int64_t)xt.panels * xt.kq * 4 / PREP_TILES;
  hipError_t e = mx_launch(mx_prep_kernel<DT>, dim3((unsigned)((waves + 3) / 4)), dim3(256), stream, xp, ldx, m, blocks,
                           xt.kt, xt.kq, waves, codes, scales);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)(plan.mblocks * plan.nblocks * plan.splits));
  auto go = [&](auto* kernel) {
    return mx_launch(kernel, grid, dim3(256), stream, xt, w, m, N, mb, nb, sp, kp, yp, part);
  };
  switch (plan.variant) {
    case 0: return go(mx_gemm4_kernel<DT, 8, 8, 2, 2>);
    case 1: return go(mx_gemm4_kernel<DT, 8, 7, 2, 2>);
    case 2: return go(mx_gemm4_kernel<DT, 8, 4, 1, 4>);
    default: return go(mx_gemm4_kernel<DT, 4, 2, 1, 4>);
  }
}

hipError_t launch_mx_gemm4(const void* x, int dtype, int64_t ldx, const MxTiled& w, int64_t M, int64_t K, int64_t N,
                           void* y, const MxGemmPlan& plan, uint8_t* ws, hipStream_t stream) {
  const hipError_t e = dtype == MX_F16 ? gemm4_dt<MX_F16>(x, ldx, w, M, K, N, y, plan, ws, stream)
                                       : gemm4_dt<MX_BF16>(x, ldx, w, M, K, N, y, plan, ws, stream);
  if (e != hipSuccess || plan.splits == 1) return e;
  return launch_mx_reduce(reinterpret_cast<const float*>(ws + plan.x_bytes), (int)plan.splits, M, N, y, dtype, stream);
}

}  // namespace wqbmm
