// mx_quant.hip -- quantising to MXFP4, reading back, and the one-time layout
// of MXFP4 weights for the products.  The format and the rounding are stated
// in include/wqbmm_mxfp4.h, the tiled layout in mx_launch.hpp.
#include <algorithm>

#include "mx_device.hpp"
#include "mx_launch.hpp"

namespace wqbmm {

// A thread takes eight consecutive values of a row, four threads a block; the
// largest magnitude is taken over the four with DPP quad permutations.  One
// pass: x is read once, the codes go out as 4 bytes a thread.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  auto dpp = [](uint32_t x, auto ctrl) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, decltype(ctrl)::value, 0xf, 0xf, false);
  };
  v = max(v, dpp(v, std::integral_constant<int, 0xB1>{}));    // lane ^ 1
  return max(v, dpp(v, std::integral_constant<int, 0x4E>{})); // lane ^ 2
}

template <int DT>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const void* __restrict__ x, int64_t ldx, uint32_t kc,
                                                          int64_t chunks, uint32_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
  // chunks and the stride are multiples of 4, so a block's four threads leave together
  for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < chunks; t += (int64_t)gridDim.x * 256) {
    const int64_t m = chunks <= 0x7fffffff ? (int64_t)((uint32_t)t / kc) : t / kc;
    const int64_t at = m * ldx + (t - m * kc) * 8;
    uint32_t top, code = 0;
    if constexpr (DT == MX_F32) {
      const mx_f4* p = reinterpret_cast<const mx_f4*>(static_cast<const float*>(x) + at);
      const mx_f4 a = p[0], b = p[1];
      const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
      top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
      top = quad_max(top);
      const uint32_t s = mx_scale_byte(top);
      if (s < 255u) code = mx_encode8_f32(v, mx_scale(s));
      if ((t & 3) == 0) scales[t >> 2] = (uint8_t)s;
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at);
      top = mx_top_bits<DT>(quad_max(mx_max16_fold(mx_max16(v, 0))));
      const uint32_t s = mx_scale_byte(top);
      if (s < 255u) code = mx_encode8<DT>(v, mx_scale(s));
      if ((t & 3) == 0) scales[t >> 2] = (uint8_t)s;
    }
    codes[t] = code;
  }
}

// A thread stores 16 bytes, so that a wave's stores are 1 KB in a row, past the
// caches: 4099 x 11008 in fp32 took 44.6 us with ordinary stores and takes 29.2
// (7.0 TB/s), and the inputs that follow find more of the cache (quantised and
// read back in turn 78.4 -> 63.8 us).  Stores past the caches of 16 bytes in every
// 32 took 67.
template <int DT>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const void* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, uint32_t kc,
                                                            int64_t chunks, void* __restrict__ y, int64_t ldy) {
  constexpr int VALUES = DT == MX_F32 ? 4 : 8;
  for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < chunks; t += (int64_t)gridDim.x * 256) {
    const int64_t m = chunks <= 0x7fffffff ? (int64_t)((uint32_t)t / kc) : t / kc;
    const int64_t at = m * ldy + (t - m * kc) * VALUES;
    const float s = mx_scale(scales[t / (kMxBlock / VALUES)]);
    if constexpr (DT == MX_F32) {
      const uint32_t c = static_cast<const uint16_t*>(codes)[t];
      const mx_f2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
      mx_f4* p = reinterpret_cast<mx_f4*>(static_cast<float*>(y) + at);
      const mx_f4 v = {a[0], a[1], b[0], b[1]};
      __builtin_nontemporal_store(v, p);
    } else {
      mx_u4* p = reinterpret_cast<mx_u4*>(static_cast<uint16_t*>(y) + at);
      const mx_u4 v = __builtin_bit_cast(mx_u4, mx_decode8<DT>(static_cast<const uint32_t*>(codes)[t], s));
      __builtin_nontemporal_store(v, p);
    }
  }
}

// One workgroup per panel of 16 rows; its four waves take the quads of
// K-tiles in turn.  A one-time conversion: simple rather than fast.
__global__ __launch_bounds__(256) void mx_tile_kernel(const uint8_t* __restrict__ codes,
                                                      const uint8_t* __restrict__ scales, int K, int64_t N,
                                                      int KT, int KQ, uint8_t* __restrict__ out_codes,
                                                      uint32_t* __restrict__ out_scales,
                                                      uint32_t* __restrict__ out_flags) {
  __shared__ int wide;                       // some value is not exact in fp16
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t p = blockIdx.x;
  const int64_t n = p * kMxPanel + (lane & 15);
  const int blocks = K / kMxBlock;
  if (threadIdx.x == 0) wide = 0;
  __syncthreads();
  bool any = false;
  for (int q = wave; q < KQ; q += 4) {
    uint32_t dword = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int kt = 4 * q + i;
      uint32_t s = 127u;
      if (kt < KT) {
        const int b = 4 * kt + (lane >> 4);
        uint4 c = make_uint4(0u, 0u, 0u, 0u);
        if (n < N && b < blocks) {
          c = *reinterpret_cast<const uint4*>(codes + n * (K / 2) + (int64_t)b * 16);
          s = scales[n * blocks + b];
          if (s != 255u && ((c.x | c.y | c.z | c.w) & 0x77777777u) == 0u) s = 127u;
        }
        *reinterpret_cast<uint4*>(out_codes + ((p * KT + kt) * 64 + lane) * 16) = c;
      }
      any |= s < 104u || s > 140u;
      dword |= s << (8 * i);
    }
    out_scales[(p * KQ + q) * 64 + lane] = dword;
  }
  if (any) atomicOr(&wide, 1);
  __syncthreads();
  if (threadIdx.x == 0) out_flags[p] = wide ? 0u : kMxFlagF16;
  // the flags fill whole 16 bytes: equal weights are equal in every byte
  if (p == gridDim.x - 1 && threadIdx.x < 3 && (p + 1 + threadIdx.x) / 4 == p / 4) out_flags[p + 1 + threadIdx.x] = 0;
}

// A thread per chunk; past 2^22 workgroups the threads loop (a grid holds fewer than 2^32 threads).
static dim3 chunk_grid(int64_t chunks) {
  return dim3((unsigned)std::min<int64_t>((chunks + 255) / 256, int64_t(1) << 22));
}

hipError_t launch_mx_quantize(const void* x, int dtype, int64_t M, int64_t K, int64_t ldx, void* codes,
                              void* scales, hipStream_t stream) {
  const uint32_t kc = (uint32_t)(K / 8);
  const int64_t chunks = M * kc;
  auto* c = static_cast<uint32_t*>(codes);
  auto* s = static_cast<uint8_t*>(scales);
  auto* kernel = dtype == MX_F16 ? mx_quantize_kernel<MX_F16>
               : dtype == MX_BF16 ? mx_quantize_kernel<MX_BF16> : mx_quantize_kernel<MX_F32>;
  return mx_launch(kernel, chunk_grid(chunks), dim3(256), stream, x, ldx, kc, chunks, c, s);
}

hipError_t launch_mx_dequantize(const void* codes, const void* scales, int64_t M, int64_t K, void* y,
                                int dtype, int64_t ldy, hipStream_t stream) {
  const uint32_t kc = (uint32_t)(dtype == MX_F32 ? K / 4 : K / 8);
  const int64_t chunks = M * kc;
  auto* c = codes;
  auto* s = static_cast<const uint8_t*>(scales);
  auto* kernel = dtype == MX_F16 ? mx_dequantize_kernel<MX_F16>
               : dtype == MX_BF16 ? mx_dequantize_kernel<MX_BF16> : mx_dequantize_kernel<MX_F32>;
  return mx_launch(kernel, chunk_grid(chunks), dim3(256), stream, c, s, kc, chunks, y, ldy);
}

hipError_t launch_mx_tile(const void* codes, const void* scales, int64_t K, int64_t N, void* w_tiled,
                          hipStream_t stream) {
  const MxTiled v = mx_view(w_tiled, K, N);
  const int k = (int)K;
  auto* c = static_cast<const uint8_t*>(codes);
  auto* s = static_cast<const uint8_t*>(scales);
  auto* oc = const_cast<uint8_t*>(v.codes);
  auto* os = reinterpret_cast<uint32_t*>(const_cast<uint8_t*>(v.scales));
  auto* of = const_cast<uint32_t*>(v.flags);
  return mx_launch(mx_tile_kernel, dim3((unsigned)v.panels), dim3(256), stream, c, s, k, N, v.kt, v.kq, oc, os, of);
}

}  // namespace wqbmm
