// mx_tile.hpp -- what the tiled MXFP4 products (mx_gemm16.hip, mx_gemm4.hip)
// share: the order of workgroup tiles, waits, and the store of a 16 x 16 result.
#pragma once

#include "mx_device.hpp"
#include "mx_launch.hpp"

namespace wqbmm {

// The workgroup's output tile and K range.  XCD x (= id % 8) runs a contiguous
// range of tiles, numbered in bands of four row blocks, column-major within a
// band, so that the tiles an XCD runs together share operands in its L2.
struct MxPlace {
  int rb, cb, split;
};
__device__ __forceinline__ MxPlace mx_place(int id, int mblocks, int nblocks, int splits) {
  constexpr int NXCD = 8, BAND = 4;
  const int tiles = mblocks * nblocks, total = tiles * splits;
  int t = id;
  if (total % NXCD == 0) t = (id % NXCD) * (total / NXCD) + id / NXCD;
  MxPlace p;
  p.split = t / tiles;
  t %= tiles;
  const int band = t / (BAND * nblocks), in_band = t % (BAND * nblocks);
  const int rows = min(BAND, mblocks - band * BAND);
  p.rb = band * BAND + in_band % rows;
  p.cb = in_band / rows;
  return p;
}

// s_waitcnt vmcnt(N) alone: bits 3:0 and 15:14 are the count, expcnt and
// lgkmcnt stay at their "no wait" values.
template <int N>
__device__ __forceinline__ void mx_wait_vm() {
  static_assert(N >= 0 && N < 64, "a 6-bit count");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
// A barrier without a fence: copies and loads in flight stay in flight.
__device__ __forceinline__ void mx_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The same, and all LDS reads.
template <int N>
__device__ __forceinline__ void mx_wait_vm_lds() {
  static_assert(N >= 0 && N < 64, "a 6-bit count");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

__device__ __forceinline__ void mx_wait_lds() { __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4)); }

// The products are written as asm, c += a . b on accumulators that keep their
// registers: through the builtin the compiler may give the sum other registers
// than c, and where the accumulators fill their half of the register file it
// then moved them about in every step.  What the compiler does not see then is
// up to the kernels: LDS reads are waited for explicitly, and the results are
// read after mx_wait_results (the last one is complete after these 32 cycles).
__device__ __forceinline__ void mx_wait_results() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }
// Between an ordinary instruction and a product that reads its result.
__device__ __forceinline__ void mx_settle() { asm volatile("s_nop 1" ::: "memory"); }
__device__ __forceinline__ void mx_keep_in_place(mx_f4& c) { asm volatile("" : "+a"(c)); }

// A buffer of `bytes` (below 2^31) at a wave-uniform address: loads take their
// address as buffer + scalar offset + lane's offset.  Every load stays inside it;
// whether the limit takes the scalar offset into account is not relied on.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t mx_buffer(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00027000);
}

// The copies of 16-bit x: K-tile kt of a row is 256 bytes, 16 chunks of 16 bytes, and
// a lane copies the chunk at mx_x_row + mx_x_chunk + 256 * kt from the tile's first
// row on.  Of `rows` rows of the tile (less than 2^22 values apart) and `left` blocks
// of the K-tile, ones past the end repeat the last row and the K-tile's first chunk:
// their products are not stored, or zeros are multiplied instead.
__host__ __device__ inline int mx_x_row(int row, int rows, int64_t ldx) {
  return (row < rows ? row : rows - 1) * (int)ldx * 2;
}
__host__ __device__ inline int mx_x_chunk(int chunk, int left) { return chunk < 4 * left ? chunk * 16 : 0; }

// fp32 partial sums: split s starts at s * M * pitch, rows are `pitch` apart, a
// multiple of 4 so that a lane's four columns are one aligned store.
__host__ __device__ inline int64_t mx_part_pitch(int64_t N) { return (N + 3) / 4 * 4; }

template <int DT>
__device__ __forceinline__ uint2 mx_pack4(mx_f4 v) {
  return make_uint2(mx_round16<DT>(v[0]) | ((uint32_t)mx_round16<DT>(v[1]) << 16),
                    mx_round16<DT>(v[2]) | ((uint32_t)mx_round16<DT>(v[3]) << 16));
}

// A wave's results: each(f) calls f(m, n, v) for each 16 x 16 tile with the
// lane's row m and its four columns from n on.
template <int DT, typename Each>
__device__ __forceinline__ void mx_store_tile(uint16_t* __restrict__ y, float* __restrict__ part, int split, int M,
                                              int64_t N, Each&& each) {
  if (part) {
    const int64_t pitch = mx_part_pitch(N);
    float* const out = part + split * (M * pitch);
    each([&](int m, int64_t n, mx_f4 v) {
      if (m < M && n < N) *reinterpret_cast<mx_f4*>(out + m * pitch + n) = v;
    });
  } else if ((N & 3) == 0) {
    each([&](int m, int64_t n, mx_f4 v) {
      if (m < M && n < N) *reinterpret_cast<uint2*>(y + m * N + n) = mx_pack4<DT>(v);
    });
  } else {
    each([&](int m, int64_t n, mx_f4 v) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (m < M && n + i < N) y[m * N + n + i] = mx_round16<DT>(v[i]);
    });
  }
}

// The same by way of LDS for N % 8 == 0: the results above leave a lane with 8
// bytes of a row, and stores of 32 bytes a row reached 2 TB/s; from LDS a wave
// stores 16 bytes a lane, whole rows of 32*TN bytes.  `mine` (aligned to 16):
// mx_stage_bytes<TN>() of LDS of this wave's own, half its rows at a time; rows lie
// 16 bytes further apart than they are long, which spreads them over the banks.
// The stores go past the caches, so that less is left to write back when the
// kernel ends (2048 x 4096 x 4096: 51.9 -> 50.8 us with 16-bit x, 25.3 -> 24.2 with MXFP4).
template <int TN>
constexpr int mx_row_bytes() { return TN * 32 + 16; }
template <int TM, int TN>
constexpr int mx_stage_bytes() { return TM / 2 * 16 * mx_row_bytes<TN>(); }
template <int DT, int TM, int TN, typename Value>
__device__ __forceinline__ void mx_store_rows(uint16_t* __restrict__ y, int M, int64_t N, int m0, int64_t n0, int lane,
                                              uint8_t* mine, Value&& value) {
  static_assert(TM % 2 == 0, "two halves");
  constexpr int H = TM / 2, CHUNKS = TN * 2;
  const int r = lane & 15, g = lane >> 4;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
#pragma unroll
    for (int t = 0; t < H; ++t)
#pragma unroll
      for (int c = 0; c < TN; ++c)
        *reinterpret_cast<uint2*>(mine + (t * 16 + r) * mx_row_bytes<TN>() + c * 32 + g * 8) =
            mx_pack4<DT>(value(c, half * H + t));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 0; i < H * 16 * CHUNKS / 64; ++i) {
      const int id = i * 64 + lane, row = id / CHUNKS, chunk = id % CHUNKS;
      const mx_u4 v = *reinterpret_cast<const mx_u4*>(mine + row * mx_row_bytes<TN>() + chunk * 16);
      const int m = m0 + half * H * 16 + row;
      const int64_t n = n0 + chunk * 8;
      if (m < M && n < N) __builtin_nontemporal_store(v, reinterpret_cast<mx_u4*>(y + m * N + n));
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

}  // namespace wqbmm
