// Results of the latent kernels from registers to memory, through a box of shared memory and a
// tensor copy. A thread holds 32 columns of its own row; written from there, a warp's 16-byte
// stores touch 32 rows each, half a sector at a time.
#pragma once

#include "ptx.cuh"

namespace fa {

constexpr int kStoreCols = 32, kStoreRows = 32;       // a warp's box
constexpr int kStoreBytes = kStoreRows * kStoreCols * 2;

// 32 accumulator columns of the warp's 32 rows times f (each thread's own), rounded, to columns col
// and rows row of tm's tensor (rows past its extent are not written). The box: 64-byte rows with the
// 64-byte swizzle, 16-byte units by pairs of rows.
template <bool kBf16>
__device__ __forceinline__ void store_box(uint8_t* box, const CUtensorMap* tm, const uint32_t (&o)[32], float f,
                                          int lane, int col, int row, int h, int b) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = pack2<kBf16>(__uint_as_float(o[8 * u + 2 * e]) * f, __uint_as_float(o[8 * u + 2 * e + 1]) * f);
    *reinterpret_cast<uint4*>(box + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_4d(tm, smem_u32(box), col, row, h, b);
    bulk_commit_group();
  }
  __syncwarp();
}

// The same in fp32: 128-byte rows with the 128-byte swizzle.
__device__ __forceinline__ void store_box_f32(uint8_t* box, const CUtensorMap* tm, const uint32_t (&o)[32], float f,
                                              int lane, int col, int row, int h, int b) {
#pragma unroll
  for (int u = 0; u < 8; ++u)
    *reinterpret_cast<float4*>(box + lane * 128 + ((u ^ (lane & 7)) << 4)) =
        make_float4(__uint_as_float(o[4 * u]) * f, __uint_as_float(o[4 * u + 1]) * f,
                    __uint_as_float(o[4 * u + 2]) * f, __uint_as_float(o[4 * u + 3]) * f);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_4d(tm, smem_u32(box), col, row, h, b);
    bulk_commit_group();
  }
  __syncwarp();
}

}  // namespace fa
