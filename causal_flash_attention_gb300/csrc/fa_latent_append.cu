// New tokens into the paged latent cache: a token's latent c (rank elements) gets its RMS
// norm, its shared key part and its heads' query parts (64 elements each) are rotated by
// its position,
//
//   row of the cache = [ c (mean_e c_e^2 + eps)^(-1/2) weight | rotated k_rope ],  q_out = rotated q_rope,
//
// with the rotation, its table of turns and the norm's conventions as in fa_heads.cu.
//
// A warp takes units of a token: the latent (8 elements a lane, rank / 256 vectors of them),
// or a group of four 64-element heads (8 lanes a head), the shared key part being head 0 of
// the first group's place in the order of work. Bound by the launch for a step's few
// tokens, by the bytes for prompts.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "fa_latent.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kWarpsA = 8;
constexpr unsigned kFullA = 0xffffffffu;

// 8 consecutive elements in fp32.
template <typename T>
__device__ __forceinline__ void load8(const T* src, float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = reinterpret_cast<const float4*>(src)[0], b = reinterpret_cast<const float4*>(src)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(src);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<std::is_same<T, __nv_bfloat16>::value>(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* dst, const float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack2<std::is_same<T, __nv_bfloat16>::value>(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// A block takes one token, or (blockIdx.y of gridDim.y) a part of its units: unit 0 the
// latent, unit 1 the shared key part, unit 2 + i query heads 4 i to 4 i + 3.
template <typename T, int RANK>
__global__ void __launch_bounds__(32 * kWarpsA)
    latent_append_kernel(const __grid_constant__ LatentAppendParams p) {
  __shared__ float2 table[kRope / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (gridDim.x * gridDim.y <= 152) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const unsigned token = blockIdx.x;   // B * Sq < 2^31
  const int b = static_cast<int>(token / p.Sq);
  const int s = static_cast<int>(token - static_cast<unsigned>(b) * p.Sq);
  // (a length may be any int32, and so far below 0 that 32 bits would wrap around)
  const long long row = static_cast<long long>(p.seq_lens[b]) - p.Sq + s;
  if (threadIdx.x < kRope / 2) {
    const long long position = p.positions ? p.positions[token] : row;
    const uint64_t turn = static_cast<uint64_t>(position) * p.turns[threadIdx.x];
    const float x = static_cast<float>(static_cast<int>((turn + 0x80000000u) >> 32)) * 0x1p-31f;
    float sn, cs;
    sincospif(x, &sn, &cs);
    table[threadIdx.x] = make_float2(cs * p.rope_scale, sn * p.rope_scale);
  }
  __syncthreads();
  const int first = static_cast<int>(blockIdx.y) * kWarpsA + warp, step = static_cast<int>(gridDim.y) * kWarpsA;
  const int units = 2 + (p.H + 3) / 4;
  long long cache_row = -1;
  if (first < 2 && row >= 0 && row / p.block_size < p.max_blocks) {
    const int pb = p.block_table[static_cast<size_t>(b) * p.max_blocks + row / p.block_size];
    if (pb >= 0 && pb < p.num_blocks) cache_row = static_cast<long long>(pb) * p.block_size + row % p.block_size;
  }
  T* const cache = static_cast<T*>(p.cache) + cache_row * (RANK + kRope);
  for (int u = first; u < units; u += step) {
    if (u == 0) {
      constexpr int N = RANK / 256;
      const T* src = static_cast<const T*>(p.latent.data) + b * p.latent.sb + s * p.latent.ss;
      float x[N][8], sum = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        load8(src + i * 256 + lane * 8, x[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(x[i][e], x[i][e], sum);
      }
      if (p.weight) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFullA, sum, o);
        // the mean plus eps at least the least normal number, as for heads: zeros stay zeros
        float r;
        asm("{\n\t.reg .f32 t;\n\tmax.NaN.f32 t, %1, %2;\n\trsqrt.approx.ftz.f32 %0, t;\n\t}"
            : "=f"(r) : "f"(sum * (1.f / RANK) + p.eps), "f"(0x1p-126f));
#pragma unroll
        for (int i = 0; i < N; ++i) {
          float w[8];
          load8(static_cast<const T*>(p.weight) + i * 256 + lane * 8, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[i][e] = x[i][e] * r * w[e];
        }
      }
      if (cache_row >= 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) store8(cache + i * 256 + lane * 8, x[i]);
      }
      continue;
    }
    const int h = u == 1 ? 0 : (u - 2) * 4 + lane / 8;
    const bool live = u == 1 ? lane < 8 : h < p.H;
    const HeadView& v = u == 1 ? p.k_rope : p.q_rope;
    const int e0 = (lane & 7) * 8;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, y[8];
    if (live) load8(static_cast<const T*>(v.data) + b * v.sb + h * v.sh + s * v.ss + e0, x);
    if (p.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 t = table[e0 / 2 + i];
        y[2 * i] = t.x * x[2 * i] - t.y * x[2 * i + 1];
        y[2 * i + 1] = t.y * x[2 * i] + t.x * x[2 * i + 1];
      }
    } else {   // the partner is four lanes away
      const float sign = e0 < kRope / 2 ? -1.f : 1.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 t = table[(e0 & (kRope / 2 - 1)) + i];
        const float o = __shfl_xor_sync(kFullA, x[i], 4);
        y[i] = t.x * x[i] + sign * t.y * o;
      }
    }
    if (u == 1) {
      if (live && cache_row >= 0) store8(cache + RANK + e0, y);
    } else if (live) {
      store8(static_cast<T*>(p.q_out.data) + b * p.q_out.sb + h * p.q_out.sh + s * p.q_out.ss + e0, y);
    }
  }
}

template <typename T>
cudaError_t launch_type(const LatentAppendParams& p, cudaStream_t stream) {
  const long long tokens = static_cast<long long>(p.B) * p.Sq;
  const int units = 2 + (p.H + 3) / 4;
  // with few tokens a warp a unit
  const int parts = tokens < 152 ? std::min((units + kWarpsA - 1) / kWarpsA, 65535) : 1;
  const dim3 grid(static_cast<unsigned>(tokens), static_cast<unsigned>(parts));
  return launch_dependent(p.rank == 512 ? latent_append_kernel<T, 512> : latent_append_kernel<T, 256>, grid,
                          dim3(32 * kWarpsA), 0, stream, p);
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendParams& p, cudaStream_t stream) {
  switch (p.dtype) {
    case 0: return launch_type<float>(p, stream);
    case 1: return launch_type<__half>(p, stream);
    default: return launch_type<__nv_bfloat16>(p, stream);
  }
}

}  // namespace fa
