// New tokens into the paged latent cache: a token's latent c (rank elements) gets its RMS
// norm, its shared key part and its heads' query parts (64 elements each) are rotated by
// its position,
//
//   row of the cache = [ c (mean_e c_e^2 + eps)^(-1/2) weight | rotated k_rope ],  q_out = rotated q_rope,
//
// with the rotation, its table of turns and the norm's conventions as in fa_heads.cu.
//
// A warp takes units of a token: the latent (8 elements a lane, rank / 256 vectors of them), or
// eight 64-element heads. Bound by the launch for a step's few tokens; for prompts by the issue of
// instructions, as which a lane has both elements of a pair and 16 in all (8 elements and the partners
// by shuffles, one token a block: 9.6 us instead of 6.2 at 3 x 1025 tokens of 16 heads, rank 512).
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

// 8 consecutive elements as they are in memory, and in fp32.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* src) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) r.v[i] = reinterpret_cast<const uint4*>(src)[i];
  return r;
}
template <typename T>
__device__ __forceinline__ void widen(const Raw8<T>& r, float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[4 * i] = __uint_as_float(r.v[i].x); x[4 * i + 1] = __uint_as_float(r.v[i].y);
      x[4 * i + 2] = __uint_as_float(r.v[i].z); x[4 * i + 3] = __uint_as_float(r.v[i].w);
    }
  } else {
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
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

// A block takes kTokens tokens with kWarpsA / kTokens warps each, or (blockIdx.y of gridDim.y) a part
// of one's units: unit 0 the latent, unit 1 + i eight heads (four lanes a head, 16 elements a lane, those
// of a pair in one lane), of which the shared key part is the first and query head h number 1 + h. A
// warp's elements are loaded one unit ahead, the first before the angles are known: they need no length.
template <typename T, int RANK, int kTokens>
__global__ void __launch_bounds__(32 * kWarpsA)
    latent_append_kernel(const __grid_constant__ LatentAppendParams p) {
  constexpr int kAngles = kRope / 2, kPer = kWarpsA / kTokens;   // warps a token
  static_assert(kTokens * kAngles <= 32 * kWarpsA - 32, "a thread an angle, a warp for the rows");
  __shared__ __align__(16) float2 table[kTokens][kAngles];
  __shared__ long long cache_rows[kTokens];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (gridDim.x * gridDim.y <= 152) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const unsigned token0 = blockIdx.x * kTokens;   // B * Sq < 2^31
  const int tokens = static_cast<int>(min(static_cast<unsigned>(kTokens), static_cast<unsigned>(p.B) * p.Sq - token0));
  const int t = warp / kPer;
  const unsigned token = token0 + (t < tokens ? t : 0);
  const int b = static_cast<int>(token / p.Sq);
  const int s = static_cast<int>(token - static_cast<unsigned>(b) * p.Sq);
  const int units = t < tokens ? 1 + (p.H + 8) / 8 : 0, step = static_cast<int>(gridDim.y) * kPer;
  int u = static_cast<int>(blockIdx.y) * kPer + warp % kPer;
  constexpr int N = RANK / 256;   // vectors of 8 elements of a lane: of the latent, and two of a head
  const int e0 = (lane & 3) * 8, e1 = e0 + kRope / 2;   // this lane's elements of a head

  auto load = [&](int unit, Raw8<T> (&x)[2]) {
    if (unit >= units) return;
    if (unit == 0) {
      const T* src = static_cast<const T*>(p.latent.data) + b * p.latent.sb + s * p.latent.ss + lane * 8;
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = load8(src + i * 256);
      return;
    }
    const int h = (unit - 1) * 8 + lane / 4 - 1;   // -1: the shared key part
    if (h >= p.H) return;
    const HeadView& v = h < 0 ? p.k_rope : p.q_rope;
    const T* src = static_cast<const T*>(v.data) + b * v.sb + max(h, 0) * v.sh + s * v.ss;
    x[0] = load8(src + e0);
    x[1] = load8(src + e1);
  };
  Raw8<T> raw[2] = {}, ahead[2] = {};
  load(u, raw);

  {
    // a token's row of its sequence (a length may be any int32, and so far below 0 that 32 bits would
    // wrap around), its angles, and its row of the cache: -1 if it is not stored
    const bool angle = threadIdx.x < kTokens * kAngles;
    const int of = angle ? static_cast<int>(threadIdx.x) / kAngles : static_cast<int>(threadIdx.x) - (32 * kWarpsA - 32);
    if (of >= 0 && of < tokens) {
      const unsigned tok = token0 + of;
      const int seq = static_cast<int>(tok / p.Sq);
      const long long row = static_cast<long long>(p.seq_lens[seq]) - p.Sq + (tok - static_cast<unsigned>(seq) * p.Sq);
      if (angle) {
        const int i = threadIdx.x % kAngles;
        const long long position = p.positions ? p.positions[tok] : row;
        const uint64_t turn = static_cast<uint64_t>(position) * p.turns[i];
        const float f = static_cast<float>(static_cast<int>((turn + 0x80000000u) >> 32)) * 0x1p-31f;
        float sn, cs;
        sincospif(f, &sn, &cs);
        table[of][i] = make_float2(cs * p.rope_scale, sn * p.rope_scale);
      } else {
        long long at = -1;
        if (row >= 0 && row / p.block_size < p.max_blocks) {
          const int pb = p.block_table[static_cast<size_t>(seq) * p.max_blocks + row / p.block_size];
          if (pb >= 0 && pb < p.num_blocks) at = static_cast<long long>(pb) * p.block_size + row % p.block_size;
        }
        cache_rows[of] = at;
      }
    }
  }
  __syncthreads();
  const long long cache_row = cache_rows[t < tokens ? t : 0];
  T* const cache = static_cast<T*>(p.cache) + cache_row * (RANK + kRope);
  for (; u < units; u += step) {
    load(u + step, ahead);
    float x[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i) widen(raw[i], x[i]);
    if (u == 0) {
      if (p.weight) {
        Raw8<T> w[N];
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = load8(static_cast<const T*>(p.weight) + i * 256 + lane * 8);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) sum = fmaf(x[i][e], x[i][e], sum);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFullA, sum, o);
        // the mean plus eps at least the least normal number, as for heads: zeros stay zeros
        float r;
        asm("{\n\t.reg .f32 t;\n\tmax.NaN.f32 t, %1, %2;\n\trsqrt.approx.ftz.f32 %0, t;\n\t}"
            : "=f"(r) : "f"(sum * (1.f / RANK) + p.eps), "f"(0x1p-126f));
#pragma unroll
        for (int i = 0; i < N; ++i) {
          float f[8];
          widen(w[i], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[i][e] = x[i][e] * r * f[e];
        }
      }
      if (cache_row >= 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) store8(cache + i * 256 + lane * 8, x[i]);
      }
    } else {
      const int h = (u - 1) * 8 + lane / 4 - 1;
      float y[2][8];
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 c = table[t][(i == 0 ? e0 : e1) / 2 + k];
            y[i][2 * k] = c.x * x[i][2 * k] - c.y * x[i][2 * k + 1];
            y[i][2 * k + 1] = c.y * x[i][2 * k] + c.x * x[i][2 * k + 1];
          }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 c = table[t][e0 + k];
          y[0][k] = c.x * x[0][k] - c.y * x[1][k];
          y[1][k] = c.y * x[0][k] + c.x * x[1][k];
        }
      }
      T* dst = cache + RANK;
      if (h >= 0) dst = static_cast<T*>(p.q_out.data) + b * p.q_out.sb + h * p.q_out.sh + s * p.q_out.ss;
      if (h < 0 ? cache_row >= 0 : h < p.H) {
        store8(dst + e0, y[0]);
        store8(dst + e1, y[1]);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) raw[i] = ahead[i];
  }
}

template <typename T, int RANK>
cudaError_t launch_rank(const LatentAppendParams& p, cudaStream_t stream) {
  constexpr int kTokens = 4, kSms = 152;
  const long long tokens = static_cast<long long>(p.B) * p.Sq;
  const int units = 1 + (p.H + 8) / 8;
  // with few tokens a warp a unit, with many four tokens a block
  const int parts = tokens < kSms ? std::min((units + kWarpsA - 1) / kWarpsA, 65535) : 1;
  const int each = tokens >= kTokens * kSms ? kTokens : 1;
  const dim3 grid(static_cast<unsigned>((tokens + each - 1) / each), static_cast<unsigned>(parts));
  return launch_dependent(each == 1 ? latent_append_kernel<T, RANK, 1> : latent_append_kernel<T, RANK, kTokens>, grid,
                          dim3(32 * kWarpsA), 0, stream, p);
}

template <typename T>
cudaError_t launch_type(const LatentAppendParams& p, cudaStream_t stream) {
  return p.rank == 512 ? launch_rank<T, 512>(p, stream) : launch_rank<T, 256>(p, stream);
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
