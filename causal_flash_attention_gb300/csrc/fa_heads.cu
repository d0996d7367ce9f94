// Query/key preparation: per-head RMS norm and rotary positions, in one pass.
//
//   n = x * (mean_e x_e^2 + eps)^(-1/2) * w            (w null: n = x)
//   y_a = m (cos t n_a - sin t n_b),  y_b = m (sin t n_a + cos t n_b)
//
// for the rope_dim / 2 pairs (a, b) of the head's first rope_dim elements,
// (i, i + rope_dim / 2) or, interleaved, (2i, 2i + 1), with t the token's
// position times the pair's frequency and m = rope_scale; the rest of the head
// is n. Backward, with r = (mean x^2 + eps)^(-1/2) and dn the gradient turned
// back by -t:
//
//   dx = r (w dn - x r^2 mean_e(w dn x)),   dw = sum over tokens, heads of dn x r.
//
// The angle. Frequencies come as turns per position in 64-bit fixed point, so
// the token's phase is one wrapping integer product, exact modulo a turn at any
// position, and no range reduction follows: its top 32 bits (a phase within
// 2^-33 of a turn) go to sincospif.
//
// Layout. A head's d elements are held by d / 8 lanes, 8 consecutive elements
// each (16-byte accesses), so a warp takes 32 / (d / 8) heads of a token at a
// time. The pair partner of the half layout sits in another lane of the same
// head (rope_dim is a multiple of 16) and is exchanged by shuffles. A warp does
// all its heads of one token, so each phase is turned into sin and cos once for
// many heads. Everything is bound by the bytes of x and y.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "fa_heads.h"

namespace fa {
namespace {

constexpr int kSms = 152;
constexpr int kWarpsH = 8;
constexpr unsigned kFull = 0xffffffffu;

template <typename T>
struct alignas(16) Vec8 { T x[8]; };

template <typename T>
__device__ __forceinline__ void load8(const void* base, long long at, float (&f)[8]) {
  const Vec8<T> v = *reinterpret_cast<const Vec8<T>*>(static_cast<const T*>(base) + at);
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = static_cast<float>(v.x[e]);
}

template <typename T>
__device__ __forceinline__ void store8(void* base, long long at, const float (&f)[8]) {
  Vec8<T> v;
#pragma unroll
  for (int e = 0; e < 8; ++e) v.x[e] = static_cast<T>(f[e]);
  *reinterpret_cast<Vec8<T>*>(static_cast<T*>(base) + at) = v;
}

// sin and cos of this lane's elements' phases at one position, times
// rope_scale: element e of the lane belongs to pair i(e), and the rotation is
// y_e = c_e n_e + s_e n_partner with the sign of the pair's side in s_e. Elements
// past rope_dim get c = 1, s = 0.
template <int D>
struct Turn {
  float c[8], s[8];
  __device__ __forceinline__ void set(const HeadsParams& p, int sub, int position) {
    const int half = p.rope_dim / 2;
    const int e0 = sub * 8;
    if (e0 >= p.rope_dim) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c[e] = 1.f;
        s[e] = 0.f;
      }
      return;
    }
    auto phase = [&](int i, float& sn, float& cs) {
      const uint64_t turn = static_cast<uint64_t>(static_cast<long long>(position)) * p.turns[i];
      // top 32 bits as a signed fraction of half a turn
      const float x = static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f;
      sincospif(x, &sn, &cs);
      sn *= p.rope_scale;
      cs *= p.rope_scale;
    };
    if (p.interleaved) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        float sn, cs;
        phase((e0 + e) / 2, sn, cs);
        c[e] = c[e + 1] = cs;
        s[e] = -sn;
        s[e + 1] = sn;
      }
    } else {
      const bool second = e0 >= half;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float sn, cs;
        phase(e0 + e - (second ? half : 0), sn, cs);
        c[e] = cs;
        s[e] = second ? sn : -sn;
      }
    }
  }
  // y = R n (sign = 1) or R^T n (sign = -1); every lane of the warp calls it
  __device__ __forceinline__ void apply(const HeadsParams& p, int lane, float sign,
                                        float (&n)[8]) const {
    constexpr int kLanes = D / 8;
    float o[8];
    if (p.interleaved) {
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = n[e ^ 1];
    } else {
      const int sub = lane % kLanes, h = p.rope_dim / 16;   // lanes of half the rotated part
      const int src = sub < h ? lane + h : (sub < 2 * h ? lane - h : lane);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = __shfl_sync(kFull, n[e], src);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) n[e] = fmaf(c[e], n[e], sign * s[e] * o[e]);
  }
};

template <int D>
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  return x;
}

__device__ __forceinline__ float dot8(const float (&a)[8], const float (&b)[8]) {
  float s0 = 0.f, s1 = 0.f;
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    s0 = fmaf(a[e], b[e], s0);
    s1 = fmaf(a[e + 1], b[e + 1], s1);
  }
  return s0 + s1;
}

// ---------------------------------------------------------------- forward --
// Warp task: one token, `passes` groups of heads from `chunk * passes` on. Head
// index h: query heads, then key heads, then (append) value heads, which are
// copied. Append: row s stands at position seq_lens[b] - S + s and its key and
// value go to that row of the sequence's pages; a position below 0 or a page
// outside the cache is not stored.
template <typename T, int D, bool kAppend>
__global__ void __launch_bounds__(32 * kWarpsH)
    heads_fwd_kernel(const __grid_constant__ HeadsParams p, int passes, int chunks) {
  constexpr int kLanes = D / 8, kHeads = 32 / kLanes;   // lanes a head, heads a pass
  const int lane = threadIdx.x & 31;
  const int sub = lane % kLanes;
  const long long task = static_cast<long long>(blockIdx.x) * kWarpsH + (threadIdx.x >> 5);
  const long long token = task / chunks;
  if (token >= static_cast<long long>(p.B) * p.S) return;
  const int chunk = static_cast<int>(task - token * chunks);
  const int b = static_cast<int>(token / p.S), s = static_cast<int>(token % p.S);
  const int H = p.Hq + (kAppend ? 2 : 1) * p.Hkv;
  int position = s;
  long long page_row = -1;   // append: row of the cache [block][Hkv][block_size], head 0
  if constexpr (kAppend) {
    position = p.seq_lens[b] - p.S + s;
    if (position >= 0 && position / p.block_size < p.max_blocks) {
      const int pb = p.block_table[static_cast<size_t>(b) * p.max_blocks + position / p.block_size];
      if (pb >= 0 && pb < p.num_blocks)
        page_row = static_cast<long long>(pb) * p.Hkv * p.block_size + position % p.block_size;
    }
  } else if (p.positions) {
    position = p.positions[token];
  }
  Turn<D> turn;
  turn.set(p, sub, position);
  const int h0 = chunk * passes * kHeads + lane / kLanes;
  for (int i = 0; i < passes; ++i) {
    const int h = h0 + i * kHeads;
    const bool live = h < H;
    const bool is_q = h < p.Hq, is_v = kAppend && h >= p.Hq + p.Hkv;
    const int hh = is_q ? h : (is_v ? h - p.Hq - p.Hkv : h - p.Hq);
    const HeadView& in = is_q ? p.q : (is_v ? p.v : p.k);
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (live) load8<T>(in.data, b * in.sb + hh * in.sh + s * in.ss + sub * 8, x);
    if (p.wq) {
      const float r = rsqrtf(head_sum<D>(dot8(x, x)) * (1.f / D) + p.eps);
      if (live && !is_v) {
        float w[8];
        load8<T>(is_q ? p.wq : p.wk, sub * 8, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * r * w[e];
      }
    }
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = x[e];
    turn.apply(p, lane, 1.f, y);
    if (!live) continue;
    if (!kAppend || is_q) {
      const HeadView& out = is_q ? p.q_out : p.k_out;
      store8<T>(out.data, b * out.sb + hh * out.sh + s * out.ss + sub * 8, y);
    } else if (page_row >= 0) {
      const long long at = (page_row + static_cast<long long>(hh) * p.block_size) * D + sub * 8;
      if (is_v) store8<T>(p.v_cache, at, x);
      else store8<T>(p.k_cache, at, y);
    }
  }
}

// --------------------------------------------------------------- backward --
// Warps stride over the tokens; each does all heads of a token. A lane's share
// of dw_q and dw_k (its 8 columns) is summed in registers over all its tokens,
// then over the block's warps, then over the blocks by the reduce kernel, always
// in the same order.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarpsH)
    heads_bwd_kernel(const __grid_constant__ HeadsParams p) {
  constexpr int kLanes = D / 8, kHeads = 32 / kLanes;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % kLanes;
  const int H = p.Hq + p.Hkv;
  const bool norm = p.wq != nullptr;
  float wq[8], wk[8], dwq[8], dwk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dwq[e] = dwk[e] = 0.f;
  if (norm) {
    load8<T>(p.wq, sub * 8, wq);
    load8<T>(p.wk, sub * 8, wk);
  }
  const long long tokens = static_cast<long long>(p.B) * p.S;
  for (long long token = static_cast<long long>(blockIdx.x) * kWarpsH + warp; token < tokens;
       token += static_cast<long long>(gridDim.x) * kWarpsH) {
    const int b = static_cast<int>(token / p.S), s = static_cast<int>(token % p.S);
    Turn<D> turn;
    turn.set(p, sub, p.positions ? p.positions[token] : s);
    for (int g = 0; g < H; g += kHeads) {
      const int h = g + lane / kLanes;
      const bool live = h < H, is_q = h < p.Hq;
      const int hh = is_q ? h : h - p.Hq;
      const HeadView& dy = is_q ? p.q_out : p.k_out;
      const HeadView& in = is_q ? p.q : p.k;
      const HeadView& dx = is_q ? p.dq : p.dk;
      float dn[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (live) {
        load8<T>(dy.data, b * dy.sb + hh * dy.sh + s * dy.ss + sub * 8, dn);
        if (norm) load8<T>(in.data, b * in.sb + hh * in.sh + s * in.ss + sub * 8, x);
      }
      turn.apply(p, lane, -1.f, dn);
      if (norm) {
        const float r = rsqrtf(head_sum<D>(dot8(x, x)) * (1.f / D) + p.eps);
        float gx[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float t = dn[e] * (x[e] * r);
          if (is_q) dwq[e] += t;
          else dwk[e] += t;
          gx[e] = dn[e] * (is_q ? wq[e] : wk[e]);
        }
        const float m = head_sum<D>(dot8(gx, x)) * (1.f / D) * r * r;
#pragma unroll
        for (int e = 0; e < 8; ++e) dn[e] = r * (gx[e] - x[e] * m);
      }
      if (live) store8<T>(dx.data, b * dx.sb + hh * dx.sh + s * dx.ss + sub * 8, dn);
    }
  }
  if (!norm) return;
  // lanes of one column group, then warps
  __shared__ float part[kWarpsH][2][D];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1) {
      dwq[e] += __shfl_xor_sync(kFull, dwq[e], o);
      dwk[e] += __shfl_xor_sync(kFull, dwk[e], o);
    }
    if (lane < kLanes) {
      part[warp][0][sub * 8 + e] = dwq[e];
      part[warp][1][sub * 8 + e] = dwk[e];
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * D; c += blockDim.x) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kWarpsH; ++w) t += part[w][c / D][c % D];
    p.dw_part[static_cast<size_t>(blockIdx.x) * 2 * D + c] = t;
  }
}

// dw = sum over blocks: one block of 256 threads per 32 of the 2 d columns, 8
// threads a column striding over the blocks.
__global__ void __launch_bounds__(256) heads_dw_kernel(const __grid_constant__ HeadsParams p) {
  __shared__ float part[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float t = 0.f;
  for (int i = warp; i < p.n_blocks; i += 8) t += p.dw_part[static_cast<size_t>(i) * 2 * p.d + c];
  part[warp][lane] = t;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int w = 1; w < 8; ++w) t += part[w][lane];
    if (c < p.d) p.dwq[c] = t;
    else p.dwk[c - p.d] = t;
  }
}

// Head groups a warp takes: all of a token's where the tokens alone fill the GPU
// with warps (one conversion of phases into sin and cos for all heads), fewer
// where they do not, down to one.
template <typename T, int D, bool kAppend>
cudaError_t launch_fwd_impl(const HeadsParams& p, cudaStream_t stream) {
  constexpr int kHeads = 32 / (D / 8);
  const int H = p.Hq + (kAppend ? 2 : 1) * p.Hkv;
  const int groups = (H + kHeads - 1) / kHeads;
  const long long tokens = static_cast<long long>(p.B) * p.S;
  const long long fill = kSms * 32LL;   // warps
  const int passes = static_cast<int>(std::max<long long>(1, std::min<long long>(groups, tokens * groups / fill)));
  const int chunks = (groups + passes - 1) / passes;
  const long long blocks = (tokens * chunks + kWarpsH - 1) / kWarpsH;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  heads_fwd_kernel<T, D, kAppend><<<static_cast<unsigned>(blocks), 32 * kWarpsH, 0, stream>>>(p, passes, chunks);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_bwd_impl(const HeadsParams& p, cudaStream_t stream) {
  heads_bwd_kernel<T, D><<<static_cast<unsigned>(p.n_blocks), 32 * kWarpsH, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.wq) return e;
  heads_dw_kernel<<<2 * D / 32, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

template <bool kAppend>
cudaError_t dispatch_fwd(const HeadsParams& p, cudaStream_t st) {
  const bool big = p.d == 128;
  switch (p.dtype) {
    case 0: return big ? launch_fwd_impl<float, 128, kAppend>(p, st) : launch_fwd_impl<float, 64, kAppend>(p, st);
    case 1: return big ? launch_fwd_impl<__half, 128, kAppend>(p, st) : launch_fwd_impl<__half, 64, kAppend>(p, st);
    default:
      return big ? launch_fwd_impl<__nv_bfloat16, 128, kAppend>(p, st)
                 : launch_fwd_impl<__nv_bfloat16, 64, kAppend>(p, st);
  }
}

}  // namespace

int heads_bwd_blocks(int B, int S) {
  const long long tokens = static_cast<long long>(B) * S;
  return static_cast<int>(std::max<long long>(1, std::min<long long>((tokens + kWarpsH - 1) / kWarpsH, kSms * 4LL)));
}

cudaError_t launch_heads_fwd(const HeadsParams& p, cudaStream_t stream) {
  return dispatch_fwd<false>(p, stream);
}
cudaError_t launch_heads_append(const HeadsParams& p, cudaStream_t stream) {
  return dispatch_fwd<true>(p, stream);
}
cudaError_t launch_heads_bwd(const HeadsParams& p, cudaStream_t stream) {
  const bool big = p.d == 128;
  switch (p.dtype) {
    case 0: return big ? launch_bwd_impl<float, 128>(p, stream) : launch_bwd_impl<float, 64>(p, stream);
    case 1: return big ? launch_bwd_impl<__half, 128>(p, stream) : launch_bwd_impl<__half, 64>(p, stream);
    default:
      return big ? launch_bwd_impl<__nv_bfloat16, 128>(p, stream)
                 : launch_bwd_impl<__nv_bfloat16, 64>(p, stream);
  }
}

}  // namespace fa
