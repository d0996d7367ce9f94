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
// position, and no range reduction follows: rounded to 32 bits (2^-33 of a turn), then to
// fp32 (another 2^-26 of a turn at most, near half a turn) it goes to sincospif.
//
// Layout. A head's d elements are held by d / 8 lanes, 8 elements each, so a warp
// takes a group of 32 / (d / 8) heads of a token at a time. Forward, a lane holds two
// chunks of 4 that are each other's partners in the half layout. Backward, it holds 8
// consecutive elements (16-byte accesses); the partner sits in another lane of
// the same head (rope_dim is a multiple of 16) and is exchanged by shuffles of
// the loaded words. A warp stays with one token, walks its query heads, then its
// key heads (then its value heads), and keeps its columns' factors in registers:
// the weights are multiplied into sin and cos once per token, so that a group
// costs a sum of squares and two products an element, in paired fp32
// instructions. A block's threads turn the phases of its tokens into sin and cos
// once, in shared memory, while the first loads are on their way.
//
// Everything is bound by the bytes of x and y as long as a group costs few
// instructions: a form that found token and head of every group by division ran
// at a quarter of this one's rate. At 8192 tokens, 32 + 8 heads, d = 128: forward 32.0 us
// in bf16 (168 MB, 5.2 TB/s) and 54.3 us in fp32 (6.2 TB/s), backward 57.0 us (252 MB,
// 4.4 TB/s: a group is still about 165 instructions there) and 87.5 us (5.8 TB/s).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "fa_heads.h"
#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kSms = 152;
constexpr int kWarpsH = 8;
constexpr unsigned kFull = 0xffffffffu;

// 8 elements as loaded: 4 words of two 16-bit elements, or 8 of one fp32.
template <typename T>
struct Raw {
  static constexpr int kWords = static_cast<int>(sizeof(T)) * 2;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* src) {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(src)[i];
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void store(T* dst) const {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i)
      reinterpret_cast<uint4*>(dst)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
  // the same in two chunks of 4 elements
  __device__ __forceinline__ void load(const T* a, const T* b) {
    if constexpr (sizeof(T) == 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(a), y = *reinterpret_cast<const uint4*>(b);
      w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
      w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(a), y = *reinterpret_cast<const uint2*>(b);
      w[0] = x.x; w[1] = x.y; w[2] = y.x; w[3] = y.y;
    }
  }
  __device__ __forceinline__ void store(T* a, T* b) const {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<uint4*>(a) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>(b) = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
      *reinterpret_cast<uint2*>(a) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(b) = make_uint2(w[2], w[3]);
    }
  }
  __device__ __forceinline__ Raw from_lane(int src) const {
    Raw r;
#pragma unroll
    for (int i = 0; i < kWords; ++i) r.w[i] = __shfl_sync(kFull, w[i], src);
    return r;
  }
  // elements 2i and 2i + 1 as a pair of fp32, and back
  __device__ __forceinline__ uint64_t pair(int i) const {
    if constexpr (sizeof(T) == 4) {
      return f2_pack(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    } else {
      const float2 f = unpack2<std::is_same<T, __nv_bfloat16>::value>(w[i]);
      return f2_pack(f.x, f.y);
    }
  }
  __device__ __forceinline__ void set_pair(int i, uint64_t v) {
    float a, b;
    f2_unpack(v, a, b);
    if constexpr (sizeof(T) == 4) {
      w[2 * i] = __float_as_uint(a);
      w[2 * i + 1] = __float_as_uint(b);
    } else {
      w[i] = pack2<std::is_same<T, __nv_bfloat16>::value>(a, b);
    }
  }
};

__device__ __forceinline__ uint64_t f2_swap(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return f2_pack(b, a);
}

// In front of a kernel's first access to memory: programmatic dependent of the kernel
// before on the stream.
__device__ __forceinline__ void wait_for_kernel_before() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// (mean x^2 + eps)^(-1/2), the sum at least the least normal number: with eps = 0 a
// head of zeros (a lane past the last head holds one) gives finite factors, not 0 * inf.
__device__ __forceinline__ float inv_rms(float mean, float eps) {
  float y;
  asm("{\n\t.reg .f32 t;\n\tmax.NaN.f32 t, %1, %2;\n\trsqrt.approx.ftz.f32 %0, t;\n\t}"
      : "=f"(y) : "f"(mean + eps), "f"(0x1p-126f));   // a NaN stays one
  return y;
}

// (cos, sin) times rope_scale of pair i at a position: entry i of a token's table.
__device__ __forceinline__ float2 cos_sin(const HeadsParams& p, long long position, int i) {
  const uint64_t turn = static_cast<uint64_t>(position) * p.turns[i];
  // top 32 bits, rounded, as a signed fraction of half a turn
  const float x = static_cast<float>(static_cast<int>((turn + 0x80000000u) >> 32)) * 0x1p-31f;
  float sn, cs;
  sincospif(x, &sn, &cs);
  return make_float2(cs * p.rope_scale, sn * p.rope_scale);
}

// The table of one token, by the warps that share it (warp `w` of `W` here).
__device__ __forceinline__ void fill_table(const HeadsParams& p, float2* table, long long position,
                                           int lane, int w, int W) {
  for (int i = w * 32 + lane; i < p.rope_dim / 2; i += 32 * W) table[i] = cos_sin(p, position, i);
}

// Forward: this lane's two chunks of 4 elements of its head. In the rotated part's half
// layout they are each other's partners (chunk A in the first half, B in the second);
// past the rotated part, and interleaved, they follow each other. One chunk of 8 and
// shuffles for the partners (the backward's layout) take a quarter longer at 8192 tokens,
// 32 + 8 heads, d = 128, bf16. The backward, with its loads of two tensors and more values
// to keep, loses what it gains (8 to 35% slower without shuffles).
template <int D>
struct Chunks {
  int a, b;            // first element of each chunk
  bool turned, halves;
  __device__ __forceinline__ Chunks(const HeadsParams& p, int lane) {
    const int sub = lane % (D / 8);
    turned = sub < p.rope_dim / 8;   // rope_dim / 8 lanes hold the rotated part
    halves = turned && !p.interleaved;
    a = halves ? sub * 4 : sub * 8;
    b = a + (halves ? p.rope_dim / 2 : 4);
  }
};

// This lane's factors from its token's table: y_e = c_e x_e + s_e x_partner, with
// the sign of the pair's side in s.
template <int D>
struct ChunkTurn {
  uint64_t c[4], s[4];
  __device__ __forceinline__ ChunkTurn(const Chunks<D>& at, const float2* table) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = f2_pack(1.f, 1.f);
      s[i] = f2_pack(0.f, 0.f);
    }
    if (!at.turned) return;
    if (at.halves) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 u = table[at.a + 2 * i], v = table[at.a + 2 * i + 1];
        c[i] = c[i + 2] = f2_pack(u.x, v.x);
        s[i] = f2_pack(-u.y, -v.y);
        s[i + 2] = f2_pack(u.y, v.y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 t = table[at.a / 2 + i];
        c[i] = f2_pack(t.x, t.x);
        s[i] = f2_pack(-t.y, t.y);
      }
    }
  }
};

// c x + s (partner of x), pair i of a lane's elements. kWhole: the half layout over the
// whole head. Else x past rope_dim takes no part of another element, were it infinite.
template <bool kWhole, int D>
__device__ __forceinline__ uint64_t turned(const HeadsParams& p, const Chunks<D>& at,
                                           const ChunkTurn<D>& f, const uint64_t (&x)[4], int i) {
  const uint64_t y = f2_mul(f.c[i], x[i]);
  if constexpr (kWhole) return f2_fma(f.s[i], x[i ^ 2], y);
  return at.turned ? f2_fma(f.s[i], p.interleaved ? f2_swap(x[i]) : x[i ^ 2], y) : y;
}

// Backward: this lane's place in its head, and where its elements' pair partners are.
template <int D>
struct Place {
  int e0;            // first element
  int partner;       // half layout: partners of e0, e0 + 1, ... (e0 past rope_dim)
  int src;           // the lane that holds them
  bool turned, second;
  __device__ __forceinline__ Place(const HeadsParams& p, int lane) {
    const int sub = lane % (D / 8), h = p.rope_dim / 16;   // h lanes hold half the rotated part
    e0 = sub * 8;
    turned = sub < 2 * h;
    second = sub >= h;
    const int shift = (p.interleaved || !turned) ? 0 : (second ? -h : h);
    partner = e0 + 8 * shift;
    src = lane + shift;
  }
};

// This lane's factors from its token's table: y_e = c_e x_e + s_e x_partner, with
// the sign of the pair's side (and `sign`: -1 turns back) in s. Elements past
// rope_dim are their own partners (`partners`) and get c = s = 1/2: y = x, infinities
// included, without a select in the inner loop (at 8192 tokens, 32 + 8 heads, d = 128, bf16,
// selects took 57.4 us for 56.8, a branch 58.0).
template <int D>
struct Turn {
  uint64_t c[4], s[4];
  __device__ __forceinline__ Turn(const HeadsParams& p, const Place<D>& at, const float2* table,
                                  float sign) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = s[i] = f2_pack(0.5f, 0.5f);
    if (!at.turned) return;
    if (p.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 t = table[at.e0 / 2 + i];
        c[i] = f2_pack(t.x, t.x);
        s[i] = f2_pack(-sign * t.y, sign * t.y);
      }
    } else {
      const float2* t = table + (at.second ? at.partner : at.e0);
      const float sg = at.second ? sign : -sign;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 a = t[2 * i], b = t[2 * i + 1];
        c[i] = f2_pack(a.x, b.x);
        s[i] = f2_pack(sg * a.y, sg * b.y);
      }
    }
  }
};

// The partners of a loaded vector's elements, past rope_dim they themselves (every lane of
// the warp calls it).
template <typename T, int D>
__device__ __forceinline__ void partners(const HeadsParams& p, const Place<D>& at, const Raw<T>& x,
                                         uint64_t (&o)[4]) {
  if (p.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = at.turned ? f2_swap(x.pair(i)) : x.pair(i);
  } else {   // (src is the lane itself past rope_dim)
    const Raw<T> r = x.from_lane(at.src);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = r.pair(i);
  }
}

template <int D>
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  return x;
}

__device__ __forceinline__ float dot(const uint64_t (&a)[4], const uint64_t (&b)[4]) {
  uint64_t t = f2_mul(a[0], b[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) t = f2_fma(a[i], b[i], t);
  float x, y;
  f2_unpack(t, x, y);
  return x + y;
}

// Tokens a block takes at a time, at most (its table: kTokens * d / 2 pairs).
constexpr int kTokens = 8;
// Resident blocks an SM and groups a warp has in flight (16-bit types; fp32, with
// twice the bytes a group, half). Against these, at 8192 tokens, 32 + 8 heads, d = 128,
// bf16: forward, 4 blocks and 4 groups, 7% longer with 4 and 3, 15% with 3 and 5, 51%
// with 5 and 3 (registers spill, as they do with 4 and 4 in the appending form, which
// takes 3); backward, persistent, 2 blocks and 4 groups (each a dy and an x), 11%
// longer with 2 and 3, 40% with 3 and 4.
constexpr int kFwdBlocks = 4, kFwdFlight = 4;
constexpr int kBwdBlocks = 2, kBwdFlight = 4;
// Warps an SM up to which tokens are spread over more warps than one: a warp's
// set-up (sin and cos, factors, offsets) is worth about five groups, so more
// warps than these cost more than they hide (2000 tokens of the same heads:
// forward 13.0 us at 16, 15.0 at 32, with three groups in flight; backward 19.6 at 8, 22.1 at 16).
constexpr int kFwdWarps = 16, kBwdWarps = 8;

// How blocks share the tokens and their head groups: a block takes `tokens`
// tokens (a power of two), kWarpsH / tokens = 2^log2_warps warps each, or, with
// one token, one of `splits` parts of its groups (blockIdx.y).
struct Shares {
  int tokens, log2_warps, splits;
  Shares(int tokens, int splits) : tokens(tokens), log2_warps(0), splits(splits) {
    while (tokens << log2_warps < kWarpsH) ++log2_warps;
  }
};

// The warp's groups of one class of H heads: g = start, start + W, ... below
// `groups`. `before` groups of the token belong to the classes before it, so
// that warps without a group of one class get the next one's.
struct Groups {
  int start, groups;
  __device__ __forceinline__ Groups(int w, int W, int before, int H, int heads) {
    groups = (H + heads - 1) / heads;
    start = (w - before) % W;
    if (start < 0) start += W;
  }
};

// ---------------------------------------------------------------- forward --
// Classes: query, key and (append) value heads, which are copied. Append: row s
// stands at position seq_lens[b] - S + s and its key and value go to that row of
// the sequence's pages; a position below 0 or a page outside the cache is not
// stored.
template <typename T, int D, bool kAppend>
__global__ void __launch_bounds__(32 * kWarpsH, kFwdBlocks)
    heads_fwd_kernel(const __grid_constant__ HeadsParams p, const Shares sh) {
  constexpr int kLanes = D / 8, kHeads = 32 / kLanes;   // lanes a head, heads a group
  constexpr int kFlight = sizeof(T) == 4 ? kFwdFlight / 2 : (kAppend ? kFwdFlight - 1 : kFwdFlight);
  constexpr int kClasses = kAppend ? 3 : 2;
  __shared__ float2 table[kTokens][D / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Chunks<D> at(p, lane);
  const bool whole = p.rope_dim == D && !p.interleaved;
  const int ab = at.b - at.a;
  const int hl = lane / kLanes;
  const int W = kWarpsH / sh.tokens * sh.splits;
  // this warp's token, and its number among the warps that share it
  const int t = warp >> sh.log2_warps;
  const int w = (warp & (kWarpsH / sh.tokens - 1)) + static_cast<int>(blockIdx.y) * kWarpsH;
  const unsigned token = blockIdx.x * sh.tokens + t;   // B * S < 2^31
  const bool live = token < static_cast<unsigned>(p.B) * p.S;
  const int b = live ? static_cast<int>(token / p.S) : 0;
  const int s = live ? static_cast<int>(token - static_cast<unsigned>(b) * p.S) : 0;
  wait_for_kernel_before();
  // Where there is at most one block an SM, the next kernel's blocks may take their
  // places beside this one's (16 tokens into the cache: 4.0 us a call, 4.3 without; 16 tokens
  // of 32 + 8 heads 2.76, 2.85); with more blocks they would fill the SMs unevenly (375 blocks,
  // 1500 tokens of 12 + 12 heads, d = 64: 5.3 us, 4.6 without; 300 to 600 tokens of 32 + 8
  // heads within 2% either way; 3075 tokens 8.5, 7.4 without).
  if (gridDim.x * gridDim.y <= kSms) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const T* in;
  long long in_step;   // between groups of the warp
  int heads;
  Groups gr(0, 1, 0, 0, 1);
  auto enter = [&](int c) {
    const HeadView& v = c == 0 ? p.q : (c == 1 ? p.k : p.v);
    heads = c == 0 ? p.Hq : p.Hkv;
    const int gq = (p.Hq + kHeads - 1) / kHeads, gk = (p.Hkv + kHeads - 1) / kHeads;
    gr = Groups(w, W, c == 0 ? 0 : (c == 1 ? gq : gq + gk), heads, kHeads);
    if (!live) gr.groups = 0;
    in = static_cast<const T*>(v.data) + b * v.sb + s * v.ss + at.a + (gr.start * kHeads + hl) * v.sh;
    in_step = v.sh * (kHeads * W);
  };
  Raw<T> raw[kFlight];
  auto load = [&](int g) {   // groups g, g + W, ...; `in` moves past them
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      if (g + u * W < gr.groups) {   // warp-uniform
        if ((g + u * W) * kHeads + hl < heads) raw[u].load(in, in + ab);
        else raw[u].zero();
        in += in_step;
      }
    }
  };
  int c = 0;
  enter(0);
  while (gr.start >= gr.groups && c < kClasses - 1) enter(++c);
  load(gr.start);

  long long position = s;
  if (live) {
    // (a length may be any int32, and so far below 0 that 32 bits would wrap around)
    if constexpr (kAppend) position = static_cast<long long>(p.seq_lens[b]) - p.S + s;
    else if (p.positions) position = p.positions[token];
  }
  fill_table(p, table[t], position, lane, warp & (kWarpsH / sh.tokens - 1), kWarpsH / sh.tokens);
  long long page_row = -1;   // append: row of the cache [block][Hkv][block_size]
  if constexpr (kAppend) {
    const int row = static_cast<int>(position);   // below 2^31 where it is not below 0
    if (live && position >= 0 && row / p.block_size < p.max_blocks) {
      const int pb = p.block_table[static_cast<size_t>(b) * p.max_blocks + row / p.block_size];
      if (pb >= 0 && pb < p.num_blocks)
        page_row = static_cast<long long>(pb) * p.Hkv * p.block_size + row % p.block_size;
    }
  }
  __syncthreads();

  for (bool loaded = true;; loaded = false) {
    const T* weight = static_cast<const T*>(c == 0 ? p.wq : p.wk);
    const bool norm = weight != nullptr;
    T* out;
    long long out_step;
    bool store = true;
    if (!kAppend || c == 0) {
      const HeadView& v = c == 0 ? p.q_out : p.k_out;
      out = static_cast<T*>(v.data) + b * v.sb + s * v.ss;
      out_step = v.sh;
    } else {
      out = static_cast<T*>(c == 1 ? p.k_cache : p.v_cache) + page_row * D;
      out_step = static_cast<long long>(p.block_size) * D;
      store = page_row >= 0;
    }
    out += at.a + (gr.start * kHeads + hl) * out_step;
    out_step *= kHeads * W;
    ChunkTurn<D> f(at, table[t]);   // the factors of x and of its partner
    if (norm && c < 2) {
      Raw<T> w;
      w.load(weight + at.a, weight + at.b);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f.c[i] = f2_mul(f.c[i], w.pair(i));
        f.s[i] = f2_mul(f.s[i], p.interleaved ? f2_swap(w.pair(i)) : w.pair(i ^ 2));
      }
    }
    auto walk = [&](auto rotates, auto whole) {
      for (int g = gr.start; g < gr.groups; g += kFlight * W, loaded = false) {
        if (!loaded) load(g);
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
          if (g + u * W < gr.groups) {   // warp-uniform
            if constexpr (rotates.value) {
              uint64_t x[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) x[i] = raw[u].pair(i);
              const float r = norm ? inv_rms(head_sum<D>(dot(x, x)) * (1.f / D), p.eps) : 1.f;
              const uint64_t rr = f2_pack(r, r);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                raw[u].set_pair(i, f2_mul(rr, turned<whole.value>(p, at, f, x, i)));
            }
            if (store && (g + u * W) * kHeads + hl < heads) raw[u].store(out, out + ab);
            out += out_step;
          }
        }
      }
    };
    if (kAppend && c == 2) walk(std::false_type{}, std::false_type{});
    else if (whole) walk(std::true_type{}, std::true_type{});
    else walk(std::true_type{}, std::false_type{});
    if (++c >= kClasses) break;
    enter(c);
  }
}

// --------------------------------------------------------------- backward --
// Blocks stride over groups of tokens, as the forward takes them (splits = 1). A
// lane's share of dw_q and dw_k (its 8 columns) is summed in registers over all
// its tokens, then over the block's warps, then over the blocks by the reduce
// kernel, always in the same order.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarpsH, kBwdBlocks)
    heads_bwd_kernel(const __grid_constant__ HeadsParams p, const Shares sh) {
  constexpr int kLanes = D / 8, kHeads = 32 / kLanes;
  constexpr int kFlight = sizeof(T) == 4 ? kBwdFlight / 2 : kBwdFlight;
  __shared__ float2 table[2][kTokens][D / 2];
  __shared__ float part[kWarpsH][2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Place<D> at(p, lane);
  const int hl = lane / kLanes;
  const int W = kWarpsH / sh.tokens;
  const int t = warp >> sh.log2_warps, w = warp & (W - 1);
  const bool norm = p.wq != nullptr;
  wait_for_kernel_before();
  uint64_t dw[2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) dw[0][i] = dw[1][i] = f2_pack(0.f, 0.f);
  const unsigned all = static_cast<unsigned>(p.B) * p.S;   // < 2^31
  int flip = 0;
  for (unsigned first = blockIdx.x * sh.tokens; first < all; first += gridDim.x * sh.tokens, flip ^= 1) {
    const unsigned token = first + t;
    const bool live = token < all;
    const int b = live ? static_cast<int>(token / p.S) : 0;
    const int s = live ? static_cast<int>(token - static_cast<unsigned>(b) * p.S) : 0;
    if (live) fill_table(p, table[flip][t], p.positions ? p.positions[token] : s, lane, w, W);
    // a token of one warp has a table of its own; else the other table's readers are
    // past it when this one is written again
    if (W == 1) __syncwarp();
    else __syncthreads();
    if (!live) continue;
    const Turn<D> turn(p, at, table[flip][t], -1.f);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const HeadView& vy = c == 0 ? p.q_out : p.k_out;
      const HeadView& vx = c == 0 ? p.q : p.k;
      const HeadView& vd = c == 0 ? p.dq : p.dk;
      const int heads = c == 0 ? p.Hq : p.Hkv;
      const Groups gr(w, W, c == 0 ? 0 : (p.Hq + kHeads - 1) / kHeads, heads, kHeads);
      const int h0 = gr.start * kHeads + hl;
      const T* dy = static_cast<const T*>(vy.data) + b * vy.sb + s * vy.ss + at.e0 + h0 * vy.sh;
      const T* xs = static_cast<const T*>(vx.data) + b * vx.sb + s * vx.ss + at.e0 + h0 * vx.sh;
      T* dx = static_cast<T*>(vd.data) + b * vd.sb + s * vd.ss + at.e0 + h0 * vd.sh;
      const int step = kHeads * W;
      uint64_t wt[4];
      if (norm) {
        Raw<T> v;
        v.load(static_cast<const T*>(c == 0 ? p.wq : p.wk) + at.e0);
#pragma unroll
        for (int i = 0; i < 4; ++i) wt[i] = v.pair(i);
      }
      for (int g = gr.start; g < gr.groups; g += kFlight * W) {
        Raw<T> ry[kFlight], rx[kFlight];
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
          ry[u].zero();
          rx[u].zero();
          if (g + u * W < gr.groups && (g + u * W) * kHeads + hl < heads) {
            ry[u].load(dy);
            if (norm) rx[u].load(xs);
          }
          dy += step * vy.sh;
          xs += step * vx.sh;
        }
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
          if (g + u * W < gr.groups) {   // warp-uniform
            uint64_t dn[4], o[4];
            partners<T, D>(p, at, ry[u], o);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              dn[i] = f2_fma(turn.c[i], ry[u].pair(i), f2_mul(turn.s[i], o[i]));
            if (norm) {
              uint64_t x[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                x[i] = rx[u].pair(i);
                o[i] = f2_mul(dn[i], wt[i]);   // g = w dn
              }
              const float r = inv_rms(head_sum<D>(dot(x, x)) * (1.f / D), p.eps);
              const float m = head_sum<D>(dot(o, x)) * (1.f / D) * r;
              const uint64_t rr = f2_pack(r, r), nm = f2_pack(-m, -m);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                x[i] = f2_mul(x[i], rr);
                dw[c][i] = f2_fma(dn[i], x[i], dw[c][i]);
                dn[i] = f2_mul(rr, f2_fma(nm, x[i], o[i]));
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) ry[u].set_pair(i, dn[i]);
            if ((g + u * W) * kHeads + hl < heads) ry[u].store(dx);
            dx += step * vd.sh;
          }
        }
      }
    }
  }
  if (!norm) return;
  // lanes of one column group, then warps
#pragma unroll
  for (int c = 0; c < 2; ++c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[2];
      f2_unpack(dw[c][i], v[0], v[1]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = kLanes; o < 32; o <<= 1) v[e] += __shfl_xor_sync(kFull, v[e], o);
        if (lane < kLanes) part[warp][c][at.e0 + 2 * i + e] = v[e];
      }
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * D; c += blockDim.x) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kWarpsH; ++i) sum += part[i][c / D][c % D];
    p.dw_part[static_cast<size_t>(blockIdx.x) * 2 * D + c] = sum;
  }
}

// dw = sum over blocks: one block of 256 threads per 32 of the 2 d columns, 8
// threads a column striding over the blocks.
__global__ void __launch_bounds__(256) heads_dw_kernel(const __grid_constant__ HeadsParams p) {
  __shared__ float part[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  wait_for_kernel_before();
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

// Tokens a block takes at a time: as many as it has warps when the tokens alone
// give every SM `warps` warps, else fewer, down to one (never more warps a token
// than it has groups).
int tokens_per_block(long long tokens, int groups, int warps) {
  int W = 1;
  while (W < kWarpsH && W < groups && tokens * W < static_cast<long long>(kSms) * warps) W *= 2;
  return kWarpsH / W;
}

int heads_bwd_tokens(int B, int Hq, int Hkv, int S, int d) {
  const int heads = 32 / (d / 8);
  return tokens_per_block(static_cast<long long>(B) * S, (Hq + heads - 1) / heads + (Hkv + heads - 1) / heads, kBwdWarps);
}

// With few tokens, as many blocks a token as give each group a warp of its own.
template <typename T, int D, bool kAppend>
cudaError_t launch_fwd_impl(const HeadsParams& p, cudaStream_t stream) {
  constexpr int kHeads = 32 / (D / 8);
  const long long tokens = static_cast<long long>(p.B) * p.S;
  const int groups = (p.Hq + kHeads - 1) / kHeads + (kAppend ? 2 : 1) * ((p.Hkv + kHeads - 1) / kHeads);
  Shares sh(tokens_per_block(tokens, groups, kFwdWarps), 1);
  if (sh.tokens == 1 && tokens < kSms) sh.splits = std::min((groups + kWarpsH - 1) / kWarpsH, 65535);
  const dim3 grid(static_cast<unsigned>((tokens + sh.tokens - 1) / sh.tokens), sh.splits);
  return launch_dependent(heads_fwd_kernel<T, D, kAppend>, grid, dim3(32 * kWarpsH), 0, stream, p, sh);
}

template <typename T, int D>
cudaError_t launch_bwd_impl(const HeadsParams& p, cudaStream_t stream) {
  const Shares sh(heads_bwd_tokens(p.B, p.Hq, p.Hkv, p.S, p.d), 1);
  const cudaError_t e = launch_dependent(heads_bwd_kernel<T, D>, dim3(static_cast<unsigned>(p.n_blocks)),
                                         dim3(32 * kWarpsH), 0, stream, p, sh);
  if (e != cudaSuccess || !p.wq) return e;
  return launch_dependent(heads_dw_kernel, dim3(2 * D / 32), dim3(256), 0, stream, p);
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

int heads_bwd_blocks(int B, int Hq, int Hkv, int S, int d) {
  const long long tokens = static_cast<long long>(B) * S;
  const int per = heads_bwd_tokens(B, Hq, Hkv, S, d);
  return static_cast<int>(std::min<long long>((tokens + per - 1) / per, static_cast<long long>(kSms) * kBwdBlocks));
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
