// Backward of latent attention in its expanded form (fa_latent_fwd.cu). With the shared
// rotated part written as the last 64 columns of every head's key, K'_j = [K_j, KR_j],
//
//   p_ij = e^(s_ij - L_i), ds_ij = p_ij (<dO_i, V_j> - D_i), D_i = <dO_i, O_i>,
//   dQ_i = scale sum_j ds_ij K'_j, [dK_j, dKR_j of the head] = scale sum_i ds_ij Q_i,
//   dV_j = sum_i p_ij dO_i, dKR_j = sum over the heads.
//
// Two kernels, each of which recomputes S and dP, instead of one that keeps everything: at
// d = 128 dK' (192 columns) and dV leave no room in tensor memory for a dQ of 192 columns
// beside S and dP, and a dQ kernel of its own needs no sum over key tiles in global
// memory (so gradients have the same bits on every call). Two products more of seven. d = 64 (128 and 64
// columns) takes the same two kernels and their layouts; forms of its own were not tried.
//   1. dQ:      a CTA per 128 query rows walks their key tiles; it also forms D and leaves
//               it with L and the rows' key ranges for the second.
//   2. dK, dV:  a CTA per 128 keys of a head walks the query rows, 64 at a time.
//   3. dKR:     adds up the heads' parts, in head order.
//
// P and dS are rounded to the inputs' type as operands of their products. bf16 has fp32's exponents; in
// fp16 dS is scaled by a power of two first, which the results leave with, since it has the size of
// dO: at |dO| = 1e-4 over 2048 keys it would be a few of fp16's least steps (dQ's and dK's errors 3 to 5
// times an output's own rounding), with short rows and |dO| |V| = 3e5 past its largest value. |dS_ij| is at most
// 2 |dO_i| max_j |V_j| (the norm of O_i is no greater than V's), so one more kernel in front takes the
// norms of V's rows, 128 keys a block; dQ scales each row by its own bound, dK and dV all rows by the greatest
// of the query tiles that see one of their keys. P, at most 1, is scaled by 2^kShiftP for dV. Packed documents of 2999 tokens, 2 x 16 heads: the norms 6 us,
// dQ 53.6 -> 55.5, dK and dV 66.7 -> 68.
// Warp roles of 1 and 2: warp 0 TMA producer, warp 1 MMA issuer, warps 2-9 softmax
// gradient, two warps a tensor-memory lane quarter with half the columns each (four with 16 columns
// each: 1 and 2% slower), in 1 also warp 10 MMA issuer of dQ. P and dS
// go back to tensor memory as the A operands of the products, so shared memory holds
// only what TMA loads.
//
// 4096 tokens, 32 heads, d = 128, bf16, causal: dQ 183 us, 1502 TFLOP/s of products executed (78%
// of a large product's rate), dK and dV 253 us, 1358 (71%), dKR 7.6; d = 64: 138, 194 and 6.9. dQ is bound
// by a tile's chain through the softmax warps (1340 cycles, 1024 of products) and by the filling of a CTA (112
// KB, a tenth of it); dK and dV by shared memory, from which products 64 rows
// wide take both operands (1600 cycles a step instead of 1280, 1950 in all): at d = 128 these columns leave no
// tensor memory for K' and V beside S^T, dP^T, P^T, dS^T and the sums. (With dS^T over dP^T and P^T over S^T V would
// have room, at the cost of the overlap between steps; at d = 64 128 columns are free. Neither was tried.)
#include <algorithm>
#include <type_traits>

#include "fa_latent.h"
#include "latent_store.cuh"
#include "ptx.cuh"
#include "score_mod.cuh"

namespace fa {
namespace {

constexpr int kThreadsQ = 352, kThreadsB = 320;   // of the dQ kernel, of the dK, dV kernel
constexpr float kLog2eB = 1.4426950408889634f;

// The shift e for which 2 bound 2^e < 2^15, half of fp16's range; bound >= 0.
__device__ __forceinline__ int shift_for(float bound) {
  const int e = 13 - (static_cast<int>(__float_as_uint(bound) >> 23) - 127);
  return min(max(e, -64), 64);   // (no bound at all, or one that is not finite)
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }
template <bool kBf16>
constexpr int kShiftP = kBf16 ? 0 : 12;   // of P and L as the dK, dV kernel takes them
__device__ __forceinline__ LatentNorms* norms_of(const LatentBwdParams& p, int bh, int key_tile) {
  return reinterpret_cast<LatentNorms*>(
      p.part + (static_cast<size_t>(bh) * p.mask.Skv + static_cast<size_t>(key_tile) * kTileN) * kRope);
}

template <bool kBf16>
__device__ __forceinline__ float dot16(const uint4& a, const uint4& b, float s) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 u = unpack2<kBf16>(x[e]), v = unpack2<kBf16>(y[e]);
    s = fmaf(u.x, v.x, s);
    s = fmaf(u.y, v.y, s);
  }
  return s;
}

// --------------------------------------------------------------- V's norms --
// The greatest norm of 128 rows of V of a head (fp16 only); a row is D / 8 lanes. Reads V once: 24.6 MB
// at 2 x 16 heads, 2999 tokens.
constexpr int kThreadsN = 256;

template <int D>
__global__ void __launch_bounds__(kThreadsN) latent_norms_kernel(const __grid_constant__ LatentBwdParams p) {
  __shared__ uint32_t tops[kThreadsN / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int BH = p.B * p.H;
  const int tile = static_cast<int>(blockIdx.x) / BH, bh = static_cast<int>(blockIdx.x) % BH;
  const int b = bh / p.H, h = bh % p.H;
  constexpr int kLanes = D / 8, kRowsPass = kThreadsN / kLanes, N = kTileN / kRowsPass;
  const int r0 = tile * kTileN + static_cast<int>(threadIdx.x) / kLanes;
  const uint16_t* src = static_cast<const uint16_t*>(p.v.data) + b * p.v.sb + h * p.v.sh + threadIdx.x % kLanes * 8;
  uint4 x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int row = r0 + i * kRowsPass;
    x[i] = row < p.mask.Skv ? *reinterpret_cast<const uint4*>(src + row * p.v.ss) : make_uint4(0u, 0u, 0u, 0u);
  }
  uint32_t top = 0;   // of squares, as bits: not negative
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float s = dot16<false>(x[i], x[i], 0.f);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    top = max(top, __float_as_uint(s));
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (threadIdx.x % 32 == 0) tops[threadIdx.x / 32] = top;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < kThreadsN / 32; ++w) top = max(top, tops[w]);
  *norms_of(p, bh, tile) = LatentNorms{sqrtf(__uint_as_float(top)), 0.f};
}

// --------------------------------------------------------------------- dQ --
// Q and dO stay in tensor memory, as A operands, for the whole CTA, which leaves shared memory to
// a deep ring of 64-key tiles (with both in shared memory there was room for two K' tiles of
// 128 keys and one of V, whose loads stood in every step: 3700 cycles for 128 keys, of 2048 of
// products), and lets products 64 keys wide run at the tensor core's rate. Tensor memory: S
// [0, 64), dP [64, 128), dQ [128, 192 + d), dS (16-bit) [192 + d, 224 + d), Q, dO behind it: 512
// columns in all at d = 128. S and dP of the next tile are formed while the warps work on this
// tile's, which they have copied to registers.
template <int D>
struct LatDqCfg {
  static constexpr int kW = D + kRope;                  // columns of a key
  static constexpr int kKeys = 64;                      // keys of a tile
  static constexpr int kKChunks = kW / kChunk, kVChunks = D / kChunk;
  static constexpr int CB = kKeys * 128;
  static constexpr int kStageBytes = (kKChunks + kVChunks) * CB;   // K', then V
  static constexpr int NS = D == 128 ? 5 : 6;
  static constexpr int kOffBar = NS * kStageBytes;
  // the rows of O, Q and dO pass through the last stages on their way in
  static constexpr int kFirst = 2;                      // stages for the first tiles meanwhile
  static constexpr int RB = kTileM * 128;               // a chunk of 128 rows
  static constexpr int kOffO = kFirst * kStageBytes, kOffQ = kOffO + kVChunks * RB, kOffDO = kOffQ + kKChunks * RB;
  static_assert(kOffDO + kVChunks * RB <= NS * kStageBytes, "O, Q and dO in the ring");
  // full[], empty[], s_full, dp_full, s_free, dp_free, ds_full, dq_done, drain, q_full, swap[4], drain2,
  // do_full, o_full, o_done
  static constexpr int kNumBars = 2 * NS + 16;
  static constexpr int kOffMisc = (kOffBar + kNumBars * 8 + 15) / 16 * 16;
  static constexpr int kOffSpan = kOffMisc + 16;        // 4 warps' (begin, end)
  static constexpr int kOffDelta = kOffSpan + 32;       // two buffers of [2][128] halves of D
  static constexpr int kOffNorm = kOffDelta + 2048;     // fp16: [2][128] halves of |dO|^2, the norm of V
  static constexpr int kSmemBytes = kOffNorm + 1024 + 16;
  static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
  static constexpr int kColDq = 128, kColDs = kColDq + kW, kColQ = kColDs + 32, kColDO = kColQ + kW / 2;
  static_assert(kColDO + D / 2 <= 512, "tensor memory");
};

template <int D, bool kBf16>
__global__ void __launch_bounds__(kThreadsQ, 1)
    latent_dq_kernel(const __grid_constant__ LatentBwdParams p) {
  using Cfg = LatDqCfg<D>;
  constexpr int NS = Cfg::NS, CB = Cfg::CB, W = Cfg::kW, KT = Cfg::kKeys;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {   // the 128-byte swizzle needs 1024-byte aligned tiles
    if (threadIdx.x == 0) atomicOr(p.status, kStatusBadLaunch);
    return;
  }
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::kOffMisc + 4);
  volatile int* issued = abort_flag + 1;   // tiles that the producer has asked for
  int2* ranges = reinterpret_cast<int2*>(smem + Cfg::kOffSpan);
  float* halves = reinterpret_cast<float*>(smem + Cfg::kOffDelta);
  float* norms = reinterpret_cast<float*>(smem + Cfg::kOffNorm);

  const uint32_t bar0 = sbase + Cfg::kOffBar;
  auto full = [&](int s) { return bar0 + 8 * s; };
  auto empty = [&](int s) { return bar0 + 8 * (NS + s); };
  const uint32_t s_full = bar0 + 8 * 2 * NS;
  const uint32_t dp_full = s_full + 8, s_free = s_full + 16, dp_free = s_full + 24, ds_full = s_full + 32;
  const uint32_t dq_done = s_full + 40, drain = s_full + 48, q_full = s_full + 56;
  auto swap = [&](int quarter) { return s_full + 64 + 8 * quarter; };
  const uint32_t drain2 = swap(4), do_full = swap(5), o_full = swap(6), o_done = swap(7);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(warp_id()), 0);
  const int lane = static_cast<int>(lane_id());
  const int BH = p.B * p.H;
  const int unit = p.n_units - 1 - static_cast<int>(blockIdx.x) / BH;   // last rows first, as in the forward
  const int bh = static_cast<int>(blockIdx.x) % BH;
  const int b = bh / p.H, h = bh % p.H;
  const int q0 = unit * kTileM;
  const int quarter = warp & 3, half = (warp - 2) >> 2;
  const int rr = quarter * 32 + lane, row = q0 + rr;
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;

  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    // one arrival per compute warp; the first phase of s_free says that Q is in tensor memory, that of
    // dp_free that dO is
    mbar_init(s_free, 8);
    mbar_init(dp_free, 8);
    mbar_init(ds_full, 8);
    mbar_init(dq_done, 1);
    mbar_init(drain, 1);
    mbar_init(drain2, 1);
    mbar_init(q_full, 1);
    mbar_init(do_full, 1);
    mbar_init(o_full, 1);
    mbar_init(o_done, 8);
    for (int i = 0; i < 4; ++i) mbar_init(swap(i), 2);   // the two warps of a lane quarter
    *abort_flag = 0;
    fence_mbar_init();
    // rows past Sq come as zeros
    asm volatile("griddepcontrol.wait;" ::: "memory");
    auto rows = [&](uint32_t bar, const CUtensorMap* tm, int off, int chunks) {
      mbar_arrive_expect_tx(bar, chunks * Cfg::RB);
      for (int c = 0; c < chunks; ++c)
        for (int r = 0; r < 2; ++r)
          tma_load_4d(sbase + off + c * Cfg::RB + r * (Cfg::RB / 2), tm, bar, c * kChunk, q0 + r * 64, h, b);
    };
    rows(q_full, &p.tm_q, Cfg::kOffQ, Cfg::kKChunks);
    rows(do_full, &p.tm_do, Cfg::kOffDO, Cfg::kVChunks);
    rows(o_full, &p.tm_o, Cfg::kOffO, Cfg::kVChunks);
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_kr);
    tma_prefetch_desc(&p.tm_v);
  }
  int row_lo = 0, row_hi = 0;
  float l2 = INFINITY;
  const bool soft = warp >= 2 && warp < 10;
  if (soft) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int2 s = p.mask.span(b, row);
    row_lo = s.x;
    row_hi = s.y;
    if (half == 0) {
      const int lo = __reduce_min_sync(0xffffffffu, row_hi > 0 ? row_lo : 0x7fffffff);
      const int hi = __reduce_max_sync(0xffffffffu, row_hi);
      if (lane == 0) ranges[quarter] = make_int2(lo, hi);
    }
  }
  tc_fence_before();
  __syncthreads();   // tensor memory, barriers, ranges
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  int lo = 0x7fffffff, hi = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    lo = min(lo, ranges[w].x);
    hi = max(hi, ranges[w].y);
  }
  const int tile0 = hi > 0 ? lo / KT : 0;
  const int n = hi > 0 ? (hi + KT - 1) / KT - tile0 : 0;

  auto load = [&](int j) {
    const uint32_t f = full(j % NS), dst = sbase + (j % NS) * Cfg::kStageBytes;
    const int y = (tile0 + j) * KT;
    mbar_arrive_expect_tx(f, Cfg::kStageBytes);
    for (int c = 0; c < Cfg::kVChunks; ++c) {
      tma_load_4d(dst + c * CB, &p.tm_k, f, c * kChunk, y, h, b);
      tma_load_4d(dst + (Cfg::kKChunks + c) * CB, &p.tm_v, f, c * kChunk, y, h, b);
    }
    tma_load_4d(dst + Cfg::kVChunks * CB, &p.tm_kr, f, 0, y, 0, b);
  };
  if (warp == 0 && lane == 0)
    for (int j = 0; j < min(n, Cfg::kFirst); ++j) load(j);
  bool ok = true;
  if (!kBf16 && warp == 0) {   // the greatest norm of V's key tiles
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float top = 0.f;
    for (int t = tile0 * KT / kTileN + lane; t * kTileN < hi; t += 32) top = fmaxf(top, __ldcg(&norms_of(p, bh, t)->v));
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    if (lane == 0) norms[256] = top;
    __syncwarp();
    asm volatile("bar.arrive 1, 288;" ::: "memory");
  }
  if (soft) {
    // This thread's halves of its row of Q and dO into tensor memory, its half of D, and L: each as
    // it lands, so that S and dP of the first tile are formed meanwhile.
    if (row < p.mask.Sq && row_hi > 0) l2 = p.lse[static_cast<size_t>(bh) * p.mask.Sq + row] * kLog2eB;
    constexpr int QU = W / 16, OU = D / 16;   // 16-byte units of a half row
    auto unit = [&](int off, int u) {   // unit u of this row, chunks of 128 rows with the 128-byte swizzle
      return *reinterpret_cast<const uint4*>(smem + off + (u >> 3) * Cfg::RB + rr * 128 + (((u & 7) ^ (rr & 7)) << 4));
    };
    auto put = [&](uint32_t landed, uint32_t there, uint32_t col, int off, int first, auto units) {
      constexpr int N = decltype(units)::value;
      // (one outcome for the warp, as for every wait: tensor-memory instructions have to find it whole)
      if (ok) ok = warp_wait(landed, 0, abort_flag, p.status);
      if (!ok) return;
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        uint32_t w[16];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 v = unit(off, first + i + k);
          w[4 * k] = v.x; w[4 * k + 1] = v.y; w[4 * k + 2] = v.z; w[4 * k + 3] = v.w;
        }
        tmem_st16(tmem + lane_off + col + (first + i) * 4, w);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(there);
    };
    put(q_full, s_free, Cfg::kColQ, Cfg::kOffQ, half * QU, std::integral_constant<int, QU>{});
    put(do_full, dp_free, Cfg::kColDO, Cfg::kOffDO, half * OU, std::integral_constant<int, OU>{});
    if (ok) ok = warp_wait(o_full, 0, abort_flag, p.status);
    float d = 0.f, square = 0.f;
    if (ok) {
#pragma unroll
      for (int u = 0; u < OU; ++u) {
        const uint4 g = unit(Cfg::kOffDO, half * OU + u);
        d = dot16<kBf16>(unit(Cfg::kOffO, half * OU + u), g, d);
        if constexpr (!kBf16) square = dot16<kBf16>(g, g, square);
      }
    }
    halves[half * 128 + rr] = d;
    if constexpr (!kBf16) norms[half * 128 + rr] = row_hi > 0 ? square : 0.f;   // a row that sees nothing has no dS
    fence_proxy_async_smem();   // the copies that follow into these stages come after the reads
    __syncwarp();
    if (lane == 0) mbar_arrive(o_done);
    // the halves of D, among these warps; fp16: of |dO|^2, and V's norm from warp 0
    asm volatile("bar.sync 1, %0;" ::"n"(kBf16 ? 256 : 288) : "memory");
  }

  if (warp == 0) {
    // ===================== TMA producer =====================
    if (lane == 0) {
      int j = min(n, Cfg::kFirst);
#ifdef FA_WAIT_TEST
      if (wait_test(kWaitProducer, p.H)) ok = mbar_wait(drain, 0, abort_flag, p.status);
#endif
      if (ok && j < n) ok = mbar_wait(o_done, 0, abort_flag, p.status);   // the other stages are free
      for (; ok && j < n; ++j) {
        if (j >= NS && !mbar_wait(empty(j % NS), (j / NS - 1) & 1, abort_flag, p.status)) break;
        load(j);
      }
      *issued = j;
    }
  } else if (warp == 1) {
    // ===================== MMA issuer of S and dP (the whole warp, one lane of it the MMAs) =====================
    if (n > 0) {
      constexpr uint32_t idesc_s = make_idesc(128, KT, kBf16, false, false);
      auto wait = [&](uint32_t bar, uint32_t parity) { return warp_wait(bar, parity, abort_flag, p.status); };
#ifdef FA_WAIT_TEST
      // wait-limit test build: nothing completes this phase before the abort
      // path's own commit, so the wait runs out
      if (wait_test(kWaitIssuer, p.H)) ok = wait(drain, 0);
#endif
      auto scores = [&](int j) -> bool {   // S = Q K'_j^T, dP = dO V_j^T
        if (!wait(full(j % NS), (j / NS) & 1)) return false;
        if (!wait(s_free, j & 1)) return false;
        tc_fence_after();
        const uint32_t st = sbase + (j % NS) * Cfg::kStageBytes;
        const uint64_t kb = make_sdesc(st, 16, 1024), vb = make_sdesc(st + Cfg::kKChunks * CB, 16, 1024);
        elected([&] {
          mma_ts_steps<W / 16, true, CB>(tmem, tmem + Cfg::kColQ, kb, idesc_s, 0u);
          tc_commit(s_full);
        });
        if (!wait(dp_free, j & 1)) return false;
        tc_fence_after();
        elected([&] {
          mma_ts_steps<D / 16, true, CB>(tmem + KT, tmem + Cfg::kColDO, vb, idesc_s, 0u);
          tc_commit(dp_full);
        });
        return true;
      };
      for (int j = 0; ok && j < n; ++j) ok = scores(j);
    }
  } else if (warp == 10) {
    // ===================== MMA issuer of dQ =====================
    // (one issuer for all: 196 us instead of 192 at 4096 tokens, 32 heads; two in the dK, dV kernel, whose
    // products wait for shared memory: 262 instead of 255)
    if (n > 0) {
      constexpr uint32_t idesc_q = make_idesc(128, W, kBf16, false, true);
      for (int j = 0; ok && j < n; ++j) {   // dQ += dS_j K'_j
        if (!(ok = warp_wait(ds_full, j & 1, abort_flag, p.status))) break;
        tc_fence_after();
        const uint64_t kb = make_sdesc(sbase + (j % NS) * Cfg::kStageBytes, CB, 1024);
        elected([&] {
          mma_ts_steps<KT / 16, false, 0>(tmem + Cfg::kColDq, tmem + Cfg::kColDs, kb, idesc_q, j > 0 ? 1u : 0u);
          tc_commit(empty(j % NS));   // (before the one that is waited for at the end: a commit
          tc_commit(dq_done);         // that arrived after the CTA had exited would be a fault)
        });
      }
    }
  } else {
    // ===================== softmax gradient, two threads a row =====================
    float delta = halves[rr] + halves[128 + rr];
    // fp16: P, and with it dS, is scaled by 2^e, a part of the exponent
    float up = 1.f, down = 1.f;
    if constexpr (!kBf16) {
      const int e = shift_for(sqrtf(norms[rr] + norms[128 + rr]) * norms[256]);
      up = static_cast<float>(e);
      down = pow2(-e);
    }
    int n_swap = 0;   // exchanges of half sums with the other warp of the rows
    if (half == 0 && h == 0 && lane == 0 && (quarter & 1) == 0) {
      const int2 u = ranges[quarter], v = ranges[quarter + 1];
      p.ranges[static_cast<size_t>(b) * (p.Sq_pad / 64) + unit * 2 + quarter / 2] =
          make_int2(min(u.x, v.x), max(u.y, v.y));
    }
    const uint32_t t_s = tmem + lane_off + half * 32;
    const float c = p.scale_log2, l2e = kBf16 ? l2 : l2 - up;
    for (int j = 0; ok && j < n; ++j) {
      ok = __all_sync(0xffffffffu, mbar_wait(s_full, j & 1, abort_flag, p.status));
      if (!ok) break;
      tc_fence_after();
      uint32_t s[32], g[32];
      tmem_ld32(t_s, s);
      tmem_wait_ld();
      tc_fence_before();   // S is in registers: the next tile's may overwrite it
      __syncwarp();
      if (lane == 0) mbar_arrive(s_free);
      const int tile_k0 = (tile0 + j) * KT, k0 = tile_k0 + half * 32;
      const bool inside = row_hi > 0 && row_lo >= tile_k0 && row_hi <= tile_k0 + KT;
      if (__any_sync(0xffffffffu, k0 < row_lo || k0 + 32 > row_hi)) {
        const uint32_t see = span_bits(row_lo, row_hi, k0);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (!((see >> i) & 1u)) s[i] = __float_as_uint(-INFINITY);
      }
      const uint64_t c2 = f2_pack(c, c), nl2 = f2_pack(-l2e, -l2e);
#pragma unroll
      for (int i = 0; i < 32; i += 2) {   // P, in fp32
        float x0, x1;
        f2_unpack(f2_fma(f2_pack(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), c2, nl2), x0, x1);
        s[i] = __float_as_uint(ex2(x0));
        s[i + 1] = __float_as_uint(ex2(x1));
      }
      ok = __all_sync(0xffffffffu, mbar_wait(dp_full, j & 1, abort_flag, p.status));
      if (!ok) break;
      tc_fence_after();
      tmem_ld32(t_s + KT, g);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(dp_free);
      // A row whose keys all lie in this tile takes D = sum_j P dP from here, in fp32. From the
      // rounded O it is off by half a step of |dO| |O|, which for rows of few keys, the ones with
      // the largest gradients, counts as much as rounding dS does: dQ's and dK's errors at packed
      // documents of 75 to 300 tokens 1.6 to 1.7 times an output's own rounding, 1.4 with this.
      if (__any_sync(0xffffffffu, inside)) {   // the same in the warp of the other half
        uint64_t sum = f2_pack(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 32; i += 2)
          sum = f2_fma(f2_pack(__uint_as_float(s[i]), __uint_as_float(s[i + 1])),
                       f2_pack(__uint_as_float(g[i]), __uint_as_float(g[i + 1])), sum);
        float a0, a1;
        f2_unpack(sum, a0, a1);
        // (buffers in turn: a warp that writes one again has seen the other arrive after reading it)
        float* const buf = halves + ((n_swap + 1) & 1) * 256;
        buf[half * 128 + rr] = a0 + a1;
        __syncwarp();
        if (lane == 0) mbar_arrive(swap(quarter));
        ok = __all_sync(0xffffffffu, mbar_wait(swap(quarter), n_swap & 1, abort_flag, p.status));
        if (!ok) break;
        ++n_swap;
        if (inside) delta = (buf[rr] + buf[128 + rr]) * down;
      }
      const uint64_t nd2 = f2_pack(-delta, -delta);
      uint32_t ds[16];
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const uint64_t x = f2_add(f2_pack(__uint_as_float(g[i]), __uint_as_float(g[i + 1])), nd2);
        float d0, d1;
        f2_unpack(f2_mul(f2_pack(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), x), d0, d1);
        ds[i / 2] = pack2<kBf16>(d0, d1);
      }
      if (j > 0) {   // dQ += dS_(j-1) K'_(j-1) has read the buffer
        ok = __all_sync(0xffffffffu, mbar_wait(dq_done, (j - 1) & 1, abort_flag, p.status));
        if (!ok) break;
        tc_fence_after();
      }
      tmem_st16(tmem + lane_off + Cfg::kColDs + half * 16, ds);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ds_full);
    }
#ifdef FA_WAIT_TEST
    if (ok && wait_test(kWaitSoftmax, p.H)) ok = warp_wait(drain, 0, abort_flag, p.status);
#endif
    if (ok && n > 0)
      ok = __all_sync(0xffffffffu, mbar_wait(dq_done, (n - 1) & 1, abort_flag, p.status));
    if (ok) {
      tc_fence_after();
      if (half == 0) {
        const size_t at = static_cast<size_t>(bh) * p.Sq_pad + row;
        p.lse2[at] = l2 - kShiftP<kBf16>;
        p.delta[at] = delta;
      }
      // through the ring's first stages, which every product has read (or none was loaded into)
      uint8_t* box = smem + (warp - 2) * (W / 64) * kStoreBytes;
#pragma unroll
      for (int cc = 0; cc < W / 64; ++cc) {
        const int col = half * (W / 2) + cc * 32;
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32(tmem + lane_off + Cfg::kColDq + col, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0u;
        }
        if (row - lane < p.mask.Sq)
          store_box<kBf16>(box + cc * kStoreBytes, &p.tm_dq, o, p.scale * down, lane, col, row - lane, h, b);
      }
      // The greatest bound of the rows, for dK and dV of the keys that they see. (In front of the loop it
      // cost 4096 tokens of 32 heads of 64 19 us of 138, packed documents 4 of 55 in warp 0 or 10.)
      if (!kBf16 && warp == 2) {
        float top = 0.f;
        for (int i = lane; i < kTileM; i += 32) top = fmaxf(top, norms[i] + norms[128 + i]);
        const uint32_t bound = __reduce_max_sync(0xffffffffu, __float_as_uint(sqrtf(top) * norms[256]));
        for (int t = tile0 * KT / kTileN + lane; t * kTileN < hi; t += 32)
          atomicMax(reinterpret_cast<unsigned*>(&norms_of(p, bh, t)->ds), bound);
      }
      if (lane == 0) bulk_wait_all();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // A wait ran out, whosever: only now is it known that nothing more is issued. Every copy lands and every
    // MMA finishes before the CTA releases its memory.
    if (threadIdx.x == 0) {
      drain_wait(q_full, 0, p.status);
      drain_wait(do_full, 0, p.status);
      drain_wait(o_full, 0, p.status);
      for (int i = max(0, *issued - NS); i < *issued; ++i) drain_wait(full(i % NS), (i / NS) & 1, p.status);
    }
    if (warp == 1 || warp == 10) {
      const uint32_t bar = warp == 1 ? drain : drain2;
      elected([&] { tc_commit(bar); });
      drain_wait(bar, 0, p.status);
    }
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ----------------------------------------------------------------- dK, dV --
// Transposed products, keys on the tensor-memory lanes, 64 query rows a step:
// S^T = K' Q^T, dP^T = V dO^T, dV += P^T dO, dK' += dS^T Q. Tensor memory: dV [0, d),
// dK' [128, 128 + d + 64), S^T [320, 384), dP^T [384, 448), P^T and dS^T (16-bit)
// [448, 480) and [480, 512).
template <int D>
struct LatDkvCfg {
  static constexpr int kW = D + kRope;
  static constexpr int kKChunks = kW / kChunk, kVChunks = D / kChunk;
  static constexpr int CB = kTileN * 128;               // a chunk of 128 keys
  static constexpr int kRows = 64;                      // query rows a step
  static constexpr int QB = kRows * 128;                // a chunk of 64 query rows
  static constexpr int NS = 3;
  static constexpr int kOffV = kKChunks * CB;           // K' first
  static constexpr int kOffQ = kOffV + kVChunks * CB;   // stages: Q, dO, L, D
  static constexpr int kStageBytes = (kKChunks + kVChunks) * QB;
  static constexpr int kStoreWarp = (2 + D / 32) * kStoreBytes;   // a warp's results on their way out
  static_assert(8 * kStoreWarp <= NS * kStageBytes && kStoreWarp % 1024 == 0, "results in the stages");
  static constexpr int kOffRow = kOffQ + NS * kStageBytes;
  static constexpr int kOffBar = kOffRow + NS * 2 * kRows * 4;
  // kv_full, full[], empty[], s_full, dp_full, s_free, ds_full, kd_done, drain
  static constexpr int kNumBars = 1 + 2 * NS + 6;
  static constexpr int kOffMisc = (kOffBar + kNumBars * 8 + 15) / 16 * 16;   // tmem, abort
  static constexpr int kOffSteps = kOffMisc + 16;       // first and last step, each warp's
  static constexpr int kSmemBytes = kOffSteps + kThreadsB / 32 * 8;
  static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
};

template <int D, bool kBf16>
__global__ void __launch_bounds__(kThreadsB, 1)
    latent_dkv_kernel(const __grid_constant__ LatentBwdParams p) {
  using Cfg = LatDkvCfg<D>;
  constexpr int NS = Cfg::NS, CB = Cfg::CB, QB = Cfg::QB, W = Cfg::kW, R = Cfg::kRows;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.status, kStatusBadLaunch);
    return;
  }
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::kOffMisc + 4);
  volatile int* issued = abort_flag + 1;   // tiles that the producer has asked for
  int2* steps = reinterpret_cast<int2*>(smem + Cfg::kOffSteps);

  const uint32_t kv_full = sbase + Cfg::kOffBar;
  auto full = [&](int s) { return kv_full + 8 * (1 + s); };
  auto empty = [&](int s) { return kv_full + 8 * (1 + NS + s); };
  const uint32_t s_full = kv_full + 8 * (1 + 2 * NS);
  const uint32_t dp_full = s_full + 8, s_free = s_full + 16, ds_full = s_full + 24;
  const uint32_t kd_done = s_full + 32, drain = s_full + 40;

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(warp_id()), 0);
  const int lane = static_cast<int>(lane_id());
  const int BH = p.B * p.H;
  const int kv0 = static_cast<int>(blockIdx.x) / BH * kTileN;   // most query rows first (causal)
  const int bh = static_cast<int>(blockIdx.x) % BH;
  const int b = bh / p.H, h = bh % p.H;
  const int n_steps = p.Sq_pad / R;

  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    mbar_init(s_free, 8);
    mbar_init(ds_full, 8);
    mbar_init(kd_done, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    mbar_arrive_expect_tx(kv_full, (Cfg::kKChunks + Cfg::kVChunks) * CB);
    for (int r = 0; r < 2; ++r) {   // boxes of 64 rows
      const int y = kv0 + r * 64, at = r * (CB / 2);
      for (int c = 0; c < Cfg::kVChunks; ++c) {
        tma_load_4d(sbase + c * CB + at, &p.tm_k, kv_full, c * kChunk, y, h, b);
        tma_load_4d(sbase + Cfg::kOffV + c * CB + at, &p.tm_v, kv_full, c * kChunk, y, h, b);
      }
      tma_load_4d(sbase + Cfg::kVChunks * CB + at, &p.tm_kr, kv_full, 0, y, 0, b);
    }
    tma_prefetch_desc(&p.tm_q);
    tma_prefetch_desc(&p.tm_do);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  // the steps with a row whose span reaches into the tile, and those between them
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the dQ kernel's L, D and ranges
  {
    const int2* ranges = p.ranges + static_cast<size_t>(b) * n_steps;
    int lo = 0x7fffffff, hi = -1;
    for (int i = threadIdx.x; i < n_steps; i += kThreadsB) {
      const int2 r = ranges[i];
      if (r.y > kv0 && r.x < kv0 + kTileN) {
        lo = min(lo, i);
        hi = i;
      }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) steps[warp] = make_int2(lo, hi);
  }
  tc_fence_before();
  __syncthreads();   // tensor memory, barriers, steps
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int i0 = 0x7fffffff, i1 = -1;
#pragma unroll
  for (int w = 0; w < kThreadsB / 32; ++w) {
    i0 = min(i0, steps[w].x);
    i1 = max(i1, steps[w].y);
  }
  if (i1 < 0) i0 = 0;
  const int n = i1 + 1 - i0;   // 0: nothing sees the tile

  if (warp == 0) {
    // ===================== TMA producer =====================
    if (lane == 0) {
      if (n == 0) drain_wait(kv_full, 0, p.status);
      int g = 0;
      bool ok = true;
#ifdef FA_WAIT_TEST
      if (wait_test(kWaitProducer, p.H)) ok = mbar_wait(drain, 0, abort_flag, p.status);
#endif
      for (; ok && g < n; ++g) {
        const int st = g % NS;
        if (g >= NS && !mbar_wait(empty(st), (g / NS - 1) & 1, abort_flag, p.status)) break;
        const uint32_t f = full(st), dst = sbase + Cfg::kOffQ + st * Cfg::kStageBytes;
        const int y = (i0 + g) * R;
        mbar_arrive_expect_tx(f, Cfg::kStageBytes + 2 * R * 4);
        for (int c = 0; c < Cfg::kKChunks; ++c) tma_load_4d(dst + c * QB, &p.tm_q, f, c * kChunk, y, h, b);
        const size_t at = static_cast<size_t>(bh) * p.Sq_pad + y;
        bulk_load(sbase + Cfg::kOffRow + st * (2 * R * 4), p.lse2 + at, R * 4, f);
        for (int c = 0; c < Cfg::kVChunks; ++c)
          tma_load_4d(dst + (Cfg::kKChunks + c) * QB, &p.tm_do, f, c * kChunk, y, h, b);
        bulk_load(sbase + Cfg::kOffRow + st * (2 * R * 4) + R * 4, p.delta + at, R * 4, f);
      }
      *issued = g;
    }
  } else if (warp == 1) {
    // ===================== MMA issuer (the whole warp, one lane of it the MMAs) =====================
    if (n > 0) {
      constexpr uint32_t idesc_s = make_idesc(128, R, kBf16, false, false);
      constexpr uint32_t idesc_v = make_idesc(128, D, kBf16, false, true);
      constexpr uint32_t idesc_k = make_idesc(128, W, kBf16, false, true);
      const uint64_t ka = make_sdesc(sbase, 16, 1024), va = make_sdesc(sbase + Cfg::kOffV, 16, 1024);
      auto wait = [&](uint32_t bar, uint32_t parity) { return warp_wait(bar, parity, abort_flag, p.status); };
      bool ok = wait(kv_full, 0);
#ifdef FA_WAIT_TEST
      if (ok && wait_test(kWaitIssuer, p.H)) ok = wait(drain, 0);   // runs out, as in the dQ kernel
#endif
      auto scores = [&](int g) -> bool {   // S^T and dP^T of step g
        if (!wait(full(g % NS), (g / NS) & 1)) return false;
        if (g > 0 && !wait(s_free, (g - 1) & 1)) return false;
        tc_fence_after();
        const uint32_t st = sbase + Cfg::kOffQ + (g % NS) * Cfg::kStageBytes;
        const uint64_t qb = make_sdesc(st, 16, 1024), ob = make_sdesc(st + Cfg::kKChunks * QB, 16, 1024);
        elected([&] {
          mma_ss_steps<4 * Cfg::kKChunks, true, CB, true, QB>(tmem + 320, ka, qb, idesc_s, 0u);
          tc_commit(s_full);
        });
        elected([&] {
          mma_ss_steps<4 * Cfg::kVChunks, true, CB, true, QB>(tmem + 384, va, ob, idesc_s, 0u);
          tc_commit(dp_full);
        });
        return true;
      };
      if (ok) ok = scores(0);
      for (int g = 0; ok && g < n; ++g) {
        if (g + 1 < n && !(ok = scores(g + 1))) break;
        if (!(ok = wait(ds_full, g & 1))) break;
        tc_fence_after();
        const uint32_t st = sbase + Cfg::kOffQ + (g % NS) * Cfg::kStageBytes;
        const uint64_t qb = make_sdesc(st, QB, 1024), ob = make_sdesc(st + Cfg::kKChunks * QB, QB, 1024);
        elected([&] {
          mma_ts_steps<4, false, 0>(tmem, tmem + 448, ob, idesc_v, g > 0 ? 1u : 0u);
          mma_ts_steps<4, false, 0>(tmem + 128, tmem + 480, qb, idesc_k, g > 0 ? 1u : 0u);
          tc_commit(empty(g % NS));
          tc_commit(kd_done);
        });
      }
    }
  } else {
    // ===================== softmax gradient, two threads a key =====================
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const int key0 = kv0 + quarter * 32;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + lane_off + 320 + half * 32;
    const float c = p.scale_log2;
    float up = 1.f, down = 1.f;   // fp16: dS is scaled, P with it by 2^kShiftP
    if constexpr (!kBf16) {
      if (n > 0) {
        const int e = shift_for(__ldcg(&norms_of(p, bh, kv0 / kTileN)->ds));
        up = pow2(e - kShiftP<kBf16>);
        down = pow2(-e);
      }
    }
    // the span of query column `lane` of this warp's half of step g
    auto span_of = [&](int g) { return p.mask.span(b, (i0 + g) * R + half * 32 + lane); };
    int2 sp = n > 0 ? span_of(0) : make_int2(0, 0);
    bool ok = true;
    for (int g = 0; g < n; ++g) {
      const int st = g % NS;
      uint32_t vis = 0xffffffffu;   // bit e: this lane's key is seen by query column e
      const bool masked = __any_sync(0xffffffffu, sp.x > key0 || sp.y < key0 + 32);
      if (masked)
        vis = transpose_bits(span_bits(sp.x, sp.y, key0), lane);
      if (g + 1 < n) sp = span_of(g + 1);
      ok = __all_sync(0xffffffffu, mbar_wait(full(st), (g / NS) & 1, abort_flag, p.status) &&
                                       mbar_wait(s_full, g & 1, abort_flag, p.status));
      if (!ok) break;
      tc_fence_after();
      const float* l2 = reinterpret_cast<const float*>(smem + Cfg::kOffRow + st * (2 * R * 4)) + half * 32;
      uint32_t s[32];
      tmem_ld32(t_s, s);
      tmem_wait_ld();
      if (masked) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (!((vis >> e) & 1u)) s[e] = __float_as_uint(-INFINITY);
      }
      const uint64_t c2 = f2_pack(c, c);
      uint32_t pk[16], ds[16];
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        const float2 l = *reinterpret_cast<const float2*>(l2 + e);
        float x0, x1;
        f2_unpack(f2_fma(f2_pack(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2, f2_pack(-l.x, -l.y)), x0, x1);
        x0 = ex2(x0);
        x1 = ex2(x1);
        pk[e / 2] = pack2<kBf16>(x0, x1);
        s[e] = __float_as_uint(kBf16 ? x0 : x0 * up);
        s[e + 1] = __float_as_uint(kBf16 ? x1 : x1 * up);
      }
      ok = __all_sync(0xffffffffu, mbar_wait(dp_full, g & 1, abort_flag, p.status));
      if (!ok) break;
      tc_fence_after();
      {
        uint32_t d[32];
        tmem_ld32(t_s + 64, d);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_free);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 dl = *reinterpret_cast<const float2*>(l2 + R + e);
          float d0, d1;
          f2_unpack(f2_mul(f2_pack(__uint_as_float(s[e]), __uint_as_float(s[e + 1])),
                           f2_sub(f2_pack(__uint_as_float(d[e]), __uint_as_float(d[e + 1])), f2_pack(dl.x, dl.y))),
                    d0, d1);
          ds[e / 2] = pack2<kBf16>(d0, d1);
        }
      }
      if (g > 0) {   // the products of step g - 1 have read P^T and dS^T
        ok = __all_sync(0xffffffffu, mbar_wait(kd_done, (g - 1) & 1, abort_flag, p.status));
        if (!ok) break;
        tc_fence_after();
      }
      tmem_st16(tmem + lane_off + 448 + half * 16, pk);
      tmem_st16(tmem + lane_off + 480 + half * 16, ds);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ds_full);
    }
#ifdef FA_WAIT_TEST
    if (ok && wait_test(kWaitSoftmax, p.H)) ok = warp_wait(drain, 0, abort_flag, p.status);
#endif
    if (ok && n > 0)
      ok = __all_sync(0xffffffffu, mbar_wait(kd_done, (n - 1) & 1, abort_flag, p.status));
    if (ok) {
      tc_fence_after();
      // warps 2-5 write dK, warps 6-9 dV, each half the shared part, through the stages of Q and dO
      const CUtensorMap* tm = half == 0 ? &p.tm_dk : &p.tm_dv;
      const float f = half == 0 ? p.scale * down : pow2(-kShiftP<kBf16>);
      uint8_t* box = smem + Cfg::kOffQ + (warp - 2) * Cfg::kStoreWarp;
      auto load = [&](int col, uint32_t (&o)[32]) {
        if (n > 0) {
          tmem_ld32(tmem + lane_off + col, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0u;
        }
      };
      if (key0 < p.mask.Skv) {
        uint32_t o[32];
        load(128 + D + half * 32, o);
        store_box_f32(box, &p.tm_part, o, down, lane, half * 32, key0, h, b);
#pragma unroll
        for (int cc = 0; cc < D / 32; ++cc) {
          load((half == 0 ? 128 : 0) + cc * 32, o);
          store_box<kBf16>(box + (cc + 2) * kStoreBytes, tm, o, f, lane, cc * 32, key0, h, b);
        }
        if (lane == 0) bulk_wait_all();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {   // as in the dQ kernel
    if (threadIdx.x == 0) {
      drain_wait(kv_full, 0, p.status);
      for (int j = max(0, *issued - NS); j < *issued; ++j) drain_wait(full(j % NS), (j / NS) & 1, p.status);
    }
    if (warp == 1) {
      elected([&] { tc_commit(drain); });
      drain_wait(drain, 0, p.status);
    }
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// -------------------------------------------------------------------- dKR --
// dKR_j = scale * the heads' parts, added in head order; 4 elements a thread. Bound by latency:
// the parts are in L2, and eight heads' loads go out together (8 elements a thread with two heads'
// at a time: 7.7 us instead of 4.7 at 2 x 16 heads, 2999 tokens).
constexpr int kDkrElems = 4;

template <bool kBf16>
__global__ void __launch_bounds__(256) latent_dkr_kernel(const __grid_constant__ LatentBwdParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long at = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  const long long tokens = static_cast<long long>(p.B) * p.mask.Skv;
  const long long token = at / (kRope / kDkrElems);
  const int e = static_cast<int>(at % (kRope / kDkrElems)) * kDkrElems;
  if (token >= tokens) return;
  const int b = static_cast<int>(token / p.mask.Skv), j = static_cast<int>(token % p.mask.Skv);
  const size_t step = static_cast<size_t>(p.mask.Skv) * kRope;
  const float* src = p.part + static_cast<size_t>(b) * p.H * step + static_cast<size_t>(j) * kRope + e;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kHeads = 8;
  for (int h = 0; h < p.H; h += kHeads) {
    float4 x[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
      if (h + i < p.H) x[i] = *reinterpret_cast<const float4*>(src + (h + i) * step);
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
      if (h + i < p.H) {
        acc.x += x[i].x; acc.y += x[i].y; acc.z += x[i].z; acc.w += x[i].w;
      }
  }
  uint16_t* dst = static_cast<uint16_t*>(p.dk_rope.data) + b * p.dk_rope.sb + j * p.dk_rope.ss + e;
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<kBf16>(acc.x * p.scale, acc.y * p.scale),
                                              pack2<kBf16>(acc.z * p.scale, acc.w * p.scale));
}

template <int D, bool kBf16>
cudaError_t launch_impl(const LatentBwdParams& p0, cudaStream_t stream) {
  auto dq = latent_dq_kernel<D, kBf16>;
  auto dkv = latent_dkv_kernel<D, kBf16>;
  cudaError_t e = cudaFuncSetAttribute(dq, cudaFuncAttributeMaxDynamicSharedMemorySize, LatDqCfg<D>::kSmemBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(dkv, cudaFuncAttributeMaxDynamicSharedMemorySize, LatDkvCfg<D>::kSmemBytes);
  if (e != cudaSuccess) return e;
  LatentBwdParams p = p0;
  const long long bh = static_cast<long long>(p.B) * p.H;
  if constexpr (!kBf16) {
    e = launch_dependent(latent_norms_kernel<D>, dim3(static_cast<unsigned>(bh * ((p.mask.Skv + kTileN - 1) / kTileN))),
                         dim3(kThreadsN), 0, stream, p);
    if (e != cudaSuccess) return e;
  }
  p.n_units = p.Sq_pad / kTileM;
  e = launch_dependent(dq, dim3(static_cast<unsigned>(bh * p.n_units)), dim3(kThreadsQ),
                       LatDqCfg<D>::kSmemBytes, stream, p);
  if (e != cudaSuccess) return e;
  p.n_units = (p.mask.Skv + kTileN - 1) / kTileN;
  e = launch_dependent(dkv, dim3(static_cast<unsigned>(bh * p.n_units)), dim3(kThreadsB),
                       LatDkvCfg<D>::kSmemBytes, stream, p);
  if (e != cudaSuccess) return e;
  const long long threads = static_cast<long long>(p.B) * p.mask.Skv * (kRope / kDkrElems);
  return launch_dependent(latent_dkr_kernel<kBf16>, dim3(static_cast<unsigned>((threads + 255) / 256)),
                          dim3(256), 0, stream, p);
}

}  // namespace

cudaError_t launch_latent_bwd(const LatentBwdParams& p, int d, bool bf16, cudaStream_t stream) {
  if (d == 128) return bf16 ? launch_impl<128, true>(p, stream) : launch_impl<128, false>(p, stream);
  return bf16 ? launch_impl<64, true>(p, stream) : launch_impl<64, false>(p, stream);
}

}  // namespace fa
