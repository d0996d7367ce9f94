// Forward of latent attention in its expanded form: every head has keys K [Skv, d] and
// values V [Skv, d] (expanded from the tokens' latents by the caller) and all heads of a
// token share a rotated key part KR [Skv, 64], so that
//
//   s_ij = scale (<Q_i[0:d], K_j> + <Q_i[d:], KR_j>),  out = softmax(s) V, LSE_i = log sum_j e^s_ij
//
// under one key range per row. The shared part is loaded beside each head's keys, as a
// third chunk of the key tile; it is never copied out to the heads in memory.
//
// P is rounded to the type of V, whose product takes it as an operand (an output is off by at most half a
// step of P |V| more); sums and maxima are in fp32.
//
// As the forward in fa_fwd.cu: T query tiles of 128 rows per CTA, TMA producer (warp 0),
// MMA issuer (warp 1), four softmax warps a tile with a thread a row, online softmax with
// a lazily moved reference maximum, P over S's columns (T = 2) or beside them (T = 1). Two
// query tiles a CTA at d = 128, which share the keys and values they load, one at d = 64,
// where two CTAs fit an SM.
//
// Bound by a step's chain: 2560 cycles of products for two query tiles of 128 rows by 128 keys,
// 3900 in all, the rest the handing over between products and softmax and the wait for K (the
// ring holds less than two tiles beside 96 KB of queries). 4096 tokens, 32 heads, d = 128, bf16,
// causal: 126 us, 1364 TFLOP/s, 71% of a large product's rate (d = 64: 84.5, 1220); a chunk of 1024 over 8192
// keys, 128 CTAs on 152 SMs: 122 us, 1320. Tried and slower at the latter: two issuing warps (151 instead of
// 134 then), both P V before both S (140), a barrier a chunk of K (128 instead of 122).
#include <type_traits>

#include "fa_latent.h"
#include "latent_store.cuh"
#include "ptx.cuh"
#include "score_mod.cuh"

namespace fa {
namespace {

constexpr float kLn2L = 0.6931471805599453f;
constexpr float kRescaleL = 8.0f;   // the reference maximum moves when exceeded by 2^8

template <int D>
struct LatFwdCfg {
  static constexpr int T = D == 128 ? 2 : 1;            // query tiles a CTA
  static constexpr int kCtasPerSm = 3 - T;
  static constexpr int kThreads = 64 + 128 * T;
  static constexpr bool kSepP = T == 1;                 // P has columns of its own
  static constexpr int kTmemCols = 256 * T;
  static constexpr int kKChunks = D / kChunk + 1;       // key chunks, the shared one last
  static constexpr int kVChunks = D / kChunk;
  static constexpr int kChunkBytes = kTileN * 128;
  static constexpr int kKBytes = kKChunks * kChunkBytes;
  // One ring of chunks for K' and V, in the order in which they are freed: K_0 V_0 K_1 V_1 ..., or
  // K_0 K_1 V_0 K_2 V_1 ... where the next S is formed ahead of P V. (Stages of two K' and one V,
  // the same memory, left every V tile's load uncovered, 2000 of 4800 cycles a step at d = 128.)
  static constexpr int kSlots = T == 2 ? 8 : 5;
  static constexpr int kOffRing = T * kKBytes;          // Q tiles first
  static constexpr int kOffBar = kOffRing + kSlots * kChunkBytes;
  // q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], pv_done[2], s_free, drain
  static constexpr int kNumBars = 1 + 8 + 8;
  static constexpr int kOffMisc = (kOffBar + kNumBars * 8 + 15) / 16 * 16;   // tmem base, abort flag
  static constexpr int kOffSpan = kOffMisc + 16;        // (begin, end) of each softmax warp's rows
  static constexpr int kSmemBytes = kOffSpan + 4 * T * 8;
  static_assert(kSmemBytes <= 232448 && (T == 2 || 2 * (kSmemBytes + 1024) <= 233472), "shared memory");
};

template <int D, bool kBf16>
__global__ void __launch_bounds__(LatFwdCfg<D>::kThreads, LatFwdCfg<D>::kCtasPerSm)
    latent_fwd_kernel(const __grid_constant__ LatentFwdParams p) {
  using Cfg = LatFwdCfg<D>;
  constexpr int T = Cfg::T, NS = Cfg::kSlots, CB = Cfg::kChunkBytes, KC = Cfg::kKChunks, VC = Cfg::kVChunks;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {   // the 128-byte swizzle needs 1024-byte aligned tiles
    if (threadIdx.x == 0) atomicOr(p.status, kStatusBadLaunch);
    return;
  }
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::kOffMisc + 4);
  volatile int* issued = abort_flag + 1;   // K and V tiles that the producer has asked for
  int2* ranges = reinterpret_cast<int2*>(smem + Cfg::kOffSpan);

  const uint32_t q_full = sbase + Cfg::kOffBar;
  auto bars = [&](int first) { return [=](int i) { return q_full + 8 * (first + i); }; };
  const auto k_full = bars(1), k_empty = bars(3), v_full = bars(5), v_empty = bars(7);   // by tile % 2
  const auto s_full = bars(9), p_full = bars(11), pv_done = bars(13);
  const uint32_t s_free = q_full + 8 * 15, drain = s_free + 8;

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(warp_id()), 0);
  const int lane = static_cast<int>(lane_id());
  // last rows first: the heaviest under the causal mask. (Under other masks the order says nothing about
  // what a tile costs: padded rows come first, and documents in any order.)
  const int BH = p.B * p.H;
  const int unit = p.n_units - 1 - static_cast<int>(blockIdx.x) / BH;
  const int bh = static_cast<int>(blockIdx.x) % BH;
  const int b = bh / p.H, h = bh % p.H;
  const int q0 = unit * T * kTileM;

  int row_lo = 0, row_hi = 0;   // a softmax thread's row
  if (warp >= 2) {
    // programmatic dependent of the kernel before: waited for in front of the first access
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int t = (warp - 2) / 4;
    const int2 s = p.mask.span(b, q0 + t * kTileM + (warp & 3) * 32 + lane);
    row_lo = s.x;
    row_hi = s.y;
    const int lo = __reduce_min_sync(0xffffffffu, row_hi > 0 ? row_lo : 0x7fffffff);
    const int hi = __reduce_max_sync(0xffffffffu, row_hi);
    if (lane == 0) ranges[t * 4 + (warp & 3)] = make_int2(lo, hi);
  }
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full(i), 1);
      mbar_init(k_empty(i), 1);
      mbar_init(v_full(i), 1);
      mbar_init(v_empty(i), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(s_full(t), 1);
      mbar_init(p_full(t), 4);   // one arrival per softmax warp
      mbar_init(pv_done(t), 1);
    }
    mbar_init(s_free, 4);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    // the queries are on their way while the spans are read (rows past Sq come as zeros)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    mbar_arrive_expect_tx(q_full, T * Cfg::kKBytes);
    for (int t = 0; t < T; ++t)
      for (int c = 0; c < Cfg::kKChunks; ++c)
        tma_load_4d(sbase + t * Cfg::kKBytes + c * CB, &p.tm_q, q_full, c * kChunk, q0 + t * kTileM, h, b);
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_kr);
    tma_prefetch_desc(&p.tm_v);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), Cfg::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (gridDim.x <= 152) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // key tiles [tile0, tile0 + n_load); query tile t takes those from first[t] to last[t]
  int first[2] = {0, 0}, last[2] = {0, 0};
  int tile0 = 0x7fffffff, tile1 = 0;
#pragma unroll
  for (int t = 0; t < T; ++t) {
    int lo = 0x7fffffff, hi = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      lo = min(lo, ranges[t * 4 + w].x);
      hi = max(hi, ranges[t * 4 + w].y);
    }
    if (hi > 0) {
      first[t] = lo / kTileN;
      last[t] = (hi + kTileN - 1) / kTileN;
      tile0 = min(tile0, first[t]);
      tile1 = max(tile1, last[t]);
    }
  }
  if (tile1 == 0) tile0 = 0;
  const int n_load = tile1 - tile0;
#pragma unroll
  for (int t = 0; t < T; ++t) {
    if (last[t] == 0) first[t] = last[t] = 0;   // sees nothing
    else {
      first[t] -= tile0;
      last[t] -= tile0;
    }
  }

  if (warp == 0) {
    // ===================== TMA producer =====================
    if (lane == 0) {
      if (n_load == 0) drain_wait(q_full, 0, p.status);   // no product waits for the queries
      // units of the ring, in order: K or V of a tile
      auto is_k = [](int u) { return Cfg::kSepP ? u == 0 || u % 2 == 1 : u % 2 == 0; };
      auto tile_of = [&](int u) { return Cfg::kSepP ? (u == 0 ? 0 : is_k(u) ? (u + 1) / 2 : u / 2 - 1) : u / 2; };
      const int n_units = 2 * n_load + (Cfg::kSepP ? 1 : 0);   // (with a K past the last tile, skipped)
      // At most three units are out at once: each pair of barriers serves every other tile, and a
      // copy announced on a barrier whose phase still waits for bytes of the tile two before it would
      // be a second arrival of a phase that expects one. (The slots alone do not see to that where
      // the last tiles' V follow one another.)
      int slot = 0, used = 0, held = 0, oldest = 0, jk = 0, jv = 0;   // jk, jv: K and V tiles issued
      bool ok = true;
#ifdef FA_WAIT_TEST
      if (wait_test(kWaitProducer, p.H)) ok = mbar_wait(drain, 0, abort_flag, p.status);
#endif
      for (int u = 0; ok && u < n_units; ++u) {
        const int j = tile_of(u), n = is_k(u) ? KC : VC;
        if (j >= n_load) continue;
        for (; used + n > NS || held == 3; ++oldest, --held) {
          const int o = tile_of(oldest);
          if (!(ok = mbar_wait(is_k(oldest) ? k_empty(o & 1) : v_empty(o & 1), (o >> 1) & 1, abort_flag, p.status))) break;
          used -= is_k(oldest) ? KC : VC;
        }
        if (!ok) break;
        const uint32_t f = is_k(u) ? k_full(j & 1) : v_full(j & 1);
        const int y = (tile0 + j) * kTileN;
        mbar_arrive_expect_tx(f, n * CB);
        for (int c = 0; c < n; ++c) {
          const uint32_t dst = sbase + Cfg::kOffRing + slot * CB;
          if (!is_k(u)) tma_load_4d(dst, &p.tm_v, f, c * kChunk, y, h, b);
          else if (c < VC) tma_load_4d(dst, &p.tm_k, f, c * kChunk, y, h, b);
          else tma_load_4d(dst, &p.tm_kr, f, 0, y, 0, b);
          slot = slot + 1 == NS ? 0 : slot + 1;
        }
        // The next tile's on their way to L2, while their slots are in use: at d = 128 the ring holds
        // less than two tiles and K is waited for in every step (chunk of 1024 over 8192 keys 126 ->
        // 122 us, 4096 tokens, 32 heads 131 -> 125).
        if (T == 2 && j + 1 < n_load) {
          for (int c = 0; c < n; ++c) {
            if (!is_k(u)) tma_prefetch_l2_4d(&p.tm_v, c * kChunk, y + kTileN, h, b);
            else if (c < VC) tma_prefetch_l2_4d(&p.tm_k, c * kChunk, y + kTileN, h, b);
            else tma_prefetch_l2_4d(&p.tm_kr, 0, y + kTileN, 0, b);
          }
        }
        used += n;
        ++held;
        if (is_k(u)) ++jk;
        else ++jv;
      }
      issued[0] = jk;
      issued[1] = jv;
    }
  } else if (warp == 1) {
    // ===================== MMA issuer (the whole warp, one lane of it the MMAs) =====================
    if (n_load > 0) {
      constexpr uint32_t idesc_qk = make_idesc(128, kTileN, kBf16, false, false);
      constexpr uint32_t idesc_pv = make_idesc(128, D, kBf16, false, true);
      auto wait = [&](uint32_t bar, uint32_t parity) { return warp_wait(bar, parity, abort_flag, p.status); };
      bool ok = wait(q_full, 0);
#ifdef FA_WAIT_TEST
      // wait-limit test build: nothing completes this phase before the abort
      // path's own commit, so the wait runs out
      if (ok && wait_test(kWaitIssuer, p.H)) ok = wait(drain, 0);
#endif
      auto active = [&](int t, int j) { return j >= first[t] && j < last[t]; };
      // the ring's slots of the K tile and the V tile in turn
      int next_slot = 0, k_slot[KC], v_slot[VC];
      auto take = [&](int (&slots)[KC]) {
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          slots[c] = next_slot;
          next_slot = next_slot + 1 == NS ? 0 : next_slot + 1;
        }
      };
      auto take_v = [&]() {
#pragma unroll
        for (int c = 0; c < VC; ++c) {
          v_slot[c] = next_slot;
          next_slot = next_slot + 1 == NS ? 0 : next_slot + 1;
        }
      };
      const uint64_t ring = make_sdesc(sbase + Cfg::kOffRing, 16, 1024);   // K-major
      const uint64_t ring_mn = make_sdesc(sbase + Cfg::kOffRing, CB, 1024);
      constexpr uint64_t kSlot = CB >> 4;
      auto issue_qk = [&](int t) {   // S_t = Q_t K^T
        const uint64_t qa = make_sdesc(sbase + t * Cfg::kKBytes, 16, 1024);
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          const uint64_t kb = ring + k_slot[c] * kSlot;
          elected([&] {
            mma_ss_steps<4, true, CB, true, CB>(tmem + t * 128, qa + c * kSlot, kb, idesc_qk, c > 0 ? 1u : 0u);
            if (c == KC - 1) tc_commit(s_full(t));
          });
        }
      };
      auto issue_pv = [&](int t, bool more) {   // O_t (+)= P_t V
        const uint32_t o_t = tmem + 128 * T + t * 128;
        const uint32_t p_t = Cfg::kSepP ? o_t + D : tmem + t * 128;
        if (VC == 2 && v_slot[VC - 1] == 0) {   // the tile's chunks are not next to each other
          const uint64_t v0 = ring_mn + v_slot[0] * kSlot, v1 = ring_mn;
          elected([&] {
            mma_ts_steps<8, false, 0>(o_t, p_t, v0, make_idesc(128, 64, kBf16, false, true), more ? 1u : 0u);
            mma_ts_steps<8, false, 0>(o_t + 64, p_t, v1, make_idesc(128, 64, kBf16, false, true), more ? 1u : 0u);
            tc_commit(pv_done(t));
          });
        } else {
          const uint64_t vb = ring_mn + v_slot[0] * kSlot;
          elected([&] {
            mma_ts_steps<8, false, 0>(o_t, p_t, vb, idesc_pv, more ? 1u : 0u);
            tc_commit(pv_done(t));
          });
        }
      };
      // Slots are freed for the loads still to come only: a commit that arrived after the CTA had
      // exited would be a fault. (A tile that no row of either query tile wants is waited for all
      // the same, so that none is in flight at the end.)
      auto commit = [&](uint32_t bar) {
        elected([&] { tc_commit(bar); });
      };
      if (ok) ok = wait(k_full(0), 0);
      if (ok) {
        tc_fence_after();
        take(k_slot);
#pragma unroll
        for (int t = 0; t < T; ++t)
          if (active(t, 0)) issue_qk(t);
        if (n_load > 1) commit(k_empty(0));
      }
      for (int j = 0; ok && j < n_load; ++j) {
        const bool last_tile = j + 1 == n_load;
        if constexpr (Cfg::kSepP) {   // S of the next tile once S has been read, then P V
          const uint32_t n = j - first[0];
          if (!last_tile) {
            take(k_slot);
            if (!(ok = wait(k_full((j + 1) & 1), ((j + 1) >> 1) & 1) && wait(s_free, n & 1))) break;
            tc_fence_after();
            issue_qk(0);
            if (j + 2 < n_load) commit(k_empty((j + 1) & 1));
          }
          take_v();
          if (!(ok = wait(v_full(j & 1), (j >> 1) & 1) && wait(p_full(0), n & 1))) break;
          tc_fence_after();
          issue_pv(0, n > 0);
          if (!last_tile) commit(v_empty(j & 1));
        } else {   // P_t V, then S_t of the next tile over P_t, for either query tile in turn
          take_v();
          if (!(ok = wait(v_full(j & 1), (j >> 1) & 1))) break;
          bool k_seen = last_tile;
#pragma unroll
          for (int t = 0; t < T; ++t) {
            const bool now = active(t, j), then = active(t, j + 1);
            const uint32_t n = j - first[t];   // tiles of this query tile before j
            if (now) {
              if (!(ok = wait(p_full(t), n & 1))) break;
              tc_fence_after();
              issue_pv(t, n > 0);
            }
            // (a commit covers all that was issued before it: V's comes before the next S)
            if (t == T - 1 && !last_tile) commit(v_empty(j & 1));
            if (!k_seen && (t == T - 1 || then)) {
              take(k_slot);
              if (!(ok = wait(k_full((j + 1) & 1), ((j + 1) >> 1) & 1))) break;
              k_seen = true;
            }
            if (then) {
              if (now && !(ok = wait(pv_done(t), n & 1))) break;   // P_t V has read P_t
              tc_fence_after();
              issue_qk(t);
            }
          }
          if (!ok) break;
          if (j + 2 < n_load) commit(k_empty((j + 1) & 1));
        }
      }
    }
  } else {
    // ===================== softmax / correction / epilogue =====================
    const int t = (warp - 2) / 4;
    const int quarter = warp & 3;               // TMEM lane quarter of this warp
    const int row = q0 + t * kTileM + quarter * 32 + lane;
    const int n = last[t] - first[t];
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_tmem = tmem + lane_off + t * 128;
    const uint32_t o_tmem = tmem + lane_off + 128 * T + t * 128;
    const uint32_t p_tmem = Cfg::kSepP ? o_tmem + D : s_tmem;
    const float c = p.scale_log2;
    float m_ref = -INFINITY;   // reference max, scaled log2 domain
    float l = 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      ok = __all_sync(0xffffffffu, mbar_wait(s_full(t), j & 1, abort_flag, p.status));
      if (!ok) break;
      tc_fence_after();
      float s[kTileN];
      {
        uint32_t raw[kTileN];
#pragma unroll
        for (int cc = 0; cc < kTileN / 32; ++cc)
          tmem_ld32(s_tmem + cc * 32, *reinterpret_cast<uint32_t(*)[32]>(raw + cc * 32));
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < kTileN; ++i) s[i] = __uint_as_float(raw[i]);
      }
      if constexpr (Cfg::kSepP) {   // the issuer may overwrite S with the next tile's
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_free);
      }
      const int kv0 = (tile0 + first[t] + j) * kTileN;
      // (branches in front of tensor-memory instructions are the warp's, which have to find it whole)
      if (__any_sync(0xffffffffu, kv0 < row_lo || kv0 + kTileN > row_hi)) {
#pragma unroll
        for (int w = 0; w < kTileN / 32; ++w) {
          const uint32_t see = span_bits(row_lo, row_hi, kv0 + w * 32);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!((see >> i) & 1u)) s[w * 32 + i] = -INFINITY;
        }
      }
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int i = 4; i + 8 <= kTileN; i += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = fmax3(mx[e], s[i + e], s[i + 4 + e]);
#pragma unroll
      for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], s[kTileN - 4 + e]);
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
      const float m_new = top > m_ref + kRescaleL ? top : m_ref;
      const float m_use = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = ex2(m_ref - m_use);   // 0 when m_ref = -inf
      const bool moved = m_new != m_ref;
      m_ref = m_new;

      const uint64_t c2 = f2_pack(c, c), nm2 = f2_pack(-m_use, -m_use);
      uint64_t sum0 = f2_pack(0.f, 0.f), sum1 = sum0;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        uint32_t pk[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float x0, x1;
          f2_unpack(f2_fma(f2_pack(s[w * 64 + 2 * i], s[w * 64 + 2 * i + 1]), c2, nm2), x0, x1);
          const float p0 = ex2(x0), p1 = ex2(x1);
          if (i & 1) sum1 = f2_add(sum1, f2_pack(p0, p1));
          else sum0 = f2_add(sum0, f2_pack(p0, p1));
          pk[i] = pack2<kBf16>(p0, p1);
        }
        if (Cfg::kSepP && w == 0 && j > 0) {
          // P_(j-1) V_(j-1) has read the P buffer (and O may be rescaled)
          ok = __all_sync(0xffffffffu, mbar_wait(pv_done(t), (j - 1) & 1, abort_flag, p.status));
          tc_fence_after();
        }
        tmem_st32(p_tmem + w * 32, pk);
      }
      if (!ok) break;
      float a0, a1, a2, a3;
      f2_unpack(sum0, a0, a1);
      f2_unpack(sum1, a2, a3);
      l = l * alpha + ((a0 + a1) + (a2 + a3));

      // O <- alpha O for rows whose reference max moved (the first P V overwrites O)
      if (j > 0 && __any_sync(0xffffffffu, moved)) {
        if constexpr (!Cfg::kSepP) {
          ok = __all_sync(0xffffffffu, mbar_wait(pv_done(t), (j - 1) & 1, abort_flag, p.status));
          if (!ok) break;
          tc_fence_after();
        }
        const float a = moved ? alpha : 1.f;
#pragma unroll
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t o[32];
          tmem_ld32(o_tmem + cc * 32, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
          tmem_st32(o_tmem + cc * 32, o);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full(t));
    }

#ifdef FA_WAIT_TEST
    if (ok && wait_test(kWaitSoftmax, p.H)) ok = warp_wait(drain, 0, abort_flag, p.status);
#endif
    if (ok && n > 0)
      ok = __all_sync(0xffffffffu, mbar_wait(pv_done(t), (n - 1) & 1, abort_flag, p.status));
    // (results leave through the query tile's own memory)
    if (ok && n == 0) ok = __all_sync(0xffffffffu, mbar_wait(q_full, 0, abort_flag, p.status));
    if (ok) {
      tc_fence_after();
      // a row that sees nothing has O = 0, l = 0 (and only its own span says so: a row of NaN
      // or -infinite scores has no sum either)
      const bool none = row_hi == 0;
      const float inv_l = none ? 0.f : 1.f / l;
      uint8_t* box = smem + t * Cfg::kKBytes + quarter * (D / 32) * kStoreBytes;
#pragma unroll
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32(o_tmem + cc * 32, o);
          tmem_wait_ld();
        }
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (none) o[i] = 0u;
        if (row - lane < p.mask.Sq)
          store_box<kBf16>(box + cc * kStoreBytes, &p.tm_out, o, inv_l, lane, cc * 32, row - lane, h, b);
      }
      if (row < p.mask.Sq)
        p.lse[static_cast<size_t>(bh) * p.mask.Sq + row] =
            none ? -INFINITY : (m_ref + __log2f(l)) * kLn2L;
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
      for (int j = max(0, issued[0] - 2); j < issued[0]; ++j) drain_wait(k_full(j & 1), (j >> 1) & 1, p.status);
      for (int j = max(0, issued[1] - 2); j < issued[1]; ++j) drain_wait(v_full(j & 1), (j >> 1) & 1, p.status);
    }
    if (warp == 1) {
      elected([&] { tc_commit(drain); });
      drain_wait(drain, 0, p.status);
    }
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::kTmemCols);
  }
}

template <int D, bool kBf16>
cudaError_t launch_impl(const LatentFwdParams& p0, cudaStream_t stream) {
  using Cfg = LatFwdCfg<D>;
  auto kernel = latent_fwd_kernel<D, kBf16>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmemBytes);
  if (e != cudaSuccess) return e;
  LatentFwdParams p = p0;
  p.n_units = (p.mask.Sq + Cfg::T * kTileM - 1) / (Cfg::T * kTileM);
  const unsigned grid = static_cast<unsigned>(static_cast<long long>(p.B) * p.H * p.n_units);   // < 2^31
  return launch_dependent(kernel, dim3(grid), dim3(Cfg::kThreads), Cfg::kSmemBytes, stream, p);
}

}  // namespace

cudaError_t launch_latent_fwd(const LatentFwdParams& p, int d, bool bf16, cudaStream_t stream) {
  if (d == 128) return bf16 ? launch_impl<128, true>(p, stream) : launch_impl<128, false>(p, stream);
  return bf16 ? launch_impl<64, true>(p, stream) : launch_impl<64, false>(p, stream);
}

}  // namespace fa
