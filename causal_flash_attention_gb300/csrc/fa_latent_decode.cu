// Latent attention in its absorbed form: one or a few new tokens per sequence over a paged
// cache that holds one row a token, [latent (rank) | rotated key part (64)], which is key
// and, its first rank elements, value of every head. For row r = (head, token) of a
// sequence, with q_r absorbed into the latent's space by the caller,
//
//   s_rj = scale <q_r, c_j>,  out_r = sum_j softmax(s)_rj c_j[0:rank],  LSE_r = log sum_j e^s_rj
//
// over the keys that the row sees: up to its own token's, in a window or not, or before the
// new tokens all and among them those of a bit mask (a tree of drafted tokens).
//
// Work is shared out as in the ragged decode (ragged_shares.cuh): the list of 64-key tiles
// of all sequences is cut into even shares. The rows of a sequence (H * Sq) are cut into
// groups of up to 64; the CTAs of a share's groups stand next to each other in the grid,
// so that they read the same tiles at the same time, from L2 all but the first.
//
// A tile is loaded once and serves both products:
//   S = Q C^T    rows x 64 keys, M = 64: Q and the tile K-major in shared memory
//   O^T += C^T P rank x rows, M = 128, rank / 128 products: the tile again, MN-major, and P,
//                in the type of the cache, as the B operand
// O stands transposed in tensor memory because rows are the short side (rank / 128 * rows
// columns: 256 at rank 512 with 64 rows; the other way around it would take all 512). The
// tile goes through a ring of 16 KB pairs of 64-column chunks, each freed as soon as its
// own part of O^T is issued.
//
// Warp roles (192 threads): warp 0 TMA producer, warp 1 MMA issuer, warps 2-5 softmax (a
// thread a row: lanes 0-15 of a warp hold rows 16 w .. 16 w + 15, the M = 64 layout) and
// O^T (all lanes).
#include <algorithm>
#include <type_traits>

#include "fa_latent.h"
#include "ptx.cuh"
#include "ragged_shares.cuh"
#include "score_mod.cuh"

namespace fa {
namespace {

constexpr int kTile = LatentPagedParams::kTileKeys;
constexpr float kLn2D = 0.6931471805599453f;
constexpr float kRescaleD = 8.0f;   // the reference maximum moves when exceeded by 2^8

template <int RANK, int NR>
struct LatDecCfg {
  static constexpr int kPairs = RANK / 128;             // pairs of 64-column chunks of a latent
  static constexpr int kChunks = RANK / kChunk + 1;
  static constexpr int CB = kTile * 128;                // bytes of a chunk of a tile
  static constexpr int kQB = NR * 128;                  // bytes of a chunk of the queries
  // the ring: pairs, and the rotated parts in one of their own
  static constexpr int NX = NR == 64 && RANK == 512 ? 2 : 3;
  static constexpr int kP = NR * 128;                   // P: [rows][64 keys]
  static constexpr int kFree = 232448 - 2048 - kChunks * kQB - kP - NX * CB;
  static constexpr int NP = kFree / (2 * CB) < 12 ? kFree / (2 * CB) : 12;
  static_assert(NP >= 2 * kPairs, "two tiles in flight");
  // queries first: a product of M = 64 reads 64 rows of a chunk, whatever stands behind its NR
  static constexpr int kOffP = kChunks * kQB;
  static constexpr int kOffX = kOffP + kP;
  static constexpr int kOffC = kOffX + NX * CB;
  static constexpr int kOffBar = kOffC + NP * 2 * CB;
  // full[NP], empty[NP], x_full[NX], x_empty[NX], q_ready, s_full[2], p_full, pv_done, drain
  static constexpr int kNumBars = 2 * NP + 2 * NX + 6;
  static constexpr int kOffMisc = (kOffBar + kNumBars * 8 + 15) / 16 * 16;   // tmem, abort
  static constexpr int kOffScan = kOffMisc + 16;        // find_share
  static constexpr int kOffRow = kOffScan + 32;         // [64] factor, [64] log2-sum of a row
  static constexpr int kSmemBytes = kOffRow + 512;
  static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
};

__device__ __forceinline__ void drain_wait_d(uint32_t bar, uint32_t parity, int* status) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > kDrainLimitCycles) {
      atomicOr(status, kStatusWaitTimeout);
      return;
    }
  }
}

// Position in a ring of N slots, and the parity of its use.
template <int N>
struct Ring {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      parity ^= 1u;
    }
  }
};

// Bits of a 64-key tile from key kv0 that a row with tree mask `w` sees: all keys before the
// new tokens (the first at key `first`), of those token t by bit t.
__device__ __forceinline__ uint64_t tree_bits(uint64_t w, int first, int kv0) {
  const int t0 = kv0 - first;   // token of the tile's first key
  if (t0 >= 64) return 0;
  if (t0 >= 0) return w >> t0;
  if (t0 <= -64) return ~0ull;
  return (w << -t0) | ((1ull << -t0) - 1);
}

template <int RANK, int NR, bool kBf16>
__global__ void __launch_bounds__(kRaggedThreads, 1)
    latent_paged_kernel(const __grid_constant__ LatentPagedParams p) {
  using Cfg = LatDecCfg<RANK, NR>;
  using Elem = typename std::conditional<kBf16, __nv_bfloat16, __half>::type;
  constexpr int NP = Cfg::NP, NX = Cfg::NX, CB = Cfg::CB, kPairs = Cfg::kPairs;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {   // the 128-byte swizzle needs 1024-byte aligned tiles
    if (threadIdx.x == 0) atomicOr(p.status, kStatusBadLaunch);
    return;
  }
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::kOffMisc + 4);
  float* row_f = reinterpret_cast<float*>(smem + Cfg::kOffRow);
  float* row_lse = row_f + 64;

  const Bars full{sbase + Cfg::kOffBar}, empty{full(NP)}, x_full{empty(NP)}, x_empty{x_full(NX)};
  const uint32_t q_ready = x_empty(NX);
  const Bars s_full{q_ready + 8};
  const uint32_t p_full = s_full(2), pv_done = p_full + 8, drain = p_full + 16;

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(warp_id()), 0);
  const int lane = static_cast<int>(lane_id());
  const int share_id = static_cast<int>(blockIdx.x) / p.groups;
  // this CTA's rows of a sequence: from token s0 of head h0 on
  const int group = static_cast<int>(blockIdx.x) % p.groups;
  const int per_head = (p.Sq + p.group_tokens - 1) / p.group_tokens;   // groups a head is cut into
  const int h0 = group / per_head * p.group_heads, s0 = group % per_head * p.group_tokens;
  const int row0 = h0 * p.Sq + s0;
  const int rows = min(p.group_heads, p.H - h0) * min(p.group_tokens, p.Sq - s0);

  if (threadIdx.x == 0) {
    for (int s = 0; s < NP; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int s = 0; s < NX; ++s) {
      mbar_init(x_full(s), 1);
      mbar_init(x_empty(s), 1);
    }
    mbar_init(q_ready, 1);   // once a segment
    mbar_init(s_full(0), 1);
    mbar_init(s_full(1), 1);
    mbar_init(p_full, 4);
    mbar_init(pv_done, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tm);
    tma_prefetch_desc(&p.tm_q);
  }
  // tensor memory: S at columns 0 and 64, O^T part m at 128 + m NR
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  const Share share = find_share(p, share_id, reinterpret_cast<int*>(smem + Cfg::kOffScan));
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // the merge kernel may be scheduled now; it waits for this grid's completion
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  Segments seg(p, share);

  if (warp == 0) {
    // ===================== TMA producer =====================
    // Lane i reads the table entry of box i of a tile and issues its copies. A box past the
    // sequence or before every row's window, or an entry outside [0, num_blocks), is loaded
    // from an out-of-range row, which the copy fills with zeros.
    const int n_boxes = kTile / p.box_rows;
    Ring<NP> at;
    Ring<NX> xt;
    int n_p = 0, n_x = 0;   // pairs and rotated parts issued
    bool stop = false;
    while (!stop && seg.next(p)) {
      const int* table = p.block_table + static_cast<size_t>(seg.b) * p.max_blocks;
      for (int j = 0; j < seg.n && !stop; ++j) {
        const int key = (seg.tile0 + j) * kTile + lane * p.box_rows;
        int pb = -1;
        if (lane < n_boxes && key < seg.keys.len && key + p.box_rows > seg.keys.first)
          pb = table[key / p.block_size];
        const bool in_range = pb >= 0 && pb < p.num_blocks;
        const int y = in_range ? key % p.block_size : p.block_size;
        const int z = in_range ? pb : 0;
        const uint32_t box = lane * p.box_rows * 128;
        for (int m = 0; m <= kPairs && !stop; ++m) {   // the rotated part goes with the last
          const bool is_x = m == kPairs;
          const uint32_t f = is_x ? x_full(xt.slot) : full(at.slot);
          int fail = 0;
          if (lane == 0) {
            const bool wait = is_x ? n_x >= NX : n_p >= NP;
            if (wait && !mbar_wait(is_x ? x_empty(xt.slot) : empty(at.slot), (is_x ? xt.parity : at.parity) ^ 1u,
                                   abort_flag, p.status))
              fail = 1;
            else
              mbar_arrive_expect_tx(f, is_x ? CB : 2 * CB);
          }
          if ((stop = __shfl_sync(0xffffffffu, fail, 0))) break;
          if (is_x) {
            if (lane < n_boxes) tma_load_3d(sbase + Cfg::kOffX + xt.slot * CB + box, &p.tm, f, RANK, y, z);
            xt.next();
            ++n_x;
          } else {
            if (lane < n_boxes) {
              const uint32_t dst = sbase + Cfg::kOffC + at.slot * 2 * CB + box;
              tma_load_3d(dst, &p.tm, f, m * 128, y, z);
              tma_load_3d(dst + CB, &p.tm, f, m * 128 + kChunk, y, z);
            }
            at.next();
            ++n_p;
          }
        }
      }
    }
    if (lane == 0 && *abort_flag) {
      // let every copy already issued land before the CTA releases its memory
      for (int i = max(0, n_p - NP); i < n_p; ++i) drain_wait_d(full(i % NP), (i / NP) & 1, p.status);
      for (int i = max(0, n_x - NX); i < n_x; ++i) drain_wait_d(x_full(i % NX), (i / NX) & 1, p.status);
    }
  } else if (warp == 1) {
    // ===================== MMA issuer (the whole warp, one lane of it the MMAs) =====================
    // Two streams of work, whichever is ready first: tile gs's S, once
    // it has landed, and tile go's O^T once its P is there. (In a fixed order, S of the next tile
    // first, a late load held up O^T, which frees the ring for the load after it.)
    constexpr uint32_t idesc_s = make_idesc(64, kTile, kBf16, false, false);
    constexpr uint32_t idesc_o = make_idesc(128, NR, kBf16, true, false);
    TileWalk walk{seg};
    Ring<NP> at_s, at_o;
    Ring<NX> xt;
    int n_seg = 0;      // segments whose queries have landed
    int gs = 0, go = 0; // the next tile of either stream
    bool begins = false;   // tile gs is its segment's first, and its queries have landed
    bool first_of[2] = {false, false};   // the same of the tiles whose S is formed, by g % 2
    const uint64_t qa = make_sdesc(sbase, 16, 1024);
    const uint64_t pb = make_sdesc(sbase + Cfg::kOffP, 16, 1024);
    auto ready = [](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_test(bar, parity)); };
    // (votes make what was loaded the same in every lane for the compiler too, and with it the
    // control flow and the descriptors: elect_one)
    bool first_s = false;
    auto next = [&]() {
      const bool more = __all_sync(0xffffffffu, walk.next(p));
      first_s = __all_sync(0xffffffffu, walk.first);
      return more;
    };
    bool ok = true, have = next();
#ifdef FA_WAIT_TEST
    // wait-limit test build: nothing completes this phase before the abort
    // path's own commit, so the wait runs out
    if (have) ok = warp_wait(drain, 0, abort_flag, p.status);
#endif
    long long idle_since = clock64();
    uint32_t idle = 0;
    while (ok && (have || go < gs)) {
      bool worked = false;
      // S_gs goes over S_(gs-2), which has been read when P_(gs-2) is there
      if (have && gs <= go + 1) {
        if (first_s && ready(q_ready, n_seg & 1)) {
          ++n_seg;
          first_s = false;
          begins = true;
        }
        // the tile's last part has landed, and so, soon or already, have the others
        if (!first_s && ready(x_full(xt.slot), xt.parity)) {
          first_of[gs & 1] = begins;
          begins = false;
          const uint32_t d = tmem + (gs & 1) * 64;
#pragma unroll
          for (int m = 0; m < kPairs; ++m) {
            if (!(ok = warp_wait(full(at_s.slot), at_s.parity, abort_flag, p.status))) break;
            tc_fence_after();
            const uint64_t cb = make_sdesc(sbase + Cfg::kOffC + at_s.slot * 2 * CB, 16, 1024);
            if (elect_one())
              mma_ss_steps<8, true, Cfg::kQB, true, CB>(d, qa + 2 * m * (Cfg::kQB >> 4), cb, idesc_s, m > 0 ? 1u : 0u);
            at_s.next();
          }
          if (!ok) break;
          const uint64_t xb = make_sdesc(sbase + Cfg::kOffX + xt.slot * CB, 16, 1024);
          if (elect_one()) {
            mma_ss_steps<4, true, Cfg::kQB, true, CB>(d, qa + 2 * kPairs * (Cfg::kQB >> 4), xb, idesc_s, 1u);
            tc_commit(s_full(gs & 1));
            tc_commit(x_empty(xt.slot));
          }
          xt.next();
          ++gs;
          have = next();
          worked = true;
        }
      }
      if (go < gs && ready(p_full, go & 1)) {
        tc_fence_after();
        const uint32_t more = first_of[go & 1] ? 0u : 1u, o_t = tmem + 128;
#pragma unroll
        for (int m = 0; m < kPairs; ++m) {   // O^T part m (+)= C_m^T P
          const uint64_t ca = make_sdesc(sbase + Cfg::kOffC + at_o.slot * 2 * CB, CB, 1024);
          if (elect_one()) {
            mma_ss_steps<kTile / 16, false, 0, true, Cfg::kP>(o_t + m * NR, ca, pb, idesc_o, more);
            tc_commit(empty(at_o.slot));
            if (m == kPairs - 1) tc_commit(pv_done);
          }
          at_o.next();
        }
        ++go;
        worked = true;
      }
      if (worked) {
        idle = 0;
      } else if ((++idle & 15u) == 0) {   // as mbar_wait
        if (idle == 16) idle_since = clock64();
        bool stop = false;
        if (lane == 0) {
          stop = *abort_flag;
          if (!stop && clock64() - idle_since > kWaitLimitCycles) {
            *abort_flag = 1;
            atomicOr(p.status, kStatusWaitTimeout);
            stop = true;
          }
        }
        ok = !__any_sync(0xffffffffu, stop);
      }
    }
    if (!ok) {
      // every MMA issued so far must finish before the TMEM is released
      if (elect_one()) tc_commit(drain);
      drain_wait_d(drain, 0, p.status);
    }
    __syncwarp();
  } else {
    // ===== queries, softmax per tile, O^T =====
    const int quarter = warp & 3;               // TMEM lane quarter of this warp
    const int tid = static_cast<int>(threadIdx.x) - 64;
    const int r = quarter * 16 + lane;          // this thread's row of the group, if any
    const bool busy = quarter * 16 < rows;      // the warp holds rows
    const bool real = lane < 16 && r < rows;
    const int s = real ? s0 + r % p.group_tokens : 0;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t o_tmem = tmem + lane_off + 128;
    const float c = p.scale_log2;
    uint8_t* const p_row = smem + Cfg::kOffP + (lane < 16 && r < NR ? r : 0) * 128;

    // A segment's queries (heads past the last come as zeros; rows past the group's are whatever
    // the memory held, and so are their scores, which nobody reads).
    auto load_q = [&](int b) {
      if (tid != 0) return;
      mbar_arrive_expect_tx(q_ready, Cfg::kChunks * p.group_heads * p.group_tokens * 128);
      for (int cc = 0; cc < Cfg::kChunks; ++cc)
        tma_load_4d(sbase + cc * Cfg::kQB, &p.tm_q, q_ready, cc * kChunk, s0, h0, b);
    };

    bool more = seg.next(p);
    if (more) load_q(seg.b);
    int n_q = 1;        // segments whose queries have been asked for
    // A wait that fails in one warp must not leave the others in a barrier: the warp goes on
    // without touching anything until the next vote, where all four learn of it.
    bool ok = true, dead = false;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar, parity & 1, abort_flag, p.status));
    };
    Ring<NP> at;        // the tile's first pair
    bool head = true;   // the share's first segment
    int g = 0;
    while (more && !dead) {
      const int b = seg.b, n = seg.n, tile0 = seg.tile0;
      const bool whole = seg.whole;
      const SeqKeys keys = seg.keys;
      more = seg.next(p);
      const int pos = keys.len - p.Sq + s;
      int row_lo = 0, row_hi = 0;   // keys of this row
      uint64_t tree = 0;
      if (real) {
        if (p.tree) {
          row_hi = keys.len;
          tree = static_cast<uint64_t>(p.tree[static_cast<size_t>(b) * p.Sq + s]);
        } else {
          row_hi = max(pos + 1, 0);
          row_lo = p.window > 0 ? max(0, pos + 1 - p.window) : 0;
        }
      }
      float m_ref = -INFINITY, l = 0.f;   // reference max, scaled log2 domain; sum of weights
      for (int j = 0; j < n; ++j, ++g) {
        const int kv0 = (tile0 + j) * kTile;
        wait(s_full(g & 1), g >> 1);
        tc_fence_after();
        if (j == n - 1 && more && ok) {   // every S of this segment has been formed
          load_q(seg.b);
          ++n_q;
        }
        const HiddenRows hidden(p, keys, kv0);
        if (hidden.any() && ok) {   // rows that nobody sees must not reach O^T through P = 0
          const int na = hidden.a1 - hidden.a0, nh = na + hidden.b1 - hidden.b0;
          Ring<NP> pair = at;
          for (int m = 0; m < kPairs; ++m, pair.next())
            for (int i = tid; i < nh * 16; i += 128) {
              const int k = i >> 4;
              const int row = k < na ? hidden.a0 + k : hidden.b0 + k - na;
              *reinterpret_cast<uint4*>(smem + Cfg::kOffC + pair.slot * 2 * CB + ((i >> 3) & 1) * CB + row * 128 + (i & 7) * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
            }
          fence_proxy_async_smem();
        }
        for (int m = 0; m < kPairs; ++m) at.next();
        float x[kTile];
        float alpha = 1.f;
        bool moved = false;
        if (busy && ok) {
          uint32_t raw[kTile];
          tmem_ld32(tmem + lane_off + (g & 1) * 64, *reinterpret_cast<uint32_t(*)[32]>(raw));
          tmem_ld32(tmem + lane_off + (g & 1) * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(raw + 32));
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < kTile; ++i) x[i] = __uint_as_float(raw[i]);
          if (kv0 < row_lo || kv0 + kTile > row_hi || (p.tree && kv0 + kTile > keys.len - p.Sq)) {
            uint32_t see[2] = {span_bits(row_lo, row_hi, kv0), span_bits(row_lo, row_hi, kv0 + 32)};
            if (p.tree) {
              const uint64_t t = tree_bits(tree, keys.len - p.Sq, kv0);
              see[0] &= static_cast<uint32_t>(t);
              see[1] &= static_cast<uint32_t>(t >> 32);
            }
#pragma unroll
            for (int i = 0; i < kTile; ++i)
              if (!((see[i / 32] >> (i & 31)) & 1u)) x[i] = -INFINITY;
          }
          float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int i = 4; i < kTile; i += 4)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], x[i + e]);
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
          const float m_new = top > m_ref + kRescaleD ? top : m_ref;
          moved = real && m_new != m_ref;
          alpha = m_new == -INFINITY ? 1.f : ex2(m_ref - m_new);   // 0 from m = -inf
          m_ref = m_new;
        }
        // P_(g-1) has been read, and its product is in O^T
        if (g > 0) wait(pv_done, g - 1);
        // O^T <- alpha O^T where a row's reference moved (the segment's first product overwrites O^T)
        if (j > 0) {
          if (row_warps_any(moved || !ok)) {
            if (real) row_f[r] = moved ? alpha : 1.f;
            if ((dead = row_warps_any(!ok))) break;
            tc_fence_after();
            for (int m = 0; m < kPairs; ++m)
#pragma unroll
              for (int cc = 0; cc < NR; cc += 16) {
                if (cc >= rows) break;
                uint32_t o[16];
                tmem_ld16(o_tmem + m * NR + cc, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  if (cc + i < rows) o[i] = __float_as_uint(__uint_as_float(o[i]) * row_f[cc + i]);
                tmem_st16(o_tmem + m * NR + cc, o);
              }
            tmem_wait_st();
            row_warps_any(false);   // the factors have been read
          }
        }
        if (!ok) continue;   // to the next vote
        if (busy) {
          const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          uint32_t pk[kTile / 2];
#pragma unroll
          for (int i = 0; i < kTile; i += 2) {
            const float p0 = ex2(fmaf(x[i], c, -m_use)), p1 = ex2(fmaf(x[i + 1], c, -m_use));
            sum[i & 3] += p0;
            sum[(i + 1) & 3] += p1;
            pk[i / 2] = pack2<kBf16>(p0, p1);
          }
          l = l * alpha + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
          if (lane < 16 && r < NR) {
#pragma unroll
            for (int u = 0; u < 8; ++u)
              *reinterpret_cast<uint4*>(p_row + ((u ^ (r & 7)) << 4)) =
                  real ? make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]) : make_uint4(0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
      }
      if (dead) break;
      if (real) {
        const PartSum sum(l, m_ref);
        row_f[r] = sum.inv;
        row_lse[r] = sum.lse2;
      }
      wait(pv_done, g - 1);
      if ((dead = row_warps_any(!ok))) break;
      tc_fence_after();
      const size_t orow = static_cast<size_t>(b) * p.R + row0;                                  // + row
      const size_t prow = (static_cast<size_t>(share_id) * 2 + (head ? 0 : 1)) * p.R + row0;    // + row
      if (tid < rows) {
        if (whole) p.lse[orow + tid] = row_lse[tid] * kLn2D;
        else p.part_lse2[prow + tid] = row_lse[tid];
      }
      for (int cc = 0; cc < rows; cc += 16) {
        float f[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(f + 4 * i) = reinterpret_cast<const float4*>(row_f + cc)[i];
#pragma unroll
        for (int m = 0; m < kPairs; ++m) {
          const int e = m * 128 + quarter * 32 + lane;   // element of the latent
          uint32_t o[16];
          tmem_ld16(o_tmem + m * NR + cc, o);
          tmem_wait_ld();
          if (whole) {
            Elem* dst = static_cast<Elem*>(p.out) + (orow + cc) * RANK + e;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (cc + i < rows) dst[i * RANK] = static_cast<Elem>(__uint_as_float(o[i]) * f[i]);
          } else {
            float* dst = p.part_out + (prow + cc) * RANK + e;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (cc + i < rows) dst[i * RANK] = __uint_as_float(o[i]) * f[i];
          }
        }
      }
      tc_fence_before();
      row_warps_any(false);   // the factors have been read
      head = false;
    }
    // the last queries asked for land before the CTA releases its memory
    if (tid == 0 && *abort_flag && share.begin < share.end) drain_wait_d(q_ready, (n_q - 1) & 1, p.status);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ merge --
// Joins the parts of sequences whose tiles lie in more than one share, in share order:
// block (c, y) takes rows y, y + gridDim.y, ... of the sequence whose second part is in
// share c. kLanes sets of rank / 4 threads take every kLanes-th part, four elements a
// thread; their sums are added in a fixed order. Also writes out = 0, LSE = -inf for
// sequences without keys.
constexpr int kMergeLanes = 4, kMergeFlight = 8;

template <typename T, int RANK>
__global__ void __launch_bounds__(kMergeLanes * RANK / 4) latent_merge_kernel(const __grid_constant__ LatentPagedParams p) {
  // programmatic dependent of the main kernel; a main kernel that follows on the stream may
  // set itself up beside this grid
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kThreads = kMergeLanes * RANK / 4;
  __shared__ float4 sums[kMergeLanes][RANK / 4];
  __shared__ float weights[kMergeLanes];
  const int c = static_cast<int>(blockIdx.x);
  const int set = threadIdx.x / (RANK / 4), e = threadIdx.x % (RANK / 4);
  for (int b = c; b < p.B; b += static_cast<int>(gridDim.x)) {
    if (seq_keys(p, b).n > 0) continue;
    for (int r = blockIdx.y; r < p.R; r += gridDim.y) {
      const size_t row = static_cast<size_t>(b) * p.R + r;
      for (int i = threadIdx.x; i < RANK; i += kThreads) static_cast<T*>(p.out)[row * RANK + i] = static_cast<T>(0.f);
      if (threadIdx.x == 0) p.lse[row] = -INFINITY;
    }
  }
  const int total = p.starts[0].w;
  const int4 start = p.starts[c];   // without meaning past the shares
  const ShareOut out(p.n_ctas, total);
  if (c == 0 || c >= out.shares) return;
  const int b = start.x, u0 = start.y;   // the sequence's units: [u0, u0 + start.z)
  const int c0 = out.of_unit(u0 + kSegmentUnits), c1 = out.of_unit(u0 + start.z - 1);
  if (c != c0 + 1 || c0 == c1) return;
  // the parts are the first segments of their shares, but for that of c0 when its share
  // begins before this sequence's units (and so with another's tiles)
  const bool tail0 = out.begin(c0) < u0;
  for (int r = blockIdx.y; r < p.R; r += gridDim.y) {
    auto part = [&](int i) { return (static_cast<size_t>(i) * 2 + ((i == c0 && tail0) ? 1 : 0)) * p.R + r; };
    float M = -INFINITY;
    for (int i = c0 + (threadIdx.x & 31); i <= c1; i += 32) M = fmaxf(M, p.part_lse2[part(i)]);
    M = warp_max(M);   // without NaN parts: their weight is NaN whatever it is
    if (M == -INFINITY) M = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
    for (int i = c0 + set; i <= c1; i += kMergeLanes * kMergeFlight) {
      float4 v[kMergeFlight];
      float lv[kMergeFlight];
#pragma unroll
      for (int k = 0; k < kMergeFlight; ++k)
        if (i + k * kMergeLanes <= c1) {
          const size_t at = part(i + k * kMergeLanes);
          v[k] = reinterpret_cast<const float4*>(p.part_out + at * RANK)[e];
          lv[k] = p.part_lse2[at];
        }
#pragma unroll
      for (int k = 0; k < kMergeFlight; ++k)
        if (i + k * kMergeLanes <= c1) {
          const float w = ex2(lv[k] - M);
          L += w;
          acc.x = fmaf(w, v[k].x, acc.x);
          acc.y = fmaf(w, v[k].y, acc.y);
          acc.z = fmaf(w, v[k].z, acc.z);
          acc.w = fmaf(w, v[k].w, acc.w);
        }
    }
    sums[set][e] = acc;
    if (e == 0) weights[set] = L;
    __syncthreads();
    if (set == 0) {
      L = weights[0];
#pragma unroll
      for (int k = 1; k < kMergeLanes; ++k) {
        const float4 v = sums[k][e];
        L += weights[k];
        acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
      }
      const PartSum sum(L, M);
      const size_t row = static_cast<size_t>(b) * p.R + r;
      constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
      reinterpret_cast<uint2*>(static_cast<T*>(p.out) + row * RANK)[e] =
          make_uint2(pack2<kBf>(acc.x * sum.inv, acc.y * sum.inv), pack2<kBf>(acc.z * sum.inv, acc.w * sum.inv));
      if (e == 0) p.lse[row] = sum.lse2 * kLn2D;
    }
    __syncthreads();
  }
}

template <int RANK, int NR, bool kBf16>
cudaError_t launch_main(const LatentPagedParams& p, cudaStream_t stream) {
  using Cfg = LatDecCfg<RANK, NR>;
  auto kernel = latent_paged_kernel<RANK, NR, kBf16>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, dim3(static_cast<unsigned>(p.n_ctas * p.groups)), dim3(kRaggedThreads),
                          Cfg::kSmemBytes, stream, p);
}

template <int RANK, bool kBf16>
cudaError_t launch_impl(const LatentPagedParams& p, cudaStream_t stream) {
  using Elem = typename std::conditional<kBf16, __nv_bfloat16, __half>::type;
  const int rows = p.group_heads * p.group_tokens;
  const cudaError_t e = rows <= 16   ? launch_main<RANK, 16, kBf16>(p, stream)
                        : rows <= 32 ? launch_main<RANK, 32, kBf16>(p, stream)
                                     : launch_main<RANK, 64, kBf16>(p, stream);
  if (e != cudaSuccess) return e;
  const int y = std::min(p.R, std::max(16, 2048 / p.n_ctas));
  return launch_dependent(latent_merge_kernel<Elem, RANK>, dim3(static_cast<unsigned>(p.n_ctas), y),
                          dim3(kMergeLanes * RANK / 4), 0, stream, p);
}

}  // namespace

cudaError_t launch_latent_paged(const LatentPagedParams& p, int rank, bool bf16, cudaStream_t stream) {
  if (rank == 512) return bf16 ? launch_impl<512, true>(p, stream) : launch_impl<512, false>(p, stream);
  return bf16 ? launch_impl<256, true>(p, stream) : launch_impl<256, false>(p, stream);
}

}  // namespace fa
