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
//                in the type of the cache, as the B operand (the product takes no other beside it:
//                half a step of P |C| in an output; sums, maxima and parts are in fp32)
// O stands transposed in tensor memory because rows are the short side (rank / 128 * rows
// columns: 256 at rank 512 with 64 rows; the other way around it would take all 512). The
// tile goes through a ring of 16 KB pairs of 64-column chunks, each freed as soon as its
// own part of O^T is formed; one barrier a tile tells that it has landed (a wait costs the
// issuer 100 cycles, three products).
//
// Bound by a tile's way through the ring, which holds two tiles beside the queries of 64 rows:
// landing, S (1325 cycles: M = 64 runs at half rate), softmax, O^T (900) and the next load. One new
// token of 16 sequences of up to 8192 rows, rank 512: 128 heads 43.1 us with the merge (36 + 7), of
// which a share of 14 tiles takes 25 and a part's 128 KB on their way out 2.4; 16 heads 27.7 (21 + 6.7),
// 67 MB, of which the loop runs at 7 TB/s and the first tiles of all SMs take 3 us to land. (Writing the
// results 32 columns of all parts at a time: 52 instead of 43.5, registers spilled.) One long sequence is bound
// by the merge, below.
//
// Warp roles (320 threads): warp 0 TMA producer, warp 1 MMA issuer, warps 2-9 softmax (lanes
// 0-15 of the two warps of a tensor-memory quarter w hold rows 16 w .. 16 w + 15, the M = 64
// layout, each warp 32 of the tile's keys) and O^T (all lanes, each warp half its parts).
#include <algorithm>
#include <type_traits>

#include "fa_latent.h"
#include "ptx.cuh"
#include "ragged_shares.cuh"
#include "score_mod.cuh"

namespace fa {
namespace {

constexpr int kTile = LatentPagedParams::kTileKeys;
constexpr int kThreadsD = 320, kSoftThreads = 256;
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
  static constexpr int NT = 8;   // tiles in the ring at a time, at most (NP / kPairs and parts of two more)
  static_assert(NP / kPairs + 2 <= NT, "a barrier a tile");
  // full[NT], empty[NP], x_empty[NX], q_ready, s_full[2], p_full, pv_done, drain
  static constexpr int kNumBars = NT + NP + NX + 6;
  static constexpr int kOffMisc = (kOffBar + kNumBars * 8 + 15) / 16 * 16;   // tmem, abort
  static constexpr int kOffScan = kOffMisc + 16;        // find_share
  static constexpr int kOffRow = kOffScan + 48;         // [64] factor, [64] log2-sum, [2][64] halves of a row
  static constexpr int kSmemBytes = kOffRow + 1024;
  static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
};

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

// Zeros in the rows of a tile (from key kv0, its first pair in slot `slot` of the ring) whose drafted tokens no
// mask has: like rows past the sequence, they must not reach O^T through P = 0. By the softmax warps; few
// tiles come here, and in line it cost all of them registers (128 heads 35.5 -> 37.2 us).
template <int NP, int kPairs>
__device__ __noinline__ void zero_unseen(const long long* masks, int Sq, int len, int kv0, uint8_t* ring, int slot, int tid) {
  constexpr int CB = kTile * 128;
  uint64_t seen = 0;
  for (int t = tid & 31; t < Sq; t += 32) seen |= static_cast<uint64_t>(masks[t]);
  seen = static_cast<uint64_t>(__reduce_or_sync(0xffffffffu, static_cast<uint32_t>(seen >> 32))) << 32 |
         __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(seen));
  const int rows = min(len - kv0, kTile);
  const uint64_t unseen = ~tree_bits(seen, len - Sq, kv0) << (kTile - rows) >> (kTile - rows);
  if (unseen == 0) return;
  for (int m = 0; m < kPairs; ++m, slot = slot + 1 == NP ? 0 : slot + 1)
    for (int i = tid; i < rows * 16; i += kSoftThreads)
      if ((unseen >> (i >> 4)) & 1)
        *reinterpret_cast<uint4*>(ring + slot * 2 * CB + ((i >> 3) & 1) * CB + (i >> 4) * 128 + (i & 7) * 16) =
            make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
}

template <int RANK, int NR, bool kBf16>
__global__ void __launch_bounds__(kThreadsD, 1)
    latent_paged_kernel(const __grid_constant__ LatentPagedParams p) {
  using Cfg = LatDecCfg<RANK, NR>;
  using Elem = typename std::conditional<kBf16, __nv_bfloat16, __half>::type;
  constexpr int NP = Cfg::NP, NX = Cfg::NX, NT = Cfg::NT, CB = Cfg::CB, kPairs = Cfg::kPairs;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {   // the 128-byte swizzle needs 1024-byte aligned tiles
    if (threadIdx.x == 0) atomicOr(p.status, kStatusBadLaunch);
    return;
  }
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::kOffMisc + 4);
  volatile int* issued = abort_flag + 1;   // tiles that the producer has asked for, and segments' queries
  float* row_f = reinterpret_cast<float*>(smem + Cfg::kOffRow);
  float* row_lse = row_f + 64;
  float* halves = row_f + 128;   // [2][64]

  const Bars full{sbase + Cfg::kOffBar}, empty{full(NT)}, x_empty{empty(NP)};
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
    for (int s = 0; s < NT; ++s) mbar_init(full(s), kTile / p.box_rows);   // an arrival a box
    for (int s = 0; s < NP; ++s) mbar_init(empty(s), 1);
    for (int s = 0; s < NX; ++s) mbar_init(x_empty(s), 1);
    mbar_init(q_ready, 1);   // once a segment
    mbar_init(s_full(0), 1);
    mbar_init(s_full(1), 1);
    mbar_init(p_full, 8);   // one arrival per softmax warp
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
  const Share share = find_share<kThreadsD>(p, share_id, reinterpret_cast<int*>(smem + Cfg::kOffScan));
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // the merge kernel may be scheduled now; it waits for this grid's completion
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  Segments seg(p, share);

  if (warp == 0) {
    // ===================== TMA producer =====================
    // Lane i takes box i of every tile, by itself: it reads the box's table entry (a tile ahead:
    // the read would stand before every tile's copies), waits for the ring's slots and issues
    // the copies (a barrier counts the boxes' arrivals). A box past the sequence or before
    // every row's window, or an entry outside [0, num_blocks), is loaded from an out-of-range
    // row, which the copy fills with zeros.
    if (lane < kTile / p.box_rows) {
      Ring<NP> at;
      Ring<NX> xt;
      int n_p = 0, n_x = 0;   // pairs and rotated parts issued
      int n_t = 0;            // tiles arrived for
      const uint32_t box_bytes = p.box_rows * 128, box = lane * box_bytes;
      auto free = [&](bool used, uint32_t bar, uint32_t parity) {
        return !used || mbar_wait(bar, parity ^ 1u, abort_flag, p.status);
      };
      int j = 0;
      auto page = [&]() -> int {   // of this lane's box of tile j of the segment
        const int key = (seg.tile0 + j) * kTile + lane * p.box_rows;
        if (key >= seg.keys.len || key + p.box_rows <= seg.keys.first) return -1;
        return p.block_table[static_cast<size_t>(seg.b) * p.max_blocks + (key >> p.block_shift)];
      };
      bool have = seg.next(p), ok = true;
      int pb = have ? page() : -1;
#ifdef FA_WAIT_TEST
      if (wait_test(kWaitProducer, p.H)) ok = mbar_wait(drain, 0, abort_flag, p.status);
#endif
      while (ok && have) {
        const bool in_range = pb >= 0 && pb < p.num_blocks;
        const int y = in_range ? ((seg.tile0 + j) * kTile + lane * p.box_rows) & (p.block_size - 1) : p.block_size;
        const int z = in_range ? pb : 0;
        if (++j == seg.n) {
          j = 0;
          have = seg.next(p);
        }
        if (have) pb = page();
        const uint32_t f = full(n_t % NT);
        // the tile's bytes are announced copy by copy, its arrival comes at the end
#pragma unroll
        for (int m = 0; m < kPairs; ++m) {
          if (!(ok = free(n_p >= NP, empty(at.slot), at.parity))) break;
          const uint32_t dst = sbase + Cfg::kOffC + at.slot * 2 * CB + box;
          mbar_expect_tx(f, 2 * box_bytes);
          tma_load_3d(dst, &p.tm, f, m * 128, y, z);
          tma_load_3d(dst + CB, &p.tm, f, m * 128 + kChunk, y, z);
          at.next();
          ++n_p;
        }
        if (!ok || !(ok = free(n_x >= NX, x_empty(xt.slot), xt.parity))) break;
        mbar_arrive_expect_tx(f, box_bytes);
        tma_load_3d(sbase + Cfg::kOffX + xt.slot * CB + box, &p.tm, f, RANK, y, z);
        xt.next();
        ++n_x;
        ++n_t;
        // The next tile's rows on their way to L2 while its slots are still in use (16 sequences of up
        // to 8192 rows, 128 heads: 46 -> 43.5 us).
        if (have && n_p + kPairs > NP && pb >= 0 && pb < p.num_blocks) {
          const int yn = ((seg.tile0 + j) * kTile + lane * p.box_rows) & (p.block_size - 1);
#pragma unroll
          for (int cc = 0; cc < Cfg::kChunks; ++cc) tma_prefetch_l2_3d(&p.tm, cc * kChunk, yn, pb);
        }
      }
      // A tile given up half-way is arrived for, and so is one that another lane went on to, so that
      // the phases complete.
      if (!ok) mbar_arrive(full(n_t++ % NT));
      const int most = __reduce_max_sync((1u << (kTile / p.box_rows)) - 1, n_t);
      for (; n_t < most; ++n_t) mbar_arrive(full(n_t % NT));
      issued[0] = most;
    }
    __syncwarp();
  } else if (warp == 1) {
    // ===================== MMA issuer (the whole warp, one lane of it the MMAs) =====================
    // Two streams of work, whichever is ready first: tile gs's S, once it has landed, and
    // tile go's O^T once its P is there. (In a fixed order, S of the next tile
    // first, a late load held up O^T, which frees the ring for the load after it.)
    constexpr uint32_t idesc_s = make_idesc(64, kTile, kBf16, false, false);
    constexpr uint32_t idesc_o = make_idesc(128, NR, kBf16, true, false);
    TileWalk walk{seg};
    Ring<NP> at_s, at_o;
    Ring<NX> xt;
    int n_seg = 0;      // segments whose queries have landed
    int gs = 0, go = 0; // the next tile of either stream
    bool first_of[2] = {false, false};   // of the tiles whose S is formed, by g % 2: a segment's first
    const uint64_t qa = make_sdesc(sbase, 16, 1024);
    const uint64_t pb = make_sdesc(sbase + Cfg::kOffP, 16, 1024);
    auto ready = [](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_test(bar, parity)); };
    // (votes make what was loaded the same in every lane for the compiler too, and with it the
    // control flow and the descriptors: elected)
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
    if (have && wait_test(kWaitIssuer, p.H)) ok = warp_wait(drain, 0, abort_flag, p.status);
#endif
    auto issue_o = [&]() {   // O^T (+)= C_go^T P
      tc_fence_after();
      const uint32_t more = first_of[go & 1] ? 0u : 1u, o_t = tmem + 128;
#pragma unroll
      for (int m = 0; m < kPairs; ++m) {   // a part a pair
        const uint64_t ca = make_sdesc(sbase + Cfg::kOffC + at_o.slot * 2 * CB, CB, 1024);
        elected([&] {
          mma_ss_steps<kTile / 16, false, 0, true, Cfg::kP>(o_t + m * NR, ca, pb, idesc_o, more);
          tc_commit(empty(at_o.slot));
          if (m == kPairs - 1) tc_commit(pv_done);
        });
        at_o.next();
      }
      ++go;
    };
    // Wait for a barrier of the S stream, issuing O^T meanwhile when its P comes first; without a
    // barrier, for the next P. Bounded as mbar_wait.
    auto until = [&](uint32_t bar, uint32_t parity) -> bool {
      long long since = 0;
      for (uint32_t idle = 0;;) {
        if (bar && ready(bar, parity)) return true;
        if (go < gs && ready(p_full, go & 1)) {
          issue_o();
          if (!bar) return true;
          idle = 0;
          continue;
        }
        if ((++idle & 15u) != 0) continue;
        if (idle == 16) since = clock64();
        bool stop = false;
        if (lane == 0) {
          stop = *abort_flag;
          if (!stop && clock64() - since > kWaitLimitCycles) {
            *abort_flag = 1;
            atomicOr(p.status, kStatusWaitTimeout);
            stop = true;
          }
        }
        if (__any_sync(0xffffffffu, stop)) return false;
      }
    };
    while (ok && have) {
      // S_gs goes over S_(gs-2), which has been read when P_(gs-2) is there
      while (ok && gs > go + 1) ok = until(0, 0);
      if (!ok) break;
      const bool begins = first_s;
      if (begins && !(ok = until(q_ready, n_seg++ & 1))) break;
      if (!(ok = until(full(gs % NT), (gs / NT) & 1))) break;
      tc_fence_after();
      const uint32_t d = tmem + (gs & 1) * 64;
#pragma unroll
      for (int m = 0; m < kPairs; ++m) {
        const uint64_t cb = make_sdesc(sbase + Cfg::kOffC + at_s.slot * 2 * CB, 16, 1024);
        elected([&] { mma_ss_steps<8, true, Cfg::kQB, true, CB>(d, qa + 2 * m * (Cfg::kQB >> 4), cb, idesc_s, m > 0 ? 1u : 0u); });
        at_s.next();
      }
      const uint64_t xb = make_sdesc(sbase + Cfg::kOffX + xt.slot * CB, 16, 1024);
      elected([&] {
        mma_ss_steps<4, true, Cfg::kQB, true, CB>(d, qa + 2 * kPairs * (Cfg::kQB >> 4), xb, idesc_s, 1u);
        tc_commit(x_empty(xt.slot));
        tc_commit(s_full(gs & 1));
      });
      xt.next();
      first_of[gs & 1] = begins;
      ++gs;
      have = next();
    }
    while (ok && go < gs) ok = until(0, 0);
  } else {
    // ===== queries, softmax per tile, O^T =====
    const int quarter = warp & 3;               // TMEM lane quarter of this warp
    const int half = (warp - 2) >> 2;           // its half of a tile's keys, and of the parts of O^T
    const int tid = static_cast<int>(threadIdx.x) - 64;
    const int r = quarter * 16 + lane;          // this thread's row of the group, if any
    const bool busy = quarter * 16 < rows;      // the warp holds rows
    const bool real = lane < 16 && r < rows;
    const int s = real ? s0 + r % p.group_tokens : 0;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t o_tmem = tmem + lane_off + 128;
    const float c = p.scale_log2;
    constexpr int kHalf = kTile / 2, kOwn = kPairs / 2;   // keys of a warp, its parts of O^T
    uint8_t* const p_row = smem + Cfg::kOffP + (lane < 16 && r < NR ? r : 0) * 128;
    auto any = [](bool flag) { return row_warps_any<kSoftThreads>(flag); };

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
    int n_q = more ? 1 : 0;   // segments whose queries have been asked for
    // A wait that fails in one warp must not leave the others in a barrier: the warp goes on
    // without touching anything until the next vote, where all learn of it.
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
            for (int i = tid; i < nh * 16; i += kSoftThreads) {
              const int k = i >> 4;
              const int row = k < na ? hidden.a0 + k : hidden.b0 + k - na;
              *reinterpret_cast<uint4*>(smem + Cfg::kOffC + pair.slot * 2 * CB + ((i >> 3) & 1) * CB + row * 128 + (i & 7) * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
            }
          fence_proxy_async_smem();
        }
        if (p.tree && kv0 + kTile > keys.len - p.Sq && ok)
          zero_unseen<NP, kPairs>(p.tree + static_cast<size_t>(b) * p.Sq, p.Sq, keys.len, kv0, smem + Cfg::kOffC, at.slot, tid);
        for (int m = 0; m < kPairs; ++m) at.next();
        float x[kHalf], top = -INFINITY;   // scores, and the greatest in the log2 domain
        __syncwarp();   // (tensor-memory instructions have to find the warp whole)
        if (busy && ok) {
          const int k0 = kv0 + half * kHalf;
          uint32_t raw[kHalf];
          tmem_ld32(tmem + lane_off + (g & 1) * 64 + half * kHalf, raw);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < kHalf; ++i) x[i] = __uint_as_float(raw[i]);
          // (lanes without a row have no say, and their scores no reader)
          if (__any_sync(0xffffffffu, real && (k0 < row_lo || k0 + kHalf > row_hi)) ||
              (p.tree && k0 + kHalf > keys.len - p.Sq)) {
            uint32_t see = span_bits(row_lo, row_hi, k0);
            if (p.tree) see &= static_cast<uint32_t>(tree_bits(tree, keys.len - p.Sq, k0));
#pragma unroll
            for (int i = 0; i < kHalf; ++i)
              if (!((see >> i) & 1u)) x[i] = -INFINITY;
          }
          float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int i = 4; i + 8 <= kHalf; i += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = fmax3(mx[e], x[i + e], x[i + 4 + e]);
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], x[kHalf - 4 + e]);
          top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
        }
        // A row's reference moves when a score of either half exceeds it by 2^8: one vote tells
        // whether any does; then the halves exchange their maxima and O^T <- alpha O^T. (A
        // segment's first tile sets it; its first product overwrites O^T.)
        if (j == 0 || any((real && top > m_ref + kRescaleD) || !ok)) {
          if (real) halves[half * 64 + r] = top;
          if (j > 0) wait(pv_done, g - 1);   // its product is in O^T
          if ((dead = any(!ok))) break;
          float alpha = 1.f;
          if (real) {
            const float both = fmaxf(halves[r], halves[64 + r]);
            const float m_new = both > m_ref + kRescaleD ? both : m_ref;
            alpha = m_new == -INFINITY ? 1.f : ex2(m_ref - m_new);   // 0 from m = -inf
            m_ref = m_new;
            l *= alpha;
          }
          if (j > 0) {
            if (real && half == 0) row_f[r] = alpha;
            any(false);
            __syncwarp();
            tc_fence_after();
            for (int m = half * kOwn; m < (half + 1) * kOwn; ++m)
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
            any(false);   // the factors have been read
          }
        }
        uint32_t pk[kHalf / 2];
        if (busy && ok) {
          const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
          const uint64_t c2 = f2_pack(c, c), nm2 = f2_pack(-m_use, -m_use);
          uint64_t sum0 = f2_pack(0.f, 0.f), sum1 = sum0;
#pragma unroll
          for (int i = 0; i < kHalf; i += 2) {
            float p0, p1;
            f2_unpack(f2_fma(f2_pack(x[i], x[i + 1]), c2, nm2), p0, p1);
            p0 = ex2(p0);
            p1 = ex2(p1);
            if (i & 2) sum1 = f2_add(sum1, f2_pack(p0, p1));
            else sum0 = f2_add(sum0, f2_pack(p0, p1));
            pk[i / 2] = pack2<kBf16>(p0, p1);
          }
          float a0, a1;
          f2_unpack(f2_add(sum0, sum1), a0, a1);
          l += a0 + a1;
        }
        if (g > 0) wait(pv_done, g - 1);   // P_(g-1) has been read
        if (!ok) continue;   // to the next vote
        if (busy && lane < 16 && r < NR) {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            *reinterpret_cast<uint4*>(p_row + (((half * 4 + u) ^ (r & 7)) << 4)) =
                real ? make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]) : make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
      }
      if (dead) break;
      // The last tile's product has every warp's P, and a warp gives its P after it has read the halves'
      // maxima: past this wait they may be overwritten, in a segment of one tile too, which has no vote
      // in between.
#ifdef FA_WAIT_TEST
      if (wait_test(kWaitSoftmax, p.H)) wait(drain, 0);
#endif
      wait(pv_done, g - 1);
      if (real) halves[half * 64 + r] = l;
      if ((dead = any(!ok))) break;
      if (real && half == 0) {
        const PartSum sum(l + halves[64 + r], m_ref);
        row_f[r] = sum.inv;
        row_lse[r] = sum.lse2;
      }
      any(false);
      __syncwarp();
      tc_fence_after();
      const size_t orow = static_cast<size_t>(b) * p.R + row0;                                  // + row
      const size_t prow = (static_cast<size_t>(share_id) * 2 + (head ? 0 : 1)) * p.R + row0;    // + row
      if (tid < rows) {
        if (whole) p.lse[orow + tid] = row_lse[tid] * kLn2D;
        else p.part_lse2[prow + tid] = row_lse[tid];
      }
      __syncwarp();
      for (int cc = 0; cc < rows; cc += 16) {
        float f[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(f + 4 * i) = reinterpret_cast<const float4*>(row_f + cc)[i];
#pragma unroll
        for (int mm = 0; mm < kOwn; ++mm) {
          const int m = half * kOwn + mm;
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
      any(false);   // the factors have been read
      head = false;
    }
    if (tid == 0) issued[1] = n_q;
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // A wait ran out, whosever: only now is it known that nothing more is issued. Every copy lands and every
    // MMA finishes before the CTA releases its memory.
    if (threadIdx.x == 0) {
      for (int i = max(0, issued[0] - NT); i < issued[0]; ++i) drain_wait(full(i % NT), (i / NT) & 1, p.status);
      if (issued[1] > 0) drain_wait(q_ready, (issued[1] - 1) & 1, p.status);
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

// ------------------------------------------------------------------ merge --
// Joins the parts of sequences whose tiles lie in more than one share, in share order: a
// warp takes 128 elements of a row. Up to as many sequences as shares, block (b, y) takes
// sequence b, found by a scan over the lengths as the main kernel's; more sequences than
// shares, block (c, y) the one whose second part is in share c. Also writes out = 0, LSE =
// -inf for sequences without keys. Bound by latency (10 KB a row from L2), and by a row's walk along its
// parts: one sequence of 8192 rows, 16 heads, leaves 128 of them, 31 of the call's 41 us; of 32768, 152, 41 of 57.
constexpr int kMergeWarps = 4, kMergeFlight = 12;

template <typename T, int RANK>
__global__ void __launch_bounds__(32 * kMergeWarps) latent_merge_kernel(const __grid_constant__ LatentPagedParams p) {
  // programmatic dependent of the main kernel; a main kernel that follows on the stream may
  // set itself up beside this grid
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kParts = RANK / 128, kRows = kMergeWarps / kParts;   // warps a row, rows a block
  constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
  __shared__ int2 sums[kMergeWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = static_cast<int>(blockIdx.y) * kRows + warp / kParts;
  const int e = warp % kParts * 128 + lane * 4;   // this lane's four elements
  int b, u0, units, total;   // a sequence, its units [u0, u0 + units), all units
  // The lengths are read before the wait: every block of the main kernel, which let this one start,
  // has waited for what ran before it, and does not write them.
  auto nothing = [&](int seq) {
    if (r >= p.R) return;
    const size_t row = static_cast<size_t>(seq) * p.R + r;
    *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + row * RANK + e) = make_uint2(0u, 0u);
    if (e == 0) p.lse[row] = -INFINITY;
  };
  if (p.B <= p.n_ctas) {
    b = static_cast<int>(blockIdx.x);
    units = units_of(seq_keys(p, b).n);
    int before = 0, all = 0;
    for (int i = threadIdx.x; i < p.B; i += 32 * kMergeWarps) {
      const int n = units_of(seq_keys(p, i).n);
      all += n;
      if (i < b) before += n;
    }
    before = __reduce_add_sync(0xffffffffu, before);
    all = __reduce_add_sync(0xffffffffu, all);
    if (lane == 0) sums[warp] = make_int2(before, all);
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    u0 = total = 0;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) {
      u0 += sums[w].x;
      total += sums[w].y;
    }
    if (units == 0) {
      nothing(b);
      return;
    }
  } else {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int i = blockIdx.x; i < p.B; i += gridDim.x)
      if (seq_keys(p, i).n == 0) nothing(i);
    total = p.starts[0].w;
    const int4 start = p.starts[blockIdx.x];   // without meaning past the shares
    b = start.x;
    u0 = start.y;
    units = start.z;
  }
  const ShareOut out(p.n_ctas, total);
  if (r >= p.R || (p.B > p.n_ctas && static_cast<int>(blockIdx.x) >= out.shares)) return;
  const int c0 = out.of_unit(u0 + kSegmentUnits), c1 = out.of_unit(u0 + units - 1);
  if (c0 == c1 || (p.B > p.n_ctas && static_cast<int>(blockIdx.x) != c0 + 1)) return;
  // the parts are the first segments of their shares, but for that of c0 when its share
  // begins before this sequence's units (and so with another's tiles)
  const bool tail0 = out.begin(c0) < u0;
  auto part = [&](int i) { return (static_cast<size_t>(i) * 2 + ((i == c0 && tail0) ? 1 : 0)) * p.R + r; };
  // a batch's loads go out together, the first batch's with those of the maximum
  float4 v[kMergeFlight];
  float lv[kMergeFlight];
  auto load = [&](int i) {
#pragma unroll
    for (int k = 0; k < kMergeFlight; ++k)
      if (i + k <= c1) {
        const size_t at = part(i + k);
        v[k] = *reinterpret_cast<const float4*>(p.part_out + at * RANK + e);
        lv[k] = p.part_lse2[at];
      }
  };
  load(c0);
  float M = -INFINITY;
  for (int i = c0 + lane; i <= c1; i += 32) M = fmaxf(M, p.part_lse2[part(i)]);
  M = warp_max(M);   // without NaN parts: their weight is NaN whatever it is
  if (M == -INFINITY) M = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float L = 0.f;
  for (int i = c0; i <= c1; i += kMergeFlight) {
    if (i > c0) load(i);
#pragma unroll
    for (int k = 0; k < kMergeFlight; ++k)
      if (i + k <= c1) {
        const float w = ex2(lv[k] - M);
        L += w;
        acc.x = fmaf(w, v[k].x, acc.x);
        acc.y = fmaf(w, v[k].y, acc.y);
        acc.z = fmaf(w, v[k].z, acc.z);
        acc.w = fmaf(w, v[k].w, acc.w);
      }
  }
  const PartSum sum(L, M);
  const size_t row = static_cast<size_t>(b) * p.R + r;
  *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + row * RANK + e) =
      make_uint2(pack2<kBf>(acc.x * sum.inv, acc.y * sum.inv), pack2<kBf>(acc.z * sum.inv, acc.w * sum.inv));
  if (e == 0) p.lse[row] = sum.lse2 * kLn2D;
}

template <int RANK, int NR, bool kBf16>
cudaError_t launch_main(const LatentPagedParams& p, cudaStream_t stream) {
  using Cfg = LatDecCfg<RANK, NR>;
  auto kernel = latent_paged_kernel<RANK, NR, kBf16>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, dim3(static_cast<unsigned>(p.n_ctas * p.groups)), dim3(kThreadsD),
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
  constexpr int kRows = kMergeWarps / (RANK / 128);
  return launch_dependent(latent_merge_kernel<Elem, RANK>,
                          dim3(static_cast<unsigned>(std::min(p.B, p.n_ctas)), static_cast<unsigned>((p.R + kRows - 1) / kRows)),
                          dim3(32 * kMergeWarps), 0, stream, p);
}

}  // namespace

cudaError_t launch_latent_paged(const LatentPagedParams& p, int rank, bool bf16, cudaStream_t stream) {
  if (rank == 512) return bf16 ? launch_impl<512, true>(p, stream) : launch_impl<512, false>(p, stream);
  return bf16 ? launch_impl<256, true>(p, stream) : launch_impl<256, false>(p, stream);
}

}  // namespace fa
