// Attention of one or a few new tokens per sequence over a paged key/value
// cache, for sequences of unequal length known on the device only.
//
// Row s of sequence b (length L_b, its new tokens included) stands at position
// p = L_b - Sq + s and sees keys max(0, p + 1 - window) <= j <= p (window 0: from
// key 0); scores may be capped and biased by distance as in the span forward.
// The query packing, the tile pipeline and the merge formula are those of the
// split-KV forward (fa_decode.cu); the division of the work is not:
//
//   - the host knows neither the lengths nor how uneven they are, so the work is
//     one list of 128-key tiles over all sequences and heads, and each of one
//     wave of CTAs takes an equal, contiguous share of it, found by a scan over
//     the lengths at its start. One long sequence among short ones spreads over
//     the GPU, and a captured graph stays balanced when the lengths change;
//   - a share is a run of segments, each a key range of one (sequence, key/value
//     head). Loads run ahead across segments. A segment that holds its whole
//     range writes out and LSE itself; the others (at most the first and the
//     last of a share) write a partial result, which the merge kernel joins in
//     the order of the shares, so results do not depend on scheduling.
//
// Up to 16 rows a key/value head (G * Sq <= 128 rows share each tile) the kernel is bound by
// the bytes of K and V: at 32 + 8 heads, d = 128, bf16, 16 sequences of 4096 keys take 50.8 us
// (5.3 TB/s) and of 8192 keys 88.8 us (6.0 TB/s). About 10 us of each call are the scan, the
// first loads, the unequal ends and the merge; one sequence of 500 keys takes 9. With more
// rows the softmax counts (the figures stand at launch_form).
//
// Rows of the cache outside a sequence's keys (the tail of its last page, keys before
// every row's window) are cleared in the V tile before use, so that whatever they hold, NaN
// included, cannot reach O through a probability of 0. A NaN among the scores that a row
// sees comes out as NaN in its out and its LSE, through the merge too.
//
// A row's last bits depend on where the shares cut its keys, and so on the lengths of the
// other sequences.
//
// Warp roles and tensor memory: as fa_decode.cu.
#include <algorithm>
#include <type_traits>

#include "fa_ragged.h"
#include "ptx.cuh"
#include "score_mod.cuh"

namespace fa {
namespace {

constexpr int kThreads = 192;
constexpr float kLn2R = 0.6931471805599453f;
constexpr float kLog2eR = 1.4426950408889634f;
constexpr float kRescaleThresholdR = 8.0f;   // same lazy-rescale rule as the forward

template <int D>
struct RagCfg {
  static constexpr int kChunks = D / kChunk;
  static constexpr int kTileBytes = kTileM * D * 2;
  static constexpr int kStages = 3;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kTileBytes;
  static constexpr int kOffV = kOffK + kStages * kTileBytes;
  static constexpr int kOffBar = kOffV + kStages * kTileBytes;
  // q_ready, k_full[S], k_empty[S], v_full[S], v_empty[S], s_full[2],
  // p_full[2], pv_done[2], drain
  static constexpr int kNumBars = 1 + 4 * kStages + 6 + 1;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kOffScan = kOffMisc + 16;            // 6 warp totals, start (b, prefix)
  static constexpr int kSmemBytes = kOffScan + 32 + 1024;   // + alignment slack
};

__device__ __forceinline__ void drain_wait_r(uint32_t bar, uint32_t parity, int* status) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > kDrainLimitCycles) {
      atomicOr(status, kStatusWaitTimeout);
      return;
    }
  }
}

// Keys of one sequence that any of its rows sees, and their tiles.
struct SeqKeys {
  int len, first;     // keys [first, len)
  int tile0, n;       // tiles [tile0, tile0 + n)
};

__device__ __forceinline__ SeqKeys seq_keys(const RaggedParams& p, int b) {
  SeqKeys s;
  s.len = min(max(p.seq_lens[b], 0), p.capacity);
  s.first = p.window > 0 ? max(0, s.len - p.Sq + 1 - p.window) : 0;
  s.tile0 = s.first / kTileN;
  s.n = s.len > 0 ? (s.len + kTileN - 1) / kTileN - s.tile0 : 0;
  return s;
}

// The list that is shared out counts units: one a key tile and kSegmentUnits for
// every (sequence, head) that has tiles, in front of them, for what a segment
// costs beside its tiles. Measured at 32 + 8 heads, d = 128, 66137 keys in 16
// sequences of 8 to 8192 and (second) 65521 + 15 x 1 keys: with no such units one
// CTA got dozens of one-tile segments, 70.1 and 119 us; 1 unit 60.5 and 69.1; 2
// units 52.5 and 54.2; 3 units 53.1 and 54.1.
constexpr int kSegmentUnits = 2;
__device__ __forceinline__ int units_of(int tiles) { return tiles > 0 ? tiles + kSegmentUnits : 0; }

// Even shares of a list of `total` units (below 2^31): the first `rest` shares
// take one unit more than the others.
struct ShareOut {
  int shares, each, rest;
  __device__ __forceinline__ ShareOut(int n_ctas, int total) {
    shares = min(n_ctas, total);
    each = shares > 0 ? total / shares : 0;
    rest = total - each * shares;
  }
  __device__ __forceinline__ int begin(int c) const { return c * each + min(c, rest); }
  __device__ __forceinline__ int of_unit(int t) const {
    const int big = rest * (each + 1);   // units of the larger shares
    return t < big ? t / (each + 1) : rest + (t - big) / each;
  }
};

// A CTA's share, found by all its threads: a scan over the sequences' units. Where it
// begins is also written for the merge: (sequence, units per head before it, its units,
// units of all sequences per head). Two barriers.
struct Share {
  int begin, end;    // units of the list
  int b, pre;        // the first unit's sequence, and units per head before it
};

__device__ __forceinline__ Share find_share(const RaggedParams& p, int cta, int* scan) {
  // launched as a programmatic dependent of whatever runs before on the stream
  // (the merge of the call before lets it start early): the barriers, tensor memory
  // and descriptors above are set up meanwhile, memory is touched from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = static_cast<int>(warp_id()), lane = static_cast<int>(lane_id());
  // thread t holds sequences [t * per, (t + 1) * per)
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b_lo = min(p.B, static_cast<int>(threadIdx.x) * per);
  const int b_hi = min(p.B, b_lo + per);
  int mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += units_of(seq_keys(p, b).n);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int pre = incl - mine, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) pre += scan[w];
    total += scan[w];
  }
  const ShareOut out(p.n_ctas, total * p.Hkv);
  Share s;
  s.begin = cta < out.shares ? out.begin(cta) : 0;
  s.end = cta < out.shares ? out.begin(cta + 1) : 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const int n = units_of(seq_keys(p, b).n);
    if (s.begin < s.end && pre * p.Hkv <= s.begin && s.begin < (pre + n) * p.Hkv) {
      scan[6] = b;
      scan[7] = pre;
      p.starts[cta] = make_int4(b, pre, n, total);
    }
    pre += n;
  }
  if (total == 0 && cta == 0 && threadIdx.x == 0) p.starts[0] = make_int4(0, 0, 0, 0);
  __syncthreads();
  s.b = s.begin < s.end ? scan[6] : 0;
  s.pre = s.begin < s.end ? scan[7] : 0;
  return s;
}

// The segments of one CTA's share, in order; every role walks its own copy.
struct Segments {
  int cur, end, pre;   // list position, end of the share, units per head before b
  int b;
  SeqKeys keys;
  // the current segment
  int kvh, tile0, n;
  bool whole;

  __device__ __forceinline__ Segments(const RaggedParams& p, const Share& s)
      : cur(s.begin), end(s.end), pre(s.pre), b(s.b) {
    if (cur < end) keys = seq_keys(p, b);
  }
  __device__ __forceinline__ bool next(const RaggedParams& p) {
    while (cur < end) {
      int units = units_of(keys.n);
      while (cur >= (pre + units) * p.Hkv) {   // cur < end <= total: some later b has units
        pre += units;
        if (++b >= p.B) return false;   // only if the lengths changed meanwhile
        keys = seq_keys(p, b);
        units = units_of(keys.n);
      }
      const int off = cur - pre * p.Hkv;
      kvh = off / units;
      const int u = off - kvh * units;
      const int take = min(units - u, end - cur);
      cur += take;
      const int t0 = max(u - kSegmentUnits, 0), t1 = max(u + take - kSegmentUnits, 0);
      if (t1 == t0) continue;   // the share ends with the units in front of a head's tiles
      n = t1 - t0;
      tile0 = keys.tile0 + t0;
      whole = n == keys.n;
      return true;
    }
    return false;
  }
};

// The tiles of a share in order, for the MMA issuers: whether there is a next
// one, and whether it begins a segment.
struct TileWalk {
  Segments& seg;
  int left = 0;
  bool first = false;
  __device__ __forceinline__ bool next(const RaggedParams& p) {
    first = left == 0;
    if (first) {
      if (!seg.next(p)) return false;
      left = seg.n;
    }
    --left;
    return true;
  }
};

// TMA producer warp of both kernels: K and V tiles of the share into rings of
// kStages. Each lane i < 128 / box_rows reads the block-table entry of box i of a
// tile and issues that box itself. A box past the sequence or before every row's
// window, or a table entry outside [0, num_blocks), is loaded from an
// out-of-range row, which the copy fills with zeros.
template <int kChunks, int kStages, class Bar>
__device__ __forceinline__ void produce(const RaggedParams& p, Segments& seg, uint32_t k_ring,
                                        uint32_t v_ring, Bar k_full, Bar k_empty, Bar v_full,
                                        Bar v_empty, volatile int* abort_flag) {
  constexpr int kTileBytes = kChunks * kTileN * 128;
  const int lane = static_cast<int>(lane_id());
  const int n_boxes = kTileN / p.box_rows;
  auto load_part = [&](const CUtensorMap* tm, uint32_t dst, uint32_t bar, int key, int pb) {
    if (lane >= n_boxes) return;
    const bool in_range = pb >= 0 && pb < p.num_blocks;
    const int y = in_range ? key % p.block_size : p.block_size;
    const int z = in_range ? pb * p.Hkv + seg.kvh : 0;
    for (int c = 0; c < kChunks; ++c)
      tma_load_3d(dst + c * (kTileN * 128) + lane * p.box_rows * 128, tm, bar, c * kChunk, y, z);
  };
  int g = 0;   // tiles whose K load has been issued
  bool stop = false;
  while (!stop && seg.next(p)) {
    const int* table = p.block_table + static_cast<size_t>(seg.b) * p.max_blocks;
    for (int j = 0; j < seg.n; ++j, ++g) {
      const int key = (seg.tile0 + j) * kTileN + lane * p.box_rows;
      const int st = g % kStages;
      const uint32_t use = static_cast<uint32_t>(g / kStages);
      int pb = -1;
      if (lane < n_boxes && key < seg.keys.len && key + p.box_rows > seg.keys.first)
        pb = table[key / p.block_size];
      int fail = 0;
      if (lane == 0) {
        if (g >= kStages && !mbar_wait(k_empty(st), (use - 1) & 1, abort_flag, p.status)) fail = 1;
        else mbar_arrive_expect_tx(k_full(st), kTileBytes);
      }
      if ((stop = __shfl_sync(0xffffffffu, fail, 0))) break;
      load_part(&p.tm_k, k_ring + st * kTileBytes, k_full(st), key, pb);
      if (lane == 0) {
        if (g >= kStages && !mbar_wait(v_empty(st), (use - 1) & 1, abort_flag, p.status)) fail = 1;
        else mbar_arrive_expect_tx(v_full(st), kTileBytes);
      }
      if ((stop = __shfl_sync(0xffffffffu, fail, 0))) {
        ++g;   // this tile's K load is in flight
        break;
      }
      load_part(&p.tm_v, v_ring + st * kTileBytes, v_full(st), key, pb);
    }
  }
  if (lane == 0 && *abort_flag) {
    // let every copy already issued land before the CTA releases its memory
    for (int gg = max(0, g - kStages); gg < g; ++gg) {
      const uint32_t par = static_cast<uint32_t>(gg / kStages) & 1;
      drain_wait_r(k_full(gg % kStages), par, p.status);
      drain_wait_r(v_full(gg % kStages), par, p.status);
    }
  }
}

// Keys of a tile that nobody sees but that were loaded with others' boxes: rows
// [a0, a1) before the window and [b0, b1) past the sequence.
struct HiddenRows {
  int a0, a1, b0, b1;
  __device__ __forceinline__ HiddenRows(const RaggedParams& p, const SeqKeys& k, int kv0) {
    a1 = min(max(k.first - kv0, 0), kTileN);
    a0 = max(a1 - (k.first & (p.box_rows - 1)), 0);
    b0 = min(max(k.len - kv0, 0), kTileN);
    b1 = min(b0 + (-k.len & (p.box_rows - 1)), kTileN);
    if (k.first < kv0 || k.first >= kv0 + kTileN) a0 = a1 = 0;
    if (k.len < kv0 || k.len >= kv0 + kTileN) b0 = b1 = 0;
  }
  __device__ __forceinline__ bool any() const { return a0 < a1 || b0 < b1; }
};

// Clears those rows of a V tile (`chunks` 64-column chunks of 128-byte rows), by
// 128 threads, a 16-byte unit each at a time.
template <int kChunks>
__device__ __forceinline__ void clear_rows(const HiddenRows& h, uint8_t* tile, int tid) {
  const int na = h.a1 - h.a0, n = na + h.b1 - h.b0;
  for (int i = tid; i < n * 8; i += 128) {
    const int r = (i >> 3) < na ? h.a0 + (i >> 3) : h.b0 + (i >> 3) - na;
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
      *reinterpret_cast<uint4*>(tile + c * (kTileN * 128) + r * 128 + (i & 7) * 16) =
          make_uint4(0u, 0u, 0u, 0u);
  }
}

// What a row's sum of weights (relative to 2^m) makes of a key range: the factor of O and
// the log2-sum. A sum of 0 is a range of which the row sees nothing (or only scores of
// -infinity): weight 0; a NaN stays one. (To tell the two apart where the range is all of
// the row's took the key form another value through its loop: 24 sequences of 4000
// keys, 8 rows of 4 tokens, d = 64: 38.2 us, 40.7 to 45.1 with it.)
struct PartSum {
  float inv, lse2;
  __device__ __forceinline__ PartSum(float l, float m) {
    inv = l == 0.f ? 0.f : 1.f / l;
    lse2 = l == 0.f ? -INFINITY : m + __log2f(l);
  }
};

// One barrier of a group of consecutive 8-byte barriers.
struct Bars {
  uint32_t base;
  __device__ __forceinline__ uint32_t operator()(int i) const { return base + 8 * i; }
};

// ------------------------------------------------- one thread per query row --
// (kLargeCap: p.large_cap. A kernel of its own: with the forms in it the other's loop is
// slower, 24 sequences of 2000 keys with 40 rows 20.2 us -> 21.4, of 4000 keys with 32
// rows at d = 64 38.1 -> 40.5.)
template <int D, bool kBf16, bool kLargeCap>
__global__ void __launch_bounds__(kThreads, 1)
    fa_ragged_kernel(const __grid_constant__ RaggedParams p) {
  using Cfg = RagCfg<D>;
  constexpr int NS = Cfg::kStages;
  using Elem = typename std::conditional<kBf16, __nv_bfloat16, __half>::type;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::kOffMisc + 4);
  int* scan = reinterpret_cast<int*>(smem + Cfg::kOffScan);

  const uint32_t q_ready = sbase + Cfg::kOffBar;
  const Bars k_full{q_ready + 8}, k_empty{k_full(NS)}, v_full{k_empty(NS)}, v_empty{v_full(NS)};
  const Bars s_full{v_empty(NS)}, p_full{s_full(2)}, pv_done{p_full(2)};
  const uint32_t drain = pv_done(2);

  const int warp = static_cast<int>(warp_id());
  const int lane = static_cast<int>(lane_id());
  const int cta = static_cast<int>(blockIdx.x);

  if (threadIdx.x == 0) {
    mbar_init(q_ready, 4);   // one arrival per row warp and segment
    for (int s = 0; s < NS; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), 1);
      mbar_init(v_full(s), 1);
      mbar_init(v_empty(s), 1);
    }
    for (int bb = 0; bb < 2; ++bb) {
      mbar_init(s_full(bb), 1);
      mbar_init(p_full(bb), 4);
      mbar_init(pv_done(bb), 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }

  tc_fence_before();
  const Share share = find_share(p, cta, scan);   // with the barriers that order the set-up
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // the merge kernel may be scheduled now; it waits for this grid's completion
  // before it reads anything
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  Segments seg(p, share);

  if (warp == 0) {
    produce<Cfg::kChunks, NS>(p, seg, sbase + Cfg::kOffK, sbase + Cfg::kOffV, k_full, k_empty,
                              v_full, v_empty, abort_flag);
  } else if (warp == 1) {
    // ===================== MMA issuer =====================
    // Tile g's Q K^T goes out ahead of tile g - 1's P V, except the first of a
    // segment, whose queries are staged after the segment before has been read.
    if (lane == 0) {
      constexpr uint32_t idesc_qk = make_idesc(128, kTileN, kBf16, false, false);
      constexpr uint32_t idesc_pv = make_idesc(128, D, kBf16, false, true);
      const uint64_t qa = make_sdesc(sbase + Cfg::kOffQ, 16, 1024);
      TileWalk walk{seg};
      int n_seg = 0;   // segments whose queries have been awaited
      auto issue_qk = [&](int g) -> bool {   // S_(g%2) = Q K_g^T
        const int st = g % NS;
        if (walk.first && !mbar_wait(q_ready, n_seg++ & 1, abort_flag, p.status)) return false;
        if (!mbar_wait(k_full(st), static_cast<uint32_t>(g / NS) & 1, abort_flag, p.status))
          return false;
        // S_(g%2) held P_(g-2), which P_(g-2) V_(g-2) must have read
        if (g >= 2 && !mbar_wait(pv_done(g & 1), static_cast<uint32_t>((g - 2) >> 1) & 1,
                                 abort_flag, p.status))
          return false;
        tc_fence_after();
        const uint64_t kb = make_sdesc(sbase + Cfg::kOffK + st * Cfg::kTileBytes, 16, 1024);
        mma_ss_product<D / 16, true, kTileM * 128, true, kTileN * 128>(tmem + (g & 1) * 128, qa, kb,
                                                                       idesc_qk, 0);
        tc_commit(s_full(g & 1));
        tc_commit(k_empty(st));
        return true;
      };
      bool ok = true, have = walk.next(p);
#ifdef FA_WAIT_TEST
      // wait-limit test build: nothing completes this phase before the abort
      // path's own commit, so the wait runs out
      if (have) ok = mbar_wait(drain, 0, abort_flag, p.status);
#endif
      if (ok && have) ok = issue_qk(0);
      for (int g = 0; ok && have; ++g) {
        const int st = g % NS;
        const bool first = walk.first;   // tile g is its segment's first
        have = walk.next(p);
        if (have && !walk.first && !(ok = issue_qk(g + 1))) break;
        if (!(ok = mbar_wait(p_full(g & 1), static_cast<uint32_t>(g >> 1) & 1, abort_flag, p.status)))
          break;
        if (!(ok = mbar_wait(v_full(st), static_cast<uint32_t>(g / NS) & 1, abort_flag, p.status)))
          break;
        tc_fence_after();
        const uint64_t vb = make_sdesc(sbase + Cfg::kOffV + st * Cfg::kTileBytes, kTileN * 128, 1024);
        mma_ts_product8<false, 0>(tmem + 256, tmem + (g & 1) * 128, vb, idesc_pv, first ? 0u : 1u);
        tc_commit(pv_done(g & 1));
        tc_commit(v_empty(st));
        if (have && walk.first && !(ok = issue_qk(g + 1))) break;
      }
      if (!ok) {
        // every MMA issued so far must finish before the TMEM is released
        tc_commit(drain);
        drain_wait_r(drain, 0, p.status);
      }
    }
  } else {
    // ===== row warps: stage Q, then softmax per key tile, then the write-out =====
    const int quarter = warp & 3;               // TMEM lane quarter of this warp
    const int r = quarter * 32 + lane;          // query-tile row
    const bool real = r < p.R;
    const bool busy = quarter * 32 < p.R;       // the warp holds real rows
    const int gq = real ? r / p.Sq : 0;
    const int s = real ? r % p.Sq : 0;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t o_tmem = tmem + lane_off + 256;
    const float c = p.mod.cap_in != 0.f ? 1.f : p.scale_log2;   // capped scores are in the log2 domain
    // Stage this row of a segment's queries into the 128-byte-swizzled K-major
    // query tile (16-byte unit u of a 128-byte row sits at unit u ^ (r % 8));
    // rows past R are zero.
    auto stage_q = [&](int b, int kvh) {
      const size_t qrow = (static_cast<size_t>(b) * p.Hq + kvh * p.G + gq) * p.Sq + s;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const Elem*>(p.q) + qrow * D);
#pragma unroll
      for (int cc = 0; cc < Cfg::kChunks; ++cc) {
        uint8_t* dst_row = smem + Cfg::kOffQ + cc * (kTileM * 128) + r * 128;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const uint4 v = real ? src[cc * 8 + u] : make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(dst_row + ((u ^ (r & 7)) << 4)) = v;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready);
    };

    bool more = seg.next(p);
    if (more) stage_q(seg.b, seg.kvh);
    bool ok = true;
    bool head = true;   // the share's first segment
    int g = 0;
    while (more && ok) {
      const int b = seg.b, kvh = seg.kvh, n = seg.n;
      const bool whole = seg.whole;
      const SeqKeys keys = seg.keys;
      const int tile0 = seg.tile0;
      const int hq = kvh * p.G + gq;
      const int pos = keys.len - p.Sq + s;
      // keys [row_lo, row_hi) of this row; rows past R see what any row does
      int row_lo = keys.first, row_hi = keys.len;
      if (real) {
        row_hi = max(pos + 1, 0);
        row_lo = p.window > 0 ? max(0, pos + 1 - p.window) : 0;
      }
      const float bias = p.mod.slopes ? p.mod.slopes[hq] * (kLog2eR / c) : 0.f;
      float m_ref = -INFINITY;   // reference max, scaled log2 domain
      float l = 0.f;
      for (int j = 0; j < n; ++j, ++g) {
        const uint32_t s_tmem = tmem + lane_off + (g & 1) * 128;
        const int kv0 = (tile0 + j) * kTileN;
        ok = __all_sync(0xffffffffu, mbar_wait(s_full(g & 1), static_cast<uint32_t>(g >> 1) & 1,
                                               abort_flag, p.status));
        if (!ok) break;
        tc_fence_after();
        const HiddenRows hidden(p, keys, kv0);
        if (hidden.any()) {
          const int st = g % NS;
          ok = __all_sync(0xffffffffu, mbar_wait(v_full(st), static_cast<uint32_t>(g / NS) & 1,
                                                 abort_flag, p.status));
          if (!ok) break;
          clear_rows<Cfg::kChunks>(hidden, smem + Cfg::kOffV + st * Cfg::kTileBytes, r);
          fence_proxy_async_smem();
        }
        if (busy) {
          float sc[kTileN];
          {
            uint32_t raw[kTileN];
#pragma unroll
            for (int cc = 0; cc < kTileN / 32; ++cc)
              tmem_ld32(s_tmem + cc * 32, *reinterpret_cast<uint32_t(*)[32]>(raw + cc * 32));
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < kTileN; ++i) sc[i] = __uint_as_float(raw[i]);
          }
          if constexpr (kLargeCap) {
            if (hidden.any()) {   // keys that may hold anything do not choose the cap's form
#pragma unroll
              for (int h = 0; h < kTileN / 32; ++h) {
                const uint32_t w = span_bits(keys.first, keys.len, kv0 + h * 32);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (!((w >> i) & 1u)) sc[h * 32 + i] = 0.f;
              }
            }
            cap_scores(sc, warp_abs_max(sc), p.mod);
          } else if (p.mod.cap_in != 0.f) {
#pragma unroll
            for (int i = 0; i < kTileN; ++i) sc[i] = cap_exact(sc[i], p.mod);
          }
          if (p.mod.slopes) {
            const float d0 = static_cast<float>(kv0 - pos);
#pragma unroll
            for (int i = 0; i < kTileN; ++i)
              sc[i] = fmaf(-bias, fabsf(d0 + static_cast<float>(i)), sc[i]);
          }
          if (kv0 < row_lo || kv0 + kTileN > row_hi) {
#pragma unroll
            for (int h = 0; h < kTileN / 32; ++h) {
              const uint32_t w = span_bits(row_lo, row_hi, kv0 + h * 32);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((w >> i) & 1u)) sc[h * 32 + i] = -INFINITY;
            }
          }
          float mx0 = sc[0], mx1 = sc[1], mx2 = sc[2], mx3 = sc[3];
#pragma unroll
          for (int i = 4; i < kTileN; i += 4) {
            mx0 = fmaxf(mx0, sc[i]);
            mx1 = fmaxf(mx1, sc[i + 1]);
            mx2 = fmaxf(mx2, sc[i + 2]);
            mx3 = fmaxf(mx3, sc[i + 3]);
          }
          const float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * c;
          float m_new = m_ref;
          if (mx > m_ref + kRescaleThresholdR) m_new = mx;
          const float m_use = (m_new == -INFINITY) ? 0.f : m_new;
          const float alpha = ex2(m_ref - m_use);   // 0 when m_ref = -inf
          const bool moved = (m_new != m_ref);
          m_ref = m_new;

          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          uint32_t pk[32];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float p0 = ex2(fmaf(sc[h * 64 + 2 * i], c, -m_use));
              const float p1 = ex2(fmaf(sc[h * 64 + 2 * i + 1], c, -m_use));
              sum[(2 * i) & 3] += p0;
              sum[(2 * i + 1) & 3] += p1;
              pk[i] = pack2<kBf16>(p0, p1);
            }
            tmem_st32(s_tmem + h * 32, pk);
          }
          l = l * alpha + ((sum[0] + sum[1]) + (sum[2] + sum[3]));

          // O <- alpha * O for rows whose reference max moved (the segment's
          // first P V overwrites O)
          if (j > 0 && __any_sync(0xffffffffu, moved)) {
            ok = __all_sync(0xffffffffu, mbar_wait(pv_done((g - 1) & 1),
                                                   static_cast<uint32_t>((g - 1) >> 1) & 1,
                                                   abort_flag, p.status));
            if (!ok) break;
            tc_fence_after();
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
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(g & 1));
      }
      if (!ok) break;
      // the next segment's queries (every Q K^T of this one has been read), then
      // this segment's result
      more = seg.next(p);
      if (more) stage_q(seg.b, seg.kvh);
      if (busy) {
        ok = __all_sync(0xffffffffu, mbar_wait(pv_done((g - 1) & 1),
                                               static_cast<uint32_t>((g - 1) >> 1) & 1, abort_flag,
                                               p.status));
        if (!ok) break;
        tc_fence_after();
        const PartSum sum(l, m_ref);
        const size_t qrow = (static_cast<size_t>(b) * p.Hq + hq) * p.Sq + s;
        const size_t prow = (static_cast<size_t>(cta) * 2 + (head ? 0 : 1)) * p.R + r;
#pragma unroll
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t o[32];
          tmem_ld32(o_tmem + cc * 32, o);
          tmem_wait_ld();
          if (!real) continue;
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<Elem*>(p.out) + qrow * D + cc * 32);
#pragma unroll
            for (int v = 0; v < 4; ++v)
              dst[v] = make_uint4(
                  pack2<kBf16>(__uint_as_float(o[8 * v]) * sum.inv, __uint_as_float(o[8 * v + 1]) * sum.inv),
                  pack2<kBf16>(__uint_as_float(o[8 * v + 2]) * sum.inv, __uint_as_float(o[8 * v + 3]) * sum.inv),
                  pack2<kBf16>(__uint_as_float(o[8 * v + 4]) * sum.inv, __uint_as_float(o[8 * v + 5]) * sum.inv),
                  pack2<kBf16>(__uint_as_float(o[8 * v + 6]) * sum.inv, __uint_as_float(o[8 * v + 7]) * sum.inv));
          } else {
            float4* dst = reinterpret_cast<float4*>(p.part_out + prow * D + cc * 32);
#pragma unroll
            for (int v = 0; v < 8; ++v)
              dst[v] = make_float4(__uint_as_float(o[4 * v]) * sum.inv, __uint_as_float(o[4 * v + 1]) * sum.inv,
                                   __uint_as_float(o[4 * v + 2]) * sum.inv, __uint_as_float(o[4 * v + 3]) * sum.inv);
          }
        }
        if (real && whole) p.lse[qrow] = sum.lse2 * kLn2R;
        if (real && !whole) p.part_lse2[prow] = sum.lse2;
        tc_fence_before();
      }
      head = false;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ----------------------------------------------------- one thread per key --
// The form for few rows (R <= NR; 16, or 32 with a cap: launch_form): the products are transposed, so that
// the keys fill the 128 tensor-memory lanes and the rows are the short side,
//
//   S^T = K Q^T  (keys x NR),   O^T += V^T P  (d x NR, P as stored: rows x keys),
//
// and each of the 128 threads takes one key's NR scores. Where the form above
// has one warp do 128 exponentials a thread (for R <= 32; the other three idle),
// here all four warps do NR each. P goes through shared memory, its own buffer,
// so the score buffers are free as soon as they are read. The running maximum of
// a row is common to all keys of a tile, so all threads: it moves only when some
// score exceeds it by 2^8, which one barrier with a vote finds out; then the
// warps exchange their maxima and rescale O^T. Row sums stay with the threads
// until the end of a segment.
//
// At d = 64 the V tile has one 64-column chunk, but the product's M is 128: its
// second half reads the 16 KB behind the tile (the next V or K buffer) into
// lanes 64 .. 127, which nobody reads.
template <int D, int NR>
struct RagTCfg {
  static constexpr int kChunks = D / kChunk;
  static constexpr int kTileBytes = kTileM * D * 2;
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kQBytes = NR * D * 2;        // [chunk][NR rows][128 bytes]
  static constexpr int kPBytes = NR * kTileN * 2;   // [64-key chunk][NR rows][128 bytes]
  static constexpr int kOffV = 0;
  static constexpr int kOffK = kStages * kTileBytes;
  static constexpr int kOffQ = 2 * kStages * kTileBytes;   // two buffers
  static constexpr int kOffP = kOffQ + 2 * kQBytes;        // two buffers
  static constexpr int kOffBar = kOffP + 2 * kPBytes;
  // k_full[S], k_empty[S], v_full[S], v_empty[S], q_ready[2], s_full[2],
  // s_free[2], p_full[2], pv_done[2], drain
  static constexpr int kNumBars = 4 * kStages + 10 + 1;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kOffScan = kOffMisc + 16;
  static constexpr int kOffRed = (kOffScan + 32 + 15) / 16 * 16;   // [2][NR][4 warps] floats
  static constexpr int kOffRow = kOffRed + 2 * NR * 16;            // [2][NR]: slope, token of the row
  static constexpr int kSmemBytes = kOffRow + 2 * NR * 4 + 1024;   // + alignment slack
  static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
};

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Sums of N columns over the warp's lanes: each exchange halves the columns a
// lane holds (the lanes of a pair keep one half each), so N columns take N
// shuffles; lane l ends with the sum of column l % N (both lanes l and l + 16 for
// N = 16).
template <int N>
__device__ __forceinline__ float column_sums(float (&v)[N], int lane) {
  static_assert(N == 16 || N == 32, "columns");
#pragma unroll
  for (int h = N / 2; h > 0; h >>= 1) {
    const bool up = (lane & h) != 0;   // keeps the upper half of its columns
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float keep = up ? v[i + h] : v[i], give = up ? v[i] : v[i + h];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, h);
    }
  }
  if (N == 16) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 16);
  return v[0];
}

// Barrier of the four row warps that tells whether any thread's flag is set.
__device__ __forceinline__ bool row_warps_any(bool flag) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any) : "r"(flag ? 1u : 0u) : "memory");
  return any != 0;
}

template <int N>
__device__ __forceinline__ void tmem_ld_n(uint32_t addr, uint32_t (&r)[N]) {
  if constexpr (N == 16) tmem_ld16(addr, r);
  else tmem_ld32(addr, r);
}
template <int N>
__device__ __forceinline__ void tmem_st_n(uint32_t addr, const uint32_t (&r)[N]) {
  if constexpr (N == 16) tmem_st16(addr, r);
  else tmem_st32(addr, r);
}

template <int D, int NR, bool kBf16, bool kLargeCap>
__global__ void __launch_bounds__(kThreads, 1)
    fa_ragged_keys_kernel(const __grid_constant__ RaggedParams p) {
  using Cfg = RagTCfg<D, NR>;
  constexpr int NS = Cfg::kStages;
  using Elem = typename std::conditional<kBf16, __nv_bfloat16, __half>::type;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::kOffMisc + 4);
  float4* red = reinterpret_cast<float4*>(smem + Cfg::kOffRed);   // [NR] maxima, one float a warp
  float4* red_sum = red + NR;                                     // [NR] sums

  const Bars k_full{sbase + Cfg::kOffBar}, k_empty{k_full(NS)}, v_full{k_empty(NS)};
  const Bars v_empty{v_full(NS)}, q_ready{v_empty(NS)}, s_full{q_ready(2)}, s_free{s_full(2)};
  const Bars p_full{s_free(2)}, pv_done{p_full(2)};
  const uint32_t drain = pv_done(2);

  const int warp = static_cast<int>(warp_id());
  const int lane = static_cast<int>(lane_id());
  const int cta = static_cast<int>(blockIdx.x);

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), 1);
      mbar_init(v_full(s), 1);
      mbar_init(v_empty(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_ready(i), 4);   // one arrival per row warp
      mbar_init(s_full(i), 1);
      mbar_init(s_free(i), 4);
      mbar_init(p_full(i), 4);
      mbar_init(pv_done(i), 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  // tensor memory: S^T buffers at columns 0 and 32, O^T at 64
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 128);
    tmem_relinquish();
  }
  tc_fence_before();
  const Share share = find_share(p, cta, reinterpret_cast<int*>(smem + Cfg::kOffScan));
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // the merge kernel may be scheduled now; it waits for this grid's completion
  // before it reads anything
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  Segments seg(p, share);

  if (warp == 0) {
    produce<Cfg::kChunks, NS>(p, seg, sbase + Cfg::kOffK, sbase + Cfg::kOffV, k_full, k_empty,
                              v_full, v_empty, abort_flag);
  } else if (warp == 1) {
    // ===================== MMA issuer =====================
    if (lane == 0) {
      constexpr uint32_t idesc_s = make_idesc(128, NR, kBf16, false, false);
      constexpr uint32_t idesc_o = make_idesc(128, NR, kBf16, true, false);
      TileWalk walk{seg};
      int n_seg = 0;   // segments begun
      auto issue_s = [&](int g) -> bool {   // S^T_(g%2) = K_g Q^T
        const int st = g % NS;
        if (walk.first) {
          if (!mbar_wait(q_ready(n_seg & 1), (n_seg >> 1) & 1, abort_flag, p.status)) return false;
          ++n_seg;
        }
        if (!mbar_wait(k_full(st), static_cast<uint32_t>(g / NS) & 1, abort_flag, p.status))
          return false;
        if (g >= 2 && !mbar_wait(s_free(g & 1), static_cast<uint32_t>((g - 2) >> 1) & 1, abort_flag,
                                 p.status))
          return false;
        tc_fence_after();
        const uint64_t ka = make_sdesc(sbase + Cfg::kOffK + st * Cfg::kTileBytes, 16, 1024);
        const uint64_t qb = make_sdesc(sbase + Cfg::kOffQ + ((n_seg - 1) & 1) * Cfg::kQBytes, 16, 1024);
        mma_ss_product<D / 16, true, kTileN * 128, true, NR * 128>(tmem + (g & 1) * 32, ka, qb,
                                                                   idesc_s, 0);
        tc_commit(s_full(g & 1));
        tc_commit(k_empty(st));
        return true;
      };
      bool ok = true, have = walk.next(p);
#ifdef FA_WAIT_TEST
      // wait-limit test build: nothing completes this phase before the abort
      // path's own commit, so the wait runs out
      if (have) ok = mbar_wait(drain, 0, abort_flag, p.status);
#endif
      if (ok && have) ok = issue_s(0);
      for (int g = 0; ok && have; ++g) {
        const int st = g % NS;
        const bool first = walk.first;   // tile g is its segment's first
        have = walk.next(p);
        if (have && !(ok = issue_s(g + 1))) break;
        if (!(ok = mbar_wait(p_full(g & 1), static_cast<uint32_t>(g >> 1) & 1, abort_flag, p.status)))
          break;
        if (!(ok = mbar_wait(v_full(st), static_cast<uint32_t>(g / NS) & 1, abort_flag, p.status)))
          break;
        tc_fence_after();
        const uint64_t va = make_sdesc(sbase + Cfg::kOffV + st * Cfg::kTileBytes, kTileN * 128, 1024);
        const uint64_t pb = make_sdesc(sbase + Cfg::kOffP + (g & 1) * Cfg::kPBytes, 16, 1024);
        mma_ss_product<kTileN / 16, false, 0, true, NR * 128>(tmem + 64, va, pb, idesc_o,
                                                              first ? 0u : 1u);
        tc_commit(pv_done(g & 1));
        tc_commit(v_empty(st));
      }
      if (!ok) {
        // every MMA issued so far must finish before the TMEM is released
        tc_commit(drain);
        drain_wait_r(drain, 0, p.status);
      }
    }
  } else {
    // ===== row warps: thread = key of the tile, and dimension of O^T =====
    const int quarter = warp & 3;               // TMEM lane quarter of this warp
    const int t = quarter * 32 + lane;          // key of the tile; dimension
    const int tid = static_cast<int>(threadIdx.x) - 64;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t o_tmem = tmem + lane_off + 64;
    const bool cap = NR == 32 || p.mod.cap_in != 0.f;
    const bool same_rows = p.Sq == 1 && !p.mod.slopes;   // rows do not differ in position or slope
    const float c = p.scale_log2;
    float* row_slope = reinterpret_cast<float*>(smem + Cfg::kOffRow);          // log2 domain
    int* row_s = reinterpret_cast<int*>(smem + Cfg::kOffRow + NR * 4);         // token of the row

    // A segment's queries: R rows that follow each other in memory. 16-byte unit
    // u of a 128-byte row r sits at unit u ^ (r % 8); rows past R are zero.
    constexpr int kUnits = NR * D / 8 / 128;    // 16-byte units a thread
    uint4 qv[kUnits];
    auto load_q = [&](const Segments& sg) {
      const size_t row0 = (static_cast<size_t>(sg.b) * p.Hq + sg.kvh * p.G) * p.Sq;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const Elem*>(p.q) + row0 * D);
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const int u = tid + i * 128;
        qv[i] = u / (D / 8) < p.R ? src[u] : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    auto stage_q = [&](int buffer) {
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const int u = tid + i * 128, row = u / (D / 8), col = u % (D / 8);
        *reinterpret_cast<uint4*>(smem + Cfg::kOffQ + buffer * Cfg::kQBytes + (col >> 3) * (NR * 128) +
                                  row * 128 + (((col & 7) ^ (row & 7)) << 4)) = qv[i];
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready(buffer));
    };
    // this thread's place in a P buffer: row r of 64-key chunk t / 64, key t % 64
    const uint32_t p_dst = sbase + Cfg::kOffP + (t >> 6) * (NR * 128) + (t & 7) * 2;
    const uint32_t p_unit = static_cast<uint32_t>((t & 63) >> 3);

    bool more = seg.next(p);
    if (more) {
      load_q(seg);
      stage_q(0);
    }
    // A wait that fails in one warp must not leave the others in a barrier: the
    // warp goes on without touching anything until the next vote, where all four
    // learn of it and leave together.
    bool ok = true;     // no wait of this warp has failed
    bool dead = false;  // voted: some warp's has
    bool head = true;   // the share's first segment
    int g = 0;
    auto wait = [&](uint32_t bar, int phase) {
      if (ok)
        ok = __all_sync(0xffffffffu, mbar_wait(bar, static_cast<uint32_t>(phase) & 1, abort_flag, p.status));
    };
    for (int n_seg = 0; more && !dead; ++n_seg) {
      const int b = seg.b, kvh = seg.kvh, n = seg.n;
      const bool whole = seg.whole;
      const SeqKeys keys = seg.keys;
      const int tile0 = seg.tile0;
      const int pos0 = keys.len - p.Sq;   // position of row s = 0
      // rows' slopes and tokens (the readers of the segment before are past its last vote)
      if (!same_rows && tid < NR) {
        const int gq = min(tid, p.R - 1) / p.Sq;
        row_s[tid] = tid < p.R ? tid - gq * p.Sq : 0;
        row_slope[tid] = p.mod.slopes ? p.mod.slopes[kvh * p.G + gq] * kLog2eR : 0.f;
      }
      more = seg.next(p);
      if (more) load_q(seg);   // the next segment's, stored after the first tile
      float m[NR], l[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        m[r] = -INFINITY;   // reference max, scaled log2 domain
        l[r] = 0.f;         // this thread's part of the row sum
      }
      for (int j = 0; j < n; ++j, ++g) {
        const int kv0 = (tile0 + j) * kTileN;
        const int key = kv0 + t;
        wait(s_full(g & 1), g >> 1);
        tc_fence_after();
        float x[NR];
        {
          uint32_t raw[NR];
          tmem_ld_n<NR>(tmem + lane_off + (g & 1) * 32, raw);
          tmem_wait_ld();
#pragma unroll
          for (int r = 0; r < NR; ++r) x[r] = __uint_as_float(raw[r]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_free(g & 1));
        if constexpr (kLargeCap) {
          if (key < keys.first || key >= keys.len) {   // a key that may hold anything does not
#pragma unroll
            for (int r = 0; r < NR; ++r) x[r] = 0.f;   // choose the cap's form
          }
          cap_scores(x, warp_abs_max(x), p.mod);
        } else if (cap) {
#pragma unroll
          for (int r = 0; r < NR; ++r) x[r] = cap_exact(x[r], p.mod);
        } else {
#pragma unroll
          for (int r = 0; r < NR; ++r) x[r] *= c;
        }
        if (j == 0 && !same_rows) row_warps_any(false);   // row_slope and row_s are written
        if (p.mod.slopes) {
#pragma unroll
          for (int r = 0; r < NR; ++r)
            x[r] = fmaf(-row_slope[r], fabsf(static_cast<float>(pos0 + row_s[r] - key)), x[r]);
        }
        // the first row sees keys up to pos0, the last from first + Sq - 1 on (window)
        if (kv0 + kTileN > pos0 + 1 || (p.window > 0 && kv0 < pos0 + p.Sq - p.window)) {
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const int pos = same_rows ? pos0 : pos0 + row_s[r];
            if (key > pos || (p.window > 0 && key <= pos - p.window)) x[r] = -INFINITY;
          }
        }
        const HiddenRows hidden(p, keys, kv0);
        if (hidden.any()) {
          const int st = g % NS;
          wait(v_full(st), g / NS);
          if (ok) clear_rows<Cfg::kChunks>(hidden, smem + Cfg::kOffV + st * Cfg::kTileBytes, tid);
        }
        float over = -INFINITY;   // how far a score exceeds its row's reference
#pragma unroll
        for (int r = 0; r < NR; ++r) over = fmaxf(over, x[r] - m[r]);
        // (a segment's first tile sets them; the last vote, at the end of the segment
        // before, was after the last use of `red`)
        if (j == 0 || row_warps_any(over > kRescaleThresholdR || !ok)) {
          // move every row's reference to its maximum so far
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const float v = warp_max(x[r]);
            if (lane == 0) reinterpret_cast<float*>(red + r)[quarter] = v;
          }
          // P_(g-1) V_(g-1) is in O^T (the segment's first product overwrites it)
          if (j > 0) wait(pv_done((g - 1) & 1), (g - 1) >> 1);
          if ((dead = row_warps_any(!ok))) break;
          tc_fence_after();
          uint32_t o[NR];
          if (j > 0) {
            tmem_ld_n<NR>(o_tmem, o);
            tmem_wait_ld();
          }
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const float4 v = red[r];
            const float m_new = fmaxf(fmaxf(m[r], fmaxf(v.x, v.y)), fmaxf(v.z, v.w));
            const float alpha = m_new == -INFINITY ? 1.f : ex2(m[r] - m_new);   // 0 from m = -inf
            m[r] = m_new;
            l[r] *= alpha;
            if (j > 0) o[r] = __float_as_uint(__uint_as_float(o[r]) * alpha);
          }
          if (j > 0) {
            tmem_st_n<NR>(o_tmem, o);
            tmem_wait_st();
          }
        }
        if (g >= 2) wait(pv_done(g & 1), (g - 2) >> 1);   // P_(g-2) V_(g-2) has read this P buffer
        if (!ok) continue;   // to the next vote
        const uint32_t dst = p_dst + (g & 1) * Cfg::kPBytes;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const float e = ex2(x[r] - (m[r] == -INFINITY ? 0.f : m[r]));
          l[r] += e;
          const uint32_t h = pack2<kBf16>(e, 0.f);
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst + r * 128 + ((p_unit ^ (r & 7)) << 4)),
                       "h"(static_cast<uint16_t>(h)) : "memory");
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(g & 1));
        if (j == 0 && more) stage_q((n_seg + 1) & 1);
      }
      if (dead) break;
      // row sums over the 128 keys
      const float sum_l = column_sums<NR>(l, lane);
      if (lane < NR) reinterpret_cast<float*>(red_sum + lane)[quarter] = sum_l;
      wait(pv_done((g - 1) & 1), (g - 1) >> 1);
      if ((dead = row_warps_any(!ok))) break;
      tc_fence_after();
      uint32_t o[NR];
      tmem_ld_n<NR>(o_tmem, o);
      tmem_wait_ld();
      tc_fence_before();
      const size_t qrow = (static_cast<size_t>(b) * p.Hq + kvh * p.G) * p.Sq;   // + r
      const size_t prow = (static_cast<size_t>(cta) * 2 + (head ? 0 : 1)) * p.R;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        if (r >= p.R) break;
        const float4 v = red_sum[r];
        const PartSum sum((v.x + v.y) + (v.z + v.w), m[r]);
        const float y = __uint_as_float(o[r]) * sum.inv;
        if (t < D) {
          if (whole) static_cast<Elem*>(p.out)[(qrow + r) * D + t] = static_cast<Elem>(y);
          else p.part_out[(prow + r) * D + t] = y;
        }
        if (tid == 0) {
          if (whole) p.lse[qrow + r] = sum.lse2 * kLn2R;
          else p.part_lse2[prow + r] = sum.lse2;
        }
      }
      head = false;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 128);
  }
}

// ------------------------------------------------------------------ merge --
// Joins the parts of (sequence, head)s whose tiles lie in more than one share, in
// share order, as the split-KV merge does: block (c, y) takes rows [kMergeRows y,
// + kMergeRows) of the one whose second part is in share c, one warp a row, each
// lane d / 32 columns. So the grid goes by the shares, not by the batch, most of
// whose rows one segment has written whole (against a warp for every row: one
// sequence of 65536 keys 51.4 -> 50.1 us). Also writes out = 0, LSE = -inf for
// sequences without keys.
constexpr int kMergeRows = 4;     // rows (warps) a block: fits beside the ragged kernel's CTA
constexpr int kMergeBatch = 20;   // 152 shares of one sequence with 8 heads: 20 parts a head
template <int PER>
struct alignas(4 * PER) PartVec { float x[PER]; };

template <typename T, int PER>
__global__ void __launch_bounds__(32 * kMergeRows) ragged_merge_kernel(const __grid_constant__ RaggedParams p) {
  // programmatic dependent of the ragged kernel: wait until that grid has
  // completed and its results are visible; a ragged kernel that follows on the
  // stream may set itself up beside this grid
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int D = 32 * PER;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = static_cast<int>(blockIdx.x);
  if (blockIdx.y == 0) {
    for (int b = c; b < p.B; b += static_cast<int>(gridDim.x)) {
      if (seq_keys(p, b).n > 0) continue;
      const long long rows = static_cast<long long>(p.Hq) * p.Sq;
      for (long long i = warp; i < rows; i += kMergeRows) {
        const long long row = b * rows + i;
        T* dst = static_cast<T*>(p.out) + row * D + lane * PER;
#pragma unroll
        for (int e = 0; e < PER; ++e) dst[e] = static_cast<T>(0.f);
        if (lane == 0) p.lse[row] = -INFINITY;
      }
    }
  }
  const int r = static_cast<int>(blockIdx.y) * kMergeRows + warp;
  const int total = p.starts[0].w;
  const int4 start = p.starts[c];   // without meaning past the shares
  const ShareOut out(p.n_ctas, total * p.Hkv);
  if (c == 0 || c >= out.shares || r >= p.R) return;
  const int b = start.x, units = start.z;
  const int kvh = (out.begin(c) - start.y * p.Hkv) / units;
  const int u0 = start.y * p.Hkv + kvh * units;   // this head's units: [u0, u0 + units)
  const int c0 = out.of_unit(u0 + kSegmentUnits), c1 = out.of_unit(u0 + units - 1);
  if (c != c0 + 1 || c0 == c1) return;
  // the parts are the first segments of their shares, but for that of c0 when
  // its share begins before this head's units (and so with another's tiles)
  const bool tail0 = out.begin(c0) < u0;
  auto part = [&](int i) {
    return (static_cast<size_t>(i) * 2 + ((i == c0 && tail0) ? 1 : 0)) * p.R + r;
  };
  // Bound by latency (a few KB a row): a batch's loads go out together, the first
  // batch's with those of the maximum over all parts.
  PartVec<PER> v[kMergeBatch];
  float lv[kMergeBatch];
  auto load = [&](int i) {
#pragma unroll
    for (int k = 0; k < kMergeBatch; ++k)
      if (i + k <= c1) {
        const size_t at = part(i + k);
        v[k] = reinterpret_cast<const PartVec<PER>*>(p.part_out + at * D)[lane];
        lv[k] = p.part_lse2[at];
      }
  };
  load(c0);
  float M = -INFINITY;
  for (int i = c0 + lane; i <= c1; i += 32) M = fmaxf(M, p.part_lse2[part(i)]);
  M = warp_max(M);   // without NaN parts: their weight is NaN whatever it is
  if (M == -INFINITY) M = 0.f;
  float acc[PER], L = 0.f;
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = 0.f;
  for (int i = c0; i <= c1; i += kMergeBatch) {
    if (i > c0) load(i);
#pragma unroll
    for (int k = 0; k < kMergeBatch; ++k)
      if (i + k <= c1) {
        const float w = ex2(lv[k] - M);
        L += w;
#pragma unroll
        for (int e = 0; e < PER; ++e) acc[e] = fmaf(w, v[k].x[e], acc[e]);
      }
  }
  const PartSum sum(L, M);
  const int gq = r / p.Sq;
  const long long row = (static_cast<long long>(b) * p.Hq + kvh * p.G + gq) * p.Sq + r - gq * p.Sq;
  T* dst = static_cast<T*>(p.out) + row * D + lane * PER;
#pragma unroll
  for (int e = 0; e < PER; ++e) dst[e] = static_cast<T>(acc[e] * sum.inv);
  if (lane == 0) p.lse[row] = sum.lse2 * kLn2R;
}

template <int smem, class Kernel>
cudaError_t launch_main(Kernel kernel, const RaggedParams& p, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, dim3(static_cast<unsigned>(p.n_ctas)), dim3(kThreads), smem, stream, p);
}

// The form by the rows R of a key/value head and whether there is a cap. Measured (us, each
// a thread a key | a thread a row; bf16; A: 40 sequences of 4000 keys, 2 key/value heads,
// B: one of 500 keys, 4 heads):
//            d = 128: A    A, cap 50          B     d = 64: A    A, cap 50          B
//   R =  4  35.9 | 41.1  36.1 | 65.8  10.1 | 11.3  26.8 | 30.6  27.4 | 56.1   9.3 | 9.4
//   R = 16  39.4 | 42.5  39.5 | 66.9  11.5 | 11.3  31.9 | 30.7  32.4 | 56.1  11.1 | 9.4
//   R = 20  51.1 | 43.2  54.4 | 67.4  14.4 | 12.0  39.2 | 31.0  42.9 | 56.0  13.5 | 9.8
//   R = 32  63.9 | 45.0  64.5 | 68.9  16.2 | 11.6  48.5 | 32.0  51.6 | 56.8  15.4 | 9.5
// A thread a key shares the exponentials of few rows among four warps; its work grows with
// the rows, that of a thread a row does not, until a cap doubles the special functions.
template <int D, bool kBf16, bool kLargeCap>
cudaError_t launch_form(const RaggedParams& p, cudaStream_t stream) {
  if (p.R <= 16)
    return launch_main<RagTCfg<D, 16>::kSmemBytes>(fa_ragged_keys_kernel<D, 16, kBf16, kLargeCap>, p, stream);
  if (p.R <= 32 && p.mod.cap_in != 0.f)
    return launch_main<RagTCfg<D, 32>::kSmemBytes>(fa_ragged_keys_kernel<D, 32, kBf16, kLargeCap>, p, stream);
  return launch_main<RagCfg<D>::kSmemBytes>(fa_ragged_kernel<D, kBf16, kLargeCap>, p, stream);
}

template <int D, bool kBf16>
cudaError_t launch_ragged_impl(const RaggedParams& p, cudaStream_t stream) {
  using Elem = typename std::conditional<kBf16, __nv_bfloat16, __half>::type;
  const cudaError_t e = p.large_cap ? launch_form<D, kBf16, true>(p, stream)
                                    : launch_form<D, kBf16, false>(p, stream);
  if (e != cudaSuccess) return e;
  // the merge overlaps its launch with the ragged kernel's tail
  return launch_dependent(ragged_merge_kernel<Elem, D / 32>,
                          dim3(static_cast<unsigned>(p.n_ctas),
                               static_cast<unsigned>((p.R + kMergeRows - 1) / kMergeRows)),
                          dim3(32 * kMergeRows), 0, stream, p);
}

}  // namespace

cudaError_t launch_ragged(const RaggedParams& p, int d, bool bf16, cudaStream_t stream) {
  if (d == 128)
    return bf16 ? launch_ragged_impl<128, true>(p, stream) : launch_ragged_impl<128, false>(p, stream);
  return bf16 ? launch_ragged_impl<64, true>(p, stream) : launch_ragged_impl<64, false>(p, stream);
}

}  // namespace fa
