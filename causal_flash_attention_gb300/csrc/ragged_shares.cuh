// How the key tiles of sequences of unequal length, known on the device only, are shared
// out over one wave of CTAs: the list of all tiles, even shares of it, and a share's
// segments. Shared by the ragged decode kernels (fa_ragged.cu, fa_latent_decode.cu).
//
// P is a kernel's parameter struct with B, Hkv (parts of a sequence's tiles that are
// listed after one another: key/value heads), Sq, window, capacity, box_rows, seq_lens,
// starts and n_ctas (shares at most), and kTileKeys, the keys of a tile.
#pragma once

#include "fa_internal.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kRaggedThreads = 192;

// Keys of one sequence that any of its rows sees, and their tiles.
struct SeqKeys {
  int len, first;     // keys [first, len)
  int tile0, n;       // tiles [tile0, tile0 + n)
};

template <class P>
__device__ __forceinline__ SeqKeys seq_keys(const P& p, int b) {
  SeqKeys s;
  s.len = min(max(p.seq_lens[b], 0), p.capacity);
  s.first = p.window > 0 ? max(0, s.len - p.Sq + 1 - p.window) : 0;
  s.tile0 = s.first / P::kTileKeys;
  s.n = s.len > 0 ? (s.len + P::kTileKeys - 1) / P::kTileKeys - s.tile0 : 0;
  return s;
}

// The list that is shared out counts units: one a key tile and kSegmentUnits for
// every (sequence, head) that has tiles, in front of them, for what a segment
// costs beside its tiles. Measured at 32 + 8 heads, d = 128, 66137 keys in 16
// sequences of 8 to 8192 and (second) 65521 + 15 x 1 keys: with no such units one
// CTA got dozens of one-tile segments, 70.1 and 119 us; 1 unit 60.5 and 69.1; 2
// units 52.5 and 54.2; 3 units 53.1 and 54.1. The latent decode (64-key tiles, a part of up to 128
// KB), with 1, 2, 3 and 5 units: 16 sequences of up to 8192 rows, 128 heads 45.0, 43.0, 43.3, 43.3 us, 16 heads
// 26.9, 27.3, 27.3, 27.2; trees over 3 x 20000 rows 40.2, 37.9, 37.8, 38.2; 60 windows of 512 rows 13.5, 12.9, 13.5,
// 13.8; 120 sequences of up to 300 rows 17.9, 18.3, 18.9, 19.0; one of 500 rows 9.7, 10.7, 10.7, 10.7.
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

// A CTA's share, found by all its kThreads threads (scan: kThreads / 32 + 2 words): a scan over the sequences' units. Where it
// begins is also written for the merge: (sequence, units per head before it, its units,
// units of all sequences per head). Two barriers.
struct Share {
  int begin, end;    // units of the list
  int b, pre;        // the first unit's sequence, and units per head before it
};

template <int kThreads = kRaggedThreads, class P>
__device__ __forceinline__ Share find_share(const P& p, int cta, int* scan) {
  constexpr int kWarps = kThreads / 32;
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
  for (int w = 0; w < kWarps; ++w) {
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
      scan[kWarps] = b;
      scan[kWarps + 1] = pre;
      p.starts[cta] = make_int4(b, pre, n, total);
    }
    pre += n;
  }
  if (total == 0 && cta == 0 && threadIdx.x == 0) p.starts[0] = make_int4(0, 0, 0, 0);
  __syncthreads();
  s.b = s.begin < s.end ? scan[kWarps] : 0;
  s.pre = s.begin < s.end ? scan[kWarps + 1] : 0;
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

  template <class P>
  __device__ __forceinline__ Segments(const P& p, const Share& s)
      : cur(s.begin), end(s.end), pre(s.pre), b(s.b) {
    if (cur < end) keys = seq_keys(p, b);
  }
  template <class P>
  __device__ __forceinline__ bool next(const P& p) {
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
  template <class P>
  __device__ __forceinline__ bool next(const P& p) {
    first = left == 0;
    if (first) {
      if (!seg.next(p)) return false;
      left = seg.n;
    }
    --left;
    return true;
  }
};

// Keys of a tile that nobody sees but that were loaded with others' boxes: rows
// [a0, a1) before the window and [b0, b1) past the sequence.
struct HiddenRows {
  int a0, a1, b0, b1;
  template <class P>
  __device__ __forceinline__ HiddenRows(const P& p, const SeqKeys& k, int kv0) {
    a1 = min(max(k.first - kv0, 0), P::kTileKeys);
    a0 = max(a1 - (k.first & (p.box_rows - 1)), 0);
    b0 = min(max(k.len - kv0, 0), P::kTileKeys);
    b1 = min(b0 + (-k.len & (p.box_rows - 1)), P::kTileKeys);
    if (k.first < kv0 || k.first >= kv0 + P::kTileKeys) a0 = a1 = 0;
    if (k.len < kv0 || k.len >= kv0 + P::kTileKeys) b0 = b1 = 0;
  }
  __device__ __forceinline__ bool any() const { return a0 < a1 || b0 < b1; }
};

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

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Barrier of the row warps (kThreads threads) that tells whether any thread's flag is set.
template <int kThreads = 128>
__device__ __forceinline__ bool row_warps_any(bool flag) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any) : "r"(flag ? 1u : 0u), "n"(kThreads) : "memory");
  return any != 0;
}

}  // namespace
}  // namespace fa
