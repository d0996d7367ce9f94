// Work list of the span backward: in what order the items run, and which of them
// are cut.
//
// A work item of the backward is a key tile of one (batch, key/value head) with
// all the steps (query tile, query head) that reach it. Under the causal mask
// the items number thousands and get shorter in order; under spans they may be
// few and uneven (78 items of 4 to 44 steps for three padded sequences of 1537
// tokens with two key/value heads: half the SMs idle, the others wait for the
// longest item). So for up to kListTiles key tiles over the batch every CTA of the
// main kernel, at its start,
//   - cuts items into slices of at most L steps where there are fewer than two
//     items an SM, with the L that leaves one or two rounds of slices over the
//     SMs, whichever is shorter with kSliceCost steps a slice for its start and
//     write-out,
//   - orders the slices by length, longest first.
// All CTAs come to the same list, in their shared memory; for 64 tiles it takes
// about three microseconds. (Made once, by a kernel in front of the pre-pass, the
// list cost 8 us of a 72 us backward; by a block of the pre-pass, 22 us.) Slices of a cut
// item leave fp32 partial dK and dV, added up in slice order by the convert kernel,
// so that dK and dV keep their bits from call to call. With more key tiles the
// items number hundreds and run uncut in index order.
#pragma once

#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kMinSlice = 8;
constexpr int kSliceCost = 3;

// Scratch of span_list, in shared memory that is free before the first load.
struct SpanScratch {
  int steps[kListTiles], len[kListTiles], slices[kListTiles];
  int longest, feasible[32];
};

// Slices and their length of a tile with so many steps.
__device__ __forceinline__ void span_cut(int steps, int L, int& slices, int& len) {
  slices = (steps + L - 1) / L;
  len = (steps + slices - 1) / slices;
}

// By all `threads` threads (a multiple of 32, at least kListTiles) of the CTA:
// entries (tile | slice << 7) into `list`, the slices' limit into *limit_out; their
// number is returned. (A call of its own: its registers are not the main loop's.)
__device__ __noinline__ int span_list(const BwdParams& p, SpanScratch& s, uint16_t* list,
                                      int* limit_out, int threads) {
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int warps = threads / 32;
  const int n = p.B * p.n_kv_tiles;   // <= kListTiles
  const int G = p.Hq / p.Hkv;
  if (tid == 0) s.longest = 1;
  __syncthreads();
  if (tid < n) {
    s.steps[tid] = G * p.plan[tid].y;
    atomicMax(&s.longest, s.steps[tid]);
  }
  __syncthreads();
  int best_L = s.longest;
  if (p.parts) {
    int best = 0x7fffffff;
    const int longest = s.longest;
    for (int rounds = 1; rounds <= 2; ++rounds) {
      const int limit = min(p.n_slots * rounds, kMaxParts);
      // the least L whose slices fit: each warp tries one L of the bracket at a time
      int lo = min(kMinSlice, longest), hi = longest + 1;   // hi: known to fit, or past the end
      while (lo < hi) {
        const int L = lo + static_cast<int>(static_cast<long long>(hi - lo) * warp / warps);
        int c = 0;
        for (int i = lane; i < n; i += 32) c += (s.steps[i] + L - 1) / L;
        c = __reduce_add_sync(0xffffffffu, c);
        if (lane == 0) s.feasible[warp] = c * p.Hkv <= limit;
        __syncthreads();
        int new_lo = lo, new_hi = hi;
        for (int w = warps - 1; w >= 0; --w) {
          const int Lw = lo + static_cast<int>(static_cast<long long>(hi - lo) * w / warps);
          if (s.feasible[w]) new_hi = Lw;
          else {
            new_lo = Lw + 1;
            break;
          }
        }
        __syncthreads();
        lo = new_lo;
        hi = new_hi;
      }
      if (lo <= longest && rounds * (lo + kSliceCost) < best) {
        best = rounds * (lo + kSliceCost);
        best_L = lo;
      }
    }
  }
  int slices = 0, len = 0;
  if (tid < n) {
    span_cut(s.steps[tid], best_L, slices, len);
    s.slices[tid] = slices;
    s.len[tid] = len;
  }
  __syncthreads();
  // slices of longer tiles (of the same length: of those with a lower index) come
  // before this one's
  int at = 0, cut = 0, total = 0;
  for (int i = 0; i < n; ++i) {
    const int k = s.slices[i], l = s.len[i];
    total += k;
    if (l > len || (l == len && i < tid)) at += k;
    if (i < tid && k > 1) ++cut;
  }
  if (tid < n) {
    for (int k = 0; k < slices; ++k) list[at + k] = static_cast<uint16_t>(tid | (k << 7));
    if (blockIdx.x == 0 && p.parts) {   // for the convert kernel
      if (slices > 1) p.splits[cut] = make_int4(tid, at, slices, 0);
      if (tid == n - 1) *p.n_splits = cut + (slices > 1 ? 1 : 0);
    }
  }
  if (tid == 0) *limit_out = best_L;
  return total;
}

}  // namespace
}  // namespace fa
