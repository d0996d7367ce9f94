// Work list of the span backward: which query tiles each key tile needs, in what
// order the items run, and which items are cut.
//
// A work item of the backward is a key tile of one (batch, key/value head) with
// all the steps (query tile, query head) that reach it. Under the causal mask
// the items number thousands and get shorter in order; under spans they may be
// few and uneven (78 items of 4 to 44 steps for three padded sequences of 1537
// tokens with two key/value heads: half the SMs idle, the others wait for the
// longest item). So one block, for up to kPlanMax key tiles,
//   - finds every key tile's range of query tiles,
//   - cuts items into slices of at most L steps where there are fewer than two
//     items an SM, with the L that leaves one or two rounds of slices over the
//     SMs, whichever is shorter with kSliceCost steps a slice for its start and
//     write-out,
//   - orders the slices by length, longest first.
// Slices of a cut item leave fp32 partial dK and dV, added up in slice order by
// the convert kernel, so that dK and dV keep their bits from call to call. Above
// kPlanMax key tiles (where the items number hundreds at least) the pre-pass
// finds the ranges with many blocks and the items run uncut in index order.
//
// The kernel runs beside the pre-pass, which is launched as its programmatic
// dependent and ends by waiting for it.
#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kThreadsP = 1024;
constexpr int kMinSlice = 8;
constexpr int kSliceCost = 3;

// Sum over the block of one value a thread.
__device__ int block_sum(int v, int* slot) {
  __syncthreads();
  if (threadIdx.x == 0) *slot = 0;
  __syncthreads();
  v = __reduce_add_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0 && v) atomicAdd(slot, v);
  __syncthreads();
  return *slot;
}

__global__ void __launch_bounds__(kThreadsP) span_plan_kernel(const SpanPlanParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ int first[kPlanMax], last[kPlanMax], size[kPlanMax], slices[kPlanMax];
  __shared__ int slot, longest;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = p.B * p.n_kv_tiles;   // <= kPlanMax
  for (int i = tid; i < n; i += kThreadsP) {
    first[i] = 0x7fffffff;
    last[i] = -1;
  }
  if (tid == 0) longest = 1;
  __syncthreads();
  // the clamped, padded spans, and every query tile's reach into the key tiles
  const int n_q = p.Sq_pad / kTileM;
  for (int t = warp; t < p.B * n_q; t += kThreadsP / 32) {
    const int b = t / n_q, qt = t - b * n_q;
    int lo = 0x7fffffff, hi = 0;
#pragma unroll
    for (int u = 0; u < kTileM / 32; ++u) {
      const int i = qt * kTileM + u * 32 + lane;
      int2 s = make_int2(0, 0);
      if (i < p.Sq) {
        const size_t at = static_cast<size_t>(b) * p.Sq + i;
        s = make_int2(max(p.key_begin[at], 0), min(p.key_end[at], p.Skv));
      }
      if (s.y <= s.x) s = make_int2(0, 0);
      else lo = min(lo, s.x);
      hi = max(hi, s.y);
      p.spans[static_cast<size_t>(b) * p.Sq_pad + i] = s;
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (hi > 0)
      for (int j = lo / kTileN + lane; j * kTileN < hi; j += 32) {
        atomicMin(&first[b * p.n_kv_tiles + j], qt);
        atomicMax(&last[b * p.n_kv_tiles + j], qt);
      }
  }
  __syncthreads();
  // steps of this thread's key tile (one tile a thread); a tile that nothing sees
  // takes one query tile's, with P = 0: its dK and dV are written as zeros
  const bool mine = tid < n;
  int i0 = 0, n_i = 1, steps = 0;
  if (mine) {
    if (last[tid] >= 0) {
      i0 = first[tid];
      n_i = last[tid] - i0 + 1;
    }
    steps = p.G * n_i;
    atomicMax(&longest, steps);
  }
  __syncthreads();
  // the longest slice
  int L = longest;
  if (p.max_parts > 0) {
    int best = 0x7fffffff;
    for (int rounds = 1; rounds <= 2; ++rounds) {
      int lo = min(kMinSlice, longest), hi = longest;   // the least L whose slices fit, if any
      const int limit = min(p.n_sm * rounds, p.max_parts);
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (block_sum(mine ? (steps + mid - 1) / mid : 0, &slot) * p.Hkv <= limit) hi = mid;
        else lo = mid + 1;
      }
      const int cost = rounds * (lo + kSliceCost);
      const bool fits = block_sum(mine ? (steps + lo - 1) / lo : 0, &slot) * p.Hkv <= limit;
      if (fits && cost < best) {
        best = cost;
        L = lo;
      }
    }
  }
  const int c = mine ? (steps + L - 1) / L : 0;    // slices of this tile
  const int len = mine ? (steps + c - 1) / c : 0;  // and their length (the last one's may be less)
  if (mine) {
    size[tid] = len;
    slices[tid] = c;
  }
  __syncthreads();
  if (mine) {
    int at = 0, part = 0, split = 0;   // slices before this tile's; partial slots and cut tiles before it
    for (int j = 0; j < n; ++j) {
      const int s = size[j], k = slices[j];
      if (s > len || (s == len && j < tid)) at += k;
      if (j < tid && k > 1) {
        part += k;
        ++split;
      }
    }
    for (int k = 0; k < c; ++k) {
      SpanSlice e;
      e.tile = tid;
      e.step0 = k * len;
      e.n_steps = min(len, steps - k * len);
      e.part = c > 1 ? part + k : -1;
      e.i_start = i0;
      e.n_i = n_i;
      p.slices[at + k] = e;
    }
    if (c > 1) p.splits[split] = make_int4(tid, part, c, 0);
    if (tid == n - 1) {
      p.head[1] = split + (c > 1 ? 1 : 0);
    }
  }
  const int total = block_sum(c, &slot);
  if (tid == 0) p.head[0] = total;
}

}  // namespace

cudaError_t launch_span_plan(const SpanPlanParams& p, cudaStream_t stream) {
  span_plan_kernel<<<1, kThreadsP, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fa
