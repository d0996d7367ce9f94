// Internal interface between the C-ABI entry points (fa_api.cu) and the
// kernel launchers (fa_fwd.cu, fa_bwd.cu, fa_simt.cu). Not installed.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace fa {

// Launch as the programmatic dependent of the kernel before it on the stream:
// the new grid may start before that one completes and synchronizes with it
// through griddepcontrol.wait, in front of its first access to memory. (A kernel that
// lets its dependents start early has all its blocks resident by then.)
template <typename... Args>
cudaError_t launch_dependent(void (*kernel)(Args...), dim3 grid, dim3 block, size_t smem,
                             cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Tile geometry shared by the tensor-core kernels: 128 query rows per tile,
// 128 key/value rows per tile, 64-element (128-byte) column chunks.
constexpr int kTileM = 128;
constexpr int kTileN = 128;
constexpr int kChunk = 64;

// Score changes of the span entry points: query row i of batch b sees keys
// key_begin[b][i] <= j < key_end[b][i] (clamped to [0, Skv)); scores are capped
// to softcap * tanh(s / softcap) and biased by -slope_h * |i + Skv - Sq - j|.
struct ScoreMod {
  const int* key_begin;   // [B][Sq]
  const int* key_end;     // [B][Sq]
  const float* slopes;    // [Hq], or null: no distance bias
  float cap_in;           // 2 log2(e) scale / softcap: e^(2 s / softcap) = 2^(cap_in <q, k>); 0: no cap
  float cap_log2;         // softcap * log2(e)
  float cap_a[5], cap_b[3];           // odd polynomials of the cap, each for unscaled
  float cap_limit_a, cap_limit_b;     // scores up to this size (0: not to be used)
  int pos_offset;         // Skv - Sq: query row i stands at position i + pos_offset
};

// Sequence lengths: Sq query rows, Skv key/value rows (equal for
// self-attention). Under the causal mask query row i stands at position
// i + kv_offset, kv_offset = Skv - Sq >= 0 (0 without the mask).
struct FwdParams {
  CUtensorMap tm_q;   // [B*Hq][Sq][d], box (64, 128, 1), 128B swizzle
  CUtensorMap tm_k;   // [B*Hkv][Skv][d]
  CUtensorMap tm_v;   // [B*Hkv][Skv][d]
  void* out;          // [B*Hq][Sq][d], same dtype as q
  float* lse;         // [B*Hq][Sq], natural log
  int B, Hq, Hkv, Sq, Skv, kv_offset;
  int causal;
  float scale_log2;   // softmax scale * log2(e)
  int n_units;        // CTAs per (batch, query head): ceil(Sq / (128 T)) for T query
                      // tiles per CTA (set by the forward's launcher)
  int kv_tiles_ahead; // 1 + ceil(kv_offset / 128): key tiles a full causal
                      // query tile qt walks is qt + kv_tiles_ahead
  int* status;        // device status word (wait timeouts)
  unsigned long long* trace;   // timeline buffer of trace builds (FA_TRACE); else null
  // CTA-pair forward (d = 128) only:
  CUtensorMap tm_k_half;   // k as tm_k with a box of 64 rows: each CTA of a pair loads half a tile
  int n_qblocks;           // ceil(Sq / 512): CTA pairs per (batch, query head)
  // span forward (fa_fwd_span) only
  ScoreMod mod;
};

// Work list of the span backward (span_plan.cuh): for up to this many key tiles
// over the batch, with partial results of so many slices of cut tiles (two rounds
// over 152 SMs).
constexpr int kListTiles = 128;
constexpr int kMaxParts = 304;

struct BwdPreParams {
  const void* out;    // [B*Hq][Sq][d]
  const void* dout;   // [B*Hq][Sq][d]
  const float* lse;   // [B*Hq][Sq]
  float* delta;       // [B*Hq][Sq_pad]   D_i = <dO_i, O_i>, 0 on padding rows
  float* lse2;        // [B*Hq][Sq_pad]   LSE_i * log2(e), +inf on padding rows
  float* dq_acc;      // [B*Hq][Sq_pad][d] fp32, zeroed here
  int* work;          // the main kernel's work-item counter, zeroed here (null: none)
  int BH, Sq, Sq_pad, d;
  int dtype;
  // span backward only (n_plan_blocks blocks more, which write spans and plan):
  int n_plan_blocks, B, Skv, n_kv_tiles;
  const int* key_begin;   // [B][Sq]
  const int* key_end;     // [B][Sq]
  int2* spans;            // [B][Sq_pad] clamped (begin, end), empty spans as (0, 0)
  int2* plan;             // [B][n_kv_tiles] (first query tile, number of query tiles)
};

struct BwdParams {
  CUtensorMap tm_q;   // [B*Hq][Sq][d]
  CUtensorMap tm_k;   // [B*Hkv][Skv][d]
  CUtensorMap tm_v;   // [B*Hkv][Skv][d]
  CUtensorMap tm_do;  // [B*Hq][Sq][d]
  CUtensorMap tm_dq;  // dq_acc as fp32 [B*Hq][Sq_pad][d], box (32, 32, 1), 128B swizzle
  CUtensorMap tm_dk;  // dk [B*Hkv][Skv][d], box (64, 32, 1), 128B swizzle (stores)
  CUtensorMap tm_dv;  // dv, as tm_dk
  const float* delta; // [B*Hq][Sq_pad]
  const float* lse2;  // [B*Hq][Sq_pad]
  float* dq_acc;      // [B*Hq][Sq_pad][d]
  void* dk;           // [B*Hkv][Skv][d]
  void* dv;           // [B*Hkv][Skv][d]
  int* work;          // work-item counter, zeroed by the pre-pass
  int B, Hq, Hkv, Sq, Skv, Sq_pad, kv_offset;
  int causal;
  float scale;        // softmax scale
  float scale_log2;   // softmax scale * log2(e)
  int n_kv_tiles;     // ceil(Skv / 128): work items per (batch, key/value head)
  int n_q_tiles;      // ceil(Sq / 128)
  int* status;
  unsigned long long* trace;   // timeline buffer of trace builds (FA_TRACE); else null
  // span backward only
  ScoreMod mod;
  const int2* spans;  // [B][Sq_pad], written by the pre-pass
  const int2* plan;   // [B][n_kv_tiles], written by the pre-pass
  int listed;         // B * n_kv_tiles <= kListTiles: items go by a work list
  int n_slots;        // SMs the list is made for
  float* parts;       // [entry * Hkv + g][dK, dV][d][128] fp32 of the slices of cut
                      // tiles, or null: nothing is cut
  int4* splits;       // cut tiles, for the convert kernel: (tile, first entry, entries, 0)
  int* n_splits;
};

struct DqConvertParams {
  const float* dq_acc;  // [B*Hq][Sq_pad][d]
  void* dq;             // [B*Hq][Sq][d]
  int BH, Sq, Sq_pad, d;
  float scale;
  int dtype;
  // span backward with cuts: blocks more, which add up the parts of cut tiles into
  // dk and dv, for up to max_pairs (cut tile, key/value head) pairs (0: no cuts)
  int max_pairs, n_part_blocks;
  const int* n_splits;
  const int4* splits;
  const float* parts;
  void* dk;
  void* dv;
  int Hkv, Skv, n_kv_tiles;
};

// Plain fp32 (SIMT) kernels for fp32 inputs.
struct SimtParams {
  const float *q, *k, *v, *out, *dout, *lse;
  float *o_out, *lse_out, *dq, *dk, *dv;
  const float* delta;   // [B*Hq][Sq_pad]
  int B, Hq, Hkv, Sq, Skv, kv_offset, d;
  int causal;
  float scale;
};

// Host-side argument checks of the backward entry points (shapes, dtype,
// scale, null and 16-byte alignment of every pointer); FA_OK or an FA_ERR_*
// code. Defined in fa_api.cu.
int check_bwd_args(const void* q, const void* k, const void* v, const void* out,
                   const void* dout, const float* lse, const void* dq, const void* dk,
                   const void* dv, int B, int Hq, int Hkv, int Sq, int Skv, int d, int causal,
                   float scale, int dtype);

// Launchers; each returns a cudaError_t from the launch.
cudaError_t launch_fwd_tc(const FwdParams& p, int d, bool bf16, cudaStream_t stream);
cudaError_t launch_fwd_span(const FwdParams& p, int d, bool bf16, cudaStream_t stream);
cudaError_t launch_fwd_pair(const FwdParams& p, bool bf16, cudaStream_t stream);
cudaError_t launch_bwd_pre(const BwdPreParams& p, cudaStream_t stream);
cudaError_t launch_bwd_tc(const BwdParams& p, int d, bool bf16, cudaStream_t stream);
cudaError_t launch_bwd_pre_span(const BwdPreParams& p, cudaStream_t stream);
cudaError_t launch_bwd_span(const BwdParams& p, int d, bool bf16, cudaStream_t stream);
cudaError_t launch_dq_convert(const DqConvertParams& p, cudaStream_t stream);
cudaError_t launch_fwd_simt(const SimtParams& p, cudaStream_t stream);
cudaError_t launch_bwd_simt(const SimtParams& p, cudaStream_t stream);

}  // namespace fa
