// Internal interface of the query/key preparation (fa_qk_norm_rope*): per-head
// norm and rotary positions, for training and for appending to a paged cache.
// Not installed.
#pragma once

#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace fa {

// Strided view [B][H][S][d] of one tensor: element strides of b, h and s; the
// d elements of a head are contiguous.
struct HeadView {
  void* data;
  long long sb, sh, ss;
};

struct HeadsParams {
  HeadView q, k, v;            // inputs (v: append only)
  HeadView q_out, k_out;       // outputs of the forward; gradients of them in the backward
  HeadView dq, dk;             // backward: gradients of q and k
  const void* wq;              // [d] norm weights, or null: no norm
  const void* wk;
  const int* positions;        // [B][S], or null: row s stands at position s
  const uint64_t* turns;       // [rope_dim / 2] turns a position in units of 2^-64
  float eps, rope_scale;
  int rope_dim, interleaved;
  int B, Hq, Hkv, S, d, dtype;
  // append only
  void* k_cache;               // [num_blocks][Hkv][block_size][d]
  void* v_cache;
  const int* block_table;      // [B][max_blocks]
  const int* seq_lens;         // [B]
  int block_size, num_blocks, max_blocks;
  // backward only
  float* dw_part;              // [blocks][2][d] partial weight gradients
  float* dwq;                  // [d]
  float* dwk;
  int n_blocks;
};

// Blocks of the backward (and partial weight gradients) for these sizes.
int heads_bwd_blocks(int B, int Hq, int Hkv, int S, int d);

cudaError_t launch_heads_fwd(const HeadsParams& p, cudaStream_t stream);
cudaError_t launch_heads_append(const HeadsParams& p, cudaStream_t stream);
cudaError_t launch_heads_bwd(const HeadsParams& p, cudaStream_t stream);

}  // namespace fa
