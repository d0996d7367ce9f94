// Internal interface of the ragged paged decode (fa_fwd_ragged_paged): sequences
// of unequal length over a paged key/value cache. Not installed.
#pragma once

#include "fa_internal.h"

namespace fa {

// Work is the list of all key tiles: for every sequence, for every key/value
// head, the tiles of 128 keys that its new rows see. The list is cut into even
// shares, one a CTA.
struct RaggedParams {
  CUtensorMap tm_k;   // [num_blocks*Hkv][block_size][d], box (64, box_rows, 1), 128B swizzle
  CUtensorMap tm_v;
  const void* q;      // [B*Hq][Sq][d]
  void* out;          // [B*Hq][Sq][d]
  float* lse;         // [B*Hq][Sq]
  const int* block_table;   // [B][max_blocks]
  const int* seq_lens;      // [B]
  float* part_out;    // [2 * CTAs][R][d] fp32 out = O / l of a part of a (sequence, head)
  float* part_lse2;   // [2 * CTAs][R]    its log2-sum-exp2 of scaled scores
  int4* starts;       // [CTAs] where each CTA's share begins, written by it (find_share)
  int B, Hq, Hkv, Sq, G, R;
  int block_size, box_rows, max_blocks, num_blocks;
  int capacity;       // keys a table row can hold (at most 2^31 - 128)
  int window;         // keys a row sees, its own position included; 0: all
  float scale_log2;
  ScoreMod mod;       // cap and slopes; key spans and pos_offset are not used here
  bool large_cap;     // the cap's form goes by the scores (cap_scores), not the exponential always
  int n_ctas;
  int* status;
};

cudaError_t launch_ragged(const RaggedParams& p, int d, bool bf16, cudaStream_t stream);

}  // namespace fa
