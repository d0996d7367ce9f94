// Internal interface of the latent attention (fa_fwd_latent, fa_bwd_latent,
// fa_fwd_latent_paged, fa_latent_append): keys and values from one latent vector a
// token, with a rotated key part that all heads share. Not installed.
#pragma once

#include "fa_heads.h"
#include "fa_internal.h"

namespace fa {

constexpr int kRope = 64;   // rotated elements of a key and of a query: one 128-byte chunk

// ---- expanded form: keys and values of every head in memory ----
// Query row i of batch b sees keys key_begin[b][i] <= j < key_end[b][i], or without
// the two arrays 0 <= j <= i + Skv - Sq.
struct LatentMask {
  const int* key_begin;   // [B][Sq], or null: causal
  const int* key_end;
  int Sq, Skv;
  // keys [x, y) of a row, (0, 0) when it sees none
  __device__ __forceinline__ int2 span(int b, int row) const {
    int2 s = make_int2(0, 0);
    if (row < Sq) {
      if (key_begin) {
        const size_t at = static_cast<size_t>(b) * Sq + row;
        s = make_int2(max(key_begin[at], 0), min(key_end[at], Skv));
      } else {
        s.y = min(row + Skv - Sq + 1, Skv);
      }
    }
    if (s.y <= s.x) s = make_int2(0, 0);
    return s;
  }
};

struct LatentFwdParams {
  CUtensorMap tm_q;    // 4-D (d + 64, Sq, H, B), box (64, 128, 1, 1), 128B swizzle
  CUtensorMap tm_k;    // (d, Skv, H, B)
  CUtensorMap tm_kr;   // (64, Skv, 1, B)
  CUtensorMap tm_v;    // (d, Skv, H, B)
  CUtensorMap tm_out;  // (d, Sq, H, B), box (32, 32, 1, 1), 64B swizzle
  float* lse;          // [B*H][Sq]
  LatentMask mask;
  int B, H;
  float scale_log2;
  int n_units;         // CTAs a (batch, head), set by the launcher
  int* status;
};

// fp16 only: what bounds |dS| of 128 keys of a head, for the power of two that dS is scaled by.
struct LatentNorms {
  float v;     // greatest norm of their rows of V
  float ds;    // greatest |dO_i| max_j |V_j| of the query tiles that see one of them: |dS| is at most twice that
};

// Backward: workspace regions, the dQ kernel's results for the dK, dV kernel among them.
struct LatentBwdParams {
  CUtensorMap tm_q;    // 4-D (d + 64, Sq, H, B), box (64, 64, 1, 1), 128B swizzle
  CUtensorMap tm_do;   // (d, Sq, H, B), box of 64 rows
  CUtensorMap tm_o;    // as tm_do
  CUtensorMap tm_k;    // (d, Skv, H, B), as the rest
  CUtensorMap tm_kr;   // (64, Skv, 1, B)
  CUtensorMap tm_v;    // (d, Skv, H, B)
  CUtensorMap tm_dq;   // as q, dK, dV as k and v: boxes (32, 32, 1, 1), 64B swizzle
  CUtensorMap tm_dk;
  CUtensorMap tm_dv;
  CUtensorMap tm_part; // fp32 (64, Skv, H, B), box (32, 32, 1, 1), 128B swizzle
  HeadView dk_rope;
  HeadView v;          // (read directly for fp16's norms)
  const float* lse;    // [B*H][Sq]
  float* lse2;         // [B*H][Sq_pad]  LSE log2(e) less kShiftP, +inf on rows that see nothing
  float* delta;        // [B*H][Sq_pad]  <dO, O>
  int2* ranges;        // [B][Sq_pad / 64] least and greatest key of 64 rows' spans, (max, 0): none
  float* part;         // [B*H][Skv][64] each head's unscaled gradient of the shared key part; in fp16, until
                       // it is written, the first two of each 128 keys hold LatentNorms
  LatentMask mask;
  int B, H, Sq_pad;
  float scale, scale_log2;
  int n_units;         // 128-row tiles of the kernel's own side, set by the launcher
  int* status;
};

// ---- absorbed form: the cache holds [latent | rotated key part] rows ----
struct LatentAppendParams {
  HeadView latent;         // [B][Sq][rank] (no heads)
  HeadView k_rope;         // [B][Sq][64] (no heads)
  HeadView q_rope, q_out;  // [B][H][Sq][64]
  void* cache;             // [num_blocks][block_size][rank + 64]
  const int* block_table;  // [B][max_blocks]
  const int* seq_lens;     // [B]
  const int* positions;    // [B][Sq], or null: a token's position is its row of the sequence
  const void* weight;      // [rank], or null: no norm
  const uint64_t* turns;   // [32] turns a position in units of 2^-64
  float eps, rope_scale;
  int interleaved, B, H, Sq, rank, block_size, num_blocks, max_blocks, dtype;
};

// The last Sq tokens of every sequence, R = H * Sq rows (head, token) of it, in groups of up to
// 64 rows, over 64-key tiles of its cache. (Names as the work's division wants them,
// ragged_shares.cuh: Hkv = 1, n_ctas the shares.)
struct LatentPagedParams {
  static constexpr int kTileKeys = 64;
  static constexpr int Hkv = 1;
  CUtensorMap tm;          // [num_blocks][block_size][rank + 64], box (64, box_rows, 1), 128B swizzle
  CUtensorMap tm_q;        // 4-D (rank + 64, Sq, H, B), box (64, group_tokens, group_heads, 1)
  void* out;               // [B][R][rank]
  float* lse;              // [B][R]
  const int* block_table;  // [B][max_blocks]
  const int* seq_lens;     // [B]
  const long long* tree;   // [B][Sq] bit t: sees new token t; or null
  float* part_out;         // [2 * n_ctas][R][rank] fp32 out = O / l of a part of a sequence
  float* part_lse2;        // [2 * n_ctas][R]       its log2-sum-exp2 of scaled scores
  int4* starts;            // [n_ctas] where each share begins
  // a group's rows: all tokens (up to 64) of group_heads heads, or 64 tokens of one head
  int B, H, Sq, R, groups, group_heads, group_tokens;
  int block_size, block_shift, box_rows, max_blocks, num_blocks;   // block_size = 2^block_shift
  int capacity;            // keys a table row can hold (at most 2^31 - 128)
  int window;              // keys a row sees, its own position included; 0: all
  float scale_log2;
  int n_ctas;
  int* status;
};

cudaError_t launch_latent_paged(const LatentPagedParams& p, int rank, bool bf16, cudaStream_t stream);
cudaError_t launch_latent_append(const LatentAppendParams& p, cudaStream_t stream);
cudaError_t launch_latent_bwd(const LatentBwdParams& p, int d, bool bf16, cudaStream_t stream);
cudaError_t launch_latent_fwd(const LatentFwdParams& p, int d, bool bf16, cudaStream_t stream);

}  // namespace fa
