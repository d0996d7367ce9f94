/*
 * fa.h — C ABI of libfa: causal scaled-dot-product flash attention, forward
 * and backward, on one NVIDIA GB300 (sm_103a).
 *
 * What is computed. For every batch b and query head h (key/value head
 * g = h / (Hq / Hkv), grouped-query attention as in "Phase 14: Flash
 * Attention 2 for SM120", section GQA 支持):
 *
 *   s_ij   = scale * <Q[b,h,i,:], K[b,g,j,:]>,  s_ij = -inf for j > i if causal
 *   P_ij   = exp(s_ij - LSE_i),   LSE_i = log(sum_j exp(s_ij))   (natural log)
 *   out_i  = sum_j P_ij V[b,g,j,:]
 *
 * ("Phase T14: 融合 Flash-Attention Kernel", section 什么是 flash-attention,
 * and its Key Design Decisions item 2: the forward keeps only LSE per row).
 * The backward recomputes P from Q, K, V and LSE, forms D_i = <dO_i, out_i>
 * (item 3 of the same section) and
 *
 *   dP_ij = <dO_i, V_j>,  dS_ij = P_ij (dP_ij - D_i)
 *   dQ_i  = scale * sum_j dS_ij K_j,  dK_j = scale * sum_i dS_ij Q_i,
 *   dV_j  = sum_i P_ij dO_i
 *
 * with dK, dV of a key/value head summed over its Hq/Hkv query heads. No S x S
 * matrix is ever stored.
 *
 * Layout. Every tensor is a dense, contiguous array in device memory:
 *   q, out, dout, dq : [B][Hq][S][d]      k, v, dk, dv : [B][Hkv][S][d]
 *   lse              : [B][Hq][S]  float32
 * Element type of q/k/v/out/dout/dq/dk/dv is `dtype` (FA_F32, FA_F16 or
 * FA_BF16). d must be 64 or 128. Every pointer must be 16-byte aligned.
 *
 * Precision. FA_BF16 / FA_F16 run on the tensor cores with fp32 accumulation;
 * P is rounded to the input type before it multiplies V (and dS before it
 * multiplies Q and K). FA_F32 runs on plain fp32 arithmetic.
 *
 * Ownership and execution. The caller owns every buffer; the library keeps no
 * pointer after a call returns and allocates no device memory. Calls are
 * asynchronous on `stream` (a cudaStream_t; NULL = legacy default stream) and
 * run on the current CUDA device, which must be the stream's device. Outputs
 * are overwritten, never accumulated into. Calls that share output or
 * workspace buffers must be ordered by the caller.
 *
 * Errors. Functions return FA_OK (0) or a negative FA_ERR_* code. Argument
 * errors are detected on the host before anything is enqueued, so a call that
 * returns an argument error has written nothing. FA_ERR_CUDA means a CUDA
 * runtime call or a kernel launch failed (the CUDA error is left for
 * cudaGetLastError to report). A kernel that gives up an internal wait (it
 * never should) sets a device status word instead of hanging; read it with
 * fa_last_device_status.
 */
#ifndef FA_H_
#define FA_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t. */
typedef struct CUstream_st* fa_stream_t;

typedef enum { FA_F32 = 0, FA_F16 = 1, FA_BF16 = 2 } fa_dtype;

enum {
  FA_OK = 0,
  FA_ERR_SHAPE = -1,        /* B, Hq, Hkv, S < 1, Hq % Hkv != 0, d not 64/128, causal with
                               Skv < Sq (fa_*_kv), a size the call refuses, or too large */
  FA_ERR_DTYPE = -2,        /* dtype not one of fa_dtype, or one the call does not take */
  FA_ERR_NULL = -3,         /* a required pointer is NULL */
  FA_ERR_ALIGN = -4,        /* a pointer (tensors 16 bytes, workspace 256, others as stated)
                               or a view's stride is not aligned */
  FA_ERR_WORKSPACE = -5,    /* workspace NULL or smaller than the call's *_workspace_bytes */
  FA_ERR_CUDA = -6,         /* a CUDA runtime call or kernel launch failed */
  FA_ERR_SCALE = -7,        /* scale not finite and > 0, or softcap, rope_scale or eps out of
                               the call's range */
  FA_ERR_TMA = -8,          /* the driver rejected a tensor-memory-access descriptor */
  FA_ERR_NOALLOC_LIMIT = -9 /* fa_bwd_noalloc: sizes need more than FA_NOALLOC_SCRATCH_BYTES */
};

/*
 * Forward pass. Writes out[B][Hq][S][d] (dtype) and lse[B][Hq][S] (float32,
 * natural-log logsumexp of the scaled, masked score row). causal != 0 masks
 * key positions j > i. scale is usually 1/sqrt(d).
 *
 * For FA_BF16 / FA_F16 at d = 128 the forward (here and in fa_fwd_kv) runs
 * either a single-CTA kernel (the default) or a CTA-pair kernel on the
 * tensor cores' 2-CTA mode ("Phase 14: Flash Attention 2 for SM120", section
 * 硬件约束); both write the same bits. The environment variable
 * FA_FWD_CTA_PAIR, read at every call, selects the pair kernel when it is "1"
 * and the single-CTA kernel when it is "0". The single-CTA kernel gives each
 * CTA one 128-row query tile (two CTAs share an SM) at d = 64 and, at
 * d = 128, when the grid has at least four such CTAs per SM, else two tiles;
 * FA_FWD_TILES ("1" or "2", read at every call) forces one form. All forms
 * write the same bits.
 */
int fa_fwd(const void* q, const void* k, const void* v, void* out, float* lse,
           int B, int Hq, int Hkv, int S, int d, int causal, float scale,
           int dtype, fa_stream_t stream);

/*
 * Bytes of device workspace fa_bwd needs for these sizes (the same for every
 * dtype): an fp32 dQ accumulator [B][Hq][S128][d], D and LSE*log2(e) rows
 * [B][Hq][S128] each, where S128 = S rounded up to a multiple of 128, each
 * region starting on a 256-byte boundary, then 256 bytes holding the
 * counter from which the main kernel's CTAs claim work items. Returns 0 for
 * invalid sizes.
 */
size_t fa_bwd_workspace_bytes(int B, int Hq, int Hkv, int S, int d);

/*
 * Backward pass. Inputs: q, k, v, out and lse from fa_fwd with the same
 * arguments, dout = dL/dout. Writes dq [B][Hq][S][d], dk and dv [B][Hkv][S][d]
 * (dtype). `workspace` is caller-owned device memory of at least
 * fa_bwd_workspace_bytes(B, Hq, Hkv, S, d) bytes, 256-byte aligned; its
 * contents on entry do not matter and are clobbered.
 */
int fa_bwd(const void* q, const void* k, const void* v, const void* out,
           const void* dout, const float* lse, void* dq, void* dk, void* dv,
           int B, int Hq, int Hkv, int S, int d, int causal, float scale,
           int dtype, void* workspace, size_t workspace_bytes,
           fa_stream_t stream);

/*
 * Separate query and key/value lengths: Sq query rows against Skv key/value
 * rows, for a chunk of queries at the end of a longer context (chunked
 * prefill, a few new tokens against a KV cache) or, without the mask, any two
 * lengths. Layout:
 *   q, out, dout, dq : [B][Hq][Sq][d]     k, v, dk, dv : [B][Hkv][Skv][d]
 *   lse              : [B][Hq][Sq]  float32
 * With causal != 0, query row i stands at sequence position i + kv_offset,
 * kv_offset = Skv - Sq, and key j is masked when j > i + kv_offset ("Phase 14:
 * Flash Attention 2 for SM120", section Causal Mask: kv_offset = kv_len -
 * q_len, for a KV cache longer than Q). Causal calls need Skv >= Sq, else
 * FA_ERR_SHAPE (rows with no visible key have no softmax). Everything else
 * (dtypes, d, alignment, ownership, errors, asynchrony) is as for fa_fwd and
 * fa_bwd, which are these calls with Sq = Skv = S.
 */
int fa_fwd_kv(const void* q, const void* k, const void* v, void* out, float* lse,
              int B, int Hq, int Hkv, int Sq, int Skv, int d, int causal,
              float scale, int dtype, fa_stream_t stream);

/* Workspace bytes of fa_bwd_kv: as fa_bwd_workspace_bytes, sized by Sq (the
 * dQ accumulator and the per-row D and LSE have one row per query). Returns 0
 * for invalid sizes. */
size_t fa_bwd_kv_workspace_bytes(int B, int Hq, int Hkv, int Sq, int Skv, int d);

int fa_bwd_kv(const void* q, const void* k, const void* v, const void* out,
              const void* dout, const float* lse, void* dq, void* dk, void* dv,
              int B, int Hq, int Hkv, int Sq, int Skv, int d, int causal,
              float scale, int dtype, void* workspace, size_t workspace_bytes,
              fa_stream_t stream);

/*
 * Split-KV forward for few query rows per head: decode (one or a few new
 * tokens, Sq small, against a long key/value cache Skv). Same arguments,
 * layouts, mask (kv_offset = Skv - Sq under causal) and results as fa_fwd_kv;
 * only the work layout differs. The G = Hq / Hkv query heads of a key/value
 * head are packed into one 128-row tile, so G * Sq must be at most 128
 * (else FA_ERR_SHAPE); the key/value sequence of each (batch, key/value head)
 * is cut into n_splits ranges of whole 128-key tiles processed in parallel,
 * each producing a partial out and log-sum-exp, which a second kernel merges
 * ("Phase 14: Flash Attention 2 for SM120", section 已知局限与后续优化方向,
 * item 1: a dedicated decode kernel that reduces in parallel along the
 * key/value dimension).
 *
 * n_splits: 0 = automatic (the largest count that keeps all B * Hkv * n_splits
 * CTAs in one wave on the GPU's 152 SMs, at least 1); otherwise the requested
 * number of ranges, reduced so that no range is empty (at most ceil(Skv/128)).
 * workspace: caller-owned device memory of at least
 * fa_fwd_splitkv_workspace_bytes(...) bytes, 256-byte aligned, for the
 * per-range partial results (fp32); it may be NULL when that size is 0 (one
 * range). FA_F32 inputs take the fa_fwd_kv path (no split, no workspace).
 */
int fa_fwd_splitkv(const void* q, const void* k, const void* v, void* out, float* lse,
                   int B, int Hq, int Hkv, int Sq, int Skv, int d, int causal,
                   float scale, int dtype, int n_splits, void* workspace,
                   size_t workspace_bytes, fa_stream_t stream);

/* Workspace bytes of fa_fwd_splitkv for these sizes and n_splits (0 =
 * automatic): B * Hkv * ranges * G * Sq rows of d + 1 floats, each region
 * 256-byte aligned; 0 when one range suffices, and 0 for invalid sizes (the
 * call reports those). */
size_t fa_fwd_splitkv_workspace_bytes(int B, int Hq, int Hkv, int Sq, int Skv, int d,
                                      int n_splits);

/*
 * fa_fwd_splitkv over a paged key/value cache: the keys and values of all
 * sequences live in fixed-size blocks of a shared pool, and a block table maps
 * each sequence's logical blocks to physical ones ("FlashAttention 与 SDPA
 * Backend", section 与 PagedAttention、KV Cache 的组合: a paged decode kernel
 * looks up the block table while it loads the K/V tiles and runs the online
 * softmax). Layouts:
 *   k_cache, v_cache : [num_blocks][Hkv][block_size][d]   (dtype)
 *   block_table      : [B][max_blocks] int32; key position t of sequence b is
 *                      row t % block_size of block block_table[b][t / block_size]
 * block_size: a power of two from 16 to 1024. Only the first
 * ceil(Skv / block_size) entries of a row are read (max_blocks must be at
 * least that); an entry outside [0, num_blocks) reads as zeros instead of
 * faulting. Every sequence has the same Skv. q, out, lse, the mask, the
 * results, n_splits and the workspace (fa_fwd_splitkv_workspace_bytes) are as
 * for fa_fwd_splitkv. FA_BF16 and FA_F16 only (FA_F32 gives FA_ERR_DTYPE).
 */
int fa_fwd_splitkv_paged(const void* q, const void* k_cache, const void* v_cache,
                         const int* block_table, void* out, float* lse,
                         int B, int Hq, int Hkv, int Sq, int Skv, int d,
                         int block_size, int num_blocks, int max_blocks, int causal,
                         float scale, int dtype, int n_splits, void* workspace,
                         size_t workspace_bytes, fa_stream_t stream);

/*
 * A strided view [B][H][S][d]: element (b, h, s, e) is at
 * data[b * stride_b + h * stride_h + s * stride_s + e] (strides in elements, of
 * any sign; data and every stride a multiple of 16 bytes, else FA_ERR_ALIGN).
 * A packed projection [B][S][Hq + 2 Hkv][d] is three such views.
 */
typedef struct {
  void* data;
  long long stride_b, stride_h, stride_s;
} fa_view;

/*
 * Queries and keys for the attention calls: an RMS norm of every head, then
 * rotary positions, in one pass. For each row x (d elements) of q and of k:
 *
 *   n = x * (mean_e x_e^2 + eps)^(-1/2) * weight       (both weights NULL: n = x;
 *       a mean plus eps below 2^-126 counts as that, so a row of zeros gives zeros)
 *   y_a = rope_scale * (cos t * n_a - sin t * n_b)
 *   y_b = rope_scale * (sin t * n_a + cos t * n_b)
 *
 * for the pairs i < rope_dim / 2 of the first rope_dim elements, (a, b) =
 * (i, i + rope_dim / 2), or (2i, 2i + 1) with interleaved != 0; y = n in the rest
 * of the head. The angle t is the row's position times the pair's frequency:
 * turns[i] is that frequency in units of 2^-64 of a turn per position
 * (frequency in radians / (2 pi) * 2^64, modulo 2^64), so angles are exact
 * modulo a turn at every int32 position. positions: [B][S] int32, or NULL for
 * position s at row s. Arithmetic is in fp32; y is rounded once.
 *
 * q, q_out have Hq heads, k, k_out Hkv, all S rows of d elements. FA_F32,
 * FA_F16 or FA_BF16; weights are [d] of that type, 16-byte aligned; turns
 * 8-byte aligned, may be NULL when rope_dim is 0. rope_dim: a multiple of 16 up
 * to d. Outputs may be their own inputs, but must not overlap them otherwise.
 * eps must be finite and >= 0 (read only with weights) and rope_scale finite
 * (else FA_ERR_SCALE); one weight without the other gives FA_ERR_NULL.
 */
int fa_qk_norm_rope(const fa_view* q, const fa_view* k, const fa_view* q_out,
                    const fa_view* k_out, const void* q_weight, const void* k_weight,
                    float eps, const int* positions, const unsigned long long* turns,
                    int rope_dim, int interleaved, float rope_scale, int B, int Hq, int Hkv,
                    int S, int d, int dtype, fa_stream_t stream);

/*
 * Backward of fa_qk_norm_rope: from dq_out, dk_out (gradients of its outputs),
 * its inputs q, k and its other arguments, writes dq, dk and the float32 weight
 * gradients dq_weight, dk_weight [d], summed over all rows and heads (the same
 * bits on every call). Without weights q, k, dq_weight, dk_weight and workspace
 * are not read and may be NULL. dq, dk may be dq_out, dk_out (same views).
 * workspace: caller-owned, 256-byte aligned, contents on entry without meaning.
 */
int fa_qk_norm_rope_bwd(const fa_view* dq_out, const fa_view* dk_out, const fa_view* q,
                        const fa_view* k, const fa_view* dq, const fa_view* dk,
                        float* dq_weight, float* dk_weight, const void* q_weight,
                        const void* k_weight, float eps, const int* positions,
                        const unsigned long long* turns, int rope_dim, int interleaved,
                        float rope_scale, int B, int Hq, int Hkv, int S, int d, int dtype,
                        void* workspace, size_t workspace_bytes, fa_stream_t stream);

/* Workspace bytes of fa_qk_norm_rope_bwd: 2 d floats for each of at most 304
 * CTAs; 0 without the norm (norm == 0) and for invalid sizes. */
size_t fa_qk_norm_rope_bwd_workspace_bytes(int B, int Hq, int Hkv, int S, int d, int norm);

/*
 * The serving form: the last Sq tokens of each of B sequences. Row s of
 * sequence b stands at position p = seq_lens[b] - Sq + s (seq_lens: [B] int32 in
 * device memory, these tokens included, as fa_fwd_ragged_paged reads it). q is
 * normed and rotated into q_out; k is normed and rotated into row p of the
 * sequence in k_cache and v copied into v_cache (layouts as for
 * fa_fwd_splitkv_paged, here of any dtype). A token at p < 0, past the block
 * table, or in a page whose entry is outside [0, num_blocks) is not stored; its
 * q_out row is written all the same. Everything else in the caches is left as
 * it was. Two tokens of a call must not share a cache row.
 */
int fa_qk_norm_rope_append(const fa_view* q, const fa_view* k, const fa_view* v,
                           const fa_view* q_out, void* k_cache, void* v_cache,
                           const int* block_table, const int* seq_lens, const void* q_weight,
                           const void* k_weight, float eps, const unsigned long long* turns,
                           int rope_dim, int interleaved, float rope_scale, int B, int Hq,
                           int Hkv, int Sq, int d, int block_size, int num_blocks,
                           int max_blocks, int dtype, fa_stream_t stream);

/*
 * One or a few new tokens of each of B sequences of unequal length over a
 * paged key/value cache. k_cache, v_cache, block_table, q, out and lse are laid
 * out as for fa_fwd_splitkv_paged; seq_lens: [B] int32 in device memory, the
 * keys of each sequence with its Sq new tokens included (values below 0 count
 * as 0, values above max_blocks * block_size as that). Row s of sequence b
 * stands at position p = seq_lens[b] - Sq + s and sees keys
 *
 *   max(0, p + 1 - window) <= j <= p        (window 0: from key 0),
 *
 * with scores capped and biased as by fa_fwd_span (distance p - j). A row that
 * sees no key (p < 0), or whose scores are all -infinity, gets out = 0 and lse =
 * -infinity; a row with a NaN or +infinity among its scores gets NaN in both.
 *
 * The lengths are read on the device only, and must not change while the call
 * runs: it needs no host copy of them, and a captured graph may be replayed
 * after they change. All key tiles
 * of all sequences are shared out evenly over one wave of CTAs whatever the
 * lengths are. Results are the same bits on every call with the same lengths (where
 * a row's keys are cut, and so its last bits, goes by the lengths of all sequences).
 *
 * Only table entries of pages that hold a key some row sees are read; an entry
 * outside [0, num_blocks) reads as zeros. The rest of the cache, rows of a
 * sequence's last page past its length included, may hold anything.
 *
 * G * Sq <= 128 with G = Hq / Hkv, block_size as for fa_fwd_splitkv_paged,
 * max_blocks >= 1, window >= 0 and B * Hkv * (ceil(max_blocks * block_size /
 * 128) + 8) < 2^31 (else FA_ERR_SHAPE); softcap as for fa_fwd_span (else
 * FA_ERR_SCALE), its error too, but softcap * 2^-20 always for caps up to 128 (a
 * warp caps 32 rows of 128 keys, or up to 32 rows of 32 keys; keys that no row
 * sees do not count there); FA_BF16 and FA_F16 only (FA_F32 gives FA_ERR_DTYPE).
 * workspace: caller-owned, at least fa_fwd_ragged_paged_workspace_bytes(...)
 * bytes, 256-byte aligned, contents on entry without meaning; calls that may
 * overlap on the GPU need one each.
 */
int fa_fwd_ragged_paged(const void* q, const void* k_cache, const void* v_cache,
                        const int* block_table, const int* seq_lens, void* out, float* lse,
                        int B, int Hq, int Hkv, int Sq, int d, int block_size, int num_blocks,
                        int max_blocks, int window, float scale, float softcap,
                        const float* slopes, int dtype, void* workspace,
                        size_t workspace_bytes, fa_stream_t stream);

/* Workspace bytes of fa_fwd_ragged_paged: two partial results of G * Sq rows of
 * d + 1 floats for each of at most 152 CTAs, and 16 bytes a CTA, each region
 * 256-byte aligned. Returns 0 for invalid sizes. */
size_t fa_fwd_ragged_paged_workspace_bytes(int B, int Hq, int Hkv, int Sq, int d,
                                           int block_size, int max_blocks);

/*
 * Attention in which every query row sees its own contiguous range of keys,
 * for packed documents, sliding windows, prefixes seen by all, and padding:
 * row i of batch b sees keys j with
 *
 *   max(key_begin[b][i], 0) <= j < min(key_end[b][i], Skv)
 *
 * in every head (key_begin, key_end: [B][Sq] int32 in device memory). Spans
 * need no order among the rows. Scores are
 *
 *   s_ij = scale * <Q_i, K_j>                                softcap == 0
 *   s_ij = softcap * tanh(scale * <Q_i, K_j> / softcap)      softcap > 0
 *   s_ij -= slopes[h] * |i + Skv - Sq - j|                   slopes != NULL
 *
 * (slopes: [Hq] float32; a distance bias on the positions of fa_fwd_kv).
 * Everything else is as for fa_fwd_kv without the causal mask, whose other
 * arguments these are; Sq and Skv are unrelated. A row that sees no key gets
 * out = 0 and lse = -infinity, and contributes nothing to any gradient; a key
 * that no row sees gets dk = dv = 0. No gradient is formed for slopes.
 *
 * Masked positions: a masked probability of 0 still multiplies V (forward) and
 * dO, Q, K (backward) of the same 128-row tile, so q, k, v, out and dout must
 * be finite everywhere, padding included. (A NaN score that a row sees gives NaN in
 * its out and lse, as in fa_fwd, and NaN gradients at least where they depend on it.)
 *
 * FA_BF16 and FA_F16 only (FA_F32 gives FA_ERR_DTYPE). softcap must be 0, or it
 * and scale / softcap within 2^-60 .. 2^60 (else FA_ERR_SCALE). A capped score is
 * off by up to softcap * 2^-20; where no score of the warp that caps it (32 rows of
 * a tile of 128 keys, masked ones included) is above 0.3 softcap, or 2^-12 softcap
 * for caps above 10^9 scale, by up to 2^-17 of itself. So the last bits of a row
 * may depend on what stands beside it. key_begin, key_end and slopes need 4-byte
 * alignment. dk and dv have the same bits on every call with the same spans (how
 * their sums are cut goes by the spans of the whole batch); dq is summed with fp32
 * additions in global memory whose order, and so its last bits, may differ.
 */
int fa_fwd_span(const void* q, const void* k, const void* v, const int* key_begin,
                const int* key_end, void* out, float* lse, int B, int Hq, int Hkv, int Sq,
                int Skv, int d, float scale, float softcap, const float* slopes, int dtype,
                fa_stream_t stream);

/* Workspace bytes of fa_bwd_span: fa_bwd_kv_workspace_bytes, then the padded
 * spans ([B][Sq rounded up to 128] pairs of int32), the query-tile range of every
 * key tile ([B][ceil(Skv / 128)] pairs) and, for at most 128 key tiles over the
 * batch and fewer than 304 pairs of a key tile and a key/value head, up to 304
 * partial results of cut tiles (2 * 128 * d floats each); each region 256-byte
 * aligned. Returns 0 for invalid sizes. */
size_t fa_bwd_span_workspace_bytes(int B, int Hq, int Hkv, int Sq, int Skv, int d);

int fa_bwd_span(const void* q, const void* k, const void* v, const int* key_begin,
                const int* key_end, const void* out, const void* dout, const float* lse,
                void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int Sq, int Skv, int d,
                float scale, float softcap, const float* slopes, int dtype, void* workspace,
                size_t workspace_bytes, fa_stream_t stream);

/*
 * Size of the fixed device scratch array behind fa_bwd_noalloc (32 MiB). A
 * call fits when fa_bwd_workspace_bytes(B, Hq, Hkv, S, d) is at most this,
 * e.g. B*Hq = 96 heads at S = 1024, d = 64 (about 25.9 MB). The limit uses
 * that one size for every dtype, although FA_F32 calls use only the D and
 * LSE rows of it.
 */
#define FA_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)

/*
 * Backward pass for callers that cannot allocate device memory (for example
 * code inside a framework or plugin callback that owns every device
 * allocation, or latency-critical code that must not call cudaMalloc/cudaFree
 * because they can synchronize the device). Same arguments and results as
 * fa_bwd, without the workspace: the scratch is a fixed
 * FA_NOALLOC_SCRATCH_BYTES array in the library's device memory, held on every
 * GPU that loads the library until the process exits. The call allocates
 * nothing. This entry point has no counterpart in the method's description;
 * it is a deployment aid.
 *
 * Errors: first fa_bwd's argument errors (FA_ERR_SHAPE, FA_ERR_DTYPE,
 * FA_ERR_SCALE, FA_ERR_NULL, FA_ERR_ALIGN), then FA_ERR_NOALLOC_LIMIT when
 * the sizes need more scratch than FA_NOALLOC_SCRATCH_BYTES; either way
 * nothing is enqueued and the scratch array is not looked up.
 *
 * Device and set-up: the array used is the current device's, so the current
 * device must be the one that owns `stream` and every pointer. The first call
 * that passes the checks with a given device current looks up the array's
 * device address on that device; make that first call before any stream
 * capture.
 *
 * Sharing: every call shares the one array and it keeps the last call's
 * contents (each call rewrites all of it that it reads, so results do not
 * depend on them). Calls whose work overlaps on the GPU (unordered streams,
 * concurrent host threads) race on the array: the caller must order them.
 */
int fa_bwd_noalloc(const void* q, const void* k, const void* v, const void* out,
                   const void* dout, const float* lse, void* dq, void* dk, void* dv,
                   int B, int Hq, int Hkv, int S, int d, int causal, float scale,
                   int dtype, fa_stream_t stream);

/* Static description of an FA_* code. */
const char* fa_strerror(int code);

/*
 * Waits for `stream`, then reads and clears the device status word of the
 * current device: 0 when no kernel has given up a wait since the last read,
 * else a bit mask (1 = an mbarrier wait ran past its limit). Returns FA_OK or
 * FA_ERR_CUDA.
 */
int fa_last_device_status(fa_stream_t stream, int* status);

/* Library version, major * 10000 + minor * 100 + patch. */
int fa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FA_H_ */
