// C-ABI entry points of the latent attention (declared in include/fa.h): argument
// checks, TMA descriptors, launches.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "../../include/fa.h"
#include "fa_latent.h"

namespace fa {
namespace {

constexpr float kLog2eLat = 1.4426950408889634f;

long long up(long long x, long long m) { return (x + m - 1) / m * m; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_sizes(int B, int H, int Sq, int Skv, int d, float scale) {
  if (B < 1 || H < 1 || Sq < 1 || Skv < 1 || (d != 64 && d != 128)) return FA_ERR_SHAPE;
  // CTAs of any kernel below 2^31, rows and keys within int32 with room for a tile
  const long long bh = static_cast<long long>(B) * H;
  if (bh > (1LL << 30) || Sq > (1 << 30) || Skv > (1 << 30) || bh * ((Sq + 127) / 128) > 0x7fffffffLL ||
      bh * ((Skv + 127) / 128) > 0x7fffffffLL || static_cast<long long>(B) * Skv * 16 / 256 > 0x7ffffffeLL)
    return FA_ERR_SHAPE;
  if (!(std::isfinite(scale) && scale > 0.f)) return FA_ERR_SCALE;
  return FA_OK;
}

// A strided view with its extents; every row of `d` elements starts on a 16-byte boundary,
// and strides are positive (the copy engine's descriptors take no others).
struct ViewOf {
  const fa_view* from;
  int H, S;
  HeadView* to;
};
int take(std::initializer_list<ViewOf> views, int B, int dtype) {
  const long long unit = dtype == FA_F32 ? 4 : 8;   // elements in 16 bytes
  for (const ViewOf& v : views)
    if (!v.from || !v.from->data) return FA_ERR_NULL;
  for (const ViewOf& v : views) {
    const long long st[3] = {v.from->stride_b, v.from->stride_h, v.from->stride_s};
    const int n[3] = {B, v.H, v.S};
    if (!aligned(v.from->data, 16)) return FA_ERR_ALIGN;
    for (int i = 0; i < 3; ++i) {
      if (n[i] == 1) continue;   // no stride to speak of
      if (st[i] % unit != 0) return FA_ERR_ALIGN;
      if (st[i] <= 0 || st[i] >= (1LL << 38)) return FA_ERR_SHAPE;
    }
    *v.to = HeadView{v.from->data, B > 1 ? st[0] : 0, v.H > 1 ? st[1] : 0, v.S > 1 ? st[2] : 0};
  }
  return FA_OK;
}

// 4-D view (d, S, H, B) of a strided 16-bit tensor; box = box_cols columns (one swizzle span, 128
// bytes of 64) x box_rows rows x box_heads heads.
bool make_map(CUtensorMap* m, const HeadView& v, int B, int H, int S, int d, int box_rows, bool bf16,
              int box_heads = 1, int box_cols = kChunk) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(S), static_cast<cuuint64_t>(H),
                              static_cast<cuuint64_t>(B)};
  auto bytes = [&](long long stride) { return static_cast<cuuint64_t>(stride > 0 ? stride * 2 : d * 2); };
  const cuuint64_t strides[3] = {bytes(v.ss), bytes(v.sh), bytes(v.sb)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows),
                             static_cast<cuuint32_t>(box_heads), 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, v.data, dims, strides,
             box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_cols == kChunk ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The same for stores, in a warp's boxes.
bool make_store_map(CUtensorMap* m, const HeadView& v, int B, int H, int S, int d, bool bf16) {
  return make_map(m, v, B, H, S, d, 32, bf16, 1, 32);
}
// [B][H][S][64] floats, contiguous, in boxes of 32 x 32.
bool make_part_map(CUtensorMap* m, float* data, int B, int H, int S) {
  EncodeTiledFn enc = encode_fn();
  const cuuint64_t row = kRope * 4, dims[4] = {kRope, static_cast<cuuint64_t>(S), static_cast<cuuint64_t>(H),
                                               static_cast<cuuint64_t>(B)};
  const cuuint64_t strides[3] = {row, row * dims[1], row * dims[1] * dims[2]};
  const cuuint32_t box[4] = {32, 32, 1, 1}, one[4] = {1, 1, 1, 1};
  return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, data, dims, strides, box, one,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int check_mask(const int* begin, const int* end) {
  if ((begin == nullptr) != (end == nullptr)) return FA_ERR_NULL;
  return aligned(begin, 4) && aligned(end, 4) ? FA_OK : FA_ERR_ALIGN;
}

struct LatentBwdWs {
  size_t lse2, delta, ranges, part, total;
};
LatentBwdWs bwd_ws(int B, int H, int Sq, int Skv) {
  LatentBwdWs w;
  const long long rows = up(Sq, kTileM), bh = static_cast<long long>(B) * H;
  w.lse2 = 0;
  w.delta = static_cast<size_t>(up(bh * rows * 4, 256));
  w.ranges = w.delta + static_cast<size_t>(up(bh * rows * 4, 256));
  w.part = w.ranges + static_cast<size_t>(up(B * (rows / 64) * 8, 256));
  w.total = w.part + static_cast<size_t>(bh) * Skv * kRope * 4;
  return w;
}

bool blocks_ok(int block_size, int num_blocks, int max_blocks) {
  return block_size >= 16 && block_size <= 1024 && (block_size & (block_size - 1)) == 0 && num_blocks >= 1 &&
         num_blocks <= (1 << 30) && max_blocks >= 1;
}

// Plan of fa_fwd_latent_paged: the rows of a sequence in groups of up to 64, and as many
// shares of the key tiles as leave all CTAs of a share's groups in one wave.
constexpr int kMaxRows = 1024;   // H * Sq
constexpr int kGroupRows = 64;
struct PagedPlan {
  int groups, group_heads, group_tokens, shares;
  size_t part_out, part_lse2, starts, total;
};
PagedPlan paged_plan(int B, int H, int Sq, int rank, int block_size, int max_blocks) {
  PagedPlan w;
  const long long R = static_cast<long long>(H) * Sq;
  w.group_tokens = std::min(Sq, kGroupRows);
  const int heads = kGroupRows / w.group_tokens;   // of a group, at most
  w.groups = Sq > kGroupRows ? H * ((Sq + kGroupRows - 1) / kGroupRows) : (H + heads - 1) / heads;
  w.group_heads = Sq > kGroupRows ? 1 : (H + w.groups - 1) / w.groups;
  const long long tiles =
      (static_cast<long long>(max_blocks) * block_size + LatentPagedParams::kTileKeys - 1) / LatentPagedParams::kTileKeys;
  w.shares = static_cast<int>(std::min<long long>(152 / w.groups, B * tiles));
  const long long rows = 2LL * w.shares * R;
  w.part_out = 0;
  w.part_lse2 = static_cast<size_t>(up(rows * rank * 4, 256));
  w.starts = w.part_lse2 + static_cast<size_t>(up(rows * 4, 256));
  w.total = w.starts + static_cast<size_t>(up(w.shares * 16LL, 256));
  return w;
}
bool paged_ok(int B, int H, int Sq, int rank, int block_size, int num_blocks, int max_blocks) {
  if (B < 1 || H < 1 || Sq < 1 || static_cast<long long>(H) * Sq > kMaxRows || (rank != 256 && rank != 512) ||
      !blocks_ok(block_size, num_blocks, max_blocks))
    return false;
  // the list of key tiles, and a few units a sequence beside them, is counted in 32 bits
  const long long tiles = (static_cast<long long>(max_blocks) * block_size + 63) / 64;
  return tiles + 8 <= 0x7fffffffLL / B;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

int fa_fwd_latent(const fa_view* q, const fa_view* k, const fa_view* k_rope, const fa_view* v,
                  const int* key_begin, const int* key_end, const fa_view* out, float* lse, int B, int H,
                  int Sq, int Skv, int d, float scale, int dtype, fa_stream_t stream) {
  if (dtype != FA_F16 && dtype != FA_BF16) return FA_ERR_DTYPE;
  int rc = check_sizes(B, H, Sq, Skv, d, scale);
  if (rc == FA_OK) rc = check_mask(key_begin, key_end);
  if (rc != FA_OK) return rc;
  LatentFwdParams p;
  std::memset(&p, 0, sizeof(p));
  HeadView vq, vk, vr, vv, vo;
  if ((rc = take({{q, H, Sq, &vq}, {k, H, Skv, &vk}, {k_rope, 1, Skv, &vr}, {v, H, Skv, &vv}, {out, H, Sq, &vo}},
                 B, dtype)) != FA_OK)
    return rc;
  if (!lse) return FA_ERR_NULL;
  if (!aligned(lse, 4)) return FA_ERR_ALIGN;
  const bool bf16 = dtype == FA_BF16;
  if (!make_map(&p.tm_q, vq, B, H, Sq, d + kRope, kTileM, bf16) || !make_map(&p.tm_k, vk, B, H, Skv, d, kTileN, bf16) ||
      !make_map(&p.tm_kr, vr, B, 1, Skv, kRope, kTileN, bf16) || !make_map(&p.tm_v, vv, B, H, Skv, d, kTileN, bf16) ||
      !make_store_map(&p.tm_out, vo, B, H, Sq, d, bf16))
    return FA_ERR_TMA;
  p.lse = lse;
  p.mask = LatentMask{key_begin, key_end, Sq, Skv};
  p.B = B;
  p.H = H;
  p.scale_log2 = scale * kLog2eLat;
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  return launch_latent_fwd(p, d, bf16, stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_bwd_latent_workspace_bytes(int B, int H, int Sq, int Skv, int d) {
  return check_sizes(B, H, Sq, Skv, d, 1.f) == FA_OK ? bwd_ws(B, H, Sq, Skv).total : 0;
}

int fa_bwd_latent(const fa_view* q, const fa_view* k, const fa_view* k_rope, const fa_view* v,
                  const int* key_begin, const int* key_end, const fa_view* out, const fa_view* dout,
                  const float* lse, const fa_view* dq, const fa_view* dk, const fa_view* dk_rope,
                  const fa_view* dv, int B, int H, int Sq, int Skv, int d, float scale, int dtype,
                  void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  if (dtype != FA_F16 && dtype != FA_BF16) return FA_ERR_DTYPE;
  int rc = check_sizes(B, H, Sq, Skv, d, scale);
  if (rc == FA_OK) rc = check_mask(key_begin, key_end);
  if (rc != FA_OK) return rc;
  LatentBwdParams p;
  std::memset(&p, 0, sizeof(p));
  HeadView vq, vk, vr, vo, vg, vdq, vdk, vdv;
  if ((rc = take({{q, H, Sq, &vq}, {k, H, Skv, &vk}, {k_rope, 1, Skv, &vr}, {v, H, Skv, &p.v}, {out, H, Sq, &vo},
                  {dout, H, Sq, &vg}, {dq, H, Sq, &vdq}, {dk, H, Skv, &vdk}, {dk_rope, 1, Skv, &p.dk_rope},
                  {dv, H, Skv, &vdv}}, B, dtype)) != FA_OK)
    return rc;
  if (!lse) return FA_ERR_NULL;
  if (!aligned(lse, 4)) return FA_ERR_ALIGN;
  const LatentBwdWs w = bwd_ws(B, H, Sq, Skv);
  if (!workspace || workspace_bytes < w.total) return FA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return FA_ERR_ALIGN;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.part = reinterpret_cast<float*>(ws + w.part);
  const bool bf16 = dtype == FA_BF16;
  if (!make_map(&p.tm_q, vq, B, H, Sq, d + kRope, 64, bf16) || !make_map(&p.tm_do, vg, B, H, Sq, d, 64, bf16) ||
      !make_map(&p.tm_o, vo, B, H, Sq, d, 64, bf16) ||
      !make_map(&p.tm_k, vk, B, H, Skv, d, 64, bf16) || !make_map(&p.tm_kr, vr, B, 1, Skv, kRope, 64, bf16) ||
      !make_map(&p.tm_v, p.v, B, H, Skv, d, 64, bf16) || !make_store_map(&p.tm_dq, vdq, B, H, Sq, d + kRope, bf16) ||
      !make_store_map(&p.tm_dk, vdk, B, H, Skv, d, bf16) || !make_store_map(&p.tm_dv, vdv, B, H, Skv, d, bf16) ||
      !make_part_map(&p.tm_part, p.part, B, H, Skv))
    return FA_ERR_TMA;
  p.lse = lse;
  p.lse2 = reinterpret_cast<float*>(ws + w.lse2);
  p.delta = reinterpret_cast<float*>(ws + w.delta);
  p.ranges = reinterpret_cast<int2*>(ws + w.ranges);
  p.mask = LatentMask{key_begin, key_end, Sq, Skv};
  p.B = B;
  p.H = H;
  p.Sq_pad = static_cast<int>(up(Sq, kTileM));
  p.scale = scale;
  p.scale_log2 = scale * kLog2eLat;
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  return launch_latent_bwd(p, d, bf16, stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_fwd_latent_paged_workspace_bytes(int B, int H, int Sq, int rank, int block_size, int max_blocks) {
  if (!paged_ok(B, H, Sq, rank, block_size, 1, max_blocks)) return 0;
  return paged_plan(B, H, Sq, rank, block_size, max_blocks).total;
}

int fa_fwd_latent_paged(const fa_view* q, const void* cache, const int* block_table, const int* seq_lens,
                        const long long* tree_masks, void* out, float* lse, int B, int H, int Sq, int rank,
                        int block_size, int num_blocks, int max_blocks, int window, float scale, int dtype,
                        void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  if (dtype != FA_F16 && dtype != FA_BF16) return FA_ERR_DTYPE;
  if (!paged_ok(B, H, Sq, rank, block_size, num_blocks, max_blocks) || window < 0 ||
      (tree_masks && (window > 0 || Sq > 64)))
    return FA_ERR_SHAPE;
  if (!(std::isfinite(scale) && scale > 0.f)) return FA_ERR_SCALE;
  LatentPagedParams p;
  std::memset(&p, 0, sizeof(p));
  HeadView vq;
  const int rc = take({{q, H, Sq, &vq}}, B, dtype);
  if (rc != FA_OK) return rc;
  if (!cache || !block_table || !seq_lens || !out || !lse) return FA_ERR_NULL;
  if (!aligned(cache, 16) || !aligned(out, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(lse, 4) || !aligned(tree_masks, 8))
    return FA_ERR_ALIGN;
  const PagedPlan w = paged_plan(B, H, Sq, rank, block_size, max_blocks);
  if (!workspace || workspace_bytes < w.total) return FA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return FA_ERR_ALIGN;
  const bool bf16 = dtype == FA_BF16;
  const int width = rank + kRope;
  p.box_rows = std::min(block_size, LatentPagedParams::kTileKeys);
  EncodeTiledFn enc = encode_fn();
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(block_size),
                              static_cast<cuuint64_t>(num_blocks)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(width) * 2, static_cast<cuuint64_t>(block_size) * width * 2};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(kChunk), static_cast<cuuint32_t>(p.box_rows), 1};
  const cuuint32_t one[3] = {1, 1, 1};
  if (!enc || enc(&p.tm, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                  const_cast<void*>(cache), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
      !make_map(&p.tm_q, vq, B, H, Sq, width, w.group_tokens, bf16, w.group_heads))
    return FA_ERR_TMA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.out = out;
  p.lse = lse;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.tree = tree_masks;
  p.part_out = reinterpret_cast<float*>(ws + w.part_out);
  p.part_lse2 = reinterpret_cast<float*>(ws + w.part_lse2);
  p.starts = reinterpret_cast<int4*>(ws + w.starts);
  p.B = B; p.H = H; p.Sq = Sq;
  p.R = H * Sq;
  p.groups = w.groups;
  p.group_heads = w.group_heads;
  p.group_tokens = w.group_tokens;
  p.block_size = block_size; p.max_blocks = max_blocks; p.num_blocks = num_blocks;
  while (1 << p.block_shift < block_size) ++p.block_shift;
  p.capacity = static_cast<int>(std::min(static_cast<long long>(max_blocks) * block_size, 0x7fffff80LL));
  // a window that no position outgrows hides nothing (and would overflow positions)
  p.window = window < p.capacity ? window : 0;
  p.scale_log2 = scale * kLog2eLat;
  p.n_ctas = w.shares;
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  return launch_latent_paged(p, rank, bf16, stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

int fa_latent_append(const fa_view* latent, const fa_view* k_rope, const fa_view* q_rope,
                     const fa_view* q_out, void* cache, const int* block_table, const int* seq_lens,
                     const int* positions, const void* weight, float eps,
                     const unsigned long long* turns, int interleaved, float rope_scale, int B, int H,
                     int Sq, int rank, int block_size, int num_blocks, int max_blocks, int dtype,
                     fa_stream_t stream) {
  if (dtype != FA_F32 && dtype != FA_F16 && dtype != FA_BF16) return FA_ERR_DTYPE;
  if (B < 1 || H < 1 || Sq < 1 || H > (1 << 20) || static_cast<long long>(B) * Sq > 0x7fffffffLL ||
      (rank != 256 && rank != 512) || !blocks_ok(block_size, num_blocks, max_blocks))
    return FA_ERR_SHAPE;
  if (!std::isfinite(rope_scale) || (weight && !(std::isfinite(eps) && eps >= 0.f))) return FA_ERR_SCALE;
  LatentAppendParams p;
  std::memset(&p, 0, sizeof(p));
  const int rc = take({{latent, 1, Sq, &p.latent}, {k_rope, 1, Sq, &p.k_rope}, {q_rope, H, Sq, &p.q_rope},
                       {q_out, H, Sq, &p.q_out}}, B, dtype);
  if (rc != FA_OK) return rc;
  if (!cache || !block_table || !seq_lens || !turns) return FA_ERR_NULL;
  if (!aligned(cache, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(positions, 4) ||
      !aligned(weight, 16) || !aligned(turns, 8))
    return FA_ERR_ALIGN;
  p.cache = cache;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.positions = positions;
  p.weight = weight;
  p.turns = reinterpret_cast<const uint64_t*>(turns);
  p.eps = eps;
  p.rope_scale = rope_scale;
  p.interleaved = interleaved != 0;
  p.B = B; p.H = H; p.Sq = Sq; p.rank = rank;
  p.block_size = block_size; p.num_blocks = num_blocks; p.max_blocks = max_blocks;
  p.dtype = dtype;
  return launch_latent_append(p, stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
