// C-ABI entry points of libfa (declared in include/fa.h): argument checks,
// TMA descriptor construction and kernel launches. No device memory is
// allocated here; the only device-resident state is the status word below.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <initializer_list>
#include <limits>

#include "../../include/fa.h"
#include "fa_decode.h"
#include "fa_heads.h"
#include "fa_internal.h"
#include "fa_ragged.h"

namespace fa {

// Sticky device status word: kernels OR kStatus* bits into it when they give
// up a wait instead of hanging.
__device__ int g_status;

namespace {

constexpr float kLog2e = 1.4426950408889634f;

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

// Device address of g_status on the current device, looked up once per
// device (the lookup is a runtime call worth microseconds of host time).
constexpr int kMaxDevices = 128;
std::atomic<int*> g_status_ptr[kMaxDevices];

int* status_ptr() {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  int* p = g_status_ptr[dev].load(std::memory_order_acquire);
  if (p) return p;
  if (cudaGetSymbolAddress(reinterpret_cast<void**>(&p), g_status) != cudaSuccess) return nullptr;
  g_status_ptr[dev].store(p, std::memory_order_release);
  return p;
}

// 3-D view [rows = BH][S][d] of a contiguous 16-bit tensor; box = 64 columns
// (128 bytes, one swizzle span) x 128 sequence rows x 1 head.
bool make_tmap(CUtensorMap* m, const void* base, int BH, int S, int d, bool bf16,
               int box_rows = kTileM) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(S),
                        static_cast<cuuint64_t>(BH)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(S) * d * 2};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(kChunk), static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                   const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// 3-D view [BH][S_pad][d] of the fp32 dQ accumulator for bulk reduce-adds;
// box = 32 columns (128 bytes) x 32 rows x 1 head, 128-byte swizzle.
bool make_tmap_acc(CUtensorMap* m, float* base, int BH, int S_pad, int d) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(S_pad),
                        static_cast<cuuint64_t>(BH)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 4, static_cast<cuuint64_t>(S_pad) * d * 4};
  cuuint32_t box[3] = {32, 32, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Sq query rows against Skv key/value rows. Under the causal mask query row i
// stands at position i + (Skv - Sq), so every row sees at least one key only
// when Skv >= Sq; fewer keys than queries is a shape error.
int check_common(int B, int Hq, int Hkv, int Sq, int Skv, int d, int causal, float scale,
                 int dtype) {
  if (dtype != FA_F32 && dtype != FA_F16 && dtype != FA_BF16) return FA_ERR_DTYPE;
  if (B < 1 || Hq < 1 || Hkv < 1 || Sq < 1 || Skv < 1 || Hq % Hkv != 0) return FA_ERR_SHAPE;
  if (d != 64 && d != 128) return FA_ERR_SHAPE;
  if (causal && Skv < Sq) return FA_ERR_SHAPE;
  // grid and index ranges: up to B*Hq*ceil(Sq/128) forward CTAs; B*Hkv*ceil(Skv/128)
  // backward work items, claimed from a 32-bit counter that runs past the
  // last item by at most one claim per CTA (so the bound keeps 2^16 of
  // headroom); element offsets in 64 bits
  const long long bh = static_cast<long long>(B) * Hq;
  const long long bhkv = static_cast<long long>(B) * Hkv;
  if (bh > (1LL << 30) || Sq > (1 << 30) || Skv > (1 << 30) ||
      bh * ((Sq + 127) / 128) > 0x7fffffffLL ||
      bhkv * ((Skv + 127) / 128) > 0x7fffffffLL - 0xffffLL)
    return FA_ERR_SHAPE;
  if (!(std::isfinite(scale) && scale > 0.f)) return FA_ERR_SCALE;
  return FA_OK;
}

inline long long round_up(long long x, long long m) { return (x + m - 1) / m * m; }

// Forward kernel for 16-bit inputs at d = 128: the CTA-pair kernel
// (fa_fwd_pair.cu, tcgen05 cta_group::2) or the single-CTA one (fa_fwd.cu).
// Both compute the same function. FA_FWD_CTA_PAIR=1 (or 0) in the environment
// selects one for every call; otherwise kPairForwardDefault does.
constexpr bool kPairForwardDefault = false;

bool use_pair_forward(int d) {
  if (d != 128) return false;
  const char* e = std::getenv("FA_FWD_CTA_PAIR");
  if (e && e[0] == '1') return true;
  if (e && e[0] == '0') return false;
  return kPairForwardDefault;
}

struct WsLayout {
  size_t dq_acc, delta, lse2, work, total;
};

WsLayout ws_layout(int B, int Hq, int Sq, int d) {
  const long long bh = static_cast<long long>(B) * Hq;
  const long long s_pad = round_up(Sq, kTileM);
  WsLayout w;
  w.dq_acc = 0;
  w.delta = static_cast<size_t>(round_up(bh * s_pad * d * 4, 256));
  w.lse2 = w.delta + static_cast<size_t>(round_up(bh * s_pad * 4, 256));
  w.work = w.lse2 + static_cast<size_t>(round_up(bh * s_pad * 4, 256));
  w.total = w.work + 256;   // the backward's work-item counter
  return w;
}

// Split-KV plan of fa_fwd_splitkv: key tiles per CTA, CTA count per (batch,
// key/value head) and the partial-result workspace. One CTA fits on an SM at a
// time and each CTA pays a start-up (barriers, tensor memory, query staging,
// first-load latency), so the automatic choice is the largest range count that
// keeps every CTA in one wave on the 152 SMs (one range when the (batch,
// key/value head) pairs alone fill the GPU), never an empty range.
constexpr int kDecodeWaveCtas = 152;
constexpr int kDecodeMaxRows = 128;   // G * Sq rows must fit one query tile

struct SplitPlan {
  int n_splits, tiles_per_split, R;
  size_t part_out, part_lse2, total;
};

SplitPlan split_plan(int B, int Hq, int Hkv, int Sq, int Skv, int d, int n_splits_req) {
  SplitPlan sp;
  const int n_tiles = (Skv + kTileN - 1) / kTileN;
  const long long bhkv = static_cast<long long>(B) * Hkv;
  long long want = n_splits_req > 0 ? n_splits_req : kDecodeWaveCtas / bhkv;
  want = std::max(1LL, std::min<long long>(want, n_tiles));
  sp.tiles_per_split = static_cast<int>((n_tiles + want - 1) / want);
  sp.n_splits = (n_tiles + sp.tiles_per_split - 1) / sp.tiles_per_split;
  sp.R = (Hq / Hkv) * Sq;
  sp.part_out = 0;
  if (sp.n_splits == 1) {
    sp.part_lse2 = sp.total = 0;
  } else {
    const long long rows = bhkv * sp.n_splits * sp.R;
    sp.part_lse2 = static_cast<size_t>(round_up(rows * d * 4, 256));
    sp.total = sp.part_lse2 + static_cast<size_t>(round_up(rows * 4, 256));
  }
  return sp;
}

// Plan of fa_fwd_ragged_paged: one wave of CTAs (fewer when the table cannot
// hold that many key tiles), two partial results a CTA.
struct RaggedPlan {
  int n_ctas, R;
  size_t part_out, part_lse2, starts, total;
};

RaggedPlan ragged_plan(int B, int Hq, int Hkv, int Sq, int d, int block_size, int max_blocks) {
  RaggedPlan rp;
  const long long tiles = (static_cast<long long>(max_blocks) * block_size + kTileN - 1) / kTileN;
  const long long bhkv = static_cast<long long>(B) * Hkv;
  rp.n_ctas = bhkv >= kDecodeWaveCtas ? kDecodeWaveCtas
                                      : static_cast<int>(std::min<long long>(kDecodeWaveCtas, bhkv * tiles));
  rp.R = (Hq / Hkv) * Sq;
  const long long rows = 2LL * rp.n_ctas * rp.R;
  rp.part_out = 0;
  rp.part_lse2 = static_cast<size_t>(round_up(rows * d * 4, 256));
  rp.starts = rp.part_lse2 + static_cast<size_t>(round_up(rows * 4, 256));
  rp.total = rp.starts + static_cast<size_t>(round_up(rp.n_ctas * 16LL, 256));
  return rp;
}

// Sizes of a paged cache, and of few query rows against it.
bool block_sizes_ok(int Hkv, int block_size, int num_blocks, int max_blocks) {
  return block_size >= 16 && block_size <= 1024 && (block_size & (block_size - 1)) == 0 &&
         num_blocks >= 1 && static_cast<long long>(num_blocks) * Hkv <= (1LL << 30) &&
         max_blocks >= 1;
}
bool paged_sizes_ok(int B, int Hq, int Hkv, int Sq, int block_size, int num_blocks, int max_blocks) {
  if (static_cast<long long>(Hq / Hkv) * Sq > kDecodeMaxRows ||
      !block_sizes_ok(Hkv, block_size, num_blocks, max_blocks))
    return false;
  // the list of key tiles, and a few units a head beside them, is counted in 32 bits
  const long long tiles = (static_cast<long long>(max_blocks) * block_size + kTileN - 1) / kTileN;
  return tiles + 8 <= 0x7fffffffLL / (static_cast<long long>(B) * Hkv);
}

// Arguments the query/key preparation entry points share.
int heads_params(HeadsParams& p, const void* wq, const void* wk, float eps, const int* positions,
                 const unsigned long long* turns, int rope_dim, int interleaved, float rope_scale,
                 int B, int Hq, int Hkv, int S, int d, int dtype) {
  int rc = check_common(B, Hq, Hkv, S, S, d, 0, 1.f, dtype);
  if (rc != FA_OK) return rc;
  if (rope_dim < 0 || rope_dim > d || rope_dim % 16 != 0 || Hq > (1 << 20) ||
      static_cast<long long>(B) * S > 0x7fffffffLL)
    return FA_ERR_SHAPE;
  if (!std::isfinite(rope_scale) || (wq && !(std::isfinite(eps) && eps >= 0.f)))
    return FA_ERR_SCALE;
  if ((rope_dim > 0 && !turns) || (wq == nullptr) != (wk == nullptr)) return FA_ERR_NULL;
  if (!aligned16(wq) || !aligned16(wk) || (reinterpret_cast<uintptr_t>(positions) & 3u) != 0 ||
      (reinterpret_cast<uintptr_t>(turns) & 7u) != 0)
    return FA_ERR_ALIGN;
  p.wq = wq;
  p.wk = wk;
  p.positions = positions;
  p.turns = reinterpret_cast<const uint64_t*>(turns);
  p.eps = eps;
  p.rope_scale = rope_scale;
  p.rope_dim = rope_dim;
  p.interleaved = interleaved != 0;
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.S = S; p.d = d; p.dtype = dtype;
  return FA_OK;
}

// Strided views: every head starts on a 16-byte boundary.
struct ViewArg {
  const fa_view* from;
  HeadView* to;
};
int take_views(std::initializer_list<ViewArg> views, int dtype) {
  const long long step = dtype == FA_F32 ? 4 : 8;   // elements in 16 bytes
  for (const ViewArg& v : views)
    if (!v.from || !v.from->data) return FA_ERR_NULL;
  for (const ViewArg& v : views) {
    if (!aligned16(v.from->data) || v.from->stride_b % step != 0 || v.from->stride_h % step != 0 ||
        v.from->stride_s % step != 0)
      return FA_ERR_ALIGN;
    *v.to = HeadView{v.from->data, v.from->stride_b, v.from->stride_h, v.from->stride_s};
  }
  return FA_OK;
}

// Arguments the span entry points add.
struct SpanArgs {
  const int* key_begin;
  const int* key_end;
  const float* slopes;
  float softcap;
};

// Scores are scaled by scale / softcap and by softcap in fp32, and by the latter's
// inverse: factors far from any use are refused before one leaves the range.
bool cap_ok(float softcap, float scale) {
  if (softcap == 0.f) return true;
  const double c = softcap, ratio = scale / c;
  return c >= 0x1p-60 && c <= 0x1p60 && ratio >= 0x1p-60 && ratio <= 0x1p60;
}

int check_span(const SpanArgs& m, float scale) {
  if (!cap_ok(m.softcap, scale)) return FA_ERR_SCALE;
  if (!m.key_begin || !m.key_end) return FA_ERR_NULL;
  if (((reinterpret_cast<uintptr_t>(m.key_begin) | reinterpret_cast<uintptr_t>(m.key_end) |
        reinterpret_cast<uintptr_t>(m.slopes)) & 3u) != 0)
    return FA_ERR_ALIGN;
  return FA_OK;
}

// Coefficients of softcap log2(e) tanh(s ratio) / s from those of tanh u / u. False: one
// would leave the range of fp32, the polynomial is not to be used.
template <int N>
bool scale_poly(const double (&from)[N], float (&to)[N], double ratio, double cap_log2) {
  bool ok = true;
  double power = cap_log2 * ratio;
  for (int i = 0; i < N; ++i, power *= ratio * ratio) {
    const double x = std::fabs(from[i] * power);
    ok = ok && x >= std::numeric_limits<float>::min() && x <= std::numeric_limits<float>::max();
    to[i] = ok ? static_cast<float>(from[i] * power) : 0.f;
  }
  return ok;
}

ScoreMod make_mod(const SpanArgs& m, int Sq, int Skv, float scale) {
  ScoreMod r;
  r.key_begin = m.key_begin;
  r.key_end = m.key_end;
  r.slopes = m.slopes;
  r.cap_in = m.softcap > 0.f ? 2.f * kLog2e * scale / m.softcap : 0.f;
  r.cap_log2 = m.softcap * kLog2e;
  // tanh u / u in powers of u^2 on |u| <= 3/4 and on |u| <= 0.3 (score_mod.cuh), scaled
  static const double a[5] = {0.9999971985816956, -0.33323076367378235, 0.13226088881492615,
                              -0.04928038269281387, 0.012318773195147514};
  static const double b[3] = {0.9999960104045702, -0.3329747978841012, 0.12522591724872847};
  const double ratio = m.softcap > 0.f ? static_cast<double>(scale) / m.softcap : 0.0;
  const double cap_log2 = static_cast<double>(m.softcap) * kLog2e;
  r.cap_limit_a = scale_poly(a, r.cap_a, ratio, cap_log2) ? static_cast<float>(0.75 / ratio) : 0.f;
  if (scale_poly(b, r.cap_b, ratio, cap_log2)) {
    r.cap_limit_b = static_cast<float>(0.3 / ratio);
  } else if (m.softcap > 0.f && ratio < 1.0) {
    // a cap some 10^9 times the scale or more: tanh u = u, to 2^-25 of it, up to u = 2^-12
    r.cap_b[0] = static_cast<float>(cap_log2 * ratio);
    r.cap_b[1] = r.cap_b[2] = 0.f;
    r.cap_limit_b = static_cast<float>(0x1p-12 / ratio);
  }
  r.pos_offset = Skv - Sq;
  return r;
}

// Extra workspace of the span backward behind ws_layout's: the padded spans, each
// key tile's query-tile range and, where items may be cut (there is a work list,
// and fewer than two items an SM), the cut tiles and their partial results.
struct SpanWs {
  size_t spans, plan, splits, parts, total;
  int max_parts;
};

SpanWs span_ws(const WsLayout& w, int B, int Hq, int Hkv, int Sq, int Skv, int d) {
  SpanWs s{};
  const long long tiles = (Skv + kTileN - 1LL) / kTileN * B, rows = round_up(Sq, kTileM) * B;
  const long long items = tiles * Hkv;
  const long long steps = static_cast<long long>(Hq / Hkv) * (rows / B / kTileM);   // of an item, at most
  if (tiles <= kListTiles && items < kMaxParts)
    s.max_parts = static_cast<int>(std::min<long long>(kMaxParts, items * steps));
  s.spans = w.total;
  s.plan = s.spans + static_cast<size_t>(round_up(rows * 8, 256));
  s.splits = s.plan + static_cast<size_t>(round_up(tiles * 8, 256));
  // the number of cut tiles, then they
  s.parts = s.splits + (s.max_parts > 0 ? static_cast<size_t>(round_up(16 + s.max_parts * 16LL, 256)) : 0);
  s.total = s.parts + static_cast<size_t>(s.max_parts) * 2 * kTileN * d * 4;
  return s;
}

}  // namespace

int check_bwd_args(const void* q, const void* k, const void* v, const void* out,
                   const void* dout, const float* lse, const void* dq, const void* dk,
                   const void* dv, int B, int Hq, int Hkv, int Sq, int Skv, int d, int causal,
                   float scale, int dtype) {
  int rc = check_common(B, Hq, Hkv, Sq, Skv, d, causal, scale, dtype);
  if (rc != FA_OK) return rc;
  if (!q || !k || !v || !out || !dout || !lse || !dq || !dk || !dv) return FA_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(dout) ||
      !aligned16(lse) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
    return FA_ERR_ALIGN;
  return FA_OK;
}

}  // namespace fa

using namespace fa;

#ifdef FA_TRACE
// Trace builds only: the device buffer kernels record their timelines into
// (kTraceCtas x kTraceRoles x kTraceSlots 64-bit entries), or null.
static unsigned long long* g_trace_buf = nullptr;
extern "C" void fa_trace_set(void* buf) { g_trace_buf = static_cast<unsigned long long*>(buf); }
#define FA_TRACE_PTR g_trace_buf
#else
#define FA_TRACE_PTR nullptr
#endif

namespace {

// Shared body of fa_bwd_kv (mod null) and fa_bwd_span.
int bwd_impl(const void* q, const void* k, const void* v, const void* out, const void* dout,
             const float* lse, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int Sq,
             int Skv, int d, int causal, float scale, int dtype, void* workspace,
             size_t workspace_bytes, fa_stream_t stream, const SpanArgs* mod) {
  int rc = check_bwd_args(q, k, v, out, dout, lse, dq, dk, dv, B, Hq, Hkv, Sq, Skv, d, causal,
                          scale, dtype);
  if (rc != FA_OK) return rc;
  const WsLayout ws = ws_layout(B, Hq, Sq, d);
  const SpanWs sws = span_ws(ws, B, Hq, Hkv, Sq, Skv, d);
  if (!workspace || workspace_bytes < (mod ? sws.total : ws.total)) return FA_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return FA_ERR_ALIGN;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* wsb = static_cast<uint8_t*>(workspace);
  const int BH = B * Hq;
  const int Sq_pad = static_cast<int>(round_up(Sq, kTileM));
  const int kv_offset = causal ? Skv - Sq : 0;

  float* delta = reinterpret_cast<float*>(wsb + ws.delta);
  float* lse2 = reinterpret_cast<float*>(wsb + ws.lse2);
  float* dq_acc = dtype == FA_F32 ? nullptr : reinterpret_cast<float*>(wsb + ws.dq_acc);
  int* status = status_ptr();
  if (!status) return FA_ERR_CUDA;

  // Everything that can fail on the host (descriptor encoding, the status
  // lookup) happens before the first kernel is enqueued.
  const bool bf16 = dtype == FA_BF16;
  BwdParams p;
  std::memset(&p, 0, sizeof(p));
  if (dtype != FA_F32 &&
      (!make_tmap(&p.tm_q, q, BH, Sq, d, bf16) || !make_tmap(&p.tm_k, k, B * Hkv, Skv, d, bf16) ||
       !make_tmap(&p.tm_v, v, B * Hkv, Skv, d, bf16) ||
       !make_tmap(&p.tm_do, dout, BH, Sq, d, bf16) ||
       !make_tmap_acc(&p.tm_dq, dq_acc, BH, Sq_pad, d) ||
       !make_tmap(&p.tm_dk, dk, B * Hkv, Skv, d, bf16, 32) ||
       !make_tmap(&p.tm_dv, dv, B * Hkv, Skv, d, bf16, 32)))
    return FA_ERR_TMA;

  BwdPreParams pre{};
  pre.out = out;
  pre.dout = dout;
  pre.lse = lse;
  pre.delta = delta;
  pre.lse2 = lse2;
  pre.dq_acc = dq_acc;
  pre.work = dtype == FA_F32 ? nullptr : reinterpret_cast<int*>(wsb + ws.work);
  pre.BH = BH; pre.Sq = Sq; pre.Sq_pad = Sq_pad; pre.d = d;
  pre.dtype = dtype;
  if (mod) {
    pre.B = B;
    pre.Skv = Skv;
    pre.n_kv_tiles = (Skv + kTileN - 1) / kTileN;
    pre.key_begin = mod->key_begin;
    pre.key_end = mod->key_end;
    p.spans = pre.spans = reinterpret_cast<int2*>(wsb + sws.spans);
    p.plan = pre.plan = reinterpret_cast<int2*>(wsb + sws.plan);
    // A list for up to four items an SM. It pays where items are long and uneven, and costs
    // its making where they are short and alike; their lengths are known on the device only.
    // With it and without: 512 items of documents (8192 tokens, 8 key/value heads, d = 128)
    // 319 and 330 us, of 4096 causal tokens (16 heads) 184 and 181, of a window of 256 (8192
    // tokens, 8 heads, d = 64) 63.5 and 60.2; 768 of documents 141 and 143, of the window 77.7
    // and 74.2; 1024 of it (d = 128) 131 and 127.5.
    const long long tiles = static_cast<long long>(B) * pre.n_kv_tiles;
    p.listed = tiles <= kListTiles && tiles * Hkv <= 4 * kDecodeWaveCtas;
    p.n_slots = kDecodeWaveCtas;
    if (sws.max_parts > 0) {
      p.n_splits = reinterpret_cast<int*>(wsb + sws.splits);
      p.splits = reinterpret_cast<int4*>(wsb + sws.splits + 16);
      p.parts = reinterpret_cast<float*>(wsb + sws.parts);
    }
  }
  if ((mod ? launch_bwd_pre_span(pre, st) : launch_bwd_pre(pre, st)) != cudaSuccess)
    return FA_ERR_CUDA;

  if (dtype == FA_F32) {
    SimtParams sp{};
    sp.q = static_cast<const float*>(q);
    sp.k = static_cast<const float*>(k);
    sp.v = static_cast<const float*>(v);
    sp.dout = static_cast<const float*>(dout);
    sp.lse = lse;
    sp.delta = delta;
    sp.dq = static_cast<float*>(dq);
    sp.dk = static_cast<float*>(dk);
    sp.dv = static_cast<float*>(dv);
    sp.B = B; sp.Hq = Hq; sp.Hkv = Hkv; sp.Sq = Sq; sp.Skv = Skv; sp.kv_offset = kv_offset;
    sp.d = d;
    sp.causal = causal != 0;
    sp.scale = scale;
    return launch_bwd_simt(sp, st) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
  }

  p.delta = delta;
  p.lse2 = lse2;
  p.dq_acc = dq_acc;
  p.work = reinterpret_cast<int*>(wsb + ws.work);
  p.dk = dk;
  p.dv = dv;
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.Sq = Sq; p.Skv = Skv; p.Sq_pad = Sq_pad;
  p.kv_offset = kv_offset;
  p.causal = causal != 0;
  p.scale = scale;
  p.scale_log2 = scale * kLog2e;
  p.n_kv_tiles = (Skv + kTileN - 1) / kTileN;
  p.n_q_tiles = (Sq + kTileM - 1) / kTileM;
  p.trace = FA_TRACE_PTR;
  p.status = status;
  if (mod) p.mod = make_mod(*mod, Sq, Skv, scale);
  if ((mod ? launch_bwd_span(p, d, bf16, st) : launch_bwd_tc(p, d, bf16, st)) != cudaSuccess)
    return FA_ERR_CUDA;

  DqConvertParams cv{};
  cv.dq_acc = dq_acc;
  cv.dq = dq;
  cv.BH = BH; cv.Sq = Sq; cv.Sq_pad = Sq_pad; cv.d = d;
  cv.scale = scale;
  cv.dtype = dtype;
  if (mod && p.parts) {
    cv.max_pairs = sws.max_parts / 2;   // a cut tile of one head has two parts at least
    cv.n_splits = p.n_splits;
    cv.splits = p.splits;
    cv.parts = p.parts;
    cv.dk = dk;
    cv.dv = dv;
    cv.Hkv = Hkv; cv.Skv = Skv; cv.n_kv_tiles = p.n_kv_tiles;
  }
  return launch_dq_convert(cv, st) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

extern "C" {

int fa_version(void) { return 1 * 10000 + 0 * 100 + 0; }

const char* fa_strerror(int code) {
  switch (code) {
    case FA_OK: return "ok";
    case FA_ERR_SHAPE:
      return "invalid shape (B, Hq, Hkv, S >= 1, Hq % Hkv == 0, d in {64, 128}, causal Skv >= Sq; "
             "paged: block_size a power of two from 16 to 1024, Hq / Hkv * Sq <= 128, window >= 0; "
             "rope_dim a multiple of 16 up to d)";
    case FA_ERR_DTYPE: return "dtype not FA_F32, FA_F16 or FA_BF16, or one this call does not take";
    case FA_ERR_NULL: return "a required pointer is NULL";
    case FA_ERR_ALIGN: return "a pointer or stride is not aligned (tensors and strides 16 bytes, workspace 256, int32 and float "
                              "arguments 4, turns 8)";
    case FA_ERR_WORKSPACE: return "workspace missing or smaller than the call's *_workspace_bytes()";
    case FA_ERR_CUDA: return "a CUDA runtime call or kernel launch failed";
    case FA_ERR_SCALE: return "scale must be finite and > 0, softcap 0 or in its range, rope_scale finite, eps finite and >= 0";
    case FA_ERR_TMA: return "the driver rejected a tensor-memory-access descriptor";
    case FA_ERR_NOALLOC_LIMIT:
      return "sizes need more scratch than fa_bwd_noalloc's fixed FA_NOALLOC_SCRATCH_BYTES";
    default: return "unknown error code";
  }
}

int fa_fwd_kv(const void* q, const void* k, const void* v, void* out, float* lse, int B,
              int Hq, int Hkv, int Sq, int Skv, int d, int causal, float scale, int dtype,
              fa_stream_t stream) {
  int rc = check_common(B, Hq, Hkv, Sq, Skv, d, causal, scale, dtype);
  if (rc != FA_OK) return rc;
  if (!q || !k || !v || !out || !lse) return FA_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(lse))
    return FA_ERR_ALIGN;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int kv_offset = causal ? Skv - Sq : 0;

  if (dtype == FA_F32) {
    SimtParams p{};
    p.q = static_cast<const float*>(q);
    p.k = static_cast<const float*>(k);
    p.v = static_cast<const float*>(v);
    p.o_out = static_cast<float*>(out);
    p.lse_out = lse;
    p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.Sq = Sq; p.Skv = Skv; p.kv_offset = kv_offset; p.d = d;
    p.causal = causal != 0;
    p.scale = scale;
    return launch_fwd_simt(p, st) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
  }

  const bool bf16 = dtype == FA_BF16;
  FwdParams p;
  std::memset(&p, 0, sizeof(p));
  if (!make_tmap(&p.tm_q, q, B * Hq, Sq, d, bf16) || !make_tmap(&p.tm_k, k, B * Hkv, Skv, d, bf16) ||
      !make_tmap(&p.tm_v, v, B * Hkv, Skv, d, bf16))
    return FA_ERR_TMA;
  p.out = out;
  p.lse = lse;
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.Sq = Sq; p.Skv = Skv; p.kv_offset = kv_offset;
  p.causal = causal != 0;
  p.scale_log2 = scale * kLog2e;
  p.kv_tiles_ahead = 1 + (kv_offset + kTileN - 1) / kTileN;
  p.trace = FA_TRACE_PTR;
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  if (use_pair_forward(d)) {
    if (!make_tmap(&p.tm_k_half, k, B * Hkv, Skv, d, bf16, kTileN / 2)) return FA_ERR_TMA;
    p.n_qblocks = (Sq + 4 * kTileM - 1) / (4 * kTileM);
    return launch_fwd_pair(p, bf16, st) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
  }
  return launch_fwd_tc(p, d, bf16, st) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

int fa_fwd(const void* q, const void* k, const void* v, void* out, float* lse, int B, int Hq,
           int Hkv, int S, int d, int causal, float scale, int dtype, fa_stream_t stream) {
  return fa_fwd_kv(q, k, v, out, lse, B, Hq, Hkv, S, S, d, causal, scale, dtype, stream);
}

size_t fa_bwd_kv_workspace_bytes(int B, int Hq, int Hkv, int Sq, int Skv, int d) {
  // the causal constraint is checked by fa_bwd_kv itself
  if (check_common(B, Hq, Hkv, Sq, Skv, d, 0, 1.f, FA_BF16) != FA_OK) return 0;
  return ws_layout(B, Hq, Sq, d).total;
}

size_t fa_bwd_workspace_bytes(int B, int Hq, int Hkv, int S, int d) {
  return fa_bwd_kv_workspace_bytes(B, Hq, Hkv, S, S, d);
}

int fa_bwd_kv(const void* q, const void* k, const void* v, const void* out, const void* dout,
              const float* lse, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int Sq,
              int Skv, int d, int causal, float scale, int dtype, void* workspace,
              size_t workspace_bytes, fa_stream_t stream) {
  return bwd_impl(q, k, v, out, dout, lse, dq, dk, dv, B, Hq, Hkv, Sq, Skv, d, causal, scale,
                  dtype, workspace, workspace_bytes, stream, nullptr);
}

int fa_bwd(const void* q, const void* k, const void* v, const void* out, const void* dout,
           const float* lse, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int S, int d,
           int causal, float scale, int dtype, void* workspace, size_t workspace_bytes,
           fa_stream_t stream) {
  return fa_bwd_kv(q, k, v, out, dout, lse, dq, dk, dv, B, Hq, Hkv, S, S, d, causal, scale, dtype,
                   workspace, workspace_bytes, stream);
}

size_t fa_fwd_splitkv_workspace_bytes(int B, int Hq, int Hkv, int Sq, int Skv, int d,
                                      int n_splits) {
  if (check_common(B, Hq, Hkv, Sq, Skv, d, 0, 1.f, FA_BF16) != FA_OK || n_splits < 0 ||
      (Hq / Hkv) * Sq > kDecodeMaxRows)
    return 0;
  return split_plan(B, Hq, Hkv, Sq, Skv, d, n_splits).total;
}

}  // extern "C"

namespace {

// Shared body of fa_fwd_splitkv and fa_fwd_splitkv_paged (block_table null:
// contiguous K/V).
int splitkv_impl(const void* q, const void* k, const void* v, void* out, float* lse, int B, int Hq,
                 int Hkv, int Sq, int Skv, int d, int causal, float scale, int dtype, int n_splits,
                 void* workspace, size_t workspace_bytes, fa_stream_t stream,
                 const int* block_table, int block_size, int max_blocks, int num_blocks) {
  const bool paged = block_table != nullptr;
  const SplitPlan sp = split_plan(B, Hq, Hkv, Sq, Skv, d, n_splits);
  if (sp.total > 0 && (!workspace || workspace_bytes < sp.total)) return FA_ERR_WORKSPACE;
  if (sp.total > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return FA_ERR_ALIGN;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool bf16 = dtype == FA_BF16;
  uint8_t* wsb = static_cast<uint8_t*>(workspace);

  DecodeParams p;
  std::memset(&p, 0, sizeof(p));
  if (paged) {
    p.box_rows = std::min(block_size, kTileN);
    if (!make_tmap(&p.tm_k, k, num_blocks * Hkv, block_size, d, bf16, p.box_rows) ||
        !make_tmap(&p.tm_v, v, num_blocks * Hkv, block_size, d, bf16, p.box_rows))
      return FA_ERR_TMA;
    p.block_table = block_table;
    p.block_size = block_size;
    p.max_blocks = max_blocks;
    p.num_blocks = num_blocks;
  } else if (!make_tmap(&p.tm_k, k, B * Hkv, Skv, d, bf16) ||
             !make_tmap(&p.tm_v, v, B * Hkv, Skv, d, bf16)) {
    return FA_ERR_TMA;
  }
  p.q = q;
  p.out = out;
  p.lse = lse;
  p.part_out = sp.total ? reinterpret_cast<float*>(wsb + sp.part_out) : nullptr;
  p.part_lse2 = sp.total ? reinterpret_cast<float*>(wsb + sp.part_lse2) : nullptr;
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.Sq = Sq; p.Skv = Skv;
  p.kv_offset = causal ? Skv - Sq : 0;
  p.causal = causal != 0;
  p.G = Hq / Hkv;
  p.R = sp.R;
  p.n_kv_tiles = (Skv + kTileN - 1) / kTileN;
  p.tiles_per_split = sp.tiles_per_split;
  p.n_splits = sp.n_splits;
  p.scale_log2 = scale * kLog2e;
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  if (launch_decode(p, d, bf16, st) != cudaSuccess) return FA_ERR_CUDA;
  if (sp.n_splits == 1) return FA_OK;

  DecodeMergeParams m;
  m.part_out = p.part_out;
  m.part_lse2 = p.part_lse2;
  m.out = out;
  m.lse = lse;
  m.B = B; m.Hq = Hq; m.Hkv = Hkv; m.Sq = Sq; m.G = p.G; m.R = p.R; m.d = d;
  m.n_splits = sp.n_splits;
  m.dtype = dtype;
  return launch_decode_merge(m, st) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

extern "C" {

int fa_fwd_splitkv(const void* q, const void* k, const void* v, void* out, float* lse, int B,
                   int Hq, int Hkv, int Sq, int Skv, int d, int causal, float scale, int dtype,
                   int n_splits, void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  int rc = check_common(B, Hq, Hkv, Sq, Skv, d, causal, scale, dtype);
  if (rc != FA_OK) return rc;
  if (n_splits < 0 || (Hq / Hkv) * Sq > kDecodeMaxRows) return FA_ERR_SHAPE;
  if (!q || !k || !v || !out || !lse) return FA_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(lse))
    return FA_ERR_ALIGN;
  if (dtype == FA_F32)   // plain fp32 arithmetic: one warp per query row, no split
    return fa_fwd_kv(q, k, v, out, lse, B, Hq, Hkv, Sq, Skv, d, causal, scale, dtype, stream);
  return splitkv_impl(q, k, v, out, lse, B, Hq, Hkv, Sq, Skv, d, causal, scale, dtype, n_splits,
                      workspace, workspace_bytes, stream, nullptr, 0, 0, 0);
}

int fa_fwd_splitkv_paged(const void* q, const void* k_cache, const void* v_cache,
                         const int* block_table, void* out, float* lse, int B, int Hq, int Hkv,
                         int Sq, int Skv, int d, int block_size, int num_blocks, int max_blocks,
                         int causal, float scale, int dtype, int n_splits, void* workspace,
                         size_t workspace_bytes, fa_stream_t stream) {
  int rc = check_common(B, Hq, Hkv, Sq, Skv, d, causal, scale, dtype);
  if (rc != FA_OK) return rc;
  if (dtype == FA_F32) return FA_ERR_DTYPE;   // the paged path runs on the tensor cores only
  if (n_splits < 0 || (Hq / Hkv) * Sq > kDecodeMaxRows) return FA_ERR_SHAPE;
  if (block_size < 16 || block_size > 1024 || (block_size & (block_size - 1)) != 0 ||
      num_blocks < 1 || static_cast<long long>(num_blocks) * Hkv > (1LL << 30) ||
      max_blocks < (Skv + block_size - 1) / block_size)
    return FA_ERR_SHAPE;
  if (!q || !k_cache || !v_cache || !block_table || !out || !lse) return FA_ERR_NULL;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      !aligned16(lse) || (reinterpret_cast<uintptr_t>(block_table) & 3u) != 0)
    return FA_ERR_ALIGN;
  return splitkv_impl(q, k_cache, v_cache, out, lse, B, Hq, Hkv, Sq, Skv, d, causal, scale, dtype,
                      n_splits, workspace, workspace_bytes, stream, block_table, block_size,
                      max_blocks, num_blocks);
}

int fa_qk_norm_rope(const fa_view* q, const fa_view* k, const fa_view* q_out, const fa_view* k_out,
                    const void* q_weight, const void* k_weight, float eps, const int* positions,
                    const unsigned long long* turns, int rope_dim, int interleaved,
                    float rope_scale, int B, int Hq, int Hkv, int S, int d, int dtype,
                    fa_stream_t stream) {
  HeadsParams p{};
  int rc = heads_params(p, q_weight, k_weight, eps, positions, turns, rope_dim, interleaved,
                        rope_scale, B, Hq, Hkv, S, d, dtype);
  if (rc == FA_OK) rc = take_views({{q, &p.q}, {k, &p.k}, {q_out, &p.q_out}, {k_out, &p.k_out}}, dtype);
  if (rc != FA_OK) return rc;
  return launch_heads_fwd(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK
                                                                                    : FA_ERR_CUDA;
}

size_t fa_qk_norm_rope_bwd_workspace_bytes(int B, int Hq, int Hkv, int S, int d, int norm) {
  if (!norm || check_common(B, Hq, Hkv, S, S, d, 0, 1.f, FA_BF16) != FA_OK) return 0;
  return static_cast<size_t>(heads_bwd_blocks(B, Hq, Hkv, S, d)) * 2 * d * 4;
}

int fa_qk_norm_rope_bwd(const fa_view* dq_out, const fa_view* dk_out, const fa_view* q,
                        const fa_view* k, const fa_view* dq, const fa_view* dk, float* dq_weight,
                        float* dk_weight, const void* q_weight, const void* k_weight, float eps,
                        const int* positions, const unsigned long long* turns, int rope_dim,
                        int interleaved, float rope_scale, int B, int Hq, int Hkv, int S, int d,
                        int dtype, void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  HeadsParams p{};
  int rc = heads_params(p, q_weight, k_weight, eps, positions, turns, rope_dim, interleaved,
                        rope_scale, B, Hq, Hkv, S, d, dtype);
  if (rc == FA_OK)
    rc = take_views({{dq_out, &p.q_out}, {dk_out, &p.k_out}, {dq, &p.dq}, {dk, &p.dk}}, dtype);
  if (rc != FA_OK) return rc;
  p.n_blocks = heads_bwd_blocks(B, Hq, Hkv, S, d);
  if (q_weight) {
    if ((rc = take_views({{q, &p.q}, {k, &p.k}}, dtype)) != FA_OK) return rc;
    if (!dq_weight || !dk_weight) return FA_ERR_NULL;
    if (((reinterpret_cast<uintptr_t>(dq_weight) | reinterpret_cast<uintptr_t>(dk_weight)) & 3u) != 0)
      return FA_ERR_ALIGN;
    if (!workspace || workspace_bytes < fa_qk_norm_rope_bwd_workspace_bytes(B, Hq, Hkv, S, d, 1))
      return FA_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return FA_ERR_ALIGN;
    p.dwq = dq_weight;
    p.dwk = dk_weight;
    p.dw_part = static_cast<float*>(workspace);
  }
  return launch_heads_bwd(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK
                                                                                    : FA_ERR_CUDA;
}

int fa_qk_norm_rope_append(const fa_view* q, const fa_view* k, const fa_view* v,
                           const fa_view* q_out, void* k_cache, void* v_cache,
                           const int* block_table, const int* seq_lens, const void* q_weight,
                           const void* k_weight, float eps, const unsigned long long* turns,
                           int rope_dim, int interleaved, float rope_scale, int B, int Hq, int Hkv,
                           int Sq, int d, int block_size, int num_blocks, int max_blocks,
                           int dtype, fa_stream_t stream) {
  HeadsParams p{};
  int rc = heads_params(p, q_weight, k_weight, eps, nullptr, turns, rope_dim, interleaved,
                        rope_scale, B, Hq, Hkv, Sq, d, dtype);
  if (rc != FA_OK) return rc;
  if (!block_sizes_ok(Hkv, block_size, num_blocks, max_blocks)) return FA_ERR_SHAPE;
  if ((rc = take_views({{q, &p.q}, {k, &p.k}, {v, &p.v}, {q_out, &p.q_out}}, dtype)) != FA_OK)
    return rc;
  if (!k_cache || !v_cache || !block_table || !seq_lens) return FA_ERR_NULL;
  if (!aligned16(k_cache) || !aligned16(v_cache) ||
      ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(seq_lens)) & 3u) != 0)
    return FA_ERR_ALIGN;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.block_size = block_size; p.num_blocks = num_blocks; p.max_blocks = max_blocks;
  return launch_heads_append(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK : FA_ERR_CUDA;
}

int fa_fwd_span(const void* q, const void* k, const void* v, const int* key_begin,
                const int* key_end, void* out, float* lse, int B, int Hq, int Hkv, int Sq, int Skv,
                int d, float scale, float softcap, const float* slopes, int dtype,
                fa_stream_t stream) {
  int rc = check_common(B, Hq, Hkv, Sq, Skv, d, 0, scale, dtype);
  if (rc != FA_OK) return rc;
  if (dtype == FA_F32) return FA_ERR_DTYPE;   // the span path runs on the tensor cores only
  const SpanArgs mod{key_begin, key_end, slopes, softcap};
  if ((rc = check_span(mod, scale)) != FA_OK) return rc;
  if (!q || !k || !v || !out || !lse) return FA_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(lse))
    return FA_ERR_ALIGN;
  const bool bf16 = dtype == FA_BF16;
  FwdParams p;
  std::memset(&p, 0, sizeof(p));
  if (!make_tmap(&p.tm_q, q, B * Hq, Sq, d, bf16) || !make_tmap(&p.tm_k, k, B * Hkv, Skv, d, bf16) ||
      !make_tmap(&p.tm_v, v, B * Hkv, Skv, d, bf16))
    return FA_ERR_TMA;
  p.out = out;
  p.lse = lse;
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.Sq = Sq; p.Skv = Skv;
  p.scale_log2 = scale * kLog2e;
  p.mod = make_mod(mod, Sq, Skv, scale);
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  return launch_fwd_span(p, d, bf16, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK : FA_ERR_CUDA;
}

size_t fa_bwd_span_workspace_bytes(int B, int Hq, int Hkv, int Sq, int Skv, int d) {
  if (check_common(B, Hq, Hkv, Sq, Skv, d, 0, 1.f, FA_BF16) != FA_OK) return 0;
  return span_ws(ws_layout(B, Hq, Sq, d), B, Hq, Hkv, Sq, Skv, d).total;
}

int fa_bwd_span(const void* q, const void* k, const void* v, const int* key_begin,
                const int* key_end, const void* out, const void* dout, const float* lse, void* dq,
                void* dk, void* dv, int B, int Hq, int Hkv, int Sq, int Skv, int d, float scale,
                float softcap, const float* slopes, int dtype, void* workspace,
                size_t workspace_bytes, fa_stream_t stream) {
  if (dtype == FA_F32) return FA_ERR_DTYPE;
  const SpanArgs mod{key_begin, key_end, slopes, softcap};
  int rc = check_common(B, Hq, Hkv, Sq, Skv, d, 0, scale, dtype);
  if (rc == FA_OK) rc = check_span(mod, scale);
  if (rc != FA_OK) return rc;
  return bwd_impl(q, k, v, out, dout, lse, dq, dk, dv, B, Hq, Hkv, Sq, Skv, d, 0, scale, dtype,
                  workspace, workspace_bytes, stream, &mod);
}

size_t fa_fwd_ragged_paged_workspace_bytes(int B, int Hq, int Hkv, int Sq, int d, int block_size,
                                           int max_blocks) {
  if (check_common(B, Hq, Hkv, Sq, Sq, d, 0, 1.f, FA_BF16) != FA_OK ||
      !paged_sizes_ok(B, Hq, Hkv, Sq, block_size, 1, max_blocks))
    return 0;
  return ragged_plan(B, Hq, Hkv, Sq, d, block_size, max_blocks).total;
}

int fa_fwd_ragged_paged(const void* q, const void* k_cache, const void* v_cache,
                        const int* block_table, const int* seq_lens, void* out, float* lse, int B,
                        int Hq, int Hkv, int Sq, int d, int block_size, int num_blocks,
                        int max_blocks, int window, float scale, float softcap,
                        const float* slopes, int dtype, void* workspace, size_t workspace_bytes,
                        fa_stream_t stream) {
  int rc = check_common(B, Hq, Hkv, Sq, Sq, d, 0, scale, dtype);
  if (rc != FA_OK) return rc;
  if (dtype == FA_F32) return FA_ERR_DTYPE;   // the paged path runs on the tensor cores only
  if (!paged_sizes_ok(B, Hq, Hkv, Sq, block_size, num_blocks, max_blocks) || window < 0)
    return FA_ERR_SHAPE;
  if (!cap_ok(softcap, scale)) return FA_ERR_SCALE;
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !out || !lse) return FA_ERR_NULL;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      !aligned16(lse) ||
      ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(seq_lens) |
        reinterpret_cast<uintptr_t>(slopes)) & 3u) != 0)
    return FA_ERR_ALIGN;
  // (the last of the checks that depend on the caller's arguments, but for its alignment: a
  // call without a workspace tells whether the others pass)
  const RaggedPlan rp = ragged_plan(B, Hq, Hkv, Sq, d, block_size, max_blocks);
  if (!workspace || workspace_bytes < rp.total) return FA_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return FA_ERR_ALIGN;
  uint8_t* wsb = static_cast<uint8_t*>(workspace);
  const bool bf16 = dtype == FA_BF16;
  RaggedParams p;
  std::memset(&p, 0, sizeof(p));
  p.box_rows = std::min(block_size, kTileN);
  if (!make_tmap(&p.tm_k, k_cache, num_blocks * Hkv, block_size, d, bf16, p.box_rows) ||
      !make_tmap(&p.tm_v, v_cache, num_blocks * Hkv, block_size, d, bf16, p.box_rows))
    return FA_ERR_TMA;
  p.mod = make_mod(SpanArgs{nullptr, nullptr, slopes, softcap}, 0, 0, scale);
  // The exponential form is off by up to softcap 2^-20: for caps up to 128 no more than
  // 2^-13 of a weight, half of what rounding it to fp16 is. Choosing the form by the scores
  // gains nothing there (4 tokens of 2 sequences of 20000 and 32768 keys, 32 + 8 heads,
  // d = 128: 46.3 us, by the scores 47.1; 40 rows of 24 sequences of 2000 keys, scores up to
  // the cap: 20.7, by the scores 23.0), so that is for larger caps.
  p.large_cap = softcap > 128.f;
  p.q = q;
  p.out = out;
  p.lse = lse;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.part_out = reinterpret_cast<float*>(wsb + rp.part_out);
  p.part_lse2 = reinterpret_cast<float*>(wsb + rp.part_lse2);
  p.starts = reinterpret_cast<int4*>(wsb + rp.starts);
  p.capacity = static_cast<int>(std::min(static_cast<long long>(max_blocks) * block_size, 0x7fffff80LL));
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.Sq = Sq;
  p.G = Hq / Hkv;
  p.R = rp.R;
  p.block_size = block_size; p.max_blocks = max_blocks; p.num_blocks = num_blocks;
  // a window that no position outgrows hides nothing (and would overflow positions)
  p.window = window < p.capacity ? window : 0;
  p.scale_log2 = scale * kLog2e;
  p.n_ctas = rp.n_ctas;
  p.status = status_ptr();
  if (!p.status) return FA_ERR_CUDA;
  return launch_ragged(p, d, bf16, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK : FA_ERR_CUDA;
}

int fa_last_device_status(fa_stream_t stream, int* status) {
  if (!status) return FA_ERR_NULL;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int value = 0;
  const int zero = 0;
  if (cudaMemcpyFromSymbolAsync(&value, g_status, sizeof(int), 0, cudaMemcpyDeviceToHost, st) !=
          cudaSuccess ||
      cudaMemcpyToSymbolAsync(g_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, st) !=
          cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return FA_ERR_CUDA;
  *status = value;
  return FA_OK;
}

}  // extern "C"
