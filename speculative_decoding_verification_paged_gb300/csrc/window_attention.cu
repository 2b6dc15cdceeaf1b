// Verify attention over a window of a paged cache, 16-bit or 4-bit (sm_103a).
//
//   out_i = sum_t e^(s_it - m_i) V_t / sum_t e^(s_it - m_i),  s_it = q_i . K_t / sqrt(D),
//
// over the tokens t <= p_i that lie in the row's window or among the first ones.
// A 4-bit cache holds codes n with a scale s and a minimum m for each token and
// head: s_it = (s_t n_t . q_i + m_t sum(q_i)) / sqrt(D), and the same for V.
//
// A unit is some packed rows (query row x head of the group) of one sequence and kv
// head, for all of which K and V are read once: over 16 bits up to 64 rows; over 4 bits
// eight warps' worth, each with 16 or 32 rows of a head (up to eight heads, whose codes
// share a token row). More rows are more units, which read K and V again. Pages that no
// row sees are not read; pages of the sinks and of the window form one list. The device
// plans the call from ctx_lens (window_plan.cuh): units go to the blocks in turns, and are
// cut where that shortens the longest block's work; a kernel of its own joins cut units
// (window_join.cuh).
//
// Softmax in one pass: a row's weights are 2^(score - reference). The reference is set
// 2^7 below the largest weight of the first keys, and again only when a later weight
// passes 2^15, so that most tiles neither search a maximum nor scale what was summed.
//
// 16 bits (window_attention.cuh): bound by HBM, K and V by tensor copies into tcgen05.
// 32 sequences with a window of 4096 tokens, 8 kv heads of 128, 16 packed rows: 548 MB
// in 105 us between events with L2 flushed, 91 among other calls, 77 to 88% of the copy
// rate; 64 ragged sequences, 4 heads of 256, 24 rows: 539 MB in 115 us, 109 among others.
//
// 4 bits (q4_attention.cuh): bound by instructions, since a byte holds four times the
// work: unpacking, and mma with 16 rows a time.
#include <math.h>

#include "q4_attention_launch.h"
#include "tensor_map.h"
#include "window_attention_launch.h"

namespace specv {
namespace wattn {

static bool desc_ok(const spec_attn_desc* d, int rows) {
  if (d == nullptr) return false;
  if (d->batch < 0 || d->num_q_heads < 1 || d->num_kv_heads < 1) return false;
  if (d->num_q_heads % d->num_kv_heads != 0) return false;
  return d->max_blocks_per_seq >= 1 && d->num_blocks >= 1 && rows >= 1;
}

static bool shape_supported(const spec_attn_desc* d, int rows) {
  const int D = d->head_dim, bs = d->block_size, G = d->num_q_heads / d->num_kv_heads;
  if (D != 64 && D != 128 && D != 256) return false;
  if (bs != 16 && bs != 32 && bs != 64 && bs != 128) return false;
  if (rows > 64 || G > kMaxRows || d->batch > kMaxBatch) return false;
  const int64_t longest = (int64_t)d->max_blocks_per_seq * bs;
  if (longest > (1 << 30) || d->num_blocks > INT32_MAX / bs) return false;
  if ((longest / 32 + 2) * d->batch > INT32_MAX) return false;
  const int groups = (rows * G + 15) / 16;  // at most
  return (longest / 128 + 2) * d->batch <= INT32_MAX / ((int64_t)d->num_kv_heads * groups);
}

// How the query rows of a kv head are cut into units.
struct Rows {
  int per, groups, packed;  // packed rows of a unit, units, and what its kernel has room for: 8, 16, 32 or 64
};
static Rows rows_for(const spec_attn_desc* d, int rows) {  // whole query rows
  const int G = d->num_q_heads / d->num_kv_heads, per = kMaxRows / G;
  Rows r;
  r.groups = (rows + per - 1) / per;
  r.per = (rows + r.groups - 1) / r.groups * G;
  for (r.packed = 8; r.packed < r.per;) r.packed *= 2;
  return r;
}
static size_t workspace_16(const spec_attn_desc* d, int rows) {
  return SPEC_ATTN_COUNTER_BYTES + kCutBytes + (size_t)kMaxPieces * rows_for(d, rows).per * (2 + d->head_dim) * 4;
}
static size_t workspace_q4(const spec_attn_desc* d, int rows) {
  const int all = rows * (d->num_q_heads / d->num_kv_heads);
  switch (d->head_dim) {
    case 64: return qattn::workspace<64>(d, rows, all);
    case 128: return qattn::workspace<128>(d, rows, all);
    default: return qattn::workspace<256>(d, rows, all);
  }
}

static int call(bool q4, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                const int32_t* ctx_lens, int32_t num_rows, int32_t window, int32_t sinks, void* out, int32_t dtype,
                const spec_attn_desc* d, void* workspace, size_t workspace_bytes, int32_t* dev_err,
                spec_stream_t stream_) {
  if (!desc_ok(d, num_rows) || window < 0 || sinks < 0) return SPEC_ERR_INVALID_ARG;
  if (dtype != SPEC_DTYPE_BF16 && dtype != SPEC_DTYPE_FP16) return SPEC_ERR_INVALID_ARG;
  if (d->batch == 0) return SPEC_OK;
  if (!q || !k_cache || !v_cache || !block_table || !ctx_lens || !out) return SPEC_ERR_INVALID_ARG;
  if (!shape_supported(d, num_rows)) return SPEC_ERR_UNSUPPORTED;
  if (q4 && spec_q4_row_bytes(d->num_kv_heads, d->head_dim) == 0) return SPEC_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache) |
       reinterpret_cast<uintptr_t>(out)) & 15)
    return SPEC_ERR_INVALID_ARG;
  if (workspace == nullptr || workspace_bytes < spec_window_attention_workspace(d, num_rows)) return SPEC_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255) != 0) return SPEC_ERR_INVALID_ARG;
  const Rows rows = rows_for(d, num_rows);
  const bool fp16 = dtype == SPEC_DTYPE_FP16;
  const int D = d->head_dim, bs = d->block_size;

  Call c;
  Params& p = c.p;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.q = static_cast<const uint8_t*>(q);
  p.out = static_cast<uint8_t*>(out);
  p.row = q4::row_bytes(d->num_kv_heads, D);
  p.k = static_cast<const uint8_t*>(k_cache);
  p.v = static_cast<const uint8_t*>(v_cache);
  p.block_table = block_table;
  p.ctx_lens = ctx_lens;
  // the first bytes are other kernels' counters, which stay zero
  p.cut_units = reinterpret_cast<CutUnit*>(ws + SPEC_ATTN_COUNTER_BYTES);
  p.stat = reinterpret_cast<float2*>(ws + SPEC_ATTN_COUNTER_BYTES + kCutBytes);
  p.opart = reinterpret_cast<float*>(p.stat + (size_t)kMaxPieces * rows.per);
  p.dev_err = dev_err;
  p.num_blocks = d->num_blocks;
  p.batch = d->batch;
  p.rows = num_rows;
  p.heads = d->num_q_heads;
  p.kv_heads = d->num_kv_heads;
  p.gqa = p.heads / p.kv_heads;
  p.by_gqa = ((1 << 20) + p.gqa - 1) / p.gqa;
  p.per = p.sub = rows.per;
  p.unit_heads = p.parts = p.pairs = 1;
  p.by_sub = ((1 << 16) + p.sub - 1) / p.sub;
  p.by_parts = 1 << 8;
  p.groups = rows.groups;
  p.head_units = p.kv_heads;
  for (p.page_shift = 0; (1 << p.page_shift) < bs;) ++p.page_shift;
  p.max_blocks = d->max_blocks_per_seq;
  const int longest = p.max_blocks * bs;  // at most 2^30
  p.window = window >= longest ? 0 : window;
  p.sinks = sinks > longest ? longest : sinks;
  p.slots = 0;
  p.fp16 = fp16;
  p.scale_log2 = (float)(1.4426950408889634 / sqrt((double)D));
  p.ref_unit = q4 ? 1.f : p.scale_log2;
  c.stream = reinterpret_cast<cudaStream_t>(stream_);

  if (q4) {
    switch (D) {
      case 64: return qattn::launch<64>(d, num_rows * p.gqa, p, c.stream);
      case 128: return qattn::launch<128>(d, num_rows * p.gqa, p, c.stream);
      default: return qattn::launch<256>(d, num_rows * p.gqa, p, c.stream);
    }
  }
  Launch l;
  int rc;
  switch (D) {
    case 64: rc = settings_16<64>(rows.packed, fp16, d->batch, &l); break;
    case 128: rc = settings_16<128>(rows.packed, fp16, d->batch, &l); break;
    default: rc = settings_16<256>(rows.packed, fp16, d->batch, &l); break;
  }
  if (rc != SPEC_OK) return rc;
  p.slots = l.slots;
  EncodeTiledFn encode = encode_fn();
  if (encode == nullptr) return SPEC_ERR_LAUNCH;
  // K and V [token rows][Hkv][D]: a box holds one head's rows of a page, 64 elements wide
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.kv_heads, (cuuint64_t)d->num_blocks * bs};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)p.kv_heads * D * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)bs}, ones[3] = {1, 1, 1};
  auto map = [&](CUtensorMap* m, const void* base) {
    return encode(m, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base),
                  dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (!map(&c.tk, k_cache) || !map(&c.tv, v_cache)) return SPEC_ERR_LAUNCH;
  switch (D) {
    case 64: return launch_16<64>(rows.packed, fp16, l, c);
    case 128: return launch_16<128>(rows.packed, fp16, l, c);
    default: return launch_16<256>(rows.packed, fp16, l, c);
  }
}

}  // namespace wattn
}  // namespace specv

using namespace specv;

extern "C" size_t spec_window_attention_workspace(const spec_attn_desc* d, int32_t num_rows) {
  if (!wattn::desc_ok(d, num_rows) || !wattn::shape_supported(d, num_rows)) return 0;
  const size_t a = wattn::workspace_16(d, num_rows), b = wattn::workspace_q4(d, num_rows);
  return a > b ? a : b;
}

extern "C" int spec_window_attention(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                                     const int32_t* ctx_lens, int32_t num_rows, int32_t window, int32_t sinks, void* out,
                                     int32_t dtype, const spec_attn_desc* d, void* workspace, size_t workspace_bytes,
                                     int32_t* dev_err, spec_stream_t stream) {
  return wattn::call(false, q, k_cache, v_cache, block_table, ctx_lens, num_rows, window, sinks, out, dtype, d, workspace,
                     workspace_bytes, dev_err, stream);
}

extern "C" int spec_q4_attention(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                                 const int32_t* ctx_lens, int32_t num_rows, int32_t window, int32_t sinks, void* out,
                                 int32_t dtype, const spec_attn_desc* d, void* workspace, size_t workspace_bytes,
                                 int32_t* dev_err, spec_stream_t stream) {
  return wattn::call(true, q, k_cache, v_cache, block_table, ctx_lens, num_rows, window, sinks, out, dtype, d, workspace,
                     workspace_bytes, dev_err, stream);
}
