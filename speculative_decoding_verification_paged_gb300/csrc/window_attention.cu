// Verify attention over a window of a paged cache, 16-bit or 4-bit (sm_103a).
//
//   out_i = sum_t e^(s_it - m_i) V_t / sum_t e^(s_it - m_i),  s_it = q_i . K_t / sqrt(D),
//
// over the tokens t <= p_i that lie in the row's window or among the first ones.
// A 4-bit cache holds codes n with a scale s and a minimum m for each token and
// head: s_it = (s_t n_t . q_i + m_t sum(q_i)) / sqrt(D).
//
// One block per query row and head; four warps take the visible tokens in turns,
// each with a running maximum and sum, and are joined at the end.
#include <math.h>

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
  const int per = kMaxRows / G, groups = (rows + per - 1) / per;
  return (longest / 128 + 2) * d->batch <= INT32_MAX / ((int64_t)d->num_kv_heads * groups);
}

// How the query rows of a kv head are cut into units.
struct Rows {
  int npt, groups, packed;  // query rows of a unit, units, and its packed rows: 8, 16, 32 or 64 at most
};
static Rows rows_for(const spec_attn_desc* d, int rows) {
  const int G = d->num_q_heads / d->num_kv_heads, per = kMaxRows / G;
  Rows r;
  r.groups = (rows + per - 1) / per;
  r.npt = (rows + r.groups - 1) / r.groups;
  for (r.packed = 8; r.packed < r.npt * G;) r.packed *= 2;
  return r;
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
  Launch l;
  int rc;
  switch (D) {
    case 64: rc = q4 ? settings_q4<64>(rows.packed, d->batch, &l) : settings_16<64>(rows.packed, fp16, d->batch, &l); break;
    case 128: rc = q4 ? settings_q4<128>(rows.packed, d->batch, &l) : settings_16<128>(rows.packed, fp16, d->batch, &l); break;
    default: rc = q4 ? settings_q4<256>(rows.packed, d->batch, &l) : settings_16<256>(rows.packed, fp16, d->batch, &l); break;
  }
  if (rc != SPEC_OK) return rc;

  Call c;
  Params& p = c.p;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.q = static_cast<const uint8_t*>(q);
  p.out = static_cast<uint8_t*>(out);
  p.row = q4::row_bytes(d->num_kv_heads, D);
  p.kpar = static_cast<const uint8_t*>(k_cache) + d->num_kv_heads * (D / 2);
  p.vpar = static_cast<const uint8_t*>(v_cache) + d->num_kv_heads * (D / 2);
  p.block_table = block_table;
  p.ctx_lens = ctx_lens;
  p.counters = reinterpret_cast<int32_t*>(ws);
  p.lse = reinterpret_cast<float*>(ws + SPEC_ATTN_COUNTER_BYTES);
  p.opart = p.lse + kMaxPieces * kMaxRows;
  p.dev_err = dev_err;
  p.num_blocks = d->num_blocks;
  p.batch = d->batch;
  p.rows = num_rows;
  p.heads = d->num_q_heads;
  p.kv_heads = d->num_kv_heads;
  p.gqa = p.heads / p.kv_heads;
  p.by_gqa = (65535 + p.gqa) / p.gqa;
  p.npt = rows.npt;
  p.groups = rows.groups;
  for (p.page_shift = 0; (1 << p.page_shift) < bs;) ++p.page_shift;
  p.max_blocks = d->max_blocks_per_seq;
  const int longest = p.max_blocks * bs;  // at most 2^30
  p.window = window >= longest ? 0 : window;
  p.sinks = sinks > longest ? longest : sinks;
  p.slots = l.slots;
  p.fp16 = fp16;
  p.scale_log2 = (float)(1.4426950408889634 / sqrt((double)D));
  c.stream = reinterpret_cast<cudaStream_t>(stream_);

  if (!q4) {
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
  }
  switch (D) {
    case 64: return q4 ? launch_q4<64>(rows.packed, l, c) : launch_16<64>(rows.packed, fp16, l, c);
    case 128: return q4 ? launch_q4<128>(rows.packed, l, c) : launch_16<128>(rows.packed, fp16, l, c);
    default: return q4 ? launch_q4<256>(rows.packed, l, c) : launch_16<256>(rows.packed, fp16, l, c);
  }
}

}  // namespace wattn
}  // namespace specv

using namespace specv;

extern "C" size_t spec_window_attention_workspace(const spec_attn_desc* d, int32_t num_rows) {
  if (!wattn::desc_ok(d, num_rows) || !wattn::shape_supported(d, num_rows)) return 0;
  const int packed = wattn::rows_for(d, num_rows).packed, n = packed < 16 ? 16 : packed;
  return SPEC_ATTN_COUNTER_BYTES + (size_t)wattn::kMaxPieces * (wattn::kMaxRows + (size_t)n * d->head_dim) * 4;
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
