// Verify attention over a tree of drafts and a paged cache (sm_103a): argument
// checks, the workspace, tensor maps and the choice of the instance.
//
//   out[i] = sum_t e^(s_it - m_i) V_t / sum_t e^(s_it - m_i),  s_it = q_i . K_t / sqrt(D),
//
// over the committed tokens and the node's own line of ancestors.
//
// Work: the nodes x heads rows that share a kv head are packed into row tiles of
// 128 (the M of the tensor core), up to two row tiles to a unit (sequence, kv head,
// group of rows). The key tiles of all units form one list that is cut over one CTA
// per SM; a unit that was cut is joined by its log-sum-exp inside the kernel: the
// pieces meet, eight at a time, at a counter, and who comes last joins.
//
// A CTA: warp 0 loads K and V pages by TMA into two rings, K ahead of V; warp 1
// issues every product as a whole uniform warp (one elected lane issues; operands in
// a branch of one lane cost a register move each: four MMAs 340 cycles, here 110);
// two softmax warpgroups for each accumulator take half of a tile's keys each. The
// scores stay in tensor memory, where P replaces them as operand A of the second
// product. The running maximum follows only when it grows by more than 2^8 (fp16: 2^4,
// and it may fall too), so that the accumulator is rarely rescaled; the row sum is fp32.
//
// Numbers: 16-bit output rounds P to 16 bits once (bf16 2.3e-3 off, 1.7e-3 with the
// output's own rounding alone; a second part of P takes 83 us for 65 in the batch of
// 32 below, 127 for 81 with 16 nodes, 722 to 768 for 546 to 552 in the long contexts;
// fp32 output is there for those who want it). fp32 output adds a second part of
// P (fp16) or two (bf16), since a single part would leave an error of half a step of
// the 16-bit type. The tensor core cuts its fp32 sums instead of rounding them, so
// with fp32 output the accumulator is folded into fp32 sums every 512 keys: at head
// dim 256 the error was 2.2e-5 without folds and is 1.8e-6 with them and the small
// parts added first.
//
// What bounds it (one GB300, L2 flushed): batch 32, 64 nodes, 32/8 heads, head dim
// 128, context 2K: 71 us of 44.5 us for its bytes; tensor pipe 38% active, DRAM 49%,
// so neither: the chain scores -> softmax -> product and the ends of units. Contexts of
// 32K to 128K: 491 to 628 us of 395 us, at about 1370 W, where the clock falls to about
// 1.6 GHz. Head dim 256, fp32 output: 462 to 521 us of 341 us, in a graph 485; there
// 430 without folds (256 KB a CTA through L2, about 5000 cycles each) and 398 with
// 16-bit output.
#include <math.h>

#include "launch_memo.h"
#include "tensor_map.h"
#include "tree_attention.cuh"

namespace specv {
namespace tattn {

constexpr int kMaxBatch = 4096;
constexpr int kMaxGqa = 128;

static bool desc_ok(const spec_attn_desc* d, int nodes) {
  if (d == nullptr) return false;
  if (d->batch < 0 || d->num_q_heads < 1 || d->num_kv_heads < 1) return false;
  if (d->num_q_heads % d->num_kv_heads != 0) return false;
  return d->max_blocks_per_seq >= 1 && d->num_blocks >= 1 && nodes >= 1;
}

static bool shape_supported(const spec_attn_desc* d, int nodes) {
  const int D = d->head_dim, bs = d->block_size;
  if (D != 64 && D != 128 && D != 256) return false;
  if (bs != 16 && bs != 32 && bs != 64 && bs != 128) return false;
  if (nodes > tree::kMaxNodes || d->num_q_heads / d->num_kv_heads > kMaxGqa || d->batch > kMaxBatch) return false;
  const int64_t longest = (int64_t)d->max_blocks_per_seq * bs;
  if (longest > INT32_MAX / 2) return false;
  // tile counts of all units are 32-bit (units: at most N row tiles a kv head)
  const int most = kRows / (d->num_q_heads / d->num_kv_heads), tiles = (nodes + most - 1) / most;
  if ((longest / 64 + 1) * d->batch > INT32_MAX / ((int64_t)d->num_kv_heads * tiles)) return false;
  return (int64_t)d->num_blocks * bs <= INT32_MAX;  // TMA row coordinates are 32-bit
}

// How the N * G query rows of a kv head are cut: row tiles of npt nodes, mt of them to a unit.
struct Rows {
  int mt, groups, npt;
};
static int streams_for(int D, int terms) {  // accumulators of the instance
  switch (D) {
    case 64: return terms == 3 ? Cfg<64, 1, 3, false>::STREAMS : Cfg<64, 1, 1, false>::STREAMS;
    case 128: return terms == 3 ? Cfg<128, 1, 3, false>::STREAMS : Cfg<128, 1, 1, false>::STREAMS;
    default: return Cfg<256, 1, 3, false>::STREAMS;
  }
}
static Rows rows_for(const spec_attn_desc* d, int nodes, int terms) {
  const int most = kRows / (d->num_q_heads / d->num_kv_heads);
  const int tiles = (nodes + most - 1) / most;
  Rows r;
  r.mt = tiles > 1 ? streams_for(d->head_dim, terms) : 1;
  r.groups = (tiles + r.mt - 1) / r.mt;
  r.npt = (nodes + r.mt * r.groups - 1) / (r.mt * r.groups);
  return r;
}

struct Layout {
  size_t lse, opart, folds, total;
};
static Layout layout_for(const spec_attn_desc* d, int nodes) {  // room for any output type
  Layout L;
  const size_t slots = 2 * (size_t)kMaxGrid * rows_for(d, nodes, 1).mt, row_tile = (size_t)kRows * d->head_dim * 4;
  L.lse = SPEC_ATTN_COUNTER_BYTES;
  L.opart = L.lse + attn::align256(slots * kRows * 4);
  L.folds = L.opart + slots * row_tile;
  L.total = L.folds + (size_t)kMaxGrid * streams_for(d->head_dim, 1) * row_tile;
  return L;
}

}  // namespace tattn
}  // namespace specv

using namespace specv;

extern "C" size_t spec_tree_attention_workspace(const spec_attn_desc* d, int32_t num_nodes) {
  if (!tattn::desc_ok(d, num_nodes) || !tattn::shape_supported(d, num_nodes)) return 0;
  return tattn::layout_for(d, num_nodes).total;
}

extern "C" int spec_tree_attention(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                                   const int32_t* ctx_lens, const int32_t* parents, int32_t num_nodes, void* out,
                                   int32_t dtype, int32_t out_dtype, const spec_attn_desc* d, void* workspace,
                                   size_t workspace_bytes, int32_t* dev_err, spec_stream_t stream_) {
  if (!tattn::desc_ok(d, num_nodes)) return SPEC_ERR_INVALID_ARG;
  if (dtype != SPEC_DTYPE_BF16 && dtype != SPEC_DTYPE_FP16) return SPEC_ERR_INVALID_ARG;
  if (out_dtype != dtype && out_dtype != SPEC_DTYPE_FP32) return SPEC_ERR_INVALID_ARG;
  if (d->batch == 0) return SPEC_OK;
  if (!q || !k_cache || !v_cache || !block_table || !ctx_lens || !parents || !out) return SPEC_ERR_INVALID_ARG;
  if (!tattn::shape_supported(d, num_nodes)) return SPEC_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache) |
       reinterpret_cast<uintptr_t>(out)) & 15)
    return SPEC_ERR_INVALID_ARG;
  const tattn::Layout L = tattn::layout_for(d, num_nodes);
  if (workspace == nullptr || workspace_bytes < L.total) return SPEC_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255) != 0) return SPEC_ERR_INVALID_ARG;

  // Parts of P: one where the output is rounded to the input type anyway; for fp32 output as many as keep 22 to 24 bits
  // of it (two fp16 parts, down to fp16's smallest step, see Cfg::SHIFT; three bf16 ones; two bf16 parts alone would be
  // 2.2e-6 off).
  const bool fp16 = dtype == SPEC_DTYPE_FP16;
  const int D = d->head_dim, terms = out_dtype != SPEC_DTYPE_FP32 ? 1 : fp16 ? 2 : 3;
  const tattn::Rows rows = tattn::rows_for(d, num_nodes, terms);
  tattn::Launch l;
  int rc;
  switch (D) {
    case 64: rc = tattn::settings<64>(rows.mt, terms, fp16, d->batch, &l); break;
    case 128: rc = tattn::settings<128>(rows.mt, terms, fp16, d->batch, &l); break;
    default: rc = tattn::settings<256>(rows.mt, terms, fp16, d->batch, &l); break;
  }
  if (rc != SPEC_OK) return rc;

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  tattn::Call c;
  tattn::Params& p = c.p;
  p.block_table = block_table;
  p.ctx_lens = ctx_lens;
  p.parents = parents;
  p.out = out;
  p.counters = reinterpret_cast<int32_t*>(ws);
  p.lse = reinterpret_cast<float*>(ws + L.lse);
  p.opart = reinterpret_cast<float4*>(ws + L.opart);
  p.folds = reinterpret_cast<float4*>(ws + L.folds);
  p.dev_err = dev_err;
  p.num_blocks = d->num_blocks;
  p.batch = d->batch;
  p.nodes = num_nodes;
  p.heads = d->num_q_heads;
  p.kv_heads = d->num_kv_heads;
  p.gqa = d->num_q_heads / d->num_kv_heads;
  p.npt = rows.npt;
  p.groups = rows.groups;
  p.page_shift = 0;
  while ((1 << p.page_shift) < d->block_size) ++p.page_shift;
  p.max_blocks = d->max_blocks_per_seq;
  p.kslots = l.kslots;
  p.vslots = l.vslots;
  p.out_f32 = out_dtype == SPEC_DTYPE_FP32;
  p.out_wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
  p.scale_log2 = (float)(1.4426950408889634 / sqrt((double)D));
  c.stream = reinterpret_cast<cudaStream_t>(stream_);

  EncodeTiledFn encode = encode_fn();
  if (encode == nullptr) return SPEC_ERR_LAUNCH;
  const CUtensorMapDataType type = fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  auto map = [&](CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                 const cuuint32_t* box) {
    return encode(m, type, rank, const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  // queries [B][N][Hq][D]: a box holds the heads of one kv head for the nodes of a row tile; nodes past N read zeros
  const cuuint64_t qd[4] = {(cuuint64_t)D, (cuuint64_t)p.heads, (cuuint64_t)num_nodes, (cuuint64_t)d->batch};
  const cuuint64_t qs[3] = {qd[0] * 2, qd[0] * qd[1] * 2, qd[0] * qd[1] * qd[2] * 2};
  const cuuint32_t qbox[4] = {64, (cuuint32_t)p.gqa, (cuuint32_t)p.npt, 1};
  // K and V [token rows][Hkv][D]: a box holds one head's rows of a page (or of a tile), 64 elements wide; where that is
  // a whole tile, all of its slices, slice by slice
  const int tk = D <= 128 ? 128 : 64;
  const bool whole = d->block_size >= tk;
  const cuuint64_t row_bytes = (cuuint64_t)p.kv_heads * D * 2;
  const cuuint64_t kd[4] = {64, (cuuint64_t)d->num_blocks * d->block_size, (cuuint64_t)D / 64, (cuuint64_t)p.kv_heads};
  const cuuint64_t ks[3] = {row_bytes, 128, (cuuint64_t)D * 2};
  const cuuint32_t kbox[4] = {64, (cuuint32_t)(whole ? tk : d->block_size), whole ? (cuuint32_t)D / 64 : 1, 1};
  if (!map(&c.tq, q, 4, qd, qs, qbox) || !map(&c.tk, k_cache, 4, kd, ks, kbox) || !map(&c.tv, v_cache, 4, kd, ks, kbox))
    return SPEC_ERR_LAUNCH;
  switch (D) {
    case 64: return tattn::launch<64>(rows.mt, terms, fp16, l, c);
    case 128: return tattn::launch<128>(rows.mt, terms, fp16, l, c);
    default: return tattn::launch<256>(rows.mt, terms, fp16, l, c);
  }
}
