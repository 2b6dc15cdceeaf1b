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

#include <type_traits>

#include "attention_device.cuh"
#include "launch_memo.h"
#include "q4_device.cuh"

namespace specv {
namespace wattn {

constexpr int kMaxBatch = 4096;
constexpr int kMaxRows = 64;  // packed query rows of a unit

struct Params {
  const uint8_t* q;
  const uint8_t* k;
  const uint8_t* v;
  uint8_t* out;
  const int32_t* block_table;
  const int32_t* ctx_lens;
  int32_t* dev_err;
  int64_t num_blocks, row;
  int rows, heads, kv_heads, gqa, page_shift, max_blocks, window, sinks;
  float scale_log2;
};

template <int D, bool FP16, bool Q4>
__global__ void __launch_bounds__(128) window_attention_kernel(const Params p) {
  constexpr int E = D / 32;  // elements of a lane
  __shared__ float s_m[4], s_l[4], s_o[4][D];
  __shared__ int s_bad;
  const int h = blockIdx.x % p.heads, i = blockIdx.x / p.heads, b = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = h / p.gqa;
  const int64_t at = (((int64_t)b * p.rows + i) * p.heads + h) * D + lane * E;
  const int ctx = p.ctx_lens[b];
  uint16_t* out = reinterpret_cast<uint16_t*>(p.out) + at;
  if (ctx < p.rows || (int64_t)ctx > ((int64_t)p.max_blocks << p.page_shift)) {
    if (warp == 0)
      for (int e = 0; e < E; ++e) out[e] = 0;
    if (ctx != 0 && threadIdx.x == 0) raise_error(p.dev_err, SPEC_DEVERR_CTX_LEN);
    return;
  }
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  const int pos = ctx - p.rows + i, bs = 1 << p.page_shift;
  const int low = p.window ? max(0, pos - p.window + 1) : 0;
  // pages are checked for the whole sequence: all its rows are zeros if one of them is bad
  const int first = p.window ? max(0, ctx - p.rows - p.window + 1) : 0;
  for (int t = threadIdx.x << p.page_shift; t < ctx; t += 128 << p.page_shift) {
    if (t + bs <= first && t >= p.sinks) continue;
    const int page = p.block_table[(int64_t)b * p.max_blocks + (t >> p.page_shift)];
    if (page < 0 || page >= p.num_blocks) s_bad = 1;
  }
  __syncthreads();
  if (s_bad) {
    if (warp == 0)
      for (int e = 0; e < E; ++e) out[e] = 0;
    if (threadIdx.x == 0) raise_error(p.dev_err, SPEC_DEVERR_BLOCK_ID);
    return;
  }
  float q[E], o[E], m = -INFINITY, l = 0.f;
  auto value = [](uint16_t w) { return q4::unpack2<FP16>(w).x; };
  for (int e = 0; e < E; ++e) {
    q[e] = value(reinterpret_cast<const uint16_t*>(p.q)[at + e]) * p.scale_log2;
    o[e] = 0.f;
  }
  auto token = [&](const uint8_t* cache, int64_t slot, float (&x)[E]) {
    if constexpr (Q4) {
      const uint8_t* row = cache + slot * p.row;
      const float2 sm = q4::unpack2<FP16>(reinterpret_cast<const uint32_t*>(row + p.kv_heads * (D / 2))[g]);
      for (int e = 0; e < E; ++e) {
        const int d = g * D + lane * E + e;
        x[e] = fmaf((float)((row[d / 2] >> (4 * (d & 1))) & 15), sm.x, sm.y);
      }
    } else {
      const uint16_t* row = reinterpret_cast<const uint16_t*>(cache) + (slot * p.kv_heads + g) * D + lane * E;
      for (int e = 0; e < E; ++e) x[e] = value(row[e]);
    }
  };
  const int sinks = min(p.sinks, low), total = sinks + pos + 1 - low;
  for (int j = warp; j < total; j += 4) {
    const int t = j < sinks ? j : low + j - sinks;
    const int64_t slot =
        ((int64_t)p.block_table[(int64_t)b * p.max_blocks + (t >> p.page_shift)] << p.page_shift) + (t & (bs - 1));
    float x[E], s = 0.f;
    token(p.k, slot, x);
    for (int e = 0; e < E; ++e) s = fmaf(q[e], x[e], s);
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (s == -INFINITY) continue;
    const float mn = fmaxf(m, s), a = exp2f(m - mn), w = exp2f(s - mn);
    token(p.v, slot, x);
    for (int e = 0; e < E; ++e) o[e] = fmaf(w, x[e], o[e] * a);
    l = l * a + w;
    m = mn;
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
  __syncthreads();
  if (warp != 0) return;
  const float top = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  float sum = 0.f;
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int w = 0; w < 4; ++w) {
    if (s_m[w] == -INFINITY && s_l[w] == 0.f) continue;
    const float a = exp2f(s_m[w] - top);
    sum += s_l[w] * a;
    for (int e = 0; e < E; ++e) o[e] += s_o[w][lane * E + e] * a;
  }
  for (int e = 0; e < E; ++e) out[e] = (uint16_t)q4::pack2<FP16>(o[e] / sum, 0.f);
}

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
  Params p;
  p.q = static_cast<const uint8_t*>(q);
  p.k = static_cast<const uint8_t*>(k_cache);
  p.v = static_cast<const uint8_t*>(v_cache);
  p.out = static_cast<uint8_t*>(out);
  p.block_table = block_table;
  p.ctx_lens = ctx_lens;
  p.dev_err = dev_err;
  p.num_blocks = d->num_blocks;
  p.row = q4::row_bytes(d->num_kv_heads, d->head_dim);
  p.rows = num_rows;
  p.heads = d->num_q_heads;
  p.kv_heads = d->num_kv_heads;
  p.gqa = p.heads / p.kv_heads;
  for (p.page_shift = 0; (1 << p.page_shift) < d->block_size;) ++p.page_shift;
  p.max_blocks = d->max_blocks_per_seq;
  p.window = window;
  p.sinks = sinks;
  p.scale_log2 = (float)(1.4426950408889634 / sqrt((double)d->head_dim));
  const dim3 grid((unsigned)(num_rows * p.heads), (unsigned)d->batch);
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  auto go = [&](auto D) {
    constexpr int kD = decltype(D)::value;
    const bool fp16 = dtype == SPEC_DTYPE_FP16;
    if (q4 && fp16) window_attention_kernel<kD, true, true><<<grid, 128, 0, stream>>>(p);
    else if (q4) window_attention_kernel<kD, false, true><<<grid, 128, 0, stream>>>(p);
    else if (fp16) window_attention_kernel<kD, true, false><<<grid, 128, 0, stream>>>(p);
    else window_attention_kernel<kD, false, false><<<grid, 128, 0, stream>>>(p);
  };
  switch (d->head_dim) {
    case 64: go(std::integral_constant<int, 64>{}); break;
    case 128: go(std::integral_constant<int, 128>{}); break;
    default: go(std::integral_constant<int, 256>{}); break;
  }
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_LAUNCH;
}

}  // namespace wattn
}  // namespace specv

using namespace specv;

extern "C" size_t spec_window_attention_workspace(const spec_attn_desc* d, int32_t num_rows) {
  if (!wattn::desc_ok(d, num_rows) || !wattn::shape_supported(d, num_rows)) return 0;
  return SPEC_ATTN_COUNTER_BYTES;
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
