// Verify attention over a tree of drafts and a paged cache (sm_103a).
//
//   out[i] = sum_t e^(s_it - m_i) V_t / sum_t e^(s_it - m_i),  s_it = q_i . K_t / sqrt(D),
//
// over the committed tokens and the node's own line of ancestors.
//
// Plain form of the kernel: one CTA per (sequence, node, query head), 128 keys
// at a time: a thread forms one key's score, the CTA the tile's maximum and
// weights, and each thread accumulates D / 128 (at least one) columns of the output.
#include <math.h>

#include <cuda_fp16.h>

#include "tree_device.cuh"

namespace specv {
namespace tattn {

constexpr int kThreads = 128;
constexpr int kMaxBatch = 4096;
constexpr int kMaxGqa = 128;

struct Params {
  const void* q;
  const void* k;
  const void* v;
  const int32_t* block_table;
  const int32_t* ctx_lens;
  const int32_t* parents;
  void* out;
  int32_t* dev_err;
  int64_t num_blocks;
  int nodes, heads, kv_heads, dim, page, max_blocks, out_dtype;
  float scale_log2;
};

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }

template <typename T>
__global__ void __launch_bounds__(kThreads) tree_attention_kernel(const Params p) {
  __shared__ int32_t s_par[tree::kMaxNodes];
  __shared__ float s_q[256], s_w[kThreads], s_red[4];
  __shared__ int32_t s_page[kThreads];
  const int tid = threadIdx.x, N = p.nodes;
  const int h = blockIdx.x % p.heads, i = blockIdx.x / p.heads % N, b = blockIdx.x / p.heads / N;
  const int g = h / (p.heads / p.kv_heads), D = p.dim;
  const int64_t row = ((int64_t)b * N + i) * p.heads + h;
  if (tid < N) s_par[tid] = p.parents[(int64_t)b * N + tid];
  for (int d = tid; d < D; d += kThreads) s_q[d] = to_f(static_cast<const T*>(p.q)[row * D + d]) * p.scale_log2;
  __syncthreads();
  const bool empty = s_par[0] == SPEC_TREE_UNUSED;
  const int ctx = empty ? 0 : p.ctx_lens[b];
  int err = 0;
  if (!empty) {
    if (__syncthreads_or(tid < N && !tree::parent_ok(s_par, tid))) err |= SPEC_DEVERR_TREE;
    if (ctx < N || (int64_t)ctx > (int64_t)p.max_blocks * p.page) err |= SPEC_DEVERR_CTX_LEN;
  }
  const uint64_t sees = tree::ancestors(s_par, i);
  const int base = ctx - N;
  float m = -INFINITY, l = 0.f, acc[2] = {0.f, 0.f};
  bool bad_page = false;
  const int span = (empty || err) ? 0 : ctx;
  for (int t0 = 0; t0 < span; t0 += kThreads) {
    const int t = t0 + tid;
    float s = -INFINITY;
    int page = 0;
    if (t < ctx) {
      page = p.block_table[(int64_t)b * p.max_blocks + t / p.page];
      if (page < 0 || page >= p.num_blocks) bad_page = true;
      else if (t < base ? sees != 0 : ((sees >> (t - base)) & 1) != 0) {
        const T* k = static_cast<const T*>(p.k) + (((int64_t)page * p.page + t % p.page) * p.kv_heads + g) * D;
        s = 0.f;
        for (int d = 0; d < D; ++d) s += s_q[d] * to_f(k[d]);
      }
    }
    s_page[tid] = page;
    float mx = s;
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (tid % 32 == 0) s_red[tid / 32] = mx;
    __syncthreads();
    const float mn = fmaxf(m, fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3])));
    const float a = m == -INFINITY ? 0.f : exp2f(m - mn);
    s_w[tid] = s == -INFINITY ? 0.f : exp2f(s - mn);
    m = mn;
    if (__syncthreads_or(bad_page)) {
      bad_page = true;
      break;
    }
    l *= a;
    acc[0] *= a;
    acc[1] *= a;
    for (int j = 0; j < kThreads && t0 + j < ctx; ++j) {
      const float w = s_w[j];
      if (w == 0.f) continue;  // keys that the row does not see may hold anything
      l += w;
      const T* v = static_cast<const T*>(p.v) + (((int64_t)s_page[j] * p.page + (t0 + j) % p.page) * p.kv_heads + g) * D;
      for (int c = 0, d = tid; d < D; ++c, d += kThreads) acc[c] += w * to_f(v[d]);
    }
    __syncthreads();
  }
  if (bad_page) err |= SPEC_DEVERR_BLOCK_ID;
  if (err && tid == 0 && h == 0) raise_error(p.dev_err, err);
  const float inv = (err == 0 && l > 0.f) ? 1.f / l : 0.f;
  for (int c = 0, d = tid; d < D; ++c, d += kThreads) {
    const float o = inv == 0.f ? 0.f : acc[c] * inv;
    if (p.out_dtype == SPEC_DTYPE_FP32) static_cast<float*>(p.out)[row * D + d] = o;
    else if (p.out_dtype == SPEC_DTYPE_BF16) static_cast<__nv_bfloat16*>(p.out)[row * D + d] = __float2bfloat16(o);
    else static_cast<__half*>(p.out)[row * D + d] = __float2half(o);
  }
}

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
  if ((int64_t)d->max_blocks_per_seq * bs > INT32_MAX / 2) return false;
  return (int64_t)d->num_blocks * bs <= INT32_MAX;
}

}  // namespace tattn
}  // namespace specv

using namespace specv;

extern "C" size_t spec_tree_attention_workspace(const spec_attn_desc* d, int32_t num_nodes) {
  if (!tattn::desc_ok(d, num_nodes) || !tattn::shape_supported(d, num_nodes)) return 0;
  return 256;
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
  if (workspace == nullptr || workspace_bytes < spec_tree_attention_workspace(d, num_nodes)) return SPEC_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255) != 0) return SPEC_ERR_INVALID_ARG;
  tattn::Params p;
  p.q = q;
  p.k = k_cache;
  p.v = v_cache;
  p.block_table = block_table;
  p.ctx_lens = ctx_lens;
  p.parents = parents;
  p.out = out;
  p.dev_err = dev_err;
  p.num_blocks = d->num_blocks;
  p.nodes = num_nodes;
  p.heads = d->num_q_heads;
  p.kv_heads = d->num_kv_heads;
  p.dim = d->head_dim;
  p.page = d->block_size;
  p.max_blocks = d->max_blocks_per_seq;
  p.out_dtype = out_dtype;
  p.scale_log2 = (float)(1.4426950408889634 / sqrt((double)d->head_dim));
  const int64_t blocks = (int64_t)d->batch * num_nodes * d->num_q_heads;
  if (blocks > INT32_MAX) return SPEC_ERR_UNSUPPORTED;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (dtype == SPEC_DTYPE_BF16) tattn::tree_attention_kernel<__nv_bfloat16><<<(unsigned)blocks, tattn::kThreads, 0, stream>>>(p);
  else tattn::tree_attention_kernel<__half><<<(unsigned)blocks, tattn::kThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_LAUNCH;
}
