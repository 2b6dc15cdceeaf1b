// Acceptance of a tree of drafts: greedy walk or speculative sampling with
// several candidates a position (sm_103a).
//
// The residual after r refused children of a node has the closed form
//   w = max(0, a p - b q),  a_0 = 1, b_0 = 0,  a' = a / Z, b' = (b + 1) / Z,
//   Z = sum max(0, a p - (b + 1) q),
// because max(0, max(0, x) / Z - q) = max(0, x / Z - q): two scalars hold it.
// Without draft probabilities the residual is p without the refused tokens.
//
// Plain form of the kernel: one CTA per row walks its nodes.
#include <math.h>

#include "tree_device.cuh"

namespace specv {
namespace tacc {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxVocab = 1 << 30;

struct Params {
  const float* logits;
  const int32_t* tokens;
  const int32_t* parents;
  const float* probs;
  const int32_t* mode;
  const float* temperature;
  int32_t* out_tokens;
  int32_t* path;
  int32_t* accept_len;
  int32_t* dev_err;
  uint32_t seed_lo, seed_hi;
  int nodes, vocab;
};

__global__ void __launch_bounds__(kThreads) tree_accept_kernel(const Params p) {
  __shared__ int32_t s_par[tree::kMaxNodes], s_tok[tree::kMaxNodes], s_out[tree::kMaxNodes], s_path[tree::kMaxNodes];
  __shared__ int32_t s_gone[tree::kMaxNodes];
  __shared__ float s_f[kWarps];
  __shared__ int32_t s_i[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x, N = p.nodes, V = p.vocab;
  if (tid < N) {
    s_par[tid] = p.parents[(int64_t)b * N + tid];
    s_tok[tid] = p.tokens[(int64_t)b * N + tid];
    s_out[tid] = s_path[tid] = -1;
  }
  __syncthreads();
  auto block_sum = [&](float v) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (lane == 0) s_f[warp] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < kWarps; ++w) v += s_f[w];
    return v;
  };
  auto block_best = [&](float v, int i, float& bv, int& bi) {  // largest value, lowest index on ties
    for (int o = 16; o > 0; o >>= 1) {
      const float ov = __shfl_xor_sync(0xffffffffu, v, o);
      const int oi = __shfl_xor_sync(0xffffffffu, i, o);
      if (ov > v || (ov == v && oi < i)) v = ov, i = oi;
    }
    __syncthreads();
    if (lane == 0) s_f[warp] = v, s_i[warp] = i;
    __syncthreads();
    bv = s_f[0];
    bi = s_i[0];
    for (int w = 1; w < kWarps; ++w)
      if (s_f[w] > bv || (s_f[w] == bv && s_i[w] < bi)) bv = s_f[w], bi = s_i[w];
  };
  const int mode = p.mode[b];
  const float T = mode == SPEC_MODE_SAMPLE ? p.temperature[b] : 1.f;
  int m = -1;
  if (s_par[0] != SPEC_TREE_UNUSED) {
    int err = 0;
    if (mode != SPEC_MODE_GREEDY && mode != SPEC_MODE_SAMPLE) err |= SPEC_DEVERR_MODE;
    if (!(T > 0.f) || !isfinite(T)) err |= SPEC_DEVERR_TEMPERATURE;
    if (__syncthreads_or(tid < N && !tree::parent_ok(s_par, tid))) err |= SPEC_DEVERR_TREE;
    if (__syncthreads_or(tid > 0 && tid < N && s_par[tid] != SPEC_TREE_UNUSED && (s_tok[tid] < 0 || s_tok[tid] >= V)))
      err |= SPEC_DEVERR_TOKEN;
    if (err) {
      if (tid == 0) raise_error(p.dev_err, err);
    } else {
      const float c2 = (1.0f / T) * 1.4426950408889634f;
      int cur = 0;
      m = 0;
      for (;;) {
        const float* l = p.logits + ((int64_t)b * N + cur) * V;
        const float* q = p.probs ? p.probs + ((int64_t)b * N + cur) * V : nullptr;
        float mx = -INFINITY;
        int at = INT32_MAX;
        for (int x = tid; x < V; x += kThreads)
          if (l[x] > mx || at == INT32_MAX) mx = l[x], at = x;
        float M;
        int top;
        block_best(mx, at, M, top);
        int next = -1, last = top;
        if (mode == SPEC_MODE_GREEDY) {
          for (int c = N - 1; c > cur; --c)
            if (s_par[c] == cur && s_tok[c] == top) next = c;
        } else {
          float s = 0.f;
          for (int x = tid; x < V; x += kThreads) s += exp2f((l[x] - M) * c2);
          const float invZ = 1.f / block_sum(s);
          float a = 1.f, bq = 0.f;
          int gone = 0;  // refused tokens (no draft probabilities)
          // the residual's weight of x, for given scalars and number of refused tokens
          auto weight = [&](int x, float a_, float b_, int n_) {
            const float w = exp2f((l[x] - M) * c2) * invZ * a_;
            if (q) return fmaxf(0.f, w - b_ * q[x]);
            for (int k = 0; k < n_; ++k)
              if (s_gone[k] == x) return 0.f;
            return w;
          };
          for (int c = cur + 1; c < N && next < 0; ++c) {
            if (s_par[c] != cur) continue;
            const int x = s_tok[c];
            const float u = word_to_uniform(philox4x32_10(0u, (uint32_t)(c - 1), (uint32_t)b, 0u, p.seed_lo, p.seed_hi).v[0]);
            if (u * (q ? q[x] : 1.f) < weight(x, a, bq, gone)) {
              next = c;
              break;
            }
            __syncthreads();
            if (tid == 0) s_gone[gone] = x;
            __syncthreads();
            float z = 0.f;
            for (int y = tid; y < V; y += kThreads) z += weight(y, a, bq + 1.f, gone + 1);
            z = block_sum(z);
            if (z > 0.f) {
              a /= z;
              bq = (bq + 1.f) / z;
              ++gone;
            }
          }
          if (next < 0) {
            float best = -1.f;
            int bx = INT32_MAX;
            for (int x = tid; x < V; x += kThreads) {
              const float w = weight(x, a, bq, gone);
              const uint32_t r = philox4x32_10((uint32_t)(x / 4), (uint32_t)cur, (uint32_t)b, 1u, p.seed_lo, p.seed_hi).v[x % 4];
              const float key = w / -logf(word_to_uniform(r));
              if (key > best) best = key, bx = x;
            }
            float kv;
            block_best(best, bx, kv, last);
          }
        }
        if (tid == 0) {
          s_path[m] = cur;
          s_out[m] = next < 0 ? last : s_tok[next];
        }
        if (next < 0) break;
        cur = next;
        ++m;
      }
    }
  }
  __syncthreads();
  if (tid < N) {
    p.out_tokens[(int64_t)b * N + tid] = s_out[tid];
    p.path[(int64_t)b * N + tid] = s_path[tid];
  }
  if (tid == 0) p.accept_len[b] = m;
}

}  // namespace tacc
}  // namespace specv

using namespace specv;

extern "C" int spec_tree_accept(const float* target_logits, const int32_t* tokens, const int32_t* parents,
                                const float* draft_probs, uint64_t philox_seed, const int32_t* mode,
                                const float* temperature, int32_t* out_tokens, int32_t* path, int32_t* accept_len,
                                int32_t batch, int32_t num_nodes, int32_t vocab, int32_t* dev_err,
                                spec_stream_t stream_) {
  if (batch < 0 || num_nodes < 1 || vocab < 1) return SPEC_ERR_INVALID_ARG;
  if (batch == 0) return SPEC_OK;
  if (!target_logits || !tokens || !parents || !mode || !temperature || !out_tokens || !path || !accept_len)
    return SPEC_ERR_INVALID_ARG;
  if (num_nodes > tree::kMaxNodes || vocab > tacc::kMaxVocab) return SPEC_ERR_UNSUPPORTED;
  tacc::Params p;
  p.logits = target_logits;
  p.tokens = tokens;
  p.parents = parents;
  p.probs = draft_probs;
  p.mode = mode;
  p.temperature = temperature;
  p.out_tokens = out_tokens;
  p.path = path;
  p.accept_len = accept_len;
  p.dev_err = dev_err;
  p.seed_lo = (uint32_t)(philox_seed & 0xFFFFFFFFu);
  p.seed_hi = (uint32_t)(philox_seed >> 32);
  p.nodes = num_nodes;
  p.vocab = vocab;
  tacc::tree_accept_kernel<<<(unsigned)batch, tacc::kThreads, 0, reinterpret_cast<cudaStream_t>(stream_)>>>(p);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_LAUNCH;
}
