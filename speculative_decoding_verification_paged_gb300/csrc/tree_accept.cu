// Acceptance of a tree of drafts: greedy walk or speculative sampling with
// several candidates a position (sm_103a).
//
// The residual after r refused children of a node has the closed form
//   w = max(0, a p - b q),  a_0 = 1, b_0 = 0,  a' = a / Z, b' = (b + 1) / Z,
//   Z = sum max(0, a p - (b + 1) q),
// because max(0, max(0, x) / Z - q) = max(0, x / Z - q): two scalars hold it.
// Without draft probabilities the residual is p without the refused tokens.
//
// Design (GB300): the chain call's (accept.cu): one thread-block cluster per row,
// its CTAs splitting the vocabulary, partials pushed into every CTA of the
// cluster and counted by mbarriers, so that all warps reach the same decision
// without a block-wide or cluster-wide barrier. The walk reads the rows of the
// nodes that it visits and no others: per node one pass for the statistics (or
// the argmax), one pass for every refused child but the last (the mass of the
// next residual; none without draft probabilities, where it is 1 minus the
// refused tokens' share), and one exponential race at the last node; all but the
// first pass over a row come from L2. Every warp keeps the row's nodes in shared
// memory of its own (lane l writes nodes l and l + 32; no block-wide barrier):
// parent, token, the uniform of its test and, for the children of the current
// node, the target logit and the draft probability, whose loads are in flight
// during the statistics pass. In registers they would spill in the race.
//
// What bounds it (one GB300, L2 flushed): 32 rows of 128K entries, sampled, 38 to 45 us
// by the draws; the roots alone are 16.4 MB, 2.4 us. DRAM is 26% busy and the stalls are on loads:
// each visited node is a chain of dependent passes over its row, and the race after
// the last one draws a uniform for every entry.
#include <math.h>

#include <type_traits>

#include "accept_device.cuh"
#include "tree_device.cuh"

namespace specv {
namespace tacc {

using namespace acc;

constexpr int kNB = 8;  // float4 groups per thread in flight together (statistics, argmax)
constexpr int kRB = 2;  // ... in the race, whose Philox words and bounds fill the registers
constexpr int kSB = 4;  // ... in a residual's sum
constexpr int64_t kPrefetchMaxBytes = 32ll << 20;  // one node's rows over the batch, at most, to prefetch
constexpr float kExactMass = 0.0625f;  // remaining mass below which it is summed instead of subtracted

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
  int batch, nodes, vocab, slice, csize;
  int vec;       // rows are 16-byte aligned: float4 loads
  int prefetch;  // see the walk
};

// A warp's copy of the row.
struct Nodes {
  int32_t par[tree::kMaxNodes], tok[tree::kMaxNodes], path[tree::kMaxNodes];
  int32_t gone[tree::kMaxNodes];  // refused tokens of the current node (no draft probabilities)
  float u[tree::kMaxNodes], ld[tree::kMaxNodes], qd[tree::kMaxNodes];
};

// Registers bound the CTAs resident per SM (512 threads at 128 registers each: with less the passes spill).
template <int T>
__global__ void __launch_bounds__(T, 512 / T) tree_accept_kernel(const Params p) {
  constexpr int kWarps = T / 32;
  constexpr int kStep = kNB * T;  // groups per batch of the block
  constexpr uint32_t kAll = 0xffffffffu;
  __shared__ Shared sh;
  __shared__ Nodes nodes_of_warp[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int csize = p.csize, rank = (int)cluster_ctarank(), nclusters = (int)(gridDim.x / (unsigned)csize);
  const int N = p.nodes, V = p.vocab;
  Nodes& nd = nodes_of_warp[warp];
  const int x0 = rank * p.slice;       // a multiple of 4: group g holds Philox counter x0/4 + g
  const int n = min(p.slice, V - x0);  // >= 1 by construction of the slice
  const int ngroups = (n + 3) >> 2;
  const bool vec = p.vec != 0;
  const int nparts = csize * kWarps;
  int xs = 0;           // exchanges so far (slot parity)
  bool joined = false;  // the start-up cluster barrier was waited on
  if (tid == 0) {
    mbar_init(&sh.xbar[0], 1);  // the local arrival sets the exchange's byte count
    mbar_init(&sh.xbar[1], 1);
    fence_mbar_init();  // visible to the cluster before any peer can push
  }
  __syncthreads();
  cluster_arrive_relaxed();

  auto load4 = [&](const float* src, int g, float fill) -> float4 {
    if (g >= ngroups) return make_float4(fill, fill, fill, fill);
    if (vec) return __ldg(reinterpret_cast<const float4*>(src) + g);
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = 4 * g + e < n ? __ldg(src + 4 * g + e) : fill;
    return make_float4(v[0], v[1], v[2], v[3]);
  };
  auto load_batch = [&](const float* src, int gb, float4 (&v)[kNB]) {
    if (vec && gb + kStep <= ngroups) {
      const float4* s4 = reinterpret_cast<const float4*>(src) + gb + tid;
#pragma unroll
      for (int i = 0; i < kNB; ++i) v[i] = __ldg(s4 + i * T);
    } else {
#pragma unroll
      for (int i = 0; i < kNB; ++i) v[i] = load4(src, gb + i * T + tid, -INFINITY);
    }
  };
  auto batch_max = [&](const float4 (&v)[kNB]) -> float {
    float m4[kNB];
#pragma unroll
    for (int i = 0; i < kNB; ++i) m4[i] = fmaxf(max3f(v[i].x, v[i].y, v[i].z), v[i].w);
#pragma unroll
    for (int w = 1; w < kNB; w *= 2)
#pragma unroll
      for (int i = 0; i + w < kNB; i += 2 * w) m4[i] = fmaxf(m4[i], m4[i + w]);
    return m4[0];
  };
  // Push this warp's partial into every CTA of the cluster, then wait for the cluster's partials.
  auto exchange = [&](float f0, float f1, int i0) -> const Part* {
    const int slot = xs & 1;
    const uint32_t parity = (uint32_t)((xs >> 1) & 1);
    ++xs;
    if (tid == 0) mbar_arrive_expect_tx(&sh.xbar[slot], (uint32_t)(nparts * (int)sizeof(Part)));
    if (lane < csize)
      st_async_v4(map_to_rank(smem_u32(&sh.xch[slot][rank * kWarps + warp]), (uint32_t)lane), f0, f1, i0, 0,
                  map_to_rank(smem_u32(&sh.xbar[slot]), (uint32_t)lane));
    if (!mbar_wait_cluster_bounded(&sh.xbar[slot], parity) && lane == 0) raise_error(p.dev_err, SPEC_DEVERR_TIMEOUT);
    return sh.xch[slot];
  };
  auto warp_best = [&](float& v, int& i) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) vi_combine(v, i, __shfl_xor_sync(kAll, v, o), __shfl_xor_sync(kAll, i, o));
  };
  auto row_best = [&](const Part* x, float& bv, int& bi) {
    bv = -INFINITY;
    bi = INT32_MAX;
    for (int t = lane; t < nparts; t += 32) vi_combine(bv, bi, x[t].f0, x[t].i0);
    warp_best(bv, bi);
  };
  auto warp_sum = [&](float v) -> float {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
  };

  for (int b = (int)(blockIdx.x / (unsigned)csize); b < p.batch; b += nclusters) {
    const float* lrow = p.logits + (int64_t)b * N * V + x0;  // node i's slice at lrow + i V
    const float* qrow = p.probs ? p.probs + (int64_t)b * N * V + x0 : nullptr;
    const int md = p.mode[b];
    const float t_row = p.temperature[b];
    float4 v[kNB];
    load_batch(lrow, 0, v);  // node 0's first batch, in flight during the checks
    __syncwarp();            // the row before is done with
    int par[2], tok[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = lane + 32 * i;
      nd.par[c] = par[i] = c < N ? p.parents[(int64_t)b * N + c] : SPEC_TREE_UNUSED;
      nd.tok[c] = tok[i] = c < N ? p.tokens[(int64_t)b * N + c] : 0;
      nd.path[c] = c == 0 ? 0 : -1;
    }
    // nodes with a property (of nodes lane and lane + 32), as a 64-bit mask
    auto nodes_with = [&](bool a, bool c) -> uint64_t {
      return (uint64_t)__ballot_sync(kAll, a) | ((uint64_t)__ballot_sync(kAll, c) << 32);
    };
    const int par0 = __shfl_sync(kAll, par[0], 0);
    int err = 0;
    if (par0 != SPEC_TREE_UNUSED) {
      if (md != SPEC_MODE_GREEDY && md != SPEC_MODE_SAMPLE) err |= SPEC_DEVERR_MODE;
      if (md == SPEC_MODE_SAMPLE && (!(t_row > 0.f) || !isfinite(t_row))) err |= SPEC_DEVERR_TEMPERATURE;
      const uint64_t used = nodes_with(par[0] != SPEC_TREE_UNUSED, par[1] != SPEC_TREE_UNUSED);
      bool bad_tree = false, bad_token = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = lane + 32 * i, q = par[i];
        if (q != SPEC_TREE_UNUSED && q != SPEC_TREE_ROOT) bad_tree |= q < 0 || q >= c || !((used >> (q & 63)) & 1);
        bad_token |= c > 0 && q != SPEC_TREE_UNUSED && (tok[i] < 0 || tok[i] >= V);
      }
      if (__any_sync(kAll, bad_tree)) err |= SPEC_DEVERR_TREE;
      if (__any_sync(kAll, bad_token)) err |= SPEC_DEVERR_TOKEN;
    }
    if (par0 == SPEC_TREE_UNUSED || err) {  // uniform across the cluster: no exchange for this row
      if (rank == 0 && warp == 0) {
        if (lane == 0) {
          if (err) raise_error(p.dev_err, err);
          p.accept_len[b] = -1;
        }
        for (int j = lane; j < N; j += 32) p.out_tokens[(int64_t)b * N + j] = p.path[(int64_t)b * N + j] = -1;
      }
      continue;
    }
    const bool greedy = md == SPEC_MODE_GREEDY;
    // logit -> log2 units of p. Exponents are c2 times a difference of logits, so that the largest has a weight of exactly 1
    // and every part of the row uses the same weights: l c2 - round(max c2) in one fma has an error of up to half a step of
    // max c2, 2^2 at a temperature of 1e-6, and another in every part. The subtraction costs 2 to 3% (32 sampled rows in a
    // graph 33.9 us for 32.9). c2 is kept finite, for temperatures near fp32's smallest.
    const float c2 = fminf((1.0f / (greedy ? 1.f : t_row)) * 1.4426950408889634f, 3.402823466e38f);
    if (!greedy) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        nd.u[lane + 32 * i] = word_to_uniform(
            philox4x32_10(0u, (uint32_t)(lane + 32 * i - 1), (uint32_t)b, 0u, p.seed_lo, p.seed_hi).v[0]);
    }
    __syncwarp();
    if (!joined) {
      cluster_wait();  // every CTA of the cluster is running
      joined = true;
    }

    int cur = 0, m = 0, last = 0;
    bool loaded = true;                      // v holds the node's first batch already
    for (;;) {
      const float* src = lrow + (int64_t)cur * V;
      const float* qsrc = qrow ? qrow + (int64_t)cur * V : nullptr;
      if (!loaded) load_batch(src, 0, v);
      loaded = false;
      const uint64_t children = nodes_with(nd.par[lane] == cur, nd.par[lane + 32] == cur);
      // Rows that the node's decision may ask for, on their way to L2 while it is made: its draft probabilities (needed as
      // soon as a child is refused) and the first child's logits.
      if (p.prefetch && children && tid == 0) {
        if (qsrc && !greedy) bulk_prefetch_l2(qsrc, (uint32_t)n * 4);
        bulk_prefetch_l2(lrow + (int64_t)(__ffsll((long long)children) - 1) * V, (uint32_t)n * 4);
      }
      int next = -1;
      if (greedy) {
        // ---- argmax of the slice (lowest index on ties), then of the row: see accept.cu
        float bv = -INFINITY;
        int idx = tid < ngroups ? x0 + 4 * tid : INT32_MAX;
        for (int gb = 0;;) {
          const float bm = batch_max(v);
          if (bm > bv) {
            bv = bm;
#pragma unroll
            for (int i = kNB - 1; i >= 0; --i) {
              const float lv[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
              for (int e = 3; e >= 0; --e)
                if (lv[e] == bm) idx = x0 + 4 * (gb + i * T + tid) + e;
            }
          }
          gb += kStep;
          if (gb >= ngroups) break;
          load_batch(src, gb, v);
        }
        warp_best(bv, idx);
        const Part* x = exchange(bv, 0.f, idx);
        float rv;
        row_best(x, rv, last);
        const uint64_t hit = children & nodes_with(nd.tok[lane] == last, nd.tok[lane + 32] == last);
        if (hit) next = __ffsll((long long)hit) - 1;
      } else {
        // the children's target logits and draft probabilities: first used after the statistics
        float ld[2] = {0.f, 0.f}, qd[2] = {1.f, 1.f};
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if ((children >> (lane + 32 * i)) & 1) {
            ld[i] = __ldg(src - x0 + nd.tok[lane + 32 * i]);
            if (qsrc) qd[i] = __ldg(qsrc - x0 + nd.tok[lane + 32 * i]);
          }
        // ---- max and sum of exp2((l - max) c2) in one pass
        float mx = -INFINITY, s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
        for (int gb = 0;;) {
          const float bm = batch_max(v);
          if (bm > mx) {
            if (mx != -INFINITY) {
              const float rs = fast_exp2((mx - bm) * c2);
              s0 *= rs;
              s1 *= rs;
              s2 *= rs;
              s3 *= rs;
            }
            mx = bm;
          }
          if (mx != -INFINITY) {
#pragma unroll
            for (int i = 0; i < kNB; ++i) {
              s0 += fast_exp2((v[i].x - mx) * c2);
              s1 += fast_exp2((v[i].y - mx) * c2);
              s2 += fast_exp2((v[i].z - mx) * c2);
              s3 += fast_exp2((v[i].w - mx) * c2);
            }
          } else {  // -inf all, or a NaN that the maximum passes over: as +inf, so that it reaches the row's sum
            bool nan = false;
#pragma unroll
            for (int i = 0; i < kNB; ++i)
              nan |= v[i].x != v[i].x || v[i].y != v[i].y || v[i].z != v[i].z || v[i].w != v[i].w;
            if (nan) {
              mx = INFINITY;
              s0 = __int_as_float(0x7fc00000);
            }
          }
          gb += kStep;
          if (gb >= ngroups) break;
          load_batch(src, gb, v);
        }
        float s = (s0 + s1) + (s2 + s3);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const float om = __shfl_xor_sync(kAll, mx, o), os = __shfl_xor_sync(kAll, s, o);
          ms_combine(mx, s, om, os, c2);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          nd.ld[lane + 32 * i] = ld[i];
          nd.qd[lane + 32 * i] = qd[i];
        }
        const Part* x = exchange(mx, s, 0);
        float M = -INFINITY, Z = 0.f;
        for (int i = lane; i < nparts; i += 32) ms_combine(M, Z, x[i].f0, x[i].f1, c2);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const float om = __shfl_xor_sync(kAll, M, o), os = __shfl_xor_sync(kAll, Z, o);
          ms_combine(M, Z, om, os, c2);
        }
        // A row without a distribution: no logit above -inf, or a NaN or +inf among them (the sum is then NaN). Uniform over
        // the cluster: every warp holds the same values.
        if (!(M > -INFINITY && Z < INFINITY)) {
          last = -1;
          break;
        }
        const float invZ = 1.f / Z;

        __syncwarp();
        int n_gone = 0;  // refused tokens (no draft probabilities)
        // One pass over the slice with the residual's weights: their sum over the row, or (race) the winner of the
        // exponential race, -1 if every weight is 0. Keys and bounds as in accept.cu.
        // Weight of an entry with pe = 2^((l - M) c2): max(0, A pe - bq q), or without q (bq 0) pe itself, 0 for a
        // refused token.
        auto pass = [&](auto race, auto with_q, float A, float bq, float& total) -> int {
          constexpr bool kRace = decltype(race)::value, kResid = decltype(with_q)::value;
          constexpr int NBat = kRace ? kRB : kSB, kRStep = NBat * T;
          bool strikes = false;  // a refused token is among this thread's entries
          for (int k = 0; k < (kResid ? 0 : n_gone); ++k) {
            const int t = nd.gone[k] - x0;
            strikes |= t >= 0 && t < n && (t >> 2) % T == tid;
          }
          float thr = 0.f, best = -1.f, sum = 0.f;
          int bx = INT32_MAX;
          auto iteration = [&](auto checked, int gb) {
            float4 l4[NBat], q4[NBat];
#pragma unroll
            for (int i = 0; i < NBat; ++i) {
              const int g = gb + i * T + tid;
              const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
              if constexpr (decltype(checked)::value) {
                l4[i] = load4(src, g, -INFINITY);
                q4[i] = kResid ? load4(qsrc, g, 0.f) : zero;
              } else {
                l4[i] = __ldg(reinterpret_cast<const float4*>(src) + g);
                q4[i] = kResid ? __ldg(reinterpret_cast<const float4*>(qsrc) + g) : zero;
              }
            }
            [[maybe_unused]] Philox4 r[NBat];
            if constexpr (kRace) {
#pragma unroll
              for (int i = 0; i < NBat; ++i)
                r[i] = philox4x32_10((uint32_t)(x0 / 4 + gb + i * T + tid), (uint32_t)cur, (uint32_t)b, 1u, p.seed_lo,
                                     p.seed_hi);
            }
            float w[NBat * 4];
#pragma unroll
            for (int i = 0; i < NBat; ++i) {
              const float lv[4] = {l4[i].x, l4[i].y, l4[i].z, l4[i].w};
              [[maybe_unused]] const float qv[4] = {q4[i].x, q4[i].y, q4[i].z, q4[i].w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float pe = fast_exp2((lv[e] - M) * c2);  // 0 past the slice (-inf logit)
                w[4 * i + e] = kResid ? fmaxf(fmaf(pe, A, -bq * qv[e]), 0.f) : pe;
              }
            }
            if (!kResid && strikes) {
              for (int k = 0; k < n_gone; ++k) {
                const int t = nd.gone[k] - x0 - 4 * (gb + tid);
#pragma unroll
                for (int i = 0; i < NBat; ++i)
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    if (t == 4 * i * T + e) w[4 * i + e] = 0.f;
              }
            }
            if constexpr (kRace) {
              float ub[NBat * 4], lb = thr, ubm = 0.f;
#pragma unroll
              for (int i = 0; i < NBat; ++i) {
                float lbe[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  // U = (2j + 1) 2^-24 for the word's top 23 bits j; U and 1 - U are exact
                  const float f1 = __uint_as_float(0x3F800000u + (r[i].v[e] >> 9));
                  const float uu = f1 - 0.999999940395355224609375f;
                  ub[4 * i + e] = w[4 * i + e] * fast_rcp(1.f - uu);
                  lbe[e] = ub[4 * i + e] * uu;
                }
                lb = max3f(lb, max3f(lbe[0], lbe[1], lbe[2]), lbe[3]);
                ubm = max3f(ubm, max3f(ub[4 * i], ub[4 * i + 1], ub[4 * i + 2]), ub[4 * i + 3]);
              }
#pragma unroll
              for (int o = 16; o > 0; o >>= 1) lb = fmaxf(lb, __shfl_xor_sync(kAll, lb, o));
              thr = lb;
              if (ubm > 0.f && ubm >= thr) {
#pragma unroll
                for (int i = 0; i < NBat; ++i) {
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    if (ub[4 * i + e] > 0.f && ub[4 * i + e] >= thr) {
                      const float key = w[4 * i + e] / -logf(word_to_uniform(r[i].v[e]));
                      if (key > best) {  // entries are visited in increasing x: ties keep the lower index
                        best = key;
                        bx = x0 + 4 * (gb + i * T + tid) + e;
                      }
                    }
                  }
                }
              }
            } else {
#pragma unroll
              for (int i = 0; i < NBat; ++i) sum += (w[4 * i] + w[4 * i + 1]) + (w[4 * i + 2] + w[4 * i + 3]);
            }
          };
          int gb = 0;
          if (vec)
            for (; gb + kRStep <= ngroups; gb += kRStep) iteration(std::false_type{}, gb);
          for (; gb < ngroups; gb += kRStep) iteration(std::true_type{}, gb);  // uniform: every lane shuffles
          if constexpr (kRace) {
            warp_best(best, bx);
            const Part* xp = exchange(best, 0.f, bx);
            float kv;
            int win;
            row_best(xp, kv, win);
            return kv > 0.f ? win : -1;
          } else {
            const Part* xp = exchange(warp_sum(sum), 0.f, 0);
            float t = 0.f;
            for (int i = lane; i < nparts; i += 32) t += xp[i].f0;
            total = warp_sum(t);
            return 0;
          }
        };

        // ---- the children in turn
        float a = 1.f, bq = 0.f;    // with draft probabilities: the residual is max(0, a p - bq q)
        float a0 = 1.f, bq0 = 0.f;  // ... before the last refusal
        float rem = 1.f;            // without: the mass of p that the refused tokens left
        for (uint64_t left = children; left;) {
          const int c = __ffsll((long long)left) - 1;
          left &= left - 1;
          const float pd = fast_exp2((nd.ld[c] - M) * c2) / Z, uc = nd.u[c], qc = nd.qd[c];
          const int t = nd.tok[c];
          bool again = false;  // a refused token once more
          for (int k = 0; k < n_gone; ++k) again |= nd.gone[k] == t;
          const float r = qsrc ? (bq == 0.f ? pd : fmaxf(0.f, fmaf(a, pd, -bq * qc))) : pd;
          if (!again && uc * (qsrc ? qc : rem) < r) {
            next = c;
            break;
          }
          if (again) continue;
          a0 = a;
          bq0 = bq;
          if (qsrc) {
            bq += 1.f;
            if (!left) break;  // the race needs no mass
          } else {
            if (lane == 0) nd.gone[n_gone] = t;
            __syncwarp();
            ++n_gone;
          }
          float mass = rem - pd;
          if (qsrc || mass < kExactMass) {
            if (qsrc) {
              pass(std::false_type{}, std::true_type{}, a * invZ, bq, mass);
            } else {
              pass(std::false_type{}, std::false_type{}, 0.f, 0.f, mass);
              mass *= invZ;
            }
          }
          if (mass > 0.f) {
            if (qsrc) {
              a /= mass;
              bq /= mass;
            } else {
              rem = mass;
            }
          } else {  // all zero: the residual stays as it was
            bq = bq0;
            if (!qsrc) --n_gone;
          }
        }
        // ---- the last token, from the residual; where that is all zero, from the one before
        if (next < 0) {
          float dummy;
          for (int attempt = 0; attempt < 3; ++attempt) {
            last = bq > 0.f ? pass(std::true_type{}, std::true_type{}, a * invZ, bq, dummy)
                            : pass(std::true_type{}, std::false_type{}, 0.f, 0.f, dummy);
            if (last >= 0 || bq == 0.f) break;
            a = a0;
            bq = bq0;
            bq0 = 0.f;
          }
        }
      }
      if (next < 0) break;
      ++m;
      if (lane == 0) nd.path[m] = next;
      cur = next;
    }
    // ---- the row's result: accepted tokens, the last token, -1 padding (one warp)
    if (rank == 0 && warp == 0) {
      __syncwarp();
      for (int j = lane; j < N; j += 32) {
        p.out_tokens[(int64_t)b * N + j] = j < m ? nd.tok[nd.path[j + 1]] : (j == m ? last : -1);
        p.path[(int64_t)b * N + j] = nd.path[j];
      }
      if (lane == 0) p.accept_len[b] = m;
    }
  }
  if (!joined) cluster_wait();
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
  if (num_nodes > tree::kMaxNodes || vocab > acc::kMaxVocab) return SPEC_ERR_UNSUPPORTED;
  // The results of a row with an error are written while other blocks of its cluster may still check it.
  const size_t rows = (size_t)batch * 4, nodes = rows * num_nodes;
  const struct {
    const void* at;
    size_t bytes;
  } results[3] = {{out_tokens, nodes}, {path, nodes}, {accept_len, rows}},
    inputs[4] = {{tokens, nodes}, {parents, nodes}, {mode, rows}, {temperature, rows}};
  for (int i = 0; i < 3; ++i) {
    for (const auto& x : inputs)
      if (tree::overlap(results[i].at, results[i].bytes, x.at, x.bytes)) return SPEC_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (tree::overlap(results[i].at, results[i].bytes, results[j].at, results[j].bytes)) return SPEC_ERR_INVALID_ARG;
  }
  const int dev = current_device();
  if (dev < 0) return SPEC_ERR_LAUNCH;
  acc::Config c;
  if (!acc::choose_config<tacc::tree_accept_kernel<256>, tacc::tree_accept_kernel<128>>(dev, batch, vocab, c))
    return SPEC_ERR_LAUNCH;
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
  p.batch = batch;
  p.nodes = num_nodes;
  p.vocab = vocab;
  p.slice = c.slice;
  p.csize = c.csize;
  p.vec = (vocab % 4 == 0) && ((reinterpret_cast<uintptr_t>(target_logits) | reinterpret_cast<uintptr_t>(draft_probs)) & 15) == 0;
  // Prefetches are free where a node's rows of the whole batch are small; on larger batches they compete with reads that
  // are sure to be needed.
  p.prefetch = p.vec && (int64_t)batch * vocab * 4 <= tacc::kPrefetchMaxBytes;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)c.csize;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int clusters = batch < c.clusters ? batch : c.clusters;
  cfg.gridDim = dim3((unsigned)(clusters * c.csize), 1, 1);
  cfg.blockDim = dim3((unsigned)c.threads, 1, 1);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream_);
  const cudaError_t e = c.threads == 256 ? cudaLaunchKernelEx(&cfg, tacc::tree_accept_kernel<256>, p)
                                         : cudaLaunchKernelEx(&cfg, tacc::tree_accept_kernel<128>, p);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_LAUNCH;
}
