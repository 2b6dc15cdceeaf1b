// Pieces shared by the acceptance kernels (chain and tree): the exchange of
// partials inside a thread-block cluster, small reductions, and the choice of
// the launch configuration. See accept.cu for the design.
#pragma once

#include <stdio.h>
#include <stdlib.h>

#include <mutex>

#include "common.cuh"
#include "launch_memo.h"

namespace specv {
namespace acc {

constexpr int kMaxCluster = 16;
constexpr int kMaxWarps = 8;
constexpr int kMaxVocab = 1 << 30;

// A partial pushed by one warp for one exchange.
struct __align__(16) Part {
  float f0;    // max logit, best race key, or the argmax value
  float f1;    // sum of exponentials relative to f0
  int32_t i0;  // argmax / race index
  int32_t pad;
};

struct Shared {
  // Exchange, push model: warp w of CTA r writes its partial into slot
  // [r * warps + w] of every CTA of the cluster with an asynchronous store that
  // counts its 16 bytes on that CTA's mbarrier xbar[e & 1], so everything read
  // after the wait is local. Two slots alternate: a CTA pushes exchange e only
  // after its own exchange e - 1 completed, which needs every peer's push of
  // e - 1, which each peer makes after it has read exchange e - 2 from the same
  // slot (its next push depends on what it read).
  Part xch[2][kMaxCluster * kMaxWarps];
  uint64_t xbar[2];  // phase k of xbar[s] completes with exchange 2k + s
};

// Split cluster barrier used once at start-up: every CTA arrives as soon as it
// runs and waits just before its first push into a peer's shared memory, so no
// CTA writes into a peer that has not started (the rule for distributed shared
// memory); by then the barrier has long completed.
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory"); }

// Combine two (max, sum of exp2((x - max) c2)) pairs; commutative, so a
// butterfly leaves the same bits in every lane.
__device__ __forceinline__ void ms_combine(float& m, float& s, float om, float os, float c2) {
  const float nm = fmaxf(m, om);
  const float a = m == -INFINITY ? 0.f : s * fast_exp2((m - nm) * c2);
  const float b = om == -INFINITY ? 0.f : os * fast_exp2((om - nm) * c2);
  m = nm;
  s = a + b;
}

// (value, index) with the larger value, the lower index on ties.
__device__ __forceinline__ void vi_combine(float& v, int& i, float ov, int oi) {
  if (ov > v || (ov == v && oi < i)) {
    v = ov;
    i = oi;
  }
}

// Largest of three (the three-input PTX form, sm_100 and later).
__device__ __forceinline__ float max3f(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Approximate reciprocal (rcp.approx: no refinement steps).
__device__ __forceinline__ float fast_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}

// 16-byte asynchronous store into a peer CTA's shared memory that also counts its
// bytes on the peer's mbarrier (complete_tx); both are shared::cluster addresses.
__device__ __forceinline__ void st_async_v4(uint32_t addr, float a, float b, int32_t c, int32_t d, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];\n"
               ::"r"(addr), "r"(__float_as_uint(a)), "r"(__float_as_uint(b)), "r"(c), "r"(d), "r"(bar)
               : "memory");
}
// Wait (bounded) for the phase of this CTA's mbarrier with the given parity, with
// cluster-scope acquire: the data peers stored into this CTA is visible after it.
__device__ __forceinline__ bool mbar_wait_cluster_bounded(uint64_t* bar, uint32_t parity,
                                                          long long limit_cycles = 2000000000LL) {
  auto try_wait = [&]() -> bool {
    uint32_t ok;
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
  };
  if (try_wait()) return true;
  const long long start = clock64();
  while (!try_wait()) {
    if (clock64() - start > limit_cycles) return false;
  }
  return true;
}

// ---------------------------------------------------------------------------
// Launch configuration
// ---------------------------------------------------------------------------

struct Config {
  int threads = 0, csize = 0, slice = 0, clusters = 0;
};

constexpr int kNumCsizes = 5;  // cluster sizes 1, 2, 4, 8, 16

// Clusters of `csize` CTAs of T threads the device can hold at once, from the
// occupancy query (0: none), worked out once per device under the caller's lock.
template <auto kern, int T>
static int resident_clusters(int dev, int li) {
  static int memo[kMaxDevices][kNumCsizes];  // 0: not asked yet; -1: none
  static bool attrs_set[kMaxDevices];
  if (!attrs_set[dev]) {
    // 16-CTA clusters are beyond the portable size
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
      (void)cudaGetLastError();
      return 0;
    }
    attrs_set[dev] = true;
  }
  if (memo[dev][li] == 0) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << li;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(1u << li, 1, 1);
    cfg.blockDim = dim3(T, 1, 1);
    int c = 0;
    if (cudaOccupancyMaxActiveClusters(&c, kern, &cfg) != cudaSuccess || c <= 0) {
      (void)cudaGetLastError();
      c = -1;
    }
    memo[dev][li] = c;
  }
  return memo[dev][li] > 0 ? memo[dev][li] : 0;
}

// Threads per CTA and cluster size. Among the configurations whose slices give
// every thread at least one float4 group (and the one-CTA clusters), prefer
// those that hold every row of the batch at once, and among them the fewest
// groups per thread and position (the shortest chain per row); at equal
// threads per row, 128-thread CTAs (finer placement over the SMs) unless they
// need 16-CTA clusters (the cluster barrier and exchange grow with the
// cluster), then the smallest cluster. Measured: serving128 49.6 us with 8 x
// 128 against 52.1 with 4 x 256; hybrid_gdn 57.0 with 8 x 256 against 57.7
// with 16 x 128. When none holds the batch, the one closest to 32 groups per
// thread (each cluster walks several rows). SPEC_ACCEPT_CONFIG="TxC" (T in
// {128, 256}, C a power of two <= 16) forces one.
template <auto kern256, auto kern128>
static bool choose_config(int dev, int batch, int vocab, Config& out) {
  static std::mutex mu;
  std::lock_guard<std::mutex> lock(mu);
  int force_t = 0, force_c = 0;
  if (const char* env = getenv("SPEC_ACCEPT_CONFIG")) {
    if (sscanf(env, "%dx%d", &force_t, &force_c) != 2) force_t = force_c = 0;
  }
  bool have = false;
  long best_score = 0;
  for (int ti = 0; ti < 2; ++ti) {
    const int T = ti == 0 ? 256 : 128;
    for (int li = kNumCsizes - 1; li >= 0; --li) {
      const int c = 1 << li;
      int slice = (vocab + c - 1) / c;
      slice = (slice + 3) & ~3;
      if ((vocab + slice - 1) / slice != c) continue;  // a CTA would own no logit
      if (c > 1 && slice < 4 * T) continue;
      if (force_t != 0 && (T != force_t || c != force_c)) continue;
      const int clusters = T == 256 ? resident_clusters<kern256, 256>(dev, li) : resident_clusters<kern128, 128>(dev, li);
      if (clusters == 0) continue;
      const long groups = ((slice / 4) + T - 1) / T;  // float4 groups per thread and position
      const bool fits = clusters >= batch;
      const long dist = groups > 32 ? groups - 32 : 32 - groups;
      const bool preferred = T == 128 ? c <= 8 : 2 * c > 8;  // see above
      const long score = fits ? groups * 1024 + (preferred ? 0 : 512) + li * 2 + (T == 256 ? 0 : 1)
                              : (1L << 40) + ((dist * 64 + li) * 2 + (T == 128 ? 0 : 1));
      if (!have || score < best_score) {
        have = true;
        best_score = score;
        out.threads = T;
        out.csize = c;
        out.slice = slice;
        out.clusters = clusters;
      }
    }
  }
  return have;
}


}  // namespace acc
}  // namespace specv
