// Launches of the tree attention's kernels for one head dim (host side).
#pragma once

#include "launch_memo.h"
#include "tree_attention.cuh"

namespace specv {
namespace tattn {

template <class C>
static int settings_of(int batch, Launch* l) {
  static LaunchMemo memo;
  const int dev = current_device();
  if (dev < 0) return SPEC_ERR_LAUNCH;
  auto kern = tree_attention_kernel<C>;
  std::lock_guard<std::mutex> lock(memo.mu);
  if (memo.grid[dev] == 0) {
    int sms = 0, optin = 0;
    cudaFuncAttributes attr;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
        cudaFuncGetAttributes(&attr, kern) != cudaSuccess)
      return SPEC_ERR_LAUNCH;
    // the register exchange inside the kernel must not ask for more than the launch brings
    if (C::STREAMS == 2 && attr.numRegs < kLaunchRegs) return SPEC_ERR_LAUNCH;
    if (!grant_smem_locked(memo, (const void*)kern, dev, (size_t)optin)) return SPEC_ERR_LAUNCH;
    memo.grid[dev] = sms > kMaxGrid ? kMaxGrid : sms;
  }
  const size_t fixed = smem_fixed<C>(batch), room = memo.granted[dev];
  const size_t fit = fixed < room ? (room - fixed) / C::SLOT : 0;
  const int slots = fit > kMaxSlots ? kMaxSlots : (int)fit;
  l->vslots = slots / 2;
  l->kslots = slots - l->vslots;
  if (l->vslots < C::kMinV) return SPEC_ERR_UNSUPPORTED;
  l->smem = fixed + (size_t)slots * C::SLOT;
  l->grid = memo.grid[dev];
  return SPEC_OK;
}

template <class C>
static int launch_of(const Launch& l, const Call& c) {
  tree_attention_kernel<C><<<l.grid, C::kThreads, l.smem, c.stream>>>(c.p, c.tq, c.tk, c.tv);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_LAUNCH;
}

// The instance for a call: fn.template operator()<Cfg>().
template <int D, int MT, class F>
static int with_terms(int terms, bool fp16, F fn) {
  if (fp16) return terms == 1 ? fn(Cfg<D, MT, 1, true>{}) : fn(Cfg<D, MT, 2, true>{});
  if constexpr (MT <= Cfg<D, 1, 3, false>::STREAMS) {
    if (terms == 3) return fn(Cfg<D, MT, 3, false>{});
  }
  return fn(Cfg<D, MT, 1, false>{});
}
template <int D, class F>
static int with_instance(int mt, int terms, bool fp16, F fn) {
  if constexpr (D <= 128) {
    if (mt == 2) return with_terms<D, 2>(terms, fp16, fn);
  }
  return with_terms<D, 1>(terms, fp16, fn);
}

template <int D>
int settings(int mt, int terms, bool fp16, int batch, Launch* l) {
  return with_instance<D>(mt, terms, fp16, [&](auto c) { return settings_of<decltype(c)>(batch, l); });
}
template <int D>
int launch(int mt, int terms, bool fp16, const Launch& l, const Call& c) {
  return with_instance<D>(mt, terms, fp16, [&](auto k) { return launch_of<decltype(k)>(l, c); });
}

}  // namespace tattn
}  // namespace specv
