// Launch settings and launches of the windowed attention's kernels: one
// translation unit for each head dim and kind of cache.
#pragma once

#include "launch_memo.h"
#include "window_attention.cuh"

namespace specv {
namespace wattn {

struct Launch {
  int grid, slots;
  size_t smem;
};
struct Call {
  Params p;
  CUtensorMap tk, tv;
  cudaStream_t stream;
};

template <class C>
static int settings_of(int batch, Launch* l) {
  static LaunchMemo memo;
  const int dev = current_device();
  if (dev < 0) return SPEC_ERR_LAUNCH;
  std::lock_guard<std::mutex> lock(memo.mu);
  if (memo.grid[dev] == 0) {
    int sms = 0, optin = 0;
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, window_attention_kernel<C>) != cudaSuccess) return SPEC_ERR_LAUNCH;
    // the registers that are dealt out inside the kernel are those that the launch brings
    if (C::DEAL && attr.numRegs < C::kLaunchRegs) return SPEC_ERR_LAUNCH;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess)
      return SPEC_ERR_LAUNCH;
    if (!grant_smem_locked(memo, (const void*)window_attention_kernel<C>, dev, (size_t)optin)) return SPEC_ERR_LAUNCH;
    memo.grid[dev] = sms;
  }
  const size_t fixed = smem_fixed<C>(batch), room = memo.granted[dev];
  const size_t fit = fixed < room ? (room - fixed) / C::SLOT : 0;
  const int least = C::Q4 ? C::RINGS : 2 * C::PARTS, most = C::Q4 ? least : kMaxSlots;
  if (fit < (size_t)least) return SPEC_ERR_UNSUPPORTED;
  l->slots = fit > (size_t)most ? most : (int)fit;
  l->smem = fixed + (size_t)l->slots * C::SLOT;
  l->grid = memo.grid[dev];
  return SPEC_OK;
}
template <class C>
static int launch_of(const Launch& l, const Call& c) {
  window_attention_kernel<C><<<l.grid, C::kThreads, l.smem, c.stream>>>(c.p, c.tk, c.tv);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_LAUNCH;
}

// fn(configuration) for a unit of at most `packed` rows.
template <int D, bool Q4, bool FP16, class F>
static int with_rows(int packed, F fn) {
  switch (packed) {
    case 8: return fn(Cfg<D, 8, Q4, FP16>{});
    case 16: return fn(Cfg<D, 16, Q4, FP16>{});
    case 32: return fn(Cfg<D, 32, Q4, FP16>{});
    default: return fn(Cfg<D, 64, Q4, FP16>{});
  }
}

template <int D>
int settings_16(int packed, bool fp16, int batch, Launch* l);
template <int D>
int launch_16(int packed, bool fp16, const Launch& l, const Call& c);
template <int D>
int settings_q4(int packed, int batch, Launch* l);
template <int D>
int launch_q4(int packed, const Launch& l, const Call& c);

}  // namespace wattn
}  // namespace specv
