// Launch settings and launches of the windowed attention's kernels: one
// translation unit for each head dim.
#pragma once

#include "launch_memo.h"
#include "window_attention.cuh"
#include "window_join.cuh"

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
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess)
      return SPEC_ERR_LAUNCH;
    if (!grant_smem_locked(memo, (const void*)window_attention_kernel<C>, dev, (size_t)optin)) return SPEC_ERR_LAUNCH;
    memo.grid[dev] = sms;
  }
  const size_t fixed = smem_fixed<C>(batch), room = memo.granted[dev];
  const size_t fit = fixed < room ? (room - fixed) / C::SLOT : 0;
  if (fit < (size_t)2 * C::PARTS) return SPEC_ERR_UNSUPPORTED;
  l->slots = fit > (size_t)kMaxSlots ? kMaxSlots : (int)fit;
  l->smem = fixed + (size_t)l->slots * C::SLOT;
  l->grid = memo.grid[dev];
  return SPEC_OK;
}
template <class C>
static int launch_of(const Launch& l, Call c) {
  c.p.cuts = may_cut(c.p, C::KEYS, C::TILE_US, 9.f);
  c.p.task_cost = C::TASK_COST;
  c.p.join_cost = C::JOIN_COST;
  c.p.piece_cost = C::PIECE_COST;
  window_attention_kernel<C><<<l.grid, C::kThreads, l.smem, c.stream>>>(c.p, c.tk, c.tv);
  if (cudaGetLastError() != cudaSuccess) return SPEC_ERR_LAUNCH;
  return c.p.cuts ? launch_join<C::D>(c.p, kMaxPieces, c.stream) : SPEC_OK;
}

// fn(configuration) for a unit of at most `packed` rows.
template <int D, bool FP16, class F>
static int with_rows(int packed, F fn) {
  switch (packed) {
    case 8: return fn(Cfg<D, 8, FP16>{});
    case 16: return fn(Cfg<D, 16, FP16>{});
    case 32: return fn(Cfg<D, 32, FP16>{});
    default: return fn(Cfg<D, 64, FP16>{});
  }
}

template <int D>
int settings_16(int packed, bool fp16, int batch, Launch* l);
template <int D>
int launch_16(int packed, bool fp16, const Launch& l, const Call& c);

}  // namespace wattn
}  // namespace specv
