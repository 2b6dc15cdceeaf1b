// Launches of the kernels of the attention over a 4-bit cache: one translation
// unit for each head dim.
#pragma once

#include "launch_memo.h"
#include "q4_attention.cuh"
#include "window_join.cuh"

namespace specv {
namespace qattn {

// Bytes of shared memory that a block may use: two share an SM's 228 KB, of which the system takes 1 KB a block.
template <class C>
static constexpr size_t budget() {
  return C::kBlocks == 2 ? 115712 : 232448;
}

// How a call is cut into units, and a unit into the work of warps. False: a tile's token rows do not fit.
template <class C>
static bool cut_up(const spec_attn_desc* d, int rows, Params* p) {
  const int all = rows * (d->num_q_heads / d->num_kv_heads), heads = d->num_kv_heads;
  const int parts = (all + C::ROWS - 1) / C::ROWS;
  p->sub = (all + parts - 1) / parts;
  p->unit_heads = heads < C::kWarps ? heads : C::kWarps;
  p->head_units = (heads + p->unit_heads - 1) / p->unit_heads;
  p->parts = C::kWarps / p->unit_heads < parts ? C::kWarps / p->unit_heads : parts;
  p->groups = (parts + p->parts - 1) / p->parts;
  p->parts = (parts + p->groups - 1) / p->groups;
  p->per = p->parts * p->sub;
  p->by_sub = ((1 << 16) + p->sub - 1) / p->sub;
  p->by_parts = ((1 << 8) + p->parts - 1) / p->parts;
  p->pairs = p->unit_heads * p->parts;
  p->seg_par = p->unit_heads * (C::D / 2);
  // copies are of multiples of 16 bytes; a unit of some of the heads has 8 of them
  p->seg = p->head_units == 1 ? (int)q4::row_bytes(heads, C::D) : p->seg_par + p->unit_heads * 4;
  const size_t fixed = Smem<C>::bytes(p->pairs, d->batch);
  if (fixed >= budget<C>()) return false;
  const size_t room = budget<C>() - fixed;
  const size_t tile = 2 * (size_t)TK * p->seg;
  for (p->splits = C::kWarps / p->pairs; p->splits >= 1; --p->splits) {
    p->slots = (int)(room / tile < kMaxSlots ? room / tile : kMaxSlots) / p->splits * p->splits;
    // The ring holds a split's tile at work and the next ones, and in the end the other splits' results. Where a tile is
    // shared by all warps, a slot stays free between their copies and their work, so that a warp does not wait for the slowest
    // to leave it: 169 us for 178 (32 sequences of 16384 tokens, 8 kv heads of 128), 691 for 781 with 64 rows, 232 for 262
    // at head dim 256.
    if (p->slots < 2 * p->splits || (size_t)(p->splits - 1) * p->pairs * C::STATE * 128 > p->slots * tile) continue;
    p->ahead = p->slots / p->splits - (p->splits == 1 && p->slots > 2 ? 2 : 1);
    return true;
  }
  return false;
}

template <class C>
static int launch_of(const spec_attn_desc* d, Params p, cudaStream_t stream) {
  static LaunchMemo memo;
  const int dev = current_device();
  if (dev < 0) return SPEC_ERR_LAUNCH;
  if (!cut_up<C>(d, p.rows, &p)) return SPEC_ERR_UNSUPPORTED;
  p.opart = reinterpret_cast<float*>(p.stat + (size_t)kMaxPieces * p.pairs * p.sub);
  // A block takes about 2.4 us for 32 keys of 8 pairs (2.2 to 2.7 measured at head dims 128 and 256, 16 and 32 rows)
  const float tile_us = (C::D == 64 ? 0.2f : 0.3f) * p.pairs;
  p.cuts = wattn::may_cut(p, C::KEYS, tile_us, 6.f);
  p.task_cost = 8.f / tile_us;
  p.join_cost = 3.f / tile_us;
  p.piece_cost = 0.05f / tile_us;
  const size_t smem = p.slots * (2 * (size_t)TK * p.seg) + Smem<C>::bytes(p.pairs, p.batch);
  int grid;
  {
    std::lock_guard<std::mutex> lock(memo.mu);
    if (memo.grid[dev] == 0) {
      int sms = 0;
      if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return SPEC_ERR_LAUNCH;
      if (!grant_smem_locked(memo, (const void*)q4_attention_kernel<C>, dev, budget<C>())) return SPEC_ERR_LAUNCH;
      memo.grid[dev] = C::kBlocks * sms;
    }
    grid = memo.grid[dev];
  }
  q4_attention_kernel<C><<<grid, C::kThreads, smem, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return SPEC_ERR_LAUNCH;
  return p.cuts ? wattn::launch_join<C::D>(p, kMaxPieces, stream) : SPEC_OK;
}
template <class C>
static size_t workspace_of(const spec_attn_desc* d, int rows) {
  Params p;
  if (!cut_up<C>(d, rows, &p)) return 0;
  return SPEC_ATTN_COUNTER_BYTES + wattn::kCutBytes + (size_t)kMaxPieces * p.pairs * p.sub * (2 + C::D) * 4;
}

// fn(configuration) for `all` packed rows of a kv head: the accumulators of 32 rows of head dim 256 do not fit the registers.
template <int D, class F>
static auto with_rows(int all, F fn) {
  if constexpr (D < 256) {
    if (all > 16) return fn(Cfg<D, 2>{});
  }
  return fn(Cfg<D, 1>{});
}

template <int D>
int launch(const spec_attn_desc* d, int all, const Params& p, cudaStream_t stream);
template <int D>
size_t workspace(const spec_attn_desc* d, int rows, int all);

}  // namespace qattn
}  // namespace specv
