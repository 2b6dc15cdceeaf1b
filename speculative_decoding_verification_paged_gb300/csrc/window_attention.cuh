// Kernel of the attention over a window of a 16-bit paged cache (see the comment
// at the top of window_attention.cu).
//
// Keys on the M side of the MMAs (tiles of 128), packed query rows on N, which may be as
// few as 16: S^T = K Q^T and O^T = V^T P^T, accumulators in tensor memory. One block an SM,
// a warp or more for each role: tensor copies of K and V (rings of their own, so that a
// barrier's phases are all waited for by one warp, in turn), the scores' MMAs, the
// products' MMAs, softmax (a thread for a key, 8 or 16 of the rows), queries in and results
// out. Nothing waits for a result that it does not need: a tile's scores are computed while
// the last one's weights are made.
//
// What bounds it: HBM for long units (24 rows of head dim 256 over whole contexts of 1024 to
// 16384 tokens: 90% of the copy rate); under a window the units' starts and ends, 20 to 25 us
// a call; with 64 packed rows the softmax and, in fp16, the second product (32 sequences with a
// window of 4096 tokens, 8 heads of 128: bf16 121 us, fp16 162, 82 us' worth of bytes); at head
// dim 64 the MMAs, half of whose lanes are dropped (the same with 16 rows: 65 us, 40 us' worth).
// Hot loops of all roles together have to fit the SM's instruction cache: unrolled by hand and
// in full, they were three times slower.
#pragma once

#include <cuda.h>

#include "attention_tc.cuh"
#include "window_plan.cuh"

namespace specv {
namespace wattn {

using attn::tc::reduce_cols;
using attn::tc::reduced_col;
using attn::tc::tmem_load_cols;
using attn::tc::tmem_store_cols;

constexpr int TK = 128;            // keys per tile (MMA M)
constexpr int kMaxSlots = 16;      // K and V tiles in shared memory
constexpr int kBarEpi = 1, kBarEnd = 2, kBarGroup0 = 3;  // named barriers: the epilogue's warps, all at the end, each softmax
                                                        // warpgroup

template <int D_, int ROWS_, bool FP16_>
struct Cfg {
  static constexpr int D = D_, ROWS = ROWS_;  // packed rows of a unit, at most
  static constexpr bool FP16 = FP16_;
  static constexpr int KEYS = TK, MAX_PIECES = kMaxPieces;
  static constexpr int N = ROWS < 16 ? 16 : ROWS;
  static constexpr int NG = ROWS <= 16 ? 1 : ROWS / 16;  // softmax warpgroups, CW rows each
  static constexpr int CW = ROWS / NG;
  static constexpr int HALVES = D == 256 ? 2 : 1;  // O^T accumulators of 128 lanes
  // Weights are two 16-bit numbers, the second one what the first has left, with an accumulator each: 22 bits in fp16 (down
  // to 2^-26, times 2^12 so that it is no subnormal; 2^-37 is the least step), 16 in bf16. With bf16 only where HBM hides the
  // second product: 32 sequences of head dim 128 with a window of 4096 tokens 103 us with one and two on 16 rows, 108 and 111
  // on 32, but 119 and 162 on 64, and 65 and 73 on 16 rows of head dim 64; 64 ragged ones of head dim 256, 24 rows, 114 and 115.
  static constexpr int BANDS = FP16 || (D >= 128 && ROWS <= 32) ? 2 : 1;
  static constexpr float LOW = FP16 ? 0x1p12f : 1.f;
  static constexpr int QB = D == 256 && N == 64 ? 1 : 2;           // query buffers
  static constexpr int NP = D == 256 && N == 64 && BANDS == 2 ? 1 : 2;  // P buffers
  static constexpr int O_COLS = BANDS * HALVES * N;
  static constexpr int SB = 2;                                     // scores of tiles
  static constexpr int OB = SB * N + 2 * O_COLS <= 512 ? 2 : 1;  // tasks whose accumulators there is room for
  static constexpr int COL_S = 0, COL_O = COL_S + SB * N;
  static constexpr int COLS = COL_O + OB * O_COLS;
  static constexpr int ALLOC = COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  static_assert(COLS <= 512, "tensor memory");
  // Tiles in shared memory; those of head dim 256 in two parts of 128 head dims.
  static constexpr int PARTS = D == 256 ? 2 : 1;
  static constexpr int SLOT = TK * D * 2 / PARTS;
  static constexpr int Q_BYTES = N * D * 2;  // D / 64 slices, rows of 64 elements
  static constexpr int P_BYTES = N * TK * 2;
  // P is the operand B of the second product, MN-major: the N rows of a key are contiguous and swizzled at that width.
  static constexpr uint32_t P_LAYOUT = N == 16 ? 6u : (N == 32 ? 4u : 2u);
  static constexpr int P_SWZ_SHIFT = N == 16 ? 2 : (N == 32 ? 1 : 0);
  static constexpr int P_SWZ_MASK = N == 16 ? 1 : (N == 32 ? 3 : 7);
  static constexpr int W_EPI = 4, W_SOFT = 8, kWarps = W_SOFT + 4 * NG;  // first warps of the roles
  static constexpr int kThreads = 32 * kWarps;
  // What a task's start and end, a join, and a piece of it cost, in tiles (us over the us of a tile at the measured copy
  // bandwidth, 45 KB a us for each SM, but 0.35 us at least).
  static constexpr float TILE_US = 2.f * PARTS * SLOT / 45000.f > 0.35f ? 2.f * PARTS * SLOT / 45000.f : 0.35f;
  static constexpr float TASK_COST = 1.f / TILE_US, JOIN_COST = 2.f / TILE_US, PIECE_COST = 0.15f / TILE_US;
  // Weights are 2^SHIFT at the largest of the tile that set a row's reference, TOP at most.
  static constexpr float SHIFT = 7.f, TOP = 32768.f;
};

// Shared memory besides the ring, in order.
template <class C>
struct Smem {
  static constexpr int Q = 0;
  static constexpr int P = Q + C::QB * C::Q_BYTES;
  static constexpr int BARS = P + C::NP * C::BANDS * C::P_BYTES;  // 96 mbarriers
  static constexpr int REF = BARS + 96 * 8;                       // [64] minus the reference of each row, a score before its scaling
  static constexpr int ALPHA = REF + 256;                         // [64]
  static constexpr int RED = ALPHA + 256;                         // [4][64]
  static constexpr int STAT = RED + 1024;                         // [OB]: [4][64] sums, [64] reference
  static constexpr int STAT_BYTES = 1024 + 256;
  static constexpr int EPI = STAT + C::OB * STAT_BYTES;  // [64] int64 and [64] floats of the epilogue
  static constexpr int MISC = EPI + 768;  // [64] plan, tensor-memory base, flags
  static constexpr int PREFIX = MISC + 256;
};
template <class C>
size_t smem_fixed(int batch) {
  return 1024 + Smem<C>::PREFIX + (((size_t)(batch + 1) * 6 + 63) & ~size_t(63));
}

// ---------------------------------------------------------------------------
// Instructions
// ---------------------------------------------------------------------------
// The MMAs are executed by a whole warp with the same operands; one elected lane issues them.
// D[tmem] (+)= A[smem] * B[smem]^T
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t id,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p, q;\n"
      ".reg .b64 a, b;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "setp.ne.b32 p, %6, 0;\n"
      "mov.b64 a, {%1, %2};\n"
      "mov.b64 b, {%3, %4};\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n"
      "}\n" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(id), "r"(accumulate)
      : "memory");
}
template <bool FP16>
__device__ __forceinline__ constexpr uint32_t mma_desc(int n, int a_mn, int b_mn) {
  return (1u << 4) | (FP16 ? 0u : (1u << 7) | (1u << 10)) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(TK >> 4) << 24);
}
// K or V rows of a head: box {64 elements, 1 head, rows} at {c0, head, row}; c0 a multiple of 8.
__device__ __forceinline__ void tma_rows(uint32_t dst, const void* map, int c0, int head, int row, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
      "[%1, {%2, %3, %4}], [%5], %6;\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(head), "r"(row), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ uint64_t l2_normal_policy() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;\n" : "=l"(pol));
  return pol;
}
// The barrier gets one arrival when all MMAs that this warp issued so far are complete.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "{\n"
      ".reg .pred q;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n"
      "}\n" ::"r"(bar)
      : "memory");
}
// ---------------------------------------------------------------------------
// Kernel
// ---------------------------------------------------------------------------
// A place in a ring of n slots, and how often its end has been passed.
struct Ring {
  int slot = 0, round = 0;
  __device__ __forceinline__ void advance(int by, int n) {
    slot += by;
    if (slot >= n) slot -= n, ++round;
  }
};

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1) window_attention_kernel(const __grid_constant__ Params p,
                                                                          const __grid_constant__ CUtensorMap tm_k,
                                                                          const __grid_constant__ CUtensorMap tm_v) {
  constexpr int D = C::D, N = C::N, CW = C::CW;
  using S = Smem<C>;
  // The products' MMA has 128 head dims. Of tiles with 64 it takes the other 64 lanes, which no one reads, from what lies
  // behind the tile: the next slot, or for the last one the area behind the ring.
  static_assert(D >= 128 || S::PREFIX >= C::SLOT, "the MMA stays inside the block's shared memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // KS slots for K, the others for V, so that a barrier's phases are all waited for by one warp, in turn (the
  // parity of a phase says nothing to a warp that has not seen the phase before)
  const int NS = p.slots, KS = NS - NS / 2;
  uint8_t* ring = smem;
  uint8_t* fixed = ring + (size_t)NS * C::SLOT;
  const uint32_t ring_u32 = smem_u32(ring), fixed_u32 = smem_u32(fixed);
  const uint32_t q_u32 = fixed_u32 + S::Q, p_u32 = fixed_u32 + S::P;
  int32_t* misc = reinterpret_cast<int32_t*>(fixed + S::MISC);
  int32_t* prefix = reinterpret_cast<int32_t*>(fixed + S::PREFIX);
  uint16_t* cut = reinterpret_cast<uint16_t*>(prefix + p.batch + 1);
  // mbarriers, 8 bytes each
  const uint32_t full = fixed_u32 + S::BARS;        // [kMaxSlots] a tile has landed
  const uint32_t empty = full + 8 * kMaxSlots;      // [kMaxSlots] its slot may be filled again
  const uint32_t q_full = empty + 8 * kMaxSlots;    // [QB] queries and their factors written
  const uint32_t s_full = q_full + 16;    // [SB] scores of a tile
  const uint32_t s_free = s_full + 16;     // [SB] and their buffer may be written again
  const uint32_t p_full = s_free + 16;     // [2] weights of a tile written
  const uint32_t pv_done = p_full + 16;    // [NP] second product of the tile that used the P buffer is complete
  const uint32_t o_full = pv_done + 16;    // [OB] a task's accumulators are complete
  const uint32_t o_free = o_full + 16;     // [OB] and have been read, with the statistics
  const uint32_t st_full = o_free + 16;    // [OB] a task's statistics are written
  static_assert(2 * kMaxSlots + 16 <= 96, "barriers fit their area");

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int grid = (int)gridDim.x, me = (int)blockIdx.x;

  make_plan<C>(p, prefix, cut, misc);
  clear_empty<C>(p, prefix);
  list_cut<C>(p, prefix, cut, misc);
  const int tasks = prefix[p.batch];
  if (me >= tasks) return;
  __syncthreads();  // the plan's area is used again below

  volatile int32_t* s_bad = misc;  // [32] a task (number & 31) met a bad page; the producer is less than 32 tasks ahead
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(misc) + 32;
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), C::ALLOC);
    tmem_relinquish();
  }
  if (tid == 0) {
#pragma unroll 1
    for (int s = 0; s < NS; ++s) {
      bar_init(full + 8 * s, 1);
      bar_init(empty + 8 * s, 1);
    }
#pragma unroll 1
    for (int j = 0; j < 16; j += 8) {
      bar_init(q_full + j, 4);
      bar_init(s_full + j, 1);
      bar_init(s_free + j, 4 * C::NG);
      bar_init(p_full + j, 4 * C::NG);
      bar_init(pv_done + j, 1);
      bar_init(o_full + j, 1);
      bar_init(o_free + j, 4);
      bar_init(st_full + j, 4 * C::NG);
    }
    fence_mbar_init();
  }
  if (tid < 32) s_bad[tid] = 0;
  // what no one writes and the tensor core reads: weights of rows behind the last one (their sums are not used)
#pragma unroll 1
  for (int i = tid; i < C::NP * C::BANDS * C::P_BYTES / 16; i += C::kThreads)
    reinterpret_cast<uint4*>(fixed + S::P)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  uint32_t tries = kMaxTries;
  auto wait = [&](uint32_t bar, int n) {  // until the bar's phase n is complete (n < 0: at once)
    if (n >= 0) bar_wait(bar, (uint32_t)(n & 1), tries);
  };
  auto leave = [&]() {  // the end of every warp but the one that gives tensor memory back
    if (tries == 1) raise_error(p.dev_err, SPEC_DEVERR_TIMEOUT);
    tc_fence_before();
    __syncwarp();
    asm volatile("bar.arrive %0, %1;\n" ::"n"(kBarEnd), "n"(C::kThreads) : "memory");
  };
  // Entry l of a task's page list, -1 behind the task's end; and whether it is a page, noted where it is not. A call of its
  // own, so that the entry can be on its way while other work is done.
  const int bs = 1 << p.page_shift, ppt_shift = 7 - p.page_shift;  // pages of a tile: 2^ppt_shift
  auto entry = [&](const Task& k, int l) {
    return l < min(k.span.pages, (k.tile0 + k.tiles) << ppt_shift)
               ? __ldg(p.block_table + (int64_t)k.b * p.max_blocks + (l < k.span.ns ? l : k.span.wp + l - k.span.ns))
               : -1;
  };
  auto checked = [&](int id, bool there, int seq) {
    const bool ok = id >= 0 && (int64_t)id < p.num_blocks;
    if (there && !ok) s_bad[seq & 31] = 1;
    return ok ? id : -1;
  };

  if (warp == 0) {
    // =================== K and V tiles by TMA ===================
    // K and V that no other unit reads again are the first to leave L2
    const uint64_t policy = p.groups == 1 ? l2_evict_first_policy() : l2_normal_policy();
    Ring at[2];  // K's and V's
    int seq = 0;
#pragma unroll 1
    for (int t = me; t < tasks; t += grid, ++seq) {
      const Task k = task_at<C>(p, prefix, cut, t);
      int win = -1, ids = 0;  // 32 entries of the page list, one a lane
#pragma unroll 1
      for (int j = 0; j < k.tiles; ++j) {
        const int l0 = (k.tile0 + j) << ppt_shift;
        if (win < 0 || l0 >= win + 32) {
          win = l0;
          ids = checked(entry(k, l0 + lane), l0 + lane < min(k.span.pages, (k.tile0 + k.tiles) << ppt_shift), seq);
          __syncwarp();
        }
#pragma unroll 1
        for (int w = 0; w < 2 * C::PARTS; ++w) {
          const bool v = w >= C::PARTS;
          const int s = v ? KS + at[1].slot : at[0].slot;
          wait(empty + 8 * s, (v ? at[1].round : at[0].round) - 1);
          if (tries == 1) break;
          if (v) at[1].advance(1, NS - KS);
          else at[0].advance(1, KS);
          if (lane == 0) bar_expect(full + 8 * s, (uint32_t)C::SLOT);
          __syncwarp();
          const CUtensorMap* map = v ? &tm_v : &tm_k;
          const int c0 = w % C::PARTS * 128;
#pragma unroll 1
          for (int pc = 0; pc < 1 << ppt_shift; ++pc) {
            const int id = __shfl_sync(0xffffffffu, ids, l0 - win + pc);
            const int row = id < 0 ? -bs : id << p.page_shift;  // outside of the cache: zeros
            if (lane == 0) {
#pragma unroll
              for (int sub = 0; sub < D / 64 / C::PARTS; ++sub)
                tma_rows(ring_u32 + s * C::SLOT + sub * TK * 128 + pc * bs * 128, map, c0 + sub * 64, k.g, row, full + 8 * s,
                         policy);
            }
          }
          __syncwarp();
        }
      }
    }
    if (tries == 1) {  // copies in flight still write here
      uint32_t few = 1000;
      for (int s = 0; s < NS; ++s) {
        const Ring& x = at[s < KS ? 0 : 1];
        const int copied = x.round + ((s < KS ? s : s - KS) < x.slot ? 1 : 0);
        if (copied > 0) bar_wait(full + 8 * s, (uint32_t)((copied - 1) & 1), few);
      }
    }
    leave();
    return;
  }
  if (warp == 1 || warp == 2) {
    // =================== MMA: one warp issues the scores, one the products ===================
    const uint32_t id_qk = mma_desc<C::FP16>(N, 0, 0), id_pv = mma_desc<C::FP16>(N, 1, 1);
    const uint64_t kmaj = smem_desc_sw128(0, 16, 1024);          // K, Q: K-major
    const uint64_t vmn = smem_desc_sw128(0, TK * 128, 1024);     // V: MN-major
    const uint64_t pmn = smem_desc(0, 16, 16 * N, C::P_LAYOUT);  // P: MN-major, groups of 8 keys
    const uint32_t kq_hi = (uint32_t)(kmaj >> 32), v_hi = (uint32_t)(vmn >> 32), w_hi = (uint32_t)(pmn >> 32);
    // Values that the compiler knows to be the same in all lanes are operands of the MMAs as they are; others would be
    // moved to uniform registers for each.
    auto uniform = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
    const uint32_t tm = uniform(tmem);
    const int n_slots = (int)uniform((uint32_t)(warp == 2 ? NS - KS : KS)), all = (int)uniform((uint32_t)tasks);
    const uint32_t q_lo = uniform((uint32_t)kmaj + (q_u32 >> 4)), k_lo = uniform((uint32_t)kmaj + (ring_u32 >> 4));
    const uint32_t v_lo = uniform((uint32_t)vmn + (ring_u32 >> 4)), p_lo = uniform((uint32_t)pmn + (p_u32 >> 4));
    const uint32_t bars = uniform(full);
    auto bar = [&](uint32_t b) { return bars + (b - full); };
    auto tiles_at = [&](int t) { return (int)uniform((uint32_t)task_at<C>(p, prefix, cut, t).tiles); };
    Ring at;  // the slot of the next K (V)
    const int first_slot = warp == 2 ? (int)uniform((uint32_t)KS) : 0;
    int i = 0, seq = 0;
#pragma unroll 1
    for (int t = me; t < all; t += grid, ++seq) {
      const int tiles = tiles_at(t);
#pragma unroll 1
      for (int j = 0; j < tiles && tries != 1; ++j, ++i) {
        if (warp == 1) {
          wait(bar(s_free) + 8 * (i % C::SB), i / C::SB - 1);
          wait(bar(q_full) + 8 * (seq % C::QB), seq / C::QB);
          const uint32_t qb = q_lo + (seq % C::QB) * (C::Q_BYTES >> 4), dst = tm + C::COL_S + (i % C::SB) * N;
#pragma unroll 1
          for (int part = 0; part < C::PARTS; ++part) {
            wait(bar(full) + 8 * (first_slot + at.slot), at.round);
            tc_fence_after();
            const uint32_t kb = k_lo + (first_slot + at.slot) * (C::SLOT >> 4), qp = qb + part * (N * 256 >> 4);
#pragma unroll
            for (int ks = 0; ks < D / 16 / C::PARTS; ++ks)
              mma_ss(dst, kb + (((ks >> 2) * TK * 128 + (ks & 3) * 32) >> 4), kq_hi,
                     qp + (((ks >> 2) * N * 128 + (ks & 3) * 32) >> 4), kq_hi, id_qk, part + ks > 0 ? 1u : 0u);
            mma_commit(bar(empty) + 8 * (first_slot + at.slot));
            at.advance(1, n_slots);
          }
          mma_commit(bar(s_full) + 8 * (i % C::SB));
        } else {
          const uint32_t o = tm + C::COL_O + (seq % C::OB) * C::O_COLS, more = j > 0 ? 1u : 0u;
          if (j == 0) wait(bar(o_free) + 8 * (seq % C::OB), seq / C::OB - 1);
          wait(bar(p_full) + 8 * (i & 1), i >> 1);
          const uint32_t pb = p_lo + (i % C::NP) * (C::BANDS * C::P_BYTES >> 4);
#pragma unroll 1
          for (int hh = 0; hh < C::HALVES; ++hh) {
            wait(bar(full) + 8 * (first_slot + at.slot), at.round);
            tc_fence_after();
            const uint32_t vb = v_lo + (first_slot + at.slot) * (C::SLOT >> 4);
#pragma unroll 1
            for (int band = 0; band < C::BANDS; ++band)
#pragma unroll
              for (int kk = 0; kk < TK / 16; ++kk)
                mma_ss(o + (band * C::HALVES + hh) * N, vb + (kk * 2048 >> 4), v_hi, pb + ((band * C::P_BYTES + kk * 32 * N) >> 4),
                       w_hi, id_pv, kk > 0 ? 1u : more);
            mma_commit(bar(empty) + 8 * (first_slot + at.slot));
            at.advance(1, n_slots);
          }
          mma_commit(bar(pv_done) + 8 * (i % C::NP));
          if (j == tiles - 1) mma_commit(bar(o_full) + 8 * (seq % C::OB));
        }
      }
    }
    if (warp == 2) {
      leave();
      return;
    }
    if (tries == 1) raise_error(p.dev_err, SPEC_DEVERR_TIMEOUT);
    __syncwarp();
    named_sync(kBarEnd, C::kThreads);  // no one uses tensor memory any more
    tc_fence_after();
    tmem_dealloc(tmem, C::ALLOC);
    return;
  }
  if (warp < C::W_EPI) {
    leave();
    return;
  }
  if (warp < C::W_SOFT) {
    // =================== epilogue: queries in, results out ===================
    const int et = tid - 32 * C::W_EPI, q4 = warp & 3;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    // Query rows of task number seq into its buffer. The buffer's last readers are done: the task QB before has been
    // written out.
    auto load_queries = [&](int t, int seq) {
      const Task k = task_at<C>(p, prefix, cut, t);
      uint8_t* dst = fixed + S::Q + (seq % C::QB) * C::Q_BYTES;
      constexpr int L = D / 8;  // threads of a row, 8 elements each
      const int c = et % L;
#pragma unroll 1
      for (int r = et / L; r < N; r += 128 / L) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (r < k.nr) x = __ldg(reinterpret_cast<const uint4*>(p.q) + out_row(p, k.b, k.g, k.r0 + r) * L + c);
        *reinterpret_cast<uint4*>(dst + (c >> 3) * N * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = x;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) bar_arrive(q_full + 8 * (seq % C::QB));
    };
    const int d0 = q4 * 32 + lane;  // head dim of this thread's lane; its neighbour's lane holds the other of a pair
    const bool odd = lane & 1;
    int64_t* e_row = reinterpret_cast<int64_t*>(fixed + S::EPI);    // [64] a row's place in the output
    float* e_fac = reinterpret_cast<float*>(fixed + S::EPI + 512);  // [64] one over the row's sum
    int seq = -C::QB;  // the first queries are loaded before the first result
#pragma unroll 1
    for (int t = me - C::QB * grid; t < tasks; t += grid, ++seq) {
      if (seq >= 0) {
        const Task k = task_at<C>(p, prefix, cut, t);
        const int ob = seq % C::OB;
        wait(st_full + 8 * ob, seq / C::OB);
        wait(o_full + 8 * ob, seq / C::OB);
        tc_fence_after();
        const bool bad = s_bad[seq & 31] != 0;
        if (bad && et == 0) raise_error(p.dev_err, SPEC_DEVERR_BLOCK_ID);
        named_sync(kBarEpi, 128);  // the last task's entries have been read, and the flag
        if (et == 0) s_bad[seq & 31] = 0;
        if (et < k.nr) {
          const float* x = reinterpret_cast<const float*>(fixed + S::STAT + ob * S::STAT_BYTES) + et;
          const float sum = (x[0] + x[64]) + (x[128] + x[192]);
          e_fac[et] = bad || (sum == 0.f && k.pieces > 1) ? 0.f : 1.f / sum;
          e_row[et] = out_row(p, k.b, k.g, k.r0 + et) * D;
          if (k.pieces > 1) __stcg(p.stat + (int64_t)k.slot * p.sub + et, make_float2(x[256], bad ? -1.f : sum));
        }
        named_sync(kBarEpi, 128);
        const uint32_t o = tmem + C::COL_O + ob * C::O_COLS + lane_off;
        float* part = p.opart + (int64_t)k.slot * p.sub * D;
        uint16_t* out = reinterpret_cast<uint16_t*>(p.out);
#pragma unroll 1
        for (int c = 0; c < k.nr; c += 8) {
#pragma unroll 1
          for (int hh = 0; hh < C::HALVES; ++hh) {
            float v[8];
            tmem_load_cols<8>(o + hh * N + c, v);
            if constexpr (C::BANDS == 2) {
              float low[8];
              tmem_load_cols<8>(o + (C::HALVES + hh) * N + c, low);
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = fmaf(low[e], 1.f / C::LOW, v[e]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= e_fac[c + e];
            if (D == 64 && q4 >= 2) continue;
            const int d = hh * 128 + d0;
            if (k.pieces == 1) {
              // pairs of head dims: one thread writes those of the even row, its neighbour those of the odd row
#pragma unroll
              for (int e = 0; e < 8; e += 2) {
                const float got = __shfl_xor_sync(0xffffffffu, odd ? v[e] : v[e + 1], 1);
                const float lo = bad ? 0.f : odd ? got : v[e], hi = bad ? 0.f : odd ? v[e + 1] : got;
                const int r = c + e + (odd ? 1 : 0);
                if (r < k.nr)
                  *reinterpret_cast<uint32_t*>(out + e_row[r] + (d & ~1)) = p.fp16 ? q4::pack2<true>(lo, hi) : q4::pack2<false>(lo, hi);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (c + e < k.nr) __stcg(part + (c + e) * D + d, v[e]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(o_free + 8 * ob);
      }
      if (t + C::QB * grid < tasks) load_queries(t + C::QB * grid, seq + C::QB);
    }
    leave();
    return;
  }
  {
    // =================== softmax ===================
    const int h = (warp - C::W_SOFT) >> 2, c0 = h * CW, q4 = warp & 3, gt = tid - 32 * C::W_SOFT - h * 128;
    const int bar_group = kBarGroup0 + h;
    float* s_ref = reinterpret_cast<float*>(fixed + S::REF);
    float* s_alpha = reinterpret_cast<float*>(fixed + S::ALPHA);
    float* s_red = reinterpret_cast<float*>(fixed + S::RED);
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const int key = q4 * 32 + lane;  // the lane of the scores that this thread reads
    int base = 0, seq = 0;
#pragma unroll 1
    for (int t = me; t < tasks; t += grid, ++seq) {
      const Task k = task_at<C>(p, prefix, cut, t);
      const int ob = seq % C::OB, first = k.ctx - p.rows + k.r0 / p.gqa;  // position of the unit's first row
      uint64_t l[CW / 2];  // pairs of rows
#pragma unroll
      for (int e = 0; e < CW / 2; ++e) l[e] = 0;
#pragma unroll 1
      for (int j = 0; j < k.tiles; ++j) {
        const int i = base + j;
        // ---- which rows see this thread's key: [r_lo, r_hi); most tiles are seen whole by all
        const int l0 = (k.tile0 + j) << ppt_shift;
        const bool early = l0 < k.span.ns;
        const int from = (early ? l0 : k.span.wp + l0 - k.span.ns) << p.page_shift;
        const bool whole = l0 + (1 << ppt_shift) <= (early ? k.span.ns : k.span.pages) && from + TK - 1 <= first &&
                           (p.window == 0 || from + TK <= p.sinks || from > first + k.nr - 1 - p.window);
        int r_lo = 0, r_hi = N;  // rows of padding see what all rows see
        bool dead = false;
        if (!whole) {
          const int lp = l0 + (key >> p.page_shift);
          const int tok = ((lp < k.span.ns ? lp : k.span.wp + lp - k.span.ns) << p.page_shift) + (key & (bs - 1));
          r_lo = max(0, tok - first) * p.gqa;
          if (p.window != 0 && tok >= p.sinks)
            r_hi = min(r_hi, (int)min((int64_t)1 << 20, max((int64_t)0, (int64_t)tok - first + p.window)) * p.gqa);
          if (lp >= k.span.pages || tok >= k.ctx) r_hi = 0;
          dead = r_lo >= min(r_hi, k.nr);
        }
        auto sees = [&](int e) { return c0 + e >= r_lo && c0 + e < r_hi; };
        wait(s_full + 8 * (i % C::SB), i / C::SB);
        tc_fence_after();
        const uint32_t t_s = tmem + C::COL_S + (i % C::SB) * N + lane_off + c0;
        const uint64_t scale2 = pack_f2(p.scale_log2, p.scale_log2);
        uint64_t y[CW / 2];  // weights
#pragma unroll 1
        for (bool settled = false;; settled = true) {
          if (j > 0 || settled) {
            float x[CW], top = 0.f;
            tmem_load_cols<CW>(t_s, x);
#pragma unroll
            for (int e = 0; e < CW; e += 4) {
              const float4 ref = *reinterpret_cast<const float4*>(s_ref + c0 + e);  // minus the reference
              // subtracted before it is scaled: the rounding of a scaled score is as large as weights are far apart
              const uint64_t z[2] = {mul_f2(add_f2(pack_f2(x[e], x[e + 1]), pack_f2(ref.x, ref.y)), scale2),
                                     mul_f2(add_f2(pack_f2(x[e + 2], x[e + 3]), pack_f2(ref.z, ref.w)), scale2)};
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const float2 f = unpack_f2(z[u]);
                y[e / 2 + u] = pack_f2(fast_exp2(f.x), fast_exp2(f.y));
              }
            }
            if (!whole) {
#pragma unroll
              for (int e = 0; e < CW; e += 2) {
                const float2 f = unpack_f2(y[e / 2]);
                y[e / 2] = pack_f2(sees(e) ? f.x : 0.f, sees(e + 1) ? f.y : 0.f);
              }
            }
            if (settled) break;
#pragma unroll
            for (int e = 0; e < CW / 2; ++e) {
              const float2 f = unpack_f2(y[e]);
              top = fmaxf(top, fmaxf(f.x, f.y));
            }
            if (!named_sync_or(bar_group, 128, top > C::TOP)) break;
          }
          // ---- new references: 2^SHIFT below the tile's largest weight of each row, if that is higher; what was summed so far is scaled down
#pragma unroll 1
          for (int c = 0; c < CW; c += 8) {
            float x[8];
            tmem_load_cols<8>(t_s + c, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float m = warp_max(sees(c + e) ? x[e] : -INFINITY);
              if (lane == 0) s_red[q4 * 64 + c0 + c + e] = m;
            }
          }
          named_sync(bar_group, 128);
          if (gt < CW) {
            const int r = c0 + gt;
            const float m = fmaxf(fmaxf(s_red[r], s_red[64 + r]), fmaxf(s_red[128 + r], s_red[192 + r]));
            const float old = j == 0 ? kUnseen : -s_ref[r], now = fmaxf(old, m - C::SHIFT / p.scale_log2);
            s_ref[r] = -now;
            s_alpha[r] = fast_exp2((old - now) * p.scale_log2);
          }
          named_sync(bar_group, 128);
          if (j > 0) {
            wait(pv_done + 8 * ((i - 1) % C::NP), (i - 1) / C::NP);
            tc_fence_after();
#pragma unroll
            for (int e = 0; e < CW / 2; ++e) {
              const uint64_t a = pack_f2(s_alpha[c0 + 2 * e], s_alpha[c0 + 2 * e + 1]);
              l[e] = mul_f2(l[e], a);
            }
#pragma unroll 1
            for (int part = 0; part < C::BANDS * C::HALVES; ++part) {
#pragma unroll 1
              for (int c = 0; c < CW; c += 8) {
                const uint32_t o = tmem + C::COL_O + ob * C::O_COLS + part * N + lane_off + c0 + c;
                float v[8];
                tmem_load_cols<8>(o, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= s_alpha[c0 + c + e];
                tmem_store_cols<8>(o, v);
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(s_free + 8 * (i % C::SB));
        // slots that no row sees may hold anything: zero their V
        if (__any_sync(0xffffffffu, dead)) {
          // What the tile's V replaces in the ring may not have landed yet: the barrier's parity would then name an
          // earlier phase. The product of the tile before says that it has.
          if (i > 0) wait(pv_done + 8 * ((i - 1) % C::NP), (i - 1) / C::NP);
#pragma unroll 1
          for (int part = 0; part < C::PARTS; ++part) {
            const int n = i * C::PARTS + part, s = KS + n % (NS - KS);
            wait(full + 8 * s, n / (NS - KS));
            if (dead) {
              uint8_t* v = ring + s * C::SLOT + key * 128;
              for (int c = h; c < D / 8 / C::PARTS; c += C::NG)
                *reinterpret_cast<uint4*>(v + (c >> 3) * TK * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
          }
        }
        // ---- sums, and the weights in 16 bits, or twice that
        uint32_t hi[CW / 2], lo[C::BANDS == 2 ? CW / 2 : 1];
#pragma unroll
        for (int e = 0; e < CW / 2; ++e) l[e] = add_f2(l[e], y[e]);
#pragma unroll
        for (int e = 0; e < CW / 2; ++e) {
          const float2 w = unpack_f2(y[e]);
          hi[e] = q4::pack2<C::FP16>(w.x, w.y);
          if constexpr (C::BANDS == 2) {
            const float2 a = q4::unpack2<C::FP16>(hi[e]);
            lo[e] = q4::pack2<C::FP16>((w.x - a.x) * C::LOW, (w.y - a.y) * C::LOW);
          }
        }
        wait(pv_done + 8 * (i % C::NP), i / C::NP - 1);  // the buffer's last product is done
        uint8_t* pb = fixed + S::P + (i % C::NP) * C::BANDS * C::P_BYTES;
        const int swz = (key >> C::P_SWZ_SHIFT) & C::P_SWZ_MASK;
#pragma unroll
        for (int c = 0; c < CW / 8; ++c) {
          const uint32_t at = (uint32_t)(key * N * 2) + ((uint32_t)(((c0 >> 3) + c) ^ swz) << 4);
          *reinterpret_cast<uint4*>(pb + at) = make_uint4(hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]);
          if constexpr (C::BANDS == 2)
            *reinterpret_cast<uint4*>(pb + C::P_BYTES + at) = make_uint4(lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]);
        }
        fence_proxy_async_smem();  // weights and zeroed V are read by the tensor core
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(p_full + 8 * (i & 1));
      }
      // ---- the task's statistics
      wait(o_free + 8 * ob, seq / C::OB - 1);
      base += k.tiles;
      float* stat = reinterpret_cast<float*>(fixed + S::STAT + ob * S::STAT_BYTES);
#pragma unroll 1
      for (int c = 0; c < CW; c += 8) {
        float v[8];
#pragma unroll
        for (int e = 0; e < CW; e += 2) {
          const float2 f = unpack_f2(l[e / 2]);
          if (e / 8 * 8 == c) {
            v[e % 8] = f.x;
            v[e % 8 + 1] = f.y;
          }
        }
        const float sum = reduce_cols<8, false>(v, lane);
        if (lane < 8) stat[q4 * 64 + c0 + c + reduced_col<8>(lane)] = sum;
      }
      if (gt < CW) stat[256 + c0 + gt] = -s_ref[c0 + gt];
      __syncwarp();
      if (lane == 0) bar_arrive(st_full + 8 * ob);
    }
    leave();
  }
}

}  // namespace wattn
}  // namespace specv
