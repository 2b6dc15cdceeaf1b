// Kernels of the tree verify attention (see the comment at the top of
// tree_attention.cu): the tcgen05 kernel, the merge of units that were cut over
// several CTAs, and their parameters, shared with the host side.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include "attention_device.cuh"
#include "tree_device.cuh"

namespace specv {
namespace tattn {

using attn::Cursor;
using attn::cursor_advance;
using attn::cursor_at;
using attn::piece_slot;

constexpr int kMaxGrid = 160;  // one CTA per SM, at most
constexpr int kMaxSlots = 10;  // K and V tiles in shared memory
constexpr int kMinSlots = 4;   // two of each
constexpr int kTmemCols = 512;
constexpr int kLaunchRegs = 168; // registers a thread that a kernel of 384 threads is launched with
constexpr int kTables = 1024;  // bytes of shared memory for barriers and small tables
constexpr int kRows = 128;     // packed query rows of a row tile (MMA M)
constexpr int kBarGroup = 1;   // named barriers: one per softmax warpgroup (1, 2),
constexpr int kBarSoftmax = 3; // all softmax threads,
constexpr int kBarTail = 4;    // softmax threads and the issuing warps

// What the merge needs of a unit cut over several CTAs; written by the CTA that holds its first piece.
struct Split {
  int32_t nseg;  // pieces; 0: no unit starts here that is cut
  int32_t b, u;  // sequence, unit of the sequence
  int32_t slot;  // partial slot of the first piece; the others are slots 2 (c + 1), 2 (c + 2), ...
};

struct Params {
  const int32_t* block_table;
  const int32_t* ctx_lens;
  const int32_t* parents;
  void* out;
  Split* split;  // [kMaxGrid]
  float* lse;    // [2 * kMaxGrid][row tiles of a unit][128], log2 units; NaN: no result
  float4* opart; // [2 * kMaxGrid][row tiles of a unit][D / 4][128], normalised
  int32_t* dev_err;
  int64_t num_blocks;
  int batch, nodes, heads, kv_heads, gqa;
  int npt;     // nodes of a row tile: its npt * gqa rows are packed node by node
  int groups;  // units per kv head
  int page_shift, max_blocks;
  int kslots, vslots;  // depths of the K and the V ring
  int out_f32;
  float scale_log2;
};

template <int D_, int MT_, int TERMS_, bool FP16_>
struct Cfg {
  static constexpr int D = D_, MT = MT_, TERMS = TERMS_;
  static constexpr bool FP16 = FP16_;
  static constexpr bool DUAL = D <= 128;  // two accumulators and two softmax warpgroups
  static constexpr int NWG = DUAL ? 2 : 1;
  static constexpr int ISSUERS = NWG;  // threads that issue MMAs
  static constexpr int TK = (D == 256 || TERMS == 3) ? 64 : 128;  // keys per tile
  static constexpr int PW = TK / 2;                               // tensor-memory columns of one part of P
  static constexpr int SW = TERMS * PW > TK ? TERMS * PW : TK;    // columns of an S / P buffer
  static constexpr int QB = (DUAL && MT == 1) ? 2 : 1;            // query buffers
  static constexpr int SUBS = D / 64;
  static constexpr int Q_TILE = kRows * D * 2;
  static constexpr int Q_BYTES = MT * Q_TILE;
  static constexpr int SLOT = TK * D * 2;
  static constexpr int kThreads = 128 + 128 * NWG;
  static constexpr int COL_O = 2 * SW;
  static constexpr int ML_BYTES = (DUAL && MT == 1) ? 2 * kRows * 8 : 0;  // (max, sum) of both warpgroups' rows
  static_assert(MT == 1 || DUAL, "two row tiles need two accumulators");
  static_assert(COL_O + NWG * D <= kTmemCols, "S / P buffers and accumulators fit tensor memory");
  static_assert(TERMS >= 1 && TERMS <= 3, "");
};

// Shared memory besides the ring: alignment, query buffers, barriers and tables, the plan.
template <class C>
size_t smem_fixed(int batch) {
  return 1024 + (size_t)C::QB * C::Q_BYTES + kTables + C::ML_BYTES + attn::align256((size_t)(batch + 2) * 4);
}

template <class C>
__device__ __forceinline__ uint32_t idesc(int n, int b_mn) {
  return (1u << 4) | (C::FP16 ? 0u : (1u << 7) | (1u << 10)) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(kRows >> 4) << 24);
}
// D[tmem] (+)= A * B^T, 16-bit inputs, fp32 accumulate; the descriptors of A and B share their high word.
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      ".reg .b64 a, b;\n"
      "setp.ne.b32 p, %5, 0;\n"
      "mov.b64 a, {%1, %3};\n"
      "mov.b64 b, {%2, %3};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n"
      "}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(id), "r"(accumulate)
      : "memory");
}
// The same with A in tensor memory.
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      ".reg .b64 b;\n"
      "setp.ne.b32 p, %5, 0;\n"
      "mov.b64 b, {%2, %3};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n"
      "}\n" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(hi), "r"(id), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// 4-D tiled copy into shared memory; c0 * element size is a multiple of 16 bytes.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* map, int c0, int c1, int c2, int c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
template <bool FP16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (FP16) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    return pack_bf16(lo, hi);
  }
}
template <bool FP16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (FP16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Bits k = 0 .. 63: bit (o + k) of m, where bits before the first are 1 (committed tokens) and behind the last 0.
__device__ __forceinline__ uint64_t window(uint64_t m, int o) {
  if (o <= -64) return ~0ull;
  if (o < 0) return (m << -o) | ((1ull << -o) - 1);
  return o < 64 ? m >> o : 0ull;
}

// Write 32 consecutive columns of one output row (element offset `at`).
template <bool FP16>
__device__ __forceinline__ void store_row32(const Params& p, int64_t at, const float (&v)[32]) {
  if (p.out_f32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else {
    uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = make_uint4(pack2<FP16>(v[8 * i], v[8 * i + 1]), pack2<FP16>(v[8 * i + 2], v[8 * i + 3]),
                        pack2<FP16>(v[8 * i + 4], v[8 * i + 5]), pack2<FP16>(v[8 * i + 6], v[8 * i + 7]));
  }
}

// Row r of row tile mt of unit u: its output offset, or -1 for a padding row.
__device__ __forceinline__ int64_t row_offset(const Params& p, int D, int MT, int b, int u, int mt, int r) {
  const int g = u / p.groups, rg = u - g * p.groups;
  const int i = (rg * MT + mt) * p.npt + r / p.gqa, j = r % p.gqa;
  if (r >= p.npt * p.gqa || i >= p.nodes) return -1;
  return (((int64_t)b * p.nodes + i) * p.heads + g * p.gqa + j) * D;
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1) tree_attention_kernel(const Params p,
                                                                        const __grid_constant__ CUtensorMap tm_q,
                                                                        const __grid_constant__ CUtensorMap tm_k,
                                                                        const __grid_constant__ CUtensorMap tm_v) {
  constexpr int D = C::D, MT = C::MT, TK = C::TK, SW = C::SW, PW = C::PW, TERMS = C::TERMS, NWG = C::NWG;
  constexpr int kThreads = C::kThreads, kSoftmaxThreads = 128 * NWG;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int RK = p.kslots, RV = p.vslots, S = RK + RV;
  uint8_t* qbuf = smem;
  uint8_t* ring = qbuf + C::QB * C::Q_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + S * C::SLOT);  // [RK of K, RV of V]: the slot's tile has landed
  uint64_t* empty = full + kMaxSlots;                                // [...]: its MMAs are done
  uint64_t* s_full = empty + kMaxSlots;  // [2]: S buffer x holds the scores of its item
  uint64_t* p_full = s_full + 2;         // [2]: its weights are written (one arrival per warp)
  uint64_t* pv_done = p_full + 2;        // [2]: the product that read them is complete
  uint64_t* q_full = pv_done + 2;        // [2]
  uint64_t* q_empty = q_full + 2;        // [2]
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(q_empty + 2);
  int32_t* s_lock = reinterpret_cast<int32_t*>(s_tmem + 1);
  int32_t* s_bad = reinterpret_cast<int32_t*>(s_tmem + 2);  // [8] per piece (seq & 7): a page id was bad
  int32_t* s_misc = s_bad + 8;                              // [32]
  uint64_t* s_used = reinterpret_cast<uint64_t*>(s_misc + 32);  // [2 warpgroups]
  int32_t* s_par = reinterpret_cast<int32_t*>(s_used + 2);      // [2 warpgroups][64]
  static_assert(8 * (2 * kMaxSlots + 10) + 8 + 32 + 128 + 16 + 2 * 64 * 4 <= kTables, "the tables fit their area");
  float2* s_ml = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(full) + kTables);  // [2 warpgroups][128]
  int32_t* s_prefix = reinterpret_cast<int32_t*>(reinterpret_cast<uint8_t*>(s_ml) + C::ML_BYTES);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = p.batch, N = p.nodes, U = p.kv_heads * p.groups;
  const int64_t max_ctx = (int64_t)p.max_blocks << p.page_shift;

  // ---- split plan (every CTA): tiles of every sequence and their prefix
  // A sequence's tiles: 0 for an empty row or a context length out of range (its rows are zeros).
  auto tiles_of = [&](int b, int& ctx) -> int {
    if (p.parents[(int64_t)b * N] == SPEC_TREE_UNUSED) {
      ctx = 0;
      return 0;
    }
    ctx = p.ctx_lens[b];
    return (ctx >= N && (int64_t)ctx <= max_ctx) ? (ctx + TK - 1) / TK : 0;
  };
  {
    const int per = (B + kThreads - 1) / kThreads;
    const int b0 = tid * per;
    int mine = 0, lo = INT32_MAX, hi = 0;
    if (tid == 0) {
      s_misc[30] = INT32_MAX;
      s_misc[31] = 0;
    }
    for (int b = b0; b < b0 + per && b < B; ++b) {
      int ctx;
      const int nt = tiles_of(b, ctx);
      s_prefix[b] = nt;
      mine += nt;
      if (nt > 0) {
        lo = min(lo, nt);
        hi = max(hi, nt);
      }
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s_misc[warp] = incl;
    __syncthreads();
    if (hi > 0) {
      atomicMin(&s_misc[30], lo);
      atomicMax(&s_misc[31], hi);
    }
    int run = incl - mine;
    for (int w = 0; w < warp; ++w) run += s_misc[w];
    if (tid == kThreads - 1) s_prefix[B] = run + mine;
    for (int b = b0; b < b0 + per && b < B; ++b) {
      const int nt = s_prefix[b];
      s_prefix[b] = run;
      run += nt;
    }
    if (tid == 0) {
      for (int s = 0; s < S; ++s) {
        mbar_init(&full[s], 1);
        mbar_init(&empty[s], MT);  // one arrival for each row tile that read it
      }
      for (int x = 0; x < 2; ++x) {
        mbar_init(&s_full[x], 1);
        mbar_init(&p_full[x], 4);
        mbar_init(&pv_done[x], 1);
        mbar_init(&q_full[x], 1);
        mbar_init(&q_empty[x], C::ISSUERS);
      }
      fence_mbar_init();
      *s_lock = 0;
      p.split[blockIdx.x].nseg = 0;
    }
    __syncthreads();
  }
  // rows of sequences without work
  for (int b = blockIdx.x; b < B; b += gridDim.x) {
    if (s_prefix[b + 1] != s_prefix[b]) continue;
    int ctx;
    tiles_of(b, ctx);
    if (tid == 0 && p.parents[(int64_t)b * N] != SPEC_TREE_UNUSED) raise_error(p.dev_err, SPEC_DEVERR_CTX_LEN);
    const int64_t bytes = (int64_t)N * p.heads * D * (p.out_f32 ? 4 : 2);
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + b * bytes);
    for (int64_t i = tid; i < bytes / 16; i += kThreads) dst[i] = make_uint4(0, 0, 0, 0);
  }
  const int64_t T = (int64_t)s_prefix[B] * U;
  if (T == 0) return;
  const int64_t W = (T + gridDim.x - 1) / gridDim.x;
  const int64_t f0 = (int64_t)blockIdx.x * W;
  const int64_t f1 = min(T, f0 + W);
  if (f0 >= f1) return;
  const int n_tiles = (int)(f1 - f0);

  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), kTmemCols);
    tmem_relinquish();
  }
  // padding rows of the query tiles (the copies write npt * gqa rows each)
  const int packed = p.npt * p.gqa;
  for (int i = tid; i < C::QB * MT * C::SUBS * (kRows - packed) * 8; i += kThreads) {
    const int rest = i / 8, slice = rest / (kRows - packed), r = packed + rest % (kRows - packed);
    *reinterpret_cast<uint4*>(qbuf + slice * kRows * 128 + r * 128 + (i % 8) * 16) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const uint32_t ring_u32 = smem_u32(ring), q_u32 = smem_u32(qbuf);
  // Every wait is bounded (about 0.2 s); a thread that gave up once waits no more and the producer stops copying, so the
  // kernel ends and SPEC_DEVERR_TIMEOUT says that its output is not to be used.
  bool lost = false;
  auto wait = [&](uint64_t* bar, int phase) {
    if (!lost && !mbar_wait_bounded(bar, (uint32_t)(phase & 1), 400000000LL)) {
      lost = true;
      raise_error(p.dev_err, SPEC_DEVERR_TIMEOUT);
    }
  };

  // Registers: 384 threads are launched with kLaunchRegs each; the warps that only issue copies and MMAs give theirs to
  // the softmax warps, which hold a row's scores (3 * 168 = 72 + 2 * 216). Each role's branch has its own
  // instruction: where branches join, the compiler would hold all that follows to the smaller number.
  if (warp == 0) {
    // =================== producer: TMA ===================
    // Tile j's K goes to slot j % RK of the K ring, its V to slot j % RV of the V ring, in the order in which they are
    // taken: K0, K1 V0, K2 V1, ... with one row tile, K0 V0, K1 V1, ... with two. A barrier's parity names its phase only
    // while the phase before is over, so every slot is used by both issuers, or by one alone (even depths, one row tile).
    if constexpr (C::DUAL) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;\n");
    const int bs = 1 << p.page_shift;
    const int BH = bs < TK ? bs : TK;
    const int pieces = TK / BH;
    const uint64_t pol = l2_evict_first_policy();  // K and V that no other unit reads again
    // Lane i < pieces copies page piece i of a tile.
    Cursor ld = cursor_at(f0, s_prefix, B, U);
    int seq = 0, win_b = -1, win_base = 0, win_val = 0, ctx = p.ctx_lens[ld.b];
    bool fresh = true;
    int zk = 0, zv = 0, gv = 0;  // token rows of the lane's piece, kv head
    auto load_tile = [&](const CUtensorMap* map, int g, int z, int first, int depth, int j) {  // ring `first`, tile j
      const int s = first + j % depth;
      if (lane == 0) {
        if (j >= depth) wait(&empty[s], j / depth - 1);
        if (!lost) mbar_arrive_expect_tx(&full[s], (uint32_t)C::SLOT);
      }
      lost = __shfl_sync(0xffffffffu, (int)lost, 0) != 0;
      if (lane < pieces && !lost) {
        const uint32_t dst = ring_u32 + s * C::SLOT + lane * BH * 128;
#pragma unroll
        for (int sub = 0; sub < C::SUBS; ++sub) {
          if (p.groups == 1) tma_load_3d_hint(dst + sub * TK * 128, map, sub * 64, g, z, &full[s], pol);
          else tma_load_3d(dst + sub * TK * 128, map, sub * 64, g, z, &full[s]);
        }
      }
    };
#pragma unroll 1
    for (int j = 0; j < n_tiles; ++j) {
      const int g = ld.g / p.groups;
      zv = zk;
      {
        // the tile's page ids, from a window of 32 of the block table's row held by the lanes
        const int n_first = (ld.tile * TK) >> p.page_shift;
        if (ld.b != win_b || n_first < win_base || n_first + pieces > win_base + 32) {
          win_b = ld.b;
          win_base = n_first;
          win_val = (n_first + lane < ((ctx + bs - 1) >> p.page_shift))
                        ? __ldg(p.block_table + (int64_t)ld.b * p.max_blocks + n_first + lane) : 0;
        }
        const int t = ld.tile * TK + lane * BH;
        const int32_t page = __shfl_sync(0xffffffffu, win_val, ((t >> p.page_shift) - win_base) & 31);
        const bool in = lane < pieces && t < ctx, ok = page >= 0 && (int64_t)page < p.num_blocks;
        zk = in && ok ? (int)(((int64_t)page << p.page_shift) + (t & (bs - 1))) : -BH;  // -BH: reads zeros
        const bool bad = __any_sync(0xffffffffu, in && !ok);
        if (lane == 0) {
          if (fresh) s_bad[seq & 7] = 0;
          if (bad) s_bad[seq & 7] = 1;
        }
      }
      load_tile(&tm_k, g, zk, 0, RK, j);
      if (MT == 2) load_tile(&tm_v, g, zk, RK, RV, j);
      else if (j > 0) load_tile(&tm_v, gv, zv, RK, RV, j - 1);
      if (fresh && lane == 0) {
        const int x = seq % C::QB;
        if (seq >= C::QB) wait(&q_empty[x], seq / C::QB - 1);
        const int n0 = (ld.g % p.groups) * MT * p.npt;
        if (!lost) mbar_arrive_expect_tx(&q_full[x], (uint32_t)(MT * packed * D * 2));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int sub = 0; sub < C::SUBS && !lost; ++sub)
            tma_load_4d(q_u32 + x * C::Q_BYTES + mt * C::Q_TILE + sub * kRows * 128, &tm_q, sub * 64, g * p.gqa,
                        n0 + mt * p.npt, ld.b, &q_full[x]);
      }
      __syncwarp();
      gv = g;
      const int before = ld.seq, b_before = ld.b;
      cursor_advance(ld, s_prefix, B, U);
      fresh = ld.seq != before;
      if (fresh) ++seq;
      if (ld.b != b_before && ld.b < B) ctx = p.ctx_lens[ld.b];
    }
    if (MT == 1) load_tile(&tm_v, gv, zk, RK, RV, n_tiles - 1);
    return;
  }

  if (warp <= C::ISSUERS) {
    // =================== MMA issuers (one thread of warp 1, and of warp 2 with two accumulators) ===================
    // Item j is tile j (one row tile) or row tile j & 1 of tile j >> 1 (two); it uses S / P buffer j & 1. An issuer's
    // MMAs run in the order of its instructions, so scores issued after a product may overwrite the weights it reads.
    if constexpr (C::DUAL) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;\n");
    if (lane == 0) {
      const uint32_t id_qk = idesc<C>(TK, 0), id_pv = idesc<C>(D, 1);
      // Descriptors differ in their low words only (start address / 16 in the low 14 bits).
      const uint64_t kmaj = smem_desc_sw128(0, 16, 1024);       // Q, K: rows of 64 elements, K-major
      const uint64_t vmn = smem_desc_sw128(0, TK * 128, 1024);  // V: MN-major, slices of 64 dims
      const uint32_t k_hi = (uint32_t)(kmaj >> 32), v_hi = (uint32_t)(vmn >> 32);
      const uint32_t q_lo = (uint32_t)kmaj + (q_u32 >> 4), k_lo = (uint32_t)kmaj + (ring_u32 >> 4);
      const uint32_t v_lo = (uint32_t)vmn + (ring_u32 >> 4);
      auto qk = [&](uint32_t s, uint32_t qb, int slot) {  // scores into buffer address s
        tc_fence_after();
        const uint32_t kb = k_lo + slot * (C::SLOT >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t qo = ((ks >> 2) * kRows * 128 + (ks & 3) * 32) >> 4;
          const uint32_t ko = ((ks >> 2) * TK * 128 + (ks & 3) * 32) >> 4;
          umma_ss(s, qb + qo, kb + ko, k_hi, id_qk, ks > 0 ? 1u : 0u);
        }
      };
      auto pv = [&](uint32_t d, uint32_t s, int slot, bool first) {  // first: nothing is in the accumulator yet
        tc_fence_after();
        const uint32_t vb = v_lo + slot * (C::SLOT >> 4);
#pragma unroll
        for (int term = 0; term < TERMS; ++term)
#pragma unroll
          for (int kk = 0; kk < TK / 16; ++kk)
            umma_ts(d, s + term * PW + kk * 8, vb + ((kk * 2048) >> 4), v_hi, id_pv,
                    (first && term == 0 && kk == 0) ? 0u : 1u);
      };
      if constexpr (C::DUAL) {
        // Issuer h owns buffer and accumulator h: scores, wait for the weights, product, next scores. The two issuers'
        // MMAs interleave, so one item's softmax runs under the other's MMAs.
        const int h = warp - 1;
        const uint32_t s = tmem + (uint32_t)(h * SW), d = tmem + (uint32_t)(C::COL_O + h * D);
        constexpr int step = MT == 1 ? 2 : 1;  // tiles from one item of an issuer to its next
        Cursor cu = cursor_at(f0, s_prefix, B, U);
        int done = 0, item = 0, sk = MT == 1 ? h : 0, sv = sk, pk = 0, pv_ = 0;  // slots and phases of the item's K and V
        // A product and the next scores are issued as one burst under a lock: if the two issuers' MMAs alternated one by
        // one, both items' results would come at the end of both, and both softmaxes would run at once, then both
        // MMA phases (measured: 5000 cycles a tile against 3000).
        bool held = false;
        auto lock = [&]() {
          const long long start = clock64();  // order is all it gives: after the limit the issue goes on without it
          while (!held && atomicCAS(s_lock, 0, 1) != 0 && clock64() - start < 100000) {
          }
          held = true;
        };
        auto unlock = [&]() {
          if (held) atomicExch(s_lock, 0);
          held = false;
        };
        for (int seq = 0; done < n_tiles; ++seq) {
          const int n = min(cu.ntiles - cu.tile, n_tiles - done), x = seq % C::QB;
          const int t_first = MT == 1 ? ((done & 1) == h ? 0 : 1) : 0;
          const uint32_t qb = q_lo + ((x * C::Q_BYTES + (MT == 2 ? h : 0) * C::Q_TILE) >> 4);
          if (held && !mbar_try_wait(&q_full[x], (uint32_t)((seq / C::QB) & 1))) unlock();
          wait(&q_full[x], seq / C::QB);  // without an item too: the buffer's last use must be over before the arrival
          if (t_first >= n) mbar_arrive(&q_empty[x]);
          for (int tt = t_first; tt < n; tt += step, ++item) {
            if (!mbar_try_wait(&full[sk], (uint32_t)(pk & 1))) {
              unlock();  // not while waiting
              wait(&full[sk], pk);
            }
            lock();
            qk(s, qb, sk);
            umma_commit(&s_full[h]);
            unlock();
            umma_commit(&empty[sk]);
            if (tt + step >= n) umma_commit(&q_empty[x]);
            if ((sk += step) >= RK) sk -= RK, ++pk;
            wait(&full[RK + sv], pv_);
            wait(&p_full[h], item);
            lock();
            pv(d, s, RK + sv, tt == t_first);
            umma_commit(&pv_done[h]);
            umma_commit(&empty[RK + sv]);
            if ((sv += step) >= RV) sv -= RV, ++pv_;
          }
          done += n;
          cu.tile += n - 1;
          cursor_advance(cu, s_prefix, B, U);
        }
        unlock();
      } else {
        // One accumulator: the scores of item j + 1 are issued before the product of item j, so they run while the
        // softmax works on item j.
        const uint32_t d = tmem + (uint32_t)C::COL_O;
        Cursor cq = cursor_at(f0, s_prefix, B, U), cv = cq;
        int left_q = min(cq.ntiles - cq.tile, n_tiles), left_v = left_q, sk = 0, pk = 0, sv = 0, pv_ = 0;
        bool q_fresh = true, v_fresh = true;
        auto issue_qk = [&](int j) {
          if (q_fresh) wait(&q_full[0], cq.seq);
          wait(&full[sk], pk);
          qk(tmem + (uint32_t)((j & 1) * SW), q_lo, sk);
          umma_commit(&s_full[j & 1]);
          umma_commit(&empty[sk]);
          if (++sk == RK) sk = 0, ++pk;
          q_fresh = --left_q == 0;
          if (q_fresh) {
            umma_commit(&q_empty[0]);
            cq.tile = cq.ntiles - 1;
            cursor_advance(cq, s_prefix, B, U);
            left_q = cq.ntiles;
          }
        };
        issue_qk(0);
        for (int j = 0; j < n_tiles; ++j) {
          if (j + 1 < n_tiles) issue_qk(j + 1);
          wait(&full[RK + sv], pv_);
          wait(&p_full[j & 1], j >> 1);
          pv(d, tmem + (uint32_t)((j & 1) * SW), RK + sv, v_fresh);
          umma_commit(&pv_done[j & 1]);
          umma_commit(&empty[RK + sv]);
          if (++sv == RV) sv = 0, ++pv_;
          v_fresh = --left_v == 0;
          if (v_fresh) {
            cv.tile = cv.ntiles - 1;
            cursor_advance(cv, s_prefix, B, U);
            left_v = cv.ntiles;
          }
        }
      }
    }
    __syncwarp();
    named_sync(kBarTail, 32 * C::ISSUERS + kSoftmaxThreads);  // the softmax warps are done with tensor memory
    if (warp == 1) {
      tc_fence_after();
      tmem_dealloc(tmem, kTmemCols);
    }
    return;
  }
  if (warp < 4) {
    if constexpr (C::DUAL) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;\n");
    return;
  }

  // =================== softmax / epilogue: one thread per row ===================
  if constexpr (C::DUAL) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;\n");
  const int h = (warp - 4) >> 2;      // warpgroup
  const int r = tid - 128 - h * 128;  // row of the row tile = tensor-memory lane
  const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
  const int bar = kBarGroup + h;
  const int mt = MT == 2 ? h : 0;
  const uint32_t t_o = tmem + (uint32_t)(C::COL_O + h * D) + lanes;  // this warpgroup's accumulator
  auto wait_pv = [&](int j) {
    wait(&pv_done[j & 1], j >> 1);
    tc_fence_after();
  };
  // The slot of item j's V tile, which has landed. The slot's tile before it was multiplied before the scores of item j
  // were issued (RV >= 2), so the parity is unambiguous.
  auto wait_v = [&](int j) -> int {
    const int tile = MT == 2 ? j >> 1 : j, s = RK + tile % RV;
    wait(&full[s], tile / RV);
    return s;
  };

  Cursor cu = cursor_at(f0, s_prefix, B, U);
  int done = 0;  // tiles of this CTA before the unit
  for (int seq = 0; done < n_tiles; ++seq) {
    const int b = cu.b, u = cu.g, n = min(cu.ntiles - cu.tile, n_tiles - done);
    const int ctx = p.ctx_lens[b], base = ctx - N;
    const int n0 = ((u % p.groups) * MT + mt) * p.npt;  // first node of the row tile
    float m = -INFINITY, l = 0.f;  // running maximum (scaled; it may lag by up to 8) and sum of the row
    bool tree_bad = false, dead = false, have_tree = false;
    uint64_t sees = 0, used = 0;
    int mine = 0;  // items of this warpgroup in the unit so far
    int last_j = -1;
    // the first tile of this warpgroup: every tile, or every other one of the CTA's
    const int t_first = (C::DUAL && MT == 1) ? ((done & 1) == h ? 0 : 1) : 0;
    for (int tt = t_first; tt < n; tt += (C::DUAL && MT == 1) ? 2 : 1) {
      const int j = MT == 2 ? 2 * (done + tt) + h : done + tt;
      const int x = j & 1;
      const uint32_t t_s = tmem + (uint32_t)(x * SW) + lanes;
      const int t0 = (cu.tile + tt) * TK;
      const bool edge = t0 + TK > base;  // the tile holds keys that not every row sees
      if (edge && !have_tree) {
        have_tree = true;
        if (r < N) s_par[h * 64 + r] = __ldg(p.parents + (int64_t)b * N + r);
        named_sync(bar, 128);
        const bool bad = r < N && !tree::parent_ok(s_par + h * 64, r);
        const uint32_t word = __ballot_sync(0xffffffffu, r < N && s_par[h * 64 + (r & 63)] != SPEC_TREE_UNUSED);
        if (r == 0) reinterpret_cast<uint32_t*>(s_used + h)[0] = word;
        if (r == 32) reinterpret_cast<uint32_t*>(s_used + h)[1] = word;
        tree_bad = named_sync_or(bar, 128, bad);
        used = s_used[h];
        const int node = n0 + r / p.gqa;
        if (r < packed && node < N) {
          sees = tree::ancestors(s_par + h * 64, node);
          dead = sees == 0;
        }
      }
      wait(&s_full[x], j >> 1);
      tc_fence_after();
      float v[TK];
#pragma unroll
      for (int c = 0; c < TK / 16; ++c) tmem_ld16(t_s + c * 16, *reinterpret_cast<float(*)[16]>(&v[c * 16]));
      tmem_wait_ld_regs<TK>(v);
      if (edge) {
        const int off = t0 - base;
        // V of slots that no row sees may hold anything: zeros, so that 0 weights give 0. With two row tiles both
        // warpgroups write them, each before its own product.
        {
          const uint64_t dead0 = ~window(used, off), dead1 = TK > 64 ? ~window(used, off + 64) : 0;
          if (dead0 | dead1) {
            uint8_t* vt = ring + wait_v(j) * C::SLOT;
            for (int i = r; i < TK * (D / 8); i += 128) {
              const int key = i / (D / 8), ch = i % (D / 8);
              if (((key < 64 ? dead0 : dead1) >> (key & 63)) & 1)
                *reinterpret_cast<uint4*>(vt + (ch >> 3) * TK * 128 + key * 128 + (((ch & 7) ^ (key & 7)) << 4)) =
                    make_uint4(0, 0, 0, 0);
            }
          }
        }
#pragma unroll
        for (int half = 0; half < TK / 64; ++half) {
          const uint64_t w = window(sees, off + 64 * half);
          const uint32_t w0 = (uint32_t)w, w1 = (uint32_t)(w >> 32);
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            if (!((w0 >> k) & 1)) v[64 * half + k] = -INFINITY;
            if (!((w1 >> k) & 1)) v[64 * half + 32 + k] = -INFINITY;
          }
        }
      }
      float mx;
      {
        float a[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = v[i];
#pragma unroll
        for (int k = 8; k < TK; k += 16)
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i] = k + 8 + i < TK ? max3(a[i], v[k + i], v[k + 8 + i]) : fmaxf(a[i], v[k + i]);
        mx = max3(max3(a[0], a[1], a[2]), max3(a[3], a[4], a[5]), fmaxf(a[6], a[7])) * p.scale_log2;
      }
      const bool grow = mx > m + 8.f;
      if (__any_sync(0xffffffffu, grow)) {
        const float mn = grow ? mx : m;
        const float a = grow ? (m == -INFINITY ? 0.f : fast_exp2(m - mn)) : 1.f;
        m = mn;
        l *= a;
        if (mine > 0) {  // the accumulator holds earlier tiles
          wait_pv(last_j);
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            float o[16];
            tmem_ld16(t_o + c, o);
            tmem_wait_ld_regs<16>(o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= a;
            tmem_st16(t_o + c, o);
          }
        }
      }
      const float ms = m == -INFINITY ? 0.f : m;
      float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
#pragma unroll
      for (int c = 0; c < TK; c += 32) {
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          v[c + i] = fast_exp2(fmaf(v[c + i], p.scale_log2, -ms));
          v[c + i + 1] = fast_exp2(fmaf(v[c + i + 1], p.scale_log2, -ms));
          v[c + i + 2] = fast_exp2(fmaf(v[c + i + 2], p.scale_log2, -ms));
          v[c + i + 3] = fast_exp2(fmaf(v[c + i + 3], p.scale_log2, -ms));
          l0 += v[c + i];
          l1 += v[c + i + 1];
          l2 += v[c + i + 2];
          l3 += v[c + i + 3];
        }
        uint32_t w[16];
#pragma unroll
        for (int term = 0; term < TERMS; ++term) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float& e0 = v[c + 2 * i];
            float& e1 = v[c + 2 * i + 1];
            w[i] = pack2<C::FP16>(e0, e1);
            if (term + 1 < TERMS) {
              const float2 f = unpack2<C::FP16>(w[i]);
              e0 -= f.x;  // exact: the next part holds what this one left
              e1 -= f.y;
            }
          }
          tmem_st16u(t_s + term * PW + c / 2, w);
        }
      }
      l += (l0 + l1) + (l2 + l3);
      tmem_wait_st();
      if (edge) fence_proxy_async_smem();  // zeroed rows of V
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[x]);
      last_j = j;
      ++mine;
    }

    // ---- the unit's rows: output, or a normalised partial and its log-sum-exp
    const bool whole = cu.tile == 0 && n == cu.ntiles;
    const int64_t u0 = (int64_t)s_prefix[b] * U + (int64_t)u * cu.ntiles;
    const int c0 = (int)(u0 / W);
    const int slot = piece_slot((int)blockIdx.x, c0, u0, W);
    if (!whole && cu.tile == 0 && tid == 128)
      p.split[blockIdx.x] = Split{(int)((u0 + cu.ntiles - 1) / W) - c0 + 1, b, u, slot};
    if (mine > 0) wait_pv(last_j);
    if (tree_bad && r == 0) raise_error(p.dev_err, SPEC_DEVERR_TREE);
    if (tree_bad || dead) l = __int_as_float(0x7fc00000);  // no result: the row is zeros
    float L = l, M = m, f[2] = {0.f, 0.f};  // factors of the accumulators
    if constexpr (C::DUAL && MT == 1) {
      // both warpgroups hold the same rows, over different keys: each writes half of the columns of their sum
      s_ml[h * kRows + r] = make_float2(m, l);
      tc_fence_before();
      named_sync(kBarSoftmax, kSoftmaxThreads);
      tc_fence_after();
      const float2 a = s_ml[r], c = s_ml[kRows + r];
      M = fmaxf(a.x, c.x);
      const float w0 = a.x == -INFINITY ? 0.f : fast_exp2(a.x - M), w1 = c.x == -INFINITY ? 0.f : fast_exp2(c.x - M);
      L = a.y * w0 + c.y * w1;
      if (a.y != a.y || c.y != c.y) L = __int_as_float(0x7fc00000);
      f[0] = w0;
      f[1] = w1;
    } else {
      f[0] = 1.f;
    }
    // read here: a warpgroup without a tile of the unit knows only now that the unit was loaded
    const bool bad = s_bad[seq & 7] != 0;
    if (bad && tid == 128) raise_error(p.dev_err, SPEC_DEVERR_BLOCK_ID);
    if (bad) L = __int_as_float(0x7fc00000);
    const bool some = L > 0.f;
    const float inv = some ? 1.f / L : 0.f;
    f[0] *= inv;
    f[1] *= inv;
    const int64_t row = row_offset(p, D, MT, b, u, mt, r);
    if (!whole && (h == 0 || MT == 2))
      p.lse[((int64_t)slot * MT + mt) * kRows + r] = some ? M + __log2f(L) : (L == 0.f ? -INFINITY : L);
    constexpr int COLS = (C::DUAL && MT == 1) ? D / 2 : D;
    const int col0 = (C::DUAL && MT == 1) ? h * COLS : 0;
    const uint32_t t_acc = (C::DUAL && MT == 1) ? tmem + (uint32_t)C::COL_O + lanes : t_o;
    // an accumulator that got no tile of the unit holds anything
    const bool has0 = !(C::DUAL && MT == 1) || (done & 1) == 0 || n > 1, has1 = (C::DUAL && MT == 1) && ((done & 1) == 1 || n > 1);
#pragma unroll 1
    for (int c = 0; c < COLS; c += 32) {
      float o[32], o1[32];
      if (has0) {
        tmem_ld16(t_acc + col0 + c, *reinterpret_cast<float(*)[16]>(&o[0]));
        tmem_ld16(t_acc + col0 + c + 16, *reinterpret_cast<float(*)[16]>(&o[16]));
      }
      if (has1) {
        tmem_ld16(t_acc + D + col0 + c, *reinterpret_cast<float(*)[16]>(&o1[0]));
        tmem_ld16(t_acc + D + col0 + c + 16, *reinterpret_cast<float(*)[16]>(&o1[16]));
      }
      tmem_wait_ld_regs<32>(o);
      if (has1) tmem_wait_ld_regs<32>(o1);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        float a = has0 ? o[i] * f[0] : 0.f;
        if (has1) a = fmaf(o1[i], f[1], a);
        o[i] = some ? a : 0.f;
      }
      if (whole) {
        if (row >= 0) store_row32<C::FP16>(p, row + col0 + c, o);
      } else {
        float4* dst = p.opart + (((int64_t)slot * MT + mt) * (D / 4) + (col0 + c) / 4) * kRows + r;
#pragma unroll
        for (int i = 0; i < 8; ++i) dst[i * kRows] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
      }
    }
    if constexpr (C::DUAL && MT == 1) {
      tc_fence_before();
      named_sync(kBarSoftmax, kSoftmaxThreads);  // both accumulators are read, s_ml is free
      tc_fence_after();
    }
    done += n;
    cu.tile += n - 1;
    cursor_advance(cu, s_prefix, B, U);
  }
  tc_fence_before();
  named_sync(kBarTail, 32 * C::ISSUERS + kSoftmaxThreads);
}

// Joins the pieces of the units that were cut: CTA (c, chunk) the 32 columns `chunk` of a row tile of the unit whose
// first piece CTA c of the kernel above held; out = sum_k w_k part_k / sum_k w_k, w_k = 2^(lse_k - max lse).
template <class C>
__global__ void __launch_bounds__(kRows) tree_merge_kernel(const Params p) {
  constexpr int D = C::D, MT = C::MT;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int4 sv = __ldcg(reinterpret_cast<const int4*>(p.split) + blockIdx.x);
  const Split s{sv.x, sv.y, sv.z, sv.w};
  if (s.nseg == 0) return;
  const int r = threadIdx.x, mt = blockIdx.y / (D / 32), c4 = (blockIdx.y % (D / 32)) * 8;
  const int64_t row = row_offset(p, D, MT, s.b, s.u, mt, r);
  if (row < 0) return;
  auto slot = [&](int k) -> int64_t { return ((k == 0 ? s.slot : 2 * ((int64_t)blockIdx.x + k)) * MT + mt); };
  float M = -INFINITY;
  bool nan = false;
#pragma unroll 4
  for (int k = 0; k < s.nseg; ++k) {
    const float v = __ldcg(p.lse + slot(k) * kRows + r);
    nan |= v != v;
    M = fmaxf(M, v);
  }
  const bool some = !nan && M > -INFINITY;
  float acc[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) acc[i] = 0.f;
  float Z = 0.f;
  if (some) {
#pragma unroll 2
    for (int k = 0; k < s.nseg; ++k) {
      const float w = fast_exp2(__ldcg(p.lse + slot(k) * kRows + r) - M);
      const float4* part = p.opart + (slot(k) * (D / 4) + c4) * kRows + r;
      Z += w;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 v = __ldcg(part + i * kRows);
        acc[4 * i] = fmaf(w, v.x, acc[4 * i]);
        acc[4 * i + 1] = fmaf(w, v.y, acc[4 * i + 1]);
        acc[4 * i + 2] = fmaf(w, v.z, acc[4 * i + 2]);
        acc[4 * i + 3] = fmaf(w, v.w, acc[4 * i + 3]);
      }
    }
    const float inv = 1.f / Z;
#pragma unroll
    for (int i = 0; i < 32; ++i) acc[i] *= inv;
  }
  store_row32<C::FP16>(p, row + c4 * 4, acc);
}

// Host side, one translation unit per head dim: the instance for a call. `settings` gets its grid and ring slots.
struct Launch {
  int grid = 0, kslots = 0, vslots = 0;
  size_t smem = 0;
};
struct Call {
  Params p;
  CUtensorMap tq, tk, tv;
  cudaStream_t stream;
};
// tile(): keys per tile of the instance for head dim D, `terms` parts of P.
inline int tile_keys(int D, int terms) { return (D == 256 || terms == 3) ? 64 : 128; }
template <int D>
int settings(int mt, int terms, bool fp16, int batch, Launch* l);
template <int D>
int launch(int mt, int terms, bool fp16, const Launch& l, const Call& c);

}  // namespace tattn
}  // namespace specv
