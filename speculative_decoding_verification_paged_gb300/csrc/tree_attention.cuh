// Kernel of the tree verify attention (see the comment at the top of
// tree_attention.cu) and its parameters, shared with the host side.
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

// Partial slot of the piece of unit [u0, ...) held by CTA c: slot 0 for a CTA's first unit, slot 1 for its last one (the
// units between are whole).
__device__ __forceinline__ int piece_slot(int c, int c0, int u0, int W) { return 2 * c + ((c == c0 && u0 > c * W) ? 1 : 0); }

constexpr int kMaxGrid = 160;  // one CTA per SM, at most
static_assert(kMaxGrid * 4 <= SPEC_ATTN_COUNTER_BYTES, "the counters keep to their area, which the chain call shares");
constexpr int kMaxSlots = 10;  // K and V tiles in shared memory
constexpr int kTmemCols = 512;
constexpr int kLaunchRegs = 96;  // registers a thread that a kernel of 640 threads is launched with
constexpr int kCutBytes = 6 * 32768;  // see tiles_per_cta
constexpr int kRadix = 8;  // runs of pieces that are joined at once
constexpr int kAlignBatch = 256;  // rows whose tile counts fit the statistics' area
constexpr int kTables = 576;   // bytes of shared memory for barriers and small tables
constexpr int kRows = 128;     // packed query rows of a row tile (MMA M)
constexpr int kBarStream = 1;  // named barriers: the softmax threads of a stream (1, 2),
constexpr int kBarSoftmax = 3; // all softmax threads,
constexpr int kBarTail = 4;    // softmax threads and the issuing warp

struct Params {
  const int32_t* block_table;
  const int32_t* ctx_lens;
  const int32_t* parents;
  void* out;
  int32_t* counters;  // [kMaxGrid], zero between calls: pieces that met at the border before CTA c
  float* lse;         // [2 * kMaxGrid][row tiles of a unit][128], log2 units; +inf: no result (NaN: scores without a value)
  float4* opart;      // [2 * kMaxGrid][row tiles of a unit][D / 4][128], normalised
  float4* folds;      // [kMaxGrid][streams][D / 4][128], see fold
  int32_t* dev_err;
  int64_t num_blocks;
  int batch, nodes, heads, kv_heads, gqa;
  int npt;     // nodes of a row tile: its npt * gqa rows are packed node by node
  int groups;  // units per kv head
  int page_shift, max_blocks;
  int kslots, vslots;  // depths of the K and the V ring
  int out_f32, out_wide;  // fp32 output; output 32-byte aligned
  float scale_log2;
};

template <int D_, int MT_, int TERMS_, bool FP16_>
struct Cfg {
  static constexpr int D = D_, MT = MT_, TERMS = TERMS_;
  static constexpr bool FP16 = FP16_;
  // Keys per tile. 128 keep the scores' MMAs at N = 128 (66 cycles each for 16 head dims; N = 64 takes 96); at D = 256
  // two tiles of 128 keys would leave no room for a ring.
  static constexpr int TK = D <= 128 ? 128 : 64;
  static constexpr int PW = TK / 2;                             // tensor-memory columns of one part of P
  static constexpr int SW = TERMS * PW > TK ? TERMS * PW : TK;  // columns of an S / P buffer
  // Streams: accumulators, each with an S / P buffer and two softmax warpgroups, which work in turns with the tensor
  // core. One accumulator with two buffers where two do not fit tensor memory.
  static constexpr int STREAMS = 2 * (SW + D) <= kTmemCols ? 2 : 1;
  static constexpr int NB = STREAMS == 2 ? 1 : 2;  // S / P buffers a stream
  static constexpr int BUFS = 2;
  static constexpr int AHEAD = BUFS / MT;  // tiles whose scores are issued before a tile's product
  static constexpr bool JOIN = STREAMS == 2 && MT == 1;  // two accumulators hold the same rows
  static constexpr int CW = TK / 2;                      // keys of a softmax thread
  static constexpr int SUBS = D / 64;
  static constexpr int Q_TILE = kRows * D * 2;
  static constexpr int Q_BYTES = MT * Q_TILE;
  static constexpr int SLOT = TK * D * 2;
  static constexpr int kSoftmaxThreads = 256 * STREAMS;
  static constexpr int kThreads = 128 + kSoftmaxThreads;
  static constexpr int COL_O = BUFS * SW;
  static constexpr int X_BYTES = 2 * STREAMS * kRows * 4 * (JOIN ? 2 : 1);  // row statistics exchanged by warpgroups
  static constexpr int kMinV = 2;                                           // V slots at least, see wait_v
  // Items after which an accumulator is folded into fp32 sums in memory, 0: never. The tensor core cuts each sum it adds
  // to instead of rounding it, so an accumulator loses about 1.3e-8 of itself with every MMA; 512 keys keep that at the
  // size of fp32's own errors. (Output of 16 bits does not show it: 1e-4 after 128K keys.)
  static constexpr int FOLD = TERMS > 1 ? 512 / TK : 0;
  // Weights are 2^SHIFT e^(s - m) for a reference m of the row that may lag behind the largest score, by up to LAG (in log2
  // units). bf16 holds weights of any size. fp16's steps are never below 2^-24: there the reference is as low as its
  // largest value allows (weights up to 2^15), and follows scores that stay more than FALL below it down, by up to DEPTH
  // in all (the fp32 accumulator and row sum have that room). A step then leaves 2^-36 min(p, 2^FALL w) of a key, p the
  // row's and w the tile's largest weight; with LAG 8 and neither shift nor fall it was 2^-25 p, all of a key 17 nats
  // below a first token that takes most of the attention. What it costs (32 sequences of 2048, 64 nodes, head dim 128, in
  // a graph, with and without): scores of standard deviation 1 65.1 to 66.3 and 65.1 to 65.6 us, of 3 78 and 70, of 6 78
  // and 76.5. The shift is added in the exponent, whose rounding grows with it: scores of deviation 1 at head dim 64 come
  // out 3.6 to 4.9e-7 off instead of 2.6 to 3.3e-7. A multiplication after it (3.0 to 4.4e-7) takes up to 4% longer.
  static constexpr float SHIFT = FP16 ? 11.f : 0.f, LAG = FP16 ? 4.f : 8.f, FALL = FP16 ? 10.f : 0.f, DEPTH = 40.f;
  static_assert(!FP16 || SHIFT + LAG <= 15.f, "weights stay below fp16's largest value");
  static_assert(X_BYTES >= kAlignBatch * 4 && kThreads >= kAlignBatch, "");
  static_assert(MT <= STREAMS, "two row tiles need two accumulators");
  static_assert(COL_O + STREAMS * D <= kTmemCols, "S / P buffers and accumulators fit tensor memory");
  static_assert(TERMS >= 1 && TERMS <= 3 && kMinV >= AHEAD, "");
};

// Shared memory besides the ring: alignment, query buffers, barriers and tables, the plan.
template <class C>
size_t smem_fixed(int batch) {
  return 1024 + (size_t)C::Q_BYTES + kTables + C::X_BYTES + (((size_t)(batch + 2) * 4 + 63) & ~size_t(63));
}

template <class C>
__device__ __forceinline__ uint32_t idesc(int n, int b_mn) {
  return (1u << 4) | (C::FP16 ? 0u : (1u << 7) | (1u << 10)) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(kRows >> 4) << 24);
}
// The tensor-core instructions below are executed by a whole warp with the same operands; one elected lane issues them.
// (Operands are then known to be uniform; in a branch of one lane each would be moved to a uniform register first.)
// D[tmem] (+)= A * B^T, 16-bit inputs, fp32 accumulate; the descriptors of A and B share their high word.
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p, q;\n"
      ".reg .b64 a, b;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "setp.ne.b32 p, %5, 0;\n"
      "mov.b64 a, {%1, %3};\n"
      "mov.b64 b, {%2, %3};\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n"
      "}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(id), "r"(accumulate)
      : "memory");
}
// The same with A in tensor memory.
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p, q;\n"
      ".reg .b64 b;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "setp.ne.b32 p, %5, 0;\n"
      "mov.b64 b, {%2, %3};\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n"
      "}\n" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(hi), "r"(id), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_commit_elect(uint64_t* bar) {
  asm volatile(
      "{\n"
      ".reg .pred q;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n"
      "}\n" ::"r"(smem_u32(bar))
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
// K or V rows of one kv head: box {64 elements, rows, slices of 64, 1 head} at {0, row, slice, head}.
__device__ __forceinline__ void tma_kv_elect(uint32_t dst, const void* map, int row, int slice, int head, uint64_t* bar,
                                             uint64_t policy, bool once) {
  if (once)
    asm volatile(
        "{\n"
        ".reg .pred q;\n"
        "elect.sync _|q, 0xffffffff;\n"
        "@q cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
        "[%1, {%2, %3, %7, %4}], [%5], %6;\n"
        "}\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(head), "r"(smem_u32(bar)), "l"(policy), "r"(slice)
        : "memory");
  else
    asm volatile(
        "{\n"
        ".reg .pred q;\n"
        "elect.sync _|q, 0xffffffff;\n"
        "@q cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %6, %4}], [%5];\n"
        "}\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(head), "r"(smem_u32(bar)), "r"(slice)
        : "memory");
}
__device__ __forceinline__ void mbar_expect_elect(uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n"
      ".reg .pred q;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n"
      "}\n" ::"r"(smem_u32(bar)),
      "r"(bytes)
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

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n"
      ".reg .b64 a, b, c, d;\n"
      "mov.b64 a, {%2, %3};\n"
      "mov.b64 b, {%4, %5};\n"
      "mov.b64 c, {%6, %7};\n"
      "fma.rn.f32x2 d, a, b, c;\n"
      "mov.b64 {%0, %1}, d;\n"
      "}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n"
      ".reg .b64 a, b, d;\n"
      "mov.b64 a, {%2, %3};\n"
      "mov.b64 b, {%4, %5};\n"
      "add.rn.f32x2 d, a, b;\n"
      "mov.b64 {%0, %1}, d;\n"
      "}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Bits k = 0 .. 63: bit (o + k) of m, where bits before the first are 1 (committed tokens) and behind the last 0.
__device__ __forceinline__ uint64_t window(uint64_t m, int o) {
  if (o <= -64) return ~0ull;
  if (o < 0) return (m << -o) | ((1ull << -o) - 1);
  return o < 64 ? m >> o : 0ull;
}

// 32 bytes at once.
__device__ __forceinline__ void store32(void* at, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
// Write 16 consecutive columns of one output row (element offset `at`).
template <bool FP16>
__device__ __forceinline__ void store_row(const Params& p, int64_t at, const float* v) {
  uint32_t w[8];
  if (p.out_f32) {
    float* o = static_cast<float*>(p.out) + at;
#pragma unroll
    for (int c = 0; c < 16; c += 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[c + i]);
      if (p.out_wide) {
        store32(o + c, w);
      } else {
        reinterpret_cast<uint4*>(o + c)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(o + c)[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(p.out) + at;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack2<FP16>(v[2 * i], v[2 * i + 1]);
    if (p.out_wide) {
      store32(o, w);
    } else {
      reinterpret_cast<uint4*>(o)[0] = make_uint4(w[0], w[1], w[2], w[3]);
      reinterpret_cast<uint4*>(o)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

// Row r of row tile mt of unit u: its output offset, or -1 for a padding row.
__device__ __forceinline__ int64_t row_offset(const Params& p, int D, int MT, int b, int u, int mt, int r) {
  const int g = u / p.groups, rg = u - g * p.groups;
  const int i = (rg * MT + mt) * p.npt + r / p.gqa, j = r % p.gqa;
  if (r >= p.npt * p.gqa || i >= p.nodes) return -1;
  return (((int64_t)b * p.nodes + i) * p.heads + g * p.gqa + j) * D;
}

// Tiles per CTA. An even split cuts a unit at every CTA's border, and each cut unit is joined from its pieces. Where all
// units have the same length (unit_tiles > 0), whole units are taken instead if the busiest CTA then has at most kCutBytes
// of K (six tiles of 32 KB) more than the even split gives it. In a graph, inputs in L2 where they fit, whole and cut: one
// tile more (one sequence of 200) 14.9 and 18.5 us, five more (batch 32, 64 nodes) 65.5 and 77.4, seven more (one of 1000;
// 40 of 1024) 26.4 and 21.0; 74.6 and 68.1. Cuts are not limited to longer pieces: for short ragged sequences pieces of at
// least two tiles take 31 us, of three 34, of one 22.
// Where there are at most as many units as CTAs (`units`, the longest of `longest` tiles), pieces do not reach over a
// unit's end (`aligned`), under the same limit: a CTA with pieces of two units ends and joins twice. One sequence in a
// graph, reaching over and aligned: 3968 tokens 46.9 and 28.2 us, 8064 51.0 and 32.9, 16000 54.1 and 40.4; four of 8000
// 63.6 and 51.1. The plan for it costs the calls that do not need it up to 0.7 us.
template <class C>
__device__ __forceinline__ int tiles_per_cta(int T, int unit_tiles, int units, int longest, int grid, int batch, bool& aligned) {
  constexpr int kMore = kCutBytes / C::SLOT;
  const int even = (T + grid - 1) / grid;
  aligned = false;
  if (unit_tiles > 0) {
    const int whole = (T / unit_tiles + grid - 1) / grid * unit_tiles;
    if (whole <= even + kMore) return whole;
  }
  if (units <= grid && batch <= kAlignBatch) {  // (padded rows can make the batch larger than its units)
    int w = longest;  // then the pieces are at most T / w + units
    if (unit_tiles > 0) w = (longest + grid / units - 1) / (grid / units);
    else if (units < grid) w = min(w, (T + grid - units - 1) / (grid - units));
    if (w <= even + kMore) {
      aligned = w > 1 && (unit_tiles == 0 || unit_tiles % w != 0);  // else they end there anyway
      return w;
    }
  }
  return even;
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1) tree_attention_kernel(const Params p,
                                                                        const __grid_constant__ CUtensorMap tm_q,
                                                                        const __grid_constant__ CUtensorMap tm_k,
                                                                        const __grid_constant__ CUtensorMap tm_v) {
  constexpr int D = C::D, MT = C::MT, TK = C::TK, SW = C::SW, PW = C::PW, TERMS = C::TERMS, NB = C::NB, BUFS = C::BUFS;
  constexpr int kThreads = C::kThreads, kSoftmaxThreads = C::kSoftmaxThreads;
  constexpr bool JOIN = C::JOIN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int RK = p.kslots, RV = p.vslots, S = RK + RV;
  uint8_t* qbuf = smem;
  uint8_t* ring = qbuf + C::Q_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + S * C::SLOT);  // [RK of K, RV of V]: the slot's tile has landed
  uint64_t* empty = full + kMaxSlots;                                // [...]: its MMAs are done
  uint64_t* s_full = empty + kMaxSlots;  // [2]: S / P buffer x holds the scores of its item
  uint64_t* p_full = s_full + 2;         // [2]: its weights are written (one arrival per warp of the stream)
  uint64_t* pv_done = p_full + 2;        // [2]: the product that read them is complete
  uint64_t* q_full = pv_done + 2;
  uint64_t* q_empty = q_full + 1;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(q_empty + 1);
  int32_t* s_bad = reinterpret_cast<int32_t*>(s_tmem + 2);  // [8] per piece (seq & 7): a page id was bad
  int32_t* s_misc = s_bad + 8;                              // [24]: per warp, then the tile counts' range
  uint64_t* s_used = reinterpret_cast<uint64_t*>(s_misc + 24);  // [2 streams]
  int8_t* s_par = reinterpret_cast<int8_t*>(s_used + 2);        // [2 streams][64]
  static_assert(8 * (2 * kMaxSlots + 8) + 8 + 32 + 96 + 16 + 2 * 64 <= kTables, "the tables fit their area");
  float* s_x = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(full) + kTables);  // [warpgroups][128] (joined: twice)
  int32_t* s_prefix = reinterpret_cast<int32_t*>(reinterpret_cast<uint8_t*>(s_x) + C::X_BYTES);

  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
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
  int live;  // sequences with work, where B <= kThreads
  {
    const int per = (B + kThreads - 1) / kThreads;
    const int b0 = tid * per;
    int mine = 0, lo = INT32_MAX, hi = 0;
    if (tid == 0) {
      s_misc[22] = INT32_MAX;
      s_misc[23] = 0;
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
      atomicMin(&s_misc[22], lo);
      atomicMax(&s_misc[23], hi);
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
        mbar_init(&empty[s], 1);
      }
      for (int x = 0; x < 2; ++x) {
        mbar_init(&s_full[x], 1);
        mbar_init(&p_full[x], 8);
        mbar_init(&pv_done[x], 1);
      }
      mbar_init(q_full, 1);
      mbar_init(q_empty, 1);
      fence_mbar_init();
    }
    live = __syncthreads_count(mine > 0);
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
  const int T = s_prefix[B] * U;  // the host made sure that it fits
  if (T == 0) return;
  bool aligned;
  const int W = tiles_per_cta<C>(T, s_misc[22] == s_misc[23] ? s_misc[23] : 0, live * U, s_misc[23], (int)gridDim.x, B,
                                 aligned);
  int f0 = min(T, (int)blockIdx.x * W), f1 = min(T, f0 + W);
  if (aligned) {  // uniform over the grid; the prefix then counts whole pieces, B <= kAlignBatch
    const int nt = tid < B ? s_prefix[tid + 1] - s_prefix[tid] : 0, padded = (nt + W - 1) / W * W;
    int incl = padded;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    __syncthreads();  // the tile counts and s_misc are read
    if (lane == 31) s_misc[warp] = incl;
    __syncthreads();
    for (int w = 0; w < warp; ++w) incl += s_misc[w];
    int32_t* real = reinterpret_cast<int32_t*>(s_x);
    if (tid < B) {
      s_prefix[tid + 1] = incl;  // s_prefix[0] is 0
      real[tid] = nt;
    }
    __syncthreads();
    f0 = (int)blockIdx.x * W;
    if (f0 >= s_prefix[B] * U) return;
    const Cursor c = cursor_at(f0, s_prefix, B, U);
    f1 = f0 + min(W, real[c.b] - c.tile);  // a unit's last piece may be shorter
  }
  if (f0 >= f1) return;
  const int n_tiles = f1 - f0;

  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), kTmemCols);
    tmem_relinquish();
  }
  // padding rows of the query tiles (the copies write npt * gqa rows each)
  const int packed = p.npt * p.gqa;
  for (int i = tid; i < MT * C::SUBS * (kRows - packed) * 8; i += kThreads) {
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

  // Registers: 640 threads are launched with kLaunchRegs each; the warps that only issue copies and MMAs give some of
  // theirs to the softmax warps (5 * 96 = 64 + 4 * 104). Each role's branch has its own instruction: where branches
  // join, the compiler would hold all that follows to the smaller number.
  if (warp == 0) {
    // =================== producer: TMA ===================
    if constexpr (C::STREAMS == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
    // Tile j's K goes to slot j % RK of the K ring, its V to slot j % RV of the V ring, in the order in which they are
    // taken: the first AHEAD tiles' K, then V0 K(AHEAD), V1 K(AHEAD + 1), ...
    const int bs = 1 << p.page_shift;
    const int BH = bs < TK ? bs : TK;  // tokens of a copy: a page, or a tile of it
    const int pieces = TK / BH;
    // K and V that no other unit reads again (in a graph: head dim 256 480 us, 518 without; batch 32 65 and 69)
    const uint64_t pol = l2_evict_first_policy();
    // Two walks over the tiles, K's AHEAD tiles before V's. The lanes hold a window of 32 entries of the block table's row
    // as token rows; entries past the context and bad ones lie far outside the cache and read zeros.
    constexpr int kNowhere = -(1 << 20);
    struct Walk {
      Cursor c;
      int left, ctx, win_b, win_base, win_row, slot, phase;
      bool win_bad;
    };
    auto load_tile = [&](Walk& w, const CUtensorMap* map, int first, int depth) {  // into ring `first`
      const int t0 = w.c.tile * TK, n0 = t0 >> p.page_shift;
      if (w.c.b != w.win_b || n0 < w.win_base || n0 + pieces > w.win_base + 32) {
        w.win_b = w.c.b;
        w.win_base = n0;
        const bool in = n0 + lane < ((w.ctx + bs - 1) >> p.page_shift);
        const int page = in ? __ldg(p.block_table + (int64_t)w.c.b * p.max_blocks + n0 + lane) : 0;
        const bool ok = page >= 0 && (int64_t)page < p.num_blocks;
        w.win_row = in && ok ? page << p.page_shift : kNowhere;
        w.win_bad = __any_sync(0xffffffffu, in && !ok);
      }
      if (w.win_bad && lane == 0) s_bad[w.c.seq & 7] = 1;  // somewhere in the sequence: all of its rows are zeros
      if (w.phase > 0) wait(&empty[first + w.slot], w.phase - 1);
      if (!lost) {
        uint64_t* bar = &full[first + w.slot];
        mbar_expect_elect(bar, (uint32_t)C::SLOT);
        const uint32_t dst = ring_u32 + (first + w.slot) * C::SLOT;
        const int g = p.groups == 1 ? w.c.g : w.c.g / p.groups, in_page = t0 & (bs - 1);
#pragma unroll
        for (int i = 0; i < TK / 16; ++i)
          if (i < pieces) {
            const int row = __shfl_sync(0xffffffffu, w.win_row, n0 - w.win_base + i) + in_page;
            if (pieces == 1) {
              tma_kv_elect(dst, map, row, 0, g, bar, pol, p.groups == 1);  // all slices
            } else {
#pragma unroll
              for (int sub = 0; sub < C::SUBS; ++sub)
                tma_kv_elect(dst + sub * TK * 128 + i * BH * 128, map, row, sub, g, bar, pol, p.groups == 1);
            }
          }
      }
      if (++w.slot == depth) w.slot = 0, ++w.phase;
      if (--w.left == 0) {
        w.c.tile = w.c.ntiles - 1;
        cursor_advance(w.c, s_prefix, B, U);
        w.left = w.c.ntiles;
        if (w.c.b < B) w.ctx = p.ctx_lens[w.c.b];
      } else {
        ++w.c.tile;
      }
    };
    Walk wk;
    wk.c = cursor_at(f0, s_prefix, B, U);
    wk.left = wk.c.ntiles - wk.c.tile;
    wk.ctx = p.ctx_lens[wk.c.b];
    wk.win_b = -1;
    wk.win_base = wk.win_row = wk.slot = wk.phase = 0;
    wk.win_bad = false;
    Walk wv = wk;
    const int steps = __shfl_sync(0xffffffffu, n_tiles, 0);
    int fresh = -1;  // the last piece whose queries were asked for
#pragma unroll 1
    for (int j = 0; j < steps + C::AHEAD; ++j) {
      if (j >= C::AHEAD) load_tile(wv, &tm_v, RK, RV);
      if (j >= steps) continue;
      const Cursor c = wk.c;
      if (c.seq != fresh && lane == 0) s_bad[c.seq & 7] = 0;  // the piece eight before is long written
      __syncwarp();
      load_tile(wk, &tm_k, 0, RK);
      if (c.seq != fresh) {
        if (c.seq > 0) wait(q_empty, c.seq - 1);
        if (!lost && lane == 0) {
          const int n0 = (c.g % p.groups) * MT * p.npt;
          mbar_arrive_expect_tx(q_full, (uint32_t)(MT * packed * D * 2));
#pragma unroll 1
          for (int i = 0; i < MT * C::SUBS; ++i) {
            const int tile = i / C::SUBS, sub = i % C::SUBS;
            tma_load_4d(q_u32 + tile * C::Q_TILE + sub * kRows * 128, &tm_q, sub * 64, (c.g / p.groups) * p.gqa,
                        n0 + tile * p.npt, c.b, q_full);
          }
        }
        __syncwarp();
      }
      fresh = c.seq;
    }
    return;
  }

  if (warp == 1) {
    // =================== MMA issuer (one warp) ===================
    // Item j is tile j (one row tile) or row tile j & 1 of tile j >> 1 (two). Its S / P buffer is j & 1, its accumulator
    // the buffer's own, or the only one. The scores run two items ahead: those of item j + 2 follow the product of item
    // j, whose weights they overwrite (MMAs run in the order of their instructions), and while the softmax works on one
    // buffer, the tensor core works on the other.
    if constexpr (C::STREAMS == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
    {
      const uint32_t id_qk = idesc<C>(TK, 0), id_pv = idesc<C>(D, 1);
      // Descriptors differ in their low words only (start address / 16 in the low 14 bits).
      const uint64_t kmaj = smem_desc_sw128(0, 16, 1024);       // Q, K: rows of 64 elements, K-major
      const uint64_t vmn = smem_desc_sw128(0, TK * 128, 1024);  // V: MN-major, slices of 64 dims
      const uint32_t k_hi = (uint32_t)(kmaj >> 32), v_hi = (uint32_t)(vmn >> 32);
      const uint32_t q_lo = (uint32_t)kmaj + (q_u32 >> 4), k_lo = (uint32_t)kmaj + (ring_u32 >> 4);
      const uint32_t v_lo = (uint32_t)vmn + ((ring_u32 + RK * C::SLOT) >> 4);
      const int n_items = __shfl_sync(0xffffffffu, n_tiles, 0) * MT;
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      // scores: the next item, its tile's slot and phase, the tiles left in its unit
      Cursor cq = cursor_at(f0, s_prefix, B, U);
      int jq = 0, sk = 0, pk = 0, left_q = __shfl_sync(0xffffffffu, min(cq.ntiles - cq.tile, n_tiles), 0);
      bool q_fresh = true;
      int q_seq = 0;
      // products: the same, and the items of the unit so far
      Cursor cv = cq;
      int sv = 0, pv = 0, left_v = left_q, in_unit = 0;
      auto scores = [&]() {
        const int x = jq & 1, mt = MT == 2 ? x : 0;
        if (mt == 0) {
          if (q_fresh) wait(q_full, q_seq);
          wait(&full[sk], pk);
          tc_fence_after();
        }
        const uint32_t qb = q_lo + ((mt * C::Q_TILE) >> 4), kb = k_lo + sk * (C::SLOT >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t qo = ((ks >> 2) * kRows * 128 + (ks & 3) * 32) >> 4;
          const uint32_t ko = ((ks >> 2) * TK * 128 + (ks & 3) * 32) >> 4;
          umma_ss(tm + (uint32_t)(x * SW), qb + qo, kb + ko, k_hi, id_qk, ks > 0 ? 1u : 0u);
        }
        umma_commit_elect(&s_full[x]);
        if (mt == MT - 1) {
          umma_commit_elect(&empty[sk]);
          if (++sk == RK) sk = 0, ++pk;
          q_fresh = --left_q == 0;
          if (q_fresh) {
            umma_commit_elect(q_empty);
            cq.tile = cq.ntiles - 1;
            cursor_advance(cq, s_prefix, B, U);
            ++q_seq;
            left_q = __shfl_sync(0xffffffffu, cq.ntiles, 0);
          }
        }
        ++jq;
      };
#pragma unroll 1
      for (int i = 0; i < BUFS && jq < n_items; ++i) scores();
#pragma unroll 1
      for (int j = 0; j < n_items; ++j) {
        const int x = j & 1, mt = MT == 2 ? x : 0;
        if (mt == 0) wait(&full[RK + sv], pv);
        wait(&p_full[x], j >> 1);
        tc_fence_after();
        const uint32_t vb = v_lo + sv * (C::SLOT >> 4), d = tm + (uint32_t)(C::COL_O + (C::STREAMS == 2 ? x * D : 0));
        const int nth = in_unit / C::STREAMS;  // item of its stream in the unit
        const bool first = C::FOLD > 0 ? nth % (C::FOLD > 0 ? C::FOLD : 1) == 0 : nth == 0;  // the accumulator starts anew
        // The small parts of P first: each sum is cut relative to what the accumulator holds by then. Over six seeds the
        // error of 200 keys at head dim 128 is 5.3 to 5.7e-7 instead of 9.8 to 10.2e-7, in the same time.
#pragma unroll
        for (int term = TERMS - 1; term >= 0; --term)
#pragma unroll
          for (int kk = 0; kk < TK / 16; ++kk)
            umma_ts(d, tm + (uint32_t)(x * SW + term * PW + kk * 8), vb + ((kk * 2048) >> 4), v_hi, id_pv,
                    (first && term == TERMS - 1 && kk == 0) ? 0u : 1u);
        umma_commit_elect(&pv_done[x]);  // before the buffer's next scores, see wait_pv
        if (mt == MT - 1) umma_commit_elect(&empty[RK + sv]);
        if (jq < n_items) scores();
        ++in_unit;
        if (mt == MT - 1) {
          if (++sv == RV) sv = 0, ++pv;
          if (--left_v == 0) {
            cv.tile = cv.ntiles - 1;
            cursor_advance(cv, s_prefix, B, U);
            left_v = __shfl_sync(0xffffffffu, cv.ntiles, 0);
            in_unit = 0;
          }
        }
      }
    }
    __syncwarp();
    named_sync(kBarTail, 32 + kSoftmaxThreads);  // the softmax warps are done with tensor memory
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
    return;
  }
  if (warp < 4) {
    if constexpr (C::STREAMS == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
    return;
  }

  // =================== softmax / epilogue: one thread per row ===================
  if constexpr (C::STREAMS == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;\n");
  const int wg = (warp - 4) >> 2, h = wg >> 1, half = wg & 1;  // warpgroup; its stream and half of a tile's keys
  const int r = tid & 127;                                     // row of the row tile = tensor-memory lane
  const int st = tid & 255;                                    // with half * 128 + r the stream's threads, in some order
  const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
  const int bar = kBarStream + h;
  const int mt = MT == 2 ? h : 0;
  constexpr int CW = C::CW;
  const uint32_t t_o = tmem + (uint32_t)(C::COL_O + h * D) + lanes;  // the stream's accumulator
  // The slot of tile `tile`'s V, which has landed. The slot's tile before it was multiplied before the scores of this one
  // were issued (RV >= AHEAD), so the parity is unambiguous.
  auto wait_v = [&](int tile) -> int {
    const int s = RK + tile % RV;
    wait(&full[s], tile / RV);
    return s;
  };
  // The product of the stream's item i is complete. Its buffer's product before it was issued before the scores of
  // item i, and the next one needs weights of this stream: the parity is unambiguous.
  auto wait_pv = [&](int i) {
    wait(&pv_done[C::STREAMS == 2 ? h : i & 1], i / NB);
    tc_fence_after();
  };

  // Adds the stream's accumulator, which holds the products up to item `last`, to its sums in memory (`again`: they hold
  // earlier folds, relative to the reference m_fold), and leaves the result there, or in the accumulator (`back`). Each half
  // of the stream does half of the columns. The loads go out before the product is waited for, 64 columns at a time.
  auto fold = [&](float m_, float m_fold, bool again, bool back, int last) {
    constexpr int CH = D / 2 < 64 ? D / 2 : 64;
    float4* sums = p.folds + ((int64_t)blockIdx.x * C::STREAMS + h) * (D / 4) * kRows + r;
    const float e = again && m_fold > -INFINITY ? fast_exp2(m_fold - m_) : 0.f;
#pragma unroll 1
    for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += CH) {
      float4 a[CH / 4];
#pragma unroll
      for (int i = 0; i < CH / 4; ++i)
        a[i] = again && r < packed ? __ldcg(sums + (c / 4 + i) * kRows) : make_float4(0.f, 0.f, 0.f, 0.f);
      if (c == half * (D / 2)) wait_pv(last);
#pragma unroll
      for (int k = 0; k < CH; k += 16) {
        float o[16];
        tmem_ld16(t_o + c + k, o);
        tmem_wait_ld_regs<16>(o);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float4& s = a[k / 4 + i];
          s.x = o[4 * i] = fmaf(s.x, e, o[4 * i]);
          s.y = o[4 * i + 1] = fmaf(s.y, e, o[4 * i + 1]);
          s.z = o[4 * i + 2] = fmaf(s.z, e, o[4 * i + 2]);
          s.w = o[4 * i + 3] = fmaf(s.w, e, o[4 * i + 3]);
        }
        if (back) tmem_st16(t_o + c + k, o);
      }
      if (!back && r < packed) {
#pragma unroll
        for (int i = 0; i < CH / 4; ++i) __stcg(sums + (c / 4 + i) * kRows, a[i]);
      }
    }
    if (back) tmem_wait_st();
  };

  // Pieces of units that are cut, joined when the CTA is done: its first unit's and its last one's.
  struct Piece {
    int b, u, c0, nseg;
  } cut[2];
  int n_cut = 0;

  Cursor cu = cursor_at(f0, s_prefix, B, U);
  int done = 0;  // tiles of this CTA before the unit
  int item = 0;  // items of this stream before the current one
  int base = p.ctx_lens[cu.b] - N, base_next = base;  // committed tokens of the unit's sequence and of the next unit's
  for (int seq = 0; done < n_tiles; ++seq, base = base_next) {
    const int n = min(cu.ntiles - cu.tile, n_tiles - done);
    if (cu.g == U - 1 && done + n < n_tiles) {  // asked for here: the unit's tiles hide the latency
      Cursor nx = cu;
      nx.tile = nx.ntiles - 1;
      cursor_advance(nx, s_prefix, B, U);
      base_next = p.ctx_lens[nx.b] - N;
    }
    float m = -INFINITY, l = 0.f;  // reference (scaled scores, see SHIFT), the thread's share of the row's sum
    [[maybe_unused]] float m_top = -INFINITY;  // the largest reference so far
    bool tree_bad = false, dead = false, have_tree = false;
    uint64_t sees = 0;
    int mine = 0;  // items of this stream in the unit so far
    [[maybe_unused]] float m_fold = -INFINITY;  // the reference of the folded sums
    // the stream's first tile: every tile, or every other one of the CTA's
#pragma unroll 1
    for (int tt = JOIN ? ((done & 1) == h ? 0 : 1) : 0; tt < n; tt += JOIN ? 2 : 1, ++item, ++mine) {
      const int x = C::STREAMS == 2 ? h : item & 1;
      const uint32_t t_s = tmem + (uint32_t)(x * SW) + lanes;
      const int off = (cu.tile + tt) * TK - base;  // the tile's first key among the tree's
      const bool edge = off + TK > 0;              // the tile holds keys that not every row sees
      if (edge && !have_tree) {
        have_tree = true;
        int par = SPEC_TREE_ROOT;
        if (st < N) {
          par = __ldg(p.parents + (int64_t)cu.b * N + st);
          s_par[h * 64 + st] = (int8_t)max(-3, min(64, par));  // what is out of range stays a bad parent
        }
        named_sync(bar, 256);
        const bool bad = st < N && !tree::parent_ok(s_par + h * 64, st);
        const uint32_t word = __ballot_sync(0xffffffffu, st < N && par != SPEC_TREE_UNUSED);
        if (st == 0) reinterpret_cast<uint32_t*>(s_used + h)[0] = word;
        if (st == 32) reinterpret_cast<uint32_t*>(s_used + h)[1] = word;
        tree_bad = named_sync_or(bar, 256, bad);
        const int node = ((cu.g % p.groups) * MT + mt) * p.npt + r / p.gqa;
        if (r < packed && node < N) {
          sees = tree::ancestors(s_par + h * 64, node);
          dead = sees == 0;
        }
      }
      wait(&s_full[x], item / NB);
      tc_fence_after();
      float v[CW];
#pragma unroll
      for (int c = 0; c < CW / 16; ++c) tmem_ld16(t_s + half * CW + c * 16, *reinterpret_cast<float(*)[16]>(&v[c * 16]));
      tmem_wait_ld_regs<CW>(v);
      if (edge) {
        // V of slots that no row sees may hold anything: zeros, so that 0 weights give 0. With two row tiles both
        // streams write them, each before its own product.
        const uint64_t dead0 = ~window(s_used[h], off), dead1 = TK > 64 ? ~window(s_used[h], off + 64) : 0;
        if (dead0 | dead1) {
          uint8_t* vt = ring + wait_v(done + tt) * C::SLOT;
          for (int i = st; i < TK * (D / 8); i += 256) {
            const int key = i / (D / 8), ch = i % (D / 8);
            if (((key < 64 ? dead0 : dead1) >> (key & 63)) & 1)
              *reinterpret_cast<uint4*>(vt + (ch >> 3) * TK * 128 + key * 128 + (((ch & 7) ^ (key & 7)) << 4)) =
                  make_uint4(0, 0, 0, 0);
          }
        }
        const uint64_t w = window(sees, off + half * CW);
        const uint32_t w0 = (uint32_t)w, w1 = (uint32_t)(w >> 32);
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          if (!((w0 >> k) & 1)) v[k] = -INFINITY;
          if (CW > 32 && !((w1 >> k) & 1)) v[CW > 32 ? 32 + k : k] = -INFINITY;
        }
      }
      float mx;
      {
        float a[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = max3(v[i], v[8 + i], v[16 + i]);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = fmaxf(a[i], v[24 + i]);
#pragma unroll
        for (int k = 32; k < CW; k += 16)
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i] = max3(a[i], v[k + i], v[k + 8 + i]);
        mx = max3(max3(a[0], a[1], a[2]), max3(a[3], a[4], a[5]), fmaxf(a[6], a[7])) * p.scale_log2;
      }
      // Both halves of a row use one reference. The barrier also tells that both have read their scores, which the weights
      // overwrite.
      tc_fence_before();
      const bool any = named_sync_or(bar, 256, mx > m + C::LAG || (C::FALL > 0.f && mx < m - C::FALL && mx > -INFINITY));
      tc_fence_after();
      if (any) {
        s_x[wg * kRows + r] = mx;
        named_sync(bar, 256);
        mx = fmaxf(mx, s_x[(wg ^ 1) * kRows + r]);
        float to = mx > m + C::LAG ? mx : m;
        bool moved = true;
        if constexpr (C::FALL > 0.f) {
          if (mx < m - C::FALL && mx > -INFINITY) to = fmaxf(mx, m_top - C::DEPTH);
          m_top = fmaxf(m_top, to);
          moved = named_sync_or(bar, 256, to != m);  // not if it was one half that is low
        }
        const float a = to == m ? 1.f : m == -INFINITY ? 0.f : fast_exp2(m - to);
        m = to;
        l *= a;
        if (mine > 0 && moved) {  // the accumulator holds earlier tiles; each half of the stream rescales half of its columns
          wait_pv(item - 1);
#pragma unroll 1
          for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 16) {
            float o[16];
            tmem_ld16(t_o + c, o);
            tmem_wait_ld_regs<16>(o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= a;
            tmem_st16(t_o + c, o);
          }
        }
      }
      const float ms = (m == -INFINITY ? 0.f : m) - C::SHIFT;
      const float2 sc = make_float2(p.scale_log2, p.scale_log2), mm = make_float2(-ms, -ms);
      float2 l0 = make_float2(0.f, 0.f), l1 = l0;
#pragma unroll
      for (int c = 0; c < CW; c += 32) {
#pragma unroll
        for (int i = c; i < c + 32; i += 4) {
          const float2 e0 = fma2(make_float2(v[i], v[i + 1]), sc, mm), e1 = fma2(make_float2(v[i + 2], v[i + 3]), sc, mm);
          v[i] = fast_exp2(e0.x);
          v[i + 1] = fast_exp2(e0.y);
          v[i + 2] = fast_exp2(e1.x);
          v[i + 3] = fast_exp2(e1.y);
          l0 = add2(l0, make_float2(v[i], v[i + 1]));
          l1 = add2(l1, make_float2(v[i + 2], v[i + 3]));
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
          tmem_st16u(t_s + term * PW + (half * CW + c) / 2, w);
        }
      }
      l0 = add2(l0, l1);
      l += l0.x + l0.y;
      tmem_wait_st();
      if constexpr (C::FOLD > 0) {
        if (mine > 0 && mine % C::FOLD == 0) {  // this item's product starts the accumulator anew
          fold(m, m_fold, mine > C::FOLD, false, item - 1);
          m_fold = m;
        }
      }
      if (edge) fence_proxy_async_smem();  // zeroed rows of V
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[x]);
    }

    // ---- the unit's rows: output, or a normalised partial and its log-sum-exp
    bool whole = cu.tile == 0 && n == cu.ntiles;
    int slot = 0, c0 = 0, nseg = 1;
    if (!whole) {
      const int u0 = s_prefix[cu.b] * U + cu.g * cu.ntiles;
      c0 = u0 / W;
      nseg = (u0 + cu.ntiles - 1) / W - c0 + 1;
      whole = nseg == 1;  // one piece, padded
      if (!whole) {
        slot = piece_slot((int)blockIdx.x, c0, u0, W);
        cut[n_cut++] = Piece{cu.b, cu.g, c0, nseg};
      }
    }
    if (mine > 0) wait_pv(item - 1);
    if constexpr (C::FOLD > 0) {
      if (mine > C::FOLD) fold(m, m_fold, true, true, item - 1);
    }
    if (tree_bad && st == 0) raise_error(p.dev_err, SPEC_DEVERR_TREE);
    if (tree_bad || dead) l = -1.f;  // no result: the row is zeros, whatever its scores were
    // Threads of a row: the two halves of its stream; with one row tile on two streams all four, which then write a
    // quarter of the columns of both accumulators' sum each.
    float L, M = m, f[2] = {1.f, 0.f};  // factors of the accumulators
    bool none;
    s_x[wg * kRows + r] = l;
    if (JOIN) s_x[(4 + wg) * kRows + r] = m;
    tc_fence_before();
    if (JOIN) named_sync(kBarSoftmax, kSoftmaxThreads);
    else named_sync(bar, 256);
    tc_fence_after();
    if constexpr (JOIN) {
      const float m0 = s_x[4 * kRows + r], m1 = s_x[6 * kRows + r];
      M = fmaxf(m0, m1);
      f[0] = m0 == -INFINITY ? 0.f : fast_exp2(m0 - M);
      f[1] = m1 == -INFINITY ? 0.f : fast_exp2(m1 - M);
      const float l0 = s_x[r], l1 = s_x[kRows + r], l2 = s_x[2 * kRows + r], l3 = s_x[3 * kRows + r];
      L = (l0 + l1) * f[0] + (l2 + l3) * f[1];
      none = l0 < 0.f || l1 < 0.f || l2 < 0.f || l3 < 0.f;
    } else {
      const float l0 = s_x[2 * h * kRows + r], l1 = s_x[(2 * h + 1) * kRows + r];
      L = l0 + l1;
      none = l0 < 0.f || l1 < 0.f;
    }
    // read here: a stream without a tile of the unit knows only now that the unit was loaded
    const bool bad = s_bad[seq & 7] != 0;
    if (bad && tid == 128) raise_error(p.dev_err, SPEC_DEVERR_BLOCK_ID);
    none |= bad;
    const bool some = !none && L != 0.f;  // a NaN makes the row NaN, by its factor
    const float inv = some ? 1.f / L : 0.f;
    f[0] *= inv;
    f[1] *= inv;
    const int64_t row = row_offset(p, D, MT, cu.b, cu.g, mt, r);
    constexpr int COLS = JOIN ? D / 4 : D / 2;  // columns of a thread
    const int part = JOIN ? wg : half;
    if (!whole && part == 0)
      p.lse[((int64_t)slot * MT + mt) * kRows + r] = some ? M + __log2f(L) : none ? INFINITY : -INFINITY;
    const uint32_t t_acc = JOIN ? tmem + (uint32_t)C::COL_O + lanes : t_o;
    // an accumulator that got no tile of the unit holds anything
    const bool has0 = !JOIN || (done & 1) == 0 || n > 1, has1 = JOIN && ((done & 1) == 1 || n > 1);
#pragma unroll
    for (int c = part * COLS; c < (part + 1) * COLS; c += 16) {
      float o[16], o1[16];
      if (has0) tmem_ld16(t_acc + c, o);
      if (has1) tmem_ld16(t_acc + D + c, o1);
      tmem_wait_ld_regs<16>(o);
      if (has1) tmem_wait_ld_regs<16>(o1);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float a = has0 ? o[i] * f[0] : 0.f;
        if (has1) a = fmaf(o1[i], f[1], a);
        o[i] = some ? a : 0.f;
      }
      if (whole) {
        if (row >= 0) store_row<C::FP16>(p, row + c, o);
      } else {
        float4* dst = p.opart + (((int64_t)slot * MT + mt) * (D / 4) + c / 4) * kRows + r;
#pragma unroll
        for (int i = 0; i < 4; ++i) dst[i * kRows] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
      }
    }
    // The next unit's first product waits for weights of every warp of its stream. With a join the other stream reads
    // this one's accumulator and statistics too.
    if constexpr (JOIN) {
      tc_fence_before();
      named_sync(kBarSoftmax, kSoftmaxThreads);
      tc_fence_after();
    }
    done += n;
    cu.tile += n - 1;
    cursor_advance(cu, s_prefix, B, U);
  }
  tc_fence_before();
  named_sync(kBarTail, 32 + kSoftmaxThreads);

  // ---- join the pieces of cut units, kRadix neighbouring runs of pieces at a time: the CTA that comes last joins them, in
  // the order of the pieces,
  //   out = sum w_k part_k / sum w_k, w_k = 2^(lse_k - max lse),
  // and goes on with the longer run; nobody waits. A group's counter is that of the border CTA behind its first run: borders
  // 1 mod kRadix on the first level, kRadix mod kRadix^2 on the second, and so on; no two groups share one. Each level costs
  // a fence, an atomic and a round trip; one CTA reads what it joins. Radix 2, 4, 8, 16, 32 in a graph: one sequence of 8000
  // 64.6, 54.6, 52.6, 57.5, 53.9 us; of 2000 at head dim 256 42.9, 37.6, 34.9, 45.0, 52.4; the largest batch at head dim
  // 256 479, 481, 482, 482, 482.
  constexpr int COLS = JOIN ? D / 4 : D / 2;
  const int part = JOIN ? wg : half;
  for (int k = 0; k < n_cut; ++k) {
    const Piece c = cut[k];
    const int u0 = s_prefix[c.b] * U + c.u * (s_prefix[c.b + 1] - s_prefix[c.b]);
    const int64_t row = row_offset(p, D, MT, c.b, c.u, mt, r);
    auto slot_of = [&](int piece) -> int64_t {  // in units of 128 rows
      return (int64_t)(piece == 0 ? piece_slot(c.c0, c.c0, u0, W) : 2 * (c.c0 + piece)) * MT + mt;
    };
    int me = (int)blockIdx.x - c.c0;
    for (int run = 1; run < c.nseg; run *= kRadix) {
      const int left = me / (kRadix * run) * (kRadix * run), runs = min(kRadix, (c.nseg - left + run - 1) / run);
      if (runs == 1) continue;                   // no neighbour on this level
      named_sync(kBarSoftmax, kSoftmaxThreads);  // the run's stores are issued, s_misc is read
      if (tid == 128) {
        int32_t* met = p.counters + c.c0 + left + run;
        __threadfence();
        const int before = atomicAdd(met, 1);
        if (before == runs - 1) *met = 0;
        __threadfence();
        s_misc[0] = before;
      }
      named_sync(kBarSoftmax, kSoftmaxThreads);
      if (s_misc[0] != runs - 1) break;
      me = left;
      const bool last = left == 0 && kRadix * run >= c.nseg;
      auto lse_at = [&](int i) { return p.lse + slot_of(left + i * run) * kRows + r; };
      float M = -INFINITY, sum = 0.f;
      bool none = false, nan = false;
#pragma unroll 8
      for (int i = 0; i < runs; ++i) {
        const float x = __ldcg(lse_at(i));
        none |= x == INFINITY;
        nan |= x != x;
        M = fmaxf(M, x);
      }
      const bool some = !none && (M > -INFINITY || nan);
#pragma unroll 8
      for (int i = 0; i < runs; ++i) sum += some ? fast_exp2(__ldcg(lse_at(i)) - M) : 0.f;
      const float inv = some ? 1.f / sum : 0.f;
#pragma unroll 1
      for (int q = part * COLS; q < (part + 1) * COLS; q += 16) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0.f;
#pragma unroll 4
        for (int i = 0; i < runs; ++i) {
          const float w = some ? fast_exp2(__ldcg(lse_at(i)) - M) * inv : 0.f;
          const float4* a = p.opart + (slot_of(left + i * run) * (D / 4) + q / 4) * kRows + r;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 x = __ldcg(a + e * kRows);
            v[4 * e] = fmaf(x.x, w, v[4 * e]);
            v[4 * e + 1] = fmaf(x.y, w, v[4 * e + 1]);
            v[4 * e + 2] = fmaf(x.z, w, v[4 * e + 2]);
            v[4 * e + 3] = fmaf(x.w, w, v[4 * e + 3]);
          }
        }
        if (!some) {  // (parts of a row without a result may be NaN)
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = 0.f;
        }
        if (last) {
          if (row >= 0) store_row<C::FP16>(p, row + q, v);
        } else {
          float4* to = p.opart + (slot_of(left) * (D / 4) + q / 4) * kRows + r;
#pragma unroll
          for (int e = 0; e < 4; ++e) __stcg(to + e * kRows, make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]));
        }
      }
      if (!last) {
        named_sync(kBarSoftmax, kSoftmaxThreads);  // everyone has read the runs' lse
        if (part == 0) __stcg(lse_at(0), some ? M + __log2f(sum) : none ? INFINITY : -INFINITY);
      }
    }
  }
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
template <int D>
int settings(int mt, int terms, bool fp16, int batch, Launch* l);
template <int D>
int launch(int mt, int terms, bool fp16, const Launch& l, const Call& c);

}  // namespace tattn
}  // namespace specv
