// Kernel of the attention over a window of a paged cache, 16-bit or 4-bit (see
// the comment at the top of window_attention.cu), and its parameters, shared with
// the host side.
#pragma once

#include <cuda.h>

#include "attention_tc.cuh"
#include "q4_device.cuh"
#include "tree_attention.cuh"

namespace specv {
namespace wattn {

using attn::tc::reduce_cols;
using attn::tc::reduced_col;
using attn::tc::tmem_load_cols;
using attn::tc::tmem_store_cols;
using tattn::umma_commit_elect;

constexpr int TK = 128;            // keys per tile (MMA M)
constexpr int kMaxBatch = 4096;
constexpr int kMaxRows = 64;       // packed query rows of a unit
constexpr int kMaxPieces = 768;    // pieces of cut units in a call
constexpr int kMaxSlots = 16;      // K and V tiles in shared memory
constexpr int kCandidates = 32;
constexpr int kPageSlots = 8;      // 4-bit: tiles whose pages, s and m are in shared memory
constexpr uint32_t kMaxTries = 500000;  // of a wait, 2 s
constexpr int kBarEpi = 1, kBarEnd = 2, kBarV = 3, kBarGroup0 = 5;  // named barriers: the epilogue's warps, all at the end,
                                                           // those that unpack V, each softmax warpgroup
constexpr float kUnseen = -3e38f;  // reference of a row that has seen no key
static_assert(kMaxPieces / 2 * 4 <= SPEC_ATTN_COUNTER_BYTES, "a counter for every cut unit");

struct Params {
  const uint8_t* q;
  uint8_t* out;
  const uint8_t* kpar;  // 4-bit: where a token's s and m begin
  const uint8_t* vpar;
  const int32_t* block_table;
  const int32_t* ctx_lens;
  int32_t* counters;  // [kMaxPieces / 2], zero between calls
  float* lse;         // [kMaxPieces][kMaxRows], log2 units; +inf: no result
  float* opart;       // [kMaxPieces][N][D], normalised
  int32_t* dev_err;
  int64_t num_blocks, row;  // pages; bytes of a 4-bit token row
  int batch, rows, heads, kv_heads, gqa;
  int by_gqa;       // 2^16 / gqa, rounded up: r / gqa = r * by_gqa >> 16 for r < 64
  int npt, groups;  // query rows of a unit (its npt * gqa packed rows), units per kv head
  int page_shift, max_blocks, window, sinks;
  int slots;  // tiles (or parts of one) that fit the ring
  int fp16;   // type of q and out (4-bit: and of s and m)
  float scale_log2;
};

template <int D_, int ROWS_, bool Q4_, bool FP16_>
struct Cfg {
  static constexpr int D = D_, ROWS = ROWS_;  // packed rows of a unit, at most
  static constexpr bool Q4 = Q4_;
  static constexpr bool FP16 = FP16_;         // type of the MMA operands (4-bit: always fp16)
  static constexpr int N = ROWS < 16 ? 16 : ROWS;
  // Softmax: ST streams, which take the tiles in turns and have an accumulator, references and sums of their own (a tile
  // is a long chain of steps for its warps), with NG warpgroups each, ROWS / NG rows of a tile.
  static constexpr int UG = ROWS <= 32 ? 2 : 1;  // 4-bit: groups of four warps that unpack K (and V), taking the tiles in turns
  static constexpr int ST = Q4 && ROWS <= 16 ? 2 : 1;
  static constexpr int NG = ROWS <= 16 ? 1 : ROWS / 16;
  static constexpr int CW = ROWS / NG;
  static constexpr int CHUNK = CW > 8 && Q4 && ROWS > 16 ? 8 : CW;  // scores that a softmax thread holds at once (registers)
  static constexpr int HALVES = D == 256 ? 2 : 1;  // O^T accumulators of 128 lanes
  // A 16-bit fp16 weight keeps its bits between 2^15 and 2^-14 only: two bands of weights, the lower one times 2^18, with
  // an accumulator each, cover 2^15 to 2^-32. (4-bit: the reference takes the values' scale along, see softmax.)
  static constexpr int BANDS = FP16 && !Q4 ? 2 : 1;
  static constexpr int QB = D == 256 && N == 64 ? 1 : 2;           // query buffers
  static constexpr int NP = D == 256 && N == 64 && BANDS == 2 ? 1 : 2;  // P buffers
  static constexpr int VB = D == 256 && N == 64 ? 1 : 2;           // 4-bit: unpacked V tiles in tensor memory (K: 2)
  static constexpr int OPERANDS = Q4 ? 2 * (D / 4) + VB * HALVES * (TK / 2) : 0;
  static constexpr int O_COLS = BANDS * HALVES * N;                 // of a stream
  static constexpr int SB = 2 * ST;                                // scores of tiles
  static constexpr int OB = OPERANDS + SB * N + 2 * ST * O_COLS <= 512 ? 2 : 1;  // tasks whose accumulators there is room for
  static constexpr int COL_K = 0, COL_V = Q4 ? 2 * (D / 4) : 0, COL_S = OPERANDS, COL_O = COL_S + SB * N;
  static constexpr int COLS = COL_O + OB * ST * O_COLS;
  static constexpr int ALLOC = COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  static_assert(COLS <= 512, "tensor memory");
  // Tiles in shared memory; those of head dim 256 in two parts of 128 head dims (16-bit).
  static constexpr int PARTS = D == 256 && !Q4 ? 2 : 1;
  static constexpr int SLOT = Q4 ? TK * D / 2 : TK * D * 2 / PARTS;
  // 4-bit: tiles that a group copies ahead; its ring holds one more.
  static constexpr int AHEAD = D == 256 ? 3 / UG : UG == 2 ? 3 : 5;
  static constexpr int RINGS = 2 * UG * (AHEAD + 1);
  // Queries: rows of 64 16-bit elements, D / 64 slices. 4-bit: of 128 8-bit ones, in three parts that add up to them.
  static constexpr int Q_SLICES = D == 256 ? 2 : 1, Q_PART = Q_SLICES * N * 128;
  static constexpr int Q_BYTES = Q4 ? 3 * Q_PART : N * D * 2;
  static constexpr int P_BYTES = N * TK * 2;
  // P is the operand B of the second product, MN-major: the N rows of a key are contiguous and swizzled at that width.
  static constexpr uint32_t P_LAYOUT = N == 16 ? 6u : (N == 32 ? 4u : 2u);
  static constexpr int P_SWZ_SHIFT = N == 16 ? 2 : (N == 32 ? 1 : 0);
  static constexpr int P_SWZ_MASK = N == 16 ? 1 : (N == 32 ? 3 : 7);
  static constexpr int W_EPI = 4, W_SOFT = 8, W_K = W_SOFT + 4 * NG * ST, W_V = W_K + 4 * UG;  // first warps of the roles
  static constexpr int kWarps = Q4 ? W_V + 4 * UG : W_K;
  static constexpr int kThreads = 32 * kWarps;
  // Registers a thread of the softmax and of the other roles, where they are dealt out anew: 32 warps are launched with 64.
  static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;
  static constexpr int kOtherRegs = 48, kSoftRegs = NG * ST == 4 ? 80 : NG * ST == 2 ? 112 : 160;
  static constexpr bool DEAL = Q4;
  static_assert(!DEAL || 4 * NG * ST * kSoftRegs + (kWarps - 4 * NG * ST) * kOtherRegs <= kWarps * kLaunchRegs, "registers");
  static_assert(!Q4 || kWarps == 32, "");
  static_assert(ST == 1 || NP == 2, "a stream has a P buffer of its own");
  static constexpr int V_WARPS = D / 32 < 4 ? D / 32 : 4;  // 4-bit: warps that unpack V, 32 head dims each (and a half)
  // What a task's start and end, a join, and a piece of it cost, in tiles (us over the us of a tile at the measured copy
  // bandwidth, 45 KB a us for each SM, but 0.35 us at least).
  static constexpr float TILE_US = 2.f * PARTS * SLOT / 45000.f > 0.35f ? 2.f * PARTS * SLOT / 45000.f : 0.35f;
  static constexpr float TASK_COST = 1.f / TILE_US, JOIN_COST = 2.f / TILE_US, PIECE_COST = 0.15f / TILE_US;
  // Weights are 2^SHIFT at the largest of the tile that set a row's reference, TOP at most.
  static constexpr float SHIFT = 7.f, TOP = 32768.f;
  static constexpr float TINY = 0x1p-60f;  // 4-bit: the smallest s that the reference follows
};

// Shared memory besides the ring, in order.
template <class C>
struct Smem {
  static constexpr int Q = 0;
  static constexpr int P = Q + C::QB * C::Q_BYTES;
  static constexpr int BARS = P + C::NP * C::BANDS * C::P_BYTES;  // 96 mbarriers
  static constexpr int REF = BARS + 96 * 8;                       // [ST][64] minus the reference of each row
  static constexpr int ALPHA = REF + C::ST * 256;                 // [ST][64]
  static constexpr int RED = ALPHA + C::ST * 256;                 // [ST][4][64]
  static constexpr int STAT = RED + C::ST * 1024;                 // [OB][ST]: [4][64] sums, [4][64] offsets, [64] reference
  static constexpr int STAT_BYTES = 2048 + 256;
  static constexpr int QC = STAT + C::OB * C::ST * STAT_BYTES;    // [QB][2][64] factors of the scores
  static constexpr int PAGES = QC + C::QB * 512;                  // [kPageSlots]: [8] pages of a tile, kv head
  static constexpr int PAR = PAGES + (C::Q4 ? kPageSlots * 48 : 0);    // [kPageSlots][2][128] s and m of K and V
  static constexpr int EPI = PAR + (C::Q4 ? kPageSlots * 1024 : 0);   // [64] int64 and three times [64] floats of the epilogue
  static constexpr int MISC = EPI + 1280;  // [64] plan, tensor-memory base, flags
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
// The same with A in tensor memory, of 16-bit elements or of e4m3.
template <bool F8>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t id, uint32_t accumulate) {
  if constexpr (F8)
    asm volatile(
        "{\n"
        ".reg .pred p, q;\n"
        ".reg .b64 b;\n"
        "elect.sync _|q, 0xffffffff;\n"
        "setp.ne.b32 p, %5, 0;\n"
        "mov.b64 b, {%2, %3};\n"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], b, %4, p;\n"
        "}\n" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(b_hi), "r"(id), "r"(accumulate)
        : "memory");
  else
    tattn::umma_ts(d, a, b_lo, b_hi, id, accumulate);
}
template <bool FP16>
__device__ __forceinline__ constexpr uint32_t mma_desc(int n, int a_mn, int b_mn) {
  return (1u << 4) | (FP16 ? 0u : (1u << 7) | (1u << 10)) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(TK >> 4) << 24);
}
__device__ __forceinline__ constexpr uint32_t mma_desc_e4m3(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(TK >> 4) << 24); }
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
// 16 lanes x 4 columns a pair of registers: thread l holds lane l / 4 (first of the pair) and l / 4 + 8 of column l % 4.
__device__ __forceinline__ void tmem_st_16x128_x4(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// 4 bytes from global to shared memory, zeros with bytes = 0; the barrier gets one arrival of this thread once all its
// copies so far are there.
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
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
// Barriers by their shared-memory address.
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(bytes) : "memory");
}
// Waits for the phase of this parity, `tries` times at most; if they run out, 1 is left of them, which says so and makes
// later waits short. A try sleeps for up to 4 us (7819 cycles measured; 1942 without the hint). Few instructions: the
// roles' loops together have to fit the instruction cache.
__device__ __forceinline__ void bar_wait(uint32_t bar, uint32_t parity, uint32_t& tries) {
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      ".reg .u32 n;\n"
      "mov.u32 n, %0;\n"
      "TRY:\n"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000000;\n"
      "@p bra DONE;\n"
      "sub.u32 n, n, 1;\n"
      "setp.ne.u32 p, n, 0;\n"
      "@p bra TRY;\n"
      "mov.u32 %0, 1;\n"
      "DONE:\n"
      "}\n"
      : "+r"(tries)
      : "r"(bar), "r"(parity)
      : "memory");
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
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  const __half2 r = __hadd2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Pairs of fp32 in one register pair.
__device__ __forceinline__ uint64_t pack_f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack_f2(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma_f2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul_f2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add_f2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Four fp32 as e4m3, the first in the low byte; what they lack of the originals is left in x.
__device__ __forceinline__ uint32_t take_e4m3(float (&x)[4]) {
  uint32_t r;
  asm("{\n"
      ".reg .b16 a, b;\n"
      "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n"
      "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n"
      "mov.b32 %0, {a, b};\n"
      "}\n"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t f;  // two fp16
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(f) : "h"((uint16_t)(r >> (16 * h))));
    const float2 v = q4::unpack2<true>(f);
    x[2 * h] -= v.x;
    x[2 * h + 1] -= v.y;
  }
  return r;
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// ---------------------------------------------------------------------------
// The plan: which tiles of which unit a block works on
// ---------------------------------------------------------------------------
// The pages that some row of a sequence sees: the first ns, and those from wp on; `pages` in all.
struct Span {
  int ns, wp, pages;
};
__device__ __forceinline__ Span span_of(const Params& p, int ctx) {
  const int np = (ctx + (1 << p.page_shift) - 1) >> p.page_shift;
  Span s = {0, 0, np};
  if (p.window != 0) {
    s.ns = min((p.sinks + (1 << p.page_shift) - 1) >> p.page_shift, np);
    s.wp = min(max(s.ns, max(0, ctx - p.rows - p.window + 1) >> p.page_shift), np);
    s.pages = s.ns + np - s.wp;
  }
  return s;
}
__device__ __forceinline__ bool ctx_ok(const Params& p, int ctx) {
  return ctx >= p.rows && (int64_t)ctx <= ((int64_t)p.max_blocks << p.page_shift);
}
__device__ __forceinline__ int tiles_of(const Params& p, int ctx) {  // 0: nothing to do
  if (!ctx_ok(p, ctx)) return 0;
  const int ppt = TK >> p.page_shift;
  return (span_of(p, ctx).pages + ppt - 1) / ppt;
}

// A task: a unit (sequence b, kv head g, query rows from i0 on), or one of the pieces that it was cut into.
struct Task {
  int b, g, i0, nr;      // nr: packed rows
  int tile0, tiles;      // its tiles of the unit's
  int pieces, first;     // pieces of the unit, slot of its first one
  int slot;              // its own
  int ctx;
  Span span;
};
// Tasks are numbered by sequence, piece, kv head and group, so that the blocks of a wave read the same tokens for all
// heads at about the same time: a line of a 4-bit token row holds several heads.
__device__ __forceinline__ Task task_at(const Params& p, const int32_t* prefix, const uint16_t* cut, int t) {
  int lo = 0, hi = p.batch;  // the last b with prefix[b] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= t) lo = mid; else hi = mid;
  }
  Task k;
  k.b = lo;
  const int units = p.kv_heads * p.groups;
  k.pieces = (prefix[lo + 1] - prefix[lo]) / units;
  const int r = t - prefix[lo], piece = r / units, unit = r - piece * units;
  k.g = unit / p.groups;
  k.i0 = (unit - k.g * p.groups) * p.npt;
  k.nr = min(p.npt, p.rows - k.i0) * p.gqa;
  k.ctx = p.ctx_lens[lo];
  k.span = span_of(p, k.ctx);
  const int ppt = TK >> p.page_shift, all = (k.span.pages + ppt - 1) / ppt;
  const int base = all / k.pieces, rest = all - base * k.pieces;
  k.tile0 = piece * base + min(piece, rest);
  k.tiles = base + (piece < rest ? 1 : 0);
  k.first = k.pieces > 1 ? (int)cut[lo] + unit * k.pieces : 0;
  k.slot = k.first + piece;
  return k;
}

// Length of the pieces. A block does ceil(tasks / blocks) tasks, one after the other; a task costs its tiles and
// something for its start and end, and cut units have to be joined. 32 lengths (no cut at all, and sixteenths of an even
// share) are tried, and the cheapest is taken.
template <class C>
__device__ __forceinline__ void make_plan(const Params& p, int32_t* prefix, uint16_t* cut, int32_t* misc) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = p.batch, units = p.kv_heads * p.groups, grid = (int)gridDim.x;
  float* cost = reinterpret_cast<float*>(misc) + 16;  // [kCandidates]
  if (tid < 2) misc[tid] = 0;  // all tiles, longest unit
  __syncthreads();
  {
    int sum = 0, most = 0;
#pragma unroll 1
    for (int b = tid; b < B; b += C::kThreads) {
      const int t = tiles_of(p, p.ctx_lens[b]);
      prefix[b] = t;  // until the prefix sums are made
      sum += t;
      most = max(most, t);
    }
    sum = __reduce_add_sync(0xffffffffu, sum);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0 && most > 0) {
      atomicAdd(&misc[0], sum);
      atomicMax(&misc[1], most);
    }
  }
  __syncthreads();
  const int longest = misc[1];
  const float share = (float)misc[0] * (float)units / (float)grid;
  auto length = [&](int c) { return c == 0 ? longest : max(1, min(longest, (int)ceilf(share * (float)c * (1.f / 16.f)))); };
  if (longest > 0) {
#pragma unroll 1
    for (int c = warp; c < kCandidates; c += C::kWarps) {
      const int len = length(c);
      int tasks = 0, pieces = 0, top = 0, parts = 1;
#pragma unroll 1
      for (int b = lane; b < B; b += 32) {
        const int t = prefix[b];
        if (t == 0) continue;
        const int k = (t + len - 1) / len;
        tasks += k;
        pieces += k > 1 ? k : 0;
        top = max(top, (t + k - 1) / k);
        parts = max(parts, k);
      }
      tasks = __reduce_add_sync(0xffffffffu, tasks);
      pieces = __reduce_add_sync(0xffffffffu, pieces);
      top = __reduce_max_sync(0xffffffffu, top);
      parts = __reduce_max_sync(0xffffffffu, parts);
      const float waves = ceilf((float)tasks * (float)units / (float)grid);
      float x = waves * ((float)top + C::TASK_COST) + (parts > 1 ? C::JOIN_COST + C::PIECE_COST * (float)parts : 0.f);
      if ((float)pieces * (float)units > (float)kMaxPieces) x = INFINITY;
      if (lane == 0) cost[c] = x;
    }
  }
  __syncthreads();
  if (warp == 0) {
    int best = 0;
#pragma unroll 1
    for (int c = 1; c < kCandidates && longest > 0; ++c)
      if (cost[c] < cost[best]) best = c;
    const int len = max(1, length(best));
    int tasks = 0, pieces = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < B; b0 += 32) {
      const int b = b0 + lane;
      const int t = b < B ? prefix[b] : 0;
      const int k = (t + len - 1) / len, kc = k > 1 ? k : 0;
      int a = k * units, c = kc * units;  // scans
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int ua = __shfl_up_sync(0xffffffffu, a, o), uc = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) {
          a += ua;
          c += uc;
        }
      }
      if (b < B) {
        prefix[b] = tasks + a - k * units;
        cut[b] = (uint16_t)(pieces + c - kc * units);
      }
      tasks += __shfl_sync(0xffffffffu, a, 31);
      pieces += __shfl_sync(0xffffffffu, c, 31);
    }
    if (lane == 0) prefix[B] = tasks;
  }
  __syncthreads();
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
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // 16-bit: KS slots for K, the others for V, so that a barrier's phases are all waited for by one warp, in turn (the
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
  const uint32_t kd_full = q_full + 16, kd_free = kd_full + 16;  // [KB] 4-bit: K unpacked
  const uint32_t vd_full = kd_free + 16, vd_free = vd_full + 16;  // [KB]
  const uint32_t s_full = vd_free + 16;    // [SB] scores of a tile
  const uint32_t s_free = s_full + 32;     // [SB] and their buffer may be written again
  const uint32_t p_full = s_free + 32;     // [2] weights of a tile written
  const uint32_t pv_done = p_full + 16;    // [NP] second product of the tile that used the P buffer is complete
  const uint32_t o_full = pv_done + 16;    // [OB] a task's accumulators are complete
  const uint32_t o_free = o_full + 16;     // [OB] and have been read, with the statistics
  const uint32_t st_full = o_free + 16;    // [OB] a task's statistics are written
  const uint32_t pg_full = st_full + 16;   // [kPageSlots] 4-bit: pages of a tile are there
  const uint32_t par_full = pg_full + 8 * kPageSlots;   // [kPageSlots] its s and m
  const uint32_t par_free = par_full + 8 * kPageSlots;  // [kPageSlots] they (and the pages) have been read
  static_assert(2 * kMaxSlots + 28 + 3 * kPageSlots <= 96, "barriers fit their area");

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int grid = (int)gridDim.x, me = (int)blockIdx.x;

  make_plan<C>(p, prefix, cut, misc);
  // sequences without a task: zeros
#pragma unroll 1
  for (int b = me; b < p.batch; b += grid) {
    if (prefix[b + 1] != prefix[b]) continue;
    if (tid == 0 && p.ctx_lens[b] != 0) raise_error(p.dev_err, SPEC_DEVERR_CTX_LEN);
    const int64_t words = (int64_t)p.rows * p.heads * D / 8;
    uint4* dst = reinterpret_cast<uint4*>(p.out) + (int64_t)b * words;
    for (int64_t i = tid; i < words; i += C::kThreads) dst[i] = make_uint4(0, 0, 0, 0);
  }
  const int tasks = prefix[p.batch];
  if (me >= tasks) return;
  __syncthreads();  // the plan's area is used again below

  volatile int32_t* s_bad = misc;  // [32] a task (number & 31) met a bad page; the producer is less than 32 tasks ahead
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(misc) + 32;
  int32_t* s_last = misc + 33;
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
    for (int j = 0; j < kPageSlots; ++j) {
      bar_init(pg_full + 8 * j, 1);
      bar_init(par_full + 8 * j, 32);
      bar_init(par_free + 8 * j, 4 * C::NG);
    }
#pragma unroll 1
    for (int j = 0; j < 16; j += 8) {
      bar_init(q_full + j, 4);
      bar_init(kd_full + j, 4);
      bar_init(kd_free + j, 1);
      bar_init(vd_full + j, 4);
      bar_init(vd_free + j, 1);
      bar_init(s_full + 2 * j, 1);
      bar_init(s_full + 2 * j + 8, 1);
      bar_init(s_free + 2 * j, 4 * C::NG);
      bar_init(s_free + 2 * j + 8, 4 * C::NG);
      bar_init(p_full + j, 4 * C::NG);
      bar_init(pv_done + j, 1);
      bar_init(o_full + j, 1);
      bar_init(o_free + j, 4);
      bar_init(st_full + j, 4 * C::NG * C::ST);
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
  auto other_regs = [&]() {
    if constexpr (C::DEAL) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(C::kOtherRegs));
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

  // Each role has its own instruction for its registers, and its own end: where branches join, the compiler would hold all
  // that follows to the smaller number.
  if (!C::Q4 && warp == 0) {
    // =================== 16-bit: K and V tiles by TMA ===================
    // K and V that no other unit reads again are the first to leave L2
    const uint64_t policy = p.groups == 1 ? l2_evict_first_policy() : l2_normal_policy();
    Ring at[2];  // K's and V's
    int seq = 0;
#pragma unroll 1
    for (int t = me; t < tasks; t += grid, ++seq) {
      const Task k = task_at(p, prefix, cut, t);
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
    other_regs();
    const uint32_t id_qk = C::Q4 ? mma_desc_e4m3(N) : mma_desc<C::FP16>(N, 0, 0), id_pv = mma_desc<C::FP16>(N, C::Q4 ? 0 : 1, 1);
    const uint64_t kmaj = smem_desc_sw128(0, 16, 1024);          // K, Q: K-major
    const uint64_t vmn = smem_desc_sw128(0, TK * 128, 1024);     // V: MN-major
    const uint64_t pmn = smem_desc(0, 16, 16 * N, C::P_LAYOUT);  // P: MN-major, groups of 8 keys
    const uint32_t kq_hi = (uint32_t)(kmaj >> 32), v_hi = (uint32_t)(vmn >> 32), w_hi = (uint32_t)(pmn >> 32);
    // Values that the compiler knows to be the same in all lanes are operands of the MMAs as they are; others would be
    // moved to uniform registers for each.
    auto uniform = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
    const uint32_t tm = uniform(tmem);
    const int n_slots = (int)uniform((uint32_t)(warp == 2 ? NS - KS : KS)), all = (int)uniform((uint32_t)tasks), q_parts = p.fp16 ? 3 : 2;
    const uint32_t q_lo = uniform((uint32_t)kmaj + (q_u32 >> 4)), k_lo = uniform((uint32_t)kmaj + (ring_u32 >> 4));
    const uint32_t v_lo = uniform((uint32_t)vmn + (ring_u32 >> 4)), p_lo = uniform((uint32_t)pmn + (p_u32 >> 4));
    const uint32_t bars = uniform(full);
    auto bar = [&](uint32_t b) { return bars + (b - full); };
    auto tiles_at = [&](int t) { return (int)uniform((uint32_t)task_at(p, prefix, cut, t).tiles); };
    Ring at;  // 16-bit: the slot of the next K (V)
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
          if constexpr (C::Q4) {
            wait(bar(kd_full) + 8 * (i & 1), i >> 1);
            tc_fence_after();
            const uint32_t a = tm + C::COL_K + (i & 1) * (D / 4);
            // bf16 queries are two e4m3 numbers, fp16 ones three; the small parts first
#pragma unroll 1
            for (int part = q_parts - 1; part >= 0; --part) {
              const uint32_t qp = qb + part * (C::Q_PART >> 4), fresh = part == q_parts - 1 ? 0u : 1u;
#pragma unroll
              for (int ks = 0; ks < D / 32; ++ks)
                mma_ts<true>(dst, a + ks * 8, qp + (((ks >> 2) * N * 128 + (ks & 3) * 32) >> 4), kq_hi, id_qk, ks > 0 ? 1u : fresh);
            }
            mma_commit(bar(s_full) + 8 * (i % C::SB));
            mma_commit(bar(kd_free) + 8 * (i & 1));
          } else {
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
          }
        } else {
          const uint32_t o = tm + C::COL_O + ((seq % C::OB) * C::ST + i % C::ST) * C::O_COLS, more = j >= C::ST ? 1u : 0u;
          if (j == 0) wait(bar(o_free) + 8 * (seq % C::OB), seq / C::OB - 1);
          wait(bar(p_full) + 8 * (i & 1), i >> 1);
          const uint32_t pb = p_lo + (i % C::NP) * (C::BANDS * C::P_BYTES >> 4);
          if constexpr (C::Q4) {
            wait(bar(vd_full) + 8 * (i % C::VB), i / C::VB);
            tc_fence_after();
#pragma unroll 1
            for (int hh = 0; hh < C::HALVES; ++hh) {
              const uint32_t a = tm + C::COL_V + ((i % C::VB) * C::HALVES + hh) * (TK / 2);
#pragma unroll 1
              for (int k4 = 0; k4 < 2; ++k4)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  mma_ts<false>(o + hh * N, a + k4 * 32 + kk * 8, pb + (k4 * 4 + kk) * (32 * N >> 4), w_hi, id_pv, k4 + kk > 0 ? 1u : more);
            }
            mma_commit(bar(pv_done) + 8 * (i % C::NP));
            mma_commit(bar(vd_free) + 8 * (i % C::VB));
          } else {
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
          }
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
    other_regs();
    if (C::Q4 && warp == 3) {
      // =================== 4-bit: the tiles' pages, and s and m of their keys ===================
      // That s and m of a tile have been read says that its codes have been copied, by its pages: the unpacking comes first.
      const uint32_t row = (uint32_t)p.row;
      int n = 0, seq = 0;
#pragma unroll 1
      for (int t = me; t < tasks; t += grid, ++seq) {
        const Task k = task_at(p, prefix, cut, t);
        int win = -1, ids = 0;  // 32 entries of the page list, one a lane
#pragma unroll 1
        for (int j = 0; j < k.tiles && tries != 1; ++j, ++n) {
          const int l0 = (k.tile0 + j) << ppt_shift, s = n % kPageSlots;
          if (win < 0 || l0 >= win + 32) {
            win = l0;
            ids = checked(entry(k, l0 + lane), l0 + lane < min(k.span.pages, (k.tile0 + k.tiles) << ppt_shift), seq);
          }
          wait(par_free + 8 * s, n / kPageSlots - 1);
          int32_t* pages = reinterpret_cast<int32_t*>(fixed + S::PAGES + s * 48);
          const int id = __shfl_sync(0xffffffffu, ids, l0 - win + (lane & ((1 << ppt_shift) - 1)));
          if (lane < 8) pages[lane] = id;
          if (lane == 8) pages[8] = k.g;
          __syncwarp();
          if (lane == 0) bar_arrive(pg_full + 8 * s);
          const uint32_t dst = fixed_u32 + S::PAR + s * 1024;
#pragma unroll 2
          for (int r = lane; r < TK; r += 32) {
            const int page = __shfl_sync(0xffffffffu, ids, l0 - win + (r >> p.page_shift));
            const uint32_t slot = ((uint32_t)max(page, 0) << p.page_shift) + (r & (bs - 1));
            const uint64_t off = (uint64_t)slot * row + 4 * k.g;
            cp_async_4(dst + r * 4, p.kpar + off, page < 0 ? 0 : 4);
            cp_async_4(dst + 512 + r * 4, p.vpar + off, page < 0 ? 0 : 4);
          }
          cp_async_arrive(par_full + 8 * s);
        }
      }
      cp_async_commit();
      cp_async_wait<0>();
    }
    leave();
    return;
  }
  if (warp < C::W_SOFT) {
    // =================== epilogue: queries in, results out ===================
    other_regs();
    const int et = tid - 32 * C::W_EPI, q4 = warp & 3;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    // packed row r's place among the rows of its sequence
    auto row_of = [&](const Task& k, int r) {
      const int i = (r * p.by_gqa) >> 16;
      return (int64_t)(k.i0 + i) * p.heads + k.g * p.gqa + (r - i * p.gqa);
    };
    // Query rows of task number seq into its buffer. The buffer's last readers are done: the task QB before has been
    // written out.
    auto load_queries = [&](int t, int seq) {
      const Task k = task_at(p, prefix, cut, t);
      uint8_t* dst = fixed + S::Q + (seq % C::QB) * C::Q_BYTES;
      constexpr int L = D / 8;  // threads of a row, 8 elements each
      const int c = et % L;
      float* qc = reinterpret_cast<float*>(fixed + S::QC) + (seq % C::QB) * 128;
#pragma unroll 1
      for (int r = et / L; r < N; r += 128 / L) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (r < k.nr) x = __ldg(reinterpret_cast<const uint4*>(p.q) + ((int64_t)k.b * p.rows * p.heads + row_of(k, r)) * L + c);
        if constexpr (C::Q4) {
          // The row times a power of two that brings its largest element to [2^7, 2^8), as a sum of e4m3 numbers (8 bits
          // are two of them, 11 are three; what is below 2^-10 is lost), in the order that the unpacking leaves the codes
          // in: 0 2 4 6 1 3 5 7.
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
          float f[8], top = 0.f, sum = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 v = p.fp16 ? q4::unpack2<true>(w[e]) : q4::unpack2<false>(w[e]);
            f[2 * e] = v.x;
            f[2 * e + 1] = v.y;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            top = fmaxf(top, fabsf(f[e]));
            sum += f[e];
          }
#pragma unroll
          for (int o = 1; o < L; o <<= 1) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
          }
          const int e2 = max(-100, min(133, 7 + 127 - (__float_as_int(top) >> 23)));
          const float f1 = pow2(e2 / 2), f2 = pow2(e2 - e2 / 2);
          float even[4], odd4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            even[e] = f[2 * e] * f1 * f2;
            odd4[e] = f[2 * e + 1] * f1 * f2;
          }
          uint8_t* to = dst + (c >> 4) * N * 128 + r * 128 + ((((c & 15) >> 1) ^ (r & 7)) << 4) + (c & 1) * 8;
#pragma unroll
          for (int part = 0; part < 3; ++part) {
            const uint32_t a = take_e4m3(even), b = take_e4m3(odd4);
            *reinterpret_cast<uint2*>(to + part * C::Q_PART) = make_uint2(a, b);
          }
          if (c == 0) {
            qc[r] = pow2(max(-126, min(127, 9 - e2))) * (top < INFINITY ? p.scale_log2 : NAN);
            qc[64 + r] = sum * p.scale_log2;
          }
        }
        if constexpr (!C::Q4) *reinterpret_cast<uint4*>(dst + (c >> 3) * N * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = x;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) bar_arrive(q_full + 8 * (seq % C::QB));
    };
    // head dim of this thread's lane, and the lane that holds its neighbour
    const int d0 = C::Q4 ? q4 * 32 + 4 * (lane & 7) + (lane >> 3) : q4 * 32 + lane;
    constexpr int NEXT = C::Q4 ? 8 : 1;
    const bool odd = lane & NEXT;
    const float unit = C::Q4 ? (odd ? 0x1p20f : 0x1p24f) : 1.f;
    int64_t* e_row = reinterpret_cast<int64_t*>(fixed + S::EPI);    // [64] a row's place in the sequence's output
    float* e_fac = reinterpret_cast<float*>(fixed + S::EPI + 512);  // [ST][64] a stream's weight over the row's sum
    float* e_off = e_fac + 128;                                     // [64] what is added to the products
    int seq = -C::QB, base = 0;  // the first queries are loaded before the first result; tiles of the tasks before
#pragma unroll 1
    for (int t = me - C::QB * grid; t < tasks; t += grid, ++seq) {
      if (seq >= 0) {
        const Task k = task_at(p, prefix, cut, t);
        const int ob = seq % C::OB;
        wait(st_full + 8 * ob, seq / C::OB);
        wait(o_full + 8 * ob, seq / C::OB);
        tc_fence_after();
        const bool bad = s_bad[seq & 31] != 0;
        if (bad && et == 0) raise_error(p.dev_err, SPEC_DEVERR_BLOCK_ID);
        const int only = C::ST == 2 && k.tiles == 1 ? base % C::ST : -1;  // the one stream that had a tile
        base += k.tiles;
        named_sync(kBarEpi, 128);  // the last task's entries have been read, and the flag
        if (et == 0) s_bad[seq & 31] = 0;
        if (et < k.nr) {
          const float* stat = reinterpret_cast<const float*>(fixed + S::STAT + ob * C::ST * S::STAT_BYTES) + et;
          float sum[C::ST], ref = -INFINITY, total = 0.f, off = 0.f;
#pragma unroll
          for (int st = 0; st < C::ST; ++st) {
            const float* x = stat + st * (S::STAT_BYTES / 4);
            sum[st] = (x[0] + x[64]) + (x[128] + x[192]);
            if (sum[st] != 0.f) ref = fmaxf(ref, x[512]);
          }
#pragma unroll
          for (int st = 0; st < C::ST; ++st) {
            const float* x = stat + st * (S::STAT_BYTES / 4);
            const float f = sum[st] != 0.f ? exp2f(x[512] - ref) : 0.f;
            total = fmaf(f, sum[st], total);
            if (C::Q4 && f != 0.f) off = fmaf(f, (x[256] + x[320]) + (x[384] + x[448]), off);
            e_fac[64 * st + et] = f;
          }
          const float inv = bad ? 0.f : 1.f / total;
#pragma unroll
          for (int st = 0; st < C::ST; ++st) e_fac[64 * st + et] *= inv;
          e_off[et] = off * inv;
          e_row[et] = row_of(k, et) * D;
          // a piece without a visible key has weight 0
          if (k.pieces > 1)
            __stcg(p.lse + (int64_t)k.slot * kMaxRows + et, bad ? INFINITY : total == 0.f ? -INFINITY : ref + log2f(total));
        }
        named_sync(kBarEpi, 128);
        const uint32_t o = tmem + C::COL_O + ob * C::ST * C::O_COLS + lane_off;
        float* part = p.opart + (int64_t)k.slot * N * D;
        uint16_t* out = reinterpret_cast<uint16_t*>(p.out) + (int64_t)k.b * p.rows * p.heads * D;
#pragma unroll 1
        for (int c = 0; c < k.nr; c += 8) {
#pragma unroll 1
          for (int hh = 0; hh < C::HALVES; ++hh) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e_off[c + e];
#pragma unroll 1
            for (int st = 0; st < C::ST; ++st) {
              if (C::ST == 2 && only >= 0 && only != st) continue;
              float x[8];
              tmem_load_cols<8>(o + st * C::O_COLS + hh * N + c, x);
              if constexpr (C::BANDS == 2) {
                float low[8];
                tmem_load_cols<8>(o + (C::HALVES + hh) * N + c, low);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = fmaf(low[e], 0x1p-18f, x[e]);
              }
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = fmaf(x[e] * unit, e_fac[64 * st + c + e], v[e]);
            }
            if (D == 64 && q4 >= 2) continue;
            const int d = hh * 128 + d0;
            if (k.pieces == 1) {
              // pairs of head dims: one thread writes those of the even row, its neighbour those of the odd row
#pragma unroll
              for (int e = 0; e < 8; e += 2) {
                const float got = __shfl_xor_sync(0xffffffffu, odd ? v[e] : v[e + 1], NEXT);
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
      if (seq < 0) continue;
      const Task k = task_at(p, prefix, cut, t);
      if (k.pieces == 1) continue;
      // ---- a cut unit is joined by whoever finishes its last piece
      named_sync(kBarEpi, 128);
      if (et == 0) {
        __threadfence();  // release the piece
        int32_t* counter = p.counters + k.first / 2;
        const int last = atomicAdd(counter, 1) == k.pieces - 1;
        if (last) {
          *counter = 0;
          __threadfence();  // acquire the others
        }
        *s_last = last;
      }
      named_sync(kBarEpi, 128);
      const bool last = *s_last != 0;
      named_sync(kBarEpi, 128);  // s_last is written again
      if (!last) continue;
#pragma unroll 1
      for (int item = et; item < k.nr * (D / 4); item += 128) {
        const int r = item / (D / 4), c = item - r * (D / 4);
        const float* lse = p.lse + (int64_t)k.first * kMaxRows + r;
        const float4* src = reinterpret_cast<const float4*>(p.opart) + (int64_t)k.first * (N * D / 4) + item;
        float top = -INFINITY;
        bool none = false;
#pragma unroll 4
        for (int w = 0; w < k.pieces; ++w) {
          const float x = __ldcg(lse + (int64_t)w * kMaxRows);
          none |= x == INFINITY;
          top = fmaxf(top, x);
        }
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll 4
        for (int w = 0; w < k.pieces; ++w) {
          const float x = __ldcg(lse + (int64_t)w * kMaxRows);
          float4 y = __ldcg(src + (int64_t)w * (N * D / 4));
          const float f = x == -INFINITY ? 0.f : exp2f(x - top);
          if (x == -INFINITY) y = make_float4(0.f, 0.f, 0.f, 0.f);
          sum += f;
          a.x = fmaf(f, y.x, a.x);
          a.y = fmaf(f, y.y, a.y);
          a.z = fmaf(f, y.z, a.z);
          a.w = fmaf(f, y.w, a.w);
        }
        const float inv = 1.f / sum;
        uint2 out = p.fp16 ? make_uint2(q4::pack2<true>(a.x * inv, a.y * inv), q4::pack2<true>(a.z * inv, a.w * inv))
                           : make_uint2(q4::pack2<false>(a.x * inv, a.y * inv), q4::pack2<false>(a.z * inv, a.w * inv));
        if (none) out = make_uint2(0, 0);
        reinterpret_cast<uint2*>(p.out)[((int64_t)k.b * p.rows * p.heads + row_of(k, r)) * (D / 4) + c] = out;
      }
    }
    leave();
    return;
  }
  if (warp < C::W_K) {
    // =================== softmax ===================
    if constexpr (C::DEAL) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(C::kSoftRegs));
    const int group = (warp - C::W_SOFT) >> 2, st = group / C::NG, h = group % C::NG, c0 = h * CW, q4 = warp & 3;
    const int gt = tid - 32 * C::W_SOFT - group * 128, bar_group = kBarGroup0 + group;
    float* s_ref = reinterpret_cast<float*>(fixed + S::REF) + st * 64;
    float* s_alpha = reinterpret_cast<float*>(fixed + S::ALPHA) + st * 64;
    float* s_red = reinterpret_cast<float*>(fixed + S::RED) + st * 256;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const int key = q4 * 32 + lane;  // the lane of the scores that this thread reads
    int base = 0, seq = 0;
#pragma unroll 1
    for (int t = me; t < tasks; t += grid, ++seq) {
      const Task k = task_at(p, prefix, cut, t);
      const int ob = seq % C::OB, first = k.ctx - p.rows + k.i0;  // position of the unit's first row
      uint64_t l[CW / 2], off[C::Q4 ? CW / 2 : 1];  // pairs of rows
#pragma unroll
      for (int e = 0; e < CW / 2; ++e) l[e] = 0;
#pragma unroll
      for (int e = 0; e < (C::Q4 ? CW / 2 : 1); ++e) off[e] = 0;
      wait(q_full + 8 * (seq % C::QB), seq / C::QB);
      const float* qc = reinterpret_cast<const float*>(fixed + S::QC) + (seq % C::QB) * 128 + c0;
      const int j0 = C::ST == 2 ? (base ^ st) & 1 : 0;
#pragma unroll 1
      for (int j = j0; j < k.tiles; j += C::ST) {
        const int i = base + j;  // of stream i % ST
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
        float ks = p.scale_log2, km = 0.f, vs = 1.f, vm = 0.f;
        if constexpr (C::Q4) {
          const int s = i % kPageSlots;
          wait(par_full + 8 * s, i / kPageSlots);
          const uint32_t* par = reinterpret_cast<const uint32_t*>(fixed + S::PAR + s * 1024) + key;
          const uint32_t a = dead ? 0u : par[0], b = dead ? 0u : par[128];
          __syncwarp();
          if (lane == 0) bar_arrive(par_free + 8 * s);
          const float2 x = p.fp16 ? q4::unpack2<true>(a) : q4::unpack2<false>(a);
          const float2 y = p.fp16 ? q4::unpack2<true>(b) : q4::unpack2<false>(b);
          ks = x.x;
          km = x.y;
          vs = y.x;
          vm = fmaf(8.f, y.x, y.y);  // the codes of V are taken from 8
        }
        wait(s_full + 8 * (i % C::SB), i / C::SB);
        tc_fence_after();
        const uint32_t t_s = tmem + C::COL_S + (i % C::SB) * N + lane_off + c0;
        const uint64_t ks2 = pack_f2(ks, ks), km2 = pack_f2(km, km), vs2 = pack_f2(vs, vs);
        uint64_t y[CW / 2];  // the softmax's weights (4-bit: those that meet V are y times s)
#pragma unroll 1
        for (bool settled = false;; settled = true) {
          if (j >= C::ST || settled) {
            float x[C::CHUNK], top = 0.f;
#pragma unroll
            for (int e = 0; e < CW; e += 4) {
              if (e % C::CHUNK == 0) tmem_load_cols<C::CHUNK>(t_s + e, x);
              const float4 ref = *reinterpret_cast<const float4*>(s_ref + c0 + e);  // minus the reference
              const float* xe = x + e % C::CHUNK;
              uint64_t z[2] = {pack_f2(ref.x, ref.y), pack_f2(ref.z, ref.w)};
              if constexpr (C::Q4) {
                const float4 qa = *reinterpret_cast<const float4*>(qc + e), qb = *reinterpret_cast<const float4*>(qc + 64 + e);
                z[0] = fma_f2(km2, pack_f2(qb.x, qb.y), z[0]);
                z[1] = fma_f2(km2, pack_f2(qb.z, qb.w), z[1]);
                z[0] = fma_f2(ks2, mul_f2(pack_f2(xe[0], xe[1]), pack_f2(qa.x, qa.y)), z[0]);
                z[1] = fma_f2(ks2, mul_f2(pack_f2(xe[2], xe[3]), pack_f2(qa.z, qa.w)), z[1]);
              } else {
                z[0] = fma_f2(pack_f2(xe[0], xe[1]), ks2, z[0]);
                z[1] = fma_f2(pack_f2(xe[2], xe[3]), ks2, z[1]);
              }
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
              const float2 f = unpack_f2(C::Q4 ? mul_f2(y[e], vs2) : y[e]);
              top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
            bool grow = top > C::TOP;
            if constexpr (C::Q4) {
              const bool tiny = fabsf(vs) < C::TINY && !dead;  // s does not bound the softmax's own weights
              if (__any_sync(0xffffffffu, tiny)) {
                float most = 0.f;
#pragma unroll
                for (int e = 0; e < CW / 2; ++e) {
                  const float2 f = unpack_f2(y[e]);
                  most = fmaxf(most, fmaxf(f.x, f.y));
                }
                grow |= tiny && most > C::TOP / C::TINY;
              }
            }
            if (!named_sync_or(bar_group, 128, grow)) break;
          }
          // ---- new references: 2^SHIFT below the tile's largest weight (4-bit: weight times s) of each row, if that is
          // higher; what was summed so far is scaled down
          const float lvs = C::Q4 ? log2f(fmaxf(fabsf(vs), C::TINY)) : 0.f;
#pragma unroll 1
          for (int c = 0; c < CW; c += 8) {
            float x[8];
            tmem_load_cols<8>(t_s + c, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float s;  // the score in log2 units, and s
              if constexpr (C::Q4) s = fmaf(ks, x[e] * qc[c + e], fmaf(km, qc[64 + c + e], lvs));
              else s = x[e] * ks;
              const float m = warp_max(sees(c + e) ? s : -INFINITY);
              if (lane == 0) s_red[q4 * 64 + c0 + c + e] = m;
            }
          }
          named_sync(bar_group, 128);
          if (gt < CW) {
            const int r = c0 + gt;
            const float m = fmaxf(fmaxf(s_red[r], s_red[64 + r]), fmaxf(s_red[128 + r], s_red[192 + r]));
            const float old = j < C::ST ? kUnseen : -s_ref[r], now = fmaxf(old, m - C::SHIFT);
            s_ref[r] = -now;
            s_alpha[r] = fast_exp2(old - now);
          }
          named_sync(bar_group, 128);
          if (j >= C::ST) {
            wait(pv_done + 8 * ((i - C::ST) % C::NP), (i - C::ST) / C::NP);
            tc_fence_after();
#pragma unroll
            for (int e = 0; e < CW / 2; ++e) {
              const uint64_t a = pack_f2(s_alpha[c0 + 2 * e], s_alpha[c0 + 2 * e + 1]);
              l[e] = mul_f2(l[e], a);
              if constexpr (C::Q4) off[e] = mul_f2(off[e], a);
            }
#pragma unroll 1
            for (int part = 0; part < C::BANDS * C::HALVES; ++part) {
#pragma unroll 1
              for (int c = 0; c < CW; c += 8) {
                const uint32_t o = tmem + C::COL_O + (ob * C::ST + st) * C::O_COLS + part * N + lane_off + c0 + c;
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
        if constexpr (!C::Q4) {
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
        }
        // ---- sums, and the weights in 16 bits
        uint32_t hi[CW / 2], lo[C::BANDS == 2 ? CW / 2 : 1];
#pragma unroll
        for (int e = 0; e < CW / 2; ++e) l[e] = add_f2(l[e], y[e]);
        if constexpr (C::Q4) {
          if (whole) {
            const uint64_t vm2 = pack_f2(vm, vm);
#pragma unroll
            for (int e = 0; e < CW / 2; ++e) {
              off[e] = fma_f2(y[e], vm2, off[e]);
              y[e] = mul_f2(y[e], vs2);
            }
          } else {  // s and m may be NaN: a row that does not see the key keeps clear of them
#pragma unroll
            for (int e = 0; e < CW; e += 2) {
              const float2 w = unpack_f2(y[e / 2]), f = unpack_f2(off[e / 2]);
              off[e / 2] = pack_f2(sees(e) ? fmaf(w.x, vm, f.x) : f.x, sees(e + 1) ? fmaf(w.y, vm, f.y) : f.y);
              y[e / 2] = pack_f2(sees(e) ? w.x * vs : 0.f, sees(e + 1) ? w.y * vs : 0.f);
            }
          }
        }
#pragma unroll
        for (int e = 0; e < CW / 2; ++e) {
          const float2 w = unpack_f2(y[e]);
          if constexpr (C::BANDS == 2) {
            const float a = w.x >= 0.0625f ? w.x : 0.f, b = w.y >= 0.0625f ? w.y : 0.f;
            hi[e] = q4::pack2<true>(a, b);
            lo[e] = q4::pack2<true>((w.x - a) * 0x1p18f, (w.y - b) * 0x1p18f);
          } else {
            hi[e] = q4::pack2<C::FP16>(w.x, w.y);
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
      float* stat = reinterpret_cast<float*>(fixed + S::STAT + (ob * C::ST + st) * S::STAT_BYTES);
#pragma unroll
      for (int which = 0; which < (C::Q4 ? 2 : 1); ++which) {
#pragma unroll 1
        for (int c = 0; c < CW; c += 8) {
          float v[8];
#pragma unroll
          for (int e = 0; e < CW; e += 2) {
            const float2 f = unpack_f2(which == 0 ? l[e / 2] : off[C::Q4 ? e / 2 : 0]);
            if (e / 8 * 8 == c) {
              v[e % 8] = f.x;
              v[e % 8 + 1] = f.y;
            }
          }
          const float sum = reduce_cols<8, false>(v, lane);
          if (lane < 8) stat[256 * which + q4 * 64 + c0 + c + reduced_col<8>(lane)] = sum;
        }
      }
      if (gt < CW) stat[512 + c0 + gt] = -s_ref[c0 + gt];
      __syncwarp();
      if (lane == 0) bar_arrive(st_full + 8 * ob);
    }
    leave();
    return;
  }
  if constexpr (C::Q4) {
    // =================== 4-bit: codes from the cache into tensor memory ===================
    // Each warp copies the rows of 32 keys with 16-byte cp.async, H tiles ahead (a tensor copy's rate goes by its rows,
    // whose 64 bytes at head dim 128 are too few). Rows are swizzled so that both ways of reading a tile are free of bank
    // conflicts.
    other_regs();
    constexpr int H = C::AHEAD + 1, UG = C::UG;
    const int q4 = warp & 3, group = ((warp - C::W_K) >> 2) % UG;  // tiles i with i % UG == group
    const bool is_k = warp < C::W_V;
    const uint32_t quarter = (uint32_t)(q4 * 32) << 16;
    constexpr int CPR = D / 32, RPI = 32 / CPR;  // 16-byte chunks of a row, rows a warp copies at once
    const int c = lane % CPR, r0 = lane / CPR;
    const uint32_t row = (uint32_t)p.row;
    const uint8_t* src = (is_k ? p.kpar : p.vpar) - (int64_t)p.kv_heads * (D / 2) + c * 16;
    const uint32_t my_ring = ((is_k ? 0 : UG) + group) * H * C::SLOT, mine = ring_u32 + my_ring;
    const uint8_t* mine_ptr = ring + my_ring;
    int total = 0, at = 0, to = 0, n = group;  // slots of the next tile to unpack and to copy, and the latter's number
#pragma unroll 1
    for (int x = me; x < tasks; x += grid) total += task_at(p, prefix, cut, x).tiles;
    auto copy = [&]() {
      if (n < total) {
        const int s = n % kPageSlots;
        wait(pg_full + 8 * s, n / kPageSlots);
        const int32_t* pages = reinterpret_cast<const int32_t*>(fixed + S::PAGES + s * 48);
        const uint32_t dst = mine + to * C::SLOT + (q4 * 32 + r0) * (D / 2);
        const uint8_t* head = src + pages[8] * (D / 2);
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // 16 rows
          const int key = q4 * 32 + half * 16, page = pages[key >> p.page_shift];
          const uint32_t slot = ((uint32_t)max(page, 0) << p.page_shift) + ((key + r0) & (bs - 1));
          const uint8_t* from = head + (uint64_t)slot * row;
#pragma unroll
          for (int r = 0; r < 16; r += RPI) {
            const int swz = D == 64 ? (r0 >> 2) & 1 : D == 128 ? (r0 >> 1) & 3 : (r0 + r) & 7;
            cp_async_16(dst + (half * 16 + r) * (D / 2) + ((c ^ swz) << 4), from + r * row, page < 0 ? 0 : 16);
          }
        }
        if (++to == H) to = 0;
        n += UG;
      }
      cp_async_commit();
    };
#pragma unroll 1
    for (int x = 0; x < C::AHEAD; ++x) copy();
    if (is_k) {
      // ---- K, one key a lane. A code c in a byte is the e4m3 number c 2^-9, the subnormal ones and those above alike: a
      // word of eight codes gives two columns, codes 0 2 4 6 and 1 3 5 7, for a mask each. The queries are split instead
      // of K being made wider.
      const int key = q4 * 32 + lane;
      const int swz = D == 64 ? (key >> 2) & 1 : D == 128 ? (key >> 1) & 3 : key & 7;
#pragma unroll 1
      for (int i = group; i < total; i += UG) {
        cp_async_wait<C::AHEAD - 1>();
        __syncwarp();
        wait(kd_free + 8 * (i & 1), (i >> 1) - 1);
        tc_fence_after();
        const uint8_t* from = mine_ptr + at * C::SLOT + key * (D / 2);
        const uint32_t dst = tmem + C::COL_K + (i & 1) * (D / 4) + quarter;
#pragma unroll 1
        for (int x = 0; x < D / 32; x += 2) {
          uint32_t v[16];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint4 q = *reinterpret_cast<const uint4*>(from + (((x + u) ^ swz) << 4));
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[8 * u + 2 * e] = w[e] & 0x0f0f0f0fu;
              v[8 * u + 2 * e + 1] = (w[e] >> 4) & 0x0f0f0f0fu;
            }
          }
          tattn::tmem_st16u(dst + x * 8, v);
        }
        if (++at == H) at = 0;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(kd_full + 8 * (i & 1));
        copy();
      }
    } else {
      // ---- V, transposed. ldmatrix takes 16-bit halves, four codes of neighbouring head dims, and gives a thread those of
      // two keys: the masks leave a pair of keys for each of four head dims. Head dim 4 g + j of 32 goes to lane 8 j + g.
      // Codes are taken from 8: the sums of the tensor core, which are cut, not rounded, stay near zero, and a weight's
      // rounding meets at most 8 s.
      const int swz = D == 64 ? (lane >> 2) & 1 : D == 128 ? (lane >> 1) & 3 : lane & 7;
#pragma unroll 1
      for (int i = group; i < total; i += UG) {
        cp_async_wait<C::AHEAD - 1>();
        named_sync(kBarV + group, 128);  // all four warps' rows are there, and the last tile has been read
        copy();
        wait(vd_free + 8 * (i % C::VB), i / C::VB - 1);
        tc_fence_after();
        if (q4 < C::V_WARPS) {  // head dim 64: the upper lanes hold anything, and so do those of the results
          const uint32_t from = mine + at * C::SLOT + lane * (D / 2);
#pragma unroll 1
          for (int hh = 0; hh < C::HALVES; ++hh) {
            const uint32_t dst = tmem + C::COL_V + ((i % C::VB) * C::HALVES + hh) * (TK / 2) + quarter;
            const uint32_t m0 = from + (((hh * 4 + q4) ^ swz) << 4);
            uint32_t r[4], next[4];
            ldmatrix_x4_trans(m0, next[0], next[1], next[2], next[3]);
#pragma unroll 1
            for (int blk = 0; blk < TK / 32; ++blk) {
              uint32_t a[8], b[8];
#pragma unroll
              for (int m = 0; m < 4; ++m) r[m] = next[m];
              if (blk + 1 < TK / 32) ldmatrix_x4_trans(m0 + (blk + 1) * 32 * (D / 2), next[0], next[1], next[2], next[3]);
#pragma unroll
              for (int m = 0; m < 4; ++m) {
                const uint32_t z = r[m] >> 8;
                a[2 * m] = hadd2(r[m] & 0x000f000fu, 0x80088008u);
                a[2 * m + 1] = hadd2(r[m] & 0x00f000f0u, 0x80808080u);
                b[2 * m] = hadd2(z & 0x000f000fu, 0x80088008u);
                b[2 * m + 1] = hadd2(z & 0x00f000f0u, 0x80808080u);
              }
              tmem_st_16x128_x4(dst + blk * 16, a);
              tmem_st_16x128_x4(dst + blk * 16 + (16u << 16), b);
            }
          }
        }
        if (++at == H) at = 0;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(vd_full + 8 * (i % C::VB));
      }
    }
    cp_async_wait<0>();
    leave();
  }
}

}  // namespace wattn
}  // namespace specv
