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
constexpr int kParamSlots = 8;     // tiles of s and m in shared memory
constexpr int kCandidates = 32;
constexpr long long kMaxCycles = 2000000000LL;  // that a wait lasts at most
constexpr int kBarEpi = 1, kBarGroup0 = 2;  // named barriers: the epilogue's warps, each softmax warpgroup
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
  int slots;  // depth of the ring
  int fp16;   // type of q and out (4-bit: and of s and m)
  float scale_log2;
};

template <int D_, int ROWS_, bool Q4_, bool FP16_>
struct Cfg {
  static constexpr int D = D_, ROWS = ROWS_;  // packed rows of a unit, at most
  static constexpr bool Q4 = Q4_;
  static constexpr bool FP16 = FP16_;         // type of the MMA operands (4-bit: always fp16)
  static constexpr int N = ROWS < 16 ? 16 : ROWS;
  static constexpr int NG = ROWS <= 8 ? 1 : 2;  // softmax warpgroups, each ROWS / NG rows of every tile
  static constexpr int CW = ROWS / NG;
  static constexpr int HALVES = D == 256 ? 2 : 1;  // O^T accumulators of 128 lanes
  // A 16-bit fp16 weight keeps its bits between 2^15 and 2^-14 only: two bands of weights, the lower one times 2^18, with
  // an accumulator each, cover 2^15 to 2^-32. (4-bit: the reference takes the values' scale along, see softmax.)
  static constexpr int BANDS = FP16 && !Q4 ? 2 : 1;
  static constexpr int QB = D == 256 && N == 64 ? 1 : 2;           // query buffers
  static constexpr int NP = D == 256 && N == 64 && BANDS == 2 ? 1 : 2;  // P buffers
  static constexpr int KB = D == 256 ? 1 : 2;                      // 4-bit: unpacked K (and V) tiles in tensor memory
  static constexpr int OPERANDS = Q4 ? KB * (D / 2 + HALVES * (TK / 2)) : 0;
  static constexpr int O_COLS = BANDS * HALVES * N;
  static constexpr int OB = OPERANDS + 2 * N + 2 * O_COLS <= 512 ? 2 : 1;  // accumulators
  static constexpr int COL_K = 0, COL_V = Q4 ? KB * (D / 2) : 0, COL_S = OPERANDS, COL_O = COL_S + 2 * N;
  static constexpr int COLS = COL_O + OB * O_COLS;
  static constexpr int ALLOC = COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  static_assert(COLS <= 512, "tensor memory");
  static constexpr int SLOT = Q4 ? TK * D / 2 : TK * D * 2;  // one K or V tile
  static constexpr int Q_BYTES = N * D * 2;
  static constexpr int P_BYTES = N * TK * 2;
  // P is the operand B of the second product, MN-major: the N rows of a key are contiguous and swizzled at that width.
  static constexpr uint32_t P_LAYOUT = N == 16 ? 6u : (N == 32 ? 4u : 2u);
  static constexpr int P_SWZ_SHIFT = N == 16 ? 2 : (N == 32 ? 1 : 0);
  static constexpr int P_SWZ_MASK = N == 16 ? 1 : (N == 32 ? 3 : 7);
  static constexpr int W_EPI = 4, W_SOFT = 8, W_K = W_SOFT + 4 * NG, W_V = W_K + 4;  // first warps of the roles
  static constexpr int kWarps = Q4 ? W_V + 4 : W_K;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int V_WARPS = D / 32 < 4 ? D / 32 : 4;  // 4-bit: warps that unpack V, 32 head dims each (and a half)
  // What a task's start and end, a join, and a piece of it cost, in tiles (us over the us of a tile at the measured copy
  // bandwidth, 45 KB a us for each SM, but 0.35 us at least).
  static constexpr float TILE_US = 2.f * SLOT / 45000.f > 0.35f ? 2.f * SLOT / 45000.f : 0.35f;
  static constexpr float TASK_COST = 1.f / TILE_US, JOIN_COST = 2.f / TILE_US, PIECE_COST = 0.15f / TILE_US;
  static constexpr float SHIFT = 7.f, LIMIT = 15.f;  // weights are 2^SHIFT at the reference's maximum, 2^LIMIT at most
};

// Shared memory besides the ring, in order.
template <class C>
struct Smem {
  static constexpr int Q = 0;
  static constexpr int P = Q + C::QB * C::Q_BYTES;
  static constexpr int BARS = P + C::NP * C::BANDS * C::P_BYTES;  // 96 mbarriers
  static constexpr int REF = BARS + 96 * 8;                       // [64] reference of each row
  static constexpr int ALPHA = REF + 256;                         // [64]
  static constexpr int RED = ALPHA + 256;                         // [4][64]
  static constexpr int STAT = RED + 1024;                         // per accumulator: [4][64] sums, [4][64] offsets, [64] reference
  static constexpr int STAT_BYTES = 2048 + 256;
  static constexpr int QC = STAT + 2 * STAT_BYTES;                // [QB][2][64] factors of the scores
  static constexpr int PAR = QC + C::QB * 512;                    // [kParamSlots][2][128] s and m of K and V
  static constexpr int EPI = PAR + (C::Q4 ? kParamSlots * 1024 : 0);   // [64] int64 and twice [64] floats of the epilogue
  static constexpr int MISC = EPI + 1024;  // [64] plan, tensor-memory base, flags
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
using tattn::umma_ts;
template <bool FP16>
__device__ __forceinline__ constexpr uint32_t mma_desc(int n, int a_mn, int b_mn) {
  return (1u << 4) | (FP16 ? 0u : (1u << 7) | (1u << 10)) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(TK >> 4) << 24);
}
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
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}
// mbarrier.try_wait that may sleep for a millisecond: a warp that asks again and again takes issue slots from those that
// work (20 of 24 warps wait at any time).
__device__ __forceinline__ bool try_wait_long(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
      "selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u)
      : "memory");
  return ok != 0;
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
static __device__ __noinline__ Task task_at(const Params& p, const int32_t* prefix, const uint16_t* cut, int t) {
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
template <class C>
__global__ void __launch_bounds__(C::kThreads, 1) window_attention_kernel(const __grid_constant__ Params p,
                                                                          const __grid_constant__ CUtensorMap tm_k,
                                                                          const __grid_constant__ CUtensorMap tm_v) {
  constexpr int D = C::D, N = C::N, CW = C::CW;
  using S = Smem<C>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int NS = p.slots;
  uint8_t* ring = smem;
  uint8_t* fixed = ring + (size_t)NS * C::SLOT;
  uint64_t* bars = reinterpret_cast<uint64_t*>(fixed + S::BARS);
  uint64_t* full = bars;                     // [kMaxSlots] a tile has landed
  uint64_t* empty = full + kMaxSlots;        // [kMaxSlots] its slot may be filled again
  uint64_t* q_full = empty + kMaxSlots;      // [QB] queries and their factors written
  uint64_t* kd_full = q_full + 2;            // [KB] 4-bit: K unpacked
  uint64_t* kd_free = kd_full + 2;
  uint64_t* vd_full = kd_free + 2;
  uint64_t* vd_free = vd_full + 2;
  uint64_t* s_full = vd_free + 2;            // [2] scores of a tile
  uint64_t* p_full = s_full + 2;             // [2] weights of a tile written
  uint64_t* pv_done = p_full + 2;            // [NP] second product of the tile that used the P buffer is complete
  uint64_t* o_full = pv_done + 2;            // [OB] a task's accumulator is complete
  uint64_t* o_free = o_full + 2;             // [OB] and has been read, with the statistics
  uint64_t* st_full = o_free + 2;            // [OB] a task's statistics are written
  uint64_t* par_full = st_full + 2;          // [kParamSlots] 4-bit: s and m of a tile
  uint64_t* par_free = par_full + kParamSlots;
  static_assert(2 * kMaxSlots + 2 * 11 + 2 * kParamSlots <= 96, "barriers fit their area");
  float* s_ref = reinterpret_cast<float*>(fixed + S::REF);
  float* s_alpha = reinterpret_cast<float*>(fixed + S::ALPHA);
  float* s_red = reinterpret_cast<float*>(fixed + S::RED);
  int32_t* misc = reinterpret_cast<int32_t*>(fixed + S::MISC);
  int32_t* prefix = reinterpret_cast<int32_t*>(fixed + S::PREFIX);
  uint16_t* cut = reinterpret_cast<uint16_t*>(prefix + p.batch + 1);

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
  volatile int32_t* s_abort = misc + 34;  // a wait ran out: nothing more is issued, and no one waits any longer
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), C::ALLOC);
    tmem_relinquish();
  }
  if (tid == 0) {
    const uint32_t readers = C::Q4 ? 4 : 1;
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], C::Q4 ? 32 : 1);
      mbar_init(&empty[s], readers);
    }
    for (int j = 0; j < 2; ++j) {
      mbar_init(&q_full[j], 4);
      mbar_init(&kd_full[j], 4);
      mbar_init(&kd_free[j], 1);
      mbar_init(&vd_full[j], 4);
      mbar_init(&vd_free[j], 1);
      mbar_init(&s_full[j], 1);
      mbar_init(&p_full[j], 4 * C::NG);
      mbar_init(&pv_done[j], 1);
      mbar_init(&o_full[j], 1);
      mbar_init(&o_free[j], 4);
      mbar_init(&st_full[j], 4 * C::NG);
    }
    for (int j = 0; j < kParamSlots; ++j) {
      mbar_init(&par_full[j], 32);
      mbar_init(&par_free[j], 4 * C::NG);
    }
    fence_mbar_init();
    for (int j = 0; j < 32; ++j) s_bad[j] = 0;
    *s_abort = 0;
  }
  // what no one writes and the tensor core reads: weights of rows behind the last one (their sums are not used)
#pragma unroll 1
  for (int i = tid; i < C::NP * C::BANDS * C::P_BYTES / 16; i += C::kThreads)
    reinterpret_cast<uint4*>(fixed + S::P)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const uint32_t ring_u32 = smem_u32(ring), q_u32 = smem_u32(fixed + S::Q), p_u32 = smem_u32(fixed + S::P);

  auto wait = [&](uint64_t* bar, int n) {  // until the bar's phase n is complete (n < 0: at once)
    if (n < 0) return;
    for (long long start = 0; !try_wait_long(bar, (uint32_t)(n & 1));) {
      const long long now = clock64();
      if (start == 0) start = now;
      if (*s_abort) break;
      if (now - start > kMaxCycles) {
        *s_abort = 1;
        raise_error(p.dev_err, SPEC_DEVERR_TIMEOUT);
      }
    }
  };

  if (C::Q4 ? warp < C::W_EPI && warp != 1 : warp == 0) {
    // =================== producers ===================
    const int bs = 1 << p.page_shift, ppt = TK >> p.page_shift;
    // 32 entries of the task's page list from entry l0 on, one a lane; -1 for those behind its end and for bad pages
    auto page_ids = [&](const Task& k, int l0, int seq) {
      const int l = l0 + lane;
      int id = -1;
      bool bad = false;
      if (l < min(k.span.pages, (k.tile0 + k.tiles) * ppt)) {
        id = __ldg(p.block_table + (int64_t)k.b * p.max_blocks + (l < k.span.ns ? l : k.span.wp + l - k.span.ns));
        bad = id < 0 || (int64_t)id >= p.num_blocks;
        if (bad) id = -1;
      }
      if (__any_sync(0xffffffffu, bad) && lane == 0) s_bad[seq & 31] = 1;
      return id;
    };
    if constexpr (C::Q4) {
      // One warp copies K, one V, with 16-byte cp.async: a tensor copy's rate goes by its rows, whose 64 bytes (head dim
      // 128) are too few. Rows are swizzled so that both ways of reading a tile are free of bank conflicts. A third warp
      // copies s and m of the keys.
      constexpr int CPR = D / 32, RPI = 32 / CPR;  // 16-byte chunks of a row, rows a warp copies at once
      const int w = warp == 0 ? 0 : 1, H = NS / 2, c = lane % CPR, r0 = lane / CPR;
      const uint32_t row = (uint32_t)p.row;
      const uint8_t* src = (w == 0 ? p.kpar : p.vpar) - (int64_t)p.kv_heads * (D / 2) + (uint64_t)r0 * row + c * 16;
      int i = 0, seq = 0;
      for (int t = me; t < tasks; t += grid, ++seq) {
        const Task k = task_at(p, prefix, cut, t);
        int win = -1, ids = 0;
        if (lane == 0 && warp == 0) s_bad[seq & 31] = 0;
        __syncwarp();
        for (int j = 0; j < k.tiles; ++j, ++i) {
          const int l0 = (k.tile0 + j) * ppt;
          if (win < 0 || l0 >= win + 32) {
            win = l0;
            ids = page_ids(k, l0, seq);
          }
          if (warp == 3) {
            const int s = i % kParamSlots;
            wait(&par_free[s], i / kParamSlots - 1);
            if (__any_sync(0xffffffffu, *s_abort)) break;
            const uint32_t dst = smem_u32(fixed + S::PAR + s * 1024);
#pragma unroll 2
            for (int r = lane; r < TK; r += 32) {
              const int id = __shfl_sync(0xffffffffu, ids, l0 - win + (r >> p.page_shift));
              const uint32_t slot = ((uint32_t)max(id, 0) << p.page_shift) + (r & (bs - 1));
              const uint64_t at = (uint64_t)slot * row + 4 * k.g;
              cp_async_4(dst + r * 4, p.kpar + at, id < 0 ? 0 : 4);
              cp_async_4(dst + 512 + r * 4, p.vpar + at, id < 0 ? 0 : 4);
            }
            cp_async_arrive(&par_full[s]);
          } else {
            const int s = (i % H) * 2 + w;
            wait(&empty[s], i / H - 1);
            if (__any_sync(0xffffffffu, *s_abort)) break;
            for (int pc = 0; pc < ppt; ++pc) {
              const int id = __shfl_sync(0xffffffffu, ids, l0 - win + pc);
              const uint32_t dst = ring_u32 + s * C::SLOT + ((pc << p.page_shift) + r0) * (D / 2);
              const uint8_t* from = src + (uint64_t)((uint32_t)max(id, 0) << p.page_shift) * row + k.g * (D / 2);
#pragma unroll 4
              for (int r = 0; r < bs; r += RPI) {
                const int swz = D == 64 ? (r0 >> 2) & 1 : D == 128 ? (r0 >> 1) & 3 : (r0 + r) & 7;
                cp_async_16(dst + r * (D / 2) + ((c ^ swz) << 4), from, id < 0 ? 0 : 16);
                from += RPI * row;
              }
            }
            cp_async_arrive(&full[s]);
          }
        }
      }
      cp_async_commit();
      cp_async_wait<0>();
    } else {
      const bool once = p.groups == 1;  // read by this block alone
      const uint64_t policy = l2_evict_first_policy();
      int at = 0, seq = 0;  // tiles loaded (K and V in turns), tasks
      for (int t = me; t < tasks; t += grid, ++seq) {
        const Task k = task_at(p, prefix, cut, t);
        int win = -1, ids = 0;
        if (lane == 0) s_bad[seq & 31] = 0;
        __syncwarp();
        for (int j = 0; j < k.tiles; ++j) {
          const int l0 = (k.tile0 + j) * ppt;
          if (win < 0 || l0 >= win + 32) {
            win = l0;
            ids = page_ids(k, l0, seq);
          }
#pragma unroll 1
          for (int w = 0; w < 2; ++w, ++at) {
            const int s = at % NS;
            wait(&empty[s], at / NS - 1);
            if (__any_sync(0xffffffffu, *s_abort)) break;
            if (lane == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)C::SLOT);
            __syncwarp();
            const CUtensorMap* map = w == 0 ? &tm_k : &tm_v;
            const uint32_t dst = ring_u32 + s * C::SLOT;
#pragma unroll 1
            for (int pc = 0; pc < ppt; ++pc) {
              const int id = __shfl_sync(0xffffffffu, ids, l0 - win + pc);
              const int row = id < 0 ? -bs : id << p.page_shift;  // outside of the cache: zeros
              if (lane == 0) {
#pragma unroll
                for (int sub = 0; sub < D / 64; ++sub) {
                  const uint32_t to = dst + sub * TK * 128 + pc * bs * 128;
                  if (once) tma_load_3d_hint(to, map, sub * 64, k.g, row, &full[s], policy);
                  else tma_load_3d(to, map, sub * 64, k.g, row, &full[s]);
                }
              }
            }
            __syncwarp();
          }
        }
      }
      if (*s_abort)  // copies in flight still write here
        for (int n = max(0, at - NS); n < at; ++n) mbar_wait_bounded(&full[n % NS], (uint32_t)((n / NS) & 1), 20000000LL);
    }
  } else if (warp == 1) {
    // =================== MMA: scores of tile i + 1, then the product of tile i ===================
    const uint32_t id_qk = mma_desc<C::FP16>(N, 0, 0), id_pv = mma_desc<C::FP16>(N, C::Q4 ? 0 : 1, 1);
    const uint64_t kmaj = smem_desc_sw128(0, 16, 1024);          // K, Q: K-major
    const uint64_t vmn = smem_desc_sw128(0, TK * 128, 1024);     // V: MN-major
    const uint64_t pmn = smem_desc(0, 16, 16 * N, C::P_LAYOUT);  // P: MN-major, groups of 8 keys
    const uint32_t kq_lo = (uint32_t)kmaj, kq_hi = (uint32_t)(kmaj >> 32), v_lo = (uint32_t)vmn, v_hi = (uint32_t)(vmn >> 32);
    const uint32_t w_lo = (uint32_t)pmn, w_hi = (uint32_t)(pmn >> 32);
    int qt = me, q_left = task_at(p, prefix, cut, me).tiles, q_seq = 0, qi = 0;  // the next tile of scores
    auto scores = [&]() {
      wait(&q_full[q_seq % C::QB], q_seq / C::QB);
      const uint32_t qb = (q_u32 + (q_seq % C::QB) * C::Q_BYTES) >> 4, dst = tmem + C::COL_S + (qi & 1) * N;
      if constexpr (C::Q4) {
        wait(&kd_full[qi % C::KB], qi / C::KB);
        tc_fence_after();
#pragma unroll 1
        for (int sl = 0; sl < D / 64; ++sl) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            umma_ts(dst, tmem + C::COL_K + (qi % C::KB) * (D / 2) + sl * 32 + ks * 8, kq_lo + qb + ((sl * N * 128 + ks * 32) >> 4),
                    kq_hi, id_qk, sl + ks > 0 ? 1u : 0u);
        }
        umma_commit_elect(&s_full[qi & 1]);
        umma_commit_elect(&kd_free[qi % C::KB]);
      } else {
        const int n = 2 * qi, s = n % NS;
        wait(&full[s], n / NS);
        tc_fence_after();
        const uint32_t kb = (ring_u32 + s * C::SLOT) >> 4;
#pragma unroll 1
        for (int sl = 0; sl < D / 64; ++sl) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma_ss(dst, kq_lo + kb + ((sl * TK * 128 + ks * 32) >> 4), kq_hi, kq_lo + qb + ((sl * N * 128 + ks * 32) >> 4),
                   kq_hi, id_qk, sl + ks > 0 ? 1u : 0u);
        }
        umma_commit_elect(&s_full[qi & 1]);
        umma_commit_elect(&empty[s]);
      }
      ++qi;
      if (--q_left == 0) {
        qt += grid;
        ++q_seq;
        if (qt < tasks) q_left = task_at(p, prefix, cut, qt).tiles;
      }
    };
    int t = me, seq = 0, tiles = q_left, j = -1;  // tile j of task t is next for the second product; -1: scores first
    for (int i = -1; t < tasks; ++i) {
      if (__any_sync(0xffffffffu, *s_abort)) break;
      if (qt < tasks) scores();
      if (j >= 0) {
        const uint32_t o = tmem + C::COL_O + (seq % C::OB) * C::O_COLS;
        if (j == 0) wait(&o_free[seq % C::OB], seq / C::OB - 1);
        wait(&p_full[i & 1], i >> 1);
        const uint32_t pb = (p_u32 + (i % C::NP) * C::BANDS * C::P_BYTES) >> 4;
        const int n = 2 * i + 1, s = n % NS;
        if constexpr (C::Q4) wait(&vd_full[i % C::KB], i / C::KB);
        else wait(&full[s], n / NS);
        tc_fence_after();
        const uint32_t vb = (ring_u32 + s * C::SLOT) >> 4;
#pragma unroll 1
        for (int part = 0; part < C::BANDS * C::HALVES; ++part) {
          const int band = part / C::HALVES, hh = part % C::HALVES;
#pragma unroll 1
          for (int k4 = 0; k4 < TK / 64; ++k4) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint32_t b = w_lo + pb + ((band * C::P_BYTES + (k4 * 4 + kk) * 32 * N) >> 4);
              const uint32_t acc = j > 0 || k4 + kk > 0 ? 1u : 0u;
              if constexpr (C::Q4)
                umma_ts(o + part * N, tmem + C::COL_V + ((i % C::KB) * C::HALVES + hh) * (TK / 2) + k4 * 32 + kk * 8, b, w_hi,
                        id_pv, acc);
              else
                mma_ss(o + part * N, v_lo + vb + ((hh * 2 * TK * 128 + (k4 * 4 + kk) * 2048) >> 4), v_hi, b, w_hi, id_pv, acc);
            }
          }
        }
        umma_commit_elect(&pv_done[i % C::NP]);
        if constexpr (C::Q4) umma_commit_elect(&vd_free[i % C::KB]);
        else umma_commit_elect(&empty[s]);
        if (j == tiles - 1) umma_commit_elect(&o_full[seq % C::OB]);
      }
      if (++j == tiles) {
        j = 0;
        ++seq;
        t += grid;
        if (t < tasks) tiles = task_at(p, prefix, cut, t).tiles;
      }
    }
  } else if (warp < C::W_EPI) {
  } else if (warp < C::W_SOFT) {
    // =================== epilogue: queries in, results out ===================
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
        if (r < k.nr) {
          x = __ldg(reinterpret_cast<const uint4*>(p.q) + ((int64_t)k.b * p.rows * p.heads + row_of(k, r)) * L + c);
        }
        if constexpr (C::Q4) {
          // fp16 times a power of two that brings the row's largest element to [2^14, 2^15); the codes come in the order
          // and with the factors that the unpacking leaves them in (see there): 0 4 1 5 2 6 3 7, odd ones 16-fold
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
          const int e2 = max(-100, min(140, 14 + 127 - (__float_as_int(top) >> 23)));
          const float f1 = pow2(e2 / 2), f2 = pow2(e2 - e2 / 2);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = f[e] * f1 * f2;
          x = make_uint4(q4::pack2<true>(f[0], f[4]), q4::pack2<true>(f[1] * 0.0625f, f[5] * 0.0625f),
                         q4::pack2<true>(f[2], f[6]), q4::pack2<true>(f[3] * 0.0625f, f[7] * 0.0625f));
          if (c == 0) {
            qc[r] = pow2(max(-126, min(127, 24 - e2))) * p.scale_log2;
            qc[64 + r] = sum * p.scale_log2;
          }
        }
        *reinterpret_cast<uint4*>(dst + (c >> 3) * N * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = x;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[seq % C::QB]);
    };
    // head dim of this thread's lane, and the lane that holds its neighbour
    const int d0 = C::Q4 ? q4 * 32 + 4 * (lane & 7) + (lane >> 3) : q4 * 32 + lane;
    constexpr int NEXT = C::Q4 ? 8 : 1;
    const bool odd = lane & NEXT;
    const float unit = C::Q4 ? (odd ? 0x1p20f : 0x1p24f) : 1.f;
    int64_t* e_row = reinterpret_cast<int64_t*>(fixed + S::EPI);        // [64] a row's place in the sequence's output
    float* e_inv = reinterpret_cast<float*>(fixed + S::EPI + 512);      // [64] 1 / its sum
    float* e_off = e_inv + 64;                                          // [64] what is added to the product
    int seq = -C::QB;  // the first queries are loaded before the first result
    for (int t = me - C::QB * grid; t < tasks; t += grid, ++seq) {
     if (seq >= 0) {
      const Task k = task_at(p, prefix, cut, t);
      const int ob = seq % C::OB;
      wait(&st_full[ob], seq / C::OB);
      wait(&o_full[ob], seq / C::OB);
      tc_fence_after();
      const bool bad = s_bad[seq & 31] != 0;
      if (bad && et == 0) raise_error(p.dev_err, SPEC_DEVERR_BLOCK_ID);
      named_sync(kBarEpi, 128);  // the last task's entries have been read
      if (et < k.nr) {
        const float* stat = reinterpret_cast<const float*>(fixed + S::STAT + ob * S::STAT_BYTES) + et;
        const float sum = (stat[0] + stat[64]) + (stat[128] + stat[192]);
        e_row[et] = row_of(k, et) * D;
        e_inv[et] = bad ? 0.f : 1.f / sum;
        if constexpr (C::Q4) e_off[et] = (stat[256] + stat[320]) + (stat[384] + stat[448]);
        // a piece without a visible key has weight 0
        if (k.pieces > 1)
          __stcg(p.lse + (int64_t)k.slot * kMaxRows + et, bad ? INFINITY : sum == 0.f ? -INFINITY : stat[512] + log2f(sum));
      }
      named_sync(kBarEpi, 128);
      const uint32_t o = tmem + C::COL_O + ob * C::O_COLS + lane_off;
      float* part = p.opart + (int64_t)k.slot * N * D;
      uint16_t* out = reinterpret_cast<uint16_t*>(p.out) + (int64_t)k.b * p.rows * p.heads * D;
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
            for (int e = 0; e < 8; ++e) v[e] = fmaf(low[e], 0x1p-18f, v[e]);
          }
          if (D == 64 && q4 >= 2) continue;
          const int d = hh * 128 + d0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if constexpr (C::Q4) v[e] = fmaf(v[e], unit, e_off[c + e]);
            v[e] *= e_inv[c + e];
          }
          if (k.pieces == 1) {
            // pairs of head dims: one thread writes those of the even row, its neighbour those of the odd row
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float got = __shfl_xor_sync(0xffffffffu, odd ? v[e] : v[e + 1], NEXT);
              const float lo = odd ? got : v[e], hi = odd ? v[e + 1] : got;
              const int r = c + e + (odd ? 1 : 0);
              if (r < k.nr)
                *reinterpret_cast<uint32_t*>(out + e_row[r] + (d & ~1)) = p.fp16 ? q4::pack2<true>(bad ? 0.f : lo, bad ? 0.f : hi)
                                                                               : q4::pack2<false>(bad ? 0.f : lo, bad ? 0.f : hi);
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
      if (lane == 0) mbar_arrive(&o_free[ob]);
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
        for (int w = 0; w < k.pieces; ++w) {
          const float x = __ldcg(lse + (int64_t)w * kMaxRows);
          if (x == -INFINITY) continue;
          const float4 y = __ldcg(src + (int64_t)w * (N * D / 4));
          const float f = exp2f(x - top);
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
  } else if (warp < C::W_K) {
    // =================== softmax ===================
    const int sw = warp - C::W_SOFT, h = sw >> 2, c0 = h * CW, q4 = warp & 3;
    const int gt = tid - 32 * C::W_SOFT - h * 128, bar_group = kBarGroup0 + h;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const int key = q4 * 32 + lane;  // the lane of the scores that this thread reads
    const int bs = 1 << p.page_shift, ppt_shift = 7 - p.page_shift;
    int i = 0, seq = 0;
    for (int t = me; t < tasks; t += grid, ++seq) {
      const Task k = task_at(p, prefix, cut, t);
      const int ob = seq % C::OB, first = k.ctx - p.rows + k.i0;  // position of the unit's first row
      float l[CW], off[C::Q4 ? CW : 1];
#pragma unroll
      for (int e = 0; e < CW; ++e) l[e] = 0.f;
#pragma unroll
      for (int e = 0; e < (C::Q4 ? CW : 1); ++e) off[e] = 0.f;
      wait(&q_full[seq % C::QB], seq / C::QB);
      const float* qc = reinterpret_cast<const float*>(fixed + S::QC) + (seq % C::QB) * 128 + c0;
      for (int j = 0; j < k.tiles; ++j, ++i) {
        // ---- which rows see this thread's key: [r_lo, r_hi)
        const int lp = ((k.tile0 + j) << ppt_shift) + (key >> p.page_shift);
        const int tok = ((lp < k.span.ns ? lp : k.span.wp + lp - k.span.ns) << p.page_shift) + (key & (bs - 1));
        int r_lo = max(0, tok - first) * p.gqa, r_hi = k.nr;
        if (p.window != 0 && tok >= p.sinks) r_hi = min(r_hi, (int)min((int64_t)1 << 20, max((int64_t)0, (int64_t)tok - first + p.window)) * p.gqa);
        if (lp >= k.span.pages || tok >= k.ctx) r_hi = 0;
        const bool dead = r_lo >= r_hi;
        const bool masked = __any_sync(0xffffffffu, r_lo > 0 || r_hi < k.nr);
        float ks = 1.f, km = 0.f, vs = 1.f, vm = 0.f, lvs = 0.f;
        if constexpr (C::Q4) {
          const int s = i % kParamSlots;
          wait(&par_full[s], i / kParamSlots);
          const uint32_t* par = reinterpret_cast<const uint32_t*>(fixed + S::PAR + s * 1024);
          const uint32_t a = dead ? 0u : par[key], b = dead ? 0u : par[128 + key];
          const float2 x = p.fp16 ? q4::unpack2<true>(a) : q4::unpack2<false>(a);
          const float2 y = p.fp16 ? q4::unpack2<true>(b) : q4::unpack2<false>(b);
          ks = x.x;
          km = x.y;
          vs = y.x;
          vm = fmaf(8.f, y.x, y.y);  // the codes of V are taken from 8
          lvs = __log2f(fmaxf(fabsf(vs), 0x1p-60f));
          __syncwarp();
          if (lane == 0) mbar_arrive(&par_free[s]);
        }
        wait(&s_full[i & 1], i >> 1);
        tc_fence_after();
        float x[CW];
        tmem_load_cols<CW>(tmem + C::COL_S + (i & 1) * N + lane_off + c0, x);
        bool grow = j == 0;
        float top = -INFINITY;
#pragma unroll
        for (int e = 0; e < CW; ++e) {
          if constexpr (C::Q4) x[e] = fmaf(ks, x[e] * qc[e], km * qc[64 + e]);
          else x[e] *= p.scale_log2;
        }
        if (masked) {
#pragma unroll
          for (int e = 0; e < CW; ++e)
            if (c0 + e < r_lo || c0 + e >= r_hi) x[e] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < CW; ++e) top = fmaxf(top, x[e] - s_ref[c0 + e]);
        grow |= top + lvs > C::LIMIT;
        if (named_sync_or(bar_group, 128, grow)) {
          // ---- new references: 2^SHIFT below the tile's largest weight (4-bit: weight times s) of each row, if that is
          // higher; what was summed so far is scaled down
#pragma unroll
          for (int e = 0; e < CW; ++e) {
            const float m = warp_max(x[e] + lvs);
            if (lane == 0) s_red[q4 * 64 + c0 + e] = m;
          }
          named_sync(bar_group, 128);
          if (gt < CW) {
            const int r = c0 + gt;
            const float m = fmaxf(fmaxf(s_red[r], s_red[64 + r]), fmaxf(s_red[128 + r], s_red[192 + r]));
            const float old = j == 0 ? kUnseen : s_ref[r], now = fmaxf(old, m - C::SHIFT);
            s_ref[r] = now;
            s_alpha[r] = fast_exp2(old - now);
          }
          named_sync(bar_group, 128);
          if (j > 0) {
            wait(&pv_done[(i - 1) % C::NP], (i - 1) / C::NP);
            tc_fence_after();
            constexpr int CH = CW < 16 ? CW : 16;
#pragma unroll
            for (int e = 0; e < CW; ++e) {
              l[e] *= s_alpha[c0 + e];
              if constexpr (C::Q4) off[e] *= s_alpha[c0 + e];
            }
#pragma unroll 1
            for (int part = 0; part < C::BANDS * C::HALVES; ++part) {
#pragma unroll
              for (int c = 0; c < CW; c += CH) {
                const uint32_t o = tmem + C::COL_O + ob * C::O_COLS + part * N + lane_off + c0 + c;
                float v[CH];
                tmem_load_cols<CH>(o, v);
#pragma unroll
                for (int e = 0; e < CH; ++e) v[e] *= s_alpha[c0 + c + e];
                tmem_store_cols<CH>(o, v);
              }
            }
          }
        }
        if constexpr (!C::Q4) {
          // slots that no row sees may hold anything: zero their V
          if (__any_sync(0xffffffffu, dead)) {
            // With two slots, K and V of the tile before may be the last that the V barrier's parity knows of; its product
            // says that they have landed.
            if (NS == 2 && i > 0) wait(&pv_done[(i - 1) % C::NP], (i - 1) / C::NP);
            const int n = 2 * i + 1, s = n % NS;
            wait(&full[s], n / NS);
            if (dead) {
              uint8_t* v = ring + s * C::SLOT + key * 128;
              for (int c = h; c < D / 8; c += C::NG)
                *reinterpret_cast<uint4*>(v + (c >> 3) * TK * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
          }
        }
        // ---- weights
#pragma unroll
        for (int e = 0; e < CW; ++e) {
          x[e] = fast_exp2(x[e] - s_ref[c0 + e]);
          l[e] += x[e];
        }
        if constexpr (C::Q4) {
          if (masked) {  // s and m of a key may be NaN for the rows that see it
#pragma unroll
            for (int e = 0; e < CW; ++e) {
              const bool see = c0 + e >= r_lo && c0 + e < r_hi;
              off[e] += see ? x[e] * vm : 0.f;
              x[e] = see ? x[e] * vs : 0.f;
            }
          } else {
#pragma unroll
            for (int e = 0; e < CW; ++e) {
              off[e] = fmaf(x[e], vm, off[e]);
              x[e] *= vs;
            }
          }
        }
        uint32_t hi[CW / 2], lo[C::BANDS == 2 ? CW / 2 : 1];
#pragma unroll
        for (int e = 0; e < CW; e += 2) {
          if constexpr (C::BANDS == 2) {
            const float a = x[e] >= 0.0625f ? x[e] : 0.f, b = x[e + 1] >= 0.0625f ? x[e + 1] : 0.f;
            hi[e / 2] = q4::pack2<true>(a, b);
            lo[e / 2] = q4::pack2<true>((x[e] - a) * 0x1p18f, (x[e + 1] - b) * 0x1p18f);
          } else {
            hi[e / 2] = q4::pack2<C::FP16>(x[e], x[e + 1]);
          }
        }
        if (i >= C::NP) wait(&pv_done[i % C::NP], i / C::NP - 1);
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
        if (lane == 0) mbar_arrive(&p_full[i & 1]);
      }
      // ---- the task's statistics
      wait(&o_free[ob], seq / C::OB - 1);
      float* stat = reinterpret_cast<float*>(fixed + S::STAT + ob * S::STAT_BYTES);
      const float sum = reduce_cols<CW, false>(l, lane);
      if (lane < CW) stat[q4 * 64 + c0 + reduced_col<CW>(lane)] = sum;
      if constexpr (C::Q4) {
        const float o = reduce_cols<CW, false>(off, lane);
        if (lane < CW) stat[256 + q4 * 64 + c0 + reduced_col<CW>(lane)] = o;
      }
      if (gt < CW) stat[512 + c0 + gt] = s_ref[c0 + gt];
      __syncwarp();
      if (lane == 0) mbar_arrive(&st_full[ob]);
    }
  } else if (warp < C::W_V) {
    // =================== 4-bit: K codes into tensor memory, one key a lane ===================
    if constexpr (C::Q4) {
      // A code c in the low bits of a 16-bit half is the fp16 number c 2^-24, four bits higher c 2^-20: masks are all
      // that it takes. A word of eight codes gives four columns, codes (0, 4), (1, 5), (2, 6), (3, 7), the second and the
      // fourth 16-fold.
      const int q4 = warp & 3, key = q4 * 32 + lane;
      int total = 0;
#pragma unroll 1
      for (int t = me; t < tasks; t += grid) total += task_at(p, prefix, cut, t).tiles;
      for (int i = 0; i < total; ++i) {
        const int s = (i % (NS / 2)) * 2;
        wait(&full[s], i / (NS / 2));
        wait(&kd_free[i % C::KB], i / C::KB - 1);
        tc_fence_after();
        const uint8_t* row = ring + s * C::SLOT + key * (D / 2);
        const int swz = D == 64 ? (key >> 2) & 1 : D == 128 ? (key >> 1) & 3 : key & 7;
        const uint32_t dst = tmem + C::COL_K + (i % C::KB) * (D / 2) + ((uint32_t)(q4 * 32) << 16);
#pragma unroll 1
        for (int c = 0; c < D / 32; c += 2) {
          uint32_t v[32];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint4 x = *reinterpret_cast<const uint4*>(row + (((c + u) ^ swz) << 4));
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[16 * u + 4 * e] = w[e] & 0x000f000fu;
              v[16 * u + 4 * e + 1] = w[e] & 0x00f000f0u;
              v[16 * u + 4 * e + 2] = (w[e] >> 8) & 0x000f000fu;
              v[16 * u + 4 * e + 3] = (w[e] >> 8) & 0x00f000f0u;
            }
          }
          tmem_st32(dst + c * 16, v);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&kd_full[i % C::KB]);
      }
    }
  } else {
    // =================== 4-bit: V codes into tensor memory, transposed ===================
    if constexpr (C::Q4) {
      // ldmatrix takes 16-bit halves, four codes of neighbouring head dims, and gives a thread those of two keys: the
      // masks leave a pair of keys for each of four head dims. Head dim 4 g + j of 32 goes to lane 8 j + g. Codes are
      // taken from 8, so that a weight's rounding meets at most 8 s.
      const int q4 = warp & 3;
      int total = 0;
#pragma unroll 1
      for (int t = me; t < tasks; t += grid) total += task_at(p, prefix, cut, t).tiles;
      if (q4 >= C::V_WARPS) {  // head dim 64: the upper lanes are not used
#pragma unroll
        for (int kb = 0; kb < C::KB; ++kb) {
          const uint32_t z[32] = {};
          tmem_st32(tmem + C::COL_V + kb * (TK / 2) + ((uint32_t)(q4 * 32) << 16), z);
          tmem_st32(tmem + C::COL_V + kb * (TK / 2) + 32 + ((uint32_t)(q4 * 32) << 16), z);
        }
        tmem_wait_st();
      }
      for (int i = 0; i < total; ++i) {
        const int s = (i % (NS / 2)) * 2 + 1;
        wait(&full[s], i / (NS / 2));
        wait(&vd_free[i % C::KB], i / C::KB - 1);
        tc_fence_after();
        if (q4 < C::V_WARPS) {
          const uint32_t base = ring_u32 + s * C::SLOT;
#pragma unroll 1
          for (int hh = 0; hh < C::HALVES; ++hh) {
            const uint32_t dst = tmem + C::COL_V + ((i % C::KB) * C::HALVES + hh) * (TK / 2) + ((uint32_t)(q4 * 32) << 16);
#pragma unroll 2
            for (int blk = 0; blk < TK / 32; ++blk) {
              const int key = blk * 32 + lane, c = hh * 4 + q4;
              const int swz = D == 64 ? (key >> 2) & 1 : D == 128 ? (key >> 1) & 3 : key & 7;
              uint32_t r[4], a[8], b[8];
              ldmatrix_x4_trans(base + key * (D / 2) + ((c ^ swz) << 4), r[0], r[1], r[2], r[3]);
#pragma unroll
              for (int m = 0; m < 4; ++m) {
                a[2 * m] = hadd2(r[m] & 0x000f000fu, 0x80088008u);
                a[2 * m + 1] = hadd2(r[m] & 0x00f000f0u, 0x80808080u);
                b[2 * m] = hadd2((r[m] >> 8) & 0x000f000fu, 0x80088008u);
                b[2 * m + 1] = hadd2((r[m] >> 8) & 0x00f000f0u, 0x80808080u);
              }
              tmem_st_16x128_x4(dst + blk * 16, a);
              tmem_st_16x128_x4(dst + blk * 16 + (16u << 16), b);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&vd_full[i % C::KB]);
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::ALLOC);
  }
}

}  // namespace wattn
}  // namespace specv
