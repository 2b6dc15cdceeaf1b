// The parts that the attention kernels over a window of a paged cache share: their
// parameters, which tiles of which unit a block works on, and the list of the units that were cut.
#pragma once

#include "pairs.cuh"
#include "q4_device.cuh"
#include "spec_verify.h"

namespace specv {
namespace wattn {

constexpr int kMaxBatch = 4096;
constexpr int kMaxRows = 64;       // packed query rows of a unit over 16 bits, and query heads of a kv head
constexpr int kMaxPieces = 768;    // pieces of cut units in a call, at most
constexpr int kCandidates = 32;
constexpr int kCutBytes = (1 + kMaxPieces / 2) * 24 + 255 & ~255;  // of the list of cut units
constexpr float kUnseen = -3e38f;  // reference of a row that has seen no key
constexpr uint32_t kMaxTries = 500000;  // of a wait, 2 s

struct CutUnit;
struct Params {
  const uint8_t* q;
  uint8_t* out;
  const uint8_t* k;  // 4-bit
  const uint8_t* v;
  const int32_t* block_table;
  const int32_t* ctx_lens;
  CutUnit* cut_units;  // [1 + kMaxPieces / 2]
  float2* stat;        // [pieces][pairs][sub]: reference of a row's weights and their sum; below 0: no result
  float* opart;        // [pieces][pairs][sub][D], normalised
  int32_t* dev_err;
  int64_t num_blocks, row;  // pages; bytes of a 4-bit token row
  int batch, rows, heads, kv_heads, gqa;
  int per, groups;  // packed rows (query row * gqa + head of the group) of a unit, row units
  int head_units;   // units of kv heads
  int by_gqa;       // 2^20 / gqa, rounded up: R / gqa = R * by_gqa >> 20 for R < 64 gqa
  int page_shift, max_blocks, window, sinks;
  int slots;  // tiles (or parts of one) that fit the ring
  // kv heads of a unit, its parts by rows, `sub` packed rows each; pairs = unit_heads * parts
  int unit_heads, parts, sub, pairs;
  int by_sub, by_parts;  // 2^16 / sub and 2^8 / parts, rounded up: quotients of what is below 256 and 8
  // 4-bit: splits that take the tiles in turns, own tiles that one is ahead of its work; bytes of a token in shared memory,
  // and where s and m begin
  int splits, ahead, seg, seg_par;
  int cuts;  // whether units may be cut, see may_cut
  float task_cost, join_cost, piece_cost;  // what a task's start and end, a join, and a piece of it cost, in tiles
  int fp16;   // type of q and out (4-bit: and of s and m)
  float scale_log2;
  float ref_unit;  // of the references in stat, in log2 units
};

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
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(r) : "f"(x));
  return r;
}
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
template <class C>
__device__ __forceinline__ int tiles_of(const Params& p, int ctx) {  // 0: nothing to do
  if (!ctx_ok(p, ctx)) return 0;
  return ((span_of(p, ctx).pages << p.page_shift) + C::KEYS - 1) / C::KEYS;
}

// A task: a unit (sequence b, head unit g, packed rows from r0 on), or one of the pieces that it was cut into.
struct Task {
  int b, g, r0, nr;
  int tile0, tiles;      // its tiles of the unit's
  int pieces, first;     // pieces of the unit, slot of its first one
  int slot;              // its own
  int ctx;
  Span span;
};
// Tasks are numbered by sequence, piece, kv head and group, so that the blocks of a wave read the same tokens for all
// heads at about the same time: a line of a 4-bit token row holds several heads.
template <class C>
__device__ __forceinline__ Task task_at(const Params& p, const int32_t* prefix, const uint16_t* cut, int t) {
  int lo = 0, hi = p.batch;  // the last b with prefix[b] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= t) lo = mid; else hi = mid;
  }
  Task k;
  k.b = lo;
  const int units = p.head_units * p.groups;
  k.pieces = (prefix[lo + 1] - prefix[lo]) / units;
  const int r = t - prefix[lo], piece = r / units, unit = r - piece * units;
  k.g = unit / p.groups;
  k.r0 = (unit - k.g * p.groups) * p.per;
  k.nr = min(p.per, p.rows * p.gqa - k.r0);
  k.ctx = p.ctx_lens[lo];
  k.span = span_of(p, k.ctx);
  const int all = ((k.span.pages << p.page_shift) + C::KEYS - 1) / C::KEYS;
  const int base = all / k.pieces, rest = all - base * k.pieces;
  k.tile0 = piece * base + min(piece, rest);
  k.tiles = base + (piece < rest ? 1 : 0);
  k.first = k.pieces > 1 ? (int)cut[lo] + unit * k.pieces : 0;
  k.slot = k.first + piece;
  return k;
}

// Whether a unit can be so long, in tiles that take `tile_us`, that cutting it pays: where not, the join's launch is left out
// with the cuts. `even_us` of tiles are even: 9 over 16 bits (8 kv heads of 128, one row: one sequence of 512 tokens, 6 us, 13
// us whole and 16 with cuts, of 1024 tokens 17 both; 20 sequences of 768 tokens 27 and 28), 6 over 4 bits, where tiles are
// shorter (one of 64 tokens, 5 us, 15 and 18, of 96 tokens 19 both, of 128 tokens 19 and 18, of 256 tokens 25 and 17).
static inline bool may_cut(const Params& p, int keys, float tile_us, float even_us) {
  const int64_t page = int64_t(1) << p.page_shift, table = (int64_t)p.max_blocks << p.page_shift;
  int64_t tokens = table;
  if (p.window != 0) tokens = (p.sinks + page - 1) / page * page + ((int64_t)p.window + p.rows + 2 * page) / page * page;
  if (tokens > table) tokens = table;
  return (float)((tokens + keys - 1) / keys) * tile_us > even_us;
}

// Length of the pieces. A block does ceil(tasks / blocks) tasks, one after the other; a task costs its tiles and
// something for its start and end, and cut units have to be joined. 32 lengths (no cut at all, and sixteenths of an even
// share) are tried, and the cheapest is taken.
template <class C>
__device__ __forceinline__ void make_plan(const Params& p, int32_t* prefix, uint16_t* cut, int32_t* misc) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = p.batch, units = p.head_units * p.groups, grid = (int)gridDim.x;
  float* cost = reinterpret_cast<float*>(misc) + 16;  // [kCandidates]
  if (tid < 2) misc[tid] = 0;  // all tiles, longest unit
  __syncthreads();
  {
    int sum = 0, most = 0;
#pragma unroll 1
    for (int b = tid; b < B; b += C::kThreads) {
      const int t = tiles_of<C>(p, p.ctx_lens[b]);
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
  // of t tiles, by the reciprocal of a piece's length: 1 to t
  auto pieces_of = [](int t, float by_len) { return max(1, (int)ceilf((float)t * by_len - 1e-3f)); };
  if (longest > 0 && p.cuts) {
#pragma unroll 1
    for (int c = warp; c < kCandidates; c += C::kWarps) {
      const float by_len = 1.f / (float)length(c);
      int tasks = 0, pieces = 0, top = 0, parts = 1;
#pragma unroll 1
      for (int b = lane; b < B; b += 32) {
        const int t = prefix[b], k = pieces_of(t, by_len);
        if (t == 0) continue;
        tasks += k;
        pieces += k > 1 ? k : 0;
        top = max(top, (int)ceilf(__fdividef((float)t, (float)k)));
        parts = max(parts, k);
      }
      tasks = __reduce_add_sync(0xffffffffu, tasks);
      pieces = __reduce_add_sync(0xffffffffu, pieces);
      top = __reduce_max_sync(0xffffffffu, top);
      parts = __reduce_max_sync(0xffffffffu, parts);
      const float waves = ceilf((float)tasks * (float)units / (float)grid);
      float x = waves * ((float)top + p.task_cost) + (parts > 1 ? p.join_cost + p.piece_cost * (float)parts : 0.f);
      if ((float)pieces * (float)units > (float)C::MAX_PIECES) x = INFINITY;
      if (lane == 0) cost[c] = x;
    }
  }
  __syncthreads();
  if (warp == 0) {
    static_assert(kCandidates == 32, "one a lane");
    const float least = longest > 0 && p.cuts ? -warp_max(-cost[lane]) : 0.f;
    const int best = longest > 0 && p.cuts ? __ffs(__ballot_sync(0xffffffffu, cost[lane] == least)) - 1 : 0;
    const float by_len = 1.f / (float)max(1, length(best));
    int tasks = 0, pieces = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < B; b0 += 32) {
      const int b = b0 + lane;
      const int t = b < B ? prefix[b] : 0;
      const int k = t == 0 ? 0 : pieces_of(t, by_len), kc = k > 1 ? k : 0;
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

// Sequences without a task: zeros.
template <class C>
__device__ __forceinline__ void clear_empty(const Params& p, const int32_t* prefix) {
#pragma unroll 1
  for (int b = (int)blockIdx.x; b < p.batch; b += (int)gridDim.x) {
    if (prefix[b + 1] != prefix[b]) continue;
    if (threadIdx.x == 0 && p.ctx_lens[b] != 0) raise_error(p.dev_err, SPEC_DEVERR_CTX_LEN);
    const int64_t words = (int64_t)p.rows * p.heads * C::D / 8;
    uint4* dst = reinterpret_cast<uint4*>(p.out) + (int64_t)b * words;
    for (int64_t i = threadIdx.x; i < words; i += C::kThreads) dst[i] = make_uint4(0, 0, 0, 0);
  }
}

// Place of packed row R of kv head g among the rows of q and out.
__device__ __forceinline__ int64_t out_row(const Params& p, int b, int g, int R) {
  const int i = R * p.by_gqa >> 20;
  return ((int64_t)b * p.rows + i) * p.heads + g * p.gqa + (R - i * p.gqa);
}

// The units that were cut, for the kernel that joins them.
struct CutUnit {
  int32_t b, g, r0, nr, pieces, first;  // of the first of the list, b is the number of the others
};
static_assert(sizeof(CutUnit) == 24, "");
template <class C>
__device__ __forceinline__ void list_cut(const Params& p, const int32_t* prefix, const uint16_t* cut, int32_t* misc) {
  if (blockIdx.x != 0 || !p.cuts) return;
  const int units = p.head_units * p.groups;
  if (threadIdx.x == 0) misc[0] = 0;
  __syncthreads();
#pragma unroll 1
  for (int b = threadIdx.x; b < p.batch; b += C::kThreads) {
    const int tasks = prefix[b + 1] - prefix[b];
    if (tasks <= units) continue;
    const int pieces = tasks / units, at = 1 + atomicAdd(&misc[0], units);
#pragma unroll 1
    for (int unit = 0; unit < units; ++unit) {
      CutUnit u;
      u.b = b;
      u.g = unit / p.groups;
      u.r0 = (unit - u.g * p.groups) * p.per;
      u.nr = min(p.per, p.rows * p.gqa - u.r0);
      u.pieces = pieces;
      u.first = (int)cut[b] + unit * pieces;
      p.cut_units[at + unit] = u;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) p.cut_units[0].b = misc[0];
}

}  // namespace wattn
}  // namespace specv
