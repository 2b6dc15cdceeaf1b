// Kernel of the attention over a 4-bit cache (see the comment at the top of
// window_attention.cu).
//
// A block has eight warps, one for each kv head of a unit (or for 16 or 32 of a head's
// rows; where there are fewer, splits of warps take the tiles in turns). A tile is 16 whole
// token rows of K and of V, contiguous in a page, so that two bulk copies bring it for all
// heads: 16-byte copies by the warps took 120 of 650 instructions for 32 keys, and tensor
// copies, which go by rows, 8.6 cycles for each of 64 bytes. From there every warp works
// alone, without a barrier inside the block but the ring's:
//
//   scores   mma m16n8k16, rows x 8 keys, the codes as fp16: c in the low bits of a half is
//            the subnormal c 2^-24, so that one mask makes two operands out of a word.
//            Queries are fp16 times a power of two of the row, bf16 ones exactly.
//   softmax  in the accumulators' lanes; s and m of a tile are spread by shared memory
//   product  rows x 8 head dims, the weights times s as fp16, codes of V by ldmatrix
//
// mma.sync instead of tcgen05: operands of the latter have to pass through tensor or shared
// memory, unpacked, and every step between unpacking, MMAs and softmax is a barrier that
// warps wait at. A kernel of that kind (K as e4m3 against queries in parts, V transposed by
// ldmatrix, unpacked into tensor memory, two softmax streams) took 228 us on 32 sequences of
// 16384 tokens, 8 kv heads of 128, 16 rows, where this one takes 169; 755 us with 64 rows
// over 655,000 tokens, here 721; 225 us for 4 heads of 256 and 24 rows, here 226: the choice
// is won on up to 16 rows, and even on more. (All of these are single calls between events
// with L2 flushed, on the same inputs.)
//
// What bounds it: 372 instructions for 16 keys, a head and 16 rows (33 of them mma), 57% of
// the issue slots used, start and end included: 84 us' worth of HBM reads in 169. With 32
// rows or head dim 256 the accumulators leave room for eight warps an SM, which issue in 41%
// of the slots and wait for their results 1.7 cycles an instruction. Each against this kernel
// as it was then: interleaving the next tile's scores with this one's product was slower (174
// us for 167), as were 16 rows a warp for 64 (778 for 709) and two warps for a head's rows,
// which exchange weights and share the head dims (224 us for 228 at head dim 256, 916 for 708
// with 64 rows). 17 to 32 rows go two MMA tiles to a warp, which unpack once for both (374 us
// for 411 in two units).
#pragma once

#include <type_traits>

#include "q4_device.cuh"
#include "window_plan.cuh"

namespace specv {
namespace qattn {

using wattn::Params;
using wattn::Task;
using wattn::bar_init;
using wattn::bar_arrive;
using wattn::bar_expect;

constexpr int TK = 16;           // keys of a tile in shared memory; all of one page
constexpr int kMaxSlots = 32;    // such tiles
constexpr int kMaxPieces = 320;  // pieces of cut units in a call

template <int D_, int MT_>
struct Cfg {
  static constexpr int D = D_, MT = MT_;
  static constexpr int ROWS = 16 * MT;  // packed rows of a warp: MT tiles of the MMA's M
  static constexpr int kWarps = 8, kThreads = 32 * kWarps;
  // Two blocks share an SM where the accumulators leave room in registers, so that one computes while the other starts or
  // ends a task.
  static constexpr int kBlocks = D == 256 || MT == 2 ? 1 : 2;
  static constexpr int KEYS = 32, MAX_PIECES = kMaxPieces;
  static constexpr int STEPS = D / 16, TILES = D / 8;  // MMAs of a row of scores, and of an accumulator's row
  static constexpr int Q_BYTES = MT * STEPS * 512;     // of a kv head's rows
  static constexpr int STATE = MT * (TILES * 4 + 6);   // registers of a lane that the join of splits hands over
  // Weights are 2^SHIFT at the largest of the keys that set a row's reference, TOP at most.
  static constexpr float SHIFT = 7.f, TOP = 32768.f, TINY = 0x1p-40f;
};

// Shared memory behind the ring, in order.
template <class C>
struct Smem {
  static constexpr int BARS = 0;                        // [2][kMaxSlots] mbarriers
  static constexpr int PAR = BARS + 2 * kMaxSlots * 8;  // [warps][8][2][4] of a pair of keys: s, s, m, m, of K and of V; fp32
  static constexpr int MISC = PAR + C::kWarps * 256;    // [64]
  static constexpr int TASK = MISC + 256;
  static constexpr int PARAMS = TASK + 64;
  // [pairs][2][ROWS] factors of the scores; then the queries, and the plan
  static constexpr int QC = PARAMS + (sizeof(Params) + 15) / 16 * 16;
  static_assert(sizeof(Task) <= 64, "");
  __host__ __device__ static int q(int pairs) { return (QC + pairs * 2 * C::ROWS * 4 + 127) & ~127; }
  __host__ __device__ static int prefix(int pairs) { return q(pairs) + pairs * C::Q_BYTES; }
  __host__ __device__ static int bytes(int pairs, int batch) { return prefix(pairs) + (((batch + 1) * 6 + 127) & ~127); }
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same from zero.
__device__ __forceinline__ void mma_f16_fresh(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// fp16, the largest one in place of what is above it: weights of rows whose scores are so large that their own rounding
// takes them past TOP.
__device__ __forceinline__ uint32_t pack_sat(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The larger one of each half, b without its sign.
__device__ __forceinline__ uint32_t max_abs(uint32_t a, uint32_t b) {
  const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&a), __habs2(*reinterpret_cast<const __half2*>(&b)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.b32 %0, [%1];\n" : "=r"(r) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];\n" : "=r"(r.x), "=r"(r.y) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// The parts of the kernel outside of its hot loop are calls of their own: inlined, they cost that loop registers. Their
// parameters are in shared memory.
template <class C>
__device__ __noinline__ void plan_call(const Params& p, int32_t* prefix, uint16_t* cut, int32_t* misc) {
  wattn::make_plan<C>(p, prefix, cut, misc);
  wattn::clear_empty<C>(p, prefix);
  wattn::list_cut<C>(p, prefix, cut, misc);
}
template <class C>
__device__ __noinline__ void task_call(const Params& p, const int32_t* prefix, const uint16_t* cut, int t, Task* to) {
  *to = wattn::task_at<C>(p, prefix, cut, t);
}
// Queries: fp16 times a power of two that brings a row's largest element to [2^14, 2^15), as operand A of the
// MMAs. Lane 4 g + t of step s holds rows g and g + 8 of the elements that meet the codes of key g that the lane has
// (see scores); those 16-fold of odd codes are divided by 16. qc: what a row's scores have to be multiplied with, a power of
// two (the codes' 2^-24 with it), and the sum of its queries divided by that.
template <class C>
__device__ __noinline__ void query_call(const Params& p, const Task* task, uint8_t* queries, float* qc) {
  constexpr int D = C::D, ROWS = C::ROWS;
  const Task k = *task;
  const int tid = threadIdx.x, lane = tid & 31;
  const bool fp16 = p.fp16;
  constexpr int L = D / 8, STEP = C::kThreads / L;  // threads of a row, 8 elements each; rows in a step
  const int c = tid % L, head0 = k.g * p.unit_heads, rows = p.pairs * p.sub;
  auto row = [&](int x) {  // row x, zeros if there is none
    const int of_pair = x * p.by_sub >> 16, h = of_pair * p.by_parts >> 8, R = k.r0 - h * p.per + x;
    uint4 got = make_uint4(0, 0, 0, 0);
    if (x < rows && R < k.r0 + k.nr && head0 + h < p.kv_heads)
      got = __ldg(reinterpret_cast<const uint4*>(p.q) + wattn::out_row(p, k.b, head0 + h, R) * L + c);
    return got;
  };
  uint4 next[2] = {row(tid / L), row(tid / L + STEP)};
  // rows behind a pair's
#pragma unroll 1
  for (int x = tid; p.sub < ROWS && x < p.pairs * C::Q_BYTES / 16; x += C::kThreads)
    reinterpret_cast<uint4*>(queries)[x] = make_uint4(0, 0, 0, 0);
#pragma unroll 1
  for (int x = tid; x < p.pairs * 2 * ROWS; x += C::kThreads) qc[x] = 0.f;
  __syncthreads();
#pragma unroll 1
  for (int rr0 = tid / L; rr0 - lane / L < rows; rr0 += 2 * STEP) {
    const uint4 now[2] = {next[0], next[1]};
    next[0] = row(rr0 + 2 * STEP);
    next[1] = row(rr0 + 3 * STEP);
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const uint4 x = now[y];
      const int rr = rr0 + y * STEP, of_pair = rr * p.by_sub >> 16, r = rr - of_pair * p.sub;
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      float f[8], top = 0.f, sum = 0.f;
      if (fp16) {
#pragma unroll
        for (int e = 0; e < 4; ++e) reinterpret_cast<float2*>(f)[e] = q4::unpack2<true>(w[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) reinterpret_cast<float2*>(f)[e] = q4::unpack2<false>(w[e]);
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
      const int e2 = max(-100, min(126, 14 + 127 - (__float_as_int(top) >> 23)));
      const float f1 = pow2(e2), f2 = pow2(e2 - 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= e & 1 ? f2 : f1;
      if (rr < rows && c == 0) {
        qc[of_pair * 2 * ROWS + r] = pow2(24 - e2);
        qc[of_pair * 2 * ROWS + ROWS + r] = sum * pow2(e2 - 24);
      }
      // word c of the row is word `at` of lane `of`'s codes, and the operands of two steps
      constexpr int WORDS = D / 32 < 4 ? D / 32 : 4;  // words of a lane in a row of up to 64 bytes
      const int of = (c / WORDS) & 3, at = c % WORDS + (c / (4 * WORDS)) * WORDS;
      const int mt = r / 16, up = (r / 8) & 1;
      uint32_t* dst = reinterpret_cast<uint32_t*>(queries + of_pair * C::Q_BYTES) + (mt * C::STEPS + 2 * at) * 128 + ((r & 7) * 4 + of) * 4 + up;
      if (rr < rows) {
        dst[0] = q4::pack2<true>(f[0], f[4]);
        dst[2] = q4::pack2<true>(f[1], f[5]);
        dst[128] = q4::pack2<true>(f[2], f[6]);
        dst[130] = q4::pack2<true>(f[3], f[7]);
      }
    }
  }
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kBlocks) q4_attention_kernel(const __grid_constant__ Params p) {
  constexpr int D = C::D, MT = C::MT, ROWS = C::ROWS, NB = 2;
  using S = Smem<C>;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t stage_bytes = 2 * TK * p.seg;  // K's tokens, then V's
  uint8_t* fixed = smem + p.slots * stage_bytes;
  int32_t* misc = reinterpret_cast<int32_t*>(fixed + S::MISC);
  int32_t* prefix = reinterpret_cast<int32_t*>(fixed + S::prefix(p.pairs));
  uint16_t* cut = reinterpret_cast<uint16_t*>(prefix + p.batch + 1);
  const uint32_t full = smem_u32(fixed + S::BARS), empty = full + 8 * kMaxSlots, ring_u32 = smem_u32(smem);
  // Values that the compiler knows to be the same in all lanes do without the registers of each thread.
  auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5), g = lane >> 2, t4 = lane & 3;
  const int grid = (int)gridDim.x, me = (int)blockIdx.x;

  // the queries are on their way to L2 while the plan is made
  {
    const int64_t all = (int64_t)p.batch * p.rows * p.heads * D * 2, bytes = all < 32 << 20 ? all : 32 << 20;
    for (int64_t at = ((int64_t)me * C::kThreads + tid) * 128; at < bytes; at += (int64_t)grid * C::kThreads * 128)
      asm volatile("prefetch.global.L2 [%0];\n" ::"l"(p.q + at));
  }
  // The calls read the parameters here: by a reference to the kernel's own they take a memory access each.
  Params* shared = reinterpret_cast<Params*>(fixed + S::PARAMS);
  if (tid == 0) *shared = p;
  __syncthreads();
  plan_call<C>(*shared, prefix, cut, misc);
  const int tasks = uniform(prefix[p.batch]);
  if (me >= tasks) return;
  __syncthreads();  // the plan's area is used again below
  volatile int32_t* s_bad = misc;  // [2] a task (number & 1) met a bad page
  if (tid == 0) {
    misc[0] = misc[1] = 0;
#pragma unroll 1
    for (int s = 0; s < p.slots; ++s) {
      bar_init(full + 8 * s, 1);
      bar_init(empty + 8 * s, (uint32_t)p.pairs);
    }
    fence_mbar_init();
  }

  // This warp: rows `part` of kv head `head` of a unit, tiles split, split + splits, ...
  const int pair = warp % p.pairs, split = warp / p.pairs, head = pair / p.parts, part = pair - head * p.parts;
  const bool works = split < p.splits;
  float* par = reinterpret_cast<float*>(fixed + S::PAR) + warp * 64;
  float* qc = reinterpret_cast<float*>(fixed + S::QC);
  uint8_t* queries = fixed + S::q(p.pairs);
  const int bs = 1 << p.page_shift;
  uint32_t tries = wattn::kMaxTries;
  int slot0 = 0, round0 = 0;  // ring slot of a task's first tile, and how often the ring has gone round
  auto advance = [&](int& slot, int& round, int by) {  // by at most `slots`
    slot += by;
    if (slot >= p.slots) slot -= p.slots, ++round;
  };

  // what this lane reads of a tile: s and m, of K in the first 16 lanes and of V in the others; codes of K and of V
  const uint32_t par_of = (lane & 15) * p.seg + (lane >> 4) * (stage_bytes >> 1) + p.seg_par + head * 4;
  const uint32_t k_of = g * p.seg + head * (D / 2) + t4 * (D == 64 ? 8 : 16);
  const uint32_t v_of = (stage_bytes >> 1) + (lane & 15) * p.seg + head * (D / 2) + (lane >> 4) * 16;
  int seq = 0;
#pragma unroll 1
  for (int t = me; t < tasks; t += grid, ++seq) {
    __syncthreads();  // the last task is done
    Task* task = reinterpret_cast<Task*>(fixed + S::TASK);
    if (tid == 0) {
      task_call<C>(*shared, prefix, cut, t, task);
      s_bad[(seq + 1) & 1] = 0;
    }
    __syncthreads();
    Task k = *task;
    k.b = uniform(k.b), k.g = uniform(k.g), k.r0 = uniform(k.r0), k.nr = uniform(k.nr), k.tile0 = uniform(k.tile0);
    k.tiles = uniform(k.tiles), k.ctx = uniform(k.ctx), k.span.ns = uniform(k.span.ns), k.span.wp = uniform(k.span.wp);
    k.span.pages = uniform(k.span.pages);
    const int head0 = k.g * p.unit_heads, kv_head = head0 + head;
    // keys of the unit's page list, and the tokens that it leaves out behind the first ones
    const int entries = k.span.pages << p.page_shift, first_keys = k.span.ns << p.page_shift;
    const int skipped = (k.span.wp - k.span.ns) << p.page_shift, key0 = k.tile0 * C::KEYS;
    const int tiles = (min(k.tiles * C::KEYS, entries - key0) + TK - 1) / TK;
    const int32_t* table = p.block_table + (int64_t)k.b * p.max_blocks;

    // ---- copies: whole token rows, or where a unit has some of the heads, their codes, and their s and m, of each row
    int ids = -1, win = -64;  // entries of the page list from `win` on, one a lane
    auto pages_at = [&](int l) {  // page l of the list is in the window
      if (l < win || l >= win + 32) {
        win = l;
        ids = -1;
        if (l + lane < k.span.pages) {
          const int x = l + lane;
          ids = __ldg(table + (x < k.span.ns ? x : k.span.wp + x - k.span.ns));
          if (ids < 0 || (int64_t)ids >= p.num_blocks) {
            ids = -1;
            s_bad[seq & 1] = 1;
          }
        }
        __syncwarp();
      }
    };
    auto issue = [&](int i, int slot, bool again, int parity) {  // tile i into a slot, whose last tile had this parity
      if (again) wattn::bar_wait(empty + 8 * slot, (uint32_t)parity, tries);
      const int from = key0 + i * TK;  // of one page, as a page has 16 tokens at least
      const uint32_t dst = ring_u32 + slot * stage_bytes, bar = full + 8 * slot;
      pages_at(from >> p.page_shift);
      const int id = __shfl_sync(0xffffffffu, ids, (from >> p.page_shift) - win);
      const uint64_t off = (uint64_t)(((uint32_t)max(id, 0) << p.page_shift) + (from & (bs - 1))) * (uint32_t)p.row;
      if (p.head_units == 1) {
        if (lane == 0) {
          const uint32_t bytes = TK * p.seg;
          bar_expect(bar, id < 0 ? 0 : 2 * bytes);
          if (id >= 0) {
            bulk_load(dst, p.k + off, bytes, bar);
            bulk_load(dst + bytes, p.v + off, bytes, bar);
          }
        }
      } else {
        const int heads = min(p.unit_heads, p.kv_heads - head0);
        const uint32_t codes = heads * (D / 2), params = (heads * 4 + 15) & ~15;
        if (lane == 0) bar_expect(bar, id < 0 ? 0 : TK * 2 * (codes + params));
        __syncwarp();
        if (lane < TK && id >= 0) {
          const uint8_t *k_row = p.k + off + lane * (uint32_t)p.row, *v_row = p.v + off + lane * (uint32_t)p.row;
          const uint32_t at = head0 * (D / 2), at_par = p.kv_heads * (D / 2) + head0 * 4;
          const uint32_t to = dst + lane * p.seg, v_to = to + TK * p.seg;
          bulk_load(to, k_row + at, codes, bar);
          bulk_load(to + p.seg_par, k_row + at_par, params, bar);
          bulk_load(v_to, v_row + at, codes, bar);
          bulk_load(v_to + p.seg_par, v_row + at_par, params, bar);
        }
      }
      __syncwarp();
    };
    int turn = pair;  // the pairs issue in turns
    auto issue_from = [&](int i, int slot, int round) {  // tile i, `splits` tiles or a multiple behind the ring's end
      if (turn == 0) {
        turn = p.pairs;
        if (i < tiles) {
          const bool over = slot >= p.slots;
          const int n = round + (over ? 1 : 0);
          issue(i, over ? slot - p.slots : slot, n > 0, n - 1 & 1);
        }
      }
      --turn;
    };
    int slot = slot0, round = round0;  // of this warp's next tile
    advance(slot, round, split);
    if (works) {
#pragma unroll 1
      for (int a = 0; a < p.ahead; ++a) issue_from(split + a * p.splits, slot + a * p.splits, round);
    }

    query_call<C>(*shared, task, queries, qc);
    __syncthreads();

    // ---- state of this lane's rows: g + 8 u of tile mt
    const int r0 = k.r0 + part * p.sub, nr = kv_head < p.kv_heads ? min(p.sub, k.r0 + k.nr - r0) : 0;
    float o[MT][C::TILES][4], extra[MT][4];  // extra: what the products have too much
    float sum[MT][2], offset[MT][2], nref[MT][2], fc[MT][2], fd[MT][2];  // nref: minus the reference; fc, fd: see query_call
    int pos[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int n = 0; n < C::TILES; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][n][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) extra[mt][e] = 0.f;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int r = mt * 16 + u * 8 + g;
        sum[mt][u] = offset[mt][u] = 0.f;
        nref[mt][u] = -wattn::kUnseen;
        fc[mt][u] = qc[pair * 2 * ROWS + r];
        fd[mt][u] = qc[pair * 2 * ROWS + ROWS + r];
        pos[mt][u] = k.ctx - p.rows + (r0 + r) / p.gqa;
      }
    }
    const int low_pos = k.ctx - p.rows + r0 / p.gqa, high_pos = k.ctx - p.rows + (r0 + nr - 1) / p.gqa;
    // tiles that all rows see whole begin at `early` at most, or from `near` to `late`
    int early = low_pos - 15, near = INT32_MAX, late = 0;
    if (p.window != 0) {
      early = min(min(first_keys - 16, p.sinks - 16), early);
      near = max(first_keys, high_pos - p.window + 1 - skipped);
      late = low_pos - 15 - skipped;
    }
    const uint32_t mine = smem_u32(queries) + pair * C::Q_BYTES + lane * 16;
    const int ahead = p.ahead * p.splits;
    bool fresh = true;

#pragma unroll 1
    for (int i = split; i < tiles && works && tries != 1; i += p.splits) {
      issue_from(i + ahead, slot + ahead, round);
      wattn::bar_wait(full + 8 * slot, (uint32_t)(round & 1), tries);
      const uint32_t at = ring_u32 + slot * stage_bytes;
      if (nr > 0) {
        const int where = key0 + i * TK;
        // token of key x of the 16; past the context: none sees it
        auto token = [&](int x) {
          const int tok = where + x + (where < first_keys ? 0 : skipped);
          return tok < k.ctx ? tok : 0x7fffffff;
        };
        auto sees = [&](int position, int tok) {
          return tok <= position && (p.window == 0 || tok < p.sinks || tok > position - p.window);
        };
        const bool whole = where <= early || (where >= near && where <= late);
        // ---- s and m to fp32
        {
          const uint32_t a = lds32(at + par_of);
          float2 x;
          if (p.fp16) x = q4::unpack2<true>(a);
          else x = q4::unpack2<false>(a);
          if (!whole) {  // what no row sees may hold anything
            const int tok = token(lane & 15);
            if (!(tok <= high_pos && (p.window == 0 || tok < p.sinks || tok > low_pos - p.window))) x = make_float2(0.f, 0.f);
          }
          if (lane < 16) x.x *= p.scale_log2, x.y *= p.scale_log2;
          if (lane >= 16) x.y = fmaf(8.f, x.x, x.y);  // the codes of V are taken from 8
          if (lane >= 24) x.x = -x.x;                 // and the last 8 keys' weights are negative (see the product)
          float* to_par = par + ((lane & 15) >> 1) * 8 + (lane >> 4) * 4 + (lane & 1);
          __syncwarp();  // the last ones have been read
          to_par[0] = x.x;
          to_par[2] = x.y;
          __syncwarp();
        }
        // ---- scores: 16 rows x 8 keys an MMA tile. Lane 4 g + t has the codes of key g from word t on: a code c in the low bits
        // of a 16-bit half is the fp16 number c 2^-24, four bits higher c 2^-20, so that a mask makes the operands of two
        // steps out of a word.
        float s[MT][NB][4];
        constexpr int WORDS = D / 32 < 4 ? D / 32 : 4;
#pragma unroll
        for (int section = 0; section < D / 32 / WORDS; ++section) {
          uint32_t w[NB][WORDS];
#pragma unroll
          for (int n8 = 0; n8 < NB; ++n8) {
            const uint32_t from_row = at + k_of + n8 * 8 * p.seg;
            if constexpr (WORDS == 4) {
              const uint4 x = lds128(from_row + section * 64);
              w[n8][0] = x.x, w[n8][1] = x.y, w[n8][2] = x.z, w[n8][3] = x.w;
            } else {
              const uint2 x = lds64(from_row);
              w[n8][0] = x.x, w[n8][1] = x.y;
            }
          }
#pragma unroll
          for (int x = 0; x < WORDS; ++x) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint4 a[MT];
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
                a[mt] = lds128(mine + (mt * C::STEPS + 2 * (section * WORDS + x) + h) * 512);
#pragma unroll
              for (int n8 = 0; n8 < NB; ++n8) {
                const uint32_t z = h ? w[n8][x] >> 8 : w[n8][x], lo = z & 0x000f000fu, hi = z & 0x00f000f0u;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                  if (section + x + h == 0) mma_f16_fresh(s[mt][n8], a[mt].x, a[mt].y, a[mt].z, a[mt].w, lo, hi);
                  else mma_f16(s[mt][n8], a[mt].x, a[mt].y, a[mt].z, a[mt].w, lo, hi);
                }
              }
            }
          }
        }
        // ---- the softmax's weights 2^(score - reference): their sums, and the weights times s as operand A, rows x 16 keys
        // a step
        uint32_t pa[MT][NB / 2][4];
        uint64_t sl[MT][2], soff[MT][2];
        const float* par_at = par + t4 * 8;  // of keys 2 t and 2 t + 1 of a tile
        auto weigh = [&](auto all) {  // whether the weights are too large for their types
          constexpr bool ALL = decltype(all)::value;  // seen by all rows
          uint32_t top = 0;  // two fp16
#pragma unroll
          for (int n8 = 0; n8 < NB; ++n8) {
            const float4 kq = *reinterpret_cast<const float4*>(par_at + n8 * 32);
            const float4 vq = *reinterpret_cast<const float4*>(par_at + n8 * 32 + 4);
            const uint64_t ks = pack_f2(kq.x, kq.y), km = pack_f2(kq.z, kq.w);
            const uint64_t vs = pack_f2(vq.x, vq.y), vm = pack_f2(vq.z, vq.w);
            const int tok0 = ALL ? 0 : token(n8 * 8 + 2 * t4), tok1 = ALL ? 0 : token(n8 * 8 + 2 * t4 + 1);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                // the score, and its distance to the reference: a power of two as the factor leaves one rounding, which is
                // zero at the score that the reference was made of
                uint64_t z = mul_f2(km, pack_f2(fd[mt][u], fd[mt][u]));
                z = fma_f2(ks, pack_f2(s[mt][n8][2 * u], s[mt][n8][2 * u + 1]), z);
                z = fma_f2(z, pack_f2(fc[mt][u], fc[mt][u]), pack_f2(nref[mt][u], nref[mt][u]));
                float2 f = unpack_f2(z), w;
                f.x = fast_exp2(f.x);
                f.y = fast_exp2(f.y);
                if constexpr (ALL) {
                  const uint64_t y = pack_f2(f.x, f.y);
                  w = unpack_f2(mul_f2(y, vs));
                  sl[mt][u] = n8 == 0 ? y : add_f2(sl[mt][u], y);
                  soff[mt][u] = n8 == 0 ? mul_f2(y, vm) : fma_f2(y, vm, soff[mt][u]);
                } else {  // s and m may be NaN: a row that does not see the key keeps clear of them
                  const bool a = sees(pos[mt][u], tok0), b = sees(pos[mt][u], tok1);
                  f.x = a ? f.x : 0.f;
                  f.y = b ? f.y : 0.f;
                  w.x = a ? f.x * vq.x : 0.f;
                  w.y = b ? f.y * vq.y : 0.f;
                  const uint64_t y = pack_f2(f.x, f.y), m = pack_f2(a ? f.x * vq.z : 0.f, b ? f.y * vq.w : 0.f);
                  sl[mt][u] = n8 == 0 ? y : add_f2(sl[mt][u], y);
                  soff[mt][u] = n8 == 0 ? m : add_f2(soff[mt][u], m);
                }
                pa[mt][n8 / 2][(n8 & 1) * 2 + u] = pack_sat(w.x, w.y);
                top = max_abs(top, pa[mt][n8 / 2][(n8 & 1) * 2 + u]);
              }
          }
          float most = 0.f;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const float2 f = unpack_f2(sl[mt][u]);
              most = fmaxf(most, fmaxf(f.x, f.y));
            }
          const float2 f = q4::unpack2<true>(top);
          return fmaxf(f.x, f.y) > C::TOP || most > C::TOP / C::TINY;
        };
#pragma unroll 1
        for (bool settled = false;; settled = true) {
          if (!fresh || settled) {
            const bool grow = whole ? weigh(std::true_type{}) : weigh(std::false_type{});
            if (settled || !__any_sync(0xffffffffu, grow)) break;
          }
          // new references: 2^SHIFT below the largest weight times s of each row, if that is higher; what was summed so far
          // is scaled down. A score of 2^27 or more has no bits for that: its weight is 1, times s as it is. The logarithms are
          // taken ahead of the choice: inside of it they became 16 branches (0.5 to 1.2 us of a small call).
          float below[NB][2];
#pragma unroll
          for (int n8 = 0; n8 < NB; ++n8)
#pragma unroll
            for (int e = 0; e < 2; ++e) below[n8][e] = log2f(fmaxf(fabsf(par_at[n8 * 32 + e + 4]), C::TINY)) - C::SHIFT;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              float m = -INFINITY;
#pragma unroll
              for (int n8 = 0; n8 < NB; ++n8)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const float* of = par_at + n8 * 32 + e;
                  const float z = __fmul_rn(fmaf(of[0], s[mt][n8][2 * u + e], __fmul_rn(of[2], fd[mt][u])), fc[mt][u]);
                  const float ref = z + (fabsf(z) < 0x1p27f ? below[n8][e] : 0.f);
                  if (whole || sees(pos[mt][u], token(n8 * 8 + 2 * t4 + e))) m = fmaxf(m, ref);
                }
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
              const float old = -nref[mt][u], now = fmaxf(old, m), alpha = fast_exp2(old - now);
              nref[mt][u] = -now;
              sum[mt][u] *= alpha;
              offset[mt][u] *= alpha;
              extra[mt][2 * u] *= alpha;
#pragma unroll
              for (int x = 0; x < C::TILES; ++x) {
                o[mt][x][2 * u] *= alpha;
                o[mt][x][2 * u + 1] *= alpha;
              }
            }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float2 a = unpack_f2(sl[mt][u]), b = unpack_f2(soff[mt][u]);
            sum[mt][u] += a.x + a.y;
            offset[mt][u] += b.x + b.y;
          }
        // ---- product with V, 32 head dims at a time. ldmatrix takes 16-bit halves, four codes of neighbouring head dims,
        // and gives a lane those of two keys: the masks leave a pair of keys, operand B, for each of four head dims. The
        // last 8 of 16 keys come as 15 - n with negative weights, -w (15 - n) = w n - 15 w: the sums of the tensor core, which
        // are cut, not rounded, stay near zero. `extra`, 8 w of the first and -7 w of the last keys, is taken off in the end;
        // that leaves the codes taken from 8, so that a weight's rounding meets at most 8 s.
#pragma unroll
        for (int step = 0; step < NB / 2; ++step)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            mma_f16(extra[mt], pa[mt][step][0], pa[mt][step][1], pa[mt][step][2], pa[mt][step][3], 0x48004800u, 0x47004700u);
        fresh = false;
        constexpr int CH = 4 / NB;  // 16-byte chunks of a row that a load takes, of 8 NB keys
        const uint32_t v_u32 = at + v_of;
#pragma unroll
        for (int c = 0; c < D / 32; c += CH) {
          uint32_t r[4];
          ldmatrix_x4_trans(v_u32 + c * 16, r[0], r[1], r[2], r[3]);
#pragma unroll
          for (int ch = 0; ch < CH; ++ch)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t b[NB];
#pragma unroll
              for (int m = 0; m < NB; ++m) {
                const uint32_t z = j & 2 ? r[ch * NB + m] >> 8 : r[ch * NB + m];
                b[m] = (m & 1 ? ~z : z) & (j & 1 ? 0x00f000f0u : 0x000f000fu);
              }
#pragma unroll
              for (int step = 0; step < NB / 2; ++step)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                  mma_f16(o[mt][(c + ch) * 4 + j], pa[mt][step][0], pa[mt][step][1], pa[mt][step][2], pa[mt][step][3],
                          b[2 * step], b[2 * step + 1]);
            }
        }
      }
      __syncwarp();
      if (lane == 0) bar_arrive(empty + 8 * slot);
      advance(slot, round, p.splits);
    }
    // the next task's first slot
    slot0 += tiles;
    round0 += slot0 / p.slots;
    slot0 %= p.slots;
    __syncthreads();  // all tiles have been read
    k = *reinterpret_cast<const Task*>(fixed + S::TASK);
    const bool bad = s_bad[seq & 1] != 0;
    if (bad && tid == 0) raise_error(p.dev_err, SPEC_DEVERR_BLOCK_ID);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int x = 0; x < C::TILES; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[mt][x][e] = fmaf(o[mt][x][e], x & 1 ? 0x1p20f : 0x1p24f, -extra[mt][e & 2]);
    if (p.splits > 1) {  // the other splits' results, by way of the ring, to the first one's warps
      float* box = reinterpret_cast<float*>(smem) + lane;
      if (works && split > 0) {
        float* to = box + ((split - 1) * p.pairs + pair) * C::STATE * 32;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int x = 0; x < C::TILES * 4; ++x) to[(mt * (C::TILES * 4 + 6) + x) * 32] = o[mt][x / 4][x % 4];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float* of = to + (mt * (C::TILES * 4 + 6) + C::TILES * 4 + 3 * u) * 32;
            of[0] = sum[mt][u];
            of[32] = offset[mt][u];
            of[64] = -nref[mt][u];
          }
        }
      }
      __syncthreads();
      if (split == 0) {
#pragma unroll 1
        for (int other = 1; other < p.splits; ++other) {
          const float* from = box + ((other - 1) * p.pairs + pair) * C::STATE * 32;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const float* of = from + (mt * (C::TILES * 4 + 6) + C::TILES * 4 + 3 * u) * 32;
              const float top = fmaxf(-nref[mt][u], of[64]);
              const float a = fast_exp2(-nref[mt][u] - top), b = fast_exp2(of[64] - top);
              nref[mt][u] = -top;
              // of a row that has seen nothing, what it would be added to counts nothing
              sum[mt][u] = sum[mt][u] * a + of[0] * b;
              offset[mt][u] = offset[mt][u] * a + of[32] * b;
#pragma unroll
              for (int x = 0; x < C::TILES * 4; ++x)
                if (((x >> 1) & 1) == u)
                  o[mt][x / 4][x % 4] = o[mt][x / 4][x % 4] * a + from[(mt * (C::TILES * 4 + 6) + x) * 32] * b;
            }
        }
      }
      fence_proxy_async_smem();  // copies write here again
    }
    // ---- results: a lane has 8 neighbouring head dims of its rows
    if (split == 0) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int r = mt * 16 + u * 8 + g;
          float a = sum[mt][u], b = offset[mt][u];
#pragma unroll
          for (int x = 1; x < 4; x <<= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, x);
            b += __shfl_xor_sync(0xffffffffu, b, x);
          }
          if (r >= nr) continue;
          const float inv = k.pieces > 1 && a == 0.f ? 0.f : 1.f / a;
          if (k.pieces == 1) {
            uint4* dst = reinterpret_cast<uint4*>(p.out) + wattn::out_row(p, k.b, kv_head, r0 + r) * (D / 8) + t4;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              float y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] = bad ? 0.f : (o[mt][c * 4 + e % 4][2 * u + e / 4] + b) * inv;
              dst[c * 4] = p.fp16 ? make_uint4(q4::pack2<true>(y[0], y[1]), q4::pack2<true>(y[2], y[3]),
                                               q4::pack2<true>(y[4], y[5]), q4::pack2<true>(y[6], y[7]))
                                  : make_uint4(q4::pack2<false>(y[0], y[1]), q4::pack2<false>(y[2], y[3]),
                                               q4::pack2<false>(y[4], y[5]), q4::pack2<false>(y[6], y[7]));
            }
          } else {
            const int64_t row = ((int64_t)k.slot * p.pairs + pair) * p.sub + r;
            if (t4 == 0) __stcg(p.stat + row, make_float2(-nref[mt][u], bad ? -1.f : a));
            float4* dst = reinterpret_cast<float4*>(p.opart) + row * (D / 4) + t4 * 2;
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                __stcg(dst + c * 8 + e,
                       bad ? make_float4(0.f, 0.f, 0.f, 0.f)
                           : make_float4((o[mt][c * 4][2 * u + e] + b) * inv, (o[mt][c * 4 + 1][2 * u + e] + b) * inv,
                                         (o[mt][c * 4 + 2][2 * u + e] + b) * inv, (o[mt][c * 4 + 3][2 * u + e] + b) * inv));
          }
        }
    }
  }
  if (tries == 1) {  // copies in flight still write here: give them far more time than they take
    raise_error(p.dev_err, SPEC_DEVERR_TIMEOUT);
    __nanosleep(1000000);
  }
}

}  // namespace qattn
}  // namespace specv
