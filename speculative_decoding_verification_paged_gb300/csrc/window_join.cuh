// The join of the units that the attention kernels over a window cut into pieces.
#pragma once

#include "window_plan.cuh"

namespace specv {
namespace wattn {

constexpr int kJoinThreads = 128;

// out = sum of W_w opart_w over the pieces w of a unit, in their order, over the sum of W_w = 2^(reference_w unit) sum_w; zeros if a
// piece has no result. References and sums come apart: next to a large reference log2 of a sum has no bits left. A piece
// without a visible key has sum 0 and holds zeros. D / 4 threads for a row, four head dims each; a block joins some rows, or
// (`split`) one, whose pieces its groups of threads take in turns.
//
// A kernel of its own: the block that happens to finish a unit's last piece would have to read 2.5 to 8 us' worth of
// partial results at the latency of L2 by itself, on code that it meets for the first time (15 us measured for 64 pieces of
// 32 rows); here all SMs share in it.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ Params p, int split) {
  constexpr int L = D / 4, GROUP = L < 32 ? L : 32, GROUPS = kJoinThreads / L, AT_ONCE = 8;
  __shared__ float4 s_part[kJoinThreads];
  __shared__ float s_sum[GROUPS];
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  if ((int)blockIdx.x >= __ldcg(&p.cut_units[0].b)) return;
  const CutUnit u = p.cut_units[1 + blockIdx.x];
  const int c = threadIdx.x % L, group = threadIdx.x / L, rows = p.pairs * p.sub, lane = threadIdx.x % GROUP;
  const int r = split ? (int)blockIdx.y : (int)blockIdx.y * GROUPS + group, part = split ? group : 0, parts = split ? GROUPS : 1;
  const int of_pair = r * p.by_sub >> 16, h = of_pair * p.by_parts >> 8, R = u.r0 - h * p.per + r, g = u.g * p.unit_heads + h;
  const bool there = r < rows && R < u.r0 + u.nr && g < p.kv_heads;
  if (split && !there) return;
  const int first = there ? r : 0;  // the threads of a row that is not there go along
  const float2* stat = p.stat + (int64_t)u.first * rows + first;
  const float4* src = reinterpret_cast<const float4*>(p.opart) + ((int64_t)u.first * rows + first) * L + c;
  const int64_t step = (int64_t)rows * L;
  float top = -INFINITY, least = 0.f;  // of the references, and of the sums
#pragma unroll 4
  for (int w = lane; w < u.pieces; w += GROUP) {
    const float2 x = __ldcg(stat + (int64_t)w * rows);
    top = fmaxf(top, x.x);
    least = fminf(least, x.y);
  }
#pragma unroll
  for (int o = 1; o < GROUP; o <<= 1) {
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
  }
  // this group's are the pieces part, part + parts, ...; the groups of a warp take as many steps, the last with weight 0
  const int steps = (u.pieces + parts - 1) / parts;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
#pragma unroll 1
  for (int w0 = 0; w0 < steps; w0 += GROUP) {
    const int piece = part + (w0 + lane) * parts;
    float weight = 0.f;
    if (piece < u.pieces) {
      const float2 x = __ldcg(stat + (int64_t)piece * rows);
      weight = exp2f((x.x - top) * p.ref_unit) * x.y;
    }
    sum += weight;
#pragma unroll 1
    for (int w1 = 0; w1 < GROUP && w0 + w1 < steps; w1 += AT_ONCE) {
      float4 y[AT_ONCE];
#pragma unroll
      for (int w = 0; w < AT_ONCE; ++w) y[w] = __ldcg(src + min(part + (w0 + w1 + w) * parts, u.pieces - 1) * step);
#pragma unroll
      for (int w = 0; w < AT_ONCE; ++w) {
        const float f = __shfl_sync(0xffffffffu, weight, w1 + w, GROUP);
        a.x = fmaf(f, y[w].x, a.x);
        a.y = fmaf(f, y[w].y, a.y);
        a.z = fmaf(f, y[w].z, a.z);
        a.w = fmaf(f, y[w].w, a.w);
      }
    }
  }
#pragma unroll
  for (int o = 1; o < GROUP; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (split) {
    s_part[threadIdx.x] = a;
    if (c == 0) s_sum[group] = sum;
    __syncthreads();
    if (group > 0) return;
#pragma unroll 1
    for (int x = 1; x < GROUPS; ++x) {
      const float4 y = s_part[x * L + c];
      a = make_float4(a.x + y.x, a.y + y.y, a.z + y.z, a.w + y.w);
      sum += s_sum[x];
    }
  }
  if (!there) return;
  const float inv = 1.f / sum;  // the row is NaN where all its scores are -inf, as in one piece
  a = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
  // Chosen, not a product with 0: what the pieces hold beside a bad page may be NaN.
  if (least < 0.f) a = make_float4(0.f, 0.f, 0.f, 0.f);
  reinterpret_cast<uint2*>(p.out)[out_row(p, u.b, g, R) * L + c] =
      p.fp16 ? make_uint2(q4::pack2<true>(a.x, a.y), q4::pack2<true>(a.z, a.w))
             : make_uint2(q4::pack2<false>(a.x, a.y), q4::pack2<false>(a.z, a.w));
}

// Behind the attention on its stream; its blocks may be there before the attention's have ended, and wait for them.
template <int D>
static int launch_join(const Params& p, int max_pieces, cudaStream_t stream) {
  const int64_t units = (int64_t)p.batch * p.head_units * p.groups;
  const int lists = (int)(units < max_pieces / 2 ? units : max_pieces / 2), rows = p.pairs * p.sub, groups = kJoinThreads / (D / 4);
  // One row a block where few units are cut, and so into many pieces; else a block has a row for each group. Over 4 bits, 128
  // rows a unit: one sequence of 8192 tokens 29 us, 36 with a row a group; two 32 and 38, four 35 and 37, eight of 2048 tokens
  // 31 both, 16 of them 37 and 35. 16 bits, 128 rows a sequence: four of 8192 tokens 39 both, eight of 4096 tokens 41 and 39.
  const int split = (int64_t)lists * rows <= 1000 ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)lists, (unsigned)(split ? rows : (rows + groups - 1) / groups));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<D>, p, split) == cudaSuccess ? SPEC_OK : SPEC_ERR_LAUNCH;
}

}  // namespace wattn
}  // namespace specv
