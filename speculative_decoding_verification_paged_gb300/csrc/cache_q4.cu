// Storing tokens into a 4-bit cache and reading them back (sm_103a).
//
// Per token and kv head, over its D elements x_e:
//   m = min x,  s = round16((max x - min x) / 15),  n_e = round((x_e - m) / s).
//
// Both directions are bound by HBM: a store reads 2 bytes and writes 1/2 + 4/D
// bytes an element, a load the reverse. A thread holds 8 elements (16 bytes of
// 16-bit values, one word of codes), so that every access of a warp is a run of
// consecutive bytes; the D / 8 lanes of a head find its range by shuffles.
//
// The code is the exact rounding of the quotient. y = (x - m) * (1 / s) in fp32 is
// near enough to place it between two integers f <= y < f + 1; whether it lies
// above f + 1/2 is decided by the sign of t - (f + 1/2) s, t = x - m, which one fma
// gives exactly. Where that is zero, what the subtraction t rounded away decides,
// and then evenness.
#include "launch_memo.h"
#include "q4_device.cuh"

namespace specv {
namespace q4 {

constexpr int kThreads = 256;

struct Params {
  const uint8_t* src[2];  // store: k, v; load: the caches
  uint8_t* dst[2];        // store: the caches; load: k_out, v_out
  int64_t stride[2];      // store: bytes from a token of k (v) to the next
  const int32_t* block_table;
  const int32_t* ctx_lens;
  int32_t* dev_err;
  int64_t num_blocks, row;  // pages; bytes of a token's row
  uint32_t chunks;          // 8-element chunks of all tokens
  uint32_t per_token;       // chunks of a token: Hkv * D / 8
  uint32_t rows;
  int page_shift, max_blocks;
};

// The cache slot of token row n of the call: -1 for padding, -2 for what has an error.
__device__ __forceinline__ int64_t slot_of(const Params& p, uint32_t n, int32_t* err) {
  const uint32_t b = n / p.rows;
  const int ctx = __ldg(p.ctx_lens + b);
  if (ctx < 0 || (int64_t)ctx > ((int64_t)p.max_blocks << p.page_shift)) {
    *err = SPEC_DEVERR_CTX_LEN;
    return -2;
  }
  const int64_t t = (int64_t)ctx - p.rows + (n - b * p.rows);
  if (t < 0) return -1;
  const int page = __ldg(p.block_table + (int64_t)b * p.max_blocks + (t >> p.page_shift));
  if (page < 0 || page >= p.num_blocks) {
    *err = SPEC_DEVERR_BLOCK_ID;
    return -2;
  }
  return ((int64_t)page << p.page_shift) + (t & ((1 << p.page_shift) - 1));
}

// One step of quantising: the code of x, given m, s and 1 / s (all times a power of two of the head where its range is
// close to fp32's ends).
__device__ __forceinline__ uint32_t code_of(float x, float m, float s, float inv) {
  const float t = x - m;
  const float f = floorf(t * inv);
  const float d = fmaf(-(f + 0.5f), s, t);
  bool up = d > 0.f;
  if (d == 0.f) {
    const float r = t - x;
    const float e = (x - (t - r)) - (m + r);  // x - m - t, exactly
    up = e > 0.f || (e == 0.f && ((int)f & 1));
  }
  return (uint32_t)min((int)f + (up ? 1 : 0), 15);
}

template <int D, bool FP16>
__global__ void __launch_bounds__(kThreads) cache_store_q4_kernel(const Params p) {
  constexpr int L = D / 8;  // lanes of a head
  const uint32_t c = blockIdx.x * kThreads + threadIdx.x;
  int64_t slot = -1;
  uint32_t n = 0, at = 0;
  int32_t err = 0;
  if (c < p.chunks) {
    n = c / p.per_token;
    at = c - n * p.per_token;
    slot = slot_of(p, n, &err);
    if (err != 0 && at == 0) raise_error(p.dev_err, err);
  }
  uint4 raw[2] = {};
  if (slot >= 0) {
#pragma unroll
    for (int w = 0; w < 2; ++w) raw[w] = __ldcs(reinterpret_cast<const uint4*>(p.src[w] + (int64_t)n * p.stride[w]) + at);
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float x[8];
    const uint32_t words[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<FP16>(words[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
    float lo = x[0], hi = x[0], sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo = fminf(lo, x[i]);
      hi = fmaxf(hi, x[i]);
      sum += fabsf(x[i]) * 0.f;  // NaN if one of them is no number or infinite
    }
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    float range = __fsub_rn(hi, lo);
    // half the range over half of 15 is the same number, in reach of fp32 for every bf16 range
    const float q = range <= 3e38f ? __fdiv_rn(range, 15.f) : __fdiv_rn(__fsub_rn(0.5f * hi, 0.5f * lo), 7.5f);
    uint32_t par = pack2<FP16>(q, lo), code = 0;
    const float s16 = unpack2<FP16>(par).x;
    if (sum != 0.f) {
      par = FP16 ? 0x7e007e00u : 0x7fc07fc0u;  // both NaN
    } else if (s16 > 0.f) {
      const float scale = s16 < 0x1p-60f ? 0x1p90f : s16 > 0x1p100f ? 0x1p-30f : 1.f;
      const float s = s16 * scale, m = lo * scale, inv = 1.f / s;
#pragma unroll
      for (int i = 0; i < 8; ++i) code |= code_of(x[i] * scale, m, s, inv) << (4 * i);
    }
    if (slot >= 0) {
      uint32_t* row = reinterpret_cast<uint32_t*>(p.dst[w] + slot * p.row);
      row[at] = code;
      if (at % L == 0) row[p.per_token + at / L] = par;
    }
  }
}

template <int D, bool FP16, bool F32>
__global__ void __launch_bounds__(kThreads) cache_load_q4_kernel(const Params p) {
  constexpr int L = D / 8;
  const uint32_t c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= p.chunks) return;
  const uint32_t n = c / p.per_token, at = c - n * p.per_token;
  int32_t err = 0;
  const int64_t slot = slot_of(p, n, &err);
  if (err != 0 && at == 0) raise_error(p.dev_err, err);
  uint32_t code[2] = {}, par[2] = {};
  if (slot >= 0) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint32_t* row = reinterpret_cast<const uint32_t*>(p.src[w] + slot * p.row);
      code[w] = __ldcs(row + at);
      par[w] = __ldg(row + p.per_token + at / L);
    }
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const float2 sm = unpack2<FP16>(par[w]);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fmaf((float)((code[w] >> (4 * i)) & 15u), sm.x, sm.y);
    if constexpr (F32) {
      float4* out = reinterpret_cast<float4*>(p.dst[w]) + (int64_t)c * 2;
      __stcs(out, make_float4(x[0], x[1], x[2], x[3]));
      __stcs(out + 1, make_float4(x[4], x[5], x[6], x[7]));
    } else {
      __stcs(reinterpret_cast<uint4*>(p.dst[w]) + c,
             make_uint4(pack2<FP16>(x[0], x[1]), pack2<FP16>(x[2], x[3]), pack2<FP16>(x[4], x[5]), pack2<FP16>(x[6], x[7])));
    }
  }
}

// What both calls check and fill in; SPEC_OK with p.chunks = 0 where there is nothing to do.
static int params_for(Params& p, const int32_t* block_table, const int32_t* ctx_lens, int32_t num_rows, int32_t dtype,
                      const spec_attn_desc* d, int32_t* dev_err) {
  if (d == nullptr || d->batch < 0 || d->num_kv_heads < 1 || d->max_blocks_per_seq < 1 || d->num_blocks < 1 || num_rows < 1)
    return SPEC_ERR_INVALID_ARG;
  if (dtype != SPEC_DTYPE_BF16 && dtype != SPEC_DTYPE_FP16) return SPEC_ERR_INVALID_ARG;
  p.chunks = 0;
  if (d->batch == 0) return SPEC_OK;
  const int D = d->head_dim, bs = d->block_size;
  if (D != 64 && D != 128 && D != 256) return SPEC_ERR_UNSUPPORTED;
  if (bs != 16 && bs != 32 && bs != 64 && bs != 128) return SPEC_ERR_UNSUPPORTED;
  if (spec_q4_row_bytes(d->num_kv_heads, D) == 0) return SPEC_ERR_UNSUPPORTED;
  const int64_t per_token = (int64_t)d->num_kv_heads * (D / 8), tokens = (int64_t)d->batch * num_rows;
  if (tokens > INT32_MAX / per_token) return SPEC_ERR_UNSUPPORTED;
  if (d->num_blocks > INT32_MAX / bs || (int64_t)d->max_blocks_per_seq * bs > (1 << 30)) return SPEC_ERR_UNSUPPORTED;
  if (block_table == nullptr || ctx_lens == nullptr) return SPEC_ERR_INVALID_ARG;
  p.block_table = block_table;
  p.ctx_lens = ctx_lens;
  p.dev_err = dev_err;
  p.num_blocks = d->num_blocks;
  p.row = row_bytes(d->num_kv_heads, D);
  p.per_token = (uint32_t)per_token;
  p.chunks = (uint32_t)(tokens * per_token);
  p.rows = (uint32_t)num_rows;
  p.max_blocks = d->max_blocks_per_seq;
  for (p.page_shift = 0; (1 << p.page_shift) < bs;) ++p.page_shift;
  return SPEC_OK;
}

static bool aligned16(const void* a, const void* b, const void* c, const void* d) {
  return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) | reinterpret_cast<uintptr_t>(c) |
           reinterpret_cast<uintptr_t>(d)) & 15) == 0;
}

template <int D>
static void launch_store(const Params& p, bool fp16, cudaStream_t stream) {
  const unsigned grid = (p.chunks + kThreads - 1) / kThreads;
  if (fp16) cache_store_q4_kernel<D, true><<<grid, kThreads, 0, stream>>>(p);
  else cache_store_q4_kernel<D, false><<<grid, kThreads, 0, stream>>>(p);
}
template <int D>
static void launch_load(const Params& p, bool fp16, bool f32, cudaStream_t stream) {
  const unsigned grid = (p.chunks + kThreads - 1) / kThreads;
  if (fp16 && f32) cache_load_q4_kernel<D, true, true><<<grid, kThreads, 0, stream>>>(p);
  else if (fp16) cache_load_q4_kernel<D, true, false><<<grid, kThreads, 0, stream>>>(p);
  else if (f32) cache_load_q4_kernel<D, false, true><<<grid, kThreads, 0, stream>>>(p);
  else cache_load_q4_kernel<D, false, false><<<grid, kThreads, 0, stream>>>(p);
}

}  // namespace q4
}  // namespace specv

using namespace specv;

extern "C" int64_t spec_q4_row_bytes(int32_t num_kv_heads, int32_t head_dim) {
  if (num_kv_heads < 1 || num_kv_heads > 65536) return 0;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
  return q4::row_bytes(num_kv_heads, head_dim);
}

extern "C" int spec_cache_store_q4(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                                   const int32_t* block_table, const int32_t* ctx_lens, int32_t num_rows, void* k_cache,
                                   void* v_cache, int32_t dtype, const spec_attn_desc* d, int32_t* dev_err,
                                   spec_stream_t stream_) {
  q4::Params p;
  const int rc = q4::params_for(p, block_table, ctx_lens, num_rows, dtype, d, dev_err);
  if (rc != SPEC_OK || p.chunks == 0) return rc;
  if (!k || !v || !k_cache || !v_cache || k_cache == v_cache || !q4::aligned16(k, v, k_cache, v_cache))
    return SPEC_ERR_INVALID_ARG;
  const int64_t least = (int64_t)d->num_kv_heads * d->head_dim;
  if (k_stride < least || v_stride < least || ((k_stride | v_stride) & 7) != 0) return SPEC_ERR_INVALID_ARG;
  p.src[0] = static_cast<const uint8_t*>(k);
  p.src[1] = static_cast<const uint8_t*>(v);
  p.stride[0] = k_stride * 2;
  p.stride[1] = v_stride * 2;
  p.dst[0] = static_cast<uint8_t*>(k_cache);
  p.dst[1] = static_cast<uint8_t*>(v_cache);
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const bool fp16 = dtype == SPEC_DTYPE_FP16;
  switch (d->head_dim) {
    case 64: q4::launch_store<64>(p, fp16, stream); break;
    case 128: q4::launch_store<128>(p, fp16, stream); break;
    default: q4::launch_store<256>(p, fp16, stream); break;
  }
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_LAUNCH;
}

extern "C" int spec_cache_load_q4(const void* k_cache, const void* v_cache, const int32_t* block_table,
                                  const int32_t* ctx_lens, int32_t num_rows, void* k_out, void* v_out, int32_t dtype,
                                  int32_t out_dtype, const spec_attn_desc* d, int32_t* dev_err, spec_stream_t stream_) {
  q4::Params p;
  const int rc = q4::params_for(p, block_table, ctx_lens, num_rows, dtype, d, dev_err);
  if (rc != SPEC_OK) return rc;
  if (out_dtype != dtype && out_dtype != SPEC_DTYPE_FP32) return SPEC_ERR_INVALID_ARG;
  if (p.chunks == 0) return SPEC_OK;
  if (!k_cache || !v_cache || !k_out || !v_out || k_out == v_out || !q4::aligned16(k_cache, v_cache, k_out, v_out))
    return SPEC_ERR_INVALID_ARG;
  p.src[0] = static_cast<const uint8_t*>(k_cache);
  p.src[1] = static_cast<const uint8_t*>(v_cache);
  p.stride[0] = p.stride[1] = 0;
  p.dst[0] = static_cast<uint8_t*>(k_out);
  p.dst[1] = static_cast<uint8_t*>(v_out);
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const bool fp16 = dtype == SPEC_DTYPE_FP16, f32 = out_dtype == SPEC_DTYPE_FP32;
  switch (d->head_dim) {
    case 64: q4::launch_load<64>(p, fp16, f32, stream); break;
    case 128: q4::launch_load<128>(p, fp16, f32, stream); break;
    default: q4::launch_load<256>(p, fp16, f32, stream); break;
  }
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_LAUNCH;
}
