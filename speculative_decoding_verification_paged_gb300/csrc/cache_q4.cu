// Storing tokens into a 4-bit cache and reading them back (sm_103a).
//
// Per token and kv head, over its D elements x_e:
//   m = min x,  s = round16((max x - min x) / 15),  n_e = round((x_e - m) / s).
//
// A store reads 2 bytes and writes 1/2 + 4/D bytes an element, a load the reverse. A
// thread holds 8 elements (16 bytes of 16-bit values, one word of codes), so that
// every access of a warp is a run of consecutive bytes; the D / 8 lanes of a head find
// its range by shuffles, least and negated greatest in the halves of one word.
//
// A load comes to 81% of the copy rate: 65,536 tokens of 8 heads of 128, 340 MB, in 62 us (56
// among other calls, whose starts and ends overlap). A store is bound by instructions, 423 a warp
// for 256 elements of K and of V, 72% of the issue slots used: the same 340 MB, 50 us' worth at
// the copy rate, in 127 us (115 among others). fp32 results are 608 MB in 136 us.
// Each element rounded by floor and an exact comparison took 1.6 times as long. Small calls are
// launches: 10 us with the host's work for 512 tokens, 2 to 3 in a graph.
//
// The code is the exact rounding of the quotient: see codes_of.
#include "launch_memo.h"
#include "pairs.cuh"
#include "q4_device.cuh"

namespace specv {
namespace q4 {

constexpr int kThreads = 256;

// Quotients by d of numbers below 2^31, by a product.
struct Quotient {
  uint32_t mul, shift, d;  // mul 0: d is 1
  __device__ __forceinline__ uint32_t of(uint32_t x) const { return mul == 0 ? x : __umulhi(x, mul) >> shift; }
};
// mul = floor(2^(31 + s) / d) + 1 with 2^s >= d: mul d is above 2^(31 + s) by 2^s at most, so that for x < 2^31 the product
// x mul / 2^(31 + s) is above x / d by less than 1 / d.
static Quotient quotient_by(uint32_t d) {
  Quotient q = {0, 0, d};
  if (d == 1) return q;
  while ((1u << q.shift) < d) ++q.shift;
  q.mul = (uint32_t)((uint64_t(1) << (31 + q.shift)) / d + 1);
  --q.shift;
  return q;
}

struct Params {
  const uint8_t* src[2];  // store: k, v; load: the caches
  uint8_t* dst[2];        // store: the caches; load: k_out, v_out
  int64_t stride[2];      // store: bytes from a token of k (v) to the next
  const int32_t* block_table;
  const int32_t* ctx_lens;
  int32_t* dev_err;
  uint32_t num_blocks, row;  // pages; bytes of a token's row
  uint32_t chunks;          // 8-element chunks of all tokens
  Quotient per_token;       // chunks of a token: Hkv * D / 8
  Quotient rows;
  uint32_t tokens;
  int page_shift, max_blocks, max_tokens;
};

// The cache slot of token row n of the call: -1 for padding, -2 for what has an error.
__device__ __forceinline__ int slot_of(const Params& p, uint32_t n, int32_t* err) {
  const uint32_t b = p.rows.of(n);
  const int ctx = __ldg(p.ctx_lens + b);
  if (ctx < 0 || ctx > p.max_tokens) {
    *err = SPEC_DEVERR_CTX_LEN;
    return -2;
  }
  const int t = ctx - (int)p.rows.d + (int)(n - b * p.rows.d);
  if (t < 0) return -1;
  const int page = __ldg(p.block_table + (int64_t)b * p.max_blocks + (t >> p.page_shift));
  if ((uint32_t)page >= p.num_blocks) {
    *err = SPEC_DEVERR_BLOCK_ID;
    return -2;
  }
  return (page << p.page_shift) + (t & ((1 << p.page_shift) - 1));
}

// The code of x, given m, s and 1 / s (all times a power of two of the head where its range is close to fp32's ends). y =
// (x - m) * (1 / s) is near enough to place the quotient between two integers f <= y < f + 1; whether it lies above f + 1/2
// is decided by the sign of t - (f + 1/2) s, t = x - m, which one fma gives exactly. Where that is zero, what the
// subtraction t rounded away decides, and then evenness.
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

// The smaller one of each half of two words of 16-bit floats; NaN if one is NaN.
template <bool FP16>
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (FP16) asm("min.NaN.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  else asm("min.NaN.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The codes of 8 elements of a head, given m and s > 0. A quotient y = (x - m) / s to within two units of its last place
// comes from the reciprocal and one step of correction, in pairs of fp32; adding 1.5 2^23 rounds it to an integer, halves to
// even. That is the rounding of the quotient itself unless y lies within 2^-19 of a half; if it is one, and x - m and
// y s have no rounding (most halves of real inputs are such), it is right, too. What is left goes the exact way (code_of),
// as does a head whose s is so coarse that quotients reach 15 1/4 and more, or lies near the ends of fp32.
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8], float m, float s, float range) {
  constexpr float MAGIC = 12582912.f;
  const float inv = __fdividef(1.f, s);
  uint32_t code = 0;
  bool exact = true;
  if (s >= 0x1p-60f && s <= 0x1p100f && range * inv < 15.25f) {
    const uint64_t m2 = pack_f2(-m, -m), inv2 = pack_f2(inv, inv), s2 = pack_f2(-s, -s);
    const uint64_t up = pack_f2(MAGIC, MAGIC), down = pack_f2(-MAGIC, -MAGIC), sign = pack_f2(-1.f, -1.f);
    uint64_t t[4], y[4], d[4];
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t[i] = add_f2(pack_f2(x[2 * i], x[2 * i + 1]), m2);
      const uint64_t y0 = mul_f2(t[i], inv2);
      y[i] = fma_f2(fma_f2(y0, s2, t[i]), inv2, y0);
      const uint64_t r = add_f2(y[i], up);
      d[i] = fma_f2(add_f2(r, down), sign, y[i]);
      const float2 e = unpack_f2(d[i]), n = unpack_f2(r);
      most = fmaxf(most, fmaxf(fabsf(e.x), fabsf(e.y)));
      code += (__float_as_uint(n.x) << 8 * i) + (__float_as_uint(n.y) << 8 * i + 4);
    }
    code -= 0x3f400000u;  // the bits of MAGIC, shifted by 0, 4 and 8 (by more they have left the word)
    if (most >= 0.5f - 0x1p-19f) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 e = unpack_f2(d[i]), q = unpack_f2(y[i]), u = unpack_f2(t[i]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float a = fabsf(h ? e.y : e.x), b = h ? q.y : q.x, v = h ? u.y : u.x, z = x[2 * i + h];
          // v = z - m: exact if neither way back has a rounding
          const bool half = a == 0.5f && fmaf(-b, s, v) == 0.f && v + m == z && z - v == m;
          exact &= a < 0.5f - 0x1p-19f || half;
        }
      }
    }
    if (exact) return code;
  }
  const float scale = s < 0x1p-60f ? 0x1p90f : s > 0x1p100f ? 0x1p-30f : 1.f, ss = s * scale, by_ss = 1.f / ss;
  code = 0;
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    float z = x[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) z = i == j ? x[j] : z;
    code |= code_of(z * scale, m * scale, ss, by_ss) << (4 * i);
  }
  return code;
}

template <int D, bool FP16>
__global__ void __launch_bounds__(kThreads) cache_store_q4_kernel(const Params p) {
  constexpr int L = D / 8;  // lanes of a head
  const uint32_t c = blockIdx.x * kThreads + threadIdx.x, n = p.per_token.of(c), at = c - n * p.per_token.d;
  int slot = -1;
  if (n < p.tokens) {
    int32_t err = 0;
    slot = slot_of(p, n, &err);
    if (err != 0 && at == 0) raise_error(p.dev_err, err);
  }
  if (!__any_sync(0xffffffffu, slot >= 0)) return;
  uint4 raw[2] = {};
  if (slot >= 0) {
#pragma unroll
    for (int w = 0; w < 2; ++w) raw[w] = __ldcs(reinterpret_cast<const uint4*>(p.src[w] + (int64_t)n * p.stride[w]) + at);
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const uint32_t words[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
    // the range of the head, as the least of the elements and of their negatives, in the halves of a word
    uint32_t low = words[0], neg = words[0] ^ 0x80008000u;
#pragma unroll
    for (int i = 1; i < 4; ++i) {
      low = min2_nan<FP16>(low, words[i]);
      neg = min2_nan<FP16>(neg, words[i] ^ 0x80008000u);
    }
    low = min2_nan<FP16>(__byte_perm(low, neg, 0x5410), __byte_perm(low, neg, 0x7632));
#pragma unroll
    for (int o = 1; o < L; o <<= 1) low = min2_nan<FP16>(low, __shfl_xor_sync(0xffffffffu, low, o));
    const float2 ends = unpack2<FP16>(low);
    const float lo = ends.x, hi = -ends.y, range = __fsub_rn(hi, lo);
    // half the range over half of 15 is the same number, in reach of fp32 for every bf16 range
    const float q = range <= 3e38f ? __fdiv_rn(range, 15.f) : __fdiv_rn(__fsub_rn(0.5f * hi, 0.5f * lo), 7.5f);
    uint32_t par = pack2<FP16>(q, lo), code = 0;
    const float s16 = unpack2<FP16>(par).x;
    if (!(fabsf(lo) < INFINITY && fabsf(hi) < INFINITY)) {
      par = FP16 ? 0x7e007e00u : 0x7fc07fc0u;  // both NaN
    } else if (s16 > 0.f) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<FP16>(words[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
      code = codes_of(x, lo, s16, range);
    }
    if (slot >= 0) {
      uint32_t* row = reinterpret_cast<uint32_t*>(p.dst[w] + (uint64_t)(uint32_t)slot * p.row);
      row[at] = code;
      if (at % L == 0) row[p.per_token.d + at / L] = par;
    }
  }
}

// T tokens a thread, `groups` tokens apart.
template <int D, bool FP16, bool F32, int T>
__global__ void __launch_bounds__(kThreads) cache_load_q4_kernel(const Params p, uint32_t groups) {
  constexpr int L = D / 8;
  const uint32_t c = blockIdx.x * kThreads + threadIdx.x, n0 = p.per_token.of(c), at = c - n0 * p.per_token.d;
  if (n0 >= groups) return;
  uint32_t code[T][2] = {}, par[T][2] = {};
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const uint32_t n = n0 + t * groups;
    if (T > 1 && n >= p.tokens) break;
    int32_t err = 0;
    const int slot = slot_of(p, n, &err);
    if (err != 0 && at == 0) raise_error(p.dev_err, err);
    if (slot >= 0) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint32_t* row = reinterpret_cast<const uint32_t*>(p.src[w] + (uint64_t)(uint32_t)slot * p.row);
        code[t][w] = __ldcs(row + at);
        par[t][w] = __ldg(row + p.per_token.d + at / L);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const uint32_t n = n0 + t * groups;
    if (T > 1 && n >= p.tokens) break;
    const uint32_t chunk = n * p.per_token.d + at;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const float2 sm = unpack2<FP16>(par[t][w]);
      const uint64_t s = pack_f2(sm.x, sm.x), m = pack_f2(sm.y, sm.y), base = pack_f2(-8388608.f, -8388608.f);
      const uint32_t even = code[t][w] & 0x0f0f0f0fu, odd = code[t][w] >> 4 & 0x0f0f0f0fu;
      float x[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // a byte n behind 0x4b0000 is the float 2^23 + n
        const uint64_t n2 = pack_f2(__uint_as_float(__byte_perm(even, 0x4b000000u, 0x7440 | i)),
                                    __uint_as_float(__byte_perm(odd, 0x4b000000u, 0x7440 | i)));
        const float2 f = unpack_f2(fma_f2(add_f2(n2, base), s, m));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
      if constexpr (F32) {
        float4* out = reinterpret_cast<float4*>(p.dst[w]) + (int64_t)chunk * 2;
        __stcs(out, make_float4(x[0], x[1], x[2], x[3]));
        __stcs(out + 1, make_float4(x[4], x[5], x[6], x[7]));
      } else {
        __stcs(reinterpret_cast<uint4*>(p.dst[w]) + chunk,
               make_uint4(pack2<FP16>(x[0], x[1]), pack2<FP16>(x[2], x[3]), pack2<FP16>(x[4], x[5]), pack2<FP16>(x[6], x[7])));
      }
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
  p.num_blocks = (uint32_t)d->num_blocks;
  p.row = (uint32_t)row_bytes(d->num_kv_heads, D);
  p.per_token = quotient_by((uint32_t)per_token);
  p.chunks = (uint32_t)(tokens * per_token);
  p.rows = quotient_by((uint32_t)num_rows);
  p.tokens = (uint32_t)tokens;
  p.max_blocks = d->max_blocks_per_seq;
  p.max_tokens = d->max_blocks_per_seq * bs;
  for (p.page_shift = 0; (1 << p.page_shift) < bs;) ++p.page_shift;
  return SPEC_OK;
}

static bool aligned16(const void* a, const void* b, const void* c, const void* d) {
  return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) | reinterpret_cast<uintptr_t>(c) |
           reinterpret_cast<uintptr_t>(d)) & 15) == 0;
}

static unsigned blocks_for(const Params& p, uint32_t tokens) {
  return (unsigned)(((int64_t)tokens * p.per_token.d + kThreads - 1) / kThreads);
}

template <int D>
static void launch_store(const Params& p, bool fp16, cudaStream_t stream) {
  if (fp16) cache_store_q4_kernel<D, true><<<blocks_for(p, p.tokens), kThreads, 0, stream>>>(p);
  else cache_store_q4_kernel<D, false><<<blocks_for(p, p.tokens), kThreads, 0, stream>>>(p);
}
template <int D, bool FP16, bool F32>
static void launch_load_as(const Params& p, cudaStream_t stream) {
  // Four tokens a thread keep more loads on their way; a call too small to fill the GPU that way is better off with one. 65,536
  // tokens of 8 heads of 128 take 62 us, 66 with one a thread; 32,768 (4 M chunks) 35 both, 24,576 29 and 27.
  const uint32_t groups = p.chunks >= 4u << 20 ? (p.tokens + 3) / 4 : p.tokens;
  if (groups < p.tokens) cache_load_q4_kernel<D, FP16, F32, 4><<<blocks_for(p, groups), kThreads, 0, stream>>>(p, groups);
  else cache_load_q4_kernel<D, FP16, F32, 1><<<blocks_for(p, groups), kThreads, 0, stream>>>(p, groups);
}
template <int D>
static void launch_load(const Params& p, bool fp16, bool f32, cudaStream_t stream) {
  if (fp16 && f32) launch_load_as<D, true, true>(p, stream);
  else if (fp16) launch_load_as<D, true, false>(p, stream);
  else if (f32) launch_load_as<D, false, true>(p, stream);
  else launch_load_as<D, false, false>(p, stream);
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
