// The paged cache between two tree steps (sm_103a): compaction of the accepted
// path, and the update of the page tables (trim, reserve, free, fork).
#include "tree_device.cuh"

namespace specv {
namespace pages {

// ---------------------------------------------------------------------------
// Compaction of the accepted path
// ---------------------------------------------------------------------------
// K and V of token base + path[j] go to token base + j. The path increases, so
// path[j] >= j: a thread that owns one column of a row's tokens and moves them
// in the order of j, reading a batch of tokens before it writes them, never
// overwrites a token it still has to read, and no two threads share a byte.
constexpr int kPathThreads = 128;
constexpr int kPathBatch = 8;

struct PathParams {
  uint8_t* k;
  uint8_t* v;
  const int32_t* block_table;
  const int32_t* ctx_lens;
  const int32_t* path;
  const int32_t* accept_len;
  int32_t* new_lens;
  int32_t* dev_err;
  int64_t num_blocks, token_bytes;
  int batch, layers, nodes, page, max_blocks;
};

template <typename Vec>
__global__ void __launch_bounds__(kPathThreads) commit_path_kernel(const PathParams p) {
  __shared__ int64_t s_src[tree::kMaxNodes], s_dst[tree::kMaxNodes];
  const int b = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x, N = p.nodes;
  const int ctx = p.ctx_lens[b], m = p.accept_len[b], base = ctx - N;
  int err = 0;
  if (m < -1 || m >= N) err |= SPEC_DEVERR_ACCEPT_LEN;
  if (m >= 0 && (ctx < N || (int64_t)ctx > (int64_t)p.max_blocks * p.page)) err |= SPEC_DEVERR_CTX_LEN;
  bool bad_path = false, bad_page = false;
  if (m >= 0 && err == 0 && tid <= m) {
    const int32_t* path = p.path + (int64_t)b * N;
    const int at = path[tid];
    if (at < 0 || at >= N || (tid == 0 ? at != 0 : path[tid - 1] >= at)) {
      bad_path = true;
    } else {
      const int ts = base + at, td = base + tid;
      const int32_t ps = p.block_table[(int64_t)b * p.max_blocks + ts / p.page];
      const int32_t pd = p.block_table[(int64_t)b * p.max_blocks + td / p.page];
      bad_page = ps < 0 || ps >= p.num_blocks || pd < 0 || pd >= p.num_blocks;
      s_src[tid] = (int64_t)ps * p.page + ts % p.page;
      s_dst[tid] = (int64_t)pd * p.page + td % p.page;
    }
  }
  if (__syncthreads_or(bad_path)) err |= SPEC_DEVERR_ACCEPT_LEN;
  if (__syncthreads_or(bad_page)) err |= SPEC_DEVERR_BLOCK_ID;
  if (layer == 0 && tid == 0) {
    if (err) raise_error(p.dev_err, err);
    p.new_lens[b] = (err || m < 0) ? max(0, base) : base + m + 1;
  }
  if (err) return;
  const int64_t cols = p.token_bytes / (int64_t)sizeof(Vec);
  const int64_t plane = (int64_t)layer * p.num_blocks * p.page;
  for (int64_t c = tid; c < 2 * cols; c += kPathThreads) {
    Vec* buf = reinterpret_cast<Vec*>(c < cols ? p.k : p.v) + (c < cols ? c : c - cols) + plane * cols;
    for (int j0 = 1; j0 <= m; j0 += kPathBatch) {
      Vec x[kPathBatch];
#pragma unroll
      for (int j = 0; j < kPathBatch; ++j)
        if (j0 + j <= m) x[j] = buf[s_src[j0 + j] * cols];
#pragma unroll
      for (int j = 0; j < kPathBatch; ++j)
        if (j0 + j <= m) buf[s_dst[j0 + j] * cols] = x[j];
    }
  }
}

// ---------------------------------------------------------------------------
// Page tables
// ---------------------------------------------------------------------------
constexpr int kTableThreads = 1024;
constexpr int32_t kNeed = -2;  // an entry that waits for a free page

// One row's partly filled page to copy.
struct Copy {
  int32_t src, dst, tokens, pad;
};

struct TableParams {
  int32_t* table;
  int32_t* refs;
  const int32_t* cur;
  const int32_t* want;
  const int32_t* src;
  // workspace
  int32_t* bad;    // [B]
  int32_t* first;  // [B] lowest row that continues from the row
  int32_t* entry;  // [B * W] new entries
  int32_t* free_;  // [B * W] pages handed out, in order
  Copy* copy;      // [B]
  int32_t* dev_err;
  int64_t num_blocks;
  int batch, width, page;
};

__global__ void __launch_bounds__(kTableThreads, 1) update_table_kernel(const TableParams p) {
  __shared__ int32_t s_warp[32];
  __shared__ int32_t s_total;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = p.batch, W = p.width;
  const int64_t E = (int64_t)B * W, room = (int64_t)W * p.page;
  // exclusive prefix of `mine` over the threads; s_total is their sum
  auto prefix = [&](int mine) {
    int incl = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < kTableThreads / 32; ++w) {
      if (w < warp) before += s_warp[w];
      all += s_warp[w];
    }
    if (tid == 0) s_total = all;
    __syncthreads();
    return before + incl - mine;
  };
  auto source = [&](int b) { return p.src ? p.src[b] : b; };

  // 1. rows whose source or lengths are out of range
  for (int b = tid; b < B; b += kTableThreads) {
    const int s = source(b);
    int err = 0;
    if (s < -1 || s >= B) err = SPEC_DEVERR_SRC_ROW;
    else if (s >= 0 && (p.want[b] < 0 || p.want[b] > room || p.cur[s] < 0 || p.cur[s] > room)) err = SPEC_DEVERR_CTX_LEN;
    if (err) raise_error(p.dev_err, err);
    p.bad[b] = err != 0;
    p.first[b] = B;
    p.copy[b] = Copy{-1, -1, 0, 0};
  }
  __syncthreads();
  // 2. kept tokens in entries that name no page
  for (int64_t e = tid; e < E; e += kTableThreads) {
    const int b = (int)(e / W), i = (int)(e - (int64_t)b * W), s = source(b);
    if (p.bad[b] || s < 0) continue;
    if ((int64_t)i * p.page < min(p.cur[s], p.want[b])) {
      const int32_t x = p.table[(int64_t)s * W + i];
      if (x < 0 || x >= p.num_blocks) {
        raise_error(p.dev_err, SPEC_DEVERR_BLOCK_ID);
        p.bad[b] = 1;
      }
    }
  }
  __syncthreads();
  // 3. the row that continues each row
  for (int b = tid; b < B; b += kTableThreads) {
    const int s = source(b);
    if (!p.bad[b] && s >= 0) atomicMin(&p.first[s], b);
  }
  __syncthreads();
  // 4. new entries, and which of them wait for a page
  const int64_t per = (E + kTableThreads - 1) / kTableThreads;
  const int64_t e0 = min(E, tid * per), e1 = min(E, e0 + per);
  int lacking = 0;
  for (int64_t e = e0; e < e1; ++e) {
    const int b = (int)(e / W), i = (int)(e - (int64_t)b * W), s = source(b);
    int32_t x;
    if (p.bad[b]) {
      x = p.table[e];
    } else if (s < 0 || (int64_t)i * p.page >= p.want[b]) {
      x = -1;
    } else {
      const int keep = min(p.cur[s], p.want[b]);
      x = p.table[(int64_t)s * W + i];
      const bool named = x >= 0 && x < p.num_blocks;
      const int owner = (p.bad[s] || source(s) == s) ? s : p.first[s];
      if ((int64_t)(i + 1) * p.page > keep && !(named && owner == b && p.refs[x] == 1)) {
        const int64_t left = (int64_t)keep - (int64_t)i * p.page;
        if (left > 0) p.copy[b] = Copy{x, -1, (int32_t)left, 0};
        x = kNeed;
        ++lacking;
      }
    }
    p.entry[e] = x;
  }
  int rank = prefix(lacking);
  const int total = s_total;
  // 5. references of the entries that changed
  for (int64_t e = e0; e < e1; ++e) {
    const int32_t was = p.table[e], x = p.entry[e];
    if (was == x) continue;
    if (was >= 0 && was < p.num_blocks) atomicSub(&p.refs[was], 1);
    if (x >= 0) atomicAdd(&p.refs[x], 1);
  }
  // a page that is copied from is not handed out in this call: the copy may still read it
  for (int b = tid; b < B; b += kTableThreads)
    if (p.copy[b].src >= 0) atomicAdd(&p.refs[p.copy[b].src], 1);
  __syncthreads();
  // 6. the lowest free pages
  const int64_t pper = (p.num_blocks + kTableThreads - 1) / kTableThreads;
  const int64_t g0 = min(p.num_blocks, tid * pper), g1 = min(p.num_blocks, g0 + pper);
  int zeros = 0;
  for (int64_t g = g0; g < g1; ++g) zeros += __ldcg(&p.refs[g]) == 0;
  int at = prefix(zeros);
  const int found = s_total;
  for (int64_t g = g0; g < g1 && at < total; ++g) {
    if (__ldcg(&p.refs[g]) != 0) continue;
    p.free_[at++] = (int32_t)g;
    p.refs[g] = 1;
  }
  __syncthreads();
  for (int b = tid; b < B; b += kTableThreads)
    if (p.copy[b].src >= 0) atomicSub(&p.refs[p.copy[b].src], 1);
  // 7. the table
  for (int64_t e = e0; e < e1; ++e) {
    int32_t x = p.entry[e];
    if (x == kNeed) {
      const int b = (int)(e / W), i = (int)(e - (int64_t)b * W), s = source(b);
      x = rank < found ? p.free_[rank] : -1;
      if (x < 0) raise_error(p.dev_err, SPEC_DEVERR_NO_PAGE);
      if (min(p.cur[s], p.want[b]) > (int64_t)i * p.page) p.copy[b].dst = x;
      ++rank;
    }
    p.table[e] = x;
  }
}

// Copies of partly filled pages: CTA (b, layer).
constexpr int kCopyThreads = 256;

template <typename Vec>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const Copy* __restrict__ copies, uint8_t* k, uint8_t* v,
                                                                   int64_t num_blocks, int page, int64_t token_bytes) {
  const Copy c = copies[blockIdx.x];
  if (c.dst < 0) return;
  const int64_t cols = token_bytes / (int64_t)sizeof(Vec), n = c.tokens * cols;
  const int64_t plane = (int64_t)blockIdx.y * num_blocks * page * cols;
  for (int side = 0; side < 2; ++side) {
    Vec* buf = reinterpret_cast<Vec*>(side ? v : k) + plane;
    const Vec* from = buf + (int64_t)c.src * page * cols;
    Vec* to = buf + (int64_t)c.dst * page * cols;
    for (int64_t e = threadIdx.x; e < n; e += kCopyThreads) to[e] = from[e];
  }
}

struct Layout {
  size_t first, entry, free_, copy, total;
};

static size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

static Layout layout_for(const spec_cache_desc* d) {
  Layout L;
  const size_t rows = up256((size_t)d->batch * 4), entries = up256((size_t)d->batch * d->max_blocks_per_seq * 4);
  L.first = rows;
  L.entry = 2 * rows;
  L.free_ = L.entry + entries;
  L.copy = L.free_ + entries;
  L.total = L.copy + up256((size_t)d->batch * sizeof(Copy));
  return L;
}

static bool tables_ok(const spec_cache_desc* d) {
  return d != nullptr && d->batch >= 0 && d->block_size >= 1 && d->max_blocks_per_seq >= 1 && d->num_blocks >= 1;
}

static bool tables_supported(const spec_cache_desc* d) {
  return d->block_size <= 65536 && (int64_t)d->batch * d->max_blocks_per_seq <= (1 << 30) && d->num_blocks <= (1 << 30) &&
         (int64_t)d->max_blocks_per_seq * d->block_size <= INT32_MAX;
}

// Bytes that every token row of both caches can be accessed with at once: 16, 4 or 1.
static int vector_bytes(const void* k, const void* v, int64_t token_bytes) {
  const uint64_t bits = reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) | (uint64_t)token_bytes;
  return (bits & 15) == 0 ? 16 : (bits & 3) == 0 ? 4 : 1;
}

}  // namespace pages
}  // namespace specv

using namespace specv;

extern "C" int spec_cache_commit_path(void* k_cache, void* v_cache, const int32_t* block_table, const int32_t* ctx_lens,
                                      const int32_t* path, const int32_t* accept_len, int32_t* new_lens,
                                      int32_t num_nodes, const spec_cache_desc* d, int32_t* dev_err,
                                      spec_stream_t stream_) {
  if (!pages::tables_ok(d) || num_nodes < 1 || d->num_layers < 0 || d->token_bytes < 1) return SPEC_ERR_INVALID_ARG;
  if (d->batch == 0 || d->num_layers == 0) return SPEC_OK;
  if (!k_cache || !v_cache || !block_table || !ctx_lens || !path || !accept_len || !new_lens || new_lens == ctx_lens)
    return SPEC_ERR_INVALID_ARG;
  if (num_nodes > tree::kMaxNodes || !pages::tables_supported(d) || d->num_layers > 65535) return SPEC_ERR_UNSUPPORTED;
  pages::PathParams p;
  p.k = static_cast<uint8_t*>(k_cache);
  p.v = static_cast<uint8_t*>(v_cache);
  p.block_table = block_table;
  p.ctx_lens = ctx_lens;
  p.path = path;
  p.accept_len = accept_len;
  p.new_lens = new_lens;
  p.dev_err = dev_err;
  p.num_blocks = d->num_blocks;
  p.token_bytes = d->token_bytes;
  p.batch = d->batch;
  p.layers = d->num_layers;
  p.nodes = num_nodes;
  p.page = d->block_size;
  p.max_blocks = d->max_blocks_per_seq;
  const dim3 grid((unsigned)d->batch, (unsigned)d->num_layers, 1);
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  switch (pages::vector_bytes(k_cache, v_cache, d->token_bytes)) {
    case 16: pages::commit_path_kernel<uint4><<<grid, pages::kPathThreads, 0, stream>>>(p); break;
    case 4: pages::commit_path_kernel<uint32_t><<<grid, pages::kPathThreads, 0, stream>>>(p); break;
    default: pages::commit_path_kernel<uint8_t><<<grid, pages::kPathThreads, 0, stream>>>(p); break;
  }
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_LAUNCH;
}

extern "C" size_t spec_cache_update_workspace(const spec_cache_desc* d) {
  if (!pages::tables_ok(d) || !pages::tables_supported(d)) return 0;
  return pages::layout_for(d).total;
}

extern "C" int spec_cache_update(int32_t* block_table, int32_t* page_refs, const int32_t* cur_lens,
                                 const int32_t* new_lens, const int32_t* src_rows, void* k_cache, void* v_cache,
                                 const spec_cache_desc* d, void* workspace, size_t workspace_bytes, int32_t* dev_err,
                                 spec_stream_t stream_) {
  if (!pages::tables_ok(d)) return SPEC_ERR_INVALID_ARG;
  const bool copies = k_cache != nullptr;
  if ((v_cache != nullptr) != copies) return SPEC_ERR_INVALID_ARG;
  if (copies && (d->num_layers < 0 || d->token_bytes < 1)) return SPEC_ERR_INVALID_ARG;
  if (d->batch == 0) return SPEC_OK;
  if (!block_table || !page_refs || !cur_lens || !new_lens) return SPEC_ERR_INVALID_ARG;
  if (!pages::tables_supported(d) || (copies && d->num_layers > 65535)) return SPEC_ERR_UNSUPPORTED;
  const pages::Layout L = pages::layout_for(d);
  if (workspace == nullptr || workspace_bytes < L.total) return SPEC_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255) != 0) return SPEC_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  pages::TableParams p;
  p.table = block_table;
  p.refs = page_refs;
  p.cur = cur_lens;
  p.want = new_lens;
  p.src = src_rows;
  p.bad = reinterpret_cast<int32_t*>(ws);
  p.first = reinterpret_cast<int32_t*>(ws + L.first);
  p.entry = reinterpret_cast<int32_t*>(ws + L.entry);
  p.free_ = reinterpret_cast<int32_t*>(ws + L.free_);
  p.copy = reinterpret_cast<pages::Copy*>(ws + L.copy);
  p.dev_err = dev_err;
  p.num_blocks = d->num_blocks;
  p.batch = d->batch;
  p.width = d->max_blocks_per_seq;
  p.page = d->block_size;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  pages::update_table_kernel<<<1, pages::kTableThreads, 0, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return SPEC_ERR_LAUNCH;
  if (!copies || d->num_layers == 0) return SPEC_OK;
  const dim3 grid((unsigned)d->batch, (unsigned)d->num_layers, 1);
  uint8_t *k = static_cast<uint8_t*>(k_cache), *v = static_cast<uint8_t*>(v_cache);
  switch (pages::vector_bytes(k_cache, v_cache, d->token_bytes)) {
    case 16: pages::copy_pages_kernel<uint4><<<grid, pages::kCopyThreads, 0, stream>>>(p.copy, k, v, d->num_blocks, d->block_size, d->token_bytes); break;
    case 4: pages::copy_pages_kernel<uint32_t><<<grid, pages::kCopyThreads, 0, stream>>>(p.copy, k, v, d->num_blocks, d->block_size, d->token_bytes); break;
    default: pages::copy_pages_kernel<uint8_t><<<grid, pages::kCopyThreads, 0, stream>>>(p.copy, k, v, d->num_blocks, d->block_size, d->token_bytes); break;
  }
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_LAUNCH;
}
