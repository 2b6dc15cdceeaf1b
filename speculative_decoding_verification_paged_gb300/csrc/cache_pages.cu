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
// In a graph one layer takes 2 us; 32 layers of batch 32 (34 MB moved, 4.9 us at copy
// rate) 6 us warm and 11 us a call, of which the host's part is about 9 us.
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
  int nodes, page, max_blocks;
};

template <typename Vec>
__global__ void __launch_bounds__(kPathThreads) commit_path_kernel(const PathParams p) {
  __shared__ int64_t s_src[tree::kMaxNodes], s_dst[tree::kMaxNodes];
  const int b = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x, N = p.nodes;
  const int ctx = p.ctx_lens[b], m = p.accept_len[b], base = ctx < N ? 0 : ctx - N;  // (rows that
  // moved nothing may hold any length)
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
    p.new_lens[b] = (err || m < 0) ? base : base + m + 1;
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
// One cluster does the whole table: the phases (checks, claims, new entries,
// references, free pages, the table) need all of one before the next, and a
// cluster barrier is the cheapest such point on the device. A warp works on a
// row, its lanes on the row's entries; free pages are found in order by a prefix
// over contiguous ranges of the reference counts. Latency bounds it: about a
// dozen dependent trips to L2. Two updates of 128 rows take 23 or 30 us in a graph,
// depending on what the process ran before; the cause of the two levels is not known.
constexpr int kTableThreads = 1024;
constexpr int kTableCtas = 8;     // the largest portable cluster
constexpr int32_t kNeed = -2;     // an entry that waits for a free page

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
  int32_t* lack;   // [B] entries of the row that wait for a page
  int32_t* entry;  // [B * W] new entries
  int32_t* free_;  // [B * W] pages handed out, in order
  int32_t* zeros;  // [kTableCtas] free pages in a CTA's range
  Copy* copy;      // [B]
  int32_t* dev_err;
  int64_t num_blocks;
  int batch, width, page;
};

// Everything that another CTA wrote is read past L1.
__device__ __forceinline__ int32_t ld(const int32_t* p) { return __ldcg(p); }

__global__ void __launch_bounds__(kTableThreads, 1) update_table_kernel(const TableParams p) {
  __shared__ int32_t s_warp[32];
  constexpr int kWarps = kTableThreads / 32;
  constexpr uint32_t kAll = 0xffffffffu;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = p.batch, W = p.width;
  const int ctas = (int)gridDim.x, cta = (int)blockIdx.x;
  const int first_row = cta * kWarps + warp, rows_apart = ctas * kWarps;
  const int64_t room = (int64_t)W * p.page;
  auto source = [&](int b) { return p.src ? p.src[b] : b; };
  const bool same = p.src == nullptr;  // every row continues itself: nobody else's entries are looked at

  if (!same) {
    for (int b = cta * kTableThreads + tid; b < B; b += ctas * kTableThreads) p.first[b] = B;
    cluster_sync_all();
  }
  // 1. rows that cannot be done: source or lengths out of range, kept tokens in entries that name no page
  for (int b = first_row; b < B; b += rows_apart) {
    const int s = source(b);
    int err = 0;
    if (s < -1 || s >= B) {
      err = SPEC_DEVERR_SRC_ROW;
    } else if (s >= 0) {
      const int cur = p.cur[s], want = p.want[b];
      if (want < 0 || want > room || cur < 0 || cur > room) {
        err = SPEC_DEVERR_CTX_LEN;
      } else {
        const int kept = (min(cur, want) + p.page - 1) / p.page;
        bool wrong = false;
        for (int i = lane; i < kept; i += 32) {
          const int32_t x = p.table[(int64_t)s * W + i];
          wrong |= x < 0 || x >= p.num_blocks;
        }
        if (__any_sync(kAll, wrong)) err = SPEC_DEVERR_BLOCK_ID;
      }
    }
    if (lane == 0) {
      if (err) raise_error(p.dev_err, err);
      p.bad[b] = err != 0;
      p.copy[b] = Copy{-1, -1, 0, 0};
      if (!same && !err && s >= 0) atomicMin(&p.first[s], b);  // 2. the row that continues each row
    }
  }
  if (!same) cluster_sync_all();
  else __syncwarp();
  // 3. new entries, and which of them wait for a page
  for (int b = first_row; b < B; b += rows_apart) {
    const bool bad = ld(&p.bad[b]) != 0;
    const int s = bad ? b : source(b);
    const int want = (bad || s < 0) ? 0 : p.want[b], keep = (bad || s < 0) ? 0 : min(p.cur[s], want);
    bool heir = same;  // row b continues row s
    if (!same && !bad && s >= 0) heir = (ld(&p.bad[s]) || source(s) == s ? s : ld(&p.first[s])) == b;
    const int entries = (want + p.page - 1) / p.page;
    int lacking = 0;
    for (int i0 = 0; i0 < W; i0 += 32) {
      const int i = i0 + lane;
      int32_t x = -1;
      bool need = false;
      if (i < W) {
        if (bad) {
          x = p.table[(int64_t)b * W + i];
        } else if (i < entries) {
          x = p.table[(int64_t)s * W + i];
          const int64_t begin = (int64_t)i * p.page;
          // a page wholly inside the kept tokens is shared; another stays if the row continues s and holds it alone
          if (begin + p.page > keep && !(heir && x >= 0 && x < p.num_blocks && p.refs[x] == 1)) {
            if (keep > begin) p.copy[b] = Copy{x, -1, (int32_t)(keep - begin), 0};
            x = kNeed;
            need = true;
          }
        }
        p.entry[(int64_t)b * W + i] = x;
      }
      lacking += __popc(__ballot_sync(kAll, need));
    }
    if (lane == 0) p.lack[b] = lacking;
  }
  cluster_sync_all();
  // 4. references of the entries that changed; a page that is copied from is not handed out in this call (the copy may
  // still read it)
  int total = 0;
  for (int b = lane; b < B; b += 32) total += ld(&p.lack[b]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
  for (int b = first_row; b < B; b += rows_apart) {
    for (int i = lane; i < W; i += 32) {
      const int32_t was = p.table[(int64_t)b * W + i], x = p.entry[(int64_t)b * W + i];
      if (was == x) continue;
      if (was >= 0 && was < p.num_blocks) atomicSub(&p.refs[was], 1);
      if (x >= 0) atomicAdd(&p.refs[x], 1);
    }
    if (lane == 0 && p.copy[b].src >= 0) atomicAdd(&p.refs[p.copy[b].src], 1);
  }
  // 5. the lowest free pages, if any row waits for one
  int found = 0;
  if (total > 0) {
    cluster_sync_all();
    // contiguous ranges of 4-page groups for the CTAs, of them for the warps: lane order is page order
    const int64_t groups = (p.num_blocks + 3) / 4, per = (groups + ctas - 1) / ctas, per_warp = (per + kWarps - 1) / kWarps;
    const int64_t cta_end = min(groups, (cta + 1) * per);
    const int64_t g0 = min(cta_end, cta * per + warp * per_warp), g1 = min(cta_end, g0 + per_warp);
    auto free_mask = [&](int64_t g) -> uint32_t {  // of the group's pages
      uint32_t m = 0;
      if (g < g1) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (4 * g + e < p.num_blocks && ld(&p.refs[4 * g + e]) == 0) m |= 1u << e;
      }
      return m;
    };
    int mine = 0;
    for (int64_t g = g0; g < g1; g += 32) mine += __popc(free_mask(g + lane));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(kAll, mine, o);
    if (lane == 0) s_warp[warp] = mine;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s_warp[w];
      all += s_warp[w];
    }
    if (tid == 0) p.zeros[cta] = all;
    cluster_sync_all();
    for (int c = 0; c < ctas; ++c) {
      const int z = ld(&p.zeros[c]);
      if (c < cta) before += z;
      found += z;
    }
    for (int64_t g = g0; g < g1 && before < total; g += 32) {
      const uint32_t m = free_mask(g + lane);
      int incl = __popc(m);
      const int own = incl;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += v;
      }
      int at = before + incl - own;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((m >> e) & 1) {
          if (at < total) {
            p.free_[at] = (int32_t)(4 * (g + lane) + e);
            p.refs[4 * (g + lane) + e] = 1;
          }
          ++at;
        }
      before += __shfl_sync(kAll, incl, 31);
    }
    cluster_sync_all();
  }
  // 6. the table
  for (int b = first_row; b < B; b += rows_apart) {
    int rank = 0;
    if (ld(&p.lack[b]) > 0)
      for (int c = lane; c < b; c += 32) rank += ld(&p.lack[c]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) rank += __shfl_xor_sync(kAll, rank, o);
    for (int i0 = 0; i0 < W; i0 += 32) {
      const int i = i0 + lane;
      int32_t x = i < W ? p.entry[(int64_t)b * W + i] : -1;
      const uint32_t needs = __ballot_sync(kAll, x == kNeed);
      if (x == kNeed) {
        const int at = rank + __popc(needs & ((1u << lane) - 1));
        x = at < found ? ld(&p.free_[at]) : -1;
        if (x < 0) raise_error(p.dev_err, SPEC_DEVERR_NO_PAGE);
        const Copy c = p.copy[b];
        if (c.src >= 0 && i == min(p.cur[source(b)], p.want[b]) / p.page) p.copy[b].dst = x;
      }
      rank += __popc(needs);
      if (i < W) p.table[(int64_t)b * W + i] = x;
    }
    if (lane == 0 && p.copy[b].src >= 0) atomicSub(&p.refs[p.copy[b].src], 1);
  }
}

// Copies of partly filled pages: CTA (row, layer, K or V). A stream at HBM speed; eight 16-byte loads a thread are in
// flight before the first store. Launched early behind the table kernel, it waits for that kernel's results. A fork with
// 235 MB of partial pages takes 43 to 48 us with the table's update (41 in a graph), 34.6 us at copy rate.
constexpr int kCopyThreads = 256;
constexpr int kCopyBatch = 8;

template <typename Vec>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const Copy* copies, uint8_t* k, uint8_t* v,
                                                                   int64_t num_blocks, int page, int64_t token_bytes) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int4 c = __ldcg(reinterpret_cast<const int4*>(copies) + blockIdx.x);  // src, dst, tokens
  if (c.x < 0 || c.y < 0) return;
  const int64_t cols = token_bytes / (int64_t)sizeof(Vec), n = c.z * cols;
  Vec* buf = reinterpret_cast<Vec*>(blockIdx.z ? v : k) + (int64_t)blockIdx.y * num_blocks * page * cols;
  const Vec* from = buf + (int64_t)c.x * page * cols;
  Vec* to = buf + (int64_t)c.y * page * cols;
  for (int64_t e0 = threadIdx.x; e0 < n; e0 += kCopyThreads * kCopyBatch) {
    Vec x[kCopyBatch];
#pragma unroll
    for (int i = 0; i < kCopyBatch; ++i)
      if (e0 + i * kCopyThreads < n) x[i] = from[e0 + i * kCopyThreads];
#pragma unroll
    for (int i = 0; i < kCopyBatch; ++i)
      if (e0 + i * kCopyThreads < n) to[e0 + i * kCopyThreads] = x[i];
  }
}

template <typename Vec>
static int launch_copies(const TableParams& p, uint8_t* k, uint8_t* v, const spec_cache_desc* d, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)d->batch, (unsigned)d->num_layers, 2);
  cfg.blockDim = dim3(kCopyThreads, 1, 1);
  cfg.stream = stream;
  const Copy* copies = p.copy;
  return cudaLaunchKernelEx(&cfg, copy_pages_kernel<Vec>, copies, k, v, d->num_blocks, (int)d->block_size, d->token_bytes) ==
                 cudaSuccess
             ? SPEC_OK
             : SPEC_ERR_LAUNCH;
}

struct Layout {
  size_t first, lack, entry, free_, zeros, copy, total;
};

static size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

static Layout layout_for(const spec_cache_desc* d) {
  Layout L;
  const size_t rows = up256((size_t)d->batch * 4), entries = up256((size_t)d->batch * d->max_blocks_per_seq * 4);
  L.first = rows;
  L.lack = 2 * rows;
  L.entry = 3 * rows;
  L.free_ = L.entry + entries;
  L.zeros = L.free_ + entries;
  L.copy = L.zeros + 256;
  L.total = L.copy + up256((size_t)d->batch * sizeof(Copy));
  return L;
}

static bool tables_ok(const spec_cache_desc* d) {
  return d != nullptr && d->batch >= 0 && d->block_size >= 1 && d->max_blocks_per_seq >= 1 && d->num_blocks >= 1;
}

static bool tables_supported(const spec_cache_desc* d) {
  return d->block_size <= 65536 && (int64_t)d->batch * d->max_blocks_per_seq <= (1 << 30) && d->num_blocks <= (1 << 30) &&
         (int64_t)d->max_blocks_per_seq * d->block_size + d->block_size - 1 <= INT32_MAX;  // lengths are rounded up to pages
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
  if (!k_cache || !v_cache || !block_table || !ctx_lens || !path || !accept_len || !new_lens) return SPEC_ERR_INVALID_ARG;
  if (num_nodes > tree::kMaxNodes || !pages::tables_supported(d) || d->num_layers > 65535) return SPEC_ERR_UNSUPPORTED;
  if (k_cache == v_cache) return SPEC_ERR_INVALID_ARG;  // two threads would move the same bytes
  // new_lens is written while the blocks of other layers still read the inputs
  const size_t rows = (size_t)d->batch * 4;
  if (tree::overlap(new_lens, rows, ctx_lens, rows) || tree::overlap(new_lens, rows, accept_len, rows) ||
      tree::overlap(new_lens, rows, path, rows * num_nodes) ||
      tree::overlap(new_lens, rows, block_table, rows * d->max_blocks_per_seq))
    return SPEC_ERR_INVALID_ARG;
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
  if (copies && d->num_layers > 0 && k_cache == v_cache) return SPEC_ERR_INVALID_ARG;
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
  p.lack = reinterpret_cast<int32_t*>(ws + L.lack);
  p.entry = reinterpret_cast<int32_t*>(ws + L.entry);
  p.free_ = reinterpret_cast<int32_t*>(ws + L.free_);
  p.zeros = reinterpret_cast<int32_t*>(ws + L.zeros);
  p.copy = reinterpret_cast<pages::Copy*>(ws + L.copy);
  p.dev_err = dev_err;
  p.num_blocks = d->num_blocks;
  p.batch = d->batch;
  p.width = d->max_blocks_per_seq;
  p.page = d->block_size;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = pages::kTableCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(pages::kTableCtas, 1, 1);
  cfg.blockDim = dim3(pages::kTableThreads, 1, 1);
  cfg.stream = stream;
  if (cudaLaunchKernelEx(&cfg, pages::update_table_kernel, p) != cudaSuccess) return SPEC_ERR_LAUNCH;
  if (!copies || d->num_layers == 0) return SPEC_OK;
  uint8_t *k = static_cast<uint8_t*>(k_cache), *v = static_cast<uint8_t*>(v_cache);
  switch (pages::vector_bytes(k_cache, v_cache, d->token_bytes)) {
    case 16: return pages::launch_copies<uint4>(p, k, v, d, stream);
    case 4: return pages::launch_copies<uint32_t>(p, k, v, d, stream);
    default: return pages::launch_copies<uint8_t>(p, k, v, d, stream);
  }
}
