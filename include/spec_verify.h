/*
 * spec_verify.h -- C ABI of the target-side verify step of chain speculative
 * decoding (a draft of k tokens is checked by one wide target pass).
 *
 * The step has three parts, one entry point each:
 *
 *   spec_verify_attention  paged GQA attention of the k+1 verify rows of every
 *                          sequence over a block-paged bf16 KV cache
 *                          (lmdeploy PR #5019, summary: "paged CuTe
 *                          verification attention"; onnxruntime-genai PR #2457,
 *                          fast-commit notes: the "wide batched verify").
 *   spec_accept            greedy prefix match or speculative (rejection)
 *                          sampling over vocab-sized logits, giving the number
 *                          of accepted drafts and the correction/bonus token
 *                          (lmdeploy PR #5019, summary: "speculative sampling";
 *                          lmdeploy PR #3945, review of reject_sampler.py;
 *                          onnxruntime-genai PR #2457: greedy speculation is
 *                          token-identical to greedy decoding).
 *   spec_commit_state      copies, for every row, the recurrent-state checkpoint
 *                          of the accepted prefix into the live gated-delta-net
 *                          state (onnxruntime-genai PR #2457, notes on per-token
 *                          state checkpoints and CommitPrefix; lmdeploy PR #5019,
 *                          fix 2: CommitAcceptedRecurrentStateKernel).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Every tensor argument is a DEVICE pointer owned by the caller. The library
 *    never allocates, frees or synchronises; each call only enqueues kernels on
 *    `stream` (a cudaStream_t; NULL = legacy default stream) and returns.
 *  - Return value: SPEC_OK, or a negative SPEC_ERR_* code. Arguments the host
 *    can check (null pointers, sizes, unsupported shapes, a workspace that is
 *    too small) are checked before anything is launched; on error nothing is
 *    enqueued. SPEC_ERR_LAUNCH reports a failed kernel launch.
 *  - `dev_err` (optional, may be NULL) is a device int32 that kernels OR
 *    SPEC_DEVERR_* bits into when they meet data they cannot use (for example
 *    a block id outside the cache). The offending unit is skipped: its outputs
 *    are written as documented per call and the rest of the batch is computed
 *    normally. No kernel traps, asserts or aborts. The caller clears the word.
 *  - All index tensors are int32, row-major, densely packed.
 */
#ifndef SPEC_VERIFY_H_
#define SPEC_VERIFY_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t, without requiring the CUDA headers. */
typedef struct CUstream_st* spec_stream_t;

/* Status codes. */
#define SPEC_OK 0
#define SPEC_ERR_INVALID_ARG (-1)   /* null pointer, negative size, bad enum   */
#define SPEC_ERR_UNSUPPORTED (-2)   /* a shape this build has no kernel for    */
#define SPEC_ERR_LAUNCH (-3)        /* cudaLaunch* failed (see cudaGetLastError) */
#define SPEC_ERR_WORKSPACE (-4)     /* workspace missing or smaller than asked  */
#define SPEC_ERR_SCRATCH_LIMIT (-5) /* shape needs more than the fixed scratch of
                                       spec_verify_attention_noalloc           */

/* Bits OR-ed into *dev_err by the kernels. */
#define SPEC_DEVERR_BLOCK_ID 1     /* block_table entry outside [0, num_blocks)  */
#define SPEC_DEVERR_TOKEN 2        /* draft token outside [0, V)                 */
#define SPEC_DEVERR_ACCEPT_LEN 4   /* accept_len outside [0, S-1]                */
#define SPEC_DEVERR_CTX_LEN 8      /* ctx_len < k+1 or > max_blocks_per_seq * bs */
#define SPEC_DEVERR_TEMPERATURE 16 /* sampling row with temperature not > 0      */
#define SPEC_DEVERR_TIMEOUT 32     /* an asynchronous copy did not arrive        */
#define SPEC_DEVERR_MODE 64        /* mode not 0/1                               */
#define SPEC_DEVERR_POOL_ROW 128   /* state-pool row index outside the pool      */
#define SPEC_DEVERR_TREE 256       /* parents do not describe a tree             */
#define SPEC_DEVERR_NO_PAGE 512    /* no free page left for a row                */
#define SPEC_DEVERR_SRC_ROW 1024   /* source row outside [-1, B)                 */

/* Human-readable name of a status code (static storage, never NULL). */
const char* spec_status_string(int status);

/* ------------------------------------------------------------------------ */
/* 1. Paged GQA verification attention                                        */
/* ------------------------------------------------------------------------ */

/* Shapes of one attention call. */
typedef struct spec_attn_desc {
  int32_t batch;              /* B: sequences                                  */
  int32_t num_q_heads;        /* Hq                                            */
  int32_t num_kv_heads;       /* Hkv; Hq % Hkv == 0, G = Hq / Hkv              */
  int32_t head_dim;           /* D in {64, 128, 256}                           */
  int32_t block_size;         /* bs: tokens per KV block, in {16, 32, 64, 128} */
  int32_t max_blocks_per_seq; /* row stride of block_table                     */
  int64_t num_blocks;         /* physical blocks in k_cache / v_cache          */
} spec_attn_desc;

/* The first bytes of an attention workspace hold arrival counters that every
 * call, of spec_verify_attention and of spec_tree_attention, returns to zero;
 * nothing else is ever written there. They alone have to be zero before the
 * workspace's first use. */
#define SPEC_ATTN_COUNTER_BYTES 4096

/* Zeroes the counters of a new attention workspace (256-byte aligned, at least
 * SPEC_ATTN_COUNTER_BYTES), asynchronously on `stream`. */
int spec_attention_workspace_init(void* workspace, size_t workspace_bytes, spec_stream_t stream);

/*
 * Bytes of device workspace spec_verify_attention needs for `d`: room for the
 * split-KV partial results (normalised partial outputs and their log-sum-exp)
 * of the largest split plan the kernel can choose, so the caller may size it
 * once from the shapes alone. Returns 0 for an invalid descriptor.
 */
size_t spec_verify_attention_workspace(const spec_attn_desc* d, int32_t k_draft);

/*
 * out[b, i, h, :] = softmax_t( q[b,i,h,:] . K[b,t,g,:] / sqrt(D) ) . V[b,t,g,:]
 * for every sequence b, verify row i in [0, k_draft], query head h, with
 * g = h / G (contiguous GQA groups) and t over the causal window
 * t <= ctx_lens[b] - (k_draft+1) + i: row 0 is the last committed token and
 * row i also sees the first i draft tokens of its own chain.
 *
 *  q           [B, k_draft+1, Hq, D] bf16
 *  k_cache     [num_blocks, bs, Hkv, D] bf16. Token t of sequence b is stored
 *  v_cache     in physical block block_table[b, t / bs], slot t % bs. The KV of
 *              the k_draft+1 verify tokens is already in the cache.
 *  block_table [B, max_blocks_per_seq] int32
 *  ctx_lens    [B] int32, tokens in the cache per sequence, verify tokens
 *              included; must lie in [k_draft+1, max_blocks_per_seq * bs].
 *  out         [B, k_draft+1, Hq, D] fp32
 *  workspace   >= spec_verify_attention_workspace(d, k_draft) bytes, 256-byte
 *              aligned, its first SPEC_ATTN_COUNTER_BYTES bytes ZERO-FILLED
 *              before its first use; the rest is scratch. Reuse it for later
 *              calls of any shape that it is large enough for, and of
 *              spec_tree_attention, on the same stream; two calls in flight at
 *              once need two workspaces.
 *
 * The key tiles of all (sequence, kv head) units are split evenly over the
 * CTAs (split-KV); a unit held by several CTAs is merged by its log-sum-exp
 * inside the same launch. When all units have the same length, CTAs take
 * whole units instead as long as the load stays close to even. The split is
 * chosen on the device from ctx_lens, so no host synchronisation is needed.
 * Calls may come from several host threads at once (each with its own
 * workspace and stream).
 * Kernels: D = 128 or 256 with (k_draft+1)*G >= 17 packed query rows runs on
 * the 5th-generation tensor cores (tcgen05, 128-key tiles, accumulators in
 * tensor memory) when that kernel's shared-memory plan fits the batch; other
 * shapes run on mma.sync tiles. The environment variable SPEC_ATTN_KERNEL=tc
 * or =mma overrides the choice for D = 128 and 256. Both give the same result
 * within rounding (fp32 accumulation in both).
 * Device errors: a sequence with an out-of-range ctx_len (SPEC_DEVERR_CTX_LEN)
 * or block id (SPEC_DEVERR_BLOCK_ID) gets out rows of zeros.
 * Supported: D in {64,128,256}; bs in {16,32,64,128}; (k_draft+1)*G <= 64.
 */
int spec_verify_attention(const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* block_table, const int32_t* ctx_lens,
                          int32_t k_draft, float* out, const spec_attn_desc* d,
                          void* workspace, size_t workspace_bytes, int32_t* dev_err,
                          spec_stream_t stream);

/*
 * Allocation-free form of spec_verify_attention (the pages have no
 * counterpart; this is a convenience of this library).
 *
 * For callers that may not allocate device memory when they call in: a
 * serving engine's per-step enqueue path that must not touch the allocator,
 * a plugin hook of an inference runtime whose enqueue contract forbids
 * allocation, or a process that reserved all device memory up front. It
 * computes the same result as spec_verify_attention but takes no workspace:
 * its scratch is a fixed array of spec_verify_attention_noalloc_limit() bytes
 * (32 MiB) inside the library, which every GPU that loads the library holds
 * until the process exits. It never calls cudaMalloc or cudaFree.
 *
 *  - The first call on a device looks up the array's device address
 *    (cudaGetSymbolAddress) with that device current; make that first call
 *    before any stream capture.
 *  - Every call shares the one array and leaves its contents behind; the call
 *    clears the part that must start at zero (an asynchronous memset on
 *    `stream`). Calls whose kernels overlap on the GPU (other streams, or
 *    other host threads) race on the array: serialise them.
 *  - A shape whose scratch would exceed the array returns
 *    SPEC_ERR_SCRATCH_LIMIT before anything is launched.
 * Arguments, layouts and device errors are those of spec_verify_attention.
 */
int spec_verify_attention_noalloc(const void* q, const void* k_cache, const void* v_cache,
                                  const int32_t* block_table, const int32_t* ctx_lens,
                                  int32_t k_draft, float* out, const spec_attn_desc* d,
                                  int32_t* dev_err, spec_stream_t stream);

/* Bytes of the fixed scratch array used by spec_verify_attention_noalloc. */
size_t spec_verify_attention_noalloc_limit(void);

/*
 * Which kernel spec_verify_attention (and its allocation-free form) launches
 * for `d` and `k_draft` on the current device, with the tile settings it is
 * built with (a convenience of this library, for callers that report
 * per-kernel figures). The choice follows the rule stated above
 * spec_verify_attention, SPEC_ATTN_KERNEL included.
 *
 *  plan   written on SPEC_OK; host memory owned by the caller.
 *
 * Returns SPEC_ERR_INVALID_ARG for an invalid descriptor or a null plan,
 * SPEC_ERR_UNSUPPORTED for a shape spec_verify_attention rejects the same way,
 * and SPEC_ERR_LAUNCH when a device query it needs fails (D = 128 or 256 with
 * 17 or more packed rows, or with SPEC_ATTN_KERNEL=tc, reads the current
 * device's shared-memory limit; other shapes need no device). Launches
 * nothing and touches no device memory.
 */
#define SPEC_ATTN_KERNEL_MMA 1 /* mma.sync m16n8k16 tiles                    */
#define SPEC_ATTN_KERNEL_TC 2  /* tcgen05 MMAs, accumulators in tensor memory */

typedef struct spec_attn_plan {
  int32_t kernel;        /* SPEC_ATTN_KERNEL_*                                   */
  int32_t m_tiles;       /* (k_draft+1)*G packed rows padded to 16*m_tiles: 1, 2, 4 */
  int32_t keys_per_tile; /* keys per K/V pipeline stage                          */
  int32_t stages;        /* K/V pipeline stages in shared memory (tcgen05: K ring
                            stages; its V ring has as many, or two with three K) */
  int32_t p_buffers;     /* tcgen05: shared-memory buffers of P; 0 for mma.sync  */
  int32_t ctas_per_sm;   /* resident CTAs per SM the kernel is compiled for      */
} spec_attn_plan;

int spec_verify_attention_plan(const spec_attn_desc* d, int32_t k_draft, spec_attn_plan* plan);

/* ------------------------------------------------------------------------ */
/* 2. Acceptance: greedy prefix match or speculative sampling                  */
/* ------------------------------------------------------------------------ */

#define SPEC_MODE_GREEDY 0
#define SPEC_MODE_SAMPLE 1

/*
 * For each row b (k = number of drafts, R = k+1 target positions):
 *
 *  Greedy rows (mode[b] == SPEC_MODE_GREEDY): a_j = argmax_v target_logits[b,j,v]
 *  (lowest index on ties). accept_len[b] = m = first j < k with
 *  draft_tokens[b,j] != a_j, else k. Emitted: d_0..d_{m-1}, a_m.
 *
 *  Sampling rows (mode[b] == SPEC_MODE_SAMPLE), T = temperature[b] > 0:
 *  p_j = softmax(target_logits[b,j,:] / T), q_j = draft_probs[b,j,:].
 *  Draft j is accepted iff u_j * q_j(d_j) < p_j(d_j), u_j uniform in (0,1);
 *  m = first rejected j, else k. The last emitted token is drawn from
 *  w = max(0, p_m - q_m) (from p_m itself if that is all zero) when m < k, and
 *  from p_k when m == k. The draw is an exponential race over the whole
 *  vocabulary: every entry x with w_x > 0 gets the key w_x / E_x, E_x = -ln U_x,
 *  and the largest key wins, which samples x with probability w_x / sum(w)
 *  without normalising w. Ties go to the lowest index; entries of zero weight
 *  never win.
 *
 *  Random numbers: Philox4x32-10 (Salmon et al., SC'11) keyed by
 *  (philox_seed low word, philox_seed high word). u_j uses word 0 of counter
 *  (0, j, b, 0); U_x of the race at position m uses word (x mod 4) of counter
 *  (x / 4, m, b, 1). A word w maps to ((w >> 9) + 0.5) * 2^-23.
 *
 *  target_logits [B, k+1, V] fp32
 *  draft_tokens  [B, k] int32
 *  draft_probs   [B, k, V] fp32, each row a distribution; or NULL: the
 *                drafts are then deterministic and q_j is one-hot at d_j, so
 *                draft j is kept iff u_j < p_j(d_j) and a rejection draws from
 *                p_m with d_m removed (the reject sampler of lmdeploy PR #3945
 *                is called with draft_probs = None)
 *  mode          [B] int32 (SPEC_MODE_*); temperature [B] fp32 (ignored for
 *                greedy rows)
 *  out_tokens    [B, k+1] int32: d_0..d_{m-1}, final token, then -1 padding
 *  accept_len    [B] int32: m in [0, k]
 *
 * Rows are read only up to the first rejection (early exit), so the bytes read
 * depend on the outcome; when the batch's rows are small (B * V * 4 bytes at
 * most 32 MB), the first float4 batch of each thread's slice of position j + 1
 * is also loaded while position j is decided. Each row is handled by one
 * thread-block cluster; the call picks the threads per CTA and the CTAs per
 * cluster so that every row of the batch is resident at once where that fits
 * (clusters walk several rows otherwise). The environment variable
 * SPEC_ACCEPT_CONFIG=TxC (T = 128 or 256 threads, C = 1, 2, 4, 8 or 16 CTAs
 * per cluster) forces one configuration, for tests and measurements; one the
 * vocabulary cannot use (fewer than 4T logits per CTA with C > 1) makes the
 * call return SPEC_ERR_LAUNCH.
 * Device errors: a row with a draft token outside [0, V) (SPEC_DEVERR_TOKEN),
 * a sampling row with temperature not > 0 (SPEC_DEVERR_TEMPERATURE), or a mode
 * other than 0/1 (SPEC_DEVERR_MODE) gets out_tokens all -1 and accept_len -1.
 * Supported: k_draft <= 31; vocab <= 2^30.
 */
int spec_accept(const float* target_logits, const int32_t* draft_tokens,
                const float* draft_probs, uint64_t philox_seed, const int32_t* mode,
                const float* temperature, int32_t* out_tokens, int32_t* accept_len,
                int32_t batch, int32_t k_draft, int32_t vocab, int32_t* dev_err,
                spec_stream_t stream);

/* ------------------------------------------------------------------------ */
/* 3. Recurrent-state commit                                                  */
/* ------------------------------------------------------------------------ */

/*
 * live_state[l, b, :] = snapshots[l, b, accept_len[b], :] for every layer l
 * and row b. Snapshot slot s holds the state after the verify step consumed
 * its input s (input 0 is the last committed token), so slot accept_len[b] is
 * the state of the accepted prefix.
 *
 *  snapshots  [L, B, S, state_elems] fp32
 *  accept_len [B] int32 (as written by spec_accept)
 *  live_state [L, B, state_elems] fp32
 *
 * The copy is bit-exact. A row whose accept_len lies outside [0, S-1] keeps
 * its live state unchanged and sets SPEC_DEVERR_ACCEPT_LEN.
 */
int spec_commit_state(const float* snapshots, const int32_t* accept_len,
                      float* live_state, int32_t num_layers, int32_t batch,
                      int32_t num_slots, int64_t state_elems, int32_t* dev_err,
                      spec_stream_t stream);

/* Checkpoint alignments of spec_commit_state_aligned. */
#define SPEC_ALIGN_TOKEN 0 /* slot j holds the state after the step's token j      */
#define SPEC_ALIGN_LAST 1  /* slot W-1 holds the state after the step's last token */

/*
 * Commit from a checkpoint window that may be wider than the step
 * (onnxruntime-genai PR #2457: the window is described by a checkpoint count
 * and an alignment, because the conv state writes slot j after local token j
 * while GatedDeltaNet writes slot W-1 after the last token). A step of
 * num_tokens = n tokens (k+1 for a verify step) fills a window of
 * num_slots = W >= n slots; with m = accept_len[b] drafts accepted the kept
 * state is the one after token m:
 *
 *   SPEC_ALIGN_TOKEN: live_state[l, b, :] = snapshots[l, b, m, :]
 *   SPEC_ALIGN_LAST:  live_state[l, b, :] = snapshots[l, b, W - n + m, :]
 *
 * snapshots [L, B, W, state_elems] fp32; accept_len [B] int32; live_state
 * [L, B, state_elems] fp32. With W = n both alignments equal spec_commit_state.
 * A row with accept_len outside [0, n-1] keeps its live state and sets
 * SPEC_DEVERR_ACCEPT_LEN. Returns SPEC_ERR_INVALID_ARG for n outside [1, W]
 * or another alignment.
 */
int spec_commit_state_aligned(const float* snapshots, const int32_t* accept_len,
                              float* live_state, int32_t num_layers, int32_t batch,
                              int32_t num_slots, int64_t state_elems, int32_t num_tokens,
                              int32_t alignment, int32_t* dev_err, spec_stream_t stream);

/*
 * Zero-copy commit: stage a different source row instead of copying state
 * (onnxruntime-genai PR #2457, CommitPrefix note: rolling back a rejected
 * draft only needs the state pool to stage another row, the checkpoint of the
 * accepted prefix, instead of the step's final state).
 *
 * The states are rows of a pool that the caller owns and that this call never
 * touches; two int32 tables of pool-row indices, updated in place, say where
 * each (layer l, row b) keeps its state:
 *
 *  live_row  [L, B]    int32: the row holding the live state of (l, b)
 *  ckpt_rows [L, B, W] int32: the W rows the verify step writes its
 *                      checkpoints to (slot s in ckpt_rows[l, b, s])
 *  accept_len [B] int32 (as written by spec_accept)
 *
 * With m = accept_len[b] and the slot s picked as in spec_commit_state_aligned
 * (s = m for SPEC_ALIGN_TOKEN, W - n + m for SPEC_ALIGN_LAST, n = num_tokens),
 * the call exchanges live_row[l, b] and ckpt_rows[l, b, s]: the chosen
 * checkpoint becomes the live state where it lies, and the former live row
 * becomes the window's free slot for the next step. Afterwards
 * pool[live_row[l, b]] holds exactly what spec_commit_state_aligned would have
 * copied, and each (l, b) still owns the same W + 1 rows. Cost: 16 bytes of
 * index traffic per (l, b) instead of two state copies.
 *
 * A row with accept_len outside [0, n-1] keeps both tables and sets
 * SPEC_DEVERR_ACCEPT_LEN. Returns SPEC_ERR_INVALID_ARG for n outside [1, W],
 * another alignment, negative sizes or a missing table.
 */
int spec_commit_select(const int32_t* accept_len, int32_t* live_row, int32_t* ckpt_rows,
                       int32_t num_layers, int32_t batch, int32_t num_slots,
                       int32_t num_tokens, int32_t alignment, int32_t* dev_err,
                       spec_stream_t stream);

/* ------------------------------------------------------------------------ */
/* 4. Gated delta rule over the verify chain (checkpoint producer)            */
/* ------------------------------------------------------------------------ */

/*
 * The GatedDeltaNet layers of a hybrid model publish their recurrent state
 * after every token of the speculative step (onnxruntime-genai PR #2457:
 * GatedDeltaNet.checkpoints, V-major float32 state, checkpoint windows;
 * lmdeploy PR #5019: GDR verify kernels); these calls compute that series for
 * one layer. The pages name the operator but not its update, which follows the
 * published Gated DeltaNet rule (Yang, Kautz, Hatamizadeh, "Gated Delta
 * Networks"). Per row b, head h and token t (R = num_tokens tokens, k+1 for a
 * verify step), with the state S V-major (S[i][c]: value i, key c):
 *
 *   a_t = exp(g_t)
 *   S_t = a_t S_{t-1} + beta_t (v_t - a_t S_{t-1} k_t) k_t^T
 *   o_t = S_t (scale q_t)
 *
 * S_0 is the live state; checkpoint slot base + t of a W-slot window
 * (W = num_slots >= R) receives S_{t+1}, the state after input t, with
 * base = 0 for SPEC_ALIGN_TOKEN and W - R for SPEC_ALIGN_LAST; other slots are
 * not written. The gates arrive computed (g is the log decay, typically <= 0);
 * q and k are used as given (any normalisation happens upstream).
 *
 *  q, k   [B, R, H, dk] fp32      v    [B, R, H, dv] fp32
 *  g, beta [B, R, H] fp32         out  [B, R, H, dv] fp32 (o_t)
 *  state_in  [B, H, dv, dk] fp32  (one row of E = H*dv*dk floats per b)
 *  snapshots [B, W, H, dv, dk] fp32
 *
 * Arithmetic is fp32 (the state stays fp32 between tokens). dk = dv = 128
 * runs the register-resident kernel (16-byte aligned states); other sizes run
 * a shared-memory kernel while dv*dk + R*(2dk+dv) + 3dv floats fit in 200 KB.
 * Returns SPEC_ERR_INVALID_ARG for R outside [1, 32], W < R, an unknown
 * alignment, non-positive sizes or missing pointers; SPEC_ERR_UNSUPPORTED for
 * a state too large for either kernel.
 */
int spec_gdn_verify(const float* q, const float* k, const float* v, const float* g,
                    const float* beta, float scale, const float* state_in, float* snapshots,
                    float* out, int32_t batch, int32_t num_tokens, int32_t num_heads,
                    int32_t dk, int32_t dv, int32_t num_slots, int32_t alignment,
                    int32_t* dev_err, spec_stream_t stream);

/*
 * The same step over a state pool, the companion of spec_commit_select: row b
 * reads its live state from pool row live_row[b] and writes checkpoint slot s
 * to pool row ckpt_rows[b, s]; a pool row holds E = H*dv*dk floats (all heads
 * of one (layer, row)). Pass the tables of one layer (live_row + l*B,
 * ckpt_rows + l*B*W). A row naming an index outside [0, pool_rows) writes
 * zeros to its out rows, touches no state and sets SPEC_DEVERR_POOL_ROW.
 */
int spec_gdn_verify_pooled(const float* q, const float* k, const float* v, const float* g,
                           const float* beta, float scale, float* pool, int64_t pool_rows,
                           const int32_t* live_row, const int32_t* ckpt_rows, float* out,
                           int32_t batch, int32_t num_tokens, int32_t num_heads, int32_t dk,
                           int32_t dv, int32_t num_slots, int32_t alignment, int32_t* dev_err,
                           spec_stream_t stream);

/* ------------------------------------------------------------------------ */
/* 5. Tree speculation: verify attention over a tree of drafts                */
/* ------------------------------------------------------------------------ */

/*
 * A tree step drafts several candidates per position. Its num_nodes = N nodes
 * of a sequence are described by `parents` [B, N] int32:
 *
 *   parents[b, i] = j, 0 <= j < i   node i is a child of node j
 *   parents[b, i] = SPEC_TREE_ROOT  node i has no parent (node 0 always)
 *   parents[b, i] = SPEC_TREE_UNUSED  no node: the slot is padding
 *
 * Node 0 is the last committed token, as row 0 of a chain step is; the chain is
 * the tree parents[b, i] = i - 1. A child of an unused node, a parent outside
 * [-2, i) or a node 0 with a parent is no tree (SPEC_DEVERR_TREE). A sequence
 * whose node 0 is unused is an empty row of a padded batch: its other inputs
 * are not looked at, and no error is set for it.
 */
#define SPEC_TREE_ROOT (-1)
#define SPEC_TREE_UNUSED (-2)

#define SPEC_DTYPE_BF16 0
#define SPEC_DTYPE_FP16 1
#define SPEC_DTYPE_FP32 2

/*
 * out[b, i, h, :] = softmax_t( q[b,i,h,:] . K[b,t,g,:] / sqrt(D) ) . V[b,t,g,:]
 * for node i of sequence b and query head h, g = h / G, over the committed
 * tokens t < base = ctx_lens[b] - N and over t = base + j for node i itself and
 * its ancestors j. Rows of unused nodes are zeros.
 *
 *  q           [B, N, Hq, D] of type `dtype` (SPEC_DTYPE_BF16 or _FP16)
 *  k_cache     [num_blocks, bs, Hkv, D] of type `dtype`; node j's K and V are in
 *  v_cache     the cache at token base + j. Slots of unused nodes and slots at
 *              or past ctx_lens[b] may hold anything, NaN included. A NaN or
 *              +inf among the scores that a row sees makes that row NaN, a score
 *              of -inf is a weight of 0; a NaN or infinity in the V of any other
 *              slot may reach every row of the sequence.
 *  block_table [B, max_blocks_per_seq] int32
 *  ctx_lens    [B] int32, tokens in the cache, the N tree slots included; must
 *              lie in [N, max_blocks_per_seq * bs]
 *  parents     [B, N] int32
 *  out         [B, N, Hq, D] of type `out_dtype`: fp32, or `dtype`. For the latter
 *              the softmax weights are rounded once to `dtype` before they meet V
 *              (an error of up to half its step of sum p |v|, beside the output's
 *              own rounding); for fp32 they keep 22 to 24 bits (fp16: down to
 *              2^-36 of the row's largest weight).
 *  workspace   >= spec_tree_attention_workspace(d, N) bytes, 256-byte aligned,
 *              its first SPEC_ATTN_COUNTER_BYTES bytes ZERO-FILLED before its
 *              first use; reusable by later calls of any shape, and of
 *              spec_verify_attention, on the same stream (two calls in flight at
 *              once, or two captured graphs that may run at once, need two
 *              workspaces).
 *
 * Device errors: a sequence with an out-of-range ctx_len (SPEC_DEVERR_CTX_LEN),
 * block id (SPEC_DEVERR_BLOCK_ID) or tree (SPEC_DEVERR_TREE) gets out rows of
 * zeros. Device pointers 16-byte aligned.
 * Supported: D in {64,128,256}; bs in {16,32,64,128}; N <= 64; G <= 128;
 * B <= 4096; with tiles = ceil(N / floor(128 / G)), at most 2^31 - 1 key tiles:
 * (max_blocks_per_seq * bs / 64 + 1) * B * Hkv * tiles; num_blocks * bs at most
 * 2^31 - 1.
 */
size_t spec_tree_attention_workspace(const spec_attn_desc* d, int32_t num_nodes);

int spec_tree_attention(const void* q, const void* k_cache, const void* v_cache,
                        const int32_t* block_table, const int32_t* ctx_lens,
                        const int32_t* parents, int32_t num_nodes, void* out, int32_t dtype,
                        int32_t out_dtype, const spec_attn_desc* d, void* workspace,
                        size_t workspace_bytes, int32_t* dev_err, spec_stream_t stream);

/* ------------------------------------------------------------------------ */
/* 6. Tree speculation: acceptance                                            */
/* ------------------------------------------------------------------------ */

/*
 * Walks the tree of each sequence from node 0. At node n:
 *
 *  Greedy rows (mode[b] == SPEC_MODE_GREEDY): a = argmax_v target_logits[b,n,v]
 *  (lowest index on ties). The first child (lowest node index) whose token is a
 *  is accepted and the walk goes on there; without one, a is emitted last.
 *
 *  Sampling rows (mode[b] == SPEC_MODE_SAMPLE), T = temperature[b] > 0:
 *  p = softmax(target_logits[b,n,:] / T). The children c of n are tried in
 *  increasing node index against the residual r, at first r = p:
 *    with draft_probs: q = draft_probs[b,n,:], the distribution every child of n
 *      was drawn from independently. c is accepted iff u_c q(x_c) < r(x_c);
 *      else r <- max(0, r - q) / sum.
 *    without (NULL): the children are deterministic. c is accepted iff
 *      u_c < r(x_c); else r <- r with x_c removed, normalised.
 *    A residual that would be all zero stays as it was.
 *  If no child is accepted, the last token is drawn from r by the exponential
 *  race of spec_accept.
 *
 *  Random numbers as in spec_accept with the node index in place of the
 *  position: u_c uses word 0 of counter (0, c - 1, b, 0), the race at node n
 *  counter (x / 4, n, b, 1). On a chain the call computes what spec_accept does,
 *  with exponents that stay exact to fp32 rounding at any T (spec_accept's lose
 *  bits where max |logit| / T is past 2^12 or so).
 *
 *  target_logits [B, N, V] fp32, row n the target's logits after node n
 *  tokens        [B, N] int32; the token of node n (node 0's is not looked at)
 *  parents       [B, N] int32; nodes other than 0 without a parent are never
 *                reached
 *  draft_probs   [B, N, V] fp32 or NULL; rows of nodes without children are not
 *                read
 *  mode          [B] int32; temperature [B] fp32 (ignored for greedy rows)
 *  out_tokens    [B, N] int32: the accepted nodes' tokens, the last token, -1s
 *  path          [B, N] int32: 0, the accepted nodes in order, -1s
 *  accept_len    [B] int32: accepted nodes, node 0 not counted
 *  The three results share no byte with one another or with the int32 and
 *  temperature inputs (refused otherwise).
 *
 * A visited node of a sampling row whose logits hold no distribution (all -inf, a
 * NaN, a +inf) ends the row: no child of it is accepted, the last token is -1.
 * Rows are read only along the accepted path; of small batches (B * V * 4 bytes
 * at most 32 MB) rows that the next decision may ask for are also prefetched.
 * SPEC_ACCEPT_CONFIG acts as in spec_accept.
 * Device errors: a row with a used node's token outside [0, V)
 * (SPEC_DEVERR_TOKEN), a bad tree (SPEC_DEVERR_TREE), mode (SPEC_DEVERR_MODE) or
 * temperature (SPEC_DEVERR_TEMPERATURE), and an empty row of a padded batch (no
 * error), get out_tokens and path all -1 and accept_len -1.
 * Supported: N <= 64; vocab <= 2^30.
 */
int spec_tree_accept(const float* target_logits, const int32_t* tokens, const int32_t* parents,
                     const float* draft_probs, uint64_t philox_seed, const int32_t* mode,
                     const float* temperature, int32_t* out_tokens, int32_t* path,
                     int32_t* accept_len, int32_t batch, int32_t num_nodes, int32_t vocab,
                     int32_t* dev_err, spec_stream_t stream);

/* ------------------------------------------------------------------------ */
/* 7. The paged cache between two steps                                       */
/* ------------------------------------------------------------------------ */

/* A cache of num_layers layers, [num_layers, num_blocks, block_size, token_bytes]
 * each for K and V, whose pages the rows of one block table name. */
typedef struct spec_cache_desc {
  int32_t batch;              /* B: rows of the block table                      */
  int32_t num_layers;         /* L                                               */
  int32_t block_size;         /* tokens per page, 1 to 65536                     */
  int32_t max_blocks_per_seq; /* row stride of block_table                       */
  int64_t num_blocks;         /* pages                                           */
  int64_t token_bytes;        /* bytes of one token's K (or V) in one layer      */
} spec_cache_desc;

/*
 * Keeps the accepted path of a tree step: in every layer, K and V of token
 * base + path[b, j] move to token base + j, j = 1 .. accept_len[b], in place,
 * base = ctx_lens[b] - N; the rest of the cache is left as it is.
 * new_lens[b] = base + accept_len[b] + 1, the row's committed tokens.
 *
 *  block_table [B, max_blocks_per_seq] int32; ctx_lens [B] int32
 *  path [B, N] int32 and accept_len [B] int32 as written by spec_tree_accept
 *  new_lens [B] int32; shares no byte with the inputs above
 *
 * K and V are two caches: one pointer for both is refused.
 * A row with accept_len -1 moves nothing and gets new_lens = max(0, base).
 * Device errors, with the same treatment: accept_len outside [-1, N - 1] or a
 * path that does not increase from 0 within [0, N) (SPEC_DEVERR_ACCEPT_LEN), a
 * ctx_len outside [N, max_blocks_per_seq * block_size] (SPEC_DEVERR_CTX_LEN), a
 * page outside [0, num_blocks) (SPEC_DEVERR_BLOCK_ID). Rows must not share the
 * pages of their tree slots. Without a row or a layer (B or L = 0) the call does
 * nothing, new_lens included. Supported: N <= 64; L <= 65535; the table's limits
 * of spec_cache_update.
 */
int spec_cache_commit_path(void* k_cache, void* v_cache, const int32_t* block_table,
                           const int32_t* ctx_lens, const int32_t* path,
                           const int32_t* accept_len, int32_t* new_lens, int32_t num_nodes,
                           const spec_cache_desc* d, int32_t* dev_err, spec_stream_t stream);

/*
 * Gives every row of the block table the pages for new_lens[b] tokens, on the
 * device: trims, reserves, frees, forks and reorders rows in one call.
 *
 *  block_table [B, max_blocks_per_seq] int32, in place; -1 means no page
 *  page_refs   [num_blocks] int32, in place: how many table entries (and other
 *              holders) name the page; a page with 0 is free
 *  cur_lens    [B] int32: tokens the rows hold; new_lens [B] int32: tokens they
 *              shall have room for
 *  src_rows    [B] int32 or NULL: the row b continues from: b itself (NULL: all
 *              rows do), another row (a fork, or a beam's reordering), or -1 to
 *              free the row
 *
 * With s = src_rows[b], row b keeps the first keep = min(cur_lens[s], new_lens[b])
 * tokens of row s. Entry i of the new row, for i < ceil(new_lens[b] / bs):
 *   - a page wholly inside the kept tokens is shared;
 *   - any other page of row s stays with the row that continues s (s itself if
 *     src_rows[s] == s, else the lowest b with that source), if no other holder
 *     has it (page_refs is 1 at entry);
 *   - else a free page is taken, and the kept tokens that the old page holds
 *     are copied into it, K and V of every layer.
 * Entries behind are -1. References are counted again, and pages that reach 0
 * are free at once (one that is copied from, after the call). Free pages are
 * handed out lowest index first, in the order of rows and entries, so the result
 * does not depend on timing.
 *
 *  k_cache, v_cache: two caches, or both NULL (then num_layers and token_bytes are not
 *              looked at and nothing is copied: for callers whose rows never
 *              share partly filled pages)
 *  workspace   >= spec_cache_update_workspace(d) bytes, 256-byte aligned, no
 *              initial contents needed; one call at a time
 *
 * Device errors: a row with a source outside [-1, B) (SPEC_DEVERR_SRC_ROW), a
 * length outside [0, max_blocks_per_seq * bs] (SPEC_DEVERR_CTX_LEN), or a kept
 * token in an entry outside [0, num_blocks) (SPEC_DEVERR_BLOCK_ID) keeps its
 * entries as they are. Entries that find no free page are -1
 * (SPEC_DEVERR_NO_PAGE). Supported: B * max_blocks_per_seq <= 2^30;
 * num_blocks <= 2^30; (max_blocks_per_seq + 1) * bs <= 2^31.
 */
size_t spec_cache_update_workspace(const spec_cache_desc* d);

int spec_cache_update(int32_t* block_table, int32_t* page_refs, const int32_t* cur_lens,
                      const int32_t* new_lens, const int32_t* src_rows, void* k_cache,
                      void* v_cache, const spec_cache_desc* d, void* workspace,
                      size_t workspace_bytes, int32_t* dev_err, spec_stream_t stream);

/* ------------------------------------------------------------------------ */
/* 8. Verify attention over a window of the cache, and over a 4-bit cache     */
/* ------------------------------------------------------------------------ */

/*
 * out[b, i, h, :] = softmax_t( q[b,i,h,:] . K[b,t,g,:] / sqrt(D) ) . V[b,t,g,:]
 * for every sequence b, row i in [0, num_rows), query head h, with g = h / G
 * (contiguous GQA groups). Row i is the token at p = ctx_lens[b] - num_rows + i;
 * it sees the tokens
 *
 *   t <= p  with  window = 0, or t > p - window, or t < sinks,
 *
 * that is the last `window` tokens, itself included, and the first `sinks`.
 * num_rows = 1 is a step of plain decoding; a verify step has k + 1 rows.
 *
 *  q           [B, num_rows, Hq, D] of type `dtype` (SPEC_DTYPE_BF16 or _FP16)
 *  k_cache     [num_blocks, bs, Hkv, D] of type `dtype`; the rows' own K and V
 *  v_cache     are in the cache already. Slots that no row of the sequence sees
 *              may hold anything, NaN included, and pages that hold only such
 *              slots are not looked at (their block_table entry may be anything).
 *              A NaN or +inf among the scores that a row sees makes that row NaN,
 *              a score of -inf is a weight of 0 (NaN where a row has no other); a NaN or infinity in the V of a
 *              slot that only other rows of the sequence see may reach the row.
 *  block_table [B, max_blocks_per_seq] int32
 *  ctx_lens    [B] int32, tokens in the cache, the rows' own included: 0 (an empty
 *              row of a padded batch: out rows of zeros, no error), or in
 *              [num_rows, max_blocks_per_seq * bs]
 *  out         [B, num_rows, Hq, D] of type `dtype`. Before they meet V the softmax
 *              weights p are rounded to two 16-bit numbers each (an error of 2^-16
 *              sum p |v| at most, beside the output's own rounding); bf16 ones at head
 *              dim 64, or where num_rows * G > 32, to one (2^-8 sum p |v|)
 *  workspace   >= spec_window_attention_workspace(d, num_rows) bytes, 256-byte
 *              aligned, its first SPEC_ATTN_COUNTER_BYTES bytes ZERO-FILLED before
 *              its first use; one workspace serves every attention call of any
 *              shape that it is large enough for, on one stream (two calls in
 *              flight at once, or two captured graphs that may run at once, need two
 *              workspaces).
 *
 * Device errors: a sequence with another ctx_len (SPEC_DEVERR_CTX_LEN) or a block
 * id outside the cache among the pages that it sees (SPEC_DEVERR_BLOCK_ID) gets out
 * rows of zeros. Device pointers 16-byte aligned.
 * Supported: D in {64,128,256}; bs in {16,32,64,128}; num_rows <= 64; G <= 64;
 * B <= 4096; max_blocks_per_seq * bs at most 2^30; num_blocks * bs,
 * (max_blocks_per_seq * bs / 32 + 2) * B and
 * (max_blocks_per_seq * bs / 128 + 2) * B * Hkv * ceil(num_rows * G / 16) at most
 * 2^31 - 1.
 */
size_t spec_window_attention_workspace(const spec_attn_desc* d, int32_t num_rows);

int spec_window_attention(const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* block_table, const int32_t* ctx_lens,
                          int32_t num_rows, int32_t window, int32_t sinks, void* out,
                          int32_t dtype, const spec_attn_desc* d, void* workspace,
                          size_t workspace_bytes, int32_t* dev_err, spec_stream_t stream);

/*
 * A cache in 4 bits. For every token and kv head the D elements x_e are held as
 *
 *   m = min x,  s = round16((max x - min x) / 15),  n_e = round((x_e - m) / s) in 0..15
 *
 * (the quotient rounded half to even; n = 0 where s = 0) and stand for n_e s + m. s
 * and m have the 16-bit type of the model, `dtype` in every call; a NaN or infinity
 * among the x makes all D elements NaN. The range is divided in fp32.
 *
 * k_cache and v_cache are [num_blocks, bs, row_bytes] bytes each, row_bytes =
 * spec_q4_row_bytes(Hkv, D). A token's row holds, for every kv head in turn, D / 2
 * bytes of codes (n_2i in the low, n_2i+1 in the high half of byte i); then, for
 * every kv head, s and m; then padding to 16 bytes, which no call looks at. A row is
 * whole in itself, so spec_cache_update and spec_cache_commit_path move tokens of
 * such caches too, with token_bytes = row_bytes.
 *
 * spec_q4_row_bytes returns 0 for D not in {64,128,256} or Hkv outside [1, 65536].
 */
int64_t spec_q4_row_bytes(int32_t num_kv_heads, int32_t head_dim);

/*
 * Writes the newest num_rows tokens of every sequence into a 4-bit cache: row i of
 * sequence b becomes token ctx_lens[b] - num_rows + i. Rows before token 0 are padding
 * (a batch of prompts of several lengths, aligned at their ends) and are not read;
 * nothing but the tokens' codes, s and m is written.
 *
 *  k, v        [B, num_rows, Hkv, D] of type `dtype`, k_stride and v_stride elements
 *              from one row to the next (at least Hkv * D, a multiple of 8): slices
 *              of a projection's output do
 *  block_table [B, max_blocks_per_seq] int32
 *  ctx_lens    [B] int32, tokens in the cache once these are in it
 *  d           num_q_heads is not looked at
 *
 * Device errors: a sequence whose ctx_len lies outside [0, max_blocks_per_seq * bs]
 * (SPEC_DEVERR_CTX_LEN) and a token whose page lies outside the cache
 * (SPEC_DEVERR_BLOCK_ID) are not written. Tokens must not share a slot. K and V are
 * two caches: one pointer for both is refused. Device pointers 16-byte aligned.
 * Supported: D in {64,128,256}; bs in {16,32,64,128}; B * num_rows * Hkv * D / 8 and
 * num_blocks * bs at most 2^31 - 1; max_blocks_per_seq * bs at most 2^30.
 */
int spec_cache_store_q4(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                        const int32_t* block_table, const int32_t* ctx_lens, int32_t num_rows,
                        void* k_cache, void* v_cache, int32_t dtype, const spec_attn_desc* d,
                        int32_t* dev_err, spec_stream_t stream);

/*
 * Reads the newest num_rows tokens of every sequence back: k_out, v_out
 * [B, num_rows, Hkv, D] of type `out_dtype` (`dtype` or fp32; n s + m is rounded to
 * fp32, then to `dtype`). Rows before token 0, rows of sequences with a bad ctx_len and
 * of tokens with a bad page (errors as above) are zeros. Limits as above.
 */
int spec_cache_load_q4(const void* k_cache, const void* v_cache, const int32_t* block_table,
                       const int32_t* ctx_lens, int32_t num_rows, void* k_out, void* v_out,
                       int32_t dtype, int32_t out_dtype, const spec_attn_desc* d,
                       int32_t* dev_err, spec_stream_t stream);

/*
 * spec_window_attention over a 4-bit cache: q and out of type `dtype`, which is that
 * of the cache's s and m too. Arguments, visibility (window = 0 for all tokens),
 * workspace, errors and limits are those of spec_window_attention; there is no
 * exception for V: what a row does not see cannot reach it.
 * q is held as fp16 times a power of two of its row (elements below 2^-24 of the row's
 * largest lose bits; a row with an element of 2^115 or more may come out as NaN), the
 * weights times s as fp16 times a power of two of the row. Where a row's largest score is
 * 2^27 or more (times log2 e), that power is set without regard to s: tokens of V with an
 * s below 2^-14 lose bits, and one above 2^15 counts as that. At all scores,
 * tokens of V with an s below 2^-60 lose bits, and elements of V of 2^40 or more may come
 * out as infinities or NaN.
 */
int spec_q4_attention(const void* q, const void* k_cache, const void* v_cache,
                      const int32_t* block_table, const int32_t* ctx_lens, int32_t num_rows,
                      int32_t window, int32_t sinks, void* out, int32_t dtype,
                      const spec_attn_desc* d, void* workspace, size_t workspace_bytes,
                      int32_t* dev_err, spec_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_VERIFY_H_ */
