"""Workloads of the tree-verification operators: their inputs, their plain forms and the library's calls.

The step of tree speculative decoding over a paged cache: attention of the N
tree nodes of every sequence, the walk that accepts a path of the tree, the
compaction of the accepted path's K and V, and the update of the page tables
(reserving, trimming, forking and freeing rows).

With `own` false, `run` computes the operators from elementary torch
operations; with `own` true it calls the library. `exact` computes the outputs
in 64 bits, sequence by sequence, written apart from the plain forms.
"""

import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one user's short prompt, a small tree: the latency of a single call
        dict(name="attention_single", op="attention", batch=1, ctx_lo=200, ctx_hi=200, nodes=8, heads=32, kv_heads=8,
             dim=128, page=64, dtype="bf16", out="f32"),
        # a handful of odd, short contexts with small heads, 16-token pages and half-precision caches
        dict(name="attention_odd_fp16", op="attention", batch=5, ctx_lo=14, ctx_hi=701, nodes=13, heads=9, kv_heads=3,
             dim=64, page=16, dtype="fp16", out="f32"),
        # a serving batch of the 8B-shaped target: 64-node trees, 256 packed rows per kv head
        dict(name="attention_batch32_tree64", op="attention", batch=32, ctx_lo=2048, ctx_hi=2048, nodes=64, heads=32,
             kv_heads=8, dim=128, page=64, dtype="bf16", out="bf16"),
        # the hybrid model's attention layer: head dim 256, ragged contexts, trees of 16
        dict(name="attention_hybrid_d256", op="attention", batch=64, ctx_lo=1024, ctx_hi=16384, nodes=16, heads=24,
             kv_heads=4, dim=256, page=64, dtype="bf16", out="f32"),
        # few sequences with very long contexts: the key axis is split
        dict(name="attention_longctx", op="attention", batch=8, ctx_lo=32768, ctx_hi=131072, nodes=32, heads=64,
             kv_heads=8, dim=128, page=128, dtype="bf16", out="bf16"),
        # the tiny vocabulary of the smallest configuration, all rows greedy: latency
        dict(name="accept_tiny_greedy", op="accept", batch=4, nodes=7, vocab=1000, mode="greedy", probs=False,
             lo=1.0, hi=1.0, noise=1.0),
        # sampled trees (children drawn from the draft's distribution) at the 8B vocabulary
        dict(name="accept_batch32_sampled", op="accept", batch=32, nodes=32, vocab=128256, mode="sample", probs=True,
             lo=1.0, hi=1.0, noise=1.5),
        # top-k trees without draft probabilities, greedy and sampling rows mixed, the largest vocabulary
        dict(name="accept_batch64_topk", op="accept", batch=64, nodes=16, vocab=248320, mode="mixed", probs=False,
             lo=0.5, hi=1.2, noise=1.5),
        # one sequence's path, few layers: latency
        dict(name="commit_path_single", op="commit", layers=4, batch=1, ctx_lo=300, ctx_hi=300, nodes=16, kv_heads=8,
             dim=128, page=64, dtype="bf16", longest=6),
        # every layer of the 8B-shaped target for a serving batch
        dict(name="commit_path_32layers", op="commit", layers=32, batch=32, ctx_lo=512, ctx_hi=1024, nodes=64,
             kv_heads=8, dim=128, page=64, dtype="bf16", longest=8),
        # page tables between two steps of a full serving batch: trim the rejected tail, reserve the next tree
        dict(name="pages_step_batch128", op="pages", layers=0, batch=128, ctx_lo=512, ctx_hi=8192, nodes=64, kv_heads=8,
             dim=128, page=64, dtype="bf16", group=1),
        # parallel sampling: groups of eight rows continue from surviving rows, partly filled pages are copied
        dict(name="pages_fork_batch32", op="pages", layers=32, batch=32, ctx_lo=256, ctx_hi=1024, nodes=32, kv_heads=8,
             dim=128, page=64, dtype="bf16", group=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "accept", "commit", "pages"])
    if op == "attention":
        kv = rng.choice([1, 2, 3, 4, 8])
        dim = rng.choice([64, 128, 256])
        nodes = rng.randint(1, 64)
        batch = _log(rng, 1, 96)
        hi = _log(rng, nodes + 1, max(nodes + 2, min(60000, 150000 // batch)))
        return dict(op=op, batch=batch, ctx_lo=min(hi, max(nodes, hi // 6)), ctx_hi=hi, nodes=nodes,
                    heads=kv * rng.choice([1, 2, 3, 4, 5, 6, 8]), kv_heads=kv, dim=dim, page=rng.choice([16, 32, 64, 128]),
                    dtype=rng.choice(["bf16", "bf16", "fp16"]), out=rng.choice(["f32", "same"]))
    if op == "accept":
        return dict(op=op, batch=_log(rng, 1, 32), nodes=rng.randint(1, 32), vocab=_log(rng, 500, 128256),
                    mode=rng.choice(["greedy", "sample", "mixed"]), probs=rng.random() < 0.5, lo=0.6, hi=1.3,
                    noise=rng.uniform(0.3, 2.0))
    if op == "commit":
        nodes = rng.randint(2, 64)
        return dict(op=op, layers=rng.randint(1, 32), batch=_log(rng, 1, 32), ctx_lo=nodes, ctx_hi=_log(rng, nodes, 1024),
                    nodes=nodes, kv_heads=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 128]),
                    page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "fp16"]), longest=rng.randint(1, nodes))
    group = rng.choice([1, 2, 3, 5, 8])
    return dict(op=op, layers=rng.randint(1, 24) if group > 1 else 0, batch=group * rng.randint(1, 32 // group),
                ctx_lo=1, ctx_hi=_log(rng, 40, 1024), nodes=rng.randint(1, 64), kv_heads=rng.choice([1, 2, 4, 8]),
                dim=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]), dtype="bf16", group=group)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _dtype(name):
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}[name]


def _trees(g, batch, nodes):
    """Random recursive trees: node i > 0 hangs under any earlier node of its sequence; the last nodes of a
    sequence may be unused (-2)."""
    i = torch.arange(nodes, device=DEV)
    parents = (torch.rand((batch, nodes), generator=g, device=DEV) * i).long().clamp(max=nodes - 1)
    parents = torch.minimum(parents, (i - 1).clamp(min=0))
    used = torch.randint((nodes + 1) // 2, nodes + 1, (batch, 1), generator=g, device=DEV)
    parents = torch.where(i < used, parents, -2)
    parents[:, 0] = -1
    return parents.to(torch.int32)


def _page_table(g, lens, page, longest, spare):
    """Tables that cover `lens` tokens a row with distinct random pages, -1 behind them, and the number of pages of
    a cache that holds any such batch (rows of up to `longest` tokens)."""
    want = (lens + page - 1) // page
    width = -(-longest // page)
    has = torch.arange(width, device=DEV)[None, :] < want[:, None]
    pages = lens.shape[0] * width + spare
    order = torch.randperm(pages, generator=g, device=DEV)
    rank = (torch.cumsum(has.reshape(-1).long(), 0) - 1).clamp(min=0).reshape(has.shape)
    return torch.where(has, order[rank], -1).to(torch.int32), pages


def _lens(case, g):
    return torch.randint(case["ctx_lo"], case["ctx_hi"] + 1, (case["batch"],), generator=g, device=DEV)


def _prepare_attention(case, g):
    B, N, D, page = case["batch"], case["nodes"], case["dim"], case["page"]
    dt = _dtype(case["dtype"])
    ctx = _lens(case, g).clamp(min=N)
    table, pages = _page_table(g, ctx, page, max(N, case["ctx_hi"]), 3)
    shape = (pages, page, case["kv_heads"], D)
    s = dict(q=torch.randn((B, N, case["heads"], D), generator=g, device=DEV, dtype=dt),
             k_cache=torch.randn(shape, generator=g, device=DEV, dtype=dt),
             v_cache=torch.randn(shape, generator=g, device=DEV, dtype=dt),
             block_table=table, ctx_lens=ctx.to(torch.int32), parents=_trees(g, B, N))
    s["out"] = torch.empty((B, N, case["heads"], D), device=DEV,
                           dtype=dt if case["out"] in ("same", case["dtype"]) else _dtype(case["out"]))
    return s


def _prepare_accept(case, g):
    B, N, V = case["batch"], case["nodes"], case["vocab"]
    parents = _trees(g, B, N)
    par = parents.long()
    logits = torch.randn((B, N, V), generator=g, device=DEV) * 3.0
    draft = logits + torch.randn((B, N, V), generator=g, device=DEV) * case["noise"]
    mode = {"greedy": torch.zeros(B, device=DEV), "sample": torch.ones(B, device=DEV),
            "mixed": (torch.rand(B, generator=g, device=DEV) < 0.5).float()}[case["mode"]].to(torch.int32)
    temp = case["lo"] + (case["hi"] - case["lo"]) * torch.rand(B, generator=g, device=DEV)
    # sibling number of each node, and the widest family
    i = torch.arange(N, device=DEV)
    same = (par[:, :, None] == par[:, None, :]) & (par[:, :, None] >= 0)
    sibling = (same & (i[None, None, :] < i[None, :, None])).sum(-1)
    widest = int(same.sum(-1).max())
    k = max(1, min(widest, V))
    up = par.clamp(min=0)
    probs = torch.softmax(draft / temp[:, None, None], -1)
    if case["probs"]:
        choice = torch.multinomial(probs.reshape(B * N, V), k, replacement=True, generator=g).reshape(B, N, k)
    else:
        choice = draft.topk(k, dim=-1).indices
    tokens = choice.gather(1, up[:, :, None].expand(B, N, k)).gather(2, sibling.clamp(max=k - 1)[:, :, None])[:, :, 0]
    seed = int(torch.randint(0, 1 << 62, (1,), generator=g, device=DEV))
    return dict(logits=logits, probs=probs if case["probs"] else None, tokens=tokens.to(torch.int32).contiguous(),
                parents=parents, mode=mode, temperature=temp.float(), seed=seed, widest=widest,
                out_tokens=torch.empty((B, N), dtype=torch.int32, device=DEV),
                path=torch.empty((B, N), dtype=torch.int32, device=DEV),
                accept_len=torch.empty((B,), dtype=torch.int32, device=DEV))


def _caches(case, g, pages):
    shape = (case["layers"], pages, case["page"], case["kv_heads"], case["dim"])
    return {n: torch.randn(shape, generator=g, device=DEV, dtype=_dtype(case["dtype"])) for n in ("k_cache", "v_cache")}


def _prepare_commit(case, g):
    B, N = case["batch"], case["nodes"]
    ctx = _lens(case, g).clamp(min=N)
    table, pages = _page_table(g, ctx, case["page"], max(N, case["ctx_hi"]), 2)
    m = torch.randint(0, min(case["longest"], N - 1) + 1, (B,), generator=g, device=DEV)
    # an accepted path: node 0, then m of the other nodes in increasing order
    score = torch.rand((B, N), generator=g, device=DEV)
    score[:, 0] = -1.0
    order = score.argsort(-1)
    j = torch.arange(N, device=DEV)
    kept = torch.where(j[None, :] <= m[:, None], order, N).sort(-1).values
    path = torch.where(kept < N, kept, -1).to(torch.int32)
    return dict(block_table=table, ctx_lens=ctx.to(torch.int32), path=path, accept_len=m.to(torch.int32),
                new_lens=torch.empty((B,), dtype=torch.int32, device=DEV), **_caches(case, g, pages))


def _prepare_pages(case, g):
    B, N, page, group = case["batch"], case["nodes"], case["page"], case["group"]
    low = _lens(case, g)
    src = None
    if group > 1:
        # every row continues from some row of its group, at the group's common length
        at = torch.arange(B, device=DEV)
        low = low[at // group * group]
        src = (at // group * group + torch.randint(0, group, (B,), generator=g, device=DEV)).to(torch.int32)
    high = low + N
    table, pages = _page_table(g, high, page, case["ctx_hi"] + N, B + 5)
    refs = torch.bincount(table[table >= 0].long(), minlength=pages).to(torch.int32)
    return dict(block_table=table, refs=refs, high=high.to(torch.int32), low=low.to(torch.int32), src_rows=src,
                **(_caches(case, g, pages) if group > 1 else {}))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = {"attention": _prepare_attention, "accept": _prepare_accept, "commit": _prepare_commit,
         "pages": _prepare_pages}[case["op"]](case, g)
    s["op"] = case["op"]
    s["page"] = case.get("page")
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _visible(parents):
    """[B, N, N]: node i sees node j (j is i or an ancestor of i); nothing for unused nodes."""
    n = parents.shape[1]
    i = torch.arange(n, device=DEV)
    edge = (parents[:, :, None] == i) | torch.eye(n, dtype=torch.bool, device=DEV)
    reach = torch.linalg.matrix_power(edge.double(), max(1, n - 1)) > 0
    return reach & (parents > -2)[:, :, None]


def _plain_attention(s):
    q, table, ctx = s["q"].float(), s["block_table"].long().clamp(min=0), s["ctx_lens"].long()
    B, N, H, D = q.shape
    K = s["k_cache"].shape[2]
    G = H // K
    T = table.shape[1] * s["page"]
    k = s["k_cache"][table].reshape(B, T, K, D).float().permute(0, 2, 3, 1)
    v = s["v_cache"][table].reshape(B, T, K, D).float().permute(0, 2, 1, 3)
    node = torch.arange(T, device=DEV)[None, :] - (ctx - N)[:, None]
    tree = _visible(s["parents"]).gather(2, node.clamp(0, N - 1)[:, None, :].expand(B, N, T))
    sees = (node < 0)[:, None, :] | (tree & ((node >= 0) & (node < N))[:, None, :])
    rows = q.reshape(B, N, K, G, D).permute(0, 2, 3, 1, 4).reshape(B, K, G * N, D) * D ** -0.5
    x = torch.matmul(rows, k).reshape(B, K, G, N, T)
    x = torch.where(sees[:, None, None], x, -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    out = torch.matmul(x.reshape(B, K, G * N, T), v).reshape(B, K, G, N, D) / x.sum(-1, keepdim=True)
    out = out.permute(0, 3, 1, 2, 4).reshape(B, N, H, D)
    return torch.where((s["parents"] > -2)[:, :, None, None], out, 0.0).to(s["out"].dtype)


def _philox(c0, c1, c2, c3, seed):
    """Philox4x32-10 on int64 tensors that hold 32-bit words."""
    low = 0xFFFFFFFF
    k0, k1 = seed & low, (seed >> 32) & low

    def product(a, x):
        lo_part = a * (x & 0xFFFF)
        hi_part = a * (x >> 16) + (lo_part >> 16)
        return hi_part >> 16, ((hi_part & 0xFFFF) << 16) | (lo_part & 0xFFFF)

    for _ in range(10):
        h0, l0 = product(0xD2511F53, c0)
        h1, l1 = product(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return c0, c1, c2, c3


def _uniform(word):
    return ((word >> 9).double() + 0.5) * 2.0 ** -23


def _plain_accept(s):
    logits, tokens, par, mode = s["logits"], s["tokens"].long(), s["parents"].long(), s["mode"]
    B, N, V = logits.shape
    i = torch.arange(N, device=DEV)
    rows = torch.arange(B, device=DEV)[:, None].expand(B, N)
    zero = torch.zeros((B, N), dtype=torch.int64, device=DEV)
    # children[b, n, r]: the r-th child of node n, N where there is none
    child = (par[:, None, :] == i[:, None])
    children = torch.where(child, i, N).sort(-1).values[:, :, : max(1, s["widest"])]
    # greedy: the argmax and the first child that holds it, of every node
    top = (logits == logits.amax(-1, keepdim=True)).to(torch.uint8).argmax(-1)
    hit = torch.where(child & (tokens[:, None, :] == top[:, :, None]), i, N).amin(-1)
    # sampling: the children of every node in turn against the residual
    p = torch.softmax(logits.double() / s["temperature"].double()[:, None, None], -1)
    q = None if s["probs"] is None else s["probs"].double()
    u = _uniform(_philox(zero, (i - 1).clamp(min=0) + zero, rows, zero, s["seed"])[0])
    weight, kept = p, torch.full_like(hit, N)
    for r in range(children.shape[2]):
        c = children[:, :, r]
        at = c.clamp(max=N - 1)
        x = tokens.gather(1, at)[:, :, None]
        total = weight.sum(-1)
        px = weight.gather(2, x)[:, :, 0] / total
        qx = torch.ones_like(px) if q is None else q.gather(2, x)[:, :, 0]
        open_ = (c < N) & (kept == N)
        take = open_ & (u.gather(1, at) * qx < px)
        kept = torch.where(take, c, kept)
        shifted = weight / total[:, :, None]
        less = shifted.scatter_add(2, x, -torch.ones_like(px)[:, :, None]) if q is None else shifted - q
        less = less.clamp(min=0.0)
        stays = ~(open_ & ~take) | (less.amax(-1) <= 0)
        weight = torch.where(stays[:, :, None], weight, less)
    group = torch.arange((V + 3) // 4, device=DEV)
    words = torch.stack(_philox(group.expand(B, N, -1), i[:, None].expand(B, N, 1), rows[:, :, None],
                                torch.ones_like(zero)[:, :, None], s["seed"]), -1).reshape(B, N, -1)[:, :, :V]
    drawn = (weight / -torch.log(_uniform(words))).argmax(-1)
    greedy = (mode == 0)[:, None]
    step, final = torch.where(greedy, hit, kept), torch.where(greedy, top, drawn)
    # the walk from node 0
    at = torch.zeros((B,), dtype=torch.int64, device=DEV)
    path, done = [at], torch.zeros((B,), dtype=torch.bool, device=DEV)
    for _ in range(N - 1):
        nxt = step.gather(1, at[:, None])[:, 0]
        done = done | (nxt == N)
        at = torch.where(done, at, nxt)
        path.append(torch.where(done, -1, nxt))
    path = torch.stack(path, 1)
    m = (path >= 0).sum(1) - 1
    after = torch.cat([path[:, 1:], path.new_full((B, 1), -1)], 1)
    last = final.gather(1, at[:, None])
    out = torch.where(after >= 0, tokens.gather(1, after.clamp(min=0)), torch.where(i == m[:, None], last, -1))
    return dict(out_tokens=out.to(torch.int32), path=path.to(torch.int32), accept_len=m.to(torch.int32))


def _plain_commit(s):
    table, ctx, path, m = s["block_table"].long(), s["ctx_lens"].long(), s["path"].long(), s["accept_len"].long()
    N, page = path.shape[1], s["page"]
    j = torch.arange(N, device=DEV)
    base = (ctx - N)[:, None]
    to = base + j
    come = base + torch.where(j <= m[:, None], path, j)
    slot = lambda t: (table.gather(1, t // page) * page + t % page).reshape(-1)  # noqa: E731
    for name in ("k_cache", "v_cache"):
        flat = s[name].reshape(s[name].shape[0], -1, s[name].shape[3] * s[name].shape[4])
        flat[:, slot(to)] = flat[:, slot(come)]
    s["new_lens"].copy_(ctx - N + m + 1)
    return dict(k_cache=s["k_cache"], v_cache=s["v_cache"], new_lens=s["new_lens"])


def _plain_update(s, cur, new, src):
    """Rows take the pages of their source row: full pages shared, the partly filled one private, missing ones the
    lowest free pages in the order of rows and positions."""
    table, refs, page = s["block_table"].long(), s["refs"].long(), s["page"]
    B, W = table.shape
    P = refs.shape[0]
    at = torch.arange(B, device=DEV)
    src = at if src is None else src.long()
    new = new.long()
    keep = torch.minimum(cur.long()[src], new)
    i = torch.arange(W, device=DEV)
    full = ((i + 1) * page <= keep[:, None])
    filled = (keep[:, None] - i * page).clamp(0, page)
    have = table[src]
    first = torch.full((B,), B, device=DEV).scatter_reduce(0, src, at, "amin")
    first = torch.where(src == at, at, first)
    mine = (first[src] == at)[:, None]
    alone = (refs[have.clamp(min=0)] == 1) & (have >= 0)
    wanted = i < ((new + page - 1) // page)[:, None]
    stays = wanted & (full | (mine & alone))
    got = torch.where(stays, have, -1)
    count = torch.zeros(P + 1, dtype=torch.int64, device=DEV)
    count.scatter_add_(0, torch.where(got >= 0, got, P).reshape(-1), torch.ones(B * W, dtype=torch.int64, device=DEV))
    count.scatter_add_(0, torch.where(table >= 0, table, P).reshape(-1), -torch.ones(B * W, dtype=torch.int64, device=DEV))
    refs = refs + count[:P]
    free = refs == 0
    ids = torch.full((P + 1,), -1, device=DEV)
    ids.scatter_(0, torch.where(free, torch.cumsum(free.long(), 0) - 1, P), torch.arange(P, device=DEV))
    ids[P] = -1
    lack = (wanted & ~stays)
    rank = (torch.cumsum(lack.reshape(-1).long(), 0) - 1).reshape(B, W)
    fresh = torch.where(lack & (rank < P), ids[rank.clamp(0, P)], -1)
    refs = torch.cat([refs, refs.new_zeros(1)]).scatter_add(
        0, torch.where(fresh >= 0, fresh, P).reshape(-1), torch.ones(B * W, dtype=torch.int64, device=DEV))[:P]
    if "k_cache" in s:
        slots = torch.arange(page, device=DEV)
        move = (lack & (filled > 0) & (fresh >= 0))[:, :, None] & (slots < filled[:, :, None])
        come = (have[:, :, None] * page + slots)[move]
        to = (fresh[:, :, None] * page + slots)[move]
        for name in ("k_cache", "v_cache"):
            flat = s[name].reshape(s[name].shape[0], -1, s[name].shape[3] * s[name].shape[4])
            flat[:, to] = flat[:, come]
    s["block_table"].copy_(torch.where(lack, fresh, got))
    s["refs"].copy_(refs)


def _plain_pages(s):
    # rows continue from their sources without the tree's tail, then reserve the next tree
    _plain_update(s, s["high"], s["low"], s["src_rows"])
    _plain_update(s, s["low"], s["high"], None)


def run(s):
    op = s["op"]
    if own:
        import speculative_decoding_verification_paged_gb300 as sv
        if op == "attention":
            if "workspace" not in s:  # kept for the program's life, like the cache
                s["workspace"] = sv.new_attention_workspace(
                    sv.spec_tree_attention_workspace(s["q"], s["k_cache"], s["block_table"]), DEV)
            return sv.spec_tree_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["ctx_lens"],
                                          s["parents"], s["out"], workspace=s["workspace"])
        if op == "accept":
            sv.spec_tree_accept(s["logits"], s["tokens"], s["parents"], s["probs"], s["seed"], s["mode"],
                                s["temperature"], s["out_tokens"], s["path"], s["accept_len"])
            return dict(out_tokens=s["out_tokens"], path=s["path"], accept_len=s["accept_len"])
        if op == "commit":
            sv.spec_cache_commit_path(s["k_cache"], s["v_cache"], s["block_table"], s["ctx_lens"], s["path"],
                                      s["accept_len"], s["new_lens"])
            return dict(k_cache=s["k_cache"], v_cache=s["v_cache"], new_lens=s["new_lens"])
        k, v, page = s.get("k_cache"), s.get("v_cache"), s["page"]
        if "workspace" not in s:
            s["workspace"] = torch.empty(sv.spec_cache_update_workspace(s["block_table"], s["refs"]),
                                         dtype=torch.uint8, device=DEV)
        sv.spec_cache_update(s["block_table"], s["refs"], s["high"], s["low"], page, src_rows=s["src_rows"], k_cache=k,
                             v_cache=v, workspace=s["workspace"])
        sv.spec_cache_update(s["block_table"], s["refs"], s["low"], s["high"], page, workspace=s["workspace"])
    elif op == "attention":
        return _plain_attention(s)
    elif op == "accept":
        return _plain_accept(s)
    elif op == "commit":
        return _plain_commit(s)
    else:
        _plain_pages(s)
    return {n: s[n] for n in ("block_table", "refs", "k_cache", "v_cache") if n in s}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    B, N = case["batch"], case["nodes"]
    mean = (case.get("ctx_lo", 0) + case.get("ctx_hi", 0)) / 2
    if case["op"] == "attention":
        mean = max(mean, N)
        size = 2 if case["out"] != "f32" else 4
        rows = B * N * case["heads"] * case["dim"]
        return dict(bytes=B * mean * case["kv_heads"] * case["dim"] * 4 + rows * (2 + size) + B * (N * 4 + mean / case["page"] * 4),
                    flops=4.0 * B * mean * N * case["heads"] * case["dim"])
    if case["op"] == "accept":
        # the root's logits at least (and its draft distribution, where a draft is refused); the walk stops early
        return dict(bytes=B * case["vocab"] * 4.0 + B * N * 16, flops=B * case["vocab"] * 4.0)
    row = case["kv_heads"] * case["dim"] * 2
    if case["op"] == "commit":
        moved = min(case["longest"], N - 1) / 2
        return dict(bytes=B * (moved * row * 4 * case["layers"] + N * 4 + 16), flops=0)
    pages = B * (mean + N) / case["page"]
    copied = B * (1 - 1 / case["group"]) * case["page"] / 2 * row * 4 * case["layers"]
    return dict(bytes=2 * (pages * 8 + pages * 8) + copied, flops=0)


# ---------------------------------------------------------------------------
# 64 bits, one sequence or row at a time
# ---------------------------------------------------------------------------
def _exact_attention(case, s):
    B, N, H, D = s["q"].shape
    K, page = case["kv_heads"], case["page"]
    out = torch.zeros((B, N, H, D), dtype=torch.float64, device=DEV)
    parents, lens = s["parents"].tolist(), s["ctx_lens"].tolist()
    for b in range(B):
        n = -(-lens[b] // page)
        ids = s["block_table"][b, :n].long()
        base = lens[b] - N
        mask = torch.zeros((N, lens[b]), dtype=torch.bool)
        for i in range(N):
            if parents[b][i] == -2:
                continue
            mask[i, :base] = True
            j = i
            while j >= 0:
                mask[i, base + j] = True
                j = parents[b][j]
        mask = mask.to(DEV)
        for h in range(K):
            k = s["k_cache"][ids, :, h].reshape(-1, D)[: lens[b]].double()
            v = s["v_cache"][ids, :, h].reshape(-1, D)[: lens[b]].double()
            for n0 in range(0, N, 16):
                qs = s["q"][b, n0:n0 + 16, h * (H // K):(h + 1) * (H // K)].double()
                x = (qs @ k.T) / math.sqrt(D)
                see = mask[n0:n0 + 16, None, :].expand_as(x)
                x = x.masked_fill(~see, -math.inf)
                live = see.any(-1, keepdim=True)
                x = torch.where(live, x, 0.0).softmax(-1)
                out[b, n0:n0 + 16, h * (H // K):(h + 1) * (H // K)] = torch.where(live, x @ v, 0.0)
    return out


def _exact_commit(case, s):
    page, N = case["page"], case["nodes"]
    got = {n: s[n].clone() for n in ("k_cache", "v_cache")}
    lens = []
    for b, (row, ctx, path, m) in enumerate(zip(s["block_table"].tolist(), s["ctx_lens"].tolist(), s["path"].tolist(),
                                                s["accept_len"].tolist())):
        for j in range(m + 1):
            a, t = ctx - N + path[j], ctx - N + j
            for n in got:
                got[n][:, row[t // page], t % page] = s[n][:, row[a // page], a % page]
        lens.append(ctx - N + m + 1)
    return dict(got, new_lens=None)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(case, s)
    if case["op"] == "commit":
        return _exact_commit(case, s)
    return None
