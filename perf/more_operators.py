"""Workloads of the operators on bounded and compressed caches: inputs, plain forms and the library's calls.

Attention of the verify rows of every sequence over a paged cache of which a row
sees a sliding window and a few first tokens; the same over a cache that holds K
and V in 4 bits (windowed or not); storing tokens into such a cache, and reading
them back.

A token of a 4-bit cache is one row of bytes: for every kv head D/2 bytes of
codes (element 2i in the low half of byte i), then for every kv head the scale
and the minimum as two 16-bit floats, then padding to 16 bytes. An element
stands for code * scale + minimum.

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
        # one user decoding token by token with a small window: the latency of a single call
        dict(name="window_single", op="window", batch=1, ctx_lo=3000, ctx_hi=3000, rows=1, heads=32, kv_heads=8, dim=128,
             page=64, dtype="bf16", window=1024, sinks=4),
        # a handful of odd, short contexts, some shorter than the window, small heads, 16-token pages, half precision
        dict(name="window_odd_fp16", op="window", batch=5, ctx_lo=14, ctx_hi=701, rows=5, heads=9, kv_heads=3, dim=64,
             page=16, dtype="fp16", window=100, sinks=3),
        # a serving batch of the 8B-shaped target, chain of three drafts
        dict(name="window_batch32", op="window", batch=32, ctx_lo=8192, ctx_hi=8192, rows=4, heads=32, kv_heads=8,
             dim=128, page=64, dtype="bf16", window=4096, sinks=64),
        # the hybrid model's attention heads (head dim 256) with a window over ragged contexts
        dict(name="window_hybrid_d256", op="window", batch=64, ctx_lo=1024, ctx_hi=16384, rows=4, heads=24, kv_heads=4,
             dim=256, page=64, dtype="bf16", window=2048, sinks=16),
        # tokens of a decoding step of a full serving batch into the 4-bit cache: latency
        dict(name="store_step_batch128", op="store", batch=128, ctx_lo=512, ctx_hi=8192, rows=4, kv_heads=8, dim=128,
             page=64, dtype="bf16"),
        # prompts of several sequences at once; the shorter ones are padded in front
        dict(name="store_prompts", op="store", batch=8, ctx_lo=1000, ctx_hi=8192, rows=8192, kv_heads=8, dim=128,
             page=64, dtype="bf16"),
        # reading back the newest tokens of a batch: latency, odd sizes
        dict(name="load_tail_odd", op="load", batch=7, ctx_lo=30, ctx_hi=900, rows=13, kv_heads=3, dim=64, page=16,
             dtype="fp16"),
        # a whole cached prefix as 16-bit K and V
        dict(name="load_prefix", op="load", batch=1, ctx_lo=65536, ctx_hi=65536, rows=65536, kv_heads=8, dim=128, page=128,
             dtype="bf16"),
        # one user, one token, full visibility over a 4-bit cache: latency
        dict(name="q4_single", op="q4", batch=1, ctx_lo=2048, ctx_hi=2048, rows=1, heads=32, kv_heads=8, dim=128, page=64,
             dtype="bf16", window=0, sinks=0),
        # a serving batch of the 8B-shaped target over a 4-bit cache
        dict(name="q4_batch32", op="q4", batch=32, ctx_lo=2048, ctx_hi=2048, rows=4, heads=32, kv_heads=8, dim=128,
             page=64, dtype="fp16", window=0, sinks=0),
        # the hybrid model's attention layer, ragged contexts, a window wider than most of them
        dict(name="q4_hybrid_d256", op="q4", batch=64, ctx_lo=1024, ctx_hi=16384, rows=4, heads=24, kv_heads=4, dim=256,
             page=64, dtype="bf16", window=8192, sinks=4),
        # few sequences with very long contexts, 64 rows a kv head: the key axis is split
        dict(name="q4_longctx", op="q4", batch=8, ctx_lo=32768, ctx_hi=131072, rows=8, heads=64, kv_heads=8, dim=128,
             page=128, dtype="bf16", window=0, sinks=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "window", "q4", "q4", "q4", "store", "load"])
    kv = rng.choice([1, 2, 3, 4, 8])
    dim = rng.choice([64, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    if op in ("store", "load"):
        batch = _log(rng, 1, 64)
        hi = _log(rng, 1, max(2, 65536 // (batch * max(1, kv * dim // 1024))))
        return dict(op=op, batch=batch, ctx_lo=max(1, hi // 5), ctx_hi=hi, rows=_log(rng, 1, hi), kv_heads=kv, dim=dim,
                    page=page, dtype=dtype)
    rows = rng.choice([1, 1, 2, 3, 4, 5, 8, 16])
    batch = _log(rng, 1, 96)
    hi = _log(rng, rows + 1, max(rows + 2, min(60000, 150000 // batch)))
    window = rng.choice([0, _log(rng, 1, 8192)]) if op == "q4" else _log(rng, 1, 8192)
    return dict(op=op, batch=batch, ctx_lo=min(hi, max(rows, hi // 6)), ctx_hi=hi, rows=rows,
                heads=kv * rng.choice([1, 2, 3, 4, 5, 6, 8]), kv_heads=kv, dim=dim, page=page, dtype=dtype, window=window,
                sinks=rng.choice([0, 1, 4, 100]) if window else 0)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _dtype(name):
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[name]


def _row_bytes(kv_heads, dim):
    return (kv_heads * (dim // 2 + 4) + 15) // 16 * 16


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


def _q4_cache(g, pages, page, kv_heads, dim, dt):
    """Codes and parameters as tokens of normally distributed K and V have them: 15 steps span about 5.3 deviations."""
    cache = torch.zeros((pages, page, 1, _row_bytes(kv_heads, dim)), dtype=torch.uint8, device=DEV)
    half = kv_heads * dim // 2
    step = max(1, (1 << 26) // (page * kv_heads * dim))
    for p in range(0, pages, step):
        part = cache[p:p + step]
        code = torch.randn((part.shape[0], page, kv_heads * dim), generator=g, device=DEV, dtype=torch.float16)
        code = code.mul_(2.8).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
        part[:, :, 0, :half] = code[..., 0::2] | (code[..., 1::2] << 4)
        scale = (torch.rand((part.shape[0], page, kv_heads), generator=g, device=DEV) * 0.1 + 0.3).to(dt)
        low = (scale.float() * -(torch.rand(scale.shape, generator=g, device=DEV) + 7.0)).to(dt)
        part[:, :, 0, half:half + 4 * kv_heads] = torch.stack([scale, low], -1).reshape(*scale.shape[:2], -1).view(torch.uint8)
    return cache


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    B, R, K, D, page, dt = (case["batch"], case["rows"], case["kv_heads"], case["dim"], case["page"], _dtype(case["dtype"]))
    op = case["op"]
    ctx = torch.randint(case["ctx_lo"], case["ctx_hi"] + 1, (B,), generator=g, device=DEV)
    if op in ("window", "q4"):
        ctx = ctx.clamp(min=R)
    table, pages = _page_table(g, ctx, page, max(R, case["ctx_hi"]), 3)
    s = dict(op=op, page=page, kv_heads=K, dim=D, block_table=table, ctx_lens=ctx.to(torch.int32),
             window=case.get("window", 0), sinks=case.get("sinks", 0))
    if op in ("window", "q4"):
        s["q"] = torch.randn((B, R, case["heads"], D), generator=g, device=DEV, dtype=dt)
        s["out"] = torch.empty_like(s["q"])
    if op == "window":
        for n in ("k_cache", "v_cache"):
            s[n] = torch.randn((pages, page, K, D), generator=g, device=DEV, dtype=dt)
    elif op == "store":
        for n in ("k_cache", "v_cache"):
            s[n] = torch.zeros((pages, page, 1, _row_bytes(K, D)), dtype=torch.uint8, device=DEV)
    else:
        for n in ("k_cache", "v_cache"):
            s[n] = _q4_cache(g, pages, page, K, D, dt)
    if op == "store":
        for n in ("k", "v"):
            s[n] = torch.randn((B, R, K, D), generator=g, device=DEV, dtype=dt)
    if op in ("store", "load"):
        for n in ("k_out", "v_out"):
            s[n] = torch.empty((B, R, K, D), device=DEV, dtype=dt)
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _unpack(rows, kv_heads, dim, dt):
    """[..., row bytes] -> values [..., kv_heads, dim] in 32 bits."""
    half = kv_heads * dim // 2
    codes = rows[..., :half]
    codes = torch.stack([codes & 15, codes >> 4], -1).reshape(*rows.shape[:-1], kv_heads, dim).float()
    par = rows[..., half:half + 4 * kv_heads].contiguous().view(dt).float().reshape(*rows.shape[:-1], kv_heads, 2)
    return codes * par[..., :1] + par[..., 1:]


def _plain_attention(s):
    q, table, ctx = s["q"].float(), s["block_table"].long().clamp(min=0), s["ctx_lens"].long()
    B, R, H, D = q.shape
    K, page = s["kv_heads"], s["page"]
    G = H // K
    # the pages that some row sees: the first ones, and the newest ones
    W = table.shape[1]
    if s["window"]:
        first = min(W, -(-s["sinks"] // page))
        count = min(W - first, (s["window"] + R - 2) // page + 2)
        last = (ctx + page - 1) // page
        at = (last - count).clamp(min=first)[:, None] + torch.arange(count, device=DEV)
        at = torch.cat([torch.arange(first, device=DEV).expand(B, first), at], 1)
    else:
        at = torch.arange(W, device=DEV).expand(B, W)
    T = at.shape[1] * page
    t = (at[:, :, None] * page + torch.arange(page, device=DEV)).reshape(B, T)
    ids = table.gather(1, at.clamp(max=W - 1))
    if s["op"] == "q4":
        k, v = (_unpack(s[n][ids][:, :, :, 0].reshape(B, T, -1), K, D, s["q"].dtype) for n in ("k_cache", "v_cache"))
    else:
        k, v = (s[n][ids].reshape(B, T, K, D).float() for n in ("k_cache", "v_cache"))
    pos = (ctx - R)[:, None] + torch.arange(R, device=DEV)
    sees = t[:, None, :] <= pos[:, :, None]
    if s["window"]:
        sees &= (t[:, None, :] > pos[:, :, None] - s["window"]) | (t[:, None, :] < s["sinks"])
    sees = sees[:, None, None]
    rows = q.reshape(B, R, K, G, D).permute(0, 2, 3, 1, 4).reshape(B, K, G * R, D) * D ** -0.5
    x = torch.matmul(rows, k.permute(0, 2, 3, 1)).reshape(B, K, G, R, T)
    x = torch.where(sees, x, -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    out = torch.matmul(x.reshape(B, K, G * R, T), v.permute(0, 2, 1, 3)).reshape(B, K, G, R, D) / x.sum(-1, keepdim=True)
    return out.permute(0, 3, 1, 2, 4).reshape(B, R, H, D).to(s["out"].dtype)


def _token_rows(s, rows):
    """Where the last `rows` tokens of every sequence lie in the cache, and which of them exist."""
    pos = s["ctx_lens"].long()[:, None] - rows + torch.arange(rows, device=DEV)
    t = pos.clamp(min=0)
    page = s["block_table"].long().gather(1, t // s["page"])
    return page * s["page"] + t % s["page"], pos >= 0


def _plain_store(s):
    B, R, K, D = s["k"].shape
    dt = s["k"].dtype
    at, there = _token_rows(s, R)
    for x, n in ((s["k"], "k_cache"), (s["v"], "v_cache")):
        low, high = x.float().amin(-1, keepdim=True), x.float().amax(-1, keepdim=True)
        scale = ((high - low) / torch.full_like(low, 15.0)).to(dt)
        # the quotient in 64 bits: it decides between neighbouring codes
        code = ((x.double() - low.double()) / torch.where(scale > 0, scale, 1.0).double()).round().clamp(0, 15).to(torch.uint8)
        code = code.reshape(B, R, K * D)
        par = torch.stack([scale[..., 0], low[..., 0].to(dt)], -1).reshape(B, R, 2 * K).view(torch.uint8)
        rows = torch.cat([code[..., 0::2] | (code[..., 1::2] << 4), par], -1)
        flat = s[n].reshape(-1, s[n].shape[-1])
        flat[at[there], :rows.shape[-1]] = rows[there]


def _plain_load(s):
    R, dt = s["k_out"].shape[1], s["k_out"].dtype
    at, there = _token_rows(s, R)
    at = torch.where(there, at, 0)
    for n in ("k", "v"):
        rows = s[n + "_cache"].reshape(-1, s[n + "_cache"].shape[-1])[at]
        x = _unpack(rows, s["kv_heads"], s["dim"], dt).to(dt)
        s[n + "_out"].copy_(torch.where(there[:, :, None, None], x, 0.0))
    return dict(k=s["k_out"], v=s["v_out"])


def run(s):
    op = s["op"]
    if own:
        import speculative_decoding_verification_paged_gb300 as sv
        if op in ("window", "q4") and "workspace" not in s:  # kept for the program's life, like the cache
            s["workspace"] = sv.new_attention_workspace(
                sv.spec_window_attention_workspace(s["q"], s["kv_heads"], s["block_table"]), DEV)
        if op == "window":
            return sv.spec_window_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["ctx_lens"], s["out"],
                                            window=s["window"], sinks=s["sinks"], workspace=s["workspace"])
        if op == "q4":
            return sv.spec_q4_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["ctx_lens"], s["kv_heads"],
                                        s["out"], window=s["window"], sinks=s["sinks"], workspace=s["workspace"])
        if op == "store":
            sv.spec_cache_store_q4(s["k"], s["v"], s["block_table"], s["ctx_lens"], s["k_cache"], s["v_cache"])
        sv.spec_cache_load_q4(s["k_cache"], s["v_cache"], s["block_table"], s["ctx_lens"], s["k_out"], s["v_out"])
        return dict(k=s["k_out"], v=s["v_out"])
    if op in ("window", "q4"):
        return _plain_attention(s)
    if op == "store":
        _plain_store(s)
    # what a store has left in 4 bits is returned as the values it stands for
    return _plain_load(s)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    B, R, K, D = case["batch"], case["rows"], case["kv_heads"], case["dim"]
    lo, hi = case["ctx_lo"], max(case["ctx_hi"], case["ctx_lo"])

    def mean(most):  # of min(ctx, most) over the contexts
        if lo == hi or most <= lo:
            return min(lo, most)
        if most >= hi:
            return (lo + hi) / 2
        return ((lo + most) / 2 * (most - lo) + most * (hi - most)) / (hi - lo)

    if case["op"] in ("store", "load"):
        n = B * mean(R) * K * D * 2.0
        moved = B * R * K * D * 2.0 * 2 + n * (0.5 + 4 / D)  # 16-bit values, codes and parameters
        return dict(bytes=moved + (n * 2 if case["op"] == "store" else 0), flops=n * 2)
    keys = mean(case["sinks"] + case["window"] + R - 1 if case["window"] else hi)
    token = 2 * (D / 2 + 4) if case["op"] == "q4" else 4 * D
    return dict(bytes=B * (keys * K * token + R * case["heads"] * D * 4 + keys / case["page"] * 4),
                flops=4.0 * B * keys * R * case["heads"] * D)


# ---------------------------------------------------------------------------
# 64 bits, one sequence at a time
# ---------------------------------------------------------------------------
def _exact_rows(case, rows, h):
    """Values [tokens, D] of kv head h of 4-bit token rows [tokens, bytes]."""
    K, D = case["kv_heads"], case["dim"]
    codes = rows[:, h * D // 2:(h + 1) * D // 2]
    par = rows[:, K * D // 2 + 4 * h:K * D // 2 + 4 * h + 4].contiguous().view(_dtype(case["dtype"])).double()
    x = torch.empty((rows.shape[0], D), dtype=torch.float64, device=DEV)
    x[:, 0::2] = (codes % 16).double()
    x[:, 1::2] = (codes // 16).double()
    return x * par[:, 0:1] + par[:, 1:2]


def _exact_attention(case, s):
    B, R, H, D = s["q"].shape
    K, page, W, S = case["kv_heads"], case["page"], case["window"], case["sinks"]
    out = torch.zeros((B, R, H, D), dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["ctx_lens"].tolist()):
        t = torch.arange(n, device=DEV)
        if W:
            t = t[(t < S) | (t > n - R - W)]
        slot = s["block_table"][b].long()[t // page] * page + t % page
        for h in range(K):
            if case["op"] == "q4":
                k, v = (_exact_rows(case, s[c].reshape(-1, s[c].shape[-1])[slot], h) for c in ("k_cache", "v_cache"))
            else:
                k, v = (s[c].reshape(-1, K, D)[slot, h].double() for c in ("k_cache", "v_cache"))
            heads = slice(h * (H // K), (h + 1) * (H // K))
            for i in range(R):
                p = n - R + i
                see = t <= p
                if W:
                    see &= (t < S) | (t > p - W)
                x = (s["q"][b, i, heads].double() @ k.T / math.sqrt(D)).masked_fill(~see, -math.inf)
                out[b, i, heads] = torch.softmax(x, -1) @ v
    return out


def _exact_values(case, s):
    B, R, K, D, page = case["batch"], case["rows"], case["kv_heads"], case["dim"], case["page"]
    got = {}
    for n in ("k", "v"):
        x = torch.zeros((B, R, K, D), dtype=torch.float64, device=DEV)
        for b, ctx in enumerate(s["ctx_lens"].tolist()):
            c = min(R, ctx)
            if case["op"] == "load":
                t = torch.arange(ctx - c, ctx, device=DEV)
                slot = s["block_table"][b].long()[t // page] * page + t % page
                rows = s[n + "_cache"].reshape(-1, s[n + "_cache"].shape[-1])[slot]
                for h in range(K):
                    x[b, R - c:, h] = _exact_rows(case, rows, h)
                continue
            y = s[n][b, R - c:].double()
            low = y.amin(-1, keepdim=True)
            step = ((y.amax(-1, keepdim=True) - low) / 15).float().to(s[n].dtype).double()
            safe = torch.where(step > 0, step, 1.0)
            x[b, R - c:] = ((y - low) / safe).round().clamp(0, 15) * step + low
        got[n] = x
    return got


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_attention(case, s) if case["op"] in ("window", "q4") else _exact_values(case, s)
