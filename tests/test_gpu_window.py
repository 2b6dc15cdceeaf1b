"""Windowed attention and the 4-bit cache on the GPU against their 64-bit definitions (window_oracle).

Attention tolerances, per element, with S = sum_t p_t |v_t|:
  * one rounding of the weights to 16 bits and one of the result, half the step of the type each: 2^-8 for bf16, 2^-11
    for fp16, relative to S and to |ref|;
  * fp32 scores, exponentials and sums: 2^-16 S, and the smallest normal number of the output type;
  * over a 4-bit cache what is rounded (to fp16) is p_t s_t, which meets codes that are at most 7.5 from their middle:
    2^-11 of Q = 7.5 sum_t p_t s_t instead of the first rounding, and 2^-16 Q for the two halves of s n + m, which are
    summed apart. fp16 weights have a least step: 2^-30 of the largest p_t s_t for each token.
"""

import numpy as np
import pytest
import torch

import window_oracle as wo

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, FP = torch.bfloat16, torch.float16
HALF = {BF: 2.0 ** -8, FP: 2.0 ** -11}


def cuda(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x)).to(DEV, dtype)


def page_tables(rng, ctx, rows, window, sinks, bs, spare=2):
    """Tables that name distinct pages where some row sees one and anything else elsewhere; and the page count."""
    W = max(1, -(-max(ctx) // bs)) + 1
    seen = [wo.pages_seen(c, rows, window, sinks, bs) if c >= rows else np.zeros(0, int) for c in ctx]
    P = sum(len(s) for s in seen) + spare
    order = rng.permutation(P)
    table = rng.choice([-1, -7, P, 2 ** 30], (len(ctx), W))
    at = 0
    for b, s in enumerate(seen):
        table[b, s] = order[at: at + len(s)]
        at += len(s)
    return table, P


def make(rng, ctx, R, H, K, D, bs, dtype, window, sinks, q4, scale=1.0):
    """One call's inputs. Slots that no row sees hold NaN (4-bit: NaN for s and m, any codes)."""
    ctx = list(ctx)
    table, P = page_tables(rng, ctx, R, window, sinks, bs)
    q = torch.from_numpy(rng.standard_normal((len(ctx), R, H, D)).astype(np.float32) * scale).to(dtype)
    caches, values, spread = [], [], None
    dead = np.ones((P, bs), bool)
    for b, c in enumerate(ctx):
        if c < R:
            continue
        t = np.flatnonzero(wo.sees(c, R, window, sinks).any(0))
        dead[table[b, t // bs], t % bs] = False
    for _ in range(2):
        x = torch.from_numpy(rng.standard_normal((P, bs, K, D)).astype(np.float32)).to(dtype)
        if q4:
            codes = np.clip(np.round(x.double().numpy() * 2.8 + 7.5), 0, 15).astype(int)
            s = wo.round16(0.3 + 0.2 * rng.random((P, bs, K)), dtype)
            m = wo.round16(-s * (7.0 + rng.random((P, bs, K))), dtype)
            s[dead], m[dead] = np.nan, np.nan
            rows = wo.pack(codes, s, m, dtype)
            values.append(wo.unpack(rows, K, D, dtype)[0])
            spread = s
            caches.append(torch.from_numpy(rows)[:, :, None, :].contiguous().to(DEV))
        else:
            x[torch.from_numpy(dead)] = float("nan")
            values.append(x.double().numpy())
            caches.append(x.to(DEV))
    return dict(q=q.to(DEV), k=caches[0], v=caches[1], table=cuda(table), ctx=cuda(ctx), K=K, window=window, sinks=sinks, q4=q4,
                host=(q.double().numpy(), values[0], values[1], spread, table, ctx), bs=bs)


def call(sv, c, ws=None, out=None, stream=None):
    out = torch.full(c["q"].shape, float("nan"), dtype=c["q"].dtype, device=DEV) if out is None else out
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    kw = dict(window=c["window"], sinks=c["sinks"], workspace=ws, dev_err=err, stream=stream)
    if c["q4"]:
        sv.spec_q4_attention(c["q"], c["k"], c["v"], c["table"], c["ctx"], c["K"], out, **kw)
    else:
        sv.spec_window_attention(c["q"], c["k"], c["v"], c["table"], c["ctx"], out, **kw)
    torch.cuda.synchronize()
    return out, int(err.item())


def reference(c, b):
    """(ref, tolerance) of sequence b."""
    q, k, v, spread, table, ctx = c["host"]
    n, bs, dtype = ctx[b], c["bs"], c["q"].dtype
    t = np.arange(n)
    see = wo.sees(n, q.shape[1], c["window"], c["sinks"])
    page = np.where(see.any(0), table[b, t // bs], 0)
    pick = lambda x: x[page, t % bs]  # noqa: E731
    ref, S, Q, top = wo.attention(q[b], pick(k), pick(v), c["window"], c["sinks"], None if spread is None else pick(spread))
    tol = 2.0 ** -16 * S + HALF[dtype] * np.abs(ref) * (1 + 2.0 ** -6) + torch.finfo(dtype).smallest_normal
    if spread is None:
        tol = tol + HALF[dtype] * S * (1 + 2.0 ** -6)
    else:
        tol = tol + 7.5 * (Q * (2.0 ** -11 + 2.0 ** -16) + top * 2.0 ** -30 * see.sum(1)[:, None])[..., None] * (1 + 2.0 ** -6)
    return ref, tol


def check(c, out):
    q, ctx = c["host"][0], c["host"][5]
    got = out.double().cpu().numpy()
    for b, n in enumerate(ctx):
        if n < q.shape[1]:
            assert not got[b].any()
            continue
        ref, tol = reference(c, b)
        assert np.isfinite(got[b]).all(), (b, np.argwhere(~np.isfinite(got[b]))[:5])
        bad = np.abs(got[b] - ref) > tol
        assert not bad.any(), (b, int(bad.sum()), np.argwhere(bad)[:5], np.abs(got[b] - ref)[bad][:5], tol[bad][:5], ref[bad][:5])


# (contexts, rows, query heads, kv heads, head dim, page, window, sinks): one token to many tiles; contexts and windows
# just below, at and above page and tile edges; an empty row; windows of one token, longer than the context, and none;
# sinks inside, next to and over the window; packed rows from 1 to 512 a kv head.
CASES = [
    ((1, 2, 17, 128, 129), 1, 4, 4, 64, 16, 0, 0),
    ((5, 16, 17, 300, 0, 701), 5, 9, 3, 64, 16, 100, 3),
    ((4, 130, 1000), 4, 8, 8, 64, 32, 1, 0),
    ((64, 127, 191, 700), 64, 8, 1, 64, 32, 64, 1),
    ((1000, 257, 3), 3, 6, 2, 64, 128, 0, 0),
    ((4, 127, 128, 129, 1000), 4, 32, 8, 128, 64, 128, 4),
    ((2048, 0, 900), 1, 32, 8, 128, 64, 0, 0),
    ((33, 161, 640), 33, 8, 2, 128, 128, 300, 16),
    ((3000, 1500), 2, 14, 2, 128, 16, 257, 100),
    ((4096, 70), 8, 16, 2, 128, 128, 0, 0),
    ((3, 700), 3, 64, 1, 128, 32, 20, 130),
    ((50, 900), 16, 24, 3, 128, 64, 10 ** 9, 5),
    ((130, 258, 1100), 1, 5, 1, 256, 32, 129, 0),
    ((16, 80, 129, 900), 16, 24, 4, 256, 64, 200, 1),
    ((4, 1300, 600), 4, 24, 4, 256, 16, 0, 0),
    ((7, 2000), 7, 16, 1, 256, 128, 1000, 10 ** 9),
]
IDS = [f"R{c[1]}-{c[2]}h{c[3]}-d{c[4]}-p{c[5]}-w{c[6]}" for c in CASES]


@pytest.mark.parametrize("q4", [False, True], ids=["16bit", "q4"])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_attention(sv, case, dtype, q4):
    ctx, R, H, K, D, bs, window, sinks = case
    c = make(np.random.default_rng(sum(ctx) + R + H + D), ctx, R, H, K, D, bs, dtype, window, sinks, q4)
    out, err = call(sv, c)
    assert err == 0
    check(c, out)


@pytest.mark.parametrize("q4", [False, True], ids=["16bit", "q4"])
@pytest.mark.parametrize("scale", [4.0, 16.0])
def test_peaked_attention(sv, q4, scale):
    """Scores of several deviations: references that move while the keys pass, weights of every size."""
    for D, dtype in ((64, FP), (128, BF), (128, FP), (256, FP)):
        c = make(np.random.default_rng(D), (3000, 700), 4, 8, 2, D, 64, dtype, 0, 0, q4, scale)
        out, err = call(sv, c)
        assert err == 0
        # scores reach 2^8 in log2 units: an fp32 one is off by a few 2^-16
        q, ctx = c["host"][0], c["host"][5]
        got = out.double().cpu().numpy()
        for b in range(len(ctx)):
            ref, tol = reference(c, b)
            v = np.nan_to_num(c["host"][2])
            tol = tol + 2.0 ** -13 * np.abs(v).max() * (scale / 16)
            assert np.all(np.abs(got[b] - ref) <= tol)


@pytest.mark.parametrize("q4", [False, True], ids=["16bit", "q4"])
def test_values_of_very_different_size(sv, q4):
    """Tokens whose V differ by factors of 2^-20 to 2^20, and a first token that takes most of the weight and has no V:
    what the rows get is made of weights far below their largest."""
    for D, dtype in ((64, FP), (128, BF), (128, FP), (256, FP)):
        rng = np.random.default_rng(D + 7)
        c = make(rng, (2500, 300), 2, 8, 2, D, 64, dtype, 0, 0, q4)
        q, k, v, spread, table, ctx = c["host"]
        fac = np.exp2(rng.integers(-6, 7, v.shape[:3]) * (3 if dtype == BF else 1))
        fac[table[0, 0], 0] = fac[table[1, 0], 0] = 0.0
        if q4:
            rows = c["v"][:, :, 0].cpu().numpy()
            val, s, m = wo.unpack(rows, 2, D, dtype)
            s, m = wo.round16(s * fac, dtype), wo.round16(m * fac, dtype)
            codes = np.stack([rows[..., : D] % 16, rows[..., : D] // 16], -1).reshape(*rows.shape[:2], 2, D)
            rows = wo.pack(codes.astype(int), s, m, dtype)
            val, s, m = wo.unpack(rows, 2, D, dtype)
            c["v"] = torch.from_numpy(rows)[:, :, None, :].contiguous().to(DEV)
            spread = s
        else:
            val = wo.round16(np.nan_to_num(v) * fac[..., None], dtype)
            c["v"] = torch.from_numpy(val).to(dtype).to(DEV)
        # the first token's key is along every query of its group
        q[...] = np.abs(q)
        c["q"] = torch.from_numpy(q).to(dtype).to(DEV)
        q = c["q"].double().cpu().numpy()
        level = 16 * np.log(2) * D ** 0.5 / (np.sqrt(2 / np.pi) * D)
        if q4:
            rows = c["k"][:, :, 0].cpu().numpy()
            kv, ks, km = wo.unpack(rows, 2, D, dtype)
            codes = np.stack([rows[..., : D] % 16, rows[..., : D] // 16], -1).reshape(*rows.shape[:2], 2, D).astype(int)
            for b in range(2):
                codes[table[b, 0], 0] = 15
                ks[table[b, 0], 0] = wo.round16(level / 15, dtype)
                km[table[b, 0], 0] = 0
            rows = wo.pack(codes, ks, km, dtype)
            k = wo.unpack(rows, 2, D, dtype)[0]
            c["k"] = torch.from_numpy(rows)[:, :, None, :].contiguous().to(DEV)
        else:
            for b in range(2):
                k[table[b, 0], 0] = wo.round16(level, dtype)
            c["k"] = torch.from_numpy(k).to(dtype).to(DEV)
        c["host"] = (q, k, val, spread, table, ctx)
        out, err = call(sv, c)
        assert err == 0
        check(c, out)


def test_scores_without_a_value(sv):
    """A NaN or +inf among the scores that a row sees makes that row NaN and no other; -inf is a weight of zero."""
    for dtype in (BF, FP):
        c = make(np.random.default_rng(5), (900, 300), 3, 8, 2, 128, 64, dtype, 500, 4, False)
        q, k, v, _, table, ctx = c["host"]
        q[..., 5] = np.abs(q[..., 5]) + 0.5
        q[0, 1, 2, 7] = np.nan                                # one row of one head
        k[table[0, 700 // 64], 700 % 64, 1, 9] = np.nan       # all rows of kv head 1
        k[table[0, 0], 2, 0, 5] = -np.inf                     # a weight of zero
        k[table[1, 299 // 64], 299 % 64, 0, 5] = np.inf       # the last token: the last row of kv head 0
        c["q"], c["k"] = torch.from_numpy(q).to(dtype).to(DEV), torch.from_numpy(k).to(dtype).to(DEV)
        out, err = call(sv, c)
        assert err == 0
        got = out.double().cpu().numpy()
        nan = np.zeros(got.shape[:3], bool)
        nan[0, 1, 2] = True
        nan[0, :, 4:] = True
        nan[1, 2, :4] = True
        assert np.array_equal(np.isnan(got), np.repeat(nan[..., None], 128, -1))
        with np.errstate(invalid="ignore"):
            for b in range(2):
                ref, tol = reference(c, b)
                ok = ~nan[b]
                assert np.all(np.abs(got[b] - ref)[ok] <= tol[ok])


def test_q4_rows_are_kept_apart(sv):
    """NaN for s or m of a token reaches the rows that see it, and no other row."""
    c = make(np.random.default_rng(6), (900, 300), 3, 8, 2, 128, 64, BF, 500, 4, True)
    table, ctx = c["host"][4], c["host"][5]
    for name, tok, g in (("v", 899, 0), ("k", 898, 1)):       # the last token's V, the one before's K
        row = c[name][table[0, tok // 64], tok % 64, 0]
        row[128 + 4 * g: 128 + 4 * g + 4] = torch.tensor([0xff, 0x7f, 0xff, 0x7f], dtype=torch.uint8, device=DEV)
    out, err = call(sv, c)
    assert err == 0
    nan = torch.zeros(out.shape[:3], dtype=torch.bool)
    nan[0, 2, :4] = True
    nan[0, 1:, 4:] = True
    assert torch.equal(out.isnan().cpu(), nan[..., None].expand(out.shape))


@pytest.mark.parametrize("q4", [False, True], ids=["16bit", "q4"])
def test_bad_sequences_are_zeros_and_flagged(sv, q4):
    rng = np.random.default_rng(8)
    for bad, bit in (("len", 8), ("short", 8), ("page", 1), ("far", 1)):
        c = make(rng, (900, 700, 2100), 3, 8, 2, 128, 64, BF, 500, 4, q4)
        if bad == "len":
            c["ctx"][1] = c["table"].shape[1] * 64 + 1
        elif bad == "short":
            c["ctx"][1] = 2
        else:
            c["table"][1, 699 // 64] = -1 if bad == "page" else c["k"].shape[0]
        out, err = call(sv, c)
        assert err == bit
        assert not out[1].any()
        c["host"] = (*c["host"][:5], [900, 0, 2100])
        check(c, out)


# ---------------------------------------------------------------------------
# The 4-bit cache
# ---------------------------------------------------------------------------
def token_case(rng, ctx, R, K, D, bs, dtype, kind="normal"):
    B = len(ctx)
    W = max(1, -(-max(ctx) // bs)) + 1
    P = B * W + 3
    table = rng.permutation(P)[: B * W].reshape(B, W)
    x = [rng.standard_normal((B, R, K, D)) * np.exp(rng.standard_normal((B, R, K, 1)) * 3) for _ in range(2)]
    if kind == "ties":
        x = [rng.integers(-15, 16, (B, R, K, D)) / 2.0 for _ in range(2)]
        x[0][..., :2] = [-7.5, 7.5]
    elif kind == "ends":                                       # equal values, tiny and huge ranges, tiny beside large
        big, small = (3e38, 1e-40) if dtype == BF else (6e4, 1e-7)
        for y in x:
            y[..., 0::4] = rng.standard_normal(y[..., 0::4].shape) * 1e-6
            pick = rng.integers(0, 4, (B, R, K, 1))
            y[...] = np.where(pick == 0, 0.75, np.where(pick == 1, np.clip(y, -1, 1) * big, np.where(pick == 2, y * small, y)))
    return table, P, [torch.from_numpy(y).to(dtype) for y in x]


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("kind", ["normal", "ties", "ends"])
@pytest.mark.parametrize("ctx,R,K,D,bs", [((1, 40, 0, 17), 1, 1, 64, 16), ((70, 5, 129), 70, 3, 64, 32), ((300, 33), 33, 8, 128, 64),
                                          ((16, 300), 20, 5, 256, 128)])
def test_store_and_load(sv, ctx, R, K, D, bs, dtype, kind):
    rng = np.random.default_rng(R + K + D)
    table, P, x = token_case(rng, ctx, R, K, D, bs, dtype, kind)
    size = wo.row_bytes(K, D)
    before = torch.from_numpy(rng.integers(0, 256, (2, P, bs, 1, size)).astype(np.uint8)).to(DEV)
    cache = before.clone()
    # rows inside wider ones, as a projection's output has them
    wide = [torch.zeros((len(ctx), R, (K + 3) * D), dtype=dtype, device=DEV) for _ in x]
    parts = []
    for w, y in zip(wide, x):
        parts.append(w[:, :, D: (K + 1) * D].unflatten(-1, (K, D)))
        parts[-1].copy_(y)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    sv.spec_cache_store_q4(parts[0], parts[1], cuda(table), cuda(ctx), cache[0], cache[1], dev_err=err)
    want = before.cpu().numpy()[:, :, :, 0]
    body = K * (D // 2 + 4)
    values = []
    for w, y in enumerate(x):
        with np.errstate(invalid="ignore"):
            codes, s, m = wo.quantise(y.double().numpy(), dtype)
        rows = wo.pack(codes, s, m, dtype)
        val = wo.unpack(rows, K, D, dtype)[0]
        for b, n in enumerate(ctx):
            for i in range(R):
                t = n - R + i
                if t < 0:
                    val[b, i] = 0
                else:
                    want[w, table[b, t // bs], t % bs, :body] = rows[b, i, :body]
        values.append(val)
    assert int(err.item()) == 0
    have = cache.cpu().numpy()[:, :, :, 0]
    off = np.argwhere(have != want)
    assert off.size == 0, (len(off), off[:5], have[have != want][:5], want[have != want][:5])
    for out_dtype in (dtype, torch.float32):
        got = [torch.full((len(ctx), R, K, D), float("nan"), dtype=out_dtype, device=DEV) for _ in x]
        sv.spec_cache_load_q4(cache[0], cache[1], cuda(table), cuda(ctx), *got, dtype=dtype, dev_err=err)
        for g, val in zip(got, values):
            with np.errstate(over="ignore"):
                ref = torch.from_numpy(val.astype(np.float32)).to(out_dtype)
            assert torch.equal(g.isnan().cpu(), ref.isnan()) and torch.equal(g.cpu().nan_to_num(), ref.nan_to_num())
    assert int(err.item()) == 0


def test_store_of_what_has_no_value(sv):
    """A NaN or infinity makes its token's head NaN, and nothing else."""
    table, P, x = token_case(np.random.default_rng(9), (20,), 20, 3, 128, 16, FP)
    x[0][0, 3, 1, 100] = float("nan")
    x[0][0, 5, 2, 0] = float("inf")
    x[1][0, 7, 0, 127] = float("-inf")
    cache = [sv.new_q4_cache(P, 16, 3, 128, DEV) for _ in x]
    sv.spec_cache_store_q4(x[0].to(DEV), x[1].to(DEV), cuda(table), cuda([20]), *cache)
    got = [torch.empty_like(y, device=DEV) for y in x]
    sv.spec_cache_load_q4(*cache, cuda(table), cuda([20]), *got)
    for g, y in zip(got, x):
        bad = ~torch.isfinite(y).all(-1)
        assert torch.equal(g.isnan().cpu(), bad[..., None].expand(y.shape))


def test_store_and_load_of_bad_rows(sv):
    """Bad lengths and pages write nothing, read as zeros and are flagged; the rest of the batch is as ever."""
    rng = np.random.default_rng(10)
    ctx = [100, 40, 90, 64]
    table, P, x = token_case(rng, ctx, 30, 2, 64, 16, BF)
    bad = table.copy()
    bad[0, 80 // 16] = P
    bad[2, 70 // 16] = -1
    lens = [100, -1, 90, table.shape[1] * 16 + 1]
    for c_table, c_lens, bits in ((bad, ctx, 1), (table, lens, 8)):
        cache = [sv.new_q4_cache(P, 16, 2, 64, DEV) for _ in x]
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        sv.spec_cache_store_q4(x[0].to(DEV), x[1].to(DEV), cuda(c_table), cuda(c_lens), *cache, dev_err=err)
        assert int(err.item()) == bits
        err.zero_()
        got = [torch.full_like(y, float("nan"), device=DEV) for y in x]
        sv.spec_cache_load_q4(*cache, cuda(c_table), cuda(c_lens), *got, dev_err=err)
        assert int(err.item()) == bits
        for g, y in zip(got, x):
            codes, s, m = wo.quantise(y.double().numpy(), BF)
            val = codes * s[..., None] + m[..., None]
            for b in range(4):
                for i in range(30):
                    t = ctx[b] - 30 + i
                    if c_lens[b] != ctx[b] or not 0 <= c_table[b, t // 16] < P:
                        val[b, i] = 0
            assert torch.equal(g.cpu(), torch.from_numpy(val.astype(np.float32)).to(BF))
        assert int(err.item()) == bits
