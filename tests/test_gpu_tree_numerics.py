"""The tree calls on inputs at the ends of their range: weights far below a row's largest, temperatures near zero,
NaN and infinities where a row sees them."""

import numpy as np
import pytest
import torch

import test_gpu_tree as tg
import tree_oracle as to
from test_gpu_tree import DEV, HALF

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# fp16: weights far below the largest
# ---------------------------------------------------------------------------
def sink_case(ctx, D, bits, sink_v, spread, at=0):
    """One sequence whose token `at` has 2^bits the weight of any other (times 2^+-spread); V has a mean, so that a
    bias of the small weights shows. 4 nodes that see the committed tokens and themselves."""
    rng = np.random.default_rng(int(D + bits * 7 + spread * 3 + at))
    N, H, K, bs = 4, 4, 2, 64
    c = tg.attention_case(rng, (ctx,), N, H, K, D, bs, torch.float16, par=np.array([[-1, -1, -1, -1]]))
    table = c["host"][0]
    q, k, v = (c[n].clone() for n in ("q", "k", "v"))
    q[...] = 0
    q[..., 0] = 8.0
    k[...] = 0
    level = rng.uniform(-1, 1, tuple(k.shape[:-1])) * spread * np.log(2) * D ** 0.5 / 8.0
    k[..., 0] = torch.from_numpy(level).to(DEV, torch.float16)
    k[table[0, at // bs], at % bs, :, 0] = bits * np.log(2) * D ** 0.5 / 8.0
    v += 0.5
    v = torch.nan_to_num(v)
    v[table[0, at // bs], at % bs] *= sink_v
    c.update(q=q, k=k, v=v, clean=[t.float().cpu().numpy() for t in (q, k, v)])
    return c


@pytest.mark.parametrize("out_dtype", [torch.float16, torch.float32], ids=["f16", "f32"])
@pytest.mark.parametrize("D,ctx,at", [(64, 20000, 0), (128, 40000, 0), (128, 9000, 8000), (256, 9000, 70)])
@pytest.mark.parametrize("bits", [14, 20, 26, 34])
@pytest.mark.parametrize("sink_v,spread", [(0.0, 0.0), (0.0, 1.5), (1.0, 1.5)])
def test_fp16_weights_far_below_the_largest(sv, bits, sink_v, spread, D, ctx, at, out_dtype):
    """Weights are held as 2^11 times their ratio to a reference m that stays within 2^4 below and 2^10 above the tile's
    largest weight w_j (or 2^-40 of the row's largest, p): a part's step of 2^-24 at most leaves 2^-36 min(p, 2^10 w_j)
    of each of a tile's 128 keys. The rest is as for other inputs: 2^-16 S, and a rounding of the weights and of the
    result for fp16 output."""
    c = sink_case(ctx, D, bits, sink_v, spread, at)
    got, err = tg.run_attention(sv, c, out_dtype)
    assert err == 0
    q, k, v = c["clean"]
    table, lens, par = c["host"]
    ref, S = to.attention(q, k, v, table, lens, par)
    base = ctx - 4
    keys = k[table[0, : -(-ctx // 64)]].reshape(-1, 2, D)[:base].astype(np.float64)
    p = np.exp(8.0 * keys[:, :, 0] / np.sqrt(D))
    p /= p.sum(0)
    tiles = np.maximum.reduceat(p, np.arange(0, base, 64), axis=0)
    top = p.max(0)
    held = np.minimum(top, np.maximum(2.0 ** 10 * tiles, 2.0 ** -40 * top)).sum(0)  # [K]
    tol = 2.0 ** -16 * S + 2.0 ** -29 * np.repeat(held, 2)[None, None, :, None] * np.abs(v).max()
    if out_dtype == torch.float16:
        tol = tol + HALF[out_dtype] * (S + np.abs(ref)) * (1 + 2.0 ** -6) + torch.finfo(out_dtype).smallest_normal
    diff = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(diff <= tol), (float((diff / S).max()), float((tol / S).min()))


@pytest.mark.parametrize("out_dtype", [torch.float16, torch.float32], ids=["f16", "f32"])
def test_fp16_scores_that_rise_and_fall(sv, out_dtype):
    """Scores whose level wanders by 2^+-30 along the sequence, in steps of a tile and within tiles, N(0,1) on top."""
    rng = np.random.default_rng(71)
    for D, ctx in ((64, (900, 5000)), (128, (700, 6000)), (256, (650, 3000))):
        N, bs = 12, 64
        c = tg.attention_case(rng, ctx, N, 8, 2, D, bs, torch.float16)
        table, lens, par = c["host"]
        q, k = torch.nan_to_num(c["q"]), c["k"]
        q[..., 0] = 8.0
        for b in range(2):
            for t in range(int(lens[b])):
                level = 20 * np.sin(t / 200.0) + (15 if t % 517 == 3 else 0)
                k[table[b, t // bs], t % bs, :, 0] = float(level * np.log(2) * D ** 0.5 / 8.0)
        c["q"], c["clean"][0] = q, q.float().cpu().numpy()
        c["clean"][1] = np.nan_to_num(k.float().cpu().numpy())
        got, err = tg.run_attention(sv, c, out_dtype)
        assert err == 0
        ref, S = to.attention(*c["clean"], *c["host"])
        # scores reach 2^6 in log2 units: an fp32 one is off by a few 2^-18, and p by as much; and the tiles' 2^-29 * 2^10
        # w_j of above, where the w_j together are at most 1
        tol = 2.0 ** -15 * S + 2.0 ** -19 * np.abs(c["clean"][2]).max() * (S > 0)
        if out_dtype == torch.float16:
            tol = tol + HALF[out_dtype] * (S + np.abs(ref)) * (1 + 2.0 ** -6) + torch.finfo(out_dtype).smallest_normal
        assert np.all(np.abs(got.double().cpu().numpy() - ref) <= tol)


# ---------------------------------------------------------------------------
# NaN and infinities that a row sees
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,out_dtype", [(torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16),
                                             (torch.float16, torch.float32)], ids=["bf16_f32", "bf16", "fp16_f32"])
@pytest.mark.parametrize("D,ctx", [(64, (300, 2500, 70)), (128, (300, 2500, 70)), (128, (2304, 2304, 2304)), (256, (300, 2500, 70))])
def test_attention_scores_without_a_value(sv, dtype, out_dtype, D, ctx):
    """A NaN or +inf among the scores that a row sees makes that row NaN, as the formula does, and no other; a score of
    -inf is a weight of zero."""
    rng = np.random.default_rng(D + ctx[0])
    N, H, K, bs = 12, 8, 2, 64
    par = random_line_trees(rng, len(ctx), N)
    c = tg.attention_case(rng, ctx, N, H, K, D, bs, dtype, par=par)
    table, lens, par = c["host"]
    q, k = c["q"], c["k"]
    q[..., 5] = q[..., 5].abs() + 0.5                                    # signs of infinities are then known
    row = lambda b, t: (int(table[b, t // bs]), t % bs)  # noqa: E731
    q[0, 2, 3, 7] = float("nan")                                         # one row of one head
    k[(*row(0, int(lens[0]) - N + 4), 1, 9)] = float("nan")              # a node: itself and its descendants
    k[(*row(1, 1200 if lens[1] > 1300 else 40), 0, 5)] = float("nan")    # a committed token: all rows of a kv head
    k[(*row(1, 30), 1, 5)] = float("-inf")                               # a weight of zero
    k[(*row(2, 10), 0, 5)] = float("inf")
    got, err = tg.run_attention(sv, c, out_dtype)
    assert err == 0
    keep = k.float().cpu().numpy()
    for b in range(len(ctx)):                                            # slots that no row sees
        for j in range(N):
            if par[b, j] == to.UNUSED:
                keep[row(b, int(lens[b]) - N + j)] = 0
        for t in range(int(lens[b]), -(-int(lens[b]) // bs) * bs):
            keep[row(b, t)] = 0
    with np.errstate(invalid="ignore"):
        ref, S = to.attention(q.float().cpu().numpy(), keep, c["clean"][2], table, lens, par)
    x = got.double().cpu().numpy()
    used = np.asarray(par) != to.UNUSED
    nan = np.isnan(ref)
    assert nan[0, 2, 3].all() and nan[1, used[1], :4].all() and nan[2, used[2], :4].all()
    assert not nan[1, :, 4:].any() and not nan[2, :, 4:].any() and not nan[0, 0].any()
    assert np.array_equal(np.isnan(x), nan)
    tol = 2.0 ** -16 * S
    if out_dtype != torch.float32:
        tol = tol + HALF[out_dtype] * (S + np.abs(ref)) * (1 + 2.0 ** -6) + torch.finfo(out_dtype).smallest_normal
    tol = tol + (2.0 ** -19 * np.abs(c["clean"][2]).max() if dtype == torch.float16 else 0.0)
    assert np.all(np.abs(x - ref)[~nan] <= tol[~nan])


def random_line_trees(rng, B, N):
    par = np.zeros((B, N), np.int64)
    for b in range(B):
        for i in range(1, N):
            par[b, i] = to.UNUSED if i >= N - b else rng.integers(0, i)
        par[b, 0] = to.ROOT
        par[b, 4] = 1
    return par


# ---------------------------------------------------------------------------
# Acceptance at temperatures near zero
# ---------------------------------------------------------------------------
def cold_case(rng, B, V, temperature, probs, offset=0.0):
    """Rows whose node 0 has a largest logit of 10 to 30 and one, at some rows, within a few temperatures of it; the
    children of every node hold the largest logit's token, the second's and one more."""
    N = 7
    c = tg.accept_case(rng, B, N, V, "sample", probs)
    c["par"] = np.tile([-1, 0, 0, 0, 1, 1, 2], (B, 1))
    c["temp"][:] = temperature
    l = np.minimum(c["logits"], 9.0)
    for b in range(B):
        for n in range(N):
            x, y = rng.choice(V, 2, replace=False)
            top = np.float32(rng.uniform(10, 30))
            l[b, n, x] = top
            if (b + n) % 3 == 0:
                l[b, n, y] = top - np.float32(temperature * rng.uniform(0, 3))
            for j, i in enumerate(np.flatnonzero(c["par"][b] == n)):
                c["tok"][b, i] = (x, y, (x + 1) % V)[(j + b) % 3]
            if probs:
                q = np.full(V, 0.2 / V, np.float32)
                q[x] += 0.5
                q[y] += 0.3
                c["probs"][b, n] = q
    c["logits"] = (l + np.float32(offset)).astype(np.float32)
    return c


@pytest.mark.parametrize("probs", [False, True])
@pytest.mark.parametrize("temperature,offset", [(1e-3, 0.0), (1e-5, 0.0), (1e-6, 0.0), (1e-8, 0.0), (1e-30, 0.0),
                                                (1e-40, 0.0), (1.0, 1e4), (0.05, -3e4), (1e4, 0.0)])
@pytest.mark.parametrize("B,V", [(160, 512), (24, 33000)])
def test_accept_at_small_temperatures_and_large_logits(sv, B, V, temperature, offset, probs):
    """Exponents of the softmax reach 10^9 and more; the decisions are those of 64 bits, and no row ends without a
    token."""
    c = cold_case(np.random.default_rng(V + int(probs)), B, V, temperature, probs, offset)
    got, err = tg.run_accept(sv, c)
    assert err == 0
    m = tg.check_accept(c, got)
    at = got[0][np.arange(B), np.maximum(m, 0)]
    assert np.all(at >= 0) and (m.max() > 0 or temperature > 1)  # (a flat distribution accepts next to nothing)


# ---------------------------------------------------------------------------
# Acceptance of rows that hold a NaN or an infinity
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("probs", [False, True])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("V", [700, 33000, 33001])
def test_accept_one_entry_without_a_value(sv, V, value, probs):
    """One NaN or +inf among the logits of an inner node (rows 1 to 3) or of a leaf (rows 4 to 6), in the first, a
    middle and the last part of the vocabulary: the row ends there with -1; the others are as without it."""
    B, N = 8, 5
    c = tg.accept_case(np.random.default_rng(81), B, N, V, "sample", probs)
    c["par"][:] = [-1, 0, 0, 1, 2]
    c["tok"][:] = np.arange(B)[:, None] * 3 + np.arange(N)
    c["logits"][4:7, 0] = -50.0
    c["logits"][[4, 5, 6], 0, c["tok"][4:7, 1]] = 50.0        # node 1 is accepted for certain,
    c["logits"][4:7, 1] = -50.0
    c["logits"][[4, 5, 6], 1, c["tok"][4:7, 3]] = 50.0        # then its child, a leaf
    good, err = tg.run_accept(sv, c)
    bad = dict(c, logits=c["logits"].copy())
    for r, x in enumerate((0, V // 2, V - 1)):
        bad["logits"][1 + r, 0, x] = value
        bad["logits"][4 + r, 3, x] = value
    got, err2 = tg.run_accept(sv, bad)
    assert err == 0 and err2 == 0
    for x, y in zip(got, good):
        assert np.array_equal(x[[0, 7]], y[[0, 7]])
    for b in (1, 2, 3):
        assert got[2][b] == 0 and got[1][b].tolist() == [0, -1, -1, -1, -1] and got[0][b].tolist() == [-1] * 5
    for b in (4, 5, 6):
        assert got[2][b] == 2 and got[1][b].tolist() == [0, 1, 3, -1, -1]
        assert got[0][b].tolist() == [int(c["tok"][b, 1]), int(c["tok"][b, 3]), -1, -1, -1]


@pytest.mark.parametrize("probs", [False, True])
@pytest.mark.parametrize("V", [1, 5, 700, 40000, 128256])
def test_accept_a_nan_among_impossible_tokens(sv, V, probs):
    """One NaN where all other entries of its neighbourhood are -inf (a masked vocabulary), or the only entry."""
    B, N = 9, 3
    c = tg.accept_case(np.random.default_rng(82), B, N, V, "sample", probs)
    c["par"][:] = [-1, 0, 0]
    keep = c["logits"][:, 0, : max(1, V // 50)].copy()
    c["logits"][:, 0] = -np.inf
    c["logits"][:, 0, : keep.shape[1]] = keep
    good, err = tg.run_accept(sv, c)
    bad = dict(c, logits=c["logits"].copy())
    for b in range(1, B):
        bad["logits"][b, 0, min(V - 1, V * b // (B - 1))] = np.nan
    got, err2 = tg.run_accept(sv, bad)
    assert err == 0 and err2 == 0
    for x, y in zip(got, good):
        assert np.array_equal(x[0], y[0])
    assert np.all(good[0][:, 0] >= 0)
    assert np.all(got[2][1:] == 0) and np.all(got[0][1:] == -1) and np.all(got[1][1:] == [0, -1, -1])


@pytest.mark.parametrize("size", [(1 << 32) + 4, 1 << 31, -(1 << 32) + 4])
def test_update_refuses_block_sizes_past_32_bits(sv, size):
    table, refs, n = (torch.zeros(s, dtype=torch.int32, device=DEV) for s in ((1, 2), (4,), (1,)))
    with pytest.raises(ValueError):
        sv.spec_cache_update(table, refs, n, n, size)
