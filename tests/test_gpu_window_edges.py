"""Windowed and 4-bit attention at the edges of what the header allows: bad pages beside values that are no numbers, scores
far past fp32's resolution of a power of two, tasks in a row with single buffers.

Tolerances are those of test_gpu_window where no other is derived."""

import numpy as np
import pytest
import torch

import window_oracle as wo
from test_gpu_window import BF, DEV, FP, HALF, call, check, make, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q4", [False, True], ids=["16bit", "q4"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [30, 9000])
def test_bad_pages_beside_nan_are_zeros(sv, q4, D, n):
    """A sequence with a bad page gets zeros whatever the pages beside it hold, whole (30 tokens are one tile) and cut: NaN
    for K and V of tokens in the bad page's tile, and far from it."""
    bs, R = 16, 3
    c = make(np.random.default_rng(n + D), (n, 300), R, 8, 2, D, bs, BF, 0, 0, q4)
    table = c["host"][4]
    for t in {n - 1, n - 2, n // 2, 20}:
        for name in "kv":
            if q4:
                c[name][table[0, t // bs], t % bs, 0, D: D + 8] = 0xff                   # s and m of both heads: NaN
            else:
                c[name][table[0, t // bs], t % bs] = float("nan")
    c["table"][0, 0] = -1
    out, err = call(sv, c)
    assert err == 1
    assert not out[0].isnan().any() and not out[0].any()
    c["host"] = (*c["host"][:5], [0, 300])
    check(c, out)


# The scores of a row are c 2^e with a whole number c for each token, exact in fp32 until the factor log2(e) / sqrt(D) meets
# them: equal ones have equal weights, and others are 2^20 apart at least, so that the definition's result is the mean of V
# over the visible tokens with the largest c.
def exact_scores(rng, D, dtype, q4, level, n, v_scale=1.0):
    bs, R, H, K = 64, 2, 4, 2
    c = make(rng, (n, 300), R, H, K, D, bs, dtype, 0, 0, q4)
    q, k, v, spread, table, ctx = c["host"]
    sign = np.where(rng.permutation(D) % 2 == 0, 1.0, -1.0)
    up = level // 2                                                                       # powers of two of q and of K
    q[...] = sign * 2.0 ** up
    q[:, :, 1::2] *= -1                                                                   # every other head: the least c
    count = rng.integers(1, 16, k.shape[:3])
    unit = 2.0 ** (level - up)
    c["q"] = torch.from_numpy(q).to(dtype).to(DEV)
    if q4:
        codes = np.broadcast_to(np.where(sign > 0, 15, 0), k.shape).astype(int)
        s = count * unit / 8
        rows = wo.pack(codes, s, -7.5 * s, dtype)                                         # +-7.5 s, m of 8 bits at most
        k = wo.unpack(rows, K, D, dtype)[0]
        assert np.array_equal(np.abs(k), np.broadcast_to(7.5 * s[..., None], k.shape))
        c["k"] = torch.from_numpy(rows)[:, :, None, :].contiguous().to(DEV)
        if v_scale != 1.0:
            rows = c["v"][:, :, 0].cpu().numpy()
            codes = np.stack([rows[..., : D] % 16, rows[..., : D] // 16], -1).reshape(*rows.shape[:2], K, D).astype(int)
            _, s, m = wo.unpack(rows, K, D, dtype)
            rows = wo.pack(codes, wo.round16(s * v_scale, dtype), wo.round16(m * v_scale, dtype), dtype)
            v, spread, _ = wo.unpack(rows, K, D, dtype)
            c["v"] = torch.from_numpy(rows)[:, :, None, :].contiguous().to(DEV)
    else:
        k = count[..., None] * unit * sign
        c["k"] = torch.from_numpy(k).to(dtype).to(DEV)
        assert np.array_equal(c["k"].double().cpu().numpy(), k)
    c["host"] = (q, k, v, spread, table, ctx)
    return c


@pytest.mark.parametrize("q4", [False, True], ids=["16bit", "q4"])
@pytest.mark.parametrize("D,dtype,level", [(64, FP, 16), (128, FP, 16), (128, BF, 16), (256, BF, 15)])
@pytest.mark.parametrize("n", [9000])
def test_equal_scores_in_pieces(sv, q4, D, dtype, level, n):
    """Scores of 2^24 in log2 units, many of them equal: their tokens share the weight equally, in whichever pieces they lie."""
    c = exact_scores(np.random.default_rng(level + n), D, dtype, q4, level, n)
    out, err = call(sv, c)
    assert err == 0
    check(c, out)


@pytest.mark.parametrize("q4", [False, True], ids=["16bit", "q4"])
@pytest.mark.parametrize("D,dtype,level", [(64, FP, 18), (128, FP, 22), (256, FP, 24), (128, BF, 18), (64, BF, 22), (128, BF, 25),
                                           (256, BF, 27), (128, BF, 60), (64, BF, 100)])
@pytest.mark.parametrize("n", [30, 9000])
def test_large_scores(sv, q4, D, dtype, level, n):
    """Scores of 2^22 to 2^110 in log2 units, whole and cut, many of them equal: a finite score, however large, is no NaN,
    and tokens of equal scores share the weight equally wherever they lie."""
    c = exact_scores(np.random.default_rng(level + n), D, dtype, q4, level, n)
    out, err = call(sv, c)
    assert err == 0
    check(c, out)


def test_large_scores_and_small_values(sv):
    """V of a 4-bit cache far below 1 under scores of 2^26 to 2^33: the reference, which is a sum of the score and log2 s,
    has no bits for the latter."""
    for level in (18, 20, 21, 22, 23, 25):
        c = exact_scores(np.random.default_rng(level), 128, BF, True, level, 700, 2.0 ** -10)
        out, err = call(sv, c)
        assert err == 0
        check(c, out)


def test_large_equal_values(sv):
    """Tokens of which all V elements are equal (s = 0), and large: 2^60 in a 4-bit cache."""
    for n in (30, 300, 9000):
        c = make(np.random.default_rng(n), (n, 40), 2, 8, 2, 128, 64, BF, 0, 0, True)
        q, k, v, spread, table, ctx = c["host"]
        rows = wo.pack(np.zeros(v.shape, int), np.zeros(v.shape[:3]), np.full(v.shape[:3], 2.0 ** 60), BF)
        c["v"] = torch.from_numpy(rows)[:, :, None, :].contiguous().to(DEV)
        c["host"] = (q, k, wo.unpack(rows, 2, 128, BF)[0], np.zeros(spread.shape), table, ctx)
        out, err = call(sv, c)
        assert err == 0
        check(c, out)


def test_q4_rows_whose_scores_are_all_minus_infinity(sv):
    """NaN, in one piece and in many, as over a 16-bit cache; the other kv head's rows are as ever."""
    for n in (30, 9000):
        c = make(np.random.default_rng(n), (n, 300), 2, 4, 2, 64, 64, BF, 0, 0, True)
        q, k, v, spread, table, ctx = c["host"]
        q[...] = np.abs(q) + 0.5
        c["q"] = torch.from_numpy(q).to(BF).to(DEV)
        pages = torch.as_tensor(table[0, : -(-n // 64)]).long().to(DEV)
        low = torch.tensor([0x80, 0xff], dtype=torch.uint8, device=DEV)                   # -inf
        c["k"][pages, :, 0, 64 + 4 + 2: 64 + 4 + 4] = low                                 # m of kv head 1
        out, err = call(sv, c)
        assert err == 0 and out[0, :, 2:].isnan().all()
        got = out.double().cpu().numpy()
        q = c["q"].double().cpu().numpy()
        c["host"] = (q, np.nan_to_num(k), np.nan_to_num(v), spread, table, ctx)
        for b, heads in ((0, slice(0, 2)), (1, slice(0, 4))):
            ref, tol = reference(c, b)
            assert np.all(np.abs(got[b] - ref)[:, heads] <= tol[:, heads])


# head dim 256 and 33 to 64 packed rows have one buffer of queries, accumulators and weights: several tasks a block, some cut
@pytest.mark.parametrize("q4", [False, True], ids=["16bit", "q4"])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("R,H,K,D", [(16, 8, 2, 256), (12, 6, 2, 256), (16, 16, 4, 128), (8, 8, 2, 64)])
def test_many_tasks_of_many_rows(sv, q4, dtype, R, H, K, D):
    rng = np.random.default_rng(R + H + D)
    ctx = [int(x) for x in rng.integers(R, 150, 330)]
    ctx[3], ctx[77], ctx[200] = 0, 0, 2500
    c = make(rng, ctx, R, H, K, D, 16, dtype, 0, 0, q4)
    out, err = call(sv, c)
    assert err == 0
    assert torch.isfinite(out.float()).all() and not out[3].any() and not out[77].any()
    pick = sorted({3, 200, 329, *range(0, 330, 11)})
    some = dict(c, host=(c["host"][0][pick], *c["host"][1:4], c["host"][4][pick], [ctx[b] for b in pick]))
    check(some, out[pick])
    again, _ = call(sv, c)
    assert torch.equal(out, again)
    # each alone gives what it gives among the others, but for the cuts: within both tolerances
    for b in (0, 200, 329):
        one = dict(c, q=c["q"][b: b + 1].contiguous(), table=c["table"][b: b + 1].contiguous(), ctx=c["ctx"][b: b + 1].contiguous(),
                   host=(c["host"][0][b: b + 1], *c["host"][1:4], c["host"][4][b: b + 1], [ctx[b]]))
        alone, err = call(sv, one)
        assert err == 0
        check(one, alone)


@pytest.mark.parametrize("q4", [False, True], ids=["16bit", "q4"])
def test_every_row_of_the_largest_batch(sv, q4):
    rng = np.random.default_rng(21)
    ctx = [int(x) for x in rng.integers(0, 20, 4096)]
    c = make(rng, ctx, 1, 2, 1, 256, 16, BF, 5, 1, q4)
    out, err = call(sv, c)
    assert err == 0
    check(c, out)


@pytest.mark.parametrize("dtype,D,R,H,K", [(BF, 128, 4, 32, 8), (BF, 128, 8, 16, 4), (BF, 256, 4, 24, 4), (BF, 256, 1, 8, 8),
                                           (FP, 64, 3, 8, 2), (FP, 128, 4, 32, 8), (FP, 128, 16, 16, 4), (FP, 256, 16, 8, 2)])
def test_weights_of_two_numbers(sv, dtype, D, R, H, K):
    """Where the weights are two 16-bit numbers they add 2^-16 of S at most, (2^-8)^2 in bf16, to the 2^-16 of fp32 scores,
    exponentials and sums (fp16: 2^-22, and a least step of 2^-37 next to weights of 2^7 or more); the rest is the rounding of
    the result."""
    c = make(np.random.default_rng(D + R), (R + 20, 700, 2100), R, H, K, D, 64, dtype, 600, 4, False)
    out, err = call(sv, c)
    assert err == 0
    q, k, v, _, table, ctx = c["host"]
    got = out.double().cpu().numpy()
    for b, n in enumerate(ctx):
        t = np.arange(n)
        page = np.where(wo.sees(n, R, 600, 4).any(0), table[b, t // 64], 0)
        ref, S, _, _ = wo.attention(q[b], k[page, t % 64], v[page, t % 64], 600, 4)
        tol = 2.0 ** -15 * S + HALF[dtype] * np.abs(ref) + torch.finfo(dtype).smallest_normal
        bad = np.abs(got[b] - ref) > tol
        assert not bad.any(), (b, int(bad.sum()), (np.abs(got[b] - ref) / S).max())
