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
