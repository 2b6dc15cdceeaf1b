"""Plain 64-bit definitions of windowed attention and of the 4-bit cache (test infrastructure).

Nothing here is shared with the library: visibility, softmax, quantising and the
layout of a token's row are written down from their definitions in numpy.
"""

import math

import numpy as np
import torch


def sees(ctx, rows, window, sinks):
    """[rows, ctx]: which tokens each of the newest `rows` tokens sees."""
    t = np.arange(ctx)[None, :]
    p = (ctx - rows + np.arange(rows))[:, None]
    near = np.ones((rows, ctx), bool) if window == 0 else (t > p - window) | (t < sinks)
    return (t <= p) & near


def attention(q, k, v, window, sinks, spread=None):
    """One sequence: q [R, H, D], k and v [ctx, K, D]. (out, sum_t p_t |v_t|, and sum_t p_t spread_t, max_t p_t spread_t
    [R, H] for spread [ctx, K])."""
    R, H, D = q.shape
    ctx, K, _ = k.shape
    G = H // K
    see = sees(ctx, R, window, sinks)
    out, S = np.zeros((R, H, D)), np.zeros((R, H, D))
    Q, top = np.zeros((R, H)), np.zeros((R, H))
    for i in range(R):
        at = np.flatnonzero(see[i])
        for h in range(H):
            g = h // G
            s = k[at, g].astype(np.float64) @ q[i, h].astype(np.float64) / math.sqrt(D)
            e = np.exp(s - s.max())
            p = e / e.sum()
            out[i, h] = p @ v[at, g].astype(np.float64)
            S[i, h] = p @ np.abs(v[at, g].astype(np.float64))
            if spread is not None:
                Q[i, h] = p @ spread[at, g]
                top[i, h] = (p * spread[at, g]).max()
    return out, S, Q, top


def round16(x, dtype):
    """fp64 -> fp32 -> `dtype`, as fp64."""
    return torch.from_numpy(np.asarray(x, np.float32)).to(dtype).double().numpy()


def row_bytes(K, D):
    return -(-K * (D // 2 + 4) // 16) * 16


def quantise(x, dtype):
    """x [..., D] (values of `dtype`, fp64): (codes [..., D], s [...], m [...])."""
    x = np.asarray(x, np.float64)
    lo, hi = x.min(-1), x.max(-1)
    with np.errstate(over="ignore", invalid="ignore"):
        s = round16((hi - lo) / 15, dtype)
    codes = np.zeros(x.shape, np.int64)
    for at in np.ndindex(*x.shape[:-1]):
        if not np.isfinite(x[at]).all():
            s[at] = lo[at] = np.nan
            continue
        if s[at] == 0:
            continue
        t = x[at] - lo[at]
        f = np.floor(t / s[at])
        over = 2 * t - (2 * f + 1) * s[at]
        codes[at] = np.minimum(f + ((over > 0) | ((over == 0) & (f % 2 == 1))), 15)
    return codes, s, lo


def pack(codes, s, m, dtype):
    """Token rows [..., row bytes] of codes [..., K, D] and s, m [..., K]; padding zero."""
    *lead, K, D = codes.shape
    rows = np.zeros((*lead, row_bytes(K, D)), np.uint8)
    flat = codes.reshape(*lead, K * D)
    rows[..., : K * D // 2] = flat[..., 0::2] + 16 * flat[..., 1::2]
    par = torch.from_numpy(np.stack([s, m], -1).reshape(*lead, 2 * K).astype(np.float32)).to(dtype).contiguous()
    rows[..., K * D // 2: K * D // 2 + 4 * K] = par.view(torch.uint8).numpy()
    return rows


def unpack(rows, K, D, dtype):
    """(values [..., K, D], s, m) of token rows."""
    lead = rows.shape[:-1]
    body = rows[..., : K * D // 2].astype(np.int64)
    codes = np.stack([body % 16, body // 16], -1).reshape(*lead, K, D)
    par = torch.from_numpy(np.ascontiguousarray(rows[..., K * D // 2: K * D // 2 + 4 * K])).view(dtype).double().numpy()
    par = par.reshape(*lead, K, 2)
    with np.errstate(invalid="ignore"):
        return codes * par[..., :1] + par[..., 1:], par[..., 0], par[..., 1]


def pages_seen(ctx, rows, window, sinks, bs):
    """Indices of the pages that some row sees."""
    if ctx == 0:
        return np.zeros(0, int)
    return np.unique(np.flatnonzero(sees(ctx, rows, window, sinks).any(0)) // bs)
