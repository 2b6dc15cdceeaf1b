"""Plain 64-bit definitions of the tree calls, one row at a time (test infrastructure).

Nothing here is shared with the library: attention, acceptance, the compaction
of the accepted path and the page-table update are written down from their
definitions in numpy and plain Python.
"""

import math

import numpy as np

ROOT, UNUSED = -1, -2


def line(parents, i):
    """Node i and its ancestors."""
    out = []
    while i >= 0:
        out.append(i)
        i = int(parents[i])
    return out


def is_tree(parents):
    for i, p in enumerate(parents):
        if p in (ROOT, UNUSED):
            continue
        if not 0 <= p < i or parents[p] == UNUSED:
            return False
    return True


def attention(q, k_cache, v_cache, table, ctx_lens, parents):
    """(out, weight): out [B, N, Hq, D] and sum_t p_t |v_t|, the scale of an error in p."""
    B, N, H, D = q.shape
    _, bs, K, _ = k_cache.shape
    G = H // K
    out = np.zeros((B, N, H, D))
    scale = np.zeros((B, N, H, D))
    for b in range(B):
        par, ctx = parents[b], int(ctx_lens[b])
        nb = k_cache.shape[0]
        if par[0] == UNUSED or not is_tree(par) or not N <= ctx <= table.shape[1] * bs:
            continue
        pages = table[b, : -(-ctx // bs)]
        if np.any((pages < 0) | (pages >= nb)):
            continue
        k = k_cache[pages].reshape(-1, K, D)[:ctx].astype(np.float64)
        v = v_cache[pages].reshape(-1, K, D)[:ctx].astype(np.float64)
        base = ctx - N
        for i in range(N):
            if par[i] == UNUSED:
                continue
            keys = list(range(base)) + sorted(base + j for j in line(par, i))
            for g in range(K):
                s = q[b, i, g * G:(g + 1) * G].astype(np.float64) @ k[keys, g].T / math.sqrt(D)
                s = np.exp(s - s.max(-1, keepdims=True))
                s /= s.sum(-1, keepdims=True)
                out[b, i, g * G:(g + 1) * G] = s @ v[keys, g]
                scale[b, i, g * G:(g + 1) * G] = s @ np.abs(v[keys, g])
    return out, scale


def philox(counter, seed):
    """Philox4x32-10 (Salmon et al., SC'11) on uint64 arrays of 32-bit words."""
    low = np.uint64(0xFFFFFFFF)
    x = [np.asarray(c, np.uint64) for c in counter]
    k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        a, c = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(c >> np.uint64(32)) ^ x[1] ^ np.uint64(k[0]), c & low, (a >> np.uint64(32)) ^ x[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return x


def uniform(word):
    return ((np.asarray(word) >> np.uint64(9)).astype(np.float64) + 0.5) * 2.0 ** -23


def race_uniforms(V, node, b, seed):
    g = np.arange(-(-V // 4), dtype=np.uint64)
    full = lambda c: np.full_like(g, c)  # noqa: E731
    words = philox([g, full(node), full(b), full(1)], seed)
    return uniform(np.stack(words, -1).reshape(-1)[:V])


def accept_row(logits, tokens, parents, probs, seed, b, mode, temperature):
    """(out_tokens, path, accept_len, margin): margin is the smallest relative distance of a decision from its
    border (a test u q < p, or the two largest keys of the race)."""
    N, V = logits.shape
    out, path = np.full(N, -1), np.full(N, -1)
    ok = parents[0] != UNUSED and is_tree(parents) and mode in (0, 1)
    ok = ok and all(0 <= tokens[i] < V for i in range(1, N) if parents[i] != UNUSED)
    if not ok or (mode == 1 and not 0 < temperature < math.inf):
        return out, path, -1, 1.0
    cur, m, margin = 0, 0, 1.0
    while True:
        l = logits[cur].astype(np.float64)
        children = [c for c in range(cur + 1, N) if parents[c] == cur]
        nxt = None
        if mode == 0:
            last = int(l.argmax())
            nxt = next((c for c in children if tokens[c] == last), None)
        else:
            p = np.exp((l - l.max()) / float(temperature))
            p /= p.sum()
            r, q = p, None if probs is None else probs[cur].astype(np.float64)
            for c in children:
                x = int(tokens[c])
                u = float(uniform(philox([0, c - 1, b, 0], seed)[0]))
                left, right = u * (1.0 if q is None else q[x]), r[x]
                margin = min(margin, abs(left - right) / max(left, right, 1e-300))
                if left < right:
                    nxt = c
                    break
                w = r.copy() if q is None else np.maximum(0.0, r - q)
                if q is None:
                    w[x] = 0.0
                if w.sum() > 0:
                    r = w / w.sum()
            if nxt is None:
                keys = r / -np.log(race_uniforms(V, cur, b, seed))
                last = int(keys.argmax())
                if V > 1:
                    top = np.partition(keys, V - 2)[V - 2:]
                    margin = min(margin, (top[1] - top[0]) / top[1])
        path[m] = cur
        if nxt is None:
            out[m] = last
            return out, path, m, margin
        out[m] = tokens[nxt]
        cur, m = nxt, m + 1


def accept(logits, tokens, parents, probs, seed, mode, temperature):
    rows = [accept_row(logits[b], tokens[b], parents[b], None if probs is None else probs[b], seed, b, int(mode[b]),
                       float(temperature[b])) for b in range(logits.shape[0])]
    return tuple(np.stack([np.asarray(r[i]) for r in rows]) for i in range(4))


def commit_path(k, v, table, ctx_lens, path, accept_len):
    """Caches [L, P, bs, ...] after the call, and the new lengths."""
    k, v = k.copy(), v.copy()
    k0, v0 = k.copy(), v.copy()
    B, N = path.shape
    bs, P = k.shape[2], k.shape[1]
    new = np.zeros(B, np.int64)
    for b in range(B):
        ctx, m = int(ctx_lens[b]), int(accept_len[b])
        base = ctx - N
        new[b] = max(0, base)
        if not 0 <= m < N or not N <= ctx <= table.shape[1] * bs:
            continue
        steps = [int(x) for x in path[b, : m + 1]]
        if steps[0] != 0 or any(y <= x for x, y in zip(steps, steps[1:])) or steps[-1] >= N:
            continue
        at = [(int(table[b, (base + t) // bs]), (base + t) % bs) for t in range(N)]
        if any(not 0 <= at[t][0] < P for j, s in enumerate(steps) for t in (j, s)):
            continue
        for j, s in enumerate(steps):
            k[:, at[j][0], at[j][1]] = k0[:, at[s][0], at[s][1]]
            v[:, at[j][0], at[j][1]] = v0[:, at[s][0], at[s][1]]
        new[b] = base + m + 1
    return k, v, new


def update(table, refs, cur, want, src, bs):
    """(table, refs, copies): copies lists (from page, to page, tokens)."""
    table, refs = np.array(table, np.int64), np.array(refs, np.int64)
    B, W = table.shape
    P = len(refs)
    src = list(range(B)) if src is None else [int(s) for s in src]
    room = W * bs
    bad = []
    for b, s in enumerate(src):
        wrong = not -1 <= s < B
        wrong = wrong or (s >= 0 and not (0 <= want[b] <= room and 0 <= cur[s] <= room))
        if not wrong and s >= 0:
            keep = min(int(cur[s]), int(want[b]))
            wrong = any(not 0 <= table[s, i] < P for i in range(-(-keep // bs)))
        bad.append(wrong)
    heir = {}
    for r in range(B):
        claims = [b for b in range(B) if not bad[b] and src[b] == r]
        heir[r] = r if bad[r] or src[r] == r else (claims[0] if claims else None)
    new = np.full((B, W), -1, np.int64)
    lack, held = [], set()
    for b, s in enumerate(src):
        if bad[b]:
            new[b] = table[b]
            continue
        if s < 0:
            continue
        keep = min(int(cur[s]), int(want[b]))
        for i in range(-(-int(want[b]) // bs)):
            e = int(table[s, i])
            tokens = min(max(keep - i * bs, 0), bs)
            if tokens == bs or (heir[s] == b and 0 <= e < P and refs[e] == 1):
                new[b, i] = e
            else:
                lack.append((b, i, e, tokens))
                if tokens:
                    held.add(e)
    refs_out = refs.copy()
    for old, sign in ((table, -1), (new, 1)):
        for e in old.reshape(-1):
            if 0 <= e < P:
                refs_out[e] += sign
    free = [g for g in range(P) if refs_out[g] == 0 and g not in held]
    copies = []
    for (b, i, e, tokens), g in zip(lack, free):
        new[b, i] = g
        refs_out[g] = 1
        if tokens:
            copies.append((e, g, tokens))
    return new, refs_out, copies
