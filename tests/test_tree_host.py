"""Tree calls without a GPU: what the host refuses before any CUDA call, and the plain definitions' own facts."""

import ctypes

import numpy as np
import pytest

import tree_oracle as to


@pytest.fixture(scope="module")
def lib():
    import speculative_decoding_verification_paged_gb300 as sv
    sv.build()
    return sv.load_library()


FAKE = ctypes.c_void_p(256)


def _desc(**kw):
    import speculative_decoding_verification_paged_gb300 as sv
    base = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=64, max_blocks_per_seq=4, num_blocks=8)
    base.update(kw)
    return sv._AttnDesc(**base)


def _cdesc(**kw):
    import speculative_decoding_verification_paged_gb300 as sv
    base = dict(batch=2, num_layers=2, block_size=16, max_blocks_per_seq=4, num_blocks=8, token_bytes=64)
    base.update(kw)
    return sv._CacheDesc(**base)


def test_tree_attention_refusals(lib):
    size = lambda n=16, **kw: lib.spec_tree_attention_workspace(ctypes.byref(_desc(**kw)), n)  # noqa: E731
    assert size() > 0
    assert size(n=0) == 0 and size(n=65) == 0 and size(num_q_heads=7) == 0 and size(head_dim=96) == 0
    assert lib.spec_tree_attention_workspace(None, 4) == 0

    def call(n=16, q=FAKE, par=FAKE, dtype=0, out_dtype=2, w=FAKE, wsb=None, **kw):
        d = _desc(**kw)
        wsb = lib.spec_tree_attention_workspace(ctypes.byref(_desc()), 16) if wsb is None else wsb
        return lib.spec_tree_attention(q, FAKE, FAKE, FAKE, FAKE, par, n, FAKE, dtype, out_dtype, ctypes.byref(d), w, wsb,
                                       None, None)

    assert call(q=None) == -1 and call(par=None) == -1
    assert call(n=0) == -1 and call(num_q_heads=7) == -1 and call(batch=-1) == -1
    assert call(dtype=2) == -1 and call(dtype=3) == -1 and call(dtype=0, out_dtype=1) == -1
    assert call(q=ctypes.c_void_p(264)) == -1              # not 16-byte aligned
    assert call(n=65) == -2 and call(head_dim=96) == -2 and call(block_size=48) == -2
    assert call(num_q_heads=258, num_kv_heads=2) == -2     # 129 query heads a kv head
    assert call(batch=4097) == -2
    assert call(w=None) == -4 and call(wsb=16) == -4
    assert call(batch=0, q=None) == 0


def test_tree_accept_refusals(lib):
    def call(B=2, N=4, V=100, logits=FAKE, path=FAKE):
        return lib.spec_tree_accept(logits, FAKE, FAKE, None, 1, FAKE, FAKE, FAKE, path, FAKE, B, N, V, None, None)

    assert call(N=0) == -1 and call(V=0) == -1 and call(B=-1) == -1
    assert call(logits=None) == -1 and call(path=None) == -1
    assert call(N=65) == -2 and call(V=(1 << 30) + 1) == -2
    assert call(B=0, logits=None) == 0


def test_commit_path_refusals(lib):
    def call(N=4, k=FAKE, new=ctypes.c_void_p(512), ctx=FAKE, **kw):
        return lib.spec_cache_commit_path(k, FAKE, FAKE, ctx, FAKE, FAKE, new, N, ctypes.byref(_cdesc(**kw)), None, None)

    assert call(k=None) == -1 and call(new=None) == -1 and call(N=0) == -1
    assert call(new=FAKE) == -1                            # new_lens is ctx_lens
    assert call(token_bytes=0) == -1 and call(block_size=0) == -1 and call(num_layers=-1) == -1
    assert call(N=65) == -2 and call(block_size=65537) == -2
    assert call(batch=0) == 0 and call(num_layers=0) == 0


def test_cache_update_refusals(lib):
    size = lambda **kw: lib.spec_cache_update_workspace(ctypes.byref(_cdesc(**kw)))  # noqa: E731
    assert size() > 0 and size(batch=64) > size()
    assert size(max_blocks_per_seq=0) == 0 and size(num_blocks=(1 << 30) + 1) == 0

    def call(table=FAKE, k=None, v=None, w=FAKE, wsb=1 << 20, **kw):
        return lib.spec_cache_update(table, FAKE, FAKE, FAKE, None, k, v, ctypes.byref(_cdesc(**kw)), w, wsb, None, None)

    assert call(table=None) == -1 and call(block_size=0) == -1
    assert call(k=FAKE) == -1 and call(v=FAKE) == -1       # one cache without the other
    assert call(k=FAKE, v=FAKE, token_bytes=0) == -1
    assert call(max_blocks_per_seq=1 << 30) == -2
    assert call(w=None) == -4 and call(wsb=64) == -4
    assert call(w=ctypes.c_void_p(264)) == -1
    assert call(batch=0, table=None) == 0


def test_a_chain_tree_accepts_what_the_chain_oracle_does(oracle_mod):
    rng = np.random.default_rng(5)
    B, k, V, seed = 40, 4, 53, 1234567890123
    N = k + 1
    logits = rng.standard_normal((B, N, V)).astype(np.float32) * 2
    drafts = rng.integers(0, V, (B, k)).astype(np.int32)
    raw = logits[:, :k] + rng.standard_normal((B, k, V)).astype(np.float32)
    probs = np.exp(raw - raw.max(-1, keepdims=True))
    probs = (probs / probs.sum(-1, keepdims=True)).astype(np.float32)
    drafts[::2] = np.take_along_axis(logits[::2, :k].argmax(-1)[..., None], np.zeros((1, 1, 1), int), -1)[..., 0]
    mode = (np.arange(B) % 3 > 0).astype(np.int32)
    temp = np.full(B, 0.9, np.float32)
    parents = np.tile(np.arange(-1, k), (B, 1))
    tokens = np.concatenate([np.zeros((B, 1), np.int32), drafts], 1)
    for q in (probs, None):
        rt, ra, margin, gap, rc = oracle_mod.accept(logits, drafts, q, seed, mode, temp)
        assert rc == 0
        full = None if q is None else np.concatenate([q, np.zeros((B, 1, V), np.float32)], 1)
        out, path, m, mg = to.accept(logits, tokens, parents, full, seed, mode, temp)
        near = (mg < 1e-9) | (margin < 1e-9)
        assert np.array_equal(out[~near], rt[~near]) and np.array_equal(m[~near], ra[~near])
        assert near.sum() == 0
        for b in range(B):
            assert path[b, : m[b] + 1].tolist() == list(range(m[b] + 1))


def test_tree_acceptance_keeps_the_target_distribution():
    """The first emitted token of a two-child tree is distributed as p, whatever q is: the frequencies over many
    seeds stay within five standard deviations of p (a fixed set of seeds)."""
    rng = np.random.default_rng(11)
    V, trials = 5, 4000
    logits = rng.standard_normal((3, V)).astype(np.float32)
    q = np.exp(rng.standard_normal(V))
    q = (q / q.sum()).astype(np.float32)
    p = np.exp(logits[0].astype(np.float64))
    p /= p.sum()
    probs = np.zeros((3, V), np.float32)
    probs[0] = q
    for deterministic in (False, True):
        count = np.zeros(V)
        for t in range(trials):
            tokens = np.array([0, 1, 3]) if deterministic else np.array([0, *rng.choice(V, 2, p=q / q.sum())])
            out = to.accept_row(logits, tokens, np.array([-1, 0, 0]), None if deterministic else probs, t, 0, 1, 1.0)[0]
            count[out[0]] += 1
        sigma = np.sqrt(trials * p * (1 - p))
        assert np.all(np.abs(count - trials * p) < 5 * sigma)


def test_plain_update_keeps_references_consistent():
    rng = np.random.default_rng(3)
    B, W, bs, P = 6, 5, 4, 40
    table, refs, _ = to.update(np.full((B, W), -1), np.zeros(P, int), np.zeros(B, int), rng.integers(1, W * bs, B), None, bs)
    cur = rng.integers(0, 5, B)
    for _ in range(20):
        src = rng.integers(-1, B, B)
        want = rng.integers(0, W * bs + 1, B)
        cur = np.array([np.count_nonzero(table[b] >= 0) * bs for b in range(B)])
        table, refs, _ = to.update(table, refs, cur, want, src, bs)
        assert np.array_equal(refs, np.bincount(table[table >= 0], minlength=P))
        for b in range(B):
            n = -(-int(want[b]) // bs) if src[b] >= 0 else 0
            assert np.all(table[b, :n] >= 0) and np.all(table[b, n:] == -1)


def test_one_tensor_for_both_caches_is_refused(lib):
    d = ctypes.byref(_cdesc())
    ws = lib.spec_cache_update_workspace(d)
    a, b, c, e, f = (ctypes.c_void_p(256 * i) for i in range(2, 7))
    assert lib.spec_cache_commit_path(FAKE, FAKE, a, b, c, e, f, 4, d, None, None) == -1
    assert lib.spec_cache_update(a, b, c, e, None, FAKE, FAKE, d, f, ws, None, None) == -1
