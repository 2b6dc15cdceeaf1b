"""Windowed attention and the 4-bit cache without a GPU: what the host refuses before any CUDA call, and the plain
definitions' own facts."""

import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import window_oracle as wo
from test_tree_host import FAKE, _desc, lib  # noqa: F401  (lib is a fixture)

OTHER = ctypes.c_void_p(4096)


def test_attention_refusals(lib):  # noqa: F811
    size = lambda n=4, **kw: lib.spec_window_attention_workspace(ctypes.byref(_desc(**kw)), n)  # noqa: E731
    assert size() >= 4096
    assert size(n=0) == 0 and size(n=65) == 0 and size(num_q_heads=7) == 0 and size(head_dim=96) == 0
    assert lib.spec_window_attention_workspace(None, 4) == 0

    for fn in (lib.spec_window_attention, lib.spec_q4_attention):
        def call(n=4, q=FAKE, k=FAKE, table=FAKE, out=FAKE, dtype=0, w=FAKE, wsb=None, window=10, sinks=2, **kw):
            wsb = size() if wsb is None else wsb
            return fn(q, k, FAKE, table, FAKE, n, window, sinks, out, dtype, ctypes.byref(_desc(**kw)), w, wsb, None, None)

        assert call(q=None) == -1 and call(k=None) == -1 and call(table=None) == -1 and call(out=None) == -1
        assert call(n=0) == -1 and call(num_q_heads=7) == -1 and call(batch=-1) == -1 and call(num_kv_heads=0) == -1
        assert call(window=-1) == -1 and call(sinks=-1) == -1
        assert call(dtype=2) == -1 and call(dtype=3) == -1
        assert call(q=ctypes.c_void_p(264)) == -1 and call(out=ctypes.c_void_p(264)) == -1   # not 16-byte aligned
        assert call(n=65) == -2 and call(head_dim=96) == -2 and call(block_size=48) == -2
        assert call(num_q_heads=130, num_kv_heads=2) == -2                                    # 65 query heads a kv head
        assert call(batch=4097) == -2
        assert call(num_blocks=1 << 25, block_size=64) == -2                                  # 2^31 token rows
        assert call(max_blocks_per_seq=(1 << 24) + 1) == -2                                   # more than 2^30 tokens
        assert call(max_blocks_per_seq=1 << 24, num_q_heads=512, num_kv_heads=256) == -2      # 2^32 key tiles
        assert call(w=None) == -4 and call(wsb=16) == -4 and call(w=ctypes.c_void_p(264)) == -1
        assert call(batch=0, q=None) == 0


def test_cache_refusals(lib):  # noqa: F811
    assert lib.spec_q4_row_bytes(8, 128) == 544 and lib.spec_q4_row_bytes(1, 128) == 80 and lib.spec_q4_row_bytes(3, 64) == 112
    assert lib.spec_q4_row_bytes(4, 256) == 528
    for heads, dim in ((0, 128), (65537, 128), (8, 96), (8, 0), (-1, 64)):
        assert lib.spec_q4_row_bytes(heads, dim) == 0

    def store(n=4, k=FAKE, v=FAKE, ks=256, vs=256, kc=FAKE, vc=OTHER, dtype=0, ctx=FAKE, **kw):
        return lib.spec_cache_store_q4(k, v, ks, vs, FAKE, ctx, n, kc, vc, dtype, ctypes.byref(_desc(**kw)), None, None)

    def load(n=4, kc=FAKE, ko=FAKE, vo=OTHER, dtype=0, out=0, ctx=FAKE, **kw):
        return lib.spec_cache_load_q4(kc, FAKE, FAKE, ctx, n, ko, vo, dtype, out, ctypes.byref(_desc(**kw)), None, None)

    assert store(k=None) == -1 and store(vc=FAKE) == -1 and store(ks=248) == -1 and store(vs=260) == -1
    assert store(k=ctypes.c_void_p(264)) == -1 and store(vc=ctypes.c_void_p(4104)) == -1
    assert load(kc=None) == -1 and load(vo=FAKE) == -1 and load(out=1) == -1 and load(dtype=2) == -1
    for call in (store, load):
        assert call(n=0) == -1 and call(ctx=None) == -1 and call(dtype=2) == -1 and call(batch=-1) == -1
        assert call(head_dim=96) == -2 and call(block_size=8) == -2
        assert call(n=1 << 26) == -2                             # 2 * 2^26 * 2 * 128 / 8 chunks
        assert call(num_blocks=1 << 25) == -2 and call(max_blocks_per_seq=(1 << 24) + 1) == -2
        assert call(batch=0) == 0
    assert load(out=2, batch=0) == 0


def test_codes_are_the_exact_rounding():
    """quantise against rational arithmetic: random values, ties, tiny values beside large ones."""
    rng = np.random.default_rng(3)
    rows = [rng.standard_normal(64) for _ in range(20)]
    rows += [rng.integers(-15, 16, 64) / 2.0 for _ in range(20)]                  # many ties
    rows += [np.concatenate([[-7.5, 7.5], rng.standard_normal(62) * 1e-9]) for _ in range(4)]
    rows += [np.full(64, 3.25), np.zeros(64)]
    for dtype in (torch.bfloat16, torch.float16):
        for x in rows:
            x = torch.from_numpy(x).to(dtype).double().numpy()
            codes, s, m = wo.quantise(x, dtype)
            assert m == x.min()
            if s == 0:
                assert not codes.any()
                continue
            for c, y in zip(codes, x):
                want = round((Fraction(float(y)) - Fraction(float(m))) / Fraction(float(s)))  # half to even
                assert c == min(want, 15)


def test_rows_unpack_to_what_was_packed():
    rng = np.random.default_rng(4)
    for K, D in ((1, 64), (3, 128), (2, 256)):
        for dtype in (torch.bfloat16, torch.float16):
            x = torch.from_numpy(rng.standard_normal((5, K, D))).to(dtype).double().numpy()
            codes, s, m = wo.quantise(x, dtype)
            rows = wo.pack(codes, s, m, dtype)
            assert rows.shape == (5, wo.row_bytes(K, D))
            got, s2, m2 = wo.unpack(rows, K, D, dtype)
            assert np.array_equal(s, s2) and np.array_equal(m, m2) and np.array_equal(got, codes * s[..., None] + m[..., None])
            # half a step, and at the upper end what s was rounded down by
            tol = s[..., None] / 2 + 15 * s[..., None] * (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11)
            assert np.all(np.abs(got - x) <= tol)


def test_which_tokens_a_row_sees():
    see = wo.sees(10, 3, 4, 2)
    assert [np.flatnonzero(r).tolist() for r in see] == [[0, 1, 4, 5, 6, 7], [0, 1, 5, 6, 7, 8], [0, 1, 6, 7, 8, 9]]
    assert wo.sees(5, 5, 0, 0).tolist() == np.tril(np.ones((5, 5), bool)).tolist()
    assert wo.pages_seen(300, 2, 20, 3, 16).tolist() == [0, 17, 18]


def test_wrong_arguments_are_named():
    import speculative_decoding_verification_paged_gb300 as sv
    with pytest.raises(ValueError, match="no 4-bit cache"):
        sv.q4_row_bytes(8, 96)
    with pytest.raises(ValueError, match="32 bits"):
        sv.q4_row_bytes(1 << 32, 128)
    cache = sv.new_q4_cache(3, 16, 2, 64, "cpu", num_layers=2)
    assert cache.shape == (2, 3, 16, 1, 80) and cache.dtype == torch.uint8 and not bool(cache.any())
    x = torch.zeros(2, 3, 4, 64)
    assert sv._token_stride(x, "k") == 256
    wide = torch.zeros(2, 3, 12 * 64)[:, :, 256:512].unflatten(-1, (4, 64))
    assert sv._token_stride(wide, "k") == 768
    with pytest.raises(ValueError, match="k must have dense heads"):
        sv._token_stride(x.transpose(1, 2), "k")
    with pytest.raises(ValueError, match="evenly spaced"):
        sv._token_stride(torch.zeros(2, 5, 4, 64)[:, :3], "k")
