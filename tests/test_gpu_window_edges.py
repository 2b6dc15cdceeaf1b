"""Windowed and 4-bit attention at the edges of what the header allows: bad pages beside values that are no numbers.

Tolerances are those of test_gpu_window where no other is derived."""

import numpy as np
import pytest

from test_gpu_window import BF, call, check, make

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
