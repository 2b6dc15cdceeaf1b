"""One workspace for every attention call on a stream: chain and tree calls of any shapes in any order."""

import numpy as np
import pytest
import torch

import test_gpu_tree as tg
from test_gpu_tree import DEV

pytestmark = pytest.mark.gpu


def chain_case(rng, ctx, k, H, K, D):
    par = np.tile(np.arange(-1, k), (len(ctx), 1))
    return dict(tg.attention_case(rng, ctx, k + 1, H, K, D, 64, torch.bfloat16, par=par), k_draft=k)


def tree_case(rng, ctx, N, H, K, D):
    return tg.attention_case(rng, ctx, N, H, K, D, 64, torch.bfloat16)


def bytes_for(sv, c):
    if "k_draft" in c:
        return sv.spec_verify_attention_workspace(c["q"], c["k"], c["table"], c["k_draft"])
    return sv.spec_tree_attention_workspace(c["q"], c["k"], c["table"])


def call(sv, c, ws):
    out = torch.full(c["q"].shape, float("nan"), device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = (c["q"], c["k"], c["v"], c["table"], c["ctx"])
    if "k_draft" in c:
        sv.spec_verify_attention(*args, c["k_draft"], out, workspace=ws, dev_err=err)
    else:
        sv.spec_tree_attention(*args, c["par"], out, workspace=ws, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return out


def cases():
    """Units cut over the SMs in each: few and many units a call, both kernels of the chain call (16 packed rows and
    32), one and two row tiles of the tree call."""
    rng = np.random.default_rng(61)
    return [
        chain_case(rng, rng.integers(100, 4000, 8), 3, 32, 8, 128),
        tree_case(rng, rng.integers(64, 3000, 6), 16, 32, 8, 128),
        chain_case(rng, rng.integers(4, 900, 150), 3, 32, 8, 128),
        tree_case(rng, (2500, 900, 64), 64, 16, 2, 128),
        chain_case(rng, (3000, 1700), 7, 32, 8, 128),
        tree_case(rng, (1500, 800), 20, 8, 2, 64),
        chain_case(rng, rng.integers(8, 700, 70), 7, 16, 4, 256),
    ]


def test_chain_and_tree_calls_share_a_workspace(sv):
    """Every order of two neighbours: each result is, bit for bit, that of a workspace of its own."""
    all_cases = cases()
    own = [call(sv, c, sv.new_attention_workspace(bytes_for(sv, c), DEV)) for c in all_cases]
    ws = sv.new_attention_workspace(max(bytes_for(sv, c) for c in all_cases), DEV)
    for i in range(len(all_cases)):
        for j in range(len(all_cases)):
            for at in (i, j):
                assert torch.equal(call(sv, all_cases[at], ws), own[at]), (i, j, at)
    for c, o in zip(all_cases, own):
        tg.check_attention(c, o)


def test_only_the_counters_need_zeros(sv):
    """A workspace that holds zeros in its first ATTN_COUNTER_BYTES bytes and NaN patterns behind them."""
    for c in cases():
        n = bytes_for(sv, c)
        want = call(sv, c, sv.new_attention_workspace(n, DEV))
        ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
        ws[: sv.ATTN_COUNTER_BYTES] = 0
        assert torch.equal(call(sv, c, ws), want)
        assert not bool(ws[: sv.ATTN_COUNTER_BYTES].any())  # zeros again, whatever the next call is


def test_small_call_then_large_call_of_the_chain(sv):
    """The counters of many units lie where a call of few units keeps nothing else."""
    rng = np.random.default_rng(62)
    small, large = chain_case(rng, (5000,), 3, 32, 8, 128), chain_case(rng, rng.integers(4, 700, 64), 3, 32, 8, 128)
    ws = sv.new_attention_workspace(max(bytes_for(sv, c) for c in (small, large)), DEV)
    call(sv, small, ws)
    tg.check_attention(large, call(sv, large, ws))


def test_a_new_workspace_zeroes_its_counters_alone(sv):
    """A call without a workspace pays for the counters, not for tens of megabytes: the rest is what the allocator's
    block held."""
    n = 48 << 20
    old = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    at = old.data_ptr()
    del old
    ws = sv.new_attention_workspace(n, DEV)
    assert ws.data_ptr() == at and not bool(ws[: sv.ATTN_COUNTER_BYTES].any())
    assert bool((ws[sv.ATTN_COUNTER_BYTES:] == 255).all())
    assert sv.new_attention_workspace(0, DEV).numel() == sv.ATTN_COUNTER_BYTES


def test_the_chain_calls_own_workspace_belongs_to_its_stream(sv):
    """A chain call on a given stream without a workspace waits for nothing on the current one, and is right when that
    is busy."""
    c = chain_case(np.random.default_rng(63), (3000, 700, 90), 3, 32, 8, 128)
    want = call(sv, c, None)
    out = torch.full_like(want, float("nan"))
    dirty = torch.full((96 << 20,), 255, dtype=torch.uint8, device=DEV)  # what a reused block would hold
    del dirty
    side, done = torch.cuda.Stream(), torch.cuda.Event()
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)
    done.record()
    sv.spec_verify_attention(c["q"], c["k"], c["v"], c["table"], c["ctx"], 3, out, stream=side)
    side.synchronize()
    assert not done.query()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_calls_without_a_workspace_in_a_graph(sv):
    """The clearing of the counters is captured with the call: replays on new inputs are right."""
    rng = np.random.default_rng(64)
    for make in (lambda: chain_case(rng, (3000, 700, 90), 3, 32, 8, 128), lambda: tree_case(rng, (2500, 900, 64), 16, 16, 2, 128)):
        c = make()
        call(sv, c, None)
        out = torch.full(c["q"].shape, float("nan"), device=DEV)
        args = (c["q"], c["k"], c["v"], c["table"], c["ctx"])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            if "k_draft" in c:
                sv.spec_verify_attention(*args, c["k_draft"], out)
            else:
                sv.spec_tree_attention(*args, c["par"], out)
        for _ in range(3):
            c["q"].copy_(torch.randn(c["q"].shape, device=DEV))
            out.fill_(float("nan"))
            g.replay()
            assert torch.equal(call(sv, c, None), out)
