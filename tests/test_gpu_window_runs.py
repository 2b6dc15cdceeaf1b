"""Windowed attention and the 4-bit cache as a program uses them: a run of the operators together, one workspace for all
attention calls, captured and replayed calls, two calls at once, caches of more than 2^32 bytes, many sequences.

Tolerances are those of test_gpu_window; what must not depend on anything is compared bit by bit."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import window_oracle as wo
from test_gpu_window import BF, DEV, FP, call, check, cuda, make

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def rounded(x, dtype):
    """What a 4-bit cache holds for x [..., K, D]: values, s."""
    codes, s, m = wo.quantise(x, dtype)
    return codes * s[..., None] + m[..., None], s


@pytest.mark.parametrize("dtype,D,window", [(BF, 128, 0), (FP, 64, 100), (BF, 256, 40)])
def test_serving_run(sv, dtype, D, window):
    """Prompts of two sequences stored at once, a step of verification, the accepted rows committed, a fork (its partial page
    copied), another step of all three, the whole cache loaded: each against the definitions."""
    rng = np.random.default_rng(D)
    K, H, bs, R, sinks, W, P = 2, 8, 32, 4, 3, 12, 40
    lens = [150, 61]
    table = np.full((3, W), -1)
    table[:2, : 6] = rng.permutation(P)[:12].reshape(2, 6)
    refs = np.zeros(P, int)
    refs[table[table >= 0]] = 1
    table, refs = cuda(table), cuda(refs)
    caches = [sv.new_q4_cache(P, bs, K, D, DEV, num_layers=1) for _ in "kv"]
    kc, vc = (c[0] for c in caches)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    have = [[None] * 3, [None] * 3]                 # K and V of every sequence, as they were given
    draw = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(dtype)  # noqa: E731

    def store(rows, ctx, seqs):
        x = [draw(len(seqs), rows, K, D) for _ in "kv"]
        sv.spec_cache_store_q4(x[0].to(DEV), x[1].to(DEV), table[seqs], cuda(ctx), kc, vc, dev_err=err)
        return [y.double().numpy() for y in x]

    def attend(ctx):
        q = draw(len(ctx), R, H, D)
        held = [[rounded(y, dtype) if y is not None else None for y in h] for h in have]
        P2, Wb = sum(-(-c // bs) for c in ctx) + 1, W
        flat, spread, at, tab = [np.zeros((P2, bs, K, D)) for _ in "kv"], np.zeros((P2, bs, K)), 0, np.zeros((len(ctx), Wb), int)
        for b, n in enumerate(ctx):
            for i in range(-(-n // bs)):
                tab[b, i] = at
                part = slice(i * bs, min(n, (i + 1) * bs))
                for w in range(2):
                    flat[w][at, : part.stop - part.start] = held[w][b][0][part]
                spread[at, : part.stop - part.start] = held[1][b][1][part]
                at += 1
        c = dict(q=q.to(DEV), k=kc, v=vc, table=table[: len(ctx)].contiguous(), ctx=cuda(ctx), K=K, window=window, sinks=sinks,
                 q4=True, bs=bs, host=(q.double().numpy(), flat[0], flat[1], spread, tab, list(ctx)))
        out, e = call(sv, c)
        assert e == 0
        check(c, out)

    x = store(150, lens, [0, 1])
    for w in range(2):
        have[w][0], have[w][1] = x[w][0], x[w][1, 150 - 61:]
    assert int(err.item()) == 0
    # a step: four rows each, of which two and one are kept (rows 0 and 2; row 0)
    x = store(R, [n + R for n in lens], [0, 1])
    step = [[np.concatenate([have[w][b], x[w][b]]) for b in range(2)] for w in range(2)]
    before = have
    have = [s + [None] for s in step]
    attend([n + R for n in lens])
    new = torch.zeros(2, dtype=torch.int32, device=DEV)
    sv.spec_cache_commit_path(*caches, table[:2].contiguous(), cuda([n + R for n in lens]),
                              cuda([[0, 2, 0, 0], [0, 0, 0, 0]]), cuda([1, 0]), new, dev_err=err)
    kept = new.cpu().tolist()
    assert kept == [152, 62]
    have = [[np.concatenate([before[w][0], x[w][0, [0, 2]]]), np.concatenate([before[w][1], x[w][1, [0]]]), None] for w in range(2)]
    # the third row continues the first; room for the next step
    lens = [kept[0] + R, kept[1] + R, kept[0] + R]
    sv.spec_cache_update(table, refs, cuda(kept + [0]), cuda(lens), bs, cuda([0, 1, 0]), *caches, dev_err=err)
    assert int(err.item()) == 0
    x = store(R, lens, [0, 1, 2])
    have = [[np.concatenate([have[w][b % 2], x[w][b]]) for b in range(3)] for w in range(2)]
    attend(lens)
    # all of it back
    n = max(lens)
    got = [torch.empty(3, n, K, D, dtype=dtype, device=DEV) for _ in "kv"]
    sv.spec_cache_load_q4(kc, vc, table, cuda(lens), *got, dev_err=err)
    assert int(err.item()) == 0
    for w in range(2):
        for b in range(3):
            want = torch.from_numpy(rounded(have[w][b], dtype)[0].astype(np.float32)).to(dtype)
            assert torch.equal(got[w][b, n - lens[b]:].cpu(), want) and not got[w][b, : n - lens[b]].any()


def test_rows_whose_scores_are_all_minus_infinity(sv):
    """NaN, in one piece and in many; the other kv head's rows are as ever."""
    for ctx in (40, 9000):
        c = make(np.random.default_rng(ctx), (ctx, 300), 2, 4, 2, 64, 64, BF, 0, 0, False)
        q, k, v, _, table, _ = c["host"]
        q[..., 3] = np.abs(q[..., 3]) + 0.5
        k[table[0, : -(-ctx // 64)], :, 1, 3] = -np.inf
        c["q"], c["k"] = torch.from_numpy(q).to(BF).to(DEV), torch.from_numpy(k).to(BF).to(DEV)
        out, err = call(sv, c)
        assert err == 0 and out[0, :, 2:].isnan().all()
        good = dict(c, q=c["q"][:, :, :2].contiguous(), k=c["k"][:, :, :1].contiguous(), v=c["v"][:, :, :1].contiguous(), K=1,
                    host=(q[:, :, :2], k[:, :, :1], v[:, :, :1], None, table, c["host"][5]))
        check(good, out[:, :, :2])


# q4 head counts that do not fit a block's eight warps: more than eight, and parts of eight at the end; one and two
@pytest.mark.parametrize("H,K,D,R,bs", [(10, 10, 128, 3, 16), (24, 12, 64, 1, 32), (34, 17, 128, 20, 64), (32, 32, 256, 1, 64),
                                        (8, 1, 64, 1, 16), (2, 1, 256, 5, 128), (20, 5, 128, 9, 32)])
def test_head_counts(sv, H, K, D, R, bs):
    rng = np.random.default_rng(H + K)
    for q4 in (False, True):
        c = make(rng, (R, 150 + R, 1200), R, H, K, D, bs, FP if K % 2 else BF, 400, 2, q4)
        out, err = call(sv, c)
        assert err == 0
        check(c, out)


@pytest.mark.parametrize("q4", [False, True], ids=["16bit", "q4"])
def test_many_ragged_sequences(sv, q4):
    """More units than blocks, empty and one-token sequences among them, one much longer than the rest: twice the same."""
    rng = np.random.default_rng(12)
    ctx = [int(x) for x in rng.integers(0, 90, 400)]
    ctx = [0 if n < 2 else n for n in ctx]
    ctx[7], ctx[391] = 9000, 777
    c = make(rng, ctx, 2, 8, 4, 64, 16, BF, 0, 0, q4)
    out, err = call(sv, c)
    assert err == 0
    check(c, out)
    again, _ = call(sv, c)
    assert torch.equal(out, again)


@pytest.mark.parametrize("q4", [False, True], ids=["16bit", "q4"])
def test_largest_batch(sv, q4):
    rng = np.random.default_rng(13)
    ctx = [int(x) for x in rng.integers(0, 20, 4096)]
    c = make(rng, ctx, 1, 2, 1, 256, 16, FP, 5, 1, q4)
    out, err = call(sv, c)
    assert err == 0
    pick = [0, 1, 2, 77, 2048, 4095] + [int(np.argmax(ctx)), int(np.argmin(ctx))]
    c["host"] = (c["host"][0][pick], *c["host"][1:4], c["host"][4][pick], [ctx[b] for b in pick])
    check(c, out[pick])


def calls_of_all_kinds(sv, rng):
    """Closures over attention calls of several kinds and shapes, each with its own output."""
    made = []
    for q4, D, R, ctx in ((True, 128, 4, (5000, 300)), (False, 64, 1, (4000, 0, 80)), (True, 64, 40, (900,)),
                          (False, 256, 4, (3000, 2500))):
        c = make(rng, ctx, R, 8, 2, D, 64, BF, 0, 0, q4)
        out = torch.empty_like(c["q"])
        made.append((lambda ws, s=None, c=c, out=out: (
            sv.spec_q4_attention(c["q"], c["k"], c["v"], c["table"], c["ctx"], c["K"], out, workspace=ws, stream=s) if c["q4"]
            else sv.spec_window_attention(c["q"], c["k"], c["v"], c["table"], c["ctx"], out, workspace=ws, stream=s)), out,
            sv.spec_window_attention_workspace(c["q"], c["K"], c["table"])))
    q = torch.randn(2, 5, 8, 128, device=DEV).to(BF)
    k = torch.randn(200, 64, 2, 128, device=DEV).to(BF)
    table, ctx = torch.randperm(200, device=DEV).int().view(2, 100), cuda([6000, 4000])
    out = torch.empty(2, 5, 8, 128, device=DEV)
    made.append((lambda ws, s=None: sv.spec_verify_attention(q, k, k, table, ctx, 4, out, workspace=ws, stream=s), out,
                 sv.spec_verify_attention_workspace(q, k, table, 4)))
    parents = cuda([[-1, 0, 0, 1, 2]] * 2)
    out2 = torch.empty(2, 5, 8, 128, device=DEV)
    made.append((lambda ws, s=None: sv.spec_tree_attention(q, k, k, table, ctx, parents, out2, workspace=ws, stream=s), out2,
                 sv.spec_tree_attention_workspace(q, k, table)))
    return made


def test_one_workspace_for_all_attention_calls(sv):
    """Calls of every kind and shape in turns over one workspace give what each gives over its own, bit by bit, eager and
    captured, two graphs over the same workspace replayed in turns."""
    torch.manual_seed(1)
    made = calls_of_all_kinds(sv, np.random.default_rng(14))
    want = []
    for f, out, size in made:
        f(sv.new_attention_workspace(size, DEV))
        torch.cuda.synchronize()
        want.append(out.clone())
    ws = sv.new_attention_workspace(max(size for _, _, size in made), DEV)

    def clear():
        for _, out, _ in made:
            out.fill_(float("nan"))

    for order in ([0, 1, 2, 3, 4, 5], [5, 3, 1, 4, 2, 0], [0, 0, 4, 1, 0, 5, 2, 3]):
        clear()
        for i in order:
            made[i][0](ws)
        torch.cuda.synchronize()
        for (_, out, _), w in zip(made, want):
            assert torch.equal(out, w)
    side = torch.cuda.Stream()
    graphs = []
    torch.cuda.synchronize()
    for part in ([0, 1, 4], [2, 3, 5, 0]):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            for i in part:
                made[i][0](ws, torch.cuda.current_stream())
        graphs.append(g)
    for _ in range(3):
        clear()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (_, out, _), w in zip(made, want):
            assert torch.equal(out, w)
    # without a workspace of the caller's
    for i in range(4):
        made[i][1].fill_(float("nan"))
        made[i][0](None)
    torch.cuda.synchronize()
    for i in range(4):
        assert torch.equal(made[i][1], want[i])


def test_two_calls_at_once(sv):
    """Streams with a workspace each, many calls in flight."""
    torch.manual_seed(2)
    made = calls_of_all_kinds(sv, np.random.default_rng(15))[:4]
    want = []
    for f, out, size in made:
        f(sv.new_attention_workspace(size, DEV))
        torch.cuda.synchronize()
        want.append(out.clone())
        out.fill_(float("nan"))
    streams = [torch.cuda.Stream() for _ in made]
    spaces = [sv.new_attention_workspace(size, DEV) for _, _, size in made]
    torch.cuda.synchronize()
    for _ in range(20):
        for (f, _, _), s, ws in zip(made, streams, spaces):
            f(ws, s)
    torch.cuda.synchronize()
    for (_, out, _), w in zip(made, want):
        assert torch.equal(out, w)


SCRIPT = """
import sys
sys.path.insert(0, sys.argv[1])
import torch
import speculative_decoding_verification_paged_gb300 as sv
torch.manual_seed(0)
dev = "cuda"
B, R, H, K, D, bs = 2, 4, 8, 2, 128, 64
table = torch.arange(2 * 60, device=dev).int().view(2, 60)
ctx = torch.tensor([3000, 900], device=dev).int()
x = [torch.randn(B, 3000, K, D, device=dev).to(torch.bfloat16) for _ in "kv"]
q = torch.randn(B, R, H, D, device=dev).to(torch.bfloat16)
kc, vc = (sv.new_q4_cache(120, bs, K, D, dev) for _ in "kv")
back = [torch.empty_like(y) for y in x]
wide = [torch.zeros(120, bs, K, D, device=dev, dtype=torch.bfloat16) for _ in "kv"]
for w, y in zip(wide, x):
    for b, n in ((0, 3000), (1, 900)):
        flat = w.view(2, -1, K, D)[b]
        flat[:n] = y[b, 3000 - n:]
outs = [torch.empty_like(q) for _ in range(2)]
size = sv.spec_window_attention_workspace(q, K, table)
ws = sv.new_attention_workspace(size, dev)
side = torch.cuda.Stream()
torch.cuda.synchronize()
def run():
    s = torch.cuda.current_stream()
    sv.spec_cache_store_q4(*x, table, ctx, kc, vc, stream=s)
    sv.spec_q4_attention(q, kc, vc, table, ctx, K, outs[0], window=500, sinks=4, workspace=ws, stream=s)
    sv.spec_cache_load_q4(kc, vc, table, ctx, *back, stream=s)
    sv.spec_window_attention(q, *wide, table, ctx, outs[1], window=500, sinks=4, workspace=ws, stream=s)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=side):   # the first calls of the process
    run()
for _ in range(2):
    for t in (*outs, *back):
        t.fill_(float("nan"))
    kc.zero_(), vc.zero_()
    g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (*outs, *back, kc, vc)]
kc.zero_(), vc.zero_()
run()
torch.cuda.synchronize()
for a, b in zip(got, (*outs, *back, kc, vc)):
    assert torch.equal(a, b)
assert torch.isfinite(outs[0]).all() and (outs[0].float() - outs[1].float()).abs().max() < 0.3
print("ok")
"""


def test_first_calls_captured(sv):
    """A process whose first calls are captured: store, attention over both kinds of cache, load."""
    r = subprocess.run([sys.executable, "-c", SCRIPT, ROOT], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-2000:]


def test_caches_past_32_bits(sv):
    """Pages at the end of caches of more than 2^32 bytes: a store, a load, and attention over both kinds."""
    rng = np.random.default_rng(16)
    for q4 in (True, False):
        c = make(rng, (700, 130), 3, 8, 8, 256, 128, BF, 0, 0, q4)
        size = c["k"][0].numel() * c["k"].element_size()
        pages = 2 ** 32 // size + 9
        small = c["k"].shape[0]
        big = []
        for name in "kv":
            x = torch.empty((pages, *c[name].shape[1:]), dtype=c[name].dtype, device=DEV)
            x[pages - small:] = c[name]
            big.append(x)
        table = c["table"].clone()
        seen = (table >= 0) & (table < small)
        table[seen] += pages - small
        table[~seen] = -1
        d = dict(c, k=big[0], v=big[1], table=table)
        out, err = call(sv, d)
        want, _ = call(sv, c)
        assert err == 0 and torch.equal(out, want)
        check(c, out)
        if q4:
            x = [torch.from_numpy(rng.standard_normal((2, 5, 8, 256))).to(BF) for _ in "kv"]
            sv.spec_cache_store_q4(x[0].to(DEV), x[1].to(DEV), table, c["ctx"], *big)
            got = [torch.empty_like(y, device=DEV) for y in x]
            sv.spec_cache_load_q4(*big, table, c["ctx"], *got)
            for g, y in zip(got, x):
                want = torch.from_numpy(rounded(y.double().numpy(), BF)[0].astype(np.float32)).to(BF)
                assert torch.equal(g.cpu(), want)
        del big, d
        torch.cuda.empty_cache()


def test_large_loads(sv):
    """As many tokens as the loads that take several a thread, an odd number of them, padded rows and a bad page among them."""
    rng = np.random.default_rng(17)
    K, D, bs, R, ctx = 8, 64, 64, 16411, [16411, 9000, 0, 16400]
    W = 260
    table = rng.permutation(4 * W).reshape(4, W)
    x = [torch.from_numpy(rng.standard_normal((4, R, K, D)).astype(np.float32)).to(FP).to(DEV) for _ in "kv"]
    cache = [sv.new_q4_cache(4 * W, bs, K, D, DEV) for _ in "kv"]
    sv.spec_cache_store_q4(*x, cuda(table), cuda(ctx), *cache)
    bad = table.copy()
    bad[1, 4] = -1
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = [torch.full_like(y, float("nan")) for y in x]
    sv.spec_cache_load_q4(*cache, cuda(bad), cuda(ctx), *got, dev_err=err)
    assert int(err.item()) == 1
    for g, y in zip(got, x):
        for b, n in enumerate(ctx):
            assert not g[b, : R - n].any()
        assert not g[1, R - 9000 + 256: R - 9000 + 320].any()
        for b, t in ((0, 0), (0, 16410), (1, 255), (1, 320), (1, 8999), (3, 16399), (3, 7000)):
            row = R - ctx[b] + t
            want = torch.from_numpy(rounded(y[b, row].double().cpu().numpy(), FP)[0].astype(np.float32)).to(FP)
            assert torch.equal(g[b, row].cpu(), want)
    # and the same token for token as loads of a few rows
    few = [torch.empty(4, 7, K, D, dtype=FP, device=DEV) for _ in "kv"]
    sv.spec_cache_load_q4(*cache, cuda(table), cuda(ctx), *few)
    for f, g in zip(few, got):
        assert torch.equal(f, g[:, R - 7:])


def test_wrong_tensors_are_named(sv):
    c = make(np.random.default_rng(18), (300, 40), 3, 8, 2, 128, 64, BF, 0, 0, True)
    d = make(np.random.default_rng(18), (300, 40), 3, 8, 2, 128, 64, BF, 0, 0, False)
    out = torch.empty_like(c["q"])
    q4 = lambda **kw: sv.spec_q4_attention(*[kw.get(n, c[n]) for n in ("q", "k", "v", "table", "ctx")], kw.get("K", 2),  # noqa: E731
                                           kw.get("out", out), workspace=kw.get("ws"))
    win = lambda **kw: sv.spec_window_attention(*[kw.get(n, d[n]) for n in ("q", "k", "v", "table", "ctx")],  # noqa: E731
                                                kw.get("out", out), workspace=kw.get("ws"))
    for f, own in ((q4, c), (win, d)):
        for bad in (dict(q=own["q"].cpu()), dict(q=own["q"].float()), dict(q=own["q"][0]), dict(out=out.float()), dict(out=out[:1]),
                    dict(v=own["v"][1:]), dict(k=own["k"].cpu()), dict(table=own["table"].long()), dict(table=own["table"][:1]),
                    dict(ctx=own["ctx"][:1]), dict(ctx=own["ctx"].cpu()), dict(out=out.transpose(1, 2)),
                    dict(ws=torch.zeros(4, device=DEV))):
            with pytest.raises((ValueError, TypeError)):
                f(**bad)
        with pytest.raises(RuntimeError):
            f(ws=torch.zeros(4096, dtype=torch.uint8, device=DEV))
    for bad in (dict(K=3), dict(k=c["k"][..., :-16], v=c["v"][..., :-16]), dict(K=0)):
        with pytest.raises((ValueError, RuntimeError)):
            q4(**bad)
    with pytest.raises(ValueError):
        win(k=d["k"].half(), v=d["v"].half())
    torch.cuda.synchronize()
