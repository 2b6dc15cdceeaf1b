"""The tree calls on the GPU against their 64-bit definitions (tree_oracle).

Attention tolerances, per element, with S = sum_t p_t |v_t| (the scale on which an
error of p acts) and `half` the largest relative error of a rounding:
  * 16-bit output: one rounding of the weights to the input type (half * S) and one
    of the result (half * |ref|), half = 2^-8 for bf16 and 2^-11 for fp16, plus the
    fp32 part below;
  * fp32 output: the weights are held to 2^-17 at least (two bf16 parts; three, or
    fp16 parts, are finer); exponentials, fp32 scores and sums are given as much
    again: 2^-16 * S.
Decisions of the acceptance must match exactly except within 1e-5 of their border.
"""

import numpy as np
import pytest
import torch

import tree_oracle as to

pytestmark = pytest.mark.gpu

DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def cuda(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x)).to(DEV, dtype)


def random_trees(rng, B, N, unused=True, kind="random"):
    par = np.zeros((B, N), np.int64)
    for b in range(B):
        used = int(rng.integers(1, N + 1)) if unused else N
        for i in range(1, N):
            if i >= used:
                par[b, i] = to.UNUSED
            elif kind == "chain":
                par[b, i] = i - 1
            elif kind == "star":
                par[b, i] = 0
            else:
                par[b, i] = rng.integers(0, i)
        par[b, 0] = to.ROOT
    return par


def attention_case(rng, ctx, N, H, K, D, bs, dtype, par=None, unused=True, spare=2):
    """Inputs of one call; slots past the context and of unused nodes hold NaN."""
    B, ctx = len(ctx), np.asarray(ctx)
    W = max(1, -(-int(ctx.max()) // bs))
    want = -(-np.maximum(ctx, 0) // bs)
    P = int(want.sum()) + spare
    order = rng.permutation(P)
    table = np.full((B, W), -1, np.int64)
    at = 0
    for b in range(B):
        table[b, : want[b]] = order[at: at + want[b]]
        at += want[b]
    par = random_trees(rng, B, N, unused) if par is None else par
    q, k, v = (torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dtype)
               for s in ((B, N, H, D), (P, bs, K, D), (P, bs, K, D)))
    clean = [t.float().numpy() for t in (q, k, v)]
    for b in range(B):
        dead = [ctx[b] - N + j for j in range(N) if par[b, j] == to.UNUSED] + list(range(ctx[b], want[b] * bs))
        for t in dead:
            if t >= 0:
                k[table[b, t // bs], t % bs] = float("nan")
                v[table[b, t // bs], t % bs] = float("nan")
    return dict(q=q.to(DEV), k=k.to(DEV), v=v.to(DEV), table=cuda(table), ctx=cuda(ctx), par=cuda(par), clean=clean,
                host=(table, ctx, par))


def run_attention(sv, c, out_dtype, **kw):
    out = torch.full(c["q"].shape, float("nan"), dtype=out_dtype, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    sv.spec_tree_attention(c["q"], c["k"], c["v"], c["table"], c["ctx"], c["par"], out, dev_err=err, **kw)
    torch.cuda.synchronize()
    return out, int(err.item())


def check_attention(c, out):
    table, ctx, par = c["host"]
    q, k, v = c["clean"]
    ref, S = to.attention(q, k, v, table, ctx, par)
    got = out.double().cpu().numpy()
    tol = 2.0 ** -16 * S
    if out.dtype != torch.float32:
        tol = tol + HALF[out.dtype] * (S + np.abs(ref)) * (1 + 2.0 ** -6)
        tol = tol + torch.finfo(out.dtype).smallest_normal  # results below the normal range keep fewer bits
    assert np.isfinite(got).all()
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got - ref)[bad][:5], tol[bad][:5])
    return ref


# (contexts, nodes, query heads, kv heads, head dim, page): one token to many tiles, contexts just below, at and above
# tile and page edges, odd head ratios, one node to 64, packed rows from 1 to 512.
ATTENTION = [
    ((1, 2, 17, 128, 129), 1, 4, 4, 64, 16),
    ((7, 64, 65, 300), 7, 9, 3, 64, 16),
    ((64, 127, 191, 700), 64, 8, 1, 64, 32),
    ((16, 128, 144, 1000, 257), 16, 32, 8, 128, 64),
    ((33, 161, 640), 33, 8, 2, 128, 128),
    ((64, 65, 200, 1500), 64, 8, 2, 128, 16),
    ((64, 512, 777), 64, 16, 2, 128, 64),
    ((50, 300), 50, 7, 1, 128, 32),
    ((20, 140, 260), 20, 71, 1, 128, 64),
    ((3, 100), 3, 128, 1, 64, 128),
    ((16, 80, 129, 900), 16, 24, 4, 256, 64),
    ((64, 300, 513), 64, 8, 2, 256, 16),
    ((5, 6, 1100), 5, 2, 2, 256, 128),
]


@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("case", ATTENTION, ids=[f"n{c[1]}_h{c[2]}_{c[3]}_d{c[4]}_p{c[5]}" for c in ATTENTION])
def test_attention(sv, case, dtype, out):
    ctx, N, H, K, D, bs = case
    c = attention_case(np.random.default_rng(N * 1000 + D), ctx, N, H, K, D, bs, dtype)
    got, err = run_attention(sv, c, dtype if out == "same" else torch.float32)
    assert err == 0
    check_attention(c, got)


@pytest.mark.parametrize("D,N,H,K", [(128, 16, 32, 8), (128, 48, 16, 2), (64, 24, 12, 2), (256, 12, 8, 1)])
def test_attention_many_sequences(sv, D, N, H, K):
    """Ragged batches whose units are cut over the SMs and merged, and equal lengths."""
    rng = np.random.default_rng(D + N)
    for ctx in (rng.integers(N, 3000, 12), np.full(40, 1024)):
        c = attention_case(rng, ctx, N, H, K, D, 64, torch.bfloat16)
        for dt in (torch.bfloat16, torch.float32):
            got, err = run_attention(sv, c, dt)
            assert err == 0
            check_attention(c, got)


@pytest.mark.parametrize("kind", ["chain", "star"])
def test_attention_extreme_trees(sv, kind):
    rng = np.random.default_rng(1)
    c = attention_case(rng, (64, 190, 450), 64, 8, 2, 128, 64, torch.bfloat16,
                       par=random_trees(rng, 3, 64, unused=False, kind=kind))
    got, err = run_attention(sv, c, torch.float32)
    assert err == 0
    check_attention(c, got)


def test_attention_of_a_chain_is_the_chain_call(sv):
    rng = np.random.default_rng(2)
    k = 3
    c = attention_case(rng, (4, 300, 1111), k + 1, 16, 4, 128, 64, torch.bfloat16,
                       par=np.tile(np.arange(-1, k), (3, 1)))
    got, err = run_attention(sv, c, torch.float32)
    out = torch.empty_like(got)
    sv.spec_verify_attention(c["q"], c["k"], c["v"], c["table"], c["ctx"], k, out)
    # each call is within 2^-16 S of the definition, S <= max |v| < 8
    assert err == 0 and (got - out).abs().max().item() <= 2 * 2.0 ** -16 * 8


def test_attention_forest_large_scores_and_rows(sv):
    """Several nodes without a parent, scores far apart (one key dominates; the running maximum keeps growing), and
    64-bit offsets into the cache are exercised by a page table that names the last pages of a large cache."""
    rng = np.random.default_rng(3)
    N, D = 12, 128
    par = np.array([[-1, -1, 0, 1, -2, 2, -1, 6, 6, -2, 8, 3]])
    c = attention_case(rng, (900,), N, 8, 2, D, 16, torch.bfloat16, par=par)
    table = c["host"][0]
    for name, i in (("k", 1),):
        t = c[name]
        for tok in range(0, 880, 37):  # ever larger keys along the sequence
            t[table[0, tok // 16], tok % 16] *= 1 + tok / 64
        c["clean"][i] = torch.nan_to_num(t).float().cpu().numpy()
    got, err = run_attention(sv, c, torch.float32)
    assert err == 0
    ref, S = to.attention(*c["clean"], *c["host"])
    # scores reach ~2^8: an fp32 score of that size is off by 2^-15 at most, and p by as much
    assert np.all(np.abs(got.double().cpu().numpy() - ref) <= (2.0 ** -16 + 2.0 ** -13) * S)


def test_attention_long_offsets(sv):
    """Pages past 2^31 elements of the cache."""
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    rng = np.random.default_rng(4)
    N, H, K, D, bs = 8, 8, 8, 128, 64
    P = (1 << 31) // (bs * K * D) + 40
    c = attention_case(rng, (200, 450), N, H, K, D, bs, torch.bfloat16)
    table, ctx, par = c["host"]
    far = table + np.where(table >= 0, P - c["k"].shape[0], 0)
    for n in ("k", "v"):
        big = torch.zeros((P, bs, K, D), dtype=torch.bfloat16, device=DEV)
        big[P - c[n].shape[0]:] = c[n]
        c[n] = big
    c["table"] = cuda(far)
    got, err = run_attention(sv, c, torch.float32)
    assert err == 0
    check_attention(c, got)


def test_attention_reports_and_skips_bad_rows(sv):
    rng = np.random.default_rng(5)
    N = 8
    par = random_trees(rng, 7, N, unused=False)
    par[1, 3] = 5                      # a later node as parent
    par[2, 4], par[2, 6] = -2, 4       # child of an unused node
    par[3, 0] = -2                     # an empty row: nothing of it is looked at
    c = attention_case(rng, (300,) * 7, N, 8, 2, 128, 16, torch.bfloat16, par=par, unused=False)
    table = c["host"][0].copy()
    ctx = c["host"][1].copy()
    table[3] = 1 << 20
    ctx[3] = -5
    ctx[4] = N - 1
    ctx[5] = table.shape[1] * 16 + 1
    table[6, 7] = c["k"].shape[0]
    c["table"], c["ctx"], c["host"] = cuda(table), cuda(ctx), (table, ctx, par)
    for dt in (torch.float32, torch.bfloat16):
        got, err = run_attention(sv, c, dt)
        assert err == sv.DEVERR["tree"] | sv.DEVERR["ctx_len"] | sv.DEVERR["block_id"]
        ref = check_attention(c, got)
        assert np.abs(ref[0]).max() > 0 and not ref[1:].any() and not got[1:].any()


@pytest.mark.parametrize("D,out_dtype", [(64, torch.float32), (128, torch.bfloat16), (256, torch.float32)])
@pytest.mark.parametrize("live", [1, 2, 5])
@pytest.mark.parametrize("B", [5, 256, 257, 700])
def test_attention_few_long_rows_of_a_padded_batch(sv, B, live, D, out_dtype):
    """A few sequences of unlike lengths, cut over many CTAs, among rows that are empty: at the batch's ends and within."""
    rng = np.random.default_rng(B + live)
    ctx = np.full(B, 8)
    par = np.full((B, 8), to.UNUSED)
    at = np.unique(np.linspace(0, B - 1, live).astype(int))
    ctx[at] = [2000, 1111, 129, 900, 8][: len(at)]
    par[at] = random_trees(rng, len(at), 8)
    c = attention_case(rng, ctx, 8, 4, 2, D, 64, torch.bfloat16, par=par)
    out, err = run_attention(sv, c, out_dtype)
    assert err == 0
    check_attention(c, out)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_attention_output_on_a_16_byte_boundary(sv, D, out_dtype):
    """An output that is 16- but not 32-byte aligned gives the same bits, and nothing around it is written."""
    c = attention_case(np.random.default_rng(31), (40, 300), 13, 8, 2, D, 64, torch.bfloat16)
    whole, err = run_attention(sv, c, out_dtype)
    pad = 16 // whole.element_size()
    flat = torch.full((whole.numel() + 2 * pad,), 7.0, dtype=out_dtype, device=DEV)
    out = flat[pad:-pad].view(whole.shape)
    assert err == 0 and out.data_ptr() % 32 == 16
    sv.spec_tree_attention(c["q"], c["k"], c["v"], c["table"], c["ctx"], c["par"], out)
    torch.cuda.synchronize()
    check_attention(c, out)
    assert torch.equal(out, whole) and bool((flat[:pad] == 7).all()) and bool((flat[-pad:] == 7).all())


def test_empty_batches(sv):
    i = lambda *s: torch.empty(s, dtype=torch.int32, device=DEV)  # noqa: E731
    q, kv = torch.empty((0, 4, 2, 64), dtype=torch.bfloat16, device=DEV), torch.zeros((3, 16, 1, 64), dtype=torch.bfloat16, device=DEV)
    out = torch.empty((0, 4, 2, 64), device=DEV)
    sv.spec_tree_attention(q, kv, kv.clone(), i(0, 2), i(0), i(0, 4), out)
    f = torch.empty((0, 4, 50), device=DEV)
    sv.spec_tree_accept(f, i(0, 4), i(0, 4), None, 1, i(0), torch.empty(0, device=DEV), i(0, 4), i(0, 4), i(0))
    torch.cuda.synchronize()


def test_own_workspaces_belong_to_the_calls_stream(sv):
    """A call on a given stream without a workspace waits for nothing on the current one, and is right when that is busy."""
    c = attention_case(np.random.default_rng(51), (700, 1500, 90), 16, 8, 2, 128, 64, torch.bfloat16)
    want, _ = run_attention(sv, c, torch.bfloat16)
    out = torch.full_like(want, float("nan"))
    table, refs, cur = cuda([[0, -1, -1], [1, -1, -1]]), cuda([1, 1, 0, 0, 0]), cuda([3, 4])
    new = cuda([9, 5])
    side, done = torch.cuda.Stream(), torch.cuda.Event()
    # A kernel's first launch in a process waits for the device (it is loaded then: 193 ms here, 0.1 ms afterwards).
    sv.spec_cache_update(table.clone(), refs.clone(), cur, new, 4)
    dirty = torch.full((96 << 20,), 255, dtype=torch.uint8, device=DEV)  # what a reused block would hold
    del dirty
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)
    done.record()
    sv.spec_tree_attention(c["q"], c["k"], c["v"], c["table"], c["ctx"], c["par"], out, stream=side)
    sv.spec_cache_update(table, refs, cur, new, 4, stream=side)
    side.synchronize()
    assert not done.query()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert table.tolist() == [[0, 2, 3], [1, 4, -1]] and refs.tolist() == [1] * 5


def test_attention_reuses_its_workspace(sv):
    """One workspace, alternating shapes and inputs, bit-equal repeats; a bad row leaves it usable."""
    rng = np.random.default_rng(6)
    a = attention_case(rng, (2000, 77, 800), 40, 16, 2, 128, 64, torch.bfloat16)
    b = attention_case(rng, (900, 900), 9, 6, 2, 256, 32, torch.bfloat16)
    need = max(sv.spec_tree_attention_workspace(x["q"], x["k"], x["table"]) for x in (a, b))
    ws = sv.new_attention_workspace(need, DEV)
    first = [run_attention(sv, x, torch.float32, workspace=ws)[0] for x in (a, b)]
    broken = dict(a, table=torch.full_like(a["table"], -1))
    assert run_attention(sv, broken, torch.float32, workspace=ws)[1] == sv.DEVERR["block_id"]
    for _ in range(3):
        for x, y in zip((a, b), first):
            assert torch.equal(run_attention(sv, x, torch.float32, workspace=ws)[0], y)
    check_attention(a, first[0])


@pytest.mark.parametrize("case", [(12, 3000, 16, 32, 8, 128, "same"), (30, 1024, 16, 32, 8, 128, "same"),
                                  (8, 2048, 64, 32, 8, 128, "same"), (16, 2000, 40, 32, 8, 64, "f32"),
                                  (16, 2000, 16, 32, 8, 128, "f32"), (16, 1500, 16, 24, 4, 256, "f32")])
def test_attention_repeats_bit_for_bit_from_cold_memory(sv, case):
    """Every other call starts with the caches out of L2, so tiles land late and out of order; the calls before the
    check run back to back or one at a time."""
    B, longest, N, H, K, D, out = case
    g = torch.Generator(device=DEV).manual_seed(B)
    ctx = torch.randint(N, longest + 1, (B,), generator=g, device=DEV).int()
    W = -(-longest // 64)
    table = torch.randperm(B * W, generator=g, device=DEV).int().view(B, W)
    k, v = (torch.randn((B * W, 64, K, D), generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    q = torch.randn((B, N, H, D), generator=g, device=DEV, dtype=torch.bfloat16)
    par = cuda(random_trees(np.random.default_rng(B), B, N))
    outs = [torch.empty((B, N, H, D), device=DEV, dtype=torch.float32 if out == "f32" else q.dtype) for _ in range(2)]
    ws = sv.new_attention_workspace(sv.spec_tree_attention_workspace(q, k, table), DEV)
    flush = torch.empty(300 << 20, dtype=torch.uint8, device=DEV)
    sv.spec_tree_attention(q, k, v, table, ctx, par, outs[0], workspace=ws)
    differ = torch.zeros((), dtype=torch.int64, device=DEV)
    for i in range(300):
        outs[1].fill_(float("nan"))
        if i % 2:
            flush.fill_(i % 251)
        if i % 4 > 1:
            torch.cuda.synchronize()
        sv.spec_tree_attention(q, k, v, table, ctx, par, outs[1], workspace=ws)
        differ += (outs[0] != outs[1]).sum()
    assert int(differ) == 0


def test_attention_on_other_streams_and_in_graphs(sv):
    """Two captured graphs with a workspace each, replayed at once on two streams with new inputs."""
    rng = np.random.default_rng(7)
    cases = [attention_case(rng, (700, 64, 1300), 20, 8, 2, 128, 64, torch.bfloat16) for _ in range(2)]
    fresh = attention_case(rng, (700, 64, 1300), 20, 8, 2, 128, 64, torch.bfloat16)
    want = [run_attention(sv, c, torch.float32)[0] for c in cases]
    outs, graphs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for c, s in zip(cases, streams):
        out = torch.zeros_like(want[0])
        ws = sv.new_attention_workspace(sv.spec_tree_attention_workspace(c["q"], c["k"], c["table"]), DEV)
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            sv.spec_tree_attention(c["q"], c["k"], c["v"], c["table"], c["ctx"], c["par"], out, workspace=ws)
        outs.append((out, ws))
        graphs.append(g)
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (out, _), w in zip(outs, want):
        assert torch.equal(out, w)
    cases[0]["q"].copy_(fresh["q"])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], run_attention(sv, cases[0], torch.float32)[0])


# ---------------------------------------------------------------------------
# Acceptance
# ---------------------------------------------------------------------------
def accept_case(rng, B, N, V, mode, with_probs, noise=1.0, temp=(0.6, 1.3), kind="random"):
    logits = (rng.standard_normal((B, N, V)) * 2).astype(np.float32)
    par = random_trees(rng, B, N, kind=kind)
    modes = {"greedy": np.zeros(B), "sample": np.ones(B), "mixed": rng.integers(0, 2, B)}[mode].astype(np.int64)
    t = rng.uniform(*temp, B).astype(np.float32)
    draft = logits + rng.standard_normal((B, N, V)).astype(np.float32) * noise
    probs = np.exp((draft - draft.max(-1, keepdims=True)) / t[:, None, None])
    probs = (probs / probs.sum(-1, keepdims=True)).astype(np.float32)
    tok = rng.integers(0, V, (B, N))
    for b in range(B):
        seen = {}
        for i in range(1, N):
            p = int(par[b, i])
            if p < 0:
                continue
            seen[p] = seen.get(p, 0) + 1
            if with_probs:
                tok[b, i] = rng.choice(V, p=probs[b, p].astype(np.float64) / probs[b, p].sum(dtype=np.float64))
            else:
                tok[b, i] = np.argsort(-draft[b, p], kind="stable")[min(seen[p] - 1, V - 1)]
    return dict(logits=logits, tok=tok, par=par, probs=probs if with_probs else None, mode=modes, temp=t,
                seed=int(rng.integers(0, 1 << 62)))


def run_accept(sv, c, **over):
    c = dict(c, **over)
    B, N, V = c["logits"].shape
    outs = [torch.full(s, -7, dtype=torch.int32, device=DEV) for s in ((B, N), (B, N), (B,))]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    probs = None if c["probs"] is None else cuda(c["probs"], torch.float32)
    sv.spec_tree_accept(cuda(c["logits"], torch.float32), cuda(c["tok"]), cuda(c["par"]), probs, c["seed"], cuda(c["mode"]),
                        cuda(c["temp"], torch.float32), *outs, dev_err=err)
    torch.cuda.synchronize()
    return [o.cpu().numpy() for o in outs], int(err.item())


def check_accept(c, got):
    out, path, m, margin = to.accept(c["logits"], c["tok"], c["par"], c["probs"], c["seed"], c["mode"], c["temp"])
    clear = margin >= 1e-5
    assert clear.mean() > 0.9
    for a, b in zip(got, (out, path, m)):
        assert np.array_equal(a[clear], b[clear])
    return m


ACCEPT = [
    (1, 1, 1), (3, 1, 7), (5, 7, 10), (16, 12, 257), (9, 64, 1000), (7, 30, 4099), (4, 13, 32003), (6, 20, 128256),
    (160, 6, 2048),
]


@pytest.mark.parametrize("mode,probs", [("greedy", False), ("sample", True), ("sample", False), ("mixed", True)])
@pytest.mark.parametrize("shape", ACCEPT, ids=["b%d_n%d_v%d" % s for s in ACCEPT])
def test_accept(sv, shape, mode, probs):
    B, N, V = shape
    c = accept_case(np.random.default_rng(V + N), B, N, V, mode, probs)
    got, err = run_accept(sv, c)
    assert err == 0
    check_accept(c, got)


@pytest.mark.parametrize("kind", ["chain", "star"])
@pytest.mark.parametrize("probs", [True, False])
def test_accept_deep_and_wide_trees(sv, kind, probs):
    """Low noise on a chain: long accepted paths; a star with high noise: many refused siblings."""
    c = accept_case(np.random.default_rng(8), 12, 40, 300, "mixed", probs, noise=0.05 if kind == "chain" else 3.0, kind=kind)
    got, err = run_accept(sv, c)
    assert err == 0
    m = check_accept(c, got)
    assert kind == "star" or m.max() > 8


@pytest.mark.parametrize("V", [1000, 1001, 32768])
def test_accept_of_a_chain_is_the_chain_call(sv, V):
    rng = np.random.default_rng(V)
    for probs in (True, False):
        c = accept_case(rng, 24, 6, V, "mixed", probs, noise=0.5, kind="chain")
        c["par"] = np.tile(np.arange(-1, 5), (24, 1))
        c["tok"][:, 1:] = np.where(c["tok"][:, 1:] >= 0, c["tok"][:, 1:], 0)
        (out, _, m), err = run_accept(sv, c)
        ct = torch.empty((24, 6), dtype=torch.int32, device=DEV)
        cm = torch.empty((24,), dtype=torch.int32, device=DEV)
        sv.spec_accept(cuda(c["logits"], torch.float32), cuda(c["tok"][:, 1:]),
                       cuda(c["probs"][:, :5], torch.float32) if probs else None, c["seed"], cuda(c["mode"]),
                       cuda(c["temp"], torch.float32), ct, cm)
        clear = to.accept(c["logits"], c["tok"], c["par"], c["probs"], c["seed"], c["mode"], c["temp"])[3] >= 1e-5
        assert err == 0 and clear.mean() > 0.9
        assert np.array_equal(out[clear], ct.cpu().numpy()[clear]) and np.array_equal(m[clear], cm.cpu().numpy()[clear])


def test_accept_refused_twins_and_certain_tokens(sv):
    """Siblings with the same token, a token of (almost) all mass, -inf logits, ties."""
    B, N, V = 6, 5, 64
    rng = np.random.default_rng(9)
    c = accept_case(rng, B, N, V, "sample", False)
    c["par"] = np.tile([-1, 0, 0, 0, 1], (B, 1))
    c["tok"][:, 1:4] = 7                       # twins: the second and third are never accepted
    c["logits"][1, :, :] = -np.inf             # all mass on one token
    c["logits"][1, :, 9] = 0.0
    c["logits"][2, :, 10:] = -np.inf           # half of the vocabulary impossible
    c["tok"][3, 1:4] = [1, 2, 3]
    c["logits"][3, 0, :] = -30.0               # three tokens with all of the mass
    c["logits"][3, 0, 1:4] = 0.0
    c["mode"][4] = c["mode"][5] = 0
    c["logits"][4, 0, :] = 1.0                 # every value ties: token 0
    c["tok"][4, 1:4] = [3, 0, 0]               # the first child that holds it is node 2
    got, err = run_accept(sv, c)
    assert err == 0
    check_accept(c, got)
    assert got[1][4].tolist()[:2] == [0, 2]
    assert got[0][1][0] == 9


def test_accept_equal_distributions_accept_the_first_child(sv):
    """p == q exactly (a uniform row): u q < p holds for every u, so the first child is accepted and the all-zero
    residual is never drawn from."""
    B, N, V = 8, 3, 512
    c = accept_case(np.random.default_rng(10), B, N, V, "sample", True)
    c["logits"][:] = 0.0
    c["probs"][:] = 1.0 / V
    c["par"] = np.tile([-1, 0, 0], (B, 1))
    (out, path, m), err = run_accept(sv, c)
    assert err == 0 and np.all(m == 1) and np.all(path[:, 1] == 1) and np.array_equal(out[:, 0], c["tok"][:, 1])


def test_accept_reports_bad_rows(sv):
    B, N, V = 8, 5, 100
    rng = np.random.default_rng(11)
    c = accept_case(rng, B, N, V, "sample", True)
    c["par"] = np.tile([-1, 0, 0, 1, 2], (B, 1))
    bits = 0
    good, _ = run_accept(sv, c)
    c["tok"][1, 3] = V
    c["tok"][2, 1] = -1
    c["par"][3, 2] = 4
    c["mode"][4] = 2
    c["temp"][5] = 0.0
    c["temp"][6] = np.nan
    c["par"][7] = [-2, 0, 5, 9, -7]            # an empty row: its other inputs do not matter
    c["tok"][0, 0] = -5                        # node 0's token is not looked at
    got, err = run_accept(sv, c)
    for n in ("token", "tree", "mode", "temperature"):
        bits |= sv.DEVERR[n]
    assert err == bits
    for a, b in zip(got, good):
        assert np.array_equal(a[0], b[0]) and np.all(a[1:] == -1)


@pytest.mark.parametrize("probs", [True, False])
def test_accept_under_every_cluster_shape(sv, monkeypatch, probs):
    """Threads a CTA and CTAs a cluster forced in turn; 16 CTAs of 256 threads need 4 * 256 logits each."""
    c = accept_case(np.random.default_rng(21), 40, 9, 16 * 1024 + 3, "mixed", probs)
    for threads in (128, 256):
        for csize in (1, 2, 4, 8, 16):
            monkeypatch.setenv("SPEC_ACCEPT_CONFIG", f"{threads}x{csize}")
            got, err = run_accept(sv, c)
            assert err == 0, (threads, csize)
            check_accept(c, got)


@pytest.mark.parametrize("probs", [True, False])
def test_accept_rows_that_hold_no_distribution(sv, probs):
    """Logits of node 0 all -inf, all NaN, or with a +inf: no probability is defined. The row ends there: no child is
    accepted by sampling and its last token is -1; other rows are as they would be without it."""
    c = accept_case(np.random.default_rng(41), 6, 5, 700, "sample", probs)
    c["par"][:] = [-1, 0, 0, 1, 2]
    c["tok"][:, 1:] %= 700
    good, err = run_accept(sv, c)
    bad = dict(c, logits=c["logits"].copy())
    bad["logits"][1, 0] = -np.inf
    bad["logits"][2, 0] = np.nan
    bad["logits"][3, 0, 17] = np.inf
    got, err2 = run_accept(sv, bad)
    assert err == 0 and err2 == 0
    for x, y in zip(got, good):
        assert np.array_equal(x[[0, 4, 5]], y[[0, 4, 5]])
    for b in (1, 2, 3):
        assert got[2][b] == 0 and got[1][b].tolist() == [0, -1, -1, -1, -1] and got[0][b].tolist() == [-1] * 5


def test_accept_unaligned_rows_and_graph(sv):
    """Logits that start 4 bytes off a 16-byte boundary, and a captured call replayed on new inputs."""
    rng = np.random.default_rng(12)
    c, d = (accept_case(rng, 5, 9, 1000, "mixed", True) for _ in range(2))
    flat = torch.empty(5 * 9 * 1000 + 1, device=DEV)
    logits = flat[1:].view(5, 9, 1000)
    probs = torch.empty((5, 9, 1000), device=DEV)
    ints = [torch.empty((5, 9), dtype=torch.int32, device=DEV) for _ in range(4)]
    mode, m = (torch.empty(5, dtype=torch.int32, device=DEV) for _ in range(2))
    temp = torch.empty(5, device=DEV)

    def load(x):
        logits.copy_(cuda(x["logits"], torch.float32))
        probs.copy_(cuda(x["probs"], torch.float32))
        ints[0].copy_(cuda(x["tok"]))
        ints[1].copy_(cuda(x["par"]))
        mode.copy_(cuda(x["mode"]))
        temp.copy_(cuda(x["temp"], torch.float32))

    call = lambda: sv.spec_tree_accept(logits, ints[0], ints[1], probs, c["seed"], mode, temp, ints[2], ints[3], m)  # noqa: E731
    load(c)
    call()
    torch.cuda.synchronize()
    check_accept(c, [t.cpu().numpy() for t in (ints[2], ints[3], m)])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    d["seed"] = c["seed"]
    load(d)
    g.replay()
    torch.cuda.synchronize()
    check_accept(d, [t.cpu().numpy() for t in (ints[2], ints[3], m)])


# ---------------------------------------------------------------------------
# The cache between two steps
# ---------------------------------------------------------------------------
def random_paths(rng, B, N, longest):
    path, m = np.full((B, N), -1), np.zeros(B, np.int64)
    for b in range(B):
        m[b] = rng.integers(0, min(longest, N - 1) + 1)
        path[b, : m[b] + 1] = [0, *np.sort(rng.choice(np.arange(1, N), m[b], replace=False))] if N > 1 else [0]
    return path, m


@pytest.mark.parametrize("layers,B,N,bs,K,D,dtype", [
    (1, 1, 1, 16, 1, 8, torch.bfloat16), (3, 5, 16, 16, 2, 64, torch.bfloat16), (2, 4, 64, 5, 3, 7, torch.float32),
    (4, 3, 64, 64, 8, 128, torch.float16), (2, 3, 9, 4, 1, 6, torch.uint8), (1, 2, 30, 1, 5, 3, torch.bfloat16),
    (2, 2, 12, 7, 20, 256, torch.float32)])
def test_commit_path(sv, layers, B, N, bs, K, D, dtype):
    rng = np.random.default_rng(N * 7 + bs)
    ctx = rng.integers(N, N + 150, B)
    W = -(-int(ctx.max()) // bs)
    P = B * W + 3
    table = rng.permutation(P)[: B * W].reshape(B, W)
    shape = (layers, P, bs, K, D)
    k, v = (torch.randint(0, 200, shape, device=DEV).to(dtype) for _ in range(2))
    path, m = random_paths(rng, B, N, N)
    m[0] = path[0].max() if N == 1 else m[0]
    want = to.commit_path(*(t.float().cpu().numpy() for t in (k, v)), table, ctx, path, m)
    new = torch.full((B,), -9, dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    sv.spec_cache_commit_path(k, v, cuda(table), cuda(ctx), cuda(path), cuda(m), new, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert np.array_equal(k.float().cpu().numpy(), want[0]) and np.array_equal(v.float().cpu().numpy(), want[1])
    assert np.array_equal(new.cpu().numpy(), want[2])


def test_commit_path_one_layer_and_bad_rows(sv):
    rng = np.random.default_rng(20)
    B, N, bs, W, P = 9, 8, 4, 10, 100
    table = rng.permutation(P)[: B * W].reshape(B, W)
    ctx = np.full(B, 33)
    path, m = random_paths(rng, B, N, N)
    m[:] = 3
    path[:] = [0, 2, 5, 6, -1, -1, -1, -1]
    m[1] = -1                      # a row that accepted nothing
    m[2] = N
    path[3, 2] = 2                 # does not increase
    path[4, 0] = 1
    ctx[5] = N - 1
    ctx[6] = W * bs + 1
    table[7, 8] = P                # a page that the path does not touch is not looked at
    path[8, 3] = N
    for cut in (0, 1):
        k, v = (torch.randn((P, bs, 2, 8 + 4 * cut), device=DEV) for _ in range(2))
        want = to.commit_path(k[None].cpu().numpy(), v[None].cpu().numpy(), table, ctx, path, m)
        new = torch.empty(B, dtype=torch.int32, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        sv.spec_cache_commit_path(k, v, cuda(table), cuda(ctx), cuda(path), cuda(m), new, dev_err=err)
        assert int(err.item()) == sv.DEVERR["accept_len"] | sv.DEVERR["ctx_len"]
        assert np.array_equal(k[None].cpu().numpy(), want[0]) and np.array_equal(v[None].cpu().numpy(), want[1])
        assert np.array_equal(new.cpu().numpy(), want[2]) and want[2][0] == 29


def test_commit_path_padded_rows_of_any_length(sv):
    """Rows that accepted nothing may hold any length: their new length is max(0, length - N)."""
    N, ctx = 8, [-2 ** 31, -2 ** 31 + 3, -1, 0, 7, 8, 9, 2 ** 31 - 1]
    B = len(ctx)
    k, v = (torch.zeros((2, 4, 4, 1, 8), device=DEV) for _ in range(2))
    new = torch.full((B,), -9, dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    path = np.full((B, N), -1)
    sv.spec_cache_commit_path(k, v, cuda(np.zeros((B, 2))), cuda(np.array(ctx)), cuda(path), cuda(np.full(B, -1)), new, dev_err=err)
    assert int(err.item()) == 0 and new.tolist() == [max(0, c - N) for c in ctx]


@pytest.mark.parametrize("entry", [6, 7])
@pytest.mark.parametrize("page", [-1, 100])
def test_commit_path_bad_page(sv, entry, page):
    """Entry 6 holds token base + 0's page, entry 7 the last source's: a bad id in either leaves the row as it was."""
    rng = np.random.default_rng(21)
    B, N, bs, W, P = 2, 8, 4, 10, 100
    table = rng.permutation(P)[: B * W].reshape(B, W)
    table[1, entry] = page
    path, m = np.tile([0, 2, 5, 6, -1, -1, -1, -1], (B, 1)), np.full(B, 3)
    k, v = (torch.randn((1, P, bs, 2, 8), device=DEV) for _ in range(2))
    want = to.commit_path(k.cpu().numpy(), v.cpu().numpy(), table, np.full(B, 33), path, m)
    new = torch.empty(B, dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    sv.spec_cache_commit_path(k, v, cuda(table), cuda(np.full(B, 33)), cuda(path), cuda(m), new, dev_err=err)
    assert int(err.item()) == sv.DEVERR["block_id"] and new.tolist() == [29, 25]
    assert np.array_equal(k.cpu().numpy(), want[0]) and np.array_equal(v.cpu().numpy(), want[1])


def run_update(sv, table, refs, cur, want, src, bs, caches=None):
    t, r = cuda(table), cuda(refs)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    sv.spec_cache_update(t, r, cuda(cur), cuda(want), bs, src_rows=None if src is None else cuda(src), dev_err=err,
                         **({} if caches is None else dict(k_cache=caches[0], v_cache=caches[1])))
    torch.cuda.synchronize()
    return t.cpu().numpy(), r.cpu().numpy(), int(err.item())


@pytest.mark.parametrize("B,W,bs,P,layers", [(1, 1, 16, 4, 1), (6, 5, 4, 80, 2), (33, 9, 16, 700, 1), (8, 140, 3, 3000, 1),
                                              (300, 7, 8, 5000, 0), (5, 4, 64, 60, 3)])
def test_update_random_walk(sv, B, W, bs, P, layers):
    """Many steps of trims, reservations, forks, reorderings and frees against the definition, contents included."""
    rng = np.random.default_rng(B * W)
    table, refs = np.full((B, W), -1), np.zeros(P, np.int64)
    refs[[1, P - 1]] = 1                          # pages some other holder keeps
    cur = np.zeros(B, np.int64)
    caches = [torch.randn((layers, P, bs, 2, 5), device=DEV) for _ in range(2)] if layers else None
    for step in range(10):
        src = None if step % 3 == 0 else rng.integers(-1 if step % 2 else 0, B, B)
        want = rng.integers(0, W * bs + 1, B)
        if step % 4 == 2:
            want = np.minimum(want, np.maximum(cur, 1))   # truncations, into shared pages too
        nt, nr, copies = to.update(table, refs, cur, want, src, bs)
        before = None if caches is None else [c.clone() for c in caches]
        gt, gr, err = run_update(sv, table, refs, cur, want, src, bs, caches)
        assert err == 0 and np.array_equal(gt, nt) and np.array_equal(gr, nr), step
        for a, b in zip(caches or [], before or []):
            for x, y, n in copies:
                b_new = b[:, x, :n].clone()
                assert torch.equal(a[:, y, :n], b_new)
            touched = torch.zeros((P, bs), dtype=torch.bool, device=DEV)
            for _, y, n in copies:
                touched[y, :n] = True
            assert torch.equal(a[:, ~touched], b[:, ~touched])
        s = np.arange(B) if src is None else src
        cur = np.where(s >= 0, want, 0)           # the rows are filled up to their room
        table, refs = gt, gr


def test_update_runs_out_of_pages_and_reports_bad_rows(sv):
    B, W, bs, P = 5, 4, 4, 9
    table = np.full((B, W), -1)
    refs = np.zeros(P, np.int64)
    t, r, err = run_update(sv, table, refs, np.zeros(B), np.full(B, 11), None, bs)
    assert err == sv.DEVERR["no_page"]
    want = to.update(table, refs, np.zeros(B, int), np.full(B, 11), None, bs)
    assert np.array_equal(t, want[0]) and np.array_equal(r, want[1])
    assert t[:3, :3].reshape(-1).tolist() == list(range(9)) and np.all(t[3:] == -1)
    # row 0: source out of range, row 1: length out of range, row 2: keeps tokens of a row without pages
    src, cur, new = np.array([7, 1, 3, 3, -1]), np.array([11, 11, 11, 5, 0]), np.array([3, 17, 5, 0, 9])
    t2, r2, err = run_update(sv, t, r, cur, new, src, bs)
    want = to.update(t, r, cur, new, src, bs)
    assert err == sv.DEVERR["src_row"] | sv.DEVERR["ctx_len"] | sv.DEVERR["block_id"]
    assert np.array_equal(t2, want[0]) and np.array_equal(r2, want[1])
    assert np.array_equal(t2[:3], t[:3])


def test_update_and_commit_in_graphs(sv):
    """The step's table calls captured once and replayed: the tables live in device memory."""
    rng = np.random.default_rng(30)
    B, W, bs, P, N = 7, 12, 8, 200, 10
    low = rng.integers(1, W * bs - N, B)
    table, refs, _ = to.update(np.full((B, W), -1), np.zeros(P, int), np.zeros(B, int), low + N, None, bs)
    t, r, lo, hi = cuda(table), cuda(refs), cuda(low), cuda(low + N)
    ws = torch.empty(sv.spec_cache_update_workspace(t, r), dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        sv.spec_cache_update(t, r, hi, lo, bs, workspace=ws)
        sv.spec_cache_update(t, r, lo, hi, bs, workspace=ws)
    for _ in range(4):
        table, refs, _ = to.update(table, refs, low + N, low, None, bs)
        table, refs, _ = to.update(table, refs, low, low + N, None, bs)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(r.cpu().numpy(), refs)


def test_bindings_refuse(sv):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
    f = lambda *s: torch.zeros(s, device=DEV)  # noqa: E731
    q, kc = f(2, 4, 8, 64).bfloat16(), f(6, 16, 2, 64).bfloat16()
    good = dict(q=q, k_cache=kc, v_cache=kc, block_table=i32(2, 3), ctx_lens=i32(2), parents=i32(2, 4), out=f(2, 4, 8, 64))
    for name, bad in (("q", q.float()), ("k_cache", kc.half()), ("v_cache", kc[:5].contiguous()), ("ctx_lens", i32(3)),
                      ("parents", i32(2, 5)), ("block_table", i32(1, 3)), ("out", f(2, 4, 8, 64).half()),
                      ("out", f(2, 4, 8, 128)[..., ::2]), ("parents", i32(2, 4).cpu())):
        with pytest.raises((ValueError, TypeError)):
            sv.spec_tree_attention(**dict(good, **{name: bad}))
    with pytest.raises(ValueError):
        sv.spec_cache_update(i32(2, 3), i32(6), i32(2), i32(2), 16, k_cache=kc, v_cache=None)
    with pytest.raises(ValueError):
        sv.spec_cache_update(i32(2, 3), i32(7), i32(2), i32(2), 16, k_cache=kc, v_cache=kc)
    with pytest.raises(sv.SpecError):
        sv.spec_cache_update(i32(2, 3), i32(6), i32(2), i32(2), 0)
    with pytest.raises(ValueError):
        sv.spec_tree_accept(f(2, 4, 9), i32(2, 4), i32(2, 4), f(2, 3, 9), 0, i32(2), f(2), i32(2, 4), i32(2, 4), i32(2))
    with pytest.raises(ValueError):
        sv.spec_cache_commit_path(kc, kc, i32(2, 3), i32(2), i32(2, 4), i32(3), i32(2))


# ---------------------------------------------------------------------------
# A run of all of them
# ---------------------------------------------------------------------------
def test_tree_decoding_emits_the_greedy_sequence(sv):
    """A small attention model decoded with trees on the paged cache (pages reserved, tree attended, path accepted and
    compacted, tail freed, every step on the device) emits, token for token, what one-token decoding by the same
    model in 64 bits on the host does; rows are forked half way and go on alike."""
    rng = np.random.default_rng(40)
    B, N, H, K, D, V, bs, L, P, W = 4, 8, 4, 2, 64, 37, 16, 2, 64, 8
    steps, start = 9, 5
    emb, wq, wk, wv = (rng.standard_normal(s) for s in ((V, 32), (L, 32, H * D), (L, 32, K * D), (L, 32, K * D)))
    head = rng.standard_normal((L, H * D, V))
    bf = lambda x: torch.from_numpy(np.asarray(x)).to(torch.bfloat16).double().numpy()  # noqa: E731

    def project(tokens, l):  # depends on the token alone, so that a compacted cache is what decoding would have written
        x = emb[tokens]
        return bf(x @ wq[l] / 6), bf(x @ wk[l] / 6), bf(x @ wv[l] / 6)

    def host_logits(seq):
        z = 0.0
        for l in range(L):
            qh, kh, vh = project(np.array(seq), l)
            for h in range(H):
                g = h // (H // K)
                s = kh[:, g * D:(g + 1) * D] @ qh[-1, h * D:(h + 1) * D] / np.sqrt(D)
                p = np.exp(s - s.max())
                z = z + (p / p.sum() @ vh[:, g * D:(g + 1) * D]) @ head[l, h * D:(h + 1) * D]
        return z

    prompts = [list(rng.integers(0, V, start)) for _ in range(B)]
    prompts[2] = prompts[3] = prompts[0]
    greedy = []
    for p in prompts:
        seq = list(p)
        for _ in range(steps * N):
            seq.append(int(host_logits(seq).argmax()))
            if len(seq) > start + 40:
                break
        greedy.append(seq)

    caches = [torch.zeros((L, P, bs, K, D), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    table, refs = cuda(np.full((B, W), -1)), cuda(np.zeros(P))
    lens = cuda(np.full(B, start - 1))            # the last prompt token is the first tree's root
    zero = cuda(np.zeros(B))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    sv.spec_cache_update(table, refs, zero, lens, bs, dev_err=err)

    def write(tokens, at):                        # K and V of tokens[b, j] at token at[b] + j
        host = table.cpu().numpy()
        for l in range(L):
            for b in range(B):
                _, kk, vv = project(tokens[b], l)
                for j in range(tokens.shape[1]):
                    t = int(at[b]) + j
                    for c, x in zip(caches, (kk, vv)):
                        c[l, host[b, t // bs], t % bs] = torch.from_numpy(x[j].reshape(K, D)).to(DEV, torch.bfloat16)

    write(np.array([p[:-1] for p in prompts]), np.zeros(B, int))
    seqs, accepted = [list(p) for p in prompts], 0
    for step in range(steps):
        if step == 4:                             # rows 2 and 3 continue from row 0
            src = cuda([0, 1, 0, 0])
            sv.spec_cache_update(table, refs, lens, lens[src.long()].contiguous(), bs, src_rows=src, k_cache=caches[0],
                                 v_cache=caches[1], dev_err=err)
            lens = lens[src.long()].contiguous()
            seqs[2], seqs[3] = list(seqs[0]), list(seqs[0])
        par = random_trees(rng, B, N, unused=True)
        tok = rng.integers(0, V, (B, N))
        for b in range(B):
            tok[b, 0] = seqs[b][-1]
            for i in range(1, N):                 # most drafts are right where their branch is
                chain = to.line(par[b], i)[1:] if par[b, i] >= 0 else []
                known = seqs[b] + [int(tok[b, j]) for j in chain[::-1][1:]]
                if known == greedy[b][: len(known)] and rng.random() < 0.7:
                    tok[b, i] = greedy[b][len(known)]
        ctx = (lens + N).to(torch.int32)
        sv.spec_cache_update(table, refs, lens, ctx, bs, dev_err=err)
        write(tok, lens.cpu().numpy())
        logits = torch.zeros((B, N, V), dtype=torch.float64, device=DEV)
        for l in range(L):
            q = torch.from_numpy(project(tok, l)[0].reshape(B, N, H, D)).to(DEV, torch.bfloat16)
            out = torch.empty((B, N, H, D), device=DEV)
            sv.spec_tree_attention(q, caches[0][l], caches[1][l], table, ctx, cuda(par), out, dev_err=err)
            logits += out.double().reshape(B, N, H * D) @ torch.from_numpy(head[l]).to(DEV)
        outs = [torch.empty(s, dtype=torch.int32, device=DEV) for s in ((B, N), (B, N), (B,))]
        sv.spec_tree_accept(logits.float(), cuda(tok), cuda(par), None, 0, zero, torch.ones(B, device=DEV), *outs, dev_err=err)
        new = torch.empty(B, dtype=torch.int32, device=DEV)
        sv.spec_cache_commit_path(*caches, table, ctx, outs[1], outs[2], new, dev_err=err)
        sv.spec_cache_update(table, refs, ctx, new, bs, dev_err=err)
        lens = new
        for b in range(B):
            m = int(outs[2][b])
            accepted += m
            seqs[b] += outs[0][b, : m + 1].tolist()
            assert seqs[b] == greedy[b][: len(seqs[b])], (step, b)
        assert np.array_equal(refs.cpu().numpy(), np.bincount(table[table >= 0].cpu().numpy(), minlength=P))
        if max(len(s) for s in seqs) > start + 30:
            break
    assert int(err.item()) == 0 and accepted > steps
