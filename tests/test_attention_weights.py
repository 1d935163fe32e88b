"""Attention weight per cached key: pins of the definition and refusals (CPU), and the kernels
against the fp64 definition (GPU)."""
import math

import numpy as np
import pytest

import oracle.fp8 as ofp8
import oracle.paged_attention as pa
from continuous_batching_gb300 import binding as bd
from continuous_batching_gb300 import workloads as wl
from oracle.bounded import lse_and_weights

torch = pytest.importorskip("torch")


# ------------------------------------------------------------------ the definition (CPU)

def test_definition_against_softmax_and_closed_forms():
    st = wl.make_step(4, 2, 64, 8, [20, 9, 1], [5, 9, 1], seed=0)
    q, k = pa.bf16_to_f64(st.q), pa.bf16_to_f64(st.k_pool)
    lse, w = lse_and_weights(q, k, st.block_table, st.cu_seqlens_q, st.ctx_lens)
    # every (row, q head) hands out a weight of one
    for s, n in enumerate(st.n_q):
        np.testing.assert_allclose(w[s].sum(axis=1), n * 2.0, rtol=1e-12)
    # against torch's softmax, one sequence
    K = torch.from_numpy(pa.gather(k, st.block_table[0], 20)).repeat_interleave(2, 0)
    a = torch.einsum("nhd,hkd->nhk", torch.from_numpy(q[:5]), K) / 8.0
    a[torch.arange(20)[None, None].expand_as(a) > torch.arange(15, 20)[:, None, None]] = -math.inf
    np.testing.assert_allclose(lse[:5], torch.logsumexp(a, -1).numpy(), rtol=1e-12)
    p = torch.softmax(a, -1).view(5, 2, 2, 20).sum((0, 2))
    np.testing.assert_allclose(w[0], p.numpy(), atol=1e-12)
    # one key: all the weight; equal keys: equal weights
    assert w[2].tolist() == [[2.0], [2.0]]
    lse, w = lse_and_weights(q, np.ones_like(k), st.block_table, st.cu_seqlens_q, st.ctx_lens)
    np.testing.assert_allclose(w[1][:, 8], 2 / 9.0, rtol=1e-12)      # seen by the last row alone


def _call(**kw):
    a = dict(q=16, kp=16, lse=16, tb=16, mb=4, cu=16, ctx=16, B=2, T=2, held=None, rows=16, w=16, n=4, m=64)
    shape = kw.pop("shape", bd.Shape.make(4, 2, 128, 16, 8))
    scale = kw.pop("scale", None)
    a.update(kw)
    f = bd.load().paged_attention_weights if scale is None else bd.load().paged_attention_weights_fp8
    return f(a["q"], a["kp"], a["lse"], a["tb"], a["mb"], a["cu"], a["ctx"], a["B"], a["T"], a["held"],
             a["rows"], a["w"], a["n"], a["m"], *(() if scale is None else (scale,)), shape, None, None)


@pytest.mark.parametrize("kw, want", [
    (dict(B=-1), bd.PA_ERR_INVALID), (dict(T=-1), bd.PA_ERR_INVALID), (dict(T=0), bd.PA_OK),
    (dict(B=0), bd.PA_OK), (dict(q=None), bd.PA_ERR_INVALID), (dict(kp=None), bd.PA_ERR_INVALID),
    (dict(lse=None), bd.PA_ERR_INVALID), (dict(tb=None), bd.PA_ERR_INVALID),
    (dict(cu=None), bd.PA_ERR_INVALID), (dict(ctx=None), bd.PA_ERR_INVALID),
    (dict(w=None), bd.PA_ERR_INVALID), (dict(m=0), bd.PA_ERR_INVALID), (dict(m=-1), bd.PA_ERR_INVALID),
    (dict(rows=None, n=1), bd.PA_ERR_INVALID), (dict(n=(1 << 18) + 1), bd.PA_ERR_SHAPE),
    (dict(m=2 ** 31 - 1), bd.PA_ERR_SHAPE), (dict(m=2 ** 31 - 4096), bd.PA_ERR_SHAPE),
    (dict(lse=20), bd.PA_ERR_INVALID), (dict(q=24), bd.PA_ERR_INVALID),
    (dict(kp=8), bd.PA_ERR_INVALID), (dict(shape=bd.Shape.make(4, 2, 32, 16, 8)), bd.PA_ERR_SHAPE),
    (dict(shape=bd.Shape.make(6, 2, 128, 16, 8)), bd.PA_ERR_SHAPE),
    (dict(shape=bd.Shape.make(4, 2, 64, 16, 8), scale=1.0), bd.PA_ERR_SHAPE),
    (dict(scale=0.0), bd.PA_ERR_INVALID), (dict(scale=float("nan")), bd.PA_ERR_INVALID),
])
def test_refusals(kw, want):
    assert _call(**kw) == want


def _step_call(**kw):
    a = dict(q=16, kp=16, vp=16, tb=16, mb=4, cu=16, ctx=16, B=2, T=2, mc=64, items=16, n_items=2, ws=16,
             wb=None, out=16, lse=16, held=None, rows=16, w=16, n=4, m=64)
    shape = bd.Shape.make(4, 2, 128, 16, 8)
    a.update(kw)
    if a["wb"] is None:
        a["wb"] = bd.pa_step_weights_workspace_bytes(shape, max(a["B"], 0), max(a["T"], 0), max(a["mc"], 0))
    return bd.load().paged_attention_step_weights(*a.values(), shape, None, None)


# Every refusal comes before the attention step's launch (it would fail here, without a device).
@pytest.mark.parametrize("kw, want", [
    (dict(T=0), bd.PA_OK), (dict(B=0), bd.PA_OK), (dict(n_items=0), bd.PA_OK), (dict(B=-1), bd.PA_ERR_INVALID),
    (dict(mc=0), bd.PA_ERR_INVALID), (dict(mc=2 ** 31 - 4096), bd.PA_ERR_SHAPE),
    (dict(m=2 ** 31 - 4096), bd.PA_ERR_SHAPE), (dict(m=0), bd.PA_ERR_INVALID), (dict(w=None), bd.PA_ERR_INVALID),
    (dict(lse=None), bd.PA_ERR_INVALID), (dict(lse=20), bd.PA_ERR_INVALID), (dict(ws=None), bd.PA_ERR_WORKSPACE),
    (dict(wb=64), bd.PA_ERR_WORKSPACE), (dict(ws=24), bd.PA_ERR_INVALID), (dict(rows=None, n=1), bd.PA_ERR_INVALID),
    (dict(B=8193, n=8193), bd.PA_ERR_SHAPE), (dict(n=(1 << 18) + 1), bd.PA_ERR_SHAPE),
])
def test_step_refusals(kw, want):
    assert _step_call(**kw) == want


# ------------------------------------------------------------------ the kernels (GPU)

def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.view(dtype)


# One weight is exp(x), x = s c - lse in base 2. Against the given lse its relative error is the
# error of x times ln 2, plus ex2's (2 units of 2^-23) and the sum's. s is an fp32 accumulation of
# D exact products: <= (D / 8 + 4) 2^-23 of the sum of magnitudes (the tensor cores add groups of
# products with at least this much), x two roundings of its own magnitude and lse's. The sum over
# n terms, all positive: in a thread 32 partial sums of a column's four, added up: (40 + n / 128)
# 2^-24 at most. With |q| |k| the bound of |s| that the test knows.
def tolerance(q, k, D, lse, n):
    s = np.abs(q).max() * np.abs(k).max() * D
    x = 1.4427 / math.sqrt(D) * s * (D / 8 + 4) * 2.0 ** -23
    x += (1.4427 / math.sqrt(D) * s + 1.4427 * np.abs(lse).max()) * 2 * 2.0 ** -24
    return min(x * 0.6932, 1e-3) + 4 * 2.0 ** -24 + (40 + n / 128) * 2.0 ** -24


def _check(st, fp8=False, held=None, order=None, extra=3, seed=0):
    rng = np.random.default_rng(seed)
    B, g = len(st.ctx_lens), st.Hq // st.Hkv
    shape = bd.Shape.make(st.Hq, st.Hkv, st.D, st.block_size, st.num_blocks)
    q = pa.bf16_to_f64(st.q)
    if fp8:
        scale = 0.0125
        codes = ofp8.quantize(st.k_pool, scale)
        k, kp = ofp8.dequantize(codes, scale), dev(codes)
    else:
        k, kp = pa.bf16_to_f64(st.k_pool), dev(st.k_pool.view(np.int16), torch.bfloat16)
    lse, _ = lse_and_weights(q, k, st.block_table, st.cu_seqlens_q, st.ctx_lens)
    lse = (lse + 0.25 * rng.random(lse.shape)).astype(np.float32)      # any reference will do
    _, want = lse_and_weights(q, k, st.block_table, st.cu_seqlens_q, st.ctx_lens, lse.astype(np.float64))
    n_rows, max_len = B + extra, int(st.ctx_lens.max()) + 13
    rows = rng.permutation(n_rows)[:B].astype(np.int32) if order is None else order
    start = rng.random((n_rows, st.Hkv, max_len)).astype(np.float32)
    w = dev(start.copy())
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (dev(st.q.view(np.int16), torch.bfloat16), kp, dev(lse), dev(st.block_table),
            dev(st.cu_seqlens_q), dev(st.ctx_lens), None if rows is None else dev(rows), w)
    kw = dict(held=None if held is None else dev(held.astype(np.int32)), err=err)
    run = (lambda: bd.paged_attention_weights_fp8(*args, scale, shape, **kw)) if fp8 else \
        (lambda: bd.paged_attention_weights(*args, shape, **kw))
    run()
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    got = w.cpu().numpy()
    expect = start.astype(np.float64)
    worst = 0.0
    for s in range(B):
        row = s if rows is None else int(rows[s])
        n, c = int(st.n_q[s]), int(st.ctx_lens[s])
        if row < 0 or n == 0:
            continue
        keep = c - n if held is None else int(held[s])
        expect[row, :, keep:c] = 0
        expect[row, :, :c] += want[s]
        sl = slice(int(st.cu_seqlens_q[s]), int(st.cu_seqlens_q[s + 1]))
        tol = tolerance(q[sl], k, st.D, lse[sl], n * g)
        d = np.abs(got[row, :, :c] - expect[row, :, :c])
        bound = tol * want[s] + 2.0 ** -24 * expect[row, :, :c] + 1e-37
        assert np.all(d <= bound), (s, float((d / bound).max()))
        worst = max(worst, float((d / bound).max()))
        expect[row, :, :c] = got[row, :, :c]
    assert np.array_equal(got, expect.astype(np.float32))            # the rest as it was, to the bit
    # the same call from the same state gives the same bits
    w.copy_(dev(start))
    run()
    assert np.array_equal(w.cpu().numpy(), got)
    return worst


SHAPES = [(4, 2, 64, 16), (32, 8, 128, 16), (8, 8, 128, 32), (8, 1, 128, 8), (16, 1, 64, 128), (4, 2, 128, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("Hq, Hkv, D, bs", SHAPES)
@pytest.mark.parametrize("ctx, n_q", [
    ([1], [1]),
    ([17, 40, 64, 100], [1, 1, 1, 1]),
    ([128, 129, 127, 256, 1, 300], [1, 1, 1, 1, 1, 1]),
    ([2049, 4000], [1, 1]),
    ([50, 9, 200], [7, 9, 3]),                              # short chunks: one query tile
    ([140, 300, 1000], [140, 257, 33]),                     # chunks from the start and behind a prior
    ([700, 20, 129, 64], [300, 1, 129, 0]),                 # mixed, one sequence without rows
])
def test_against_the_definition(Hq, Hkv, D, bs, ctx, n_q):
    _check(wl.make_step(Hq, Hkv, D, bs, ctx, n_q, seed=len(ctx) + D))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq, Hkv, bs", [(32, 8, 16), (8, 8, 32), (8, 1, 8), (16, 1, 128)])
@pytest.mark.parametrize("ctx, n_q", [
    ([1, 40, 129], [1, 1, 1]), ([2049, 700], [1, 1]), ([50, 9, 200], [7, 9, 3]),
    ([140, 300, 700, 20], [140, 257, 33, 1]),
])
def test_fp8_against_the_definition(Hq, Hkv, bs, ctx, n_q):
    _check(wl.make_step(Hq, Hkv, 128, bs, ctx, n_q, seed=5), fp8=True)


@pytest.mark.gpu
def test_many_sequences():
    """More sequences than threads (the deal over rounds of them), single tiles, many items."""
    rng = np.random.default_rng(2)
    ctx = rng.integers(1, 200, 900)
    _check(wl.make_step(2, 2, 64, 8, ctx, np.ones(900, int), seed=9))
    n_q = np.minimum(ctx, rng.integers(0, 90, 900))
    _check(wl.make_step(4, 2, 64, 8, ctx, n_q, seed=10))


@pytest.mark.gpu
def test_rows_held_and_windows():
    st = wl.make_step(8, 2, 128, 16, [300, 77, 129], [20, 1, 129], seed=4)
    _check(st, order=np.array([2, 0, 1], np.int32), extra=0)
    _check(st, order=None, extra=0)
    _check(st, order=np.array([4, -1, 1], np.int32))
    # an observation window: the last rows alone give weight, everything is set afresh
    _check(st, held=np.array([0, 0, 0]))
    _check(st, held=np.array([300, 50, 129]))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq, Hkv, D, fp8", [(8, 2, 128, False), (8, 8, 64, False), (16, 2, 128, True)])
def test_a_sequences_bits_do_not_depend_on_the_batch(Hq, Hkv, D, fp8):
    """However the key tiles are dealt (four, three, two or one to an item), a sum has the same bits."""
    ctx, n_q = [1500, 700, 2048, 130, 90, 901], [700, 1, 300, 130, 20, 515]
    st = wl.make_step(Hq, Hkv, D, 16, ctx, n_q, seed=12)
    shape = bd.Shape.make(st.Hq, st.Hkv, st.D, st.block_size, st.num_blocks)
    q = dev(st.q.view(np.int16), torch.bfloat16)
    kp = dev(ofp8.quantize(st.k_pool, 0.0125)) if fp8 else dev(st.k_pool.view(np.int16), torch.bfloat16)
    gen = torch.Generator("cuda").manual_seed(3)
    lse = 4 + torch.rand(st.T, Hq, device="cuda", generator=gen)
    start = torch.rand(len(ctx), Hkv, 2100, device="cuda", generator=gen)

    def run(seqs):
        w = start.clone()
        at = [slice(int(st.cu_seqlens_q[s]), int(st.cu_seqlens_q[s + 1])) for s in seqs]
        cu = np.concatenate([[0], np.cumsum([n_q[s] for s in seqs])]).astype(np.int32)
        i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
        args = (torch.cat([q[a] for a in at]), kp, torch.cat([lse[a] for a in at]), dev(st.block_table[list(seqs)]),
                dev(cu), i32([ctx[s] for s in seqs]), i32(list(seqs)), w)
        if fp8:
            bd.paged_attention_weights_fp8(*args, 0.0125, shape)
        else:
            bd.paged_attention_weights(*args, shape)
        return w

    whole = run(range(len(ctx)))
    for seqs in [[s] for s in range(len(ctx))] + [[4, 0], [2, 5, 1], [5, 4, 3, 2, 1, 0], [0] + [1, 3, 4]]:
        part = run(seqs)
        for s in range(len(ctx)):
            assert torch.equal(part[s], whole[s] if s in seqs else start[s]), (seqs, s)


@pytest.mark.gpu
def test_stale_keys_and_values_outside_leave_no_trace():
    """NaN and infinity in the rows behind ctx, in blocks of nobody and in the q rows of another
    sequence reach only what they belong to."""
    st = wl.make_step(8, 2, 128, 16, [130, 77, 200], [1, 40, 140], seed=6, num_blocks=40)
    for s, c in enumerate(st.ctx_lens):
        last = st.block_table[s][(c - 1) // 16]
        st.k_pool[last, (c - 1) % 16 + 1:] = 0x7FC0
    used = set(st.block_table[st.block_table >= 0].tolist())
    st.k_pool[[b for b in range(40) if b not in used]] = 0x7F80
    clean = st.k_pool.copy()
    _check_like(st, clean)


def _check_like(st, pool):
    shape = bd.Shape.make(st.Hq, st.Hkv, st.D, st.block_size, st.num_blocks)
    q = pa.bf16_to_f64(st.q)
    k = np.nan_to_num(pa.bf16_to_f64(pool), nan=0.0, posinf=0.0)
    lse, want = lse_and_weights(q, k, st.block_table, st.cu_seqlens_q, st.ctx_lens)
    qd = dev(st.q.view(np.int16), torch.bfloat16)
    for broken in (None, 1):                       # then sequence 1's q is NaN
        qb = qd.clone()
        if broken is not None:
            qb[int(st.cu_seqlens_q[1]):int(st.cu_seqlens_q[2])] = float("nan")
        w = torch.zeros(3, st.Hkv, 256, device="cuda")
        bd.paged_attention_weights(qb, dev(pool.view(np.int16), torch.bfloat16), dev(lse.astype(np.float32)),
                                   dev(st.block_table), dev(st.cu_seqlens_q), dev(st.ctx_lens), None, w, shape)
        got = w.cpu().numpy()
        for s, c in enumerate(st.ctx_lens):
            if s == broken:
                continue
            np.testing.assert_allclose(got[s, :, :c], want[s], rtol=1e-4, atol=1e-9)
            assert not got[s, :, c:].any()


@pytest.mark.gpu
def test_bad_metadata_is_skipped_and_flagged():
    st = wl.make_step(4, 2, 64, 16, [40, 50, 60], [1, 1, 1], seed=8)
    shape = bd.Shape.make(st.Hq, st.Hkv, st.D, st.block_size, st.num_blocks)
    q, kp = dev(st.q.view(np.int16), torch.bfloat16), dev(st.k_pool.view(np.int16), torch.bfloat16)
    lse = torch.zeros(3, 4, device="cuda")

    def run(cu=st.cu_seqlens_q, ctx=st.ctx_lens, table=st.block_table, rows=None, held=None, max_len=64):
        w = torch.full((3, 2, max_len), -1.0, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        i = lambda a: None if a is None else dev(np.asarray(a, np.int32))
        bd.paged_attention_weights(q, kp, lse, i(table), i(cu), i(ctx), i(rows), w, shape, held=i(held), err=err)
        w = w.cpu().numpy()
        return [bool((w[s] != -1).any()) for s in range(3)], int(err.item())

    assert run() == ([True] * 3, 0)
    assert run(ctx=[40, 65, 60]) == ([True, False, True], bd.PA_DEVERR_META)        # behind max_len
    assert run(ctx=[40, 0, 60]) == ([True, False, True], bd.PA_DEVERR_META)         # n_q > ctx
    assert run(ctx=[40, 50, 70], max_len=128) == ([True, True, False], bd.PA_DEVERR_META)  # behind the table
    assert run(cu=[0, 1, 2, 9]) == ([True, True, False], bd.PA_DEVERR_META)         # behind T
    assert run(rows=[0, 3, 2]) == ([True, False, True], bd.PA_DEVERR_META)
    assert run(rows=[1, 2, 2]) == ([False, True, False], bd.PA_DEVERR_META)         # one row twice
    assert run(rows=[0, -5, 2]) == ([True, False, True], 0)
    assert run(held=[40, 51, -1]) == ([True, False, False], bd.PA_DEVERR_META)
    table = st.block_table.copy()
    table[1, 0] = st.num_blocks
    assert run(table=table) == ([True] * 3, bd.PA_DEVERR_BLOCK)
    table[1, 0] = -1
    assert run(table=table) == ([True] * 3, bd.PA_DEVERR_BLOCK)


@pytest.mark.gpu
def test_streams_and_a_graph_that_follows_its_metadata():
    st = wl.make_step(8, 2, 128, 16, [300, 77], [1, 30], seed=11)
    shape = bd.Shape.make(st.Hq, st.Hkv, st.D, st.block_size, st.num_blocks)
    q, kp = dev(st.q.view(np.int16), torch.bfloat16), dev(st.k_pool.view(np.int16), torch.bfloat16)
    lse = torch.full((31, 8), 5.0, device="cuda")
    table, cu, ctx = dev(st.block_table), dev(st.cu_seqlens_q), dev(st.ctx_lens)
    rows = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    w = torch.zeros(2, 2, 320, device="cuda")
    run = lambda **kw: bd.paged_attention_weights(q, kp, lse, table, cu, ctx, rows, w, shape, **kw)
    run()
    want = w.clone()
    torch.cuda.synchronize()
    w.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run(stream=side)
    side.synchronize()
    assert torch.equal(w, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    w.zero_()
    graph.replay()
    assert torch.equal(w, want)
    # the same graph on other lengths
    ctx.copy_(torch.tensor([123, 64], dtype=torch.int32))
    w.zero_()
    run()
    torch.cuda.synchronize()
    direct = w.clone()
    w.zero_()
    graph.replay()
    assert torch.equal(w, direct) and not torch.equal(direct, want)


# ------------------------------------------------------------------ the step that keeps them (GPU)

def _step_case(st, fp8=False, shared=False, seed=0):
    """paged_attention_step_lse and _weights of a step: outputs with the plain step's bits, the
    definition's log-sum-exps and weights."""
    rng = np.random.default_rng(seed)
    B, g = len(st.ctx_lens), st.Hq // st.Hkv
    shape = bd.Shape.make(st.Hq, st.Hkv, st.D, st.block_size, st.num_blocks)
    q = pa.bf16_to_f64(st.q)
    scales = (0.0125, 0.02) if fp8 else ()
    if fp8:
        codes = ofp8.quantize(st.k_pool, scales[0])
        k, kp, vp = ofp8.dequantize(codes, scales[0]), dev(codes), dev(ofp8.quantize(st.v_pool, scales[1]))
    else:
        k = pa.bf16_to_f64(st.k_pool)
        kp, vp = (dev(x.view(np.int16), torch.bfloat16) for x in (st.k_pool, st.v_pool))
    plan = bd.pa_plan_step_shared(shape, st.cu_seqlens_q, st.ctx_lens, st.block_table) if shared else \
        bd.pa_plan_step(shape, st.cu_seqlens_q, st.ctx_lens)
    items = dev(plan.view(np.int32).reshape(-1))
    max_ctx = int(st.ctx_lens.max())
    qd, table, cu, ctx = dev(st.q.view(np.int16), torch.bfloat16), dev(st.block_table), dev(st.cu_seqlens_q), dev(st.ctx_lens)
    nan = lambda *s, dtype=torch.float32: torch.full(s, float("nan"), dtype=dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = nan(bd.pa_workspace_bytes(shape, st.T, max_ctx) // 4 + 1)
    want_out, out, out2 = (nan(st.T, st.Hq, st.D, dtype=torch.bfloat16) for _ in range(3))
    pre = (qd, kp, vp, table, cu, ctx, max_ctx, items, *scales)
    s8 = "_fp8" if fp8 else ""
    getattr(bd, "paged_attention_step" + s8)(*pre, ws, want_out, shape, err)
    lse = nan(st.T, st.Hq)
    getattr(bd, "paged_attention_step" + s8 + "_lse")(*pre, ws, out, lse, shape, err)
    want_lse, want = lse_and_weights(q, k, st.block_table, st.cu_seqlens_q, st.ctx_lens)
    got_lse = lse.cpu().numpy()
    tol = tolerance(q, k, st.D, want_lse, st.T * g) + 16 * 2.0 ** -24
    # the sum's relative error is the logarithm's absolute one; then two roundings of lse's size
    assert np.all(np.abs(got_lse - want_lse) <= tol + 2.0 ** -22 * np.maximum(np.abs(want_lse), 1))
    bits = lambda t: t.view(torch.int16)
    assert torch.equal(bits(out), bits(want_out))
    rows = rng.permutation(B + 2)[:B].astype(np.int32)
    start = rng.random((B + 2, st.Hkv, max_ctx + 5)).astype(np.float32)
    w = dev(start.copy())
    ws2 = nan((bd.pa_step_weights_workspace_bytes(shape, B, st.T, max_ctx) + 3) // 4)
    lse2 = nan(st.T, st.Hq)
    step = lambda: getattr(bd, "paged_attention_step_weights" + s8)(*pre, ws2, out2, lse2, dev(rows), w, shape, err=err)
    step()
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert torch.equal(bits(out2), bits(want_out)) and torch.equal(lse2, lse)
    got = w.cpu().numpy()
    expect = start.astype(np.float64)
    for s in range(B):
        n, c, r = int(st.n_q[s]), int(st.ctx_lens[s]), rows[s]
        if n == 0:
            continue
        expect[r, :, c - n:c] = 0
        expect[r, :, :c] += want[s]
        d = np.abs(got[r, :, :c] - expect[r, :, :c])
        # the kernel's own lse stands in: its error is the weights' as well
        assert np.all(d <= 3 * tol * want[s] + 2.0 ** -24 * expect[r, :, :c] + 1e-37), s
        expect[r, :, :c] = got[r, :, :c]
    assert np.array_equal(got, expect.astype(np.float32))
    # against paged_attention_weights from the same log-sum-exps
    w2 = dev(start.copy())
    getattr(bd, "paged_attention_weights" + s8)(qd, kp, lse, table, cu, ctx, dev(rows), w2, *scales[:1], shape)
    np.testing.assert_allclose(w2.cpu().numpy(), got, rtol=1e-5, atol=1e-7)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq, Hkv, D, bs", SHAPES)
@pytest.mark.parametrize("ctx, n_q", [
    ([1], [1]), ([17, 128, 64, 100], [1, 1, 1, 1]), ([2049, 2048, 4500], [1, 1, 1]),
    ([140, 300, 2100], [140, 257, 33]), ([700, 20, 129, 64, 2500], [130, 1, 129, 0, 1]),
])
def test_step_against_the_definition(Hq, Hkv, D, bs, ctx, n_q):
    _step_case(wl.make_step(Hq, Hkv, D, bs, ctx, n_q, seed=len(ctx) + D))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq, Hkv, bs", [(32, 8, 16), (8, 8, 32), (16, 1, 128)])
@pytest.mark.parametrize("ctx, n_q", [([17, 128, 64, 3000], [1, 1, 1, 1]), ([700, 20, 2129], [130, 1, 129])])
def test_fp8_step_against_the_definition(Hq, Hkv, bs, ctx, n_q):
    _step_case(wl.make_step(Hq, Hkv, 128, bs, ctx, n_q, seed=5), fp8=True)


@pytest.mark.gpu
def test_step_with_shared_prefixes():
    """Rows of GROUP and RESUME items keep their scores as well (each under its own sequence)."""
    for Hq, D in ((8, 64), (32, 128)):
        _step_case(wl.make_prefix_step(Hq, 8, D, 16, prompts=2, samples=5, prompt_tokens=640, cont_max=900, seed=2),
                   shared=True)
    _step_case(wl.make_prefix_step(32, 8, 128, 16, prompts=2, samples=3, prompt_tokens=640, cont_max=2500, seed=3),
               fp8=True, shared=True)


@pytest.mark.gpu
def test_step_refusals_and_contexts_behind_the_bound():
    st = wl.make_step(4, 2, 64, 16, [40, 150, 60], [1, 1, 1], seed=8)
    shape = bd.Shape.make(st.Hq, st.Hkv, st.D, st.block_size, st.num_blocks)
    q, kp, vp = (dev(x.view(np.int16), torch.bfloat16) for x in (st.q, st.k_pool, st.v_pool))
    items = dev(bd.pa_plan_step(shape, st.cu_seqlens_q, st.ctx_lens).view(np.int32).reshape(-1))
    out, lse = torch.empty(3, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 4, device="cuda")
    need = bd.pa_step_weights_workspace_bytes(shape, 3, 3, 160) // 4

    def run(max_ctx=160, ws=need, max_len=160, rows=(0, 1, 2), n=3):
        w = torch.full((n, 2, max_len), -1.0, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        bd.paged_attention_step_weights(q, kp, vp, dev(st.block_table), dev(st.cu_seqlens_q), dev(st.ctx_lens), max_ctx,
                                        items, None if ws is None else torch.empty(ws, device="cuda"), out, lse,
                                        torch.tensor(rows, dtype=torch.int32, device="cuda"), w, shape, err=err)
        return [bool((w[s] != -1).any()) for s in range(n)], int(err.item())

    assert run() == ([True] * 3, 0)
    for bad in (dict(ws=None), dict(ws=need - 1), dict(max_ctx=0)):
        with pytest.raises(bd.PagedAttnError):
            run(**bad)
    # sequence 1 is longer than the bound the caller gave: its scores have no room, it adds nothing
    assert run(max_ctx=100) == ([True, False, True], bd.PA_DEVERR_META)
    assert run(max_ctx=149) == ([True, False, True], bd.PA_DEVERR_META)   # one key, within the same tile
    assert run(max_ctx=150) == ([True] * 3, 0)
    assert run(max_len=100) == ([True, False, True], bd.PA_DEVERR_META)
    assert run(rows=(0, 2, 2)) == ([True, False, False], bd.PA_DEVERR_META)
    assert run(rows=(0, -1, 2)) == ([True, False, True], 0)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ctx, max_ctx", [(2200, 2048), (2200, 2199), (400, 399)])
def test_step_chunk_behind_the_bound_takes_no_part(ctx, max_ctx, fp8):
    """A chunk longer than max_ctx: rows that reach a split behind the bound are refused by the step and
    have no log-sum-exp (here NaN is left in the buffer). Its state row stays as it was."""
    st = wl.make_step(8, 2, 128, 16, [40, ctx, 60], [1, 300, 20], seed=8)
    shape = bd.Shape.make(st.Hq, st.Hkv, st.D, st.block_size, st.num_blocks)
    scales, s8 = ((0.0125, 0.02), "_fp8") if fp8 else ((), "")
    pools = [dev(ofp8.quantize(x, s)) for x, s in zip((st.k_pool, st.v_pool), scales)] if fp8 else \
        [dev(x.view(np.int16), torch.bfloat16) for x in (st.k_pool, st.v_pool)]
    q, table, cu, lens = dev(st.q.view(np.int16), torch.bfloat16), dev(st.block_table), dev(st.cu_seqlens_q), dev(st.ctx_lens)
    items = dev(bd.pa_plan_step(shape, st.cu_seqlens_q, st.ctx_lens).view(np.int32).reshape(-1))
    step = getattr(bd, "paged_attention_step_weights" + s8)

    def run(bound):
        ws = torch.empty((bd.pa_step_weights_workspace_bytes(shape, 3, st.T, bound) + 3) // 4, device="cuda")
        out = torch.empty(st.T, st.Hq, st.D, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((st.T, st.Hq), float("nan"), device="cuda")
        w = torch.full((3, st.Hkv, ctx + 9), 0.25, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        step(q, *pools, table, cu, lens, bound, items, *scales, ws, out, lse, None, w, shape, err=err)
        return w, int(err.item())

    want, err = run(ctx)
    assert err == 0 and bool((want[1] != 0.25).any()) and bool(torch.isfinite(want).all())
    got, err = run(max_ctx)
    assert err == bd.PA_DEVERR_META
    assert bool((got[1] == 0.25).all())
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


# A state much larger than what a step adds: the bound is one rounding of the total (half a step,
# 2^-24 of it at most) on top of the increment's own tolerance. The starting states are such that a
# part of the increment (a head's weight) is below half a step of theirs.
def _large_state(st, start, step, fp8=False):
    shape = bd.Shape.make(st.Hq, st.Hkv, st.D, st.block_size, st.num_blocks)
    q = pa.bf16_to_f64(st.q)
    scales, s8 = ((0.0125, 0.02), "_fp8") if fp8 else ((), "")
    if fp8:
        k = ofp8.dequantize(ofp8.quantize(st.k_pool, scales[0]), scales[0])
        kp, vp = (dev(ofp8.quantize(x, s)) for x, s in zip((st.k_pool, st.v_pool), scales))
    else:
        k = pa.bf16_to_f64(st.k_pool)
        kp, vp = (dev(x.view(np.int16), torch.bfloat16) for x in (st.k_pool, st.v_pool))
    lse64, want = lse_and_weights(q, k, st.block_table, st.cu_seqlens_q, st.ctx_lens)
    B, max_ctx = len(st.ctx_lens), int(st.ctx_lens.max())
    state = (start * (1 + np.random.default_rng(1).random((B, st.Hkv, max_ctx)))).astype(np.float32)
    w, held, err = dev(state.copy()), dev(st.ctx_lens), torch.zeros(1, dtype=torch.int32, device="cuda")
    qd, table, cu, ctx = dev(st.q.view(np.int16), torch.bfloat16), dev(st.block_table), dev(st.cu_seqlens_q), dev(st.ctx_lens)
    if step:
        items = dev(bd.pa_plan_step(shape, st.cu_seqlens_q, st.ctx_lens).view(np.int32).reshape(-1))
        ws = torch.empty((bd.pa_step_weights_workspace_bytes(shape, B, st.T, max_ctx) + 3) // 4, device="cuda")
        out = torch.empty(st.T, st.Hq, st.D, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(st.T, st.Hq, device="cuda")
        getattr(bd, "paged_attention_step_weights" + s8)(qd, kp, vp, table, cu, ctx, max_ctx, items, *scales, ws, out,
                                                         lse, None, w, shape, held=held, err=err)
    else:
        getattr(bd, "paged_attention_weights" + s8)(qd, kp, dev(lse64.astype(np.float32)), table, cu, ctx, None, w,
                                                    *scales[:1], shape, held=held, err=err)
    got = w.cpu().numpy()
    assert int(err.item()) == 0
    tol = 3 * (tolerance(q, k, st.D, lse64, st.T * st.Hq // st.Hkv) + 16 * 2.0 ** -24)
    for s in range(B):
        c = int(st.ctx_lens[s])
        total = state[s, :, :c].astype(np.float64) + want[s]
        d = np.abs(got[s, :, :c] - total)
        assert np.all(d <= tol * want[s] + 2.0 ** -24 * total), (s, float((d / (2.0 ** -24 * total)).max()))
        assert np.array_equal(got[s, :, c:], state[s, :, c:])


@pytest.mark.gpu
@pytest.mark.parametrize("step", [True, False])
@pytest.mark.parametrize("Hq, Hkv, D, fp8", [(16, 1, 128, False), (16, 2, 64, False), (32, 2, 128, True)])
def test_decode_rows_into_a_large_state_round_once(Hq, Hkv, D, fp8, step):
    _large_state(wl.make_step(Hq, Hkv, D, 16, [300, 2100, 129], [1, 1, 1], seed=3), 1e5, step, fp8)


@pytest.mark.gpu
@pytest.mark.parametrize("step", [True, False])
@pytest.mark.parametrize("seqs", [1, 5, 14])
def test_chunks_into_a_large_state_round_once(seqs, step):
    """Four query tiles to a chunk, its key tiles dealt one, two and up to four to an item: the step's
    weights are added up before the old sum joins them."""
    ctx = [1000 - 37 * s for s in range(seqs)]
    _large_state(wl.make_step(64, 8, 64, 16, ctx, [60] * seqs, seed=seqs), 5e6, step)


@pytest.mark.gpu
def test_fp8_chunks_into_a_large_state_round_once():
    _large_state(wl.make_step(64, 8, 128, 16, [1000, 700, 300], [60, 100, 17], seed=2), 5e6, True, fp8=True)


@pytest.mark.gpu
@pytest.mark.parametrize("chunks", [False, True])
def test_rows_named_twice_among_thousands(chunks):
    """Those that share a state row drop out, wherever they lie in the deal; the others are as without
    them, and the call stays one of microseconds."""
    B, Hkv = 6001, 2
    rng = np.random.default_rng(B)
    ctx = rng.integers(1, 60, B)
    n_q = np.minimum(ctx, rng.integers(0, 50, B)) if chunks else np.ones(B, int)
    st = wl.make_step(8, Hkv, 64, 8, ctx, n_q, seed=9)
    shape = bd.Shape.make(st.Hq, st.Hkv, st.D, st.block_size, st.num_blocks)
    q, kp = dev(st.q.view(np.int16), torch.bfloat16), dev(st.k_pool.view(np.int16), torch.bfloat16)
    lse = torch.full((st.T, st.Hq), 3.0, device="cuda")
    table, cu, lens = dev(st.block_table), dev(st.cu_seqlens_q), dev(st.ctx_lens)
    plain = rng.permutation(B + 40)[:B].astype(np.int32)
    start = torch.rand(B + 40, Hkv, 64, device="cuda")

    def run(rows):
        w, err, r = start.clone(), torch.zeros(1, dtype=torch.int32, device="cuda"), dev(rows)
        call = lambda: bd.paged_attention_weights(q, kp, lse, table, cu, lens, r, w, shape, err=err)
        call()
        got = w.clone(), int(err.item())
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        times = []
        for _ in range(3):
            a.record()
            call()
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return *got, min(times)

    whole, err, t_plain = run(plain)
    assert err == 0
    active = np.flatnonzero(n_q > 0)
    rows = plain.copy()
    groups = [active[[3, -2]], active[[1000, 1001, 4000]], active[[0, 2500]]]
    out = set()
    for g in groups:
        rows[g] = plain[g[0]]
        out |= set(g.tolist())
    idle = np.flatnonzero(n_q == 0)
    if len(idle):
        rows[idle[0]] = plain[active[70]]           # a sequence without query rows shares nothing
    got, err, t = run(rows)
    assert err == bd.PA_DEVERR_META
    want = start.clone()
    live = torch.from_numpy(plain[[s for s in active.tolist() if s not in out]].astype(np.int64)).cuda()
    want[live] = whole[live]
    assert torch.equal(got, want)
    assert t < 3 * t_plain + 0.3, (t, t_plain)      # milliseconds; a scan of all pairs takes tens of them


@pytest.mark.gpu
def test_step_of_a_decode_row_and_a_chunk_that_name_one_state_row():
    """Decode rows and chunks are summed by different kernels: both drop out, whichever else is there."""
    st = wl.make_step(8, 2, 64, 16, [40, 350, 60, 500, 90], [1, 300, 1, 120, 7], seed=8)
    shape = bd.Shape.make(st.Hq, st.Hkv, st.D, st.block_size, st.num_blocks)
    q, kp, vp = (dev(x.view(np.int16), torch.bfloat16) for x in (st.q, st.k_pool, st.v_pool))
    items = dev(bd.pa_plan_step(shape, st.cu_seqlens_q, st.ctx_lens).view(np.int32).reshape(-1))
    out, lse = torch.empty(st.T, 8, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(st.T, 8, device="cuda")
    ws = torch.empty(bd.pa_step_weights_workspace_bytes(shape, 5, st.T, 500) // 4, device="cuda")

    def run(rows):
        w, err = torch.full((6, 2, 512), 0.5, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        bd.paged_attention_step_weights(q, kp, vp, dev(st.block_table), dev(st.cu_seqlens_q), dev(st.ctx_lens), 500, items,
                                        ws, out, lse, dev(np.asarray(rows, np.int32)), w, shape, err=err)
        return w, int(err.item())

    want, err = run([0, 1, 2, 3, 4])
    assert err == 0
    for rows, alone in (([0, 0, 2, 3, 4], [2, 3, 4]), ([0, 1, 2, 2, 2], [0, 1]), ([5, 1, 2, 1, 5], [2])):
        got, err = run(rows)
        assert err == bd.PA_DEVERR_META
        for r in range(6):
            assert torch.equal(got[r], want[r]) if r in alone else bool((got[r] == 0.5).all()), (rows, r)
