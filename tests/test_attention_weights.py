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
    (dict(m=2 ** 31 - 1), bd.PA_ERR_SHAPE), (dict(q=24), bd.PA_ERR_INVALID),
    (dict(kp=8), bd.PA_ERR_INVALID), (dict(shape=bd.Shape.make(4, 2, 32, 16, 8)), bd.PA_ERR_SHAPE),
    (dict(shape=bd.Shape.make(6, 2, 128, 16, 8)), bd.PA_ERR_SHAPE),
    (dict(shape=bd.Shape.make(4, 2, 64, 16, 8), scale=1.0), bd.PA_ERR_SHAPE),
    (dict(scale=0.0), bd.PA_ERR_INVALID), (dict(scale=float("nan")), bd.PA_ERR_INVALID),
])
def test_refusals(kw, want):
    assert _call(**kw) == want


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
    assert run(rows=[0, 2, 2]) == ([False] * 3, bd.PA_DEVERR_META)                  # one row twice
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
