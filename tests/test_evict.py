"""Eviction by accumulated attention weight: pins of the definition and refusals (CPU), and the
kernel against the definition (GPU). Everything here is equal to the bit: entries move, nothing is
computed."""
import math

import numpy as np
import pytest

from continuous_batching_gb300 import binding as bd
from oracle.bounded import evict

torch = pytest.importorskip("torch")


# ------------------------------------------------------------------ the definition (CPU)

def test_definition_on_small_cases():
    pos = np.arange(8)
    w = np.array([5.0, 1, 7, 7, 2, 9, 0, 3])
    # budget 4, nothing protected: 9, 7, 7, 5 stay: 0, 2, 3 in place, 5 into the hole at 1
    assert evict(w, pos, 8, 4, 0, 0).tolist() == [0, 5, 2, 3]
    # ties go to the lower index
    assert evict(np.ones(6), np.arange(6), 6, 3, 0, 0).tolist() == [0, 1, 2]
    # the last two tokens and the first are protected
    assert evict(w, pos, 8, 4, 2, 1).tolist() == [0, 5, 6, 7]
    # positions, not places, are protected
    assert evict(w, pos[::-1], 8, 4, 2, 0).tolist() == [0, 1, 2, 5]
    # more protected than the budget: the lower indices
    assert evict(w, pos, 8, 3, 8, 0).tolist() == [0, 1, 2]
    assert evict(w, pos, 8, 9, 1, 1).tolist() == list(range(8))
    assert evict(np.array([1.0, math.nan, math.inf, 2]), np.arange(4), 4, 2, 0, 0).tolist() == [2, 1]


def _call(**kw):
    a = dict(kp=16, vp=16, eb=2, tb=16, mb=4, ctx=16, bu=16, nt=16, kept=None, rows=16, B=2, recent=1,
             sink=0, w=16, wo=16, p=16, po=16, n=4, m=64)
    shape = kw.pop("shape", bd.Shape.make(4, 2, 128, 16, 8))
    a.update(kw)
    return bd.load().paged_evict(*[a[k] for k in ("kp", "vp", "eb", "tb", "mb", "ctx", "bu", "nt", "kept", "rows",
                                                  "B", "recent", "sink", "w", "wo", "p", "po", "n", "m")],
                                 shape, None, None)


@pytest.mark.parametrize("kw, want", [
    (dict(B=0), bd.PA_OK), (dict(B=-1), bd.PA_ERR_INVALID), (dict(eb=4), bd.PA_ERR_SHAPE),
    (dict(recent=-1), bd.PA_ERR_INVALID), (dict(sink=-1), bd.PA_ERR_INVALID),
    (dict(kp=None), bd.PA_ERR_INVALID), (dict(w=None), bd.PA_ERR_INVALID), (dict(po=None), bd.PA_ERR_INVALID),
    (dict(bu=None), bd.PA_ERR_INVALID), (dict(nt=None), bd.PA_ERR_INVALID), (dict(m=0), bd.PA_ERR_INVALID),
    (dict(rows=None, n=1), bd.PA_ERR_INVALID), (dict(m=(1 << 19) + 1), bd.PA_ERR_SHAPE),
    (dict(B=65536), bd.PA_ERR_SHAPE), (dict(kp=8), bd.PA_ERR_INVALID),
    (dict(wo=16 + 4 * 64), bd.PA_ERR_INVALID), (dict(po=16 + 4), bd.PA_ERR_INVALID),   # half over itself
    (dict(shape=bd.Shape.make(4, 2, 128, 12, 8)), bd.PA_ERR_SHAPE),
])
def test_refusals(kw, want):
    assert _call(**kw) == want


# ------------------------------------------------------------------ the kernel (GPU)

def _run(ctx, budget, Hkv=2, D=64, bs=16, fp8=False, recent=3, sink=1, kept=None, seed=0, in_place=False,
         weights=None, max_len=None, extra_rows=2, rows=True, want_err=0):
    rng = np.random.default_rng(seed)
    B = len(ctx)
    ctx = np.asarray(ctx, np.int32)
    budget = np.broadcast_to(np.asarray(budget, np.int32), (B,)).copy()
    kept = np.zeros(B, np.int32) if kept is None else np.asarray(kept, np.int32)
    n_tokens = (ctx + 2 * kept).astype(np.int32)
    nblk = -(-ctx // bs)
    nb = int(nblk.sum()) + 3
    perm = rng.permutation(nb)
    table = np.full((B, max(int(nblk.max()), 1) + 1), -1, np.int32)
    at = 0
    for s in range(B):
        table[s, :nblk[s]] = perm[at:at + nblk[s]]
        at += nblk[s]
    max_len = int(ctx.max()) + 7 if max_len is None else max_len
    n_rows = B + extra_rows
    order = rng.permutation(n_rows)[:B].astype(np.int32) if rows else np.arange(B, dtype=np.int32)
    w = rng.lognormal(0, 2, (n_rows, Hkv, max_len)).astype(np.float32) if weights is None else \
        weights(rng, (n_rows, Hkv, max_len)).astype(np.float32)
    pos = np.stack([[rng.permutation(4 * max_len)[:max_len] for _ in range(Hkv)] for _ in range(n_rows)]).astype(np.int32)
    for s in range(B):                                    # kept entries: distinct tokens before the new ones
        for h in range(Hkv):
            pos[order[s], h, :kept[s]] = rng.permutation(int(n_tokens[s] - ctx[s] + kept[s]))[:kept[s]]
    e, np_e = (torch.uint8, np.uint8) if fp8 else (torch.int16, np.int16)
    pools = [rng.integers(0, 120, (nb, bs, Hkv, D)).astype(np_e) for _ in "kv"]
    d = lambda a: torch.from_numpy(a.copy()).cuda()
    kp, vp = (d(x) if fp8 else d(x).view(torch.bfloat16) for x in pools)
    wi, pi = d(w), d(pos)
    wo = wi if in_place else torch.full_like(wi, -5.0)
    po = pi if in_place else torch.full_like(pi, -5)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    shape = bd.Shape.make(Hkv, Hkv, D, bs, nb)
    bd.paged_evict(kp, vp, d(table), d(ctx), d(budget), d(n_tokens), d(kept) if kept.any() else None,
                   d(order) if rows else None, recent, sink, wi, wo, pi, po, shape, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == want_err
    flat = [x.reshape(nb * bs, Hkv, D) for x in pools]
    want = [f.copy() for f in flat]
    ww = w.copy() if in_place else np.full_like(w, -5.0)
    wp = pos.copy() if in_place else np.full_like(pos, -5)
    moved = 0
    for s in range(B):
        slot = [int(table[s][j // bs]) * bs + j % bs for j in range(int(ctx[s]))]
        for h in range(Hkv):
            r = order[s]
            j = np.arange(ctx[s])
            p = np.where(j < kept[s], pos[r, h, :ctx[s]], n_tokens[s] - ctx[s] + j)
            src = evict(w[r, h, :ctx[s]].astype(np.float64), p, int(n_tokens[s]), int(budget[s]), recent, sink)
            for i, f in enumerate(src):
                if f != i:
                    moved += 1
                    for a, b in zip(want, flat):
                        a[slot[i], h] = b[slot[f], h]
            ww[r, h, :len(src)] = w[r, h, src]
            wp[r, h, :len(src)] = p[src]
    got = [(x if fp8 else x.view(torch.int16)).cpu().numpy().reshape(nb * bs, Hkv, D) for x in (kp, vp)]
    np.testing.assert_array_equal(po.cpu().numpy(), wp)
    np.testing.assert_array_equal(wo.cpu().numpy().view(np.int32), ww.view(np.int32))
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    return moved


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("ctx, budget", [
    ([1], 1), ([1, 2, 3], 1), ([33, 32, 31, 64, 65], 32), ([40, 10, 100], [20, 10, 200]),
    ([257, 300, 129], 128), ([2049, 2049], 2048), ([5000, 1025], 1000), ([9000], 4097),
])
def test_against_the_definition(ctx, budget, in_place):
    _run(ctx, budget, in_place=in_place, seed=len(ctx))


@pytest.mark.gpu
@pytest.mark.parametrize("Hkv, D, bs, fp8", [(1, 64, 8, False), (8, 128, 16, False), (3, 128, 128, True),
                                             (2, 64, 32, True), (8, 128, 64, True)])
def test_layouts(Hkv, D, bs, fp8):
    _run([700, 130, 1500], 128, Hkv=Hkv, D=D, bs=bs, fp8=fp8, recent=40, sink=4, seed=D)
    _run([129, 129, 129, 129], 128, Hkv=Hkv, D=D, bs=bs, fp8=fp8, recent=16, sink=4, kept=[128] * 4, in_place=True)


@pytest.mark.gpu
@pytest.mark.parametrize("max_len, C", [(900, 1), (2048, 2), (4100, 4), (20000, 8), (100000, 8), (300000, 8)])
def test_cluster_sizes_and_long_slices(max_len, C):
    """Every cluster size, slices that are held in shared memory and longer ones."""
    assert _run([min(max_len, 70000)], 500, Hkv=1, recent=100, max_len=max_len, extra_rows=0, seed=C) > 0
    _run([min(max_len, 3000), 600], [599, 600], Hkv=1, max_len=max_len, extra_rows=0, seed=C)


@pytest.mark.gpu
def test_ties_zeros_negative_and_non_finite_weights():
    some = lambda rng, shape: rng.choice([0.0, -0.0, 1.0, 1.0, 2.0, -3.0, np.inf, -np.inf, np.nan, 1e-40], shape)
    for n in ([300, 77], [4000]):
        _run(n, 50, weights=some, recent=5, seed=len(n))
    _run([3000, 3000], 1500, weights=lambda rng, shape: np.ones(shape), recent=0, sink=0)
    _run([3000, 3000], 1500, weights=lambda rng, shape: np.zeros(shape), recent=700, sink=4)


@pytest.mark.gpu
def test_protection():
    _run([600, 600], 100, recent=100, sink=0)             # all that stays is recent
    _run([600, 600], 100, recent=300, sink=8)             # more protected than the budget holds
    _run([600], 100, recent=1 << 30, sink=1 << 30)        # everything is
    _run([400, 300], 120, recent=30, sink=4, kept=[120, 300], in_place=True)
    _run([400, 300], 120, recent=30, sink=4, kept=[350, 120], in_place=True)   # a budget that was lowered
    _run([60, 70], 120, recent=30, sink=4, kept=[50, 0])  # nothing to evict: positions are filled in
    _run([60, 70], 120, rows=False, extra_rows=0, in_place=True)


@pytest.mark.gpu
def test_many_sequences():
    rng = np.random.default_rng(1)
    _run(rng.integers(1, 260, 700), rng.integers(1, 200, 700), Hkv=2, bs=8, seed=3)


@pytest.mark.gpu
def test_bad_metadata_is_skipped_and_flagged():
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    shape = bd.Shape.make(2, 2, 64, 16, 8)

    def run(table=((0, 1), (2, 3)), ctx=(30, 30), budget=(10, 10), n=(30, 30), kept=(0, 0), rows=(0, 1), max_len=32):
        kp = torch.randint(0, 99, (8, 16, 2, 64), device="cuda").to(torch.bfloat16)
        vp, before = kp.clone(), kp.clone()
        w = torch.rand(2, 2, max_len, device="cuda") + torch.arange(max_len, device="cuda")
        p = torch.zeros(2, 2, max_len, dtype=torch.int32, device="cuda")
        wo, po = torch.full_like(w, -1), torch.full_like(p, -1)
        err = i([0])
        bd.paged_evict(kp, vp, i(table), i(ctx), i(budget), i(n), i(kept), i(rows), 2, 0, w, wo, p, po, shape, err=err)
        done = [bool((wo[r] != -1).any()) for r in range(2)]
        moved = [bool((kp[b] != before[b]).any()) for b in (0, 2)]
        return done, moved, int(err.item())

    both, none = [True, True], [False, False]
    assert run() == (both, both, 0)
    for bad in (dict(ctx=(30, 33)), dict(ctx=(30, -1)), dict(budget=(10, 0)), dict(n=(30, 29)), dict(kept=(0, 31)),
                dict(kept=(0, -1)), dict(ctx=(30, 40), n=(30, 40), max_len=64), dict(rows=(0, 2))):
        assert run(**bad) == ([True, False], [True, False], bd.PA_DEVERR_META), bad
    assert run(rows=(1, 1)) == (none, none, bd.PA_DEVERR_META)
    assert run(rows=(0, -1)) == ([True, False], [True, False], 0)
    assert run(table=((0, 1), (2, 8))) == (both, [True, False], bd.PA_DEVERR_BLOCK)
    assert run(table=((0, 1), (2, -1))) == (both, [True, False], bd.PA_DEVERR_BLOCK)


@pytest.mark.gpu
def test_binding_refusals_streams_and_graphs():
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    shape = bd.Shape.make(2, 2, 64, 16, 8)
    kp0 = torch.randn(8, 16, 2, 64, device="cuda").to(torch.bfloat16)
    w = torch.rand(2, 2, 48, device="cuda")
    a = dict(kp=kp0.clone(), vp=kp0.clone(), table=i([[0, 1, 2], [3, 4, 5]]), ctx=i([40, 33]), budget=i([20, 20]),
             n=i([40, 33]), kept=None, rows=None, recent=4, sink=1, w=w, wo=torch.zeros_like(w),
             p=torch.zeros(2, 2, 48, dtype=torch.int32, device="cuda"),
             po=torch.zeros(2, 2, 48, dtype=torch.int32, device="cuda"), shape=shape)
    run = lambda stream=None, **kw: bd.paged_evict(*{**a, **kw}.values(), stream=stream)
    for bad in (dict(w=w.double()), dict(w=w[:, :1]), dict(wo=w[:1]), dict(p=a["p"].long()), dict(ctx=i([40])),
                dict(kp=kp0.half()), dict(vp=kp0.view(torch.uint8)), dict(table=a["table"].cpu()),
                dict(budget=i([20])), dict(po=a["po"].transpose(1, 2))):
        with pytest.raises(ValueError):
            run(**bad)
    run()
    torch.cuda.synchronize()
    want = a["kp"].clone(), a["wo"].clone(), a["po"].clone()
    state = lambda: (a["kp"], a["wo"], a["po"])

    def reset():
        a["kp"].copy_(kp0), a["vp"].copy_(kp0), a["wo"].zero_(), a["po"].zero_()
        torch.cuda.synchronize()

    reset()
    side = torch.cuda.Stream()
    run(stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(state(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    reset()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(state(), want))


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("ctx, budget, max_len", [(60, 20, 64), (3000, 1000, 3000)])
def test_an_entry_that_cannot_move_leaves_the_hole_its_own(ctx, budget, max_len, in_place):
    """Blocks outside the pool among the strays' and among the holes': K, V, weight and position of such a
    move stay together, in both places."""
    rng = np.random.default_rng(ctx)
    bs, Hkv, D = 16, 2, 64
    n = -(-ctx // bs)
    shape = bd.Shape.make(Hkv, Hkv, D, bs, n)
    table = rng.permutation(n).astype(np.int32)[None]
    bad = [0, n - 2, n // 2] if n > 10 else [0, n - 2]
    table[0, bad] = [n, -1, n + 5][:len(bad)]
    flat = [rng.integers(0, 120, (n * bs, Hkv, D)).astype(np.int16) for _ in "kv"]
    w = rng.lognormal(0, 2, (1, Hkv, max_len)).astype(np.float32)
    kept, n_tokens = ctx // 3, 2 * ctx
    pos = np.stack([[rng.permutation(n_tokens - ctx)[:max_len] if n_tokens - ctx >= max_len else
                     rng.permutation(max_len) for _ in range(Hkv)]]).astype(np.int32)
    d = lambda a: torch.from_numpy(a.copy()).cuda()
    kp, vp = (d(x.reshape(n, bs, Hkv, D)).view(torch.bfloat16) for x in flat)
    wi, pi = d(w), d(pos)
    wo, po = (wi, pi) if in_place else (torch.full_like(wi, -5), torch.full_like(pi, -5))
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    err = i(0)
    bd.paged_evict(kp, vp, d(table), i(ctx), i(budget), i(n_tokens), i(kept), None, 4, 1, wi, wo, pi, po, shape, err=err)
    assert int(err.item()) == bd.PA_DEVERR_BLOCK
    got_w, got_p = wo.cpu().numpy()[0], po.cpu().numpy()[0]
    got = [x.view(torch.int16).cpu().numpy().reshape(n * bs, Hkv, D) for x in (kp, vp)]
    want = [x.copy() for x in flat]
    slot = [int(table[0, j // bs]) * bs + j % bs if 0 <= table[0, j // bs] < n else -1 for j in range(ctx)]
    stayed = 0
    for h in range(Hkv):
        j = np.arange(ctx)
        p = np.where(j < kept, pos[0, h, :ctx], n_tokens - ctx + j)
        src = evict(w[0, h, :ctx].astype(np.float64), p, n_tokens, budget, 4, 1)
        for to, f in enumerate(src):
            if f == to:
                continue
            if slot[f] < 0 or slot[to] < 0:
                src[to] = to
                stayed += 1
            else:
                for a, b in zip(want, flat):
                    a[slot[to], h] = b[slot[f], h]
        np.testing.assert_array_equal(got_w[h, :budget], w[0, h, src])
        np.testing.assert_array_equal(got_p[h, :budget], p[src])
    assert stayed > 4
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
