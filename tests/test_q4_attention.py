"""The attention step over a 4-bit cache: the plan and the refusals on the CPU; on the GPU its outputs
against the definition in 64 bits, bit for bit invariances, graphs, bad pages and metadata."""
import ctypes as C

import numpy as np
import pytest

import oracle.paged_attention as pa
import oracle.q4 as q4
from continuous_batching_gb300 import binding as bd
from continuous_batching_gb300 import workloads as wl

torch = pytest.importorskip("torch")


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bf16(bits):
    return dev(bits.view(np.int16)).view(torch.bfloat16)


def bits_of(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


class Case:
    """A step over pools whose unwritten bytes are NaN parameters: lens is [(rows, context)]."""

    def __init__(self, lens, Hq=8, Hkv=2, D=128, bs=16, seed=0, spare=2, offset=0.0):
        rng = np.random.default_rng(seed)
        self.lens, self.Hq, self.Hkv, self.D, self.bs = lens, Hq, Hkv, D, bs
        ctx = np.array([c for _, c in lens], np.int32)
        self.ctx, self.cu = ctx, np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)
        need = [-(-int(c) // bs) for c in ctx]
        self.nb = sum(need) + spare
        self.table = np.full((len(lens), max(max(need), 1) + 1), -1, np.int32)
        order = rng.permutation(self.nb)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n
        self.shape = bd.Shape.make(Hq, Hkv, D, bs, self.nb)
        self.T = int(self.cu[-1])
        self.q = wl.random_bf16(rng, (self.T, Hq, D))
        self.pools = []
        for is_v in (False, True):
            pool = np.full((self.nb, Hkv, bs * (D // 2 + D // 8)), 0xFF, np.uint8)
            x = pa.bf16_to_f64(wl.random_bf16(rng, (int(ctx.sum()), Hkv, D)))
            x = wl.f32_to_bf16_bits((x + offset * rng.standard_normal((1, Hkv, D))).astype(np.float32))
            slots = np.concatenate([self.table[s][np.arange(c) // bs] * bs + np.arange(c) % bs for s, c in enumerate(ctx) if c] or [np.zeros(0, int)])
            self.pools.append(q4.write(pool, x, slots, bs, is_v))

    def rounded(self):
        """K and V as bf16 (what a step over expanded contexts computes on), NaN bytes as 0."""
        return [np.nan_to_num(pa.bf16_to_f64(q4._to_bf16_bits(q4.values(p, self.bs, self.D, i == 1)))) for i, p in enumerate(self.pools)]

    def exact(self, k=None, v=None):
        if k is None:
            k, v = (np.nan_to_num(q4.values(p, self.bs, self.D, i == 1).astype(np.float64)) for i, p in enumerate(self.pools))
        return pa.attention(pa.bf16_to_f64(self.q), k, v, self.table, self.cu, self.ctx, self.Hq)

    def bound(self):
        """How far an output of rows read from the codes may be off, per value. Three parts:
        the output's rounding, 2^-8 of it; the roundings of a term p (s (u - 8) + (m + 8 s)): p to two bf16
        (2^-8 of what the first leaves, 2^-16), the product of the second part and s (2^-8 of 2^-8), and to one bf16 the
        whole product p s (2^-8 of the first summand) or the centre m + 8 s (2^-8 of the second), so 2^-8 + 2^-15
        of p (|s (u - 8)| + |m + 8 s|); and what fp32 does to a score: products and sums of a group stay
        below 144 sum |q| (codes as 128 + u), of which 2^-20 covers the sums of 32 products and four groups at 2^-23
        each (a tensor core may truncate), times the scale. A score off by e moves a weight by exp(e) - 1, and so the
        result by at most that of twice the magnitudes (numerator and denominator)."""
        k, v = self.pools
        D, g = self.D, self.Hq // self.Hkv
        out = np.abs(self.exact()) * 2.0 ** -8
        q = pa.bf16_to_f64(self.q)
        mag = np.zeros((self.nb, self.bs, self.Hkv, D))
        ks = np.zeros((self.nb, self.bs, self.Hkv, D // 32))
        for b in range(self.nb):
            for h in range(self.Hkv):
                pv = v[b, h, self.bs * (D // 2):].view("<u2").reshape(self.bs, D // 32, 2)
                s, m = (np.nan_to_num(np.repeat(pa.bf16_to_f64(pv[..., i]), 32, -1)) for i in (0, 1))
                c = v[b, h, :self.bs * (D // 2)].reshape(self.bs, D // 2)
                u = np.stack([c & 15, c >> 4], -1).reshape(self.bs, D)[:, q4.column_nibble(D, True)].astype(float)
                mag[b, :, h] = s * np.abs(u - 8) + np.abs(m + 8 * s)
                ks[b, :, h] = np.nan_to_num(pa.bf16_to_f64(k[b, h, self.bs * (D // 2):].view("<u2").reshape(self.bs, D // 32, 2)[..., 0]))
        kv = np.nan_to_num(q4.values(k, self.bs, D, False).astype(np.float64))
        big = pa.attention(q, kv, mag, self.table, self.cu, self.ctx, self.Hq)
        e = np.abs(q).reshape(self.T, self.Hq, D // 32, 32).sum(-1) @ np.full(D // 32, ks.max()) * 144 * 2.0 ** -20 / np.sqrt(D)
        return out + (2.0 ** -8 + 2.0 ** -15 + 2 * np.expm1(2 * e)[..., None] + 2.0 ** -18) * big

    def plan(self, direct_rows=None, limits=None):
        return bd.pa_plan_step_q4(self.shape, self.cu, self.ctx, direct_rows, limits, device="cuda")

    def run(self, direct_rows=None, plan=None, pools=None, table=None, cu=None, ctx=None, expect=0):
        plan = plan or self.plan(direct_rows)
        ws = torch.empty(bd.pa_q4_workspace_bytes(self.shape, plan) // 4 + 1, device="cuda")
        ws.fill_(float("nan"))
        out = torch.full((self.T, self.Hq, self.D), 9.0, dtype=torch.bfloat16, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        k, v = pools or [dev(p) for p in self.pools]
        bd.paged_attention_step_q4(bf16(self.q), k, v, dev(self.table if table is None else table), dev(self.cu if cu is None else cu),
                                   dev(self.ctx if ctx is None else ctx), plan, ws, out, self.shape, err=err)
        assert int(err.item()) == expect
        return bits_of(out)

    def check_direct(self, direct_rows):
        got = pa.bf16_to_f64(self.run(direct_rows))
        far, most = np.abs(got - self.exact()), self.bound()
        assert np.isfinite(got).all() and (far <= most).all(), float((far / np.maximum(most, 1e-30)).max())


# ------------------------------------------------------------------------------------ plan

def _items(words, at, n):
    return words[at:at + n * bd.ITEM_INTS].view(bd.WORK_ITEM_DTYPE)


def _split(ctx):
    return 512 if ctx <= 6144 else 768 if ctx <= 12288 else 1024 if ctx <= 32768 else 2048


@pytest.mark.parametrize("direct_rows", [0, 8, 16, 64])
@pytest.mark.parametrize("Hq, Hkv", [(8, 8), (8, 2), (32, 2)])
def test_plan_covers_every_row_once(direct_rows, Hq, Hkv):
    rng = np.random.default_rng(direct_rows + Hq)
    n_q = rng.integers(0, 40, 30)
    n_q[:10] = 1
    ctx = np.maximum(n_q, rng.integers(1, 9000, 30)).astype(np.int32)
    ctx[3], ctx[4] = 33000, 0
    n_q[4] = 0
    cu = np.concatenate([[0], np.cumsum(n_q)]).astype(np.int32)
    shape = bd.Shape.make(Hq, Hkv, 128, 16, 4)
    g = Hq // Hkv
    exact = bd.pa_plan_step_q4(shape, cu, ctx, direct_rows)
    limits = bd.pa_q4_plan_limits(shape, 30, int(cu[-1]), 33000, direct_rows, 3000)
    for plan in (exact, bd.pa_plan_step_q4(shape, cu, ctx, limits=limits)):
        s, w = plan.sizes, plan.words
        direct = _items(w, 0, s.n_direct)
        at = s.n_direct * bd.ITEM_INTS
        first = w[at:at + 153] if s.n_direct else np.zeros(1, np.int32)
        at += 153 if s.n_direct else 0
        fold = w[at:at + s.n_fold]
        at += s.n_fold
        chunk = _items(w, at, s.n_chunk)
        at += s.n_chunk * bd.ITEM_INTS
        blocks = w[at:at + 2 * s.n_expand].reshape(-1, 2)
        table = w[at + 2 * s.n_expand:s.words].reshape(30 if s.n_chunk else 0, s.expand_cols)
        seen, places = {}, set()
        n_real = int((direct["n_q"] > 0).sum())
        assert first[0] == 0 and (np.diff(first) >= 0).all() and first[-1] == n_real and (direct[n_real:]["n_q"] == 0).all()
        cost = [int((direct["n_tiles"][a:b] + 1).sum()) for a, b in zip(first, first[1:])]
        # every item goes to the list of the least cost, so no two differ by more than an item's (here rounded up)
        assert not cost or max(cost) - min(cost) <= direct["n_tiles"].max() + 2
        for i in range(n_real):
            it = direct[i]
            q = int(it["seq"])
            keys = int(ctx[q] - cu[q + 1] + it["q_start"] + it["n_q"])
            assert n_q[q] * g <= direct_rows and it["kind"] == bd.PA_ITEM_DIRECT and it["n_q"] * g <= (16 if direct_rows > 8 else 8)
            assert it["n_splits"] == -(-keys // _split(ctx[q])) and 0 <= it["split"] < it["n_splits"]
            place = int(it["tile0"] + it["split"])
            assert place not in places and place < s.n_direct
            places.add(place)
            for t in range(it["q_start"], it["q_start"] + it["n_q"]):
                seen.setdefault((t, int(it["kv_head"])), []).append(int(it["split"]))
            assert (i in fold) == (it["split"] == 0 and it["n_splits"] > 1)
        wide = [q for q in range(30) if n_q[q] * g > direct_rows]
        for q in range(30):
            nb = -(-int(ctx[q]) // 128)
            if q in wide:
                mine = [i for i in range(len(blocks)) if blocks[i, 0] == q]
                assert blocks[mine, 1].tolist() == list(range(nb)) and table[q, :nb].tolist() == mine and (table[q, nb:] == -1).all()
            else:
                assert len(table) == 0 or (table[q] == -1).all()
                for t in range(cu[q], cu[q + 1]):
                    for h in range(Hkv):
                        assert len(seen[t, h]) == max(seen[t, h]) + 1 == len(set(seen[t, h]))
        assert {int(i["seq"]) for i in chunk if i["n_q"] > 0} == set(wide)


def test_plan_refuses():
    shape = bd.Shape.make(8, 2, 128, 16, 64)
    cu, ctx = np.array([0, 1, 31], np.int32), np.array([700, 90], np.int32)
    lim = lambda **kw: bd.pa_q4_plan_limits(shape, **{**dict(B=2, T=31, max_ctx=700, direct_rows=8, max_expand=2), **kw})
    bd.pa_plan_step_q4(shape, cu, ctx, limits=lim())
    for bad in (dict(B=3), dict(T=32), dict(max_ctx=699), dict(max_expand=0)):
        with pytest.raises(bd.PagedAttnError) as e:
            bd.pa_plan_step_q4(shape, cu, ctx, limits=lim(**bad))
        assert e.value.status == bd.PA_ERR_INVALID, bad
    for bad in (dict(B=-1), dict(T=-1), dict(direct_rows=-1), dict(max_expand=-1)):
        with pytest.raises(bd.PagedAttnError):
            lim(**bad)
    with pytest.raises(bd.PagedAttnError):
        bd.pa_plan_step_q4(shape, np.array([0, 1, 100], np.int32), ctx, 8)      # more rows than context
    s = lim()
    s.words += 1                                          # sizes that are not one plan's
    with pytest.raises(bd.PagedAttnError):
        bd.pa_plan_step_q4(shape, cu, ctx, limits=s)


@pytest.mark.parametrize("cu, ctx", [([0], []), ([0, 0], [0]), ([0, 0, 0], [5, 900])])
def test_plans_of_no_rows(cu, ctx):
    shape = bd.Shape.make(8, 2, 128, 16, 64)
    cu, ctx = np.array(cu, np.int32), np.array(ctx, np.int32)
    plan = bd.pa_plan_step_q4(shape, cu, ctx)
    assert plan.sizes.words == 0 and bd.pa_q4_workspace_bytes(shape, plan) == 0
    limits = bd.pa_q4_plan_limits(shape, len(ctx), 0, 900, 8, 0)
    assert bd.pa_plan_step_q4(shape, cu, ctx, limits=limits).sizes.T == 0
    with pytest.raises(ValueError):
        bd.pa_plan_step_q4(shape, cu[1:], ctx)


def test_contexts_near_the_end_of_32_bits_are_refused():
    shape, most = bd.Shape.make(8, 2, 128, 128, 64), 2 ** 31 - 1 - 4096
    cu = np.array([0, 1], np.int32)
    for ctx, rows in ((most + 1, 8), (2 ** 31 - 1, 8), (2 ** 31 - 1, 0)):
        with pytest.raises(bd.PagedAttnError) as e:
            bd.pa_plan_step_q4(shape, cu, np.array([ctx], np.int32), rows)
        assert e.value.status == bd.PA_ERR_SHAPE
        with pytest.raises(bd.PagedAttnError) as e:
            bd.pa_q4_plan_limits(shape, 1, 1, ctx, rows)
        assert e.value.status == bd.PA_ERR_SHAPE
    sizes = bd.pa_plan_step_q4(shape, cu, np.array([most], np.int32), 8).sizes
    assert sizes.n_direct == 2 * -(-most // 2048) and bd.pa_q4_plan_limits(shape, 1, 1, most, 8).n_direct >= sizes.n_direct
    # the largest key that q4_direct_kernel looks up: of the eight tiles, of a pair's 64 keys, after the last eight of a split
    assert most - 1 + (2 * (-(-2048 // 64) + 14) + 1) * 32 + 24 < 2 ** 31
    # sizes that no call gave
    sizes.max_ctx = most + 1
    lib = bd.load()
    assert lib.paged_attention_step_q4(4096, 4096, 4096, 4096, 1 << 24, 4096, 4096, C.byref(sizes), 4096, 4096, 1 << 40, 4096, C.byref(shape), None, None) == bd.PA_ERR_SHAPE
    with pytest.raises(bd.PagedAttnError):
        bd.pa_plan_step_q4(shape, cu, np.array([most], np.int32), limits=sizes)


def test_step_refuses():
    lib, shape = bd.load(), bd.Shape.make(8, 2, 128, 16, 64)
    sizes = bd.pa_plan_step_q4(shape, np.array([0, 1], np.int32), np.array([700], np.int32), 8).sizes
    need = bd.pa_q4_workspace_bytes(shape, sizes)
    assert need > 0

    def call(q=4096, kp=4096, vp=4096, table=4096, mb=44, cu=4096, ctx=4096, sz=sizes, words=4096, ws=4096, n=need, out=4096, sh=shape):
        return lib.paged_attention_step_q4(q, kp, vp, table, mb, cu, ctx, None if sz is None else C.byref(sz), words, ws, n, out, C.byref(sh), None, None)

    for kw in (dict(q=None), dict(q=4104), dict(kp=None), dict(vp=4100), dict(table=None), dict(mb=-1), dict(cu=None), dict(ctx=None), dict(sz=None), dict(words=None), dict(out=None),
               dict(out=4098), dict(ws=4100)):
        assert call(**kw) == bd.PA_ERR_INVALID, kw
    assert call(ws=None) == bd.PA_ERR_WORKSPACE and call(n=need - 1) == bd.PA_ERR_WORKSPACE
    assert call(sh=bd.Shape.make(24, 2, 128, 16, 64)) == bd.PA_ERR_SHAPE
    assert call(sh=bd.Shape.make(32, 2, 128, 16, 64)) == bd.PA_ERR_INVALID       # groups of 16 in tiles of 8
    empty = bd.pa_plan_step_q4(shape, np.array([0, 0], np.int32), np.array([5], np.int32), 8).sizes
    assert call(sz=empty, q=None, words=None) == bd.PA_OK
    bad = bd.Q4Sizes.from_buffer_copy(sizes)
    bad.n_direct = -1
    assert call(sz=bad) == bd.PA_ERR_INVALID


def test_runner_limits_without_chunks():
    """A runner that only decodes has no room for chunks, in its plan and its workspace; one for a chunk has that
    chunk's. Contexts of 16,384 and 64 sequences, 32 / 8 heads of 128."""
    shape = bd.Shape.make(32, 8, 128, 16, 64)
    runner = lambda T, chunks, rows=None: bd.StepRunner(shape, device="cpu", kv_bits=4, direct_rows=rows,
                                                        limits=bd.StepLimits(64, T, 1024, 16384, max_chunks=chunks))
    r = runner(64, 0)
    assert r.q4_sizes.n_chunk == r.q4_sizes.n_expand == 0
    # the splits' parts alone: of every row and head, at most 16 splits of 1,024 keys, tiles of 8 rows of 130 numbers
    assert r.ws.numel() * 4 <= 64 * 8 * 16 * 8 * 130 * 4 + 256
    table = np.full((64, 1), -1, np.int32)
    slots = np.full(64, -1, np.int32)
    ctx = np.full(64, 9000, np.int32)
    r.prepare(np.arange(65, dtype=np.int32), ctx, table, slots)
    # the bytes of an expanded context of 16,384: K and V in bf16
    one = 2 * 16384 * 8 * 128 * 2
    chunky = runner(576, 1)
    assert chunky.q4_sizes.n_expand == 128 and chunky.ws.numel() * 4 <= one + 576 * 8 * 16 * 16 * 130 * 4 + 1024
    n = np.ones(64, np.int32)
    n[7] = 513
    cu = lambda n: np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    chunky.prepare(cu(n), ctx, table, np.full(576, -1, np.int32))
    n[7], n[9] = 257, 257
    with pytest.raises(ValueError):
        chunky.prepare(cu(n), ctx, table, np.full(576, -1, np.int32))
    n = np.ones(64, np.int32)
    n[:15], n[20] = 0, 16
    with pytest.raises(ValueError):
        r.prepare(cu(n), ctx, table, slots)
    runner(64, None).prepare(cu(n), ctx, table, slots)
    runner(64, 1).prepare(cu(n), ctx, table, slots)
    with pytest.raises(ValueError):
        bd.StepLimits(64, 64, 1024, 16384, max_chunks=-1)


# ------------------------------------------------------------------------------------- GPU

SHAPES = [(8, 8, 128, 16), (8, 4, 64, 8), (8, 2, 128, 32), (16, 2, 128, 128), (8, 1, 64, 64), (32, 2, 128, 16), (16, 1, 64, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("Hq, Hkv, D, bs", SHAPES)
def test_single_rows_read_from_the_codes(Hq, Hkv, D, bs):
    """Contexts around tiles, warps, splits and the places where the split's length changes."""
    ctx = [1, 2, 8, 31, 32, 33, 127, 128, 129, 160, 511, 512, 513, 640, 1025, 4095, 4096, 4097, 6144, 6145]
    Case([(1, c) for c in ctx], Hq, Hkv, D, bs, seed=Hq + D).check_direct(16)


@pytest.mark.gpu
def test_a_long_context():
    Case([(1, 33000), (1, 32768), (3, 32769), (2, 12289), (1, 12288)], 8, 1, 128, 16, seed=5).check_direct(24)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq, Hkv, D, bs", SHAPES)
def test_few_rows_read_from_the_codes(Hq, Hkv, D, bs):
    """Several tokens per sequence: prompts of a few tokens, tiles with a part of the rows, a split that
    begins between the rows' positions, sequences without rows among them."""
    lens = [(2, 2), (3, 3), (5, 700), (1, 90), (0, 40), (4, 514), (7, 515), (0, 0), (2, 33), (6, 130), (8, 1027)]
    Case(lens, Hq, Hkv, D, bs, seed=Hkv).check_direct(8 * max(Hq // Hkv, 2))


@pytest.mark.gpu
def test_keys_with_a_common_offset():
    """Columns whose keys share a large offset: the minimum carries it, the codes the rest."""
    Case([(1, 300), (2, 77)], seed=11, offset=6.0).check_direct(16)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq, Hkv, D, bs", SHAPES)
@pytest.mark.parametrize("direct_rows", [0, 16])
def test_chunks_over_expanded_contexts(Hq, Hkv, D, bs, direct_rows):
    """Chunks, and with direct_rows 0 single rows, against the definition on K and V rounded to bf16, as the bf16 step is tested."""
    from tests.gpu_util import assert_close
    c = Case([(70, 70), (1, 2500), (129, 700), (33, 2300), (0, 5), (1, 3), (40, 41)], Hq, Hkv, D, bs, seed=bs)
    assert_close(c.run(direct_rows), c.exact(*c.rounded()), f"q4 chunks {Hq}/{Hkv}/{D} rows {direct_rows}")


@pytest.mark.gpu
def test_bits_do_not_depend_on_the_batch():
    """A sequence alone, among others and in another place of pool and step; single tokens and the same rows
    as drafted tokens (contexts whose splits have one length); tiles of 8 and of 16 rows."""
    lens = [(1, 700), (4, 2500), (1, 5000), (2, 40), (3, 1500)]
    a = Case(lens, seed=3)
    for rows in (8, 16):
        whole = a.run(rows)
        assert np.array_equal(whole, a.run(rows))
        for s, (n, c) in enumerate(lens):
            if n * 4 > rows:
                continue
            b = Case([(n, c)], seed=17)
            b.q = a.q[a.cu[s]:a.cu[s + 1]]
            nb = -(-c // 16)
            for pool, src in zip(b.pools, a.pools):
                pool[b.table[0, :nb]] = src[a.table[s, :nb]]
            assert np.array_equal(b.run(rows), whole[a.cu[s]:a.cu[s + 1]])
    wide, narrow = a.run(16), a.run(8)
    for s, (n, c) in enumerate(lens):
        if n <= 2:
            assert np.array_equal(wide[a.cu[s]:a.cu[s + 1]], narrow[a.cu[s]:a.cu[s + 1]])
    # row i of sequence 1 by itself: context shorter by what follows it
    for i in range(4):
        one = Case([(1, 2500 - 3 + i)], seed=19)
        one.q = a.q[a.cu[1] + i:a.cu[1] + i + 1]
        nb = -(-int(one.ctx[0]) // 16)
        for pool, src in zip(one.pools, a.pools):
            pool[one.table[0, :nb]] = src[a.table[1, :nb]]
        assert np.array_equal(one.run(8)[0], wide[a.cu[1] + i])


@pytest.mark.gpu
def test_one_way_for_all_rows():
    """direct_rows 0: a token has the same bits as a single row and within a chunk."""
    a = Case([(60, 2100)], seed=23)
    chunk = a.run(0)
    for i in (0, 17, 59):
        one = Case([(1, 2100 - 59 + i), (1, 9)], seed=29)
        one.q[0] = a.q[i]
        nb = -(-int(one.ctx[0]) // 16)
        for pool, src in zip(one.pools, a.pools):
            pool[one.table[0, :nb]] = src[a.table[0, :nb]]
        assert np.array_equal(one.run(0)[0], chunk[i])


@pytest.mark.gpu
def test_numbers_that_are_none_stay_with_the_rows_that_see_them():
    """A NaN or infinity in K or V of a later token does not reach earlier rows, heads or groups."""
    c = Case([(4, 300), (1, 300)], seed=31)
    clean = c.run(16)
    slot = lambda s, p: int(c.table[s, p // 16]) * 16 + p % 16
    for is_v in (False, True):
        for p in (297, 298, 299):
            pools = [x.copy() for x in c.pools]
            x = np.full((1, 2, 128), 0x3F80, np.uint16)
            x[0, 1, 70] = 0x7F80 if p == 298 else 0x7FC0  # head 1, group 2
            other = q4.write(pools[is_v], x, [slot(0, p)], 16, is_v)
            b, o = divmod(slot(0, p), 16)
            pools[is_v][b, 1] = other[b, 1]
            got = c.run(16, pools=[dev(x) for x in pools])
            val = pa.bf16_to_f64(got)
            assert np.array_equal(got[:, :4], clean[:, :4]) and np.array_equal(got[4:], clean[4:])
            for i in range(4):
                if 296 + i < p:
                    assert np.array_equal(got[i], clean[i])
                elif is_v:
                    assert np.isnan(val[i, 4:, 64:96]).all() and np.isfinite(val[i, 4:, :64]).all() and np.isfinite(val[i, 4:, 96:]).all()
                else:
                    assert np.isnan(val[i, 4:]).all()
    c.q[2, 3, 9] = 0x7FC0                                 # a NaN in one row's q
    got = c.run(16)
    keep = np.ones((5, 8), bool)
    keep[2, 3] = False
    assert np.array_equal(got[keep], clean[keep]) and np.isnan(pa.bf16_to_f64(got[2, 3])).all()


@pytest.mark.gpu
def test_bad_pages_and_metadata():
    c = Case([(1, 600), (2, 300), (40, 200)], seed=37)
    clean = c.run(8)
    table = c.table.copy()
    table[0, 5], table[2, 1] = c.nb, -1                   # outside the pool: keys of value 0
    got = c.run(8, table=table, expect=bd.PA_DEVERR_BLOCK)
    k, v = (np.nan_to_num(q4.values(p, 16, 128, i == 1).astype(np.float64)) for i, p in enumerate(c.pools))
    k, v = (np.concatenate([x, np.zeros((1, *x.shape[1:]))]) for x in (k, v))
    zero = np.where((table < 0) | (table >= c.nb), c.nb, table)
    want = pa.attention(pa.bf16_to_f64(c.q), k, v, zero, c.cu, c.ctx, 8)
    np.testing.assert_allclose(pa.bf16_to_f64(got), want, atol=2e-2)
    assert np.array_equal(got[1:3], clean[1:3])
    nine = wl.f32_to_bf16_bits(np.float32(9))
    # contexts and rows other than the planned ones: those sequences are left out, the rest is as it was
    for s, ctx, cu in ((0, 1300, None), (0, 0, None), (1, 1, None), (2, 39, None), (2, 300, None), (0, -4, None), (0, 2 ** 31 - 1, None),
                       (1, None, [0, 1, 2, 43]), (2, None, [0, 1, 3, 4])):
        x, y = c.ctx.copy(), c.cu if cu is None else np.array(cu, np.int32)
        if ctx is not None:
            x[s] = ctx
        # (a longer chunk's context runs into the table's -1 entries as well)
        got = c.run(8, ctx=x, cu=y, expect=bd.PA_DEVERR_META | (bd.PA_DEVERR_BLOCK if ctx == 300 else 0))
        for t in range(3):
            rows = slice(c.cu[t], c.cu[t + 1])
            if t == s:
                assert (got[rows] == nine).all(), (s, ctx, cu)
            elif cu is None:
                assert np.array_equal(got[rows], clean[rows])
    # a context that the table does not cover
    short = c.table[:, :20].copy()
    got = c.run(8, table=short, expect=bd.PA_DEVERR_META)
    assert (got[0] == nine).all() and np.array_equal(got[1:], clean[1:])
    # words that are no plan: nothing is written
    plan = c.plan(8)
    plan.words.fill_(2 ** 31 - 1)
    assert (c.run(plan=plan, expect=bd.PA_DEVERR_META) == nine).all()


@pytest.mark.gpu
def test_a_captured_step_follows_its_plan():
    """One graph under limits replays steps of other contexts, with and without chunks; two graphs with a
    workspace each on two streams at once."""
    steps = [Case([(1, 700), (1, 90), (30, 2200)], seed=41), Case([(4, 4), (1, 5100), (27, 27)], seed=43), Case([(2, 1000), (1, 513), (29, 129)], seed=47)]
    nb = max(c.nb for c in steps)
    shape = bd.Shape.make(8, 2, 128, 16, nb)
    lim = bd.pa_q4_plan_limits(shape, 3, 32, 5200, 16, 60)

    class Slot:
        def __init__(self):
            self.k, self.v = (torch.zeros(bd.pa_q4_pool_shape(shape), dtype=torch.uint8, device="cuda") for _ in "kv")
            self.q, self.out = (torch.zeros(32, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in "qo")
            self.table = torch.full((3, 330), -1, dtype=torch.int32, device="cuda")
            self.cu, self.ctx = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (4, 3))
            self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
            self.ws = torch.empty(bd.pa_q4_workspace_bytes(shape, lim) // 4 + 1, device="cuda")
            self.plan = None
            self.stream = torch.cuda.Stream()

        def load(self, c):
            for to, x in ((self.k, c.pools[0]), (self.v, c.pools[1])):
                to[:c.nb].copy_(dev(x))
            self.q.copy_(bf16(c.q))
            self.out.fill_(9.0)
            self.table.fill_(-1)
            self.table[:, :c.table.shape[1]].copy_(dev(c.table))
            self.cu.copy_(dev(c.cu))
            self.ctx.copy_(dev(c.ctx))
            p = bd.pa_plan_step_q4(shape, c.cu, c.ctx, limits=lim, device="cuda")
            if self.plan is None:
                self.plan = p
            else:
                self.plan.words.copy_(p.words)

        def call(self):
            bd.paged_attention_step_q4(self.q, self.k, self.v, self.table, self.cu, self.ctx, self.plan, self.ws, self.out, shape, err=self.err)

    slots = [Slot(), Slot()]
    graphs = []
    for s in slots:
        s.load(steps[0])
        s.call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.call()
        graphs.append(g)
    want = [c.run(16) for c in steps]
    for a, b in ((0, 1), (1, 2), (2, 0)):
        slots[0].load(steps[a])
        slots[1].load(steps[b])
        torch.cuda.synchronize()
        for _ in range(3):
            for s, g in zip(slots, graphs):
                with torch.cuda.stream(s.stream):
                    g.replay()
        torch.cuda.synchronize()
        for s, i in zip(slots, (a, b)):
            assert int(s.err.item()) == 0 and np.array_equal(bits_of(s.out), want[i])


def _chain(case, plan, n=8):
    """n steps whose outputs are the next one's q, captured, against the same steps one by one."""
    k, v, table, cu, ctx = (dev(x) for x in (*case.pools, case.table, case.cu, case.ctx))
    ws = torch.empty(bd.pa_q4_workspace_bytes(case.shape, plan) // 4, device="cuda")
    rows = [bf16(case.q)] + [torch.zeros(case.T, case.Hq, case.D, dtype=torch.bfloat16, device="cuda") for _ in range(n)]

    def step(i):
        bd.paged_attention_step_q4(rows[i], k, v, table, cu, ctx, plan, ws, rows[i + 1], case.shape)

    for i in range(n):
        step(i)
        torch.cuda.synchronize()
    want = [bits_of(r) for r in rows]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(n):
            step(i)
    for _ in range(3):
        for r in rows[1:]:
            r.zero_()
        ws.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for r, w in zip(rows, want):
            np.testing.assert_array_equal(bits_of(r), w)


@pytest.mark.gpu
def test_a_chain_of_captured_steps_without_splits():
    # room for splits that no context of these steps has: each step still ends after its rows are written
    case = Case([(1, 1 + s % 256) for s in range(600)], Hq=8, Hkv=8, D=64, bs=16, seed=41)
    limits = bd.pa_q4_plan_limits(case.shape, 600, 600, 5000, 8, 0)
    assert limits.n_fold > 0
    _chain(case, bd.pa_plan_step_q4(case.shape, case.cu, case.ctx, limits=limits, device="cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("chunks, rows", [(1, 250), (6, 3), (40, 2)])
def test_a_chain_of_captured_steps_with_chunks(chunks, rows):
    # the rows read from the codes start while the chunks' attention ends: whichever of them is last, the next step
    # waits for it
    case = Case([(100, 900 - 3 * s) for s in range(chunks)] + [(1, 31 + 13 * s) for s in range(rows)], seed=46)
    plan = case.plan(16)
    assert plan.sizes.n_direct > 0 and plan.sizes.n_chunk > 0
    _chain(case, plan)


@pytest.mark.gpu
def test_lists_longer_than_a_cta_holds():
    # 2,600 sequences of 8 heads over 152 lists: 136 or 137 items a list, 128 of which are held on chip
    rng = np.random.default_rng(42)
    case = Case([(1, int(c)) for c in rng.integers(1, 41, 2600)], Hq=8, Hkv=8, D=64, bs=8, seed=42)
    first = np.diff(case.plan(8).words.cpu().numpy()[case.plan(8).sizes.n_direct * bd.ITEM_INTS:][:153])
    assert first.max() > 128
    case.check_direct(8)


@pytest.mark.gpu
def test_two_streams_at_once():
    cases = [Case([(1, 900 + 37 * s) for s in range(20)], seed=43), Case([(3, 5000 - 91 * s) for s in range(9)], seed=44)]
    want = [c.run(16) for c in cases]
    plans = [c.plan(16) for c in cases]
    held = []
    for c, p in zip(cases, plans):
        held.append([bf16(c.q), *(dev(x) for x in (*c.pools, c.table, c.cu, c.ctx)), p,
                     torch.empty(bd.pa_q4_workspace_bytes(c.shape, p) // 4, device="cuda"),
                     torch.zeros(c.T, c.Hq, c.D, dtype=torch.bfloat16, device="cuda"), c.shape])
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, h in zip(streams, held):
            with torch.cuda.stream(s):
                bd.paged_attention_step_q4(*h)
    torch.cuda.synchronize()
    for h, w in zip(held, want):
        np.testing.assert_array_equal(bits_of(h[-2]), w)


@pytest.mark.gpu
@pytest.mark.parametrize("power", [-100, -20, 20, 100])
@pytest.mark.parametrize("direct_rows", [8, 16])
def test_queries_of_every_magnitude(power, direct_rows):
    # q 2^n over K 2^-n: the same scores, bit for bit, since every scaling on the way is by a power of two
    case = Case([(1, 300), (1, 7), (2, 1000)], Hq=8, Hkv=2, seed=45)
    want = case.run(direct_rows)
    case.q = wl.f32_to_bf16_bits((pa.bf16_to_f64(case.q) * 2.0 ** power).astype(np.float32))
    rows = case.pools[0].reshape(case.nb, case.Hkv, -1)
    params = np.ascontiguousarray(rows[..., case.bs * (case.D // 2):]).view("<u2")
    with np.errstate(invalid="ignore"):
        scaled = wl.f32_to_bf16_bits((pa.bf16_to_f64(params) * 2.0 ** -power).astype(np.float32))
    rows[..., case.bs * (case.D // 2):] = np.where(params == 0xFFFF, params, scaled).astype("<u2").view(np.uint8)
    np.testing.assert_array_equal(case.run(direct_rows), want)


@pytest.mark.gpu
def test_pools_behind_two_gigabytes():
    """Pages at the end of pools of more than 2^31 bytes give the bits of the same pages in small ones."""
    a = Case([(1, 900), (3, 140), (50, 310)], 16, 8, 128, 128, seed=53)
    small = a.run(16)
    per = 8 * 128 * 80
    nb = 2 ** 31 // per + 40
    shape = bd.Shape.make(16, 8, 128, 128, nb)
    pools = [torch.empty(bd.pa_q4_pool_shape(shape), dtype=torch.uint8, device="cuda") for _ in "kv"]
    shift = nb - a.nb
    for p, x in zip(pools, a.pools):
        p[shift:].copy_(dev(x))
    table = np.where(a.table >= 0, a.table + shift, -1).astype(np.int32)
    a.shape = shape
    assert np.array_equal(a.run(16, pools=pools, table=table), small)


@pytest.mark.gpu
def test_a_run_as_it_is_used():
    """Prompts in chunks, then single and drafted tokens: norm + rotation + write, step; a fork whose first
    write copies its page, and a compaction between steps, the pages of K and V together."""
    rng = np.random.default_rng(61)
    Hq, Hkv, D, bs, nb = 8, 2, 128, 16, 64
    shape = bd.Shape.make(Hq, Hkv, D, bs, nb)
    f = 1e4 ** (-np.arange(D // 2) / (D // 2))
    rope = bd.pa_rope_pairs(f, device="cuda")
    w = dev((1 + 0.1 * rng.standard_normal(D)).astype(np.float32)).bfloat16()
    kp, vp = (torch.full(bd.pa_q4_pool_shape(shape), 255, dtype=torch.uint8, device="cuda") for _ in "kv")
    alloc = bd.Allocator(nb, bs)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ctx = {}

    def copy(pairs):
        if pairs:
            bd.paged_copy_pages(dev(np.array(pairs, np.int32)), [kp, vp], err=err)

    def step(new, rows=None):
        seqs = list(new)
        for s in seqs:
            if s not in ctx:
                alloc.admit(s, new[s])
                ctx[s] = 0
            ctx[s] += new[s]
            alloc.ensure_capacity(s, ctx[s])
            copy(alloc.cow(s, ctx[s] - new[s], new[s]))
        lens = np.array([ctx[s] for s in seqs], np.int32)
        cu, slots, table = alloc.build_step(seqs, lens, [new[s] for s in seqs], max_blocks=24)
        T = int(cu[-1])
        x = bf16(wl.random_bf16(rng, (T, Hq + 2 * Hkv, D)))
        q = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        pos = np.concatenate([np.arange(ctx[s] - new[s], ctx[s]) for s in seqs]).astype(np.int32)
        bd.paged_qk_norm_rope_write_q4(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], w, w, 1e-6, rope, dev(pos), dev(slots), q, kp, vp, shape, err=err)
        plan = bd.pa_plan_step_q4(shape, cu, lens, rows, device="cuda")
        ws = torch.empty(bd.pa_q4_workspace_bytes(shape, plan) // 4 + 1, device="cuda")
        out = torch.empty_like(q)
        bd.paged_attention_step_q4(q, kp, vp, dev(table), dev(cu), dev(lens), plan, ws, out, shape, err=err)
        k, v = (np.nan_to_num(q4.values(p.cpu().numpy(), bs, D, i == 1).astype(np.float64)) for i, p in enumerate((kp, vp)))
        want = pa.attention(pa.bf16_to_f64(bits_of(q)), k, v, table, cu, lens, Hq)
        got = pa.bf16_to_f64(bits_of(out))
        # the rounding of K, V, p and the output to bf16, as of the bf16 step
        assert np.all(np.abs(got - want) <= 2.0 ** -5 * np.sqrt((want ** 2).mean(-1, keepdims=True)) + 1e-3)

    step({0: 90, 1: 33, 2: 64})
    step({0: 1, 1: 1, 2: 40})
    alloc.fork(0, 7)
    ctx[7] = ctx[0]
    step({0: 1, 7: 4, 1: 1, 2: 1})
    alloc.free_seq(1)
    del ctx[1]
    alloc.trim(2, 50)
    ctx[2] = 50
    pairs = alloc.compact()
    assert pairs
    copy(pairs)
    alloc.check_consistent()
    step({0: 2, 7: 1, 2: 1, 9: 20})
    step({0: 1, 7: 1, 2: 1, 9: 1}, rows=0)
    assert int(err.item()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fixed", [False, True])
def test_step_runner(fixed):
    """StepRunner over 4-bit pools: write and step of its own plans, with limits as a captured graph."""
    lens = [[(1, 500), (1, 33), (20, 260)], [(1, 501), (20, 53), (1, 261)]]
    a = Case(lens[0], seed=71)
    if not fixed:
        runner = bd.StepRunner(a.shape, kv_bits=4).prepare(a.cu, a.ctx, a.table)
        k, v = (dev(p) for p in a.pools)
        kn, vn = (wl.random_bf16(np.random.default_rng(s), (a.T, 2, 128)) for s in (1, 2))
        out = torch.empty(a.T, 8, 128, dtype=torch.bfloat16, device="cuda")
        runner.run(bf16(a.q), bf16(kn), bf16(vn), k, v, out)
        slots = bd.pa_compute_slots(a.shape, a.table, a.cu, a.ctx)
        a.pools = [q4.write(p, x, slots, 16, i == 1) for i, (p, x) in enumerate(zip(a.pools, (kn, vn)))]
        assert np.array_equal(k.cpu().numpy(), a.pools[0]) and np.array_equal(v.cpu().numpy(), a.pools[1])
        assert runner.device_error() == 0 and np.array_equal(bits_of(out), a.run())
        return
    runner = bd.StepRunner(a.shape, limits=bd.StepLimits(3, 22, 40, 520), kv_bits=4)
    k, v = (dev(p) for p in a.pools)
    q, out = (torch.empty(a.T, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in "qo")
    for i, l in enumerate(lens):
        c = Case(l, seed=71 + i, spare=2)
        if c.nb > a.nb:
            continue
        runner.prepare(c.cu, c.ctx, c.table)
        k.zero_(), v.zero_()
        k[:c.nb].copy_(dev(c.pools[0])), v[:c.nb].copy_(dev(c.pools[1]))
        q.copy_(bf16(c.q))
        if i == 0:
            runner.capture(q, None, None, k, v, out, write=False)
        out.zero_()
        runner.replay()
        torch.cuda.synchronize()
        assert runner.device_error() == 0 and np.array_equal(bits_of(out), c.run(8))


def test_runner_refuses():
    with pytest.raises(ValueError):
        bd.StepRunner(bd.Shape.make(8, 2, 128, 16, 4), device="cpu", kv_bits=8)
    with pytest.raises(ValueError):
        bd.StepRunner(bd.Shape.make(8, 2, 128, 16, 4), device="cpu", kv_bits=4, kv_scales=(1.0, 1.0))


@pytest.mark.gpu
@pytest.mark.parametrize("direct_rows", [0, 8])
def test_a_table_too_narrow_for_a_chunk(direct_rows):
    """A chunk, and with direct_rows 0 a single row, whose context the block table does not cover: its rows are not
    written (the workspace holds nothing of that context), the others are as they were."""
    c = Case([(1, 600), (40, 700), (2, 300), (1, 2500)], seed=73)
    clean = c.run(direct_rows)
    got = c.run(direct_rows, table=c.table[:, :40].copy(), expect=bd.PA_DEVERR_META)
    nine = wl.f32_to_bf16_bits(np.float32(9))
    assert (got[1:41] == nine).all() and (got[43] == nine).all()
    assert np.array_equal(got[[0, 41, 42]], clean[[0, 41, 42]])


@pytest.mark.gpu
@pytest.mark.parametrize("direct_rows", [0, 16])
def test_the_largest_values(direct_rows):
    """Values up to the largest bf16 number, where one key has all of a row's weight: the middle of their group
    (minimum + 8 scale) enters as it is, also in tiles that hold later keys, unwritten ones and NaN."""
    c = Case([(1, 1), (3, 3), (1, 40)], seed=79)
    k, v = np.zeros((44, 2, 128), np.uint16), np.zeros((44, 2, 128), np.uint16)
    ramp = wl.f32_to_bf16_bits(np.linspace(2.0, 3.3, 128, dtype=np.float32) * np.float32(1e38))
    v[0, 0], v[0, 1] = 0x7F7F, 0xFF7F                     # constant groups: scale 0
    v[1] = ramp                                           # all that the first of three rows sees
    if direct_rows:
        v[3] = 0x7FC0                                     # the last row's
    at = 4 + 35
    v[at] = ramp
    k[at] = wl.f32_to_bf16_bits(np.float32(4))            # a score 181 above the others'
    c.q = wl.f32_to_bf16_bits(np.full((5, 8, 128), 4, np.float32))
    slots = [int(c.table[s, p // 16]) * 16 + p % 16 for s, n in ((0, 1), (1, 3), (2, 40)) for p in range(n)]
    c.pools = [q4.write(p, x, slots, 16, i == 1) for i, (p, x) in enumerate(zip(c.pools, (k, v)))]
    got = pa.bf16_to_f64(c.run(direct_rows))[[0, 1, 4]]
    want = np.repeat(q4.values(c.pools[1], 16, 128, True).astype(np.float64).reshape(-1, 2, 128)[slots][[0, 1, at]], 4, 1)
    # Roundings to bf16, 2^-8 of what is rounded each: the output's and the middle's (s (u - 8) has p = 1 and is exact);
    # the middle is at most 1.1 of the value. Expanded, the value's alone.
    assert (np.abs(got - want) <= (2.1 * 2.0 ** -8 + 2.0 ** -15) * np.abs(want)).all()


def test_tiles_of_eight_and_sixteen_rows():
    """What decides the tiles' rows: direct_rows, the group, rows beyond one a sequence, chunks; every plan with the
    same tokens covered."""
    def tiles(n_q, Hq, Hkv, rows, ctx=900, limits=None):
        shape = bd.Shape.make(Hq, Hkv, 128, 16, 4)
        cu = np.concatenate([[0], np.cumsum(n_q)]).astype(np.int32)
        if limits is not None:
            limits = bd.pa_q4_plan_limits(shape, len(n_q), int(cu[-1]), 1000, rows, limits)
        plan = bd.pa_plan_step_q4(shape, cu, np.full(len(n_q), ctx, np.int32), rows if limits is None else None, limits)
        it = _items(plan.words, 0, plan.sizes.n_direct)
        it = it[it["n_q"] > 0]
        few = [t for s, n in enumerate(n_q) if n * (Hq // Hkv) <= rows for t in range(cu[s], cu[s + 1])]
        seen = sorted(t for i in it[(it["split"] == 0) & (it["kv_head"] == 0)] for t in range(i["q_start"], i["q_start"] + i["n_q"]))
        assert seen == few
        return int(it["n_q"].max()) * (Hq // Hkv)

    for limits in (None, 0):
        assert tiles([4, 4, 1], 8, 2, 48, limits=limits) == 16 and tiles([4, 1], 8, 2, 16, limits=limits) == 16
        assert tiles([4, 0, 0, 0], 8, 2, 48, limits=limits) == 8                   # no more rows than sequences
        assert tiles([1, 1], 32, 2, 48, limits=limits) == 16                       # groups of 16
        assert tiles([2, 2], 8, 2, 8, limits=limits) == 8
    for limits in (None, 100):
        assert tiles([4, 40], 8, 2, 48, limits=limits) == 8                        # a chunk beside them
        assert tiles([3, 40], 32, 2, 48, limits=limits) == 16
    assert tiles([4, 4, 1], 8, 2, 48, limits=100) == 8                             # room for chunks


@pytest.mark.gpu
@pytest.mark.parametrize("max_chunks", [None, 3])
def test_a_captured_runner_gives_the_eager_ones_bits(max_chunks):
    """Write and step of a runner with limits, captured once, replayed for steps whose chunks, few tokens and single
    tokens change places, and for the first one again: the pools' bytes and the outputs' bits of a runner without."""
    lens = [[(1, 500), (12, 33), (46, 260), (1, 700)], [(46, 300), (1, 501), (1, 53), (12, 261)], [(20, 20), (13, 700), (26, 26), (1, 90)],
            [(9, 90), (4, 300), (46, 46), (1, 1)]]
    cases = [Case(l, seed=83 + i) for i, l in enumerate(lens)]
    shape = bd.Shape.make(8, 2, 128, 16, max(c.nb for c in cases))
    eager = bd.StepRunner(shape, kv_bits=4)
    fixed = bd.StepRunner(shape, kv_bits=4, limits=bd.StepLimits(4, 60, 50, 800, max_chunks=max_chunks))
    pool = lambda: torch.zeros(bd.pa_q4_pool_shape(shape), dtype=torch.uint8, device="cuda")
    sides = [[torch.zeros(60, 8, 128, dtype=torch.bfloat16, device="cuda"), *(torch.zeros(60, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in "kv"),
              pool(), pool(), torch.zeros(60, 8, 128, dtype=torch.bfloat16, device="cuda")] for _ in "ab"]
    for turn, i in enumerate((0, 1, 2, 3, 0)):
        c, rng = cases[i], np.random.default_rng(i)
        new = [bf16(wl.random_bf16(rng, (60, 2, 128))) for _ in "kv"]
        for q, kn, vn, k, v, out in sides:
            q.copy_(bf16(c.q)), kn.copy_(new[0]), vn.copy_(new[1]), out.zero_()
            for p, x in ((k, c.pools[0]), (v, c.pools[1])):
                p.fill_(255)
                p[:c.nb].copy_(dev(x))
        for runner in (eager, fixed):
            runner.prepare(c.cu, c.ctx, c.table)
        eager.run(*sides[0])
        if turn == 0:
            q, kn, vn, k, v, out = sides[1]
            fixed.capture(q, kn, vn, k, v, out, write=True)
            out.zero_()
        fixed.replay()
        torch.cuda.synchronize()
        assert eager.device_error() == fixed.device_error() == 0
        for a, b in zip(sides[0][3:], sides[1][3:]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), turn


@pytest.mark.gpu
def test_bits_do_not_depend_on_the_tiles():
    """Sequences of several tokens in tiles of 16 rows and, with a chunk beside them, of 8."""
    lens = [(4, 700), (12, 33), (7, 2500), (1, 5000), (3, 514), (12, 6150)]
    a = Case(lens, seed=89)
    b = Case(lens + [(40, 600)], seed=89)
    b.q[:a.T] = a.q
    for s, (_, x) in enumerate(lens):
        n = -(-x // 16)
        for to, src in zip(b.pools, a.pools):
            to[b.table[s, :n]] = src[a.table[s, :n]]
    assert np.array_equal(a.run(48), b.run(48)[:a.T])


def test_arguments_that_would_have_no_effect_are_refused():
    shape = bd.Shape.make(8, 2, 128, 16, 4)
    with pytest.raises(ValueError):
        bd.StepRunner(shape, device="cpu", direct_rows=8)
    with pytest.raises(ValueError):
        bd.StepRunner(shape, device="cpu", direct_rows=8, kv_scales=(1.0, 1.0))
    cu, ctx = np.array([0, 1], np.int32), np.array([7], np.int32)
    limits = bd.pa_q4_plan_limits(shape, 1, 1, 100, 8)
    with pytest.raises(ValueError):
        bd.pa_plan_step_q4(shape, cu, ctx, 16, limits)
    assert bd.pa_plan_step_q4(shape, cu, ctx, 8, limits).sizes.direct_rows == 8


def _held(pool, bs, D, is_v):
    """A pool's codes [nb, bs, Hkv, D], and every column's scale and minimum."""
    nb, H, _ = pool.shape
    c = pool[:, :, :bs * (D // 2)].reshape(nb, H, bs, D // 2)
    u = np.stack([c & 15, c >> 4], -1).reshape(nb, H, bs, D)[..., q4.column_nibble(D, is_v)]
    p = np.ascontiguousarray(pool[:, :, bs * (D // 2):]).view("<u2").reshape(nb, H, bs, D // 32, 2)
    return [x.transpose(0, 2, 1, 3).astype(np.float64) for x in (u, *(np.repeat(pa.bf16_to_f64(p[..., i]), 32, -1) for i in (0, 1)))]


@pytest.mark.gpu
@pytest.mark.parametrize("D, Hq, Hkv", [(128, 8, 2), (64, 16, 2)])
def test_roundings_of_rows_read_from_the_codes(D, Hq, Hkv):
    """What the roundings add up to, and how far a score may be off.

    The error against 64 bits is a sum of independent roundings: of the output, of every p scale, of every middle.
    These are made here, in 64 bits otherwise; were p itself rounded to one bf16 as well, its roundings would come
    on top. The kernel has to be nearer to the first than to the second (its p is relative to another reference,
    which changes the roundings but not their size).
    Per value, an output is off by at most 2^-8 of itself and the roundings' 2^-8 + 2^-15 of p (|s (u - 8)| + |m + 8 s|),
    as in Case.bound, and by what fp32 does to its scores: a group's 32 products, q (u 2^-24) in fp32, are two sums
    of 16 and an accumulator, the minima's product three parts of four groups, and a tensor core may cut each of
    a sum's 17 addends at 2^-23 of the largest: 2 * 17 * 2^-23 < 2^-17 of sum |q| 15 s, and 2^-18 of sum |q| |m| for its 13
    addends; the products with the scales and their sum over the groups are 2^-24 each of these, 8 of them: 2^-21."""
    c = Case([(1, 1500), (1, 900), (2, 700), (1, 2100)], Hq, Hkv, D, 16, seed=97)
    (ku, ks, km), (vu, vs, vm) = (_held(p, 16, D, i == 1) for i, p in enumerate(c.pools))
    exact, q, g = c.exact(), pa.bf16_to_f64(c.q), Hq // Hkv
    got = pa.bf16_to_f64(c.run(16))
    near = lambda x: pa.bf16_to_f64(wl.f32_to_bf16_bits(np.asarray(x, np.float32)))
    two, one, most = (np.empty_like(exact) for _ in range(3))
    for s, (n, x) in enumerate(c.lens):
        block = c.table[s, np.arange(x) // 16]
        at = lambda a: a[block, np.arange(x) % 16]
        for i in range(n):
            t, seen = c.cu[s] + i, x - n + i + 1
            for h in range(Hq):
                U, S, M, u, sc, m = (at(a)[:seen, h // g] for a in (ku, ks, km, vu, vs, vm))
                a = (S * U + M) @ q[t, h] / np.sqrt(D)
                p = np.exp(a - a.max())
                for to, r in ((two, p), (one, near(p))):
                    to[t, h] = near((near(r[:, None] * sc) * (u - 8) + r[:, None] * near(m + 8 * sc)).sum(0) / r.sum())
                e = ((2.0 ** -17 + 2.0 ** -21) * (15 * S @ np.abs(q[t, h])) + (2.0 ** -18 + 2.0 ** -21) * (np.abs(M) @ np.abs(q[t, h]))).max() / np.sqrt(D)
                big = (p[:, None] * (np.abs(sc * (u - 8)) + np.abs(m + 8 * sc))).sum(0) / p.sum()
                most[t, h] = np.abs(exact[t, h]) * 2.0 ** -8 + (2.0 ** -8 + 2.0 ** -15 + 2.0 ** -18 + 2 * np.expm1(2 * e)) * big
    off = [np.sqrt(((y - exact) ** 2).sum() / (exact ** 2).sum()) for y in (got, two, one)]
    assert off[1] < off[2] and off[0] < np.sqrt(off[1] * off[2]), off
    assert (np.abs(got - exact) <= most).all(), float((np.abs(got - exact) / most).max())


def _expanded(c, kinds):
    """The rows of a case over expanded contexts with the roundings of K, V and p given (bf16 or f16) and the output's,
    in 64 bits otherwise."""
    near = {"bf16": lambda x: pa.bf16_to_f64(wl.f32_to_bf16_bits(np.asarray(x, np.float32))), "f16": lambda x: np.asarray(x, np.float16).astype(np.float64)}
    q, g = pa.bf16_to_f64(c.q), c.Hq // c.Hkv
    k, v = (q4.values(p, c.bs, c.D, i == 1).astype(np.float64) for i, p in enumerate(c.pools))
    out = np.empty((c.T, c.Hq, c.D))
    for s, (n, x) in enumerate(c.lens):
        at = c.table[s, np.arange(x) // c.bs], np.arange(x) % c.bs
        ks, vs = near[kinds[0]](k[at]), near[kinds[1]](v[at])
        a = np.einsum("nhgd,khd->hgnk", q[c.cu[s]:c.cu[s + 1]].reshape(n, c.Hkv, g, c.D), ks) / np.sqrt(c.D)
        a[..., np.arange(x) > np.arange(x - n, x)[:, None]] = -np.inf
        p = np.exp(a - a.max(-1, keepdims=True))
        o = np.einsum("hgnk,khd->nhgd", near[kinds[2]](p), vs) / p.sum(-1).transpose(2, 0, 1)[..., None]
        out[c.cu[s]:c.cu[s + 1]] = near["bf16"](o.reshape(n, c.Hq, c.D))
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("D, Hq, Hkv", [(128, 8, 2), (64, 8, 1)])
@pytest.mark.parametrize("power", [-60, -18, -12, -8, 0, 8, 13, 16, 100])
def test_roundings_of_rows_over_expanded_contexts(D, Hq, Hkv, power):
    """The error against 64 bits is that of K and the output rounded to bf16, V and p to f16 (simulated here), for V of
    every magnitude that f16 holds, and elsewhere no larger than with bf16 for all. The border between two
    simulations is their geometric mean; 60,000 outputs leave each uncertain by less than 1 %."""
    c = Case([(40, 700), (26, 1300)], Hq, Hkv, D, 16, seed=101)
    params = np.ascontiguousarray(c.pools[1][:, :, c.bs * (D // 2):]).view("<u2")
    with np.errstate(invalid="ignore"):
        scaled = wl.f32_to_bf16_bits((pa.bf16_to_f64(params) * 2.0 ** power).astype(np.float32))
    c.pools[1][:, :, c.bs * (D // 2):] = np.where(params == 0xFFFF, params, scaled).astype("<u2").view(np.uint8)
    exact = c.exact()
    far = lambda y: np.sqrt((((y - exact) / 2.0 ** power) ** 2).sum() / ((exact / 2.0 ** power) ** 2).sum())
    got, low = far(pa.bf16_to_f64(c.run(0))), far(_expanded(c, ("bf16", "bf16", "bf16")))
    if -12 <= power <= 13:
        # (every block's largest value lies between 1 and 6: in f16's part of the magnitudes, 2^-12 to 65,504)
        high = far(_expanded(c, ("bf16", "f16", "f16")))
        assert high < 0.8 * low and got < np.sqrt(high * low), (got, high, low)
    else:
        assert got < 1.05 * low, (got, low)


@pytest.mark.gpu
def test_blocks_of_both_types_of_values():
    """Blocks of 128 keys whose V is too small for f16, fits, and is too large, one behind the other: every row against
    64 bits. A row's error is four roundings of at most 2^-8 / sqrt(3) of its size each (0.0045 together);
    twice that is left for the few keys of a row at a block's begin. A NaN leaves the bits of the other groups' columns."""
    c = Case([(384, 384), (40, 200)], seed=103)
    at = np.concatenate([c.table[0][np.arange(384) // 16] * 16 + np.arange(384) % 16, c.table[1][np.arange(200) // 16] * 16 + np.arange(200) % 16])
    x = pa.bf16_to_f64(wl.random_bf16(np.random.default_rng(5), (584, 2, 128)))
    x[:384] *= np.repeat(2.0 ** np.array([-30.0, 0.0, 30.0]), 128)[:, None, None]
    c.pools[1] = q4.write(c.pools[1], wl.f32_to_bf16_bits(x.astype(np.float32)), at, 16, True)
    got, exact = pa.bf16_to_f64(c.run(8)), c.exact()
    off = np.sqrt(((got - exact) ** 2).sum((1, 2)) / (exact ** 2).sum((1, 2)))
    assert off.max() < 0.009, (off.max(), off.argmax())
    clean = c.run(8)
    bits = wl.f32_to_bf16_bits(x[-1:].astype(np.float32))
    bits[0, 1, 40] = 0x7FC0
    c.pools[1] = q4.write(c.pools[1], bits, at[-1:], 16, True)
    got = c.run(8)
    keep = np.ones((8, 128), bool)
    keep[4:, 32:64] = False
    assert np.array_equal(got[:, keep], clean[:, keep]) and np.isnan(pa.bf16_to_f64(got[-1, 4:, 32:64])).all()


@pytest.mark.gpu
@pytest.mark.parametrize("direct_rows", [0, 16])
def test_a_captured_step_follows_the_values_types(direct_rows):
    """Replays of one graph while V changes between magnitudes that f16 holds, holds in some blocks, in none: each gives
    the bits of a step called for those pools."""
    c = Case([(40, 900), (1, 2100), (129, 300)], seed=107)
    k, v, table, cu, ctx = (dev(x) for x in (*c.pools, c.table, c.cu, c.ctx))
    plan = c.plan(direct_rows)
    ws = torch.empty(bd.pa_q4_workspace_bytes(c.shape, plan) // 4, device="cuda")
    q, out = bf16(c.q), torch.zeros(c.T, 8, 128, dtype=torch.bfloat16, device="cuda")
    step = lambda: bd.paged_attention_step_q4(q, k, v, table, cu, ctx, plan, ws, out, c.shape)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    params = np.ascontiguousarray(c.pools[1][:, :, 16 * 64:]).view("<u2")
    plain = c.pools[1].copy()
    some = np.zeros(c.nb, bool)
    some[c.table[0, 20:30]] = some[c.table[1, 3]] = True
    for power, where in ((0, some), (30, some), (-30, some), (0, some), (40, ~some), (40, some | True), (0, some)):
        with np.errstate(invalid="ignore"):
            scaled = wl.f32_to_bf16_bits((pa.bf16_to_f64(params) * 2.0 ** power).astype(np.float32))
        scaled = np.where((params != 0xFFFF) & where[:, None, None], scaled, params)
        c.pools[1] = plain.copy()
        c.pools[1][:, :, 16 * 64:] = scaled.astype("<u2").view(np.uint8)
        v.copy_(dev(c.pools[1]))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = bits_of(out)
        assert np.array_equal(got, c.run(plan=plan)) and np.array_equal(got, c.run(direct_rows))
        exact = c.exact()
        off = np.sqrt(((pa.bf16_to_f64(got) - exact) ** 2).sum((1, 2)) / (exact ** 2).sum((1, 2)))
        assert off.max() < 0.009, (power, off.max())          # (as in test_blocks_of_both_types_of_values)
