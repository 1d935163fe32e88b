"""The bounded cache as it is used: prompts in chunks, then single tokens, every step norm + rotation +
write, attention with weights, eviction down to a budget and the freed blocks handed back; each stage
against the fp64 definitions on the state the device had before it (GPU), and the allocator's part of
it (CPU)."""
import numpy as np
import pytest

import oracle.fp8 as ofp8
import oracle.paged_attention as pa
from continuous_batching_gb300 import binding as bd
from oracle.bounded import evict, lse_and_weights, norm_rope

torch = pytest.importorskip("torch")


def test_shared_blocks_are_found_and_made_private_before_an_eviction():
    """An eviction writes the first `budget` entries: the read-only rule over them names shared blocks,
    copy-on-write replaces them, trim gives the tail back."""
    a = bd.Allocator(12, 16)
    a.admit(1, 70)                                    # 5 blocks
    a.fork(1, 2)
    with pytest.raises(bd.ReadOnlyBlock):
        a.slots(2, 0, 40)
    pairs = a.cow(2, 0, 40)
    assert [old for old, _ in pairs] == a.table(1)[:3]
    a.slots(2, 0, 40)
    a.trim(2, 40)
    assert len(a.table(2)) == 3 and len(a.table(1)) == 5 and a.num_free == 12 - 8
    a.check_consistent()


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_prompts_then_tokens_under_a_budget(fp8):
    rng = np.random.default_rng(7)
    Hq, Hkv, D, bs, nb = 4, 2, 128, 16, 40
    g = Hq // Hkv
    budget, recent, sink, chunk, n_decode = 48, 8, 2, 32, 14
    prompts = [70, 25, 48]
    B, max_len = 3, 112
    shape = bd.Shape.make(Hq, Hkv, D, bs, nb)
    f = 10000.0 ** (-np.arange(D // 2) / (D // 2))
    rope = bd.pa_rope_pairs(f, device="cuda")
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    wq, wk = (dev((1 + 0.2 * rng.standard_normal(D)).astype(np.float32)).to(torch.bfloat16) for _ in "qk")
    e = torch.uint8 if fp8 else torch.bfloat16
    kp, vp = (torch.zeros(nb, bs, Hkv, D, dtype=e, device="cuda") for _ in "kv")
    scales = (0.02, 0.02) if fp8 else ()
    s8 = "_fp8" if fp8 else ""
    values = lambda p, s: (ofp8.dequantize(p.cpu().numpy(), s) if fp8 else pa.bf16_to_f64(_bits(p)))
    weights = torch.full((B + 1, Hkv, max_len), 9e9, device="cuda")
    positions = torch.full((B + 1, Hkv, max_len), -7, dtype=torch.int32, device="cuda")
    rows = np.array([2, 0, 3], np.int32)
    alloc = bd.Allocator(nb, bs)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ctx, seen, kept = [0] * B, [0] * B, [0] * B
    for s in range(B):
        alloc.admit(s, 1)
    ws = None
    evicted = 0
    while min(seen[s] - prompts[s] for s in range(B)) < n_decode:
        n_new = [min(chunk, prompts[s] - seen[s]) if seen[s] < prompts[s] else 1 for s in range(B)]
        for s in range(B):
            ctx[s] += n_new[s]
            seen[s] += n_new[s]
            alloc.ensure_capacity(s, ctx[s])
        cu, slots, table = alloc.build_step(range(B), ctx, n_new, max_blocks=8)
        T = int(cu[-1])
        pos = np.concatenate([np.arange(seen[s] - n_new[s], seen[s]) for s in range(B)]).astype(np.int32)
        qkv = dev(rng.standard_normal((T, Hq + 2 * Hkv, D)).astype(np.float32)).to(torch.bfloat16)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        q_out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        getattr(bd, "paged_qk_norm_rope_write" + s8)(q, k, v, wq, wk, 1e-6, rope, dev(pos), dev(slots), q_out, kp, vp,
                                                     *scales, shape, err=err)
        want, mag = norm_rope(pa.bf16_to_f64(_bits(q)), pa.bf16_to_f64(_bits(wq)), 1e-6, f, np.zeros(D // 2, int),
                              pos[None], False)
        assert np.all(np.abs(pa.bf16_to_f64(_bits(q_out)) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * mag)
        ctx_np, cu_np = np.array(ctx, np.int32), cu
        max_ctx = max(ctx)
        need = bd.pa_step_weights_workspace_bytes(shape, B, T, max_ctx) // 4 + 1
        if ws is None or ws.shape[0] < need:
            ws = torch.empty(need, device="cuda")
        items = dev(bd.pa_plan_step_shared(shape, cu_np, ctx_np, table).view(np.int32).reshape(-1))
        out, lse = torch.empty_like(q_out), torch.empty(T, Hq, device="cuda")
        before = weights.cpu().numpy().astype(np.float64)
        getattr(bd, "paged_attention_step_weights" + s8)(
            q_out, kp, vp, dev(table), dev(cu_np), dev(ctx_np), max_ctx, items, *scales, ws, out, lse, dev(rows), weights,
            shape, err=err)
        q64, k64, v64 = pa.bf16_to_f64(_bits(q_out)), values(kp, 0.02), values(vp, 0.02)
        want_lse, w = lse_and_weights(q64, k64, table, cu_np, ctx_np)
        np.testing.assert_allclose(lse.cpu().numpy(), want_lse, atol=2e-5, rtol=1e-6)
        ref = pa.attention(q64, k64, v64, table, cu_np, ctx_np, Hq)
        got = pa.bf16_to_f64(_bits(out))
        assert np.abs(got - ref).max() <= 2.0 ** -5 * np.sqrt((ref ** 2).mean(-1)).max() + 1e-4
        now = weights.cpu().numpy()
        for s in range(B):
            old = before[rows[s], :, :ctx[s]].copy()
            old[:, ctx[s] - n_new[s]:] = 0
            np.testing.assert_allclose(now[rows[s], :, :ctx[s]], old + w[s], rtol=1e-4, atol=1e-7)
            assert abs(w[s].sum() - n_new[s] * Hq) < 1e-6      # every row hands out a weight of one per head
        # ---- down to the budget
        k0, v0 = (p.cpu().clone() if fp8 else p.view(torch.int16).cpu().clone() for p in (kp, vp))
        pos0 = positions.cpu().numpy()
        for s in range(B):
            alloc.slots(s, 0, min(ctx[s], budget))             # nothing shared
        bd.paged_evict(kp, vp, dev(table), dev(ctx_np), dev(np.full(B, budget, np.int32)), dev(np.array(seen, np.int32)),
                       dev(np.array(kept, np.int32)), dev(rows), recent, sink, weights, weights, positions, positions,
                       shape, err=err)
        assert int(err.item()) == 0
        k1, v1 = (p.cpu() if fp8 else p.view(torch.int16).cpu() for p in (kp, vp))
        w1, pos1 = weights.cpu().numpy(), positions.cpu().numpy()
        for s in range(B):
            r, c = rows[s], ctx[s]
            slot = np.array([table[s][j // bs] * bs + j % bs for j in range(c)])
            for h in range(Hkv):
                j = np.arange(c)
                p = np.where(j < kept[s], pos0[r, h, :c], seen[s] - c + j)
                src = evict(now[r, h, :c].astype(np.float64), p, seen[s], budget, recent, sink)
                evicted += int((src != np.arange(len(src))).sum())
                assert np.array_equal(pos1[r, h, :len(src)], p[src])
                assert np.array_equal(w1[r, h, :len(src)], now[r, h, src])
                for a, b in ((k0, k1), (v0, v1)):
                    assert torch.equal(b.view(nb * bs, Hkv, D)[slot[:len(src)], h], a.view(nb * bs, Hkv, D)[slot[src], h])
                # each head's entries are distinct tokens, the last and the first among them
                got = set(pos1[r, h, :len(src)].tolist())
                assert len(got) == len(src) and set(range(max(0, seen[s] - recent), seen[s])) <= got
                assert set(range(min(sink, seen[s]))) <= got
            ctx[s] = kept[s] = min(c, budget)
            alloc.trim(s, ctx[s])
        alloc.check_consistent()
        assert alloc.num_free >= nb - 3 * (budget // bs)
    # 17 steps. Sequence 1 ends with 25 + 16 = 41 tokens and never evicts. At least the protected last
    # tokens behind the budget move, per head: sequence 0 8 (of 64 entries), 6 (of 54), then one in
    # each of 14 steps; sequence 2 one in each of 15
    assert ctx == [budget, 41, budget] and evicted >= Hkv * (8 + 6 + 14 + 15)


@pytest.mark.gpu
def test_offsets_that_pass_32_bits():
    """Blocks at the end of a pool of more than 2^31 elements, and a state row behind as many: the bits
    of the same calls at the start of small ones."""
    Hq, Hkv, D, bs, n, budget, max_len = 16, 8, 128, 128, 300, 130, 1 << 19
    torch.manual_seed(3)
    q, k, v = (torch.randn(n, h, D, device="cuda").bfloat16() for h in (Hq, Hkv, Hkv))
    w = torch.rand(D, device="cuda").bfloat16()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cu, ctx = np.array([0, n], np.int32), np.array([n], np.int32)

    def run(num_blocks, blocks, n_rows, row):
        shape = bd.Shape.make(Hq, Hkv, D, bs, num_blocks)
        kp, vp = (torch.empty(num_blocks, bs, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        weights = torch.empty(n_rows, Hkv, max_len, device="cuda")
        places = torch.empty(n_rows, Hkv, max_len, dtype=torch.int32, device="cuda")
        q_out, out, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(n, Hq, device="cuda")
        table, err = i32(*blocks)[None], i32(0)
        at = torch.arange(n, dtype=torch.int32, device="cuda")
        slots = (table[0][(at // bs).long()] * bs + at % bs).int()
        rope = bd.pa_rope_pairs(1e4 ** (-np.arange(D // 2) / (D // 2)), device="cuda")
        bd.paged_qk_norm_rope_write(q, k, v, w, w, 1e-6, rope, at, slots, q_out, kp, vp, shape, err=err)
        items = torch.from_numpy(bd.pa_plan_step(shape, cu, ctx).view(np.int32).reshape(-1)).cuda()
        ws = torch.empty(bd.pa_step_weights_workspace_bytes(shape, 1, n, n) // 4 + 4, device="cuda")
        bd.paged_attention_step_weights(q_out, kp, vp, table, i32(0, n), i32(n), n, items, ws, out, lse, i32(row),
                                        weights, shape, err=err)
        before = weights[row, :, :n].clone()
        bd.paged_evict(kp, vp, table, i32(n), i32(budget), i32(n), None, i32(row), 8, 2, weights, weights, places,
                       places, shape, err=err)
        assert int(err.item()) == 0
        rows = table[0].long()
        return [x.cpu() for x in (q_out, out, lse, before, kp[rows][:, :40], vp[rows][:, :40],
                                  weights[row, :, :budget], places[row, :, :budget])]

    far_blocks, far_rows = 2 ** 31 // (bs * Hkv * D) + 64, 2 ** 31 // (Hkv * max_len) + 8
    near = run(8, (7, 0, 5), 1, 0)
    far = run(far_blocks, (far_blocks - 1, far_blocks - 8, far_blocks - 3), far_rows, far_rows - 1)
    for a, b in zip(near, far):
        assert torch.equal(a, b)


class _Cache:
    """Four sequences with their pools, state and buffers; run queues a step and an eviction."""
    Hq, Hkv, D, bs, nb, max_len = 16, 8, 128, 16, 600, 4000
    ctx, n_q = np.array([3001, 1700, 40, 3333], np.int32), np.array([1, 300, 40, 1], np.int32)
    shape = bd.Shape.make(Hq, Hkv, D, bs, nb)

    def __init__(self, seed):
        torch.manual_seed(seed)
        B, cu = len(self.ctx), np.concatenate([[0], np.cumsum(self.n_q)]).astype(np.int32)
        T, self.longest = int(cu[-1]), int(self.ctx.max())
        i32 = lambda x: torch.as_tensor(np.asarray(x, np.int32)).cuda()
        half = lambda *s: torch.randn(*s, device="cuda").bfloat16()
        self.q, self.k, self.v = half(T, self.Hq, self.D), half(T, self.Hkv, self.D), half(T, self.Hkv, self.D)
        blocks, table, slots = torch.randperm(self.nb).numpy(), np.zeros((B, -(-self.longest // self.bs)), np.int32), []
        for s, c in enumerate(self.ctx):
            n = -(-int(c) // self.bs)
            table[s, :n], blocks = blocks[:n], blocks[n:]
            new = np.arange(c - self.n_q[s], c)
            slots.append(table[s, new // self.bs] * self.bs + new % self.bs)
        self.table, self.slots, self.cu = i32(table), i32(np.concatenate(slots)), i32(cu)
        self.pos = i32(np.concatenate([np.arange(c - n, c) for c, n in zip(self.ctx, self.n_q)]))
        self.ctx_d, self.rows, self.budget, self.err = i32(self.ctx), i32([2, 0, 3, 1]), i32([1500] * B), i32([0])
        self.rope = bd.pa_rope_pairs(1e4 ** (-np.arange(self.D // 2) / (self.D // 2)), device="cuda")
        self.items = torch.from_numpy(bd.pa_plan_step(self.shape, cu, self.ctx).view(np.int32).reshape(-1)).cuda()
        need = bd.pa_step_weights_workspace_bytes(self.shape, B, T, self.longest)
        self.ws = torch.empty(need // 4 + 4, device="cuda")
        pool, state = (self.nb, self.bs, self.Hkv, self.D), (B, self.Hkv, self.max_len)
        self.first = [half(*pool), half(*pool), torch.rand(*state, device="cuda"),
                      torch.zeros(state, dtype=torch.int32, device="cuda"), torch.zeros_like(self.q),
                      torch.zeros_like(self.q), torch.zeros(T, self.Hq, device="cuda")]
        self.now = [x.clone() for x in self.first]

    def reset(self):
        for x, y in zip(self.now, self.first):
            x.copy_(y)

    def run(self, stream=None):
        kp, vp, weights, places, q_out, out, lse = self.now
        bd.paged_qk_norm_rope_write(self.q, self.k, self.v, None, None, 1e-6, self.rope, self.pos, self.slots, q_out,
                                    kp, vp, self.shape, err=self.err, stream=stream)
        bd.paged_attention_step_weights(q_out, kp, vp, self.table, self.cu, self.ctx_d, self.longest, self.items,
                                        self.ws, out, lse, self.rows, weights, self.shape, err=self.err, stream=stream)
        bd.paged_evict(kp, vp, self.table, self.ctx_d, self.budget, self.ctx_d, None, self.rows, 16, 2, weights,
                       weights, places, places, self.shape, err=self.err, stream=stream)


@pytest.mark.gpu
def test_two_caches_at_once():
    """Calls of two caches queued in turn on two streams, by themselves and as replayed graphs: the bits
    of each cache alone."""
    caches, streams = [_Cache(1), _Cache(2)], [torch.cuda.Stream(), torch.cuda.Stream()]
    want = []
    for c in caches:
        c.run()
        torch.cuda.synchronize()
        want.append([x.clone() for x in c.now])

    def check():
        torch.cuda.synchronize()
        for c, w in zip(caches, want):
            assert int(c.err.item()) == 0
            for x, y in zip(c.now, w):
                assert torch.equal(x, y)
            c.reset()
        torch.cuda.synchronize()

    for c in caches:
        c.reset()
    torch.cuda.synchronize()
    for _ in range(4):
        for c, s in zip(caches, streams):
            c.run(s)
        check()
    graphs = []
    for c, s in zip(caches, streams):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            c.run()
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        check()
