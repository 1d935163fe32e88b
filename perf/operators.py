"""What is measured of the operators around a bounded paged KV cache.

Four kinds of calls, each with a plain form in elementary torch operations and the call a user makes:

- ``rope``: per-head RMS norm of q and k, rotation by position (one or several axes), q to its
  buffer and K / V through the slot mapping into the paged pools;
- ``weights``: the attention weight every cached key received from a step's query rows, added to a
  running sum per (sequence, KV head, cache index), from the rows' log-sum-exp;
- ``step``: the attention step of a bounded cache: outputs, log-sum-exp and the running weights;
- ``evict``: per (sequence, KV head) the ``budget`` entries to keep, and the compaction of the paged
  cache, weights and token positions.

Shapes are those of the repository's workloads: 32 / 8 or 64 / 8 heads of 128 (and small ones of
64), blocks of 16 or 32, lognormal or long-tailed contexts, 512-row chunks, bf16 and e4m3 caches.
"""
import math
import random

import torch

own = False

DEV = "cuda"
K_SCALE, V_SCALE = 0.0125, 0.015625


# ---------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one sequence generating: the smallest call, where latency counts
        dict(name="rope_one_token", op="rope", T=1, Hq=32, Hkv=8, D=128, bs=16, rot=128, axes=1, inter=False, norm=True, fp8=False),
        # a decode batch of 128 rows of the long-tail shape
        dict(name="rope_decode", op="rope", T=128, Hq=64, Hkv=8, D=128, bs=32, rot=128, axes=1, inter=False, norm=True, fp8=False),
        # a long prompt's prefill, q / k / v as views of one packed projection
        dict(name="rope_prompt", op="rope", T=16384, Hq=32, Hkv=8, D=128, bs=16, rot=128, axes=1, inter=False, norm=True, fp8=False),
        # image and text tokens of a flat step: three axes, adjacent pairs, e4m3 cache
        dict(name="rope_axes_fp8", op="rope", T=2096, Hq=32, Hkv=8, D=128, bs=16, rot=128, axes=3, inter=True, norm=True, fp8=True),
        # one long sequence decoding
        dict(name="weights_one", op="weights", kind="fixed", B=1, n_q=1, lo=16001, hi=16001, lens=1, Hq=32, Hkv=8, D=128, bs=16, fp8=False),
        # the decode batch (lognormal contexts, median 2048)
        dict(name="weights_decode", op="weights", kind="lognormal", B=64, n_q=1, lo=2048, hi=16384, lens=2, Hq=32, Hkv=8, D=128, bs=16, fp8=False),
        # long-tailed contexts over an e4m3 cache, groups of 8
        dict(name="weights_tail_fp8", op="weights", kind="tail", B=32, n_q=1, lo=1024, hi=40000, lens=3, Hq=64, Hkv=8, D=128, bs=32, fp8=True),
        # chunked prefill: 512-row segments behind prior tokens
        dict(name="weights_chunks", op="weights", kind="uniform", B=4, n_q=512, lo=600, hi=9512, lens=5, Hq=32, Hkv=8, D=128, bs=16, fp8=False),
        # a decode step of a bounded cache
        dict(name="step_decode", op="step", kind="uniform", B=32, n_q=1, lo=4000, hi=16384, lens=6, Hq=32, Hkv=8, D=128, bs=16, fp8=False),
        # a ragged chunk with heads of 64
        dict(name="step_chunk_d64", op="step", kind="uniform", B=3, n_q=257, lo=300, hi=2500, lens=7, Hq=16, Hkv=8, D=64, bs=16, fp8=False),
        # every step of a full cache: one entry out per sequence and head
        dict(name="evict_step", op="evict", B=64, lo=2049, hi=2049, budget=2048, again=True, recent=256, sink=4, lens=8, Hkv=8, D=128, bs=16, fp8=False),
        # prompts cut down to a budget once they are in
        dict(name="evict_prompt", op="evict", B=8, lo=4000, hi=40000, budget=2048, again=False, recent=128, sink=4, lens=9, Hkv=8, D=128, bs=16, fp8=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "weights", "weights", "step", "evict"])
    Hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 4, 8])
    fp8 = rng.random() < 0.35
    D = 128 if fp8 else rng.choice([64, 128, 128])
    bs = rng.choice([8, 16, 16, 32, 64])
    c = dict(op=op, Hkv=Hkv, D=D, bs=bs, fp8=fp8)
    if op == "rope":
        c.update(Hq=Hkv * g, T=_log(rng, 1, 9000), rot=rng.choice([D, D, D // 2]), axes=rng.choice([1, 1, 2, 3]), inter=rng.random() < 0.5, norm=rng.random() < 0.8)
        return c
    if op == "evict":
        budget = _log(rng, 32, 4096)
        again = rng.random() < 0.5
        lo = budget + _log(rng, 1, 64) if again else budget + _log(rng, 16, 4096)
        hi = lo if again else lo + _log(rng, 1, 16000)
        c.update(B=_log(rng, 1, min(64, max(8, 16384 // budget))), lo=lo, hi=hi, budget=budget, again=again, recent=rng.randint(1, budget // 2), sink=rng.choice([0, 1, 4]), lens=rng.randrange(1 << 30))
        return c
    n_q = 1 if rng.random() < 0.5 else _log(rng, 2, 512)
    hi = _log(rng, max(64, n_q), 16000 if n_q == 1 else 8000)
    B = _log(rng, 1, min(64, max(4, 300000 // hi))) if n_q == 1 else rng.randint(1, 4 if n_q * hi < 1e6 else 2)
    c.update(Hq=Hkv * g if n_q == 1 else min(32, Hkv * g), kind="uniform", B=B, n_q=n_q, lo=max(n_q, hi // rng.choice([1, 2, 16])), hi=hi, lens=rng.randrange(1 << 30))
    return c


def _lens(c):
    """Query rows and context of every sequence (fixed by the case): ctx counts the rows."""
    r = random.Random(c["lens"])
    out = []
    for i in range(c["B"]):
        kind = c.get("kind", "uniform")
        if kind == "lognormal":
            x = min(c["hi"], max(16, int(r.lognormvariate(math.log(c["lo"]), 1.0))))
        elif kind == "tail":
            x = r.randint(c["lo"], 4 * c["lo"]) if i % 10 else r.randint(int(0.4 * c["hi"]), c["hi"])
        else:
            x = r.randint(c["lo"], c["hi"])
        out.append((min(c.get("n_q", 1), x), x))
    return out


# ------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _pool(g, fp8, *shape):
    x = _randn(g, *shape)
    if fp8:
        return (x / K_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.to(torch.bfloat16)


def _table(g, ctxs, bs, num_blocks):
    """Block tables over a permuted pool, -1 behind a sequence's last block."""
    perm = torch.randperm(num_blocks, generator=g, device=DEV).to(torch.int32).cpu()
    width = max(-(-x // bs) for x in ctxs)
    t = torch.full((len(ctxs), width), -1, dtype=torch.int32)
    at = 0
    for i, x in enumerate(ctxs):
        n = -(-x // bs)
        t[i, :n] = perm[at:at + n]
        at += n
    return t


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c = case
    g = _gen(seed)
    s = {"case": c}
    if c["op"] == "rope":
        T, Hq, Hkv, D, bs = c["T"], c["Hq"], c["Hkv"], c["D"], c["bs"]
        packed = _randn(g, T, (Hq + 2 * Hkv) * D).to(torch.bfloat16)
        s["q"] = packed[:, :Hq * D].view(T, Hq, D)
        s["k"] = packed[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        s["v"] = packed[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        s["wq"] = (1 + 0.1 * _randn(g, D)).to(torch.bfloat16) if c["norm"] else None
        s["wk"] = (1 + 0.1 * _randn(g, D)).to(torch.bfloat16) if c["norm"] else None
        n = c["rot"] // 2
        s["inv_freq"] = 10000.0 ** (-torch.arange(n, dtype=torch.float64) / n)
        s["axis"] = torch.arange(n) % c["axes"]
        # far positions among them; every axis moves on its own
        s["pos"] = torch.randint(0, 131072, (c["axes"], T), generator=g, device=DEV, dtype=torch.int32)
        nb = -(-T // bs) + 3
        s["slots"] = torch.randperm(nb * bs, generator=g, device=DEV)[:T].to(torch.int32)
        s["k_pool"], s["v_pool"] = _pool(g, c["fp8"], nb, bs, Hkv, D), _pool(g, c["fp8"], nb, bs, Hkv, D)
        s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
        s["freq_dev"], s["axis_dev"] = s["inv_freq"].to(DEV), s["axis"].to(DEV)
        if own:
            from continuous_batching_gb300 import binding as bd
            s["shape"] = bd.Shape.make(Hq, Hkv, D, bs, nb)
            s["rope"] = bd.pa_rope_pairs(s["inv_freq"].numpy(), s["axis"].numpy(), device=DEV)
        return s
    Hkv, D, bs, B = c["Hkv"], c["D"], c["bs"], c["B"]
    lens = _lens(c)
    ctxs = [x for _, x in lens]
    nb = sum(-(-x // bs) for x in ctxs) + 2
    s["table_host"] = _table(g, ctxs, bs, nb)
    s["table"] = s["table_host"].to(DEV)
    s["ctx"] = _int(ctxs)
    s["k_pool"], s["v_pool"] = _pool(g, c["fp8"], nb, bs, Hkv, D), None
    # the state rows of the sequences are theirs for life: not the step's order
    n_rows = B + 2
    s["rows"] = torch.randperm(n_rows, generator=g, device=DEV)[:B].to(torch.int32)
    L = max(ctxs)
    s["L"] = L
    max_len = L + 5
    if c["op"] == "evict":
        s["v_pool"] = _pool(g, c["fp8"], nb, bs, Hkv, D)
        # accumulated weights: heavy-tailed
        s["weights"] = torch.exp(1.5 * _randn(g, n_rows, Hkv, max_len))
        s["weights_out"] = torch.zeros_like(s["weights"])
        s["budget"] = _int([c["budget"]] * B)
        kept = c["budget"] if c["again"] else 0
        s["kept"] = _int([kept] * B)
        # tokens seen so far; before, the cache was cut to `kept` entries of random tokens
        seen = [x + 3 * kept for x in ctxs]
        s["seen"] = _int(seen)
        s["positions"] = torch.zeros(n_rows, Hkv, max_len, dtype=torch.int32, device=DEV)
        if kept:
            s["positions"][:, :, :kept] = torch.rand(n_rows, Hkv, 4 * kept, generator=g, device=DEV).argsort(-1)[:, :, :kept].to(torch.int32)
        s["positions_out"] = torch.zeros_like(s["positions"])
        if own:
            from continuous_batching_gb300 import binding as bd
            s["shape"] = bd.Shape.make(Hkv, Hkv, D, bs, nb)
        return s
    Hq = c["Hq"]
    cu = [0]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    T = cu[-1]
    s["cu"], s["T"], s["n_max"] = _int(cu), T, max(n for n, _ in lens)
    s["q"] = _randn(g, T, Hq, D).to(torch.bfloat16)
    s["weights"] = torch.rand(n_rows, Hkv, max_len, generator=g, device=DEV) * 4
    if c["op"] == "weights":
        # what the attention step before it has left: the rows' log-sum-exp
        s["lse"] = _plain_scores(s)[1]
        if own:
            from continuous_batching_gb300 import binding as bd
            s["shape"] = bd.Shape.make(Hq, Hkv, D, bs, nb)
        return s
    s["v_pool"] = _pool(g, c["fp8"], nb, bs, Hkv, D)
    s["out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.empty(T, Hq, dtype=torch.float32, device=DEV)
    if own:
        from continuous_batching_gb300 import binding as bd
        import numpy as np
        sh = s["shape"] = bd.Shape.make(Hq, Hkv, D, bs, nb)
        items = bd.pa_plan_step(sh, np.asarray(cu, np.int32), np.asarray(ctxs, np.int32))
        s["items"] = torch.from_numpy(items.view(np.int32).reshape(-1).copy()).to(DEV)
        need = bd.pa_step_weights_workspace_bytes(sh, B, T, L)
        s["ws"] = torch.empty((need + 3) // 4, dtype=torch.float32, device=DEV)
    return s


# ---------------------------------------------------------------------------------- plain forms

def _values(x, scale, fp8):
    """What a cache's stored elements stand for, in 32 bits."""
    return x.view(torch.float8_e4m3fn).float() * scale if fp8 else x.float()


def _gather(s, pool, scale):
    """[B, L, Hkv, D] of a paged pool in 32 bits (any block where the table has none)."""
    c = s["case"]
    j = torch.arange(s["L"], device=DEV)
    slots = s["table"].clamp(min=0)[:, j // c["bs"]].long() * c["bs"] + j % c["bs"]
    return _values(pool.view(-1, c["Hkv"], c["D"])[slots], scale, c["fp8"])


def _plain_scores(s):
    """Masked scaled scores [B, Hkv, g, n_max, L] of padded query rows, their lse [T, Hq], and the
    row index of every (sequence, padded row) with the mask of real ones."""
    c = s["case"]
    B, Hkv, g, n, L, D = c["B"], c["Hkv"], c["Hq"] // c["Hkv"], s["n_max"], s["L"], c["D"]
    cu, ctx = s["cu"].long(), s["ctx"].long()
    i = torch.arange(n, device=DEV)
    n_q = cu[1:] - cu[:-1]
    real = i < n_q[:, None]
    at = (cu[:-1, None] + i).clamp(max=s["T"] - 1)
    q = s["q"].float()[at].view(B, n, Hkv, g, D)
    k = _gather(s, s["k_pool"], K_SCALE)
    x = torch.einsum("bnhgd,blhd->bhgnl", q, k) * (1 / math.sqrt(D))
    pos = (ctx - n_q)[:, None] + i
    seen = (torch.arange(L, device=DEV) <= pos[..., None]) & real[..., None]
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1).clamp(min=-1e30)
    lse = m + torch.log(torch.exp(x - m[..., None]).sum(-1))
    rows = lse.permute(0, 3, 1, 2).reshape(B, n, Hkv * g)[real]
    return x, rows, at, real


def _plain_add(s, p):
    """The running weights with the step's p [B, Hkv, L] added: entries behind those of earlier
    steps start afresh, the rest of the state stays."""
    n_q = (s["cu"][1:] - s["cu"][:-1]).long()
    j = torch.arange(s["L"], device=DEV)
    ctx = s["ctx"].long()
    rows = s["rows"].long()
    w = s["weights"][rows, :, :s["L"]]
    new = torch.where((j < (ctx - n_q)[:, None])[:, None], w, 0) + p
    s["weights"][rows, :, :s["L"]] = torch.where((j < ctx[:, None])[:, None], new, w)


def _plain_rope(s):
    c = s["case"]
    D, r, n = c["D"], c["rot"], c["rot"] // 2
    a = s["pos"].double()[s["axis_dev"]].t() * s["freq_dev"]
    cos, sin = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]

    def turn(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
        u, v = (x[..., 0:r:2], x[..., 1:r:2]) if c["inter"] else (x[..., :n], x[..., n:r])
        u, v = u * cos - v * sin, u * sin + v * cos
        y = torch.stack([u, v], -1).flatten(-2) if c["inter"] else torch.cat([u, v], -1)
        return torch.cat([y, x[..., r:]], -1)

    s["q_out"].copy_(turn(s["q"], s["wq"]))
    at = s["slots"].long()
    for pool, x, scale in ((s["k_pool"], turn(s["k"], s["wk"]), K_SCALE), (s["v_pool"], s["v"].float(), V_SCALE)):
        if c["fp8"]:
            x = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        pool.view(-1, c["Hkv"], D)[at] = x.to(pool.dtype)


def _plain_evict(s):
    c = s["case"]
    B, Hkv, D, bs, L = c["B"], c["Hkv"], c["D"], c["bs"], s["L"]
    rows, ctx = s["rows"].long(), s["ctx"].long()
    j = torch.arange(L, device=DEV)
    w = s["weights"][rows, :, :L]
    since = (s["seen"].long() - ctx)[:, None, None] + j
    pos = torch.where(j < s["kept"].long()[:, None, None], s["positions"][rows, :, :L].long(), since)
    guarded = (pos < c["sink"]) | (pos >= s["seen"].long()[:, None, None] - c["recent"])
    valid = (j < ctx[:, None])[:, None].expand(B, Hkv, L)
    key = torch.where(valid, torch.where(guarded, math.inf, w), -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    length = torch.minimum(ctx, s["budget"].long())[:, None, None]
    keep = torch.zeros_like(valid).scatter(-1, order, (j < length).expand(B, Hkv, L))
    hole, stray = (j < length) & ~keep, (j >= length) & keep
    # the k-th stray moves into the k-th hole
    by_rank = torch.zeros_like(order).scatter(-1, torch.where(stray, stray.cumsum(-1) - 1, L - 1), torch.where(stray, j, 0))
    source = torch.where(hole, by_rank.gather(-1, (hole.cumsum(-1) - 1).clamp(min=0)), j)
    b, h, i = torch.nonzero(hole, as_tuple=True)
    table = s["table"].long()
    src = source[b, h, i]
    to, frm = table[b, i // bs] * bs + i % bs, table[b, src // bs] * bs + src % bs
    for pool in (s["k_pool"], s["v_pool"]):
        flat = pool.view(-1, Hkv, D)
        flat[to, h] = flat[frm, h]
    inside = (j < length).expand(B, Hkv, L)
    for to, x in ((s["weights_out"], w), (s["positions_out"], pos.int())):
        to[rows, :, :L] = torch.where(inside, x.gather(-1, source), to[rows, :, :L])


def run(state):
    s = state
    c = s["case"]
    fp8 = c["fp8"]
    scales = (K_SCALE, V_SCALE)
    if own:
        from continuous_batching_gb300 import binding as bd
    if c["op"] == "rope":
        if own and fp8:
            bd.paged_qk_norm_rope_write_fp8(s["q"], s["k"], s["v"], s["wq"], s["wk"], 1e-6, s["rope"], s["pos"], s["slots"], s["q_out"], s["k_pool"], s["v_pool"], *scales, s["shape"], interleaved=c["inter"])
        elif own:
            bd.paged_qk_norm_rope_write(s["q"], s["k"], s["v"], s["wq"], s["wk"], 1e-6, s["rope"], s["pos"], s["slots"], s["q_out"], s["k_pool"], s["v_pool"], s["shape"], interleaved=c["inter"])
        else:
            _plain_rope(s)
        e = torch.float8_e4m3fn if fp8 else torch.bfloat16
        return {"q": s["q_out"], "k": s["k_pool"].view(e), "v": s["v_pool"].view(e)}
    if c["op"] == "weights":
        if own and fp8:
            bd.paged_attention_weights_fp8(s["q"], s["k_pool"], s["lse"], s["table"], s["cu"], s["ctx"], s["rows"], s["weights"], K_SCALE, s["shape"])
        elif own:
            bd.paged_attention_weights(s["q"], s["k_pool"], s["lse"], s["table"], s["cu"], s["ctx"], s["rows"], s["weights"], s["shape"])
        else:
            x, _, at, real = _plain_scores(s)
            lse = s["lse"][at].masked_fill(~real[..., None], math.inf)
            lse = lse.view(c["B"], s["n_max"], c["Hkv"], -1).permute(0, 2, 3, 1)
            _plain_add(s, torch.exp(x - lse[..., None]).sum((2, 3)))
        return {"weights": s["weights"]}
    if c["op"] == "step":
        if own and fp8:
            bd.paged_attention_step_weights_fp8(s["q"], s["k_pool"], s["v_pool"], s["table"], s["cu"], s["ctx"], s["L"], s["items"], *scales, s["ws"], s["out"], s["lse"], s["rows"], s["weights"], s["shape"])
        elif own:
            bd.paged_attention_step_weights(s["q"], s["k_pool"], s["v_pool"], s["table"], s["cu"], s["ctx"], s["L"], s["items"], s["ws"], s["out"], s["lse"], s["rows"], s["weights"], s["shape"])
        else:
            x, lse, at, real = _plain_scores(s)
            m = x.amax(-1, keepdim=True).clamp(min=-1e30)
            p = torch.exp(x - m)
            p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
            o = torch.einsum("bhgnl,blhd->bnhgd", p, _gather(s, s["v_pool"], V_SCALE))
            s["out"].copy_(o.reshape(c["B"], s["n_max"], c["Hq"], c["D"])[real])
            s["lse"].copy_(lse)
            _plain_add(s, p.sum((2, 3)))
        return {"out": s["out"], "lse": s["lse"], "weights": s["weights"]}
    if own:
        bd.paged_evict(s["k_pool"], s["v_pool"], s["table"], s["ctx"], s["budget"], s["seen"], s["kept"], s["rows"], c["recent"], c["sink"], s["weights"], s["weights_out"], s["positions"], s["positions_out"], s["shape"])
    else:
        _plain_evict(s)
    e = torch.float8_e4m3fn if fp8 else torch.bfloat16
    return {"k": s["k_pool"].view(e), "v": s["v_pool"].view(e), "weights": s["weights_out"], "positions": s["positions_out"]}


# ----------------------------------------------------------------------------------- the work

def work(case):
    c = case
    es = 1 if c["fp8"] else 2
    Hkv, D = c["Hkv"], c["D"]
    if c["op"] == "rope":
        T, Hq = c["T"], c["Hq"]
        read = T * (Hq + 2 * Hkv) * D * 2 + T * 4 * (c["axes"] + 1)
        return {"bytes": read + T * Hq * D * 2 + T * 2 * Hkv * D * es, "flops": T * (Hq + Hkv) * D * 7}
    lens = _lens(c)
    if c["op"] == "evict":
        # an entry's place says nothing about its weight: the strays are the recent ones and the
        # expected share of the others that are kept
        n = 0
        for _, x in lens:
            free = max(1, x - c["recent"] - c["sink"])
            inside = max(0, c["budget"] - c["recent"] - c["sink"]) / free
            strays = min(x - c["budget"], c["recent"]) + inside * max(0, x - c["budget"] - c["recent"])
            kept = c["budget"] if c["again"] else 0
            n += Hkv * (4 * x + 4 * kept + 8 * c["budget"] + strays * 4 * D * es)
        return {"bytes": n, "flops": 0}
    Hq = c["Hq"]
    T = sum(n for n, _ in lens)
    pairs = sum(n * (x - n) + n * (n + 1) // 2 for n, x in lens)
    ctx = sum(x for _, x in lens)
    b = ctx * Hkv * D * es + T * Hq * (D * 2 + 4) + 8 * ctx * Hkv - 4 * T * Hkv
    if c["op"] == "weights":
        return {"bytes": b, "flops": 2 * D * Hq * pairs}
    return {"bytes": b + ctx * Hkv * D * es + T * Hq * D * 2, "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------------- the definition, in 64 bits

def _stored(x, fp8, scale=1.0):
    return x.view(torch.float8_e4m3fn).double() * scale if fp8 else x.double()


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    fp8, Hkv, D, bs = c["fp8"], c["Hkv"], c["D"], c["bs"]
    if c["op"] == "rope":
        half = c["rot"] // 2
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                           torch.stack([s["pos"][int(a)].double() * float(f) for a, f in zip(s["axis"], s["inv_freq"])], -1))

        def rotated(x, w):
            y = x.double()
            if w is not None:
                y = y / (y.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
            first = range(0, c["rot"], 2) if c["inter"] else range(half)
            first = torch.tensor(list(first), device=DEV)
            second = first + (1 if c["inter"] else half)
            z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
            y = y.clone()
            y[..., first], y[..., second] = z.real, z.imag
            return y

        out = {"q": rotated(s["q"], s["wq"])}
        for name, x, scale in (("k", rotated(s["k"], s["wk"]), K_SCALE), ("v", s["v"].double(), V_SCALE)):
            pool = _stored(s[name + "_pool"], fp8)
            flat = pool.view(-1, Hkv, D)
            flat[s["slots"].long()] = (x / scale).clamp(-448, 448) if fp8 else x
            out[name] = pool
        return out
    lens = _lens(c)
    table = s["table_host"].long().to(DEV)
    if c["op"] == "evict":
        pools = [_stored(s["k_pool"], fp8), _stored(s["v_pool"], fp8)]
        flat = [p.view(-1, Hkv, D) for p in pools]
        w_out = s["weights_out"].double()
        for b, (_, x) in enumerate(lens):
            row, keep_n = int(s["rows"][b]), min(x, c["budget"])
            seen, kept = int(s["seen"][b]), int(s["kept"][b])
            slot = table[b].repeat_interleave(bs)[:x] * bs + torch.arange(x, device=DEV) % bs
            for h in range(Hkv):
                pos = torch.arange(x, device=DEV) + (seen - x)
                pos[:kept] = s["positions"][row, h, :kept].long()
                w = s["weights"][row, h, :x].double()
                rank = torch.where((pos < c["sink"]) | (pos >= seen - c["recent"]), 1e300, w)
                chosen = torch.argsort(-rank, stable=True)[:keep_n]
                flag = torch.zeros(x, dtype=torch.bool, device=DEV)
                flag[chosen] = True
                holes = (~flag[:keep_n]).nonzero().flatten()
                strays = flag[keep_n:].nonzero().flatten() + keep_n
                final = w.clone()
                final[holes] = w[strays]
                w_out[row, h, :keep_n] = final[:keep_n]
                for f in flat:
                    f[slot[holes], h] = f[slot[strays], h]
        return {"k": pools[0], "v": pools[1], "weights": w_out, "positions": None}
    Hq, g = c["Hq"], c["Hq"] // Hkv
    weights = s["weights"].double()
    outs, lses, at = [], [], 0
    for b, (n, x) in enumerate(lens):
        slot = table[b].repeat_interleave(bs)[:x] * bs + torch.arange(x, device=DEV) % bs
        k = _stored(s["k_pool"].view(-1, Hkv, D)[slot], fp8, K_SCALE if fp8 else 1.0)
        q = s["q"][at:at + n].double().view(n, Hkv, g, D)
        later = torch.arange(x, device=DEV) > torch.arange(x - n, x, device=DEV)[:, None]
        row = int(s["rows"][b])
        o = torch.empty(n, Hkv, g, D, dtype=torch.float64, device=DEV)
        e = torch.empty(n, Hkv, g, dtype=torch.float64, device=DEV)
        for h in range(Hkv):
            a = torch.matmul(q[:, h].transpose(0, 1), k[:, h].t()) / math.sqrt(D)
            a[:, later] = -math.inf
            e[:, h] = torch.logsumexp(a, -1).t()
            given = s["lse"][at:at + n].double().view(n, Hkv, g)[:, h] if c["op"] == "weights" else e[:, h]
            p = torch.exp(a - given.t()[..., None])
            total = p.sum((0, 1))
            total[:x - n] += weights[row, h, :x - n]
            weights[row, h, :x] = total
            if c["op"] == "step":
                v = _stored(s["v_pool"].view(-1, Hkv, D)[slot, h], fp8, V_SCALE if fp8 else 1.0)
                o[:, h] = torch.matmul(p, v).transpose(0, 1)
        outs.append(o.view(n, Hq, D))
        lses.append(e.view(n, Hq))
        at += n
    if c["op"] == "weights":
        return {"weights": weights}
    return {"out": torch.cat(outs), "lse": torch.cat(lses), "weights": weights}
