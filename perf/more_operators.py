"""What is measured of the operators around a paged KV cache held in 4 bits, and of moving pages.

Four kinds of calls, each with a plain form in elementary torch operations and the call a user makes:

- ``write``: new K / V rows quantised to 4-bit codes with a scale and a minimum per group of 32 columns,
  scattered through the slot mapping, and the rows a slot mapping names read back in bf16;
- ``rope``: per-head RMS norm of q and k, rotation by position and the 4-bit write in one pass;
- ``step``: attention of one flat ragged step over the 4-bit pools (single tokens, a few tokens,
  chunks, mixed);
- ``pages``: pages copied to other places of the pools of all layers in one call, what a fork's first
  write and a compaction of the pool need.

A pool is [num_blocks, Hkv, block_size * (D/2 + D/8)] bytes: per block and head the codes of its tokens
(D/2 bytes each), then their group parameters, (scale, minimum) in bf16. Code n of 8 of word
(c * D/32 + g) of a K row belongs to column 32 g + 8 c + n, code n of 4 of half-word (r * D/32 + g) of a
V row to column 32 g + 4 r + n. A code u stands for scale * u + minimum.

Shapes are those of the repository's workloads: 32 / 8 or 64 / 8 heads of 128 (and small ones of
64), blocks of 8 to 64, lognormal or long-tailed contexts, 512-row chunks.
"""
import math
import random

import torch

own = False

DEV = "cuda"
GROUP = 32


# ---------------------------------------------------------------------------------- the cases

def listed():
    return [
        # a decode batch's new rows, strided parts of one projection
        dict(name="write_decode", op="write", T=64, Hkv=8, D=128, bs=16),
        # a long prompt's rows
        dict(name="write_prompt", op="write", T=16384, Hkv=8, D=128, bs=16),
        # one sequence generating: the smallest call
        dict(name="rope_one_token", op="rope", T=1, Hq=32, Hkv=8, D=128, bs=16, rot=128, inter=False, norm=True),
        # a prompt through norm, rotation and write
        dict(name="rope_prompt", op="rope", T=8192, Hq=32, Hkv=8, D=128, bs=16, rot=128, inter=False, norm=True),
        # one long sequence decoding
        dict(name="step_one", op="step", kind="fixed", B=1, n_q=1, lo=16001, hi=16001, chunks=0, lens=1, Hq=32, Hkv=8, D=128, bs=16),
        # the decode batch (lognormal contexts, median 2048)
        dict(name="step_decode", op="step", kind="lognormal", B=64, n_q=1, lo=2048, hi=16384, chunks=0, lens=2, Hq=32, Hkv=8, D=128, bs=16),
        # long-tailed contexts, groups of 8 query heads
        dict(name="step_tail", op="step", kind="tail", B=32, n_q=1, lo=1024, hi=40000, chunks=0, lens=3, Hq=64, Hkv=8, D=128, bs=32),
        # four drafted tokens per sequence checked at once, heads of 64
        dict(name="step_draft_d64", op="step", kind="uniform", B=12, n_q=4, lo=700, hi=6000, chunks=0, lens=4, Hq=16, Hkv=4, D=64, bs=8),
        # chunked prefill: 512-row segments behind prior tokens
        dict(name="step_chunks", op="step", kind="uniform", B=4, n_q=512, lo=600, hi=9512, chunks=4, lens=5, Hq=32, Hkv=8, D=128, bs=16),
        # decode rows and one ragged chunk in one flat step
        dict(name="step_mixed", op="step", kind="uniform", B=33, n_q=257, lo=900, hi=9000, chunks=1, lens=6, Hq=32, Hkv=8, D=128, bs=16),
        # the pages that forked sequences write next, in every layer
        dict(name="pages_fork", op="pages", pools=64, blocks=128, pairs=6, Hkv=8, D=128, bs=16, fp8=False),
        # the upper part of the pools moved into the holes of the lower one
        dict(name="pages_compact", op="pages", pools=16, blocks=3000, pairs=701, Hkv=8, D=128, bs=16, fp8=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "rope", "step", "step", "step", "step", "pages"])
    Hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 4, 8, 16])
    D = rng.choice([64, 128, 128])
    bs = rng.choice([8, 16, 16, 32, 64, 128])
    c = dict(op=op, Hkv=Hkv, D=D, bs=bs)
    if op == "write":
        c.update(T=_log(rng, 1, 9000))
        return c
    if op == "rope":
        c.update(Hq=Hkv * min(g, 8), T=_log(rng, 1, 6000), rot=rng.choice([D, D, D // 2]), inter=rng.random() < 0.5, norm=rng.random() < 0.8)
        return c
    if op == "pages":
        blocks = _log(rng, 16, 1500)
        c.update(Hkv=max(2, Hkv), pools=_log(rng, 2, 48), blocks=blocks, pairs=rng.randint(1, max(1, blocks // 3)), fp8=rng.random() < 0.4)
        c["pools"] = min(c["pools"], max(2, (1 << 30) // (blocks * bs * c["Hkv"] * D * 2)))
        return c
    kind = rng.choice(["single", "single", "few", "chunk", "mixed"])
    if kind == "single":
        n_q, chunks = 1, 0
        hi = _log(rng, 32, 16000)
        B = _log(rng, 1, min(96, max(4, 300000 // hi)))
    elif kind == "few":
        n_q, chunks = rng.randint(2, 12), 0
        hi = _log(rng, 32, 9000)
        B = _log(rng, 1, min(32, max(4, 60000 // hi)))
    else:
        n_q = _log(rng, 13, 512)
        hi = _log(rng, max(64, n_q), 8000)
        chunks = rng.randint(1, 3)
        B = chunks + (_log(rng, 1, 32) if kind == "mixed" else 0)
    c.update(Hq=min(64, Hkv * g), kind="uniform", B=B, n_q=n_q, lo=max(1, hi // rng.choice([1, 2, 16])), hi=hi, chunks=chunks, lens=rng.randrange(1 << 30))
    return c


def _lens(c):
    """Query rows and context of every sequence (fixed by the case): ctx counts the rows. Where there
    are chunks, the last of the sequences bring them and the others single tokens."""
    r = random.Random(c["lens"])
    out = []
    for i in range(c["B"]):
        if c["kind"] == "lognormal":
            x = min(c["hi"], max(16, int(r.lognormvariate(math.log(c["lo"]), 1.0))))
        elif c["kind"] == "tail":
            x = r.randint(c["lo"], 4 * c["lo"]) if i % 10 else r.randint(int(0.4 * c["hi"]), c["hi"])
        else:
            x = r.randint(c["lo"], c["hi"])
        n = c["n_q"] if not c["chunks"] or i >= c["B"] - c["chunks"] else 1
        out.append((min(n, x), x))
    return out


# ------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _row_bytes(D):
    return D // 2 + D // 8


def _to_pool(codes, params):
    """[blocks, bs, Hkv, D/2] and [blocks, bs, Hkv, D/8] bytes -> the pool."""
    b = codes.shape[0]
    h = codes.shape[2]
    return torch.cat([codes.transpose(1, 2).reshape(b, h, -1), params.transpose(1, 2).reshape(b, h, -1)], -1)


def _pool(g, is_v, blocks, bs, Hkv, D):
    """A pool of quantised normal values."""
    parts = []
    n = max(1, (1 << 25) // (bs * Hkv * D))
    for at in range(0, blocks, n):
        parts.append(_to_pool(*_quantise(_randn(g, min(n, blocks - at), bs, Hkv, D).to(torch.bfloat16).float(), is_v)))
    return torch.cat(parts)


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


def prepare(case, seed):
    c = case
    g = _gen(seed)
    s = {"case": c}
    Hkv, D, bs = c["Hkv"], c["D"], c["bs"]
    if own:
        from continuous_batching_gb300 import binding as bd
    if c["op"] == "pages":
        # layers' K and V pools; live pages among them are copied to free ones
        x = _randn(g, c["pools"], c["blocks"], bs, Hkv, D)
        s["all"] = x.to(torch.float8_e4m3fn) if c["fp8"] else x.to(torch.bfloat16)
        ids = torch.randperm(c["blocks"], generator=g, device=DEV)[:2 * c["pairs"]].to(torch.int32)
        s["pairs"] = ids.view(-1, 2).contiguous()
        s["pools"] = list(s["all"].unbind(0))
        return s
    if c["op"] in ("write", "rope"):
        T = c["T"]
        Hq = c.get("Hq", 0)
        packed = _randn(g, T, (Hq + 2 * Hkv) * D).to(torch.bfloat16)
        s["q"] = packed[:, :Hq * D].view(T, Hq, D)
        s["k"] = packed[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        s["v"] = packed[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        nb = -(-T // bs) + 3
        s["slots"] = torch.randperm(nb * bs, generator=g, device=DEV)[:T].to(torch.int32)
        s["k_pool"], s["v_pool"] = _pool(g, False, nb, bs, Hkv, D), _pool(g, True, nb, bs, Hkv, D)
        s["k_out"] = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=DEV)
        s["v_out"] = torch.empty_like(s["k_out"])
        if c["op"] == "rope":
            s["wq"] = (1 + 0.1 * _randn(g, D)).to(torch.bfloat16) if c["norm"] else None
            s["wk"] = (1 + 0.1 * _randn(g, D)).to(torch.bfloat16) if c["norm"] else None
            n = c["rot"] // 2
            s["inv_freq"] = 10000.0 ** (-torch.arange(n, dtype=torch.float64) / n)
            s["freq_dev"] = s["inv_freq"].to(DEV)
            s["pos"] = torch.randint(0, 131072, (T,), generator=g, device=DEV, dtype=torch.int32)
            s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
            if own:
                s["rope"] = bd.pa_rope_pairs(s["inv_freq"].numpy(), device=DEV)
        if own:
            s["shape"] = bd.Shape.make(max(Hq, Hkv), Hkv, D, bs, nb)
        return s
    lens = _lens(c)
    ctxs = [x for _, x in lens]
    nb = sum(-(-x // bs) for x in ctxs) + 2
    s["table_host"] = _table(g, ctxs, bs, nb)
    s["table"] = s["table_host"].to(DEV)
    s["ctx"] = _int(ctxs)
    s["k_pool"], s["v_pool"] = _pool(g, False, nb, bs, Hkv, D), _pool(g, True, nb, bs, Hkv, D)
    cu = [0]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    T = cu[-1]
    s["cu"], s["T"], s["L"] = _int(cu), T, max(ctxs)
    s["q"] = _randn(g, T, c["Hq"], D).to(torch.bfloat16)
    s["out"] = torch.empty(T, c["Hq"], D, dtype=torch.bfloat16, device=DEV)
    # sequences of one or few rows, and chunks
    n_small = c["B"] - c["chunks"]
    s["classes"] = [(a, b) for a, b in ((0, n_small), (n_small, c["B"])) if a < b]
    s["classes"] = [(a, b, max(n for n, _ in lens[a:b]), max(x for _, x in lens[a:b])) for a, b in s["classes"]]
    if own:
        import numpy as np
        sh = s["shape"] = bd.Shape.make(c["Hq"], Hkv, D, bs, nb)
        s["plan"] = bd.pa_plan_step_q4(sh, np.asarray(cu, np.int32), np.asarray(ctxs, np.int32), device=DEV)
        need = bd.pa_q4_workspace_bytes(sh, s["plan"])
        s["ws"] = torch.empty((need + 3) // 4, dtype=torch.float32, device=DEV)
    return s


# ---------------------------------------------------------------------------------- plain forms

def _quantise(x, is_v):
    """[..., D] in 32 bits -> code bytes [..., D/2] and parameter bytes [..., D/8]."""
    D = x.shape[-1]
    G = D // GROUP
    y = x.unflatten(-1, (G, GROUP))
    lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    # (a division by a plain number would be done as a product with its reciprocal)
    scale = ((hi - lo) / torch.full_like(lo, 15)).to(torch.bfloat16)
    step = scale.float()
    u = torch.where(step > 0, torch.round((y - lo) / step.clamp(min=1e-45)).clamp(0, 15), 0).to(torch.uint8)
    n = 4 if is_v else 8
    u = u.unflatten(-1, (GROUP // n, n)).transpose(-3, -2).flatten(-3)
    codes = u[..., 0::2] | (u[..., 1::2] << 4)
    params = torch.cat([scale, lo.to(torch.bfloat16)], -1).contiguous().view(torch.uint8).flatten(-2)
    return codes, params


def _params(b, G):
    """Parameter bytes [..., 4 G] -> scales and minima [..., G, 1] in 32 bits."""
    p = b.contiguous().view(torch.bfloat16).float().unflatten(-1, (G, 2))
    return p[..., :1], p[..., 1:]


def _codes(b, is_v, D):
    """Code bytes [..., D/2] -> the codes of every group in column order [..., G, 32]."""
    n = 4 if is_v else 8
    u = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    return u.unflatten(-1, (GROUP // n, D // GROUP, n)).transpose(-3, -2).flatten(-2)


def _values(codes, params, is_v, D):
    scale, lo = _params(params, D // GROUP)
    return (_codes(codes, is_v, D).float() * scale + lo).flatten(-2)


def _split(pool, c):
    """The pool's code rows [blocks, Hkv, bs, D/2] and parameter rows [blocks, Hkv, bs, D/8]."""
    n = c["bs"] * c["D"] // 2
    return pool[..., :n].unflatten(-1, (c["bs"], -1)), pool[..., n:].unflatten(-1, (c["bs"], -1))


def _plain_write(s, k, v):
    c = s["case"]
    at = s["slots"].long()
    b, o = at // c["bs"], at % c["bs"]
    for name, x in (("k", k), ("v", v)):
        codes, params = _split(s[name + "_pool"], c)
        new_codes, new_params = _quantise(x, name == "v")
        codes[b, :, o], params[b, :, o] = new_codes, new_params


def _plain_read(s):
    c = s["case"]
    at = s["slots"].long()
    b, o = at // c["bs"], at % c["bs"]
    for name in "kv":
        codes, params = _split(s[name + "_pool"], c)
        s[name + "_out"].copy_(_values(codes[b, :, o], params[b, :, o], name == "v", c["D"]))


def _plain_turn(s):
    c = s["case"]
    r, n = c["rot"], c["rot"] // 2
    a = s["pos"].double()[:, None] * s["freq_dev"]
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
    return turn(s["k"], s["wk"]).to(torch.bfloat16).float()


def _plain_attend(s, a, b, n, L):
    """Attention of sequences a .. b - 1, padded to n query rows and L keys."""
    c = s["case"]
    Hkv, g, D, bs = c["Hkv"], c["Hq"] // c["Hkv"], c["D"], c["bs"]
    blocks = s["table"][a:b, :-(-L // bs)].clamp(min=0).long()

    def gathered(name):
        codes, params = _split(s[name + "_pool"][blocks], c)
        return _values(codes, params, name == "v", D).transpose(1, 2).flatten(2, 3)

    k = gathered("k")                              # [b - a, Hkv, keys, D]
    cu, ctx = s["cu"].long(), s["ctx"][a:b].long()
    i = torch.arange(n, device=DEV)
    first, n_q = cu[a:b], cu[a + 1:b + 1] - cu[a:b]
    real = i < n_q[:, None]
    at = (first[:, None] + i).clamp(max=s["T"] - 1)
    q = s["q"].float()[at].view(b - a, n, Hkv, g, D)
    x = torch.einsum("bnhgd,bhld->bhgnl", q, k) * (1 / math.sqrt(D))
    pos = (ctx - n_q)[:, None] + i
    seen = (torch.arange(k.shape[2], device=DEV) <= pos[..., None]) & real[..., None]
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(x - m)
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = torch.einsum("bhgnl,bhld->bnhgd", p, gathered("v"))
    s["out"][at[real]] = o.reshape(b - a, n, c["Hq"], D)[real].to(torch.bfloat16)


def run(state):
    s = state
    c = s["case"]
    if own:
        from continuous_batching_gb300 import binding as bd
    if c["op"] == "pages":
        if own:
            bd.paged_copy_pages(s["pairs"], s["pools"])
        else:
            pairs = s["pairs"].long()
            s["all"][:, pairs[:, 1]] = s["all"][:, pairs[:, 0]]
        return {"pools": s["all"]}
    if c["op"] in ("write", "rope"):
        if own and c["op"] == "write":
            bd.paged_kv_write_q4(s["k"], s["v"], s["slots"], s["k_pool"], s["v_pool"], s["shape"])
        elif own:
            bd.paged_qk_norm_rope_write_q4(s["q"], s["k"], s["v"], s["wq"], s["wk"], 1e-6, s["rope"], s["pos"], s["slots"], s["q_out"], s["k_pool"], s["v_pool"], s["shape"], interleaved=c["inter"])
        else:
            _plain_write(s, s["k"].float() if c["op"] == "write" else _plain_turn(s), s["v"].float())
        if own:
            bd.paged_kv_read_q4(s["slots"], s["k_pool"], s["v_pool"], s["k_out"], s["v_out"], s["shape"])
        else:
            _plain_read(s)
        out = {"k": s["k_out"], "v": s["v_out"]}
        if c["op"] == "rope":
            out["q"] = s["q_out"]
        return out
    if own:
        bd.paged_attention_step_q4(s["q"], s["k_pool"], s["v_pool"], s["table"], s["cu"], s["ctx"], s["plan"], s["ws"], s["out"], s["shape"])
    else:
        for part in s["classes"]:
            _plain_attend(s, *part)
    return {"out": s["out"]}


# ----------------------------------------------------------------------------------- the work

def work(case):
    c = case
    Hkv, D, bs = c["Hkv"], c["D"], c["bs"]
    if c["op"] == "pages":
        return {"bytes": 2 * c["pools"] * c["pairs"] * bs * Hkv * D * (1 if c["fp8"] else 2) + 8 * c["pairs"], "flops": 0}
    if c["op"] in ("write", "rope"):
        T, Hq = c["T"], c.get("Hq", 0)
        # rows in, codes out; codes in again, rows out
        n = T * Hkv * 2 * (2 * D * 2 + 2 * _row_bytes(D)) + 8 * T
        return {"bytes": n + T * Hq * D * 4 + (4 * T if Hq else 0), "flops": T * (Hq + Hkv) * D * 7 if Hq else 0}
    lens = _lens(c)
    Hq = c["Hq"]
    T = sum(n for n, _ in lens)
    pairs = sum(n * (x - n) + n * (n + 1) // 2 for n, x in lens)
    return {"bytes": sum(x for _, x in lens) * Hkv * 2 * _row_bytes(D) + 2 * T * Hq * D * 2, "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------------- the definition, in 64 bits

def _bf16(x):
    """The nearest bf16 number, ties to even, in 64 bits."""
    b = x.contiguous().view(torch.int64)
    return (b + (1 << 44) - 1 + ((b >> 45) & 1) >> 45 << 45).view(torch.float64)


def _held(x):
    """What a cache in 4 bits holds of [..., D] and gives back in bf16."""
    y = x.unflatten(-1, (-1, GROUP))
    lo, hi = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
    step = _bf16((hi - lo) / 15)
    u = torch.round((y - lo) / step).clamp(0, 15)
    return _bf16(torch.where(step == 0, lo, lo + u * step).flatten(-2))


def _decoded(pool, slot, h, c, is_v):
    """Rows `slot` of head h of a pool in 64 bits, by the layout's formula."""
    D, bs = c["D"], c["bs"]
    G = D // GROUP
    col = torch.arange(D, device=DEV)
    g, e = col // 32, col % 32
    nibble = ((e // 4) * G + g) * 4 + e % 4 if is_v else ((e // 8) * G + g) * 8 + e % 8
    rows = pool[slot // bs, h]
    at = (slot % bs)[:, None]
    byte = rows.gather(1, at * (D // 2) + nibble // 2)
    u = (byte >> (4 * (nibble % 2)).to(torch.uint8)) & 15
    p = bs * D // 2 + at * (D // 8) + 4 * g
    word = [rows.gather(1, p + i).long() for i in range(4)]
    scale, lo = ((word[i] + 256 * word[i + 1] << 16).int().view(torch.float32).double() for i in (0, 2))
    return u.double() * scale + lo


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    Hkv, D, bs = c["Hkv"], c["D"], c["bs"]
    if c["op"] == "pages":
        out = s["all"].double()
        for a, b in s["pairs"].tolist():
            out[:, b] = out[:, a]
        return {"pools": out}
    if c["op"] == "write":
        return {"k": _held(s["k"].double()), "v": _held(s["v"].double())}
    if c["op"] == "rope":
        half = c["rot"] // 2
        angle = s["pos"].double()[:, None] * s["inv_freq"].to(DEV)
        turned = torch.polar(torch.ones_like(angle), angle)

        def rotated(x, w):
            y = x.double()
            if w is not None:
                y = y / (y.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
            first = torch.arange(0, c["rot"], 2, device=DEV) if c["inter"] else torch.arange(half, device=DEV)
            second = first + (1 if c["inter"] else half)
            z = torch.complex(y[..., first], y[..., second]) * turned[:, None]
            y = y.clone()
            y[..., first], y[..., second] = z.real, z.imag
            return y

        return {"q": rotated(s["q"], s["wq"]), "k": _held(_bf16(rotated(s["k"], s["wk"]))), "v": _held(s["v"].double())}
    Hq, g = c["Hq"], c["Hq"] // Hkv
    table = s["table_host"].long().to(DEV)
    outs, at = [], 0
    for b, (n, x) in enumerate(_lens(c)):
        slot = table[b].repeat_interleave(bs)[:x] * bs + torch.arange(x, device=DEV) % bs
        q = s["q"][at:at + n].double().view(n, Hkv, g, D)
        later = torch.arange(x, device=DEV) > torch.arange(x - n, x, device=DEV)[:, None]
        o = torch.empty(n, Hkv, g, D, dtype=torch.float64, device=DEV)
        for h in range(Hkv):
            w = torch.matmul(q[:, h].transpose(0, 1), _decoded(s["k_pool"], slot, h, c, False).t()) / math.sqrt(D)
            w[:, later] = -math.inf
            w = torch.exp(w - torch.logsumexp(w, -1, keepdim=True))
            o[:, h] = torch.matmul(w, _decoded(s["v_pool"], slot, h, c, True)).transpose(0, 1)
        outs.append(o.view(n, Hq, D))
        at += n
    return {"out": torch.cat(outs)}
