"""Per-head norm, rotation and KV write: pins of the definition and refusals (CPU), and the kernel
against the fp64 definition (GPU)."""
import numpy as np
import pytest

import oracle.fp8 as ofp8
import oracle.paged_attention as pa
from continuous_batching_gb300 import binding as bd
from continuous_batching_gb300 import workloads as wl
from oracle.bounded import norm_rope

torch = pytest.importorskip("torch")


# ------------------------------------------------------------------ the definition (CPU)

def test_definition_against_complex_rotation_and_closed_forms():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 16))
    f = np.array([1.0, 0.3, 0.02, 0.001])
    pos = np.array([[0, 1, 7, 1000, 65537], [3, 2, 1, 0, -5]])
    axes = [0, 1, 0, 1]
    for inter in (False, True):
        y, _ = norm_rope(x, None, 0.0, f, axes, pos, inter)
        u = x[..., 0:8:2] if inter else x[..., :4]
        v = x[..., 1:8:2] if inter else x[..., 4:8]
        z = (u + 1j * v) * np.exp(1j * np.stack([pos[a] * w for a, w in zip(axes, f)], -1))[:, None]
        got = (y[..., 0:8:2] + 1j * y[..., 1:8:2]) if inter else y[..., :4] + 1j * y[..., 4:8]
        np.testing.assert_allclose(got, z, atol=1e-12)
        np.testing.assert_array_equal(y[..., 8:], x[..., 8:])       # untouched columns
        # a rotation keeps the product of two rows that are equally far apart
        np.testing.assert_allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
    y, _ = norm_rope(x, np.full(16, 2.0), 0.0, f[:0], [], pos, False)
    np.testing.assert_allclose((y ** 2).mean(-1), 4.0)


def test_pairs_hold_the_fraction_of_a_turn():
    f = np.array([1.0, 1e-4, 0.0, -0.25, 2 * np.pi, 100.0, -1e-30, 2.5])
    p = bd.pa_rope_pairs(f, np.arange(8) % 3)
    assert p["axis"].tolist() == [0, 1, 2, 0, 1, 2, 0, 1]
    for i in range(8):
        turns = float(f[i]) / (2 * np.pi)
        got = int(p["step"][i]) / 2.0 ** 64
        d = (got - turns) % 1.0
        assert min(d, 1 - d) <= 2.0 ** -53 * max(1.0, abs(turns)) * 4, i
    assert int(p["step"][2]) == 0


def test_pair_refusals():
    with pytest.raises(bd.PagedAttnError):
        bd.pa_rope_pairs([1.0, np.nan])
    with pytest.raises(bd.PagedAttnError):
        bd.pa_rope_pairs([1.0, np.inf])
    with pytest.raises(bd.PagedAttnError):
        bd.pa_rope_pairs([1.0, 1.0], [0, 2], n_axes=2)
    with pytest.raises(bd.PagedAttnError):
        bd.pa_rope_pairs([1.0, 1.0], [0, -1], n_axes=2)
    with pytest.raises(ValueError):
        bd.pa_rope_pairs([1.0, 1.0], [0])
    assert len(bd.pa_rope_pairs([])) == 0


def _call(**kw):
    """The C entry with addresses that are never read: every refusal comes before a launch."""
    a = dict(q=16, qs=512, k=16, ks=256, v=16, vs=256, wq=16, wk=16, eps=1e-6, rope=16, n=32, inter=0,
             pos=16, axes=1, slots=16, T=4, out=32, kp=16, vp=16)
    shape = kw.pop("shape", bd.Shape.make(4, 2, 128, 16, 8))
    scales = kw.pop("scales", None)
    a.update(kw)
    f = bd.load().paged_qk_norm_rope_write if scales is None else bd.load().paged_qk_norm_rope_write_fp8
    return f(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["wq"], a["wk"], a["eps"], a["rope"],
             a["n"], a["inter"], a["pos"], a["axes"], a["slots"], a["T"], a["out"], a["kp"], a["vp"],
             *(scales or ()), shape, None, None)


@pytest.mark.parametrize("kw, want", [
    (dict(T=-1), bd.PA_ERR_INVALID), (dict(T=0), bd.PA_OK), (dict(eps=-1.0), bd.PA_ERR_INVALID),
    (dict(eps=float("nan")), bd.PA_ERR_INVALID), (dict(n=3), bd.PA_ERR_SHAPE),
    (dict(n=68), bd.PA_ERR_SHAPE), (dict(n=-4), bd.PA_ERR_SHAPE), (dict(q=None), bd.PA_ERR_INVALID),
    (dict(kp=None), bd.PA_ERR_INVALID), (dict(slots=None), bd.PA_ERR_INVALID),
    (dict(pos=None), bd.PA_ERR_INVALID), (dict(rope=None), bd.PA_ERR_INVALID),
    (dict(axes=0), bd.PA_ERR_INVALID), (dict(qs=504), bd.PA_ERR_INVALID),
    (dict(ks=260), bd.PA_ERR_INVALID), (dict(vs=128), bd.PA_ERR_INVALID),
    (dict(q=24), bd.PA_ERR_INVALID), (dict(wq=8), bd.PA_ERR_INVALID), (dict(vp=8), bd.PA_ERR_INVALID),
    (dict(q=32, qs=1024), bd.PA_ERR_INVALID),                     # in place over another layout
    (dict(shape=bd.Shape.make(4, 2, 96, 16, 8)), bd.PA_ERR_SHAPE),
    (dict(scales=(0.0, 1.0)), bd.PA_ERR_INVALID), (dict(scales=(1.0, float("inf"))), bd.PA_ERR_INVALID),
])
def test_refusals(kw, want):
    assert _call(**kw) == want


# ------------------------------------------------------------------ the kernel (GPU)

def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def _f64(t):
    return pa.bf16_to_f64(_bits(t))


HALF = torch.finfo(torch.bfloat16).eps / 2     # relative half step
HALF8 = 2.0 ** -4                              # e4m3; its smallest half step is 2^-10
# fp32 in between, relative to the sum of magnitudes that meet in an element, in units of 2^-24:
# the mean of squares (128 terms in a tree over lanes of 8: <= 12 roundings, halved by the square
# root) 6, rsqrt 4, its product with weight and value 2, sine and cosine 4, their argument
# (2^-25 of a half turn: 1.6 in radians) 2, the rotation 3
F32 = 24 * 2.0 ** -24


def _check(Hq, Hkv, D, bs, T, n_pairs, n_axes, inter, norm, fp8, packed, far=131072, in_place=False,
           seed=0):
    rng = np.random.default_rng(seed)
    dev = "cuda"
    width = (Hq + 2 * Hkv) * D
    src = torch.from_numpy(rng.standard_normal((T, width)).astype(np.float32)).to(dev).to(torch.bfloat16)
    if packed:
        q, k, v = src[:, :Hq * D], src[:, Hq * D:(Hq + Hkv) * D], src[:, (Hq + Hkv) * D:]
        q, k, v = q.view(T, Hq, D), k.view(T, Hkv, D), v.view(T, Hkv, D)
    else:
        q = src[:, :Hq * D].reshape(T, Hq, D).contiguous()
        k = src[:, Hq * D:(Hq + Hkv) * D].reshape(T, Hkv, D).contiguous()
        v = src[:, (Hq + Hkv) * D:].reshape(T, Hkv, D).contiguous()
    wq, wk = [(1 + 0.3 * torch.randn(D, device=dev)).to(torch.bfloat16) if norm else None for _ in "qk"]
    nb = T // bs + 2
    slots = rng.permutation(nb * bs)[:T].astype(np.int32)
    slots[rng.random(T) < 0.1] = -1                                  # rows that write nothing
    f = 10000.0 ** (-np.arange(n_pairs) / max(n_pairs, 1))
    axes = rng.integers(0, n_axes, n_pairs).astype(np.int32)
    pos = rng.integers(-far if far > 0 else 0, abs(far) + 1, (n_axes, T)).astype(np.int32)
    rope = bd.pa_rope_pairs(f, axes, n_axes, device=dev) if n_pairs else None
    shape = bd.Shape.make(Hq, Hkv, D, bs, nb)
    e = torch.uint8 if fp8 else torch.bfloat16
    kp0 = torch.randint(0, 120, (nb, bs, Hkv, D), device=dev, dtype=torch.uint8) if fp8 else \
        torch.randn(nb, bs, Hkv, D, device=dev).to(e)
    vp0 = kp0.flip(0).clone()
    kp, vp = kp0.clone(), vp0.clone()
    q64, k64 = _f64(q), _f64(k)
    out = q if in_place else torch.full((T, Hq, D), float("nan"), dtype=torch.bfloat16, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    ks, vs = 0.013, 0.009
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    args = (q, k, v, wq, wk, 1e-5, rope, d(pos) if n_pairs else None, d(slots), out, kp, vp)
    if fp8:
        bd.paged_qk_norm_rope_write_fp8(*args, ks, vs, shape, interleaved=inter, err=err)
    else:
        bd.paged_qk_norm_rope_write(*args, shape, interleaved=inter, err=err)
    assert int(err.item()) == 0
    w64 = [None if w is None else _f64(w) for w in (wq, wk)]
    y, mag = norm_rope(q64, w64[0], 1e-5, f, axes, pos, inter)
    # the table's frequencies and the definition's products are doubles: their angles differ by
    # up to 2^-52 of |position * frequency|
    angle = float(np.abs(pos).max(initial=0)) * float(np.abs(f).max(initial=0)) * 2.0 ** -51
    slack = F32 + angle
    assert np.all(np.abs(_f64(out) - y) <= HALF * np.abs(y) + (1 + HALF) * slack * mag + 1e-38)
    yk, magk = norm_rope(k64, w64[1], 1e-5, f, axes, pos, inter)
    w = slots >= 0
    if fp8:
        got = ofp8.decode_e4m3(kp.cpu().numpy()).reshape(-1, Hkv, D)[slots[w]]
        x, m = yk[w] / np.float64(np.float32(ks)), magk[w] / ks
        lim = np.clip(x, -448, 448)
        assert np.all(np.abs(got - lim) <= np.maximum(HALF8 * np.abs(x), 2.0 ** -10) +
                      (1 + HALF8) * (slack + 2.0 ** -24) * m)
        ref_k, ref_v = kp0.clone(), vp0.clone()
        bd.paged_kv_write_fp8(k.contiguous(), v.contiguous(), d(slots), ref_k, ref_v, ks, vs, shape)
    else:
        got = pa.bf16_to_f64(_bits(kp)).reshape(-1, Hkv, D)[slots[w]]
        assert np.all(np.abs(got - yk[w]) <= HALF * np.abs(yk[w]) + (1 + HALF) * slack * magk[w] + 1e-38)
        ref_k, ref_v = kp0.clone(), vp0.clone()
        bd.paged_kv_write(k.contiguous(), v.contiguous(), d(slots), ref_k, ref_v, shape)
    as_int = lambda t: t.view(torch.uint8 if fp8 else torch.int16)
    assert torch.equal(as_int(vp), as_int(ref_v))                   # v goes the plain write's way
    rest = np.setdiff1d(np.arange(nb * bs), slots[w])
    flat = lambda t: as_int(t).view(nb * bs, -1).cpu().numpy()[rest]
    assert np.array_equal(flat(kp), flat(kp0))                      # other slots as they were
    if n_pairs == 0 and not norm:
        assert torch.equal(as_int(kp), as_int(ref_k))               # nothing to do: a plain write


@pytest.mark.gpu
@pytest.mark.parametrize("Hq, Hkv, D, bs, T, n_pairs, n_axes, inter, norm, fp8, packed", [
    (32, 8, 128, 16, 1, 64, 1, False, True, False, True),
    (32, 8, 128, 16, 33, 64, 1, True, True, False, True),
    (64, 8, 128, 32, 128, 64, 3, False, True, False, False),
    (4, 2, 64, 16, 5, 32, 1, False, True, False, False),
    (4, 2, 64, 16, 77, 32, 2, True, False, False, True),
    (4, 2, 64, 8, 64, 16, 1, False, True, False, True),             # half of the columns turn
    (8, 8, 128, 64, 19, 32, 3, True, True, False, True),
    (1, 1, 64, 8, 5000, 32, 1, False, True, False, True),           # several tokens per CTA
    (1, 1, 128, 8, 5001, 64, 1, True, True, True, True),
    (2, 1, 128, 16, 40, 4, 1, False, False, False, False),
    (16, 1, 128, 128, 31, 0, 1, False, True, False, True),          # norm only
    (16, 2, 64, 128, 31, 0, 1, False, False, False, True),          # neither: the plain write
    (16, 2, 64, 16, 31, 0, 1, True, False, True, True),
    (32, 8, 128, 16, 70, 64, 3, False, True, True, True),
    (32, 8, 128, 16, 2, 48, 2, True, True, True, False),
])
def test_against_the_definition(Hq, Hkv, D, bs, T, n_pairs, n_axes, inter, norm, fp8, packed):
    _check(Hq, Hkv, D, bs, T, n_pairs, n_axes, inter, norm, fp8, packed)


@pytest.mark.gpu
@pytest.mark.parametrize("far", [0, 2 ** 24, 2 ** 31 - 1])
def test_far_positions(far):
    _check(4, 2, 128, 16, 64, 64, 2, False, True, False, False, far=far, seed=3)


@pytest.mark.gpu
def test_in_place():
    _check(8, 2, 128, 16, 50, 64, 1, False, True, False, False, in_place=True)
    _check(8, 2, 64, 16, 50, 32, 1, True, True, False, False, in_place=True)


@pytest.mark.gpu
def test_bad_slots_axes_and_large_values():
    dev = "cuda"
    shape = bd.Shape.make(2, 2, 64, 16, 2)
    T = 4
    big = torch.full((T, 2, 64), 3e38, device=dev).to(torch.bfloat16)
    rope = bd.pa_rope_pairs(np.ones(32), np.full(32, 2), n_axes=3, device=dev)
    kp = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device=dev)
    vp = kp.clone()
    out = torch.zeros(T, 2, 64, dtype=torch.bfloat16, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    pos = torch.zeros(1, T, dtype=torch.int32, device=dev)
    slots = torch.tensor([0, 32, 2 ** 31 - 1, -7], dtype=torch.int32, device=dev)
    bd.paged_qk_norm_rope_write(big, big, big, None, None, 0.0, rope, pos, slots, out, kp, vp, shape, err=err)
    assert int(err.item()) == bd.PA_DEVERR_SLOT | bd.PA_DEVERR_META
    assert torch.equal(out, big)                                    # position 0 turns nothing
    assert torch.equal(kp.view(-1, 2, 64)[0], big[0]) and not kp.view(-1, 2, 64)[1:].any()
    assert torch.equal(vp.view(-1, 2, 64)[0], big[0]) and not vp.view(-1, 2, 64)[1:].any()


@pytest.mark.gpu
def test_binding_refusals_streams_and_graphs():
    dev = "cuda"
    shape = bd.Shape.make(4, 2, 64, 16, 4)
    T = 6
    mk = lambda h: torch.randn(T, h, 64, device=dev).to(torch.bfloat16)
    q, k, v = mk(4), mk(2), mk(2)
    kp, vp = (torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device=dev) for _ in "kv")
    out = torch.empty_like(q)
    slots = torch.arange(T, dtype=torch.int32, device=dev)
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    rope = bd.pa_rope_pairs(np.ones(32), device=dev)
    ok = lambda **kw: bd.paged_qk_norm_rope_write(*[kw.get(n, d) for n, d in (
        ("q", q), ("k", k), ("v", v), ("wq", None), ("wk", None), ("eps", 1e-6), ("rope", rope),
        ("pos", pos), ("slots", slots), ("out", out), ("kp", kp), ("vp", vp), ("shape", shape))],
        stream=kw.get("stream"))
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q.transpose(0, 1)), dict(k=mk(4)),
                dict(pos=pos.long()), dict(pos=pos[:3]), dict(pos=None), dict(slots=slots.long()),
                dict(out=out.float()), dict(kp=kp[:2]), dict(kp=kp.view(torch.uint8)),
                dict(wq=torch.ones(64, device=dev)), dict(rope=rope[:, :1])):
        with pytest.raises(ValueError):
            ok(**bad)
    ok()
    torch.cuda.synchronize()
    want, want_k = out.clone(), kp.clone()
    out.zero_(), kp.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ok(stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(kp, want_k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ok()
    out.zero_(), kp.zero_()
    q.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want * 2) and torch.equal(kp, want_k)


def _turn_digits(bits):
    """2 pi in units of 2^-bits, from Machin's formula."""
    one = 1 << (bits + 32)

    def arctan_of_inverse(n):
        total, term, k = 0, one // n, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total

    return 2 * (16 * arctan_of_inverse(5) - 4 * arctan_of_inverse(239)) >> 32


def test_pairs_are_the_nearest_of_their_unit():
    """A step is f / 2 pi turns, rounded once to units of 2^-64 turn: the quotient is known to more bits
    than a double's, so a far position's phase is off by the step's half unit times the position."""
    rng = np.random.default_rng(0)
    f = np.concatenate([10000.0 ** (-np.arange(64) / 64), [1.0, -1.0, 0.5, 2 * np.pi, -2 * np.pi, 6.25, 100.0, 1e6, 1e-19,
                                                           -1e-19, 0.0, 5e-324, -5e-324], rng.standard_normal(200)])
    bits = 1200
    turn = _turn_digits(bits)
    got = bd.pa_rope_pairs(f)["step"]
    for x, step in zip(f.tolist(), got.tolist()):
        m, d = x.as_integer_ratio()
        want = (m << (bits + 64 + 20)) // (d * turn)             # turns in units of 2^-84
        off = ((step << 20) - want) % (1 << 84)
        off = min(off, (1 << 84) - off)
        # half a unit, and what a double-double quotient leaves of it (2^-100 of the turns)
        assert off <= (1 << 19) + 2 + abs(want) // (1 << 100), (x, off / 2 ** 20)
