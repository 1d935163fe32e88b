"""The 4-bit cache's write, read and norm + rotation + write: bytes and values against the definition, on
the CPU the definition itself and the refusals."""
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


# ------------------------------------------------------------------------------- definition

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("is_v", [False, True])
def test_bytes_hold_the_quantised_values(D, is_v):
    rng = np.random.default_rng(3)
    bits = wl.random_bf16(rng, (7, 2, D))
    bits[0, 0, :32] = bits[0, 0, 0]                       # a constant group: scale 0
    slots = np.array([9, 3, -1, 31, 0, 16, 15])
    pool = q4.write(q4.empty_pool(4, 2, 8, D), bits, slots, 8, is_v)
    vals = q4.values(pool, 8, D, is_v).reshape(32, 2, D)
    u, scale, low = q4.quantise(bits)
    for t, s in enumerate(slots):
        if s < 0:
            continue
        x = pa.bf16_to_f64(bits[t])
        step = np.repeat(pa.bf16_to_f64(scale[t]), 32, -1)
        # rounding to the nearest code: half a step; the scale's own rounding (2^-8 of it) over up to 15 steps
        # adds at most 15 * 2^-8 / 2 behind the last code where the scale was rounded down
        assert np.all(np.abs(vals[s] - x) <= (0.5 + 15 * 2.0 ** -8) * step + 1e-30)
    assert np.array_equal(vals[9, 0, :32], np.full(32, pa.bf16_to_f64(bits[0, 0, 0])))
    assert sorted(q4.column_nibble(D, is_v).tolist()) == list(range(D))


def test_groups_that_hold_no_numbers_read_as_nan():
    bits = wl.random_bf16(np.random.default_rng(4), (5, 1, 64))
    for t, b in enumerate([0x7FC0, 0x7F80, 0xFF80]):      # NaN, +inf, -inf
        bits[t, 0, 40] = b
    bits[3, 0, 0], bits[3, 0, 1] = 0x7F7F, 0xFF7F         # the range passes fp32
    vals = q4.values(q4.write(q4.empty_pool(1, 1, 8, 64), bits, range(5), 8, False), 8, 64, False)[0, :, 0]
    for t in range(3):
        assert np.isnan(vals[t, 32:]).all() and np.isfinite(vals[t, :32]).all()
    assert np.isnan(vals[3, :32]).all() and np.isfinite(vals[4]).all()


# --------------------------------------------------------------------------------- refusals

def _write(lib, **kw):
    a = dict(k=4096, ks=256, v=4096, vs=256, slots=4096, T=4, kp=4096, vp=4096, shape=bd.Shape.make(8, 2, 128, 16, 4))
    a.update(kw)
    return lib.paged_kv_write_q4(a["k"], a["ks"], a["v"], a["vs"], a["slots"], a["T"], a["kp"], a["vp"], C.byref(a["shape"]), None, None)


@pytest.mark.parametrize("kw, status", [
    (dict(T=-1), bd.PA_ERR_INVALID), (dict(k=None), bd.PA_ERR_INVALID), (dict(v=4104), bd.PA_ERR_INVALID),
    (dict(kp=4100), bd.PA_ERR_INVALID), (dict(ks=248), bd.PA_ERR_INVALID), (dict(vs=260), bd.PA_ERR_INVALID),
    (dict(slots=None), bd.PA_ERR_INVALID), (dict(shape=bd.Shape.make(8, 2, 96, 16, 4)), bd.PA_ERR_SHAPE),
    (dict(shape=bd.Shape.make(8, 2, 128, 24, 4)), bd.PA_ERR_SHAPE), (dict(T=0, k=None), bd.PA_OK)])
def test_write_refuses(kw, status):
    assert _write(bd.load(), **kw) == status


def test_read_refuses():
    lib, sh = bd.load(), bd.Shape.make(8, 2, 128, 16, 4)
    call = lambda slots=4096, T=4, kp=4096, vp=4096, ko=4096, vo=4096: lib.paged_kv_read_q4(slots, T, kp, vp, ko, vo, C.byref(sh), None, None)
    assert call(T=-2) == bd.PA_ERR_INVALID and call(ko=None) == bd.PA_ERR_INVALID and call(vo=4098) == bd.PA_ERR_INVALID
    assert call(kp=None) == bd.PA_ERR_INVALID and call(slots=None) == bd.PA_ERR_INVALID and call(T=0, slots=None) == bd.PA_OK


# -------------------------------------------------------------------------------------- GPU

def pools(rng, nb, Hkv, bs, D):
    return [dev(rng.integers(0, 256, (nb, Hkv, bs * (D // 2 + D // 8)), dtype=np.uint8)) for _ in "kv"]


@pytest.mark.gpu
@pytest.mark.parametrize("T, Hkv, D, bs", [(1, 1, 128, 8), (1, 8, 64, 16), (37, 8, 128, 16), (64, 3, 64, 128), (301, 2, 128, 64), (2048, 8, 128, 32)])
def test_write_and_read_are_the_definition(T, Hkv, D, bs):
    """Every byte of the pools, those of tokens that were not written among them, and every value read."""
    rng = np.random.default_rng(T + D)
    nb = -(-T // bs) + 2
    sh = bd.Shape.make(Hkv, Hkv, D, bs, nb)
    k, v = (wl.random_bf16(rng, (T, Hkv, D)) for _ in "kv")
    k[0, 0, 1:32] = k[0, 0, 0]                            # a constant group
    v[T // 2, 0, 5] = 0x7F80                              # an infinity
    k[T // 2, 0, 6] = 0x7FC1                              # a NaN
    k[-1, -1, 32:64] = wl.f32_to_bf16_bits(np.float32(100) + np.arange(32, dtype=np.float32) / 8)
    slots = rng.permutation(nb * bs)[:T].astype(np.int32)
    if T > 8:
        slots[rng.integers(0, T, 3)] = -1
    kp, vp = pools(rng, nb, Hkv, bs, D)
    k0, v0 = kp.cpu().numpy(), vp.cpu().numpy()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bd.paged_kv_write_q4(bf16(k), bf16(v), dev(slots), kp, vp, sh, err=err)
    k1, v1 = q4.write(k0, k, slots, bs, False), q4.write(v0, v, slots, bs, True)
    assert np.array_equal(kp.cpu().numpy(), k1) and np.array_equal(vp.cpu().numpy(), v1)
    ko, vo = (torch.full((T, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    bd.paged_kv_read_q4(dev(slots), kp, vp, ko, vo, sh, err=err)
    on = slots >= 0
    for got, pool, is_v in ((ko, k1, False), (vo, v1, True)):
        want = q4.values(pool, bs, D, is_v).reshape(nb * bs, Hkv, D)[slots]
        want = pa.bf16_to_f64(q4._to_bf16_bits(want))
        got = pa.bf16_to_f64(bits_of(got))
        assert np.array_equal(got[on], want[on], equal_nan=True) and np.all(got[~on] == 7.0)
    assert int(err.item()) == 0


@pytest.mark.gpu
def test_strided_rows_and_slots_outside_the_pool():
    rng = np.random.default_rng(8)
    T, Hkv, D, bs, nb = 21, 2, 128, 16, 3
    sh = bd.Shape.make(4, Hkv, D, bs, nb)
    packed = wl.random_bf16(rng, (T, 8, D))
    slots = rng.permutation(nb * bs)[:T].astype(np.int32)
    kp, vp = pools(rng, nb, Hkv, bs, D)
    k0, v0 = kp.cpu().numpy(), vp.cpu().numpy()
    x = bf16(packed)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots[4], slots[9] = nb * bs, 2 ** 31 - 1
    bd.paged_kv_write_q4(x[:, 4:6], x[:, 6:], dev(slots), kp, vp, sh, err=err)
    assert int(err.item()) == bd.PA_DEVERR_SLOT
    inside = np.where(slots < nb * bs, slots, -1)
    assert np.array_equal(kp.cpu().numpy(), q4.write(k0, packed[:, 4:6], inside, bs, False))
    assert np.array_equal(vp.cpu().numpy(), q4.write(v0, packed[:, 6:], inside, bs, True))
    out = torch.full((T, Hkv, D), 3.0, dtype=torch.bfloat16, device="cuda")
    err.zero_()
    bd.paged_kv_read_q4(dev(slots), kp, vp, out, torch.empty_like(out), sh, err=err)
    assert int(err.item()) == bd.PA_DEVERR_SLOT and bool((out[[4, 9]] == 3.0).all())
    with pytest.raises(ValueError):                       # columns of another stride
        bd.paged_kv_write_q4(x[:, :2].transpose(0, 1).contiguous().transpose(0, 1)[:, :, ::2], x[:, 6:], dev(slots), kp, vp, sh)
    with pytest.raises(ValueError):                       # a bf16 pool
        bd.paged_kv_write_q4(x[:, 4:6], x[:, 6:], dev(slots), torch.zeros(nb, bs, Hkv, D, dtype=torch.bfloat16, device="cuda"), vp, sh)


@pytest.mark.gpu
@pytest.mark.parametrize("D, rot, inter, norm, T", [(128, 128, False, True, 67), (128, 64, False, True, 5), (128, 24, False, False, 9), (128, 128, True, True, 300),
                                                    (64, 64, False, True, 33), (64, 32, False, False, 2), (64, 16, True, True, 11), (128, 0, False, True, 17)])
def test_norm_rotation_and_write_is_the_bf16_form_quantised(D, rot, inter, norm, T):
    """The pools' bytes are those of paged_kv_write_q4 of what paged_qk_norm_rope_write writes, and q is its q."""
    rng = np.random.default_rng(rot + T)
    Hq, Hkv, bs, nb = 6, 3, 16, -(-T // 16) + 1
    sh = bd.Shape.make(Hq, Hkv, D, bs, nb)
    x = bf16(wl.random_bf16(rng, (T, Hq + 2 * Hkv, D)))
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    w = bf16(wl.random_bf16(rng, (D,))) if norm else None
    rope = bd.pa_rope_pairs(1e4 ** (-np.arange(rot // 2) / max(rot // 2, 1)), device="cuda") if rot else None
    pos = dev(rng.integers(0, 1 << 20, T).astype(np.int32))
    slots = rng.permutation(nb * bs)[:T].astype(np.int32)
    if T > 8:
        slots[3] = -1
    plain = [torch.zeros(nb, bs, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    q0, q1 = (torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in "ab")
    bd.paged_qk_norm_rope_write(q, k, v, w, w, 1e-6, rope, pos, dev(slots), q0, *plain, sh, interleaved=inter)
    kp, vp = pools(rng, nb, Hkv, bs, D)
    k0, v0 = kp.cpu().numpy(), vp.cpu().numpy()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bd.paged_qk_norm_rope_write_q4(q, k, v, w, w, 1e-6, rope, pos, dev(slots), q1, kp, vp, sh, interleaved=inter, err=err)
    assert int(err.item()) == 0 and np.array_equal(bits_of(q0), bits_of(q1))
    rows = [bits_of(p).reshape(nb * bs, Hkv, D)[slots] for p in plain]
    assert np.array_equal(kp.cpu().numpy(), q4.write(k0, rows[0], slots, bs, False))
    assert np.array_equal(vp.cpu().numpy(), q4.write(v0, rows[1], slots, bs, True))


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -60, 2.0 ** -92, 2.0 ** -126, 2.0 ** -131, 2.0 ** 60, 2.0 ** 89, 2.0 ** 122])
def test_codes_at_every_magnitude(scale):
    """Values of a few bits (their quotients fall on ties often), groups whose scale is subnormal or large,
    and groups around an offset."""
    rng = np.random.default_rng(17)
    T, Hkv, D, bs = 512, 4, 128, 16
    x = rng.integers(-24, 25, (T, Hkv, D)).astype(np.float64)
    x[::3] = rng.integers(-7, 8, x[::3].shape) * 0.5 + 3.0
    x[1::3] = rng.standard_normal(x[1::3].shape) * 4
    bits = wl.f32_to_bf16_bits((x * scale).astype(np.float32))
    sh = bd.Shape.make(Hkv, Hkv, D, bs, T // bs)
    kp, vp = pools(rng, T // bs, Hkv, bs, D)
    slots = np.arange(T, dtype=np.int32)
    bd.paged_kv_write_q4(bf16(bits), bf16(bits), dev(slots), kp, vp, sh)
    for pool, is_v in ((kp, False), (vp, True)):
        want = q4.write(q4.empty_pool(T // bs, Hkv, bs, D), bits, slots, bs, is_v)
        assert np.array_equal(pool.cpu().numpy(), want)
