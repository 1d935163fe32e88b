"""The 4-bit cache in numpy (test infrastructure only): its quantisation, its bytes and its values.

Per group of 32 columns of a token and head: minimum = min x, scale = bf16((max x - min x) / 15),
code = clamp(rint((x - minimum) / scale), 0, 15) in fp32, all codes 0 where the scale is 0; the value is
scale * code + minimum. A group with a NaN or an infinity, or whose range passes fp32, is NaN.

Bytes of a (block, head): the tokens' code rows, then their parameter rows (per group scale and minimum,
bf16). In a code row, nibble n of 32-bit word c G + g holds column 32 g + 8 c + n (K), nibble n of
16-bit word r G + g column 32 g + 4 r + n (V), with G = D / 32.
"""
import numpy as np


def _to_bf16_bits(x):
    b = np.ascontiguousarray(x, np.float32).view(np.uint32)
    out = ((b + np.uint32(0x7FFF) + ((b >> np.uint32(16)) & np.uint32(1))) >> np.uint32(16)).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), out)


def _from_bf16_bits(b):
    return (np.ascontiguousarray(b, np.uint16).astype(np.uint32) << np.uint32(16)).view(np.float32)


def quantise(bits):
    """bf16 bit patterns [..., D] -> codes uint8 [..., D/32, 32], scale and minimum bits [..., D/32]."""
    x = _from_bf16_bits(bits)
    x = x.reshape(*x.shape[:-1], -1, 32)
    with np.errstate(all="ignore"):
        lo, hi = x.min(-1), x.max(-1)
        span = (hi - lo).astype(np.float32)
        bad = ~(np.isfinite(x).all(-1) & np.isfinite(span))
        scale = _to_bf16_bits(span / np.float32(15))
        s = _from_bf16_bits(scale)[..., None]
        u = np.rint((x - lo[..., None]) / np.where(s > 0, s, np.float32(1)))
    u = np.where((s > 0) & ~bad[..., None], np.clip(u, 0, 15), 0).astype(np.uint8)
    low = _to_bf16_bits(lo)
    return u, np.where(bad, np.uint16(0x7FC0), scale), np.where(bad, np.uint16(0x7FC0), low)


def column_nibble(D, is_v):
    """The nibble of a code row that each column has."""
    col = np.arange(D)
    g, e, G = col // 32, col % 32, D // 32
    return ((e // 4) * G + g) * 4 + e % 4 if is_v else ((e // 8) * G + g) * 8 + e % 8


def empty_pool(num_blocks, Hkv, bs, D):
    return np.zeros((num_blocks, Hkv, bs * (D // 2 + D // 8)), np.uint8)


def write(pool, bits, slots, bs, is_v):
    """A copy of the pool with rows bits [T, Hkv, D] at slots (negative: not written)."""
    pool = pool.copy()
    D = bits.shape[-1]
    u, scale, low = quantise(bits)
    nib = np.empty(bits.shape, np.uint8)
    nib[..., column_nibble(D, is_v)] = u.reshape(bits.shape)
    codes = nib[..., 0::2] | (nib[..., 1::2] << 4)
    params = np.stack([scale, low], -1).astype("<u2").view(np.uint8).reshape(*bits.shape[:2], D // 8)
    for t, slot in enumerate(slots):
        if slot < 0:
            continue
        b, o = slot // bs, slot % bs
        pool[b, :, o * (D // 2):(o + 1) * (D // 2)] = codes[t]
        at = bs * (D // 2) + o * (D // 8)
        pool[b, :, at:at + D // 8] = params[t]
    return pool


def values(pool, bs, D, is_v):
    """What a pool stands for: float32 [num_blocks, bs, Hkv, D]."""
    nb, H, _ = pool.shape
    codes = pool[:, :, :bs * (D // 2)].reshape(nb, H, bs, D // 2)
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(nb, H, bs, D)
    u = nib[..., column_nibble(D, is_v)].astype(np.float32)
    p = np.ascontiguousarray(pool[:, :, bs * (D // 2):]).view("<u2").reshape(nb, H, bs, D // 32, 2)
    with np.errstate(all="ignore"):
        s, m = (np.repeat(_from_bf16_bits(p[..., i]), 32, -1) for i in (0, 1))
        # the product of a bf16 and 4 bits is exact in fp32
        return (s * u + m).astype(np.float32).transpose(0, 2, 1, 3)
