// The 4-bit cache's layout and its quantisation, shared by the kernels that write and read it.
//
// A pool is [num_blocks, Hkv, block_size * kRow<D>] bytes. The tokens of a block and head lie together:
// first their code rows (D / 2 bytes each), then their parameter rows (D / 8 bytes each: for every
// group of 32 columns the scale and the minimum, bf16). So a reader of one head takes whole blocks in
// runs of contiguous bytes, and a token's bytes are its own (writers of two tokens share none).
//
// Within a code row the order is that of the tensor-core fragments the codes are read into, with
// G = D / 32 groups:
//   K: 32-bit word c G + g holds columns 32 g + 8 c + n in nibbles n = 0 .. 7
//   V: 16-bit word r G + g holds columns 32 g + 4 r + n in nibbles n = 0 .. 3
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "sm103.h"

namespace {

constexpr int kQ4Group = 32;

// bytes per token and head, codes and parameters
template <int D>
constexpr int kQ4Codes = D / 2;
template <int D>
constexpr int kQ4Params = D / 8;
template <int D>
constexpr int kQ4Row = kQ4Codes<D> + kQ4Params<D>;

// Offset of the bytes of (block, head).
template <int D>
__device__ __forceinline__ int64_t q4_base(int64_t block, int Hkv, int head, int bs) {
    return (block * Hkv + head) * (int64_t(bs) * kQ4Row<D>);
}

// Two bf16 at a time; NaN where one of a pair is.
__device__ __forceinline__ uint32_t q4_max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t q4_min2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Lane l of a row's D / (2 W) lanes (consecutive lanes of a warp, all of them active) holds columns
// 2 W l .. 2 W l + 2 W - 1 as bf16 pairs w[0 .. W - 1], W 4 or 8; 16 / W lanes hold a group. Gives the lane's codes
// (column 2 W l + 8 i + n in nibble n of word i) and its group's (scale | minimum << 16):
//   minimum = min x;  scale = bf16((max x - min x) / 15);  code = clamp(rint((x - minimum) / scale), 0, 15)
// with fp32 subtractions and divisions rounded to nearest (the minimum is a bf16 value itself, so
// storing it loses nothing). All codes are 0 where the scale is 0. A group that holds a NaN or an
// infinity, or whose range passes fp32, is stored as NaN: every value of it reads as NaN.
//
// The division by the group's scale s is one reciprocal and, per element, a product and a correction by its
// exact remainder (Markstein 1990): q = d y, then q + (d - q s) y. This is the quotient rounded to
// nearest: before its rounding it is off by at most 2^-46 of itself (the remainder is exact and y is
// off by 2^-24), while d / s, d of 24 bits and s of 8, is at least 2^-33 of itself away from every point half way
// between two fp32 numbers (such a point has 25 bits, and no multiple of s by it has 24). The division by 15
// likewise. Ranges so small or so large that a step could leave fp32's normal numbers divide as usual. (16,384
// tokens of 8 heads of 128: 60 us with a division per element and fp32 extremes, bound by instructions, 23 with
// this one, 15.1 with packed extremes and 16 columns a lane in the write.)
template <int W>
__device__ __forceinline__ void q4_quantise(const uint32_t (&w)[W], uint32_t (&codes)[W / 4], uint32_t& params) {
    uint32_t top = w[0], low = w[0];
#pragma unroll
    for (int i = 1; i < W; ++i) {
        top = q4_max2(top, w[i]);
        low = q4_min2(low, w[i]);
    }
    // (max, -min), so that one maximum serves both
    constexpr uint32_t kSign = 0x80000000u;
    top = q4_max2(__byte_perm(top, low, 0x5410) ^ kSign, __byte_perm(top, low, 0x7632) ^ kSign);
#pragma unroll
    for (int m = 1; m < 16 / W; m <<= 1) top = q4_max2(top, __shfl_xor_sync(0xffffffffu, top, m));
    const float hi = __uint_as_float(top << 16), lo = __uint_as_float((top & 0xFFFF0000u) ^ kSign);
    const float range = __fsub_rn(hi, lo);
#pragma unroll
    for (int k = 0; k < W / 4; ++k) codes[k] = 0;
    if (!(range < INFINITY)) {                      // (NaN, too)
        params = 0x7FC07FC0u;
        return;
    }
    // u + 1.5 2^23 rounds to an integer, ties to even; the words' upper parts add up to a constant
    constexpr float kRound = 12582912.f;
    constexpr uint32_t kUpper = 0x4B400000u * 0x11111111u;
    const bool usual = range >= 0x1p-80f && range <= 0x1p90f;
    float t;
    if (usual) {
        constexpr float y = 1.f / 15.f;
        t = __fmul_rn(range, y);
        t = fmaf(fmaf(-t, 15.f, range), y, t);
    } else {
        t = __fdiv_rn(range, 15.f);
    }
    const __nv_bfloat16 s = __float2bfloat16_rn(t);
    const float sf = __bfloat162float(s);
    params = uint32_t(__bfloat16_as_ushort(s)) | (__float_as_uint(lo) & 0xFFFF0000u);
    if (usual) {
        const float y = __frcp_rn(sf);
        const uint64_t y2 = f2(y, y), n2 = f2(-sf, -sf), lo2 = f2(-lo, -lo), round2 = f2(kRound, kRound);
#pragma unroll
        for (int i = W - 1; i >= 0; --i) {          // two elements at a time
            const uint64_t d = add2(f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)), lo2);
            uint64_t q = mul2(d, y2);
            q = fma2(fma2(q, n2, d), y2, q);        // (at most 15.06: no code but 0 .. 15)
            float u, v;
            f2_split(add2(q, round2), u, v);
            codes[i / 4] = (codes[i / 4] * 16u + __float_as_uint(v)) * 16u + __float_as_uint(u);
        }
    } else {
        if (!(sf > 0.f)) return;
#pragma unroll
        for (int k = 0; k < W / 4; ++k) {
#pragma unroll 1
            for (int i = 7; i >= 0; --i) {
                const uint32_t x = i < 4 ? (i < 2 ? w[4 * k] : w[4 * k + 1]) : (i < 6 ? w[4 * k + 2] : w[4 * k + 3]);
                const float q = __fdiv_rn(__fsub_rn(__uint_as_float(i & 1 ? x & 0xFFFF0000u : x << 16), lo), sf);
                codes[k] = codes[k] * 16u + __float_as_uint(fminf(q, 15.f) + kRound);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < W / 4; ++k) codes[k] -= kUpper;
}

// A V row's 16-bit words pair the groups g and g + 1 (g even) of one r. Lanes (g, c) hold r = 2 c in
// their low and r = 2 c + 1 in their high half; the even lane takes the pair of r = 2 c, the odd one that of
// r = 2 c + 1.
__device__ __forceinline__ uint32_t q4_pair_groups(uint32_t codes, int l) {
    const bool odd = (l >> 2) & 1;
    const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? codes & 0xFFFFu : codes >> 16, 4);
    return odd ? (codes & 0xFFFF0000u) | other : (codes & 0xFFFFu) | (other << 16);
}

// 32-bit word of a code row that lane l writes (after q4_pair_groups for V).
template <int D, bool IS_V>
__device__ __forceinline__ int q4_word(int l) {
    constexpr int G = D / kQ4Group;
    const int g = l >> 2, c = l & 3;
    return IS_V ? (2 * c + (g & 1)) * (G / 2) + (g >> 1) : c * G + g;
}

// Stores one row of a lane group; `at` is q4_base of the row's block and head, o its token in the block.
template <int D, bool IS_V>
__device__ __forceinline__ void q4_store_row(uint8_t* pool, int64_t at, int bs, int o, int l,
                                             uint32_t codes, uint32_t params) {
    uint8_t* row = pool + at + o * kQ4Codes<D>;
    reinterpret_cast<uint32_t*>(row)[q4_word<D, IS_V>(l)] = codes;
    if ((l & 3) == 0)
        reinterpret_cast<uint32_t*>(pool + at + bs * kQ4Codes<D> + o * kQ4Params<D>)[l >> 2] = params;
}

// The same of lanes with 16 columns, g = l / 2 and c = 2 (l % 2) and the next, codes[0] and codes[1].
__device__ __forceinline__ void q4_pair_groups2(uint32_t (&codes)[2], int l) {
    // the even group's lane takes r = 4 (l % 2) and the next, the odd one's the two behind them
    const bool odd = (l >> 1) & 1;
    const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? codes[0] : codes[1], 2);
    const uint32_t even_half = odd ? other : codes[0], odd_half = odd ? codes[1] : other;
    codes[0] = __byte_perm(even_half, odd_half, 0x5410);
    codes[1] = __byte_perm(even_half, odd_half, 0x7632);
}

template <int D, bool IS_V>
__device__ __forceinline__ void q4_store_row2(uint8_t* pool, int64_t at, int bs, int o, int l,
                                              const uint32_t (&codes)[2], uint32_t params) {
    constexpr int G = D / kQ4Group;
    const int g = l >> 1, c = l & 1;
    uint32_t* const row = reinterpret_cast<uint32_t*>(pool + at + o * kQ4Codes<D>);
    if constexpr (IS_V) {
        uint32_t* const to = row + (4 * c + 2 * (g & 1)) * (G / 2) + (g >> 1);
        to[0] = codes[0];
        to[G / 2] = codes[1];
    } else {
        uint32_t* const to = row + 2 * c * G + g;
        to[0] = codes[0];
        to[G] = codes[1];
    }
    if (c == 0) reinterpret_cast<uint32_t*>(pool + at + bs * kQ4Codes<D> + o * kQ4Params<D>)[g] = params;
}

// What reads the cache back takes a row by four lanes: lane c its D / 8 bytes of codes from c D / 8 on (w: G words)
// and all of the row's parameters (p), and gives columns 32 g + 8 c .. + 7 of every group g. In a V row these bytes are
// the halves r = 2 c and r = 2 c + 1.
template <int D, bool IS_V>
__device__ __forceinline__ uint4 q4_columns(const uint32_t (&w)[D / kQ4Group],
                                            const uint32_t (&p)[D / kQ4Group], int g) {
    constexpr int G = D / kQ4Group;
    const uint32_t x = IS_V ? __byte_perm(w[g / 2], w[G / 2 + g / 2], g & 1 ? 0x7632 : 0x5410) : w[g];
    const uint32_t scale = __byte_perm(p[g], 0, 0x1010), low = __byte_perm(p[g], 0, 0x3232);
    // the value scale * u + minimum in one rounding, two columns n and n + 4 at a time: u as bf16 128 + u, less 128
    uint32_t y[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        uint32_t u = ((x >> (4 * n)) & 0x000F000Fu) | 0x43004300u;
        asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(u) : "r"(0x43004300u));
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y[n]) : "r"(u), "r"(scale), "r"(low));
    }
    return make_uint4(__byte_perm(y[0], y[1], 0x5410), __byte_perm(y[2], y[3], 0x5410),
                      __byte_perm(y[0], y[1], 0x7632), __byte_perm(y[2], y[3], 0x7632));
}

// Two values in f16, rounded to odd (cut, the last bit set where bits were cut off): an output that is one value alone
// is then that value rounded to bf16 once.
__device__ __forceinline__ uint32_t q4_odd_f16(float lo, float hi) {
    uint32_t h;
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
    // the 13 bits that f16 does not have, plus 2^13 - 1: bit 13 is set where they are not all zeros
    const uint32_t cut = (__byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x5410) & 0x1FFF1FFFu) + 0x1FFF1FFFu;
    return h | ((cut >> 13) & 0x00010001u);
}

// The columns of a V row in f16: in fp32, where the value is off by 2^-24 at most, then one rounding (below 2^-14 more
// bits are cut off than are looked at).
template <int D>
__device__ __forceinline__ uint4 q4_columns_f16(const uint32_t (&w)[D / kQ4Group], const uint32_t (&p)[D / kQ4Group],
                                                int g) {
    constexpr int G = D / kQ4Group;
    const uint32_t x = __byte_perm(w[g / 2], w[G / 2 + g / 2], g & 1 ? 0x7632 : 0x5410);
    const float scale = __uint_as_float(p[g] << 16), low = __uint_as_float(p[g] & 0xFFFF0000u);
    uint32_t y[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        uint32_t u = ((x >> (4 * n)) & 0x000F000Fu) | 0x43004300u;
        asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(u) : "r"(0x43004300u));
        y[n] = q4_odd_f16(fmaf(__uint_as_float(u << 16), scale, low), fmaf(__uint_as_float(u & 0xFFFF0000u), scale, low));
    }
    return make_uint4(__byte_perm(y[0], y[1], 0x5410), __byte_perm(y[2], y[3], 0x5410),
                      __byte_perm(y[0], y[1], 0x7632), __byte_perm(y[2], y[3], 0x7632));
}

// A row's parameters; `at` is q4_base of the block and head, o the token in it.
template <int D>
__device__ __forceinline__ void q4_load_params(const uint8_t* pool, int64_t at, int bs, int o, uint32_t (&p)[D / kQ4Group]) {
    const uint8_t* params = pool + at + bs * kQ4Codes<D> + o * kQ4Params<D>;
    if constexpr (D == 128) {
        const uint4 b = __ldg(reinterpret_cast<const uint4*>(params));
        p[0] = b.x, p[1] = b.y, p[2] = b.z, p[3] = b.w;
    } else {
        const uint2 b = __ldg(reinterpret_cast<const uint2*>(params));
        p[0] = b.x, p[1] = b.y;
    }
}

// A lane's codes and its row's parameters.
template <int D>
__device__ __forceinline__ void q4_load_row(const uint8_t* pool, int64_t at, int bs, int o, int c,
                                            uint32_t (&w)[D / kQ4Group], uint32_t (&p)[D / kQ4Group]) {
    const uint8_t* codes = pool + at + o * kQ4Codes<D> + c * (D / 8);
    if constexpr (D == 128) {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(codes));
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    } else {
        const uint2 a = __ldg(reinterpret_cast<const uint2*>(codes));
        w[0] = a.x, w[1] = a.y;
    }
    q4_load_params<D>(pool, at, bs, o, p);
}

}  // namespace
