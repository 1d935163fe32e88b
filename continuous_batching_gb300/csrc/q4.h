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

// Lane l of a row's D / 8 lanes (consecutive lanes of a warp, all of them active) holds columns
// 8 l .. 8 l + 7 as bf16 pairs w[0 .. 3]; its group is l / 4. Gives the lane's eight codes (column
// 8 l + n in nibble n) and its group's (scale | minimum << 16):
//   minimum = min x;  scale = bf16((max x - min x) / 15);  code = clamp(rint((x - minimum) / scale), 0, 15)
// with fp32 subtractions and divisions rounded to nearest (the minimum is a bf16 value itself, so
// storing it loses nothing). All codes are 0 where the scale is 0. A group that holds a NaN or an
// infinity, or whose range passes fp32, is stored as NaN: every value of it reads as NaN.
__device__ __forceinline__ void q4_quantise8(const uint32_t (&w)[4], uint32_t& codes,
                                             uint32_t& params) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    float lo = x[0], hi = x[0];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        nan = nan || x[i] != x[i];
    }
    if (nan) hi = INFINITY;
#pragma unroll
    for (int m = 1; m <= 2; m <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
    }
    const float range = __fsub_rn(hi, lo);
    codes = 0;
    if (!(range < INFINITY)) {
        params = 0x7FC07FC0u;
        return;
    }
    const __nv_bfloat16 s = __float2bfloat16_rn(__fdiv_rn(range, 15.f));
    const float sf = __bfloat162float(s);
    params = uint32_t(__bfloat16_as_ushort(s)) | (__float_as_uint(lo) & 0xFFFF0000u);
    if (sf > 0.f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float u = rintf(__fdiv_rn(__fsub_rn(x[i], lo), sf));
            codes |= uint32_t(fminf(u, 15.f)) << (4 * i);
        }
    }
}

// A V row's 16-bit words pair the groups g and g + 1 (g even) of one r. Lanes (g, c) hold r = 2 c in
// their low and r = 2 c + 1 in their high half; the even lane takes the pair of r = 2 c, the odd one that of
// r = 2 c + 1. The exchange is its own inverse (a reader's words become the lane's eight codes).
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

// The value a code stands for: scale * code + minimum in one rounding to fp32 (the product is exact).
__device__ __forceinline__ float q4_value(uint32_t code, uint32_t params) {
    return fmaf(__uint_as_float(params << 16), float(code), __uint_as_float(params & 0xFFFF0000u));
}

}  // namespace
