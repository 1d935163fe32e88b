// Per-head RMS norm of q and k, rotation by position and the KV write, in one pass: what stands
// between a layer's projections and paged_attention_step.
//
//   y = x * rsqrt(mean_d(x^2) + eps) * w                      (q and k heads; skipped without w)
//   (y_i, y_j) -> (y_i cos a - y_j sin a, y_i sin a + y_j cos a),  a = position[axis] * frequency
//   q -> q_out (bf16), k -> its slot of the K pool, v -> its slot of the V pool unchanged
// with the pairs (i, i + r/2) or (2i, 2i+1) of the first r of D columns; the others pass through.
// Everything between the bf16 input and the single rounding of the output is fp32.
//
// Angles. A pair's frequency is held as turns per position, rounded to units of 2^-64 turn
// (pa_rope_pair.step). position * step in 64-bit integers, wrapping, is that step's phase modulo one
// turn exactly, for positions of any size and sign: nothing is lost to range reduction, and what the
// step's rounding makes of it is 2^-65 turn a position (2^-34 turn at 2^31). The phase's top
// 32 bits go to fp32 (2^-25 of half a turn) and sincospif. Reading the sines from a table instead
// would read 8 bytes a pair and token from memory, against none here.
//
// Bound by memory: (Hq + 2 Hkv) D read and written per token. D / 8 lanes hold a head, each lane
// the elements of four pairs (two 8-byte pieces r/2 apart, or one of 16 bytes for adjacent
// pairs), so a pair never crosses lanes and the norm is the only exchange (log2(D / 8) shuffles).
// A warp takes some rounds of one token's heads, all of one kind at a time, so its lanes' four sines
// (each lane computes its share and gets the rest from its neighbours) and the products of weights
// and sines serve them from registers and nothing is shared between warps. What it costs beyond
// memory is instructions: per head, 4 shuffles and some 50 others, the arithmetic in packed pairs.
//
// Measured: 16,384 tokens of 32 + 2 x 8 heads of 128 (403 MB) in 75 us, 5.4 TB/s, 79 % of the measured
// copy rate; replayed in a graph, one token 2.5 us, 128 tokens of 64 + 2 x 8 heads 3.4 us, 2,096
// tokens into an fp8 pool (47 MB) 14.3 us; 8,192 tokens of 32 + 2 x 8 heads into 4-bit pools (178 MB) 44.7 us, 4.0 TB/s
// (bf16 pools, 201 MB, 40.7), bound by the latency of a head's load, norm and exchange: 1, 3 or 4 heads in flight 50
// to 51 us, 3 or 5 CTAs a multiprocessor 57 and 53.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.h"
#include "q4.h"
#include "sm103.h"

using namespace pa_detail;

namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 2;          // heads a lane group has in flight
constexpr int kMaxRounds = 24;     // heads a lane group takes, where there are tokens enough

struct RopeParams {
    const __nv_bfloat16 *q, *k, *v, *wq, *wk;
    int64_t q_stride, k_stride, v_stride;      // elements between tokens
    const pa_rope_pair* rope;
    const int32_t* positions;                  // [n_axes, T]
    const int32_t* slots;
    __nv_bfloat16* q_out;
    void *k_pool, *v_pool;
    int64_t num_slots;
    int32_t* err;
    int32_t T, Hq, Hkv, n_pairs, n_axes;
    int32_t warps;                             // per token
    int32_t log2bs;                            // of the tokens a block (4-bit pools)
    float eps, k_scale, v_scale;
};

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Four values -> four codes e4m3(x / s): the same division and rounding as paged_kv_write_fp8,
// from the fp32 value, so that a K element is rounded once.
__device__ __forceinline__ uint32_t e4m3x4(const float* x, float s) {
    uint16_t a, b;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(a) : "f"(__fdiv_rn(x[1], s)), "f"(__fdiv_rn(x[0], s)));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(b) : "f"(__fdiv_rn(x[3], s)), "f"(__fdiv_rn(x[2], s)));
    return uint32_t(a) | (uint32_t(b) << 16);
}

enum Kind { kQ, kK, kV };
enum Cache { kBf16, kFp8, kQ4 };               // what the pools hold

template <int D, bool INTER, Cache C>
__global__ void __launch_bounds__(kThreads, 4) norm_rope_kernel(const RopeParams p) {
    constexpr bool F8 = C == kFp8;
    constexpr int kLanes = D / 8;              // lanes per head
    constexpr int kHeads = 32 / kLanes;        // heads a warp has at a time: a round
    // the attention kernel that follows waits for this grid before it reads anything; this one
    // in turn waits for what came before it
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const int64_t wid = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = wid / p.warps;
    if (t >= p.T) return;
    const int part = int(wid - t * p.warps);
    const int sub = (threadIdx.x & 31) / kLanes;
    const int l = threadIdx.x % kLanes;
    const bool turns = l < p.n_pairs / 4;      // the lane's elements rotate
    // the lane's two four-element pieces: adjacent pairs lie in one 16-byte piece
    const int a = INTER ? 8 * l : turns ? 4 * l : 8 * l;
    const int b = INTER ? 8 * l + 4 : turns ? p.n_pairs + 4 * l : 8 * l + 4;

    const int32_t slot = p.slots[t];
    const bool writes = slot >= 0 && slot < p.num_slots;
    if (slot >= p.num_slots && part == 0 && (threadIdx.x & 31) == 0 && p.err)
        atomicOr(p.err, PA_DEVERR_SLOT);

    float co[4], si[4];                        // of the lane's pairs
    bool have = false;
    const auto sines = [&]() {
        have = true;
#pragma unroll
        for (int e = 0; e < 4; ++e) co[e] = 1.f, si[e] = 0.f;
        // a pair's lanes in the warp's lane groups share its sines: each computes 4 / kHeads
#pragma unroll
        for (int k = 0; k < 4 / kHeads; ++k) {
            const int e = k * kHeads + sub;
            float c = 1.f, s = 0.f;
            if (turns) {
                const pa_rope_pair f = p.rope[4 * l + e];
                int axis = f.axis;
                if (axis < 0 || axis >= p.n_axes) {
                    if (p.err) atomicOr(p.err, PA_DEVERR_META);
                    axis = 0;
                }
                const int64_t pos = p.positions[int64_t(axis) * p.T + t];
                const uint64_t phase = uint64_t(pos) * f.step;
                sincospif(float(int32_t(phase >> 32)) * 0x1p-31f, &s, &c);
            }
#pragma unroll
            for (int g = 0; g < kHeads; ++g) {
                co[k * kHeads + g] = __shfl_sync(0xffffffffu, c, g * kLanes + l);
                si[k * kHeads + g] = __shfl_sync(0xffffffffu, s, g * kLanes + l);
            }
        }
    };

    // rounds r0 .. r1 - 1 of one kind's heads
    const auto run = [&](auto kind, const __nv_bfloat16* src, const __nv_bfloat16* weight, int heads,
                         int r0, int r1) {
        constexpr Kind K = decltype(kind)::value;
        if (r0 >= r1 || (K != kQ && !writes)) return;
        src += sub * D;
        const auto load = [&](int r, uint2& xa, uint2& xb) {
            if (r >= r1 || r * kHeads + sub >= heads) return;
            const __nv_bfloat16* s = src + r * (kHeads * D);
            if constexpr (INTER) {
                const uint4 w = *reinterpret_cast<const uint4*>(s + 8 * l);
                xa = make_uint2(w.x, w.y);
                xb = make_uint2(w.z, w.w);
            } else {
                xa = *reinterpret_cast<const uint2*>(s + a);
                xb = *reinterpret_cast<const uint2*>(s + b);
            }
        };
        uint2 xa[kUnits] = {}, xb[kUnits] = {};
#pragma unroll
        for (int i = 0; i < kUnits; ++i) load(r0 + i, xa[i], xb[i]);
        // With weights (wu, wv) of a pair's elements: (u, v) -> r (u wu c - v wv s, u wu s + v wv c),
        // r the norm's factor (c = 1, s = 0 in lanes that do not turn).
        uint64_t uc[2], us[2], vc[2], vs[2];
        const bool norm = K != kV && weight;
        if constexpr (K != kV) {
            if (!have) sines();
            float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
            if (weight) {
                const uint2 wa = __ldg(reinterpret_cast<const uint2*>(weight + a));
                const uint2 wb = __ldg(reinterpret_cast<const uint2*>(weight + b));
                w[0] = lo16(wa.x), w[1] = hi16(wa.x), w[2] = lo16(wa.y), w[3] = hi16(wa.y);
                w[4] = lo16(wb.x), w[5] = hi16(wb.x), w[6] = lo16(wb.y), w[7] = hi16(wb.y);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * e, j = 2 * e + 1;
                const float wui = INTER ? w[2 * i] : w[i], wvi = INTER ? w[2 * i + 1] : w[4 + i];
                const float wuj = INTER ? w[2 * j] : w[j], wvj = INTER ? w[2 * j + 1] : w[4 + j];
                uc[e] = f2(wui * co[i], wuj * co[j]);
                us[e] = f2(wui * si[i], wuj * si[j]);
                vc[e] = f2(wvi * co[i], wvj * co[j]);
                vs[e] = f2(-wvi * si[i], -wvj * si[j]);
            }
        }
        // Rows in column order (4-bit pools): piece i of four columns, of half = n_pairs / 4 in either half of the
        // rotated ones, is the first piece of lane i or the second of lane i - half, and behind those lane i / 2's own. In
        // the first of two exchanges even lanes give their first piece and odd ones their second, in the other the
        // rest, and every lane takes one of its two pieces from each.
        int from_a = l, from_b = l;
        bool a_second = l & 1;
        if constexpr (C == kQ4 && !INTER && K != kQ) {
            const int half = p.n_pairs / 4;
            const auto from = [&](int i) { return i < half ? i : i < 2 * half ? i - half : l; };
            const auto in_a = [&](int i) {
                const bool second = i < half ? false : i < 2 * half ? true : (i & 1) != 0;
                return ((from(i) & 1) != 0) == second;
            };
            a_second = !in_a(2 * l);
            from_a = from(2 * l + a_second);
            from_b = from(2 * l + !a_second);
        }
        const int64_t row = K == kQ ? t * p.Hq : int64_t(slot) * p.Hkv;
#pragma unroll 1
        for (int rb = r0; rb < r1; rb += kUnits) {
#pragma unroll
            for (int i = 0; i < kUnits; ++i) {
                const int r = rb + i;
                if (r >= r1) break;
                const int h = r * kHeads + sub;
                uint2 ya = xa[i], yb = xb[i];
                load(r + kUnits, xa[i], xb[i]);
                float x[8];
                if (K != kV || F8) {
                    x[0] = lo16(ya.x), x[1] = hi16(ya.x), x[2] = lo16(ya.y), x[3] = hi16(ya.y);
                    x[4] = lo16(yb.x), x[5] = hi16(yb.x), x[6] = lo16(yb.y), x[7] = hi16(yb.y);
                }
                if constexpr (K != kV) {
                    uint64_t u[2], v[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        u[e] = INTER ? f2(x[4 * e], x[4 * e + 2]) : f2(x[2 * e], x[2 * e + 1]);
                        v[e] = INTER ? f2(x[4 * e + 1], x[4 * e + 3])
                                     : f2(x[4 + 2 * e], x[5 + 2 * e]);
                    }
                    uint64_t q2 = mul2(u[0], u[0]);
                    q2 = fma2(u[1], u[1], q2);
                    q2 = fma2(v[0], v[0], q2);
                    q2 = fma2(v[1], v[1], q2);
                    float f = 1.f;
                    if (norm) {
                        float s0, s1;
                        f2_split(q2, s0, s1);
                        float ss = s0 + s1;
#pragma unroll
                        for (int m = kLanes / 2; m; m >>= 1)
                            ss += __shfl_xor_sync(0xffffffffu, ss, m);
                        f = rsqrtf(ss * (1.f / D) + p.eps);
                    }
                    const uint64_t ff = f2(f, f);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        u[e] = mul2(u[e], ff);
                        v[e] = mul2(v[e], ff);
                        uint64_t nu = mul2(u[e], uc[e]), nv = mul2(v[e], vc[e]);
                        if (turns) {                   // else the other's infinity would leak in
                            nu = fma2(v[e], vs[e], nu);
                            nv = fma2(u[e], us[e], nv);
                        }
                        float u0, u1, v0, v1;
                        f2_split(nu, u0, u1);
                        f2_split(nv, v0, v1);
                        if constexpr (INTER) {
                            x[4 * e] = u0, x[4 * e + 1] = v0, x[4 * e + 2] = u1, x[4 * e + 3] = v1;
                        } else {
                            x[2 * e] = u0, x[2 * e + 1] = u1, x[4 + 2 * e] = v0, x[5 + 2 * e] = v1;
                        }
                    }
                    if (!F8 || K == kQ) {
                        ya = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
                        yb = make_uint2(pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
                    }
                }
                if constexpr (C == kQ4 && K != kQ) {
                    // The row in column order, lane l columns 8 l .. 8 l + 7
                    uint32_t w[4] = {ya.x, ya.y, yb.x, yb.y};
                    if constexpr (!INTER) {
                        const bool odd = l & 1;
                        const uint32_t p0 = odd ? yb.x : ya.x, p1 = odd ? yb.y : ya.y;
                        const uint32_t q0 = odd ? ya.x : yb.x, q1 = odd ? ya.y : yb.y;
                        const uint32_t x0 = __shfl_sync(0xffffffffu, p0, from_a, kLanes);
                        const uint32_t x1 = __shfl_sync(0xffffffffu, p1, from_a, kLanes);
                        const uint32_t y0 = __shfl_sync(0xffffffffu, q0, from_b, kLanes);
                        const uint32_t y1 = __shfl_sync(0xffffffffu, q1, from_b, kLanes);
                        w[0] = a_second ? y0 : x0, w[1] = a_second ? y1 : x1;
                        w[2] = a_second ? x0 : y0, w[3] = a_second ? x1 : y1;
                    }
                    uint32_t codes[1], params;
                    q4_quantise<4>(w, codes, params);
                    if constexpr (K == kV) codes[0] = q4_pair_groups(codes[0], l);
                    if (h >= heads) continue;
                    const int block = slot >> p.log2bs;
                    q4_store_row<D, K == kV>(static_cast<uint8_t*>(K == kV ? p.v_pool : p.k_pool),
                                             q4_base<D>(block, p.Hkv, h, 1 << p.log2bs), 1 << p.log2bs,
                                             slot - (block << p.log2bs), l, codes[0], params);
                    continue;
                }
                if (h >= heads) continue;
                const int64_t at = (row + h) * D;
                if constexpr (F8 && K != kQ) {
                    uint8_t* dst = static_cast<uint8_t*>(K == kV ? p.v_pool : p.k_pool) + at;
                    const float s = K == kV ? p.v_scale : p.k_scale;
                    const uint32_t ca = e4m3x4(x, s), cb = e4m3x4(x + 4, s);
                    if constexpr (INTER) {
                        *reinterpret_cast<uint2*>(dst + a) = make_uint2(ca, cb);
                    } else {
                        *reinterpret_cast<uint32_t*>(dst + a) = ca;
                        *reinterpret_cast<uint32_t*>(dst + b) = cb;
                    }
                } else {
                    __nv_bfloat16* dst =
                        (K == kQ ? p.q_out : static_cast<__nv_bfloat16*>(K == kV ? p.v_pool
                                                                                 : p.k_pool)) + at;
                    if constexpr (INTER) {
                        *reinterpret_cast<uint4*>(dst + a) = make_uint4(ya.x, ya.y, yb.x, yb.y);
                    } else {
                        *reinterpret_cast<uint2*>(dst + a) = ya;
                        *reinterpret_cast<uint2*>(dst + b) = yb;
                    }
                }
            }
        }
    };
    const int rq = (p.Hq + kHeads - 1) / kHeads, rk = (p.Hkv + kHeads - 1) / kHeads;
    const int rounds = rq + 2 * rk;
    const int r0 = rounds * part / p.warps, r1 = rounds * (part + 1) / p.warps;
    run(std::integral_constant<Kind, kQ>(), p.q + t * p.q_stride, p.wq, p.Hq, r0, min(r1, rq));
    run(std::integral_constant<Kind, kK>(), p.k + t * p.k_stride, p.wk, p.Hkv, max(r0 - rq, 0),
        min(r1 - rq, rk));
    run(std::integral_constant<Kind, kV>(), p.v + t * p.v_stride, nullptr, p.Hkv,
        max(r0 - rq - rk, 0), min(r1 - rq - rk, rk));
}

template <int D, bool INTER, Cache C>
int32_t launch_rope(RopeParams& p, cudaStream_t stream) {
    constexpr int kHeads = 256 / D;            // heads a warp has at a time
    // Warps per token: few, so that each has kMaxRounds rounds of heads to its sines, unless there
    // are too few tokens to fill the GPU with (16 warps an SM); at most one for every round. 128 and
    // 2,096 tokens: 3.4 and 14.3 us, with 8 warps an SM 4.6 and 22.5, with 32 3.7 and 17.6.
    const int rounds = (p.Hq + kHeads - 1) / kHeads + 2 * ((p.Hkv + kHeads - 1) / kHeads);
    const int64_t fill = (16 * int64_t(PA_PLAN_CTAS) + p.T - 1) / p.T;
    p.warps = int(std::min<int64_t>(rounds, std::max<int64_t>((rounds + kMaxRounds - 1) / kMaxRounds,
                                                              fill)));
    const int64_t blocks = (int64_t(p.T) * p.warps * 32 + kThreads - 1) / kThreads;
    if (blocks > INT32_MAX) return PA_ERR_SHAPE;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return note_cuda(cudaLaunchKernelEx(&cfg, norm_rope_kernel<D, INTER, C>, p));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int32_t norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                  int64_t v_stride, const void* q_weight, const void* k_weight, float eps,
                  const pa_rope_pair* rope, int32_t n_pairs, int32_t interleaved,
                  const int32_t* positions, int32_t n_axes, const int32_t* slot_mapping, int32_t T,
                  void* q_out, void* k_pool, void* v_pool, Cache cache, float k_scale, float v_scale,
                  const pa_shape* shape, int32_t* err_flag, cudaStream_t stream) {
    int32_t st = check_shape(shape);
    if (st) return st;
    const int D = shape->head_dim;
    if (T < 0 || !(eps >= 0.f) || !(eps < INFINITY)) return PA_ERR_INVALID;
    if (n_pairs < 0 || n_pairs % 4 || 2 * n_pairs > D) return PA_ERR_SHAPE;
    if (T == 0) return PA_OK;
    if (!q || !k || !v || !q_out || !k_pool || !v_pool || !slot_mapping) return PA_ERR_INVALID;
    if (n_pairs > 0 && (!rope || !positions || n_axes < 1)) return PA_ERR_INVALID;
    const int64_t q_row = int64_t(shape->num_q_heads) * D, kv_row = int64_t(shape->num_kv_heads) * D;
    if (q_stride < q_row || k_stride < kv_row || v_stride < kv_row) return PA_ERR_INVALID;
    if ((q_stride | k_stride | v_stride) % 8) return PA_ERR_INVALID;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) ||
        !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(q_weight) || !aligned16(k_weight) ||
        !aligned16(rope))
        return PA_ERR_INVALID;
    // in place only over the same layout: otherwise a head could be overwritten before it is read
    if (q == q_out && q_stride != q_row) return PA_ERR_INVALID;
    RopeParams p;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.wq = static_cast<const __nv_bfloat16*>(q_weight);
    p.wk = static_cast<const __nv_bfloat16*>(k_weight);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.rope = rope;
    p.positions = positions;
    p.slots = slot_mapping;
    p.q_out = static_cast<__nv_bfloat16*>(q_out);
    p.k_pool = k_pool;
    p.v_pool = v_pool;
    p.num_slots = int64_t(shape->num_blocks) * shape->block_size;
    p.err = err_flag;
    p.T = T;
    p.Hq = shape->num_q_heads;
    p.Hkv = shape->num_kv_heads;
    p.n_pairs = n_pairs;
    p.n_axes = n_axes;
    p.eps = eps;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.log2bs = 0;
    while ((1 << p.log2bs) < shape->block_size) ++p.log2bs;
    const auto launch = [&](auto held) {
        constexpr Cache C = decltype(held)::value;
        if (D == 128)
            return interleaved ? launch_rope<128, true, C>(p, stream) : launch_rope<128, false, C>(p, stream);
        return interleaved ? launch_rope<64, true, C>(p, stream) : launch_rope<64, false, C>(p, stream);
    };
    if (cache == kFp8) return launch(std::integral_constant<Cache, kFp8>());
    if (cache == kQ4) return launch(std::integral_constant<Cache, kQ4>());
    return launch(std::integral_constant<Cache, kBf16>());
}

}  // namespace

namespace {

// f / 2 pi turns modulo one turn, rounded to the nearest 2^-64 of a turn. The quotient is carried in
// two doubles (quotient and what it leaves of f, 2 pi in two doubles itself; their 2^-100 is enough for
// |f| < 2^30): one double's 53 bits would be off by 2^10 units for a frequency of a turn, which a far
// position multiplies.
uint64_t turn_step(double f) {
    constexpr double kTwoPi = 0x1.921fb54442d18p+2, kTwoPiLow = 0x1.1a62633145c07p-52;
    const double turns = std::fabs(f) / kTwoPi;
    const double left = std::fma(-turns, kTwoPi, std::fabs(f)) - turns * kTwoPiLow;
    double low = left / kTwoPi;
    low -= std::nearbyint(low);                     // (not zero for frequencies of 2^53 turns or more)
    // the fraction of `turns` in units, exactly; its whole units apart from the rest
    const double units = std::ldexp(turns - std::floor(turns), 64), whole = std::floor(units);
    const double rest = std::nearbyint((units - whole) + std::ldexp(low, 64));   // |rest| <= 2^63 + 1
    const uint64_t step = uint64_t(whole) + (rest < 0 ? ~uint64_t(-rest) + 1 : uint64_t(rest));
    return f < 0 ? ~step + 1 : step;
}

}  // namespace

extern "C" int32_t pa_rope_pairs(const double* inv_freq, const int32_t* axes, int32_t n_pairs,
                                 int32_t n_axes, pa_rope_pair* out) {
    if (n_pairs < 0 || n_axes < 1) return PA_ERR_INVALID;
    if (n_pairs == 0) return PA_OK;
    if (!inv_freq || !out) return PA_ERR_INVALID;
    for (int32_t i = 0; i < n_pairs; ++i) {
        if (!std::isfinite(inv_freq[i])) return PA_ERR_INVALID;
        if (axes && (axes[i] < 0 || axes[i] >= n_axes)) return PA_ERR_BOUNDS;
    }
    for (int32_t i = 0; i < n_pairs; ++i) {
        out[i].step = turn_step(inv_freq[i]);
        out[i].axis = axes ? axes[i] : 0;
        out[i].reserved = 0;
    }
    return PA_OK;
}

extern "C" int32_t paged_qk_norm_rope_write(
    const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
    int64_t v_stride, const void* q_weight, const void* k_weight, float eps,
    const pa_rope_pair* rope, int32_t n_pairs, int32_t interleaved, const int32_t* positions,
    int32_t n_axes, const int32_t* slot_mapping, int32_t T, void* q_out, void* k_pool,
    void* v_pool, const pa_shape* shape, int32_t* err_flag, pa_stream_t stream) {
    return norm_rope(q, q_stride, k, k_stride, v, v_stride, q_weight, k_weight, eps, rope, n_pairs,
                     interleaved, positions, n_axes, slot_mapping, T, q_out, k_pool, v_pool, kBf16,
                     1.f, 1.f, shape, err_flag, stream);
}

extern "C" int32_t paged_qk_norm_rope_write_fp8(
    const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
    int64_t v_stride, const void* q_weight, const void* k_weight, float eps,
    const pa_rope_pair* rope, int32_t n_pairs, int32_t interleaved, const int32_t* positions,
    int32_t n_axes, const int32_t* slot_mapping, int32_t T, void* q_out, void* k_pool,
    void* v_pool, float k_scale, float v_scale, const pa_shape* shape, int32_t* err_flag,
    pa_stream_t stream) {
    if (!(k_scale > 0.f) || !(v_scale > 0.f) || !(k_scale < INFINITY) || !(v_scale < INFINITY))
        return PA_ERR_INVALID;
    return norm_rope(q, q_stride, k, k_stride, v, v_stride, q_weight, k_weight, eps, rope, n_pairs,
                     interleaved, positions, n_axes, slot_mapping, T, q_out, k_pool, v_pool, kFp8,
                     k_scale, v_scale, shape, err_flag, stream);
}

extern "C" int32_t paged_qk_norm_rope_write_q4(
    const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
    int64_t v_stride, const void* q_weight, const void* k_weight, float eps,
    const pa_rope_pair* rope, int32_t n_pairs, int32_t interleaved, const int32_t* positions,
    int32_t n_axes, const int32_t* slot_mapping, int32_t T, void* q_out, void* k_pool,
    void* v_pool, const pa_shape* shape, int32_t* err_flag, pa_stream_t stream) {
    return norm_rope(q, q_stride, k, k_stride, v, v_stride, q_weight, k_weight, eps, rope, n_pairs,
                     interleaved, positions, n_axes, slot_mapping, T, q_out, k_pool, v_pool, kQ4,
                     1.f, 1.f, shape, err_flag, stream);
}
