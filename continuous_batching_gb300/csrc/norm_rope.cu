// Per-head RMS norm of q and k, rotation by position and the KV write, in one pass: what stands
// between a layer's projections and paged_attention_step.
//
//   y = x * rsqrt(mean_d(x^2) + eps) * w                      (q and k heads; skipped without w)
//   (y_i, y_j) -> (y_i cos a - y_j sin a, y_i sin a + y_j cos a),  a = position[axis] * frequency
//   q -> q_out (bf16), k -> its slot of the K pool, v -> its slot of the V pool unchanged
// with the pairs (i, i + r/2) or (2i, 2i+1) of the first r of D columns; the others pass through.
// Everything between the bf16 input and the single rounding of the output is fp32.
//
// Angles. A pair's frequency is held as turns per position in units of 2^-64 turn
// (pa_rope_pair.step), so position * step in 64-bit integers, wrapping, IS the phase modulo one
// turn, exactly, for positions of any size and sign: nothing is lost to range reduction. Its top
// 32 bits go to fp32 (2^-25 of half a turn) and sincospif. The sines are computed once per token
// and shared by its heads through shared memory; reading them from a table instead would read
// 8 bytes a pair and token from memory, against none here.
//
// Bound by memory: (Hq + 2 Hkv) D read and written per token. D / 8 lanes hold a head, each lane
// the elements of four pairs (two 8-byte pieces r/2 apart, or one of 16 bytes for adjacent
// pairs), so a pair never crosses lanes and the norm is the only exchange (log2(D / 8) shuffles).
// A group of lanes loads up to kUnits heads before it waits for the sines.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "common.h"

using namespace pa_detail;

namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;          // heads a lane group has in flight
constexpr int kMaxTokens = 8;      // tokens per CTA

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
    int32_t T, Hq, Hkv, n_pairs, n_axes, tokens;
    float eps, k_scale, v_scale;
};

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&r);
}

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

template <int D, bool INTER, bool F8>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const RopeParams p) {
    constexpr int kLanes = D / 8;              // lanes per head
    constexpr int kGroups = kThreads / kLanes;
    __shared__ float2 trig[kMaxTokens][D / 2]; // (cos, sin) of a token's pairs
    // the attention kernel that follows waits for this grid before it reads anything; this one
    // in turn waits for what came before it
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const int heads = p.Hq + 2 * p.Hkv;
    const int t0 = int(blockIdx.x) * p.tokens;
    const int nt = min(p.tokens, p.T - t0);
    const int total = nt * heads;
    const int l = threadIdx.x % kLanes;
    const int group = threadIdx.x / kLanes;
    const int n_rot = p.n_pairs / 4;           // lanes whose elements rotate
    const bool turns = l < n_rot;
    // the lane's two four-element pieces: adjacent pairs lie in one 16-byte piece
    const int a = INTER ? 8 * l : turns ? 4 * l : 8 * l;
    const int b = INTER ? 8 * l + 4 : turns ? p.n_pairs + 4 * l : 8 * l + 4;

    for (int u0 = group; u0 - group < total; u0 += kGroups * kUnits) {
        uint2 xa[kUnits], xb[kUnits];
        int tok[kUnits], head[kUnits];
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int u = u0 + i * kGroups;
            tok[i] = u < total ? u / heads : -1;
            head[i] = u - tok[i] * heads;
            if (tok[i] < 0) continue;
            const int64_t t = t0 + tok[i];
            const int h = head[i];
            const __nv_bfloat16* src =
                h < p.Hq           ? p.q + t * p.q_stride + h * D
                : h < p.Hq + p.Hkv ? p.k + t * p.k_stride + (h - p.Hq) * D
                                   : p.v + t * p.v_stride + (h - p.Hq - p.Hkv) * D;
            if constexpr (INTER) {
                const uint4 w = *reinterpret_cast<const uint4*>(src + a);
                xa[i] = make_uint2(w.x, w.y);
                xb[i] = make_uint2(w.z, w.w);
            } else {
                xa[i] = *reinterpret_cast<const uint2*>(src + a);
                xb[i] = *reinterpret_cast<const uint2*>(src + b);
            }
        }
        if (u0 == group) {
            for (int e = threadIdx.x; e < nt * p.n_pairs; e += kThreads) {
                const int t = e / p.n_pairs, i = e - t * p.n_pairs;
                const pa_rope_pair f = p.rope[i];
                int axis = f.axis;
                if (axis < 0 || axis >= p.n_axes) {
                    if (p.err) atomicOr(p.err, PA_DEVERR_META);
                    axis = 0;
                }
                const int64_t pos = p.positions[int64_t(axis) * p.T + t0 + t];
                const uint64_t phase = uint64_t(pos) * f.step;
                float s, c;
                sincospif(float(int32_t(phase >> 32)) * 0x1p-31f, &s, &c);
                trig[t][i] = make_float2(c, s);
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            // a group's lanes agree on the unit, but a warp holds several groups
            const bool on = tok[i] >= 0;
            const int h = head[i];
            const bool is_v = h >= p.Hq + p.Hkv;
            float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (on) {
                x[0] = lo16(xa[i].x);
                x[1] = hi16(xa[i].x);
                x[2] = lo16(xa[i].y);
                x[3] = hi16(xa[i].y);
                x[4] = lo16(xb[i].x);
                x[5] = hi16(xb[i].x);
                x[6] = lo16(xb[i].y);
                x[7] = hi16(xb[i].y);
            }
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int m = kLanes / 2; m; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
            if (!on) continue;
            if (!is_v) {
                const __nv_bfloat16* w = h < p.Hq ? p.wq : p.wk;
                if (w) {
                    const float r = rsqrtf(ss * (1.f / D) + p.eps);
                    const uint2 wa = __ldg(reinterpret_cast<const uint2*>(w + a));
                    const uint2 wb = __ldg(reinterpret_cast<const uint2*>(w + b));
                    x[0] *= r * lo16(wa.x);
                    x[1] *= r * hi16(wa.x);
                    x[2] *= r * lo16(wa.y);
                    x[3] *= r * hi16(wa.y);
                    x[4] *= r * lo16(wb.x);
                    x[5] *= r * hi16(wb.x);
                    x[6] *= r * lo16(wb.y);
                    x[7] *= r * hi16(wb.y);
                }
                if (turns) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 cs = trig[tok[i]][4 * l + e];
                        float& u = INTER ? x[2 * e] : x[e];
                        float& v = INTER ? x[2 * e + 1] : x[4 + e];
                        const float nu = u * cs.x - v * cs.y;
                        v = u * cs.y + v * cs.x;
                        u = nu;
                    }
                }
            }
            const int64_t t = t0 + tok[i];
            if (h < p.Hq) {
                __nv_bfloat16* dst = p.q_out + (t * p.Hq + h) * D;
                const uint2 ya = make_uint2(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]));
                const uint2 yb = make_uint2(bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
                if constexpr (INTER) {
                    *reinterpret_cast<uint4*>(dst + a) = make_uint4(ya.x, ya.y, yb.x, yb.y);
                } else {
                    *reinterpret_cast<uint2*>(dst + a) = ya;
                    *reinterpret_cast<uint2*>(dst + b) = yb;
                }
                continue;
            }
            const int32_t slot = p.slots[t];
            if (slot < 0) continue;                       // "no write" marker
            if (slot >= p.num_slots) {
                if (l == 0 && p.err) atomicOr(p.err, PA_DEVERR_SLOT);
                continue;
            }
            const int kvh = is_v ? h - p.Hq - p.Hkv : h - p.Hq;
            const int64_t at = (int64_t(slot) * p.Hkv + kvh) * D;
            if constexpr (F8) {
                uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_pool : p.k_pool) + at;
                const float s = is_v ? p.v_scale : p.k_scale;
                const uint32_t ya = e4m3x4(x, s), yb = e4m3x4(x + 4, s);
                if constexpr (INTER) {
                    *reinterpret_cast<uint2*>(dst + a) = make_uint2(ya, yb);
                } else {
                    *reinterpret_cast<uint32_t*>(dst + a) = ya;
                    *reinterpret_cast<uint32_t*>(dst + b) = yb;
                }
            } else {
                __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_v ? p.v_pool : p.k_pool) + at;
                // v goes through unchanged: its bits, not a round trip
                const uint2 ya = is_v ? xa[i] : make_uint2(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]));
                const uint2 yb = is_v ? xb[i] : make_uint2(bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
                if constexpr (INTER) {
                    *reinterpret_cast<uint4*>(dst + a) = make_uint4(ya.x, ya.y, yb.x, yb.y);
                } else {
                    *reinterpret_cast<uint2*>(dst + a) = ya;
                    *reinterpret_cast<uint2*>(dst + b) = yb;
                }
            }
        }
    }
}

template <int D, bool INTER, bool F8>
int32_t launch_rope(RopeParams& p, cudaStream_t stream) {
    constexpr int kGroups = kThreads / (D / 8);
    const int heads = p.Hq + 2 * p.Hkv;
    // Tokens per CTA: one, unless a token has so few heads that most lane groups would idle and
    // there are tokens enough to fill the GPU all the same.
    int tokens = std::min(kMaxTokens, std::max(1, kGroups * kUnits / heads));
    while (tokens > 1 && (p.T + tokens - 1) / tokens < 4 * PA_PLAN_CTAS) --tokens;
    p.tokens = tokens;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned((p.T + tokens - 1) / tokens));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return note_cuda(cudaLaunchKernelEx(&cfg, norm_rope_kernel<D, INTER, F8>, p));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int32_t norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                  int64_t v_stride, const void* q_weight, const void* k_weight, float eps,
                  const pa_rope_pair* rope, int32_t n_pairs, int32_t interleaved,
                  const int32_t* positions, int32_t n_axes, const int32_t* slot_mapping, int32_t T,
                  void* q_out, void* k_pool, void* v_pool, bool fp8, float k_scale, float v_scale,
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
    const bool inter = interleaved != 0;
    if (D == 128) {
        if (fp8) return inter ? launch_rope<128, true, true>(p, stream)
                              : launch_rope<128, false, true>(p, stream);
        return inter ? launch_rope<128, true, false>(p, stream)
                     : launch_rope<128, false, false>(p, stream);
    }
    if (fp8) return inter ? launch_rope<64, true, true>(p, stream)
                          : launch_rope<64, false, true>(p, stream);
    return inter ? launch_rope<64, true, false>(p, stream)
                 : launch_rope<64, false, false>(p, stream);
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
        const double turns = inv_freq[i] / 6.283185307179586477;
        // the fraction of a turn, in [0, 1); a tiny negative one would round up to a whole turn
        double frac = turns - std::floor(turns);
        if (frac >= 1.0) frac = 0.0;
        out[i].step = uint64_t(std::ldexp(frac, 64));
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
                     interleaved, positions, n_axes, slot_mapping, T, q_out, k_pool, v_pool, false,
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
                     interleaved, positions, n_axes, slot_mapping, T, q_out, k_pool, v_pool, true,
                     k_scale, v_scale, shape, err_flag, stream);
}
