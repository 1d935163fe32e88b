// A KV cache held in 4 bits: the write, the read back, and the attention step over it.
//
// Layout and quantisation: q4.h. A value is scale * code + minimum per group of 32 columns.
//
// Rows of few tokens (direct_rows or fewer per sequence and KV head: single tokens, drafted tokens) are computed from the codes
// themselves, never expanded to memory; see q4_direct_kernel. Sequences with more rows (chunks) have
// their context expanded once to bf16 in the workspace and go through the tcgen05 step of the bf16
// cache: the products are then the cost, and an expansion of a few us serves every row tile.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "common.h"
#include "q4.h"
#include "sm103.h"

using namespace pa_detail;

namespace {

constexpr int kMaxDevices = 64;

cudaLaunchConfig_t dependent_launch(cudaLaunchAttribute* pdl, dim3 grid, int threads, size_t smem,
                                    cudaStream_t stream) {
    pdl->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl->val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cfg;
}

__device__ __forceinline__ void dependent_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------------------- write and read

struct RowsParams {
    const __nv_bfloat16 *k, *v;         // write: the new rows
    __nv_bfloat16 *k_out, *v_out;       // read: [T, Hkv, D]
    int64_t k_stride, v_stride;         // elements between tokens
    const int32_t* slots;
    uint8_t *k_pool, *v_pool;
    int64_t num_slots, rows;            // rows: T * Hkv
    int32_t Hkv, bs;
    int32_t* err;
};

constexpr int kRowsThreads = 256;
constexpr int kRowsPer = 2;             // rows a lane group takes, so that their loads are in flight together

// D / 8 lanes take a (token, head) of K and of V: 16 bytes each in, a 4-byte word of codes out, the words
// of a row side by side. Bound by memory (656 bytes a token and head for D = 128, K and V, in and out).
template <int D>
__global__ void __launch_bounds__(kRowsThreads) q4_write_kernel(const RowsParams p) {
    constexpr int kLanes = D / 8;
    constexpr int kGroups = kRowsThreads / kLanes;
    dependent_start();
    const int l = threadIdx.x % kLanes;
    const int64_t row0 = int64_t(blockIdx.x) * (kGroups * kRowsPer) + threadIdx.x / kLanes;
    uint4 k[kRowsPer], v[kRowsPer];
    int32_t slot[kRowsPer];
    int head[kRowsPer];
#pragma unroll
    for (int i = 0; i < kRowsPer; ++i) {
        const int64_t row = row0 + i * kGroups;
        slot[i] = -1;
        if (row < p.rows) {
            const int64_t t = row / p.Hkv;
            head[i] = int(row - t * p.Hkv);
            slot[i] = p.slots[t];
            k[i] = *reinterpret_cast<const uint4*>(p.k + t * p.k_stride + head[i] * D + 8 * l);
            v[i] = *reinterpret_cast<const uint4*>(p.v + t * p.v_stride + head[i] * D + 8 * l);
            if (slot[i] >= p.num_slots) {
                if (l == 0 && p.err) atomicOr(p.err, PA_DEVERR_SLOT);
                slot[i] = -1;
            }
        } else {
            k[i] = v[i] = make_uint4(0, 0, 0, 0);
        }
    }
#pragma unroll
    for (int i = 0; i < kRowsPer; ++i) {
        uint32_t kc, kp, vc, vp;
        q4_quantise8({k[i].x, k[i].y, k[i].z, k[i].w}, kc, kp);
        q4_quantise8({v[i].x, v[i].y, v[i].z, v[i].w}, vc, vp);
        vc = q4_pair_groups(vc, l);
        if (slot[i] < 0) continue;
        const int block = slot[i] / p.bs, o = slot[i] - block * p.bs;
        const int64_t at = q4_base<D>(block, p.Hkv, head[i], p.bs);
        q4_store_row<D, false>(p.k_pool, at, p.bs, o, l, kc, kp);
        q4_store_row<D, true>(p.v_pool, at, p.bs, o, l, vc, vp);
    }
}

// Eight columns of a row from its code word and the group's parameters, as bf16.
__device__ __forceinline__ uint4 q4_expand8(uint32_t codes, uint32_t params) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = q4_value((codes >> (4 * i)) & 15u, params);
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                      pack_bf16(x[6], x[7]));
}

template <int D>
__global__ void __launch_bounds__(kRowsThreads) q4_read_kernel(const RowsParams p) {
    constexpr int kLanes = D / 8;
    constexpr int kGroups = kRowsThreads / kLanes;
    dependent_start();
    const int l = threadIdx.x % kLanes;
    const int64_t row0 = int64_t(blockIdx.x) * (kGroups * kRowsPer) + threadIdx.x / kLanes;
    uint32_t kc[kRowsPer], kp[kRowsPer], vc[kRowsPer], vp[kRowsPer];
    bool on[kRowsPer];
#pragma unroll
    for (int i = 0; i < kRowsPer; ++i) {
        const int64_t row = row0 + i * kGroups;
        kc[i] = kp[i] = vc[i] = vp[i] = 0;
        on[i] = false;
        if (row >= p.rows) continue;
        const int64_t t = row / p.Hkv;
        const int head = int(row - t * p.Hkv);
        const int32_t slot = p.slots[t];
        if (slot < 0) continue;
        if (slot >= p.num_slots) {
            if (l == 0 && p.err) atomicOr(p.err, PA_DEVERR_SLOT);
            continue;
        }
        on[i] = true;
        const int block = slot / p.bs, o = slot - block * p.bs;
        const int64_t at = q4_base<D>(block, p.Hkv, head, p.bs);
        const int64_t codes = at + o * kQ4Codes<D>;
        const int64_t params = at + p.bs * kQ4Codes<D> + o * kQ4Params<D>;
        kc[i] = reinterpret_cast<const uint32_t*>(p.k_pool + codes)[q4_word<D, false>(l)];
        vc[i] = reinterpret_cast<const uint32_t*>(p.v_pool + codes)[q4_word<D, true>(l)];
        kp[i] = reinterpret_cast<const uint32_t*>(p.k_pool + params)[l >> 2];
        vp[i] = reinterpret_cast<const uint32_t*>(p.v_pool + params)[l >> 2];
    }
#pragma unroll
    for (int i = 0; i < kRowsPer; ++i) {
        const uint32_t v = q4_pair_groups(vc[i], l);
        if (!on[i]) continue;
        const int64_t to = (row0 + i * kGroups) * D + 8 * l;
        *reinterpret_cast<uint4*>(p.k_out + to) = q4_expand8(kc[i], kp[i]);
        *reinterpret_cast<uint4*>(p.v_out + to) = q4_expand8(v, vp[i]);
    }
}

// ------------------------------------------------------------------------------ expansion

struct ExpandParams {
    const uint8_t *k_pool, *v_pool;
    const int32_t *table, *cu, *ctx;
    const int32_t* list;                // [n][2]: sequence, 128-token block of it
    const int32_t* ex_table;            // [B][cols]: place of every block in the expanded pools, -1
    int32_t* ex_ctx;                    // [B]: the context of the sequences that are expanded, else 0
    __nv_bfloat16 *k_out, *v_out;       // [n][128][Hkv][D]
    int32_t* err;
    int32_t n, B, cols, max_blocks, num_blocks, Hkv, g, bs, direct_rows;
};

// CTA (i, h): block i of the plan's list, head h: 128 tokens of K and V to bf16, one rounding each.
// The values are those of paged_kv_read_q4. Bound by its writes (512 bytes a token and head, 160 read).
// The sequences whose context is expanded whole are told to the attention by ex_ctx; the others (rows that
// are read directly, metadata that the plan was not made for) have a context of 0 there.
template <int D>
__global__ void __launch_bounds__(256) q4_expand_kernel(const ExpandParams p) {
    constexpr int kLanes = D / 8;
    constexpr int kGroups = 256 / kLanes;
    dependent_start();
    const int64_t id = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
    for (int64_t s = id; s < p.B; s += int64_t(gridDim.x) * gridDim.y * 256) {
        const int64_t n_q = int64_t(p.cu[s + 1]) - p.cu[s];
        const int c = p.ctx[s];
        const int64_t blocks = (int64_t(c) + 127) / 128;
        const bool whole = n_q * p.g > p.direct_rows && c > 0 && blocks <= p.cols &&
                           p.ex_table[s * p.cols + blocks - 1] >= 0;
        p.ex_ctx[s] = whole ? c : 0;
    }
    const int seq = p.list[2 * blockIdx.x], first = p.list[2 * blockIdx.x + 1];
    if (seq < 0) return;                                        // padding of the plan
    const int head = blockIdx.y;
    const int ctx = seq < p.B ? p.ctx[seq] : 0;
    if (seq >= p.B || first < 0 || int64_t(first) * 128 >= ctx ||
        (int64_t(ctx) + p.bs - 1) / p.bs > p.max_blocks) {
        if (threadIdx.x == 0 && p.err) atomicOr(p.err, PA_DEVERR_META);
        return;
    }
    const int l = threadIdx.x % kLanes;
    const int32_t* table = p.table + int64_t(seq) * p.max_blocks;
#pragma unroll 2
    for (int i = 0; i < 128 / kGroups; ++i) {
        const int tok = i * kGroups + threadIdx.x / kLanes;
        const int key = first * 128 + tok;                      // < ctx + 128
        uint32_t kc = 0, vc = 0, kp = 0, vp = 0;
        bool on = key < ctx;
        if (on) {
            const int32_t block = table[key / p.bs];
            if (block >= 0 && block < p.num_blocks) {
                const int o = key % p.bs;
                const int64_t at = q4_base<D>(block, p.Hkv, head, p.bs);
                const int64_t codes = at + o * kQ4Codes<D>;
                const int64_t params = at + p.bs * kQ4Codes<D> + o * kQ4Params<D>;
                kc = reinterpret_cast<const uint32_t*>(p.k_pool + codes)[q4_word<D, false>(l)];
                vc = reinterpret_cast<const uint32_t*>(p.v_pool + codes)[q4_word<D, true>(l)];
                kp = reinterpret_cast<const uint32_t*>(p.k_pool + params)[l >> 2];
                vp = reinterpret_cast<const uint32_t*>(p.v_pool + params)[l >> 2];
            } else if (p.err) {
                atomicOr(p.err, PA_DEVERR_BLOCK);               // its keys read as 0
            }
        }
        const uint32_t v = q4_pair_groups(vc, l);
        if (!on) continue;
        const int64_t to = ((int64_t(blockIdx.x) * 128 + tok) * p.Hkv + head) * D + 8 * l;
        *reinterpret_cast<uint4*>(p.k_out + to) = q4_expand8(kc, kp);
        *reinterpret_cast<uint4*>(p.v_out + to) = q4_expand8(v, vp);
    }
}

// ------------------------------------------------------------------- rows read from the codes
//
// An item is one KV head, one tile of query rows (tokens x heads of its group, at most 8 NT of them)
// and one split of the sequence's keys. Each of the CTA's four warps takes every fourth tile of 32 keys and keeps its own
// online softmax; the warps' results are joined in a fixed order at the item's end, the splits' by
// q4_fold_kernel. A split's length depends on the sequence's context alone (q4_split_keys), so a row's
// bits do not depend on the batch.
//
// Why mma.sync and not tcgen05: the contraction's free dimension is at most 8 NT columns, so the tensor
// rate is no concern; what is, is the way of the codes to the tensor core. tcgen05 would take them expanded to
// 16 bits from shared memory or TMEM: four times the cache's bytes written and read once more (the e4m3 path of
// attention.cu, which does this, takes 2.5 T elements/s). mma.sync takes them from
// the registers that unpacked them. So (keys x columns) is the A operand, and with the row order of q4.h
// a lane's 16-byte piece of a row is its fragments:
//   S^T = K Q^T     A = K codes as 128 + u (bf16: the code in the mantissa, no conversion), B = Q^T
//   S = sum_g s_g (q . (128 + u))_g + (m_g - 128 s_g) sum(q_g)
// exact products and fp32 sums: K is never rounded beyond its code.
//   O^T = V^T P^T   A = V codes as u - 8 (exact), B = P^T with the group's scale in it, rounded to bf16
//   O = sum_j bf16(p_j s_jg) (u_j - 8) + sum_j p_j (m_jg + 8 s_jg)        (the second sum in fp32)
// The tensor core turns P^T's layout by movmatrix. u - 8 instead of u: a rounding of p s then weighs as
// much as that of p against a bf16 V; u alone would double it.
//
// Loads: cp.async into a ring of kStages tiles per warp (codes and parameters; keys behind the context
// and blocks outside the pool are filled with zeros), no barrier but the warp's own.
struct DirectParams {
    const __nv_bfloat16* q;
    const uint8_t *k_pool, *v_pool;
    const int32_t *table, *cu, *ctx;
    const pa_work_item* items;
    float* part;                        // [n_items][8 NT][D + 2]: splits' (acc, m, l)
    __nv_bfloat16* out;
    int32_t* err;
    int32_t n_items, B, T, max_blocks, num_blocks, Hq, Hkv, log2g, log2bs, max_ctx;
    float c;                            // log2(e) / sqrt(D)
};

constexpr int kWarps = PA_Q4_WARPS;
constexpr int kKeys = 32;               // keys of a warp's tile

template <int D>
struct Ring {
    static constexpr int kStages = 3;
    static constexpr int kCodes = kKeys * kQ4Codes<D>;
    static constexpr int kParams = kKeys * kQ4Params<D>;
    static constexpr int kStage = 2 * (kCodes + kParams);       // K codes, V codes, K, V parameters
    static constexpr int kWarp = kStages * kStage;
    static constexpr int kBytes = kWarps * kWarp;
};

// What the warps leave for the join at an item's end, over the ring: rows of D + 4 floats (so that a
// quarter warp's 16-byte stores meet every bank once), then (m, l).
template <int D, int NT>
struct Join {
    static constexpr int kRow = D + 4;
    static constexpr int kMl = kWarps * 8 * NT * kRow;          // floats
    static constexpr int kBytes = (kMl + kWarps * 8 * NT * 2) * 4;
};

template <int D, int NT>
constexpr int kDirectSmem = Ring<D>::kBytes > Join<D, NT>::kBytes ? Ring<D>::kBytes
                                                                  : Join<D, NT>::kBytes;

template <int D>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[D / kQ4Group]) {
    if constexpr (D == 128) {
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr) : "memory");
    } else {
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
    }
}

// A lane's part of a V row: its 16-bit words of all groups, two to a register.
template <int D>
__device__ __forceinline__ void lds_halves(uint32_t addr, uint32_t (&w)[D / kQ4Group / 2]) {
    if constexpr (D == 128) {
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
    } else {
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr) : "memory");
    }
}

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool on) {
    const uint32_t n = on ? BYTES : 0;                          // 0: the place is filled with zeros
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(n), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// D (+)= A B, A 16 x 16 and B 16 x 8 bf16, fp32 accumulator.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
                 "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t w) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(w));
    return r;
}

// Nibble K of both 16-bit halves as bf16 128 + u.
template <int K>
__device__ __forceinline__ uint32_t biased(uint32_t w) {
    return ((w >> (4 * K)) & 0x000F000Fu) | 0x43004300u;
}
// ... as bf16 u - 8.
template <int K>
__device__ __forceinline__ uint32_t centred(uint32_t w) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(biased<K>(w)), "r"(0x43084308u));
    return r;
}

__device__ __forceinline__ float scale_of(uint32_t params) { return __uint_as_float(params << 16); }
__device__ __forceinline__ float min_of(uint32_t params) {
    return __uint_as_float(params & 0xFFFF0000u);
}

// A lane (r = lane / 4, c = lane % 4) holds of every 16-key block the scores of keys r and r + 8 with
// rows 2 c and 2 c + 1 of each column tile; of O^T four adjacent columns 32 g + 4 r + .. of the same rows.
template <int D, int NT>
struct Rows {
    static constexpr int G = D / kQ4Group;
    uint32_t qb[NT][G][4];              // Q^T fragments of the group's two steps
    uint64_t qs[NT][G];                 // sums of q over the group, rows 2 c and 2 c + 1
    float o[NT][2 * G][4];
    uint64_t z[NT][G];                  // sum of p (m + 8 s), this lane's keys
    uint64_t l[NT];                     // sum of p, this lane's keys
    float m[NT][2];                     // reference maximum, in raw scores
    int pos[NT][2];                     // position of the row
};

// Two keys' weights for two rows: p * scale as bf16 pairs, p (m + 8 s) onto z.
__device__ __forceinline__ void q4_weigh(uint64_t p0, uint64_t p1, uint64_t s0, uint64_t s1, uint64_t m0,
                                         uint64_t m1, uint32_t& w0, uint32_t& w1, uint64_t& z) {
    float a, b;
    f2_split(mul2(p0, s0), a, b);
    w0 = pack_bf16(a, b);
    f2_split(mul2(p1, s1), a, b);
    w1 = pack_bf16(a, b);
    z = fma2(p0, m0, z);
    z = fma2(p1, m1, z);
}

// One tile of 32 keys, from key0 on. MASK: some key lies behind some row.
template <int D, int NT, bool MASK>
__device__ __forceinline__ void q4_tile(uint32_t stage, Rows<D, NT>& R, float c, int key0, int lane) {
    constexpr int G = D / kQ4Group;
    using L = Ring<D>;
    const int r = lane >> 2, cc = lane & 3;
    float x[NT][2][4];                  // [column tile][16 keys][key r: rows 2c, 2c + 1; key r + 8]
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t ka[G], kb[G], pa[G], pb[G];
        const uint32_t row = stage + (16 * h + r) * kQ4Codes<D> + cc * (4 * G);
        lds_words<D>(row, ka);
        lds_words<D>(row + 8 * kQ4Codes<D>, kb);
        const uint32_t par = stage + 2 * L::kCodes + (16 * h + r) * kQ4Params<D>;
        lds_words<D>(par, pa);
        lds_words<D>(par + 8 * kQ4Params<D>, pb);
        uint64_t sa[NT], sb[NT];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float raw[NT][4];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                raw[j][0] = raw[j][1] = raw[j][2] = raw[j][3] = 0.f;
                mma(raw[j], biased<0>(ka[g]), biased<0>(kb[g]), biased<1>(ka[g]), biased<1>(kb[g]),
                    R.qb[j][g][0], R.qb[j][g][1]);
                mma(raw[j], biased<2>(ka[g]), biased<2>(kb[g]), biased<3>(ka[g]), biased<3>(kb[g]),
                    R.qb[j][g][2], R.qb[j][g][3]);
            }
            const float s0 = scale_of(pa[g]), s1 = scale_of(pb[g]);
            const float m0 = fmaf(-128.f, s0, min_of(pa[g])), m1 = fmaf(-128.f, s1, min_of(pb[g]));
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint64_t ra = f2(raw[j][0], raw[j][1]), rb = f2(raw[j][2], raw[j][3]);
                sa[j] = g ? fma2(ra, f2(s0, s0), sa[j]) : mul2(ra, f2(s0, s0));
                sb[j] = g ? fma2(rb, f2(s1, s1), sb[j]) : mul2(rb, f2(s1, s1));
                sa[j] = fma2(R.qs[j][g], f2(m0, m0), sa[j]);
                sb[j] = fma2(R.qs[j][g], f2(m1, m1), sb[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            f2_split(sa[j], x[j][h][0], x[j][h][1]);
            f2_split(sb[j], x[j][h][2], x[j][h][3]);
        }
    }
    // online softmax; the reference maximum moves when the rows' maximum outgrows it by 2^8
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        float mx[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if constexpr (MASK) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        if (key0 + 16 * h + 8 * b + r > R.pos[j][e]) x[j][h][2 * b + e] = -INFINITY;
            }
            mx[e] = fmaxf(fmaxf(x[j][0][e], x[j][0][2 + e]), fmaxf(x[j][1][e], x[j][1][2 + e]));
        }
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) {
            mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], d));
            mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], d));
        }
        float a[2], nmc[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float old = R.m[j][e], now = fmaxf(old, mx[e]);
            const bool move = old == -INFINITY ? now != -INFINITY : (now - old) * c > 8.f;
            R.m[j][e] = move ? now : old;
            const float use = R.m[j][e] == -INFINITY ? 0.f : R.m[j][e];
            a[e] = !move || old == -INFINITY ? 1.f : ex2((old - use) * c);
            nmc[e] = -use * c;
        }
        if (__any_sync(0xffffffffu, a[0] != 1.f || a[1] != 1.f)) {
            const uint64_t a2 = f2(a[0], a[1]);
            R.l[j] = mul2(R.l[j], a2);
#pragma unroll
            for (int g = 0; g < G; ++g) R.z[j][g] = mul2(R.z[j][g], a2);
#pragma unroll
            for (int t = 0; t < 2 * G; ++t) {
                R.o[j][t][0] *= a[0];
                R.o[j][t][1] *= a[1];
                R.o[j][t][2] *= a[0];
                R.o[j][t][3] *= a[1];
            }
        }
        const uint64_t n2 = f2(nmc[0], nmc[1]), c2 = f2(c, c);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float& u = x[j][h][2 * b];
                float& v = x[j][h][2 * b + 1];
                f2_split(fma2(f2(u, v), c2, n2), u, v);
                u = ex2(u);
                v = ex2(v);
                R.l[j] = add2(R.l[j], f2(u, v));
            }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        // keys 2 c, 2 c + 1 and those 8 behind them: even keys of eight lie before odd ones
        uint32_t v[4][G / 2], pa[G], pb[G];
        const uint32_t row = stage + L::kCodes + (16 * h + cc) * kQ4Codes<D> + r * (2 * G);
#pragma unroll
        for (int k = 0; k < 4; ++k) lds_halves<D>(row + 4 * k * kQ4Codes<D>, v[k]);
        const uint32_t par = stage + 2 * L::kCodes + L::kParams + (16 * h + r) * kQ4Params<D>;
        lds_words<D>(par, pa);
        lds_words<D>(par + 8 * kQ4Params<D>, pb);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float s0 = scale_of(pa[g]), s1 = scale_of(pb[g]);
            const float m0 = fmaf(8.f, s0, min_of(pa[g])), m1 = fmaf(8.f, s1, min_of(pb[g]));
            const uint32_t sel = g & 1 ? 0x7632 : 0x5410;
            const uint32_t lo = __byte_perm(v[0][g / 2], v[1][g / 2], sel);
            const uint32_t hi = __byte_perm(v[2][g / 2], v[3][g / 2], sel);
            const uint32_t a0 = centred<0>(lo), a1 = centred<1>(lo), a2 = centred<2>(lo), a3 = centred<3>(lo);
            const uint32_t b0 = centred<0>(hi), b1 = centred<1>(hi), b2 = centred<2>(hi), b3 = centred<3>(hi);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                uint32_t w0, w1;
                if constexpr (MASK) {
                    // a masked key's parameters may be anything (its p is 0): they are taken as 0, with the
                    // arithmetic of the other branch, so that a row's bits do not depend on its tile's others
                    const bool on0 = key0 + 16 * h + r <= R.pos[j][0], on1 = key0 + 16 * h + r <= R.pos[j][1];
                    const bool on2 = key0 + 16 * h + 8 + r <= R.pos[j][0], on3 = key0 + 16 * h + 8 + r <= R.pos[j][1];
                    q4_weigh(f2(x[j][h][0], x[j][h][1]), f2(x[j][h][2], x[j][h][3]),
                             f2(on0 ? s0 : 0.f, on1 ? s0 : 0.f), f2(on2 ? s1 : 0.f, on3 ? s1 : 0.f),
                             f2(on0 ? m0 : 0.f, on1 ? m0 : 0.f), f2(on2 ? m1 : 0.f, on3 ? m1 : 0.f), w0, w1,
                             R.z[j][g]);
                } else {
                    q4_weigh(f2(x[j][h][0], x[j][h][1]), f2(x[j][h][2], x[j][h][3]), f2(s0, s0), f2(s1, s1),
                             f2(m0, m0), f2(m1, m1), w0, w1, R.z[j][g]);
                }
                w0 = transpose8(w0);
                w1 = transpose8(w1);
                mma(R.o[j][2 * g], a0, a1, b0, b1, w0, w1);
                mma(R.o[j][2 * g + 1], a2, a3, b2, b3, w0, w1);
            }
        }
    }
}

template <int D, int NT>
__global__ void __launch_bounds__(32 * kWarps, NT == 1 ? 3 : 2) q4_direct_kernel(const DirectParams p) {
    constexpr int G = D / kQ4Group;
    constexpr int kCols = 8 * NT;
    using L = Ring<D>;
    using J = Join<D, NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    dependent_start();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, cc = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * L::kWarp;
    float* const join = reinterpret_cast<float*>(smem);
    const int bs = 1 << p.log2bs, gq = 1 << p.log2g;

    for (int idx = blockIdx.x; idx < p.n_items;) {
        const pa_work_item it = p.items[idx];
        if (it.n_q == 0) break;                                 // padding: no more work
        // ---- the item against the metadata it points at
        bool good = it.kind == PA_ITEM_DIRECT && it.seq >= 0 && it.seq < p.B && it.kv_head >= 0 &&
                    it.kv_head < p.Hkv && it.n_q > 0 && it.n_q <= (kCols >> p.log2g) && it.q_start >= 0 &&
                    it.q_start <= p.T - it.n_q && it.split >= 0 && it.n_splits > it.split &&
                    it.tile0 >= 0 && it.tile0 <= p.n_items - it.n_splits;
        int ctx = 0, pos0 = 0, k_begin = 0, k_end = 0;
        if (good) {
            ctx = p.ctx[it.seq];
            const int cu0 = p.cu[it.seq], cu1 = p.cu[it.seq + 1];
            good = ctx > 0 && ctx <= p.max_ctx && cu0 <= it.q_start && it.q_start + it.n_q <= cu1 &&
                   int64_t(cu1) - cu0 <= ctx && (int64_t(ctx) + bs - 1) / bs <= p.max_blocks;
            pos0 = ctx - cu1 + it.q_start;                      // position of the first row
            const int keys = pos0 + it.n_q;                     // up to the last row
            const int64_t len = good ? q4_split_keys(ctx) : 1;
            good = good && (keys + len - 1) / len == it.n_splits;
            k_begin = int(it.split * len);
            k_end = int(min(int64_t(keys), k_begin + len));
        }
        if (!good && threadIdx.x == 0 && p.err) atomicOr(p.err, PA_DEVERR_META);
        if (good) {
            const int rows = it.n_q << p.log2g;
            Rows<D, NT> R;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int row = 8 * j + r;
                const bool on = row < rows;
                const __nv_bfloat16* src =
                    p.q + (int64_t(it.q_start + (on ? row >> p.log2g : 0)) * p.Hq + it.kv_head * gq +
                           (on ? row & (gq - 1) : 0)) * D;
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (on) w = __ldg(reinterpret_cast<const uint4*>(src + 32 * g + 8 * cc));
                    R.qb[j][g][0] = __byte_perm(w.x, w.z, 0x5410);      // columns 0, 4
                    R.qb[j][g][1] = __byte_perm(w.x, w.z, 0x7632);      // 1, 5
                    R.qb[j][g][2] = __byte_perm(w.y, w.w, 0x5410);      // 2, 6
                    R.qb[j][g][3] = __byte_perm(w.y, w.w, 0x7632);      // 3, 7
                    float s = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s += scale_of(R.qb[j][g][i]) + min_of(R.qb[j][g][i]);
                    s += __shfl_xor_sync(0xffffffffu, s, 1);
                    s += __shfl_xor_sync(0xffffffffu, s, 2);
                    R.qs[j][g] = f2(__shfl_sync(0xffffffffu, s, 8 * cc),
                                    __shfl_sync(0xffffffffu, s, 8 * cc + 4));
                    R.z[j][g] = 0;
                }
#pragma unroll
                for (int t = 0; t < 2 * G; ++t)
                    R.o[j][t][0] = R.o[j][t][1] = R.o[j][t][2] = R.o[j][t][3] = 0.f;
                R.l[j] = 0;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    R.m[j][e] = -INFINITY;
                    // rows behind the last one see what the last one sees
                    R.pos[j][e] = pos0 + (min(8 * j + 2 * cc + e, rows - 1) >> p.log2g);
                }
            }
            // ---- the warp's tiles: keys k_begin + 32 (warp + kWarps n)
            const int n_keys = k_end - k_begin;
            const int tiles = (n_keys + kKeys - 1) / kKeys;
            const int n = tiles > warp ? (tiles - warp + kWarps - 1) / kWarps : 0;
            const int32_t* table = p.table + int64_t(it.seq) * p.max_blocks;
            // lane i holds the block of eight keys i % 4 of tile i / 4 of the next eight tiles
            const auto blocks_from = [&](int tile) {
                const int key = k_begin + (warp + kWarps * (tile + (lane >> 2))) * kKeys + 8 * (lane & 3);
                int b = -1;
                if (tile + (lane >> 2) < n && key < k_end) {
                    b = __ldg(table + (key >> p.log2bs));
                    if (b < 0 || b >= p.num_blocks) {
                        if (p.err) atomicOr(p.err, PA_DEVERR_BLOCK);
                        b = -1;                                 // its keys read as 0
                    }
                }
                return b;
            };
            int blocks = blocks_from(0), blocks_next = blocks_from(8);
            const auto issue = [&](int tile) {
                if (tile < n) {
                    if (tile && (tile & 7) == 0) {
                        blocks = blocks_next;
                        blocks_next = blocks_from(tile + 8);
                    }
                    const int key0 = k_begin + (warp + kWarps * tile) * kKeys;
                    const uint32_t stage = ring + (tile % L::kStages) * L::kStage;
                    constexpr int kPieces = kQ4Codes<D> / 16;           // of a code row
                    constexpr int kAtOnce = 32 / kPieces;               // keys the warp's lanes cover
                    const int piece = lane % kPieces;
#pragma unroll
                    for (int i = 0; i < kKeys / kAtOnce; ++i) {
                        const int place = i * kAtOnce + lane / kPieces;     // row in the stage
                        const int b = __shfl_sync(0xffffffffu, blocks, (tile & 7) * 4 + place / 8);
                        const int w = place & 7;
                        // V: even keys of eight first (see q4_tile)
                        const int v_key = (place & ~7) + (w < 4 ? 2 * w : 2 * w - 7);
                        const int64_t at = q4_base<D>(b < 0 ? 0 : b, p.Hkv, it.kv_head, bs) + 16 * piece;
                        cp_async<16>(stage + place * kQ4Codes<D> + 16 * piece,
                                     p.k_pool + at + ((key0 + place) & (bs - 1)) * kQ4Codes<D>,
                                     b >= 0 && key0 + place < k_end);
                        cp_async<16>(stage + L::kCodes + place * kQ4Codes<D> + 16 * piece,
                                     p.v_pool + at + ((key0 + v_key) & (bs - 1)) * kQ4Codes<D>,
                                     b >= 0 && key0 + v_key < k_end);
                    }
                    const int b = __shfl_sync(0xffffffffu, blocks, (tile & 7) * 4 + lane / 8);
                    const int64_t at = q4_base<D>(b < 0 ? 0 : b, p.Hkv, it.kv_head, bs) +
                                       bs * kQ4Codes<D> + ((key0 + lane) & (bs - 1)) * kQ4Params<D>;
                    const uint32_t to = stage + 2 * L::kCodes + lane * kQ4Params<D>;
                    const bool on = b >= 0 && key0 + lane < k_end;
                    cp_async<kQ4Params<D>>(to, p.k_pool + at, on);
                    cp_async<kQ4Params<D>>(to + L::kParams, p.v_pool + at, on);
                }
                cp_commit();
            };
#pragma unroll
            for (int i = 0; i < L::kStages - 1; ++i) issue(i);
            for (int i = 0; i < n; ++i) {
                cp_wait<L::kStages - 2>();
                __syncwarp();                                   // every lane's copies, every lane done
                issue(i + L::kStages - 1);
                const int key0 = k_begin + (warp + kWarps * i) * kKeys;
                const uint32_t stage = ring + (i % L::kStages) * L::kStage;
                if (key0 + kKeys - 1 <= pos0) q4_tile<D, NT, false>(stage, R, p.c, key0, lane);
                else q4_tile<D, NT, true>(stage, R, p.c, key0, lane);
            }
            cp_wait<0>();
            // ---- join the warps: rows in shared memory, over the ring
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float l[2];
                f2_split(R.l[j], l[0], l[1]);
#pragma unroll
                for (int d = 4; d <= 16; d <<= 1) {
                    l[0] += __shfl_xor_sync(0xffffffffu, l[0], d);
                    l[1] += __shfl_xor_sync(0xffffffffu, l[1], d);
                }
                float* to = join + (warp * kCols + 8 * j + 2 * cc) * J::kRow + 4 * r;
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    float z[2];
                    f2_split(R.z[j][g], z[0], z[1]);
#pragma unroll
                    for (int d = 4; d <= 16; d <<= 1) {
                        z[0] += __shfl_xor_sync(0xffffffffu, z[0], d);
                        z[1] += __shfl_xor_sync(0xffffffffu, z[1], d);
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *reinterpret_cast<float4*>(to + e * J::kRow + 32 * g) =
                            make_float4(R.o[j][2 * g][e] + z[e], R.o[j][2 * g][2 + e] + z[e],
                                        R.o[j][2 * g + 1][e] + z[e], R.o[j][2 * g + 1][2 + e] + z[e]);
                }
                if (r == 0) {
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *reinterpret_cast<float2*>(join + J::kMl + (warp * kCols + 8 * j + 2 * cc + e) * 2) =
                            make_float2(R.m[j][e], l[e]);
                }
            }
            __syncthreads();
            constexpr int kPer = D / 4;                         // threads of a row
            for (int u = threadIdx.x; u < rows * kPer; u += 32 * kWarps) {
                const int row = u / kPer, col = (u % kPer) * 4;
                float M = -INFINITY, Lsum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
                float2 ml[kWarps];
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    ml[w] = *reinterpret_cast<const float2*>(join + J::kMl + (w * kCols + row) * 2);
                    M = fmaxf(M, ml[w].x);
                }
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float f = ml[w].x == -INFINITY ? 0.f : ex2((ml[w].x - M) * p.c);
                    const float4 a = *reinterpret_cast<const float4*>(join + (w * kCols + row) * J::kRow + col);
                    Lsum = fmaf(ml[w].y, f, Lsum);
                    acc[0] = fmaf(a.x, f, acc[0]);
                    acc[1] = fmaf(a.y, f, acc[1]);
                    acc[2] = fmaf(a.z, f, acc[2]);
                    acc[3] = fmaf(a.w, f, acc[3]);
                }
                if (it.n_splits == 1) {
                    const float inv = __frcp_rn(Lsum);
                    const int64_t at = (int64_t(it.q_start + (row >> p.log2g)) * p.Hq + it.kv_head * gq +
                                        (row & (gq - 1))) * D + col;
                    *reinterpret_cast<uint2*>(p.out + at) = make_uint2(
                        pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
                } else {
                    float* part = p.part + int64_t(it.tile0 + it.split) * (kCols * (D + 2));
                    *reinterpret_cast<float4*>(part + row * D + col) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                    if (col == 0)
                        *reinterpret_cast<float2*>(part + kCols * D + 2 * row) = make_float2(M, Lsum);
                }
            }
            __syncthreads();                                    // the ring is free again
        }
        if (it.next <= 0) break;
        if (it.next <= idx || it.next >= p.n_items) {
            if (threadIdx.x == 0 && p.err) atomicOr(p.err, PA_DEVERR_META);
            break;
        }
        idx = it.next;
    }
}

// Joins the splits of a tile of rows and head, in ascending order: one CTA per entry of the plan's fold
// list (items of split 0 with more splits behind them), a warp per row at a time. A part whose row has no
// key in its split holds m = -infinity and l = 0.
template <int D, int NT>
__global__ void __launch_bounds__(128) q4_fold_kernel(const DirectParams p, const int32_t* fold) {
    constexpr int kCols = 8 * NT;
    constexpr int kPart = kCols * (D + 2);
    constexpr int kBatch = 8;
    dependent_start();
    const int idx = fold[blockIdx.x];
    if (idx < 0) return;                                        // padding
    if (idx >= p.n_items) {
        if (threadIdx.x == 0 && p.err) atomicOr(p.err, PA_DEVERR_META);
        return;
    }
    const pa_work_item it = p.items[idx];
    if (it.kind != PA_ITEM_DIRECT || it.split != 0 || it.n_splits < 2 || it.tile0 < 0 ||
        it.tile0 > p.n_items - it.n_splits || it.n_q < 1 || it.n_q > (kCols >> p.log2g) ||
        it.q_start < 0 || it.q_start > p.T - it.n_q || it.kv_head < 0 || it.kv_head >= p.Hkv ||
        it.seq < 0 || it.seq >= p.B) {
        if (threadIdx.x == 0 && p.err) atomicOr(p.err, PA_DEVERR_META);
        return;
    }
    // an item that the direct kernel refused has left no parts
    const int ctx = p.ctx[it.seq], cu0 = p.cu[it.seq], cu1 = p.cu[it.seq + 1];
    if (ctx <= 0 || ctx > p.max_ctx || cu0 > it.q_start || it.q_start + it.n_q > cu1 ||
        int64_t(cu1) - cu0 > ctx)
        return;
    const int64_t keys = ctx - cu1 + it.q_start + it.n_q, len = q4_split_keys(ctx);
    if ((keys + len - 1) / len != it.n_splits || (int64_t(ctx) + (1 << p.log2bs) - 1) >> p.log2bs > p.max_blocks)
        return;
    const int gq = 1 << p.log2g, rows = it.n_q << p.log2g;
    constexpr int kPer = D / 4;
    for (int u = threadIdx.x; u < rows * kPer; u += 128) {
        const int row = u / kPer, col = (u % kPer) * 4;
        const float* part = p.part + int64_t(it.tile0) * kPart;
        float M = -INFINITY, Lsum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
        for (int s0 = 0; s0 < it.n_splits; s0 += kBatch) {
            float2 ml[kBatch];
            float4 a[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (s0 + i < it.n_splits) {
                    const float* from = part + int64_t(s0 + i) * kPart;
                    a[i] = *reinterpret_cast<const float4*>(from + row * D + col);
                    ml[i] = *reinterpret_cast<const float2*>(from + kCols * D + 2 * row);
                }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (s0 + i >= it.n_splits) break;
                const float now = fmaxf(M, ml[i].x);
                const float fa = M == -INFINITY ? 0.f : ex2((M - now) * p.c);
                const float fb = ml[i].x == -INFINITY ? 0.f : ex2((ml[i].x - now) * p.c);
                Lsum = Lsum * fa + ml[i].y * fb;
                acc[0] = acc[0] * fa + a[i].x * fb;
                acc[1] = acc[1] * fa + a[i].y * fb;
                acc[2] = acc[2] * fa + a[i].z * fb;
                acc[3] = acc[3] * fa + a[i].w * fb;
                M = now;
            }
        }
        const float inv = __frcp_rn(Lsum);
        const int64_t at = (int64_t(it.q_start + (row >> p.log2g)) * p.Hq + it.kv_head * gq +
                            (row & (gq - 1))) * D + col;
        *reinterpret_cast<uint2*>(p.out + at) = make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv),
                                                           pack_bf16(acc[2] * inv, acc[3] * inv));
    }
}

// ------------------------------------------------------------------------------- host side

template <int D, int NT>
int32_t launch_direct(const DirectParams& p, const int32_t* fold, int32_t n_fold, cudaStream_t stream) {
    static std::atomic<bool> raised[kMaxDevices];               // zero-initialised: not raised yet
    int dev = 0;
    int32_t st = note_cuda(cudaGetDevice(&dev));
    if (st) return st;
    if (dev < 0 || dev >= kMaxDevices) return PA_ERR_INVALID;
    constexpr int smem = kDirectSmem<D, NT>;
    if (!raised[dev].load(std::memory_order_acquire)) {
        st = note_cuda(cudaFuncSetAttribute(q4_direct_kernel<D, NT>,
                                            cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
        if (st) return st;
        raised[dev].store(true, std::memory_order_release);
    }
    cudaLaunchAttribute pdl;
    const int lists = NT == 1 ? PA_Q4_LISTS_8 : PA_Q4_LISTS_16;
    auto cfg = dependent_launch(&pdl, dim3(unsigned(std::min(p.n_items, lists))), 32 * kWarps, smem, stream);
    st = note_cuda(cudaLaunchKernelEx(&cfg, q4_direct_kernel<D, NT>, p));
    if (st || n_fold == 0) return st;
    cfg = dependent_launch(&pdl, dim3(unsigned(n_fold)), 128, 0, stream);
    return note_cuda(cudaLaunchKernelEx(&cfg, q4_fold_kernel<D, NT>, p, fold));
}

int ilog2(int x) {
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int32_t check_rows(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                   const int32_t* slots, int32_t T, const void* k_pool, const void* v_pool,
                   const pa_shape* shape) {
    const int64_t row = int64_t(shape->num_kv_heads) * shape->head_dim;
    if (!k || !v || !slots || !k_pool || !v_pool) return PA_ERR_INVALID;
    if (k_stride < row || v_stride < row || (k_stride | v_stride) % 8) return PA_ERR_INVALID;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_pool) || !aligned16(v_pool)) return PA_ERR_INVALID;
    return PA_OK;
}

template <bool WRITE>
int32_t launch_rows(RowsParams& p, int32_t T, const int32_t* slots, void* k_pool, void* v_pool,
                    const pa_shape* shape, int32_t* err, cudaStream_t stream) {
    p.slots = slots;
    p.k_pool = static_cast<uint8_t*>(k_pool);
    p.v_pool = static_cast<uint8_t*>(v_pool);
    p.num_slots = int64_t(shape->num_blocks) * shape->block_size;
    p.rows = int64_t(T) * shape->num_kv_heads;
    p.Hkv = shape->num_kv_heads;
    p.bs = shape->block_size;
    p.err = err;
    const int per = kRowsThreads / (shape->head_dim / 8) * kRowsPer;
    const int64_t blocks = (p.rows + per - 1) / per;
    if (blocks > INT32_MAX) return PA_ERR_SHAPE;
    cudaLaunchAttribute pdl;
    auto cfg = dependent_launch(&pdl, dim3(unsigned(blocks)), kRowsThreads, 0, stream);
    if (shape->head_dim == 128)
        return note_cuda(cudaLaunchKernelEx(&cfg, WRITE ? q4_write_kernel<128> : q4_read_kernel<128>, p));
    return note_cuda(cudaLaunchKernelEx(&cfg, WRITE ? q4_write_kernel<64> : q4_read_kernel<64>, p));
}

// Parts of the workspace, each a multiple of 256 bytes.
struct Space {
    size_t parts, partials, expanded, ctx, total;   // sizes: split parts, decode partials, one pool, contexts
};

Space space_of(const pa_shape* s, const pa_q4_plan* p) {
    const auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    Space w{};
    const int D = s->head_dim, g = s->num_q_heads / s->num_kv_heads;
    const int cols = p->direct_rows > 8 ? 16 : 8;
    if (p->n_fold > 0) w.parts = up(size_t(p->n_direct) * cols * (D + 2) * 4);
    if (p->n_chunk > 0) {
        // single tokens are among the expanded rows only where a group is larger than direct_rows
        if (p->direct_rows < g && p->max_ctx > PA_SPLIT_TOKENS)
            w.partials = up(pa_workspace_bytes(s, p->T, p->max_ctx));
        w.expanded = up(size_t(p->n_expand) * 128 * s->num_kv_heads * D * 2);
        w.ctx = up(size_t(p->B) * 4);
    }
    w.total = w.parts + w.partials + 2 * w.expanded + w.ctx;
    return w;
}

}  // namespace

extern "C" int32_t paged_kv_write_q4(const void* k_new, int64_t k_stride, const void* v_new,
                                     int64_t v_stride, const int32_t* slot_mapping, int32_t T,
                                     void* k_pool, void* v_pool, const pa_shape* shape,
                                     int32_t* err_flag, pa_stream_t stream) {
    int32_t st = check_shape(shape);
    if (st) return st;
    if (T < 0) return PA_ERR_INVALID;
    if (T == 0) return PA_OK;
    if ((st = check_rows(k_new, k_stride, v_new, v_stride, slot_mapping, T, k_pool, v_pool, shape)))
        return st;
    RowsParams p{};
    p.k = static_cast<const __nv_bfloat16*>(k_new);
    p.v = static_cast<const __nv_bfloat16*>(v_new);
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    return launch_rows<true>(p, T, slot_mapping, k_pool, v_pool, shape, err_flag, stream);
}

extern "C" int32_t paged_kv_read_q4(const int32_t* slot_mapping, int32_t T, const void* k_pool,
                                    const void* v_pool, void* k_out, void* v_out,
                                    const pa_shape* shape, int32_t* err_flag, pa_stream_t stream) {
    int32_t st = check_shape(shape);
    if (st) return st;
    if (T < 0) return PA_ERR_INVALID;
    if (T == 0) return PA_OK;
    const int64_t row = int64_t(shape->num_kv_heads) * shape->head_dim;
    if ((st = check_rows(k_out, row, v_out, row, slot_mapping, T, k_pool, v_pool, shape))) return st;
    RowsParams p{};
    p.k_out = static_cast<__nv_bfloat16*>(k_out);
    p.v_out = static_cast<__nv_bfloat16*>(v_out);
    return launch_rows<false>(p, T, slot_mapping, const_cast<void*>(k_pool), const_cast<void*>(v_pool),
                              shape, err_flag, stream);
}

extern "C" size_t pa_q4_workspace_bytes(const pa_shape* shape, const pa_q4_plan* plan) {
    if (check_shape(shape) || !plan) return 0;
    return space_of(shape, plan).total;
}

extern "C" int32_t paged_attention_step_q4(const void* q, const void* k_pool, const void* v_pool,
                                           const int32_t* block_table, int32_t max_blocks,
                                           const int32_t* cu_seqlens_q, const int32_t* ctx_lens,
                                           const pa_q4_plan* plan, const int32_t* words,
                                           void* workspace, size_t ws_bytes, void* out,
                                           const pa_shape* shape, int32_t* err_flag,
                                           pa_stream_t stream) {
    int32_t st = check_shape(shape);
    if (st) return st;
    if (!plan || max_blocks < 0) return PA_ERR_INVALID;
    const pa_q4_plan& P = *plan;
    if ((st = check_q4_plan(shape, P))) return st;
    if (P.T == 0 || P.words == 0) return PA_OK;
    if (!q || !k_pool || !v_pool || !block_table || !cu_seqlens_q || !ctx_lens || !words || !out)
        return PA_ERR_INVALID;
    if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out)) return PA_ERR_INVALID;
    if (int64_t(shape->num_blocks) * shape->block_size > INT32_MAX) return PA_ERR_SHAPE;
    const Space w = space_of(shape, plan);
    if (w.total > 0 && (!workspace || ws_bytes < w.total)) return PA_ERR_WORKSPACE;
    if (w.total > 0 && !aligned16(workspace)) return PA_ERR_INVALID;
    uint8_t* at = static_cast<uint8_t*>(workspace);
    const int D = shape->head_dim, Hq = shape->num_q_heads, Hkv = shape->num_kv_heads, g = Hq / Hkv;
    const Q4Words f = q4_words(P);
    if (P.n_direct > 0) {
        DirectParams p{};
        p.q = static_cast<const __nv_bfloat16*>(q);
        p.k_pool = static_cast<const uint8_t*>(k_pool);
        p.v_pool = static_cast<const uint8_t*>(v_pool);
        p.table = block_table;
        p.cu = cu_seqlens_q;
        p.ctx = ctx_lens;
        p.items = reinterpret_cast<const pa_work_item*>(words + f.direct);
        p.part = reinterpret_cast<float*>(at);
        p.out = static_cast<__nv_bfloat16*>(out);
        p.err = err_flag;
        p.n_items = P.n_direct;
        p.B = P.B;
        p.T = P.T;
        p.max_blocks = max_blocks;
        p.num_blocks = shape->num_blocks;
        p.Hq = Hq;
        p.Hkv = Hkv;
        p.log2g = ilog2(g);
        p.log2bs = ilog2(shape->block_size);
        // without a fold no row may have a second split: its part would have no place
        p.max_ctx = P.n_fold > 0 ? P.max_ctx : int32_t(std::min<int64_t>(P.max_ctx, q4_one_split()));
        p.c = float(1.4426950408889634 / std::sqrt(double(D)));
        const int32_t* fold = words + f.fold;
        const bool wide = P.direct_rows > 8;
        st = D == 128 ? (wide ? launch_direct<128, 2>(p, fold, P.n_fold, stream)
                              : launch_direct<128, 1>(p, fold, P.n_fold, stream))
                      : (wide ? launch_direct<64, 2>(p, fold, P.n_fold, stream)
                              : launch_direct<64, 1>(p, fold, P.n_fold, stream));
        if (st) return st;
    }
    if (P.n_chunk == 0) return PA_OK;
    ExpandParams e{};
    e.k_pool = static_cast<const uint8_t*>(k_pool);
    e.v_pool = static_cast<const uint8_t*>(v_pool);
    e.table = block_table;
    e.cu = cu_seqlens_q;
    e.ctx = ctx_lens;
    e.list = words + f.expand;
    e.ex_table = words + f.table;
    e.k_out = reinterpret_cast<__nv_bfloat16*>(at + w.parts + w.partials);
    e.v_out = reinterpret_cast<__nv_bfloat16*>(at + w.parts + w.partials + w.expanded);
    e.ex_ctx = reinterpret_cast<int32_t*>(at + w.parts + w.partials + 2 * w.expanded);
    e.err = err_flag;
    e.n = P.n_expand;
    e.B = P.B;
    e.cols = P.expand_cols;
    e.max_blocks = max_blocks;
    e.num_blocks = shape->num_blocks;
    e.Hkv = Hkv;
    e.g = g;
    e.bs = shape->block_size;
    e.direct_rows = P.direct_rows;
    cudaLaunchAttribute pdl;
    auto cfg = dependent_launch(&pdl, dim3(unsigned(P.n_expand), unsigned(Hkv)), 256, 0, stream);
    st = note_cuda(D == 128 ? cudaLaunchKernelEx(&cfg, q4_expand_kernel<128>, e)
                            : cudaLaunchKernelEx(&cfg, q4_expand_kernel<64>, e));
    if (st) return st;
    pa_shape ex = *shape;
    ex.block_size = 128;
    ex.num_blocks = P.n_expand;
    return attention_step_expanded(q, e.k_out, e.v_out, e.ex_table, e.cols, cu_seqlens_q, e.ex_ctx, P.B,
                                   P.T, P.max_ctx,
                                   reinterpret_cast<const pa_work_item*>(words + f.chunk), P.n_chunk,
                                   w.partials ? at + w.parts : nullptr, out, &ex, err_flag, stream);
}
