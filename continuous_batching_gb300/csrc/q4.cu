// A KV cache held in 4 bits: the write, the read back, and the attention step over it.
//
// Layout and quantisation: q4.h. A value is scale * code + minimum per group of 32 columns.
//
// Sequences of few rows (tokens x heads of a group, direct_rows or fewer: single tokens, drafted tokens) are
// computed from the codes themselves, never expanded to memory; see q4_direct_kernel. Sequences with more rows
// (chunks) have their context expanded once to 16 bits in the workspace and go through the tcgen05 step of
// the bf16 cache: the products are then the cost, and an expansion of a few us serves every row tile. V and P are
// f16 there, three bits more than bf16, where V's magnitudes allow.
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

int ilog2(int x) {
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

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
    int64_t num_slots;
    uint32_t rows;                      // T * Hkv
    uint32_t div;                       // (row * div) >> div_shift is row / Hkv, for rows below 2^31
    int32_t div_shift;
    int32_t Hkv, log2bs;
    int32_t* err;
};

constexpr int kRowsThreads = 256;

// D / 16 lanes take a (token, head) of K and of V: 32 bytes of each in, two 4-byte words of codes out, the words of a
// row side by side. 672 bytes a token and head of 128 (K and V, in and out); 16,384 tokens of 8 heads take 15.1 us,
// 5.85 TB/s. Lanes of 8 columns, two rows of each, took 23: half as many values to every extreme, scale and address.
template <int D>
__global__ void __launch_bounds__(kRowsThreads) q4_write_kernel(const RowsParams p) {
    constexpr int kLanes = D / 16;
    dependent_start();
    const int l = threadIdx.x % kLanes, bs = 1 << p.log2bs;
    const uint32_t row = blockIdx.x * uint32_t(kRowsThreads / kLanes) + threadIdx.x / kLanes;
    uint32_t k[8] = {}, v[8] = {};
    int32_t slot = -1;
    int head = 0;
    if (row < p.rows) {
        const uint32_t t = uint32_t((uint64_t(row) * p.div) >> p.div_shift);
        head = int(row - t * uint32_t(p.Hkv));
        slot = p.slots[t];
        const uint4* const ks = reinterpret_cast<const uint4*>(p.k + int64_t(t) * p.k_stride + head * D + 16 * l);
        const uint4* const vs = reinterpret_cast<const uint4*>(p.v + int64_t(t) * p.v_stride + head * D + 16 * l);
        const uint4 k0 = ks[0], k1 = ks[1], v0 = vs[0], v1 = vs[1];
        k[0] = k0.x, k[1] = k0.y, k[2] = k0.z, k[3] = k0.w, k[4] = k1.x, k[5] = k1.y, k[6] = k1.z, k[7] = k1.w;
        v[0] = v0.x, v[1] = v0.y, v[2] = v0.z, v[3] = v0.w, v[4] = v1.x, v[5] = v1.y, v[6] = v1.z, v[7] = v1.w;
        if (slot >= p.num_slots) {
            if (l == 0 && p.err) atomicOr(p.err, PA_DEVERR_SLOT);
            slot = -1;
        }
    }
    uint32_t kc[2], kp, vc[2], vp;
    q4_quantise<8>(k, kc, kp);
    q4_quantise<8>(v, vc, vp);
    q4_pair_groups2(vc, l);
    if (slot < 0) return;
    const int o = slot & (bs - 1);
    const int64_t at = q4_base<D>(slot >> p.log2bs, p.Hkv, head, bs);
    q4_store_row2<D, false>(p.k_pool, at, bs, o, l, kc, kp);
    q4_store_row2<D, true>(p.v_pool, at, bs, o, l, vc, vp);
}

// Four lanes take a (token, head) of K and of V, all of their loads in flight. Bound by memory (672 bytes a token and
// head for D = 128, in and out): 16,384 tokens of 8 heads just written, part of them still in L2, take 11.6 us.
template <int D>
__global__ void __launch_bounds__(kRowsThreads) q4_read_kernel(const RowsParams p) {
    constexpr int G = D / kQ4Group;
    dependent_start();
    const int c = threadIdx.x & 3, bs = 1 << p.log2bs;
    const uint32_t row = blockIdx.x * uint32_t(kRowsThreads / 4) + threadIdx.x / 4;
    if (row >= p.rows) return;
    const uint32_t t = uint32_t((uint64_t(row) * p.div) >> p.div_shift);
    const int head = int(row - t * uint32_t(p.Hkv));
    const int32_t slot = p.slots[t];
    if (slot < 0) return;
    if (slot >= p.num_slots) {
        if (c == 0 && p.err) atomicOr(p.err, PA_DEVERR_SLOT);
        return;
    }
    const int o = slot & (bs - 1);
    const int64_t at = q4_base<D>(slot >> p.log2bs, p.Hkv, head, bs);
    uint32_t kw[G], kp[G], vw[G], vp[G];
    q4_load_row<D>(p.k_pool, at, bs, o, c, kw, kp);
    q4_load_row<D>(p.v_pool, at, bs, o, c, vw, vp);
    const int64_t to = int64_t(row) * D + 8 * c;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        *reinterpret_cast<uint4*>(p.k_out + to + 32 * g) = q4_columns<D, false>(kw, kp, g);
        *reinterpret_cast<uint4*>(p.v_out + to + 32 * g) = q4_columns<D, true>(vw, vp, g);
    }
}

// ------------------------------------------------------------------------------ expansion

struct ExpandParams {
    const uint8_t *k_pool, *v_pool;
    const int32_t *table, *cu, *ctx;
    const int32_t* list;                // [n][2]: sequence, 128-token block of it
    const int32_t* ex_table;            // [B][cols]: place of every block in the expanded pools, -1
    int32_t* ex_ctx;                    // [B]: the context of the sequences that are expanded, else 0
    int32_t* queue;                     // of the rows read from the codes (see DirectParams): back to 0
    __nv_bfloat16 *k_out, *v_out;       // [n][128][Hkv][D]; V in f16 where v16 says so
    uint8_t* v16;                       // [n][Hkv]
    int32_t* err;
    int32_t B, cols, max_blocks, num_blocks, Hkv, g, log2bs, direct_rows;
};

// CTA (i, h): block i of the plan's list, head h: 128 tokens of K to bf16, the values of paged_kv_read_q4, and of V to
// f16, 3 bits more, where the block's largest |V| lies in 2^-12 .. 65,504 or is 0 (groups that are NaN aside), so that
// what is too small for f16's bits is off by 2^-12 of the largest or less; else V is bf16, too.
// Bound by memory (512 bytes a token and head written, 160 read): 21,900 tokens of 8 heads take 18 us ahead of the
// attention that reads them, 3 of them for V's type: its values wait for all of the block's parameters, while K's are
// written. (Every warp looking at all of the parameters, without a barrier: 2 us more.)
// The sequences whose context is expanded whole are told to the attention by ex_ctx; the others (rows that
// are read directly, metadata that the plan was not made for, a context that the block table does not cover) have a
// context of 0 there, by which the attention refuses their items.
template <int D>
__global__ void __launch_bounds__(256) q4_expand_kernel(const ExpandParams p) {
    constexpr int G = D / kQ4Group, kGroups = 256 / 4;          // rows at a time
    dependent_start();
    const int bs = 1 << p.log2bs;
    const int64_t id = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
    if (id == 0) *p.queue = 0;
    for (int64_t s = id; s < p.B; s += int64_t(gridDim.x) * gridDim.y * 256) {
        const int64_t n_q = int64_t(p.cu[s + 1]) - p.cu[s];
        const int c = p.ctx[s];
        const int64_t blocks = (int64_t(c) + 127) / 128;
        const bool whole = n_q * p.g > p.direct_rows && c > 0 && blocks <= p.cols &&
                           (int64_t(c) + bs - 1) / bs <= p.max_blocks && p.ex_table[s * p.cols + blocks - 1] >= 0;
        p.ex_ctx[s] = whole ? c : 0;
    }
    const int seq = p.list[2 * blockIdx.x], first = p.list[2 * blockIdx.x + 1];
    const int head = blockIdx.y;
    uint8_t* const v16 = p.v16 + int64_t(blockIdx.x) * p.Hkv + head;
    if (seq < 0) {                                              // padding of the plan
        if (threadIdx.x == 0) *v16 = 1;
        return;
    }
    const int ctx = seq < p.B ? p.ctx[seq] : 0;
    if (seq >= p.B || first < 0 || int64_t(first) * 128 >= ctx ||
        (int64_t(ctx) + bs - 1) / bs > p.max_blocks) {
        if (threadIdx.x == 0) *v16 = 1;
        if (threadIdx.x == 0 && p.err) atomicOr(p.err, PA_DEVERR_META);
        return;
    }
    const int c = threadIdx.x & 3;
    const int32_t* table = p.table + int64_t(seq) * p.max_blocks;
    constexpr int kTimes = 128 / kGroups;
    uint32_t kw[kTimes][G] = {}, kp[kTimes][G] = {}, vw[kTimes][G] = {}, vp[kTimes][G] = {};
    const int tok = threadIdx.x / 4, key = first * 128 + tok;       // the first row's; key < ctx + 128
#pragma unroll
    for (int i = 0; i < kTimes; ++i) {
        if (key + i * kGroups >= ctx) break;
        const int32_t block = table[(key + i * kGroups) >> p.log2bs];
        if (block >= 0 && block < p.num_blocks) {
            const int64_t at = q4_base<D>(block, p.Hkv, head, bs);
            q4_load_row<D>(p.v_pool, at, bs, (key + i * kGroups) & (bs - 1), c, vw[i], vp[i]);
            q4_load_row<D>(p.k_pool, at, bs, (key + i * kGroups) & (bs - 1), c, kw[i], kp[i]);
        } else if (p.err) {
            atomicOr(p.err, PA_DEVERR_BLOCK);                   // its keys read as 0
        }
    }
    float big = 0.f;                                            // (fmaxf passes NaN over)
#pragma unroll
    for (int i = 0; i < kTimes; ++i)
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float low = __uint_as_float(vp[i][g] & 0xFFFF0000u);
            big = fmaxf(big, fmaxf(fabsf(low), fabsf(fmaf(15.f, __uint_as_float(vp[i][g] << 16), low))));
        }
    // (no negative numbers: they order as whole ones do)
    __shared__ uint32_t warp_big[256 / 32];
    const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(big));
    if ((threadIdx.x & 31) == 0) warp_big[threadIdx.x >> 5] = most;
    const auto out = [&](int i, int g) { return ((int64_t(blockIdx.x) * 128 + tok + i * kGroups) * p.Hkv + head) * D + 8 * c + 32 * g; };
#pragma unroll
    for (int i = 0; i < kTimes; ++i) {
        if (key + i * kGroups >= ctx) break;
#pragma unroll
        for (int g = 0; g < G; ++g)
            *reinterpret_cast<uint4*>(p.k_out + out(i, g)) = q4_columns<D, false>(kw[i], kp[i], g);
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 256 / 32; ++w) big = fmaxf(big, __uint_as_float(warp_big[w]));
    const bool half = big <= 65504.f && (big >= 0x1p-12f || big == 0.f);
    if (threadIdx.x == 0) *v16 = half;
#pragma unroll
    for (int i = 0; i < kTimes; ++i) {
        if (key + i * kGroups >= ctx) break;
#pragma unroll
        for (int g = 0; g < G; ++g)
            *reinterpret_cast<uint4*>(p.v_out + out(i, g)) =
                half ? q4_columns_f16<D>(vw[i], vp[i], g) : q4_columns<D, true>(vw[i], vp[i], g);
    }
}

// ------------------------------------------------------------------- rows read from the codes
//
// An item is one KV head, one tile of query rows (tokens x heads of its group, at most 8 NT of them)
// and one split of the sequence's keys: the work of two warps, which take every second one of the split's tiles of 32
// keys, keep their online softmax, and join at its end. A CTA's pairs draw items from its list (one CTA and list a
// multiprocessor, dealt by cost on the host), so that a warp waits for nothing but its own loads, and the first one of
// a pair for the second's part. A row's splits are joined in a fixed order by q4_fold_kernel. A split's length
// depends on the sequence's context alone (q4_split_keys), so a row's bits do not depend on the batch.
// A pair and not a warp: an item costs a warp about as much beside its tiles as a tile and a half does (q, state,
// results), so its tiles should be many, and splits few; but a sequence by itself wants short chains. One warp a split,
// of half the length: decode batch 74.5 us, long tail 59, one sequence 21.3, four drafted tokens 14.1, where pairs take
// 72.8 / 57 / 20.5 / 13.7; four warps a split of 1,024 keys or more 77.5 / 61 / 14.2 / 13.7.
//
// Why mma.sync and not tcgen05: the contraction's free dimension is at most 8 NT columns, so the tensor
// rate is no concern; what is, is the way of the codes to the tensor core. tcgen05 would take them expanded to
// 16 bits from shared memory or TMEM: four times the cache's bytes written and read once more (the e4m3 path of
// attention.cu, which does this, takes 2.5 T elements/s). mma.sync takes them from
// the registers that unpacked them. So (keys x columns) is the A operand, and with the row order of q4.h
// a lane's 16-byte piece of a row is its fragments:
//   S^T = K Q^T     A = K codes as f16 subnormals, u 2^-24 and 16 u 2^-24 (no conversion: a mask), B = Q^T and
//                   Q^T / 16 in f16, each row of q times a power of two
//   S = sum_g s_g (q . codes)_g + sum_g m_g sum(q_g)
// with exact products and fp32 sums: K is never rounded beyond its code. The second sum is a product too, of the
// minima and sum(q_g) in three bf16 parts.
//   O^T = V^T P^T   A = V codes as u - 8 (bf16: the code in the mantissa, less 136), B = w = bf16(p s_g)
//   O = sum_j w_j (u_j - 8) + sum_j p_j bf16(m_jg + 8 s_jg)
// u - 8 and not u: |u - 8| s is the size of the value's distance from its group's middle, u s twice that, and so
// would the roundings of w be. p is a sum of two bf16 (16 bits: p itself rounded to one would add an error
// as large as that of w; against 64 bits the output's would be 0.0028 so and is 0.0023 to 0.0024, at 1.4 us of the decode
// batch below); w = fma(p_hi, s, p_lo s) rounds once. P^T's layout is turned by movmatrix, once for all groups.
// A masked key's parameters may be anything (it may not have been written yet), and 0 times them too: its w
// are cleared for the rows that do not see it, its centre is clamped to numbers. What is not finite still
// reaches the rows that see it, through w (the write makes such a group's scale NaN, too).
//
// Loads: cp.async into a ring of kStages tiles per warp (codes and parameters; blocks outside the pool are
// filled with zeros, keys of a block behind the last row may hold anything and are masked), no barrier
// but the warp's own.
//
// Measured, with the join, calls one behind the other: 64 sequences of median 2,048 (up to 16,384) keys, 32 / 8 heads
// of 128 (314 MB of cache): 73 us, 4.3 TB/s; 32 of 1,000 to 40,000 keys, 64 / 8 heads: 57; 12 of 4 rows, 16 / 4
// heads of 64: 13.7; one of 16,001 keys: 20.7. 32 single rows beside a chunk of 257: 85, 14 more when they waited for
// the chunk's 72 CTAs (or these for them). What bounds it: replayed in graphs, where the four take 76, 60, 17 and 24 us,
// the same kernel without its arithmetic, copies, items and join alone, takes 61, 49, 10 and 12. So of the first's 30 us above
// its bytes (46) half is the way of the bytes and half the arithmetic beyond it, a tile's chain of products and softmax
// with three warps a scheduler; a sequence by itself is its 16 tiles of one warp, one behind the other.
// Tried without gain: 16 warps of 128 registers, a third stage, the next tile's scores between the
// values' products, K as e4m3 (its mma.sync is emulated), splits joined inside this kernel (20 to 40 us more), the
// next item's first tiles or its L2 lines asked for ahead (3 to 6 us more).
struct DirectParams {
    const __nv_bfloat16* q;
    const uint8_t *k_pool, *v_pool;
    const int32_t *table, *cu, *ctx;
    const pa_work_item* items;
    const int32_t* lists;               // [PA_PLAN_CTAS + 1]: the first item of every CTA's
    int32_t* queue;                     // behind an attention over chunks: the next item, for all CTAs; else null
    float* part;                        // [n_items][8 NT][D + 2]: splits' (acc, m, l)
    __nv_bfloat16* out;
    int32_t* err;
    int32_t n_items, B, T, max_blocks, num_blocks, Hq, Hkv, log2g, log2bs, max_ctx;
    float c;                            // log2(e) / sqrt(D)
    uint32_t bits;                      // 0x43004300
};

// warps of a CTA (one a multiprocessor): what the registers hold
template <int NT>
constexpr int kWarps = NT == 1 ? 12 : 8;
constexpr uint32_t kEights = 0x41004100u;   // two bf16
constexpr int kKeys = 32;               // keys of a warp's tile
constexpr int kHeld = 128;              // items of a list that a CTA keeps in shared memory
constexpr float kNone = 3e38f;          // minus a maximum that every score passes

template <int D>
struct Ring {
    static constexpr int kStages = 2;
    static constexpr int kCodes = kKeys * kQ4Codes<D>;
    static constexpr int kParams = kKeys * kQ4Params<D>;
    static constexpr int kStage = 2 * (kCodes + kParams);       // K codes, V codes, K, V parameters
    static constexpr int kWarp = kStages * kStage;
};

// what a pair's second warp hands to the first: a float4 of each lane for every product tile, (l, maxima) and z
template <int D, int NT>
constexpr int kHanded = NT * (2 * (D / kQ4Group) + 2) * 512;

// n is the number of splits of `len` keys that `keys` take
__device__ __forceinline__ bool split_in(int64_t keys, int64_t len, int n) {
    return n * len >= keys && (n - 1) * len < keys;
}

// barriers of two warps
__device__ __forceinline__ void pair_sync(int id) {
    asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory");
}
__device__ __forceinline__ void pair_arrive(int id) {
    __syncwarp();
    asm volatile("bar.arrive %0, 64;" ::"r"(id) : "memory");
}

template <int D>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[D / kQ4Group]) {
    if constexpr (D == 128) {
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
    } else {
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
    }
}

// A lane's part of a V row: its 16-bit words of all groups, two to a register.
template <int D>
__device__ __forceinline__ void lds_halves(uint32_t addr, uint32_t (&w)[D / kQ4Group / 2]) {
    if constexpr (D == 128) {
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
    } else {
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
    }
}

__device__ __forceinline__ uint32_t lds_word(uint32_t addr) {
    uint32_t w;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(addr));
    return w;
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

// D = A B and D += A B, A 16 x 16 and B 16 x 8 bf16 (or f16), fp32 accumulator.
#define PA_Q4_MMA(NAME, SHAPE, TYPE)                                                                          \
    __device__ __forceinline__ void NAME(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,         \
                                         uint32_t a3, uint32_t b0, uint32_t b1) {                      \
        asm("mma.sync.aligned." SHAPE ".row.col.f32." TYPE "." TYPE ".f32 {%0, %1, %2, %3}, "           \
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"                                            \
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])                                           \
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));                                   \
    }                                                                                                  \
    __device__ __forceinline__ void NAME##0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,      \
                                            uint32_t a3, uint32_t b0, uint32_t b1) {                   \
        asm("mma.sync.aligned." SHAPE ".row.col.f32." TYPE "." TYPE ".f32 {%0, %1, %2, %3}, "           \
            "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"                                        \
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])                                           \
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));                         \
    }
PA_Q4_MMA(mma, "m16n8k16", "bf16")
PA_Q4_MMA(mma_f16_, "m16n8k16", "f16")
#undef PA_Q4_MMA

__device__ __forceinline__ uint32_t mul_bf16(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t fma_bf16(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
// NaN and infinities become the largest numbers, numbers stay.
__device__ __forceinline__ uint32_t finite_bf16(uint32_t a) {
    asm("max.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(0xFF7FFF7Fu));
    asm("min.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(0x7F7F7F7Fu));
    return a;
}

__device__ __forceinline__ uint32_t transpose8(uint32_t w) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(w));
    return r;
}

// Nibble K of both 16-bit halves as bf16 u - 8. bits: 128 twice, in a register that the compiler does not know
// the value of (with two constants it makes two instructions of mask and exponent).
template <int K>
__device__ __forceinline__ uint32_t centred(uint32_t w, uint32_t bits) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(((w >> (4 * K)) & 0x000F000Fu) | bits), "r"(0x43084308u));
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
    uint32_t qm[NT][2];                 // ... of the minima's product
    float o[NT][2 * G][4];
    float z[NT][4];                     // sums of p (m + 8 s): lane row r holds group r % G
    uint64_t l[NT];                     // sum of p, this lane's keys
    float c[NT][2];                     // scores to base 2: log2(e) / sqrt(D) and q's power of two
    float nm[NT][2];                    // minus the reference maximum, in base 2; kNone: no key yet
    int pos0, rows, log2g;              // position of the first row, rows, heads of a token

    // Position of a row; those behind the last one see what the last one sees.
    __device__ __forceinline__ int pos(int row) const { return pos0 + (min(row, rows - 1) >> log2g); }
    uint32_t bits;                      // of 128, twice (see centred)
};

// The rows of column tile j from q (w: columns 32 g + 8 c .. + 7 of row 8 j + r), and their state at the start.
template <int D, int NT>
__device__ __forceinline__ void q4_take_q(Rows<D, NT>& R, const uint4 (&w)[D / kQ4Group], int j, float c_plain,
                                          int lane) {
    constexpr int G = D / kQ4Group;
    const int cc = lane & 3;
    float v[G][8], big = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        v[g][0] = scale_of(w[g].x), v[g][1] = min_of(w[g].x), v[g][2] = scale_of(w[g].y), v[g][3] = min_of(w[g].y);
        v[g][4] = scale_of(w[g].z), v[g][5] = min_of(w[g].z), v[g][6] = scale_of(w[g].w), v[g][7] = min_of(w[g].w);
#pragma unroll
        for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(v[g][i]));
    }
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
    // q 2^e, its largest element below 2^15: a bf16's 8 bits are kept down to 2^-29 of it (in the halves
    // divided by 16, 2^-25). Exponent 255, an infinity, is taken like the largest number's: infinities and NaN
    // stay what they are.
    const int e = 14 + 127 - int(max(__float_as_uint(big) >> 23, 24u));     // 2^e and 2^-e are fp32 numbers
    const float up = __uint_as_float(uint32_t(127 + e) << 23);
    const float c = c_plain * __uint_as_float(uint32_t(127 - e) << 23) * 0x1p24f;
    R.c[j][0] = __shfl_sync(0xffffffffu, c, 8 * cc);
    R.c[j][1] = __shfl_sync(0xffffffffu, c, 8 * cc + 4);
    float sum[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[g][i] *= up;
        // nibbles 0, 4 | 1, 5 | 2, 6 | 3, 7 are the steps' operands
        R.qb[j][g][0] = pack_f16(v[g][0], v[g][4]);
        R.qb[j][g][1] = pack_f16(v[g][1] * 0.0625f, v[g][5] * 0.0625f);
        R.qb[j][g][2] = pack_f16(v[g][2], v[g][6]);
        R.qb[j][g][3] = pack_f16(v[g][3] * 0.0625f, v[g][7] * 0.0625f);
        float t = ((v[g][0] + v[g][1]) + (v[g][2] + v[g][3])) + ((v[g][4] + v[g][5]) + (v[g][6] + v[g][7]));
        t += __shfl_xor_sync(0xffffffffu, t, 1);
        t += __shfl_xor_sync(0xffffffffu, t, 2);
        sum[g] = t * 0x1p-24f;
    }
    // The minima's product. Every lane of a row holds all its minima, groups 0 and 1 in the first half of the
    // step and 2 and 3 in the second; against them stand part c of sum(q_g) (lanes c < 3) or nothing.
    uint32_t part[2] = {0, 0};
#pragma unroll
    for (int g = 0; g < G; ++g) {
        float t = sum[g];
        const __nv_bfloat16 p0 = __float2bfloat16_rn(t);
        t -= __bfloat162float(p0);
        const __nv_bfloat16 p1 = __float2bfloat16_rn(t);
        t -= __bfloat162float(p1);
        const __nv_bfloat16 p2 = __float2bfloat16_rn(t);
        const uint32_t b = __bfloat16_as_ushort(cc == 0 ? p0 : cc == 1 ? p1 : p2);
        part[g / 2] |= b << (16 * (g & 1));
    }
    R.qm[j][0] = cc < 3 ? part[0] : 0;
    R.qm[j][1] = cc < 3 ? part[1] : 0;              // (two groups: nothing)
#pragma unroll
    for (int t = 0; t < 2 * G; ++t) R.o[j][t][0] = R.o[j][t][1] = R.o[j][t][2] = R.o[j][t][3] = 0.f;
    R.z[j][0] = R.z[j][1] = R.z[j][2] = R.z[j][3] = 0.f;
    R.l[j] = 0;
    R.nm[j][0] = R.nm[j][1] = kNone;
}

// Scores of 16 keys of a tile (h: which half) from its stage, in units of 1 / R.c.
template <int D, int NT>
__device__ __forceinline__ void q4_scores(uint32_t stage, const Rows<D, NT>& R, int h, int lane,
                                          float (&x)[NT][2][4]) {
    constexpr int G = D / kQ4Group;
    using L = Ring<D>;
    const int r = lane >> 2, cc = lane & 3;
    uint32_t ka[G], kb[G], pa[G], pb[G];
    const uint32_t row = stage + (16 * h + r) * kQ4Codes<D> + cc * (4 * G);
    lds_words<D>(row, ka);
    lds_words<D>(row + 8 * kQ4Codes<D>, kb);
    const uint32_t par = stage + 2 * L::kCodes + (16 * h + r) * kQ4Params<D>;
    lds_words<D>(par, pa);
    lds_words<D>(par + 8 * kQ4Params<D>, pb);
    const uint32_t m0 = __byte_perm(pa[0], pa[1], 0x7632), m1 = __byte_perm(pb[0], pb[1], 0x7632);
    const uint32_t m2 = __byte_perm(pa[G - 2], pa[G - 1], 0x7632), m3 = __byte_perm(pb[G - 2], pb[G - 1], 0x7632);
#pragma unroll
    for (int j = 0; j < NT; ++j) mma0(x[j][h], m0, m1, m2, m3, R.qm[j][0], R.qm[j][1]);
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const float s0 = scale_of(pa[g]), s1 = scale_of(pb[g]);
        const uint32_t ha = ka[g] >> 8, hb = kb[g] >> 8;
        constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            float t[4];
            mma_f16_0(t, ka[g] & kLow, kb[g] & kLow, ka[g] & kHigh, kb[g] & kHigh, R.qb[j][g][0], R.qb[j][g][1]);
            mma_f16_(t, ha & kLow, hb & kLow, ha & kHigh, hb & kHigh, R.qb[j][g][2], R.qb[j][g][3]);
            x[j][h][0] = fmaf(t[0], s0, x[j][h][0]);
            x[j][h][1] = fmaf(t[1], s0, x[j][h][1]);
            x[j][h][2] = fmaf(t[2], s1, x[j][h][2]);
            x[j][h][3] = fmaf(t[3], s1, x[j][h][3]);
        }
    }
}

// Online softmax of a tile of 32 keys from key0 on: p as bf16 pairs of keys 2 c, 2 c + 1 (and 8 behind them) of
// row r, and what that rounding leaves. masked: some key lies behind some row. The reference maximum moves when
// the rows' maximum outgrows it by 2^8.
template <int D, int NT>
__device__ __forceinline__ void q4_softmax(Rows<D, NT>& R, float (&x)[NT][2][4], bool masked, int key0,
                                           int lane, uint32_t (&p)[NT][2][2], uint32_t (&rest)[NT][2][2]) {
    constexpr int G = D / kQ4Group;
    const int r = lane >> 2;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        float mx[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (masked) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        if (key0 + 16 * h + 8 * b + r > R.pos(8 * j + 2 * (lane & 3) + e)) x[j][h][2 * b + e] = -INFINITY;
            }
            mx[e] = fmaxf(fmaxf(x[j][0][e], x[j][0][2 + e]), fmaxf(x[j][1][e], x[j][1][2 + e]));
        }
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) {
            mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], d));
            mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], d));
        }
        // in base 2 above the reference
        const float up0 = fmaf(mx[0], R.c[j][0], R.nm[j][0]), up1 = fmaf(mx[1], R.c[j][1], R.nm[j][1]);
        if (__any_sync(0xffffffffu, up0 > 8.f || up1 > 8.f)) {
            // the result's factors, 1 for a row that stays
            float a[2] = {1.f, 1.f};
            if (up0 > 8.f) {
                const float now = -mx[0] * R.c[j][0];
                a[0] = ex2(now - R.nm[j][0]);
                R.nm[j][0] = now;
            }
            if (up1 > 8.f) {
                const float now = -mx[1] * R.c[j][1];
                a[1] = ex2(now - R.nm[j][1]);
                R.nm[j][1] = now;
            }
            const uint64_t a2 = f2(a[0], a[1]);
            R.l[j] = mul2(R.l[j], a2);
            R.z[j][0] *= a[0];
            R.z[j][1] *= a[1];
#pragma unroll
            for (int t = 0; t < 2 * G; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) R.o[j][t][e] *= a[e & 1];
        }
        const uint64_t n2 = f2(R.nm[j][0], R.nm[j][1]), c2 = f2(R.c[j][0], R.c[j][1]);
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
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const uint32_t hi = pack_bf16(x[j][h][2 * b], x[j][h][2 * b + 1]);
                float u, v;
                const uint64_t both = f2(x[j][h][2 * b], x[j][h][2 * b + 1]);
                f2_split(fma2(f2(scale_of(hi), min_of(hi)), f2(-1.f, -1.f), both), u, v);
                p[j][h][b] = transpose8(hi);
                rest[j][h][b] = transpose8(pack_bf16(u, v));
            }
        }
    }
}

// O of 16 keys of a tile (h: which half) from its stage and p. MASK: some key lies behind some row.
template <int D, int NT, bool MASK>
__device__ __forceinline__ void q4_values(uint32_t stage, Rows<D, NT>& R, const uint32_t (&p)[NT][2][2],
                                          const uint32_t (&rest)[NT][2][2], int h, int key0, int lane) {
    constexpr int G = D / kQ4Group;
    using L = Ring<D>;
    const int r = lane >> 2, cc = lane & 3;
    // Keys 2 c, 2 c + 1 and those 8 behind them. Of eight keys the even ones lie before the odd ones, and (D = 128) of
    // four such rows the first halves before the second, so that what half a warp reads is contiguous.
    const uint32_t row = stage + L::kCodes + 16 * h * kQ4Codes<D> + cc * 32 +
                         (D == 128 ? (r >> 2) * 128 + (r & 3) * 8 : r * 4);
    const uint32_t par = stage + 2 * L::kCodes + L::kParams + (16 * h + 2 * cc) * kQ4Params<D>;
    uint32_t v[4][G / 2], zp[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        lds_halves<D>(row + 4 * k * kQ4Codes<D>, v[k]);
        zp[k] = lds_word(par + ((k >> 1) * 8 + (k & 1)) * kQ4Params<D> + 4 * (r % G));
    }
    uint32_t keep0[NT], keep1[NT];
    uint32_t z0 = fma_bf16(__byte_perm(zp[0], zp[1], 0x5410), kEights, __byte_perm(zp[0], zp[1], 0x7632));
    uint32_t z1 = fma_bf16(__byte_perm(zp[2], zp[3], 0x5410), kEights, __byte_perm(zp[2], zp[3], 0x7632));
    if constexpr (MASK) {
        z0 = finite_bf16(z0);
        z1 = finite_bf16(z1);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        mma(R.z[j], z0, 0u, z1, 0u, p[j][h][0], p[j][h][1]);
        mma(R.z[j], z0, 0u, z1, 0u, rest[j][h][0], rest[j][h][1]);
        if constexpr (MASK) {
            const int seen = R.pos(8 * j + r) - (key0 + 16 * h + 2 * cc);     // >= 0: key 2 c, and so on
            keep0[j] = (seen >= 0 ? 0xFFFFu : 0u) | (seen >= 1 ? 0xFFFF0000u : 0u);
            keep1[j] = (seen >= 8 ? 0xFFFFu : 0u) | (seen >= 9 ? 0xFFFF0000u : 0u);
        }
    }
    uint32_t pv[4][G];
#pragma unroll
    for (int k = 0; k < 4; ++k) lds_words<D>(par + ((k >> 1) * 8 + (k & 1)) * kQ4Params<D>, pv[k]);
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const uint32_t sel = g & 1 ? 0x7632 : 0x5410;
        const uint32_t lo = __byte_perm(v[0][g / 2], v[1][g / 2], sel), hi = __byte_perm(v[2][g / 2], v[3][g / 2], sel);
        const uint32_t s0 = __byte_perm(pv[0][g], pv[1][g], 0x5410), s1 = __byte_perm(pv[2][g], pv[3][g], 0x5410);
        const uint32_t a0 = centred<0>(lo, R.bits), a1 = centred<1>(lo, R.bits);
        const uint32_t a2 = centred<2>(lo, R.bits), a3 = centred<3>(lo, R.bits);
        const uint32_t b0 = centred<0>(hi, R.bits), b1 = centred<1>(hi, R.bits);
        const uint32_t b2 = centred<2>(hi, R.bits), b3 = centred<3>(hi, R.bits);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            uint32_t w0 = fma_bf16(p[j][h][0], s0, mul_bf16(rest[j][h][0], s0));
            uint32_t w1 = fma_bf16(p[j][h][1], s1, mul_bf16(rest[j][h][1], s1));
            if constexpr (MASK) {
                w0 &= keep0[j];
                w1 &= keep1[j];
            }
            mma(R.o[j][2 * g], a0, a1, b0, b1, w0, w1);
            mma(R.o[j][2 * g + 1], a2, a3, b2, b3, w0, w1);
        }
    }
}

template <int D, int NT>
__global__ void __launch_bounds__(32 * kWarps<NT>, 1) q4_direct_kernel(const DirectParams p) {
    constexpr int G = D / kQ4Group;
    constexpr int kCols = 8 * NT;
    using L = Ring<D>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ pa_work_item held[kHeld];
    __shared__ int next_item, drawn[kWarps<NT> / 2][2];
    // Behind the attention over the step's chunks this kernel starts while that one ends: it reads nothing of it (what
    // came before that one has completed, or it would not have let this one start), and waits for it at its end, for
    // the sake of the next one. (In this order: q4_fold_kernel reads the metadata before it waits for this kernel.)
    if (!p.queue) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, cc = lane & 3;
    const int pair = warp >> 1, half = warp & 1;
    const uint32_t ring = smem_u32(smem) + warp * L::kWarp;
    float4* const handed = reinterpret_cast<float4*>(smem + kWarps<NT> * L::kWarp + pair * kHanded<D, NT>) + lane;
    const int bs = 1 << p.log2bs, gq = 1 << p.log2g;
    // by itself: the CTA's list; else the whole plan, since CTAs start when the chunks leave them a multiprocessor
    int first = p.queue ? 0 : p.lists[blockIdx.x], last = p.lists[p.queue ? PA_PLAN_CTAS : blockIdx.x + 1];
    if (first < 0 || last < first || last > p.n_items) {
        if (threadIdx.x == 0 && p.err) atomicOr(p.err, PA_DEVERR_META);
        first = last = 0;               // (n_items is far from where the counter would wrap)
    }
    const int n_held = p.queue ? 0 : min(last - first, kHeld);
    if (threadIdx.x == 0) next_item = first;
    // the list's first items, so that a warp that draws one has it at once
    constexpr int kWords = sizeof(pa_work_item) / 4;
    for (int i = threadIdx.x; i < n_held * kWords; i += 32 * kWarps<NT>)
        reinterpret_cast<int32_t*>(held)[i] = reinterpret_cast<const int32_t*>(p.items + first)[i];
    __syncthreads();

    // The pair's second warp draws its items, one ahead of the first warp: what it arrives with at the barrier `ready` is
    // its part of an item and the next item's index. It may hand over another part once the first warp has arrived at
    // `taken`. Both pass them once for every index drawn, whatever they find there.
    const auto draw = [&](int turn) {
        int idx = 0;
        if (lane == 0) {
            if (p.queue)
                idx = atomicAdd(p.queue, 1);
            else
                idx = atomicAdd(&next_item, 1);
            drawn[pair][turn & 1] = idx;
        }
        return __shfl_sync(0xffffffffu, idx, 0);
    };
    const int ready = 1 + 2 * pair, taken = 2 + 2 * pair;
    int idx;
    if (half) {
        idx = draw(0);
        __syncwarp();
        pair_sync(ready);
    } else {
        pair_sync(ready);
        idx = drawn[pair][0];
    }
    // an item that is not worked on
    const auto pass = [&](int turn) {
        if (half) {
            if (turn > 0) pair_sync(taken);
            idx = draw(turn + 1);
            pair_arrive(ready);
        } else {
            pair_sync(ready);
            idx = drawn[pair][(turn + 1) & 1];
            pair_arrive(taken);
        }
    };
    for (int turn = 0;; ++turn) {
        if (idx < 0 || idx >= last) {
            if (half && turn > 0) pair_sync(taken);
            break;
        }
        const pa_work_item* const at_item = !p.queue && idx - first < kHeld ? held + (idx - first) : p.items + idx;
        const pa_work_item it = *at_item;
        // ---- The item by itself, then against the metadata it points at: what the loads of q, of the first blocks and
        // of the metadata need is in the item (next: the context it was planned for), so that they
        // are all on the way at once.
        const int ctx = it.next;
        bool good = it.kind == PA_ITEM_DIRECT && it.seq >= 0 && it.seq < p.B && it.kv_head >= 0 &&
                    it.kv_head < p.Hkv && it.n_q > 0 && it.n_q <= (kCols >> p.log2g) && it.q_start >= 0 &&
                    it.q_start <= p.T - it.n_q && it.split >= 0 && it.n_splits > it.split &&
                    it.tile0 >= 0 && it.tile0 <= p.n_items - it.n_splits && ctx > 0 && ctx <= p.max_ctx &&
                    (int64_t(ctx) + bs - 1) / bs <= p.max_blocks && it.split * q4_split_keys(ctx) < ctx;
        if (!good) {
            if (lane == 0 && p.err) atomicOr(p.err, PA_DEVERR_META);
            pass(turn);
            continue;
        }
        const int ctx_now = __ldg(p.ctx + it.seq), cu0 = __ldg(p.cu + it.seq), cu1 = __ldg(p.cu + it.seq + 1);
        const int len = int(q4_split_keys(ctx)), k_begin = it.split * len, k_last = min(ctx, k_begin + len);
        const int32_t* table = p.table + int64_t(it.seq) * p.max_blocks;
        // (the split's keys up to the context: the last row may lie before it)
        const auto block_of = [&](int tile) {
            const int key = k_begin + (2 * (tile + (lane >> 2)) + half) * kKeys + 8 * (lane & 3);
            return key < k_last ? max(__ldg(table + (key >> p.log2bs)), -1) : -2;
        };
        int block = block_of(0);
        const int rows = it.n_q << p.log2g;
        uint4 qw[NT][G];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int row = 8 * j + r;
            const __nv_bfloat16* src = p.q + (int64_t(it.q_start + (row >> p.log2g)) * p.Hq + it.kv_head * gq +
                                              (row & (gq - 1))) * D + 8 * cc;
#pragma unroll
            for (int g = 0; g < G; ++g)
                qw[j][g] = row < rows ? __ldg(reinterpret_cast<const uint4*>(src + 32 * g)) : make_uint4(0, 0, 0, 0);
        }
        const int pos0 = ctx - (cu1 - it.q_start);              // position of the first row
        const int keys = pos0 + it.n_q;                         // up to the last row
        good = ctx_now == ctx && cu0 <= it.q_start && it.q_start + it.n_q <= cu1 &&
               int64_t(cu1) - cu0 <= ctx && split_in(keys, len, it.n_splits);
        if (!good) {
            if (lane == 0 && p.err) atomicOr(p.err, PA_DEVERR_META);
            pass(turn);
            continue;
        }
        const int k_end = min(keys, k_begin + len);
        // tiles of 32 keys: the pair's warps take every second one
        const int n = ((k_end - k_begin + kKeys - 1) / kKeys + 1 - half) / 2;
        // Lane i looks after the eight keys i % 4 of tile i / 4 of eight tiles: where their code rows and their
        // parameter rows begin, in units of 16 bytes, and (a bit of `there`) whether their block is there.
        constexpr int kRow16 = kQ4Codes<D> / 16, kPar8 = 8 * kQ4Params<D> / 16;
        uint32_t codes_at = 0, params_at = 0, there = 0;
        const auto turn_to = [&](int tile) {                // the eight tiles from `tile` on
            const int key = k_begin + (2 * (tile + (lane >> 2)) + half) * kKeys + 8 * (lane & 3);
            const bool on = block >= 0 && block < p.num_blocks;
            if (!on && block != -2 && p.err) atomicOr(p.err, PA_DEVERR_BLOCK);   // its keys read as 0
            there = __ballot_sync(0xffffffffu, on);
            const int o = key & (bs - 1);
            const uint32_t at = (uint32_t(on ? block : 0) * p.Hkv + it.kv_head) * (bs * kQ4Row<D> / 16);
            codes_at = at + o * kRow16;
            params_at = at + bs * kRow16 + (o >> 3) * kPar8;
            block = block_of(tile + 8);
        };
        constexpr int kPieces = kRow16;                     // 16-byte pieces of a code row
        constexpr int kAtOnce = 32 / kPieces;               // keys the warp's lanes cover
        // the lane's piece of a unit's eight code rows, in 16 bytes: K as it lies, V as q4_values reads it
        const uint32_t k_lane = lane % (8 * kPieces);
        const uint32_t v_lane = D == 128 ? ((lane & 6) + (lane >> 4)) * kPieces + ((lane >> 2) & 2) + (lane & 1)
                                         : (lane & 6) * kPieces + ((lane >> 3) & 1) * kPieces + (lane & 1);
        uint32_t stage_in = ring;
        const auto issue = [&](int tile) {
            if (tile < n) {
                if ((tile & 7) == 0) turn_to(tile);
                const int u0 = (tile & 7) * 4;
                const bool all = ((there >> u0) & 15u) == 15u;
#pragma unroll
                for (int i = 0; i < kKeys / kAtOnce; ++i) {
                    const int unit = u0 + (i * kAtOnce + lane / kPieces) / 8;
                    const uint32_t at = __shfl_sync(0xffffffffu, codes_at, unit);
                    const bool on = all || ((there >> unit) & 1u);
                    const uint32_t to = stage_in + i * (kAtOnce * kQ4Codes<D>) + 16 * lane;
                    cp_async<16>(to, p.k_pool + uint64_t(at + k_lane) * 16, on);
                    cp_async<16>(to + L::kCodes, p.v_pool + uint64_t(at + v_lane) * 16, on);
                }
                const uint32_t at = __shfl_sync(0xffffffffu, params_at, u0 + lane / 8);
                const bool on = all || ((there >> (u0 + lane / 8)) & 1u);
                const uint32_t to = stage_in + 2 * L::kCodes + lane * kQ4Params<D>;
                const int64_t par = int64_t(uint64_t(at) * 16) + (lane & 7) * kQ4Params<D>;
                cp_async<kQ4Params<D>>(to, p.k_pool + par, on);
                cp_async<kQ4Params<D>>(to + L::kParams, p.v_pool + par, on);
                stage_in = stage_in == ring + (L::kStages - 1) * L::kStage ? ring : stage_in + L::kStage;
            }
            cp_commit();
        };
#pragma unroll
        for (int i = 0; i < L::kStages; ++i) issue(i);
        // ---- Q, while the first tiles are on their way
        Rows<D, NT> R;
        R.bits = __shfl_sync(0xffffffffu, p.bits, 0);
        R.pos0 = pos0;
        R.rows = rows;
        R.log2g = p.log2g;
#pragma unroll
        for (int j = 0; j < NT; ++j) q4_take_q<D, NT>(R, qw[j], j, p.c, lane);
        uint32_t stage = ring;
        for (int i = 0, key0 = k_begin + half * kKeys; i < n; ++i, key0 += 2 * kKeys) {
            cp_wait<L::kStages - 1>();
            __syncwarp();                                   // every lane's copies
            float x[NT][2][4];
            uint32_t prob[NT][2][2], rest[NT][2][2];
            const bool masked = key0 + kKeys - 1 > pos0;
            q4_scores<D, NT>(stage, R, 0, lane, x);
            q4_scores<D, NT>(stage, R, 1, lane, x);
            q4_softmax<D, NT>(R, x, masked, key0, lane, prob, rest);
            if (masked) {
                q4_values<D, NT, true>(stage, R, prob, rest, 0, key0, lane);
                q4_values<D, NT, true>(stage, R, prob, rest, 1, key0, lane);
            } else {
                q4_values<D, NT, false>(stage, R, prob, rest, 0, key0, lane);
                q4_values<D, NT, false>(stage, R, prob, rest, 1, key0, lane);
            }
            __syncwarp();                                   // every lane has read the stage
            issue(i + L::kStages);
            stage = stage == ring + (L::kStages - 1) * L::kStage ? ring : stage + L::kStage;
        }
        cp_wait<0>();
        // ---- the second warp's part goes to the first
        if (half) {
            if (turn > 0) pair_sync(taken);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float4* const to = handed + j * (2 * G + 2) * 32;
#pragma unroll
                for (int t = 0; t < 2 * G; ++t)
                    to[32 * t] = make_float4(R.o[j][t][0], R.o[j][t][1], R.o[j][t][2], R.o[j][t][3]);
                float l0, l1;
                f2_split(R.l[j], l0, l1);
                to[32 * 2 * G] = make_float4(l0, l1, R.nm[j][0], R.nm[j][1]);
                to[32 * (2 * G + 1)] = make_float4(R.z[j][0], R.z[j][1], R.z[j][2], R.z[j][3]);
            }
            idx = draw(turn + 1);
            pair_arrive(ready);
            continue;
        }
        pair_sync(ready);
        idx = drawn[pair][(turn + 1) & 1];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const float4* const from = handed + j * (2 * G + 2) * 32;
            const float4 s = from[32 * 2 * G], z = from[32 * (2 * G + 1)];
            const float m0 = fminf(R.nm[j][0], s.z), m1 = fminf(R.nm[j][1], s.w);    // minus the maxima
            const float a0 = ex2(m0 - R.nm[j][0]), a1 = ex2(m1 - R.nm[j][1]), b0 = ex2(m0 - s.z), b1 = ex2(m1 - s.w);
            float l0, l1;
            f2_split(R.l[j], l0, l1);
            R.l[j] = f2(l0 * a0 + s.x * b0, l1 * a1 + s.y * b1);
            R.z[j][0] = R.z[j][0] * a0 + z.x * b0;
            R.z[j][1] = R.z[j][1] * a1 + z.y * b1;
            R.nm[j][0] = m0;
            R.nm[j][1] = m1;
#pragma unroll
            for (int t = 0; t < 2 * G; ++t) {
                const float4 o = from[32 * t];
                R.o[j][t][0] = R.o[j][t][0] * a0 + o.x * b0;
                R.o[j][t][1] = R.o[j][t][1] * a1 + o.y * b1;
                R.o[j][t][2] = R.o[j][t][2] * a0 + o.z * b0;
                R.o[j][t][3] = R.o[j][t][3] * a1 + o.w * b1;
            }
        }
        pair_arrive(taken);
        // ---- the rows' results: finished where they have one split, else left for the fold
        const pa_work_item done = *at_item;                     // (again: not kept in registers meanwhile)
        const bool whole = done.n_splits == 1;
        float* const part = p.part + int64_t(done.tile0 + done.split) * (kCols * (D + 2));
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            float l[2];
            f2_split(R.l[j], l[0], l[1]);
#pragma unroll
            for (int d = 4; d <= 16; d <<= 1) {
                l[0] += __shfl_xor_sync(0xffffffffu, l[0], d);
                l[1] += __shfl_xor_sync(0xffffffffu, l[1], d);
            }
            const float f[2] = {whole ? __frcp_rn(l[0]) : 1.f, whole ? __frcp_rn(l[1]) : 1.f};
#pragma unroll
            for (int g = 0; g < G; ++g) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float z = __shfl_sync(0xffffffffu, R.z[j][e], 4 * g + cc);
                    const int row = 8 * j + 2 * cc + e;
                    if (row >= rows) continue;
                    const float y[4] = {(R.o[j][2 * g][e] + z) * f[e], (R.o[j][2 * g][2 + e] + z) * f[e],
                                        (R.o[j][2 * g + 1][e] + z) * f[e], (R.o[j][2 * g + 1][2 + e] + z) * f[e]};
                    const int col = 32 * g + 4 * r;
                    if (whole) {
                        const int64_t at = (int64_t(done.q_start + (row >> p.log2g)) * p.Hq + done.kv_head * gq +
                                            (row & (gq - 1))) * D + col;
                        *reinterpret_cast<uint2*>(p.out + at) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
                    } else {
                        *reinterpret_cast<float4*>(part + row * D + col) = make_float4(y[0], y[1], y[2], y[3]);
                    }
                }
            }
            if (r == 0 && !whole) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    *reinterpret_cast<float2*>(part + kCols * D + 2 * (8 * j + 2 * cc + e)) =
                        make_float2(-R.nm[j][e], l[e]);
            }
        }
        __syncwarp();                                       // the ring is free again
    }
    if (p.queue) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Joins the splits of the rows of a tile and head: a warp per row, CTAs of the plan's fold list (items of split 0 with
// more splits behind them). Eight splits are joined in ascending order, then the eights, likewise: an order that
// the number of splits alone decides. Maxima are in base 2; a part whose row has no key in its split holds -kNone
// and l = 0.
//
// Bound by latency: the way to the parts (list, item, metadata) lies before the wait for the direct kernel, the loads
// of the next eight are on their way while one is joined, and the CTAs are few (a CTA per row, or per tile and eight,
// took twice as long; the last warp of a tile doing this inside the direct kernel 20 to 40 us, row after row).
constexpr int kFoldWarps = 4, kEight = 8;

template <int D, int NT>
__global__ void __launch_bounds__(32 * kFoldWarps) q4_fold_kernel(const DirectParams p, const int32_t* fold) {
    constexpr int kCols = 8 * NT, kPart = kCols * (D + 2), kLane = D / 32;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // Every thread waits for the direct kernel, also one that has nothing to do: were this grid to end before that one,
    // the next kernel, which waits for this grid alone, would start too early.
    const auto wait = [] { asm volatile("griddepcontrol.wait;" ::: "memory"); };
    // (what precedes the direct kernel has completed before this one starts, and that one writes none of these)
    const int idx = fold[blockIdx.x];
    if (idx < 0) return wait();                                 // padding
    const pa_work_item it = p.items[min(idx, p.n_items - 1)];
    const int row = blockIdx.y * kFoldWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const bool good = idx < p.n_items && it.kind == PA_ITEM_DIRECT && it.split == 0 && it.n_splits >= 2 && it.tile0 >= 0 &&
                      it.tile0 <= p.n_items - it.n_splits && it.n_q >= 1 && it.n_q <= (kCols >> p.log2g) &&
                      it.q_start >= 0 && it.q_start <= p.T - it.n_q && it.kv_head >= 0 && it.kv_head < p.Hkv &&
                      it.seq >= 0 && it.seq < p.B;
    if (!good) {
        if (row == 0 && lane == 0 && p.err) atomicOr(p.err, PA_DEVERR_META);
        return wait();
    }
    if (row >= it.n_q << p.log2g) return wait();
    // an item that the direct kernel refused has left no parts
    const int ctx = p.ctx[it.seq], cu0 = p.cu[it.seq], cu1 = p.cu[it.seq + 1];
    if (ctx <= 0 || ctx != it.next || ctx > p.max_ctx || cu0 > it.q_start || it.q_start + it.n_q > cu1 ||
        int64_t(cu1) - cu0 > ctx)
        return wait();
    const int64_t keys = ctx - (cu1 - it.q_start) + it.n_q, len = q4_split_keys(ctx);
    if (!split_in(keys, len, it.n_splits) || (int64_t(ctx) + (1 << p.log2bs) - 1) >> p.log2bs > p.max_blocks)
        return wait();
    wait();
    const int n_splits = it.n_splits;
    const float* const part = p.part + int64_t(it.tile0) * kPart + row * D + kLane * lane;
    const float* const stat = p.part + int64_t(it.tile0) * kPart + kCols * D + 2 * row;
    float a[2][kEight][kLane];
    float2 ml[2];
    // lane i has (m, l) of the eight's split i; those behind the last weigh nothing
    const auto load = [&](int s0, float (&a)[kEight][kLane], float2& ml) {
        ml = make_float2(-kNone, 0.f);
        if (s0 + lane < n_splits && lane < kEight)
            ml = *reinterpret_cast<const float2*>(stat + int64_t(s0 + lane) * kPart);
#pragma unroll
        for (int i = 0; i < kEight; ++i) {
            if (s0 + i >= n_splits) continue;
            if constexpr (kLane == 4) {
                const float4 v = *reinterpret_cast<const float4*>(part + int64_t(s0 + i) * kPart);
                a[i][0] = v.x, a[i][1] = v.y, a[i][2] = v.z, a[i][3] = v.w;
            } else {
                const float2 v = *reinterpret_cast<const float2*>(part + int64_t(s0 + i) * kPart);
                a[i][0] = v.x, a[i][1] = v.y;
            }
        }
    };
    float M = -kNone, Lsum = 0.f, sum[kLane] = {};
    const auto join = [&](int s0, const float (&a)[kEight][kLane], float2 ml) {
        float m = ml.x;
#pragma unroll
        for (int d = 1; d < kEight; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        m = __shfl_sync(0xffffffffu, m, 0);
        const float f = ex2(ml.x - m), fl = f * ml.y;
        float l = 0.f, out[kLane] = {};
#pragma unroll
        for (int i = 0; i < kEight; ++i) {
            const float fi = __shfl_sync(0xffffffffu, f, i);
            l += __shfl_sync(0xffffffffu, fl, i);
            if (s0 + i >= n_splits) continue;
#pragma unroll
            for (int c = 0; c < kLane; ++c) out[c] = fmaf(a[i][c], fi, out[c]);
        }
        const float now = fmaxf(M, m), fa = ex2(M - now), fb = ex2(m - now);
        Lsum = Lsum * fa + l * fb;
#pragma unroll
        for (int c = 0; c < kLane; ++c) sum[c] = sum[c] * fa + out[c] * fb;
        M = now;
    };
    load(0, a[0], ml[0]);
    for (int s0 = 0; s0 < n_splits; s0 += 2 * kEight) {
        load(s0 + kEight, a[1], ml[1]);
        join(s0, a[0], ml[0]);
        load(s0 + 2 * kEight, a[0], ml[0]);
        if (s0 + kEight < n_splits) join(s0 + kEight, a[1], ml[1]);
    }
    const float inv = __frcp_rn(Lsum);
    __nv_bfloat16* const out = p.out + (int64_t(it.q_start + (row >> p.log2g)) * p.Hq + (it.kv_head << p.log2g) +
                                        (row & ((1 << p.log2g) - 1))) * D + kLane * lane;
#pragma unroll
    for (int c = 0; c < kLane; c += 2)
        *reinterpret_cast<uint32_t*>(out + c) = pack_bf16(sum[c] * inv, sum[c + 1] * inv);
}

// ------------------------------------------------------------------------------- host side

template <int D, int NT>
int32_t launch_direct(const DirectParams& p, const int32_t* fold, int32_t n_fold, int32_t fold_rows,
                      cudaStream_t stream) {
    static std::atomic<bool> raised[kMaxDevices];               // zero-initialised: not raised yet
    int dev = 0;
    int32_t st = note_cuda(cudaGetDevice(&dev));
    if (st) return st;
    if (dev < 0 || dev >= kMaxDevices) return PA_ERR_INVALID;
    constexpr int smem = kWarps<NT> * Ring<D>::kWarp + kWarps<NT> / 2 * kHanded<D, NT>;
    if (!raised[dev].load(std::memory_order_acquire)) {
        st = note_cuda(cudaFuncSetAttribute(q4_direct_kernel<D, NT>,
                                            cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
        if (st) return st;
        raised[dev].store(true, std::memory_order_release);
    }
    cudaLaunchAttribute pdl;
    auto cfg = dependent_launch(&pdl, dim3(PA_PLAN_CTAS), 32 * kWarps<NT>, smem, stream);
    st = note_cuda(cudaLaunchKernelEx(&cfg, q4_direct_kernel<D, NT>, p));
    if (st || n_fold == 0) return st;
    const dim3 grid{unsigned(n_fold), unsigned((fold_rows + kFoldWarps - 1) / kFoldWarps)};
    cfg = dependent_launch(&pdl, grid, 32 * kFoldWarps, 0, stream);
    return note_cuda(cudaLaunchKernelEx(&cfg, q4_fold_kernel<D, NT>, p, fold));
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
    const int64_t rows = int64_t(T) * shape->num_kv_heads;
    if (rows > INT32_MAX) return PA_ERR_SHAPE;
    p.rows = uint32_t(rows);
    p.Hkv = shape->num_kv_heads;
    // ceil(2^(31 + k) / Hkv), 2^(k - 1) < Hkv <= 2^k: too large by less than 1, so the quotient's error is below
    // row / 2^(31 + k), less than the 1 / Hkv that is between it and the next whole number
    p.div_shift = 31 + ilog2(p.Hkv);
    p.div = uint32_t(((uint64_t(1) << p.div_shift) + p.Hkv - 1) / p.Hkv);
    p.log2bs = ilog2(shape->block_size);
    p.err = err;
    const int per = kRowsThreads / (WRITE ? shape->head_dim / 16 : 4);
    const int64_t blocks = (rows + per - 1) / per;
    cudaLaunchAttribute pdl;
    auto cfg = dependent_launch(&pdl, dim3(unsigned(blocks)), kRowsThreads, 0, stream);
    if (shape->head_dim == 128)
        return note_cuda(cudaLaunchKernelEx(&cfg, WRITE ? q4_write_kernel<128> : q4_read_kernel<128>, p));
    return note_cuda(cudaLaunchKernelEx(&cfg, WRITE ? q4_write_kernel<64> : q4_read_kernel<64>, p));
}

// Parts of the workspace, each a multiple of 256 bytes.
struct Space {
    // sizes: split parts, decode partials, one pool, contexts and queue, types of V
    size_t parts, partials, expanded, ctx, types, total;
};

Space space_of(const pa_shape* s, const pa_q4_plan* p) {
    const auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    Space w{};
    const int D = s->head_dim, g = s->num_q_heads / s->num_kv_heads;
    const int cols = q4_tile_rows(g, *p);
    if (p->n_fold > 0) w.parts = up(size_t(p->n_direct) * cols * (D + 2) * 4);
    if (p->n_chunk > 0) {
        // single tokens are among the expanded rows only where a group is larger than direct_rows
        if (p->direct_rows < g && p->max_ctx > PA_SPLIT_TOKENS)
            w.partials = up(pa_workspace_bytes(s, p->T, p->max_ctx));
        w.expanded = up(size_t(p->n_expand) * 128 * s->num_kv_heads * D * 2);
        w.ctx = up((size_t(p->B) + 1) * 4);
        w.types = up(size_t(p->n_expand) * s->num_kv_heads);
    }
    w.total = w.parts + w.partials + 2 * w.expanded + w.ctx + w.types;
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
    // places in a pool are counted in 16 bytes, in 32 bits
    if (int64_t(shape->num_blocks) * shape->num_kv_heads * (shape->block_size * (shape->head_dim / 8) * 5 / 16) >
        int64_t(UINT32_MAX))
        return PA_ERR_SHAPE;
    const Space w = space_of(shape, plan);
    if (w.total > 0 && (!workspace || ws_bytes < w.total)) return PA_ERR_WORKSPACE;
    if (w.total > 0 && !aligned16(workspace)) return PA_ERR_INVALID;
    uint8_t* at = static_cast<uint8_t*>(workspace);
    const int D = shape->head_dim, Hq = shape->num_q_heads, Hkv = shape->num_kv_heads, g = Hq / Hkv;
    const Q4Words f = q4_words(P);
    int32_t* queue = nullptr;
    if (P.n_chunk > 0) {
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
        e.queue = queue = e.ex_ctx + P.B;
        e.v16 = reinterpret_cast<uint8_t*>(e.ex_ctx) + w.ctx;
        e.err = err_flag;
        e.B = P.B;
        e.cols = P.expand_cols;
        e.max_blocks = max_blocks;
        e.num_blocks = shape->num_blocks;
        e.Hkv = Hkv;
        e.g = g;
        e.log2bs = ilog2(shape->block_size);
        e.direct_rows = P.direct_rows;
        cudaLaunchAttribute pdl;
        auto cfg = dependent_launch(&pdl, dim3(unsigned(P.n_expand), unsigned(Hkv)), 256, 0, stream);
        st = note_cuda(D == 128 ? cudaLaunchKernelEx(&cfg, q4_expand_kernel<128>, e)
                                : cudaLaunchKernelEx(&cfg, q4_expand_kernel<64>, e));
        if (st) return st;
        pa_shape ex = *shape;
        ex.block_size = 128;
        ex.num_blocks = P.n_expand;
        st = attention_step_expanded(q, e.k_out, e.v_out, e.ex_table, e.cols, cu_seqlens_q, e.ex_ctx, P.B,
                                     P.T, P.max_ctx, e.v16,
                                     reinterpret_cast<const pa_work_item*>(words + f.chunk), P.n_chunk,
                                     w.partials ? at + w.parts : nullptr, out, &ex, err_flag, stream);
        if (st) return st;
    }
    if (P.n_direct == 0) return PA_OK;
    DirectParams p{};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k_pool = static_cast<const uint8_t*>(k_pool);
    p.v_pool = static_cast<const uint8_t*>(v_pool);
    p.table = block_table;
    p.cu = cu_seqlens_q;
    p.ctx = ctx_lens;
    p.items = reinterpret_cast<const pa_work_item*>(words + f.direct);
    p.lists = words + f.lists;
    p.queue = queue;
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
    p.bits = 0x43004300u;
    const int32_t* fold = words + f.fold;
    const bool wide = q4_tile_rows(g, P) > 8;
    return D == 128 ? (wide ? launch_direct<128, 2>(p, fold, P.n_fold, P.fold_rows, stream)
                            : launch_direct<128, 1>(p, fold, P.n_fold, P.fold_rows, stream))
                    : (wide ? launch_direct<64, 2>(p, fold, P.n_fold, P.fold_rows, stream)
                            : launch_direct<64, 1>(p, fold, P.n_fold, P.fold_rows, stream));
}
