// Eviction from a paged cache by accumulated attention weight, per (sequence, KV head): which
// `budget` of the ctx entries stay, and the compaction of K, V, weights and token positions.
//
// Rank of an entry: protected ones first (token position < sink, or among the last `recent`
// tokens), then the larger weight, ties to the lower index. The first `budget` stay. An entry that
// stays and lies behind the budget (a stray) moves into the place of one that goes and lies before
// it (a hole), the k-th into the k-th; the others stay where they are. The order of keys means
// nothing to attention (the rotation is in them), so only the strays' rows are read and written:
// one row per head where a full cache makes room for one token, against the whole cache if it
// were kept in order. Each entry's position is carried along for the next call's protection.
//
// A cluster of C CTAs takes one (sequence, head): each reads its slice of the weights once (held
// as ordered 32-bit keys in shared memory; entries before the budget are copied to the output on
// the way), up to three radix passes (11, 11, 10 bits) over histograms find the key of rank `budget`,
// and two bitmaps (above it, equal to it) give the holes and strays. A pass's non-empty bins are
// added up in the first CTA's shared memory, which finds the bin and tells the others: tens of
// bins (pulling whole histograms from each other took 25 us a pass). Nothing depends on the order
// of atomics: they count. Then the CTAs share the moves. Bound by latency when few rows move (the
// passes' barriers), by the strays' K and V rows otherwise.
//
// Shared memory and the cluster's size follow max_len: the contexts are the device's to know.
//
// Measured (8 KV heads of 128): 64 full caches of 2,049 entries in a graph, 10.1 us with state rows of
// 2,054 entries (one wave of CTAs), 14.2 with rows of 8,192 to 131,072 (two waves, for the bitmaps and
// keys that longer contexts would need), 24.1 with 524,288; eight prompts of
// 4,000 .. 40,000 cut to 2,048 (123 MB) 42 us, of a CTA's time on average 5 up to the first histogram, 9
// in the passes and bitmaps, 6 to list the moves and 10 in them (where memory is at its limit).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "common.h"

namespace cg = cooperative_groups;
using namespace pa_detail;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;                // of a radix pass
constexpr int kPer = kBins / kThreads;     // bins a thread scans
constexpr int kWindow = 1024;              // moves listed at a time
constexpr int kBatch = 8;                  // loads a thread has in flight
constexpr int kCache = 8192;               // keys a CTA holds; a longer slice is read once a pass
constexpr int kMaxLen = 1 << 19;           // entries: the bitmaps lie in shared memory
constexpr int kMaxCluster = 8;

struct EvictParams {
    uint4 *k_pool, *v_pool;
    const int32_t *table, *ctx, *budget, *n_tokens, *kept, *rows;
    const float* w_in;
    float* w_out;
    const int32_t* pos_in;
    int32_t* pos_out;
    int32_t* err;
    int32_t B, max_blocks, Hkv, log2bs, num_blocks, n_rows, max_len, recent, sink;
    int32_t log2_vecs;                     // 16-byte vectors of one head's row
    int32_t cache;                         // keys there is room for
};

// Shared memory after the fixed part: the keep bitmap of all entries, the slice's equal bitmap,
// the slice's keys.
struct Fixed {
    int32_t hist[kBins];                   // the CTA's own counts
    int32_t all[kBins];                    // the cluster's, in the first CTA
    int32_t hole[kWindow], stray[kWindow];
    int32_t warp_sum[kWarps];
    int32_t bin, need, count, equal, clash;
};

__device__ __forceinline__ uint32_t order_key(float w) {
    if (w != w) return 0xFFFFFFFEu;                    // NaN: above every number
    const uint32_t u = __float_as_uint(w + 0.f);       // -0 ranks as 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Inclusive sum over the block (and the total); every thread calls it.
__device__ __forceinline__ int block_scan(int x, int32_t* warp_sum, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();                                   // the previous call's sums have been read
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const int v = warp_sum[w];
        if (w < warp) before += v;
        total += v;
    }
    return x + before;
}

// kMany: more than one CTA per (sequence, head).
template <bool kMany>
__global__ void __launch_bounds__(kThreads, 4) evict_kernel(const EvictParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    Fixed& sh = *reinterpret_cast<Fixed*>(smem);
    cg::cluster_group cluster = cg::this_cluster();
    const int C = kMany ? int(cluster.num_blocks()) : 1;
    const int rank = kMany ? int(cluster.block_rank()) : 0;
    const auto sync_all = [&]() {
        if constexpr (kMany) cluster.sync();
        else __syncthreads();
    };
    const int h = int(blockIdx.y), s = int(blockIdx.z);
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < kBins; i += kThreads) {
        sh.hist[i] = 0;
        if (kMany) sh.all[i] = 0;
    }
    if (tid == 0) sh.clash = 0;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- the sequence, the same for every CTA of the cluster
    const int row = p.rows ? p.rows[s] : s;
    const int ctx = p.ctx[s], budget = p.budget[s], n_tokens = p.n_tokens[s];
    const int kept = p.kept ? p.kept[s] : 0;
    if (row < 0) return;                               // takes no part
    __syncthreads();
    if (p.rows)
        for (int i = tid; i < p.B; i += kThreads)
            if (i != s && p.rows[i] == row) sh.clash = 1;
    __syncthreads();
    if (ctx < 0 || ctx > p.max_len || budget < 1 || kept < 0 || kept > ctx || n_tokens < ctx ||
        row >= p.n_rows || sh.clash ||
        ((int64_t(ctx) + (1 << p.log2bs) - 1) >> p.log2bs) > p.max_blocks) {
        if (tid == 0 && p.err) atomicOr(p.err, PA_DEVERR_META);
        return;
    }
    const int64_t state = (int64_t(row) * p.Hkv + h) * p.max_len;
    const float* w_in = p.w_in + state;
    float* w_out = p.w_out + state;
    const int32_t* pos_in = p.pos_in + state;
    int32_t* pos_out = p.pos_out + state;
    const bool same_w = w_in == w_out, same_pos = pos_in == pos_out;
    const int len = min(ctx, budget);
    const int since = n_tokens - ctx;                  // position of entry j >= kept: since + j
    const int recent_from = n_tokens - min(p.recent, n_tokens);
    const auto position = [&](int j) { return j < kept ? pos_in[j] : since + j; };
    const auto rank_key = [&](int pos, float w) {
        return pos < p.sink || pos >= recent_from ? 0xFFFFFFFFu : order_key(w);
    };
    const int words = (ctx + 31) / 32;
    const int w0 = int(int64_t(words) * rank / C), w1 = int(int64_t(words) * (rank + 1) / C);
    const int j0 = 32 * w0, j1 = min(ctx, 32 * w1);
    uint32_t* keep = reinterpret_cast<uint32_t*>(smem + sizeof(Fixed));
    uint32_t* equal = keep + words;
    uint32_t* cached = equal + (words / C + 1);
    const bool hold = j1 - j0 <= p.cache;
    const bool cut = ctx > budget;                     // something goes
    // the first CTA's counts start at zero before another adds to them (awaited below)
    if constexpr (kMany)
        if (cut) cluster.barrier_arrive();

    // ---- the slice's keys, counted by their top bits; what lies before the budget goes to the
    // output as if it stayed (an evicted entry's place is overwritten by its stray later, behind a
    // barrier of the cluster)
    for (int base = j0; base < j1; base += kThreads * kBatch) {
        float w[kBatch];
        int pos[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int j = base + i * kThreads + tid;
            if (j < j1) {
                w[i] = w_in[j];
                pos[i] = position(j);
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int j = base + i * kThreads + tid;
            if (base + i * kThreads >= j1) break;
            uint32_t k = 0;
            if (j < j1) {
                k = rank_key(pos[i], w[i]);
                if (j < len) {
                    if (!same_w) w_out[j] = w[i];
                    if (!same_pos || j >= kept) pos_out[j] = pos[i];
                }
            }
            if (!cut) continue;
            if (j < j1 && hold) cached[j - j0] = k;
            // the protected all fall in one bin: one count for a warp's
            const bool guarded = j < j1 && k == 0xFFFFFFFFu;
            const uint32_t all = __ballot_sync(0xffffffffu, guarded);
            if (guarded) {
                if (lane == __ffs(all) - 1) atomicAdd(&sh.hist[kBins - 1], __popc(all));
            } else if (j < j1) {
                atomicAdd(&sh.hist[k >> 21], 1);
            }
        }
    }
    if (!cut) return;
    const auto key_of = [&](int j) {
        return hold ? cached[j - j0] : rank_key(position(j), w_in[j]);
    };

    // ---- the key of rank `len`, and how many of its equals stay
    uint32_t prefix = 0;
    int need = len, count = ctx, shift = 32;
    // (where all of a bin stay its lower bits need not be looked at: mostly the third pass)
#pragma unroll 1
    for (int pass = 0; pass < 3 && need < count; ++pass) {
        shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const int bits = pass == 2 ? 10 : 11;
        if (pass > 0)
            for (int j = j0 + tid; j < j1; j += kThreads) {
                const uint32_t k = key_of(j);
                if (k >> (shift + bits) == prefix)
                    atomicAdd(&sh.hist[k >> shift & ((1 << bits) - 1)], 1);
            }
        int4* own = reinterpret_cast<int4*>(sh.hist) + tid * (kPer / 4);
        if constexpr (kMany) {
            if (pass == 0) cluster.barrier_wait();
            __syncthreads();
            int32_t* all = cluster.map_shared_rank(sh.all, 0) + tid * kPer;
#pragma unroll
            for (int e = 0; e < kPer / 4; ++e) {
                const int4 v = own[e];
                if (v.x) atomicAdd(all + 4 * e, v.x);
                if (v.y) atomicAdd(all + 4 * e + 1, v.y);
                if (v.z) atomicAdd(all + 4 * e + 2, v.z);
                if (v.w) atomicAdd(all + 4 * e + 3, v.w);
                own[e] = make_int4(0, 0, 0, 0);
            }
        }
        sync_all();
        if (rank == 0) {
            int4* from = kMany ? reinterpret_cast<int4*>(sh.all) + tid * (kPer / 4) : own;
            int n[kPer], sum = 0, total;
#pragma unroll
            for (int e = 0; e < kPer / 4; ++e) {
                const int4 v = from[e];
                from[e] = make_int4(0, 0, 0, 0);
                n[4 * e] = v.x;
                n[4 * e + 1] = v.y;
                n[4 * e + 2] = v.z;
                n[4 * e + 3] = v.w;
                sum += v.x + v.y + v.z + v.w;
            }
            // rank `need` from the top is index count - need from the bottom
            const int index = count - need;
            int upto = block_scan(sum, sh.warp_sum, total);
            int below = upto - sum;
            if (below <= index && index < upto) {
#pragma unroll
                for (int e = 0; e < kPer; ++e) {
                    if (below <= index && index < below + n[e])
                        for (int r = 0; r < C; ++r) {
                            Fixed* to = kMany ? cluster.map_shared_rank(&sh, r) : &sh;
                            to->bin = tid * kPer + e;
                            to->need = need - (count - below - n[e]);
                            to->count = n[e];
                        }
                    below += n[e];
                }
            }
        }
        sync_all();
        prefix = prefix << bits | uint32_t(sh.bin);
        need = sh.need;
        count = sh.count;
    }

    // ---- the slice's entries above it and equal to it; equal ones stay from the lowest index on
    const bool ties = need < count;
    for (int w = w0 + warp; w < w1; w += kWarps) {
        const int j = 32 * w + lane;
        const uint32_t k = j < j1 ? key_of(j) >> shift : 0u;
        const uint32_t gt = __ballot_sync(0xffffffffu, j < j1 && k > prefix);
        const uint32_t eq = __ballot_sync(0xffffffffu, j < j1 && k == prefix);
        if (lane == 0) {
            keep[w] = ties ? gt : gt | eq;
            equal[w - w0] = eq;
        }
    }
    __syncthreads();
    const int n_words = w1 - w0;
    if (ties) {                                        // the same for the whole cluster
        const int per = (n_words + kThreads - 1) / kThreads;
        const int a = min(n_words, tid * per), b = min(n_words, a + per);
        int mine = 0, total;
        for (int w = a; w < b; ++w) mine += __popc(equal[w]);
        int before = block_scan(mine, sh.warp_sum, total) - mine;
        if constexpr (kMany) {
            if (tid == 0) sh.equal = total;
            cluster.sync();
            for (int r = 0; r < rank; ++r) before += *cluster.map_shared_rank(&sh.equal, r);
        }
        for (int w = a; w < b; ++w) {
            uint32_t e = equal[w];
            const int has = __popc(e), take = min(has, max(0, need - before));
            for (int i = has; i > take; --i) e ^= 0x80000000u >> __clz(e);   // the highest go
            keep[w0 + w] |= e;
            before += has;
        }
        __syncthreads();
    }
    if constexpr (kMany) {
        // every CTA gets the others' words; nothing of another CTA is touched after the barrier
        for (int r = 0; r < C; ++r) {
            if (r == rank) continue;
            uint32_t* other = cluster.map_shared_rank(keep, r);
            for (int w = w0 + tid; w < w1; w += kThreads) other[w] = keep[w];
        }
        cluster.sync();
    }

    // ---- holes and strays, this CTA's share of the moves a window at a time
    const auto bits_of = [&](int w, bool holes) {
        const int below = len - 32 * w;                // entries of the word that lie before len
        const uint32_t in = below >= 32 ? 0xffffffffu : below <= 0 ? 0u : (1u << below) - 1;
        return holes ? ~keep[w] & in : keep[w] & ~in;
    };
    // Both kinds' ranks, a word per thread and kThreads words at a time (neighbouring words are
    // dense in holes: a thread with several of them would list them alone): the number before the
    // thread's word and in the whole round, holes in the lower 16 bits, strays in the upper ones
    static_assert(32 * kThreads < 1 << 16, "a round's counts fit 16 bits");
    const auto round_scan = [&](int w, int& all) {
        const int n = w < words ? __popc(bits_of(w, true)) | __popc(bits_of(w, false)) << 16 : 0;
        return block_scan(n, sh.warp_sum, all) - n;
    };
    int moves = 0;                                     // as many as there are holes
    for (int r = 0; 32 * r < len; r += kThreads) {
        int all;
        round_scan(r + tid, all);
        moves += all & 0xffff;
    }
    const int m0 = int(int64_t(moves) * rank / C), m1 = int(int64_t(moves) * (rank + 1) / C);
    const auto list = [&](int32_t* to, int at, int w, bool holes, int first, int end) {
        if (at >= end || at + 32 <= first) return;
        for (uint32_t m = bits_of(w, holes); m; m &= m - 1, ++at)
            if (at >= first && at < end) to[at - first] = 32 * w + __ffs(m) - 1;
    };
    const int32_t* table = p.table + int64_t(s) * p.max_blocks;
    // the slot of entry j, -1 where the table leads outside the pool
    const auto slot_of = [&](int j) {
        const int b = table[j >> p.log2bs];
        return b < 0 || b >= p.num_blocks ? -1
                                          : (b << p.log2bs) + (j & ((1 << p.log2bs) - 1));
    };
    const int log2_parts = p.log2_vecs + 1;            // vectors of a row's K and V
    const int part_mask = (1 << log2_parts) - 1, vec_mask = (1 << p.log2_vecs) - 1;
    for (int first = m0; first < m1; first += kWindow) {
        const int end = min(m1, first + kWindow);
        __syncthreads();
        for (int r = 0, holes = 0, strays = 0; r < words; r += kThreads) {
            const int w = r + tid;
            int all;
            const int before = round_scan(w, all);
            if (w < words) {
                list(sh.hole, holes + (before & 0xffff), w, true, first, end);
                list(sh.stray, strays + (before >> 16), w, false, first, end);
            }
            holes += all & 0xffff;
            strays += all >> 16;
        }
        __syncthreads();
        for (int e = tid; e < end - first; e += kThreads) {
            const int to = sh.hole[e], from = sh.stray[e];
            const int dst = slot_of(to), src = slot_of(from);
            const bool inside = dst >= 0 && src >= 0;
            if (inside) {
                w_out[to] = w_in[from];
                pos_out[to] = position(from);
            } else if (p.err) {
                // the hole keeps its own entry whole: weight and position are in the output already
                atomicOr(p.err, PA_DEVERR_BLOCK);
            }
            sh.hole[e] = inside ? dst : -1;            // the lists hold slots from here on
            sh.stray[e] = src;
        }
        __syncthreads();
        const int total = (end - first) << log2_parts;
        for (int e0 = tid; e0 < total; e0 += kBatch * kThreads) {
            uint4 v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int e = e0 + i * kThreads;
                if (e >= total || sh.hole[e >> log2_parts] < 0) continue;
                const int part = e & part_mask;
                const int64_t at = (int64_t(sh.stray[e >> log2_parts]) * p.Hkv + h) << p.log2_vecs;
                v[i] = (part > vec_mask ? p.v_pool : p.k_pool)[at + (part & vec_mask)];
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int e = e0 + i * kThreads;
                if (e >= total || sh.hole[e >> log2_parts] < 0) continue;
                const int part = e & part_mask;
                const int64_t at = (int64_t(sh.hole[e >> log2_parts]) * p.Hkv + h) << p.log2_vecs;
                (part > vec_mask ? p.v_pool : p.k_pool)[at + (part & vec_mask)] = v[i];
            }
        }
    }
}

constexpr int kMaxDevices = 64;
// the largest: the fixed part, two bitmaps of kMaxLen and the keys
constexpr int kMaxSmem = int(sizeof(Fixed)) + 2 * kMaxLen / 8 + 4 + 4 * kCache;
static_assert(kMaxSmem <= 227 * 1024, "shared memory of one CTA");

}  // namespace

extern "C" int32_t paged_evict(void* k_pool, void* v_pool, int32_t elem_bytes,
                               const int32_t* block_table, int32_t max_blocks,
                               const int32_t* ctx_lens, const int32_t* budget,
                               const int32_t* n_tokens, const int32_t* kept, const int32_t* rows,
                               int32_t B, int32_t recent, int32_t sink, const float* weights,
                               float* weights_out, const int32_t* positions,
                               int32_t* positions_out, int32_t n_rows, int32_t max_len,
                               const pa_shape* shape, int32_t* err_flag, pa_stream_t stream) {
    int32_t st = check_shape(shape);
    if (st) return st;
    if (elem_bytes != 1 && elem_bytes != 2) return PA_ERR_SHAPE;
    if (B < 0 || max_blocks < 0 || recent < 0 || sink < 0 || n_rows < 0 || max_len < 0)
        return PA_ERR_INVALID;
    if (B == 0) return PA_OK;
    if (!k_pool || !v_pool || !block_table || !ctx_lens || !budget || !n_tokens || !weights ||
        !weights_out || !positions || !positions_out || max_len == 0 || (!rows && n_rows < B))
        return PA_ERR_INVALID;
    if (max_len > kMaxLen || B > 65535 || shape->num_kv_heads > 65535 ||
        int64_t(shape->num_blocks) * shape->block_size > INT32_MAX)
        return PA_ERR_SHAPE;
    const auto aligned = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
    if (!aligned(k_pool) || !aligned(v_pool)) return PA_ERR_INVALID;
    // weights and positions are replaced in place or written elsewhere, not half over themselves
    const size_t bytes = size_t(n_rows) * shape->num_kv_heads * max_len * 4;
    const auto overlaps = [&](const void* a, const void* b) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
        return x != y && x < y + bytes && y < x + bytes;
    };
    if (overlaps(weights, weights_out) || overlaps(positions, positions_out))
        return PA_ERR_INVALID;
    int dev = 0;
    if ((st = note_cuda(cudaGetDevice(&dev)))) return st;
    if (dev < 0 || dev >= kMaxDevices) return PA_ERR_INVALID;
    static std::atomic<bool> raised[kMaxDevices];
    if (!raised[dev].load(std::memory_order_acquire)) {
        constexpr auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
        if ((st = note_cuda(cudaFuncSetAttribute(evict_kernel<false>, attr, kMaxSmem)))) return st;
        if ((st = note_cuda(cudaFuncSetAttribute(evict_kernel<true>, attr, kMaxSmem)))) return st;
        raised[dev].store(true, std::memory_order_release);
    }
    EvictParams p;
    p.k_pool = static_cast<uint4*>(k_pool);
    p.v_pool = static_cast<uint4*>(v_pool);
    p.table = block_table;
    p.ctx = ctx_lens;
    p.budget = budget;
    p.n_tokens = n_tokens;
    p.kept = kept;
    p.rows = rows;
    p.w_in = weights;
    p.w_out = weights_out;
    p.pos_in = positions;
    p.pos_out = positions_out;
    p.err = err_flag;
    p.B = B;
    p.max_blocks = max_blocks;
    p.Hkv = shape->num_kv_heads;
    p.log2bs = 0;
    while ((1 << p.log2bs) < shape->block_size) ++p.log2bs;
    p.num_blocks = shape->num_blocks;
    p.n_rows = n_rows;
    p.max_len = max_len;
    p.recent = recent;
    p.sink = sink;
    p.log2_vecs = 0;
    while ((16 << p.log2_vecs) < shape->head_dim * elem_bytes) ++p.log2_vecs;
    // CTAs per (sequence, head): as many as the GPU holds at once, each with a thousand entries
    int C = kMaxCluster;
    while (C > 1 && (int64_t(B) * p.Hkv * C > 4 * PA_PLAN_CTAS || max_len / C < 1024)) C /= 2;
    const int words = (max_len + 31) / 32, slice = 32 * (words / C + 1);
    p.cache = std::min(kCache, slice);
    const size_t smem = sizeof(Fixed) + 4 * size_t(words) + 4 * size_t(words / C + 1) +
                        4 * size_t(p.cache);
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = unsigned(C);
    attrs[1].val.clusterDim.y = 1;
    attrs[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(C), unsigned(p.Hkv), unsigned(B));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attrs;
    cfg.numAttrs = C > 1 ? 2 : 1;
    return note_cuda(C > 1 ? cudaLaunchKernelEx(&cfg, evict_kernel<true>, p)
                           : cudaLaunchKernelEx(&cfg, evict_kernel<false>, p));
}
