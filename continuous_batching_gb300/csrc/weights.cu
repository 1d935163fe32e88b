// The attention weight every cached key received from a step's query rows:
//
//   w[row(s)][kvh][j] (+)= sum over rows i of s with pos_i >= j, q heads h of the group, of
//                          exp(q_ih . k_j / sqrt(D) - lse_ih)
//
// lse being the rows' log-sum-exp, which the attention step gives. With it a key's sum needs one
// look at the key and no second pass over the row.
//
// S^T = K Q^T: the MMA's 128 rows (A) are the keys of one tile and its columns (B) the (token,
// head-in-group) pairs of one KV head, so that a key is a TMEM lane. The thread that reads the
// lane adds its columns' exponentials in a register: no exchange between lanes, no atomics, one
// writer per entry, and an order of additions that is fixed. A stale key behind ctx (NaN even)
// stays in its own lane, which is not written; a stale or foreign query stays in its own column,
// which is not read.
//
// Two forms, chosen per sequence:
//   FEW   all its columns fit one query tile (n_q * g <= 128; a decode row among them): the query
//         tile stays, key tiles stream past it. Bound by the read of K (a 32 KB tile per 128 keys
//         against 16 .. 128 MMA columns); K is read once, no other pass touches it.
//   MANY  a prefill chunk: one or two key tiles stay, query tiles (128 columns) stream past them
//         from L2. Bound by the tensor pipe and the exponentials (per element one fused
//         multiply-add and one addition, packed in pairs, and one ex2).
// Work is dealt by cost, on the device: every (sequence, KV head, key tile) in order has a cost
// (4 for a FEW tile, 2 for each query tile a MANY tile meets), CTA c takes the tiles that start in
// its 1/G of the total. No plan is made or uploaded, so a captured graph needs nothing renewed but
// its metadata.
//
// Warps: 0-15 four epilogue warpgroups, 16 scheduler and loader of what stays, 17 and 20 MMA issuers,
// 18 loader of what streams, 19 log-sum-exps; over an fp8 cache 24-27 turn codes and q to f16. The
// stream's tiles alternate between the two issuers, each with two of the four accumulators (128
// TMEM columns each): an issuer's waits, commits and address arithmetic, made slow by the warps it
// shares its scheduler with, run while the other's MMAs keep the tensor pipe busy (one issuer left
// it idle for more than half of the time). FEW: each tile has one accumulator and one warpgroup.
// MANY: a query tile has an accumulator for each of its two key tiles, and each of these is read by
// two warpgroups, 64 columns each, whose sums meet in shared memory at the item's end.
// Shared memory: seven 32 KB slots. Two sets of two for what stays (an item loads while the one
// before it runs) and three stages for what streams; where no sequence is MANY, each set is one
// slot, and the two others are stages as well (five tiles of K in flight). Every wait is bounded.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "common.h"
#include "sm103.h"
#include "tensor_map.h"
#include "tmem_ldst.h"

using namespace pa_detail;

namespace {

constexpr int kBaseThreads = 672;
template <bool F8>
constexpr int kThreadsFor = F8 ? kBaseThreads + 128 : kBaseThreads;
constexpr int kTurners = kBaseThreads / 32;    // the first f16 warp of an fp8 cache
constexpr int kCols = 128;                     // columns of a query tile
constexpr int kSlot = 32768;                   // one tile, 128 rows of D = 128
constexpr int kHalf = 16384;                   // its 64-column halves
constexpr int kStay = 0;                       // 2 sets x 2 slots
constexpr int kMaxStages = 5;
constexpr int kCtl = 7 * kSlot;
constexpr int kBytes = kCtl + 3072;
static_assert(kBytes <= 227 * 1024, "shared memory of one CTA");
constexpr int kLseSlots = 2;
constexpr int kMaxRows = 1 << 18;              // state rows whose repeats are looked for
constexpr int64_t kCostFew = 4, kCostMany = 2; // of a key tile; of a key tile and query tile

// Stream tile n (counted over all items) has stage n % n_stages and issuer n % 2. The barriers that
// issuers wait on for it are numbered n % (2 n_stages), n_stages being odd: each is only ever waited
// on by one of them, which keeps its parity's meaning sound.
enum Bar {
    kStayFull = 0,     // + set: TMA -> issuers (or the f16 warps)
    kStayEmpty = 2,    // + set: both issuers -> loader
    kStreamFull = 4,   // + n % (2 n_stages)
    kStreamEmpty = 14, // + stage: its issuer -> loader
    kAccFull = 19,     // + accumulator, FEW: issuer -> its warpgroup
    kAccEmpty = 23,    // + accumulator, FEW: 128 arrivals -> issuer
    kPairFull = 27,    // + n % 2, MANY: issuer -> the warpgroups (one for both key tiles)
    kPairEmpty = 29,   // + n % 2, MANY: 512 arrivals -> issuer
    kLseFull = 31,     // + slot: 32 arrivals -> the warpgroups
    kLseEmpty = 33,    // + slot: 512 arrivals
    kItemFull = 35,    // + slot (4)
    kItemEmpty = 39,   // + slot: every consumer thread
    kPartFull = 43,    // + key tile of a pair: 128 arrivals, its second warpgroup -> its first
    kPartEmpty = 45,   // + key tile: 128 arrivals
    kDrain = 47,       // + issuer
    kStayReady = 49,   // + set, fp8 only: 128 arrivals of the f16 warps
    kStreamReady = 51, // + n % (2 n_stages)
    kNumBars = 61
};
constexpr int kHolderOff = 8 * kNumBars;
constexpr int kAbortOff = kHolderOff + 4;
constexpr int kRingOff = 512;                  // 4 items of 64 bytes
constexpr int kLseOff = kRingOff + 4 * 64;     // kLseSlots x 128 floats
constexpr int kPartOff = kLseOff + kLseSlots * 512;   // 2 x 128 floats
constexpr int kScanOff = kLseOff;              // before the pipeline starts
static_assert(kAbortOff + 4 <= kRingOff && kPartOff + 2 * 512 <= 3072, "control area");

// Stage st of the stream: slots 4, 5, 6, and without MANY sequences the sets' second slots 1, 3.
__device__ __forceinline__ uint32_t stage_at(int st) {
    return uint32_t(st < 3 ? 4 + st : st == 3 ? 1 : 3) * kSlot;
}

struct Params {
    const float* lse;            // [T][Hq]
    const int32_t* block_table;
    const int32_t* cu;
    const int32_t* ctx;
    const int32_t* held;         // entries that hold a sum already; NULL: ctx - n_q
    const int32_t* rows;         // state rows; NULL: the sequence's index
    float* weights;              // [n_rows][Hkv][max_len]
    int32_t* err;
    int32_t B, T, max_blocks, Hq, Hkv, g, bs, num_blocks, n_rows, max_len;
    int32_t skip_decode;         // sequences of one row are another kernel's
    float c;                     // log2(e) / sqrt(D), times the K scale of an fp8 cache
};

// What the sequences' metadata says, checked. cost 0: nothing to do (no rows, no state row, or
// metadata that does not fit, which sets bad).
struct Seq {
    int n_q, ctx, pos0, cu0, row, held;
    int n_tiles, n_qt;           // key tiles; query tiles
    bool few, bad;
    int64_t head_cost;
};

// Query tiles that key tile t does not meet: their rows all come before it.
__device__ __forceinline__ int first_qt(const Seq& q, int t, int log2qt) {
    return max(0, t * kTileKeys - q.pos0) >> log2qt;
}

// Cost of a head's key tiles before tile t.
__device__ __forceinline__ int64_t cost_before(const Seq& q, int t, int log2qt) {
    if (q.few) return kCostFew * t;
    // tiles up to u meet every query tile
    const int u = min(t, (q.pos0 + (1 << log2qt) - 1) / kTileKeys + 1);
    int64_t f = int64_t(u) * q.n_qt;
    for (int i = u; i < t; ++i) f += q.n_qt - first_qt(q, i, log2qt);
    return kCostMany * f;
}

// The first tile whose start is at or behind x.
__device__ __forceinline__ int tile_at(const Seq& q, int64_t x, int log2qt) {
    if (x <= 0) return 0;
    if (x >= q.head_cost) return q.n_tiles;
    if (q.few) return int((x + kCostFew - 1) / kCostFew);
    const int u = min(q.n_tiles, (q.pos0 + (1 << log2qt) - 1) / kTileKeys + 1);
    const int64_t per = kCostMany * q.n_qt;
    if (x <= per * u) return int((x + per - 1) / per);
    int64_t f = per * u;
    int t = u;
    for (; t < q.n_tiles && f < x; ++t) f += kCostMany * (q.n_qt - first_qt(q, t, log2qt));
    return t;
}

// Another sequence with query rows names sequence s's state row: both would race on it.
__device__ __noinline__ bool shares_row(const int32_t* rows, const int32_t* cu, int B, int s) {
    for (int i = 0; i < B; ++i)
        if (i != s && rows[i] == rows[s] && cu[i + 1] != cu[i]) return true;
    return false;
}

// repeated: some row is named twice (the sequences that do are then looked for).
__device__ __forceinline__ Seq load_seq(const Params& p, int s, int log2qt, bool repeated) {
    Seq q;
    const int c0 = p.cu[s], c1 = p.cu[s + 1];
    q.row = p.rows ? p.rows[s] : s;
    q.ctx = p.ctx[s];
    const int64_t n = int64_t(c1) - c0;
    q.bad = false;
    q.head_cost = 0;
    if (n == 0 || q.row < 0 || (p.skip_decode && n == 1)) return q;
    q.n_q = int(n);
    q.cu0 = c0;
    q.held = p.held ? p.held[s] : q.ctx - q.n_q;
    if (n < 0 || c0 < 0 || c1 > p.T || q.n_q > q.ctx || q.ctx > p.max_len ||
        (int64_t(q.ctx) + p.bs - 1) / p.bs > p.max_blocks || q.row >= p.n_rows || q.held < 0 ||
        q.held > q.ctx || (repeated && shares_row(p.rows, p.cu, p.B, s))) {
        q.bad = true;
        return q;
    }
    q.pos0 = q.ctx - q.n_q;
    q.n_tiles = (q.ctx + kTileKeys - 1) / kTileKeys;
    q.n_qt = (q.n_q + (1 << log2qt) - 1) >> log2qt;
    q.few = q.n_qt == 1;
    q.head_cost = cost_before(q, q.n_tiles, log2qt);
    return q;
}

// One unit of work, published by the scheduler: FEW: query tile 0 against key tiles t0 .. t0 + nt
// - 1; MANY: key tiles t0 (and t0 + 1 with nt 2) against query tiles qt0 .. n_qt - 1.
struct Item {
    int seq, kvh, t0, nt, qt0, n_qt, cu0, n_q, pos0, ctx, held, last;
    int64_t state;               // index of entry 0 in weights
    int pad[2];
};
static_assert(sizeof(Item) == 64, "item slot size");

__device__ __forceinline__ Item read_item(uint32_t at) {
    union {
        uint4 v[4];
        Item i;
    } u;
#pragma unroll
    for (int k = 0; k < 4; ++k) u.v[k] = ld_shared_v4(at + 16 * k);
    return u.i;
}

// Where column col's log-sum-exp lies in its slot: the order in which add16 takes them.
__device__ __forceinline__ int lse_place(int col) {
    return (col & ~15) + ((col & 7) >> 1) * 4 + ((col >> 3) & 1) * 2 + (col & 1);
}

// A thread's share of 16 columns for the 32 keys of its warp (tcgen05.ld 16x256b, the lower and
// the upper 16 lanes): keys rs + 8 k (rs = lane / 4, k = 0 .. 3) and columns 8 cc + 2 q4 + {0, 1}
// (q4 = lane % 4, cc = 0, 1). One 16-byte read of log-sum-exps so serves 16 elements: with a lane
// per key it served four, and those reads took a quarter of the shared-memory bandwidth that the
// MMAs' operands need. Adds 2^(s c + n) to the packed sum of each of the four keys.
__device__ __forceinline__ void add16(const uint32_t (&lo)[8], const uint32_t (&hi)[8], float4 n,
                                      uint64_t c2, uint64_t (&a)[4]) {
#pragma unroll
    for (int cc = 0; cc < 2; ++cc) {
        const uint64_t n2 = cc ? f2(n.z, n.w) : f2(n.x, n.y);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t* s = (k < 2 ? lo : hi) + 4 * cc + 2 * (k & 1);
            float x0, x1;
            f2_split(fma2(f2(__uint_as_float(s[0]), __uint_as_float(s[1])), c2, n2), x0, x1);
            a[k] = add2(a[k], f2(ex2(x0), ex2(x1)));
        }
    }
}

// A K slot's code rows r0 .. r0 + 31 expanded to f16 by one warp, like expand_codes but with 16 rows
// read before any is written: the reads' latency is paid twice a tile, not eight times. Rows from
// `rows` on hold nothing that counts; their (stale) codes are turned as well.
__device__ __forceinline__ void expand_rows(uint32_t slot, int r0, int rows, int lane) {
    const uint32_t c = lane & 7, j0 = 2 * (c & 3), hi = c >> 2;
#pragma unroll 1
    for (int b = r0; b < min(rows, r0 + 32); b += 16) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = ld_shared_v4(slot + kHalf + uint32_t(b + 4 * i + (lane >> 3)) * 128 + c * 16);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t R = uint32_t(b + 4 * i + (lane >> 3)), x = R & 7;
            uint32_t f[8];
            e4m3x4_to_f16x4(v[i].x, f[0], f[1]);
            e4m3x4_to_f16x4(v[i].y, f[2], f[3]);
            e4m3x4_to_f16x4(v[i].z, f[4], f[5]);
            e4m3x4_to_f16x4(v[i].w, f[6], f[7]);
            const uint32_t rb = slot + hi * kHalf + R * 128;
            st_shared_v4(rb + ((j0 ^ x) << 4), f[0], f[1], f[2], f[3]);
            st_shared_v4(rb + (((j0 + 1) ^ x) << 4), f[4], f[5], f[6], f[7]);
        }
    }
}

template <int D, bool F8>
__global__ void __launch_bounds__(kThreadsFor<F8>, 1)
    attn_weights_kernel(const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_q1,
                        const __grid_constant__ CUtensorMap tm_qn, const Params p) {
    static_assert(!F8 || D == 128, "the fp8 cache is supported at head_dim 128");
    constexpr int kChunks = D / 64;
    constexpr int kThreads = kThreadsFor<F8>;
    constexpr int kStayUse = F8 ? kStayReady : kStayFull;
    constexpr int kStreamUse = F8 ? kStreamReady : kStreamFull;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sb = smem_u32(smem);
    const uint32_t bars = sb + kCtl;
    volatile int* abort_word = reinterpret_cast<volatile int*>(smem + kCtl + kAbortOff);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const auto bar = [&](int b) { return bars + 8 * b; };
    const int log2qt = 7 - (__ffs(p.g) - 1);         // tokens of a query tile: 128 / g
    const int log2bs = __ffs(p.bs) - 1;
    if (sb & 1023) {                                 // the swizzled tiles need this alignment
        if (threadIdx.x == 0 && p.err) atomicOr(p.err, PA_DEVERR_META);
        return;
    }

    if (threadIdx.x == 0) {
        for (int b = 0; b < kNumBars; ++b)
            mbar_init(bar(b), b >= kStayReady                         ? 128
                              : b >= kDrain                           ? 1
                              : b >= kPartFull                        ? 128
                              // issuers 2, stream loader and log-sum-exps 64, epilogue 512, f16 128
                              : b >= kItemEmpty                       ? 2 + 64 + 512 + (F8 ? 128 : 0)
                              : b >= kItemFull                        ? 1
                              : b >= kLseEmpty                        ? 512
                              : b >= kLseFull                         ? 32
                              : b >= kPairEmpty                       ? 512
                              : b >= kPairFull                        ? 1
                              : b >= kAccEmpty                        ? 128
                              : b >= kStayEmpty && b < kStreamFull    ? 2
                                                                      : 1);
        *abort_word = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 17) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         bars + kHolderOff),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // a programmatic dependent: nothing the kernel before it wrote is read before this point
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- this CTA's share: repeated state rows, the total cost, where the share starts
    uint32_t* once = reinterpret_cast<uint32_t*>(smem + kStay);
    int64_t* scan = reinterpret_cast<int64_t*>(smem + kCtl + kScanOff);   // [32] warps
    int64_t* found = scan + 32;                      // start offset of the first sequence
    int* found_s = reinterpret_cast<int*>(scan + 33);
    int* repeated = found_s + 1;
    if (threadIdx.x == 0) {
        *found_s = p.B;
        *found = 0;
        *repeated = 0;
    }
    if (p.rows)
        for (int i = threadIdx.x; i < (p.n_rows + 31) / 32; i += kThreads) once[i] = 0;
    // the first round's metadata, read before the barriers
    Seq mine_seq;
    mine_seq.head_cost = 0;
    mine_seq.bad = false;
    mine_seq.few = true;
    if (int(threadIdx.x) < p.B) mine_seq = load_seq(p, int(threadIdx.x), log2qt, false);
    __syncthreads();
    if (p.rows) {
        for (int s = threadIdx.x; s < p.B; s += kThreads) {
            const int row = p.rows[s];
            if (row < 0 || row >= p.n_rows || p.cu[s + 1] == p.cu[s]) continue;
            const uint32_t bit = 1u << (row & 31);
            if (atomicOr(once + (row >> 5), bit) & bit) *repeated = 1;
        }
        __syncthreads();
    }
    const bool twice = *repeated != 0;
    int64_t total = 0;
    bool bad = false, some_many = false;
    // inclusive sums over the sequences of one round of kThreads; returns the thread's own
    const auto round_scan = [&](int64_t x, int64_t& sum) {
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        __syncthreads();
        if (lane == 31) scan[warp] = x;
        __syncthreads();
        sum = 0;
        int64_t before = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w == warp) before = sum;
            sum += scan[w];
        }
        return x + before;
    };
    int64_t mine = 0, upto = 0;
    for (int s0 = 0; s0 < p.B; s0 += kThreads) {
        const int s = s0 + int(threadIdx.x);
        mine = 0;
        if (s < p.B) {
            const Seq q = s0 == 0 && !twice ? mine_seq : load_seq(p, s, log2qt, twice);
            mine = q.head_cost * p.Hkv;
            bad = bad || q.bad;
            some_many = some_many || (q.head_cost > 0 && !q.few);
        }
        int64_t sum;
        upto = round_scan(mine, sum) + total;
        total += sum;
    }
    if (bad && blockIdx.x == 0 && p.err) atomicOr(p.err, PA_DEVERR_META);
    const int64_t lo = total * int64_t(blockIdx.x) / int64_t(gridDim.x);
    const int64_t hi = total * (int64_t(blockIdx.x) + 1) / int64_t(gridDim.x);
    if (p.B <= kThreads) {
        if (mine > 0 && upto - mine <= lo && lo < upto) {
            *found_s = int(threadIdx.x);
            *found = upto - mine;
        }
    } else if (lo < hi) {
        int64_t run = 0;
        for (int s0 = 0; s0 < p.B && run <= lo; s0 += kThreads) {
            const int s = s0 + int(threadIdx.x);
            mine = s < p.B ? load_seq(p, s, log2qt, twice).head_cost * p.Hkv : 0;
            int64_t sum;
            upto = round_scan(mine, sum) + run;
            if (mine > 0 && upto - mine <= lo && lo < upto) {
                *found_s = s;
                *found = upto - mine;
            }
            run += sum;
        }
    }
    // the rows' bits were written through the generic proxy where TMA writes next
    fence_proxy_async();
    tc_fence_before();
    const int n_stages = __syncthreads_or(some_many) ? 3 : kMaxStages;
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + kCtl + kHolderOff);
    const int start_s = *reinterpret_cast<volatile int*>(found_s);
    const int64_t start_at = *reinterpret_cast<volatile int64_t*>(found);
    __syncthreads();                                 // the scan's words belong to the ring now

    volatile Item* ring = reinterpret_cast<volatile Item*>(smem + kCtl + kRingOff);
    // takes the next item: every consumer thread (or the one lane that stands for a warp) calls it
    const auto next_item = [&](int ic, Item& I) {
        if (!wait_bounded(bar(kItemFull + (ic & 3)), (ic >> 2) & 1, abort_word)) return false;
        I = read_item(sb + kCtl + kRingOff + (ic & 3) * 64);
        mbar_arrive(bar(kItemEmpty + (ic & 3)));
        return I.last == 0;
    };
    // the K tile of key tile t into `slot` (all lanes; lane 0 has waited for the slot): one box per
    // block and 64-column half, or over an fp8 cache one box of codes per block into the second
    // half, where they are expanded. `id`: the lane's block.
    const auto blocks_of = [&](const Item& I, int t) {
        return (min(kTileKeys, I.ctx - t * kTileKeys) + p.bs - 1) >> log2bs;
    };
    const auto load_k = [&](uint32_t slot, uint32_t full, const Item& I, int nblk, int id) {
        if (lane >= nblk) return;
        const uint32_t dst = slot + lane * p.bs * 128;
        if constexpr (F8) {
            tma_load_3d(dst + kHalf, &tm_k, full, 0, I.kvh, id * p.bs);
        } else {
#pragma unroll
            for (int h = 0; h < kChunks; ++h)
                tma_load_3d(dst + h * kHalf, &tm_k, full, 64 * h, I.kvh, id * p.bs);
        }
    };
    const auto k_bytes = [&](int nblk) { return uint32_t(nblk) * p.bs * (F8 ? 128 : 128 * kChunks); };
    // the block in the lane's entry of the table, counted from key tile t's first, up to key tile
    // `end`; one outside the pool reads zeros
    const auto block_id = [&](const Item& I, int t, int end) {
        const int e = (t << (7 - log2bs)) + lane;
        if (e << log2bs >= min(I.ctx, end * kTileKeys)) return -1;
        const int b = __ldg(p.block_table + int64_t(I.seq) * p.max_blocks + e);
        if (b >= 0 && b < p.num_blocks) return b;
        if (p.err) atomicOr(p.err, PA_DEVERR_BLOCK);
        return -1;
    };
    // query tile qt: 128 rows (token, head-in-group), or one token's g rows
    const auto load_q = [&](uint32_t slot, uint32_t full, const Item& I, int qt) {
        const bool one = I.n_q == 1;
        mbar_expect_tx(full, uint32_t(one ? p.g : kCols) * 128 * kChunks);
        for (int h = 0; h < kChunks; ++h)
            tma_load_3d(slot + h * kHalf, one ? &tm_q1 : &tm_qn, full, 64 * h, I.kvh * p.g,
                        I.cu0 + (qt << log2qt));
    };

    if (warp == 16) {
        // ------------------------------------------------ scheduler, loader of what stays
        int ic = 0, ok = 1;
        // publishes an item and loads its query tile or key tiles
        const auto emit = [&](Item& I, bool few) {
            if (lane == 0) {
                if (ic >= 4)
                    ok = wait_bounded(bar(kItemEmpty + (ic & 3)), ((ic >> 2) - 1) & 1, abort_word);
                if (ok) {
                    volatile Item* v = ring + (ic & 3);
                    v->seq = I.seq;
                    v->kvh = I.kvh;
                    v->t0 = I.t0;
                    v->nt = I.nt;
                    v->qt0 = I.qt0;
                    v->n_qt = I.n_qt;
                    v->cu0 = I.cu0;
                    v->n_q = I.n_q;
                    v->pos0 = I.pos0;
                    v->ctx = I.ctx;
                    v->held = I.held;
                    v->last = I.last;
                    v->state = I.state;
                    mbar_arrive(bar(kItemFull + (ic & 3)));
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok || I.last) return;
            const int set = ic & 1;
            int id[2] = {-1, -1};
            if (!few)
                for (int r = 0; r < I.nt; ++r) id[r] = block_id(I, I.t0 + r, I.t0 + r + 1);
            if (lane == 0 && ic >= 2)
                ok = wait_bounded(bar(kStayEmpty + set), ((ic >> 1) - 1) & 1, abort_word);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) return;
            const uint32_t slot = sb + kStay + set * 2 * kSlot;
            if (few) {
                if (lane == 0) load_q(slot, bar(kStayFull + set), I, 0);
            } else {
                // one barrier for both tiles: its one arrival carries the bytes of both
                const int n0 = blocks_of(I, I.t0), n1 = I.nt == 2 ? blocks_of(I, I.t0 + 1) : 0;
                if (lane == 0) mbar_expect_tx(bar(kStayFull + set), k_bytes(n0 + n1));
                __syncwarp();
                load_k(slot, bar(kStayFull + set), I, n0, id[0]);
                load_k(slot + kSlot, bar(kStayFull + set), I, n1, id[1]);
            }
            ++ic;
        };
        int64_t base = start_at;
        for (int s = start_s; s < p.B && base < hi && ok; ++s) {
            const Seq q = load_seq(p, s, log2qt, twice);
            if (q.head_cost == 0) continue;
            Item I;
            I.seq = s;
            I.cu0 = q.cu0;
            I.n_q = q.n_q;
            I.pos0 = q.pos0;
            I.ctx = q.ctx;
            I.held = q.held;
            I.last = 0;
            I.n_qt = q.n_qt;
            for (int h = base < lo ? int((lo - base) / q.head_cost) : 0; h < p.Hkv && ok; ++h) {
                const int64_t hb = base + h * q.head_cost;
                if (hb >= hi) break;
                const int ta = tile_at(q, lo - hb, log2qt), tb = tile_at(q, hi - hb, log2qt);
                I.kvh = h;
                I.state = (int64_t(q.row) * p.Hkv + h) * p.max_len;
                if (q.few) {
                    if (ta >= tb) continue;
                    I.t0 = ta;
                    I.nt = tb - ta;
                    I.qt0 = 0;
                    emit(I, true);
                } else {
                    for (int t = ta; t < tb && ok; t += 2) {
                        I.t0 = t;
                        I.nt = min(2, tb - t);
                        I.qt0 = first_qt(q, t, log2qt);
                        emit(I, false);
                    }
                }
            }
            base += q.head_cost * p.Hkv;
        }
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        if (ok) {
            Item I = {};
            I.last = 1;
            emit(I, true);
        }
        if (lane == 0) {
            // never leave with copies in flight into this CTA's shared memory
            for (int i = max(0, ic - 2); i < ic; ++i)
                wait_drain(bar(kStayFull + (i & 1)), (i >> 1) & 1);
        }
    } else if (warp == 17 || warp == 20) {
        // ------------------------------------------------ MMA issuers
        if (lane == 0) {
            const int me = warp == 20;           // takes the stream tiles n with n % 2 == me
            int n = 0, st = 0, fb = 0;           // stream tile, its stage and full barrier
            uint32_t ph = 0;                     // parity of the barriers of this turn of fb
            // accumulators me, me + 2 (FEW) or both (MANY) handed to the epilogue and not seen back,
            // and the parity of their next return
            uint32_t few_out = 0, few_ph = 0, pair_out = 0, pair_ph = 0;
            bool ok = true;
            const auto few_back = [&](int h) {
                if (!(few_out >> h & 1)) return;
                ok = ok && wait_bounded(bar(kAccEmpty + me + 2 * h), few_ph >> h & 1, abort_word);
                few_out &= ~(1u << h);
                few_ph ^= 1u << h;
            };
            const auto pair_back = [&]() {
                if (!pair_out) return;
                ok = ok && wait_bounded(bar(kPairEmpty + me), pair_ph, abort_word);
                pair_out = 0;
                pair_ph ^= 1;
            };
            const uint32_t idesc_full = make_idesc(128, kCols, false, F8);
            for (int ic = 0;; ++ic) {
                Item I;
                if (!next_item(ic, I)) break;
                const int set = ic & 1;
                const bool few = I.n_qt == 1;
                const uint64_t stay = make_sdesc(sb + kStay + set * 2 * kSlot, 16, 1024);
                if (!(ok = wait_bounded(bar(kStayUse + set), (ic >> 1) & 1, abort_word))) break;
                const int end = n + (few ? I.nt : I.n_qt - I.qt0);
                const int last_cols = (I.n_q - ((I.n_qt - 1) << log2qt)) * p.g;
                const uint32_t idesc_last = make_idesc(128, (last_cols + 15) & ~15, false, F8);
                for (; n < end; ++n) {
                    if ((n & 1) == me) {
                        const uint64_t stage = make_sdesc(sb + stage_at(st), 16, 1024);
                        pair_back();
                        if (few) {
                            const int h = n >> 1 & 1, acc = n & 3;
                            few_back(h);
                            if (!ok || !(ok = wait_bounded(bar(kStreamUse + fb), ph, abort_word)))
                                break;
                            tc_fence_after();
                            issue_s_group<D>(1u, tmem + acc * kCols, stage, stay, idesc_last);
                            tc_commit_if(1u, bar(kAccFull + acc));
                            few_out |= 1u << h;
                        } else {
                            const uint32_t idesc = n + 1 == end ? idesc_last : idesc_full;
                            few_back(0);
                            few_back(1);
                            if (!ok || !(ok = wait_bounded(bar(kStreamUse + fb), ph, abort_word)))
                                break;
                            tc_fence_after();
                            issue_s_group<D>(1u, tmem + me * kCols, stay, stage, idesc);
                            if (I.nt == 2)
                                issue_s_group<D>(1u, tmem + (me + 2) * kCols, stay + (kSlot >> 4),
                                                 stage, idesc);
                            tc_commit_if(1u, bar(kPairFull + me));
                            pair_out = 1;
                        }
                        tc_commit_if(1u, bar(kStreamEmpty + st));
                    }
                    if (++st == n_stages) st = 0;
                    if (++fb == 2 * n_stages) {
                        fb = 0;
                        ph ^= 1;
                    }
                }
                if (!ok) break;
                tc_commit_if(1u, bar(kStayEmpty + set));
            }
            // every MMA has finished before TMEM is released
            tc_commit_if(1u, bar(kDrain + me));
            wait_drain(bar(kDrain + me), 0);
        }
    } else if (warp == 18) {
        // ------------------------------------------------ loader of what streams
        int st = 0, fb = 0, ph = 1, n_done = 0, ok = 1;   // a fresh barrier's phase 1 counts as past
        const int per_tile = kTileKeys >> log2bs, per_load = 32 / per_tile;   // blocks; tiles
        for (int ic = 0; ok; ++ic) {
            Item I;
            ok = next_item(ic, I);
            if (!__all_sync(0xffffffffu, ok)) break;
            const bool few = I.n_qt == 1;
            const int n = few ? I.nt : I.n_qt - I.qt0, end = I.t0 + I.nt;
            // the lanes hold the blocks of per_load tiles, and those of the next ones on their way
            int ids = -1, next = few ? block_id(I, I.t0, end) : -1;
            for (int i = 0; i < n; ++i) {
                const int at = i & (per_load - 1);
                if (few && at == 0) {
                    ids = next;
                    next = i + per_load < n ? block_id(I, I.t0 + i + per_load, end) : -1;
                }
                if (lane == 0) ok = wait_bounded(bar(kStreamEmpty + st), ph, abort_word);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                const uint32_t slot = sb + stage_at(st), full = bar(kStreamFull + fb);
                if (few) {
                    const int nblk = blocks_of(I, I.t0 + i);
                    const int id = __shfl_sync(0xffffffffu, ids, (at * per_tile + lane) & 31);
                    if (lane == 0) mbar_expect_tx(full, k_bytes(nblk));
                    __syncwarp();
                    load_k(slot, full, I, nblk, id);
                } else if (lane == 0) {
                    load_q(slot, full, I, I.qt0 + i);
                }
                ++n_done;
                if (++fb == 2 * n_stages) fb = 0;
                if (++st == n_stages) {
                    st = 0;
                    ph ^= 1;
                }
            }
        }
        if (lane == 0) {
            // never leave with copies in flight into this CTA's shared memory
            for (int i = max(0, n_done - n_stages); i < n_done; ++i)
                wait_drain(bar(kStreamFull + i % (2 * n_stages)), (i / (2 * n_stages)) & 1);
        }
    } else if (warp == 19) {
        // ------------------------------------------------ log-sum-exps, negated, in base 2
        int n_done = 0, ok = 1;
        for (int ic = 0; ok; ++ic) {
            Item I;
            ok = next_item(ic, I);
            if (!__all_sync(0xffffffffu, ok)) break;
            const auto fetch = [&](int qt) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int col = 4 * lane + e;
                    const int tok = (qt << log2qt) + (col >> (7 - log2qt));
                    v[e] = 0.f;
                    if (tok < I.n_q)
                        v[e] = -1.4426950408889634f *
                               __ldg(p.lse + int64_t(I.cu0 + tok) * p.Hq + I.kvh * p.g +
                                     (col & (p.g - 1)));
                }
                return make_float4(v[0], v[1], v[2], v[3]);
            };
            float4 next = fetch(I.qt0);
            for (int qt = I.qt0; qt < I.n_qt; ++qt, ++n_done) {
                const float4 v = next;
                if (qt + 1 < I.n_qt) next = fetch(qt + 1);
                const int slot = n_done % kLseSlots;
                if (lane == 0 && n_done >= kLseSlots)
                    ok = wait_bounded(bar(kLseEmpty + slot), (n_done / kLseSlots - 1) & 1,
                                      abort_word);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                float* to = reinterpret_cast<float*>(smem + kCtl + kLseOff) + slot * 128;
                *reinterpret_cast<float2*>(to + lse_place(4 * lane)) = make_float2(v.x, v.y);
                *reinterpret_cast<float2*>(to + lse_place(4 * lane + 2)) = make_float2(v.z, v.w);
                mbar_arrive(bar(kLseFull + slot));
            }
        }
    } else if (warp >= kTurners) {
        // ------------------------------------------------ codes and q to f16 (fp8 cache)
        if constexpr (F8) {
            const int w = warp - kTurners;
            // the MMAs take f16 operands: 32 rows a warp of a K tile's codes are expanded, or of a
            // query tile rounded in place (a 16-byte chunk keeps its place, so the swizzle holds)
            const auto turn_k = [&](uint32_t slot, const Item& I, int t) {
                const int rows =
                    ((min(kTileKeys, I.ctx - t * kTileKeys) + p.bs - 1) >> log2bs) << log2bs;
                expand_rows(slot, 32 * w, rows, lane);
            };
            const auto turn_q = [&](uint32_t slot, int rows) {
                for (int i = threadIdx.x - kBaseThreads; i < rows * 16; i += 128) {
                    const uint32_t a = slot + ((i >> 3) & 1) * kHalf + (i >> 4) * 128 + (i & 7) * 16;
                    const uint4 v = ld_shared_v4(a);
                    st_shared_v4(a, bf16x2_to_f16x2(v.x), bf16x2_to_f16x2(v.y),
                                 bf16x2_to_f16x2(v.z), bf16x2_to_f16x2(v.w));
                }
            };
            int st = 0, fb = 0, ph = 0;
            bool ok = true;
            for (int ic = 0; ok; ++ic) {
                Item I;
                if (!next_item(ic, I)) break;
                const bool few = I.n_qt == 1;
                const int set = ic & 1;
                const uint32_t stay = sb + kStay + set * 2 * kSlot;
                if (!(ok = wait_bounded(bar(kStayFull + set), (ic >> 1) & 1, abort_word))) break;
                if (few) turn_q(stay, I.n_q == 1 ? p.g : kCols);
                else
                    for (int r = 0; r < I.nt; ++r) turn_k(stay + r * kSlot, I, I.t0 + r);
                fence_proxy_async();
                mbar_arrive(bar(kStayReady + set));
                const int n = few ? I.nt : I.n_qt - I.qt0;
                for (int i = 0; i < n; ++i) {
                    if (!(ok = wait_bounded(bar(kStreamFull + fb), ph, abort_word))) break;
                    const uint32_t slot = sb + stage_at(st);
                    if (few) turn_k(slot, I, I.t0 + i);
                    else turn_q(slot, kCols);
                    fence_proxy_async();
                    mbar_arrive(bar(kStreamReady + fb));
                    if (++st == n_stages) st = 0;
                    if (++fb == 2 * n_stages) {
                        fb = 0;
                        ph ^= 1;
                    }
                }
            }
        }
    } else {
        // ------------------------------------------------ epilogue warpgroups
        const int w = warp >> 2;             // FEW: accumulator w; MANY: the pair's key tile w >> 1,
                                             // columns 64 (w & 1) .. + 63
        const uint32_t tm = tmem + (uint32_t(32 * (warp & 3)) << 16);
        const int q4 = lane & 3, rs = lane >> 2;
        // after the sums over the four threads of a key have met, thread q4 has key rs + 8 q4
        const int key_in_tile = 32 * (warp & 3) + rs + 8 * q4;
        const uint64_t c2 = f2(p.c, p.c);
        int n = 0, few_ph = 0, pair_ph = 0, n_lse = 0, n_part = 0;
        bool ok = true;
        const float4* lse_smem = reinterpret_cast<const float4*>(smem + kCtl + kLseOff) + q4;
        float* part = reinterpret_cast<float*>(smem + kCtl + kPartOff) + (w >> 1) * 128;
        uint64_t a[4];                       // the thread's part of its four keys' sums
        const auto clear = [&]() {
#pragma unroll
            for (int k = 0; k < 4; ++k) a[k] = f2(0.f, 0.f);
        };
        // adds columns c0 .. c1 - 1 of the accumulator at ta: query rows from position `at` on, the
        // warp's keys from `kw` on; `empty` takes the accumulator back
        const auto add_columns = [&](uint32_t ta, const float4* nl, int c0, int c1, int at, int kw,
                                     uint32_t empty) {
            tc_fence_after();
            if (c1 - c0 == 64 && kw + 31 <= at) {
                ta += c0;
                nl += c0 / 4;
                uint32_t lo0[8], hi0[8], lo1[8], hi1[8];
                tmem_ld_16x256b_x2(ta, lo0);
                tmem_ld_16x256b_x2(ta + (16u << 16), hi0);
#pragma unroll
                for (int c = 0; c < 64; c += 32) {
                    tmem_wait_ld();
                    tmem_ld_16x256b_x2(ta + c + 16, lo1);
                    tmem_ld_16x256b_x2(ta + c + 16 + (16u << 16), hi1);
                    add16(lo0, hi0, nl[c / 4], c2, a);
                    tmem_wait_ld();
                    if (c + 32 < 64) {
                        tmem_ld_16x256b_x2(ta + c + 32, lo0);
                        tmem_ld_16x256b_x2(ta + c + 32 + (16u << 16), hi0);
                    } else {
                        tc_fence_before();
                        mbar_arrive(empty);
                    }
                    add16(lo1, hi1, nl[c / 4 + 4], c2, a);
                }
                return;
            }
            for (int c = c0; c < c1; c += 16) {
                uint32_t lo[8], hi[8];
                tmem_ld_16x256b_x2(ta + c, lo);
                tmem_ld_16x256b_x2(ta + c + (16u << 16), hi);
                const float4 l = nl[c / 4];
                const float nv[4] = {l.x, l.y, l.z, l.w};
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    // the first column whose row comes at or after the key
                    const int from = max(0, kw + rs + 8 * k - at) << (7 - log2qt);
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) {
                        const uint32_t* s = (k < 2 ? lo : hi) + 4 * cc + 2 * (k & 1);
                        float e[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int col = c + 8 * cc + 2 * q4 + i;
                            const float x = ex2(fmaf(__uint_as_float(s[i]), p.c, nv[2 * cc + i]));
                            e[i] = col >= from && col < c1 ? x : 0.f;
                        }
                        a[k] = add2(a[k], f2(e[0], e[1]));
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(empty);
        };
        // the sum of key key_in_tile
        const auto total_of_key = [&]() {
            float mine = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float x0, x1;
                f2_split(a[k], x0, x1);
                float x = x0 + x1;
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                if (q4 == k) mine = x;
            }
            return mine;
        };
        for (int ic = 0; ok; ++ic) {
            Item I;
            if (!next_item(ic, I)) break;
            const auto wait_lse = [&]() {
                return ok = wait_bounded(bar(kLseFull + n_lse % kLseSlots), (n_lse / kLseSlots) & 1,
                                         abort_word);
            };
            const auto done_lse = [&]() { mbar_arrive(bar(kLseEmpty + n_lse++ % kLseSlots)); };
            if (I.n_qt == 1) {
                if (!wait_lse()) break;
                const float4* nl = lse_smem + (n_lse % kLseSlots) * 32;
                // the item's first tile of this warpgroup, then every fourth
                for (int i = (w - n) & 3; i < I.nt; i += 4) {
                    const int kb = (I.t0 + i) * kTileKeys, j = kb + key_in_tile;
                    float* dst = p.weights + I.state + j;
                    const float old = j < I.held ? *dst : 0.f;
                    if (!(ok = wait_bounded(bar(kAccFull + w), few_ph, abort_word))) break;
                    few_ph ^= 1;
                    clear();
                    add_columns(tm + w * kCols, nl, 0, I.n_q * p.g, I.pos0, kb + 32 * (warp & 3),
                                bar(kAccEmpty + w));
                    const float sum = total_of_key();
                    if (j < I.ctx) *dst = old + sum;
                }
                if (!ok) break;
                n += I.nt;
                done_lse();
                continue;
            }
            const int r = w >> 1, c0 = 64 * (w & 1);
            const bool my = r < I.nt;
            const int kb = (I.t0 + r) * kTileKeys, j = kb + key_in_tile;
            float* dst = p.weights + I.state + j;
            const float old = my && !(w & 1) && j < I.held ? *dst : 0.f;
            clear();
            for (int qt = I.qt0; qt < I.n_qt; ++qt, ++n) {
                if (!wait_lse()) break;
                const int pair = n & 1;
                if (!(ok = wait_bounded(bar(kPairFull + pair), pair_ph >> pair & 1, abort_word)))
                    break;
                pair_ph ^= 1 << pair;
                const int c1 = min(c0 + 64, (I.n_q - (qt << log2qt)) * p.g);
                if (my && c0 < c1)
                    add_columns(tm + (pair + 2 * r) * kCols, lse_smem + (n_lse % kLseSlots) * 32, c0,
                                c1, I.pos0 + (qt << log2qt), kb + 32 * (warp & 3),
                                bar(kPairEmpty + pair));
                else
                    mbar_arrive(bar(kPairEmpty + pair));
                done_lse();
            }
            if (!ok) break;
            if (!my) continue;
            const float sum = total_of_key();
            if (w & 1) {
                if (n_part > 0 &&
                    !(ok = wait_bounded(bar(kPartEmpty + r), (n_part - 1) & 1, abort_word)))
                    break;
                part[key_in_tile] = sum;
                mbar_arrive(bar(kPartFull + r));
            } else {
                if (!(ok = wait_bounded(bar(kPartFull + r), n_part & 1, abort_word))) break;
                const float all = sum + part[key_in_tile];
                mbar_arrive(bar(kPartEmpty + r));
                if (j < I.ctx) *dst = old + all;
            }
            ++n_part;
        }
    }
    if (*abort_word && threadIdx.x == 0 && p.err) atomicOr(p.err, PA_DEVERR_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == 17) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                     : "memory");
    }
}

constexpr int kMaxDevices = 64;

template <int D, bool F8>
int32_t launch_weights(const CUtensorMap& k, const CUtensorMap& q1, const CUtensorMap& qn,
                       const Params& p, cudaStream_t stream) {
    int dev = 0;
    int32_t st = note_cuda(cudaGetDevice(&dev));
    if (st) return st;
    // the shared-memory limit is raised once per device (idempotent: threads may race to it)
    static std::atomic<bool> raised[kMaxDevices];
    if (dev < 0 || dev >= kMaxDevices) return PA_ERR_INVALID;
    if (!raised[dev].load(std::memory_order_acquire)) {
        if ((st = note_cuda(cudaFuncSetAttribute(attn_weights_kernel<D, F8>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 kBytes))))
            return st;
        raised[dev].store(true, std::memory_order_release);
    }
    const int64_t tiles =
        int64_t(p.B) * p.Hkv * ((int64_t(p.max_len) + kTileKeys - 1) / kTileKeys);
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(std::min<int64_t>(tiles, PA_PLAN_CTAS)));
    cfg.blockDim = dim3(kThreadsFor<F8>);
    cfg.dynamicSmemBytes = kBytes;
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return note_cuda(cudaLaunchKernelEx(&cfg, attn_weights_kernel<D, F8>, k, q1, qn, p));
}

// ------------------------------------------------ decode rows of a step that kept their scores
// One thread per four keys of a (sequence, KV head): the group's raw scores, stored by the
// attention kernel, against the rows' log-sum-exps. A decode step so pays 4 g bytes per key and
// KV head written and read again (in L2, mostly) in place of a second read of K's 2 D.
constexpr int kDecodeKeys = 1024;      // per block of 256 threads
__global__ void __launch_bounds__(256)
    decode_weights_kernel(const float* __restrict__ scores, int64_t scores_ld, const Params p) {
    __shared__ float nl[16];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int s = int(blockIdx.z), h = int(blockIdx.y);
    const int c0 = p.cu[s], ctx = p.ctx[s];
    const int row = p.rows ? p.rows[s] : s;
    const int j0 = int(blockIdx.x) * kDecodeKeys;
    if (p.cu[s + 1] - c0 != 1 || row < 0 || (j0 >= ctx && j0 > 0)) return;
    const int held = p.held ? p.held[s] : ctx - 1;
    bool bad = c0 < 0 || c0 >= p.T || ctx < 1 || ctx > p.max_len || ctx > scores_ld ||
               (int64_t(ctx) + p.bs - 1) / p.bs > p.max_blocks || row >= p.n_rows || held < 0 ||
               held > ctx;
    if (p.rows)
        for (int i = threadIdx.x; i < p.B; i += 256)
            bad = bad || (i != s && p.rows[i] == row && p.cu[i + 1] != p.cu[i]);
    if (threadIdx.x < p.g)
        nl[threadIdx.x] = bad ? 0.f
                              : -1.4426950408889634f *
                                    p.lse[int64_t(c0) * p.Hq + h * p.g + threadIdx.x];
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0 && j0 == 0 && h == 0 && p.err) atomicOr(p.err, PA_DEVERR_META);
        return;
    }
    const int j = j0 + 4 * int(threadIdx.x);
    if (j >= ctx) return;
    // scores_ld is a multiple of 128: a thread's four lie within the row
    const float* sc = scores + (int64_t(s) * p.Hq + h * p.g) * scores_ld + j;
    float* w = p.weights + (int64_t(row) * p.Hkv + h) * p.max_len + j;
    float sum[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = j + e < held ? w[e] : 0.f;
    for (int i = 0; i < p.g; ++i) {
        const float4 x = __ldcs(reinterpret_cast<const float4*>(sc + int64_t(i) * scores_ld));
        sum[0] += ex2(fmaf(x.x, p.c, nl[i]));
        sum[1] += ex2(fmaf(x.y, p.c, nl[i]));
        sum[2] += ex2(fmaf(x.z, p.c, nl[i]));
        sum[3] += ex2(fmaf(x.w, p.c, nl[i]));
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (j + e < ctx) w[e] = sum[e];
}

// Scores kept for a step: rows of a whole number of tiles.
int64_t scores_row(int32_t max_ctx) {
    return (int64_t(max_ctx) + kTileKeys - 1) / kTileKeys * kTileKeys;
}
size_t partials_bytes(const pa_shape* s, int32_t T, int32_t max_ctx) {
    return (pa_workspace_bytes(s, T, max_ctx) + 255) & ~size_t(255);
}

int32_t attention_weights(const void* q, const void* k_pool, const float* lse,
                          const int32_t* block_table, int32_t max_blocks, const int32_t* cu,
                          const int32_t* ctx, int32_t B, int32_t T, const int32_t* held,
                          const int32_t* rows, float* weights, int32_t n_rows, int32_t max_len,
                          bool fp8, float k_scale, const pa_shape* s, int32_t* err,
                          cudaStream_t stream, const float* scores = nullptr,
                          int32_t max_ctx = 0) {
    int32_t st = check_shape(s);
    if (st) return st;
    if (fp8 && s->head_dim != 128) return PA_ERR_SHAPE;
    if (B < 0 || T < 0 || max_blocks < 0 || n_rows < 0 || max_len < 0) return PA_ERR_INVALID;
    if (T == 0 || B == 0) return PA_OK;
    if (!q || !k_pool || !lse || !block_table || !cu || !ctx || !weights) return PA_ERR_INVALID;
    if (max_len == 0 || (!rows && n_rows < B)) return PA_ERR_INVALID;
    if (n_rows > kMaxRows || int64_t(s->num_blocks) * s->block_size > INT32_MAX ||
        max_len > INT32_MAX - kTileKeys)
        return PA_ERR_SHAPE;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_pool)) & 15)
        return PA_ERR_INVALID;
    const int D = s->head_dim, g = s->num_q_heads / s->num_kv_heads;
    const int64_t slots = int64_t(s->num_blocks) * s->block_size;
    CUtensorMap k, q1, qn;
    st = fp8 ? make_map_codes(&k, k_pool, D, s->num_kv_heads, slots, s->block_size)
             : make_map(&k, k_pool, D, s->num_kv_heads, slots, 1, s->block_size);
    if (st) return st;
    if ((st = make_map(&q1, q, D, s->num_q_heads, T, g, 1))) return st;
    if ((st = make_map(&qn, q, D, s->num_q_heads, T, g, kCols / g))) return st;
    Params p;
    p.lse = lse;
    p.block_table = block_table;
    p.cu = cu;
    p.ctx = ctx;
    p.held = held;
    p.rows = rows;
    p.weights = weights;
    p.err = err;
    p.B = B;
    p.T = T;
    p.max_blocks = max_blocks;
    p.Hq = s->num_q_heads;
    p.Hkv = s->num_kv_heads;
    p.g = g;
    p.bs = s->block_size;
    p.num_blocks = s->num_blocks;
    p.n_rows = n_rows;
    p.max_len = max_len;
    p.c = float(1.4426950408889634 / std::sqrt(double(D))) * k_scale;
    p.skip_decode = scores != nullptr;
    if (scores) {
        cudaLaunchAttribute pdl[1];
        pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        pdl[0].val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(unsigned((max_ctx + kDecodeKeys - 1) / kDecodeKeys), unsigned(p.Hkv),
                           unsigned(B));
        cfg.blockDim = dim3(256);
        cfg.stream = stream;
        cfg.attrs = pdl;
        cfg.numAttrs = 1;
        if ((st = note_cuda(cudaLaunchKernelEx(&cfg, decode_weights_kernel, scores,
                                               scores_row(max_ctx), p))))
            return st;
    }
    if (fp8) return launch_weights<128, true>(k, q1, qn, p, stream);
    if (D == 128) return launch_weights<128, false>(k, q1, qn, p, stream);
    return launch_weights<64, false>(k, q1, qn, p, stream);
}

}  // namespace

extern "C" int32_t paged_attention_weights(
    const void* q, const void* k_pool, const float* lse, const int32_t* block_table,
    int32_t max_blocks, const int32_t* cu_seqlens_q, const int32_t* ctx_lens, int32_t B,
    int32_t T, const int32_t* held, const int32_t* rows, float* weights, int32_t n_rows,
    int32_t max_len, const pa_shape* shape, int32_t* err_flag, pa_stream_t stream) {
    return attention_weights(q, k_pool, lse, block_table, max_blocks, cu_seqlens_q, ctx_lens, B, T,
                             held, rows, weights, n_rows, max_len, false, 1.f, shape, err_flag,
                             stream);
}

extern "C" int32_t paged_attention_weights_fp8(
    const void* q, const void* k_pool, const float* lse, const int32_t* block_table,
    int32_t max_blocks, const int32_t* cu_seqlens_q, const int32_t* ctx_lens, int32_t B,
    int32_t T, const int32_t* held, const int32_t* rows, float* weights, int32_t n_rows,
    int32_t max_len, float k_scale, const pa_shape* shape, int32_t* err_flag,
    pa_stream_t stream) {
    if (!(k_scale > 0.f) || !(k_scale < INFINITY)) return PA_ERR_INVALID;
    return attention_weights(q, k_pool, lse, block_table, max_blocks, cu_seqlens_q, ctx_lens, B, T,
                             held, rows, weights, n_rows, max_len, true, k_scale, shape, err_flag,
                             stream);
}

// ------------------------------------------------ the step of a bounded cache
namespace {

int32_t step_weights(const void* q, const void* k_pool, const void* v_pool,
                     const int32_t* block_table, int32_t max_blocks, const int32_t* cu,
                     const int32_t* ctx, int32_t B, int32_t T, int32_t max_ctx,
                     const pa_work_item* items, int32_t n_items, bool fp8, float k_scale,
                     float v_scale, void* workspace, size_t ws_bytes, void* out, float* lse,
                     const int32_t* held, const int32_t* rows, float* weights, int32_t n_rows,
                     int32_t max_len, const pa_shape* s, int32_t* err, cudaStream_t stream) {
    int32_t st = check_shape(s);
    if (st) return st;
    if (B < 0 || T < 0 || n_items < 0 || max_ctx < 0) return PA_ERR_INVALID;
    if (T == 0 || B == 0 || n_items == 0) return PA_OK;
    // both halves' checks come before either launches
    if (!q || !k_pool || !v_pool || !block_table || !cu || !ctx || !items || !out || !lse ||
        !weights || max_len <= 0 || max_ctx == 0 || n_rows < 0 || (!rows && n_rows < B))
        return PA_ERR_INVALID;
    if (B > 65535 || s->num_kv_heads > 65535 || n_rows > kMaxRows ||
        max_len > INT32_MAX - kTileKeys || max_ctx > INT32_MAX - kTileKeys ||
        int64_t(s->num_blocks) * s->block_size > INT32_MAX)
        return PA_ERR_SHAPE;
    if (!workspace || ws_bytes < pa_step_weights_workspace_bytes(s, B, T, max_ctx))
        return PA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 15) return PA_ERR_INVALID;
    float* scores = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                             partials_bytes(s, T, max_ctx));
    if ((st = attention_step_stats(q, k_pool, v_pool, block_table, max_blocks, cu, ctx, B, T,
                                   max_ctx, items, n_items, fp8, k_scale, v_scale, workspace,
                                   ws_bytes, out, lse, scores, scores_row(max_ctx), s, err,
                                   stream)))
        return st;
    return attention_weights(q, k_pool, lse, block_table, max_blocks, cu, ctx, B, T, held, rows,
                             weights, n_rows, max_len, fp8, k_scale, s, err, stream, scores,
                             max_ctx);
}

}  // namespace

extern "C" size_t pa_step_weights_workspace_bytes(const pa_shape* shape, int32_t B, int32_t T,
                                                  int32_t max_ctx) {
    if (check_shape(shape) || B < 0 || T < 0 || max_ctx < 0) return 0;
    return partials_bytes(shape, T, max_ctx) +
           size_t(B) * shape->num_q_heads * size_t(scores_row(max_ctx)) * sizeof(float);
}

extern "C" int32_t paged_attention_step_weights(
    const void* q, const void* k_pool, const void* v_pool, const int32_t* block_table,
    int32_t max_blocks, const int32_t* cu_seqlens_q, const int32_t* ctx_lens, int32_t B,
    int32_t T, int32_t max_ctx, const pa_work_item* items, int32_t n_items, void* workspace,
    size_t ws_bytes, void* out, float* lse, const int32_t* held, const int32_t* rows,
    float* weights, int32_t n_rows, int32_t max_len, const pa_shape* shape, int32_t* err_flag,
    pa_stream_t stream) {
    return step_weights(q, k_pool, v_pool, block_table, max_blocks, cu_seqlens_q, ctx_lens, B, T,
                        max_ctx, items, n_items, false, 1.f, 1.f, workspace, ws_bytes, out, lse,
                        held, rows, weights, n_rows, max_len, shape, err_flag, stream);
}

extern "C" int32_t paged_attention_step_weights_fp8(
    const void* q, const void* k_pool, const void* v_pool, const int32_t* block_table,
    int32_t max_blocks, const int32_t* cu_seqlens_q, const int32_t* ctx_lens, int32_t B,
    int32_t T, int32_t max_ctx, const pa_work_item* items, int32_t n_items, float k_scale,
    float v_scale, void* workspace, size_t ws_bytes, void* out, float* lse, const int32_t* held,
    const int32_t* rows, float* weights, int32_t n_rows, int32_t max_len, const pa_shape* shape,
    int32_t* err_flag, pa_stream_t stream) {
    if (!(k_scale > 0.f) || !(v_scale > 0.f) || !(k_scale < INFINITY) || !(v_scale < INFINITY))
        return PA_ERR_INVALID;
    if (shape && shape->head_dim != 128) return PA_ERR_SHAPE;
    return step_weights(q, k_pool, v_pool, block_table, max_blocks, cu_seqlens_q, ctx_lens, B, T,
                        max_ctx, items, n_items, true, k_scale, v_scale, workspace, ws_bytes, out,
                        lse, held, rows, weights, n_rows, max_len, shape, err_flag, stream);
}
