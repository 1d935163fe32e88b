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
//   MANY  a prefill chunk: up to four key tiles stay, query tiles (128 columns) stream past them
//         from L2. Bound by each accumulator's chain (product, read, hand back): the tensor pipe and
//         the exponentials (per element one fused multiply-add and one addition, packed in pairs,
//         and one ex2) are each busy two thirds of the time. With two key tiles staying, the 32 KB a
//         query tile takes out of L2 for each of their products was what bound it.
// Work is dealt by cost, on the device, to groups of CTAs, one for each of 8 (4, 2, 1) neighbouring
// KV heads: every (sequence, heads, key tile) in order has a cost (kCostFew for a FEW tile, kCostMany
// for each query tile a MANY tile meets), a group takes the tiles that start in its share of the
// total. The heads of a token lie side by side in memory; read at about the same time, whole rows of
// DRAM are used. No plan is made or uploaded, so a captured graph needs nothing renewed but its
// metadata.
//
// Warps: 0-15 four epilogue warpgroups, 16 scheduler and loader of what stays, 17 and 19 MMA issuers,
// 18 loader of what streams; over an fp8 cache 20-23 turn codes and q to f16. There are four
// accumulators of 128 TMEM columns, warpgroup w reads accumulator w: FEW's stream tiles take them in
// turn, a MANY item's key tile r has accumulator r; with two key tiles the query tiles alternate
// between accumulators r and r + 2, with one they take all four in turn, and the sums meet in memory
// at the item's end. A key's sum is the same whichever way its tile came to be taken: query tiles are
// summed in four classes (qt % 4), these are added up in the order 0, 2, 1, 3, and the old sum joins
// last, in one rounding (a class may be below half a step of a large old sum).
// Issuer i fills accumulators i and i + 2: its waits, commits and address arithmetic, made slow by the
// warps it shares its scheduler with, run while the other's MMAs keep the tensor pipe busy (strict
// turns of the two, 0, 1, 2, 3, were slower: 92 us where the chunks below then took 87).
// Shared memory: seven 32 KB slots. Four in a ring for what stays (the next item's tiles load as this
// one's are done with) and three stages for what streams; where no sequence is MANY, two for what
// stays and five stages (five tiles of K in flight). Every wait is bounded.
//
// Measured (8 KV heads of 128, group 4): 64 decode rows at 2k .. 16k keys 93 us, 5.6 TB/s, 82 % of the
// measured copy rate; one at 16,001 keys 11.7 us (some 7 of them up to the first tile: launch,
// metadata, deal, first loads); four chunks of 512 rows at up to 9,512 keys 84 us, 1.03 PFLOP/s, 54 %
// of the measured matrix rate; 32 decode rows at up to 40,000 keys over an fp8 cache (group 8) 50 us, 4.05
// TB/s, 60 % (its 16 KB tiles leave half the bytes in flight; with no expansion at all it took 46.6).
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

constexpr int kBaseThreads = 640;
constexpr int kTurnWarps = 4;                  // turn an fp8 cache's codes, 32 rows of a tile each
template <bool F8>
constexpr int kThreadsFor = F8 ? kBaseThreads + 32 * kTurnWarps : kBaseThreads;
constexpr int kTurners = kBaseThreads / 32;    // the first f16 warp of an fp8 cache
constexpr int kCols = 128;                     // columns of a query tile
constexpr int kSlot = 32768;                   // one tile, 128 rows of D = 128
constexpr int kHalf = 16384;                   // its 64-column halves
constexpr int kMaxStages = 5;
constexpr int kCtl = 7 * kSlot;
constexpr int kCtlBytes = 3 * 1024;            // barriers, items, log-sum-exps
constexpr int kBytes = kCtl + kCtlBytes;
static_assert(kBytes <= 227 * 1024, "shared memory of one CTA");
constexpr int kMaxRows = 1 << 18;              // state rows whose repeats are looked for
constexpr int kMaxLen = INT32_MAX - 32 * 128;  // keys: a warp's 32 blocks more are counted in 32 bits
constexpr int kMaxSeqs = 8192;                 // sequences whose costs are held while they are dealt
// before the pipeline starts: a bit per state row in slot 0 (named) and in slot 6 (named again), the
// first sequences' metadata from slot 1, a cost per sequence from slot 4
constexpr int kMeta = kSlot, kCosts = 4 * kSlot, kAgain = 6 * kSlot;
constexpr int kMetaSeqs = 3 * kSlot / 32;
static_assert(kMaxRows / 8 <= kSlot && kMaxSeqs * 8 <= 2 * kSlot, "scratch of the deal");
constexpr int64_t kShared = -1;                // cost of a sequence whose state row another one names
// Cost of a key tile, and of a key tile and query tile. Their ratio counts in a batch with both kinds
// alone, and it weighs streamed keys too heavily there: 48 decode rows at 2k .. 16k keys beside four
// 512-row chunks (32 / 8 heads of 128) take 261 us, the two kinds by themselves 151 and 87; with 5 : 3
// 231, 5 : 4 246, 5 : 1 443. Over an e4m3 cache 288 (5 : 3 236, 5 : 4 241), head_dim 64 244 (192, 180).
constexpr int64_t kCostFew = 5, kCostMany = 2;

// A role that waits on a barrier waits for each of its phases in turn: parity tells only neighbours
// apart. Warps arrive once, not 32 times.
enum Bar {
    kStayFull = 0,     // + slot: TMA -> issuers (or the f16 warps)
    kStayEmpty = 4,    // + slot: both issuers -> loader
    kStreamFull = 8,   // + stage: TMA -> issuers (or the f16 warps)
    kStreamEmpty = 13, // + stage: both issuers -> loader
    kAccFull = 18,     // + accumulator: its issuer -> its warpgroup
    kAccEmpty = 22,    // + accumulator: 4 arrivals -> its issuer
    kLseFull = 26,     // + slot (4), MANY: the stream's loader -> the warpgroups
    kLseEmpty = 30,    // + slot, MANY: 16 arrivals
    kItemFull = 34,    // + slot (4)
    kItemEmpty = 38,   // + slot: every consumer warp
    kPartDone = 42,    // + key tile of two: 4 arrivals, warpgroup r -> r + 2
    kPartSeen = 44,    // + key tile of two: 4 arrivals, r + 2 -> r: it has read the old sum
    kChainDone = 46,   // + place, one key tile: 4 arrivals, a warpgroup -> the next
    kChainSeen = 49,   // one key tile: 4 arrivals, the last -> the first: it has read the old sum
    kDrain = 50,       // + issuer
    kStayReady = 52,   // + slot, fp8 only: the f16 warps
    kStreamReady = 56, // + stage
    kNumBars = 61
};
constexpr int kHolderOff = 8 * kNumBars;
constexpr int kAbortOff = kHolderOff + 4;
constexpr int kRingOff = 512;                  // 4 items of 64 bytes
constexpr int kLseOff = kRingOff + 4 * 64;     // MANY: 4 x 128 log-sum-exps
constexpr int kTwiceOff = kLseOff + 4 * 512;   // whether some state row is named twice
static_assert(kAbortOff + 4 <= kRingOff && kTwiceOff + 4 <= kCtlBytes, "control area");

// A bounded wait. Twenty warps wait here, the issuers among them; with 32 polls at a time in place of 4
// their polling cost 512-row chunks 90.3 us instead of 87.0, and a decode batch 94.0 instead of 92.7
// (one poll at a time: 86.6 and 92.7, but an fp8 tail 51.3 instead of 50.9).
__device__ __forceinline__ bool await(uint32_t bar, uint32_t parity, volatile int* abort_word) {
    return wait_bounded<4>(bar, parity, abort_word);
}

// Slots of stage st of the stream, and of tile k of what stays.
__device__ __forceinline__ uint32_t stage_at(int st) {
    return uint32_t(st < 3 ? 4 + st : st == 3 ? 1 : 3) * kSlot;
}
__device__ __forceinline__ uint32_t stay_at(int s, int n_stay) {
    return uint32_t(n_stay == 4 ? s : 2 * s) * kSlot;
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
    int32_t heads;               // CTAs of a group: neighbouring KV heads
    int32_t skip_decode;         // sequences of one row are another kernel's
    int32_t max_ctx;             // a step's bound: rows of longer contexts may have no lse
    float c;                     // log2(e) / sqrt(D), times the K scale of an fp8 cache
};

// What the sequences' metadata says, checked. cost 0: nothing to do (no rows, no state row, or
// metadata that does not fit, which sets bad).
struct Seq {
    int n_q, ctx, pos0, cu0, row, held;
    bool any;                    // it has query rows
    int n_tiles, n_qt;           // key tiles; query tiles
    bool few, bad;
    int64_t head_cost;
};

// Query tiles that key tile t does not meet: their rows all come before it.
__device__ __forceinline__ int first_qt(const Seq& q, int t, int log2qt) {
    return max(0, t * kTileKeys - q.pos0) >> log2qt;
}

// Cost of a head's key tiles before tile t: a tile costs the query tiles that the first of its four
// meets (an item passes all of them by its four tiles).
__device__ __forceinline__ int64_t cost_before(const Seq& q, int t, int log2qt) {
    if (q.few) return kCostFew * t;
    // tiles up to u meet every query tile
    const int u = min(t, ((q.pos0 + (1 << log2qt) - 1) / kTileKeys + 4) & ~3);
    int64_t f = int64_t(u) * q.n_qt;
    for (int i = u; i < t; ++i) f += q.n_qt - first_qt(q, i & ~3, log2qt);
    return kCostMany * f;
}

// Quotients of costs: nearly always of 32 bits.
__device__ __noinline__ int64_t quot_64(int64_t a, int64_t b) { return a / b; }
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? int64_t(uint32_t(a) / uint32_t(b)) : quot_64(a, b);
}

// The first tile whose start is at or behind x.
__device__ __forceinline__ int tile_at(const Seq& q, int64_t x, int log2qt) {
    if (x <= 0) return 0;
    if (x >= q.head_cost) return q.n_tiles;
    if (q.few) return int(quot(x + kCostFew - 1, kCostFew));
    const int u = min(q.n_tiles, ((q.pos0 + (1 << log2qt) - 1) / kTileKeys + 4) & ~3);
    const int64_t per = kCostMany * q.n_qt;
    if (x <= per * u) return int(quot(x + per - 1, per));
    int64_t f = per * u;
    int t = u;
    for (; t < q.n_tiles && f < x; ++t) f += kCostMany * (q.n_qt - first_qt(q, t & ~3, log2qt));
    return t;
}

// The order in which an item's query tiles qt0 .. n_qt - 1 stream: class by class with three or four
// key tiles (each accumulator's warpgroup sums one class after the other), classes 0 and 1 before 2 and
// 3 with two (a warpgroup takes the even or the odd ones), as they come with one (a warpgroup each).
__device__ __forceinline__ int first_in_class(int c, int qt0) { return qt0 + ((c - qt0) & 3); }
__device__ __forceinline__ int first_in_half(int h, int qt0) {          // >= qt0, qt & 2 == h
    return (qt0 & 2) == h ? qt0 : (qt0 | 1) + 1;
}
__device__ __forceinline__ int next_class(int c) { return 0x3132 >> (4 * c) & 3; }   // 0, 2, 1, 3
__device__ __forceinline__ int stream_first(int qt0, int n_qt, int nt) {
    if (nt == 1) return qt0;
    if (nt == 2) {
        const int qt = first_in_half(0, qt0);
        return qt < n_qt ? qt : first_in_half(2, qt0);
    }
    int c = 0, qt = first_in_class(0, qt0);
    while (qt >= n_qt) {
        c = next_class(c);
        qt = first_in_class(c, qt0);
    }
    return qt;
}
// The one behind qt (there is one).
__device__ __forceinline__ int stream_next(int qt, int qt0, int n_qt, int nt) {
    if (nt == 1) return qt + 1;
    if (nt == 2) {
        const int next = qt & 1 ? qt + 3 : qt + 1;
        return next < n_qt || (qt & 2) ? next : first_in_half(2, qt0);
    }
    int c = qt & 3;
    for (qt += 4; qt >= n_qt; qt = first_in_class(c, qt0)) c = next_class(c);
    return qt;
}

// What follows from n_q and ctx.
__device__ __forceinline__ void derive(Seq& q, int log2qt) {
    q.pos0 = q.ctx - q.n_q;
    q.n_tiles = (q.ctx + kTileKeys - 1) / kTileKeys;
    q.n_qt = (q.n_q + (1 << log2qt) - 1) >> log2qt;
    q.few = q.n_qt == 1;
    q.head_cost = cost_before(q, q.n_tiles, log2qt);
}

// shared: another sequence with query rows names s's state row (both would race on it).
__device__ __forceinline__ Seq load_seq(const Params& p, int s, int log2qt, bool shared) {
    Seq q;
    const int c0 = p.cu[s], c1 = p.cu[s + 1];
    q.row = p.rows ? p.rows[s] : s;
    q.ctx = p.ctx[s];
    const int64_t n = int64_t(c1) - c0;
    q.bad = false;
    q.few = true;
    q.head_cost = 0;
    q.any = n != 0;
    if (n == 0 || q.row < 0 || (p.skip_decode && n == 1)) return q;
    q.n_q = int(n);
    q.cu0 = c0;
    q.held = p.held ? p.held[s] : q.ctx - q.n_q;
    if (n < 0 || c0 < 0 || c1 > p.T || q.n_q > q.ctx || q.ctx > min(p.max_len, p.max_ctx) ||
        (int64_t(q.ctx) + p.bs - 1) / p.bs > p.max_blocks || q.row >= p.n_rows || q.held < 0 ||
        q.held > q.ctx || shared) {
        q.bad = true;
        return q;
    }
    derive(q, log2qt);
    return q;
}

// One unit of work, published by the scheduler: FEW: query tile 0 against key tiles t0 .. t0 + nt
// - 1; MANY: key tiles t0 .. t0 + nt - 1 (nt <= 4) against query tiles qt0 .. n_qt - 1.
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
// (q4 = lane % 4, cc = 0, 1). One 16-byte read of log-sum-exps (n, negated, in base 2) so serves 16
// elements: with a lane per key it served four, and those reads took a quarter of the shared-memory
// bandwidth that the MMAs' operands need. Adds 2^(s c + n) to the packed sum of each of the four
// keys.
__device__ __forceinline__ void add16(const uint32_t* lo, const uint32_t* hi, float4 n,
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

// A K slot's code rows r0 .. r0 + 15 (128-byte swizzled, like what they become) expanded to f16 by one
// warp, all of them read before any is written, so that the reads' latency is paid once. Eight lanes
// take one half of the code rows x and x ^ 5 of a swizzle's eight: their reads, and each of their
// two writes, so meet all the banks once (a row of codes to eight lanes met half of them twice when it
// was written). Rows behind the tile's keys hold nothing that counts; their (stale) codes are turned
// as well.
__device__ __forceinline__ void expand_rows(uint32_t slot, int r0, int lane) {
    const uint32_t cc = lane & 3, hi = (lane >> 3) & 1, j0 = 2 * cc;
    const auto row = [&](int i) {                        // pair 2 i + lane / 16
        const uint32_t pair = 2 * i + (lane >> 4), x = pair & 3;
        return uint32_t(r0) + 8 * (pair >> 2) + (lane & 4 ? x ^ 5 : x);
    };
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t R = row(i);
        v[i] = ld_shared_v4(slot + kHalf + R * 128 + (((4 * hi + cc) ^ (R & 7)) << 4));
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t R = row(i), x = R & 7;
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

    // the metadata's and the tables' lines on their way into L2, dealt over the grid's CTAs (up to 8 a
    // lane; a prefetch reads nothing that the kernel before might still write)
    if (warp == 18) {
        const int64_t l_b = (int64_t(p.B) + 31) / 32;
        const int64_t all = 3 * l_b + (int64_t(p.B) * p.max_blocks + 31) / 32;
        int64_t l = int64_t(blockIdx.x) * 32 + lane;
        for (int k = 0; k < 8 && l < all; ++k, l += int64_t(gridDim.x) * 32) {
            const int32_t* at = l < l_b ? p.cu + l * 32
                                : l < 2 * l_b ? p.ctx + (l - l_b) * 32
                                : l < 3 * l_b ? (p.rows ? p.rows + (l - 2 * l_b) * 32 : nullptr)
                                              : p.block_table + (l - 3 * l_b) * 32;
            if (at) prefetch_l2(at);
        }
    }
    if (threadIdx.x < kNumBars) {
        const int b = threadIdx.x;
        mbar_init(bar(b), b >= kStayReady                             ? kTurnWarps
                          : b >= kDrain                               ? 1
                          : b >= kPartDone                            ? 4
                          // issuers 2, stream loader 1, epilogue 16, f16 warps
                          : b >= kItemEmpty                           ? 2 + 1 + 16 + (F8 ? kTurnWarps : 0)
                          : b >= kItemFull                            ? 1
                          : b >= kLseEmpty                            ? 16
                          : b >= kLseFull                             ? 1
                          : b >= kAccEmpty                            ? 4
                          : b >= kAccFull                             ? 1
                          : b >= kStreamEmpty                         ? 2
                          : b >= kStreamFull                          ? 1
                          : b >= kStayEmpty                           ? 2
                                                                      : 1);
        if (b == 0) *abort_word = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 17) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         bars + kHolderOff),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    uint32_t* once = reinterpret_cast<uint32_t*>(smem);
    uint32_t* again = reinterpret_cast<uint32_t*>(smem + kAgain);
    int64_t* costs = reinterpret_cast<int64_t*>(smem + kCosts);
    volatile int* repeated = reinterpret_cast<volatile int*>(smem + kCtl + kTwiceOff);
    if (p.rows)
        for (int i = threadIdx.x; i < (p.n_rows + 31) / 32; i += kThreads) once[i] = again[i] = 0;
    if (threadIdx.x == 0) *repeated = 0;
    if (warp == 18 && lane < 3)
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(
                         lane == 0 ? &tm_k : lane == 1 ? &tm_q1 : &tm_qn))
                     : "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + kCtl + kHolderOff);
    // a programmatic dependent: nothing the kernel before it wrote is read before this point
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- every sequence's cost, and whether two name one state row
    int n_stages;
    {
        bool bad = false, some = false, some_many = false;
        for (int s = threadIdx.x; s < p.B; s += kThreads) {
            const Seq q = load_seq(p, s, log2qt, false);
            if (p.rows && q.row >= 0 && q.row < p.n_rows && q.any) {
                const uint32_t bit = 1u << (q.row & 31);
                if (atomicOr(once + (q.row >> 5), bit) & bit) {
                    atomicOr(again + (q.row >> 5), bit);
                    *repeated = 1;
                }
            }
            costs[s] = q.head_cost;
            if (s < kMetaSeqs) {
                int4* m = reinterpret_cast<int4*>(smem + kMeta) + 2 * s;
                m[0] = make_int4(q.n_q, q.ctx, q.cu0, q.row);
                m[1].x = q.held;
            }
            bad = bad || q.bad;
            some = some || q.head_cost > 0;
            some_many = some_many || (q.head_cost > 0 && !q.few);
        }
        if (bad && blockIdx.x == 0 && p.err) atomicOr(p.err, PA_DEVERR_META);
        // these words were written through the generic proxy where TMA writes next
        fence_proxy_async();
        n_stages = __syncthreads_or(some_many) ? 3 : kMaxStages;
        if (*repeated) {                             // rare: those that share a row drop out
            for (int s = threadIdx.x; s < p.B; s += kThreads) {
                const int row = p.rows[s];
                if (row < 0 || row >= p.n_rows || p.cu[s + 1] == p.cu[s] ||
                    !(again[row >> 5] >> (row & 31) & 1))
                    continue;
                costs[s] = kShared;
                if (blockIdx.x == 0 && p.err) atomicOr(p.err, PA_DEVERR_META);
            }
            fence_proxy_async();
            __syncthreads();
        }
        // behind a step of decode rows alone there is nothing left: 1.3 us earlier out
        if (p.skip_decode && !__syncthreads_or(some)) {
            if (warp == 17)
                asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                             "r"(512)
                             : "memory");
            return;
        }
    }
    const int n_stay = n_stages == 3 ? 4 : 2;

    volatile Item* ring = reinterpret_cast<volatile Item*>(smem + kCtl + kRingOff);
    // a whole warp's arrival, after what its lanes have read or written
    const auto warp_arrive = [&](uint32_t b) {
        __syncwarp();
        if (lane == 0) mbar_arrive(b);
    };
    // takes the next item; called by whole warps, or by the one lane that stands for an issuer's
    const auto next_item = [&](int ic, Item& I, bool alone = false) {
        if (!await(bar(kItemFull + (ic & 3)), (ic >> 2) & 1, abort_word)) return false;
        I = read_item(sb + kCtl + kRingOff + (ic & 3) * 64);
        if (alone) mbar_arrive(bar(kItemEmpty + (ic & 3)));
        else warp_arrive(bar(kItemEmpty + (ic & 3)));
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
        int ks = 0, kph = 1, n_loaded = 0;               // next slot of what stays, parity, tiles so far
        // publishes an item and loads its query tile or key tiles
        const auto emit = [&](Item& I, bool few) {
            if (lane == 0) {
                if (ic >= 4)
                    ok = await(bar(kItemEmpty + (ic & 3)), ((ic >> 2) - 1) & 1, abort_word);
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
            ++ic;
            int ids[4];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                ids[r] = !few && r < I.nt ? block_id(I, I.t0 + r, I.t0 + r + 1) : -1;
            for (int r = 0; r < (few ? 1 : I.nt); ++r) {
                const int id = r == 0 ? ids[0] : r == 1 ? ids[1] : r == 2 ? ids[2] : ids[3];
                if (lane == 0) ok = await(bar(kStayEmpty + ks), kph, abort_word);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) return;
                const uint32_t slot = sb + stay_at(ks, n_stay), full = bar(kStayFull + ks);
                if (few) {
                    if (lane == 0) load_q(slot, full, I, 0);
                } else {
                    const int nblk = blocks_of(I, I.t0 + r);
                    if (lane == 0) mbar_expect_tx(full, k_bytes(nblk));
                    __syncwarp();
                    load_k(slot, full, I, nblk, id);
                }
                ++n_loaded;
                if (++ks == n_stay) {
                    ks = 0;
                    kph ^= 1;
                }
            }
        };
        // ---- the share: this CTA's range of the total cost, and the sequence it starts in
        // (the tiles take the costs' place while later sequences are read: which of them share a row is
        // kept as bits, those of sequences 1024 k + 32 l .. + 31 in lane l's word k)
        const bool twice = *repeated != 0;
        uint32_t shared[kMaxSeqs / 1024];
        if (twice) {
            for (int s0 = 0; s0 < p.B; s0 += 32) {
                const bool out = s0 + lane < p.B && costs[s0 + lane] == kShared;
                const uint32_t word = __ballot_sync(0xffffffffu, out);
                if (lane == (s0 >> 5 & 31)) shared[s0 >> 10] = word;
                if (out) costs[s0 + lane] = 0;
            }
            fence_proxy_async();
            __syncwarp();
        }
        const auto is_shared = [&](int s) {          // s the same for the whole warp
            if (!twice) return false;
            return (__shfl_sync(0xffffffffu, shared[s >> 10], s >> 5 & 31) >> (s & 31) & 1) != 0;
        };
        const int per = (p.B + 31) / 32;             // sequences a lane adds up
        int64_t mine = 0;
        for (int i = 0, s = lane * per; i < per && s < p.B; ++i, ++s) mine += costs[s];
        int64_t upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += y;
        }
        const int blocks = p.Hkv / p.heads, groups = int(gridDim.x) / p.heads;
        const int group = int(blockIdx.x) / p.heads, member = int(blockIdx.x) - group * p.heads;
        const int64_t total = __shfl_sync(0xffffffffu, upto, 31) * blocks;
        const int64_t each = quot(total, groups), rest = total - each * groups;
        const auto bound = [&](int c) { return each * c + int64_t(uint32_t(rest) * c / groups); };
        const int64_t lo = bound(group), hi = bound(group + 1);
        // the last lane whose sequences start at or before lo
        const uint32_t before = __ballot_sync(0xffffffffu, (upto - mine) * blocks <= lo);
        const int from = 31 - __clz(before);
        int64_t base = __shfl_sync(0xffffffffu, upto - mine, from) * blocks;
        int first_s = from * per;
        while (first_s < p.B && base + costs[first_s] * blocks <= lo) base += costs[first_s++] * blocks;
        // the first sequence's metadata is still at hand; the next ones are read again
        Seq q;
        if (first_s < min(p.B, kMetaSeqs)) {
            const int4* m = reinterpret_cast<const int4*>(smem + kMeta) + 2 * first_s;
            const int4 v = m[0];
            q.n_q = v.x;
            q.ctx = v.y;
            q.cu0 = v.z;
            q.row = v.w;
            q.held = m[1].x;
            derive(q, log2qt);
        } else if (first_s < p.B) {
            q = load_seq(p, first_s, log2qt, false);
        }
        __syncwarp();                                // costs and metadata make room for the tiles
        for (int s = first_s; s < p.B && base < hi && ok; ++s) {
            if (s > first_s) q = load_seq(p, s, log2qt, is_shared(s));
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
            for (int h = base < lo ? int(quot(lo - base, q.head_cost)) : 0; h < blocks && ok; ++h) {
                const int64_t hb = base + h * q.head_cost;
                if (hb >= hi) break;
                const int ta = tile_at(q, lo - hb, log2qt), tb = tile_at(q, hi - hb, log2qt);
                I.kvh = h * p.heads + member;
                I.state = (int64_t(q.row) * p.Hkv + I.kvh) * p.max_len;
                if (q.few) {
                    if (ta >= tb) continue;
                    I.t0 = ta;
                    I.nt = tb - ta;
                    I.qt0 = 0;
                    emit(I, true);
                } else {
                    for (int t = ta; t < tb && ok; t += I.nt) {
                        I.t0 = t;
                        I.nt = min(4, tb - t);
                        I.qt0 = first_qt(q, t, log2qt);
                        emit(I, false);
                    }
                }
            }
            base += q.head_cost * blocks;
        }
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        if (ok) {
            Item I = {};
            I.last = 1;
            emit(I, true);
        }
        if (lane == 0) {
            // never leave with copies in flight into this CTA's shared memory
            for (int i = max(0, n_loaded - n_stay); i < n_loaded; ++i)
                wait_drain(bar(kStayFull + i % n_stay), (i / n_stay) & 1);
        }
    } else if (warp == 17 || warp == 19) {
        // ------------------------------------------------ MMA issuers
        if (lane == 0) {
            const int me = warp == 19;           // fills accumulators me and me + 2
            int n = 0, st = 0, ph = 0;           // stream tile, its stage and the stage's parity
            int ks = 0, kph = 0;                 // next slot of what stays and its parity
            uint32_t eph = 3;                    // parities of the two accumulators' next return
            bool ok = true;
            // (the first look in line: mostly the phase is past, and the issuer's own time counts)
            const auto wait = [&](int b, uint32_t parity) {
                return mbar_try_wait(bar(b), parity) || await(bar(b), parity, abort_word);
            };
            const auto take_back = [&](int h) {
                ok = wait(kAccEmpty + me + 2 * h, eph >> h & 1);
                eph ^= 1u << h;
                return ok;
            };
            const uint32_t idesc_full = make_idesc(128, kCols, false, F8);
            for (int ic = 0;; ++ic) {
                Item I;
                if (!next_item(ic, I, true)) break;
                const bool few = I.n_qt == 1;
                const int n_tiles = few ? 1 : I.nt, first = ks;
                for (int r = 0; r < n_tiles && ok; ++r) {
                    ok = await(bar(kStayUse + ks), kph, abort_word);
                    if (++ks == n_stay) {
                        ks = 0;
                        kph ^= 1;
                    }
                }
                if (!ok) break;
                const auto first_slot = [&](int r) { return (first + r) & (n_stay - 1); };
                const auto stay = [&](int r) {
                    return make_sdesc(sb + stay_at(first_slot(r), n_stay), 16, 1024);
                };
                const uint64_t stay0 = stay(few || I.nt == 1 ? 0 : me), stay1 = stay(few ? 0 : me + 2);
                const int last_cols = (I.n_q - ((I.n_qt - 1) << log2qt)) * p.g;
                const uint32_t idesc_last = make_idesc(128, (last_cols + 15) & ~15, false, F8);
                const auto next_stage = [&]() {
                    if (++st == n_stages) {
                        st = 0;
                        ph ^= 1;
                    }
                };
                if (few) {
                    for (const int end = n + I.nt; n < end; ++n) {
                        if (!(ok = wait(kStreamUse + st, ph))) break;
                        const int acc = n & 3;
                        if ((acc & 1) == me) {
                            if (!take_back(acc >> 1)) break;
                            tc_fence_after();
                            issue_s_group<D>(1u, tmem + acc * kCols,
                                             make_sdesc(sb + stage_at(st), 16, 1024), stay0,
                                             idesc_last);
                            tc_commit_if(1u, bar(kAccFull + acc));
                            tc_commit_if(1u, bar(kStreamEmpty + st));
                        } else {
                            mbar_arrive(bar(kStreamEmpty + st));
                        }
                        next_stage();
                    }
                } else {
                    const uint64_t stage0 = make_sdesc(sb + stage_at(0), 16, 1024);
                    const bool two = me + 2 < I.nt;
                    const int end = n + I.n_qt - I.qt0;
                    int qt = stream_first(I.qt0, I.n_qt, I.nt);
                    for (; n < end; ++n) {
                        // (three stages, side by side)
                        const uint64_t stage = stage0 + uint32_t(st) * (kSlot / 16);
                        const uint32_t idesc = qt + 1 == I.n_qt ? idesc_last : idesc_full;
                        if (!(ok = wait(kStreamUse + st, ph))) break;
                        if (I.nt == 1 ? (qt & 1) == me : me < I.nt) {
                            const int h = I.nt == 1 ? qt >> 1 & 1 : I.nt == 2 ? qt & 1 : 0;
                            if (!take_back(h)) break;
                            tc_fence_after();
                            issue_s_group<D>(1u, tmem + (me + 2 * h) * kCols, stay0, stage, idesc);
                            tc_commit_if(1u, bar(kAccFull + me + 2 * h));
                        }
                        if (two) {
                            // (the first tile's slot is not needed any more once the last query
                            // tile's product is in the pipe)
                            if (n + 1 == end) tc_commit_if(1u, bar(kStayEmpty + first_slot(me)));
                            if (!take_back(1)) break;
                            tc_fence_after();
                            issue_s_group<D>(1u, tmem + (me + 2) * kCols, stay1, stage, idesc);
                            tc_commit_if(1u, bar(kAccFull + me + 2));
                        }
                        tc_commit_if(1u, bar(kStreamEmpty + st));
                        if (n + 1 < end) qt = stream_next(qt, I.qt0, I.n_qt, I.nt);
                        next_stage();
                    }
                }
                if (!ok) break;
                for (int r = 0; r < n_tiles; ++r)
                    if (few || r != me || me + 2 >= I.nt)
                        tc_commit_if(1u, bar(kStayEmpty + first_slot(r)));
            }
            // every MMA has finished before TMEM is released
            tc_commit_if(1u, bar(kDrain + me));
            wait_drain(bar(kDrain + me), 0);
        }
    } else if (warp == 18) {
        // ------------------------------------------------ loader of what streams
        int n_lse = 0;                                    // MANY tiles so far
        int st = 0, ph = 1, n_done = 0, ok = 1;   // a fresh barrier's phase 1 counts as past
        const int per_tile = kTileKeys >> log2bs, per_load = 32 / per_tile;   // blocks; tiles
        for (int ic = 0; ok; ++ic) {
            Item I;
            ok = next_item(ic, I);
            if (!__all_sync(0xffffffffu, ok)) break;
            const bool few = I.n_qt == 1;
            const int n = few ? I.nt : I.n_qt - I.qt0, end = I.t0 + I.nt;
            // the lanes hold the blocks of per_load tiles, and those of the next ones on their way
            int ids = few ? block_id(I, I.t0, end) : -1, next = -1;
            // the lane's four log-sum-exps of a query tile, negated, in base 2
            const auto fetch_lse = [&](int qt) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int col = 4 * lane + e, tok = (qt << log2qt) + (col >> (7 - log2qt));
                    v[e] = 0.f;
                    if (tok < I.n_q)
                        v[e] = -1.4426950408889634f *
                               __ldg(p.lse + int64_t(I.cu0 + tok) * p.Hq + I.kvh * p.g +
                                     (col & (p.g - 1)));
                }
                return make_float4(v[0], v[1], v[2], v[3]);
            };
            int qt = few ? 0 : stream_first(I.qt0, I.n_qt, I.nt);
            float4 l_next = few ? make_float4(0.f, 0.f, 0.f, 0.f) : fetch_lse(qt);
            for (int i = 0; i < n; ++i) {
                const int at = i & (per_load - 1);
                if (few && at == 0 && i > 0) ids = next;
                if (lane == 0) ok = await(bar(kStreamEmpty + st), ph, abort_word);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                const uint32_t slot = sb + stage_at(st), full = bar(kStreamFull + st);
                if (few) {
                    const int nblk = blocks_of(I, I.t0 + i);
                    const int id = __shfl_sync(0xffffffffu, ids, (at * per_tile + lane) & 31);
                    if (lane == 0) mbar_expect_tx(full, k_bytes(nblk));
                    __syncwarp();
                    load_k(slot, full, I, nblk, id);
                    if (at == 0 && i + per_load < n) next = block_id(I, I.t0 + i + per_load, end);
                } else {
                    const int lse_slot = n_lse & 3;
                    if (lane == 0) {
                        load_q(slot, full, I, qt);
                        ok = await(bar(kLseEmpty + lse_slot), (n_lse >> 2 & 1) ^ 1,
                                          abort_word);
                    }
                    const float4 v = l_next;
                    if (i + 1 < n) {
                        qt = stream_next(qt, I.qt0, I.n_qt, I.nt);
                        l_next = fetch_lse(qt);
                    }
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (ok) {
                        float* to = reinterpret_cast<float*>(smem + kCtl + kLseOff) +
                                    lse_slot * 128;
                        *reinterpret_cast<float2*>(to + lse_place(4 * lane)) =
                            make_float2(v.x, v.y);
                        *reinterpret_cast<float2*>(to + lse_place(4 * lane + 2)) =
                            make_float2(v.z, v.w);
                        warp_arrive(bar(kLseFull + lse_slot));
                        ++n_lse;
                    }
                }
                ++n_done;
                if (++st == n_stages) {
                    st = 0;
                    ph ^= 1;
                }
                if (!ok) break;
            }
        }
        if (lane == 0) {
            // never leave with copies in flight into this CTA's shared memory
            for (int i = max(0, n_done - n_stages); i < n_done; ++i)
                wait_drain(bar(kStreamFull + i % n_stages), (i / n_stages) & 1);
        }
    } else if (warp >= kTurners) {
        // ------------------------------------------------ codes and q to f16 (fp8 cache)
        if constexpr (F8) {
            const int w = warp - kTurners;
            // the MMAs take f16 operands: 32 rows a warp of a K tile's codes are expanded, or a
            // query tile is rounded in place (a 16-byte chunk keeps its place, so the swizzle holds)
            const auto turn_k = [&](uint32_t slot, const Item& I, int t) {
                const int rows = I.ctx - t * kTileKeys;
                if (32 * w < rows) expand_rows(slot, 32 * w, lane);
                if (32 * w + 16 < rows) expand_rows(slot, 32 * w + 16, lane);
            };
            const auto turn_q = [&](uint32_t slot, int rows) {
                for (int i = threadIdx.x - kBaseThreads; i < rows * 16; i += 32 * kTurnWarps) {
                    const uint32_t a = slot + ((i >> 3) & 1) * kHalf + (i >> 4) * 128 + (i & 7) * 16;
                    const uint4 v = ld_shared_v4(a);
                    st_shared_v4(a, bf16x2_to_f16x2(v.x), bf16x2_to_f16x2(v.y),
                                 bf16x2_to_f16x2(v.z), bf16x2_to_f16x2(v.w));
                }
            };
            int st = 0, ph = 0, ks = 0, kph = 0;
            bool ok = true;
            for (int ic = 0; ok; ++ic) {
                Item I;
                if (!next_item(ic, I)) break;
                const bool few = I.n_qt == 1;
                for (int r = 0; r < (few ? 1 : I.nt); ++r) {
                    if (!(ok = await(bar(kStayFull + ks), kph, abort_word))) break;
                    const uint32_t slot = sb + stay_at(ks, n_stay);
                    if (few) turn_q(slot, I.n_q == 1 ? p.g : kCols);
                    else turn_k(slot, I, I.t0 + r);
                    fence_proxy_async();
                    warp_arrive(bar(kStayReady + ks));
                    if (++ks == n_stay) {
                        ks = 0;
                        kph ^= 1;
                    }
                }
                const int n = few ? I.nt : I.n_qt - I.qt0;
                for (int i = 0; i < n && ok; ++i) {
                    if (!(ok = await(bar(kStreamFull + st), ph, abort_word))) break;
                    const uint32_t slot = sb + stage_at(st);
                    if (few) turn_k(slot, I, I.t0 + i);
                    else turn_q(slot, kCols);
                    fence_proxy_async();
                    warp_arrive(bar(kStreamReady + st));
                    if (++st == n_stages) {
                        st = 0;
                        ph ^= 1;
                    }
                }
            }
        }
    } else {
        // ------------------------------------------------ epilogue warpgroups
        const int w = warp >> 2;             // reads accumulator w
        const uint32_t tm = tmem + w * kCols + (uint32_t(32 * (warp & 3)) << 16);
        const int q4 = lane & 3, rs = lane >> 2;
        // after the sums over the four threads of a key have met, thread q4 has key rs + 8 q4
        const int key_in_tile = 32 * (warp & 3) + rs + 8 * q4;
        const uint64_t c2 = f2(p.c, p.c);
        int n = 0, acc_ph = 0, n_lse = 0, n_part = 0, n_chain = 0;
        const uint32_t full = bar(kAccFull + w), empty = bar(kAccEmpty + w);
        const float4* lse_smem = reinterpret_cast<const float4*>(smem + kCtl + kLseOff) + q4;
        bool ok = true;
        const int log2g = 7 - log2qt;
        uint64_t a[4];                       // the thread's part of its four keys' sums
        const auto clear = [&]() {
#pragma unroll
            for (int k = 0; k < 4; ++k) a[k] = f2(0.f, 0.f);
        };
        // log-sum-exps of columns col, col + 1 (col even) of the query tile from token `tok` on,
        // negated, in base 2; columns behind the sequence's rows read nothing
        const auto lse_pair = [&](const Item& I, int tok, int col) {
            const int i = tok + (col >> log2g);
            const float* l = p.lse + int64_t(I.cu0 + i) * p.Hq + I.kvh * p.g;
            float x = 0.f, y = 0.f;
            if (log2g > 0) {
                if (i < I.n_q) {
                    const float2 v = __ldg(reinterpret_cast<const float2*>(l + (col & (p.g - 1))));
                    x = v.x;
                    y = v.y;
                }
            } else {
                if (i < I.n_q) x = __ldg(l);
                if (i + 1 < I.n_q) y = __ldg(l + p.Hq);
            }
            return mul2(f2(x, y), f2(-1.4426950408889634f, -1.4426950408889634f));
        };
        // adds the first `cols` columns of the accumulator (query tile from token tok on), masked by
        // causality, and hands it back; the warp's keys are those from kw on. nl: the log-sum-exps
        // in shared memory, or NULL
        const auto add_masked = [&](const Item& I, int tok, int cols, int kw, const float4* nl) {
            const int at = I.pos0 + tok;
            for (int c = 0; c < cols; c += 16) {
                uint32_t lo[8], hi[8];
                tmem_ld_16x256b_x2(tm + c, lo);
                tmem_ld_16x256b_x2(tm + c + (16u << 16), hi);
                float nv[4];
                if (nl) {
                    const float4 v = nl[c / 4];
                    nv[0] = v.x, nv[1] = v.y, nv[2] = v.z, nv[3] = v.w;
                } else {
                    f2_split(lse_pair(I, tok, c + 2 * q4), nv[0], nv[1]);
                    f2_split(lse_pair(I, tok, c + 8 + 2 * q4), nv[2], nv[3]);
                }
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    // the first column whose row comes at or after the key
                    const int from = max(0, kw + rs + 8 * k - at) << log2g;
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) {
                        const uint32_t* s = (k < 2 ? lo : hi) + 4 * cc + 2 * (k & 1);
                        float e[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int col = c + 8 * cc + 2 * q4 + i;
                            const float x = ex2(fmaf(__uint_as_float(s[i]), p.c, nv[2 * cc + i]));
                            e[i] = col >= from && col < cols ? x : 0.f;
                        }
                        a[k] = add2(a[k], f2(e[0], e[1]));
                    }
                }
            }
            tc_fence_before();
            warp_arrive(empty);
        };
        // the same for a whole query tile that every key of the warp comes before
        const auto add_all = [&](const float4* nl) {
            // 16 columns at a time, the next ones on their way (half or all of the accumulator in
            // registers first, to hand it back earlier, made the whole kernel a fourth slower)
            uint32_t lo0[8], hi0[8], lo1[8], hi1[8];
            tmem_ld_16x256b_x2(tm, lo0);
            tmem_ld_16x256b_x2(tm + (16u << 16), hi0);
#pragma unroll
            for (int c = 0; c < kCols; c += 32) {
                tmem_wait_ld();
                tmem_ld_16x256b_x2(tm + c + 16, lo1);
                tmem_ld_16x256b_x2(tm + c + 16 + (16u << 16), hi1);
                add16(lo0, hi0, nl[c / 4], c2, a);
                tmem_wait_ld();
                if (c + 32 < kCols) {
                    tmem_ld_16x256b_x2(tm + c + 32, lo0);
                    tmem_ld_16x256b_x2(tm + c + 32 + (16u << 16), hi0);
                } else {
                    tc_fence_before();
                    warp_arrive(empty);
                }
                add16(lo1, hi1, nl[c / 4 + 4], c2, a);
            }
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
            if (I.n_qt == 1) {
                // the item's first tile of this warpgroup, then every fourth
                for (int i = (w - n) & 3; i < I.nt; i += 4) {
                    const int kb = (I.t0 + i) * kTileKeys, j = kb + key_in_tile;
                    float* dst = p.weights + I.state + j;
                    const float old = j < I.held ? *dst : 0.f;
                    if (!(ok = await(full, acc_ph, abort_word))) break;
                    acc_ph ^= 1;
                    clear();
                    tc_fence_after();
                    add_masked(I, 0, I.n_q * p.g, kb + 32 * (warp & 3), nullptr);
                    const float sum = total_of_key();
                    if (j < I.ctx) *dst = old + sum;
                }
                n += I.nt;
                continue;
            }
            // key tile r: all query tiles, or with one or two key tiles those with qt & mod == w's
            const int mod = I.nt == 1 ? 3 : I.nt == 2 ? 1 : 0;
            const int r = I.nt == 1 ? 0 : I.nt == 2 ? w & 1 : w;
            const int turn = I.nt == 1 ? w : w >> 1;
            const bool my = r < I.nt;
            const int kb = (I.t0 + r) * kTileKeys, j = kb + key_in_tile, kw = kb + 32 * (warp & 3);
            float* dst = p.weights + I.state + j;
            // the warpgroups' order: 0, 2, 1, 3 with one key tile, r, r + 2 with two
            const int place = mod == 0 ? 0 : mod == 1 ? w >> 1 : w == 0 ? 0 : w == 2 ? 1 : w == 1 ? 2 : 3;
            const int hops = mod == 0 ? 0 : mod == 1 ? 1 : 3;
            // the one that has class 0 begins; the classes are added in the order 0, 2, 1, 3, those of
            // another warpgroup once they are there (at most two: kept apart). The last one adds the
            // old sum: it reads it here, before the first may write the entry
            const bool opens = place == 0, ends = place == hops;
            const float old = my && ends && j < I.held ? *dst : 0.f;
            const int seen = bar(mod == 1 ? kPartSeen + r : kChainSeen);
            if (mod != 0 && ends) warp_arrive(seen);
            float sum = 0.f, later = 0.f;
            int qt = stream_first(I.qt0, I.n_qt, I.nt), now = -1;
            const auto close = [&]() {                   // the class that was being summed
                const float s = total_of_key();
                if (opens) sum += s;
                else if (mod == 1 && now >= 2) later = s;
                else sum = s;
                clear();
            };
            clear();
            for (int i = I.qt0; i < I.n_qt; ++i, ++n, ++n_lse) {
                const int tok = qt << log2qt, cols = min(kCols, (I.n_q - tok) * p.g);
                const int at = I.pos0 + tok;             // the tile's first row
                const float4* nl = lse_smem + (n_lse & 3) * 32;
                if (!(ok = await(bar(kLseFull + (n_lse & 3)), n_lse >> 2 & 1, abort_word)))
                    break;
                if (my && (qt & mod) == (turn & mod)) {
                    if (now >= 0 && now != (qt & 3)) close();
                    now = qt & 3;
                    if (!(ok = await(full, acc_ph, abort_word))) break;
                    acc_ph ^= 1;
                    tc_fence_after();
                    if (kw > at + ((cols - 1) >> log2g)) warp_arrive(empty);   // all rows come before
                    else if (cols == kCols && kw + 31 <= at) add_all(nl);
                    else add_masked(I, tok, cols, kw, nl);
                }
                warp_arrive(bar(kLseEmpty + (n_lse & 3)));
                if (i + 1 < I.n_qt) qt = stream_next(qt, I.qt0, I.n_qt, I.nt);
            }
            if (!ok) break;
            if (!my) continue;
            if (now >= 0) close();
            if (mod == 0) {
                if (j < I.ctx) *dst = old + sum;
                continue;
            }
            int& n_hops = mod == 1 ? n_part : n_chain;
            // from place to place; the next item's first hand-over waits for the last one's look at
            // its entries, and so for the end of this item's
            const int done = bar(mod == 1 ? kPartDone + r : kChainDone + place);
            if (opens) {
                if (!(ok = await(seen, n_hops & 1, abort_word))) break;
                if (j < I.ctx) *dst = sum;
            } else {
                if (!(ok = await(mod == 1 ? done : done - 8, n_hops & 1, abort_word))) break;
                if (j < I.ctx) {
                    const float all = (*dst + sum) + later;
                    *dst = ends ? old + all : all;
                }
            }
            if (!ends) warp_arrive(done);
            ++n_hops;
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
    // whole groups: 152 is a multiple of 8
    const int64_t tiles = int64_t(p.B) * (p.Hkv / p.heads) *
                          ((int64_t(p.max_len) + kTileKeys - 1) / kTileKeys) * p.heads;
    static_assert(PA_PLAN_CTAS % 8 == 0, "groups of up to 8 CTAs");
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
// Scores kept for a step: rows of a whole number of tiles.
__host__ __device__ int64_t scores_row(int32_t max_ctx) {
    return (int64_t(max_ctx) + kTileKeys - 1) / kTileKeys * kTileKeys;
}

// One thread per four keys of a (sequence, KV head): the group's raw scores, stored by the
// attention kernel, against the rows' log-sum-exps. A decode step so pays 4 g bytes per key and
// KV head written and read again in place of a second read of K's 2 D (D over an e4m3 cache): 32 rows at
// 4k .. 16k keys (8 KV heads of 128, group 4) take 261 us, 230 of them the plain step, 15 this kernel (56
// MB read); the step followed by a pass over K 360. Larger groups gain less, but gain: 32 rows at 8,000
// keys, kept scores against a second pass, group 8 202 / 271 us, group 16 (4 KV heads) 132 / 158, over
// e4m3 149 / 171, head_dim 64 101 / 120. As a part of the kernel above (a warp per key tile, one, two or
// four tiles at a time) 265 to 271. The grid covers max_ctx, whose idle blocks leave at once: 32 rows of
// 2,000 keys 79 us at a bound of 2,000 or 10,000, 85 at 40,000.
constexpr int kDecodeKeys = 1024;      // per block of 256 threads
__global__ void __launch_bounds__(256)
    decode_weights_kernel(const float* __restrict__ scores, const Params p) {
    __shared__ float nl[16];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int s = int(blockIdx.z), h = int(blockIdx.y);
    const int c0 = p.cu[s], ctx = p.ctx[s];
    const int row = p.rows ? p.rows[s] : s;
    const int j0 = int(blockIdx.x) * kDecodeKeys;
    if (p.cu[s + 1] - c0 != 1 || row < 0 || (j0 >= ctx && j0 > 0)) return;
    const int held = p.held ? p.held[s] : ctx - 1;
    bool bad = c0 < 0 || c0 >= p.T || ctx < 1 || ctx > p.max_len || ctx > p.max_ctx ||
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
    // a row of scores is a whole number of tiles: a thread's four lie within it
    const int64_t scores_ld = scores_row(p.max_ctx);
    const float* sc = scores + (int64_t(s) * p.Hq + h * p.g) * scores_ld + j;
    float* w = p.weights + (int64_t(row) * p.Hkv + h) * p.max_len + j;
    // the old sum joins once, rounded once: a head's weight may be below half a step of it
    float old[4], sum[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        old[e] = j + e < held ? w[e] : 0.f;
        sum[e] = 0.f;
    }
    for (int i = 0; i < p.g; ++i) {
        const float4 x = __ldcs(reinterpret_cast<const float4*>(sc + int64_t(i) * scores_ld));
        sum[0] += ex2(fmaf(x.x, p.c, nl[i]));
        sum[1] += ex2(fmaf(x.y, p.c, nl[i]));
        sum[2] += ex2(fmaf(x.z, p.c, nl[i]));
        sum[3] += ex2(fmaf(x.w, p.c, nl[i]));
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (j + e < ctx) w[e] = old[e] + sum[e];
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
                          int32_t max_ctx = INT32_MAX) {
    int32_t st = check_shape(s);
    if (st) return st;
    if (fp8 && s->head_dim != 128) return PA_ERR_SHAPE;
    if (B < 0 || T < 0 || max_blocks < 0 || n_rows < 0 || max_len < 0) return PA_ERR_INVALID;
    if (T == 0 || B == 0) return PA_OK;
    if (B > kMaxSeqs) return PA_ERR_SHAPE;
    if (!q || !k_pool || !lse || !block_table || !cu || !ctx || !weights) return PA_ERR_INVALID;
    if (max_len == 0 || (!rows && n_rows < B)) return PA_ERR_INVALID;
    if (n_rows > kMaxRows || int64_t(s->num_blocks) * s->block_size > INT32_MAX ||
        max_len > kMaxLen)
        return PA_ERR_SHAPE;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_pool)) & 15 ||
        reinterpret_cast<uintptr_t>(lse) & 7)
        return PA_ERR_INVALID;
    const int D = s->head_dim, g = s->num_q_heads / s->num_kv_heads;
    const int64_t slots = int64_t(s->num_blocks) * s->block_size;
    CUtensorMap k, q1, qn;
    st = fp8 ? make_map_codes(&k, k_pool, D, s->num_kv_heads, slots, s->block_size,
                              CU_TENSOR_MAP_SWIZZLE_128B)
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
    p.heads = p.Hkv % 8 == 0 ? 8 : p.Hkv % 4 == 0 ? 4 : p.Hkv % 2 == 0 ? 2 : 1;
    p.bs = s->block_size;
    p.num_blocks = s->num_blocks;
    p.n_rows = n_rows;
    p.max_len = max_len;
    p.c = float(1.4426950408889634 / std::sqrt(double(D))) * k_scale;
    p.skip_decode = scores != nullptr;
    p.max_ctx = max_ctx;
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
        if ((st = note_cuda(cudaLaunchKernelEx(&cfg, decode_weights_kernel, scores, p))))
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
    if (B > kMaxSeqs || s->num_kv_heads > 65535 || n_rows > kMaxRows ||
        max_len > kMaxLen || max_ctx > kMaxLen ||
        int64_t(s->num_blocks) * s->block_size > INT32_MAX)
        return PA_ERR_SHAPE;
    if (!workspace || ws_bytes < pa_step_weights_workspace_bytes(s, B, T, max_ctx))
        return PA_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 15) || (reinterpret_cast<uintptr_t>(lse) & 7))
        return PA_ERR_INVALID;
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
