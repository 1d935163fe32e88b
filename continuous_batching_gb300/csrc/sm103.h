// Device-side building blocks shared by the library's tcgen05 kernels: mbarriers with bounded
// waits, TMA tile loads, tcgen05 fences and commits, shared-memory descriptors, the S = A B^T MMA
// group, the packed fp32 arithmetic and the expansion of fp8 codes.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.h"

namespace {

constexpr int kTileKeys = PA_TILE_KEYS;

constexpr unsigned long long kWaitLimitNs = 1000000000ull;   // one second per wait

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(bar)
                 : "memory");
}

// The MMA warp runs its whole loop with all 32 lanes, so that its control flow never
// diverges; the instructions that one thread must issue take the issuing lane as a predicate.
__device__ __forceinline__ void mbar_arrive_if(uint32_t issue, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t.reg .b64 st;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q mbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(bar), "r"(issue)
        : "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile(
        "{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar),
        "r"(bytes)
        : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ void prefetch_l2(const void* a) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(a));
}

__device__ __forceinline__ unsigned long long global_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// Waits for the phase of `bar` with the given parity. Gives up when another role has set
// the CTA's abort word or after limit_ns; then sets the abort word and returns false. Between two
// looks at the abort word and the clock, which leave the other warps' work in peace for a while, it
// polls POLLS times.
template <int POLLS = 32>
__device__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort_word,
                             unsigned long long limit_ns = kWaitLimitNs) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_ns();
    for (;;) {
        for (int i = 0; i < POLLS; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*abort_word) return false;
        if (global_ns() - t0 > limit_ns) {
            *abort_word = 1;
            return false;
        }
    }
}

// Waits for an mbarrier phase that the CTA's own copies or MMAs complete, before the CTA
// leaves: it ignores the abort word (the copies are in flight whatever happened) but still
// gives up after kWaitLimitNs.
__device__ void wait_drain(uint32_t bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return;
    const unsigned long long t0 = global_ns();
    while (!mbar_try_wait(bar, parity))
        if (global_ns() - t0 > kWaitLimitNs) return;
}

__device__ __forceinline__ void fence_proxy_async() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int32_t x, int32_t y, int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int32_t x, int32_t y, int32_t z, int32_t w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_commit_if(uint32_t issue, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(issue)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// The MMA groups of one tile, each in one asm block: the issuing warp shares its scheduler
// with two softmax warps that take most issue slots, so every instruction between two MMAs
// costs tensor-pipe time. The predicates are set once per group, and a step k only adds its
// offset / 16 to the low word of a shared-memory descriptor (the start-address field, bits
// 0-13, never carries: shared addresses stay below 2^18).
//
// S group: D[tmem] = sum_k A_k B_k^T with A = Q, B = K (both K-major in shared memory); step k
// reads 16 columns at byte offset (k / 4) * 16384 + (k % 4) * 32 of both operands.
#define PA_S_STEP(OFF, PRED)                                                                   \
    "add.u32 x, al, " #OFF ";\n\tadd.u32 y, bl, " #OFF ";\n\tmov.b64 a, {x, ah};\n\t"            \
    "mov.b64 b, {y, bh};\n\t@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, " PRED ";\n\t"
template <int D>
__device__ __forceinline__ void issue_s_group(uint32_t issue, uint32_t d, uint64_t qdesc,
                                              uint64_t kdesc, uint32_t idesc) {
    static_assert(D == 64 || D == 128, "head_dim");
    if constexpr (D == 128) {
        asm volatile(
            "{\n\t.reg .pred q, pt, pf;\n\t.reg .b32 al, ah, bl, bh, x, y;\n\t.reg .b64 a, b;\n\t"
            "setp.ne.b32 q, %4, 0;\n\tsetp.eq.b32 pt, %4, %4;\n\tsetp.ne.b32 pf, %4, %4;\n\t"
            "mov.b64 {al, ah}, %1;\n\tmov.b64 {bl, bh}, %2;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, pf;\n\t"
            PA_S_STEP(2, "pt") PA_S_STEP(4, "pt") PA_S_STEP(6, "pt") PA_S_STEP(1024, "pt")
            PA_S_STEP(1026, "pt") PA_S_STEP(1028, "pt") PA_S_STEP(1030, "pt") "}" ::"r"(d),
            "l"(qdesc), "l"(kdesc), "r"(idesc), "r"(issue)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred q, pt, pf;\n\t.reg .b32 al, ah, bl, bh, x, y;\n\t.reg .b64 a, b;\n\t"
            "setp.ne.b32 q, %4, 0;\n\tsetp.eq.b32 pt, %4, %4;\n\tsetp.ne.b32 pf, %4, %4;\n\t"
            "mov.b64 {al, ah}, %1;\n\tmov.b64 {bl, bh}, %2;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, pf;\n\t"
            PA_S_STEP(2, "pt") PA_S_STEP(4, "pt") PA_S_STEP(6, "pt") "}" ::"r"(d), "l"(qdesc),
            "l"(kdesc), "r"(idesc), "r"(issue)
            : "memory");
    }
}
#undef PA_S_STEP

// Instruction descriptor, kind::f16: fp32 accumulator (bits 4-5 = 1), A and B bf16 (bits 7-9,
// 10-12 = 1) or both f16 (0), A K-major, B K-major or MN-major (bit 16), N >> 3 at bits
// 17-22, M >> 4 at bits 24-28.
__host__ __device__ constexpr uint32_t make_idesc(int M, int N, bool b_mn_major, bool f16) {
    return (1u << 4) | ((f16 ? 0u : 1u) << 7) | ((f16 ? 0u : 1u) << 10) |
           ((b_mn_major ? 1u : 0u) << 16) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

// Shared-memory matrix descriptor: start address >> 4 (bits 0-13), leading-dimension byte
// offset >> 4 (16-29), stride-dimension byte offset >> 4 (32-45), descriptor version 1
// (bit 46), 128-byte swizzle (layout type 2, bits 61-63). Operand tiles sit at 1024-byte
// aligned addresses in rows of 128 bytes, 8-row swizzle atoms.
__device__ __forceinline__ uint64_t make_sdesc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return uint64_t((addr & 0x3FFFF) >> 4) | (uint64_t((lbo >> 4) & 0x3FFF) << 16) |
           (uint64_t((sbo >> 4) & 0x3FFF) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// 2^x on the special-function unit (ex2.approx, flush-to-zero). Every place that takes an
// exponential in this library calls this one helper, so all of them round the same way.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Packed fp32 pairs (lo, hi) in one 64-bit register for the f32x2 instructions. They are used
// where every row goes through the same instructions whatever its item (the softmax and the
// rescale); the fold of split partials stays scalar like the combine kernel it must match.
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f2_split(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Maximum of 32 values (exact in any order).
__device__ __forceinline__ float max32(const float (&v)[32]) {
    float t[11];
#pragma unroll
    for (int k = 0; k < 10; ++k) t[k] = max3(v[3 * k], v[3 * k + 1], v[3 * k + 2]);
    t[10] = fmaxf(v[30], v[31]);
    const float u0 = max3(t[0], t[1], t[2]), u1 = max3(t[3], t[4], t[5]);
    const float u2 = max3(t[6], t[7], t[8]), u3 = fmaxf(t[9], t[10]);
    return fmaxf(max3(u0, u1, u2), u3);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

// Four e4m3 codes (lowest byte first) -> two f16x2 words (exact: every e4m3 value is an f16
// value).
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// Expands the 128-byte code rows r_begin .. rows - 1 of a K (IS_V false) or V ring slot to f16
// in place (8 lanes per row, 4 rows per pass). rows - r_begin is a multiple of 8 (whole blocks
// of at least 8 rows), so every pass has 4 valid rows. Row R's codes sit unswizzled where the
// row's second 64-column f16 half goes (K slots: [half][key row]; V slots: [block][half][row]);
// its f16 halves go to the 128-byte swizzled rows TMA would have written. A row is read by its
// 8 lanes before any lane writes over it.
template <bool IS_V>
__device__ __forceinline__ void expand_codes(uint32_t slot, int r_begin, int rows, int bs,
                                             int log2bs, int lane) {
    const int c = lane & 7;                    // code chunk: columns 16 c .. 16 c + 15
    const uint32_t j0 = uint32_t(2 * (c & 3)); // its first f16 chunk within the half
    const uint32_t hi = uint32_t(c >> 2);      // the half it goes to
    for (int R0 = r_begin; R0 + 4 <= rows; R0 += 4) {        // warp-uniform: whole passes
        const int R = R0 + (lane >> 3);
        uint32_t b0, half_step;
        if constexpr (IS_V) {
            b0 = slot + uint32_t(R >> log2bs) * uint32_t(bs * 256) + uint32_t(R & (bs - 1)) * 128;
            half_step = uint32_t(bs * 128);
        } else {
            b0 = slot + uint32_t(R) * 128;
            half_step = uint32_t(kTileKeys * 128);
        }
        const uint32_t b1 = b0 + half_step;
        const uint4 v = ld_shared_v4(b1 + uint32_t(c) * 16);
        __syncwarp();
        uint32_t f[8];
        e4m3x4_to_f16x4(v.x, f[0], f[1]);
        e4m3x4_to_f16x4(v.y, f[2], f[3]);
        e4m3x4_to_f16x4(v.z, f[4], f[5]);
        e4m3x4_to_f16x4(v.w, f[6], f[7]);
        const uint32_t rb = b0 + hi * half_step;
        const uint32_t x = uint32_t(R & 7);    // 128-byte swizzle: chunk ^ (row & 7)
        st_shared_v4(rb + ((j0 ^ x) << 4), f[0], f[1], f[2], f[3]);
        st_shared_v4(rb + (((j0 + 1) ^ x) << 4), f[4], f[5], f[6], f[7]);
    }
}

// Two bf16 (lower half first) -> two f16, rounded to nearest and saturated at +-65504.
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w) {
    uint32_t r;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;"
        : "=r"(r)
        : "f"(__uint_as_float(w & 0xFFFF0000u)), "f"(__uint_as_float(w << 16)));
    return r;
}
__device__ __forceinline__ void st_shared_zero16(uint32_t addr) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0) : "memory");
}

}  // namespace
