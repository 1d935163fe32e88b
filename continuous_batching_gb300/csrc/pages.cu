// Copies of pages within the pools of all layers: what a fork's first writes (pa_alloc_cow) and a
// compaction (pa_alloc_compact) ask for.
//
// A page is a pool's bytes of one block, whatever it holds (bf16, e4m3 or 4-bit codes). A warp takes
// kChunk bytes of one page of one pool at a time, all of its loads in flight before its first store, so an SM
// has about 128 KB on the way; consecutive warps take consecutive chunks of a page. Bound by memory: each byte
// is read and written once (701 pages of 32 KB in 16 pools: 109.9 us, 6.7 TB/s, 98 % of a copy's rate; 6 in 64 pools 3.9 us
// in a graph, and 32 to 35 as a call of the Python binding, which looks at 64 tensors).
#include <cuda_runtime.h>

#include <algorithm>

#include "common.h"

using namespace pa_detail;

namespace {

constexpr int kThreads = 256;
constexpr int kLoads = 4;                          // 16-byte loads of a lane
constexpr int kChunk = 32 * 16 * kLoads;
constexpr int kPools = 128;                        // of one launch: its parameters hold their addresses

struct Pages {
    pa_pages pool[kPools];
    const int32_t* pairs;
    int32_t* err;
    int32_t n_pairs, num_blocks;
    int32_t chunks;                                // of the largest page
    int64_t units;                                 // pools * pairs * chunks
};

__global__ void __launch_bounds__(kThreads) copy_pages_kernel(const __grid_constant__ Pages p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int64_t step = int64_t(gridDim.x) * (kThreads / 32);
    for (int64_t u = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); u < p.units; u += step) {
        const int64_t w = u / p.chunks;
        const int chunk = int(u - w * p.chunks);
        const int pool = int(w / p.n_pairs);
        const int64_t pair = w - int64_t(pool) * p.n_pairs;
        const int64_t bytes = p.pool[pool].page_bytes;
        const int64_t first = int64_t(chunk) * kChunk;
        if (first >= bytes) continue;              // a smaller page than the largest
        const int32_t from = p.pairs[2 * pair], to = p.pairs[2 * pair + 1];
        if (from < 0 || from >= p.num_blocks || to < 0 || to >= p.num_blocks || from == to) {
            if (lane == 0 && p.err) atomicOr(p.err, PA_DEVERR_BLOCK);
            continue;
        }
        uint8_t* const base = static_cast<uint8_t*>(p.pool[pool].pool) + first + 16 * lane;
        const uint8_t* src = base + from * bytes;
        uint8_t* dst = base + to * bytes;
        uint4 v[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            if (first + 512 * i + 16 * lane < bytes) v[i] = __ldcs(reinterpret_cast<const uint4*>(src + 512 * i));
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            if (first + 512 * i + 16 * lane < bytes) *reinterpret_cast<uint4*>(dst + 512 * i) = v[i];
    }
}

}  // namespace

extern "C" int32_t paged_copy_pages(const int32_t* pairs, int32_t n_pairs, const pa_pages* pools,
                                    int32_t n_pools, int32_t num_blocks, int32_t* err_flag,
                                    pa_stream_t stream) {
    if (n_pairs < 0 || n_pools < 0 || num_blocks < 0 || (n_pools > 0 && !pools)) return PA_ERR_INVALID;
    for (int32_t i = 0; i < n_pools; ++i)
        if (!pools[i].pool || (reinterpret_cast<uintptr_t>(pools[i].pool) & 15) ||
            pools[i].page_bytes <= 0 || pools[i].page_bytes % 16)
            return PA_ERR_INVALID;
    for (int32_t i = 0; i < n_pools; ++i)
        if (pools[i].page_bytes > (int64_t(1) << 40)) return PA_ERR_SHAPE;
    if (n_pairs == 0 || n_pools == 0) return PA_OK;
    if (!pairs) return PA_ERR_INVALID;
    for (int32_t at = 0; at < n_pools; at += kPools) {
        const int32_t n = std::min(n_pools - at, kPools);
        Pages p{};
        int64_t largest = 0;
        for (int32_t i = 0; i < n; ++i) {
            p.pool[i] = pools[at + i];
            largest = std::max(largest, pools[at + i].page_bytes);
        }
        p.pairs = pairs;
        p.err = err_flag;
        p.n_pairs = n_pairs;
        p.num_blocks = num_blocks;
        p.chunks = int32_t((largest + kChunk - 1) / kChunk);
        p.units = int64_t(n) * n_pairs * p.chunks;
        const int64_t blocks = (p.units + kThreads / 32 - 1) / (kThreads / 32);
        cudaLaunchAttribute pdl[1];
        pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        pdl[0].val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(unsigned(std::min<int64_t>(blocks, int64_t(1) << 30)));
        cfg.blockDim = dim3(kThreads);
        cfg.stream = stream;
        cfg.attrs = pdl;
        cfg.numAttrs = 1;
        const int32_t st = note_cuda(cudaLaunchKernelEx(&cfg, copy_pages_kernel, p));
        if (st) return st;
    }
    return PA_OK;
}
