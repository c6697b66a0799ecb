// Pages of the K/V caches: copied (forks), moved with the block-table entries
// that name them (compaction), counted, and a request's row forked.
//
// All of it is indexed copying, bound by HBM: a page is read once and written
// once, 16 bytes per lane, and the tables are read in place.  One launch covers
// the pages of up to 32 layers' K and V.  Measured: 1500 pages of 32 KiB in 4
// layers' K and V with 1024 tables, 786 MB, 131 us (6.0 TB/s read and written); 24
// pages in 32 layers, 101 MB, 17 us.
#include <algorithm>

#include "ric_internal.h"

namespace ric {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;                                   // 16-byte loads in flight per lane
constexpr int64_t kChunkVec = (int64_t)kThreads * kUnroll;   // 16 KiB of a page per workgroup

__device__ __forceinline__ void copy_vec(const u32x4* in, u32x4* out, int64_t v0, int64_t n) {
    u32x4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t j = v0 + u * kThreads + threadIdx.x;
        if (j < n) v[u] = __builtin_nontemporal_load(in + j);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t j = v0 + u * kThreads + threadIdx.x;
        if (j < n) __builtin_nontemporal_store(v[u], out + j);
    }
}

}  // namespace

// blockIdx.y < 2 * layers: one 16 KiB piece of one page of one cache.  The last
// y: the block tables, one wave per row; each entry is looked up among the
// sorted sources (binary search in LDS) and replaced by its destination.  No
// destination is a source, so the order of pieces, rows and launches is free.
__global__ __launch_bounds__(kThreads) void page_copy_kernel(PageParams p, int chunks) {
    const int y = blockIdx.y;
    if (y < 2 * p.num_layers) {
        const int pair = blockIdx.x / chunks;
        if (pair >= p.num_pairs) return;
        const int64_t v0 = (int64_t)(blockIdx.x - pair * chunks) * kChunkVec;
        const uint8_t* base = (y & 1) ? p.vc[y >> 1] : p.kc[y >> 1];
        const u32x4* in = reinterpret_cast<const u32x4*>(base + (int64_t)p.pairs[2 * pair] * p.block_bytes);
        u32x4* out = reinterpret_cast<u32x4*>(const_cast<uint8_t*>(base) + (int64_t)p.pairs[2 * pair + 1] * p.block_bytes);
        copy_vec(in, out, v0, p.block_bytes >> 4);
        return;
    }
    extern __shared__ int32_t sources[];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int first = blockIdx.x * (kThreads / 64);
    if (first >= p.rows) return;
    for (int k = threadIdx.x; k < p.num_pairs; k += kThreads) sources[k] = p.pairs[2 * k];
    __syncthreads();
    for (int r = first + wave; r < p.rows; r += gridDim.x * (kThreads / 64)) {
        const int nb = min(p.num_blocks[r], (int)p.blk_stride);
        int32_t* row = p.blocks + (int64_t)r * p.blk_stride;
        for (int j = lane; j < nb; j += 64) {
            const int32_t id = row[j];
            int lo = 0, hi = p.num_pairs;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (sources[mid] < id) lo = mid + 1; else hi = mid;
            }
            if (lo < p.num_pairs && sources[lo] == id) row[j] = p.pairs[2 * lo + 1];
        }
    }
}

hipError_t launch_page_copy(const PageParams& p, hipStream_t s) {
    const int chunks = (int)((p.block_bytes / 16 + kChunkVec - 1) / kChunkVec);
    const int64_t copies = p.num_layers ? (int64_t)p.num_pairs * chunks : 0;
    const int64_t row_groups = ((int64_t)p.rows + 3) / 4;
    // a few pages of many requests: the tables still take up to 256 workgroups
    const int64_t x = copies > 0 ? std::max(copies, std::min<int64_t>(row_groups, 256)) : row_groups;
    if (p.num_pairs == 0 || x == 0) return hipSuccess;
    hipLaunchKernelGGL(page_copy_kernel, dim3((uint32_t)x, 2 * p.num_layers + (p.rows > 0 ? 1 : 0)), dim3(kThreads),
                       p.rows > 0 ? (size_t)p.num_pairs * 4 : 0, s, p, chunks > 0 ? chunks : 1);
    return hipGetLastError();
}

// Counts of table entries per page: cleared by a kernel (not a memset: the call
// may be captured), then one wave per row adds its entries.  Integer sums, so the
// order of the atomics does not matter.
__global__ __launch_bounds__(kThreads) void clear_refs_kernel(int32_t* refs, int32_t pool) {
    const int i = blockIdx.x * kThreads + threadIdx.x;
    if (i < pool) refs[i] = 0;
}

__global__ __launch_bounds__(kThreads) void count_refs_kernel(const int32_t* blocks, int64_t blk_stride,
                                                              const int32_t* num_blocks, int32_t rows, int32_t pool,
                                                              int32_t* refs) {
    const int r = blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
    if (r >= rows) return;
    const int nb = min(num_blocks[r], (int)blk_stride);
    for (int j = threadIdx.x & 63; j < nb; j += 64) {
        const int32_t id = blocks[(int64_t)r * blk_stride + j];
        if (id >= 0 && id < pool) atomicAdd(refs + id, 1);
    }
}

hipError_t launch_block_refs(const int32_t* blocks, int64_t blk_stride, const int32_t* num_blocks, int32_t rows,
                             int32_t pool, int32_t* refs, hipStream_t s) {
    hipLaunchKernelGGL(clear_refs_kernel, dim3((pool + kThreads - 1) / kThreads), dim3(kThreads), 0, s, refs, pool);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || rows == 0) return e;
    hipLaunchKernelGGL(count_refs_kernel, dim3((rows + 3) / 4), dim3(kThreads), 0, s, blocks, blk_stride, num_blocks,
                       rows, pool, refs);
    return hipGetLastError();
}

// blockIdx.y < 2 * layers: the valid rows of the parent's partly filled page.
// The last y (first launch only): the parent's history and shared page ids.
__global__ __launch_bounds__(kThreads) void fork_kernel(ForkParams p) {
    const int y = blockIdx.y;
    if (y < 2 * p.num_layers) {
        const int32_t src = p.blocks[(int64_t)p.parent * p.blk_stride + p.num_shared];
        const int64_t page = (int64_t)p.block_size * p.row_bytes;
        const int64_t n = (int64_t)p.tail_rows * p.row_bytes / 16;
        const int64_t v0 = (int64_t)blockIdx.x * kChunkVec;
        if (v0 >= n || src < 0 || src >= p.pool) return;
        uint8_t* base = (y & 1) ? p.vc[y >> 1] : p.kc[y >> 1];
        copy_vec(reinterpret_cast<const u32x4*>(base + src * page),
                 reinterpret_cast<u32x4*>(base + p.tail_block * page), v0, n);
        return;
    }
    const int step = gridDim.x * kThreads;
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < p.num_tokens; i += step)
        p.tokens[(int64_t)p.child * p.tok_stride + i] = p.tokens[(int64_t)p.parent * p.tok_stride + i];
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < p.num_shared; i += step)
        p.blocks[(int64_t)p.child * p.blk_stride + i] = p.blocks[(int64_t)p.parent * p.blk_stride + i];
}

hipError_t launch_fork(const ForkParams& p, bool rows, hipStream_t s) {
    const int64_t tail = ((int64_t)p.tail_rows * p.row_bytes / 16 + kChunkVec - 1) / kChunkVec;
    const int64_t x = std::max<int64_t>(p.num_layers ? tail : 0, rows ? std::min<int64_t>((p.num_tokens + 1023) / 1024, 64) : 0);
    hipLaunchKernelGGL(fork_kernel, dim3((uint32_t)std::max<int64_t>(x, 1), 2 * p.num_layers + (rows ? 1 : 0)),
                       dim3(kThreads), 0, s, p);
    return hipGetLastError();
}

}  // namespace ric
