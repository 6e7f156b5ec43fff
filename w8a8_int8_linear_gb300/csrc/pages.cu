// Pages of a cache: copies of pages, and forks of sequences, in all layers'
// caches at once.
//
// A page is copied in parts of 16 KB, a CTA each: bytes bound it, and every
// thread has four 16-byte loads in flight before its stores.  The indices stay on
// the device; one that is not in the cache moves nothing.  150 pages of 64 KB in 16
// caches take 48 us (0.98 of the copy bandwidth), 15 forks of one 128 KB page in 32
// caches 13, a few small pages 1.7.
#include <cuda_runtime.h>

#include <cstdint>

#include "operators.h"

namespace w8a8 {

namespace {

constexpr int kThreads = 256;
constexpr int kAtOnce = 4;
constexpr int64_t kPart = kThreads * kAtOnce * 16;

// Part `part` of page src of a cache to page dst.
__device__ __forceinline__ void copy_part(const PageCaches& c, int cache, int src, int dst, int64_t part) {
    uint8_t* base = static_cast<uint8_t*>(c.base[cache]);
    const uint8_t* from = base + src * c.stride[cache];
    uint8_t* to = base + dst * c.stride[cache];
    const int64_t at = part * kPart + threadIdx.x * 16;
    uint4 w[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
        if (at + i * kThreads * 16 < c.page_bytes)
            w[i] = *reinterpret_cast<const uint4*>(from + at + i * kThreads * 16);
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
        if (at + i * kThreads * 16 < c.page_bytes) *reinterpret_cast<uint4*>(to + at + i * kThreads * 16) = w[i];
}

__device__ __forceinline__ bool inside(int i, int n) { return static_cast<unsigned>(i) < static_cast<unsigned>(n); }

// blockIdx.x: parts of the pages of all caches, a page's side by side
__global__ void __launch_bounds__(kThreads)
    copy_pages_kernel(const __grid_constant__ PageCaches c, const int* src, const int* dst, int64_t first) {
    const unsigned parts = static_cast<unsigned>((c.page_bytes + kPart - 1) / kPart);
    const unsigned page = blockIdx.x / parts, cache = page % c.count;
    const int64_t i = first + page / c.count;
    const int s = src[i], d = dst[i];
    if (inside(s, c.pages) && inside(d, c.pages) && s != d) copy_part(c, cache, s, d, blockIdx.x % parts);
}

// the same for the pairs' last pages, and for each pair a CTA for its row of the table
__global__ void __launch_bounds__(kThreads)
    fork_kernel(const __grid_constant__ PageCaches c, const ForkArgs f, int64_t first) {
    const unsigned parts = static_cast<unsigned>((c.page_bytes + kPart - 1) / kPart);
    const unsigned copies = parts * c.count, of_pair = copies + f.tables;
    const int64_t i = first + blockIdx.x / of_pair;
    const unsigned what = blockIdx.x % of_pair;
    const int src = f.src[i], dst = f.dst[i], page = f.page[i];
    if (!inside(src, f.rows) || !inside(dst, f.rows) || src == dst || !inside(page, c.pages)) return;
    const int len = min(max(f.k_lens[src], 0), f.max_pages * f.page_size), full = len / f.page_size;
    const int* row = f.table + src * f.table_stride;
    if (what < copies) {
        if (len % f.page_size == 0) return;
        const int from = row[full];
        if (inside(from, c.pages) && from != page) copy_part(c, what / parts, from, page, what % parts);
        return;
    }
    int* to = f.table + dst * f.table_stride;
    for (int k = threadIdx.x; k < min(full + 1, f.max_pages); k += kThreads) to[k] = k < full ? row[k] : page;
    if (threadIdx.x == 0) f.k_lens[dst] = len;
}

// Launches of at most 2^31 - 1 CTAs over n pairs.
template <typename F>
cudaError_t over_pairs(int64_t n, int64_t ctas_of_pair, F launch) {
    const int64_t most = 0x7FFFFFFF / ctas_of_pair;
    for (int64_t first = 0; first < n; first += most) {
        const int64_t pairs = n - first < most ? n - first : most;
        launch(static_cast<unsigned>(pairs * ctas_of_pair), first);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

int64_t parts_of(const PageCaches& c) { return (c.page_bytes + kPart - 1) / kPart; }

}  // namespace

cudaError_t launch_copy_pages(const PageCaches& c, const int* src, const int* dst, int64_t n, cudaStream_t st) {
    return over_pairs(n, parts_of(c) * c.count, [&](unsigned grid, int64_t first) {
        copy_pages_kernel<<<grid, kThreads, 0, st>>>(c, src, dst, first);
    });
}

cudaError_t launch_fork_sequences(const PageCaches& c, const ForkArgs& f, cudaStream_t st) {
    return over_pairs(f.n, parts_of(c) * c.count + f.tables, [&](unsigned grid, int64_t first) {
        fork_kernel<<<grid, kThreads, 0, st>>>(c, f, first);
    });
}

}  // namespace w8a8
