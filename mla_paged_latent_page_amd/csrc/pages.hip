// Page upkeep of a paged cache: copies of pages, forks of requests, compaction of
// accepted rows, and the return of pages without references.  Bit copies of 16-byte
// pieces over all layers and kv halves; every kernel is bound by memory or, for a few
// rows, by its chain of index loads.  Forking 16 parents to 112 children in 16 layers:
// 30 us for 278 MB (children of one parent read its page from the caches); a few beams: 3.5 us.
// Freeing: 5 to 11 us for the references, one compare-and-swap per page, and the walk over all
// counts by one workgroup, which keeps the list in order: 3.5 us for pools of 300 pages; both kernels
// 6, 14 and 95 us for 8 requests of 16 pages in pools of 300, 20,000 and 200,000.
#include <algorithm>

#include "step.hpp"

namespace mla {
namespace {

constexpr uint32_t kNoPage = 0xFFFFFFFFu;
constexpr uint32_t kJustFreed = 0x80000000u;   // a count that reached 0 in this call

// Copy the first `rows` token rows (and their scales) of page src to page dst in one
// layer and kv half (z = layer * kvs + kv), the block taking pieces part, part + parts, ...
__device__ inline void copy_page_rows(const PageArgs& a, uint32_t src, uint32_t dst, uint32_t z, uint32_t rows,
                                      uint32_t part, uint32_t parts)
{
    const uint32_t layer = z / a.kvs, kv = z - layer * a.kvs;
    const int64_t plane = (int64_t)layer * a.sl + (int64_t)kv * a.sk;
    const char* s = a.pool + (int64_t)src * a.sp + plane;
    char* d = a.pool + (int64_t)dst * a.sp + plane;
    const uint32_t G = (uint32_t)a.granules, total = rows * G;   // page_size * granules < 2^31
    constexpr int U = 4;
    for (uint32_t i = part * (U * 256) + threadIdx.x; i < total; i += parts * (U * 256)) {
        u32x4 v[U];
        int64_t o[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t k = min(i + u * 256, total - 1);
            const uint32_t r = k / G;
            o[u] = (int64_t)r * a.st + (int64_t)(k - r * G) * 16;
            v[u] = ld16(s + o[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u * 256 < total)
                st16(d + o[u], v[u]);
    }
    if (a.scales && part == 0) {
        const int64_t splane = (int64_t)layer * a.ssl + (int64_t)kv * a.ssk;
        const float* ss = a.scales + (int64_t)src * a.ssp + splane;
        float* sd = a.scales + (int64_t)dst * a.ssp + splane;
        const uint32_t n = rows * (uint32_t)a.nblk;
        for (uint32_t i = threadIdx.x; i < n; i += 256) {
            const uint32_t r = i / (uint32_t)a.nblk;
            const int64_t at = (int64_t)r * a.sst + (i - r * (uint32_t)a.nblk);
            sd[at] = ss[at];
        }
    }
}

// Grid: (parts of a page, layer x kv, pair).
__global__ void __launch_bounds__(256) copy_pages_kernel(PageArgs a)
{
    const uint32_t src = a.a[blockIdx.z], dst = a.b[blockIdx.z];
    if (src >= a.num_pages || dst >= a.num_pages || src == dst)
        return;
    for (uint32_t z = blockIdx.y; z < a.layers * a.kvs; z += gridDim.y)
        copy_page_rows(a, src, dst, z, a.page_size, blockIdx.x, gridDim.x);
}

// Grid: (parts of a page, layer x kv, pair).  The first block of a pair also does its
// table row, its counts (integer atomics: any order gives the same) and its length;
// nothing that another block of the call reads is written (no child is a parent).
__global__ void __launch_bounds__(256) fork_kernel(PageArgs a)
{
    const uint32_t parent = a.a[blockIdx.z], child = a.b[blockIdx.z];
    if (parent >= a.batch || child >= a.batch || parent == child)
        return;
    const uint64_t room = (uint64_t)a.max_pages * a.page_size;
    const uint32_t len = (uint32_t)min((uint64_t)a.cache_len[parent], room);
    const uint32_t full = len / a.page_size, part = len - full * a.page_size;
    const uint32_t fresh = part ? a.c[blockIdx.z] : kNoPage;
    if (part && fresh >= a.num_pages)
        return;
    const uint32_t* from = a.page_table + (size_t)parent * a.max_pages;
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        uint32_t* to = a.page_table + (size_t)child * a.max_pages;
        for (uint32_t i = threadIdx.x; i < full; i += 256) {
            const uint32_t pg = from[i];
            to[i] = pg;
            if (pg < a.num_pages)
                atomicAdd(a.refs + pg, 1u);
        }
        if (threadIdx.x == 0) {
            if (part) {
                to[full] = fresh;
                a.refs[fresh] = 1u;
            }
            a.cache_len[child] = len;
        }
    }
    if (part) {
        const uint32_t src = from[full];
        if (src < a.num_pages && src != fresh)
            for (uint32_t z = blockIdx.y; z < a.layers * a.kvs; z += gridDim.y)
                copy_page_rows(a, src, fresh, z, part, blockIdx.x, gridDim.x);
    }
}

// One block per listed request; the first listing of a request frees it.
__global__ void __launch_bounds__(256) free_requests_kernel(PageArgs a)
{
    const uint32_t req = a.a[blockIdx.x];
    if (req >= a.batch)
        return;
    __shared__ int again;
    if (threadIdx.x == 0)
        again = 0;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < blockIdx.x; i += 256)
        if (a.a[i] == req)
            again = 1;
    __syncthreads();
    if (again)
        return;
    const uint64_t room = (uint64_t)a.max_pages * a.page_size;
    const uint64_t len = min((uint64_t)a.cache_len[req], room);
    const uint32_t pages = (uint32_t)((len + a.page_size - 1) / a.page_size);
    uint32_t* row = a.page_table + (size_t)req * a.max_pages;
    for (uint32_t i = threadIdx.x; i < pages; i += 256) {
        const uint32_t pg = row[i];
        row[i] = kNoPage;
        if (pg >= a.num_pages)
            continue;
        // The last holder leaves the mark that collect_kernel looks for; a count of 0
        // (marked or not) stays as it is.
        uint32_t old = a.refs[pg];
        while (old != 0 && old != kJustFreed) {
            const uint32_t want = old == 1 ? kJustFreed : old - 1;
            const uint32_t got = atomicCAS(a.refs + pg, old, want);
            if (got == old)
                break;
            old = got;
        }
    }
    __syncthreads();   // every thread has read the length
    if (threadIdx.x == 0)
        a.cache_len[req] = 0;
}

// One block walks the counts in order, 16 per thread and step, and appends the marked
// pages: the list does not depend on the order in which the references went.  (num_pages is
// below 2^31: neither the walk nor the sums wrap.)
constexpr int COLLECT_THREADS = 1024, COLLECT_EACH = 16;
__global__ void __launch_bounds__(COLLECT_THREADS) collect_kernel(PageArgs a)
{
    __shared__ uint32_t wave_sum[COLLECT_THREADS / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t base = min(a.free_count[0], a.num_pages);
    for (uint32_t p0 = 0; p0 < a.num_pages; p0 += COLLECT_THREADS * COLLECT_EACH) {
        const uint32_t first = p0 + threadIdx.x * COLLECT_EACH;
        uint32_t marks = 0;
#pragma unroll
        for (int i = 0; i < COLLECT_EACH; ++i)
            if (first + i < a.num_pages && a.refs[first + i] == kJustFreed)
                marks |= 1u << i;
        const uint32_t mine = (uint32_t)__popc(marks);
        uint32_t scan = mine;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t up = __shfl_up(scan, d);
            scan += lane >= d ? up : 0u;
        }
        if (lane == 63)
            wave_sum[wave] = scan;
        __syncthreads();
        uint32_t before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < COLLECT_THREADS / 64; ++w) {
            before += w < wave ? wave_sum[w] : 0u;
            all += wave_sum[w];
        }
        uint32_t at = base + before + scan - mine;
        while (marks) {
            const uint32_t pg = first + (uint32_t)__ffs(marks) - 1;
            marks &= marks - 1;
            a.refs[pg] = 0;
            if (at < a.num_pages)
                a.free_list[at] = pg;
            ++at;
        }
        base += all;
        __syncthreads();
    }
    if (threadIdx.x == 0)
        a.free_count[0] = min(base, a.num_pages);
}

// The value that lane k holds, in a scalar register.
__device__ inline uint32_t lane_of(uint32_t v, int k) { return (uint32_t)__builtin_amdgcn_readlane((int)v, k); }

// Page and slot of position p of request b; no page if it has none.  (Always loads: two calls
// side by side then wait once.)  A length and a token's index are 32 bits each, their sum is not.
__device__ inline void slot_of(const PageArgs& a, uint32_t b, uint64_t p, uint32_t& page, uint32_t& slot)
{
    const bool there = p < (uint64_t)a.max_pages * a.page_size;
    const uint64_t q = there ? p : 0u;
    const uint32_t lp = q >> 32 ? (uint32_t)(q / a.page_size) : (uint32_t)q / a.page_size;
    const uint32_t pg = a.page_table[(size_t)b * a.max_pages + lp];
    page = there && pg < a.num_pages ? pg : kNoPage;
    slot = (uint32_t)q - lp * a.page_size;
}

// A wave owns 64 16-byte columns (or scales) of one request, layer and kv half and moves them
// for the accepted rows in ascending order, eight rows at a time: all eight are read before the
// first is stored, and a later source a[k] >= k is never an earlier destination i < k, so no
// lane has to wait for another.  The pages and slots of 64 rows are looked up at once, one row
// per lane.  Few rows are bound by the chain of loads (offsets, accepted list, page table, then
// one round per eight rows): 8 requests, 4 layers 4.1 us, 128 requests, 24 layers of an e4m3 cache
// 6.8 us; 40 of 60 drafted rows of 64 requests in 24 bf16 layers move at 5.2 TB/s (27 us).
// Grid: (columns, layer x kv, request).
constexpr int COMPACT_THREADS = 64;
template <bool SCALES>
__global__ void __launch_bounds__(COMPACT_THREADS) compact_kernel(PageArgs a)
{
    constexpr int U = 8;
    const int lane = threadIdx.x;
    const int col = blockIdx.x * COMPACT_THREADS + lane;
    const bool in_row = col < a.granules, in_scales = SCALES && !in_row && col < a.granules + a.nblk;
    const int row_col = min(col, a.granules - 1), scale_col = max(min(col - a.granules, a.nblk - 1), 0);
    for (uint32_t b = blockIdx.z; b < a.batch; b += gridDim.z) {
        const uint32_t total = (uint32_t)a.count;
        const uint32_t lo = min(a.b[b], total), hi = min(a.b[b + 1], total);
        const uint64_t len = a.cache_len[b];
        for (uint32_t i0 = lo; i0 < hi; i0 += 64) {
            const int n = (int)min(hi - i0, 64u);
            const uint32_t i = i0 - lo + lane, from = a.a[i0 + min(lane, n - 1)];
            uint32_t from_page, from_slot, to_page, to_slot;
            slot_of(a, b, len + from, from_page, from_slot);
            slot_of(a, b, len + i, to_page, to_slot);
            const uint64_t moves = __ballot(lane < n && from != i && from_page != kNoPage && to_page != kNoPage);
            for (uint32_t z = blockIdx.y; z < a.layers * a.kvs; z += gridDim.y) {
                const int64_t layer = z / a.kvs, kv = z % a.kvs;
                char* rows = a.pool + layer * a.sl + kv * a.sk + (int64_t)row_col * 16;
                float* scales = a.scales + layer * a.ssl + kv * a.ssk + scale_col;
                for (int k0 = 0; k0 < n; k0 += U) {
                    // Every lane loads in every round (a branch would wait for the loads before
                    // it); rows without a move read the pool's first one.
                    u32x4 v[U];
                    float s[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const bool move = moves >> (k0 + u) & 1;
                        const int64_t page = move ? lane_of(from_page, k0 + u) : 0u;
                        const int64_t slot = move ? lane_of(from_slot, k0 + u) : 0u;
                        v[u] = ld16(rows + page * a.sp + slot * a.st);
                        if constexpr (SCALES)
                            s[u] = scales[page * a.ssp + slot * a.sst];
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        if (!(moves >> (k0 + u) & 1))
                            continue;
                        const int64_t page = lane_of(to_page, k0 + u), slot = lane_of(to_slot, k0 + u);
                        if (in_row)
                            st16(rows + page * a.sp + slot * a.st, v[u]);
                        if (in_scales)
                            scales[page * a.ssp + slot * a.sst] = s[u];
                    }
                }
            }
        }
    }
}

constexpr unsigned kMaxGridYZ = 65535;

unsigned page_parts(const PageArgs& a)
{
    const int64_t pieces = (int64_t)a.page_size * a.granules;
    return (unsigned)std::min<int64_t>((pieces + 1023) / 1024, 64);
}

}  // namespace

hipError_t launch_copy_pages(const PageArgs& a, hipStream_t s)
{
    const unsigned planes = a.layers * a.kvs;
    for (int i0 = 0; i0 < a.count; i0 += kMaxGridYZ) {
        PageArgs c = a;
        c.a += i0;
        c.b += i0;
        c.count = std::min(a.count - i0, (int)kMaxGridYZ);
        const dim3 grid(page_parts(a), std::min(planes, kMaxGridYZ), c.count);
        log_launch("copy_pages_kernel", grid.x * grid.y * grid.z, 256, "count=%d", c.count);
        hipLaunchKernelGGL(copy_pages_kernel, grid, dim3(256), 0, s, c);
        if (hipError_t e = hipGetLastError())
            return e;
    }
    return hipSuccess;
}

hipError_t launch_fork(const PageArgs& a, hipStream_t s)
{
    for (int i0 = 0; i0 < a.count; i0 += kMaxGridYZ) {
        PageArgs c = a;
        c.a += i0;
        c.b += i0;
        c.c += i0;
        c.count = std::min(a.count - i0, (int)kMaxGridYZ);
        const dim3 grid(page_parts(a), std::min((unsigned)(a.layers * a.kvs), kMaxGridYZ), c.count);
        log_launch("fork_kernel", grid.x * grid.y * grid.z, 256, "count=%d", c.count);
        hipLaunchKernelGGL(fork_kernel, grid, dim3(256), 0, s, c);
        if (hipError_t e = hipGetLastError())
            return e;
    }
    return hipSuccess;
}

hipError_t launch_free(const PageArgs& a, hipStream_t s)
{
    log_launch("free_requests_kernel", a.count, 256, "count=%d", a.count);
    hipLaunchKernelGGL(free_requests_kernel, dim3(a.count), dim3(256), 0, s, a);
    if (hipError_t e = hipGetLastError())
        return e;
    log_launch("collect_kernel", 1, COLLECT_THREADS, "pages=%u", a.num_pages);
    hipLaunchKernelGGL(collect_kernel, dim3(1), dim3(COLLECT_THREADS), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_compact(const PageArgs& a, hipStream_t s)
{
    const unsigned cols = (a.granules + a.nblk + COMPACT_THREADS - 1) / COMPACT_THREADS;
    const dim3 grid(cols, std::min((unsigned)(a.layers * a.kvs), kMaxGridYZ), std::min(a.batch, kMaxGridYZ));
    log_launch("compact_kernel", grid.x * grid.y * grid.z, COMPACT_THREADS, "accepted=%d batch=%u", a.count, a.batch);
    auto* kernel = a.scales ? compact_kernel<true> : compact_kernel<false>;
    hipLaunchKernelGGL(kernel, grid, dim3(COMPACT_THREADS), 0, s, a);
    return hipGetLastError();
}

}  // namespace mla
