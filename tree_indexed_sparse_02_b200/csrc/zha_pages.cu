// zha_pages.cu -- zha_paged_plan: block tables, slot maps and lengths of one
// step from the requests' lengths.
//
// Everything follows from three prefix sums over the sequences: pages that
// come back, new tokens, new pages. Each CTA of one thread-block cluster
// forms them for itself in shared memory (a few loads per sequence), then the
// cluster's threads walk the returned pages, the new pages and the token rows
// as flat lists, finding an element's sequence by bisection. One cluster
// barrier orders the pushes onto the free stack before the pops and lets the
// lengths be updated in place. Bound by latency: a chain of three dependent
// loads, two scans and the barrier. B200, per launch in a graph: 64 requests of
// one token 6.5 us with 1, 8 or 16 CTAs; 700 requests with 44,507 tokens 12.1 us
// with 8, 9.1 us with 16 (one CTA of an earlier form: 57 us).
#include <cooperative_groups.h>

#include "zha_paged.h"

namespace cg = cooperative_groups;

namespace zha {

namespace {

constexpr int kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;
constexpr int kRun = 4;                  // token rows a thread writes at a time
// Sums stop here: more than any pool or token buffer holds, and two of them fit 32 bits.
constexpr uint32_t kMany = (1u << 30) + 1;

__device__ __forceinline__ uint32_t add(uint32_t x, uint32_t y) { return min(x + y, kMany); }
__device__ __forceinline__ uint2 add(uint2 x, uint2 y) { return make_uint2(add(x.x, y.x), add(x.y, y.y)); }
__device__ __forceinline__ uint2 up(uint2 x, int o) {
    return make_uint2(__shfl_up_sync(0xffffffffu, x.x, o), __shfl_up_sync(0xffffffffu, x.y, o));
}
__device__ __forceinline__ uint2 warp_scan(uint2 x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint2 y = up(x, o);
        if (lane >= o) x = add(x, y);
    }
    return x;
}

// Sums of two values per thread over the threads before it, and over all of them. `sums` is this scan's own.
__device__ __forceinline__ uint2 block_scan(uint2 v, uint2 *sums, uint2 &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint2 x = warp_scan(v, lane);
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    const uint2 w = warp_scan(sums[lane], lane);
    total = make_uint2(__shfl_sync(0xffffffffu, w.x, 31), __shfl_sync(0xffffffffu, w.y, 31));
    // exclusive: the warps before this one, then the lanes before this one
    uint2 before = make_uint2(__shfl_sync(0xffffffffu, w.x, (warp + 31) & 31), __shfl_sync(0xffffffffu, w.y, (warp + 31) & 31));
    if (warp == 0) before = make_uint2(0, 0);
    uint2 lanes = up(x, 1);
    if (lane == 0) lanes = make_uint2(0, 0);
    return add(before, lanes);
}

constexpr uint32_t kUnserved = 0x80000000u;      // of need_pre: this sequence is not served

// Last b in [0, n) with pre[b] <= x, marks aside (pre ascends, pre[0] = 0).
__device__ __forceinline__ int find(const uint32_t *pre, int n, uint32_t x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((pre[mid] & ~kUnserved) <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads, 1) paged_plan_kernel(const __grid_constant__ PlanArgs a) {
    extern __shared__ uint32_t sm[];
    __shared__ uint2 sums[2][kPlanWarps];
    __shared__ uint32_t sh_taken;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int B = a.B, lps = a.lps, ps = 1 << lps;
    int *len = reinterpret_cast<int *>(sm);
    uint32_t *back_pre = sm + B, *tok_pre = back_pre + B, *need_pre = tok_pre + B;   // sums over earlier sequences
    if (threadIdx.x == 0) sh_taken = 0;

    pdl_wait();
    const int n_free = *a.n_free;
    const int64_t cap = (int64_t)a.max_pages << lps;
    const int per = (B + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min((int)threadIdx.x * per, B), b1 = min(b0 + per, B);
    auto valid = [&](int l) { return l >= 0 && l <= cap; };
    auto pages = [&](int n) { return (int)(((uint32_t)n + ps - 1) >> lps); };

    uint2 own = make_uint2(0, 0), total;                           // pages that come back, new tokens
    for (int b = b0; b < b1; ++b) {
        const int n = a.n_new[b], l = a.lens[b];
        len[b] = l;
        if (!valid(l)) set_status(a.status, ZHA_ERR_INVALID_ARG);
        own = add(own, make_uint2(n < 0 && valid(l) ? pages(l) : 0, min((uint32_t)max(n, 0), kMany)));
    }
    const uint2 pre = block_scan(own, sums[0], total);
    const bool pool_ok = n_free >= 0 && n_free <= a.n_pages && n_free + total.x <= (uint32_t)a.n_pages;
    if (!pool_ok && threadIdx.x == 0) set_status(a.status, ZHA_ERR_INVALID_ARG);
    const uint32_t have = pool_ok ? n_free + total.x : 0;
    // pages a sequence of l tokens asks for with n more that end at row tok_end; -1: it cannot be served
    auto wants = [&](int l, int n, uint32_t tok_end) {
        if (!pool_ok || !valid(l) || n < 0 || l + (int64_t)n > cap || tok_end > (uint32_t)a.max_tokens) return -1;
        return pages(l + n) - pages(l);
    };
    uint2 at = pre;
    uint32_t need = 0;
    for (int b = b0; b < b1; ++b) {
        const int n = a.n_new[b], l = len[b];
        back_pre[b] = at.x;
        tok_pre[b] = at.y;
        at = add(at, make_uint2(n < 0 && valid(l) ? pages(l) : 0, min((uint32_t)max(n, 0), kMany)));
        need = add(need, (uint32_t)max(wants(l, n, at.y), 0));
    }
    uint2 total_need;
    uint32_t np = block_scan(make_uint2(need, 0), sums[1], total_need).x;
    uint32_t top_need = 0, end = pre.y;
    for (int b = b0; b < b1; ++b) {
        const int n = a.n_new[b], l = len[b];
        end = add(end, min((uint32_t)max(n, 0), kMany));
        const int w = wants(l, n, end);
        const bool served = w == 0 || (w > 0 && np + w <= have);
        need_pre[b] = np | (served ? 0 : kUnserved);
        np = add(np, (uint32_t)max(w, 0));
        if (served) top_need = w > 0 ? np : top_need;
        else if (n > 0 && valid(l)) set_status(a.status, pool_ok ? ZHA_ERR_CAPACITY : ZHA_ERR_INVALID_ARG);
    }
    // who is served is a prefix of those who ask for pages: their need is its largest sum
    top_need = __reduce_max_sync(0xffffffffu, top_need);
    if ((threadIdx.x & 31) == 0 && top_need) atomicMax(&sh_taken, top_need);
    __syncthreads();
    const uint32_t taken = sh_taken;

    const int gt = rank * kPlanThreads + threadIdx.x, gn = ranks * kPlanThreads;
    if (pool_ok)
        for (uint32_t j = gt; j < total.x; j += gn) {              // pages that come back
            const int b = find(back_pre, B, j);
            const int page = a.table[(int64_t)b * a.max_pages + (j - back_pre[b])];
            if ((unsigned)page >= (unsigned)a.n_pages) set_status(a.status, ZHA_ERR_INVALID_ARG);
            a.free_pages[n_free + j] = page;
        }
    // pushes before pops; and every CTA has read the lengths before one of them writes the new ones
    cluster.sync();

    const int32_t *top = a.free_pages + (int)have - 1;
    for (uint32_t j = gt; j < taken; j += gn) {                    // new pages
        const int b = find(need_pre, B, j);
        const int page = __ldcg(top - j);
        if ((unsigned)page >= (unsigned)a.n_pages) set_status(a.status, ZHA_ERR_INVALID_ARG);
        a.table[(int64_t)b * a.max_pages + pages(len[b]) + (j - need_pre[b])] = page;
    }
    // token rows, a run of kRun per thread: neighbours are mostly of one sequence and one page
    const uint32_t tokens = min(total.y, (uint32_t)a.max_tokens);
    const bool vec = ((reinterpret_cast<uintptr_t>(a.positions) | reinterpret_cast<uintptr_t>(a.slots) |
                       reinterpret_cast<uintptr_t>(a.seq_ids)) & 15u) == 0;
    const int runs = (a.max_tokens - 1) / kRun + 1;
    for (int r = gt; r < runs; r += gn) {
        const uint32_t i0 = (uint32_t)r * kRun;
        int pos[kRun], slot[kRun], seq[kRun];
        int b = i0 < tokens ? find(tok_pre, B, i0) : B, col = -1, page = -1;
        uint32_t next = b + 1 < B ? tok_pre[b + 1] : kMany;
#pragma unroll
        for (int u = 0; u < kRun; ++u) {
            const uint32_t i = i0 + u;
            pos[u] = 0;
            slot[u] = seq[u] = -1;
            if (i >= tokens) continue;
            while (i >= next) {
                ++b;
                next = b + 1 < B ? tok_pre[b + 1] : kMany;
                col = -1;
            }
            if (need_pre[b] & kUnserved) continue;
            const int p = len[b] + (int)(i - tok_pre[b]), c = p >> lps;
            if (c != col) {
                const int old = pages(len[b]);
                col = c;
                page = c < old ? a.table[(int64_t)b * a.max_pages + c] : __ldcg(top - (need_pre[b] + (c - old)));
                if ((unsigned)page >= (unsigned)a.n_pages) set_status(a.status, ZHA_ERR_INVALID_ARG);
            }
            if ((unsigned)page >= (unsigned)a.n_pages) continue;
            pos[u] = p;
            slot[u] = (page << lps) | (p & (ps - 1));
            seq[u] = b;
        }
        if (vec && i0 + kRun <= (uint32_t)a.max_tokens) {
            reinterpret_cast<int4 *>(a.positions)[r] = make_int4(pos[0], pos[1], pos[2], pos[3]);
            reinterpret_cast<int4 *>(a.slots)[r] = make_int4(slot[0], slot[1], slot[2], slot[3]);
            reinterpret_cast<int4 *>(a.seq_ids)[r] = make_int4(seq[0], seq[1], seq[2], seq[3]);
        } else {
#pragma unroll
            for (int u = 0; u < kRun; ++u)
                if (i0 + u < (uint32_t)a.max_tokens) {
                    a.positions[i0 + u] = pos[u];
                    a.slots[i0 + u] = slot[u];
                    a.seq_ids[i0 + u] = seq[u];
                }
        }
    }
    if (rank == 0) {
        for (int b = b0; b < b1; ++b) {
            const int n = a.n_new[b], l = len[b];
            a.cu_new[b] = min(tok_pre[b], (uint32_t)a.max_tokens);
            a.lens_out[b] = !(need_pre[b] & kUnserved) ? l + n : (n < 0 && pool_ok && valid(l)) ? 0 : l;
        }
        if (threadIdx.x == 0) {
            a.cu_new[B] = tokens;
            *a.n_free_out = pool_ok ? (int)(have - taken) : n_free;
        }
    }
}

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs &a, cudaStream_t st) {
    const size_t smem = 4 * (size_t)a.B * sizeof(uint32_t);
    // 16 CTAs where such a cluster fits the device, else the portable 8
    static int ranks_of[64] = {};
    int dev = 0, ranks = 8;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && ranks_of[dev]) {
        ranks = ranks_of[dev];
    } else {
        const int most = 4 * kPagedMaxBatch * (int)sizeof(uint32_t);
        cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
        if (cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess) {
            cudaLaunchConfig_t q{};
            cudaLaunchAttribute at{};
            int fit = 0;
            q.gridDim = dim3(16);
            q.blockDim = dim3(kPlanThreads);
            q.dynamicSmemBytes = most;
            at.id = cudaLaunchAttributeClusterDimension;
            at.val.clusterDim.x = 16;
            at.val.clusterDim.y = at.val.clusterDim.z = 1;
            q.attrs = &at;
            q.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&fit, paged_plan_kernel, &q) == cudaSuccess && fit > 0) ranks = 16;
        }
        (void)cudaGetLastError();
        if (dev >= 0 && dev < 64) ranks_of[dev] = ranks;
    }
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(ranks);
    c.blockDim = dim3(kPlanThreads);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = ranks;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = 2;
    ProfScope ps("paged_plan", st);
    return cudaLaunchKernelEx(&c, paged_plan_kernel, a);
}

}  // namespace zha
