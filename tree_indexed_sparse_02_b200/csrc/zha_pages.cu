// zha_pages.cu -- zha_paged_plan: block tables, slot maps and lengths of one
// step from the requests' lengths.
//
// Everything follows from three prefix sums over the sequences: pages that
// come back, new tokens, new pages. Every CTA of one thread-block cluster
// forms them for itself in shared memory (a few loads per sequence), then the
// cluster's threads walk the returned pages, the new pages and the token rows
// as flat lists, finding an element's sequence by bisection. The cluster
// barriers order the pushes onto the free stack before the pops and let the
// lengths be updated in place.
#include <cooperative_groups.h>

#include "zha_paged.cuh"

namespace cg = cooperative_groups;

namespace zha {

namespace {

constexpr int kPlanThreads = 1024;

__device__ __forceinline__ int saturate(int64_t x) { return x > 0x7fffffff ? 0x7fffffff : (int)x; }

// Exclusive prefix sum of one value per thread over the block, and the total.
__device__ int64_t block_scan(int64_t v, int64_t *warp_sums, int64_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int64_t base = 0, all = 0;
    for (int w = 0; w < nw; ++w) {
        const int64_t s = warp_sums[w];
        if (w < warp) base += s;
        all += s;
    }
    total = all;
    return base + x - v;
}

// Last b in [0, n) with pre[b] <= x (pre ascending, pre[0] <= x).
__device__ __forceinline__ int find(const int *pre, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(PlanArgs a) {
    extern __shared__ int sm[];
    __shared__ int64_t warp_sums[32];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int B = a.B, lps = a.lps, ps = 1 << lps;
    int *len = sm, *back_pre = len + B, *tok_pre = back_pre + B + 1, *need_pre = tok_pre + B + 1;
    // need_pre: low 31 bits the pages asked for by earlier sequences (ascending), sign bit: not served
    constexpr int kUnserved = (int)0x80000000;

    pdl_wait();
    const int n_free = *a.n_free;
    const int64_t cap = (int64_t)a.max_pages << lps;
    const int per = (B + blockDim.x - 1) / blockDim.x;
    const int b0 = min((int)threadIdx.x * per, B), b1 = min(b0 + per, B);
    auto valid = [&](int l) { return l >= 0 && l <= cap; };
    auto pages = [&](int64_t n) { return (int)((n + ps - 1) >> lps); };

    int64_t back = 0, toks = 0, total_back, total_tok;
    for (int b = b0; b < b1; ++b) {
        const int n = a.n_new[b], l = a.lens[b];
        len[b] = l;
        if (!valid(l)) set_status(a.status, ZHA_ERR_INVALID_ARG);
        else if (n < 0) back += pages(l);
        if (n > 0) toks += n;
    }
    int64_t bp = block_scan(back, warp_sums, total_back), tp = block_scan(toks, warp_sums, total_tok);
    const bool pool_ok = n_free >= 0 && n_free <= a.n_pages && n_free + total_back <= a.n_pages;
    if (!pool_ok && threadIdx.x == 0) set_status(a.status, ZHA_ERR_INVALID_ARG);
    // pages sequence b asks for, given the end of its token rows; -1: it cannot be served
    auto wants = [&](int l, int n, int64_t tok_end) {
        if (!pool_ok || !valid(l) || n < 0 || l + (int64_t)n > cap || tok_end > a.max_tokens) return -1;
        return pages(l + (int64_t)n) - pages(l);
    };
    int64_t need = 0, total_need, tq = tp;
    for (int b = b0; b < b1; ++b) {
        const int n = a.n_new[b];
        back_pre[b] = saturate(bp);
        tok_pre[b] = saturate(tq);
        if (n < 0 && valid(len[b])) bp += pages(len[b]);
        if (n > 0) tq += n;
        need += max(wants(len[b], n, tq), 0);
    }
    if (threadIdx.x == 0) tok_pre[B] = saturate(total_tok);
    int64_t np = block_scan(need, warp_sums, total_need);
    const int64_t have = pool_ok ? n_free + total_back : 0;
    int64_t taken = 0, total_taken;
    tq = tp;
    for (int b = b0; b < b1; ++b) {
        const int n = a.n_new[b];
        if (n > 0) tq += n;
        const int w = wants(len[b], n, tq);
        const bool served = w == 0 || (w > 0 && np + w <= have);
        need_pre[b] = saturate(np) | (served ? 0 : kUnserved);
        if (served) taken += w;
        else if (n > 0 && valid(len[b])) set_status(a.status, pool_ok ? ZHA_ERR_CAPACITY : ZHA_ERR_INVALID_ARG);
        np += max(w, 0);
    }
    block_scan(taken, warp_sums, total_taken);       // (ends with every thread past the writes above)
    __syncthreads();

    const int gt = rank * blockDim.x + threadIdx.x, gn = ranks * blockDim.x;
    if (pool_ok)
        for (int j = gt; j < (int)total_back; j += gn) {           // pages that come back
            const int b = find(back_pre, B, j);
            const int page = a.table[(int64_t)b * a.max_pages + (j - back_pre[b])];
            if ((unsigned)page >= (unsigned)a.n_pages) set_status(a.status, ZHA_ERR_INVALID_ARG);
            a.free_pages[n_free + j] = page;
        }
    // pushes before pops; and every CTA has read the lengths before one of them writes the new ones
    cluster.sync();

    const int top = (int)have - 1;
    auto need_of = [&](int b) { return need_pre[b] & ~kUnserved; };
    // the served sequences' needs are the first total_taken units of the prefix sum
    for (int j = gt; j < (int)total_taken; j += gn) {              // new pages
        int b = 0, hi = B;
        while (hi - b > 1) {
            const int mid = (b + hi) >> 1;
            if (need_of(mid) <= j) b = mid;
            else hi = mid;
        }
        const int page = __ldcg(a.free_pages + (top - j));
        if ((unsigned)page >= (unsigned)a.n_pages) set_status(a.status, ZHA_ERR_INVALID_ARG);
        a.table[(int64_t)b * a.max_pages + pages(len[b]) + (j - need_of(b))] = page;
    }
    for (int i = gt; i < a.max_tokens; i += gn) {                  // token rows
        int pos = 0, slot = -1, seq = -1;
        if (i < total_tok) {
            const int b = find(tok_pre, B, i);
            if (need_pre[b] >= 0) {
                const int p = len[b] + (i - tok_pre[b]), col = p >> lps, old = pages(len[b]);
                const int page = col < old ? a.table[(int64_t)b * a.max_pages + col]
                                           : __ldcg(a.free_pages + (top - (need_of(b) + col - old)));
                if ((unsigned)page < (unsigned)a.n_pages) {
                    pos = p;
                    slot = (page << lps) | (p & (ps - 1));
                    seq = b;
                } else {
                    set_status(a.status, ZHA_ERR_INVALID_ARG);
                }
            }
        }
        a.positions[i] = pos;
        a.slots[i] = slot;
        a.seq_ids[i] = seq;
    }
    if (rank == 0) {
        for (int b = b0; b < b1; ++b) {
            const int n = a.n_new[b];
            a.cu_new[b] = min(tok_pre[b], a.max_tokens);
            a.lens_out[b] = need_pre[b] >= 0 ? len[b] + n : (n < 0 && pool_ok && valid(len[b])) ? 0 : len[b];
        }
        if (threadIdx.x == 0) {
            a.cu_new[B] = min(tok_pre[B], a.max_tokens);
            *a.n_free_out = pool_ok ? (int)(have - total_taken) : n_free;
        }
    }
}

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs &a, cudaStream_t st) {
    const size_t smem = (4 * (size_t)a.B + 3) * sizeof(int);
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (4 * kPagedMaxBatch + 3) * (int)sizeof(int));
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    const int ranks = 1;
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
