// zha_paged_attn.cu -- zha_paged_decode: exact softmax attention of single
// query rows over a paged key/value cache.
//
// Simplest form: one CTA per (row, KV head); each warp takes every 4th token
// with the head's coordinates spread over its lanes, keeps a running maximum
// and sum per query head, and the four warps' parts are joined at the end.
#include "zha_paged.cuh"

namespace zha {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWarps = 4;

// The tokens [lo, hi) that row r attends and the sequence they belong to
// (-1: the row is left as it is).
struct RowSpan {
    int seq, lo, hi;
};

__device__ __forceinline__ RowSpan row_span(const PagedAttnArgs &a, int r) {
    RowSpan s{r, 0, 0};
    if (a.seq_ids) {
        s.seq = a.seq_ids[r];
        if (s.seq >= a.batch) {
            set_status(a.status, ZHA_ERR_INVALID_ARG);
            s.seq = -1;
        }
        if (s.seq < 0) return RowSpan{-1, 0, 0};
    }
    int n = a.lens[s.seq];
    if (n < 0 || n > ((int64_t)a.max_pages << a.lps)) {
        set_status(a.status, ZHA_ERR_CAPACITY);
        n = 0;
    } else if (a.positions) {
        const int p = a.positions[r];
        if (p < 0 || p >= n) set_status(a.status, ZHA_ERR_INVALID_ARG);
        n = (p < 0 || p >= n) ? 0 : p + 1;
    }
    s.hi = n;
    s.lo = (a.window > 0 && n > a.window) ? n - a.window : 0;
    return s;
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) paged_simple_kernel(PagedAttnArgs a) {
    constexpr int E = D / 32;
    __shared__ float sm_m[kWarps][16], sm_l[kWarps][16], sm_o[kWarps][16][D];
    const int r = blockIdx.x, kvh = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    const RowSpan sp = row_span(a, r);
    if (sp.seq < 0) return;
    const int64_t head = (int64_t)r * a.Hq + kvh * a.G;
    float q[16][E], o[16][E], m[16], l[16];
#pragma unroll
    for (int h = 0; h < 16; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            q[h][e] = h < a.G ? to_f32(static_cast<const T *>(a.q)[(head + h) * D + lane + 32 * e]) : 0.f;
            o[h][e] = 0.f;
        }
    }
    const float s2 = a.s * kLog2e;
    for (int t = sp.lo + warp; t < sp.hi; t += kWarps) {
        const int page = a.table[(int64_t)sp.seq * a.max_pages + (t >> a.lps)];
        if ((unsigned)page >= (unsigned)a.n_pages) {
            set_status(a.status, ZHA_ERR_INVALID_ARG);
            continue;
        }
        const int64_t row = ((((int64_t)page * a.Hkv + kvh) << a.lps) + (t & ((1 << a.lps) - 1))) * D;
        float k[E], v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            k[e] = to_f32(static_cast<const T *>(a.kpool)[row + lane + 32 * e]);
            v[e] = to_f32(static_cast<const T *>(a.vpool)[row + lane + 32 * e]);
        }
#pragma unroll
        for (int h = 0; h < 16; ++h) {
            if (h >= a.G) break;
            float x = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) x = fmaf(q[h][e], k[e], x);
            x = warp_sum(x) * s2;
            const float mn = x > m[h] || x != x ? x : m[h];
            const float c = m[h] == mn ? 1.f : exp2f(m[h] - mn), p = mn == -INFINITY ? 0.f : exp2f(x - mn);
            m[h] = mn;
            l[h] = l[h] * c + p;
#pragma unroll
            for (int e = 0; e < E; ++e) o[h][e] = fmaf(p, v[e], o[h][e] * c);
        }
    }
#pragma unroll
    for (int h = 0; h < 16; ++h) {
        if (lane == 0) {
            sm_m[warp][h] = m[h];
            sm_l[warp][h] = l[h];
        }
#pragma unroll
        for (int e = 0; e < E; ++e) sm_o[warp][h][lane + 32 * e] = o[h][e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.G * D; i += blockDim.x) {
        const int h = i / D, e = i % D;
        float M = -INFINITY, L = 0.f, acc = 0.f;
        for (int w = 0; w < kWarps; ++w) M = (sm_m[w][h] > M || sm_m[w][h] != sm_m[w][h]) ? sm_m[w][h] : M;
        for (int w = 0; w < kWarps; ++w) {
            if (sm_m[w][h] == -INFINITY) continue;
            const float f = exp2f(sm_m[w][h] - M);
            L += sm_l[w][h] * f;
            acc += sm_o[w][h][e] * f;
        }
        static_cast<T *>(a.out)[(head + h) * D + e] = from_f32<T>(L == 0.f ? 0.f : acc / L);
        if (a.lse && e == 0) a.lse[head + h] = L == 0.f ? -INFINITY : M * kLn2 + logf(L);
    }
}

}  // namespace

size_t paged_attn_workspace(const PagedAttnArgs &) { return 256; }

cudaError_t launch_paged_attention(const PagedAttnArgs &a, cudaStream_t st) {
    ProfScope ps("paged_decode", st);
    const dim3 grid(a.rows, a.Hkv), blk(kWarps * 32);
    if (a.dtype == ZHA_BF16)
        return a.d == 128 ? launch_pdl(paged_simple_kernel<__nv_bfloat16, 128>, grid, blk, 0, st, a)
                          : launch_pdl(paged_simple_kernel<__nv_bfloat16, 64>, grid, blk, 0, st, a);
    return a.d == 128 ? launch_pdl(paged_simple_kernel<float, 128>, grid, blk, 0, st, a)
                      : launch_pdl(paged_simple_kernel<float, 64>, grid, blk, 0, st, a);
}

}  // namespace zha
