// zha_paged_attn.cu -- zha_paged_decode: exact softmax attention of single
// query rows over a paged key/value cache, in one launch.
//
// For a row's query heads q_h over the tokens t it attends (base 2, with
// x = s log2(e) q.k):  m = max x_t,  l = sum 2^(x_t - m),
// o = sum 2^(x_t - m) v_t;  out = o / l,  lse = (m + log2 l) ln 2.
// (m, l, o) of disjoint token sets join by rescaling to the larger m, so any
// split of the tokens gives the same result.
//
// Bound: one read of the attended K and V rows from HBM (8 flops a byte at 8
// query heads per KV head, far below the tensor cores' rate).
//
// Work: the K/V rows of a (row, KV head) -- a group -- are cut into tiles of
// 16 KB of K and 16 KB of V; all groups' tiles form one list, and every CTA
// (two per SM) takes an equal contiguous part of it, whatever the rows'
// lengths are. A group that lies inside one CTA's part is written directly;
// of any other, each CTA that holds a piece leaves (m, l, o) in the workspace
// and the last one to arrive joins the pieces in their order.
//
// Inside a CTA the copies of the next two tiles (16-byte cp.async gathers by
// page, across group borders) are in flight while one is computed: S = Q K^T
// with each of the four warps on a quarter of the tile's tokens, the common
// row maximum and the weights through shared memory, then O += P V with each
// warp on a quarter of the head's coordinates. So O is spread over the CTA
// and a group's end needs no exchange, which keeps short rows cheap.
#include "zha_paged.cuh"

namespace zha {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kStages = 3;
constexpr int kRows = 16;                // query heads of a group, padded to the MMA's rows
constexpr int kTileBytes = 16384;        // of K, and of V
constexpr int kMaxWorkers = 148 * 2;
constexpr int kMinTiles = 4;             // tiles of a CTA's part at least
constexpr int kOffSlots = 4, kDescSlots = 8;
constexpr int kJoin = 64;                // pieces joined at a time

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

__device__ __forceinline__ uint32_t smem_at(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }
__device__ __forceinline__ void ldsm4(uint32_t at, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t at, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo, each with tf32's 11 significant bits (22 in all)
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo) {
    asm("cvt.rna.tf32.f32 %0, %1;\n" : "=r"(hi) : "f"(x));
    asm("cvt.rna.tf32.f32 %0, %1;\n" : "=r"(lo) : "f"(x - __uint_as_float(hi)));
}
// NaN if either is NaN
__device__ __forceinline__ float max_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
// main + corr, or main alone where the correction is not finite: the small
// parts of a split operand would turn an infinite factor into NaN.
__device__ __forceinline__ float with_correction(float main, float corr) {
    return fabsf(corr) <= 3.0e38f ? main + corr : main;
}

// A piece of a group in the workspace: (m, l) of its G heads, padded to whole
// float4s, then o as [G][D].
__host__ __device__ __forceinline__ int piece_ml(int G) { return (2 * G + 3) & ~3; }
__host__ __device__ __forceinline__ int piece_floats(int G, int d) { return piece_ml(G) + G * d; }

// One tile of a group.
struct Tile {
    int r, kvh;
    int len;          // tiles of the group
    int flags;
    int64_t g0;       // the group's first tile in the list of all tiles
};
enum { kFirst = 1, kLast = 2, kWhole = 4 };   // of this CTA's piece of the group; the piece is the group

template <typename T, int D>
struct Shared {
    static constexpr int TT = kTileBytes / (D * (int)sizeof(T));   // tokens of a tile
    // P as [16][TT] high parts, then low parts, rows padded against bank conflicts
    static constexpr int PS = sizeof(T) == 2 ? TT + 8 : TT + 4;
    uint8_t ring[kStages][2 * kTileBytes];
    union {
        alignas(16) T p[2][kRows][PS];
        float weight[kJoin][kRows];
    };
    int64_t off[kOffSlots][TT];          // byte offset of each token's row in its pool, -1: none
    Tile tile[kDescSlots];
    float mx[kWarps * 2][kRows], sum[kWarps * 2][kRows];
    int64_t scan[kWarps];
    int64_t start_before;
    int start_row, last;
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 2) paged_attn_kernel(PagedAttnArgs a, float *parts, int32_t *arrived) {
    using S = Shared<T, D>;
    constexpr bool kBf16 = sizeof(T) == 2;
    constexpr int TT = S::TT;
    constexpr int ROWB = D * (int)sizeof(T), CH = ROWB / 16;       // bytes and 16-byte chunks of a row
    constexpr int NT = TT / 32;                                     // 8-token columns of S per warp
    constexpr int NJ = D / 32;                                      // 8-wide columns of O per warp
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    S &sm = *reinterpret_cast<S *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gq = lane >> 2, t4 = lane & 3;
    pdl_wait();

    // ---- this CTA's part [w0, w1) of the list of all tiles, and the row it begins in
    const int per = (a.rows + kThreads - 1) / kThreads;
    const int ra = min(tid * per, a.rows), rb = min(ra + per, a.rows);
    auto tiles_of = [&](int r) {
        const RowSpan s = row_span(a, r);
        return (s.hi - s.lo + TT - 1) / TT;
    };
    int64_t mine = 0;
    for (int r = ra; r < rb; ++r) mine += tiles_of(r);
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sm.scan[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sm.scan[w];
        all += sm.scan[w];
    }
    const int64_t W = all * a.Hkv;
    const int64_t want = (W + kMinTiles - 1) / kMinTiles;
    const int P = want < gridDim.x ? (int)want : (int)gridDim.x;    // CTAs that get a part
    const int64_t w0 = (int)blockIdx.x < P ? W * blockIdx.x / P : 0;
    const int64_t w1 = (int)blockIdx.x < P ? W * (blockIdx.x + 1) / P : 0;
    const int n = (int)(w1 - w0);

    if (n > 0) {
        if (w0 >= before * a.Hkv && w0 < (before + mine) * a.Hkv) {
            int64_t at = before;
            for (int r = ra; r < rb; ++r) {
                const int t = tiles_of(r);
                if (w0 < (at + t) * a.Hkv) {
                    sm.start_row = r;
                    sm.start_before = at;
                    break;
                }
                at += t;
            }
        }
        __syncthreads();

        // ---- the reading end: which tile's pages are looked up next
        int c_r = sm.start_row, c_len = tiles_of(c_r);
        int64_t c_g0 = sm.start_before * a.Hkv;
        int c_kvh = (int)((w0 - c_g0) / c_len);
        c_g0 += (int64_t)c_kvh * c_len;
        int c_i = (int)(w0 - c_g0);
        RowSpan c_span = row_span(a, c_r);
        // looks up the page of this thread's token of tile k (of this CTA's part), leaves the tile's
        // description, and moves on; returns the page (-1: no token)
        int look_in = 0;                   // row inside the page, head included
        auto look = [&](int k) -> int {
            int page = -1;
            if (k < n) {
                const int pos = c_span.lo + c_i * TT + tid;
                if (tid < TT && pos < c_span.hi) {
                    page = __ldg(a.table + (int64_t)c_span.seq * a.max_pages + (pos >> a.lps));
                    look_in = (c_kvh << a.lps) + (pos & ((1 << a.lps) - 1));
                }
                if (tid == 0) {
                    Tile d;
                    d.r = c_r;
                    d.kvh = c_kvh;
                    d.len = c_len;
                    d.g0 = c_g0;
                    const bool first = k == 0 || c_i == 0, last = k == n - 1 || c_i == c_len - 1;
                    const bool whole = c_g0 >= w0 && c_g0 + c_len <= w1;
                    d.flags = (first ? kFirst : 0) | (last ? kLast : 0) | (whole ? kWhole : 0);
                    sm.tile[k % kDescSlots] = d;
                }
                if (++c_i == c_len && k + 1 < n) {
                    c_i = 0;
                    c_g0 += c_len;
                    if (++c_kvh == a.Hkv) {
                        c_kvh = 0;
                        do {
                            c_span = row_span(a, ++c_r);
                            c_len = (c_span.hi - c_span.lo + TT - 1) / TT;
                        } while (c_len == 0);
                    }
                }
            }
            return page;
        };
        const int64_t page_rows = (int64_t)a.Hkv << a.lps;
        auto put_off = [&](int k, int page, int in, bool asked) {
            if (tid < TT) {
                const bool ok = (unsigned)page < (unsigned)a.n_pages;
                if (asked && !ok) set_status(a.status, ZHA_ERR_INVALID_ARG);
                sm.off[k % kOffSlots][tid] = ok ? (page * page_rows + in) * ROWB : -1;
            }
        };
        const uint32_t ring = smem_at(sm.ring);
        const char *kpool = static_cast<const char *>(a.kpool), *vpool = static_cast<const char *>(a.vpool);
        auto issue = [&](int k) {
            if (k < n) {
                const uint32_t kb = ring + (k % kStages) * 2 * kTileBytes, vb = kb + kTileBytes;
#pragma unroll
                for (int j = 0; j < TT * CH / kThreads; ++j) {
                    const int c = tid + j * kThreads, row = c / CH, ch = c % CH;
                    const int64_t o = sm.off[k % kOffSlots][row];
                    const bool ok = o >= 0;
                    const int64_t at = (ok ? o : 0) + ch * 16;
                    // 16-byte chunks are permuted in a row so that the reads below meet no bank twice
                    const int ks = kBf16 ? (ch ^ (row & 7)) : (ch ^ ((row & 1) << 2));
                    const int vs = kBf16 ? (ch ^ (row & 7)) : (ch ^ ((row & 3) << 1));
                    cp16(kb + row * ROWB + ks * 16, kpool + at, ok);
                    cp16(vb + row * ROWB + vs * 16, vpool + at, ok);
                }
            }
            cp_commit();
        };

        // ---- before the first tile: pages of four tiles, copies of two
        int next_page, next_in;
        bool next_asked;
        {
            int pg[3], in[3];
            bool as[3];
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                as[k] = k < n && tid < TT && c_span.lo + c_i * TT + tid < c_span.hi;
                pg[k] = look(k);
                in[k] = look_in;
            }
            next_asked = 3 < n && tid < TT && c_span.lo + c_i * TT + tid < c_span.hi;
            next_page = look(3);
            next_in = look_in;
#pragma unroll
            for (int k = 0; k < 3; ++k) put_off(k, pg[k], in[k], as[k]);
        }
        __syncthreads();
        issue(0);
        issue(1);

        // Q fragments: bf16 as they are; fp32 split in two tf32 parts
        constexpr int KS = kBf16 ? D / 16 : D / 8;
        uint32_t qf[KS][4], ql[kBf16 ? 1 : KS][4];
        float o[NJ][4], m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NJ; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
        const float s2 = a.s * kLog2e;

        auto load_q = [&](int r, int kvh) {
            const T *q = static_cast<const T *>(a.q) + ((int64_t)r * a.Hq + kvh * a.G) * D;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int h = gq + 8 * half;
                const bool ok = h < a.G;
                if constexpr (kBf16) {
                    const uint32_t *row = reinterpret_cast<const uint32_t *>(q + (ok ? h : 0) * D);
#pragma unroll
                    for (int st = 0; st < KS; ++st) {
                        qf[st][half] = ok ? row[st * 8 + t4] : 0u;
                        qf[st][2 + half] = ok ? row[st * 8 + 4 + t4] : 0u;
                    }
                } else {
                    // coordinates of 16 are dealt to the k slots so that a lane's are 4 in a row
                    const float4 *row = reinterpret_cast<const float4 *>(q + (ok ? h : 0) * D);
#pragma unroll
                    for (int st = 0; st < KS; st += 2) {
                        const float4 x = ok ? row[st * 2 + t4] : make_float4(0.f, 0.f, 0.f, 0.f);
                        split_tf32(x.x, qf[st][half], ql[st][half]);
                        split_tf32(x.y, qf[st][2 + half], ql[st][2 + half]);
                        split_tf32(x.z, qf[st + 1][half], ql[st + 1][half]);
                        split_tf32(x.w, qf[st + 1][2 + half], ql[st + 1][2 + half]);
                    }
                }
            }
        };
        // this lane's coordinate of column c (0, 1) of O's column block j
        auto dim_of = [&](int j, int c) {
            return warp * (D / 4) + (kBf16 ? 8 * j + 2 * t4 + c : (2 * t4 + c) * NJ + j);
        };

        for (int it = 0; it < n; ++it) {
            cp_wait<1>();
            __syncthreads();               // tile `it` has landed; everyone is done with tile it - 1
            issue(it + 2);
            put_off(it + 3, next_page, next_in, next_asked);
            next_asked = it + 4 < n && tid < TT && c_span.lo + c_i * TT + tid < c_span.hi;
            next_page = look(it + 4);
            next_in = look_in;
            const Tile d = sm.tile[it % kDescSlots];
            if (d.flags & kFirst) load_q(d.r, d.kvh);
            const uint8_t *kt = sm.ring[it % kStages], *vt = kt + kTileBytes;
            const int64_t *off = sm.off[it % kOffSlots];
            const int tok0 = warp * (TT / 4);

            // ---- S = Q K^T of this warp's tokens
            float x[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if constexpr (kBf16) {
                    float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
                    const int row = tok0 + nt * 8 + (lane & 7);
#pragma unroll
                    for (int kp = 0; kp < D / 32; ++kp) {
                        uint32_t b[4];
                        ldsm4(smem_at(kt) + row * ROWB + (((4 * kp + (lane >> 3)) ^ (row & 7)) << 4), b);
                        mma_bf16(s0, qf[2 * kp], b[0], b[1]);
                        mma_bf16(s1, qf[2 * kp + 1], b[2], b[3]);
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u) x[nt][u] = s0[u] + s1[u];
                } else {
                    // three tf32 products (the low parts' product, 2^-22 of the whole, is left out)
                    float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f}, cr[4] = {0.f, 0.f, 0.f, 0.f};
                    const int row = tok0 + nt * 8 + gq;
#pragma unroll
                    for (int kp = 0; kp < D / 16; ++kp) {
                        const float4 kx = *reinterpret_cast<const float4 *>(
                            kt + row * ROWB + (((4 * kp + t4) ^ ((row & 1) << 2)) << 4));
                        uint32_t h[4], w[4];
                        split_tf32(kx.x, h[0], w[0]);
                        split_tf32(kx.y, h[1], w[1]);
                        split_tf32(kx.z, h[2], w[2]);
                        split_tf32(kx.w, h[3], w[3]);
                        mma_tf32(s0, qf[2 * kp], h[0], h[1]);
                        mma_tf32(s1, qf[2 * kp + 1], h[2], h[3]);
                        mma_tf32(cr, qf[2 * kp], w[0], w[1]);
                        mma_tf32(cr, ql[2 * kp], h[0], h[1]);
                        mma_tf32(cr, qf[2 * kp + 1], w[2], w[3]);
                        mma_tf32(cr, ql[2 * kp + 1], h[2], h[3]);
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u) x[nt][u] = with_correction(s0[u] + s1[u], cr[u]);
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const bool seen = off[tok0 + nt * 8 + 2 * t4 + (u & 1)] >= 0;
                    x[nt][u] = seen ? x[nt][u] * s2 : -INFINITY;
                }
            }
            // ---- row maxima over the tile
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float mx = -INFINITY;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mx = max_nan(mx, max_nan(x[nt][2 * r], x[nt][2 * r + 1]));
                mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                if (t4 == 0) sm.mx[warp][gq + 8 * r] = mx;
            }
            __syncthreads();
            float corr[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float mx = m_run[r];
#pragma unroll
                for (int w = 0; w < kWarps; ++w) mx = max_nan(mx, sm.mx[w][gq + 8 * r]);
                corr[r] = m_run[r] == mx ? 1.f : exp2f(m_run[r] - mx);
                m_run[r] = mx;
                float ls = 0.f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float p[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        p[u] = mx == -INFINITY ? 0.f : exp2f(x[nt][2 * r + u] - mx);
                        ls += p[u];
                    }
                    const int at = tok0 + nt * 8 + 2 * t4;
                    // weights keep 16 (bf16) or 22 (tf32) bits in two parts: one bf16 part alone would
                    // cost half an ulp of the output
                    if constexpr (kBf16) {
                        const __nv_bfloat162 hi = __floats2bfloat162_rn(p[0], p[1]);
                        const float2 hf = __bfloat1622float2(hi);
                        *reinterpret_cast<__nv_bfloat162 *>(&sm.p[0][gq + 8 * r][at]) = hi;
                        *reinterpret_cast<__nv_bfloat162 *>(&sm.p[1][gq + 8 * r][at]) =
                            __floats2bfloat162_rn(p[0] - hf.x, p[1] - hf.y);
                    } else {
                        uint32_t h[2], w[2];
                        split_tf32(p[0], h[0], w[0]);
                        split_tf32(p[1], h[1], w[1]);
                        *reinterpret_cast<uint2 *>(&sm.p[0][gq + 8 * r][at]) = make_uint2(h[0], h[1]);
                        *reinterpret_cast<uint2 *>(&sm.p[1][gq + 8 * r][at]) = make_uint2(w[0], w[1]);
                    }
                }
                l_run[r] = l_run[r] * corr[r] + ls;
            }
            __syncthreads();
            // ---- the tile's P V in accumulators of its own (the MMA truncates its sums: kept short), then into O
            float pv[NJ][4], pc[NJ][4];
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int u = 0; u < 4; ++u) pv[j][u] = pc[j][u] = 0.f;
            if constexpr (kBf16) {
#pragma unroll
                for (int kp = 0; kp < TT / 16; ++kp) {
                    uint32_t ph[4], pl[4];
                    const int prow = lane & 15, pcol = kp * 16 + (lane >> 4) * 8;
                    ldsm4(smem_at(&sm.p[0][prow][pcol]), ph);
                    ldsm4(smem_at(&sm.p[1][prow][pcol]), pl);
                    const int row = kp * 16 + (lane & 15);
#pragma unroll
                    for (int jp = 0; jp < NJ / 2; ++jp) {
                        uint32_t b[4];
                        const int ch = warp * (D / 32) + 2 * jp + (lane >> 4);
                        ldsm4t(smem_at(vt) + row * ROWB + ((ch ^ (row & 7)) << 4), b);
                        mma_bf16(pv[2 * jp], ph, b[0], b[1]);
                        mma_bf16(pv[2 * jp + 1], ph, b[2], b[3]);
                        mma_bf16(pc[2 * jp], pl, b[0], b[1]);
                        mma_bf16(pc[2 * jp + 1], pl, b[2], b[3]);
                    }
                }
            } else {
#pragma unroll
                for (int kp = 0; kp < TT / 8; ++kp) {
                    uint32_t ph[4], pl[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int prow = gq + 8 * (u & 1), pcol = kp * 8 + t4 + 4 * (u >> 1);
                        ph[u] = __float_as_uint(sm.p[0][prow][pcol]);
                        pl[u] = __float_as_uint(sm.p[1][prow][pcol]);
                    }
                    // NJ coordinates in a row per lane: column gq of each of the NJ column blocks
                    float v0[NJ], v1[NJ];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int row = kp * 8 + t4 + 4 * e;
                        const int byte = (warp * (D / 4) + gq * NJ) * 4;
                        const uint8_t *src = vt + row * ROWB + (((byte >> 4) ^ ((row & 3) << 1)) << 4) + (byte & 15);
                        float *dst = e ? v1 : v0;
                        if constexpr (NJ == 4) *reinterpret_cast<float4 *>(dst) = *reinterpret_cast<const float4 *>(src);
                        else *reinterpret_cast<float2 *>(dst) = *reinterpret_cast<const float2 *>(src);
                    }
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        uint32_t h0, h1, w0_, w1_;
                        split_tf32(v0[j], h0, w0_);
                        split_tf32(v1[j], h1, w1_);
                        mma_tf32(pv[j], ph, h0, h1);
                        mma_tf32(pc[j], ph, w0_, w1_);
                        mma_tf32(pc[j], pl, h0, h1);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int u = 0; u < 4; ++u) o[j][u] = fmaf(o[j][u], corr[u >> 1], with_correction(pv[j][u], pc[j][u]));

            if (!(d.flags & kLast)) continue;
            // ---- the end of this CTA's piece of the group: the sums of the warps
            float L[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float l = l_run[r];
                l += __shfl_xor_sync(0xffffffffu, l, 1);
                l += __shfl_xor_sync(0xffffffffu, l, 2);
                if (t4 == 0) sm.sum[warp][gq + 8 * r] = l;
            }
            __syncthreads();
            const int64_t head = (int64_t)d.r * a.Hq + d.kvh * a.G;
            float *part = nullptr;
            if (!(d.flags & kWhole)) {
                // slot 2c holds the piece that begins with CTA c's part, slot 2c + 1 the other
                const int64_t slot = 2 * (int64_t)blockIdx.x + (d.g0 > w0 ? 1 : 0);
                part = parts + slot * piece_floats(a.G, D);
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                L[r] = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) L[r] += sm.sum[w][gq + 8 * r];
                const int h = gq + 8 * r;
                if (h < a.G) {
                    if (part) {
                        if (warp == 0 && t4 == 0) {
                            part[2 * h] = m_run[r];
                            part[2 * h + 1] = L[r];
                        }
#pragma unroll
                        for (int j = 0; j < NJ; ++j)
#pragma unroll
                            for (int c = 0; c < 2; ++c) part[piece_ml(a.G) + h * D + dim_of(j, c)] = o[j][2 * r + c];
                    } else {
                        T *out = static_cast<T *>(a.out) + (head + h) * D;
#pragma unroll
                        for (int j = 0; j < NJ; ++j)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                out[dim_of(j, c)] = from_f32<T>(L[r] == 0.f ? 0.f : o[j][2 * r + c] / L[r]);
                        if (a.lse && warp == 0 && t4 == 0)
                            a.lse[head + h] = L[r] == 0.f ? -INFINITY : (m_run[r] + log2f(L[r])) * kLn2;
                    }
                }
                m_run[r] = -INFINITY;
                l_run[r] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < NJ; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
            if (!part) continue;

            // ---- the last piece to arrive joins them all
            const int c_first = (int)(((d.g0 + 1) * P - 1) / W), c_last = (int)(((d.g0 + d.len) * P - 1) / W);
            const int pieces = c_last - c_first + 1;
            __threadfence();
            __syncthreads();
            int32_t *counter = arrived + (int64_t)d.r * a.Hkv + d.kvh;
            if (tid == 0) sm.last = atomicAdd(counter, 1) == pieces - 1;
            __syncthreads();
            if (!sm.last) continue;
            __threadfence();
            if (tid == 0) *counter = 0;
            auto piece = [&](int i) {
                const int c = c_first + i;
                const bool second = i == 0 && W * c / P < d.g0;
                return parts + (2 * (int64_t)c + (second ? 1 : 0)) * piece_floats(a.G, D);
            };
            const int jh = tid & 15, ji = tid >> 4;        // this thread's head and first piece of the statistics
            float M = -INFINITY;
            if (jh < a.G)
                for (int i = ji; i < pieces; i += kThreads / 16) M = max_nan(M, __ldcg(piece(i) + 2 * jh));
            sm.mx[ji][jh] = M;
            __syncthreads();
            M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kThreads / 16; ++w) M = max_nan(M, sm.mx[w][jh]);
            constexpr int ITEMS = kRows * D / 4 / kThreads;
            float4 acc[ITEMS];
#pragma unroll
            for (int e = 0; e < ITEMS; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
            float Ls = 0.f;
            for (int base = 0; base < pieces; base += kJoin) {
                const int cnt = min(kJoin, pieces - base);
                __syncthreads();
                if (jh < a.G)
                    for (int i = ji; i < cnt; i += kThreads / 16) {
                        const float2 ml = __ldcg(reinterpret_cast<const float2 *>(piece(base + i)) + jh);
                        const float f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
                        sm.weight[i][jh] = f;
                        Ls += f == 0.f ? 0.f : ml.y * f;
                    }
                __syncthreads();
#pragma unroll
                for (int e = 0; e < ITEMS; ++e) {
                    const int at = tid + e * kThreads, h = at / (D / 4);
                    if (h < a.G) {
#pragma unroll 8
                        for (int i = 0; i < cnt; ++i) {
                            const float4 v = __ldcg(reinterpret_cast<const float4 *>(piece(base + i) + piece_ml(a.G)) + at);
                            const float f = sm.weight[i][h];
                            acc[e].x = fmaf(v.x, f, acc[e].x);
                            acc[e].y = fmaf(v.y, f, acc[e].y);
                            acc[e].z = fmaf(v.z, f, acc[e].z);
                            acc[e].w = fmaf(v.w, f, acc[e].w);
                        }
                    }
                }
            }
            sm.sum[ji][jh] = Ls;
            __syncthreads();
            auto total = [&](int h) {
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < kThreads / 16; ++w) s += sm.sum[w][h];
                return s;
            };
#pragma unroll
            for (int e = 0; e < ITEMS; ++e) {
                const int at = tid + e * kThreads, h = at / (D / 4);
                if (h < a.G) {
                    const float l = total(h), v[4] = {acc[e].x, acc[e].y, acc[e].z, acc[e].w};
                    float y[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) y[c] = l == 0.f ? 0.f : v[c] / l;
                    store_vec<4>(static_cast<T *>(a.out) + head * D + (int64_t)at * 4, y);
                }
            }
            if (a.lse && ji == 0 && jh < a.G) {
                const float l = total(jh);
                a.lse[head + jh] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
            }
        }
        cp_wait<0>();
    }
    // ---- rows that attend nothing
    for (int r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const RowSpan s = row_span(a, r);
        if (s.seq < 0 || s.hi > s.lo) continue;
        T *out = static_cast<T *>(a.out) + (int64_t)r * a.Hq * D;
        for (int i = tid; i < a.Hq * D; i += kThreads) out[i] = from_f32<T>(0.f);
        if (a.lse)
            for (int i = tid; i < a.Hq; i += kThreads) a.lse[(int64_t)r * a.Hq + i] = -INFINITY;
    }
    // no early trigger: a kernel behind this one may read `out` before its own wait
}

template <typename T, int D>
cudaError_t launch(const PagedAttnArgs &a, float *parts, int32_t *arrived, cudaStream_t st) {
    const size_t smem = sizeof(Shared<T, D>);
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    // no more CTAs than the longest possible rows would keep busy
    const int64_t longest = min64((int64_t)a.max_pages << a.lps, a.window > 0 ? a.window : INT64_MAX);
    const int64_t tiles = (longest + Shared<T, D>::TT - 1) / Shared<T, D>::TT * a.Hkv * a.rows;
    const int grid = (int)max64(1, min64(kMaxWorkers, (tiles + kMinTiles - 1) / kMinTiles));
    ProfScope ps("paged_decode", st);
    return launch_pdl(paged_attn_kernel<T, D>, dim3(grid), dim3(kThreads), smem, st, a, parts, arrived);
}

size_t pieces_bytes(const PagedAttnArgs &a) { return (size_t)kMaxWorkers * 2 * piece_floats(a.G, a.d) * sizeof(float); }

}  // namespace

// Two pieces per CTA, then the arrival counters of the groups (behind the
// part whose size is the configuration's alone: a call of fewer rows finds
// its counters where one of more rows does).
size_t paged_attn_workspace(const PagedAttnArgs &a) { return pieces_bytes(a) + (size_t)a.rows * a.Hkv * sizeof(int32_t); }

cudaError_t launch_paged_attention(const PagedAttnArgs &a, cudaStream_t st) {
    float *parts = static_cast<float *>(a.ws);
    int32_t *arrived = reinterpret_cast<int32_t *>(static_cast<char *>(a.ws) + pieces_bytes(a));
    if (a.dtype == ZHA_BF16)
        return a.d == 128 ? launch<__nv_bfloat16, 128>(a, parts, arrived, st)
                          : launch<__nv_bfloat16, 64>(a, parts, arrived, st);
    return a.d == 128 ? launch<float, 128>(a, parts, arrived, st) : launch<float, 64>(a, parts, arrived, st);
}

}  // namespace zha
