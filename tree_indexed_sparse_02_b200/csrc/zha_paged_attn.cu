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
// query heads per KV head, far below the tensor cores' rate). B200, launches in
// a graph: 4 rows of 262,144 tokens, 32/4 heads, d 128, bf16 334 us (2.15 GB:
// 6.43 TB/s, 98% of the measured copy; 315 to 343 us from card to card); 64 rows
// of 16 to 16,384 tokens 77 us (85%); one row of 200 tokens 8.2 us (latency: code
// and translations are cold in every launch); fp32, 6 rows of 60,001 tokens,
// 16/2 heads, d 64, 83 us (68%, bound by its instructions). Rows of one sequence
// share nothing: a prompt's rows each read their prefix (4,096 tokens 2.6 ms).
//
// Work: the K/V rows of a (row, KV head) -- a group -- are cut into tiles of
// 16 KB of K and 16 KB of V; all groups' tiles form one list, and every CTA
// (two or three per SM) takes an equal contiguous part of it, whatever the
// rows' lengths are: with a fixed number of CTAs per group the longest row of a
// ragged batch set the time. A part's ends move to a group's border where one
// is near. A group that lies inside one CTA's part is written directly; of any
// other, each CTA that holds a piece leaves (m, l, o) in the workspace, and the
// last to arrive joins the pieces in their order (in two levels where they are
// many). The counters end at zero.
//
// Inside a CTA a fifth warp walks the tiles ahead of the other four: it looks
// pages up (a batch of tiles ahead) and copies runs of up to 16 rows of a page
// by TMA into a ring of two or three tiles, across the groups' borders. (Tiles
// begin on any such box, so that little is copied that a window or a length
// leaves out; pages of 8 to 256 rows take the same time.) The
// four warps compute S = Q K^T, each on a quarter of the tile's tokens, share
// the row maxima and the weights through shared memory, and then O += P V, each
// on a quarter of the head's coordinates: O is spread over the CTA and a
// group's end needs no exchange, which keeps short rows cheap.
#include "zha_paged.h"
#include <type_traits>

#include "zha_tc.cuh"

namespace zha {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWarps = 4, kMath = kWarps * 32, kThreads = kMath + 32;
constexpr int kRows = 16;                // query heads of a group, padded to the MMA's rows
constexpr int kTileBytes = 16384;        // of K, and of V
constexpr int kSms = 148, kMaxWorkers = kSms * 3;
constexpr int kMinTiles = 3;             // tiles of a CTA's part at least (one row of 4,000 tokens: 13.7 us; 4: 15.3, 6: 17.5)
constexpr int kBox = 16;                 // rows of a page copied at a time, at most
constexpr int kDirect = 16;              // pieces of a group joined at once; more in two levels
constexpr int kSnap = 2;                 // a CTA's part begins at a group's border if one is this near (in tiles). 256 rows of 300 tokens:
                                         // 34.7 us, with 1 36.2; 16 rows of 2,000: 17.9 us, with 3 19.4
constexpr long long kWaitCycles = 4000000000ll;   // ~2 s: a wait that long is an error

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
// NaN if either is NaN
__device__ __forceinline__ float max_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
    return r;
}
// barriers of the four computing warps (the copying warp takes no part)
__device__ __forceinline__ void math_sync() { asm volatile("bar.sync 1, 128;\n" ::: "memory"); }
__device__ __forceinline__ bool math_any(bool x) {
    int r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.or.pred q, 1, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}\n"
                 : "=r"(r) : "r"((int)x) : "memory");
    return r != 0;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
// arrive on an mbarrier once this thread's cp.async copies so far have landed
__device__ __forceinline__ void cp_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %3, %3, %4}], [%2];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(w)
        : "memory");
}

// A piece of a group in the workspace: (m, l) of its G heads, padded to whole
// float4s, then o as [G][D].
__host__ __device__ __forceinline__ int piece_ml(int G) { return (2 * G + 3) & ~3; }
__host__ __device__ __forceinline__ int piece_floats(int G, int d) { return piece_ml(G) + G * d; }

// One tile of a group, as the copying warp describes it to the others.
struct alignas(16) Tile {
    int r, kvh;
    int flags;
    int base, lo, hi; // first token, and the tokens the row attends
    int c_first, pieces;      // a split group's last tile here: the first CTA that has a piece of it, and how many do
    uint32_t bad[4];  // tokens whose page number is no page
};
// first and last tile of this CTA's piece of the group; the piece begins and ends with the group; some token is
// not attended
enum { kFirst = 1, kLast = 2, kHead = 4, kTail = 8, kEdge = 16 };

// GP: query heads of a group, padded (fp32: 8 or 16; the bf16 MMA always has 16 rows).
template <typename T, int D, int GP>
struct Shared {
    static constexpr bool kBf16 = sizeof(T) == 2;
    // CTAs per SM and tiles in a CTA's ring. fp32 with few heads is bound by its instructions' latency: a third CTA
    // hides more of it than a third tile (16 heads do not fit its registers).
    static constexpr int kCtas = !kBf16 && GP == 8 ? 3 : 2, kStages = kCtas == 3 ? 2 : 3;
    static constexpr int TT = kTileBytes / (D * (int)sizeof(T));   // tokens of a tile
    static constexpr int ROWB = D * (int)sizeof(T), CH = ROWB / 16;       // bytes and 16-byte chunks of a row
    // K then V of a tile: blocks of 8 tokens, [ROWB / 128][8][128 bytes], 16-byte chunks XOR-swizzled by the row
    // (the 128-byte swizzle of a TMA copy)
    uint8_t ring[kStages][2 * kTileBytes];
    // The weights. bf16: as MMA operand rows [head][token], in two parts (16 bits, which moves about one output in a
    // thousand by a bf16 step; one bf16 part alone would cost half an ulp of the output), padded against bank conflicts; fp32: [token][head].
    typedef typename std::conditional<kBf16, __nv_bfloat16[2][kRows][TT + 8], float[TT][kRows]>::type Weights;
    alignas(16) Weights p;
    alignas(16) float score[!kBf16 && D == 128 && GP == 16 ? TT : 1][kRows];     // between a tile's scores and its weights
    // the queries of a piece, in one of QS places; bf16 rows are padded (read as fragments: no bank twice)
    static constexpr int QROW = ROWB + (kBf16 ? 16 : 0), QS = kBf16 || GP == 8 ? 2 : 1;
    alignas(16) uint8_t q[QS][kBf16 ? kRows : GP][QROW];
    Tile tile[kStages];
    alignas(16) float corr[kRows];
    float mx[kWarps][kRows], sum[kWarps][kRows];
    // of the rows that this part's two ends fall into: the row, tiles before it, its own tiles (of each head)
    int edge_row[2], edge_before[2], edge_tiles[2];
    int scan[kThreads / 32];
    uint64_t full[kStages], empty[kStages], q_empty[QS];
    int n, last, abort;

    // byte offset of a token's 16-byte chunk in K or V of a tile
    static __device__ __forceinline__ int at(int t, int ch) {
        return (t >> 3) * 8 * ROWB + (ch >> 3) * 1024 + (t & 7) * 128 + (((ch & 7) ^ (t & 7)) << 4);
    }
    // token t of the tile in stage st is outside the row's range or on no page
    __device__ __forceinline__ bool hidden(const Tile &d, int st, int t) const {
        const int pos = d.base + t;
        return pos < d.lo || pos >= d.hi || ((tile[st].bad[t >> 5] >> (t & 31)) & 1u);
    }
    // clears this warp's coordinates of the hidden tokens' value rows, which no other warp reads (their weights are
    // 0, but 0 times what the rows hold can be NaN)
    __device__ __forceinline__ void clear_hidden(const Tile &d, int st, int warp, int lane) {
        for (int i = lane; i < TT * CH / 4; i += 32) {
            const int t = i / (CH / 4), ch = warp * (CH / 4) + i % (CH / 4);
            if (hidden(d, st, t)) *reinterpret_cast<uint4 *>(ring[st] + kTileBytes + at(t, ch)) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();          // before a later copy lands there
        __syncwarp();
    }
};

// Joins cnt pieces in slots s0, s1, s1 + step, ... of the workspace, eight at a time; the result goes to the
// group's output, or back into slot s0. Each thread does its float4s of the heads' o with a running maximum of
// its own, so that nothing waits but for the loads. (Small code on purpose: it runs once or twice in a CTA's
// life, from a cold instruction cache.)
template <typename T, int D>
__device__ __forceinline__ void join(const PagedAttnArgs &a, float *parts, int cnt, int s0, int s1, int step, int64_t head,
                                     bool back) {
    constexpr int FLY = 8, Q = D / 4;          // float4s of a head
    const int items = a.G * Q, pf = piece_floats(a.G, D);
    float *first = parts + (int64_t)s0 * pf;
#pragma unroll 1
    for (int base = threadIdx.x & ~31; base < items; base += kMath) {
        // a head's float4s are lanes of one warp
        const bool mine = base + (threadIdx.x & 31) < items;
        const int at = mine ? base + (threadIdx.x & 31) : items - 1, h = at / Q;
        float M = -INFINITY, L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int i0 = 0; i0 < cnt; i0 += FLY) {
            float4 v[FLY];
            float2 ml[FLY];
#pragma unroll
            for (int u = 0; u < FLY; ++u) {
                const int i = i0 + u;
                const float *piece = i == 0 || i >= cnt ? first : parts + (int64_t)(s1 + (i - 1) * step) * pf;
                ml[u] = __ldcg(reinterpret_cast<const float2 *>(piece) + h);
                v[u] = __ldcg(reinterpret_cast<const float4 *>(piece + piece_ml(a.G)) + at);
                if (i >= cnt) ml[u] = make_float2(-INFINITY, 0.f);
            }
            float mx = M;
#pragma unroll
            for (int u = 0; u < FLY; ++u) mx = max_nan(mx, ml[u].x);
            const float ref = mx == -INFINITY ? 0.f : mx, c = ex2(M - ref);
            M = mx;
            L *= c;
            acc.x *= c;
            acc.y *= c;
            acc.z *= c;
            acc.w *= c;
#pragma unroll
            for (int u = 0; u < FLY; ++u) {
                if (ml[u].x == -INFINITY) continue;        // a piece without weight
                const float f = ex2(ml[u].x - ref);
                L = fmaf(ml[u].y, f, L);
                acc.x = fmaf(v[u].x, f, acc.x);
                acc.y = fmaf(v[u].y, f, acc.y);
                acc.z = fmaf(v[u].z, f, acc.z);
                acc.w = fmaf(v[u].w, f, acc.w);
            }
        }
        if (back) {
            __syncwarp();                          // piece s0 has been read
            if (mine) reinterpret_cast<float4 *>(first + piece_ml(a.G))[at] = acc;
            if (mine && at % Q == 0) reinterpret_cast<float2 *>(first)[h] = make_float2(M, L);
        } else if (mine) {
            const float inv = L == 0.f ? 0.f : 1.f / L, y[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
            store_vec<4>(static_cast<T *>(a.out) + head * D + (int64_t)at * 4, y);
            if (a.lse && at % Q == 0) a.lse[head + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
        }
    }
}

// Announces this CTA's piece (or set of pieces) at a counter; true in the CTA that is the last of `of`. (The
// barrier puts every thread's stores before thread 0's fence, which publishes them; the pieces are read past L1.)
__device__ __forceinline__ bool arrive(int32_t *counter, int of, int &sm_last) {
    math_sync();
    if (threadIdx.x == 0) {
        __threadfence();
        const bool last = atomicAdd(counter, 1) == of - 1;
        if (last) {
            __threadfence();
            *counter = 0;
        }
        sm_last = last;
    }
    math_sync();
    return sm_last != 0;
}

// The last piece of a group to arrive joins them all; with many pieces the last of a set of about sqrt(pieces)
// joins the set into its first piece's place, and the last set to arrive joins the sets.
template <typename T, int D>
__device__ __forceinline__ void join_group(const PagedAttnArgs &a, float *parts, int32_t *arrived, const Tile &d, int64_t head,
                                           int &sm_last) {
    const int pieces = d.pieces, slot0 = 2 * d.c_first + 1, mine = (int)blockIdx.x - d.c_first;
    int set = pieces;
    if (pieces > kDirect) {
        set = kDirect / 2;
        while (set * set < pieces) ++set;
    }
    const int i0 = mine / set * set, in_set = min(set, pieces - i0), sets = (pieces + set - 1) / set;
    const int set0 = i0 == 0 ? slot0 : 2 * (d.c_first + i0);
    int32_t *counter = arrived + set0;
    int cnt = in_set, s0 = set0, s1 = 2 * (d.c_first + i0 + 1), step = 2;
    bool back = sets > 1;
#pragma unroll 1
    while (arrive(counter, cnt, sm_last)) {
        join<T, D>(a, parts, cnt, s0, s1, step, head, back);
        if (!back) break;
        counter = arrived + 2 * kMaxWorkers + slot0;       // now the sets
        cnt = sets;
        s0 = slot0;
        s1 = 2 * (d.c_first + set);
        step = 2 * set;
        back = false;
    }
}

// This CTA's place for its piece of a split group (null: the piece is the group): slot 2c + 1 for a group's first
// piece, 2c for another.
__device__ __forceinline__ float *piece_place(const PagedAttnArgs &a, float *parts, int flags) {
    if ((flags & (kHead | kTail)) == (kHead | kTail)) return nullptr;
    return parts + (2 * (int64_t)blockIdx.x + (flags & kHead ? 1 : 0)) * piece_floats(a.G, a.d);
}

// bf16: S and O on tensor cores, m16n8k16 with the heads as rows.
template <int D>
__device__ __forceinline__ void math_bf16(const PagedAttnArgs &a, Shared<__nv_bfloat16, D, kRows> &sm, float *parts,
                                          int32_t *arrived, int n) {
    using T = __nv_bfloat16;
    using S = Shared<T, D, kRows>;
    constexpr int TT = S::TT, ROWB = S::ROWB;
    constexpr int NT = TT / 32;              // 8-token columns of S per warp
    constexpr int NJ = D / 32;               // 8-wide columns of O per warp
    constexpr int KS = D / 16;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gq = lane >> 2, t4 = lane & 3;
    volatile int *abort = &sm.abort;
    uint32_t qf[KS][4];                      // Q fragments
    float o[NJ][4], m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NJ; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    const float s2 = a.s * kLog2e;
    const int tok0 = warp * (TT / 4);
    // byte offsets of this lane's reads of K (two values of bit 2 of the chunk) and of V
    uint32_t ko[2], vo[NJ / 2];
#pragma unroll
    for (int b = 0; b < 2; ++b) ko[b] = S::at(tok0 + (lane & 7), 4 * b + (lane >> 3));
#pragma unroll
    for (int jp = 0; jp < NJ / 2; ++jp) vo[jp] = S::at(lane & 15, warp * (D / 32) + 2 * jp + (lane >> 4));

    int seg = -1;
    for (int it = 0; it < n; ++it) {
        const int st = it % S::kStages;
        const bool ok = mbar_wait_bounded(smem_u32(&sm.full[st]), (it / S::kStages) & 1, kWaitCycles, abort, a.status);
        const Tile d = sm.tile[st];
        if (d.flags & kFirst) {
            ++seg;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int h = gq + 8 * half;
                const uint32_t *row = reinterpret_cast<const uint32_t *>(sm.q[seg % S::QS][h]);
#pragma unroll
                for (int st = 0; st < KS; ++st) {
                    qf[st][half] = h < a.G ? row[st * 8 + t4] : 0u;
                    qf[st][2 + half] = h < a.G ? row[st * 8 + 4 + t4] : 0u;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.q_empty[seg % S::QS]));
        }
        const uint32_t kt = smem_u32(sm.ring[st]), vt = kt + kTileBytes;

        // ---- S = Q K^T of this warp's tokens
        float x[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kp = 0; kp < D / 32; ++kp) {
                uint32_t b[4];
                ldsm4(kt + ko[kp & 1] + nt * 8 * ROWB + (kp >> 1) * 1024, b);
                mma_bf16(s0, qf[2 * kp], b[0], b[1]);
                mma_bf16(s1, qf[2 * kp + 1], b[2], b[3]);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) x[nt][u] = (s0[u] + s1[u]) * s2;
        }
        if (d.flags & kEdge) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (sm.hidden(d, st, tok0 + nt * 8 + 2 * t4 + (u & 1))) x[nt][u] = -INFINITY;
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
        if (math_any(!ok)) break;          // a wait ran out: every warp leaves here
        float corr[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float mx = m_run[r];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mx = max_nan(mx, sm.mx[w][gq + 8 * r]);
            const float ref = mx == -INFINITY ? 0.f : mx;
            corr[r] = ex2(m_run[r] - ref);
            m_run[r] = mx;
            float ls = 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float p0 = ex2(x[nt][2 * r] - ref), p1 = ex2(x[nt][2 * r + 1] - ref);
                ls += p0 + p1;
                const int at = tok0 + nt * 8 + 2 * t4, h = gq + 8 * r;
                const __nv_bfloat162 hi = __floats2bfloat162_rn(p0, p1);
                const float2 hf = __bfloat1622float2(hi);
                *reinterpret_cast<__nv_bfloat162 *>(&sm.p[0][h][at]) = hi;
                *reinterpret_cast<__nv_bfloat162 *>(&sm.p[1][h][at]) = __floats2bfloat162_rn(p0 - hf.x, p1 - hf.y);
            }
            l_run[r] = l_run[r] * corr[r] + ls;
        }
        math_sync();
        // ---- the tile's P V in accumulators of its own (the MMA truncates its sums: kept short), then into O
        float pv[NJ][4];
        auto weigh = [&](bool low) {
#pragma unroll
            for (int j = 0; j < NJ; ++j) pv[j][0] = pv[j][1] = pv[j][2] = pv[j][3] = 0.f;
#pragma unroll
            for (int kp = 0; kp < TT / 16; ++kp) {
                uint32_t ph[4], pl[4];
                const int prow = lane & 15, pcol = kp * 16 + (lane >> 4) * 8;
                ldsm4(smem_u32(&sm.p[0][prow][pcol]), ph);
                if (low) ldsm4(smem_u32(&sm.p[1][prow][pcol]), pl);
#pragma unroll
                for (int jp = 0; jp < NJ / 2; ++jp) {
                    uint32_t b[4];
                    ldsm4t(vt + vo[jp] + kp * 16 * ROWB, b);
                    mma_bf16(pv[2 * jp], ph, b[0], b[1]);
                    mma_bf16(pv[2 * jp + 1], ph, b[2], b[3]);
                    if (low) {
                        mma_bf16(pv[2 * jp], pl, b[0], b[1]);
                        mma_bf16(pv[2 * jp + 1], pl, b[2], b[3]);
                    }
                }
            }
        };
        auto finite = [&]() {
            float odd = 0.f;               // stays 0 if everything is
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int u = 0; u < 4; ++u) odd = fmaf(pv[j][u], 0.f, odd);
            return !__any_sync(0xffffffffu, odd != 0.f);
        };
        weigh(true);
        if (!finite()) {
            // What hidden tokens' value rows hold came in: clear them and do the tile again. An attended infinite
            // value times a low part can be NaN where the product is infinite: what is not finite then is taken
            // from the high parts.
            if (d.flags & kEdge) sm.clear_hidden(d, st, warp, lane);
            weigh(true);
            if (!finite()) {
                float both[NJ][4];
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int u = 0; u < 4; ++u) both[j][u] = pv[j][u];
                weigh(false);
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int u = 0; u < 4; ++u) pv[j][u] = fabsf(both[j][u]) <= 3.0e38f ? both[j][u] : pv[j][u];
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.empty[st]));
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int u = 0; u < 4; ++u) o[j][u] = fmaf(o[j][u], corr[u >> 1], pv[j][u]);

        if (!(d.flags & kLast)) continue;
        // ---- the end of this CTA's piece of the group: the sums of the warps
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float l = l_run[r];
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            if (t4 == 0) sm.sum[warp][gq + 8 * r] = l;
        }
        math_sync();
        const int64_t head = (int64_t)d.r * a.Hq + d.kvh * a.G;
        float *part = piece_place(a, parts, d.flags);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float L = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) L += sm.sum[w][gq + 8 * r];
            const int h = gq + 8 * r;
            if (h < a.G) {
                if (part) {
                    if (warp == 0 && t4 == 0) reinterpret_cast<float2 *>(part)[h] = make_float2(m_run[r], L);
                } else if (a.lse && warp == 0 && t4 == 0) {
                    a.lse[head + h] = L == 0.f ? -INFINITY : (m_run[r] + log2f(L)) * kLn2;
                }
                const float inv = part ? 1.f : L == 0.f ? 0.f : 1.f / L;
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const float y[2] = {o[j][2 * r] * inv, o[j][2 * r + 1] * inv};
                    const int at = h * D + warp * (D / 4) + 8 * j + 2 * t4;
                    if (part) store_vec<2>(part + piece_ml(a.G) + at, y);
                    else store_vec<2>(static_cast<T *>(a.out) + head * D + at, y);
                }
            }
            m_run[r] = -INFINITY;
            l_run[r] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
        if (part) join_group<T, D>(a, parts, arrived, d, head, sm.last);
    }
}

// Two fp32 products and sums at once.
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;\n" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
struct Four {                                // 16 bytes: four floats as two pairs
    uint64_t a, b;
};
__device__ __forceinline__ Four load4(const void *p) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(p);
    return Four{v.x, v.y};
}

// fp32, on the CUDA cores two lanes wide (fma.rn.f32x2): products and sums keep fp32's precision, which tensor
// cores reach only with three or more passes over split operands.
//   S: 16 lanes share a token's coordinates (a chunk or two each) and take TC tokens and 8 heads at a time; the 16
//      partial sums are exchanged so that a lane ends with one head's scores of TC / 2 tokens.
//   O: a lane has 4 coordinates of all heads for every NG-th token; the NG parts meet at the end of the piece.
template <int D, int GP>
__device__ __forceinline__ void math_f32(const PagedAttnArgs &a, Shared<float, D, GP> &sm, float *parts, int32_t *arrived,
                                         int n) {
    using S = Shared<float, D, GP>;
    constexpr int TT = S::TT;
    constexpr int WT = TT / 4;               // tokens of a warp
    constexpr int CL = D / 64;               // chunks of a lane in S
    constexpr int TC = GP == 8 ? 4 : 2;      // tokens of a lane at a time (registers)
    constexpr int NC = WT / (2 * TC);        // times
    constexpr int NO = GP / 8;               // octets of heads
    constexpr int NX = NC * TC / 2;          // scores a lane ends with, for each octet
    constexpr int CW = D / 16;               // chunks of a warp in O: lanes side by side
    constexpr int NG = 32 / CW;              // groups of lanes, by token
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int dq = lane & 15, ts = lane >> 4, hd = lane & 7, th = (lane >> 3) & 1;
    const int oc = lane % CW, og = lane / CW;
    const int tok0 = warp * WT;
    volatile int *abort = &sm.abort;
    uint64_t o[GP][2];
    float m_run[NO], l_run[NO];
#pragma unroll
    for (int h = 0; h < GP; ++h) o[h][0] = o[h][1] = 0ull;
#pragma unroll
    for (int e = 0; e < NO; ++e) {
        m_run[e] = -INFINITY;
        l_run[e] = 0.f;
    }
    const float s2 = a.s * kLog2e;
    // token of score e of a lane
    auto tok_of = [&](int e) { return tok0 + ts + 2 * ((e / (TC / 2)) * TC + th * (TC / 2) + e % (TC / 2)); };

    int seg = -1;
    for (int it = 0; it < n; ++it) {
        const int st = it % S::kStages;
        const bool ok = mbar_wait_bounded(smem_u32(&sm.full[st]), (it / S::kStages) & 1, kWaitCycles, abort, a.status);
        const Tile d = sm.tile[st];
        if (d.flags & kFirst) ++seg;
        const uint8_t *kt = sm.ring[st], *vt = kt + kTileBytes, *qp = sm.q[seg % S::QS][0];

        // ---- S, an octet of heads at a time. 16 heads of 128 coordinates: loops stay rolled and the scores go to
        // shared memory (unrolled, with the scores in registers, they spill: 160 instead of 116 us at 6 x 20,001
        // tokens); otherwise unrolling is faster by a tenth.
        constexpr bool kRoll = D == 128 && GP == 16;
        float kept[kRoll ? 1 : NO][kRoll ? 1 : NX];
        const bool edge = d.flags & kEdge;
#pragma unroll(kRoll ? 1 : NO)
        for (int e = 0; e < NO; ++e) {
            float mx = -INFINITY;
#pragma unroll(kRoll ? 1 : NC)
            for (int c = 0; c < NC; ++c) {
                Four k[TC][CL];
#pragma unroll
                for (int i = 0; i < TC; ++i)
#pragma unroll
                    for (int j = 0; j < CL; ++j) k[i][j] = load4(kt + S::at(tok0 + ts + 2 * (c * TC + i), dq + 16 * j));
                float v[TC][8];
#pragma unroll
                for (int h = 0; h < 8; ++h) {
                    // (heads beyond the group repeat its last one; their results are dropped)
                    const uint8_t *row = qp + min(8 * e + h, a.G - 1) * S::QROW;
                    Four q[CL];
#pragma unroll
                    for (int j = 0; j < CL; ++j) q[j] = load4(row + (dq + 16 * j) * 16);
#pragma unroll
                    for (int i = 0; i < TC; ++i) {
                        uint64_t acc = 0ull;
#pragma unroll
                        for (int j = 0; j < CL; ++j) {
                            acc = fma2(k[i][j].a, q[j].a, acc);
                            acc = fma2(k[i][j].b, q[j].b, acc);
                        }
                        const float2 f = unpack2(acc);
                        v[i][h] = f.x + f.y;
                    }
                }
                // sums over the 16 lanes: by halves of the tokens, then of the heads
#pragma unroll
                for (int i = 0; i < TC / 2; ++i) {
                    float w[8], u[4], y[2];
#pragma unroll
                    for (int h = 0; h < 8; ++h) {
                        const float keep = th ? v[i + TC / 2][h] : v[i][h], give = th ? v[i][h] : v[i + TC / 2][h];
                        w[h] = keep + __shfl_xor_sync(0xffffffffu, give, 8);
                    }
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const bool up = lane & 4;
                        const float keep = up ? w[h + 4] : w[h], give = up ? w[h] : w[h + 4];
                        u[h] = keep + __shfl_xor_sync(0xffffffffu, give, 4);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const bool up = lane & 2;
                        const float keep = up ? u[h + 2] : u[h], give = up ? u[h] : u[h + 2];
                        y[h] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
                    }
                    const bool up = lane & 1;
                    const float keep = up ? y[1] : y[0], give = up ? y[0] : y[1];
                    float x = (keep + __shfl_xor_sync(0xffffffffu, give, 1)) * s2;
                    const int t = tok_of(c * (TC / 2) + i);
                    if (edge && sm.hidden(d, st, t)) x = -INFINITY;
                    if constexpr (kRoll) sm.score[t][8 * e + hd] = x;
                    else kept[e][c * (TC / 2) + i] = x;
                    mx = max_nan(mx, x);
                }
            }
            mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            if (lane < 8) sm.mx[warp][8 * e + lane] = mx;
        }
        if (edge) sm.clear_hidden(d, st, warp, lane);
        if (math_any(!ok)) break;          // a wait ran out: every warp leaves here
#pragma unroll
        for (int e = 0; e < NO; ++e) {
            const int h = 8 * e + hd;
            float mx = m_run[e];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mx = max_nan(mx, sm.mx[w][h]);
            const float ref = mx == -INFINITY ? 0.f : mx, corr = ex2(m_run[e] - ref);
            m_run[e] = mx;
            float ls = 0.f;
#pragma unroll
            for (int i = 0; i < NX; ++i) {
                const int t = tok_of(i);
                float x;
                if constexpr (kRoll) x = sm.score[t][h];
                else x = kept[e][i];
                const float p = ex2(x - ref);
                ls += p;
                sm.p[t][h] = p;
            }
            l_run[e] = l_run[e] * corr + ls;
            if (tid < 8) sm.corr[h] = corr;
        }
        math_sync();
        // ---- O
#pragma unroll
        for (int h = 0; h < GP; h += 4) {
            const float4 c = *reinterpret_cast<const float4 *>(&sm.corr[h]);
            const float cc[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint64_t c2 = pack2(cc[u], cc[u]);
                o[h + u][0] = fma2(o[h + u][0], c2, 0ull);
                o[h + u][1] = fma2(o[h + u][1], c2, 0ull);
            }
        }
#pragma unroll(GP == 8 ? 4 : 1)
        for (int i = 0; i < TT / NG; ++i) {
            // (neighbouring groups four rows apart: 8 lanes' 16-byte reads meet no bank twice)
            const int t = NG == 4 ? og + 4 * i : (og >> 1) + 4 * (og & 1) + 8 * i;
            const Four v = load4(vt + S::at(t, warp * CW + oc));
#pragma unroll
            for (int h = 0; h < GP; h += 4) {
                const float4 p = *reinterpret_cast<const float4 *>(&sm.p[t][h]);
                const float pp[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint64_t p2 = pack2(pp[u], pp[u]);
                    o[h + u][0] = fma2(v.a, p2, o[h + u][0]);
                    o[h + u][1] = fma2(v.b, p2, o[h + u][1]);
                }
            }
        }
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(smem_u32(&sm.empty[st]));
            if (d.flags & kLast) mbar_arrive(smem_u32(&sm.q_empty[seg % S::QS]));
        }
        if (!(d.flags & kLast)) continue;
        // ---- the end of this CTA's piece of the group: the sums of the warps, and O's parts of the NG groups of
        // lanes, by halves of the heads
#pragma unroll
        for (int e = 0; e < NO; ++e) {
            float l = l_run[e];
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            if (lane < 8) sm.sum[warp][8 * e + lane] = l;
        }
        int h0 = 0;                        // first head of what this lane keeps
        auto halve = [&]<int BIT, int KEEP>() {
            const bool up = lane & BIT;
#pragma unroll
            for (int h = 0; h < KEEP; ++h)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint64_t mine = up ? o[h + KEEP][c] : o[h][c], give = up ? o[h][c] : o[h + KEEP][c];
                    const float2 f = unpack2(mine), g = unpack2(give);
                    o[h][c] = pack2(f.x + __shfl_xor_sync(0xffffffffu, g.x, BIT), f.y + __shfl_xor_sync(0xffffffffu, g.y, BIT));
                }
            h0 += up ? KEEP : 0;
        };
        halve.template operator()<16, GP / 2>();
        halve.template operator()<8, GP / 4>();
        if constexpr (NG == 8) halve.template operator()<4, GP / 8>();
        math_sync();
        const int64_t head = (int64_t)d.r * a.Hq + d.kvh * a.G;
        float *part = piece_place(a, parts, d.flags);
        auto total = [&](int h) {
            float L = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) L += sm.sum[w][h];
            return L;
        };
#pragma unroll
        for (int u = 0; u < GP / NG; ++u) {
            const int h = h0 + u;
            if (h >= a.G) continue;
            const float L = part ? 1.f : total(h), inv = L == 0.f ? 0.f : 1.f / L;
            const float2 f = unpack2(o[u][0]), g = unpack2(o[u][1]);
            const float y[4] = {f.x * inv, f.y * inv, g.x * inv, g.y * inv};
            store_vec<4>((part ? part + piece_ml(a.G) : static_cast<float *>(a.out) + head * D) + h * D + (warp * CW + oc) * 4, y);
        }
        if (warp == 0 && lane < 8) {
#pragma unroll
            for (int e = 0; e < NO; ++e) {
                const int h = 8 * e + lane;
                if (h >= a.G) continue;
                const float L = total(h);
                if (part) reinterpret_cast<float2 *>(part)[h] = make_float2(m_run[e], L);
                else if (a.lse) a.lse[head + h] = L == 0.f ? -INFINITY : (m_run[e] + log2f(L)) * kLn2;
            }
        }
#pragma unroll
        for (int h = 0; h < GP; ++h) o[h][0] = o[h][1] = 0ull;
#pragma unroll
        for (int e = 0; e < NO; ++e) {
            m_run[e] = -INFINITY;
            l_run[e] = 0.f;
        }
        if (part) join_group<float, D>(a, parts, arrived, d, head, sm.last);
    }
}

template <typename T, int D, int GP, bool kTma>
__global__ void __launch_bounds__(kThreads, Shared<T, D, GP>::kCtas)
paged_attn_kernel(const __grid_constant__ PagedAttnArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  float *parts, int32_t *arrived) {
    using S = Shared<T, D, GP>;
    constexpr bool kBf16 = S::kBf16;
    constexpr int TT = S::TT, ROWB = S::ROWB, CH = S::CH;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    S &sm = *reinterpret_cast<S *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int box = min(1 << a.lps, kBox);      // rows of a page copied at a time; tiles begin on a box
    volatile int *abort = &sm.abort;
    if (tid == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(smem_u32(&sm.full[i]), kTma ? 1 : 33);
            mbar_init(smem_u32(&sm.empty[i]), kWarps);
        }
        for (int i = 0; i < S::QS; ++i) mbar_init(smem_u32(&sm.q_empty[i]), kWarps);
        sm.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        fence_proxy_async_smem();
        if (kTma) {
            asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
            asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&vmap)) : "memory");
        }
    }
    __syncthreads();
    pdl_wait();

    // ---- this CTA's part [w0, w1) of the list of all tiles, and the row it begins in: prefix sums over the
    // rows, by the copying warp alone where it holds them all. (The others get its count, so that they cannot
    // disagree on it.)
    auto tiles_of = [&](const RowSpan &s) { return s.hi > s.lo ? (s.hi - (s.lo & -box) + TT - 1) / TT : 0; };
    const bool few = a.rows <= 32;
    int w0 = 0, w1 = 0, share = 1, start_row = 0, start_before = 0;
    if (!few || warp == kWarps) {
        const int per = few ? 1 : (a.rows + kThreads - 1) / kThreads;
        const int ra = min((few ? lane : tid) * per, a.rows), rb = min(ra + per, a.rows);
        int mine = 0;
        for (int r = ra; r < rb; ++r) mine += tiles_of(row_span(a, r));
        int before = mine;               // first inclusive, of this warp's lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += y;
        }
        int W = __shfl_sync(0xffffffffu, before, 31);
        before -= mine;
        if (!few) {
            if (lane == 0) sm.scan[warp] = W;
            __syncthreads();
            W = 0;
#pragma unroll 1
            for (int w = 0; w < kThreads / 32; ++w) {
                if (w < warp) before += sm.scan[w];
                W += sm.scan[w];
            }
        }
        W *= a.Hkv;
        // Parts of `share` tiles, their ends moved to a group's border where one is within kSnap tiles: a piece of
        // a few tiles costs more to join than to compute.
        share = max(kMinTiles, (W + (int)gridDim.x - 1) / (int)gridDim.x);
        const int first_tile = min((int64_t)blockIdx.x * share, (int64_t)W);
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {    // (a loop, not two copies: the code is cold)
            int edge = e ? min(first_tile + share, W) : first_tile;
            const bool own = edge >= before * a.Hkv && edge < (before + mine) * a.Hkv;
            int row = ra, t = mine, at = before;
            if (few) {
                const int src = (__ffs(__ballot_sync(0xffffffffu, own)) - 1) & 31;
                row = __shfl_sync(0xffffffffu, ra, src);
                t = __shfl_sync(0xffffffffu, mine, src);
                at = __shfl_sync(0xffffffffu, before, src);
            } else {
                if (own) {
                    for (row = ra; row < rb; ++row) {
                        t = tiles_of(row_span(a, row));
                        if (edge < (at + t) * a.Hkv) break;
                        at += t;
                    }
                    sm.edge_row[e] = min(row, a.rows - 1);
                    sm.edge_tiles[e] = t;
                    sm.edge_before[e] = at;
                }
                __syncthreads();
                row = sm.edge_row[e];
                t = sm.edge_tiles[e];
                at = sm.edge_before[e];
            }
            if (e == 0) {
                start_row = row;
                start_before = at;
            }
            if (edge > 0 && edge < W) {
                const int i = (edge - at * a.Hkv) % t;
                if (t - i <= kSnap) edge += t - i;
                else if (i <= kSnap) edge -= i;
            }
            if (e == 0) w0 = edge;
            else w1 = edge;
        }
    }
    if (tid == kMath) sm.n = w1 - w0;
    __syncthreads();
    const int n = sm.n;

    if (warp == kWarps) {
        // ================= the copying warp
        if (n == 0) return;
        // where a walk over the list stands: tile i of the group (r, kvh), whose len tiles begin at g0
        struct Walk {
            int r, kvh, i, len, g0;
            RowSpan span;
        };
        Walk next;
        next.r = start_row;
        next.span = row_span(a, next.r);
        next.len = tiles_of(next.span);
        next.g0 = start_before * a.Hkv;
        next.kvh = (w0 - next.g0) / next.len;
        next.g0 += next.kvh * next.len;
        next.i = w0 - next.g0;
        auto next_row = [&]() {
            next.kvh = 0;
            do {
                next.span = row_span(a, ++next.r);
                next.len = tiles_of(next.span);
            } while (next.len == 0 && next.r + 1 < a.rows);
        };
        if (next.kvh == a.Hkv) next_row();         // the start moved up to the end of its row
        // A lane looks up one box's page of one of the next `batch` tiles of a group (TMA), or the pages of
        // the tokens lane, lane + 32, ... of the next tile (small pages), a batch ahead of the copies.
        constexpr int NP = kTma ? 1 : TT / 32;
        const int lbox = 31 - __clz(box), boxes = kTma ? TT >> lbox : 1, lboxes = 31 - __clz(boxes);
        const int batch = kTma ? 32 >> lboxes : 1;
        const int lt = kTma ? lane >> lboxes : 0, lb = kTma ? lane & (boxes - 1) : 0;
        int page_next[NP];
        auto token = [&](const Walk &c, int i) {
            return (c.span.lo & -box) + (c.i + lt) * TT + (kTma ? lb * box : lane + 32 * i);
        };
        auto look = [&]() {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int pos = token(next, i);
                page_next[i] = next.i + lt < next.len && pos < next.span.hi
                                   ? __ldg(a.table + (int64_t)next.span.seq * a.max_pages + (pos >> a.lps)) : -1;
            }
        };
        look();
        int k = 0, seg = -1;               // tiles issued, pieces begun
        int st = 0, round = 0;             // place in the ring, times round it
        int left = 0, off = 0;             // tiles left of the batch, and the next one's place in it
        int64_t row[NP];                   // first row of this lane's copy in its pool, -1: none
        uint32_t good[NP], bad[NP];        // lanes whose copy is one; whose page number is no page
        Tile d;
        int ci = 0, last_ci = 0;           // the next tile's place in its group, and the piece's last one
        for (; k < n; ++k, --left, ++off, ++ci) {
            if (left == 0) {
                // what the tiles of a batch have in common
                const Walk c = next;
                off = 0;
                ci = c.i;
                last_ci = c.len - 1;
                left = min(batch, c.len - c.i);
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    const int pos = token(c, i);
                    const bool in = lt < left && pos < c.span.hi, ok = in && (unsigned)page_next[i] < (unsigned)a.n_pages;
                    row[i] = ok ? (((int64_t)page_next[i] * a.Hkv + c.kvh) << a.lps) + (pos & ((1 << a.lps) - 1)) : -1;
                    good[i] = __ballot_sync(0xffffffffu, ok);
                    bad[i] = __ballot_sync(0xffffffffu, in && !ok);
                    if (in && !ok) set_status(a.status, ZHA_ERR_INVALID_ARG);
                }
                d.r = c.r;
                d.kvh = c.kvh;
                d.lo = c.span.lo;
                d.hi = c.span.hi;
                d.base = (c.span.lo & -box) + ci * TT;
                d.flags = (c.g0 >= w0 ? kHead : 0) | (c.g0 + c.len <= w1 ? kTail : 0);
                // of a split group: the parts that begin inside it, not near its borders
                const int lo = (c.g0 + kSnap) / share + 1, hi = (c.g0 + c.len - kSnap - 1) / share;
                d.c_first = lo - 1;
                d.pieces = hi - lo + 2;
                if (k + left < n) {
                    next.i += left;
                    if (next.i == next.len) {
                        next.i = 0;
                        next.g0 += next.len;
                        if (++next.kvh == a.Hkv) next_row();
                    }
                    look();
                }
            }
            const bool first = k == 0 || ci == 0;
            Tile t = d;
            t.flags |= (first ? kFirst : 0) | (k == n - 1 || ci == last_ci ? kLast : 0) |
                       (d.base < d.lo || d.base + TT > d.hi ? kEdge : 0);
            d.base += TT;
            t.bad[0] = t.bad[1] = t.bad[2] = t.bad[3] = 0;
            const uint32_t mine = kTma ? ((1u << boxes) - 1u) << (off << lboxes) : 0xffffffffu;   // the tile's lanes
#pragma unroll
            for (int i = 0; i < NP; ++i)
                if (bad[i] & mine) {
                    t.flags |= kEdge;
                    if constexpr (kTma) {
                        const uint32_t b = (bad[0] & mine) >> (off << lboxes);     // one bit a box
#pragma unroll
                        for (int w = 0; w < (TT + 31) / 32; ++w)
                            for (int e = 0; e < 32; ++e)
                                if ((b >> ((32 * w + e) >> lbox)) & 1u) t.bad[w] |= 1u << e;
                    } else {
                        t.bad[i] = bad[i];
                    }
                }
            if (round > 0 && !__all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&sm.empty[st]), (round - 1) & 1, kWaitCycles,
                                                                        abort, a.status)))
                break;
            seg += first;
            // a piece's queries come with its first tile, once the warps hold those that were in their place
            if (first && seg >= S::QS && !__all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&sm.q_empty[seg % S::QS]),
                                                                                    (seg / S::QS - 1) & 1, kWaitCycles, abort, a.status)))
                break;
            const uint32_t kb = smem_u32(sm.ring[st]), vb = kb + kTileBytes, full = smem_u32(&sm.full[st]);
            if (lane == 0) sm.tile[st] = t;
            if constexpr (kTma) {
                const bool ok = row[0] >= 0 && lt == off;
                const uint32_t cnt = __popc(good[0] & mine);
                if (lane == 0) mbar_expect_tx(full, cnt * 2u * (uint32_t)box * ROWB + (first ? a.G * ROWB : 0));
                __syncwarp();
                if (ok) {
                    const uint32_t at = (uint32_t)lb * box * ROWB;
                    tma_load_4d(kb + at, &kmap, (int)(row[0] >> 3), full);
                    tma_load_4d(vb + at, &vmap, (int)(row[0] >> 3), full);
                }
            } else {
#pragma unroll 4
                for (int j = 0; j < TT * CH / 32; ++j) {
                    const int tok = (j * 32) / CH + lane / CH, ch = (j * 32) % CH + lane % CH;
                    const int64_t rw = __shfl_sync(0xffffffffu, row[0], tok & 31);
                    int64_t r2 = rw;
#pragma unroll
                    for (int i = 1; i < NP; ++i) {
                        const int64_t x = __shfl_sync(0xffffffffu, row[i], tok & 31);
                        if ((tok >> 5) == i) r2 = x;
                    }
                    const bool ok = r2 >= 0;
                    const int64_t at = (ok ? r2 : 0) * ROWB + ch * 16;
                    const uint32_t to = S::at(tok, ch);
                    cp16(kb + to, static_cast<const char *>(a.kpool) + at, ok);
                    cp16(vb + to, static_cast<const char *>(a.vpool) + at, ok);
                }
                cp_arrive(full);
                __syncwarp();
                if (lane == 0) mbar_expect_tx(full, first ? a.G * ROWB : 0);
                __syncwarp();
            }
            if (first && lane < a.G)
                bulk_load(smem_u32(sm.q[seg % S::QS][lane]), static_cast<const T *>(a.q) + ((int64_t)t.r * a.Hq + t.kvh * a.G + lane) * D,
                          ROWB, full);
            if (++st == S::kStages) {
                st = 0;
                ++round;
            }
        }
        // The copies in flight land before the CTA may end, also where another warp has given up on one (it does not
        // wait for those behind it).
        for (int j = k < S::kStages ? 0 : k - S::kStages; j < k; ++j)
            mbar_wait_bounded(smem_u32(&sm.full[j % S::kStages]), (j / S::kStages) & 1, kWaitCycles, nullptr, a.status);
        return;
    }

    // ================= the computing warps
    if constexpr (kBf16) math_bf16<D>(a, sm, parts, arrived, n);
    else math_f32<D, GP>(a, sm, parts, arrived, n);
    // ---- rows that attend nothing
    for (int r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const RowSpan s = row_span(a, r);
        if (s.seq < 0 || s.hi > s.lo) continue;
        T *out = static_cast<T *>(a.out) + (int64_t)r * a.Hq * D;
        for (int i = tid; i < a.Hq * D; i += kMath) out[i] = from_f32<T>(0.f);
        if (a.lse)
            for (int i = tid; i < a.Hq; i += kMath) a.lse[(int64_t)r * a.Hq + i] = -INFINITY;
    }
    // no early trigger: a kernel behind this one may read `out` before its own wait
}

// The pool as [rows / 8][D * sizeof(T) / 128][8][128 bytes]: a box is `box` rows in the ring's layout.
template <typename T, int D>
bool pool_map(CUtensorMap *map, const void *pool, const PagedAttnArgs &a, int box) {
    constexpr int ROWB = D * (int)sizeof(T), E = 128 / (int)sizeof(T);
    const uint64_t rows = ((uint64_t)a.n_pages << a.lps) * a.Hkv;
    const cuuint64_t dims[4] = {(cuuint64_t)E, 8, ROWB / 128, rows / 8};
    const cuuint64_t strides[3] = {ROWB, 128, 8 * ROWB};
    const cuuint32_t boxd[4] = {(cuuint32_t)E, 8, ROWB / 128, (cuuint32_t)(box / 8)};
    const cuuint32_t step[4] = {1, 1, 1, 1};
    return tensor_map_encoder()(map, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4,
                                const_cast<void *>(pool), dims, strides, boxd, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, int GP, bool kTma>
cudaError_t launch(const PagedAttnArgs &a, float *parts, int32_t *arrived, cudaStream_t st) {
    const size_t smem = sizeof(Shared<T, D, GP>);
    using S = Shared<T, D, GP>;
    static_assert(S::kCtas * (sizeof(S) + 1024) <= 228 * 1024, "the CTAs fit an SM's shared memory");
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel<T, D, GP, kTma>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    CUtensorMap kmap{}, vmap{};
    if (kTma) {
        const int box = (1 << a.lps) < kBox ? 1 << a.lps : kBox;
        if (!tensor_map_encoder() || !pool_map<T, D>(&kmap, a.kpool, a, box) || !pool_map<T, D>(&vmap, a.vpool, a, box))
            return cudaErrorNotSupported;
    }
    // no more CTAs than the longest possible rows would keep busy
    const int64_t longest = min64((int64_t)a.max_pages << a.lps, a.window > 0 ? (int64_t)a.window + kBox : INT64_MAX);
    const int64_t tiles = (longest + Shared<T, D, GP>::TT - 1) / Shared<T, D, GP>::TT * a.Hkv * a.rows;
    const int grid = (int)max64(1, min64(kSms * S::kCtas, (tiles + kMinTiles - 1) / kMinTiles));
    ProfScope ps("paged_decode", st);
    return launch_pdl(paged_attn_kernel<T, D, GP, kTma>, dim3(grid), dim3(kThreads), smem, st, a, kmap, vmap, parts, arrived);
}

// Pages of 8 rows and more are copied by TMA, whose boxes are whole blocks of 8 rows; smaller ones row by row.
template <typename T, int D, int GP>
cudaError_t launch_page(const PagedAttnArgs &a, float *parts, int32_t *arrived, cudaStream_t st) {
    return a.lps >= 3 ? launch<T, D, GP, true>(a, parts, arrived, st) : launch<T, D, GP, false>(a, parts, arrived, st);
}

template <int D>
cudaError_t launch_dim(const PagedAttnArgs &a, float *parts, int32_t *arrived, cudaStream_t st) {
    if (a.dtype == ZHA_BF16) return launch_page<__nv_bfloat16, D, kRows>(a, parts, arrived, st);
    return a.G <= 8 ? launch_page<float, D, 8>(a, parts, arrived, st) : launch_page<float, D, 16>(a, parts, arrived, st);
}

size_t pieces_bytes(const PagedAttnArgs &a) { return (size_t)kMaxWorkers * 2 * piece_floats(a.G, a.d) * sizeof(float); }

}  // namespace

// A counter per piece for sets and one for groups, then two pieces per CTA. (The counters come first: their place
// is the same for all configurations, so that one workspace serves several.)
constexpr size_t kCounterBytes = 4 * kMaxWorkers * sizeof(int32_t);
static_assert(kCounterBytes % 16 == 0, "pieces are whole float4s");

size_t paged_attn_workspace(const PagedAttnArgs &a) { return kCounterBytes + pieces_bytes(a); }

cudaError_t launch_paged_attention(const PagedAttnArgs &a, cudaStream_t st) {
    int32_t *arrived = static_cast<int32_t *>(a.ws);
    float *parts = reinterpret_cast<float *>(static_cast<char *>(a.ws) + kCounterBytes);
    return a.d == 128 ? launch_dim<128>(a, parts, arrived, st) : launch_dim<64>(a, parts, arrived, st);
}

}  // namespace zha
