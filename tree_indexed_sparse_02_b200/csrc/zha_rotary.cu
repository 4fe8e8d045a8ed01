// zha_rotary.cu -- rotary positions of queries and keys, alone
// (zha_rotary_apply) or together with the scatter of keys and values into the
// paged cache (zha_paged_write): one kernel, one read of every input and one
// write of every output.
//
// Pair (x, y) of a head at position n turns by the angle a = 2 pi n freq:
//   x' = m (x cos a - y sin a),  y' = m (x sin a + y cos a);
// the transposed map (the gradient) has the sine's sign flipped.
//
// A warp works on one token (or a share of its heads, where tokens are few).
// A head is NP lanes' work, each with two 16-byte chunks that hold whole
// pairs, so a lane turns the same coordinates of every head it meets: its
// cosines and sines stay in registers, formed once per token by the whole warp
// (one or two per lane, dealt out by shuffles).
#include "zha_paged.h"

namespace zha {

namespace {

constexpr int kWarps = 8;                // per CTA
constexpr int kFillWarps = 148 * 32;     // warps that fill the GPU: with fewer tokens, a token gets several
constexpr int kDepth = 2;                // heads whose loads a lane has in flight (16,384 tokens: 48.6 us; 3: 49.9, 4: 50.8)

template <typename T>
struct Vec {                             // 16 bytes
    static constexpr int N = 16 / sizeof(T);
    uint4 raw;
    __device__ __forceinline__ void load(const T *p) { raw = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<uint4 *>(p) = raw; }
    __device__ __forceinline__ T *at() { return reinterpret_cast<T *>(&raw); }
};

__device__ __forceinline__ void turn(float &x, float &y, float2 cs) {
    const float a = x * cs.x - y * cs.y, b = x * cs.y + y * cs.x;
    x = a;
    y = b;
}

// (m cos, m sin) of n * f turns. The turns are reduced in fp64 to a quarter
// turn around the nearest multiple, so that a position of 2^30 costs no bits.
// What is left is rounded to fp32 and its sine and cosine taken there: a few
// units of 2^-24 of the pair's size, as the products' own roundings are (fp32,
// 1,537 tokens against 64 bits: 2.7e-8 of the result's norm; with sines, cosines
// and m in fp64, rounded once, and torch's products: 3.0e-8).
__device__ __forceinline__ float2 cos_sin(int n, double f, float m, float sign) {
    const double t = 4.0 * (double)n * f;
    const double k = rint(t);
    const float r = (float)(t - k);                  // quarter turns, in [-1/2, 1/2]
    float s, c;
    sincospif(0.5f * r, &s, &c);
    const int quad = (int)((long long)k & 3);
    const float cc = (quad & 1) ? s : c, ss = (quad & 1) ? c : s;
    return make_float2(m * ((quad == 1 || quad == 2) ? -cc : cc), sign * m * ((quad >= 2) ? -ss : ss));
}

// The two chunks of a lane, c of NP, and the pairs in them:
//   kHalf         chunk c of the first half of the rotated part and its
//                 partner in the second, then chunks that pass through;
//   kInterleaved  chunks c and c + NP, each of V / 2 whole pairs (also where
//                 nothing is rotated);
//   kStaged       the same chunks of a half layout whose halves are not whole
//                 chunks: the partners come through shared memory.
enum { kHalf = 0, kInterleaved = 1, kStaged = 2 };

template <typename T, int D, int MODE>
__global__ void __launch_bounds__(kWarps * 32, 4) rotary_kernel(const __grid_constant__ RotaryArgs a, int share) {
    constexpr int V = Vec<T>::N, NP = D / (2 * V), HW = 32 / NP;   // HW: heads of a warp at a time
    constexpr int PL = D / 64;                                      // pairs whose sine a lane forms
    __shared__ Vec<T> staged[MODE == kStaged ? kWarps : 1][MODE == kStaged ? 64 : 1];
    __shared__ float2 table[MODE == kStaged ? kWarps : 1][MODE == kStaged ? D / 2 : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = lane & (NP - 1), hs = lane / NP;
    const int job = blockIdx.x * kWarps + warp, t = job / share, part = job - t * share;
    if (t >= a.n_tokens) return;
    const int half = a.rd >> 1;
    pdl_wait();

    int64_t row = 0;                     // the token's cache row
    if (a.slots) {
        const int s = a.slots[t];
        if (s >= a.n_slots && lane == 0) set_status(a.status, ZHA_ERR_INVALID_ARG);
        if (s < 0 || s >= a.n_slots) return;
        row = ((int64_t)(s >> a.lps) * a.Hk << a.lps) + (s & ((1 << a.lps) - 1));
    }
    // elements of the lane's two chunks in a head: of queries and keys, and of values
    const int nrot = half / V, va = c * V, vb = (c + NP) * V;
    int ea = va, eb = vb;
    if (MODE == kHalf) {
        ea = c < nrot ? c * V : a.rd + (c - nrot) * V;
        eb = c < nrot ? half + c * V : a.rd + (c - nrot + NP - nrot) * V;
    }
    // heads hs + HW j, j = part, part + share, ...: queries, then keys, then values
    const int heads = a.Hq + a.Hk + (a.v ? a.Hk : 0);
    struct Place {
        const T *src;
        T *dst;
        int ea, eb;
        bool rotate;
    };
    auto place = [&](int h) {
        Place p;
        p.rotate = h < a.Hq + a.Hk;
        p.ea = p.rotate ? ea : va;
        p.eb = p.rotate ? eb : vb;
        if (h < a.Hq) {
            p.src = static_cast<const T *>(a.q) + t * a.q_stride + h * D;
            p.dst = static_cast<T *>(a.q_out) + t * a.q_out_stride + h * D;
        } else if (p.rotate) {
            h -= a.Hq;
            p.src = static_cast<const T *>(a.k) + t * a.k_stride + h * D;
            p.dst = a.slots ? static_cast<T *>(a.kpool) + (row + ((int64_t)h << a.lps)) * D
                            : static_cast<T *>(a.k_out) + t * a.k_out_stride + h * D;
        } else {
            h -= a.Hq + a.Hk;
            p.src = static_cast<const T *>(a.v) + t * a.v_stride + h * D;
            p.dst = static_cast<T *>(a.vpool) + (row + ((int64_t)h << a.lps)) * D;
        }
        return p;
    };

    Vec<T> x[kDepth], y[kDepth];
    auto load = [&](int h, Vec<T> &u, Vec<T> &v) {
        u.raw = v.raw = make_uint4(0, 0, 0, 0);
        if (h < heads) {
            const Place p = place(h);
            u.load(p.src + p.ea);
            v.load(p.src + p.eb);
        }
    };
    const int step = HW * share;
    int h0 = hs + HW * part;
#pragma unroll
    for (int e = 0; e < kDepth; ++e) load(h0 + e * step, x[e], y[e]);

    // cosines and sines: the warp's lanes form the token's pairs, then each takes those of its chunks
    float2 cs[V];
    {
        float2 mine[PL];
#pragma unroll
        for (int e = 0; e < PL; ++e) {
            const int p = lane * PL + e;
            mine[e] = p < half ? cos_sin(a.positions[t], a.freq[p], a.mscale, a.sign) : make_float2(1.f, 0.f);
            if (MODE == kStaged) table[warp][p] = mine[e];
        }
        if (MODE == kStaged) {
            __syncwarp();
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int p = MODE == kHalf ? c * V + k : (k < V / 2 ? c * (V / 2) + k : (c + NP) * (V / 2) + k - V / 2);
                const int from = (p / PL) & 31, e = MODE == kHalf || V / 2 % PL == 0 ? k % PL : p % PL;
                cs[k].x = __shfl_sync(0xffffffffu, mine[e].x, from);
                cs[k].y = __shfl_sync(0xffffffffu, mine[e].y, from);
            }
        }
    }

    for (; h0 - hs < heads; h0 += kDepth * step) {
#pragma unroll
        for (int e = 0; e < kDepth; ++e) {
            const int h = h0 + e * step;
            Vec<T> u = x[e], v = y[e];
            load(h + kDepth * step, x[e], y[e]);
            if (MODE == kStaged) {
                __syncwarp();
                staged[warp][hs * 2 * NP + c] = u;
                staged[warp][hs * 2 * NP + NP + c] = v;
                __syncwarp();
            }
            if (h >= heads) continue;
            const Place p = place(h);
            if (p.rotate) {
                if (MODE == kHalf) {
                    if (c < nrot) {
#pragma unroll
                        for (int k = 0; k < V; ++k) {
                            float f = to_f32(u.at()[k]), g = to_f32(v.at()[k]);
                            turn(f, g, cs[k]);
                            u.at()[k] = from_f32<T>(f);
                            v.at()[k] = from_f32<T>(g);
                        }
                    }
                } else if (MODE == kInterleaved) {
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        Vec<T> &w = k < V / 2 ? u : v;
                        const int i = k < V / 2 ? 2 * k : 2 * k - V;
                        if ((k < V / 2 ? va : vb) + i >= a.rd) continue;
                        float f = to_f32(w.at()[i]), g = to_f32(w.at()[i + 1]);
                        turn(f, g, cs[k]);
                        w.at()[i] = from_f32<T>(f);
                        w.at()[i + 1] = from_f32<T>(g);
                    }
                } else {
                    const T *head = reinterpret_cast<const T *>(&staged[warp][hs * 2 * NP]);
#pragma unroll
                    for (int k = 0; k < 2 * V; ++k) {
                        const int i = (k < V ? va : vb - V) + k;
                        if (i >= a.rd) continue;
                        const int q = i < half ? i : i - half;
                        float f = to_f32(head[q]), g = to_f32(head[q + half]);
                        turn(f, g, table[warp][q]);
                        (k < V ? u : v).at()[k % V] = from_f32<T>(i < half ? f : g);
                    }
                }
            }
            u.store(p.dst + p.ea);
            v.store(p.dst + p.eb);
        }
    }
    // no early trigger: a kernel behind this one may read q_out before its own wait
}

template <typename T, int D, int MODE>
cudaError_t launch_mode(const RotaryArgs &a, cudaStream_t st) {
    constexpr int HW = 32 / (D / (2 * Vec<T>::N));
    // warps per token: one where tokens alone fill the GPU, more where they do not, up to one for each HW heads
    const int most = (a.Hq + a.Hk + (a.v ? a.Hk : 0) + HW - 1) / HW, want = kFillWarps / a.n_tokens;
    const int share = want < 1 ? 1 : want > most ? most : want;
    const int64_t jobs = (int64_t)a.n_tokens * share;
    if (jobs > INT32_MAX - kWarps) return cudaErrorInvalidValue;
    ProfScope ps(a.slots ? "paged_write" : "rotary", st);
    return launch_pdl(rotary_kernel<T, D, MODE>, dim3((unsigned)((jobs + kWarps - 1) / kWarps)), dim3(kWarps * 32), 0, st, a, share);
}

template <typename T, int D>
cudaError_t launch_dim(const RotaryArgs &a, cudaStream_t st) {
    if (a.rd == 0 || a.layout == ZHA_ROPE_INTERLEAVED) return launch_mode<T, D, kInterleaved>(a, st);
    if ((a.rd / 2) % Vec<T>::N == 0) return launch_mode<T, D, kHalf>(a, st);
    return launch_mode<T, D, kStaged>(a, st);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs &a, cudaStream_t st) {
    if (a.dtype == ZHA_BF16)
        return a.d == 128 ? launch_dim<__nv_bfloat16, 128>(a, st) : launch_dim<__nv_bfloat16, 64>(a, st);
    return a.d == 128 ? launch_dim<float, 128>(a, st) : launch_dim<float, 64>(a, st);
}

}  // namespace zha
