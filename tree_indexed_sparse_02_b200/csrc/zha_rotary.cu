// zha_rotary.cu -- rotary positions of queries and keys, alone
// (zha_rotary_apply) or together with the scatter of keys and values into the
// paged cache (zha_paged_write): one kernel, one read of every input and one
// write of every output.
//
// Pair (x, y) of a head at position n turns by the angle a = 2 pi n freq:
//   x' = m (x cos a - y sin a),  y' = m (x sin a + y cos a);
// the transposed map (the gradient) has the sine's sign flipped.
#include "zha_paged.cuh"

namespace zha {

namespace {

constexpr int kThreads = 256;

// n / D for n < 2^16 and D < 2^16 by one multiplication.
struct Div {
    uint64_t m;
    int D;
    explicit Div(int d = 1) : m(((uint64_t(1) << 32) + d - 1) / d), D(d) {}
    __device__ __forceinline__ int of(int n) const { return (int)(((uint64_t)(uint32_t)n * m) >> 32); }
};

struct Shape {
    int items_rot;          // items of a q or k head
    int items_v;            // items of a v head
    int items_q;            // items of a token's q heads; then k, then v heads
    int items_qk, items_all;
    int tok;                // tokens per CTA
    int per;                // items of each token per CTA (blockIdx.y chooses which)
    Div by_per, by_rot;
};

template <typename T>
struct Vec {                // 16 bytes
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

enum { kHalfVec = 0, kPairVec = 1, kScalar = 2 };

// MODE kHalfVec: an item of a q/k head is a 16-byte chunk of the first half
// with its partner in the second, or a chunk that passes through;
// kPairVec (interleaved): a 16-byte chunk; kScalar (half layouts whose halves
// are not whole chunks): one pair, or one coordinate that passes through.
template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads) rotary_kernel(RotaryArgs a, Shape sh) {
    constexpr int V = Vec<T>::N;
    extern __shared__ float2 cs[];                   // [tok][rd / 2]
    __shared__ int64_t row[64];                      // cache row of each token, -1: skip
    const int t0 = blockIdx.x * sh.tok, i0 = blockIdx.y * sh.per;
    const int nt = min(sh.tok, a.n_tokens - t0), ni = min(sh.per, sh.items_all - i0);
    const int half = a.rd >> 1;
    pdl_wait();
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int t = i / half, p = i - t * half;
        cs[i] = cos_sin(a.positions[t0 + t], a.freq[p], a.mscale, a.sign);
    }
    if (a.slots && threadIdx.x < nt) {
        const int s = a.slots[t0 + threadIdx.x];
        if (s >= a.n_slots && blockIdx.y == 0) set_status(a.status, ZHA_ERR_INVALID_ARG);
        row[threadIdx.x] = (s < 0 || s >= a.n_slots)
                               ? -1
                               : ((int64_t)(s >> a.lps) * a.Hk << a.lps) + (s & ((1 << a.lps) - 1));
    }
    __syncthreads();
    for (int idx = threadIdx.x; idx < nt * sh.per; idx += kThreads) {
        const int t = sh.by_per.of(idx), it = idx - t * sh.per + i0;
        if (it - i0 >= ni) continue;
        const int64_t tk = t0 + t;
        const int64_t rw = a.slots ? row[t] : 0;
        if (rw < 0) continue;
        if (it >= sh.items_qk) {                     // values: copied
            const int j = it - sh.items_qk, h = j / sh.items_v, c = j - h * sh.items_v;
            Vec<T> x;
            x.load(static_cast<const T *>(a.v) + tk * a.v_stride + h * a.d + c * V);
            x.store(static_cast<T *>(a.vpool) + (rw + ((int64_t)h << a.lps)) * a.d + c * V);
            continue;
        }
        const bool is_k = it >= sh.items_q;
        const int j = is_k ? it - sh.items_q : it;
        const int h = sh.by_rot.of(j), c = j - h * sh.items_rot;
        const T *src;
        T *dst;
        if (!is_k) {
            src = static_cast<const T *>(a.q) + tk * a.q_stride + h * a.d;
            dst = static_cast<T *>(a.q_out) + tk * a.q_out_stride + h * a.d;
        } else {
            src = static_cast<const T *>(a.k) + tk * a.k_stride + h * a.d;
            dst = a.slots ? static_cast<T *>(a.kpool) + (rw + ((int64_t)h << a.lps)) * a.d
                          : static_cast<T *>(a.k_out) + tk * a.k_out_stride + h * a.d;
        }
        const float2 *w = cs + t * half;
        if (MODE == kHalfVec) {
            const int nrot = half / V;
            if (c < nrot) {
                Vec<T> x, y;
                x.load(src + c * V);
                y.load(src + half + c * V);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float u = to_f32(x.at()[e]), v = to_f32(y.at()[e]);
                    turn(u, v, w[c * V + e]);
                    x.at()[e] = from_f32<T>(u);
                    y.at()[e] = from_f32<T>(v);
                }
                x.store(dst + c * V);
                y.store(dst + half + c * V);
            } else {
                Vec<T> x;
                x.load(src + a.rd + (c - nrot) * V);
                x.store(dst + a.rd + (c - nrot) * V);
            }
        } else if (MODE == kPairVec) {
            Vec<T> x;
            x.load(src + c * V);
#pragma unroll
            for (int e = 0; e < V; e += 2) {
                const int p = (c * V + e) >> 1;
                if (p < half) {
                    float u = to_f32(x.at()[e]), v = to_f32(x.at()[e + 1]);
                    turn(u, v, w[p]);
                    x.at()[e] = from_f32<T>(u);
                    x.at()[e + 1] = from_f32<T>(v);
                }
            }
            x.store(dst + c * V);
        } else {
            if (c < half) {
                float u = to_f32(src[c]), v = to_f32(src[half + c]);
                turn(u, v, w[c]);
                dst[c] = from_f32<T>(u);
                dst[half + c] = from_f32<T>(v);
            } else {
                dst[half + c] = src[half + c];
            }
        }
    }
    // no early trigger: a kernel behind this one may read q_out before its own wait
}

template <typename T, int MODE>
cudaError_t launch_mode(const RotaryArgs &a, cudaStream_t st) {
    constexpr int V = Vec<T>::N;
    Shape sh;
    const int half = a.rd / 2;
    sh.items_rot = MODE == kHalfVec ? half / V + (a.d - a.rd) / V : MODE == kPairVec ? a.d / V : half + (a.d - a.rd);
    sh.items_v = a.d / V;
    sh.items_q = a.Hq * sh.items_rot;
    sh.items_qk = sh.items_q + a.Hk * sh.items_rot;
    sh.items_all = sh.items_qk + (a.v ? a.Hk * sh.items_v : 0);
    sh.per = sh.items_all < 1024 ? sh.items_all : 1024;
    sh.tok = 1024 / sh.per;
    if (sh.tok > 16) sh.tok = 16;
    sh.by_per = Div(sh.per);
    sh.by_rot = Div(sh.items_rot);
    const dim3 grid((a.n_tokens + sh.tok - 1) / sh.tok, (sh.items_all + sh.per - 1) / sh.per);
    ProfScope ps(a.slots ? "paged_write" : "rotary", st);
    return launch_pdl(rotary_kernel<T, MODE>, grid, dim3(kThreads), sizeof(float2) * sh.tok * (half ? half : 1), st, a, sh);
}

template <typename T>
cudaError_t launch_type(const RotaryArgs &a, cudaStream_t st) {
    constexpr int V = Vec<T>::N;
    if (a.rd == 0 || a.layout == ZHA_ROPE_INTERLEAVED) return launch_mode<T, kPairVec>(a, st);
    if ((a.rd / 2) % V == 0) return launch_mode<T, kHalfVec>(a, st);
    return launch_mode<T, kScalar>(a, st);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs &a, cudaStream_t st) {
    return a.dtype == ZHA_BF16 ? launch_type<__nv_bfloat16>(a, st) : launch_type<float>(a, st);
}

}  // namespace zha
