// zha_paged_api.cu -- the extern "C" entry points of the paged cache and the
// rotary positions: argument checks and dispatch.
#include <limits.h>
#include <math.h>

#include "zha_paged.h"

namespace {

bool pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// The launch's error is the call's; it is not left for the host program's next look at the last error.
zha_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return ZHA_OK;
    (void)cudaGetLastError();
    return ZHA_ERR_CUDA;
}

int log2i(int x) {
    int l = 0;
    while ((1 << l) < x) ++l;
    return l;
}

zha_status check_paged(const zha_paged_config *c) {
    if (!c) return ZHA_ERR_INVALID_ARG;
    if (c->batch < 1 || c->n_q_heads < 1 || c->n_kv_heads < 1 || c->page_size < 1 || c->n_pages < 1 ||
        c->max_pages < 1 || c->window < 0 || !(c->scale == c->scale) || isinf(c->scale))
        return ZHA_ERR_INVALID_ARG;
    if (c->reserved[0] || c->reserved[1]) return ZHA_ERR_INVALID_ARG;
    if (c->n_q_heads % c->n_kv_heads) return ZHA_ERR_INVALID_ARG;
    if (c->n_q_heads / c->n_kv_heads > 16) return ZHA_ERR_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128) return ZHA_ERR_UNSUPPORTED;
    if (c->dtype != ZHA_BF16 && c->dtype != ZHA_F32) return ZHA_ERR_UNSUPPORTED;
    if (!pow2(c->page_size) || c->page_size > 1024) return ZHA_ERR_UNSUPPORTED;
    if (c->batch > zha::kPagedMaxBatch || c->n_kv_heads > 65535) return ZHA_ERR_UNSUPPORTED;
    if ((int64_t)c->n_pages * c->page_size > (1 << 30) || (int64_t)c->max_pages * c->page_size > (1 << 30))
        return ZHA_ERR_UNSUPPORTED;
    return ZHA_OK;
}

// Rows of one attention call: counts of query heads and of tiles (of 32 tokens at least) stay in int32.
bool rows_ok(const zha_paged_config *c, int32_t n_rows) {
    return (int64_t)n_rows * c->n_q_heads <= (1 << 24) &&
           (int64_t)n_rows * c->n_kv_heads <= (int64_t(1) << 35) / c->page_size / c->max_pages;
}

zha_status check_rotary(const zha_rotary *r, int head_dim) {
    if (r->rotary_dim < 2 || (r->rotary_dim & 1) || r->rotary_dim > head_dim || r->reserved) return ZHA_ERR_INVALID_ARG;
    if (r->layout != ZHA_ROPE_HALF && r->layout != ZHA_ROPE_INTERLEAVED) return ZHA_ERR_INVALID_ARG;
    if (!isfinite(r->mscale) || !r->freq || (reinterpret_cast<uintptr_t>(r->freq) & 7u)) return ZHA_ERR_INVALID_ARG;
    return ZHA_OK;
}

// A token stride in elements: 0 is contiguous, anything else at least one
// token and a multiple of 16 bytes.
bool stride_ok(int64_t *stride, int heads, int d, int es) {
    const int64_t row = (int64_t)heads * d;
    if (*stride == 0) *stride = row;
    return *stride >= row && (*stride * es) % 16 == 0 && *stride < (int64_t(1) << 30);
}

// What a write refuses before it enqueues anything; strides of 0 become the contiguous ones.
zha_status check_write(const zha_paged_config *cfg, const zha_rotary *rotary, int32_t n_tokens, const void *q,
                       int64_t *q_stride, const void *k_new, int64_t *k_stride, const void *v_new, int64_t *v_stride,
                       const int32_t *positions, const int32_t *slots, const void *q_out, const void *kpool,
                       const void *vpool) {
    zha_status s = check_paged(cfg);
    if (s != ZHA_OK) return s;
    if (rotary && (s = check_rotary(rotary, cfg->head_dim)) != ZHA_OK) return s;
    if (n_tokens < 0) return ZHA_ERR_INVALID_ARG;
    if (n_tokens == 0) return ZHA_OK;
    if (n_tokens > (1 << 30) || cfg->n_q_heads > 1024 || cfg->n_kv_heads > 1024) return ZHA_ERR_UNSUPPORTED;
    if (!q != !q_out) return ZHA_ERR_INVALID_ARG;
    if (!k_new || !v_new || !slots || !kpool || !vpool || (rotary && !positions)) return ZHA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(q_out) || !aligned16(kpool) ||
        !aligned16(vpool))
        return ZHA_ERR_INVALID_ARG;
    const int es = cfg->dtype == ZHA_BF16 ? 2 : 4, d = cfg->head_dim;
    if ((q && !stride_ok(q_stride, cfg->n_q_heads, d, es)) || !stride_ok(k_stride, cfg->n_kv_heads, d, es) ||
        !stride_ok(v_stride, cfg->n_kv_heads, d, es))
        return ZHA_ERR_INVALID_ARG;
    return ZHA_OK;
}

zha::PagedAttnArgs attn_args(const zha_paged_config *c, int rows) {
    zha::PagedAttnArgs a{};
    a.rows = rows;
    a.batch = c->batch;
    a.Hq = c->n_q_heads;
    a.Hkv = c->n_kv_heads;
    a.G = c->n_q_heads / c->n_kv_heads;
    a.d = c->head_dim;
    a.dtype = c->dtype;
    a.lps = log2i(c->page_size);
    a.n_pages = c->n_pages;
    a.max_pages = c->max_pages;
    a.window = c->window;
    a.s = c->scale > 0.f ? c->scale : 1.f / sqrtf((float)c->head_dim);
    return a;
}

}  // namespace

extern "C" {

zha_status zha_paged_check_config(const zha_paged_config *cfg) { return check_paged(cfg); }

zha_status zha_paged_plan(const zha_paged_config *cfg, int32_t *table, const int32_t *lens,
                          const int32_t *n_new, int32_t *free_pages, const int32_t *n_free,
                          int32_t *lens_out, int32_t *n_free_out, const zha_token_map *map,
                          int32_t *dev_status, void *stream) {
    zha_status s = check_paged(cfg);
    if (s != ZHA_OK) return s;
    if (!table || !lens || !n_new || !free_pages || !n_free || !lens_out || !n_free_out || !map)
        return ZHA_ERR_INVALID_ARG;
    if (!map->positions || !map->slots || !map->seq_ids || !map->cu_new || map->max_tokens < 1 || map->reserved)
        return ZHA_ERR_INVALID_ARG;
    if (map->max_tokens > (1 << 30)) return ZHA_ERR_UNSUPPORTED;
    zha::PlanArgs a{};
    a.B = cfg->batch;
    a.lps = log2i(cfg->page_size);
    a.n_pages = cfg->n_pages;
    a.max_pages = cfg->max_pages;
    a.max_tokens = map->max_tokens;
    a.table = table;
    a.free_pages = free_pages;
    a.lens = lens;
    a.n_new = n_new;
    a.n_free = n_free;
    a.lens_out = lens_out;
    a.n_free_out = n_free_out;
    a.positions = map->positions;
    a.slots = map->slots;
    a.seq_ids = map->seq_ids;
    a.cu_new = map->cu_new;
    a.status = dev_status;
    return cuda_status(zha::launch_paged_plan(a, static_cast<cudaStream_t>(stream)));
}

zha_status zha_rotary_freqs(int32_t rotary_dim, double base, int32_t scaling, double factor,
                            int64_t original_len, double *freq, float *mscale) {
    if (rotary_dim < 2 || rotary_dim > 256 || (rotary_dim & 1) || !freq || !mscale) return ZHA_ERR_INVALID_ARG;
    if (!(base > 1.0) || isinf(base)) return ZHA_ERR_INVALID_ARG;
    if (scaling < ZHA_ROPE_PLAIN || scaling > ZHA_ROPE_YARN) return ZHA_ERR_INVALID_ARG;
    if (scaling != ZHA_ROPE_PLAIN && (!(factor > 0.0) || isinf(factor))) return ZHA_ERR_INVALID_ARG;
    if (scaling == ZHA_ROPE_YARN && (factor < 1.0 || original_len < 1)) return ZHA_ERR_INVALID_ARG;
    const double turn = 6.283185307179586476925286766559;
    const double rd = rotary_dim;
    if (scaling == ZHA_ROPE_NTK && rotary_dim > 2) base *= pow(factor, rd / (rd - 2.0));
    if (!(base > 0.0) || isinf(base)) return ZHA_ERR_INVALID_ARG;
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = pow(base, -2.0 * i / rd);
        if (scaling == ZHA_ROPE_LINEAR) f /= factor;
        if (scaling == ZHA_ROPE_YARN) {
            double g = (original_len * f / turn - 1.0) / 31.0;
            g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
            f = (1.0 - g) * f / factor + g * f;
        }
        freq[i] = f / turn;
    }
    *mscale = scaling == ZHA_ROPE_YARN ? (float)(0.1 * log(factor) + 1.0) : 1.f;
    return ZHA_OK;
}

zha_status zha_rotary_apply(const zha_rotary *rotary, int32_t head_dim, int32_t dtype,
                            int32_t n_tokens, int32_t n_q_heads, int32_t n_k_heads, const void *q,
                            int64_t q_stride, const void *k, int64_t k_stride, const int32_t *positions,
                            void *q_out, int64_t q_out_stride, void *k_out, int64_t k_out_stride,
                            int32_t transpose, void *stream) {
    if (!rotary) return ZHA_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128) return ZHA_ERR_UNSUPPORTED;
    if (dtype != ZHA_BF16 && dtype != ZHA_F32) return ZHA_ERR_UNSUPPORTED;
    zha_status s = check_rotary(rotary, head_dim);
    if (s != ZHA_OK) return s;
    if (n_tokens < 0) return ZHA_ERR_INVALID_ARG;
    if (n_tokens == 0) return ZHA_OK;
    if (n_tokens > (1 << 30)) return ZHA_ERR_UNSUPPORTED;
    if ((!q && !k) || !q != !q_out || !k != !k_out) return ZHA_ERR_INVALID_ARG;
    if ((q && n_q_heads < 1) || (k && n_k_heads < 1)) return ZHA_ERR_INVALID_ARG;
    const int Hq = q ? n_q_heads : 0, Hk = k ? n_k_heads : 0;
    if (Hq > 1024 || Hk > 1024) return ZHA_ERR_UNSUPPORTED;
    if (!positions || !aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out))
        return ZHA_ERR_INVALID_ARG;
    const int es = dtype == ZHA_BF16 ? 2 : 4;
    if (q && (!stride_ok(&q_stride, Hq, head_dim, es) || !stride_ok(&q_out_stride, Hq, head_dim, es)))
        return ZHA_ERR_INVALID_ARG;
    if (k && (!stride_ok(&k_stride, Hk, head_dim, es) || !stride_ok(&k_out_stride, Hk, head_dim, es)))
        return ZHA_ERR_INVALID_ARG;
    zha::RotaryArgs a{};
    a.freq = rotary->freq;
    a.rd = rotary->rotary_dim;
    a.layout = rotary->layout;
    a.mscale = rotary->mscale;
    a.sign = transpose ? -1.f : 1.f;
    a.n_tokens = n_tokens;
    a.Hq = Hq;
    a.Hk = Hk;
    a.d = head_dim;
    a.dtype = dtype;
    a.q = q;
    a.k = k;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.positions = positions;
    a.q_out = q_out;
    a.k_out = k_out;
    a.q_out_stride = q_out_stride;
    a.k_out_stride = k_out_stride;
    return cuda_status(zha::launch_rotary(a, static_cast<cudaStream_t>(stream)));
}

zha_status zha_paged_write_check(const zha_paged_config *cfg, const zha_rotary *rotary, int32_t n_tokens,
                                 const void *q, int64_t q_stride, const void *k_new, int64_t k_stride,
                                 const void *v_new, int64_t v_stride, const int32_t *positions,
                                 const int32_t *slots, const void *q_out, const void *kpool, const void *vpool) {
    return check_write(cfg, rotary, n_tokens, q, &q_stride, k_new, &k_stride, v_new, &v_stride, positions, slots, q_out, kpool,
                       vpool);
}

zha_status zha_paged_write(const zha_paged_config *cfg, const zha_rotary *rotary, int32_t n_tokens,
                           const void *q, int64_t q_stride, const void *k_new, int64_t k_stride,
                           const void *v_new, int64_t v_stride, const int32_t *positions,
                           const int32_t *slots, void *q_out, void *kpool, void *vpool,
                           int32_t *dev_status, void *stream) {
    const zha_status s = check_write(cfg, rotary, n_tokens, q, &q_stride, k_new, &k_stride, v_new, &v_stride, positions, slots,
                                     q_out, kpool, vpool);
    if (s != ZHA_OK || n_tokens == 0) return s;
    const int d = cfg->head_dim;
    zha::RotaryArgs a{};
    if (rotary) {
        a.freq = rotary->freq;
        a.rd = rotary->rotary_dim;
        a.layout = rotary->layout;
        a.mscale = rotary->mscale;
    }
    a.sign = 1.f;
    a.n_tokens = n_tokens;
    a.Hq = q ? cfg->n_q_heads : 0;
    a.Hk = cfg->n_kv_heads;
    a.d = d;
    a.dtype = cfg->dtype;
    a.q = q;
    a.k = k_new;
    a.v = v_new;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.positions = positions;
    a.slots = slots;
    a.q_out = q_out;
    a.q_out_stride = (int64_t)cfg->n_q_heads * d;
    a.kpool = kpool;
    a.vpool = vpool;
    a.lps = log2i(cfg->page_size);
    a.n_slots = (int64_t)cfg->n_pages * cfg->page_size;
    a.status = dev_status;
    return cuda_status(zha::launch_rotary(a, static_cast<cudaStream_t>(stream)));
}

size_t zha_paged_workspace_bytes(const zha_paged_config *cfg, int32_t n_rows) {
    if (check_paged(cfg) != ZHA_OK || n_rows < 1 || !rows_ok(cfg, n_rows)) return 0;
    return zha::paged_attn_workspace(attn_args(cfg, n_rows));
}

zha_status zha_paged_decode(const zha_paged_config *cfg, int32_t n_rows, const void *q, const void *kpool,
                            const void *vpool, const int32_t *table, const int32_t *lens,
                            const int32_t *seq_ids, const int32_t *positions, void *out, float *lse,
                            void *workspace, int32_t *dev_status, void *stream) {
    zha_status s = check_paged(cfg);
    if (s != ZHA_OK) return s;
    if (n_rows < 0 || (!seq_ids && n_rows > cfg->batch)) return ZHA_ERR_INVALID_ARG;
    if (n_rows == 0) return ZHA_OK;
    if (!rows_ok(cfg, n_rows)) return ZHA_ERR_UNSUPPORTED;
    if (!q || !kpool || !vpool || !table || !lens || !out || !workspace) return ZHA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(kpool) || !aligned16(vpool) || !aligned16(out) || !aligned16(workspace))
        return ZHA_ERR_INVALID_ARG;
    zha::PagedAttnArgs a = attn_args(cfg, n_rows);
    a.q = q;
    a.kpool = kpool;
    a.vpool = vpool;
    a.table = table;
    a.lens = lens;
    a.seq_ids = seq_ids;
    a.positions = positions;
    a.out = out;
    a.lse = lse;
    a.ws = workspace;
    a.status = dev_status;
    return cuda_status(zha::launch_paged_attention(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
