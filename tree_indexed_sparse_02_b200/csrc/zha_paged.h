// zha_paged.h -- arguments of the paged-cache kernels and their launchers.
// Internal to libzha.
#pragma once

#include "zha_common.cuh"

namespace zha {

constexpr int kPagedMaxBatch = 4096;     // the plan kernel holds every sequence in shared memory

__host__ __device__ inline int div_up(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

struct PlanArgs {
    int B, lps, n_pages, max_pages;      // lps: log2(page_size)
    int max_tokens;
    int32_t *table, *free_pages;
    const int32_t *lens, *n_new, *n_free;
    int32_t *lens_out, *n_free_out;
    int32_t *positions, *slots, *seq_ids, *cu_new;
    int32_t *status;
};
cudaError_t launch_paged_plan(const PlanArgs &a, cudaStream_t st);

// One launch rotates queries and keys and, for a cache write (slots != null),
// scatters keys and values; without slots k goes to k_out.
struct RotaryArgs {
    const double *freq;                  // null: no rotation (rd = 0)
    int rd, layout;
    float mscale, sign;                  // sign: -1 for the transposed map
    int n_tokens, Hq, Hk, d, dtype;
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;        // elements
    const int32_t *positions, *slots;
    void *q_out, *k_out;
    int64_t q_out_stride, k_out_stride;
    void *kpool, *vpool;                 // cache write
    int lps;
    int64_t n_slots;
    int32_t *status;
};
cudaError_t launch_rotary(const RotaryArgs &a, cudaStream_t st);

struct PagedAttnArgs {
    int rows, batch, Hq, Hkv, G, d, dtype;
    int lps, n_pages, max_pages, window;
    float s;
    const void *q, *kpool, *vpool;
    const int32_t *table, *lens, *seq_ids, *positions;
    void *out;
    float *lse;
    void *ws;
    int32_t *status;
};
size_t paged_attn_workspace(const PagedAttnArgs &a);
cudaError_t launch_paged_attention(const PagedAttnArgs &a, cudaStream_t st);

}  // namespace zha
