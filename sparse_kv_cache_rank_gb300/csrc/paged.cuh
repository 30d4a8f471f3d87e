// paged.cuh -- the paged cache and the ragged batch that the paged operators share: pages
// [n_pages, page, n_kv, hd] of keys and of values, a page table [B, max_pages], and the new
// rows of sequence b at q_start[b] .. q_start[b+1] of the flattened batch, the last of them
// at position kv_len[b] - 1.
#pragma once

#include "internal.h"

namespace dllm {

constexpr int kPagedMaxSeqs = 1024;   // sequences of a batch

struct PagedSeqs {
    const int32_t *q_start;      // [B + 1] ascending
    const int32_t *kv_len;       // [B] keys of the sequence, its new rows included
    const int32_t *page_table;   // [B, max_pages]
    int B, max_pages;
    int page_log2;               // rows of a page (a power of two)
    int n_pages;

    // Keys that the row at position pos sees: all of them (mask_block == 0), else the
    // blocks of mask_block positions up to its own (1: causal).
    __device__ __forceinline__ static int visible(int pos, int len, int mask_block) {
        if (mask_block == 0) return len;
        if (pos < 0) return 0;
        const long long end = ((long long)pos / mask_block + 1) * mask_block;
        return end < len ? (int)end : len;
    }
    // New rows of sequence b: the first one's row of the batch, their number (which sets their
    // positions) and how many of them there are inside [0, T) and below max_new.
    __device__ __forceinline__ int rows(int b, int T, int max_new, int &start, int &n_new) const {
        start = q_start[b];
        const int end = q_start[b + 1];
        n_new = end - start;
        if (start < 0 || end <= start || start >= T) return 0;
        return min(min(n_new, max_new), T - start);
    }
    // Keys of sequence b that the table can hold (a longer kv_len is cut there).
    __device__ __forceinline__ int keys(int b) const {
        const int len = kv_len[b];
        const long long cap = (long long)max_pages << page_log2;
        return len < 0 ? 0 : (len < cap ? len : (int)cap);
    }
};

__device__ __forceinline__ float ex2(float x) {   // 2^x, relative error ~2^-22; 2^-inf = 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// paged_append.cu: Q may be NULL (keys and values alone); strides in elements.
cudaError_t paged_append(const void *Q, const void *K, const void *V, long long qs, long long ks, long long vs,
                         const void *gq, const void *gk, float eps, const float *inv_freq,
                         const int32_t *pos_base, void *q_out, void *k_pages, void *v_pages, const PagedSeqs &sq,
                         int T, int n_q, int n_kv, int hd, int in_dtype, int dtype, unsigned *status, cudaStream_t st);

// paged_append_f8.cu: 8-bit pages with a scale for each page and head; Q_out and the gains are bf16.
struct AppendF8 {
    const void *src[3];       // Q (may be NULL), K, V
    long long stride[3];      // elements between rows
    const bf16 *gamma[2];     // of Q and K, or NULL
    const float *inv_freq;    // [hd/2] or NULL
    const int32_t *pos_base;  // [B] or NULL
    bf16 *q_out;
    uint8_t *pages[2], *scale[2];   // of K and V
    PagedSeqs sq;
    int T, n_q, n_kv;         // n_q = 0 without Q
    float eps;
};
cudaError_t paged_append_f8(const AppendF8 &a, int hd, int in_dtype, unsigned *status, cudaStream_t st);

struct PagedAttn {
    const void *Q, *k_pages, *v_pages;
    long long q_stride;   // elements between rows of Q
    void *A;
    float *lse;           // [T, n_q] or NULL
    PagedSeqs sq;
    int T, max_new, n_q, n_kv, hd, mask_block;
    float scale;
};
// paged_attention.cu: fp32, operands split into TF32 parts; paged_attention_tc.cu: bf16.
// Two launches each, partial results in ws.
size_t paged_attention_f32_ws_bytes(int max_new, int n_q, int n_kv, int hd);
cudaError_t paged_attention_f32(const PagedAttn &p, void *ws, cudaStream_t st);
size_t paged_attention_tc_ws_bytes(int max_new, int n_q, int n_kv, int hd);
cudaError_t paged_attention_tc(const PagedAttn &p, void *ws, unsigned *status, cudaStream_t st);

// paged_attention_f8.cu: 8-bit pages, bf16 queries and results.  Two launches, partial results in ws.
size_t paged_attention_f8_ws_bytes(int max_new, int n_q, int n_kv, int hd);
cudaError_t paged_attention_f8(const PagedAttn &p, const uint8_t *k_scale, const uint8_t *v_scale, void *ws, unsigned *status,
                               cudaStream_t st);

// The attention weight that each key receives; dtype by the function.
struct PagedWeights {
    const void *Q, *k_pages;
    const uint8_t *k_scale;      // 8-bit pages
    long long q_stride;
    const float *lse;            // [T, n_q]
    const int32_t *pos_base;     // [B] or NULL
    const float *score;          // [B, n_kv, slots]
    float *score_out;            // may be score
    int32_t *slot_pos;           // [B, n_kv, slots] or NULL
    int slots;
    PagedSeqs sq;
    int T, max_new, n_q, n_kv, hd, mask_block;
    float scale;
};
// paged_weights_tc.cu: bf16 queries, bf16 or 8-bit pages; paged_weights_f32.cu: fp32.
cudaError_t paged_weights_tc(const PagedWeights &p, bool f8, unsigned *status, cudaStream_t st);
cudaError_t paged_weights_f32(const PagedWeights &p, cudaStream_t st);

// paged_evict.cu: slots given up by their scores.  Two launches, lists in ws.
struct PagedEvict {
    void *k_pages, *v_pages;
    uint8_t *k_scale, *v_scale;         // 8-bit pages, else NULL
    const int32_t *kv_len, *keep;       // [B]
    const int32_t *pos_base;            // [B] or NULL
    const float *score;                 // [B, n_kv, slots]
    const int32_t *slot_pos;
    float *score_out;                   // may be their inputs
    int32_t *slot_pos_out, *kv_len_out, *pos_base_out;
    PagedSeqs sq;                       // (q_start unused)
    int slots, n_kv, recent;
};
size_t paged_evict_ws_bytes(int B, int n_kv, int slots, bool f8);
cudaError_t paged_evict(const PagedEvict &p, int row_bytes, void *ws, unsigned *status, cudaStream_t st);

// sample.cu: one token per row of logits [B * M, V].
struct SampleArgs {
    const void *logits;
    const float *u, *temperature, *top_p, *min_p;   // u [B * M]; the others [B], NULL = off
    const int32_t *top_k;
    const uint8_t *valid;                           // [B * M] or NULL
    int32_t *token;
    float *prob;
    int rows, M, V;
};
int sample_max_vocab();
int sample_launches(int V);
size_t sample_ws_bytes(int rows, int V);
cudaError_t sample_tokens(const SampleArgs &a, int dtype, void *ws, cudaStream_t st);

}  // namespace dllm
