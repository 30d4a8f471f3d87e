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

// paged_append.cu: Q may be NULL (keys and values alone); strides in elements.
cudaError_t paged_append(const void *Q, const void *K, const void *V, long long qs, long long ks, long long vs,
                         const void *gq, const void *gk, float eps, const float *inv_freq, void *q_out,
                         void *k_pages, void *v_pages, const PagedSeqs &sq, int T, int n_q, int n_kv, int hd,
                         int in_dtype, int dtype, unsigned *status, cudaStream_t st);

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
