// paged_attention.cu -- attention of ragged new rows over a paged cache on the CUDA cores
// (fp32).
//
//   A[t, h] = softmax_j(<Q[t, h], K_j> scale) V_j  over the keys j < visible(pos(t)),
// zeros for a row that sees none.  One CTA (4 warps) per (row, head); warp w takes every
// fourth key; each lane holds hd / 32 dims, so a score is a warp all-reduce over one
// coalesced key row.  The warps keep the running max / sum form in fp32 and are merged in
// warp order.
#include "paged.cuh"

namespace dllm {
namespace {

constexpr int kW = 4;

template <class T, int EPL>
__global__ void __launch_bounds__(kW * 32) k_paged_attention(const T *__restrict__ Q, long long q_stride,
                                                             const T *__restrict__ Kp, const T *__restrict__ Vp,
                                                             T *__restrict__ A, float *__restrict__ lse,
                                                             PagedSeqs sq, int max_new, int n_q, int n_kv, int mask_block,
                                                             float scale) {
    constexpr int hd = EPL * 32;
    __shared__ float wm[kW], wl[kW];
    __shared__ float wacc[kW][hd];
    griddep_wait();
    griddep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x, h = blockIdx.y;
    int cnt = 0;
    for (int i = threadIdx.x; i < (sq.B + 127) / 128 * 128; i += kW * 32)
        cnt += __syncthreads_count(i < sq.B && sq.q_start[i + 1] <= t);
    const int b = cnt;
    if (b >= sq.B || t < sq.q_start[b] || t - sq.q_start[b] >= max_new) return;   // not a row of a sequence: left as it was
    const int len = sq.keys(b);
    const int pos = sq.kv_len[b] - (sq.q_start[b + 1] - t);
    const int lim = PagedSeqs::visible(pos, len, mask_block);
    const int g = h / (n_q / n_kv);
    const size_t row = (size_t)n_kv * hd;
    float q[EPL], acc[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
        q[e] = to_f32<T>(Q[(size_t)t * q_stride + (size_t)h * hd + lane * EPL + e]) * scale;
        acc[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int j = warp; j < lim; j += kW) {
        const int id = sq.page_table[(size_t)b * sq.max_pages + (j >> sq.page_log2)];
        if (id < 0 || id >= sq.n_pages) continue;   // no page: the key is absent
        const size_t at = (((size_t)id << sq.page_log2) + (j & ((1 << sq.page_log2) - 1))) * row + (size_t)g * hd + lane * EPL;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < EPL; ++e) s = fmaf(q[e], to_f32<T>(Kp[at + e]), s);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        const float nm = fmaxf(m, s);
        const float c = nm == -INFINITY ? 1.f : expf(m - nm), p = nm == -INFINITY ? 0.f : expf(s - nm);
        l = l * c + p;
#pragma unroll
        for (int e = 0; e < EPL; ++e) acc[e] = fmaf(p, to_f32<T>(Vp[at + e]), acc[e] * c);
        m = nm;
    }
    if (lane == 0) {
        wm[warp] = m;
        wl[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < EPL; ++e) wacc[warp][lane * EPL + e] = acc[e];
    __syncthreads();
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kW; ++w) M = fmaxf(M, wm[w]);
    float den = 0.f, c[kW];
#pragma unroll
    for (int w = 0; w < kW; ++w) {
        c[w] = wm[w] == -INFINITY ? 0.f : expf(wm[w] - M);
        den = fmaf(wl[w], c[w], den);
    }
    const float inv = den != 0.f ? 1.0f / den : 0.f;
    for (int e = threadIdx.x; e < hd; e += kW * 32) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kW; ++w) v = c[w] == 0.f ? v : fmaf(wacc[w][e], c[w], v);
        A[((size_t)t * n_q + h) * hd + e] = from_f32<T>(v * inv);
    }
    if (lse && threadIdx.x == 0) lse[(size_t)t * n_q + h] = den != 0.f ? M + logf(den) : -INFINITY;
}

template <class T>
cudaError_t launch(const PagedAttn &p, cudaStream_t st) {
    const dim3 grid(p.T, p.n_q);
    if (p.hd == 64)
        return launch_kernel(k_paged_attention<T, 2>, grid, dim3(kW * 32), 0, st, 1, static_cast<const T *>(p.Q), p.q_stride,
                             static_cast<const T *>(p.k_pages), static_cast<const T *>(p.v_pages),
                             static_cast<T *>(p.A), p.lse, p.sq, p.max_new, p.n_q, p.n_kv, p.mask_block, p.scale);
    return launch_kernel(k_paged_attention<T, 4>, grid, dim3(kW * 32), 0, st, 1, static_cast<const T *>(p.Q), p.q_stride,
                         static_cast<const T *>(p.k_pages), static_cast<const T *>(p.v_pages), static_cast<T *>(p.A),
                         p.lse, p.sq, p.max_new, p.n_q, p.n_kv, p.mask_block, p.scale);
}

}  // namespace

cudaError_t paged_attention_f32(const PagedAttn &p, cudaStream_t st) { return launch<float>(p, st); }

}  // namespace dllm
