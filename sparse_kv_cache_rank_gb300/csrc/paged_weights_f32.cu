// paged_weights_f32.cu -- the attention weight that every key of an fp32 paged cache receives, on the CUDA cores:
//
//   score[b, g, j] <- (old score, or 0 for the new rows' own keys)
//                     + sum over rows t of b and heads h of g that see j of exp(scale <Q[t, h], K_j> - lse[t, h])
//
// Four lanes share four keys, a quarter of the dims each, in registers; 32 rows of queries at a time stand in shared
// memory.  A load of four dims serves four keys that way (a load hands out 128 bytes a clock, broadcast or not: with a key
// a thread, and a load for four FMAs, that took 14 of 21 us), and three shuffles a row leave each lane one key's sum.
// Sums are in the order of the rows, the same every time.
#include <climits>

#include "paged_tc.cuh"

namespace dllm {
namespace {

constexpr int kKeys = 128;       // keys of an item, threads of a CTA
constexpr int kRows = 32;        // rows in shared memory

struct WeightArgs32 {
    PagedWeights p;
    int G;
};

template <int HD> __global__ void __launch_bounds__(kKeys) k_paged_weights_f32(const WeightArgs32 a) {
    __shared__ __align__(16) float sq[kRows][HD];
    __shared__ float slse[kRows];
    __shared__ int slim[kRows];
    __shared__ long long pre[kPagedMaxSeqs + 1];
    const PagedWeights &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, B = p.sq.B;
    griddep_wait();
    griddep_launch();
    auto tiles_of = [&](int b, int &start, int &n, int &n_new) -> int {
        n = p.sq.rows(b, p.T, p.max_new, start, n_new);
        if (n <= 0) return 0;
        return (int)(((long long)min(p.sq.keys(b), p.slots) + kKeys - 1) / kKeys);
    };
    for (int b = tid; b < B; b += kKeys) {
        int start, n, n_new;
        pre[b + 1] = (long long)tiles_of(b, start, n, n_new) * p.n_kv;
    }
    __syncthreads();
    if (tid < 32) {
        long long run = 0;
        for (int b0 = 0; b0 < B; b0 += 32) {
            long long x = b0 + lane < B ? pre[b0 + lane + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (b0 + lane < B) pre[b0 + lane + 1] = run + x;
            run += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) pre[0] = 0;
    }
    __syncthreads();
    int b = 0;
    for (long long at = blockIdx.x; at < pre[B]; at += gridDim.x) {
        while (at >= pre[b + 1]) ++b;
        int start, n, n_new;
        const int tiles = tiles_of(b, start, n, n_new);
        const long long off = at - pre[b];
        const int g = (int)(off / tiles), k0 = (int)(off - (long long)g * tiles) * kKeys, key = k0 + tid;
        const int len = min(p.sq.keys(b), p.slots), pos0 = p.sq.kv_len[b] - n_new;
        int id = -1;
        if (key < len) id = p.sq.page_table[(size_t)b * p.sq.max_pages + (key >> p.sq.page_log2)];
        const bool here = (unsigned)id < (unsigned)p.sq.n_pages;
        const size_t at_slot = ((size_t)b * p.n_kv + g) * p.slots + key;
        const float old = key < len && key < pos0 ? p.score[at_slot] : 0.f;   // (early: with the keys)
        float4 k[4][HD / 16];        // dims 16 e + 4 c .. of the four lanes' keys
        const int c = lane & 3;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at_key = (key & ~3) + i, at_id = __shfl_sync(0xffffffffu, id, (lane & ~3) + i);
            const bool there = (unsigned)at_id < (unsigned)p.sq.n_pages;
            const float4 *src = static_cast<const float4 *>(p.k_pages) +
                                ((((size_t)(there ? at_id : 0) << p.sq.page_log2) + (at_key & ((1 << p.sq.page_log2) - 1))) * p.n_kv + g) * (HD / 4);
#pragma unroll
            for (int e = 0; e < HD / 16; ++e) k[i][e] = there ? src[4 * e + c] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        // the first token whose row sees key k0
        const int m = p.mask_block;
        const long long first = m == 0 ? 0 : (long long)(k0 / m) * m - pos0;
        const int rows = n * a.G;
        float sum = 0.f;
        for (long long r0 = first > 0 ? first * a.G : 0; r0 < rows; r0 += kRows) {
            __syncthreads();
            for (int i = tid; i < kRows * (HD / 4); i += kKeys) {
                const int j = i / (HD / 4), e = i - j * (HD / 4), row = (int)r0 + j, tok = row / a.G;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (row < rows)
                    v = reinterpret_cast<const float4 *>(static_cast<const float *>(p.Q) + (size_t)(start + tok) * p.q_stride +
                                                         (size_t)(g * a.G + row - tok * a.G) * HD)[e];
                reinterpret_cast<float4 *>(sq[j])[e] = v;
            }
            if (tid < kRows) {
                const int row = (int)r0 + tid, tok = row / a.G;
                float l = 0.f;
                int lim = 0;                 // no row, or one without keys, or without a number
                if (row < rows) {
                    const float v = p.lse[(size_t)(start + tok) * p.n_q + g * a.G + row - tok * a.G];
                    if (isfinite(v)) {
                        l = v;
                        lim = PagedSeqs::visible(pos0 + tok, len, m);
                    }
                }
                slse[tid] = l;
                slim[tid] = lim;
            }
            __syncthreads();
#pragma unroll 2
            for (int j = 0; j < kRows; ++j) {
                float2 d[4] = {};
#pragma unroll
                for (int e = 0; e < HD / 16; ++e) {
                    const float4 v = reinterpret_cast<const float4 *>(sq[j])[4 * e + c];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        d[i] = fma2(make_float2(v.x, v.y), make_float2(k[i][e].x, k[i][e].y), d[i]);
                        d[i] = fma2(make_float2(v.z, v.w), make_float2(k[i][e].z, k[i][e].w), d[i]);
                    }
                }
                // the four lanes' shares: two keys to each half of them, then one to each
                const bool up = c & 2, odd = c & 1;
                float x = d[0].x + d[0].y, y = d[1].x + d[1].y, z = d[2].x + d[2].y, w = d[3].x + d[3].y;
                const float x1 = __shfl_xor_sync(0xffffffffu, up ? x : z, 2), y1 = __shfl_xor_sync(0xffffffffu, up ? y : w, 2);
                x = (up ? z : x) + x1;
                y = (up ? w : y) + y1;
                const float s = (odd ? y : x) + __shfl_xor_sync(0xffffffffu, odd ? x : y, 1);
                if (here && key < slim[j]) sum += expf(s * p.scale - slse[j]);
            }
        }
        if (key < len) {
            p.score_out[at_slot] = old + sum;
            if (key >= pos0 && p.slot_pos) p.slot_pos[at_slot] = key + (p.pos_base ? p.pos_base[b] : 0);
        }
    }
}

}  // namespace

cudaError_t paged_weights_f32(const PagedWeights &p, cudaStream_t st) {
    const WeightArgs32 a{p, p.n_q / p.n_kv};
    const dim3 grid(4 * num_sms());
    if (p.hd == 64) return launch_kernel(k_paged_weights_f32<64>, grid, dim3(kKeys), 0, st, 1, a);
    return launch_kernel(k_paged_weights_f32<128>, grid, dim3(kKeys), 0, st, 1, a);
}

}  // namespace dllm
