// paged_append.cu -- new rows enter a paged cache: RMS norm of every query and key head,
// rotary rotation of the head by its position, and the scatter of keys and values into
// their pages, in one pass over the projection's output.
//
//   x' = x rsqrt(mean_j x_j^2 + eps) gamma          (queries and keys, where gamma is given)
//   (y_i, y_{i+h}) = (x'_i c - x'_{i+h} s, x'_{i+h} c + x'_i s),  h = hd / 2,
//                    (c, s) = (cos, sin)(pos inv_freq_i)   (queries and keys, with a table)
//
// Every element is read once and written once with a handful of operations in between, so
// the bytes bound it.  A head is held by hd / 16 lanes, each with 8 consecutive dims of the
// lower half and the 8 they pair with in the upper half: 16-byte accesses, the rotation
// inside a thread, the norm a shuffle over the head's lanes.  The angle is formed in 64
// bits (position times frequency, reduced by 2 pi) because 32 bits lose it: at position
// 10^5 one fp32 rounding of the product is already 4e-3 rad.  It is computed once per row
// and shared by the row's heads through shared memory.
#include "paged.cuh"

namespace dllm {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendUnroll = 3;   // head slices in flight per thread
constexpr int kAppendTok = 8;      // most rows of a CTA

template <class T> struct Vec8;   // 8 consecutive elements as loaded
template <> struct Vec8<bf16> {
    uint4 a;
    __device__ __forceinline__ void load(const bf16 *p) { a = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <> struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = *reinterpret_cast<const float4 *>(p);
        b = *reinterpret_cast<const float4 *>(p + 4);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};

__device__ __forceinline__ void store8(bf16 *p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);   // one rounding per output
        w[i] = *reinterpret_cast<const uint32_t *>(&t);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

struct AppendArgs {
    const void *src[3];       // Q (may be NULL), K, V
    long long stride[3];      // elements between rows
    const void *gamma[2];     // of Q and K, or NULL
    const float *inv_freq;    // [hd/2] or NULL
    void *q_out, *k_pages, *v_pages;
    PagedSeqs sq;
    int T, n_q, n_kv, tok;    // tok: rows of a CTA; n_q = 0 without Q
    float eps;
};

// cos and sin of pos * f with the product and its reduction in 64 bits: what is left is
// the rounding of the reduced angle (|r| <= pi) to 32 bits, 1.2e-7 rad at most.
__device__ __forceinline__ float2 turn(int pos, float f) {
    const double a = (double)pos * (double)f;
    const double k = rint(a * 0.15915494309189535);
    const double r = fma(-k, 2.4492935982947064e-16, fma(-k, 6.283185307179586, a));
    float s, c;
    sincosf((float)r, &s, &c);
    return make_float2(c, s);
}

template <class TI, class TC, int HD>
__global__ void __launch_bounds__(kAppendThreads) k_paged_append(const AppendArgs a, unsigned *status) {
    constexpr int L = HD / 16;       // lanes of a head
    constexpr int H = HD / 2;
    __shared__ float2 cs[kAppendTok][H];
    __shared__ int s_cnt[kAppendTok], s_pos[kAppendTok];
    __shared__ long long s_slot[kAppendTok];   // row of the page pool, or -1
    griddep_wait();
    griddep_launch();
    const int heads = a.n_q + 2 * a.n_kv;
    const int t0 = blockIdx.x * a.tok;
    const int nt = min(a.tok, a.T - t0);
    const int items = nt * heads * L;
    const int tid = threadIdx.x;

    struct Item {
        Vec8<TI> lo, hi;
        int tok, head, l;
    };
    Item it[kAppendUnroll];
    auto fetch = [&](int base) {
#pragma unroll
        for (int u = 0; u < kAppendUnroll; ++u) {
            const int i = base + u * kAppendThreads + tid;
            it[u].tok = -1;
            if (i < items) {
                const int l = i % L, th = i / L;
                const int tk = th / heads, h = th - tk * heads;
                const int w = h < a.n_q ? 0 : (h < a.n_q + a.n_kv ? 1 : 2);
                const int hh = h - (w == 0 ? 0 : (w == 1 ? a.n_q : a.n_q + a.n_kv));
                const TI *p = static_cast<const TI *>(a.src[w]) + (size_t)(t0 + tk) * a.stride[w] +
                              (size_t)hh * HD + l * 8;
                it[u].lo.load(p);
                it[u].hi.load(p + H);
                it[u].tok = tk;
                it[u].head = h;
                it[u].l = l;
            }
        }
    };
    // the rows' data is on its way while the CTA finds out where they belong
    fetch(0);
    if (tid < kAppendTok) s_cnt[tid] = 0;
    __syncthreads();
    for (int i = tid; i < (a.sq.B + 31) / 32 * 32; i += kAppendThreads) {   // sequences that end at or before a row
        const int end = i < a.sq.B ? a.sq.q_start[i + 1] : INT_MAX;
        for (int j = 0; j < nt; ++j) {
            const unsigned m = __ballot_sync(0xffffffffu, end <= t0 + j);
            if ((tid & 31) == 0 && m) atomicAdd(&s_cnt[j], __popc(m));
        }
    }
    __syncthreads();
    if (tid < nt) {
        const int b = s_cnt[tid], t = t0 + tid;
        int pos = -1;
        long long slot = -1;
        if (b < a.sq.B && t >= a.sq.q_start[b]) {
            pos = a.sq.kv_len[b] - (a.sq.q_start[b + 1] - t);
            if (pos >= 0) {
                const int pg = pos >> a.sq.page_log2;
                const int id = pg < a.sq.max_pages ? a.sq.page_table[(size_t)b * a.sq.max_pages + pg] : -1;
                if (id >= 0 && id < a.sq.n_pages)
                    slot = ((long long)id << a.sq.page_log2) + (pos & ((1 << a.sq.page_log2) - 1));
                else
                    raise_status(status, DLLM_STATUS_PAGE);
            }
        }
        s_pos[tid] = pos;
        s_slot[tid] = slot;
    }
    __syncthreads();
    if (a.inv_freq) {
        for (int i = tid; i < nt * H; i += kAppendThreads) {
            const int j = i / H, e = i - j * H;
            cs[j][e] = s_pos[j] >= 0 ? turn(s_pos[j], a.inv_freq[e]) : make_float2(1.f, 0.f);
        }
        __syncthreads();
    }
    // whole warps go through the loop together (the norm's shuffles)
    for (int base = 0; base < items; base += kAppendUnroll * kAppendThreads) {
        if (base > 0) fetch(base);
#pragma unroll
        for (int u = 0; u < kAppendUnroll; ++u) {
            const bool on = it[u].tok >= 0;
            const int tk = on ? it[u].tok : 0, h = on ? it[u].head : 0, l = on ? it[u].l : 0;
            float x[8], y[8];
            if (on) {
                it[u].lo.get(x);
                it[u].hi.get(y);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = y[e] = 0.f;
            }
            const int w = h < a.n_q ? 0 : (h < a.n_q + a.n_kv ? 1 : 2);
            const int hh = h - (w == 0 ? 0 : (w == 1 ? a.n_q : a.n_q + a.n_kv));
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], fmaf(y[e], y[e], ss));
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (!on || s_pos[tk] < 0) continue;
            if (w < 2) {
                const TC *gm = static_cast<const TC *>(a.gamma[w]);
                if (gm) {
                    const float r = rsqrtf(ss * (1.0f / HD) + a.eps);
                    Vec8<TC> g0, g1;
                    float f0[8], f1[8];
                    g0.load(gm + l * 8);
                    g1.load(gm + H + l * 8);
                    g0.get(f0);
                    g1.get(f1);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        x[e] *= r * f0[e];
                        y[e] *= r * f1[e];
                    }
                }
                if (a.inv_freq) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 t = cs[tk][l * 8 + e];
                        const float p = x[e] * t.x - y[e] * t.y;
                        y[e] = y[e] * t.x + x[e] * t.y;
                        x[e] = p;
                    }
                }
            }
            TC *dst;
            if (w == 0) {
                dst = static_cast<TC *>(a.q_out) + ((size_t)(t0 + tk) * a.n_q + hh) * HD;
            } else {
                const long long slot = s_slot[tk];
                if (slot < 0) continue;
                dst = static_cast<TC *>(w == 1 ? a.k_pages : a.v_pages) + ((size_t)slot * a.n_kv + hh) * HD;
            }
            store8(dst + l * 8, x);
            store8(dst + H + l * 8, y);
        }
    }
}

template <class TI, class TC>
cudaError_t launch_append(const AppendArgs &a, int hd, unsigned *status, cudaStream_t st) {
    const dim3 grid((a.T + a.tok - 1) / a.tok);
    if (hd == 64)
        return launch_kernel(k_paged_append<TI, TC, 64>, grid, dim3(kAppendThreads), 0, st, 1, a, status);
    return launch_kernel(k_paged_append<TI, TC, 128>, grid, dim3(kAppendThreads), 0, st, 1, a, status);
}

}  // namespace

cudaError_t paged_append(const void *Q, const void *K, const void *V, long long qs, long long ks, long long vs,
                         const void *gq, const void *gk, float eps, const float *inv_freq, void *q_out,
                         void *k_pages, void *v_pages, const PagedSeqs &sq, int T, int n_q, int n_kv, int hd,
                         int in_dtype, int dtype, unsigned *status, cudaStream_t st) {
    AppendArgs a{};
    a.src[0] = Q;
    a.src[1] = K;
    a.src[2] = V;
    a.stride[0] = qs;
    a.stride[1] = ks;
    a.stride[2] = vs;
    a.gamma[0] = gq;
    a.gamma[1] = gk;
    a.inv_freq = inv_freq;
    a.q_out = q_out;
    a.k_pages = k_pages;
    a.v_pages = v_pages;
    a.sq = sq;
    a.T = T;
    a.n_q = Q ? n_q : 0;
    a.n_kv = n_kv;
    a.eps = eps;
    a.tok = 1;
    if (in_dtype == DLLM_BF16) return launch_append<bf16, bf16>(a, hd, status, st);
    if (dtype == DLLM_BF16) return launch_append<float, bf16>(a, hd, status, st);
    return launch_append<float, float>(a, hd, status, st);
}

}  // namespace dllm
