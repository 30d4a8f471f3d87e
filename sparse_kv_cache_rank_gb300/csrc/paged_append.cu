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
// and shared by the row's heads; a warp keeps its lanes' angles in registers over all heads it
// takes, with the loads of the next turn under way.
//
// 7374 ragged rows of 64 heads of 128 dims, normed, bf16: 67 us, 5.3 TB/s (85 us with
// the angles read again for every head).  A block of 32 rows or 64 single ones takes about 11 us of which
// the launch's own cost on the host is most.
#include "paged.cuh"

namespace dllm {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendWarps = kAppendThreads / 32;   // most rows of a CTA

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
    int T, n_q, n_kv, wpt;    // wpt: warps of a row (a divisor of kAppendWarps); n_q = 0 without Q
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
    constexpr int PER = 32 / L;      // heads of a warp at a time
    __shared__ float2 cs[kAppendWarps][H];
    __shared__ int s_cnt[kAppendWarps], s_pos[kAppendWarps];
    __shared__ long long s_slot[kAppendWarps];   // row of the page pool, or -1
    __shared__ __align__(16) TC gain[2][HD];
    griddep_wait();
    griddep_launch();
    const int heads = a.n_q + 2 * a.n_kv;
    const int rows = kAppendWarps / a.wpt;       // of a CTA
    const int t0 = blockIdx.x * rows;
    const int nt = min(rows, a.T - t0);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tk = warp / a.wpt, l = lane % L;
    const bool on = tk < nt;
    const size_t t = (size_t)(t0 + (on ? tk : 0));
    const int h0 = (warp - tk * a.wpt) * PER + lane / L, step = a.wpt * PER;   // this lane's heads

    struct Item {
        Vec8<TI> lo, hi;
    };
    auto fetch = [&](Item &x, int h) {
        if (on && h < heads) {
            const TI *p = h < a.n_q             ? static_cast<const TI *>(a.src[0]) + t * a.stride[0] + (size_t)h * HD
                          : h < a.n_q + a.n_kv ? static_cast<const TI *>(a.src[1]) + t * a.stride[1] + (size_t)(h - a.n_q) * HD
                                                : static_cast<const TI *>(a.src[2]) + t * a.stride[2] +
                                                      (size_t)(h - a.n_q - a.n_kv) * HD;
            x.lo.load(p + l * 8);
            x.hi.load(p + H + l * 8);
        }
    };
    // the first heads are on their way while the CTA finds out where its rows belong
    Item cur;
    fetch(cur, h0);
    if (tid < kAppendWarps) s_cnt[tid] = 0;
    for (int i = tid; i < 2 * HD; i += kAppendThreads)
        if (const TC *g = static_cast<const TC *>(a.gamma[i / HD])) gain[i / HD][i % HD] = g[i % HD];
    __syncthreads();
    for (int i = tid; i < (a.sq.B + 31) / 32 * 32; i += kAppendThreads) {   // sequences that end at or before a row
        const int end = i < a.sq.B ? a.sq.q_start[i + 1] : INT_MAX;
        for (int j = 0; j < nt; ++j) {
            const unsigned m = __ballot_sync(0xffffffffu, end <= t0 + j);
            if (lane == 0 && m) atomicAdd(&s_cnt[j], __popc(m));
        }
    }
    __syncthreads();
    if (tid < nt) {
        const int b = s_cnt[tid], row = t0 + tid;
        int pos = -1;
        long long slot = -1;
        if (b < a.sq.B && row >= a.sq.q_start[b]) {
            pos = a.sq.kv_len[b] - (a.sq.q_start[b + 1] - row);
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
    if (a.inv_freq)
        for (int i = tid; i < nt * H; i += kAppendThreads) {
            const int j = i / H, e = i - j * H;
            cs[j][e] = s_pos[j] >= 0 ? turn(s_pos[j], a.inv_freq[e]) : make_float2(1.f, 0.f);
        }
    __syncthreads();
    if (!on || s_pos[tk] < 0) return;            // (whole warps)
    const long long slot = s_slot[tk];
    // the row's angles and the gains of this lane's dims serve all its heads
    float2 c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = a.inv_freq ? cs[tk][l * 8 + e] : make_float2(1.f, 0.f);
    for (int hw = h0 - lane / L; hw < heads; hw += step) {   // whole warps (the norm's shuffles)
        const int h = hw + lane / L;
        Item ahead;
        fetch(ahead, h + step);
        float x[8], y[8];
        cur.lo.get(x);
        cur.hi.get(y);
        const int w = h < a.n_q ? 0 : (h < a.n_q + a.n_kv ? 1 : 2);
        const void *gm = w < 2 ? a.gamma[w] : nullptr;
        if (a.gamma[0] || a.gamma[1]) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], fmaf(y[e], y[e], ss));
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (gm) {
                const float r = rsqrtf(ss * (1.0f / HD) + a.eps);
                float f0[8], f1[8];
                Vec8<TC> g0, g1;
                g0.load(gain[w] + l * 8);
                g1.load(gain[w] + H + l * 8);
                g0.get(f0);
                g1.get(f1);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] *= r * f0[e];
                    y[e] *= r * f1[e];
                }
            }
        }
        if (w < 2 && a.inv_freq) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float p = x[e] * c[e].x - y[e] * c[e].y;
                y[e] = y[e] * c[e].x + x[e] * c[e].y;
                x[e] = p;
            }
        }
        if (h < heads && (w == 0 || slot >= 0)) {
            TC *dst = w == 0 ? static_cast<TC *>(a.q_out) + (t * a.n_q + h) * HD
                      : w == 1 ? static_cast<TC *>(a.k_pages) + ((size_t)slot * a.n_kv + (h - a.n_q)) * HD
                               : static_cast<TC *>(a.v_pages) + ((size_t)slot * a.n_kv + (h - a.n_q - a.n_kv)) * HD;
            store8(dst + l * 8, x);
            store8(dst + H + l * 8, y);
        }
        cur = ahead;
    }
}

template <class TI, class TC>
cudaError_t launch_append(const AppendArgs &a, int hd, unsigned *status, cudaStream_t st) {
    const int rows = kAppendWarps / a.wpt;
    const dim3 grid((a.T + rows - 1) / rows);
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
    // Warps of a row: as many as its heads occupy while that still leaves CTAs to spare for the GPU
    // (a short call's rows end sooner), one or two for long ones (the row's setup is shared): 7374 rows of 96
    // heads take 91, 76, 71, 69 us with 8, 4, 2, 1 warps a row.
    const int per = 512 / hd, turns = (a.n_q + 2 * n_kv + per - 1) / per;   // a warp's turns for a whole row
    a.wpt = kAppendWarps;
    while (a.wpt > 1 && (a.wpt / 2 >= turns || (long long)T * a.wpt > kAppendWarps * 8LL * num_sms())) a.wpt /= 2;
    if (in_dtype == DLLM_BF16) return launch_append<bf16, bf16>(a, hd, status, st);
    if (dtype == DLLM_BF16) return launch_append<float, bf16>(a, hd, status, st);
    return launch_append<float, float>(a, hd, status, st);
}

}  // namespace dllm
