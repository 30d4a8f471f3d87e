// paged_append_f8.cu -- new rows enter 8-bit pages: RMS norm and rotary rotation of the query and key
// heads as in paged_append.cu, then keys and values as E4M3 codes under one power of two for each
// page and head.
//
//   a   = max |x| over the page's new rows;   e = the least exponent with a <= 448 2^e  (-64 .. 63)
//   2^e = the page's scale, or the larger of it and the scale before where earlier rows stay in the page
//   code(x) = E4M3(x 2^-e)       earlier rows whose scale grew: E4M3(value 2^-e), a shift of the exponent
//
// A power of two costs a floating format nothing but range at the lower end, makes growth exact for all
// codes that stay normal, and leaves the reader's products exact.
//
// A CTA has the rows that enter one page (a segment) and a share of the heads; each of its warps takes
// a head at a time.  A head's rows are read twice, for the maximum and for the codes (the second time from
// L1 or L2), so the unit needs no registers for a page of rows and no barrier.  The rotation's angles
// are formed once per segment, in 64 bits, for all heads.  The bytes bound it.
#include <climits>

#include "e4m3.cuh"
#include "paged_rows.cuh"

namespace dllm {
namespace {

constexpr int kF8Threads = 256;
constexpr int kF8Warps = kF8Threads / 32;

__device__ __forceinline__ uint2 codes8(const float (&v)[8], float f) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e4m3x2(v[2 * i] * f, v[2 * i + 1] * f);
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// Angles as 64-bit fractions of a turn: one division by 2 pi in 64 bits for a frequency (2^-54 of a turn for each position
// at most), an integer product that wraps as the angle does for a position (the 64-bit floating pipe has two operations a
// clock and SM), and what is handed to the sine is off by one rounding of |angle| <= pi, 1.9e-7 rad.
__device__ __forceinline__ uint64_t turn_step(float f) {
    const double q = (double)f * 0.15915494309189535;
    return (uint64_t)((q - floor(q)) * 18446744073709551616.0);
}
__device__ __forceinline__ float2 turn_at(uint64_t turns) {
    float s, c;
    sincospif((float)(int)(turns >> 32) * 4.656612873077393e-10f, &s, &c);   // (2^-31: half turns)
    return make_float2(c, s);
}

struct Piece {          // rows of one sequence that enter one page
    int b, id;          // id: the page, or -1
    int row, n;         // first row of the batch, number of rows
    int pos;            // position of the first
};

// Segment `index` of the batch, by the whole CTA: sequences in order, their pages in order.
__device__ __forceinline__ Piece find_piece(const PagedSeqs &sq, int T, int index, unsigned *status, bool report) {
    __shared__ long long part[kF8Warps];
    __shared__ Piece found;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = (sq.B + kF8Threads - 1) / kF8Threads;
    // rows [lo, hi) of sequence b inside the batch and from position 0 on -> pages that they touch
    auto span = [&](int b, int &start, long long &pos0, int &lo, int &hi) -> long long {
        int n_new;
        hi = sq.rows(b, T, INT_MAX, start, n_new);
        if (hi <= 0) return 0;
        pos0 = (long long)sq.kv_len[b] - n_new;
        lo = pos0 < 0 ? (-pos0 < hi ? (int)-pos0 : hi) : 0;
        if (lo >= hi) return 0;
        return ((pos0 + hi - 1) >> sq.page_log2) - ((pos0 + lo) >> sq.page_log2) + 1;
    };
    if (tid == 0) found.n = 0;
    long long mine = 0;
    for (int j = 0; j < per; ++j) {
        const int b = tid * per + j;
        int start, lo, hi;
        long long pos0;
        if (b < sq.B) mine += span(b, start, pos0, lo, hi);
    }
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) part[warp] = x;
    __syncthreads();
    long long at = x - mine;
    for (int w = 0; w < warp; ++w) at += part[w];
    if (index >= at && index < at + mine) {
        for (int j = 0; j < per; ++j) {
            const int b = tid * per + j;
            int start = 0, lo = 0, hi = 0;
            long long pos0 = 0;
            const long long cnt = b < sq.B ? span(b, start, pos0, lo, hi) : 0;
            if (index >= at && index < at + cnt) {
                const long long page = ((pos0 + lo) >> sq.page_log2) + (index - at);
                const long long first = max(pos0 + lo, page << sq.page_log2);
                const long long last = min(pos0 + hi, (page + 1) << sq.page_log2);
                int id = page < sq.max_pages ? sq.page_table[(size_t)b * sq.max_pages + page] : -1;
                if ((unsigned)id >= (unsigned)sq.n_pages) id = -1;
                if (id < 0 && report) raise_status(status, DLLM_STATUS_PAGE);
                found = Piece{b, id, start + (int)(first - pos0), (int)(last - first), (int)first};
            }
            at += cnt;
        }
    }
    __syncthreads();
    return found;
}

template <class TI, int HD>
__global__ void __launch_bounds__(kF8Threads) k_paged_append_f8(const AppendF8 a, unsigned *status) {
    constexpr int L = HD / 16;       // lanes of a head's row: 8 dims of each half
    constexpr int H = HD / 2;
    constexpr int PER = 32 / L;      // rows of a warp at a time
    extern __shared__ __align__(16) float2 cs[];   // [rows][H], a lane's 8 in pairs L pairs apart (no bank conflicts)
    __shared__ uint64_t step[H];
    griddep_wait();
    griddep_launch();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Piece p = find_piece(a.sq, a.T, blockIdx.x, status, blockIdx.y == 0);
    if (p.n <= 0) return;
    if (a.inv_freq) {
        if (tid < H) step[tid] = turn_step(a.inv_freq[tid]);
        __syncthreads();
        const long long base = (long long)p.pos + (a.pos_base ? a.pos_base[p.b] : 0);
        for (int i = tid; i < p.n * H; i += kF8Threads) {
            const int r = i / H, e = i % H;
            cs[r * H + ((e & 7) >> 1) * (2 * L) + (e >> 3) * 2 + (e & 1)] = turn_at((uint64_t)(base + r) * step[e]);
        }
        __syncthreads();
    }
    const int l = lane % L, rr = lane / L;
    const int heads = a.n_q + 2 * a.n_kv, off0 = p.pos & ((1 << a.sq.page_log2) - 1);
    for (int u = blockIdx.y * kF8Warps + warp; u < heads; u += gridDim.y * kF8Warps) {
        // keys and values first: they take longest
        const int w = u < a.n_kv ? 1 : (u < 2 * a.n_kv ? 2 : 0);
        const int h = w == 1 ? u : (w == 2 ? u - a.n_kv : u - 2 * a.n_kv);
        if (w > 0 && p.id < 0) continue;
        const TI *src = static_cast<const TI *>(a.src[w]) + (size_t)p.row * a.stride[w] + (size_t)h * HD + l * 8;
        const bf16 *gm = w < 2 ? a.gamma[w] : nullptr;
        float g0[8], g1[8];
        if (gm) {
            Vec8<bf16> v0, v1;
            v0.load(gm + l * 8);
            v1.load(gm + H + l * 8);
            v0.get(g0);
            v1.get(g1);
        }
        auto value = [&](int r, float (&x)[8], float (&y)[8]) {   // row r of the segment (whole warps), normed and turned
            Vec8<TI> lo{}, hi{};
            if (r < p.n) {
                lo.load(src + (size_t)r * a.stride[w]);
                hi.load(src + (size_t)r * a.stride[w] + H);
            }
            lo.get(x);
            hi.get(y);
            if (gm) {
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], fmaf(y[e], y[e], ss));
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float f = rsqrtf(ss * (1.0f / HD) + a.eps);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] *= f * g0[e];
                    y[e] *= f * g1[e];
                }
            }
            if (w < 2 && a.inv_freq && r < p.n) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float4 c = *reinterpret_cast<const float4 *>(cs + r * H + e * L + l * 2);
                    const float t = x[e] * c.x - y[e] * c.y, u = x[e + 1] * c.z - y[e + 1] * c.w;
                    y[e] = y[e] * c.x + x[e] * c.y;
                    y[e + 1] = y[e + 1] * c.z + x[e + 1] * c.w;
                    x[e] = t;
                    x[e + 1] = u;
                }
            }
        };
        if (w == 0) {
            for (int r0 = 0; r0 < p.n; r0 += PER) {
                float x[8], y[8];
                value(r0 + rr, x, y);
                if (r0 + rr < p.n) {
                    bf16 *dst = a.q_out + ((size_t)(p.row + r0 + rr) * a.n_q + h) * HD + l * 8;
                    store8(dst, x);
                    store8(dst + H, y);
                }
            }
            continue;
        }
        float top = 0.f;
#pragma unroll 2
        for (int r0 = 0; r0 < p.n; r0 += PER) {
            float x[8], y[8];
            value(r0 + rr, x, y);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fmaxf(fabsf(x[e]), fabsf(y[e])));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        uint8_t *sp = a.scale[w - 1] + (size_t)p.id * a.n_kv + h;
        uint8_t *page = a.pages[w - 1] + (((size_t)p.id << a.sq.page_log2) * a.n_kv + h) * HD;
        const size_t row_bytes = (size_t)a.n_kv * HD;
        int now = e8m0_for(top);
        if (off0 > 0) {              // earlier rows stay in the page
            const int old = *sp;
            if (old < now) {
                const float f = __uint_as_float((uint32_t)max(old - now + 127, 0) << 23);   // 2^(old - now); 0 from 2^-127 on
                for (int i = lane; i < off0 * (HD / 4); i += 32) {
                    uint32_t *c = reinterpret_cast<uint32_t *>(page + (size_t)(i / (HD / 4)) * row_bytes) + i % (HD / 4);
                    const float2 x = f32_of_e4m3x2(*c & 0xffffu), y = f32_of_e4m3x2(*c >> 16);
                    *c = e4m3x2(x.x * f, x.y * f) | e4m3x2(y.x * f, y.y * f) << 16;
                }
            }
            now = max(now, old);
        }
        __syncwarp();                // (the old scale has been read by every lane)
        if (lane == 0) *sp = (uint8_t)now;
        const float f = e8m0_inverse(now);
        uint8_t *dst = page + (size_t)off0 * row_bytes + l * 8;
#pragma unroll 2
        for (int r0 = 0; r0 < p.n; r0 += PER) {
            float x[8], y[8];
            value(r0 + rr, x, y);
            if (r0 + rr < p.n) {
                *reinterpret_cast<uint2 *>(dst + (size_t)(r0 + rr) * row_bytes) = codes8(x, f);
                *reinterpret_cast<uint2 *>(dst + (size_t)(r0 + rr) * row_bytes + H) = codes8(y, f);
            }
        }
    }
}

template <class TI, int HD>
cudaError_t launch_append_f8(const AppendF8 &a, unsigned *status, cudaStream_t st) {
    const int page = 1 << a.sq.page_log2;
    // segments: a sequence's rows touch at most two pages more than they fill, and a page each
    const long long most = (long long)a.T / page + 2LL * a.sq.B;
    const int segs = (int)(most < a.T ? most : a.T);
    const int heads = a.n_q + 2 * a.n_kv, full = (heads + kF8Warps - 1) / kF8Warps;
    // CTAs of a segment: one per 8 heads while that does not fill the GPU several times over
    int split = full;
    while (split > 1 && (long long)segs * split > 8LL * num_sms()) split = (split + 1) / 2;
    const size_t smem = a.inv_freq ? (size_t)(page < a.T ? page : a.T) * (HD / 2) * sizeof(float2) : 0;
    static size_t allowed[64] = {};   // per device: the shared-memory limit as raised so far
    int dev = 0;
    cudaGetDevice(&dev);
    if (smem > 48 * 1024 && (dev < 0 || dev >= 64 || allowed[dev] < 128 * 1024)) {
        const cudaError_t e = cudaFuncSetAttribute(k_paged_append_f8<TI, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 1024);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) allowed[dev] = 128 * 1024;
    }
    return launch_kernel(k_paged_append_f8<TI, HD>, dim3(segs, split), dim3(kF8Threads), smem, st, 1, a, status);
}

}  // namespace

cudaError_t paged_append_f8(const AppendF8 &a, int hd, int in_dtype, unsigned *status, cudaStream_t st) {
    if (in_dtype == DLLM_BF16)
        return hd == 64 ? launch_append_f8<bf16, 64>(a, status, st) : launch_append_f8<bf16, 128>(a, status, st);
    return hd == 64 ? launch_append_f8<float, 64>(a, status, st) : launch_append_f8<float, 128>(a, status, st);
}

}  // namespace dllm
