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
// A CTA has the rows that enter one page (a segment) and a share of the heads; a group of its warps takes a head at a
// time, up to four 32-lane loads of rows a warp, which stay in registers between the maximum and the codes.  The rotation's
// angles are formed once per segment for all its heads, those in the first rows' way.
//
// 7374 ragged rows of 96 heads of 128 dims (bf16, normed, pages of 64): 82 us, 3.6 TB/s.  It was 146 us with the angles
// in 64-bit floating point and their lanes' reads in each other's banks, 98 us without those two, 90 us with the rows read
// once (registers for them leave two CTAs an SM), 84 us with packed arithmetic; what is left is the chain from the sequence
// tables to the first rows, once for each of 1476 CTAs, and two passes of norm and rotation for the keys.
#include <climits>

#include "e4m3.cuh"
#include "paged_rows.cuh"
#include "paged_tc.cuh"

namespace dllm {
namespace {

constexpr int kF8Threads = 256;
constexpr int kF8Warps = kF8Threads / 32;

__device__ __forceinline__ uint2 codes8(const float2 (&v)[4], float f) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = mul2(v[i], make_float2(f, f));
        c[i] = e4m3x2(t.x, t.y);
    }
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}
template <class T> __device__ __forceinline__ void pairs(const Vec8<T> &v, float2 (&x)[4]) {
    float t[8];
    v.get(t);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_float2(t[2 * i], t[2 * i + 1]);
}
__device__ __forceinline__ void store8(bf16 *p, const float2 (&v)[4], uint32_t flip) {   // (flip: sign bits turned over)
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(v[i].x, v[i].y);   // one rounding per output
        w[i] = *reinterpret_cast<const uint32_t *>(&t) ^ flip;
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
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

// gw: warps of a group, a power of two; share: heads of a CTA.
template <class TI, int HD>
__global__ void __launch_bounds__(kF8Threads, 2) k_paged_append_f8(const AppendF8 a, int gw, int share, unsigned *status) {
    constexpr int L = HD / 16;       // lanes of a head's row: 8 dims of each half
    constexpr int H = HD / 2;
    constexpr int PER = 32 / L;      // rows of a warp at a time
    extern __shared__ __align__(16) float cs[];    // [rows][2 H]: a lane's 8 dims as 4 times 2 cosines and 2 sines, L fours apart
                                                   // (no bank conflicts)
    __shared__ uint64_t steps[H];
    __shared__ float tops[2][kF8Warps];
    griddep_wait();
    griddep_launch();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (a.inv_freq && tid < H) steps[tid] = turn_step(a.inv_freq[tid]);   // (find_piece has barriers)
    const Piece p = find_piece(a.sq, a.T, blockIdx.x, status, blockIdx.y == 0);
    if (p.n <= 0) return;
    const int heads = a.n_q + 2 * a.n_kv, off0 = p.pos & ((1 << a.sq.page_log2) - 1);
    const int u0 = blockIdx.y * share, u1 = min(u0 + share, heads);   // this CTA's heads: of keys, queries, values
    const int l = lane % L, wi = warp & (gw - 1), group = warp / gw, groups = kF8Warps / gw;
    const int rr = wi * PER + lane / L, turn = gw * PER;   // this lane's first row, rows of the group at a time
    // head u's rows: the first ones are on their way while the angles are formed
    auto place = [&](int u, int &w, int &h) -> const TI * {
        w = u < a.n_kv ? 1 : (u < a.n_kv + a.n_q ? 0 : 2);
        h = w == 1 ? u : (w == 0 ? u - a.n_kv : u - a.n_kv - a.n_q);
        return static_cast<const TI *>(a.src[w]) + (size_t)p.row * a.stride[w] + (size_t)h * HD + l * 8;
    };
    auto load = [&](const TI *src, long long stride, int r, Vec8<TI> &x, Vec8<TI> &y) {
        if (r < p.n) {
            x.load(src + (size_t)r * stride);
            y.load(src + (size_t)r * stride + H);
        } else {
            x = Vec8<TI>{};
            y = Vec8<TI>{};
        }
    };
    Vec8<TI> lo[4], hi[4];
    auto fetch = [&](int u) {
        if (u >= u1) return;
        int w, h;
        const TI *src = place(u, w, h);
        if (w > 0 && p.id < 0) return;
#pragma unroll
        for (int k = 0; k < 4; ++k) load(src, a.stride[w], rr + k * turn, lo[k], hi[k]);
    };
    fetch(u0 + group);
    if (a.inv_freq && u0 < a.n_kv + a.n_q) {
        const long long base = (long long)p.pos + (a.pos_base ? a.pos_base[p.b] : 0);
        for (int i = tid; i < p.n * H; i += kF8Threads) {
            const int r = i / H, e = i % H;
            const float2 c = turn_at((uint64_t)(base + r) * steps[e]);
            float *at = cs + r * HD + ((e & 7) >> 1) * (4 * L) + (e >> 3) * 4 + (e & 1);
            at[0] = c.x;
            at[2] = c.y;
        }
        __syncthreads();
    }
    int flip = 0;
    for (int u = u0 + group; u < u1; u += groups) {
        if (u != u0 + group) fetch(u);
        int w, h;
        const TI *src = place(u, w, h);
        if (w > 0 && p.id < 0) continue;
        uint8_t *sp = w > 0 ? a.scale[w - 1] + (size_t)p.id * a.n_kv + h : nullptr;
        const int old = w > 0 && off0 > 0 ? *sp : 0;   // (earlier rows stay in the page)
        const bf16 *gm = w < 2 ? a.gamma[w] : nullptr;
        const bool turns = w < 2 && a.inv_freq;
        Vec8<bf16> v0{}, v1{};
        if (gm) {
            v0.load(gm + l * 8);
            v1.load(gm + H + l * 8);
        }
        // Normed and turned (whole warps); where they turn, the lower half comes out with the other sign: (y s - x c, y c + x s)
        // needs no sign turned on the way.
        auto value = [&](int r, const Vec8<TI> &vx, const Vec8<TI> &vy, float2 (&x)[4], float2 (&y)[4]) {
            pairs(vx, x);
            pairs(vy, y);
            if (gm) {
                float2 s2 = make_float2(0.f, 0.f), g0[4], g1[4];
                pairs(v0, g0);
                pairs(v1, g1);
#pragma unroll
                for (int e = 0; e < 4; ++e) s2 = fma2(x[e], x[e], fma2(y[e], y[e], s2));
                float ss = s2.x + s2.y;
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float f = rsqrtf(ss * (1.0f / HD) + a.eps);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = mul2(x[e], mul2(g0[e], make_float2(f, f)));
                    y[e] = mul2(y[e], mul2(g1[e], make_float2(f, f)));
                }
            }
            if (turns && r < p.n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 c = *reinterpret_cast<const float4 *>(cs + r * HD + e * (4 * L) + l * 4);
                    const float2 co = make_float2(c.x, c.y), si = make_float2(c.z, c.w);
                    const float2 xs = mul2(x[e], si), xc = mul2(x[e], co);
                    x[e] = fma2(y[e], si, make_float2(-xc.x, -xc.y));
                    y[e] = fma2(y[e], co, xs);
                }
            }
        };
        // rows past the fourth load of a warp (pages of more than 4 turns) are read again
        auto rows = [&](auto &&each) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k * turn >= p.n) return;
                float2 x[4], y[4];
                value(rr + k * turn, lo[k], hi[k], x, y);
                if (rr + k * turn < p.n) each(rr + k * turn, x, y);
            }
#pragma unroll 1
            for (int r0 = 4 * turn; r0 < p.n; r0 += turn) {
                Vec8<TI> vx, vy;
                float2 x[4], y[4];
                load(src, a.stride[w], rr + r0, vx, vy);
                value(rr + r0, vx, vy, x, y);
                if (rr + r0 < p.n) each(rr + r0, x, y);
            }
        };
        if (w == 0) {
            rows([&](int r, const float2 (&x)[4], const float2 (&y)[4]) {
                bf16 *dst = a.q_out + ((size_t)(p.row + r) * a.n_q + h) * HD + l * 8;
                store8(dst, x, turns ? 0x80008000u : 0u);
                store8(dst + H, y, 0u);
            });
            continue;
        }
        float top = 0.f;
        rows([&](int, const float2 (&x)[4], const float2 (&y)[4]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                top = fmaxf(top, fmaxf(fabsf(x[e].x), fabsf(x[e].y)));
                top = fmaxf(top, fmaxf(fabsf(y[e].x), fabsf(y[e].y)));
            }
        });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (gw > 1) {                // (the places of a head are written again two heads on, with a barrier between)
            if (lane == 0) tops[flip][warp] = top;
            __syncwarp();
            named_bar_sync(1 + group, gw * 32);
            for (int i = 0; i < gw; ++i) top = fmaxf(top, tops[flip][group * gw + i]);
            flip ^= 1;
        }
        uint8_t *page = a.pages[w - 1] + (((size_t)p.id << a.sq.page_log2) * a.n_kv + h) * HD;
        const size_t row_bytes = (size_t)a.n_kv * HD;
        int now = e8m0_for(top);
        if (off0 > 0) {
            if (old < now) {
                const float f = __uint_as_float((uint32_t)max(old - now + 127, 0) << 23);   // 2^(old - now); 0 from 2^-127 on
                for (int i = wi * 32 + lane; i < off0 * (HD / 4); i += gw * 32) {
                    uint32_t *c = reinterpret_cast<uint32_t *>(page + (size_t)(i / (HD / 4)) * row_bytes) + i % (HD / 4);
                    const float2 x = f32_of_e4m3x2(*c & 0xffffu), y = f32_of_e4m3x2(*c >> 16);
                    *c = e4m3x2(x.x * f, x.y * f) | e4m3x2(y.x * f, y.y * f) << 16;
                }
            }
            now = max(now, old);
        }
        __syncwarp();                // (the old scale has been read by every lane, before the barrier by every warp)
        if (lane == 0 && wi == 0) *sp = (uint8_t)now;
        const float f = e8m0_inverse(now);
        uint8_t *dst = page + (size_t)off0 * row_bytes + l * 8;
        rows([&](int r, const float2 (&x)[4], const float2 (&y)[4]) {
            *reinterpret_cast<uint2 *>(dst + (size_t)r * row_bytes) = codes8(x, turns ? -f : f);
            *reinterpret_cast<uint2 *>(dst + (size_t)r * row_bytes + H) = codes8(y, f);
        });
    }
}

template <class TI, int HD>
cudaError_t launch_append_f8(const AppendF8 &a, unsigned *status, cudaStream_t st) {
    const int page = 1 << a.sq.page_log2;
    // segments: a sequence's rows touch at most two pages more than they fill, and a page each
    const long long most = (long long)a.T / page + 2LL * a.sq.B;
    const int segs = (int)(most < a.T ? most : a.T);
    // warps of a head: a page's rows in four loads
    const int most_rows = page < a.T ? page : a.T;
    int gw = 1;
    while (gw < kF8Warps && most_rows > gw * 4 * (512 / HD)) gw *= 2;
    const int heads = a.n_q + 2 * a.n_kv, groups = kF8Warps / gw, full = (heads + groups - 1) / groups;
    // CTAs of a segment: a group of warps per head while that does not fill the GPU several times over
    int split = full;
    while (split > 1 && (long long)segs * split > 16LL * num_sms()) split = (split + 1) / 2;
    const int share = (heads + split - 1) / split;
    const size_t smem = a.inv_freq ? (size_t)most_rows * (HD / 2) * sizeof(float2) : 0;
    static size_t allowed[64] = {};   // per device: the shared-memory limit as raised so far
    int dev = 0;
    cudaGetDevice(&dev);
    if (smem > 48 * 1024 && (dev < 0 || dev >= 64 || allowed[dev] < 128 * 1024)) {
        const cudaError_t e = cudaFuncSetAttribute(k_paged_append_f8<TI, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 1024);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) allowed[dev] = 128 * 1024;
    }
    return launch_kernel(k_paged_append_f8<TI, HD>, dim3(segs, (heads + share - 1) / share), dim3(kF8Threads), smem, st, 1, a, gw, share, status);
}

}  // namespace

cudaError_t paged_append_f8(const AppendF8 &a, int hd, int in_dtype, unsigned *status, cudaStream_t st) {
    if (in_dtype == DLLM_BF16)
        return hd == 64 ? launch_append_f8<bf16, 64>(a, status, st) : launch_append_f8<bf16, 128>(a, status, st);
    return hd == 64 ? launch_append_f8<float, 64>(a, status, st) : launch_append_f8<float, 128>(a, status, st);
}

}  // namespace dllm
