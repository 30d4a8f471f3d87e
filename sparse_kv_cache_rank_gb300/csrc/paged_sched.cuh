// paged_sched.cuh -- how the attention over a paged cache is cut into equal work, for batches
// whose lengths only the device knows.
//
// The G = n_q / n_kv query heads of a key head read the same keys, so the rows that share them
// are the sequence's new tokens times G: row token * G + head of the group.  A *unit* of work is
// `unit_rows` such rows of one sequence and key head over the key tiles that its last row
// sees.  Every CTA lays the units end to end by itself (sequence, key head, rows), counts
// their key tiles, and takes the slice of that line that its index gives it: equal numbers of
// key tiles whatever the lengths.  A unit cut by a slice's end leaves unnormalised partial
// results (O, m, l) in the workspace; a second kernel joins them in the order of the keys,
// the same order every time.  (The lengths are device data, so the host cannot lay out the slices;
// a CTA needs 2.4 us for it, most of them the latency of dependent loads and divisions.)
#pragma once

#include "paged.cuh"

namespace dllm {

struct PagedPart {     // one per CTA: the split unit whose first slice it computed
    int nseg, slot, tok0, row0, nrows, g, pad[2];
};

struct PagedSched {
    PagedSeqs sq;
    int T, n_q, n_kv, G;
    int unit_rows;                      // rows of a unit
    int key_tile, max_new, mask_block;
    float *part_o;                      // [2 grid][unit_rows][hd]
    float2 *part_ml;                    // [2 grid][unit_rows]: reference m (log2), sum l
    PagedPart *meta;                    // [grid]
    float *lse;                         // [T, n_q] or NULL
};

// Key tiles of a unit whose last row is of the sequence's new token `last` (at least one, so
// that a unit whose rows see nothing still writes its zeros).
__device__ __forceinline__ int unit_tiles(const PagedSched &a, int len_raw, int len, int n_new, int last) {
    const int lim = PagedSeqs::visible(len_raw - n_new + last, len, a.mask_block);
    const int n = (int)(((long long)lim + a.key_tile - 1) / a.key_tile);
    return n > 0 ? n : 1;
}

struct Seg {            // a slice of a unit
    int b, g;
    int row0, nrows;    // rows of the sequence (token * G + head)
    int start, pos0;    // row of the batch and position of the sequence's first new token
    int len;            // keys of the sequence
    int k0, k1, n;      // key tiles [k0, k1) of n
};

// The units of a CTA's slice, one after another (fp32: every thread walks them by itself; bf16: the TMA warp does
// and hands them to the other roles).
struct Walker {
    int b, g, u, kt;
    long long left;
    int start, n_new, rows, len_raw, len;   // of sequence b

    __device__ __forceinline__ void load(const PagedSched &a) {
        rows = a.sq.rows(b, a.T, a.max_new, start, n_new) * a.G;
        len_raw = a.sq.kv_len[b];
        len = a.sq.keys(b);
    }
    __device__ __forceinline__ bool next(const PagedSched &a, Seg &s) {
        if (left <= 0) return false;
        s.b = b;
        s.g = g;
        s.row0 = u * a.unit_rows;
        s.nrows = min(a.unit_rows, rows - s.row0);
        s.start = start;
        s.pos0 = len_raw - n_new;
        s.len = len;
        s.n = unit_tiles(a, len_raw, len, n_new, (s.row0 + s.nrows - 1) / a.G);
        s.k0 = kt;
        const long long e = kt + left;
        s.k1 = e < s.n ? (int)e : s.n;
        left -= s.k1 - s.k0;
        kt = 0;
        if (left > 0) {   // more in this slice: the next unit
            if ((u + 1) * a.unit_rows < rows) {
                ++u;
            } else {
                u = 0;
                if (++g == a.n_kv) {
                    g = 0;
                    do {
                        ++b;
                        load(a);
                    } while (rows <= 0 && b + 1 < a.sq.B);
                }
            }
        }
        return true;
    }
};

// Where the CTA's slice starts, by all its threads (multiples of 32): pre is scratch of B + 1
// words, out receives b, g, u, kt (ints), then left and the slice length (long longs).  The
// caller synchronises afterwards.
__device__ __forceinline__ void schedule_start(const PagedSched &a, long long *pre, int *out) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nthr = blockDim.x;
    const int B = a.sq.B;
    auto count = [&](int b, int first, int step) -> long long {   // tiles of a key head, strided over its units
        int start, n_new;
        const int rows = a.sq.rows(b, a.T, a.max_new, start, n_new) * a.G;
        const int raw = a.sq.kv_len[b], len = a.sq.keys(b);
        long long s = 0;
        for (int r = first * a.unit_rows; r < rows; r += step * a.unit_rows)
            s += unit_tiles(a, raw, len, n_new, (min(r + a.unit_rows, rows) - 1) / a.G);
        return s;
    };
    if ((long long)a.max_new * a.G <= a.unit_rows) {   // a unit per key head
        for (int b = tid; b < B; b += nthr) pre[b + 1] = count(b, 0, 1) * a.n_kv;
    } else {
        for (int b = warp; b < B; b += nthr / 32) {
            long long s = count(b, lane, 32);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane == 0) pre[b + 1] = s * a.n_kv;
        }
    }
    __syncthreads();
    if (warp == 0) {
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
        __syncwarp();
        const long long chunk = (run + gridDim.x - 1) / gridDim.x;
        const long long at = (long long)blockIdx.x * chunk;
        const long long left = run - at < chunk ? run - at : chunk;
        int b = 0, g = 0, u = 0, kt = 0;
        if (left > 0) {
            // the sequence that tile `at` belongs to
            for (int b0 = 0; b0 < B; b0 += 32)
                b += __popc(__ballot_sync(0xffffffffu, b0 + lane < B && pre[b0 + lane + 1] <= at));
            const long long base = b > 0 ? pre[b] : 0;
            const long long off = at - base, per = (pre[b + 1] - base) / a.n_kv;
            g = (int)(off / per);
            long long rem = off - g * per;
            // the unit: 32 at a time
            int start, n_new;
            const int rows = a.sq.rows(b, a.T, a.max_new, start, n_new) * a.G;
            const int raw = a.sq.kv_len[b], len = a.sq.keys(b);
            for (int u0 = 0;; u0 += 32) {
                const int r = (u0 + lane) * a.unit_rows;
                const int n = r < rows ? unit_tiles(a, raw, len, n_new, (min(r + a.unit_rows, rows) - 1) / a.G) : 0;
                long long x = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o) x += y;
                }
                const long long tot = __shfl_sync(0xffffffffu, x, 31);
                if (rem < tot || tot == 0) {
                    const unsigned m = __ballot_sync(0xffffffffu, x > rem);
                    const int l = m ? __ffs(m) - 1 : 0;
                    u = u0 + l;
                    kt = (int)(rem - __shfl_sync(0xffffffffu, x - n, l));
                    break;
                }
                rem -= tot;
            }
        }
        if (lane == 0) {
            out[0] = b;
            out[1] = g;
            out[2] = u;
            out[3] = kt;
            *reinterpret_cast<long long *>(out + 4) = left;
            *reinterpret_cast<long long *>(out + 6) = chunk;
        }
    }
}

__device__ __forceinline__ Walker walk_from(const PagedSched &a, const int *out) {
    Walker w;
    w.b = out[0];
    w.g = out[1];
    w.u = out[2];
    w.kt = out[3];
    w.left = *reinterpret_cast<const long long *>(out + 4);
    if (w.left > 0) w.load(a);
    return w;
}

// What the join has to know of a cut unit, by the CTA that has its first tile.
__device__ __forceinline__ PagedPart part_of(const Seg &s, int slot, long long chunk) {
    PagedPart p{};
    p.nseg = 1 + (int)((s.n - s.k1 + chunk - 1) / chunk);
    p.slot = slot;
    p.tok0 = s.start;
    p.row0 = s.row0;
    p.nrows = s.nrows;
    p.g = s.g;
    return p;
}

__device__ __forceinline__ float ex2(float x) {   // 2^x, relative error ~2^-22; 2^-inf = 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A row's log-sum-exp from its reference (log2) and sum: -inf without a key, the sum's NaN as it is.
__device__ __forceinline__ float row_lse(float m, float l) {
    return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// Joins the slices of the units that were cut, in the order of their keys:
//   M = max m_s,  L = sum l_s 2^(m_s - M),  O = sum O_s 2^(m_s - M) / L
// One warp per row, every row of a launch at once: it is a chain of three loads (what was cut, m and l,
// O), not bytes, that costs (3 us after 16 slices of 32 rows).  A warp for every fourth row took 9 us longer
// there: 24 against 15.4 us with the attention before it.
template <class T, int HD>
__global__ void __launch_bounds__(256) k_paged_join(const PagedSched a, T *A) {
    griddep_wait();
    griddep_launch();
    const PagedPart pm = a.meta[blockIdx.x];
    if (pm.nseg <= 0) return;
    constexpr int E = HD / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int r = blockIdx.y * 8 + warp; r < pm.nrows; r += gridDim.y * 8) {
        auto at = [&](int s) -> size_t {   // the first slice, then the next CTAs' first ones
            return (size_t)(s == 0 ? pm.slot : 2 * (blockIdx.x + s)) * a.unit_rows + r;
        };
        // a lane per slice for (m, l); then the slices' rows, several on their way at once
        float M = -INFINITY, m = -INFINITY, l = 0.f;
        bool nan = false;   // in a slice's sum: the row has a score that is no number
        for (int s0 = 0; s0 < pm.nseg; s0 += 32) {
            const float2 ml = s0 + lane < pm.nseg ? a.part_ml[at(s0 + lane)] : make_float2(-INFINITY, 0.f);
            if (s0 == 0) {
                m = ml.x;
                l = ml.y;
            }
            M = fmaxf(M, ml.x);
            nan |= ml.y != ml.y;
        }
        nan = __any_sync(0xffffffffu, nan);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        float L = 0.f, o[E] = {};
        for (int s0 = 0; M != -INFINITY && s0 < pm.nseg; s0 += 32) {
            if (s0 > 0) {
                const float2 ml = s0 + lane < pm.nseg ? a.part_ml[at(s0 + lane)] : make_float2(-INFINITY, 0.f);
                m = ml.x;
                l = ml.y;
            }
            const float f = m == -INFINITY ? 0.f : ex2(m - M);
            const float lf = m == -INFINITY ? 0.f : l * f;
#pragma unroll 4
            for (int s = 0; s < min(32, pm.nseg - s0); ++s) {   // in the order of the keys
                const float fs = __shfl_sync(0xffffffffu, f, s);
                L += __shfl_sync(0xffffffffu, lf, s);
                const float *src = a.part_o + at(s0 + s) * HD + lane * E;
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = fs == 0.f ? o[e] : fmaf(src[e], fs, o[e]);   // (without keys: not written to)
            }
        }
        if (nan) L = NAN;
        const float inv = L == 0.f ? 0.f : 1.0f / L;
        const int row = pm.row0 + r;
        const size_t out = (size_t)(pm.tok0 + row / a.G) * a.n_q + pm.g * a.G + row % a.G;
        T *dst = A + out * HD + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) dst[e] = from_f32<T>(o[e] * inv);
        if (a.lse && lane == 0) a.lse[out] = row_lse(M, L);
    }
}

// Workspace of a launch of `grid` CTAs: partial results, their (m, l), the cut units.
inline size_t paged_up256(size_t x) { return (x + 255) & ~size_t(255); }
inline size_t paged_part_bytes(int grid, int unit_rows, int hd) {
    const size_t rows = 2 * (size_t)grid * unit_rows;
    return paged_up256(rows * hd * 4) + paged_up256(rows * 8) + paged_up256((size_t)grid * sizeof(PagedPart)) + 256;
}
inline PagedSched paged_sched(const PagedAttn &p, int grid, int unit_rows, int key_tile, void *ws) {
    PagedSched a{};
    a.sq = p.sq;
    a.T = p.T;
    a.n_q = p.n_q;
    a.n_kv = p.n_kv;
    a.G = p.n_q / p.n_kv;
    a.unit_rows = unit_rows;
    a.key_tile = key_tile;
    a.max_new = p.max_new;
    a.mask_block = p.mask_block;
    a.lse = p.lse;
    const size_t rows = 2 * (size_t)grid * unit_rows;
    uint8_t *w = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(ws) + 255) & ~uintptr_t(255));
    a.part_o = reinterpret_cast<float *>(w);
    w += paged_up256(rows * p.hd * 4);
    a.part_ml = reinterpret_cast<float2 *>(w);
    w += paged_up256(rows * 8);
    a.meta = reinterpret_cast<PagedPart *>(w);
    return a;
}
template <class T, int HD>
cudaError_t paged_join(const PagedSched &a, int grid, T *A, cudaStream_t st) {
    const int ry = (a.unit_rows + 7) / 8;   // a warp per row
    return launch_kernel(k_paged_join<T, HD>, dim3(grid, ry), dim3(256), 0, st, 1, a, A);
}

}  // namespace dllm
