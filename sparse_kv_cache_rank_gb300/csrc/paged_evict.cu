// paged_evict.cu -- slots of a paged cache are given up, in each sequence and key head those whose keys have
// the lowest accumulated attention weight:
//
//   L = kv_len[b], K = min(keep[b], L).  Order of the slots j < L: protected ones (their token among the last `recent`
//   positions) before others, then by descending score, then by ascending slot; the first K stay.
//   The i-th slot below K that does not stay receives the i-th slot from K on that does (key, value, score, position).
//
// Attention does not depend on the order of its keys and their rotation is in them, so only rows from K on move, into
// holes below K: as few as can be, and no row is read after another is written onto it.
//
// Launch 1, a CTA per (sequence, key head): scores as ordered integers; the K-th largest, ties by slot; then holes and
// rows to move are listed in the order of the slots, for 8-bit pages with the moved rows' scales.  Launch 2 moves the
// rows, a few lanes each; for 8-bit pages a warp takes a page's holes: its scale becomes the largest of the rows that come
// in and, if any stay, of its own; rows that stay or come are rounded to it (E4M3(code old / new)).  Every byte that
// launch 2 reads of a page is from K on or in the warp's own page.
//
// What bounds it: the scores and positions read once, 4 rows' bytes a move, and its entry in the lists: 20 bytes, written,
// filled in by a second pass once the order is known, and read.
#include <climits>

#include "e4m3.cuh"
#include "paged.cuh"

namespace dllm {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kPer = 8;                        // slots of a thread at a time
constexpr int kBins = 2 * kSelThreads;

struct EvictArgs {
    PagedEvict p;
    int *moves;                                // [B, n_kv] number of moves
    int *holes;                                // [B, n_kv, half] slots to fill
    int4 *list;                                // [B, n_kv, half]: slot that moves, its row of the pool (-1: none), its key's
                                               // scale | its value's << 8
    int *first;                                // [B, n_kv, pages]: moves before a page's first slot (8-bit pages)
    int half, pages;
};

// Scores as integers in their order; NaN below all, -0 as 0.
__device__ __forceinline__ uint32_t ordered(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive sum over the CTA's threads and the total; two barriers.
__device__ __forceinline__ int cta_scan(int v, int *warp_sums, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    const int w = lane < kSelWarps ? warp_sums[lane] : 0;
    int before = lane < warp ? w : 0, all = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, o);
        all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    __syncthreads();
    total = all;
    return before + x - v;
}

// Where among the slots j0 + e 512 + thread, in their order, a flag's slot stands: exclusive counts of the flags
// (and of the second ones, << 16: at most 4096 of each), by ballots; `cell` holds kSelWarps N counts.
template <int N>
__device__ __forceinline__ void ranks(const bool (&f)[N], const bool (&f2)[N], int *cell, int *sums, int (&out)[N], int &total) {
    static_assert(N * kSelWarps <= kSelThreads, "a count a thread");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned m[N], m2[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
        m[e] = __ballot_sync(0xffffffffu, f[e]);
        m2[e] = __ballot_sync(0xffffffffu, f2[e]);
        if (lane == 0) cell[e * kSelWarps + warp] = __popc(m[e]) | __popc(m2[e]) << 16;
    }
    __syncthreads();
    const int v = threadIdx.x < kSelWarps * N ? cell[threadIdx.x] : 0;
    const int x = cta_scan(v, sums, total);
    if (threadIdx.x < kSelWarps * N) cell[threadIdx.x] = x;
    __syncthreads();
    const unsigned below = (1u << lane) - 1;
#pragma unroll
    for (int e = 0; e < N; ++e)
        out[e] = cell[e * kSelWarps + warp] + (__popc(m[e] & below) | __popc(m2[e] & below) << 16);
    __syncthreads();
}

struct Head {               // a CTA's sequence and key head
    int b, g, L, K;
    long long safe_from;    // positions from here on are protected
};
// False if there is nothing to give up (scores and positions copied, no moves).
__device__ __forceinline__ bool head_of(const EvictArgs &a, Head &x) {
    const PagedEvict &p = a.p;
    x.b = blockIdx.x / p.n_kv;
    x.g = blockIdx.x - x.b * p.n_kv;
    x.L = min(p.sq.keys(x.b), p.slots);
    x.K = min(max(p.keep[x.b], 0), x.L);
    x.safe_from = (long long)x.L + (p.pos_base ? p.pos_base[x.b] : 0) - p.recent;
    if (x.K < x.L) return true;
    if (threadIdx.x == 0) a.moves[blockIdx.x] = 0;
    const size_t at = (size_t)blockIdx.x * p.slots;
    if (p.score_out != p.score || p.slot_pos_out != p.slot_pos)
        for (int j = threadIdx.x; j < x.L; j += kSelThreads) {
            p.score_out[at + j] = p.score[at + j];
            p.slot_pos_out[at + j] = p.slot_pos[at + j];
        }
    return false;
}

// The border among the scores is closed in on by counting those between two values into 1024 bins of equal width and
// going on within the bin in which the K-th largest lies: four rounds for 32 bits, two or three as a rule.  (Equal bins
// between the least and the largest spread the counts; by the leading bits, thousands of additions meet in the few bins
// that scores of one magnitude share; a search bit by bit looks at every score 32 times.)  The first `cached` slots'
// scores are kept in shared memory as ordered integers, with a bit for the protected ones; later ones are read again in
// every round.  Loads go out eight to a thread before the first is looked at: of 512 threads with registers for
// that, two CTAs an SM, 27 us at 256 heads of up to 8192 slots where 1024 threads with half the registers took 44.
__global__ void __launch_bounds__(kSelThreads, 2) k_evict_select(const EvictArgs a, int cached) {
    extern __shared__ uint32_t su[];           // [cached] scores, [cached / 32] bits
    __shared__ int hist[kBins];                // (later the cells of the ranks)
    __shared__ int sums[32];
    __shared__ uint32_t s_lo, s_hi;
    __shared__ int s_want, s_all;
    const PagedEvict &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31;
    griddep_wait();
    griddep_launch();
    Head x;
    if (!head_of(a, x)) return;
    const int L = x.L, K = x.K;
    const size_t at = (size_t)blockIdx.x * p.slots;
    const float *score = p.score + at;
    const int32_t *tag = p.slot_pos + at;
    uint32_t *bits = su + cached;
    const bool copies = p.score_out != p.score, copies_pos = p.slot_pos_out != p.slot_pos, by_pos = p.recent > 0;
    int mine = 0;
    for (int j0 = 0; j0 < L; j0 += kPer * kSelThreads) {   // (whole warps)
        float sc[kPer];
        int32_t tg[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int j = j0 + e * kSelThreads + tid;
            sc[e] = j < L ? score[j] : 0.f;
            tg[e] = j < L && (by_pos || copies_pos) ? tag[j] : 0;
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int j = j0 + e * kSelThreads + tid;
            const bool safe = j < L && by_pos && tg[e] >= x.safe_from;
            const unsigned m = __ballot_sync(0xffffffffu, safe);
            if (j < cached) {                  // (a multiple of 512)
                if (lane == 0) bits[j >> 5] = m;
                su[j] = ordered(sc[e]);
            }
            mine += safe;
            // kept scores into place; those of the holes among them are written again when their rows move
            if (j < K) {
                if (copies) p.score_out[at + j] = sc[e];
                if (copies_pos) p.slot_pos_out[at + j] = tg[e];
            }
        }
    }
    int n_safe;
    cta_scan(mine, sums, n_safe);
    auto value = [&](int j) { return j < cached ? su[j] : ordered(score[j]); };
    auto is_safe = [&](int j) { return j < cached ? (bits[j >> 5] >> (j & 31) & 1) != 0 : by_pos && tag[j] >= x.safe_from; };
    const bool among_safe = n_safe >= K;       // the border runs through the protected ones: all others go
    int want = among_safe ? K : K - n_safe;    // how many of its class stay
    const bool none = want == 0;
    // least and largest of the class
    uint32_t lo = 0xffffffffu, hi = 0;
    if (tid == 0) {
        s_lo = lo;
        s_hi = hi;
        s_all = 0;
    }
#pragma unroll 4
    for (int j = tid; j < L; j += kSelThreads)
        if (is_safe(j) == among_safe) {
            const uint32_t u = value(j);
            lo = min(lo, u);
            hi = max(hi, u);
        }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    __syncthreads();
    if (lane == 0) {
        atomicMin(&s_lo, lo);
        atomicMax(&s_hi, hi);
    }
    __syncthreads();
    lo = s_lo;
    hi = s_hi;
    while (!none && lo < hi) {
        const int shift = max(0, 32 - __clz(hi - lo) - 10);
        hist[tid] = hist[tid + kSelThreads] = 0;
        __syncthreads();
#pragma unroll 8
        for (int j = tid; j < L; j += kSelThreads) {
            const uint32_t u = value(j);
            if (u >= lo && u <= hi && is_safe(j) == among_safe) atomicAdd(&hist[(u - lo) >> shift], 1);
        }
        __syncthreads();
        // thread t has bins 1023 - 2 t and the one below: the bin in which the count from above reaches `want`
        const int bin = kBins - 1 - 2 * tid, c0 = hist[bin], c1 = hist[bin - 1];
        int total;
        const int before = cta_scan(c0 + c1, sums, total);
        if (before < want && before + c0 + c1 >= want) {
            const bool upper = before + c0 >= want;
            const int left = want - before - (upper ? 0 : c0);
            const uint32_t from = lo + ((uint32_t)(upper ? bin : bin - 1) << shift), last = from + ((1u << shift) - 1);
            s_want = left;
            s_lo = from;
            s_hi = last < hi ? last : hi;      // (no wrap: bins lie within lo .. lo + 1024 2^shift - 1, which may pass 2^32)
            if (last < from) s_hi = hi;
            s_all = left == (upper ? c0 : c1);
        }
        __syncthreads();
        want = s_want;
        lo = s_lo;
        hi = s_hi;
    }
    // Of the class, scores above lo stay, and the first `want` slots of those equal to it (no order needed if that is all
    // of them).  Holes and slots that move go into the lists in the order of the slots.
    const bool all = s_all;
    int eq_run = 0, hole_run = 0, src_run = 0;
    int *holes = a.holes + (size_t)blockIdx.x * a.half;
    int4 *list = a.list + (size_t)blockIdx.x * a.half;
    __syncthreads();
    for (int j0 = 0; j0 < L; j0 += kSelThreads * kPer) {
        bool stays[kPer], equal[kPer], src[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int j = j0 + e * kSelThreads + tid;
            stays[e] = equal[e] = src[e] = false;
            if (j < L) {
                const bool safe = is_safe(j);
                if (safe != among_safe) {
                    stays[e] = safe;           // a protected one beside a border among the others
                } else if (!none) {
                    const uint32_t u = value(j);
                    stays[e] = all ? u >= lo : u > lo;
                    equal[e] = !all && u == lo;
                }
            }
        }
        int rank[kPer], total;
        if (!all && !none) {
            ranks(equal, src, hist, sums, rank, total);
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                if (equal[e]) stays[e] = eq_run + rank[e] < want;
            eq_run += total;
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int j = j0 + e * kSelThreads + tid;
            src[e] = j >= K && stays[e];
            equal[e] = j < K && !stays[e];     // holes
        }
        ranks(equal, src, hist, sums, rank, total);
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int j = j0 + e * kSelThreads + tid, h = hole_run + (rank[e] & 0xffff);
            if (p.k_scale && j < K && (j & ((1 << p.sq.page_log2) - 1)) == 0)
                a.first[(size_t)blockIdx.x * a.pages + (j >> p.sq.page_log2)] = h;
            if (equal[e]) holes[h] = j;
            if (src[e]) list[src_run + (rank[e] >> 16)].x = j;
        }
        hole_run += total & 0xffff;
        src_run += total >> 16;
    }
    if (tid == 0) a.moves[blockIdx.x] = hole_run;
    // where the slots that move lie, and their scales: all of the CTA's threads have one
    __syncthreads();
    for (int i0 = 0; i0 < src_run; i0 += 4 * kSelThreads) {
        int j[4], id[4], sk[4], sv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = i0 + e * kSelThreads + tid;
            j[e] = i < src_run ? list[i].x : -1;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            id[e] = j[e] >= 0 ? p.sq.page_table[(size_t)x.b * p.sq.max_pages + (j[e] >> p.sq.page_log2)] : -1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const size_t at_scale = (size_t)id[e] * p.n_kv + x.g;
            const bool here = p.k_scale && (unsigned)id[e] < (unsigned)p.sq.n_pages;
            sk[e] = here ? p.k_scale[at_scale] : 0;
            sv[e] = here ? p.v_scale[at_scale] : 0;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (j[e] >= 0)
                list[i0 + e * kSelThreads + tid] =
                    make_int4(j[e], (unsigned)id[e] < (unsigned)p.sq.n_pages ? (id[e] << p.sq.page_log2) + (j[e] & ((1 << p.sq.page_log2) - 1)) : -1,
                              sk[e] | sv[e] << 8, 0);
    }
}

// Lengths and positions, by the first threads of launch 2 (nothing in it reads them).
__device__ __forceinline__ void write_lengths(const PagedEvict &p) {
    for (int b = blockIdx.y * blockDim.x + threadIdx.x; b < p.sq.B; b += gridDim.y * blockDim.x) {
        const int raw = p.kv_len[b], L = min(p.sq.keys(b), p.slots), K = min(max(p.keep[b], 0), L);
        // (a length past the table or the arrays is left to itself unless slots are given up)
        if (K < L) {
            const int base = p.pos_base ? p.pos_base[b] : 0;
            p.kv_len_out[b] = K;
            if (p.pos_base_out) p.pos_base_out[b] = base + (L - K);
        } else {
            p.kv_len_out[b] = raw;
            if (p.pos_base_out) p.pos_base_out[b] = p.pos_base ? p.pos_base[b] : 0;
        }
    }
}

__device__ __forceinline__ long long pool_row(const PagedSeqs &sq, int b, int slot) {
    const int id = sq.page_table[(size_t)b * sq.max_pages + (slot >> sq.page_log2)];
    return (unsigned)id < (unsigned)sq.n_pages ? ((long long)id << sq.page_log2) + (slot & ((1 << sq.page_log2) - 1)) : -1;
}

// Rows of `units` 16-byte units (a power of two, at most 32), as many a warp as there is room for, two turns' loads under
// way at a time.
__global__ void __launch_bounds__(256) k_evict_move(const EvictArgs a, int units, unsigned *status) {
    const PagedEvict &p = a.p;
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31, per = 32 / units, u = lane % units;
    const int bg = blockIdx.x;
    if (bg == 0) write_lengths(p);
    const int b = bg / p.n_kv, g = bg - b * p.n_kv;
    const int n = a.moves[bg], stride = gridDim.y * 8 * per;
    const int *holes = a.holes + (size_t)bg * a.half;
    const int4 *list = a.list + (size_t)bg * a.half;
    const size_t at = (size_t)bg * p.slots;
    const uint4 *k = static_cast<const uint4 *>(p.k_pages), *v = static_cast<const uint4 *>(p.v_pages);
    for (int i = (blockIdx.y * 8 + (threadIdx.x >> 5)) * per + lane / units; i < n; i += 2 * stride) {
        int4 m[2];
        int hole[2];
        long long dst[2];
        uint4 x[2], y[2];
        float sc[2];
        int32_t tg[2];
        bool ok[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            ok[j] = false;
            if (i + j * stride < n) {
                m[j] = list[i + j * stride];
                hole[j] = holes[i + j * stride];
                dst[j] = pool_row(p.sq, b, hole[j]);
                ok[j] = dst[j] >= 0 && m[j].y >= 0;
                if (ok[j]) {
                    const size_t s = ((size_t)m[j].y * p.n_kv + g) * units + u;
                    x[j] = k[s];
                    y[j] = v[s];
                }
                if (u == 0) {
                    sc[j] = p.score[at + m[j].x];
                    tg[j] = p.slot_pos[at + m[j].x];
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (i + j * stride < n) {
                if (ok[j]) {
                    const size_t d = ((size_t)dst[j] * p.n_kv + g) * units + u;
                    static_cast<uint4 *>(p.k_pages)[d] = x[j];
                    static_cast<uint4 *>(p.v_pages)[d] = y[j];
                } else if (u == 0) {
                    raise_status(status, DLLM_STATUS_PAGE);
                }
                if (u == 0) {
                    p.score_out[at + hole[j]] = sc[j];
                    p.slot_pos_out[at + hole[j]] = tg[j];
                }
            }
    }
}

// 16 codes under the scale byte `from` to the byte `to` (from <= to).
__device__ __forceinline__ uint4 shifted(uint4 c, int from, int to) {
    if (from == to) return c;
    const float f = __uint_as_float((uint32_t)max(from - to + 127, 0) << 23);   // 2^(from - to); 0 from 2^-127 on
    uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 lo = f32_of_e4m3x2(w[i] & 0xffffu), hi = f32_of_e4m3x2(w[i] >> 16);
        w[i] = e4m3x2(lo.x * f, lo.y * f) | e4m3x2(hi.x * f, hi.y * f) << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 8-bit pages: `gl` lanes (a power of two, a row's units at least) take the holes of one page, keys and values side by
// side.  A page's moves are few (four of 16 slots, say), so what it takes is the chain of loads to them; pages side by side
// in a warp, and many warps, hide it: 31 us at 256 heads of up to 8192 slots (60 where every other page's rows are rounded
// to a larger scale), 37 us with a page a warp, 46 with the next page's moves read ahead, which took 80 registers.
__global__ void __launch_bounds__(256, 6) k_evict_move_f8(const EvictArgs a, int units, int gl, unsigned *status) {
    const PagedEvict &p = a.p;
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31, l = lane & (gl - 1), per = gl / units, u = l % units, r = l / units;
    const int bg = blockIdx.x;
    if (bg == 0) write_lengths(p);
    const int b = bg / p.n_kv, g = bg - b * p.n_kv;
    const int n = a.moves[bg], page = 1 << p.sq.page_log2;
    if (n == 0) return;
    const int4 *list = a.list + (size_t)bg * a.half;
    const int *holes = a.holes + (size_t)bg * a.half, *before = a.first + (size_t)bg * a.pages;
    const size_t at = (size_t)bg * p.slots;
    const int L = min(p.sq.keys(b), p.slots), K = min(max(p.keep[b], 0), L);   // (n > 0: kv_len_out is K, so K stays what it was)
    const int pages = (K + page - 1) >> p.sq.page_log2, abreast = 32 / gl;
    uint4 *kr = static_cast<uint4 *>(p.k_pages), *vr = static_cast<uint4 *>(p.v_pages);
    for (int pg0 = (blockIdx.y * 8 + (threadIdx.x >> 5)) * abreast; pg0 < pages; pg0 += gridDim.y * 8 * abreast) {   // (whole warps)
        const int pg = pg0 + lane / gl, s0 = pg << p.sq.page_log2, s1 = min(s0 + page, K);
        int i0 = 0, i1 = 0, id = -1;
        if (pg < pages) {
            i0 = before[pg];
            i1 = pg + 1 < pages ? before[pg + 1] : n;
            id = p.sq.page_table[(size_t)b * p.sq.max_pages + pg];
        }
        const bool here = (unsigned)id < (unsigned)p.sq.n_pages;
        // the largest scales that come in (0: rows without a page); the scores on the way
        int in_k = 0, in_v = 0;
        bool lost = !here && i0 < i1;
        for (int i = i0 + l; i < i1; i += gl) {
            const int4 m = list[i];
            const int hole = holes[i];
            in_k = max(in_k, m.z & 255);
            in_v = max(in_v, m.z >> 8);
            lost |= m.y < 0;
            p.score_out[at + hole] = p.score[at + m.x];
            p.slot_pos_out[at + hole] = p.slot_pos[at + m.x];
        }
        if (lost) raise_status(status, DLLM_STATUS_PAGE);
        __syncwarp();
        for (int o = gl / 2; o > 0; o >>= 1) {
            in_k = max(in_k, __shfl_xor_sync(0xffffffffu, in_k, o));
            in_v = max(in_v, __shfl_xor_sync(0xffffffffu, in_v, o));
        }
        const bool comes = here && in_k > 0, stay = i1 - i0 < s1 - s0;   // some of the page's rows stay
        const size_t scale_at = (size_t)(comes ? id : 0) * p.n_kv + g;
        int old_k = 0, old_v = 0;
        if (comes && stay) {
            old_k = p.k_scale[scale_at];
            old_v = p.v_scale[scale_at];
        }
        const int now_k = max(old_k, in_k), now_v = max(old_v, in_v);
        // this lane's 16 bytes of the page's first row
        const size_t base = (((size_t)(comes ? id : 0) << p.sq.page_log2) * p.n_kv + g) * units + u, row = (size_t)p.n_kv * units;
        const bool grows = comes && stay && (now_k > old_k || now_v > old_v);
        if (__any_sync(0xffffffffu, grows))
            // rows that stay: the slots between the holes, 32 at a time
            for (int j0 = 0; j0 < page; j0 += 32) {
                const int left = s1 - s0 - j0;
                unsigned m = !grows || left <= 0 ? 0u : (left < 32 ? (1u << left) - 1 : 0xffffffffu);
                unsigned h = 0;
                for (int i = i0 + l; i < i1; i += gl)
                    if ((unsigned)(holes[i] - s0 - j0) < 32u) h |= 1u << (holes[i] - s0 - j0);
                __syncwarp();
                for (int o = gl / 2; o > 0; o >>= 1) h |= __shfl_xor_sync(0xffffffffu, h, o);
                m &= ~h;
                for (int j = r; j < 32; j += per) {
                    if (!(m >> j & 1)) continue;
                    const size_t x = base + (j0 + j) * row;
                    uint4 k, v;
                    if (now_k > old_k) k = kr[x];
                    if (now_v > old_v) v = vr[x];
                    if (now_k > old_k) kr[x] = shifted(k, old_k, now_k);
                    if (now_v > old_v) vr[x] = shifted(v, old_v, now_v);
                }
                __syncwarp();
            }
        if (comes) {
            for (int i = i0 + r; i < i1; i += per) {
                const int4 m = list[i];
                if (m.y < 0) continue;
                const size_t s = ((size_t)m.y * p.n_kv + g) * units + u, d = base + (holes[i] - s0) * row;
                const uint4 x = kr[s], y = vr[s];
                kr[d] = shifted(x, m.z & 255, now_k);
                vr[d] = shifted(y, m.z >> 8, now_v);
            }
        }
        __syncwarp();                          // (the old scales have been read by every lane)
        if (comes && l == 0) {
            p.k_scale[scale_at] = (uint8_t)now_k;
            p.v_scale[scale_at] = (uint8_t)now_v;
        }
    }
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

// (pages have 8 slots at least)
size_t paged_evict_ws_bytes(int B, int n_kv, int slots, bool f8) {
    const size_t heads = (size_t)B * n_kv, half = (size_t)slots / 2 + 1;
    return up256(heads * 4) + up256(heads * half * 4) + up256(heads * half * 16) + (f8 ? up256(heads * ((size_t)slots / 8 + 1) * 4) : 0) + 256;
}

cudaError_t paged_evict(const PagedEvict &p, int row_bytes, void *ws, unsigned *status, cudaStream_t st) {
    const size_t heads = (size_t)p.sq.B * p.n_kv;
    EvictArgs a{};
    a.p = p;
    a.half = p.slots / 2 + 1;
    a.pages = p.slots / 8 + 1;
    uint8_t *w = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(ws) + 255) & ~uintptr_t(255));
    a.moves = reinterpret_cast<int *>(w);
    w += up256(heads * 4);
    a.holes = reinterpret_cast<int *>(w);
    w += up256(heads * a.half * 4);
    a.list = reinterpret_cast<int4 *>(w);
    w += up256(heads * a.half * 16);
    a.first = reinterpret_cast<int *>(w);
    // shared memory for two CTAs an SM
    const int cached = (p.slots < 24576 ? p.slots + kSelThreads - 1 : 24576) / kSelThreads * kSelThreads;
    const int smem = cached * 4 + cached / 8;
    static bool configured[64] = {};   // per device: raise the shared-memory limit once
    int dev = 0;
    cudaGetDevice(&dev);
    if (smem > 40 * 1024 && (dev < 0 || dev >= 64 || !configured[dev])) {
        const cudaError_t e = cudaFuncSetAttribute(k_evict_select, cudaFuncAttributeMaxDynamicSharedMemorySize, 24576 * 4 + 24576 / 8);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    cudaError_t e = launch_kernel(k_evict_select, dim3((unsigned)heads), dim3(kSelThreads), smem, st, 1, a, cached);
    if (e != cudaSuccess) return e;
    // CTAs of a head: enough to fill the GPU four times over (heads differ in their moves), a warp having at least a few rows
    long long want = 24LL * num_sms() / (long long)heads + 1;
    const long long most = ((long long)p.slots / 2 + 63) / 64;
    if (want > most) want = most;
    const dim3 grid((unsigned)heads, (unsigned)(want < 1 ? 1 : want));
    const int units = row_bytes / 16;
    if (!p.k_scale) return launch_kernel(k_evict_move, grid, dim3(256), 0, st, 1, a, units, status);
    // lanes of a page: two slots each, so that a page's moves are done in a turn or two
    const int page = 1 << p.sq.page_log2, gl = page / 2 < units ? units : (page / 2 < 32 ? page / 2 : 32);
    return launch_kernel(k_evict_move_f8, grid, dim3(256), 0, st, 1, a, units, gl, status);
}

}  // namespace dllm
