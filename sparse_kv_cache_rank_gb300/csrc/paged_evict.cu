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
// Launch 1, a CTA per (sequence, key head): scores as ordered integers; the K-th by three passes of radix
// counting, ties by slot; then one pass in the order of the slots lists holes and rows to move.  For 8-bit pages the
// moved rows' scales go into the list too.  Launch 2 moves the rows, a warp each; for 8-bit pages a warp takes a
// page's holes: its scale becomes the largest of the rows that come in and, if any stay, of its own; rows that
// stay or come are rounded to it (E4M3(code old / new)).  Every byte that launch 2 reads of a page is from K on or in
// the warp's own page.
//
// What bounds it: the scores and positions read once, 16 bytes of lists a move, 4 rows' bytes a move.
#include <climits>

#include "e4m3.cuh"
#include "paged.cuh"

namespace dllm {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kPer = 4;                        // consecutive slots of a thread in the listing pass
constexpr int kBins = 2048;

struct EvictArgs {
    PagedEvict p;
    int *moves;                                // [B, n_kv] number of moves
    int2 *list;                                // [B, n_kv, half]: slot to fill, slot that moves
    uint16_t *scales;                          // [B, n_kv, half]: its key's scale, its value's << 8
    int half;
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
    const int w = warp_sums[lane];             // (32 warps)
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

__global__ void __launch_bounds__(kSelThreads) k_evict_select(const EvictArgs a) {
    __shared__ int hist[kBins];
    __shared__ int sums[32];
    __shared__ int s_bin, s_rest;
    const PagedEvict &p = a.p;
    const int tid = threadIdx.x, b = blockIdx.x / p.n_kv, g = blockIdx.x - b * p.n_kv;
    griddep_wait();
    griddep_launch();
    const int L = min(p.sq.keys(b), p.slots), K = min(max(p.keep[b], 0), L);
    const int base = p.pos_base ? p.pos_base[b] : 0;
    const size_t at = (size_t)blockIdx.x * p.slots;
    const float *score = p.score + at;
    const int32_t *tag = p.slot_pos + at;
    const long long old_from = (long long)L + base - p.recent;   // positions from here on are protected
    auto is_safe = [&](int j) { return p.recent > 0 && tag[j] >= old_from; };
    if (K == L) {                              // nothing to give up
        if (tid == 0) a.moves[blockIdx.x] = 0;
        if (p.score_out != p.score || p.slot_pos_out != p.slot_pos)
            for (int j = tid; j < L; j += kSelThreads) {
                p.score_out[at + j] = score[j];
                p.slot_pos_out[at + j] = tag[j];
            }
        return;
    }
    // protected slots: all stay, or (more of them than K) the K best of them
    int mine = 0, n_safe = 0;
    if (p.recent > 0) {
        for (int j = tid; j < L; j += kSelThreads) mine += is_safe(j);
        cta_scan(mine, sums, n_safe);
    }
    const bool among_safe = n_safe >= K;       // the border runs through the protected ones
    int rest = among_safe ? K : K - n_safe;    // how many of its class stay
    // the rest-th largest key of the class, 11 + 11 + 10 bits at a time
    uint32_t prefix = 0;
    for (int pass = 0; rest > 0 && pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bins = pass == 2 ? 1024 : 2048;
        for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        for (int j = tid; j < L; j += kSelThreads) {
            const uint32_t u = ordered(score[j]);
            const bool in = pass == 0 || (u >> (pass == 1 ? 21 : 10)) == prefix;
            if (in && is_safe(j) == among_safe) atomicAdd(&hist[(u >> shift) & (bins - 1)], 1);
        }
        __syncthreads();
        // the bin in which the count from above reaches rest; thread t has bins - 1 - 2t and the one below
        const int hi = bins - 1 - 2 * tid;
        const int c0 = hi >= 0 ? hist[hi] : 0, c1 = hi >= 1 ? hist[hi - 1] : 0;
        int total;
        const int before = cta_scan(c0 + c1, sums, total);
        if (before < rest && before + c0 + c1 >= rest) {
            s_bin = before + c0 >= rest ? hi : hi - 1;
            s_rest = before + c0 >= rest ? rest - before : rest - before - c0;
        }
        __syncthreads();
        prefix = prefix << (pass == 2 ? 10 : 11) | (uint32_t)s_bin;
        rest = s_rest;
        __syncthreads();
    }
    // now: of the class, keys above `prefix` stay, and the first `rest` slots of those equal to it
    const bool none = (among_safe ? K : K - n_safe) == 0;
    int eq_run = 0, hole_run = 0, src_run = 0;
    int2 *list = a.list + (size_t)blockIdx.x * a.half;
    uint16_t *scales = a.scales + (size_t)blockIdx.x * a.half;
    for (int j0 = 0; j0 < L; j0 += kSelThreads * kPer) {
        const int first = j0 + tid * kPer;
        bool stays[kPer], equal[kPer];
        int eq = 0;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int j = first + e;
            stays[e] = equal[e] = false;
            if (j < L) {
                const bool safe = is_safe(j);
                if (safe != among_safe) {
                    stays[e] = safe;           // a protected one beside a border among the others
                } else if (!none) {
                    const uint32_t u = ordered(score[j]);
                    stays[e] = u > prefix;
                    equal[e] = u == prefix;
                    eq += equal[e];
                }
            }
        }
        int total;
        int before = eq_run + cta_scan(eq, sums, total);
        eq_run += total;
        int holes = 0, srcs = 0;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            if (equal[e]) stays[e] = before++ < rest;
            const int j = first + e;
            holes += j < K && !stays[e];
            srcs += j >= K && j < L && stays[e];
        }
        // (both counts in one scan: at most 4096 of each)
        const int both = cta_scan(holes | srcs << 16, sums, total);
        int h = hole_run + (both & 0xffff), s = src_run + (both >> 16);
        hole_run += total & 0xffff;
        src_run += total >> 16;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int j = first + e;
            if (j < K && !stays[e]) {
                list[h++].x = j;
            } else if (j < K) {
                if (p.score_out != p.score) p.score_out[at + j] = score[j];
                if (p.slot_pos_out != p.slot_pos) p.slot_pos_out[at + j] = tag[j];
            } else if (j < L && stays[e]) {
                list[s].y = j;
                if (p.k_scale) {
                    const int id = p.sq.page_table[(size_t)b * p.sq.max_pages + (j >> p.sq.page_log2)];
                    const bool here = (unsigned)id < (unsigned)p.sq.n_pages;
                    const size_t x = (size_t)(here ? id : 0) * p.n_kv + g;
                    scales[s] = here ? (uint16_t)(p.k_scale[x] | p.v_scale[x] << 8) : 0;
                }
                ++s;
            }
        }
    }
    if (tid == 0) a.moves[blockIdx.x] = hole_run;
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

// Rows of `units` 16-byte units (a power of two, at most 32), as many a warp as there is room for.
__global__ void __launch_bounds__(256) k_evict_move(const EvictArgs a, int units, unsigned *status) {
    const PagedEvict &p = a.p;
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31, per = 32 / units, u = lane % units;
    const int bg = blockIdx.x;
    if (bg == 0) write_lengths(p);
    const int b = bg / p.n_kv, g = bg - b * p.n_kv;
    const int n = a.moves[bg], stride = gridDim.y * 8 * per;
    const int2 *list = a.list + (size_t)bg * a.half;
    const size_t at = (size_t)bg * p.slots;
    for (int i = (blockIdx.y * 8 + (threadIdx.x >> 5)) * per + lane / units; i < n; i += stride) {
        const int2 m = list[i];
        const long long dst = pool_row(p.sq, b, m.x), src = pool_row(p.sq, b, m.y);
        if (dst >= 0 && src >= 0) {
            const uint4 *k = static_cast<const uint4 *>(p.k_pages), *v = static_cast<const uint4 *>(p.v_pages);
            const size_t s = ((size_t)src * p.n_kv + g) * units + u, d = ((size_t)dst * p.n_kv + g) * units + u;
            const uint4 x = k[s], y = v[s];
            static_cast<uint4 *>(p.k_pages)[d] = x;
            static_cast<uint4 *>(p.v_pages)[d] = y;
        } else if (u == 0) {
            raise_status(status, DLLM_STATUS_PAGE);
        }
        if (u == 0) {
            p.score_out[at + m.x] = p.score[at + m.y];
            p.slot_pos_out[at + m.x] = p.slot_pos[at + m.y];
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

// 8-bit pages: a warp takes the holes of one page, keys and then values.
__global__ void __launch_bounds__(256) k_evict_move_f8(const EvictArgs a, int units, unsigned *status) {
    const PagedEvict &p = a.p;
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31, per = 32 / units, u = lane % units, r = lane / units;
    const int bg = blockIdx.x;
    if (bg == 0) write_lengths(p);
    const int b = bg / p.n_kv, g = bg - b * p.n_kv;
    const int n = a.moves[bg], page = 1 << p.sq.page_log2;
    if (n == 0) return;
    const int2 *list = a.list + (size_t)bg * a.half;
    const uint16_t *scales = a.scales + (size_t)bg * a.half;
    const size_t at = (size_t)bg * p.slots;
    const int L = min(p.sq.keys(b), p.slots), K = min(max(p.keep[b], 0), L);   // (n > 0: kv_len_out is K, so K stays what it was)
    const int pages = (K + page - 1) >> p.sq.page_log2;
    auto lower = [&](int slot) {               // first move whose hole is at or past `slot`
        int lo = 0, hi = n;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (list[mid].x < slot) lo = mid + 1;
            else hi = mid;
        }
        return lo;
    };
    for (int pg = blockIdx.y * 8 + (threadIdx.x >> 5); pg < pages; pg += gridDim.y * 8) {
        const int s0 = pg << p.sq.page_log2, s1 = min(s0 + page, K);
        const int i0 = lower(s0), i1 = lower(s1);
        if (i0 == i1) continue;
        for (int i = i0 + lane; i < i1; i += 32) {
            const int2 m = list[i];
            p.score_out[at + m.x] = p.score[at + m.y];
            p.slot_pos_out[at + m.x] = p.slot_pos[at + m.y];
        }
        const int id = p.sq.page_table[(size_t)b * p.sq.max_pages + pg];
        if ((unsigned)id >= (unsigned)p.sq.n_pages) {
            if (lane == 0) raise_status(status, DLLM_STATUS_PAGE);
            continue;
        }
        // the largest scales that come in (0: rows without a page)
        int in_k = 0, in_v = 0;
        for (int i = i0 + lane; i < i1; i += 32) {
            in_k = max(in_k, scales[i] & 255);
            in_v = max(in_v, scales[i] >> 8);
        }
        in_k = __reduce_max_sync(0xffffffffu, in_k);
        in_v = __reduce_max_sync(0xffffffffu, in_v);
        const bool stay = i1 - i0 < s1 - s0;   // some of the page's rows stay
#pragma unroll 1
        for (int w = 0; w < 2; ++w) {
            uint8_t *sp = (w ? p.v_scale : p.k_scale) + (size_t)id * p.n_kv + g;
            uint4 *rows = static_cast<uint4 *>(w ? p.v_pages : p.k_pages);
            const int old = *sp, in = w ? in_v : in_k, now = stay ? max(old, in) : in;
            __syncwarp();
            if (in > 0) {                      // (0: nothing comes)
                if (stay && now > old) {
                    // rows that stay: the slots of the page between the holes
                    for (int j = s0 + r; j < s1; j += per) {
                        const int i = lower(j);
                        if (i < n && list[i].x == j) continue;
                        uint4 *x = rows + ((((size_t)id << p.sq.page_log2) + (j - s0)) * p.n_kv + g) * units + u;
                        *x = shifted(*x, old, now);
                    }
                }
                for (int i = i0 + r; i < i1; i += per) {
                    const int2 m = list[i];
                    const long long src = pool_row(p.sq, b, m.y);
                    if (src < 0) {
                        if (u == 0) raise_status(status, DLLM_STATUS_PAGE);
                        continue;
                    }
                    const uint4 x = rows[((size_t)src * p.n_kv + g) * units + u];
                    rows[((((size_t)id << p.sq.page_log2) + (m.x - s0)) * p.n_kv + g) * units + u] =
                        shifted(x, w ? scales[i] >> 8 : scales[i] & 255, now);
                }
                if (lane == 0) *sp = (uint8_t)now;
            } else if (lane == 0) {
                raise_status(status, DLLM_STATUS_PAGE);
            }
            __syncwarp();
        }
    }
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

size_t paged_evict_ws_bytes(int B, int n_kv, int slots, bool f8) {
    const size_t heads = (size_t)B * n_kv, half = (size_t)slots / 2 + 1;
    return up256(heads * 4) + up256(heads * half * 8) + (f8 ? up256(heads * half * 2) : 0) + 256;
}

cudaError_t paged_evict(const PagedEvict &p, int row_bytes, void *ws, unsigned *status, cudaStream_t st) {
    const size_t heads = (size_t)p.sq.B * p.n_kv;
    EvictArgs a{};
    a.p = p;
    a.half = p.slots / 2 + 1;
    uint8_t *w = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(ws) + 255) & ~uintptr_t(255));
    a.moves = reinterpret_cast<int *>(w);
    w += up256(heads * 4);
    a.list = reinterpret_cast<int2 *>(w);
    w += up256(heads * a.half * 8);
    a.scales = reinterpret_cast<uint16_t *>(w);
    cudaError_t e = launch_kernel(k_evict_select, dim3((unsigned)heads), dim3(kSelThreads), 0, st, 1, a);
    if (e != cudaSuccess) return e;
    // CTAs of a head: enough to fill the GPU, a warp having at least a few rows
    long long want = 4LL * num_sms() / (long long)heads + 1;
    const long long most = ((long long)p.slots / 2 + 63) / 64;
    if (want > most) want = most;
    const dim3 grid((unsigned)heads, (unsigned)(want < 1 ? 1 : want));
    return launch_kernel(p.k_scale ? k_evict_move_f8 : k_evict_move, grid, dim3(256), 0, st, 1, a, row_bytes / 16, status);
}

}  // namespace dllm
