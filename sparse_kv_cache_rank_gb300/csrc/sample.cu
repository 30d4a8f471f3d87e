// sample.cu -- one token per row of logits from a given uniform number: temperature, top-k,
// top-p and min-p, then the inverse of the kept tokens' cumulative distribution.
//
//   z_v = fp32(l_v fp32(1 / T)),   w_v = exp(z_v - max z)
//   order: z descending, equal z by lower id.  Every filter keeps a prefix of that order:
//     top-k   the first k;   top-p  the tokens whose mass before them is < p (mass of the
//     first k);   min-p  the tokens with w >= min_p;   the first token always stays
//   token = the lowest kept id whose cumulative kept mass (in id order) exceeds u * total
//
// A row is read once.  Its vocabulary is cut into slices, one per CTA of a cluster, and each
// CTA keeps its scaled slice in shared memory; everything after the load works there, and the
// CTAs exchange only histograms and sums through distributed shared memory.
//
// The prefix's end is found by a radix descent over the order instead of a sort: a
// histogram over bins of the distance to the maximum, then over ever narrower ranges of the
// ordered keys of the bin where the count (top-k) or the mass (top-p) crosses its target,
// until the bin stays or goes whole or holds one value, whose ties the ids order.
//
// Masses are whole numbers, units of 2^-44 of the largest weight (sums of up to 2^18 tokens
// fit 64 bits): their sums are exact in any order, so neither atomics nor the cut into slices
// can move a border.  exp itself is formed to 2^-38 (weight44): an fp32 exponential's
// 2^-23 would move the running sums across the border of a neighbouring token once in a
// few hundred rows of a large vocabulary.
#include <cfloat>

#include "paged.cuh"

namespace dllm {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = kThreads;    // a bin per thread
constexpr int kMaxCluster = 16;
constexpr int kSlice = 16384;      // most tokens of a CTA: 6 bytes each, two CTAs share an SM
constexpr int kSmall = 512;        // candidates up to which one CTA ranks them directly
constexpr float kBinsPerUnit = 16.f;

// ---------------------------------------------------------------- exp in fixed point
constexpr double kLn2_64 = 0.69314718055994530942 / 64;
constexpr double kC1 = (double)(long long)(kLn2_64 * 262144.0) / 262144.0;                       // 12 bits
constexpr double kC2 = (double)(long long)((kLn2_64 - kC1) * 4294967296.0) / 4294967296.0;       // 11 bits
constexpr double kC3 = kLn2_64 - kC1 - kC2;

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

struct ExpTable {
    u64 fix[64];    // 2^(-j/64) in units of 2^-60
    float hi[64];   // the same as a sum of two fp32
    float lo[64];
};

// exp(-(top - z)) in units of 2^-44, off by at most 2^-38 relative; 0 from a distance of 32 on.
// With n = round(64 d / ln 2) and n = 64 k + j:  exp(-d) = 2^-k 2^(-j/64) exp(r), where
// r = n ln2/64 - d lies within ln2/128 and is formed from a three-part ln2/64 whose first two
// products are exact; exp(r) - 1 by its series to r^4 (the rest is below 2^-43).
__device__ __forceinline__ u64 weight44(float top, float z, const ExpTable &tb) {
    if (z == top) return 1ull << 44;   // also for an infinite maximum
    const float d = top - z;
    if (!(d < 32.f)) return 0;
    const float bb = d - top;          // top - z = d + dl exactly
    const float dl = (top - (d - bb)) - (z + bb);
    const float nf = rintf(d * (float)(1.0 / kLn2_64));
    const float r1 = fmaf(-nf, (float)kC1, d);          // exact
    const float p2 = nf * (float)kC2;                   // exact
    const float rh = r1 - p2;
    const float rb = rh - r1;
    const float re = (r1 - (rh - rb)) - (p2 + rb);      // r1 - p2 = rh + re exactly
    const float th = -rh, tl = fmaf(nf, (float)kC3, -(re + dl));
    const float p = fmaf(th * th, fmaf(th, fmaf(th, 1.f / 24.f, 1.f / 6.f), 0.5f), fmaf(tl, fmaf(th * 0.5f, th, th), tl));   // exp(r) - 1 - th
    const int n = (int)nf, j = n & 63, k = n >> 6;
    const float Th = tb.hi[j];
    const float a = Th * th;
    const float rest = fmaf(Th, th, -a) + fmaf(Th, p, tb.lo[j] * th);
    const float unit = __int_as_float((127 + 44 - k) << 23);   // 2^(44 - k)
    return (tb.fix[j] >> (16 + k)) + (u64)(__float2ll_rn(a * unit) + __float2ll_rn(rest * unit));
}

// ---------------------------------------------------------------- ordered keys
__device__ __forceinline__ uint32_t order_key(float z) {   // ascending with z (no NaN, no -0)
    const uint32_t u = __float_as_uint(z);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ int distance_bin(float top, float z) {
    const float d = z == top ? 0.f : (top - z) * kBinsPerUnit;
    return d < (float)(kBins - 1) ? (int)d : kBins - 1;
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ u64 ld_dsmem_u64(uint32_t addr) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_dsmem_u64(uint32_t addr, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

struct Shared {
    ExpTable tb;
    union {
        u64 hist[2][kBins];
        struct {                   // the candidates of the whole row, by id (one CTA's)
            float z[kSmall];
            uint32_t id[kSmall];
            u64 cum[kSmall];       // weights by rank, then their running sum
        } g;
    };
    u64 xch[8][kMaxCluster];       // values of the cluster's CTAs, one line per exchange
    u64 warp[kWarps], warp2[kWarps];
    u64 found_before, found_val;
    int found_bin, cnt[kWarps];
};

// One row's state, the same in every thread of the cluster except the slice.
struct Row {
    Shared *sh;
    float *z;                      // this CTA's slice
    unsigned short *list;          // kept candidates of warp w from w * chunk on
    float top;
    int n, chunk, cs, rank;        // slice length, tokens of a warp, cluster size and rank
    bool listed;                   // candidates in list (else every finite token of the slice)
    int level;                     // radix levels so far (histogram buffer parity)
};

// Each CTA's value for exchange line x, visible to all of the cluster after the sync.
__device__ __forceinline__ void exchange(const Row &r, int x, u64 v) {
    if (threadIdx.x < (unsigned)r.cs)
        st_dsmem_u64(mapa_shared(smem_u32(&r.sh->xch[x][r.rank]), threadIdx.x), v);
    cluster_sync_all();
}

// Sum of one value per warp (lane 0's) over the CTA, in every thread.
__device__ __forceinline__ u64 block_sum(const Row &r, u64 v) {
    const int warp = threadIdx.x >> 5;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) r.sh->warp[warp] = v;
    __syncthreads();
    u64 s = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += r.sh->warp[w];
    return s;
}

// Inclusive running sum over the CTA's threads, and the total.
__device__ __forceinline__ u64 block_scan_u64(const Row &r, u64 v, u64 &total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    u64 x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) r.sh->warp[warp] = x;
    __syncthreads();
    u64 before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const u64 y = r.sh->warp[w];
        before += w < warp ? y : 0;
        all += y;
    }
    total = all;
    return before + x;
}

// Calls f(index in the slice, valid) for the warp's candidates in index order, 32 at a time.
template <class F>
__device__ __forceinline__ void each(const Row &r, F &&f) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int base = warp * r.chunk;
    const int m = r.listed ? r.sh->cnt[warp] : max(0, min(r.chunk, r.n - base));
    for (int i = 0; i < m; i += 32) {
        const bool ok = i + lane < m;
        f(ok ? (r.listed ? (int)r.list[base + i + lane] : base + i + lane) : 0, ok);
    }
}

// The bin of the cluster's histogram h where the running sum from `acc` on reaches target (-1:
// nowhere); the sum before it and its own value.
__device__ int crossing(const Row &r, const u64 *h, u64 acc, u64 target, u64 &before, u64 &val) {
    Shared &sh = *r.sh;
    u64 a = 0;
    const uint32_t la = smem_u32(&h[threadIdx.x]);
    for (int c = 0; c < r.cs; ++c) a += ld_dsmem_u64(mapa_shared(la, (uint32_t)c));
    if (threadIdx.x == 0) sh.found_bin = -1;
    u64 total;
    const u64 upto = acc + block_scan_u64(r, a, total);
    if (upto >= target && upto - a < target) {
        sh.found_bin = threadIdx.x;
        sh.found_before = upto - a;
        sh.found_val = a;
    }
    __syncthreads();
    const int bin = sh.found_bin;
    if (bin >= 0) {
        before = sh.found_before;
        val = sh.found_val;
    }
    __syncthreads();
    return bin;
}

// Zeroes the next histogram of the two (the other may still be read by the cluster).
__device__ __forceinline__ u64 *next_hist(Row &r) {
    u64 *h = r.sh->hist[r.level & 1];
    ++r.level;
    h[threadIdx.x] = 0;
    __syncthreads();
    return h;
}

// The end of a prefix of the order: keys above `key` are in, and of those equal to it the
// first `ties` in id order.
struct Cut {
    uint32_t key;
    u64 ties;
};

constexpr u64 kAllTies = ~0ull;

// Descends to the place where the running sum over the order (of 1 per candidate, or of its
// weight with kMass) reaches `target`; everything when it never does.
template <bool kMass>
__device__ Cut descend(Row &r, u64 target) {
    Shared &sh = *r.sh;
    uint32_t klo = 0, khi = order_key(r.top);
    int bin0 = -1;                 // the distance bin that is being narrowed (-1: first level)
    int shift = 0;
    u64 acc = 0;                   // before the bin
    for (;;) {
        u64 *h = next_hist(r);
        if (bin0 >= 0) {
            const uint32_t range = khi - klo;
            shift = range < kBins ? 0 : 23 - __clz(range);   // range >> shift < kBins
        }
        each(r, [&](int i, bool ok) {
            const float z = r.z[i];
            if (!ok || z == -INFINITY) return;
            int bin = distance_bin(r.top, z);
            if (bin0 >= 0) {
                const uint32_t k = order_key(z);
                if (bin != bin0 || k < klo || k > khi) return;
                bin = (int)((khi - k) >> shift);
            }
            const u64 v = kMass ? weight44(r.top, z, sh.tb) : 1ull;
            if (v) atomicAdd(&h[bin], v);
        });
        cluster_sync_all();
        u64 val;
        const int bin = crossing(r, h, acc, target, acc, val);
        if (bin < 0) return Cut{0, kAllTies};   // never reached: everything stays
        if (bin0 < 0) {
            // the keys of the bin, with room for the rounding of its borders
            bin0 = bin;
            if (bin < kBins - 1 && r.top < INFINITY) {
                const float zl = r.top - (float)(bin + 1) / kBinsPerUnit;
                klo = order_key(zl - fabsf(zl) * 1e-6f - fabsf(r.top) * 1e-6f - 1e-6f);
                if (bin > 0) {
                    const float zh = r.top - (float)bin / kBinsPerUnit;
                    const uint32_t k = order_key(zh + fabsf(zh) * 1e-6f + fabsf(r.top) * 1e-6f + 1e-6f);
                    if (k < khi) khi = k;
                }
            }
        } else {
            const uint32_t h1 = khi - ((uint32_t)bin << shift);
            const uint32_t l1 = h1 - ((1u << shift) - 1u);
            khi = h1;
            klo = l1 > klo && l1 <= h1 ? l1 : klo;
            if (!kMass && acc + val == target) return Cut{klo, kAllTies};   // the bin goes in whole
        }
        if (khi == klo) {   // one value: its ties in id order
            if (kMass) {
                const u64 w = weight44(r.top, key_value(khi), sh.tb);
                return Cut{khi, (target - acc + w - 1) / w};
            }
            return Cut{khi, target - acc};
        }
    }
}

// Keeps the candidates inside the cut (and of at least `floor44` weight) as the new list.
__device__ void keep(Row &r, const Cut &cut, u64 floor44, int x) {
    Shared &sh = *r.sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned below = (1u << lane) - 1u;
    u64 tie0 = 0;
    if (cut.ties != kAllTies) {   // ids of equal values before this warp's
        u64 c = 0;
        each(r, [&](int i, bool ok) {
            const float z = r.z[i];
            c += __popc(__ballot_sync(0xffffffffu, ok && z != -INFINITY && order_key(z) == cut.key));
        });
        __syncthreads();
        if (lane == 0) sh.warp2[warp] = c;
        const u64 mine = block_sum(r, c);
        exchange(r, x, mine);
        for (int k = 0; k < r.rank; ++k) tie0 += sh.xch[x][k];
        for (int w = 0; w < warp; ++w) tie0 += sh.warp2[w];
    }
    int kept = 0;
    const int base = warp * r.chunk;
    each(r, [&](int i, bool ok) {
        const float z = r.z[i];
        const uint32_t k = order_key(z);
        ok = ok && z != -INFINITY;
        const bool tie = ok && k == cut.key;
        const unsigned tm = __ballot_sync(0xffffffffu, tie);
        bool in = ok && (k > cut.key || (tie && (cut.ties == kAllTies || tie0 + __popc(tm & below) < cut.ties)));
        tie0 += __popc(tm);
        if (in && floor44) in = z == r.top || weight44(r.top, z, sh.tb) >= floor44;
        const unsigned im = __ballot_sync(0xffffffffu, in);
        if (in) r.list[base + kept + __popc(im & below)] = (unsigned short)i;   // never ahead of the reading
        kept += __popc(im);
        __syncwarp();
    });
    __syncwarp();
    if (lane == 0) sh.cnt[warp] = kept;
    r.listed = true;
    __syncthreads();
}

// Keeps the candidates that pred(z) holds for as the new list; returns the CTA's number.
template <class P>
__device__ u64 keep_if(Row &r, P &&pred) {
    Shared &sh = *r.sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int base = warp * r.chunk;
    int kept = 0;
    each(r, [&](int i, bool ok) {
        const float z = r.z[i];
        const bool in = ok && z != -INFINITY && pred(z);
        const unsigned im = __ballot_sync(0xffffffffu, in);
        if (in) r.list[base + kept + __popc(im & ((1u << lane) - 1u))] = (unsigned short)i;
        kept += __popc(im);
        __syncwarp();
    });
    __syncwarp();
    if (lane == 0) sh.cnt[warp] = kept;
    r.listed = true;
    return block_sum(r, (u64)kept);
}

// Weight of the CTA's candidates; sh.warp2[w] = warp w's.
__device__ u64 mass(Row &r) {
    Shared &sh = *r.sh;
    u64 s = 0;
    each(r, [&](int i, bool ok) {
        const float z = r.z[i];
        if (ok && z != -INFINITY) s += weight44(r.top, z, sh.tb);
    });
    s = warp_sum(s);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh.warp2[threadIdx.x >> 5] = s;
    return block_sum(r, s);
}

struct Filters {
    u64 k;          // 0: off
    float p;        // >= 1: off
    u64 floor44;    // 0: off
};

__device__ __forceinline__ u64 mass_target(float p, u64 total) {   // tokens with less before them stay
    const double t = ceil((double)p * (double)total);
    return t >= 1.0 ? (u64)t : 1ull;
}
__device__ __forceinline__ u64 drawn(float u, u64 total) {         // u * total, below total
    const u64 t = u > 0.f ? (u64)((double)(u < 1.f ? u : 1.f) * (double)total) : 0;
    return t < total ? t : total - 1;
}

__device__ __forceinline__ void answer(const SampleArgs &a, const Row &r, int row, int id, float z, u64 total) {
    a.token[row] = id;
    // (its weight anew: a rare token's has few of the fixed point's bits)
    const double w = z == r.top ? 1.0 : exp((double)z - (double)r.top);
    a.prob[row] = (float)(w * 17592186044416.0 / (double)total);   // 2^44
}

// All filters and the draw over at most kSmall candidates, gathered by id in CTA 0's shared
// memory: each thread ranks one by counting.  total: the mass that top-p refers to without
// top-k.
__device__ void finish_small(const SampleArgs &a, const Row &r, int row, int n, const Filters &f, u64 total) {
    Shared &sh = *r.sh;
    const int e = threadIdx.x;
    const float z = e < n ? sh.g.z[e] : -INFINITY;
    int rank = 0;
    for (int j = 0; j < n; ++j) {
        const float y = sh.g.z[j];
        rank += y > z || (y == z && j < e);
    }
    const u64 w = e < n ? weight44(r.top, z, sh.tb) : 0;
    if (e < n) sh.g.cum[rank] = w;
    __syncthreads();
    u64 all;
    const u64 wr = e < n ? sh.g.cum[e] : 0;
    const u64 upto = block_scan_u64(r, wr, all);
    if (e < n) sh.g.cum[e] = upto;
    __syncthreads();
    const bool byk = f.k > 0;
    if (byk) total = sh.g.cum[(f.k < (u64)n ? (int)f.k : n) - 1];
    bool in = e < n && (!byk || (u64)rank < f.k);
    if (in && f.p < 1.f) in = sh.g.cum[rank] - w < mass_target(f.p, total);
    if (in && f.floor44) in = rank == 0 || w >= f.floor44;
    u64 kept;
    const u64 run = block_scan_u64(r, in ? w : 0, kept);
    const u64 t = drawn(a.u[row], kept);
    if (in && run > t && run - w <= t) answer(a, r, row, (int)sh.g.id[e], z, kept);
}

// Loads the slice as scaled fp32 logits; returns (ordered key of the thread's maximum, then
// the complement of its id).
template <class TL>
__device__ __forceinline__ u64 load_slice(const TL *l, int n, int v0, float inv, float *z) {
    constexpr int E = 16 / sizeof(TL), U = 4;
    u64 best = 0;
    auto put = [&](int i, float x) {
        x = x * inv + 0.f;               // + 0: -0 counts as 0
        if (x != x) x = -INFINITY;       // a NaN logit is never drawn
        z[i] = x;
        const u64 k = ((u64)order_key(x) << 32) | (uint32_t)~(uint32_t)(v0 + i);
        best = k > best ? k : best;
    };
    const int tid = threadIdx.x;
    // up to the first 16-byte boundary, then 16-byte loads, several in flight
    const int mis = (int)((reinterpret_cast<uintptr_t>(l) & 15) / sizeof(TL));
    const int head = min(n, mis ? E - mis : 0);
    if (tid < head) put(tid, to_f32<TL>(l[tid]));
    const int nv = (n - head) / E;
    const uint4 *lv = reinterpret_cast<const uint4 *>(l + head);
    for (int i0 = tid; i0 < nv; i0 += U * kThreads) {
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * kThreads < nv) x[u] = lv[i0 + u * kThreads];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u * kThreads >= nv) break;
            const int at = head + (i0 + u * kThreads) * E;
            const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (sizeof(TL) == 4) {
                    put(at + q, __uint_as_float(w[q]));
                } else {
                    put(at + 2 * q, __uint_as_float(w[q] << 16));
                    put(at + 2 * q + 1, __uint_as_float(w[q] & 0xffff0000u));
                }
            }
        }
    }
    const int tail = head + nv * E + tid;
    if (tail < n) put(tail, to_f32<TL>(l[tail]));
    return best;
}

template <class TL>
__global__ void __launch_bounds__(kThreads, 2) k_sample(const SampleArgs a, int slice) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Shared &sh = *reinterpret_cast<Shared *>(smem_raw);
    Row r;
    r.sh = &sh;
    r.z = reinterpret_cast<float *>(smem_raw + sizeof(Shared));
    r.list = reinterpret_cast<unsigned short *>(r.z + slice);
    r.cs = gridDim.z;
    r.rank = blockIdx.z;
    r.chunk = slice / kWarps;
    r.listed = false;
    r.level = 0;
    const int row = blockIdx.x, b = row / a.M, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int v0 = min(a.V, r.rank * slice);
    r.n = min(slice, a.V - v0);
    cluster_arrive();     // (waited for before the first write into another CTA)
    if (tid < 64) {
        const double t = exp2(-(double)tid / 64.0);
        sh.tb.fix[tid] = (u64)llrint(t * 1152921504606846976.0);   // 2^60
        sh.tb.hi[tid] = (float)t;
        sh.tb.lo[tid] = (float)(t - (double)(float)t);
    }
    griddep_wait();
    griddep_launch();
    const bool off = a.valid && !a.valid[row];   // the same in the whole cluster
    const float temp = a.temperature ? a.temperature[b] : 1.f;
    const bool greedy = !(temp > 0.f);
    const float inv = greedy ? 1.f : 1.0f / temp;
    u64 best = off ? 0 : load_slice<TL>(static_cast<const TL *>(a.logits) + (size_t)row * a.V + v0, r.n, v0, inv, r.z);
    const uint32_t mine_key = (uint32_t)(best >> 32);   // the thread's own maximum
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const u64 y = __shfl_xor_sync(0xffffffffu, best, o);
        best = y > best ? y : best;
    }
    if (lane == 0) sh.warp[warp] = best;
    cluster_wait();
    __syncthreads();
    if (off) {
        if (r.rank == 0 && tid == 0) {
            a.token[row] = -1;
            a.prob[row] = 0.f;
        }
        return;
    }
#pragma unroll
    for (int w = 0; w < kWarps; ++w) best = sh.warp[w] > best ? sh.warp[w] : best;
    exchange(r, 0, best);
    for (int c = 0; c < r.cs; ++c) best = sh.xch[0][c] > best ? sh.xch[0][c] : best;
    r.top = key_value((uint32_t)(best >> 32));
    if (greedy || r.top == -INFINITY || best == 0) {
        if (r.rank == 0 && tid == 0) {
            const bool none = r.top == -INFINITY || best == 0;
            a.token[row] = none ? -1 : (int)~(uint32_t)best;
            a.prob[row] = none ? 0.f : 1.f;
        }
        return;           // (no other CTA touches this one's memory any more)
    }
    const u64 one = 1ull << 44;
    const int k = a.top_k ? a.top_k[b] : 0;
    const float mp = a.min_p ? a.min_p[b] : 0.f;
    Filters f;
    f.k = k > 0 && k < a.V ? (u64)k : 0;
    f.p = a.top_p ? a.top_p[b] : 1.f;
    if (!(f.p < 1.f)) f.p = 1.f;
    f.floor44 = mp > 0.f ? (mp < 1.f ? (u64)ceil((double)mp * (double)one) : one) : 0;

    u64 total = 0;        // mass of the row (what top-p refers to without top-k)
    u64 found = 0;        // this CTA's candidates, once listed
    bool any = false;     // a filter that shortens the list is on
    if (f.k) {
        // The k largest of the threads' maxima are k tokens, so the k-th token is not below
        // the k-th maximum: the bins up to that one's hold the top k.
        u64 *h = next_hist(r);
        if (mine_key > order_key(-INFINITY)) atomicAdd(&h[distance_bin(r.top, key_value(mine_key))], 1ull);
        cluster_sync_all();
        u64 before, val;
        const int bin = crossing(r, h, 0, f.k, before, val);
        if (bin >= 0 && bin < kBins - 1) {
            found = keep_if(r, [&](float z) { return distance_bin(r.top, z) <= bin; });
            any = true;
        }
    } else if (f.p < 1.f) {
        // Tokens below (1 - p) / V of the largest cannot be needed: V of them and everything
        // after them weigh less than (1 - p) of the total.  The mass per bin of the others
        // says which bin the cut falls into.
        const float far = -logf(fmaxf((1.f - f.p) / (float)a.V, 1e-30f)) + 0.25f;
        u64 *h = next_hist(r);
        u64 s = 0;
        each(r, [&](int i, bool ok) {
            const float z = r.z[i];
            if (!ok || z == -INFINITY) return;
            const u64 w = weight44(r.top, z, sh.tb);
            s += w;
            if (w && (z == r.top || r.top - z < far)) atomicAdd(&h[distance_bin(r.top, z)], w);
        });
        exchange(r, 1, block_sum(r, warp_sum(s)));
        for (int c = 0; c < r.cs; ++c) total += sh.xch[1][c];
        u64 before, val;
        const int bin = crossing(r, h, 0, mass_target(f.p, total), before, val);
        if (bin >= 0 && bin < kBins - 1) {
            found = keep_if(r, [&](float z) { return distance_bin(r.top, z) <= bin; });
            any = true;
        }
    } else if (f.floor44) {
        const float far = -logf(fmaxf(mp, 1e-30f)) * 1.0001f + 1e-3f;
        found = keep_if(r, [&](float z) { return z == r.top || r.top - z < far; });
        any = true;
    }
    if (any) {
        exchange(r, 2, found);
        u64 n = 0, before = 0;
        for (int c = 0; c < r.cs; ++c) {
            if (c < r.rank) before += sh.xch[2][c];
            n += sh.xch[2][c];
        }
        if (n <= kSmall) {
            // gather in id order in CTA 0 (the histograms have been read: exchange 2 came after)
            int at = (int)before;
            for (int w = 0; w < warp; ++w) at += sh.cnt[w];
            for (int i = lane; i < sh.cnt[warp]; i += 32) {
                const int x = r.list[warp * r.chunk + i];
                st_dsmem_f32(mapa_shared(smem_u32(&sh.g.z[at + i]), 0), r.z[x]);
                st_dsmem_f32(mapa_shared(smem_u32(&sh.g.id[at + i]), 0), __uint_as_float((uint32_t)(v0 + x)));
            }
            cluster_sync_all();
            if (r.rank == 0) finish_small(a, r, row, (int)n, f, total);
            return;
        }
    }
    // many candidates: the cuts by descent over the bins' keys
    if (f.k) keep(r, descend<false>(r, f.k), 0, 3);
    if (f.p < 1.f) {
        if (f.k) {
            exchange(r, 4, mass(r));
            for (int c = 0; c < r.cs; ++c) total += sh.xch[4][c];
        }
        keep(r, descend<true>(r, mass_target(f.p, total)), f.floor44, 5);
    } else if (f.floor44) {
        keep(r, Cut{0, kAllTies}, f.floor44, 5);
    }
    // draw
    const u64 mine = mass(r);
    exchange(r, 6, mine);
    u64 before = 0;
    total = 0;
    for (int c = 0; c < r.cs; ++c) {
        if (c < r.rank) before += sh.xch[6][c];
        total += sh.xch[6][c];
    }
    const u64 target = drawn(a.u[row], total);
    if (target >= before && target < before + mine) {   // one CTA of the cluster
        int w = 0;
        u64 at = before;
        while (target >= at + sh.warp2[w]) at += sh.warp2[w++];
        // warp w's candidates, a part for each warp of the CTA
        const int m = r.listed ? sh.cnt[w] : min(r.chunk, r.n - w * r.chunk);
        const int part = ((m + kWarps - 1) / kWarps + 31) / 32 * 32;
        const int i0 = warp * part, i1 = min(m, i0 + part);
        auto item = [&](int i) { return r.listed ? (int)r.list[w * r.chunk + i] : w * r.chunk + i; };
        auto weight = [&](int i) -> u64 {
            if (i >= i1) return 0;
            const float z = r.z[item(i)];
            return z == -INFINITY ? 0 : weight44(r.top, z, sh.tb);
        };
        u64 s = 0;
        for (int i = i0; i < i1; i += 32) s += weight(i + lane);
        s = warp_sum(s);
        __syncthreads();
        if (lane == 0) sh.warp[warp] = s;
        __syncthreads();
        for (int p = 0; p < warp; ++p) at += sh.warp[p];
        if (target >= at && target < at + s) {
            for (int i = i0; i < i1; i += 32) {
                const u64 wt = weight(i + lane);
                u64 x = wt;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const u64 y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o) x += y;
                }
                if (at + x > target && at + x - wt <= target) {
                    const int j = item(i + lane);
                    answer(a, r, row, v0 + j, r.z[j], total);
                }
                at += __shfl_sync(0xffffffffu, x, 31);
            }
        }
    }
    cluster_sync_all();   // nobody leaves while its histograms may still be read
}

}  // namespace

int sample_max_vocab() { return kMaxCluster * kSlice; }

cudaError_t sample_tokens(const SampleArgs &a, int dtype, cudaStream_t st) {
    if (a.rows <= 0) return cudaSuccess;
    int cs = 1;
    while (cs < kMaxCluster && (a.V + cs - 1) / cs > kSlice) cs *= 2;
    int slice = (a.V + cs - 1) / cs;
    slice = (slice + kThreads - 1) / kThreads * kThreads;   // whole 32-token steps for every warp
    const size_t smem = sizeof(Shared) + (size_t)slice * 6;
    static bool configured[64] = {};   // per device: shared-memory limit, clusters of 16
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        const int most = (int)(sizeof(Shared) + (size_t)kSlice * 6);
        for (auto kern : {reinterpret_cast<const void *>(k_sample<float>), reinterpret_cast<const void *>(k_sample<bf16>)}) {
            cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
            if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
        }
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    auto kern = dtype == DLLM_BF16 ? k_sample<bf16> : k_sample<float>;
    return launch_kernel(kern, dim3(a.rows, 1, cs), dim3(kThreads), smem, st, cs, a, slice);
}

}  // namespace dllm
