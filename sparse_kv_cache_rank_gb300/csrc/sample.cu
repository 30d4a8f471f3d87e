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
// can move a border.  Weights above 2^-20 of the largest are formed to 2^-36 of themselves
// (weight44): an fp32 exponential's 2^-23 would move the running sums across the border of
// a neighbouring token once in a few hundred rows of a large vocabulary.  Below, the fp32
// exponential is as good: its error is 2^-43 of the largest weight.
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
constexpr double kC1 = (double)(long long)(kLn2_64 * 262144.0) / 262144.0;   // its first 12 bits
constexpr float kHeavy = 14.f;     // distance to the maximum up to which weights are formed in full

struct ExpTable {                  // 2^(-j/64)
    u64 fix[64];                   // in units of 2^-44
    int t31[64];                   // in units of 2^-31
};

constexpr double exp_series(double x) {   // |x| < 0.7: the remainder after 24 terms is below 2^-80
    double s = 1.0;
    for (int k = 24; k > 0; --k) s = 1.0 + s * x / k;
    return s;
}
constexpr ExpTable make_table() {
    ExpTable t{};
    for (int j = 0; j < 64; ++j) {
        const double e = exp_series(-j * kLn2_64);
        t.fix[j] = (u64)(e * 17592186044416.0 + 0.5);
        const double x = e * 2147483648.0 + 0.5;
        t.t31[j] = x >= 2147483647.0 ? 2147483647 : (int)x;
    }
    return t;
}
__constant__ const ExpTable c_table = make_table();

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// exp(-(top - z)) in units of 2^-44 for a distance of kHeavy on: the fp32 exponential.
__device__ __forceinline__ uint32_t weight44_light(float top, float z) {
    const float d = top - z, bb = d - top;
    const float dl = (top - (d - bb)) - (z + bb);   // top - z = d + dl exactly
    const float e = expf(-d);
    return __float2uint_rn(fmaf(-e, dl, e) * 17592186044416.f);
}

// exp(-(top - z)) in units of 2^-44, off by at most 2^-36 relative (and half a unit).
// With n = round(64 d / ln 2) and n = 64 k + j:  exp(-d) = 2^-k 2^(-j/64) exp(-r), where
// r = d - n ln2/64 lies within ln2/128.  d - n C1 is exact in fp32; it, n (ln2/64 - C1) and the
// rounding of d are then added in units of 2^-38, and exp(-r) - 1 = -r + (r^2/2 - r^3/6 + r^4/24)
// needs fp32 in its second part alone.
__device__ __forceinline__ u64 weight44(float top, float z, const ExpTable &tb) {
    if (z == top) return 1ull << 44;   // also for an infinite maximum
    const float d = top - z;
    if (!(d < kHeavy)) return weight44_light(top, z);
    constexpr float kUnit = 274877906944.f;   // 2^38
    const float bb = d - top;
    const float dl = (top - (d - bb)) - (z + bb);
    const float t = fmaf(d, (float)(1.0 / kLn2_64), 12582912.f);   // its low bits: the rounded product
    const int n = __float_as_int(t) - 0x4B400000;
    const float r1 = fmaf(-(t - 12582912.f), (float)kC1, d);
    constexpr uint32_t kRest = (uint32_t)((kLn2_64 - kC1) * 1125899906842624.0 + 0.5);   // 2^50
    const int r = __float2int_rn(r1 * kUnit) - (int)__umulhi((uint32_t)n << 20, kRest) + __float2int_rn(dl * kUnit);
    const float rf = (float)r * (1.0f / kUnit);
    const float s = rf * rf * fmaf(rf, fmaf(rf, kUnit / 24.f, -kUnit / 6.f), kUnit * 0.5f);
    const int e = __float2int_rn(s) - r;      // exp(-r) - 1
    const int j = n & 63, k = n >> 6;
    const u64 w = tb.fix[j] + (u64)(((long long)e * tb.t31[j]) >> 25);
    return (w + ((1ull << k) >> 1)) >> k;
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

struct alignas(16) Shared {
    ExpTable tb;
    union {
        u64 hist[2][kBins];
        struct {                   // the candidates of the whole row, by id (one CTA's)
            float z[kSmall];
            uint32_t id[kSmall];
            u64 cum[kSmall];       // weights by rank, then their running sum
        } g;
    };
    u64 bins[kBins];               // a histogram summed over the cluster
    u64 xch[8][kMaxCluster];       // values of the cluster's CTAs, one line per exchange
    u64 warp[kWarps], warp2[kWarps];
    u64 found_before, found_val, cut[2];
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
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) r.sh->warp[warp] = v;
    __syncthreads();
    return warp_sum(lane < kWarps ? r.sh->warp[lane] : 0);
}

// Sum of exchange line x over the cluster, and over the CTAs before this one.
__device__ __forceinline__ u64 line_sum(const Row &r, int x, u64 &before) {
    const int lane = threadIdx.x & 31;
    const u64 v = lane < r.cs ? r.sh->xch[x][lane] : 0;
    before = warp_sum(lane < r.rank ? v : 0);
    return warp_sum(v);
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
    const u64 y = lane < kWarps ? r.sh->warp[lane] : 0;
    total = warp_sum(y);
    return warp_sum(lane < warp ? y : 0) + x;
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
    // Each CTA adds up its share of the bins (a bin's parts in neighbouring lanes) and hands the
    // sums to all: one remote load and one remote store per thread.
    const int cs = r.cs, c = threadIdx.x & (cs - 1);
    const int own = r.rank * (kBins / cs) + threadIdx.x / cs;
    u64 a = ld_dsmem_u64(mapa_shared(smem_u32(&h[own]), (uint32_t)c));
    for (int o = cs >> 1; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    st_dsmem_u64(mapa_shared(smem_u32(&sh.bins[own]), (uint32_t)c), a);
    cluster_sync_all();
    a = sh.bins[threadIdx.x];
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

// Adds to a bin whose sum within the CTA stays below 2^32.
__device__ __forceinline__ void add32(u64 *bin, uint32_t v) { atomicAdd(reinterpret_cast<unsigned *>(bin), v); }

// Adds a mass: two 32-bit atomics with the carry between them (shared memory has no native 64-bit
// add); the high half of a CTA's sum stays below 2^32.
__device__ __forceinline__ void add64(u64 *bin, u64 v) {
    unsigned *p = reinterpret_cast<unsigned *>(bin);
    const unsigned lo = (unsigned)v;
    const unsigned old = atomicAdd(p, lo);
    const unsigned hi = (unsigned)(v >> 32) + (old + lo < lo ? 1u : 0u);
    if (hi) atomicAdd(p + 1, hi);
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
            if (kMass) {
                const u64 v = weight44(r.top, z, sh.tb);
                if (v) add64(&h[bin], v);
            } else {
                add32(&h[bin], 1);
            }
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

// The cut inside distance bin `bin`, whose members (at most kSmall in the cluster, `before` of
// them in the CTAs before this one) one CTA gathers and ranks: the running sum starts at
// acc and the cut is where it reaches target.
template <bool kMass>
__device__ Cut rank_bin(Row &r, int bin, int before, int n, u64 acc, u64 target) {
    Shared &sh = *r.sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = threadIdx.x;
    // members of the CTA's warps, then their places
    int c = 0;
    each(r, [&](int i, bool ok) {
        const float z = r.z[i];
        c += __popc(__ballot_sync(0xffffffffu, ok && z != -INFINITY && distance_bin(r.top, z) == bin));
    });
    __syncthreads();
    if (lane == 0) sh.warp[warp] = (u64)c;
    __syncthreads();
    int at = before + (int)warp_sum(lane < warp ? sh.warp[lane < kWarps ? lane : 0] : 0);
    each(r, [&](int i, bool ok) {
        const float z = r.z[i];
        const bool in = ok && z != -INFINITY && distance_bin(r.top, z) == bin;
        const unsigned m = __ballot_sync(0xffffffffu, in);
        if (in) st_dsmem_f32(mapa_shared(smem_u32(&sh.g.z[at + __popc(m & ((1u << lane) - 1u))]), 0), z);
        at += __popc(m);
    });
    cluster_sync_all();
    if (r.rank == 0) {
        const float z = e < n ? sh.g.z[e] : -INFINITY;
        int rank = 0, tie = 0, ties = 0;
        if (warp * 32 < n)
            for (int j = 0; j < n; ++j) {
                const float y = sh.g.z[j];
                rank += y > z;
                ties += y == z;
                tie += y == z && j < e;
            }
        rank += tie;
        const u64 w = e < n ? (kMass ? weight44(r.top, z, sh.tb) : 1ull) : 0;
        if (e < n) sh.g.cum[rank] = w;
        __syncthreads();
        u64 all;
        const u64 upto = block_scan_u64(r, e < n ? sh.g.cum[e] : 0, all);
        if (e < n) sh.g.cum[e] = upto;
        __syncthreads();
        // (the bin holds the crossing, so one member is it)
        if (e < n && acc + sh.g.cum[rank] >= target && acc + sh.g.cum[rank] - w < target)
            for (int k = 0; k < r.cs; ++k) {
                st_dsmem_u64(mapa_shared(smem_u32(&sh.cut[0]), (uint32_t)k), order_key(z));
                st_dsmem_u64(mapa_shared(smem_u32(&sh.cut[1]), (uint32_t)k), tie + 1 < ties ? (u64)(tie + 1) : kAllTies);
            }
    }
    cluster_sync_all();
    return Cut{(uint32_t)sh.cut[0], sh.cut[1]};
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
        line_sum(r, x, tie0);
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

// Lists the tokens nearer to the maximum than `far` (>= kHeavy) and returns the weight of all of
// the CTA's, listed or not (sh.warp2[w] = warp w's); f(z, weight) for the listed ones.  The
// few cheap operations per token come first, the full exponential runs over the dense list.
template <class F>
__device__ u64 list_near(Row &r, float far, F &&f) {
    Shared &sh = *r.sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int base = warp * r.chunk, m = max(0, min(r.chunk, r.n - base));
    int kept = 0;
    u64 s = 0;
    for (int i = lane; i < (m + 31) / 32 * 32; i += 32) {
        const float z = i < m ? r.z[base + i] : -INFINITY;
        const bool in = z == r.top || r.top - z < far;
        if (!in) s += weight44_light(r.top, z);      // 0 for -inf
        const unsigned im = __ballot_sync(0xffffffffu, in);
        if (in) r.list[base + kept + __popc(im & ((1u << lane) - 1u))] = (unsigned short)(base + i);
        kept += __popc(im);
    }
    __syncwarp();
    for (int i = lane; i < kept; i += 32) {
        const float z = r.z[r.list[base + i]];
        const u64 w = weight44(r.top, z, sh.tb);
        s += w;
        f(z, w);
    }
    s = warp_sum(s);
    __syncthreads();
    if (lane == 0) {
        sh.cnt[warp] = kept;
        sh.warp2[warp] = s;
    }
    r.listed = true;
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

// Elements of the slice before its first 16-byte boundary.
template <class TL>
__device__ __forceinline__ int slice_head(const TL *l, int n) {
    constexpr int E = 16 / sizeof(TL);
    const int mis = (int)((reinterpret_cast<uintptr_t>(l) & 15) / sizeof(TL));
    return min(n, mis ? E - mis : 0);
}

// Loads the slice as scaled fp32 logits (z + head is 16-byte aligned); returns the thread's maximum.
template <class TL>
__device__ __forceinline__ float load_slice(const TL *l, int n, int head, float inv, float *z) {
    constexpr int E = 16 / sizeof(TL), U = 8;
    float best = -INFINITY;
    auto scaled = [&](float x) {
        x = fmaxf(fmaf(x, inv, 0.f), -INFINITY);   // -0 counts as 0, a NaN logit is never drawn
        best = fmaxf(best, x);
        return x;
    };
    const int tid = threadIdx.x;
    if (tid < head) z[tid] = scaled(to_f32<TL>(l[tid]));
    const int nv = (n - head) / E;
    const uint4 *lv = reinterpret_cast<const uint4 *>(l + head);
    float4 *zv = reinterpret_cast<float4 *>(z + head);
    for (int i0 = tid; i0 < nv; i0 += U * kThreads) {   // 16-byte loads, several in flight
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * kThreads < nv) x[u] = lv[i0 + u * kThreads];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kThreads;
            if (i >= nv) break;
            const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
            float y[E];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (sizeof(TL) == 4) {
                    y[q] = scaled(__uint_as_float(w[q]));
                } else {
                    y[(2 * q) % E] = scaled(__uint_as_float(w[q] << 16));
                    y[(2 * q + 1) % E] = scaled(__uint_as_float(w[q] & 0xffff0000u));
                }
            }
#pragma unroll
            for (int q = 0; q < E / 4; ++q)
                zv[i * (E / 4) + q] = make_float4(y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]);
        }
    }
    const int tail = head + nv * E + tid;
    if (tail < n) z[tail] = scaled(to_f32<TL>(l[tail]));
    return best;
}

template <class TL>
__global__ void __launch_bounds__(kThreads, 2) k_sample(const SampleArgs a, int slice) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Shared &sh = *reinterpret_cast<Shared *>(smem_raw);
    Row r;
    r.sh = &sh;
    r.z = reinterpret_cast<float *>(smem_raw + sizeof(Shared));
    r.list = reinterpret_cast<unsigned short *>(r.z + slice + 4);   // (z may start up to 3 further)
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
        sh.tb.fix[tid] = c_table.fix[tid];
        sh.tb.t31[tid] = c_table.t31[tid];
    }
    griddep_wait();
    griddep_launch();
    const bool off = a.valid && !a.valid[row];   // the same in the whole cluster
    const float temp = a.temperature ? a.temperature[b] : 1.f;
    const bool greedy = !(temp > 0.f && 1.0f / temp < INFINITY);
    const float inv = greedy ? 1.f : 1.0f / temp;
    const TL *l = static_cast<const TL *>(a.logits) + (size_t)row * a.V + v0;
    const int head = slice_head(l, r.n);
    r.z += -head & 3;
    const float mine_max = off ? 0.f : load_slice(l, r.n, head, inv, r.z);
    float top = mine_max;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) sh.warp[warp] = __float_as_uint(top);
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
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, __uint_as_float((uint32_t)sh.warp[w]));
    exchange(r, 0, __float_as_uint(top));
    for (int c = 0; c < r.cs; ++c) top = fmaxf(top, __uint_as_float((uint32_t)sh.xch[0][c]));
    r.top = top;
    if (greedy || top == -INFINITY) {
        // the lowest id of the maximum: each CTA's first, the lowest CTA that has one
        int first = INT_MAX;
        if (top > -INFINITY)
            for (int i = tid; i < r.n; i += kThreads)
                if (r.z[i] == top) {
                    first = i;
                    break;
                }
        first = __reduce_min_sync(0xffffffffu, first);
        if (lane == 0) sh.cnt[warp] = first;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) first = min(first, sh.cnt[w]);
        exchange(r, 1, (u64)(uint32_t)first);
        if (r.rank == 0 && tid == 0) {
            int id = -1;
            for (int c = r.cs - 1; c >= 0; --c)
                if (sh.xch[1][c] != (u64)INT_MAX) id = c * slice + (int)sh.xch[1][c];
            a.token[row] = id;
            a.prob[row] = id < 0 ? 0.f : 1.f;
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
    int bin = -1;         // top-p without top-k: the distance bin of the cut,
    u64 acc = 0;          // the mass before it,
    int in_bin = 0, in_bin0 = 0;   // its members in the cluster and in the CTAs before this one
    if (f.k) {
        // The k largest of the threads' maxima are k tokens, so the k-th token is not below
        // the k-th maximum: the bins up to that one's hold the top k.
        u64 *h = next_hist(r);
        if (mine_max > -INFINITY) add32(&h[distance_bin(top, mine_max)], 1);
        cluster_sync_all();
        u64 before, val;
        const int most = crossing(r, h, 0, f.k, before, val);
        if (most >= 0 && most < kBins - 1) {
            found = keep_if(r, [&](float z) { return distance_bin(top, z) <= most; });
            any = true;
        }
    } else if (f.p < 1.f) {
        // Tokens below (1 - p) / V of the largest cannot be needed: V of them and everything
        // after them weigh less than (1 - p) of the total.  The others are listed (with all
        // whose weights are formed in full); their mass per bin says into which bin the cut falls.
        const float far = -logf(fmaxf((1.f - f.p) / (float)a.V, 1e-30f)) + 0.25f;
        u64 *h = next_hist(r);
        const u64 s = list_near(r, fmaxf(far, kHeavy), [&](float z, u64 w) {
            if (w) add64(&h[distance_bin(top, z)], w);
        });
        exchange(r, 1, s);
        u64 before, val;
        total = line_sum(r, 1, before);
        bin = crossing(r, h, 0, mass_target(f.p, total), acc, val);
        if (bin >= 0 && bin < kBins - 1) {
            u64 c = 0;
            found = keep_if(r, [&](float z) {
                const int d = distance_bin(top, z);
                c += d == bin;
                return d <= bin;
            });
            found |= block_sum(r, warp_sum(c)) << 32;
            any = true;
        }
    } else if (f.floor44) {
        const float far = -logf(fmaxf(mp, 1e-30f)) * 1.0001f + 1e-3f;
        found = keep_if(r, [&](float z) { return z == top || top - z < far; });
        any = true;
    }
    if (any) {
        exchange(r, 2, found);
        u64 before;
        const u64 sums = line_sum(r, 2, before);
        const uint32_t n = (uint32_t)sums;
        in_bin = (int)(sums >> 32);
        in_bin0 = (int)(before >> 32);
        if (n <= kSmall) {
            // gather in id order in CTA 0 (the histograms have been read: exchange 2 came after)
            int at = (int)(uint32_t)before;
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
            u64 before;
            total = line_sum(r, 4, before);
        }
        const u64 target = mass_target(f.p, total);
        keep(r, any && bin >= 0 && in_bin <= kSmall ? rank_bin<true>(r, bin, in_bin0, in_bin, acc, target)
                                                    : descend<true>(r, target),
             f.floor44, 5);
    } else if (f.floor44) {
        keep(r, Cut{0, kAllTies}, f.floor44, 5);
    }
    // draw
    u64 mine;
    if (r.listed) {
        mine = mass(r);
    } else {   // no filter shortened anything: every token
        mine = list_near(r, kHeavy, [](float, u64) {});
        r.listed = false;
    }
    exchange(r, 6, mine);
    u64 before;
    total = line_sum(r, 6, before);
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
    const size_t smem = sizeof(Shared) + 16 + (size_t)slice * 6;
    static bool configured[64] = {};   // per device: shared-memory limit, clusters of 16
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        const int most = (int)(sizeof(Shared) + 16 + (size_t)kSlice * 6);
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
