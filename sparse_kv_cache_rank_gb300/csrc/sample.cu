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
constexpr int kBins = 1024;
constexpr int kMaxCluster = 8;
constexpr int kSlice = 16384;      // tokens per CTA up to which a smaller cluster is taken
constexpr int kSliceMax = 32768;   // largest slice (192 KB of shared memory)
constexpr float kBinsPerUnit = 32.f;

// ---------------------------------------------------------------- exp in fixed point
constexpr double kLn2_64 = 0.69314718055994530942 / 64;
constexpr double kC1 = (double)(long long)(kLn2_64 * 262144.0) / 262144.0;                       // 12 bits
constexpr double kC2 = (double)(long long)((kLn2_64 - kC1) * 4294967296.0) / 4294967296.0;       // 11 bits
constexpr double kC3 = kLn2_64 - kC1 - kC2;

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
    u64 hist[2][kBins];
    u64 xch[8][kMaxCluster];       // values of the cluster's CTAs, one line per exchange
    u64 warp[kWarps], warp2[kWarps];
    u64 found_before;
    int found_bin, cnt[kWarps], ties[kWarps];
    u64 found_val;
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
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t klo = 0, khi = order_key(r.top);
    int bin0 = -1;                 // the distance bin that is being narrowed (-1: first level)
    int shift = 0;
    u64 acc = 0;                   // before the bin
    for (;;) {
        u64 *h = sh.hist[r.level & 1];
        ++r.level;
        for (int i = tid; i < kBins; i += kThreads) h[i] = 0;
        __syncthreads();
        if (bin0 >= 0) {
            const uint32_t range = khi - klo;
            shift = range < kBins ? 0 : 22 - __clz(range);   // range >> shift < kBins
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
        // bins 2 tid and 2 tid + 1 over the cluster, then where the running sum crosses
        u64 a0 = 0, a1 = 0;
        const uint32_t la = smem_u32(&h[2 * tid]);
        for (int c = 0; c < r.cs; ++c) {
            const uint32_t p = mapa_shared(la, (uint32_t)c);
            a0 += ld_dsmem_u64(p);
            a1 += ld_dsmem_u64(p + 8);
        }
        u64 x = a0 + a1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (tid == 0) sh.found_bin = -1;
        if (lane == 31) sh.warp2[warp] = x;
        __syncthreads();
        u64 before = acc;
        for (int w = 0; w < warp; ++w) before += sh.warp2[w];
        before += x - (a0 + a1);
        if (before < target && before + a0 >= target) {
            sh.found_bin = 2 * tid;
            sh.found_before = before;
            sh.found_val = a0;
        } else if (before + a0 < target && before + a0 + a1 >= target) {
            sh.found_bin = 2 * tid + 1;
            sh.found_before = before + a0;
            sh.found_val = a1;
        }
        __syncthreads();
        const int bin = sh.found_bin;
        const u64 val = sh.found_val;
        acc = bin >= 0 ? sh.found_before : acc;
        __syncthreads();
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
                const u64 w = weight44(r.top, __uint_as_float(khi & 0x80000000u ? khi & 0x7fffffffu : ~khi), sh.tb);
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

template <class TL>
__global__ void __launch_bounds__(kThreads) k_sample(const SampleArgs a, int slice) {
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
    if (tid < 64) {
        const double t = exp2(-(double)tid / 64.0);
        sh.tb.fix[tid] = (u64)llrint(t * 1152921504606846976.0);   // 2^60
        sh.tb.hi[tid] = (float)t;
        sh.tb.lo[tid] = (float)(t - (double)(float)t);
    }
    griddep_wait();
    griddep_launch();
    if (a.valid && !a.valid[row]) {   // the same in the whole cluster
        if (r.rank == 0 && tid == 0) {
            a.token[row] = -1;
            a.prob[row] = 0.f;
        }
        return;
    }
    const float temp = a.temperature ? a.temperature[b] : 1.f;
    const bool greedy = !(temp > 0.f);
    const float inv = greedy ? 1.f : 1.0f / temp;
    // load, scale, maximum (its lowest id)
    const TL *l = static_cast<const TL *>(a.logits) + (size_t)row * a.V + v0;
    u64 best = 0;   // ordered key of the maximum, then the complement of its id
    for (int i = tid; i < r.n; i += kThreads) {
        float z = to_f32<TL>(l[i]) * inv + 0.f;     // + 0: -0 counts as 0
        if (z != z) z = -INFINITY;                  // a NaN logit is never drawn
        r.z[i] = z;
        const u64 k = ((u64)order_key(z) << 32) | (uint32_t)~(uint32_t)(v0 + i);
        best = k > best ? k : best;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const u64 y = __shfl_xor_sync(0xffffffffu, best, o);
        best = y > best ? y : best;
    }
    if (lane == 0) sh.warp[warp] = best;
    cluster_sync_all();   // (the whole cluster runs: its shared memory may be written)
#pragma unroll
    for (int w = 0; w < kWarps; ++w) best = sh.warp[w] > best ? sh.warp[w] : best;
    exchange(r, 0, best);
    for (int c = 0; c < r.cs; ++c) best = sh.xch[0][c] > best ? sh.xch[0][c] : best;
    const uint32_t kt = (uint32_t)(best >> 32);
    r.top = __uint_as_float(kt & 0x80000000u ? kt & 0x7fffffffu : ~kt);
    if (greedy || r.top == -INFINITY) {
        if (r.rank == 0 && tid == 0) {
            const bool none = r.top == -INFINITY;
            a.token[row] = none ? -1 : (int)~(uint32_t)best;
            a.prob[row] = none ? 0.f : 1.f;
        }
        cluster_sync_all();   // nobody leaves while its exchange line may still be written
        return;
    }
    const int k = a.top_k ? a.top_k[b] : 0;
    const float tp = a.top_p ? a.top_p[b] : 1.f;
    const float mp = a.min_p ? a.min_p[b] : 0.f;
    const u64 one = 1ull << 44;
    const u64 floor44 = mp > 0.f ? (mp < 1.f ? (u64)ceil((double)mp * (double)one) : one) : 0;
    if (k > 0 && k < a.V) {
        const Cut c = descend<false>(r, (u64)k);
        keep(r, c, 0, 1);
    }
    if (tp < 1.f) {
        u64 total = 0;
        exchange(r, 2, mass(r));
        for (int c = 0; c < r.cs; ++c) total += sh.xch[2][c];
        const double t = ceil((double)tp * (double)total);
        const Cut c = descend<true>(r, t >= 1.0 ? (u64)t : 1ull);
        keep(r, c, floor44, 3);
    } else if (floor44) {
        keep(r, Cut{0, kAllTies}, floor44, 3);
    }
    // draw
    const u64 mine = mass(r);
    exchange(r, 4, mine);
    u64 total = 0, before = 0;
    for (int c = 0; c < r.cs; ++c) {
        if (c < r.rank) before += sh.xch[4][c];
        total += sh.xch[4][c];
    }
    const float u = a.u[row];
    u64 target = u > 0.f ? (u64)((double)(u < 1.f ? u : 1.f) * (double)total) : 0;
    if (target >= total) target = total - 1;
    if (target >= before && target < before + mine) {   // one CTA of the cluster
        int w = 0;
        u64 at = before;
        while (target >= at + sh.warp2[w]) at += sh.warp2[w++];
        if (warp == w) {
            bool done = false;
            each(r, [&](int i, bool ok) {
                if (done) return;
                const float z = r.z[i];
                const u64 wt = ok && z != -INFINITY ? weight44(r.top, z, sh.tb) : 0;
                u64 x = wt;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const u64 y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o) x += y;
                }
                const unsigned m = __ballot_sync(0xffffffffu, at + x > target);
                if (m) {
                    if (lane == __ffs(m) - 1) {
                        a.token[row] = v0 + i;
                        // (its weight anew: a rare token's has few of the fixed point's bits)
                        const double w = z == r.top ? 1.0 : exp((double)z - (double)r.top);
                        a.prob[row] = (float)(w * (double)one / (double)total);
                    }
                    done = true;
                }
                at += __shfl_sync(0xffffffffu, x, 31);
            });
        }
    }
    cluster_sync_all();   // nobody leaves while its histograms or lines may still be read or written
}

}  // namespace

int sample_max_vocab() { return kMaxCluster * kSliceMax; }

cudaError_t sample_tokens(const SampleArgs &a, int dtype, cudaStream_t st) {
    if (a.rows <= 0) return cudaSuccess;
    int cs = 1;
    while (cs < kMaxCluster && (a.V + cs - 1) / cs > kSlice) cs *= 2;
    int slice = (a.V + cs - 1) / cs;
    slice = (slice + kThreads - 1) / kThreads * kThreads;   // whole 32-token steps for every warp
    const size_t smem = sizeof(Shared) + (size_t)slice * 6;
    static bool configured[64] = {};   // per device: raise the shared-memory limit once
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        const int most = (int)(sizeof(Shared) + (size_t)kSliceMax * 6);
        cudaError_t e = cudaFuncSetAttribute(k_sample<float>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(k_sample<bf16>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    auto kern = dtype == DLLM_BF16 ? k_sample<bf16> : k_sample<float>;
    return launch_kernel(kern, dim3(a.rows, 1, cs), dim3(kThreads), smem, st, cs, a, slice);
}

}  // namespace dllm
