// sample.cu -- one token per row of logits from a given uniform number: temperature, top-k,
// top-p and min-p, then the inverse of the kept tokens' cumulative distribution.
//
//   z_v = fp32(l_v fp32(1 / T)),   w_v = exp(z_v - max z)
//   order: z descending, equal z by lower id.  Every filter keeps a prefix of that order:
//     top-k   the first k;   top-p  the tokens whose mass before them is < p (mass of the
//     first k);   min-p  the tokens with w >= min_p;   the first token always stays
//   token = the lowest kept id whose cumulative kept mass (in id order) exceeds u * total
//
// Two launches, no sort:
//   k_sample_stats  streams the logits once, a CTA per chunk of 4096 tokens of a row, held in
//                   shared memory: the chunk's maximum, and what the row's filters need of it: its mass,
//                   and counts (top-k) or mass (top-p) per eighth unit of z below the maximum; and
//                   a list of its foremost tokens, which mostly holds all that the row needs of it.
//                   Some 65 instructions a token, most of them the exponential in fixed point, bound it and
//                   not the logits' bytes: 256 rows of 152064 fp32 logits without a filter take 88 us in
//                   all, 1.8 TB/s; 256 of 126464 with top-k, which need no exponential here, 61 us.
//   k_sample_draw   one CTA per row joins the chunks.  Without a filter the mass says which chunk
//                   holds the drawn token, and that chunk alone is read again.  With one, the
//                   eighth units say from where on tokens can stay; those come together in
//                   shared memory from the chunks' lists (a chunk whose list falls short is read
//                   again).  Up to 128 are ranked by counting; of more, the prefix's end is found
//                   by a radix descent over the pair (z, id), which no two tokens share, and the
//                   drawn token by two histograms over the id.  Where more than 12288 come together and
//                   top-p alone decides, only the tokens of the unit in which the prefix ends are
//                   taken, and what is above them is known by its mass (64 rows of 152064 nearly flat
//                   logits: 116 us, 620 us when every pass reads the row again, as other filters still do).
//                   Chains of dependent steps bound it, 13 to 20 us a row and up to 43 for 7000 candidates.
//
// Masses are whole numbers, units of 2^-44 of the largest weight (sums of up to 2^18 tokens
// fit 64 bits): their sums are the same in any order, so atomics cannot move a border and a call
// repeats itself.  exp itself is formed to 2^-36 of each weight (weight44): an fp32
// exponential's 2^-23 would move the running sums across the border of a neighbouring token
// once in a few hundred rows of a large vocabulary.
// A chunk's mass is summed in units of its own maximum and then scaled to the row's, which adds as much again: a
// border is placed to within 2^-35 of the mass and V 2^-43 of the largest weight.  Where the eighth units take part in
// it (more than 12288 candidates under top-p alone) they are rounded to 2^-36 of their chunk's maximum, V 2^-36 in all.  Chunks
// start at 16-byte boundaries, so equal logits at another address can be cut elsewhere and fall to the other side
// of a border inside those bounds.
#include <cfloat>

#include "paged.cuh"

namespace dllm {
namespace {

using u64 = unsigned long long;

constexpr int kStatThreads = 128;
constexpr int kPer = 32;                          // tokens of a thread
constexpr int kChunk = kStatThreads * kPer;       // tokens of a chunk
constexpr int kMaxVocab = 262144;
constexpr int kKept = 1024;                       // most listed tokens of a chunk
constexpr int kMaxChunks = kMaxVocab / kChunk + 1;
constexpr int kCoarse = 128;                      // bins of an eighth unit below the chunk's maximum
constexpr float kPerUnit = 8.f;

constexpr int kThreads = 512;                     // of the drawing CTA
constexpr int kWarps = kThreads / 32;
constexpr int kBins = kThreads;                   // a bin per thread
constexpr int kSmall = 128;                       // candidates ranked by counting
constexpr int kList = 12288;                      // candidates held in shared memory

// ---------------------------------------------------------------- exp in fixed point
constexpr double kLn2_64 = 0.69314718055994530942 / 64;
constexpr double kC1 = (double)(long long)(kLn2_64 * 262144.0) / 262144.0;   // its first 12 bits

struct ExpTable {                  // 2^(-j/64)
    u64 fix[64];                   // in units of 2^-45
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
        t.fix[j] = (u64)(e * 35184372088832.0 + 0.5);
        const double x = e * 2147483648.0 + 0.5;
        t.t31[j] = x >= 2147483647.0 ? 2147483647 : (int)x;
    }
    return t;
}
__constant__ const ExpTable c_table = make_table();


// exp(-(top - z)) in units of 2^-44, off by at most 2^-36 relative (and half a unit); 0 from a
// distance of 32 on.  With n = round(64 d / ln 2) and n = 64 k + j:
// exp(-d) = 2^-k 2^(-j/64) exp(-r), where r = d - n ln2/64 lies within ln2/128.  d - n C1 is exact
// in fp32; it, n (ln2/64 - C1) and the rounding of d are then added in units of 2^-38, and
// exp(-r) - 1 = -r + (r^2/2 - r^3/6 + r^4/24) needs fp32 in its second part alone.
// (finite: of a finite top; 40 in place of larger distances, whose low parts mean nothing, is shifted out.)
__device__ __forceinline__ u64 weight44_finite(float top, float z, const ExpTable &tb) {
    const float d = fminf(top - z, 40.f);
    constexpr float kUnit = 274877906944.f;   // 2^38
    const float bb = d - top;
    const float dl = (top - (d - bb)) - (z + bb);                  // top - z = d + dl exactly
    const float t = fmaf(d, (float)(1.0 / kLn2_64), 12582912.f);   // its low bits: the rounded product
    const int n = __float_as_int(t) - 0x4B400000;
    const float r1 = fmaf(-(t - 12582912.f), (float)kC1, d);
    constexpr uint32_t kRest = (uint32_t)((kLn2_64 - kC1) * 1125899906842624.0 + 0.5);   // 2^50
    const int r = (int)((uint32_t)__float2int_rn(r1 * kUnit) - __umulhi((uint32_t)n << 20, kRest) + (uint32_t)__float2int_rn(dl * kUnit));
    const float rf = (float)r * (1.0f / kUnit);
    const float s = rf * rf * fmaf(rf, fmaf(rf, kUnit / 24.f, -kUnit / 6.f), kUnit * 0.5f);
    const int e = (int)((uint32_t)__float2int_rn(s) - (uint32_t)r);   // exp(-r) - 1
    const int j = n & 63, k = n >> 6;
    const u64 w = tb.fix[j] + (u64)(((long long)e * tb.t31[j]) >> 24);   // units of 2^-45
    return ((w >> k) + 1) >> 1;
}
__device__ __forceinline__ u64 weight44(float top, float z, const ExpTable &tb) {
    return z == top ? 1ull << 44 : top < INFINITY ? weight44_finite(top, z, tb) : 0;   // (infinite: its equals alone)
}

__device__ __forceinline__ void load_table(ExpTable &tb) {
    if (threadIdx.x < 64) {
        tb.fix[threadIdx.x] = c_table.fix[threadIdx.x];
        tb.t31[threadIdx.x] = c_table.t31[threadIdx.x];
    }
}

// ---------------------------------------------------------------- small helpers
__device__ __forceinline__ uint32_t order_key(float z) {   // ascending with z (no NaN, no -0)
    const uint32_t u = __float_as_uint(z);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
// Eighth unit of z (a whole number as float).
__device__ __forceinline__ float eighth(float z) { return floorf(z * kPerUnit); }

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Adds a mass in shared memory: two 32-bit atomics with the carry between them (there is no
// native 64-bit add); the high half of a sum stays below 2^32.
__device__ __forceinline__ void add64(u64 *bin, u64 v) {
    unsigned *p = reinterpret_cast<unsigned *>(bin);
    const unsigned lo = (unsigned)v;
    const unsigned old = atomicAdd(p, lo);
    const unsigned hi = (unsigned)(v >> 32) + (old + lo < lo ? 1u : 0u);
    if (hi) atomicAdd(p + 1, hi);
}

// A row's settings and what they ask of its chunks.
struct RowSet {
    float inv;        // 1 / T
    float p;          // >= 1: off
    u64 k;            // 0: off
    u64 floor44;      // min-p in weight units, 0: off
    float min_p;
    bool off, greedy;
    __device__ __forceinline__ RowSet(const SampleArgs &a, int row) {
        const int b = row / a.M;
        off = a.valid && !a.valid[row];
        const float t = a.temperature ? a.temperature[b] : 1.f;
        inv = 1.0f / t;
        greedy = !(t > 0.f && inv < INFINITY);
        if (greedy) inv = 1.f;
        const int kk = a.top_k ? a.top_k[b] : 0;
        k = kk > 0 && kk < a.V ? (u64)kk : 0;
        p = a.top_p ? a.top_p[b] : 1.f;
        if (!(p < 1.f)) p = 1.f;
        min_p = a.min_p ? a.min_p[b] : 0.f;
        floor44 = min_p > 0.f ? (min_p < 1.f ? __float2ull_ru(min_p * 17592186044416.f) : 1ull << 44) : 0;
    }
    // Distance to the maximum beyond which min-p leaves nothing.
    __device__ __forceinline__ float reach() const { return -logf(fminf(fmaxf(min_p, 1e-30f), 1.f)) * 1.0001f + 1e-3f; }
    __device__ __forceinline__ bool by_mass() const { return !greedy && !k && p < 1.f; }
    __device__ __forceinline__ bool open() const { return !greedy && !k && p >= 1.f && !floor44; }
};

struct ChunkStat {
    float top;        // maximum of the chunk's scaled logits, -inf: none
    int id;           // its lowest id (greedy rows)
    u64 mass;         // sum of weight44(top, z) (rows without filter, or with top-p alone)
    float low;        // tokens with z >= low are listed (+inf: too many, n > kKept)
    int n;            // how many
};

// The vectors of a row: position q = id + mis counts from the 16-byte boundary at or before
// the row, so that vector v holds q = v E .. v E + E - 1.
template <class TL> struct RowView {
    static constexpr int E = 16 / sizeof(TL);
    const TL *l;
    int V, mis;
    float inv;
    __device__ __forceinline__ RowView(const SampleArgs &a, int row, float inv_) {
        l = static_cast<const TL *>(a.logits) + (size_t)row * a.V;
        V = a.V;
        mis = (int)((reinterpret_cast<uintptr_t>(l) & 15) / sizeof(TL));
        inv = inv_;
    }
    __device__ __forceinline__ int vectors() const { return (V + mis + E - 1) / E; }
    // Raw vector v; outside the row: NaN.
    __device__ __forceinline__ uint4 raw(int v) const {
        const int id = v * E - mis;
        if (id >= 0 && id + E <= V) return *reinterpret_cast<const uint4 *>(l + id);
        uint32_t w[4] = {~0u, ~0u, ~0u, ~0u};
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (id + e >= 0 && id + e < V) {
                if (sizeof(TL) == 4) {
                    w[e % 4] = reinterpret_cast<const uint32_t *>(l)[id + e];
                } else {
                    const uint32_t x = reinterpret_cast<const uint16_t *>(l)[id + e];
                    w[e / 2] = e & 1 ? (w[e / 2] & 0xffffu) | (x << 16) : (w[e / 2] & 0xffff0000u) | x;
                }
            }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // Its scaled logit e: -0 counts as 0, NaN (never drawn) as -inf.
    __device__ __forceinline__ float scaled(const uint4 &x, int e) const {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        const float y = sizeof(TL) == 4 ? __uint_as_float(w[e % 4])
                                        : __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
        return fmaxf(fmaf(y, inv, 0.f), -INFINITY);
    }
    __device__ __forceinline__ void scaled(const uint4 &x, float *z) const {
#pragma unroll
        for (int e = 0; e < E; ++e) z[e] = scaled(x, e);
    }
};

// ---------------------------------------------------------------- first launch: the chunks
template <class TL>
__global__ void __launch_bounds__(kStatThreads, 12) k_sample_stats(const SampleArgs a, ChunkStat *stat, u64 *coarse,
                                                               uint2 *list, int nc) {
    using View = RowView<TL>;
    constexpr int E = View::E, NV = kPer / E;
    __shared__ ExpTable tb;
    __shared__ float s_top[kStatThreads / 32];
    __shared__ u64 s_mass[kStatThreads / 32];
    __shared__ int s_id[kStatThreads / 32];
    __shared__ uint32_t s_bin[2][kCoarse];           // counts; masses in units of 2^-36, two digits of 18 bits
    __shared__ float s_low;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    load_table(tb);
    if (tid < kCoarse) s_bin[0][tid] = s_bin[1][tid] = 0;
    griddep_wait();
    griddep_launch();
    const int row = blockIdx.x / nc, c = blockIdx.x - row * nc;
    const RowSet rs(a, row);
    if (rs.off) return;
    const View view(a, row, rs.inv);
    // thread's vectors: c * kChunk / E + u * kStatThreads + tid
    // They stay in shared memory, and each phase is a loop of four tokens a turn: unrolled over registers, the
    // exponentials alone outgrow the instruction cache (256 rows of 152064: 126 us, 97 in loops).
    __shared__ float4 s_z[kPer / 4 * kStatThreads];
    const int v0 = c * (kChunk / E) + tid, nv = view.vectors();
    float top = -INFINITY;
    {
        uint4 x[NV];
#pragma unroll
        for (int u = 0; u < NV; ++u) x[u] = v0 + u * kStatThreads < nv ? view.raw(v0 + u * kStatThreads) : make_uint4(~0u, ~0u, ~0u, ~0u);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float z[E];
            view.scaled(x[u], z);
#pragma unroll
            for (int e = 0; e < E; ++e) top = fmaxf(top, z[e]);
#pragma unroll
            for (int e = 0; e < E; e += 4) s_z[(u * E + e) / 4 * kStatThreads + tid] = make_float4(z[e], z[e + 1], z[e + 2], z[e + 3]);
        }
    }
    auto each = [&](auto &&f) {           // f(z, id)
#pragma unroll 1
        for (int i = 0; i < kPer; i += 4) {
            const float4 z = s_z[i / 4 * kStatThreads + tid];
            const int id = (v0 + i / E * kStatThreads) * E + i % E - view.mis;
            f(z.x, id);
            f(z.y, id + 1);
            f(z.z, id + 2);
            f(z.w, id + 3);
        }
    };
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) s_top[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kStatThreads / 32; ++w) top = fmaxf(top, s_top[w]);
    ChunkStat st{top, INT_MAX, 0, INFINITY, 0};
    if (rs.greedy) {
        int id = INT_MAX;
        each([&](float z, int i) {
            if (z == top) id = min(id, i);
        });
        id = __reduce_min_sync(0xffffffffu, id);
        if (lane == 0) s_id[warp] = id;
        __syncthreads();
        for (int w = 0; w < kStatThreads / 32; ++w) st.id = min(st.id, s_id[w]);
    } else if (top > -INFINITY) {
        const bool mass = rs.by_mass(), count = rs.k > 0;
        const float q0 = eighth(top);
        auto bin_of = [&](float y) -> int {   // the last one: everything further (and -inf)
            const float q = y == top ? 0.f : q0 - eighth(y);
            return q < (float)(kCoarse - 1) ? (int)q : kCoarse - 1;
        };
        if (mass || rs.open()) {
            u64 s = 0;
            // (an infinite maximum's units stay empty: the second launch asks such a row for none)
            if (!(top < INFINITY)) each([&](float y, int) { s += y == top ? 1ull << 44 : 0; });
            else if (!mass) each([&](float y, int) { s += weight44_finite(top, y, tb); });
            else each([&](float y, int) {
                const u64 w = weight44_finite(top, y, tb);
                s += w;
                const u64 v = (w + 128) >> 8;             // (a chunk's sum of 18-bit digits fits 32 bits)
                if (v) {
                    const int bin = bin_of(y);
                    atomicAdd(&s_bin[0][bin], (uint32_t)v & 0x3ffffu);
                    if (v >> 18) atomicAdd(&s_bin[1][bin], (uint32_t)(v >> 18));
                }
            });
            s = warp_sum(s);
            if (lane == 0) s_mass[warp] = s;
        } else if (count) {
            each([&](float y, int) {
                const int bin = bin_of(y);
                if (bin < kCoarse - 1) atomicAdd(&s_bin[0][bin], 1u);
            });
        }
        __syncthreads();
        if (mass || rs.open())
            for (int w = 0; w < kStatThreads / 32; ++w) st.mass += s_mass[w];
        auto unit = [&](int b) { return mass ? ((u64)s_bin[0][b] << 8) + ((u64)s_bin[1][b] << 26) : (u64)s_bin[0][b]; };
        if ((mass || count) && tid < kCoarse) {
            u64 *row_units = coarse + (size_t)row * nc * kCoarse;
            if (mass) row_units[c * kCoarse + tid] = unit(tid);
            else reinterpret_cast<uint32_t *>(row_units)[c * kCoarse + tid] = s_bin[0][tid];
        }
        if (!rs.open()) {
            // From where on tokens are listed: the chunk's first k (no other can be among the row's),
            // or all but a quarter of (1 - p) of the mass in the bins (a guess that the second launch checks),
            // and not below what min-p leaves.
            if (warp == 0) {
                constexpr int B = kCoarse / 32;
                u64 v[B], x = 0;
#pragma unroll
                for (int b = 0; b < B; ++b) x += v[b] = mass || count ? unit(lane * B + b) : 0;
                const u64 own = x;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const u64 y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o) x += y;
                }
                u64 at = x - own;
                const u64 need = count ? rs.k : (u64)((float)__shfl_sync(0xffffffffu, x, 31) * (0.75f + 0.25f * fmaxf(rs.p, 0.f)));
                int bin = INT_MAX;
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    at += v[b];
                    if (bin == INT_MAX && at >= need) bin = lane * B + b;
                }
                bin = __reduce_min_sync(0xffffffffu, bin);
                float low = -INFINITY;
                if ((mass || count) && bin < kCoarse - 1 && fabsf(q0) < 4194304.f) low = (q0 - (float)bin) / kPerUnit;
                if (rs.floor44 && !rs.k) low = fmaxf(low, top - rs.reach());
                if (low == -INFINITY || top == INFINITY) low = top;   // nothing known: the foremost alone
                if (lane == 0) s_low = low;
            }
            __syncthreads();
            const float low = s_low;
            uint2 *out = list + ((size_t)row * nc + c) * kKept;
            int mine = 0;
            each([&](float y, int) { mine += y >= low; });
            int at = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, at, o);
                if (lane >= o) at += y;
            }
            if (lane == 31) s_id[warp] = at;
            __syncthreads();
            at -= mine;
#pragma unroll
            for (int w = 0; w < kStatThreads / 32; ++w) {
                if (w < warp) at += s_id[w];
                st.n += s_id[w];
            }
            if (mine && at + mine <= kKept)
                each([&](float y, int i) {
                    if (y >= low) out[at++] = make_uint2(__float_as_uint(y), (uint32_t)i);
                });
            st.low = st.n <= kKept ? low : INFINITY;
        }
    }
    if (tid == 0) stat[(size_t)row * nc + c] = st;
}

// ---------------------------------------------------------------- second launch: the rows
struct alignas(16) Shared {
    ExpTable tb;
    ChunkStat st[kMaxChunks];
    u64 scale[kMaxChunks];         // weight44 of the chunk's maximum in the row,
    float scale_lo[kMaxChunks];    // 2^28 of it as a ratio, a little less
    u64 mass[kMaxChunks];          // the chunk's mass in the row's units
    int off[kMaxChunks];           // its eighth units below the row's first
    u64 bins[kBins];
    unsigned cnt[kBins];
    u64 warp[kWarps];
    u64 val, before, total;
    float top, from;
    int n, where;
    float z[kList];
    uint32_t id[kList];
};

__device__ __forceinline__ u64 block_sum(Shared &sh, u64 v) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    v = warp_sum(v);
    __syncthreads();
    if (lane == 0) sh.warp[warp] = v;
    __syncthreads();
    return warp_sum(lane < kWarps ? sh.warp[lane] : 0);
}

// Inclusive running sum over the CTA's threads.
__device__ __forceinline__ u64 block_scan(Shared &sh, u64 v) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    __syncthreads();
    if (lane == 31) sh.warp[warp] = v;
    __syncthreads();
    return v + warp_sum(lane < warp ? sh.warp[lane] : 0);
}

// The bin in which the running sum of sh.bins, starting at acc, reaches target (-1: none).  acc
// becomes the sum before it and val its own.
__device__ __forceinline__ int crossing(Shared &sh, u64 target, u64 &acc, u64 &val) {
    const u64 v = sh.bins[threadIdx.x];
    if (threadIdx.x == 0) sh.where = -1;
    const u64 upto = acc + block_scan(sh, v);
    if (upto >= target && upto - v < target) {
        sh.where = threadIdx.x;
        sh.before = upto - v;
        sh.val = v;
    }
    __syncthreads();
    const int bin = sh.where;
    if (bin >= 0) {
        acc = sh.before;
        val = sh.val;
    }
    __syncthreads();
    return bin;
}

// f * total for f in [0, 1), exactly, rounded down (or up).  (Whole numbers: the GPU's 64-bit
// floating-point rate is a small fraction of its integer rate.)
__device__ __forceinline__ u64 share(float f, u64 total, bool up) {
    const uint32_t bits = __float_as_uint(f), e = bits >> 23;
    const u64 m = e ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
    const int s = 150 - (int)(e ? e : 1);      // f = m 2^-s, s >= 24
    const u64 lo = total * m, hi = __umul64hi(total, m);
    if (s >= 128) return up && (lo | hi) ? 1 : 0;
    const u64 q = s >= 64 ? hi >> (s - 64) : (hi << (64 - s)) | (lo >> s);
    const u64 rest = s >= 64 ? lo | (s > 64 ? hi << (128 - s) : 0) : lo << (64 - s);
    return q + (up && rest ? 1 : 0);
}
__device__ __forceinline__ u64 mass_target(float p, u64 total) {   // tokens with less before them stay
    const u64 t = p > 0.f ? share(p, total, true) : 0;
    return t ? t : 1;
}
__device__ __forceinline__ u64 drawn(float u, u64 total) {         // u * total, below total
    if (!(u < 1.f)) return u >= 1.f ? total - 1 : 0;
    const u64 t = u > 0.f ? share(u, total, false) : 0;
    return t < total ? t : total - 1;
}

// total: the kept mass in units of 2^-44
__device__ __forceinline__ void answer(int32_t *token, float *prob, int id, float z, float top, u64 total,
                                       const ExpTable &tb) {
    *token = id;
    // (a rare token's weight has too few of the fixed point's bits)
    const double w = z == top || top - z < 12.f ? (double)weight44(top, z, tb) : exp((double)z - (double)top) * 17592186044416.0;
    *prob = (float)(w / (double)total);
}

// No filter: every token can be drawn.
template <class TL>
__device__ void draw_open(const SampleArgs &a, Shared &sh, const RowView<TL> &view, int row, int nc) {
    constexpr int E = RowView<TL>::E, NV = kChunk / kThreads / E;   // a thread's consecutive vectors
    const int tid = threadIdx.x;
    if (tid < 32) {   // the chunk, in the order of the ids
        const u64 t = drawn(a.u[row], sh.total);
        u64 run = 0;
        for (int c0 = 0; c0 < nc; c0 += 32) {
            const u64 m = c0 + tid < nc ? sh.mass[c0 + tid] : 0;
            u64 x = m;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 y = __shfl_up_sync(0xffffffffu, x, o);
                if (tid >= o) x += y;
            }
            if (run + x > t && run + x - m <= t) {   // and the place in it, in its own units
                sh.where = c0 + tid;
                sh.val = (u64)((double)(t - (run + x - m)) * (17592186044416.0 / (double)sh.scale[c0 + tid]));
            }
            run += __shfl_sync(0xffffffffu, x, 31);
        }
    }
    __syncthreads();
    const int c = sh.where;
    u64 target = sh.val;
    if (target >= sh.st[c].mass) target = sh.st[c].mass - 1;
    const float ctop = sh.st[c].top;
    const int v0 = c * (kChunk / E) + tid * NV, nv = view.vectors();
    float z[NV * E];
    u64 s = 0;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        view.scaled(v0 + u < nv ? view.raw(v0 + u) : make_uint4(~0u, ~0u, ~0u, ~0u), z + u * E);
#pragma unroll
        for (int e = 0; e < E; ++e) s += weight44(ctop, z[u * E + e], sh.tb);
    }
    u64 at = block_scan(sh, s) - s;
    if (target < at || target >= at + s) return;
    for (int i = 0; i < NV * E; ++i) {
        const u64 w = weight44(ctop, z[i], sh.tb);
        if (target < at + w) {
            answer(a.token + row, a.prob + row, v0 * E + i - view.mis, z[i], sh.top, sh.total, sh.tb);
            return;
        }
        at += w;
    }
}

// Up to kSmall listed candidates, ranked by counting: `per` neighbouring lanes share one.  (256 rows with top-k
// 50: 61.3 us, 64.7 by the radix descent.)
__device__ void draw_small(const SampleArgs &a, Shared &sh, int row, int n, const RowSet &rs, u64 total) {
    int per = 1;
    while (per < 16 && kThreads / (2 * per) >= n) per *= 2;
    const int e = threadIdx.x / per, part = threadIdx.x & (per - 1);
    const bool on = e < n, own = on && part == 0;
    const float z = on ? sh.z[e] : -INFINITY;
    const uint32_t id = on ? sh.id[e] : 0xffffffffu;
    const bool busy = (threadIdx.x & ~31) / per < n;
    int rank = 0;
    if (busy) {
#pragma unroll 4
        for (int j = part; j < n; j += per) {
            const float y = sh.z[j];
            rank += y > z || (y == z && sh.id[j] < id);
        }
        for (int o = per >> 1; o > 0; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    }
    const u64 w = on ? weight44(sh.top, z, sh.tb) : 0;
    sh.bins[threadIdx.x] = 0;
    __syncthreads();
    if (own) sh.bins[rank] = w;
    __syncthreads();
    const u64 upto = block_scan(sh, sh.bins[threadIdx.x]);
    __syncthreads();
    sh.bins[threadIdx.x] = upto;
    __syncthreads();
    if (rs.k) total = sh.bins[(rs.k < (u64)n ? (int)rs.k : n) - 1];
    bool in = on && (!rs.k || (u64)rank < rs.k);
    if (in && rs.p < 1.f) in = sh.bins[rank] - w < mass_target(rs.p, total);
    if (in && rs.floor44) in = rank == 0 || w >= rs.floor44;
    __syncthreads();
    if (own) sh.bins[e] = in ? w : 0;      // kept weights in the list's order
    const u64 kept = block_sum(sh, own && in ? w : 0);
    u64 below = 0;                // kept mass of lower ids
    if (busy) {
#pragma unroll 4
        for (int j = part; j < n; j += per) below += sh.id[j] < id ? sh.bins[j] : 0;
        for (int o = per >> 1; o > 0; o >>= 1) below += __shfl_xor_sync(0xffffffffu, below, o);
    }
    const u64 t = drawn(a.u[row], kept);
    if (own && in && below <= t && t < below + w) answer(a.token + row, a.prob + row, (int)id, z, sh.top, kept, sh.tb);
}

// Descending order as one number: z's key above the lowest candidate's, then the id.
__device__ __forceinline__ u64 key_of(float z, uint32_t id, uint32_t base) {
    return (u64)(order_key(z) - base) << 18 | (u64)(kMaxVocab - 1 - id);
}

// The lowest key of the order's prefix of the candidates that each(f) calls f(z, id) for, from the key
// `lowest` up to z = ztop, whose count (or mass), with acc before them, reaches target; `lowest` if none does.
template <class Each>
__device__ __forceinline__ u64 descend(Shared &sh, bool by_mass, u64 target, u64 acc, float ztop, uint32_t base, u64 lowest,
                                       Each &&each) {
    const int tid = threadIdx.x;
    const float top = sh.top;
    u64 hi = (u64)(order_key(ztop) - base) << 18 | (u64)(kMaxVocab - 1), lo = lowest, val = 0;
    for (;;) {
        const int bits = 64 - __clzll((long long)(hi - lo));
        const int shift = bits > 9 ? bits - 9 : 0;
        __syncthreads();
        sh.bins[tid] = 0;
        sh.cnt[tid] = 0;
        __syncthreads();
        each([&](float z, uint32_t id) {
            const u64 k = key_of(z, id, base);
            if (k < lo || k > hi) return;
            const int bin = (int)((hi - k) >> shift);
            atomicAdd(&sh.cnt[bin], 1u);
            if (by_mass) {
                const u64 w = weight44(top, z, sh.tb);
                if (w) add64(&sh.bins[bin], w);
            } else {
                atomicAdd(reinterpret_cast<unsigned *>(&sh.bins[bin]), 1u);
            }
        });
        __syncthreads();
        const int bin = crossing(sh, target, acc, val);
        if (bin < 0) return lowest;                // never reached: all stay
        const u64 h = hi - ((u64)bin << shift);
        const u64 l = h - ((1ull << shift) - 1ull);
        hi = h;
        if (l > lo && l <= h) lo = l;
        const int m = (int)sh.cnt[bin];
        // whole bin, one candidate, or one key
        if (acc + val == target || m == 1 || hi == lo) return lo;
        if (m <= kSmall) {                         // few: each looks at the others
            __syncthreads();
            if (tid == 0) sh.where = 0;
            __syncthreads();
            each([&](float z, uint32_t id) {
                const u64 k = key_of(z, id, base);
                if (k < lo || k > hi) return;
                const int at = atomicAdd(&sh.where, 1);
                sh.bins[at] = k;
                sh.bins[kSmall + at] = by_mass ? weight44(top, z, sh.tb) : 1ull;
            });
            __syncthreads();
            if (tid < m) {
                const u64 k = sh.bins[tid], w = sh.bins[kSmall + tid];
                u64 before = acc;
                for (int j = 0; j < m; ++j) before += sh.bins[j] > k ? sh.bins[kSmall + j] : 0;
                if (before < target && before + w >= target) sh.val = k;
            }
            __syncthreads();
            return sh.val;
        }
    }
}

// The filters and the draw over many candidates (those from `low` on): each(f) calls f(z, id)
// for every one of them, by all threads.  total as for draw_small.
template <class Each>
__device__ __forceinline__ void draw_many(const SampleArgs &a, Shared &sh, int row, const RowSet &rs, float low, u64 total,
                                          Each &&each) {
    const float top = sh.top;
    const uint32_t base = order_key(low);
    u64 lowest = 0;
    if (rs.k) lowest = descend(sh, false, rs.k, 0, top, base, lowest, each);
    if (rs.p < 1.f) {
        if (rs.k) {
            u64 s = 0;
            each([&](float z, uint32_t id) { s += key_of(z, id, base) >= lowest ? weight44(top, z, sh.tb) : 0; });
            total = block_sum(sh, s);
        }
        lowest = descend(sh, true, mass_target(rs.p, total), 0, top, base, lowest, each);
    }
    auto weight = [&](float z, uint32_t id) -> u64 {
        if (key_of(z, id, base) < lowest) return 0;
        const u64 w = weight44(top, z, sh.tb);
        return w >= rs.floor44 ? w : 0;
    };
    __syncthreads();
    sh.bins[threadIdx.x] = 0;
    __syncthreads();
    each([&](float z, uint32_t id) {
        const u64 w = weight(z, id);
        if (w) add64(&sh.bins[id / kBins], w);
    });
    __syncthreads();
    const u64 kept = block_sum(sh, sh.bins[threadIdx.x]);
    const u64 t = drawn(a.u[row], kept);
    u64 acc = 0, val = 0;
    const int part = crossing(sh, t + 1, acc, val);
    __syncthreads();
    sh.bins[threadIdx.x] = 0;
    sh.cnt[threadIdx.x] = 0;
    __syncthreads();
    each([&](float z, uint32_t id) {
        if ((int)(id / kBins) != part) return;
        sh.bins[id % kBins] = weight(z, id);
        sh.cnt[id % kBins] = __float_as_uint(z);
    });
    __syncthreads();
    const int at = crossing(sh, t + 1, acc, val);
    if (threadIdx.x == 0) answer(a.token + row, a.prob + row, part * kBins + at, __uint_as_float(sh.cnt[at]), top, kept, sh.tb);
}

// The mass of a row's eighth unit in chunk c (to a unit of 2^-44), from the chunk's own eighth units (coarse of
// the row), which start off[c] below the row's.
__device__ __forceinline__ u64 unit_mass(const Shared &sh, const u64 *exact, int c, int unit) {
    const int b = unit - sh.off[c];                       // (every chunk reaches down to the last but one)
    const u64 m = b >= 0 && unit < kCoarse - 1 ? exact[c * kCoarse + b] : 0, f = sh.scale[c];
    return __umul64hi(m, f) << 20 | (m * f) >> 44;
}

// Puts the row's tokens from `low` to below zhi (NaN: all) into the list and their number into sh.n (zero before);
// with more than fit, any of them and any larger number.  list: the row's chunks' own.
template <class TL>
__device__ __forceinline__ void gather(Shared &sh, const RowView<TL> &view, const uint2 *list, int nc, float low, float zhi) {
    constexpr int E = RowView<TL>::E;
    const int tid = threadIdx.x, lane = tid & 31, nv = view.vectors();
    auto wanted = [&](float z) { return z >= low && !(z >= zhi); };
    // a warp's places for `in` candidates of each lane: one atomic
    auto places = [&](int in) -> int {
        int at = in;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, at, o);
            if (lane >= o) at += y;
        }
        int base = 0;
        if (lane == 31 && at) base = atomicAdd(&sh.n, at);
        return __shfl_sync(0xffffffffu, base, 31) + at - in;
    };
    auto put = [&](int at, float z, uint32_t id) {
        if (at < kList) {
            sh.z[at] = z;
            sh.id[at] = id;
        }
    };
    for (int c = tid >> 5; c < nc; c += kWarps) {
        const ChunkStat st = sh.st[c];
        if (!(st.top >= low)) continue;
        if (__shfl_sync(0xffffffffu, *reinterpret_cast<volatile int *>(&sh.n), 0) > kList) break;   // (they are not used)
        if (st.n <= kKept && st.low <= low) {   // (low may be infinite itself)
            const uint2 *src = list + (size_t)c * kKept;
            constexpr int U = 8;   // entries of a lane at a time, one atomic for the warp's
            for (int i = lane; i < (st.n + 31) / 32 * 32; i += U * 32) {
                uint2 x[U];
                int in = 0;
#pragma unroll
                for (int u = 0; u < U; ++u) x[u] = i + u * 32 < st.n ? src[i + u * 32] : make_uint2(~0u, 0);
#pragma unroll
                for (int u = 0; u < U; ++u) in += wanted(__uint_as_float(x[u].x));
                int at = places(in);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (wanted(__uint_as_float(x[u].x))) put(at++, __uint_as_float(x[u].x), x[u].y);
            }
        } else {   // its list does not reach down to there
            constexpr int U = 16 / E * 2;   // 32 tokens of a lane at a time
            const int end = min(nv, (c + 1) * (kChunk / E));
            for (int vw = c * (kChunk / E); vw < end; vw += U * 32) {
                const int v0 = vw + lane;
                uint4 x[U];
#pragma unroll
                for (int u = 0; u < U; ++u) x[u] = v0 + u * 32 < end ? view.raw(v0 + u * 32) : make_uint4(~0u, ~0u, ~0u, ~0u);
                int in = 0;
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int e = 0; e < E; ++e) in += wanted(view.scaled(x[u], e));
                int at = places(in);
                if (in)
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            const float z = view.scaled(x[u], e);
                            if (wanted(z)) put(at++, z, (uint32_t)((v0 + u * 32) * E + e - view.mis));
                        }
            }
        }
    }
}

// top-p alone over more candidates than the list holds: the chunks' exact eighth units say in which unit the
// prefix ends, and only that unit's tokens are listed.  What is above them needs no other look than at the
// chunk that is drawn.  false: they do not fit either.
// Not inlined: its registers would cost the other rows theirs.
template <class TL>
__device__ __noinline__ bool draw_wide(Shared &sh, const RowView<TL> view, float p, float u01, int32_t *token, float *prob,
                                       const u64 *exact, const uint2 *list, int nc) {
    constexpr int E = RowView<TL>::E, NV = kChunk / kThreads / E;   // a thread's consecutive vectors of a chunk
    const int tid = threadIdx.x, lane = tid & 31;
    const float top = sh.top, q0 = eighth(top);
    __syncthreads();
    sh.bins[tid] = 0;
    if (tid == 0) sh.n = 0;
    __syncthreads();
    u64 sum = 0, above = 0, val;
    for (int c = tid / kCoarse; c < nc; c += kThreads / kCoarse) sum += unit_mass(sh, exact, c, tid % kCoarse);
    if (sum) add64(&sh.bins[tid % kCoarse], sum);
    __syncthreads();
    const int unit = crossing(sh, mass_target(p, sh.total), above, val);
    if (unit < 0) return false;
    const float low = (q0 - (float)unit) / kPerUnit;
    const float zhi = unit > 0 ? low + 1.f / kPerUnit : __uint_as_float(0x7fffffffu);
    gather(sh, view, list, nc, low, zhi);
    __syncthreads();
    const int n = sh.n;
    if (n > kList) return false;
    const uint32_t base = order_key(low);
    auto listed = [&](auto &&f) {
        for (int i = tid; i < n; i += kThreads) f(sh.z[i], sh.id[i]);
    };
    const u64 lowest = descend(sh, true, mass_target(p, sh.total), above, fminf(zhi, top), base, 0, listed);
    // kept mass of the chunks
    __syncthreads();
    sh.bins[tid] = 0;
    __syncthreads();
    for (int c = tid >> 5; c < nc; c += kWarps) {
        u64 s = 0;
        if (sh.st[c].top > -INFINITY)
            for (int u = lane; u < unit; u += 32) s += unit_mass(sh, exact, c, u);
        s = warp_sum(s);
        if (lane == 0) sh.bins[c] = s;
    }
    __syncthreads();
    listed([&](float z, uint32_t id) {
        const u64 w = key_of(z, id, base) >= lowest ? weight44(top, z, sh.tb) : 0;
        if (w) add64(&sh.bins[((int)id + view.mis) / kChunk], w);
    });
    __syncthreads();
    const u64 kept = block_sum(sh, sh.bins[tid]);
    const u64 t = drawn(u01, kept);
    u64 acc = 0;
    const int c = crossing(sh, t + 1, acc, val);
    // the token in it
    const int v0 = c * (kChunk / E) + tid * NV, nv = view.vectors();
    float z[NV * E];
    u64 w[NV * E], s = 0;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        view.scaled(v0 + u < nv ? view.raw(v0 + u) : make_uint4(~0u, ~0u, ~0u, ~0u), z + u * E);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int i = u * E + e;
            const bool in = z[i] >= zhi || (z[i] >= low && key_of(z[i], (uint32_t)(v0 * E + i - view.mis), base) >= lowest);
            s += w[i] = in ? weight44(top, z[i], sh.tb) : 0;
        }
    }
    const u64 all = block_sum(sh, s);
    if (!all) return false;                        // (a chunk of weights that are nothing in the row's units)
    const u64 want = t - acc < all ? t - acc : all - 1;   // (units of 2^-44 apart from the sums above)
    u64 at = block_scan(sh, s) - s;
#pragma unroll
    for (int i = 0; i < NV * E; ++i) {
        if (want >= at && want < at + w[i]) answer(token, prob, v0 * E + i - view.mis, z[i], top, kept, sh.tb);
        at += w[i];
    }
    return true;
}

// Rows of one chunk in one launch: the CTA holds the row and every token is a candidate.
template <class TL>
__global__ void __launch_bounds__(kThreads) k_sample_row(const SampleArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Shared &sh = *reinterpret_cast<Shared *>(smem_raw);
    using View = RowView<TL>;
    constexpr int E = View::E;
    const int row = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    load_table(sh.tb);
    griddep_wait();
    griddep_launch();
    const RowSet rs(a, row);
    const View view(a, row, rs.inv);
    float top = -INFINITY;
    if (!rs.off)
        for (int v = tid; v < view.vectors(); v += kThreads) {
            float z[E];
            view.scaled(view.raw(v), z);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int id = v * E + e - view.mis;
                if (id >= 0 && id < a.V) sh.z[id] = z[e];
                top = fmaxf(top, z[e]);
            }
        }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) sh.warp[warp] = __float_as_uint(top);
    if (tid == 0) sh.where = INT_MAX;
    __syncthreads();
    top = __uint_as_float((uint32_t)sh.warp[lane % kWarps]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (tid == 0) sh.top = top;
    __syncthreads();
    if (rs.off || rs.greedy || top == -INFINITY) {
        int id = INT_MAX;
        if (!rs.off && top > -INFINITY)
            for (int i = tid; i < a.V; i += kThreads)
                if (sh.z[i] == top) id = min(id, i);
        id = __reduce_min_sync(0xffffffffu, id);
        if (lane == 0 && id != INT_MAX) atomicMin(&sh.where, id);
        __syncthreads();
        if (tid == 0) {
            const bool none = sh.where == INT_MAX;
            a.token[row] = none ? -1 : sh.where;
            a.prob[row] = none ? 0.f : 1.f;
        }
        return;
    }
    auto each = [&](auto &&f) {
        for (int i = tid; i < a.V; i += kThreads) {
            const float z = sh.z[i];
            if (z > -INFINITY) f(z, (uint32_t)i);
        }
    };
    u64 total = 0;
    if (rs.by_mass()) {
        each([&](float z, uint32_t) { total += weight44(top, z, sh.tb); });
        total = block_sum(sh, total);
    }
    // (below a distance of 32 no token has weight; one that top-k counts may lie there)
    draw_many(a, sh, row, rs, rs.k ? -FLT_MAX : fmaxf(top - 33.f, -FLT_MAX), total, [&](auto &&f) {
        const float from = rs.k ? -FLT_MAX : fmaxf(top - 33.f, -FLT_MAX);
        each([&](float z, uint32_t id) {
            if (z >= from) f(z, id);
        });
    });
}

template <class TL>
__global__ void __launch_bounds__(kThreads, 2) k_sample_draw(const SampleArgs a, const ChunkStat *stat, const u64 *coarse,
                                                          const uint2 *list, int nc) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Shared &sh = *reinterpret_cast<Shared *>(smem_raw);
    using View = RowView<TL>;
    constexpr int E = View::E;
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    load_table(sh.tb);
    sh.bins[tid] = 0;
    if (tid == 0) sh.n = 0;
    griddep_wait();
    griddep_launch();
    ChunkStat mine{};
    if (tid < nc) mine = stat[(size_t)row * nc + tid];   // (not written for a row that is off)
    const RowSet rs(a, row);
    if (rs.off) {
        if (tid == 0) {
            a.token[row] = -1;
            a.prob[row] = 0.f;
        }
        return;
    }
    if (tid < nc) sh.st[tid] = mine;
    __syncthreads();
    if (tid < 32) {
        float top = -INFINITY;
        for (int c = lane; c < nc; c += 32) top = fmaxf(top, sh.st[c].top);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        int id = INT_MAX;
        if (rs.greedy)
            for (int c = lane; c < nc; c += 32)
                if (sh.st[c].top == top) id = min(id, sh.st[c].id);
        id = __reduce_min_sync(0xffffffffu, id);
        if (lane == 0) {
            sh.top = top;
            if (rs.greedy || top == -INFINITY) {
                a.token[row] = top == -INFINITY ? -1 : id;
                a.prob[row] = top == -INFINITY ? 0.f : 1.f;
            }
        }
    }
    __syncthreads();
    const float top = sh.top;
    if (rs.greedy || top == -INFINITY) return;
    const View view(a, row, rs.inv);
    if (rs.by_mass() || rs.open()) {   // the mass of the row
        if (tid < 32) {
            u64 s = 0;
            for (int c = lane; c < nc; c += 32) {
                const u64 f = weight44(top, sh.st[c].top, sh.tb), m = sh.st[c].mass;
                const u64 x = __umul64hi(m, f) << 20 | (m * f) >> 44;   // m f / 2^44
                sh.scale[c] = f;
                sh.scale_lo[c] = (float)f * (0.99999f / 65536.f);
                sh.mass[c] = x;
                s += x;
            }
            s = warp_sum(s);
            if (lane == 0) sh.total = s;
        }
        __syncthreads();
        if (rs.open()) {
            draw_open(a, sh, view, row, nc);
            return;
        }
    }
    // ---------------- from which eighth unit on tokens can stay
    const float q0 = eighth(top);
    float from = -INFINITY;
    const u64 *units = coarse + (size_t)row * nc * kCoarse;
    u64 total = rs.by_mass() ? sh.total : 0;
    if (rs.by_mass() || rs.k) {
        // counts, or a mass, of the row's eighth units: thread = (unit, a part of the chunks); a chunk's own
        // units start off[c] below the row's.  The mass from the row's maximum down to a unit is a lower bound: its tokens'
        // roundings add 2^-37 each at most, 2^-19 in all, and scale_lo takes 10^-5 (2^-17) off the largest weight alone.
        if (tid < nc) {
            const float q = sh.st[tid].top == top ? 0.f : q0 - eighth(sh.st[tid].top);
            sh.off[tid] = q < (float)kCoarse ? (int)q : kCoarse;   // (one without a token: its units are not read)
        }
        __syncthreads();
        const int unit = tid % kCoarse;
        u64 sum = 0;
#pragma unroll 5
        for (int c = tid / kCoarse; c < nc; c += kThreads / kCoarse) {
            const int b = unit - sh.off[c];                       // (every chunk reaches down to the last but one)
            uint32_t v = 0;
            if (b >= 0 && unit < kCoarse - 1)
                v = rs.k ? reinterpret_cast<const uint32_t *>(units)[c * kCoarse + b] : (uint32_t)(units[c * kCoarse + b] >> 28);
            sum += rs.k ? (u64)v : (u64)(__uint2float_rd(v) * sh.scale_lo[c]);
        }
        if (sum) add64(&sh.bins[unit], sum);
        __syncthreads();
        u64 acc = 0, val;
        const int bin = crossing(sh, rs.k ? rs.k : mass_target(rs.p, total) + 1, acc, val);
        if (bin >= 0 && fabsf(q0) < 4194304.f) from = q0 - (float)bin;
    }
    if (top == INFINITY) from = INFINITY;
    // ---------------- the candidates: z >= low, which is never above top
    float low = fmaxf(from / kPerUnit, -FLT_MAX);
    // (with top-k its tokens' whole mass is wanted; not in eighth units, which overflow for the largest tops)
    if (rs.floor44 && !rs.k) low = fmaxf(low, top - rs.reach());
    const int nv = view.vectors();
    list += (size_t)row * nc * kKept;
    __syncthreads();   // (sh.n is zero)
    gather(sh, view, list, nc, low, __uint_as_float(0x7fffffffu));
    __syncthreads();
    const int n = sh.n;
    if (n > kList && rs.by_mass() && !rs.floor44 && fabsf(q0) < 4194304.f &&
        draw_wide<TL>(sh, view, rs.p, a.u[row], a.token + row, a.prob + row, units, list, nc))
        return;
    if (n <= kSmall) {
        draw_small(a, sh, row, n, rs, total);
        return;
    }
    // f(z, id) for every candidate: from the list, or from the row again where it did not fit
    auto each = [&](auto &&f) {
        if (n <= kList) {
#pragma unroll 2
            for (int i = tid; i < n; i += kThreads) f(sh.z[i], sh.id[i]);
        } else {
            for (int v = tid; v < nv; v += kThreads) {
                float z[E];
                view.scaled(view.raw(v), z);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (z[e] >= low) f(z[e], (uint32_t)(v * E + e - view.mis));
            }
        }
    };
    draw_many(a, sh, row, rs, low, total, each);
}

int chunks_of(int V) { return (V + 7 + kChunk - 1) / kChunk; }   // (up to 7 tokens before the boundary)

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

int sample_max_vocab() { return kMaxVocab; }
int sample_launches(int V) { return V <= kChunk ? 1 : 2; }

size_t sample_ws_bytes(int rows, int V) {
    if (V <= kChunk) return 256;   // one launch, which has everything in shared memory
    const size_t n = (size_t)rows * chunks_of(V);
    return up256(n * sizeof(ChunkStat)) + up256(n * kCoarse * 8) + n * kKept * 8 + 256;   // room to align the caller's base
}

cudaError_t sample_tokens(const SampleArgs &a, int dtype, void *ws, cudaStream_t st) {
    if (a.rows <= 0) return cudaSuccess;
    const bool b16 = dtype == DLLM_BF16;
    const int nc = chunks_of(a.V);
    uint8_t *w = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(ws) + 255) & ~uintptr_t(255));
    ChunkStat *stat = reinterpret_cast<ChunkStat *>(w);
    w += up256((size_t)a.rows * nc * sizeof(ChunkStat));
    u64 *coarse = reinterpret_cast<u64 *>(w);
    uint2 *list = reinterpret_cast<uint2 *>(w + up256((size_t)a.rows * nc * kCoarse * 8));
    static bool configured[64] = {};   // per device: raise the shared-memory limit once
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        for (auto kern : {reinterpret_cast<const void *>(k_sample_draw<float>), reinterpret_cast<const void *>(k_sample_draw<bf16>),
                          reinterpret_cast<const void *>(k_sample_row<float>), reinterpret_cast<const void *>(k_sample_row<bf16>)}) {
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared));
            if (e != cudaSuccess) return e;
        }
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    // A row of one chunk leaves nothing to stream: one launch (V = 4096, one row: 16.1 us, two launches
    // 21.4 us).
    if (a.V <= kChunk)
        return launch_kernel(b16 ? k_sample_row<bf16> : k_sample_row<float>, dim3(a.rows), dim3(kThreads), sizeof(Shared), st, 1, a);
    cudaError_t e = launch_kernel(b16 ? k_sample_stats<bf16> : k_sample_stats<float>, dim3((unsigned)(a.rows * nc)), dim3(kStatThreads), 0, st,
                                  1, a, stat, coarse, list, nc);
    if (e != cudaSuccess) return e;
    return launch_kernel(b16 ? k_sample_draw<bf16> : k_sample_draw<float>, dim3(a.rows), dim3(kThreads), sizeof(Shared), st, 1,
                         a, stat, coarse, list, nc);
}

}  // namespace dllm
