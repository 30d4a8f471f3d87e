// paged_attention.cu -- attention of ragged new rows over a paged cache in fp32.
//
//   A[t, h] = softmax_j(<Q[t, h], K_j> scale) V_j  over the keys j < visible(pos(t))
//
// Work is cut as in paged_sched.cuh: units of 32 rows (token, head of the group) over 64-key
// tiles, two CTAs per SM (hd 64) or one.  Both products run on the tensor cores with every fp32
// operand split into two TF32 parts, x = hi + lo: hi is x rounded to 11 bits, lo the exact rest cut
// to 11 bits, so hi + lo is off by 2^-21 |x| at most, to either side.  Three of the four partial products
// are summed in fp32:
//   <q, k> = hi hi + hi lo + lo hi     (lo lo, 2^-22 of a product at most, is left out)
// which is about as near to 64 bits as fp32 multiply-adds are (1e-6 of the outputs' norm or less).  Sums of
// a tile start at zero and join the outputs by an fp32 addition: the tensor cores round their sums downwards,
// which over 2 10^5 keys came to 10^-5 (3 10^-7 now).
// Warp-level products (16 x 8 x 8) are taken rather than tcgen05's 128-row ones: a unit has 32 rows
// at most, the operands have to pass through registers to be split in any case, and outputs in
// registers are rescaled in place.
//
// A turn of the loop: S of tile t (16 rows x 16 keys per warp; the queries stay in registers, split)
// to shared memory, and O += P V of tile t - 1 (16 rows x hd / 4 dims per warp), which do not wait
// for one another; then the softmax of tile t by 8 threads per row (running maximum and sum in
// fp32), weights back split.  K of the next tile and V of this one come in by cp.async meanwhile.
// Units of 16 rows or fewer are another instance, whose warps take other keys and dims in place of
// the second 16 rows.
//
// Latency bounds short caches (4 x 2001 keys: 18% of the tensor pipe's cycles, 0.38 of the issue slots), products
// and splits long ones; single rows read K and V at 4 TB/s.  8 fp32 heads of 64 dims, 32 rows each, 4 x 2001
// keys: 28 us (fp32 multiply-adds: 36 us, bound by their operands' shared-memory reads); 16 x 8001
// keys: 194 us (299); 64 single rows, 28 heads on 4 of 128 dims, 4096 keys: 253 us (619).
#include "paged_sched.cuh"

namespace dllm {
namespace {

constexpr int kR = 32;        // rows of a unit
constexpr int kK = 64;        // keys of a tile
constexpr int kT = 256;       // threads: 8 warps

__device__ __forceinline__ void cp16(void *dst, const void *src, bool on) {   // zeros when off
    const int n = on ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

struct F32Args {
    PagedSched s;
    const float *Q, *Kp, *Vp;
    long long q_stride;
    float *A;
    float scale_log2;
};

template <int HD> struct F32Cfg {
    static constexpr int LK = HD + 16;                   // row pitches: no two lanes of an access meet in a bank
    static constexpr int LV = HD + 4, LP = kK + 8;       // (K: 16 bytes of 2 rows; V: rows 2c, 2c + 1; P: 8 bytes of 4 rows)
    static constexpr int kPerSm = HD == 64 ? 2 : 1;      // CTAs per SM (shared memory)
    static constexpr int kWords = 2 * kK * (LK + LV) + 3 * kR * LP + kR;
    static constexpr size_t kSmem = (size_t)kWords * 4 + 2 * kK;
};

// x = hi + lo in TF32 (see above).  cvt.rna.tf32 in place of the two whole-number operations cost 10%.
__device__ __forceinline__ void split(float x, uint32_t &hi, uint32_t &lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi)) & 0xffffe000u;
}
// d += a b: a 16 x 8 (rows lane / 4 and + 8; columns lane % 4 and + 4), b 8 x 8 (rows lane % 4 and + 4, column
// lane / 4), d 16 x 8 (rows as a; columns 2 (lane % 4) and + 1).
__device__ __forceinline__ void mma8(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// TWO: units of more than 16 rows.
template <int HD, bool TWO>
__global__ void __launch_bounds__(kT, F32Cfg<HD>::kPerSm) k_paged_attention_f32(const F32Args a) {
    using C = F32Cfg<HD>;
    constexpr int LK = C::LK, LV = C::LV, LP = C::LP, V4 = HD / 4;
    constexpr int NI = kK * V4 / kT;          // 16-byte pieces of K (and of V) that a thread loads per tile
    constexpr int NS = TWO ? 2 : 1;           // 8-key tiles of a warp's scores
    constexpr int NO = HD / (TWO ? 32 : 64);  // 8-dim tiles of a warp's outputs
    extern __shared__ __align__(16) float sm[];
    float *sK = sm, *sV = sK + 2 * kK * LK;   // [2][kK] rows each
    float *sS = sV + 2 * kK * LV;             // scores
    float *sP = sS + kR * LP;                 // weights: hi, lo
    float *sF = sP + 2 * kR * LP;             // per row: the tile's rescaling; at the end 1 / sum
    uint8_t *pages = reinterpret_cast<uint8_t *>(sF + kR);   // key has a page, of two tiles
    __shared__ __align__(16) int w0[8];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    static_assert((kPagedMaxSeqs + 1) * 8 <= 2 * kK * LK * 4, "the schedule's sums fit the idle K ring");
    griddep_wait();
    griddep_launch();
    schedule_start(a.s, reinterpret_cast<long long *>(sm), w0);
    __syncthreads();
    const long long chunk = *reinterpret_cast<const long long *>(w0 + 6);
    Walker wk = walk_from(a.s, w0);
    if (tid == 0) a.s.meta[blockIdx.x].nseg = 0;
    const int G = a.s.G, lg = a.s.sq.page_log2;
    const int fr = lane >> 2, fc = lane & 3;         // this lane's row and column of the products' operands
    const int row = tid >> 3, part = tid & 7;        // softmax: keys 4 part .. + 3 and 32 + 4 part .. + 3
    const int lj = tid / V4, le = (tid % V4) * 4;    // loads: key lj + (kT / V4) i, dims le ..
    // 16 rows x 16 keys and x hd / 4 dims per warp (TWO), or 16 rows x 8 keys and x hd / 8 dims
    const int mt = TWO ? warp & 1 : 0, n0 = (TWO ? warp >> 1 : warp) * NS, o0 = (TWO ? warp >> 1 : warp) * NO;
    const unsigned stride = (unsigned)a.s.n_kv * HD;
    bool first = true;
    Seg sg;
    while (wk.next(a.s, sg)) {
        const int32_t *tab = a.s.sq.page_table + (size_t)sg.b * a.s.sq.max_pages;
        const float *gK = a.Kp + (size_t)sg.g * HD + le, *gV = a.Vp + (size_t)sg.g * HD + le;
        int ids[NI];                                 // pages of the next tile of K to load
        unsigned at[NI];                             // pool rows of the last one (~0: none), for its V
        auto look = [&](int kt) {
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int key = kt * kK + lj + i * (kT / V4);
                ids[i] = key < sg.len ? tab[key >> lg] : -1;
            }
        };
        auto load_k = [&](int kt) {
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int j = lj + i * (kT / V4);
                const bool on = (unsigned)ids[i] < (unsigned)a.s.sq.n_pages;
                at[i] = on ? ((unsigned)ids[i] << lg) + ((kt * kK + j) & ((1 << lg) - 1)) : ~0u;
                cp16(sK + ((kt & 1) * kK + j) * LK + le, gK + (size_t)(on ? at[i] : 0) * stride, on);
                if (le == 0) pages[(kt & 1) * kK + j] = on;
            }
        };
        auto load_v = [&](int kt) {
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const bool on = at[i] != ~0u;
                cp16(sV + ((kt & 1) * kK + lj + i * (kT / V4)) * LV + le, gV + (size_t)(on ? at[i] : 0) * stride, on);
            }
        };
        look(sg.k0);
        float4 qv[2][HD / 16];                       // under way while the first keys are asked for
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int rw = sg.row0 + min(mt * 16 + fr + 8 * x, sg.nrows - 1);   // (rows past the unit's: copies, never written)
            const float *q = a.Q + (size_t)(sg.start + rw / G) * a.q_stride + (size_t)(sg.g * G + rw % G) * HD + 4 * fc;
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) qv[x][kk] = *reinterpret_cast<const float4 *>(q + 16 * kk);
        }
        __syncthreads();   // the previous segment (or the schedule) is done with shared memory
        load_k(sg.k0);
        cp_commit();
        if (sg.k0 + 1 < sg.k1) look(sg.k0 + 1);
        uint32_t qh[HD / 16][2][4], ql[HD / 16][2][4];   // dims 16 kk + 4 fc + e: columns fc (e even) and fc + 4 of product e / 2
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) {
                split(qv[x][kk].x, qh[kk][0][x], ql[kk][0][x]);
                split(qv[x][kk].y, qh[kk][0][2 + x], ql[kk][0][2 + x]);
                split(qv[x][kk].z, qh[kk][1][x], ql[kk][1][x]);
                split(qv[x][kk].w, qh[kk][1][2 + x], ql[kk][1][2 + x]);
            }
        const int lim = row < sg.nrows ? PagedSeqs::visible(sg.pos0 + (sg.row0 + row) / G, sg.len, a.s.mask_block) : 0;
        float m = -INFINITY, l = 0.f;
        float o[NO][4] = {};
        // turn kt: S of tile kt and O of tile kt - 1, then the softmax of tile kt
        for (int kt = sg.k0; kt <= sg.k1; ++kt) {
            cp_wait<0>();
            __syncthreads();                     // K of kt and V of kt - 1 are here, its weights too; the rings' other halves are free
            if (kt < sg.k1) {
                load_v(kt);
                if (kt + 1 < sg.k1) {
                    load_k(kt + 1);
                    if (kt + 2 < sg.k1) look(kt + 2);
                }
                cp_commit();
                // ---- S
                const float *kb = sK + ((kt & 1) * kK + n0 * 8 + fr) * LK + 4 * fc;
                float s[NS][4] = {}, z[NS][4] = {};   // hi hi; the rest (products that do not wait for one another)
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk)
#pragma unroll
                    for (int j = 0; j < NS; ++j) {
                        const float4 v = *reinterpret_cast<const float4 *>(kb + j * 8 * LK + 16 * kk);
                        uint32_t h[4], w[4];
                        split(v.x, h[0], w[0]);
                        split(v.y, h[1], w[1]);
                        split(v.z, h[2], w[2]);
                        split(v.w, h[3], w[3]);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            mma8(z[j], ql[kk][x], h[2 * x], h[2 * x + 1]);
                            mma8(z[j], qh[kk][x], w[2 * x], w[2 * x + 1]);
                            mma8(s[j], qh[kk][x], h[2 * x], h[2 * x + 1]);
                        }
                    }
#pragma unroll
                for (int j = 0; j < NS; ++j) {
                    float *d = sS + (mt * 16 + fr) * LP + (n0 + j) * 8 + 2 * fc;
                    *reinterpret_cast<float2 *>(d) = make_float2(s[j][0] + z[j][0], s[j][1] + z[j][1]);
                    *reinterpret_cast<float2 *>(d + 8 * LP) = make_float2(s[j][2] + z[j][2], s[j][3] + z[j][3]);
                }
            }
            if (kt > sg.k0) {   // ---- O
                const float f0 = sF[mt * 16 + fr], f1 = sF[mt * 16 + fr + 8];   // (rows past the unit's: anything, never written)
                float y[NO][4] = {};
                const float *vb = sV + (((kt - 1) & 1) * kK + 2 * fc) * LV + o0 * 8 + fr;
                const uint32_t *pb = reinterpret_cast<const uint32_t *>(sP) + (mt * 16 + fr) * LP + 2 * fc;
#pragma unroll 4
                for (int ks = 0; ks < 8; ++ks) {
                    uint32_t h[4], w[4];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint2 ph = *reinterpret_cast<const uint2 *>(pb + x * 8 * LP + 8 * ks);
                        const uint2 pl = *reinterpret_cast<const uint2 *>(pb + (kR + x * 8) * LP + 8 * ks);
                        h[x] = ph.x;
                        h[2 + x] = ph.y;
                        w[x] = pl.x;
                        w[2 + x] = pl.y;
                    }
#pragma unroll
                    for (int j = 0; j < NO; ++j) {
                        uint32_t vh0, vl0, vh1, vl1;
                        split(vb[8 * ks * LV + 8 * j], vh0, vl0);
                        split(vb[(8 * ks + 1) * LV + 8 * j], vh1, vl1);
                        mma8(y[j], w, vh0, vh1);
                        mma8(y[j], h, vl0, vl1);
                        mma8(y[j], h, vh0, vh1);
                    }
                }
#pragma unroll
                for (int j = 0; j < NO; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[j][e] = fmaf(o[j][e], e < 2 ? f0 : f1, y[j][e]);
            }
            if (kt == sg.k1) break;
            __syncthreads();
            // ---- softmax
            if (row < sg.nrows) {                // (8 lanes of a row together)
                const unsigned mask = 0xffu << (lane & 24);
                float *p = sP + row * LP + 4 * part;
                const uint8_t *here = pages + (kt & 1) * kK + 4 * part;
                float s[8];
                const float *raw = sS + row * LP + 4 * part;
                *reinterpret_cast<float4 *>(s) = *reinterpret_cast<const float4 *>(raw);
                *reinterpret_cast<float4 *>(s + 4) = *reinterpret_cast<const float4 *>(raw + 32);
                const uint32_t on0 = *reinterpret_cast<const uint32_t *>(here), on1 = *reinterpret_cast<const uint32_t *>(here + 32);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[e] *= a.scale_log2;
                if ((kt + 1) * kK > lim || (on0 & on1) != 0x01010101u) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int key = kt * kK + 4 * part + (e & 3) + (e >> 2) * 32;
                        if (key >= lim || !(((e < 4 ? on0 : on1) >> (8 * (e & 3))) & 1)) s[e] = -INFINITY;
                    }
                }
                float mx = s[0];
#pragma unroll
                for (int e = 1; e < 8; ++e) mx = fmaxf(mx, s[e]);
#pragma unroll
                for (int c = 4; c > 0; c >>= 1) mx = fmaxf(mx, __shfl_xor_sync(mask, mx, c));
                const float mn = fmaxf(m, mx);
                const float f = mn == -INFINITY ? 1.f : ex2(m - mn);
                const float ref = mn == -INFINITY ? 0.f : mn;
                uint32_t h[8], w[8];
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x = ex2(s[e] - ref);
                    sum += x;
                    split(x, h[e], w[e]);
                }
                l = l * f + sum;                 // this thread's keys
                m = mn;
                *reinterpret_cast<uint4 *>(p) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4 *>(p + 32) = make_uint4(h[4], h[5], h[6], h[7]);
                *reinterpret_cast<uint4 *>(p + kR * LP) = make_uint4(w[0], w[1], w[2], w[3]);
                *reinterpret_cast<uint4 *>(p + kR * LP + 32) = make_uint4(w[4], w[5], w[6], w[7]);
                if (part == 0) sF[row] = f;
            }
        }
        const bool whole = sg.k0 == 0 && sg.k1 == sg.n;
        const int slot = blockIdx.x * 2 + (first ? 0 : 1);
        first = false;
        if (tid == 0 && sg.k0 == 0 && !whole) a.s.meta[blockIdx.x] = part_of(sg, slot, chunk);
        float L = l;
#pragma unroll
        for (int c = 4; c > 0; c >>= 1) L += __shfl_xor_sync(0xffffffffu, L, c);
        __syncthreads();                         // the rescalings have been read
        if (part == 0 && row < sg.nrows) {
            sF[row] = !whole ? 1.f : L == 0.f ? 0.f : 1.0f / L;
            const int rw = sg.row0 + row;
            if (!whole) a.s.part_ml[(size_t)slot * a.s.unit_rows + row] = make_float2(m, L);
            else if (a.s.lse)
                a.s.lse[(size_t)(sg.start + rw / G) * a.s.n_q + sg.g * G + rw % G] = row_lse(m, L);
        }
        __syncthreads();
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int r = mt * 16 + fr + 8 * x;
            if (r >= sg.nrows) continue;
            const float f = sF[r];
            const int rw = sg.row0 + r;
            const size_t out = (size_t)(sg.start + rw / G) * a.s.n_q + sg.g * G + rw % G;
            float *dst = (whole ? a.A + out * HD : a.s.part_o + ((size_t)slot * a.s.unit_rows + r) * HD) + 2 * fc;
#pragma unroll
            for (int j = 0; j < NO; ++j)
                *reinterpret_cast<float2 *>(dst + (o0 + j) * 8) = make_float2(o[j][2 * x] * f, o[j][2 * x + 1] * f);
        }
    }
}

int f32_rows(int max_new, int G) {
    const long long r = (long long)max_new * G;
    return r < kR ? (int)r : kR;
}

template <int HD, bool TWO>
cudaError_t launch_f32(const F32Args &a, int grid, cudaStream_t st) {
    static bool configured[64] = {};   // per device: raise the shared-memory limit once
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(k_paged_attention_f32<HD, TWO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)F32Cfg<HD>::kSmem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    const cudaError_t e = launch_kernel(k_paged_attention_f32<HD, TWO>, dim3(grid), dim3(kT), F32Cfg<HD>::kSmem, st, 1, a);
    return e != cudaSuccess ? e : paged_join<float, HD>(a.s, grid, a.A, st);
}

}  // namespace

size_t paged_attention_f32_ws_bytes(int max_new, int n_q, int n_kv, int hd) {
    return paged_part_bytes((hd == 64 ? F32Cfg<64>::kPerSm : F32Cfg<128>::kPerSm) * num_sms(), f32_rows(max_new, n_q / n_kv), hd);
}

cudaError_t paged_attention_f32(const PagedAttn &p, void *ws, cudaStream_t st) {
    const int grid = (p.hd == 64 ? F32Cfg<64>::kPerSm : F32Cfg<128>::kPerSm) * num_sms();
    F32Args a{};
    a.s = paged_sched(p, grid, f32_rows(p.max_new, p.n_q / p.n_kv), kK, ws);
    a.Q = static_cast<const float *>(p.Q);
    a.Kp = static_cast<const float *>(p.k_pages);
    a.Vp = static_cast<const float *>(p.v_pages);
    a.q_stride = p.q_stride;
    a.A = static_cast<float *>(p.A);
    a.scale_log2 = p.scale * 1.4426950408889634f;
    // (64 single rows over 4096 keys with 7 rows a unit: 253 us, 381 in the instance for 32; with 3: 129, 188)
    if (a.s.unit_rows > 16)
        return p.hd == 128 ? launch_f32<128, true>(a, grid, st) : launch_f32<64, true>(a, grid, st);
    return p.hd == 128 ? launch_f32<128, false>(a, grid, st) : launch_f32<64, false>(a, grid, st);
}

}  // namespace dllm
