// paged_attention_f8.cu -- attention of ragged new rows over 8-bit pages on the sm_103a tensor
// cores: E4M3 codes with a power-of-two scale for each page and head, 2^k for keys, 2^v for values.
//
//   A[t, h] = sum_j w_j 2^{v_j} V_j / sum_j w_j,   w_j = 2^(c 2^{k_j} <Q[t, h], K_j>)
//
// The codes are fed to the tensor cores as they lie in the pages (kind::f8f6f4, twice the rate
// of bf16); nothing is widened.  The other operand of each product is two E4M3 numbers:
//   q 2^-e    = q1 + q2 / 32      (a bf16 query has 8 bits, an E4M3 number 4: exact but for what lies
//                                  2^-22 below the row's largest element, which 2^e brings to [128, 256))
//   w' 2^-m   = w1 + w2 / 32      (8 bits of each weight; floor 2^-19 of the row's largest)
// so a product costs what it does in bf16 and reads half the bytes.  Both parts stand side by side
// in the N dimension:
//   S^T [128 keys, q1 rows | q2 rows]  =  K [128 keys, hd]   [q1 | q2]^T
//   O^T [hd, w1 rows | w2 rows]       += V^T [hd, 128 keys]  [w1 | w2]
// Keys and dims are the 128 lanes, rows the columns: a few rows cost a few columns, a thread
// has one key, and the key's scales, presence and position are values of its own.  The value's scale
// goes into the weight before it is rounded, w' = w 2^v, and the running reference m is that of
// c s + v, so that what is rounded to 8 bits is what counts in the result; the sum of w is kept in
// fp32 without it.  m moves (O and sums rescaled) when a weight would pass 2^8, that is when a score
// exceeds the row's largest so far by 4 in log2.
//
// Work is cut as in paged_sched.cuh, one CTA per SM.  A unit has up to R rows of a sequence and key
// head.  Streams work through key tiles in turn, each with an S^T, an O^T and weights of its own, so that the
// tensor cores and the loads run on while a stream's softmax does:
//   R = 8, 16, 32:  4 streams of 4 warps;     R = 64: 2 streams of 8 warps (32 rows each four);
//   SHARE (R = 64): 2 streams with 64 rows each of a unit of 128, sharing every K and V tile.
// The streams' (O, m, sum) are joined at the end of a slice.
//
// Threads: warp 0 TMA, warp 1 MMA issue, warps 2 and 3 split the queries, then 16 softmax warps:
// thread = key of the tile.
#include <climits>

#include "e4m3.cuh"
#include "paged_sched.cuh"
#include "paged_tc.cuh"

namespace dllm {
namespace {

constexpr int kTile = 128;              // keys of a tile
constexpr int kThreads = 128 + 512;
constexpr float kTop = 8.f;             // log2 of the largest weight
constexpr float kSlack = 4.f;           // the reference puts a row's largest weight this far below it
constexpr float kNoRef = 3e38f;         // minus the reference of a row that has seen no key

struct F8Args {
    PagedSched s;
    bf16 *A;
    const bf16 *Q;
    long long q_stride;
    const uint8_t *k_scale, *v_scale;   // [n_pages, n_kv]
    int box, boxes;                     // keys of a TMA box and boxes of a tile
    float scale_log2;
};

struct RingSeg {
    Seg s;
    int go;             // 0: no more
};

template <int HD, int R, bool SHARE> struct Cfg {
    static constexpr int NS = SHARE ? 2 : (R == 64 ? 2 : 4);   // streams
    static constexpr int RT = R < 32 ? R : 32;                 // rows of a thread
    static constexpr int CH = RT < 16 ? RT : 16;               // rows that it has in registers at a time
    static constexpr int GS = R / RT;                          // groups (of 4 warps) of a stream
    static constexpr int UR = SHARE ? 128 : R;                 // rows of a unit
    static constexpr int N = 2 * R;                            // columns of a stream's products
    static constexpr int AHEAD = SHARE ? 1 : NS;               // tiles by which K runs ahead of V
    static constexpr int TB = kTile * HD;                      // bytes of a tile
    static constexpr int WROW = N < 32 ? 32 : N;               // bytes of a key's weights
    static constexpr int WB = kTile * WROW;
    static constexpr int QB = (SHARE ? 2 : 1) * N * HD;        // bytes of a unit's queries
    static constexpr int WORDS = 4 * UR /* rs, lim: two buffers */ + 4 * RT + 16 * RT /* xm */ + 16 * RT /* sums */ +
                                 (SHARE ? 1 : NS) * UR + 2 * UR;
    static constexpr int FIX = 2 * QB + NS * WB + WORDS * 4 + 1024;
    static constexpr int SLOTS = (227 * 1024 - FIX) / TB < 20 ? (227 * 1024 - FIX) / TB : 20;
    static constexpr int BARS = 2 * 2 + 2 * SLOTS + 2 * NS + 1 + 2 * kSegs;
    static constexpr size_t kSmem = 2 * QB + NS * WB + (size_t)SLOTS * TB + WORDS * 4 + BARS * 8 + 64 + kSegs * (int)sizeof(RingSeg);
    static_assert(kSmem <= 227 * 1024 && SLOTS >= AHEAD + 3, "shared memory");
};

// kind::f8f6f4, both operands E4M3, fp32 D.  Bits as in idesc_bf16 with formats 0; 15 and 16: A, B MN-major.
constexpr uint32_t idesc_e4m3(int N, int mn_major) {
    return (1u << 4) | (uint32_t(mn_major) << 15) | (uint32_t(mn_major) << 16) | (uint32_t(N >> 3) << 17) | (uint32_t(128 >> 4) << 24);
}
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
}
// Descriptor of rows of `ROW` bytes swizzled within them (128-, 64- or 32-byte mode), 8 rows a group.
// K-major: the rows are M or N; MN-major: the rows are K.  No operand here is wider than a row but
// A = V^T of 64 dims, whose second half (leading offset 0) repeats the first.
template <int ROW> __device__ __forceinline__ uint64_t smem_desc_rows(uint32_t saddr) {
    constexpr uint64_t mode = ROW == 128 ? 2 : (ROW == 64 ? 4 : 6);
    uint64_t d = 0;
    d |= uint64_t((saddr & 0x3FFFFu) >> 4);
    d |= uint64_t((8 * ROW) >> 4) << 32;
    d |= uint64_t(1) << 46;
    d |= mode << 61;
    return d;
}
// Byte offset of 16-byte unit u of row r in that layout.
template <int ROW> __device__ __forceinline__ int row_unit(int r, int u) {
    return r * ROW + ((u ^ ((r * ROW >> 7) & (ROW / 16 - 1))) << 4);
}

// 32 lanes x C consecutive columns; readable after tmem_ld_wait_n on the same array.
template <int C> __device__ __forceinline__ void tmem_ld_n(uint32_t taddr, float *v) {
    if constexpr (C == 2) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "r"(taddr));
    } else if constexpr (C == 4) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(taddr));
    } else if constexpr (C == 8) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                     : "r"(taddr));
    } else {
        static_assert(C == 16);
        tmem_ld_x16(taddr, slice16(v));
    }
}
template <int C> __device__ __forceinline__ void tmem_ld_wait_n(float *v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < C; ++i) asm volatile("" : "+f"(v[i]));   // (no use of them moves above the wait)
}
template <int C> __device__ __forceinline__ void tmem_st_n(uint32_t taddr, const float *v) {
    if constexpr (C == 8) {
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "f"(v[0]),
                     "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                     : "memory");
    } else {
        static_assert(C == 16);
        uint32_t b[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) b[i] = __float_as_uint(v[i]);
        tmem_st_x16(taddr, b);
    }
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
// Named barrier that also tells whether any thread's flag is set.
__device__ __forceinline__ bool bar_any(int id, int nthreads, bool flag) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "barrier.cta.red.or.pred p, %2, %3, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)flag), "r"(id), "r"(nthreads)
        : "memory");
    return r != 0;
}
// Sums over the warp of C values a lane; lane l receives that of value l * C / 32.
template <int C> __device__ __forceinline__ float warp_sums(float (&v)[C], int lane) {
    int cnt = C;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (cnt > 1) {
            cnt >>= 1;
#pragma unroll
            for (int k = 0; k < C / 2; ++k)
                if (k < cnt) {
                    const float give = (lane & o) ? v[k] : v[k + cnt], keep = (lane & o) ? v[k + cnt] : v[k];
                    v[k] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        }
    }
    return v[0];
}

template <int HD, int R, bool SHARE>
__global__ void __launch_bounds__(kThreads, 1)
    k_paged_attention_f8(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const F8Args a,
                         unsigned *status) {
    using C = Cfg<HD, R, SHARE>;
    constexpr int SLOTS = C::SLOTS, TB = C::TB, NS = C::NS, RT = C::RT, CH = C::CH, UR = C::UR, N = C::N, WROW = C::WROW;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *ring = smem;
    uint8_t *sQ = ring + SLOTS * TB;                                // two units' queries
    uint8_t *sW = sQ + 2 * C::QB;                                   // the streams' weights
    float *rs = reinterpret_cast<float *>(sW + NS * C::WB);         // [2][UR] scale of a row's query
    int *lims = reinterpret_cast<int *>(rs + 2 * UR);               // [2][UR] keys that a row sees
    float *nm = reinterpret_cast<float *>(lims + 2 * UR);           // [4 groups][RT] minus the reference
    float *xm = nm + 4 * RT;                                        // [4][4 warps][RT] maxima
    float *ls = xm + 16 * RT;                                       // [4][4][RT] sums
    float *fj = ls + 16 * RT;                                       // [streams][UR] factors of the join
    float *Lr = fj + (SHARE ? 1 : NS) * UR, *Mr = Lr + UR;          // [UR]
    uint64_t *bars = reinterpret_cast<uint64_t *>(Mr + UR);
    uint64_t *q_full = bars, *q_empty = bars + 2;
    uint64_t *full = bars + 4, *empty = full + SLOTS;
    uint64_t *s_full = empty + SLOTS, *p_full = s_full + NS, *o_full = p_full + NS;
    uint64_t *seg_full = o_full + 1, *seg_empty = seg_full + kSegs;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + C::BARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *w0 = reinterpret_cast<int *>(tmem_slot + 2);               // the walker's start
    RingSeg *segs = reinterpret_cast<RingSeg *>(tmem_slot + 14);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (smem_u32(smem) & 1023u) {   // the swizzled tiles need it; the same in every CTA
        if (tid == 0) raise_status(status, DLLM_STATUS_SMEM_LAYOUT);
        griddep_wait();
        if (tid == 0) a.s.meta[blockIdx.x].nseg = 0;
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 2);
            mbar_init(&q_empty[i], 1 + 16);     // MMA thread, softmax warps
        }
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < NS; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4 * C::GS);
        }
        mbar_init(o_full, 1);
        for (int i = 0; i < kSegs; ++i) {
            mbar_init(&seg_full[i], 1);
            mbar_init(&seg_empty[i], 1 + 2 + 16);   // MMA thread, query warps, softmax warps
        }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    griddep_wait();
    griddep_launch();
    schedule_start(a.s, reinterpret_cast<long long *>(ring), w0);   // (in the idle ring)
    fence_async_smem();   // the ring's generic writes before TMA's
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const long long chunk = *reinterpret_cast<const long long *>(w0 + 6);
    // Slice k, or null at the end.  The wait does not look at the abort flag and lasts longer than the
    // others: the TMA warp hands out a slice, or the end, in any case, and warps that meet at
    // named barriers must not part.
    auto seg_at = [&](uint32_t k) -> const RingSeg * {
        for (int tries = 0; tries < 4; ++tries)
            if (mbar_drain_ok(&seg_full[k % kSegs], (k / kSegs) & 1)) {
                const RingSeg *r = &segs[k % kSegs];
                return r->go ? r : nullptr;
            }
        return nullptr;
    };
    // Where in the ring's order a slice of n tiles has its K and V tiles: AHEAD K tiles, then V(t), K(t + AHEAD)
    auto k_at = [](int t, int n) -> uint32_t { return t < C::AHEAD ? t : 2 * t - C::AHEAD + 1; };
    auto v_at = [](int t, int n) -> uint32_t { return min(C::AHEAD, n) + t + min(t, max(n - C::AHEAD, 0)); };

    if (warp == 0) {
        // ---------------- TMA producer: lane = box of a tile
        uint32_t seq = 0, sk = 0;
        bool ok = true;
        Walker wk = walk_from(a.s, w0);
        const int page_log2 = a.s.sq.page_log2;
        const int absent = a.s.sq.n_pages << page_log2;          // a row outside the pool: zeros
        const int in_page = (lane * a.box) & ((1 << page_log2) - 1);   // (tiles start on pages, or pages hold tiles)
        for (;; ++sk) {
            Seg sg{};
            const bool go = wk.next(a.s, sg) && ok;
            if (lane == 0) {
                mbar_drain(&seg_empty[sk % kSegs], ((sk / kSegs) & 1) ^ 1);
                segs[sk % kSegs] = RingSeg{sg, go};
                mbar_arrive(&seg_full[sk % kSegs]);
            }
            __syncwarp();
            if (!go) break;
            const int n = sg.k1 - sg.k0;
            const int32_t *tab = a.s.sq.page_table + (size_t)sg.b * a.s.sq.max_pages;
            // Page of this lane's box of a tile (-1: none, or past the keys); the value is first looked at
            // when the box is loaded, a tile later.
            auto page_of = [&](int tile) -> int {
                const int key = (sg.k0 + tile) * kTile + lane * a.box;
                return lane < a.boxes && tile < n && key < sg.len ? tab[key >> page_log2] : -1;
            };
            auto row_of = [&](int tile, int id) -> int {                 // pool row
                if ((unsigned)id >= (unsigned)a.s.sq.n_pages) return absent;
                const int off = page_log2 > 7 ? ((sg.k0 + tile) * kTile) & ((1 << page_log2) - 1) : 0;
                return (id << page_log2) + in_page + off;
            };
            auto load = [&](const CUtensorMap *tm, int row) -> bool {
                const uint32_t s = seq % SLOTS, ph = (seq / SLOTS) & 1;
                bool go = true;
                if (lane == 0) {
                    go = mbar_wait(&empty[s], ph ^ 1, abort_flag, status);
                    if (go) mbar_arrive_expect_tx(&full[s], TB);
                }
                go = __shfl_sync(0xffffffffu, go, 0);
                if (!go) return false;
                if (lane < a.boxes) tma_load_3d(ring + s * TB + lane * a.box * HD, tm, &full[s], 0, sg.g, row);
                ++seq;
                return true;
            };
            int ids[C::AHEAD + 1];
#pragma unroll
            for (int j = 0; j <= C::AHEAD; ++j) ids[j] = page_of(j);
#pragma unroll
            for (int j = 0; j < C::AHEAD; ++j)
                if (ok && j < n) ok = load(&tmK, row_of(j, ids[j]));
            for (int t = 0; ok && t < n; ++t) {
                const int later = page_of(t + C::AHEAD + 1);
                ok = load(&tmV, row_of(t, ids[0]));
                if (ok && t + C::AHEAD < n) ok = load(&tmK, row_of(t + C::AHEAD, ids[C::AHEAD]));
#pragma unroll
                for (int j = 0; j < C::AHEAD; ++j) ids[j] = ids[j + 1];
                ids[C::AHEAD] = later;
            }
        }
        if (lane == 0 && *abort_flag)   // every issued copy must land before the CTA can exit
            for (uint32_t i = seq > SLOTS ? seq - SLOTS : 0; i < seq; ++i) mbar_drain(&full[i % SLOTS], (i / SLOTS) & 1);
    } else if (warp == 1) {
        if (lane == 0) {   // ---------------- MMA issuer
            const uint32_t aq = smem_u32(sQ), ar = smem_u32(ring), aw = smem_u32(sW);
            uint32_t seq = 0, pn[NS] = {};
            bool ok = true;
            auto take = [&](uint32_t q) -> bool { return mbar_wait(&full[q % SLOTS], (q / SLOTS) & 1, abort_flag, status); };
            for (uint32_t sk = 0;; ++sk) {
                const RingSeg *rsg = seg_at(sk);
                if (!rsg) break;
                const int n = rsg->s.k1 - rsg->s.k0;
                mbar_arrive(&seg_empty[sk % kSegs]);
                if (!ok) continue;   // (aborted: only takes the slices off the ring)
                ok = mbar_wait(&q_full[sk & 1], (sk >> 1) & 1, abort_flag, status);
                const uint32_t qb = aq + (sk & 1) * C::QB;
                auto issue_s = [&](int i, uint32_t q, bool last) {
                    const uint32_t kb = ar + (q % SLOTS) * TB;
#pragma unroll
                    for (int kk = 0; kk < HD / 32; ++kk)
                        mma_e4m3(tmem + i * N, smem_desc_rows<HD>(kb + kk * 32),
                                 smem_desc_rows<HD>(qb + (SHARE ? i * N * HD : 0) + kk * 32), idesc_e4m3(N, 0), kk > 0);
                    mma_commit(&s_full[i]);
                    if (last) mma_commit(&empty[q % SLOTS]);
                };
                auto issue_pv = [&](int i, uint32_t q, bool first, bool last) {
                    const uint32_t vb = ar + (q % SLOTS) * TB;
#pragma unroll
                    for (int kk = 0; kk < kTile / 32; ++kk)
                        mma_e4m3(tmem + (NS + i) * N, smem_desc_rows<HD>(vb + kk * 32 * HD),
                                 smem_desc_rows<WROW>(aw + i * C::WB + kk * 32 * WROW), idesc_e4m3(N, 1), !first || kk > 0);
                    if (last) mma_commit(&empty[q % SLOTS]);
                };
                if (SHARE) {
                    if (ok) ok = take(seq);
                    if (ok) {
                        tc_fence_after();
                        issue_s(0, seq, false);
                        issue_s(1, seq, true);
                    }
                    for (int t = 0; ok && t < n; ++t) {
                        const bool more = t + 1 < n;
                        for (int i = 0; ok && i < 2; ++i) {
                            ok = mbar_wait(&p_full[i], pn[i] & 1, abort_flag, status);
                            ++pn[i];
                            if (ok && i == 0) ok = take(seq + v_at(t, n));
                            if (ok && i == 0 && more) ok = take(seq + k_at(t + 1, n));
                            if (!ok) break;
                            tc_fence_after();
                            issue_pv(i, seq + v_at(t, n), t == 0, i == 1);
                            if (more) issue_s(i, seq + k_at(t + 1, n), i == 1);
                        }
                    }
                } else {
                    for (int t = 0; ok && t < NS && t < n; ++t) {
                        ok = take(seq + t);
                        if (!ok) break;
                        tc_fence_after();
                        issue_s(t, seq + t, true);
                    }
                    int i = 0;
                    for (int t = 0; ok && t < n; ++t) {
                        ok = mbar_wait(&p_full[i], pn[i] & 1, abort_flag, status);
                        ++pn[i];
                        if (ok) ok = take(seq + v_at(t, n));
                        if (!ok) break;
                        tc_fence_after();
                        issue_pv(i, seq + v_at(t, n), t < NS, true);
                        if (t + NS < n) {
                            ok = take(seq + k_at(t + NS, n));
                            if (!ok) break;
                            tc_fence_after();
                            issue_s(i, seq + k_at(t + NS, n), true);
                        }
                        i = i + 1 == NS ? 0 : i + 1;
                    }
                }
                if (!ok) continue;
                seq += 2 * n;
                mma_commit(&q_empty[sk & 1]);
                mma_commit(o_full);
            }
            if (!ok) {   // nothing of this thread may still run when TMEM is freed
                mma_commit(&s_full[0]);
                mbar_drain(&s_full[0], 0);
                mbar_drain(&s_full[0], 1);
            }
        }
    } else if (warp < 4) {
        // ---------------- queries: two E4M3 numbers an element, the row's power of two beside them
        constexpr int E = HD / 32;                       // elements of a lane
        bool ok = true;
        for (uint32_t sk = 0;; ++sk) {
            const RingSeg *rsg = seg_at(sk);
            if (!rsg) break;
            const Seg sg = rsg->s;
            __syncwarp();
            if (lane == 0) mbar_arrive(&seg_empty[sk % kSegs]);
            if (ok) ok = mbar_wait(&q_empty[sk & 1], ((sk >> 1) & 1) ^ 1, abort_flag, status);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) continue;
            uint8_t *qb = sQ + (sk & 1) * C::QB;
            constexpr int AT = UR < 16 ? UR / 2 : 8;     // rows at a time
#pragma unroll 1
            for (int u0 = (warp - 2) * AT; u0 < UR; u0 += 2 * AT) {
                uint32_t raw[AT][E / 2];
#pragma unroll
                for (int j = 0; j < AT; ++j) {
                    const int ur = u0 + j, row = sg.row0 + ur, tok = row / a.s.G;
                    const bool live = ur < sg.nrows;
                    const bf16 *p = a.Q + (size_t)(sg.start + tok) * a.q_stride + (size_t)(sg.g * a.s.G + row - tok * a.s.G) * HD;
#pragma unroll
                    for (int e = 0; e < E / 2; ++e)
                        raw[j][e] = live ? reinterpret_cast<const uint32_t *>(p)[lane * (E / 2) + e] : 0u;
                    if (lane == 0)
                        lims[(sk & 1) * UR + ur] = live ? PagedSeqs::visible(sg.pos0 + tok, sg.len, a.s.mask_block) : INT_MAX;
                }
#pragma unroll
                for (int j = 0; j < AT; ++j) {
                    const int ur = u0 + j;
                    uint32_t top = 0;                    // magnitude bits: NaN above infinity above all others
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) top = max(top, max(raw[j][e] & 0x7fffu, (raw[j][e] >> 16) & 0x7fffu));
                    top = __reduce_max_sync(0xffffffffu, top);
                    const int ex = min(max((int)(top >> 7), 10), 254);      // biased exponent of the largest
                    const float f = __uint_as_float((uint32_t)(261 - ex) << 23);   // 2^(7 - (ex - 127))
                    if (lane == 0)   // a query that is not finite gives NaN
                        rs[(sk & 1) * UR + ur] = top >= 0x7f80u ? NAN : __uint_as_float((uint32_t)max(ex - 7, 1) << 23);
                    uint32_t c1 = 0, c2 = 0;
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) {
                        const float x = __uint_as_float(raw[j][e] << 16) * f, y = __uint_as_float(raw[j][e] & 0xffff0000u) * f;
                        const uint32_t c = e4m3x2(x, y);
                        const float2 b = f32_of_e4m3x2(c);
                        c1 |= c << (16 * e);
                        c2 |= e4m3x2((x - b.x) * 32.f, (y - b.y) * 32.f) << (16 * e);
                    }
                    const int n1 = SHARE ? (ur >> 6) * N + (ur & 63) : ur;   // row of the operand; R further: the second part
                    const int at = lane * E;
                    uint8_t *d1 = qb + row_unit<HD>(n1, at >> 4) + (at & 15), *d2 = qb + row_unit<HD>(n1 + R, at >> 4) + (at & 15);
                    if (E == 4) {
                        *reinterpret_cast<uint32_t *>(d1) = c1;
                        *reinterpret_cast<uint32_t *>(d2) = c2;
                    } else {
                        *reinterpret_cast<uint16_t *>(d1) = (uint16_t)c1;
                        *reinterpret_cast<uint16_t *>(d2) = (uint16_t)c2;
                    }
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[sk & 1]);
        }
    } else {
        // ---------------- softmax: group of four warps (a stream's, or half a stream's rows), lane quarter
        const int w = warp - 4, group = w >> 2, q = warp & 3;
        const int i = group / C::GS, rb = (group % C::GS) * RT;    // stream, first row within it
        const int kl = q * 32 + lane;                              // key of the tile
        const uint32_t lanes = (uint32_t)(q * 32) << 16;
        const uint32_t tS = tmem + i * N + lanes + rb, tO = tmem + (NS + i) * N + lanes + rb;
        const int st = w * 32 + lane;
        float *nmg = nm + group * RT;
        uint8_t *wrow = sW + i * C::WB;
        uint32_t sn = 0, on = 0, seq0 = 0;
        bool first_seg = true;
        if (st == 0) a.s.meta[blockIdx.x].nseg = 0;
        for (int r = st & 127; r < RT; r += 128) nmg[r] = kNoRef;
        named_bar_sync(1 + group, 128);
        for (uint32_t sk = 0;; ++sk) {
            const RingSeg *rsg = seg_at(sk);
            if (!rsg) break;
            const Seg &sg = rsg->s;
            const int n = sg.k1 - sg.k0, len = sg.len;
            const int t0 = SHARE ? 0 : i, step = SHARE ? 1 : NS;
            const int page_log2 = a.s.sq.page_log2, n_kv = a.s.n_kv, g = sg.g;
            const int32_t *tab = a.s.sq.page_table + (size_t)sg.b * a.s.sq.max_pages;
            const int kbase = sg.k0 * kTile + kl;
            // page of this thread's key of tile t (-1: none), and its scales; looked up one and two tiles ahead
            auto page_of = [&](int t) -> int {
                const int key = kbase + t * kTile;
                const int id = t < n && key < len ? tab[key >> page_log2] : -1;
                return (unsigned)id < (unsigned)a.s.sq.n_pages ? id : -1;
            };
            auto scales_of = [&](int id) -> int {          // key's | value's << 8; -1: no key
                if (id < 0) return -1;
                const size_t at = (size_t)id * n_kv + g;
                return a.k_scale[at] | (int)a.v_scale[at] << 8;
            };
            int sc_next = scales_of(page_of(t0)), id_next = page_of(t0 + step);
            mbar_wait(&q_full[sk & 1], (sk >> 1) & 1, abort_flag, status);   // rs, lims
            const int ur0 = (SHARE ? i * 64 : 0) + rb;     // first row of the unit
            const float *rsg_ = rs + (sk & 1) * UR + ur0;
            const int *lim = lims + (sk & 1) * UR + ur0;
            const int lim0 = lim[0];                       // (no row sees fewer keys)
            float l[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) l[r] = 0.f;
            for (int t = t0; t < n; t += step) {
                const int sc = sc_next;
                sc_next = scales_of(id_next);
                id_next = page_of(t + 2 * step);
                const bool here = sc >= 0;
                const int key = kbase + t * kTile;
                const float aj = here ? a.scale_log2 * e8m0_f32(sc & 255) : 0.f;
                const float vs = here ? e8m0_f32(sc >> 8) : 0.f;
                const float ev = here ? (float)((sc >> 8) - 127) : 0.f;
                const bool all_seen = __all_sync(0xffffffffu, here && key < lim0);
                mbar_wait(&s_full[i], sn & 1, abort_flag, status);
                ++sn;
                __syncwarp();
                tc_fence_after();
                const bool fresh = t < C::NS && (!SHARE || t == 0);   // the stream's first tile of the slice
#pragma unroll
                for (int c = 0; c < RT; c += CH) {
                    float x[CH];
                    // scores in log2, less the rows' references (or as they are)
                    auto scores = [&](bool whole) {
                        float s2[CH];
                        tmem_ld_n<CH>(tS + c, x);
                        tmem_ld_n<CH>(tS + R + c, s2);
                        tmem_ld_wait_n<CH>(x);
                        tmem_ld_wait_n<CH>(s2);
#pragma unroll
                        for (int r = 0; r < CH; r += 4) {
                            const float4 f = *reinterpret_cast<const float4 *>(rsg_ + c + r);
                            float4 m = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (!whole) m = *reinterpret_cast<const float4 *>(nmg + c + r);
                            const float2 k32 = make_float2(0.03125f, 0.03125f), aj2 = make_float2(aj, aj);
                            float2 u = fma2(make_float2(s2[r], s2[r + 1]), k32, make_float2(x[r], x[r + 1]));
                            float2 v = fma2(make_float2(s2[r + 2], s2[r + 3]), k32, make_float2(x[r + 2], x[r + 3]));
                            u = fma2(mul2(u, aj2), make_float2(f.x, f.y), make_float2(m.x, m.y));
                            v = fma2(mul2(v, aj2), make_float2(f.z, f.w), make_float2(m.z, m.w));
                            x[r] = u.x;
                            x[r + 1] = u.y;
                            x[r + 2] = v.x;
                            x[r + 3] = v.y;
                        }
                        if (!all_seen) {
#pragma unroll
                            for (int r = 0; r < CH; ++r)
                                if (!here || key >= lim[c + r]) x[r] = -INFINITY;
                        }
                    };
                    scores(false);
                    float top = fmaxf(x[0], x[1]);
#pragma unroll
                    for (int r = 2; r < CH; r += 2) top = fmaxf(top, fmaxf(x[r], x[r + 1]));
                    if (bar_any(1 + group, 128, top > kTop - ev)) {
                        // a weight would pass 2^8 (or a row's first key): the references move
                        scores(true);
#pragma unroll
                        for (int r = 0; r < CH; ++r) {
                            float v = x[r] + ev;
#pragma unroll
                            for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
                            if (lane == 0) xm[(group * 4 + q) * RT + c + r] = v;
                        }
                        named_bar_sync(1 + group, 128);
                        float f[CH];
#pragma unroll
                        for (int r = 0; r < CH; ++r) {
                            float v = xm[group * 4 * RT + c + r];
#pragma unroll
                            for (int x4 = 1; x4 < 4; ++x4) v = fmaxf(v, xm[(group * 4 + x4) * RT + c + r]);
                            const float old = nmg[c + r], now = fminf(old, kSlack - v);   // (minus the references; v = -inf keeps it)
                            f[r] = old == kNoRef ? 1.f : ex2(now - old);
                            l[c + r] *= f[r];
                        }
                        if (!fresh) {
                            float o[CH];
#pragma unroll
                            for (int part = 0; part < 2; ++part) {
                                tmem_ld_n<CH>(tO + part * R + c, o);
                                tmem_ld_wait_n<CH>(o);
#pragma unroll
                                for (int r = 0; r < CH; ++r) o[r] *= f[r];
                                tmem_st_n<CH>(tO + part * R + c, o);
                            }
                            tmem_st_wait();
                        }
                        named_bar_sync(1 + group, 128);   // every warp has the old references
                        if (q == 0 && lane < CH) {
                            float v = xm[group * 4 * RT + c + lane];
#pragma unroll
                            for (int x4 = 1; x4 < 4; ++x4) v = fmaxf(v, xm[(group * 4 + x4) * RT + c + lane]);
                            nmg[c + lane] = fminf(nmg[c + lane], kSlack - v);
                        }
                        named_bar_sync(1 + group, 128);
                        scores(false);
                    }
                    // weights: their sum as they are, their two parts with the value's scale
                    uint32_t p1[CH / 4], p2[CH / 4];
                    const float2 vs2 = make_float2(vs, vs);
#pragma unroll
                    for (int r = 0; r < CH; r += 2) {
                        const float2 p = make_float2(ex2(x[r]), ex2(x[r + 1]));
                        l[c + r] += p.x;
                        l[c + r + 1] += p.y;
                        const float2 pv = mul2(p, vs2);
                        const __half2 h = __floats2half2_rn(pv.x, pv.y);   // 11 bits: three more than the two parts keep
                        const uint32_t c1 = e4m3x2_of_half2(*reinterpret_cast<const uint32_t *>(&h));
                        const uint32_t b = half2_of_e4m3x2(c1);
                        const __half2 d = __hmul2(__hsub2(h, *reinterpret_cast<const __half2 *>(&b)), __float2half2_rn(32.f));
                        const uint32_t c2 = e4m3x2_of_half2(*reinterpret_cast<const uint32_t *>(&d));
                        if (r & 2) {
                            p1[r >> 2] |= c1 << 16;
                            p2[r >> 2] |= c2 << 16;
                        } else {
                            p1[r >> 2] = c1;
                            p2[r >> 2] = c2;
                        }
                    }
                    if constexpr (CH == 8) {
                        *reinterpret_cast<uint4 *>(wrow + row_unit<WROW>(kl, 0)) = make_uint4(p1[0], p1[1], p2[0], p2[1]);
                    } else {
                        *reinterpret_cast<uint4 *>(wrow + row_unit<WROW>(kl, (rb + c) >> 4)) = make_uint4(p1[0], p1[1], p1[2], p1[3]);
                        *reinterpret_cast<uint4 *>(wrow + row_unit<WROW>(kl, (R + rb + c) >> 4)) = make_uint4(p2[0], p2[1], p2[2], p2[3]);
                    }
                }
                if (rb == 0 && (!SHARE || i == 0)) {
                    // a page that ends inside this tile: its slots past the keys are zeroed in V
                    const int e = len - (sg.k0 + t) * kTile;
                    const int page = 1 << page_log2;
                    const int end = min(kTile, ((len + page - 1) & ~(page - 1)) - (sg.k0 + t) * kTile);
                    if (e > 0 && e < end) {
                        const uint32_t vsl = seq0 + v_at(t, n);
                        mbar_wait(&full[vsl % SLOTS], (vsl / SLOTS) & 1, abort_flag, status);
                        uint8_t *vt = ring + (vsl % SLOTS) * TB;
                        for (int y = st & 127; y < (end - e) * (HD / 16); y += 128)
                            *reinterpret_cast<uint4 *>(vt + e * HD + y * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[i]);
            }
            seq0 += 2 * n;
            // ---------------- the segment's rows: out, or left for the join
            const bool whole = sg.k0 == 0 && sg.k1 == sg.n;
            const int slot = blockIdx.x * 2 + (first_seg ? 0 : 1);
            if (st == 0 && sg.k0 == 0 && !whole) a.s.meta[blockIdx.x] = part_of(sg, slot, chunk);
            first_seg = false;
            {
                const float sum = warp_sums<RT>(l, lane);
                constexpr int rep = 32 / RT;
                if (lane % rep == 0) ls[(group * 4 + q) * RT + lane / rep] = sum;
            }
            named_bar_sync(9, 512);
            if (st < UR) {                                 // thread = row of the unit
                float M = -INFINITY, L = 0.f;
                const int ng = SHARE ? 1 : NS;
                float ms[NS], sums[NS];
#pragma unroll
                for (int x = 0; x < ng; ++x) {
                    const int gr = SHARE ? st / RT : x * C::GS + st / RT, r = st % RT;
                    const float m = -nm[gr * RT + r];
                    ms[x] = m == -kNoRef ? -INFINITY : m;
                    sums[x] = (ls[gr * 4 * RT + r] + ls[(gr * 4 + 1) * RT + r]) + (ls[(gr * 4 + 2) * RT + r] + ls[(gr * 4 + 3) * RT + r]);
                    M = fmaxf(M, ms[x]);
                }
#pragma unroll
                for (int x = 0; x < ng; ++x) {
                    const float f = ms[x] == -INFINITY ? 0.f : ex2(ms[x] - M);
                    fj[x * UR + st] = f;
                    L += ms[x] == -INFINITY ? sums[x] : sums[x] * f;   // (0, or NaN of a query that is not finite)
                }
                Lr[st] = L;
                Mr[st] = M;
            }
            mbar_wait(o_full, on & 1, abort_flag, status);
            ++on;
            tc_fence_after();
            named_bar_sync(9, 512);
            // lane = dim, columns = rows: each group of warps takes a quarter of the unit's rows
            constexpr int OR = UR / 4, OC = OR < 16 ? OR : 16;
            const int d = (q * 32 + lane) & (HD - 1);
            if (q * 32 < HD) {
#pragma unroll 1
                for (int r0 = group * OR; r0 < group * OR + OR; r0 += OC) {
                    if (r0 >= sg.nrows) break;
                    float o[OC];
#pragma unroll
                    for (int r = 0; r < OC; ++r) o[r] = 0.f;
#pragma unroll
                    for (int x = 0; x < (SHARE ? 1 : NS); ++x) {
                        if (!SHARE && x >= n) break;       // (a stream without a tile)
                        float o1[OC], o2[OC];
                        const uint32_t tx = tmem + lanes + (SHARE ? (NS + (r0 >> 6)) * N + (r0 & 63) : (NS + x) * N + r0);
                        tmem_ld_n<OC>(tx, o1);
                        tmem_ld_n<OC>(tx + R, o2);
                        tmem_ld_wait_n<OC>(o1);
                        tmem_ld_wait_n<OC>(o2);
#pragma unroll
                        for (int r = 0; r < OC; ++r) {
                            const float f = fj[x * UR + r0 + r];
                            const float v = fmaf(o2[r], 0.03125f, o1[r]);
                            o[r] = f == 0.f ? o[r] : fmaf(v, f, o[r]);
                        }
                    }
#pragma unroll
                    for (int r = 0; r < OC; ++r) {
                        const int ur = r0 + r;
                        if (ur < sg.nrows) {
                            const float L = Lr[ur], M = Mr[ur];
                            const int tok = (sg.row0 + ur) / a.s.G;
                            const size_t out_row = (size_t)(sg.start + tok) * a.s.n_q + sg.g * a.s.G + (sg.row0 + ur - tok * a.s.G);
                            const size_t part_row = (size_t)slot * UR + ur;
                            if (whole) {
                                a.A[out_row * HD + d] = __float2bfloat16_rn(L == 0.f ? 0.f : o[r] / L);
                                if (d == 0 && a.s.lse) a.s.lse[out_row] = row_lse(M, L);
                            } else {
                                a.s.part_o[part_row * HD + d] = o[r];
                                if (d == 0) a.s.part_ml[part_row] = make_float2(M, L);
                            }
                        }
                    }
                }
            }
            __syncwarp();
            tc_fence_before();
            if (lane == 0) {
                mbar_arrive(&seg_empty[sk % kSegs]);
                mbar_arrive(&q_empty[sk & 1]);
            }
            named_bar_sync(9, 512);   // O, sums and references have been read
            for (int r = st & 127; r < RT; r += 128) nmg[r] = kNoRef;
            named_bar_sync(1 + group, 128);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- host side
// Rows of a stream, and whether two streams share tiles, by the rows that share a key head's keys.
struct Form {
    int rows, share;
};
Form form_for(int max_new, int G) {
    const long long rows = (long long)max_new * G;
    if (rows <= 8) return {8, 0};
    if (rows <= 16) return {16, 0};
    if (rows <= 32) return {32, 0};
    return {64, rows > 64};
}

template <int HD, int R, bool SHARE>
cudaError_t launch_f8(const F8Args &a, int grid, const CUtensorMap &tk, const CUtensorMap &tv, unsigned *status,
                      cudaStream_t st) {
    static bool configured[64] = {};   // per device: raise the shared-memory limit once
    int dev = 0;
    cudaGetDevice(&dev);
    constexpr int smem = (int)Cfg<HD, R, SHARE>::kSmem;
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(k_paged_attention_f8<HD, R, SHARE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    const cudaError_t e = launch_kernel(k_paged_attention_f8<HD, R, SHARE>, dim3(grid), dim3(kThreads), smem, st, 1, tk, tv, a, status);
    if (e != cudaSuccess) return e;
    return paged_join<bf16, HD>(a.s, grid, a.A, st);
}

template <int HD>
cudaError_t launch_form(Form f, const F8Args &a, int grid, const CUtensorMap &tk, const CUtensorMap &tv, unsigned *status,
                        cudaStream_t st) {
    if (f.share) return launch_f8<HD, 64, true>(a, grid, tk, tv, status, st);
    if (f.rows == 64) return launch_f8<HD, 64, false>(a, grid, tk, tv, status, st);
    if (f.rows == 32) return launch_f8<HD, 32, false>(a, grid, tk, tv, status, st);
    return f.rows == 16 ? launch_f8<HD, 16, false>(a, grid, tk, tv, status, st)
                        : launch_f8<HD, 8, false>(a, grid, tk, tv, status, st);
}

}  // namespace

size_t paged_attention_f8_ws_bytes(int max_new, int n_q, int n_kv, int hd) {
    const Form f = form_for(max_new, n_q / n_kv);
    return paged_part_bytes(num_sms(), f.share ? 128 : f.rows, hd);
}

cudaError_t paged_attention_f8(const PagedAttn &p, const uint8_t *k_scale, const uint8_t *v_scale, void *ws, unsigned *status,
                               cudaStream_t st) {
    const Form f = form_for(p.max_new, p.n_q / p.n_kv);
    const int page = 1 << p.sq.page_log2, grid = num_sms();
    F8Args a{};
    a.s = paged_sched(p, grid, f.share ? 128 : f.rows, kTile, ws);
    a.A = static_cast<bf16 *>(p.A);
    a.Q = static_cast<const bf16 *>(p.Q);
    a.q_stride = p.q_stride;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.box = page < kTile ? page : kTile;
    a.boxes = kTile / a.box;
    a.scale_log2 = p.scale * 1.4426950408889634f;
    CUtensorMap tk, tv;
    const uint64_t hd = (uint64_t)p.hd, rows = (uint64_t)p.sq.n_pages << p.sq.page_log2;
    const CUtensorMapSwizzle sw = p.hd == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    if (!map3d(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, sw, p.k_pages, hd, (uint64_t)p.n_kv, rows, hd, hd * p.n_kv, (uint32_t)hd, 1,
               (uint32_t)a.box) ||
        !map3d(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, sw, p.v_pages, hd, (uint64_t)p.n_kv, rows, hd, hd * p.n_kv, (uint32_t)hd, 1,
               (uint32_t)a.box))
        return cudaErrorInvalidValue;
    return p.hd == 128 ? launch_form<128>(f, a, grid, tk, tv, status, st) : launch_form<64>(f, a, grid, tk, tv, status, st);
}

}  // namespace dllm
