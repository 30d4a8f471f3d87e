// paged_attention_f8.cu -- attention of ragged new rows over 8-bit pages on the sm_103a tensor
// cores: E4M3 codes with a power-of-two scale for each page and head, 2^k for keys, 2^v for values.
//
//   A[t, h] = sum_j w_j 2^{v_j} V_j / sum_j w_j,   w_j = 2^(c 2^{k_j} <Q[t, h], K_j>)
//
// The codes are fed to the tensor cores as they lie in the pages (kind::f8f6f4, twice the rate
// of bf16); nothing is widened.  The other operand of each product is two E4M3 numbers:
//   q 2^-e    = q1 + q2           (a bf16 query has 8 bits, an E4M3 number 4: exact but for what lies
//                                  2^-17 below the row's largest element, which 2^e brings to [128, 256))
//   w' 2^-m   = w1 + w2 / 32      (8 bits of each weight, or to 2^-15: 2^-13 of its tile's largest at most)
// so a product costs what it does in bf16 and reads half the bytes.
//   S^T [128 keys, rows]         =  K [128 keys, hd] q1^T + K q2^T
//   O^T [hd, w1 rows | w2 rows] += V^T [hd, 128 keys]  [w1 | w2]
// Keys and dims are the 128 lanes, rows the columns: a few rows cost a few columns, a thread
// has one key, and the key's scales, presence and position are values of its own.  The value's scale
// goes into the weight before it is rounded, w' = w 2^v, and the running reference m is that of
// c s + v, so that what is rounded to 8 bits is what counts in the result; the sum of w is kept in
// fp32 without it.  m moves, up or down, when in a tile of keys a row's largest weight would pass 2^8 or stay below 2^-2, and
// O and the sums are multiplied by a power of two.  So a weight is held to 2^-13 of the largest in its own tile, and (a row's
// largest so far is never below 2^2) to 2^-17 of the row's: thousands of small ones behind one key far above them all come
// out right, where a reference that only rises rounds each to 0.  It falls by 2^24 below its highest at most (weights below
// 2^-41 of the row's largest may be lost; O and the sums stay in range).  What finds a row that stays below costs prompts 60 us
// and blocks 5 us; a window of 2^1 .. 2^8 took 1420 us instead of 1146 (a move holds up both streams for two tiles' time), one
// warp of four that looks for all, the others only after it, no less than all.  Rows near the window's ends move along with one
// that has to: prompts behind one key that stands out take 1175 us, 1585 while each row moved by itself; 1133 without one.
//
// Work is cut as in paged_sched.cuh, one CTA per SM.  A unit has up to R rows of a sequence and key
// head.  Streams of four warps work through key tiles in turn, each with an S^T, an O^T and weights of its
// own, so that the tensor cores and the loads run on while a stream's softmax does:
//   R = 8, 16, 32: 4 streams;   R = 64: 2;
//   SHARE (R = 64): 2 streams with 64 rows each of a unit of 128, sharing every K and V tile.
// The streams' (O, m, sum) are joined at the end of a slice.
//
// Threads: warp 0 loads K tiles, warps 1 and 2 issue the products for S and for O, warp 3 loads V tiles for up to
// 32 rows (warp 0 does for more), then the streams' 16 warps: thread = key of the tile, with up to 32 rows in its
// registers.  S of a stream's next tile is formed as soon as this one's scores are
// in registers.  (One warp issues a box in 55 cycles and a tile of 8 boxes in 650: pages of 16 rows were
// bound by it at 4.6 TB/s.)
#include <climits>

#include "e4m3.cuh"
#include "paged_sched.cuh"
#include "paged_tc.cuh"

namespace dllm {
namespace {

constexpr int kTile = 128;              // keys of a tile
constexpr float kTop = 8.f, kLow = -2.f; // log2 of a row's largest weight in a tile: no more, and no less if the reference may fall
// Where a reference that moves puts it (or up to 1 below: whole numbers, exact factors): in the middle, but a tile that passed
// the top is one of the largest to come.  When a row's has to move, those of rows above kRaised or below kNear move along.
constexpr float kFirst = 3.f, kRaised = 6.f, kNear = 1.f;
constexpr float kDrop = 24.f;           // how far the reference falls below its highest
constexpr int kInfos = 20;              // tiles whose scales are at hand
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
    static constexpr int NS = R <= 32 ? 4 : 2;                 // streams
    static constexpr int RT = R < 32 ? R : 32;                 // rows of a thread
    static constexpr int GS = R / RT;                          // groups of four warps of a stream
    static constexpr bool SPLIT = R <= 32;                     // K and V are loaded by two warps
    static constexpr int THREADS = 128 + 512;
    static constexpr int UR = SHARE ? 128 : R;                 // rows of a unit
    static constexpr int N = 2 * R;                            // columns of a stream's O^T
    static constexpr int QR = R < 16 ? 16 : R;                 // of its S^T (16 at least)
    static constexpr int AHEAD = SHARE ? 1 : NS;               // tiles by which K runs ahead of V
    static constexpr int TB = kTile * HD;                      // bytes of a tile
    static constexpr int WROW = N < 32 ? 32 : N;               // bytes of a key's weights
    static constexpr int WB = kTile * WROW;
    static constexpr int QB = (SHARE ? 2 : 1) * 2 * QR * HD;   // bytes of a unit's queries
    static constexpr int WORDS = 4 * UR /* rs, lim: two buffers */ + 4 * 11 * RT /* nm, fm, hm, xm, ls */ + 36 /* lows, held */ +
                                 (SHARE ? 1 : NS) * UR + 4 * UR + kInfos * 16 * 4;
    static constexpr int FIX = 2 * QB + NS * WB + WORDS * 4 + 1024;
    static constexpr int SLOTS = (227 * 1024 - FIX) / TB < 20 ? (227 * 1024 - FIX) / TB : 20;
    static constexpr int KSLOTS = SLOTS / 2;                   // of them for K
    static constexpr int BARS = 2 + 2 * SLOTS + 4 * NS + 1 + 2 * kSegs + 2;
    static constexpr size_t kSmem = 2 * QB + NS * WB + (size_t)SLOTS * TB + WORDS * 4 + BARS * 8 + 64 + kSegs * (int)sizeof(RingSeg);
    static_assert(kSmem <= 227 * 1024 && KSLOTS >= 2, "shared memory");
};

// kind::f8f6f4, both operands E4M3, fp32 D.  Bits as in idesc_bf16 with formats 0; 15 and 16: A, B MN-major.
constexpr uint32_t idesc_e4m3(int N, int mn_major) {
    return (1u << 4) | (uint32_t(mn_major) << 15) | (uint32_t(mn_major) << 16) | (uint32_t(N >> 3) << 17) | (uint32_t(128 >> 4) << 24);
}
// Shared-memory descriptors as their two words: the low one has the address (and no leading offset), the
// high one, the same for all tiles of a layout, the stride of 8 rows of `ROW` bytes, which are swizzled within
// themselves (128-, 64- or 32-byte mode).  K-major: the rows are M or N; MN-major: the rows are K.  No operand
// here is wider than a row but A = V^T of 64 dims, whose second half (leading offset 0) repeats the first.
template <int ROW> __device__ __forceinline__ constexpr uint32_t desc_hi() {
    return uint32_t((8 * ROW) >> 4) | (1u << 14) | ((ROW == 128 ? 2u : (ROW == 64 ? 4u : 6u)) << 29);
}
__device__ __forceinline__ void mma_e4m3(uint32_t leader, uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                         uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc), "r"(leader)
        : "memory");
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
    } else if constexpr (C == 16) {
        tmem_ld_x16(taddr, slice16(v));
    } else {
        static_assert(C == 32);
        tmem_ld_x32(taddr, *reinterpret_cast<float(*)[32]>(v));
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
// Named barrier of whole warps whose lanes may have parted before it.
__device__ __forceinline__ void meet(int id, int nthreads) {
    __syncwarp();
    named_bar_sync(id, nthreads);
}
// Reduces C <= 32 values a lane over the warp, in v[0]; lane l receives that of value l * C / 32.
template <int C, class F> __device__ __forceinline__ void warp_reduce(float (&v)[C], int lane, F op) {
    int cnt = C;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (cnt > 1) {
            cnt >>= 1;
#pragma unroll
            for (int k = 0; k < C / 2; ++k)
                if (k < cnt) {
                    const float give = (lane & o) ? v[k] : v[k + cnt], keep = (lane & o) ? v[k + cnt] : v[k];
                    v[k] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
                }
        } else {
            v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
        }
    }
}

template <int HD, int R, bool SHARE>
__global__ void __launch_bounds__(Cfg<HD, R, SHARE>::THREADS, 1)
    k_paged_attention_f8(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const F8Args a,
                         unsigned *status) {
    using C = Cfg<HD, R, SHARE>;
    constexpr int SLOTS = C::SLOTS, TB = C::TB, NS = C::NS, RT = C::RT, UR = C::UR, N = C::N, QR = C::QR, WROW = C::WROW;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *ring = smem;
    uint8_t *sQ = ring + SLOTS * TB;                                // two units' queries
    uint8_t *sW = sQ + 2 * C::QB;                                   // the streams' weights
    float *rs = reinterpret_cast<float *>(sW + NS * C::WB);         // [2][UR] scale of a row's query
    int *lims = reinterpret_cast<int *>(rs + 2 * UR);               // [2][UR] keys that a row sees
    float *nm = reinterpret_cast<float *>(lims + 2 * UR);           // [4 groups][RT] minus the reference
    float *fm = nm + 4 * RT;                                        // [4][RT] log2 of a moved reference's factor
    float *hm = fm + 4 * RT;                                        // [4][RT] minus the highest reference so far
    float *xm = hm + 4 * RT;                                        // [4][4 warps][RT] maxima
    float *ls = xm + 16 * RT;                                       // [4][4][RT] sums
    float *fj = ls + 16 * RT;                                    // [streams][UR] factors of the join
    float *Lr = fj + (SHARE ? 1 : NS) * UR, *Mr = Lr + UR, *inv = Mr + UR;   // [UR]
    int *rowof = reinterpret_cast<int *>(inv + UR);                 // [UR] row and head of the batch
    uint32_t *lows = reinterpret_cast<uint32_t *>(rowof + UR);      // [2 tiles][4 groups][4 warps] rows without a weight of 2^kLow
    uint32_t *held = lows + 32;                                     // [4 groups] rows whose reference does not fall
    float4 *info = reinterpret_cast<float4 *>(held + 4);            // [kInfos][16 boxes] factors of a box, see load_k
    uint64_t *bars = reinterpret_cast<uint64_t *>(info + kInfos * 16);
    uint64_t *q_full = bars;
    uint64_t *full = bars + 2, *empty = full + SLOTS;
    uint64_t *s_full = empty + SLOTS, *s_empty = s_full + NS, *p_full = s_empty + NS, *p_empty = p_full + NS, *o_full = p_empty + NS;
    uint64_t *seg_full = o_full + 1, *seg_empty = seg_full + kSegs, *fin = seg_empty + kSegs;
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
            mbar_init(&q_full[i], 16);
        }
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < NS; ++i) {
            mbar_init(&s_full[i], 2);             // the product, and the S warp for the tile's scales
            mbar_init(&s_empty[i], 4 * C::GS);
            mbar_init(&p_full[i], 4 * C::GS);
            mbar_init(&p_empty[i], 1);
        }
        mbar_init(o_full, 1);
        mbar_init(&fin[0], 1);
        mbar_init(&fin[1], 1);
        for (int i = 0; i < kSegs; ++i) {
            mbar_init(&seg_full[i], 1);
            mbar_init(&seg_empty[i], (C::SPLIT ? 3 : 2) + 16);   // product, V and softmax warps
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
    // Slice k, or null at the end, the same for all lanes.  The wait does not look at the abort flag and lasts longer than
    // the others: the TMA warp hands out a slice, or the end, in any case, and warps that meet at
    // named barriers must not part.
    auto seg_of_warp = [&](uint32_t k) -> const RingSeg * {
        const bool got = mbar_wait_through(&seg_full[k % kSegs], (k / kSegs) & 1, 4);
        const RingSeg *r = &segs[k % kSegs];
        return __all_sync(0xffffffffu, got) && r->go ? r : nullptr;
    };
    // K and V tiles go through a ring each (slots 0 .. KSLOTS - 1 and KSLOTS .. SLOTS - 1): loaded by one warp and used in
    // that order, a slot is never waited for two laps ahead, which its barriers' phase could not tell apart.
    struct Place {
        uint32_t first, count, slot, lap;
        __device__ __forceinline__ void next() {
            if (++slot == first + count) {
                slot = first;
                lap ^= 1;
            }
        }
    };
    const Place k_ring{0, C::KSLOTS, 0, 0}, v_ring{C::KSLOTS, SLOTS - C::KSLOTS, C::KSLOTS, 0};
    // By a whole warp.  Every lane asks; the vote brings them together again before an instruction that takes the warp as one.
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status));
    };

    if (warp == 0 || (C::SPLIT && warp == 3)) {
        // ---------------- loads: lane = box of a tile
        const int page_log2 = a.s.sq.page_log2;
        const int absent = a.s.sq.n_pages << page_log2;                // a row outside the pool: zeros
        const int in_page = (lane * a.box) & ((1 << page_log2) - 1);   // (tiles start on pages, or pages hold tiles)
        uint32_t sent = 0, laps = 0;                                   // slots that this warp has loaded into, their last laps
        Place kat = k_ring, vat = v_ring;
        bool ok = true;
        // Page of this lane's box of a tile (-1: none, or past the keys); the value is first looked at
        // when the box is loaded, a tile or more later.
        auto page_of = [&](const Seg &sg, int tile) -> int {
            const int key = (sg.k0 + tile) * kTile + lane * a.box;
            int id = -1;
            if (lane < a.boxes && tile < sg.k1 - sg.k0 && key < sg.len)
                id = a.s.sq.page_table[(size_t)sg.b * a.s.sq.max_pages + (key >> page_log2)];
            return id;
        };
        auto row_of = [&](const Seg &sg, int tile, int id) -> int {    // pool row of this lane's box
            const int off = page_log2 > 7 ? ((sg.k0 + tile) * kTile) & ((1 << page_log2) - 1) : 0;
            return (unsigned)id < (unsigned)a.s.sq.n_pages ? (id << page_log2) + in_page + off : absent;
        };
        auto issue = [&](const CUtensorMap *tm, Place &at, const Seg &sg, int row) {
            if (lane < a.boxes) tma_load_3d(ring + at.slot * TB + lane * a.box * HD, tm, &full[at.slot], 0, sg.g, row);
            sent |= 1u << at.slot;
            laps = (laps & ~(1u << at.slot)) | at.lap << at.slot;
        };
        auto load_v = [&](const Seg &sg, int tile, int id) {
            if (!ok || !(ok = wait(&empty[vat.slot], vat.lap ^ 1))) return;
            if (lane == 0) mbar_arrive_expect_tx(&full[vat.slot], TB);
            __syncwarp();
            issue(&tmV, vat, sg, row_of(sg, tile, id));
            vat.next();
        };
        // A box's scales go along with its keys: (c 2^k, 2^v, v), zeros without a page.  An entry is written anew kInfos
        // tiles later, when K is at most KSLOTS ahead of S and S at most NS ahead of the streams.
        static_assert(kInfos >= C::KSLOTS + 2 * NS, "scales");
        struct Scales {
            int k, v;
        };
        auto scales_of = [&](const Seg &sg, int id) -> Scales {
            Scales x{-1, -1};
            if ((unsigned)id < (unsigned)a.s.sq.n_pages) {
                const size_t at = (size_t)id * a.s.n_kv + sg.g;
                x.k = a.k_scale[at];
                x.v = a.v_scale[at];
            }
            return x;
        };
        uint32_t inf = 0;
        auto load_k = [&](const Seg &sg, int tile, int id, const Scales &x) {
            if (!ok || !(ok = wait(&empty[kat.slot], kat.lap ^ 1))) return;
            issue(&tmK, kat, sg, row_of(sg, tile, id));
            if (lane < 16)
                info[inf * 16 + lane] = x.k < 0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                                                : make_float4(a.scale_log2 * e8m0_f32(x.k), e8m0_f32(x.v), (float)(x.v - 127), 0.f);
            inf = (inf + 1) % kInfos;
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(&full[kat.slot], TB);   // (the phase ends with this arrival at the earliest)
            kat.next();
        };
        if (warp == 0) {
            // A slice is handed out before the loads of the one before it, so that its queries are ready in time.
            uint32_t sk = 0;
            auto hand_out = [&](const Seg &x, bool go) {
                if (lane == 0) {
                    mbar_wait_through(&seg_empty[sk % kSegs], ((sk / kSegs) & 1) ^ 1, 1);
                    segs[sk % kSegs] = RingSeg{x, go};
                    mbar_arrive(&seg_full[sk % kSegs]);
                    if (sk == 0) a.s.meta[blockIdx.x].nseg = 0;
                    if (go && x.k0 == 0 && x.k1 < x.n) a.s.meta[blockIdx.x] = part_of(x, blockIdx.x * 2 + (sk > 0), chunk);
                }
                ++sk;
                __syncwarp();
            };
            Walker wk = walk_from(a.s, w0);
            Seg sg{}, nx{};
            bool have = wk.next(a.s, sg);
            hand_out(sg, have);
            while (have) {
                const bool more = wk.next(a.s, nx) && ok;
                hand_out(nx, more);
                const int n = sg.k1 - sg.k0;
                // pages are looked up two tiles, scales one tile before they are needed
                constexpr int LEAD = C::AHEAD;
                int ids[LEAD + 2];
#pragma unroll
                for (int j = 0; j < LEAD + 2; ++j) ids[j] = page_of(sg, j);
                Scales sc[LEAD + 1];
#pragma unroll
                for (int j = 0; j <= LEAD; ++j) sc[j] = scales_of(sg, ids[j]);
#pragma unroll
                for (int j = 0; j < LEAD; ++j)
                    if (j < n) load_k(sg, j, ids[j], sc[j]);
                Scales next_sc = sc[LEAD];
                for (int t = 0; ok && t < n; ++t) {
                    const Scales now = next_sc;
                    next_sc = scales_of(sg, ids[LEAD + 1]);
                    const int later = page_of(sg, t + LEAD + 2);
                    if (!C::SPLIT) load_v(sg, t, ids[0]);
                    if (t + LEAD < n) load_k(sg, t + LEAD, ids[LEAD], now);
#pragma unroll
                    for (int j = 0; j < LEAD + 1; ++j) ids[j] = ids[j + 1];
                    ids[LEAD + 1] = later;
                }
                sg = nx;
                have = more;
            }
        } else {
            for (uint32_t sk = 0;; ++sk) {
                const RingSeg *rsg = seg_of_warp(sk);
                if (!rsg) break;
                const Seg sg = rsg->s;
                __syncwarp();
                if (lane == 0) mbar_arrive(&seg_empty[sk % kSegs]);
                const int n = sg.k1 - sg.k0;
                int ids[3];
#pragma unroll
                for (int j = 0; j < 3; ++j) ids[j] = page_of(sg, j);
                for (int t = 0; ok && t < n; ++t) {
                    const int later = page_of(sg, t + 3);
                    load_v(sg, t, ids[0]);
                    ids[0] = ids[1];
                    ids[1] = ids[2];
                    ids[2] = later;
                }
            }
        }
        if (lane == 0 && *abort_flag)   // every issued copy must land before the CTA can exit
            for (uint32_t i = 0; i < SLOTS; ++i)
                if (sent >> i & 1) mbar_drain(&full[i], laps >> i & 1);
    } else if (warp == 1 || warp == 2) {
        // ---------------- products: warp 1 S = K q, warp 2 O += V w.  The whole warp walks along, so that addresses
        // stay in uniform registers (a lane alone took 75 cycles for each product); one lane issues.
        const uint32_t lead = elect_one();
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t aq = smem_u32(sQ) >> 4, ar = smem_u32(ring) >> 4, aw = smem_u32(sW) >> 4;
        uint32_t ph = 0;                        // bit i = phase of the stream's barrier
        Place at = warp == 1 ? k_ring : v_ring;
        bool ok = true;
        for (uint32_t sk = 0;; ++sk) {
            const RingSeg *rsg = seg_of_warp(sk);
            if (!rsg) break;
            const int n = __shfl_sync(0xffffffffu, rsg->s.k1 - rsg->s.k0, 0);
            __syncwarp();
            if (lane == 0) mbar_arrive(&seg_empty[sk % kSegs]);
            if (!ok) continue;   // (aborted: only takes the slices off the ring)
            if (warp == 1) {
                ok = wait(&q_full[sk & 1], (sk >> 1) & 1);
                const uint32_t qb = aq + (sk & 1) * (C::QB >> 4);
                int i = 0;
                for (int t = 0; ok && t < n; ++t) {
                    ok = wait(&full[at.slot], at.lap);
                    const uint32_t kb = ar + at.slot * (TB >> 4);
#pragma unroll 1
                    for (int j = 0; ok && j < (SHARE ? 2 : 1); ++j) {
                        const int x = SHARE ? j : i;
                        ok = wait(&s_empty[x], ((ph >> x) & 1) ^ 1);
                        if (!ok) break;
                        ph ^= 1u << x;
                        tc_fence_after();
                        // the first part of the queries, then the second, QR rows further
#pragma unroll
                        for (int kk = 0; kk < 2 * HD / 32; ++kk)
                            mma_e4m3(lead, tm + x * QR, kb + kk % (HD / 32) * 2, desc_hi<HD>(),
                                     qb + (SHARE ? j * (2 * QR * HD >> 4) : 0) + (kk / (HD / 32) * QR * HD >> 4) + kk % (HD / 32) * 2,
                                     desc_hi<HD>(), idesc_e4m3(QR, 0), kk > 0);
                        commit_if(lead, &s_full[x]);
                        if (lane == 0) mbar_arrive(&s_full[x]);   // hands the tile's scales on, as this warp got them with its keys
                    }
                    if (!ok) break;
                    commit_if(lead, &empty[at.slot]);
                    i = i + 1 == NS ? 0 : i + 1;
                    at.next();
                }
            } else {
                int i = 0;
                for (int t = 0; ok && t < n; ++t) {
                    ok = wait(&full[at.slot], at.lap);
                    const uint32_t vb = ar + at.slot * (TB >> 4);
#pragma unroll 1
                    for (int j = 0; ok && j < (SHARE ? 2 : 1); ++j) {
                        const int x = SHARE ? j : i;
                        ok = wait(&p_full[x], (ph >> x) & 1);
                        if (!ok) break;
                        ph ^= 1u << x;
                        tc_fence_after();
                        const uint32_t wb = aw + x * (C::WB >> 4);
#pragma unroll
                        for (int kk = 0; kk < kTile / 32; ++kk)
                            mma_e4m3(lead, tm + NS * QR + x * N, vb + kk * 2 * HD, desc_hi<HD>(), wb + kk * 2 * WROW, desc_hi<WROW>(),
                                     idesc_e4m3(N, 1), kk > 0 ? 1 : t >= C::AHEAD);
                        commit_if(lead, &p_empty[x]);
                    }
                    if (!ok) break;
                    commit_if(lead, &empty[at.slot]);
                    i = i + 1 == NS ? 0 : i + 1;
                    at.next();
                }
                if (ok) commit_if(lead, o_full);
            }
        }
        // Nothing of this thread may still run when TMEM is freed, and no arrival that a commit still owes may come when the
        // CTA has gone: its barriers' place is the next one's by then.
        if (lead) {
            mma_commit(&fin[warp - 1]);
            mbar_drain(&fin[warp - 1], 0);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ---------------- softmax: group gr (a stream's, or half of its rows: rb and on), lane quarter q
        const int st = tid - 128, gr = st >> 7, q = warp & 3;
        const int i = gr / C::GS, rb = gr % C::GS * RT;
        const int kl = q * 32 + lane;                              // key of the tile
        const uint32_t lanes = (uint32_t)(q * 32) << 16;
        const uint32_t tS = tmem + i * QR + lanes + rb, tO = tmem + NS * QR + i * N + lanes + rb;
        const int page_log2 = a.s.sq.page_log2;
        float *nmg = nm + gr * RT, *fmg = fm + gr * RT, *hmg = hm + gr * RT, *xmg = xm + gr * 4 * RT, *lsg = ls + gr * 4 * RT;
        uint8_t *wrow = sW + i * C::WB;
        uint32_t sn = 0, on = 0, seq0 = 0;
        if (kl < RT) nmg[kl] = kNoRef;
        meet(1 + gr, 128);
        constexpr int step = SHARE ? 1 : NS;
        const int t0 = SHARE ? 0 : i;
        const int box = kl / a.box;
        // Queries of slice sk, by all these warps: two E4M3 numbers an element, the row's power of two beside them; a
        // thread has 16 elements of a row.  Their buffer's last user was slice sk - 2, which every warp has left behind.
        auto prepare = [&](uint32_t sk, const Seg &sg) {
            constexpr int LR = HD / 16;
            uint8_t *qb = sQ + (sk & 1) * C::QB;
#pragma unroll 1
            for (int p = st; p < UR * LR; p += 512) {       // (whole warps)
                const int ur = p / LR, lr = p % LR, row = sg.row0 + ur, tok = row / a.s.G;
                uint32_t raw[8] = {};
                int lim = INT_MAX;
                if (ur < sg.nrows) {
                    const bf16 *src = a.Q + (size_t)(sg.start + tok) * a.q_stride + (size_t)(sg.g * a.s.G + row - tok * a.s.G) * HD;
                    const uint4 x = reinterpret_cast<const uint4 *>(src)[2 * lr], y = reinterpret_cast<const uint4 *>(src)[2 * lr + 1];
                    raw[0] = x.x;
                    raw[1] = x.y;
                    raw[2] = x.z;
                    raw[3] = x.w;
                    raw[4] = y.x;
                    raw[5] = y.y;
                    raw[6] = y.z;
                    raw[7] = y.w;
                    if (lr == 0) lim = PagedSeqs::visible(sg.pos0 + tok, sg.len, a.s.mask_block);
                }
                uint32_t top = 0;                    // magnitude bits: NaN above infinity above all others
#pragma unroll
                for (int e = 0; e < 8; ++e) top = max(top, max(raw[e] & 0x7fffu, (raw[e] >> 16) & 0x7fffu));
#pragma unroll
                for (int o = LR / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                const int ex = min(max((int)(top >> 7), 10), 254);             // biased exponent of the largest
                const float f = __uint_as_float((uint32_t)(261 - ex) << 23);   // 2^(7 - (ex - 127))
                uint32_t c1[4], c2[4];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x = __uint_as_float(raw[e] << 16) * f, y = __uint_as_float(raw[e] & 0xffff0000u) * f;
                    const uint32_t c = e4m3x2(x, y);
                    const float2 b = f32_of_e4m3x2(c);
                    const uint32_t d = e4m3x2(x - b.x, y - b.y);
                    if (e & 1) {
                        c1[e >> 1] |= c << 16;
                        c2[e >> 1] |= d << 16;
                    } else {
                        c1[e >> 1] = c;
                        c2[e >> 1] = d;
                    }
                }
                const int n1 = SHARE ? (ur >> 6) * 2 * QR + (ur & 63) : ur;   // row of the operand; QR further: the second part
                *reinterpret_cast<uint4 *>(qb + row_unit<HD>(n1, lr)) = make_uint4(c1[0], c1[1], c1[2], c1[3]);
                *reinterpret_cast<uint4 *>(qb + row_unit<HD>(n1 + QR, lr)) = make_uint4(c2[0], c2[1], c2[2], c2[3]);
                if (lr == 0) {                       // a query that is not finite gives NaN
                    rs[(sk & 1) * UR + ur] = top >= 0x7f80u ? NAN : __uint_as_float((uint32_t)(ex - 7) << 23);
                    lims[(sk & 1) * UR + ur] = lim;
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[sk & 1]);
        };
        const RingSeg *rsg = seg_of_warp(0);
        if (rsg) prepare(0, rsg->s);
        for (uint32_t sk = 0; rsg; ++sk) {
            const Seg &sg = rsg->s;
            const int n = sg.k1 - sg.k0, len = sg.len;
            const int kbase = sg.k0 * kTile + kl;
            wait(&q_full[sk & 1], (sk >> 1) & 1);              // rs, lims
            const float *rsu = rs + (sk & 1) * UR + (SHARE ? i * 64 : 0) + rb;
            const int *lim = lims + (sk & 1) * UR + (SHARE ? i * 64 : 0) + rb;
            const int lim0 = lim[0];                       // (no row sees fewer keys)
            // the tile in which the last page ends with slots that hold no key
            const int page = 1 << page_log2, last_page = (len + page - 1) & ~(page - 1);
            const int tail = (len & (kTile - 1)) && len < last_page ? (len >> 7) - sg.k0 : -1;
            float2 l[RT / 2];
#pragma unroll
            for (int r = 0; r < RT / 2; ++r) l[r] = make_float2(0.f, 0.f);
            for (int t = t0; t < n; t += step) {
                const int key = kbase + t * kTile;
                wait(&s_full[i], sn & 1);
                ++sn;
                const float4 f4 = info[((seq0 + t) % kInfos) * 16 + box];
                const float aj = f4.x, vs = f4.y, ev = f4.z;
                const bool here = vs > 0.f;                 // (aj may be too small for a number)
                const bool all_seen = __all_sync(0xffffffffu, here && key < lim0);
                tc_fence_after();
                const bool fresh = t == t0;                // the stream's first tile of the slice
                float x[RT];
                // scores in log2, less the rows' references (or as they are)
                auto scores = [&](bool whole) {
#pragma unroll
                    for (int c = 0; c < RT; c += 32) tmem_ld_n<RT>(tS + c, x + c);
                    tmem_ld_wait_n<RT>(x);
                    const float2 aj2 = make_float2(aj, aj);
#pragma unroll
                    for (int r = 0; r < RT; r += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(rsu + r);
                        float4 m = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (!whole) m = *reinterpret_cast<const float4 *>(nmg + r);
                        const float2 u = fma2(mul2(make_float2(x[r], x[r + 1]), aj2), make_float2(f.x, f.y), make_float2(m.x, m.y));
                        const float2 v = fma2(mul2(make_float2(x[r + 2], x[r + 3]), aj2), make_float2(f.z, f.w), make_float2(m.z, m.w));
                        x[r] = u.x;
                        x[r + 1] = u.y;
                        x[r + 2] = v.x;
                        x[r + 3] = v.y;
                    }
                    if (!all_seen) {
#pragma unroll
                        for (int r = 0; r < RT; ++r)
                            if (!here || key >= lim[r]) x[r] = -INFINITY;
                    }
                };
                // The rows' maxima over the tile, value scales included, and the references that follow from them
                // (x is lost)
                auto refer = [&](bool first) {
#pragma unroll
                    for (int r = 0; r < RT; ++r) x[r] += ev;
                    warp_reduce(x, lane, [](float u, float v) { return fmaxf(u, v); });
                    constexpr int rep = 32 / RT;
                    if (lane % rep == 0) xmg[q * RT + lane / rep] = x[0];
                    meet(1 + gr, 128);
                    if (kl < RT) {
                        const float old = first ? kNoRef : nmg[kl];      // minus the references; without a key they stay
                        const float most = fmaxf(fmaxf(xmg[kl], xmg[RT + kl]), fmaxf(xmg[2 * RT + kl], xmg[3 * RT + kl]));
                        const float high = old == kNoRef ? kNoRef : hmg[kl];
                        const bool above = most + old > kRaised, below = most + old < kNear && most > -INFINITY;
                        const float place = above && old != kNoRef ? kRaised : kFirst;
                        const float now = above || below ? fminf(floorf(place - most), high + kDrop) : old;
                        nmg[kl] = now;
                        fmg[kl] = old == kNoRef ? 0.f : now - old;
                        hmg[kl] = fminf(high, now);
                        const bool stuck = now == high + kDrop || (SHARE ? i * 64 : 0) + rb + kl >= sg.nrows;
                        const unsigned h = __ballot_sync(RT == 32 ? 0xffffffffu : (1u << RT) - 1, stuck);
                        if (kl == 0) held[gr] = __brev(h) >> (32 - RT);
                    }
                    meet(1 + gr, 128);
                };
                bool move = fresh;
                if (!fresh) {
                    scores(false);
                    float top = fmaxf(x[0], x[1]);
#pragma unroll
                    for (int r = 2; r < RT; r += 2) top = fmaxf(top, fmaxf(x[r], x[r + 1]));
                    // rows none of whose keys here has a weight of 2^kLow (of row r in bit RT - 1 - r)
                    uint32_t low = 0;
#pragma unroll
                    for (int r = 0; r < RT; ++r) low = __funnelshift_l(__float_as_uint(x[r] - (kLow - ev)), low, 1);
                    low = __reduce_and_sync(0xffffffffu, low);
                    uint32_t *lw = lows + (sn & 1) * 16 + gr * 4;     // (another place in the next tile, whose first warps may be ahead)
                    if (lane == 0) lw[q] = low;
                    __syncwarp();
                    move = bar_any(1 + gr, 128, top > kTop - ev);   // a weight would pass 2^8 (or a row's first key)
                    const uint4 all = *reinterpret_cast<const uint4 *>(lw);
                    move |= (all.x & all.y & all.z & all.w & ~held[gr]) != 0;
                }
                if (move) {
                    scores(true);
                    refer(fresh);
                    if (!fresh) {
                        wait(&p_empty[i], sn & 1);
                        tc_fence_after();
                        constexpr int OC = RT < 16 ? RT : 16;
#pragma unroll
                        for (int c = 0; c < RT; c += OC) {
                            float f[OC];
#pragma unroll
                            for (int r = 0; r < OC; r += 4) {
                                const float4 g = *reinterpret_cast<const float4 *>(fmg + c + r);
                                f[r] = g.x;
                                f[r + 1] = g.y;
                                f[r + 2] = g.z;
                                f[r + 3] = g.w;
                            }
#pragma unroll
                            for (int r = 0; r < OC; r += 2)    // (of O what 2^d loses is lost beside what comes)
                                l[(c + r) / 2] = make_float2(sum_times_ex2(l[(c + r) / 2].x, f[r]), sum_times_ex2(l[(c + r) / 2].y, f[r + 1]));
#pragma unroll
                            for (int r = 0; r < OC; ++r) f[r] = ex2(f[r]);
#pragma unroll
                            for (int part = 0; part < 2; ++part) {
                                float o[OC];
                                tmem_ld_n<OC>(tO + part * R + c, o);
                                tmem_ld_wait_n<OC>(o);
#pragma unroll
                                for (int r = 0; r < OC; ++r) o[r] *= f[r];
                                tmem_st_n<OC>(tO + part * R + c, o);
                            }
                        }
                        tmem_st_wait();
                    }
                    scores(false);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_empty[i]);
                // weights: their sum as they are, their two parts with the value's scale
                if (sn > 1) wait(&p_empty[i], sn & 1);   // the tile before has been multiplied
                const float2 vs2 = make_float2(vs, vs);
                constexpr int WC = RT < 16 ? RT : 16;
#pragma unroll
                for (int c = 0; c < RT; c += WC) {
                    uint32_t p1[WC / 4], p2[WC / 4];
#pragma unroll
                    for (int r = 0; r < WC; r += 2) {
                        const float2 p = make_float2(ex2(x[c + r]), ex2(x[c + r + 1]));
                        l[(c + r) / 2] = add2(l[(c + r) / 2], p);
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
                    if constexpr (WC == 8) {
                        *reinterpret_cast<uint4 *>(wrow + row_unit<WROW>(kl, 0)) = make_uint4(p1[0], p1[1], p2[0], p2[1]);
                    } else {
                        *reinterpret_cast<uint4 *>(wrow + row_unit<WROW>(kl, (rb + c) >> 4)) = make_uint4(p1[0], p1[1], p1[2], p1[3]);
                        *reinterpret_cast<uint4 *>(wrow + row_unit<WROW>(kl, (R + rb + c) >> 4)) = make_uint4(p2[0], p2[1], p2[2], p2[3]);
                    }
                }
                if (t == tail && rb == 0 && (!SHARE || i == 0)) {
                    // a page that ends inside this tile: its slots past the keys are zeroed in V
                    const int e = len & (kTile - 1), end = min(kTile, last_page - (len - e));
                    constexpr uint32_t VS = SLOTS - C::KSLOTS;
                    const uint32_t vsl = seq0 + t, slot = C::KSLOTS + vsl % VS;
                    wait(&full[slot], (vsl / VS) & 1);
                    uint8_t *vt = ring + slot * TB;
                    for (int y = kl; y < (end - e) * (HD / 16); y += 128)
                        *reinterpret_cast<uint4 *>(vt + e * HD + y * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[i]);
            }
            seq0 += n;
            // ---------------- the segment's rows: out, or left for the join
            const bool whole = sg.k0 == 0 && sg.k1 == sg.n;
            const int cut = blockIdx.x * 2 + (sk > 0);
            {
                float lr[RT];
#pragma unroll
                for (int r = 0; r < RT; ++r) lr[r] = r & 1 ? l[r / 2].y : l[r / 2].x;
                warp_reduce(lr, lane, [](float u, float v) { return u + v; });
                constexpr int rep = 32 / RT;
                if (lane % rep == 0) lsg[q * RT + lane / rep] = lr[0];
            }
            const RingSeg *next = seg_of_warp(sk + 1);
            if (next) prepare(sk + 1, next->s);
            meet(9, 512);
            if (st < UR) {                                 // thread = row of the unit
                constexpr int ng = SHARE ? 1 : NS;
                float M = -INFINITY, L = 0.f, ms[ng], sums[ng];
#pragma unroll
                for (int x = 0; x < ng; ++x) {
                    const int j = SHARE ? st / RT : x * C::GS + st / RT, r = st % RT;   // the row's group
                    const float m = -nm[j * RT + r], *v = ls + j * 4 * RT + r;
                    ms[x] = m == -kNoRef ? -INFINITY : m;
                    sums[x] = (v[0] + v[RT]) + (v[2 * RT] + v[3 * RT]);
                    M = fmaxf(M, ms[x]);
                }
#pragma unroll
                for (int x = 0; x < ng; ++x) {
                    const float f = ms[x] == -INFINITY ? 0.f : ex2(ms[x] - M);
                    fj[x * UR + st] = f;
                    L += ms[x] == -INFINITY ? sums[x] : sum_times_ex2(sums[x], ms[x] - M);   // (0, or NaN of a query that is not finite)
                }
                Lr[st] = L;
                Mr[st] = M;
                inv[st] = L == 0.f ? 0.f : 1.0f / L;
                const int tok = (sg.row0 + st) / a.s.G;
                rowof[st] = (sg.start + tok) * a.s.n_q + sg.g * a.s.G + (sg.row0 + st - tok * a.s.G);
            }
            wait(o_full, on & 1);
            ++on;
            tc_fence_after();
            meet(9, 512);
            if (st < sg.nrows) {
                if (!whole) a.s.part_ml[(size_t)cut * UR + st] = make_float2(Mr[st], Lr[st]);
                else if (a.s.lse) a.s.lse[rowof[st]] = row_lse(Mr[st], Lr[st]);
            }
            __syncwarp();
            // lane = dim, columns = rows: the streams' warps share the unit's rows
            constexpr int OC = UR / 4 < 8 ? UR / 4 : 8;
            if (q * 32 < HD) {
#pragma unroll 1
                for (int r0 = gr * OC; r0 < sg.nrows; r0 += 4 * OC) {
                    constexpr int ng = SHARE ? 1 : NS, two = ng < 2 ? 1 : 2;   // two streams' loads under way at a time
                    float o[OC];
#pragma unroll
                    for (int r = 0; r < OC; ++r) o[r] = 0.f;
#pragma unroll 1
                    for (int x0 = 0; x0 < ng && (SHARE || x0 < n); x0 += two) {
                        float part[two][2][OC];
#pragma unroll
                        for (int x = 0; x < two; ++x) {    // (a stream without a tile has factors 0)
                            const uint32_t tx = tmem + lanes + NS * QR + (SHARE ? (r0 >> 6) * N + (r0 & 63) : (x0 + x) * N + r0);
                            tmem_ld_n<OC>(tx, part[x][0]);
                            tmem_ld_n<OC>(tx + R, part[x][1]);
                        }
#pragma unroll
                        for (int x = 0; x < two; ++x) {
                            tmem_ld_wait_n<OC>(part[x][0]);
                            tmem_ld_wait_n<OC>(part[x][1]);
#pragma unroll
                            for (int r = 0; r < OC; ++r) {
                                const float f = fj[(x0 + x) * UR + r0 + r];
                                const float v = fmaf(part[x][1][r], 0.03125f, part[x][0][r]);
                                o[r] = f == 0.f ? o[r] : fmaf(v, f, o[r]);
                            }
                        }
                    }
                    if (whole) {
#pragma unroll
                        for (int r = 0; r < OC; ++r)
                            if (r0 + r < sg.nrows) a.A[(size_t)rowof[r0 + r] * HD + kl] = __float2bfloat16_rn(o[r] * inv[r0 + r]);
                    } else {
                        float *dst = a.s.part_o + ((size_t)cut * UR + r0) * HD + kl;
#pragma unroll
                        for (int r = 0; r < OC; ++r)
                            if (r0 + r < sg.nrows) dst[r * HD] = o[r];
                    }
                }
            }
            __syncwarp();
            tc_fence_before();
            if (lane == 0) {
                mbar_arrive(&seg_empty[sk % kSegs]);
            }
            meet(9, 512);   // O, sums and references have been read
            if (kl < RT) nmg[kl] = kNoRef;
            meet(1 + gr, 128);
            rsg = next;
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
    const cudaError_t e = launch_kernel(k_paged_attention_f8<HD, R, SHARE>, dim3(grid), dim3(Cfg<HD, R, SHARE>::THREADS), smem, st, 1, tk, tv, a, status);
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
    // (a line of L2 may not bring in the next head's row)
    const CUtensorMapSwizzle sw = p.hd == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    const CUtensorMapL2promotion l2 = p.hd == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
    if (!map3d(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, sw, p.k_pages, hd, (uint64_t)p.n_kv, rows, hd, hd * p.n_kv, (uint32_t)hd, 1,
               (uint32_t)a.box, l2) ||
        !map3d(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, sw, p.v_pages, hd, (uint64_t)p.n_kv, rows, hd, hd * p.n_kv, (uint32_t)hd, 1,
               (uint32_t)a.box, l2))
        return cudaErrorInvalidValue;
    return p.hd == 128 ? launch_form<128>(f, a, grid, tk, tv, status, st) : launch_form<64>(f, a, grid, tk, tv, status, st);
}

}  // namespace dllm
