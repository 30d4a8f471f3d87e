// paged_attention_tc.cu -- attention of ragged new rows over a paged cache on the sm_103a
// tensor cores (bf16).
//
//   A[t, h] = softmax_j(<Q[t, h], K_j> scale) V_j  over the keys j < visible(pos(t))
//
// Work is cut as in paged_sched.cuh, one CTA per SM.  A 128-row tile holds the rows (token, head
// of the group) of floor(128 / G) tokens, loaded by one TMA box of [tokens, G heads, 64 dims];
// a unit is one or two such tiles over 128-key tiles.
//
// Pipeline of a CTA, two streams i = 0, 1, so that while one's softmax runs the tensor cores work
// for the other:
//   NQ = 2: the streams are the unit's two row tiles and share every K and V tile;
//   NQ = 1: both streams have the same rows and take the key tiles in turn; their (O, m, l)
//           are joined at the end;
//   NQ = 0: as 1 for 32 rows or fewer.  The rows stand in all four lane quarters of the S tile, so that
//           every warp has 16 of the tile's keys for each row, where 1 leaves three warps of four idle;
//           the weights go through shared memory, one copy.
//   S_i = Q_i K^T      tcgen05.mma into TMEM (128 columns)
//   P_i = 2^(S_i c - m) softmax warps, bf16 (one rounding of each weight, as the product takes bf16),
//                      written back over S_i in TMEM (keys 0..63 from column 0 on, keys 64..127 from
//                      column 64 on: each warpgroup over its own)
//   O_i += P_i V       tcgen05.mma, A from TMEM (NQ = 0: from shared memory), V MN-major; O_i stays in TMEM
// m is the reference of the exponentials and is only moved (O_i and l rescaled) when a tile's
// maximum exceeds it by more than 8 in log2: fp32 sums and bf16 weights keep their relative
// precision below that.
// K and V tiles go through one ring in the order of their use; pages shorter than a tile
// are loaded box by box, one lane each; boxes without a page (or past the keys) read as
// zeros from outside the pool.  Values past the last key of a page that ends inside a tile
// may be anything (NaN included): they are zeroed in shared memory before the product.
//
// Threads: warp 0 TMA, warp 1 MMA issue, then two warpgroups per stream: thread = (row, half of
// the tile's keys).
//
// What bounds it.  Few rows per key (a block or a token of each sequence): the bytes of K and V.
// 64 tokens, 28 heads on 4 of 128 dims, 64 x up to 8192 keys: 144 us, 5.8 TB/s (the loads alone take as
// long); 16 blocks of 32 rows, 32 heads, 4096 keys: 145 us.  Long prompts: the chain from a
// tile's scores through its softmax to its product, of which two are under way at a time.  2 x 4096 rows over
// 8192 keys, 28 heads: 652 us,
// 1.02 PFLOP/s (the products alone: 404 us).  One block of 32 rows over 1024 keys: 15.5 us, a chain of
// latencies (the schedule 2.4, first loads and scores 3, a slice's end 3.3, the join 3 to 5).
#include <climits>

#include "paged_sched.cuh"
#include "paged_tc.cuh"

namespace dllm {

namespace {

constexpr int kTile = 128;              // rows of a query tile, keys of a key tile
constexpr int kBox = 128 * 128;         // one 64-dim box of 128 rows: 16 KB
constexpr int kThreads = 64 + 512;
constexpr float kLazy = 8.f;            // log2 by which a maximum may exceed the reference

struct PtcArgs {
    PagedSched s;
    bf16 *A;
    int tile_tok;                       // tokens of a row tile
    int box, box_log2, boxes;           // rows of a TMA box of K / V and boxes of a tile
    float scale_log2;
};

// D[tmem] (+)= A[tmem] * B[smem]: A's row r is lane r, two bf16 of K per 32-bit column.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void tmem_ld_wait32(float (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]),
                   "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]),
                   "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27])
                 :
                 : "memory");
    asm volatile("" : "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31]));   // (30 operands at most per statement)
}

// The slices that the CTA works through, from the TMA warp (which walks the schedule, ahead of the
// others) to the MMA thread and the softmax warps.
struct RingSeg {
    Seg s;
    int holes;          // a key of the slice lacks a page
    int go;             // 0: no more
};

// Does a row that sees the keys below lim (<= s.len) have one in slice s?
__device__ __forceinline__ bool sees_key(const int32_t *tab, int page_log2, int n_pages, const Seg &s, int lim, bool holes) {
    if (!holes || lim <= s.k0 * kTile) return lim > s.k0 * kTile;
    const int end = (min(s.k1 * kTile, lim) + (1 << page_log2) - 1) >> page_log2;
    bool any = false;
#pragma unroll 1
    for (int p = s.k0 * kTile >> page_log2; p < end && !any; ++p) any = (unsigned)tab[p] < (unsigned)n_pages;
    return any;
}

template <int HD, int NQ> struct Cfg {
    static constexpr int CH = HD / 64;
    static constexpr int TB = CH * kBox;                       // bytes of a 128-row tile
    static constexpr int QT = NQ == 2 ? 2 : 1;                  // row tiles in shared memory
    static constexpr int SLOTS = HD == 128 ? (NQ != 1 ? 5 : 6) : 8;
    static constexpr int PB = NQ == 0 ? 32 * 256 : 0;           // bytes of a stream's weights (32 rows)
    static constexpr int BARS = 2 + 2 * SLOTS + 6 + 2 * kSegs;
    static constexpr size_t kSmem = (size_t)QT * TB + 2 * PB + (size_t)SLOTS * TB + 2 * 2 * 128 * 4 + BARS * 8 + 64 + kSegs * (int)sizeof(RingSeg);
};

template <int HD, int NQ>
__global__ void __launch_bounds__(kThreads, 1)
    k_paged_attention_tc(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const PtcArgs a, unsigned *status) {
    using C = Cfg<HD, NQ>;
    constexpr int SLOTS = C::SLOTS, TB = C::TB, CH = C::CH;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *sQ = smem;
    uint8_t *sP = sQ + C::QT * TB;        // (NQ == 0; the product reads on into the ring, rows that nobody uses)
    uint8_t *ring = sP + 2 * C::PB;
    float *xmax = reinterpret_cast<float *>(ring + SLOTS * TB);   // [2 streams][2 halves][128]
    uint64_t *bars = reinterpret_cast<uint64_t *>(xmax + 2 * 2 * 128);
    uint64_t *q_full = bars, *q_empty = bars + 1;
    uint64_t *full = bars + 2, *empty = full + SLOTS;
    uint64_t *s_full = empty + SLOTS, *p_full = s_full + 2, *o_full = p_full + 2;
    uint64_t *seg_full = o_full + 2, *seg_empty = seg_full + kSegs;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + C::BARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *w0 = reinterpret_cast<int *>(tmem_slot + 2);             // the walker's start
    RingSeg *segs = reinterpret_cast<RingSeg *>(tmem_slot + 14);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (smem_u32(smem) & 1023u) {   // the swizzled tiles need it; the same in every CTA
        if (tid == 0) raise_status(status, DLLM_STATUS_SMEM_LAYOUT);
        griddep_wait();
        if (tid == 0) a.s.meta[blockIdx.x].nseg = 0;
        return;
    }
    if (tid == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 8);
            mbar_init(&o_full[i], 1);
        }
        for (int i = 0; i < kSegs; ++i) {
            mbar_init(&seg_full[i], 1);
            mbar_init(&seg_empty[i], 1 + 16);   // MMA thread, softmax warps
        }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmQ);
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

    if (warp == 0) {
        // ---------------- TMA producer: lane = (box of a tile, 64-dim half), 32 of them at most
        const int box = lane % a.boxes, half = lane / a.boxes;
        uint32_t seq = 0, qn = 0, sk = 0;
        bool ok = true;
        Walker wk = walk_from(a.s, w0);
        Seg sg, nx{};
        bool have = wk.next(a.s, nx);
        // Does any key of a slice lack a page?  Looked up 32 pages at a time, for the next slice while
        // this one's tiles go out.
        int scan_p = 0, scan_end = 0;
        bool scan_gap = false;
        int scan_id = 0;               // (looked at one step later)
        const int32_t *scan_tab = nullptr;
        auto scan_begin = [&](const Seg &x) {
            scan_tab = a.s.sq.page_table + (size_t)x.b * a.s.sq.max_pages;
            scan_p = (x.k0 * kTile >> a.s.sq.page_log2) + lane;
            scan_end = (min(x.k1 * kTile, x.len) + (1 << a.s.sq.page_log2) - 1) >> a.s.sq.page_log2;
            scan_gap = false;
            scan_id = 0;
        };
        auto scan = [&] {
            scan_gap |= (unsigned)scan_id >= (unsigned)a.s.sq.n_pages;
            scan_id = scan_p < scan_end ? scan_tab[scan_p] : 0;
            scan_p += 32;
        };
        if (have) scan_begin(nx);
        for (;; ++sk) {
            sg = nx;
            const bool go = have && ok;
            auto hand_out = [&](bool gap) {
                if (lane == 0) {
                    mbar_drain(&seg_empty[sk % kSegs], ((sk / kSegs) & 1) ^ 1);
                    segs[sk % kSegs] = RingSeg{sg, gap, go};
                    mbar_arrive(&seg_full[sk % kSegs]);
                }
                __syncwarp();
            };
            if (!go) {
                hand_out(false);
                break;
            }
            const int n = sg.k1 - sg.k0;
            const int32_t *tab = a.s.sq.page_table + (size_t)sg.b * a.s.sq.max_pages;
            const int absent = a.s.sq.n_pages << a.s.sq.page_log2;   // a row outside the pool: zeros
            // Page of this lane's box of a tile (-1: none, or past the keys); the value is first looked at
            // when the box is loaded, a tile later.
            auto page_of = [&](int tile) -> int {
                const int key = (sg.k0 + tile) * kTile + box * a.box;
                return lane < a.boxes * CH && tile < n && key < sg.len ? tab[key >> a.s.sq.page_log2] : -1;
            };
            const int in_page = (box * a.box) & ((1 << a.s.sq.page_log2) - 1);   // (tiles start on pages, or pages hold tiles)
            auto row_of = [&](int tile, int id) -> int {                 // pool row
                if ((unsigned)id >= (unsigned)a.s.sq.n_pages) return absent;
                const int off = a.s.sq.page_log2 > 7 ? ((sg.k0 + tile) * kTile) & ((1 << a.s.sq.page_log2) - 1) : 0;
                return (id << a.s.sq.page_log2) + in_page + off;
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
                if (lane < a.boxes * CH)
                    tma_load_3d(ring + s * TB + half * kBox + box * a.box * 128, tm, &full[s], half * 64, sg.g, row);
                ++seq;
                return true;
            };
            // K tiles run NQ == 2: one, NQ != 2: two ahead of the V tiles; rows are looked up a tile ahead
            constexpr int AHEAD = NQ == 2 ? 1 : 2;
            int ids[AHEAD + 1];
#pragma unroll
            for (int j = 0; j <= AHEAD; ++j) ids[j] = page_of(j);
#pragma unroll
            for (int j = 0; j < AHEAD; ++j)
                if (ok && j < n) ok = load(&tmK, row_of(j, ids[j]));
            while (__any_sync(0xffffffffu, scan_p < scan_end)) {   // (what the slice before left)
#pragma unroll
                for (int x = 0; x < 4; ++x) scan();
            }
            scan();
            hand_out(__any_sync(0xffffffffu, scan_gap));
            have = wk.next(a.s, nx);
            // the queries: their buffer is free once the segment before has formed its last scores
            if (ok && lane == 0) {
                ok = mbar_wait(q_empty, (qn & 1) ^ 1, abort_flag, status);
                if (ok) {
                    constexpr int COPIES = NQ == 0 ? 4 : 1;   // the 32 rows once per lane quarter
                    mbar_arrive_expect_tx(q_full, (uint32_t)(C::QT * COPIES * a.tile_tok * a.s.G * HD * 2));
                    for (int i = 0; i < C::QT; ++i)
                        for (int x = 0; x < COPIES; ++x)
                            for (int c = 0; c < CH; ++c)
                                tma_load_3d(sQ + i * TB + c * kBox + x * 32 * 128, &tmQ, q_full, c * 64, sg.g * a.s.G,
                                            sg.start + sg.row0 / a.s.G + i * a.tile_tok);
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (ok) ++qn;
            if (have) scan_begin(nx);
            for (int t = 0; ok && t < n; ++t) {
                const int later = page_of(t + AHEAD + 1);
                scan();
                ok = load(&tmV, row_of(t, ids[0]));
                if (ok && t + AHEAD < n) ok = load(&tmK, row_of(t + AHEAD, ids[AHEAD]));
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) ids[j] = ids[j + 1];
                ids[AHEAD] = later;
            }
        }
        if (lane == 0 && *abort_flag) {   // every issued copy must land before the CTA can exit
            if (qn) mbar_drain(q_full, (qn - 1) & 1);
            for (uint32_t i = seq > SLOTS ? seq - SLOTS : 0; i < seq; ++i) mbar_drain(&full[i % SLOTS], (i / SLOTS) & 1);
        }
    } else if (warp == 1) {
        if (lane == 0) {   // ---------------- MMA issuer
            const uint32_t id_s = idesc_bf16(128, kTile, 0), id_pv = idesc_bf16(128, HD, 1);
            const uint32_t aq = smem_u32(sQ), ar = smem_u32(ring), ap = smem_u32(sP);
            uint32_t seq = 0, qn = 0, pn[2] = {0, 0};
            bool ok = true;
            auto take = [&](uint32_t q) -> bool { return mbar_wait(&full[q % SLOTS], (q / SLOTS) & 1, abort_flag, status); };
            for (uint32_t sk = 0;; ++sk) {
                const RingSeg *rsg = seg_at(sk);
                if (!rsg) break;
                const int n = rsg->s.k1 - rsg->s.k0;
                mbar_arrive(&seg_empty[sk % kSegs]);
                if (!ok) continue;   // (aborted: only takes the slices off the ring)
                const int ni[2] = {NQ == 2 ? n : (n + 1) / 2, NQ == 2 ? n : n / 2};
                ok = mbar_wait(q_full, qn & 1, abort_flag, status);
                auto issue_s = [&](int i, uint32_t q, bool last) {
                    const uint32_t kb = ar + (q % SLOTS) * TB, qb = aq + (NQ == 2 ? i : 0) * TB;
#pragma unroll
                    for (int kk = 0; kk < HD / 16; ++kk) {
                        const uint32_t off = (uint32_t)((kk >> 2) * kBox + (kk & 3) * 32);
                        mma_bf16(tmem + i * 128, smem_desc_sw128(qb + off, 16, 1024), smem_desc_sw128(kb + off, 16, 1024),
                                 id_s, kk > 0);
                    }
                    mma_commit(&s_full[i]);
                    if (last) mma_commit(&empty[q % SLOTS]);
                };
                auto issue_pv = [&](int i, uint32_t q, bool first, bool last) {
                    const uint32_t vb = ar + (q % SLOTS) * TB;
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        if (NQ == 0)
                            mma_bf16(tmem + 256 + i * 128, smem_desc_sw128(ap + i * C::PB + (kk >> 2) * (C::PB / 2) + (kk & 3) * 32, 16, 1024),
                                     smem_desc_sw128(vb + kk * 16 * 128, kBox, 1024), id_pv, !first || kk > 0);
                        else mma_bf16_ts(tmem + 256 + i * 128, tmem + i * 128 + (kk >> 2) * 64 + (kk & 3) * 8,
                                    smem_desc_sw128(vb + kk * 16 * 128, kBox, 1024), id_pv, !first || kk > 0);
                    if (last) mma_commit(&empty[q % SLOTS]);
                };
                int scores = ni[0] + ni[1];
                // first scores
                for (int i = 0; ok && i < 2; ++i) {
                    if (ni[i] == 0) continue;
                    const uint32_t q = seq + (NQ == 2 ? 0 : i);
                    if (NQ != 2 || i == 0) ok = take(q);
                    if (!ok) break;
                    tc_fence_after();
                    issue_s(i, q, NQ != 2 || i == 1);
                    if (--scores == 0) mma_commit(q_empty);
                }
                seq += NQ == 2 ? 1 : (n > 1 ? 2 : 1);
                for (int u = 0; ok && u < ni[0]; ++u) {
                    for (int i = 0; ok && i < 2; ++i) {
                        if (u >= ni[i]) continue;
                        const bool lastuse = NQ != 2 || i == 1;
                        const bool more = u + 1 < ni[i];
                        ok = mbar_wait(&p_full[i], pn[i] & 1, abort_flag, status);
                        ++pn[i];
                        if (ok && (NQ != 2 || i == 0)) ok = take(seq);
                        if (!ok) break;
                        tc_fence_after();
                        issue_pv(i, seq, u == 0, lastuse);
                        if (more) {
                            if (NQ != 2 || i == 0) ok = take(seq + 1);
                            if (!ok) break;
                            tc_fence_after();
                            issue_s(i, seq + 1, lastuse);
                            if (--scores == 0) mma_commit(q_empty);   // every product of Q has been issued
                        }
                        if (lastuse) seq += more ? 2 : 1;
                    }
                }
                if (!ok) continue;
                mma_commit(&o_full[0]);
                mma_commit(&o_full[1]);
                ++qn;
            }
            if (!ok) {   // nothing of this thread may still run when TMEM is freed
                mma_commit(&s_full[0]);
                mbar_drain(&s_full[0], 0);
                mbar_drain(&s_full[0], 1);
            }
        }
    } else {
        // ---------------- softmax: stream i, lane quarter q, half hf of the keys
        const int w = warp - 2;
        const int i = w >> 3, hf = (w >> 2) & 1, q = warp & 3;
        const int r = q * 32 + lane;
        const uint32_t lanes = (uint32_t)(q * 32) << 16;
        const uint32_t tS = tmem + i * 128 + lanes, tO = tmem + 256 + i * 128 + lanes;
        const int st = (w & 7) * 32 + lane;          // thread of the stream
        const int tile_rows = a.tile_tok * a.s.G;
        uint32_t sn = 0, on = 0, seq0 = 0;
        bool first_seg = true;
        if (w == 0 && lane == 0) a.s.meta[blockIdx.x].nseg = 0;
        for (uint32_t sk = 0;; ++sk) {
            const RingSeg *rsg = seg_at(sk);
            if (!rsg) break;
            const Seg &sg = rsg->s;
            const bool holes = rsg->holes;
            const int n = sg.k1 - sg.k0;
            const int ni = NQ == 2 ? n : (n + 1 - i) / 2;
            const int rr = NQ == 0 ? lane : r;                     // row of the tile
            const int ur = (NQ == 2 ? i * tile_rows : 0) + rr;     // row of the unit
            const bool live = rr < tile_rows && ur < sg.nrows;
            const int row_tok = (sg.row0 + ur) / a.s.G;            // token of the sequence
            // (a row of no token sees everything: nothing of it is used, and its warp need not mask)
            const int lim = live ? PagedSeqs::visible(sg.pos0 + row_tok, sg.len, a.s.mask_block) : INT_MAX;
            const bool warp_live = __any_sync(0xffffffffu, live);
            float m = -INFINITY, l = 0.f;
            for (int u = 0; u < ni; ++u) {
                const int t = NQ == 2 ? u : 2 * u + i, kt = sg.k0 + t;
                unsigned pages = 0xffffffffu;   // boxes that have a page (those past the keys count as present: lim cuts them)
                if (holes) {
                    const int32_t *tab = a.s.sq.page_table + (size_t)sg.b * a.s.sq.max_pages;
                    const int key = kt * kTile + lane * a.box;
                    const int id = lane < a.boxes && key < sg.len ? tab[key >> a.s.sq.page_log2] : 0;
                    pages = __ballot_sync(0xffffffffu, id >= 0 && id < a.s.sq.n_pages);
                }
                mbar_wait(&s_full[i], sn & 1, abort_flag, status);
                ++sn;
                __syncwarp();
                tc_fence_after();
                if (NQ == 0) {
                    // 32 rows, each in all lane quarters: a thread has 16 of the tile's keys
                    const int sl = hf * 4 + q, k0 = sl * 16;
                    const int nv = lim - kt * kTile - k0;
                    float v[16];
                    tmem_ld_x16(tS + k0, v);
                    tmem_ld_wait(v);
                    if (holes || __any_sync(0xffffffffu, nv < 16)) {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (j >= nv || !((pages >> ((k0 + j) >> a.box_log2)) & 1)) v[j] = -INFINITY;
                    }
                    float mx = v[0];
#pragma unroll
                    for (int j = 1; j < 15; j += 2) mx = fmaxf(mx, fmaxf(v[j], v[j + 1]));
                    mx = fmaxf(mx, v[15]) * a.scale_log2;
                    xmax[(i * 8 + sl) * 32 + lane] = mx;
                    __syncwarp();
                    named_bar_sync(1 + i, 256);
#pragma unroll
                    for (int x = 0; x < 8; ++x) mx = fmaxf(mx, xmax[(i * 8 + x) * 32 + lane]);
                    if (u == 0) {
                        m = mx;
                    } else if (__any_sync(0xffffffffu, mx > m + kLazy)) {   // (the same in the row's eight threads)
                        const float mn = fmaxf(m, mx);
                        const float f = mn == -INFINITY ? 1.f : ex2(m - mn);
                        m = mn;
                        l *= f;
                        if (q == 0) {
#pragma unroll
                            for (int c = 0; c < HD / 2; c += 16) {
                                float o[16];
                                uint32_t ob[16];
                                tmem_ld_x16(tO + hf * (HD / 2) + c, o);
                                tmem_ld_wait(o);
#pragma unroll
                                for (int e = 0; e < 16; ++e) ob[e] = __float_as_uint(o[e] * f);
                                tmem_st_x16(tO + hf * (HD / 2) + c, ob);
                            }
                            tmem_st_wait();
                        }
                    }
                    const float mr = m == -INFINITY ? 0.f : m;
                    uint32_t pk[8];
                    float lt = 0.f;
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const float p0 = ex2(fmaf(v[j], a.scale_log2, -mr)), p1 = ex2(fmaf(v[j + 1], a.scale_log2, -mr));
                        lt += p0 + p1;
                        const __nv_bfloat162 pp = __floats2bfloat162_rn(p0, p1);
                        pk[j >> 1] = *reinterpret_cast<const uint32_t *>(&pp);
                    }
                    l += lt;
                    // row `lane` of the weights, keys k0 ..: two 16-byte units of the swizzled row
                    uint8_t *pr = sP + i * C::PB + hf * (C::PB / 2) + (lane >> 3) * 1024 + (lane & 7) * 128;
                    *reinterpret_cast<uint4 *>(pr + (((2 * q) ^ (lane & 7)) * 16)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    *reinterpret_cast<uint4 *>(pr + (((2 * q + 1) ^ (lane & 7)) * 16)) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
                    fence_async_smem();
                } else if (warp_live) {
                    const int nv = lim - kt * kTile - hf * 64;     // keys of this half that the row sees
                    float v0[32], v1[32];
                    tmem_ld_x32(tS + hf * 64, v0);
                    tmem_ld_x32(tS + hf * 64 + 32, v1);
                    tmem_ld_wait32(v0);
                    tmem_ld_wait32(v1);
                    if (holes || __any_sync(0xffffffffu, nv < 64)) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            if (j >= nv || !((pages >> ((hf * 64 + j) >> a.box_log2)) & 1)) v0[j] = -INFINITY;
                            if (j + 32 >= nv || !((pages >> ((hf * 64 + 32 + j) >> a.box_log2)) & 1)) v1[j] = -INFINITY;
                        }
                    }
                    float x0 = v0[0], x1 = v1[0];
#pragma unroll
                    for (int j = 1; j < 31; j += 2) {
                        x0 = fmaxf(x0, fmaxf(v0[j], v0[j + 1]));
                        x1 = fmaxf(x1, fmaxf(v1[j], v1[j + 1]));
                    }
                    float mx = fmaxf(fmaxf(x0, v0[31]), fmaxf(x1, v1[31]));
                    mx *= a.scale_log2;
                    xmax[(i * 2 + hf) * 128 + r] = mx;
                    __syncwarp();
                    named_bar_sync(1 + i * 4 + q, 64);
                    mx = fmaxf(mx, xmax[(i * 2 + (hf ^ 1)) * 128 + r]);
                    if (u == 0) {
                        m = mx;
                    } else if (__any_sync(0xffffffffu, mx > m + kLazy)) {
                        const float mn = fmaxf(m, mx);
                        const float f = mn == -INFINITY ? 1.f : ex2(m - mn);
                        m = mn;
                        l *= f;
#pragma unroll
                        for (int c = 0; c < HD / 2; c += 16) {
                            float o[16];
                            uint32_t ob[16];
                            tmem_ld_x16(tO + hf * (HD / 2) + c, o);
                            tmem_ld_wait(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) ob[e] = __float_as_uint(o[e] * f);
                            tmem_st_x16(tO + hf * (HD / 2) + c, ob);
                        }
                    }
                    const float mr = m == -INFINITY ? 0.f : m;
                    float2 ls = make_float2(0.f, 0.f);
                    const float2 sc = make_float2(a.scale_log2, a.scale_log2), sh = make_float2(-mr, -mr);
                    auto weights = [&](int c, float (&v)[32]) {
                        uint32_t pk[16];
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            const float2 x = fma2(make_float2(v[j], v[j + 1]), sc, sh);
                            const float2 p = make_float2(ex2(x.x), ex2(x.y));
                            ls = add2(ls, p);
                            const __nv_bfloat162 pp = __floats2bfloat162_rn(p.x, p.y);
                            pk[j >> 1] = *reinterpret_cast<const uint32_t *>(&pp);
                        }
                        tmem_st_x16(tS + hf * 64 + c, pk);   // (over this half's scores)
                    };
                    weights(0, v0);
                    weights(16, v1);
                    l += ls.x + ls.y;
                    tmem_st_wait();
                }
                if (NQ != 2 || i == 0) {
                    // a page that ends inside this tile: its slots past the keys are zeroed in V
                    const int e = sg.len - kt * kTile;
                    const int page = 1 << a.s.sq.page_log2;
                    const int end = min(kTile, ((sg.len + page - 1) & ~(page - 1)) - kt * kTile);
                    if (e > 0 && e < end) {
                        const uint32_t vs = seq0 + (NQ == 2 ? 2 * u + 1 : t + min(n, t + 2));
                        mbar_wait(&full[vs % SLOTS], (vs / SLOTS) & 1, abort_flag, status);
                        uint8_t *vt = ring + (vs % SLOTS) * TB;
                        for (int x = st; x < (end - e) * 8 * CH; x += 256) {
                            const int c = x / ((end - e) * 8), y = x - c * (end - e) * 8;
                            *reinterpret_cast<uint4 *>(vt + c * kBox + (e + (y >> 3)) * 128 + (y & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                        }
                        fence_async_smem();
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[i]);
            }
            seq0 += 2 * n;
            // ---------------- the segment's rows: out, or left for the join
            const bool whole = sg.k0 == 0 && sg.k1 == sg.n;
            const int slot = blockIdx.x * 2 + (first_seg ? 0 : 1);
            if (w == 0 && lane == 0 && sg.k0 == 0 && !whole) a.s.meta[blockIdx.x] = part_of(sg, slot, chunk);
            first_seg = false;
            const size_t out_row = (size_t)(sg.start + row_tok) * a.s.n_q + sg.g * a.s.G + (sg.row0 + ur - row_tok * a.s.G);
            const size_t part_row = (size_t)slot * a.s.unit_rows + ur;
            constexpr int CW = NQ == 2 ? HD / 2 : HD / 4;    // columns of this thread
            const int c0 = (NQ == 2 ? hf : i * 2 + hf) * CW;
            float M = m, L, f0 = 1.f, f1 = 0.f;
            // (o_full also says that every warp of the stream is done with xmax)
            mbar_wait(&o_full[i], on & 1, abort_flag, status);
            if (NQ != 2) mbar_wait(&o_full[i ^ 1], on & 1, abort_flag, status);
            if (NQ == 0) {
                xmax[(i * 8 + hf * 4 + q) * 32 + lane] = l;
                __syncwarp();
                named_bar_sync(1 + i, 256);
                L = 0.f;
#pragma unroll
                for (int x = 0; x < 8; ++x) L += xmax[(i * 8 + x) * 32 + lane];
            } else {
                xmax[(i * 2 + hf) * 128 + r] = l;
                __syncwarp();
                named_bar_sync(1 + i * 4 + q, 64);
                L = xmax[i * 256 + r] + xmax[i * 256 + 128 + r];
            }
            if (NQ == 2) {
                named_bar_sync(1 + i * 4 + q, 64);
            } else {
                named_bar_sync(9, 512);
                xmax[(i * 2 + hf) * 128 + r] = hf == 0 ? L : (ni > 0 ? m : -INFINITY);
                named_bar_sync(9, 512);
                const float m0 = xmax[128 + r], m1 = xmax[384 + r];
                M = fmaxf(m0, m1);
                f0 = m0 == -INFINITY ? 0.f : ex2(m0 - M);
                f1 = m1 == -INFINITY ? 0.f : ex2(m1 - M);
                L = xmax[r] * f0 + xmax[256 + r] * f1;
            }
            ++on;
            tc_fence_after();
            // No weight although the row sees a key: every score is -inf (an infinity in its query), and the formula NaN.
            if (live && L == 0.f &&
                sees_key(a.s.sq.page_table + (size_t)sg.b * a.s.sq.max_pages, a.s.sq.page_log2, a.s.sq.n_pages, sg, lim, holes))
                L = NAN;
            if (warp_live && (NQ != 0 || q == 0)) {
                const float inv = whole ? 1.0f / L : 1.f;
                const uint32_t t0 = (NQ == 2 ? tO : tmem + 256 + lanes) + c0;
#pragma unroll
                for (int c = 0; c < CW; c += 16) {
                    float o[16];
                    __syncwarp();
                    tmem_ld_x16(t0 + c, o);
                    tmem_ld_wait(o);
                    if (NQ != 2) {
                        float o1[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = f0 == 0.f ? 0.f : o[e] * f0;
                        if (n > 1) {
                            tmem_ld_x16(t0 + 128 + c, o1);
                            tmem_ld_wait(o1);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = f1 == 0.f ? o[e] : fmaf(o1[e], f1, o[e]);
                        }
                    }
                    if (live && whole) {
                        uint32_t pk[8];
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const __nv_bfloat162 pp = __floats2bfloat162_rn(L == 0.f ? 0.f : o[e] * inv, L == 0.f ? 0.f : o[e + 1] * inv);
                            pk[e >> 1] = *reinterpret_cast<const uint32_t *>(&pp);
                        }
                        uint4 *dst = reinterpret_cast<uint4 *>(a.A + out_row * HD + c0 + c);
                        dst[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                        dst[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
                    } else if (live) {
                        float4 *dst = reinterpret_cast<float4 *>(a.s.part_o + part_row * HD + c0 + c);
#pragma unroll
                        for (int e = 0; e < 16; e += 4) dst[e >> 2] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                }
                if (live && c0 == 0) {
                    if (!whole) a.s.part_ml[part_row] = make_float2(M, L);
                    else if (a.s.lse) a.s.lse[out_row] = row_lse(M, L);
                }
            }
            __syncwarp();
            tc_fence_before();
            if (lane == 0) mbar_arrive(&seg_empty[sk % kSegs]);
            if (NQ != 2) named_bar_sync(9, 512);   // both streams' O and sums have been read
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
struct Units {
    int tile_tok, nq, rows;
};

// Which instance, by the rows that share a key head's keys in a sequence.  Measured: up to 32 rows, NQ = 0
// against 1: 144 against 162 us (64 single tokens, 7 heads a group), 145 against 165 us (16 blocks of 32
// rows).  One tile holds them, NQ = 1 against 2: 172 against 206 us (64 rows), 185 against 219 us (128).
// More, NQ = 2 against 1: 242 against 259 us (200 rows), 652 against 719 us (4096).
Units units_for(int max_new, int G) {
    Units u;
    if ((long long)max_new * G <= 32) {   // few rows: their softmax spread over all warps
        u.tile_tok = 32 / G;
        u.nq = 0;
    } else {
        u.tile_tok = kTile / G;
        u.nq = max_new > u.tile_tok ? 2 : 1;   // two row tiles where one does not hold a sequence's new rows
    }
    const int tok = u.tile_tok * (u.nq == 2 ? 2 : 1);
    u.rows = (max_new < tok ? max_new : tok) * G;
    return u;
}

template <int HD, int NQ>
cudaError_t launch_tc(const PtcArgs &a, int grid, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                      unsigned *status, cudaStream_t st) {
    static bool configured[64] = {};   // per device: raise the shared-memory limit once
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(k_paged_attention_tc<HD, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)Cfg<HD, NQ>::kSmem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    cudaError_t e = launch_kernel(k_paged_attention_tc<HD, NQ>, dim3(grid), dim3(kThreads), Cfg<HD, NQ>::kSmem, st, 1,
                                  tq, tk, tv, a, status);
    if (e != cudaSuccess) return e;
    return paged_join<bf16, HD>(a.s, grid, a.A, st);
}

}  // namespace

size_t paged_attention_tc_ws_bytes(int max_new, int n_q, int n_kv, int hd) {
    return paged_part_bytes(num_sms(), units_for(max_new, n_q / n_kv).rows, hd);
}

cudaError_t paged_attention_tc(const PagedAttn &p, void *ws, unsigned *status, cudaStream_t st) {
    const int G = p.n_q / p.n_kv;
    const Units u = units_for(p.max_new, G);
    const int page = 1 << p.sq.page_log2, grid = num_sms();
    PtcArgs a{};
    a.s = paged_sched(p, grid, u.rows, kTile, ws);
    a.A = static_cast<bf16 *>(p.A);
    a.tile_tok = u.tile_tok;
    a.box = page < kTile ? page : kTile;
    a.box_log2 = p.sq.page_log2 < 7 ? p.sq.page_log2 : 7;
    a.boxes = kTile / a.box;
    a.scale_log2 = p.scale * 1.4426950408889634f;
    CUtensorMap tq, tk, tv;
    const uint64_t hd = (uint64_t)p.hd, rows = (uint64_t)p.sq.n_pages << p.sq.page_log2;
    if (!map3d_bf16(&tq, p.Q, hd, (uint64_t)p.n_q, (uint64_t)p.T, hd * 2, (uint64_t)p.q_stride * 2, (uint32_t)G,
               (uint32_t)u.tile_tok) ||
        !map3d_bf16(&tk, p.k_pages, hd, (uint64_t)p.n_kv, rows, hd * 2, hd * 2 * p.n_kv, 1, (uint32_t)a.box) ||
        !map3d_bf16(&tv, p.v_pages, hd, (uint64_t)p.n_kv, rows, hd * 2, hd * 2 * p.n_kv, 1, (uint32_t)a.box))
        return cudaErrorInvalidValue;
    if (u.nq == 0)
        return p.hd == 128 ? launch_tc<128, 0>(a, grid, tq, tk, tv, status, st) : launch_tc<64, 0>(a, grid, tq, tk, tv, status, st);
    if (p.hd == 128)
        return u.nq == 2 ? launch_tc<128, 2>(a, grid, tq, tk, tv, status, st) : launch_tc<128, 1>(a, grid, tq, tk, tv, status, st);
    return u.nq == 2 ? launch_tc<64, 2>(a, grid, tq, tk, tv, status, st) : launch_tc<64, 1>(a, grid, tq, tk, tv, status, st);
}

}  // namespace dllm
