// paged_attention_tc.cu -- attention of ragged new rows over a paged cache on the sm_103a
// tensor cores (bf16).
//
//   A[t, h] = softmax_j(<Q[t, h], K_j> scale) V_j  over the keys j < visible(pos(t))
//
// Rows.  The G = n_q / n_kv query heads of a key head read the same keys, so a row of a
// 128-row tile is one (token, head of the group): floor(128 / G) tokens a tile, loaded by one
// TMA box of [tokens, G heads, 64 dims].  A *unit* of work is one or two such tiles (NQ) of
// one sequence and key head, over the 128-key tiles that its last row sees.
//
// Schedule.  One CTA per SM.  The lengths are device data, so every CTA lays the units end to
// end by itself (sequence, key head, tile), counts their key tiles, and takes the slice of
// that line that its index gives it: equal numbers of key tiles whatever the lengths.  A unit
// cut by a slice's end leaves unnormalised partial results in the workspace, which a second
// kernel joins in the order of the keys (the same order every time).
//
// Pipeline of a CTA, two streams i = 0, 1:
//   NQ = 2: the streams are the unit's two row tiles and share every K and V tile;
//   NQ = 1: both streams have the same rows and take the key tiles in turn; their (O, m, l)
//           are joined at the end.
//   S_i = Q_i K^T      tcgen05.mma into TMEM (128 columns)
//   P_i = 2^(S_i c - m) softmax warps, bf16, written back over S_i in TMEM
//   O_i += P_i V       tcgen05.mma, A from TMEM, V MN-major; O_i stays in TMEM
// While one stream's softmax runs the tensor cores work for the other.  m is the reference
// of the exponentials and is only moved (O_i and l rescaled) when a tile's maximum exceeds it by
// more than 2^8: fp32 sums and bf16 weights keep their relative precision below that.
// K and V tiles go through one ring in the order of their use; pages shorter than a tile
// are loaded box by box, one lane each; boxes without a page (or past the keys) read as
// zeros from outside the pool.  Values past the last key of a page that ends inside a tile
// may be anything (NaN included): they are zeroed in shared memory before the product.
//
// Threads: warp 0 TMA, warp 1 MMA issue, then two warpgroups per stream: thread = (row, half of
// the tile's keys).
#include <cudaTypedefs.h>

#include "paged.cuh"

namespace dllm {

PFN_cuTensorMapEncodeTiled_v12000 tmap_encoder();

namespace {

constexpr int kTile = 128;              // rows of a query tile, keys of a key tile
constexpr int kBox = 128 * 128;         // one 64-dim box of 128 rows: 16 KB
constexpr int kThreads = 64 + 512;
constexpr float kLazy = 8.f;            // log2 by which a maximum may exceed the reference

struct PartMeta {      // one per CTA: the split unit whose first slice it computed
    int nseg, slot, tok0, ntok, g, pad[3];
};

struct PtcArgs {
    PagedSeqs sq;
    bf16 *A;
    float *lse;
    int n_q, n_kv, G;
    int tile_tok, unit_tok;             // tokens of a row tile and of a unit
    int T, max_new, mask_block;
    int box, box_log2, boxes;           // rows of a TMA box of K / V and boxes of a tile
    float scale_log2;
    float *part_o;                      // [2 grid][unit_rows][hd]
    float2 *part_ml;                    // [2 grid][unit_rows]
    PartMeta *meta;                     // [grid]
    int unit_rows;
};

__device__ __forceinline__ float ex2(float x) {   // 2^x, relative error ~2^-22; 2^-inf = 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *tm, uint64_t *bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]: A's row r is lane r, two bf16 of K per 32-bit column.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---------------------------------------------------------------- the line of units
// Key tiles of the unit whose last row is the sequence's new row `last` (at least one, so that
// a unit whose rows see nothing still writes its zeros).
__device__ __forceinline__ int unit_tiles(const PtcArgs &a, int len_raw, int len, int n_new, int last) {
    const int lim = PagedSeqs::visible(len_raw - n_new + last, len, a.mask_block);
    const int n = (lim + kTile - 1) / kTile;
    return n > 0 ? n : 1;
}

struct Seg {            // a slice of a unit
    int b, g, tok0;     // tok0: first token (of the batch)
    int n_tok;          // tokens of the unit
    int pos0;           // position of its first token
    int len;            // keys of the sequence
    int k0, k1, n;      // key tiles [k0, k1) of n
};

// The units of a CTA's slice, one after another; every role walks them by itself.
struct Walker {
    int b, g, qt, kt;
    long long left;
    int start, n_new, n_eff, len_raw, len;   // of sequence b

    __device__ __forceinline__ void load(const PtcArgs &a) {
        n_eff = a.sq.rows(b, a.T, a.max_new, start, n_new);
        len_raw = a.sq.kv_len[b];
        len = a.sq.keys(b);
    }
    __device__ __forceinline__ bool next(const PtcArgs &a, Seg &s) {
        if (left <= 0) return false;
        const int t = qt * a.unit_tok;
        s.b = b;
        s.g = g;
        s.tok0 = start + t;
        s.n_tok = min(a.unit_tok, n_eff - t);
        s.pos0 = len_raw - n_new + t;
        s.len = len;
        s.n = unit_tiles(a, len_raw, len, n_new, t + s.n_tok - 1);
        s.k0 = kt;
        const long long e = kt + left;
        s.k1 = e < s.n ? (int)e : s.n;
        left -= s.k1 - s.k0;
        kt = 0;
        if (left > 0) {   // more in this slice: the next unit
            if ((qt + 1) * a.unit_tok < n_eff) {
                ++qt;
            } else {
                qt = 0;
                if (++g == a.n_kv) {
                    g = 0;
                    do {
                        ++b;
                        load(a);
                    } while (n_eff <= 0 && b + 1 < a.sq.B);
                }
            }
        }
        return true;
    }
};

template <int HD, int NQ> struct Cfg {
    static constexpr int CH = HD / 64;
    static constexpr int TB = CH * kBox;                       // bytes of a 128-row tile
    static constexpr int SLOTS = HD == 128 ? (NQ == 2 ? 5 : 6) : 8;
    static constexpr int BARS = 2 + 2 * SLOTS + 6;
    static constexpr size_t kSmem = (size_t)NQ * TB + (size_t)SLOTS * TB + 2 * 2 * 128 * 4 + BARS * 8 + 64;
};

template <int HD, int NQ>
__global__ void __launch_bounds__(kThreads, 1)
    k_paged_attention_tc(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const PtcArgs a, unsigned *status) {
    using C = Cfg<HD, NQ>;
    constexpr int SLOTS = C::SLOTS, TB = C::TB, CH = C::CH;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *sQ = smem;
    uint8_t *ring = sQ + NQ * TB;
    float *xmax = reinterpret_cast<float *>(ring + SLOTS * TB);   // [2 streams][2 halves][128]
    uint64_t *bars = reinterpret_cast<uint64_t *>(xmax + 2 * 2 * 128);
    uint64_t *q_full = bars, *q_empty = bars + 1;
    uint64_t *full = bars + 2, *empty = full + SLOTS;
    uint64_t *s_full = empty + SLOTS, *p_full = s_full + 2, *o_full = p_full + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + C::BARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *w0 = reinterpret_cast<int *>(tmem_slot + 2);             // the walker's start: b, g, qt, kt, left

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nthr = kThreads;

    if (smem_u32(smem) & 1023u) {   // the swizzled tiles need it; the same in every CTA
        if (tid == 0) raise_status(status, DLLM_STATUS_SMEM_LAYOUT);
        griddep_wait();
        if (tid == 0) a.meta[blockIdx.x].nseg = 0;
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
    // ---------------- schedule: prefix of the sequences' key tiles (in the idle ring)
    {
        long long *pre = reinterpret_cast<long long *>(ring);   // [B + 1]
        const int B = a.sq.B;
        const bool one_unit = a.max_new <= a.unit_tok;
        auto count = [&](int b, int first, int step) -> long long {   // tiles of a key head, strided over its units
            int start, n_new;
            const int n_eff = a.sq.rows(b, a.T, a.max_new, start, n_new);
            const int raw = a.sq.kv_len[b], len = a.sq.keys(b);
            long long s = 0;
            for (int t = first * a.unit_tok; t < n_eff; t += step * a.unit_tok)
                s += unit_tiles(a, raw, len, n_new, min(t + a.unit_tok, n_eff) - 1);
            return s;
        };
        if (one_unit) {
            for (int b = tid; b < B; b += nthr) pre[b + 1] = count(b, 0, 1) * a.n_kv;
        } else {
            for (int b = warp; b < B; b += nthr / 32) {
                long long s = count(b, lane, 32);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                if (lane == 0) pre[b + 1] = s * a.n_kv;
            }
        }
        __syncthreads();
        if (warp == 0) {
            long long run = 0;
            for (int b0 = 0; b0 < B; b0 += 32) {
                long long x = b0 + lane < B ? pre[b0 + lane + 1] : 0;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o) x += y;
                }
                if (b0 + lane < B) pre[b0 + lane + 1] = run + x;
                run += __shfl_sync(0xffffffffu, x, 31);
            }
            __syncwarp();
            const long long chunk = (run + gridDim.x - 1) / gridDim.x;
            const long long at = (long long)blockIdx.x * chunk;
            long long left = run - at < chunk ? run - at : chunk;
            int b = 0, g = 0, qt = 0, kt = 0;
            if (left > 0) {
                // the sequence that tile `at` belongs to
                int c = 0;
                for (int b0 = 0; b0 < B; b0 += 32)
                    c += __popc(__ballot_sync(0xffffffffu, b0 + lane < B && pre[b0 + lane + 1] <= at));
                b = c;
                const long long off = at - (b > 0 ? pre[b] : 0);
                const long long per = (pre[b + 1] - (b > 0 ? pre[b] : 0)) / a.n_kv;
                g = (int)(off / per);
                long long rem = off - g * per;
                // the unit: 32 at a time
                int start, n_new;
                const int n_eff = a.sq.rows(b, a.T, a.max_new, start, n_new), raw = a.sq.kv_len[b], len = a.sq.keys(b);
                for (int u0 = 0;; u0 += 32) {
                    const int t = (u0 + lane) * a.unit_tok;
                    const int n = t < n_eff ? unit_tiles(a, raw, len, n_new, min(t + a.unit_tok, n_eff) - 1) : 0;
                    long long x = n;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const long long y = __shfl_up_sync(0xffffffffu, x, o);
                        if (lane >= o) x += y;
                    }
                    const long long tot = __shfl_sync(0xffffffffu, x, 31);
                    if (rem < tot || tot == 0) {
                        const unsigned m = __ballot_sync(0xffffffffu, x > rem);
                        const int l = m ? __ffs(m) - 1 : 0;
                        qt = u0 + l;
                        kt = (int)(rem - __shfl_sync(0xffffffffu, x - n, l));
                        break;
                    }
                    rem -= tot;
                }
            }
            if (lane == 0) {
                w0[0] = b;
                w0[1] = g;
                w0[2] = qt;
                w0[3] = kt;
                *reinterpret_cast<long long *>(w0 + 4) = left;
                *reinterpret_cast<long long *>(w0 + 6) = chunk;
            }
        }
        fence_async_smem();   // the ring's generic writes before TMA's
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const long long chunk = *reinterpret_cast<const long long *>(w0 + 6);
    Walker wk;
    wk.b = w0[0];
    wk.g = w0[1];
    wk.qt = w0[2];
    wk.kt = w0[3];
    wk.left = *reinterpret_cast<const long long *>(w0 + 4);
    if (wk.left > 0) wk.load(a);
    Seg sg;

    if (warp == 0) {
        // ---------------- TMA producer: lane = box of a tile
        uint32_t seq = 0, qn = 0;
        bool ok = true;
        while (ok && wk.next(a, sg)) {
            if (lane == 0) ok = mbar_wait(q_empty, (qn & 1) ^ 1, abort_flag, status);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(q_full, (uint32_t)(NQ * a.tile_tok * a.G * HD * 2));
                for (int i = 0; i < NQ; ++i)
                    for (int c = 0; c < CH; ++c)
                        tma_load_3d(sQ + i * TB + c * kBox, &tmQ, q_full, c * 64, sg.g * a.G, sg.tok0 + i * a.tile_tok);
            }
            ++qn;
            const int n = sg.k1 - sg.k0;
            const int32_t *tab = a.sq.page_table + (size_t)sg.b * a.sq.max_pages;
            const int absent = a.sq.n_pages << a.sq.page_log2;   // a row outside the pool: zeros
            auto row_of = [&](int tile) -> int {                 // pool row of this lane's box
                if (lane >= a.boxes || tile >= n) return absent;
                const int key = (sg.k0 + tile) * kTile + lane * a.box;
                if (key >= sg.len) return absent;
                const int id = tab[key >> a.sq.page_log2];
                return id >= 0 && id < a.sq.n_pages ? (id << a.sq.page_log2) + (key & ((1 << a.sq.page_log2) - 1)) : absent;
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
                if (lane < a.boxes)
                    for (int c = 0; c < CH; ++c)
                        tma_load_3d(ring + s * TB + c * kBox + lane * a.box * 128, tm, &full[s], c * 64, sg.g, row);
                ++seq;
                return true;
            };
            // K tiles run NQ == 2: one, NQ == 1: two ahead of the V tiles; rows are looked up a tile ahead
            constexpr int AHEAD = NQ == 2 ? 1 : 2;
            int rows[AHEAD + 1];
#pragma unroll
            for (int j = 0; j <= AHEAD; ++j) rows[j] = row_of(j);
#pragma unroll
            for (int j = 0; j < AHEAD; ++j)
                if (ok && j < n) ok = load(&tmK, rows[j]);
            for (int t = 0; ok && t < n; ++t) {
                const int nx = row_of(t + AHEAD + 1);
                ok = load(&tmV, rows[0]);
                if (ok && t + AHEAD < n) ok = load(&tmK, rows[AHEAD]);
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) rows[j] = rows[j + 1];
                rows[AHEAD] = nx;
            }
        }
        if (lane == 0 && *abort_flag) {   // every issued copy must land before the CTA can exit
            if (qn) mbar_drain(q_full, (qn - 1) & 1);
            for (uint32_t i = seq > SLOTS ? seq - SLOTS : 0; i < seq; ++i) mbar_drain(&full[i % SLOTS], (i / SLOTS) & 1);
        }
    } else if (warp == 1) {
        if (lane == 0) {   // ---------------- MMA issuer
            const uint32_t id_s = idesc_bf16(128, kTile, 0), id_pv = idesc_bf16(128, HD, 1);
            const uint32_t aq = smem_u32(sQ), ar = smem_u32(ring);
            uint32_t seq = 0, qn = 0, pn[2] = {0, 0};
            bool ok = true;
            auto take = [&](uint32_t q) -> bool { return mbar_wait(&full[q % SLOTS], (q / SLOTS) & 1, abort_flag, status); };
            while (ok && wk.next(a, sg)) {
                const int n = sg.k1 - sg.k0;
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
                        mma_bf16_ts(tmem + 256 + i * 128, tmem + i * 128 + kk * 8,
                                    smem_desc_sw128(vb + kk * 16 * 128, kBox, 1024), id_pv, !first || kk > 0);
                    if (last) mma_commit(&empty[q % SLOTS]);
                };
                // first scores
                for (int i = 0; ok && i < 2; ++i) {
                    if (ni[i] == 0) continue;
                    const uint32_t q = seq + (NQ == 2 ? 0 : i);
                    if (NQ == 1 || i == 0) ok = take(q);
                    if (!ok) break;
                    tc_fence_after();
                    issue_s(i, q, NQ == 1 || i == 1);
                }
                seq += NQ == 2 ? 1 : (n > 1 ? 2 : 1);
                for (int u = 0; ok && u < ni[0]; ++u) {
                    for (int i = 0; ok && i < 2; ++i) {
                        if (u >= ni[i]) continue;
                        const bool lastuse = NQ == 1 || i == 1;
                        const bool more = u + 1 < ni[i];
                        ok = mbar_wait(&p_full[i], pn[i] & 1, abort_flag, status);
                        ++pn[i];
                        if (ok && (NQ == 1 || i == 0)) ok = take(seq);
                        if (!ok) break;
                        tc_fence_after();
                        issue_pv(i, seq, u == 0, lastuse);
                        if (more) {
                            if (NQ == 1 || i == 0) ok = take(seq + 1);
                            if (!ok) break;
                            tc_fence_after();
                            issue_s(i, seq + 1, lastuse);
                        }
                        if (lastuse) seq += more ? 2 : 1;
                    }
                }
                if (!ok) break;
                mma_commit(q_empty);   // every product of Q is done
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
        const int row_tok = r / a.G, row_h = r - row_tok * a.G;
        const int st = (w & 7) * 32 + lane;          // thread of the stream
        uint32_t sn = 0, on = 0, seq0 = 0;
        bool first_seg = true;
        if (w == 0 && lane == 0) a.meta[blockIdx.x].nseg = 0;
        while (wk.next(a, sg)) {
            const int n = sg.k1 - sg.k0;
            const int ni = NQ == 2 ? n : (n + 1 - i) / 2;
            const int tk = (NQ == 2 ? i * a.tile_tok : 0) + row_tok;
            const bool live = row_tok < a.tile_tok && tk < sg.n_tok;
            const int lim = live ? PagedSeqs::visible(sg.pos0 + tk, sg.len, a.mask_block) : 0;
            const bool warp_live = __any_sync(0xffffffffu, live);
            const int32_t *tab = a.sq.page_table + (size_t)sg.b * a.sq.max_pages;
            float m = -INFINITY, l = 0.f;
            for (int u = 0; u < ni; ++u) {
                const int t = NQ == 2 ? u : 2 * u + i, kt = sg.k0 + t;
                // boxes that have a page (those past the keys count as present: lim cuts them)
                bool here = true;
                if (lane < a.boxes) {
                    const int key = kt * kTile + lane * a.box;
                    if (key < sg.len) {
                        const int id = tab[key >> a.sq.page_log2];
                        here = id >= 0 && id < a.sq.n_pages;
                    }
                }
                const unsigned pages = __ballot_sync(0xffffffffu, here);
                mbar_wait(&s_full[i], sn & 1, abort_flag, status);
                ++sn;
                __syncwarp();
                tc_fence_after();
                if (warp_live) {
                    float v[64];
#pragma unroll
                    for (int c = 0; c < 64; c += 16) tmem_ld_x16(tS + hf * 64 + c, slice16(v + c));
#pragma unroll
                    for (int c = 0; c < 64; c += 16) tmem_ld_wait(slice16(v + c));
                    const int nv = lim - kt * kTile - hf * 64;
                    if (nv < 64) {
#pragma unroll
                        for (int j = 0; j < 64; ++j)
                            if (j >= nv) v[j] = -INFINITY;
                    }
                    if (pages != 0xffffffffu) {
#pragma unroll
                        for (int j = 0; j < 64; ++j)
                            if (!((pages >> ((hf * 64 + j) >> a.box_log2)) & 1)) v[j] = -INFINITY;
                    }
                    float x0 = v[0], x1 = v[1], x2 = v[2], x3 = v[3];
#pragma unroll
                    for (int j = 4; j < 64; j += 4) {
                        x0 = fmaxf(x0, v[j]);
                        x1 = fmaxf(x1, v[j + 1]);
                        x2 = fmaxf(x2, v[j + 2]);
                        x3 = fmaxf(x3, v[j + 3]);
                    }
                    float mx = fmaxf(fmaxf(x0, x1), fmaxf(x2, x3)) * a.scale_log2;
                    xmax[(i * 2 + hf) * 128 + r] = mx;
                    __syncwarp();
                    named_bar_sync(1 + i * 4 + q, 64);   // both halves have read S, too
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
                    float l0 = 0.f, l1 = 0.f;
                    uint32_t pk[32];
#pragma unroll
                    for (int j = 0; j < 64; j += 2) {
                        const float p0 = ex2(fmaf(v[j], a.scale_log2, -mr));
                        const float p1 = ex2(fmaf(v[j + 1], a.scale_log2, -mr));
                        l0 += p0;
                        l1 += p1;
                        const __nv_bfloat162 pp = __floats2bfloat162_rn(p0, p1);
                        pk[j >> 1] = *reinterpret_cast<const uint32_t *>(&pp);
                    }
                    tmem_st_x16(tS + hf * 32, pk);
                    tmem_st_x16(tS + hf * 32 + 16, pk + 16);
                    l += l0 + l1;
                    tmem_st_wait();
                }
                if (NQ == 1 || i == 0) {
                    // a page that ends inside this tile: its slots past the keys are zeroed in V
                    const int e = sg.len - kt * kTile;
                    const int page = 1 << a.sq.page_log2;
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
            if (w == 0 && lane == 0 && sg.k0 == 0 && !whole) {
                PartMeta pm{};
                pm.nseg = 1 + (int)((sg.n - sg.k1 + chunk - 1) / chunk);
                pm.slot = slot;
                pm.tok0 = sg.tok0;
                pm.ntok = sg.n_tok;
                pm.g = sg.g;
                a.meta[blockIdx.x] = pm;
            }
            first_seg = false;
            const size_t out_row = ((size_t)(sg.tok0 + tk) * a.n_q + sg.g * a.G + row_h);
            const size_t part_row = (size_t)slot * a.unit_rows + (size_t)tk * a.G + row_h;
            constexpr int CW = NQ == 2 ? HD / 2 : HD / 4;    // columns of this thread
            const int c0 = (NQ == 2 ? hf : i * 2 + hf) * CW;
            float M = m, L, f0 = 1.f, f1 = 0.f;
            // (o_full also says that every warp of the stream is done with xmax)
            mbar_wait(&o_full[i], on & 1, abort_flag, status);
            if (NQ == 1) mbar_wait(&o_full[i ^ 1], on & 1, abort_flag, status);
            xmax[(i * 2 + hf) * 128 + r] = l;
            __syncwarp();
            named_bar_sync(1 + i * 4 + q, 64);
            L = xmax[i * 256 + r] + xmax[i * 256 + 128 + r];
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
            if (warp_live) {
                const float inv = whole ? (L > 0.f ? 1.0f / L : 0.f) : 1.f;
                const uint32_t t0 = (NQ == 2 ? tO : tmem + 256 + lanes) + c0;
#pragma unroll
                for (int c = 0; c < CW; c += 16) {
                    float o[16];
                    __syncwarp();
                    tmem_ld_x16(t0 + c, o);
                    tmem_ld_wait(o);
                    if (NQ == 1) {
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
                            const __nv_bfloat162 pp = __floats2bfloat162_rn(L > 0.f ? o[e] * inv : 0.f, L > 0.f ? o[e + 1] * inv : 0.f);
                            pk[e >> 1] = *reinterpret_cast<const uint32_t *>(&pp);
                        }
                        uint4 *dst = reinterpret_cast<uint4 *>(a.A + out_row * HD + c0 + c);
                        dst[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                        dst[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
                    } else if (live) {
                        float4 *dst = reinterpret_cast<float4 *>(a.part_o + part_row * HD + c0 + c);
#pragma unroll
                        for (int e = 0; e < 16; e += 4) dst[e >> 2] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                }
                if (live && c0 == 0) {
                    if (!whole) a.part_ml[part_row] = make_float2(M, L);
                    else if (a.lse) a.lse[out_row] = L > 0.f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
                }
            }
            __syncwarp();
            tc_fence_before();
            if (NQ == 1) named_bar_sync(9, 512);   // both streams' O and sums have been read
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

// Joins the slices of the units that were cut, in the order of their keys: one warp per row.
template <int HD>
__global__ void __launch_bounds__(256) k_paged_join(const PtcArgs a) {
    griddep_wait();
    griddep_launch();
    const PartMeta pm = a.meta[blockIdx.x];
    if (pm.nseg <= 0) return;
    constexpr int E = HD / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = pm.ntok * a.G;
    for (int r = blockIdx.y * 8 + warp; r < rows; r += gridDim.y * 8) {
        auto at = [&](int s) -> size_t {   // the first slice, then the next CTAs' first ones
            return (size_t)(s == 0 ? pm.slot : 2 * (blockIdx.x + s)) * a.unit_rows + r;
        };
        float M = -INFINITY;
        for (int s = 0; s < pm.nseg; ++s) M = fmaxf(M, a.part_ml[at(s)].x);
        float L = 0.f, o[E] = {};
        if (M != -INFINITY)
            for (int s = 0; s < pm.nseg; ++s) {
                const size_t p = at(s);
                const float2 ml = a.part_ml[p];
                if (ml.x == -INFINITY) continue;
                const float f = ex2(ml.x - M);
                L = fmaf(ml.y, f, L);
                const float *src = a.part_o + p * HD + lane * E;
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = fmaf(src[e], f, o[e]);
            }
        const float inv = L > 0.f ? 1.0f / L : 0.f;
        const size_t row = (size_t)(pm.tok0 + r / a.G) * a.n_q + pm.g * a.G + r % a.G;
        bf16 *dst = a.A + row * HD + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2)
            *reinterpret_cast<__nv_bfloat162 *>(dst + e) = __floats2bfloat162_rn(o[e] * inv, o[e + 1] * inv);
        if (a.lse && lane == 0) a.lse[row] = L > 0.f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
    }
}

// ---------------------------------------------------------------- host side
bool map3d(CUtensorMap *tm, const void *base, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t s1, uint64_t s2,
           uint32_t b1, uint32_t b2) {
    auto enc = tmap_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {d0, d1, d2};
    cuuint64_t strides[2] = {s1, s2};   // bytes
    cuuint32_t box[3] = {64, b1, b2};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Units {
    int tile_tok, unit_tok, nq, unit_rows;
};

Units units_for(int max_new, int G) {
    Units u;
    u.tile_tok = kTile / G;
    u.nq = max_new > u.tile_tok ? 2 : 1;   // two row tiles where one does not hold a sequence's new rows
    u.unit_tok = u.tile_tok * u.nq;
    u.unit_rows = (max_new < u.unit_tok ? max_new : u.unit_tok) * G;
    return u;
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

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
    int ry = (a.unit_rows + 31) / 32;   // a block's 8 warps take 4 rows each
    return launch_kernel(k_paged_join<HD>, dim3(grid, ry < 1 ? 1 : ry), dim3(256), 0, st, 1, a);
}

}  // namespace

size_t paged_attention_tc_ws_bytes(int max_new, int n_q, int n_kv, int hd) {
    const Units u = units_for(max_new, n_q / n_kv);
    const size_t slots = 2 * (size_t)num_sms();
    return up256(slots * u.unit_rows * hd * 4) + up256(slots * u.unit_rows * 8) + up256((size_t)num_sms() * sizeof(PartMeta)) +
           256;   // room to align the caller's base
}

cudaError_t paged_attention_tc(const PagedAttn &p, void *ws, unsigned *status, cudaStream_t st) {
    const int G = p.n_q / p.n_kv;
    const Units u = units_for(p.max_new, G);
    const int page = 1 << p.sq.page_log2, grid = num_sms();
    PtcArgs a{};
    a.sq = p.sq;
    a.A = static_cast<bf16 *>(p.A);
    a.lse = p.lse;
    a.n_q = p.n_q;
    a.n_kv = p.n_kv;
    a.G = G;
    a.tile_tok = u.tile_tok;
    a.unit_tok = u.unit_tok;
    a.T = p.T;
    a.max_new = p.max_new;
    a.mask_block = p.mask_block;
    a.box = page < kTile ? page : kTile;
    a.box_log2 = p.sq.page_log2 < 7 ? p.sq.page_log2 : 7;
    a.boxes = kTile / a.box;
    a.scale_log2 = p.scale * 1.4426950408889634f;
    a.unit_rows = u.unit_rows;
    uint8_t *w = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(ws) + 255) & ~uintptr_t(255));
    const size_t slots = 2 * (size_t)grid;
    a.part_o = reinterpret_cast<float *>(w);
    w += up256(slots * u.unit_rows * p.hd * 4);
    a.part_ml = reinterpret_cast<float2 *>(w);
    w += up256(slots * u.unit_rows * 8);
    a.meta = reinterpret_cast<PartMeta *>(w);
    CUtensorMap tq, tk, tv;
    const uint64_t hd = (uint64_t)p.hd, rows = (uint64_t)p.sq.n_pages << p.sq.page_log2;
    if (!map3d(&tq, p.Q, hd, (uint64_t)p.n_q, (uint64_t)p.T, hd * 2, (uint64_t)p.q_stride * 2, (uint32_t)G,
               (uint32_t)u.tile_tok) ||
        !map3d(&tk, p.k_pages, hd, (uint64_t)p.n_kv, rows, hd * 2, hd * 2 * p.n_kv, 1, (uint32_t)a.box) ||
        !map3d(&tv, p.v_pages, hd, (uint64_t)p.n_kv, rows, hd * 2, hd * 2 * p.n_kv, 1, (uint32_t)a.box))
        return cudaErrorInvalidValue;
    if (p.hd == 128)
        return u.nq == 2 ? launch_tc<128, 2>(a, grid, tq, tk, tv, status, st) : launch_tc<128, 1>(a, grid, tq, tk, tv, status, st);
    return u.nq == 2 ? launch_tc<64, 2>(a, grid, tq, tk, tv, status, st) : launch_tc<64, 1>(a, grid, tq, tk, tv, status, st);
}

}  // namespace dllm
