// paged_weights_tc.cu -- the attention weight that every key of a paged cache receives from the new rows,
// on the sm_103a tensor cores (bf16 or 8-bit pages):
//
//   score[b, g, j] <- (old score, or 0 for the new rows' own keys)
//                     + sum over rows t of b and heads h of g that see j of 2^(c <Q[t, h], K_j> - lse2[t, h])
//
// with the log-sum-exp that the attention left, so that one pass over the keys and no running maximum is
// needed.  Keys are the 128 lanes, rows the columns of S^T = K Q^T: a thread has one key and adds up the row's
// weights by itself, in the order of the rows; no atomics, the same sum every time.
//
// Work: the key tiles of all (sequence, key head) laid end to end, one CTA per SM.  Where one row tile
// holds a sequence's rows a CTA takes consecutive tiles, so that the queries stay where they are; otherwise every
// grid-th one, as the first tiles of a causal prompt are seen by all rows and the last by few.
//
// Roles: warp 0 finds the items and their pages, warp 1 issues the products, warp 2 loads keys, warp 3 loads
// queries and their log-sum-exp; two groups of four warps take the row tiles in turn.  8-bit keys are widened by eight
// more warps, a key a thread, into TMEM, from where the product takes its first operand (their scale is the thread's own
// factor): through shared memory they would cross it six times, more than its rate at the rate of DRAM.  With few rows the
// keys become fp16, one conversion for two of them, and the queries are brought to fp16 as they come, each row times the
// power of two that puts its largest element into [2^14, 2^15): exact but for what lies 2^-28 below that, and there
// to 2^-39 of it.  With many rows the queries, which change with every key tile, stay bf16 and the keys become bf16 (exactly).
//
// Keys bound it: blocks of 32 rows of 16 sequences over up to 4096 keys (bf16, 32 heads) take 75.5 us, 5.7 TB/s (113 us
// when the rows behind a sequence's last one in its tile were masked instead of zeroed, which left every tile of such a
// sequence to the path that compares each score's row).  Single rows of 64 sequences over up to 8192 keys of 8 bits (28
// heads on 4) take 62 us, 3.6 TB/s: a tile is 16 KB, 0.5 us of a CTA's time, and the product warp's turn takes that (102 us
// with the pages of one tile at a time looked up; 70 us with both groups of warps at every tile and that warp's barriers
// asked one after another).
#include <climits>
#include <cstddef>

#include "e4m3.cuh"
#include "paged_tc.cuh"

namespace dllm {
namespace {

constexpr int kTile = 128;
constexpr int kItems = 12;
constexpr int kMost = 4;                // key tiles whose pages are looked up at a time

struct WeightArgs {
    PagedSeqs sq;
    const float *lse;
    const int32_t *pos_base;            // [B] or NULL
    const uint8_t *k_scale;             // [n_pages, n_kv], 8-bit pages
    const float *score;                 // [B, n_kv, slots]
    float *score_out;
    int32_t *slot_pos;                  // [B, n_kv, slots] or NULL
    int slots;
    int T, n_q, n_kv, G, max_new, mask_block;
    int tile_tok;                       // tokens of a row tile
    int box, boxes;
    int spread;                         // take every grid-th item
    float scale_log2;
};

struct Item {                           // (the first kFields words: a lane of the warp that finds it writes one each)
    int b, g, kt, go;
    int start, n, pos0, len;            // first row, computed rows, position of the first, keys
    int r0, nrt;                        // row tiles [r0, nrt) see the key tile
    int same, last;                     // the queries of the item before are kept; the next one's are others
    int qn, jn;                         // loads of queries, and row tiles, up to the first of this item
    int row[16];                        // pool rows of the tile's boxes
    float aj[16];                       // scale_log2 times the key's scale, 0 without a page
};

constexpr int kFields = 14;
constexpr int kLims = 8;                // loads of queries whose lse, limits and factors are at hand

template <int HD, int N, bool F8> struct Cfg {
    static constexpr int GRP0 = F8 ? 12 : 4;                       // first warp of the two groups
    static constexpr int THREADS = (GRP0 + 8) * 32;
    static constexpr int KB = kTile * HD * (F8 ? 1 : 2);           // bytes of a key tile
    static constexpr int QB = N * HD * 2;
    static constexpr bool HALF = F8 && N < 128;                    // products in fp16
    static_assert(offsetof(Item, row) == kFields * 4, "words of an item");
    static constexpr int FIX = 2 * QB + kLims * (N * 12 + 4) + 128 * 4 + (kPagedMaxSeqs + 1) * 8 + kItems * (int)sizeof(Item) + 1024;
    static constexpr int SLOTS = (227 * 1024 - FIX) / KB < 10 ? (227 * 1024 - FIX) / KB : 10;
    static constexpr int BARS = 6 + 2 * SLOTS + 4 + 8 + 2 * kItems;
    static constexpr size_t kSmem = (size_t)SLOTS * KB + 2 * QB + kLims * (N * 12 + 4) + 128 * 4 + (kPagedMaxSeqs + 1) * 8 +
                                    kItems * sizeof(Item) + BARS * 8 + 32;
    static_assert(kSmem <= 227 * 1024 && SLOTS >= 3, "shared memory");
    // A group that takes every other tile must not ask a barrier two laps ahead, which its phase could not tell from none: items
    // of a slot are all one group's, and keys of tile k are asked for when all products up to tile k - 4 are done.
    static_assert(kItems % 2 == 0 && (!F8 || SLOTS >= 4), "laps");
    static constexpr int DCOLS = N < 32 ? 32 : N;                  // columns of a row tile's scores
    static constexpr int ND = N < 128 ? 4 : 2;                     // row tiles in TMEM, the groups' in turn
};

// Whether the phase is over, without a wait.
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// Shared-memory descriptors (128-byte swizzle, 8 rows of 128 bytes a group) as their two words: the low one has the
// address, the high one is the same for all.
constexpr uint32_t kDescHi = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\tmov.b64 x, {%1, %6};\n\tmov.b64 y, {%2, %6};\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(lead),
        "r"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 y;\n\tmov.b64 y, {%2, %6};\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(lead),
        "r"(kDescHi)
        : "memory");
}
template <int HD, int N, bool F8>
__global__ void __launch_bounds__(Cfg<HD, N, F8>::THREADS, 1)
    k_paged_weights(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK, const WeightArgs a,
                    unsigned *status) {
    using C = Cfg<HD, N, F8>;
    constexpr int SLOTS = C::SLOTS, KB = C::KB, CH = HD / 64, ND = C::ND;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *ring = smem;
    uint8_t *sQ = ring + SLOTS * KB;                                // two row tiles
    float *lse2 = reinterpret_cast<float *>(sQ + 2 * C::QB);        // [kLims][N]
    int *lims = reinterpret_cast<int *>(lse2 + kLims * N);          // [kLims][N]
    float *rs = reinterpret_cast<float *>(lims + kLims * N);        // [kLims][N] a row's power of two (HALF)
    int *least = lims + 2 * kLims * N;                                      // [kLims] the fewest keys that a row of a tile sees
    float *part = reinterpret_cast<float *>(least + kLims);             // [128] the second group's sums
    long long *pre = reinterpret_cast<long long *>(part + 128);
    Item *items = reinterpret_cast<Item *>(pre + kPagedMaxSeqs + 1);
    uint64_t *bars = reinterpret_cast<uint64_t *>(items + kItems);
    uint64_t *q_full = bars, *q_empty = bars + 2, *k_full = bars + 4, *k_empty = k_full + SLOTS;
    uint64_t *a_full = k_empty + SLOTS, *a_empty = a_full + 2, *d_full = a_empty + 2, *d_empty = d_full + 4;
    uint64_t *i_full = d_empty + 4, *i_empty = i_full + kItems, *q_part = i_empty + kItems, *fin = q_part + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + C::BARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (smem_u32(smem) & 1023u) {   // the swizzled tiles need it; the same in every CTA
        if (tid == 0) raise_status(status, DLLM_STATUS_SMEM_LAYOUT);
        griddep_wait();
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 2);               // the load, and the log-sum-exp
            mbar_init(&q_empty[i], 1);
            mbar_init(&a_full[i], 4);
            mbar_init(&a_empty[i], 1);
        }
        for (int i = 0; i < C::ND; ++i) {
            mbar_init(&d_full[i], 1);
            mbar_init(&d_empty[i], 4);
        }
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], F8 ? 4 : 1);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&i_full[i], 1);
            mbar_init(&i_empty[i], 3 + (F8 ? 4 : 0) + (a.spread ? 8 : 4));   // (groups of four: who has the tile)
        }
        mbar_init(q_part, 1);
        mbar_init(fin, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    // rows of a query tile that no load fills read as zeros
    for (int i = tid; i < 2 * C::QB / 16; i += C::THREADS) reinterpret_cast<uint4 *>(sQ)[i] = make_uint4(0, 0, 0, 0);
    griddep_wait();
    griddep_launch();
    // key tiles of every sequence, summed up
    const int B = a.sq.B;
    auto tiles_of = [&](int b, int &start, int &n, int &n_new) -> int {
        n = a.sq.rows(b, a.T, a.max_new, start, n_new);
        if (n <= 0) return 0;
        return (int)(((long long)min(a.sq.keys(b), a.slots) + kTile - 1) / kTile);
    };
    for (int b = tid; b < B; b += C::THREADS) {
        int start, n, n_new;
        pre[b + 1] = (long long)tiles_of(b, start, n, n_new) * a.n_kv;
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
        if (lane == 0) pre[0] = 0;
    }
    fence_async_smem();   // generic writes before TMA's and the products' reads
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const long long total = pre[B];
    // By a whole warp, every lane of which asks: what the wait shows is shown to each.
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status));
    };
    // Item k, or null at the end: handed out in any case, so the wait does not look at the abort flag.
    auto item_at = [&](uint32_t k) -> const Item * {
        const bool got = mbar_wait_through(&i_full[k % kItems], (k / kItems) & 1, 4);
        const Item *r = &items[k % kItems];
        return __all_sync(0xffffffffu, got) && r->go ? r : nullptr;
    };
    auto item_done = [&](uint32_t k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&i_empty[k % kItems]);
    };

    if (warp == 0) {
        // ---------------- items: pages are looked up two, scales one turn ahead, a turn being up to four tiles of a head (a turn
        // takes the latency of a load, longer than the products and weights of a tile)
        const long long chunk = (total + gridDim.x - 1) / gridDim.x;
        long long at = a.spread ? blockIdx.x : (long long)blockIdx.x * chunk;
        const long long end = a.spread ? total : (at + chunk < total ? at + chunk : total);
        const long long step = a.spread ? gridDim.x : 1;
        const int page_log2 = a.sq.page_log2;
        int b = 0, start = 0, n = 0, n_new = 0, len = 0, pos0 = 0, tiles = 0, nrt = 0, g = 0, kt = 0;
        const int box_log2 = __ffs(a.box) - 1, boxes_log2 = __ffs(a.boxes) - 1;
        struct Next {
            int go, b, g, kt, nt, start, n, pos0, len, r0, nrt;
            int id[2], k[2];            // this lane's boxes (number lane and lane + 32 of the nt tiles): page, scale
        };
        auto find = [&](Next &x) {
            x.go = at < end;
            x.nt = 0;
            x.id[0] = x.id[1] = -1;
            x.k[0] = x.k[1] = 127;
            if (!x.go) return;
            bool moved = n == 0;
            while (at >= pre[b + 1]) {
                ++b;
                moved = true;
            }
            if (moved) {
                tiles = tiles_of(b, start, n, n_new);
                pos0 = a.sq.kv_len[b] - n_new;
                len = min(a.sq.keys(b), a.slots);
                nrt = (n + a.tile_tok - 1) / a.tile_tok;
            }
            if (moved || a.spread) {
                const long long off = at - pre[b];
                g = (int)(off / tiles);
                kt = (int)(off - (long long)g * tiles);
            } else if (kt == tiles) {       // (the next tiles: no divisions, this warp paces the small ones)
                kt = 0;
                ++g;
            }
            x.b = b;
            x.g = g;
            x.kt = kt;
            x.nt = 1;
            if (!a.spread) {
                const long long left = end - at;
                x.nt = min(kMost, tiles - kt);
                if (x.nt > left) x.nt = (int)left;
            }
            x.start = start;
            x.n = n;
            x.pos0 = pos0;
            x.len = len;
            x.nrt = nrt;
            // row tiles from the first position on whose row sees key kt * 128 (with one row tile masked all the same)
            const int k0 = kt * kTile, m = a.mask_block;
            x.r0 = 0;
            if (nrt > 1) {
                const long long p = m == 0 ? 0 : (m == 1 ? (long long)k0 : (long long)(k0 / m) * m) - pos0;
                x.r0 = p < a.tile_tok ? 0 : (p >= n ? nrt : (int)p / a.tile_tok);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int key = k0 + ((lane + 32 * j) << box_log2);    // (boxes follow one another through the tiles)
                if (lane + 32 * j < x.nt << boxes_log2 && key < len)
                    x.id[j] = a.sq.page_table[(size_t)b * a.sq.max_pages + (key >> page_log2)];
            }
            if (!a.spread) kt += x.nt;
            at += a.spread ? step : x.nt;
        };
        auto scale = [&](Next &x) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (F8 && (unsigned)x.id[j] < (unsigned)a.sq.n_pages) x.k[j] = a.k_scale[(size_t)x.id[j] * a.n_kv + x.g];
        };
        Next cur{}, n1{}, n2{};
        find(cur);
        find(n1);
        scale(cur);
        bool same = false;
        uint32_t slot = 0, lap = 0;
        int qn = 0, jn = 0;
        bool ended = false;
        for (bool go = true; go;) {
            find(n2);
            scale(n1);
            const bool follows = cur.go && n1.go && n1.b == cur.b && n1.g == cur.g && cur.nrt == 1;
            go = cur.go && !__any_sync(0xffffffffu, *abort_flag);
            // this lane's word of the turn's items, and its boxes' rows and factors
            const int words[kFields] = {cur.b, cur.g, cur.kt, go, cur.start, cur.n, cur.pos0, cur.len, cur.r0, cur.nrt, same, 0, qn - same, jn};
            int word = 0, row[2];
            float aj[2];
#pragma unroll
            for (int i = 0; i < kFields; ++i) word = lane == i ? words[i] : word;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const bool here = (unsigned)cur.id[j] < (unsigned)a.sq.n_pages;
                const int in_page = (cur.kt * kTile + ((lane + 32 * j) << box_log2)) & ((1 << page_log2) - 1);
                row[j] = here ? (cur.id[j] << page_log2) + in_page : a.sq.n_pages << page_log2;   // (outside the pool: zeros)
                // (above 0 where there is a page, even if the product is too small for a number)
                aj[j] = here ? fmaxf(a.scale_log2 * (F8 ? e8m0_f32(cur.k[j]) : 1.f), 1.4e-45f) : 0.f;
            }
            const int nt = go ? cur.nt : 1;       // (one item says that there are no more)
#pragma unroll 1
            for (int t = 0; t < nt; ++t) {
                mbar_wait_through(&i_empty[slot], lap ^ 1, 1);
                __syncwarp();
                Item &it = items[slot];
                if (lane == 11) word = t == nt - 1 && !follows;
                if (lane < kFields) (&it.b)[lane] = word;
                if (lane == 2) ++word;            // the next tile
                if (lane == 10) word = 1;         // with the same queries
                if (lane == 13) ++word;           // (one row tile each)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int x = lane + 32 * j, box = x & (a.boxes - 1);
                    if (go && x >> boxes_log2 == t) {
                        it.row[box] = row[j];
                        it.aj[box] = aj[j];
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&i_full[slot]);
                if (++slot == kItems) {
                    slot = 0;
                    lap ^= 1;
                }
            }
            // (a turn of several tiles has one row tile, one load)
            qn += cur.nrt > 1 ? cur.nrt - cur.r0 : !same;
            jn += cur.nrt > 1 ? cur.nrt - cur.r0 : nt;
            if (!go && !ended) {                  // every other item is a group's: an end for each
                ended = go = true;
                cur.go = 0;
                continue;
            }
            same = follows;
            cur = n1;
            n1 = n2;
        }
    } else if (warp == 1) {
        // ---------------- products
        const uint32_t lead = elect_one();
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t aq = smem_u32(sQ) >> 4, ar = smem_u32(ring) >> 4;
        const uint32_t id_s = idesc_bf16(128, N, 0) & (C::HALF ? ~(1u << 7 | 1u << 10) : ~0u);   // (formats 0: fp16)
        uint32_t slot = 0, lap = 0, qn = 0, jn = 0;
        bool ok = true;
        struct Words {
            int go, r0, nrt, same, last;
        };
        auto words_of = [&](const Item *it) -> Words { return it ? Words{it->go, it->r0, it->nrt, it->same, it->last} : Words{}; };
        Words now = words_of(item_at(0));
        for (uint32_t k = 0; now.go; ++k) {
            const int r0 = now.r0, nrt = now.nrt, same = now.same, last = now.last;
            item_done(k);
            bool known = false;
            Words next{};
            if (ok) {
                // The barriers of the first row tile, and the next item's, are all asked before an answer is looked at: one
                // after another they take this warp longer than anything else.
                const bool fresh = nrt > 1 || !same;
                uint64_t *in = F8 ? &a_full[k & 1] : &k_full[slot];
                const uint32_t in_phase = F8 ? (k >> 1) & 1 : lap;
                const bool t_in = mbar_test(in, in_phase), t_q = !fresh || mbar_test(&q_full[qn & 1], (qn >> 1) & 1),
                           t_d = mbar_test(&d_empty[jn % ND], ((jn / ND) & 1) ^ 1),
                           t_i = mbar_test(&i_full[(k + 1) % kItems], ((k + 1) / kItems) & 1);
                known = __all_sync(0xffffffffu, t_i);
                if (known) next = words_of(&items[(k + 1) % kItems]);
                bool q_in = __all_sync(0xffffffffu, t_q), d_free = __all_sync(0xffffffffu, t_d);
                ok = __all_sync(0xffffffffu, t_in) || wait(in, in_phase);
                const uint32_t kb = ar + slot * (KB >> 4);
                for (int r = r0; ok && r < nrt; ++r, ++jn) {
                    if (fresh) {
                        ok = q_in || wait(&q_full[qn & 1], (qn >> 1) & 1);
                        ++qn;
                    }
                    const uint32_t qi = (qn - 1) & 1, qb = aq + qi * (C::QB >> 4);
                    if (ok) ok = d_free || wait(&d_empty[jn % ND], ((jn / ND) & 1) ^ 1);
                    if (!ok) break;
                    q_in = d_free = false;
                    tc_fence_after();
                    const uint32_t d = tm + (jn % ND) * C::DCOLS;
#pragma unroll
                    for (int kk = 0; kk < HD / 16; ++kk) {
                        const uint32_t qo = (uint32_t)((kk >> 2) * N * 128 + (kk & 3) * 32) >> 4;
                        if (F8) mma_ts(lead, d, tm + 256 + (k & 1) * 64 + kk * 8, qb + qo, id_s, kk > 0);
                        else mma_ss(lead, d, kb + (((kk >> 2) * kTile * 128 + (kk & 3) * 32) >> 4), qb + qo, id_s, kk > 0);
                    }
                    commit_if(lead, &d_full[jn % ND]);
                    if (nrt > 1 || last) commit_if(lead, &q_empty[qi]);
                }
                if (ok) {
                    if (!F8) commit_if(lead, &k_empty[slot]);
                    else if (a.spread) commit_if(lead, &a_empty[k & 1]);   // (else the tile's one d_full says it)
                    if (!F8 && ++slot == SLOTS) {
                        slot = 0;
                        lap ^= 1;
                    }
                }
            }
            now = known ? next : words_of(item_at(k + 1));
        }
        // Nothing of this thread may still run when TMEM is freed, and no arrival that a commit still owes may come when the
        // CTA has gone: its barriers' place is the next one's by then.
        if (lead) {
            mma_commit(fin);
            mbar_drain(fin, 0);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ---------------- keys: lane = (box, 64-dim half of bf16)
        const int box = lane % a.boxes, half = lane / a.boxes;
        uint32_t slot = 0, lap = 0, sent = 0, laps = 0;
        bool ok = true;
        for (uint32_t k = 0;; ++k) {
            const Item *it = item_at(k);
            if (!it) break;
            const int g = it->g, row = it->row[box & 15];
            item_done(k);
            if (!ok || !(ok = wait(&k_empty[slot], lap ^ 1))) continue;
            if (lane == 0) mbar_arrive_expect_tx(&k_full[slot], KB);
            __syncwarp();
            if (F8) {
                if (lane < a.boxes) tma_load_3d(ring + slot * KB + box * a.box * HD, &tmK, &k_full[slot], 0, g, row);
            } else if (lane < a.boxes * CH) {
                tma_load_3d(ring + slot * KB + half * kTile * 128 + box * a.box * 128, &tmK, &k_full[slot], half * 64, g, row);
            }
            sent |= 1u << slot;
            laps = (laps & ~(1u << slot)) | lap << slot;
            if (++slot == SLOTS) {
                slot = 0;
                lap ^= 1;
            }
        }
        if (lane == 0 && *abort_flag)   // every issued copy must land before the CTA can exit
            for (uint32_t i = 0; i < SLOTS; ++i)
                if (sent >> i & 1) mbar_drain(&k_full[i], laps >> i & 1);
    } else if (warp == 3) {
        // ---------------- queries, their log-sum-exp (log2) and the keys that they see
        uint32_t qn = 0, parts = 0;
        bool ok = true;
        const int rows = a.tile_tok * a.G;
        for (uint32_t k = 0;; ++k) {
            const Item *it = item_at(k);
            if (!it) break;
            const int r0 = it->r0, nrt = it->nrt, same = it->same, start = it->start, n = it->n, g = it->g, pos0 = it->pos0, len = it->len;
            item_done(k);
            if (same) continue;
            for (int r = r0; ok && r < nrt; ++r, ++qn) {
                ok = wait(&q_empty[qn & 1], ((qn >> 1) & 1) ^ 1);
                if (!ok) break;
                // The products with load qn - 2 are done, so the groups are with all row tiles but the last four (ND) of them, and
                // no load before qn - 6 is looked at any more.
                static_assert(kLims >= 2 + C::ND + 1, "loads at hand");
                uint8_t *qb = sQ + (qn & 1) * C::QB;
                // The rows that follow a sequence's last one in its last tile are another's: zeros take their place (weight 0
                // without a mask for every score; what they hold may be no numbers).
                const int mine = min(rows, (n - r * a.tile_tok) * a.G);
                const bool touch = C::HALF || mine < rows;   // rows are written here before the products may read them
                uint64_t *bar = touch ? q_part : &q_full[qn & 1];
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, (uint32_t)(rows * HD * 2));
                    for (int c = 0; c < CH; ++c) tma_load_3d(qb + c * N * 128, &tmQ, bar, c * 64, g * a.G, start + r * a.tile_tok);
                }
                if (touch) {
                    ok = wait(q_part, parts & 1);
                    ++parts;
                    if (!ok) break;
                    for (int i = lane; i < (rows - mine) * 8 * CH; i += 32) {
                        const int c = i / ((rows - mine) * 8), x = i - c * (rows - mine) * 8;
                        *reinterpret_cast<uint4 *>(qb + c * N * 128 + mine * 128 + x * 16) = make_uint4(0, 0, 0, 0);
                    }
                    if constexpr (C::HALF) {
                        __syncwarp();
                        constexpr int LR = 32 / N, U = HD / 8 / LR;   // lanes of a row, 16-byte units of a lane
                        const int row = lane / LR, u0 = lane % LR * U;
                        auto unit = [&](int u) {                      // (starting elsewhere in each row: fewer bank conflicts)
                            const int x = u0 + ((u + row) & (U - 1));
                            return reinterpret_cast<uint4 *>(qb + (x >> 3) * N * 128 + row * 128 + (x & 7) * 16);
                        };
                        uint32_t top = 0;
                        for (int u = 0; u < U; ++u) {
                            const uint4 v = *unit(u);
                            for (uint32_t w : {v.x, v.y, v.z, v.w}) top = max(top, max(w & 0x7fffu, (w >> 16) & 0x7fffu));
                        }
                        if (LR == 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                        const int ex = min(max((int)(top >> 7), 15), 254);             // biased exponent of the largest
                        const float f = __uint_as_float((uint32_t)(268 - ex) << 23);   // 2^(14 - (ex - 127))
                        for (int u = 0; u < U; ++u) {
                            uint4 v = *unit(u);
                            for (uint32_t *w : {&v.x, &v.y, &v.z, &v.w}) {
                                const __half2 h = __floats2half2_rn(__uint_as_float(*w << 16) * f, __uint_as_float(*w & 0xffff0000u) * f);
                                *w = *reinterpret_cast<const uint32_t *>(&h);
                            }
                            *unit(u) = v;
                        }
                        if (lane % LR == 0) rs[qn % kLims * N + row] = __uint_as_float((uint32_t)(ex - 14) << 23);
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&q_full[qn & 1]);
                }
                float *l2 = lse2 + qn % kLims * N;
                int *lm = lims + qn % kLims * N, lim0 = INT_MAX;
                for (int i = lane; i < N; i += 32) {
                    const int tok = r * a.tile_tok + i / a.G;
                    float l = INFINITY;         // (no row: the products are zeros, the weights too)
                    int lim = 0;                // a row without keys, or without a number: sees nothing here
                    if (i < mine) {
                        l = 0.f;
                        const float v = a.lse[(size_t)(start + tok) * a.n_q + g * a.G + i % a.G];
                        if (isfinite(v)) {
                            l = v * 1.4426950408889634f;
                            lim = PagedSeqs::visible(pos0 + tok, len, a.mask_block);
                        }
                    }
                    l2[i] = -l;
                    lm[i] = lim;
                    if (i < mine) lim0 = min(lim0, lim);
                }
                lim0 = __reduce_min_sync(0xffffffffu, lim0);
                if (lane == 0) least[qn % kLims] = lim0;
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_full[qn & 1]);
            }
        }
        if (lane == 0 && *abort_flag) {
            for (uint32_t i = qn > 2 ? qn - 2 : 0; i < qn; ++i) mbar_drain(&q_full[i & 1], (i >> 1) & 1);
            if (parts) mbar_drain(q_part, (parts - 1) & 1);
        }
    } else if (F8 && warp < 12) {
        // ---------------- 8-bit keys widened, a key a thread, into TMEM: two groups of four warps, every other tile each
        const int group = (warp - 4) >> 2;
        const int q = warp & 3, r = q * 32 + lane;
        const uint32_t lanes = (uint32_t)(q * 32) << 16;
        uint32_t at = group, phase = 0;
        bool ok = true;
        for (uint32_t k = group;; k += 2) {
            const Item *it = item_at(k);
            if (!it) break;
            item_done(k);
            if (!ok || !(ok = wait(&k_full[at], phase))) continue;
            const uint8_t *kt = ring + at * KB;
            uint4 raw[HD / 16];
#pragma unroll
            for (int u = 0; u < HD / 16; ++u)
                raw[u] = *reinterpret_cast<const uint4 *>(kt + r * HD + ((u ^ ((r * HD >> 7) & (HD / 16 - 1))) << 4));
            __syncwarp();
            if (lane == 0) mbar_arrive(&k_empty[at]);
            at += 2;
            if (at >= SLOTS) {
                at -= SLOTS;
                phase ^= 1;
            }
            // the product with the tile before last, whose place these keys take
            if (a.spread) ok = wait(&a_empty[k & 1], ((k >> 1) & 1) ^ 1);
            else if (k >= 2) ok = wait(&d_full[(k - 2) % ND], ((k - 2) / ND) & 1);
            if (!ok) continue;
            tc_fence_after();
#pragma unroll
            for (int u = 0; u < HD / 16; u += 2) {
                const uint32_t w[8] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w, raw[u + 1].x, raw[u + 1].y, raw[u + 1].z, raw[u + 1].w};
                uint32_t o[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const uint32_t two = e & 1 ? w[e >> 1] >> 16 : w[e >> 1] & 0xffffu;
                    if constexpr (C::HALF) {
                        o[e] = half2_of_e4m3x2(two);
                        continue;
                    }
                    const float2 f = f32_of_e4m3x2(two);
                    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);   // (exact)
                    o[e] = *reinterpret_cast<const uint32_t *>(&h);
                }
                tmem_st_x16(tmem + 256 + (k & 1) * 64 + lanes + u * 8, o);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&a_full[k & 1]);
        }
    } else {
        // ---------------- weights: group of four warps, a key a thread
        const int gr = (warp - C::GRP0) >> 2, q = warp & 3, kl = q * 32 + lane;
        const uint32_t lanes = (uint32_t)(q * 32) << 16;
        const int box = kl / a.box;
        // (one row tile an item: every other item is the group's)
        for (uint32_t k = a.spread ? 0 : gr;; k += a.spread ? 1 : 2) {
            const Item *it = item_at(k);
            if (!it) break;
            const int r0 = it->r0, nrt = it->nrt, qn = it->qn - r0;
            uint32_t jn = it->jn;
            const float aj = it->aj[box];
            const int b = it->b, g = it->g, key = it->kt * kTile + kl, len = it->len, pos0 = it->pos0;
            item_done(k);
            const size_t head_at = ((size_t)b * a.n_kv + g) * a.slots;
            // A key tile of one row tile is one group's, of more the first group writes it.  Old sums early.
            const bool here = aj > 0.f, mine = nrt - r0 == 1 ? (int)(jn & 1) == gr : gr == 0;
            const float old = mine && key < len && key < pos0 ? a.score[head_at + key] : 0.f;
            float2 acc = make_float2(0.f, 0.f), acc2 = acc;
#pragma unroll 1
            for (int r = r0; r < nrt; ++r, ++jn) {
                if ((int)(jn & 1) == gr) {
                    const uint32_t qi = (uint32_t)(qn + r) % kLims;   // (there before the products were: no wait of its own)
                    const float *l2 = lse2 + qi * N;
                    const int *lm = lims + qi * N;
                    wait(&d_full[jn % ND], (jn / ND) & 1);
                    const bool all_seen = __all_sync(0xffffffffu, here && key < least[qi]);
                    const uint32_t tD = tmem + (jn % ND) * C::DCOLS + lanes;
                    __syncwarp();
                    tc_fence_after();
                    constexpr int W = N < 32 ? N : 32;
#pragma unroll 1
                    for (int c = 0; c < N; c += W) {
                        float x[W];
                        if constexpr (W == 32) tmem_ld_x32(tD + c, x);
                        else tmem_ld_x16(tD + c, x);
                        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                        for (int i = 0; i < W; ++i) asm volatile("" : "+f"(x[i]));
                        const float2 aj2 = make_float2(aj, aj);
#pragma unroll
                        for (int i = 0; i < W; i += 4) {
                            const float4 l = *reinterpret_cast<const float4 *>(l2 + c + i);
                            if constexpr (C::HALF) {
                                const float4 f = *reinterpret_cast<const float4 *>(rs + qi * N + c + i);
                                const float2 s0 = mul2(make_float2(x[i], x[i + 1]), make_float2(f.x, f.y));
                                const float2 s1 = mul2(make_float2(x[i + 2], x[i + 3]), make_float2(f.z, f.w));
                                x[i] = s0.x;
                                x[i + 1] = s0.y;
                                x[i + 2] = s1.x;
                                x[i + 3] = s1.y;
                            }
                            const float2 u = fma2(make_float2(x[i], x[i + 1]), aj2, make_float2(l.x, l.y));
                            const float2 v = fma2(make_float2(x[i + 2], x[i + 3]), aj2, make_float2(l.z, l.w));
                            x[i] = u.x;
                            x[i + 1] = u.y;
                            x[i + 2] = v.x;
                            x[i + 3] = v.y;
                        }
                        if (!all_seen) {
#pragma unroll
                            for (int i = 0; i < W; ++i)
                                if (!here || key >= lm[c + i]) x[i] = -INFINITY;
                        }
#pragma unroll
                        for (int i = 0; i < W; i += 4) {
                            acc = add2(acc, make_float2(ex2(x[i]), ex2(x[i + 1])));
                            acc2 = add2(acc2, make_float2(ex2(x[i + 2]), ex2(x[i + 3])));
                        }
                    }
                    // the scores have been read, and what came with the queries: the next product may come
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&d_empty[jn % ND]);
                }
            }
            float sum = (acc.x + acc.y) + (acc2.x + acc2.y);
            if (nrt - r0 > 1) {              // both groups have had row tiles of this key tile
                __syncwarp();
                if (gr == 1) part[kl] = sum;
                named_bar_sync(1, 256);
                if (gr == 0) sum += part[kl];
                named_bar_sync(1, 256);
            }
            if (mine && key < len) {
                a.score_out[head_at + key] = old + sum;
                if (key >= pos0 && a.slot_pos) a.slot_pos[head_at + key] = key + (a.pos_base ? a.pos_base[b] : 0);
            }
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
template <int HD, int N, bool F8>
cudaError_t launch_weights(const WeightArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, unsigned *status, cudaStream_t st) {
    static bool configured[64] = {};   // per device: raise the shared-memory limit once
    int dev = 0;
    cudaGetDevice(&dev);
    using C = Cfg<HD, N, F8>;
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(k_paged_weights<HD, N, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    return launch_kernel(k_paged_weights<HD, N, F8>, dim3(num_sms()), dim3(C::THREADS), C::kSmem, st, 1, tq, tk, a, status);
}
template <int HD, bool F8>
cudaError_t launch_rows(int n, const WeightArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, unsigned *status, cudaStream_t st) {
    if (n == 16) return launch_weights<HD, 16, F8>(a, tq, tk, status, st);
    return n == 32 ? launch_weights<HD, 32, F8>(a, tq, tk, status, st) : launch_weights<HD, 128, F8>(a, tq, tk, status, st);
}

}  // namespace

cudaError_t paged_weights_tc(const PagedWeights &p, bool f8, unsigned *status, cudaStream_t st) {
    const int G = p.n_q / p.n_kv, page = 1 << p.sq.page_log2;
    const long long all = (long long)p.max_new * G;
    const int n = all <= 16 ? 16 : (all <= 32 ? 32 : 128);         // rows of a tile: as many as there are, where they are few
    WeightArgs a{};
    a.sq = p.sq;
    a.lse = p.lse;
    a.pos_base = p.pos_base;
    a.k_scale = p.k_scale;
    a.score = p.score;
    a.score_out = p.score_out;
    a.slot_pos = p.slot_pos;
    a.slots = p.slots;
    a.T = p.T;
    a.n_q = p.n_q;
    a.n_kv = p.n_kv;
    a.G = G;
    a.max_new = p.max_new;
    a.mask_block = p.mask_block;
    a.tile_tok = n / G < p.max_new ? n / G : p.max_new;
    a.box = page < kTile ? page : kTile;
    a.boxes = kTile / a.box;
    a.spread = p.max_new > a.tile_tok;
    a.scale_log2 = p.scale * 1.4426950408889634f;
    CUtensorMap tq, tk;
    const uint64_t hd = (uint64_t)p.hd, rows = (uint64_t)p.sq.n_pages << p.sq.page_log2;
    if (!map3d_bf16(&tq, p.Q, hd, (uint64_t)p.n_q, (uint64_t)p.T, hd * 2, (uint64_t)p.q_stride * 2, (uint32_t)G, (uint32_t)a.tile_tok))
        return cudaErrorInvalidValue;
    const bool wide = p.hd == 128;
    if (f8 ? !map3d(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, wide ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, p.k_pages, hd,
                    (uint64_t)p.n_kv, rows, hd, hd * p.n_kv, (uint32_t)hd, 1, (uint32_t)a.box,
                    wide ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_64B)
           : !map3d_bf16(&tk, p.k_pages, hd, (uint64_t)p.n_kv, rows, hd * 2, hd * 2 * p.n_kv, 1, (uint32_t)a.box))
        return cudaErrorInvalidValue;
    if (f8) return wide ? launch_rows<128, true>(n, a, tq, tk, status, st) : launch_rows<64, true>(n, a, tq, tk, status, st);
    return wide ? launch_rows<128, false>(n, a, tq, tk, status, st) : launch_rows<64, false>(n, a, tq, tk, status, st);
}

}  // namespace dllm
