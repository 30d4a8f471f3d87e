// paged_attention.cu -- attention of ragged new rows over a paged cache on the CUDA cores
// (fp32).
//
//   A[t, h] = softmax_j(<Q[t, h], K_j> scale) V_j  over the keys j < visible(pos(t))
//
// Work is cut as in paged_sched.cuh: units of 32 rows (token, head of the group) over 64-key
// tiles, two CTAs per SM (hd 64) or one.  A CTA holds its rows' queries in shared memory and takes
// one key tile after another, the next one's K and V coming in by cp.async meanwhile; a thread
// forms 2 x 4 scores and
// later 2 x HD/16 outputs from 16-byte shared loads, and each row's running maximum and sum
// (fp32) are kept by the 16 lanes that hold its scores.  fp32 multiply-adds bound it from
// about 8 rows on; tensor cores would round the products to TF32.
#include "paged_sched.cuh"

namespace dllm {
namespace {

constexpr int kR = 32;        // rows of a unit
constexpr int kK = 64;        // keys of a tile
constexpr int kT = 256;

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
    static constexpr int LD = HD + 4;                    // row pitch: 16-byte reads of 8 rows meet no bank twice
    static constexpr int kPerSm = HD == 64 ? 2 : 1;      // CTAs per SM (shared memory)
    static constexpr size_t kSmem = (size_t)(kR * LD + 4 * kK * LD + kR * (kK + 4)) * 4 + 2 * kK + 64;
};

template <int HD>
__global__ void __launch_bounds__(kT, F32Cfg<HD>::kPerSm) k_paged_attention_f32(const F32Args a) {
    constexpr int LD = F32Cfg<HD>::LD, V4 = HD / 4;
    extern __shared__ __align__(16) float sm[];
    float *sQ = sm, *ring = sQ + kR * LD, *sP = ring + 4 * kK * LD;   // ring: K, V of two tiles; sP [kR][kK + 4]
    uint8_t *pages = reinterpret_cast<uint8_t *>(sP + kR * (kK + 4));  // key has a page, of two tiles
    __shared__ __align__(16) int w0[8];
    __shared__ long long pre[kPagedMaxSeqs + 1];
    const int tid = threadIdx.x;
    griddep_wait();
    griddep_launch();
    schedule_start(a.s, pre, w0);
    __syncthreads();
    const long long chunk = *reinterpret_cast<const long long *>(w0 + 6);
    Walker wk = walk_from(a.s, w0);
    if (tid == 0) a.s.meta[blockIdx.x].nseg = 0;
    // thread = rows 2 ty, 2 ty + 1; scores of keys tx + 16 j; outputs of dims 4 tx.. (and 64 + 4 tx..)
    const int ty = tid >> 4, tx = tid & 15;
    const int G = a.s.G;
    bool first = true;
    Seg sg;
    while (wk.next(a.s, sg)) {
        const int32_t *tab = a.s.sq.page_table + (size_t)sg.b * a.s.sq.max_pages;
        auto load = [&](int kt) {   // K and V of a tile into its half of the ring
            float *dK = ring + (kt & 1) * 2 * kK * LD, *dV = dK + kK * LD;
            for (int i = tid; i < kK * V4; i += kT) {
                const int j = i / V4, e = i - j * V4, key = kt * kK + j;
                int id = -1;
                if (key < sg.len) id = tab[key >> a.s.sq.page_log2];
                const bool on = id >= 0 && id < a.s.sq.n_pages;
                const size_t row = on ? ((size_t)id << a.s.sq.page_log2) + (key & ((1 << a.s.sq.page_log2) - 1)) : 0;
                const size_t at = (row * a.s.n_kv + sg.g) * HD + e * 4;
                cp16(dK + j * LD + e * 4, a.Kp + at, on);
                cp16(dV + j * LD + e * 4, a.Vp + at, on);
                if (e == 0) pages[(kt & 1) * kK + j] = on;
            }
            cp_commit();
        };
        __syncthreads();   // the previous segment is done with shared memory
        for (int i = tid; i < kR * V4; i += kT) {
            const int r = i / V4, e = i - r * V4;
            const bool on = r < sg.nrows;
            const int row = sg.row0 + (on ? r : 0);
            const size_t t = (size_t)(sg.start + row / G);
            cp16(sQ + r * LD + e * 4, a.Q + t * a.q_stride + (size_t)(sg.g * G + row % G) * HD + e * 4, on);
        }
        load(sg.k0);
        int lim[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int r = 2 * ty + x;
            lim[x] = r < sg.nrows ? PagedSeqs::visible(sg.pos0 + (sg.row0 + r) / G, sg.len, a.s.mask_block) : 0;
        }
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        float o[2][V4 / 16][4] = {};
        for (int kt = sg.k0; kt < sg.k1; ++kt) {
            cp_wait<0>();
            __syncthreads();                     // the tile is here; the other half of the ring and P are free
            if (kt + 1 < sg.k1) load(kt + 1);
            const float *sK = ring + (kt & 1) * 2 * kK * LD, *sV = sK + kK * LD;
            const uint8_t *here = pages + (kt & 1) * kK;
            float s[2][4] = {};
#pragma unroll 4
            for (int d = 0; d < HD; d += 4) {
                const float4 q0 = *reinterpret_cast<const float4 *>(sQ + (2 * ty) * LD + d);
                const float4 q1 = *reinterpret_cast<const float4 *>(sQ + (2 * ty + 1) * LD + d);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 k = *reinterpret_cast<const float4 *>(sK + (tx + 16 * j) * LD + d);
                    s[0][j] = fmaf(q0.x, k.x, fmaf(q0.y, k.y, fmaf(q0.z, k.z, fmaf(q0.w, k.w, s[0][j]))));
                    s[1][j] = fmaf(q1.x, k.x, fmaf(q1.y, k.y, fmaf(q1.z, k.z, fmaf(q1.w, k.w, s[1][j]))));
                }
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = tx + 16 * j;
                    s[x][j] = kt * kK + key < lim[x] && here[key] ? s[x][j] * a.scale_log2 : -INFINITY;
                    mx = fmaxf(mx, s[x][j]);
                }
#pragma unroll
                for (int c = 8; c > 0; c >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, c));
                const float mn = fmaxf(m[x], mx);
                const float f = mn == -INFINITY ? 1.f : exp2f(m[x] - mn);
                const float ref = mn == -INFINITY ? 0.f : mn;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = exp2f(s[x][j] - ref);
                    sum += p;
                    sP[(2 * ty + x) * (kK + 4) + tx + 16 * j] = p;
                }
                l[x] = l[x] * f + sum;           // this lane's keys
                m[x] = mn;
#pragma unroll
                for (int c = 0; c < V4 / 16; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[x][c][e] *= f;
            }
            __syncwarp();                        // (a row's weights are written and read by one warp)
            const int end = min(kK, sg.len - kt * kK);   // (values past the keys were read as zeros)
#pragma unroll 2
            for (int j = 0; j < end; j += 4) {
                const float4 p0 = *reinterpret_cast<const float4 *>(sP + (2 * ty) * (kK + 4) + j);
                const float4 p1 = *reinterpret_cast<const float4 *>(sP + (2 * ty + 1) * (kK + 4) + j);
                const float w[2][4] = {{p0.x, p0.y, p0.z, p0.w}, {p1.x, p1.y, p1.z, p1.w}};
#pragma unroll
                for (int y = 0; y < 4; ++y)
#pragma unroll
                    for (int c = 0; c < V4 / 16; ++c) {
                        const float4 v = *reinterpret_cast<const float4 *>(sV + (j + y) * LD + c * 64 + tx * 4);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            o[x][c][0] = fmaf(w[x][y], v.x, o[x][c][0]);
                            o[x][c][1] = fmaf(w[x][y], v.y, o[x][c][1]);
                            o[x][c][2] = fmaf(w[x][y], v.z, o[x][c][2]);
                            o[x][c][3] = fmaf(w[x][y], v.w, o[x][c][3]);
                        }
                    }
            }
        }
        cp_wait<0>();
        const bool whole = sg.k0 == 0 && sg.k1 == sg.n;
        const int slot = blockIdx.x * 2 + (first ? 0 : 1);
        first = false;
        if (tid == 0 && sg.k0 == 0 && !whole) a.s.meta[blockIdx.x] = part_of(sg, slot, chunk);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float L = l[x];
#pragma unroll
            for (int c = 8; c > 0; c >>= 1) L += __shfl_xor_sync(0xffffffffu, L, c);
            const int r = 2 * ty + x;
            if (r >= sg.nrows) continue;
            const float inv = whole ? (L > 0.f ? 1.0f / L : 0.f) : 1.f;
            const int row = sg.row0 + r;
            const size_t out = (size_t)(sg.start + row / G) * a.s.n_q + sg.g * G + row % G;
            const size_t part = (size_t)slot * a.s.unit_rows + r;
            float *dst = whole ? a.A + out * HD : a.s.part_o + part * HD;
#pragma unroll
            for (int c = 0; c < V4 / 16; ++c)
                *reinterpret_cast<float4 *>(dst + c * 64 + tx * 4) =
                    make_float4(o[x][c][0] * inv, o[x][c][1] * inv, o[x][c][2] * inv, o[x][c][3] * inv);
            if (tx == 0) {
                if (!whole) a.s.part_ml[part] = make_float2(m[x], L);
                else if (a.s.lse) a.s.lse[out] = L > 0.f ? (m[x] + log2f(L)) * 0.6931471805599453f : -INFINITY;
            }
        }
    }
}

int f32_rows(int max_new, int G) {
    const long long r = (long long)max_new * G;
    return r < kR ? (int)r : kR;
}

template <int HD>
cudaError_t launch_f32(const F32Args &a, int grid, cudaStream_t st) {
    static bool configured[64] = {};   // per device: raise the shared-memory limit once
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(k_paged_attention_f32<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)F32Cfg<HD>::kSmem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    const cudaError_t e = launch_kernel(k_paged_attention_f32<HD>, dim3(grid), dim3(kT), F32Cfg<HD>::kSmem, st, 1, a);
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
    return p.hd == 128 ? launch_f32<128>(a, grid, st) : launch_f32<64>(a, grid, st);
}

}  // namespace dllm
