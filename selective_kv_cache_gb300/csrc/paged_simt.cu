// paged_simt.cu -- attention over fp32 pages on the CUDA cores, fp32
// throughout (the tensor cores would round the products).
//
//   x_rj = cap(scale <q_r, k_j>) + alpha loc_j + beta snk_j - slope |g_r - j|
//   o_r  = sum_j softmax_j(x_rj) v_j,   j in [lo_r, hi_r)
//
// One pass over the keys with a running maximum and sum (base 2).  A CTA of
// four warps walks its share of units (32 keys of one (item, head)).  A warp
// owns four of the item's 16 rows, its lanes the 32 keys for the scores and the
// head's dims for the output, so softmax statistics are warp reductions and the
// output stays in registers.  The next K tile is copied while the output's
// products run and the next V tile while the scores' do, so one buffer of each
// is enough and four CTAs fit an SM.  Shared memory's reads bound it: 8
// wavefronts of K and q for 16 products a lane.  Measured: 4.49 ms, 21 TFLOP/s, at
// 8 x 300 rows over 4096 keys of a 32/8-head model; 25 us at 2 x 64 rows over 1024
// keys of 4 heads of 64.  Tiles twice as tall and wide (255 registers, two CTAs an
// SM) took 4.10 ms and 31 us.
#include <type_traits>

#include "paged.h"
#include "ptx.cuh"

namespace kvr {
namespace {

constexpr int kThreads = 128, kRows = 16, kKeys = 32;

__device__ __forceinline__ void copy16(void* dst, const uint8_t* src, bool take) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(take ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copy_wait1() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

// 32 rows of K or V from key0 on; keys outside [klo, khi) become zeros, whatever their slots hold.
template <int DH, int LD>
__device__ __forceinline__ void stage(const PagedAttn& a, const PagedItem& it, int h, const uint8_t* base, int key0,
                                      float (*dst)[LD]) {
    constexpr int kVec = DH / 4;
#pragma unroll
    for (int e0 = 0; e0 < kKeys * kVec; e0 += kThreads) {
        const int e = e0 + threadIdx.x, kk = e / kVec, v = e % kVec, key = key0 + kk;
        const uint8_t* src = base;
        const bool take = key >= it.klo && key < it.khi;
        if (take) {
            const int id =
                paged_id(a.p, a.p.table[(int64_t)it.seq * a.p.max_pages + (key >> a.p.page_shift)]);
            src += paged_row(a.p, id, key & ((1 << a.p.page_shift) - 1), h) * (DH * 4) + 16 * v;
        }
        copy16(&dst[kk][4 * v], src, take);
    }
}

template <int DH>
struct alignas(16) SimtTiles {
    float k[kKeys][DH + 4];   // padded: lanes read different keys' rows
    float v[kKeys][DH];
    float q[kRows][DH];
    float p[4][kKeys][4];
    PagedItem items[kPagedInline];
};

template <int DH>
__global__ void __launch_bounds__(kThreads) paged_simt_kernel(PagedAttn a) {
    constexpr int kLane = DH / 32;   // dims of a lane
    using Dims = std::conditional_t<kLane == 2, float2, float4>;
    extern __shared__ __align__(16) uint8_t smem[];
    SimtTiles<DH>& sm = *reinterpret_cast<SimtTiles<DH>*>(smem);
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.G;
    constexpr float kLog2e = 1.4426950408889634f;
    PagedShare sh;
    int u1;
    if (a.planned) {
        sh = a.shares[blockIdx.x];
        u1 = a.shares[blockIdx.x + 1].u0;
    } else {
        sh = paged_inline_share(a, sm.items, &u1);
    }
    for (PagedWalk w(a, sh, u1); w.live(); w.next(a, a.planned ? a.items : sm.items)) {
        const PagedItem& it = w.it;
        const int n = w.n, h = w.h;
        const int b = it.seq, row0 = it.row0, live = it.rows * G;
        const int key_first = (it.klo / kKeys + w.off) * kKeys;
        __syncthreads();
        stage<DH, DH + 4>(a, it, h, a.p.k, key_first, sm.k);
        copy_commit();
        stage<DH, DH>(a, it, h, a.p.v, key_first, sm.v);
        copy_commit();
#pragma unroll
        for (int e0 = 0; e0 < kRows * DH; e0 += 4 * kThreads) {
            const int e = e0 + 4 * threadIdx.x, m = e / DH, d = e % DH;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (m < live)
                x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) +
                                                     (int64_t)(row0 + m / G) * a.q_stride +
                                                     (int64_t)(h * G + m % G) * DH + d);
            *reinterpret_cast<float4*>(&sm.q[m][d]) = x;
        }
        int lo[4], hi[4], g[4];
        float slope[4], m_run[4], l_run[4], o[4][kLane];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = 4 * warp + j;
            lo[j] = hi[j] = g[j] = 0;
            slope[j] = 0.f;
            if (m < live) {
                paged_interval(a, row0 + m / G, it.kv, &lo[j], &hi[j]);
                g[j] = a.r.pos[row0 + m / G];
                if (a.slopes) slope[j] = a.slopes[h * G + m % G];
            }
            m_run[j] = -INFINITY;
            l_run[j] = 0.f;
#pragma unroll
            for (int d = 0; d < kLane; ++d) o[j][d] = 0.f;
        }
        for (int s = 0; s < n; ++s) {
            const int key0 = key_first + s * kKeys, key = key0 + lane;
            float bias = 0.f;
            if (a.loc && (a.loc[(int64_t)b * a.words + (key0 >> 5)] >> lane) & 1u) bias += a.alpha;
            if (a.snk && (a.snk[(int64_t)b * a.words + (key0 >> 5)] >> lane) & 1u) bias += a.beta;
            copy_wait1();
            __syncthreads();
            // scores: lane = key
            float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
            for (int d = 0; d < DH; d += 4) {
                const float4 k4 = *reinterpret_cast<const float4*>(&sm.k[lane][d]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 q4 = *reinterpret_cast<const float4*>(&sm.q[4 * warp + j][d]);
                    x[j] = fmaf(q4.x, k4.x, fmaf(q4.y, k4.y, fmaf(q4.z, k4.z, fmaf(q4.w, k4.w, x[j]))));
                }
            }
            __syncthreads();
            if (s + 1 < n) stage<DH, DH + 4>(a, it, h, a.p.k, key0 + kKeys, sm.k);
            copy_commit();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float y = x[j] * a.scale;
                if (a.softcap > 0.f) y = a.softcap * tanhf(y / a.softcap);
                y += bias;
                y = fmaf(-slope[j], (float)abs(g[j] - key), y);
                y = key >= lo[j] && key < hi[j] ? y * kLog2e : -INFINITY;
                float mx = y;
#pragma unroll
                for (int z = 16; z > 0; z >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, z));
                const float m_new = fmaxf(m_run[j], mx);
                const float base = m_new == -INFINITY ? 0.f : m_new;
                const float p = exp2f(y - base);
                const float f = exp2f(m_run[j] - base);
                float sum = p;
#pragma unroll
                for (int z = 16; z > 0; z >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, z);
                m_run[j] = m_new;
                l_run[j] = l_run[j] * f + sum;
#pragma unroll
                for (int d = 0; d < kLane; ++d) o[j][d] *= f;
                sm.p[warp][lane][j] = p;
            }
            copy_wait1();
            __syncthreads();
#pragma unroll 4
            for (int kk = 0; kk < kKeys; ++kk) {
                const float4 p4 = *reinterpret_cast<const float4*>(sm.p[warp][kk]);
                float v[kLane];
                *reinterpret_cast<Dims*>(v) = *reinterpret_cast<const Dims*>(&sm.v[kk][kLane * lane]);
#pragma unroll
                for (int d = 0; d < kLane; ++d) {
                    o[0][d] = fmaf(p4.x, v[d], o[0][d]);
                    o[1][d] = fmaf(p4.y, v[d], o[1][d]);
                    o[2][d] = fmaf(p4.z, v[d], o[2][d]);
                    o[3][d] = fmaf(p4.w, v[d], o[3][d]);
                }
            }
            __syncthreads();
            if (s + 1 < n) stage<DH, DH>(a, it, h, a.p.v, key0 + kKeys, sm.v);
            copy_commit();
        }
        const bool whole = w.whole();
        const size_t slot = ((size_t)blockIdx.x * 2 + (w.first ? 0 : 1)) * a.tile_rows;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = 4 * warp + j;
            if (m >= live) continue;
            if (whole) {
                const float inv = l_run[j] > 0.f ? 1.0f / l_run[j] : 0.f;
                float* out = static_cast<float*>(a.out) + (int64_t)(row0 + m / G) * a.out_stride +
                             (int64_t)(h * G + m % G) * DH + kLane * lane;
#pragma unroll
                for (int d = 0; d < kLane; ++d) out[d] = o[j][d] * inv;
            } else {
#pragma unroll
                for (int d = 0; d < kLane; ++d) a.part_o[(slot + m) * DH + kLane * lane + d] = o[j][d];
                if (lane == 0) {
                    a.part_ml[2 * (slot + m)] = m_run[j];
                    a.part_ml[2 * (slot + m) + 1] = l_run[j];
                }
            }
        }
    }
}

template <int DH>
cudaError_t launch(const PagedAttn& a, cudaStream_t s) {
    constexpr int kSmem = (int)sizeof(SimtTiles<DH>);
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(paged_simt_kernel<DH>, kSmem, &allowed);
    if (e != cudaSuccess) return e;
    KVR_LAUNCH(paged_simt_kernel<DH>, dim3((unsigned)a.n_cta), dim3(kThreads), kSmem, s, a);
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_paged_simt(int head_dim, const PagedAttn& a, cudaStream_t s) {
    return head_dim == 64 ? launch<64>(a, s) : launch<128>(a, s);
}

}  // namespace kvr
