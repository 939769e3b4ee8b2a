// paged_simt.cu -- attention over the paged cache on the CUDA cores, fp32
// throughout.
//
//   x_rj = cap(scale <q_r, k_j>) + alpha loc_j + beta snk_j - slope |g_r - j|
//   o_r  = sum_j softmax_j(x_rj) v_j,   j in [lo_r, hi_r)
//
// One pass over the keys with a running maximum and sum (base 2).  A CTA of
// four warps walks its share of units (32 keys of one (item, head)): the K and
// V tiles are staged in shared memory as fp32; a warp owns four of the tile's
// 16 rows, its lanes the 32 keys for the scores and the head's dims for the
// output, so softmax statistics are warp reductions and the output stays in
// registers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged.h"

namespace kvr {
namespace {

constexpr int kThreads = 128, kRows = 16, kKeys = 32;

template <int FMT, int DH, int NG>
__global__ void __launch_bounds__(kThreads) paged_simt_kernel(PagedAttn a) {
    constexpr int LD = DH + 4, kLane = DH / 32;   // padded K row; dims of a lane
    __shared__ float sK[kKeys][LD];
    __shared__ float sV[kKeys][DH];
    __shared__ float sQ[kRows][DH];
    __shared__ float sP[4][kKeys][4];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.G;
    constexpr float kLog2e = 1.4426950408889634f;
    for (PagedWalk w(a, a.shares[blockIdx.x], a.shares[blockIdx.x + 1].u0); w.live(); w.next(a, a.items)) {
        const PagedItem& it = w.it;
        const int n = w.n, h = w.h, off = w.off;
        const int b = it.seq, row0 = it.row0, np = it.rows, kv = it.kv;
        __syncthreads();
        for (int e = threadIdx.x; e < kRows * DH; e += kThreads) {
            const int m = e / DH, d = e % DH;
            float x = 0.f;
            if (m < np * G) {
                const int64_t at = (int64_t)(row0 + m / G) * a.q_stride + (int64_t)(h * G + m % G) * DH + d;
                x = FMT == KVR_F32 ? reinterpret_cast<const float*>(a.q)[at]
                                   : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.q)[at]);
            }
            sQ[m][d] = x;
        }
        int lo[4], hi[4], g[4];
        float slope[4], m_run[4], l_run[4], o[4][kLane];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = 4 * warp + j;
            lo[j] = hi[j] = g[j] = 0;
            slope[j] = 0.f;
            if (m < np * G) {
                paged_interval(a, row0 + m / G, kv, &lo[j], &hi[j]);
                g[j] = a.r.pos[row0 + m / G];
                if (a.slopes) slope[j] = a.slopes[h * G + m % G];
            }
            m_run[j] = -INFINITY;
            l_run[j] = 0.f;
#pragma unroll
            for (int d = 0; d < kLane; ++d) o[j][d] = 0.f;
        }
        for (int s = 0; s < n; ++s) {
            const int key0 = (it.klo / kKeys + off + s) * kKeys;
            __syncthreads();
            // keys outside [klo, khi) are staged as zeros, whatever their slots hold
            constexpr int kVec = FMT == KVR_INT4 ? 8 : DH * (FMT == KVR_F32 ? 4 : 2) / 16;
            for (int e = threadIdx.x; e < kKeys * kVec; e += kThreads) {
                const int kk = e / kVec, v = e % kVec, key = key0 + kk;
                float x[2][16];
#pragma unroll
                for (int d = 0; d < 16; ++d) x[0][d] = x[1][d] = 0.f;
                if (key >= it.klo && key < it.khi) {
                    const int id = paged_id(a.p, a.p.table[(int64_t)b * a.p.max_pages + (key >> a.p.page_shift)]);
                    const int64_t row = paged_row(a.p, id, key & ((1 << a.p.page_shift) - 1), h);
#pragma unroll
                    for (int kv2 = 0; kv2 < 2; ++kv2) {
                        const uint8_t* base = kv2 ? a.p.v : a.p.k;
                        if (FMT == KVR_F32) {
                            const float4 w = reinterpret_cast<const float4*>(base + row * (DH * 4))[v];
                            x[kv2][0] = w.x, x[kv2][1] = w.y, x[kv2][2] = w.z, x[kv2][3] = w.w;
                        } else if (FMT == KVR_BF16) {
                            const uint4 w = reinterpret_cast<const uint4*>(base + row * (DH * 2))[v];
                            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                            for (int d = 0; d < 4; ++d) {
                                x[kv2][2 * d] = __uint_as_float(ws[d] << 16);
                                x[kv2][2 * d + 1] = __uint_as_float(ws[d] & 0xffff0000u);
                            }
                        } else {
                            const uint2 w = *reinterpret_cast<const uint2*>(base + row * 64 + 8 * v);
                            const __half2* meta =
                                reinterpret_cast<const __half2*>((kv2 ? a.p.vs : a.p.ks) + row * (4 * NG));
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const float2 so = __half22float2(meta[q * NG / 4]);
                                const uint32_t unit = (q < 2 ? w.x : w.y) >> (16 * (q & 1));
#pragma unroll
                                for (int d = 0; d < 4; ++d)
                                    x[kv2][4 * q + d] = fmaf((float)((unit >> (4 * d)) & 15u), so.x, so.y);
                            }
                        }
                    }
                }
                if (FMT == KVR_INT4) {
#pragma unroll
                    for (int d = 0; d < 16; ++d) {
                        sK[kk][32 * (d / 4) + 4 * v + d % 4] = x[0][d];
                        sV[kk][32 * (d / 4) + 4 * v + d % 4] = x[1][d];
                    }
                } else {
                    constexpr int E = FMT == KVR_F32 ? 4 : 8;
#pragma unroll
                    for (int d = 0; d < E; ++d) {
                        sK[kk][v * E + d] = x[0][d];
                        sV[kk][v * E + d] = x[1][d];
                    }
                }
            }
            __syncthreads();
            // scores: lane = key
            float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
            for (int d = 0; d < DH; d += 4) {
                const float4 k4 = *reinterpret_cast<const float4*>(&sK[lane][d]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 q4 = *reinterpret_cast<const float4*>(&sQ[4 * warp + j][d]);
                    x[j] = fmaf(q4.x, k4.x, fmaf(q4.y, k4.y, fmaf(q4.z, k4.z, fmaf(q4.w, k4.w, x[j]))));
                }
            }
            const int key = key0 + lane;
            float bias = 0.f;
            if (a.loc && (a.loc[(int64_t)b * a.words + (key0 >> 5)] >> lane) & 1u) bias += a.alpha;
            if (a.snk && (a.snk[(int64_t)b * a.words + (key0 >> 5)] >> lane) & 1u) bias += a.beta;
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
                sP[warp][lane][j] = p;
            }
            __syncwarp();
#pragma unroll 4
            for (int kk = 0; kk < kKeys; ++kk) {
                const float4 p4 = *reinterpret_cast<const float4*>(sP[warp][kk]);
                float v[kLane];
#pragma unroll
                for (int d = 0; d < kLane; ++d) v[d] = sV[kk][kLane * lane + d];
#pragma unroll
                for (int d = 0; d < kLane; ++d) {
                    o[0][d] = fmaf(p4.x, v[d], o[0][d]);
                    o[1][d] = fmaf(p4.y, v[d], o[1][d]);
                    o[2][d] = fmaf(p4.z, v[d], o[2][d]);
                    o[3][d] = fmaf(p4.w, v[d], o[3][d]);
                }
            }
        }
        const bool whole = w.whole();
        const size_t slot = ((size_t)blockIdx.x * 2 + (w.first ? 0 : 1)) * a.tile_rows;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = 4 * warp + j;
            if (m >= np * G) continue;
            if (whole) {
                const float inv = l_run[j] > 0.f ? 1.0f / l_run[j] : 0.f;
                const int64_t at =
                    (int64_t)(row0 + m / G) * a.out_stride + (int64_t)(h * G + m % G) * DH + kLane * lane;
#pragma unroll
                for (int d = 0; d < kLane; ++d) {
                    if (FMT == KVR_F32) reinterpret_cast<float*>(a.out)[at + d] = o[j][d] * inv;
                    else reinterpret_cast<__nv_bfloat16*>(a.out)[at + d] = __float2bfloat16(o[j][d] * inv);
                }
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

}  // namespace

cudaError_t launch_paged_simt(int format, int head_dim, int group, const PagedAttn& a, cudaStream_t s) {
    const dim3 grid((unsigned)a.n_cta), block(kThreads);
    if (format == KVR_F32 && head_dim == 64) KVR_LAUNCH(paged_simt_kernel<KVR_F32, 64, 0>, grid, block, 0, s, a);
    else if (format == KVR_F32) KVR_LAUNCH(paged_simt_kernel<KVR_F32, 128, 0>, grid, block, 0, s, a);
    else if (format == KVR_BF16) KVR_LAUNCH(paged_simt_kernel<KVR_BF16, 128, 0>, grid, block, 0, s, a);
    else if (group == 32) KVR_LAUNCH(paged_simt_kernel<KVR_INT4, 128, 4>, grid, block, 0, s, a);
    else if (group == 64) KVR_LAUNCH(paged_simt_kernel<KVR_INT4, 128, 2>, grid, block, 0, s, a);
    else KVR_LAUNCH(paged_simt_kernel<KVR_INT4, 128, 1>, grid, block, 0, s, a);
    return cudaSuccess;
}

}  // namespace kvr
