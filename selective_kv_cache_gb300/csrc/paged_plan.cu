// paged_plan.cu -- sharing one paged attention call over the GPU, and merging
// what was split.
//
// The call's work is a line (paged.h: PagedShare) cut into equal shares,
// whatever the sequences' lengths, which only the device knows.  A run that one
// CTA holds whole is written by it; the others leave unnormalised partial rows
// (at most two per CTA: its first and its last run), merged afterwards in key
// order, so the bits depend on nothing but the inputs.
//
// All kernels here are latency, not bandwidth: a warp per item reads a few
// words per row, one block scans the items, the merge reads each partial once,
// from L2.
#include <cuda_bf16.h>

#include "paged.h"

namespace kvr {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kCoarse = 4096;

__global__ void __launch_bounds__(256) items_kernel(PagedAttn a) {
    pdl_trigger();
    const int i = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (i >= a.n_items) return;
    const PagedItem it = paged_item<32>(a, i, lane);
    if (lane == 0) a.items[i] = it;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PagedAttn a) {
    __shared__ int coarse[kCoarse];
    __shared__ int warp_sum[32];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int step = (a.n_items + kCoarse - 1) / kCoarse;   // items per coarse entry
    int carry = 0;
    for (int base = 0; base < a.n_items; base += kPlanThreads) {
        const int i = base + threadIdx.x;
        const int units = i < a.n_items ? a.items[i].units : 0;
        const int cost = units ? units + a.run_cost : 0;
        int incl = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) warp_sum[w] = incl;
        __syncthreads();
        if (w == 0) {
            int v = warp_sum[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += y;
            }
            warp_sum[lane] = v;
        }
        __syncthreads();
        const int before = carry + (w ? warp_sum[w - 1] : 0) + incl - cost;
        carry += warp_sum[31];
        if (i < a.n_items) {
            a.items[i].before = before;
            if (i % step == 0) coarse[i / step] = before;
        }
        __syncthreads();
    }
    const int H = a.p.n_kv_heads;
    const long long T = (long long)carry * H;
    const int n = paged_shares(a, T);
    for (int c = threadIdx.x; c <= a.n_cta; c += kPlanThreads) {
        PagedShare sh{-1, 0, 0, (int)T, (int)T, {}};
        if (c < n) {
            const int u0 = (int)(T * c / n);
            const int x = u0 / H;   // before_i <= u0 / H exactly when H before_i <= u0
            int l = 0, r = (a.n_items + step - 1) / step - 1;
            while (l < r) {   // last coarse entry at or below x
                const int m = (l + r + 1) >> 1;
                if (coarse[m] <= x) l = m;
                else r = m - 1;
            }
            int i = l * step;
            while (i + 1 < a.n_items && a.items[i + 1].before <= x) ++i;
            sh = paged_share(a, u0, i, a.items[i]);
        }
        a.shares[c] = sh;
    }
}

__device__ __forceinline__ void store4(float* o, float4 v) { *reinterpret_cast<float4*>(o) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* o, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(o) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

constexpr int kMergeRows = 16, kMergeBatch = 8;

// Block (c - 1, y): rows 16 y .. of the run that share c enters in its middle,
// if share c is the first to do so.  Items of up to 16 rows (kWarps = 16): the
// warps are dealt to the rows (one each, or several to a row when there are
// few), a row's warps take its partials in turn, eight loads in flight a lane,
// four dims a lane (lanes past head_dim idle), and are joined through shared
// memory, in order.  A long sequence has a partial per CTA, so it is the loads
// in flight that count: 57 partials of 4 rows 12 -> 5 us against a warp per
// row.  Larger items (kWarps = 4) have many rows and few partials: a warp takes
// rows in turn, and the blocks are small, since most find nothing to do.
template <typename T, int DH, int kWarps>
__global__ void __launch_bounds__(32 * kWarps) merge_kernel(PagedAttn a) {
    __shared__ float sO[kWarps][DH];
    __shared__ float2 sML[kWarps];
    pdl_wait();
    const int c = blockIdx.x + 1;
    const PagedShare sh = a.shares[c];
    const int prev = a.shares[c - 1].u0;
    if (sh.item < 0 || sh.off == 0) return;
    if (prev > sh.run + a.run_cost) return;   // an earlier share began past its first unit
    const PagedItem it = sh.first;
    const int end = sh.run + a.run_cost + it.units;
    const int rows = min(it.rows * a.G - (int)blockIdx.y * kMergeRows, kMergeRows);
    if (rows <= 0) return;
    // partials: shares c - 1, c, ... that begin before the end
    int parts = 1;
    for (int k0 = c;; k0 += 32 * kWarps) {
        const int k = k0 + threadIdx.x;
        const int n = __syncthreads_count(k < a.n_cta && a.shares[k].item >= 0 && a.shares[k].u0 < end);
        parts += n;
        if (n < 32 * kWarps) break;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // warps of a row: 16 / (rows rounded up to a power of two)
    const int wpr = kWarps == 16 ? 16 >> (32 - __clz(rows - 1)) : 1;
    const size_t stride = (size_t)2 * a.tile_rows;   // rows from one share's first slot to the next's
    for (int m = warp / wpr; m < kMergeRows; m += kWarps) {   // one round when kWarps = 16
    const int sub = warp % wpr, row = blockIdx.y * kMergeRows + m;
    if (kWarps < 16 && m >= rows) break;
    const size_t first = (size_t)(c - 1) * stride + (prev >= sh.run ? 0 : a.tile_rows) + row;
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = sub; m < rows && k0 < parts; k0 += wpr * kMergeBatch) {
        float2 ml[kMergeBatch];
        float4 o[kMergeBatch];
#pragma unroll
        for (int x = 0; x < kMergeBatch; ++x) {
            const int k = k0 + x * wpr;
            ml[x] = make_float2(-INFINITY, 0.f);
            o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k < parts) {
                const size_t at = k == 0 ? first : (size_t)(c - 1 + k) * stride + row;
                ml[x] = *reinterpret_cast<const float2*>(a.part_ml + 2 * at);
                if (lane < DH / 4) o[x] = *reinterpret_cast<const float4*>(a.part_o + at * DH + 4 * lane);
            }
        }
        float top = M;
#pragma unroll
        for (int x = 0; x < kMergeBatch; ++x) top = fmaxf(top, ml[x].x);
        const float f = M == -INFINITY ? 0.f : exp2f(M - top);
        M = top;
        L *= f;
        acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
        for (int x = 0; x < kMergeBatch; ++x) {
            // a share that saw no key of the row takes no part
            const float w = ml[x].x == -INFINITY ? 0.f : exp2f(ml[x].x - M);
            if (w != 0.f) {
                L = fmaf(w, ml[x].y, L);
                acc.x = fmaf(w, o[x].x, acc.x);
                acc.y = fmaf(w, o[x].y, acc.y);
                acc.z = fmaf(w, o[x].z, acc.z);
                acc.w = fmaf(w, o[x].w, acc.w);
            }
        }
    }
    if (wpr > 1) {   // block-uniform
        if (lane == 0) sML[warp] = make_float2(M, L);
        if (lane < DH / 4) *reinterpret_cast<float4*>(&sO[warp][4 * lane]) = acc;
        __syncthreads();
        if (sub || m >= rows) return;
        float top = M;
        for (int w = 1; w < wpr; ++w) top = fmaxf(top, sML[warp + w].x);
        const float f = M == -INFINITY ? 0.f : exp2f(M - top);
        L *= f;
        acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
        for (int w = 1; w < wpr; ++w) {
            const float2 ml = sML[warp + w];
            const float g = ml.x == -INFINITY ? 0.f : exp2f(ml.x - top);
            if (g == 0.f) continue;
            L = fmaf(g, ml.y, L);
            if (lane < DH / 4) {
                const float4 o = *reinterpret_cast<const float4*>(&sO[warp + w][4 * lane]);
                acc.x = fmaf(g, o.x, acc.x);
                acc.y = fmaf(g, o.y, acc.y);
                acc.z = fmaf(g, o.z, acc.z);
                acc.w = fmaf(g, o.w, acc.w);
            }
        }
    } else if (m >= rows) {
        return;
    }
    const float inv = L > 0.f ? 1.0f / L : 0.f;
    if (lane < DH / 4)
        store4(reinterpret_cast<T*>(a.out) + (int64_t)(it.row0 + row / a.G) * a.out_stride +
                   (int64_t)(sh.head * a.G + row % a.G) * DH + 4 * lane,
               make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    }
}

template <typename T, int DH>
cudaError_t merge(const PagedAttn& a, cudaStream_t s) {
    const dim3 grid((unsigned)a.n_cta - 1, (unsigned)((a.positions * a.G + kMergeRows - 1) / kMergeRows));
    if (a.tile_rows <= kMergeRows) KVR_LAUNCH(merge_kernel<T, DH, 16>, grid, dim3(32 * 16), 0, s, a);
    else if constexpr (sizeof(T) == 2) KVR_LAUNCH(merge_kernel<T, DH, 4>, grid, dim3(32 * 4), 0, s, a);
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_paged_plan(const PagedAttn& a, cudaStream_t s) {
    KVR_LAUNCH(items_kernel, dim3((unsigned)((a.n_items + 7) / 8)), dim3(256), 0, s, a);
    KVR_LAUNCH(plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, a);
    return cudaSuccess;
}

cudaError_t launch_paged_merge(int dtype, int head_dim, const PagedAttn& a, cudaStream_t s) {
    if (a.n_cta < 2) return cudaSuccess;
    if (dtype == KVR_BF16) return merge<__nv_bfloat16, 128>(a, s);
    return head_dim == 64 ? merge<float, 64>(a, s) : merge<float, 128>(a, s);
}

}  // namespace kvr
