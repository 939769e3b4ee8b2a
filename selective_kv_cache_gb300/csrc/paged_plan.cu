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

// Partials of the run that ends at `end` and that share c - 1 begins: its own
// and those of shares c, c + 1, ... that begin before the end.
__device__ __forceinline__ int count_parts(const PagedAttn& a, int c, int end) {
    int parts = 1;
    for (int k0 = c;; k0 += blockDim.x) {
        const int k = k0 + threadIdx.x;
        const int n = __syncthreads_count(k < a.n_cta && a.shares[k].item >= 0 && a.shares[k].u0 < end);
        parts += n;
        if (n < (int)blockDim.x) return parts;
    }
}

// Block c - 1: the rows of the run that share c enters in its middle, if share c
// is the first to do so.  Items of up to 16 rows: the warps are dealt to the
// rows (one each, or several to a row when there are few), a row's warps take
// its partials in turn, eight loads in flight a lane, four dims a lane (lanes
// past head_dim idle), and are joined through shared memory, in order.  A long
// sequence has a partial per CTA, so it is the loads in flight that count: 57
// partials of 4 rows 12 -> 5 us against a warp per row.
template <typename T, int DH>
__global__ void __launch_bounds__(32 * 16) merge_kernel(PagedAttn a) {
    constexpr int kWarps = 16;
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
    const int rows = it.rows * a.G;   // at most 16
    const int parts = count_parts(a, c, end);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // warps of a row: 16 / (rows rounded up to a power of two)
    const int wpr = kWarps >> (32 - __clz(rows - 1));
    const size_t stride = (size_t)2 * a.tile_rows;   // rows from one share's first slot to the next's
    const int m = warp / wpr, sub = warp % wpr, row = m;
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

// The same for items of two 128-row tiles, whose partials lie chunk by chunk
// of four dims, [32][tile_rows] (the attention's lanes are rows): block (c - 1,
// y) takes rows 32 y .., a lane a row and a warp eight of the chunks, so that
// loads are whole lines, and turns them through shared memory into rows.  Few
// partials each; most blocks find nothing to do, so they are small.
__global__ void __launch_bounds__(128) merge_tiles_kernel(PagedAttn a) {
    __shared__ float sO[32][132];
    pdl_wait();
    const int c = blockIdx.x + 1;
    const PagedShare sh = a.shares[c];
    const int prev = a.shares[c - 1].u0;
    if (sh.item < 0 || sh.off == 0 || prev > sh.run + a.run_cost) return;
    const PagedItem it = sh.first;
    const int per_tile = 128 / a.G, t = blockIdx.y >> 2;            // row tile
    const int rows = min(it.rows - t * per_tile, per_tile) * a.G;   // its rows
    const int m0 = 32 * (blockIdx.y & 3);
    if (m0 >= rows) return;
    const int parts = count_parts(a, c, sh.run + a.run_cost + it.units);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, m = t * 128 + m0 + lane;
    float M = -INFINITY, L = 0.f;
    float4 acc[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool live = m0 + lane < rows;
    for (int k = 0; k < parts && live; ++k) {
        const size_t slot = ((size_t)2 * (c - 1 + k) + (k == 0 && prev < sh.run ? 1 : 0)) * a.tile_rows;
        const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + 2 * (slot + m));
        float4 o[8];
#pragma unroll
        for (int x = 0; x < 8; ++x)
            o[x] = *reinterpret_cast<const float4*>(a.part_o + slot * 128 +
                                                    4 * ((size_t)(8 * warp + x) * a.tile_rows + m));
        if (ml.x == -INFINITY) continue;   // saw no key of the row
        const float top = fmaxf(M, ml.x), f = M == -INFINITY ? 0.f : exp2f(M - top), g = exp2f(ml.x - top);
        M = top;
        L = L * f + g * ml.y;
#pragma unroll
        for (int x = 0; x < 8; ++x)
            acc[x] = make_float4(fmaf(g, o[x].x, acc[x].x * f), fmaf(g, o[x].y, acc[x].y * f),
                                 fmaf(g, o[x].z, acc[x].z * f), fmaf(g, o[x].w, acc[x].w * f));
    }
    const float inv = L > 0.f ? 1.0f / L : 0.f;
#pragma unroll
    for (int x = 0; x < 8; ++x)
        *reinterpret_cast<float4*>(&sO[lane][4 * (8 * warp + x)]) =
            make_float4(acc[x].x * inv, acc[x].y * inv, acc[x].z * inv, acc[x].w * inv);
    __syncthreads();
    for (int i = warp; i < 32 && m0 + i < rows; i += 4) {
        const int r = m0 + i;
        store4(reinterpret_cast<__nv_bfloat16*>(a.out) + (int64_t)(it.row0 + t * per_tile + r / a.G) * a.out_stride +
                   (int64_t)(sh.head * a.G + r % a.G) * 128 + 4 * lane,
               *reinterpret_cast<const float4*>(&sO[i][4 * lane]));
    }
}

}  // namespace

cudaError_t launch_paged_plan(const PagedAttn& a, cudaStream_t s) {
    KVR_LAUNCH(items_kernel, dim3((unsigned)((a.n_items + 7) / 8)), dim3(256), 0, s, a);
    KVR_LAUNCH(plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, a);
    return cudaSuccess;
}

cudaError_t launch_paged_merge(int dtype, int head_dim, const PagedAttn& a, cudaStream_t s) {
    if (a.n_cta < 2) return cudaSuccess;
    const dim3 grid((unsigned)a.n_cta - 1), block(32 * 16);
    if (a.tile_rows > kMergeRows) KVR_LAUNCH(merge_tiles_kernel, dim3(grid.x, 8), dim3(128), 0, s, a);
    else if (dtype == KVR_BF16) KVR_LAUNCH(merge_kernel<__nv_bfloat16, 128>, grid, block, 0, s, a);
    else if (head_dim == 64) KVR_LAUNCH(merge_kernel<float, 64>, grid, block, 0, s, a);
    else KVR_LAUNCH(merge_kernel<float, 128>, grid, block, 0, s, a);
    return cudaSuccess;
}

}  // namespace kvr
