// paged_plan.cu -- sharing one paged attention call over the GPU, and merging
// what was split.
//
// The call's work is a line of units: for each item (a run of packed rows of
// one sequence), for each K/V head, the runs of unit_keys keys its rows can
// see.  CTA c takes units [c T / n, (c + 1) T / n): equal shares whatever the
// sequences' lengths, which only the device knows.  An (item, head) that one
// CTA holds whole is written by it; the others leave unnormalised partial rows
// (at most two per CTA: its first and its last), merged afterwards in key
// order, so the bits depend on nothing but the inputs.
//
// Both kernels here are latency, not bandwidth: the plan is one block reading
// a few words per row; the merge reads each partial once, from L2.
#include <cuda_bf16.h>

#include "paged.h"

namespace kvr {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kCoarse = 4096;

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PagedAttn a) {
    __shared__ int coarse[kCoarse];
    __shared__ int warp_sum[32];
    __shared__ int s_total;
    pdl_trigger();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int step = (a.n_items + kCoarse - 1) / kCoarse;   // items per coarse entry
    int carry = 0;
    for (int base = 0; base < a.n_items; base += kPlanThreads) {
        const int i = base + threadIdx.x;
        PagedItem it{};
        if (i < a.n_items) it = paged_item(a, i);
        int incl = it.units;
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
        it.before = carry + (w ? warp_sum[w - 1] : 0) + incl - it.units;
        carry += warp_sum[31];
        if (i < a.n_items) {
            a.items[i] = it;
            if (i % step == 0) coarse[i / step] = it.before;
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) s_total = carry;
    __syncthreads();
    const int H = a.p.n_kv_heads;
    const long long T = (long long)s_total * H;
    const int n = (int)min((long long)a.n_cta, T);
    for (int c = threadIdx.x; c <= a.n_cta; c += kPlanThreads) {
        PagedShare sh{-1, 0, 0, (int)T, {}};
        if (c < n) {
            sh.u0 = (int)(T * c / n);
            const int x = sh.u0 / H;   // before_i <= u0 / H exactly when H before_i <= u0
            int l = 0, r = (a.n_items + step - 1) / step - 1;
            while (l < r) {   // last coarse entry at or below x
                const int m = (l + r + 1) >> 1;
                if (coarse[m] <= x) l = m;
                else r = m - 1;
            }
            int i = l * step;
            while (i + 1 < a.n_items && a.items[i + 1].before <= x) ++i;
            sh.first = a.items[i];
            const int rem = sh.u0 - H * sh.first.before, units = sh.first.units;
            sh.item = i;
            sh.head = rem / units;
            sh.off = rem - sh.head * units;
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

constexpr int kMergeWarps = 16, kMergeRows = 16, kMergeBatch = 8;

// Block (c - 1, y): rows 16 y .. of the (item, head) that share c enters in
// its middle, if share c is the first to do so.  The 16 warps are dealt to the
// rows (one each, or several to a row when there are few), a row's warps take
// its partials in turn, eight loads in flight a lane, four dims a lane (lanes
// past head_dim idle); a row's warps are joined through shared memory, in
// order.  A long sequence has a partial per CTA, so it is the loads in flight that
// count here: 57 partials of 4 rows 12 -> 4 us against a warp per row.
template <typename T, int DH>
__global__ void __launch_bounds__(32 * kMergeWarps) merge_kernel(PagedAttn a) {
    __shared__ float sO[kMergeWarps][DH];
    __shared__ float2 sML[kMergeWarps];
    pdl_wait();
    const int c = blockIdx.x + 1;
    const PagedShare sh = a.shares[c];
    const int prev = a.shares[c - 1].u0;
    if (sh.item < 0 || sh.off == 0) return;
    const int start = sh.u0 - sh.off;
    if (prev > start) return;
    const PagedItem it = sh.first;
    const int end = start + it.units;
    const int rows = min(it.rows * a.G - (int)blockIdx.y * kMergeRows, kMergeRows);
    if (rows <= 0) return;
    // partials: shares c - 1, c, ... that begin before the end
    int parts = 1;
    for (int k0 = c;; k0 += 32 * kMergeWarps) {
        const int k = k0 + threadIdx.x;
        const int n = __syncthreads_count(k < a.n_cta && a.shares[k].item >= 0 && a.shares[k].u0 < end);
        parts += n;
        if (n < 32 * kMergeWarps) break;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wpr = kMergeWarps >> (32 - __clz(rows - 1));   // warps of a row: 16 / (rows rounded up to a power of two)
    const int m = warp / wpr, sub = warp % wpr, row = blockIdx.y * kMergeRows + m;
    const size_t stride = (size_t)2 * a.tile_rows;   // rows from one share's first slot to the next's
    const size_t first = (size_t)(c - 1) * stride + (prev == start ? 0 : a.tile_rows) + row;
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

}  // namespace

cudaError_t launch_paged_plan(const PagedAttn& a, cudaStream_t s) {
    KVR_LAUNCH(plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, a);
    return cudaSuccess;
}

cudaError_t launch_paged_merge(int dtype, int head_dim, const PagedAttn& a, cudaStream_t s) {
    if (a.n_cta < 2) return cudaSuccess;
    const dim3 grid((unsigned)a.n_cta - 1, (unsigned)((a.positions * a.G + kMergeRows - 1) / kMergeRows));
    if (dtype == KVR_BF16) KVR_LAUNCH(merge_kernel<__nv_bfloat16, 128>, grid, dim3(32 * kMergeWarps), 0, s, a);
    else if (head_dim == 64) KVR_LAUNCH(merge_kernel<float, 64>, grid, dim3(32 * kMergeWarps), 0, s, a);
    else KVR_LAUNCH(merge_kernel<float, 128>, grid, dim3(32 * kMergeWarps), 0, s, a);
    return cudaSuccess;
}

}  // namespace kvr
