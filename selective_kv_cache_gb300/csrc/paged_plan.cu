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

// Keys that the rows of item i can see, its units, and the checks of its
// sequence's row range.
__device__ __forceinline__ PagedItem make_item(const PagedAttn& a, int i) {
    PagedItem it{};
    const int b = i / a.tiles, t = i - b * a.tiles;
    int row0;
    const int n = paged_seq_rows(a.p, a.r, b, &row0);
    if (t == 0) {
        if (n > a.max_rows) paged_err(a.p, DEV_ERR_INDEX, n);
        const int kv = a.p.kv_len[b];
        if (kv < 0 || kv > a.p.capacity) paged_err(a.p, DEV_ERR_INDEX, kv);
    }
    const int r0 = t * a.positions, r1 = min(min(n, a.max_rows), r0 + a.positions);
    if (r0 >= r1) return it;
    const int kv = paged_kv_len(a.p, b);
    int lo = 0x7fffffff, hi = 0;
    for (int r = row0 + r0; r < row0 + r1; ++r) {
        if (a.r.pos[r] < 0) paged_err(a.p, DEV_ERR_INDEX, a.r.pos[r]);
        int l, h;
        paged_interval(a, r, kv, &l, &h);
        if (l < h) {
            lo = min(lo, l);
            hi = max(hi, h);
        }
    }
    if (lo >= hi) lo = hi = 0;   // nothing visible: one unit without keys, which writes the zeros
    it.klo = lo;
    it.khi = hi;
    it.seq = b;
    it.kv = kv;
    it.row0 = row0 + r0;
    it.rows = r1 - r0;
    it.units = max(1, (hi + a.unit_keys - 1) / a.unit_keys - lo / a.unit_keys);
    return it;
}

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
        if (i < a.n_items) it = make_item(a, i);
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

constexpr int kMergeRows = 8;   // rows of a merge block, one per warp

// Block (c - 1, rows): the (item, head) that share c enters in its middle, if
// share c is the first to do so.  One warp per row, four dims per lane (dims
// past head_dim idle): the maxima and weights of up to 32 partials at a time
// in the lanes, then each partial's row scaled and added in share order.
template <typename T, int DH>
__global__ void __launch_bounds__(32 * kMergeRows) merge_kernel(PagedAttn a) {
    pdl_wait();
    const int c = blockIdx.x + 1;
    const PagedShare sh = a.shares[c];
    if (sh.item < 0 || sh.off == 0) return;
    const int start = sh.u0 - sh.off, prev = a.shares[c - 1].u0;
    if (prev > start) return;
    const PagedItem it = sh.first;
    const int end = start + it.units, row0 = it.row0, n = it.rows;
    const int row = blockIdx.y * kMergeRows + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (row >= n * a.G) return;
    const size_t stride = (size_t)2 * a.tile_rows;   // rows from one share's first slot to the next's
    const size_t first = (size_t)(c - 1) * stride + (prev == start ? 0 : a.tile_rows) + row;
    float M = -INFINITY;
    for (int k0 = 0;; k0 += 32) {
        const int k = k0 + lane;   // partial k belongs to share c - 1 + k
        const bool live = c - 1 + k < a.n_cta && (k == 0 || (a.shares[c - 1 + k].item >= 0 && a.shares[c - 1 + k].u0 < end));
        if (live) M = fmaxf(M, a.part_ml[2 * (k == 0 ? first : (size_t)(c - 1 + k) * stride + row)]);
        if (!__all_sync(0xffffffffu, live)) break;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0;; k0 += 32) {
        const int k = k0 + lane;
        const bool live = c - 1 + k < a.n_cta && (k == 0 || (a.shares[c - 1 + k].item >= 0 && a.shares[c - 1 + k].u0 < end));
        const size_t at = k == 0 ? first : (size_t)(c - 1 + k) * stride + row;
        float w = 0.f, l = 0.f;
        if (live) {
            const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + 2 * at);
            w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);   // a share that saw no key of the row takes no part
            l = w * ml.y;
        }
        const int parts = __popc(__ballot_sync(0xffffffffu, live));
#pragma unroll 4
        for (int i = 0; i < parts; ++i) {
            const float wi = __shfl_sync(0xffffffffu, w, i);
            L += __shfl_sync(0xffffffffu, l, i);
            if (wi != 0.f && lane < DH / 4) {
                const size_t ai = k0 + i == 0 ? first : (size_t)(c - 1 + k0 + i) * stride + row;
                const float4 o = *reinterpret_cast<const float4*>(a.part_o + ai * DH + 4 * lane);
                acc.x += wi * o.x;
                acc.y += wi * o.y;
                acc.z += wi * o.z;
                acc.w += wi * o.w;
            }
        }
        if (parts < 32) break;
    }
    const float inv = L > 0.f ? 1.0f / L : 0.f;
    if (lane < DH / 4)
        store4(reinterpret_cast<T*>(a.out) + (int64_t)(row0 + row / a.G) * a.out_stride +
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
    if (dtype == KVR_BF16) KVR_LAUNCH(merge_kernel<__nv_bfloat16, 128>, grid, dim3(32 * kMergeRows), 0, s, a);
    else if (head_dim == 64) KVR_LAUNCH(merge_kernel<float, 64>, grid, dim3(32 * kMergeRows), 0, s, a);
    else KVR_LAUNCH(merge_kernel<float, 128>, grid, dim3(32 * kMergeRows), 0, s, a);
    return cudaSuccess;
}

}  // namespace kvr
