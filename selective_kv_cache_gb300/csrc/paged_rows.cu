// paged_rows.cu -- rows into and out of the paged cache.
//
// Append: k'_r = R_{g_r} k_r (rotate-half pairs (i, i + dh/2)) and v_r go to
// slot g_r of their sequence, queries are rotated beside them ("Budgeted
// KV-Cache Repair for Evolving Contexts", Sec. 13.2, Eq. 21, for a cache in
// pages).  Read is the inverse of the write.  Both move each byte once and do
// a few flops on it: HBM-bound for prompts, launch-bound for decode steps.
//
// A CTA takes a few packed rows, about three (row, head) units per group of
// eight or sixteen threads: one warp finds the rows' sequences and slots (three
// dependent loads) while every thread already has its units' rows on their
// way.  Threads of a unit own whole rotation pairs, so nothing is exchanged
// between them but the extrema of a 4-bit group.
// Rotation: fp32, products and sum rounded separately, so
// that a plain elementwise evaluation gives the same bits.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "paged.h"

namespace kvr {
namespace {

constexpr int kRowThreads = 128, kMaxRows = 16, kBatch = 3;   // units a thread has in flight

__device__ __forceinline__ void unpack8(uint4 u, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// The pair (x, y) turned by (cos, sin).
__device__ __forceinline__ void turn(float& x, float& y, float2 cs) {
    const float a = __fsub_rn(__fmul_rn(x, cs.x), __fmul_rn(y, cs.y));
    y = __fadd_rn(__fmul_rn(y, cs.x), __fmul_rn(x, cs.y));
    x = a;
}

// A vector pair of one row: elements [v*E, v*E + E) and the same + dh/2.
template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
    static constexpr int E = 8;
    static __device__ __forceinline__ void rotate(uint4& lo, uint4& hi, const float2* cs) {
        float x[8], y[8];
        unpack8(lo, x);
        unpack8(hi, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) turn(x[e], y[e], cs[e]);
        lo = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
        hi = make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
    }
};
template <>
struct Pair<float> {
    static constexpr int E = 4;
    static __device__ __forceinline__ void rotate(uint4& lo, uint4& hi, const float2* cs) {
        float* x = reinterpret_cast<float*>(&lo);
        float* y = reinterpret_cast<float*>(&hi);
#pragma unroll
        for (int e = 0; e < 4; ++e) turn(x[e], y[e], cs[e]);
    }
};

// Slots of the CTA's rows in shared memory, by warp 0, lane i for row i: the page
// row of head 0 and the position, page row -1 for a row that is not to be
// touched.  A row's sequence is the number of ends cu[b + 1] <= r.  Offsets that do
// not begin at 0, fall or pass n_rows are reported, and no row is touched; kAppend
// checks what a write needs besides.  The caller synchronises.
struct RowSlot {
    int64_t at;
    int g;
};
template <bool kAppend>
__device__ __forceinline__ void find_slots(const PagedRowIo& a, RowSlot* slots) {
    if (threadIdx.x >= 32) return;
    const int lane = threadIdx.x, r0 = blockIdx.x * a.rows_per_block, r = r0 + lane;
    int b = 0, malformed = -1, last = a.r.cu[0];
    if (last != 0) malformed = 0;
    for (int b0 = 0; b0 < a.p.batch; b0 += 32) {
        const bool in = b0 + lane < a.p.batch;
        const int end = in ? a.r.cu[b0 + lane + 1] : 0x7fffffff;
        int begin = __shfl_up_sync(0xffffffffu, end, 1);
        if (lane == 0) begin = last;
        last = __shfl_sync(0xffffffffu, end, 31);
        if (in && (end < begin || end > a.r.n_rows)) malformed = b0 + lane;
        for (int i = 0; i < a.rows_per_block; ++i) {
            const int n = __popc(__ballot_sync(0xffffffffu, end <= r0 + i));
            if (lane == i) b += n;
        }
    }
    const bool usable = !__any_sync(0xffffffffu, malformed >= 0);
    if (malformed >= 0) paged_err(a.p.err, DEV_ERR_INDEX, malformed);
    if (lane >= a.rows_per_block) return;
    int64_t at = -1;
    int g = 0;
    if (usable && r < a.r.n_rows && b < a.p.batch) {   // else behind the last sequence: left alone
        g = a.r.pos[r];
        int bad = 0;
        if (g < 0 || g >= a.p.capacity || (kAppend && a.rope && g >= a.rope_len)) bad = DEV_ERR_INDEX;
        else if (kAppend && r > a.r.cu[b] && a.r.pos[r - 1] >= g) bad = DEV_ERR_ORDER;
        int id = 0;
        if (!bad) {
            id = a.p.table[(int64_t)b * a.p.max_pages + (g >> a.p.page_shift)];
            if ((unsigned)id >= (unsigned)a.p.n_pages) bad = DEV_ERR_INDEX;
        }
        if (bad) paged_err(a.p.err, bad, g);
        else at = paged_row(a.p, id, g & ((1 << a.p.page_shift) - 1), 0);
    }
    slots[lane] = RowSlot{at, g};
}

// Unit x of the CTA: row i of its rows, head u (K heads, V heads, query heads).
struct RowUnit {
    int i, u;
    int64_t r;
    bool live;
};
__device__ __forceinline__ RowUnit unit_of(const PagedRowIo& a, int x) {
    const int total = a.rows_per_block * a.units, y = min(x, total - 1), i = y / a.units;
    const int64_t r = (int64_t)blockIdx.x * a.rows_per_block + i;
    return RowUnit{i, y - i * a.units, r, x < total && r < a.r.n_rows};
}
__device__ __forceinline__ const uint8_t* unit_src(const PagedRowIo& a, const RowUnit& x, int bytes) {
    const int H = a.p.n_kv_heads;
    return x.u < H ? a.k_in + x.r * a.k_stride + (int64_t)x.u * bytes
         : x.u < 2 * H ? a.v_in + x.r * a.v_stride + (int64_t)(x.u - H) * bytes
                       : a.q_in + x.r * a.q_stride + (int64_t)(x.u - 2 * H) * bytes;
}

template <typename T, int DH>
__global__ void __launch_bounds__(kRowThreads) append_kernel(PagedRowIo a) {
    constexpr int E = Pair<T>::E, VT = DH / 2 / E;   // elements per vector, threads per unit
    constexpr int kBytes = DH * (int)sizeof(T), kStep = kRowThreads / VT;
    __shared__ RowSlot slots[kMaxRows];
    const int v = threadIdx.x % VT, H = a.p.n_kv_heads, total = a.rows_per_block * a.units;
    float2 cs[E];   // of the row in hand
    int in_hand = -1;
    for (int x0 = 0; x0 < total; x0 += kBatch * kStep) {
        uint4 lo[kBatch], hi[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const RowUnit x = unit_of(a, x0 + j * kStep + threadIdx.x / VT);
            if (!x.live) continue;
            const uint4* src = reinterpret_cast<const uint4*>(unit_src(a, x, kBytes));
            lo[j] = src[v];
            hi[j] = src[v + VT];
        }
        if (x0 == 0) {
            find_slots<true>(a, slots);
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const RowUnit x = unit_of(a, x0 + j * kStep + threadIdx.x / VT);
            const RowSlot slot = slots[x.i];
            if (!x.live || slot.at < 0) continue;
            if (a.rope && (x.u < H || x.u >= 2 * H)) {
                if (x.i != in_hand) {
                    in_hand = x.i;
#pragma unroll
                    for (int e = 0; e < E; e += 2) {
                        const float4 w =
                            *reinterpret_cast<const float4*>(a.rope + (int64_t)slot.g * (DH / 2) + v * E + e);
                        cs[e] = make_float2(w.x, w.y);
                        cs[e + 1] = make_float2(w.z, w.w);
                    }
                }
                Pair<T>::rotate(lo[j], hi[j], cs);
            }
            uint4* dst = reinterpret_cast<uint4*>(
                x.u < H ? a.p.k + (slot.at + x.u * a.p.head_stride) * kBytes
                : x.u < 2 * H ? a.p.v + (slot.at + (x.u - H) * a.p.head_stride) * kBytes
                              : a.q_out + (x.r * a.n_q_heads + x.u - 2 * H) * kBytes);
            dst[v] = lo[j];
            dst[v + VT] = hi[j];
        }
    }
}

// 4-bit pages: thread v of a row's eight owns the unit quadruple u = v, 8 + v,
// 16 + v, 24 + v (dims 32 i + 4 v .. + 3): whole rotation pairs, and the 8
// bytes at place 4 v of the packed row.  The extrema of 32 dims are those of
// the eight threads' i-th units; wider groups join their units.
__device__ __forceinline__ void extremum8(float& lo, float& hi) {
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
}

template <int NG>
__global__ void __launch_bounds__(kRowThreads) append_int4_kernel(PagedRowIo a) {
    constexpr int kJoin = 4 / NG, kStep = kRowThreads / 8;
    __shared__ RowSlot slots[kMaxRows];
    const int v = threadIdx.x % 8, H = a.p.n_kv_heads, total = a.rows_per_block * a.units;
    // every thread of a warp runs the same rounds: the shuffles below need
    // the whole warp
    for (int x0 = 0; x0 < total; x0 += kBatch * kStep) {
        uint2 raw[kBatch][4];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const RowUnit un = unit_of(a, x0 + j * kStep + threadIdx.x / 8);
            const uint8_t* src = unit_src(a, un, 256) + 8 * v;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                raw[j][i] = un.live ? *reinterpret_cast<const uint2*>(src + 64 * i) : make_uint2(0u, 0u);
        }
        if (x0 == 0) {
            find_slots<true>(a, slots);
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const RowUnit un = unit_of(a, x0 + j * kStep + threadIdx.x / 8);
            const RowSlot slot = slots[un.i];
            const int u = un.u;
            const int64_t r = un.r, row = slot.at;
            const bool live = un.live && row >= 0, is_q = u >= 2 * H, is_v = !is_q && u >= H;
            float x[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint2 w = raw[j][i];
                x[4 * i] = __uint_as_float(w.x << 16);
                x[4 * i + 1] = __uint_as_float(w.x & 0xffff0000u);
                x[4 * i + 2] = __uint_as_float(w.y << 16);
                x[4 * i + 3] = __uint_as_float(w.y & 0xffff0000u);
            }
            if (a.rope && live && !is_v) {
                const float4* cs = reinterpret_cast<const float4*>(a.rope + (int64_t)slot.g * 64 + 4 * v);
#pragma unroll
                for (int i = 0; i < 2; ++i) {   // dims 4v.. and 32 + 4v.. with their pairs 64 further
                    const float4 c0 = cs[16 * i], c1 = cs[16 * i + 1];
                    turn(x[4 * i], x[4 * i + 8], make_float2(c0.x, c0.y));
                    turn(x[4 * i + 1], x[4 * i + 9], make_float2(c0.z, c0.w));
                    turn(x[4 * i + 2], x[4 * i + 10], make_float2(c1.x, c1.y));
                    turn(x[4 * i + 3], x[4 * i + 11], make_float2(c1.z, c1.w));
                }
            }
            if (live && is_q) {
                uint8_t* dst = a.q_out + (r * a.n_q_heads + u - 2 * H) * 256;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<uint2*>(dst + 64 * i + 8 * v) =
                        make_uint2(pack2(x[4 * i], x[4 * i + 1]), pack2(x[4 * i + 2], x[4 * i + 3]));
            }
            if (__all_sync(0xffffffffu, !live || is_q)) continue;   // nothing to quantise in this warp
            float lo[NG], hi[NG];
#pragma unroll
            for (int e = 0; e < 16; ++e)   // 15 s + o stays in fp16's range
                x[e] = fminf(fmaxf(x[e], -32768.f), 32768.f);
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                lo[n] = hi[n] = x[4 * kJoin * n];
#pragma unroll
                for (int e = 1; e < 4 * kJoin; ++e) {
                    lo[n] = fminf(lo[n], x[4 * kJoin * n + e]);
                    hi[n] = fmaxf(hi[n], x[4 * kJoin * n + e]);
                }
                extremum8(lo[n], hi[n]);
            }
            if (!live || is_q) continue;
            const int64_t at = row + (u - (is_v ? H : 0)) * a.p.head_stride;
            __half2* meta = reinterpret_cast<__half2*>((is_v ? a.p.vs : a.p.ks) + at * (4 * NG));
            uint32_t unit[4];
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                // scale and offset are rounded to fp16 first and the codes chosen
                // against the rounded ones, so their rounding costs range, not
                // bias: a value is off by half a step plus at most the offset's
                // rounding (2^-11 of it)
                const __half sh = __float2half_rn(__fmul_rn(__fsub_rn(hi[n], lo[n]), 1.0f / 15.0f));
                const __half oh = __float2half_rn(lo[n]);
                const float s = __half2float(sh), o = __half2float(oh);
                const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
                if (v == n) meta[n] = __halves2half2(sh, oh);   // NG <= 4 of the eight threads
#pragma unroll
                for (int i = n * kJoin; i < (n + 1) * kJoin; ++i) {
                    // 2^23 + 2^22 leaves the rounded code in the low bits; bits 16 and up of the
                    // sum are not used
                    uint32_t c[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        c[e] = __float_as_uint(
                            __fadd_rn(fminf(fmaxf(__fmul_rn(__fsub_rn(x[4 * i + e], o), inv), 0.f), 15.f), 12582912.f));
                    unit[i] = c[0] + (c[1] << 4) + (c[2] << 8) + (c[3] << 12);
                }
            }
            *reinterpret_cast<uint2*>((is_v ? a.p.v : a.p.k) + at * 64 + 8 * v) =
                make_uint2(__byte_perm(unit[0], unit[1], 0x5410), __byte_perm(unit[2], unit[3], 0x5410));
        }
    }
}

// NG = 0: rows copied as they are (VT 16-byte vectors); else 4-bit rows.  K heads first, then V heads;
// when only one of the two is wanted, its heads alone.
template <int VT, int NG>
__global__ void __launch_bounds__(kRowThreads) read_kernel(PagedRowIo a) {
    constexpr int kPerUnit = NG ? 8 : VT, kStep = kRowThreads / kPerUnit, MB = NG ? 4 * NG : 4;
    __shared__ RowSlot slots[kMaxRows];
    const int v = threadIdx.x % kPerUnit, H = a.p.n_kv_heads, total = a.rows_per_block * a.units;
    find_slots<false>(a, slots);
    __syncthreads();
    for (int x0 = 0; x0 < total; x0 += kBatch * kStep) {
        uint4 w[kBatch];
        uint32_t meta[kBatch][NG ? NG : 1];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const RowUnit x = unit_of(a, x0 + j * kStep + threadIdx.x / kPerUnit);
            const int64_t row = slots[x.i].at;
            if (!x.live || row < 0) continue;
            const bool is_v = x.u >= H || !a.k_out;
            const int64_t at = row + (x.u >= H ? x.u - H : x.u) * a.p.head_stride;
            if constexpr (NG == 0) {
                w[j] = reinterpret_cast<const uint4*>((is_v ? a.p.v : a.p.k) + at * VT * 16)[v];
            } else {
                const uint2 c = *reinterpret_cast<const uint2*>((is_v ? a.p.v : a.p.k) + at * 64 + 8 * v);
                w[j].x = c.x;
                w[j].y = c.y;
                const uint8_t* m = (is_v ? a.p.vs : a.p.ks) + at * MB;
                if constexpr (NG == 4) {
                    const uint4 z = *reinterpret_cast<const uint4*>(m);
                    meta[j][0] = z.x, meta[j][1] = z.y, meta[j][2] = z.z, meta[j][3] = z.w;
                } else if constexpr (NG == 2) {
                    const uint2 z = *reinterpret_cast<const uint2*>(m);
                    meta[j][0] = z.x, meta[j][1] = z.y;
                } else {
                    meta[j][0] = *reinterpret_cast<const uint32_t*>(m);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const RowUnit x = unit_of(a, x0 + j * kStep + threadIdx.x / kPerUnit);
            if (!x.live || slots[x.i].at < 0) continue;
            const bool is_v = x.u >= H || !a.k_out;
            const int h = x.u >= H ? x.u - H : x.u;
            uint8_t* dst = is_v ? a.v_out + x.r * a.v_stride : a.k_out + x.r * a.k_stride;
            if constexpr (NG == 0) {
                reinterpret_cast<uint4*>(dst + (int64_t)h * VT * 16)[v] = w[j];
            } else {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const float2 so = __half22float2(*reinterpret_cast<const __half2*>(&meta[j][g * NG / 4]));
                    const uint32_t unit = (g < 2 ? w[j].x : w[j].y) >> (16 * (g & 1));
                    float y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = fmaf((float)((unit >> (4 * e)) & 15u), so.x, so.y);
                    *reinterpret_cast<uint2*>(dst + (int64_t)h * 256 + 64 * g + 8 * v) =
                        make_uint2(pack2(y[0], y[1]), pack2(y[2], y[3]));
                }
            }
        }
    }
}

// Rows of a CTA: about kBatch units for each group of threads, while there are
// CTAs for every SM.
int rows_per_block(int n_rows, int units, int threads_per_unit) {
    const int want = kBatch * (kRowThreads / threads_per_unit) / units;
    return std::max(1, std::min(std::min(want, kMaxRows), n_rows / (2 * kNumSMs)));
}

}  // namespace

cudaError_t launch_paged_append(int format, int head_dim, int group, const PagedRowIo& a_in, cudaStream_t s) {
    PagedRowIo a = a_in;
    const int per_unit = format == KVR_F32 && head_dim == 128 ? 16 : 8;
    a.units = 2 * a.p.n_kv_heads + (a.q_in ? a.n_q_heads : 0);
    a.rows_per_block = rows_per_block(a.r.n_rows, a.units, per_unit);
    const dim3 grid((unsigned)((a.r.n_rows + a.rows_per_block - 1) / a.rows_per_block)), block(kRowThreads);
    if (format == KVR_BF16) KVR_LAUNCH(append_kernel<__nv_bfloat16, 128>, grid, block, 0, s, a);
    else if (format == KVR_F32 && head_dim == 64) KVR_LAUNCH(append_kernel<float, 64>, grid, block, 0, s, a);
    else if (format == KVR_F32) KVR_LAUNCH(append_kernel<float, 128>, grid, block, 0, s, a);
    else if (group == 32) KVR_LAUNCH(append_int4_kernel<4>, grid, block, 0, s, a);
    else if (group == 64) KVR_LAUNCH(append_int4_kernel<2>, grid, block, 0, s, a);
    else KVR_LAUNCH(append_int4_kernel<1>, grid, block, 0, s, a);
    return cudaSuccess;
}

cudaError_t launch_paged_read(int format, int head_dim, int group, const PagedRowIo& a_in, cudaStream_t s) {
    PagedRowIo a = a_in;
    const int per_unit = format == KVR_INT4 ? 8 : (format == KVR_F32 && head_dim == 128 ? 32 : 16);
    a.units = (a.k_out && a.v_out ? 2 : 1) * a.p.n_kv_heads;
    a.rows_per_block = rows_per_block(a.r.n_rows, a.units, per_unit);
    const dim3 grid((unsigned)((a.r.n_rows + a.rows_per_block - 1) / a.rows_per_block)), block(kRowThreads);
    if (format == KVR_INT4) {
        if (group == 32) KVR_LAUNCH(read_kernel<16, 4>, grid, block, 0, s, a);
        else if (group == 64) KVR_LAUNCH(read_kernel<16, 2>, grid, block, 0, s, a);
        else KVR_LAUNCH(read_kernel<16, 1>, grid, block, 0, s, a);
    } else if (format == KVR_F32 && head_dim == 128) {
        KVR_LAUNCH(read_kernel<32, 0>, grid, block, 0, s, a);
    } else {   // bf16 of 128 dims, fp32 of 64: 256-byte rows
        KVR_LAUNCH(read_kernel<16, 0>, grid, block, 0, s, a);
    }
    return cudaSuccess;
}

}  // namespace kvr
