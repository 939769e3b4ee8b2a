// linear.cuh -- what the projection kernels share: widening of codes, cluster
// instructions, rows out.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "rows.h"

namespace kvr {

// 16 codes to fp16, in order: b ^ 0x80 under the exponent of 1024 is 1152 + b, less 1152 is b, exact.
__device__ __forceinline__ void widen16(uint4 u, uint32_t* h) {
    const uint32_t w[4] = {u.x ^ 0x80808080u, u.y ^ 0x80808080u, u.z ^ 0x80808080u, u.w ^ 0x80808080u};
    const __half2 off = __half2half2(__ushort_as_half((unsigned short)0xe480));   // -1152
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t x = __byte_perm(w[i], 0x64646464u, e ? 0x4342 : 0x4140);
            const __half2 y = __hadd2(*reinterpret_cast<const __half2*>(&x), off);
            h[2 * i + e] = *reinterpret_cast<const uint32_t*>(&y);
        }
    }
}

__device__ __forceinline__ uint4 lds128(uint32_t address) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(address) : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t address, const uint32_t* v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(address), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// the shared-memory address of another block of the cluster
__device__ __forceinline__ uint32_t peer_address(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ int load_peer(uint32_t address) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(address) : "memory");
    return v;
}
__device__ __forceinline__ float4 load_peer4(uint32_t address) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(address)
                 : "memory");
    return v;
}

__device__ __forceinline__ void write_out(const Linear& a, int64_t at, float y) {
    if (a.dtype == KVR_F32) static_cast<float*>(a.out)[at] = y;
    else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(y);
}
// Features f .. f + 3 of one row; vec: out_vec4.
__device__ __forceinline__ void write4(const Linear& a, int vec, int row, int f, const float* y) {
    const int64_t at = (int64_t)row * a.out_stride + f;
    if (vec && f + 4 <= a.n_out) {
        if (a.dtype == KVR_F32) {
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(y[0], y[1], y[2], y[3]);
        } else {
            const __nv_bfloat162 p = __floats2bfloat162_rn(y[0], y[1]), q = __floats2bfloat162_rn(y[2], y[3]);
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q));
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (f + i < a.n_out) write_out(a, at + i, y[i]);
}
inline int out_vec4(const Linear& a) {
    return a.out_stride % 4 == 0 && reinterpret_cast<uintptr_t>(a.out) % (a.dtype == KVR_F32 ? 16 : 8) == 0;
}

// Of 32 accumulator columns in registers a lane holds its feature, a column is
// a row of the output.  Rows and features past the ends are not written; any
// alignment: a store is 32 features of one row.
template <typename T>
__device__ __forceinline__ void write_lanes(const Linear& a, int row, int f, const float* v, float sx, float sw, float bias,
                                            int left) {
    T* o = static_cast<T*>(a.out) + (int64_t)row * a.out_stride + f;
    const bool in = f < a.n_out;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float y = v[i] * __shfl_sync(0xffffffffu, sx, i) * sw + bias;
        if (in && i < left) {
            if constexpr (sizeof(T) == 4) *o = y;
            else *o = __float2bfloat16_rn(y);
        }
        o += a.out_stride;
    }
}
// bf16, even sizes: neighbouring lanes exchange, the even one takes both
// features of the first of two rows, the odd one of the second; a store is 64
// bytes of each.
__device__ __forceinline__ void write_pairs(const Linear& a, int row, int f, const float* v, float sx, float sw, float bias,
                                            int left) {
    const int odd = f & 1;
    const float sw2 = __shfl_xor_sync(0xffffffffu, sw, 1), bias2 = __shfl_xor_sync(0xffffffffu, bias, 1);
    const float s0 = odd ? sw2 : sw, s1 = odd ? sw : sw2, b0 = odd ? bias2 : bias, b1 = odd ? bias : bias2;
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + (int64_t)(row + odd) * a.out_stride + (f - odd);
    const int64_t step = 2 * a.out_stride;
    left = f < a.n_out ? left - odd : 0;
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        const float got = __shfl_xor_sync(0xffffffffu, odd ? v[i] : v[i + 1], 1);
        const float s = __shfl_sync(0xffffffffu, sx, i + odd);
        const __nv_bfloat162 y = __floats2bfloat162_rn((odd ? got : v[i]) * s * s0 + b0, (odd ? v[i + 1] : got) * s * s1 + b1);
        if (i < left) *reinterpret_cast<__nv_bfloat162*>(o) = y;
        o += step;
    }
}
enum : int { kOutF32, kOutBf16, kOutPairs };
inline int out_kind(const Linear& a) {
    const bool even = a.n_out % 2 == 0 && a.out_stride % 2 == 0 && reinterpret_cast<uintptr_t>(a.out) % 4 == 0;
    return a.dtype == KVR_F32 ? kOutF32 : even ? kOutPairs : kOutBf16;
}
__device__ __forceinline__ void write32(const Linear& a, int kind, int row, int f, const float* v, float sx, float sw,
                                        float bias, int left) {
    if (kind == kOutPairs) write_pairs(a, row, f, v, sx, sw, bias, left);
    else if (kind == kOutF32) write_lanes<float>(a, row, f, v, sx, sw, bias, left);
    else write_lanes<__nv_bfloat16>(a, row, f, v, sx, sw, bias, left);
}

}  // namespace kvr
