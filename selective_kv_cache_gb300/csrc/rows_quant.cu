// rows_quant.cu -- packed rows into eight bits: RMSNorm with the residual's
// addition, the gated activation, plain rows; and back.
//
// For the fp32 values y of a row: top = max |y|, s = top / 127, code =
// rint(y / s).  A norm's y is h w r with r = 1 / sqrt(mean h^2 + eps), and r
// > 0 is one number a row: top = r max |h w| and the codes are those of h w,
// so the sum of squares and the maximum are found in one pass and one
// exchange, and nothing waits for r but the scale.
//
// HBM-bound: every byte moves once.  A group of threads holds a row in
// registers (up to 32 values a thread, unrounded) between its loads and its
// stores; rows wider than 1024 threads hold are read twice.  Maxima are taken
// on the bits of |y| as unsigned numbers, where NaN lies above infinity: a row
// that is not finite shows in its maximum.
#include <cuda_bf16.h>

#include <algorithm>

#include "rows.h"

namespace kvr {
namespace {

constexpr float kTiny = 1.17549435e-38f;   // 2^-126

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }

// V consecutive elements at p as fp32: vectors of 16 bytes where V = 8
template <typename T, int V>
__device__ __forceinline__ void load(const T* p, float* x) {
    if constexpr (V == 1) {
        x[0] = to_f<T>(*p);
    } else if constexpr (sizeof(T) == 4) {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const float* x) {
    if constexpr (V == 1) {
        *p = from_f<T>(x[0]);
    } else if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// rint(y * inv) in the low byte: adding 1.5 * 2^23 leaves the integer, rounded
// to nearest even, in the low bits of the sum.
__device__ __forceinline__ uint32_t code_bits(float y, float inv) {
    return __float_as_uint(fmaf(y, inv, 12582912.f));
}
template <int V>
__device__ __forceinline__ void store_codes(int8_t* p, const float* y, float inv, bool bad) {
    if constexpr (V == 1) {
        *p = bad ? (int8_t)0 : (int8_t)(code_bits(y[0], inv) & 0xffu);
    } else {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t lo = __byte_perm(code_bits(y[4 * i], inv), code_bits(y[4 * i + 1], inv), 0x0040);
            const uint32_t hi = __byte_perm(code_bits(y[4 * i + 2], inv), code_bits(y[4 * i + 3], inv), 0x0040);
            w[i] = bad ? 0u : __byte_perm(lo, hi, 0x5410);
        }
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    }
}

// g / (1 + exp(-g)) * u.  bf16 rows take the approximate exponential and
// division (2^-20 of the value), fp32 rows the accurate ones.
template <typename T>
__device__ __forceinline__ float gated(float g, float u) {
    if constexpr (sizeof(T) == 4) return g / (1.f + expf(-g)) * u;
    return __fdividef(g, 1.f + __expf(-g)) * u;
}

// The V values at element i of a row, as the row's operator has them before
// the quantiser: h (norm, the sum of x and residual), the gated value, or x.
template <RowOp kOp, typename T, int V>
__device__ __forceinline__ void row_values(const RowsQuant& a, const T* x, const T* res, int i, float* v) {
    load<T, V>(x + i, v);
    if constexpr (kOp == RowOp::Norm) {
        if (res) {
            float r[V];
            load<T, V>(res + i, r);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] += r[e];
        }
    }
    if constexpr (kOp == RowOp::Swiglu) {
        float u[V];
        load<T, V>(x + a.d + i, u);
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = gated<T>(v[e], u[e]);
    }
}

// Sum and maximum over the threads of a row's group: a warp by itself, or the
// whole block.
template <bool kWarp, bool kSum>
__device__ __forceinline__ void row_reduce(float& sum, uint32_t& top) {
    top = __reduce_max_sync(0xffffffffu, top);
    if constexpr (kSum) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if constexpr (!kWarp) {
        __shared__ float sums[32];
        __shared__ uint32_t tops[32];
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = blockDim.x >> 5;
        if (lane == 0) {
            sums[warp] = sum;
            tops[warp] = top;
        }
        __syncthreads();
        top = __reduce_max_sync(0xffffffffu, lane < n ? tops[lane] : 0u);
        if constexpr (kSum) {
            sum = lane < n ? sums[lane] : 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
    }
}

// kV: 8 (vectors) or 1; kSlots: groups of kV values a thread holds, 0: the row
// is read twice.  kWarp: a warp a row, several rows a block; else a block a row.
constexpr int block_most(int values, bool warp) {
    return warp ? 128 : values == 8 ? 256 : values == 16 ? 512 : 1024;
}
template <RowOp kOp, typename T, int kV, int kSlots, bool kWarp>
__global__ void __launch_bounds__(block_most(kV * kSlots, kWarp)) rows_quant_kernel(const __grid_constant__ RowsQuant a) {
    constexpr bool kNorm = kOp == RowOp::Norm;
    // 32 values a thread leave no registers for their weights, which are read again (from L1)
    constexpr bool kKeepW = kNorm && kSlots > 0 && kSlots * kV <= 16;
    const int lane = kWarp ? threadIdx.x & 31 : threadIdx.x, step = (kWarp ? 32 : blockDim.x) * kV;
    const int64_t row = kWarp ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= a.n_rows) return;
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.x_stride;
    const T* res = kNorm && a.res ? reinterpret_cast<const T*>(a.res) + row * a.res_stride : nullptr;
    const T* weight = reinterpret_cast<const T*>(a.weight);
    constexpr int kHold = kSlots > 0 ? kSlots : 1;
    float v[kHold][kV], w[kKeepW ? kHold : 1][kV];
    float sum = 0.f;
    uint32_t top = 0u;
    auto take = [&](const float* h, const float* wt) {
#pragma unroll
        for (int e = 0; e < kV; ++e) {
            if constexpr (kNorm) sum = fmaf(h[e], h[e], sum);
            top = max(top, __float_as_uint(kNorm ? h[e] * wt[e] : h[e]) & 0x7fffffffu);
        }
    };
    if constexpr (kSlots > 0) {
#pragma unroll
        for (int k = 0; k < kSlots; ++k) {
            const int i = lane * kV + k * step;
            if (i < a.d) {
                row_values<kOp, T, kV>(a, x, res, i, v[k]);
                if constexpr (kKeepW) load<T, kV>(weight + i, w[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < kSlots; ++k) {
            const int i = lane * kV + k * step;
            if (i < a.d) {
                if constexpr (kNorm && !kKeepW) load<T, kV>(weight + i, w[0]);
                take(v[k], w[kKeepW ? k : 0]);
            }
        }
    } else {
        for (int i = lane * kV; i < a.d; i += step) {
            row_values<kOp, T, kV>(a, x, res, i, v[0]);
            if constexpr (kNorm) load<T, kV>(weight + i, w[0]);
            take(v[0], w[0]);
        }
    }
    row_reduce<kWarp, kNorm>(sum, top);
    const float r = kNorm ? rsqrtf(sum / (float)a.d + a.eps) : 1.f;
    const bool bad = top >= 0x7f800000u || (kNorm && !(r <= 3.4028234e38f));
    // of the values before r: r lies in the scale alone
    const float s0 = __uint_as_float(top) * (1.f / 127.f);
    const float scale = kNorm ? s0 * r : s0;
    const bool none = !bad && (s0 < kTiny || scale < kTiny);
    const float inv = bad || none ? 0.f : 1.f / s0;
    if (a.codes && lane == 0) a.scales[row] = bad ? __int_as_float(0x7fffffff) : none ? 0.f : scale;
    auto put = [&](int i, const float* h, const float* wt) {
        float y[kV];
#pragma unroll
        for (int e = 0; e < kV; ++e) y[e] = kNorm ? h[e] * wt[e] : h[e];
        if (a.codes) store_codes<kV>(a.codes + row * a.code_stride + i, y, inv, bad);
        if constexpr (kNorm) {
            if (a.sum) store<T, kV>(reinterpret_cast<T*>(a.sum) + row * a.sum_stride + i, h);
        }
        if (a.out) {
            if constexpr (kNorm) {
#pragma unroll
                for (int e = 0; e < kV; ++e) y[e] = h[e] * r * wt[e];
            }
            store<T, kV>(reinterpret_cast<T*>(a.out) + row * a.out_stride + i, y);
        }
    };
    if constexpr (kSlots > 0) {
#pragma unroll
        for (int k = 0; k < kSlots; ++k) {
            const int i = lane * kV + k * step;
            if (i < a.d) {
                if constexpr (kNorm && !kKeepW) load<T, kV>(weight + i, w[0]);
                put(i, v[k], w[kKeepW ? k : 0]);
            }
        }
    } else {
        // a thread writes only the elements that it has just read, so outputs may be inputs
        for (int i = lane * kV; i < a.d; i += step) {
            row_values<kOp, T, kV>(a, x, res, i, v[0]);
            if constexpr (kNorm) load<T, kV>(weight + i, w[0]);
            put(i, v[0], w[0]);
        }
    }
}

// codes to values; kV = 16 codes a thread in vectors, or one
template <typename T, int kV>
__global__ void __launch_bounds__(256) rows_dequantise_kernel(const int8_t* codes, int64_t code_stride,
                                                              const float* scales, T* out, int64_t out_stride, int n_rows,
                                                              int d) {
    const int per = (d + kV - 1) / kV;
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < (int64_t)n_rows * per; t += (int64_t)gridDim.x * 256) {
        const int64_t row = t / per;
        const int i = (int)(t - row * per) * kV;
        const int8_t* c = codes + row * code_stride + i;
        T* o = out + row * out_stride + i;
        const float s = scales[row];
        if constexpr (kV == 1) {
            *o = from_f<T>(s * (float)*c);
        } else {
            const uint4 u = *reinterpret_cast<const uint4*>(c);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
            float y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = s * (float)(int8_t)(w[e / 4] >> (8 * (e % 4)));
            store<T, 8>(o, y);
            store<T, 8>(o + 8, y + 8);
        }
    }
}

template <RowOp kOp, typename T, int kV>
cudaError_t launch_as(const RowsQuant& a, cudaStream_t s) {
    constexpr int kPer = kV == 8 ? 1 : 8;   // slots of a step of eight values a thread
    const int n = (a.d + kV - 1) / kV;      // groups of a row
    if (n <= 32 * kPer) {
        const int per_block = 4;
        KVR_LAUNCH((rows_quant_kernel<kOp, T, kV, kPer, true>), dim3((a.n_rows + per_block - 1) / per_block),
                   dim3(32 * per_block), 0, s, a);
        return cudaSuccess;
    }
    auto block = [&](int slots) { return dim3(std::min(1024, ((n + slots - 1) / slots + 31) / 32 * 32)); };
    if (n <= 256 * kPer)
        KVR_LAUNCH((rows_quant_kernel<kOp, T, kV, kPer, false>), dim3(a.n_rows), block(kPer), 0, s, a);
    else if (n <= 1024 * kPer)
        KVR_LAUNCH((rows_quant_kernel<kOp, T, kV, 2 * kPer, false>), dim3(a.n_rows), block(2 * kPer), 0, s, a);
    else if (n <= 4096 * kPer)
        KVR_LAUNCH((rows_quant_kernel<kOp, T, kV, 4 * kPer, false>), dim3(a.n_rows), block(4 * kPer), 0, s, a);
    else
        KVR_LAUNCH((rows_quant_kernel<kOp, T, kV, 0, false>), dim3(a.n_rows), dim3(1024), 0, s, a);
    return cudaSuccess;
}

bool in_vectors(const void* p, int64_t stride, int size, int bytes) {
    return p == nullptr || ((reinterpret_cast<uintptr_t>(p) % bytes) == 0 && (stride * size) % bytes == 0);
}

template <RowOp kOp, typename T>
cudaError_t launch_op(const RowsQuant& a, cudaStream_t s) {
    const int es = sizeof(T);
    const bool vec = a.d % 8 == 0 && in_vectors(a.x, a.x_stride, es, 16) && in_vectors(a.res, a.res_stride, es, 16) &&
                     in_vectors(a.sum, a.sum_stride, es, 16) && in_vectors(a.out, a.out_stride, es, 16) &&
                     in_vectors(a.weight, 0, es, 16) && in_vectors(a.codes, a.code_stride, 1, 8);
    return vec ? launch_as<kOp, T, 8>(a, s) : launch_as<kOp, T, 1>(a, s);
}

}  // namespace

cudaError_t launch_rows_quant(RowOp op, int dtype, const RowsQuant& a, cudaStream_t s) {
    const bool f32 = dtype == KVR_F32;
    switch (op) {
        case RowOp::Norm:
            return f32 ? launch_op<RowOp::Norm, float>(a, s) : launch_op<RowOp::Norm, __nv_bfloat16>(a, s);
        case RowOp::Swiglu:
            return f32 ? launch_op<RowOp::Swiglu, float>(a, s) : launch_op<RowOp::Swiglu, __nv_bfloat16>(a, s);
        default:
            return f32 ? launch_op<RowOp::Quantise, float>(a, s) : launch_op<RowOp::Quantise, __nv_bfloat16>(a, s);
    }
}

cudaError_t launch_rows_dequantise(int dtype, int n_rows, int d, const int8_t* codes, int64_t code_stride,
                                   const float* scales, void* out, int64_t out_stride, cudaStream_t s) {
    const int es = dtype == KVR_F32 ? 4 : 2;
    const bool vec = d % 16 == 0 && in_vectors(codes, code_stride, 1, 16) && in_vectors(out, out_stride, es, 16);
    const int64_t units = (int64_t)n_rows * (vec ? d / 16 : d);
    const dim3 grid((unsigned)std::min<int64_t>((units + 255) / 256, 1 << 20));
    auto go = [&](auto* o) -> cudaError_t {
        using T = std::remove_pointer_t<decltype(o)>;
        if (vec)
            KVR_LAUNCH((rows_dequantise_kernel<T, 16>), grid, dim3(256), 0, s, codes, code_stride, scales, o, out_stride,
                       n_rows, d);
        else
            KVR_LAUNCH((rows_dequantise_kernel<T, 1>), grid, dim3(256), 0, s, codes, code_stride, scales, o, out_stride,
                       n_rows, d);
        return cudaSuccess;
    };
    return dtype == KVR_F32 ? go(static_cast<float*>(out)) : go(static_cast<__nv_bfloat16*>(out));
}

}  // namespace kvr
