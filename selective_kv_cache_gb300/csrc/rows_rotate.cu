// rows_rotate.cu -- the rotary map on query and key heads of packed rows, and
// its table.
//
// Pair i of a head at position g turns by g f_i.  f_i is kept as a fraction of
// a turn times 2^64, so g f_i modulo one turn is an integer product that wraps:
// exact for every 32-bit position, negative ones too, where a product in fp32
// has lost the angle at a position of 2^24 and one in fp64 costs this GPU's
// scarce fp64 units.  The upper 32 bits, less the nearest quarter turn, go to
// sincospi: at most 2^-25 of an eighth turn is rounded away.
//
// HBM-bound: heads in and out once.  A block takes a few rows: each thread has
// its units (two vectors that hold whole pairs) on their way while the block
// fills the rows' (cos, sin) in shared memory, once a row instead of once a
// head.  Rotation in fp32, products and sums rounded separately, so that a
// plain elementwise evaluation gives the same bits.
#include <cuda_bf16.h>

#include <algorithm>

#include "rows.h"

namespace kvr {
namespace {

constexpr int kThreads = 256, kBatch = 4, kMaxRows = 16;   // units a thread has in flight; rows a block

__device__ __forceinline__ float2 cos_sin(uint64_t turns, int g, float m, bool inverse) {
    const uint32_t t = (uint32_t)((turns * (uint64_t)(int64_t)g) >> 32);
    const uint32_t quarter = (t + 0x20000000u) >> 30;
    const float x = (float)(int32_t)(t - (quarter << 30)) * 0x1p-31f;   // half turns, in [-1/4, 1/4]
    float s, c;
    sincospif(x, &s, &c);
    float cq = (quarter & 1u) ? -s : c, sq = (quarter & 1u) ? c : s;
    if (quarter & 2u) {
        cq = -cq;
        sq = -sq;
    }
    return make_float2(cq * m, inverse ? -(sq * m) : sq * m);
}

__device__ __forceinline__ void turn(float& x, float& y, float2 cs) {
    const float a = __fsub_rn(__fmul_rn(x, cs.x), __fmul_rn(y, cs.y));
    y = __fadd_rn(__fmul_rn(y, cs.x), __fmul_rn(x, cs.y));
    x = a;
}

template <typename T>
struct Vec;   // 16 bytes of T as fp32
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void get(uint4 u, float* x) {
        x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y); x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 put(const float* x) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(uint4 u, float* x) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 put(const float* x) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Quotients by a divisor of a launch, for numerators below 2^31: umulhi with
// ceil(2^(31 + l) / d), l = ceil(log2 d), and a shift by l - 1.
struct Div {
    uint32_t d, mul, shift;
    explicit Div(uint32_t n) : d(n), mul(0), shift(0) {
        if (n == 1) return;
        uint32_t l = 0;
        while ((1u << l) < n) ++l;
        mul = (uint32_t)(((uint64_t(1) << (31 + l)) + n - 1) / n);
        shift = l - 1;
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t x) const { return d == 1 ? x : __umulhi(x, mul) >> shift; }
};

struct RotateDev {
    RowsRotate a;
    float m;
    int rows_per_block, units, turned, heads;   // units of a head, those of them that turn; heads of a row
    Div by_units, by_heads;
};

// A head's units: `turned` of them hold two vectors of whole pairs, the others
// two vectors that are copied (or left alone in place).
template <typename T, int kLayout>
__device__ __forceinline__ void unit_offsets(const RotateDev& d, int u, int* first, int* second) {
    constexpr int N = Vec<T>::N;
    if (u < d.turned && kLayout == KVR_ROPE_HALF) {
        *first = u * N;
        *second = u * N + d.a.rope.rotary_dim / 2;
    } else {
        *first = 2 * u * N;
        *second = *first + N;
    }
}

template <typename T, int kLayout>
__global__ void __launch_bounds__(kThreads) rows_rotate_kernel(const __grid_constant__ RotateDev d) {
    constexpr int N = Vec<T>::N;
    extern __shared__ float2 cs[];   // [rows_per_block][rotary_dim / 2]
    const RowsRotate& a = d.a;
    const int dh = a.rope.head_dim, half = a.rope.rotary_dim / 2;
    const int64_t row0 = (int64_t)blockIdx.x * d.rows_per_block;
    const int rows = (int)min((int64_t)d.rows_per_block, a.n_rows - row0);
    const int total = rows * d.heads * d.units;
    bool ready = false;
    for (int base = 0; base < total; base += kThreads * kBatch) {
        uint4 x[kBatch][2];
        T* to[kBatch];
        int row[kBatch], unit[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int i = base + k * kThreads + threadIdx.x;
            to[k] = nullptr;
            if (i >= total) continue;
            const int j = (int)d.by_units(i);
            unit[k] = i - j * d.units;
            row[k] = (int)d.by_heads(j);
            int h = j - row[k] * d.heads;
            const int which = h >= a.heads[0];
            if (which) h -= a.heads[0];
            const T* in = reinterpret_cast<const T*>(a.in[which]) + (row0 + row[k]) * a.in_stride[which] + h * dh;
            T* out = reinterpret_cast<T*>(a.out[which]) + (row0 + row[k]) * a.out_stride[which] + h * dh;
            if (unit[k] >= d.turned && in == out) continue;   // copied dims in place
            int f, s;
            unit_offsets<T, kLayout>(d, unit[k], &f, &s);
            x[k][0] = *reinterpret_cast<const uint4*>(in + f);
            x[k][1] = *reinterpret_cast<const uint4*>(in + s);
            to[k] = out;
        }
        if (!ready) {
            for (int i = threadIdx.x; i < rows * half; i += kThreads) {
                const int r = i / half;
                cs[i] = cos_sin(a.rope.turns[i - r * half], a.pos[row0 + r], d.m, a.inverse);
            }
            __syncthreads();
            ready = true;
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (!to[k]) continue;
            int f, s;
            unit_offsets<T, kLayout>(d, unit[k], &f, &s);
            if (unit[k] < d.turned) {
                float p[N], q[N];
                Vec<T>::get(x[k][0], p);
                Vec<T>::get(x[k][1], q);
                const float2* c = cs + row[k] * half;
                if constexpr (kLayout == KVR_ROPE_HALF) {
#pragma unroll
                    for (int e = 0; e < N; ++e) turn(p[e], q[e], c[unit[k] * N + e]);
                } else {
#pragma unroll
                    for (int e = 0; e < N / 2; ++e) {
                        turn(p[2 * e], p[2 * e + 1], c[unit[k] * N + e]);
                        turn(q[2 * e], q[2 * e + 1], c[unit[k] * N + N / 2 + e]);
                    }
                }
                x[k][0] = Vec<T>::put(p);
                x[k][1] = Vec<T>::put(q);
            }
            *reinterpret_cast<uint4*>(to[k] + f) = x[k][0];
            *reinterpret_cast<uint4*>(to[k] + s) = x[k][1];
        }
    }
}

// Any alignment and size: a unit is one pair, or two of the dims that stay.
template <typename T>
__global__ void __launch_bounds__(kThreads) rows_rotate_pairs_kernel(const __grid_constant__ RotateDev d, int layout) {
    extern __shared__ float2 cs[];
    const RowsRotate& a = d.a;
    const int dh = a.rope.head_dim, half = a.rope.rotary_dim / 2;
    const int64_t row0 = (int64_t)blockIdx.x * d.rows_per_block;
    const int rows = (int)min((int64_t)d.rows_per_block, a.n_rows - row0);
    for (int i = threadIdx.x; i < rows * half; i += kThreads) {
        const int r = i / half;
        cs[i] = cos_sin(a.rope.turns[i - r * half], a.pos[row0 + r], d.m, a.inverse);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * d.heads * d.units; i += kThreads) {
        const int j = (int)d.by_units(i), u = i - j * d.units, row = (int)d.by_heads(j);
        int h = j - row * d.heads;
        const int which = h >= a.heads[0];
        if (which) h -= a.heads[0];
        const T* in = reinterpret_cast<const T*>(a.in[which]) + (row0 + row) * a.in_stride[which] + h * dh;
        T* out = reinterpret_cast<T*>(a.out[which]) + (row0 + row) * a.out_stride[which] + h * dh;
        const bool turns = u < half;
        if (!turns && in == out) continue;
        const int f = turns && layout == KVR_ROPE_HALF ? u : 2 * u, s = turns && layout == KVR_ROPE_HALF ? u + half : f + 1;
        T x = in[f], y = in[s];
        if (turns) {
            float p = (float)x, q = (float)y;
            turn(p, q, cs[row * half + u]);
            x = (T)p;
            y = (T)q;
        }
        out[f] = x;
        out[s] = y;
    }
}

__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ kvr_rope rope, int64_t n, float2* table) {
    const int half = rope.rotary_dim / 2;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int g = (int)(i / half);
        table[i] = cos_sin(rope.turns[i - (int64_t)g * half], g, rope.attn, false);
    }
}

template <typename T>
cudaError_t launch_as(const RowsRotate& a, cudaStream_t s) {
    constexpr int N = Vec<T>::N, es = sizeof(T);
    const int dh = a.rope.head_dim, rot = a.rope.rotary_dim;
    bool vec = rot % (2 * N) == 0 && dh % (2 * N) == 0;
    for (int w = 0; w < 2; ++w)
        if (a.heads[w])
            vec = vec && reinterpret_cast<uintptr_t>(a.in[w]) % 16 == 0 && reinterpret_cast<uintptr_t>(a.out[w]) % 16 == 0 &&
                  a.in_stride[w] * es % 16 == 0 && a.out_stride[w] * es % 16 == 0;
    const int units = vec ? dh / (2 * N) : dh / 2, heads = a.heads[0] + a.heads[1];
    // rows that fill a block's batch, fewer where there are not enough rows for the GPU
    int rows = std::max(1, std::min(kMaxRows, kThreads * kBatch / (units * heads)));
    rows = std::min(rows, std::max(1, a.n_rows / (2 * kNumSMs)));
    const RotateDev d{a, a.inverse ? 1.f / a.rope.attn : a.rope.attn, rows, units, vec ? rot / (2 * N) : rot / 2, heads,
                      Div(units), Div(heads)};
    const dim3 grid((unsigned)((a.n_rows + (int64_t)rows - 1) / rows));
    const size_t smem = sizeof(float2) * rows * (rot / 2);
    if (!vec)
        KVR_LAUNCH((rows_rotate_pairs_kernel<T>), grid, dim3(kThreads), smem, s, d, a.rope.layout);
    else if (a.rope.layout == KVR_ROPE_HALF)
        KVR_LAUNCH((rows_rotate_kernel<T, KVR_ROPE_HALF>), grid, dim3(kThreads), smem, s, d);
    else
        KVR_LAUNCH((rows_rotate_kernel<T, KVR_ROPE_INTERLEAVED>), grid, dim3(kThreads), smem, s, d);
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_rows_rotate(int dtype, const RowsRotate& a, cudaStream_t s) {
    return dtype == KVR_F32 ? launch_as<float>(a, s) : launch_as<__nv_bfloat16>(a, s);
}

cudaError_t launch_rope_table(const kvr_rope& rope, int rope_len, float2* table, cudaStream_t s) {
    const int64_t n = (int64_t)rope_len * (rope.rotary_dim / 2);
    KVR_LAUNCH(rope_table_kernel, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 16 * kNumSMs)), dim3(256), 0, s, rope,
               n, table);
    return cudaSuccess;
}

}  // namespace kvr
