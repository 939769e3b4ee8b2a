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

constexpr int kThreads = 128, kMaxRows = 16;   // rows a block
// Units a thread has in flight.  7680 rows of 32/8 heads x 128 in bf16: 27.8 us with two of 128 threads (5.7 TB/s),
// 28.4 with three, 26.8 with one, which 28/4 heads have nothing of; 29 to 32 with 256 threads.
template <int kBytes>
constexpr int kBatchOf = kBytes == 16 ? 2 : 4;

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

// A vector of kBytes (16, 8 or 4) as fp32.
template <typename T, int kBytes>
struct Vec {
    static constexpr int N = kBytes / (int)sizeof(T), W = kBytes / 4;
    uint32_t w[W];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (W == 4) *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p);
        else if constexpr (W == 2) *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
        else w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (W == 4) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (W == 2) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t*>(p) = w[0];
    }
    __device__ __forceinline__ void get(float* x) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (sizeof(T) == 4) x[i] = __uint_as_float(w[i]);
            else x[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        }
    }
    __device__ __forceinline__ void put(const float* x) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = __float_as_uint(x[i]);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
    }
};

struct RotateDev {
    RowsRotate a;
    float m;
    int rows_per_block, units, turned, heads;   // units of a head, those of them that turn; heads of a row
    Div by_units, by_heads;
};

// A head's units: `turned` of them hold two vectors of whole pairs, the others
// two vectors that are copied (or left alone in place).
template <int N, int kLayout>
__device__ __forceinline__ void unit_offsets(const RotateDev& d, int u, int* first, int* second) {
    if (u < d.turned && kLayout == KVR_ROPE_HALF) {
        *first = u * N;
        *second = u * N + d.a.rope.rotary_dim / 2;
    } else {
        *first = 2 * u * N;
        *second = *first + N;
    }
}

template <typename T, int kLayout, int kBytes>
__global__ void __launch_bounds__(kThreads, 8) rows_rotate_kernel(const __grid_constant__ RotateDev d) {
    using V = Vec<T, kBytes>;
    constexpr int N = V::N, kBatch = kBatchOf<kBytes>;
    extern __shared__ float2 cs[];   // [rows_per_block][N][turned units]: pair e of every unit side by side, for the banks' sake
    const RowsRotate& a = d.a;
    const int dh = a.rope.head_dim, half = a.rope.rotary_dim / 2, turned = d.turned;
    const int64_t row0 = (int64_t)blockIdx.x * d.rows_per_block;
    const int rows = (int)min((int64_t)d.rows_per_block, a.n_rows - row0);
    const int total = rows * d.heads * d.units;
    bool ready = false;
    for (int base = 0; base < total; base += kThreads * kBatch) {
        V x[kBatch][2];
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
            unit_offsets<N, kLayout>(d, unit[k], &f, &s);
            x[k][0].load(in + f);
            x[k][1].load(in + s);
            to[k] = out;
        }
        if (!ready) {
            for (int i = threadIdx.x; i < rows * half; i += kThreads) {
                const int r = i / half, p = i - r * half;
                cs[r * half + p % N * turned + p / N] = cos_sin(a.rope.turns[p], a.pos[row0 + r], d.m, a.inverse);
            }
            __syncthreads();
            ready = true;
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (!to[k]) continue;
            int f, s;
            unit_offsets<N, kLayout>(d, unit[k], &f, &s);
            if (unit[k] < d.turned) {
                float p[N], q[N];
                x[k][0].get(p);
                x[k][1].get(q);
                const float2* c = cs + row[k] * half + unit[k];
                if constexpr (kLayout == KVR_ROPE_HALF) {
#pragma unroll
                    for (int e = 0; e < N; ++e) turn(p[e], q[e], c[e * turned]);
                } else {
#pragma unroll
                    for (int e = 0; e < N / 2; ++e) {
                        turn(p[2 * e], p[2 * e + 1], c[e * turned]);
                        turn(q[2 * e], q[2 * e + 1], c[(N / 2 + e) * turned]);
                    }
                }
                x[k][0].put(p);
                x[k][1].put(q);
            }
            x[k][0].store(to[k] + f);
            x[k][1].store(to[k] + s);
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
    constexpr int es = sizeof(T);
    const int dh = a.rope.head_dim, rot = a.rope.rotary_dim, layout = a.rope.layout;
    // the widest vector that whole units are made of, each of two
    auto fits = [&](int bytes) {
        const int n = bytes / es;
        bool ok = rot % (2 * n) == 0 && dh % (2 * n) == 0 && (n > 1 || layout == KVR_ROPE_HALF);
        for (int w = 0; w < 2; ++w)
            if (a.heads[w])
                ok = ok && reinterpret_cast<uintptr_t>(a.in[w]) % bytes == 0 && reinterpret_cast<uintptr_t>(a.out[w]) % bytes == 0 &&
                     a.in_stride[w] * es % bytes == 0 && a.out_stride[w] * es % bytes == 0;
        return ok;
    };
    const int bytes = fits(16) ? 16 : fits(8) ? 8 : fits(4) ? 4 : 0, n = bytes / es;
    const int units = n ? dh / (2 * n) : dh / 2, heads = a.heads[0] + a.heads[1];
    // rows that fill a block's batch, fewer where there are not enough rows for the GPU
    int rows = std::max(1, std::min(kMaxRows, kThreads * (bytes == 16 ? kBatchOf<16> : kBatchOf<8>) / (units * heads)));
    rows = std::min(rows, std::max(1, a.n_rows / (2 * kNumSMs)));
    const RotateDev d{a, a.inverse ? 1.f / a.rope.attn : a.rope.attn, rows, units, n ? rot / (2 * n) : rot / 2, heads,
                      Div(units), Div(heads)};
    const dim3 grid((unsigned)((a.n_rows + (int64_t)rows - 1) / rows));
    const size_t smem = sizeof(float2) * rows * (rot / 2);
    if (n == 0) {
        KVR_LAUNCH((rows_rotate_pairs_kernel<T>), grid, dim3(kThreads), smem, s, d, layout);
        return cudaSuccess;
    }
    auto go = [&](auto half, auto interleaved) -> cudaError_t {
        KVR_LAUNCH(layout == KVR_ROPE_HALF ? half : interleaved, grid, dim3(kThreads), smem, s, d);
        return cudaSuccess;
    };
    constexpr int H = KVR_ROPE_HALF, I = KVR_ROPE_INTERLEAVED;
    if (bytes == 16) return go(rows_rotate_kernel<T, H, 16>, rows_rotate_kernel<T, I, 16>);
    if (bytes == 8) return go(rows_rotate_kernel<T, H, 8>, rows_rotate_kernel<T, I, 8>);
    return go(rows_rotate_kernel<T, H, 4>, rows_rotate_kernel<T, es == 4 ? H : I, 4>);
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
