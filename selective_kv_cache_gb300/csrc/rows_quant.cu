// rows_quant.cu -- packed rows into eight bits: RMSNorm with the residual's
// addition, the gated activation, plain rows; and back.
//
// For the fp32 values y of a row: top = max |y|, s = top / 127, code =
// rint(y / s).  A norm's y is h w r with r = 1 / sqrt(mean h^2 + eps), and r
// > 0 is one number a row: top = r max |h w| and the codes are those of h w,
// so the sum of squares and the maximum are found in one pass and one
// exchange, and nothing waits for r but the scale.
//
// HBM-bound: every byte moves once.  A warp or a block holds a row in registers
// between its loads and its stores, and has the next row's on their way
// meanwhile; rows wider than a block's registers are read twice.  A thread's
// unit is eight elements.  Rows that do not begin on 16 bytes, and widths that
// are not a multiple of eight, move in aligned 16-byte pieces all the same: a
// unit is shifted out of the pieces that hold it, and on the way out lanes
// hand the bytes of a piece to the lane that writes it.
// Instructions count as much as bytes (a row of 1536 in bf16 has 28 of them an
// element to spare at HBM's rate), so a thread has many elements, and a norm's
// sum leaves as soon as it is formed, which leaves h w alone to be kept.
// Maxima hand NaN on, and meet as unsigned numbers, where NaN lies above
// infinity: a row that is not finite shows in its maximum.
#include <cuda_bf16.h>

#include <algorithm>

#include "rows.h"

namespace kvr {
namespace {

constexpr float kTiny = 1.17549435e-38f;   // 2^-126

// words of a unit of eight elements
template <typename T>
constexpr int kWords = 2 * (int)sizeof(T);

// 16 bytes of lo | hi from byte `at` on, 0 < at < 16 a multiple of the element's size
__device__ __forceinline__ void shifted(const uint32_t* lo, const uint32_t* hi, uint32_t at, uint32_t* out) {
    uint32_t w[7];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = lo[i];
#pragma unroll
    for (int i = 0; i < 3; ++i) w[4 + i] = hi[i];
    uint32_t last = hi[3];
    if (at & 8) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 2];
        w[5] = last;
    }
    if (at & 4) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    const uint32_t bits = 8 * (at & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = __funnelshift_r(w[i], w[i + 1], bits);
}

// n of a unit's eight elements (0 to 8) at p.
template <typename T, bool kAligned>
__device__ __forceinline__ void load_unit(const T* p, int n, uint32_t* w) {
    constexpr int kPieces = kWords<T> / 4;
    if constexpr (kAligned) {
        if (n > 0) {
#pragma unroll
            for (int k = 0; k < kPieces; ++k) reinterpret_cast<uint4*>(w)[k] = reinterpret_cast<const uint4*>(p)[k];
        }
    } else {
        // aligned pieces, those that hold an element of the unit: they share its 16 bytes, so nothing else is touched
        const uint32_t off = (uint32_t)reinterpret_cast<uintptr_t>(p) & 15u;
        const uint4* from = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) - off);
        uint32_t c[4 * (kPieces + 1)];
#pragma unroll
        for (int k = 0; k <= kPieces; ++k)
            reinterpret_cast<uint4*>(c)[k] = 16 * k < (int)(n * sizeof(T) + off) && n > 0 ? from[k] : make_uint4(0u, 0u, 0u, 0u);
        if (off == 0) {
#pragma unroll
            for (int k = 0; k < 4 * kPieces; ++k) w[k] = c[k];
        } else {
#pragma unroll
            for (int k = 0; k < kPieces; ++k) shifted(c + 4 * k, c + 4 * k + 4, off, w + 4 * k);
        }
    }
}

template <typename T>
__device__ __forceinline__ void store_one(T* p, const uint32_t* w, int e) {   // element e of a unit's words
    if constexpr (sizeof(T) == 4) {
        reinterpret_cast<uint32_t*>(p)[e] = w[e];
    } else {
        reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
    }
}
// The same way out; consecutive lanes hold consecutive units, all lanes of the warp call.
template <typename T, bool kAligned>
__device__ __forceinline__ void store_unit(T* p, int n, const uint32_t* w) {
    constexpr int kPieces = kWords<T> / 4, E = 16 / (int)sizeof(T);   // elements of a piece
    if constexpr (kAligned) {
        if (n > 0) {
#pragma unroll
            for (int k = 0; k < kPieces; ++k) reinterpret_cast<uint4*>(p)[k] = reinterpret_cast<const uint4*>(w)[k];
        }
    } else {
        const uint32_t off = (uint32_t)reinterpret_cast<uintptr_t>(p) & 15u;   // one for all units of a row
        const int lane = threadIdx.x & 31, head = off ? (int)(16 - off) / (int)sizeof(T) : 0;   // elements before a border
        uint32_t next[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) next[i] = __shfl_down_sync(0xffffffffu, w[i], 1);
        int n_next = __shfl_down_sync(0xffffffffu, n, 1);
        if (lane == 31) n_next = 0;
        // piece k begins `head` elements into the unit's k-th 16 bytes; the last takes the next lane's first elements
        const bool last = n == 8 && n_next >= head;
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            uint32_t c[4];
            const uint32_t* hi = k + 1 < kPieces ? w + 4 * k + 4 : next;
            if (off) {
                shifted(w + 4 * k, hi, 16 - off, c);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) c[i] = w[4 * k + i];
            }
            const int first = k * E + head;
            if (k + 1 < kPieces ? n >= first + E : last) {
                *reinterpret_cast<uint4*>(p + first) = make_uint4(c[0], c[1], c[2], c[3]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e >= first && e < n && e < first + E) store_one(p, w, e);
            }
        }
        const bool taken = __shfl_up_sync(0xffffffffu, (int)last, 1) != 0 && lane > 0;
        if (!taken) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < head && e < n) store_one(p, w, e);
        }
    }
}

template <typename T>
__device__ __forceinline__ void unpack(const uint32_t* w, float* x) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (sizeof(T) == 4) x[i] = __uint_as_float(w[i]);
        else x[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
}
template <typename T>
__device__ __forceinline__ void pack(const float* x, uint32_t* w) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
}

// rint(y * inv) of two values in the low bytes: adding 1.5 * 2^23 leaves the
// integer, rounded to nearest even, in the low bits of the sum.  The products are
// rounded by themselves, as the formula in fp32 has it: fused with the addition,
// places next to a half go to the other code.  The assembler fuses a pair's
// product with a pair's addition, and a product plus a zero that it knows, so the
// zero comes from the launch.  5632 x 4096 of bf16 from L2, us: fused one by one
// 8.0, not fused 8.6, in pairs 7.8.
__device__ __forceinline__ void code_bits(float y0, float y1, float inv, float zero, uint32_t* w) {
    asm("{\n\t.reg .b64 y, i, m, z;\n\t"
        "mov.b64 y, {%2, %3};\n\t"
        "mov.b64 i, {%4, %4};\n\t"
        "mov.b64 z, {%5, %5};\n\t"
        "mov.b64 m, {%6, %6};\n\t"
        "fma.rn.f32x2 y, y, i, z;\n\t"
        "add.rn.f32x2 y, y, m;\n\t"
        "mov.b64 {%0, %1}, y;\n\t}"
        : "=r"(w[0]), "=r"(w[1])
        : "f"(y0), "f"(y1), "f"(inv), "f"(zero), "f"(12582912.f));
}
__device__ __forceinline__ void store_codes(int8_t* p, int n, const float* y, float inv, float zero, bool bad, bool whole) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t c[4];
        code_bits(y[4 * i], y[4 * i + 1], inv, zero, c);
        code_bits(y[4 * i + 2], y[4 * i + 3], inv, zero, c + 2);
        w[i] = bad ? 0u : __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    }
    if (whole && n == 8) {   // whole: the codes' units are 8-byte aligned
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) p[e] = (int8_t)(w[e / 4] >> (8 * (e % 4)));
    }
}

// g / (1 + exp(-g)) * u.  bf16 rows take the approximate exponential, off by 2 +
// 1.2 |g| ulp, and division: (6 + 1.2 |g|) 2^-23 of the value with the roundings,
// below half a step of bf16 for all g.  fp32 rows take the accurate ones.  Where
// exp(-g) passes fp32's range, or 2^126 in the approximate division, the quotient
// is 0 in place of something below 2^-119.
template <typename T>
__device__ __forceinline__ float gated(float g, float u) {
    if constexpr (sizeof(T) == 4) return g / (1.f + expf(-g)) * u;
    return __fdividef(g, 1.f + __expf(-g)) * u;
}

// What a thread reads of one unit: the row's, and the residual's or the up half's.
template <RowOp kOp, typename T, bool kAligned>
struct Unit {
    uint32_t a[kWords<T>], b[kOp == RowOp::Quantise ? 1 : kWords<T>];
    __device__ __forceinline__ void load(const RowsQuant& q, int64_t row, int i, int n) {
        const T* x = reinterpret_cast<const T*>(q.x) + row * q.x_stride + i;
        load_unit<T, kAligned>(x, n, a);
        if constexpr (kOp == RowOp::Norm) {
            if (q.res) load_unit<T, kAligned>(reinterpret_cast<const T*>(q.res) + row * q.res_stride + i, n, b);
        }
        if constexpr (kOp == RowOp::Swiglu) load_unit<T, kAligned>(x + q.d, n, b);
    }
    // the values before the quantiser: h (norm), the gated value, or x
    __device__ __forceinline__ void values(const RowsQuant& q, float* v) const {
        unpack<T>(a, v);
        if constexpr (kOp != RowOp::Quantise) {
            if (kOp == RowOp::Swiglu || q.res) {
                float o[8];
                unpack<T>(b, o);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = kOp == RowOp::Swiglu ? gated<T>(v[e], o[e]) : v[e] + o[e];
            }
        }
    }
};

// max(|a|, |b|, c), NaN if one of them is
__device__ __forceinline__ float top3(float a, float b, float c) {
    float d;
    asm("{\n\t.reg .f32 x, y;\n\tabs.f32 x, %1;\n\tabs.f32 y, %2;\n\tmax.NaN.f32 %0, x, y, %3;\n\t}" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Sum and maximum over the threads of a row: a warp by itself, or the whole
// block, through slot `turn` of two.
template <bool kWarp, bool kSum>
__device__ __forceinline__ void row_reduce(float& sum, uint32_t& top, int turn) {
    top = __reduce_max_sync(0xffffffffu, top);
    if constexpr (kSum) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if constexpr (!kWarp) {
        __shared__ float sums[2][32];
        __shared__ uint32_t tops[2][32];
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = blockDim.x >> 5;
        if (lane == 0) {
            sums[turn][warp] = sum;
            tops[turn][warp] = top;
        }
        __syncthreads();
        top = __reduce_max_sync(0xffffffffu, lane < n ? tops[turn][lane] : 0u);
        if constexpr (kSum) {
            sum = lane < n ? sums[turn][lane] : 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
    }
}

// Threads of a block at most, and blocks an SM at least.  Rows of bf16 leave
// registers for the next row's units beside this one's.
constexpr int block_most(int slots, bool warp, int size, bool aligned) {
    return warp ? 128 : slots == 1 ? 256 : slots == 2 ? (aligned ? 512 : 1024) : slots == 4 && size == 2 ? 640 : 1024;
}
constexpr int blocks_least(int slots, bool warp, int size, bool aligned) {
    return warp ? (slots == 1 ? 8 : 5) : slots == 1 ? 4 : slots == 2 && size == 2 && aligned ? 2 : 1;
}

// kSlots: units a thread holds of a row, 0: the row is read twice.  kWarp: a
// warp a row, several rows a block; else a block a row.
template <RowOp kOp, typename T, bool kAligned, int kSlots, bool kWarp>
__global__ void __launch_bounds__(block_most(kSlots, kWarp, sizeof(T), kAligned), blocks_least(kSlots, kWarp, sizeof(T), kAligned))
    rows_quant_kernel(const __grid_constant__ RowsQuant a) {
    constexpr bool kNorm = kOp == RowOp::Norm;
    // the next row's loads go out before this one's exchange; units that are shifted would wait for them there
    constexpr bool kAhead = kSlots > 0 && sizeof(T) == 2 && kAligned;
    constexpr bool kKeepW = kNorm && (kSlots == 1 || kSlots == 2);   // else the weights are read for every row, from L1
    constexpr int kHold = kSlots > 0 ? kSlots : 1;
    const int lane = kWarp ? threadIdx.x & 31 : threadIdx.x, step = kWarp ? 32 : blockDim.x;
    const int64_t per_block = kWarp ? blockDim.x >> 5 : 1, stride = gridDim.x * per_block;
    int64_t row = blockIdx.x * per_block + (kWarp ? threadIdx.x >> 5 : 0);
    const T* weight = reinterpret_cast<const T*>(a.weight);
    auto count = [&](int k) { return min(8, max(0, a.d - 8 * (lane + k * step))); };
    float wt[kKeepW ? kHold : 1][8];
    auto load_weight = [&](int k, float* w) {
        uint32_t raw[kWords<T>];
        load_unit<T, kAligned>(weight + 8 * (lane + k * step), count(k), raw);
        unpack<T>(raw, w);
    };
    if constexpr (kKeepW) {
#pragma unroll
        for (int k = 0; k < kHold; ++k) load_weight(k, wt[k]);
    }
    Unit<kOp, T, kAligned> u[kAhead ? kHold : 1];
    if constexpr (kAhead) {
        if (row < a.n_rows) {
#pragma unroll
            for (int k = 0; k < kHold; ++k) u[k].load(a, row, 8 * (lane + k * step), count(k));
        }
    }
    for (int turn = 0; row < a.n_rows; row += stride, turn ^= 1) {
        float v[kHold][8];   // h w, or the value
        float sum = 0.f, top = 0.f;
        // Unit k of the row into v; `first`: for the statistics, with the sum on its way out.  Outputs may be inputs:
        // a unit is written by its own warp, from what its lanes have read by then.
        auto take = [&](int k, const Unit<kOp, T, kAligned>& from, float* v, bool first) {
            const int n = count(k);
            from.values(a, v);
            if constexpr (kNorm) {
                if (a.sum && (kSlots > 0 || !first)) {   // a row that is read twice: in the second reading
                    uint32_t o[kWords<T>];
                    pack<T>(v, o);
                    if constexpr (!kAligned) __syncwarp();
                    store_unit<T, kAligned>(reinterpret_cast<T*>(a.sum) + row * a.sum_stride + 8 * (lane + k * step), n, o);
                }
            }
            if (n > 0) {
                if constexpr (!kAligned) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e >= n) v[e] = 0.f;
                }
                if constexpr (kNorm) {
                    float* w = wt[kKeepW ? k : 0];
                    if constexpr (!kKeepW) load_weight(k, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        sum = fmaf(v[e], v[e], sum);
                        v[e] = kAligned || e < n ? v[e] * w[e] : 0.f;
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; e += 2) top = top3(v[e], v[e + 1], top);
            }
        };
        if constexpr (kAhead) {
#pragma unroll
            for (int k = 0; k < kHold; ++k) take(k, u[k], v[k], true);
            if (row + stride < a.n_rows) {
#pragma unroll
                for (int k = 0; k < kHold; ++k) u[k].load(a, row + stride, 8 * (lane + k * step), count(k));
            }
        } else if constexpr (kSlots > 0) {
            // two units' loads together, as many as registers hold
            constexpr int kTogether = kSlots < 2 ? 1 : 2;
#pragma unroll
            for (int k0 = 0; k0 < kHold; k0 += kTogether) {
                Unit<kOp, T, kAligned> now[kTogether];
#pragma unroll
                for (int k = 0; k < kTogether; ++k) now[k].load(a, row, 8 * (lane + (k0 + k) * step), count(k0 + k));
#pragma unroll
                for (int k = 0; k < kTogether; ++k) take(k0 + k, now[k], v[k0 + k], true);
            }
        } else {
            for (int k = 0; 8 * (k * step) < a.d; ++k) {
                u[0].load(a, row, 8 * (lane + k * step), count(k));
                take(k, u[0], v[0], true);
            }
        }
        uint32_t top_bits = __float_as_uint(top);
        row_reduce<kWarp, kNorm>(sum, top_bits, turn);
        float r = 1.f;
        bool bad = top_bits >= 0x7f800000u;
        // A row's own scale decides whether it is zeros.  Where h w are tiny and r is large, h w go up by 2^32 and r down,
        // so that the scale before r is no subnormal number: 2^-149 / 127 * 2^32 is 2^-124.
        const bool tiny = kNorm && top_bits < 0x12800000u;   // 2^-90
        if constexpr (kNorm) {
            const float q = sum / (float)a.d + a.eps;
            r = rsqrtf(q);
            // A sum past fp32's range would make zeros of the row, one that has lost its squares below it a wrong root: NaN.
            // (Zeros need no root but a finite one.)
            if (!bad && !((q >= kTiny || (top_bits == 0u && q > 0.f)) && q <= 3.4028234e38f)) {
                bad = true;
                r = __int_as_float(0x7fffffff);
            }
            if (tiny) {
                top_bits = __float_as_uint(__uint_as_float(top_bits) * 0x1p32f);
                r *= 0x1p-32f;
                if constexpr (kSlots > 0) {
#pragma unroll
                    for (int k = 0; k < kHold; ++k)
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[k][e] *= 0x1p32f;
                }
            }
        }
        // of the values before r: r lies in the scale alone
        const float s0 = __uint_as_float(top_bits) * (1.f / 127.f);
        const float scale = kNorm ? s0 * r : s0;
        const bool none = !bad && scale < kTiny;
        const float inv = bad || none ? 0.f : 1.f / s0;
        if (a.codes && lane == 0) a.scales[row] = bad ? __int_as_float(0x7fffffff) : none ? 0.f : scale;
        auto put = [&](int k, const float* v) {
            const int i = 8 * (lane + k * step), n = count(k);
            if (a.codes && n > 0) store_codes(a.codes + row * a.code_stride + i, n, v, inv, a.zero, bad, a.codes_aligned);
            if (a.out) {
                float y[8];
                uint32_t o[kWords<T>];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = kNorm ? v[e] * r : v[e];
                pack<T>(y, o);
                store_unit<T, kAligned>(reinterpret_cast<T*>(a.out) + row * a.out_stride + i, n, o);
            }
        };
        if constexpr (kSlots > 0) {
#pragma unroll
            for (int k = 0; k < kHold; ++k) put(k, v[k]);
        } else {
            for (int k = 0; 8 * (k * step) < a.d; ++k) {
                u[0].load(a, row, 8 * (lane + k * step), count(k));
                take(k, u[0], v[0], false);
                if (tiny) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[0][e] *= 0x1p32f;
                }
                put(k, v[0]);
            }
        }
    }
}

// codes to values: 16 a thread in vectors, or a unit of eight whatever the
// alignment, 32 units of a row a warp
template <typename T>
__global__ void __launch_bounds__(256) rows_dequantise_kernel(const int8_t* codes, int64_t code_stride, const float* scales,
                                                              T* out, int64_t out_stride, int64_t total, Div per) {
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += (int64_t)gridDim.x * 256) {
        const int64_t row = total < (int64_t(1) << 31) ? per((uint32_t)t) : t / per.d;
        const int i = (int)(t - row * per.d) * 16;
        const uint4 u = *reinterpret_cast<const uint4*>(codes + row * code_stride + i);
        const float s = scales[row];
        T* o = out + row * out_stride + i;
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        float y[16];
        uint32_t packed[2 * kWords<T>];
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = s * (float)(int8_t)(w[e / 4] >> (8 * (e % 4)));
        pack<T>(y, packed);
        pack<T>(y + 8, packed + kWords<T>);
        store_unit<T, true>(o, 8, packed);
        store_unit<T, true>(o + 8, 8, packed + kWords<T>);
    }
}
template <typename T>
__global__ void __launch_bounds__(256) rows_dequantise_any_kernel(const int8_t* codes, int64_t code_stride, const float* scales,
                                                                  T* out, int64_t out_stride, int64_t total, Div per,
                                                                  int d, int codes_aligned) {
    const int lane = threadIdx.x & 31;
    for (int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); t < total; t += (int64_t)gridDim.x * 8) {   // a warp's
        const int64_t row = total < (int64_t(1) << 31) ? per((uint32_t)t) : t / per.d;
        const int i = (int)(t - row * per.d) * 256 + 8 * lane, n = min(8, max(0, d - i));
        const int8_t* c = codes + row * code_stride + i;
        const float s = scales[row];
        uint32_t w[2] = {0u, 0u}, packed[kWords<T>];
        if (codes_aligned && n == 8) {
            const uint2 u = *reinterpret_cast<const uint2*>(c);
            w[0] = u.x;
            w[1] = u.y;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) w[e / 4] |= (uint32_t)(uint8_t)c[e] << (8 * (e % 4));
        }
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = s * (float)(int8_t)(w[e / 4] >> (8 * (e % 4)));
        pack<T>(y, packed);
        store_unit<T, false>(out + row * out_stride + i, n, packed);
    }
}

// Blocks of a kernel that the GPU holds at once, asked for once per block size.
template <auto kKernel>
int resident(int threads) {
    static std::atomic<uint32_t> seen{0};   // threads, blocks an SM
    const uint32_t v = seen.load(std::memory_order_relaxed);
    if ((int)(v >> 16) == threads) return (int)(v & 0xffffu) * kNumSMs;
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kKernel, threads, 0) != cudaSuccess || n < 1) n = 1;
    seen.store((uint32_t)threads << 16 | (uint32_t)n, std::memory_order_relaxed);
    return n * kNumSMs;
}

template <RowOp kOp, typename T, bool kAligned, int kSlots, bool kWarp>
cudaError_t launch_with(const RowsQuant& a, int units, cudaStream_t s) {
    constexpr auto kernel = rows_quant_kernel<kOp, T, kAligned, kSlots, kWarp>;
    const int slots = std::max(kSlots, 1);
    const int threads = kWarp ? 128 : kSlots == 0 ? 1024 : ((units + slots - 1) / slots + 31) / 32 * 32;
    const int blocks = kWarp ? (int)((a.n_rows + int64_t(3)) / 4) : a.n_rows;
    KVR_LAUNCH(kernel, dim3(std::min(blocks, resident<kernel>(threads))), dim3(threads), 0, s, a);
    return cudaSuccess;
}

// A warp a row up to 512 elements, a block above.  Units a thread, measured:
// fp32 of 1024, 8000 rows gated: one 14.6 us, two 17.3, four 26; bf16 of 1536,
// 98304 rows stored: two 103 us, four 78; of 4096, 5632 rows stored: 18.5 and
// 14.5; 4000 rows of 5001, added and normed: two 55 us, four 73.
template <RowOp kOp, typename T, bool kAligned>
cudaError_t launch_as(const RowsQuant& a, cudaStream_t s) {
    const int units = (a.d + 7) / 8;
    if (units <= 32) return launch_with<kOp, T, kAligned, 1, true>(a, units, s);
    if (units <= 64) return launch_with<kOp, T, kAligned, 2, true>(a, units, s);
    constexpr bool kMost = sizeof(T) == 2 && kAligned && kOp != RowOp::Norm;
    if constexpr (sizeof(T) == 4) {
        if (units <= 256) return launch_with<kOp, T, kAligned, 1, false>(a, units, s);
    }
    if constexpr (!kMost) {
        if (units <= (kAligned || sizeof(T) == 4 ? 1024 : 2048)) return launch_with<kOp, T, kAligned, 2, false>(a, units, s);
    }
    if (units <= 2560) return launch_with<kOp, T, kAligned, 4, false>(a, units, s);
    return launch_with<kOp, T, kAligned, 0, false>(a, units, s);
}

bool in_vectors(const void* p, int64_t stride, int size, int bytes) {
    return p == nullptr || ((reinterpret_cast<uintptr_t>(p) % bytes) == 0 && (stride * size) % bytes == 0);
}

template <RowOp kOp, typename T>
cudaError_t launch_op(const RowsQuant& a, cudaStream_t s) {
    const int es = sizeof(T);
    const bool vec = a.d % 8 == 0 && in_vectors(a.x, a.x_stride, es, 16) && in_vectors(a.res, a.res_stride, es, 16) &&
                     in_vectors(a.sum, a.sum_stride, es, 16) && in_vectors(a.out, a.out_stride, es, 16) &&
                     in_vectors(a.weight, 0, es, 16);
    RowsQuant b = a;
    b.codes_aligned = in_vectors(a.codes, a.code_stride, 1, 8);
    return vec ? launch_as<kOp, T, true>(b, s) : launch_as<kOp, T, false>(b, s);
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
    const int codes_aligned = in_vectors(codes, code_stride, 1, 8);
    auto go = [&](auto* o) -> cudaError_t {
        using T = std::remove_pointer_t<decltype(o)>;
        const Div per(vec ? d / 16 : (d + 255) / 256);   // 16 codes a thread, 256 a warp
        const int64_t total = (int64_t)n_rows * per.d;
        const dim3 grid((unsigned)std::min<int64_t>((total + (vec ? 255 : 7)) / (vec ? 256 : 8), 1 << 20));
        if (vec)
            KVR_LAUNCH((rows_dequantise_kernel<T>), grid, dim3(256), 0, s, codes, code_stride, scales, o, out_stride, total,
                       per);
        else
            KVR_LAUNCH((rows_dequantise_any_kernel<T>), grid, dim3(256), 0, s, codes, code_stride, scales, o, out_stride,
                       total, per, d, codes_aligned);
        return cudaSuccess;
    };
    return dtype == KVR_F32 ? go(static_cast<float*>(out)) : go(static_cast<__nv_bfloat16*>(out));
}

}  // namespace kvr
