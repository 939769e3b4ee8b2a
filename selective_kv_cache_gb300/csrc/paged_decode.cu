// paged_decode.cu -- attention of a few rows per K/V head over the paged cache
// (bf16 and 4-bit pages): decode steps and drafted tokens, up to 16 rows
// (positions x query heads of the K/V head) per item.
//
//   S^T = K Q^T (16 keys x 8 rows per mma),  O^T += V^T P^T,
//   running maximum and sum in base 2, one pass over the keys.
//
// Bound by reading K and V once.  There are 8 to 16 rows against 128-row
// tensor-memory tiles, so the wide matrix unit would leave 9/10 of its rows
// empty and, for 4-bit pages, want every key written back to shared memory as
// 16-bit values first.  Here K and V are the *A* operand of mma.sync m16n8k16 and
// go from global memory to the registers in the operand's own layout; nothing
// is staged in shared memory and no row is padded beyond 8.
//   K (rows = keys): lane (r, t) = (lane / 4, lane % 4) holds dims in 16-byte
//     chunks of keys r and r + 8; the contraction may take the dims in any
//     order as long as Q does, so the chunks are loaded as they lie.
//   V (rows = dims): lane (r, t) holds 16 dims of keys 2t, 2t + 1, 2t + 8,
//     2t + 9; a byte permute of two keys' words makes the (key, key + 1) pairs.
//   P^T comes from S^T's accumulator by movmatrix (8x8 transposes).
// 4-bit pages: the codes themselves are the operand (128 + c for K, c - 8 for
//   V: both exact in bf16, one logic op and one subtraction per two values);
//   scales and offsets are applied to S in fp32 (s (acc) + (o - 128 s) sum q)
//   and to P (p s, per group; the offsets' part sum p (o + 8 s) is kept in
//   fp32).  So 4-bit keys add no rounding, and P s is rounded once to bf16,
//   as P is for bf16 pages (2^-8 of a weight at most).
// The warps of a CTA take every kWarps-th run of keys, each with its own
// maximum, sum and output, joined through shared memory when the CTA is done
// with an (item, head).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged.h"

namespace kvr {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLazy = 8.0f;   // log2 of the largest P before the maximum is raised

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// bf16 pair (128 + low nibbles of the two halves)
__device__ __forceinline__ uint32_t code_pair(uint32_t x) { return (x & 0x000f000fu) | 0x43004300u; }
// the same pair less 136: code - 8, exact
__device__ __forceinline__ uint32_t centred(uint32_t x) {
    const uint32_t m = 0xc308c308u;   // -136
    const __nv_bfloat162 y =
        __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&m));
    return *reinterpret_cast<const uint32_t*>(&y);
}
// K and V are read once: they need not displace what is reused
__device__ __forceinline__ uint4 ld16(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ld8(const uint8_t* p) {
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
// Scale-offset pairs of one row: NG words
template <int NG>
__device__ __forceinline__ void ld_meta(const uint8_t* p, uint32_t* m) {
    if (NG == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        m[0] = v.x, m[1] = v.y, m[2] = v.z, m[3] = v.w;
    } else if (NG == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        m[0] = v.x, m[1] = v.y;
    } else {
        m[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}
__device__ __forceinline__ float2 so(uint32_t m) { return __half22float2(*reinterpret_cast<const __half2*>(&m)); }

// One 16-key block in registers.
template <int NG>
struct KBlock {
    uint4 w[2];            // keys r, r + 8
    uint32_t m[2][NG];
};
template <>
struct KBlock<0> {
    uint4 w[2][4];
};
template <int NG>
struct VBlock {
    uint2 w[4];            // keys 2t, 2t + 1, 2t + 8, 2t + 9
    uint32_t m[2][NG];     // of keys r, r + 8
};
template <>
struct VBlock<0> {
    uint4 w[4][2];
};

// NG: 0 = bf16 pages, else the scale groups of a 4-bit row.  NT: 8-row tiles of an
// item.  NB: 16-key blocks of a warp's step.  kExtra: cap, biases or slopes.
template <int NG, int NT, bool kExtra>
struct Decode {
    static constexpr int NB = NG ? 2 : 1;
    static constexpr int kUnit = 16 * NB * kWarps;
    static constexpr int RB = NG ? 64 : 256;    // bytes of a row
    static constexpr int GN = NG ? NG : 1;
    static constexpr int LDO = 132;             // padded output row in shared memory
};

template <int NG, int NT, bool kExtra, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas) paged_decode_kernel(PagedAttn a) {
    using D = Decode<NG, NT, kExtra>;
    constexpr int NB = D::NB, GN = D::GN, RB = D::RB;
    __shared__ float sO[kWarps][8][D::LDO];
    __shared__ float sM[kWarps][8 * NT], sL[kWarps][8 * NT];
    pdl_wait();
    pdl_trigger();
    const PagedShare sh = a.shares[blockIdx.x];
    if (sh.item < 0) return;
    const int u1 = a.shares[blockIdx.x + 1].u0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
    const int H = a.p.n_kv_heads, G = a.G, shift = a.p.page_shift, in_page = (1 << shift) - 1;
    const float sl2 = a.scale * kLog2e;
    PagedItem it = sh.first;
    int i = sh.item, h = sh.head, off = sh.off, u = sh.u0;
    bool first = true;
    // byte offsets of this lane inside a 16-key block of one head's rows
    const int64_t ss = a.p.slot_stride;
    const int64_t k_at = r * ss * RB + 16 * t, k8 = 8 * ss * RB;
    const int64_t v_at = 2 * t * ss * RB + (NG ? 8 : 32) * r;
    const int64_t m_at = r * ss * (4 * GN), m8 = 8 * ss * (4 * GN);

    while (u < u1) {
        const int n = min(it.units - off, u1 - u);
        const int rows = it.rows * G;
        const int* table = a.p.table + (int64_t)it.seq * a.p.max_pages;
        // 16-key blocks [kb0, kb_end) hold the item's keys; this warp's steps
        // start at kb and go on kWarps * NB blocks at a time
        const int kb_first = it.klo >> 4, kb_end = (it.khi + 15) >> 4;
        int kb = (it.klo / D::kUnit + off) * (kWarps * NB) + warp * NB;
        const int kb_stop = min(kb_end, (it.klo / D::kUnit + off + n) * (kWarps * NB));

        KBlock<NG> K[NB];
        VBlock<NG> V[NB];
        int64_t row[NB];       // page row (slot 0 of the block) of the blocks being loaded
        int pid[NB];           // page ids of the step after them
        auto fetch_ids = [&](int k) {
#pragma unroll
            for (int x = 0; x < NB; ++x)
                pid[x] = k + x >= kb_first && k + x < kb_stop ? table[(k + x) >> (shift - 4)] : 0;
        };
        auto place = [&](int k) {
#pragma unroll
            for (int x = 0; x < NB; ++x)
                row[x] = paged_row(a.p, paged_id(a.p, pid[x]), ((k + x) << 4) & in_page, h);
        };
        auto load_k = [&](int k) {
#pragma unroll
            for (int x = 0; x < NB; ++x) {
                if (k + x >= kb_stop) continue;
                const uint8_t* p = a.p.k + row[x] * RB + k_at;
                if constexpr (NG == 0) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        K[x].w[0][c] = ld16(p + 64 * c);
                        K[x].w[1][c] = ld16(p + k8 + 64 * c);
                    }
                } else {
                    K[x].w[0] = ld16(p);
                    K[x].w[1] = ld16(p + k8);
                    const uint8_t* q = a.p.ks + row[x] * (4 * GN) + m_at;
                    ld_meta<NG>(q, K[x].m[0]);
                    ld_meta<NG>(q + m8, K[x].m[1]);
                }
            }
        };
        auto load_v = [&](int k) {
#pragma unroll
            for (int x = 0; x < NB; ++x) {
                if (k + x >= kb_stop) continue;
                const uint8_t* p = a.p.v + row[x] * RB + v_at;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint8_t* pj = p + ((j & 1) + 8 * (j >> 1)) * ss * RB;
                    if constexpr (NG == 0) {
                        V[x].w[j][0] = ld16(pj);
                        V[x].w[j][1] = ld16(pj + 16);
                    } else {
                        V[x].w[j] = ld8(pj);
                    }
                }
                if constexpr (NG != 0) {
                    const uint8_t* q = a.p.vs + row[x] * (4 * GN) + m_at;
                    ld_meta<NG>(q, V[x].m[0]);
                    ld_meta<NG>(q + m8, V[x].m[1]);
                }
            }
        };
        if (kb + NB <= kb_first) kb += kWarps * NB;   // a first step wholly before klo
        fetch_ids(kb);
        place(kb);
        load_k(kb);
        load_v(kb);
        fetch_ids(kb + kWarps * NB);

        // Q as the B operand: row n = 8 nt + r, this lane's dims
        uint32_t q[NT][16];
        float qs[NT][2][GN];       // sums of q over a scale group, rows 2t and 2t + 1
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int m = 8 * nt + r;
            float sums[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint4 w = make_uint4(0u, 0u, 0u, 0u);
                if (m < rows)
                    w = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.q) +
                                                        (int64_t)(it.row0 + m / G) * a.q_stride +
                                                        (int64_t)(h * G + m % G) * 128 + 32 * c + 8 * t);
                if constexpr (NG == 0) {
                    q[nt][4 * c] = w.x, q[nt][4 * c + 1] = w.y, q[nt][4 * c + 2] = w.z, q[nt][4 * c + 3] = w.w;
                } else {   // pairs (dim e, dim e + 4), as the codes' nibbles pair up
                    q[nt][4 * c] = __byte_perm(w.x, w.z, 0x5410);
                    q[nt][4 * c + 1] = __byte_perm(w.x, w.z, 0x7632);
                    q[nt][4 * c + 2] = __byte_perm(w.y, w.w, 0x5410);
                    q[nt][4 * c + 3] = __byte_perm(w.y, w.w, 0x7632);
                    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sums[c] += __uint_as_float(ws[e] << 16) + __uint_as_float(ws[e] & 0xffff0000u);
                }
            }
            if constexpr (NG != 0) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    sums[c] += __shfl_xor_sync(0xffffffffu, sums[c], 1);
                    sums[c] += __shfl_xor_sync(0xffffffffu, sums[c], 2);
                }
                float grp[GN];
#pragma unroll
                for (int g = 0; g < GN; ++g) {
                    grp[g] = 0.f;
#pragma unroll
                    for (int c = 0; c < 4 / GN; ++c) grp[g] += sums[g * (4 / GN) + c];
                    qs[nt][0][g] = __shfl_sync(0xffffffffu, grp[g], 8 * t);
                    qs[nt][1][g] = __shfl_sync(0xffffffffu, grp[g], 8 * t + 4);
                }
            }
        }
        // the intervals of rows 2t, 2t + 1 (rows that do not exist: the item's)
        // and the keys every row sees
        int lo[NT][2], hi[NT][2], gpos[NT][2], all_lo = it.klo, all_hi = it.khi;
        float slope[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int m = 8 * nt + 2 * t + e;
                lo[nt][e] = it.klo, hi[nt][e] = it.khi, gpos[nt][e] = 0, slope[nt][e] = 0.f;
                if (m < rows) {
                    paged_interval(a, it.row0 + m / G, it.kv, &lo[nt][e], &hi[nt][e]);
                    if (kExtra && a.slopes) {
                        gpos[nt][e] = a.r.pos[it.row0 + m / G];
                        slope[nt][e] = a.slopes[h * G + m % G] * kLog2e;
                    }
                }
                all_lo = max(all_lo, lo[nt][e]);
                all_hi = min(all_hi, hi[nt][e]);
            }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, o));
            all_hi = min(all_hi, __shfl_xor_sync(0xffffffffu, all_hi, o));
        }

        float o[NT][8][4], corr[NT][2][GN], m_run[NT][2], l_run[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int d = 0; d < 8; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][d][e] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m_run[nt][e] = -INFINITY;
                l_run[nt][e] = 0.f;
#pragma unroll
                for (int g = 0; g < GN; ++g) corr[nt][e][g] = 0.f;
            }
        }

        for (; kb < kb_stop; kb += kWarps * NB) {
            const int next = kb + kWarps * NB;
            // ---- scores S^T of the step's keys
            float x[NB][NT][4];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if constexpr (NG == 0) {
                        float c0[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint4 p = K[b].w[0][c], s = K[b].w[1][c];
                            mma16816(c0, p.x, s.x, p.y, s.y, q[nt][4 * c], q[nt][4 * c + 1]);
                            mma16816(c1, p.z, s.z, p.w, s.w, q[nt][4 * c + 2], q[nt][4 * c + 3]);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[b][nt][e] = c0[e] + c1[e];
                    } else {
                        const uint4 p = K[b].w[0], s = K[b].w[1];
                        // 32-dim block g: units of the lane's two chunks
                        const uint32_t ph[4] = {__byte_perm(p.x, p.z, 0x5410), __byte_perm(p.x, p.z, 0x7632),
                                                __byte_perm(p.y, p.w, 0x5410), __byte_perm(p.y, p.w, 0x7632)};
                        const uint32_t sh_[4] = {__byte_perm(s.x, s.z, 0x5410), __byte_perm(s.x, s.z, 0x7632),
                                                 __byte_perm(s.y, s.w, 0x5410), __byte_perm(s.y, s.w, 0x7632)};
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[b][nt][e] = 0.f;
#pragma unroll
                        for (int g = 0; g < GN; ++g) {
                            float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int j = g * (4 / GN); j < (g + 1) * (4 / GN); ++j) {
                                mma16816(c, code_pair(ph[j]), code_pair(sh_[j]), code_pair(ph[j] >> 4),
                                         code_pair(sh_[j] >> 4), q[nt][4 * j], q[nt][4 * j + 1]);
                                mma16816(c, code_pair(ph[j] >> 8), code_pair(sh_[j] >> 8), code_pair(ph[j] >> 12),
                                         code_pair(sh_[j] >> 12), q[nt][4 * j + 2], q[nt][4 * j + 3]);
                            }
                            const float2 s0 = so(K[b].m[0][g]), s1 = so(K[b].m[1][g]);
                            const float o0 = fmaf(-128.f, s0.x, s0.y), o1 = fmaf(-128.f, s1.x, s1.y);
                            x[b][nt][0] = fmaf(s0.x, c[0], fmaf(o0, qs[nt][0][g], x[b][nt][0]));
                            x[b][nt][1] = fmaf(s0.x, c[1], fmaf(o0, qs[nt][1][g], x[b][nt][1]));
                            x[b][nt][2] = fmaf(s1.x, c[2], fmaf(o1, qs[nt][0][g], x[b][nt][2]));
                            x[b][nt][3] = fmaf(s1.x, c[3], fmaf(o1, qs[nt][1][g], x[b][nt][3]));
                        }
                    }
                }
            }
            // K's registers are free: the next step's keys
            place(next);
            load_k(next);
            // ---- logits in base 2
            float ls = sl2;   // what is left to multiply x by
            if (kExtra) {
                ls = 1.f;
                const float cap_in = a.softcap > 0.f ? 2.f * sl2 / a.softcap : 0.f;
                const float cap_out = a.softcap * kLog2e;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    float bias[2] = {0.f, 0.f};
                    const int64_t word = (int64_t)it.seq * a.words + ((kb + b) >> 1);
                    const int bit = 16 * ((kb + b) & 1) + r;
                    if (a.loc && kb + b < kb_stop) {
                        const uint32_t w = a.loc[word] >> bit;
                        bias[0] += (w & 1u) ? a.alpha * kLog2e : 0.f;
                        bias[1] += (w >> 8 & 1u) ? a.alpha * kLog2e : 0.f;
                    }
                    if (a.snk && kb + b < kb_stop) {
                        const uint32_t w = a.snk[word] >> bit;
                        bias[0] += (w & 1u) ? a.beta * kLog2e : 0.f;
                        bias[1] += (w >> 8 & 1u) ? a.beta * kLog2e : 0.f;
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float y = x[b][nt][e];
                            // cap tanh(u) = cap (1 - 2 / (1 + exp(2u)))
                            y = a.softcap > 0.f ? cap_out - 2.f * cap_out * __fdividef(1.f, 1.f + ex2(y * cap_in))
                                                : y * sl2;
                            const int key = 16 * (kb + b) + r + 8 * (e >> 1);
                            y = fmaf(-slope[nt][e & 1], (float)abs(gpos[nt][e & 1] - key), y + bias[e >> 1]);
                            x[b][nt][e] = y;
                        }
                }
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int key0 = 16 * (kb + b);
                if (key0 < all_lo || key0 + 16 > all_hi) {   // warp-uniform: some row does not see some of the keys
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = key0 + r + 8 * (e >> 1);
                            if (key < lo[nt][e & 1] || key >= hi[nt][e & 1]) x[b][nt][e] = -INFINITY;
                        }
                    if (key0 < it.klo || key0 + 16 > it.khi) {   // keys nobody sees: whatever V's slots hold is not used
                        if constexpr (NG == 0) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int key = key0 + 2 * t + (j & 1) + 8 * (j >> 1);
                                if (key < it.klo || key >= it.khi)
                                    V[b].w[j][0] = V[b].w[j][1] = make_uint4(0u, 0u, 0u, 0u);
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const int key = key0 + r + 8 * j;
                                if (key < it.klo || key >= it.khi)
#pragma unroll
                                    for (int g = 0; g < GN; ++g) V[b].m[j][g] = 0u;
                            }
                        }
                    }
                }
            }
            // ---- running maximum: raised only when a row's passes it by 2^kLazy
            bool raise = false;
            float mx[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mx[nt][e] = fmaxf(x[0][nt][e], x[0][nt][e + 2]);
#pragma unroll
                    for (int b = 1; b < NB; ++b) mx[nt][e] = fmaxf(mx[nt][e], fmaxf(x[b][nt][e], x[b][nt][e + 2]));
                    mx[nt][e] *= ls;
                    raise |= mx[nt][e] > m_run[nt][e] + kLazy;
                }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = mx[nt][e];
#pragma unroll
                        for (int w = 4; w < 32; w <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
                        m = fmaxf(m, m_run[nt][e]);
                        const float f = m == -INFINITY ? 1.f : ex2(m_run[nt][e] - m);
                        m_run[nt][e] = m;
                        l_run[nt][e] *= f;
#pragma unroll
                        for (int g = 0; g < GN; ++g) corr[nt][e][g] *= f;
#pragma unroll
                        for (int d = 0; d < 8; ++d) {
                            o[nt][d][e] *= f;
                            o[nt][d][e + 2] *= f;
                        }
                    }
            }
            // ---- P and O^T += V^T P^T
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                if (kb + b >= kb_stop) continue;   // warp-uniform
                uint32_t pb[NT][GN][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float m0 = m_run[nt][0] == -INFINITY ? 0.f : m_run[nt][0];
                    const float m1 = m_run[nt][1] == -INFINITY ? 0.f : m_run[nt][1];
                    const float p0 = ex2(fmaf(x[b][nt][0], ls, -m0)), p1 = ex2(fmaf(x[b][nt][1], ls, -m1));
                    const float p2 = ex2(fmaf(x[b][nt][2], ls, -m0)), p3 = ex2(fmaf(x[b][nt][3], ls, -m1));
                    l_run[nt][0] += p0 + p2;
                    l_run[nt][1] += p1 + p3;
                    if constexpr (NG == 0) {
                        pb[nt][0][0] = transpose8(pack2(p0, p1));
                        pb[nt][0][1] = transpose8(pack2(p2, p3));
                    } else {
#pragma unroll
                        for (int g = 0; g < GN; ++g) {
                            const float2 s0 = so(V[b].m[0][g]), s1 = so(V[b].m[1][g]);
                            const float o0 = fmaf(8.f, s0.x, s0.y), o1 = fmaf(8.f, s1.x, s1.y);
                            corr[nt][0][g] = fmaf(p0, o0, fmaf(p2, o1, corr[nt][0][g]));
                            corr[nt][1][g] = fmaf(p1, o0, fmaf(p3, o1, corr[nt][1][g]));
                            pb[nt][g][0] = transpose8(pack2(p0 * s0.x, p1 * s0.x));
                            pb[nt][g][1] = transpose8(pack2(p2 * s1.x, p3 * s1.x));
                        }
                    }
                }
                if constexpr (NG == 0) {
#pragma unroll
                    for (int d = 0; d < 8; ++d) {
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint4 v = V[b].w[j][d >> 2];
                            w[j] = (d & 3) == 0 ? v.x : (d & 3) == 1 ? v.y : (d & 3) == 2 ? v.z : v.w;
                        }
                        const uint32_t a0 = __byte_perm(w[0], w[1], 0x5410), a1 = __byte_perm(w[0], w[1], 0x7632);
                        const uint32_t a2 = __byte_perm(w[2], w[3], 0x5410), a3 = __byte_perm(w[2], w[3], 0x7632);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816(o[nt][d], a0, a1, a2, a3, pb[nt][0][0], pb[nt][0][1]);
                    }
                } else {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {   // 32-dim blocks
                        const uint32_t sel = (g & 1) ? 0x7632 : 0x5410;
                        const uint32_t w0 = __byte_perm(g < 2 ? V[b].w[0].x : V[b].w[0].y,
                                                        g < 2 ? V[b].w[1].x : V[b].w[1].y, sel);
                        const uint32_t w1 = __byte_perm(g < 2 ? V[b].w[2].x : V[b].w[2].y,
                                                        g < 2 ? V[b].w[3].x : V[b].w[3].y, sel);
#pragma unroll
                        for (int s = 0; s < 2; ++s) {   // dims 32 g + 4 r + 2 s, + 1
                            const uint32_t a0 = centred(code_pair(w0 >> (8 * s)));
                            const uint32_t a1 = centred(code_pair(w0 >> (8 * s + 4)));
                            const uint32_t a2 = centred(code_pair(w1 >> (8 * s)));
                            const uint32_t a3 = centred(code_pair(w1 >> (8 * s + 4)));
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816(o[nt][2 * g + s], a0, a1, a2, a3, pb[nt][g * GN / 4][0],
                                         pb[nt][g * GN / 4][1]);
                        }
                    }
                }
            }
            load_v(next);
            fetch_ids(next + kWarps * NB);
        }

        // ---- join the warps: rows 2t, 2t + 1 of each tile
        const bool whole = n == it.units;
        const size_t slot = ((size_t)blockIdx.x * 2 + (first ? 0 : 1)) * a.tile_rows;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = l_run[nt][e];
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
                if (r == 0) {
                    sM[warp][8 * nt + 2 * t + e] = m_run[nt][e];
                    sL[warp][8 * nt + 2 * t + e] = l;
                }
                if constexpr (NG != 0) {
#pragma unroll
                    for (int g = 0; g < GN; ++g)
#pragma unroll
                        for (int w = 4; w < 32; w <<= 1)
                            corr[nt][e][g] += __shfl_xor_sync(0xffffffffu, corr[nt][e][g], w);
                }
            }
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int m = 8 * nt + 2 * t + e;
                float M = sM[0][m];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) M = fmaxf(M, sM[w][m]);
                const float f = m_run[nt][e] == -INFINITY ? 0.f : ex2(m_run[nt][e] - M);
                float* dst = sO[warp][2 * t + e];
                if constexpr (NG == 0) {   // dims 16 r + 2 d (+ 1)
#pragma unroll
                    for (int d = 0; d < 8; d += 2)
                        *reinterpret_cast<float4*>(dst + 16 * r + 2 * d) =
                            make_float4(o[nt][d][e] * f, o[nt][d][e + 2] * f, o[nt][d + 1][e] * f, o[nt][d + 1][e + 2] * f);
                } else {                   // dims 32 g + 4 r + 2 s (+ 1)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const float c = corr[nt][e][g * GN / 4];
                        *reinterpret_cast<float4*>(dst + 32 * g + 4 * r) =
                            make_float4((o[nt][2 * g][e] + c) * f, (o[nt][2 * g][e + 2] + c) * f,
                                        (o[nt][2 * g + 1][e] + c) * f, (o[nt][2 * g + 1][e + 2] + c) * f);
                    }
                }
            }
            __syncthreads();
            for (int x = threadIdx.x; x < 8 * 32; x += kThreads) {
                const int m = 8 * nt + x / 32, d = 4 * (x % 32);
                if (m >= rows) continue;
                float M = sM[0][m];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) M = fmaxf(M, sM[w][m]);
                float L = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float4 v = *reinterpret_cast<const float4*>(&sO[w][m & 7][d]);
                    acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
                    L += sM[w][m] == -INFINITY ? 0.f : sL[w][m] * ex2(sM[w][m] - M);
                }
                if (whole) {
                    const float inv = L > 0.f ? 1.0f / L : 0.f;
                    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) +
                                              (int64_t)(it.row0 + m / G) * a.out_stride +
                                              (int64_t)(h * G + m % G) * 128 + d) =
                        make_uint2(pack2(acc.x * inv, acc.y * inv), pack2(acc.z * inv, acc.w * inv));
                } else {
                    *reinterpret_cast<float4*>(a.part_o + (slot + m) * 128 + d) = acc;
                    if (d == 0) *reinterpret_cast<float2*>(a.part_ml + 2 * (slot + m)) = make_float2(M, L);
                }
            }
            __syncthreads();
        }
        first = false;
        u += n;
        off = 0;
        if (++h == H) {
            h = 0;
            if (u < u1) {
                do it = a.items[++i];
                while (it.units == 0);
            }
        }
    }
}

template <int NG, int NT, bool kExtra>
cudaError_t launch(const PagedAttn& a, cudaStream_t s) {
    constexpr int kCtas = paged_decode_ctas(NG != 0, NT);
    KVR_LAUNCH(paged_decode_kernel<NG, NT, kExtra, kCtas>, dim3((unsigned)a.n_cta), dim3(kThreads), 0, s, a);
    return cudaSuccess;
}
template <int NG>
cudaError_t launch_ng(const PagedAttn& a, cudaStream_t s) {
    const bool extra = a.softcap > 0.f || a.loc || a.snk || a.slopes;
    if (a.tile_rows == 8) return extra ? launch<NG, 1, true>(a, s) : launch<NG, 1, false>(a, s);
    return extra ? launch<NG, 2, true>(a, s) : launch<NG, 2, false>(a, s);
}

}  // namespace

int paged_decode_unit(int format) { return format == KVR_INT4 ? Decode<1, 1, false>::kUnit : Decode<0, 1, false>::kUnit; }

cudaError_t launch_paged_decode(int format, int group, const PagedAttn& a, cudaStream_t s) {
    if (format == KVR_BF16) return launch_ng<0>(a, s);
    if (group == 32) return launch_ng<4>(a, s);
    if (group == 64) return launch_ng<2>(a, s);
    return launch_ng<1>(a, s);
}

}  // namespace kvr
