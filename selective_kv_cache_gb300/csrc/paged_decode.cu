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
// come out of shared memory in the operand's own layout, without a
// transposing load, and no row is padded beyond 8.  Each warp copies its own
// 16-key blocks asynchronously into a ring of its own a few steps ahead, so
// the bytes in flight cost no registers and no warp waits for another.
//   K (rows = keys): lane (r, t) = (lane / 4, lane % 4) holds dims in 16-byte
//     chunks of keys r and r + 8; the contraction may take the dims in any
//     order as long as Q does, so the chunks are taken as they lie.
//   V (rows = dims): lane (r, t) holds 16 dims of keys 2t, 2t + 1, 2t + 8,
//     2t + 9; a byte permute of two keys' words makes the (key, key + 1) pairs.
//   P^T comes from S^T's accumulator by movmatrix (8x8 transposes).
// 4-bit pages, in fp16: a code under its mask is the fp16 subnormal c 2^-24
//   (16 c 2^-24 for the odd nibbles, whose q is divided by 16), which the mma
//   multiplies exactly, so K is one logic op per two values and adds no
//   rounding; scales are applied to S in fp32, the offsets' part sum_g o_g sum
//   q comes from one mma over the (scale, offset) words.  q is scaled by a
//   power of two per row to [128, 256) at its largest.  V is brought to its
//   value in fp16, s (c - 8) + (o + 8 s) in two packed FMAs (2^-11 relative), and P is fp16:
//   its smallest steps, 2^-25 of the running maximum's weight, are lost in sums
//   that are at least 1.
// The warps of a CTA take every kWarps-th run of keys, each with its own
// maximum, sum and output, joined through shared memory when the CTA is done
// with an (item, head).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged.h"
#include "ptx.cuh"

namespace kvr {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLazy = 8.0f;   // log2 of the largest P before the maximum is raised

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
__device__ __forceinline__ void mma16816h(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2h(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    const __half2 y = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b),
                              *reinterpret_cast<const __half2*>(&c));
    return *reinterpret_cast<const uint32_t*>(&y);
}
// (x & mask) | 0x6400 in both halves, one operation
__device__ __forceinline__ uint32_t with_1024(uint32_t x, uint32_t mask) {
    uint32_t y;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(y) : "r"(x), "r"(mask), "r"(0x64006400u));
    return y;
}
// code - 8 of the even and of the odd nibble of each half, exact
__device__ __forceinline__ uint32_t even8(uint32_t x) {   // (1024 + c) - 1032
    return hfma2(with_1024(x, 0x000f000fu), 0x3c003c00u, 0xe408e408u);
}
__device__ __forceinline__ uint32_t odd8(uint32_t x) {    // (1024 + 16 c) / 16 - 72
    return hfma2(with_1024(x, 0x00f000f0u), 0x2c002c00u, 0xd480d480u);
}
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const uint8_t* src) {
    if constexpr (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
// Scale-offset pairs of one row: NG words
template <int NG>
__device__ __forceinline__ void lds_meta(uint32_t a, uint32_t* m) {
    if constexpr (NG == 4) {
        const uint4 v = lds16(a);
        m[0] = v.x, m[1] = v.y, m[2] = v.z, m[3] = v.w;
    } else if constexpr (NG == 2) {
        const uint2 v = lds8(a);
        m[0] = v.x, m[1] = v.y;
    } else {
        m[0] = lds4(a);
    }
}
// A row's scale: finite and not zero, so that 0 and -inf stay what they are under it.
__device__ __forceinline__ float logit_scale(float sl2, float back) { return fminf(fmaxf(sl2 * back, 2e-38f), 2e38f); }
__device__ __forceinline__ float scale_of(uint32_t m) { return __low2float(*reinterpret_cast<const __half2*>(&m)); }

// NG: 0 = bf16 pages, else the scale groups of a 4-bit row.  NT: 8-row tiles of an item.
template <int NG, int NT>
struct Decode {
    static constexpr int NB = NG ? 2 : 1;            // 16-key blocks of a warp's step
    static constexpr int kUnit = 16 * NB * kWarps;
    static constexpr int RB = NG ? 64 : 256;         // bytes of a row
    static constexpr int GN = NG ? NG : 1;
    static constexpr int MB = NG ? 4 * NG : 0;       // bytes of a row's (scale, offset) pairs
    // a block in the ring: K rows, V rows, K pairs, V pairs
    static constexpr int kV = 16 * RB, kKm = 32 * RB, kVm = kKm + 16 * MB, kBlock = kVm + 16 * MB;
    static constexpr int kCtas = paged_decode_ctas(NG != 0, NT);
    static constexpr int kStages = 3;
    static constexpr int kRing = kStages * NB * kBlock;
    static constexpr int LDO = 132;                  // padded output row of the join
    static constexpr int kJoin = kWarps * 8 * LDO * 4;
    static constexpr int kSmem = kWarps * kRing > kJoin ? kWarps * kRing : kJoin;
};

// kExtra: cap, biases or slopes
template <int NG, int NT, bool kExtra>
__global__ void __launch_bounds__(kThreads, Decode<NG, NT>::kCtas) paged_decode_kernel(PagedAttn a) {
    using D = Decode<NG, NT>;
    constexpr int NB = D::NB, GN = D::GN, RB = D::RB, MB = D::MB, S = D::kStages;
    extern __shared__ __align__(128) uint8_t smem[];   // the warps' rings; the outputs to join over them
    float(*sO)[8][D::LDO] = reinterpret_cast<float(*)[8][D::LDO]>(smem);
    __shared__ float sM[kWarps][8 * NT], sL[kWarps][8 * NT];
    __shared__ PagedItem items[kPagedInline];
    pdl_wait();
    pdl_trigger();
    PagedShare sh;
    int u1;
    if (a.planned) {
        sh = a.shares[blockIdx.x];
        u1 = a.shares[blockIdx.x + 1].u0;
    } else {
        sh = paged_inline_share(a, items, &u1);
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
    const int G = a.G, shift = a.p.page_shift, in_page = (1 << shift) - 1;
    const float sl2 = a.scale * kLog2e;
    const PagedItem* all_items = a.planned ? a.items : items;
    const int slot_b = (int)a.p.slot_stride * RB, page_b = (int)a.p.page_stride * RB;   // below 2^31 (checked)
    const int slot_m = (int)a.p.slot_stride * MB, page_m = (int)a.p.page_stride * MB;
    const uint32_t ring = smem_u32(smem) + warp * D::kRing;
    // Where this lane's copies land in a block and where it reads.  A read
    // takes 8 lanes (16 bytes each) or 16 (8 bytes) at a time; rows and chunks
    // are placed so that those hit different banks.
    //   4 bits: K rows as they are.  V: lane (r, t) reads 8 bytes of keys
    //     2t + j: row (b3 b2 b1 b0) lies at (b3 b2 b0 b1), its 16-byte chunks
    //     exchanged by 2 b2.
    //   bf16: K chunk c of row r at c ^ 4 (r & 1); V chunk c of key k at
    //     c ^ ((c >> 1) & 1) ^ 2 ((k >> 1) & 3).
    const uint32_t k_put = NG ? 16 * lane : (lane >> 4) * 256 + 16 * ((lane & 15) ^ (4 * (lane >> 4)));
    const uint32_t v_put = NG ? ((r & 4) | ((r & 1) << 1) | ((r >> 1) & 1)) * 64 + 16 * (t ^ (2 * (r >> 2)))
                              : (lane >> 4) * 256 + 16 * ((lane & 15) ^ ((lane >> 1) & 1));
    const uint32_t k_get = NG ? 64 * r + 16 * t : 256 * r + 16 * (t ^ (4 * (r & 1)));
    const uint32_t v_get = D::kV + (NG ? (4 * (t >> 1) + (t & 1)) * 64 + 16 * ((r >> 1) ^ (2 * (t >> 1))) + 8 * (r & 1)
                                       : 512 * t + 16 * (2 * (r ^ t) + (r & 1)));

    for (PagedWalk run(a, sh, u1); run.live(); run.next(a, all_items)) {
        const PagedItem it = run.it;
        const int n = run.n, off = run.off, h = run.h;
        const int rows = it.rows * G;
        const int* table = a.p.table + (int64_t)it.seq * a.p.max_pages;
        // 16-key blocks [kb0, kb_end) hold the item's keys; this warp's steps
        // start at kb and go on kWarps * NB blocks at a time
        const int kb_first = it.klo >> 4, kb_end = (it.khi + 15) >> 4;
        int kb = (it.klo / D::kUnit + off) * (kWarps * NB) + warp * NB;
        const int kb_stop = min(kb_end, (it.klo / D::kUnit + off + n) * (kWarps * NB));

        // this lane's copies: rows of slot 0 of page 0
        const int64_t head = (int64_t)h * a.p.head_stride;
        const int copy_row = NG ? r : lane >> 4;
        const uint8_t* k_src = a.p.k + head * RB + (int64_t)copy_row * slot_b + (NG ? 16 * t : 16 * (lane & 15));
        const uint8_t* v_src = a.p.v + head * RB + (int64_t)copy_row * slot_b + (NG ? 16 * t : 16 * (lane & 15));
        const uint8_t* m_src = (lane < 16 ? a.p.ks : a.p.vs) + head * MB + (int64_t)(lane & 15) * slot_m;
        int pid[NB];           // page ids, one step ahead of the copies
        auto fetch_ids = [&](int k) {
#pragma unroll
            for (int x = 0; x < NB; ++x)
                pid[x] = k + x >= kb_first && k + x < kb_stop ? table[(k + x) >> (shift - 4)] : 0;
        };
        auto copy_step = [&](int k, uint32_t dst) {
#pragma unroll
            for (int x = 0; x < NB; ++x) {
                if (k + x < kb_stop) {   // warp-uniform
                    const int page = paged_id(a.p, pid[x]), at = ((k + x) << 4) & in_page;
                    const int64_t off_b = (int64_t)page * page_b + (int64_t)at * slot_b;
                    const uint32_t d = dst + x * D::kBlock;
                    constexpr int kRowsApart = NG ? 8 : 2;   // rows between a lane's copies
#pragma unroll
                    for (int c = 0; c < 16 / kRowsApart; ++c) {
                        const int64_t o = off_b + (int64_t)(c * kRowsApart) * slot_b;
                        copy_async<16>(d + k_put + c * kRowsApart * RB, k_src + o);
                        copy_async<16>(d + D::kV + (NG ? v_put : v_put ^ (32 * (c & 3))) + c * kRowsApart * RB,
                                       v_src + o);
                    }
                    if constexpr (NG != 0)
                        copy_async<MB>(d + D::kKm + lane * MB, m_src + (int64_t)page * page_m + (int64_t)at * slot_m);
                }
            }
            copy_commit();
        };
        if (kb + NB <= kb_first) kb += kWarps * NB;   // a first step wholly before klo
        fetch_ids(kb);
#pragma unroll
        for (int x = 0; x < S; ++x) {
            copy_step(kb + x * kWarps * NB, ring + x * NB * D::kBlock);
            fetch_ids(kb + (x + 1) * kWarps * NB);
        }

        // Q as the B operand: row n = 8 nt + r, this lane's dims; lsr: what turns
        // rows 2t, 2t + 1 of the products into base-2 logits
        uint32_t q[NT][16];
        uint32_t q_off[NT][2];     // 4 bits: the group sums of q, high and low part, against the offsets
        float lsr[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int m = 8 * nt + r;
            uint4 w[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                w[c] = make_uint4(0u, 0u, 0u, 0u);
                if (m < rows)
                    w[c] = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.q) +
                                                           (int64_t)(it.row0 + m / G) * a.q_stride +
                                                           (int64_t)(h * G + m % G) * 128 + 32 * c + 8 * t);
            }
            if constexpr (NG == 0) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    q[nt][4 * c] = w[c].x, q[nt][4 * c + 1] = w[c].y;
                    q[nt][4 * c + 2] = w[c].z, q[nt][4 * c + 3] = w[c].w;
                }
                lsr[nt][0] = lsr[nt][1] = sl2;
            } else {
                uint32_t top = 0u;   // largest exponent of the row
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t ws[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = max(top, max(ws[e] & 0x7f80u, (ws[e] >> 16) & 0x7f80u));
                }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int ex = min(max((int)(top >> 7), 8), 253);           // biased; q 2^(134 - ex) is below 256
                const float f = __uint_as_float((uint32_t)(261 - ex) << 23);
                const float back = __uint_as_float((uint32_t)(ex - 7) << 23);      // 2^(ex - 134)
                float sums[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t ws[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[2 * e] = __uint_as_float(ws[e] << 16) * f;
                        v[2 * e + 1] = __uint_as_float(ws[e] & 0xffff0000u) * f;
                    }
                    if constexpr (NG == 4) {   // pairs (dim e, dim e + 4) of block c, as its two units pair up
                        q[nt][4 * c] = pack2h(v[0], v[4]);
                        q[nt][4 * c + 1] = pack2h(v[1] * 0.0625f, v[5] * 0.0625f);
                        q[nt][4 * c + 2] = pack2h(v[2], v[6]);
                        q[nt][4 * c + 3] = pack2h(v[3] * 0.0625f, v[7] * 0.0625f);
                    } else {                   // pairs (block c, block c + 1): this block's half of each word
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint32_t hb = pack2h(v[e] * ((e & 1) ? 0.0625f : 1.f), 0.f) & 0xffffu;
                            uint32_t& dst = q[nt][8 * (c / 2) + e];
                            dst = (c & 1) ? dst | (hb << 16) : hb;
                        }
                    }
                    sums[c] = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
                    sums[c] += __shfl_xor_sync(0xffffffffu, sums[c], 1);
                    sums[c] += __shfl_xor_sync(0xffffffffu, sums[c], 2);
                }
                // lane t takes scale group t
                float own = NG == 4 ? (t == 0 ? sums[0] : t == 1 ? sums[1] : t == 2 ? sums[2] : sums[3])
                          : NG == 2 ? (t == 0 ? sums[0] + sums[1] : t == 1 ? sums[2] + sums[3] : 0.f)
                                    : (t == 0 ? (sums[0] + sums[1]) + (sums[2] + sums[3]) : 0.f);
                const float own_hi = __half2float(__float2half_rn(own));
                q_off[nt][0] = pack2h(0.f, own_hi);
                q_off[nt][1] = pack2h(0.f, own - own_hi);
                lsr[nt][0] = logit_scale(sl2, __shfl_sync(0xffffffffu, back, 8 * t));
                lsr[nt][1] = logit_scale(sl2, __shfl_sync(0xffffffffu, back, 8 * t + 4));
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

        float o[NT][8][4], m_run[NT][2], l_run[NT][2];
        float m_neg[NT][2];        // -m_run, 0 before the first key
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int d = 0; d < 8; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][d][e] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m_run[nt][e] = -INFINITY;
                m_neg[nt][e] = 0.f;
                l_run[nt][e] = 0.f;
            }
        }

        uint32_t stage = ring;
        for (; kb < kb_stop; kb += kWarps * NB) {
            copy_wait<S - 1>();
            __syncwarp();
            // ---- scores S^T of the step's keys
            float x[NB][NT][4];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const uint32_t at = stage + b * D::kBlock;
                uint4 kw[2][NG ? 1 : 4];
                uint32_t km[2][GN];
                if constexpr (NG == 0) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        kw[0][c] = lds16(at + (k_get ^ (64 * c)));
                        kw[1][c] = lds16(at + (k_get ^ (64 * c)) + 8 * RB);
                    }
                } else {
                    kw[0][0] = lds16(at + k_get);
                    kw[1][0] = lds16(at + k_get + 8 * RB);
                    lds_meta<NG>(at + D::kKm + r * MB, km[0]);
                    lds_meta<NG>(at + D::kKm + (r + 8) * MB, km[1]);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if constexpr (NG == 0) {
                        float c0[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint4 p = kw[0][c], s = kw[1][c];
                            mma16816(c0, p.x, s.x, p.y, s.y, q[nt][4 * c], q[nt][4 * c + 1]);
                            mma16816(c1, p.z, s.z, p.w, s.w, q[nt][4 * c + 2], q[nt][4 * c + 3]);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[b][nt][e] = c0[e] + c1[e];
                    } else {
                        const uint4 p = kw[0][0], s = kw[1][0];
                        // NG = 4: the units of one 32-dim block from the lane's two
                        // chunks; else a word's two units share their scale
                        const uint32_t ph[4] = {NG == 4 ? __byte_perm(p.x, p.z, 0x5410) : p.x,
                                                NG == 4 ? __byte_perm(p.x, p.z, 0x7632) : p.z,
                                                NG == 4 ? __byte_perm(p.y, p.w, 0x5410) : p.y,
                                                NG == 4 ? __byte_perm(p.y, p.w, 0x7632) : p.w};
                        const uint32_t sh_[4] = {NG == 4 ? __byte_perm(s.x, s.z, 0x5410) : s.x,
                                                 NG == 4 ? __byte_perm(s.x, s.z, 0x7632) : s.z,
                                                 NG == 4 ? __byte_perm(s.y, s.w, 0x5410) : s.y,
                                                 NG == 4 ? __byte_perm(s.y, s.w, 0x7632) : s.w};
                        constexpr uint32_t kEven = 0x000f000fu, kOdd = 0x00f000f0u;
                        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int g = 0; g < GN; ++g) {
                            float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int j = g * (4 / GN); j < (g + 1) * (4 / GN); ++j) {
                                const uint32_t p8 = ph[j] >> 8, s8 = sh_[j] >> 8;
                                mma16816h(c, ph[j] & kEven, sh_[j] & kEven, ph[j] & kOdd, sh_[j] & kOdd, q[nt][4 * j],
                                          q[nt][4 * j + 1]);
                                mma16816h(c, p8 & kEven, s8 & kEven, p8 & kOdd, s8 & kOdd, q[nt][4 * j + 2],
                                          q[nt][4 * j + 3]);
                            }
                            const float s0 = scale_of(km[0][g]), s1 = scale_of(km[1][g]);
                            sum[0] = fmaf(s0, c[0], sum[0]);
                            sum[1] = fmaf(s0, c[1], sum[1]);
                            sum[2] = fmaf(s1, c[2], sum[2]);
                            sum[3] = fmaf(s1, c[3], sum[3]);
                        }
                        uint32_t w0 = km[0][0], w1 = km[1][0];   // lane t: the words of group t
                        if constexpr (NG == 2) {
                            w0 = (t & 1) ? km[0][1] : w0;
                            w1 = (t & 1) ? km[1][1] : w1;
                        } else if constexpr (NG == 4) {
                            w0 = (t & 2) ? ((t & 1) ? km[0][3] : km[0][2]) : ((t & 1) ? km[0][1] : w0);
                            w1 = (t & 2) ? ((t & 1) ? km[1][3] : km[1][2]) : ((t & 1) ? km[1][1] : w1);
                        }
                        float c[4] = {0.f, 0.f, 0.f, 0.f};
                        mma16816h(c, w0, w1, w0, w1, q_off[nt][0], q_off[nt][1]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[b][nt][e] = fmaf(sum[e], 16777216.f, c[e]);
                    }
                }
            }
            // ---- logits in base 2
            if (kExtra) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[b][nt][e] *= lsr[nt][e & 1];
                if (a.softcap > 0.f) {
                    const float cap_out = a.softcap * kLog2e, cap_in = 1.f / cap_out;
                    auto capped = [&](auto f) {
#pragma unroll
                        for (int b = 0; b < NB; ++b)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; e += 2) {
                                    const float2 y = f(make_float2(x[b][nt][e], x[b][nt][e + 1]));
                                    x[b][nt][e] = y.x * cap_out, x[b][nt][e + 1] = y.y * cap_out;
                                }
                    };
                    if (a.softcap <= kCapQuotient) {
                        const float in_q = cap_in * kTwoLog2e;
                        capped([=](float2 y) {
                            return make_float2(tanh_quotient(y.x * in_q), tanh_quotient(y.y * in_q));
                        });
                    } else {
                        capped([=](float2 y) { return tanh_either(make_float2(y.x * cap_in, y.y * cap_in)); });
                    }
                }
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
                            const int key = 16 * (kb + b) + r + 8 * (e >> 1);
                            x[b][nt][e] = fmaf(-slope[nt][e & 1], (float)abs(gpos[nt][e & 1] - key),
                                               x[b][nt][e] + bias[e >> 1]);
                        }
                }
            }
            // warp-uniform: some row does not see some of the step's keys
            const bool partial = 16 * kb < all_lo || 16 * (kb + NB) > all_hi;
            if (partial) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = 16 * (kb + b) + r + 8 * (e >> 1);
                            if (key < lo[nt][e & 1] || key >= hi[nt][e & 1]) x[b][nt][e] = -INFINITY;
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
                    if (!kExtra) mx[nt][e] *= lsr[nt][e];
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
                        m_neg[nt][e] = m == -INFINITY ? 0.f : -m;
                        l_run[nt][e] *= f;
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
                uint32_t pb[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float m0 = m_neg[nt][0], m1 = m_neg[nt][1];
                    const float f0 = kExtra ? 1.f : lsr[nt][0], f1 = kExtra ? 1.f : lsr[nt][1];
                    const float p0 = ex2(fmaf(x[b][nt][0], f0, m0)), p1 = ex2(fmaf(x[b][nt][1], f1, m1));
                    const float p2 = ex2(fmaf(x[b][nt][2], f0, m0)), p3 = ex2(fmaf(x[b][nt][3], f1, m1));
                    l_run[nt][0] += p0 + p2;
                    l_run[nt][1] += p1 + p3;
                    pb[nt][0] = transpose8(NG ? pack2h(p0, p1) : pack2(p0, p1));
                    pb[nt][1] = transpose8(NG ? pack2h(p2, p3) : pack2(p2, p3));
                }
                // keys nobody sees: whatever their slots hold is not used
                const int key0 = 16 * (kb + b);
                const uint32_t at = stage + b * D::kBlock;
                auto unseen = [&](int j) {
                    const int key = key0 + 2 * t + (j & 1) + 8 * (j >> 1);
                    return key < it.klo || key >= it.khi;
                };
                if constexpr (NG == 0) {
                    uint4 vw[4][2];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t p = at + v_get + (j & 1) * RB + (j >> 1) * 8 * RB;
                        vw[j][0] = lds16(p);
                        vw[j][1] = lds16(p ^ 16u);
                    }
                    if (partial) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (unseen(j)) vw[j][0] = vw[j][1] = make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int d = 0; d < 8; ++d) {
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint4 v = vw[j][d >> 2];
                            w[j] = (d & 3) == 0 ? v.x : (d & 3) == 1 ? v.y : (d & 3) == 2 ? v.z : v.w;
                        }
                        const uint32_t a0 = __byte_perm(w[0], w[1], 0x5410), a1 = __byte_perm(w[0], w[1], 0x7632);
                        const uint32_t a2 = __byte_perm(w[2], w[3], 0x5410), a3 = __byte_perm(w[2], w[3], 0x7632);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816(o[nt][d], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                    }
                } else {
                    uint2 vw[4];
                    uint32_t vm[4][GN];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        vw[j] = lds8(at + v_get + (j & 1) * 128 + (j >> 1) * 512);
                        lds_meta<NG>(at + D::kVm + (2 * t + (j & 1) + 8 * (j >> 1)) * MB, vm[j]);
                    }
                    if (partial) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (unseen(j))
#pragma unroll
                                for (int g = 0; g < GN; ++g) vm[j][g] = 0u;
                    }
#pragma unroll
                    for (int g = 0; g < 4; ++g) {   // 32-dim blocks
                        const uint32_t sel = (g & 1) ? 0x7632 : 0x5410;
                        const int n = g * GN / 4;   // its scale group
                        uint32_t v[2][4];           // (key, key + 1) pairs of dims 32 g + 4 r + d
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t w = __byte_perm(g < 2 ? vw[2 * j].x : vw[2 * j].y,
                                                           g < 2 ? vw[2 * j + 1].x : vw[2 * j + 1].y, sel);
                            const uint32_t s = __byte_perm(vm[2 * j][n], vm[2 * j + 1][n], 0x5410);
                            const uint32_t o8 =
                                hfma2(s, 0x48004800u, __byte_perm(vm[2 * j][n], vm[2 * j + 1][n], 0x7632));
                            v[j][0] = hfma2(even8(w), s, o8);
                            v[j][1] = hfma2(odd8(w), s, o8);
                            v[j][2] = hfma2(even8(w >> 8), s, o8);
                            v[j][3] = hfma2(odd8(w >> 8), s, o8);
                        }
#pragma unroll
                        for (int d = 0; d < 4; d += 2)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816h(o[nt][2 * g + d / 2], v[0][d], v[0][d + 1], v[1][d], v[1][d + 1], pb[nt][0],
                                          pb[nt][1]);
                    }
                }
            }
            __syncwarp();   // every lane has read the stage
            copy_step(kb + S * kWarps * NB, stage);
            fetch_ids(kb + (S + 1) * kWarps * NB);
            stage = stage == ring + (S - 1) * NB * D::kBlock ? ring : stage + NB * D::kBlock;
        }
        copy_wait<0>();
        __syncthreads();   // the join's outputs lie over every warp's ring

        // ---- join the warps: rows 2t, 2t + 1 of each tile
        const bool whole = run.whole();
        const size_t slot = ((size_t)blockIdx.x * 2 + (run.first ? 0 : 1)) * a.tile_rows;
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
                            make_float4(o[nt][d][e] * f, o[nt][d][e + 2] * f, o[nt][d + 1][e] * f,
                                        o[nt][d + 1][e + 2] * f);
                } else {                   // dims 32 g + 4 r + 2 s (+ 1)
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        *reinterpret_cast<float4*>(dst + 32 * g + 4 * r) =
                            make_float4(o[nt][2 * g][e] * f, o[nt][2 * g][e + 2] * f, o[nt][2 * g + 1][e] * f,
                                        o[nt][2 * g + 1][e + 2] * f);
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
    }
}

template <int NG, int NT, bool kExtra>
cudaError_t launch(const PagedAttn& a, cudaStream_t s) {
    constexpr int kSmem = Decode<NG, NT>::kSmem;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(paged_decode_kernel<NG, NT, kExtra>, kSmem, &allowed);
    if (e != cudaSuccess) return e;
    KVR_LAUNCH(paged_decode_kernel<NG, NT, kExtra>, dim3((unsigned)a.n_cta), dim3(kThreads), kSmem, s, a);
    return cudaSuccess;
}
template <int NG>
cudaError_t launch_ng(const PagedAttn& a, cudaStream_t s) {
    const bool extra = a.softcap > 0.f || a.loc || a.snk || a.slopes;
    if (a.tile_rows == 8) return extra ? launch<NG, 1, true>(a, s) : launch<NG, 1, false>(a, s);
    return extra ? launch<NG, 2, true>(a, s) : launch<NG, 2, false>(a, s);
}

}  // namespace

int paged_decode_unit(int format) { return format == KVR_INT4 ? Decode<1, 1>::kUnit : Decode<0, 1>::kUnit; }

cudaError_t launch_paged_decode(int format, int group, const PagedAttn& a, cudaStream_t s) {
    if (format == KVR_BF16) return launch_ng<0>(a, s);
    if (group == 32) return launch_ng<4>(a, s);
    if (group == 64) return launch_ng<2>(a, s);
    return launch_ng<1>(a, s);
}

}  // namespace kvr
