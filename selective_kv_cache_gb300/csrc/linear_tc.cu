// linear_tc.cu -- projection of many 8-bit rows on the sm_103a tensor cores:
//   y[r][f] = s_r t_f sum_k a[r][k] w[f][k] + bias[f]
//
// This GPU's integer tensor rate is a small part of its fp16 one, and 8-bit
// integers are exact in fp16, as are their products in the fp32 accumulator:
// so the products run as fp16 (kind::f16) on operands that are widened on the
// way.  The weights, which are read once, stay in eight bits up to the SM and
// are widened there; the rows, which every feature tile reads again, are
// widened once into the workspace by a small kernel before this one.
//
// Two CTAs (a cluster) work on one tile of 256 features by up to 256 rows with
// paired products (cta_group::2): each holds 128 features of the weights and
// half of the rows, so the rows' tile crosses shared memory half as often.
// The widened weights are the A operand in tensor memory: written once with
// tcgen05.st, they never return through shared memory, whose port the rows'
// tile needs.
//   warp 0       TMA: per stage 128 features x 128 codes and N/2 rows x 128
//                fp16 (two swizzle atoms)
//   warp 1       products, in the leader CTA: four of K = 16 a 64-code chunk
//   warps 4-11   accumulators out, two warps a TMEM lane quarter
//   warps 12-27  widening: four sets of four warps take the 64-code chunks in turn,
//                a thread a feature.  A chunk takes a set about 800 cycles, most of them
//                latency, so four of them keep up with the copies.
// Barriers: full (copies landed, own CTA) -> widening warps of both CTAs ->
// a_ready (leader) -> products -> a_free, empty (both CTAs).  That the peer's
// rows have landed the issuing thread knows from the peer's widening warps,
// which wait for the same stage.
//
// Tensor memory: accumulators of two tiles (side by side up to N = 192; above,
// they share columns, which the epilogue reads first), and four chunks of widened
// weights behind them, eight up to N = 128.
//
// Work: pairs take whole tiles in turn.  The tiles that are left after the last
// whole turn, or all of them where there are few, may be split: a cluster then
// holds several pairs, each takes its part of k, writes it to the workspace as
// fp32, and the cluster's CTAs add the parts as integers, a share of the rows
// each, as soon as all have arrived on their barriers.  How many pairs a
// cluster has, and how wide a tile is, go by a model of the time (make_plan).
// Every wait is bounded.
#include <algorithm>

#include "linear.cuh"
#include "ptx.cuh"

namespace kvr {
namespace {

constexpr int kSets = 4, kOuts = 2;                // sets of widening warps; warps a lane quarter that write out
constexpr int kThreads = 32 * (4 + 4 * kOuts + 4 * kSets);
static_assert(kSets == 4, "two sets take the halves of every other stage");
constexpr int kStageK = 128;                      // codes of a stage: two chunks
constexpr uint32_t kStageA = 128 * 128;           // 128 features x 128 bytes
constexpr int kSmemMost = 227 * 1024;
constexpr int kSuper = 8;                         // row tiles that are walked beside one another

struct LinearTc {
    Linear a;
    int out_as, vec;
    float* part;            // [split tile][split][N][256]
    int N, m_tiles, n_tiles, KB, stages;
    int whole, rest;        // tiles taken whole, tiles split
    int split, clusters;    // pairs of a cluster, clusters of the grid
    uint32_t base1;         // columns of the second accumulator
    int shared_cols;        // whether the two share columns
    uint32_t col_a, slots;  // widened chunks: their first column and their number, 4 or 8
};

// ---------------------------------------------------------------- paired instructions
// One arrival on the leader CTA's barrier at this offset.  What it tells of are
// tensor memory's contents, ordered by the tcgen05 fences, and copies that have
// landed; nothing in ordinary memory is handed over, so neither side names the
// cluster's scope: with .release.cluster and .acquire.cluster a stage took 2500 cycles, the
// fences' round trips, in place of 1400.
__device__ __forceinline__ void arrive_leader(uint64_t* bar, uint32_t leader) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(peer_address(bar, leader)) : "memory");
}
// One arrival on another CTA's barrier that hands over what this warp wrote to
// the workspace, and the wait for it.
__device__ __forceinline__ void arrive_release(uint64_t* bar, uint32_t rank) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(peer_address(bar, rank)) : "memory");
}
__device__ __forceinline__ bool warp_wait_acquire(uint64_t* bar, uint32_t parity) {
    uint32_t ok = 0;
    const long long t0 = clock64();
    do {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
    } while (!ok && clock64() - t0 <= kWaitLimitCycles);
    return __all_sync(0xffffffffu, ok != 0) != 0;
}
__device__ __forceinline__ bool try_wait_pair(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// A barrier that the other CTA's threads or products arrive on; the whole warp gets the answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
    bool ok = try_wait_pair(bar, parity);
    if (!ok) {
        const long long t0 = clock64();
        while (!(ok = try_wait_pair(bar, parity)) && clock64() - t0 <= kWaitLimitCycles) {
        }
    }
    return __all_sync(0xffffffffu, ok) != 0;
}
__device__ __forceinline__ void pair_alloc(uint32_t* slot) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_dealloc(uint32_t taddr) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(taddr) : "memory");
}
// D (+)= A[tmem of both CTAs] B[smem of both]^T, fp16, K = 16
__device__ __forceinline__ void pair_mma(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// arrive on both CTAs' barriers at this offset when the products issued so far are done
__device__ __forceinline__ void pair_commit(uint64_t* bar, uint32_t leader) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)(3u << leader))
        : "memory");
}

// ---------------------------------------------------------------- work
// A pair's work in order: whole tiles, then its parts of split ones.
struct Piece {
    int tile, kb0, kb1, rest;   // rest: number of the split tile, or below 0
};
struct Walk {
    int next, pair, cluster, part;
    __device__ __forceinline__ Walk(const LinearTc& g, int id)
        : next(id), pair(id), cluster(id / g.split), part(id - id / g.split * g.split) {}
    __device__ __forceinline__ bool take(const LinearTc& g, Piece* p) {
        if (next < g.whole) {
            *p = Piece{next, 0, g.KB, -1};
            next += g.split * g.clusters;
            return true;
        }
        if (cluster >= g.rest) return false;
        *p = Piece{g.whole + cluster, g.KB * part / g.split, g.KB * (part + 1) / g.split, cluster};
        cluster += g.clusters;
        return true;
    }
};
// Tiles in order: groups of kSuper row tiles, in a group feature tile by feature tile.
__device__ __forceinline__ void tile_coords(const LinearTc& g, int tile, int* m, int* n) {
    const int sg = tile / (g.m_tiles * kSuper), n0 = sg * kSuper, w = min(kSuper, g.n_tiles - n0);
    const int i = tile - n0 * g.m_tiles;
    *m = i / w;
    *n = n0 + i - *m * w;
}

// ---------------------------------------------------------------- widening
// rows of codes to rows of fp16, `pitch` elements apart
__global__ void __launch_bounds__(256) widen_kernel(const int8_t* x, int64_t stride, __half* out, int pitch, int k, int n_rows) {
    pdl_trigger();
    const int per = (k + 15) / 16;
    for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < (int64_t)n_rows * per; t += (int64_t)gridDim.x * 256) {
        const int64_t r = t / per;
        const int i = (int)(t - r * per) * 16;
        const int8_t* p = x + r * stride + i;
        __half* o = out + r * pitch + i;
        if (i + 16 <= k) {
            uint32_t h[8];
            widen16(*reinterpret_cast<const uint4*>(p), h);
            reinterpret_cast<uint4*>(o)[0] = make_uint4(h[0], h[1], h[2], h[3]);
            reinterpret_cast<uint4*>(o)[1] = make_uint4(h[4], h[5], h[6], h[7]);
        } else {
            for (int e = 0; i + e < k; ++e) o[e] = __int2half_rn(p[e]);
        }
    }
}

// ---------------------------------------------------------------- output
// A lane holds its feature, a column is a row of the output.
__device__ __forceinline__ void write_part(float* o, const float* v, int left) {
    if (left >= 32) {
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i * 256] = v[i];
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < left) o[i * 256] = v[i];
    }
}
__global__ void __launch_bounds__(kThreads) linear_tc_kernel(const __grid_constant__ CUtensorMap tmA,
                                                            const __grid_constant__ CUtensorMap tmB,
                                                            const __grid_constant__ LinearTc g) {
    extern __shared__ uint8_t smem_raw[];
    // the same offset in both CTAs: dynamic shared memory begins at one address in all of a grid's blocks
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int stages = g.stages;
    const uint32_t half_rows = g.N / 2, atomB = half_rows * 128, stage_bytes = kStageA + 2 * atomB;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + (size_t)stages * stage_bytes);
    uint64_t* empty = full + stages;
    uint64_t* a_ready = empty + stages;   // [slots], the leader's
    uint64_t* a_free = a_ready + 8;       // [slots]
    uint64_t* acc_full = a_free + 8;      // [2]
    uint64_t* acc_empty = acc_full + 2;   // [2], the leader's
    uint64_t* cols_free = acc_empty + 2;  // the leader's: the columns that both accumulators use are read
    uint64_t* all_done = cols_free + 1;
    uint64_t* joined = all_done + 1;      // the cluster's parts of a split tile, of this CTA's features, are written
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(joined + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank(), leader = rank & ~1u, half = rank & 1u;   // half: of the tile's features and rows
    const int pair = blockIdx.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int t = 0; t < 8; ++t) {
            mbar_init(&a_ready[t], 8);
            mbar_init(&a_free[t], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 8 * kOuts);
        }
        mbar_init(cols_free, 8 * kOuts);
        mbar_init(all_done, 1);
        mbar_init(joined, 4 * kOuts * g.split);
        fence_mbar_init();
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
    }
    if (warp == 1) pair_alloc(tmem_slot);
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // the other CTA's barriers are initialised
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t slots = g.slots, lap = slots == 8 ? 3 : 2;   // chunk q: slot q % slots, its use number q >> lap
    bool ok = true;
    pdl_trigger();

    if (warp == 0) {
        // ------------------------------------------------------------ copies
        if (lane == 0) {
            auto load_a = [&](int s, int m, int kb) {
                tma_load_2d(smem + (size_t)s * stage_bytes, &tmA, &full[s], kb * kStageK, m * 256 + (int)half * 128);
            };
            // no kernel of the call writes the weights: the ring's first ones go out before the wait for the rows
            int pre = 0;
            Piece p;
            int m, n;
            for (Walk w(g, pair); pre < stages && w.take(g, &p);) {
                tile_coords(g, p.tile, &m, &n);
                for (int kb = p.kb0; kb < p.kb1 && pre < stages; ++kb, ++pre) {
                    mbar_arrive_expect_tx(&full[pre], stage_bytes);
                    load_a(pre, m, kb);
                }
            }
            pdl_wait();
            int it = 0, s = 0;
            uint32_t phase = 1;
            for (Walk w(g, pair); ok && w.take(g, &p);) {
                tile_coords(g, p.tile, &m, &n);
                for (int kb = p.kb0; kb < p.kb1; ++kb, ++it) {
                    if (it >= pre) {
                        if (!mbar_wait(&empty[s], phase)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(&full[s], stage_bytes);
                        load_a(s, m, kb);
                    }
                    uint8_t* b = smem + (size_t)s * stage_bytes + kStageA;
                    tma_load_2d(b, &tmB, &full[s], kb * kStageK, n * g.N + (int)(half * half_rows));
                    tma_load_2d(b + atomB, &tmB, &full[s], kb * kStageK + 64, n * g.N + (int)(half * half_rows));
                    if (++s == stages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) {   // let every copy still in flight land before the CTA exits
                for (int i = (it > stages ? it - stages : 0); i < it; ++i)
                    mbar_wait(&full[i % stages], (uint32_t)(i / stages) & 1u);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        const bool issuer = elect_one();
        if (half == 0) {
            const uint32_t idesc = (1u << 4) | ((uint32_t)(g.N >> 3) << 17) | ((256u >> 4) << 24);   // fp16, fp32 sums
            const uint64_t descB = sdesc_sw128(smem_u32(smem) + kStageA, 16, 1024);
            int s = 0, local = 0;
            uint32_t q = 0;
            Piece p;
            for (Walk w(g, pair); ok && w.take(g, &p); ++local) {
                const int ab = local & 1;
                if (!warp_wait(&acc_empty[ab], ((uint32_t)(local >> 1) & 1u) ^ 1u) ||
                    (g.shared_cols && local > 0 && !warp_wait(cols_free, (uint32_t)(local - 1) & 1u))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + (ab ? g.base1 : 0u);
                for (int kb = p.kb0; kb < p.kb1; ++kb) {
                    const uint64_t db = descB + (uint64_t)(((uint32_t)s * stage_bytes) >> 4);
#pragma unroll
                    for (uint32_t h = 0; h < 2; ++h, ++q) {
                        const uint32_t t = q & (slots - 1);
                        if (!warp_wait(&a_ready[t], (q >> lap) & 1u)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (issuer) {
#pragma unroll
                            for (uint32_t kk = 0; kk < 4; ++kk)
                                pair_mma(d, tmem + g.col_a + 32 * t + 8 * kk, db + (uint64_t)((h * atomB >> 4) + 2 * kk), idesc,
                                         (h > 0 || kk > 0) ? 1u : (kb > p.kb0 ? 1u : 0u));
                            pair_commit(&a_free[t], leader);
                            if (h == 1) pair_commit(&empty[s], leader);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    if (++s == stages) s = 0;
                }
                if (!ok) break;
                if (issuer) pair_commit(&acc_full[ab], leader);
                __syncwarp();
            }
            if (issuer) pair_commit(all_done, leader);
            __syncwarp();
        }
        if (!warp_wait(all_done, 0)) ok = false;
    } else if (warp >= 4 + 4 * kOuts) {
        // ------------------------------------------------------------ widening
        const int set = (warp - 4 - 4 * kOuts) >> 2, chunk = set & 1, quarter = warp & 3, row = 32 * quarter + lane;
        const uint32_t dst = tmem + ((uint32_t)(32 * quarter) << 16) + g.col_a;
        int s = 0, turn = set >> 1, pending = -1;   // this set's stages: every kSets / 2-th
        uint32_t phase = 0, q = set;
        // A chunk is handed over when the next one's codes are in registers, so that its stores complete meanwhile,
        // or at once where those have not come yet.
        auto hand_over = [&]() {
            if (pending < 0) return;
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_leader(&a_ready[pending], leader);
            pending = -1;
        };
        Piece p;
        for (Walk w(g, pair); ok && w.take(g, &p);) {
            for (int kb = p.kb0; kb < p.kb1; ++kb) {
                const int stage = s;
                const uint32_t parity = phase;
                if (++s == stages) {
                    s = 0;
                    phase ^= 1u;
                }
                if (turn-- != 0) continue;
                turn = kSets / 2 - 1;
                const uint32_t t = q & (slots - 1);
                if (!__all_sync(0xffffffffu, mbar_test(&full[stage], parity))) {
                    hand_over();
                    if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], parity))) {
                        ok = false;
                        break;
                    }
                }
                const uint8_t* a = smem + (size_t)stage * stage_bytes + row * 128;
                uint32_t h[32];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    widen16(*reinterpret_cast<const uint4*>(a + (((4 * chunk + c) ^ (row & 7)) << 4)), h + 8 * c);
                hand_over();
                if (!warp_wait(&a_free[t], ((q >> lap) & 1u) ^ 1u)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                tmem_st16_async(dst + 32 * t, h);
                tmem_st16_async(dst + 32 * t + 16, h + 16);
                pending = (int)t;
                q += kSets;
            }
        }
        hand_over();
    } else if (warp >= 4) {
        // ------------------------------------------------------------ accumulators out
        const int part = (warp - 4) >> 2, quarter = warp & 3, fo = (int)half * 128 + quarter * 32 + lane;   // this lane's feature in the tile
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        int local = 0, splits = 0;
        Piece p;
        for (Walk w(g, pair); w.take(g, &p); ++local) {
            const int ab = local & 1;
            int m, n;
            tile_coords(g, p.tile, &m, &n);
            const int row0 = n * g.N, f = m * 256 + fo, rows = min(g.N, g.a.n_rows - row0);
            const float sw = f < g.a.n_out ? g.a.w_scale[f] : 0.f, bias = f < g.a.n_out && g.a.bias ? g.a.bias[f] : 0.f;
            if (!warp_wait(&acc_full[ab], (uint32_t)(local >> 1) & 1u)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t src = tmem + lane_base + (ab ? g.base1 : 0u);
            float* tile_parts = g.part + (size_t)max(p.rest, 0) * g.split * g.N * 256;   // [split][N][256]
            float* mine = tile_parts + (size_t)w.part * g.N * 256;
            auto drain = [&](int lo, int hi) {
                for (int c = lo + 32 * part; c < hi; c += 32 * kOuts) {
                    const float sx = c + lane < rows ? g.a.x_scale[row0 + c + lane] : 0.f;
                    float v[32];
                    tmem_ld32(src + (uint32_t)c, v);
                    const int left = rows - c;
                    if (p.rest >= 0) write_part(mine + c * 256 + fo, v, left);
                    else write32(g.a, g.out_as, row0 + c, f, v, sx, sw, bias, left);
                }
            };
            if (g.shared_cols) {   // the columns that the next tile's accumulator shares first
                const int lo = ab ? 0 : (int)g.base1, hi = ab ? g.N - (int)g.base1 : g.N;
                drain(lo, hi);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_leader(cols_free, leader);
                drain(0, lo);
                drain(hi, g.N);
            } else {
                drain(0, g.N);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_leader(&acc_empty[ab], leader);
            if (p.rest < 0) continue;
            // the parts of this CTA's features, a share of the rows: a row a warp, four features a lane
            if (lane < g.split) arrive_release(joined, 2 * lane + half);
            const int f4 = m * 256 + (int)half * 128 + 4 * lane;
            const int c1 = min(rows, g.N * (w.part + 1) / g.split);
            float sw4[4], bias4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sw4[i] = f4 + i < g.a.n_out ? g.a.w_scale[f4 + i] : 0.f;
                bias4[i] = f4 + i < g.a.n_out && g.a.bias ? g.a.bias[f4 + i] : 0.f;
            }
            if (!warp_wait_acquire(joined, (uint32_t)(splits++) & 1u)) {
                ok = false;
                break;
            }
            for (int c = g.N * w.part / g.split + (warp - 4); c < c1; c += 4 * kOuts) {
                const float* from = tile_parts + c * 256 + half * 128 + 4 * lane;
                float4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < g.split) v[i] = __ldcg(reinterpret_cast<const float4*>(from + (size_t)i * g.N * 256));
                const float sx = g.a.x_scale[row0 + c];
                int sum[4] = {0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < g.split) {
                        sum[0] += __float2int_rn(v[i].x);
                        sum[1] += __float2int_rn(v[i].y);
                        sum[2] += __float2int_rn(v[i].z);
                        sum[3] += __float2int_rn(v[i].w);
                    }
                float y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = (float)sum[i] * sx * sw4[i] + bias4[i];
                write4(g.a, g.vec, row0 + c, f4, y);
            }
        }
    }
    if (!ok) atomicOr(g.a.err, DEV_ERR_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // no product or arrival of the pair is on its way any more
    if (warp == 1) {
        tc_fence_after();
        pair_dealloc(tmem);
    }
}

// Clusters of 1, 2, 3 and 4 pairs that a GB300 holds at once, one CTA an SM
// (cudaOccupancyMaxActiveClusters): its GPCs are not multiples of a cluster.
constexpr int kClusters[5] = {0, 76, 36, 23, 15};

struct Plan {
    int N, m_tiles, n_tiles, KB, stages, whole, rest, split, clusters, pitch;
    size_t rows_bytes, part_bytes;
};
// The width of a tile and the pairs of a cluster that take the shortest time in
// cycles: a stage of 128 codes takes its products' 4 N, or what copying and
// widening the weights take; a tile's end stops the products of a
// wide one while shared columns are read; a split tile's parts are joined.
Plan make_plan(int n_out, int k, int n_rows) {
    Plan best{};
    double least = 1e300;
    for (int N = 32; N <= 256; N += 32) {
        for (int split = 1; split <= 4; ++split) {
            Plan p{};
            p.N = N;
            p.split = split;
            p.m_tiles = (n_out + 255) / 256;
            p.n_tiles = (n_rows + N - 1) / N;
            p.KB = (k + kStageK - 1) / kStageK;
            if (split > p.KB || (N > 32 && N - 32 >= n_rows)) continue;
            const long long tiles = (long long)p.m_tiles * p.n_tiles;
            const int pairs = split * kClusters[split];
            p.whole = split == 1 ? (int)tiles : (int)(tiles / pairs * pairs);
            p.rest = (int)(tiles - p.whole);
            const int turns = (p.whole + pairs - 1) / pairs, rest_turns = (p.rest + kClusters[split] - 1) / kClusters[split];
            const double stage = std::max(850.0, 4.0 * N), end = N > 192 ? 4000 : 500;
            const double t = turns * (p.KB * stage + end) +
                             rest_turns * ((p.KB + split - 1) / split * stage + 3000 + 16.0 * N);
            if (t >= least) continue;
            least = t;
            p.clusters = (int)std::min<long long>(kClusters[split], p.whole ? (p.whole + split - 1) / split + p.rest : p.rest);
            best = p;
        }
    }
    Plan p = best;
    const int stage = kStageA + p.N * 128;
    // even, so that a stage always belongs to the same two of the four sets: a set that skipped a stage's earlier use
    // could not tell its phases apart
    p.stages = std::min(12, (kSmemMost - 2048) / stage / 2 * 2);
    p.pitch = (k + 7) / 8 * 8;
    p.rows_bytes = ((size_t)n_rows * p.pitch * 2 + 255) / 256 * 256;
    p.part_bytes = (size_t)p.rest * p.split * p.N * 256 * 4;
    return p;
}

}  // namespace

size_t linear_tc_workspace(int n_out, int k, int n_rows) {
    const Plan p = make_plan(n_out, k, n_rows);
    return p.rows_bytes + p.part_bytes;
}

cudaError_t launch_linear_tc(const Linear& a, cudaStream_t s, std::string* why) {
    const Plan p = make_plan(a.n_out, a.k, a.n_rows);
    LinearTc g{};
    g.a = a;
    __half* rows = static_cast<__half*>(a.workspace);
    g.part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + p.rows_bytes);
    g.N = p.N;
    g.m_tiles = p.m_tiles;
    g.n_tiles = p.n_tiles;
    g.KB = p.KB;
    g.stages = p.stages;
    g.whole = p.whole;
    g.rest = p.rest;
    g.split = p.split;
    g.clusters = p.clusters;
    g.out_as = out_kind(a);
    g.vec = out_vec4(a);
    g.slots = p.N <= 128 ? 8 : 4;
    g.col_a = 512 - 32 * g.slots;
    g.shared_cols = 2 * p.N > (int)g.col_a;
    g.base1 = g.shared_cols ? g.col_a - p.N : p.N;
    CUtensorMap ta, tb;
    if (!make_tmap_2d_sw128(&ta, 1, a.w, a.k, a.n_out, a.w_stride, kStageK, 128, why) ||
        !make_tmap_2d_sw128(&tb, 2, rows, a.k, a.n_rows, (uint64_t)p.pitch * 2, 64, p.N / 2, why))
        return cudaErrorInvalidValue;
    const int64_t units = (int64_t)a.n_rows * ((a.k + 15) / 16);
    KVR_LAUNCH(widen_kernel, dim3((unsigned)std::min<int64_t>((units + 255) / 256, 16 * kNumSMs)), dim3(256), 0, s, a.x,
               a.x_stride, rows, p.pitch, a.k, a.n_rows);
    const size_t smem = 1024 + (size_t)p.stages * (kStageA + p.N * 128) + 1024;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(linear_tc_kernel, kSmemMost, &done);
    if (e != cudaSuccess) return e;
    return launch_clusters(2 * p.split, linear_tc_kernel, dim3(2 * p.split * p.clusters), dim3(kThreads), smem, s, ta, tb, g);
}

}  // namespace kvr
