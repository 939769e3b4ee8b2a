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
//   warps 4-19   accumulators out, four warps a TMEM lane quarter
//   warps 20-27  widening: two sets of four warps, for the halves of every stage, a
//                thread a feature
// Barriers: full (copies landed, own CTA) -> widening warps of both CTAs ->
// a_ready (leader) -> products -> a_free, empty (both CTAs).  That the peer's
// rows have landed the issuing thread knows from the peer's widening warps,
// which wait for the same stage.
//
// Tensor memory: accumulators of two tiles (side by side up to N = 192; above,
// they share columns, which the epilogue reads first), and four chunks of widened
// weights behind them, eight up to N = 128.
//
// The pairs take tiles in turn, whole; how wide a tile is goes by a model of the
// time (make_plan).  Every wait is bounded.
#include <algorithm>

#include "linear.cuh"
#include "ptx.cuh"

namespace kvr {
namespace {

constexpr int kPairs = kNumSMs / 2;
constexpr int kOuts = 4;                          // warps a lane quarter that write out
constexpr int kThreads = 32 * (4 + 4 * kOuts + 8);
constexpr int kStageK = 128;                      // codes of a stage: two chunks
constexpr uint32_t kStageA = 128 * 128;           // 128 features x 128 bytes
constexpr int kSmemMost = 227 * 1024;
constexpr int kSuper = 8;                         // row tiles that are walked beside one another

struct LinearTc {
    Linear a;
    int out_as;
    int N, m_tiles, n_tiles, KB, stages, tiles, pairs;
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
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(peer_address(bar, 0)) : "memory");
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
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// ---------------------------------------------------------------- work
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
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(all_done + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t half = cta_rank();   // this CTA's half of the tile's features and rows
    const int pair = blockIdx.x >> 1;

    auto load_a = [&](int s, int m, int kb) {
        tma_load_2d(smem + (size_t)s * stage_bytes, &tmA, &full[s], kb * kStageK, m * 256 + (int)half * 128);
    };
    const int pre = min(stages, (g.tiles - pair + g.pairs - 1) / g.pairs * g.KB);   // first stages of this pair's tiles
    if (warp == 0) {
        // a barrier or two a lane: one thread takes 50 cycles for each
        if (lane < stages) {
            mbar_init(&full[lane], 1);
            mbar_init(&empty[lane], 1);
        }
        if (lane < 8) {
            mbar_init(&a_ready[lane], 8);
            mbar_init(&a_free[lane], 1);
        } else if (lane < 10) {
            mbar_init(&acc_full[lane - 8], 1);
            mbar_init(&acc_empty[lane - 8], 8 * kOuts);
        } else if (lane == 10) {
            mbar_init(cols_free, 8 * kOuts);
            mbar_init(all_done, 1);
        }
        fence_mbar_init();
        __syncwarp();
    }
    if (warp == 1) pair_alloc(tmem_slot);
    tc_fence_before();
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    if (threadIdx.x == 0) {
        // no kernel of the call writes the weights: the ring's first ones go out while the other CTA sets up
        prefetch_tmap(&tmB);
        int tile = pair, kb = 0, m, n;
        tile_coords(g, tile, &m, &n);
        for (int it = 0; it < pre; ++it) {
            mbar_arrive_expect_tx(&full[it], stage_bytes);
            load_a(it, m, kb);
            if (++kb == g.KB && it + 1 < pre) {
                kb = 0;
                tile_coords(g, tile += g.pairs, &m, &n);
            }
        }
    }
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");   // the other CTA's barriers are initialised
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t slots = g.slots, lap = slots == 8 ? 3 : 2;   // chunk q: slot q % slots, its use number q >> lap
    bool ok = true;
    pdl_trigger();

    if (warp == 0) {
        // ------------------------------------------------------------ copies
        if (lane == 0) {
            pdl_wait();
            int it = 0, s = 0;
            uint32_t phase = 1;
            for (int tile = pair; ok && tile < g.tiles; tile += g.pairs) {
                int m, n;
                tile_coords(g, tile, &m, &n);
                for (int kb = 0; kb < g.KB; ++kb, ++it) {
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
            // whatever the others met, every copy lands before the CTA exits
            for (int i = max(0, it - stages); i < it; ++i) mbar_wait(&full[i % stages], (uint32_t)(i / stages) & 1u);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        const bool issuer = elect_one();
        if (half == 0) {
            const uint32_t idesc = (1u << 4) | ((uint32_t)(g.N >> 3) << 17) | ((256u >> 4) << 24);   // fp16, fp32 sums
            const uint64_t descB = sdesc_sw128(smem_u32(smem) + kStageA, 16, 1024);
            int s = 0, local = 0;
            uint32_t q = 0;
            for (int tile = pair; ok && tile < g.tiles; tile += g.pairs, ++local) {
                const int ab = local & 1;
                if (!warp_wait(&acc_empty[ab], ((uint32_t)(local >> 1) & 1u) ^ 1u) ||
                    (g.shared_cols && local > 0 && !warp_wait(cols_free, (uint32_t)(local - 1) & 1u))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + (ab ? g.base1 : 0u);
                for (int kb = 0; kb < g.KB; ++kb) {
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
                                         (h > 0 || kk > 0) ? 1u : (kb > 0 ? 1u : 0u));
                            pair_commit(&a_free[t]);
                            if (h == 1) pair_commit(&empty[s]);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    if (++s == stages) s = 0;
                }
                if (!ok) break;
                if (issuer) pair_commit(&acc_full[ab]);
                __syncwarp();
            }
            if (issuer) pair_commit(all_done);
            __syncwarp();
        }
    } else if (warp >= 4 + 4 * kOuts) {
        // ------------------------------------------------------------ widening
        const int chunk = (warp - 4 - 4 * kOuts) >> 2, quarter = warp & 3, row = 32 * quarter + lane;
        const uint32_t dst = tmem + ((uint32_t)(32 * quarter) << 16) + g.col_a;
        // Every stage's and every slot's uses are one set's, in order, so that it can tell their phases apart.
        int s = 0, pending = -1;
        uint32_t phase = 0;
        // A chunk is handed over when the next one is half widened, so that its stores complete meanwhile, or at once
        // where that one's codes have not come.
        auto hand_over = [&]() {
            if (pending < 0) return;
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_leader(&a_ready[pending]);
            pending = -1;
        };
        const uint32_t from = smem_u32(smem) + row * 128;
        uint4 c[4];
        auto fetch = [&](int stage) {
            const uint32_t a = from + (uint32_t)stage * stage_bytes;
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = lds128(a + (((4 * chunk + i) ^ (row & 7)) << 4));
        };
        const int total = (g.tiles - pair + g.pairs - 1) / g.pairs * g.KB;
        bool have = false;
        for (int it = 0; it < total; ++it) {
            const uint32_t q = 2 * it + chunk, t = q & (slots - 1);
            if (!have) {
                hand_over();
                if (!__all_sync(0xffffffffu, mbar_wait(&full[s], phase))) {
                    ok = false;
                    break;
                }
                fetch(s);
            }
            if (!warp_wait(&a_free[t], ((q >> lap) & 1u) ^ 1u)) {
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t h[32];
            widen16(c[0], h);
            widen16(c[1], h + 8);
            hand_over();
            tmem_st16_async(dst + 32 * t, h);
            widen16(c[2], h + 16);
            widen16(c[3], h + 24);
            if (++s == stages) {
                s = 0;
                phase ^= 1u;
            }
            have = it + 1 < total && __all_sync(0xffffffffu, mbar_test(&full[s], phase));
            if (have) fetch(s);
            tmem_st16_async(dst + 32 * t + 16, h + 16);
            pending = (int)t;
        }
        hand_over();
    } else if (warp >= 4) {
        // ------------------------------------------------------------ accumulators out
        const int part = (warp - 4) >> 2, quarter = warp & 3, fo = (int)half * 128 + quarter * 32 + lane;   // this lane's feature in the tile
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        int local = 0;
        for (int tile = pair; tile < g.tiles; tile += g.pairs, ++local) {
            const int ab = local & 1;
            int m, n;
            tile_coords(g, tile, &m, &n);
            const int row0 = n * g.N, f = m * 256 + fo, rows = min(g.N, g.a.n_rows - row0);
            const float sw = f < g.a.n_out ? g.a.w_scale[f] : 0.f, bias = f < g.a.n_out && g.a.bias ? g.a.bias[f] : 0.f;
            if (!warp_wait(&acc_full[ab], (uint32_t)(local >> 1) & 1u)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t src = tmem + lane_base + (ab ? g.base1 : 0u);
            auto drain = [&](int lo, int hi) {
                for (int c = lo + 32 * part; c < hi; c += 32 * kOuts) {
                    const float sx = c + lane < rows ? g.a.x_scale[row0 + c + lane] : 0.f;
                    float v[32];
                    tmem_ld32(src + (uint32_t)c, v);
                    write32(g.a, g.out_as, row0 + c, f, v, sx, sw, bias, rows - c);
                }
            };
            if (g.shared_cols) {   // the columns that the next tile's accumulator shares first
                const int lo = ab ? 0 : (int)g.base1, hi = ab ? g.N - (int)g.base1 : g.N;
                drain(lo, hi);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_leader(cols_free);
                drain(0, lo);
                drain(hi, g.N);
            } else {
                drain(0, g.N);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_leader(&acc_empty[ab]);
        }
    }
    tc_fence_before();
    __syncthreads();
    // The last products' end on both CTAs.  Waited for here, when the accumulators are out, so that this wait spans no more
    // than another's: the other CTA's warp 1 has nothing to do before, and a call may take longer than a wait's limit.
    if (warp == 1 && !warp_wait(all_done, 0)) ok = false;
    if (!ok) atomicOr(g.a.err, DEV_ERR_TIMEOUT);
    cluster_sync();   // no product or arrival of the pair is on its way any more
    if (warp == 1) {
        tc_fence_after();
        pair_dealloc(tmem);
    }
}

int pitch_of(int k) { return (k + 7) / 8 * 8; }   // elements of a widened row

struct Plan {
    int N, m_tiles, n_tiles, KB, stages, tiles, pairs;
    double cycles;
};
// The width of a tile that takes the shortest time in cycles: a stage of 128
// codes takes its products' 4 N, or what the widening takes; a tile's end stops
// a wide one's products while shared columns are read.
Plan make_plan(int n_out, int k, int n_rows) {
    Plan p{};
    p.m_tiles = (n_out + 255) / 256;
    p.KB = (k + kStageK - 1) / kStageK;
    double least = 1e300;
    for (int N = 32; N <= 256; N += 32) {
        const int n_tiles = (n_rows + N - 1) / N;
        const long long turns = ((long long)p.m_tiles * n_tiles + kPairs - 1) / kPairs;
        const double t = (double)turns * (p.KB * std::max(650.0, 4.05 * N) + (N > 192 ? 4000 : 0)) + 20.0 * N;
        if (t >= least) continue;
        least = t;
        p.N = N;
        p.n_tiles = n_tiles;
    }
    p.cycles = least;
    p.tiles = p.m_tiles * p.n_tiles;
    p.pairs = std::min(kPairs, p.tiles);
    p.stages = std::min(12, (kSmemMost - 2048) / ((int)kStageA + p.N * 128));
    return p;
}

}  // namespace

double linear_tc_us(int n_out, int k, int n_rows) { return 5.5 + make_plan(n_out, k, n_rows).cycles / 1900; }

size_t linear_tc_workspace(int k, int n_rows) { return (size_t)n_rows * pitch_of(k) * 2; }

cudaError_t launch_linear_tc(const Linear& a, cudaStream_t s, std::string* why) {
    const Plan p = make_plan(a.n_out, a.k, a.n_rows);
    const int pitch = pitch_of(a.k);
    LinearTc g{};
    g.a = a;
    __half* rows = static_cast<__half*>(a.workspace);
    g.N = p.N;
    g.m_tiles = p.m_tiles;
    g.n_tiles = p.n_tiles;
    g.KB = p.KB;
    g.stages = p.stages;
    g.tiles = p.tiles;
    g.pairs = p.pairs;
    g.out_as = out_kind(a);
    g.slots = p.N <= 128 ? 8 : 4;
    g.col_a = 512 - 32 * g.slots;
    g.shared_cols = 2 * p.N > (int)g.col_a;
    g.base1 = g.shared_cols ? g.col_a - p.N : p.N;
    CUtensorMap ta, tb;
    if (!make_tmap_2d_sw128(&ta, 1, a.w, a.k, a.n_out, a.w_stride, kStageK, 128, why) ||
        !make_tmap_2d_sw128(&tb, 2, rows, a.k, a.n_rows, (uint64_t)pitch * 2, 64, p.N / 2, why))
        return cudaErrorInvalidValue;
    const int64_t units = (int64_t)a.n_rows * ((a.k + 15) / 16);
    KVR_LAUNCH(widen_kernel, dim3((unsigned)std::min<int64_t>((units + 255) / 256, 16 * kNumSMs)), dim3(256), 0, s, a.x,
               a.x_stride, rows, pitch, a.k, a.n_rows);
    const size_t smem = 1024 + (size_t)p.stages * (kStageA + p.N * 128) + 1024;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(linear_tc_kernel, kSmemMost, &done);
    return e != cudaSuccess ? e : launch_clusters(2, linear_tc_kernel, dim3(2 * p.pairs), dim3(kThreads), smem, s, ta, tb, g);
}

}  // namespace kvr
