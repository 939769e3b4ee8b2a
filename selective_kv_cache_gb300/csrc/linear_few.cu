// linear_few.cu -- projection of a batch of 8-bit rows (a decode batch, drafts)
// on the sm_103a tensor cores, in one launch:
//   y[r][f] = s_r t_f sum_k a[r][k] w[f][k] + bias[f]
//
// HBM-bound: the weights come in once, 128 features by up to 64 rows a block
// (more rows: as many blocks side by side, the weights then from L2).
// Both operands are widened to fp16 on the way (8-bit integers, their products
// and the fp32 sums up to 2^24 are exact; above, the accumulator cuts each step
// of 16 products off, by up to 2^-23): the weights into tensor memory, the A
// operand, the rows into shared memory.  A cluster's blocks split k, and join
// their sums as integers over distributed shared memory: nothing goes through
// the workspace.  Where there are more tiles than clusters, a cluster has several
// and its blocks share their stages, so that all SMs have the same to do.
//   warp 0     TMA: per stage 128 features x 128 codes and N rows x 128 codes
//   warp 1     products, eight of K = 16 a stage
//   warps 2..  widening, in sets of four that take the stages in turn, each into
//              a slot of its own: a thread a feature and up to four pieces of the
//              rows; then they write the sums out
// A stage is bound by its widened weights' way into tensor memory (770 cycles),
// which takes four sets to keep busy.  They are one block of four sets an SM, or
// two blocks of two, so that one streams while the other starts or ends
// (make_plan).  A block's shared memory leaves no room on its SM for more
// tensor memory than there is (linear_few_smem), so blocks of other clusters do
// not wait for one another's: an allocation is no bounded wait, and two clusters
// that each hold what the other's second block waits for would never end.  Every
// other wait is bounded.
//
// Where 19.2 us of 64 rows, 14336 -> 4096 go (clock64, cycles): set up at 1700,
// the first stage there at 5000, all 28 widened at 26000, products and sums out
// at 29500, the cluster together at 31000, joined over distributed shared memory
// at 33500, out at 34700.
#include <algorithm>

#include "linear.cuh"
#include "ptx.cuh"

namespace kvr {
namespace {

constexpr uint32_t kStageA = 128 * 128;
// by the number of sets: a block's threads, blocks an SM, columns, shared memory
// Tensor memory in columns of 64: accumulators of the tiles that a block works on, then a slot for each set.
constexpr int kTilesMost = 4;
template <int kSets>
constexpr int kThreadsOf = 64 + 128 * kSets;
template <int kSets>
constexpr int kBlocksOf = kSets == 2 ? 2 : 1;
template <int kSets>
constexpr int kSmemOf = (kSets == 2 ? 113 : 227) * 1024;

struct LinearFew {
    Linear a;
    int N, split, tiles, KB, stages, out_as, vec;   // vec: four features of an output row are one aligned store
    Div by_split, by_clusters, by_KB;
};

// kSpread: a cluster has several tiles, whose stages its blocks share evenly.
template <int kSets, bool kSpread>
__global__ void __launch_bounds__(kThreadsOf<kSets>, kBlocksOf<kSets>)
    linear_few_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ LinearFew g) {
    constexpr int kThreads = kThreadsOf<kSets>;
    constexpr uint32_t kCols = kSets == 2 ? 256 : 512, kColA = kSpread ? 64 * kTilesMost : 64;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int stages = g.stages;
    const uint32_t tile = (uint32_t)g.N * 128, stage_bytes = kStageA + tile;   // N rows of 128 codes, or of 64 widened ones
    uint8_t* wide = smem + (size_t)stages * stage_bytes;                       // [kSets][2 chunks]
    uint64_t* full = reinterpret_cast<uint64_t*>(wide + 2 * kSets * tile);
    uint64_t* empty = full + stages;
    uint64_t* ready = empty + stages;   // [kSets]
    uint64_t* freed = ready + kSets;    // [kSets]
    uint64_t* done = freed + kSets;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    uint32_t* unread = tmem_slot + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // The cluster's tiles are [t0, t0 + T), their stages in a row [0, T KB), this block's [lo(rank), lo(rank + 1)).
    const int split = g.split, cluster = (int)g.by_split(blockIdx.x), rank = (int)blockIdx.x - cluster * split;
    const int t0 = kSpread ? (int)g.by_clusters(g.tiles * cluster) : cluster;
    const int T = kSpread ? (int)g.by_clusters(g.tiles * (cluster + 1)) - t0 : 1;
    auto lo = [&](int p) { return (int)g.by_split(T * g.KB * p); };
    const int u0 = lo(rank), n_kb = lo(rank + 1) - u0, first = kSpread ? (int)g.by_KB(u0) : 0;
    int kb = u0 - first * g.KB, f_next = (t0 + first) * 128;   // of the next stage
    const int row0 = blockIdx.y * g.N, rows = min(g.N, g.a.n_rows - row0);   // of this block's tile
    auto copies = [&](int s) {
        mbar_arrive_expect_tx(&full[s], stage_bytes);
        uint8_t* d = smem + (size_t)s * stage_bytes;
        tma_load_2d(d, &tmA, &full[s], kb * 128, f_next);
        tma_load_2d(d + kStageA, &tmB, &full[s], kb * 128, row0);
        if (++kb == g.KB && kSpread) {
            kb = 0;
            f_next += 128;
        }
    };

    if (warp == 0) {
        // a barrier a lane: one thread takes 50 cycles for each
        if (lane < stages) {
            mbar_init(&full[lane], 1);
            mbar_init(&empty[lane], 4);
        } else if (lane >= 16 && lane < 16 + kSets) {
            mbar_init(&ready[lane - 16], 4);
            mbar_init(&freed[lane - 16], 1);
        } else if (lane == 31) {
            mbar_init(done, 1);
        }
        fence_mbar_init();
        __syncwarp();
    }
    if (threadIdx.x == 0) {
        for (int it = 0; it < min(stages, n_kb); ++it) copies(it);   // the ring fills while the block sets up
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;

    if (warp == 0) {
        if (lane == 0) {
            int s = 0, it = stages;
            uint32_t phase = 0;
            for (; it < n_kb; ++it) {
                if (!mbar_wait(&empty[s], phase)) {
                    ok = false;
                    break;
                }
                copies(s);
                if (++s == stages) {
                    s = 0;
                    phase ^= 1u;
                }
            }
            // whatever the others met, every copy lands before the block exits
            const int sent = min(it, n_kb);
            for (int i = max(0, sent - stages); i < sent; ++i) mbar_wait(&full[i % stages], (uint32_t)(i / stages) & 1u);
        }
        __syncwarp();
    } else if (warp == 1) {
        const uint32_t idesc = (1u << 4) | ((uint32_t)(g.N >> 3) << 17) | ((128u >> 4) << 24);   // fp16, fp32 sums
        const uint64_t descB = sdesc_sw128(smem_u32(wide), 16, 1024);
        const bool issuer = elect_one();
        uint32_t acc = tmem;
        bool fresh = true;
        for (int it = 0; it < n_kb; ++it) {
            const uint32_t t = it % kSets;
            if (!__all_sync(0xffffffffu, mbar_wait(&ready[t], (uint32_t)(it / kSets) & 1u))) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (issuer) {
#pragma unroll
                for (uint32_t kk = 0; kk < 8; ++kk)
                    mma_bf16_ta(acc, tmem + kColA + 64 * t + 8 * kk,
                                descB + (uint64_t)(((2 * t + kk / 4) * tile >> 4) + 2 * (kk % 4)), idesc, !fresh || kk > 0);
                mma_commit(&freed[t]);
            }
            __syncwarp();
            fresh = kSpread && ++kb == g.KB;
            if (fresh) {
                kb = 0;
                acc += 64;
            }
        }
        if (issuer) mma_commit(done);
        __syncwarp();
        if (!__all_sync(0xffffffffu, mbar_wait(done, 0))) ok = false;
    } else {
        const int set = (warp - 2) >> 2, quarter = warp & 3, row = 32 * quarter + lane;
        const uint32_t dst = tmem + ((uint32_t)(32 * quarter) << 16), slot = dst + kColA + 64 * set;
        // Piece p of the rows' tile: row p / 8, its 16 codes p % 8, which become two 16-byte pieces of a chunk's row.
        // A thread's pieces lie 16 rows apart: the same swizzle.
        const uint32_t r = row >> 3, piece = row & 7;
        const uint32_t from = smem_u32(smem) + row * 128, from_b = smem_u32(smem) + kStageA + r * 128 + ((piece ^ (r & 7)) << 4);
        const uint32_t to_b = smem_u32(wide) + (2 * set + (piece >> 2)) * tile + r * 128;
        const uint32_t lo = ((2 * (piece & 3)) ^ (r & 7)) << 4, hi = ((2 * (piece & 3) + 1) ^ (r & 7)) << 4;
        int s = set % stages;
        uint32_t phase = (uint32_t)(set / stages) & 1u, use = 1;
        uint4 c[8], b[4];
        auto fetch = [&]() {
            const uint32_t at = (uint32_t)s * stage_bytes;
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i] = lds128(from + at + ((i ^ (row & 7)) << 4));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                b[i] = 16 * i < g.N ? lds128(from_b + at + 2048 * i) : make_uint4(0u, 0u, 0u, 0u);
        };
        // The stage goes back once its codes are in registers.  An arrival does not wait for loads whose values nothing
        // has used, and the copy that it allows would overtake them: so a word of every vector decides on a store that
        // precedes the arrival, and that the assembler cannot drop.  Where it happens, nobody reads what it writes.  What
        // this relies on: a vector's words arrive together, the predicate needs one of each, and a warp issues its
        // instructions in order, so the arrival is not issued before the predicate is known.
        auto give_back = [&]() {
            uint32_t seen = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) seen ^= c[i].w;
#pragma unroll
            for (int i = 0; i < 4; ++i) seen ^= b[i].w;
            asm volatile(
                "{\n\t.reg .pred p;\n\t"
                "setp.eq.u32 p, %0, 0x5bd1e995;\n\t"
                "@p st.volatile.shared.u32 [%1], %0;\n\t}\n" ::"r"(seen),
                "r"(smem_u32(unread))
                : "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
        };
        bool have = false;
        for (int it = set; it < n_kb; it += kSets, use ^= 1u) {
            if (!have) {
                if (!__all_sync(0xffffffffu, mbar_wait(&full[s], phase))) {
                    ok = false;
                    break;
                }
                fetch();
                give_back();
            }
            if (!__all_sync(0xffffffffu, mbar_wait(&freed[set], use))) {
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t h[32];
#pragma unroll
            for (int i = 0; i < 4; ++i) widen16(c[i], h + 8 * i);
            tmem_st16_async(slot, h);
            tmem_st16_async(slot + 16, h + 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (16 * i >= g.N) break;
                uint32_t y[8];
                widen16(b[i], y);
                sts128(to_b + 2048 * i + lo, y);
                sts128(to_b + 2048 * i + hi, y + 4);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) widen16(c[4 + i], h + 8 * i);
            tmem_st16_async(slot + 32, h);
            tmem_st16_async(slot + 48, h + 16);
            // the next stage's codes on their way while these stores complete
            for (int i = 0; i < kSets; ++i)
                if (++s == stages) {
                    s = 0;
                    phase ^= 1u;
                }
            have = it + kSets < n_kb && __all_sync(0xffffffffu, mbar_test(&full[s], phase));
            if (have) fetch();
            fence_proxy_async_smem();
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ready[set]);
            if (have) give_back();
        }
        // ---------------------------------------------------------------- sums out
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(done, 0)) != 0;
        if (ok) {
            tc_fence_after();
            // chunks of 32 rows of a tile, one or two a tile
            const int twice = g.N > 32, chunks = (kSpread ? (int)g.by_KB(u0 + n_kb - 1) - first + 1 : 1) << twice;
            for (int i = set; i < chunks; i += kSets) {
                const int j = i >> twice, c = 32 * (i - (j << twice)), begin = (first + j) * g.KB, f = (t0 + first + j) * 128 + row;
                const bool whole = kSpread ? u0 <= begin && begin + g.KB <= u0 + n_kb : split == 1;   // all of the tile's stages
                const float sw = whole && f < g.a.n_out ? g.a.w_scale[f] : 0.f;
                const float bias = whole && f < g.a.n_out && g.a.bias ? g.a.bias[f] : 0.f;
                const float sx = whole && c + lane < rows ? g.a.x_scale[row0 + c + lane] : 0.f;
                float v[32];
                tmem_ld32(dst + (uint32_t)(64 * j + c), v);
                if (whole) {
                    write32(g.a, g.out_as, row0 + c, f, v, sx, sw, bias, rows - c);
                } else {   // into the ring, which nothing uses any more: [N][128], a second one for the last tile
                    float* o = reinterpret_cast<float*>(smem) + ((kSpread && u0 < begin ? g.N : 0) + c) * 128 + row;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (c + i < g.N) o[i * 128] = v[i];
                }
            }
        }
    }
    if (!ok) atomicOr(g.a.err, DEV_ERR_TIMEOUT);
    tc_fence_before();
    if (split > 1) {
        // The tiles that blocks share: a row a warp, four features a lane; this block's rows are [r0, r1).
        const int r0 = g.N * rank / split, r1 = min(g.N * (rank + 1) / split, rows);
        float sw[4], bias[4];
        auto features = [&](int t) {
            const int f = (t0 + t) * 128 + 4 * lane;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sw[i] = f + i < g.a.n_out ? g.a.w_scale[f + i] : 0.f;
                bias[i] = f + i < g.a.n_out && g.a.bias ? g.a.bias[f + i] : 0.f;
            }
        };
        const int from = lane < split ? lo(lane) : T * g.KB, to = lane < split ? lo(lane + 1) : 0;   // block `lane`'s stages
        // bit p: block p has stages of tile t
        auto has = [&](int t) { return __ballot_sync(0xffffffffu, from < (t + 1) * g.KB && to > t * g.KB); };
        auto shared_from = [&](int t) {
            for (; kSpread && t < T; ++t) {
                const uint32_t in = has(t);
                if (in & (in - 1)) break;
            }
            return t;
        };
        int t = shared_from(0);
        if (t < T) features(t);   // on their way while the others finish
        constexpr int kWarps = kThreads / 32;   // at most 64 rows: a lane holds the scale of one of its warp's
        const int mine = r0 + warp + kWarps * lane;
        const float scales = mine < r1 ? g.a.x_scale[row0 + mine] : 0.f;
        cluster_sync();
        while (t < T) {
            const uint32_t in = kSpread ? has(t) : (1u << split) - 1;
            const uint32_t second = kSpread ? __ballot_sync(0xffffffffu, from < t * g.KB) : 0u;   // whose sums lie in the second
            for (int r = r0 + warp, i = 0; r < r1; r += kWarps, ++i) {
                const float sx = __shfl_sync(0xffffffffu, scales, i);
                float4 v[8];
#pragma unroll
                for (int p = 0; p < 8; ++p)
                    if (in >> p & 1u)
                        v[p] = load_peer4(peer_address(smem + (size_t)(((second >> p & 1u ? g.N : 0) + r) * 128 + 4 * lane) * 4,
                                                       (uint32_t)p));
                int sum[4] = {0, 0, 0, 0};
#pragma unroll
                for (int p = 0; p < 8; ++p)
                    if (in >> p & 1u) {
                        sum[0] += __float2int_rn(v[p].x);
                        sum[1] += __float2int_rn(v[p].y);
                        sum[2] += __float2int_rn(v[p].z);
                        sum[3] += __float2int_rn(v[p].w);
                    }
                float y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = (float)sum[i] * sx * sw[i] + bias[i];
                write4(g.a, g.vec, row0 + r, (t0 + t) * 128 + 4 * lane, y);
            }
            t = shared_from(t + 1);
            if (t < T) features(t);
        }
        cluster_sync();   // no block leaves while another reads its sums
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

}  // namespace

namespace {
struct Plan {
    int row_tiles, N, tiles, KB, sets, split, clusters;
    double us;   // estimated
};

// Clusters of `split` blocks of four sets that the GPU holds at once: a cluster's blocks share a GPC.
int clusters_at_once(int split) {
    static std::atomic<int> known[9];
    int n = known[split].load(std::memory_order_relaxed);
    if (n > 0) return n;
    static std::atomic<uint64_t> done{0};
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(split);
    cfg.blockDim = dim3(kThreadsOf<4>);
    cfg.dynamicSmemBytes = kSmemOf<4>;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (allow_smem(linear_few_kernel<4, false>, kSmemOf<4>, &done) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, linear_few_kernel<4, false>, &cfg) != cudaSuccess || n < 1)
        return 0;
    known[split].store(n, std::memory_order_relaxed);
    return n;
}

Plan make_plan(int n_out, int k, int n_rows) {
    Plan p{};
    p.row_tiles = (n_rows + 63) / 64;
    p.N = ((n_rows + p.row_tiles - 1) / p.row_tiles + 15) / 16 * 16;
    p.tiles = (n_out + 127) / 128;
    p.KB = (k + 127) / 128;
    const long long blocks = (long long)p.tiles * p.row_tiles;
    const double wide = std::max(0, p.N - 16) / 48.0;   // more rows than 16 of a tile, as a part of 48
    // Two sets: a block an SM as long as each has two stages, two an SM where each keeps six; all of them resident at
    // once.  1536 -> 2048 in twos 8.5 us, fours 6.7, eights 8.4.  Threes and sixes fit the GPCs badly.
    p.sets = 2;
    p.clusters = p.tiles;
    p.split = 1;
    while (p.split < 8 && ((2 * p.split * blocks <= kNumSMs && p.KB >= 4 * p.split) ||
                           (2 * p.split * blocks <= 2 * kNumSMs && p.KB >= 12 * p.split)))
        p.split *= 2;
    const double waves = (double)((blocks * p.split + 2 * kNumSMs - 1) / (2 * kNumSMs));
    const int stages = (p.KB + p.split - 1) / p.split;
    // starting and joining, and a stage: with two blocks on the busiest SM, with one
    p.us = blocks * p.split > kNumSMs ? 8.0 + (0.55 + 0.25 * wide) * waves * stages : 5.0 + (0.5 + 0.2 * wide) * stages;
    // Four sets: all clusters at once, a cluster's blocks share its T tiles' stages evenly, where each keeps six.  64 rows:
    // 14336 -> 4096 in fours 19.2 us (two sets in eights 20.5), 18944 -> 3584 in fives 20.6 (23.8), 4096 -> 4096 in fours
    // 10.8 (11.5), 4096 -> 28672 three tiles a pair 30.3 (34.2); 128 rows, 18944 -> 3584 two tiles in fives 32.3 (one in
    // twos 36.9); 48 rows, 4096 -> 12288 unsplit 16.3 (19.6).
    for (int split = 1; split <= 8; ++split) {
        const int room = split == 1 ? kNumSMs : clusters_at_once(split), clusters = std::min(p.tiles, room / p.row_tiles);
        if (clusters < 1) continue;
        const int T = (p.tiles + clusters - 1) / clusters, share = (T * p.KB + split - 1) / split;
        const int touched = T == 1 ? 1 : split == 1 ? T : (T + split - 1) / split + 1;   // tiles of a block at most
        if (touched > kTilesMost || share < 6) continue;
        const double us = (split > 1 ? 6.8 : 5.0) + (0.28 + 0.14 * wide) * share + (T > 1 ? 3.0 : 0.0);
        if (us >= p.us) continue;
        p.us = us;
        p.sets = 4;
        p.split = split;
        p.clusters = clusters;
    }
    return p;
}

template <int kSets, bool kSpread>
cudaError_t launch(LinearFew& g, const Plan& p, cudaStream_t s, std::string* why) {
    const Linear& a = g.a;
    const int smem = linear_few_smem(kSets, g.N, &g.stages);
    CUtensorMap ta, tb;
    if (!make_tmap_2d_sw128(&ta, 1, a.w, a.k, a.n_out, a.w_stride, 128, 128, why) ||
        !make_tmap_2d_sw128(&tb, 1, a.x, a.k, a.n_rows, a.x_stride, 128, g.N, why))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(linear_few_kernel<kSets, kSpread>, kSmemOf<kSets>, &done);
    if (e != cudaSuccess) return e;
    return launch_clusters((unsigned)g.split, linear_few_kernel<kSets, kSpread>, dim3(p.clusters * p.split, p.row_tiles),
                           dim3(kThreadsOf<kSets>), (size_t)smem, s, ta, tb, g);
}
}  // namespace

int linear_few_smem(int sets, int N, int* stages) {
    const int tile = N * 128, stage = (int)kStageA + tile, most = sets == 2 ? kSmemOf<2> : kSmemOf<4>;
    const int fixed = 1024 + 2 * sets * tile + 512;   // the ring's size also holds the [N][128] sums
    // A multiple of the sets, so that a stage always belongs to the same one: a set that skipped a stage's earlier
    // use could not tell its phases apart.
    *stages = std::min(8, (most - 1024 - fixed) / stage / sets * sets);
    // Two sets take 256 of an SM's 512 columns: more than a third of its 228 KB (a block costs 1 KB more than it asks
    // for), which 48 rows a tile with their 69.5 KB would leave.
    return std::max(fixed + *stages * stage, sets == 2 ? 76 * 1024 : 0);
}

double linear_few_us(int n_out, int k, int n_rows) { return make_plan(n_out, k, n_rows).us; }

cudaError_t launch_linear_few(const Linear& a, cudaStream_t s, std::string* why) {
    const Plan p = make_plan(a.n_out, a.k, a.n_rows);
    LinearFew g{a, p.N, p.split, p.tiles, p.KB, 0, out_kind(a), out_vec4(a), Div(p.split), Div(p.clusters), Div(p.KB)};
    if (p.sets == 2) return launch<2, false>(g, p, s, why);
    return p.clusters == p.tiles ? launch<4, false>(g, p, s, why) : launch<4, true>(g, p, s, why);
}

}  // namespace kvr
