// linear_few.cu -- projection of a batch of 8-bit rows (a decode batch, drafts)
// on the sm_103a tensor cores, in one launch:
//   y[r][f] = s_r t_f sum_k a[r][k] w[f][k] + bias[f]
//
// HBM-bound: the weights come in once, 128 features by up to 64 rows a block.
// Both operands are widened to fp16 on the way (8-bit integers, their products
// and the fp32 sums up to 2^24 are exact): the weights into tensor memory, the A
// operand, the rows into shared memory.  A cluster's blocks split k, and join
// their sums as integers over distributed shared memory: nothing goes through
// the workspace.  Two blocks an SM, so that one streams while the other starts
// or ends.
//   warp 0     TMA: per stage 128 features x 128 codes and N rows x 128 codes
//   warp 1     products, four of K = 16 a 64-code chunk
//   warps 2-9  widening, in two sets of four: set 0 takes the first 64 codes of every
//              stage, set 1 the second, a thread a feature and two pieces of
//              the rows; then they write the sums out
// Every wait is bounded.
#include <algorithm>

#include "linear.cuh"
#include "ptx.cuh"

namespace kvr {
namespace {

constexpr int kThreads = 320, kSlots = 4;
constexpr uint32_t kStageA = 128 * 128;
constexpr uint32_t kCols = 256, kColA = 128;   // accumulator (up to 64 columns), then four chunks of 32
constexpr int kSmemMost = 113 * 1024;          // two blocks an SM

struct LinearFew {
    Linear a;
    int N, split, KB, stages, out_as;
};

__global__ void __launch_bounds__(kThreads, 2) linear_few_kernel(const __grid_constant__ CUtensorMap tmA,
                                                                const __grid_constant__ CUtensorMap tmB,
                                                                const __grid_constant__ LinearFew g) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int stages = g.stages;
    const uint32_t tile = (uint32_t)g.N * 128, stage_bytes = kStageA + tile;   // N rows of 128 codes, or of 64 widened ones
    uint8_t* wide = smem + (size_t)stages * stage_bytes;                       // [kSlots]
    uint64_t* full = reinterpret_cast<uint64_t*>(wide + kSlots * tile);
    uint64_t* empty = full + stages;
    uint64_t* ready = empty + stages;   // [kSlots]
    uint64_t* freed = ready + kSlots;   // [kSlots]
    uint64_t* done = freed + kSlots;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = g.split, rank = (int)blockIdx.x % split, f0 = (int)blockIdx.x / split * 128;
    const int kb0 = g.KB * rank / split, n_kb = g.KB * (rank + 1) / split - kb0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 8);
        }
        for (int t = 0; t < kSlots; ++t) {
            mbar_init(&ready[t], 4);
            mbar_init(&freed[t], 1);
        }
        mbar_init(done, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kCols);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;

    if (warp == 0) {
        if (lane == 0) {
            int s = 0, it = 0;
            uint32_t phase = 1;
            for (; it < n_kb; ++it) {
                if (!mbar_wait(&empty[s], phase)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(&full[s], stage_bytes);
                uint8_t* d = smem + (size_t)s * stage_bytes;
                tma_load_2d(d, &tmA, &full[s], (kb0 + it) * 128, f0);
                tma_load_2d(d + kStageA, &tmB, &full[s], (kb0 + it) * 128, 0);
                if (++s == stages) {
                    s = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) {   // let every copy still in flight land before the block exits
                for (int i = (it > stages ? it - stages : 0); i < it; ++i)
                    mbar_wait(&full[i % stages], (uint32_t)(i / stages) & 1u);
            }
        }
    } else if (warp == 1) {
        const uint32_t idesc = (1u << 4) | ((uint32_t)(g.N >> 3) << 17) | ((128u >> 4) << 24);   // fp16, fp32 sums
        const uint64_t descB = sdesc_sw128(smem_u32(wide), 16, 1024);
        const bool issuer = elect_one();
        for (int q = 0; q < 2 * n_kb; ++q) {
            const uint32_t t = q & (kSlots - 1);
            if (!__all_sync(0xffffffffu, mbar_wait(&ready[t], (uint32_t)(q / kSlots) & 1u))) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (issuer) {
#pragma unroll
                for (uint32_t kk = 0; kk < 4; ++kk)
                    mma_bf16_ta(tmem, tmem + kColA + 32 * t + 8 * kk, descB + (uint64_t)((t * tile >> 4) + 2 * kk), idesc,
                                q > 0 || kk > 0);
                mma_commit(&freed[t]);
            }
            __syncwarp();
        }
        if (issuer) mma_commit(done);
        __syncwarp();
        if (!__all_sync(0xffffffffu, mbar_wait(done, 0))) ok = false;
    } else {
        const int half = (warp - 2) >> 2, quarter = warp & 3, row = 32 * quarter + lane;
        const uint32_t dst = tmem + ((uint32_t)(32 * quarter) << 16);
        int s = 0, pending = -1;
        uint32_t phase = 0;
        // A chunk is handed over when the next one's codes are in registers, or at once where those have not come.
        auto hand_over = [&]() {
            if (pending < 0) return;
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ready[pending]);
            pending = -1;
        };
        for (int it = 0; it < n_kb; ++it) {
            const int q = 2 * it + half;
            const uint32_t t = q & (kSlots - 1);
            if (!__all_sync(0xffffffffu, mbar_test(&full[s], phase))) {
                hand_over();
                if (!__all_sync(0xffffffffu, mbar_wait(&full[s], phase))) {
                    ok = false;
                    break;
                }
            }
            const uint8_t* a = smem + (size_t)s * stage_bytes;
            uint4 c[4], b[2];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                c[i] = *reinterpret_cast<const uint4*>(a + row * 128 + (((4 * half + i) ^ (row & 7)) << 4));
            // piece p of the rows: row p / 4, 16 codes p % 4 of the chunk
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int p = row + 128 * i, r = p >> 2;
                if (r < g.N)
                    b[i] = *reinterpret_cast<const uint4*>(a + kStageA + r * 128 + (((4 * half + (p & 3)) ^ (r & 7)) << 4));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
            uint32_t h[32];
#pragma unroll
            for (int i = 0; i < 4; ++i) widen16(c[i], h + 8 * i);
            hand_over();
            if (!__all_sync(0xffffffffu, mbar_wait(&freed[t], ((uint32_t)(q / kSlots) & 1u) ^ 1u))) {
                ok = false;
                break;
            }
            tc_fence_after();
            tmem_st16_async(dst + kColA + 32 * t, h);
            tmem_st16_async(dst + kColA + 32 * t + 16, h + 16);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int p = row + 128 * i, r = p >> 2;
                if (r < g.N) {
                    uint32_t y[8];
                    widen16(b[i], y);
                    uint8_t* o = wide + t * tile + r * 128;
                    *reinterpret_cast<uint4*>(o + (((2 * (p & 3)) ^ (r & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
                    *reinterpret_cast<uint4*>(o + (((2 * (p & 3) + 1) ^ (r & 7)) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
                }
            }
            fence_proxy_async_smem();
            pending = (int)t;
            if (++s == stages) {
                s = 0;
                phase ^= 1u;
            }
        }
        hand_over();
        // ---------------------------------------------------------------- sums out
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(done, 0)) != 0;
        if (ok) {
            tc_fence_after();
            const int f = f0 + row, left = min(g.a.n_rows, g.N);
            const float sw = f < g.a.n_out ? g.a.w_scale[f] : 0.f, bias = f < g.a.n_out && g.a.bias ? g.a.bias[f] : 0.f;
            for (int c = 32 * half; c < g.N; c += 64) {
                float v[32];
                tmem_ld32(dst + (uint32_t)c, v);
                if (split == 1) {
                    const float sx = c + lane < left ? g.a.x_scale[c + lane] : 0.f;
                    write32(g.a, g.out_as, c, f, v, sx, sw, bias, left - c);
                } else {   // into the ring, which nothing uses any more: [N][128]
                    float* o = reinterpret_cast<float*>(smem) + c * 128 + row;
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
        cluster_sync();
        // this block's rows of the tile, four features a thread
        const int r0 = g.N * rank / split, n = min(g.N * (rank + 1) / split, g.a.n_rows) - r0;
        for (int i = threadIdx.x; i < n * 32; i += kThreads) {
            const int r = r0 + i / 32, f = 4 * (i % 32);
            int sum[4] = {0, 0, 0, 0};
            for (int p = 0; p < split; ++p) {
                const float4 v = load_peer4(peer_address(smem + (size_t)(r * 128 + f) * 4, (uint32_t)((rank + p) % split)));
                sum[0] += __float2int_rn(v.x);
                sum[1] += __float2int_rn(v.y);
                sum[2] += __float2int_rn(v.z);
                sum[3] += __float2int_rn(v.w);
            }
            if (f0 + f < g.a.n_out) write4(g.a, r, f0 + f, sum);
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

cudaError_t launch_linear_few(const Linear& a, cudaStream_t s, std::string* why) {
    LinearFew g{};
    g.a = a;
    g.N = std::max(16, (a.n_rows + 15) / 16 * 16);
    g.KB = (a.k + 127) / 128;
    const int tiles = (a.n_out + 127) / 128;
    // Blocks a cluster: those on the busiest SM times their share of k, and a
    // little for joining.
    double best = 1e30;
    for (int c = 1; c <= std::min(8, std::max(1, g.KB / 2)); ++c) {
        const double t = (double)((tiles * c + kNumSMs - 1) / kNumSMs) * ((g.KB + c - 1) / c) + 0.25 * c;
        if (t < best) {
            best = t;
            g.split = c;
        }
    }
    const uint32_t tile = g.N * 128, stage = kStageA + tile;
    const uint32_t fixed = 1024 + kSlots * tile + 512;   // the ring's size also holds the [N][128] sums
    g.stages = (kSmemMost - 1024 - (int)fixed) / (int)stage;
    g.stages = std::min(g.stages, 8);
    g.out_as = out_kind(a);
    CUtensorMap ta, tb;
    if (!make_tmap_2d_sw128(&ta, 1, a.w, a.k, a.n_out, a.w_stride, 128, 128, why) ||
        !make_tmap_2d_sw128(&tb, 1, a.x, a.k, a.n_rows, a.x_stride, 128, g.N, why))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(linear_few_kernel, kSmemMost, &done);
    if (e != cudaSuccess) return e;
    return launch_clusters((unsigned)g.split, linear_few_kernel, dim3(tiles * g.split), dim3(kThreads),
                           fixed + (size_t)g.stages * stage, s, ta, tb, g);
}

}  // namespace kvr
