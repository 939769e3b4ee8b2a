// linear_mma.cu -- projection of a few 8-bit rows: y[r][f] = s_r t_f sum_k
// a[r][k] w[f][k] + bias[f], the sums as 32-bit integers (m16n8k32 on signed
// bytes: products and sums exact).
//
// A decode step's handful of rows reads every weight byte once and does 2 n_rows
// operations on it: HBM-bound.  Weights are the M operand, loaded straight into
// registers: K may be taken in any order as long as both operands take the
// same, so a thread's fragments are 16 consecutive bytes of one weight row, and
// four threads read 64 of it.  A warp holds 32 features; the block's eight warps
// and the cluster's blocks take every 64-byte step in turn, so that they read
// neighbouring bytes at a time, and the partial sums meet in shared memory, the
// cluster's over distributed shared memory: one launch, no workspace, any order
// of addition the same integer.  A warp holds two steps in registers and loads
// each again right after its products, three blocks on an SM.
#include "linear.cuh"

namespace kvr {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kRows = kLinearMmaRows, kUnroll = 2;   // rows of a block; 64-byte steps a warp has in flight
constexpr int kMT = 2, kFeatures = 16 * kMT;   // weight tiles of a warp, features of a block

__device__ __forceinline__ void mma_s8(int* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 load_stream(const int8_t* p) {   // weights: read once
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
// The row's last pieces: one that holds a code lies in the row up to 16-byte
// alignment.  The rows' codes behind k are made zeros, the weights' then do not count.
__device__ __forceinline__ uint4 load_tail(const int8_t* p, int left, bool zeros) {
    uint4 v = left > 0 ? *reinterpret_cast<const uint4*>(p) : make_uint4(0u, 0u, 0u, 0u);
    if (zeros) {
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = left - 4 * i;
            w[i] = n >= 4 ? w[i] : n <= 0 ? 0u : w[i] & (0xffffffffu >> (32 - 8 * n));
        }
    }
    return v;
}

__global__ void __launch_bounds__(kThreads, 3) linear_mma_kernel(const __grid_constant__ Linear a, int split) {
    constexpr int kTile = kFeatures * kRows;
    __shared__ int part[kWarps][kTile];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int rank = (int)blockIdx.x % split, f0 = (int)blockIdx.x / split * kFeatures;
    // rows past the end are read as the last one and not written
    const int8_t* wp[kMT][2];
#pragma unroll
    for (int m = 0; m < kMT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) wp[m][h] = a.w + (int64_t)min(f0 + 16 * m + 8 * h + g, a.n_out - 1) * a.w_stride + 16 * t;
    const int8_t* xp = a.x + (int64_t)min(g, a.n_rows - 1) * a.x_stride + 16 * t;
    int acc[kMT][4] = {};
    auto products = [&](const uint4 (&w)[kMT][2], uint4 x) {
#pragma unroll
        for (int m = 0; m < kMT; ++m) {
            mma_s8(acc[m], w[m][0].x, w[m][1].x, w[m][0].y, w[m][1].y, x.x, x.y);
            mma_s8(acc[m], w[m][0].z, w[m][1].z, w[m][0].w, w[m][1].w, x.z, x.w);
        }
    };
    const int steps = a.k / 64, stride = kWarps * split;
    // a ring of kUnroll steps in registers: each is loaded again as soon as its products are out
    uint4 w[kUnroll][kMT][2], x[kUnroll];
    auto fetch = [&](int u, int step) {
#pragma unroll
        for (int m = 0; m < kMT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) w[u][m][h] = load_stream(wp[m][h] + 64 * step);
        x[u] = *reinterpret_cast<const uint4*>(xp + 64 * step);
    };
    const int first = rank * kWarps + warp;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
        if (first + u * stride < steps) fetch(u, first + u * stride);
    for (int s = first; s < steps; s += stride * kUnroll) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (s + u * stride < steps) products(w[u], x[u]);
            if (s + (u + kUnroll) * stride < steps) fetch(u, s + (u + kUnroll) * stride);
        }
    }
    if (rank == split - 1 && warp == kWarps - 1 && a.k % 64) {
        const int at = 64 * steps, left = a.k - at - 16 * t;
        uint4 w[kMT][2];
#pragma unroll
        for (int m = 0; m < kMT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) w[m][h] = load_tail(wp[m][h] + at, left, false);
        products(w, load_tail(xp + at, left, true));
    }
#pragma unroll
    for (int m = 0; m < kMT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)   // row 2 t + i % 2, feature g + 8 (i / 2) of the tile
            part[warp][(2 * t + (i & 1)) * kFeatures + 16 * m + g + 8 * (i >> 1)] = acc[m][i];
    __syncthreads();
    for (int i = threadIdx.x; i < kTile; i += kThreads) {
        int v = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += part[w][i];
        part[0][i] = v;   // entry i is this thread's alone
    }
    if (split > 1) cluster_sync();
    else __syncthreads();
    // The cluster's blocks would take the tile's entries in turn; there are as many as threads, so the first one adds up and
    // writes them all.
    for (int i = rank * kThreads + threadIdx.x; i < kTile; i += split * kThreads) {
        const int r = i / kFeatures, f = f0 + i % kFeatures;
        int v = part[0][i];
        for (int p = 1; p < split; ++p) v += load_peer(peer_address(&part[0][i], (rank + p) % split));
        if (r >= a.n_rows || f >= a.n_out) continue;
        write_out(a, (int64_t)r * a.out_stride + f, (float)v * a.x_scale[r] * a.w_scale[f] + (a.bias ? a.bias[f] : 0.f));
    }
    if (split > 1) cluster_sync();   // no block leaves while the first reads its sums
}

}  // namespace

cudaError_t launch_linear_mma(const Linear& a, cudaStream_t s) {
    const int groups = (a.n_out + kFeatures - 1) / kFeatures, steps = a.k / 64;
    // The fewest shares of K that give the SMs one and a half blocks each, as long as a warp keeps
    // two steps: 14336 -> 4096 one share 20.2 us, two 15.0, three 14.8, four 17.8, eight 20.8;
    // 18944 -> 3584 25.2, 18.5, 18.0, 20.9, 22.7; 8960 -> 1536 one 12.3, three 7.7, five 6.9, eight 8.3.
    int split = 1;
    while (split < 8 && 2 * groups * split < 3 * kNumSMs && steps >= 2 * (split + 1) * kWarps) ++split;
    return launch_clusters(split, linear_mma_kernel, dim3(groups * split), dim3(kThreads), 0, s, a, split);
}

}  // namespace kvr
