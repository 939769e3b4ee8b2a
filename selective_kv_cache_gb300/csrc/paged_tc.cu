// paged_tc.cu -- attention of many rows over the paged cache on the sm_103a
// tensor cores (bf16 and 4-bit pages): prompts and refreshed rows, what
// paged_decode.cu would have to read the keys too often for.
//
//   x_rj = cap(scale <q_r, k_j>) + alpha loc_j + beta snk_j - slope |g_r - j|
//   o_r  = sum_j softmax_j(x_rj) v_j,   j in [lo_r, hi_r)
//
// A CTA walks its share of units: 128 keys of one (item, K/V head), an item
// being up to two tiles of 128 MMA rows (positions x the head's G query
// heads) that share every K and V tile.  The two tiles alternate on the tensor
// pipe: while one's softmax runs, the other's products do, and a tile's next
// scores go over its P as soon as the product with V has read it, so that two
// score buffers and two outputs fill tensor memory exactly.
//   warp 0      bf16: K and V pages by TMA into a ring of five 32 KB tiles, a
//               copy per page and 64-column half (one lane each), K_0 V_0 K_1 V_1 ...
//   warp 1      tcgen05.mma: S_t = Q_t K^T, O_t += P_t V.  One lane issues all
//               products; they complete in order, so "S_t of tile j is done" also
//               says that tile j - 1's product with V is.  The warp runs the loop
//               together: in one thread's code the descriptors passed through its
//               registers, 100-130 cycles a product (4096 rows 378 us in place of 304 then).
//   warp 2      Q of the next run by TMA, as soon as the last scores are done
//               with its tile (4 bits: the softmax warps then scale it to fp16 in place).
//   warps 4-11  softmax, four warps a row tile, one thread a row: no exchange
//               between threads.  Base 2; the running maximum is raised, and O
//               rescaled in tensor memory, only when it grows by more than
//               2^8.  P goes to tensor memory in 16 bits (bf16; fp16 for 4-bit
//               pages) as the A operand: 2^-8 (2^-11) of a weight at most.
//   warp 3      4 bits: the scale pairs of the packed tiles that warp 0's copies bring
//   warps 12-15 4 bits only: packed tiles, which come in three ahead, to their values
//               in fp16, s (c - 8) + (o + 8 s) in two packed FMAs, written into the
//               ring in the operand's swizzle.  A word's nibbles come out in
//               pairs (e, e + 4), so the 8 dims of a chunk lie in the order 0 4 1
//               5 2 6 3 7; Q is stored in that order and O read back from it.
// Biases of keys (the same for every row) are written to shared memory once a
// tile and read as broadcasts; a cap well above a whole tile's logits is its series
// on the FMA pipe, where two special functions a key (12 cycles of a warp) would bound
// the tile.  4096 rows over 8192 keys: 280 us plain, 332 with biases, 428 with slopes,
// 475 capped (620 with logits near the cap, 833 there for caps above 64, whose small
// logits go by the series one by one).
// A unit is four 128^3 products (2048 cycles of the pipe) and 2 x 128 x 128
// exponentials (1024).  Measured: 1.47 PFLOP/s at 4096 rows over 8192 keys of a
// 32/8-head model (0.28 ms), under 3000 cycles a unit, close to the chain of a row
// tile that bounds it: softmax 1450, its two products 1024, three hand-overs of
// 100-150; 1.48 PFLOP/s at 8192 causal rows (0.37 ms).  4 bits: 1.26 PFLOP/s there
// (0.44 ms); softmax and conversion share the issue slots, 3000 of a unit's 3700
// cycles.  The group count is a template argument: a pair per 32 dims whatever the
// group took 8 % longer.  Rows leave as one 32-byte store a thread: with 16-byte
// halves exchanged between neighbours a run's end took 4500 cycles in place of 3000.
// The runs' bookkeeping lives in shared memory, a copy per warp: a spilled register
// costs an L2 round trip here, where shared memory takes all but a few KB of L1.  The
// kernels with biases or slopes still spill, 60 bytes a thread in bf16 and 122 or 142
// in 4 bits (-Xptxas -v); plain and capped ones none.
// Every wait is bounded; on a timeout the CTA records it, drains its copies and
// products, frees tensor memory and returns.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <string>

#include "paged.h"
#include "ptx.cuh"

namespace kvr {
namespace {

constexpr uint32_t kHalf = 16384;               // 128 rows x 128 B
constexpr uint32_t kTile = 2 * kHalf;           // 128 x 128 16-bit values
constexpr uint32_t kOffQ = 0;                   // two row tiles
constexpr uint32_t kOffRing = 2 * kTile;
// bf16: five tiles of ring.  4 bits: four, and in the fifth's place three
// packed tiles (128 rows of codes, then their scale pairs) on their way in.
constexpr int kStaged = 3;
constexpr uint32_t kStageCodes = 128 * 64, kStage = kStageCodes + 128 * 16;
constexpr uint32_t kOffStage = kOffRing + 4 * kTile;
constexpr uint32_t kOffBar = kOffRing + 5 * kTile;
constexpr uint32_t kOffWalk = kOffBar + 256;    // a PagedWalk per warp
constexpr uint32_t kWalkBytes = 72;
constexpr uint32_t kOffBias = kOffWalk + 16 * kWalkBytes;   // of each row tile's 128 keys, fp32
constexpr uint32_t kSmem = kOffBias + 2 * 512;
static_assert(sizeof(PagedWalk) <= kWalkBytes && kStaged * kStage <= kTile && kSmem <= 232448, "shared memory layout");
// TMEM columns of tile t: S (P over its first 64) at 128 t, O at 256 + 128 t
constexpr uint32_t kColS = 0, kColO = 256, kTmem = 0;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLazy = 8.0f;

__device__ __forceinline__ float max3f(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    const __half2 y = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b),
                              *reinterpret_cast<const __half2*>(&c));
    return *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ uint32_t with_1024(uint32_t x, uint32_t mask) {
    uint32_t y;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(y) : "r"(x), "r"(mask), "r"(0x64006400u));
    return y;
}
// code - 8 of the even and of the odd nibble of each half, exact
__device__ __forceinline__ uint32_t even8(uint32_t x) {
    return hfma2(with_1024(x, 0x000f000fu), 0x3c003c00u, 0xe408e408u);
}
__device__ __forceinline__ uint32_t odd8(uint32_t x) {
    return hfma2(with_1024(x, 0x00f000f0u), 0x2c002c00u, 0xd480d480u);
}
// 128 consecutive columns of this thread's lane: four loads, one wait
__device__ __forceinline__ void tmem_ld128(uint32_t taddr, float* v) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
#define KVR_LD32(OFF)                                                                                              \
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"    \
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"                        \
                 : "=r"(r[OFF]), "=r"(r[OFF + 1]), "=r"(r[OFF + 2]), "=r"(r[OFF + 3]), "=r"(r[OFF + 4]),            \
                   "=r"(r[OFF + 5]), "=r"(r[OFF + 6]), "=r"(r[OFF + 7]), "=r"(r[OFF + 8]), "=r"(r[OFF + 9]),        \
                   "=r"(r[OFF + 10]), "=r"(r[OFF + 11]), "=r"(r[OFF + 12]), "=r"(r[OFF + 13]), "=r"(r[OFF + 14]),   \
                   "=r"(r[OFF + 15]), "=r"(r[OFF + 16]), "=r"(r[OFF + 17]), "=r"(r[OFF + 18]), "=r"(r[OFF + 19]),   \
                   "=r"(r[OFF + 20]), "=r"(r[OFF + 21]), "=r"(r[OFF + 22]), "=r"(r[OFF + 23]), "=r"(r[OFF + 24]),   \
                   "=r"(r[OFF + 25]), "=r"(r[OFF + 26]), "=r"(r[OFF + 27]), "=r"(r[OFF + 28]), "=r"(r[OFF + 29]),   \
                   "=r"(r[OFF + 30]), "=r"(r[OFF + 31])                                                             \
                 : "r"(taddr + (OFF)) : "memory")
    KVR_LD32(0);
    KVR_LD32(32);
    KVR_LD32(64);
    KVR_LD32(96);
#undef KVR_LD32
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    // no use of a destination moves above the wait
#pragma unroll
    for (int i = 0; i < 128; i += 16)
        asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                     "+r"(r[i + 6]), "+r"(r[i + 7]), "+r"(r[i + 8]), "+r"(r[i + 9]), "+r"(r[i + 10]), "+r"(r[i + 11]),
                     "+r"(r[i + 12]), "+r"(r[i + 13]), "+r"(r[i + 14]), "+r"(r[i + 15])::"memory");
}
// a sector of a row; 32-byte aligned
__device__ __forceinline__ void store32(void* p, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// N bytes, or zeros
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const uint8_t* src, bool take) {
    if constexpr (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(take ? N : 0)
                     : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
// The warp waits and stays together.  All lanes poll (one instruction) and vote: a
// shuffle of one lane's answer takes longer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}
// kind::f16 with fp16 A/B, fp32 D
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int a_mn_major, int b_mn_major) {
    return (1u << 4) | ((uint32_t)a_mn_major << 15) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}

template <int N>
__device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ int first_key(const PagedWalk& w, int s) { return ((w.it.klo >> 7) + w.off + s) << 7; }
__device__ __forceinline__ int row_tiles(const PagedWalk& w, int per_tile) { return w.it.rows > per_tile ? 2 : 1; }

// NG: scale groups of a 4-bit row, 0 for bf16 pages.  kScore: 0 products alone, 1 with
// biases, 2 also slopes, 3 also capped (kernels of their own: with the others' code in
// it a biased call spilled more, 343 us in place of 333)
template <int NG, int kScore>
__global__ void __launch_bounds__(NG ? 512 : 384, 1)
    paged_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const __grid_constant__ CUtensorMap tmQ, PagedAttn a) {
    constexpr bool kInt4 = NG != 0, kExtra = kScore != 0, kSlopes = kScore >= 2, kCap = kScore == 3;
    constexpr int kRing = kInt4 ? 4 : 5;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    if (sbase & 1023u) {   // the swizzle's atoms need it; the declaration asks for it
        if (threadIdx.x == 0) paged_err(a.p.err, DEV_ERR_INDEX, (int)sbase);
        return;
    }
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBar);   // [kRing] a K or V tile has landed
    uint64_t* empty = full + kRing;                                 // [kRing] its products are done
    uint64_t* q_full = empty + kRing;                               // [2] Q_t is in place
    uint64_t* q_empty = q_full + 2;                                 // [2] a run's last scores are done with Q_t
    uint64_t* s_full = q_empty + 2;                                 // [2] S_t is done
    uint64_t* p_full = s_full + 2;                                  // [2] P_t is in tensor memory
    uint64_t* o_done = p_full + 2;                                  // [2] a run's last product with V is done
    uint64_t* q_raw = o_done + 2;                                   // [2] 4 bits: Q_t has landed in bf16
    uint64_t* drained = q_raw + 2;                                  // every product issued is done
    uint64_t* c_full = drained + 1;                                 // [kStaged] 4 bits: a tile's codes have landed
    uint64_t* c_empty = c_full + kStaged;                           // [kStaged] and have been read
    uint64_t* b_full = c_empty + kStaged;                           // [2] a tile's biases are written
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(b_full + 2);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int G = a.G, per_tile = 128 / G;
    PagedWalk& w = *reinterpret_cast<PagedWalk*>(smem + kOffWalk + warp * kWalkBytes);
    auto advance = [&]() {
        __syncwarp();
        if (lane == 0) w.next(a, a.items);
        __syncwarp();
    };

    if (threadIdx.x == 0) {
        for (int i = 0; i < kRing; ++i) mbar_init(&full[i], kInt4 ? 4 : 1);
        for (int i = 0; i < kRing; ++i) mbar_init(&empty[i], 1);
        mbar_init(drained, 1);
        for (int i = 0; i < kStaged; ++i) {
            mbar_init(&c_full[i], 33);
            mbar_init(&c_empty[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], kInt4 ? 4 : 1);
            mbar_init(&q_raw[i], 1);
            mbar_init(&q_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&b_full[i], 4);
            mbar_init(&o_done[i], 1);
        }
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        prefetch_tmap(&tmQ);
    }
    if (warp == 2)   // rows of a tile that no position fills (128 % G): zeros for good
        for (int i = lane; i < 2 * (128 - per_tile * G) * 16; i += 32) {
            const int t = i / ((128 - per_tile * G) * 16), j = i % ((128 - per_tile * G) * 16);
            sts16(sbase + kOffQ + (uint32_t)t * kTile + (uint32_t)(j & 1) * kHalf +
                      (uint32_t)(per_tile * G + (j >> 4)) * 128u + (uint32_t)((j >> 1) & 7) * 16u,
                  make_uint4(0u, 0u, 0u, 0u));
            fence_proxy_async_smem();
        }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    pdl_wait();
    if (lane == 0) w = PagedWalk(a, a.shares[blockIdx.x], a.shares[blockIdx.x + 1].u0);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    pdl_trigger();
    bool ok = true;

    // registers to the softmax, which holds a row of scores a thread: 72 + 2 x
    // 216 of 3 x 168 a thread (bf16), 72 + 2 x 176 + 88 of 4 x 128 (4 bits)
    if (warp < 4) {
        reg_dec<72>();
        if (warp == 0) {
            // ------------------------------------------------------------ K and V copies
            // into the ring, or 4-bit codes into the staged tiles: a lane per page (bf16:
            // and operand half), so tiles of 16-slot pages take 8 copies (16)
            constexpr int kSlots = kInt4 ? kStaged : kRing;
            constexpr uint32_t kPitch = kInt4 ? kStage : kTile;
            constexpr int kRowLog = kInt4 ? 6 : 7;   // bytes of a row in a copy
            uint64_t* landed = kInt4 ? c_full : full;
            uint64_t* freed = kInt4 ? c_empty : empty;
            uint8_t* ring = smem + (kInt4 ? kOffStage : kOffRing);
            const int shift = min(a.p.page_shift, 7), pages = 128 >> shift;   // pages of a tile
            const int half = kInt4 ? 0 : lane & 1, pg = kInt4 ? lane : lane >> 1;
            const uint32_t dst_off = (uint32_t)half * kHalf + ((uint32_t)pg << (shift + kRowLog));
            int x = 0;   // tiles so far
            for (; w.live() && ok; advance()) {
                const int* table = a.p.table + (int64_t)w.it.seq * a.p.max_pages;
                const int n = w.n, klo = w.it.klo, khi = w.it.khi, head = w.h;
                const int key_base = first_key(w, 0) + (pg << shift);
                for (int s = 0; s < n && ok; ++s) {
                    const int k0 = key_base + 128 * s;
                    // pages none of whose keys is visible are not touched
                    const bool mine = pg < pages && k0 < khi && k0 + (1 << shift) > klo;
                    const int id = mine ? paged_id(a.p, table[k0 >> a.p.page_shift]) : 0;
                    const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, mine)) << (shift + kRowLog);
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv, ++x) {
                        const int slot = x % kSlots;
                        // a full barrier is armed again only after every poller of its last phase has passed it:
                        // what frees the slot waited for it
                        if (x >= kSlots && !warp_wait(&freed[slot], (uint32_t)(x / kSlots - 1) & 1u)) {
                            ok = false;
                            break;
                        }
                        if (lane == 0) mbar_arrive_expect_tx(&landed[slot], bytes);
                        __syncwarp();
                        if (mine)
                            tma_load_4d(ring + slot * kPitch + dst_off, kv ? &tmV : &tmK, &landed[slot], 64 * half,
                                        k0 & ((1 << a.p.page_shift) - 1), head, id);
                    }
                }
            }
            // let every copy still in flight land before the CTA exits
            if (!ok)
                for (int y = max(x - kSlots, 0); y < x; ++y)
                    warp_wait(&landed[y % kSlots], (uint32_t)(y / kSlots) & 1u);
        } else if (warp == 1) {
            // -------------------------------------------------------------- products
            // the warp stays together and one lane issues, so that addresses and
            // descriptors are uniform values, made once a warp and not moved from a
            // thread's registers for every product
            const bool leader = elect_one();
            const uint32_t id_s = kInt4 ? idesc_f16(128, 128, 0, 0) : idesc_bf16(128, 128, 0, 0);
            const uint32_t id_o = kInt4 ? idesc_f16(128, 128, 0, 1) : idesc_bf16(128, 128, 0, 1);   // V is MN-major
            uint32_t runs = 0, ps = 0;   // bit t: parity of the runs and of the P tiles of row tile t
            int slot = 0;                // the ring's next tile and its parity
            uint32_t par = 0;
            auto step = [&]() {
                if (++slot == kRing) slot = 0, par ^= 1u;
            };
            // descriptors advance by addresses / 16 in their low bits
            const uint64_t q_desc = sdesc_sw128(sbase + kOffQ, 16, 1024);
            const uint64_t k_desc = sdesc_sw128(sbase + kOffRing, 16, 1024);
            const uint64_t v_desc = sdesc_sw128(sbase + kOffRing, kHalf, 1024);
            auto scores = [&](int t, int k_slot) {
                const uint64_t qd = q_desc + (uint64_t)(t * (kTile >> 4));
                const uint64_t kd = k_desc + (uint64_t)(k_slot * (kTile >> 4));
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    const uint32_t o = ((uint32_t)(kk >> 2) * kHalf + (uint32_t)(kk & 3) * 32u) >> 4;
                    mma_bf16(kTmem + kColS + 128u * t, qd + o, kd + o, id_s, kk > 0);
                }
                mma_commit(&s_full[t]);
            };
            int n = __shfl_sync(0xffffffffu, w.n, 0);
            while (n > 0 && ok) {
                const int nt = __shfl_sync(0xffffffffu, row_tiles(w, per_tile), 0);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (t >= nt || !ok) continue;
                    ok = warp_wait(&q_full[t], (runs >> t) & 1u) && (t || warp_wait(&full[slot], par));
                    if (!ok) continue;
                    runs ^= 1u << t;
                    tc_fence_after();
                    if (leader) {
                        scores(t, slot);
                        if (n == 1) mma_commit(&q_empty[t]);
                        if (t == nt - 1) mma_commit(&empty[slot]);
                    }
                }
                step();
                for (int s = 0; s < n && ok; ++s) {
                    const int v_slot = slot;
                    const uint32_t v_par = par;
                    step();
                    const bool more = s + 1 < n;   // its K tile is the next
                    const uint64_t vd = v_desc + (uint64_t)(v_slot * (kTile >> 4));
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (t >= nt || !ok) continue;
                        ok = (t || warp_wait(&full[v_slot], v_par)) && warp_wait(&p_full[t], (ps >> t) & 1u);
                        if (!ok) continue;
                        ps ^= 1u << t;
                        tc_fence_after();
                        if (leader) {
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk)
                                mma_bf16_ta(kTmem + kColO + 128u * t, kTmem + kColS + 128u * t + (uint32_t)kk * 8u,
                                            vd + (uint64_t)(kk * 128), id_o, (s > 0 || kk > 0));
                        }
                        // waited for while the pipe works on the product with V
                        if (!t && more && !(ok = warp_wait(&full[slot], par))) continue;
                        if (leader) {
                            if (more) scores(t, slot);
                            if (s + 2 == n) mma_commit(&q_empty[t]);
                            if (s + 1 == n) mma_commit(&o_done[t]);
                            if (t == nt - 1) {
                                mma_commit(&empty[v_slot]);
                                if (more) mma_commit(&empty[slot]);
                            }
                        }
                        __syncwarp();
                    }
                    if (more) step();
                }
                advance();
                n = __shfl_sync(0xffffffffu, w.n, 0);
            }
            if (leader) mma_commit(drained);
            if (!warp_wait(drained, 0)) ok = false;
        } else if (warp == 2) {
            // ------------------------------------------------------------- Q by TMA
            if (lane == 0) {
                uint64_t* landed = kInt4 ? q_raw : q_full;
                uint32_t begun = 0, runs = 0;   // bit t: row tile t has begun a run; parity of its runs
                for (; w.live() && ok; w.next(a, a.items))
                    for (int t = 0; t < row_tiles(w, per_tile); ++t) {
                        // the run before this one; its own parity is the other
                        if (((begun >> t) & 1u) && !mbar_wait(&q_empty[t], ((runs >> t) & 1u) ^ 1u)) {
                            ok = false;
                            break;
                        }
                        uint8_t* dst = smem + kOffQ + (uint32_t)t * kTile;
                        mbar_arrive_expect_tx(&landed[t], 2u * 128u * (uint32_t)(per_tile * G));
                        tma_load_3d(dst, &tmQ, &landed[t], 0, w.h * G, w.it.row0 + t * per_tile);
                        tma_load_3d(dst + kHalf, &tmQ, &landed[t], 64, w.h * G, w.it.row0 + t * per_tile);
                        begun |= 1u << t;
                        runs ^= 1u << t;
                    }
                for (int t = 0; t < 2; ++t)   // the last copies land before the CTA exits
                    if (((begun >> t) & 1u) && !mbar_wait(&landed[t], ((runs >> t) & 1u) ^ 1u)) ok = false;
            }
        } else if constexpr (kInt4) {
            // ------------------------------------------------------------ scale pairs
            // lane: keys lane + 32 i of a tile; a key nobody sees gets zeros: 0 * (c - 8) + 0
            constexpr int mb = 4 * NG;   // bytes of a row's pairs
            const int in_page = (1 << a.p.page_shift) - 1;
            const int page_m = (int)a.p.page_stride * mb, slot_m = (int)a.p.slot_stride * mb;   // below 2^31 (checked)
            int x = 0;   // tiles so far
            for (; w.live() && ok; advance()) {
                const int* table = a.p.table + (int64_t)w.it.seq * a.p.max_pages;
                const int n = w.n, klo = w.it.klo, khi = w.it.khi, key_base = first_key(w, 0) + lane;
                const int64_t head = w.h * a.p.head_stride * mb;
                for (int s = 0; s < n && ok; ++s) {
                    int id[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = key_base + 128 * s + 32 * i;
                        id[i] = -1;
                        if (key >= klo && key < khi) id[i] = table[key >> a.p.page_shift] & 0x7fffffff;
                    }
                    int64_t at[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        at[i] = id[i] < 0 ? 0 : head + (int64_t)paged_id(a.p, id[i]) * page_m +
                                                    (int64_t)((key_base + 128 * s + 32 * i) & in_page) * slot_m;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv, ++x) {
                        const int stage = x % kStaged;
                        if (x >= kStaged && !warp_wait(&c_empty[stage], (uint32_t)(x / kStaged - 1) & 1u)) {
                            ok = false;
                            break;
                        }
                        const uint8_t* pairs = kv ? a.p.vs : a.p.ks;
                        const uint32_t d = sbase + kOffStage + (uint32_t)stage * kStage + kStageCodes +
                                           (uint32_t)(mb * lane);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t dst = d + (uint32_t)(32 * mb * i);
                            copy_async<mb>(dst, pairs + at[i], id[i] >= 0);
                        }
                        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                                         smem_u32(&c_full[stage]))
                                     : "memory");
                    }
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else if (warp < 12) {
        reg_inc<kInt4 ? 176 : 216>();
        // -------------------------------------------------------------- softmax
        const int t = warp >= 8 ? 1 : 0, m = 32 * (warp & 3) + lane;
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = kTmem + kColS + 128u * t + lane_base, to = kTmem + kColO + 128u * t + lane_base;
        const float sl2 = a.scale * kLog2e;
        int g = 0, tile = 0, runs = 0, biases = 0;   // tiles of the CTA; tiles, runs and biased tiles of this row tile
        auto skip = [&]() {   // to the next run this row tile has rows in; the units passed are counted
            while (w.live() && t >= row_tiles(w, per_tile)) {
                g += w.n;
                advance();
            }
        };
        float lsr_next = sl2;   // what turns the row's products into base-2 logits
        // 4 bits: this thread's row of Q to fp16, scaled by a power of two to [128,
        // 256) at its largest, in place (the permuted order stays within a chunk)
        auto load_q = [&]() {
            if constexpr (kInt4) {
                if (!(ok = warp_wait(&q_raw[t], (uint32_t)runs & 1u))) return;
                const uint32_t dst = sbase + kOffQ + (uint32_t)t * kTile + (uint32_t)m * 128u;
                uint4 q[16];
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    q[c] = lds16(dst + (uint32_t)(c >> 3) * kHalf + (uint32_t)(((c & 7) ^ (m & 7)) << 4));
                uint32_t top = 0u;
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const uint32_t ws[4] = {q[c].x, q[c].y, q[c].z, q[c].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = max(top, max(ws[e] & 0x7f80u, (ws[e] >> 16) & 0x7f80u));
                }
                const int ex = min(max((int)(top >> 7), 8), 253);
                const float f = __uint_as_float((uint32_t)(261 - ex) << 23);      // 2^(134 - ex)
                // 2^(ex - 134); finite and not zero, so that 0 and -inf stay what they are under it
                lsr_next = fminf(fmaxf(sl2 * __uint_as_float((uint32_t)(ex - 7) << 23), 2e-38f), 2e38f);
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const uint32_t ws[4] = {q[c].x, q[c].y, q[c].z, q[c].w};
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[2 * e] = __uint_as_float(ws[e] << 16) * f;
                        x[2 * e + 1] = __uint_as_float(ws[e] & 0xffff0000u) * f;
                    }
                    sts16(dst + (uint32_t)(c >> 3) * kHalf + (uint32_t)(((c & 7) ^ (m & 7)) << 4),
                          make_uint4(pack_f16(x[0], x[4]), pack_f16(x[1], x[5]), pack_f16(x[2], x[6]),
                                     pack_f16(x[3], x[7])));
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_full[t]);
            }
        };
        // what this thread's row of a run sees
        struct Sees {
            int lo, hi, pos;
            float slope;
            bool live;   // a row of the item
        };
        Sees next{};
        auto load_row = [&]() {
            const int p = t * per_tile + m / G;
            next.lo = w.it.klo, next.hi = w.it.khi;
            next.live = m < per_tile * G && p < w.it.rows;
            if (next.live) {
                paged_interval(a, w.it.row0 + p, w.it.kv, &next.lo, &next.hi);
                if (kSlopes && a.slopes) {
                    next.pos = a.r.pos[w.it.row0 + p];
                    next.slope = a.slopes[w.h * G + m % G] * kLog2e;
                }
            }
        };
        const bool sectors = !(reinterpret_cast<uintptr_t>(a.out) & 31u) && a.out_stride % 16 == 0;
        skip();
        if (w.live()) {
            load_row();
            load_q();
        }
        while (w.live() && ok) {
            const Sees me = next;
            const int all_lo = __reduce_max_sync(0xffffffffu, me.lo), all_hi = __reduce_min_sync(0xffffffffu, me.hi);
            const int n = w.n, klo = w.it.klo, khi = w.it.khi, key_base = first_key(w, 0), seq = w.it.seq;
            const float lsr = lsr_next;
            float m_run = -INFINITY, m_neg = 0.f, l_run = 0.f;
            for (int s = 0; s < n; ++s, ++g, ++tile) {
                const int key0 = key_base + 128 * s;
                uint32_t lw = 0u, sw = 0u;   // lane: mask word lane % 4, on its way during the wait
                if (kExtra && (a.loc || a.snk)) {
                    const int64_t word = (int64_t)seq * a.words + min((key0 >> 5) + (lane & 3), a.words - 1);
                    if (a.loc) lw = a.loc[word];
                    if (a.snk) sw = a.snk[word];
                }
                if (!warp_wait(&s_full[t], (uint32_t)tile & 1u)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // the keys' biases are the same for every row: each warp writes those of 32
                // keys, to be read as broadcasts.  The last tile's have been read: its P
                // was waited for before these scores.
                const bool biased = kExtra && __any_sync(0xffffffffu, (lw | sw) != 0u);
                if (biased) {
                    lw = __shfl_sync(0xffffffffu, lw, warp & 3);
                    sw = __shfl_sync(0xffffffffu, sw, warp & 3);
                    const float bias = ((lw >> lane) & 1u ? a.alpha * kLog2e : 0.f) +
                                       ((sw >> lane) & 1u ? a.beta * kLog2e : 0.f);
                    reinterpret_cast<float*>(smem + kOffBias + 512 * t)[m] = bias;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&b_full[t]);
                }
                float x[128], ls = lsr;
                tmem_ld128(ts, x);
                if constexpr (kExtra) {
                    if constexpr (kCap) {
                        // u = in x; finite, so that a product of zero stays zero under the ranges' ends
                        const float cap_out = a.softcap * kLog2e, in = fminf(lsr / cap_out, 1e38f);
                        // The warp's choice comes from its rows' logits of a tile that they all see
                        // whole: what other columns and rows hold decides nothing.
                        float top_abs = 0.f;
#pragma unroll
                        for (int k = 0; k < 128; k += 2) top_abs = max3f(top_abs, fabsf(x[k]), fabsf(x[k + 1]));
                        const bool whole = key0 >= all_lo && key0 + 128 <= all_hi;
                        const float2 in2 = make_float2(in, in);
                        if (whole && __all_sync(0xffffffffu, !me.live || top_abs * in <= kTanhSeries)) {
#pragma unroll
                            for (int k = 0; k < 128; k += 2) {
                                const float2 y = tanh_series(__fmul2_rn(make_float2(x[k], x[k + 1]), in2));
                                x[k] = y.x, x[k + 1] = y.y;
                            }
                        } else if (a.softcap <= kCapQuotient) {
                            const float in_q = in * kTwoLog2e;
#pragma unroll
                            for (int k = 0; k < 128; ++k) x[k] = tanh_quotient(x[k] * in_q);
                        } else {
#pragma unroll
                            for (int k = 0; k < 128; k += 2) {
                                const float2 y = tanh_either(__fmul2_rn(make_float2(x[k], x[k + 1]), in2));
                                x[k] = y.x, x[k + 1] = y.y;
                            }
                        }
                        ls = cap_out;
                    }
                    if (biased) {
                        if (!warp_wait(&b_full[t], (uint32_t)biases++ & 1u)) {
                            ok = false;
                            break;
                        }
                        const float4* bias = reinterpret_cast<const float4*>(smem + kOffBias + 512 * t);
                        const float2 l2 = make_float2(ls, ls);
#pragma unroll
                        for (int k = 0; k < 128; k += 16) {
                            float4 b[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) b[i] = bias[k / 4 + i];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float* y = x + k + 4 * i;
                                const float2 u = __ffma2_rn(make_float2(y[0], y[1]), l2, make_float2(b[i].x, b[i].y));
                                const float2 v = __ffma2_rn(make_float2(y[2], y[3]), l2, make_float2(b[i].z, b[i].w));
                                y[0] = u.x, y[1] = u.y, y[2] = v.x, y[3] = v.y;
                            }
                        }
                        ls = 1.f;
                    }
                    if (kSlopes && a.slopes) {   // the distance's roundings, 2^-24 of it, are the product's own size
                        const float ahead = (float)(me.pos - key0);
#pragma unroll
                        for (int k = 0; k < 128; ++k) x[k] = fmaf(-me.slope, fabsf(ahead - (float)k), x[k] * ls);
                        ls = 1.f;
                    }
                }
                if (key0 + 128 > all_hi) {   // warp-uniform, as the next
                    const int h = me.hi - key0;
#pragma unroll
                    for (int k = 0; k < 128; ++k)
                        if (k >= h) x[k] = -INFINITY;
                }
                if (key0 < all_lo) {
                    const int l = me.lo - key0;
#pragma unroll
                    for (int k = 0; k < 128; ++k)
                        if (k < l) x[k] = -INFINITY;
                }
                float mx[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    mx[i] = fmaxf(x[i], x[i + 8]);
#pragma unroll
                    for (int q = 1; q < 8; ++q) mx[i] = max3f(mx[i], x[i + 16 * q], x[i + 16 * q + 8]);
                }
                const float top =
                    max3f(max3f(mx[0], mx[1], mx[2]), max3f(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * ls;
                const bool raise = top > m_run + kLazy;
                if (__any_sync(0xffffffffu, raise)) {
                    const float f = raise ? ex2(m_run - top) : 1.f;
                    if (s > 0) {
                        // the scores of this tile being done, so is the product of the one before: O stands still
#pragma unroll 1
                        for (int c = 0; c < 8; ++c) {
                            float o[16];
                            tmem_ld16(to + 16u * c, o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= f;
                            tmem_st16(to + 16u * c, o);
                        }
                    }
                    if (raise) l_run *= f, m_run = top, m_neg = -top;
                }
                // weights against the running maximum, in 16 bits, and their sum
                const float2 sc = make_float2(ls, ls), nm = make_float2(m_neg, m_neg);
                float2 acc[2] = {};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int k = 32 * c + 2 * e;
                        const float2 y = __ffma2_rn(make_float2(x[k], x[k + 1]), sc, nm);
                        const float2 z = make_float2(ex2(y.x), ex2(y.y));
                        pk[e] = kInt4 ? pack_f16(z.x, z.y) : pack_bf16(z.x, z.y);
                        acc[e & 1] = __fadd2_rn(acc[e & 1], z);
                    }
                    tmem_st16_async(ts + 16u * c, pk);
                }
                const float2 all = __fadd2_rn(acc[0], acc[1]);
                l_run += all.x + all.y;
                // keys nobody sees: whatever their slots held is not used.  Both row
                // tiles write the same zeros, each before its own product.
                if (!kInt4 && (key0 < klo || key0 + 128 > khi)) {
                    const int vx = 2 * g + 1, key = key0 + m;
                    if (!warp_wait(&full[vx % kRing], (uint32_t)(vx / kRing) & 1u)) {
                        ok = false;
                        break;
                    }
                    if (key < klo || key >= khi) {
                        const uint32_t d = sbase + kOffRing + (uint32_t)(vx % kRing) * kTile + (uint32_t)m * 128u;
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            sts16(d + 16u * c, make_uint4(0u, 0u, 0u, 0u));
                            sts16(d + kHalf + 16u * c, make_uint4(0u, 0u, 0u, 0u));
                        }
                    }
                    fence_proxy_async_smem();
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[t]);
            }
            if (!ok) break;
            // ---- where the run's rows go
            const int p = t * per_tile + m / G;
            const int64_t row = w.it.row0 + p;
            const int head = w.h * G + m % G;
            const bool whole = w.whole(), valid = m < per_tile * G && p < w.it.rows;
            const size_t slot = ((size_t)blockIdx.x * 2 + (w.first ? 0 : 1)) * a.tile_rows;
            // ---- the next run's rows and Q, so that its first scores are on their way meanwhile
            advance();
            skip();
            ++runs;
            if (w.live()) {
                load_row();
                load_q();
            }
            // ---- the run's rows
            if (!ok || !warp_wait(&o_done[t], (uint32_t)(runs - 1) & 1u)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const float inv = l_run > 0.f ? 1.0f / l_run : 0.f;
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + row * a.out_stride + (int64_t)head * 128;
            // partials lie chunk by chunk of four dims, [32][tile_rows], so that the
            // lanes' rows are neighbours; whole rows leave as 32-byte sectors
            float* po = a.part_o + slot * 128 + 4 * (size_t)(t * 128 + m);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                float y[64];
                tmem_ld32x2(to + 64u * hf, y);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float o[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e)   // 4 bits: column 2 k + b of a chunk of 8 is dim k + 4 b
                        o[e] = kInt4 ? y[16 * c + (e & 8) + 2 * (e & 3) + ((e >> 2) & 1)] : y[16 * c + e];
                    const int d = 64 * hf + 16 * c;
                    if (whole) {
                        uint32_t k[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) k[e] = pack_bf16(o[2 * e] * inv, o[2 * e + 1] * inv);
                        if (valid && sectors) {
                            store32(out + d, k);
                        } else if (valid) {
                            *reinterpret_cast<uint4*>(out + d) = make_uint4(k[0], k[1], k[2], k[3]);
                            *reinterpret_cast<uint4*>(out + d + 8) = make_uint4(k[4], k[5], k[6], k[7]);
                        }
                    } else if (valid) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *reinterpret_cast<float4*>(po + (size_t)(d / 4 + e) * 4 * a.tile_rows) =
                                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                }
            }
            if (valid && !whole)
                *reinterpret_cast<float2*>(a.part_ml + 2 * (slot + t * 128 + m)) = make_float2(m_run, l_run);
            tc_fence_before();
        }
    } else if constexpr (kInt4) {
        reg_dec<88>();
        // -------------------------------------------------------------- 4-bit tiles to fp16
        // a warp's keys are 32 of the tile: lane (kr, q) takes keys kr + 8 i, the 16 bytes
        // that hold dims 8 q.. of each 32-dim block.  Eight lanes that read or write
        // together hold keys p and p ^ 5, whose codes and whose swizzled chunks lie in
        // different banks.
        const int q = lane & 3, kr = 32 * (warp & 3) + ((lane >> 3) ^ ((lane & 4) ? 5 : 0));
        constexpr int mb = 4 * NG;
        const uint32_t stage0 = sbase + kOffStage;
        int x = 0;   // tiles so far
        for (; w.live() && ok; advance())
            for (int left = 2 * w.n; left > 0; --left, ++x) {
                const int slot = x % kRing, stage = x % kStaged;
                if (!warp_wait(&c_full[stage], (uint32_t)(x / kStaged) & 1u) ||
                    (x >= kRing && !warp_wait(&empty[slot], (uint32_t)(x / kRing - 1) & 1u))) {
                    ok = false;
                    break;
                }
                const uint32_t d = stage0 + (uint32_t)stage * kStage;
                uint4 cw[4];
                uint32_t cm[4][NG];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = kr + 8 * i;
                    cw[i] = lds16(d + 64u * k + 16u * q);
                    const uint32_t dm = d + kStageCodes + (uint32_t)(mb * k);
                    if constexpr (NG == 4) {
                        const uint4 v = lds16(dm);
                        cm[i][0] = v.x, cm[i][1] = v.y, cm[i][2] = v.z, cm[i][3] = v.w;
                    } else {
#pragma unroll
                        for (int g = 0; g < NG; ++g) cm[i][g] = lds4(dm + 4u * g);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&c_empty[stage]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = kr + 8 * i;
                    const uint32_t dst = sbase + kOffRing + (uint32_t)slot * kTile + (uint32_t)k * 128u;
                    uint4 v[4];
#pragma unroll
                    for (int b = 0; b < 4; ++b) {   // 32-dim block: units of the chunk's two 8-byte halves
                        const uint32_t z = __byte_perm(b < 2 ? cw[i].x : cw[i].y, b < 2 ? cw[i].z : cw[i].w,
                                                       (b & 1) ? 0x7632 : 0x5410);
                        const uint32_t pair = cm[i][b * NG / 4], sc = __byte_perm(pair, 0u, 0x1010);
                        const uint32_t o8 = hfma2(sc, 0x48004800u, __byte_perm(pair, 0u, 0x3232));
                        v[b] = make_uint4(hfma2(even8(z), sc, o8), hfma2(odd8(z), sc, o8),
                                          hfma2(even8(z >> 8), sc, o8), hfma2(odd8(z >> 8), sc, o8));
                    }
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        sts16(dst + (uint32_t)(b >> 1) * kHalf + (uint32_t)(((4 * (b & 1) + q) ^ (k & 7)) << 4), v[b]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[slot]);
            }
    }
    if (!ok && lane == 0) paged_err(a.p.err, DEV_ERR_TIMEOUT, warp);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(kTmem, 512);
}

template <int NG, int kScore>
cudaError_t launch(const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& q, const PagedAttn& a,
                   cudaStream_t s) {
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(paged_tc_kernel<NG, kScore>, (int)kSmem, &allowed);
    if (e != cudaSuccess) return e;
    KVR_LAUNCH((paged_tc_kernel<NG, kScore>), dim3((unsigned)a.n_cta), dim3(NG ? 512 : 384), kSmem, s, k, v, q, a);
    return cudaSuccess;
}
template <int NG>
cudaError_t launch_ng(const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& q, const PagedAttn& a,
                      cudaStream_t s) {
    if (a.softcap > 0.f) return launch<NG, 3>(k, v, q, a, s);
    if (a.slopes) return launch<NG, 2>(k, v, q, a, s);
    return a.loc || a.snk ? launch<NG, 1>(k, v, q, a, s) : launch<NG, 0>(k, v, q, a, s);
}

}  // namespace

cudaError_t launch_paged_tc(int format, int group, const PagedAttn& a, cudaStream_t s, std::string* why) {
    CUtensorMap k{}, v{}, q{};
    // Q as (dim, head, row): a box is a row tile of one K/V head, positions x query heads
    if (!make_tmap_3d_bf16(&q, a.q, 128, (uint64_t)a.n_q_heads, (uint64_t)a.r.n_rows, 256, (uint64_t)a.q_stride * 2, 64,
                           (uint32_t)a.G, (uint32_t)(128 / a.G), why))
        return cudaErrorInvalidValue;
    // pages as (dim, slot, head, page); a box is one page's share of a 128-key tile:
    // half a row wide, or a row of codes
    const bool int4 = format == KVR_INT4;
    const uint64_t row = int4 ? 64 : 256;
    const uint64_t dims[4] = {int4 ? row : 128, 1ull << a.p.page_shift, (uint64_t)a.p.n_kv_heads,
                              (uint64_t)a.p.n_pages};
    const uint64_t strides[3] = {(uint64_t)a.p.slot_stride * row, (uint64_t)a.p.head_stride * row,
                                 (uint64_t)a.p.page_stride * row};
    const uint32_t box[4] = {64, 1u << (a.p.page_shift < 7 ? a.p.page_shift : 7), 1, 1};
    auto pages = int4 ? make_tmap_4d_bytes : make_tmap_4d_bf16;
    if (!pages(&k, a.p.k, dims, strides, box, why) || !pages(&v, a.p.v, dims, strides, box, why))
        return cudaErrorInvalidValue;
    if (!int4) return launch_ng<0>(k, v, q, a, s);
    if (group == 32) return launch_ng<4>(k, v, q, a, s);
    if (group == 64) return launch_ng<2>(k, v, q, a, s);
    return launch_ng<1>(k, v, q, a, s);
}

}  // namespace kvr
