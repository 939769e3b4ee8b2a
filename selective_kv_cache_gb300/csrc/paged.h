// paged.h -- the paged cache's device view, and how its attention shares work
// over the GPU (paged_api.cu, paged_rows.cu, paged_plan.cu, paged_simt.cu).
#pragma once
#include <atomic>

#include "kvr_internal.h"

namespace kvr {

enum : int { DEV_ERR_ORDER = 8 };   // appended positions of a sequence do not ascend

constexpr int kPagedMaxGroup = 16;   // query heads per K/V head
constexpr int kPagedInline = 256;    // calls of up to this many items need no plan launch, but in paged_tc.cu

struct PagedView {
    uint8_t* k;
    uint8_t* v;
    uint8_t* ks;
    uint8_t* vs;
    const int* table;
    const int* kv_len;
    int* err;
    int64_t page_stride, head_stride, slot_stride;
    int n_pages, batch, max_pages, page_shift, n_kv_heads, capacity;   // capacity = max_pages * page_size
};

// Packed rows of a call: sequence b owns rows [cu[b], cu[b+1]).
struct PagedRows {
    const int* cu;
    const int* pos;
    int n_rows;
};

struct PagedRowIo {   // append and read
    PagedView p;
    PagedRows r;
    const uint8_t* k_in;
    const uint8_t* v_in;
    const uint8_t* q_in;
    uint8_t* k_out;
    uint8_t* v_out;
    uint8_t* q_out;
    int64_t k_stride, v_stride, q_stride;   // bytes
    const float2* rope;
    int rope_len, n_q_heads;
    int units, rows_per_block;              // (row, head) units of a row; set by the launcher
};
cudaError_t launch_paged_append(int format, int head_dim, int group, const PagedRowIo& a, cudaStream_t s);
cudaError_t launch_paged_read(int format, int head_dim, int group, const PagedRowIo& a, cudaStream_t s);

// Up to `positions` packed rows of one sequence, for each K/V head: `units`
// times unit_keys keys, from the unit that holds key klo.
struct PagedItem {
    int klo, khi;     // keys any of its rows may see: [klo, khi)
    int units;        // >= 1 when it has rows, else 0
    int before;       // cost of one head of all earlier items
    int seq, kv;      // its sequence and that one's length
    int row0, rows;   // its packed rows
};
// The call's work is a line of runs, (item, head) by (item, head), each as long
// as its units plus run_cost for starting it; CTA c's equal share of the line
// is [u0(c), u0(c + 1)).  A share that begins or ends in a run's start does not
// split the run.
struct PagedShare {
    int item, head, off;   // the run it begins in and its first unit there
    int u0, run;           // its place on the line, and that run's
    PagedItem first;       // that item, so that a CTA's first loads wait for one record only
};
struct PagedAttn {
    PagedView p;
    PagedRows r;
    const void* q;
    void* out;
    int64_t q_stride, out_stride;   // elements
    int n_q_heads, G, max_rows;
    int positions;                  // packed rows of an item
    int tiles, n_items;             // items of a sequence, of the call (tiles * batch)
    int unit_keys, run_cost, n_cta, tile_rows;   // tile_rows >= positions * G: rows of a partial
    float scale, softcap, alpha, beta;
    const uint32_t* loc;
    const uint32_t* snk;
    const float* slopes;
    const int* key_begin;
    const int* key_end;
    int words;
    int planned;                    // items and shares come from launch_paged_plan (else the kernel derives them)
    // workspace
    PagedItem* items;               // [n_items], when planned
    PagedShare* shares;             // [n_cta + 1]; u0 of the last used + 1 is the end; item < 0: no work
    float* part_o;                  // [n_cta][2][tile_rows][head_dim], unnormalised
    float* part_ml;                 // [n_cta][2][tile_rows][2]: running max in base 2, sum
};
cudaError_t launch_paged_plan(const PagedAttn& a, cudaStream_t s);
cudaError_t launch_paged_merge(int dtype, int head_dim, const PagedAttn& a, cudaStream_t s);
// Up to 16 rows an item, fp32 pages, units of 32 keys.
cudaError_t launch_paged_simt(int head_dim, const PagedAttn& a, cudaStream_t s);

// Tensor map of bytes, dims[0] innermost, strides of dims 1-3, boxes not swizzled (api.cu).
bool make_tmap_4d_bytes(CUtensorMap* out, const void* base, const uint64_t dims[4], const uint64_t strides_bytes[3],
                        const uint32_t box[4], std::string* why);
// Items of two tiles of 128 / G positions each, bf16 or 4-bit pages, units of 128 keys.
cudaError_t launch_paged_tc(int format, int group, const PagedAttn& a, cudaStream_t s, std::string* why);
// Up to 16 rows (positions * G) an item, bf16 or 4-bit pages.
cudaError_t launch_paged_decode(int format, int group, const PagedAttn& a, cudaStream_t s);
int paged_decode_unit(int format);
// its CTAs resident per SM (registers: the blocks in flight and the output)
constexpr int paged_decode_ctas(bool int4, int row_tiles) {
    return int4 && row_tiles == 1 ? 3 : 2;
}

#ifdef __CUDACC__
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Capped logits, cap tanh(u) with u = x / cap.  The quotient 1 - 2 / (1 + exp(2u)) is
// off by about 2^-22 whatever u is, so a logit by cap 2^-22: up to a cap of 64,
// 2^-16, far below what weights in 16 bits show.  A larger cap would drown logits far
// below it, so there u up to 2/5 goes by the series to u^9, off by 2^-20 of u at most.
constexpr float kTanhSeries = 0.4f, kCapQuotient = 64.f;
__device__ __forceinline__ float2 tanh_series(float2 u) {
    const float2 v = __fmul2_rn(u, u);
    float2 y = __ffma2_rn(v, make_float2(62.f / 2835.f, 62.f / 2835.f), make_float2(-17.f / 315.f, -17.f / 315.f));
    y = __ffma2_rn(v, y, make_float2(2.f / 15.f, 2.f / 15.f));
    y = __ffma2_rn(v, y, make_float2(-1.f / 3.f, -1.f / 3.f));
    return __ffma2_rn(__fmul2_rn(u, v), y, u);
}
constexpr float kTwoLog2e = 2.f * 1.4426950408889634f;
__device__ __forceinline__ float tanh_quotient(float e2u) {   // of 2u in base 2
    return fmaf(-2.f, __fdividef(1.f, 1.f + ex2(e2u)), 1.f);
}
// Which of the two is a matter of the logit alone.
__device__ __forceinline__ float2 tanh_either(float2 u) {
    const float2 y = tanh_series(u);
    return make_float2(fabsf(u.x) <= kTanhSeries ? y.x : tanh_quotient(u.x * kTwoLog2e),
                       fabsf(u.y) <= kTanhSeries ? y.y : tanh_quotient(u.y * kTwoLog2e));
}

// Dynamic shared memory above 48 KB for a kernel: set once per device.
template <typename... A>
cudaError_t allow_smem(void (*kernel)(A...), int bytes, std::atomic<uint64_t>* done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (done->load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_relaxed);
    return e;
}

__device__ __forceinline__ void paged_err(int* err, int bit, int detail) {
    if (atomicOr(&err[0], bit) == 0) err[1] = detail;
}

// First page row of (page, head), in rows; a page outside the pool is
// reported and page 0 taken in its place, so no access leaves the pool.
__device__ __forceinline__ int paged_id(const PagedView& p, int id) {
    if ((unsigned)id >= (unsigned)p.n_pages) {
        paged_err(p.err, DEV_ERR_INDEX, id);
        return 0;
    }
    return id;
}
__device__ __forceinline__ int64_t paged_row(const PagedView& p, int page, int slot, int head) {
    return page * p.page_stride + slot * p.slot_stride + head * p.head_stride;
}

// Rows of sequence b; offsets that begin before or past 0 (the first sequence's),
// fall or pass n_rows give none and are reported.
__device__ __forceinline__ int paged_seq_rows(const PagedView& p, const PagedRows& r, int b, int* row0) {
    const int a = r.cu[b], e = r.cu[b + 1];
    *row0 = a;
    if (a < 0 || (b == 0 && a != 0) || e < a || e > r.n_rows) {
        paged_err(p.err, DEV_ERR_INDEX, b);
        return 0;
    }
    return e - a;
}

// Keys a row of sequence b may see: [lo, hi), both brought into [0, kv_len] so
// that differences with key numbers stay in range whatever the arrays hold.
__device__ __forceinline__ void paged_interval(const PagedAttn& a, int row, int kv_len, int* lo, int* hi) {
    const int g = a.r.pos[row];
    *lo = a.key_begin ? min(max(a.key_begin[row], 0), kv_len) : 0;
    *hi = max(min(a.key_end ? a.key_end[row] : (g < 0x7fffffff ? g + 1 : g), kv_len), 0);
}
__device__ __forceinline__ int paged_kv_len(const PagedView& p, int b) {
    return min(max(p.kv_len[b], 0), p.capacity);
}

// Keys that the rows of item i can see, its units, and the checks of its
// sequence's row range.  Lanes lane, lane + step, ... of a step-wide group share
// the rows and all get the answer (step 1: a thread for itself).
template <int kStep>
__device__ __forceinline__ PagedItem paged_item(const PagedAttn& a, int i, int lane) {
    PagedItem it{};
    const int b = i / a.tiles, t = i - b * a.tiles;
    int row0;
    const int n = paged_seq_rows(a.p, a.r, b, &row0);
    if (t == 0 && lane == 0) {
        if (n > a.max_rows) paged_err(a.p.err, DEV_ERR_INDEX, n);
        const int kv = a.p.kv_len[b];
        if (kv < 0 || kv > a.p.capacity) paged_err(a.p.err, DEV_ERR_INDEX, kv);
    }
    const int r0 = t * a.positions, r1 = min(min(n, a.max_rows), r0 + a.positions);
    if (r0 >= r1) return it;
    const int kv = paged_kv_len(a.p, b);
    int lo = 0x7fffffff, hi = 0, least = 0;
    for (int r = row0 + r0 + lane; r < row0 + r1; r += kStep) {
        least = min(least, a.r.pos[r]);
        int l, h;
        paged_interval(a, r, kv, &l, &h);
        if (l < h) {
            lo = min(lo, l);
            hi = max(hi, h);
        }
    }
    if (least < 0) paged_err(a.p.err, DEV_ERR_INDEX, least);
    if (kStep == 32) {
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
    }
    if (lo >= hi) lo = hi = 0;   // nothing visible: one unit without keys, which writes the zeros
    it.klo = lo;
    it.khi = hi;
    it.seq = b;
    it.kv = kv;
    it.row0 = row0 + r0;
    it.rows = r1 - r0;
    it.units = max(1, (hi + a.unit_keys - 1) / a.unit_keys - lo / a.unit_keys);
    return it;
}

// Shares in use of a line of length T: each longer than a run's start, so none is without units.
__device__ __forceinline__ int paged_shares(const PagedAttn& a, long long T) {
    return (int)min((long long)a.n_cta, T > 0 ? max(T / (a.run_cost + 1), 1ll) : 0ll);
}
// Share c of n, given the item its place falls into.
__device__ __forceinline__ PagedShare paged_share(const PagedAttn& a, int u0, int i, const PagedItem& it) {
    const int H = a.p.n_kv_heads, len = it.units + a.run_cost, rem = u0 - H * it.before, head = rem / len;
    const int run = H * it.before + head * len;
    return PagedShare{i, head, max(u0 - run - a.run_cost, 0), u0, run, it};
}

// The call's items in shared memory and this CTA's share of their units, derived
// by every CTA of 128 threads for itself from the lengths and positions: a few
// dependent loads and a scan, instead of two launches before this one.  Thread i
// takes items 2 i, 2 i + 1.
__device__ __forceinline__ PagedShare paged_inline_share(const PagedAttn& a, PagedItem* items, int* u1) {
    constexpr int kWarps = kPagedInline / 64;
    __shared__ int sums[kWarps];
    __shared__ PagedShare out;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    PagedItem it[2] = {};
#pragma unroll
    for (int e = 0; e < 2; ++e)
        if (2 * (int)threadIdx.x + e < a.n_items) it[e] = paged_item<1>(a, 2 * threadIdx.x + e, 0);
    const int cost[2] = {it[0].units ? it[0].units + a.run_cost : 0, it[1].units ? it[1].units + a.run_cost : 0};
    int incl = cost[0] + cost[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int total = 0, before = incl - cost[0] - cost[1];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    const int H = a.p.n_kv_heads;
    const long long T = (long long)total * H;
    const int n = paged_shares(a, T), c = blockIdx.x;
    const int u0 = c < n ? (int)(T * c / n) : (int)T;
    if (threadIdx.x == 0) out = PagedShare{-1, 0, 0, u0, u0, {}};
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        it[e].before = before + (e ? cost[0] : 0);
        const int i = 2 * threadIdx.x + e;
        if (i < a.n_items) items[i] = it[e];
        const long long rem = (long long)u0 - (long long)H * it[e].before;
        if (c < n && rem >= 0 && rem < (long long)H * cost[e]) out = paged_share(a, u0, i, it[e]);
    }
    __syncthreads();
    const PagedShare sh = out;
    *u1 = c + 1 < n ? (int)(T * (c + 1) / n) : (int)T;
    if (threadIdx.x == 0) {   // for the merge
        a.shares[c] = sh;
        if (c == (int)gridDim.x - 1) a.shares[c + 1] = PagedShare{-1, 0, 0, (int)T, (int)T, {}};
    }
    return sh;
}

// The runs of a CTA's share in order: n units of head h of item i from unit off.
struct PagedWalk {
    PagedItem it;
    int i, h, off, run, u1, n;
    bool first;   // the share's first run: its partial goes to slot 0, another's to slot 1
    __device__ __forceinline__ PagedWalk(const PagedAttn& a, const PagedShare& sh, int end)
        : it(sh.first), i(sh.item), h(sh.head), off(sh.off), run(sh.run), u1(end), first(true) {
        n = sh.item < 0 ? 0 : min(it.units, u1 - run - a.run_cost) - off;
    }
    __device__ __forceinline__ bool live() const { return n > 0; }
    __device__ __forceinline__ bool whole() const { return n == it.units; }
    __device__ __forceinline__ void next(const PagedAttn& a, const PagedItem* items) {
        run += it.units + a.run_cost;
        off = 0;
        first = false;
        if (++h == a.p.n_kv_heads) {
            h = 0;
            if (run < u1) {
                do it = items[++i];
                while (it.units == 0);
            }
        }
        n = min(it.units, u1 - run - a.run_cost);
    }
};
#endif

}  // namespace kvr
