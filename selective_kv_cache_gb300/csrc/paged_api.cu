// paged_api.cu -- the paged cache's C entry points: host-side validation, the
// choice of kernel, and the workspace's layout.
#include <algorithm>
#include <cmath>
#include <string>

#include "paged.h"

namespace kvr {
namespace {

#define KVR_CHECK_LAUNCH(expr, what)                            \
    do {                                                        \
        cudaError_t e_ = (expr);                                \
        if (e_ != cudaSuccess) return cuda_fail(e_, what);      \
    } while (0)

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

kvr_status fail(kvr_status st, const char* msg) {
    set_error(msg);
    return st;
}

int element(const kvr_pages* p) { return p->format == KVR_F32 ? 4 : 2; }   // bytes of a q/k/v/out element

kvr_status check_pages(const kvr_pages* p) {
    if (!p) return fail(KVR_EINVAL, "pages is NULL");
    if (p->format != KVR_F32 && p->format != KVR_BF16 && p->format != KVR_INT4)
        return fail(KVR_EINVAL, "pages: unknown format");
    if (p->n_kv_heads < 1 || p->n_pages < 1 || p->batch < 1 || p->max_pages < 1)
        return fail(KVR_EINVAL, "pages: n_kv_heads, n_pages, batch and max_pages must be positive");
    if (p->head_dim != 128 && !(p->format == KVR_F32 && p->head_dim == 64))
        return fail(KVR_EUNSUPPORTED, "pages: head_dim must be 128 (64 or 128 in fp32)");
    if (p->page_size < 16 || p->page_size > 256 || (p->page_size & (p->page_size - 1)))
        return fail(KVR_EUNSUPPORTED, "pages: page_size must be 16, 32, 64, 128 or 256");
    if (p->format == KVR_INT4 ? (p->group != 32 && p->group != 64 && p->group != 128) : p->group != 0)
        return fail(KVR_EINVAL, "pages: group must be 32, 64 or 128 for 4-bit pages and 0 otherwise");
    if (p->n_kv_heads > 65535 || (int64_t)p->max_pages * p->page_size > (int64_t(1) << 30) ||
        p->batch > (1 << 20))
        return fail(KVR_EUNSUPPORTED, "pages: more than 65535 heads, 2^20 sequences or 2^30 positions of a sequence");
    if (p->page_stride < 1 || p->head_stride < 1 || p->slot_stride < 1)
        return fail(KVR_EINVAL, "pages: strides must be positive");
    if (p->page_stride > (int64_t(1) << 21) || p->slot_stride > (int64_t(1) << 21) ||
        p->head_stride > (int64_t(1) << 31))
        return fail(KVR_EUNSUPPORTED, "pages: page and slot strides above 2^21 rows or head strides above 2^31");
    if (!p->k || !p->v || !aligned16(p->k) || !aligned16(p->v))
        return fail(KVR_EINVAL, "pages: k and v must be non-NULL and 16-byte aligned");
    if (p->format == KVR_INT4 && (!p->k_scale || !p->v_scale || !aligned16(p->k_scale) || !aligned16(p->v_scale)))
        return fail(KVR_EINVAL, "pages: 4-bit pages need 16-byte aligned scale arrays");
    if (!p->page_table || !p->kv_len || !p->err || !aligned4(p->page_table) || !aligned4(p->kv_len) ||
        !aligned4(p->err))
        return fail(KVR_EINVAL, "pages: page_table, kv_len and err must be non-NULL int32 arrays");
    return KVR_OK;
}

kvr_status check_rows(int32_t n_rows, const int32_t* cu_rows, const int32_t* positions) {
    if (n_rows < 0) return fail(KVR_EINVAL, "n_rows is negative");
    if (n_rows > 0 && (!cu_rows || !positions || !aligned4(cu_rows) || !aligned4(positions)))
        return fail(KVR_EINVAL, "cu_rows and positions must be non-NULL int32 arrays");
    return KVR_OK;
}

// A packed-row operand: `heads` heads of head_dim elements every `stride`.
bool row_operand(const kvr_pages* p, const void* x, int64_t stride, int heads) {
    return x && aligned16(x) && stride >= (int64_t)heads * p->head_dim && (stride * element(p)) % 16 == 0;
}

PagedView view(const kvr_pages* p) {
    PagedView v{};
    v.k = static_cast<uint8_t*>(p->k);
    v.v = static_cast<uint8_t*>(p->v);
    v.ks = static_cast<uint8_t*>(p->k_scale);
    v.vs = static_cast<uint8_t*>(p->v_scale);
    v.table = p->page_table;
    v.kv_len = p->kv_len;
    v.err = p->err;
    v.page_stride = p->page_stride;
    v.head_stride = p->head_stride;
    v.slot_stride = p->slot_stride;
    v.n_pages = p->n_pages;
    v.batch = p->batch;
    v.max_pages = p->max_pages;
    v.n_kv_heads = p->n_kv_heads;
    v.capacity = p->max_pages * p->page_size;
    while ((1 << v.page_shift) < p->page_size) ++v.page_shift;
    return v;
}

// Geometry of an attention call: which kernel, its item and share sizes.
struct Geometry {
    int G, positions, tiles, n_items, unit_keys, run_cost, n_cta, tile_rows;
    bool decode, tc;
};
constexpr int kSimtRows = 16, kSimtKeys = 32;

kvr_status geometry(const kvr_pages* p, int32_t n_q_heads, int32_t n_rows, int32_t max_rows, Geometry* g) {
    if (n_q_heads < 1 || n_q_heads % p->n_kv_heads)
        return fail(KVR_EINVAL, "n_q_heads must be a multiple of n_kv_heads");
    g->G = n_q_heads / p->n_kv_heads;
    if (g->G > kPagedMaxGroup) return fail(KVR_EUNSUPPORTED, "more than 16 query heads per K/V head");
    if (max_rows < 1) return fail(KVR_EINVAL, "max_rows must be positive");
    max_rows = std::min(max_rows, n_rows);
    // Which kernel, from what the host knows: row groups of 16 of a K/V head
    // (passes over its keys on mma.sync) and the most 128-key units there can be.
    // The mma.sync kernel reads the keys once per pass, needs no plan and splits
    // finely; the tcgen05 one reads them once, at 1.6 us (bf16) and 2 us (4 bits) a
    // unit of up to 256 rows, and starts later.  Measured (us, mma.sync / tcgen05,
    // 8 K/V heads, rows per head): bf16, one sequence of 8192 keys 64 rows 30 / 39,
    // 128 rows 39 / 40; 3 x 5001 keys 48 rows 29 / 32, 64 rows 35 / 33; 8 x 8192 24
    // rows 57 / 54, 64 rows 95 / 56.  4 bits: 32 x 8192 32 rows 124 / 149, 48 rows
    // 162 / 141; 8 x 8192 48 rows 52 / 53, 64 rows 67 / 55; 3 x 5001 64 rows 31 / 36,
    // 128 rows 38 / 35; 1 x 8192 128 rows 36 / 43.
    // The rule knows the table's width, not the lengths, so sequences of 2048 keys in
    // a table of 131072 go to tcgen05 sooner than in one of their own width: bf16, one
    // sequence 32 rows 28 us in place of 26, 64 rows 30 in place of 27, 8 sequences 32
    // rows 39 in place of 44; 4 bits, one sequence 64 rows 32 in place of 24, 8
    // sequences 64 rows 40 in place of 48.
    const int64_t passes = ((int64_t)max_rows * g->G + 15) / 16;
    const int64_t bound = std::min<int64_t>(passes, 9) * p->batch * p->n_kv_heads *   // below 2^63; not asked past 8
                          (((int64_t)p->max_pages * p->page_size + 127) / 128);
    g->decode = p->format == KVR_BF16 ? passes == 1 || (passes <= 8 && bound <= 3600)
                                      : p->format == KVR_INT4 && (passes <= 2 || (passes <= 8 && bound <= 5500));
    g->tc = p->format != KVR_F32 && !g->decode;
    if (g->decode) {
        g->tile_rows = max_rows * g->G <= 8 ? 8 : 16;
        g->unit_keys = paged_decode_unit(p->format);
        g->n_cta = paged_decode_ctas(p->format == KVR_INT4, g->tile_rows / 8) * kNumSMs;
    } else if (g->tc) {
        g->tile_rows = 256;
        g->unit_keys = 128;
        // a run's start and end (rows and Q looked up, first scores and last product with
        // nothing beside them, O out), in units; 2, 4 and 6: 8192 causal rows 390, 366,
        // 376 us (4 bits 498, 441, 450), packed documents 114, 103, 105
        g->run_cost = 4;
        g->n_cta = kNumSMs;
    } else {
        g->tile_rows = kSimtRows;
        g->unit_keys = kSimtKeys;
        g->n_cta = 4 * kNumSMs;
    }
    g->positions = g->tc ? 2 * (128 / g->G) : g->tile_rows / g->G;
    g->tiles = (max_rows + g->positions - 1) / g->positions;
    const int64_t items = (int64_t)g->tiles * p->batch;
    // A run's start is worth more when there are runs for every CTA anyway; with few,
    // splitting them finely is.  0, 1 and 3 (us): decode 64 x 300 keys 39, 37, 33 (4
    // bits 29, 27, 26), 4 drafted rows x 3 x 5001 keys 29, 25, 25, 1 x 1000 keys 17,
    // 17, 19.  In fp32 the units themselves outweigh it (4 x 500 keys 19 with 0, 23 with 1).
    // These are captured calls alone on the GPU with inputs out of L2; one call after
    // another takes less (1 x 1000 keys 12).
    if (!g->tc) g->run_cost = !g->decode ? 0 : items * p->n_kv_heads >= g->n_cta ? 3 : 1;
    // shares and items are counted in 32 bits
    const int64_t units = ((int64_t)p->max_pages * p->page_size + g->unit_keys - 1) / g->unit_keys + g->run_cost;
    if (items > (int64_t(1) << 28) || units * p->n_kv_heads >= (int64_t(1) << 31) ||
        items * (units * p->n_kv_heads) >= (int64_t(1) << 31))   // each factor first: the product of all can pass 2^63
        return fail(KVR_EUNSUPPORTED, "batch * rows * keys is too large for one call");
    g->n_items = (int)items;
    return KVR_OK;
}

struct Ws {
    size_t items, shares, part_o, part_ml, total;
};
Ws ws_layout(const kvr_pages* p, const Geometry& g) {
    auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
    const size_t rows = (size_t)g.n_cta * 2 * g.tile_rows;
    Ws w;
    w.items = 0;
    w.shares = w.items + al((size_t)g.n_items * sizeof(PagedItem));
    w.part_o = w.shares + al((size_t)(g.n_cta + 1) * sizeof(PagedShare));
    w.part_ml = w.part_o + al(rows * p->head_dim * sizeof(float));
    w.total = w.part_ml + al(rows * 2 * sizeof(float));
    return w;
}

}  // namespace
}  // namespace kvr

using namespace kvr;

extern "C" {

kvr_status kvr_paged_append(const kvr_pages* p, int32_t n_rows, const int32_t* cu_rows, const int32_t* positions,
                            const void* k_rows, int64_t k_stride, const void* v_rows, int64_t v_stride,
                            const float* rope, int32_t rope_len, const void* q_rows, int64_t q_stride, void* q_out,
                            int32_t n_q_heads, void* stream) {
    pdl_begin_call();   // no overlap with work enqueued before this call
    kvr_status st = check_pages(p);
    if (st != KVR_OK) return st;
    if ((st = check_rows(n_rows, cu_rows, positions)) != KVR_OK) return st;
    if (n_rows == 0) return KVR_OK;
    if (!row_operand(p, k_rows, k_stride, p->n_kv_heads) || !row_operand(p, v_rows, v_stride, p->n_kv_heads))
        return fail(KVR_EINVAL, "append: K/V rows must be non-NULL, 16-byte aligned and at least a row apart");
    if (rope && (rope_len < 1 || !aligned16(rope)))
        return fail(KVR_EINVAL, "append: the rope table needs rope_len >= 1 and 16-byte alignment");
    if ((q_rows == nullptr) != (q_out == nullptr)) return fail(KVR_EINVAL, "append: q_rows and q_out go together");
    if (q_rows) {
        if (n_q_heads < 1 || n_q_heads > 65535) return fail(KVR_EINVAL, "append: n_q_heads out of range");
        if (!row_operand(p, q_rows, q_stride, n_q_heads) || !aligned16(q_out))
            return fail(KVR_EINVAL, "append: query rows must be 16-byte aligned and at least a row apart");
        if (q_rows == q_out && n_rows > 1 && q_stride != (int64_t)n_q_heads * p->head_dim)
            return fail(KVR_EINVAL, "append: queries are rotated in place only when they are packed");
    }
    PagedRowIo a{};
    const int es = element(p);
    a.p = view(p);
    a.r = PagedRows{cu_rows, positions, n_rows};
    a.k_in = static_cast<const uint8_t*>(k_rows);
    a.v_in = static_cast<const uint8_t*>(v_rows);
    a.q_in = static_cast<const uint8_t*>(q_rows);
    a.q_out = static_cast<uint8_t*>(q_out);
    a.k_stride = k_stride * es;
    a.v_stride = v_stride * es;
    a.q_stride = q_stride * es;
    a.rope = reinterpret_cast<const float2*>(rope);
    a.rope_len = rope_len;
    a.n_q_heads = n_q_heads;
    KVR_CHECK_LAUNCH(launch_paged_append(p->format, p->head_dim, p->group, a, reinterpret_cast<cudaStream_t>(stream)),
                     "paged append");
    return KVR_OK;
}

kvr_status kvr_paged_read(const kvr_pages* p, int32_t n_rows, const int32_t* cu_rows, const int32_t* positions,
                          void* k_out, int64_t k_stride, void* v_out, int64_t v_stride, void* stream) {
    pdl_begin_call();   // no overlap with work enqueued before this call
    kvr_status st = check_pages(p);
    if (st != KVR_OK) return st;
    if ((st = check_rows(n_rows, cu_rows, positions)) != KVR_OK) return st;
    if (n_rows == 0) return KVR_OK;
    if ((k_out && !row_operand(p, k_out, k_stride, p->n_kv_heads)) ||
        (v_out && !row_operand(p, v_out, v_stride, p->n_kv_heads)))
        return fail(KVR_EINVAL, "read: output rows must be 16-byte aligned and at least a row apart");
    if (!k_out && !v_out) return KVR_OK;
    PagedRowIo a{};
    const int es = element(p);
    a.p = view(p);
    a.r = PagedRows{cu_rows, positions, n_rows};
    a.k_out = static_cast<uint8_t*>(k_out);
    a.v_out = static_cast<uint8_t*>(v_out);
    a.k_stride = k_stride * es;
    a.v_stride = v_stride * es;
    KVR_CHECK_LAUNCH(launch_paged_read(p->format, p->head_dim, p->group, a, reinterpret_cast<cudaStream_t>(stream)),
                     "paged read");
    return KVR_OK;
}

size_t kvr_paged_workspace_bytes(const kvr_pages* p, int32_t n_q_heads, int32_t n_rows, int32_t max_rows) {
    Geometry g;
    if (check_pages(p) != KVR_OK || n_rows < 1 || geometry(p, n_q_heads, n_rows, max_rows, &g) != KVR_OK) return 0;
    return ws_layout(p, g).total;
}

kvr_status kvr_paged_attend(const kvr_pages* p, const kvr_score_opts* opts, int32_t n_q_heads, int32_t n_rows,
                            int32_t max_rows, const int32_t* cu_rows, const int32_t* positions, const void* q,
                            int64_t q_stride, void* out, int64_t out_stride, void* workspace, size_t ws_bytes,
                            void* stream) {
    pdl_begin_call();   // no overlap with work enqueued before this call
    kvr_status st = check_pages(p);
    if (st != KVR_OK) return st;
    if ((st = check_rows(n_rows, cu_rows, positions)) != KVR_OK) return st;
    kvr_score_opts o{};
    if (opts) o = *opts;
    // within these a product with log2 e or 2 / softcap is neither infinite nor zero
    auto usable = [](float x) { return x == 0.f || (x >= 0x1p-64f && x <= 0x1p64f); };
    if (!usable(o.scale) || !usable(o.softcap) || !std::isfinite(o.alpha) || !std::isfinite(o.beta))
        return fail(KVR_EINVAL, "attend: scale and softcap must be 0 or in [2^-64, 2^64], alpha and beta finite");
    if (!aligned4(o.local_bits) || !aligned4(o.sink_bits) || !aligned4(o.slopes) || !aligned4(o.key_begin) ||
        !aligned4(o.key_end))
        return fail(KVR_EINVAL, "attend: misaligned option array");
    if (n_rows == 0) return KVR_OK;
    Geometry g;
    if ((st = geometry(p, n_q_heads, n_rows, max_rows, &g)) != KVR_OK) return st;
    if (!row_operand(p, q, q_stride, n_q_heads) || !row_operand(p, out, out_stride, n_q_heads))
        return fail(KVR_EINVAL, "attend: q and out rows must be non-NULL, 16-byte aligned and at least a row apart");
    const Ws w = ws_layout(p, g);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || ws_bytes < w.total)
        return fail(KVR_EINVAL, "attend: workspace is NULL, not 256-byte aligned or below kvr_paged_workspace_bytes");
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    PagedAttn a{};
    a.p = view(p);
    a.r = PagedRows{cu_rows, positions, n_rows};
    a.q = q;
    a.out = out;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.n_q_heads = n_q_heads;
    a.G = g.G;
    a.max_rows = std::min(max_rows, n_rows);
    a.positions = g.positions;
    a.tiles = g.tiles;
    a.n_items = g.n_items;
    a.unit_keys = g.unit_keys;
    a.run_cost = g.run_cost;
    a.n_cta = g.n_cta;
    a.tile_rows = g.tile_rows;
    a.scale = o.scale > 0.f ? o.scale : (float)(1.0 / std::sqrt((double)p->head_dim));
    a.softcap = o.softcap;
    // a bias this large decides alone; clamped so that logits in base 2 stay finite
    a.alpha = std::min(std::max(o.alpha, -1e37f), 1e37f);
    a.beta = std::min(std::max(o.beta, -1e37f), 1e37f);
    a.loc = o.alpha != 0.f ? o.local_bits : nullptr;
    a.snk = o.beta != 0.f ? o.sink_bits : nullptr;
    a.slopes = o.slopes;
    a.key_begin = o.key_begin;
    a.key_end = o.key_end;
    a.words = (a.p.capacity + 31) / 32;
    a.items = reinterpret_cast<PagedItem*>(ws + w.items);
    a.shares = reinterpret_cast<PagedShare*>(ws + w.shares);
    a.part_o = reinterpret_cast<float*>(ws + w.part_o);
    a.part_ml = reinterpret_cast<float*>(ws + w.part_ml);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    std::string why;
    a.planned = g.tc || g.n_items > kPagedInline;
    if (a.planned) KVR_CHECK_LAUNCH(launch_paged_plan(a, s), "paged plan");
    if (g.decode) KVR_CHECK_LAUNCH(launch_paged_decode(p->format, p->group, a, s), "paged attention");
    else if (g.tc)
        KVR_CHECK_LAUNCH(launch_paged_tc(p->format, p->group, a, s, &why), ("paged attention " + why).c_str());
    else KVR_CHECK_LAUNCH(launch_paged_simt(p->head_dim, a, s), "paged attention");
    KVR_CHECK_LAUNCH(launch_paged_merge(p->format == KVR_F32 ? KVR_F32 : KVR_BF16, p->head_dim, a, s), "paged merge");
    return KVR_OK;
}

kvr_status kvr_paged_status(const kvr_pages* p, void* stream) {
    if (!p || !p->err) return fail(KVR_EINVAL, "pages or its err is NULL");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int32_t w[4] = {0, 0, 0, 0};
    cudaError_t e = cudaMemcpyAsync(w, p->err, sizeof(w), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e, "paged status");
    if (w[0] == 0) return KVR_OK;
    e = cudaMemsetAsync(p->err, 0, sizeof(w), s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e, "paged status");
    if (w[0] & DEV_ERR_TIMEOUT) return fail(KVR_ETIMEOUT, "a device-side wait timed out");
    set_error(std::string("device-side check failed:") + ((w[0] & DEV_ERR_INDEX) ? " index out of range" : "") +
              ((w[0] & DEV_ERR_ORDER) ? " positions do not ascend" : "") + " (" + std::to_string(w[1]) + ")");
    return KVR_EDEVICE;
}

}  // extern "C"
