// rows_api.cu -- the packed-row operators' C entry points: host-side
// validation and the rotary frequencies.
#include <algorithm>
#include <cmath>

#include "rows.h"

namespace kvr {
namespace {

#define KVR_CHECK_LAUNCH(expr, what)                            \
    do {                                                        \
        cudaError_t e_ = (expr);                                \
        if (e_ != cudaSuccess) return cuda_fail(e_, what);      \
    } while (0)

kvr_status fail(kvr_status st, const char* msg) {
    set_error(msg);
    return st;
}

constexpr int32_t kMaxWidth = 1 << 20;
constexpr int64_t kMaxStride = int64_t(1) << 29;   // 2^31 rows of it in bytes stay below 2^63

// rows of `width` elements of `size` bytes each, `stride` elements apart
bool rows_ok(const void* p, int64_t width, int64_t stride, int size) {
    return p && reinterpret_cast<uintptr_t>(p) % size == 0 && stride >= width && stride <= kMaxStride;
}
bool dtype_ok(int32_t dtype) { return dtype == KVR_F32 || dtype == KVR_BF16; }
int size_of(int32_t dtype) { return dtype == KVR_F32 ? 4 : 2; }

kvr_status check_shape(int32_t dtype, int32_t n_rows, int32_t d) {
    if (!dtype_ok(dtype)) return fail(KVR_EINVAL, "rows: dtype must be KVR_F32 or KVR_BF16");
    if (n_rows < 0 || d < 1 || d > kMaxWidth) return fail(KVR_EINVAL, "rows: n_rows or width out of range");
    return KVR_OK;
}
kvr_status check_codes(const int8_t* codes, int64_t stride, const float* scales, int32_t d) {
    if (!rows_ok(codes, d, stride, 1) || !rows_ok(scales, 1, 1, 4))
        return fail(KVR_EINVAL, "rows: codes and scales must be non-NULL and aligned, codes at least a row apart");
    return KVR_OK;
}
// out, codes and scales of the operators that may leave one of the two forms out
kvr_status check_outputs(int32_t dtype, int32_t d, const void* out, int64_t out_stride, const int8_t* codes,
                         int64_t code_stride, const float* scales) {
    if (!out && !codes) return fail(KVR_EINVAL, "rows: neither out nor codes is given");
    if (out && !rows_ok(out, d, out_stride, size_of(dtype)))
        return fail(KVR_EINVAL, "rows: out must be aligned to its elements and at least a row apart");
    if (codes || scales) return check_codes(codes, code_stride, scales, d);
    return KVR_OK;
}

kvr_status check_weights(const kvr_linear_weights* w) {
    if (!w) return fail(KVR_EINVAL, "weights is NULL");
    if (w->n_out < 1 || w->n_out > kMaxWidth || w->k < 1 || w->k > 65536)
        return fail(KVR_EINVAL, "weights: n_out or k out of range");
    if (!rows_ok(w->codes, w->k, w->stride, 16) || w->stride % 16)
        return fail(KVR_EINVAL, "weights: codes must be 16-byte aligned, their stride a multiple of 16 and at least a row");
    if (!rows_ok(w->scales, 1, 1, 4) || (w->bias && !rows_ok(w->bias, 1, 1, 4)) || !rows_ok(w->err, 1, 1, 4))
        return fail(KVR_EINVAL, "weights: scales, bias and err must be aligned, scales and err not NULL");
    return KVR_OK;
}
// Which kernel a call takes, measured on GB300 with weights from HBM (us):
//   rows x k -> n_out        integer    batch    tiles
//    8 x  4096 ->  6144          8.2     11.0     17.4
//    8 x  4096 -> 28672         22.7     25.8     31.4
//    9 x  4096 ->  6144         12.0     11.3     17.4
//   16 x 14336 ->  4096         25.1     15.7     42.1
//   64 x  4096 -> 28672                  30.3     32.2
//   64 x 14336 ->  4096                  19.2     43.9
//   96 x  4096 -> 28672                  40.0     32.9
//  128 x  1536 ->  2048                   7.5     10.5
//  128 x  4096 ->  4096                  13.1     17.7
//  128 x 18944 ->  3584                  32.3     57.1
//  192 x 14336 ->  4096                  41.8     45.1
//  256 x  4096 ->  4096                  17.2     17.9
//  320 x  4096 ->  4096                  25.0     18.2
//  256 x  8960 ->  1536                  19.5     30.5
//  320 x  1536 ->  2048                   9.0     10.5
// 1024 x  1536 ->  2048                  14.6     12.2
// Above 64 rows the batch kernel reads the weights once for every 64 of them,
// and splits k where the tiles are few: the two estimates decide.
enum class LinearWay { Mma, Few, Tc };
LinearWay linear_way(int n_out, int k, int n_rows) {
    if (n_rows <= kLinearMmaRows) return LinearWay::Mma;
    if (n_rows <= 64) return LinearWay::Few;
    return n_rows <= 4096 && linear_few_us(n_out, k, n_rows) < linear_tc_us(n_out, k, n_rows) ? LinearWay::Few : LinearWay::Tc;
}
// grows with n_rows, whichever kernel takes them
size_t linear_workspace(const kvr_linear_weights& w, int32_t n_rows) {
    return std::max<size_t>(256, n_rows > 64 ? linear_tc_workspace(w.k, n_rows) : 0);
}

kvr_status check_rope(const kvr_rope* r) {
    if (!r) return fail(KVR_EINVAL, "rope is NULL");
    if (r->head_dim < 2 || r->head_dim > 256 || r->head_dim % 2 || r->rotary_dim < 2 || r->rotary_dim > r->head_dim ||
        r->rotary_dim % 2)
        return fail(KVR_EINVAL, "rope: head_dim and rotary_dim must be even, rotary_dim <= head_dim <= 256");
    if (r->layout != KVR_ROPE_HALF && r->layout != KVR_ROPE_INTERLEAVED) return fail(KVR_EINVAL, "rope: unknown layout");
    if (!(r->attn >= 0x1p-64f && r->attn <= 0x1p64f)) return fail(KVR_EINVAL, "rope: attn must lie in [2^-64, 2^64]");
    return KVR_OK;
}

}  // namespace
}  // namespace kvr

using namespace kvr;

extern "C" {

kvr_status kvr_rows_norm(int32_t dtype, int32_t n_rows, int32_t d, const void* x, int64_t x_stride,
                         const void* residual, int64_t residual_stride, void* sum_out, int64_t sum_stride,
                         const void* weight, float eps, void* out, int64_t out_stride, int8_t* codes,
                         int64_t code_stride, float* scales, void* stream) {
    pdl_begin_call();   // no overlap with work enqueued before this call
    kvr_status st = check_shape(dtype, n_rows, d);
    if (st != KVR_OK) return st;
    const int es = size_of(dtype);
    if (!rows_ok(x, d, x_stride, es) || !rows_ok(weight, d, d, es) || (residual && !rows_ok(residual, d, residual_stride, es)) ||
        (sum_out && !rows_ok(sum_out, d, sum_stride, es)))
        return fail(KVR_EINVAL, "norm: x and weight must be non-NULL, every array aligned to its elements, rows at least "
                                "a row apart");
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(KVR_EINVAL, "norm: eps must be finite and not negative");
    if ((st = check_outputs(dtype, d, out, out_stride, codes, code_stride, scales)) != KVR_OK) return st;
    auto clash = [&](const void* o, int64_t os, const void* i, int64_t is) { return o && o == i && os != is && n_rows > 1; };
    if (clash(sum_out, sum_stride, x, x_stride) || clash(sum_out, sum_stride, residual, residual_stride) ||
        clash(out, out_stride, x, x_stride) || clash(out, out_stride, residual, residual_stride) || (out && out == sum_out))
        return fail(KVR_EINVAL, "norm: an output in an input's place takes its stride, and out is not sum_out");
    if (n_rows == 0) return KVR_OK;
    RowsQuant a{};
    a.x = static_cast<const uint8_t*>(x);
    a.res = static_cast<const uint8_t*>(residual);
    a.weight = static_cast<const uint8_t*>(weight);
    a.sum = static_cast<uint8_t*>(sum_out);
    a.out = static_cast<uint8_t*>(out);
    a.codes = codes;
    a.scales = scales;
    a.x_stride = x_stride;
    a.res_stride = residual_stride;
    a.sum_stride = sum_stride;
    a.out_stride = out_stride;
    a.code_stride = code_stride;
    a.n_rows = n_rows;
    a.d = d;
    a.eps = eps;
    KVR_CHECK_LAUNCH(launch_rows_quant(RowOp::Norm, dtype, a, reinterpret_cast<cudaStream_t>(stream)), "rows norm");
    return KVR_OK;
}

kvr_status kvr_rows_swiglu(int32_t dtype, int32_t n_rows, int32_t d, const void* gate_up, int64_t stride, void* out,
                           int64_t out_stride, int8_t* codes, int64_t code_stride, float* scales, void* stream) {
    pdl_begin_call();
    kvr_status st = check_shape(dtype, n_rows, d);
    if (st != KVR_OK) return st;
    if (!rows_ok(gate_up, 2 * (int64_t)d, stride, size_of(dtype)))
        return fail(KVR_EINVAL, "swiglu: gate_up must be non-NULL, aligned to its elements and at least 2 d apart");
    if ((st = check_outputs(dtype, d, out, out_stride, codes, code_stride, scales)) != KVR_OK) return st;
    if (out == gate_up) return fail(KVR_EINVAL, "swiglu: out may not be gate_up");
    if (n_rows == 0) return KVR_OK;
    RowsQuant a{};
    a.x = static_cast<const uint8_t*>(gate_up);
    a.out = static_cast<uint8_t*>(out);
    a.codes = codes;
    a.scales = scales;
    a.x_stride = stride;
    a.out_stride = out_stride;
    a.code_stride = code_stride;
    a.n_rows = n_rows;
    a.d = d;
    KVR_CHECK_LAUNCH(launch_rows_quant(RowOp::Swiglu, dtype, a, reinterpret_cast<cudaStream_t>(stream)), "rows swiglu");
    return KVR_OK;
}

kvr_status kvr_rows_quantise(int32_t dtype, int32_t n_rows, int32_t d, const void* x, int64_t x_stride, int8_t* codes,
                             int64_t code_stride, float* scales, void* stream) {
    pdl_begin_call();
    kvr_status st = check_shape(dtype, n_rows, d);
    if (st != KVR_OK) return st;
    if (!rows_ok(x, d, x_stride, size_of(dtype)))
        return fail(KVR_EINVAL, "quantise: x must be non-NULL, aligned to its elements and at least a row apart");
    if ((st = check_codes(codes, code_stride, scales, d)) != KVR_OK) return st;
    if (n_rows == 0) return KVR_OK;
    RowsQuant a{};
    a.x = static_cast<const uint8_t*>(x);
    a.codes = codes;
    a.scales = scales;
    a.x_stride = x_stride;
    a.code_stride = code_stride;
    a.n_rows = n_rows;
    a.d = d;
    KVR_CHECK_LAUNCH(launch_rows_quant(RowOp::Quantise, dtype, a, reinterpret_cast<cudaStream_t>(stream)), "rows quantise");
    return KVR_OK;
}

kvr_status kvr_rows_dequantise(int32_t dtype, int32_t n_rows, int32_t d, const int8_t* codes, int64_t code_stride,
                               const float* scales, void* out, int64_t out_stride, void* stream) {
    pdl_begin_call();
    kvr_status st = check_shape(dtype, n_rows, d);
    if (st != KVR_OK) return st;
    if ((st = check_codes(codes, code_stride, scales, d)) != KVR_OK) return st;
    if (!rows_ok(out, d, out_stride, size_of(dtype)))
        return fail(KVR_EINVAL, "dequantise: out must be non-NULL, aligned to its elements and at least a row apart");
    if (n_rows == 0) return KVR_OK;
    KVR_CHECK_LAUNCH(launch_rows_dequantise(dtype, n_rows, d, codes, code_stride, scales, out, out_stride,
                                            reinterpret_cast<cudaStream_t>(stream)),
                     "rows dequantise");
    return KVR_OK;
}

kvr_status kvr_rope_init(kvr_rope* rope, int32_t head_dim, int32_t rotary_dim, int32_t layout, int32_t scaling,
                         double theta, double factor, double low, double high, int32_t original_len,
                         float attn_factor) {
    if (!rope) return fail(KVR_EINVAL, "rope is NULL");
    kvr_rope r{};
    r.head_dim = head_dim;
    r.rotary_dim = rotary_dim;
    r.layout = layout;
    r.attn = 1.f;
    kvr_status st = check_rope(&r);
    if (st != KVR_OK) return st;
    if (scaling < KVR_ROPE_PLAIN || scaling > KVR_ROPE_YARN) return fail(KVR_EINVAL, "rope: unknown scaling");
    if (!(theta > 1.0) || !std::isfinite(theta) || !(factor >= 1.0) || !std::isfinite(factor))
        return fail(KVR_EINVAL, "rope: theta must be above 1 and factor at least 1");
    const bool banded = scaling == KVR_ROPE_BANDS || scaling == KVR_ROPE_YARN;
    if (banded && (!(low > 0.0) || !(high > low) || !std::isfinite(high) || original_len < 1))
        return fail(KVR_EINVAL, "rope: need 0 < low < high and original_len >= 1");
    if (scaling == KVR_ROPE_NTK && rotary_dim < 4) return fail(KVR_EINVAL, "rope: this scaling needs rotary_dim of 4 or more");
    const double two_pi = 6.283185307179586476925, rot = rotary_dim;
    const double base = scaling == KVR_ROPE_NTK ? theta * std::pow(factor, rot / (rot - 2)) : theta;
    if (!std::isfinite(base)) return fail(KVR_EINVAL, "rope: theta is out of range with this factor");
    // pair numbers at which the trained length holds `high` and `low` turns
    auto pair_at = [&](double t) { return rot * std::log(original_len / (two_pi * t)) / (2 * std::log(theta)); };
    double first = 0, last = 0;
    if (scaling == KVR_ROPE_YARN) {
        first = std::max(0.0, std::floor(pair_at(high)));
        last = std::min(rot - 1, std::ceil(pair_at(low)));
        r.attn = (float)(0.1 * std::log(factor) + 1.0);
    }
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot), keep = 1.0;   // keep: the part of f that is not interpolated
        if (scaling == KVR_ROPE_LINEAR) keep = 0.0;
        if (scaling == KVR_ROPE_BANDS) keep = std::min(1.0, std::max(0.0, (original_len * f / two_pi - low) / (high - low)));
        if (scaling == KVR_ROPE_YARN) keep = 1.0 - std::min(1.0, std::max(0.0, (i - first) / std::max(last - first, 1e-3)));
        f = f * (keep + (1.0 - keep) / factor);
        r.turns[i] = (uint64_t)std::ldexp(f / two_pi, 64);   // f <= 1: below a sixth of a turn
    }
    if (attn_factor != 0.f) r.attn = attn_factor;
    if ((st = check_rope(&r)) != KVR_OK) return st;
    *rope = r;
    return KVR_OK;
}

kvr_status kvr_rope_table(const kvr_rope* rope, int32_t rope_len, float* table, void* stream) {
    pdl_begin_call();
    kvr_status st = check_rope(rope);
    if (st != KVR_OK) return st;
    if (rope_len < 0 || !table || reinterpret_cast<uintptr_t>(table) % 8)
        return fail(KVR_EINVAL, "rope table: rope_len must not be negative, table 8-byte aligned and not NULL");
    if (rope_len == 0) return KVR_OK;
    KVR_CHECK_LAUNCH(launch_rope_table(*rope, rope_len, reinterpret_cast<float2*>(table),
                                       reinterpret_cast<cudaStream_t>(stream)),
                     "rope table");
    return KVR_OK;
}

kvr_status kvr_rows_rotate(const kvr_rope* rope, int32_t dtype, int32_t n_rows, const int32_t* positions, const void* q,
                           int64_t q_stride, int32_t n_q_heads, void* q_out, int64_t q_out_stride, const void* k,
                           int64_t k_stride, int32_t n_kv_heads, void* k_out, int64_t k_out_stride, uint32_t flags,
                           void* stream) {
    pdl_begin_call();
    kvr_status st = check_rope(rope);
    if (st != KVR_OK) return st;
    if (!dtype_ok(dtype)) return fail(KVR_EINVAL, "rotate: dtype must be KVR_F32 or KVR_BF16");
    if (n_rows < 0 || (flags & ~KVR_ROPE_INVERSE)) return fail(KVR_EINVAL, "rotate: n_rows or flags out of range");
    if (n_q_heads < 0 || n_kv_heads < 0 || n_q_heads > 65535 || n_kv_heads > 65535 || n_q_heads + n_kv_heads == 0)
        return fail(KVR_EINVAL, "rotate: head counts out of range");
    if (!positions || reinterpret_cast<uintptr_t>(positions) % 4)
        return fail(KVR_EINVAL, "rotate: positions must be non-NULL and aligned");
    RowsRotate a{};
    a.rope = *rope;
    const void* in[2] = {q, k};
    void* out[2] = {q_out, k_out};
    const int64_t is[2] = {q_stride, k_stride}, os[2] = {q_out_stride, k_out_stride};
    const int32_t heads[2] = {n_q_heads, n_kv_heads};
    for (int w = 0; w < 2; ++w) {
        const int64_t width = (int64_t)heads[w] * rope->head_dim;
        if (heads[w] == 0 ? in[w] || out[w]
                          : !rows_ok(in[w], width, is[w], size_of(dtype)) || !rows_ok(out[w], width, os[w], size_of(dtype)))
            return fail(KVR_EINVAL, "rotate: heads need aligned rows and outputs at least a row apart, and no heads neither");
        if (heads[w] && in[w] == out[w] && is[w] != os[w] && n_rows > 1)
            return fail(KVR_EINVAL, "rotate: an output in its input's place takes its stride");
        a.in[w] = static_cast<const uint8_t*>(in[w]);
        a.out[w] = static_cast<uint8_t*>(out[w]);
        a.in_stride[w] = is[w];
        a.out_stride[w] = os[w];
        a.heads[w] = heads[w];
    }
    if (n_rows == 0) return KVR_OK;
    a.pos = positions;
    a.n_rows = n_rows;
    a.inverse = (flags & KVR_ROPE_INVERSE) != 0;
    KVR_CHECK_LAUNCH(launch_rows_rotate(dtype, a, reinterpret_cast<cudaStream_t>(stream)), "rows rotate");
    return KVR_OK;
}

size_t kvr_linear_workspace_bytes(const kvr_linear_weights* w, int32_t n_rows) {
    if (check_weights(w) != KVR_OK || n_rows < 1 || n_rows > kMaxWidth * 4) return 0;
    return linear_workspace(*w, n_rows);
}

kvr_status kvr_linear(const kvr_linear_weights* w, int32_t n_rows, const int8_t* codes, int64_t stride,
                      const float* scales, int32_t dtype, void* out, int64_t out_stride, void* workspace,
                      size_t ws_bytes, void* stream) {
    pdl_begin_call();
    kvr_status st = check_weights(w);
    if (st != KVR_OK) return st;
    if (!dtype_ok(dtype)) return fail(KVR_EINVAL, "linear: dtype must be KVR_F32 or KVR_BF16");
    if (n_rows < 0 || n_rows > kMaxWidth * 4) return fail(KVR_EINVAL, "linear: n_rows out of range");
    if (!rows_ok(codes, w->k, stride, 16) || stride % 16 || !rows_ok(scales, 1, 1, 4))
        return fail(KVR_EINVAL, "linear: row codes must be 16-byte aligned, their stride a multiple of 16 and at least a "
                                "row, scales aligned");
    if (!rows_ok(out, w->n_out, out_stride, size_of(dtype)))
        return fail(KVR_EINVAL, "linear: out must be non-NULL, aligned to its elements and at least a row apart");
    if (n_rows == 0) return KVR_OK;
    const size_t need = linear_workspace(*w, n_rows);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || ws_bytes < need)
        return fail(KVR_EINVAL, "linear: workspace is NULL, not 256-byte aligned or below kvr_linear_workspace_bytes");
    Linear a{};
    a.w = w->codes;
    a.w_scale = w->scales;
    a.bias = w->bias;
    a.x = codes;
    a.x_scale = scales;
    a.out = out;
    a.w_stride = w->stride;
    a.x_stride = stride;
    a.out_stride = out_stride;
    a.n_out = w->n_out;
    a.k = w->k;
    a.n_rows = n_rows;
    a.dtype = dtype;
    a.err = w->err;
    a.workspace = workspace;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    std::string why;
    cudaError_t e = cudaSuccess;
    switch (linear_way(w->n_out, w->k, n_rows)) {
        case LinearWay::Mma: e = launch_linear_mma(a, s); break;
        case LinearWay::Few: e = launch_linear_few(a, s, &why); break;
        case LinearWay::Tc: e = launch_linear_tc(a, s, &why); break;
    }
    if (e != cudaSuccess) return cuda_fail(e, ("linear " + why).c_str());
    return KVR_OK;
}

kvr_status kvr_linear_status(const kvr_linear_weights* w, void* stream) {
    if (!w || !w->err) return fail(KVR_EINVAL, "linear: weights or their err are NULL");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int32_t e4[4] = {0, 0, 0, 0};
    cudaError_t e = cudaMemcpyAsync(e4, w->err, sizeof(e4), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e, "linear status");
    if (e4[0] == 0) return KVR_OK;
    e = cudaMemsetAsync(w->err, 0, sizeof(e4), s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e, "linear status");
    return fail((e4[0] & DEV_ERR_TIMEOUT) ? KVR_ETIMEOUT : KVR_EDEVICE, "linear: a device-side wait timed out");
}

}  // extern "C"
