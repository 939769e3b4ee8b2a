// rows.h -- packed-row operators: norms and gates into eight bits, the rotary
// map, and projections by 8-bit weights (rows_api.cu, rows_quant.cu,
// rows_rotate.cu, linear_*.cu).
#pragma once
#include "kvr_internal.h"

namespace kvr {

// Quotients by a divisor of a launch, for numerators below 2^31: umulhi with
// ceil(2^(31 + l) / d), l = ceil(log2 d), and a shift by l - 1.
struct Div {
    uint32_t d, mul, shift;
    explicit Div(uint32_t n) : d(n), mul(0), shift(0) {
        if (n == 1) return;
        uint32_t l = 0;
        while ((1u << l) < n) ++l;
        mul = (uint32_t)(((uint64_t(1) << (31 + l)) + n - 1) / n);
        shift = l - 1;
    }
#ifdef __CUDACC__
    __device__ __forceinline__ uint32_t operator()(uint32_t x) const { return d == 1 ? x : __umulhi(x, mul) >> shift; }
#endif
};

enum class RowOp { Norm, Swiglu, Quantise };

struct RowsQuant {
    const uint8_t* x;       // Norm: rows; Swiglu: gate, up halves; Quantise: rows
    const uint8_t* res;     // Norm, nullable
    const uint8_t* weight;  // Norm
    uint8_t* sum;           // Norm, nullable
    uint8_t* out;           // nullable
    int8_t* codes;          // nullable, with scales
    float* scales;
    int64_t x_stride, res_stride, sum_stride, out_stride, code_stride;   // elements
    int n_rows, d;
    float eps;
    int codes_aligned;      // set by the launcher
    float zero = 0.f;       // one that the compiler does not know
};
cudaError_t launch_rows_quant(RowOp op, int dtype, const RowsQuant& a, cudaStream_t s);
cudaError_t launch_rows_dequantise(int dtype, int n_rows, int d, const int8_t* codes, int64_t code_stride,
                                   const float* scales, void* out, int64_t out_stride, cudaStream_t s);

struct RowsRotate {
    kvr_rope rope;
    const uint8_t* in[2];   // queries, keys
    uint8_t* out[2];
    int64_t in_stride[2], out_stride[2];   // elements
    int heads[2];
    const int* pos;
    int n_rows;
    bool inverse;
};
cudaError_t launch_rows_rotate(int dtype, const RowsRotate& a, cudaStream_t s);
struct Linear {
    const int8_t* w;
    const float* w_scale;
    const float* bias;      // nullable
    const int8_t* x;
    const float* x_scale;
    void* out;
    int64_t w_stride, x_stride, out_stride;   // bytes, bytes, elements
    int n_out, k, n_rows, dtype;
    int* err;
    void* workspace;
};
constexpr int kLinearMmaRows = 8;   // up to these rows the integer kernel takes a call
cudaError_t launch_linear_mma(const Linear& a, cudaStream_t s);

double linear_few_us(int n_out, int k, int n_rows);   // estimated time
// A block's dynamic shared memory and ring, with two or four widening sets and N rows a tile.
int linear_few_smem(int sets, int N, int* stages);
cudaError_t launch_linear_few(const Linear& a, cudaStream_t s, std::string* why);
// Many rows; needs linear_tc_workspace bytes of workspace.
double linear_tc_us(int n_out, int k, int n_rows);
size_t linear_tc_workspace(int k, int n_rows);
cudaError_t launch_linear_tc(const Linear& a, cudaStream_t s, std::string* why);

cudaError_t launch_rope_table(const kvr_rope& rope, int rope_len, float2* table, cudaStream_t s);

}  // namespace kvr
