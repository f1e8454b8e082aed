// gemm.cuh -- the matrix product behind the decoder layers (host interface of gemm.cu).
#pragma once

#include "layers_common.cuh"

namespace gs {

// A factor of the product over the contracted index k: element (row, k) lies at
// p[row * ld + k] when k is the fast index, at p[k * ld + row] otherwise.
struct GemmFactor {
    const void* p;
    int64_t ld;
    bool k_fast;
};

enum class GemmKind {
    kLinear,   // y = act(sum * x_scale * w_scale + bias) + residual, z before act
    kGlu,      // b[0] gate, b[1] up: y = act(g) * u, z = g, z2 = u
    kSum,      // y = a[0] b[0]^T + a[1] b[1]^T
    kTwo       // y = a[0] b[0]^T, y2 = a[1] b[1]^T
};

struct GemmCall {
    GemmKind kind;
    int64_t m, n, k;
    int type;                 // of the factors: BF16, F16, E4M3
    GemmFactor a[2], b[2];    // [m][k], [n][k]
    const float* x_scale;     // [m]
    const float* w_scale[2];  // [n]
    const void* bias;         // [n]
    int bias_type;
    const void* residual;     // [m][n] of out_type
    int64_t ldr;
    void* y;
    int64_t ldy;
    void* y2;
    int64_t ldy2;
    void* z;                  // 16 bits, z_type
    int64_t ldz;
    void* z2;
    int64_t ldz2;
    int out_type, z_type, act;
};

// Scratch that a call needs; it depends on sizes, types, presence and alignment.
gs_status gemm_ws_bytes(const GemmCall& c, size_t* bytes);
gs_status gemm_run(const GemmCall& c, void* ws, cudaStream_t st);

// out[r * ld + c] = sum over parts, in order, of partial[part][r][c] (rows of `pitch`).
gs_status join_partials(const float* partial, int64_t parts, int64_t rows, int64_t cols, int64_t pitch, void* out,
                        int64_t ld, int type, cudaStream_t st);

}  // namespace gs
