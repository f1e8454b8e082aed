// gemm.cuh -- the matrix product behind the decoder layers (host interface of gemm.cu).
#pragma once

#include "layers_common.cuh"

namespace gs {

// A factor of the product over the contracted index k: element (row, k) lies at
// p[row * ld + k] when k is the fast index, at p[k * ld + row] otherwise.  Base and
// pitch are multiples of 16 bytes (the TMA needs both).
struct GemmFactor {
    const void* p;
    int64_t ld;
    bool k_fast;
};

enum class GemmKind {
    kLinear,   // y = act(sum * x_scale * w_scale + bias) + residual, z before act
    kGlu,      // b[0] gate, b[1] up: y = act(g) * u, z = g, z2 = u
    kGluGrad,  // b[0] gate, b[1] up, residual dh: y = dh * u * act'(g), y2 = dh * act(g) (16-byte rows, one ld)
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

// How a call runs: kernel, tile shape, splits of k.  It depends on sizes, types and on
// which arrays are there, not on where.
struct GemmPlan {
    int nb, ranks;   // the few-rows kernel: rows of x a CTA takes (0: not used), CTAs that split k
    bool pair;
    int bn, sms;
    int64_t tile_m, out_cols, tiles_m, tiles_n, units, k_blocks;
    int splits, terms, probs, k_elems, esz;
    int64_t pitch;   // of the partial sums
    size_t bytes;    // of the partial sums: the call's scratch
};
GemmPlan gemm_plan(const GemmCall& c);
// Whether a CTA's part of the contraction ends well within the bound of a wait for it (a
// default plan: no product, fits).
bool gemm_fits(const GemmPlan& p);

// Multiprocessors of the current device (0 if there is none).
int device_sms();

// Sums of partial rows, up to four of them in one launch (a launch costs the host more
// than a small sum the GPU):  out[r * ld + c] = sum over parts, in a fixed order, of
// partial[part][r][c], rows of `pitch` floats.
struct JoinJobs {
    struct Job {
        const float* partial;
        void* out;
        int64_t count, ld;          // floats of a part; of out
        uint32_t rows, cols, pitch, first;   // first: block
        int parts, type, vec, slices;
    } job[4];
    int jobs = 0;
    unsigned blocks = 0;
    gs_status add(const float* partial, int64_t parts, int64_t rows, int64_t cols, int64_t pitch, void* out, int64_t ld,
                  int type);
    gs_status run(cudaStream_t st) const;   // nothing to do without jobs
};

// The partial sums of a call whose plan splits k are joined by `joins`, run later.
gs_status gemm_run(const GemmCall& c, const GemmPlan& plan, void* ws, JoinJobs* joins, cudaStream_t st);

// The gradients of a narrow gated layer (glu_narrow.cu), from x, dh and the weights: rows
// of 16-byte base and pitch but for dx, which may be NULL; dw: NULL, or glu_narrow_blocks
// partial sums [hidden][pitch] each.
struct GluNarrowCall {
    int64_t rows, features, hidden;
    int type, act;
    const void *x, *dh, *w_gate, *w_up;
    int64_t ldx, lddh, ldwg, ldwu;
    void* dx;
    int64_t lddx;
    float *dw_gate, *dw_up;
    int64_t pitch;
};
bool glu_narrow_fits(int64_t features, int64_t hidden);
int64_t glu_narrow_blocks(int64_t rows);
gs_status glu_narrow_grad(const GluNarrowCall& c, cudaStream_t st);
// Whether a wait of that kernel ran out; clears the mark.  The device is idle.
gs_status glu_narrow_wait_report(int* expired);

}  // namespace gs
