// norm.cu -- root-mean-square norm with the residual's addition (16-, 32- or
// 8-bit output), its gradients, and row quantisation to e4m3.
//
// One pass over the data: a group of threads holds a whole row in registers,
// reduces its sum of squares (and largest magnitude) and writes the result.
// HBM bounds all three; there is no reuse beyond a row.  The group is the
// smallest power of two of threads that covers the row at kVec elements a
// thread (16-byte accesses where every row allows them, single elements
// otherwise), so narrow rows share a warp and wide ones take a block.
#include "gemm.cuh"

namespace gs {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kTiny = 0x1p-100f;

__device__ __forceinline__ float max_nan(float a, float b)   // NaN if either is
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

struct Sum {
    __device__ static float join(float a, float b) { return a + b; }
};
struct Max {
    __device__ static float join(float a, float b) { return max_nan(a, b); }
};

// Reduction over the `group` threads of a row: a warp's lanes by butterfly (all
// lanes get the same bits, the joins being commutative), then the group's warps
// through shared memory, in order.
template <class Op>
__device__ __forceinline__ float group_reduce(float v, int group, float* sm)
{
    const int in_warp = group < 32 ? group : 32;
    for (int o = in_warp >> 1; o > 0; o >>= 1) v = Op::join(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (group <= 32) return v;
    const int warp = threadIdx.x >> 5, first = threadIdx.x / group * (group >> 5), last = first + (group >> 5);
    __syncthreads();   // the previous row's readers are done
    if ((threadIdx.x & 31) == 0) sm[warp] = v;
    __syncthreads();
    float r = sm[first];
    for (int w = first + 1; w < last; ++w) r = Op::join(r, sm[w]);
    return r;
}

template <int VEC>
__device__ __forceinline__ void load_vec(const void* p, int64_t i, int type, float (&v)[VEC])
{
    if constexpr (VEC == 8) load8(p, i, type, v);
    else v[0] = load_elem(p, i, type);
}
template <int VEC>
__device__ __forceinline__ void store_vec(void* p, int64_t i, int type, const float (&v)[VEC])
{
    if constexpr (VEC == 8) store8(p, i, type, v);
    else store_elem(p, i, type, v[0]);
}

// NORM: gs_rms_norm; otherwise gs_quantize_rows (weight 1, no rstd).
// A block takes blockDim / group rows at a time.
template <int VEC, int NV, bool NORM>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(gs_rms_norm_args a, int group)
{
    __shared__ float sm[32];
    const int lane = threadIdx.x % group;
    const int rows_per_block = blockDim.x / group;
    const int nvec = (int)((a.cols + VEC - 1) / VEC);
    const float inv_cols = 1.0f / (float)a.cols;
    const bool q8 = a.y_type == GS_E4M3;
    const int64_t step = (int64_t)gridDim.x * rows_per_block;
    // every thread of a warp runs the same number of rounds (the reductions use whole warps)
    for (int64_t row0 = (int64_t)blockIdx.x * rows_per_block; row0 < a.rows; row0 += step) {
        const int64_t row = row0 + threadIdx.x / group;
        const bool live = row < a.rows;
        float s[NV][VEC];
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = lane + j * group;
#pragma unroll
            for (int e = 0; e < VEC; ++e) s[j][e] = 0.0f;
            if (live && c < nvec) {
                load_vec<VEC>(a.x, row * a.ldx + (int64_t)c * VEC, a.type, s[j]);
                if (NORM && a.residual) {
                    float r[VEC];
                    load_vec<VEC>(a.residual, row * a.ldr + (int64_t)c * VEC, a.type, r);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) s[j][e] += r[e];
                }
            }
        }
        float rstd = 1.0f;
        if (NORM) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = lane + j * group;
                if (a.sum && live && c < nvec) store_vec<VEC>(a.sum, row * a.lds + (int64_t)c * VEC, a.type, s[j]);
#pragma unroll
                for (int e = 0; e < VEC; ++e) ss = __fmaf_rn(s[j][e], s[j][e], ss);
            }
            ss = group_reduce<Sum>(ss, group, sm);
            rstd = 1.0f / sqrtf(ss * inv_cols + a.eps);
            if (a.rstd && live && lane == 0) a.rstd[row] = rstd;
        }
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = lane + j * group;
            if (c < nvec) {
                if (NORM) {
                    float w[VEC];
                    load_vec<VEC>(a.weight, (int64_t)c * VEC, a.weight_type, w);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) s[j][e] = q8 ? s[j][e] * w[e] : (s[j][e] * rstd) * w[e];
                }
                if (q8) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) top = max_nan(top, fabsf(s[j][e]));
                }
            }
        }
        if (q8) {
            // e4m3 keeps 4 significant bits; the row's largest magnitude goes to 448
            top = max_nan(group_reduce<Max>(top, group, sm), kTiny);
            const float to8 = kE4m3Max / top;
            if (live && lane == 0) a.y_scale[row] = (top / kE4m3Max) * rstd;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) s[j][e] *= to8;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = lane + j * group;
            if (live && c < nvec) store_vec<VEC>(a.y, row * a.ldy + (int64_t)c * VEC, a.y_type, s[j]);
        }
    }
}

// Gradients.  dweight: every thread keeps its columns' sums over the rows it
// visits; a block joins its groups in order and writes one partial row, and
// join_partials_kernel (linear.cu) adds the blocks' rows in order.
template <int VEC, int NV>
__global__ void __launch_bounds__(1024) norm_bwd_kernel(gs_rms_norm_bwd_args a, int group, float* partial)
{
    extern __shared__ float part[];   // [rows_per_block][cols rounded up] when a block holds several groups
    __shared__ float sm[32];
    const int lane = threadIdx.x % group;
    const int rows_per_block = blockDim.x / group;
    const int nvec = (int)((a.cols + VEC - 1) / VEC);
    const float inv_cols = 1.0f / (float)a.cols;
    const int64_t step = (int64_t)gridDim.x * rows_per_block;
    float w[NV][VEC], acc[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = lane + j * group;
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[j][e] = acc[j][e] = 0.0f;
        if (c < nvec) load_vec<VEC>(a.weight, (int64_t)c * VEC, a.weight_type, w[j]);
    }
    for (int64_t row0 = (int64_t)blockIdx.x * rows_per_block; row0 < a.rows; row0 += step) {
        const int64_t row = row0 + threadIdx.x / group;
        const bool live = row < a.rows;
        float s[NV][VEC], g[NV][VEC];
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = lane + j * group;
#pragma unroll
            for (int e = 0; e < VEC; ++e) s[j][e] = g[j][e] = 0.0f;
            if (live && c < nvec) {
                load_vec<VEC>(a.sum, row * a.lds + (int64_t)c * VEC, a.type, s[j]);
                load_vec<VEC>(a.dy, row * a.lddy + (int64_t)c * VEC, a.dy_type, g[j]);
            }
        }
        const float rstd = live ? a.rstd[row] : 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                acc[j][e] = __fmaf_rn(g[j][e], s[j][e] * rstd, acc[j][e]);
                g[j][e] *= w[j][e];
                dot = __fmaf_rn(g[j][e], s[j][e], dot);
            }
        if (a.dx) {
            dot = group_reduce<Sum>(dot, group, sm);
            const float c2 = dot * inv_cols * rstd * rstd;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = lane + j * group;
                if (live && c < nvec) {
                    float d[VEC];
#pragma unroll
                    for (int e = 0; e < VEC; ++e) d[e] = 0.0f;
                    if (a.dsum) load_vec<VEC>(a.dsum, row * a.ldds + (int64_t)c * VEC, a.type, d);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) d[e] = __fmaf_rn(rstd, __fmaf_rn(-s[j][e], c2, g[j][e]), d[e]);
                    store_vec<VEC>(a.dx, row * a.lddx + (int64_t)c * VEC, a.type, d);
                }
            }
        }
    }
    if (!a.dweight) return;
    float* out = partial + (int64_t)blockIdx.x * a.cols;
    if (rows_per_block == 1) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int c = (lane + j * group) * VEC + e;
                if (c < a.cols) out[c] = acc[j][e];
            }
        return;
    }
    const int width = NV * group * VEC;
    float* mine = part + (threadIdx.x / group) * width;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) mine[(lane + j * group) * VEC + e] = acc[j][e];
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
        float t = 0.0f;
        for (int r = 0; r < rows_per_block; ++r) t += part[r * width + c];
        out[c] = t;
    }
}

struct Shape {
    int nv, group, threads;
};

// The group: the smallest power of two of threads that covers the row with one
// vector each, at most 1024; then as many vectors a thread as that leaves.
Shape shape_for(int64_t cols, int vec)
{
    const int64_t nvec = (cols + vec - 1) / vec;
    Shape s;
    s.group = 1;
    while (s.group < nvec && s.group < (vec == 8 ? 1024 : 32)) s.group *= 2;
    if (vec == 1)
        while (s.group < 1024 && nvec > 8 * (int64_t)s.group) s.group *= 2;
    s.nv = 1;
    while ((int64_t)s.nv * s.group < nvec) s.nv *= 2;
    s.threads = s.group < 256 ? 256 : s.group;
    return s;
}

int sm_count()
{
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return sms;
}

template <bool NORM>
gs_status run_fwd(const gs_rms_norm_args& a, cudaStream_t st)
{
    const bool vec = a.cols % 8 == 0 && rows16(a.x, a.ldx, a.type) &&
                     (!a.residual || rows16(a.residual, a.ldr, a.type)) && (!a.sum || rows16(a.sum, a.lds, a.type)) &&
                     (!NORM || aligned16(a.weight)) &&
                     (a.y_type == GS_E4M3 ? ((uintptr_t)a.y & 7u) == 0 && a.ldy % 8 == 0 : rows16(a.y, a.ldy, a.y_type));
    const Shape s = shape_for(a.cols, vec ? 8 : 1);
    const int rpb = s.threads / s.group;
    const int sms = sm_count();
    if (sms <= 0) return GS_ERR_CUDA;
    const int64_t want = (a.rows + rpb - 1) / rpb, most = (int64_t)sms * (2048 / s.threads);
    const int grid = (int)(want < most ? want : most);
#define GS_FWD(V, N) norm_fwd_kernel<V, N, NORM><<<grid, s.threads, 0, st>>>(a, s.group)
    if (vec) {
        if (s.nv == 1) GS_FWD(8, 1);
        else GS_FWD(8, 2);
    } else if (s.nv <= 1) GS_FWD(1, 1);
    else if (s.nv == 2) GS_FWD(1, 2);
    else if (s.nv == 4) GS_FWD(1, 4);
    else if (s.nv == 8) GS_FWD(1, 8);
    else GS_FWD(1, 16);
#undef GS_FWD
    GS_LAUNCH_CHECK();
    return GS_OK;
}

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" gs_status gs_rms_norm(const gs_rms_norm_args* args, void* stream)
{
    GS_NVTX_RANGE("gs_rms_norm");
    if (!args) return GS_ERR_INVALID_ARG;
    const gs_rms_norm_args& a = *args;
    if (!size_ok(a.rows, 0) || !size_ok(a.cols, 1) || a.cols > GS_NORM_MAX_COLS) return GS_ERR_INVALID_ARG;
    if (!type_float(a.type) || !type_float(a.weight_type) || !(type_float(a.y_type) || a.y_type == GS_E4M3))
        return GS_ERR_INVALID_ARG;
    if (!(a.eps >= 0.0f) || a.eps > 3.4e38f) return GS_ERR_INVALID_ARG;
    if (!a.weight || !vec_ok(a.weight, a.weight_type)) return GS_ERR_INVALID_ARG;
    if (a.rows == 0) return GS_OK;
    if (!mat_ok(a.x, a.ldx, a.cols, a.type) || !mat_ok(a.y, a.ldy, a.cols, a.y_type)) return GS_ERR_INVALID_ARG;
    if (a.residual && !mat_ok(a.residual, a.ldr, a.cols, a.type)) return GS_ERR_INVALID_ARG;
    if (a.sum && !mat_ok(a.sum, a.lds, a.cols, a.type)) return GS_ERR_INVALID_ARG;
    if ((a.y_type == GS_E4M3) != (a.y_scale != nullptr)) return GS_ERR_INVALID_ARG;
    if (!vec_ok(a.y_scale, GS_F32) || !vec_ok(a.rstd, GS_F32)) return GS_ERR_INVALID_ARG;
    return run_fwd<true>(a, (cudaStream_t)stream);
}

extern "C" gs_status gs_quantize_rows(const gs_quantize_rows_args* args, void* stream)
{
    GS_NVTX_RANGE("gs_quantize_rows");
    if (!args) return GS_ERR_INVALID_ARG;
    const gs_quantize_rows_args& q = *args;
    if (!size_ok(q.rows, 0) || !size_ok(q.cols, 1) || q.cols > GS_NORM_MAX_COLS || !type_float(q.type))
        return GS_ERR_INVALID_ARG;
    if (q.rows == 0) return GS_OK;
    if (!mat_ok(q.x, q.ldx, q.cols, q.type) || !mat_ok(q.q, q.ldq, q.cols, GS_E4M3)) return GS_ERR_INVALID_ARG;
    if (!q.scale || !vec_ok(q.scale, GS_F32)) return GS_ERR_INVALID_ARG;
    gs_rms_norm_args a = {};
    a.rows = q.rows, a.cols = q.cols;
    a.x = q.x, a.ldx = q.ldx, a.type = q.type;
    a.y = q.q, a.ldy = q.ldq, a.y_type = GS_E4M3, a.y_scale = q.scale;
    return run_fwd<false>(a, (cudaStream_t)stream);
}

extern "C" gs_status gs_rms_norm_bwd(const gs_rms_norm_bwd_args* args, void* ws, size_t* ws_bytes, void* stream)
{
    GS_NVTX_RANGE("gs_rms_norm_bwd");
    if (!args) return GS_ERR_INVALID_ARG;
    const gs_rms_norm_bwd_args& a = *args;
    if (!size_ok(a.rows, 0) || !size_ok(a.cols, 1) || a.cols > GS_NORM_MAX_COLS) return GS_ERR_INVALID_ARG;
    if (!type_float(a.type) || !type_float(a.dy_type) || !type_float(a.weight_type)) return GS_ERR_INVALID_ARG;
    const int sms = sm_count();
    // one partial row per block; the size is the same whatever the alignment of the arrays
    const int64_t blocks = 2 * (sms > 0 ? sms : 152);
    const size_t need = a.dweight ? (size_t)round_up(blocks * a.cols * 4, 256) : 0;
    const WsCheck wc = ws_check(ws, ws_bytes, need);
    if (wc == WsCheck::kBad) return GS_ERR_INVALID_ARG;
    if (wc == WsCheck::kQuery) return GS_OK;
    if (!a.weight || !vec_ok(a.weight, a.weight_type) || !vec_ok(a.dweight, a.weight_type)) return GS_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    if (a.rows == 0) {
        if (a.dweight) GS_CUDA_TRY(cudaMemsetAsync(a.dweight, 0, (size_t)a.cols * type_bytes(a.weight_type), st));
        return GS_OK;
    }
    if (!mat_ok(a.dy, a.lddy, a.cols, a.dy_type) || !mat_ok(a.sum, a.lds, a.cols, a.type) || !a.rstd ||
        !vec_ok(a.rstd, GS_F32))
        return GS_ERR_INVALID_ARG;
    if (a.dsum && !mat_ok(a.dsum, a.ldds, a.cols, a.type)) return GS_ERR_INVALID_ARG;
    if (a.dx && !mat_ok(a.dx, a.lddx, a.cols, a.type)) return GS_ERR_INVALID_ARG;
    if (!a.dx && !a.dweight) return GS_OK;
    if (sms <= 0) return GS_ERR_CUDA;
    const bool vec = a.cols % 8 == 0 && rows16(a.dy, a.lddy, a.dy_type) && rows16(a.sum, a.lds, a.type) &&
                     (!a.dsum || rows16(a.dsum, a.ldds, a.type)) && (!a.dx || rows16(a.dx, a.lddx, a.type)) &&
                     aligned16(a.weight);
    const int v = vec ? 8 : 1;
    Shape s = shape_for(a.cols, v);
    if (s.threads < 512) s.threads = 512;
    const int rpb = s.threads / s.group;
    const int64_t want = (a.rows + rpb - 1) / rpb;
    const int grid = (int)(want < blocks ? want : blocks);
    const size_t smem = rpb > 1 && a.dweight ? (size_t)rpb * s.nv * s.group * v * 4 : 0;   // at most 32 KB
    float* part = (float*)ws;
#define GS_BWD(V, N) norm_bwd_kernel<V, N><<<grid, s.threads, smem, st>>>(a, s.group, part)
    if (vec) {
        if (s.nv == 1) GS_BWD(8, 1);
        else GS_BWD(8, 2);
    } else if (s.nv <= 1) GS_BWD(1, 1);
    else if (s.nv == 2) GS_BWD(1, 2);
    else if (s.nv == 4) GS_BWD(1, 4);
    else if (s.nv == 8) GS_BWD(1, 8);
    else GS_BWD(1, 16);
#undef GS_BWD
    GS_LAUNCH_CHECK();
    if (a.dweight) return join_partials(part, grid, 1, a.cols, a.cols, a.dweight, a.cols, a.weight_type, st);
    return GS_OK;
}
