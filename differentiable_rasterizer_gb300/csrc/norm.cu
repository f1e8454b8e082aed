// norm.cu -- root-mean-square norm with the residual's addition (16-, 32- or
// 8-bit output), its gradients, and row quantisation to e4m3.
//
// One pass over the data: a group of threads holds a whole row in registers,
// reduces its sum of squares (and largest magnitude) and writes the result.
// HBM bounds all three; there is no reuse beyond a row.  The group is the
// smallest power of two of threads that covers the row at kVec elements a
// thread (16-byte accesses where every row allows them, single elements
// otherwise), so narrow rows share a warp and wide ones take a block.
#include <type_traits>

#include "gemm.cuh"
#include "rows.cuh"

namespace gs {
namespace {

using namespace rows;

// NORM: gs_rms_norm; otherwise gs_quantize_rows (weight 1, no rstd).
// A group takes R rows at a time, all their loads in flight together; with R rows
// the lanes share out the rows' scalar work (root, quotients), which otherwise
// costs every lane as many instructions as the row's elements.
template <int T, int VEC, int NV, int R, bool NORM>
__global__ void __launch_bounds__(R > 1 || NV * VEC == 32 ? 256 : 1024) norm_fwd_kernel(const __grid_constant__ gs_rms_norm_args a, int group)
{
    __shared__ float sm[32];
    wait_for_predecessor();
    const int lane = threadIdx.x % group;
    const int64_t rows_per_block = (int64_t)(blockDim.x / group) * R;
    const int nvec = (int)((a.cols + VEC - 1) / VEC);
    const float inv_cols = 1.0f / (float)a.cols;
    const bool q8 = a.y_type == GS_E4M3;
    const int64_t step = (int64_t)gridDim.x * rows_per_block;
    float w[NV][VEC];
    if (NORM) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) w[j][e] = 0.0f;
            if (lane + j * group < nvec) load_vec<VEC>(a.weight, (int64_t)(lane + j * group) * VEC, a.weight_type, w[j]);
        }
    }
    // every thread of a warp runs the same number of rounds (the reductions use whole warps)
    for (int64_t row0 = (int64_t)blockIdx.x * rows_per_block; row0 < a.rows; row0 += step) {
        const int64_t row = row0 + (int64_t)(threadIdx.x / group) * R;
        float s[R][NV][VEC];
        Raw<T, VEC> xr[R][NV], rr[R][NV];
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = lane + j * group;
                raw_zero(xr[i][j]);
                raw_zero(rr[i][j]);
                if (row + i < a.rows && c < nvec) {
                    raw_load(xr[i][j], a.x, (row + i) * a.ldx + (int64_t)c * VEC, T);
                    if (NORM && a.residual) raw_load(rr[i][j], a.residual, (row + i) * a.ldr + (int64_t)c * VEC, T);
                }
            }
        float ss[R], top[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            ss[i] = top[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = lane + j * group;
                raw_values(xr[i][j], T, s[i][j]);
                if (NORM) {
                    float r[VEC];
                    raw_values(rr[i][j], T, r);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        s[i][j][e] += r[e];
                        ss[i] = __fmaf_rn(s[i][j][e], s[i][j][e], ss[i]);
                    }
                    if (a.sum && row + i < a.rows && c < nvec)
                        store_vec<VEC>(a.sum, (row + i) * a.lds + (int64_t)c * VEC, T, s[i][j]);
                    if (q8) {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) s[i][j][e] *= w[j][e];
                    }
                }
                if (q8) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) top[i] = max_nan(top[i], fabsf(s[i][j][e]));
                }
            }
        }
        // scalar work: every lane for R == 1, lane i (mod R) for row i otherwise
        float rstd[R], to8[R];
        if (NORM) {
#pragma unroll
            for (int i = 0; i < R; ++i) ss[i] = group_reduce<Sum>(ss[i], group, sm);
        }
        if (q8) {   // e4m3 keeps 4 significant bits; the row's largest magnitude goes to 448
#pragma unroll
            for (int i = 0; i < R; ++i) top[i] = max_nan(group_reduce<Max>(top[i], group, sm), kTiny);
        }
        const int mine = R == 1 ? 0 : lane % R;
        float my_ss = ss[0], my_top = top[0];
#pragma unroll
        for (int i = 1; i < R; ++i)
            if (mine == i) my_ss = ss[i], my_top = top[i];
        const float my_rstd = NORM ? 1.0f / sqrtf(my_ss * inv_cols + a.eps) : 1.0f;
        const float my_to8 = q8 ? kE4m3Max / my_top : 1.0f;
        if (lane < R && row + mine < a.rows) {
            if (NORM && a.rstd) a.rstd[row + mine] = my_rstd;
            if (q8) a.y_scale[row + mine] = (my_top / kE4m3Max) * my_rstd;
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float factor = q8 ? my_to8 : my_rstd;
            rstd[i] = to8[i] = R == 1 ? factor : __shfl_sync(0xffffffffu, factor, (threadIdx.x & 31) / group * group + i);
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = lane + j * group;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    if (q8) s[i][j][e] *= to8[i];
                    else s[i][j][e] = (s[i][j][e] * rstd[i]) * w[j][e];
                }
                if (row + i < a.rows && c < nvec)
                    store_vec<VEC>(a.y, (row + i) * a.ldy + (int64_t)c * VEC, a.y_type, s[i][j]);
            }
    }
}

// Gradients.  dweight: every thread keeps its columns' sums over the rows it
// visits; a block joins its groups in order and writes one partial row, and
// JoinJobs (linear.cu) adds the blocks' rows in order.
// R rows a group at a time, their loads in flight together.
template <int T, int TDY, int VEC, int NV, int R>
__global__ void __launch_bounds__(R > 1 ? 256 : 1024) norm_bwd_kernel(const __grid_constant__ gs_rms_norm_bwd_args a, int group, float* partial)
{
    extern __shared__ float part[];   // [groups][columns rounded up] when a block holds several groups
    __shared__ float sm[32];
    wait_for_predecessor();
    const int lane = threadIdx.x % group;
    const int groups = blockDim.x / group;
    const int nvec = (int)((a.cols + VEC - 1) / VEC);
    const float inv_cols = 1.0f / (float)a.cols;
    const int64_t step = (int64_t)gridDim.x * groups * R;
    float w[NV][VEC], acc[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = lane + j * group;
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[j][e] = acc[j][e] = 0.0f;
        if (c < nvec) load_vec<VEC>(a.weight, (int64_t)c * VEC, a.weight_type, w[j]);
    }
    for (int64_t row0 = (int64_t)blockIdx.x * groups * R; row0 < a.rows; row0 += step) {
        const int64_t row = row0 + (int64_t)(threadIdx.x / group) * R;
        float s[R][NV][VEC], g[R][NV][VEC], rstd[R];
        Raw<T, VEC> sr[R][NV], dr[R][NV];
        Raw<TDY, VEC> gr[R][NV];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            rstd[i] = row + i < a.rows ? a.rstd[row + i] : 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = lane + j * group;
                raw_zero(sr[i][j]);
                raw_zero(gr[i][j]);
                raw_zero(dr[i][j]);
                if (row + i < a.rows && c < nvec) {
                    raw_load(sr[i][j], a.sum, (row + i) * a.lds + (int64_t)c * VEC, T);
                    raw_load(gr[i][j], a.dy, (row + i) * a.lddy + (int64_t)c * VEC, a.dy_type);
                    if (a.dx && a.dsum) raw_load(dr[i][j], a.dsum, (row + i) * a.ldds + (int64_t)c * VEC, T);
                }
            }
        }
        float dot[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            dot[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                raw_values(sr[i][j], T, s[i][j]);
                raw_values(gr[i][j], a.dy_type, g[i][j]);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    acc[j][e] = __fmaf_rn(g[i][j][e], s[i][j][e] * rstd[i], acc[j][e]);
                    g[i][j][e] *= w[j][e];
                    dot[i] = __fmaf_rn(g[i][j][e], s[i][j][e], dot[i]);
                }
            }
        }
        if (!a.dx) continue;
#pragma unroll
        for (int i = 0; i < R; ++i) dot[i] = group_reduce<Sum>(dot[i], group, sm);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float c2 = dot[i] * inv_cols * rstd[i] * rstd[i];
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = lane + j * group;
                float d[VEC];
                raw_values(dr[i][j], T, d);
#pragma unroll
                for (int e = 0; e < VEC; ++e) d[e] = __fmaf_rn(rstd[i], __fmaf_rn(-s[i][j][e], c2, g[i][j][e]), d[e]);
                if (row + i < a.rows && c < nvec)
                    store_vec<VEC>(a.dx, (row + i) * a.lddx + (int64_t)c * VEC, T, d);
            }
        }
    }
    if (!a.dweight) return;
    float* out = partial + (int64_t)blockIdx.x * a.cols;
    if (groups == 1) {
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
        for (int r = 0; r < groups; ++r) t += part[r * width + c];
        out[c] = t;
    }
}

template <int V>
using Type = std::integral_constant<int, V>;

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
    while ((int64_t)s.nv * s.group < nvec) s.nv *= vec == 8 ? 2 : 4;
    s.threads = s.group < 256 ? 256 : s.group;
    return s;
}

template <bool NORM>
gs_status run_fwd(const gs_rms_norm_args& a, cudaStream_t st)
{
    const bool vec = a.cols % 8 == 0 && rows16(a.x, a.ldx, a.type) &&
                     (!a.residual || rows16(a.residual, a.ldr, a.type)) && (!a.sum || rows16(a.sum, a.lds, a.type)) &&
                     (!NORM || aligned16(a.weight)) &&
                     (a.y_type == GS_E4M3 ? ((uintptr_t)a.y & 7u) == 0 && a.ldy % 8 == 0 : rows16(a.y, a.ldy, a.y_type));
    Shape s = shape_for(a.cols, vec ? 8 : 1);
    const int sms = device_sms();
    if (sms <= 0) return GS_ERR_CUDA;
    // rows of 257 to 1024 in a warp, four vectors a lane, once there are warps enough: no
    // barrier of the block between the two reductions
    if (vec && s.group > 32 && a.cols <= 1024 && a.rows >= 4ll * sms) {
        s.group = 32;
        s.nv = 4;
        s.threads = 256;
    }
    // two rows a group where a group is within a warp, holds one vector a lane and there
    // are rows enough to fill the SMs all the same (1,000,000 x 256 to 8 bits, R rows in
    // B blocks an SM: R 1 368 us, R 4 B 2 355, R 4 B 8 300, R 2 B 4 298: 6.0 TB/s)
    const bool two = vec && s.group >= 2 && s.group <= 32 && s.nv == 1 && a.rows >= (int64_t)sms * 4 * (s.threads / s.group) * 2;
    const int rpb = s.threads / s.group * (two ? 2 : 1);
    const int64_t want = (a.rows + rpb - 1) / rpb, most = (int64_t)sms * (two ? 4 : 2048 / s.threads);
    const int grid = (int)(want < most ? want : most);
    const auto run = [&](auto t) -> gs_status {
        constexpr int T = decltype(t)::value;
#define GS_FWD(V, N, R) return launch_after(norm_fwd_kernel<T, V, N, R, NORM>, dim3(grid), s.threads, 0, 1, st, a, s.group)
        if (vec) {
            if (two) GS_FWD(8, 1, 2);
            else if (s.nv == 1) GS_FWD(8, 1, 1);
            else if (s.nv == 4) GS_FWD(8, 4, 1);
            else GS_FWD(8, 2, 1);
        } else if (s.nv <= 1) GS_FWD(1, 1, 1);
        else if (s.nv <= 4) GS_FWD(1, 4, 1);
        else GS_FWD(1, 16, 1);
#undef GS_FWD
    };
    if (a.type == GS_F32) return run(Type<GS_F32>());
    if (a.type == GS_BF16) return run(Type<GS_BF16>());
    return run(Type<GS_F16>());
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
    const int sms = device_sms();
    // one partial row per block; the size is the same whatever the alignment of the arrays
    const int64_t blocks = 3 * (sms > 0 ? sms : 152);
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
    const Shape s = shape_for(a.cols, v);
    const int groups = s.threads / s.group;
    const bool two = vec && s.threads == 256 && s.nv == 1 && a.rows >= blocks * groups * 2;   // rows enough to fill the SMs
    const int64_t rpb = groups * (two ? 2 : 1), want = (a.rows + rpb - 1) / rpb;
    const int grid = (int)(want < blocks ? want : blocks);
    const size_t smem = groups > 1 && a.dweight ? (size_t)groups * s.nv * s.group * v * 4 : 0;   // at most 16 KB
    float* part = (float*)ws;
    const auto run = [&](auto t, auto tdy) -> gs_status {
        constexpr int T = decltype(t)::value, TDY = decltype(tdy)::value;
#define GS_BWD(V, N, R) return launch_after(norm_bwd_kernel<T, TDY, V, N, R>, dim3(grid), s.threads, smem, 1, st, a, s.group, part)
        if (vec) {
            if (two) GS_BWD(8, 1, 2);
            else if (s.nv == 1) GS_BWD(8, 1, 1);
            else GS_BWD(8, 2, 1);
        } else if (s.nv <= 1) GS_BWD(1, 1, 1);
        else if (s.nv <= 4) GS_BWD(1, 4, 1);
        else GS_BWD(1, 16, 1);
#undef GS_BWD
    };
    const auto pick = [&](auto t) -> gs_status {
        if (a.dy_type == a.type) return run(t, t);
        return run(t, Type<kAnyType>());
    };
    gs_status status = a.type == GS_F32 ? pick(Type<GS_F32>()) : (a.type == GS_BF16 ? pick(Type<GS_BF16>()) : pick(Type<GS_F16>()));
    if (status != GS_OK) return status;
    JoinJobs joins;
    if (a.dweight) {
        status = joins.add(part, grid, 1, a.cols, a.cols, a.dweight, a.cols, a.weight_type);
        if (status != GS_OK) return status;
    }
    return joins.run(st);
}
