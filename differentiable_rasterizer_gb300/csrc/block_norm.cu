// block_norm.cu -- the norm after a block, its gate and residual scale, and the norm
// before the next block, with their gradients.
//
//   a = h rms(h)^-1 post,  s = scale x + gate a,  y = s rms(s)^-1 weight
//
// One pass over the rows: a group of threads holds a row in registers from h and x to s
// and y (backward: from dy, ds, s and h to dx and dh), with two reductions in between.
// HBM bounds both; the group is the smallest power of two of threads that covers the row
// at VEC elements a thread, as in norm.cu, so narrow rows share a warp and wide ones take
// a block.  As separate norm, product, sum and norm a row would cross HBM nine times in
// place of four.
#include <type_traits>

#include "gemm.cuh"
#include "rows.cuh"

namespace gs {
namespace {

using namespace rows;

// A vector that may be absent, in fp32.
template <int VEC>
__device__ __forceinline__ void load_or_one(const void* p, int64_t i, int type, bool there, float (&v)[VEC])
{
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = 1.0f;
    if (p && there) load_vec<VEC>(p, i, type, v);
}

template <int T, int VEC, int NV>
__global__ void __launch_bounds__(512) block_norm_kernel(const __grid_constant__ gs_block_norm_args a, int group)
{
    __shared__ float sm[32];
    wait_for_predecessor();
    const int lane = threadIdx.x % group, rows_per_block = blockDim.x / group;
    const int nvec = (int)((a.cols + VEC - 1) / VEC);
    const float inv_cols = 1.0f / (float)a.cols;
    const bool q8 = a.y_type == GS_E4M3 && a.y;
    // every thread of a warp runs the same number of rounds (the reductions use whole warps)
    for (int64_t row0 = (int64_t)blockIdx.x * rows_per_block; row0 < a.rows; row0 += (int64_t)gridDim.x * rows_per_block) {
        const int64_t row = row0 + threadIdx.x / group;
        const bool here = row < a.rows;
        Raw<T, VEC> hr[NV], xr[NV], gr[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = lane + j * group;
            raw_zero(hr[j]);
            raw_zero(xr[j]);
            raw_zero(gr[j]);
            if (here && c < nvec) {
                raw_load(hr[j], a.h, row * a.ldh + (int64_t)c * VEC, T);
                raw_load(xr[j], a.x, row * a.ldx + (int64_t)c * VEC, T);
                if (a.gate_rows) raw_load(gr[j], a.gate, row * a.ldg + (int64_t)c * VEC, T);
            }
        }
        float s[NV][VEC], rstd_post = 1.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) raw_values(hr[j], T, s[j]);
        if (a.post_weight) {
            float ss = 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) ss = __fmaf_rn(s[j][e], s[j][e], ss);
            rstd_post = 1.0f / sqrtf(group_reduce<Sum>(ss, group, sm) * inv_cols + a.eps);
            if (a.rstd_post && here && lane == 0) a.rstd_post[row] = rstd_post;
        }
        float ss = 0.0f, top = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = lane + j * group;
            float x[VEC], g[VEC], w[VEC];
            raw_values(xr[j], T, x);
            load_or_one<VEC>(a.post_weight, (int64_t)c * VEC, a.post_type, c < nvec, w);
            if (a.gate_rows) raw_values(gr[j], T, g);
            else load_or_one<VEC>(a.gate, (int64_t)c * VEC, a.gate_type, c < nvec, g);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float n = a.post_weight ? (s[j][e] * rstd_post) * w[e] : s[j][e];
                s[j][e] = __fmaf_rn(a.scale, x[e], g[e] * n);
                if (VEC == 8 || c < nvec) ss = __fmaf_rn(s[j][e], s[j][e], ss);
            }
            if (here && c < nvec) store_vec<VEC>(a.s, row * a.lds + (int64_t)c * VEC, T, s[j]);
        }
        if (!a.y) continue;
        ss = group_reduce<Sum>(ss, group, sm);
        const float rstd = 1.0f / sqrtf(ss * inv_cols + a.eps);
        if (a.rstd && here && lane == 0) a.rstd[row] = rstd;
        float factor = rstd;
        if (q8) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = lane + j * group;
                float w[VEC];
                load_or_one<VEC>(a.weight, (int64_t)c * VEC, a.weight_type, c < nvec, w);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    s[j][e] *= w[e];
                    top = max_nan(top, fabsf(s[j][e]));
                }
            }
            top = max_nan(group_reduce<Max>(top, group, sm), kTiny);
            factor = kE4m3Max / top;
            if (here && lane == 0) a.y_scale[row] = (top / kE4m3Max) * rstd;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = lane + j * group;
            if (q8) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) s[j][e] *= factor;
            } else {
                float w[VEC];
                load_or_one<VEC>(a.weight, (int64_t)c * VEC, a.weight_type, c < nvec, w);
#pragma unroll
                for (int e = 0; e < VEC; ++e) s[j][e] = (s[j][e] * factor) * w[e];
            }
            if (here && c < nvec) store_vec<VEC>(a.y, row * a.ldy + (int64_t)c * VEC, a.y_type, s[j]);
        }
    }
}

// Sums over rows: every thread keeps its columns' over the rows it visits, a block joins
// its groups' in order into partial rows, and JoinJobs adds the blocks' in order.
// partial: [3][blocks][cols]: dweight, dpost, dgate.
template <int T, int TDY, int VEC, int NV>
__global__ void __launch_bounds__(512) block_norm_bwd_kernel(const __grid_constant__ gs_block_norm_bwd_args a,
                                                                                     int group, float* partial)
{
    extern __shared__ float part[];   // [groups][columns rounded up] when a block holds several groups
    __shared__ float sm[32];
    wait_for_predecessor();
    const int lane = threadIdx.x % group, groups = blockDim.x / group;
    const int nvec = (int)((a.cols + VEC - 1) / VEC);
    const float inv_cols = 1.0f / (float)a.cols;
    const bool post = a.post_weight != nullptr, gate_sum = a.dgate && !a.gate_rows;
    float acc[3][NV][VEC];
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[k][j][e] = 0.0f;
    for (int64_t row0 = (int64_t)blockIdx.x * groups; row0 < a.rows; row0 += (int64_t)gridDim.x * groups) {
        const int64_t row = row0 + threadIdx.x / group;
        const bool here = row < a.rows;
        Raw<T, VEC> hr[NV], sr[NV], dr[NV], gr[NV];
        Raw<TDY, VEC> yr[NV];
        const float rstd = a.dy && here ? a.rstd[row] : 0.0f, rstd_post = post && here ? a.rstd_post[row] : 1.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = lane + j * group;
            raw_zero(hr[j]);
            raw_zero(sr[j]);
            raw_zero(dr[j]);
            raw_zero(gr[j]);
            raw_zero(yr[j]);
            if (here && c < nvec) {
                const int64_t at = (int64_t)c * VEC;
                if (a.dy) {
                    raw_load(yr[j], a.dy, row * a.lddy + at, a.dy_type);
                    raw_load(sr[j], a.s, row * a.lds + at, T);
                }
                if (a.ds) raw_load(dr[j], a.ds, row * a.ldds + at, T);
                if (post || a.dgate) raw_load(hr[j], a.h, row * a.ldh + at, T);
                if (a.gate_rows) raw_load(gr[j], a.gate, row * a.ldg + at, T);
            }
        }
        float g[NV][VEC];   // the gradient of s, then of a times post
#pragma unroll
        for (int j = 0; j < NV; ++j) raw_values(dr[j], T, g[j]);
        if (a.dy) {
            float dot = 0.0f;
            float s[NV][VEC], w[NV][VEC];
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = lane + j * group;
                float dy[VEC];
                raw_values(sr[j], T, s[j]);
                raw_values(yr[j], a.dy_type, dy);
                load_or_one<VEC>(a.weight, (int64_t)c * VEC, a.weight_type, c < nvec, w[j]);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    acc[0][j][e] = __fmaf_rn(dy[e], s[j][e] * rstd, acc[0][j][e]);
                    w[j][e] *= dy[e];
                    dot = __fmaf_rn(w[j][e], s[j][e], dot);
                }
            }
            const float c2 = group_reduce<Sum>(dot, group, sm) * inv_cols * rstd * rstd;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) g[j][e] = __fmaf_rn(rstd, __fmaf_rn(-s[j][e], c2, w[j][e]), g[j][e]);
        }
        float h[NV][VEC], dot = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = lane + j * group;
            const int64_t at = (int64_t)c * VEC;
            float w[VEC], gate[VEC], v[VEC];
            raw_values(hr[j], T, h[j]);
            load_or_one<VEC>(a.post_weight, at, a.post_type, c < nvec, w);
            if (a.gate_rows) raw_values(gr[j], T, gate);
            else load_or_one<VEC>(a.gate, at, a.gate_type, c < nvec, gate);
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[e] = a.scale * g[j][e];
            if (a.dx && here && c < nvec) store_vec<VEC>(a.dx, row * a.lddx + at, T, v);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float unit = h[j][e] * rstd_post;
                v[e] = g[j][e] * (post ? unit * w[e] : h[j][e]);   // the gate's gradient
                acc[2][j][e] += v[e];
                g[j][e] *= gate[e];
                acc[1][j][e] = __fmaf_rn(g[j][e], unit, acc[1][j][e]);
                if (post) g[j][e] *= w[e];
                dot = __fmaf_rn(g[j][e], h[j][e], dot);
            }
            if (a.dgate && a.gate_rows && here && c < nvec) store_vec<VEC>(a.dgate, row * a.lddg + at, T, v);
        }
        if (!a.dh) continue;
        const float c2 = post ? group_reduce<Sum>(dot, group, sm) * inv_cols * rstd_post * rstd_post : 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = lane + j * group;
            if (post) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) g[j][e] = rstd_post * __fmaf_rn(-h[j][e], c2, g[j][e]);
            }
            if (here && c < nvec) store_vec<VEC>(a.dh, row * a.lddh + (int64_t)c * VEC, T, g[j]);
        }
    }
    const bool wanted[3] = {a.dweight != nullptr, a.dpost != nullptr, gate_sum};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        if (!wanted[k]) continue;
        float* out = partial + ((int64_t)k * gridDim.x + blockIdx.x) * a.cols;
        if (groups == 1) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int c = (lane + j * group) * VEC + e;
                    if (c < a.cols) out[c] = acc[k][j][e];
                }
            continue;
        }
        const int width = NV * group * VEC;
        float* mine = part + (threadIdx.x / group) * width;
        __syncthreads();   // the sums before have been read
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) mine[(lane + j * group) * VEC + e] = acc[k][j][e];
        __syncthreads();
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
            float t = 0.0f;
            for (int r = 0; r < groups; ++r) t += part[r * width + c];
            out[c] = t;
        }
    }
}

template <int V>
using Type = std::integral_constant<int, V>;

// The group: the smallest power of two of threads that covers the row with one vector
// each, at most 512; then as many vectors a thread as that leaves.
struct Shape {
    int nv, group, threads;
};
Shape shape_for(int64_t cols, int vec)
{
    const int64_t nvec = (cols + vec - 1) / vec, widest = 512;
    Shape s;
    s.group = 1;
    while (s.group < nvec && s.group < (vec == 8 ? widest : 32)) s.group *= 2;
    if (vec == 1)
        while (s.group < widest && nvec > 8 * (int64_t)s.group) s.group *= 2;
    s.nv = 1;
    while ((int64_t)s.nv * s.group < nvec) s.nv *= vec == 8 ? 2 : 4;
    s.threads = s.group < 256 ? 256 : s.group;
    return s;
}

bool norm_sizes_ok(int64_t rows, int64_t cols, int type) { return size_ok(rows, 0) && size_ok(cols, 1) && cols <= GS_NORM_MAX_COLS && type_float(type); }

bool weight_ok(const void* p, int type) { return !p || (type_float(type) && vec_ok(p, type)); }

bool weight16(const void* p) { return !p || aligned16(p); }

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" gs_status gs_block_norm(const gs_block_norm_args* args, void* stream)
{
    GS_NVTX_RANGE("gs_block_norm");
    if (!args) return GS_ERR_INVALID_ARG;
    const gs_block_norm_args& a = *args;
    if (!norm_sizes_ok(a.rows, a.cols, a.type) || !(a.eps >= 0.0f) || a.eps > 3.4e38f || !(fabsf(a.scale) <= 3.4e38f))
        return GS_ERR_INVALID_ARG;
    if (!weight_ok(a.post_weight, a.post_type) || !weight_ok(a.weight, a.weight_type) || (a.gate_rows && !a.gate) ||
        (!a.gate_rows && !weight_ok(a.gate, a.gate_type)))
        return GS_ERR_INVALID_ARG;
    if ((a.rstd_post && !a.post_weight) || (a.rstd && !a.weight) || !vec_ok(a.rstd_post, GS_F32) || !vec_ok(a.rstd, GS_F32))
        return GS_ERR_INVALID_ARG;
    if (a.weight && !type_float(a.y_type) && a.y_type != GS_E4M3) return GS_ERR_INVALID_ARG;
    if (!vec_ok(a.y_scale, GS_F32) || (a.weight && a.y_type == GS_E4M3) != (a.y_scale != nullptr)) return GS_ERR_INVALID_ARG;
    if (!a.weight && a.y) return GS_ERR_INVALID_ARG;
    if (a.rows == 0) return GS_OK;
    if (!mat_ok(a.h, a.ldh, a.cols, a.type) || !mat_ok(a.x, a.ldx, a.cols, a.type) || !mat_ok(a.s, a.lds, a.cols, a.type))
        return GS_ERR_INVALID_ARG;
    if (a.gate_rows && !mat_ok(a.gate, a.ldg, a.cols, a.type)) return GS_ERR_INVALID_ARG;
    if (a.weight && !mat_ok(a.y, a.ldy, a.cols, a.y_type)) return GS_ERR_INVALID_ARG;
    const int sms = device_sms();
    if (sms <= 0) return GS_ERR_CUDA;
    const bool vec = a.cols % 8 == 0 && rows16(a.h, a.ldh, a.type) && rows16(a.x, a.ldx, a.type) && rows16(a.s, a.lds, a.type) &&
                     weight16(a.post_weight) && weight16(a.weight) && (a.gate_rows ? rows16(a.gate, a.ldg, a.type) : weight16(a.gate)) &&
                     (!a.weight || (a.y_type == GS_E4M3 ? ((uintptr_t)a.y & 7u) == 0 && a.ldy % 8 == 0 : rows16(a.y, a.ldy, a.y_type)));
    const Shape s = shape_for(a.cols, vec ? 8 : 1);
    const int64_t rpb = s.threads / s.group, want = (a.rows + rpb - 1) / rpb, most = (int64_t)sms * (2048 / s.threads);
    const int grid = (int)(want < most ? want : most);
    cudaStream_t st = (cudaStream_t)stream;
    const auto run = [&](auto t) -> gs_status {
        constexpr int T = decltype(t)::value;
#define GS_FWD(V, N) return launch_after(block_norm_kernel<T, V, N>, dim3(grid), s.threads, 0, 1, st, a, s.group)
        if (vec) {
            if (s.nv == 1) GS_FWD(8, 1);
            else if (s.nv == 2) GS_FWD(8, 2);
            else GS_FWD(8, 4);
        } else if (s.nv <= 1) GS_FWD(1, 1);
        else if (s.nv <= 4) GS_FWD(1, 4);
        else if (s.nv <= 16) GS_FWD(1, 16);
        else GS_FWD(1, 32);
#undef GS_FWD
    };
    if (a.type == GS_F32) return run(Type<GS_F32>());
    if (a.type == GS_BF16) return run(Type<GS_BF16>());
    return run(Type<GS_F16>());
}

extern "C" gs_status gs_block_norm_bwd(const gs_block_norm_bwd_args* args, void* ws, size_t* ws_bytes, void* stream)
{
    GS_NVTX_RANGE("gs_block_norm_bwd");
    if (!args) return GS_ERR_INVALID_ARG;
    const gs_block_norm_bwd_args& a = *args;
    if (!norm_sizes_ok(a.rows, a.cols, a.type) || !(fabsf(a.scale) <= 3.4e38f)) return GS_ERR_INVALID_ARG;
    if (!weight_ok(a.post_weight, a.post_type) || !weight_ok(a.weight, a.weight_type) || (a.gate_rows && !a.gate) ||
        (!a.gate_rows && !weight_ok(a.gate, a.gate_type)))
        return GS_ERR_INVALID_ARG;
    if ((a.dweight && !a.weight) || (a.dpost && !a.post_weight) || (a.dgate && !a.gate)) return GS_ERR_INVALID_ARG;
    if (!vec_ok(a.dweight, a.weight_type) || !vec_ok(a.dpost, a.post_type) || (!a.gate_rows && !vec_ok(a.dgate, a.gate_type)))
        return GS_ERR_INVALID_ARG;
    if (a.weight && !type_float(a.dy_type)) return GS_ERR_INVALID_ARG;
    const int sms = device_sms();
    const int64_t blocks = 3 * (sms > 0 ? sms : 152);   // the size is the same whatever the alignment of the arrays
    const bool gate_sum = a.dgate && !a.gate_rows;
    const size_t need = a.dweight || a.dpost || gate_sum ? (size_t)round_up(3 * blocks * a.cols * 4, 256) : 0;
    const WsCheck wc = ws_check(ws, ws_bytes, need);
    if (wc == WsCheck::kBad) return GS_ERR_INVALID_ARG;
    if (wc == WsCheck::kQuery) return GS_OK;
    cudaStream_t st = (cudaStream_t)stream;
    if (a.rows == 0) {
        if (a.dweight) GS_CUDA_TRY(cudaMemsetAsync(a.dweight, 0, (size_t)a.cols * type_bytes(a.weight_type), st));
        if (a.dpost) GS_CUDA_TRY(cudaMemsetAsync(a.dpost, 0, (size_t)a.cols * type_bytes(a.post_type), st));
        if (gate_sum) GS_CUDA_TRY(cudaMemsetAsync(a.dgate, 0, (size_t)a.cols * type_bytes(a.gate_type), st));
        return GS_OK;
    }
    if (!a.dy != !a.weight || !a.dy != !a.rstd || !vec_ok(a.rstd, GS_F32) || (!a.dy && !a.ds)) return GS_ERR_INVALID_ARG;
    if (!a.post_weight != !a.rstd_post || !vec_ok(a.rstd_post, GS_F32)) return GS_ERR_INVALID_ARG;
    const auto mat = [&](const void* p, int64_t ld, bool used, int type) { return !used || mat_ok(p, ld, a.cols, type); };
    const bool reads_h = a.post_weight || a.dgate, row_gate = a.gate_rows != 0, row_dgate = row_gate && a.dgate;
    if (!mat(a.dy, a.lddy, a.dy, a.dy_type) || !mat(a.s, a.lds, a.dy, a.type) || !mat(a.ds, a.ldds, a.ds, a.type) ||
        !mat(a.h, a.ldh, reads_h, a.type) || !mat(a.gate, a.ldg, row_gate, a.type) || !mat(a.dgate, a.lddg, row_dgate, a.type) ||
        !mat(a.dx, a.lddx, a.dx, a.type) || !mat(a.dh, a.lddh, a.dh, a.type))
        return GS_ERR_INVALID_ARG;
    if (!a.dx && !a.dh && !a.dweight && !a.dpost && !a.dgate) return GS_OK;
    if (sms <= 0) return GS_ERR_CUDA;
    const auto wide = [&](const void* p, int64_t ld, bool used, int type) { return !used || rows16(p, ld, type); };
    const bool vec = a.cols % 8 == 0 && wide(a.dy, a.lddy, a.dy, a.dy_type) && wide(a.s, a.lds, a.dy, a.type) &&
                     wide(a.ds, a.ldds, a.ds, a.type) && wide(a.h, a.ldh, reads_h, a.type) && wide(a.gate, a.ldg, row_gate, a.type) &&
                     wide(a.dgate, a.lddg, row_dgate, a.type) && wide(a.dx, a.lddx, a.dx, a.type) && wide(a.dh, a.lddh, a.dh, a.type) &&
                     weight16(a.weight) && weight16(a.post_weight) && (row_gate || weight16(a.gate));
    const int v = vec ? 8 : 1;
    const Shape s = shape_for(a.cols, v);
    const int groups = s.threads / s.group;
    const int64_t want = (a.rows + groups - 1) / groups;
    const int grid = (int)(want < blocks ? want : blocks);
    const size_t smem = groups > 1 && need ? (size_t)groups * s.nv * s.group * v * 4 : 0;   // at most 16 KB
    float* part = (float*)ws;
    const auto run = [&](auto t, auto tdy) -> gs_status {
        constexpr int T = decltype(t)::value, TDY = decltype(tdy)::value;
#define GS_BWD(V, N) return launch_after(block_norm_bwd_kernel<T, TDY, V, N>, dim3(grid), s.threads, smem, 1, st, a, s.group, part)
        if (vec) {
            if (s.nv == 1) GS_BWD(8, 1);
            else if (s.nv == 2) GS_BWD(8, 2);
            else GS_BWD(8, 4);
        } else if (s.nv <= 1) GS_BWD(1, 1);
        else if (s.nv <= 4) GS_BWD(1, 4);
        else if (s.nv <= 16) GS_BWD(1, 16);
        else GS_BWD(1, 32);
#undef GS_BWD
    };
    const auto pick = [&](auto t) -> gs_status {
        if (!a.dy || a.dy_type == a.type) return run(t, t);
        return run(t, Type<kAnyType>());
    };
    gs_status status = a.type == GS_F32 ? pick(Type<GS_F32>()) : (a.type == GS_BF16 ? pick(Type<GS_BF16>()) : pick(Type<GS_F16>()));
    if (status != GS_OK) return status;
    JoinJobs joins;
    const int64_t step = (int64_t)grid * a.cols;
    if (a.dweight) status = joins.add(part, grid, 1, a.cols, a.cols, a.dweight, a.cols, a.weight_type);
    if (status == GS_OK && a.dpost) status = joins.add(part + step, grid, 1, a.cols, a.cols, a.dpost, a.cols, a.post_type);
    if (status == GS_OK && gate_sum) status = joins.add(part + 2 * step, grid, 1, a.cols, a.cols, a.dgate, a.cols, a.gate_type);
    return status == GS_OK ? joins.run(st) : status;
}
