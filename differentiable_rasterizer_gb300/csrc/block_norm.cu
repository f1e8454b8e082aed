// block_norm.cu -- the norm after a block, its gate and residual scale, and the norm
// before the next block, with their gradients.
//
//   a = h rms(h)^-1 post,  s = scale x + gate a,  y = s rms(s)^-1 weight
//
// One pass over the rows: a group of threads holds a row in registers from h and x to s
// and y (backward: from dy, ds, s and h to dx and dh), with two reductions in between.
// HBM bounds both.  The group is the smallest power of two of threads that covers the row
// at NV vectors of VEC elements a thread: eight (16-byte accesses) where every row allows
// them, else two, so that narrow rows share a warp and rows of up to 512 columns need no
// barrier.  As separate norm, product, sum and norm a row would cross HBM nine times in
// place of four.
//   1,000,000 x 256 bf16  303 us at HBM's rate; 500 with weights fetched for each row
//   20,011 x 331 f16      single elements and barriers: 138 us, gradients 362
#include <type_traits>

#include "gemm.cuh"
#include "rows.cuh"

namespace gs {
namespace {

using namespace rows;

// VEC consecutive elements of a row as they lie in memory.  Of two, in 16 bits one access
// where they start on 4 bytes.
template <int T, int VEC>
struct Cells {
    Raw<T, 8> raw;
    __device__ __forceinline__ void zero() { raw_zero(raw); }
    __device__ __forceinline__ void load(const void* p, int64_t i, int, int type) { raw_load(raw, p, i, type); }
    __device__ __forceinline__ void values(int type, float (&v)[8]) const { raw_values(raw, type, v); }
};
template <>
struct Cells<GS_F32, 2> {
    float a, b;
    __device__ __forceinline__ void zero() { a = b = 0.0f; }
    __device__ __forceinline__ void load(const void* p, int64_t i, int n, int)
    {
        a = ((const float*)p)[i];
        if (n > 1) b = ((const float*)p)[i + 1];
    }
    __device__ __forceinline__ void values(int, float (&v)[2]) const { v[0] = a, v[1] = b; }
};
template <>
struct Cells<kAnyType, 2> : Cells<GS_F32, 2> {
    __device__ __forceinline__ void load(const void* p, int64_t i, int n, int type)
    {
        a = load_elem(p, i, type);
        if (n > 1) b = load_elem(p, i + 1, type);
    }
};
template <int T>
struct CellsHalf {
    uint32_t w;
    __device__ __forceinline__ void zero() { w = 0; }
    __device__ __forceinline__ void load(const void* p, int64_t i, int n, int)
    {
        const uint16_t* at = (const uint16_t*)p + i;
        if (n > 1 && ((uintptr_t)at & 3u) == 0) w = *reinterpret_cast<const uint32_t*>(at);
        else w = at[0] | (n > 1 ? (uint32_t)at[1] << 16 : 0u);
    }
    __device__ __forceinline__ void values(int, float (&v)[2]) const
    {
        const float2 f = unpack_half2(w, T);
        v[0] = f.x, v[1] = f.y;
    }
};
template <>
struct Cells<GS_BF16, 2> : CellsHalf<GS_BF16> {};
template <>
struct Cells<GS_F16, 2> : CellsHalf<GS_F16> {};

template <int VEC>
__device__ __forceinline__ void store_cells(void* p, int64_t i, int n, int type, const float (&v)[VEC])
{
    if constexpr (VEC == 8) store8(p, i, type, v);
    else if (n > 1 && type != GS_F32 && type != GS_E4M3 && ((uintptr_t)((uint16_t*)p + i) & 3u) == 0)
        *reinterpret_cast<uint32_t*>((uint16_t*)p + i) = pack_half2(v[0], v[1], type);
    else
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (e < n) store_elem(p, i + e, type, v[e]);
}

// The thread's columns of a vector over them; 1 where there is none, 0 beyond the row.
template <int VEC>
__device__ __forceinline__ void load_weight(const void* p, int64_t i, int n, int type, float (&v)[VEC])
{
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = e < n ? 1.0f : 0.0f;
    if (!p || n <= 0) return;
    if constexpr (VEC == 8) load8(p, i, type, v);
    else
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (e < n) v[e] = load_elem(p, i + e, type);
}

// Weights of up to KEEP columns a thread stay in registers, of more they are fetched from
// the first-level cache for every row.
template <int VEC, int NV, int KEEP>
struct Weight {
    static constexpr bool kKeep = VEC * NV <= KEEP;
    float v[kKeep ? NV : 1][VEC];
    const void* p;
    int type, lane, group, cols;
    __device__ __forceinline__ void init(const void* p_, int type_, int lane_, int group_, int cols_)
    {
        p = p_, type = type_, lane = lane_, group = group_, cols = cols_;
        if constexpr (kKeep)
#pragma unroll
            for (int j = 0; j < NV; ++j) load_weight<VEC>(p, col(j), cols - col(j), type, v[j]);
    }
    __device__ __forceinline__ int col(int j) const { return (lane + j * group) * VEC; }
    __device__ __forceinline__ void get(int j, float (&w)[VEC]) const
    {
        if constexpr (kKeep)
#pragma unroll
            for (int e = 0; e < VEC; ++e) w[e] = v[j][e];
        else load_weight<VEC>(p, col(j), cols - col(j), type, w);
    }
};

// R rows a group at a time, their loads in flight together.
template <int T, int VEC, int NV, int R>
__global__ void __launch_bounds__(512) block_norm_kernel(const __grid_constant__ gs_block_norm_args a, int group)
{
    __shared__ float sm[32];
    wait_for_predecessor();
    const int lane = threadIdx.x % group, cols = (int)a.cols;
    const int64_t rows_per_block = (int64_t)(blockDim.x / group) * R;
    const float inv_cols = 1.0f / (float)a.cols;
    const bool q8 = a.y_type == GS_E4M3 && a.y;
    Weight<VEC, NV, 16> weight, post, gate;
    weight.init(a.weight, a.weight_type, lane, group, cols);
    post.init(a.post_weight, a.post_type, lane, group, cols);
    gate.init(a.gate_rows ? nullptr : a.gate, a.gate_type, lane, group, cols);
    // every thread of a warp runs the same number of rounds (the reductions use whole warps)
    for (int64_t row0 = (int64_t)blockIdx.x * rows_per_block; row0 < a.rows; row0 += (int64_t)gridDim.x * rows_per_block) {
        const int64_t row = row0 + (int64_t)(threadIdx.x / group) * R;
        Cells<T, VEC> hr[R][NV], xr[R][NV], gr[R][NV];
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = weight.col(j), n = cols - c;
                hr[i][j].zero(), xr[i][j].zero(), gr[i][j].zero();
                if (row + i < a.rows && n > 0) {
                    hr[i][j].load(a.h, (row + i) * a.ldh + c, n, T);
                    xr[i][j].load(a.x, (row + i) * a.ldx + c, n, T);
                    if (a.gate_rows) gr[i][j].load(a.gate, (row + i) * a.ldg + c, n, T);
                }
            }
        float s[R][NV][VEC], rstd_post[R], ss[R], top[R], factor[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            ss[i] = top[i] = 0.0f;
            rstd_post[i] = 1.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                hr[i][j].values(T, s[i][j]);
#pragma unroll
                for (int e = 0; e < VEC; ++e) ss[i] = __fmaf_rn(s[i][j][e], s[i][j][e], ss[i]);
            }
        }
        if (a.post_weight) {
#pragma unroll
            for (int i = 0; i < R; ++i) ss[i] = group_reduce<Sum>(ss[i], group, sm);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                rstd_post[i] = 1.0f / sqrtf(ss[i] * inv_cols + a.eps);
                if (a.rstd_post && row + i < a.rows && lane == 0) a.rstd_post[row + i] = rstd_post[i];
            }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) ss[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = weight.col(j), n = cols - c;
            float w[VEC], p[VEC], g0[VEC];
            post.get(j, p);
            gate.get(j, g0);
            if (q8) weight.get(j, w);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float x[VEC], g[VEC];
                xr[i][j].values(T, x);
                gr[i][j].values(T, g);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float unit = a.post_weight ? (s[i][j][e] * rstd_post[i]) * p[e] : s[i][j][e];
                    s[i][j][e] = __fmaf_rn(a.scale, x[e], (a.gate_rows ? g[e] : g0[e]) * unit);
                    ss[i] = __fmaf_rn(s[i][j][e], s[i][j][e], ss[i]);
                }
                if (row + i < a.rows && n > 0) store_cells<VEC>(a.s, (row + i) * a.lds + c, n, T, s[i][j]);
                if (q8)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        s[i][j][e] *= w[e];
                        top[i] = max_nan(top[i], fabsf(s[i][j][e]));
                    }
            }
        }
        if (!a.y) continue;
#pragma unroll
        for (int i = 0; i < R; ++i) ss[i] = group_reduce<Sum>(ss[i], group, sm);
        if (q8) {   // e4m3 keeps 4 significant bits; the row's largest magnitude goes to 448
#pragma unroll
            for (int i = 0; i < R; ++i) top[i] = max_nan(group_reduce<Max>(top[i], group, sm), kTiny);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float rstd = 1.0f / sqrtf(ss[i] * inv_cols + a.eps);
            factor[i] = q8 ? kE4m3Max / top[i] : rstd;
            if (row + i < a.rows && lane == 0) {
                if (a.rstd) a.rstd[row + i] = rstd;
                if (q8) a.y_scale[row + i] = (top[i] / kE4m3Max) * rstd;
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = weight.col(j), n = cols - c;
            float w[VEC];
            if (!q8) weight.get(j, w);
#pragma unroll
            for (int i = 0; i < R; ++i) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) s[i][j][e] = q8 ? s[i][j][e] * factor[i] : (s[i][j][e] * factor[i]) * w[e];
                if (row + i < a.rows && n > 0) store_cells<VEC>(a.y, (row + i) * a.ldy + c, n, a.y_type, s[i][j]);
            }
        }
    }
}

// Sums over rows: every thread keeps its columns' over the rows it visits, a block joins
// its groups' in order into partial rows, and JoinJobs adds the blocks' in order.
// partial: [3][blocks][cols]: dweight, dpost, dgate.
template <int T, int TDY, int VEC, int NV, int R>
__global__ void __launch_bounds__(512) block_norm_bwd_kernel(const __grid_constant__ gs_block_norm_bwd_args a, int group, float* partial)
{
    extern __shared__ float part[];   // [groups][columns rounded up] when a block holds several groups
    __shared__ float sm[32];
    wait_for_predecessor();
    const int lane = threadIdx.x % group, groups = blockDim.x / group, cols = (int)a.cols;
    const float inv_cols = 1.0f / (float)a.cols;
    const bool post = a.post_weight != nullptr, gate_sum = a.dgate && !a.gate_rows;
    Weight<VEC, NV, 8> weight, post_weight, gate;   // beside the sums
    weight.init(a.weight, a.weight_type, lane, group, cols);
    post_weight.init(a.post_weight, a.post_type, lane, group, cols);
    gate.init(a.gate_rows ? nullptr : a.gate, a.gate_type, lane, group, cols);
    float acc[3][NV][VEC];
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[k][j][e] = 0.0f;
    const int64_t step = (int64_t)gridDim.x * groups * R;
    for (int64_t row0 = (int64_t)blockIdx.x * groups * R; row0 < a.rows; row0 += step) {
        const int64_t row = row0 + (int64_t)(threadIdx.x / group) * R;
        Cells<T, VEC> hr[R][NV], sr[R][NV], dr[R][NV], gr[R][NV];
        Cells<TDY, VEC> yr[R][NV];
        float rstd[R], rstd_post[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const bool here = row + i < a.rows;
            rstd[i] = a.dy && here ? a.rstd[row + i] : 0.0f;
            rstd_post[i] = post && here ? a.rstd_post[row + i] : 1.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = weight.col(j), n = cols - c;
                hr[i][j].zero(), sr[i][j].zero(), dr[i][j].zero(), gr[i][j].zero(), yr[i][j].zero();
                if (here && n > 0) {
                    if (a.dy) {
                        yr[i][j].load(a.dy, (row + i) * a.lddy + c, n, a.dy_type);
                        sr[i][j].load(a.s, (row + i) * a.lds + c, n, T);
                    }
                    if (a.ds) dr[i][j].load(a.ds, (row + i) * a.ldds + c, n, T);
                    if (post || a.dgate) hr[i][j].load(a.h, (row + i) * a.ldh + c, n, T);
                    if (a.gate_rows) gr[i][j].load(a.gate, (row + i) * a.ldg + c, n, T);
                }
            }
        }
        float g[R][NV][VEC], dot[R], c2[R];   // g: dy * weight, the gradient of s, that of a times post
#pragma unroll
        for (int i = 0; i < R; ++i) dot[i] = c2[i] = 0.0f;
        if (a.dy) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float w[VEC];
                weight.get(j, w);
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    float s[VEC], dy[VEC];
                    sr[i][j].values(T, s);
                    yr[i][j].values(a.dy_type, dy);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        acc[0][j][e] = __fmaf_rn(dy[e], s[e] * rstd[i], acc[0][j][e]);
                        g[i][j][e] = dy[e] * w[e];
                        dot[i] = __fmaf_rn(g[i][j][e], s[e], dot[i]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < R; ++i) dot[i] = group_reduce<Sum>(dot[i], group, sm);
#pragma unroll
            for (int i = 0; i < R; ++i) c2[i] = dot[i] * inv_cols * rstd[i] * rstd[i], dot[i] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = weight.col(j), n = cols - c;
            float w[VEC], g0[VEC];
            post_weight.get(j, w);
            gate.get(j, g0);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float h[VEC], v[VEC], gates[VEC];
                hr[i][j].values(T, h);
                dr[i][j].values(T, v);
                gr[i][j].values(T, gates);
                if (a.dy) {
                    float s[VEC];
                    sr[i][j].values(T, s);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) g[i][j][e] = __fmaf_rn(rstd[i], __fmaf_rn(-s[e], c2[i], g[i][j][e]), v[e]);
                } else
#pragma unroll
                    for (int e = 0; e < VEC; ++e) g[i][j][e] = v[e];
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[e] = a.scale * g[i][j][e];
                const bool there = row + i < a.rows && n > 0;
                if (a.dx && there) store_cells<VEC>(a.dx, (row + i) * a.lddx + c, n, T, v);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float unit = h[e] * rstd_post[i];
                    v[e] = g[i][j][e] * (post ? unit * w[e] : h[e]);   // the gate's gradient
                    acc[2][j][e] += v[e];
                    g[i][j][e] *= a.gate_rows ? gates[e] : g0[e];
                    acc[1][j][e] = __fmaf_rn(g[i][j][e], unit, acc[1][j][e]);
                    if (post) g[i][j][e] *= w[e];
                    dot[i] = __fmaf_rn(g[i][j][e], h[e], dot[i]);
                }
                if (a.dgate && a.gate_rows && there) store_cells<VEC>(a.dgate, (row + i) * a.lddg + c, n, T, v);
            }
        }
        if (!a.dh) continue;
        if (post) {
#pragma unroll
            for (int i = 0; i < R; ++i) dot[i] = group_reduce<Sum>(dot[i], group, sm);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            c2[i] = dot[i] * inv_cols * rstd_post[i] * rstd_post[i];
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = weight.col(j), n = cols - c;
                float h[VEC];
                hr[i][j].values(T, h);
                if (post)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) g[i][j][e] = rstd_post[i] * __fmaf_rn(-h[e], c2[i], g[i][j][e]);
                if (row + i < a.rows && n > 0) store_cells<VEC>(a.dh, (row + i) * a.lddh + c, n, T, g[i][j]);
            }
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
                for (int e = 0; e < VEC; ++e)
                    if (weight.col(j) + e < cols) out[weight.col(j) + e] = acc[k][j][e];
            continue;
        }
        const int width = NV * group * VEC;
        float* mine = part + (threadIdx.x / group) * width;
        __syncthreads();   // the sums before have been read
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) mine[weight.col(j) + e] = acc[k][j][e];
        __syncthreads();
        for (int c = threadIdx.x; c < cols; c += blockDim.x) {
            float t = 0.0f;
            for (int r = 0; r < groups; ++r) t += part[r * width + c];
            out[c] = t;
        }
    }
}

template <int V>
using Type = std::integral_constant<int, V>;

struct Shape {
    int nv, group, threads;
};
// Vectors of eight: one a thread within a warp, two where that keeps a row within it, then as
// many as 512 threads need.  Pairs: two a thread for rows within a warp, else eight, or sixteen.
Shape shape_for(int64_t cols, bool vec)
{
    const int64_t n = vec ? (cols + 7) / 8 : (cols + 1) / 2;
    Shape s;
    if (vec) s.nv = n <= 32 ? 1 : (n <= 1024 ? 2 : 4);
    else s.nv = n <= 64 ? 2 : (n <= 4096 ? 8 : 16);
    s.group = 1;
    while ((int64_t)s.group * s.nv < n) s.group *= 2;
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
    const Shape s = shape_for(a.cols, vec);
    // two rows a group where there are rows enough to fill the SMs all the same
    const bool two = vec && s.nv == 1 && a.rows >= (int64_t)sms * 4 * (s.threads / s.group) * 2;
    const int64_t rpb = s.threads / s.group * (two ? 2 : 1), want = (a.rows + rpb - 1) / rpb, most = (int64_t)sms * (two ? 4 : 2048 / s.threads);
    const int grid = (int)(want < most ? want : most);
    cudaStream_t st = (cudaStream_t)stream;
    const auto run = [&](auto t) -> gs_status {
        constexpr int T = decltype(t)::value;
#define GS_FWD(V, N, R) return launch_after(block_norm_kernel<T, V, N, R>, dim3(grid), s.threads, 0, 1, st, a, s.group)
        if (vec) {
            if (two) GS_FWD(8, 1, 2);
            else if (s.nv == 1) GS_FWD(8, 1, 1);
            else if (s.nv == 2) GS_FWD(8, 2, 1);
            else GS_FWD(8, 4, 1);
        } else if (s.nv == 2) GS_FWD(2, 2, 1);
        else if (s.nv == 8) GS_FWD(2, 8, 1);
        else GS_FWD(2, 16, 1);
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
    const bool same = !a.dy || a.dy_type == a.type;   // dy of another type goes by pairs
    const bool vec = same && a.cols % 8 == 0 && wide(a.dy, a.lddy, a.dy, a.dy_type) && wide(a.s, a.lds, a.dy, a.type) &&
                     wide(a.ds, a.ldds, a.ds, a.type) && wide(a.h, a.ldh, reads_h, a.type) && wide(a.gate, a.ldg, row_gate, a.type) &&
                     wide(a.dgate, a.lddg, row_dgate, a.type) && wide(a.dx, a.lddx, a.dx, a.type) && wide(a.dh, a.lddh, a.dh, a.type) &&
                     weight16(a.weight) && weight16(a.post_weight) && (row_gate || weight16(a.gate));
    const int v = vec ? 8 : 2;
    const Shape s = shape_for(a.cols, vec);
    const int groups = s.threads / s.group;
    const bool two = vec && s.nv == 1 && a.rows >= blocks * groups * 2;   // rows enough to fill the SMs
    const int64_t rpb = groups * (two ? 2 : 1), want = (a.rows + rpb - 1) / rpb;
    const int grid = (int)(want < blocks ? want : blocks);
    const size_t smem = groups > 1 && need ? (size_t)groups * s.nv * s.group * v * 4 : 0;   // at most 16 KB
    float* part = (float*)ws;
    const auto run = [&](auto t, auto tdy) -> gs_status {
        constexpr int T = decltype(t)::value, TDY = decltype(tdy)::value;
#define GS_BWD(V, N, R) return launch_after(block_norm_bwd_kernel<T, TDY, V, N, R>, dim3(grid), s.threads, smem, 1, st, a, s.group, part)
        if constexpr (T == TDY)
            if (vec) {
                if (two) GS_BWD(8, 1, 2);
                else if (s.nv == 1) GS_BWD(8, 1, 1);
                else if (s.nv == 2) GS_BWD(8, 2, 1);
                else GS_BWD(8, 4, 1);
            }
        if (s.nv == 2) GS_BWD(2, 2, 1);
        else if (s.nv == 8) GS_BWD(2, 8, 1);
        else GS_BWD(2, 16, 1);
#undef GS_BWD
    };
    const auto pick = [&](auto t) -> gs_status {
        if (same) return run(t, t);
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
