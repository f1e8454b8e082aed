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
#include <type_traits>

#include "gemm.cuh"
#include "rows.cuh"

namespace gs {
namespace {

using namespace rows;

// VEC consecutive elements of a row as they lie in memory, and as pairs in fp32.  Two elements
// are fetched one by one, whatever their alignment: a branch on it between loads would make
// each wait for the one before.
template <int T, int VEC>
struct Cells {
    Raw<T, 8> raw;
    __device__ __forceinline__ void zero() { raw_zero(raw); }
    __device__ __forceinline__ void load(const void* p, int64_t i, int, int type) { raw_load(raw, p, i, type); }
    __device__ __forceinline__ void values(int type, uint64_t (&v)[4]) const
    {
        float f[8];
        raw_values(raw, type, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = pair(f[2 * e], f[2 * e + 1]);
    }
};
template <int T>
struct Cells<T, 2> {
    Raw<T, 1> a, b;
    __device__ __forceinline__ void zero() { raw_zero(a), raw_zero(b); }
    __device__ __forceinline__ void load(const void* p, int64_t i, int n, int type)
    {
        raw_load(a, p, i, type);
        if (n > 1) raw_load(b, p, i + 1, type);
    }
    __device__ __forceinline__ void values(int type, uint64_t (&v)[1]) const
    {
        float x[1], y[1];
        raw_values(a, type, x);
        raw_values(b, type, y);
        v[0] = pair(x[0], y[0]);
    }
};

template <int VEC>
__device__ __forceinline__ void store_cells(void* p, int64_t i, int n, int type, const uint64_t (&v)[VEC / 2])
{
    float f[VEC];
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) {
        const float2 t = unpair(v[e]);
        f[2 * e] = t.x, f[2 * e + 1] = t.y;
    }
    if constexpr (VEC == 8) store8(p, i, type, f);
    else if (n > 1 && (type == GS_BF16 || type == GS_F16) && ((uintptr_t)((uint16_t*)p + i) & 3u) == 0)
        *reinterpret_cast<uint32_t*>((uint16_t*)p + i) = pack_half2(f[0], f[1], type);
    else
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (e < n) store_elem(p, i + e, type, f[e]);
}

// The thread's columns of a vector over them; 1 where there is none, 0 beyond the row.
template <int VEC>
__device__ __forceinline__ void load_weight(const void* p, int64_t i, int n, int type, uint64_t (&v)[VEC / 2])
{
    float f[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = e < n ? 1.0f : 0.0f;
    if (p && n > 0) {
        if constexpr (VEC == 8) load8(p, i, type, f);
        else
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (e < n) f[e] = load_elem(p, i + e, type);
    }
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) v[e] = pair(f[2 * e], f[2 * e + 1]);
}

// The product of one or two vectors over the columns.  Of up to 16 columns a thread they stay
// in registers, of more they are fetched from the first-level cache for every row.
template <int VEC, int NV>
struct Weight {
    static constexpr bool kKeep = VEC * NV <= 16;
    uint64_t v[kKeep ? NV : 1][VEC / 2];
    const void *p, *q;
    int p_type, q_type, lane, group, cols;
    __device__ __forceinline__ Weight(const void* p_, int p_type_, const void* q_, int q_type_, int lane_, int group_, int cols_)
        : p(p_), q(q_), p_type(p_type_), q_type(q_type_), lane(lane_), group(group_), cols(cols_)
    {
        if constexpr (kKeep)
#pragma unroll
            for (int j = 0; j < NV; ++j) fetch(j, v[j]);
    }
    __device__ __forceinline__ int col(int j) const { return (lane + j * group) * VEC; }
    __device__ __forceinline__ void fetch(int j, uint64_t (&w)[VEC / 2]) const
    {
        load_weight<VEC>(p, col(j), cols - col(j), p_type, w);
        if (q) {
            uint64_t t[VEC / 2];
            load_weight<VEC>(q, col(j), cols - col(j), q_type, t);
#pragma unroll
            for (int e = 0; e < VEC / 2; ++e) w[e] = mul2(w[e], t[e]);
        }
    }
    __device__ __forceinline__ void get(int j, uint64_t (&w)[VEC / 2]) const
    {
        if constexpr (kKeep)
#pragma unroll
            for (int e = 0; e < VEC / 2; ++e) w[e] = v[j][e];
        else fetch(j, w);
    }
};

__device__ __forceinline__ uint64_t both(float v) { return pair(v, v); }
__device__ __forceinline__ float sum_of(uint64_t v)
{
    const float2 f = unpair(v);
    return f.x + f.y;
}

// Threads of a block at most, and blocks an SM: one vector of eight a thread wants many warps
// of few registers; eight pairs a thread, each element in a register, need more than 128.
template <int VEC, int NV>
constexpr int kThreads = (VEC == 2 && NV == 8) || (VEC == 8 && NV == 1) ? 256 : 512;
template <int T, int VEC, int NV>
constexpr int kForwardBlocks = VEC == 8 && NV == 1 ? (T == GS_F32 ? 3 : 4) : 1;
template <int T, int VEC, int NV>
constexpr int kBackwardBlocks = VEC == 8 && NV == 1 ? (T == GS_F32 ? 2 : 3) : 1;

template <int T, int VEC, int NV>
__global__ void __launch_bounds__(kThreads<VEC, NV>, kForwardBlocks<T, VEC, NV>) block_norm_kernel(const __grid_constant__ gs_block_norm_args a, int group)
{
    constexpr int P = VEC / 2;
    constexpr bool kAhead = VEC * NV == 8;   // the next row's loads before this one's work
    __shared__ float sm[32];
    wait_for_predecessor();
    const int lane = threadIdx.x % group, cols = (int)a.cols;
    const int64_t step = (int64_t)gridDim.x * (blockDim.x / group);
    const float inv_cols = 1.0f / (float)a.cols;
    const bool q8 = a.y_type == GS_E4M3 && a.y;
    const Weight<VEC, NV> weight(a.weight, a.weight_type, nullptr, 0, lane, group, cols);
    const Weight<VEC, NV> post(a.post_weight, a.post_type, a.gate_rows ? nullptr : a.gate, a.gate_type, lane, group, cols);
    const uint64_t scale = both(a.scale);
    Cells<T, VEC> hr[NV], xr[NV], gr[NV];
    const auto load = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = weight.col(j), n = cols - c;
            hr[j].zero(), xr[j].zero();
            if (row < a.rows && n > 0) {
                hr[j].load(a.h, row * a.ldh + c, n, T);
                xr[j].load(a.x, row * a.ldx + c, n, T);
            }
        }
    };
    int64_t row = (int64_t)blockIdx.x * (blockDim.x / group) + threadIdx.x / group;
    if (kAhead) load(row);
    // every thread of a warp runs the same number of rounds (the reductions use whole warps)
    for (int64_t row0 = row - threadIdx.x / group; row0 < a.rows; row0 += step, row += step) {
        const bool here = row < a.rows;
        if (!kAhead) load(row);
        if (a.gate_rows)
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = weight.col(j), n = cols - c;
                gr[j].zero();
                if (here && n > 0) gr[j].load(a.gate, row * a.ldg + c, n, T);
            }
        uint64_t s[NV][P], x[NV][P], q = both(0.0f);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            hr[j].values(T, s[j]);
            xr[j].values(T, x[j]);
#pragma unroll
            for (int e = 0; e < P; ++e) q = fma2(s[j][e], s[j][e], q);
        }
        if (kAhead) load(row + step);
        float rstd_post = 1.0f;
        if (a.post_weight) {
            rstd_post = rsqrtf(group_reduce<Sum>(sum_of(q), group, sm) * inv_cols + a.eps);
            if (a.rstd_post && here && lane == 0) a.rstd_post[row] = rstd_post;
        }
        float top = 0.0f;
        q = both(0.0f);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = weight.col(j), n = cols - c;
            uint64_t p[P];
            post.get(j, p);   // with the gate's vector
#pragma unroll
            for (int e = 0; e < P; ++e) s[j][e] = mul2(mul2(s[j][e], both(rstd_post)), p[e]);
            if (a.gate_rows) {
                uint64_t g[P];
                gr[j].values(T, g);
#pragma unroll
                for (int e = 0; e < P; ++e) s[j][e] = mul2(s[j][e], g[e]);
            }
#pragma unroll
            for (int e = 0; e < P; ++e) {
                s[j][e] = fma2(scale, x[j][e], s[j][e]);
                q = fma2(s[j][e], s[j][e], q);
            }
            if (here && n > 0) store_cells<VEC>(a.s, row * a.lds + c, n, T, s[j]);
            if (q8) {
                uint64_t w[P];
                weight.get(j, w);
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    s[j][e] = mul2(s[j][e], w[e]);
                    const float2 f = unpair(s[j][e]);
                    top = max_nan(top, max_nan(fabsf(f.x), fabsf(f.y)));
                }
            }
        }
        if (!a.y) continue;
        const float rstd = rsqrtf(group_reduce<Sum>(sum_of(q), group, sm) * inv_cols + a.eps);
        float factor = rstd;
        if (q8) {   // e4m3 keeps 4 significant bits; the row's largest magnitude goes to 448
            top = max_nan(group_reduce<Max>(top, group, sm), kTiny);
            factor = kE4m3Max / top;
            if (here && lane == 0) a.y_scale[row] = (top / kE4m3Max) * rstd;
        }
        if (a.rstd && here && lane == 0) a.rstd[row] = rstd;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = weight.col(j), n = cols - c;
#pragma unroll
            for (int e = 0; e < P; ++e) s[j][e] = mul2(s[j][e], both(factor));
            if (!q8) {
                uint64_t w[P];
                weight.get(j, w);
#pragma unroll
                for (int e = 0; e < P; ++e) s[j][e] = mul2(s[j][e], w[e]);
            }
            if (here && n > 0) store_cells<VEC>(a.y, row * a.ldy + c, n, a.y_type, s[j]);
        }
    }
}

// Sums over rows: every thread keeps its columns' over the rows it visits, a block joins
// its groups' in order into partial rows, and JoinJobs adds the blocks' in order.
//   A = sum of g h rstd_post gives two of them where the gate is a vector: dgate = post A,
//   dpost = gate A; where it is rows, dpost sums g h rstd_post gate.
// partial: [3][blocks][cols]: dweight, dpost, dgate.
template <int T, int TDY, int VEC, int NV>
__global__ void __launch_bounds__(kThreads<VEC, NV>, kBackwardBlocks<T, VEC, NV>) block_norm_bwd_kernel(const __grid_constant__ gs_block_norm_bwd_args a,
                                                                                                   int group, float* partial)
{
    constexpr int P = VEC / 2;
    extern __shared__ float part[];   // [groups][columns rounded up] when a block holds several groups
    __shared__ float sm[32];
    wait_for_predecessor();
    const int lane = threadIdx.x % group, groups = blockDim.x / group, cols = (int)a.cols;
    const float inv_cols = 1.0f / (float)a.cols;
    const bool post = a.post_weight != nullptr;
    const void* gate = a.gate_rows ? nullptr : a.gate;
    const Weight<VEC, NV> weight(a.weight, a.weight_type, nullptr, 0, lane, group, cols);
    const Weight<VEC, NV> post_weight(a.post_weight, a.post_type, gate, a.gate_type, lane, group, cols);
    const uint64_t scale = both(a.scale);
    uint64_t acc[2][NV][P];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < P; ++e) acc[k][j][e] = both(0.0f);
    for (int64_t row0 = (int64_t)blockIdx.x * groups; row0 < a.rows; row0 += (int64_t)gridDim.x * groups) {
        const int64_t row = row0 + threadIdx.x / group;
        const bool here = row < a.rows;
        Cells<T, VEC> hr[NV], sr[NV], dr[NV], gr[NV];
        Cells<TDY, VEC> yr[NV];
        const float rstd = a.dy && here ? a.rstd[row] : 0.0f, rstd_post = post && here ? a.rstd_post[row] : 1.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = weight.col(j), n = cols - c;
            hr[j].zero(), sr[j].zero(), dr[j].zero(), gr[j].zero(), yr[j].zero();
            if (here && n > 0) {
                if (a.dy) {
                    yr[j].load(a.dy, row * a.lddy + c, n, a.dy_type);
                    sr[j].load(a.s, row * a.lds + c, n, T);
                }
                if (a.ds) dr[j].load(a.ds, row * a.ldds + c, n, T);
                if (post || a.dgate) hr[j].load(a.h, row * a.ldh + c, n, T);
                if (a.gate_rows) gr[j].load(a.gate, row * a.ldg + c, n, T);
            }
        }
        uint64_t g[NV][P], q = both(0.0f);   // g: dy * weight, the gradient of s, that of h / rms(h)
        float c2 = 0.0f;
        if (a.dy) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                uint64_t s[P], dy[P], w[P];
                weight.get(j, w);
                sr[j].values(T, s);
                yr[j].values(a.dy_type, dy);
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    acc[0][j][e] = fma2(dy[e], mul2(s[e], both(rstd)), acc[0][j][e]);
                    g[j][e] = mul2(dy[e], w[e]);
                    q = fma2(g[j][e], s[e], q);
                }
            }
            c2 = -group_reduce<Sum>(sum_of(q), group, sm) * inv_cols * rstd * rstd;
        }
        q = both(0.0f);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = weight.col(j), n = cols - c;
            const bool there = here && n > 0;
            uint64_t h[P], v[P], w[P];
            post_weight.get(j, w);   // with the gate's vector
            hr[j].values(T, h);
            dr[j].values(T, v);
            if (a.dy) {
                uint64_t s[P];
                sr[j].values(T, s);
#pragma unroll
                for (int e = 0; e < P; ++e) g[j][e] = fma2(both(rstd), fma2(s[e], both(c2), g[j][e]), v[e]);
            } else
#pragma unroll
                for (int e = 0; e < P; ++e) g[j][e] = v[e];
            if (a.dx && there) {
#pragma unroll
                for (int e = 0; e < P; ++e) v[e] = mul2(scale, g[j][e]);
                store_cells<VEC>(a.dx, row * a.lddx + c, n, T, v);
            }
            if (a.gate_rows) {
                uint64_t gates[P];
                gr[j].values(T, gates);
                if (a.dgate && there) {
#pragma unroll
                    for (int e = 0; e < P; ++e) v[e] = mul2(g[j][e], mul2(mul2(h[e], both(rstd_post)), w[e]));
                    store_cells<VEC>(a.dgate, row * a.lddg + c, n, T, v);
                }
#pragma unroll
                for (int e = 0; e < P; ++e) g[j][e] = mul2(g[j][e], gates[e]);
            }
#pragma unroll
            for (int e = 0; e < P; ++e) {
                acc[1][j][e] = fma2(g[j][e], mul2(h[e], both(rstd_post)), acc[1][j][e]);
                g[j][e] = mul2(g[j][e], w[e]);
                q = fma2(g[j][e], h[e], q);
            }
        }
        if (!a.dh) continue;
        if (post) c2 = -group_reduce<Sum>(sum_of(q), group, sm) * inv_cols * rstd_post * rstd_post;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = weight.col(j), n = cols - c;
            if (post) {
                uint64_t h[P];
                hr[j].values(T, h);
#pragma unroll
                for (int e = 0; e < P; ++e) g[j][e] = mul2(both(rstd_post), fma2(h[e], both(c2), g[j][e]));
            }
            if (here && n > 0) store_cells<VEC>(a.dh, row * a.lddh + c, n, T, g[j]);
        }
    }
    const auto write = [&](int which, const uint64_t (&v)[NV][P], const void* by, int by_type) {
        float* out = partial + ((int64_t)which * gridDim.x + blockIdx.x) * a.cols;
        const int width = NV * group * VEC;
        float* mine = groups == 1 ? out : part + (threadIdx.x / group) * width;
        __syncthreads();   // the sums before have been read
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = weight.col(j);
            uint64_t w[P];
            load_weight<VEC>(by, c, cols - c, by_type, w);
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const float2 f = unpair(mul2(v[j][e], w[e]));
                if (groups > 1 || c + 2 * e < cols) mine[c + 2 * e] = f.x;
                if (groups > 1 || c + 2 * e + 1 < cols) mine[c + 2 * e + 1] = f.y;
            }
        }
        if (groups == 1) return;
        __syncthreads();
        for (int c = threadIdx.x; c < cols; c += blockDim.x) {
            float t = 0.0f;
            for (int r = 0; r < groups; ++r) t += part[r * width + c];
            out[c] = t;
        }
    };
    if (a.dweight) write(0, acc[0], nullptr, 0);
    if (a.dpost) write(1, acc[1], gate, a.gate_type);
    if (a.dgate && !a.gate_rows) write(2, acc[1], a.post_weight, a.post_type);
}

template <int V>
using Type = std::integral_constant<int, V>;

struct Shape {
    int nv, group, threads;
};
// Vectors of eight: one a thread within a warp, two where that keeps a row within it, then as
// many as 512 threads need.  Pairs: two a thread for rows within a warp, else eight (256
// threads at most), or sixteen.
Shape shape_for(int64_t cols, bool vec, bool forward)
{
    const int64_t n = vec ? (cols + 7) / 8 : (cols + 1) / 2;
    Shape s;
    if (vec) s.nv = n <= 32 ? 1 : (n <= 1024 ? 2 : 4);
    else s.nv = n <= 64 ? 2 : (n <= 2048 ? 8 : 16);
    s.group = 1;
    while ((int64_t)s.group * s.nv < n) s.group *= 2;
    s.threads = s.group > (forward ? 32 : 256) ? s.group : 256;
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
    const Shape s = shape_for(a.cols, vec, true);
    const int64_t rpb = s.threads / s.group, want = (a.rows + rpb - 1) / rpb, most = (int64_t)sms * (1024 / s.threads);
    const int grid = (int)(want < most ? want : most);
    cudaStream_t st = (cudaStream_t)stream;
    const auto run = [&](auto t) -> gs_status {
        constexpr int T = decltype(t)::value;
#define GS_FWD(V, N) return launch_after(block_norm_kernel<T, V, N>, dim3(grid), s.threads, 0, 1, st, a, s.group)
        if (vec) {
            if (s.nv == 1) GS_FWD(8, 1);
            else if (s.nv == 2) GS_FWD(8, 2);
            else GS_FWD(8, 4);
        } else if (s.nv == 2) GS_FWD(2, 2);
        else if (s.nv == 8) GS_FWD(2, 8);
        else GS_FWD(2, 16);
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
    const Shape s = shape_for(a.cols, vec, false);
    const int groups = s.threads / s.group;
    const int64_t want = (a.rows + groups - 1) / groups;
    const int grid = (int)(want < blocks ? want : blocks);
    const size_t smem = groups > 1 && need ? (size_t)groups * s.nv * s.group * v * 4 : 0;   // at most 16 KB
    float* part = (float*)ws;
    const auto run = [&](auto t, auto tdy) -> gs_status {
        constexpr int T = decltype(t)::value, TDY = decltype(tdy)::value;
#define GS_BWD(V, N) return launch_after(block_norm_bwd_kernel<T, TDY, V, N>, dim3(grid), s.threads, smem, 1, st, a, s.group, part)
        if constexpr (T == TDY)
            if (vec) {
                if (s.nv == 1) GS_BWD(8, 1);
                else if (s.nv == 2) GS_BWD(8, 2);
                else GS_BWD(8, 4);
            }
        if (s.nv == 2) GS_BWD(2, 2);
        else if (s.nv == 8) GS_BWD(2, 8);
        else GS_BWD(2, 16);
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
