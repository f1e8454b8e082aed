// linear.cu -- entry points of gs_linear, gs_glu and their gradients: argument
// checks, the elementwise passes in front of the gradients' products, and the
// fixed-order joins of partial sums.  The products are in gemm.cu.
#include <type_traits>

#include "gemm.cuh"

namespace gs {
namespace {

// Gradient in front of the products: dz = dy * act'(z) rounded to the operands'
// type, and (DB) its column sums unrounded.  HBM bound: every value is read and
// written once.  A block owns tx VEC columns and takes 256 / tx rows at
// a time, gridDim.y blocks in turn; a thread keeps its columns' sums in registers over all its rows,
// the block joins them in row order and writes one partial row.
constexpr int kElemThreads = 256;
constexpr int kElemRows = 2;   // rows of a thread in flight (100,000 x 256, relu: 2 rows 22 us, 4 rows 28 us)

struct DzParams {
    const void* dy;
    const void* z;
    void* dz;         // NULL: column sums only
    float* partial;   // [gridDim.y][n] or NULL
    int64_t m, n, lddy, ldz, lddz;
    int dy_type;
};

template <int T, int TDY, int VEC, int ACT>
__global__ void __launch_bounds__(kElemThreads) dz_kernel(const __grid_constant__ DzParams p, int tx)
{
    wait_for_predecessor();
    __shared__ float part[kElemThreads * VEC];
    const int ty = kElemThreads / tx;                 // rows a block takes at a time
    const int x = threadIdx.x % tx, y = threadIdx.x / tx;
    const int64_t col = ((int64_t)blockIdx.x * tx + x) * VEC;
    float sum[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum[e] = 0.0f;
    if (col < p.n) {
        const int64_t step = (int64_t)gridDim.y * ty;
        for (int64_t row = (int64_t)blockIdx.y * ty + y; row < p.m; row += kElemRows * step) {
            Raw<TDY, VEC> gr[kElemRows];
            Raw<T, VEC> zr[kElemRows];
#pragma unroll
            for (int i = 0; i < kElemRows; ++i) {
                raw_zero(gr[i]);
                raw_zero(zr[i]);
                if (row + i * step < p.m) {
                    raw_load(gr[i], p.dy, (row + i * step) * p.lddy + col, p.dy_type);
                    if (ACT != GS_ACT_NONE) raw_load(zr[i], p.z, (row + i * step) * p.ldz + col, T);
                }
            }
#pragma unroll
            for (int i = 0; i < kElemRows; ++i) {
                float g[VEC], z[VEC];
                raw_values(gr[i], p.dy_type, g);
                if (ACT != GS_ACT_NONE) {
                    raw_values(zr[i], T, z);
                    if constexpr (VEC == 8) {
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            uint64_t value, slope;
                            act_both2<ACT, true, true>(pair(z[e], z[e + 1]), value, slope);
                            const float2 f = unpair(mul2(pair(g[e], g[e + 1]), slope));
                            g[e] = f.x, g[e + 1] = f.y;
                        }
                    } else g[0] *= act_slope(z[0], ACT);
                }
                if (p.dz && row + i * step < p.m) store_vec<VEC>(p.dz, (row + i * step) * p.lddz + col, T, g);
#pragma unroll
                for (int e = 0; e < VEC; ++e) sum[e] += g[e];
            }
        }
    }
    if (!p.partial) return;
#pragma unroll
    for (int e = 0; e < VEC; ++e) part[(y * tx + x) * VEC + e] = sum[e];
    __syncthreads();
    for (int i = threadIdx.x; i < tx * VEC; i += kElemThreads) {
        const int64_t c = (int64_t)blockIdx.x * tx * VEC + i;
        if (c >= p.n) continue;
        float t = 0.0f;
        for (int r = 0; r < ty; ++r) t += part[r * tx * VEC + i];
        p.partial[(int64_t)blockIdx.y * p.n + c] = t;
    }
}

struct GluGradParams {
    const void *dh, *g, *u;
    void *dg, *du;
    int64_t m, n, lddh, ldg, ldu, ldd;
};

// dg = dh * u * act'(g), du = dh * act(g).  HBM bound: three reads, two writes.
template <int T, int VEC, int ACT>
__global__ void __launch_bounds__(kElemThreads) glu_grad_kernel(const __grid_constant__ GluGradParams p, int tx)
{
    wait_for_predecessor();
    const int ty = kElemThreads / tx;
    const int64_t col = ((int64_t)blockIdx.x * tx + threadIdx.x % tx) * VEC;
    if (col >= p.n) return;
    const int64_t step = (int64_t)gridDim.y * ty;
    for (int64_t row = (int64_t)blockIdx.y * ty + threadIdx.x / tx; row < p.m; row += 2 * step) {
        Raw<T, VEC> dr[2], gr[2], ur[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t r = row + i * step;
            if (r >= p.m) continue;
            raw_load(dr[i], p.dh, r * p.lddh + col, T);
            raw_load(gr[i], p.g, r * p.ldg + col, T);
            raw_load(ur[i], p.u, r * p.ldu + col, T);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t r = row + i * step;
            if (r >= p.m) continue;
            float d[VEC], g[VEC], u[VEC];
            raw_values(dr[i], T, d);
            raw_values(gr[i], T, g);
            raw_values(ur[i], T, u);
            if constexpr (VEC == 8) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    uint64_t value, slope;
                    act_both2<ACT, false, false>(pair(g[e], g[e + 1]), value, slope);
                    const uint64_t q = pair(d[e], d[e + 1]);
                    const float2 a = unpair(mul2(mul2(q, pair(u[e], u[e + 1])), slope)), b = unpair(mul2(q, value));
                    g[e] = a.x, g[e + 1] = a.y;
                    u[e] = b.x, u[e + 1] = b.y;
                }
            } else {
                float value, slope;
                act_both<false>(g[0], ACT, value, slope);
                g[0] = d[0] * u[0] * slope;
                u[0] = d[0] * value;
            }
            store_vec<VEC>(p.dg, r * p.ldd + col, T, g);
            store_vec<VEC>(p.du, r * p.ldd + col, T, u);
        }
    }
}

// Sums of partial rows, in the order of the parts.  A thread takes four columns of one
// row (one where rows are not aligned); with slices > 1 it takes every slices-th part,
// and the block adds the slices in a tree.  Few parts of a large result: one slice, one
// pass at the reads' bandwidth; many parts of a small one (a decoder's weights over a
// million rows): up to 64.
template <int VEC>
__device__ __forceinline__ void join_job(const JoinJobs::Job& q, float4* sm)
{
    const int wide = 256 / q.slices, x = threadIdx.x % wide, y = threadIdx.x / wide;
    const uint32_t per_row = (q.cols + VEC - 1) / VEC;
    const uint32_t i = (blockIdx.x - q.first) * wide + x, r = i / per_row, c = (i - r * per_row) * VEC;
    const bool live = r < q.rows;
    float t[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) t[e] = 0.0f;
    if (live) {
        const float* at = q.partial + (int64_t)r * q.pitch + c;
#pragma unroll 4
        for (int p = y; p < q.parts; p += q.slices) {
            if constexpr (VEC == 4) {
                const float4 f = *reinterpret_cast<const float4*>(at + p * q.count);
                t[0] += f.x, t[1] += f.y, t[2] += f.z, t[3] += f.w;
            } else t[0] += at[p * q.count];
        }
    }
    if (q.slices > 1) {   // the same for the whole block: halves added to halves, a fixed tree
        float4* const mine = sm + threadIdx.x;
        *mine = make_float4(t[0], t[VEC > 1 ? 1 : 0], t[VEC > 1 ? 2 : 0], t[VEC > 1 ? 3 : 0]);
        for (int half = q.slices / 2; half > 0; half /= 2) {
            __syncthreads();
            if (y < half) {
                const float4 o = mine[half * wide], m = *mine;
                *mine = make_float4(m.x + o.x, m.y + o.y, m.z + o.z, m.w + o.w);
            }
        }
        if (y > 0) return;
        t[0] = mine->x;
        if constexpr (VEC > 1) t[1] = mine->y, t[2] = mine->z, t[3] = mine->w;
    }
    if (!live) return;
    const int64_t to = (int64_t)r * q.ld + c;
    if constexpr (VEC == 4) {
        const size_t bytes = q.type == GS_F32 ? 4 : 2;
        if (c + 4 <= q.cols && (((uintptr_t)q.out + (size_t)to * bytes) & (4 * bytes - 1)) == 0) {
            if (q.type == GS_F32) *reinterpret_cast<float4*>((float*)q.out + to) = make_float4(t[0], t[1], t[2], t[3]);
            else
                *reinterpret_cast<uint2*>((uint16_t*)q.out + to) =
                    make_uint2(pack_half2(t[0], t[1], q.type), pack_half2(t[2], t[3], q.type));
            return;
        }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e)
        if (c + e < q.cols) store_elem(q.out, to + e, q.type, t[e]);
}

__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ JoinJobs p)
{
    wait_for_predecessor();
    __shared__ float4 sm[256];
    int j = 0;
    while (j + 1 < p.jobs && blockIdx.x >= p.job[j + 1].first) ++j;
    if (p.job[j].vec) join_job<4>(p.job[j], sm);
    else join_job<1>(p.job[j], sm);
}

// Thread columns of an elementwise block: a power of two that covers the row
// when it is narrow, a block's width at most.
int thread_cols(int64_t n, int vec)
{
    int tx = 1;
    while (tx < 64 && (int64_t)tx * vec < n) tx *= 2;
    return tx;
}

// Multiprocessors, also where a size is asked for without a device.
int64_t sms_or_default() { return device_sms() > 0 ? device_sms() : 152; }

int64_t slabs_for(int64_t m, int64_t n, int vec)
{
    const int tx = thread_cols(n, vec), ty = kElemThreads / tx;
    const int64_t cb = (n + (int64_t)tx * vec - 1) / ((int64_t)tx * vec);
    int64_t s = (4 * sms_or_default() + cb - 1) / cb;   // about four blocks an SM over the column blocks
    const int64_t most = (m + ty - 1) / ty;
    return s < most ? s : (most > 0 ? most : 1);
}

gs_status check_sizes(int64_t rows, int64_t in, int64_t out)
{
    return size_ok(rows, 0) && size_ok(in, 1) && size_ok(out, 1) ? GS_OK : GS_ERR_INVALID_ARG;
}

gs_status zero_rows(void* p, int64_t ld, int64_t rows, int64_t cols, int type, cudaStream_t st)
{
    const size_t e = type_bytes(type);
    GS_CUDA_TRY(cudaMemset2DAsync(p, (size_t)ld * e, 0, (size_t)cols * e, (size_t)rows, st));
    return GS_OK;
}

// Offsets of the parts of a workspace.
struct Scratch {
    size_t used = 0;
    size_t take(size_t bytes)
    {
        const size_t at = used;
        used += (size_t)round_up((int64_t)bytes, 256);
        return at;
    }
};

// Rows of any alignment to rows of 16-byte base and pitch: eight 2-byte or sixteen
// 1-byte elements a thread, one 16-byte store.  All factors of a call in one launch.
struct PackJobs {
    struct {
        const void* src;
        uint4* dst;
        int64_t ld, rows, cols, pieces;
        unsigned first;   // block
    } job[4];
    int jobs = 0;
};
template <typename E>
__global__ void __launch_bounds__(256) pack_rows_kernel(const __grid_constant__ PackJobs p)
{
    wait_for_predecessor();
    constexpr int kPer = 16 / sizeof(E);
    int j = 0;
    while (j + 1 < p.jobs && blockIdx.x >= p.job[j + 1].first) ++j;
    const unsigned end = j + 1 < p.jobs ? p.job[j + 1].first : gridDim.x;
    const auto& q = p.job[j];
    const E* src = (const E*)q.src;
    const int64_t total = q.rows * q.pieces, step = (int64_t)(end - q.first) * blockDim.x;
    for (int64_t i = (int64_t)(blockIdx.x - q.first) * blockDim.x + threadIdx.x; i < total; i += step) {
        const int64_t r = i / q.pieces, c0 = i % q.pieces * kPer;
        union {
            uint4 v;
            E e[kPer];
        } v;
#pragma unroll
        for (int e = 0; e < kPer; ++e) v.e[e] = c0 + e < q.cols ? src[r * q.ld + c0 + e] : (E)0;
        q.dst[i] = v.v;
    }
}

// A call's factor as the products take it: where it lies if its rows are aligned, else
// a copy in the workspace, made by pack_all.
struct Rows {
    const void* p = nullptr;
    int64_t ld = 0;
    const void* src = nullptr;   // set where a copy is made
    int64_t src_ld = 0, rows = 0, cols = 0;
    size_t at = 0;
};

Rows aligned_rows(Scratch& sc, bool used, const void* p, int64_t ld, int64_t rows, int64_t cols, int type)
{
    Rows r;
    r.p = p, r.ld = ld;
    if (!used || rows16(p, ld, type)) return r;
    const int64_t esz = type_bytes(type);
    r.src = p, r.src_ld = ld, r.rows = rows, r.cols = cols;
    r.ld = round_up(cols * esz, 16) / esz;
    r.at = sc.take((size_t)(rows * r.ld * esz));
    r.p = nullptr;
    return r;
}

gs_status pack_all(Rows* const* list, int n, char* base, int type, cudaStream_t st)
{
    PackJobs jobs;
    unsigned blocks = 0;
    const int64_t esz = type_bytes(type), most = 16 * sms_or_default();
    for (int i = 0; i < n; ++i) {
        Rows& r = *list[i];
        if (!r.src) continue;
        r.p = base + r.at;
        auto& job = jobs.job[jobs.jobs++];
        job.src = r.src, job.dst = (uint4*)r.p;
        job.ld = r.src_ld, job.rows = r.rows, job.cols = r.cols, job.pieces = r.ld * esz / 16;
        job.first = blocks;
        const int64_t want = (job.rows * job.pieces + 255) / 256;
        blocks += (unsigned)(want < most ? want : most);
    }
    if (!blocks) return GS_OK;
    return launch_after(esz == 2 ? pack_rows_kernel<uint16_t> : pack_rows_kernel<uint8_t>, dim3(blocks), 256, 0, 1, st, jobs);
}

}  // namespace

gs_status JoinJobs::add(const float* partial, int64_t parts, int64_t rows, int64_t cols, int64_t pitch, void* out, int64_t ld,
                        int type)
{
    if (jobs == 4) return GS_ERR_INVALID_ARG;
    Job& q = job[jobs++];
    q.vec = pitch % 4 == 0 && aligned16(partial);
    const int64_t threads = rows * (q.vec ? (cols + 3) / 4 : cols);
    // one thread a result where they fill the SMs; else so many that they do, eight parts each at least
    q.slices = 1;
    while (q.slices < 64 && threads * q.slices < sms_or_default() * 512 && parts >= 8 * q.slices) q.slices *= 2;
    const int64_t wide = 256 / q.slices, n = (threads + wide - 1) / wide;
    if (n + blocks > 0x7fffffll || threads > 0x7fffffffll) return GS_ERR_INVALID_ARG;
    q.partial = partial, q.out = out, q.count = rows * pitch, q.ld = ld;
    q.rows = (uint32_t)rows, q.cols = (uint32_t)cols, q.pitch = (uint32_t)pitch, q.first = blocks;
    q.parts = (int)parts, q.type = type;
    blocks += (unsigned)n;
    return GS_OK;
}

gs_status JoinJobs::run(cudaStream_t st) const
{
    if (!jobs) return GS_OK;
    return launch_after(join_kernel, dim3(blocks), 256, 0, 1, st, *this);
}

}  // namespace gs

using namespace gs;

extern "C" gs_status gs_linear(const gs_linear_args* args, void* ws, size_t* ws_bytes, void* stream)
{
    GS_NVTX_RANGE("gs_linear");
    if (!args) return GS_ERR_INVALID_ARG;
    const gs_linear_args& a = *args;
    if (check_sizes(a.rows, a.in_features, a.out_features) != GS_OK) return GS_ERR_INVALID_ARG;
    if (!(type_half(a.type) || a.type == GS_E4M3) || !type_float(a.out_type) || !act_ok(a.act)) return GS_ERR_INVALID_ARG;
    if (a.type != GS_E4M3 && (a.x_scale || a.w_scale)) return GS_ERR_INVALID_ARG;
    if (a.bias && (!type_float(a.bias_type) || !vec_ok(a.bias, a.bias_type))) return GS_ERR_INVALID_ARG;
    if (!vec_ok(a.x_scale, GS_F32) || !vec_ok(a.w_scale, GS_F32)) return GS_ERR_INVALID_ARG;
    if (!mat_ok(a.w, a.ldw, a.in_features, a.type)) return GS_ERR_INVALID_ARG;
    if (a.rows > 0) {
        if (!mat_ok(a.x, a.ldx, a.in_features, a.type) || !mat_ok(a.y, a.ldy, a.out_features, a.out_type))
            return GS_ERR_INVALID_ARG;
        if (a.residual && !mat_ok(a.residual, a.ldr, a.out_features, a.out_type)) return GS_ERR_INVALID_ARG;
        if (a.z && (!type_half(a.type) || !mat_ok(a.z, a.ldz, a.out_features, a.type))) return GS_ERR_INVALID_ARG;
    }
    GemmCall c = {};
    c.kind = GemmKind::kLinear;
    c.m = a.rows, c.n = a.out_features, c.k = a.in_features, c.type = a.type;
    c.x_scale = a.x_scale, c.w_scale[0] = a.w_scale;
    c.bias = a.bias, c.bias_type = a.bias_type, c.act = a.act;
    c.residual = a.residual, c.ldr = a.ldr;
    c.y = a.y, c.ldy = a.ldy, c.out_type = a.out_type;
    c.z = a.z, c.ldz = a.ldz, c.z_type = a.type;
    c.a[0].k_fast = c.b[0].k_fast = true;
    GemmPlan plan = {};
    Scratch sc;
    Rows x, w;
    size_t at = 0;
    if (a.rows > 0) {
        plan = gemm_plan(c);
        if (!gemm_fits(plan)) return GS_ERR_INVALID_ARG;
        x = aligned_rows(sc, true, a.x, a.ldx, c.m, c.k, a.type);
        w = aligned_rows(sc, true, a.w, a.ldw, c.n, c.k, a.type);
        at = sc.take(plan.bytes);
    }
    const WsCheck wc = ws_check(ws, ws_bytes, sc.used);
    if (wc == WsCheck::kBad) return GS_ERR_INVALID_ARG;
    if (wc == WsCheck::kQuery || a.rows == 0) return GS_OK;
    cudaStream_t st = (cudaStream_t)stream;
    Rows* const list[] = {&x, &w};
    gs_status s = pack_all(list, 2, (char*)ws, a.type, st);
    if (s != GS_OK) return s;
    c.a[0] = {x.p, x.ld, true}, c.b[0] = {w.p, w.ld, true};
    JoinJobs joins;
    s = gemm_run(c, plan, (char*)ws + at, &joins, st);
    return s != GS_OK ? s : joins.run(st);
}

extern "C" gs_status gs_linear_bwd(const gs_linear_bwd_args* args, void* ws, size_t* ws_bytes, void* stream)
{
    GS_NVTX_RANGE("gs_linear_bwd");
    if (!args) return GS_ERR_INVALID_ARG;
    const gs_linear_bwd_args& a = *args;
    const int64_t m = a.rows, k = a.in_features, n = a.out_features;
    if (check_sizes(m, k, n) != GS_OK) return GS_ERR_INVALID_ARG;
    if (!type_half(a.type) || !type_float(a.dy_type) || !act_ok(a.act)) return GS_ERR_INVALID_ARG;
    if (a.dw && ((a.dw_type != a.type && a.dw_type != GS_F32) || !mat_ok(a.dw, a.lddw, k, a.dw_type)))
        return GS_ERR_INVALID_ARG;
    if (a.db && (!type_float(a.db_type) || !vec_ok(a.db, a.db_type))) return GS_ERR_INVALID_ARG;
    if (m > 0) {
        if (!mat_ok(a.dy, a.lddy, n, a.dy_type)) return GS_ERR_INVALID_ARG;
        if (a.act != GS_ACT_NONE && !mat_ok(a.z, a.ldz, n, a.type)) return GS_ERR_INVALID_ARG;
        if (a.dx && (!mat_ok(a.dx, a.lddx, k, a.type) || !mat_ok(a.w, a.ldw, k, a.type))) return GS_ERR_INVALID_ARG;
        if (a.dw && !mat_ok(a.x, a.ldx, k, a.type)) return GS_ERR_INVALID_ARG;
    }
    const bool plain = a.act == GS_ACT_NONE && a.dy_type == a.type;   // dz is dy
    const bool products = a.dx || a.dw;
    const bool make_dz = !plain && products;
    const int64_t lddz = round_up(n, 8);
    const bool vec = n % 8 == 0 && rows16(a.dy, a.lddy, a.dy_type) &&
                     (a.act == GS_ACT_NONE || rows16(a.z, a.ldz, a.type));
    Scratch sc;
    const size_t at_dz = make_dz ? sc.take((size_t)m * lddz * 2) : 0;
    const size_t at_db = a.db ? sc.take((size_t)slabs_for(m, n, vec ? 8 : 1) * n * 4) : 0;
    GemmCall cx = {}, cw = {};
    cx.kind = cw.kind = GemmKind::kLinear;
    cx.type = cw.type = a.type;
    cx.a[0].k_fast = true;   // the others' fast index is not the contracted one
    cx.m = m, cx.n = k, cx.k = n;
    cx.y = a.dx, cx.ldy = a.lddx, cx.out_type = a.type;
    cw.m = n, cw.n = k, cw.k = m;
    cw.y = a.dw, cw.ldy = a.lddw, cw.out_type = a.dw_type;
    GemmPlan px = {}, pw = {};
    if (m > 0 && a.dx) px = gemm_plan(cx);
    if (m > 0 && a.dw) pw = gemm_plan(cw);
    if (!gemm_fits(px) || !gemm_fits(pw)) return GS_ERR_INVALID_ARG;
    Rows dz = aligned_rows(sc, m > 0 && products && !make_dz, a.dy, a.lddy, m, n, a.type);
    Rows w = aligned_rows(sc, m > 0 && a.dx, a.w, a.ldw, n, k, a.type);
    Rows x = aligned_rows(sc, m > 0 && a.dw, a.x, a.ldx, m, k, a.type);
    const size_t at_x = sc.take(px.bytes), at_w = sc.take(pw.bytes);
    const WsCheck wc = ws_check(ws, ws_bytes, sc.used);
    if (wc == WsCheck::kBad) return GS_ERR_INVALID_ARG;
    if (wc == WsCheck::kQuery) return GS_OK;
    cudaStream_t st = (cudaStream_t)stream;
    if (m == 0) {
        if (a.dw && zero_rows(a.dw, a.lddw, n, k, a.dw_type, st) != GS_OK) return GS_ERR_CUDA;
        if (a.db && zero_rows(a.db, n, 1, n, a.db_type, st) != GS_OK) return GS_ERR_CUDA;
        return GS_OK;
    }
    char* base = (char*)ws;
    JoinJobs joins;
    if (make_dz || a.db) {
        DzParams p = {};
        p.dy = a.dy, p.z = a.z, p.dz = make_dz ? base + at_dz : nullptr;
        p.partial = a.db ? (float*)(base + at_db) : nullptr;
        p.m = m, p.n = n, p.lddy = a.lddy, p.ldz = a.ldz, p.lddz = lddz;
        p.dy_type = a.dy_type;
        const int v = vec ? 8 : 1, tx = thread_cols(n, v);
        const int64_t slabs = slabs_for(m, n, v);
        const dim3 grid((unsigned)((n + (int64_t)tx * v - 1) / ((int64_t)tx * v)), (unsigned)slabs);
        const gs_status launched = for_type_act(a.type, a.act, [&](auto t, auto act) {
            constexpr int T = decltype(t)::value, ACT = decltype(act)::value;
            const bool same = a.dy_type == a.type;
            return launch_after(vec ? (same ? dz_kernel<T, T, 8, ACT> : dz_kernel<T, kAnyType, 8, ACT>)
                                    : (same ? dz_kernel<T, T, 1, ACT> : dz_kernel<T, kAnyType, 1, ACT>),
                                grid, kElemThreads, 0, 1, st, p, tx);
        });
        if (launched != GS_OK) return launched;
        if (a.db) {
            const gs_status s = joins.add(p.partial, slabs, 1, n, n, a.db, n, a.db_type);
            if (s != GS_OK) return s;
        }
        if (make_dz) dz.p = base + at_dz, dz.ld = lddz;
    }
    Rows* const list[] = {&dz, &w, &x};
    const gs_status packed = pack_all(list, 3, base, a.type, st);
    if (packed != GS_OK) return packed;
    cx.a[0] = {dz.p, dz.ld, true}, cx.b[0] = {w.p, w.ld, false};
    cw.a[0] = {dz.p, dz.ld, false}, cw.b[0] = {x.p, x.ld, false};
    if (a.dx) {
        const gs_status s = gemm_run(cx, px, base + at_x, &joins, st);
        if (s != GS_OK) return s;
    }
    if (a.dw) {
        const gs_status s = gemm_run(cw, pw, base + at_w, &joins, st);
        if (s != GS_OK) return s;
    }
    return joins.run(st);
}

extern "C" gs_status gs_glu(const gs_glu_args* args, void* ws, size_t* ws_bytes, void* stream)
{
    GS_NVTX_RANGE("gs_glu");
    if (!args) return GS_ERR_INVALID_ARG;
    const gs_glu_args& a = *args;
    if (check_sizes(a.rows, a.in_features, a.hidden) != GS_OK) return GS_ERR_INVALID_ARG;
    if (!(type_half(a.type) || a.type == GS_E4M3) || !type_half(a.out_type) || !act_ok(a.act)) return GS_ERR_INVALID_ARG;
    if (a.type != GS_E4M3 && (a.out_type != a.type || a.x_scale || a.gate_scale || a.up_scale)) return GS_ERR_INVALID_ARG;
    if (!vec_ok(a.x_scale, GS_F32) || !vec_ok(a.gate_scale, GS_F32) || !vec_ok(a.up_scale, GS_F32))
        return GS_ERR_INVALID_ARG;
    if (!mat_ok(a.w_gate, a.ldwg, a.in_features, a.type) || !mat_ok(a.w_up, a.ldwu, a.in_features, a.type))
        return GS_ERR_INVALID_ARG;
    if (!a.g != !a.u) return GS_ERR_INVALID_ARG;
    if (a.rows > 0) {
        if (!mat_ok(a.x, a.ldx, a.in_features, a.type) || !mat_ok(a.h, a.ldh, a.hidden, a.out_type))
            return GS_ERR_INVALID_ARG;
        if (a.g && (!mat_ok(a.g, a.ldg, a.hidden, a.out_type) || !mat_ok(a.u, a.ldu, a.hidden, a.out_type)))
            return GS_ERR_INVALID_ARG;
    }
    GemmCall c = {};
    c.kind = GemmKind::kGlu;
    c.m = a.rows, c.n = a.hidden, c.k = a.in_features, c.type = a.type;
    c.x_scale = a.x_scale, c.w_scale[0] = a.gate_scale, c.w_scale[1] = a.up_scale;
    c.act = a.act;
    c.y = a.h, c.ldy = a.ldh, c.out_type = c.z_type = a.out_type;
    c.z = a.g, c.ldz = a.ldg, c.z2 = a.u, c.ldz2 = a.ldu;
    c.a[0].k_fast = c.b[0].k_fast = true;
    GemmPlan plan = {};
    Scratch sc;
    Rows x, wg, wu;
    if (a.rows > 0) {
        plan = gemm_plan(c);
        if (!gemm_fits(plan)) return GS_ERR_INVALID_ARG;
        x = aligned_rows(sc, true, a.x, a.ldx, c.m, c.k, a.type);
        wg = aligned_rows(sc, true, a.w_gate, a.ldwg, c.n, c.k, a.type);
        wu = aligned_rows(sc, true, a.w_up, a.ldwu, c.n, c.k, a.type);
    }
    const WsCheck wc = ws_check(ws, ws_bytes, sc.used);
    if (wc == WsCheck::kBad) return GS_ERR_INVALID_ARG;
    if (wc == WsCheck::kQuery || a.rows == 0) return GS_OK;
    cudaStream_t st = (cudaStream_t)stream;
    Rows* const list[] = {&x, &wg, &wu};
    const gs_status s = pack_all(list, 3, (char*)ws, a.type, st);
    if (s != GS_OK) return s;
    c.a[0] = {x.p, x.ld, true};
    c.b[0] = {wg.p, wg.ld, true}, c.b[1] = {wu.p, wu.ld, true};
    return gemm_run(c, plan, nullptr, nullptr, st);   // a gated layer never splits k
}

// Checked arguments, at least one row.
static gs_status narrow_glu_bwd(const gs_glu_bwd_args& a, void* ws, size_t* ws_bytes, cudaStream_t st)
{
    Scratch sc;
    Rows x = aligned_rows(sc, true, a.x, a.ldx, a.rows, a.in_features, a.type);
    Rows dh = aligned_rows(sc, true, a.dh, a.lddh, a.rows, a.hidden, a.type);
    Rows wg = aligned_rows(sc, true, a.w_gate, a.ldwg, a.hidden, a.in_features, a.type);
    Rows wu = aligned_rows(sc, true, a.w_up, a.ldwu, a.hidden, a.in_features, a.type);
    const int64_t pitch = round_up(a.in_features, 4), blocks = glu_narrow_blocks(a.rows);
    const size_t bytes = a.dw_gate ? (size_t)(blocks * a.hidden * pitch) * 4 : 0;
    const size_t at_g = sc.take(bytes), at_u = sc.take(bytes);
    const WsCheck wc = ws_check(ws, ws_bytes, sc.used);
    if (wc == WsCheck::kBad) return GS_ERR_INVALID_ARG;
    if (wc == WsCheck::kQuery) return GS_OK;
    char* base = (char*)ws;
    Rows* const list[] = {&x, &dh, &wg, &wu};
    gs_status s = pack_all(list, 4, base, a.type, st);
    if (s != GS_OK) return s;
    GluNarrowCall c = {};
    c.rows = a.rows, c.features = a.in_features, c.hidden = a.hidden, c.type = a.type, c.act = a.act;
    c.x = x.p, c.ldx = x.ld, c.dh = dh.p, c.lddh = dh.ld;
    c.w_gate = wg.p, c.ldwg = wg.ld, c.w_up = wu.p, c.ldwu = wu.ld;
    c.dx = a.dx, c.lddx = a.lddx, c.pitch = pitch;
    if (a.dw_gate) c.dw_gate = (float*)(base + at_g), c.dw_up = (float*)(base + at_u);
    s = glu_narrow_grad(c, st);
    if (s != GS_OK || !a.dw_gate) return s;
    JoinJobs joins;
    s = joins.add(c.dw_gate, blocks, a.hidden, a.in_features, pitch, a.dw_gate, a.lddwg, a.dw_type);
    if (s == GS_OK) s = joins.add(c.dw_up, blocks, a.hidden, a.in_features, pitch, a.dw_up, a.lddwu, a.dw_type);
    return s != GS_OK ? s : joins.run(st);
}

extern "C" gs_status gs_glu_bwd(const gs_glu_bwd_args* args, void* ws, size_t* ws_bytes, void* stream)
{
    GS_NVTX_RANGE("gs_glu_bwd");
    if (!args) return GS_ERR_INVALID_ARG;
    const gs_glu_bwd_args& a = *args;
    const int64_t m = a.rows, k = a.in_features, f = a.hidden;
    if (check_sizes(m, k, f) != GS_OK) return GS_ERR_INVALID_ARG;
    if (!type_half(a.type) || !act_ok(a.act) || !a.dw_gate != !a.dw_up || !a.g != !a.u) return GS_ERR_INVALID_ARG;
    if (a.dw_gate && ((a.dw_type != a.type && a.dw_type != GS_F32) || !mat_ok(a.dw_gate, a.lddwg, k, a.dw_type) ||
                      !mat_ok(a.dw_up, a.lddwu, k, a.dw_type)))
        return GS_ERR_INVALID_ARG;
    if (m > 0) {
        if (!mat_ok(a.dh, a.lddh, f, a.type)) return GS_ERR_INVALID_ARG;
        if (a.g && (!mat_ok(a.g, a.ldg, f, a.type) || !mat_ok(a.u, a.ldu, f, a.type))) return GS_ERR_INVALID_ARG;
        if (a.dx && !mat_ok(a.dx, a.lddx, k, a.type)) return GS_ERR_INVALID_ARG;
        if ((a.dx || !a.g) && (!mat_ok(a.w_gate, a.ldwg, k, a.type) || !mat_ok(a.w_up, a.ldwu, k, a.type)))
            return GS_ERR_INVALID_ARG;
        if ((a.dw_gate || !a.g) && !mat_ok(a.x, a.ldx, k, a.type)) return GS_ERR_INVALID_ARG;
    }
    const bool again = !a.g;   // the projections are computed again
    if (again && m > 0 && (a.dx || a.dw_gate) && glu_narrow_fits(k, f)) return narrow_glu_bwd(a, ws, ws_bytes, (cudaStream_t)stream);
    const int64_t ldd = round_up(f, 8);
    Scratch sc;
    const size_t at_dg = sc.take((size_t)m * ldd * 2), at_du = sc.take((size_t)m * ldd * 2);
    GemmCall cx = {}, cw = {};
    cx.kind = GemmKind::kSum, cw.kind = GemmKind::kTwo;
    cx.type = cw.type = a.type;
    cx.m = m, cx.n = k, cx.k = f;
    cx.a[0].k_fast = cx.a[1].k_fast = true;
    cx.y = a.dx, cx.ldy = a.lddx, cx.out_type = a.type;
    cw.m = f, cw.n = k, cw.k = m;
    cw.y = a.dw_gate, cw.ldy = a.lddwg, cw.y2 = a.dw_up, cw.ldy2 = a.lddwu, cw.out_type = a.dw_type;
    GemmCall cg = {};
    cg.kind = GemmKind::kGluGrad;
    cg.m = m, cg.n = f, cg.k = k, cg.type = a.type;
    cg.a[0].k_fast = cg.b[0].k_fast = cg.b[1].k_fast = true;
    cg.residual = a.dh, cg.ldr = a.lddh, cg.act = a.act, cg.out_type = a.type;
    cg.ldy = cg.ldy2 = ldd;
    GemmPlan px = {}, pw = {}, pg = {};
    if (m > 0 && a.dx) px = gemm_plan(cx);
    if (m > 0 && a.dw_gate) pw = gemm_plan(cw);
    if (m > 0 && again) pg = gemm_plan(cg);
    if (!gemm_fits(px) || !gemm_fits(pw) || !gemm_fits(pg)) return GS_ERR_INVALID_ARG;
    Rows x = aligned_rows(sc, m > 0 && (again || a.dw_gate), a.x, a.ldx, m, k, a.type);
    Rows wg = aligned_rows(sc, m > 0 && (again || a.dx), a.w_gate, a.ldwg, f, k, a.type);
    Rows wu = aligned_rows(sc, m > 0 && (again || a.dx), a.w_up, a.ldwu, f, k, a.type);
    const size_t at_x = sc.take(px.bytes), at_w = sc.take(pw.bytes);
    const WsCheck wc = ws_check(ws, ws_bytes, sc.used);
    if (wc == WsCheck::kBad) return GS_ERR_INVALID_ARG;
    if (wc == WsCheck::kQuery) return GS_OK;
    cudaStream_t st = (cudaStream_t)stream;
    if (m == 0) {
        if (a.dw_gate && (zero_rows(a.dw_gate, a.lddwg, f, k, a.dw_type, st) != GS_OK ||
                          zero_rows(a.dw_up, a.lddwu, f, k, a.dw_type, st) != GS_OK))
            return GS_ERR_CUDA;
        return GS_OK;
    }
    if (!a.dx && !a.dw_gate) return GS_OK;
    char* base = (char*)ws;
    JoinJobs joins;
    Rows* const list[] = {&x, &wg, &wu};
    const gs_status packed = pack_all(list, 3, base, a.type, st);
    if (packed != GS_OK) return packed;
    if (again) {
        cg.a[0] = {x.p, x.ld, true};
        cg.b[0] = {wg.p, wg.ld, true}, cg.b[1] = {wu.p, wu.ld, true};
        cg.y = base + at_dg, cg.y2 = base + at_du;
        const gs_status s = gemm_run(cg, pg, nullptr, nullptr, st);
        if (s != GS_OK) return s;
    }
    GluGradParams p = {};
    p.dh = a.dh, p.g = a.g, p.u = a.u, p.dg = base + at_dg, p.du = base + at_du;
    p.m = m, p.n = f, p.lddh = a.lddh, p.ldg = a.ldg, p.ldu = a.ldu, p.ldd = ldd;
    const bool vec = f % 8 == 0 && rows16(a.dh, a.lddh, a.type) && rows16(a.g, a.ldg, a.type) &&
                     rows16(a.u, a.ldu, a.type);
    const int v = vec ? 8 : 1, tx = thread_cols(f, v), ty = kElemThreads / tx;
    int64_t gy = (m + 2 * ty - 1) / (2 * ty);
    if (gy > 65535) gy = 65535;
    const dim3 grid((unsigned)((f + (int64_t)tx * v - 1) / ((int64_t)tx * v)), (unsigned)gy);
    if (!again) {
        const gs_status launched = for_type_act(a.type, a.act, [&](auto t, auto act) {
            constexpr int T = decltype(t)::value, ACT = decltype(act)::value;
            return launch_after(vec ? glu_grad_kernel<T, 8, ACT> : glu_grad_kernel<T, 1, ACT>, grid, kElemThreads, 0, 1, st, p,
                                tx);
        });
        if (launched != GS_OK) return launched;
    }
    cx.a[0] = {p.dg, ldd, true}, cx.a[1] = {p.du, ldd, true};
    cx.b[0] = {wg.p, wg.ld, false}, cx.b[1] = {wu.p, wu.ld, false};
    cw.a[0] = {p.dg, ldd, false}, cw.a[1] = {p.du, ldd, false};
    cw.b[0] = cw.b[1] = {x.p, x.ld, false};
    if (a.dx) {
        const gs_status s = gemm_run(cx, px, base + at_x, &joins, st);
        if (s != GS_OK) return s;
    }
    if (a.dw_gate) {
        const gs_status s = gemm_run(cw, pw, base + at_w, &joins, st);
        if (s != GS_OK) return s;
    }
    return joins.run(st);
}
