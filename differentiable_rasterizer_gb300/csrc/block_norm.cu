// block_norm.cu -- the norm after a block, its gate and residual scale, and the norm
// before the next block, with their gradients.
//
//   a = h rms(h)^-1 post,  s = scale x + gate a,  y = s rms(s)^-1 weight
//
// One pass over the rows: a group of threads holds a row in registers from h and x to s
// and y (backward: from dy, ds, s and h to dx and dh), with two reductions in between.
// HBM bounds both.  The group is the least number of threads that covers the row at eight
// columns a thread: a power of two within a warp (narrow rows share one and rows of up to 256
// columns need no barrier), whole warps beyond it.  As separate norm, product, sum and norm a row would
// cross HBM nine times in place of four.
//   1,000,000 x 256 bf16 334 us, 6.1 TB/s (302 at the copy's rate; without the next row's loads
//   ahead 449, with weights fetched for each row 500), its gradients 520 us, 5.9 TB/s
//   20,011 x 331 f16, a gate a value: 33 and 59 us, 250,000 x 197 172 and 300 (floors 72 and
//   116).  Their instructions bound them: issue slots are 71 and 64 % busy with 7 and 6 warps a
//   scheduler; of a warp's nine and eight cycles an instruction some two are the instructions' own
//   latency, one and a half that another warp is chosen, one and a quarter loads, less than one the
//   row's barriers (single elements 20,011 x 331 138 and 364 us; the next row's pieces ahead in
//   shared memory, or whole pieces written with the neighbour's columns, no faster)
//   8,000 x 5928 bf16 132 and 203 us (floors 56 and 84): one row an SM at a time, whose two
//   reductions nothing covers
#include <type_traits>

#include "gemm.cuh"
#include "rows.cuh"

namespace gs {
namespace {

using namespace rows;

// A matrix's rows as a thread reads them, eight columns at a time.  Rows of 16-byte base and
// pitch: whole pieces, of which a row's last may lie in its padding (see piece_rows).  Others of 16-bit
// elements: the four or five 32-bit words that the eight columns lie in, shifted by an element
// where the row starts within a word (two pieces of 16 bytes shifted together took 15
// instructions more a matrix: 250,000 x 197 268 and 410 us against 230 and 367); single
// elements in the first and the last row, whose words may reach beyond the matrix, and in fp32.
struct Source {
    const void* p;
    int64_t ld;
    int type;
    bool aligned;
    __device__ __forceinline__ Source(const void* p_, int64_t ld_, int type_)
        : p(p_), ld(ld_), type(type_), aligned(piece_rows(p_, ld_, type_)) {}
    // Words that hold columns of this row lie in the matrix.
    __device__ __forceinline__ bool inside(int64_t row, int64_t rows) const { return row > 0 && row + 1 < rows; }
    // Whether a row of 16-bit elements, and with it every eighth column, starts within a word.
    __device__ __forceinline__ uint32_t odd(int64_t row) const { return ((uint32_t)((uintptr_t)p >> 1) + ((uint32_t)row & (uint32_t)ld)) & 1u; }
};

// WHOLE: every matrix's rows are whole pieces.
template <int T, bool WHOLE>
constexpr bool kShifts = !WHOLE && (T == GS_BF16 || T == GS_F16);
template <int T, bool WHOLE>
struct Cells {
    Raw<T, 8> raw;
    uint32_t last;   // a fifth word
    __device__ __forceinline__ void zero()
    {
        raw_zero(raw);
        last = 0;
    }
};
// Elements from one to the other, of the eight at p.
__device__ __forceinline__ uint32_t element_bits(const void* p, int64_t i, int type)
{
    return type == GS_F32 ? ((const uint32_t*)p)[i] : ((const uint16_t*)p)[i];
}

template <int T, bool WHOLE>
__device__ __forceinline__ void fetch(Cells<T, WHOLE>& to, const Source& m, int64_t row, int64_t rows, int col, int cols)
{
    const int n = cols - col, type = T == kAnyType ? m.type : T;
    const int64_t at = row * m.ld + col;
    if constexpr (WHOLE) {
        raw_load(to.raw, m.p, at, type);
        return;
    }
    const bool inside = m.inside(row, rows);
    if (m.aligned && (inside || (cols & 7) == 0)) {
        raw_load(to.raw, m.p, at, type);
    } else if (kShifts<T, WHOLE> && inside) {
        const int odd = (int)m.odd(row), end = odd + (n < 8 ? n : 8);
        const uint32_t* word = reinterpret_cast<const uint32_t*>((const uint16_t*)m.p + (at - odd));
        uint32_t w[5];
#pragma unroll
        for (int e = 0; e < 5; ++e) w[e] = 2 * e < end ? word[e] : 0;
        to.raw.q[0] = make_uint4(w[0], w[1], w[2], w[3]);
        to.last = w[4];
    } else {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = e < n ? element_bits(m.p, at + e, type) : 0;
        if (type == GS_F32) {
            to.raw.q[0] = make_uint4(w[0], w[1], w[2], w[3]);
            if constexpr (T == GS_F32 || T == kAnyType) to.raw.q[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else
            to.raw.q[0] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
    }
}

// The values, in pairs; 0 beyond the row.
template <int T, bool WHOLE>
__device__ __forceinline__ void values(const Cells<T, WHOLE>& c, const Source& m, int64_t row, int64_t rows, int col, int cols, uint64_t (&v)[4])
{
    const int n = cols - col, type = T == kAnyType ? m.type : T;
    Raw<T, 8> raw = c.raw;
    if constexpr (kShifts<T, WHOLE>) {
        const uint32_t by = m.inside(row, rows) ? m.odd(row) * 16 : 0;
        const uint4 w = raw.q[0];
        raw.q[0] = make_uint4(__funnelshift_r(w.x, w.y, by), __funnelshift_r(w.y, w.z, by), __funnelshift_r(w.z, w.w, by), __funnelshift_r(w.w, c.last, by));
    }
    float f[8];
    raw_values(raw, type, f);
    if (!WHOLE && n < 8) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e >= n) f[e] = 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = pair(f[2 * e], f[2 * e + 1]);
}

// Eight columns to a row, whole where the row's place (aligned) and its end allow it; 16-bit
// ones of other rows in words.
__device__ __forceinline__ void store(void* p, int64_t at, int n, int type, bool aligned, const uint64_t (&v)[4])
{
    float f[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 t = unpair(v[e]);
        f[2 * e] = t.x, f[2 * e + 1] = t.y;
    }
    if (aligned && n >= 8) store8(p, at, type, f);
    else if (type == GS_BF16 || type == GS_F16) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = pack_half2(f[2 * e], f[2 * e + 1], type);
        uint16_t* to = (uint16_t*)p + at;
        if (n < 8) {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < n) to[e] = (uint16_t)(w[e >> 1] >> (e & 1) * 16);
        } else if (((uintptr_t)to & 3u) == 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) reinterpret_cast<uint32_t*>(to)[e] = w[e];
        } else {
            to[0] = (uint16_t)w[0];
#pragma unroll
            for (int e = 0; e < 3; ++e) reinterpret_cast<uint32_t*>(to + 1)[e] = __funnelshift_r(w[e], w[e + 1], 16);
            to[7] = (uint16_t)(w[3] >> 16);
        }
    } else
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) store_elem(p, at + e, type, f[e]);
}
__device__ __forceinline__ bool rows_aligned(const void* p, int64_t ld, int type)
{
    const int e = type_bytes(type), piece = type == GS_E4M3 ? 8 : 16;
    return ((uintptr_t)p & (uintptr_t)(piece - 1)) == 0 && ld * e % piece == 0;
}

// The thread's columns of a vector over them; 1 where there is none, 0 beyond the row.
__device__ __forceinline__ void load_weight(const void* p, int col, int n, int type, uint64_t (&v)[4])
{
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = e < n ? 1.0f : 0.0f;
    if (p && n >= 8 && ((uintptr_t)p & 15u) == 0) load8(p, col, type, f);
    else if (p)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) f[e] = load_elem(p, col + e, type);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = pair(f[2 * e], f[2 * e + 1]);
}

// The product of one or two vectors over the columns.  Of up to 16 columns a thread they stay
// in registers, of more they are fetched from the first-level cache for every row.
template <int NV>
struct Weight {
    static constexpr bool kKeep = NV <= 2;
    uint64_t v[kKeep ? NV : 1][4];
    const void *p, *q;
    int p_type, q_type, lane, group, cols;
    __device__ __forceinline__ Weight(const void* p_, int p_type_, const void* q_, int q_type_, int lane_, int group_, int cols_)
        : p(p_), q(q_), p_type(p_type_), q_type(q_type_), lane(lane_), group(group_), cols(cols_)
    {
        if constexpr (kKeep)
#pragma unroll
            for (int j = 0; j < NV; ++j) product(j, v[j]);
    }
    __device__ __forceinline__ int col(int j) const { return (lane + j * group) * 8; }
    __device__ __forceinline__ void product(int j, uint64_t (&w)[4]) const
    {
        load_weight(p, col(j), cols - col(j), p_type, w);
        if (q) {
            uint64_t t[4];
            load_weight(q, col(j), cols - col(j), q_type, t);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = mul2(w[e], t[e]);
        }
    }
    __device__ __forceinline__ void get(int j, uint64_t (&w)[4]) const
    {
        if constexpr (kKeep)
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = v[j][e];
        else product(j, w);
    }
};

__device__ __forceinline__ uint64_t both(float v) { return pair(v, v); }
__device__ __forceinline__ float sum_of(uint64_t v)
{
    const float2 f = unpair(v);
    return f.x + f.y;
}

// Threads of a block at most, and blocks an SM, which set the registers: one vector a thread
// wants many warps of few.  Of unaligned rows 64 without the next row's loads ahead: 250,000 x 197
// 172 us; 80 with them 184, 97 with them 230; gradients with 80 300 us, with 117 309.
template <int T, int NV, bool WHOLE>
constexpr int kForwardThreads = NV == 1 && !(T == GS_F32 && WHOLE) ? 1024 : 512;
template <int NV>
constexpr int kBackwardThreads = NV == 1 ? 256 : 512;
template <int T, int NV, bool WHOLE>
constexpr int kBackwardBlocks = NV == 1 ? (T != GS_F32 ? 3 : 2) : 1;

template <int T, int NV, bool WHOLE>
__global__ void __launch_bounds__(kForwardThreads<T, NV, WHOLE>) block_norm_kernel(const __grid_constant__ gs_block_norm_args a, int group)
{
    constexpr int P = 4;
    constexpr bool kAhead = NV == 1 && WHOLE;   // the next row's loads before this one's work
    __shared__ float sm[32];
    wait_for_predecessor();
    const int lane = threadIdx.x % group, cols = (int)a.cols;
    const int64_t step = (int64_t)gridDim.x * (blockDim.x / group);
    const float inv_cols = 1.0f / (float)a.cols;
    const bool q8 = a.y_type == GS_E4M3 && a.y;
    const Weight<NV> weight(a.weight, a.weight_type, nullptr, 0, lane, group, cols);
    const Weight<NV> post(a.post_weight, a.post_type, a.gate_rows ? nullptr : a.gate, a.gate_type, lane, group, cols);
    const uint64_t scale = both(a.scale);
    const Source sh(a.h, a.ldh, T), sx(a.x, a.ldx, T), sg(a.gate, a.ldg, T);
    const bool s_aligned = rows_aligned(a.s, a.lds, T), y_aligned = rows_aligned(a.y, a.ldy, a.y_type);
    Cells<T, WHOLE> hr[NV], xr[NV], gr[NV];
    const auto load = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = weight.col(j), n = cols - c;
            hr[j].zero(), xr[j].zero();
            if (row < a.rows && n > 0) {
                fetch(hr[j], sh, row, a.rows, c, cols);
                fetch(xr[j], sx, row, a.rows, c, cols);
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
                if (here && n > 0) fetch(gr[j], sg, row, a.rows, c, cols);
            }
        uint64_t s[NV][P], x[NV][P], q = both(0.0f);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            values(hr[j], sh, row, a.rows, weight.col(j), cols, s[j]);
            values(xr[j], sx, row, a.rows, weight.col(j), cols, x[j]);
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
                values(gr[j], sg, row, a.rows, c, cols, g);
#pragma unroll
                for (int e = 0; e < P; ++e) s[j][e] = mul2(s[j][e], g[e]);
            }
#pragma unroll
            for (int e = 0; e < P; ++e) {
                s[j][e] = fma2(scale, x[j][e], s[j][e]);
                q = fma2(s[j][e], s[j][e], q);
            }
            if (here && n > 0) store(a.s, row * a.lds + c, n, T, s_aligned, s[j]);
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
            if (here && n > 0) store(a.y, row * a.ldy + c, n, a.y_type, y_aligned, s[j]);
        }
    }
}

// Sums over rows: every thread keeps its columns' over the rows it visits, a block joins
// its groups' in order into partial rows, and JoinJobs adds the blocks' in order.
//   A = sum of g h rstd_post gives two of them where the gate is a vector: dgate = post A,
//   dpost = gate A; where it is rows, dpost sums g h rstd_post gate.
// partial: [3][blocks][cols]: dweight, dpost, dgate.
template <int T, int TDY, int NV, bool WHOLE>
__global__ void __launch_bounds__(kBackwardThreads<NV>, kBackwardBlocks<T, NV, WHOLE>) block_norm_bwd_kernel(const __grid_constant__ gs_block_norm_bwd_args a,
                                                                                               int group, float* partial)
{
    constexpr int P = 4;
    extern __shared__ float part[];   // [groups][columns rounded up] when a block holds several groups
    __shared__ float sm[32];
    wait_for_predecessor();
    const int lane = threadIdx.x % group, groups = blockDim.x / group, cols = (int)a.cols;
    const float inv_cols = 1.0f / (float)a.cols;
    const bool post = a.post_weight != nullptr;
    const void* gate = a.gate_rows ? nullptr : a.gate;
    const Weight<NV> weight(a.weight, a.weight_type, nullptr, 0, lane, group, cols);
    const Weight<NV> post_weight(a.post_weight, a.post_type, gate, a.gate_type, lane, group, cols);
    const uint64_t scale = both(a.scale);
    const Source sy(a.dy, a.lddy, a.dy_type), ss(a.s, a.lds, T), sd(a.ds, a.ldds, T), sh(a.h, a.ldh, T), sg(a.gate, a.ldg, T);
    const bool dx_aligned = rows_aligned(a.dx, a.lddx, T), dh_aligned = rows_aligned(a.dh, a.lddh, T), dg_aligned = rows_aligned(a.dgate, a.lddg, T);
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
        Cells<T, WHOLE> hr[NV], sr[NV], dr[NV], gr[NV];
        Cells<TDY, WHOLE> yr[NV];
        const float rstd = a.dy && here ? a.rstd[row] : 0.0f, rstd_post = post && here ? a.rstd_post[row] : 1.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = weight.col(j), n = cols - c;
            hr[j].zero(), sr[j].zero(), dr[j].zero(), gr[j].zero(), yr[j].zero();
            if (here && n > 0) {
                if (a.dy) {
                    fetch(yr[j], sy, row, a.rows, c, cols);
                    fetch(sr[j], ss, row, a.rows, c, cols);
                }
                if (a.ds) fetch(dr[j], sd, row, a.rows, c, cols);
                if (post || a.dgate) fetch(hr[j], sh, row, a.rows, c, cols);
                if (a.gate_rows) fetch(gr[j], sg, row, a.rows, c, cols);
            }
        }
        uint64_t g[NV][P], q = both(0.0f);   // g: dy * weight, the gradient of s, that of h / rms(h)
        float c2 = 0.0f;
        if (a.dy) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                uint64_t s[P], dy[P], w[P];
                weight.get(j, w);
                values(sr[j], ss, row, a.rows, weight.col(j), cols, s);
                values(yr[j], sy, row, a.rows, weight.col(j), cols, dy);
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
            values(hr[j], sh, row, a.rows, c, cols, h);
            values(dr[j], sd, row, a.rows, c, cols, v);
            if (a.dy) {
                uint64_t s[P];
                values(sr[j], ss, row, a.rows, c, cols, s);
#pragma unroll
                for (int e = 0; e < P; ++e) g[j][e] = fma2(both(rstd), fma2(s[e], both(c2), g[j][e]), v[e]);
            } else
#pragma unroll
                for (int e = 0; e < P; ++e) g[j][e] = v[e];
            if (a.dx && there) {
#pragma unroll
                for (int e = 0; e < P; ++e) v[e] = mul2(scale, g[j][e]);
                store(a.dx, row * a.lddx + c, n, T, dx_aligned, v);
            }
            if (a.gate_rows) {
                uint64_t gates[P];
                values(gr[j], sg, row, a.rows, c, cols, gates);
                if (a.dgate && there) {
#pragma unroll
                    for (int e = 0; e < P; ++e) v[e] = mul2(g[j][e], mul2(mul2(h[e], both(rstd_post)), w[e]));
                    store(a.dgate, row * a.lddg + c, n, T, dg_aligned, v);
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
                values(hr[j], sh, row, a.rows, c, cols, h);
#pragma unroll
                for (int e = 0; e < P; ++e) g[j][e] = mul2(both(rstd_post), fma2(h[e], both(c2), g[j][e]));
            }
            if (here && n > 0) store(a.dh, row * a.lddh + c, n, T, dh_aligned, g[j]);
        }
    }
    const auto write = [&](int which, const uint64_t (&v)[NV][P], const void* by, int by_type) {
        float* out = partial + ((int64_t)which * gridDim.x + blockIdx.x) * a.cols;
        const int width = NV * group * 8;
        float* mine = groups == 1 ? out : part + (threadIdx.x / group) * width;
        __syncthreads();   // the sums before have been read
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = weight.col(j);
            uint64_t w[P];
            load_weight(by, c, cols - c, by_type, w);
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
// One vector a thread up to `widest` threads, then two or four; in_warp: two for rows that a
// warp holds so (forward of fp32 pieces: 20,000 x 512 39 -> 35 us).  Up to a warp a power of two of
// threads, beyond it whole warps (of 2049 columns, 257 vectors, 288 threads in place
// of 512: 16,000 rows 183 -> 111 us).
Shape shape_for(int64_t cols, int widest, bool in_warp)
{
    const int64_t n = (cols + 7) / 8;
    Shape s;
    s.nv = n <= widest && !(in_warp && n > 32 && n <= 64) ? 1 : (n <= 1024 ? 2 : 4);
    const int lanes = (int)((n + s.nv - 1) / s.nv);
    s.group = 1;
    while (s.group < 32 && s.group < lanes) s.group *= 2;
    if (lanes > 32) s.group = (lanes + 31) / 32 * 32;
    s.threads = s.group < 256 ? 256 / s.group * s.group : s.group;
    return s;
}
// Blocks of the grid: those that the SMs hold at a time, whose threads take `threads` in all of
// one SM (what is beyond would wait for a second turn: 20,011 x 331 gradients 73 -> 60 us).
int64_t grid_for(int64_t sms, const Shape& s, int threads) { return sms * (s.threads < threads ? threads / s.threads : 1); }

bool norm_sizes_ok(int64_t rows, int64_t cols, int type) { return size_ok(rows, 0) && size_ok(cols, 1) && cols <= GS_NORM_MAX_COLS && type_float(type); }

bool weight_ok(const void* p, int type) { return !p || (type_float(type) && vec_ok(p, type)); }

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
    const bool whole = a.cols % 8 == 0 && a.cols <= 8192 && rows16(a.h, a.ldh, a.type) && rows16(a.x, a.ldx, a.type) &&
                       (!a.gate_rows || rows16(a.gate, a.ldg, a.type));
    // one vector a thread up to 1024 threads where pieces are whole (8,000 x 5928 147 -> 132 us), else
    // up to 512 (unaligned 5925 columns 163 us, with 1024 175)
    const Shape s = shape_for(a.cols, whole && a.type != GS_F32 ? 1024 : 512, a.type == GS_F32 && whole);
    const int64_t rpb = s.threads / s.group, want = (a.rows + rpb - 1) / rpb, most = grid_for(sms, s, s.nv == 1 && !(a.type == GS_F32 && whole) ? 1024 : 512);
    const int grid = (int)(want < most ? want : most);
    cudaStream_t st = (cudaStream_t)stream;
    const auto run = [&](auto t) -> gs_status {
        constexpr int T = decltype(t)::value;
#define GS_FWD(N, W) return launch_after(block_norm_kernel<T, N, W>, dim3(grid), s.threads, 0, 1, st, a, s.group)
        if constexpr (T == GS_F32)
            if (whole && s.nv == 2) GS_FWD(2, true);
        if (whole) GS_FWD(1, true);   // 16-bit: 1024 threads hold the widest of whole pieces
        if (s.nv == 1) GS_FWD(1, false);
        else if (s.nv == 2) GS_FWD(2, false);
        else GS_FWD(4, false);
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
    const Shape s = shape_for(a.cols, 256, false);
    const int64_t blocks = grid_for(sms > 0 ? sms : 152, s, s.nv == 1 && a.type != GS_F32 ? 768 : 512);   // whatever the arrays' alignment
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
    const auto wide = [&](const void* p, int64_t ld, bool used) { return !used || rows16(p, ld, a.type); };
    const bool same = !a.dy || a.dy_type == a.type;
    const bool whole = same && a.cols % 8 == 0 && a.cols <= 8192 && wide(a.dy, a.lddy, a.dy) && wide(a.s, a.lds, a.dy) &&
                       wide(a.ds, a.ldds, a.ds) && wide(a.h, a.ldh, reads_h) && wide(a.gate, a.ldg, row_gate);
    const int groups = s.threads / s.group;
    const int64_t want = (a.rows + groups - 1) / groups;
    const int grid = (int)(want < blocks ? want : blocks);
    const size_t smem = groups > 1 && need ? (size_t)groups * s.nv * s.group * 32 : 0;   // at most 16 KB
    float* part = (float*)ws;
    const auto run = [&](auto t, auto tdy) -> gs_status {
        constexpr int T = decltype(t)::value, TDY = decltype(tdy)::value;
#define GS_BWD(N, W) return launch_after(block_norm_bwd_kernel<T, TDY, N, W>, dim3(grid), s.threads, smem, 1, st, a, s.group, part)
        if constexpr (T == TDY)
            if (whole) {
                if (s.nv == 1) GS_BWD(1, true);
                else GS_BWD(2, true);
            }
        if (s.nv == 1) GS_BWD(1, false);
        else if (s.nv == 2) GS_BWD(2, false);
        else GS_BWD(4, false);
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
