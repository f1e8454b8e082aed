// clip.cu -- the norm over many tensors, and the tensors scaled to a largest one.
//
//   norm = sqrt(sum v^2),  out = v min(1, max_norm / norm)
//
// Two launches over pieces of kPiece values: the pieces' sums of squares, one partial sum a
// block; then every block adds the partial sums in order and scales its pieces, the last
// ones first, which the level-two cache still holds.  HBM bounds both.  The tensors' table
// travels in the launch's parameters.
#include <algorithm>

#include "gemm.cuh"

namespace gs {
namespace {

constexpr int kThreads = 256, kPiece = 8192, kBlocksPerSm = 4;
static_assert(kPiece % (kThreads * 8) == 0, "whole vectors of every thread");

template <int N>
struct Table {
    const void* p[N];
    void* out[N];
    uint64_t size[N];       // values, the types in the top byte
    uint32_t first[N + 1];  // piece
    uint32_t count;
    float* norm;
    double* partial;        // a block
    uint32_t blocks;
    float max_norm;
};

struct Piece {
    const void* p;
    void* out;
    int64_t at;
    int n, type, out_type;   // n: values, at most kPiece
};
template <int N>
__device__ __forceinline__ Piece piece_at(const Table<N>& t, uint32_t i)
{
    uint32_t lo = 0, hi = t.count;   // the last tensor whose first piece is not behind i
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) >> 1;
        if (t.first[mid] <= i) lo = mid;
        else hi = mid;
    }
    Piece r;
    r.p = t.p[lo], r.out = t.out[lo];
    const uint64_t s = t.size[lo];
    r.type = (int)(s >> 56) & 15, r.out_type = (int)(s >> 60);
    r.at = (int64_t)(i - t.first[lo]) * kPiece;
    const int64_t left = (int64_t)(s & 0xffffffffffffffull) - r.at;
    r.n = left < kPiece ? (int)left : kPiece;
    return r;
}
__device__ __forceinline__ bool vector_aligned(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// Squares by size: values beyond 2^60 times 2^-64 and those below 2^-60 times 2^100 each in
// a sum of their own.  A vector goes by its largest value, beside which what the others
// lose is nothing.
struct Squares {
    float mid = 0.0f, big = 0.0f, small = 0.0f;
    __device__ __forceinline__ void add(const float (&v)[8])
    {
        float top = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
        if (top > 0x1p60f) {
#pragma unroll
            for (int e = 0; e < 8; ++e) big = __fmaf_rn(v[e] * 0x1p-64f, v[e] * 0x1p-64f, big);
        } else if (top < 0x1p-60f && top > 0.0f) {
#pragma unroll
            for (int e = 0; e < 8; ++e) small = __fmaf_rn(v[e] * 0x1p100f, v[e] * 0x1p100f, small);
        } else {
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s = __fmaf_rn(v[e], v[e], s);
            mid += s;
        }
    }
    __device__ __forceinline__ double total() const { return (double)mid + (double)big * 0x1p128 + (double)small * 0x1p-200; }
};

// Eight values of a piece from i on; 0 beyond its end.
__device__ __forceinline__ void load_piece(const Piece& q, int i, bool vec, float (&v)[8])
{
    if (vec && i + 8 <= q.n) {
        load8(q.p, q.at + i, q.type, v);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = i + e < q.n ? load_elem(q.p, q.at + i + e, q.type) : 0.0f;
}

// The block's sum, in a fixed order; all threads get it.
__device__ __forceinline__ double block_sum(double v, double* sm)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    double r = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) r += sm[w];
    return r;
}

template <int N>
__global__ void __launch_bounds__(kThreads) squares_kernel(const __grid_constant__ Table<N> t)
{
    __shared__ double sm[kThreads / 32];
    wait_for_predecessor();
    double sum = 0.0;
    for (uint32_t i = blockIdx.x; i < t.first[t.count]; i += t.blocks) {
        const Piece q = piece_at(t, i);
        const bool vec = vector_aligned(q.p);
        Squares s;
#pragma unroll 4
        for (int e = threadIdx.x * 8; e < q.n; e += kThreads * 8) {
            float v[8];
            load_piece(q, e, vec, v);
            s.add(v);
        }
        sum += s.total();
    }
    sum = block_sum(sum, sm);
    if (threadIdx.x == 0) t.partial[blockIdx.x] = sum;
}

template <int N>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ Table<N> t)
{
    __shared__ double sm[kThreads / 32];
    wait_for_predecessor();
    double sum = 0.0;
    for (uint32_t i = threadIdx.x; i < t.blocks; i += kThreads) sum += t.partial[i];
    const float norm = (float)sqrt(block_sum(sum, sm));
    if (blockIdx.x == 0 && threadIdx.x == 0) *t.norm = norm;
    const float factor = norm > t.max_norm && norm < INFINITY ? t.max_norm / norm : 1.0f;   // NaN: 1
    const uint32_t pieces = t.first[t.count];
    for (uint32_t i = blockIdx.x; i < pieces; i += t.blocks) {
        const Piece q = piece_at(t, pieces - 1 - i);
        if (factor == 1.0f && q.p == q.out) continue;
        const bool vec = vector_aligned(q.p), out_vec = vector_aligned(q.out);
#pragma unroll 4
        for (int e = threadIdx.x * 8; e < q.n; e += kThreads * 8) {
            float v[8];
            load_piece(q, e, vec, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] *= factor;
            if (out_vec && e + 8 <= q.n) store8(q.out, q.at + e, q.out_type, v);
            else
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (e + k < q.n) store_elem(q.out, q.at + e + k, q.out_type, v[k]);
        }
    }
}

template <int N>
gs_status run(const gs_clip_norm_args& a, double* partial, uint32_t blocks, cudaStream_t st)
{
    Table<N> t;
    uint32_t pieces = 0;
    t.count = 0;
    for (int64_t i = 0; i < a.count; ++i) {
        const gs_clip_tensor& q = a.tensors[i];
        if (q.size == 0) continue;
        t.p[t.count] = q.p, t.out[t.count] = q.out;
        t.size[t.count] = (uint64_t)q.size | (uint64_t)q.type << 56 | (uint64_t)q.out_type << 60;
        t.first[t.count++] = pieces;
        pieces += (uint32_t)((q.size + kPiece - 1) / kPiece);
    }
    t.first[t.count] = pieces;
    t.norm = a.norm, t.max_norm = a.max_norm, t.partial = partial;
    t.blocks = pieces < blocks ? (pieces ? pieces : 1) : blocks;
    const gs_status s = launch_after(squares_kernel<N>, dim3(t.blocks), kThreads, 0, 1, st, t);
    return s != GS_OK ? s : launch_after(scale_kernel<N>, dim3(t.blocks), kThreads, 0, 1, st, t);
}

// Whether two of the tensors' inputs or outputs share memory, but for a tensor's own two.
bool overlap(const gs_clip_norm_args& a)
{
    struct Span {
        uintptr_t from, to;
    };
    Span spans[2 * GS_CLIP_MAX_TENSORS];
    int64_t n = 0;
    for (int64_t i = 0; i < a.count; ++i) {
        const gs_clip_tensor& q = a.tensors[i];
        if (q.size == 0) continue;
        spans[n++] = {(uintptr_t)q.p, (uintptr_t)q.p + (uintptr_t)q.size * type_bytes(q.type)};
        if (q.out != q.p) spans[n++] = {(uintptr_t)q.out, (uintptr_t)q.out + (uintptr_t)q.size * type_bytes(q.out_type)};
    }
    std::sort(spans, spans + n, [](const Span& x, const Span& y) { return x.from < y.from; });
    for (int64_t i = 1; i < n; ++i)
        if (spans[i].from < spans[i - 1].to) return true;
    return false;
}

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" gs_status gs_clip_norm(const gs_clip_norm_args* args, void* ws, size_t* ws_bytes, void* stream)
{
    GS_NVTX_RANGE("gs_clip_norm");
    if (!args) return GS_ERR_INVALID_ARG;
    const gs_clip_norm_args& a = *args;
    if (a.count < 0 || a.count > GS_CLIP_MAX_TENSORS || (a.count > 0 && !a.tensors) || !(a.max_norm >= 0.0f)) return GS_ERR_INVALID_ARG;
    int64_t pieces = 0;
    for (int64_t i = 0; i < a.count; ++i) {
        const gs_clip_tensor& q = a.tensors[i];
        if (!type_float(q.type) || !type_float(q.out_type) || q.size < 0 || q.size > 1ll << 44) return GS_ERR_INVALID_ARG;
        if (q.size == 0) continue;
        if (!q.p || !q.out || !vec_ok(q.p, q.type) || !vec_ok(q.out, q.out_type)) return GS_ERR_INVALID_ARG;
        if (q.p == q.out && q.type != q.out_type) return GS_ERR_INVALID_ARG;
        pieces += (q.size + kPiece - 1) / kPiece;
    }
    if (pieces > 0x7fffffffll || overlap(a)) return GS_ERR_INVALID_ARG;
    const int sms = device_sms();
    const uint32_t blocks = (uint32_t)((sms > 0 ? sms : 152) * kBlocksPerSm);
    const WsCheck wc = ws_check(ws, ws_bytes, (size_t)round_up((int64_t)blocks * 8, 256));
    if (wc == WsCheck::kBad) return GS_ERR_INVALID_ARG;
    if (wc == WsCheck::kQuery) return GS_OK;
    if (!a.norm || !vec_ok(a.norm, GS_F32)) return GS_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    return a.count <= 64 ? run<64>(a, (double*)ws, blocks, st) : run<GS_CLIP_MAX_TENSORS>(a, (double*)ws, blocks, st);
}
