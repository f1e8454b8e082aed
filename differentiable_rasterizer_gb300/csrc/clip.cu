// clip.cu -- the norm over many tensors, and the tensors scaled to a largest one.
//
//   norm = sqrt(sum v^2),  out = v min(1, max_norm / norm)
//
// The values are cut into pieces.  Two launches: the pieces' sums of squares, one partial sum
// a block; then every block adds the partial sums in order and scales its pieces, the last
// ones first, which the level-two cache still holds.  HBM bounds both: 144 tensors of
// 3.2e8 bf16 values to fp32 read them twice.  Up to kSmallPieces pieces (a decoder's weights)
// stay in the shared memory of a cluster's CTAs between their sum and their scaling: one
// launch, one read.  The tensors' table travels in the launch's parameters.
#include <algorithm>
#include <atomic>

#include "gemm.cuh"
#include "tc_common.cuh"

namespace gs {
namespace {

constexpr int kThreads = 256, kPiece = 8192, kBlocksPerSm = 4;
constexpr int kVectors = kPiece / (kThreads * 8);   // of a thread and piece
static_assert(kPiece % (kThreads * 8) == 0, "whole vectors of every thread");
constexpr int kFewTensors = 64;   // a table of few is quicker to launch with
constexpr int kCluster = 8, kSmallEach = 6, kSmallPieces = kCluster * kSmallEach, kSmallSmem = kSmallEach * kPiece * 4;

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

// Squares by size: values beyond 2^50 times 2^-64 and those below 2^-60 times 2^100 each in
// a sum of their own.  A vector goes by its largest value, beside which what the others
// lose is nothing.
struct Squares {
    float mid = 0.0f, big = 0.0f, small = 0.0f;
    __device__ __forceinline__ void add(const float (&v)[8])
    {
        float top = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
        if (top > 0x1p50f) {
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
};
// The sum over a thread's pieces: in fp32 with what each addition loses beside it (Knuth's
// two-sum).  In fp64, of which an SM adds two a cycle, it took as long as the loads.
// A piece's 32 squares of a thread pass twelve roundings at most (eight in a vector's sum, four
// vectors), and a vector goes wholly by its largest value: 12 2^-24 of the sum, half of it in the
// root; the two-sum's rest and the fp64 sums add next to nothing: the norm is within 2^-21.
struct Total {
    float high = 0.0f, low = 0.0f;
    double rest = 0.0;
    __device__ __forceinline__ void add(const Squares& s)
    {
        const float sum = high + s.mid, part = sum - high;
        low += (high - (sum - part)) + (s.mid - part);
        high = sum;
        if (s.big != 0.0f || s.small != 0.0f) rest += (double)s.big * 0x1p128 + (double)s.small * 0x1p-200;   // NaN too
    }
    __device__ __forceinline__ double value() const
    {
        return (high < INFINITY ? (double)high + (double)low : (double)high) + rest;   // an infinity's low is NaN
    }
};

// A thread's values of a piece: vectors threadIdx.x, threadIdx.x + kThreads, ... of eight; 0
// beyond its end.  Whole pieces on 16 bytes: all loads first, then use(vector, values).
template <int T, class Use>
__device__ __forceinline__ void whole_piece(const Piece& q, Use use)
{
    Raw<T, 8> raw[kVectors];
#pragma unroll
    for (int k = 0; k < kVectors; ++k) raw_load(raw[k], q.p, q.at + (threadIdx.x + k * kThreads) * 8, T);
#pragma unroll
    for (int k = 0; k < kVectors; ++k) {
        float v[8];
        raw_values(raw[k], T, v);
        use(threadIdx.x + k * kThreads, v);
    }
}
template <class Use>
__device__ __forceinline__ void for_values(const Piece& q, Use use)
{
    if (q.n == kPiece && vector_aligned(q.p)) {
        if (q.type == GS_F32) whole_piece<GS_F32>(q, use);
        else if (q.type == GS_BF16) whole_piece<GS_BF16>(q, use);
        else whole_piece<GS_F16>(q, use);
        return;
    }
    for (int i = threadIdx.x; i * 8 < q.n; i += kThreads) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = i * 8 + e < q.n ? load_elem(q.p, q.at + i * 8 + e, q.type) : 0.0f;
        use(i, v);
    }
}
__device__ __forceinline__ void store_scaled(const Piece& q, int i, const float (&v)[8], float factor)
{
    float s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = v[e] * factor;
    const int at = i * 8;
    if (at + 8 <= q.n && vector_aligned(q.out)) {
        if (q.out_type == GS_F32 && ((uintptr_t)q.out & 31u) == 0) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(s[e]);
            tc::st_global32((float*)q.out + q.at + at, w);
        } else store8(q.out, q.at + at, q.out_type, s);
    } else
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (at + e < q.n) store_elem(q.out, q.at + at + e, q.out_type, s[e]);
}
__device__ __forceinline__ float factor_of(float norm, float max_norm)
{
    return norm > max_norm && norm < INFINITY ? max_norm / norm : 1.0f;   // NaN: 1
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
    Total total;
    const uint32_t pieces = t.first[t.count];
    for (uint32_t i = blockIdx.x; i < pieces; i += t.blocks) {
        Squares s;
        for_values(piece_at(t, i), [&](int, const float (&v)[8]) { s.add(v); });
        total.add(s);
    }
    const double sum = block_sum(total.value(), sm);
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
    const float factor = factor_of(norm, t.max_norm);
    const uint32_t pieces = t.first[t.count];
    for (uint32_t i = blockIdx.x; i < pieces; i += t.blocks) {
        const Piece q = piece_at(t, pieces - 1 - i);
        if (factor == 1.0f && q.p == q.out) continue;
        for_values(q, [&](int k, const float (&v)[8]) { store_scaled(q, k, v, factor); });
    }
}

// A cluster takes all pieces, CTA r pieces r, r + 8, ...
template <int N>
__global__ void __launch_bounds__(kThreads) small_kernel(const __grid_constant__ Table<N> t)
{
    extern __shared__ __align__(16) float kept[];   // [kSmallEach][kPiece]
    __shared__ double sm[kThreads / 32];
    __shared__ __align__(8) double mine;
    wait_for_predecessor();
    const uint32_t pieces = t.first[t.count];
    Total total;
    for (uint32_t i = blockIdx.x, k = 0; i < pieces; i += kCluster, ++k) {
        Squares s;
        for_values(piece_at(t, i), [&](int at, const float (&v)[8]) {
            s.add(v);
            store8(kept + k * kPiece, at * 8, GS_F32, v);
        });
        total.add(s);
    }
    const double sum = block_sum(total.value(), sm);
    if (threadIdx.x == 0) mine = sum;
    tc::cluster_sync();
    double all = 0.0;
    for (uint32_t r = 0; r < kCluster; ++r) {
        const uint32_t at = tc::map_rank(tc::smem_addr(&mine), r);
        all += __hiloint2double(__float_as_int(tc::ld_cluster_f32(at + 4)), __float_as_int(tc::ld_cluster_f32(at)));
    }
    tc::cluster_sync();   // a CTA's sum is read until here
    const float norm = (float)sqrt(all), factor = factor_of(norm, t.max_norm);
    if (blockIdx.x == 0 && threadIdx.x == 0) *t.norm = norm;
    for (uint32_t i = blockIdx.x, k = 0; i < pieces; i += kCluster, ++k) {
        const Piece q = piece_at(t, i);
        if (factor == 1.0f && q.p == q.out) continue;
        for (int at = threadIdx.x; at * 8 < q.n; at += kThreads) {   // its own values
            float v[8];
            load8(kept + k * kPiece, at * 8, GS_F32, v);
            store_scaled(q, at, v, factor);
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
    if constexpr (N == kFewTensors) if (pieces <= kSmallPieces) {
        static std::atomic<uint64_t> done{0};
        const gs_status s = allow_smem(small_kernel<N>, kSmallSmem, done);
        const size_t each = (pieces + kCluster - 1) / kCluster;
        return s != GS_OK ? s : launch_after(small_kernel<N>, dim3(kCluster), kThreads, each * kPiece * 4, kCluster, st, t);
    }
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
    int64_t pieces = 0, filled = 0;
    for (int64_t i = 0; i < a.count; ++i) {
        const gs_clip_tensor& q = a.tensors[i];
        if (!type_float(q.type) || !type_float(q.out_type) || q.size < 0 || q.size > 1ll << 44) return GS_ERR_INVALID_ARG;
        if (q.size == 0) continue;
        if (!q.p || !q.out || !vec_ok(q.p, q.type) || !vec_ok(q.out, q.out_type)) return GS_ERR_INVALID_ARG;
        if (q.p == q.out && q.type != q.out_type) return GS_ERR_INVALID_ARG;
        pieces += (q.size + kPiece - 1) / kPiece;
        ++filled;
    }
    if (pieces > 0x7fffffffll || overlap(a)) return GS_ERR_INVALID_ARG;
    const int sms = device_sms();
    const uint32_t blocks = (uint32_t)((sms > 0 ? sms : 152) * kBlocksPerSm);
    const WsCheck wc = ws_check(ws, ws_bytes, (size_t)round_up((int64_t)blocks * 8, 256));
    if (wc == WsCheck::kBad) return GS_ERR_INVALID_ARG;
    if (wc == WsCheck::kQuery) return GS_OK;
    if (!a.norm || !vec_ok(a.norm, GS_F32)) return GS_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    return filled <= kFewTensors ? run<kFewTensors>(a, (double*)ws, blocks, st) : run<GS_CLIP_MAX_TENSORS>(a, (double*)ws, blocks, st);
}
