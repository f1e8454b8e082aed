// attention.cuh -- what the attention kernels (attention.cu, attention_bwd.cu) share:
// sequences and the tiles of their packed rows, tensor maps, and the tcgen05 forms that
// take a factor from TMEM.
//
// A tile has up to 128 packed rows: tokens of one sequence times the query heads of one
// key head, (token, head) with the head fast.  The heads of a group share a tile's keys
// that way, whatever their number, and the gradients of keys and values sum over them in
// the contraction.  A group that does not divide 128 leaves the tile's last rows unused.
#pragma once

#include "gemm.cuh"
#include "tc_common.cuh"

namespace gs {
namespace attn {

using namespace tc;

constexpr int kRows = 128;                 // of a tile, packed rows or keys
constexpr uint32_t kBox = kRows * 128;     // bytes of a tile's 64 columns
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// ------------------------------------------------------------------ sequences
struct Sequences {
    const int32_t* q_starts;   // NULL: one sequence of all rows
    const int32_t* k_starts;
    const int32_t* k_lengths;
    int64_t q_rows, k_rows;
    uint32_t count;
};
struct Sequence {
    int q0, lq, k0, lk;   // first rows and lengths
    uint32_t number;
};

// Starts and lengths as they are held within the arrays.
__host__ __device__ __forceinline__ int held(int64_t v, int64_t lo, int64_t hi) { return (int)(v < lo ? lo : (v > hi ? hi : v)); }

__device__ __forceinline__ Sequence sequence_at(const Sequences& p, uint32_t s)
{
    Sequence r;
    r.number = s;
    if (!p.q_starts) {
        r.q0 = r.k0 = 0;
        r.lq = (int)p.q_rows;
        r.lk = (int)p.k_rows;
    } else {
        r.q0 = held(p.q_starts[s], 0, p.q_rows);
        r.lq = held(p.q_starts[s + 1], r.q0, p.q_rows) - r.q0;
        r.k0 = held(p.k_starts[s], 0, p.k_rows);
        r.lk = held(p.k_starts[s + 1], r.k0, p.k_rows) - r.k0;
    }
    if (p.k_lengths) r.lk = held(p.k_lengths[s], 0, r.lk);
    return r;
}

// Unit u of those that every sequence's rows (KEYS: keys) are cut into, `tokens` each:
// its sequence and the unit's number within it, of `units`.  Called by whole warps; false
// beyond the last unit.  32 starts a round, from the first on, in every warp: nothing beside a
// tile for some hundred sequences, what a call costs for many thousands (391 sequences of 256
// rows, 4 heads of 16: forward 119 us; 3,907: 6.4 ms; 15,625 of 64: 55 ms).
template <bool KEYS>
__device__ __forceinline__ bool find_unit(const Sequences& p, uint32_t u, int tokens, Sequence& seq, uint32_t& unit, uint32_t& units)
{
    const uint32_t lane = threadIdx.x & 31;
    for (uint32_t base = 0; base < p.count; base += 32) {
        const uint32_t s = base + lane;
        Sequence mine = {0, 0, 0, 0, 0};
        if (s < p.count) mine = sequence_at(p, s);
        const int length = KEYS ? mine.lk : mine.lq;
        const uint32_t n = ((uint32_t)length + (uint32_t)tokens - 1) / (uint32_t)tokens;
        uint32_t end = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t below = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= (uint32_t)o) end += below;
        }
        const uint32_t after = __ballot_sync(0xffffffffu, u < end);
        if (after) {
            const int l = __ffs(after) - 1;
            seq.q0 = __shfl_sync(0xffffffffu, mine.q0, l);
            seq.lq = __shfl_sync(0xffffffffu, mine.lq, l);
            seq.k0 = __shfl_sync(0xffffffffu, mine.k0, l);
            seq.lk = __shfl_sync(0xffffffffu, mine.lk, l);
            seq.number = base + (uint32_t)l;
            units = __shfl_sync(0xffffffffu, n, l);
            unit = u - (__shfl_sync(0xffffffffu, end, l) - units);
            return true;
        }
        u -= __shfl_sync(0xffffffffu, end, 31);
    }
    return false;
}
// The sequence that a row belongs to, from the starts: count if to none.
__host__ __device__ __forceinline__ uint32_t sequence_of(const int32_t* starts, uint32_t count, int64_t row)
{
    if (!starts) return 0;
    uint32_t lo = 0, hi = count;   // the first that ends behind the row
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (starts[mid + 1] > row) hi = mid;
        else lo = mid + 1;
    }
    return lo < count && starts[lo] <= row ? lo : count;
}
// Keys that the tokens up to `last` of a sequence see.
__host__ __device__ __forceinline__ int keys_seen(const Sequence& s, int last, bool causal)
{
    const int e = causal ? last + 1 - s.lq + s.lk : s.lk;   // in this order within 32 bits
    return e < 0 ? 0 : (e < s.lk ? e : s.lk);
}
// log2 of what the forward's f16 terms are held times: a term below f16's normal numbers is off
// by 2^-25, so that all keys of a row are off by 2^-13 of its largest together, a quarter of
// f16's half unit.  12 at most, which leaves the maximum 2^3 to grow.  4099 tokens, 16 heads of
// 128, causal, a few of whose keys draw far more weight than the first tile's: 65 us with 0 and 1, 67 with 4, 72 with
// 10: every raise rescales o.
__host__ __device__ __forceinline__ int held_up(int keys)
{
    int up = 0;
    while (up < 12 && keys > 4096 << up) ++up;
    return up;
}
// Queries that see a key come from this token of the sequence on.
__host__ __device__ __forceinline__ int first_query(const Sequence& s, int key, bool causal)
{
    const int t = causal ? key - (s.lk - s.lq) : 0;
    return t < 0 ? 0 : t;
}
// Packed rows of the tile of `tokens` tokens from t0 on that a key counts for.  Cut in tokens:
// a sequence's packed rows may be more than 2^31.
struct Columns {
    int from, to;
};
__host__ __device__ __forceinline__ Columns columns_of(const Sequence& s, int key, int t0, int tokens, int group, bool causal)
{
    const int left = s.lq - t0, hidden = first_query(s, key, causal) - t0;
    return {(hidden < 0 ? 0 : (hidden < tokens ? hidden : tokens)) * group, (left < tokens ? left : tokens) * group};
}

// The units' number at most, known without the starts.
inline int64_t units_at_most(int64_t rows, int64_t sequences, bool starts, int64_t tokens)
{
    const int64_t n = starts ? rows / tokens + (sequences < rows ? sequences : rows) : (rows + tokens - 1) / tokens;
    return n > 1 ? n : 1;
}

// Zeros to the rows of no sequence, row r of [rows][heads][dim] 16-bit elements (p) and
// of [rows][heads] floats (f), by the grid's blocks in turn.
struct Fill {
    uint16_t* p;
    int64_t row, head;
    float* f;
    int heads, dim;
};
__device__ __forceinline__ void fill_rows(const Fill& out, const int32_t* starts, uint32_t sequences, int64_t rows)
{
    if (!starts) return;
    const int64_t first = held(starts[0], 0, rows), last = held(starts[sequences], first, rows), none = first + rows - last;
    for (int64_t i = blockIdx.x; i < none; i += gridDim.x) {
        const int64_t r = i < first ? i : last + (i - first);
        for (int e = threadIdx.x; e < out.heads * out.dim; e += blockDim.x)
            out.p[r * out.row + e / out.dim * out.head + e % out.dim] = 0;
        if (out.f)
            for (int h = threadIdx.x; h < out.heads; h += blockDim.x) out.f[r * out.heads + h] = 0.0f;
    }
}

// ------------------------------------------------------------------ copies
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
// A tile: CHUNKS boxes of 64 columns.
template <int CHUNKS>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, int head, int row, uint32_t bar)
{
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) tma_load_3d(dst + c * kBox, map, 64 * c, head, row, bar);
}
// Zeros to rows [from, 128) of a tile of CHUNKS boxes, by a whole warp, before a product
// contracts over them: a box has a row in each 128 bytes.
template <int CHUNKS>
__device__ __forceinline__ void zero_rows(uint32_t tile, int from, int lane)
{
    for (uint32_t at = (uint32_t)from * 128 + lane * 16; at < kBox; at += 512)
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) st_shared16(tile + c * kBox + at, make_uint4(0, 0, 0, 0));
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
}

// ------------------------------------------------------------------ TMEM
// D[tmem] (+)= A B^T with A in TMEM (16-bit pairs, the lower k in the low half; 16 k are
// eight columns) and B in shared memory.
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, uint32_t add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(add)
        : "memory");
}

#define GS_R8(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])
#define GS_IO8(v, i) "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3]), "+r"(v[i + 4]), "+r"(v[i + 5]), "+r"(v[i + 6]), "+r"(v[i + 7])
#define GS_I8(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])
// 32 columns of this warp's 32 lanes, as tmem_ld16.
__device__ __forceinline__ void tmem_ld32(uint32_t tmem, uint32_t* v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, "
        "%26, %27, %28, %29, %30, %31}, [%32];"
        : GS_R8(v, 0), GS_R8(v, 8), GS_R8(v, 16), GS_R8(v, 24)
        : "r"(tmem));
}
__device__ __forceinline__ void tmem_ld32_wait(uint32_t* v)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" : GS_IO8(v, 0), GS_IO8(v, 8), GS_IO8(v, 16), GS_IO8(v, 24) : : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t tmem, const uint32_t* v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, "
        "%27, %28, %29, %30, %31, %32};" ::"r"(tmem),
        GS_I8(v, 0), GS_I8(v, 8), GS_I8(v, 16), GS_I8(v, 24)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t tmem, const uint32_t* v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(tmem),
        GS_I8(v, 0), GS_I8(v, 8)
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
#undef GS_R8
#undef GS_IO8
#undef GS_I8

// A tile's descriptor as the contracted rows of a product (k slow, 64 columns a box).
__device__ __forceinline__ uint32_t desc_rows(uint32_t addr) { return (addr >> 4) | ((kBox >> 4) << 16); }

// The greatest of three in one instruction.
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Three warpgroups start with 168 registers a thread, all that the SM has: the third, of
// few registers, leaves the other two 224 (2 x 224 + 56 = 3 x 168); two that start with 128
// (two blocks an SM) 200 and 56; five that start with 96, 104 four times and 56.  Whole
// warpgroups call these.
template <int N>
__device__ __forceinline__ void many_registers()
{
    static_assert(N == 224 || N == 200 || N == 104, "of three warpgroups, of two, of five");
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void few_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 56;"); }

// ------------------------------------------------------------------ rows out
// 32 columns from col of a row of `cols` 16-bit elements; vec: 2 the row starts on 32
// bytes, 1 on 16, 0 neither.
template <int T>
__device__ __forceinline__ void store_row32(uint16_t* row, int col, int cols, int vec, const float* v)
{
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = pack_half2(v[2 * j], v[2 * j + 1], T);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int left = cols - col - 16 * e;
        uint16_t* to = row + col + 16 * e;
        if (vec == 2 && left >= 16) {
            const uint32_t s[8] = {w[8 * e],     w[8 * e + 1], w[8 * e + 2], w[8 * e + 3],
                                   w[8 * e + 4], w[8 * e + 5], w[8 * e + 6], w[8 * e + 7]};
            st_global32(to, s);
            continue;
        }
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const int b = 8 * e + 4 * f;
            if (vec && left >= 8 * f + 8)
                *reinterpret_cast<uint4*>(to + 8 * f) = make_uint4(w[b], w[b + 1], w[b + 2], w[b + 3]);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (8 * f + j < left) to[8 * f + j] = (uint16_t)(w[b + (j >> 1)] >> (16 * (j & 1)));
        }
    }
}

// ------------------------------------------------------------------ host side
// A [rows][heads][dim] operand.
struct Tensor3 {
    const void* p;
    int64_t row, head;
};
// Strides of at least dim; out: no two elements share a place, so that one of the two
// strides spans the other's dimension.
bool tensor_ok(const void* p, int64_t row, int64_t head, int64_t rows, int64_t heads, int64_t dim, bool out);
// Base and strides as the tensor copies take them.
bool tensor_tma(const void* p, int64_t row, int64_t head, int64_t rows, int64_t heads);
// Rows of an output: 2 all on 32 bytes, 1 on 16, 0 neither.
int tensor_vec(const void* p, int64_t row, int64_t head, int64_t rows, int64_t heads);

// Operands that the tensor copies cannot take are copied once a call to rows of dim
// rounded up to 8 elements in the workspace.
inline int64_t packed_bytes(int64_t rows, int64_t heads, int64_t dim) { return round_up(rows * heads * round_up(dim, 8) * 2, 256); }
struct PackList {
    struct Job {
        const uint16_t* from;
        uint16_t* to;
        int64_t row, head, rows;
        int heads;
        unsigned first;   // block
    } job[4];
    int jobs = 0, dim = 0, pitch = 0;
    unsigned blocks = 0;
    // t as it is if the copies take it, else its place at `to` (moved on past it).
    Tensor3 add(const Tensor3& t, int64_t rows, int64_t heads, int64_t dim, char*& to);
    gs_status run(cudaStream_t st) const;
};
// Boxes of 64 columns of `box_heads` heads of box_rows rows.
inline gs_status tile_map(CUtensorMap* map, const Tensor3& t, int type, int64_t rows, int64_t heads, int64_t dim, int box_heads,
                          int box_rows)
{
    // the stride of a dimension of one is never used: one that the map takes
    const int64_t head = heads > 1 ? t.head : round_up(dim, 8), row = rows > 1 ? t.row : round_up(dim, 8);
    return make_map3(map, t.p, type, {dim, heads, rows}, {head, row}, {64, box_heads, box_rows});
}

// What every attention call checks of its sizes.
inline bool sizes_ok(int64_t q_rows, int64_t k_rows, int64_t sequences, int heads, int kv_heads, int dim, int type, float scale,
                     const void* q_starts, const void* k_starts)
{
    constexpr int64_t most = 0x7fffffffll - 1024;   // a tile past the last row still has a number
    if (!size_ok(q_rows, 0) || !size_ok(k_rows, 0) || !size_ok(sequences, 0) || q_rows > most || k_rows > most) return false;
    if (!q_starts != !k_starts || (!q_starts && sequences != 1)) return false;
    if (((uintptr_t)q_starts & 3u) || ((uintptr_t)k_starts & 3u)) return false;
    if (kv_heads < 1 || heads < kv_heads || heads % kv_heads || heads / kv_heads > GS_ATTENTION_MAX_GROUP || heads > 65536) return false;
    return dim >= 1 && dim <= GS_ATTENTION_MAX_DIM && type_half(type) && scale > 0.0f && scale <= 0x1p127f;   // times log2(e) finite
}

// Whether a wait of the file's kernels ran out; clears the mark.  The device is idle.
gs_status forward_wait_report(int* expired);
gs_status backward_wait_report(int* expired);

}  // namespace attn
}  // namespace gs
