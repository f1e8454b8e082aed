// gemm.cu -- the matrix product behind the decoder layers on the tensor cores.
//
//   D[m][n] = sum_k A[m][k] B[n][k], fp32 accumulators, epilogue on the way out
//
// One persistent CTA an SM (or a pair of CTAs on two SMs), 18 warps with fixed roles:
//   warp 0      TMA producer: tiles of A and B into a ring of 128-byte-swizzled stages
//   warp 1      issues tcgen05.mma into one of two to four TMEM accumulators
//   warps 2-17  epilogue: accumulator -> registers -> scale, bias, activation, gate ->
//               shared memory -> residual, row stores, while the next tiles accumulate.
//               Sixteen warps of few registers and short rolled loops: eight warps with
//               a whole row of 32 columns each in registers issued one instruction in
//               three cycles, waiting for instruction fetches and for each other
//               (1,000,000 x 64 -> 128 gated layer: 289 us)
// Either factor may have k as its fast or its slow index (the gradients contract over
// rows and over output features), so no operand is ever transposed in memory.
//
// What bounds it: with large k the tensor cores; a CTA's 128 x 128 tile takes
// 2 x 16 KB from shared memory per 64 k for 128 x 128 x 64 products, as much as
// shared memory delivers, so wide problems use the pair: 256 x 256 over two SMs, each
// holding half of B, half the shared-memory bytes a product.  With small k (a
// Gaussian decoder's layers) HBM, through the epilogue's stores.
#include <atomic>
#include <type_traits>

#include "attention.cuh"
#include "gemm.cuh"
#include "tc_common.cuh"

namespace gs {
namespace {

using namespace tc;

constexpr int kWarps = 18;
constexpr int kThreads = kWarps * 32;
constexpr int kEpiWarps = 16;
constexpr int kRowsA = 128;                      // accumulator rows of a CTA
constexpr int kStageRow = 128;                   // bytes of k a stage holds per row
constexpr int kGroupCols = 64;                   // output columns of a group of four epilogue warps
constexpr int kFewRows = 64;                     // up to here the weights' bytes are what a product costs
constexpr int kGroupM = 8;                       // m-tiles that run together (L2 reuse of B)

struct Params {
    CUtensorMap a[2], b[2];
    int64_t m, n;
    const float* x_scale;
    const float* w_scale[2];
    const void* bias;
    const void* residual;
    void* yp[2];
    void* zp;
    void* z2p;
    int64_t ldr, ldy[2], ldz, ldz2;
    int64_t part;             // elements of one partial sum
    uint32_t k_blocks;        // of one term
    uint32_t tiles_m, tiles_n, units;
    uint32_t splits, terms, probs;   // k ranges; products summed; independent products
    int k_elems;              // k of a stage
    int a_fast, b_fast, e4m3;
    uint32_t idesc;
    int bias_type, out_type, z_type, act;
    int y_vec, r_vec, z_vec, partial;
};

__device__ int g_wait_expired;

template <int BN, bool PAIR, bool GLU>
struct Shape {
    static constexpr int kTileM = PAIR ? 256 : 128;
    static constexpr int kRowsB = PAIR ? BN / 2 : BN;                  // rows of B a CTA holds
    static constexpr int kBytesA = kRowsA * kStageRow;
    static constexpr int kBytesB = kRowsB * kStageRow;
    static constexpr int kStageBytes = kBytesA + kBytesB;
    // Staging of an epilogue warp: 32 rows of 128 bytes, or of 64 in the wide pair, whose
    // sixth stage is worth more (32768 x 1024 -> 4096: 4, 5 stages 167, 162 us).
    static constexpr int kSlotRow = BN == 256 ? 64 : 128;
    static constexpr int kSlot = 32 * kSlotRow;
    static constexpr int kStages = BN == 128 && !PAIR ? 5 : 6;
    // Four groups of epilogue warps, 64 output columns each: all on one tile, or tiles in turn.
    static constexpr int kOutCols = GLU ? BN / 2 : BN;
    static constexpr int kGroupsTile = kOutCols / kGroupCols;
    static constexpr int kTurns = 4 / kGroupsTile;
    static constexpr int kAccs = kTurns > 2 ? kTurns : 2;              // accumulators in TMEM
    static constexpr int kTmemCols = kAccs * BN;
    static_assert(kTmemCols <= 512, "TMEM of an SM");
    static constexpr int kBars = kStages * 2 + kAccs * 2 + 2;          // even: what follows is 16-byte aligned
    static constexpr int kSmem = kStages * kStageBytes + kEpiWarps * kSlot + kBars * 8 + 16 + kEpiWarps * 32 * 4;
};

struct Unit {
    uint32_t prob, split, tm, tn, kb0, kb1;
};

__device__ __forceinline__ Unit decode(const Params& p, uint32_t u)
{
    Unit r;
    const uint32_t kb = p.k_blocks * p.terms;
    r.split = r.prob = 0;
    r.kb0 = 0;
    r.kb1 = kb;
    if (p.splits > 1) {
        const uint32_t per_split = p.tiles_m * p.tiles_n * p.probs;
        r.split = u / per_split;
        u -= r.split * per_split;
        r.kb0 = (uint32_t)((uint64_t)kb * r.split / p.splits);
        r.kb1 = (uint32_t)((uint64_t)kb * (r.split + 1) / p.splits);
    }
    if (p.probs > 1) {
        r.prob = u & 1;
        u >>= 1;
    }
    if (p.tiles_n == 1) {
        r.tm = u;
        r.tn = 0;
        return r;
    }
    const uint32_t per_group = kGroupM * p.tiles_n, first = u / per_group * kGroupM, in = u % per_group;
    const uint32_t rows = p.tiles_m - first < kGroupM ? p.tiles_m - first : kGroupM;
    r.tn = in / rows;
    r.tm = first + (in - r.tn * rows);
    return r;
}

// Byte of 16-byte piece j of row r in a staging slot of 32 rows of ROW bytes, swizzled
// so that neither a piece of eight rows nor the pieces of 128 bytes share a bank.
template <int ROW>
__device__ __forceinline__ uint32_t slot_piece(int r, int j)
{
    return ROW == 128 ? r * 128 + ((j ^ (r & 7)) << 4) : r * 64 + ((j ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ uint16_t ld_shared_u16(uint32_t a)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float ld_shared_f32(uint32_t a)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// 16 values of a thread's row into a slot: in 16 bits (pieces 2 step, 2 step + 1 of
// ROW / 2 columns) or in fp32 (four pieces of ROW / 4 columns).  mine: the address of
// piece 0 of the thread's row, which the swizzle makes the others' but for an xor.
template <int T>
__device__ __forceinline__ void slot_put_half(uint32_t mine, int step, const float (&v)[16])
{
    const uint32_t at = mine ^ (step << 5);
#pragma unroll
    for (int j = 0; j < 2; ++j)
        st_shared16(at ^ (j << 4),
                    make_uint4(pack_half2(v[8 * j], v[8 * j + 1], T), pack_half2(v[8 * j + 2], v[8 * j + 3], T),
                               pack_half2(v[8 * j + 4], v[8 * j + 5], T), pack_half2(v[8 * j + 6], v[8 * j + 7], T)));
}
__device__ __forceinline__ void slot_put(uint32_t mine, int step, const float (&v)[16])
{
    const uint32_t at = mine ^ (step << 6);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        st_shared16(at ^ (j << 4), make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                                              __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3])));
}

// Address of piece j of row r0 + R i of a slot, for the i-th of the rows a thread visits
// R apart (R 4 only under 128-byte rows): a constant away from the first but for the
// swizzle's third bit.
template <int ROW, int R>
__device__ __forceinline__ uint32_t slot_walk(uint32_t first, int i)
{
    return (ROW == 128 && R == 4 ? first ^ ((i & 1) << 6) : first) + i * R * ROW;
}

// A slot of ROW / 2 16-bit columns to memory (base: the chunk's first element): 16 bytes
// a thread where the rows are aligned (vec); single elements otherwise and where a row
// ends inside a piece.  Plain stores: they need no proxy fence and no wait before the
// slot is used again, and write nothing beside the matrix (a TMA store writes whole
// 16-byte pieces).
template <int ROW>
__device__ __forceinline__ void store_half(uint32_t slot, uint16_t* base, int64_t ld, int rows, int cols, bool vec, int lane)
{
    constexpr int kCols = ROW / 2, kPieces = ROW / 16, kRows = 32 / kPieces;
    if (vec) {
        const int j = lane % kPieces, r0 = lane / kPieces, left = cols - 8 * j;
        const uint32_t from = slot + slot_piece<ROW>(r0, j);
        uint16_t* at = base + r0 * ld + 8 * j;
        const int64_t step = kRows * ld;
        if (left >= 8) {
#pragma unroll
            for (int i = 0; i < 32 / kRows; ++i, at += step)
                if (r0 + kRows * i < rows) *reinterpret_cast<uint4*>(at) = ld_shared16(slot_walk<ROW, kRows>(from, i));
        } else if (left > 0) {
#pragma unroll 2
            for (int i = 0; i < 32 / kRows; ++i, at += step) {
                if (r0 + kRows * i >= rows) break;
                const uint4 q = ld_shared16(slot_walk<ROW, kRows>(from, i));
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int e = 0; e < 7; ++e)
                    if (e < left) at[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
            }
        }
    } else {
        for (int c = lane; c < cols; c += 32) {
            uint16_t* at = base + c;
#pragma unroll 8
            for (int r = 0; r < 32; ++r, at += ld) {
                const uint16_t v = ld_shared_u16(slot + slot_piece<ROW>(r, c >> 3) + 2 * (c & 7));
                if (r < rows) *at = v;
            }
        }
    }
}

// A chunk of 32 rows of ROW / 4 columns on its way out: 16 bytes of a row a thread
// where y's and the residual's rows are aligned, a column a thread otherwise.
template <int ROW, int OSZ>
struct Chunk {
    static constexpr int kCols = ROW / 4, kPer = 16 / OSZ, kPieces = kCols / kPer, kRows = 32 / kPieces, kSteps = 32 / kRows;
    static constexpr int kColThreads = 32 / kCols;             // threads that share a column, rows in turn
    static constexpr int kWords = 32 / kColThreads * OSZ / 4;  // a thread's rows of a column, packed
    static_assert(kWords <= 4 * kSteps, "the residual's registers hold either layout");
};

// The residual's part of kSteps / PARTS of a chunk's steps in that layout.  In 16 bits
// a whole chunk is fetched before the accumulator is read; in 32 its registers would
// spill, and it is fetched in parts on the way out.
template <int ROW, int OSZ>
struct Residual {
    static constexpr int kParts = OSZ == 4 ? 2 : 1, kSteps = Chunk<ROW, OSZ>::kSteps / kParts;
    uint4 q[kSteps];
};
template <int ROW, int OSZ>
__device__ __forceinline__ void fetch_residual(Residual<ROW, OSZ>& res, int part, const char* base, int64_t ld, int rows,
                                               int cols, bool vec, int lane)
{
    using C = Chunk<ROW, OSZ>;
    using R = Residual<ROW, OSZ>;
    if (!vec) {
        constexpr int kVisits = 32 / C::kColThreads / R::kParts;
        uint32_t w[4 * R::kSteps];
#pragma unroll
        for (int i = 0; i < 4 * R::kSteps; ++i) w[i] = 0;
        const int c = lane % C::kCols, r0 = lane / C::kCols + part * kVisits * C::kColThreads;
        const char* at = base + (r0 * ld + c) * OSZ;
#pragma unroll
        for (int i = 0; i < kVisits; ++i, at += C::kColThreads * ld * OSZ) {
            if (c >= cols || r0 + i * C::kColThreads >= rows) continue;
            if constexpr (OSZ == 4) w[i] = *(const uint32_t*)at;
            else w[i >> 1] |= (uint32_t)(*(const uint16_t*)at) << (16 * (i & 1));
        }
#pragma unroll
        for (int i = 0; i < R::kSteps; ++i) res.q[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        return;
    }
    const int j = lane % C::kPieces, r0 = lane / C::kPieces + part * R::kSteps * C::kRows, left = cols - C::kPer * j;
    const char* at = base + (r0 * ld + C::kPer * j) * OSZ;
    const int64_t step = C::kRows * ld * OSZ;
#pragma unroll
    for (int i = 0; i < R::kSteps; ++i, at += step) {
        res.q[i] = make_uint4(0, 0, 0, 0);
        if (r0 + i * C::kRows >= rows) continue;
        if (left >= C::kPer) res.q[i] = *reinterpret_cast<const uint4*>(at);
        else if (left > 0) {   // the row ends inside this piece
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < C::kPer - 1; ++e) {
                if (e >= left) continue;
                if constexpr (OSZ == 4) w[e] = ((const uint32_t*)at)[e];
                else w[e >> 1] |= (uint32_t)((const uint16_t*)at)[e] << (16 * (e & 1));
            }
            res.q[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// A slot of fp32 columns to memory, the residual (from, or the 16-bit one in res) added
// and rounded once.
template <int ROW, int OSZ, int T>
__device__ __forceinline__ void store_chunk(uint32_t slot, Residual<ROW, OSZ>& res, const char* from, int64_t ldr, char* base,
                                            int64_t ld, int rows, int cols, bool vec, int lane)
{
    using C = Chunk<ROW, OSZ>;
    using R = Residual<ROW, OSZ>;
    const bool add = from != nullptr;
#pragma unroll 1
    for (int part = 0; part < R::kParts; ++part) {
        if (R::kParts > 1 && add) fetch_residual(res, part, from, ldr, rows, cols, vec, lane);
        if (vec) {
            const int j = lane % C::kPieces, r0 = lane / C::kPieces + part * R::kSteps * C::kRows, left = cols - C::kPer * j;
            if (left <= 0) continue;
            const uint32_t first = slot + slot_piece<ROW>(r0, OSZ == 4 ? j : 2 * j);
            char* at = base + (r0 * ld + C::kPer * j) * OSZ;
            const int64_t step = C::kRows * ld * OSZ;
#pragma unroll
            for (int i = 0; i < R::kSteps; ++i, at += step) {
                if (r0 + i * C::kRows >= rows) break;
                const uint32_t a = slot_walk<ROW, C::kRows>(first, i);
                uint4 out = ld_shared16(a);
                if constexpr (OSZ == 4) {
                    if (add) {
                        out.x = __float_as_uint(__uint_as_float(out.x) + __uint_as_float(res.q[i].x));
                        out.y = __float_as_uint(__uint_as_float(out.y) + __uint_as_float(res.q[i].y));
                        out.z = __float_as_uint(__uint_as_float(out.z) + __uint_as_float(res.q[i].z));
                        out.w = __float_as_uint(__uint_as_float(out.w) + __uint_as_float(res.q[i].w));
                    }
                } else {
                    const uint4 hi = ld_shared16(a ^ 16);   // piece 2 j + 1
                    const float2 r = unpack_half2(res.q[i].x, T), g = unpack_half2(res.q[i].y, T),
                                 b = unpack_half2(res.q[i].z, T), d = unpack_half2(res.q[i].w, T);
                    out = make_uint4(pack_half2(__uint_as_float(out.x) + r.x, __uint_as_float(out.y) + r.y, T),
                                     pack_half2(__uint_as_float(out.z) + g.x, __uint_as_float(out.w) + g.y, T),
                                     pack_half2(__uint_as_float(hi.x) + b.x, __uint_as_float(hi.y) + b.y, T),
                                     pack_half2(__uint_as_float(hi.z) + d.x, __uint_as_float(hi.w) + d.y, T));
                }
                if (left >= C::kPer) *reinterpret_cast<uint4*>(at) = out;
                else {   // the row ends inside this piece
                    const uint32_t w[4] = {out.x, out.y, out.z, out.w};
#pragma unroll
                    for (int e = 0; e < C::kPer - 1; ++e) {
                        if (e >= left) continue;
                        if constexpr (OSZ == 4) ((uint32_t*)at)[e] = w[e];
                        else ((uint16_t*)at)[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
                    }
                }
            }
        } else if (lane % C::kCols < cols) {
            constexpr int kVisits = 32 / C::kColThreads / R::kParts;
            const int c = lane % C::kCols, rr = lane / C::kCols + part * kVisits * C::kColThreads;
            char* at = base + (rr * ld + c) * OSZ;
#pragma unroll
            for (int i = 0; i < kVisits; ++i, at += C::kColThreads * ld * OSZ) {
                const int r = rr + i * C::kColThreads;
                float v = ld_shared_f32(slot + slot_piece<ROW>(r, c >> 2) + 4 * (c & 3));
                const int word = OSZ == 4 ? i : i >> 1;
                const uint4 q = res.q[word >> 2];
                const uint32_t w = (word & 3) == 0 ? q.x : ((word & 3) == 1 ? q.y : ((word & 3) == 2 ? q.z : q.w));
                if (add) v += OSZ == 4 ? __uint_as_float(w) : (i & 1 ? unpack_half2(w, T).y : unpack_half2(w, T).x);
                if (r < rows) store_elem(at, 0, T, v);
            }
        }
    }
}

template <int T>
__device__ __forceinline__ void pack_half16(uint32_t (&w)[8], const float (&v)[16])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = pack_half2(v[2 * j], v[2 * j + 1], T);
}

template <int ACT, bool FINE, bool GLU>
__device__ __forceinline__ void activate(float (&v)[16])
{
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
        const float2 f = unpair(act_value2<ACT, FINE, GLU>(pair(v[j], v[j + 1])));
        v[j] = f.x, v[j + 1] = f.y;
    }
}
template <bool FINE, bool GLU>
__device__ __forceinline__ void activate(float (&v)[16], int act)
{
    if (act == GS_ACT_SILU) activate<GS_ACT_SILU, FINE, GLU>(v);
    else if (act == GS_ACT_GELU) activate<GS_ACT_GELU, FINE, GLU>(v);
    else if (act == GS_ACT_RELU) activate<GS_ACT_RELU, FINE, GLU>(v);
}

// The loops of the producer's and the MMA warp's elected lanes.  One thread's
// instructions come five or more cycles apart, so a k-block must cost few of them:
// the factors' orders are constants, the ring is stepped, addresses are added to
// (with all of that in the loop a k-block took 500 cycles whatever its products:
// 2048 x 4096 -> 1024 19 us).
// load_tiles returns the stages it has filled.  It stops when its own wait has run out,
// not when another role gives up: a stage is freed in both CTAs of a pair by one commit,
// so both producers stop behind the same copies, and the first CTA's barriers, which count
// both CTAs' bytes, tell when all of them have landed.
template <int BN, bool PAIR, bool GLU, bool A_FAST, bool B_FAST>
__device__ __forceinline__ uint32_t load_tiles(const Params& p, uint32_t first, uint32_t step, uint32_t rank, uint32_t stages,
                                           uint32_t bar_full, uint32_t bar_empty, volatile int* gave_up)
{
    using S = Shape<BN, PAIR, GLU>;
    const uint32_t full0 = PAIR ? map_rank(bar_full, 0) : bar_full;   // the pair counts at its first CTA
    const int k_elems = p.k_elems;
    const uint32_t k_blocks = p.k_blocks, units = p.units;
    Ring<S::kStages> ring;
    uint32_t issued = 0;
    for (uint32_t u = first; u < units; u += step) {
        const Unit q = decode(p, u);
        const int row_a = (int)(q.tm * S::kTileM + rank * kRowsA);
        const int row_b = GLU ? (int)(q.tn * (BN / 2)) : (int)(q.tn * BN + rank * S::kRowsB);
        uint32_t kb = q.kb0;
        while (kb < q.kb1) {   // the k-blocks of one term
            const uint32_t term = kb >= k_blocks ? 1 : 0, which = p.probs > 1 ? q.prob : term;
            const uint32_t end = term == 0 && q.kb1 > k_blocks ? k_blocks : q.kb1;
            const CUtensorMap *a = &p.a[which], *b = &p.b[GLU && PAIR ? rank : which];
            int k = (int)(kb - term * k_blocks) * k_elems;
            for (; kb < end; ++kb, k += k_elems, ++issued) {
                if (!mbar_wait_alone(bar_empty + 8 * ring.s, ring.parity ^ 1)) {
                    *gave_up = 1;
                    return issued;
                }
                const uint32_t full = full0 + 8 * ring.s, sa = stages + ring.s * S::kStageBytes, sb = sa + S::kBytesA;
                if (rank == 0) mbar_expect(bar_full + 8 * ring.s, S::kStageBytes * (PAIR ? 2 : 1));
                if constexpr (A_FAST) tma_load_2d<PAIR>(sa, a, k, row_a, full);
                else
#pragma unroll
                    for (int i = 0; i < kRowsA / 64; ++i) tma_load_2d<PAIR>(sa + i * 8192, a, row_a + 64 * i, k, full);
                if constexpr (GLU && !PAIR) {
                    tma_load_2d<PAIR>(sb, &p.b[0], k, row_b, full);
                    tma_load_2d<PAIR>(sb + S::kBytesB / 2, &p.b[1], k, row_b, full);
                } else if constexpr (B_FAST) tma_load_2d<PAIR>(sb, b, k, row_b, full);
                else
#pragma unroll
                    for (int i = 0; i < S::kRowsB / 64; ++i) tma_load_2d<PAIR>(sb + i * 8192, b, row_b + 64 * i, k, full);
                ring.next();
            }
        }
    }
    return issued;
}

template <int BN, bool PAIR, bool GLU, bool A_FAST, bool B_FAST, bool E4M3>
__device__ __forceinline__ void issue_products(const Params& p, uint32_t first, uint32_t step, uint32_t stages,
                                               uint32_t bar_full, uint32_t bar_empty, uint32_t bar_acc, uint32_t bar_free,
                                               uint32_t tmem, volatile int* gave_up)
{
    using S = Shape<BN, PAIR, GLU>;
    constexpr uint32_t kStepA = k_step(A_FAST), kStepB = k_step(B_FAST);
    const uint32_t lo_a = desc_lo(stages, A_FAST), lo_b = desc_lo(stages + S::kBytesA, B_FAST), idesc = p.idesc;
    const uint32_t units = p.units;
    Ring<S::kStages> ring;
    Ring<S::kAccs> acc;
    for (uint32_t u = first; u < units; u += step) {
        const Unit q = decode(p, u);
        if (!mbar_wait(bar_free + 8 * acc.s, acc.parity ^ 1, gave_up)) return;
        tc_fence_after();
        const uint32_t d = tmem + acc.s * BN;
        uint32_t add = 0;
        for (uint32_t kb = q.kb1 - q.kb0; kb > 0; --kb) {
            if (!mbar_wait(bar_full + 8 * ring.s, ring.parity, gave_up)) return;
            tc_fence_after();
            const uint32_t a = lo_a + ring.s * (S::kStageBytes >> 4), b = lo_b + ring.s * (S::kStageBytes >> 4);
            mma<PAIR, E4M3>(d, a, kDescHi, b, kDescHi, idesc, add);
#pragma unroll
            for (uint32_t i = 1; i < 4; ++i)
                mma<PAIR, E4M3>(d, a + i * kStepA, kDescHi, b + i * kStepB, kDescHi, idesc, 1);
            add = 1;
            mma_commit<PAIR>(bar_empty + 8 * ring.s);   // the stage is free once these are done
            ring.next();
        }
        mma_commit<PAIR>(bar_acc + 8 * acc.s);
        acc.next();
    }
}

// dh's part of a chunk (C 16-bit columns) into the first half of a slot's rows, 16 bytes a
// thread, several threads a row (a thread a row instead kept the L1 at 71 %: 200 us a
// million rows of 64 -> 128); then each thread takes its own row.
template <int ROW>
__device__ __forceinline__ void stage_rows(uint32_t slot, const uint16_t* base, int64_t ld, int rows, int cols, bool vec,
                                           int lane)
{
    constexpr int kPieces = ROW / 32, kRows = 32 / kPieces;   // of a half row
    const int j = lane % kPieces, r0 = lane / kPieces, left = cols - 8 * j;
    const uint16_t* at = base + r0 * ld + 8 * j;
    const int64_t step = kRows * ld;
    uint4 q[32 / kRows];
#pragma unroll
    for (int i = 0; i < 32 / kRows; ++i, at += step) {
        q[i] = make_uint4(0, 0, 0, 0);
        if (r0 + i * kRows >= rows) continue;
        if (vec && left >= 8) q[i] = *reinterpret_cast<const uint4*>(at);
        else {
            uint32_t t[4] = {0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < left) t[e >> 1] |= (uint32_t)at[e] << (16 * (e & 1));
            q[i] = make_uint4(t[0], t[1], t[2], t[3]);
        }
    }
#pragma unroll
    for (int i = 0; i < 32 / kRows; ++i) st_shared16(slot + slot_piece<ROW>(r0 + i * kRows, j), q[i]);
}

// The activation at run time.
__device__ __forceinline__ void glu_gradient_by(float (&g)[16], float (&u)[16], const float (&dh)[16], int act)
{
    if (act == GS_ACT_SILU) glu_gradient<GS_ACT_SILU>(g, u, dh);
    else if (act == GS_ACT_GELU) glu_gradient<GS_ACT_GELU>(g, u, dh);
    else if (act == GS_ACT_RELU) glu_gradient<GS_ACT_RELU>(g, u, dh);
    else glu_gradient<GS_ACT_NONE>(g, u, dh);
}

// GLU: B's rows are half gate, half up; the epilogue joins column c with c + BN/2.
// GRAD: it takes dh where a residual would be and gives dg and du.
// OSZ: bytes of an output element.
template <int BN, bool PAIR, bool GLU, int OSZ, bool GRAD = false>
__global__ void __launch_bounds__(kThreads, 1) gemm_kernel(const __grid_constant__ Params p)
{
    using S = Shape<BN, PAIR, GLU>;
    extern __shared__ __align__(1024) char smem_raw[];   // the swizzle patterns repeat every 1024 bytes
    const uint32_t base = smem_addr(smem_raw);
    if (base & 1023u) {   // every thread sees the same address; there is no padding to move within
        g_wait_expired = 1;
        return;
    }
    const uint32_t stages = base, slots = base + S::kStages * S::kStageBytes;
    const uint32_t bars = slots + kEpiWarps * S::kSlot;
    const uint32_t bar_full = bars, bar_empty = bars + S::kStages * 8, bar_acc = bar_empty + S::kStages * 8,
                   bar_free = bar_acc + S::kAccs * 8, bar_drain = bar_free + S::kAccs * 8;
    char* tail = smem_raw + (bars + S::kBars * 8 - base);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail);
    volatile int* gave_up = reinterpret_cast<volatile int*>(tail + 4);
    float* columns = reinterpret_cast<float*>(tail + 16);   // [warp][2][16]: scale, bias (or the second scale)

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_rank() : 0;
    const uint32_t first = PAIR ? blockIdx.x >> 1 : blockIdx.x, step = PAIR ? gridDim.x >> 1 : gridDim.x;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(bar_full + 8 * i, 1);
            mbar_init(bar_empty + 8 * i, 1);
        }
        for (int i = 0; i < S::kAccs; ++i) {
            mbar_init(bar_acc + 8 * i, 1);
            mbar_init(bar_free + 8 * i, 4 * S::kGroupsTile * (PAIR ? 2 : 1));
        }
        mbar_init(bar_drain, 1);
        *gave_up = 0;
        mbar_init_fence();
    }
    if (warp == 1) tmem_alloc<PAIR>(smem_addr(tmem_slot), S::kTmemCols);
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();   // both CTAs' barriers exist before any copy or commit reaches them
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    wait_for_predecessor();

    if (warp == 0) {
        if (elect_one()) {
            prefetch_map(&p.a[0]);
            prefetch_map(&p.b[0]);
            uint32_t issued = 0;
            if (p.b_fast) issued = load_tiles<BN, PAIR, GLU, true, true>(p, first, step, rank, stages, bar_full, bar_empty, gave_up);
            else if constexpr (!GLU) {
                if (p.a_fast) issued = load_tiles<BN, PAIR, GLU, true, false>(p, first, step, rank, stages, bar_full, bar_empty, gave_up);
                else issued = load_tiles<BN, PAIR, GLU, false, false>(p, first, step, rank, stages, bar_full, bar_empty, gave_up);
            }
            // the block does not leave before its copies have landed (the pair: at its last cluster barrier)
            bool landed = true;
            if (rank == 0)
                last_copies<S::kStages>(issued, [&](uint32_t s, uint32_t parity) { landed = landed && mbar_wait_alone(bar_full + 8 * s, parity); });
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            const auto issue = [&](auto a_fast, auto b_fast, auto e4m3) {
                issue_products<BN, PAIR, GLU, decltype(a_fast)::value, decltype(b_fast)::value, decltype(e4m3)::value>(
                    p, first, step, stages, bar_full, bar_empty, bar_acc, bar_free, tmem, gave_up);
            };
            const std::true_type yes;
            const std::false_type no;
            if (p.e4m3) issue(yes, yes, yes);
            else if (p.b_fast) issue(yes, yes, no);
            else if constexpr (!GLU) {
                if (p.a_fast) issue(yes, no, no);
                else issue(no, no, no);
            }
            if (*gave_up) {
                mma_commit<PAIR>(bar_drain);
                mbar_wait_alone(bar_drain, 0);
            }
        }
    } else {
        // -------------------------------------------------------------- epilogue
        const int quarter = warp & 3, group = (warp - 2) >> 2;
        const int turn = group / S::kGroupsTile, col_group = group % S::kGroupsTile;
        const uint32_t slot = slots + (warp - 2) * S::kSlot;
        const uint32_t free0 = PAIR ? map_rank(bar_free, 0) : bar_free;
        float* const factors = columns + (warp - 2) * 32;
        const bool has_factors = p.e4m3 || p.bias;
        const int passes = p.zp ? (GLU ? 3 : 2) : 1;
        const uint32_t mine = slot + slot_piece<S::kSlotRow>(lane, 0);
        const uint32_t m = (uint32_t)p.m, n = (uint32_t)p.n;
        const auto factor = [&](uint32_t col) -> float {
            if (lane < 16) return p.w_scale[0] && col < n ? p.w_scale[0][col] : 1.0f;
            if constexpr (GLU) return p.w_scale[1] && col < n ? p.w_scale[1][col] : 1.0f;
            else return p.bias && col < n ? load_elem(p.bias, col, p.bias_type) : 0.0f;
        };
        uint32_t tile = 0;
        for (uint32_t u = first; u < p.units; u += step, ++tile) {
            if (S::kTurns > 1 && (int)(tile % S::kTurns) != turn) continue;
            const uint32_t acc = tile % S::kAccs;
            const Unit q = decode(p, u);
            const uint32_t row0 = q.tm * S::kTileM + rank * kRowsA + quarter * 32;
            const uint32_t col0 = q.tn * S::kOutCols + col_group * kGroupCols;
            const bool live = row0 < m && col0 < n;
            const int rows = live ? (int)(m - row0 < 32 ? m - row0 : 32) : 0, cols = live ? (int)(n - col0) : 0;
            const float xs = p.x_scale && lane < rows ? p.x_scale[row0 + lane] : 1.0f;
            // the columns' factors, 16 columns at a time: lanes 0-15 the first, 16-31 the
            // second; they and the residual's way into L2 start before the accumulator is waited for
            float f0 = 1.0f, f1 = 1.0f, f2 = 1.0f, f3 = 1.0f;
            if (has_factors && live) {
                const uint32_t col = col0 + (lane & 15);
                f0 = factor(col), f1 = factor(col + 16), f2 = factor(col + 32), f3 = factor(col + 48);
            }
            if ((!GLU || GRAD) && p.residual && lane < rows) {
                const char* at = (const char*)p.residual + ((int64_t)(row0 + lane) * p.ldr + col0) * OSZ;
                asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
                if (OSZ == 4 && cols > 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + 128));
            }
            if (!__all_sync(0xffffffffu, mbar_wait(bar_acc + 8 * acc, (tile / S::kAccs) & 1, gave_up))) break;
            tc_fence_after();
            const uint32_t d = tmem + ((uint32_t)(quarter * 32) << 16) + acc * BN + col_group * kGroupCols;

            // 16 columns from c on, as pass `pass` of `passes` wants them: gate, up, product
            // (pass 0, 1, last of a gated layer); pre-activation, activation (pass 0, last)
            const auto columns16 = [&](int c, int pass, float (&v)[16]) {
                const bool last = pass == passes - 1;
                if (has_factors) {
                    const float f = c < 32 ? (c == 0 ? f0 : f1) : (c == 32 ? f2 : f3);
                    __syncwarp();   // the last readers are done
                    factors[lane] = f;
                    __syncwarp();
                }
                uint32_t raw[16];
                tmem_ld16(d + c + (GLU && !last && pass == 1 ? BN / 2 : 0), raw);
                if constexpr (GLU) {
                    if (last) {
                        uint32_t up[16];
                        tmem_ld16(d + c + BN / 2, up);
                        tmem_ld_wait(raw);
                        tmem_ld_wait(up);
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(raw[j]);
                        if (p.e4m3) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                v[j] *= xs * factors[j];
                                up[j] = __float_as_uint(__uint_as_float(up[j]) * (xs * factors[16 + j]));
                            }
                        }
                        activate<OSZ == 4, GLU>(v, p.act);
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] *= __uint_as_float(up[j]);
                        return;
                    }
                    tmem_ld_wait(raw);
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(raw[j]);
                    if (p.e4m3) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] *= xs * factors[pass * 16 + j];
                    }
                } else {
                    tmem_ld_wait(raw);
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(raw[j]);
                    if (has_factors) {
                        if (p.e4m3) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) v[j] *= xs * factors[j];
                        }
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            const float2 f = unpair(add2(pair(v[j], v[j + 1]), pair(factors[16 + j], factors[17 + j])));
                            v[j] = f.x, v[j + 1] = f.y;
                        }
                    }
                    if (last) activate<OSZ == 4, GLU>(v, p.act);
                }
            };

            if constexpr (GRAD) {   // a slot's row: dg, then du, of a quarter of its bytes' columns
                constexpr int kCols = S::kSlotRow / 4, kHalf = S::kSlotRow / 32;   // pieces of dg
                const uint16_t* from = (const uint16_t*)p.residual + (int64_t)row0 * p.ldr + col0;
                const int j = lane % (2 * kHalf);
                // lanes whose piece is du's see its rows kHalf pieces to the left
                uint16_t* to = (uint16_t*)p.yp[j < kHalf ? 0 : 1] + (int64_t)row0 * p.ldy[0] + col0 - (j < kHalf ? 0 : 8 * kHalf);
#pragma unroll 1
                for (int c = 0; c < kGroupCols && c < cols; c += kCols, to += kCols, from += kCols) {
                    const int part = cols - c < kCols ? cols - c : kCols;
                    uint32_t dh[kCols / 2];
                    __syncwarp();   // the slot's last readers are done
                    stage_rows<S::kSlotRow>(slot, from, p.ldr, rows, part, p.r_vec, lane);
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < kCols / 8; ++e) {
                        const uint4 q = ld_shared16(mine ^ (e << 4));
                        dh[4 * e] = q.x, dh[4 * e + 1] = q.y, dh[4 * e + 2] = q.z, dh[4 * e + 3] = q.w;
                    }
#pragma unroll
                    for (int s = 0; s < kCols / 16; ++s) {
                        uint32_t raw[16], up[16];
                        tmem_ld16(d + c + 16 * s, raw);
                        tmem_ld16(d + c + 16 * s + BN / 2, up);
                        float g[16], u[16], v[16];
                        if (p.out_type == GS_BF16) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float2 f = unpack_half2(dh[8 * s + e], GS_BF16);
                                v[2 * e] = f.x, v[2 * e + 1] = f.y;
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float2 f = unpack_half2(dh[8 * s + e], GS_F16);
                                v[2 * e] = f.x, v[2 * e + 1] = f.y;
                            }
                        }
                        tmem_ld_wait(raw);
                        tmem_ld_wait(up);
#pragma unroll
                        for (int e = 0; e < 16; ++e) g[e] = __uint_as_float(raw[e]), u[e] = __uint_as_float(up[e]);
                        glu_gradient_by(g, u, v, p.act);
                        if (p.out_type == GS_BF16) {
                            slot_put_half<GS_BF16>(mine, s, g);
                            slot_put_half<GS_BF16>(mine ^ (kHalf << 4), s, u);
                        } else {
                            slot_put_half<GS_F16>(mine, s, g);
                            slot_put_half<GS_F16>(mine ^ (kHalf << 4), s, u);
                        }
                    }
                    __syncwarp();
                    store_half<S::kSlotRow>(slot, to, p.ldy[0], rows, j < kHalf ? part : part + 8 * kHalf, true, lane);
                }
            }
            for (int pass = 0; !GRAD && live && pass < passes; ++pass) {
                const bool last = pass == passes - 1;
                if (GLU || !last || (OSZ == 2 && !p.residual)) {   // in 16 bits
                    constexpr int kCols = S::kSlotRow / 2;
                    const int type = last ? p.out_type : p.z_type;
                    const int64_t ld = last ? p.ldy[q.prob] : (GLU && pass == 1 ? p.ldz2 : p.ldz);
                    uint16_t* to = (uint16_t*)(last ? p.yp[q.prob] : (GLU && pass == 1 ? p.z2p : p.zp)) + row0 * ld + col0;
                    // The wide pair's slots hold half lines: where a thread's 32 bytes are a sector they go
                    // straight out (1,000,000 x 64 -> 192 95 us staged, 81 so; gated 100,000 x 256 -> 512
                    // 54, 45; in the other shapes up to 7 % slower).
                    if (BN == 256 && cols >= kGroupCols && (((uintptr_t)to | (uintptr_t)(ld * 2)) & 31) == 0) {
                        to += lane * ld;
#pragma unroll 1
                        for (int c = 0; c < kGroupCols; c += 16) {
                            float v[16];
                            columns16(c, pass, v);
                            uint32_t w[8];
                            if (type == GS_BF16) pack_half16<GS_BF16>(w, v);
                            else pack_half16<GS_F16>(w, v);
                            if (lane < rows) st_global32(to + c, w);
                        }
                        continue;
                    }
#pragma unroll 1
                    for (int c = 0; c < kGroupCols && c < cols; c += kCols, to += kCols) {
                        __syncwarp();   // the slot's last readers are done
#pragma unroll 1
                        for (int s = 0; s < kCols / 16; ++s) {
                            float v[16];
                            columns16(c + 16 * s, pass, v);
                            if (type == GS_BF16) slot_put_half<GS_BF16>(mine, s, v);
                            else slot_put_half<GS_F16>(mine, s, v);
                        }
                        __syncwarp();
                        store_half<S::kSlotRow>(slot, to, ld, rows, cols - c < kCols ? cols - c : kCols,
                                                last ? p.y_vec : p.z_vec, lane);
                    }
                } else if constexpr (!GLU) {   // in fp32, the residual added on the way out
                    constexpr int kCols = S::kSlotRow / 4;
                    const bool add = p.residual != nullptr, vec = p.y_vec && (p.r_vec || !add);
                    const int64_t ld = p.ldy[p.partial ? 0 : q.prob];
                    char* to = (char*)p.yp[p.partial ? 0 : q.prob] + (row0 * ld + col0) * OSZ;
                    if (p.partial) to += (int64_t)(q.prob * p.splits + q.split) * p.part * OSZ;
                    const char* from = add ? (const char*)p.residual + (row0 * p.ldr + col0) * OSZ : nullptr;
#pragma unroll 1
                    for (int c = 0; c < kGroupCols && c < cols; c += kCols, to += kCols * OSZ) {
                        const int part = cols - c < kCols ? cols - c : kCols;
                        Residual<S::kSlotRow, OSZ> res;
                        if (OSZ == 2) fetch_residual(res, 0, from, p.ldr, rows, part, vec, lane);
                        __syncwarp();
#pragma unroll   // both steps' TMEM reads in flight
                        for (int s = 0; s < kCols / 16; ++s) {
                            float v[16];
                            columns16(c + 16 * s, pass, v);
                            slot_put(mine, s, v);
                        }
                        __syncwarp();
                        if constexpr (OSZ == 4)
                            store_chunk<S::kSlotRow, 4, GS_F32>(slot, res, from, p.ldr, to, ld, rows, part, vec, lane);
                        else if (p.out_type == GS_BF16)
                            store_chunk<S::kSlotRow, 2, GS_BF16>(slot, res, from, p.ldr, to, ld, rows, part, vec, lane);
                        else store_chunk<S::kSlotRow, 2, GS_F16>(slot, res, from, p.ldr, to, ld, rows, part, vec, lane);
                        if (add) from += kCols * OSZ;
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR) mbar_arrive_cluster(free0 + 8 * acc);
                else mbar_arrive(bar_free + 8 * acc);
            }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0 && *gave_up) atomicExch(&g_wait_expired, 1);
    tc_fence_before();
    if constexpr (PAIR) cluster_sync();   // the peer's commits and arrivals have reached this CTA's barriers
    if (warp == 1) {
        tc_fence_after();
        tmem_free<PAIR>(tmem, S::kTmemCols);
    }
}

// ------------------------------------------------------------------ few rows
// With few rows (single tokens, small batches) the weights' bytes are the floor, so
// the roles are turned: a CTA holds 128 rows of the weights as the MMA's M side
// (64 of gate and 64 of up for a gated layer) and at most NB rows of x as its N
// side, and the CTAs of a cluster split k, so that enough SMs stream the weights
// (4096 x 1024: 32 tiles x 4).  Their partial sums meet in shared memory across the
// cluster, added in rank order, and every CTA finishes its share of the outputs:
// one launch, no workspace, no atomics.
struct RowsParams {
    CUtensorMap x, w[2];
    int64_t m, n;
    const float* x_scale;
    const float* w_scale[2];
    const void* bias;
    const void* residual;
    void *y, *z, *z2;
    int64_t ldr, ldy, ldz, ldz2;
    uint32_t k_blocks, tiles_n, idesc;
    int k_elems, e4m3, bias_type, out_type, z_type, act;
};

constexpr int kRowsThreads = 256;

template <int NB, bool GLU>
struct RowsShape {
    static constexpr int kBytesW = 128 * kStageRow, kBytesX = NB * kStageRow, kStageBytes = kBytesW + kBytesX;
    static constexpr int kStages = NB == 64 ? 8 : 10;
    static constexpr int kSmem = kStages * kStageBytes + kStages * 16 + 32;
    static constexpr int kTmemCols = NB < 32 ? 32 : NB;
};

template <int NB, bool GLU>
__global__ void __launch_bounds__(kRowsThreads, 1) rows_kernel(const __grid_constant__ RowsParams p)
{
    using S = RowsShape<NB, GLU>;
    extern __shared__ __align__(1024) char smem_raw[];
    const uint32_t stages = smem_addr(smem_raw);
    if (stages & 1023u) {
        g_wait_expired = 1;
        return;
    }
    const uint32_t bar_full = stages + S::kStages * S::kStageBytes, bar_empty = bar_full + S::kStages * 8,
                   bar_acc = bar_empty + S::kStages * 8;
    char* tail = smem_raw + (bar_acc + 8 - stages);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail);
    volatile int* gave_up = reinterpret_cast<volatile int*>(tail + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t ranks;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
    const uint32_t rank = cluster_rank();
    const uint32_t tile = blockIdx.x / ranks, tn = tile % p.tiles_n, tm = tile / p.tiles_n;
    constexpr int kFeatures = GLU ? 64 : 128;
    const int64_t n0 = (int64_t)tn * kFeatures, m0 = (int64_t)tm * NB;
    const uint32_t kb0 = (uint32_t)((uint64_t)p.k_blocks * rank / ranks),
                   kb1 = (uint32_t)((uint64_t)p.k_blocks * (rank + 1) / ranks);

    // One lane makes the barriers and starts the first copies before the block has met.
    const uint32_t kb_first = kb1 - kb0 < S::kStages ? kb1 : kb0 + S::kStages;   // end of the ring's first round
    const auto send = [&](uint32_t s, uint32_t kb) {
        const int k = (int)kb * p.k_elems;
        const uint32_t sw = stages + s * S::kStageBytes, full = bar_full + 8 * s;
        mbar_expect(full, S::kStageBytes);
        tma_load_2d<false>(sw, &p.w[0], k, (int)n0, full);
        if constexpr (GLU) tma_load_2d<false>(sw + S::kBytesW / 2, &p.w[1], k, (int)n0, full);
        tma_load_2d<false>(sw + S::kBytesW, &p.x, k, (int)m0, full);
    };
    if (warp == 0 && elect_one()) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(bar_full + 8 * i, 1);
            mbar_init(bar_empty + 8 * i, 1);
        }
        mbar_init(bar_acc, 1);
        *gave_up = 0;
        mbar_init_fence();
        wait_for_predecessor();
        for (uint32_t kb = kb0; kb < kb_first; ++kb) send(kb - kb0, kb);
    }
    if (warp == 1) tmem_alloc<false>(smem_addr(tmem_slot), S::kTmemCols);
    wait_for_predecessor();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        if (elect_one()) {
            Ring<S::kStages> ring;   // round 1 on: a stage is sent again once its products are done
            uint32_t sent = kb_first - kb0;
            for (uint32_t kb = kb_first; kb < kb1; ++kb, ++sent) {
                if (!mbar_wait(bar_empty + 8 * ring.s, ring.parity, gave_up)) break;
                send(ring.s, kb);
                ring.next();
            }
            bool landed = true;   // the ring is not used again before the copies have landed
            last_copies<S::kStages>(sent, [&](uint32_t s, uint32_t parity) { landed = landed && mbar_wait_alone(bar_full + 8 * s, parity); });
        }
    } else if (warp == 1) {
        if (elect_one()) {
            const uint32_t lo_w = desc_lo(stages, true), lo_x = desc_lo(stages + S::kBytesW, true), idesc = p.idesc;
            Ring<S::kStages> ring;
            uint32_t add = 0;
            for (uint32_t kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait(bar_full + 8 * ring.s, ring.parity, gave_up)) break;
                tc_fence_after();
                const uint32_t w = lo_w + ring.s * (S::kStageBytes >> 4), x = lo_x + ring.s * (S::kStageBytes >> 4);
#pragma unroll
                for (uint32_t i = 0; i < 4; ++i) {
                    if (p.e4m3) mma<false, true>(tmem, w + i * k_step(true), kDescHi, x + i * k_step(true), kDescHi, idesc, add);
                    else mma<false, false>(tmem, w + i * k_step(true), kDescHi, x + i * k_step(true), kDescHi, idesc, add);
                    add = 1;
                }
                mma_commit<false>(bar_empty + 8 * ring.s);
                ring.next();
            }
            mma_commit<false>(bar_acc);   // every product so far, also after giving up
            if (!mbar_wait_alone(bar_acc, 0)) *gave_up = 1;
        }
    }
    __syncwarp();
    mbar_wait(bar_acc, 0, gave_up);
    __syncthreads();   // copies and products are done; the ring is free for the partial sums
    tc_fence_after();
    // partial[row][feature]: 128 features a row
    if (warp < 4) {
        const uint32_t d = tmem + ((uint32_t)(warp * 32) << 16);
#pragma unroll
        for (int c = 0; c < NB; c += 16) {
            uint32_t raw[16];
            tmem_ld16(d + c, raw);
            tmem_ld_wait(raw);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float v = kb1 > kb0 ? __uint_as_float(raw[j]) : 0.0f;   // a rank without k adds nothing
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(stages + (uint32_t)(((c + j) * 128 + warp * 32 + lane) * 4)),
                             "f"(v)
                             : "memory");
            }
        }
    }
    cluster_sync();
    const int rows = p.m - m0 < NB ? (int)(p.m - m0) : NB;
    const int left = p.n - n0 < kFeatures ? (int)(p.n - n0) : kFeatures;
    uint32_t peer[8];
#pragma unroll
    for (uint32_t r = 0; r < 8; ++r) peer[r] = map_rank(stages, r < ranks ? r : 0);
    // four features of a row a thread, or one where that gives every thread at most one
    const int width = rows * kFeatures <= (int)(ranks * kRowsThreads) ? 1 : 4;
    for (int i = (int)(rank * kRowsThreads + threadIdx.x); i < rows * (kFeatures / width); i += (int)(ranks * kRowsThreads)) {
        const int r = i / (kFeatures / width), f = i % (kFeatures / width) * width;
        if (f >= left) continue;
        const int64_t row = m0 + r;
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f}, u[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (uint32_t q = 0; q < 8; ++q) {
            if (q >= ranks) break;
            if (width == 1) {
                v[0] += ld_cluster_f32(peer[q] + (uint32_t)((r * 128 + f) * 4));
                if constexpr (GLU) u[0] += ld_cluster_f32(peer[q] + (uint32_t)((r * 128 + 64 + f) * 4));
                continue;
            }
            const float4 a = ld_cluster_f32x4(peer[q] + (uint32_t)((r * 128 + f) * 4));
            v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
            if constexpr (GLU) {
                const float4 b = ld_cluster_f32x4(peer[q] + (uint32_t)((r * 128 + 64 + f) * 4));
                u[0] += b.x, u[1] += b.y, u[2] += b.z, u[3] += b.w;
            }
        }
        const float xs = p.x_scale ? p.x_scale[row] : 1.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (e >= width || f + e >= left) break;
            const int64_t col = n0 + f + e;
            float o = v[e];
            if (p.e4m3) {
                o *= xs * (p.w_scale[0] ? p.w_scale[0][col] : 1.0f);
                if constexpr (GLU) u[e] *= xs * (p.w_scale[1] ? p.w_scale[1][col] : 1.0f);
            }
            if (!GLU && p.bias) o += load_elem(p.bias, col, p.bias_type);
            if (p.z) {
                store_elem(p.z, row * p.ldz + col, p.z_type, o);
                if constexpr (GLU) store_elem(p.z2, row * p.ldz2 + col, p.z_type, u[e]);
            }
            o = act_value(o, p.act, p.out_type == GS_F32);
            if constexpr (GLU) o *= u[e];
            else if (p.residual) o += load_elem(p.residual, row * p.ldr + col, p.out_type);
            v[e] = o;
        }
        const int64_t at = row * p.ldy + n0 + f;
        if (width == 4 && f + 4 <= left && p.out_type != GS_F32 && ((uintptr_t)((uint16_t*)p.y + at) & 7u) == 0)
            *reinterpret_cast<uint2*>((uint16_t*)p.y + at) =
                make_uint2(pack_half2(v[0], v[1], p.out_type), pack_half2(v[2], v[3], p.out_type));
        else
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < width && f + e < left) store_elem(p.y, at + e, p.out_type, v[e]);
    }
    if (threadIdx.x == 0 && *gave_up) atomicExch(&g_wait_expired, 1);
    tc_fence_before();
    cluster_sync();   // the peers have read this CTA's sums
    if (warp == 1) {
        tc_fence_after();
        tmem_free<false>(tmem, S::kTmemCols);
    }
}

// ------------------------------------------------------------------ host
// Tile shapes: B's columns and whether two SMs share a tile.
struct Tile {
    int bn;
    bool pair;
    double per_kb;   // cycles a k-block (128 bytes of k) takes
    double per_clk;  // bytes a cycle its epilogue moves
    double values;   // its epilogue's arithmetic, relative
};
// A k-block of the three smaller tiles takes 350 to 420 cycles against 128, 256 and 256 of
// products, whatever its bytes (one factor alone: the same), its MMAs (one of four: 330) or
// the ring's depth; the wide pair's 520 against 512.  So that alone keeps the tensor cores fed.
// These rates and the cycles below are fitted to the times of all four shapes at 62
// sizes (500 to 1,000,000 rows, k 32 to 4096, plain, with activation, gated, 8 bits,
// gradients): the choice is within 10 % of the best shape (100,000 x 256 -> 1024: 61 us
// with the narrow pair, 55 with the wide one; gated 100,000 x 256 -> 512: 55, 47).
constexpr Tile kTiles[4] = {{64, false, 480, 22.5, 0.92}, {128, false, 560, 22, 0.95}, {128, true, 550, 19, 0.89}, {256, true, 800, 19.3, 1.15}};

// Cycles of a call with a tile shape: waves of tiles, each bound by its k-blocks or by
// its epilogue's arithmetic and traffic, and a start-up.
double cost(const GemmCall& c, const Tile& t, int sms, GemmPlan* out)
{
    GemmPlan& p = *out;
    const bool glu = c.kind == GemmKind::kGlu || c.kind == GemmKind::kGluGrad;
    p.pair = t.pair;
    p.bn = t.bn;
    p.tile_m = t.pair ? 256 : 128;
    p.out_cols = glu ? t.bn / 2 : t.bn;
    p.tiles_m = (c.m + p.tile_m - 1) / p.tile_m;
    p.tiles_n = (c.n + p.out_cols - 1) / p.out_cols;
    p.esz = type_bytes(c.type);
    p.k_elems = kStageRow / p.esz;
    p.k_blocks = (c.k + p.k_elems - 1) / p.k_elems;
    p.terms = c.kind == GemmKind::kSum ? 2 : 1;
    p.probs = c.kind == GemmKind::kTwo ? 2 : 1;
    const int64_t tiles = p.tiles_m * p.tiles_n * p.probs, slots = t.pair ? sms / 2 : sms, kb = p.k_blocks * p.terms;
    // Few tiles: split k over the idle SMs, at least four k-blocks each, where nothing
    // but the sum is asked for (the gradients): the partial sums are joined in order.
    const bool sum_only = !glu && !c.bias && !c.residual && !c.z && c.act == GS_ACT_NONE &&
                          !c.x_scale && !c.w_scale[0];
    const double live = (double)(c.n < p.out_cols ? c.n : p.out_cols);
    // the weights' gradients: a plan, and so an order, that does not depend on the type they are rounded to
    const int bytes = (c.a[0].k_fast ? type_bytes(c.out_type) : 4) * (c.residual ? 2 : 1) + (c.z ? (glu ? 4 : 2) : 0);
    const double per_value = t.values * (glu ? 0.048 : (c.act != GS_ACT_NONE ? 0.185 : (c.type == GS_E4M3 ? 0.048 : 0.0)));
    double best = 0;
    int64_t most = sum_only ? slots / tiles : 1;
    if (most > kb / 4) most = kb / 4;
    if (most < 1) most = 1;
    for (int64_t s = 1; s <= most; s = s == most ? most + 1 : (s + s / 2 + 1 < most ? s + s / 2 + 1 : most)) {
        const double main = t.per_kb * (double)((kb + s - 1) / s);
        const double epi = 390 + 128.0 * live * (per_value + (s > 1 ? 4 : bytes) / t.per_clk);
        const double waves = (double)((tiles * s + slots - 1) / slots);
        // the join: a launch, and every partial sum read once at about 20 bytes a cycle and SM
        const double join = s > 1 ? 4500 + (double)s * c.m * c.n * p.probs * 4 / (sms * 20.0) : 0;
        const double v = 6400 + waves * (main > epi ? main : epi) + (main > epi ? epi : main) + join;
        if (s == 1 || v < best) {
            best = v;
            p.splits = (int)s;
        }
    }
    p.units = tiles * p.splits;
    return best;
}

int64_t stored_rows(const GemmFactor& f, int64_t rows, int64_t k) { return f.k_fast ? rows : k; }
int64_t stored_cols(const GemmFactor& f, int64_t rows, int64_t k) { return f.k_fast ? k : rows; }

template <int NB, bool GLU>
gs_status launch_rows(const RowsParams& p, unsigned grid, int ranks, cudaStream_t st)
{
    using S = RowsShape<NB, GLU>;
    static_assert(S::kSmem <= 232448, "shared memory of an SM");
    auto* kernel = rows_kernel<NB, GLU>;
    static std::atomic<uint64_t> done{0};
    const gs_status s = allow_smem(kernel, S::kSmem, done);
    if (s != GS_OK) return s;
    return launch_after(kernel, dim3(grid), kRowsThreads, S::kSmem, (unsigned)ranks, st, p);
}

template <int BN, bool PAIR, bool GLU, int OSZ, bool GRAD = false>
gs_status launch(const Params& p, int grid, cudaStream_t st)
{
    using S = Shape<BN, PAIR, GLU>;
    static_assert(S::kSmem <= 232448, "shared memory of an SM");
    auto* kernel = gemm_kernel<BN, PAIR, GLU, OSZ, GRAD>;
    static std::atomic<uint64_t> done{0};
    const gs_status s = allow_smem(kernel, S::kSmem, done);
    if (s != GS_OK) return s;
    return launch_after(kernel, dim3((unsigned)grid), kThreads, S::kSmem, PAIR ? 2 : 1, st, p);
}

}  // namespace

// Read once a device: the count does not change while a process runs.
int device_sms()
{
    static std::atomic<int> known[64];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev < 64 && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

namespace tc {

static gs_status encode_map(CUtensorMap* map, const void* p, int type, int dims, const cuuint64_t* size, const cuuint64_t* pitch,
                            const cuuint32_t* box)
{
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return (Encode)f;
    }();
    if (!encode) return GS_ERR_CUDA;
    const CUtensorMapDataType dt = type == GS_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : type == GS_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                   : type == GS_F16  ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                     : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const cuuint32_t unit[3] = {1, 1, 1};
    const CUresult r = encode(map, dt, (cuuint32_t)dims, const_cast<void*>(p), size, pitch, box, unit,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? GS_OK : GS_ERR_CUDA;
}

gs_status make_map(CUtensorMap* map, const void* p, int type, int64_t rows, int64_t cols, int64_t ld, int box_rows,
                   int box_cols)
{
    const cuuint64_t size[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t pitch[1] = {(cuuint64_t)(ld * type_bytes(type))};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    return encode_map(map, p, type, 2, size, pitch, box);
}

gs_status make_map3(CUtensorMap* map, const void* p, int type, const int64_t (&size)[3], const int64_t (&pitch)[2],
                    const int (&box)[3])
{
    const int64_t e = type_bytes(type);
    const cuuint64_t sizes[3] = {(cuuint64_t)size[0], (cuuint64_t)size[1], (cuuint64_t)size[2]};
    const cuuint64_t pitches[2] = {(cuuint64_t)(pitch[0] * e), (cuuint64_t)(pitch[1] * e)};
    const cuuint32_t boxes[3] = {(cuuint32_t)box[0], (cuuint32_t)box[1], (cuuint32_t)box[2]};
    return encode_map(map, p, type, 3, sizes, pitches, boxes);
}

}  // namespace tc

static thread_local int t_tile = -1;   // gs_layer_tile

GemmPlan gemm_plan(const GemmCall& c)
{
    const int known = device_sms(), sms = known > 0 ? known : 152;
    GemmPlan best, p;
    double at = 0;
    const bool glu = c.kind == GemmKind::kGlu || c.kind == GemmKind::kGluGrad;
    const bool forced = t_tile >= (glu ? 1 : 0);
    const int first = forced ? t_tile : (glu ? 1 : 0), last = forced ? t_tile : 3;
    for (int i = first; i <= last; ++i) {
        const double v = cost(c, kTiles[i], sms, &p);
        if (i == first || v < at) {
            at = v;
            best = p;
        }
    }
    p = best;
    p.sms = sms;
    p.nb = 0;
    if (!forced && (c.kind == GemmKind::kLinear || c.kind == GemmKind::kGlu) && c.a[0].k_fast && c.b[0].k_fast && c.m <= kFewRows) {
        p.nb = c.m <= 16 ? 16 : (c.m <= 32 ? 32 : 64);
        const int64_t tiles = ((c.n + (glu ? 63 : 127)) / (glu ? 64 : 128)) * ((c.m + p.nb - 1) / p.nb);
        p.ranks = 1;
        while (p.ranks < 8 && tiles * p.ranks * 2 <= sms && p.k_blocks >= 2 * p.ranks) p.ranks *= 2;
        p.splits = 1;
    }
    p.pitch = round_up(c.n, 4);
    p.bytes = p.splits > 1 ? (size_t)round_up((int64_t)p.splits * p.probs * c.m * p.pitch * 4, 256) : 0;
    return p;
}

// The epilogue waits for a whole unit's contraction under kWaitCycles (4e9 cycles), and a
// k-block takes at most about 1500 cycles (the wide pair's 64 KB with all SMs on HBM).
constexpr int64_t kMostKBlocks = 1 << 21;

bool gemm_fits(const GemmPlan& p)
{
    const int64_t parts = p.nb ? p.ranks : p.splits;
    return p.k_blocks * p.terms <= kMostKBlocks * (parts > 0 ? parts : 1);
}

gs_status gemm_run(const GemmCall& c, const GemmPlan& plan, void* ws, JoinJobs* joins, cudaStream_t st)
{
    if (plan.units > 0x7fffffffll || c.m > 0x7fffff00ll || c.n > 0x7fffff00ll || c.k > 0x7fffff00ll)
        return GS_ERR_INVALID_ARG;
    const GemmFactor f[4] = {c.a[0], c.a[1], c.b[0], c.b[1]};
    const bool glu = c.kind == GemmKind::kGlu || c.kind == GemmKind::kGluGrad;
    if (plan.nb) {
        RowsParams r = {};
        gs_status s = tc::make_map(&r.x, f[0].p, c.type, c.m, c.k, f[0].ld, plan.nb, plan.k_elems);
        if (s == GS_OK) s = tc::make_map(&r.w[0], f[2].p, c.type, c.n, c.k, f[2].ld, glu ? 64 : 128, plan.k_elems);
        if (s == GS_OK && glu) s = tc::make_map(&r.w[1], f[3].p, c.type, c.n, c.k, f[3].ld, 64, plan.k_elems);
        if (s != GS_OK) return s;
        r.m = c.m, r.n = c.n;
        r.x_scale = c.x_scale, r.w_scale[0] = c.w_scale[0], r.w_scale[1] = c.w_scale[1];
        r.bias = c.bias, r.bias_type = c.bias_type, r.act = c.act;
        r.residual = c.residual, r.ldr = c.ldr;
        r.y = c.y, r.ldy = c.ldy, r.out_type = c.out_type;
        r.z = c.z, r.ldz = c.ldz, r.z2 = c.z2, r.ldz2 = c.ldz2, r.z_type = c.z_type;
        r.k_blocks = (uint32_t)plan.k_blocks, r.k_elems = plan.k_elems, r.e4m3 = c.type == GS_E4M3;
        const int64_t tiles_n = (c.n + (glu ? 63 : 127)) / (glu ? 64 : 128), tiles_m = (c.m + plan.nb - 1) / plan.nb;
        if (tiles_n * tiles_m * plan.ranks > 0x7fffffffll) return GS_ERR_INVALID_ARG;
        r.tiles_n = (uint32_t)tiles_n;
        r.idesc = tc::instr_desc(c.type, true, true, plan.nb, 128);
        const unsigned grid = (unsigned)(tiles_n * tiles_m * plan.ranks);
        if (glu)
            return plan.nb == 16   ? launch_rows<16, true>(r, grid, plan.ranks, st)
                   : plan.nb == 32 ? launch_rows<32, true>(r, grid, plan.ranks, st)
                                   : launch_rows<64, true>(r, grid, plan.ranks, st);
        return plan.nb == 16   ? launch_rows<16, false>(r, grid, plan.ranks, st)
               : plan.nb == 32 ? launch_rows<32, false>(r, grid, plan.ranks, st)
                               : launch_rows<64, false>(r, grid, plan.ranks, st);
    }

    Params p = {};
    const int rows_b = plan.pair || glu ? plan.bn / 2 : plan.bn;
    for (int i = 0; i < 4; ++i) {
        if (!f[i].p) continue;
        const int64_t rows = i < 2 ? c.m : c.n;
        CUtensorMap* map = i < 2 ? &p.a[i] : &p.b[i - 2];
        const gs_status s = tc::make_map(map, f[i].p, c.type, stored_rows(f[i], rows, c.k), stored_cols(f[i], rows, c.k),
                                         f[i].ld, f[i].k_fast ? (i < 2 ? kRowsA : rows_b) : 64,
                                         f[i].k_fast ? plan.k_elems : 64);
        if (s != GS_OK) return s;
    }
    p.partial = plan.splits > 1;
    const int out_type = p.partial ? GS_F32 : c.out_type;
    void* y[2] = {c.y, c.y2};
    const int64_t ldy[2] = {c.ldy, c.ldy2};
    if (p.partial) {
        p.yp[0] = ws;
        p.ldy[0] = plan.pitch;
        p.part = c.m * plan.pitch;
        p.y_vec = 1;
    } else {
        for (int i = 0; i < 2; ++i) p.yp[i] = y[i], p.ldy[i] = ldy[i];
        p.y_vec = rows16(c.y, c.ldy, c.out_type) && (plan.probs == 1 || rows16(c.y2, c.ldy2, c.out_type));
        if (c.residual) {
            p.residual = c.residual;
            p.ldr = c.ldr;
            p.r_vec = rows16(c.residual, c.ldr, c.out_type);
        }
        if (c.z) {
            p.zp = c.z, p.ldz = c.ldz, p.z2p = c.z2, p.ldz2 = c.ldz2;
            p.z_vec = rows16(c.z, c.ldz, c.z_type) && (!glu || rows16(c.z2, c.ldz2, c.z_type));
        }
        p.x_scale = c.x_scale;
        p.w_scale[0] = c.w_scale[0], p.w_scale[1] = c.w_scale[1];
        p.bias = c.bias, p.bias_type = c.bias_type, p.act = c.act;
    }
    p.m = c.m, p.n = c.n;
    p.out_type = out_type, p.z_type = c.z_type;
    p.k_blocks = (uint32_t)plan.k_blocks, p.tiles_m = (uint32_t)plan.tiles_m, p.tiles_n = (uint32_t)plan.tiles_n;
    p.units = (uint32_t)plan.units;
    p.splits = plan.splits, p.terms = plan.terms, p.probs = plan.probs, p.k_elems = plan.k_elems;
    p.a_fast = c.a[0].k_fast, p.b_fast = c.b[0].k_fast;
    p.e4m3 = c.type == GS_E4M3;
    p.idesc = tc::instr_desc(c.type, c.a[0].k_fast, c.b[0].k_fast, plan.bn, (int)plan.tile_m);
    const int64_t most = plan.pair ? plan.sms / 2 : plan.sms;
    const int grid = (int)(plan.units < most ? plan.units : most) * (plan.pair ? 2 : 1);
    gs_status s;
    const auto pick = [&](auto osz) {
        constexpr int OSZ = decltype(osz)::value;
        if (plan.pair) return plan.bn == 256 ? launch<256, true, false, OSZ>(p, grid, st) : launch<128, true, false, OSZ>(p, grid, st);
        return plan.bn == 128 ? launch<128, false, false, OSZ>(p, grid, st) : launch<64, false, false, OSZ>(p, grid, st);
    };
    if (c.kind == GemmKind::kGluGrad)
        s = !plan.pair         ? launch<128, false, true, 2, true>(p, grid, st)
            : plan.bn == 256 ? launch<256, true, true, 2, true>(p, grid, st)
                             : launch<128, true, true, 2, true>(p, grid, st);
    else if (glu)
        s = !plan.pair         ? launch<128, false, true, 2>(p, grid, st)
            : plan.bn == 256 ? launch<256, true, true, 2>(p, grid, st)
                             : launch<128, true, true, 2>(p, grid, st);
    else if (out_type == GS_F32) s = pick(std::integral_constant<int, 4>());
    else s = pick(std::integral_constant<int, 2>());
    if (s != GS_OK || !p.partial) return s;
    const float* partial = (const float*)ws;
    for (int i = 0; i < plan.probs; ++i) {
        s = joins->add(partial + (int64_t)i * plan.splits * c.m * plan.pitch, plan.splits, c.m, c.n, plan.pitch, y[i], ldy[i],
                       c.out_type);
        if (s != GS_OK) return s;
    }
    return GS_OK;
}

}  // namespace gs

using namespace gs;

extern "C" gs_status gs_layer_tile(int32_t tile)
{
    GS_NVTX_RANGE("gs_layer_tile");
    if (tile < -1 || tile > 3) return GS_ERR_INVALID_ARG;
    t_tile = tile;
    return GS_OK;
}

extern "C" gs_status gs_wait_report(int32_t* expired)
{
    GS_NVTX_RANGE("gs_wait_report");
    if (!expired) return GS_ERR_INVALID_ARG;
    *expired = 0;
    int v = 0;
    const int zero = 0;
    GS_CUDA_TRY(cudaDeviceSynchronize());
    GS_CUDA_TRY(cudaMemcpyFromSymbol(&v, g_wait_expired, sizeof v));
    if (v) GS_CUDA_TRY(cudaMemcpyToSymbol(g_wait_expired, &zero, sizeof zero));
    for (gs_status (*report)(int*) : {glu_narrow_wait_report, attn::forward_wait_report, attn::backward_wait_report}) {
        int other = 0;
        const gs_status s = report(&other);
        if (s != GS_OK) return s;
        v |= other;
    }
    *expired = v;
    return v ? GS_ERR_TIMEOUT : GS_OK;
}
