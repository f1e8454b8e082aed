// gemm.cu -- the matrix product behind the decoder layers on the tensor cores.
//
//   D[m][n] = sum_k A[m][k] B[n][k], fp32 accumulators, epilogue on the way out
//
// One persistent CTA an SM (or a pair of CTAs on two SMs), 10 warps with fixed roles:
//   warp 0      TMA producer: tiles of A and B into a ring of 128-byte-swizzled stages
//   warp 1      issues tcgen05.mma into one of two TMEM accumulators
//   warps 2-9   epilogue: accumulator -> registers -> scale, bias, activation, gate,
//               residual -> shared memory -> TMA store, while the next tile accumulates
// Either factor may have k as its fast or its slow index (the gradients contract over
// rows and over output features), so no operand is ever transposed in memory.
//
// What bounds it: with large k the tensor cores; a CTA's 128 x 128 tile takes
// 2 x 16 KB from shared memory per 64 k for 128 x 128 x 64 products, as much as
// shared memory delivers, so wide problems use the pair: 256 x 256 over two SMs, each
// holding half of B, half the shared-memory bytes a product.  With small k (a
// Gaussian decoder's layers) HBM, through the epilogue's stores.
#include "gemm.cuh"
#include "tc_common.cuh"

namespace gs {
namespace {

using namespace tc;

constexpr int kWarps = 10;
constexpr int kThreads = kWarps * 32;
constexpr int kEpiWarps = 8;
constexpr int kRowsA = 128;                      // accumulator rows of a CTA
constexpr int kStageRow = 128;                   // bytes of k a stage holds per row
constexpr int kSlotBytes = 8192;                 // staging of one epilogue warp
constexpr int kChunk = 32;                       // columns an epilogue warp handles at a time
constexpr int kGroupM = 8;                       // m-tiles that run together (L2 reuse of B)

struct Params {
    CUtensorMap a[2], b[2], y[2], r, z, z2;
    int64_t m, n;
    const float* x_scale;
    const float* w_scale[2];
    const void* bias;
    const void* residual;
    void* yp[2];
    void* zp;
    void* z2p;
    int64_t ldr, ldy[2], ldz, ldz2;
    int64_t k_blocks;         // of one term
    int64_t tiles_m, tiles_n, units;
    int splits, terms, probs; // k ranges; products summed; independent products
    int k_elems;              // k of a stage
    int a_fast, b_fast, e4m3;
    uint32_t idesc;
    int bias_type, out_type, z_type, act;
    int y_tma, r_tma, z_tma, partial;
};

__device__ int g_wait_expired;

template <int BN, bool PAIR>
struct Shape {
    static constexpr int kTileM = PAIR ? 256 : 128;
    static constexpr int kRowsB = PAIR ? BN / 2 : BN;                  // rows of B a CTA holds
    static constexpr int kBytesA = kRowsA * kStageRow;
    static constexpr int kBytesB = kRowsB * kStageRow;
    static constexpr int kStageBytes = kBytesA + kBytesB;
    static constexpr int kStages = BN == 64 ? 6 : 5;
    static constexpr int kTmemCols = 2 * BN;
    static constexpr int kBars = kStages * 2 + 4 + kEpiWarps * 4 + 2;   // even: what follows is 16-byte aligned
    static constexpr int kSmem = kStages * kStageBytes + kEpiWarps * kSlotBytes + kBars * 8 + 16 +
                                 kEpiWarps * 2 * kChunk * 4;
};

struct Unit {
    int prob, split;
    int64_t tm, tn, kb0, kb1;
};

__device__ __forceinline__ Unit decode(const Params& p, int64_t u)
{
    Unit r;
    const int64_t tiles = p.tiles_m * p.tiles_n, per_split = tiles * p.probs;
    r.split = (int)(u / per_split);
    const int64_t rest = u % per_split;
    r.prob = (int)(rest % p.probs);
    const int64_t t = rest / p.probs;
    const int64_t per_group = kGroupM * p.tiles_n, first = t / per_group * kGroupM, in = t % per_group;
    const int64_t rows = p.tiles_m - first < kGroupM ? p.tiles_m - first : kGroupM;
    r.tm = first + in % rows;
    r.tn = in / rows;
    const int64_t kb = p.k_blocks * p.terms;
    r.kb0 = kb * r.split / p.splits;
    r.kb1 = kb * (r.split + 1) / p.splits;
    return r;
}

// Byte of 16-byte piece j of row r in a staging slot: 64-byte rows under the 64-byte
// swizzle (16-bit elements), 128-byte rows under the 128-byte swizzle (32-bit ones).
template <int ESZ>
__device__ __forceinline__ uint32_t slot_piece(int r, int j)
{
    return ESZ == 2 ? r * 64 + ((j ^ ((r >> 1) & 3)) << 4) : r * 128 + ((j ^ (r & 7)) << 4);
}
// Byte of element c of row r.
template <int ESZ>
__device__ __forceinline__ uint32_t slot_elem(int r, int c)
{
    return slot_piece<ESZ>(r, c * ESZ >> 4) + ((c * ESZ) & 15);
}

__device__ __forceinline__ void st_shared16(uint32_t a, uint4 v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

// A row's 32 values into a slot, rounded to the output's type, and a slot's row added.
template <int T>
__device__ __forceinline__ void slot_write_half(uint32_t slot, int row, const float (&v)[kChunk])
{
#pragma unroll
    for (int j = 0; j < 4; ++j)
        st_shared16(slot + slot_piece<2>(row, j),
                    make_uint4(pack_half2(v[8 * j], v[8 * j + 1], T), pack_half2(v[8 * j + 2], v[8 * j + 3], T),
                               pack_half2(v[8 * j + 4], v[8 * j + 5], T), pack_half2(v[8 * j + 6], v[8 * j + 7], T)));
}
template <int T>
__device__ __forceinline__ void slot_add_half(uint32_t slot, int row, float (&v)[kChunk])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint4 q = ld_shared16(slot + slot_piece<2>(row, j));
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack_half2(w[i], T);
            v[8 * j + 2 * i] += f.x;
            v[8 * j + 2 * i + 1] += f.y;
        }
    }
}
template <int ESZ>
__device__ __forceinline__ void slot_write(uint32_t slot, int row, const float (&v)[kChunk], int type)
{
    if constexpr (ESZ == 2) {
        if (type == GS_BF16) slot_write_half<GS_BF16>(slot, row, v);
        else slot_write_half<GS_F16>(slot, row, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            st_shared16(slot + slot_piece<4>(row, j),
                        make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                                   __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3])));
    }
}
template <int ESZ>
__device__ __forceinline__ void slot_add(uint32_t slot, int row, float (&v)[kChunk], int type)
{
    if constexpr (ESZ == 2) {
        if (type == GS_BF16) slot_add_half<GS_BF16>(slot, row, v);
        else slot_add_half<GS_F16>(slot, row, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint4 q = ld_shared16(slot + slot_piece<4>(row, j));
            v[4 * j] += __uint_as_float(q.x);
            v[4 * j + 1] += __uint_as_float(q.y);
            v[4 * j + 2] += __uint_as_float(q.z);
            v[4 * j + 3] += __uint_as_float(q.w);
        }
    }
}

// Rows of any alignment: the warp moves a chunk between a slot and memory, one row
// of consecutive columns at a time.
template <int ESZ>
__device__ __forceinline__ void slot_to_rows(uint32_t slot, void* p, int64_t ld, int64_t row0, int64_t col0, int64_t m,
                                             int64_t n, int lane)
{
    const int64_t col = col0 + lane;
    if (col >= n) return;
    const int rows = m - row0 < 32 ? (int)(m - row0) : 32;
    for (int r = 0; r < rows; ++r) {
        const uint32_t a = slot + slot_elem<ESZ>(r, lane);
        if constexpr (ESZ == 2) {
            uint16_t v;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
            ((uint16_t*)p)[(row0 + r) * ld + col] = v;
        } else {
            uint32_t v;
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
            ((uint32_t*)p)[(row0 + r) * ld + col] = v;
        }
    }
}
template <int ESZ>
__device__ __forceinline__ void rows_to_slot(uint32_t slot, const void* p, int64_t ld, int64_t row0, int64_t col0,
                                             int64_t m, int64_t n, int lane)
{
    const int64_t col = col0 + lane;
#pragma unroll 8
    for (int r = 0; r < 32; ++r) {
        const uint32_t a = slot + slot_elem<ESZ>(r, lane);
        const bool live = col < n && row0 + r < m;
        if constexpr (ESZ == 2) {
            const uint16_t v = live ? ((const uint16_t*)p)[(row0 + r) * ld + col] : (uint16_t)0;
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"(v) : "memory");
        } else {
            const uint32_t v = live ? ((const uint32_t*)p)[(row0 + r) * ld + col] : 0u;
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
        }
    }
}

// GLU: B's rows are half gate, half up; the epilogue joins column c with c + BN/2.
// OSZ: bytes of an output element.
template <int BN, bool PAIR, bool GLU, int OSZ>
__global__ void __launch_bounds__(kThreads, 1) gemm_kernel(const __grid_constant__ Params p)
{
    using S = Shape<BN, PAIR>;
    extern __shared__ __align__(1024) char smem_raw[];   // the swizzle patterns repeat every 1024 bytes
    const uint32_t base = smem_addr(smem_raw);
    if (base & 1023u) {   // every thread sees the same address; there is no padding to move within
        g_wait_expired = 1;
        return;
    }
    const uint32_t stages = base, slots = base + S::kStages * S::kStageBytes;
    const uint32_t bars = slots + kEpiWarps * kSlotBytes;
    const uint32_t bar_full = bars, bar_empty = bars + S::kStages * 8, bar_acc = bar_empty + S::kStages * 8,
                   bar_free = bar_acc + 16, bar_res = bar_free + 16, bar_drain = bar_res + kEpiWarps * 32;
    char* tail = smem_raw + (bars + S::kBars * 8 - base);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail);
    volatile int* gave_up = reinterpret_cast<volatile int*>(tail + 4);
    float* columns = reinterpret_cast<float*>(tail + 16);   // [warp][2][chunk]: scale, bias (or the second scale)

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_rank() : 0;
    const int64_t first = PAIR ? blockIdx.x >> 1 : blockIdx.x, step = PAIR ? gridDim.x >> 1 : gridDim.x;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(bar_full + 8 * i, 1);
            mbar_init(bar_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_acc + 8 * i, 1);
            mbar_init(bar_free + 8 * i, kEpiWarps * (PAIR ? 2 : 1));
        }
        for (int i = 0; i < kEpiWarps * 4; ++i) mbar_init(bar_res + 8 * i, 1);
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

    if (warp == 0) {
        if (lane == 0) {
            // ---------------------------------------------------------- producer
            prefetch_map(&p.a[0]);
            prefetch_map(&p.b[0]);
            const uint32_t full0 = PAIR ? map_rank(bar_full, 0) : bar_full;   // the pair counts at its first CTA
            uint32_t it = 0;
            bool ok = true;
            for (int64_t u = first; u < p.units && ok; u += step) {
                const Unit q = decode(p, u);
                const int row_a = (int)(q.tm * S::kTileM + rank * kRowsA);
                const int row_b = GLU ? (int)(q.tn * (BN / 2)) : (int)(q.tn * BN + rank * S::kRowsB);
                for (int64_t kb = q.kb0; kb < q.kb1; ++kb, ++it) {
                    const int s = it % S::kStages;
                    if (!mbar_wait(bar_empty + 8 * s, ((it / S::kStages) & 1) ^ 1, gave_up)) {
                        ok = false;
                        break;
                    }
                    const int term = kb >= p.k_blocks ? 1 : 0;
                    const int k = (int)((kb - term * p.k_blocks) * p.k_elems);
                    const int which = p.probs > 1 ? q.prob : term;
                    if (rank == 0) mbar_expect(bar_full + 8 * s, S::kStageBytes * (PAIR ? 2 : 1));
                    const uint32_t full = full0 + 8 * s, sa = stages + s * S::kStageBytes, sb = sa + S::kBytesA;
                    if (p.a_fast) tma_load_2d<PAIR>(sa, &p.a[which], k, row_a, full);
                    else
#pragma unroll
                        for (int i = 0; i < kRowsA / 64; ++i)
                            tma_load_2d<PAIR>(sa + i * 8192, &p.a[which], row_a + 64 * i, k, full);
                    if constexpr (GLU) {
                        if constexpr (PAIR) tma_load_2d<PAIR>(sb, &p.b[rank], k, row_b, full);
                        else {
                            tma_load_2d<PAIR>(sb, &p.b[0], k, row_b, full);
                            tma_load_2d<PAIR>(sb + S::kBytesB / 2, &p.b[1], k, row_b, full);
                        }
                    } else if (p.b_fast) tma_load_2d<PAIR>(sb, &p.b[which], k, row_b, full);
                    else
#pragma unroll
                        for (int i = 0; i < S::kRowsB / 64; ++i)
                            tma_load_2d<PAIR>(sb + i * 8192, &p.b[which], row_b + 64 * i, k, full);
                }
            }
            if (!ok && rank == 0) {   // given up: let the copies in flight land before the block leaves
                volatile int still = 0;
                const uint32_t from = it > S::kStages ? it - S::kStages : 0;
                for (uint32_t i = from; i < it; ++i)
                    mbar_wait(bar_full + 8 * (i % S::kStages), (i / S::kStages) & 1, &still);
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            // ---------------------------------------------------------- tensor cores
            const uint64_t desc_a = smem_desc(0, p.a_fast), desc_b = smem_desc(0, p.b_fast);
            const uint32_t step_a = k_step(p.a_fast), step_b = k_step(p.b_fast);
            uint32_t it = 0, tile = 0;
            bool ok = true;
            for (int64_t u = first; u < p.units && ok; u += step, ++tile) {
                const Unit q = decode(p, u);
                const uint32_t acc = tile & 1;
                if (!mbar_wait(bar_free + 8 * acc, ((tile >> 1) & 1) ^ 1, gave_up)) break;
                tc_fence_after();
                const uint32_t d = tmem + acc * BN;
                for (int64_t kb = q.kb0; kb < q.kb1; ++kb, ++it) {
                    const int s = it % S::kStages;
                    if (!mbar_wait(bar_full + 8 * s, (it / S::kStages) & 1, gave_up)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = stages + s * S::kStageBytes, sb = sa + S::kBytesA;
                    uint64_t da = desc_a | (sa >> 4), db = desc_b | (sb >> 4);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool add = kb > q.kb0 || i > 0;
                        if (p.e4m3) mma<PAIR, true>(d, da, db, p.idesc, add);
                        else mma<PAIR, false>(d, da, db, p.idesc, add);
                        da += step_a;
                        db += step_b;
                    }
                    mma_commit<PAIR>(bar_empty + 8 * s);   // the stage is free once these are done
                }
                if (ok) mma_commit<PAIR>(bar_acc + 8 * acc);
            }
            if (*gave_up) {
                volatile int still = 0;
                mma_commit<PAIR>(bar_drain);
                mbar_wait(bar_drain, 0, &still);
            }
        }
    } else {
        // -------------------------------------------------------------- epilogue
        const int ew = warp - 2, quarter = warp & 3, half = ew >> 2;
        constexpr int kOutCols = GLU ? BN / 2 : BN;
        constexpr int kChunks = kOutCols / 2 / kChunk > 0 ? kOutCols / 2 / kChunk : 1;
        static_assert(kChunks * kChunk * 2 == kOutCols, "two halves of whole chunks");
        const uint32_t slot = slots + ew * kSlotBytes;
        const uint32_t res = bar_res + ew * 32;
        const uint32_t free0 = PAIR ? map_rank(bar_free, 0) : bar_free;
        float* col_a = columns + ew * 2 * kChunk;
        float* col_b = col_a + kChunk;
        // staging: buffers of y and where the saved projections go
        const bool save = p.zp != nullptr;
        const int bufs = OSZ == 4 ? (save ? 1 : 2) : (GLU ? (save ? 1 : 4) : (save ? 2 : 4));
        const uint32_t buf_bytes = kChunk * 32 * OSZ;
        const uint32_t z_at = OSZ == 4 ? 4096 : (GLU ? 2048 : 4096);
        const bool has_res = !GLU && p.residual != nullptr;
        uint32_t chunk_no = 0, tile = 0;
        bool ok = true;
        for (int64_t u = first; u < p.units && ok; u += step, ++tile) {
            const Unit q = decode(p, u);
            const uint32_t acc = tile & 1;
            const int64_t row0 = q.tm * S::kTileM + rank * kRowsA + quarter * 32;
            const int64_t base_col = q.tn * kOutCols + half * (kOutCols / 2);
            const bool rows_live = row0 < p.m;
            const int chunks = !rows_live || base_col >= p.n
                                   ? 0
                                   : (int)((p.n - base_col + kChunk - 1) / kChunk < kChunks
                                               ? (p.n - base_col + kChunk - 1) / kChunk
                                               : kChunks);
            // residual chunks are fetched one ahead; the first before the accumulator is waited for
            auto fetch = [&](uint32_t no, int c) {
                const uint32_t b = no % bufs;
                if (lane == 0) {
                    mbar_expect(res + 8 * b, buf_bytes);
                    tma_load_2d<false>(slot + b * buf_bytes, &p.r, (int)(base_col + c * kChunk), (int)row0, res + 8 * b);
                }
            };
            if (has_res && p.r_tma && chunks > 0 && bufs > 1) {
                if (lane == 0) {   // the buffer's last store has been read
                    if (bufs == 2) bulk_wait_read<1>();
                    else bulk_wait_read<3>();
                }
                fetch(chunk_no, 0);
            }
            const float xs = p.x_scale && row0 + lane < p.m ? p.x_scale[row0 + lane] : 1.0f;
            // column factors of the warp's chunks, one a lane, fetched before the accumulator is waited for
            float ca[kChunks], cb[kChunks];
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const int64_t col = base_col + c * kChunk + lane;
                const bool live = c < chunks && col < p.n;
                ca[c] = p.w_scale[0] && live ? p.w_scale[0][col] : 1.0f;
                if constexpr (GLU) cb[c] = p.w_scale[1] && live ? p.w_scale[1][col] : 1.0f;
                else cb[c] = p.bias && live ? load_elem(p.bias, col, p.bias_type) : 0.0f;
            }
            if (!__all_sync(0xffffffffu, mbar_wait(bar_acc + 8 * acc, (tile >> 1) & 1, gave_up))) {
                ok = false;
                // a residual chunk may be in flight: let it land
                if (has_res && p.r_tma && chunks > 0 && bufs > 1) {
                    volatile int still = 0;
                    mbar_wait(res + 8 * (chunk_no % bufs), (chunk_no / bufs) & 1, &still);
                }
                break;
            }
            __syncwarp();
            tc_fence_after();
            const uint32_t d = tmem + ((uint32_t)(quarter * 32) << 16) + acc * BN + half * (kOutCols / 2);
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                if (c >= chunks) break;
                const int64_t col0 = base_col + c * kChunk;
                const uint32_t b = chunk_no % bufs, ys = slot + b * buf_bytes;
                const uint32_t zs = slot + z_at + (bufs == 2 ? b * 2048 : 0);
                uint32_t raw[kChunk], raw2[GLU ? kChunk : 1];
                tmem_ld32(d + c * kChunk, raw);
                if constexpr (GLU) tmem_ld32(d + BN / 2 + c * kChunk, raw2);
                if (p.e4m3 || p.bias) {
                    __syncwarp();   // the last chunk's readers are done
                    col_a[lane] = ca[c];
                    col_b[lane] = cb[c];
                }
                if (has_res && !p.r_tma) {
                    if (lane == 0) bulk_wait_read<0>();
                    __syncwarp();
                    rows_to_slot<OSZ>(ys, p.residual, p.ldr, row0, col0, p.m, p.n, lane);
                }
                if (has_res && p.r_tma) {
                    if (bufs == 1) {
                        if (lane == 0) bulk_wait_read<0>();
                        fetch(chunk_no, c);
                    } else if (c + 1 < chunks) {
                        if (lane == 0) {
                            if (bufs == 2) bulk_wait_read<0>();
                            else bulk_wait_read<2>();
                        }
                        fetch(chunk_no + 1, c + 1);
                    }
                } else if (lane == 0) {
                    if (bufs == 1) bulk_wait_read<0>();
                    else if (bufs == 2) bulk_wait_read<1>();
                    else bulk_wait_read<3>();
                }
                __syncwarp();
                float v[kChunk];
                tmem_ld_wait(raw);
                if constexpr (GLU) {
                    tmem_ld_wait(raw2);
                    float g[kChunk];
#pragma unroll
                    for (int j = 0; j < kChunk; ++j) {
                        g[j] = __uint_as_float(raw[j]);
                        v[j] = __uint_as_float(raw2[j]);
                    }
                    if (p.e4m3) {
#pragma unroll
                        for (int j = 0; j < kChunk; ++j) {
                            g[j] *= xs * col_a[j];
                            v[j] *= xs * col_b[j];
                        }
                    }
                    if (save) {
                        slot_write<2>(slot + z_at, lane, g, p.z_type);
                        slot_write<2>(slot + z_at + 2048, lane, v, p.z_type);
                    }
                    if (p.act == GS_ACT_SILU) {
#pragma unroll
                        for (int j = 0; j < kChunk; ++j) v[j] *= act_value(g[j], GS_ACT_SILU);
                    } else if (p.act == GS_ACT_GELU) {
#pragma unroll
                        for (int j = 0; j < kChunk; ++j) v[j] *= act_value(g[j], GS_ACT_GELU);
                    } else {
#pragma unroll
                        for (int j = 0; j < kChunk; ++j) v[j] *= act_value(g[j], p.act);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < kChunk; ++j) v[j] = __uint_as_float(raw[j]);
                    if (p.e4m3) {
#pragma unroll
                        for (int j = 0; j < kChunk; ++j) v[j] *= xs * col_a[j];
                    }
                    if (p.bias) {
#pragma unroll
                        for (int j = 0; j < kChunk; ++j) v[j] += col_b[j];
                    }
                    if (save) slot_write<2>(zs, lane, v, p.z_type);
                    if (p.act == GS_ACT_SILU) {
#pragma unroll
                        for (int j = 0; j < kChunk; ++j) v[j] = act_value(v[j], GS_ACT_SILU);
                    } else if (p.act == GS_ACT_GELU) {
#pragma unroll
                        for (int j = 0; j < kChunk; ++j) v[j] = act_value(v[j], GS_ACT_GELU);
                    } else if (p.act == GS_ACT_RELU) {
#pragma unroll
                        for (int j = 0; j < kChunk; ++j) v[j] = act_value(v[j], GS_ACT_RELU);
                    }
                    if (has_res) {
                        if (p.r_tma && !__all_sync(0xffffffffu, mbar_wait(res + 8 * b, (chunk_no / bufs) & 1, gave_up))) {
                            ok = false;
                            break;
                        }
                        slot_add<OSZ>(ys, lane, v, p.out_type);
                    }
                }
                slot_write<OSZ>(ys, lane, v, p.out_type);
                fence_async_smem();
                __syncwarp();
                // a TMA store writes whole 16-byte pieces: the last chunk of a row that ends
                // inside a piece goes by plain stores, which touch nothing beside it
                const bool ragged = col0 + kChunk > p.n;
                const bool y_tma = p.y_tma && (p.partial || !(ragged && (p.n * OSZ & 15)));
                const bool z_tma = p.z_tma && !(ragged && (p.n & 7));
                if (lane == 0) {
                    if (y_tma)
                        tma_store_3d(&p.y[p.partial ? 0 : q.prob], ys, (int)col0, (int)row0,
                                     p.partial ? q.prob * p.splits + q.split : 0);
                    if (save && z_tma) {
                        tma_store_3d(&p.z, GLU ? slot + z_at : zs, (int)col0, (int)row0, 0);
                        if constexpr (GLU) tma_store_3d(&p.z2, slot + z_at + 2048, (int)col0, (int)row0, 0);
                    }
                    bulk_commit();
                }
                if (!y_tma)
                    slot_to_rows<OSZ>(ys, q.prob ? p.yp[1] : p.yp[0], q.prob ? p.ldy[1] : p.ldy[0], row0, col0, p.m, p.n,
                                      lane);
                if (save && !z_tma) {
                    slot_to_rows<2>(GLU ? slot + z_at : zs, p.zp, p.ldz, row0, col0, p.m, p.n, lane);
                    if constexpr (GLU) slot_to_rows<2>(slot + z_at + 2048, p.z2p, p.ldz2, row0, col0, p.m, p.n, lane);
                }
                ++chunk_no;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR) mbar_arrive_cluster(free0 + 8 * acc);
                else mbar_arrive(bar_free + 8 * acc);
            }
        }
        if (lane == 0) bulk_wait_all();
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

// Rows of any alignment to rows of 16-byte pitch (the TMA needs both): eight
// 2-byte or sixteen 1-byte elements a thread, one 16-byte store.
template <typename E>
__global__ void __launch_bounds__(256) pack_rows_kernel(const E* src, int64_t ld, int64_t rows, int64_t cols, uint4* dst,
                                                        int64_t pieces)
{
    constexpr int kPer = 16 / sizeof(E);
    const int64_t total = rows * pieces, step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += step) {
        const int64_t r = i / pieces, c0 = i % pieces * kPer;
        union {
            uint4 q;
            E e[kPer];
        } v;
#pragma unroll
        for (int j = 0; j < kPer; ++j) v.e[j] = c0 + j < cols ? src[r * ld + c0 + j] : (E)0;
        dst[i] = v.q;
    }
}

// ------------------------------------------------------------------ host
struct Plan {
    bool pair;
    int bn;
    int64_t tile_m, out_cols, tiles_m, tiles_n, units, k_blocks;
    int splits, terms, probs, k_elems, esz;
    size_t pack_at[4], partial_at, bytes;   // a0, a1, b0, b1: offset + 1, 0 where used in place
    int64_t pitch;                          // of the partial sums
};

int device_sms()
{
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 152;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) return 152;
    return sms;
}

// Cycles of a configuration: waves of tiles, each bound by its products, the shared
// memory and TMA traffic that feeds them, or its epilogue, and a start-up.
double cost(const GemmCall& c, int bn, bool pair, int sms, Plan* out)
{
    Plan& p = *out;
    const bool glu = c.kind == GemmKind::kGlu;
    p.pair = pair;
    p.bn = bn;
    p.tile_m = pair ? 256 : 128;
    p.out_cols = glu ? bn / 2 : bn;
    p.tiles_m = (c.m + p.tile_m - 1) / p.tile_m;
    p.tiles_n = (c.n + p.out_cols - 1) / p.out_cols;
    p.esz = type_bytes(c.type);
    p.k_elems = kStageRow / p.esz;
    p.k_blocks = (c.k + p.k_elems - 1) / p.k_elems;
    p.terms = c.kind == GemmKind::kSum ? 2 : 1;
    p.probs = c.kind == GemmKind::kTwo ? 2 : 1;
    const int64_t tiles = p.tiles_m * p.tiles_n * p.probs, slots = pair ? sms / 2 : sms, kb = p.k_blocks * p.terms;
    // Few tiles: split k over the idle SMs, at least four k-blocks each, where nothing
    // but the sum is asked for (the gradients): the partial sums are joined in order.
    const bool sum_only = c.kind != GemmKind::kGlu && !c.bias && !c.residual && !c.z && c.act == GS_ACT_NONE &&
                          !c.x_scale && !c.w_scale[0];
    int64_t splits = 1;
    if (sum_only && tiles < slots) {
        splits = slots / tiles;
        if (splits > kb / 4) splits = kb / 4;
        if (splits < 1) splits = 1;
    }
    p.splits = (int)splits;
    p.units = tiles * splits;
    const double per_kb = bn == 64 ? 200 : (bn == 128 ? 330 : 520);
    const double main = per_kb * (double)((kb + splits - 1) / splits), epi = 10.0 * bn + 300;
    const double waves = (double)((p.units + slots - 1) / slots);
    const double join = splits > 1 ? 4000 + (double)splits * c.m * c.n * p.probs * 8 / (sms * 20.0) : 0;
    return 2500 + waves * (main > epi ? main : epi) + (main > epi ? epi : main) + join;
}

int64_t stored_rows(const GemmFactor& f, int64_t rows, int64_t k) { return f.k_fast ? rows : k; }
int64_t stored_cols(const GemmFactor& f, int64_t rows, int64_t k) { return f.k_fast ? k : rows; }

Plan make_plan(const GemmCall& c)
{
    const int sms = device_sms();
    Plan best, p;
    double at = 0;
    const bool glu = c.kind == GemmKind::kGlu;
    const int bns[3] = {64, 128, 256};
    for (int i = glu ? 1 : 0; i < 3; ++i) {
        const double v = cost(c, bns[i], bns[i] == 256, sms, &p);
        if (i == (glu ? 1 : 0) || v < at) {
            at = v;
            best = p;
        }
    }
    p = best;
    size_t used = 0;
    const GemmFactor* f[4] = {&c.a[0], &c.a[1], &c.b[0], &c.b[1]};
    for (int i = 0; i < 4; ++i) {
        p.pack_at[i] = 0;
        if (!f[i]->p || rows16(f[i]->p, f[i]->ld, c.type)) continue;
        if (i & 1 && f[i]->p == f[i - 1]->p) {   // kTwo: both products read the same factor
            p.pack_at[i] = p.pack_at[i - 1];
            continue;
        }
        const int64_t rows = i < 2 ? c.m : c.n;
        p.pack_at[i] = used + 1;
        used += (size_t)round_up(stored_rows(*f[i], rows, c.k) * round_up(stored_cols(*f[i], rows, c.k) * p.esz, 16), 256);
    }
    p.partial_at = used;
    p.pitch = round_up(c.n, 4);
    if (p.splits > 1) used += (size_t)round_up((int64_t)p.splits * p.probs * c.m * p.pitch * 4, 256);
    p.bytes = used;
    return p;
}

using Kernel = void (*)(const Params);

template <int BN, bool PAIR, bool GLU, int OSZ>
gs_status launch(const Params& p, int grid, cudaStream_t st)
{
    using S = Shape<BN, PAIR>;
    static_assert(S::kSmem <= 232448, "shared memory of an SM");
    auto* kernel = gemm_kernel<BN, PAIR, GLU, OSZ>;
    GS_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = PAIR ? 2 : 1;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 1 : 0;
    GS_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, p));
    return GS_OK;
}

}  // namespace

namespace tc {

gs_status make_map(CUtensorMap* map, const void* p, int type, int64_t rows, int64_t cols, int64_t ld, int box_rows,
                   int box_cols, int64_t depth)
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
    const int esz = type_bytes(type);
    const CUtensorMapDataType dt = type == GS_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : type == GS_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                   : type == GS_F16  ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                     : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const int dims = depth > 0 ? 3 : 2;
    const cuuint64_t size[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)(depth > 0 ? depth : 1)};
    const cuuint64_t pitch[2] = {(cuuint64_t)(ld * esz), (cuuint64_t)(ld * esz) * (cuuint64_t)rows};
    const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
    const cuuint32_t unit[3] = {1, 1, 1};
    const CUresult r = encode(map, dt, dims, const_cast<void*>(p), size, pitch, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              box_cols * esz == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? GS_OK : GS_ERR_CUDA;
}

}  // namespace tc

gs_status gemm_ws_bytes(const GemmCall& c, size_t* bytes)
{
    *bytes = make_plan(c).bytes;
    return GS_OK;
}

gs_status gemm_run(const GemmCall& c, void* ws, cudaStream_t st)
{
    const Plan plan = make_plan(c);
    if (plan.units > 0x7fffffffll || c.m > 0x7fffff00ll || c.n > 0x7fffff00ll || c.k > 0x7fffff00ll)
        return GS_ERR_INVALID_ARG;
    char* base = (char*)ws;
    GemmFactor f[4] = {c.a[0], c.a[1], c.b[0], c.b[1]};
    for (int i = 0; i < 4; ++i) {
        if (!plan.pack_at[i]) continue;
        const int64_t rows = stored_rows(f[i], i < 2 ? c.m : c.n, c.k), cols = stored_cols(f[i], i < 2 ? c.m : c.n, c.k);
        const int64_t pieces = round_up(cols * plan.esz, 16) / 16;
        uint4* dst = (uint4*)(base + plan.pack_at[i] - 1);
        if (!(i & 1 && plan.pack_at[i] == plan.pack_at[i - 1])) {
            const int64_t blocks = (rows * pieces + 255) / 256;
            const unsigned grid = (unsigned)(blocks < 152 * 16 ? blocks : 152 * 16);
            if (plan.esz == 2)
                pack_rows_kernel<uint16_t><<<grid, 256, 0, st>>>((const uint16_t*)f[i].p, f[i].ld, rows, cols, dst, pieces);
            else
                pack_rows_kernel<uint8_t><<<grid, 256, 0, st>>>((const uint8_t*)f[i].p, f[i].ld, rows, cols, dst, pieces);
            GS_LAUNCH_CHECK();
        }
        f[i].p = dst;
        f[i].ld = pieces * 16 / plan.esz;
    }

    Params p = {};
    const bool glu = c.kind == GemmKind::kGlu;
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
        p.y_tma = 1;
        const gs_status s = tc::make_map(&p.y[0], base + plan.partial_at, GS_F32, c.m, plan.pitch, plan.pitch, 32, kChunk,
                                         (int64_t)plan.splits * plan.probs);
        if (s != GS_OK) return s;
    } else {
        p.y_tma = rows16(c.y, c.ldy, c.out_type) && (plan.probs == 1 || rows16(c.y2, c.ldy2, c.out_type));
        for (int i = 0; i < plan.probs; ++i) {
            p.yp[i] = y[i];
            p.ldy[i] = ldy[i];
            if (!p.y_tma) continue;
            const gs_status s = tc::make_map(&p.y[i], y[i], out_type, c.m, c.n, ldy[i], 32, kChunk, 1);
            if (s != GS_OK) return s;
        }
        if (c.residual) {
            p.residual = c.residual;
            p.ldr = c.ldr;
            p.r_tma = rows16(c.residual, c.ldr, c.out_type);
            if (p.r_tma) {
                const gs_status s = tc::make_map(&p.r, c.residual, c.out_type, c.m, c.n, c.ldr, 32, kChunk);
                if (s != GS_OK) return s;
            }
        }
        if (c.z) {
            p.zp = c.z, p.ldz = c.ldz, p.z2p = c.z2, p.ldz2 = c.ldz2;
            p.z_tma = rows16(c.z, c.ldz, c.z_type) && (!glu || rows16(c.z2, c.ldz2, c.z_type));
            if (p.z_tma) {
                gs_status s = tc::make_map(&p.z, c.z, c.z_type, c.m, c.n, c.ldz, 32, kChunk, 1);
                if (s == GS_OK && glu) s = tc::make_map(&p.z2, c.z2, c.z_type, c.m, c.n, c.ldz2, 32, kChunk, 1);
                if (s != GS_OK) return s;
            }
        }
        p.x_scale = c.x_scale;
        p.w_scale[0] = c.w_scale[0], p.w_scale[1] = c.w_scale[1];
        p.bias = c.bias, p.bias_type = c.bias_type, p.act = c.act;
    }
    p.m = c.m, p.n = c.n;
    p.out_type = out_type, p.z_type = c.z_type;
    p.k_blocks = plan.k_blocks, p.tiles_m = plan.tiles_m, p.tiles_n = plan.tiles_n, p.units = plan.units;
    p.splits = plan.splits, p.terms = plan.terms, p.probs = plan.probs, p.k_elems = plan.k_elems;
    p.a_fast = c.a[0].k_fast, p.b_fast = c.b[0].k_fast;
    p.e4m3 = c.type == GS_E4M3;
    p.idesc = tc::instr_desc(c.type, c.a[0].k_fast, c.b[0].k_fast, plan.bn, (int)plan.tile_m);
    const int sms = device_sms();
    const int64_t most = plan.pair ? sms / 2 : sms;
    const int grid = (int)(plan.units < most ? plan.units : most) * (plan.pair ? 2 : 1);
    gs_status s;
    if (glu) s = plan.pair ? launch<256, true, true, 2>(p, grid, st) : launch<128, false, true, 2>(p, grid, st);
    else if (out_type == GS_F32)
        s = plan.pair         ? launch<256, true, false, 4>(p, grid, st)
            : plan.bn == 128 ? launch<128, false, false, 4>(p, grid, st)
                             : launch<64, false, false, 4>(p, grid, st);
    else
        s = plan.pair         ? launch<256, true, false, 2>(p, grid, st)
            : plan.bn == 128 ? launch<128, false, false, 2>(p, grid, st)
                             : launch<64, false, false, 2>(p, grid, st);
    if (s != GS_OK || !p.partial) return s;
    const float* partial = (const float*)(base + plan.partial_at);
    for (int i = 0; i < plan.probs; ++i) {
        s = join_partials(partial + (int64_t)i * plan.splits * c.m * plan.pitch, plan.splits, c.m, c.n, plan.pitch, y[i],
                          ldy[i], c.out_type, st);
        if (s != GS_OK) return s;
    }
    return GS_OK;
}

}  // namespace gs

using namespace gs;

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
    *expired = v;
    return v ? GS_ERR_TIMEOUT : GS_OK;
}
