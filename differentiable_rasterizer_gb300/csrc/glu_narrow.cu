// glu_narrow.cu -- gradients of a narrow gated layer in one pass over its rows.
//
//   g = x Wg^T, u = x Wu^T            (computed again: features are few)
//   dg = dh u act'(g), du = dh act(g) (rounded to 16 bits, factors of the products below)
//   dx = dg Wg + du Wu,  dWg = dg^T x, dWu = du^T x
//
// for at most 64 features and 128 hidden columns (a per-Gaussian decoder's layer), where
// both weights, a tile of 128 rows with its dg and du, and all accumulators fit on one SM:
// only x and dh are read and dx is written, 2 (2 features + hidden) bytes a row.  As three
// products dg and du cross HBM three times (1,000,000 x 64 -> 128: 1.5 GB of 2.0): 122 us
// against 411 there, 24 against 56 for 100,000 rows, 10 against 15.5 for one.  What bounds
// it at 128 hidden columns is the turn of a stage, at 4.2 TB/s (copy, TMEM reads and
// arithmetic, products whose factors shared memory delivers at 48 cycles each; without
// most products 109 us before the stages were halves, without the activation 119); at 64
// HBM at 5.1 TB/s (75 us).
//
// A persistent CTA an SM, 18 warps: a TMA producer, an MMA issuer, 16 epilogue warps.
// TMEM, fp32: two buffers of 64 gate and 64 up columns (a half of the hidden columns
// each), two of dx, and dWg and dWu, which stay for all of the CTA's rows and end as its
// partial sum.  dg takes dh's place in shared memory; the same
// tiles are k-fast factors of dx and k-slow factors of the weights' gradients, and the
// weights are k-fast for g and u and k-slow for dx.
#include <atomic>

#include "gemm.cuh"
#include "tc_common.cuh"

namespace gs {
namespace {

using namespace tc;

constexpr int kWarps = 18, kThreads = kWarps * 32;
constexpr int kTileRows = 128, kHalf = 64;             // rows of a tile; hidden columns of a half
constexpr uint32_t kBox = kTileRows * 128;             // bytes of 128 rows of 64 columns
constexpr uint32_t kTmemDw = 320, kTmemCols = 512;     // columns: two of g and u, dx, the weights' gradients, dx
__device__ __forceinline__ uint32_t dx_buffer(uint32_t b) { return b ? 448 : 256; }
constexpr int kStages = 4, kMostX = 4;

enum Bar {
    kWFull = 0,
    kXFull = 1,                    // x of a tile has landed
    kXEmpty = kXFull + kMostX,     // its products are done
    kFull = kXEmpty + kMostX,      // dh of a unit has landed
    kEmpty = kFull + kStages,      // its products are done
    kGradFull = kEmpty + kStages,  // its dg and du are written
    kGuFull = kGradFull + kStages, // a buffer's g and u are there
    kGuFree = kGuFull + 2,         // and read
    kDxFull = kGuFree + 2,         // a buffer's dx is there
    kDxFree = kDxFull + 2,
    kDone = kDxFree + 2,
    kDrain,
    kBars
};

// HALVES: of the hidden columns, 64 each.  A unit is a half of a tile; unit u's buffer of
// g and u and its eight epilogue warps are number u % 2, its stage u % 4.
template <int HALVES>
struct Shape {
    static constexpr int kStagesX = HALVES == 1 ? 4 : 3;
    static constexpr uint32_t kWeights = HALVES * kBox;     // per half: 64 rows of Wg, 64 of Wu
    static constexpr uint32_t kStage = 2 * kBox;            // dh, then dg in its place; du
    static constexpr uint32_t kAtX = kWeights + kStages * kStage, kAtBars = kAtX + kStagesX * kBox;
    static constexpr int kSmem = kAtBars + ((kBars * 8 + 15) & ~15) + 16;
    static_assert(kSmem <= 232448, "shared memory of an SM");
    static constexpr int kDxCols = HALVES == 1 ? 32 : 16;   // of an epilogue warp
};

struct Params {
    CUtensorMap x, dh, wg, wu;
    void* dx;          // NULL: not asked for
    float* dw[2];      // NULL, or a partial sum [hidden][pitch] a CTA
    int64_t lddx;
    uint32_t m, tiles, idesc_gu, idesc_dx, idesc_dw;
    int features, hidden, pitch, dx_vec;
};

// The CTA's tiles: blockIdx.x, blockIdx.x + gridDim.x, ...
__device__ __forceinline__ uint32_t own_tiles(const Params& p) { return (p.tiles - blockIdx.x + gridDim.x - 1) / gridDim.x; }

__device__ int g_narrow_wait_expired;

__device__ __forceinline__ void prefetch_2d(const CUtensorMap* map, int x, int y)
{
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}

template <int HALVES>
__device__ __forceinline__ void load_rows(const Params& p, uint32_t smem, uint32_t bars, volatile int* gave_up)
{
    using S = Shape<HALVES>;
    mbar_expect(bars + 8 * kWFull, S::kWeights);
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
        tma_load_2d<false>(smem + h * kBox, &p.wg, 0, h * kHalf, bars + 8 * kWFull);
        tma_load_2d<false>(smem + h * kBox + kBox / 2, &p.wu, 0, h * kHalf, bars + 8 * kWFull);
    }
    Ring<S::kStagesX> rx;
    Ring<kStages> ru;
    uint32_t xs = 0, units = 0;
    bool ok = true;
    for (uint32_t t = blockIdx.x; ok && t < p.tiles; t += gridDim.x) {
        const int row = (int)(t * kTileRows);
        // a stage is empty for a short time only: its next tile is on its way into L2 by then
        const uint64_t ahead = (uint64_t)t + (uint64_t)S::kStagesX * gridDim.x;
        const bool more = ahead < p.tiles;
        const int row_ahead = (int)(ahead * kTileRows);
        if (!mbar_wait(bars + 8 * (kXEmpty + rx.s), rx.parity ^ 1, gave_up)) break;
        mbar_expect(bars + 8 * (kXFull + rx.s), kBox);
        tma_load_2d<false>(smem + S::kAtX + rx.s * kBox, &p.x, 0, row, bars + 8 * (kXFull + rx.s));
        if (more) prefetch_2d(&p.x, 0, row_ahead);
        rx.next();
        ++xs;
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
            ok = ok && mbar_wait(bars + 8 * (kEmpty + ru.s), ru.parity ^ 1, gave_up);
            if (!ok) break;
            mbar_expect(bars + 8 * (kFull + ru.s), kBox);
            tma_load_2d<false>(smem + S::kWeights + ru.s * S::kStage, &p.dh, h * kHalf, row, bars + 8 * (kFull + ru.s));
            if (more) prefetch_2d(&p.dh, h * kHalf, row_ahead);
            ru.next();
            ++units;
        }
    }
    // the block does not leave before its copies have landed
    bool landed = mbar_wait_alone(bars + 8 * kWFull, 0);
    last_copies<S::kStagesX>(xs, [&](uint32_t s, uint32_t parity) { landed = landed && mbar_wait_alone(bars + 8 * (kXFull + s), parity); });
    last_copies<kStages>(units, [&](uint32_t s, uint32_t parity) { landed = landed && mbar_wait_alone(bars + 8 * (kFull + s), parity); });
}

// Two kinds of work in the order in which they become ready: a unit's g and u, when its x
// has landed and its buffer is read; its part of dx and of the weights' gradients, when its
// dg and du are written.  (In a fixed order, the next tile's g and u first, a late copy
// held the products back that free the stage of the copy after it: 160 us the million rows.)
template <int HALVES>
__device__ __forceinline__ void issue_products(const Params& p, uint32_t smem, uint32_t bars, uint32_t tmem, volatile int* gave_up)
{
    using S = Shape<HALVES>;
    const uint32_t steps_x = (uint32_t)(p.features + 15) / 16, units = own_tiles(p) * HALVES;
    if (!mbar_wait(bars + 8 * kWFull, 0, gave_up)) return;
    Ring<S::kStagesX> xg, xd;   // x of the next unit of either kind
    uint32_t next = 0, v = 0, idle = 0;
    long long since = 0;
    while (v < units) {
        bool did = false;
        const uint32_t b = next & 1;
        if (next < units && mbar_test(bars + 8 * (kXFull + xg.s), xg.parity) &&
            mbar_test(bars + 8 * (kGuFree + b), (next >> 1 & 1) ^ 1)) {
            tc_fence_after();
            const uint32_t x = desc_lo(smem + S::kAtX + xg.s * kBox, true), w = desc_lo(smem + next % HALVES * kBox, true);
            for (uint32_t j = 0; j < steps_x; ++j)
                mma<false, false>(tmem + b * 128, x + j * k_step(true), kDescHi, w + j * k_step(true), kDescHi, p.idesc_gu, j > 0);
            mma_commit<false>(bars + 8 * (kGuFull + b));
            ++next;
            if (next % HALVES == 0) xg.next();
            did = true;
        }
        const uint32_t i = v / HALVES, h = v % HALVES, s = v % kStages;
        if (v < next && mbar_test(bars + 8 * (kGradFull + s), v / kStages & 1) &&
            (!p.dx || h > 0 || mbar_test(bars + 8 * (kDxFree + (i & 1)), (i >> 1 & 1) ^ 1))) {
            tc_fence_after();
            const uint32_t at = smem + S::kWeights + s * S::kStage;
            if (p.dx) {
#pragma unroll
                for (uint32_t w = 0; w < 2; ++w) {   // dg Wg, du Wu
                    const uint32_t a = desc_lo(at + w * kBox, true), c = desc_lo(smem + h * kBox + w * (kBox / 2), false);
#pragma unroll
                    for (uint32_t j = 0; j < 4; ++j)
                        mma<false, false>(tmem + dx_buffer(i & 1), a + j * k_step(true), kDescHi, c + j * k_step(false), kDescHi,
                                          p.idesc_dx, h > 0 || w > 0 || j > 0);
                }
                if (h == HALVES - 1) mma_commit<false>(bars + 8 * (kDxFull + (i & 1)));
            }
            if (p.dw[0]) {
                // k is the row, M the half's 64 columns of dg and, a box on, of du
                const uint32_t a = (at >> 4) | ((kBox >> 4) << 16), c = desc_lo(smem + S::kAtX + xd.s * kBox, false);
#pragma unroll
                for (uint32_t j = 0; j < kTileRows / 16; ++j)
                    mma<false, false>(tmem + kTmemDw + h * 64, a + j * k_step(false), kDescHi, c + j * k_step(false), kDescHi,
                                      p.idesc_dw, i > 0 || j > 0);
            }
            mma_commit<false>(bars + 8 * (kEmpty + s));
            if (h == HALVES - 1) {
                mma_commit<false>(bars + 8 * (kXEmpty + xd.s));
                xd.next();
            }
            ++v;
            did = true;
        }
        if (did) idle = 0;
        else if (++idle % 256 == 0) {   // bounded as every wait is
            const long long now = clock64();
            if (idle == 256) since = now;
            if (*gave_up) return;
            if (now - since > kWaitCycles) {
                *gave_up = 1;
                return;
            }
        }
    }
    mma_commit<false>(bars + 8 * kDone);
}

// kDxCols columns of dx of the CTA's i-th tile to memory: a thread has its row's.
template <int T, int HALVES>
__device__ __forceinline__ bool store_dx(const Params& p, uint32_t i, uint32_t row, int col, uint32_t tmem, uint32_t bars, int lane,
                                         volatile int* gave_up)
{
    constexpr int kCols = Shape<HALVES>::kDxCols;
    const uint32_t b = i & 1;
    if (!__all_sync(0xffffffffu, mbar_wait(bars + 8 * (kDxFull + b), i >> 1 & 1, gave_up))) return false;
    tc_fence_after();
#pragma unroll 1
    for (int c = 0; c < kCols; c += 16, col += 16) {
        uint32_t v[16];
        tmem_ld16(tmem + dx_buffer(b) + col, v);
        tmem_ld_wait(v);
        if (c + 16 == kCols) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars + 8 * (kDxFree + b));
        }
        const int left = row < p.m ? p.features - col : 0;
        uint16_t* to = (uint16_t*)p.dx + (int64_t)row * p.lddx + col;
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = pack_half2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]), T);
        if (p.dx_vec == 2 && left >= 16) {   // whole sectors
            st_global32(to, w);
            continue;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (p.dx_vec && left >= 8 * e + 8)
                *reinterpret_cast<uint4*>(to + 8 * e) = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
            else
#pragma unroll
                for (int j = 8 * e; j < 8 * e + 8; ++j)
                    if (j < left) to[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
        }
    }
    return true;
}

template <int T, int ACT, int HALVES>
__global__ void __launch_bounds__(kThreads, 1) glu_narrow_kernel(const __grid_constant__ Params p)
{
    using S = Shape<HALVES>;
    extern __shared__ __align__(1024) char smem_raw[];
    const uint32_t smem = smem_addr(smem_raw);
    if (smem & 1023u) {   // every thread sees the same address; there is no padding to move within
        g_narrow_wait_expired = 1;
        return;
    }
    const uint32_t bars = smem + S::kAtBars;
    char* tail = smem_raw + S::kAtBars + ((kBars * 8 + 15) & ~15);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail);
    volatile int* gave_up = reinterpret_cast<volatile int*>(tail + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kBars; ++i) {
            const bool group = (i >= kGradFull && i < kGuFull) || (i >= kGuFree && i < kDxFull), dx = i >= kDxFree && i < kDone;
            mbar_init(bars + 8 * i, group ? 8 : (dx ? 8 * HALVES : 1));
        }
        *gave_up = 0;
        mbar_init_fence();
    }
    if (warp == 1) tmem_alloc<false>(smem_addr(tmem_slot), kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    wait_for_predecessor();

    if (warp == 0) {
        if (elect_one()) load_rows<HALVES>(p, smem, bars, gave_up);
    } else if (warp == 1) {
        if (elect_one()) {
            issue_products<HALVES>(p, smem, bars, tmem, gave_up);
            if (*gave_up) {
                mma_commit<false>(bars + 8 * kDrain);
                mbar_wait_alone(bars + 8 * kDrain, 0);
            }
        }
    } else {
        // 32 rows and 32 columns of the units of a group: a half, or every other tile
        const int quarter = warp & 3, part = (warp - 2) >> 2 & 1, col = part * 32;
        const uint32_t group = (uint32_t)(warp - 2) >> 3;
        const uint32_t row = quarter * 32 + lane, mine = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t piece = row * 128 + (((uint32_t)(col >> 3) ^ (row & 7)) << 4);   // its columns' first 16 bytes in a box
        const int dx_col = HALVES == 1 ? col : (int)group * 32 + part * 16;
        constexpr uint32_t kTurn = 2 / HALVES;   // tiles from one of a group's units to the next
        const uint32_t tiles = own_tiles(p);
        const auto row_of = [&](uint32_t i) { return (blockIdx.x + i * gridDim.x) * kTileRows + row; };
        const int live = p.hidden - (HALVES == 1 ? 0 : (int)group * kHalf) - col;   // columns of the layer from col on
        bool ok = true;
        uint32_t i = HALVES == 1 ? group : 0, u = group;
        for (; i < tiles; i += kTurn, u += 2) {
            const uint32_t at = smem + S::kWeights + u % kStages * S::kStage + piece;
            ok = __all_sync(0xffffffffu, mbar_wait(bars + 8 * (kFull + u % kStages), u / kStages & 1, gave_up) &&
                                             mbar_wait(bars + 8 * (kGuFull + group), u >> 1 & 1, gave_up));
            if (!ok) break;
            tc_fence_after();
            uint32_t raw[2][16], up[2][16];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                tmem_ld16(mine + group * 128 + col + 16 * c, raw[c]);
                tmem_ld16(mine + group * 128 + 64 + col + 16 * c, up[c]);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                tmem_ld_wait(raw[c]);
                tmem_ld_wait(up[c]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars + 8 * (kGuFree + group));
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const uint32_t a = at ^ (c << 5);
                const uint4 d0 = ld_shared16(a), d1 = ld_shared16(a ^ 16);
                const uint32_t dh[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
                float g[16], u[16], d[16];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 f = unpack_half2(dh[e], T);
                    d[2 * e] = f.x, d[2 * e + 1] = f.y;
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) g[e] = __uint_as_float(raw[c][e]), u[e] = __uint_as_float(up[c][e]);
                glu_gradient<ACT>(g, u, d);
                if (live < 32) {   // beyond the layer: zeros, though an infinite x times no weight were none
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (e + 16 * c >= live) g[e] = u[e] = 0.0f;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    st_shared16(a ^ (e << 4), make_uint4(pack_half2(g[8 * e], g[8 * e + 1], T), pack_half2(g[8 * e + 2], g[8 * e + 3], T),
                                                         pack_half2(g[8 * e + 4], g[8 * e + 5], T), pack_half2(g[8 * e + 6], g[8 * e + 7], T)));
                    st_shared16((a ^ (e << 4)) + kBox,
                                make_uint4(pack_half2(u[8 * e], u[8 * e + 1], T), pack_half2(u[8 * e + 2], u[8 * e + 3], T),
                                           pack_half2(u[8 * e + 4], u[8 * e + 5], T), pack_half2(u[8 * e + 6], u[8 * e + 7], T)));
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the products read what was just written
            __syncwarp();
            if (lane == 0) mbar_arrive(bars + 8 * (kGradFull + u % kStages));
            if (i >= kTurn && p.dx) {   // the dx of the tile before is ready by now
                ok = store_dx<T, HALVES>(p, i - kTurn, row_of(i - kTurn), dx_col, mine, bars, lane, gave_up);
                if (!ok) break;
            }
        }
        if (ok && p.dx && i >= kTurn) ok = store_dx<T, HALVES>(p, i - kTurn, row_of(i - kTurn), dx_col, mine, bars, lane, gave_up);
        if (ok && p.dw[0] && __all_sync(0xffffffffu, mbar_wait(bars + 8 * kDone, 0, gave_up))) {
            tc_fence_after();
            // lanes: a half's 64 rows of dWg, then of dWu
            const uint32_t half = HALVES == 1 ? 0 : group, which = row >> 6;
            const int hidden = (int)(half * kHalf + (row & 63)), from = HALVES == 1 ? (int)group * 32 + part * 16 : col;
#pragma unroll 1
            for (int c = from; c < from + 16 * HALVES; c += 16) {
                uint32_t v[16];
                tmem_ld16(mine + kTmemDw + half * 64 + c, v);
                tmem_ld_wait(v);
                float* to = p.dw[which] + ((int64_t)blockIdx.x * p.hidden + hidden) * p.pitch + c;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (hidden < p.hidden && c + 4 * e < p.pitch)
                        *reinterpret_cast<uint4*>(to + 4 * e) = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
            }
            tc_fence_before();
        }
    }
    __syncthreads();
    if (threadIdx.x == 0 && *gave_up) atomicExch(&g_narrow_wait_expired, 1);
    if (warp == 1) {
        tc_fence_after();
        tmem_free<false>(tmem, kTmemCols);
    }
}

template <int T, int ACT, int HALVES>
gs_status launch(const Params& p, unsigned grid, cudaStream_t st)
{
    static std::atomic<uint64_t> done{0};
    const gs_status s = allow_smem(glu_narrow_kernel<T, ACT, HALVES>, Shape<HALVES>::kSmem, done);
    if (s != GS_OK) return s;
    return launch_after(glu_narrow_kernel<T, ACT, HALVES>, dim3(grid), kThreads, Shape<HALVES>::kSmem, 1, st, p);
}

}  // namespace

bool glu_narrow_fits(int64_t features, int64_t hidden) { return features <= 64 && hidden <= 2 * kHalf; }

int64_t glu_narrow_blocks(int64_t rows)
{
    const int64_t tiles = (rows + kTileRows - 1) / kTileRows, sms = device_sms() > 0 ? device_sms() : 152;
    return tiles < sms ? tiles : sms;
}

gs_status glu_narrow_grad(const GluNarrowCall& c, cudaStream_t st)
{
    if (c.rows > 0x7fffff00ll) return GS_ERR_INVALID_ARG;
    Params p = {};
    gs_status s = make_map(&p.x, c.x, c.type, c.rows, c.features, c.ldx, kTileRows, kHalf);
    if (s == GS_OK) s = make_map(&p.dh, c.dh, c.type, c.rows, c.hidden, c.lddh, kTileRows, kHalf);
    if (s == GS_OK) s = make_map(&p.wg, c.w_gate, c.type, c.hidden, c.features, c.ldwg, kHalf, kHalf);
    if (s == GS_OK) s = make_map(&p.wu, c.w_up, c.type, c.hidden, c.features, c.ldwu, kHalf, kHalf);
    if (s != GS_OK) return s;
    p.dx = c.dx, p.lddx = c.lddx, 
    p.dx_vec = c.dx && rows16(c.dx, c.lddx, c.type) ? (((uintptr_t)c.dx | (uintptr_t)(c.lddx * 2)) % 32 == 0 ? 2 : 1) : 0;
    p.dw[0] = c.dw_gate, p.dw[1] = c.dw_up, p.pitch = (int)c.pitch;
    p.m = (uint32_t)c.rows, p.tiles = (uint32_t)((c.rows + kTileRows - 1) / kTileRows);
    p.features = (int)c.features, p.hidden = (int)c.hidden;
    p.idesc_gu = instr_desc(c.type, true, true, 2 * kHalf, kTileRows);
    p.idesc_dx = instr_desc(c.type, true, false, 64, kTileRows);
    p.idesc_dw = instr_desc(c.type, false, false, 64, 2 * kHalf);
    const unsigned grid = (unsigned)glu_narrow_blocks(c.rows);
    return for_type_act(c.type, c.act, [&](auto t, auto act) {
        constexpr int T = decltype(t)::value, ACT = decltype(act)::value;
        return c.hidden <= kHalf ? launch<T, ACT, 1>(p, grid, st) : launch<T, ACT, 2>(p, grid, st);
    });
}

gs_status glu_narrow_wait_report(int* expired)
{
    const int zero = 0;
    GS_CUDA_TRY(cudaMemcpyFromSymbol(expired, g_narrow_wait_expired, sizeof *expired));
    if (*expired) GS_CUDA_TRY(cudaMemcpyToSymbol(g_narrow_wait_expired, &zero, sizeof zero));
    return GS_OK;
}

}  // namespace gs
