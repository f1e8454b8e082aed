// attention.cu -- attention over packed sequences, forward.
//
//   t = scale q k^T,  p = exp(t - m),  o = (p v) / sum p,   m the rows' running maximum
//
// One pass over the keys, 128 at a time, for one or two tiles of 128 packed rows a CTA.
// Warps have fixed roles:
//   four a tile     softmax, a row a thread: scores TMEM -> registers -> p in 16 bits back
//                   over the scores, the sum in fp32
//   one             TMA producer: q, then keys and values in a ring
//   one a tile      a lane issues tcgen05.mma: scores from shared memory, p v with p from TMEM
// While one tile's softmax works, the tensor cores compute the other's products (of the
// CTA, or of the second CTA on the SM).  TMEM, fp32: a tile's scores (p in their first 64
// columns) and its o.  The products of a tile's p with v and of its next scores, which
// overwrite p, are issued in that order by one lane and run in it.
//
// What bounds it: for 128 columns the products (128 x 128 x 16 at 64 cycles each: 2048 cycles a
// pair of tiles), for 64 and fewer the softmax beside them (128 exponentials a row at 32 a
// cycle and SM).  16384 tokens, 8 heads of 128, causal, bf16: 356 us, 1.54 PFLOP/s; 8192 of 64:
// 162 us.  A step's chain of waits (some 350 cycles each beside products whose factors keep
// shared memory busy) sets the rest: see issue().
//
// The maximum that a row's terms are taken to is raised only when a tile of keys exceeds
// it by more than 2^15: o and the sum are then rescaled (rare after the first tiles), and
// terms stay within 2^15 in between, which f16 holds and the fp32 sums do not mind.  p is
// rounded to 16 bits because the tensor cores take 16-bit factors; the sum takes it unrounded.
// f16's smallest step, 2^-24, would round away what the keys of a long context weigh together
// (2^-25 of the row's largest for each): terms are held times a power of two that grows with the
// keys, and the maximum is raised so much earlier (see held_up).
//
// Few rows against many keys (single tokens) leave most SMs idle: the keys of a tile are
// then split over several CTAs, whose sums and maxima join_kernel puts together in a
// fixed order.
#include <atomic>
#include <cmath>

#include "attention.cuh"

namespace gs {
namespace attn {
namespace {

constexpr float kMost = 15.0f;   // log2 of the largest term

// TILES: of a CTA.  With one, two CTAs share an SM; two only with 128 columns (see plan_for).
template <int DP, int TILES>
struct Shape {
    static_assert(TILES == 1 || (TILES == 2 && DP == 128), "the shapes that plan_for chooses from");
    static constexpr int kChunks = DP / 64;
    static constexpr uint32_t kTile = kChunks * kBox;
    static constexpr int kStages = TILES == 1 && DP == 128 ? 2 : 5;
    static constexpr int kSoftmaxWarps = 4 * TILES, kThreads = (kSoftmaxWarps + 4) * 32;
    static constexpr uint32_t kTmemCols = 256 * TILES, kTmemO = 128 * TILES;
    static constexpr uint32_t kAtRing = TILES * kTile, kAtBars = kAtRing + kStages * kTile;
    static constexpr int kQFull = 0, kFull = 2, kEmpty = kFull + kStages, kScores = kEmpty + kStages, kTerms = kScores + 2,
                         kSums = kTerms + 4, kClear = kSums + 2, kDone = kClear + 1, kBars = kDone + 2;
    static constexpr int kSmem = kAtBars + ((kBars * 8 + 15) & ~15) + 16;
    static_assert(kSmem <= 232448 / (3 - TILES) - (2 - TILES) * 1024, "shared memory of an SM");
};

struct Params {
    CUtensorMap q, k, v;
    Sequences seqs;
    Fill fill;
    uint16_t* o;
    int64_t o_row, o_head;
    float* lse;
    float* part;          // splits > 1: [split][q row][head][DP] sums of p v
    float2* part_stats;   // [split][q row][head] what their terms are taken to, and the sums of p
    float scale2;         // scale log2(e)
    uint32_t splits, kv_heads;
    int group, tokens;    // query heads of a key head, tokens of a tile
    int dim, o_vec, causal, zero;
    uint32_t idesc_s, idesc_o;
};

__device__ int g_attention_wait_expired;

// A CTA's work: a unit of one or two tiles of a key head, and its part of the keys' tiles.
struct Work {
    Sequence seq;
    uint32_t split, head;
    int t0;            // the first token of the unit
    int from;          // the first tile of keys
    int n[2];          // tiles of keys from there for either tile of the unit
};

template <int TILES>
__device__ __forceinline__ bool find_work(const Params& p, Work& w)
{
    const uint32_t rest = blockIdx.x / p.splits;
    w.split = blockIdx.x % p.splits;
    w.head = rest % p.kv_heads;
    uint32_t unit, units;
    const int tokens = p.tokens * TILES;
    if (!find_unit<false>(p.seqs, rest / p.kv_heads, tokens, w.seq, unit, units)) return false;
    if (p.causal) unit = units - 1 - unit;   // the longest first
    w.t0 = (int)unit * tokens;
    int tiles[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = w.t0 + i * p.tokens;
        int last = t + p.tokens - 1;
        last = last < w.seq.lq ? last : w.seq.lq - 1;
        tiles[i] = i < TILES && t < w.seq.lq ? (keys_seen(w.seq, last, p.causal) + kRows - 1) / kRows : 0;
    }
    const int most = tiles[0] > tiles[1] ? tiles[0] : tiles[1];
    const int each = (most + (int)p.splits - 1) / (int)p.splits;
    w.from = (int)w.split * each;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int n = tiles[i] - w.from;
        n = n < 0 ? 0 : n;
        w.n[i] = n < each ? n : each;
    }
    return true;
}

template <int DP, int TILES>
__device__ __forceinline__ void load(const Params& p, const Work& w, int n, uint32_t smem, uint32_t bars, volatile int* gave_up)
{
    using S = Shape<DP, TILES>;
    const uint32_t q_bytes = (uint32_t)(S::kChunks * p.tokens * p.group) * 128;
#pragma unroll
    for (int i = 0; i < TILES; ++i)
        if (w.n[i] > 0) {
            mbar_expect(bars + 8 * (S::kQFull + i), q_bytes);
            load_tile<S::kChunks>(smem + i * S::kTile, &p.q, w.head * p.group, w.seq.q0 + w.t0 + i * p.tokens, bars + 8 * (S::kQFull + i));
        }
    Ring<S::kStages> ring;
    uint32_t issued = 0;
    int row = w.seq.k0 + w.from * kRows;
    for (int j = 0; j < 2 * n; ++j, ++issued, ring.next()) {
        if (!mbar_wait(bars + 8 * (S::kEmpty + ring.s), ring.parity ^ 1, gave_up)) break;
        mbar_expect(bars + 8 * (S::kFull + ring.s), S::kTile);
        load_tile<S::kChunks>(smem + S::kAtRing + ring.s * S::kTile, j & 1 ? &p.v : &p.k, w.head, row, bars + 8 * (S::kFull + ring.s));
        if (j & 1) row += kRows;
    }
    // the block does not leave before its copies have landed
    bool landed = true;
#pragma unroll
    for (int i = 0; i < TILES; ++i) landed = landed && (w.n[i] == 0 || mbar_wait_alone(bars + 8 * (S::kQFull + i), 0));
    last_copies<S::kStages>(issued, [&](uint32_t s, uint32_t parity) { landed = landed && mbar_wait_alone(bars + 8 * (S::kFull + s), parity); });
}

// A lane issues the products of tile i.  (Of both tiles in turn one lane is too slow: each
// of its waits takes some 350 cycles beside products whose factors come from shared memory,
// 900 TFLOP/s where two lanes reach 1,100.)
template <int DP, int TILES>
__device__ __forceinline__ void issue(const Params& p, const Work& w, int i, int n, uint32_t smem, uint32_t bars, uint32_t tmem, volatile int* gave_up)
{
    using S = Shape<DP, TILES>;
    const int mine = i ? w.n[1] : w.n[0];
    const uint32_t steps = (uint32_t)(p.dim + 15) / 16, score = tmem + i * 128, sum = tmem + S::kTmemO + i * DP;
    const bool ragged = w.seq.lk < (w.from + n) * kRows;
    const auto scores = [&](uint32_t tile) {
        const uint32_t a = desc_lo(smem + i * S::kTile, true), b = desc_lo(tile, true);
#pragma unroll
        for (uint32_t s = 0; s < DP / 16; ++s) {
            const uint32_t at = (s >> 2) * (kBox >> 4) + (s & 3) * k_step(true);
            if (s < steps) mma<false, false>(score, a + at, kDescHi, b + at, kDescHi, p.idesc_s, s > 0);
        }
        mma_commit<false>(bars + 8 * (S::kScores + i));
    };
    Ring<S::kStages> ring;   // copies in the order K(0), V(0), K(1), ...
    if (mine > 0) {
        if (!mbar_wait(bars + 8 * S::kFull, 0, gave_up) || !mbar_wait(bars + 8 * (S::kQFull + i), 0, gave_up)) return;
        scores(smem + S::kAtRing);
        mma_commit<false>(bars + 8 * S::kEmpty);
        ring.next();
    }
    for (int j = 0; j < mine; ++j) {
        const uint32_t values = ring.s, b = desc_rows(smem + S::kAtRing + values * S::kTile);
        if (!mbar_wait(bars + 8 * (S::kFull + values), ring.parity, gave_up)) return;
        ring.next();
        const uint32_t keys = ring.s;
        const bool more = j + 1 < mine;
        if (more && !mbar_wait(bars + 8 * (S::kFull + keys), ring.parity, gave_up)) return;
        if (ragged && j == n - 1 && !mbar_wait(bars + 8 * S::kClear, 0, gave_up)) return;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (!mbar_wait(bars + 8 * (S::kTerms + 2 * i + half), j & 1, gave_up)) return;
            tc_fence_after();
#pragma unroll
            for (int s = 4 * half; s < 4 * half + 4; ++s)
                mma_tmem(sum, score + s * 8, b + s * k_step(false), kDescHi, p.idesc_o, j > 0 || s > 0);
        }
        if (more) scores(smem + S::kAtRing + keys * S::kTile);
        mma_commit<false>(bars + 8 * (S::kSums + i));
        mma_commit<false>(bars + 8 * (S::kEmpty + values));
        if (more) {
            mma_commit<false>(bars + 8 * (S::kEmpty + keys));
            ring.next();
        }
    }
    // copies that only the other tile reads: both lanes free a stage
    for (int c = 2 * mine; c < 2 * n; ++c, ring.next()) {
        if (!mbar_wait(bars + 8 * (S::kFull + ring.s), ring.parity, gave_up)) return;
        mbar_arrive(bars + 8 * (S::kEmpty + ring.s));
    }
}

// The rows of the last values that are behind the sequence, other sequences' perhaps: zero,
// for the product contracts over them.  By the loading warp, once all copies are under way
// (no stage is filled again, so the barrier's parity tells the last copy).
template <int DP, int TILES>
__device__ __forceinline__ void clear_values(const Work& w, int n, uint32_t smem, uint32_t bars, int lane, volatile int* gave_up)
{
    using S = Shape<DP, TILES>;
    const int live = w.seq.lk - (w.from + n - 1) * kRows;
    if (live >= kRows || *gave_up) return;
    const uint32_t copy = 2 * n - 1;
    if (!__all_sync(0xffffffffu, mbar_wait(bars + 8 * (S::kFull + copy % S::kStages), copy / S::kStages & 1, gave_up))) return;
    zero_rows<S::kChunks>(smem + S::kAtRing + copy % S::kStages * S::kTile, live, lane);
    if (lane == 0) mbar_arrive(bars + 8 * S::kClear);
}

// A row a thread: i the tile, r the row.
template <int T, int DP, int TILES>
__device__ __forceinline__ void softmax(const Params& p, const Work& w, int i, int r, uint32_t bars, uint32_t tmem, volatile int* gave_up)
{
    using S = Shape<DP, TILES>;
    const int n = i ? w.n[1] : w.n[0], t0 = w.t0 + i * p.tokens;
    const int token = t0 + r / p.group, head = (int)w.head * p.group + r % p.group;
    const bool live = r < p.tokens * p.group && token < w.seq.lq;
    const int seen = keys_seen(w.seq, token, p.causal);                 // this row's keys
    const int all = keys_seen(w.seq, t0, p.causal);                     // every row's
    const uint32_t scores = tmem + i * 128, sums = tmem + S::kTmemO + i * DP;
    const float up = T == GS_F16 ? (float)held_up(w.seq.lk) : 0.0f;
    float m = -INFINITY;
    uint64_t l2[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)};
    bool ok = true;
    for (int j = 0; j < n; ++j) {
        ok = __all_sync(0xffffffffu, mbar_wait(bars + 8 * (S::kScores + i), j & 1, gave_up));
        if (!ok) break;
        tc_fence_after();
        uint32_t s[128];
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        const int first = (w.from + j) * kRows, left = seen - first;
        const bool cut = first + kRows > all;
        tmem_ld32(scores, s);
        tmem_ld32_wait(s);
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
            if (c < 96) tmem_ld32(scores + c + 32, s + c + 32);   // on its way while these are compared
            if (cut) {
#pragma unroll
                for (int e = c; e < c + 32; ++e)
                    if (e >= left) s[e] = 0xff800000u;   // -infinity, whatever the hidden key gave
            }
#pragma unroll
            for (int e = c; e < c + 32; e += 8)
#pragma unroll
                for (int k = 0; k < 4; ++k) top[k] = max3(top[k], __uint_as_float(s[e + k]), __uint_as_float(s[e + 4 + k]));
            if (c < 96) tmem_ld32_wait(s + c + 32);
        }
        const float new_m = max3(fmaxf(top[0], top[1]), top[2], top[3]) * p.scale2;
        const bool raise = new_m > m + (kMost - up);   // from -infinity: by any score
        if (j == 0) m = new_m;
        else if (__any_sync(0xffffffffu, raise)) {
            // the sums so far, to the new maximum: the product that last added to them is done
            const float to = raise ? new_m : m, by = m == to ? 1.0f : exp2_fast(m - to);
            ok = __all_sync(0xffffffffu, mbar_wait(bars + 8 * (S::kSums + i), (j - 1) & 1, gave_up));
            if (!ok) break;
            tc_fence_after();
            m = to;
#pragma unroll
            for (int e = 0; e < 2; ++e) l2[e] = mul2(l2[e], pair(by, by));
#pragma unroll 1
            for (int c = 0; c < DP; c += 32) {
                uint32_t o[32];
                tmem_ld32(sums + c, o);
                tmem_ld32_wait(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * by);
                tmem_st32(sums + c, o);
            }
        }
        const float less = m == -INFINITY ? 0.0f : up - m;   // no key yet: every term 0
        const uint64_t scale = pair(p.scale2, p.scale2), minus = pair(less, less);
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
            uint32_t h[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float2 x = unpair(fma2(pair(__uint_as_float(s[c + 2 * e]), __uint_as_float(s[c + 2 * e + 1])), scale, minus));
                const float a = exp2_fast(x.x), b = exp2_fast(x.y);
                l2[e & 1] = add2(l2[e & 1], pair(a, b));
                h[e] = pack_half2(a, b, T);
            }
            tmem_st16(scores + c / 2, h);
            if (c & 32) {   // a half of the terms, whose product starts with it
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if ((threadIdx.x & 31) == 0) mbar_arrive(bars + 8 * (S::kTerms + 2 * i + c / 64));
            }
        }
    }
    if (n > 0 && ok) ok = __all_sync(0xffffffffu, mbar_wait(bars + 8 * (S::kSums + i), (n - 1) & 1, gave_up));
    if (!ok) return;
    tc_fence_after();
    const float2 la = unpair(l2[0]), lb = unpair(l2[1]);
    const float l = (la.x + la.y) + (lb.x + lb.y);
    const int64_t row = w.seq.q0 + token;
    if (p.splits > 1) {
        const int64_t at = ((int64_t)w.split * p.seqs.q_rows + row) * (p.group * p.kv_heads) + head;
        if (live) p.part_stats[at] = make_float2(m - up, l);
        if (n == 0) return;
        float* to = p.part + at * DP;
#pragma unroll 1
        for (int c = 0; c < DP; c += 32) {
            uint32_t o[32];
            tmem_ld32(sums + c, o);
            tmem_ld32_wait(o);
            if (live)
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<uint4*>(to + c + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
    } else {
        const bool none = l == 0.0f;
        if (live && p.lse) p.lse[row * (p.group * p.kv_heads) + head] = none ? -INFINITY : (m - up + log2f(l)) * kLn2;
        const float by = none ? 0.0f : 1.0f / l;
        uint16_t* to = p.o + row * p.o_row + head * p.o_head;
#pragma unroll 1
        for (int c = 0; c < DP; c += 32) {
            float v[32];
            uint32_t o[32];
            if (n > 0) {
                tmem_ld32(sums + c, o);
                tmem_ld32_wait(o);
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = n > 0 && !none ? __uint_as_float(o[e]) * by : 0.0f;
            if (live && c < p.dim) store_row32<T>(to, c, p.dim, p.o_vec, v);
        }
    }
    tc_fence_before();
}

template <int T, int DP, int TILES>
__global__ void __launch_bounds__(Shape<DP, TILES>::kThreads, 3 - TILES) attention_kernel(const __grid_constant__ Params p)
{
    using S = Shape<DP, TILES>;
    extern __shared__ __align__(1024) char smem_raw[];
    const uint32_t smem = smem_addr(smem_raw);
    if (smem & 1023u) {   // every thread sees the same address; there is no padding to move within
        g_attention_wait_expired = 1;
        return;
    }
    const uint32_t bars = smem + S::kAtBars;
    char* tail = smem_raw + S::kAtBars + ((S::kBars * 8 + 15) & ~15);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail);
    volatile int* gave_up = reinterpret_cast<volatile int*>(tail + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kBars; ++i)
            mbar_init(bars + 8 * i, i >= S::kTerms && i < S::kSums ? 4 : (i >= S::kEmpty && i < S::kScores ? TILES : 1));
        *gave_up = 0;
        mbar_init_fence();
    }
    wait_for_predecessor_alone();
    if (p.zero) fill_rows(p.fill, p.seqs.q_starts, p.seqs.count, p.seqs.q_rows);
    Work w;
    if (!find_work<TILES>(p, w)) return;   // the same for every warp
    if (warp == S::kSoftmaxWarps) tmem_alloc<false>(smem_addr(tmem_slot), S::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    let_successor_start();
    const int n = w.n[0] > w.n[1] ? w.n[0] : w.n[1];

    if (warp >= S::kSoftmaxWarps) {
        few_registers();
        const int i = warp - S::kSoftmaxWarps - 1;
        if (i < 0) {
            if (n > 0) {
                if (elect_one()) load<DP, TILES>(p, w, n, smem, bars, gave_up);
                __syncwarp();
                clear_values<DP, TILES>(w, n, smem, bars, lane, gave_up);
            }
        } else if (i < TILES && elect_one()) {
            issue<DP, TILES>(p, w, i, n, smem, bars, tmem, gave_up);
            mma_commit<false>(bars + 8 * (S::kDone + i));   // the block does not leave before its products are done
            if (!mbar_wait_alone(bars + 8 * (S::kDone + i), 0)) *gave_up = 1;
        }
    } else {
        many_registers<TILES == 2 ? 224 : 200>();
        const int i = warp >> 2, r = threadIdx.x & 127;
        if (w.t0 + i * p.tokens < w.seq.lq)
            softmax<T, DP, TILES>(p, w, i, r, bars, tmem + ((uint32_t)((warp & 3) * 32) << 16), gave_up);
    }
    __syncthreads();
    if (threadIdx.x == 0 && *gave_up) atomicExch(&g_attention_wait_expired, 1);
    if (warp == S::kSoftmaxWarps) {
        tc_fence_after();
        tmem_free<false>(tmem, S::kTmemCols);
    }
}

// The parts of a row's keys: o = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s.  A block a
// row: its warps take the parts in turn, their sums are added in order.  (A warp a row waited
// for one part after the other: 20 us for 33 of them, 4 so.)
constexpr int kJoinWarps = 8;
template <int T, int DP>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ Params p)
{
    __shared__ float sums[kJoinWarps][DP + 1];
    wait_for_predecessor();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t heads = p.group * p.kv_heads, all = p.seqs.q_rows * heads, row = blockIdx.x / heads;
    if (p.seqs.q_starts && (row < p.seqs.q_starts[0] || row >= p.seqs.q_starts[p.seqs.count])) return;   // of no sequence
    const float2* stats = p.part_stats + blockIdx.x;
    const float* part = p.part + (int64_t)blockIdx.x * DP;
    float m = -INFINITY;
    for (uint32_t s = lane; s < p.splits; s += 32) m = fmaxf(m, stats[s * all].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    constexpr int kPer = DP / 32;
    float l = 0.0f, v[kPer] = {};
#pragma unroll 4
    for (uint32_t s = warp; s < p.splits; s += kJoinWarps) {
        const float2 st = stats[s * all];
        if (st.y == 0.0f) continue;   // no key of this part is seen; of no keys at all there is nothing to read
        const float by = exp2_fast(st.x - m);
        const float* from = part + s * all * DP + lane * kPer;
        l = __fmaf_rn(by, st.y, l);
        float t[kPer];
        if constexpr (kPer == 4) *reinterpret_cast<float4*>(t) = *reinterpret_cast<const float4*>(from);
        else *reinterpret_cast<float2*>(t) = *reinterpret_cast<const float2*>(from);
#pragma unroll
        for (int e = 0; e < kPer; ++e) v[e] = __fmaf_rn(by, t[e], v[e]);
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) sums[warp][lane * kPer + e] = v[e];
    if (lane == 0) sums[warp][DP] = l;
    __syncthreads();
    const int c = threadIdx.x;
    if (c > DP) return;
    float total = 0.0f, mine = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) total += sums[w][DP], mine += sums[w][c];
    const bool none = total == 0.0f;
    if (c == DP && p.lse) p.lse[blockIdx.x] = none ? -INFINITY : (m + log2f(total)) * kLn2;
    if (c < p.dim) store_elem(p.o + row * p.o_row + (blockIdx.x - row * heads) * p.o_head, c, T, none ? 0.0f : mine / total);
}

__global__ void __launch_bounds__(256) pack_kernel(const __grid_constant__ PackList p)
{
    wait_for_predecessor();
    int j = 0;
    while (j + 1 < p.jobs && blockIdx.x >= p.job[j + 1].first) ++j;
    const auto& q = p.job[j];
    const unsigned blocks = (j + 1 < p.jobs ? p.job[j + 1].first : p.blocks) - q.first;
    const int64_t lines = q.rows * q.heads;   // a warp a line
    for (int64_t i = (int64_t)(blockIdx.x - q.first) * 8 + (threadIdx.x >> 5); i < lines; i += (int64_t)blocks * 8) {
        const int64_t r = i / q.heads, h = i - r * q.heads;
        for (int c = threadIdx.x & 31; c < p.dim; c += 32) q.to[i * p.pitch + c] = q.from[r * q.row + h * q.head + c];
    }
}

}  // namespace

bool tensor_ok(const void* p, int64_t row, int64_t head, int64_t rows, int64_t heads, int64_t dim, bool out)
{
    constexpr int64_t most = 1ll << 38;   // the tensor copies take strides below 2^40 bytes
    if (!p || ((uintptr_t)p & 1u)) return false;
    if (rows > 1 && (row < dim || row > most)) return false;
    if (heads > 1 && (head < dim || head > most)) return false;
    if (!out || rows <= 1 || heads <= 1) return true;
    return row >= (heads - 1) * head + dim || (__int128)head >= (__int128)(rows - 1) * row + dim;
}
bool tensor_tma(const void* p, int64_t row, int64_t head, int64_t rows, int64_t heads)
{
    return aligned16(p) && (rows <= 1 || row % 8 == 0) && (heads <= 1 || head % 8 == 0);
}
int tensor_vec(const void* p, int64_t row, int64_t head, int64_t rows, int64_t heads)
{
    const uint64_t bits = (uint64_t)(uintptr_t)p | (rows > 1 ? (uint64_t)row * 2 : 0) | (heads > 1 ? (uint64_t)head * 2 : 0);
    return bits % 32 == 0 ? 2 : (bits % 16 == 0 ? 1 : 0);
}

Tensor3 PackList::add(const Tensor3& t, int64_t rows, int64_t heads, int64_t d, char*& to)
{
    if (tensor_tma(t.p, t.row, t.head, rows, heads)) return t;
    dim = (int)d, pitch = (int)round_up(d, 8);
    const int64_t want = (rows * heads + 63) / 64;   // eight lines a warp
    job[jobs++] = {(const uint16_t*)t.p, (uint16_t*)to, t.row, t.head, rows, (int)heads, blocks};
    blocks += (unsigned)(want < 1216 ? want : 1216);
    const Tensor3 r = {to, pitch * heads, pitch};
    to += packed_bytes(rows, heads, d);
    return r;
}
gs_status PackList::run(cudaStream_t st) const
{
    return blocks ? launch_after(pack_kernel, dim3(blocks), 256, 0, 1, st, *this) : GS_OK;
}

gs_status forward_wait_report(int* expired)
{
    const int zero = 0;
    GS_CUDA_TRY(cudaMemcpyFromSymbol(expired, g_attention_wait_expired, sizeof *expired));
    if (*expired) GS_CUDA_TRY(cudaMemcpyToSymbol(g_attention_wait_expired, &zero, sizeof zero));
    return GS_OK;
}

namespace {

// How a call is cut: tiles of a unit, and parts of the keys.
struct Plan {
    int group, tokens, tiles, dp;
    uint32_t splits;
    int64_t units, items;   // units at most; times key heads and splits
    size_t part, stats;     // bytes of the parts' sums and of their maxima
    size_t packs, bytes;
};

Plan plan_for(const gs_attention_args& a)
{
    Plan r = {};
    r.group = a.heads / a.kv_heads;
    r.tokens = kRows / r.group;
    r.dp = a.dim <= 64 ? 64 : 128;
    const int known = device_sms();
    const int64_t sms = known > 0 ? known : 152;
    const bool starts = a.q_starts != nullptr;
    const int64_t one = units_at_most(a.q_rows, a.sequences, starts, r.tokens);
    const int64_t two = units_at_most(a.q_rows, a.sequences, starts, 2 * (int64_t)r.tokens);
    const int64_t sequences = a.sequences > 0 ? a.sequences : 1, keys = a.k_rows / sequences;
    // Two tiles a CTA read their keys once; two CTAs an SM hide each other's first and last
    // steps, and for 64 columns and fewer, where the softmax bounds both, each other's
    // barriers.  us with one and two: 8192 tokens of 64 causal 162, 185; 24 sequences of up to
    // 1024 56, 66; of 128: 64 x 512 151, 163; 16 x 2048 293, 310; 4099 69, 69; 16384 463, 416.
    r.tiles = r.dp == 128 && keys >= 4096 && a.q_rows > sequences * r.tokens && two * a.kv_heads >= sms ? 2 : 1;
    r.units = r.tiles == 2 ? two : one;
    r.splits = 1;
    const int64_t ctas = r.units * a.kv_heads, key_tiles = (keys + kRows - 1) / kRows;
    const int64_t rows = ((a.q_rows + sequences - 1) / sequences < r.tokens ? (a.q_rows + sequences - 1) / sequences : r.tokens) * r.group;
    if (r.tiles == 1 && key_tiles > 1 && (ctas < sms || rows <= 32) && a.q_rows * a.heads <= 0x7fffffffll) {
        // Parts of the keys: what they save in waiting, of a CTA alone (1.4 us a tile of keys) or
        // for the last one (a third of its share of HBM's time), against a wave's start and end
        // and the parts' sums.  us by parts: 1 token against 4097 keys 39 (1), 13 (8), 11 (32), 65536
        // keys 765 (1), 22 (64); 32 tokens against up to 16384 keys 306 (1), 251 (4), 244 (8),
        // 264 (24); 64 against up to 2000 82 (1), 88 (2).
        const double slots = 2.0 * sms, tile_bytes = 512.0 * r.dp, byte_us = 1.0 / 6.5e6;
        double best = 0;
        for (int64_t s = 1; s <= key_tiles && s <= 256; ++s) {
            const int64_t each = (key_tiles + s - 1) / s;
            if (s > 1 && (key_tiles + s - 2) / (s - 1) == each) continue;   // fewer parts are as long
            const double waves = std::ceil((double)(ctas * s) / slots), busy = (double)(ctas * s) < slots ? (double)(ctas * s) : slots;
            const double tile_us = 1.4 > tile_bytes * busy * byte_us ? 1.4 : tile_bytes * busy * byte_us;
            const double work = (double)(ctas * key_tiles) * tile_bytes * byte_us, alone = waves * (double)each * 1.4;
            const double us = (work > alone ? work : alone) + waves + 0.3 * (double)each * tile_us +
                              (s > 1 ? 2.5 + 0.05 * (double)s + (double)(a.q_rows * a.heads * s) * r.dp * 8 / 4e6 : 0.0);
            if (s == 1 || us < best) best = us, r.splits = (uint32_t)s;
        }
    }
    r.items = ctas * r.splits;
    if (r.splits > 1) {
        r.part = (size_t)(r.splits * a.q_rows * a.heads * r.dp * 4);   // a multiple of 256
        r.stats = (size_t)round_up(r.splits * a.q_rows * a.heads * 8, 256);
    }
    if (!tensor_tma(a.q, a.q_row, a.q_head, a.q_rows, a.heads)) r.packs += packed_bytes(a.q_rows, a.heads, a.dim);
    if (!tensor_tma(a.k, a.k_row, a.k_head, a.k_rows, a.kv_heads)) r.packs += packed_bytes(a.k_rows, a.kv_heads, a.dim);
    if (!tensor_tma(a.v, a.v_row, a.v_head, a.k_rows, a.kv_heads)) r.packs += packed_bytes(a.k_rows, a.kv_heads, a.dim);
    r.bytes = r.part + r.stats + r.packs;
    return r;
}

template <int T, int DP, int TILES>
gs_status launch(const Params& p, const Plan& plan, cudaStream_t st)
{
    using S = Shape<DP, TILES>;
    static std::atomic<uint64_t> done{0};
    gs_status s = allow_smem(attention_kernel<T, DP, TILES>, S::kSmem, done);
    if (s != GS_OK) return s;
    s = launch_after(attention_kernel<T, DP, TILES>, dim3((unsigned)plan.items), S::kThreads, S::kSmem, 1, st, p);
    if (s != GS_OK || plan.splits == 1) return s;
    return launch_after(join_kernel<T, DP>, dim3((unsigned)(p.seqs.q_rows * plan.group * p.kv_heads)), kJoinWarps * 32, 0, 1, st, p);
}

}  // namespace
}  // namespace attn
}  // namespace gs

using namespace gs;
using namespace gs::attn;

extern "C" gs_status gs_attention(const gs_attention_args* args, void* ws, size_t* ws_bytes, void* stream)
{
    GS_NVTX_RANGE("gs_attention");
    if (!args) return GS_ERR_INVALID_ARG;
    const gs_attention_args& a = *args;
    if (!sizes_ok(a.q_rows, a.k_rows, a.sequences, a.heads, a.kv_heads, a.dim, a.type, a.scale, a.q_starts, a.k_starts))
        return GS_ERR_INVALID_ARG;
    if (((uintptr_t)a.k_lengths & 3u) || ((uintptr_t)a.lse & 3u)) return GS_ERR_INVALID_ARG;
    if (a.q_rows > 0 && (!tensor_ok(a.q, a.q_row, a.q_head, a.q_rows, a.heads, a.dim, false) ||
                         !tensor_ok(a.o, a.o_row, a.o_head, a.q_rows, a.heads, a.dim, true)))
        return GS_ERR_INVALID_ARG;
    if (a.k_rows > 0 && (!tensor_ok(a.k, a.k_row, a.k_head, a.k_rows, a.kv_heads, a.dim, false) ||
                         !tensor_ok(a.v, a.v_row, a.v_head, a.k_rows, a.kv_heads, a.dim, false)))
        return GS_ERR_INVALID_ARG;
    const Plan plan = plan_for(a);
    if (plan.items > 0x7fffffffll) return GS_ERR_INVALID_ARG;
    const WsCheck wc = ws_check(ws, ws_bytes, plan.bytes);
    if (wc == WsCheck::kBad) return GS_ERR_INVALID_ARG;
    if (wc == WsCheck::kQuery) return GS_OK;
    if (a.q_rows == 0) return GS_OK;
    cudaStream_t st = (cudaStream_t)stream;
    Params p = {};
    char* to = (char*)ws + plan.part + plan.stats;
    PackList packs;
    const Tensor3 q = packs.add({a.q, a.q_row, a.q_head}, a.q_rows, a.heads, a.dim, to);
    gs_status s = tile_map(&p.q, q, a.type, a.q_rows, a.heads, a.dim, plan.group, plan.tokens);
    if (s == GS_OK && a.k_rows > 0) {   // without keys nothing is read from them
        const Tensor3 k = packs.add({a.k, a.k_row, a.k_head}, a.k_rows, a.kv_heads, a.dim, to);
        const Tensor3 v = packs.add({a.v, a.v_row, a.v_head}, a.k_rows, a.kv_heads, a.dim, to);
        s = tile_map(&p.k, k, a.type, a.k_rows, a.kv_heads, a.dim, 1, kRows);
        if (s == GS_OK) s = tile_map(&p.v, v, a.type, a.k_rows, a.kv_heads, a.dim, 1, kRows);
    }
    if (s == GS_OK) s = packs.run(st);
    if (s != GS_OK) return s;
    p.seqs = {a.q_starts, a.k_starts, a.k_lengths, a.q_rows, a.k_rows, (uint32_t)a.sequences};
    p.fill = {(uint16_t*)a.o, a.o_row, a.o_head, a.lse, a.heads, a.dim};
    p.zero = a.fill && a.q_starts;
    p.o = (uint16_t*)a.o, p.o_row = a.o_row, p.o_head = a.o_head, p.lse = a.lse;
    p.part = (float*)ws, p.part_stats = (float2*)((char*)ws + plan.part);
    p.scale2 = a.scale * kLog2e;
    p.splits = plan.splits, p.kv_heads = (uint32_t)a.kv_heads, p.group = plan.group, p.tokens = plan.tokens;
    p.dim = a.dim, p.causal = a.causal != 0;
    p.o_vec = tensor_vec(a.o, a.o_row, a.o_head, a.q_rows, a.heads);
    p.idesc_s = instr_desc(a.type, true, true, kRows, kRows);
    p.idesc_o = instr_desc(a.type, true, false, (int)round_up(a.dim, 16), kRows);
    const auto run = [&](auto type) {
        constexpr int T = decltype(type)::value;
        if (plan.dp == 64) return launch<T, 64, 1>(p, plan, st);
        return plan.tiles == 1 ? launch<T, 128, 1>(p, plan, st) : launch<T, 128, 2>(p, plan, st);
    };
    return a.type == GS_BF16 ? run(std::integral_constant<int, GS_BF16>()) : run(std::integral_constant<int, GS_F16>());
}
