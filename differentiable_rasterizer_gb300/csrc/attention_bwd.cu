// attention_bwd.cu -- the gradients of attention over packed sequences.
//
//   p = exp(scale q k^T - lse),  r = do v^T,  delta = sum of p r (a row),  ds = p (r - delta)
//   dv = p^T do,  dk = scale ds^T q,  dq = scale ds k
//
// Scores and r are computed again from the tiles, so that nothing of the size of queries
// times keys is stored.  Three launches: delta, one or two tiles of queries a CTA against
// their keys; dk and dv, a tile of keys a CTA against its queries (where tiles are few, against
// a part of them, and a fourth launch adds the parts in order); dq, tiles of queries again.
// dq could come out of the second's products, but its sum runs over the CTAs there: atomics
// would make its bits depend on the run.  delta is do . o, but o has been rounded: in bf16
// that alone puts 4e-3 of dq's norm (where few keys carry the weight, 1e-2) beside the 2e-3 of
// the factors' and results' roundings, for delta multiplies the keys' mean, and dq is what
// remains of the keys beside it.  So nine products of a pair of tiles in place of five.  (The
// forward holds o in fp32 and could hand on what o's rounding leaves, in 16 bits more: an output
// and an argument that the calls do not have.)
//
// The kernels keep p and ds out of shared memory: a tile's scores are computed with the
// rows that stay (keys, or queries) as TMEM lanes, p and ds take their place in TMEM as 16
// bits, and are the first factor of the next products from there.
//
// p and ds are rounded to 16 bits because the tensor cores take 16-bit factors: with the
// results' own rounding, 2.4e-3 of a gradient's norm in bf16.  ds in two 16-bit parts leaves dq
// with its own rounding, 1.7e-3, but four products a tile where there were three: all gradients
// 1634 -> 1818 us, 469 -> 522 for 4096 tokens of 16 heads; one part.
//
// What bounds them: the chain of waits from scores to terms to the next scores; 16384 tokens, 8
// heads of 128, causal, bf16: delta 255 us, dk and dv 834, dq 482 (two tiles a CTA hide each
// other's chains; a tile of keys has its SM to itself, 3,170 cycles a tile of queries where
// the four products take 2,050).
//
// f16 holds neither small p nor small ds among its normal numbers: p is taken times 2^12
// (at most 1 times that), ds times the power of two that brings its bound, 2 dim max|do|
// max|v|, to 2^15; the sums are scaled back at the end.  v's maximum is that of the sequence and
// key head, do's that of the row for dq, whose rows are TMEM lanes, and of the sequence's
// rows and the key head for dk, which sums over them: rows of no sequence and other
// sequences change nothing.  A launch behind delta's takes the maxima.
#include <atomic>
#include <cmath>

#include "attention.cuh"

namespace gs {
namespace attn {
namespace {

constexpr int kKeyWarps = 16, kKeyThreads = (kKeyWarps + 4) * 32, kTmemCols = 512;
constexpr int kStatRows = kRows + 4;   // of a copy of row statistics, which starts on 16 bytes

__device__ int g_attention_bwd_wait_expired;

// log2 of what p is held times as a factor.
template <int T>
constexpr float kUp = T == GS_F16 ? 12.0f : 0.0f;
template <int T>
constexpr float kDown = T == GS_F16 ? 0x1p-12f : 1.0f;

struct Params {
    CUtensorMap q, k, v, d_o;
    Sequences seqs;
    Fill fill_dq, fill_dk, fill_dv;
    float* stats;            // planes of [key head][token][head of the group]: kUp - lse log2(e) (-infinite for a row that sees no key), -delta
    const float* lse;
    float* most;             // F16: a sequence's and key head's largest finite |do|; behind them |v|; a row's |do| in a third plane of stats
    uint16_t *dq, *dk, *dv;
    int64_t dq_row, dq_head, dk_row, dk_head, dv_row, dv_head;
    int64_t stat_pitch, stat_plane;   // of a key head; to the second plane
    float* part;             // parts > 1: [part][key row][key head][dv, dk][DP] sums
    float scale, scale2;     // scale2: scale log2(e)
    uint32_t kv_heads, parts;
    int group, tokens, dim, causal, zero, dq_vec, dk_vec, dv_vec;
    uint32_t idesc_s, idesc_d;
};

// ------------------------------------------------------------------ F16's largest values
// Infinities and NaN are left out: what they reach is not finite whatever the power, and the
// rest keeps its digits.  So are, for dk, rows of do that see no key.
struct MostParams {
    const uint16_t *d_o, *v;
    int64_t do_row, do_head, v_row, v_head;
    Sequences seqs;
    const float* lse;        // of do's rows
    float* row_most;         // of do's rows, laid out as stats
    uint32_t* most;          // [2][sequences][key heads] bits of |do| and |v|, cleared by delta's launch
    int64_t stat_pitch, q_each, k_each;   // rows of a block, multiples of kMostRows
    uint32_t q_blocks, q_chunks, k_chunks;   // blocks of do; of a key head, do's and v's
    uint32_t kv_heads;
    int group, dim, do_vec, v_vec;
};
constexpr int kMostRows = 16;   // at a time, sixteen lanes each

// A block some rows of a key head: of do (all heads of the group) or of v.  Sixteen lanes a
// row, eight elements a lane.  Magnitudes are compared as bits, so that the order of the
// atomics does not matter; one a block for each sequence that its last rows are of (with one
// for each sixteen lanes all gradients of 5 x 1111 queries on 2049 keys, six heads of 72, took
// 10 us more: they wait for one another at a long sequence's place).
__global__ void __launch_bounds__(256) most_kernel(const __grid_constant__ MostParams p)
{
    __shared__ uint32_t at_end[2][kMostRows];
    wait_for_predecessor();
    const bool is_do = blockIdx.x < p.q_blocks;
    const uint32_t i = is_do ? blockIdx.x : blockIdx.x - p.q_blocks, chunks = is_do ? p.q_chunks : p.k_chunks;
    const uint32_t head = i / chunks;
    const int64_t rows = is_do ? p.seqs.q_rows : p.seqs.k_rows, each = is_do ? p.q_each : p.k_each, start = (int64_t)(i % chunks) * each;
    const int64_t end = start + each < rows ? start + each : rows;
    const int32_t* starts = is_do ? p.seqs.q_starts : p.seqs.k_starts;
    const int heads = is_do ? p.group : 1, vec = is_do ? p.do_vec : p.v_vec;
    const int64_t pitch = is_do ? p.do_row : p.v_row, head_pitch = is_do ? p.do_head : p.v_head;
    const uint16_t* from = (is_do ? p.d_o : p.v) + (int64_t)head * heads * head_pitch;
    uint32_t* most = p.most + (is_do ? 0 : (int64_t)p.seqs.count * p.kv_heads) + head;
    const int sub = threadIdx.x % 16, col = sub * 8;
    uint32_t s = p.seqs.count, top = 0;   // the sequence so far and its largest
    int64_t first = 0, last = 0;          // its rows
    const auto flush = [&] {
        if (sub == 0 && s < p.seqs.count && top > 0) {
            uint32_t* to = most + (int64_t)s * p.kv_heads;
            if (*(volatile uint32_t*)to < top) atomicMax(to, top);
        }
    };
    // whole warps run the same number of rounds: each is two rows
    for (int64_t row0 = start; row0 < end; row0 += kMostRows) {
        const int64_t row = row0 + threadIdx.x / 16;
        uint32_t mine = 0;
#pragma unroll 4
        for (int h = 0; h < heads; ++h) {
            uint32_t m = 0;
            if (row < end && col < p.dim) {
                const uint16_t* at = from + row * pitch + h * head_pitch + col;
                uint32_t w[4];
                if (vec) {
                    const uint4 q = *reinterpret_cast<const uint4*>(at);
                    w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
                } else
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = (col + 2 * e < p.dim ? at[2 * e] : 0u) | (col + 2 * e + 1 < p.dim ? (uint32_t)at[2 * e + 1] : 0u) << 16;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t lo = w[e] & 0x7fffu, hi = w[e] >> 16 & 0x7fffu;
                    if (lo < 0x7c00u && lo > m) m = lo;
                    if (hi < 0x7c00u && hi > m) m = hi;
                }
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) {
                const uint32_t other = __shfl_xor_sync(0xffffffffu, m, o);
                m = other > m ? other : m;
            }
            if (is_do && row < end) {
                if (sub == 0) p.row_most[head * p.stat_pitch + row * heads + h] = __half2float(__ushort_as_half((unsigned short)m));
                // of a row that sees no key every ds is 0
                if (p.lse[row * (int64_t)(p.kv_heads * heads) + head * heads + h] == -INFINITY) m = 0;
            }
            mine = m > mine ? m : mine;
        }
        if (row >= end) continue;
        if (row < first || row >= last) {
            flush();
            s = sequence_of(starts, p.seqs.count, row), top = 0;
            first = !starts ? 0 : (s < p.seqs.count ? starts[s] : row), last = !starts ? rows : (s < p.seqs.count ? starts[s + 1] : row + 1);
        }
        const uint32_t value = __float_as_uint(__half2float(__ushort_as_half((unsigned short)mine)));
        top = value > top ? value : top;
    }
    if (sub == 0) at_end[0][threadIdx.x / 16] = s, at_end[1][threadIdx.x / 16] = top;
    __syncthreads();
    bool mine = true;
#pragma unroll
    for (int i = 0; i < kMostRows; ++i)
        if (at_end[0][i] == s) {
            mine = mine && i >= (int)threadIdx.x / 16;   // the first with this sequence takes all
            top = at_end[1][i] > top ? at_end[1][i] : top;
        }
    if (mine) flush();
}

// The power of two that ds is held times, from the largest |do| and |v|.
template <int T>
__device__ __forceinline__ int ds_exponent(int dim, float a, float b)
{
    if constexpr (T != GS_F16) return 0;
    // finite 16-bit numbers, 2^-24 to 2^16; zeros: any power does
    const float bound = 2.0f * (float)dim * a * b;
    if (!(bound > 0.0f)) return 0;
    return 15 - (((__float_as_int(bound) >> 23) & 255) - 126);   // bound <= 2^(exponent - 126)
}
// Of v's and, for dk, of do's magnitudes in a sequence.
__device__ __forceinline__ float most_v(const Params& p, const Sequence& s, uint32_t head)
{
    return p.most[((int64_t)p.seqs.count + s.number) * p.kv_heads + head];
}
__device__ __forceinline__ float most_do(const Params& p, const Sequence& s, uint32_t head) { return p.most[(int64_t)s.number * p.kv_heads + head]; }
__device__ __forceinline__ float power2(int e) { return __int_as_float((e + 127) << 23); }   // -126..127

// ------------------------------------------------------------------ dk, dv
// A CTA a tile of 128 keys of a key head.  TMEM lanes are keys:
//   S = K Q^T, R = V dO^T (columns are packed query rows), dV += P dO, dK += dS Q
// Sixteen warps, four of them 32 columns of S and R each; P and dS take the first half of
// their own columns' place.  (Eight warps of 64 columns waited for TMEM and shared memory most
// of their time: 3,440 cycles a tile, where the products take 2,050.)  The products of a tile of queries are issued as
//   dV(i), S(i + 1), dK(i), R(i + 1)
// so that P and dS are made while the other two run.
template <int DP>
struct KeyShape {
    static constexpr int kChunks = DP / 64;
    static constexpr uint32_t kTile = kChunks * kBox;
    static constexpr int kStagesQ = 3, kStagesO = DP == 128 ? 2 : 3;
    static constexpr uint32_t kAtQ = 2 * kTile, kAtO = kAtQ + kStagesQ * kTile, kAtStats = kAtO + kStagesO * kTile;
    static constexpr uint32_t kStatBytes = kStatRows * 4;   // of a plane
    static constexpr uint32_t kAtBars = kAtStats + 4 * kStatBytes;
    static constexpr int kKV = 0, kQFull = 1, kQEmpty = kQFull + kStagesQ, kOFull = kQEmpty + kStagesQ, kOEmpty = kOFull + kStagesO,
                         kStatFull = kOEmpty + kStagesO, kStatEmpty = kStatFull + 2, kS = kStatEmpty + 2, kR = kS + 1, kP = kR + 1,
                         kDs = kP + 1, kClearQ = kDs + 1, kClearO = kClearQ + 1, kDone = kClearO + 1, kBars = kDone + 2;
    static constexpr int kSmem = kAtBars + ((kBars * 8 + 15) & ~15) + 16;
    static_assert(kSmem <= 232448 && kStatBytes % 16 == 0, "shared memory of an SM");
};
constexpr uint32_t kTmemR = 128, kTmemDv = 256;   // S at 0, R, dV, dK at kTmemDv + DP

struct KeyWork {
    Sequence seq;
    uint32_t head;
    int key0, first, n;   // first key; first token of the first tile of queries; tiles
    int each;             // tiles of a part
};
// Work number i: a tile of keys of a head, all of its queries.
__device__ __forceinline__ bool find_keys(const Params& p, uint32_t i, KeyWork& w)
{
    uint32_t unit, units;
    w.head = i % p.kv_heads;
    if (!find_unit<true>(p.seqs, i / p.kv_heads, kRows, w.seq, unit, units)) return false;
    w.key0 = (int)unit * kRows;          // the first keys are seen by the most queries
    w.first = first_query(w.seq, w.key0, p.causal);
    const int left = w.seq.lq - w.first;
    w.n = left <= 0 ? 0 : (left + p.tokens - 1) / p.tokens;
    w.each = (w.n + (int)p.parts - 1) / (int)p.parts;
    return true;
}
// A part of them.
__device__ __forceinline__ void take_part(const Params& p, uint32_t part, KeyWork& w)
{
    const int from = (int)part * w.each, n = w.n - from;
    w.first += from * p.tokens;
    w.n = n < 0 ? 0 : (n < w.each ? n : w.each);
}

template <int DP>
__device__ __forceinline__ void load_queries(const Params& p, const KeyWork& w, uint32_t smem, uint32_t bars, volatile int* gave_up)
{
    using S = KeyShape<DP>;
    mbar_expect(bars + 8 * S::kKV, 2 * S::kTile);
    load_tile<S::kChunks>(smem, &p.k, w.head, w.seq.k0 + w.key0, bars + 8 * S::kKV);
    load_tile<S::kChunks>(smem + S::kTile, &p.v, w.head, w.seq.k0 + w.key0, bars + 8 * S::kKV);
    const uint32_t bytes = (uint32_t)(S::kChunks * p.tokens * p.group) * 128;
    const float* stats = p.stats + w.head * p.stat_pitch;
    Ring<S::kStagesQ> rq;
    Ring<S::kStagesO> ro;
    Ring<2> rs;
    uint32_t nq = 0, no = 0, ns = 0;
    bool ok = true;
    for (int i = 0; i < w.n; ++i) {
        const int row = w.seq.q0 + w.first + i * p.tokens, head = w.head * p.group;
        ok = mbar_wait(bars + 8 * (S::kQEmpty + rq.s), rq.parity ^ 1, gave_up);
        if (!ok) break;
        mbar_expect(bars + 8 * (S::kQFull + rq.s), bytes);
        load_tile<S::kChunks>(smem + S::kAtQ + rq.s * S::kTile, &p.q, head, row, bars + 8 * (S::kQFull + rq.s));
        rq.next(), ++nq;
        ok = mbar_wait(bars + 8 * (S::kStatEmpty + rs.s), rs.parity ^ 1, gave_up);
        if (!ok) break;
        mbar_expect(bars + 8 * (S::kStatFull + rs.s), 2 * S::kStatBytes);
        const int64_t at = (int64_t)row * p.group & ~3ll;   // four are 16 bytes
#pragma unroll
        for (int plane = 0; plane < 2; ++plane)
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                             smem + S::kAtStats + (2 * rs.s + plane) * S::kStatBytes),
                         "l"(stats + plane * p.stat_plane + at), "r"(S::kStatBytes), "r"(bars + 8 * (S::kStatFull + rs.s))
                         : "memory");
        rs.next(), ++ns;
        ok = mbar_wait(bars + 8 * (S::kOEmpty + ro.s), ro.parity ^ 1, gave_up);
        if (!ok) break;
        mbar_expect(bars + 8 * (S::kOFull + ro.s), bytes);
        load_tile<S::kChunks>(smem + S::kAtO + ro.s * S::kTile, &p.d_o, head, row, bars + 8 * (S::kOFull + ro.s));
        ro.next(), ++no;
    }
    // the block does not leave before its copies have landed
    bool landed = mbar_wait_alone(bars + 8 * S::kKV, 0);
    last_copies<S::kStagesQ>(nq, [&](uint32_t s, uint32_t parity) { landed = landed && mbar_wait_alone(bars + 8 * (S::kQFull + s), parity); });
    last_copies<2>(ns, [&](uint32_t s, uint32_t parity) { landed = landed && mbar_wait_alone(bars + 8 * (S::kStatFull + s), parity); });
    last_copies<S::kStagesO>(no, [&](uint32_t s, uint32_t parity) { landed = landed && mbar_wait_alone(bars + 8 * (S::kOFull + s), parity); });
}

// Rows of the last tiles that hold no query of the sequence are other sequences': zero, for
// they are contracted over.  (Rows behind the packed ones are zeroed once, at the start.)
// By the loading warp, once all copies are under way.
template <int DP>
__device__ __forceinline__ void clear_queries(const Params& p, const KeyWork& w, uint32_t smem, uint32_t bars, int lane, volatile int* gave_up)
{
    using S = KeyShape<DP>;
    const int live = (w.seq.lq - w.first - (w.n - 1) * p.tokens) * p.group;
    if (live >= p.tokens * p.group || *gave_up) return;
    const uint32_t copy = w.n - 1, q = copy % S::kStagesQ, o = copy % S::kStagesO;
    if (!__all_sync(0xffffffffu, mbar_wait(bars + 8 * (S::kQFull + q), copy / S::kStagesQ & 1, gave_up))) return;
    zero_rows<S::kChunks>(smem + S::kAtQ + q * S::kTile, live, lane);
    if (lane == 0) mbar_arrive(bars + 8 * S::kClearQ);
    if (!__all_sync(0xffffffffu, mbar_wait(bars + 8 * (S::kOFull + o), copy / S::kStagesO & 1, gave_up))) return;
    zero_rows<S::kChunks>(smem + S::kAtO + o * S::kTile, live, lane);
    if (lane == 0) mbar_arrive(bars + 8 * S::kClearO);
}

// Two lanes issue, each the products around what it waits for: S and dV (P's), R and dK
// (dS's).  S(i + 1) takes P(i)'s place after dV(i), R(i + 1) dS(i)'s after dK(i).
template <int DP>
__device__ __forceinline__ void issue_keys(const Params& p, const KeyWork& w, bool second, uint32_t smem, uint32_t bars, uint32_t tmem,
                                           volatile int* gave_up)
{
    using S = KeyShape<DP>;
    const uint32_t steps = (uint32_t)(p.dim + 15) / 16;
    const bool ragged = (w.seq.lq - w.first - (w.n - 1) * p.tokens) * p.group < p.tokens * p.group;
    // first lane: a is K, the rows Q, the sum's rows dO; second: V, dO, Q
    const uint32_t at_rows = smem + (second ? S::kAtO : S::kAtQ), at_sum = smem + (second ? S::kAtQ : S::kAtO);
    const uint32_t rows_full = bars + 8 * (second ? S::kOFull : S::kQFull), sum_full = bars + 8 * (second ? S::kQFull : S::kOFull);
    const uint32_t rows_empty = bars + 8 * (second ? S::kOEmpty : S::kQEmpty), sum_empty = bars + 8 * (second ? S::kQEmpty : S::kOEmpty);
    const uint32_t rows_stages = second ? S::kStagesO : S::kStagesQ, sum_stages = second ? S::kStagesQ : S::kStagesO;
    const uint32_t terms = tmem + (second ? kTmemR : 0), sum = tmem + kTmemDv + (second ? DP : 0);
    const uint32_t a = desc_lo(smem + (second ? S::kTile : 0), true), done = bars + 8 * (second ? S::kR : S::kS);
    const uint32_t ready = bars + 8 * (second ? S::kDs : S::kP);
    const uint32_t rows_clear = bars + 8 * (second ? S::kClearO : S::kClearQ), sum_clear = bars + 8 * (second ? S::kClearQ : S::kClearO);
    uint32_t rs = 0, rp = 0, ss = 0, sp = 0;   // stage and parity of the next tile of rows, and of the sum's
    const auto rows_product = [&](int i) {      // [keys] x [queries]
        if (!mbar_wait(rows_full + 8 * rs, rp, gave_up) || (ragged && i == w.n - 1 && !mbar_wait(rows_clear, 0, gave_up))) return false;
        const uint32_t b = desc_lo(at_rows + rs * S::kTile, true);
#pragma unroll
        for (uint32_t s = 0; s < DP / 16; ++s) {
            const uint32_t at = (s >> 2) * (kBox >> 4) + (s & 3) * k_step(true);
            if (s < steps) mma<false, false>(terms, a + at, kDescHi, b + at, kDescHi, p.idesc_s, s > 0);
        }
        mma_commit<false>(done);
        mma_commit<false>(rows_empty + 8 * rs);
        if (++rs == rows_stages) rs = 0, rp ^= 1;
        return true;
    };
    if (!mbar_wait(bars + 8 * S::kKV, 0, gave_up) || !rows_product(0)) return;
    for (int i = 0; i < w.n; ++i) {
        if (!mbar_wait(sum_full + 8 * ss, sp, gave_up) || (ragged && i == w.n - 1 && !mbar_wait(sum_clear, 0, gave_up))) return;
        if (!mbar_wait(ready, i & 1, gave_up)) return;
        tc_fence_after();
        const uint32_t b = desc_rows(at_sum + ss * S::kTile);
#pragma unroll
        for (int s = 0; s < kRows / 16; ++s)   // quarters of 32 queries, 16 columns each, 32 apart
            mma_tmem(sum, terms + (s >> 1) * 32 + (s & 1) * 8, b + s * k_step(false), kDescHi, p.idesc_d, i > 0 || s > 0);
        if (i + 1 < w.n) {
            mma_commit<false>(sum_empty + 8 * ss);
            if (!rows_product(i + 1)) return;
        }
        if (++ss == sum_stages) ss = 0, sp ^= 1;
    }
}

__device__ __forceinline__ float ld_shared_f1(uint32_t a)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// Four consecutive statistics from the one at `at`, which lies `odd` after a multiple of
// four: a copy starts on 16 bytes, the tile's rows where they start.
struct Stats4 {
    uint64_t v[2];
    __device__ __forceinline__ void load(uint32_t at, bool even)
    {
        if (even) {
            const uint4 q = ld_shared16(at);
            v[0] = pair(__uint_as_float(q.x), __uint_as_float(q.y)), v[1] = pair(__uint_as_float(q.z), __uint_as_float(q.w));
        } else
            v[0] = pair(ld_shared_f1(at), ld_shared_f1(at + 4)), v[1] = pair(ld_shared_f1(at + 8), ld_shared_f1(at + 12));
    }
};
__device__ __forceinline__ uint64_t both(float v) { return pair(v, v); }

// A key a thread (row r of the tile), 32 columns: those of `quarter`.
template <int T, int DP>
__device__ __forceinline__ void key_terms(const Params& p, const KeyWork& w, int quarter, int r, uint32_t smem, uint32_t bars, uint32_t tmem,
                                          int exponent, volatile int* gave_up)
{
    using S = KeyShape<DP>;
    const uint64_t by_ds = both(power2(exponent) * kDown<T>), scale2 = both(p.scale2);
    const int key = w.key0 + r;
    const uint32_t mine = tmem + quarter * 32;
    bool ok = true;
    Ring<2> rs;
    for (int i = 0; i < w.n; ++i, rs.next()) {
        const int t0 = w.first + i * p.tokens;
        // columns of this tile that count for this key: from the first query that sees it to the last of the sequence
        const Columns all = columns_of(w.seq, key, t0, p.tokens, p.group, p.causal);
        const int from = all.from - quarter * 32, to = all.to - quarter * 32;
        const bool cut = to < 32 || __any_sync(0xffffffffu, from > 0);
        const uint32_t odd = (uint32_t)((int64_t)(w.seq.q0 + t0) * p.group) & 3;
        const uint32_t stats = smem + S::kAtStats + 2 * rs.s * S::kStatBytes + (odd + (uint32_t)quarter * 32) * 4;
        ok = __all_sync(0xffffffffu, mbar_wait(bars + 8 * (S::kStatFull + rs.s), rs.parity, gave_up) &&
                                         mbar_wait(bars + 8 * S::kS, i & 1, gave_up));
        if (!ok) break;
        tc_fence_after();
        uint32_t s[32], h[16];
        tmem_ld32(mine, s);
        Stats4 l[4];   // half of them at a time
#pragma unroll
        for (int e = 0; e < 4; ++e) l[e].load(stats + e * 16, odd == 0);
        tmem_ld32_wait(s);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            Stats4& q = l[e / 2 & 3];
            const float2 x = unpair(fma2(pair(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), scale2, q.v[e & 1]));
            s[2 * e] = __float_as_uint(exp2_fast(x.x)), s[2 * e + 1] = __float_as_uint(exp2_fast(x.y));
            if (e < 8 && (e & 1)) q.load(stats + (e / 2 + 4) * 16, odd == 0);
        }
        if (cut) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if (e < from || e >= to) s[e] = 0;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) h[e] = pack_half2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]), T);
        tmem_st16(mine, h);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(bars + 8 * S::kP);
#pragma unroll
        for (int e = 0; e < 4; ++e) l[e].load(stats + S::kStatBytes + e * 16, odd == 0);
        ok = __all_sync(0xffffffffu, mbar_wait(bars + 8 * S::kR, i & 1, gave_up));
        if (!ok) break;
        tc_fence_after();
        uint32_t d[32];
        tmem_ld32(mine + kTmemR, d);
        tmem_ld32_wait(d);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            Stats4& q = l[e / 2 & 3];
            uint64_t x = add2(pair(__uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1])), q.v[e & 1]);
            if (e < 8 && (e & 1)) q.load(stats + S::kStatBytes + (e / 2 + 4) * 16, odd == 0);
            if constexpr (T == GS_F16) x = mul2(x, by_ds);
            const float2 f = unpair(mul2(x, pair(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]))));
            d[2 * e] = __float_as_uint(f.x), d[2 * e + 1] = __float_as_uint(f.y);
        }
        if (cut) {   // 0 times whatever the hidden rows give
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if (e < from || e >= to) d[e] = 0;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) h[e] = pack_half2(__uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1]), T);
        tmem_st16(mine + kTmemR, h);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) {
            mbar_arrive(bars + 8 * S::kDs);
            mbar_arrive(bars + 8 * (S::kStatEmpty + rs.s));
        }
    }
    // the first eight warps write dV, the others dK, half of the columns each
    const int half = quarter >> 1;
    if (w.n > 0 && ok) ok = __all_sync(0xffffffffu, mbar_wait(bars + 8 * (S::kDone + half), 0, gave_up));
    if (!ok) return;
    tc_fence_after();
    const bool live = key < w.seq.lk;
    const int64_t row = w.seq.k0 + key;
    const float by = half == 0 ? kDown<T> : p.scale * power2(-exponent);
    uint16_t* to = half == 0 ? p.dv + row * p.dv_row + w.head * p.dv_head : p.dk + row * p.dk_row + w.head * p.dk_head;
#pragma unroll 1
    for (int c = (quarter & 1) * (DP / 2); c < (quarter & 1) * (DP / 2) + DP / 2; c += 32) {
        float f[32];
        uint32_t v[32];
        if (w.n > 0) {
            tmem_ld32(tmem + kTmemDv + half * DP + c, v);
            tmem_ld32_wait(v);
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) f[e] = w.n > 0 ? __uint_as_float(v[e]) * by : 0.0f;
        if (p.parts > 1) {
            float* part = p.part + ((((int64_t)(blockIdx.x % p.parts) * p.seqs.k_rows + row) * p.kv_heads + w.head) * 2 + half) * DP + c;
            if (live)
#pragma unroll
                for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4*>(part + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
        } else if (live && c < p.dim) store_row32<T>(to, c, p.dim, half == 0 ? p.dv_vec : p.dk_vec, f);
    }
    tc_fence_before();
}

template <int T, int DP>
__global__ void __launch_bounds__(kKeyThreads, 1) keys_kernel(const __grid_constant__ Params p)
{
    using S = KeyShape<DP>;
    extern __shared__ __align__(1024) char smem_raw[];
    const uint32_t smem = smem_addr(smem_raw);
    if (smem & 1023u) {   // every thread sees the same address; there is no padding to move within
        g_attention_bwd_wait_expired = 1;
        return;
    }
    const uint32_t bars = smem + S::kAtBars;
    char* tail = smem_raw + S::kAtBars + ((S::kBars * 8 + 15) & ~15);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail);
    volatile int* gave_up = reinterpret_cast<volatile int*>(tail + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kBars; ++i)
            mbar_init(bars + 8 * i, i == S::kP || i == S::kDs || (i >= S::kStatEmpty && i < S::kS)                ? kKeyWarps
                                    : (i >= S::kQEmpty && i < S::kOFull) || (i >= S::kOEmpty && i < S::kStatFull) ? 2
                                                                                                                  : 1);
        *gave_up = 0;
        mbar_init_fence();
    }
    wait_for_predecessor_alone();
    if (p.zero) {
        fill_rows(p.fill_dk, p.seqs.k_starts, p.seqs.count, p.seqs.k_rows);
        fill_rows(p.fill_dv, p.seqs.k_starts, p.seqs.count, p.seqs.k_rows);
    }
    KeyWork w;
    if (!find_keys(p, blockIdx.x / p.parts, w)) return;   // the same for every warp
    if (p.parts > 1) {
        take_part(p, blockIdx.x % p.parts, w);
        if (w.n == 0) return;   // the join knows
    }
    if (warp == kKeyWarps) tmem_alloc<false>(smem_addr(tmem_slot), kTmemCols);
    const int packed = p.tokens * p.group;
    if (packed < kRows && w.n > 0)   // rows that no copy writes
        for (int t = warp; t < S::kStagesQ + S::kStagesO; t += kKeyThreads / 32) zero_rows<S::kChunks>(smem + S::kAtQ + t * S::kTile, packed, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    let_successor_start();
    if (warp < kKeyWarps) {
        many_registers<104>();
        const int exponent = T == GS_F16 && w.n > 0 ? ds_exponent<T>(p.dim, most_do(p, w.seq, w.head), most_v(p, w.seq, w.head)) : 0;
        key_terms<T, DP>(p, w, warp >> 2, threadIdx.x & 127, smem, bars, tmem + ((uint32_t)((warp & 3) * 32) << 16), exponent, gave_up);
    } else {
        few_registers();
        if (warp == kKeyWarps) {
            if (w.n > 0) {
                if (elect_one()) load_queries<DP>(p, w, smem, bars, gave_up);
                __syncwarp();
                clear_queries<DP>(p, w, smem, bars, lane, gave_up);
            }
        } else if (warp < kKeyWarps + 3 && elect_one()) {
            const int second = warp - kKeyWarps - 1;
            if (w.n > 0) issue_keys<DP>(p, w, second, smem, bars, tmem, gave_up);
            mma_commit<false>(bars + 8 * (S::kDone + second));   // the block does not leave before its products are done
            if (!mbar_wait_alone(bars + 8 * (S::kDone + second), 0)) *gave_up = 1;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0 && *gave_up) atomicExch(&g_attention_bwd_wait_expired, 1);
    if (warp == kKeyWarps) {
        tc_fence_after();
        tmem_free<false>(tmem, kTmemCols);
    }
}

// The parts' sums of a tile of keys, added in order.  A thread 32 columns of a row.
template <int T, int DP>
__global__ void __launch_bounds__(256) keys_join_kernel(const __grid_constant__ Params p)
{
    wait_for_predecessor();
    KeyWork w;
    if (!find_keys(p, blockIdx.x, w)) return;
    const int parts = w.each ? (w.n + w.each - 1) / w.each : 0;
    int rows = w.seq.lk - w.key0;
    rows = rows < kRows ? rows : kRows;
    constexpr int kSteps = 2 * DP / 32;   // of a row: dv, then dk
    for (int i = threadIdx.x; i < rows * kSteps; i += 256) {
        const int64_t row = w.seq.k0 + w.key0 + i / kSteps;
        const int half = i % kSteps / (kSteps / 2), c = i % (kSteps / 2) * 32;
        const float* from = p.part + ((row * p.kv_heads + w.head) * 2 + half) * DP + c;
        float f[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) f[e] = 0.0f;
        for (int k = 0; k < parts; ++k, from += p.seqs.k_rows * p.kv_heads * 2 * DP)
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                const float4 v = *reinterpret_cast<const float4*>(from + e);
                f[e] += v.x, f[e + 1] += v.y, f[e + 2] += v.z, f[e + 3] += v.w;
            }
        uint16_t* to = half == 0 ? p.dv + row * p.dv_row + w.head * p.dv_head : p.dk + row * p.dk_row + w.head * p.dk_head;
        if (c < p.dim) store_row32<T>(to, c, p.dim, half == 0 ? p.dv_vec : p.dk_vec, f);
    }
}

// ------------------------------------------------------------------ dq
// A CTA one or two tiles of packed query rows; two take turns as in the forward.  TMEM lanes
// are query rows: S = Q K^T; P in registers; R = dO V^T in S's place; dS in 16 bits in
// its place; dQ += dS K.  Values are done with early, keys late: rings of their own.
template <int DP, int TILES>
struct QueryShape {
    static constexpr int kChunks = DP / 64;
    static constexpr uint32_t kTile = kChunks * kBox;
    static constexpr int kStagesK = DP == 128 ? 2 : 3, kStagesV = DP == 128 ? 1 : 2;
    static constexpr int kTermWarps = 4 * TILES, kThreads = (kTermWarps + 4) * 32;
    static constexpr uint32_t kTmemCols = 256 * TILES, kTmemDq = 128 * TILES;
    static constexpr uint32_t kAtK = 2 * TILES * kTile, kAtV = kAtK + kStagesK * kTile, kAtBars = kAtV + kStagesV * kTile;
    static constexpr int kQFull = 0, kKFull = 2, kKEmpty = kKFull + kStagesK, kVFull = kKEmpty + kStagesK, kVEmpty = kVFull + kStagesV,
                         kS = kVEmpty + kStagesV, kP = kS + 2, kR = kP + 2, kDs = kR + 2, kClear = kDs + 2, kDone = kClear + 1,
                         kBars = kDone + 2;
    static constexpr int kSmem = kAtBars + ((kBars * 8 + 15) & ~15) + 16;
    static_assert(kSmem <= 232448, "shared memory of an SM");
};

struct QueryWork {
    Sequence seq;
    uint32_t head;
    int t0, n[2];
};
template <int TILES>
__device__ __forceinline__ bool find_queries(const Params& p, QueryWork& w)
{
    uint32_t unit, units;
    w.head = blockIdx.x % p.kv_heads;
    const int tokens = p.tokens * TILES;
    if (!find_unit<false>(p.seqs, blockIdx.x / p.kv_heads, tokens, w.seq, unit, units)) return false;
    if (p.causal) unit = units - 1 - unit;   // the longest first
    w.t0 = (int)unit * tokens;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = w.t0 + i * p.tokens;
        int last = t + p.tokens - 1;
        last = last < w.seq.lq ? last : w.seq.lq - 1;
        w.n[i] = i < TILES && t < w.seq.lq ? (keys_seen(w.seq, last, p.causal) + kRows - 1) / kRows : 0;
    }
    return true;
}

template <int DP, int TILES>
__device__ __forceinline__ void load_keys(const Params& p, const QueryWork& w, int n, uint32_t smem, uint32_t bars, volatile int* gave_up)
{
    using S = QueryShape<DP, TILES>;
    const uint32_t bytes = (uint32_t)(S::kChunks * p.tokens * p.group) * 128;
#pragma unroll
    for (int i = 0; i < TILES; ++i)
        if (w.n[i] > 0) {
            const int row = w.seq.q0 + w.t0 + i * p.tokens, head = w.head * p.group;
            mbar_expect(bars + 8 * (S::kQFull + i), 2 * bytes);
            load_tile<S::kChunks>(smem + 2 * i * S::kTile, &p.q, head, row, bars + 8 * (S::kQFull + i));
            load_tile<S::kChunks>(smem + (2 * i + 1) * S::kTile, &p.d_o, head, row, bars + 8 * (S::kQFull + i));
        }
    Ring<S::kStagesK> rk;
    Ring<S::kStagesV> rv;
    uint32_t nk = 0, nv = 0;
    int row = w.seq.k0;
    for (int j = 0; j < n; ++j, row += kRows) {
        if (!mbar_wait(bars + 8 * (S::kKEmpty + rk.s), rk.parity ^ 1, gave_up)) break;
        mbar_expect(bars + 8 * (S::kKFull + rk.s), S::kTile);
        load_tile<S::kChunks>(smem + S::kAtK + rk.s * S::kTile, &p.k, w.head, row, bars + 8 * (S::kKFull + rk.s));
        rk.next(), ++nk;
        if (!mbar_wait(bars + 8 * (S::kVEmpty + rv.s), rv.parity ^ 1, gave_up)) break;
        mbar_expect(bars + 8 * (S::kVFull + rv.s), S::kTile);
        load_tile<S::kChunks>(smem + S::kAtV + rv.s * S::kTile, &p.v, w.head, row, bars + 8 * (S::kVFull + rv.s));
        rv.next(), ++nv;
    }
    // the block does not leave before its copies have landed
    bool landed = true;
#pragma unroll
    for (int i = 0; i < TILES; ++i) landed = landed && (w.n[i] == 0 || mbar_wait_alone(bars + 8 * (S::kQFull + i), 0));
    last_copies<S::kStagesK>(nk, [&](uint32_t s, uint32_t parity) { landed = landed && mbar_wait_alone(bars + 8 * (S::kKFull + s), parity); });
    last_copies<S::kStagesV>(nv, [&](uint32_t s, uint32_t parity) { landed = landed && mbar_wait_alone(bars + 8 * (S::kVFull + s), parity); });
}

// Keys behind the sequence are contracted over in dQ: zero, by the loading warp, once all
// copies are under way.
template <int DP, int TILES>
__device__ __forceinline__ void clear_keys(const QueryWork& w, int n, uint32_t smem, uint32_t bars, int lane, volatile int* gave_up)
{
    using S = QueryShape<DP, TILES>;
    const int live = w.seq.lk - (n - 1) * kRows;
    if (live >= kRows || *gave_up) return;
    const uint32_t copy = n - 1, s = copy % S::kStagesK;
    if (!__all_sync(0xffffffffu, mbar_wait(bars + 8 * (S::kKFull + s), copy / S::kStagesK & 1, gave_up))) return;
    zero_rows<S::kChunks>(smem + S::kAtK + s * S::kTile, live, lane);
    if (lane == 0) mbar_arrive(bars + 8 * S::kClear);
}

// A lane issues the products of tile i: R(j) once P(j) is in registers, dQ(j) once dS(j) is
// written and, right behind it, S(j + 1) in dS's place.
template <int DP, int TILES>
__device__ __forceinline__ void issue_queries(const Params& p, const QueryWork& w, int i, int n, uint32_t smem, uint32_t bars, uint32_t tmem,
                                              volatile int* gave_up)
{
    using S = QueryShape<DP, TILES>;
    const int mine = i ? w.n[1] : w.n[0];
    const uint32_t steps = (uint32_t)(p.dim + 15) / 16, here = tmem + i * 128;
    const bool ragged = w.seq.lk < n * kRows;
    const auto rows_product = [&](uint32_t at_a, uint32_t at_b) {
        const uint32_t a = desc_lo(at_a, true), b = desc_lo(at_b, true);
#pragma unroll
        for (uint32_t s = 0; s < DP / 16; ++s) {
            const uint32_t at = (s >> 2) * (kBox >> 4) + (s & 3) * k_step(true);
            if (s < steps) mma<false, false>(here, a + at, kDescHi, b + at, kDescHi, p.idesc_s, s > 0);
        }
    };
    const auto keys_landed = [&](const Ring<S::kStagesK>& r) { return mbar_wait(bars + 8 * (S::kKFull + r.s), r.parity, gave_up); };
    const auto values_landed = [&](const Ring<S::kStagesV>& r) { return mbar_wait(bars + 8 * (S::kVFull + r.s), r.parity, gave_up); };
    // the rows are cleared behind the last copies, which wait for products before these
    const auto cleared = [&](int j) { return !ragged || j + 1 < n || mbar_wait(bars + 8 * S::kClear, 0, gave_up); };
    Ring<S::kStagesK> rk;
    Ring<S::kStagesV> rv;
    const auto scores = [&](int j) {
        if (!cleared(j)) return false;
        rows_product(smem + 2 * i * S::kTile, smem + S::kAtK + rk.s * S::kTile);
        mma_commit<false>(bars + 8 * (S::kS + i));
        return true;
    };
    if (mine > 0 && (!mbar_wait(bars + 8 * (S::kQFull + i), 0, gave_up) || !keys_landed(rk) || !scores(0))) return;
    for (int j = 0; j < mine; ++j) {
        if (!values_landed(rv) || !mbar_wait(bars + 8 * (S::kP + i), j & 1, gave_up)) return;
        tc_fence_after();
        rows_product(smem + (2 * i + 1) * S::kTile, smem + S::kAtV + rv.s * S::kTile);
        mma_commit<false>(bars + 8 * (S::kR + i));
        mma_commit<false>(bars + 8 * (S::kVEmpty + rv.s));
        rv.next();
        const uint32_t keys = rk.s;
        rk.next();
        const bool more = j + 1 < mine;
        if (more && !keys_landed(rk)) return;
        if (!mbar_wait(bars + 8 * (S::kDs + i), j & 1, gave_up)) return;
        tc_fence_after();
        const uint32_t b = desc_rows(smem + S::kAtK + keys * S::kTile);
#pragma unroll
        for (int s = 0; s < kRows / 16; ++s)
            mma_tmem(tmem + S::kTmemDq + i * DP, here + s * 8, b + s * k_step(false), kDescHi, p.idesc_d, j > 0 || s > 0);
        if (more && !scores(j + 1)) return;
        mma_commit<false>(bars + 8 * (S::kKEmpty + keys));
    }
    // copies that only the other tile reads: both lanes free a stage
    for (int j = mine; j < n; ++j, rk.next(), rv.next()) {
        if (!keys_landed(rk)) return;
        mbar_arrive(bars + 8 * (S::kKEmpty + rk.s));
        if (!values_landed(rv)) return;
        mbar_arrive(bars + 8 * (S::kVEmpty + rv.s));
    }
}

// A row a thread: i the tile, r the row.
template <int T, int DP, int TILES>
__device__ __forceinline__ void query_terms(const Params& p, const QueryWork& w, int i, int r, uint32_t bars, uint32_t tmem, volatile int* gave_up)
{
    using S = QueryShape<DP, TILES>;
    const int n = i ? w.n[1] : w.n[0], t0 = w.t0 + i * p.tokens;
    const int token = t0 + r / p.group;
    const bool live = r < p.tokens * p.group && token < w.seq.lq;
    const int64_t row = w.seq.q0 + token;
    const float* st = p.stats + w.head * p.stat_pitch + row * p.group + r % p.group;
    const uint64_t less = both(live ? st[0] - kUp<T> : -INFINITY), minus = both(live ? st[p.stat_plane] : 0.0f);   // p is no factor here
    const int seen = live ? keys_seen(w.seq, token, p.causal) : 0;
    const int all = keys_seen(w.seq, t0, p.causal);
    const int exponent = T == GS_F16 && live && n > 0 ? ds_exponent<T>(p.dim, st[2 * p.stat_plane], most_v(p, w.seq, w.head)) : 0;
    const uint64_t by_ds = both(power2(exponent)), scale2 = both(p.scale2);
    const uint32_t here = tmem + i * 128;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
        ok = __all_sync(0xffffffffu, mbar_wait(bars + 8 * (S::kS + i), j & 1, gave_up));
        if (!ok) break;
        tc_fence_after();
        uint32_t s[128];
#pragma unroll
        for (int c = 0; c < 128; c += 32) tmem_ld32(here + c, s + c);
#pragma unroll
        for (int c = 0; c < 128; c += 32) tmem_ld32_wait(s + c);
        tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(bars + 8 * (S::kP + i));   // read: R takes its place
#pragma unroll
        for (int c = 0; c < 128; c += 2) {
            const float2 x = unpair(fma2(pair(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), scale2, less));
            s[c] = __float_as_uint(exp2_fast(x.x)), s[c + 1] = __float_as_uint(exp2_fast(x.y));
        }
        const int left = seen - j * kRows;
        const bool cut = (j + 1) * kRows > all;
        ok = __all_sync(0xffffffffu, mbar_wait(bars + 8 * (S::kR + i), j & 1, gave_up));
        if (!ok) break;
        tc_fence_after();
        uint32_t d[2][32];
        tmem_ld32(here, d[0]);
        tmem_ld32_wait(d[0]);
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
            uint32_t(&v)[32] = d[c / 32 & 1];
            if (c < 96) tmem_ld32(here + c + 32, d[c / 32 + 1 & 1]);   // on its way during this part
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
                uint64_t x = add2(pair(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), minus);
                if constexpr (T == GS_F16) x = mul2(x, by_ds);
                const float2 f = unpair(mul2(x, pair(__uint_as_float(s[c + e]), __uint_as_float(s[c + e + 1]))));
                v[e] = __float_as_uint(f.x), v[e + 1] = __float_as_uint(f.y);
            }
            if (cut) {   // 0 whatever the hidden keys give
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (c + e >= left) v[e] = 0;
            }
            uint32_t h[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) h[e] = pack_half2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]), T);
            if (c < 96) tmem_ld32_wait(d[c / 32 + 1 & 1]);
            tmem_st16(here + c / 2, h);   // behind what has been read
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(bars + 8 * (S::kDs + i));
    }
    if (n > 0 && ok) ok = __all_sync(0xffffffffu, mbar_wait(bars + 8 * (S::kDone + i), 0, gave_up));
    if (!ok) return;
    tc_fence_after();
    const float by = p.scale * power2(-exponent);
    uint16_t* to = p.dq + row * p.dq_row + ((int)w.head * p.group + r % p.group) * p.dq_head;
#pragma unroll 1
    for (int c = 0; c < DP; c += 32) {
        float f[32];
        uint32_t v[32];
        if (n > 0) {
            tmem_ld32(tmem + S::kTmemDq + i * DP + c, v);
            tmem_ld32_wait(v);
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) f[e] = n > 0 ? __uint_as_float(v[e]) * by : 0.0f;
        if (live && c < p.dim) store_row32<T>(to, c, p.dim, p.dq_vec, f);
    }
    tc_fence_before();
}

// ------------------------------------------------------------------ delta
// The queries' blocks once more: S and R in places of their own, read as they come, the
// rows' sums of p r in registers.  Nothing waits for a term, so that the products run ahead.
template <int DP, int TILES>
__device__ __forceinline__ void issue_delta(const Params& p, const QueryWork& w, int i, int n, uint32_t smem, uint32_t bars, uint32_t tmem,
                                            volatile int* gave_up)
{
    using S = QueryShape<DP, TILES>;
    const int mine = i ? w.n[1] : w.n[0];
    const uint32_t steps = (uint32_t)(p.dim + 15) / 16;
    const auto rows_product = [&](uint32_t d, uint32_t at_a, uint32_t at_b) {
        const uint32_t a = desc_lo(at_a, true), b = desc_lo(at_b, true);
#pragma unroll
        for (uint32_t s = 0; s < DP / 16; ++s) {
            const uint32_t at = (s >> 2) * (kBox >> 4) + (s & 3) * k_step(true);
            if (s < steps) mma<false, false>(d, a + at, kDescHi, b + at, kDescHi, p.idesc_s, s > 0);
        }
    };
    Ring<S::kStagesK> rk;
    Ring<S::kStagesV> rv;
    if (mine > 0 && !mbar_wait(bars + 8 * (S::kQFull + i), 0, gave_up)) return;
    for (int j = 0; j < n; ++j, rk.next(), rv.next()) {
        if (!mbar_wait(bars + 8 * (S::kKFull + rk.s), rk.parity, gave_up)) return;
        if (j < mine) {
            if (j > 0 && !mbar_wait(bars + 8 * (S::kP + i), (j - 1) & 1, gave_up)) return;   // S has been read
            tc_fence_after();
            rows_product(tmem + i * 128, smem + 2 * i * S::kTile, smem + S::kAtK + rk.s * S::kTile);
            mma_commit<false>(bars + 8 * (S::kS + i));
            mma_commit<false>(bars + 8 * (S::kKEmpty + rk.s));
        } else mbar_arrive(bars + 8 * (S::kKEmpty + rk.s));
        if (!mbar_wait(bars + 8 * (S::kVFull + rv.s), rv.parity, gave_up)) return;
        if (j < mine) {
            if (j > 0 && !mbar_wait(bars + 8 * (S::kDs + i), (j - 1) & 1, gave_up)) return;   // R has been read
            tc_fence_after();
            rows_product(tmem + (TILES + i) * 128, smem + (2 * i + 1) * S::kTile, smem + S::kAtV + rv.s * S::kTile);
            mma_commit<false>(bars + 8 * (S::kR + i));
            mma_commit<false>(bars + 8 * (S::kVEmpty + rv.s));
        } else mbar_arrive(bars + 8 * (S::kVEmpty + rv.s));
    }
}

// A row a thread: i the tile, r the row.
template <int T, int DP, int TILES>
__device__ __forceinline__ void delta_terms(const Params& p, const QueryWork& w, int i, int r, uint32_t bars, uint32_t tmem, volatile int* gave_up)
{
    using S = QueryShape<DP, TILES>;
    const int n = i ? w.n[1] : w.n[0], t0 = w.t0 + i * p.tokens;
    const int token = t0 + r / p.group;
    const bool live = r < p.tokens * p.group && token < w.seq.lq;
    const int64_t row = w.seq.q0 + token;
    const float lse = live ? p.lse[row * (p.group * p.kv_heads) + (int)w.head * p.group + r % p.group] : -INFINITY;
    const uint64_t less = both(lse == -INFINITY ? -INFINITY : lse * -kLog2e), scale2 = both(p.scale2);
    const int seen = live ? keys_seen(w.seq, token, p.causal) : 0;
    const int all = keys_seen(w.seq, t0, p.causal);
    uint64_t sum[2] = {both(0.0f), both(0.0f)};
    for (int j = 0; j < n; ++j) {
        if (!__all_sync(0xffffffffu, mbar_wait(bars + 8 * (S::kS + i), j & 1, gave_up))) return;
        tc_fence_after();
        uint32_t s[128];
#pragma unroll
        for (int c = 0; c < 128; c += 32) tmem_ld32(tmem + i * 128 + c, s + c);
#pragma unroll
        for (int c = 0; c < 128; c += 32) tmem_ld32_wait(s + c);
        tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(bars + 8 * (S::kP + i));
#pragma unroll
        for (int c = 0; c < 128; c += 2) {
            const float2 x = unpair(fma2(pair(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), scale2, less));
            s[c] = __float_as_uint(exp2_fast(x.x)), s[c + 1] = __float_as_uint(exp2_fast(x.y));
        }
        const int left = seen - j * kRows;
        const bool cut = (j + 1) * kRows > all;
        if (!__all_sync(0xffffffffu, mbar_wait(bars + 8 * (S::kR + i), j & 1, gave_up))) return;
        tc_fence_after();
        uint32_t d[2][32];
        tmem_ld32(tmem + (TILES + i) * 128, d[0]);
        tmem_ld32_wait(d[0]);
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
            uint32_t(&v)[32] = d[c / 32 & 1];
            if (c < 96) tmem_ld32(tmem + (TILES + i) * 128 + c + 32, d[c / 32 + 1 & 1]);   // on its way during this part
            if (cut) {   // 0 times whatever the hidden keys give
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (c + e >= left) s[c + e] = v[e] = 0;
            }
#pragma unroll
            for (int e = 0; e < 32; e += 2)
                sum[e / 2 & 1] = fma2(pair(__uint_as_float(s[c + e]), __uint_as_float(s[c + e + 1])),
                                      pair(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), sum[e / 2 & 1]);
            if (c < 96) tmem_ld32_wait(d[c / 32 + 1 & 1]);
        }
        tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(bars + 8 * (S::kDs + i));
    }
    if (!live) return;
    const float2 a = unpair(sum[0]), b = unpair(sum[1]);
    float* to = p.stats + w.head * p.stat_pitch + row * p.group + r % p.group;
    // a row that sees no key: every p is 2^-infinity
    to[0] = lse == -INFINITY ? -INFINITY : __fmaf_rn(lse, -kLog2e, kUp<T>);
    to[p.stat_plane] = lse == -INFINITY ? 0.0f : -((a.x + a.y) + (b.x + b.y));
}

template <int T, int DP, int TILES, bool DELTA>
__global__ void __launch_bounds__(QueryShape<DP, TILES>::kThreads, 3 - TILES) queries_kernel(const __grid_constant__ Params p)
{
    using S = QueryShape<DP, TILES>;
    extern __shared__ __align__(1024) char smem_raw[];
    const uint32_t smem = smem_addr(smem_raw);
    if (smem & 1023u) {
        g_attention_bwd_wait_expired = 1;
        return;
    }
    const uint32_t bars = smem + S::kAtBars;
    char* tail = smem_raw + S::kAtBars + ((S::kBars * 8 + 15) & ~15);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail);
    volatile int* gave_up = reinterpret_cast<volatile int*>(tail + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kBars; ++i) {
            const bool warps = (i >= S::kP && i < S::kR) || (i >= S::kDs && i < S::kClear);
            const bool lanes = (i >= S::kKEmpty && i < S::kVFull) || (i >= S::kVEmpty && i < S::kS);
            mbar_init(bars + 8 * i, warps ? 4 : (lanes ? TILES : 1));
        }
        *gave_up = 0;
        mbar_init_fence();
    }
    wait_for_predecessor_alone();
    if (DELTA && T == GS_F16)
        for (int64_t i = (int64_t)blockIdx.x * S::kThreads + threadIdx.x; i < 2 * (int64_t)p.seqs.count * p.kv_heads; i += (int64_t)gridDim.x * S::kThreads)
            p.most[i] = 0.0f;
    if (!DELTA && p.zero) fill_rows(p.fill_dq, p.seqs.q_starts, p.seqs.count, p.seqs.q_rows);
    QueryWork w;
    if (!find_queries<TILES>(p, w)) return;   // the same for every warp
    if (warp == S::kTermWarps) tmem_alloc<false>(smem_addr(tmem_slot), S::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    let_successor_start();
    const int n = w.n[0] > w.n[1] ? w.n[0] : w.n[1];
    if (warp >= S::kTermWarps) {
        few_registers();
        const int i = warp - S::kTermWarps - 1;
        if (i < 0) {
            if (n > 0) {
                if (elect_one()) load_keys<DP, TILES>(p, w, n, smem, bars, gave_up);
                __syncwarp();
                if constexpr (!DELTA) clear_keys<DP, TILES>(w, n, smem, bars, lane, gave_up);
            }
        } else if (i < TILES && elect_one()) {
            if constexpr (DELTA) issue_delta<DP, TILES>(p, w, i, n, smem, bars, tmem, gave_up);
            else issue_queries<DP, TILES>(p, w, i, n, smem, bars, tmem, gave_up);
            mma_commit<false>(bars + 8 * (S::kDone + i));   // the block does not leave before its products are done
            if (!mbar_wait_alone(bars + 8 * (S::kDone + i), 0)) *gave_up = 1;
        }
    } else {
        many_registers<TILES == 2 ? 224 : 200>();
        const int i = warp >> 2;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        if (w.t0 + i * p.tokens < w.seq.lq) {
            if constexpr (DELTA) delta_terms<T, DP, TILES>(p, w, i, threadIdx.x & 127, bars, lanes, gave_up);
            else query_terms<T, DP, TILES>(p, w, i, threadIdx.x & 127, bars, lanes, gave_up);
        }
    }
    __syncthreads();
    if (threadIdx.x == 0 && *gave_up) atomicExch(&g_attention_bwd_wait_expired, 1);
    if (warp == S::kTermWarps) {
        tc_fence_after();
        tmem_free<false>(tmem, S::kTmemCols);
    }
}

struct Plan {
    int group, tokens, tiles, dp;
    uint32_t parts;
    int64_t query_items, key_items, stat_pitch, stat_plane;
    size_t stats, most, part, packs, bytes;
};
Plan plan_for(const gs_attention_bwd_args& a)
{
    Plan r = {};
    r.group = a.heads / a.kv_heads;
    r.tokens = kRows / r.group;
    r.dp = a.dim <= 64 ? 64 : 128;
    const int known = device_sms();
    const int64_t sms = known > 0 ? known : 152;
    const bool starts = a.q_starts != nullptr;
    const int64_t two = units_at_most(a.q_rows, a.sequences, starts, 2 * (int64_t)r.tokens);
    // as in the forward: two CTAs an SM of 64 columns and fewer, whose shared memory allows it; of
    // more, two tiles a CTA where there are CTAs enough all the same, and tokens for both
    r.tiles = r.dp == 128 && two * a.kv_heads >= sms && a.q_rows > a.sequences * r.tokens ? 2 : 1;
    r.query_items = (r.tiles == 2 ? two : units_at_most(a.q_rows, a.sequences, starts, r.tokens)) * a.kv_heads;
    r.key_items = units_at_most(a.k_rows, a.sequences, starts, kRows) * a.kv_heads;
    // Parts of a tile of keys' queries: what the longest takes (1.6 us a tile of queries) or the
    // SMs' share of all, against the blocks' starts and the parts' sums.  us by parts, all
    // gradients: 2048 tokens, 1 key head of 64 236 (1), 126 (3), 97 (8), 104 (16); 16384, 1 of
    // 128 1248 (1), 911 (3), 991 (6); 4096, 4 of 64 297 (1), 228 (2), 239 (3); 4096, 16 of 128
    // without a mask 465 (1), 555 (2).
    r.parts = 1;
    const int64_t sequences = a.sequences > 0 ? a.sequences : 1, query_tiles = (a.q_rows / sequences + r.tokens - 1) / r.tokens;
    double best = 0;
    for (int64_t n = 1; n <= 32 && (n == 1 || 2 * n <= query_tiles); ++n) {
        const double longest = std::ceil((double)query_tiles / (double)n) * 1.6;
        const double work = (double)(r.key_items * query_tiles) * (a.causal ? 0.8 : 1.6) / (double)sms;
        const double us = (work > longest ? work : longest) + 0.15 * longest + 4.0 * (double)(r.key_items * n) / (double)sms +
                          (n > 1 ? 6 + 0.4 * (double)n + (double)(n * a.k_rows * a.kv_heads) * r.dp * 16 / 2e6 : 0.0);
        if (n == 1 || us < best) best = us, r.parts = (uint32_t)n;
    }
    if (r.parts > 1) r.part = (size_t)round_up(r.parts * a.k_rows * a.kv_heads * r.dp * 8, 256);
    r.stat_pitch = round_up(a.q_rows * r.group, 4);
    // the last copy of a plane's statistics reads up to a tile past the last row
    r.stat_plane = round_up(a.kv_heads * r.stat_pitch + kStatRows, 64);
    const bool f16 = a.type == GS_F16;
    r.stats = (size_t)r.stat_plane * (f16 ? 12 : 8);
    r.most = f16 ? (size_t)round_up(a.sequences * a.kv_heads * 8, 256) : 0;
    if (!tensor_tma(a.q, a.q_row, a.q_head, a.q_rows, a.heads)) r.packs += packed_bytes(a.q_rows, a.heads, a.dim);
    if (!tensor_tma(a.d_o, a.do_row, a.do_head, a.q_rows, a.heads)) r.packs += packed_bytes(a.q_rows, a.heads, a.dim);
    if (!tensor_tma(a.k, a.k_row, a.k_head, a.k_rows, a.kv_heads)) r.packs += packed_bytes(a.k_rows, a.kv_heads, a.dim);
    if (!tensor_tma(a.v, a.v_row, a.v_head, a.k_rows, a.kv_heads)) r.packs += packed_bytes(a.k_rows, a.kv_heads, a.dim);
    r.bytes = r.part + r.stats + r.most + r.packs;
    return r;
}

template <class K>
gs_status launch_one(K* kernel, int smem, int threads, std::atomic<uint64_t>& done, int64_t items, const Params& p, cudaStream_t st)
{
    const gs_status s = allow_smem(kernel, smem, done);
    return s != GS_OK ? s : launch_after(kernel, dim3((unsigned)items), (unsigned)threads, (size_t)smem, 1, st, p);
}
template <int T, int DP, bool DELTA>
gs_status launch_queries(const Params& p, const Plan& plan, cudaStream_t st)
{
    static std::atomic<uint64_t> one_done{0}, two_done{0};
    if constexpr (DP == 128)
        if (plan.tiles == 2)
            return launch_one(queries_kernel<T, DP, 2, DELTA>, QueryShape<DP, 2>::kSmem, QueryShape<DP, 2>::kThreads, two_done, plan.query_items, p, st);
    return launch_one(queries_kernel<T, DP, 1, DELTA>, QueryShape<DP, 1>::kSmem, QueryShape<DP, 1>::kThreads, one_done, plan.query_items, p, st);
}
// F16's largest magnitudes, after delta's launch.
gs_status largest_values(const gs_attention_bwd_args& a, const Params& p, cudaStream_t st)
{
    const int known = device_sms();
    const int64_t sms = known > 0 ? known : 152;
    MostParams t = {};
    t.d_o = (const uint16_t*)a.d_o, t.do_row = a.do_row, t.do_head = a.do_head;
    t.v = (const uint16_t*)a.v, t.v_row = a.v_row, t.v_head = a.v_head;
    t.seqs = p.seqs, t.lse = p.lse, t.row_most = p.stats + 2 * p.stat_plane, t.most = (uint32_t*)p.most, t.stat_pitch = p.stat_pitch;
    t.kv_heads = p.kv_heads, t.group = p.group, t.dim = p.dim;
    t.do_vec = a.dim % 8 == 0 && tensor_tma(a.d_o, a.do_row, a.do_head, a.q_rows, a.heads);
    t.v_vec = a.dim % 8 == 0 && tensor_tma(a.v, a.v_row, a.v_head, a.k_rows, a.kv_heads);
    // some four blocks an SM for either
    t.q_each = round_up((a.q_rows * a.kv_heads + 4 * sms - 1) / (4 * sms), kMostRows);
    t.k_each = round_up((a.k_rows * a.kv_heads + 4 * sms - 1) / (4 * sms), kMostRows);
    t.q_chunks = (uint32_t)((a.q_rows + t.q_each - 1) / t.q_each), t.k_chunks = (uint32_t)((a.k_rows + t.k_each - 1) / t.k_each);
    t.q_blocks = t.q_chunks * t.kv_heads;
    return launch_after(most_kernel, dim3(t.q_blocks + t.k_chunks * t.kv_heads), 256, 0, 1, st, t);
}

template <int T, int DP>
gs_status launch(const gs_attention_bwd_args& a, const Params& p, const Plan& plan, bool pairs, cudaStream_t st)
{
    static std::atomic<uint64_t> done{0};
    gs_status s = pairs ? launch_queries<T, DP, true>(p, plan, st) : GS_OK;
    if (T == GS_F16 && s == GS_OK && pairs) s = largest_values(a, p, st);
    if (s == GS_OK && p.dk) s = launch_one(keys_kernel<T, DP>, KeyShape<DP>::kSmem, kKeyThreads, done, plan.key_items * plan.parts, p, st);
    if (s == GS_OK && p.dk && plan.parts > 1) s = launch_after(keys_join_kernel<T, DP>, dim3((unsigned)plan.key_items), 256, 0, 1, st, p);
    return s == GS_OK && p.dq ? launch_queries<T, DP, false>(p, plan, st) : s;
}

}  // namespace

gs_status backward_wait_report(int* expired)
{
    const int zero = 0;
    GS_CUDA_TRY(cudaMemcpyFromSymbol(expired, g_attention_bwd_wait_expired, sizeof *expired));
    if (*expired) GS_CUDA_TRY(cudaMemcpyToSymbol(g_attention_bwd_wait_expired, &zero, sizeof zero));
    return GS_OK;
}

}  // namespace attn
}  // namespace gs

using namespace gs;
using namespace gs::attn;

extern "C" gs_status gs_attention_bwd(const gs_attention_bwd_args* args, void* ws, size_t* ws_bytes, void* stream)
{
    GS_NVTX_RANGE("gs_attention_bwd");
    if (!args) return GS_ERR_INVALID_ARG;
    const gs_attention_bwd_args& a = *args;
    if (!sizes_ok(a.q_rows, a.k_rows, a.sequences, a.heads, a.kv_heads, a.dim, a.type, a.scale, a.q_starts, a.k_starts))
        return GS_ERR_INVALID_ARG;
    if (!a.dk != !a.dv && a.k_rows > 0) return GS_ERR_INVALID_ARG;
    if (a.q_rows > 0) {
        if (!tensor_ok(a.q, a.q_row, a.q_head, a.q_rows, a.heads, a.dim, false) ||
            !tensor_ok(a.d_o, a.do_row, a.do_head, a.q_rows, a.heads, a.dim, false) || !a.lse || ((uintptr_t)a.lse & 3u))
            return GS_ERR_INVALID_ARG;
        if (a.dq && !tensor_ok(a.dq, a.dq_row, a.dq_head, a.q_rows, a.heads, a.dim, true)) return GS_ERR_INVALID_ARG;
    }
    if (a.k_rows > 0) {
        if (!tensor_ok(a.k, a.k_row, a.k_head, a.k_rows, a.kv_heads, a.dim, false) ||
            !tensor_ok(a.v, a.v_row, a.v_head, a.k_rows, a.kv_heads, a.dim, false))
            return GS_ERR_INVALID_ARG;
        if (a.dk && (!tensor_ok(a.dk, a.dk_row, a.dk_head, a.k_rows, a.kv_heads, a.dim, true) ||
                     !tensor_ok(a.dv, a.dv_row, a.dv_head, a.k_rows, a.kv_heads, a.dim, true)))
            return GS_ERR_INVALID_ARG;
    }
    const Plan plan = plan_for(a);
    if (plan.query_items > 0x7fffffffll || plan.key_items * plan.parts > 0x7fffffffll) return GS_ERR_INVALID_ARG;
    const WsCheck wc = ws_check(ws, ws_bytes, plan.bytes);
    if (wc == WsCheck::kBad) return GS_ERR_INVALID_ARG;
    if (wc == WsCheck::kQuery) return GS_OK;
    cudaStream_t st = (cudaStream_t)stream;
    const bool dq = a.dq && a.q_rows > 0, dk = a.dk && a.k_rows > 0;
    if (!dq && !dk) return GS_OK;
    float* stats = (float*)((char*)ws + plan.part);
    float* most = plan.most ? (float*)((char*)ws + plan.part + plan.stats) : nullptr;
    char* to = (char*)ws + plan.part + plan.stats + plan.most;
    PackList packs;
    Params p = {};
    gs_status s = GS_OK;
    if (a.q_rows > 0 && a.k_rows > 0) {   // without a pair of query and key the kernels read nothing and write zeros
        const Tensor3 q = packs.add({a.q, a.q_row, a.q_head}, a.q_rows, a.heads, a.dim, to);
        const Tensor3 d = packs.add({a.d_o, a.do_row, a.do_head}, a.q_rows, a.heads, a.dim, to);
        const Tensor3 k = packs.add({a.k, a.k_row, a.k_head}, a.k_rows, a.kv_heads, a.dim, to);
        const Tensor3 v = packs.add({a.v, a.v_row, a.v_head}, a.k_rows, a.kv_heads, a.dim, to);
        s = tile_map(&p.q, q, a.type, a.q_rows, a.heads, a.dim, plan.group, plan.tokens);
        if (s == GS_OK) s = tile_map(&p.d_o, d, a.type, a.q_rows, a.heads, a.dim, plan.group, plan.tokens);
        if (s == GS_OK) s = tile_map(&p.k, k, a.type, a.k_rows, a.kv_heads, a.dim, 1, kRows);
        if (s == GS_OK) s = tile_map(&p.v, v, a.type, a.k_rows, a.kv_heads, a.dim, 1, kRows);
        if (s == GS_OK) s = packs.run(st);
        if (s != GS_OK) return s;
    }
    p.seqs = {a.q_starts, a.k_starts, nullptr, a.q_rows, a.k_rows, (uint32_t)a.sequences};
    p.zero = a.fill && a.q_starts;
    p.fill_dq = {(uint16_t*)a.dq, a.dq_row, a.dq_head, nullptr, a.heads, a.dim};
    p.fill_dk = {(uint16_t*)a.dk, a.dk_row, a.dk_head, nullptr, a.kv_heads, a.dim};
    p.fill_dv = {(uint16_t*)a.dv, a.dv_row, a.dv_head, nullptr, a.kv_heads, a.dim};
    p.stats = stats, p.lse = a.lse, p.most = most, p.stat_pitch = plan.stat_pitch, p.stat_plane = plan.stat_plane;
    p.dq = dq ? (uint16_t*)a.dq : nullptr, p.dq_row = a.dq_row, p.dq_head = a.dq_head;
    p.dk = dk ? (uint16_t*)a.dk : nullptr, p.dk_row = a.dk_row, p.dk_head = a.dk_head;
    p.dv = (uint16_t*)a.dv, p.dv_row = a.dv_row, p.dv_head = a.dv_head;
    p.scale = a.scale, p.scale2 = a.scale * kLog2e;
    p.part = (float*)ws, p.parts = plan.parts;
    p.kv_heads = (uint32_t)a.kv_heads, p.group = plan.group, p.tokens = plan.tokens, p.dim = a.dim;
    p.causal = a.causal != 0;
    p.dq_vec = tensor_vec(a.dq, a.dq_row, a.dq_head, a.q_rows, a.heads);
    p.dk_vec = tensor_vec(a.dk, a.dk_row, a.dk_head, a.k_rows, a.kv_heads);
    p.dv_vec = tensor_vec(a.dv, a.dv_row, a.dv_head, a.k_rows, a.kv_heads);
    p.idesc_s = instr_desc(a.type, true, true, kRows, kRows);
    p.idesc_d = instr_desc(a.type, true, false, (int)round_up(a.dim, 16), kRows);
    const bool pairs = a.q_rows > 0 && a.k_rows > 0;
    if (a.type == GS_BF16) return plan.dp == 64 ? launch<GS_BF16, 64>(a, p, plan, pairs, st) : launch<GS_BF16, 128>(a, p, plan, pairs, st);
    return plan.dp == 64 ? launch<GS_F16, 64>(a, p, plan, pairs, st) : launch<GS_F16, 128>(a, p, plan, pairs, st);
}
