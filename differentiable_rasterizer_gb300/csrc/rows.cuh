// rows.cuh -- reductions over a row that a group of threads holds (norm.cu, block_norm.cu).
#pragma once

#include "layers_common.cuh"

namespace gs {
namespace rows {

constexpr float kE4m3Max = 448.0f;
constexpr float kTiny = 0x1p-100f;

__device__ __forceinline__ float max_nan(float a, float b)   // NaN if either is
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Rows that are read in pieces of eight columns from every eighth on, but for the last row's end:
// of 16-byte base and pitch.  A piece may end in the row's padding, and of fp32 rows whose pitch is
// not a multiple of eight in the next row's first four columns.  At a pitch of four a row of fewer
// columns has not so many: its pieces would reach behind the matrix.
__host__ __device__ __forceinline__ bool piece_rows(const void* p, int64_t ld, int type)
{
    return ((uintptr_t)p & 15u) == 0 && ld >= 8 && ld * type_bytes(type) % 16 == 0;
}

struct Sum {
    __device__ static float join(float a, float b) { return a + b; }
};
struct Max {
    __device__ static float join(float a, float b) { return max_nan(a, b); }
};

// Reduction over the `group` threads of a row: a warp's lanes by butterfly (all
// lanes get the same bits, the joins being commutative), then the group's warps
// through shared memory, in order.
template <class Op>
__device__ __forceinline__ float group_reduce(float v, int group, float* sm)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {   // unrolled: a step that the group has not leaves v as it is
        const float other = __shfl_xor_sync(0xffffffffu, v, o);
        v = o < group ? Op::join(v, other) : v;
    }
    if (group <= 32) return v;
    // the group's own barrier: other rows of the block go their way
    const int warp = threadIdx.x >> 5, first = threadIdx.x / group * (group >> 5), last = first + (group >> 5);
    const int barrier = 1 + threadIdx.x / group;   // at most 8 groups of 64 in a block
    asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(group) : "memory");   // the previous row's readers are done
    if ((threadIdx.x & 31) == 0) sm[warp] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(group) : "memory");
    float r = sm[first];
    for (int w = first + 1; w < last; ++w) r = Op::join(r, sm[w]);
    return r;
}

}  // namespace rows
}  // namespace gs
