// layers_common.cuh -- element types, conversions and activations shared by the
// decoder layers (norm.cu, linear.cu, gemm.cu, glu_narrow.cu).
#pragma once

#include <atomic>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "gs_common.cuh"

namespace gs {

__host__ __device__ constexpr int type_bytes(int t) { return t == GS_F32 ? 4 : (t == GS_E4M3 ? 1 : 2); }

inline bool type_float(int t) { return t == GS_F32 || t == GS_BF16 || t == GS_F16; }
inline bool type_half(int t) { return t == GS_BF16 || t == GS_F16; }
inline bool act_ok(int a) { return a >= GS_ACT_NONE && a <= GS_ACT_GELU; }

// A matrix of the given columns and leading dimension: present, wide enough and
// aligned to its elements.
inline bool mat_ok(const void* p, int64_t ld, int64_t cols, int type)
{
    return p && ld >= cols && ld <= 0x7fffffffll && ((uintptr_t)p % (uintptr_t)type_bytes(type)) == 0;
}
inline bool vec_ok(const void* p, int type) { return ((uintptr_t)p % (uintptr_t)type_bytes(type)) == 0; }
inline bool size_ok(int64_t v, int64_t lo) { return v >= lo && v <= 0x7fffffffll; }

// Rows that 16-byte accesses and tensor copies can take as they lie.
inline bool rows16(const void* p, int64_t ld, int type)
{
    return aligned16(p) && (ld * type_bytes(type)) % 16 == 0;
}

inline int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// The host-side workspace convention: ws == NULL with ws_bytes reports the size;
// ws_bytes == NULL runs a call that needs none; otherwise the size must suffice.
enum class WsCheck { kRun, kQuery, kBad };
inline WsCheck ws_check(void* ws, size_t* ws_bytes, size_t need)
{
    if (!ws_bytes) return need == 0 ? WsCheck::kRun : WsCheck::kBad;
    if (!ws) {
        *ws_bytes = need;
        return WsCheck::kQuery;
    }
    return *ws_bytes < need || ((uintptr_t)ws & 255u) ? WsCheck::kBad : WsCheck::kRun;
}

// ------------------------------------------------------------------ launches
// The layers' kernels follow one another closely (a training step of a layer is four to
// eight), so each is launched as a dependent of the one before: its blocks may be set up
// while that one still runs, and wait for its end, with all its writes visible, in
// wait_for_predecessor, which every thread calls before it touches memory.
__device__ __forceinline__ void wait_for_predecessor()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
}

template <class... P, class... A>
gs_status launch_after(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, unsigned cluster, cudaStream_t st,
                       const A&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    GS_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, args...));
    return GS_OK;
}

// Sets a kernel's shared memory once on each device.
template <class K>
inline gs_status allow_smem(K* kernel, int bytes, std::atomic<uint64_t>& done)
{
    int dev = 0;
    GS_CUDA_TRY(cudaGetDevice(&dev));
    const uint64_t bit = 1ull << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return GS_OK;
    GS_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    if (dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
    return GS_OK;
}

// Calls f with the 16-bit type and the activation as constants.
template <class F>
gs_status for_type_act(int type, int act, F f)
{
    const auto with_type = [&](auto t) -> gs_status {
        if (act == GS_ACT_SILU) return f(t, std::integral_constant<int, GS_ACT_SILU>());
        if (act == GS_ACT_GELU) return f(t, std::integral_constant<int, GS_ACT_GELU>());
        if (act == GS_ACT_RELU) return f(t, std::integral_constant<int, GS_ACT_RELU>());
        return f(t, std::integral_constant<int, GS_ACT_NONE>());
    };
    return type == GS_BF16 ? with_type(std::integral_constant<int, GS_BF16>())
                           : with_type(std::integral_constant<int, GS_F16>());
}

// ------------------------------------------------------------------ elements
__device__ __forceinline__ float load_elem(const void* p, int64_t i, int type)
{
    if (type == GS_F32) return ((const float*)p)[i];
    if (type == GS_BF16) return __bfloat162float(((const __nv_bfloat16*)p)[i]);
    if (type == GS_F16) return __half2float(((const __half*)p)[i]);
    __nv_fp8_e4m3 q;
    q.__x = ((const __nv_fp8_storage_t*)p)[i];
    return (float)q;
}

// fp32 -> e4m3: nearest even, saturating at 448, NaN kept.
__device__ __forceinline__ uint8_t e4m3_bits(float v)
{
    return (uint8_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ void store_elem(void* p, int64_t i, int type, float v)
{
    if (type == GS_F32) ((float*)p)[i] = v;
    else if (type == GS_BF16) ((__nv_bfloat16*)p)[i] = __float2bfloat16_rn(v);
    else if (type == GS_F16) ((__half*)p)[i] = __float2half_rn(v);
    else ((uint8_t*)p)[i] = e4m3_bits(v);
}

// Two values in 16 bits each, the first in the low half.
__device__ __forceinline__ uint32_t pack_half2(float a, float b, int type)
{
    if (type == GS_BF16) {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&h);
    }
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ float2 unpack_half2(uint32_t v, int type)
{
    if (type == GS_BF16)   // a bfloat16 is the upper half of the float of the same value
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    return __half22float2(*reinterpret_cast<__half2*>(&v));
}

// Eight consecutive elements, 16-byte aligned (f32: two accesses).
__device__ __forceinline__ void load8(const void* p, int64_t i, int type, float v[8])
{
    if (type == GS_F32) {
        const float4 a = *reinterpret_cast<const float4*>((const float*)p + i);
        const float4 b = *reinterpret_cast<const float4*>((const float*)p + i + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        return;
    }
    const uint4 a = *reinterpret_cast<const uint4*>((const uint16_t*)p + i);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = unpack_half2(w[j], type);
        v[2 * j] = f.x, v[2 * j + 1] = f.y;
    }
}

__device__ __forceinline__ void store8(void* p, int64_t i, int type, const float v[8])
{
    if (type == GS_F32) {
        *reinterpret_cast<float4*>((float*)p + i) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>((float*)p + i + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else if (type == GS_E4M3) {
        uint32_t w[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * j], v[4 * j + 1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * j + 2], v[4 * j + 3]), __NV_SATFINITE,
                                                         __NV_E4M3);
            w[j] = lo | (hi << 16);
        }
        *reinterpret_cast<uint2*>((uint8_t*)p + i) = make_uint2(w[0], w[1]);
    } else {
        *reinterpret_cast<uint4*>((uint16_t*)p + i) =
            make_uint4(pack_half2(v[0], v[1], type), pack_half2(v[2], v[3], type), pack_half2(v[4], v[5], type),
                       pack_half2(v[6], v[7], type));
    }
}

// Elements as they lie in memory, and their values.  The type is a template argument
// (GS_F32, GS_BF16, GS_F16, or kAnyType with the type at run time): a branch on the
// type between a load and its conversion makes every load wait for the one before
// (the norm's forward over 1,000,000 x 256 took 479 us with such branches).
constexpr int kAnyType = -1;

template <int T, int VEC>
struct Raw {
    uint4 q[T == GS_F32 || T == kAnyType ? 2 : 1];
};
template <>
struct Raw<GS_F32, 1> {
    float f;
};
template <>
struct Raw<GS_BF16, 1> {
    uint16_t h;
};
template <>
struct Raw<GS_F16, 1> {
    uint16_t h;
};
template <>
struct Raw<kAnyType, 1> {
    float f;
};

template <int T, int VEC>
__device__ __forceinline__ void raw_load(Raw<T, VEC>& r, const void* p, int64_t i, int type)
{
    if constexpr (VEC == 8) {
        if (T == GS_F32 || (T == kAnyType && type == GS_F32)) {
            r.q[0] = *reinterpret_cast<const uint4*>((const float*)p + i);
            if constexpr (T == GS_F32 || T == kAnyType) r.q[1] = *reinterpret_cast<const uint4*>((const float*)p + i + 4);
        } else r.q[0] = *reinterpret_cast<const uint4*>((const uint16_t*)p + i);
    } else if constexpr (T == GS_F32) r.f = ((const float*)p)[i];
    else if constexpr (T == kAnyType) r.f = load_elem(p, i, type);
    else r.h = ((const uint16_t*)p)[i];
}

template <int T, int VEC>
__device__ __forceinline__ void raw_zero(Raw<T, VEC>& r)
{
    if constexpr (VEC == 8) {
        r.q[0] = make_uint4(0, 0, 0, 0);
        if constexpr (T == GS_F32 || T == kAnyType) r.q[1] = make_uint4(0, 0, 0, 0);
    } else if constexpr (T == GS_F32 || T == kAnyType) r.f = 0.0f;
    else r.h = 0;
}

template <int T, int VEC>
__device__ __forceinline__ void raw_values(const Raw<T, VEC>& r, int type, float (&v)[VEC])
{
    if constexpr (VEC == 8) {
        if (T == GS_F32 || (T == kAnyType && type == GS_F32)) {
            constexpr int hi = T == GS_F32 || T == kAnyType ? 1 : 0;
            const uint32_t w[8] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w, r.q[hi].x, r.q[hi].y, r.q[hi].z, r.q[hi].w};
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
        } else {
            const uint32_t w[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = unpack_half2(w[j], T == kAnyType ? type : T);
                v[2 * j] = f.x, v[2 * j + 1] = f.y;
            }
        }
    } else if constexpr (T == GS_F32 || T == kAnyType) v[0] = r.f;
    else v[0] = unpack_half2(r.h, T).x;
}

template <int VEC>
__device__ __forceinline__ void load_vec(const void* p, int64_t i, int type, float (&v)[VEC])
{
    if constexpr (VEC == 8) load8(p, i, type, v);
    else v[0] = load_elem(p, i, type);
}
template <int VEC>
__device__ __forceinline__ void store_vec(void* p, int64_t i, int type, const float (&v)[VEC])
{
    if constexpr (VEC == 8) store8(p, i, type, v);
    else store_elem(p, i, type, v[0]);
}

// ------------------------------------------------------------------ activations
// The hardware's exponential and reciprocal, subnormals to zero (their callers' sums
// with 1 hide them; without .ftz each costs four instructions more).
__device__ __forceinline__ float exp2_fast(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp_fast(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// sigma(v): relative error below 2^-21 + |v| 2^-23 (the instructions' 2 and 1 ulp; two
// roundings of |v| log2 e, which the exponential multiplies by |v|).  For v below about
// -88 the exponential is infinite and the reciprocal 0, as it should be.
__device__ __forceinline__ float sigmoid_fast(float v) { return rcp_fast(1.0f + exp2_fast(-1.4426950408889634f * v)); }

// Phi(v), the normal distribution function, and e = exp(-v^2 / 2), which its slope
// shares:  Phi(-|v|) = (c1 t + ... + cN t^N) e,  t = 1 / (1 + p |v|).
// The form is that of Abramowitz & Stegun, Handbook of Mathematical Functions, 7.1.26;
// the coefficients are minimax fits of the relative error over 0 <= |v| <= 13.4 (beyond, e
// is below fp32's normal range): eight terms 1.3e-7, for what stays in fp32; six 4.7e-6,
// for what is rounded to 16 bits, where that is a 50th of f16's half unit (1,000,000 x 64
// -> 128: six 107 us, eight 117 in one coding; the epilogue is bound by issue slots).
// Taken on the negative side and chosen by the sign, so that the tail keeps its digits: with
// the instructions' errors Phi is within 2^-20 (2^-17 of six terms) + v^2 2^-23 of itself,
// the latter from rounding v^2.  1/2 + sign(v) (1/2 - Phi(-|v|)) would lose the tail in the
// subtraction, GELU below -5 with it.
// An erff and a second exponential cost three times as many instructions, which
// is what bounded the elementwise gradients and the epilogues.
template <bool FINE>
struct Phi {
    static constexpr int kTerms = FINE ? 8 : 6;
    static constexpr float kP = FINE ? 0.3f : 0.31f;
    __host__ __device__ static constexpr float c(int i)   // of t^(i + 1)
    {
        constexpr float fine[8] = {0.119625784f,   0.120807543f, 0.0995807424f, 0.129654914f,
                                   -0.0557424501f, 0.208583161f, -0.158493474f, 0.0359837115f};
        constexpr float coarse[6] = {0.123860702f, 0.12044128f, 0.133429766f, 0.0157447252f, 0.180450335f, -0.0739291385f};
        return FINE ? fine[i] : coarse[i];
    }
};
template <bool FINE>
__device__ __forceinline__ float normal_cdf(float v, float& e)
{
    using F = Phi<FINE>;
    const float t = rcp_fast(__fmaf_rn(fabsf(v), F::kP, 1.0f));
    e = exp2_fast(v * v * (-0.5f * 1.4426950408889634f));
    float q = F::c(F::kTerms - 1);
#pragma unroll
    for (int i = F::kTerms - 2; i >= 0; --i) q = __fmaf_rn(t, q, F::c(i));
    q = q * t * e;
    return __float_as_int(v) < 0 ? q : 1.0f - q;
}

// fine: the value is not rounded to 16 bits.
__device__ __forceinline__ float act_value(float v, int act, bool fine)
{
    if (act == GS_ACT_RELU) return v < 0.0f ? 0.0f : v;   // NaN stays NaN
    if (act == GS_ACT_SILU) return v * sigmoid_fast(v);
    if (act == GS_ACT_GELU) {
        float e;
        return v * (fine ? normal_cdf<true>(v, e) : normal_cdf<false>(v, e));
    }
    return v;
}

// Two floats in one 64-bit register: sm_103a adds, multiplies and fuses them in one
// instruction, rounding each as the single one does.
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Phi of two values, to the bit as normal_cdf computes it, in codings that the callers'
// registers suit best (all measured, the others being spilled or issued worse): CHOICE, the
// last step as a choice by sign, or (1 or 0) minus the tail with its sign set, without
// predicates; FOLD, t's divisor one value at a time, which takes |v| along.
//   gated layer's value          choice           1,000,000 x 64 -> 128 111 us, signed 118
//   product's value              signed, folded   100,000 x 256 -> 256 56 us, choice 60
//   gated layer's gradients      signed           1,000,000 x 64 x 128 149 us, choice 162
//   elementwise gradient         choice           100,000 x 256 37.5 us, signed 39.5
template <bool FINE, bool CHOICE, bool FOLD>
__device__ __forceinline__ uint64_t normal_cdf2(uint64_t v, uint64_t& e)
{
    using F = Phi<FINE>;
    const auto both = [](float c) { return pair(c, c); };
    const float2 f = unpair(v);
    const float2 d = FOLD ? make_float2(__fmaf_rn(fabsf(f.x), F::kP, 1.0f), __fmaf_rn(fabsf(f.y), F::kP, 1.0f))
                          : unpair(fma2(pair(fabsf(f.x), fabsf(f.y)), both(F::kP), both(1.0f)));
    const uint64_t t = pair(rcp_fast(d.x), rcp_fast(d.y));
    const float2 x = unpair(mul2(mul2(v, v), both(-0.5f * 1.4426950408889634f)));
    e = pair(exp2_fast(x.x), exp2_fast(x.y));
    uint64_t q = both(F::c(F::kTerms - 1));
#pragma unroll
    for (int i = F::kTerms - 2; i >= 0; --i) q = fma2(t, q, both(F::c(i)));
    q = mul2(mul2(q, t), e);
    const float2 p = unpair(q);
    if constexpr (!CHOICE) {
        float hx, hy;   // 0 below zero (-0 too), else 1
        asm("set.ge.f32.s32 %0, %1, 0;" : "=f"(hx) : "r"(__float_as_int(f.x)));
        asm("set.ge.f32.s32 %0, %1, 0;" : "=f"(hy) : "r"(__float_as_int(f.y)));
        return add2(pair(hx, hy), pair(copysignf(p.x, -f.x), copysignf(p.y, -f.y)));
    } else
        return pair(__float_as_int(f.x) < 0 ? p.x : 1.0f - p.x, __float_as_int(f.y) < 0 ? p.y : 1.0f - p.y);
}

template <int ACT, bool FINE, bool GLU>
__device__ __forceinline__ uint64_t act_value2(uint64_t v)
{
    if constexpr (ACT == GS_ACT_SILU) {
        const float2 x = unpair(mul2(v, pair(-1.4426950408889634f, -1.4426950408889634f)));
        const float2 d = unpair(add2(pair(exp2_fast(x.x), exp2_fast(x.y)), pair(1.0f, 1.0f)));
        return mul2(v, pair(rcp_fast(d.x), rcp_fast(d.y)));
    } else if constexpr (ACT == GS_ACT_GELU) {
        uint64_t e;
        return mul2(v, normal_cdf2<FINE, GLU, !GLU>(v, e));
    } else {
        const float2 f = unpair(v);
        return pair(act_value(f.x, ACT, FINE), act_value(f.y, ACT, FINE));
    }
}

// act(v) and act'(v), from one sigma or one Phi.
template <bool FINE>
__device__ __forceinline__ void act_both(float v, int act, float& value, float& slope)
{
    if (act == GS_ACT_SILU) {
        const float p = sigmoid_fast(v);
        value = v * p;
        slope = p * __fmaf_rn(v, 1.0f - p, 1.0f);
    } else if (act == GS_ACT_GELU) {
        float e;
        const float c = normal_cdf<FINE>(v, e);
        value = v * c;
        slope = __fmaf_rn(v * 0.39894228040143268f, e, c);
    } else if (act == GS_ACT_RELU) {
        value = v < 0.0f ? 0.0f : v;
        slope = v > 0.0f ? 1.0f : (v != v ? v : 0.0f);
    } else {
        value = v;
        slope = 1.0f;
    }
}

template <int ACT, bool FINE, bool CHOICE>
__device__ __forceinline__ void act_both2(uint64_t v, uint64_t& value, uint64_t& slope)
{
    const auto both = [](float c) { return pair(c, c); };
    if constexpr (ACT == GS_ACT_SILU) {
        const float2 x = unpair(mul2(v, both(-1.4426950408889634f)));
        const float2 d = unpair(add2(pair(exp2_fast(x.x), exp2_fast(x.y)), both(1.0f)));
        const uint64_t p = pair(rcp_fast(d.x), rcp_fast(d.y));
        value = mul2(v, p);
        slope = mul2(p, fma2(v, fma2(p, both(-1.0f), both(1.0f)), both(1.0f)));
    } else if constexpr (ACT == GS_ACT_GELU) {
        uint64_t e;
        const uint64_t c = normal_cdf2<FINE, CHOICE, false>(v, e);
        value = mul2(v, c);
        slope = fma2(mul2(v, both(0.39894228040143268f)), e, c);
    } else {
        const float2 f = unpair(v);
        float2 a, b;
        act_both<FINE>(f.x, ACT, a.x, b.x);
        act_both<FINE>(f.y, ACT, a.y, b.y);
        value = pair(a.x, a.y);
        slope = pair(b.x, b.y);
    }
}

__device__ __forceinline__ float act_slope(float v, int act)
{
    float value, slope;
    act_both<true>(v, act, value, slope);
    return slope;
}

// 16 columns of the gated layer's gradient: dg = dh u act'(g), du = dh act(g).
template <int ACT>
__device__ __forceinline__ void glu_gradient(float (&g)[16], float (&u)[16], const float (&dh)[16])
{
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
        uint64_t value, slope;
        act_both2<ACT, false, false>(pair(g[j], g[j + 1]), value, slope);
        const uint64_t d = pair(dh[j], dh[j + 1]);
        const float2 a = unpair(mul2(mul2(d, pair(u[j], u[j + 1])), slope)), b = unpair(mul2(d, value));
        g[j] = a.x, g[j + 1] = a.y;
        u[j] = b.x, u[j + 1] = b.y;
    }
}

}  // namespace gs
