// ssm_common.cuh -- device pieces shared by the selective scan's forward, step
// and backward: activations to float32 accuracy, channel pairs, thread layout.
#pragma once

#include "rdm_common.cuh"
#include "ssm_launch.h"

namespace rdm {
namespace ssm {

// Two float32 operations an instruction (sm_100's packed forms), each rounded as
// the single one.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(r)) : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t&>(r))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(r)) : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return r;
}
__device__ __forceinline__ float2 ex22(float2 x) { return make_float2(ex2_fast(x.x), ex2_fast(x.y)); }
__device__ __forceinline__ float2 two(float x) { return make_float2(x, x); }

// exp(delta A) as 2^(delta A log2 e).  ex2.approx comes out low by 2e-8 of its value
// on average where decays lie (measured on the card: 0.5 to 2.6e-8 for exponents
// from -0.001 to -1), which a long memory adds up token by token (dA of 2048 tokens
// 1.8e-6 off, against 1.0e-6 for float32 with a correctly rounded exponential); an
// exponent larger by as much costs nothing in the same multiply-add (0.8e-6).  It is
// the mean of exponents between -1 and 0; below -1 it is less than half a step of the
// exponent itself, and decays forget soon enough for neither to matter.  The folds
// over whole segments go without.  A step of zero still gives 1.
__device__ __forceinline__ float2 decay2(float2 delta, float2 A2) { return ex22(fma2(delta, A2, two(2.5e-8f))); }

// softplus(x) = max(x, 0) + log1p(e^-|x|).  The steps sit near 1e-3..1e-1, where
// the logarithm's argument is close to 1 and lg2.approx (absolute error 2^-22)
// would leave only 12 of their bits; so log1p(y) = 2 atanh(s), s = y / (2 + y),
// as 2 s P(s^2) with s^2 <= 1/9 (P fitted here, relative error 4e-9), which the
// float32 states and gradients need.
__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 rcp2(float2 x) { return make_float2(rcp_fast(x.x), rcp_fast(x.y)); }
__device__ __forceinline__ float max0(float x) {  // NaN stays NaN
    float y;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 softplus2(float2 x) {
    // e^-|x| = 2^t (1 + r ln 2), t the rounded product |x| log2 e and r what the
    // rounding left: near |x| = 7 that is 4e-7 of the result, and of a small step.
    // (|x| up to 200 only, where e^-|x| is 0 in any case and r stays finite.)
    const float2 a = make_float2(fmaxf(-fabsf(x.x), -200.0f), fmaxf(-fabsf(x.y), -200.0f));
    const float2 t = mul2(a, two(kLog2e));
    const float2 r = fma2(a, two(1.925963033500644e-08f), fma2(a, two(kLog2e), make_float2(-t.x, -t.y)));
    float2 y = ex22(t);
    y = fma2(y, mul2(r, two(kLn2)), y);
    const float2 s = mul2(y, rcp2(add2(y, two(2.0f))));
    const float2 q = mul2(s, s);
    float2 v = two(0.2817833423614502f);
    v = fma2(v, q, two(0.27960604429244995f));
    v = fma2(v, q, two(0.40024909377098083f));
    v = fma2(v, q, two(0.6666631698608398f));
    v = fma2(v, q, two(2.0f));
    return fma2(s, v, make_float2(max0(x.x), max0(x.y)));
}
__device__ __forceinline__ float2 sigmoid2(float2 x) { return rcp2(add2(ex22(mul2(x, two(-kLog2e))), two(1.0f))); }
__device__ __forceinline__ float2 silu2(float2 x) { return mul2(x, sigmoid2(x)); }
__device__ __forceinline__ float softplus(float x) { return softplus2(two(x)).x; }
__device__ __forceinline__ float silu(float x) { return x * rcp_fast(1.0f + ex2_fast(-x * kLog2e)); }
// d silu(x) / dx = s (1 + x (1 - s)), s = sigmoid(x)

__device__ __forceinline__ float2 dsilu2(float2 x, float2 s) {
    const float2 r = make_float2(1.0f - s.x, 1.0f - s.y);
    return mul2(s, fma2(x, r, two(1.0f)));
}

// 16 bytes from global into shared memory without passing registers; zeros where
// `there` is false.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(there ? 16 : 0)
                 : "memory");
}

// Two neighbouring channels of a row.
template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
    using Raw = uint32_t;
    static __device__ __forceinline__ Raw zero() { return 0u; }
    static __device__ __forceinline__ float2 f(Raw r) {
        return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
    }
    static __device__ __forceinline__ Raw r(float a, float b) {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<Raw*>(&h);
    }
};
template <>
struct Pair<float> {
    using Raw = float2;
    static __device__ __forceinline__ Raw zero() { return make_float2(0.0f, 0.0f); }
    static __device__ __forceinline__ float2 f(Raw r) { return r; }
    static __device__ __forceinline__ Raw r(float a, float b) { return make_float2(a, b); }
};
template <typename T>
__device__ __forceinline__ typename Pair<T>::Raw ldpair(const T* p) {
    return __ldg(reinterpret_cast<const typename Pair<T>::Raw*>(p));
}
template <typename T>
__device__ __forceinline__ void stpair(T* p, float a, float b) {
    *reinterpret_cast<typename Pair<T>::Raw*>(p) = Pair<T>::r(a, b);
}
// Four neighbouring values as loaded, and as float32.
template <typename T>
struct Four;
template <>
struct Four<float> {
    using Raw = float4;
    static __device__ __forceinline__ Raw zero() { return make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
    static __device__ __forceinline__ Raw ld(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
    static __device__ __forceinline__ float2 lo(Raw r) { return make_float2(r.x, r.y); }
    static __device__ __forceinline__ float2 hi(Raw r) { return make_float2(r.z, r.w); }
};
template <>
struct Four<__nv_bfloat16> {
    using Raw = uint2;
    static __device__ __forceinline__ Raw zero() { return make_uint2(0u, 0u); }
    static __device__ __forceinline__ Raw ld(const __nv_bfloat16* p) { return __ldg(reinterpret_cast<const uint2*>(p)); }
    static __device__ __forceinline__ float2 lo(Raw r) {
        return make_float2(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u));
    }
    static __device__ __forceinline__ float2 hi(Raw r) {
        return make_float2(__uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
    }
};
template <typename T>
__device__ __forceinline__ float4 ld4(const T* p) {
    const typename Four<T>::Raw r = Four<T>::ld(p);
    const float2 a = Four<T>::lo(r), b = Four<T>::hi(r);
    return make_float4(a.x, a.y, b.x, b.y);
}

// Sums of four values over the LPC lanes of a channel (LPC >= 4 neighbouring
// lanes): lane l ends with the sum of value l & 3.  Three shuffles for the first
// four lanes instead of the eight of four separate sums.
template <int LPC>
__device__ __forceinline__ float lane_sum4(float a0, float a1, float a2, float a3) {
    const int lane = threadIdx.x & 31;
    const bool hi = lane & 2, odd = lane & 1;
    const float s0 = hi ? a0 : a2, s1 = hi ? a1 : a3;
    float k0 = hi ? a2 : a0, k1 = hi ? a3 : a1;
    k0 += __shfl_xor_sync(0xffffffffu, s0, 2);
    k1 += __shfl_xor_sync(0xffffffffu, s1, 2);
    const float s = odd ? k0 : k1;
    float k = odd ? k1 : k0;
    k += __shfl_xor_sync(0xffffffffu, s, 1);
#pragma unroll
    for (int o = 4; o < LPC; o <<= 1) k += __shfl_xor_sync(0xffffffffu, k, o);
    return k;
}

// Tokens of sequence b, 0..T; out of range sets the status word and counts as
// the nearest end.
__device__ __forceinline__ int seq_len(const SsmParams& p, int b) {
    if (!p.lengths) return p.T;
    const int n = p.lengths[b];
    if (n < 0 || n > p.T) {
        if (threadIdx.x == 0) atomicOr(p.err, 2u);  // kErrBadValue
        return n < 0 ? 0 : p.T;
    }
    return n;
}

// Thread layout: each channel's N states lie on N/4 neighbouring lanes, four a
// lane; a block has CPB channels of one head.
template <int N, int CPB>
struct Lay {
    static constexpr int LPC = N / 4;
    static constexpr int THREADS = CPB * LPC;
    // Shared-memory place of channel c in the [token quad][place][4] arrays: even
    // and odd channels apart, so that the threads that write pairs of channels
    // and the lanes that read neighbouring ones both spread over the banks.
    static constexpr int ODD = CPB / 2 + 4;
    static constexpr int PLACES = CPB + 4;
    static __device__ __forceinline__ int place(int c) { return (c >> 1) + (c & 1) * ODD; }
};

}  // namespace ssm
}  // namespace rdm
