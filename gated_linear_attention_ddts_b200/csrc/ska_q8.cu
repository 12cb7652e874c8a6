// ska_q8.cu -- sliding-window shared-key attention for single tokens (ska.cu)
// over a ring cache held in 8 bits, with a scale for each block of tokens and
// head:
//
//   k_u = k_scale[u / R] K8[u]    v_u = v_scale[u / R] V8[u]
//   s_u = scale q . k_u           o = sum_u softmax(s)_u v_u
//
// The tokens of the block being written stay in bf16 (the tail) until the block
// is full and are then rounded once, with the scale of the whole block; a token
// is never rounded twice, and a cache that a prompt filled equals one that was
// filled token by token.  Slots of that block that the tail does not reach yet
// still hold the round before, with the scale of then.
//
// Codes: e4m3 with the least power of two that keeps the block's largest
// magnitude within 448 (scaling is then exact and the only rounding is e4m3's
// own, 2^-4 of a value at most), or int8 with the largest magnitude over 127
// (2^-8 of the block's largest magnitude at most).  Values that are not finite
// do not count for the scale; e4m3 keeps NaN, infinities become the largest code.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "launch.h"
#include "rdm_common.cuh"
#include "ska_launch.h"
#include "ska_q8_launch.h"
#include "tc_common.cuh"

namespace rdm {
namespace {

using tc::unpack8;

// ------------------------------------------------------------------ rounding a block
__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a <= 3.4e38f ? a : 0.0f;  // neither infinite nor NaN (bf16 ends at 3.39e38)
}

// The scale of a block whose largest magnitude is `most`; 1 for a block of zeros.
template <bool I8>
__device__ __forceinline__ float block_scale(float most) {
    if (most == 0.0f) return 1.0f;
    if (I8) return __fdiv_rn(most, 127.0f);
    // most = m 2^e, 1 <= m < 2, and 448 = 1.75 2^8
    const unsigned bits = __float_as_uint(most);
    int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((unsigned)(max(e, -126) + 127) << 23);
}

template <bool I8>
__device__ __forceinline__ unsigned char encode(float x, float scale, float inv) {
    if (I8) return (unsigned char)(signed char)max(-127, min(127, __float2int_rn(__fdiv_rn(x, scale))));
    return __nv_cvt_float_to_fp8(x * inv, __NV_SATFINITE, __NV_E4M3);
}

template <bool I8>
__device__ __forceinline__ float decode8(unsigned char c) {
    if (I8) return (float)(signed char)c;
    __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
    return __half2float(__half(h));
}

constexpr int kThreads = 128;

// Rounds `rows` rows of D values (row r at src + r * D) into dst and *scale, by
// the whole CTA of kThreads.
template <bool I8, int D>
__device__ void round_block(const __nv_bfloat16* src, int rows, unsigned char* dst, float* scale) {
    __shared__ float red[kThreads / 32];
    const int n8 = rows * (D / 8);
    float most = 0.0f;
    for (int i = threadIdx.x; i < n8; i += blockDim.x) {
        float f[8];
        unpack8(reinterpret_cast<const uint4*>(src)[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) most = fmaxf(most, finite_abs(f[e]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = most;
    __syncthreads();
    most = red[0];
    for (int w = 1; w < (int)blockDim.x / 32; ++w) most = fmaxf(most, red[w]);
    const float s = block_scale<I8>(most), inv = I8 ? 0.0f : __fdiv_rn(1.0f, s);
    for (int i = threadIdx.x; i < n8; i += blockDim.x) {
        float f[8];
        unpack8(reinterpret_cast<const uint4*>(src)[i], f);
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e >> 2] |= (uint32_t)encode<I8>(f[e], s, inv) << (8 * (e & 3));
        reinterpret_cast<uint2*>(dst)[i] = make_uint2(w[0], w[1]);
    }
    if (threadIdx.x == 0) *scale = s;
    __syncthreads();
}

// ------------------------------------------------------------------ fill from a prompt
// One CTA per (block of slots, sequence, head; the shared key counts as a head).
template <bool I8, int D>
__device__ void fill_block(const SkaQ8FillParams& p, const __nv_bfloat16* src, int blk, int len, unsigned char* dst,
                           float* scale, __nv_bfloat16* tail) {
    const int w = p.c.window, R = p.c.block;
    const int at = blk * R, stop = min(at + R, w);
    const int last = len - 1, round = last / w, cur = last % w;
    int r = round;  // the last round in which the block became full
    if (cur < stop - 1) --r;
    if (at <= cur && cur < stop - 1) {  // the block being written
        const __nv_bfloat16* s = src + ((size_t)round * w + at) * D;
        for (int i = threadIdx.x; i < (cur - at + 1) * (D / 8); i += kThreads)
            reinterpret_cast<uint4*>(tail)[i] = reinterpret_cast<const uint4*>(s)[i];
    }
    if (r < 0) return;
    round_block<I8, D>(src + ((size_t)r * w + at) * D, stop - at, dst + (size_t)at * D, scale + blk);
}

template <bool I8>
__global__ void __launch_bounds__(kThreads) ska_q8_fill_kernel(const SkaQ8FillParams p) {
    const SkaQ8Cache& c = p.c;
    const int nb = (c.window + c.block - 1) / c.block;
    const int blk = blockIdx.x % nb, row = blockIdx.x / nb, b = row / (c.H + 1), h = row % (c.H + 1) - 1;
    int len = p.lengths ? p.lengths[b] : p.T;
    if (len < 0 || len > p.T) {
        if (threadIdx.x == 0) atomicOr(p.err, kErrBadValue);
        len = len < 0 ? 0 : p.T;
    }
    if (blk == 0 && h < 0 && threadIdx.x == 0) c.pos[b] = len;
    if (len == 0) return;
    if (h < 0) {
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.k) + (size_t)b * p.T * c.dk;
        unsigned char* dst = c.k + (size_t)b * c.window * c.dk;
        __nv_bfloat16* tail = static_cast<__nv_bfloat16*>(c.k_tail) + (size_t)b * c.block * c.dk;
        if (c.dk == 64) fill_block<I8, 64>(p, src, blk, len, dst, c.k_scale + (size_t)b * nb, tail);
        else fill_block<I8, 128>(p, src, blk, len, dst, c.k_scale + (size_t)b * nb, tail);
        return;
    }
    const size_t bh = (size_t)b * c.H + h;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.v) + bh * p.T * c.dv;
    unsigned char* dst = c.v + bh * c.window * c.dv;
    __nv_bfloat16* tail = static_cast<__nv_bfloat16*>(c.v_tail) + bh * c.block * c.dv;
    if (c.dv == 64) fill_block<I8, 64>(p, src, blk, len, dst, c.v_scale + bh * nb, tail);
    else fill_block<I8, 128>(p, src, blk, len, dst, c.v_scale + bh * nb, tail);
}

// ------------------------------------------------------------------ one token
// One CTA per (b, h).  First version: scores of all slots in shared memory.
template <bool I8, int DK, int DV>
__global__ void __launch_bounds__(kThreads) ska_q8_decode_kernel(const SkaQ8DecodeParams p) {
    extern __shared__ float sc[];  // [window]
    __shared__ float qs[DK];
    __shared__ float red[kThreads / 32];
    __shared__ float part[kThreads / (DV / 8)][DV];
    const SkaQ8Cache& c = p.c;
    const int b = blockIdx.x / c.H, h = blockIdx.x % c.H, tid = threadIdx.x;
    const int pos = c.pos[b];
    if (pos < 0) {
        if (tid == 0) atomicOr(p.err, kErrBadValue);
        return;
    }
    const int w = c.window, R = c.block, nb = (w + R - 1) / R;
    const int n = pos < w ? pos + 1 : w, cur = pos % w, at = cur / R * R, fill = cur - at;
    const size_t bh = (size_t)b * c.H + h;
    const __nv_bfloat16* kin = static_cast<const __nv_bfloat16*>(p.k) + (size_t)b * DK;
    const __nv_bfloat16* vin = static_cast<const __nv_bfloat16*>(p.v) + bh * DV;
    __nv_bfloat16* kt = static_cast<__nv_bfloat16*>(c.k_tail) + (size_t)b * R * DK;
    __nv_bfloat16* vt = static_cast<__nv_bfloat16*>(c.v_tail) + bh * R * DV;
    if (h == 0 && tid < DK) kt[(size_t)fill * DK + tid] = kin[tid];
    if (tid < DV) vt[(size_t)fill * DV + tid] = vin[tid];
    if (tid < DK) qs[tid] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[bh * DK + tid]) * p.scale * kLog2e;
    __syncthreads();
    float mx = -INFINITY;
    for (int u = tid; u < n; u += kThreads) {
        float a = 0.0f;
        if (u >= at && u <= cur) {  // from the tail; the new key from the inputs
            const __nv_bfloat16* r = u == cur ? kin : kt + (size_t)(u - at) * DK;
            for (int i = 0; i < DK; ++i) a = fmaf(qs[i], __bfloat162float(r[i]), a);
        } else {
            const unsigned char* r = c.k + ((size_t)b * w + u) * DK;
            for (int i = 0; i < DK; ++i) a = fmaf(qs[i], decode8<I8>(r[i]), a);
            a *= c.k_scale[(size_t)b * nb + u / R];
        }
        sc[u] = a;
        mx = fmaxf(mx, a);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    __syncthreads();
    float sum = 0.0f;
    for (int u = tid; u < n; u += kThreads) {
        const float e = ex2_fast(sc[u] - mx);
        sc[u] = e;
        sum += e;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((tid & 31) == 0) red[tid >> 5] = sum;
    __syncthreads();
    sum = red[0] + red[1] + red[2] + red[3];
    constexpr int XP = DV / 8, LG = kThreads / XP;
    const int x = tid % XP, lg = tid / XP;
    float acc[8] = {};
    for (int u = lg; u < n; u += LG) {
        const float pu = sc[u];
        if (u >= at && u <= cur) {
            const __nv_bfloat16* r = vt + (size_t)(u - at) * DV + 8 * x;
            for (int e = 0; e < 8; ++e) acc[e] = fmaf(pu, __bfloat162float(r[e]), acc[e]);
        } else {
            const unsigned char* r = c.v + (bh * w + u) * DV + 8 * x;
            const float ps = pu * c.v_scale[bh * nb + u / R];
            for (int e = 0; e < 8; ++e) acc[e] = fmaf(ps, decode8<I8>(r[e]), acc[e]);
        }
    }
    for (int e = 0; e < 8; ++e) part[lg][8 * x + e] = acc[e];
    __syncthreads();
    if (tid < DV) {
        float a = 0.0f;
        for (int l = 0; l < LG; ++l) a += part[l][tid];
        static_cast<__nv_bfloat16*>(p.o)[bh * DV + tid] = __float2bfloat16_rn(a / sum);
    }
    if (cur == w - 1 || fill == R - 1) {  // the block is full (its slots are read from the tail in this step)
        if (h == 0) {
            __syncthreads();
            round_block<I8, DK>(kt, fill + 1, c.k + ((size_t)b * w + at) * DK, c.k_scale + (size_t)b * nb + at / R);
        }
        round_block<I8, DV>(vt, fill + 1, c.v + (bh * w + at) * DV, c.v_scale + bh * nb + at / R);
    }
}

__global__ void ska_q8_advance_kernel(int* pos, int B) {
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b < B && pos[b] >= 0) pos[b] += 1;
}

template <bool I8, int DK, int DV>
cudaError_t launch_decode_cfg(const SkaQ8DecodeParams& p, cudaStream_t s) {
    auto kern = ska_q8_decode_kernel<I8, DK, DV>;
    const size_t smem = (size_t)p.c.window * 4;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)(p.c.B * p.c.H), kThreads, smem, s>>>(p);
    return cudaGetLastError();
}

template <bool I8>
cudaError_t launch_decode_t(const SkaQ8DecodeParams& p, cudaStream_t s) {
    if (p.c.dk == 64)
        return p.c.dv == 64 ? launch_decode_cfg<I8, 64, 64>(p, s) : launch_decode_cfg<I8, 64, 128>(p, s);
    return p.c.dv == 64 ? launch_decode_cfg<I8, 128, 64>(p, s) : launch_decode_cfg<I8, 128, 128>(p, s);
}

}  // namespace

cudaError_t launch_ska_q8_fill(const SkaQ8FillParams& p, cudaStream_t s) {
    const int nb = (p.c.window + p.c.block - 1) / p.c.block;
    const unsigned grid = (unsigned)((long long)nb * p.c.B * (p.c.H + 1));
    if (p.c.int8) ska_q8_fill_kernel<true><<<grid, kThreads, 0, s>>>(p);
    else ska_q8_fill_kernel<false><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

size_t ska_q8_decode_workspace(const SkaQ8DecodeParams&) { return 0; }

cudaError_t launch_ska_q8_decode(const SkaQ8DecodeParams& p, cudaStream_t s) {
    const cudaError_t e = p.c.int8 ? launch_decode_t<true>(p, s) : launch_decode_t<false>(p, s);
    if (e != cudaSuccess || !p.advance) return e;
    ska_q8_advance_kernel<<<(p.c.B + 255) / 256, 256, 0, s>>>(p.c.pos, p.c.B);
    return cudaGetLastError();
}

}  // namespace rdm
