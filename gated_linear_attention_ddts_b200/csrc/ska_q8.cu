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

// Four values as codes.  int8 rounds x / scale; x times the rounded reciprocal is
// within 3 2^-24 of that quotient (relative), 3e-5 at most below 128, so only next
// to a border between two codes does the division itself have to decide (`exact`:
// for all, where values or the reciprocal are not finite).  Adding 1.5 2^23 rounds
// to nearest even and leaves the code in the low byte.
__device__ __noinline__ uint32_t int8_codes(float4 x, float scale) {
    auto code = [&](float v) { return (uint32_t)(max(-127, min(127, __float2int_rn(__fdiv_rn(v, scale)))) & 0xff); };
    return code(x.x) | code(x.y) << 8 | code(x.z) << 16 | code(x.w) << 24;
}
template <bool I8>
__device__ __forceinline__ uint32_t encode4(const float* x, float scale, float inv, bool exact) {
    if (!I8) {
        const unsigned lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0] * inv, x[1] * inv), __NV_SATFINITE, __NV_E4M3);
        const unsigned hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2] * inv, x[3] * inv), __NV_SATFINITE, __NV_E4M3);
        return lo | hi << 16;
    }
    uint32_t u[4];
    float off = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float t = x[e] * inv, r = t + 12582912.0f;
        u[e] = __float_as_uint(r);
        off = fmaxf(off, fabsf(t - (r - 12582912.0f)));
    }
    if (exact || off > 0.4999f) return int8_codes(make_float4(x[0], x[1], x[2], x[3]), scale);
    return __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
}

// The larger magnitude of each half of two bf16 pairs, as bits: those of values
// that are not finite are 0x7f80 and above.
__device__ __forceinline__ uint32_t max_bits(uint32_t m, uint4 v) {
    m = __vmaxu2(m, v.x & 0x7fff7fffu);
    m = __vmaxu2(m, v.y & 0x7fff7fffu);
    m = __vmaxu2(m, v.z & 0x7fff7fffu);
    return __vmaxu2(m, v.w & 0x7fff7fffu);
}
__device__ __forceinline__ uint32_t warp_max_bits(uint32_t m) {
    const uint32_t x = max(m & 0xffffu, m >> 16);
    return __reduce_max_sync(0xffffffffu, x);
}
// The largest finite magnitude among pieces i, i + step, ... below n of a block.
__device__ __noinline__ uint32_t finite_bits(const uint4* src, int i, int step, int n) {
    uint32_t m = 0;
    for (; i < n; i += step) {
        const uint4 v = src[i];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t b = (w[e >> 1] >> (16 * (e & 1))) & 0x7fffu;
            if (b < 0x7f80u) m = max(m, b);
        }
    }
    return m;
}
// `m` and the bits as a value: the block's largest finite magnitude.
__device__ __forceinline__ float bits_value(uint32_t m) { return __uint_as_float(m << 16); }

constexpr int kThreads = 128;

// Rounds `rows` rows of D values (row r at src + r * D) into dst and *scale, by
// the whole CTA of TH threads; at most 64 rows, read once and kept in registers.
template <bool I8, int D, int TH>
__device__ void round_block(const __nv_bfloat16* src, int rows, unsigned char* dst, float* scale) {
    __shared__ uint32_t red[2][TH / 32];
    constexpr int K = 64 * (D / 8) / TH;
    const int n8 = rows * (D / 8);
    uint4 v[K];
    uint32_t most = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = threadIdx.x + k * TH;
        v[k] = make_uint4(0, 0, 0, 0);
        if (i < n8) v[k] = reinterpret_cast<const uint4*>(src)[i];
        most = max_bits(most, v[k]);
    }
    most = warp_max_bits(most);
    if ((threadIdx.x & 31) == 0) red[0][threadIdx.x >> 5] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < TH / 32; ++w) most = max(most, red[0][w]);
    const bool odd = most >= 0x7f80u;
    if (odd) {
        most = __reduce_max_sync(0xffffffffu, finite_bits(reinterpret_cast<const uint4*>(src), threadIdx.x, TH, n8));
        if ((threadIdx.x & 31) == 0) red[1][threadIdx.x >> 5] = most;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < TH / 32; ++w) most = max(most, red[1][w]);
    }
    const float s = block_scale<I8>(bits_value(most)), inv = __fdiv_rn(1.0f, s);
    const bool exact = odd || !(inv < INFINITY);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = threadIdx.x + k * TH;
        if (i >= n8) break;
        float f[8];
        unpack8(v[k], f);
        reinterpret_cast<uint2*>(dst)[i] = make_uint2(encode4<I8>(f, s, inv, exact), encode4<I8>(f + 4, s, inv, exact));
    }
    if (threadIdx.x == 0) *scale = s;
    __syncthreads();
}

// ------------------------------------------------------------------ fill from a prompt
// One to four warps a block (64 values a lane), all of a block's rows in registers
// between the search for its largest magnitude and the rounding: each value is
// read once.  kThreads / 32 warps a CTA, on neighbouring blocks of one head.
template <int D, int R>
constexpr int kBlockWarps = R * D <= 2048 ? 1 : R * D / 2048;

template <bool I8, int D, int R>
__device__ void fill_blocks(const SkaQ8Cache& c, const __nv_bfloat16* src, int first, int len, unsigned char* dst,
                            float* scale, __nv_bfloat16* tail) {
    constexpr int WPB = kBlockWarps<D, R>, K = R * (D / 8) / (32 * WPB);
    __shared__ uint32_t red[2][kThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, idx = (warp % WPB) * 32 + lane;
    const int blk = first + warp / WPB, w = c.window;
    const int at = blk * R, stop = min(at + R, w);
    const int last = len - 1, cur = last % w;
    int round = last / w;  // the last round in which the block became full
    if (at <= cur && cur < stop - 1) {  // the block being written
        const __nv_bfloat16* s = src + ((size_t)round * w + at) * D;
        for (int i = idx; i < (cur - at + 1) * (D / 8); i += 32 * WPB)
            reinterpret_cast<uint4*>(tail)[i] = reinterpret_cast<const uint4*>(s)[i];
    }
    if (cur < stop - 1) --round;
    const int n8 = at < w && round >= 0 ? (stop - at) * (D / 8) : 0;
    const uint4* s4 = reinterpret_cast<const uint4*>(src + ((size_t)max(round, 0) * w + at) * D);
    uint4 v[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = idx + k * 32 * WPB;
        v[k] = i < n8 ? __ldg(s4 + i) : make_uint4(0, 0, 0, 0);
    }
    uint32_t most = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) most = max_bits(most, v[k]);
    most = warp_max_bits(most);
    auto join = [&](int turn) {  // over the block's warps
        if (WPB == 1) return;
        if (lane == 0) red[turn][warp] = most;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < WPB; ++k) most = max(most, red[turn][warp / WPB * WPB + k]);
    };
    join(0);
    const bool odd = most >= 0x7f80u;
    if (WPB == 1 ? odd : __syncthreads_or(odd)) {
        if (odd) most = __reduce_max_sync(0xffffffffu, finite_bits(s4, idx, 32 * WPB, n8));
        join(1);
    }
    if (n8 == 0) return;
    const float s = block_scale<I8>(bits_value(most)), inv = __fdiv_rn(1.0f, s);
    const bool exact = odd || !(inv < INFINITY);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = idx + k * 32 * WPB;
        if (i >= n8) break;
        float f[8];
        unpack8(v[k], f);
        reinterpret_cast<uint2*>(dst + (size_t)at * D)[i] = make_uint2(encode4<I8>(f, s, inv, exact), encode4<I8>(f + 4, s, inv, exact));
    }
    if (idx == 0) scale[blk] = s;
}

template <int D, int R>
__host__ __device__ constexpr int blocks_per_cta() {
    return kThreads / 32 / kBlockWarps<D, R>;
}
// CTAs that a row of nb blocks takes.
template <int R>
__host__ __device__ inline int row_ctas(int d, int nb) {
    const int per = d == 64 ? blocks_per_cta<64, R>() : blocks_per_cta<128, R>();
    return (nb + per - 1) / per;
}

template <bool I8, int R>
__global__ void __launch_bounds__(kThreads) ska_q8_fill_kernel(const SkaQ8FillParams p) {
    const SkaQ8Cache& c = p.c;
    const int nb = (c.window + R - 1) / R;
    const int kctas = row_ctas<R>(c.dk, nb), vctas = row_ctas<R>(c.dv, nb);
    const int per = kctas + c.H * vctas, b = blockIdx.x / per, i = blockIdx.x % per;
    int len = p.lengths ? p.lengths[b] : p.T;
    if (len < 0 || len > p.T) {
        if (threadIdx.x == 0) atomicOr(p.err, kErrBadValue);
        len = len < 0 ? 0 : p.T;
    }
    if (i == 0 && threadIdx.x == 0) c.pos[b] = len;
    if (len == 0) return;
    if (i < kctas) {
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.k) + (size_t)b * p.T * c.dk;
        unsigned char* dst = c.k + (size_t)b * c.window * c.dk;
        __nv_bfloat16* tail = static_cast<__nv_bfloat16*>(c.k_tail) + (size_t)b * R * c.dk;
        float* scale = c.k_scale + (size_t)b * nb;
        if (c.dk == 64) fill_blocks<I8, 64, R>(c, src, i * blocks_per_cta<64, R>(), len, dst, scale, tail);
        else fill_blocks<I8, 128, R>(c, src, i * blocks_per_cta<128, R>(), len, dst, scale, tail);
        return;
    }
    const int h = (i - kctas) / vctas, j = (i - kctas) % vctas;
    const size_t bh = (size_t)b * c.H + h;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.v) + bh * p.T * c.dv;
    unsigned char* dst = c.v + bh * c.window * c.dv;
    __nv_bfloat16* tail = static_cast<__nv_bfloat16*>(c.v_tail) + bh * R * c.dv;
    float* scale = c.v_scale + bh * nb;
    if (c.dv == 64) fill_blocks<I8, 64, R>(c, src, j * blocks_per_cta<64, R>(), len, dst, scale, tail);
    else fill_blocks<I8, 128, R>(c, src, j * blocks_per_cta<128, R>(), len, dst, scale, tail);
}

// ------------------------------------------------------------------ one token
// A CTA of eight warps takes a group of up to eight heads of one sequence and a
// range of its slots, 512 at a time:
//   scores  16 slots a warp, mma (slots x d_k) (d_k x 8 heads), the shared key rows
//           read once for the group's heads; into shared memory
//   weights a warp (or 8 / heads of them) per head: running maxima and sum, then
//           e = 2^(s + log2 v_scale - m' + 15) in f16, the rest of e times 2^11 in
//           f16: the block's scale is part of the exponent, so blocks of any scale meet
//           in one accumulator.  m' is the largest s + log2 v_scale, so e is at most
//           2^15, f16's last power of two; its parts have 22 bits down to 2^-14, fewer
//           below, and end at 2^-36, 2^-51 of the heaviest.  (Two halves of a weight of
//           at most 1 end at 2^-24 both: 32767 tokens behind one of 16 nats more, whose
//           value was zero, came out 6% off.)  Blocks of zeros count for nothing.
//   values  mma (d_v x 16 slots) (16 slots x the weights' two parts), the codes turned
//           into f16 pairs in registers (exact: e4m3 and int8 both fit f16's 11 bits)
// Without the tensor cores the conversions and products of the values alone would
// cost about 70 of an SM's 128 lane operations a clock at the memory's rate; with
// them each byte of V costs a quarter of a byte permutation, half a conversion and
// 1/256 of an mma a warp.  (Tried: mma on the codes themselves, e4m3 or int8, the
// weights in four parts of that type: right to 2^-24, but more instructions in all,
// 103 us against 85 at B256 H16 d128 window 512.)
// The tail's slots are scored with the others; their values follow behind the sweep,
// in bf16, under weights of at most 1 in three parts of bf16 (24 bits at any size): they
// have no scale, so the sums of the cache are brought to the scores' own exponent first
// and the tail has no say in m' (with a say in it, values of 1e-4 lost 5%).
// Each warp's tiles (the keys', then the values' of its head) come through a ring
// of its own, four tiles ahead (two or five measure the same).  Bound: the phases
// before and behind the sweep of V, in which little is on its way: a kernel that only
// streams the same V through the same rings takes 45 us, this one 82 (3.7 TB/s), of
// which the tail's rows cost 13; the bf16 rings' kernel (ska.cu) takes 119 for 1.9
// times the bytes.  One sequence, window 32768: 25 us, a second kernel joining 74
// splits included.  Registers are at the limit of two CTAs an SM (128); 16 bytes spill at
// d_k = d_v = 128, 32 at 64, none at the others.
constexpr int kWarps = 8, kDecThreads = 32 * kWarps, kChunk = 512, kStride = kChunk + 4, kRing = 4;

template <int DK, int DV>
struct Q8Smem {
    uint4 ring[kWarps][kRing][16 * (DK > DV ? DK : DV) / 16];
    float sc[kWarps][kStride];
    float sct[kWarps][64];             // the tail's scores
    __half wt[kWarps][2][kChunk];
    __nv_bfloat16 qs[kWarps][DK + 8];  // rows 16 bytes off one another's banks
    float part[kWarps][DV];
    float stat[kWarps][2];
    float lvs[kWarps][32];             // log2 of the chunk's value scales, by head and block
    float mx[kWarps][kWarps][2];       // a warp's largest scores by head, without and with the scales
    __half zero[16];
};

// Place of 16-byte piece x of row r in a tile of 16 rows, such that the lanes that
// read together (KEYS: rows g and pieces l4; else rows 2 l4 and pieces by g) spread
// over the banks.
template <int D, bool KEYS>
__device__ __forceinline__ int tile_place(int r, int x) {
    if (D == 128) return r * 8 + (KEYS ? x ^ ((r & 1) << 2) : x ^ (((r >> 1) & 3) << 1));
    const int line = r >> 1, at = (r & 1) * 4 + x;
    return line * 8 + (KEYS ? at : at ^ ((line & 3) << 1));
}
__device__ __forceinline__ void copy_piece(uint32_t dst, const unsigned char* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Starts the copy of a tile of 16 rows at `src`, which is contiguous.  Lane's
// pieces are 32 apart, and so are their places, up to one bit for every second.
template <int D, bool KEYS>
__device__ __forceinline__ void copy_tile(uint32_t dst, const unsigned char* src) {
    const int lane = threadIdx.x & 31;
    const int place = tile_place<D, KEYS>(lane / (D / 16), lane % (D / 16));
    const uint32_t at = dst + 16 * place, odd = D == 128 && !KEYS ? dst + 16 * (place ^ 4) : at;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) copy_piece((j & 1 ? odd : at) + 512 * j, src + 16 * lane + 512 * j);
}
// The same for a tile of which only rows [lo, hi) are in the cache: the others as
// the nearest that is.
template <int D, bool KEYS>
__device__ __noinline__ void copy_edge(uint32_t dst, const unsigned char* base, int t0, int lo, int hi) {
    const int lane = threadIdx.x & 31;
    for (int i = lane; i < D; i += 32) {
        const int r = i / (D / 16), x = i % (D / 16);
        const int u = min(max(t0 + r, lo), hi - 1);
        copy_piece(dst + 16 * tile_place<D, KEYS>(r, x), base + (size_t)u * D + 16 * x);
    }
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a <= 3.4e38f ? a : 0.0f;  // neither infinite nor NaN (bf16 ends at 3.39e38)
}

// A block of zeros has the scale 1, which is no measure of anything: the exponent of its
// value scale becomes -inf, so it neither lowers the weights of other blocks nor gets
// one.  `one`: the lane's block (`rows` of them at `block`) has the scale 1, which some
// other blocks have too, so their codes tell: the first 16 bytes, and if those are
// zeros all of it, eight lanes a block.  (A head that is all zeros reads its codes twice
// for it: B1 H16 d128 window 512 18 us instead of 11, B256 138 instead of 83.)
template <bool I8, int DV>
__device__ __noinline__ float without_zeros(const unsigned char* block, int rows, bool one, float exponent) {
    constexpr unsigned ALL = 0xffffffffu;
    constexpr uint32_t MAGNITUDE = I8 ? 0xffffffffu : 0x7f7f7f7fu;
    const int lane = threadIdx.x & 31, part = lane >> 3;
    const auto bits = [](const uint4& x) { return (x.x | x.y | x.z | x.w) & MAGNITUDE; };
    unsigned left = __ballot_sync(ALL, one && bits(*reinterpret_cast<const uint4*>(block)) == 0);
    while (left) {  // four blocks: part k of the warp has the k-th that is left
        unsigned mine = left;
        for (int k = 0; k < part; ++k) mine &= mine - 1;
        const int src = mine ? __ffs(mine) - 1 : 0;
        const uint4* q = reinterpret_cast<const uint4*>(__shfl_sync(ALL, reinterpret_cast<unsigned long long>(block), src));
        const int n = __shfl_sync(ALL, rows, src) * (DV / 16);
        uint32_t any = 0;
        if (mine) {
#pragma unroll 16
            for (int i = lane & 7; i < n; i += 8) any |= bits(q[i]);
        }
        const unsigned full = __ballot_sync(ALL, any != 0);
        const int at = __popc(left & ((1u << lane) - 1));
        if ((left >> lane & 1) && at < 4 && (full >> 8 * at & 0xff) == 0) exponent = -INFINITY;
        for (int k = 0; k < 4; ++k) left &= left - 1;
    }
    return exponent;
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Four codes as two f16 pairs.
template <bool I8>
__device__ __forceinline__ uint2 f16_pairs(uint32_t w) {
    if (I8) {  // 0x6400 | (code + 128) is 1024 + code + 128 in f16
        const uint32_t u = w ^ 0x80808080u;
        const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
        uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
        __half2 a = __hsub2(*reinterpret_cast<__half2*>(&lo), off), b = __hsub2(*reinterpret_cast<__half2*>(&hi), off);
        return make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
    }
    uint2 r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(r.x), "=r"(r.y) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}

// Heads of a group, groups, splits of the window and slots of each.
struct Q8Plan {
    int G, groups, splits, range;
    int cluster;   // the groups of a sequence form a cluster, and pos is advanced in the kernel
    float *m, *l, *o;  // partial results [B,H,splits], [B,H,splits], [B,H,splits,dv]
};

template <bool I8, int DK, int DV>
__global__ void __launch_bounds__(kDecThreads, 2) ska_q8_decode_kernel(const SkaQ8DecodeParams p, const Q8Plan pl) {
    constexpr int KW = DK / 16;    // words of codes a lane has of a key row
    constexpr int VB = DV / 8;     // value columns a lane has
    constexpr int MT = DV / 16;    // value tiles of 16 columns
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Q8Smem<DK, DV>& sm = *reinterpret_cast<Q8Smem<DK, DV>*>(smem_raw);
    auto& sc = sm.sc;
    auto& wt = sm.wt;
    auto& qs = sm.qs;
    auto& part = sm.part;
    auto& stat = sm.stat;
    const SkaQ8Cache& c = p.c;
    chain_next();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, l4 = lane & 3;
    const int group = blockIdx.x % pl.groups, b = blockIdx.x / pl.groups, split = blockIdx.y;
    const int h0 = group * pl.G, nh = min(pl.G, c.H - h0);
    const int w = c.window, R = c.block, nb = (w + R - 1) / R, rs = 31 - __clz(R);
    const int s0 = split * pl.range, wend = min(s0 + pl.range, w);  // this split's slots
    const size_t bh0 = (size_t)b * c.H + h0;
    // this warp's head: several warps share one where there are few
    const int wph = kWarps / nh, hd = min(warp / wph, nh - 1), sub = warp % wph;
    const bool busy = warp < wph * nh;
    const unsigned char* kc = c.k + (size_t)b * w * DK;
    const unsigned char* vc = c.v + (bh0 + hd) * w * DV;

    // What does not depend on the position is asked for before it is known: the
    // queries, the first chunk's scales and its key tiles (those behind the last
    // token too; their scores are not taken).
    const int pos = c.pos[b];
    uint4 q4 = make_uint4(0, 0, 0, 0);
    if (tid < nh * (DK / 8)) q4 = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + bh0 * DK)[tid];
    float ks_next, vs_next;  // a block a lane (32 of 16 slots at most)
    auto fetch_scales = [&](int c0) {
        const int blk = (c0 >> rs) + lane;
        ks_next = blk < nb ? c.k_scale[(size_t)b * nb + blk] : 1.0f;
        vs_next = warp < nh && blk < nb ? c.v_scale[(bh0 + warp) * nb + blk] : 1.0f;
    };
    fetch_scales(s0);
    // This warp's tiles in the order in which it takes them: of each chunk first the
    // keys' (every eighth tile), then the values' (every wph-th).
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(sm.ring[warp][0]);
    constexpr uint32_t TILE = sizeof(sm.ring[0][0]);
    int pc = s0, pk = s0 + 16 * warp, pv = s0 + 16 * sub;  // the next to ask for
    uint32_t slot_in = ring, slot_out = ring;
    auto ask_key = [&]() {
        if (pk + 16 > w) copy_edge<DK, true>(slot_in, kc, pk, pk, w);
        else copy_tile<DK, true>(slot_in, kc + (size_t)pk * DK);
        pk += 16 * kWarps;
        slot_in = slot_in == ring + (kRing - 1) * TILE ? ring : slot_in + TILE;
    };
    int asked = 0;
    for (; asked < kRing && pk < min(s0 + kChunk, wend); ++asked) {
        ask_key();
        asm volatile("cp.async.commit_group;" ::: "memory");
    }

    if (pl.cluster) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // pos is read
    const int n = pos < 0 ? 0 : pos < w ? pos + 1 : w;
    const int cur = pos < 0 ? 0 : pos % w, at = cur & ~(R - 1), fill = cur - at;
    const int s1 = min(wend, n);
    const bool tail_here = pos >= 0 && at >= s0 && at < s0 + pl.range;
    if (pos < 0 && tid == 0) atomicOr(p.err, kErrBadValue);
    const __nv_bfloat16* kin = static_cast<const __nv_bfloat16*>(p.k) + (size_t)b * DK;
    const __nv_bfloat16* vin = static_cast<const __nv_bfloat16*>(p.v) + bh0 * DV;
    __nv_bfloat16* kt = static_cast<__nv_bfloat16*>(c.k_tail) + (size_t)b * R * DK;
    __nv_bfloat16* vt = static_cast<__nv_bfloat16*>(c.v_tail) + bh0 * R * DV;

    // m of the scores, m2 of the cache's with the scales in them, 15 less
    float m = -INFINITY, m2 = -3e38f, l = 0.0f;
    float acc[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = 0.0f;

    // An edge tile holds slots of the block being written or behind the last token.
    auto is_edge = [&](int t0) { return (t0 & ~(R - 1)) == at || t0 + 16 > s1; };
    auto bounds = [&](int t0, int& lo, int& hi) {  // slots of a tile that are in the cache
        lo = (t0 & ~(R - 1)) == at ? max(t0, cur + 1) : t0;
        hi = min(t0 + 16, s1);
    };
    auto next_chunk = [&]() {
        pc += kChunk;
        pk = pc + 16 * warp;
        pv = pc + 16 * sub;
    };
    auto ask = [&]() {
        if (pc < s1) {
            const int c1 = min(pc + kChunk, s1), ke = min(pc + kChunk, wend);
            if (pk < ke) {
                ask_key();
            } else if (busy && pv < c1) {
                if (is_edge(pv)) {
                    int lo, hi;
                    bounds(pv, lo, hi);
                    if (lo >= hi) lo = pv, hi = s1;  // none of them: copied and not used
                    copy_edge<DV, false>(slot_in, vc, pv, lo, hi);
                } else {
                    copy_tile<DV, false>(slot_in, vc + (size_t)pv * DV);
                }
                pv += 16 * wph;
                slot_in = slot_in == ring + (kRing - 1) * TILE ? ring : slot_in + TILE;
            }
            if (pk >= ke && (!busy || pv >= c1)) next_chunk();
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto arrived = [&]() {  // the oldest tile that was asked for
        asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
        __syncwarp();
        const uint32_t t = slot_out;
        slot_out = slot_out == ring + (kRing - 1) * TILE ? ring : slot_out + TILE;
        return t;
    };

    if (s0 < s1) {
        if (!busy && pk >= min(pc + kChunk, wend)) next_chunk();
        for (; asked < kRing; ++asked) ask();
        // the new token's row of the tail (read from the inputs below), and the rows
        // before it toward L2
        if (tail_here) {
            if (group == 0 && tid < DK / 8)
                reinterpret_cast<uint4*>(kt + (size_t)fill * DK)[tid] = reinterpret_cast<const uint4*>(kin)[tid];
            for (int i = tid; i < nh * (DV / 8); i += kDecThreads) {
                const int hh = i / (DV / 8), x = i % (DV / 8);
                reinterpret_cast<uint4*>(vt + ((size_t)hh * R + fill) * DV)[x] =
                    reinterpret_cast<const uint4*>(vin + (size_t)hh * DV)[x];
            }
            for (int i = tid; i < fill * DK / 64; i += kDecThreads) prefetch_l2(kt + 64 * i);
            for (int i = tid; i < nh * fill * DV / 64; i += kDecThreads) {
                const int hh = i / (fill * DV / 64), x = i % (fill * DV / 64);
                prefetch_l2(vt + (size_t)hh * R * DV + 64 * x);
            }
        }
        // queries: as they are for the tail, and as f16 for the codes, each head's
        // times a power of two that puts its largest near 2^14 (exact)
        if (tid < kWarps * (DK / 8)) reinterpret_cast<uint4*>(qs[tid / (DK / 8)])[tid % (DK / 8)] = q4;
        if (tid < 16) sm.zero[tid] = __half(0.0f);
        __syncthreads();
        // lane's dimensions of a row: 16 l4 .. + 15, and 64 more on for d_k = 128; heads by g
        uint32_t qf[KW][2];
        float qmul;
        {
            float qv[KW][4], most = 0.0f;
#pragma unroll
            for (int j = 0; j < KW; ++j) {
                const uint2 u = *reinterpret_cast<const uint2*>(&qs[g][(j >> 2) * 64 + l4 * 16 + (j & 3) * 4]);
                qv[j][0] = __uint_as_float(u.x << 16);
                qv[j][1] = __uint_as_float(u.x & 0xffff0000u);
                qv[j][2] = __uint_as_float(u.y << 16);
                qv[j][3] = __uint_as_float(u.y & 0xffff0000u);
#pragma unroll
                for (int e = 0; e < 4; ++e) most = fmaxf(most, finite_abs(qv[j][e]));
            }
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
            int e2 = most > 0.0f ? (int)(__float_as_uint(most) >> 23) - 127 - 14 : 0;  // most in 2^(e2+14) .. 2^(e2+15)
            e2 = max(-126, e2);
            const float inv = __uint_as_float((unsigned)(127 - e2) << 23);
            qmul = __uint_as_float((unsigned)(127 + e2) << 23) * (p.scale * kLog2e);
#pragma unroll
            for (int j = 0; j < KW; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const __half2 hv = __floats2half2_rn(qv[j][2 * e] * inv, qv[j][2 * e + 1] * inv);
                    qf[j][e] = *reinterpret_cast<const uint32_t*>(&hv);
                }
        }
        // multipliers of the two heads whose scores this lane gets from an mma
        const float qm0 = __shfl_sync(0xffffffffu, qmul, 8 * l4), qm1 = __shfl_sync(0xffffffffu, qmul, 8 * l4 + 4);

        for (int c0 = s0; c0 < s1; c0 += kChunk) {
            const int c1 = min(c0 + kChunk, s1);
            const float ksl = ks_next;
            if (warp < nh) {
                // blocks of the chunk with a slot whose value comes from the codes
                const int first = c0 + (lane << rs);
                const bool one = vs_next == 1.0f && lane < kChunk >> rs && first < s1 && (first != at || pos >= w);
                float e = __log2f(vs_next);
                if (__any_sync(0xffffffffu, one))
                    e = without_zeros<I8, DV>(c.v + ((bh0 + warp) * w + (one ? first : 0)) * DV, min(R, w - first), one, e);
                sm.lvs[warp][lane] = e;
            }
            if (c0 + kChunk < s1) fetch_scales(c0 + kChunk);
            __syncthreads();
            float cm[2] = {-INFINITY, -INFINITY}, cn[2] = {-3e38f, -3e38f};  // of heads 2 l4 and 2 l4 + 1
            // ---- scores
            const int ke = min(c0 + kChunk, wend);
            for (int t0 = c0 + 16 * warp; t0 < ke; t0 += 16 * kWarps) {
                int lo, hi;
                bounds(t0, lo, hi);
                const float ks = __shfl_sync(0xffffffffu, ksl, (t0 - c0) >> rs);
                const uint32_t tile = arrived();
                uint32_t ka[2][KW];
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int x = 0; x < DK / 64; ++x) {
                        const uint4 v = lds128(tile + 16 * tile_place<DK, true>(g + 8 * r, 4 * x + l4));
                        ka[r][4 * x] = v.x; ka[r][4 * x + 1] = v.y; ka[r][4 * x + 2] = v.z; ka[r][4 * x + 3] = v.w;
                    }
                __syncwarp();
                ask();
                if (lo >= hi) continue;  // all of them in the tail
                float s[4] = {0.0f, 0.0f, 0.0f, 0.0f}, s2[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // two chains of products
#pragma unroll
                for (int j = 0; j < KW; ++j) {
                    const uint2 x = f16_pairs<I8>(ka[0][j]), y = f16_pairs<I8>(ka[1][j]);
                    const uint32_t a[4] = {x.x, y.x, x.y, y.y};
                    mma_f16(j & 1 ? s2 : s, a, qf[j][0], qf[j][1]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) s[e] += s2[e];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int u = t0 + g + 8 * r;
                    if (u < lo || u >= hi) continue;
                    const float a = s[2 * r] * (ks * qm0), e = s[2 * r + 1] * (ks * qm1);
                    sc[2 * l4][u - c0] = a;
                    sc[2 * l4 + 1][u - c0] = e;
                    cm[0] = fmaxf(cm[0], a);
                    cm[1] = fmaxf(cm[1], e);
                    cn[0] = fmaxf(cn[0], a + sm.lvs[2 * l4][(t0 - c0) >> rs]);
                    cn[1] = fmaxf(cn[1], e + sm.lvs[2 * l4 + 1][(t0 - c0) >> rs]);
                }
            }
            const bool tail_now = tail_here && at >= c0 && at < c0 + kChunk;
            if (tail_now)
                for (int t0 = 16 * warp; t0 <= fill; t0 += 16 * kWarps) {
                    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    const __nv_bfloat16* row[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int i = min(t0 + g + 8 * r, fill);
                        row[r] = i == fill ? kin : kt + (size_t)i * DK;
                    }
#pragma unroll
                    for (int j = 0; j < KW; ++j) {
                        const int d = (j >> 2) * 64 + l4 * 16 + (j & 3) * 4;
                        const uint2 x = *reinterpret_cast<const uint2*>(row[0] + d), y = *reinterpret_cast<const uint2*>(row[1] + d);
                        const uint2 qv = *reinterpret_cast<const uint2*>(&qs[g][d]);
                        const uint32_t a[4] = {x.x, y.x, x.y, y.y};
                        mma_bf16(s, a, qv.x, qv.y);
                    }
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int i = t0 + g + 8 * r;
                        if (i > fill) continue;
                        const float a = s[2 * r] * (p.scale * kLog2e), e = s[2 * r + 1] * (p.scale * kLog2e);
                        sc[2 * l4][at - c0 + i] = sm.sct[2 * l4][i] = a;
                        sc[2 * l4 + 1][at - c0 + i] = sm.sct[2 * l4 + 1][i] = e;
                        cm[0] = fmaxf(cm[0], a);
                        cm[1] = fmaxf(cm[1], e);
                    }
                }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    cm[k] = fmaxf(cm[k], __shfl_xor_sync(0xffffffffu, cm[k], o));
                    cn[k] = fmaxf(cn[k], __shfl_xor_sync(0xffffffffu, cn[k], o));
                }
                if (g == 0) {
                    sm.mx[warp][2 * l4 + k][0] = cm[k];
                    sm.mx[warp][2 * l4 + k][1] = cn[k];
                }
            }
            __syncthreads();
            // ---- weights of this warp's head, and its values
            if (busy) {
                float nm = m, nm2 = m2;
#pragma unroll
                for (int k = 0; k < kWarps; ++k) {
                    nm = fmaxf(nm, sm.mx[k][hd][0]);
                    nm2 = fmaxf(nm2, sm.mx[k][hd][1] - 15.0f);
                }
                const float f2 = ex2_fast(m2 - nm2);
                l *= m == nm ? 1.0f : ex2_fast(m - nm);
                m = nm;
                m2 = nm2;
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][e] *= f2;
                const int tiles = (c1 - c0 + 15) / 16;
                const int mine = ((tiles - sub + wph - 1) / wph) * 16;
                for (int i = 4 * lane; i < mine; i += 128) {  // four neighbouring slots a lane
                    const int x = 16 * (sub + wph * (i >> 4)) + (i & 15), u = c0 + x;
                    const float ls = sm.lvs[hd][x >> rs] - m2;
                    const float4 s4 = *reinterpret_cast<const float4*>(&sc[hd][x]);
                    const float sv[4] = {s4.x, s4.y, s4.z, s4.w};
                    float e[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const bool in = u + k < c1;
                        l += in ? ex2_fast(sv[k] - m) : 0.0f;
                        e[k] = in && (u + k < at || u + k > cur) ? ex2_fast(sv[k] + ls) : 0.0f;
                    }
                    const __half2 h0 = __floats2half2_rn(e[0], e[1]), h1 = __floats2half2_rn(e[2], e[3]);
                    const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
                    const __half2 r0 = __floats2half2_rn((e[0] - f0.x) * 2048.0f, (e[1] - f0.y) * 2048.0f);
                    const __half2 r1 = __floats2half2_rn((e[2] - f1.x) * 2048.0f, (e[3] - f1.y) * 2048.0f);
                    *reinterpret_cast<uint2*>(&wt[warp][0][i]) =
                        make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
                    *reinterpret_cast<uint2*>(&wt[warp][1][i]) =
                        make_uint2(*reinterpret_cast<const uint32_t*>(&r0), *reinterpret_cast<const uint32_t*>(&r1));
                }
                __syncwarp();
                // lanes g = 0 and 1 have the weights' two parts, the others zeros
                uint32_t wp = (uint32_t)__cvta_generic_to_shared(g < 2 ? &wt[warp][g][2 * l4] : &sm.zero[2 * l4]);
                const uint32_t wstep = g < 2 ? 32 : 0;
                // rows 2 l4 and 2 l4 + 1; 8 on lies 8 rows further
                const uint32_t off0 = VB == 16 ? 16 * tile_place<DV, false>(2 * l4, g)
                                               : 16 * tile_place<DV, false>(2 * l4, g >> 1) + 8 * (g & 1);
                const uint32_t off1 = VB == 16 ? 16 * tile_place<DV, false>(2 * l4 + 1, g)
                                               : 16 * tile_place<DV, false>(2 * l4 + 1, g >> 1) + 8 * (g & 1);
#pragma unroll 2
                for (int t0 = c0 + 16 * sub; t0 < c1; t0 += 16 * wph, wp += wstep) {
                    const uint32_t tile = arrived();
                    uint32_t v[4][VB / 4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {  // tokens 2 l4, 2 l4 + 1, and 8 on
                        const uint32_t a = tile + (r & 1 ? off1 : off0) + (r & 2 ? 8 * DV : 0);
                        if (VB == 16) {
                            const uint4 x = lds128(a);
                            v[r][0] = x.x; v[r][1] = x.y; v[r][VB / 4 - 2] = x.z; v[r][VB / 4 - 1] = x.w;
                        } else {
                            const uint2 x = lds64(a);
                            v[r][0] = x.x; v[r][1] = x.y;
                        }
                    }
                    const uint32_t b0 = lds32(wp), b1 = lds32(wp + 16);
                    __syncwarp();
                    ask();
                    if (is_edge(t0)) {
                        int lo, hi;
                        bounds(t0, lo, hi);
                        if (lo >= hi) continue;  // all of them in the tail
                    }
#pragma unroll
                    for (int i = 0; i < MT; ++i) {  // columns VB g + 2 i and + 1
                        const unsigned sel = i & 1 ? 0x7362u : 0x5140u;
                        const uint2 x = f16_pairs<I8>(__byte_perm(v[0][i >> 1], v[1][i >> 1], sel));
                        const uint2 y = f16_pairs<I8>(__byte_perm(v[2][i >> 1], v[3][i >> 1], sel));
                        const uint32_t a[4] = {x.x, x.y, y.x, y.y};
                        mma_f16(acc[i], a, b0, b1);
                    }
                }
            }
            if (c0 + kChunk < s1) __syncthreads();
        }
        if (busy) {
            // From here on the sums are relative to m.  In two steps: the scales alone may be
            // past float32's exponents.
            const float f = ex2_fast(0.5f * (m2 - m)), f1 = f * 0x1p-11f;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                acc[i][0] = acc[i][0] * f * f;
                acc[i][1] = acc[i][1] * f1 * f;
                acc[i][2] = acc[i][2] * f * f;
                acc[i][3] = acc[i][3] * f1 * f;
            }
            if (tail_here)
                for (int t0 = 16 * sub; t0 <= fill; t0 += 16 * wph) {
                    const __nv_bfloat16* row[4];
                    float e[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int i = t0 + 2 * l4 + (r & 1) + 4 * (r & 2), ic = min(i, fill);
                        row[r] = (ic == fill ? vin + (size_t)hd * DV : vt + ((size_t)hd * R + ic) * DV) + VB * g;
                        e[r] = i <= fill ? ex2_fast(sm.sct[hd][ic] - m) : 0.0f;
                        for (int x = 0; x < g && x < 3; ++x) e[r] -= __bfloat162float(__float2bfloat16_rn(e[r]));
                        if (g > 2) e[r] = 0.0f;
                    }
                    const uint32_t b0 = bf16_pair(e[0], e[1]), b1 = bf16_pair(e[2], e[3]);
#pragma unroll
                    for (int x = 0; x < VB / 8; ++x) {  // eight columns of the four rows at once
                        uint32_t v[4][4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const uint4 q = *reinterpret_cast<const uint4*>(row[r] + 8 * x);
                            v[r][0] = q.x; v[r][1] = q.y; v[r][2] = q.z; v[r][3] = q.w;
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t a[4] = {__byte_perm(v[0][i], v[1][i], 0x5410), __byte_perm(v[0][i], v[1][i], 0x7632),
                                                   __byte_perm(v[2][i], v[3][i], 0x5410), __byte_perm(v[2][i], v[3][i], 0x7632)};
                            mma_bf16(acc[4 * x + i], a, b0, b1);
                        }
                    }
                }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // key tiles that no position needed
    // ---- join the parts of the weights, then the warps of a head
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) {
        stat[warp][0] = m;
        stat[warp][1] = l;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        float x = acc[i][0] + acc[i][1], y = acc[i][2] + acc[i][3];
        x += __shfl_down_sync(0xffffffffu, x, 1);
        y += __shfl_down_sync(0xffffffffu, y, 1);
        if (l4 == 0) {
            part[warp][VB * g + 2 * i] = x;
            part[warp][VB * g + 2 * i + 1] = y;
        }
    }
    __syncthreads();
    if (pos >= 0)
        for (int i = tid; i < nh * DV; i += kDecThreads) {
            const int hh = i / DV, x = i % DV, w0 = hh * wph;
            // the warps of a head saw the same scores, so their maxima agree
            float a = 0.0f, sum = 0.0f;
            for (int k = 0; k < wph; ++k) {
                a += part[w0 + k][x];
                sum += stat[w0 + k][1];
            }
            const size_t bh = bh0 + hh;
            if (pl.splits == 1) {
                static_cast<__nv_bfloat16*>(p.o)[bh * DV + x] = __float2bfloat16_rn(a / sum);
            } else {
                const size_t at2 = bh * pl.splits + split;
                if (s0 < s1) pl.o[at2 * DV + x] = a;
                if (x == 0) {
                    pl.m[at2] = s0 < s1 ? stat[w0][0] : -INFINITY;
                    pl.l[at2] = sum;
                }
            }
        }
    // ---- the block if it is full with the new token
    if (tail_here) {
        if (cur == w - 1 || fill == R - 1) {
            __syncthreads();
            if (group == 0)
                round_block<I8, DK, kDecThreads>(kt, fill + 1, c.k + ((size_t)b * w + at) * DK, c.k_scale + (size_t)b * nb + at / R);
            for (int hh = 0; hh < nh; ++hh)
                round_block<I8, DV, kDecThreads>(vt + (size_t)hh * R * DV, fill + 1, c.v + ((bh0 + hh) * w + at) * DV,
                                    c.v_scale + (bh0 + hh) * nb + at / R);
        }
    }
    if (pl.cluster) {
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (p.advance && group == 0 && tid == 0 && pos >= 0) c.pos[b] = pos + 1;
    }
}

// Joins the splits of a window, one CTA a head, and advances the positions.
constexpr int kJoinThreads = 256, kMostSplits = 128;
template <int DV>
__global__ void __launch_bounds__(kJoinThreads) ska_q8_join_kernel(const SkaQ8DecodeParams p, const Q8Plan pl) {
    chain_wait();
    constexpr int ROWS = kJoinThreads / DV;
    __shared__ float f[kMostSplits], red[2][kJoinThreads / 32], part[ROWS][DV];
    const SkaQ8Cache& c = p.c;
    const int bh = blockIdx.x, tid = threadIdx.x, b = bh / c.H, pos = c.pos[b];
    if (pos < 0) return;
    // a split's share is 2^(m_k - m); one without slots has m_k = -inf and no values
    float m = tid < pl.splits ? pl.m[(size_t)bh * pl.splits + tid] : -INFINITY;
    const float l = tid < pl.splits ? pl.l[(size_t)bh * pl.splits + tid] : 0.0f;
    float mx = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if ((tid & 31) == 0) red[0][tid >> 5] = mx;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kJoinThreads / 32; ++k) mx = fmaxf(mx, red[0][k]);
    const float share = m == -INFINITY ? 0.0f : ex2_fast(m - mx);
    if (tid < pl.splits) f[tid] = share;
    float sum = share * l;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((tid & 31) == 0) red[1][tid >> 5] = sum;
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kJoinThreads / 32; ++k) sum += red[1][k];
    const int x = tid % DV, row = tid / DV;
    const float* o = pl.o + (size_t)bh * pl.splits * DV + x;
    float a = 0.0f;
#pragma unroll 8
    for (int k = row; k < pl.splits; k += ROWS) {
        const float v = o[(size_t)k * DV];
        a = f[k] == 0.0f ? a : fmaf(f[k], v, a);
    }
    part[row][x] = a;
    __syncthreads();
    if (tid < DV) {
#pragma unroll
        for (int k = 1; k < ROWS; ++k) a += part[k][x];
        static_cast<__nv_bfloat16*>(p.o)[(size_t)bh * DV + x] = __float2bfloat16_rn(a / sum);
    }
    // a sequence's other CTAs only ask whether pos is negative
    if (p.advance && bh % c.H == 0 && tid == 0) c.pos[b] = pos + 1;
}

__global__ void ska_q8_advance_kernel(int* pos, int B) {
    chain_wait();
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b < B && pos[b] >= 0) pos[b] += 1;
}

// Heads of a group.  More heads share one read of the keys and make fewer CTAs, but
// leave fewer warps to a head: a CTA of G heads takes about 9 + 3.9 G us for 512 slots
// (G = 1 .. 8, d 128, two CTAs an SM), so the group is the one whose rounds of two CTAs
// an SM cost least: the smallest that fits one round, large ones for large batches.
// Measured (us, G = 1 / 2 / 4 / 8; H16 d128, * the choice): window 512 of B1 10.4* / 12.3 /
// 16.0 / 23.9, B16 13.3* / 16.1 / 16.4 / 24.2, B32 25.3 / 17.7* / 19.8 / 29.0, B64 44.1 /
// 33.4 / 25.1* / 29.3, B256 160 / 119 / 91 / 79*; window 32768 of B1 31.4 / 24.6 / 23.7* /
// 25.7; window 4096 of B8 32.5 / 24.8 / 22.5* / 22.6.  B128 H12: 65.8 / 47.3 / 45.6, and
// 37.8* with G = 6.  The cost was fitted at d 128 and 512 slots; at d 64 the choice is
// within 6% of the best of G = 1, 2, 3, 4, 6, 8 for windows of 20 (B1 H12 7.5 against 7.3, B32 H16
// 9.7 / 9.2, B128 H16 14.6, B256 H12 22.0), 64 (B256 H24 43.5), 128 (B256 H12 33.6), 512 (B1 9.2, B32 13.4
// against 13.1, B128 H12 31.0, B256 H16 56.0), 4096 (B8 H16 19.4) and 32768 (B1 18.7).
int group_heads(int B, int H, int window) {
    const long long round = 2LL * sm_count(), chunks = (window + kChunk - 1) / kChunk;
    int best = 1;
    double least = 0.0;
    for (int G = 1; G <= 8 && G <= H; ++G) {
        const long long ctas = B * chunks * ((H + G - 1) / G);
        const double cost = (double)((ctas + round - 1) / round) * (9.0 + 3.9 * G);
        if (G == 1 || cost < least) {
            least = cost;
            best = G;
        }
    }
    return best;
}

Q8Plan plan(const SkaQ8DecodeParams& p) {
    Q8Plan pl;
    pl.G = group_heads(p.c.B, p.c.H, p.c.window);
    pl.groups = (p.c.H + pl.G - 1) / pl.G;
    const long long units = (long long)p.c.B * pl.groups;
    // two CTAs an SM; each split of at least 256 slots, in multiples of the largest block
    long long P = units > 0 ? 2LL * sm_count() / units : 1;
    // windows of a chunk stay whole (10.4 us for B1 H16 window 512; 10.5 for window 1024 split in four)
    const long long most = p.c.window <= kChunk ? 1 : (p.c.window + 255) / 256;  // at most kMostSplits, the window at most 32768
    if (P > most) P = most;
    if (P < 1) P = 1;
    const int range = (int)((p.c.window + P - 1) / P + 63) / 64 * 64;
    pl.range = range;
    pl.splits = (p.c.window + range - 1) / range;
    pl.cluster = 0;
    pl.m = pl.l = pl.o = nullptr;
    return pl;
}

size_t plan_bytes(const SkaQ8DecodeParams& p, const Q8Plan& pl) {
    return pl.splits == 1 ? 0 : (size_t)p.c.B * p.c.H * pl.splits * (p.c.dv + 2) * 4;
}

// The groups of a sequence that run as one cluster, which advances the position itself;
// beyond, a second kernel does.  More than eight need the opt-in size.  Measured (us on
// the GPU, second kernel / cluster): 12 groups of B2 window 300 9.4 / 9.4, of B20 window
// 512 13.1 / 13.5: what a cluster of twelve saves is the second launch's 2 us of host time
// in calls that the host bounds.  16 groups find room on the GPU less often: of B1
// 10.4 / 10.4, of B8 10.5 / 13.1, of B16 13.1 / 21.5.  (Between 12 and 16: not measured.)
constexpr int kMostCluster = 12;

template <bool I8, int DK, int DV>
cudaError_t launch_decode_cfg(const SkaQ8DecodeParams& p, Q8Plan pl, cudaStream_t s) {
    const size_t need = plan_bytes(p, pl);
    if (need && p.ws_bytes < need) {
        pl.splits = 1;
        pl.range = (p.c.window + 63) / 64 * 64;
    }
    if (pl.splits > 1) {
        const size_t rows = (size_t)p.c.B * p.c.H * pl.splits;
        pl.o = static_cast<float*>(p.ws);
        pl.m = pl.o + rows * DV;
        pl.l = pl.m + rows;
    }
    pl.cluster = pl.splits == 1 && pl.groups <= kMostCluster;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)p.c.B * pl.groups), pl.splits);
    cfg.blockDim = dim3(kDecThreads);
    cfg.dynamicSmemBytes = sizeof(Q8Smem<DK, DV>);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    if (pl.cluster) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = pl.groups;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    auto kern = ska_q8_decode_kernel<I8, DK, DV>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cfg.dynamicSmemBytes);
    if (e == cudaSuccess && pl.cluster && pl.groups > 8)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kern, p, pl);
    if (e != cudaSuccess) return e;
    if (pl.splits > 1) {
        e = launch_chained(ska_q8_join_kernel<DV>, dim3((unsigned)(p.c.B * p.c.H)), kJoinThreads, 0, s, p, pl);
    } else if (!pl.cluster && p.advance) {
        e = launch_chained(ska_q8_advance_kernel, dim3((p.c.B + 255) / 256), 256, 0, s, p.c.pos, p.c.B);
    }
    return e;
}

template <bool I8>
cudaError_t launch_decode_t(const SkaQ8DecodeParams& p, cudaStream_t s) {
    const Q8Plan pl = plan(p);
    if (p.c.dk == 64)
        return p.c.dv == 64 ? launch_decode_cfg<I8, 64, 64>(p, pl, s) : launch_decode_cfg<I8, 64, 128>(p, pl, s);
    return p.c.dv == 64 ? launch_decode_cfg<I8, 128, 64>(p, pl, s) : launch_decode_cfg<I8, 128, 128>(p, pl, s);
}

}  // namespace

namespace {
template <bool I8, int R>
cudaError_t launch_fill(const SkaQ8FillParams& p, cudaStream_t s) {
    const int nb = (p.c.window + R - 1) / R;
    const long long grid = p.c.B * (row_ctas<R>(p.c.dk, nb) + (long long)p.c.H * row_ctas<R>(p.c.dv, nb));
    ska_q8_fill_kernel<I8, R><<<(unsigned)grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}
}  // namespace

cudaError_t launch_ska_q8_fill(const SkaQ8FillParams& p, cudaStream_t s) {
    switch (p.c.block) {
        case 16: return p.c.int8 ? launch_fill<true, 16>(p, s) : launch_fill<false, 16>(p, s);
        case 32: return p.c.int8 ? launch_fill<true, 32>(p, s) : launch_fill<false, 32>(p, s);
        default: return p.c.int8 ? launch_fill<true, 64>(p, s) : launch_fill<false, 64>(p, s);
    }
}

size_t ska_q8_decode_workspace(const SkaQ8DecodeParams& p) { return plan_bytes(p, plan(p)); }

cudaError_t launch_ska_q8_decode(const SkaQ8DecodeParams& p, cudaStream_t s) {
    return p.c.int8 ? launch_decode_t<true>(p, s) : launch_decode_t<false>(p, s);
}

}  // namespace rdm
