// ssm_bwd.cu -- reverse mode of the selective state space scan (ssm.cu).  With
// go the gradient of the output, p_t = go silu(z_t) the gradient of y before the
// gate and G_t the gradient of s_t with all that follows it:
//
//   G_t = C_t p_t + exp(delta_{t+1} A) G_{t+1}           (G_T takes grad_ST too)
//   dC_t = sum_c p s_t        dB_t = sum_c G_t delta u       dz = go y silu'(z)
//   q_t = sum_n G_t B_t       w_t = G_t exp(delta A) s_{t-1}
//   ddelta = u q + sum_n w A  dA = sum_t w delta             du = delta q + d p
//   dzc = du silu'(zc)        dx_t = sum_i w_i dzc_{t+i}     dw_i = sum_t dzc_t x_{t-i}
//
// A block has CPB channels of one (b, h), four states a thread, and walks its
// chunks of 16 tokens backwards.  From the state saved before a chunk it runs the
// recurrence forward again, keeps the states before each four tokens, then takes
// the fours backwards, their own states and decays in registers.  Sums over n are
// shuffles within a channel's lanes for four tokens at a time, sums over channels
// (dB, dC) a transposing reduction over the warp's channels, then shared memory over
// the block's warps, then one row of partial sums per block that a last kernel adds
// up in a fixed order: no atomics, so the same call gives the same bits.  Sequences
// are cut into segments as in the forward; a first launch then runs G alone over
// each segment but the first from zero, and each block folds the segments behind its
// own.  The convolution's reach over a segment's end is added by the last kernel.
// Bound: instructions (145 a warp, token and 128 states, 54% of the issue slots) and
// the shared-memory pipe (41%); the exponentials, the floor, are 27%.  B4 H24 T2048
// D64 N16 bf16: forward and backward 554 us.  float32 is at the limit of the registers
// from N = 32 on: 12 to 16 bytes spill there, none elsewhere.
#include "launch.h"
#include "ssm_common.cuh"

namespace rdm {
namespace {

using namespace ssm;

constexpr int kQuads = kSsmChunk / 4;
constexpr int kPar = 7;  // per-channel sums: dt_bias, feedthrough, conv bias, four taps

struct BwdWork {
    int P, len, nblk;        // segments, tokens of each, blocks of channels a head
    float *local, *dsum;     // [seg][B,H,D,N], [seg][B,H,D]: G at a segment's begin from zero, its sum of delta
    float *part;             // [B,H,nblk,T,2N] sums over a block's channels: dB, dC
    float *pA, *pPar;        // [seg,B][H,D,N], [seg,B][kPar][H,D]
    float *edge;             // [seg][B,H][2][3][D]: dx of the last three tokens so far, dzc of the first three
    float *saved;
};

template <int N>
struct Red {
    static constexpr int F = N <= 32 ? 16 : N == 64 ? 8 : 2;  // tokens between two sums over the warps
};

// Threads of the element-wise warps: one for each two channels by four tokens of
// a chunk.
template <int CPB>
constexpr int kEw = kQuads * (CPB / 2) < 32 ? 32 : kQuads * (CPB / 2);

template <typename T, int N, int CPB, bool LOCAL>
struct BwdSmem {
    using L = Lay<N, CPB>;
    using Arr = float[kQuads][L::PLACES][4];
    static constexpr int M = LOCAL ? 1 : 2;
    Arr D[2], P[2];              // delta, p
    Arr U[M];
    Arr Y[M], Q[M], E[M];        // sums over n: C s, G B, w A
    Arr F[M], S[M], Z[M];        // silu'(zc), d delta / d dt, go silu'(z); the element-wise threads' own
    float C5[M][LOCAL ? 1 : kQuads + 1][L::PLACES][4];  // dzc, and the chunk behind's first four
    typename Four<T>::Raw B[LOCAL ? 1 : 3][kSsmChunk][N / 4];
    typename Four<T>::Raw C[3][kSsmChunk][N / 4];
    float R[LOCAL ? 1 : L::THREADS / 32][LOCAL ? 1 : Red<N>::F][2 * N];
    float par[kPar][kQuads][CPB];
};

template <int ID, int THREADS>
__device__ __forceinline__ void part_sync() {
    asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(THREADS) : "memory");
}

// Blocks an SM for a block's scan threads: what their registers leave room for.
constexpr int resident(int threads) { return threads > 128 ? 1 : threads > 64 ? 2 : 4; }

// Scan warps and element-wise warps, a chunk apart as in the forward: while the
// scan warps run chunk k (forward, then backwards), the others finish chunk k - 1
// and make delta, u and p of chunk k + 1.
template <typename T, int N, int CPB, bool LOCAL>
__global__ void __launch_bounds__(CPB * N / 4 + kEw<CPB>, resident(CPB * N / 4))
    ssm_bwd_kernel(const SsmBwdParams bp, const BwdWork wk) {
    using L = Lay<N, CPB>;
    using Raw = typename Pair<T>::Raw;
    using Quad = typename Four<T>::Raw;
    constexpr int LPC = L::LPC, TH = L::THREADS, EW = kEw<CPB>, UNITS = kQuads * (CPB / 2), WARPS = TH / 32, F = Red<N>::F;
    constexpr int CW = 32 / LPC;  // channels a warp
    if (!LOCAL) chain_wait();
    chain_next();
    extern __shared__ __align__(16) unsigned char smem_raw[];
    BwdSmem<T, N, CPB, LOCAL>& sm = *reinterpret_cast<BwdSmem<T, N, CPB, LOCAL>*>(smem_raw);
    const SsmParams& p = bp.f;
    const int bh = blockIdx.x / wk.nblk, blk = blockIdx.x % wk.nblk, c0 = blk * CPB;
    const int b = bh / p.H, h = bh % p.H, seg = blockIdx.y + (LOCAL ? 1 : 0);
    const int len = seq_len(p, b);
    const int begin = seg * wk.len, segend = min(begin + wk.len, p.T);
    const int end = min(segend, len);
    if (LOCAL && begin >= len) return;
    const int chunks = end > begin ? (end - begin + kSsmChunk - 1) / kSsmChunk : 0;
    const int tlast = begin + (chunks - 1) * kSsmChunk;  // first token of the chunk that is taken first
    const size_t row0 = (size_t)bh * p.T;
    const size_t states = (size_t)p.B * p.H * p.D;

    if (threadIdx.x >= TH) {  // ---------------- element-wise warps
        const int tid = threadIdx.x - TH;
        const T* x = static_cast<const T*>(p.x) + row0 * p.D + c0;
        const T* dt = static_cast<const T*>(p.dt) + row0 * p.D + c0;
        const T* z = p.z ? static_cast<const T*>(p.z) + row0 * p.D + c0 : nullptr;
        const T* gy = static_cast<const T*>(bp.gy) + row0 * p.D + c0;
        T* dx = static_cast<T*>(bp.dx) + row0 * p.D + c0;
        T* ddt = static_cast<T*>(bp.ddt) + row0 * p.D + c0;
        T* dz = static_cast<T*>(bp.dz) + row0 * p.D + c0;
        const T* cs = p.cs_in ? static_cast<const T*>(p.cs_in) + (size_t)bh * (p.W - 1) * p.D + c0 : nullptr;
        const size_t grow = (size_t)(b * p.G + h / (p.H / p.G)) * p.T;
        const T* Bm = static_cast<const T*>(p.Bm) + grow * N;
        const T* Cm = static_cast<const T*>(p.Cm) + grow * N;
        // channels cp, cp + 1 of tokens 4 uq .. 4 uq + 3 of a chunk
        const bool has_unit = tid < UNITS;
        const int uq = min(tid / (CPB / 2), kQuads - 1), cp = 2 * (tid % (CPB / 2)), pl = cp >> 1;
        const unsigned off = (unsigned)(4 * uq) * p.D + cp;
        float w[4][2] = {}, cb[2] = {0.0f, 0.0f}, bias[2] = {0.0f, 0.0f}, feed[2] = {0.0f, 0.0f};
        float par[kPar][2] = {};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int hc = h * p.D + c0 + cp + e;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < p.W) w[i][e] = p.cw[(size_t)hc * p.W + i];
            if (p.cb) cb[e] = p.cb[hc];
            if (p.dt_bias) bias[e] = p.dt_bias[hc];
            if (p.dfeed) feed[e] = p.dfeed[hc];
        }
        if (!LOCAL && has_unit && uq == 0)
            for (int e = 0; e < 2; ++e)
                *reinterpret_cast<float4*>(sm.C5[0][kQuads][pl + e * L::ODD]) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        Raw xr[7], dr[4], gr[4], zr[4], xf[4];
        // input t of the unit's channels, from before the sequence too
        auto input = [&](int t) {
            if (t >= 0) return ldpair(x + (size_t)t * p.D + cp);
            return cs && t >= 1 - p.W ? ldpair(cs + (size_t)(p.W - 1 + t) * p.D + cp) : Pair<T>::zero();
        };
        auto fetch = [&](int k) {
            if (!has_unit || k >= chunks) return;
            const int t0 = tlast - k * kSsmChunk, tq = t0 + 4 * uq;
            const bool in = t0 >= 4 && t0 + kSsmChunk <= end;
            const T *dtt = dt + (size_t)t0 * p.D, *gyt = gy + (size_t)t0 * p.D, *zt = z + (size_t)t0 * p.D, *xt = x + (size_t)t0 * p.D;
            if (!LOCAL)
#pragma unroll
                for (int i = 0; i < 7; ++i) {
                    xr[i] = Pair<T>::zero();
                    if (i < 3 && p.W < 4 - i) continue;  // 3 - i tokens back: not in the filter
                    if (in) xr[i] = ldpair(xt + (i - 3) * p.D + off);
                    else if (tq - 3 + i < end) xr[i] = input(tq - 3 + i);
                }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool live = in || tq + j < end;
                dr[j] = live ? ldpair(dtt + j * p.D + off) : Pair<T>::zero();
                gr[j] = live ? ldpair(gyt + j * p.D + off) : Pair<T>::zero();
                zr[j] = z && live ? ldpair(zt + j * p.D + off) : Pair<T>::zero();
            }
        };
        auto fetch_x = [&](int k) {
            if (!has_unit) return;
            const int tq = tlast - k * kSsmChunk + 4 * uq;
#pragma unroll
            for (int j = 0; j < 4; ++j) xf[j] = tq + j < end ? ldpair(x + (size_t)(tq + j) * p.D + cp) : Pair<T>::zero();
        };
        auto copy_bc = [&](int k) {
            constexpr int PER = 16 / (int)sizeof(T), ROW = N / PER;  // values in 16 bytes, pieces of a token
            if (k < chunks) {
                const int t0 = tlast - k * kSsmChunk;
                for (int i = tid; i < kSsmChunk * ROW; i += EW) {
                    const bool there = t0 + i / ROW < end;
                    const size_t at = there ? (size_t)t0 * N + i * PER : 0;
                    if (!LOCAL) copy16(reinterpret_cast<char*>(&sm.B[k % 3][0][0]) + 16 * i, Bm + at, there);
                    copy16(reinterpret_cast<char*>(&sm.C[k % 3][0][0]) + 16 * i, Cm + at, there);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        using Two = float2[2][2];  // [channel][tokens 0 1, 2 3]
        auto unpack = [&](const Raw* r, Two& o) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 a = Pair<T>::f(r[j]);
                (&o[0][j >> 1].x)[j & 1] = a.x;
                (&o[1][j >> 1].x)[j & 1] = a.y;
            }
        };
        auto put = [&](float (&arr)[kQuads][L::PLACES][4], const Two& v) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
                *reinterpret_cast<float4*>(arr[uq][pl + e * L::ODD]) = make_float4(v[e][0].x, v[e][0].y, v[e][1].x, v[e][1].y);
        };
        auto get = [&](const float (&arr)[kQuads][L::PLACES][4], Two& v) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float4 a = *reinterpret_cast<const float4*>(arr[uq][pl + e * L::ODD]);
                v[e][0] = make_float2(a.x, a.y);
                v[e][1] = make_float2(a.z, a.w);
            }
        };
        auto stage = [&](int k) {
            if (!has_unit || k >= chunks) return;
            const int t0 = tlast - k * kSsmChunk, tq = t0 + 4 * uq, m = k & 1;
            Two d, g;
            unpack(dr, d);
            unpack(gr, g);
            if (p.preact) {
                Two sg;
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 a = add2(d[e][i], two(bias[e]));
                        d[e][i] = softplus2(a);
                        if (!LOCAL) sg[e][i] = sigmoid2(a);
                    }
                if (!LOCAL) put(sm.S[m], sg);
            }
            if (z) {
                Two zz;
                unpack(zr, zz);
                Two gz;
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 sg = sigmoid2(zz[e][i]);
                        if (!LOCAL) gz[e][i] = mul2(g[e][i], dsilu2(zz[e][i], sg));
                        g[e][i] = mul2(g[e][i], mul2(zz[e][i], sg));
                    }
                if (!LOCAL) put(sm.Z[m], gz);
            }
            Two u;
            if (!LOCAL) {
                if (p.W) {
                    float2 xv[7];
#pragma unroll
                    for (int i = 0; i < 7; ++i) xv[i] = Pair<T>::f(xr[i]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float z0 = cb[0], z1 = cb[1];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (i < p.W) {
                                z0 = fmaf(w[i][0], xv[3 + j - i].x, z0);
                                z1 = fmaf(w[i][1], xv[3 + j - i].y, z1);
                            }
                        (&u[0][j >> 1].x)[j & 1] = z0;
                        (&u[1][j >> 1].x)[j & 1] = z1;
                    }
                    if (p.silu) {
                        Two f;
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const float2 sg = sigmoid2(u[e][i]);
                                f[e][i] = dsilu2(u[e][i], sg);
                                u[e][i] = mul2(u[e][i], sg);
                            }
                        put(sm.F[m], f);
                    }
                } else {
                    unpack(xr + 3, u);
                }
            }
            if (t0 + kSsmChunk > end) {  // tokens behind the end: no step, no input, no gradient
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (tq + j >= end) {
                            (&d[e][j >> 1].x)[j & 1] = 0.0f;
                            (&g[e][j >> 1].x)[j & 1] = 0.0f;
                            if (!LOCAL) (&u[e][j >> 1].x)[j & 1] = 0.0f;
                        }
            }
            put(sm.D[m], d);
            put(sm.P[m], g);
            if (!LOCAL) put(sm.U[m], u);
        };
        // The gradients of dt and z, dzc of the convolution; then, once all of the
        // chunk's dzc are there, those of x and the taps.
        auto finish = [&](int k) {
            const int t0 = tlast - k * kSsmChunk, tq = t0 + 4 * uq, m = k & 1;
            const bool in = t0 + kSsmChunk <= end;
            Two zc;
            if (has_unit) {
                Two d, u, pp, q, e2, sg;
                get(sm.D[m], d);
                get(sm.U[m], u);
                get(sm.P[m], pp);
                get(sm.Q[m], q);
                get(sm.E[m], e2);
                float ps[3][2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float2 s1 = two(0.0f), s2 = two(0.0f);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        sg[e][i] = fma2(u[e][i], q[e][i], mul2(e2[e][i], two(kLn2)));
                        zc[e][i] = fma2(d[e][i], q[e][i], mul2(two(feed[e]), pp[e][i]));
                        s1 = fma2(pp[e][i], u[e][i], s1);
                    }
                    ps[1][e] = s1.x + s1.y;
                }
                if (p.preact) {
                    get(sm.S[m], e2);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int i = 0; i < 2; ++i) sg[e][i] = mul2(sg[e][i], e2[e][i]);
                }
                if (p.W && p.silu) {
                    get(sm.F[m], e2);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int i = 0; i < 2; ++i) zc[e][i] = mul2(zc[e][i], e2[e][i]);
                }
                if (!in)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (tq + j >= end) (&sg[e][j >> 1].x)[j & 1] = (&zc[e][j >> 1].x)[j & 1] = 0.0f;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 a = add2(sg[e][0], sg[e][1]), c = add2(zc[e][0], zc[e][1]);
                    ps[0][e] = a.x + a.y;
                    ps[2][e] = c.x + c.y;
                    *reinterpret_cast<float4*>(sm.C5[m][uq][pl + e * L::ODD]) = make_float4(zc[e][0].x, zc[e][0].y, zc[e][1].x, zc[e][1].y);
#pragma unroll
                    for (int i = 0; i < 3; ++i) par[i][e] += ps[i][e];
                }
                T* out = ddt + (size_t)t0 * p.D;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (in || tq + j < end) stpair(out + j * p.D + off, (&sg[0][j >> 1].x)[j & 1], (&sg[1][j >> 1].x)[j & 1]);
                if (z) {
                    Two y, gz;
                    get(sm.Y[m], y);
                    get(sm.Z[m], gz);
                    out = dz + (size_t)t0 * p.D;
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int i = 0; i < 2; ++i) y[e][i] = mul2(fma2(two(feed[e]), u[e][i], y[e][i]), gz[e][i]);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (in || tq + j < end) stpair(out + j * p.D + off, (&y[0][j >> 1].x)[j & 1], (&y[1][j >> 1].x)[j & 1]);
                }
            }
            part_sync<2, EW>();
            if (has_unit) {
                float2 xv[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) xv[j] = Pair<T>::f(xf[j]);
                float o[2][4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float4 n = *reinterpret_cast<const float4*>(sm.C5[m][uq + 1][pl + e * L::ODD]);
                    const float v[8] = {zc[e][0].x, zc[e][0].y, zc[e][1].x, zc[e][1].y, n.x, n.y, n.z, n.w};
                    float pw[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        o[e][j] = p.W ? 0.0f : v[j];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (i < p.W) {  // token j + i takes tap i of this one
                                o[e][j] = fmaf(w[i][e], v[j + i], o[e][j]);
                                pw[i] = fmaf(v[j + i], e ? xv[j].y : xv[j].x, pw[i]);
                            }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) par[3 + i][e] += pw[i];
                    if (uq == 0)  // for the chunk before
                        *reinterpret_cast<float4*>(sm.C5[m ^ 1][kQuads][pl + e * L::ODD]) = make_float4(v[0], v[1], v[2], v[3]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int t = tq + j;
                    if (t0 + kSsmChunk + 3 <= end) {  // no end near
                        stpair(dx + (size_t)t0 * p.D + j * p.D + off, o[0][j], o[1][j]);
                        continue;
                    }
                    if (t >= end) continue;
                    if (p.W > 1 && end < len && t >= end - 3) {  // the next segment's dzc are still to be added
                        float* ed = wk.edge + (((size_t)seg * p.B * p.H + bh) * 2 * 3 + (t - (end - 3))) * p.D + c0 + cp;
                        ed[0] = o[0][j];
                        ed[1] = o[1][j];
                        continue;
                    }
                    if (bp.gcs && t >= len - (p.W - 1)) {
                        const float2 g = Pair<T>::f(ldpair(static_cast<const T*>(bp.gcs) +
                            ((size_t)bh * (p.W - 1) + t - (len - (p.W - 1))) * p.D + c0 + cp));
                        o[0][j] += g.x;
                        o[1][j] += g.y;
                    }
                    stpair(dx + (size_t)t * p.D + cp, o[0][j], o[1][j]);
                }
            }
        };
        copy_bc(0);
        copy_bc(1);
        fetch(0);
        stage(0);
        fetch(1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
        for (int k = 0; k <= chunks; ++k) {  // one turn more than the scan warps: the last chunk's gradients
            if (!LOCAL && k > 0) finish(k - 1);
            if (k == chunks) break;
            copy_bc(k + 2);
            stage(k + 1);
            fetch(k + 2);
            if (!LOCAL) fetch_x(k);
            asm volatile("cp.async.wait_group 1;" ::: "memory");  // B and C of chunk k + 1 are there
            __syncthreads();
        }
        if (LOCAL) return;
        if (has_unit) {
            // the first chunk's dzc (zeros where there is none): what reaches back over the begin
            const int m = (chunks + 1) & 1;
            float first[2][3] = {};
            if (uq == 0 && chunks > 0)
                for (int e = 0; e < 2; ++e)
                    for (int j = 0; j < 3; ++j) first[e][j] = sm.C5[m][0][pl + e * L::ODD][j];
            if (uq == 0 && chunks > 0)
#pragma unroll
                for (int r = 1; r < 4; ++r) {  // input r tokens before the begin
                    if (r >= p.W) continue;
                    const float2 v = Pair<T>::f(input(begin - r));
#pragma unroll
                    for (int i = 1; i < 4; ++i)
                        if (i >= r && i < p.W) {
                            par[3 + i][0] = fmaf(first[0][i - r], v.x, par[3 + i][0]);
                            par[3 + i][1] = fmaf(first[1][i - r], v.y, par[3 + i][1]);
                        }
                }
#pragma unroll
            for (int i = 0; i < kPar; ++i)
                for (int e = 0; e < 2; ++e) sm.par[i][uq][cp + e] = par[i][e];
            if (seg > 0 && begin < len && uq == 0) {  // dzc of the first three tokens, for the end of the segment before
                float* ed = wk.edge + (((size_t)seg * p.B * p.H + bh) * 2 + 1) * 3 * p.D + c0 + cp;
                for (int j = 0; j < 3; ++j)
                    for (int e = 0; e < 2; ++e) ed[(size_t)j * p.D + e] = first[e][j];
            }
            if (seg == 0 && bp.dcs && uq == 0)
                for (int r = 0; r < p.W - 1; ++r) {  // input r - (W-1) before the sequence
                    float o[2] = {0.0f, 0.0f};
#pragma unroll
                    for (int j = 0; j < 3; ++j)
#pragma unroll
                        for (int i = 1; i < 4; ++i)
                            if (j <= r && i == p.W - 1 - r + j) {
                                o[0] = fmaf(w[i][0], first[0][j], o[0]);
                                o[1] = fmaf(w[i][1], first[1][j], o[1]);
                            }
                    if (bp.gcs && r - len >= 0) {  // a sequence so short that it is carried out again
                        const float2 g = Pair<T>::f(ldpair(static_cast<const T*>(bp.gcs) +
                            ((size_t)bh * (p.W - 1) + r - len) * p.D + c0 + cp));
                        o[0] += g.x;
                        o[1] += g.y;
                    }
                    stpair(static_cast<T*>(bp.dcs) + ((size_t)bh * (p.W - 1) + r) * p.D + c0 + cp, o[0], o[1]);
                }
            // rows behind the end have no gradient
            for (int t = max(begin, len) + uq; t < segend; t += kQuads) {
                stpair(dx + (size_t)t * p.D + cp, 0.0f, 0.0f);
                stpair(ddt + (size_t)t * p.D + cp, 0.0f, 0.0f);
                if (z) stpair(dz + (size_t)t * p.D + cp, 0.0f, 0.0f);
            }
        }
        part_sync<2, EW>();
        for (int i = tid; i < kPar * CPB; i += EW) {
            const int k = i / CPB, c = i % CPB;
            float a = 0.0f;
#pragma unroll
            for (int q = 0; q < kQuads; ++q) a += sm.par[k][q][c];
            wk.pPar[((size_t)(seg * p.B + b) * kPar + k) * p.H * p.D + h * p.D + c0 + c] = a;
        }
        return;
    }

    // -------------------------------------------- scan warps
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ch = tid / LPC, sl = tid % LPC, place = L::place(ch);
    const size_t srow = ((size_t)bh * p.D + c0 + ch) * N + 4 * sl;
    const size_t nc = (p.T + kSsmChunk - 1) / kSsmChunk;
    const size_t srow_saved = ((size_t)bh * nc * p.D + c0 + ch) * N + 4 * sl, sstep = (size_t)p.D * N;
    float2 A2[2], G[2] = {two(0.0f), two(0.0f)}, dA[2] = {two(0.0f), two(0.0f)};
    float dsum = 0.0f;
    {
        const float4 a = ld4(p.A + ((size_t)h * p.D + c0 + ch) * N + 4 * sl);
        A2[0] = make_float2(a.x * kLog2e, a.y * kLog2e);
        A2[1] = make_float2(a.z * kLog2e, a.w * kLog2e);
    }
    float4 next_state = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (!LOCAL) {
        if (chunks > 0) next_state = *reinterpret_cast<const float4*>(wk.saved + srow_saved + tlast / kSsmChunk * sstep);
        if (bp.gST) {
            const float4 v = ld4(bp.gST + srow);
            G[0] = make_float2(v.x, v.y);
            G[1] = make_float2(v.z, v.w);
        }
        for (int j = wk.P - 1; j > seg; --j) {  // the segments behind this one
            if (j * wk.len >= len) continue;
            const float4 v = *reinterpret_cast<const float4*>(wk.local + j * states * N + srow);
            const float2 ds = two(wk.dsum[j * states + (size_t)bh * p.D + c0 + ch]);
            G[0] = fma2(ex22(mul2(A2[0], ds)), G[0], make_float2(v.x, v.y));
            G[1] = fma2(ex22(mul2(A2[1], ds)), G[1], make_float2(v.z, v.w));
        }
    }
    __syncthreads();
    for (int k = 0; k < chunks; ++k) {
        const int t0 = tlast - k * kSsmChunk, m = k & 1, m3 = k % 3;
        if (LOCAL) {
#pragma unroll
            for (int q = kQuads - 1; q >= 0; --q) {
                const float4 d4 = *reinterpret_cast<const float4*>(sm.D[m][q][place]);
                const float4 p4 = *reinterpret_cast<const float4*>(sm.P[m][q][place]);
                const float dd[4] = {d4.x, d4.y, d4.z, d4.w}, pp[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
                for (int j = 3; j >= 0; --j) {
                    const Quad cq = sm.C[m3][4 * q + j][sl];
                    const float2 d2 = two(dd[j]), p2 = two(pp[j]);
                    G[0] = mul2(decay2(d2, A2[0]), fma2(Four<T>::lo(cq), p2, G[0]));
                    G[1] = mul2(decay2(d2, A2[1]), fma2(Four<T>::hi(cq), p2, G[1]));
                    dsum += dd[j];
                }
            }
            __syncthreads();
            continue;
        }
        // First the states before each four tokens (kept, 12 registers), then for each
        // four tokens, the last first, their states forward (16 registers) and back.
        // (With all sixteen states kept, and every decay evaluated twice, the code of
        // a chunk outgrew the instruction cache: 642 us against 586 a training step.)
        float2 before[kQuads][2];
        before[0][0] = make_float2(next_state.x, next_state.y);
        before[0][1] = make_float2(next_state.z, next_state.w);
        if (k + 1 < chunks)
            next_state = *reinterpret_cast<const float4*>(wk.saved + srow_saved + (t0 / kSsmChunk - 1) * sstep);
#pragma unroll
        for (int q = 0; q < kQuads - 1; ++q) {
            const float4 d4 = *reinterpret_cast<const float4*>(sm.D[m][q][place]);
            const float4 u4 = *reinterpret_cast<const float4*>(sm.U[m][q][place]);
            const float dd[4] = {d4.x, d4.y, d4.z, d4.w}, uu[4] = {u4.x, u4.y, u4.z, u4.w};
            float2 s[2] = {before[q][0], before[q][1]};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const Quad bq = sm.B[m3][4 * q + j][sl];
                const float2 d2 = two(dd[j]), du = two(dd[j] * uu[j]);
                s[0] = fma2(decay2(d2, A2[0]), s[0], mul2(du, Four<T>::lo(bq)));
                s[1] = fma2(decay2(d2, A2[1]), s[1], mul2(du, Four<T>::hi(bq)));
            }
            before[q + 1][0] = s[0];
            before[q + 1][1] = s[1];
        }
        float2 dAc[2] = {two(0.0f), two(0.0f)};  // this chunk's part: long sums in two steps
#pragma unroll 1
        for (int q = kQuads - 1; q >= 0; --q) {
            const float4 d4 = *reinterpret_cast<const float4*>(sm.D[m][q][place]);
            const float4 u4 = *reinterpret_cast<const float4*>(sm.U[m][q][place]);
            const float4 p4 = *reinterpret_cast<const float4*>(sm.P[m][q][place]);
            const float dd[4] = {d4.x, d4.y, d4.z, d4.w}, uu[4] = {u4.x, u4.y, u4.z, u4.w},
                        pp[4] = {p4.x, p4.y, p4.z, p4.w};
            float2 s[2] = {before[0][0], before[0][1]};
#pragma unroll
            for (int i = 1; i < kQuads; ++i)
                if (q == i) s[0] = before[i][0], s[1] = before[i][1];
            float2 hist[4][2], dec[4][2];
            const float2 s0[2] = {s[0], s[1]};
            float yy[4], qq[4], ee[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const Quad bq = sm.B[m3][4 * q + j][sl];
                const float2 d2 = two(dd[j]), du = two(dd[j] * uu[j]);
                dec[j][0] = decay2(d2, A2[0]);
                dec[j][1] = decay2(d2, A2[1]);
                s[0] = fma2(dec[j][0], s[0], mul2(du, Four<T>::lo(bq)));
                s[1] = fma2(dec[j][1], s[1], mul2(du, Four<T>::hi(bq)));
                hist[j][0] = s[0];
                hist[j][1] = s[1];
            }
#pragma unroll
            for (int j = 3; j >= 0; --j) {
                const Quad bq = sm.B[m3][4 * q + j][sl], cq = sm.C[m3][4 * q + j][sl];
                const float du1 = dd[j] * uu[j];
                const float2 d2 = two(dd[j]), p2 = two(pp[j]), du = two(du1);
                const float2 b2[2] = {Four<T>::lo(bq), Four<T>::hi(bq)}, c2[2] = {Four<T>::lo(cq), Four<T>::hi(cq)};
                float v[8];
                float2 qs, es, ys;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    ys = i ? fma2(hist[j][i], c2[i], ys) : mul2(hist[j][i], c2[i]);
                    G[i] = fma2(c2[i], p2, G[i]);
                    qs = i ? fma2(G[i], b2[i], qs) : mul2(G[i], b2[i]);
                    // (s_t - delta u B_t, the same by the recurrence, cancels where decays are strong)
                    const float2 back = mul2(G[i], dec[j][i]), ww = mul2(back, j ? hist[j - 1][i] : s0[i]);
                    es = i ? fma2(ww, A2[i], es) : mul2(ww, A2[i]);
                    dAc[i] = fma2(ww, d2, dAc[i]);
                    const float2 gb = mul2(G[i], du), gc = mul2(p2, hist[j][i]);
                    v[2 * i] = gb.x;
                    v[2 * i + 1] = gb.y;
                    v[4 + 2 * i] = gc.x;
                    v[5 + 2 * i] = gc.y;
                    G[i] = back;
                }
                yy[j] = ys.x + ys.y;
                qq[j] = qs.x + qs.y;
                ee[j] = es.x + es.y;
                // over the warp's channels: each step halves what a lane holds
                int first = 0, count = 8;
#pragma unroll
                for (int o = 16; o >= LPC && o >= 4; o >>= 1) {
                    if (count == 1) break;
                    const bool up = lane & o;
                    count >>= 1;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < count) {
                            const float send = up ? v[i] : v[count + i];
                            const float keep = up ? v[count + i] : v[i];
                            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                        }
                    first += up ? count : 0;
                }
                float* r = &sm.R[warp][(4 * q + j) % F][(first >> 2) * N + 4 * sl + (first & 3)];
                if (CW == 8) {
                    r[0] = v[0];
                } else if (CW == 4) {
                    *reinterpret_cast<float2*>(r) = make_float2(v[0], v[1]);
                } else {
                    *reinterpret_cast<float4*>(r) = make_float4(v[0], v[1], v[2], v[3]);
                    if (CW == 1) *reinterpret_cast<float4*>(r + N) = make_float4(v[4], v[5], v[6], v[7]);
                }
                if (F < 4 ? j % F == 0 : j == 0 && 4 * q % F == 0) {  // F tokens are in: the block's sums
                    part_sync<1, TH>();
                    const int tf = t0 + 4 * q + j;
                    float* out = wk.part + (((size_t)bh * wk.nblk + blk) * p.T + tf) * 2 * N;
                    for (int i = 4 * tid; i < F * 2 * N; i += 4 * TH) {
                        float4 a = *reinterpret_cast<const float4*>(&sm.R[0][0][0] + i);
#pragma unroll
                        for (int o = 1; o < WARPS; ++o) {
                            const float4 c = *reinterpret_cast<const float4*>(&sm.R[o][0][0] + i);
                            a.x += c.x; a.y += c.y; a.z += c.z; a.w += c.w;
                        }
                        if (tf + i / (2 * N) < end) *reinterpret_cast<float4*>(out + i) = a;
                    }
                    part_sync<1, TH>();
                }
            }
            const float rq = lane_sum4<LPC>(qq[0], qq[1], qq[2], qq[3]);
            const float re = lane_sum4<LPC>(ee[0], ee[1], ee[2], ee[3]);
            const float ry = lane_sum4<LPC>(yy[0], yy[1], yy[2], yy[3]);
            if (sl < 4) {
                sm.Q[m][q][place][sl] = rq;
                sm.E[m][q][place][sl] = re;
                sm.Y[m][q][place][sl] = ry;
            }
        }
        dA[0] = add2(dA[0], dAc[0]);
        dA[1] = add2(dA[1], dAc[1]);
        __syncthreads();
    }
    const float4 g4 = make_float4(G[0].x, G[0].y, G[1].x, G[1].y);
    if (LOCAL) {
        *reinterpret_cast<float4*>(wk.local + seg * states * N + srow) = g4;
        if (sl == 0) wk.dsum[seg * states + (size_t)bh * p.D + c0 + ch] = dsum;
        return;
    }
    // this segment's sums for A
    *reinterpret_cast<float4*>(wk.pA + ((size_t)(seg * p.B + b) * p.H * p.D + h * p.D + c0 + ch) * N + 4 * sl) =
        make_float4(dA[0].x, dA[0].y, dA[1].x, dA[1].y);
    if (seg == 0 && bp.dS0) *reinterpret_cast<float4*>(bp.dS0 + srow) = g4;
}

// The sums over blocks, sequences and segments, each in a fixed order, and the rows
// where the convolution reaches over a segment's end.  First dB and dC: one thread
// has four neighbouring values of a group's row (dB and dC side by side); then the
// weights' gradients and the edges, one value a thread.
template <typename T>
__global__ void __launch_bounds__(256) ssm_finish_kernel(const SsmBwdParams bp, const BwdWork wk, const unsigned rowblocks) {
    chain_wait();
    const SsmParams& p = bp.f;
    if (blockIdx.x < rowblocks) {
        const int per = p.N / 2;  // float4 of a row
        const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
        if (i >= (size_t)p.B * p.G * p.T * per) return;
        const int n = (int)(i % per) * 4;
        const size_t row = i / per;
        const int t = (int)(row % p.T), bg = (int)(row / p.T), b = bg / p.G, g = bg % p.G;
        const int hpg = p.H / p.G, rows = hpg * wk.nblk;
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (t < seq_len(p, b)) {
            const size_t step = (size_t)p.T * 2 * p.N;
            const float* part = wk.part + (((size_t)b * p.H + g * hpg) * wk.nblk * p.T + t) * 2 * p.N + n;
#pragma unroll 8
            for (int k = 0; k < rows; ++k) {
                const float4 v = *reinterpret_cast<const float4*>(part + k * step);
                a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
            }
        }
        T* out = static_cast<T*>(n < p.N ? bp.dB : bp.dC) + row * p.N + (n < p.N ? n : n - p.N);
        stpair(out, a.x, a.y);
        stpair(out + 2, a.z, a.w);
        return;
    }
    const size_t hd = (size_t)p.H * p.D, na = hd * p.N, np = hd * kPar;
    const size_t ne = wk.P > 1 && p.W > 1 ? (size_t)(wk.P - 1) * p.B * p.H * 3 * p.D : 0;
    size_t i = (size_t)(blockIdx.x - rowblocks) * 256 + threadIdx.x;
    const int parts = wk.P * p.B;
    if (i < na) {
        float a = 0.0f;
#pragma unroll 8
        for (int k = 0; k < parts; ++k) a += wk.pA[k * na + i];
        bp.dA[i] = a;
        return;
    }
    i -= na;
    if (i < np) {
        const int k = (int)(i / hd), hc = (int)(i % hd);
        float* out = k == 0 ? bp.ddt_bias : k == 1 ? bp.ddfeed : k == 2 ? bp.dcb : (k - 3 < p.W ? bp.dcw : nullptr);
        if (!out) return;
        float a = 0.0f;
#pragma unroll 8
        for (int j = 0; j < parts; ++j) a += wk.pPar[j * np + i];
        out[k < 3 ? hc : (size_t)hc * p.W + k - 3] = a;
        return;
    }
    i -= np;
    if (i < ne) {
        const int c = (int)(i % p.D), r = (int)(i / p.D % 3);
        const size_t sb = i / p.D / 3;  // segment, sequence and head
        const int seg = (int)(sb / (p.B * p.H)), bh = (int)(sb % (p.B * p.H)), b = bh / p.H, h = bh % p.H;
        const int len = seq_len(p, b), end = (seg + 1) * wk.len, t = end - 3 + r;
        if (end >= len) return;
        float o = wk.edge[(sb * 6 + r) * p.D + c];
        const float* next = wk.edge + ((sb + (size_t)p.B * p.H) * 6 + 3) * p.D + c;
        for (int j = 3 - r; j < p.W; ++j)  // tap j reaches token t + j, j - (3 - r) behind the segment's end
            o = fmaf(p.cw[((size_t)h * p.D + c) * p.W + j], next[(size_t)(j - (3 - r)) * p.D], o);
        if (bp.gcs && t >= len - (p.W - 1))
            o += ldf(static_cast<const T*>(bp.gcs) + ((size_t)bh * (p.W - 1) + t - (len - (p.W - 1))) * p.D + c);
        stf(static_cast<T*>(bp.dx) + ((size_t)bh * p.T + t) * p.D + c, o);
    }
}

int channels_per_block(int D, int N) {
    const int most = N == 16 ? 32 : N == 32 ? 16 : 8;
    return D < most ? D : most;
}

// Segments a sequence: the count of least cost, where a round is as many blocks as run at
// a time, a segment costs its tokens and a chunk to start and end, and the first launch for
// the states is a tenth of the work of all segments but one; each of at least two chunks,
// and whole sequences unless a cut saves 3% by this count.
// Measured, a training step with D64 N16 bf16 (us, whole sequences / this rule's P):
// B1 H24 T4096 857 / 321 (6), B2 H24 T4096 947 / 616 (3), B4 H24 T2048 653 / 554 (3),
// B1 H3 T4096 769 / 72 (49), B1 H4 T512 110 / 29 (16), B3 H20 T2048 499 / 383 (7); it
// keeps P = 1 at B16 H24 T512, 507 against 547 of P = 3, at B32 H24 T128, 266 against
// 330, and at B5 H24 T777, 273 against 298 of P = 6.  Four blocks an SM, B2 H24 T2048
// D16 N16: 386 / 104 (12; 153 with the 6 that two an SM would ask for).  One, N128 T2048:
// B2 H8 D64 791 (1) against 869 of P = 3, B1 H4 D16 561 / 75 (18).
int segments(const SsmParams& p) {
    const int cpb = channels_per_block(p.D, p.N);
    const long long blocks = (long long)p.B * p.H * (p.D / cpb), round = (long long)resident(cpb * p.N / 4) * sm_count();
    const int most = p.T / (2 * kSsmChunk) < 64 ? p.T / (2 * kSsmChunk) : 64;
    int best = 1;
    double whole = 0, least = 0;
    for (int P = 1; P == 1 || P <= most; ++P) {
        const long long rounds = (blocks * P + round - 1) / round;
        const double cost = rounds * ((double)p.T / P + kSsmChunk) * (1.0 + 0.1 * (P - 1) / P);
        if (P == 1) whole = cost;
        if (P == 1 || cost < least) {
            least = cost;
            best = P;
        }
    }
    return least < 0.97 * whole ? best : 1;
}

size_t up(size_t n) { return (n + 63) / 64 * 64; }  // floats, so that each part starts on 256 bytes

// Lays the scratch out; returns its bytes.
size_t layout(const SsmBwdParams& bp, BwdWork* wk) {
    const SsmParams& p = bp.f;
    wk->P = segments(p);
    const int chunks = (p.T + kSsmChunk - 1) / kSsmChunk;
    wk->len = (chunks + wk->P - 1) / wk->P * kSsmChunk;
    wk->nblk = p.D / channels_per_block(p.D, p.N);
    float* base = static_cast<float*>(p.ws);
    size_t at = 0;
    auto take = [&](float** q, size_t n) {
        *q = base ? base + at : nullptr;
        at += up(n);
    };
    const size_t states = (size_t)p.B * p.H * p.D;
    take(&wk->local, wk->P > 1 ? wk->P * states * p.N : 0);
    take(&wk->dsum, wk->P > 1 ? wk->P * states : 0);
    take(&wk->part, (size_t)p.B * p.H * wk->nblk * p.T * 2 * p.N);
    take(&wk->pA, (size_t)wk->P * states * p.N);
    take(&wk->pPar, (size_t)wk->P * states * kPar);
    take(&wk->edge, wk->P > 1 ? (size_t)wk->P * p.B * p.H * 6 * p.D : 0);
    if (p.saved) {
        wk->saved = p.saved;
    } else {
        take(&wk->saved, states * chunks * p.N);
        // the forward's own segments
        SsmParams f = p;
        f.y = nullptr;
        at += up((ssm_fwd_workspace(f) + 3) / 4);
    }
    return at * 4;
}

template <typename T, int N, int CPB, bool LOCAL>
cudaError_t launch_bwd_pass(const SsmBwdParams& bp, const BwdWork& wk, cudaStream_t s) {
    auto kern = ssm_bwd_kernel<T, N, CPB, LOCAL>;
    constexpr int smem = sizeof(BwdSmem<T, N, CPB, LOCAL>);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid((unsigned)((long long)bp.f.B * bp.f.H * wk.nblk), LOCAL ? wk.P - 1 : wk.P);
    if (!LOCAL && wk.P > 1) return launch_chained(kern, grid, CPB * N / 4 + kEw<CPB>, smem, s, bp, wk);
    kern<<<grid, CPB * N / 4 + kEw<CPB>, smem, s>>>(bp, wk);
    return cudaGetLastError();
}

template <typename T, int N, int CPB>
cudaError_t launch_bwd(const SsmBwdParams& bp, const BwdWork& wk, cudaStream_t s) {
    if (wk.P > 1) {
        const cudaError_t e = launch_bwd_pass<T, N, CPB, true>(bp, wk, s);
        if (e != cudaSuccess) return e;
    }
    return launch_bwd_pass<T, N, CPB, false>(bp, wk, s);
}

template <typename T>
cudaError_t launch_bwd_t(const SsmBwdParams& bp, const BwdWork& wk, cudaStream_t s) {
    const SsmParams& p = bp.f;
    cudaError_t e;
    switch (p.N) {
        case 16: e = p.D >= 32 ? launch_bwd<T, 16, 32>(bp, wk, s) : launch_bwd<T, 16, 16>(bp, wk, s); break;
        case 32: e = launch_bwd<T, 32, 16>(bp, wk, s); break;
        case 64: e = launch_bwd<T, 64, 8>(bp, wk, s); break;
        default: e = launch_bwd<T, 128, 8>(bp, wk, s); break;
    }
    if (e != cudaSuccess) return e;
    const unsigned rowblocks = (unsigned)(((size_t)p.B * p.G * p.T * (p.N / 2) + 255) / 256);
    const size_t hd = (size_t)p.H * p.D;
    const size_t n = hd * (p.N + kPar) + (wk.P > 1 && p.W > 1 ? (size_t)(wk.P - 1) * p.B * p.H * 3 * p.D : 0);
    return launch_chained(ssm_finish_kernel<T>, dim3(rowblocks + (unsigned)((n + 255) / 256)), 256, 0, s, bp, wk, rowblocks);
}

}  // namespace

size_t ssm_bwd_workspace(const SsmBwdParams& bp) {
    BwdWork wk;
    SsmBwdParams q = bp;
    q.f.ws = nullptr;
    return layout(q, &wk);
}

cudaError_t launch_ssm_bwd(const SsmBwdParams& bp, cudaStream_t s) {
    BwdWork wk;
    const size_t bytes = layout(bp, &wk);
    if (!bp.f.saved) {  // the states of the forward, into the scratch
        SsmParams f = bp.f;
        f.y = nullptr;
        f.ST = nullptr;
        f.cs_out = nullptr;
        f.saved = wk.saved;
        const size_t need = ssm_fwd_workspace(f);
        f.ws = static_cast<char*>(bp.f.ws) + bytes - up((need + 3) / 4) * 4;
        f.ws_bytes = need;
        const cudaError_t e = launch_ssm_fwd(f, s);
        if (e != cudaSuccess) return e;
    }
    return bp.f.bf16 ? launch_bwd_t<__nv_bfloat16>(bp, wk, s) : launch_bwd_t<float>(bp, wk, s);
}

}  // namespace rdm
