// ssm_bwd.cu -- reverse mode of the selective state space scan (ssm.cu).  With
// go the gradient of the output, p_t = go silu(z_t) the gradient of y before the
// gate and G_t the gradient of s_t with all that follows it:
//
//   G_t = C_t p_t + exp(delta_{t+1} A) G_{t+1}           (G_T takes grad_ST too)
//   dC_t = sum_c p s_t        dB_t = sum_c G_t delta u       dz = go y silu'(z)
//   q_t = sum_n G_t B_t       w_t = G_t (s_t - delta u B_t) = G_t exp(delta A) s_{t-1}
//   ddelta = u q + sum_n w A  dA = sum_t w delta             du = delta q + d p
//   dzc = du silu'(zc)        dx_t = sum_i w_i dzc_{t+i}     dw_i = sum_t dzc_t x_{t-i}
//
// A block has CPB channels of one (b, h), four states a thread, and walks its
// chunks of 16 tokens backwards.  From the state saved before a chunk it runs
// the recurrence forward again, keeping all 16 states of the chunk in registers
// (64 of them), then backwards; sums over n are shuffles within a channel's
// lanes for four tokens at a time, sums over channels (dB, dC) a transposing
// reduction over the warp's channels, then shared memory over the block's warps,
// then one row of partial sums per block that a last kernel adds up in a fixed
// order: no atomics, so the same call gives the same bits.  Sequences are cut
// into segments as in the forward; a first launch then runs G alone over each
// segment but the first from zero, and each block folds the segments behind its
// own.  The convolution's reach over a segment's end is added by the last kernel.
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

// A chunk's delta, u, p of the block's channels into shared memory, and the
// factors that the last stage needs; tokens at or behind `end` count as zeros.
template <typename T, int N, int CPB, bool LOCAL>
__global__ void __launch_bounds__(CPB * N / 4) ssm_bwd_kernel(const SsmBwdParams bp, const BwdWork wk) {
    using L = Lay<N, CPB>;
    constexpr int LPC = L::LPC, TH = L::THREADS, UNITS = kQuads * (CPB / 2), WARPS = TH / 32, F = Red<N>::F;
    constexpr int CW = 32 / LPC;  // channels a warp
    static_assert(UNITS <= TH, "one unit a thread");
    __shared__ __align__(16) float sD[kQuads][L::PLACES][4];
    __shared__ __align__(16) float sU[kQuads][L::PLACES][4];
    __shared__ __align__(16) float sP[kQuads][L::PLACES][4];
    __shared__ __align__(16) float sY[LOCAL ? 1 : kQuads][L::PLACES][4];
    __shared__ __align__(16) float sQ[LOCAL ? 1 : kQuads][L::PLACES][4];
    __shared__ __align__(16) float sE[LOCAL ? 1 : kQuads][L::PLACES][4];
    __shared__ __align__(16) float sF[LOCAL ? 1 : kQuads][L::PLACES][4];      // silu'(zc)
    __shared__ __align__(16) float sS[LOCAL ? 1 : kQuads][L::PLACES][4];      // d delta / d dt
    __shared__ __align__(16) float sZ[LOCAL ? 1 : kQuads + 1][L::PLACES][4];  // dzc, and the next chunk's first four
    __shared__ __align__(16) float sB[LOCAL ? 1 : kSsmChunk][N];
    __shared__ __align__(16) float sC[kSsmChunk][N];
    __shared__ __align__(16) float sR[LOCAL ? 1 : WARPS][LOCAL ? 1 : F][2 * N];
    const SsmParams& p = bp.f;
    const int bh = blockIdx.x / wk.nblk, blk = blockIdx.x % wk.nblk, c0 = blk * CPB;
    const int b = bh / p.H, h = bh % p.H, seg = blockIdx.y + (LOCAL ? 1 : 0);
    const int len = seq_len(p, b);
    const int begin = seg * wk.len, segend = min(begin + wk.len, p.T);
    const int end = min(segend, len);
    const int tid = threadIdx.x;
    if (LOCAL && begin >= len) return;
    const size_t row0 = (size_t)bh * p.T;
    const T* x = static_cast<const T*>(p.x) + row0 * p.D + c0;
    const T* dt = static_cast<const T*>(p.dt) + row0 * p.D + c0;
    const T* z = p.z ? static_cast<const T*>(p.z) + row0 * p.D + c0 : nullptr;
    const T* gy = static_cast<const T*>(bp.gy) + row0 * p.D + c0;
    const size_t grow = (size_t)(b * p.G + h / (p.H / p.G)) * p.T;
    const T* Bm = static_cast<const T*>(p.Bm) + grow * N;
    const T* Cm = static_cast<const T*>(p.Cm) + grow * N;
    const T* cs = p.cs_in ? static_cast<const T*>(p.cs_in) + (size_t)bh * (p.W - 1) * p.D + c0 : nullptr;
    const size_t states = (size_t)p.B * p.H * p.D;

    const int ch = tid / LPC, sl = tid % LPC, place = L::place(ch);
    const size_t srow = ((size_t)bh * p.D + c0 + ch) * N + 4 * sl;
    float A2[4], G[4] = {0.0f, 0.0f, 0.0f, 0.0f}, dA[4] = {0.0f, 0.0f, 0.0f, 0.0f}, dsum = 0.0f;
    {
        const float4 a = ld4(p.A + ((size_t)h * p.D + c0 + ch) * N + 4 * sl);
        A2[0] = a.x * kLog2e; A2[1] = a.y * kLog2e; A2[2] = a.z * kLog2e; A2[3] = a.w * kLog2e;
    }
    if (!LOCAL) {
        if (bp.gST) {
            const float4 v = ld4(bp.gST + srow);
            G[0] = v.x; G[1] = v.y; G[2] = v.z; G[3] = v.w;
        }
        for (int j = wk.P - 1; j > seg; --j) {  // the segments behind this one
            if (j * wk.len >= len) continue;
            const float4 v = *reinterpret_cast<const float4*>(wk.local + j * states * N + srow);
            const float ds = wk.dsum[j * states + (size_t)bh * p.D + c0 + ch];
            G[0] = fmaf(ex2_fast(A2[0] * ds), G[0], v.x);
            G[1] = fmaf(ex2_fast(A2[1] * ds), G[1], v.y);
            G[2] = fmaf(ex2_fast(A2[2] * ds), G[2], v.z);
            G[3] = fmaf(ex2_fast(A2[3] * ds), G[3], v.w);
        }
    }
    // the element-wise stages: channels cp, cp + 1 of tokens 4 uq .. 4 uq + 3 of the chunk
    const bool has_unit = tid < UNITS;
    const int uq = tid / (CPB / 2), cp = 2 * (tid % (CPB / 2)), pl = cp >> 1;
    float w[4][2] = {}, cb[2] = {0.0f, 0.0f}, bias[2] = {0.0f, 0.0f}, feed[2] = {0.0f, 0.0f};
    float par[kPar][2] = {};
    if (has_unit) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int hc = h * p.D + c0 + cp + e;
            for (int i = 0; i < p.W; ++i) w[i][e] = p.cw[(size_t)hc * p.W + i];
            if (p.cb) cb[e] = p.cb[hc];
            if (p.dt_bias) bias[e] = p.dt_bias[hc];
            if (p.dfeed) feed[e] = p.dfeed[hc];
        }
        if (!LOCAL && uq == 0)
            for (int e = 0; e < 2; ++e)
                *reinterpret_cast<float4*>(sZ[kQuads][pl + e * L::ODD]) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    // inputs tq - 3 .. tq + 3 of the unit's channels
    auto window = [&](int tq, float2* xv) {
#pragma unroll
        for (int i = 0; i < 7; ++i) {
            const int t = tq - 3 + i;
            xv[i] = make_float2(0.0f, 0.0f);
            if (i < 3 && p.W < 4 - i) continue;
            if (t >= 0) {
                if (t < end) xv[i] = Pair<T>::f(ldpair(x + (size_t)t * p.D + cp));
            } else if (cs && t >= 1 - p.W) {
                xv[i] = Pair<T>::f(ldpair(cs + (size_t)(p.W - 1 + t) * p.D + cp));
            }
        }
    };

    if (end > begin)
    for (int t0 = begin + (end - begin - 1) / kSsmChunk * kSsmChunk; t0 >= begin; t0 -= kSsmChunk) {
        if (has_unit) {
            const int tq = t0 + 4 * uq;
            float2 xv[7];
            if (!LOCAL) window(tq, xv);
            float dv[2][4], uv[2][4], pv[2][4], fv[2][4], sv[2][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool live = tq + j < end;
                const size_t at = (size_t)(tq + j) * p.D + cp;
                float2 d = make_float2(0.0f, 0.0f), g = d;
                if (live) {
                    d = Pair<T>::f(ldpair(dt + at));
                    g = Pair<T>::f(ldpair(gy + at));
                    if (z) {
                        const float2 zz = Pair<T>::f(ldpair(z + at));
                        g.x *= silu(zz.x);
                        g.y *= silu(zz.y);
                    }
                }
                float2 f = make_float2(1.0f, 1.0f), u = make_float2(0.0f, 0.0f), sg = f;
                if (!LOCAL) {
                    u = xv[3 + j];
                    if (p.W) {
                        float2 zc = make_float2(cb[0], cb[1]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (i < p.W) {
                                zc.x = fmaf(w[i][0], xv[3 + j - i].x, zc.x);
                                zc.y = fmaf(w[i][1], xv[3 + j - i].y, zc.y);
                            }
                        u = zc;
                        if (p.silu) {
                            const float s0 = sigmoid(zc.x), s1 = sigmoid(zc.y);
                            u = make_float2(zc.x * s0, zc.y * s1);
                            f = make_float2(dsilu(zc.x, s0), dsilu(zc.y, s1));
                        }
                    }
                }
                if (p.preact) {
                    d.x += bias[0];
                    d.y += bias[1];
                    if (!LOCAL) sg = make_float2(sigmoid(d.x), sigmoid(d.y));
                    d = make_float2(softplus(d.x), softplus(d.y));
                }
                dv[0][j] = live ? d.x : 0.0f; dv[1][j] = live ? d.y : 0.0f;
                pv[0][j] = g.x; pv[1][j] = g.y;
                uv[0][j] = live ? u.x : 0.0f; uv[1][j] = live ? u.y : 0.0f;
                fv[0][j] = f.x; fv[1][j] = f.y;
                sv[0][j] = sg.x; sv[1][j] = sg.y;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int k = pl + e * L::ODD;
                *reinterpret_cast<float4*>(sD[uq][k]) = make_float4(dv[e][0], dv[e][1], dv[e][2], dv[e][3]);
                *reinterpret_cast<float4*>(sP[uq][k]) = make_float4(pv[e][0], pv[e][1], pv[e][2], pv[e][3]);
                if (!LOCAL) {
                    *reinterpret_cast<float4*>(sU[uq][k]) = make_float4(uv[e][0], uv[e][1], uv[e][2], uv[e][3]);
                    *reinterpret_cast<float4*>(sF[uq][k]) = make_float4(fv[e][0], fv[e][1], fv[e][2], fv[e][3]);
                    *reinterpret_cast<float4*>(sS[uq][k]) = make_float4(sv[e][0], sv[e][1], sv[e][2], sv[e][3]);
                }
            }
        }
        for (int i = tid; i < kSsmChunk * N / 4; i += TH) {
            const int t = t0 + i / (N / 4), n = 4 * (i % (N / 4));
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f), u = v;
            if (t < end) {
                u = ld4(Cm + (size_t)t * N + n);
                if (!LOCAL) v = ld4(Bm + (size_t)t * N + n);
            }
            *reinterpret_cast<float4*>(&sC[t - t0][n]) = u;
            if (!LOCAL) *reinterpret_cast<float4*>(&sB[t - t0][n]) = v;
        }
        __syncthreads();
        if (LOCAL) {
#pragma unroll
            for (int q = kQuads - 1; q >= 0; --q) {
                const float4 d4 = *reinterpret_cast<const float4*>(sD[q][place]);
                const float4 p4 = *reinterpret_cast<const float4*>(sP[q][place]);
                const float dd[4] = {d4.x, d4.y, d4.z, d4.w}, pp[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
                for (int j = 3; j >= 0; --j) {
                    const float4 cc = *reinterpret_cast<const float4*>(&sC[4 * q + j][4 * sl]);
                    G[0] = ex2_fast(dd[j] * A2[0]) * fmaf(cc.x, pp[j], G[0]);
                    G[1] = ex2_fast(dd[j] * A2[1]) * fmaf(cc.y, pp[j], G[1]);
                    G[2] = ex2_fast(dd[j] * A2[2]) * fmaf(cc.z, pp[j], G[2]);
                    G[3] = ex2_fast(dd[j] * A2[3]) * fmaf(cc.w, pp[j], G[3]);
                    dsum += dd[j];
                }
            }
            __syncthreads();
            continue;
        }
        // forward over the chunk from its saved state
        float hist[kSsmChunk][4];
        {
            const size_t nc = (p.T + kSsmChunk - 1) / kSsmChunk;
            const size_t at = (((size_t)bh * nc + t0 / kSsmChunk) * p.D + c0 + ch) * N + 4 * sl;
            const float4 v = *reinterpret_cast<const float4*>(wk.saved + at);
            float s[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int q = 0; q < kQuads; ++q) {
                const float4 d4 = *reinterpret_cast<const float4*>(sD[q][place]);
                const float4 u4 = *reinterpret_cast<const float4*>(sU[q][place]);
                const float dd[4] = {d4.x, d4.y, d4.z, d4.w}, uu[4] = {u4.x, u4.y, u4.z, u4.w};
                float yy[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int t = 4 * q + j;
                    const float4 bb = *reinterpret_cast<const float4*>(&sB[t][4 * sl]);
                    const float4 cc = *reinterpret_cast<const float4*>(&sC[t][4 * sl]);
                    const float du = dd[j] * uu[j];
                    s[0] = fmaf(ex2_fast(dd[j] * A2[0]), s[0], du * bb.x);
                    s[1] = fmaf(ex2_fast(dd[j] * A2[1]), s[1], du * bb.y);
                    s[2] = fmaf(ex2_fast(dd[j] * A2[2]), s[2], du * bb.z);
                    s[3] = fmaf(ex2_fast(dd[j] * A2[3]), s[3], du * bb.w);
                    yy[j] = fmaf(s[0], cc.x, fmaf(s[1], cc.y, fmaf(s[2], cc.z, s[3] * cc.w)));
#pragma unroll
                    for (int i = 0; i < 4; ++i) hist[t][i] = s[i];
                }
                if (z) {
                    const float r = lane_sum4<LPC>(yy[0], yy[1], yy[2], yy[3]);
                    if (sl < 4) sY[q][place][sl] = r;
                }
            }
        }
        // and backwards
        float dAc[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // this chunk's part: long sums in two steps
#pragma unroll
        for (int q = kQuads - 1; q >= 0; --q) {
            const float4 d4 = *reinterpret_cast<const float4*>(sD[q][place]);
            const float4 u4 = *reinterpret_cast<const float4*>(sU[q][place]);
            const float4 p4 = *reinterpret_cast<const float4*>(sP[q][place]);
            const float dd[4] = {d4.x, d4.y, d4.z, d4.w}, uu[4] = {u4.x, u4.y, u4.z, u4.w},
                        pp[4] = {p4.x, p4.y, p4.z, p4.w};
            float qq[4], ee[4];
#pragma unroll
            for (int j = 3; j >= 0; --j) {
                const int t = 4 * q + j;
                const float4 b4 = *reinterpret_cast<const float4*>(&sB[t][4 * sl]);
                const float4 c4 = *reinterpret_cast<const float4*>(&sC[t][4 * sl]);
                const float bb[4] = {b4.x, b4.y, b4.z, b4.w}, cc[4] = {c4.x, c4.y, c4.z, c4.w};
                const float du = dd[j] * uu[j];
                float v[8];
                float qs = 0.0f, es = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    G[i] = fmaf(cc[i], pp[j], G[i]);
                    qs = fmaf(G[i], bb[i], qs);
                    const float ww = G[i] * fmaf(-du, bb[i], hist[t][i]);
                    es = fmaf(ww, A2[i], es);
                    dAc[i] = fmaf(ww, dd[j], dAc[i]);
                    v[i] = G[i] * du;
                    v[4 + i] = pp[j] * hist[t][i];
                    G[i] *= ex2_fast(dd[j] * A2[i]);
                }
                qq[j] = qs;
                ee[j] = es;
                // over the warp's channels: each step halves what a lane holds
                const int lane = tid & 31, wrp = tid >> 5;
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
                float* r = &sR[wrp][t % F][(first >> 2) * N + 4 * sl + (first & 3)];
                if (CW == 8) {
                    r[0] = v[0];
                } else if (CW == 4) {
                    *reinterpret_cast<float2*>(r) = make_float2(v[0], v[1]);
                } else {
                    *reinterpret_cast<float4*>(r) = make_float4(v[0], v[1], v[2], v[3]);
                    if (CW == 1) *reinterpret_cast<float4*>(r + N) = make_float4(v[4], v[5], v[6], v[7]);
                }
                if (t % F == 0) {  // F tokens are in: the block's sums
                    __syncthreads();
                    float* out = wk.part + (((size_t)bh * wk.nblk + blk) * p.T + t0 + t) * 2 * N;
                    for (int i = tid; i < F * 2 * N; i += TH) {
                        float a = 0.0f;
#pragma unroll
                        for (int k = 0; k < WARPS; ++k) a += (&sR[k][0][0])[i];
                        if (t0 + t + i / (2 * N) < end) out[i] = a;
                    }
                    __syncthreads();
                }
            }
            const float rq = lane_sum4<LPC>(qq[0], qq[1], qq[2], qq[3]);
            const float re = lane_sum4<LPC>(ee[0], ee[1], ee[2], ee[3]);
            if (sl < 4) {
                sQ[q][place][sl] = rq;
                sE[q][place][sl] = re;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) dA[i] += dAc[i];
        __syncthreads();
        // element-wise: the gradients of dt and z, dzc of the convolution
        if (has_unit) {
            const int tq = t0 + 4 * uq;
            float ps[3][2] = {};
            float zc[2][4], ddt[2][4], dz[2][4] = {};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int k = pl + e * L::ODD;
                const float4 D = *reinterpret_cast<const float4*>(sD[uq][k]);
                const float4 U = *reinterpret_cast<const float4*>(sU[uq][k]);
                const float4 Pq = *reinterpret_cast<const float4*>(sP[uq][k]);
                const float4 Q = *reinterpret_cast<const float4*>(sQ[uq][k]);
                const float4 E = *reinterpret_cast<const float4*>(sE[uq][k]);
                const float4 Fz = *reinterpret_cast<const float4*>(sF[uq][k]);
                const float4 S = *reinterpret_cast<const float4*>(sS[uq][k]);
                const float d[4] = {D.x, D.y, D.z, D.w}, u[4] = {U.x, U.y, U.z, U.w}, pq[4] = {Pq.x, Pq.y, Pq.z, Pq.w},
                            qv[4] = {Q.x, Q.y, Q.z, Q.w}, ev[4] = {E.x, E.y, E.z, E.w}, f[4] = {Fz.x, Fz.y, Fz.z, Fz.w},
                            sg[4] = {S.x, S.y, S.z, S.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool live = tq + j < end;
                    ddt[e][j] = live ? fmaf(u[j], qv[j], ev[j] * kLn2) * sg[j] : 0.0f;
                    zc[e][j] = live ? fmaf(d[j], qv[j], feed[e] * pq[j]) * f[j] : 0.0f;
                    ps[0][e] += ddt[e][j];
                    ps[1][e] = fmaf(pq[j], u[j], ps[1][e]);
                    ps[2][e] += zc[e][j];
                }
                *reinterpret_cast<float4*>(sZ[uq][k]) = make_float4(zc[e][0], zc[e][1], zc[e][2], zc[e][3]);
                if (z) {
                    const float4 Yq = *reinterpret_cast<const float4*>(sY[uq][k]);
                    dz[e][0] = fmaf(feed[e], u[0], Yq.x); dz[e][1] = fmaf(feed[e], u[1], Yq.y);
                    dz[e][2] = fmaf(feed[e], u[2], Yq.z); dz[e][3] = fmaf(feed[e], u[3], Yq.w);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (tq + j >= end) continue;
                const size_t at = (size_t)(tq + j) * p.D + cp;
                stpair(static_cast<T*>(bp.ddt) + row0 * p.D + c0 + at, ddt[0][j], ddt[1][j]);
                if (z) {
                    const float2 zz = Pair<T>::f(ldpair(z + at)), g = Pair<T>::f(ldpair(gy + at));
                    stpair(static_cast<T*>(bp.dz) + row0 * p.D + c0 + at, g.x * dz[0][j] * dsilu(zz.x, sigmoid(zz.x)),
                           g.y * dz[1][j] * dsilu(zz.y, sigmoid(zz.y)));
                }
            }
#pragma unroll
            for (int i = 0; i < 3; ++i)
                for (int e = 0; e < 2; ++e) par[i][e] += ps[i][e];
        }
        __syncthreads();
        if (has_unit) {  // through the convolution
            const int tq = t0 + 4 * uq;
            float2 xv[7];
            window(tq, xv);
            float o[2][4], pw[4][2] = {};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int k = pl + e * L::ODD;
                const float4 a = *reinterpret_cast<const float4*>(sZ[uq][k]);
                const float4 n = *reinterpret_cast<const float4*>(sZ[uq + 1][k]);
                const float v[8] = {a.x, a.y, a.z, a.w, n.x, n.y, n.z, n.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    o[e][j] = p.W ? 0.0f : v[j];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < p.W) {
                            o[e][j] = fmaf(w[i][e], v[j + i], o[e][j]);
                            pw[i][e] = fmaf(v[j], e ? xv[3 + j - i].y : xv[3 + j - i].x, pw[i][e]);
                        }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                for (int e = 0; e < 2; ++e) par[3 + i][e] += pw[i][e];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = tq + j;
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
                stpair(static_cast<T*>(bp.dx) + (row0 + t) * p.D + c0 + cp, o[0][j], o[1][j]);
            }
        }
        __syncthreads();
        if (has_unit && uq == 0)
            for (int e = 0; e < 2; ++e) {
                const int k = pl + e * L::ODD;
                *reinterpret_cast<float4*>(sZ[kQuads][k]) = *reinterpret_cast<const float4*>(sZ[0][k]);
            }
        // sZ's last quad is read again only behind the next chunk's barriers
    }
    if (LOCAL) {
        *reinterpret_cast<float4*>(wk.local + seg * states * N + srow) = make_float4(G[0], G[1], G[2], G[3]);
        if (sl == 0) wk.dsum[seg * states + (size_t)bh * p.D + c0 + ch] = dsum;
        return;
    }
    // this segment's sums for the weights
    *reinterpret_cast<float4*>(wk.pA + ((size_t)(seg * p.B + b) * p.H * p.D + h * p.D + c0 + ch) * N + 4 * sl) =
        make_float4(dA[0], dA[1], dA[2], dA[3]);
    __syncthreads();
    float* scratch = &sR[0][0][0];  // [kPar][kQuads][CPB]
    static_assert(kPar * kQuads * CPB <= WARPS * F * 2 * N, "per-channel sums fit the reduction buffer");
    if (has_unit)
#pragma unroll
        for (int i = 0; i < kPar; ++i)
            for (int e = 0; e < 2; ++e) scratch[(i * kQuads + uq) * CPB + cp + e] = par[i][e];
    __syncthreads();
    for (int i = tid; i < kPar * CPB; i += TH) {
        const int k = i / CPB, c = i % CPB;
        float a = 0.0f;
#pragma unroll
        for (int q = 0; q < kQuads; ++q) a += scratch[(k * kQuads + q) * CPB + c];
        wk.pPar[((size_t)(seg * p.B + b) * kPar + k) * p.H * p.D + h * p.D + c0 + c] = a;
    }
    // dzc of the segment's first three tokens, for the end of the one before
    if (seg > 0 && begin < len && has_unit && uq == 0) {
        float* ed = wk.edge + (((size_t)seg * p.B * p.H + bh) * 2 + 1) * 3 * p.D + c0 + cp;
        for (int j = 0; j < 3; ++j)
            for (int e = 0; e < 2; ++e) ed[(size_t)j * p.D + e] = sZ[0][pl + e * L::ODD][j];
    }
    if (seg == 0) {
        if (bp.dS0) *reinterpret_cast<float4*>(bp.dS0 + srow) = make_float4(G[0], G[1], G[2], G[3]);
        if (bp.dcs && has_unit && uq == 0)
            for (int r = 0; r < p.W - 1; ++r) {  // input r - (W-1) before the sequence
                float o[2];
                for (int e = 0; e < 2; ++e) {
                    o[e] = 0.0f;
                    if (len > 0)
                        for (int j = 0; j <= r; ++j) o[e] = fmaf(w[p.W - 1 - r + j][e], sZ[0][pl + e * L::ODD][j], o[e]);
                }
                if (bp.gcs && r - len >= 0) {  // a sequence so short that it is carried out again
                    const float2 g = Pair<T>::f(ldpair(static_cast<const T*>(bp.gcs) +
                        ((size_t)bh * (p.W - 1) + r - len) * p.D + c0 + cp));
                    o[0] += g.x;
                    o[1] += g.y;
                }
                stpair(static_cast<T*>(bp.dcs) + ((size_t)bh * (p.W - 1) + r) * p.D + c0 + cp, o[0], o[1]);
            }
    }
    // rows behind the end have no gradient
    for (int t = max(begin, len) + tid / (CPB / 2); t < segend; t += TH / (CPB / 2)) {
        const size_t at = (row0 + t) * p.D + c0 + cp;
        stpair(static_cast<T*>(bp.dx) + at, 0.0f, 0.0f);
        stpair(static_cast<T*>(bp.ddt) + at, 0.0f, 0.0f);
        if (z) stpair(static_cast<T*>(bp.dz) + at, 0.0f, 0.0f);
    }
}

// dB, dC: each group's rows of partial sums, in order.  One thread has four
// neighbouring values of a row (dB and dC side by side).
template <typename T>
__global__ void __launch_bounds__(256) ssm_bc_grad_kernel(const SsmBwdParams bp, const BwdWork wk) {
    const SsmParams& p = bp.f;
    const int per = p.N / 2;  // float4 of a row
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (size_t)p.B * p.G * p.T * per) return;
    const int n = (int)(i % per) * 4;
    const size_t row = i / per;
    const int t = (int)(row % p.T), bg = (int)(row / p.T), b = bg / p.G, g = bg % p.G;
    const int hpg = p.H / p.G, rows = hpg * wk.nblk;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (t < seq_len(p, b)) {
        const float* part = wk.part + (((size_t)b * p.H + g * hpg) * wk.nblk * p.T + t) * 2 * p.N + n;
        for (int k = 0; k < rows; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(part + (size_t)k * p.T * 2 * p.N);
            a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
        }
    }
    T* out = static_cast<T*>(n < p.N ? bp.dB : bp.dC) + row * p.N + (n < p.N ? n : n - p.N);
    stpair(out, a.x, a.y);
    stpair(out + 2, a.z, a.w);
}

// The weights' gradients over sequences and segments, in order, and the rows
// where the convolution reaches over a segment's end.
template <typename T>
__global__ void __launch_bounds__(256) ssm_finish_kernel(const SsmBwdParams bp, const BwdWork wk) {
    const SsmParams& p = bp.f;
    const size_t hd = (size_t)p.H * p.D, na = hd * p.N, np = hd * kPar;
    const size_t ne = wk.P > 1 && p.W > 1 ? (size_t)(wk.P - 1) * p.B * p.H * 3 * p.D : 0;
    size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    const int parts = wk.P * p.B;
    if (i < na) {
        float a = 0.0f;
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

int segments(const SsmParams& p) {
    const long long blocks = (long long)p.B * p.H * (p.D / channels_per_block(p.D, p.N));
    const long long want = 4LL * sm_count();
    if (blocks * 2 > want) return 1;
    long long P = want / blocks;
    const long long most = p.T / (8 * kSsmChunk);
    if (P > most) P = most;
    if (P > 64) P = 64;
    return P < 2 ? 1 : (int)P;
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

template <typename T, int N, int CPB>
cudaError_t launch_bwd(const SsmBwdParams& bp, const BwdWork& wk, cudaStream_t s) {
    const unsigned blocks = (unsigned)((long long)bp.f.B * bp.f.H * wk.nblk);
    if (wk.P > 1) {
        ssm_bwd_kernel<T, N, CPB, true><<<dim3(blocks, wk.P - 1), CPB * N / 4, 0, s>>>(bp, wk);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    ssm_bwd_kernel<T, N, CPB, false><<<dim3(blocks, wk.P), CPB * N / 4, 0, s>>>(bp, wk);
    return cudaGetLastError();
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
    const size_t rows = (size_t)p.B * p.G * p.T * (p.N / 2);
    if (rows) {
        ssm_bc_grad_kernel<T><<<(unsigned)((rows + 255) / 256), 256, 0, s>>>(bp, wk);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    const size_t hd = (size_t)p.H * p.D;
    const size_t n = hd * (p.N + kPar) + (wk.P > 1 && p.W > 1 ? (size_t)(wk.P - 1) * p.B * p.H * 3 * p.D : 0);
    ssm_finish_kernel<T><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(bp, wk);
    return cudaGetLastError();
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
