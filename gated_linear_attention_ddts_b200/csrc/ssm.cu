// ssm.cu -- selective state space scan (Gu and Dao, "Mamba: Linear-Time Sequence
// Modeling with Selective State Spaces", arXiv 2312.00752, Section 3) with its
// short causal convolution, for prompts and for single tokens.  Per channel
// (h, c), state n, token t, the head's group g:
//
//   u_t = silu(bias + sum_{i<W} w_i x_{t-i})   (x_t itself without a convolution)
//   delta_t = softplus(dt_t + dt_bias)
//   s_t[n] = exp(delta_t A[n]) s_{t-1}[n] + delta_t u_t B_t[n]
//   y_t = (sum_n C_t[n] s_t[n] + d u_t) silu(z_t)
//
// The decays differ by channel and state, so there is no matrix product in it:
// the recurrence runs on the CUDA cores in float32, and its floor is the
// exponential unit (one ex2 per channel, token and state; 16 a clock and SM): 61 us
// for B8 H24 D64 N16 of ragged T up to 2048 (11608 tokens), 84 with the six of delta,
// u and the gate; it takes 164, HBM would take 22.
//
// Forward: a block has CPB channels of one (b, h), four states a thread, and
// walks its tokens in tiles of 32.  Threads first make delta and u of the tile
// (two channels by four tokens a thread) in shared memory, then run the
// recurrence, sums over n by shuffles for four tokens at a time, then finish y
// with the skip and the gate in the same layout as the loads.  Where the
// channels alone do not fill the card, each sequence is cut into P segments: a
// first launch runs every segment but the last from a zero state and leaves its
// end state and its sum of delta; in the second each block folds the segments
// before its own, s <- local + exp(A sum delta) s, and runs for good.
#include <type_traits>

#include "launch.h"
#include "ssm_common.cuh"

namespace rdm {
namespace {

using namespace ssm;

constexpr int kTile = 32;

// Segments of a scan: `len` tokens each (a multiple of kTile); local[seg][b][h][D][N]
// and dsum[seg][b][h][D] from the first launch.
struct SegArgs {
    int P, len;
    float *local, *dsum;
};

// Threads of the element-wise warps: one for each two channels by four tokens of
// a tile.
template <int CPB>
constexpr int kEw = (kTile / 4) * (CPB / 2) < 32 ? 32 : (kTile / 4) * (CPB / 2);

// B and C are staged in their own type: four bf16 states are one 8-byte read a
// lane, half of the shared-memory wavefronts of float32 (which bounded the loop
// before the exponentials did).
template <typename T, int N, int CPB, bool LOCAL>
struct FwdSmem {
    float D[2][kTile / 4][Lay<N, CPB>::PLACES][4];
    float U[2][kTile / 4][Lay<N, CPB>::PLACES][4];
    float Y[LOCAL ? 1 : 2][LOCAL ? 1 : kTile / 4][Lay<N, CPB>::PLACES][4];
    typename Four<T>::Raw B[3][kTile][N / 4];
    typename Four<T>::Raw C[LOCAL ? 1 : 3][LOCAL ? 1 : kTile][N / 4];
};

// Two kinds of warps, a tile apart, one block barrier a tile: while the scan warps
// run the recurrence over tile k, the element-wise warps finish y of tile k - 1
// and make delta and u of tile k + 1, whose inputs they fetched a tile ago.  With
// one kind doing all three in turn only 58% of the issue slots were used (2.6
// warps a scheduler at B8 H24 D64, each waiting for itself): 190 us against 165.
template <typename T, int N, int CPB, bool LOCAL>
__global__ void __launch_bounds__(CPB * N / 4 + kEw<CPB>, CPB * N / 4 > 128 ? 2 : CPB * N / 4 > 64 ? 3 : 5)
    ssm_fwd_kernel(const SsmParams p, const SegArgs sg) {
    using L = Lay<N, CPB>;
    constexpr int LPC = L::LPC, TH = L::THREADS, EW = kEw<CPB>, UNITS = (kTile / 4) * (CPB / 2);
    using Quad = typename Four<T>::Raw;
    using Raw = typename Pair<T>::Raw;
    if (LOCAL) chain_next();
    else chain_wait();
    extern __shared__ __align__(16) unsigned char smem_raw[];
    FwdSmem<T, N, CPB, LOCAL>& sm = *reinterpret_cast<FwdSmem<T, N, CPB, LOCAL>*>(smem_raw);
    auto &sD = sm.D, &sU = sm.U;
    auto& sY = sm.Y;
    auto& sB = sm.B;
    auto& sC = sm.C;
    const int nblk = p.D / CPB;
    const int bh = blockIdx.x / nblk, c0 = (blockIdx.x % nblk) * CPB;
    const int b = bh / p.H, h = bh % p.H, seg = blockIdx.y;
    const int len = seq_len(p, b);
    const int begin = seg * sg.len;
    if (LOCAL ? begin + sg.len >= len : (seg > 0 && begin >= len)) return;  // nothing after or in it
    const int end = LOCAL ? begin + sg.len : min(begin + sg.len, len);
    const int tiles = (end - begin + kTile - 1) / kTile;
    const size_t row0 = (size_t)bh * p.T;
    const T* x = static_cast<const T*>(p.x) + row0 * p.D + c0;
    const T* cs = p.cs_in ? static_cast<const T*>(p.cs_in) + (size_t)bh * (p.W - 1) * p.D + c0 : nullptr;

    if (threadIdx.x >= TH) {  // ---------------- element-wise warps
        const int tid = threadIdx.x - TH;
        const T* dt = static_cast<const T*>(p.dt) + row0 * p.D + c0;
        const T* z = p.z ? static_cast<const T*>(p.z) + row0 * p.D + c0 : nullptr;
        T* y = static_cast<T*>(p.y) + row0 * p.D + c0;
        const size_t grow = (size_t)(b * p.G + h / (p.H / p.G)) * p.T;
        const T* Bm = static_cast<const T*>(p.Bm) + grow * N;
        const T* Cm = static_cast<const T*>(p.Cm) + grow * N;
        // channels cp, cp + 1 of tokens 4 uq .. 4 uq + 3 of a tile
        const bool has_unit = tid < UNITS;
        const int uq = tid / (CPB / 2), cp = 2 * (tid % (CPB / 2)), pl = cp >> 1;
        const unsigned off = (unsigned)(4 * uq) * p.D + cp;
        float w[4][2] = {}, cb[2] = {0.0f, 0.0f}, bias[2] = {0.0f, 0.0f}, feed[2] = {0.0f, 0.0f};
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
        Raw xr[7], dr[4], zr[4];
        // A tile whose tokens are all there and not the sequence's first needs no tests.
        auto whole = [&](int t0) { return t0 >= 4 && t0 + kTile <= end; };
        auto fetch = [&](int t0, auto inner) {
            constexpr bool IN = decltype(inner)::value;
            const T *xt = x + (size_t)t0 * p.D, *dtt = dt + (size_t)t0 * p.D;
            const int tq = t0 + 4 * uq;
#pragma unroll
            for (int i = 0; i < 7; ++i) {
                const int t = tq - 3 + i;
                xr[i] = Pair<T>::zero();
                if (i < 3 && p.W < 4 - i) continue;  // 3 - i tokens back: not in the filter
                if (IN) {
                    xr[i] = ldpair(xt + (i - 3) * p.D + off);
                } else if (t >= 0) {
                    if (t < end) xr[i] = ldpair(x + (size_t)t * p.D + cp);
                } else if (cs && t >= 1 - p.W) {
                    xr[i] = ldpair(cs + (size_t)(p.W - 1 + t) * p.D + cp);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) dr[j] = IN || tq + j < end ? ldpair(dtt + j * p.D + off) : Pair<T>::zero();
        };
        auto fetch_z = [&](int t0) {
            const T* zt = z + (size_t)t0 * p.D;
            const int tq = t0 + 4 * uq;
#pragma unroll
            for (int j = 0; j < 4; ++j) zr[j] = tq + j < end ? ldpair(zt + j * p.D + off) : Pair<T>::zero();
        };
        auto copy_bc = [&](int tile) {
            constexpr int PER = 16 / (int)sizeof(T), ROW = N / PER;  // values in 16 bytes, pieces of a token
            const int t0 = begin + tile * kTile;
            for (int i = tid; i < kTile * ROW; i += EW) {
                const bool there = t0 + i / ROW < end;
                const size_t at = (size_t)(there ? t0 : 0) * N + (there ? i * PER : 0);
                copy16(reinterpret_cast<char*>(&sB[tile % 3][0][0]) + 16 * i, Bm + at, there);
                if (!LOCAL) copy16(reinterpret_cast<char*>(&sC[tile % 3][0][0]) + 16 * i, Cm + at, there);
            }
        };
        auto stage = [&](int tile, auto inner) {
            constexpr bool IN = decltype(inner)::value;
            const int tq = begin + tile * kTile + 4 * uq;
            // two neighbouring tokens of a channel an instruction
            float2 d[2][2], u[2][2];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 a = Pair<T>::f(dr[j]);
                (&d[0][j >> 1].x)[j & 1] = a.x;
                (&d[1][j >> 1].x)[j & 1] = a.y;
            }
            if (p.preact) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int m = 0; m < 2; ++m) d[e][m] = softplus2(add2(d[e][m], two(bias[e])));
            }
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
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int m = 0; m < 2; ++m) u[e][m] = silu2(u[e][m]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 a = Pair<T>::f(xr[3 + j]);
                    (&u[0][j >> 1].x)[j & 1] = a.x;
                    (&u[1][j >> 1].x)[j & 1] = a.y;
                }
            }
            if (!IN) {  // tokens behind the end leave the state as it is
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (tq + j >= end) (&d[e][j >> 1].x)[j & 1] = (&u[e][j >> 1].x)[j & 1] = 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int at = pl + e * L::ODD;
                *reinterpret_cast<float4*>(sD[tile & 1][uq][at]) = make_float4(d[e][0].x, d[e][0].y, d[e][1].x, d[e][1].y);
                *reinterpret_cast<float4*>(sU[tile & 1][uq][at]) = make_float4(u[e][0].x, u[e][0].y, u[e][1].x, u[e][1].y);
            }
        };
        auto finish = [&](int tile, auto inner) {  // y of the unit, with the skip and the gate
            constexpr bool IN = decltype(inner)::value;
            const int t0 = begin + tile * kTile, tq = t0 + 4 * uq;
            T* yt = y + (size_t)t0 * p.D;
            float2 yv[2][2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float4 a = *reinterpret_cast<const float4*>(sY[tile & 1][uq][pl + e * L::ODD]);
                const float4 u = *reinterpret_cast<const float4*>(sU[tile & 1][uq][pl + e * L::ODD]);
                yv[e][0] = fma2(two(feed[e]), make_float2(u.x, u.y), make_float2(a.x, a.y));
                yv[e][1] = fma2(two(feed[e]), make_float2(u.z, u.w), make_float2(a.z, a.w));
            }
            if (z) {
                float2 g[2][2];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 a = Pair<T>::f(zr[j]);
                    (&g[0][j >> 1].x)[j & 1] = a.x;
                    (&g[1][j >> 1].x)[j & 1] = a.y;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int m = 0; m < 2; ++m) yv[e][m] = mul2(yv[e][m], silu2(g[e][m]));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (IN || tq + j < end) stpair(yt + j * p.D + off, (&yv[0][j >> 1].x)[j & 1], (&yv[1][j >> 1].x)[j & 1]);
        };
        using Yes = std::true_type;
        using No = std::false_type;
        auto fetch_any = [&](int tile) {
            const int t0 = begin + tile * kTile;
            if (!has_unit || tile >= tiles) return;
            if (whole(t0)) fetch(t0, Yes());
            else fetch(t0, No());
        };
        auto stage_any = [&](int tile) {
            if (!has_unit || tile >= tiles) return;
            if (whole(begin + tile * kTile)) stage(tile, Yes());
            else stage(tile, No());
        };
        auto copy_any = [&](int tile) {
            if (tile < tiles) copy_bc(tile);
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        const bool out = !LOCAL && p.y && has_unit;
        copy_any(0);
        copy_any(1);
        fetch_any(0);
        stage_any(0);
        fetch_any(1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
        for (int k = 0; k <= tiles; ++k) {  // one turn more than the scan warps: the last tile's y
            if (k > 0 && out) {
                if (whole(begin + (k - 1) * kTile)) finish(k - 1, Yes());
                else finish(k - 1, No());
            }
            if (k == tiles) break;
            copy_any(k + 2);
            stage_any(k + 1);
            fetch_any(k + 2);
            if (out && z) fetch_z(begin + k * kTile);
            asm volatile("cp.async.wait_group 1;" ::: "memory");  // B and C of tile k + 1 are there
            __syncthreads();
        }
    } else {  // ------------------------------- scan warps
        const int tid = threadIdx.x;
        // states 4 sl .. 4 sl + 3 of channel ch
        const int ch = tid / LPC, sl = tid % LPC, place = L::place(ch);
        const size_t srow = ((size_t)bh * p.D + c0 + ch) * N + 4 * sl;
        const size_t states = (size_t)p.B * p.H * p.D;
        float2 A2[2], s[2] = {two(0.0f), two(0.0f)};
        float dsum = 0.0f;
        {
            const float4 a = ld4(p.A + ((size_t)h * p.D + c0 + ch) * N + 4 * sl);
            A2[0] = make_float2(a.x * kLog2e, a.y * kLog2e);
            A2[1] = make_float2(a.z * kLog2e, a.w * kLog2e);
        }
        if (!LOCAL) {
            if (p.S0) {
                const float4 v = ld4(p.S0 + srow);
                s[0] = make_float2(v.x, v.y);
                s[1] = make_float2(v.z, v.w);
            }
            for (int j = 0; j < seg; ++j) {  // the segments before this one
                const float4 v = *reinterpret_cast<const float4*>(sg.local + j * states * N + srow);
                const float2 ds = two(sg.dsum[j * states + (size_t)bh * p.D + c0 + ch]);
                s[0] = fma2(ex22(mul2(A2[0], ds)), s[0], make_float2(v.x, v.y));
                s[1] = fma2(ex22(mul2(A2[1], ds)), s[1], make_float2(v.z, v.w));
            }
        }
        __syncthreads();
        for (int k = 0; k < tiles; ++k) {
            const int t0 = begin + k * kTile, m = k & 1, m3 = k % 3;
#pragma unroll 4
            for (int q = 0; q < kTile / 4; ++q) {
                if (!LOCAL && p.saved && (q & 3) == 0 && t0 + 4 * q < end) {
                    const size_t nc = (p.T + kSsmChunk - 1) / kSsmChunk;
                    const size_t at = (((size_t)bh * nc + (t0 + 4 * q) / kSsmChunk) * p.D + c0 + ch) * N + 4 * sl;
                    *reinterpret_cast<float4*>(p.saved + at) = make_float4(s[0].x, s[0].y, s[1].x, s[1].y);
                }
                const float4 d4 = *reinterpret_cast<const float4*>(sD[m][q][place]);
                const float4 u4 = *reinterpret_cast<const float4*>(sU[m][q][place]);
                const float dd[4] = {d4.x, d4.y, d4.z, d4.w}, uu[4] = {u4.x, u4.y, u4.z, u4.w};
                float yy[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const Quad bq = sB[m3][4 * q + j][sl];
                    const float2 d2 = two(dd[j]), du = two(dd[j] * uu[j]);
                    s[0] = fma2(decay2(d2, A2[0]), s[0], mul2(du, Four<T>::lo(bq)));
                    s[1] = fma2(decay2(d2, A2[1]), s[1], mul2(du, Four<T>::hi(bq)));
                    if (LOCAL) {
                        dsum += dd[j];
                    } else {
                        const Quad cq = sC[m3][4 * q + j][sl];
                        const float2 v = fma2(s[1], Four<T>::hi(cq), mul2(s[0], Four<T>::lo(cq)));
                        yy[j] = v.x + v.y;
                    }
                }
                if (!LOCAL) {
                    const float r = lane_sum4<LPC>(yy[0], yy[1], yy[2], yy[3]);
                    if (sl < 4) sY[m][q][place][sl] = r;
                }
            }
            __syncthreads();
        }
        if (LOCAL) {
            *reinterpret_cast<float4*>(sg.local + seg * states * N + srow) = make_float4(s[0].x, s[0].y, s[1].x, s[1].y);
            if (sl == 0) sg.dsum[seg * states + (size_t)bh * p.D + c0 + ch] = dsum;
        } else if (end == len && p.ST) {
            *reinterpret_cast<float4*>(p.ST + srow) = make_float4(s[0].x, s[0].y, s[1].x, s[1].y);
        }
    }
    if (!LOCAL && end == len && p.cs_out) {  // the last W-1 inputs, some of them perhaps carried in
        T* out = static_cast<T*>(p.cs_out) + (size_t)bh * (p.W - 1) * p.D + c0;
        for (int i = threadIdx.x; i < (p.W - 1) * CPB; i += TH + EW) {
            const int r = i / CPB, c = i % CPB, t = len - (p.W - 1) + r;
            float v = 0.0f;
            if (t >= 0) v = ldf(x + (size_t)t * p.D + c);
            else if (cs) v = ldf(cs + (size_t)(p.W - 1 + t) * p.D + c);
            stf(out + (size_t)r * p.D + c, v);
        }
    }
}

// ------------------------------------------------------------------ single tokens
constexpr int kStepThreads = 256;

// A block has 1024 / N channels of R sequences, four states a thread; one read of A
// serves the R sequences.  A stream of the state, read and written once.  One
// thread per channel and sequence makes delta, u and the gate while the states are
// on their way (in the first version every lane of a channel did, and the loads of
// the 16 or 32 of them bounded it: B256 H16 D128 N64 142 us); its inputs, B and C
// are asked for before the states, so that nothing waits behind them.
template <typename T, int N, int R>
__global__ void __launch_bounds__(kStepThreads) ssm_step_kernel(const SsmStepParams p) {
    constexpr int LPC = N / 4, CB = kStepThreads / LPC, ITEMS = (R * CB + kStepThreads - 1) / kStepThreads;
    constexpr int HB = CB <= 16 ? 1 : CB / 16;  // heads a block may reach into (D >= 16)
    constexpr int QUADS = R * HB * LPC, BCQ = (QUADS + kStepThreads - 1) / kStepThreads;
    using Quad = typename Four<T>::Raw;
    __shared__ float4 sm[R][CB];  // delta, u, factor of the output, skip
    __shared__ __align__(16) Quad sB[QUADS];
    __shared__ __align__(16) Quad sC[QUADS];
    const int ds = 31 - __clz(p.D), hd = p.H << ds, nblk = (hd + CB - 1) / CB, hpg = p.H / p.G;
    const int first = (blockIdx.x % nblk) * CB, b0 = (blockIdx.x / nblk) * R, h0 = first >> ds;
    const int tid = threadIdx.x, ch = tid / LPC, sl = tid % LPC;
    const int hc = first + ch, hcc = min(hc, hd - 1);  // threads without a channel follow the last one and store nothing
    // ---- ask for everything
    float xv[ITEMS], dv[ITEMS], zv[ITEMS];
    T raw[ITEMS], old[ITEMS][3];
#pragma unroll
    for (int m = 0; m < ITEMS; ++m) {
        const int i = tid + m * kStepThreads, r = i / CB, k = first + i % CB, b = b0 + r;
        xv[m] = dv[m] = zv[m] = 0.0f;
        if (r < R && k < hd && b < p.B) {
            const size_t row = (size_t)b * hd + k;
            raw[m] = static_cast<const T*>(p.x)[row];
            dv[m] = ldf(static_cast<const T*>(p.dt) + row);
            if (p.z) zv[m] = ldf(static_cast<const T*>(p.z) + row);
            if (p.W > 1) {
                const T* cs = static_cast<const T*>(p.cs) + ((((size_t)b * p.H + (k >> ds)) * (p.W - 1)) << ds) + (k & (p.D - 1));
#pragma unroll
                for (int j = 1; j < 4; ++j)
                    if (j < p.W) old[m][j - 1] = cs[(size_t)(p.W - 1 - j) << ds];
            }
        }
    }
    Quad bq[BCQ], cq[BCQ];
#pragma unroll
    for (int m = 0; m < BCQ; ++m) {
        const int i = tid + m * kStepThreads, n = i % LPC, hh = i / LPC % HB, r = i / LPC / HB;
        if (i < QUADS) {
            const size_t at = ((size_t)min(b0 + r, p.B - 1) * p.G + min(h0 + hh, p.H - 1) / hpg) * N + 4 * n;
            bq[m] = Four<T>::ld(static_cast<const T*>(p.Bm) + at);
            cq[m] = Four<T>::ld(static_cast<const T*>(p.Cm) + at);
        }
    }
    float* S = p.S + ((size_t)b0 * hd + hcc) * N + 4 * sl;
    const size_t next = (size_t)hd * N;
    float4 s4[R];
#pragma unroll
    for (int r = 0; r < R; ++r) s4[r] = *reinterpret_cast<const float4*>(S + (b0 + r < p.B ? r * next : 0));
    const float4 a4 = ld4(p.A + (size_t)hcc * N + 4 * sl);
    // ---- per channel and sequence
#pragma unroll
    for (int m = 0; m < ITEMS; ++m) {
        const int i = tid + m * kStepThreads, r = i / CB, k = first + i % CB, b = b0 + r;
        if (r < R && k < hd && b < p.B) {
            float u = ldf(&raw[m]), d = dv[m];
            if (p.W) {
                float acc = fmaf(p.cw[(size_t)k * p.W], u, p.cb ? p.cb[k] : 0.0f);
                T* cs = static_cast<T*>(p.cs) + ((((size_t)b * p.H + (k >> ds)) * (p.W - 1)) << ds) + (k & (p.D - 1));
#pragma unroll
                for (int j = 1; j < 4; ++j)
                    if (j < p.W) {
                        acc = fmaf(p.cw[(size_t)k * p.W + j], ldf(&old[m][j - 1]), acc);
                        cs[(size_t)(p.W - 1 - j) << ds] = j == 1 ? raw[m] : old[m][j > 1 ? j - 2 : 0];
                    }
                u = p.silu ? silu(acc) : acc;
            }
            if (p.preact) d = softplus(d + (p.dt_bias ? p.dt_bias[k] : 0.0f));
            sm[r][i % CB] = make_float4(d, u, p.z ? silu(zv[m]) : 1.0f, p.dfeed ? p.dfeed[k] * u : 0.0f);
        }
    }
#pragma unroll
    for (int m = 0; m < BCQ; ++m) {
        const int i = tid + m * kStepThreads;
        if (i < QUADS) {
            sB[i] = bq[m];
            sC[i] = cq[m];
        }
    }
    __syncthreads();
    // ---- the states
    const float2 A2[2] = {make_float2(a4.x * kLog2e, a4.y * kLog2e), make_float2(a4.z * kLog2e, a4.w * kLog2e)};
    const int hh = (hcc >> ds) - h0;
#pragma unroll
    for (int q = 0; q < R; q += 4) {
        float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int r = q; r < R && r < q + 4; ++r) {
            const float4 v = sm[r][ch];
            const Quad bb = sB[(r * HB + hh) * LPC + sl], cc = sC[(r * HB + hh) * LPC + sl];
            const float2 d2 = two(v.x), du = two(v.x * v.y);
            const float2 lo = fma2(decay2(d2, A2[0]), make_float2(s4[r].x, s4[r].y), mul2(du, Four<T>::lo(bb)));
            const float2 hi = fma2(decay2(d2, A2[1]), make_float2(s4[r].z, s4[r].w), mul2(du, Four<T>::hi(bb)));
            const float2 t = fma2(hi, Four<T>::hi(cc), mul2(lo, Four<T>::lo(cc)));
            y[r - q] = t.x + t.y;
            if (hc < hd && b0 + r < p.B) *reinterpret_cast<float4*>(S + r * next) = make_float4(lo.x, lo.y, hi.x, hi.y);
        }
        const float sum = lane_sum4<LPC>(y[0], y[1], y[2], y[3]);  // lane sl < 4 has sequence q + sl's
        const int r = q + sl;
        if (sl < 4 && r < R && hc < hd && b0 + r < p.B) {
            const float4 v = sm[r][ch];
            stf(static_cast<T*>(p.y) + (size_t)(b0 + r) * hd + hc, (sum + v.w) * v.z);
        }
    }
}

// Channels a block and segments a sequence.  Measured at H24 D64 N16 bf16, 8192
// tokens in all (us, P = 1 against the best P):
//   B1 (48 blocks of 32 channels) 410 / 172 (P = 24)   B2 (96) 209 / 165 (P = 16)
//   B4 (192) 152 / 156 (P = 3)
// so sequences stay whole where the blocks reach the number of SMs (the first
// launch of a cut scan repeats nearly all of the work), and else are cut for six
// blocks an SM, each segment of at least two tiles.  Whole sequences of at most two
// blocks an SM run 16 channels a block (B4: 132 us); with more, 32 is faster
// (B8 T2048: 213 against 245).
// N = 128 (256 scan threads a block, two blocks an SM) keeps them whole from three
// quarters of the SMs on: B1 D64 T4096 whole / cut, 64 blocks 322 / 198, 104 blocks
// 323 / 292, 112 blocks 323 / 331, 128 blocks 323 / 386, 144 blocks 323 / 387.  The others
// at 128 blocks, T4096: N64 233 / 206, N32 219 / 210, N16 207 / 225 (f32 238 / 231).
struct Cut {
    int cpb, P;
};
Cut cut(const SsmParams& p) {
    Cut c;
    c.cpb = p.N == 16 ? 32 : p.N == 32 ? 16 : 8;
    if (c.cpb > p.D) c.cpb = p.D;
    const long long blocks = (long long)p.B * p.H * (p.D / c.cpb), sms = sm_count();
    c.P = 1;
    if (blocks >= (p.N == 128 ? sms * 3 / 4 : sms)) {
        if (p.N == 16 && blocks < 2 * sms) c.cpb = 16;
        return c;
    }
    long long P = 6 * sms / blocks;
    const long long most = p.T / (2 * kTile);
    if (P > most) P = most;
    if (P > 64) P = 64;
    c.P = P < 2 ? 1 : (int)P;
    return c;
}
int segment_len(int T, int P) {
    const int tiles = (T + kTile - 1) / kTile;
    return (tiles + P - 1) / P * kTile;
}

template <typename T, int N, int CPB, bool LOCAL>
cudaError_t launch_fwd_pass(const SsmParams& p, const SegArgs& sg, cudaStream_t s) {
    auto kern = ssm_fwd_kernel<T, N, CPB, LOCAL>;
    constexpr int smem = sizeof(FwdSmem<T, N, CPB, LOCAL>);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid((unsigned)((long long)p.B * p.H * (p.D / CPB)), LOCAL ? sg.P - 1 : sg.P);
    if (!LOCAL && sg.P > 1) return launch_chained(kern, grid, CPB * N / 4 + kEw<CPB>, smem, s, p, sg);
    kern<<<grid, CPB * N / 4 + kEw<CPB>, smem, s>>>(p, sg);
    return cudaGetLastError();
}

template <typename T, int N, int CPB>
cudaError_t launch_fwd(const SsmParams& p, const SegArgs& sg, cudaStream_t s) {
    if (sg.P > 1) {
        const cudaError_t e = launch_fwd_pass<T, N, CPB, true>(p, sg, s);
        if (e != cudaSuccess) return e;
    }
    return launch_fwd_pass<T, N, CPB, false>(p, sg, s);
}

template <typename T>
cudaError_t launch_fwd_t(const SsmParams& p, const SegArgs& sg, int cpb, cudaStream_t s) {
    switch (p.N) {
        case 16: return cpb == 32 ? launch_fwd<T, 16, 32>(p, sg, s) : launch_fwd<T, 16, 16>(p, sg, s);
        case 32: return launch_fwd<T, 32, 16>(p, sg, s);
        case 64: return launch_fwd<T, 64, 8>(p, sg, s);
        default: return launch_fwd<T, 128, 8>(p, sg, s);
    }
}

template <typename T, int N>
cudaError_t launch_step(const SsmStepParams& p, cudaStream_t s) {
    constexpr int CB = kStepThreads / (N / 4);
    const long long nblk = ((long long)p.H * p.D + CB - 1) / CB;
    // Eight sequences a block (one read of A for eight states, 128 bytes a thread on
    // their way) where blocks of one sequence would be more than the SMs hold at a
    // time, about six each; fewer go out one by one and spread over the SMs.  Measured
    // (us, one / eight): H16 D128 N64 of B4 3.15 / 3.19, B8 5.0 / 3.6, B32 11.6 / 7.0,
    // B256 99.5 / 51.5; H24 D64 N16 of B16 3.0 / 4.0, B32 3.7 / 4.2, B48 5.1 / 4.2, B256
    // 20.5 / 13.8; H32 D128 N128, groups of eight not full, B2 5.5 / 5.2, B3 6.3 / 5.4, B5
    // 8.9 / 5.5, B9 15.0 / 9.5, B17 32.4 / 21.2.
    const bool many = nblk * p.B > 6LL * sm_count();
    const long long grid = nblk * (many ? (p.B + 7) / 8 : p.B);
    if (many) ssm_step_kernel<T, N, 8><<<(unsigned)grid, kStepThreads, 0, s>>>(p);
    else ssm_step_kernel<T, N, 1><<<(unsigned)grid, kStepThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_step_t(const SsmStepParams& p, cudaStream_t s) {
    switch (p.N) {
        case 16: return launch_step<T, 16>(p, s);
        case 32: return launch_step<T, 32>(p, s);
        case 64: return launch_step<T, 64>(p, s);
        default: return launch_step<T, 128>(p, s);
    }
}

}  // namespace

size_t ssm_fwd_workspace(const SsmParams& p) {
    const int P = cut(p).P;
    return P < 2 ? 0 : (size_t)(P - 1) * p.B * p.H * p.D * (p.N + 1) * 4;
}

cudaError_t launch_ssm_fwd(const SsmParams& p, cudaStream_t s) {
    SegArgs sg;
    const Cut c = cut(p);
    sg.P = p.ws && p.ws_bytes >= ssm_fwd_workspace(p) ? c.P : 1;
    sg.len = segment_len(p.T, sg.P);
    sg.local = static_cast<float*>(p.ws);
    sg.dsum = sg.local + (size_t)(sg.P - 1) * p.B * p.H * p.D * p.N;
    return p.bf16 ? launch_fwd_t<__nv_bfloat16>(p, sg, c.cpb, s) : launch_fwd_t<float>(p, sg, c.cpb, s);
}

cudaError_t launch_ssm_step(const SsmStepParams& p, cudaStream_t s) {
    return p.bf16 ? launch_step_t<__nv_bfloat16>(p, s) : launch_step_t<float>(p, s);
}

}  // namespace rdm
