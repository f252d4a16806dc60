// Gradients of the selective scan from an empty start.  With g = dout silu(z)
// (the gradient of y) and lambda_t the gradient of the state h_t:
//     lambda_t = C_t g_t + a_{t+1} lambda_{t+1}
//     dC_t = sum_c g h_t            dB_t = sum_c lambda_t dt u
//     du = dt sum_n lambda B + skip g
//     q_n = lambda_n a_n h_{t-1,n}, ddt = u sum_n lambda B + sum_n A q,  draw = ddt sigmoid(raw + dt_bias)
//     dA_n = sum_t dt q_n           dskip = sum_t g u,  ddt_bias = sum_t draw,  dz = dout y silu'(z)
// The states are not kept by the forward call: they are formed again.
//
// Chunks of tokens run in parallel.  scan_grad_chunks leaves every chunk's start
// state and the gradient that the chunk behind hands to it; k_bwd_main walks its
// chunk forwards once, keeping the state at every 4th token in shared memory, then
// backwards, 4 tokens at a time: their decays and states are formed again into
// registers, and lambda runs back over them.
//
// What bounds k_bwd_main: issue.  A token of 32 channels takes 490 instructions at N =
// 16, 152 of them packed FMAs, MULs and exponentials, about 100 the two sums over
// lanes (halving exchanges: a value costs a shuffle, an add and two selects), the rest
// staging and the per-element functions; 62% of the issue slots are used with three
// warps a scheduler, and 68% of the shared-memory pipe.  At [4, 4096, 1024] bf16: 337
// us, beside 129 for the summaries, 24 for their chain and 23 for the last sums; 620
// us with one channel a thread in plain FMAs, 449 with both channels' states in 255
// registers and two blocks an SM, 396 before dt was kept for the way back.
#include <type_traits>

#include "ssm_internal.h"

namespace favor {

constexpr int kBwdThreads = 128;
constexpr int kBwdSub = 4;          // tokens whose states are in registers at a time
constexpr int kBwdTile = 16;        // tokens staged in shared memory at a time
constexpr int kBwdNS = 4;           // states a thread, of
constexpr int kBwdCH = 2;           // channels
// Tokens of a chunk: the kept states take 4 KB for every 4 of them.  At N = 16 in bf16 three blocks of 74 KB
// share an SM (64 tokens and two blocks, before the states were formed a channel at a time: 4% slower), at N =
// 32 in either type too; fp32 at N = 16, bf16 at N = 8 and either at N = 64 have two (92 to 110 KB), fp32 at
// N = 8 one (142 KB).
constexpr int kBwdChunk = 32;

struct BwdPlan {
    int tiles, tpg, Dg, nC;
};

struct BwdWs {
    ScanWs s;
    float* dA;      // [B][nC][D][N]
    float* dskip;   // [B][nC][D]
    float* dbias;   // [B][nC][D]
    float* bc;      // [tpg][B][L][G][N/4][2][4] per channel tile: dB, dC of 4 states
};

static BwdWs bwd_layout(float* ws, const BwdPlan& pl, int B, int L, int D, int N, int G, size_t* total) {
    BwdWs w;
    const size_t rows = (size_t)B * pl.nC;
    float* at = ws;
    w.s.hs = at; at += rows * D * N;
    w.s.mu = at; at += rows * D * N;
    w.dA = at; at += rows * D * N;
    w.bc = at; at += (size_t)pl.tpg * B * L * G * 2 * N;
    w.s.sdt = at; at += rows * D;
    w.dskip = at; at += rows * D;
    w.dbias = at; at += rows * D;
    *total = (size_t)(at - ws);
    return w;
}

static BwdPlan bwd_plan(const SsmHandle& h, int L) {
    BwdPlan pl;
    const int CPB = kBwdThreads * kBwdNS * kBwdCH / h.N;
    pl.Dg = h.D / h.G;
    pl.tpg = (pl.Dg + CPB - 1) / CPB;
    pl.tiles = pl.tpg * h.G;
    pl.nC = (L + kBwdChunk - 1) / kBwdChunk;
    return pl;
}

size_t scan_backward_ws(const SsmHandle& h) {
    size_t n = 0;
    bwd_layout(nullptr, bwd_plan(h, h.max_L), h.max_B, h.max_L, h.D, h.N, h.G, &n);
    return n;
}

// Sums v[0..W) over the lanes that differ in the bits of lane at and above BIT:
// while more than one value is left each step halves the values a lane holds (a
// lane with the bit set keeps the upper half), then plain butterflies.  `first`
// becomes the index of the lane's v[0].
template <int W, int BIT, int END>
struct LaneSum {
    static __device__ __forceinline__ void go(float* v, unsigned& first) {
        if constexpr (BIT < END) {
            if constexpr (W % 2 == 0) {
                const bool up = threadIdx.x & BIT;
#pragma unroll
                for (int i = 0; i < W / 2; ++i) {
                    const float keep = up ? v[i + W / 2] : v[i], give = up ? v[i] : v[i + W / 2];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, give, BIT);
                }
                first += up ? W / 2 : 0;
                LaneSum<W / 2, BIT * 2, END>::go(v, first);
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], BIT);
                LaneSum<W, BIT * 2, END>::go(v, first);
            }
        }
    }
};
constexpr int lane_sum_left(int W, int lanes) { return lanes > 1 && W % 2 == 0 ? lane_sum_left(W / 2, lanes / 2) : W; }

template <typename T, int N, int V>
struct BwdShared {
    static constexpr int LPC = N / kBwdNS, CPB = kBwdThreads * kBwdCH / LPC, PAIRS = CPB / 2, CV = CPB / V;
    static constexpr int CHUNK = kBwdChunk, W = kBwdThreads / 32;
    // Channel cl of a tile sits at place (cl % VP) (CPB / VP) + cl / VP of a shared row, as in the
    // forward kernel; the narrow path keeps the places, and with them the order of the sums.
    static constexpr int VP = 16 / (int)sizeof(T), PV = CPB / VP;
    static __device__ __forceinline__ int place(int cl) { return cl % VP * PV + cl / VP; }
    static constexpr bool ASYNC = sizeof(Pack<T, V>) >= 4;   // asynchronous copies move 4 bytes at least
    static constexpr int VECS = kBwdTile * CV, NV = (VECS + kBwdThreads - 1) / kBwdThreads;
    static constexpr int BV = V > 1 ? 16 / (int)sizeof(T) : 1;
    static constexpr int BC = kBwdTile * N / BV, EB = (BC + kBwdThreads - 1) / kBwdThreads;
    static constexpr int PAD = PV < 16 ? PV / 2 : 4;   // the rows that one warp's element lanes touch start on other banks
    float4 keep[CHUNK / kBwdSub][kBwdCH][kBwdThreads];
    // of a channel pair, each: (dt, dt u) and g, then (y, lambda B) and A q
    float4 dx[kBwdTile][PAIRS + PAD];
    float2 g[kBwdTile][PAIRS + PAD];
    alignas(16) float bc[2][kBwdTile][N];
    // dB, dC of 4 tokens from each warp, [token][part][8], go where the warp kept the states before them
    static constexpr bool ALIAS = LPC * kBwdSub * 8 * sizeof(float) <= sizeof(float4) * 32 * kBwdCH;
    alignas(16) float red[ALIAS ? 1 : W][ALIAS ? 1 : kBwdTile / kBwdSub][ALIAS ? 4 : kBwdSub * LPC * 8];
    __device__ __forceinline__ float* part_sums(int warp, int sub, int o) {
        if constexpr (ALIAS) return reinterpret_cast<float*>(&keep[sub][o >> 7][warp * 32]) + (o & 127);
        else return &red[warp][sub % (kBwdTile / kBwdSub)][o];
    }
    float d[CHUNK][CPB];   // dt of the chunk, a row's places turned by its number against bank conflicts
    static __device__ __forceinline__ int turned(int tt, int place) { return place ^ ((tt & 3) << 3 & (CPB - 1)); }
    Pack<T, V> raw[2][4][NV][kBwdThreads];
    Pack<T, BV> rawbc[2][2][EB > 1 ? EB * kBwdThreads : BC];
    alignas(16) float sbias[CPB], sskip[CPB];   // by place
};

template <typename T, int N, int V>
__global__ void __launch_bounds__(kBwdThreads, 3) k_bwd_main(ScanArgs p, BwdPlan pl, BwdWs ws, int D, int G) {
    using S = BwdShared<T, N, V>;
    constexpr int NS = kBwdNS, CH = kBwdCH, LPC = S::LPC, CPB = S::CPB, CV = S::CV, NV = S::NV, BV = S::BV, EB = S::EB;
    constexpr int TL = kBwdTile, SUB = kBwdSub;
    extern __shared__ __align__(16) unsigned char smem[];
    S& sm = *reinterpret_cast<S*>(smem);

    const int tile = blockIdx.x % pl.tiles, rest = blockIdx.x / pl.tiles;
    const int b = rest % p.B, chunk = rest / p.B;
    const int len = row_len(p.lens, b, p.L);
    const int t0 = chunk * S::CHUNK, t1 = min(t0 + S::CHUNK, len);
    const int g = tile / pl.tpg, cl = (tile % pl.tpg) * CPB, c0 = g * pl.Dg + cl, cn = min(CPB, pl.Dg - cl);
    const size_t row = (size_t)b * p.L, wr = ((size_t)b * pl.nC + chunk) * D;
    // state lanes: the channels at places 2q and 2q + 1 of the tile, states part*4 .. +3
    const int q = threadIdx.x / LPC, part = threadIdx.x % LPC, warp = threadIdx.x / 32;
    int ch[CH];
    bool live[CH];
    size_t cn0[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int at = q * CH + c;
        ch[c] = at % S::PV * S::VP + at / S::PV;
        live[c] = ch[c] < cn;
        if (!live[c]) ch[c] = 0;
        cn0[c] = (size_t)(c0 + ch[c]) * N + part * NS;
    }
    // rows of the chunk behind the row's end: no gradient
    const int tz = max(t0, t1), nz = min(t0 + S::CHUNK, p.L) - tz;
    for (int i = threadIdx.x; i < nz * cn; i += kBwdThreads) {
        const size_t at = (row + tz + i / cn) * D + c0 + i % cn;
        from_f(((T*)p.du)[at], 0.f);
        from_f(((T*)p.ddt)[at], 0.f);
        if (p.z) from_f(((T*)p.dz)[at], 0.f);
    }
    if (t0 >= t1) {   // and zeros for the sums over rows
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            if (!live[c]) continue;
            *reinterpret_cast<float4*>(ws.dA + wr * N + cn0[c]) = make_float4(0.f, 0.f, 0.f, 0.f);
            if (part == 0) ws.dskip[wr + c0 + ch[c]] = ws.dbias[wr + c0 + ch[c]] = 0.f;
        }
        return;
    }
    const T* src[4] = {(const T*)p.u, (const T*)p.dt, (const T*)p.z, (const T*)p.dout};
    const T* mat[2] = {(const T*)p.Bm + (row * G + g) * N, (const T*)p.Cm + (row * G + g) * N};
    Pack<T, V> rr[4][S::ASYNC ? 1 : NV];
    T rbc[2][S::ASYNC ? 1 : EB];
    // tile at t: nk = 2 tensors (forwards: u, dt, B) or 4 (backwards)
    auto fetch = [&](int t, int slot, bool back) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k >= 2 && !back) break;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int i = v * kBwdThreads + threadIdx.x, tt = i / CV, c = i % CV * V;
                const bool ok = i < S::VECS && t >= t0 && t + tt < t1 && c < cn && (k != 2 || p.z);
                const T* at = ok ? src[k] + (row + t + tt) * D + c0 + c : src[0];
                if constexpr (S::ASYNC) copy_async(&sm.raw[slot][k][v][threadIdx.x], at, ok);
                else rr[k][v] = ok ? load_pack<T, V>(at) : zero_pack<T, V>();
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (k && !back) break;
#pragma unroll
            for (int i = 0; i < EB; ++i) {
                const int e = i * kBwdThreads + threadIdx.x, tt = e / (N / BV), n = e % (N / BV) * BV;
                const bool ok = e < S::BC && t >= t0 && t + tt < t1;
                const T* at = ok ? mat[k] + (size_t)(t + tt) * G * N + n : mat[k];
                if constexpr (S::ASYNC) {
                    if (e < S::BC) copy_async(&sm.rawbc[slot][k][e], at, ok);
                } else {
                    from_f(rbc[k][i], 0.f);
                    if (ok) rbc[k][i] = *at;
                }
            }
        }
        if constexpr (S::ASYNC) copy_commit();
    };
    // the tile's elements arrive: dt, dt u (and g) for the state lanes, B (and C)
    auto arrive = [&](int t, int slot, bool back) {
        if constexpr (S::ASYNC) {
            copy_wait<1>();
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k >= 2 && !back) break;
#pragma unroll
                for (int v = 0; v < NV; ++v) sm.raw[slot][k][v][threadIdx.x] = rr[k][v];
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (k && !back) break;
#pragma unroll
                for (int i = 0; i < EB; ++i) {
                    const int e = i * kBwdThreads + threadIdx.x;
                    if (e < S::BC) sm.rawbc[slot][k][e].v[0] = rbc[k][i];
                }
            }
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int i = v * kBwdThreads + threadIdx.x, tt = i / CV, cv = i % CV;
            if (i >= S::VECS) break;
            const Pack<T, V> ru = sm.raw[slot][0][v][threadIdx.x], rd = sm.raw[slot][1][v][threadIdx.x];
            float d[V + V % 2];
            if constexpr (V == 1) d[1] = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e)
                d[e] = back ? sm.d[t - t0 + tt][S::turned(tt, S::place(cv * V + e))]
                            : to_f(rd.v[e]) + sm.sbias[S::place(cv * V + e)];
            if (!back) {
#pragma unroll
                for (int e = 0; e < V; e += 2) softplus_2<T>(d[e], d[e + 1]);
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int at = S::place(cv * V + e);
                if (!back) sm.d[t - t0 + tt][S::turned(tt, at)] = d[e];
                reinterpret_cast<float2*>(&sm.dx[tt][0])[at] = make_float2(d[e], d[e] * to_f(ru.v[e]));
            }
            if (back) {
                const Pack<T, V> rz = sm.raw[slot][2][v][threadIdx.x], ro = sm.raw[slot][3][v][threadIdx.x];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float gg = to_f(ro.v[e]);
                    if (p.z) gg *= to_f(rz.v[e]) * sigmoid_f<T>(to_f(rz.v[e]));
                    reinterpret_cast<float*>(&sm.g[tt][0])[S::place(cv * V + e)] = gg;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (k && !back) break;
#pragma unroll
            for (int i = 0; i < EB; ++i) {
                const int e = i * kBwdThreads + threadIdx.x;
                if (e < S::BC) {
                    const Pack<T, BV> m = sm.rawbc[slot][k][e];
                    float* to = &sm.bc[k][0][0] + e * BV;
#pragma unroll
                    for (int x = 0; x < BV; ++x) to[x] = to_f(m.v[x]);
                }
            }
        }
        __syncthreads();
    };

    // The tiles forwards, t0 .. last, and back from last to t0 are one sequence: the place that `ahead`
    // would have if the way forwards went on.
    const int last = t0 + (t1 - 1 - t0) / TL * TL;
    auto fetch_ahead = [&](int ahead, int slot) {
        const bool back = ahead > last;
        fetch(back ? 2 * last + TL - ahead : ahead, slot, back);
    };
    for (int c = threadIdx.x; c < CPB; c += kBwdThreads) {
        sm.sbias[S::place(c)] = c < cn && p.dt_bias ? p.dt_bias[c0 + c] : 0.f;
        sm.sskip[S::place(c)] = c < cn && p.skip ? p.skip[c0 + c] : 0.f;
    }
    fetch_ahead(t0, 0);
    if constexpr (S::ASYNC) fetch_ahead(t0 + TL, 1);
    // states of a thread as packed pairs; a place without a channel stays zero throughout
    uint64_t A2[CH][2], h[CH][2], mu[CH][2], dA[CH][2];
    const uint64_t mean2 = pack2(kEx2Mean, kEx2Mean);
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            A2[c][n] = live[c] ? pack2(p.A[cn0[c] + 2 * n] * kLog2e, p.A[cn0[c] + 2 * n + 1] * kLog2e) : 0ull;
            h[c][n] = live[c] ? *reinterpret_cast<const uint64_t*>(ws.s.hs + wr * N + cn0[c] + 2 * n) : 0ull;
            mu[c][n] = live[c] ? *reinterpret_cast<const uint64_t*>(ws.s.mu + wr * N + cn0[c] + 2 * n) : 0ull;
            dA[c][n] = 0ull;
        }

    __syncthreads();   // sbias

    // forwards: the state before every 4th token
    int slot = 0;
    for (int t = t0; t < t1; t += TL, slot ^= 1) {
        const int nt = min(TL, t1 - t);
        arrive(t, slot, false);
        if constexpr (!S::ASYNC) fetch_ahead(t + TL, 0);
        for (int tt = 0; tt < nt; tt += SUB) {
#pragma unroll
            for (int c = 0; c < CH; ++c)
                *reinterpret_cast<ulonglong2*>(&sm.keep[(t - t0 + tt) / SUB][c][threadIdx.x]) = make_ulonglong2(h[c][0], h[c][1]);
            if (t == last && tt + SUB >= nt) break;   // the states behind are not asked for
#pragma unroll
            for (int k = 0; k < SUB; ++k) {
                const float4 d4 = sm.dx[tt + k][q];
                const float dd[CH] = {d4.x, d4.z}, xx[CH] = {d4.y, d4.w};
                const ulonglong2 bb = *reinterpret_cast<const ulonglong2*>(&sm.bc[0][tt + k][part * NS]);
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const uint64_t d2 = pack2(dd[c], dd[c]), x2 = pack2(xx[c], xx[c]);
                    h[c][0] = fma2(x2, bb.x, mul2(ex2_2(fma2(A2[c][0], d2, mean2)), h[c][0]));
                    h[c][1] = fma2(x2, bb.y, mul2(ex2_2(fma2(A2[c][1], d2, mean2)), h[c][1]));
                }
            }
        }
        __syncthreads();
        if constexpr (S::ASYNC) fetch_ahead(t + 2 * TL, slot);
    }
    // backwards
    float dskip = 0.f, dbias = 0.f;   // of the channel at place threadIdx.x

    for (int t = last; t >= t0; t -= TL, slot ^= 1) {
        const int nt = min(TL, t1 - t);
        arrive(t, slot, true);
        if constexpr (!S::ASYNC) fetch(t - TL, 0, true);
        auto sub = [&](int s0, int ns, auto full) {
            constexpr bool FULL = decltype(full)::value;
            uint64_t accB[SUB][2], accC[SUB][2];
            // one channel after the other: decays and states of both at once would take 64 registers more
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                uint64_t a[SUB][2], hp[SUB][2], hc[2];
                float v[SUB * 3];
                const ulonglong2 k2 = *reinterpret_cast<const ulonglong2*>(&sm.keep[(t - t0 + s0) / SUB][c][threadIdx.x]);
                hc[0] = k2.x;
                hc[1] = k2.y;
#pragma unroll
                for (int k = 0; k < SUB; ++k) {
                    if (FULL || k < ns) {
                        const float2 dx = reinterpret_cast<const float2*>(&sm.dx[s0 + k][q])[c];
                        const ulonglong2 bb = *reinterpret_cast<const ulonglong2*>(&sm.bc[0][s0 + k][part * NS]);
                        const uint64_t d2 = pack2(dx.x, dx.x), x2 = pack2(dx.y, dx.y);
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            a[k][n] = ex2_2(fma2(A2[c][n], d2, mean2));
                            hp[k][n] = hc[n];
                            hc[n] = fma2(x2, n ? bb.y : bb.x, mul2(a[k][n], hc[n]));
                        }
                    }
                }
#pragma unroll
                for (int k = SUB - 1; k >= 0; --k) {
                    if (FULL || k < ns) {
                        const int tt = s0 + k;
                        const float2 dx = reinterpret_cast<const float2*>(&sm.dx[tt][q])[c];
                        const float gg = reinterpret_cast<const float*>(&sm.g[tt][q])[c];
                        const ulonglong2 bb = *reinterpret_cast<const ulonglong2*>(&sm.bc[0][tt][part * NS]);
                        const ulonglong2 cc = *reinterpret_cast<const ulonglong2*>(&sm.bc[1][tt][part * NS]);
                        const uint64_t d2 = pack2(dx.x, dx.x), x2 = pack2(dx.y, dx.y), g2 = pack2(gg, gg);
                        uint64_t y2, lb2, aq2;
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            const uint64_t Bn = n ? bb.y : bb.x, Cn = n ? cc.y : cc.x;
                            const uint64_t lam = fma2(Cn, g2, mu[c][n]);
                            accB[k][n] = c ? fma2(lam, x2, accB[k][n]) : mul2(lam, x2);
                            accC[k][n] = c ? fma2(hc[n], g2, accC[k][n]) : mul2(hc[n], g2);
                            y2 = n ? fma2(hc[n], Cn, y2) : mul2(hc[n], Cn);
                            lb2 = n ? fma2(lam, Bn, lb2) : mul2(lam, Bn);
                            mu[c][n] = mul2(a[k][n], lam);
                            const uint64_t qq = mul2(mu[c][n], hp[k][n]);
                            aq2 = n ? fma2(qq, A2[c][n], aq2) : mul2(qq, A2[c][n]);
                            dA[c][n] = fma2(qq, d2, dA[c][n]);
                            hc[n] = hp[k][n];
                        }
                        float lo, hi;
                        unpack2(y2, lo, hi);
                        v[k * 3] = lo + hi;
                        unpack2(lb2, lo, hi);
                        v[k * 3 + 1] = lo + hi;
                        unpack2(aq2, lo, hi);
                        v[k * 3 + 2] = lo + hi;
                    } else {
                        v[k * 3] = v[k * 3 + 1] = v[k * 3 + 2] = 0.f;
                        accB[k][0] = accB[k][1] = accC[k][0] = accC[k][1] = 0ull;
                    }
                }
                // y, lambda B, A q of the 4 tokens, summed over the channel's lanes
                constexpr int LEFT = lane_sum_left(SUB * 3, LPC);
                static_assert(LEFT % 3 == 0, "whole tokens are left with a lane");
                unsigned first = 0;
                LaneSum<SUB * 3, 1, LPC>::go(v, first);
                __syncwarp();   // every lane of the channel has read what is overwritten here
#pragma unroll
                for (int i = 0; i < LEFT; ++i) {
                    const int k = first / 3 + i / 3, j = i % 3;
                    if (!FULL && k >= ns) continue;
                    if (j < 2) reinterpret_cast<float*>(&sm.dx[s0 + k][q])[c * 2 + j] = v[i];
                    else reinterpret_cast<float*>(&sm.g[s0 + k][q])[c] = v[i];
                }
            }
            // dB, dC of the 4 tokens' 4 states, summed over the warp's channels
            float w[SUB * 8];
#pragma unroll
            for (int k = 0; k < SUB; ++k)
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    unpack2(accB[k][n], w[k * 8 + 2 * n], w[k * 8 + 2 * n + 1]);
                    unpack2(accC[k][n], w[k * 8 + 4 + 2 * n], w[k * 8 + 4 + 2 * n + 1]);
                }
            constexpr int LEFTW = lane_sum_left(SUB * 8, 32 / LPC);
            unsigned fw = 0;   // a multiple of LEFTW
            LaneSum<SUB * 8, LPC, 32>::go(w, fw);
            if constexpr (LEFTW % 4 == 0) {
#pragma unroll
                for (int i = 0; i < LEFTW; i += 4)
                    *reinterpret_cast<float4*>(sm.part_sums(warp, (t - t0 + s0) / SUB, ((fw / 8 + i / 8) * LPC + part) * 8 + fw % 8 + i % 8)) =
                        make_float4(w[i], w[i + 1], w[i + 2], w[i + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < LEFTW; ++i)
                    *sm.part_sums(warp, (t - t0 + s0) / SUB, (fw / 8 * LPC + part) * 8 + fw % 8 + i) = w[i];
            }
        };
        int s0 = (nt - 1) / SUB * SUB;
        if (nt % SUB) {
            sub(s0, nt - s0, std::false_type());
            s0 -= SUB;
        }
        for (; s0 >= 0; s0 -= SUB) sub(s0, SUB, std::true_type());
        __syncthreads();
        for (int i = threadIdx.x; i < nt * 2 * N; i += kBwdThreads) {
            float s = 0.f;
            const int tt = i / (2 * N), j = i % (2 * N);
#pragma unroll
            for (int w = 0; w < S::W; ++w) s += *sm.part_sums(w, (t - t0 + tt) / SUB, tt % SUB * 2 * N + j);
            ws.bc[((((size_t)(tile % pl.tpg) * p.B + b) * p.L + t + tt) * G + g) * 2 * N + j] = s;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int i = v * kBwdThreads + threadIdx.x, tt = i / CV, cv = i % CV;
            if (i >= S::VECS || tt >= nt || cv * V >= cn) continue;
            const Pack<T, V> ru = sm.raw[slot][0][v][threadIdx.x], rd = sm.raw[slot][1][v][threadIdx.x];
            const Pack<T, V> rz = sm.raw[slot][2][v][threadIdx.x], ro = sm.raw[slot][3][v][threadIdx.x];
            Pack<T, V> ou, od, oz;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int at = S::place(cv * V + e), pr = at >> 1, hf = at & 1;
                const float raw = to_f(rd.v[e]) + sm.sbias[at], sk = sm.sskip[at];
                const float d = sm.d[t - t0 + tt][S::turned(tt, at)], uu = to_f(ru.v[e]), oo = to_f(ro.v[e]);
                const float2 yl = reinterpret_cast<const float2*>(&sm.dx[tt][pr])[hf];
                const float y = yl.x, lb = yl.y;
                const float aq = reinterpret_cast<const float*>(&sm.g[tt][pr])[hf] * kLn2;   // A was scaled by log2 e
                float gg = oo;
                if (p.z) {
                    const float zz = to_f(rz.v[e]), sg = sigmoid_f<T>(zz);
                    gg *= zz * sg;
                    from_f(oz.v[e], oo * fmaf(sk, uu, y) * (sg * (1.f + zz * (1.f - sg))));
                }
                from_f(ou.v[e], fmaf(d, lb, sk * gg));
                const float dr = fmaf(uu, lb, aq) * sigmoid_f<T>(raw);
                from_f(od.v[e], dr);
                reinterpret_cast<float2*>(&sm.dx[tt][pr])[hf] = make_float2(gg * uu, dr);
            }
            const size_t at = (row + t + tt) * D + c0 + cv * V;
            *reinterpret_cast<Pack<T, V>*>((T*)p.du + at) = ou;
            *reinterpret_cast<Pack<T, V>*>((T*)p.ddt + at) = od;
            if (p.z) *reinterpret_cast<Pack<T, V>*>((T*)p.dz + at) = oz;
        }
        if constexpr (S::ASYNC) fetch(t - 2 * TL, slot, true);
        __syncthreads();
        if (threadIdx.x < CPB) {
            for (int tt = 0; tt < nt; ++tt) {
                const float2 e = reinterpret_cast<const float2*>(&sm.dx[tt][0])[threadIdx.x];
                dskip += e.x;
                dbias += e.y;
            }
        }
        __syncthreads();
    }
    if constexpr (S::ASYNC) copy_wait<0>();
#pragma unroll
    for (int c = 0; c < CH; ++c)
        if (live[c])
            *reinterpret_cast<ulonglong2*>(ws.dA + wr * N + cn0[c]) = make_ulonglong2(dA[c][0], dA[c][1]);
    if (threadIdx.x < CPB) {
        const int c = threadIdx.x % S::PV * S::VP + threadIdx.x / S::PV;
        if (c < cn) {
            ws.dskip[wr + c0 + c] = dskip;
            ws.dbias[wr + c0 + c] = dbias;
        }
    }
}

// dB, dC: the channel tiles' parts, in order, rounded once; zero behind a row's end.
template <typename T>
__global__ void __launch_bounds__(256) k_bwd_bc(ScanArgs p, BwdPlan pl, BwdWs ws, int N, int G) {
    const size_t n = (size_t)p.B * p.L * G * 2 * N, i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const size_t tg = i / (2 * N);
    const int j = (int)(i % (2 * N)), t = (int)(tg / G % p.L), b = (int)(tg / G / p.L);
    float s = 0.f;
    if (t < row_len(p.lens, b, p.L)) {
#pragma unroll 8
        for (int k = 0; k < pl.tpg; ++k) s += ws.bc[k * n + i];
    }
    T* o = (T*)(j & 4 ? p.dC : p.dB) + tg * N + j / 8 * 4 + (j & 3);
    from_f(*o, s);
}

// Sums of the parameters' gradients over the chunks of every row, in a fixed order.
__global__ void __launch_bounds__(256) k_bwd_params(ScanArgs p, BwdWs ws, int rows, int D, int N) {
    const size_t DN = (size_t)D * N, all = DN + 2 * D, i = (size_t)blockIdx.x * 32 + (threadIdx.x & 31);
    const float* src = i < DN ? ws.dA + i : i < DN + D ? ws.dskip + (i - DN) : ws.dbias + (i - DN - D);
    const float sum = block_column_sum(i < all ? src : nullptr, i < DN ? DN : D, rows);
    if (threadIdx.x >= 32 || i >= all) return;
    if (i < DN) p.dA[i] = sum;
    else if (i < DN + D) { if (p.dskip) p.dskip[i - DN] = sum; }
    else if (p.ddt_bias) p.ddt_bias[i - DN - D] = sum;
}

template <typename T, int N, int V>
static void bwd_launch(const SsmHandle& h, const ScanArgs& a, const BwdPlan& pl, const BwdWs& ws, cudaStream_t st) {
    using S = BwdShared<T, N, V>;
    static_assert(S::CPB <= kBwdThreads, "a thread for every channel");
    // the attribute's failure shows as the launch's
    cudaFuncSetAttribute(k_bwd_main<T, N, V>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(S));
    k_bwd_main<T, N, V><<<(unsigned)pl.tiles * a.B * pl.nC, kBwdThreads, sizeof(S), st>>>(a, pl, ws, h.D, h.G);
}

template <typename T, int V>
static void bwd_by_n(const SsmHandle& h, const ScanArgs& a, const BwdPlan& pl, const BwdWs& ws, cudaStream_t st) {
    if (h.N == 8) bwd_launch<T, 8, V>(h, a, pl, ws, st);
    else if (h.N == 16) bwd_launch<T, 16, V>(h, a, pl, ws, st);
    else if (h.N == 32) bwd_launch<T, 32, V>(h, a, pl, ws, st);
    else bwd_launch<T, 64, V>(h, a, pl, ws, st);
}

favor_status scan_backward(const SsmHandle& h, const ScanArgs& a, cudaStream_t st) {
    const bool f32 = h.dtype == FAVOR_DTYPE_F32;
    const BwdPlan pl = bwd_plan(h, a.L);
    size_t total = 0;
    const BwdWs ws = bwd_layout(h.ws, pl, a.B, a.L, h.D, h.N, h.G, &total);
    const bool vec = scan_grad_chunks(h, a, ws.s, kBwdChunk, st);
    if (f32 && vec) bwd_by_n<float, 4>(h, a, pl, ws, st);
    else if (f32) bwd_by_n<float, 1>(h, a, pl, ws, st);
    else if (vec) bwd_by_n<__nv_bfloat16, 8>(h, a, pl, ws, st);
    else bwd_by_n<__nv_bfloat16, 1>(h, a, pl, ws, st);
    const size_t bc = (size_t)a.B * a.L * h.G * 2 * h.N;
    const unsigned grid = (unsigned)((bc + 255) / 256);
    if (f32) k_bwd_bc<float><<<grid, 256, 0, st>>>(a, pl, ws, h.N, h.G);
    else k_bwd_bc<__nv_bfloat16><<<grid, 256, 0, st>>>(a, pl, ws, h.N, h.G);
    const size_t par = (size_t)h.D * (h.N + 2);
    k_bwd_params<<<(unsigned)((par + 31) / 32), 256, 0, st>>>(a, ws, a.B * pl.nC, h.D, h.N);
    count_launch(3);
    return check_launch("favor_ssm_scan_backward");
}

}  // namespace favor
