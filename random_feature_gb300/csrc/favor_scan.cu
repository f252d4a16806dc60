// Selective state space scan, per channel c with N states (the state is decayed
// by a rate that depends on the token):
//     dt = softplus(raw + dt_bias),  a_n = exp(dt A_n),  h_n <- a_n h_n + dt u B_n,
//     y = sum_n C_n h_n + skip u,    out = y silu(z)
// u, raw, z, out are [B, L, D]; B and C [B, L, G, N], group g serving the channels
// g D/G .. (g+1) D/G - 1.  States and every sum are fp32.
#include <initializer_list>
#include <type_traits>

#include "ssm_internal.h"

namespace favor {

constexpr int kScanThreads = 128;
enum { SCAN_OUT, SCAN_SUM, SCAN_GRAD };

// How a launch cuts channels and tokens.  A block is 128 threads over CPB
// channels of one group of one row, for one chunk of tokens walked in tiles of
// TT.  A thread holds 8 states of 2 channels, LPC = N / 8 lanes a channel pair.
//
// What bounds it: at N = 16 a token of 32 channels (one warp's) takes 110
// instructions, 32 of them packed FMAs and MULs and 20 of the exponential unit.  On
// this device an instruction's operands come from the registers two 32-bit words a
// clock (measured: fma.f32x2 of three distinct operands issues every 3.1 clocks, of
// two every 2.2, mul.f32x2 every 2.1, a plain fma 1.5, ex2 every 4.0), so the packed
// ones take 85 clocks of a quarter SM, the exponentials 80, the issue 110; they
// overlap in part.  Measured with full waves: 150 clocks.  At [16, 512, 8192], us:
// 328 so; without the exponentials 324, without the loads of B and C 314, without dt's
// and the gate's functions 287 (they stood in a copy); one channel a thread, whose
// lanes do not share the loads of B and C, 344; a token's decays formed between the
// updates of the one before, 342; 5 blocks an SM in 102 registers, 342; 3 in 168,
// 367; plain FMAs, 366.  Tokens a step of the walk: 8 against 4 is 2% faster.
//
// kScanPerSm, the blocks an SM that the registers allow, is also what the chunks are counted by.
// Shared memory allows as many to SCAN_OUT for N = 8 and 16, and for N = 32 in fp32; in bf16 3 for
// N = 32, and 2 for N = 64 in either type.  There the chunks come to two waves of blocks.  SCAN_GRAD
// has 3, 3, 2 and 1 blocks an SM in bf16 for N = 8, 16, 32, 64, in fp32 4, 4, 3 and 2.
constexpr int kScanNS = 8, kScanCH = 2, kScanPerSm = 4;

struct ScanPlan {
    int tiles;     // channel tiles a row (over all groups)
    int tpg;       // channel tiles a group
    int Dg;        // channels a group
    int nC, Lc;    // chunks, tokens a chunk
    int per;       // chunks a block (SCAN_GRAD; else 1)
};

// MODE: SCAN_OUT writes the outputs.  Where a row has several chunks they start
// from ws.hs, which k_scan_chain has formed from the chunks' summaries: SCAN_SUM
// leaves there the state that a chunk (all but a row's last) would end with from
// an empty start, and the sum of its dt, whose exponential decays what came before.
// SCAN_GRAD is the same for the backward call, over every chunk, with what the
// chunk hands to the one before it when nothing is handed to it: with g the
// gradient of y and P_t the product of a up to token t, sum_t P_t C_t g_t.
//
// A tile passes through three steps: every thread turns 8 elements (token,
// channel) into dt and dt u in shared memory; the state lanes walk the tile's
// tokens and leave y there; every thread turns its elements' y into outputs.  The
// elements come by asynchronous copies, two tiles deep, each thread
// copying what it alone reads (no barrier between them); 16-bit rows that do not start on 16
// bytes go through registers one tile ahead.
// Channel cl of a tile sits at place (cl % V) CV + cl / V of a shared row, so
// that the V channels of a thread's access land V different rows' width apart
// and neighbouring threads write neighbouring words; the state lanes take the
// places in order.
template <typename T, int N, int V, int MODE>
struct ScanShared {
    static constexpr int LPC = N / kScanNS, CPB = kScanThreads * kScanCH / LPC;
    static constexpr int EPT = V > 1 ? 32 / (int)sizeof(T) : 8;        // elements a thread, two copies of 16 bytes
    static constexpr int TT = EPT * kScanThreads / CPB, NV = EPT / V, CV = CPB / V;
    static constexpr bool ASYNC = sizeof(Pack<T, V>) >= 4;             // asynchronous copies move 4 bytes at least
    static constexpr int NT = MODE == SCAN_OUT ? 3 : MODE == SCAN_SUM ? 2 : 4;   // u, dt, z, dout
    static constexpr int NM = MODE == SCAN_SUM ? 1 : 2;                // B, C
    static constexpr int BV = V > 1 ? 16 / (int)sizeof(T) : 1;         // elements of B and C a copy
    static constexpr int BC = TT * N / BV, EB = (BC + kScanThreads - 1) / kScanThreads;
    Pack<T, V> raw[2][NT][NV][kScanThreads];
    Pack<T, BV> rawbc[2][NM][EB][kScanThreads];
    static constexpr int PAD = CV < 32 ? (CV < 2 ? 2 : CV) : 0;   // the rows that one warp's element lanes touch start on other banks
    alignas(16) float2 sdt[TT][CPB + PAD];      // (dt, dt u), then (y, )
    alignas(16) float sg[MODE == SCAN_GRAD ? TT : 1][CPB + PAD];
    alignas(16) float sbias[CV][V], sskip[CV][V];
    alignas(16) float bc[NM][TT][N];
};

template <typename T, int N, int V, int MODE>
__global__ void __launch_bounds__(kScanThreads, kScanPerSm)
k_scan(ScanArgs p, ScanPlan pl, ScanWs ws, int D, int G) {
    using S = ScanShared<T, N, V, MODE>;
    constexpr bool OUT = MODE == SCAN_OUT, GRAD = MODE == SCAN_GRAD;
    constexpr int LPC = S::LPC, CPB = S::CPB, TT = S::TT, NV = S::NV, CV = S::CV, BV = S::BV, BC = S::BC, EB = S::EB;
    constexpr int NS = kScanNS, CH = kScanCH;
    constexpr int GK = LPC < 2 ? 1 : LPC / 2;   // tokens whose y are summed over the lanes together: LPC values
    constexpr int UN = TT < 8 ? TT : 8;         // tokens a step of the walk, a multiple of GK
    extern __shared__ __align__(16) unsigned char smem[];
    S& sm = *reinterpret_cast<S*>(smem);

    const int tile = blockIdx.x % pl.tiles, rest = blockIdx.x / pl.tiles;
    const int b = rest % p.B;
    int chunk = rest / p.B * pl.per;
    const int len = row_len(p.lens, b, p.L);
    const int t0 = chunk * pl.Lc, t1 = min(t0 + pl.Lc * pl.per, len);
    if (t0 >= t1 || (MODE == SCAN_SUM && t1 == len)) return;
    const int page = OUT && p.state ? block_page(p.pg, b) : 0;
    const int g = tile / pl.tpg, cl = (tile % pl.tpg) * CPB, c0 = g * pl.Dg + cl, cn = min(CPB, pl.Dg - cl);
    const size_t row = (size_t)b * p.L;
    const T* u = (const T*)p.u + row * D + c0;
    const T* dt = (const T*)p.dt + row * D + c0;
    const T* z = p.z && MODE != SCAN_SUM ? (const T*)p.z + row * D + c0 : nullptr;
    const T* dout = GRAD ? (const T*)p.dout + row * D + c0 : nullptr;
    T* out = OUT ? (T*)p.out + row * D + c0 : nullptr;
    if (page < 0) {   // the row takes no part
        if (OUT)
            for (long long i = threadIdx.x; i < (long long)(t1 - t0) * cn; i += kScanThreads)
                from_f(out[(size_t)(t0 + i / cn) * D + i % cn], 0.f);
        return;
    }
    const T* Bm = (const T*)p.Bm + (row * G + g) * N;
    const T* Cm = (const T*)p.Cm + (row * G + g) * N;

    // element lanes: vector v is V channels of one token of the tile
    int ev_t[NV], ev_c[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int i = v * kScanThreads + threadIdx.x;
        ev_t[v] = i / CV;
        ev_c[v] = i % CV;
    }
    // registers of the narrow path, one tile ahead of the shared slots
    Pack<T, V> rr[S::ASYNC ? 1 : S::NT][S::ASYNC ? 1 : NV];
    T rbc[S::ASYNC ? 1 : S::NM][S::ASYNC ? 1 : EB];
    auto fetch = [&](int t, int slot) {
        const T* src[4] = {u, dt, z, dout};
#pragma unroll
        for (int k = 0; k < S::NT; ++k)
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const bool ok = t + ev_t[v] < t1 && ev_c[v] * V < cn && (k != 2 || z);
                const T* at = ok ? src[k] + (size_t)(t + ev_t[v]) * D + ev_c[v] * V : u;
                if constexpr (S::ASYNC) {
                    copy_async(&sm.raw[slot][k][v][threadIdx.x], at, ok);
                } else {
                    rr[k][v] = ok ? load_pack<T, V>(at) : zero_pack<T, V>();
                }
            }
        const T* mat[2] = {Bm, Cm};
#pragma unroll
        for (int k = 0; k < S::NM; ++k)
#pragma unroll
            for (int i = 0; i < EB; ++i) {
                const int e = i * kScanThreads + threadIdx.x, tt = e / (N / BV), n = e % (N / BV) * BV;
                const bool ok = e < BC && t + tt < t1;
                const T* at = ok ? mat[k] + (size_t)(t + tt) * G * N + n : mat[k];
                if constexpr (S::ASYNC) {
                    if (e < BC) copy_async(&sm.rawbc[slot][k][i][threadIdx.x], at, ok);
                } else {
                    from_f(rbc[k][i], 0.f);
                    if (ok) rbc[k][i] = *at;
                }
            }
        if constexpr (S::ASYNC) copy_commit();
    };
    // the tile's elements are in this thread's slots
    auto arrive = [&](int slot) {
        if constexpr (S::ASYNC) {
            copy_wait<1>();
        } else {
#pragma unroll
            for (int k = 0; k < S::NT; ++k)
#pragma unroll
                for (int v = 0; v < NV; ++v) sm.raw[slot][k][v][threadIdx.x] = rr[k][v];
#pragma unroll
            for (int k = 0; k < S::NM; ++k)
#pragma unroll
                for (int i = 0; i < EB; ++i) sm.rawbc[slot][k][i][threadIdx.x].v[0] = rbc[k][i];
        }
    };
    fetch(t0, 0);
    if constexpr (S::ASYNC) fetch(t0 + TT, 1);

    // state lanes: the channels at places 2q and 2q + 1, states part*8 .. +7
    const int q = threadIdx.x / LPC, part = threadIdx.x % LPC;
    int ch[CH];
    bool live[CH];
    size_t cn0[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int at = q * CH + c;
        ch[c] = at % CV * V + at / CV;
        live[c] = ch[c] < cn;
        if (!live[c]) ch[c] = 0;
        cn0[c] = (size_t)(c0 + ch[c]) * N + part * NS;
        if (part == 0) {
            sm.sbias[at % CV][at / CV] = live[c] && p.dt_bias ? p.dt_bias[c0 + ch[c]] : 0.f;
            sm.sskip[at % CV][at / CV] = live[c] && p.skip ? p.skip[c0 + ch[c]] : 0.f;
        }
    }
    uint64_t A2[CH][NS / 2], h[CH][NS / 2];
    uint64_t P[GRAD ? CH : 1][NS / 2], mu[GRAD ? CH : 1][NS / 2];
    const uint64_t mean2 = pack2(kEx2Mean, kEx2Mean);
    float* stp = OUT && p.state ? p.state + (size_t)page * D * N : nullptr;
    // Several chunks: one of them writes the page while others start, so they start from the workspace.
    const float* start = !OUT ? nullptr : pl.nC > 1 ? ws.hs + ((size_t)b * pl.nC + chunk) * D * N : stp;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int n = 0; n < NS / 2; ++n) {
            A2[c][n] = pack2(p.A[cn0[c] + 2 * n] * kLog2e, p.A[cn0[c] + 2 * n + 1] * kLog2e);
            h[c][n] = start ? *reinterpret_cast<const uint64_t*>(start + cn0[c] + 2 * n) : 0ull;
            if (GRAD) {
                P[c][n] = pack2(1.f, 1.f);
                mu[c][n] = 0ull;
            }
        }
    float total_dt[CH] = {};

    // K tokens from tt on: the states move on, the lane's part of their y comes back, token by
    // token its channels.  The decays do not wait for the states, so they are formed first.
    auto tokens = [&](int tt, auto kc, float* y) {
        constexpr int K = decltype(kc)::value;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float4 d4 = *reinterpret_cast<const float4*>(&sm.sdt[tt + k][q * CH]);
            const float dd[CH] = {d4.x, d4.z}, xx[CH] = {d4.y, d4.w};
            uint64_t a[CH][NS / 2];
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const uint64_t d2 = pack2(dd[c], dd[c]);
#pragma unroll
                for (int n = 0; n < NS / 2; ++n) a[c][n] = ex2_2(fma2(A2[c][n], d2, mean2));
                if (!OUT) total_dt[c] += dd[c];
            }
            const ulonglong2* B2 = reinterpret_cast<const ulonglong2*>(&sm.bc[0][tt + k][part * NS]);
            const ulonglong2* C2 = reinterpret_cast<const ulonglong2*>(&sm.bc[S::NM - 1][tt + k][part * NS]);
            uint64_t y2[CH], x2[CH], g2[CH];
            float2 gg;
            if (GRAD) gg = *reinterpret_cast<const float2*>(&sm.sg[tt + k][q * CH]);
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                x2[c] = pack2(xx[c], xx[c]);
                if (GRAD) g2[c] = c ? pack2(gg.y, gg.y) : pack2(gg.x, gg.x);
            }
#pragma unroll
            for (int n = 0; n < NS / 4; ++n) {
                const ulonglong2 bb = B2[n];
                ulonglong2 cc;
                if (MODE != SCAN_SUM) cc = C2[n];
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    h[c][2 * n] = fma2(x2[c], bb.x, mul2(a[c][2 * n], h[c][2 * n]));
                    h[c][2 * n + 1] = fma2(x2[c], bb.y, mul2(a[c][2 * n + 1], h[c][2 * n + 1]));
                    if (GRAD) {
                        P[c][2 * n] = mul2(P[c][2 * n], a[c][2 * n]);
                        P[c][2 * n + 1] = mul2(P[c][2 * n + 1], a[c][2 * n + 1]);
                        mu[c][2 * n] = fma2(P[c][2 * n], mul2(g2[c], cc.x), mu[c][2 * n]);
                        mu[c][2 * n + 1] = fma2(P[c][2 * n + 1], mul2(g2[c], cc.y), mu[c][2 * n + 1]);
                    }
                    if (OUT) {
                        y2[c] = n ? fma2(h[c][2 * n], cc.x, y2[c]) : mul2(h[c][2 * n], cc.x);
                        y2[c] = fma2(h[c][2 * n + 1], cc.y, y2[c]);
                    }
                }
            }
            if (OUT) {
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    float y0, y1;
                    unpack2(y2[c], y0, y1);
                    y[k * CH + c] = y0 + y1;
                }
            }
        }
    };
    // y of GK tokens from tt on, summed over a channel's lanes: at each bit of part a lane keeps
    // half of its values, the upper half where the bit is set.
    auto finish = [&](int tt, float* y, int nt) {
        if constexpr (LPC == 1) {
            sm.sdt[tt][q * CH].x = y[0];
            sm.sdt[tt][q * CH + 1].x = y[1];
        } else {
            int k = 0;
#pragma unroll
            for (int o = 1, w = LPC / 2; o < LPC; o <<= 1, w >>= 1) {
                const bool up = part & o;
#pragma unroll
                for (int i = 0; i < w; ++i) {
                    const float keep = up ? y[i + w] : y[i], give = up ? y[i] : y[i + w];
                    y[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
                k += up ? w : 0;
            }
            if (GK == 1 || tt + k / CH < nt) sm.sdt[tt + k / CH][q * CH + k % CH].x = y[0];
        }
    };

    auto bias_of = [](const float (&f)[V]) {
        Pack<float, V> r;
        if constexpr (V >= 4) {
#pragma unroll
            for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(&r.v[i]) = *reinterpret_cast<const float4*>(&f[i]);
        } else {
            r.v[0] = f[0];
        }
        return r;
    };
    // the state (OUT: into the page by the row's last chunk; else, with the sum of dt, into the workspace)
    auto leave = [&]() {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            if (!live[c]) continue;
            const size_t r = ((size_t)b * pl.nC + chunk) * D;
            float* to = !OUT ? ws.hs + r * N : stp && t1 == len ? stp : nullptr;
#pragma unroll
            for (int n = 0; n < NS / 2; ++n) {
                if (to) *reinterpret_cast<uint64_t*>(to + cn0[c] + 2 * n) = h[c][n];
                if (GRAD) *reinterpret_cast<uint64_t*>(ws.mu + r * N + cn0[c] + 2 * n) = mu[c][n];
            }
            if (!OUT && part == 0) ws.sdt[r + c0 + ch[c]] = total_dt[c];
        }
    };
    auto next_chunk = [&]() {
        leave();
        ++chunk;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            total_dt[c] = 0.f;
#pragma unroll
            for (int n = 0; n < NS / 2; ++n) {
                h[c][n] = mu[GRAD ? c : 0][n] = 0ull;
                P[GRAD ? c : 0][n] = pack2(1.f, 1.f);
            }
        }
    };
    int slot = 0;
    for (int t = t0; t < t1; t += TT, slot ^= 1) {
        const int nt = min(TT, t1 - t);
        if (t == t0) __syncthreads();           // sbias
        arrive(slot);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const Pack<T, V> ru = sm.raw[slot][0][v][threadIdx.x], rd = sm.raw[slot][1][v][threadIdx.x];
            const Pack<float, V> bias = bias_of(sm.sbias[ev_c[v]]);
            float d[V + V % 2];
            if constexpr (V == 1) d[1] = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) d[e] = to_f(rd.v[e]) + bias.v[e];
#pragma unroll
            for (int e = 0; e < V; e += 2) softplus_2<T>(d[e], d[e + 1]);
#pragma unroll
            for (int e = 0; e < V; ++e)
                sm.sdt[ev_t[v]][e * CV + ev_c[v]] = make_float2(d[e], d[e] * to_f(ru.v[e]));
            if constexpr (GRAD) {
                const Pack<T, V> rz = sm.raw[slot][2][v][threadIdx.x], ro = sm.raw[slot][3][v][threadIdx.x];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float g = to_f(ro.v[e]);
                    if (z) g *= to_f(rz.v[e]) * sigmoid_f<T>(to_f(rz.v[e]));
                    sm.sg[ev_t[v]][e * CV + ev_c[v]] = g;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < S::NM; ++k)
#pragma unroll
            for (int i = 0; i < EB; ++i) {
                const int e = i * kScanThreads + threadIdx.x;
                if (e < BC) {
                    const Pack<T, BV> m = sm.rawbc[slot][k][i][threadIdx.x];
                    float* to = &sm.bc[k][0][0] + e * BV;
#pragma unroll
                    for (int x = 0; x < BV; ++x) to[x] = to_f(m.v[x]);
                }
            }
        __syncthreads();
        if constexpr (!S::ASYNC) fetch(t + TT, 0);
        int tt = 0;
        for (; tt + UN <= nt; tt += UN) {
            if (GRAD && t + tt == t0 + (chunk - rest / p.B * pl.per + 1) * pl.Lc) next_chunk();
            float y[UN * CH];
            tokens(tt, std::integral_constant<int, UN>(), y);
            if (OUT) {
#pragma unroll
                for (int k = 0; k < UN; k += GK) finish(tt + k, y + k * CH, nt);
            }
        }
        for (; tt < nt; tt += GK) {
            if (GRAD && t + tt == t0 + (chunk - rest / p.B * pl.per + 1) * pl.Lc) next_chunk();
            float y[GK * CH] = {};
#pragma unroll
            for (int k = 0; k < GK; ++k)
                if (tt + k < nt) tokens(tt + k, std::integral_constant<int, 1>(), y + k * CH);
            if (OUT) finish(tt, y, nt);
        }
        __syncthreads();
        if constexpr (OUT) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (ev_t[v] >= nt || ev_c[v] * V >= cn) continue;
                const Pack<T, V> ru = sm.raw[slot][0][v][threadIdx.x], rz = sm.raw[slot][S::NT - 1][v][threadIdx.x];
                const Pack<float, V> skip = bias_of(sm.sskip[ev_c[v]]);
                Pack<T, V> o;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float y = fmaf(skip.v[e], to_f(ru.v[e]), sm.sdt[ev_t[v]][e * CV + ev_c[v]].x);
                    if (z) {
                        const float zz = to_f(rz.v[e]);
                        y *= zz * sigmoid_f<T>(zz);
                    }
                    from_f(o.v[e], y);
                }
                *reinterpret_cast<Pack<T, V>*>(out + (size_t)(t + ev_t[v]) * D + ev_c[v] * V) = o;
            }
        }
        if constexpr (S::ASYNC) fetch(t + 2 * TT, slot);
    }
    if constexpr (S::ASYNC) copy_wait<0>();
    leave();
}

// Per (row, channel, state), in the chunks' order: ws.hs from each chunk's own end to
// its start, h <- decay of the chunk h + its own end, from the row's page (backward
// call: from zero); there also ws.mu, the chunks' order reversed, from what each hands
// on to what it is handed.  8 chunks' loads go ahead of the stores.
template <bool GRAD>
__global__ void __launch_bounds__(128) k_scan_chain(ScanArgs p, ScanPlan pl, ScanWs ws, int D, int N) {
    const int DN = D * N, nb = (DN + 127) / 128, b = blockIdx.x / nb, i = blockIdx.x % nb * 128 + threadIdx.x, c = i / N;
    const int page = !GRAD && p.state ? block_page(p.pg, b) : 0;
    const int used = (row_len(p.lens, b, p.L) + pl.Lc - 1) / pl.Lc;
    if (page < 0 || i >= DN) return;
    const float A = p.A[i] * kLog2e;
    const size_t r = (size_t)b * pl.nC;
    const float* sdt = ws.sdt + r * D + c;
    float h = !GRAD && p.state ? p.state[(size_t)page * DN + i] : 0.f, mu = 0.f;
    float *hs = ws.hs + r * DN + i, *ms = GRAD ? ws.mu + r * DN + i : nullptr;
    constexpr int K = 8;
    float e[K], s[K], f[K], w[K];   // chunks j0 .., and (backward call) used-1-j0, downwards
    auto fetch = [&](int j0) {
        // the last one's own end is not asked for, nor what the first hands back
        const int n = used - 1 - j0;
        const float *ph = hs + (size_t)j0 * DN, *ps = sdt + (size_t)j0 * D;
        const float *pm = GRAD ? ms + (size_t)max(n, 0) * DN : nullptr, *pw = sdt + (size_t)max(n, 0) * D;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            e[k] = k < n ? ph[k * DN] : 0.f;
            s[k] = k < n ? ps[k * D] : 0.f;
            if (GRAD) {
                f[k] = k < n ? pm[-k * DN] : 0.f;
                w[k] = k < n ? pw[-k * D] : 0.f;
            }
        }
    };
    fetch(0);
    for (int j0 = 0; j0 < used; j0 += K) {
        float e0[K], s0[K], f0[K], w0[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            e0[k] = e[k];
            s0[k] = ex2_approx(A * s[k]);
            if (GRAD) {
                f0[k] = f[k];
                w0[k] = ex2_approx(A * w[k]);
            }
        }
        fetch(j0 + K);
        float* ph = hs + (size_t)j0 * DN;
        float* pm = GRAD ? ms + (size_t)(used - 1 - j0) * DN : nullptr;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (j0 + k >= used) break;
            ph[k * DN] = h;
            h = fmaf(s0[k], h, e0[k]);
            if (GRAD) {
                pm[-k * DN] = mu;
                mu = fmaf(w0[k], mu, f0[k]);
            }
        }
    }
}

// One token a row.  A thread holds 4 states (16 bytes) of CH channels, LPC = N/4
// lanes a channel; what is done once a channel (dt, the gate, the output) is done
// by one lane each (213 instructions a thread of 4 states otherwise: 20 us instead of
// 14.4 for 256 rows of [2048, 16]).  Bound by the state, read and written once: its
// loads are issued before anything that waits; 5.0 TB/s.
template <typename T, int N>
__global__ void __launch_bounds__(kScanThreads) k_scan_step(ScanArgs p, int D, int G, int cblocks, bool wide) {
    constexpr int LPC = N / 4, CH = LPC < 4 ? LPC : 4, Q = kScanThreads / LPC;
    const int cb = blockIdx.x % cblocks, b = blockIdx.x / cblocks, part = threadIdx.x % LPC, q = threadIdx.x / LPC;
    const int c0 = cb * Q * CH + q, Dg = D / G;
    // the lane's own channel: the index that the sums over lanes below leave with it
    const int own = CH == 4 ? (part & 1) * 2 + (part >> 1 & 1) : part & 1;
    int page = row_page(p.pg, b);
    float* sp = p.state + ((size_t)(page < 0 ? 0 : page) * D + c0) * N + part * 4;
    const float* A = p.A + (size_t)c0 * N + part * 4;
    float4 h[CH], a[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const bool in = c0 + i * Q < D;
        h[i] = in ? *reinterpret_cast<const float4*>(sp + i * Q * N) : make_float4(0.f, 0.f, 0.f, 0.f);
        a[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (in && wide) a[i] = *reinterpret_cast<const float4*>(A + i * Q * N);
        if (in && !wide) a[i] = make_float4(A[i * Q * N], A[i * Q * N + 1], A[i * Q * N + 2], A[i * Q * N + 3]);
    }
    const int co = min(c0 + own * Q, D - 1);
    const size_t at = (size_t)b * D + co;
    const float uu = to_f(((const T*)p.u)[at]);
    const float raw = to_f(((const T*)p.dt)[at]) + (p.dt_bias ? p.dt_bias[co] : 0.f);
    const float zz = p.z ? to_f(((const T*)p.z)[at]) : 0.f;
    const float sk = p.skip ? p.skip[co] : 0.f;
    float bm[4], cm[4];
    auto load_bc = [&](int c) {
        const size_t bc = ((size_t)b * G + min(c, D - 1) / Dg) * N + part * 4;
        if (wide) {
            const Pack<T, 4> b4 = load_pack<T, 4>((const T*)p.Bm + bc), c4 = load_pack<T, 4>((const T*)p.Cm + bc);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                bm[k] = to_f(b4.v[k]);
                cm[k] = to_f(c4.v[k]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                bm[k] = to_f(((const T*)p.Bm)[bc + k]);
                cm[k] = to_f(((const T*)p.Cm)[bc + k]);
            }
        }
    };
    load_bc(c0);
    if (block_page_taken(p.pg, b, page)) page = -1;
    const bool mine = part < CH && c0 + own * Q < D;
    if (page < 0) {   // the row takes no part
        if (mine) from_f(((T*)p.out)[at], 0.f);
        return;
    }
    const float d = softplus_f<T>(raw), x = d * uu, dl = d * kLog2e;
    float y[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        if (i && G > 1) load_bc(c0 + i * Q);
        // the lane of this channel's group that holds channel i
        const int src = (threadIdx.x & 31 & ~(LPC - 1)) + (CH == 4 ? (i >> 1) + (i & 1) * 2 : i);
        const float di = __shfl_sync(0xffffffffu, dl, src), xi = __shfl_sync(0xffffffffu, x, src);
        h[i].x = fmaf(ex2_approx(fmaf(a[i].x, di, kEx2Mean)), h[i].x, xi * bm[0]);
        h[i].y = fmaf(ex2_approx(fmaf(a[i].y, di, kEx2Mean)), h[i].y, xi * bm[1]);
        h[i].z = fmaf(ex2_approx(fmaf(a[i].z, di, kEx2Mean)), h[i].z, xi * bm[2]);
        h[i].w = fmaf(ex2_approx(fmaf(a[i].w, di, kEx2Mean)), h[i].w, xi * bm[3]);
        if (c0 + i * Q < D) *reinterpret_cast<float4*>(sp + i * Q * N) = h[i];
        y[i] = fmaf(h[i].x, cm[0], h[i].y * cm[1]) + fmaf(h[i].z, cm[2], h[i].w * cm[3]);
    }
#pragma unroll
    for (int o = 1, w = CH / 2; o < LPC; o <<= 1, w >>= 1) {
        if (w) {
            const bool up = part & o;
#pragma unroll
            for (int i = 0; i < w; ++i) {
                const float keep = up ? y[i + w] : y[i], give = up ? y[i] : y[i + w];
                y[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
        } else {
            y[0] += __shfl_xor_sync(0xffffffffu, y[0], o);
        }
    }
    if (!mine) return;
    float v = fmaf(sk, uu, y[0]);
    if (p.z) v *= zz * sigmoid_f<T>(zz);
    from_f(((T*)p.out)[at], v);
}

// ------------------------------------------------------------------ launches
// Cutting the tokens into chunks fills the SMs, but runs every exponential of all
// but the last chunk twice: with room for 3 chunks or more it pays (1024 tokens,
// 192 blocks of channels: 205 us in 3 chunks, 227 uncut), with 2 it does not
// (256 blocks: 271 and 227 us).  A chunk is 32 tokens at least (12 blocks of 1000
// tokens: 26 us, 34 with 64).
constexpr int kScanMinChunk = 32;

static ScanPlan scan_plan(const SsmHandle& h, int B, int L, int CPB, int TT) {
    ScanPlan pl;
    pl.Dg = h.D / h.G;
    pl.tpg = (pl.Dg + CPB - 1) / CPB;
    pl.tiles = pl.tpg * h.G;
    long long want = (long long)h.num_sms * kScanPerSm / ((long long)pl.tiles * B);
    const int most = (L + kScanMinChunk - 1) / kScanMinChunk;
    if (want < 3) want = 1;
    if (want > most) want = most;
    pl.Lc = (int)((L + want - 1) / want);
    pl.Lc = (pl.Lc + TT - 1) / TT * TT;
    pl.nC = (L + pl.Lc - 1) / pl.Lc;
    pl.per = 1;
    return pl;
}

// Several chunks come only while tiles * B * chunks <= SMs * kScanPerSm; a tile has
// 128 * 16 states and at most 256 channels.
size_t scan_prompt_ws(const SsmHandle& h) {
    return (size_t)h.num_sms * kScanPerSm * (kScanThreads * kScanNS * kScanCH + 256);
}

template <typename T, int N, int V>
static void scan_launch(const SsmHandle& h, const ScanArgs& a, cudaStream_t st) {
    using S = ScanShared<T, N, V, SCAN_OUT>;
    const ScanPlan pl = scan_plan(h, a.B, a.L, S::CPB, S::TT);
    const ScanWs ws = {h.ws, h.ws + (size_t)a.B * pl.nC * h.D * N, nullptr};
    auto launch = [&](auto kernel, size_t smem, int chunks) {
        // the attribute's failure shows as the launch's
        if (smem > 48 * 1024) cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        kernel<<<(unsigned)pl.tiles * a.B * chunks, kScanThreads, smem, st>>>(a, pl, ws, h.D, h.G);
        count_launch();
    };
    if (pl.nC > 1) {
        launch(k_scan<T, N, V, SCAN_SUM>, sizeof(ScanShared<T, N, V, SCAN_SUM>), pl.nC - 1);
        k_scan_chain<false><<<(unsigned)((h.D * N + 127) / 128) * a.B, 128, 0, st>>>(a, pl, ws, h.D, N);
        count_launch();
    }
    launch(k_scan<T, N, V, SCAN_OUT>, sizeof(S), pl.nC);
}

// The chunk starts and incoming gradients of a backward call, into ws.hs and ws.mu.
template <typename T, int N, int V>
static void grad_launch(const SsmHandle& h, const ScanArgs& a, const ScanWs& ws, int Lc, cudaStream_t st) {
    using S = ScanShared<T, N, V, SCAN_GRAD>;
    ScanPlan pl;
    pl.Dg = h.D / h.G;
    pl.tpg = (pl.Dg + S::CPB - 1) / S::CPB;
    pl.tiles = pl.tpg * h.G;
    pl.Lc = Lc;
    pl.nC = (a.L + Lc - 1) / Lc;
    // Chunks a block: more, up to 256 tokens, while four waves of blocks remain (a block of one chunk
    // of 32 tokens: 2% slower at [4, 8192, 1024], 13% at N = 64, whose tile is 64 tokens)
    pl.per = 1;
    while (pl.per * Lc < 256 && (long long)pl.tiles * a.B * (pl.nC / pl.per) >= 4LL * h.num_sms * kScanPerSm) pl.per *= 2;
    cudaFuncSetAttribute(k_scan<T, N, V, SCAN_GRAD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(S));
    k_scan<T, N, V, SCAN_GRAD><<<(unsigned)pl.tiles * a.B * ((pl.nC + pl.per - 1) / pl.per), kScanThreads, sizeof(S), st>>>(a, pl, ws, h.D,
                                                                                                      h.G);
    k_scan_chain<true><<<(unsigned)((h.D * N + 127) / 128) * a.B, 128, 0, st>>>(a, pl, ws, h.D, N);
    count_launch(2);
}

template <typename T, int V>
static void grad_by_n(const SsmHandle& h, const ScanArgs& a, const ScanWs& ws, int Lc, cudaStream_t st) {
    if (h.N == 8) grad_launch<T, 8, V>(h, a, ws, Lc, st);
    else if (h.N == 16) grad_launch<T, 16, V>(h, a, ws, Lc, st);
    else if (h.N == 32) grad_launch<T, 32, V>(h, a, ws, Lc, st);
    else grad_launch<T, 64, V>(h, a, ws, Lc, st);
}

// 16-byte accesses need every row of a group to start on one (rows of B and C are N >= 8 elements).
static bool wide_rows(const SsmHandle& h, const ScanArgs& a) {
    const int v = h.dtype == FAVOR_DTYPE_F32 ? 4 : 8;
    for (const void* p : {a.u, a.dt, a.z, a.dout, a.Bm, a.Cm, (const void*)a.out, (const void*)a.du, (const void*)a.ddt,
                          (const void*)a.dz})
        if (!is_aligned16(p)) return false;
    return h.D % v == 0 && (h.D / h.G) % v == 0;
}

bool scan_grad_chunks(const SsmHandle& h, const ScanArgs& a, const ScanWs& ws, int Lc, cudaStream_t st) {
    const bool vec = wide_rows(h, a);
    if (h.dtype == FAVOR_DTYPE_F32 && vec) grad_by_n<float, 4>(h, a, ws, Lc, st);
    else if (h.dtype == FAVOR_DTYPE_F32) grad_by_n<float, 1>(h, a, ws, Lc, st);
    else if (vec) grad_by_n<__nv_bfloat16, 8>(h, a, ws, Lc, st);
    else grad_by_n<__nv_bfloat16, 1>(h, a, ws, Lc, st);
    return vec;
}

template <typename T, int V>
static void scan_by_n(const SsmHandle& h, const ScanArgs& a, cudaStream_t st) {
    if (h.N == 8) scan_launch<T, 8, V>(h, a, st);
    else if (h.N == 16) scan_launch<T, 16, V>(h, a, st);
    else if (h.N == 32) scan_launch<T, 32, V>(h, a, st);
    else scan_launch<T, 64, V>(h, a, st);
}

favor_status scan_prompt(const SsmHandle& h, const ScanArgs& a, cudaStream_t st) {
    const bool f32 = h.dtype == FAVOR_DTYPE_F32;
    const bool vec = wide_rows(h, a);
    if (f32 && vec) scan_by_n<float, 4>(h, a, st);
    else if (f32) scan_by_n<float, 1>(h, a, st);
    else if (vec) scan_by_n<__nv_bfloat16, 8>(h, a, st);
    else scan_by_n<__nv_bfloat16, 1>(h, a, st);
    return check_launch("favor_ssm_scan");
}

template <typename T, int N>
static void step_launch(const SsmHandle& h, const ScanArgs& a, cudaStream_t st) {
    const int per = kScanThreads / (N / 4) * (N / 4 < 4 ? N / 4 : 4), cb = (h.D + per - 1) / per;
    k_scan_step<T, N><<<(unsigned)cb * a.B, kScanThreads, 0, st>>>(
        a, h.D, h.G, cb, is_aligned16(a.A) && is_aligned16(a.Bm) && is_aligned16(a.Cm));
}

template <typename T>
static void step_by_n(const SsmHandle& h, const ScanArgs& a, cudaStream_t st) {
    if (h.N == 8) step_launch<T, 8>(h, a, st);
    else if (h.N == 16) step_launch<T, 16>(h, a, st);
    else if (h.N == 32) step_launch<T, 32>(h, a, st);
    else step_launch<T, 64>(h, a, st);
}

favor_status scan_step(const SsmHandle& h, const ScanArgs& a, cudaStream_t st) {
    if (h.dtype == FAVOR_DTYPE_F32) step_by_n<float>(h, a, st);
    else step_by_n<__nv_bfloat16>(h, a, st);
    count_launch();
    return check_launch("favor_ssm_scan_step");
}

}  // namespace favor
