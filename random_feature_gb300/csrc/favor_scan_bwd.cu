// Gradients of the selective scan from an empty start.  With g = dout silu(z)
// (the gradient of y) and lambda_t the gradient of the state h_t:
//     lambda_t = C_t g_t + a_{t+1} lambda_{t+1}
//     dC_t = sum_c g h_t            dB_t = sum_c lambda_t dt u
//     du = dt sum_n lambda B + skip g
//     q_n = lambda_n a_n h_{t-1,n}, ddt = u sum_n lambda B + sum_n A q,  draw = ddt sigmoid(raw + dt_bias)
//     dA_n = sum_t dt q_n           dskip = sum_t g u,  ddt_bias = sum_t draw,  dz = dout y silu'(z)
// The states are not kept by the forward call: they are formed again.
//
// Chunks of kBwdChunk tokens run in parallel.  k_bwd_summary gives each chunk's
// end from an empty start, its decay (sum of dt), and what it hands to the
// chunk before, a_first lambda_first from an empty end, as sum_t P_t C_t g_t with P_t
// the running product of a; k_bwd_chain turns these into every chunk's start
// state and incoming gradient; k_bwd_main walks a chunk forwards, keeping the
// state at every 8th token, then backwards in tiles, where 8 tokens' states
// and decays are held in registers.
#include "ssm_internal.h"

namespace favor {

constexpr int kBwdThreads = 128;
constexpr int kBwdChunk = 128;
constexpr int kBwdSub = 8;          // tokens whose states are in registers at a time
constexpr int kBwdTile = 16;        // tokens staged in shared memory at a time
constexpr int kBwdNS = 4;           // states a thread

struct BwdPlan {
    int tiles, tpg, Dg, nC;
};

struct BwdWs {
    float* hs;      // [B][nC][D][N] chunk ends, then chunk starts
    float* mu;      // [B][nC][D][N] gradients handed back by a chunk, then handed to it
    float* sdt;     // [B][nC][D]
    float* dA;      // [B][nC][D][N]
    float* dskip;   // [B][nC][D]
    float* dbias;   // [B][nC][D]
    float* bc;      // [tpg][B][L][G][2N] per channel tile: dB, dC
};

static BwdWs bwd_layout(float* ws, const BwdPlan& pl, int B, int L, int D, int N, int G, size_t* total) {
    BwdWs w;
    const size_t rows = (size_t)B * pl.nC;
    float* at = ws;
    w.hs = at; at += rows * D * N;
    w.mu = at; at += rows * D * N;
    w.dA = at; at += rows * D * N;
    w.bc = at; at += (size_t)pl.tpg * B * L * G * 2 * N;
    w.sdt = at; at += rows * D;
    w.dskip = at; at += rows * D;
    w.dbias = at; at += rows * D;
    *total = (size_t)(at - ws);
    return w;
}

static BwdPlan bwd_plan(const SsmHandle& h, int L) {
    BwdPlan pl;
    const int CPB = kBwdThreads * kBwdNS / h.N;
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

// Elements (tokens x channels) of a staged tile, V channels an access.
template <typename T, int N, int V, int TL>
struct Elems {
    static constexpr int CPB = kBwdThreads * kBwdNS / N;
    static constexpr int CV = CPB / V;
    static constexpr int NV = (TL * CPB / V + kBwdThreads - 1) / kBwdThreads;
};

template <typename T, int N, int V>
__global__ void __launch_bounds__(kBwdThreads) k_bwd_summary(ScanArgs p, BwdPlan pl, BwdWs ws, int D, int G) {
    using E = Elems<T, N, V, kBwdTile>;
    constexpr int NS = kBwdNS, LPC = N / NS, CPB = E::CPB;
    __shared__ float s_dt[kBwdTile][CPB], s_x[kBwdTile][CPB], s_g[kBwdTile][CPB];
    __shared__ __align__(16) float sB[kBwdTile][N], sC[kBwdTile][N];
    const int tile = blockIdx.x % pl.tiles, rest = blockIdx.x / pl.tiles;
    const int b = rest % p.B, chunk = rest / p.B;
    const int len = row_len(p.lens, b, p.L);
    const int t0 = chunk * kBwdChunk, t1 = min(t0 + kBwdChunk, len);
    if (t0 >= t1) return;
    const int g = tile / pl.tpg, cl = (tile % pl.tpg) * CPB, c0 = g * pl.Dg + cl, cn = min(CPB, pl.Dg - cl);
    const size_t row = (size_t)b * p.L;
    const int ch = threadIdx.x / LPC, part = threadIdx.x % LPC;
    const bool live = ch < cn;
    const size_t cn0 = (size_t)(c0 + (live ? ch : 0)) * N + part * NS;
    float A[NS], h[NS], mu[NS], P[NS], sum_dt = 0.f;
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        A[n] = p.A[cn0 + n] * kLog2e;
        h[n] = mu[n] = 0.f;
        P[n] = 1.f;
    }
    for (int t = t0; t < t1; t += kBwdTile) {
        const int nt = min(kBwdTile, t1 - t);
#pragma unroll
        for (int v = 0; v < E::NV; ++v) {
            const int i = v * kBwdThreads + threadIdx.x, tt = i / E::CV, c = i % E::CV * V;
            if (tt >= kBwdTile) continue;
            const bool ok = tt < nt && c < cn;
            const size_t at = (row + t + tt) * D + c0 + c;
            const Pack<T, V> ru = ok ? load_pack<T, V>((const T*)p.u + at) : zero_pack<T, V>();
            const Pack<T, V> rd = ok ? load_pack<T, V>((const T*)p.dt + at) : zero_pack<T, V>();
            const Pack<T, V> ro = ok ? load_pack<T, V>((const T*)p.dout + at) : zero_pack<T, V>();
            Pack<T, V> rz = zero_pack<T, V>();
            if (ok && p.z) rz = load_pack<T, V>((const T*)p.z + at);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float bias = ok && p.dt_bias && c + e < cn ? p.dt_bias[c0 + c + e] : 0.f;
                const float d = softplus_f(to_f(rd.v[e]) + bias);
                float gg = to_f(ro.v[e]);
                if (p.z) gg *= to_f(rz.v[e]) * sigmoid_f<T>(to_f(rz.v[e]));
                s_dt[tt][c + e] = d;
                s_x[tt][c + e] = d * to_f(ru.v[e]);
                s_g[tt][c + e] = gg;
            }
        }
        for (int i = threadIdx.x; i < kBwdTile * N; i += kBwdThreads) {
            const int tt = i / N, n = i % N;
            const size_t at = ((row + t + tt) * G + g) * N + n;
            sB[tt][n] = tt < nt ? to_f(((const T*)p.Bm)[at]) : 0.f;
            sC[tt][n] = tt < nt ? to_f(((const T*)p.Cm)[at]) : 0.f;
        }
        __syncthreads();
        for (int tt = 0; tt < nt; ++tt) {
            const float d = s_dt[tt][ch], x = s_x[tt][ch], gg = s_g[tt][ch];
            sum_dt += d;
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                const float a = ex2_approx(A[n] * d);
                h[n] = fmaf(a, h[n], x * sB[tt][part * NS + n]);
                P[n] *= a;
                mu[n] = fmaf(P[n], gg * sC[tt][part * NS + n], mu[n]);
            }
        }
        __syncthreads();
    }
    if (!live) return;
    const size_t r = ((size_t)b * pl.nC + chunk) * D;
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        ws.hs[r * N + cn0 + n] = h[n];
        ws.mu[r * N + cn0 + n] = mu[n];
    }
    if (part == 0) ws.sdt[r + c0 + ch] = sum_dt;
}

// Per (row, channel, state): chunk ends -> chunk starts, forwards; what chunks hand
// back -> what each is handed, backwards.
__global__ void __launch_bounds__(256) k_bwd_chain(ScanArgs p, BwdPlan pl, BwdWs ws, int D, int N) {
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x, DN = (size_t)D * N;
    if (i >= (size_t)p.B * DN) return;
    const int b = (int)(i / DN);
    const size_t cn = i % DN;
    const int c = (int)(cn / N);
    const int used = (row_len(p.lens, b, p.L) + kBwdChunk - 1) / kBwdChunk;
    const float A = p.A[cn] * kLog2e;
    const size_t r0 = (size_t)b * pl.nC;
    float h = 0.f;
#pragma unroll 8
    for (int j = 0; j < used; ++j) {
        float* at = ws.hs + (r0 + j) * DN + cn;
        const float e = *at, s = ws.sdt[(r0 + j) * D + c];
        *at = h;
        h = fmaf(ex2_approx(A * s), h, e);
    }
    float mu = 0.f;
#pragma unroll 8
    for (int j = used - 1; j >= 0; --j) {
        float* at = ws.mu + (r0 + j) * DN + cn;
        const float e = *at, s = ws.sdt[(r0 + j) * D + c];
        *at = mu;
        mu = fmaf(ex2_approx(A * s), mu, e);
    }
}

// Sums v[0..W) over the lanes that differ in the bits of lane at and above
// `bit`: while more than one value is left each step halves the values a lane
// holds (a lane with the bit set keeps the upper half), then plain butterflies.
// On return v[0] (.. v[W / lanes)) of a lane holds its share.
template <int W, int BIT>
struct LaneSum {
    static __device__ __forceinline__ void go(float* v) {
        if constexpr (BIT < 32) {
            if constexpr (W > 1) {
                const bool up = threadIdx.x & BIT;
#pragma unroll
                for (int i = 0; i < W / 2; ++i) {
                    const float keep = up ? v[i + W / 2] : v[i], give = up ? v[i] : v[i + W / 2];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, give, BIT);
                }
                LaneSum<W / 2, BIT * 2>::go(v);
            } else {
                v[0] += __shfl_xor_sync(0xffffffffu, v[0], BIT);
                LaneSum<1, BIT * 2>::go(v);
            }
        }
    }
};

template <typename T, int N, int V>
__global__ void __launch_bounds__(kBwdThreads) k_bwd_main(ScanArgs p, BwdPlan pl, BwdWs ws, int D, int G) {
    using E = Elems<T, N, V, kBwdTile>;
    constexpr int NS = kBwdNS, LPC = N / NS, CPB = E::CPB, CW = 32 / LPC, W = kBwdThreads / 32;
    // values of dB | dC (4 + 4 a lane) left with a lane after the sum over its warp's channels
    constexpr int LEFT = CW >= 8 ? 1 : 8 / CW;
    extern __shared__ __align__(16) unsigned char smem[];
    float4* keep = reinterpret_cast<float4*>(smem);                       // [chunk / sub][threads]
    typedef float Row[CPB];
    Row* s_dt = reinterpret_cast<Row*>(keep + (size_t)(kBwdChunk / kBwdSub) * kBwdThreads);   // [tile] -> lb
    Row* s_u = s_dt + kBwdTile;                                           // -> sum A q
    Row* s_g = s_u + kBwdTile;                                            // -> y
    typedef float NRow[N];
    NRow* sB = reinterpret_cast<NRow*>(s_g + kBwdTile);
    NRow* sC = sB + kBwdTile;
    float* red = reinterpret_cast<float*>(sC + kBwdTile);                 // [W][tile][2N]

    const int tile = blockIdx.x % pl.tiles, rest = blockIdx.x / pl.tiles;
    const int b = rest % p.B, chunk = rest / p.B;
    const int len = row_len(p.lens, b, p.L);
    const int t0 = chunk * kBwdChunk, t1 = min(t0 + kBwdChunk, len);
    const int g = tile / pl.tpg, cl = (tile % pl.tpg) * CPB, c0 = g * pl.Dg + cl, cn = min(CPB, pl.Dg - cl);
    const size_t row = (size_t)b * p.L, wr = ((size_t)b * pl.nC + chunk) * D;
    const int ch = threadIdx.x / LPC, part = threadIdx.x % LPC, warp = threadIdx.x / 32;
    const bool live = ch < cn;
    const size_t cn0 = (size_t)(c0 + (live ? ch : 0)) * N + part * NS;
    if (t0 >= t1) {   // behind the row's end: nothing but zeros for the sums over rows
        if (live) {
#pragma unroll
            for (int n = 0; n < NS; ++n) ws.dA[wr * N + cn0 + n] = 0.f;
            if (part == 0) ws.dskip[wr + c0 + ch] = ws.dbias[wr + c0 + ch] = 0.f;
        }
        return;
    }
    float A[NS], h[NS], mu[NS], dA[NS];
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        A[n] = p.A[cn0 + n] * kLog2e;
        h[n] = ws.hs[wr * N + cn0 + n];
        mu[n] = ws.mu[wr * N + cn0 + n];
        dA[n] = 0.f;
    }
    Pack<T, V> ru[E::NV], rd[E::NV], ro[E::NV], rz[E::NV];
    float acc_skip[E::NV][V], acc_bias[E::NV][V];
#pragma unroll
    for (int v = 0; v < E::NV; ++v)
#pragma unroll
        for (int e = 0; e < V; ++e) acc_skip[v][e] = acc_bias[v][e] = 0.f;

    // stage tokens t .. t+15: dt, u (forward walk), and g, B, C
    auto stage = [&](int t, int nt, bool back) {
#pragma unroll
        for (int v = 0; v < E::NV; ++v) {
            const int i = v * kBwdThreads + threadIdx.x, tt = i / E::CV, c = i % E::CV * V;
            if (tt >= kBwdTile) continue;
            const bool ok = tt < nt && c < cn;
            const size_t at = (row + t + tt) * D + c0 + c;
            ru[v] = ok ? load_pack<T, V>((const T*)p.u + at) : zero_pack<T, V>();
            rd[v] = ok ? load_pack<T, V>((const T*)p.dt + at) : zero_pack<T, V>();
            if (back) {
                ro[v] = ok ? load_pack<T, V>((const T*)p.dout + at) : zero_pack<T, V>();
                rz[v] = ok && p.z ? load_pack<T, V>((const T*)p.z + at) : zero_pack<T, V>();
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float bias = ok && p.dt_bias && c + e < cn ? p.dt_bias[c0 + c + e] : 0.f;
                s_dt[tt][c + e] = softplus_f(to_f(rd[v].v[e]) + bias);
                s_u[tt][c + e] = to_f(ru[v].v[e]);
                if (back) {
                    float gg = to_f(ro[v].v[e]);
                    if (p.z) gg *= to_f(rz[v].v[e]) * sigmoid_f<T>(to_f(rz[v].v[e]));
                    s_g[tt][c + e] = gg;
                }
            }
        }
        for (int i = threadIdx.x; i < kBwdTile * N; i += kBwdThreads) {
            const int tt = i / N, n = i % N;
            const size_t at = ((row + t + tt) * G + g) * N + n;
            sB[tt][n] = tt < nt ? to_f(((const T*)p.Bm)[at]) : 0.f;
            if (back) sC[tt][n] = tt < nt ? to_f(((const T*)p.Cm)[at]) : 0.f;
        }
    };

    // forwards: the state at the start of every 8 tokens
    for (int t = t0; t < t1; t += kBwdTile) {
        const int nt = min(kBwdTile, t1 - t);
        stage(t, nt, false);
        __syncthreads();
        for (int tt = 0; tt < nt; ++tt) {
            if (tt % kBwdSub == 0)
                keep[(size_t)((t - t0 + tt) / kBwdSub) * kBwdThreads + threadIdx.x] = make_float4(h[0], h[1], h[2], h[3]);
            const float d = s_dt[tt][ch], x = d * s_u[tt][ch];
#pragma unroll
            for (int n = 0; n < NS; ++n) h[n] = fmaf(ex2_approx(A[n] * d), h[n], x * sB[tt][part * NS + n]);
        }
        __syncthreads();
    }
    // backwards
    for (int t = t0 + (t1 - 1 - t0) / kBwdTile * kBwdTile; t >= t0; t -= kBwdTile) {
        const int nt = min(kBwdTile, t1 - t);
        stage(t, nt, true);
        __syncthreads();
        for (int s0 = (nt - 1) / kBwdSub * kBwdSub; s0 >= 0; s0 -= kBwdSub) {
            const int ns = min(kBwdSub, nt - s0);
            float a[kBwdSub][NS], hp[kBwdSub][NS], hc[NS];
            const float4 k4 = keep[(size_t)((t - t0 + s0) / kBwdSub) * kBwdThreads + threadIdx.x];
            hc[0] = k4.x; hc[1] = k4.y; hc[2] = k4.z; hc[3] = k4.w;
#pragma unroll
            for (int k = 0; k < kBwdSub; ++k) {
                if (k < ns) {
                    const float d = s_dt[s0 + k][ch], x = d * s_u[s0 + k][ch];
#pragma unroll
                    for (int n = 0; n < NS; ++n) {
                        a[k][n] = ex2_approx(A[n] * d);
                        hp[k][n] = hc[n];
                        hc[n] = fmaf(a[k][n], hc[n], x * sB[s0 + k][part * NS + n]);
                    }
                }
            }
#pragma unroll
            for (int k = kBwdSub - 1; k >= 0; --k) {
                if (k < ns) {
                    const int tt = s0 + k;
                    const float d = s_dt[tt][ch], uu = s_u[tt][ch], gg = s_g[tt][ch], x = d * uu;
                    float y = 0.f, lb = 0.f, aq = 0.f, v[8];
#pragma unroll
                    for (int n = 0; n < NS; ++n) {
                        const float Bn = sB[tt][part * NS + n], Cn = sC[tt][part * NS + n];
                        const float lam = fmaf(Cn, gg, mu[n]);
                        y = fmaf(hc[n], Cn, y);
                        lb = fmaf(lam, Bn, lb);
                        v[n] = live ? lam * x : 0.f;
                        v[4 + n] = live ? gg * hc[n] : 0.f;
                        mu[n] = a[k][n] * lam;
                        const float q = mu[n] * hp[k][n];
                        aq = fmaf(q, A[n], aq);
                        dA[n] = fmaf(q, d, dA[n]);
                        hc[n] = hp[k][n];
                    }
#pragma unroll
                    for (int o = 1; o < LPC; o <<= 1) {
                        y += __shfl_xor_sync(0xffffffffu, y, o);
                        lb += __shfl_xor_sync(0xffffffffu, lb, o);
                        aq += __shfl_xor_sync(0xffffffffu, aq, o);
                    }
                    if (part == 0) {
                        s_dt[tt][ch] = lb;
                        s_u[tt][ch] = aq * 0.6931471805599453f;   // A was scaled by log2 e
                        s_g[tt][ch] = y;
                    }
                    LaneSum<8, LPC>::go(v);
                    // the index of v[i]: dB or dC, state n, from the lane bits that chose the halves
                    const int cb = (threadIdx.x % 32) / LPC;
                    float* rr = red + ((size_t)warp * kBwdTile + tt) * 2 * N;
                    const int first = (cb & 1 ? 4 : 0) + (CW > 2 && (cb & 2) ? 2 : 0) + (CW > 4 && (cb & 4) ? 1 : 0);
                    if (CW <= 8 || cb < 8) {
#pragma unroll
                        for (int i = 0; i < LEFT; ++i) {
                            const int j = first + i;
                            rr[(j >= 4 ? N : 0) + part * NS + (j & 3)] = v[i];
                        }
                    }
                }
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < nt * 2 * N; i += kBwdThreads) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) s += red[(size_t)w * kBwdTile * 2 * N + i];
            const int tt = i / (2 * N), j = i % (2 * N);
            ws.bc[((((size_t)(tile % pl.tpg) * p.B + b) * p.L + t + tt) * G + g) * 2 * N + j] = s;
        }
#pragma unroll
        for (int v = 0; v < E::NV; ++v) {
            const int i = v * kBwdThreads + threadIdx.x, tt = i / E::CV, c = i % E::CV * V;
            if (tt >= nt || c >= cn) continue;
            Pack<T, V> ou, od, oz;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int cc = c0 + c + e;
                const float raw = to_f(rd[v].v[e]) + (p.dt_bias ? p.dt_bias[cc] : 0.f), sk = p.skip ? p.skip[cc] : 0.f;
                const float d = softplus_f(raw), uu = to_f(ru[v].v[e]), oo = to_f(ro[v].v[e]);
                const float lb = s_dt[tt][c + e], aq = s_u[tt][c + e];
                float gg = oo;
                if (p.z) {
                    const float zz = to_f(rz[v].v[e]), sg = sigmoid_f<T>(zz);
                    gg *= zz * sg;
                    from_f(oz.v[e], oo * fmaf(sk, uu, s_g[tt][c + e]) * (sg * (1.f + zz * (1.f - sg))));
                }
                from_f(ou.v[e], fmaf(d, lb, sk * gg));
                const float dr = fmaf(uu, lb, aq) / (1.f + expf(-raw));
                from_f(od.v[e], dr);
                acc_skip[v][e] = fmaf(gg, uu, acc_skip[v][e]);
                acc_bias[v][e] += dr;
            }
            const size_t at = (row + t + tt) * D + c0 + c;
            *reinterpret_cast<Pack<T, V>*>((T*)p.du + at) = ou;
            *reinterpret_cast<Pack<T, V>*>((T*)p.ddt + at) = od;
            if (p.z) *reinterpret_cast<Pack<T, V>*>((T*)p.dz + at) = oz;
        }
        __syncthreads();
    }
    if (live) {
#pragma unroll
        for (int n = 0; n < NS; ++n) ws.dA[wr * N + cn0 + n] = dA[n];
    }
    // dskip, ddt_bias of the chunk: the element lanes' sums, added per channel in a fixed order
    float* s_a = reinterpret_cast<float*>(keep);   // [tile rows][CPB], the kept states are done with
    float* s_b = s_a + kBwdTile * CPB;
#pragma unroll
    for (int v = 0; v < E::NV; ++v) {
        const int i = v * kBwdThreads + threadIdx.x, tt = i / E::CV, c = i % E::CV * V;
        if (tt >= kBwdTile) continue;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            s_a[tt * CPB + c + e] = acc_skip[v][e];
            s_b[tt * CPB + c + e] = acc_bias[v][e];
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < cn; c += kBwdThreads) {
        float sa = 0.f, sb = 0.f;
#pragma unroll
        for (int tt = 0; tt < kBwdTile; ++tt) {
            sa += s_a[tt * CPB + c];
            sb += s_b[tt * CPB + c];
        }
        ws.dskip[wr + c0 + c] = sa;
        ws.dbias[wr + c0 + c] = sb;
    }
}

// dB, dC: the channel tiles' parts, in order, rounded once.  Rows behind a
// sequence's end are left as they were.
template <typename T>
__global__ void __launch_bounds__(256) k_bwd_bc(ScanArgs p, BwdPlan pl, BwdWs ws, int N, int G) {
    const size_t n = (size_t)p.B * p.L * G * 2 * N, i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const size_t tg = i / (2 * N);
    const int j = (int)(i % (2 * N)), t = (int)(tg / G % p.L), b = (int)(tg / G / p.L);
    if (t >= row_len(p.lens, b, p.L)) return;
    float s = 0.f;
    for (int k = 0; k < pl.tpg; ++k) s += ws.bc[k * n + i];
    T* o = j < N ? (T*)p.dB + tg * N + j : (T*)p.dC + tg * N + j - N;
    from_f(*o, s);
}

// Sums of the parameters' gradients over the chunks of every row.
__global__ void __launch_bounds__(256) k_bwd_params(ScanArgs p, BwdWs ws, int rows, int D, int N) {
    __shared__ float s[8][33];
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
    const size_t DN = (size_t)D * N, all = DN + 2 * D, i = (size_t)blockIdx.x * 32 + lane;
    const float* src = i < DN ? ws.dA + i : i < DN + D ? ws.dskip + (i - DN) : ws.dbias + (i - DN - D);
    const size_t step = i < DN ? DN : D;
    float acc = 0.f;
    if (i < all)
        for (int r = y; r < rows; r += 8) acc += src[r * step];
    s[y][lane] = acc;
    __syncthreads();
    if (y || i >= all) return;
#pragma unroll
    for (int k = 1; k < 8; ++k) acc += s[k][lane];
    if (i < DN) p.dA[i] = acc;
    else if (i < DN + D) { if (p.dskip) p.dskip[i - DN] = acc; }
    else if (p.ddt_bias) p.ddt_bias[i - DN - D] = acc;
}

template <typename T, int N, int V>
static favor_status bwd_launch(const SsmHandle& h, const ScanArgs& a, cudaStream_t st) {
    const BwdPlan pl = bwd_plan(h, a.L);
    size_t total = 0;
    const BwdWs ws = bwd_layout(h.ws, pl, a.B, a.L, h.D, N, h.G, &total);
    const unsigned grid = (unsigned)pl.tiles * a.B * pl.nC;
    constexpr int CPB = Elems<T, N, V, kBwdTile>::CPB;
    const size_t smem = (size_t)(kBwdChunk / kBwdSub) * kBwdThreads * 16 + 3 * kBwdTile * CPB * 4 +
                        2 * kBwdTile * N * 4 + (size_t)(kBwdThreads / 32) * kBwdTile * 2 * N * 4;
    if (cudaFuncSetAttribute(k_bwd_main<T, N, V>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return check_launch("favor_ssm_scan_backward");
    k_bwd_summary<T, N, V><<<grid, kBwdThreads, 0, st>>>(a, pl, ws, h.D, h.G);
    const size_t chain = (size_t)a.B * h.D * N;
    k_bwd_chain<<<(unsigned)((chain + 255) / 256), 256, 0, st>>>(a, pl, ws, h.D, N);
    k_bwd_main<T, N, V><<<grid, kBwdThreads, smem, st>>>(a, pl, ws, h.D, h.G);
    const size_t bc = (size_t)a.B * a.L * h.G * 2 * N;
    k_bwd_bc<T><<<(unsigned)((bc + 255) / 256), 256, 0, st>>>(a, pl, ws, N, h.G);
    const size_t par = (size_t)h.D * (N + 2);
    k_bwd_params<<<(unsigned)((par + 31) / 32), 256, 0, st>>>(a, ws, a.B * pl.nC, h.D, N);
    count_launch(5);
    return check_launch("favor_ssm_scan_backward");
}

template <typename T, int V>
static favor_status bwd_by_n(const SsmHandle& h, const ScanArgs& a, cudaStream_t st) {
    if (h.N == 8) return bwd_launch<T, 8, V>(h, a, st);
    if (h.N == 16) return bwd_launch<T, 16, V>(h, a, st);
    if (h.N == 32) return bwd_launch<T, 32, V>(h, a, st);
    return bwd_launch<T, 64, V>(h, a, st);
}

favor_status scan_backward(const SsmHandle& h, const ScanArgs& a, cudaStream_t st) {
    const bool f32 = h.dtype == FAVOR_DTYPE_F32;
    const int v = 4;
    const bool vec = h.D % v == 0 && (h.D / h.G) % v == 0 && is_aligned16(a.u) && is_aligned16(a.dt) &&
                     is_aligned16(a.z) && is_aligned16(a.dout) && is_aligned16(a.du) && is_aligned16(a.ddt) &&
                     is_aligned16(a.dz);
    if (f32 && vec) return bwd_by_n<float, 4>(h, a, st);
    if (f32) return bwd_by_n<float, 1>(h, a, st);
    if (vec) return bwd_by_n<__nv_bfloat16, 4>(h, a, st);
    return bwd_by_n<__nv_bfloat16, 1>(h, a, st);
}

}  // namespace favor
