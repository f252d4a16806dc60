// Selective state space scan, per channel c with N states (the state is decayed
// by a rate that depends on the token):
//     dt = softplus(raw + dt_bias),  a_n = exp(dt A_n),  h_n <- a_n h_n + dt u B_n,
//     y = sum_n C_n h_n + skip u,    out = y silu(z)
// u, raw, z, out are [B, L, D]; B and C [B, L, G, N], group g serving the channels
// g D/G .. (g+1) D/G - 1.  States and every sum are fp32.
#include "ssm_internal.h"

namespace favor {

constexpr int kScanThreads = 128;

// Two floats in one 64-bit register pair: the packed FMA / MUL issue two states'
// arithmetic in one slot.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t ex2_2(uint64_t v) {
    float lo, hi;
    unpack2(v, lo, hi);
    return pack2(ex2_approx(lo), ex2_approx(hi));
}

// How a launch cuts channels and tokens.  A block is 128 threads over CPB
// channels of one group of one row, LPC = N / NS lanes a channel (NS states in
// each lane's registers), for one chunk of tokens, walked in tiles of 8 LPC.
struct ScanPlan {
    int tiles;     // channel tiles a row (over all groups)
    int tpg;       // channel tiles a group
    int Dg;        // channels a group
    int nC, Lc;    // chunks, tokens a chunk
};

// Chunk summaries in the workspace: for chunk j, the state it would end with from
// an empty start, and the sum of its dt (whose exponential decays the start).
struct ScanWs {
    float* hend;   // [B][nC][D][N]
    float* sdt;    // [B][nC][D]
    float* h0;     // [B][D][N] the rows' own starts (the last chunk writes the page that they came from)
};

// SUMMARY: the first pass of a call with several chunks, every chunk but the last
// of a row from an empty state, without C, z or outputs.  Otherwise the pass that
// writes the outputs; a chunk's start is folded from the summaries before it.
template <typename T, int N, int NS, int V, bool SUMMARY>
__global__ void __launch_bounds__(kScanThreads)
k_scan(ScanArgs p, ScanPlan pl, ScanWs ws, int D, int G) {
    constexpr int LPC = N / NS, CPB = kScanThreads / LPC, TT = 8 * LPC, NV = 8 / V, CV = CPB / V;
    constexpr int EB = TT * N / kScanThreads > 0 ? TT * N / kScanThreads : 1;
    __shared__ float2 sdt[TT][CPB];             // (dt, dt u); .x becomes y
    __shared__ __align__(16) float sB[TT][N];
    __shared__ __align__(16) float sC[TT][N];

    const int tile = blockIdx.x % pl.tiles, rest = blockIdx.x / pl.tiles;
    const int b = rest % p.B, chunk = rest / p.B;
    const int len = row_len(p.lens, b, p.L);
    const int t0 = chunk * pl.Lc, t1 = min(t0 + pl.Lc, len);
    if (t0 >= t1 || (SUMMARY && t1 == len)) return;
    const int page = p.state ? block_page(p.pg, b) : 0;
    const int g = tile / pl.tpg, cl = (tile % pl.tpg) * CPB, c0 = g * pl.Dg + cl, cn = min(CPB, pl.Dg - cl);
    const size_t row = (size_t)b * p.L;
    const T* u = (const T*)p.u + row * D + c0;
    const T* dt = (const T*)p.dt + row * D + c0;
    const T* z = p.z && !SUMMARY ? (const T*)p.z + row * D + c0 : nullptr;
    T* out = (T*)p.out + row * D + c0;
    if (page < 0) {   // the row takes no part
        if (!SUMMARY)
            for (int i = threadIdx.x; i < (t1 - t0) * cn; i += kScanThreads)
                from_f(out[(size_t)(t0 + i / cn) * D + i % cn], 0.f);
        return;
    }
    const T* Bm = (const T*)p.Bm + (row * G + g) * N;
    const T* Cm = (const T*)p.Cm + (row * G + g) * N;

    // state lanes: channel ch, states part*NS .. +NS-1
    const int ch = threadIdx.x / LPC, part = threadIdx.x % LPC;
    const bool live = ch < cn;
    uint64_t A2[NS / 2], h[NS / 2];
    const size_t cn0 = (size_t)(c0 + (live ? ch : 0)) * N + part * NS;
#pragma unroll
    for (int n = 0; n < NS / 2; ++n)
        A2[n] = pack2(p.A[cn0 + 2 * n] * kLog2e, p.A[cn0 + 2 * n + 1] * kLog2e);
    float* stp = p.state ? p.state + (size_t)page * D * N + cn0 : nullptr;
#pragma unroll
    for (int n = 0; n < NS / 2; ++n)
        h[n] = stp && chunk == 0 && (SUMMARY || t1 == len) ? *reinterpret_cast<const uint64_t*>(stp + 2 * n) : 0ull;
    if (SUMMARY && stp && chunk == 0) {
#pragma unroll
        for (int n = 0; n < NS / 2; ++n)
            if (live) *reinterpret_cast<uint64_t*>(ws.h0 + (size_t)b * D * N + cn0 + 2 * n) = h[n];
    }
    if (!SUMMARY && stp && chunk == 0 && t1 < len) {
#pragma unroll
        for (int n = 0; n < NS / 2; ++n) h[n] = *reinterpret_cast<const uint64_t*>(ws.h0 + (size_t)b * D * N + cn0 + 2 * n);
    }
    if (!SUMMARY && chunk > 0) {
        // the chunks before, from the row's start (which chunk 0's end holds already)
#pragma unroll 4
        for (int j = 0; j < chunk; ++j) {
            const size_t r = ((size_t)b * pl.nC + j) * D;
            const float s = ws.sdt[r + c0 + (live ? ch : 0)];
            const uint64_t s2 = pack2(s, s);
#pragma unroll
            for (int n = 0; n < NS / 2; ++n) {
                const uint64_t e = *reinterpret_cast<const uint64_t*>(ws.hend + r * N + cn0 + 2 * n);
                h[n] = fma2(ex2_2(mul2(A2[n], s2)), h[n], e);
            }
        }
    }
    float total_dt = 0.f;

    // element lanes: vector v is V channels of one token of the tile
    int ev_t[NV], ev_c[NV];
    float bias[NV][V], skip[NV][V];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int i = v * kScanThreads + threadIdx.x;
        ev_t[v] = i / CV;
        ev_c[v] = i % CV * V;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const bool ok = ev_c[v] + e < cn;
            bias[v][e] = ok && p.dt_bias ? p.dt_bias[c0 + ev_c[v] + e] : 0.f;
            skip[v][e] = ok && p.skip && !SUMMARY ? p.skip[c0 + ev_c[v] + e] : 0.f;
        }
    }
    Pack<T, V> ru[NV], rd[NV], rz[NV];
    T rB[EB], rC[EB];
    auto fetch = [&](int t) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const bool ok = t + ev_t[v] < t1 && ev_c[v] < cn;
            const size_t at = (size_t)(t + ev_t[v]) * D + ev_c[v];
            ru[v] = ok ? load_pack<T, V>(u + at) : zero_pack<T, V>();
            rd[v] = ok ? load_pack<T, V>(dt + at) : zero_pack<T, V>();
            if (!SUMMARY) rz[v] = ok && z ? load_pack<T, V>(z + at) : zero_pack<T, V>();
        }
#pragma unroll
        for (int i = 0; i < EB; ++i) {
            const int e = i * kScanThreads + threadIdx.x, tt = e / N, n = e % N;
            const bool ok = tt < TT && t + tt < t1;
            const size_t at = (size_t)(t + tt) * G * N + n;
            from_f(rB[i], 0.f);
            from_f(rC[i], 0.f);
            if (ok) rB[i] = Bm[at];
            if (ok && !SUMMARY) rC[i] = Cm[at];
        }
    };
    fetch(t0);
    for (int t = t0; t < t1; t += TT) {
        const int nt = min(TT, t1 - t);
        Pack<T, V> cu[NV], cz[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = softplus_f(to_f(rd[v].v[e]) + bias[v][e]);
                sdt[ev_t[v]][ev_c[v] + e] = make_float2(d, d * to_f(ru[v].v[e]));
            }
            cu[v] = ru[v];
            cz[v] = rz[v];
        }
#pragma unroll
        for (int i = 0; i < EB; ++i) {
            const int e = i * kScanThreads + threadIdx.x, tt = e / N, n = e % N;
            if (tt < TT) {
                sB[tt][n] = to_f(rB[i]);
                if (!SUMMARY) sC[tt][n] = to_f(rC[i]);
            }
        }
        __syncthreads();
        if (t + TT < t1) fetch(t + TT);
#pragma unroll 4
        for (int tt = 0; tt < nt; ++tt) {
            const float2 dd = sdt[tt][ch];
            const uint64_t d2 = pack2(dd.x, dd.x), x2 = pack2(dd.y, dd.y);
            uint64_t y2 = 0;
            const ulonglong2* B2 = reinterpret_cast<const ulonglong2*>(&sB[tt][part * NS]);
            const ulonglong2* C2 = reinterpret_cast<const ulonglong2*>(&sC[tt][part * NS]);
#pragma unroll
            for (int n = 0; n < NS / 4; ++n) {
                const ulonglong2 bb = B2[n];
                h[2 * n] = fma2(ex2_2(mul2(A2[2 * n], d2)), h[2 * n], mul2(x2, bb.x));
                h[2 * n + 1] = fma2(ex2_2(mul2(A2[2 * n + 1], d2)), h[2 * n + 1], mul2(x2, bb.y));
                if (!SUMMARY) {
                    const ulonglong2 cc = C2[n];
                    y2 = fma2(h[2 * n], cc.x, y2);
                    y2 = fma2(h[2 * n + 1], cc.y, y2);
                }
            }
            if (SUMMARY) {
                total_dt += dd.x;
            } else {
                float y0, y1;
                unpack2(y2, y0, y1);
                float y = y0 + y1;
#pragma unroll
                for (int o = 1; o < LPC; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
                if (part == 0) sdt[tt][ch].x = y;
            }
        }
        __syncthreads();
        if (!SUMMARY) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (ev_t[v] >= nt || ev_c[v] >= cn) continue;
                Pack<T, V> o;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float y = fmaf(skip[v][e], to_f(cu[v].v[e]), sdt[ev_t[v]][ev_c[v] + e].x);
                    if (z) {
                        const float zz = to_f(cz[v].v[e]);
                        y *= zz * sigmoid_f<T>(zz);
                    }
                    from_f(o.v[e], y);
                }
                *reinterpret_cast<Pack<T, V>*>(out + (size_t)(t + ev_t[v]) * D + ev_c[v]) = o;
            }
        }
    }
    if (!live) return;
    if (SUMMARY) {
        const size_t r = ((size_t)b * pl.nC + chunk) * D;
#pragma unroll
        for (int n = 0; n < NS / 2; ++n) *reinterpret_cast<uint64_t*>(ws.hend + r * N + cn0 + 2 * n) = h[n];
        if (part == 0) ws.sdt[r + c0 + ch] = total_dt;
    } else if (stp && t1 == len) {
#pragma unroll
        for (int n = 0; n < NS / 2; ++n) *reinterpret_cast<uint64_t*>(stp + 2 * n) = h[n];
    }
}

// One token a row: a thread holds 4 states (16 bytes) of a channel, N/4 lanes a
// channel.  Bound by the state, read and written once.
template <typename T, int N>
__global__ void __launch_bounds__(kScanThreads) k_scan_step(ScanArgs p, int D, int G, int cblocks) {
    constexpr int LPC = N / 4;
    const int cb = blockIdx.x % cblocks, b = blockIdx.x / cblocks;
    const int i = cb * kScanThreads + threadIdx.x, c = i / LPC, part = i % LPC;
    const bool in = c < D;
    const int cc = in ? c : 0, g = cc / (D / G);
    const float* A = p.A + (size_t)cc * N + part * 4;
    const float a0 = A[0], a1 = A[1], a2 = A[2], a3 = A[3];
    const T* Bm = (const T*)p.Bm + ((size_t)b * G + g) * N + part * 4;
    const T* Cm = (const T*)p.Cm + ((size_t)b * G + g) * N + part * 4;
    float bm[4], cm[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) { bm[k] = to_f(Bm[k]); cm[k] = to_f(Cm[k]); }
    const size_t at = (size_t)b * D + cc;
    const float uu = to_f(((const T*)p.u)[at]);
    const float raw = to_f(((const T*)p.dt)[at]) + (p.dt_bias ? p.dt_bias[cc] : 0.f);
    const float zz = p.z ? to_f(((const T*)p.z)[at]) : 0.f;
    const float sk = p.skip ? p.skip[cc] : 0.f;
    const int page = block_page(p.pg, b);
    if (page < 0) {   // the row takes no part
        if (in && part == 0) from_f(((T*)p.out)[at], 0.f);
        return;
    }
    float4* sp = reinterpret_cast<float4*>(p.state + ((size_t)page * D + cc) * N + part * 4);
    float4 h = *sp;
    const float d = softplus_f(raw), x = d * uu, dl = d * kLog2e;
    h.x = fmaf(ex2_approx(a0 * dl), h.x, x * bm[0]);
    h.y = fmaf(ex2_approx(a1 * dl), h.y, x * bm[1]);
    h.z = fmaf(ex2_approx(a2 * dl), h.z, x * bm[2]);
    h.w = fmaf(ex2_approx(a3 * dl), h.w, x * bm[3]);
    if (in) *sp = h;
    float y = fmaf(h.x, cm[0], h.y * cm[1]) + fmaf(h.z, cm[2], h.w * cm[3]);
#pragma unroll
    for (int o = 1; o < LPC; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (in && part == 0) {
        y = fmaf(sk, uu, y);
        if (p.z) y *= zz * sigmoid_f<T>(zz);
        from_f(((T*)p.out)[at], y);
    }
}

// ------------------------------------------------------------------ launches
template <int N> struct ScanNS { static constexpr int value = N < 16 ? N : 16; };

// Blocks that a call should have before its tokens are cut into chunks: cutting
// runs every exponential twice.
static int scan_target(const SsmHandle& h) { return h.num_sms * 8; }
constexpr int kScanMinChunk = 64;

template <int N>
static ScanPlan scan_plan(const SsmHandle& h, int B, int L) {
    constexpr int LPC = N / ScanNS<N>::value, CPB = kScanThreads / LPC, TT = 8 * LPC;
    ScanPlan pl;
    pl.Dg = h.D / h.G;
    pl.tpg = (pl.Dg + CPB - 1) / CPB;
    pl.tiles = pl.tpg * h.G;
    const long long blocks = (long long)pl.tiles * B;
    long long want = scan_target(h) / blocks;
    const int most = (L + kScanMinChunk - 1) / kScanMinChunk;
    if (want > most) want = most;
    if (want < 1) want = 1;
    pl.Lc = (int)((L + want - 1) / want);
    pl.Lc = (pl.Lc + TT - 1) / TT * TT;
    pl.nC = (L + pl.Lc - 1) / pl.Lc;
    return pl;
}

// Several chunks come only while tiles * B * chunks <= scan_target, each of at
// most 128 channels.
size_t scan_prompt_ws(const SsmHandle& h) { return (size_t)scan_target(h) * kScanThreads * (2 * h.N + 1); }

template <typename T, int N, int V>
static void scan_launch(const SsmHandle& h, const ScanArgs& a, cudaStream_t st) {
    constexpr int NS = ScanNS<N>::value;
    const ScanPlan pl = scan_plan<N>(h, a.B, a.L);
    ScanWs ws;
    ws.hend = h.ws;
    ws.h0 = ws.hend + (size_t)a.B * pl.nC * h.D * N;
    ws.sdt = ws.h0 + (size_t)a.B * h.D * N;
    if (pl.nC > 1) {
        k_scan<T, N, NS, V, true><<<(unsigned)pl.tiles * a.B * (pl.nC - 1), kScanThreads, 0, st>>>(a, pl, ws, h.D, h.G);
        count_launch();
    }
    k_scan<T, N, NS, V, false><<<(unsigned)pl.tiles * a.B * pl.nC, kScanThreads, 0, st>>>(a, pl, ws, h.D, h.G);
    count_launch();
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
    const int v = f32 ? 4 : 8;
    // 16-byte accesses of u, dt, z, out need every row of a group to start on one
    const bool vec = h.D % v == 0 && (h.D / h.G) % v == 0 && is_aligned16(a.u) && is_aligned16(a.dt) &&
                     is_aligned16(a.z) && is_aligned16(a.out);
    if (f32 && vec) scan_by_n<float, 4>(h, a, st);
    else if (f32) scan_by_n<float, 1>(h, a, st);
    else if (vec) scan_by_n<__nv_bfloat16, 8>(h, a, st);
    else scan_by_n<__nv_bfloat16, 1>(h, a, st);
    return check_launch("favor_ssm_scan");
}

template <typename T, int N>
static void step_launch(const SsmHandle& h, const ScanArgs& a, cudaStream_t st) {
    const int cb = (h.D * (N / 4) + kScanThreads - 1) / kScanThreads;
    k_scan_step<T, N><<<(unsigned)cb * a.B, kScanThreads, 0, st>>>(a, h.D, h.G, cb);
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
