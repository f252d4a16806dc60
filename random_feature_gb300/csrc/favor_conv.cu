// Short causal convolution over tokens, one filter of K taps a channel:
//     p[t, c] = bias[c] + sum_k w[c, k] x[t - K + 1 + k, c],   out = p or p * sigmoid(p)
// with the inputs before the first token taken from a window page [K-1, D]
// (zeros without one).  Nothing but bytes: 2K + 5 operations an element against
// one read and one write.  A thread owns 4 neighbouring channels (one where the
// rows do not start on 16 bytes) for a run of tokens, the filter in registers; the
// run's rows come through asynchronous copies, some tokens deep, into slots that
// only their thread reads, so that the bytes in flight cost no registers.  Only the
// K-1 rows before a run are read twice (from L2).
#include <initializer_list>

#include "ssm_internal.h"

namespace favor {

constexpr int kConvThreads = 128;

template <typename T>
__device__ __forceinline__ float silu_f(float p) { return p * sigmoid_f<T>(p); }

// d silu(p) / dp = s (1 + p (1 - s)), s = sigmoid(p).
template <typename T>
__device__ __forceinline__ float dsilu_f(float p) {
    const float s = sigmoid_f<T>(p);
    return s * (1.f + p * (1.f - s));
}

template <int V, int K>
__device__ __forceinline__ void load_taps(const float* weight, const float* bias, int c, float (&w)[V][K],
                                          float (&b)[V]) {
    if constexpr (V >= 4) {   // 16 bytes at a time: c is a multiple of V
#pragma unroll
        for (int i = 0; i < V * K; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(weight + (size_t)c * K + i);
            w[i / K][i % K] = f.x;
            w[(i + 1) / K][(i + 1) % K] = f.y;
            w[(i + 2) / K][(i + 2) % K] = f.z;
            w[(i + 3) / K][(i + 3) % K] = f.w;
        }
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 f = bias ? *reinterpret_cast<const float4*>(bias + c + i) : make_float4(0.f, 0.f, 0.f, 0.f);
            b[i] = f.x;
            b[i + 1] = f.y;
            b[i + 2] = f.z;
            b[i + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) w[0][k] = weight[(size_t)c * K + k];
        b[0] = bias ? bias[c] : 0.f;
    }
}

// Grid: channel blocks x runs x rows.  A run of R tokens is walked 8 at a time (4 in
// fp32), the two steps after it in flight.  [4, 8192, 1024] bf16: 29 us (4.6 TB/s; 43
// with the next rows in registers, 55 with 8 tokens a thread and no overlap).
constexpr int kConvStages = 3;

// Blocks an SM: their registers and rings allow for them.
constexpr int kConvPerSm = 6;
template <typename T>
__host__ __device__ constexpr int conv_bwd_per_sm() { return sizeof(T) == 2 ? 4 : 3; }

template <typename T, int V, int K>
__global__ void __launch_bounds__(kConvThreads, kConvPerSm) k_conv(ConvArgs a, int D, int cblocks, int runs, int R) {
    constexpr int U = sizeof(T) == 4 ? 4 : 8;
    const int cb = blockIdx.x % cblocks, rest = blockIdx.x / cblocks;
    const int run = rest % runs, b = rest / runs;
    const int page = a.window ? block_page(a.pg, b) : 0;
    const int len = row_len(a.lens, b, a.L);
    const int t0 = run * R, t1 = min(len, t0 + R);
    const int c = (cb * kConvThreads + threadIdx.x) * V;
    if (t0 >= t1 || c >= D) return;
    const T* x = (const T*)a.x + (size_t)b * a.L * D + c;
    T* out = (T*)a.out + (size_t)b * a.L * D + c;
    if (page < 0) {   // the row takes no part
        for (int t = t0; t < t1; ++t) *reinterpret_cast<Pack<T, V>*>(out + (size_t)t * D) = zero_pack<T, V>();
        return;
    }
    T* win = a.window ? (T*)a.window + (size_t)page * (K - 1) * D + c : nullptr;
    float w[V][K], bias[V];
    __shared__ Pack<T, V> ring[V > 1 ? kConvStages : 1][U][kConvThreads];
    Pack<T, V> r[U + K - 1], ahead[V > 1 ? 1 : U];   // rows t-K+1 .. t+7; narrow rows: t+8 ..
    auto fetch = [&](int t, int slot) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const bool ok = t + i < t1;
            if constexpr (V > 1) copy_async(&ring[slot][i][threadIdx.x], ok ? x + (size_t)(t + i) * D : x, ok);
            else ahead[i] = ok ? load_pack<T, V>(x + (size_t)(t + i) * D) : zero_pack<T, V>();
        }
        if constexpr (V > 1) copy_commit();
    };
#pragma unroll
    for (int s = 0; s < (V > 1 ? kConvStages - 1 : 1); ++s) fetch(t0 + s * U, s);
    load_taps<V, K>(a.weight, a.bias, c, w, bias);
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
        const int t = t0 - (K - 1) + i;
        r[i] = t >= 0 ? load_pack<T, V>(x + (size_t)t * D)
                      : win ? load_pack<T, V>(win + (size_t)(t + K - 1) * D) : zero_pack<T, V>();
    }
    // The first run alone reads the window, so its thread also moves it on: the
    // last K-1 of (window, inputs), row K-1 + len - (K-1) + i = len + i of that list.
    if (win && run == 0) {
        Pack<T, V> last[K - 1];
#pragma unroll
        for (int i = 0; i < K - 1; ++i) {
            const int t = len - (K - 1) + i;
            last[i] = load_pack<T, V>(t >= 0 ? x + (size_t)t * D : win + (size_t)(t + K - 1) * D);
        }
#pragma unroll
        for (int i = 0; i < K - 1; ++i) *reinterpret_cast<Pack<T, V>*>(win + (size_t)i * D) = last[i];
    }
    int slot = 0;
    for (int t = t0; t < t1; t += U) {
        if constexpr (V > 1) copy_wait<kConvStages - 2>();
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if constexpr (V > 1) r[K - 1 + i] = ring[slot][i][threadIdx.x];
            else r[K - 1 + i] = ahead[i];
        }
        // the slot before this one was read in the last step
        if constexpr (V > 1) fetch(t + (kConvStages - 1) * U, slot ? slot - 1 : kConvStages - 1);
        else fetch(t + U, 0);
        slot = slot + 1 < kConvStages ? slot + 1 : 0;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (t + i >= t1) break;
            Pack<T, V> o;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float p = bias[e];
#pragma unroll
                for (int k = 0; k < K; ++k) p = fmaf(w[e][k], to_f(r[i + k].v[e]), p);
                from_f(o.v[e], a.silu ? silu_f<T>(p) : p);
            }
            *reinterpret_cast<Pack<T, V>*>(out + (size_t)(t + i) * D) = o;
        }
#pragma unroll
        for (int i = 0; i < K - 1; ++i) r[i] = r[U + i];
    }
    if constexpr (V > 1) copy_wait<0>();
}

// One token a row: x [B, D], the window moves on by one.
template <typename T, int V, int K>
__global__ void __launch_bounds__(kConvThreads) k_conv_step(ConvArgs a, int D, int cblocks) {
    const int cb = blockIdx.x % cblocks, b = blockIdx.x / cblocks;
    const int c = (cb * kConvThreads + threadIdx.x) * V;
    int page = row_page(a.pg, b);
    const bool in = c < D;
    T* win = (T*)a.window + (size_t)(page < 0 ? 0 : page) * (K - 1) * D + (in ? c : 0);
    T* out = (T*)a.out + (size_t)b * D + c;
    Pack<T, V> r[K];
    float w[V][K], bias[V];
    if (in) {   // in flight while the earlier rows are looked through
#pragma unroll
        for (int i = 0; i < K - 1; ++i) r[i] = load_pack<T, V>(win + (size_t)i * D);
        r[K - 1] = load_pack<T, V>((const T*)a.x + (size_t)b * D + c);
        load_taps<V, K>(a.weight, a.bias, c, w, bias);
    }
    if (block_page_taken(a.pg, b, page)) page = -1;
    if (!in) return;
    if (page < 0) {   // the row takes no part
        *reinterpret_cast<Pack<T, V>*>(out) = zero_pack<T, V>();
        return;
    }
    Pack<T, V> o;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float p = bias[e];
#pragma unroll
        for (int k = 0; k < K; ++k) p = fmaf(w[e][k], to_f(r[k].v[e]), p);
        from_f(o.v[e], a.silu ? silu_f<T>(p) : p);
    }
    *reinterpret_cast<Pack<T, V>*>(out) = o;
#pragma unroll
    for (int i = 0; i < K - 1; ++i) *reinterpret_cast<Pack<T, V>*>(win + (size_t)i * D) = r[i + 1];
}

// Gradients of a call that starts from an empty window.  g[t] = dout[t] silu'(p[t]):
//     dx[t] = sum_k w[k] g[t + K - 1 - k],   dw[k] = sum_t g[t] x[t - K + 1 + k],   dbias = sum_t g[t]
// A run of R tokens is walked with the last K-1 inputs and gradients in
// registers, g being formed again for the K-1 tokens behind the run ([8, 4096, 1536]
// fp32: 111 us, 5.4 TB/s; 153 with the next rows in registers instead of the ring).
// The run's sums of dw and dbias go to a row of the workspace, added in a fixed order by
// k_conv_reduce.  fp32 storage adds 4 tokens first: a term passes through R / 4 + rows / 128 +
// 11 additions of fp32, R tokens a run.  16-bit storage adds them one by one: its gates are
// good to 2^-19, and the additions in between cost 3% (80.3 to 82.6 us at [8, 4096, 1536]).
template <typename T, int V, int K>
__global__ void __launch_bounds__(kConvThreads, conv_bwd_per_sm<T>())
k_conv_bwd(ConvArgs a, int D, int cblocks, int runs, int R, float* part) {
    const int cb = blockIdx.x % cblocks, rest = blockIdx.x / cblocks;
    const int run = rest % runs, b = rest / runs;
    const int c = (cb * kConvThreads + threadIdx.x) * V;
    if (c >= D) return;
    const int len = row_len(a.lens, b, a.L);
    const int t0 = run * R, t1 = min(t0 + R, len);
    const T* x = (const T*)a.x + (size_t)b * a.L * D + c;
    const T* dout = (const T*)a.dout + (size_t)b * a.L * D + c;
    T* dx = (T*)a.dx + (size_t)b * a.L * D + c;
    for (int t = max(t0, len); t < min(t0 + R, a.L); ++t)   // behind the row's end: no gradient
        *reinterpret_cast<Pack<T, V>*>(dx + (size_t)t * D) = zero_pack<T, V>();
    float w[V][K], bias[V];
    load_taps<V, K>(a.weight, a.bias, c, w, bias);
    float xs[V][K], gs[V][K], dw[V][K], db[V];   // xs: x[t-K+1 .. t]; gs: g[t-K+1 .. t]
#pragma unroll
    for (int e = 0; e < V; ++e) {
        db[e] = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) { xs[e][k] = gs[e][k] = dw[e][k] = 0.f; }
    }
    if (t0 < t1) {
#pragma unroll
        for (int i = 0; i < K - 1; ++i) {
            const int t = t0 - (K - 1) + i;
            if (t >= 0) {
                const Pack<T, V> r = load_pack<T, V>(x + (size_t)t * D);
#pragma unroll
                for (int e = 0; e < V; ++e) xs[e][i + 1] = to_f(r.v[e]);
            }
        }
    }
    constexpr int U = 4, STAGES = 3;   // tokens a step, steps in the ring
    constexpr bool FOUR = sizeof(T) == 4;
    __shared__ Pack<T, V> ring[V > 1 ? STAGES : 1][2][U][kConvThreads];
    Pack<T, V> ahead[2][V > 1 ? 1 : U];
    const int tend = t0 < t1 ? min(len, t1 + K - 1) : t0;
    auto fetch = [&](int t, int slot) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const bool ok = t + i < tend;
            const size_t at = ok ? (size_t)(t + i) * D : 0;
            if constexpr (V > 1) {
                copy_async(&ring[slot][0][i][threadIdx.x], x + at, ok);
                copy_async(&ring[slot][1][i][threadIdx.x], dout + at, ok);
            } else {
                ahead[0][i] = ok ? load_pack<T, V>(x + at) : zero_pack<T, V>();
                ahead[1][i] = ok ? load_pack<T, V>(dout + at) : zero_pack<T, V>();
            }
        }
        if constexpr (V > 1) copy_commit();
    };
#pragma unroll
    for (int s = 0; s < (V > 1 ? STAGES - 1 : 1); ++s) fetch(t0 + s * U, s);
    int slot = 0;
    for (int t4 = t0; t4 < t1 + K - 1 && t0 < t1; t4 += U) {
        Pack<T, V> rx[U], rg[U];
        if constexpr (V > 1) copy_wait<STAGES - 2>();
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if constexpr (V > 1) {
                rx[i] = ring[slot][0][i][threadIdx.x];
                rg[i] = ring[slot][1][i][threadIdx.x];
            } else {
                rx[i] = ahead[0][i];
                rg[i] = ahead[1][i];
            }
        }
        if constexpr (V > 1) fetch(t4 + (STAGES - 1) * U, slot ? slot - 1 : STAGES - 1);
        else fetch(t4 + U, 0);
        slot = slot + 1 < STAGES ? slot + 1 : 0;
        Pack<T, V> o[U];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float dw4[K], db4;   // of these tokens, or the run's sums themselves
#pragma unroll
            for (int k = 0; k < K; ++k) dw4[k] = FOUR ? 0.f : dw[e][k];
            db4 = FOUR ? 0.f : db[e];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const bool in = t4 + i < len, own = t4 + i < t1;
#pragma unroll
                for (int k = 0; k + 1 < K; ++k) { xs[e][k] = xs[e][k + 1]; gs[e][k] = gs[e][k + 1]; }
                xs[e][K - 1] = to_f(rx[i].v[e]);
                float g = to_f(rg[i].v[e]);
                if (a.silu) {
                    float p = bias[e];
#pragma unroll
                    for (int k = 0; k < K; ++k) p = fmaf(w[e][k], xs[e][k], p);
                    g *= dsilu_f<T>(p);
                }
                if (!in) g = 0.f;
                gs[e][K - 1] = g;
                if (own) {
                    db4 += g;
#pragma unroll
                    for (int k = 0; k < K; ++k) dw4[k] = fmaf(g, xs[e][k], dw4[k]);
                }
                // dx of token t-K+1: taps k meet g[t-K+1 + K-1-k] = gs[K-1-k]
                float s = 0.f;
#pragma unroll
                for (int k = 0; k < K; ++k) s = fmaf(w[e][k], gs[e][K - 1 - k], s);
                from_f(o[i].v[e], s);
            }
            db[e] = FOUR ? db[e] + db4 : db4;
#pragma unroll
            for (int k = 0; k < K; ++k) dw[e][k] = FOUR ? dw[e][k] + dw4[k] : dw4[k];
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int t = t4 + i - (K - 1);
            if (t >= t0 && t < t1) *reinterpret_cast<Pack<T, V>*>(dx + (size_t)t * D) = o[i];
        }
    }
    if constexpr (V > 1) copy_wait<0>();
    float* row = part + (size_t)(b * runs + run) * D * (K + 1) + (size_t)c;
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int k = 0; k < K; ++k) row[(size_t)k * D + e] = dw[e][k];
        row[(size_t)K * D + e] = db[e];
    }
}

// part [rows][K+1][D] summed over rows in a fixed order.
__global__ void __launch_bounds__(256) k_conv_reduce(const float* part, int rows, int D, int K, float* dweight,
                                                     float* dbias) {
    const int n = D * (K + 1), i = blockIdx.x * 32 + (threadIdx.x & 31);
    const float sum = block_column_sum(i < n ? part + i : nullptr, n, rows);
    if (threadIdx.x < 32 && i < n) {
        const int k = i / D, c = i % D;
        if (k < K) dweight[(size_t)c * K + k] = sum;
        else if (dbias) dbias[c] = sum;
    }
}

// Whether rows of 16-byte columns (and the parameters with them) start on 16 bytes.
static bool vector_rows(const SsmHandle& h, std::initializer_list<const void*> ptrs) {
    const int v = h.dtype == FAVOR_DTYPE_F32 ? 4 : 8;
    if (h.D % v) return false;
    for (const void* p : ptrs)
        if (p && !is_aligned16(p)) return false;
    return true;
}

// Calls f<T, V, K>() for the handle's storage type, access width and taps.
template <template <typename, int, int> class F, typename... A>
static void conv_dispatch(const SsmHandle& h, bool vec, A... args) {
    const bool f32 = h.dtype == FAVOR_DTYPE_F32;
#define FAVOR_CONV_K(T, V)                              \
    do {                                                \
        if (h.K == 2) F<T, V, 2>::go(h, args...);       \
        else if (h.K == 3) F<T, V, 3>::go(h, args...);  \
        else F<T, V, 4>::go(h, args...);                \
    } while (0)
    if (f32 && vec) FAVOR_CONV_K(float, 4);
    else if (f32) FAVOR_CONV_K(float, 1);
    else if (vec) FAVOR_CONV_K(__nv_bfloat16, 8);
    else FAVOR_CONV_K(__nv_bfloat16, 1);
#undef FAVOR_CONV_K
}

static int conv_cblocks(int D, int V) { return (D + kConvThreads * V - 1) / (kConvThreads * V); }

// Tokens a run so that the blocks come to whole waves of per_sm on every SM: as many waves as runs of
// kConvRunTokens would take, and then as few tokens as that leaves, `least` at least ([4, 8192, 1024] bf16
// in runs of 72, one wave, is 9% faster than in runs of 32, 2.2 waves).  The runs a row are rounded down, so that a
// run has under 2 kConvRunTokens + U tokens.
constexpr int kConvRunTokens = 256;

static int run_tokens(const SsmHandle& h, int cb, int B, int L, int per_sm, int U, int least) {
    const long long slots = (long long)h.num_sms * per_sm, columns = (long long)cb * B;
    const long long waves = (columns * L + slots * kConvRunTokens - 1) / (slots * kConvRunTokens);
    long long runs = slots * waves / columns;
    if (runs < 1) runs = 1;
    long long R = (L + runs - 1) / runs;
    if (R < least) R = least;
    return (int)((R + U - 1) / U * U);
}

template <typename T, int V, int K>
struct ConvPrompt {
    static void go(const SsmHandle& h, const ConvArgs& a, cudaStream_t st) {
        constexpr int VP = V < 4 ? V : 4;
        const int cb = conv_cblocks(h.D, VP);
        const int R = run_tokens(h, cb, a.B, a.L, kConvPerSm, 8, 8), runs = (a.L + R - 1) / R;
        k_conv<T, VP, K><<<(unsigned)cb * runs * a.B, kConvThreads, 0, st>>>(a, h.D, cb, runs, R);
    }
};

template <typename T, int V, int K>
struct ConvStep {
    static void go(const SsmHandle& h, const ConvArgs& a, cudaStream_t st) {
        const int cb = conv_cblocks(h.D, V);
        k_conv_step<T, V, K><<<(unsigned)cb * a.B, kConvThreads, 0, st>>>(a, h.D, cb);
    }
};

// Tokens of a backward run at least: the K-1 tokens formed twice and the run's row
// of partial sums stay small next to it.
constexpr int kConvBwdRun = 16;

template <typename T, int V, int K>
struct ConvBwd {
    static void go(const SsmHandle& h, const ConvArgs& a, cudaStream_t st) {
        constexpr int VB = V < 4 ? V : 4;   // the sums of 8 channels would take 144 registers
        const int cb = conv_cblocks(h.D, VB);
        const int R = run_tokens(h, cb, a.B, a.L, conv_bwd_per_sm<T>(), 4, kConvBwdRun), runs = (a.L + R - 1) / R;
        k_conv_bwd<T, VB, K><<<(unsigned)cb * runs * a.B, kConvThreads, 0, st>>>(a, h.D, cb, runs, R, h.ws);
        const int n = h.D * (K + 1);
        k_conv_reduce<<<(n + 31) / 32, 256, 0, st>>>(h.ws, a.B * runs, h.D, K, a.dweight, a.dbias);
    }
};

// A row of partial sums a run.  run_tokens gives B rows (one run each) or slots * waves / cblocks at most,
// and waves < cblocks B L / (kConvRunTokens slots) + 1: together less than B + B L / kConvRunTokens + slots.
size_t conv_backward_ws(const SsmHandle& h) {
    const size_t slots = (size_t)h.num_sms * conv_bwd_per_sm<__nv_bfloat16>();   // the larger of the two
    const size_t rows = (size_t)h.max_B * (1 + (h.max_L + kConvRunTokens - 1) / kConvRunTokens) + slots;
    return rows * h.D * (h.K + 1);
}

favor_status conv_prompt(const SsmHandle& h, const ConvArgs& a, cudaStream_t st) {
    conv_dispatch<ConvPrompt>(h, vector_rows(h, {a.x, a.out, a.window, a.weight, a.bias}), a, st);
    count_launch();
    return check_launch("favor_conv_causal");
}

favor_status conv_step(const SsmHandle& h, const ConvArgs& a, cudaStream_t st) {
    conv_dispatch<ConvStep>(h, vector_rows(h, {a.x, a.out, a.window, a.weight, a.bias}), a, st);
    count_launch();
    return check_launch("favor_conv_causal_step");
}

favor_status conv_backward(const SsmHandle& h, const ConvArgs& a, cudaStream_t st) {
    conv_dispatch<ConvBwd>(h, vector_rows(h, {a.x, a.dout, a.dx, a.weight, a.bias}), a, st);
    count_launch(2);
    return check_launch("favor_conv_causal_backward");
}

}  // namespace favor
