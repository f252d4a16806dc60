// Short causal convolution over tokens, one filter of K taps a channel:
//     p[t, c] = bias[c] + sum_k w[c, k] x[t - K + 1 + k, c],   out = p or p * sigmoid(p)
// with the inputs before the first token taken from a window page [K-1, D]
// (zeros without one).  Nothing but bytes: 2K + 5 operations an element against
// one read and one write, so a thread owns a 16-byte column of channels (one
// channel where the rows do not start on 16 bytes) for a run of tokens, loads
// the run's rows up front and keeps them in registers; only the K-1 rows before
// a run are read twice (from L2).
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
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int k = 0; k < K; ++k) w[i][k] = weight[(size_t)(c + i) * K + k];
        b[i] = bias ? bias[c + i] : 0.f;
    }
}

// Grid: channel blocks x runs x rows.  A run is R tokens.
template <typename T, int V, int K, int R>
__global__ void __launch_bounds__(kConvThreads) k_conv(ConvArgs a, int D, int cblocks, int runs) {
    const int cb = blockIdx.x % cblocks, rest = blockIdx.x / cblocks;
    const int run = rest % runs, b = rest / runs;
    const int page = a.window ? block_page(a.pg, b) : 0;
    const int len = row_len(a.lens, b, a.L);
    const int t0 = run * R, n = min(R, len - t0);
    const int c = (cb * kConvThreads + threadIdx.x) * V;
    if (n <= 0 || c >= D) return;
    const T* x = (const T*)a.x + (size_t)b * a.L * D + c;
    T* out = (T*)a.out + (size_t)b * a.L * D + c;
    if (page < 0) {   // the row takes no part
        for (int i = 0; i < n; ++i) *reinterpret_cast<Pack<T, V>*>(out + (size_t)(t0 + i) * D) = zero_pack<T, V>();
        return;
    }
    T* win = a.window ? (T*)a.window + (size_t)page * (K - 1) * D + c : nullptr;
    float w[V][K], bias[V];
    load_taps<V, K>(a.weight, a.bias, c, w, bias);
    // rows t0-K+1 .. t0+R-1
    Pack<T, V> r[R + K - 1];
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
        const int t = t0 - (K - 1) + i;
        r[i] = t >= 0 ? load_pack<T, V>(x + (size_t)t * D)
                      : win ? load_pack<T, V>(win + (size_t)(t + K - 1) * D) : zero_pack<T, V>();
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
        r[K - 1 + i] = i < n ? load_pack<T, V>(x + (size_t)(t0 + i) * D) : zero_pack<T, V>();
    // The first run alone reads the window, so its thread also moves it on: the
    // last K-1 of (window, inputs), row K-1 + len - (K-1) + i = len + i of that list.
    Pack<T, V> last[K - 1];
    if (win && run == 0) {
#pragma unroll
        for (int i = 0; i < K - 1; ++i) {
            const int t = len - (K - 1) + i;
            last[i] = load_pack<T, V>(t >= 0 ? x + (size_t)t * D : win + (size_t)(t + K - 1) * D);
        }
#pragma unroll
        for (int i = 0; i < K - 1; ++i) *reinterpret_cast<Pack<T, V>*>(win + (size_t)i * D) = last[i];
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (i >= n) break;
        Pack<T, V> o;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float p = bias[e];
#pragma unroll
            for (int k = 0; k < K; ++k) p = fmaf(w[e][k], to_f(r[i + k].v[e]), p);
            from_f(o.v[e], a.silu ? silu_f<T>(p) : p);
        }
        *reinterpret_cast<Pack<T, V>*>(out + (size_t)(t0 + i) * D) = o;
    }
}

// One token a row: x [B, D], the window moves on by one.
template <typename T, int V, int K>
__global__ void __launch_bounds__(kConvThreads) k_conv_step(ConvArgs a, int D, int cblocks) {
    const int cb = blockIdx.x % cblocks, b = blockIdx.x / cblocks;
    const int c = (cb * kConvThreads + threadIdx.x) * V;
    const int page = block_page(a.pg, b);
    if (c >= D) return;
    T* out = (T*)a.out + (size_t)b * D + c;
    if (page < 0) {   // the row takes no part
        *reinterpret_cast<Pack<T, V>*>(out) = zero_pack<T, V>();
        return;
    }
    T* win = (T*)a.window + (size_t)page * (K - 1) * D + c;
    Pack<T, V> r[K];
#pragma unroll
    for (int i = 0; i < K - 1; ++i) r[i] = load_pack<T, V>(win + (size_t)i * D);
    r[K - 1] = load_pack<T, V>((const T*)a.x + (size_t)b * D + c);
    float w[V][K], bias[V];
    load_taps<V, K>(a.weight, a.bias, c, w, bias);
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
// registers, g being formed again for the K-1 tokens behind the run.  The run's
// sums of dw and dbias go to a row of the workspace, added in a fixed order by
// k_conv_reduce.
template <typename T, int V, int K>
__global__ void __launch_bounds__(kConvThreads)
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
    for (int t = t0; t < t1 + K - 1 && t0 < t1; ++t) {
        const bool in = t < len;
        const Pack<T, V> rx = in ? load_pack<T, V>(x + (size_t)t * D) : zero_pack<T, V>();
        const Pack<T, V> rg = in ? load_pack<T, V>(dout + (size_t)t * D) : zero_pack<T, V>();
        const bool own = t < t1;
        Pack<T, V> o;
#pragma unroll
        for (int e = 0; e < V; ++e) {
#pragma unroll
            for (int k = 0; k + 1 < K; ++k) { xs[e][k] = xs[e][k + 1]; gs[e][k] = gs[e][k + 1]; }
            xs[e][K - 1] = to_f(rx.v[e]);
            float g = to_f(rg.v[e]);
            if (a.silu) {
                float p = bias[e];
#pragma unroll
                for (int k = 0; k < K; ++k) p = fmaf(w[e][k], xs[e][k], p);
                g *= dsilu_f<T>(p);
            }
            if (!in) g = 0.f;
            gs[e][K - 1] = g;
            if (own) {
                db[e] += g;
#pragma unroll
                for (int k = 0; k < K; ++k) dw[e][k] = fmaf(g, xs[e][k], dw[e][k]);
            }
            // dx of token t-K+1: taps k meet g[t-K+1 + K-1-k] = gs[K-1-k]
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) s = fmaf(w[e][k], gs[e][K - 1 - k], s);
            from_f(o.v[e], s);
        }
        if (t - (K - 1) >= t0) *reinterpret_cast<Pack<T, V>*>(dx + (size_t)(t - (K - 1)) * D) = o;
    }
    float* row = part + (size_t)(b * runs + run) * D * (K + 1) + (size_t)c;
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
        for (int k = 0; k < K; ++k) row[(size_t)k * D + e] = dw[e][k];
        row[(size_t)K * D + e] = db[e];
    }
}

// part [rows][K+1][D] summed over rows, in the rows' order within each of 8 lanes
// and the lanes' order at the end.
__global__ void __launch_bounds__(256) k_conv_reduce(const float* part, int rows, int D, int K, float* dweight,
                                                     float* dbias) {
    __shared__ float s[8][33];
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int n = D * (K + 1), i = blockIdx.x * 32 + lane;
    float acc = 0.f;
    if (i < n)
        for (int r = y; r < rows; r += 8) acc += part[(size_t)r * n + i];
    s[y][lane] = acc;
    __syncthreads();
    if (y == 0 && i < n) {
#pragma unroll
        for (int k = 1; k < 8; ++k) acc += s[k][lane];
        const int k = i / D, c = i % D;
        if (k < K) dweight[(size_t)c * K + k] = acc;
        else if (dbias) dbias[c] = acc;
    }
}

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

constexpr int kConvRun = 8;

template <typename T, int V, int K>
struct ConvPrompt {
    static void go(const SsmHandle& h, const ConvArgs& a, cudaStream_t st) {
        const int cb = conv_cblocks(h.D, V), runs = (a.L + kConvRun - 1) / kConvRun;
        k_conv<T, V, K, kConvRun><<<(unsigned)cb * runs * a.B, kConvThreads, 0, st>>>(a, h.D, cb, runs);
    }
};

template <typename T, int V, int K>
struct ConvStep {
    static void go(const SsmHandle& h, const ConvArgs& a, cudaStream_t st) {
        const int cb = conv_cblocks(h.D, V);
        k_conv_step<T, V, K><<<(unsigned)cb * a.B, kConvThreads, 0, st>>>(a, h.D, cb);
    }
};

// Tokens of a backward run: long enough that the K-1 tokens formed twice and the
// run's row of partial sums stay small next to it.
constexpr int kConvBwdRun = 64;

template <typename T, int V, int K>
struct ConvBwd {
    static void go(const SsmHandle& h, const ConvArgs& a, cudaStream_t st) {
        const int cb = conv_cblocks(h.D, V), runs = (a.L + kConvBwdRun - 1) / kConvBwdRun;
        k_conv_bwd<T, V, K><<<(unsigned)cb * runs * a.B, kConvThreads, 0, st>>>(a, h.D, cb, runs, kConvBwdRun, h.ws);
        const int n = h.D * (K + 1);
        k_conv_reduce<<<(n + 31) / 32, 256, 0, st>>>(h.ws, a.B * runs, h.D, K, a.dweight, a.dbias);
    }
};

size_t conv_backward_ws(const SsmHandle& h) {
    return (size_t)h.max_B * ((h.max_L + kConvBwdRun - 1) / kConvBwdRun) * h.D * (h.K + 1);
}

favor_status conv_prompt(const SsmHandle& h, const ConvArgs& a, cudaStream_t st) {
    conv_dispatch<ConvPrompt>(h, vector_rows(h, {a.x, a.out, a.window}), a, st);
    count_launch();
    return check_launch("favor_conv_causal");
}

favor_status conv_step(const SsmHandle& h, const ConvArgs& a, cudaStream_t st) {
    conv_dispatch<ConvStep>(h, vector_rows(h, {a.x, a.out, a.window}), a, st);
    count_launch();
    return check_launch("favor_conv_causal_step");
}

favor_status conv_backward(const SsmHandle& h, const ConvArgs& a, cudaStream_t st) {
    conv_dispatch<ConvBwd>(h, vector_rows(h, {a.x, a.dout, a.dx}), a, st);
    count_launch(2);
    return check_launch("favor_conv_causal_backward");
}

}  // namespace favor
