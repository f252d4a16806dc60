// Internal declarations of the selective scan, the short causal convolution and
// the state pages: the handle, the launch arguments and the shared device code.
#pragma once

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cstddef>
#include <cstdint>
#include <mutex>

#include "favor_internal.h"

namespace favor {

// Everything a favor_ssm handle owns.  Device pointers unless noted.
struct SsmHandle {
    int D, N, G, K;
    favor_dtype dtype;
    int max_B, max_L;
    bool training;          // the backward calls' workspace exists
    int device, num_sms;
    float* ws;              // one area, laid out per call by the launchers below
    size_t ws_floats;
    // Held while a call that uses ws is enqueued: it is several launches, and another host thread's,
    // on the same stream, must not come between them.
    mutable std::mutex enqueue;
};

// Rows b of a call and where their state lives.
struct PageArgs {
    const int* pages;       // [B] page of row b (null: page b)
    int n_pages;
};

struct ConvArgs {
    const void* x;
    const float* weight;    // [D][K]
    const float* bias;      // [D] or null
    void* window;           // [n_pages][K-1][D] or null
    PageArgs pg;
    const int* lens;        // [B] or null
    void* out;
    const void* dout;       // backward
    void* dx;
    float* dweight;
    float* dbias;           // may be null
    int B, L, silu;
};

struct ScanArgs {
    const void *u, *dt, *Bm, *Cm, *z;    // z may be null
    const float *A, *skip, *dt_bias;     // skip, dt_bias may be null
    float* state;           // [n_pages][D][N] or null (zero start, end not kept)
    PageArgs pg;
    const int* lens;
    void* out;
    const void* dout;       // backward
    void *du, *ddt, *dB, *dC, *dz;       // dz null when z is
    float *dA, *dskip, *ddt_bias;        // null when the parameter is
    int B, L;
};

favor_status conv_prompt(const SsmHandle& h, const ConvArgs& a, cudaStream_t st);
favor_status conv_step(const SsmHandle& h, const ConvArgs& a, cudaStream_t st);
favor_status conv_backward(const SsmHandle& h, const ConvArgs& a, cudaStream_t st);
favor_status scan_prompt(const SsmHandle& h, const ScanArgs& a, cudaStream_t st);
favor_status scan_step(const SsmHandle& h, const ScanArgs& a, cudaStream_t st);
favor_status scan_backward(const SsmHandle& h, const ScanArgs& a, cudaStream_t st);

// Per chunk of tokens, in the workspace (see favor_scan.cu).
struct ScanWs {
    float* hs;      // [B][nC][D][N] the chunk's own end, then its start
    float* sdt;     // [B][nC][D] sum of dt
    float* mu;      // [B][nC][D][N] backward: what it hands back, then what it is handed
};
// Chunk starts and incoming gradients of a backward call with chunks of Lc tokens; whether its rows
// take 16-byte accesses.
bool scan_grad_chunks(const SsmHandle& h, const ScanArgs& a, const ScanWs& ws, int Lc, cudaStream_t st);

// Workspace (floats) the calls of a handle with these sizes can need.
size_t scan_prompt_ws(const SsmHandle& h);
size_t scan_backward_ws(const SsmHandle& h);
size_t conv_backward_ws(const SsmHandle& h);

// ------------------------------------------------------------------ device code
// V consecutive elements moved as one access of V * sizeof(T) bytes (<= 16).
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
    T v[V];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& d, float x) { d = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T* p) {
    return *reinterpret_cast<const Pack<T, V>*>(p);
}
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> zero_pack() {
    Pack<T, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) from_f(r.v[i], 0.f);
    return r;
}

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// log2 e and ln 2 in two parts (Cody and Waite's split): the nearest float and what it leaves.
constexpr double kLog2eExact = 1.4426950408889634074;
constexpr float kLog2e = (float)kLog2eExact, kLog2eRest = (float)(kLog2eExact - (double)kLog2e);
constexpr double kLn2Exact = 0.69314718055994530942;
constexpr float kLn2 = (float)kLn2Exact, kLn2Rest = (float)(kLn2Exact - (double)kLn2);

// One pack (4, 8 or 16 bytes) global -> shared, asynchronously; zeros where !ok (src is not read then).
template <typename P>
__device__ __forceinline__ void copy_async(P* dst, const void* src, bool ok) {
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    if constexpr (sizeof(P) == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src), "r"(ok ? 16 : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(src), "n"((int)sizeof(P)),
                     "r"(ok ? (int)sizeof(P) : 0)
                     : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Wait until at most N of this thread's committed groups are still in flight.
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ex2.approx rounds towards smaller results: its mean relative error on this
// device is -0.32 to -0.35 steps of 2^-24 for exponents in [-0.5, -0.003], where most
// decays lie.  Exponents carry this offset, 0.32 * 2^-24 * log2 e, which leaves -0.03 to
// 0.03 there; an exponent of 0 still gives 1.  Without it dA of a 777-token scan in fp32
// is 1.3e-6 off instead of 6e-7.  Between -0.003 and -1e-7 the mean is -0.09 to -0.18
// without the offset and 0.14 to 0.23 with it, about that of expf (0.26): at an exponent
// of -r a token that comes to 0.2 * 2^-24 / r of a long memory.  Half the offset has
// -0.02 to 0.07 there, and -0.16 to -0.25 in the range above.  Below -0.5 an offset is lost.
constexpr float kEx2Mean = 2.75e-8f;

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


// ln(1 + e^x) = max(x, 0) + log1p(e), e = e^-|x| <= 1, with
// log1p(e) = 2 atanh(s), s = e / (2 + e) <= 1/3: the odd series up to s^13 leaves
// s^14 / 15 < 1.4e-8 of the sum.  Two values at a time for the packed FMA.  The
// product of |x| and log2 e is off by half a step, |x| 2^-24 of e and so of the result
// (3e-6 at -50): of no weight beside a raw step of 16 bits, which leaves |x| 2^-9.  fp32
// storage multiplies e = 2^t by 1 + d, d = -|x| - t ln 2 with ln 2 in two parts (Cody and
// Waite's reduction): [8, 4096, 1536] with 16 states 463 us, 457 without.
template <typename T>
__device__ __forceinline__ void softplus_2(float& x0, float& x1) {
    const float t0 = -fabsf(x0) * kLog2e, t1 = -fabsf(x1) * kLog2e;
    float e0 = ex2_approx(t0), e1 = ex2_approx(t1);
    if constexpr (sizeof(T) == 4) {
        float d0, d1;
        const uint64_t t = pack2(-t0, -t1), e = pack2(e0, e1);
        unpack2(fma2(t, pack2(kLn2Rest, kLn2Rest), fma2(t, pack2(kLn2, kLn2), pack2(-fabsf(x0), -fabsf(x1)))), d0, d1);
        // infinite t leave no d, and e = 0 (the minimum with a NaN is the other operand; e keeps a NaN of x)
        unpack2(fma2(e, pack2(fminf(d0, 1.f), fminf(d1, 1.f)), e), e0, e1);
    }
    const uint64_t s = mul2(pack2(e0, e1), pack2(rcp_approx(2.f + e0), rcp_approx(2.f + e1)));
    const uint64_t q = mul2(s, s);
    uint64_t r = fma2(q, pack2(1.f / 13.f, 1.f / 13.f), pack2(1.f / 11.f, 1.f / 11.f));
    r = fma2(r, q, pack2(1.f / 9.f, 1.f / 9.f));
    r = fma2(r, q, pack2(1.f / 7.f, 1.f / 7.f));
    r = fma2(r, q, pack2(1.f / 5.f, 1.f / 5.f));
    r = fma2(r, q, pack2(1.f / 3.f, 1.f / 3.f));
    r = fma2(r, q, pack2(1.f, 1.f));
    unpack2(fma2(mul2(s, pack2(2.f, 2.f)), r, pack2(fmaxf(x0, 0.f), fmaxf(x1, 0.f))), x0, x1);
}
template <typename T>
__device__ __forceinline__ float softplus_f(float x) {
    float y = x;
    softplus_2<T>(x, y);
    return x;
}

// 1 / (1 + e^-x).  For 16-bit storage the approximate forms (relative error
// below 2^-19 for |x| < 16) are far under the output's rounding of 2^-9.  fp32
// storage multiplies e by 1 + r ln 2, r what the rounded product with log2 e lacks
// of the exact one, taken from the two parts by fused multiply-adds; and takes one
// Newton step, s + s (1 - d s), on the reciprocal (e is kept finite for it; a NaN
// comes back through x itself in every product this is used in).
template <typename T>
__device__ __forceinline__ float sigmoid_f(float x) {
    const float t = -x * kLog2e;
    float e = ex2_approx(t);
    if (sizeof(T) == 2) return rcp_approx(1.f + e);
    const float r = fmaf(-x, kLog2eRest, fmaf(-x, kLog2e, -t));
    if (fabsf(x) < 100.f) e = fmaf(e, r * kLn2, e);   // not of infinities
    e = fminf(e, 1e38f);
    const float d = 1.f + e, s = rcp_approx(d);
    return fmaf(s, fmaf(-d, s, 1.f), s);
}

// v[0..N) added two by two, N a power of two.
template <int N>
__device__ __forceinline__ float sum_two_by_two(float* v) {
#pragma unroll
    for (int n = N / 2; n > 0; n >>= 1)
#pragma unroll
        for (int k = 0; k < n; ++k) v[k] += v[k + n];
    return v[0];
}
// For a block of 256 threads: lane l of every warp has a column, whose `rows` values lie `step`
// floats apart from `at` on (null: none).  Warp 0's lanes get their sums.  Warp y has rows y, y + 8,
// ..; 16 of them are loaded together and added two by two before they meet the warp's sum, so that a
// term passes through rows / 128 + 7 additions.
__device__ __forceinline__ float block_column_sum(const float* at, size_t step, int rows) {
    constexpr int W = 8, P = 16;
    __shared__ float s[W][33];
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
    float sum = 0.f, v[P];
    if (at) {
        at += y * step;
        step *= W;
        for (int left = (rows - y + W - 1) / W; left > 0; left -= P) {
#pragma unroll
            for (int k = 0; k < P; ++k, at += step) v[k] = k < left ? *at : 0.f;
            sum += sum_two_by_two<P>(v);
        }
    }
    s[y][lane] = sum;
    __syncthreads();
    if (y) return 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) v[k] = s[k][lane];
    return sum_two_by_two<W>(v);
}

// Page of row b, or -1 if it is outside the pool (padding rows).
__device__ __forceinline__ int row_page(const PageArgs& pg, int b) {
    const int page = pg.pages ? pg.pages[b] : b;
    return page < 0 || page >= pg.n_pages ? -1 : page;
}
// Whether an earlier row of the call names row b's page too: such a row takes no
// part, so that no page is written by two rows.  For every thread of the block.
__device__ __forceinline__ bool block_page_taken(const PageArgs& pg, int b, int page) {
    if (!pg.pages) return false;
    int dup = 0;
    for (int j = threadIdx.x; j < b; j += blockDim.x) dup |= pg.pages[j] == page;
    return __syncthreads_or(dup);
}
// Page of row b, or -1 if the row takes no part.
__device__ __forceinline__ int block_page(const PageArgs& pg, int b) {
    const int page = row_page(pg, b);
    return block_page_taken(pg, b, page) ? -1 : page;
}

// Length of row b: lens[b] clamped to [0, L].
__device__ __forceinline__ int row_len(const int* lens, int b, int L) {
    if (!lens) return L;
    const int n = lens[b];
    return n < 0 ? 0 : n > L ? L : n;
}

}  // namespace favor
