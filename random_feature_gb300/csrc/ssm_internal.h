// Internal declarations of the selective scan, the short causal convolution and
// the state pages: the handle, the launch arguments and the shared device code.
#pragma once

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cstddef>
#include <cstdint>

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
constexpr float kLog2e = 1.4426950408889634f;

// ln(1 + e^x) = max(x, 0) + log1p(e^-|x|).
__device__ __forceinline__ float softplus_f(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }

// 1 / (1 + e^-x).  For 16-bit storage the approximate forms (relative error
// below 2^-20) are far under the output's rounding of 2^-9; fp32 storage takes
// the accurate ones.
template <typename T>
__device__ __forceinline__ float sigmoid_f(float x) {
    if (sizeof(T) == 2) return __fdividef(1.f, 1.f + ex2_approx(-x * kLog2e));
    return 1.f / (1.f + expf(-x));
}

// Page of row b, or -1 if the row takes no part: a page outside the pool
// (padding rows), or one that an earlier row of the call already names, so that
// no page is written by two rows.  Every thread of the block gets the answer.
__device__ __forceinline__ int block_page(const PageArgs& pg, int b) {
    if (!pg.pages) return b < pg.n_pages ? b : -1;
    const int page = pg.pages[b];
    int dup = 0;
    for (int j = threadIdx.x; j < b; j += blockDim.x) dup |= pg.pages[j] == page;
    dup = __syncthreads_or(dup);
    return (page < 0 || page >= pg.n_pages || dup) ? -1 : page;
}

// Length of row b: lens[b] clamped to [0, L].
__device__ __forceinline__ int row_len(const int* lens, int b, int L) {
    if (!lens) return L;
    const int n = lens[b];
    return n < 0 ? 0 : n > L ? L : n;
}

}  // namespace favor
