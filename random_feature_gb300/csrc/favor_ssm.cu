// Host side of the selective scan and the short causal convolution: argument
// checks, handle lifetime, workspace.  Every check runs before anything is
// enqueued; a failing call launches nothing.
#include <initializer_list>
#include <mutex>
#include <new>

#include "ssm_internal.h"

using namespace favor;

namespace {

struct Span {
    const void* p;
    size_t bytes;
};

bool overlap(const Span& a, const Span& b) {
    if (!a.p || !b.p) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.bytes && y < x + a.bytes;
}

// No output may overlap an input or another output.
bool any_overlap(const Span* out, int n_out, const Span* in, int n_in) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j)
            if (overlap(out[i], in[j])) return true;
        for (int j = i + 1; j < n_out; ++j)
            if (overlap(out[i], out[j])) return true;
    }
    return false;
}

size_t esize(const SsmHandle& h) { return h.dtype == FAVOR_DTYPE_F32 ? 4 : 2; }

favor_status check_call(const char* fn, favor_ssm hd, int B, int L) {
    set_error(FAVOR_OK, "%s", "");
    if (!hd) return set_error(FAVOR_ERR_INVALID_ARG, "%s: handle is NULL", fn);
    const SsmHandle* h = reinterpret_cast<const SsmHandle*>(hd);
    if (B < 1 || L < 1) return set_error(FAVOR_ERR_INVALID_ARG, "%s: B=%d L=%d must be >= 1", fn, B, L);
    if (B > h->max_B || L > h->max_L)
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: B=%d L=%d exceed the handle's max_B=%d max_L=%d", fn, B, L,
                         h->max_B, h->max_L);
    int cur = -1;
    if (cudaGetDevice(&cur) != cudaSuccess || cur != h->device) {
        cudaGetLastError();
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: current device %d is not the handle's device %d", fn, cur,
                         h->device);
    }
    return FAVOR_OK;
}

// The pages of a call's rows: n_pages pages of `page` bytes at `pool`.
favor_status check_pages(const char* fn, const void* pool, const int* pages, int n_pages, int B, size_t page,
                         bool required) {
    if (!pool) {
        if (required) return set_error(FAVOR_ERR_INVALID_ARG, "%s: null state pointer", fn);
        if (pages) return set_error(FAVOR_ERR_INVALID_ARG, "%s: pages without a state", fn);
        return FAVOR_OK;
    }
    if (n_pages < 1) return set_error(FAVOR_ERR_INVALID_ARG, "%s: n_pages=%d must be >= 1", fn, n_pages);
    if (!pages && n_pages < B)
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: n_pages=%d is below B=%d and no pages are given", fn, n_pages, B);
    if ((size_t)n_pages > ((size_t)1 << 42) / page)
        return set_error(FAVOR_ERR_UNSUPPORTED, "%s: pool of more than 2^42 bytes", fn);
    return FAVOR_OK;
}

// Whether every tensor starts on an element of it.
bool aligned(size_t es, std::initializer_list<const void*> tensors, std::initializer_list<const void*> words) {
    for (const void* p : tensors)
        if (reinterpret_cast<uintptr_t>(p) % es) return false;
    for (const void* p : words)
        if (reinterpret_cast<uintptr_t>(p) % 4) return false;
    return true;
}

}  // namespace

extern "C" {

favor_status favor_ssm_create(favor_ssm* out, int D, int N, int G, int K, favor_dtype dtype, int max_B, int max_L,
                              int training) {
    set_error(FAVOR_OK, "%s", "");
    if (!out) return set_error(FAVOR_ERR_INVALID_ARG, "favor_ssm_create: out is NULL");
    *out = nullptr;
    if (D < 1 || N < 1 || G < 1 || K < 1 || max_B < 1 || max_L < 1)
        return set_error(FAVOR_ERR_INVALID_ARG,
                         "favor_ssm_create: sizes must be >= 1 (D=%d N=%d G=%d K=%d max_B=%d max_L=%d)", D, N, G, K,
                         max_B, max_L);
    if (dtype != FAVOR_DTYPE_F32 && dtype != FAVOR_DTYPE_BF16)
        return set_error(FAVOR_ERR_INVALID_ARG, "favor_ssm_create: unknown dtype %d", (int)dtype);
    if (D % G) return set_error(FAVOR_ERR_INVALID_ARG, "favor_ssm_create: D=%d is not a multiple of G=%d", D, G);
    if (N != 8 && N != 16 && N != 32 && N != 64)
        return set_error(FAVOR_ERR_UNSUPPORTED, "favor_ssm_create: N=%d (supported: 8, 16, 32, 64)", N);
    if (K < 2 || K > 4) return set_error(FAVOR_ERR_UNSUPPORTED, "favor_ssm_create: K=%d (supported: 2, 3, 4)", K);
    if (D > (1 << 20) || (long long)max_B * max_L > (1LL << 30) || (long long)max_B * max_L > (1LL << 36) / D)
        return set_error(FAVOR_ERR_UNSUPPORTED, "favor_ssm_create: D or max_B*max_L*D too large");
    if ((long long)max_B * D > (1LL << 30) || (long long)max_B * N > (1LL << 36) / D || (long long)max_B * max_L * N > (1LL << 36) / G)
        return set_error(FAVOR_ERR_UNSUPPORTED, "favor_ssm_create: max_B*D, max_B*D*N or max_B*max_L*G*N too large");
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return set_error(FAVOR_ERR_CUDA, "favor_ssm_create: no usable CUDA device");
    }
    SsmHandle* h = new (std::nothrow) SsmHandle();
    if (!h) return set_error(FAVOR_ERR_NOMEM, "favor_ssm_create: host allocation failed");
    h->D = D; h->N = N; h->G = G; h->K = K; h->dtype = dtype; h->max_B = max_B; h->max_L = max_L;
    h->training = training != 0;
    h->device = dev;
    cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, dev);
    if (h->num_sms < 1) h->num_sms = 1;
    h->ws_floats = scan_prompt_ws(*h);
    if (h->training) {
        const size_t b = scan_backward_ws(*h), c = conv_backward_ws(*h);
        if (b > h->ws_floats) h->ws_floats = b;
        if (c > h->ws_floats) h->ws_floats = c;
    }
    const cudaError_t e = cudaMalloc(&h->ws, h->ws_floats * sizeof(float));
    if (e != cudaSuccess) {
        const favor_status st = e == cudaErrorMemoryAllocation ? FAVOR_ERR_NOMEM : FAVOR_ERR_CUDA;
        set_error(st, "favor_ssm_create: cudaMalloc of %zu bytes: %s", h->ws_floats * sizeof(float),
                  cudaGetErrorString(e));
        cudaGetLastError();
        delete h;
        return st;
    }
    *out = reinterpret_cast<favor_ssm>(h);
    return FAVOR_OK;
}

favor_status favor_ssm_destroy(favor_ssm hd) {
    if (!hd) return FAVOR_OK;
    SsmHandle* h = reinterpret_cast<SsmHandle*>(hd);
    int cur = 0;
    cudaGetDevice(&cur);
    if (cur != h->device) cudaSetDevice(h->device);
    cudaDeviceSynchronize();
    cudaFree(h->ws);
    if (cur != h->device) cudaSetDevice(cur);
    delete h;
    cudaGetLastError();
    return FAVOR_OK;
}

static favor_status conv_call(const char* fn, favor_ssm hd, const void* x, const float* weight, const float* bias,
                              int silu, void* window, const int* pages, int n_pages, const int* lens, void* out,
                              int B, int L, bool step, void* stream) {
    favor_status st = check_call(fn, hd, B, L);
    if (st != FAVOR_OK) return st;
    const SsmHandle& h = *reinterpret_cast<const SsmHandle*>(hd);
    if (!x || !weight || !out) return set_error(FAVOR_ERR_INVALID_ARG, "%s: null pointer", fn);
    const size_t es = esize(h), page = (size_t)(h.K - 1) * h.D * es, n = (size_t)B * L * h.D * es;
    st = check_pages(fn, window, pages, n_pages, B, page, step);
    if (st != FAVOR_OK) return st;
    if (!aligned(es, {x, out, window}, {weight, bias, pages, lens}))
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: a pointer is not aligned to its element", fn);
    const Span outs[] = {{out, n}, {window, window ? page * n_pages : 0}};
    const Span ins[] = {{x, n}, {weight, (size_t)h.D * h.K * 4}, {bias, (size_t)h.D * 4},
                        {pages, (size_t)B * 4}, {lens, (size_t)B * 4}};
    if (any_overlap(outs, 2, ins, 5))
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: out and window must not overlap another argument", fn);
    ConvArgs a = {};
    a.x = x; a.weight = weight; a.bias = bias; a.window = window; a.pg = {pages, n_pages}; a.lens = lens; a.out = out;
    a.B = B; a.L = L; a.silu = silu != 0;
    return (step ? conv_step : conv_prompt)(h, a, reinterpret_cast<cudaStream_t>(stream));
}

favor_status favor_conv_causal(favor_ssm h, const void* x, const float* weight, const float* bias, int silu,
                               void* window, const int* pages, int n_pages, const int* lens, void* out, int B, int L,
                               void* stream) {
    return conv_call("favor_conv_causal", h, x, weight, bias, silu, window, pages, n_pages, lens, out, B, L, false,
                     stream);
}

favor_status favor_conv_causal_step(favor_ssm h, const void* x, const float* weight, const float* bias, int silu,
                                    void* window, const int* pages, int n_pages, void* out, int B, void* stream) {
    return conv_call("favor_conv_causal_step", h, x, weight, bias, silu, window, pages, n_pages, nullptr, out, B, 1,
                     true, stream);
}

favor_status favor_conv_causal_backward(favor_ssm hd, const void* x, const float* weight, const float* bias, int silu,
                                        const int* lens, const void* dout, void* dx, float* dweight, float* dbias,
                                        int B, int L, void* stream) {
    const char* fn = "favor_conv_causal_backward";
    favor_status st = check_call(fn, hd, B, L);
    if (st != FAVOR_OK) return st;
    const SsmHandle& h = *reinterpret_cast<const SsmHandle*>(hd);
    if (!x || !weight || !dout || !dx || !dweight) return set_error(FAVOR_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!h.training) return set_error(FAVOR_ERR_UNSUPPORTED, "%s: the handle was created without training", fn);
    const size_t es = esize(h), n = (size_t)B * L * h.D * es;
    if (!aligned(es, {x, dout, dx}, {weight, bias, lens, dweight, dbias}))
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: a pointer is not aligned to its element", fn);
    const Span outs[] = {{dx, n}, {dweight, (size_t)h.D * h.K * 4}, {dbias, (size_t)h.D * 4}};
    const Span ins[] = {{x, n}, {dout, n}, {weight, (size_t)h.D * h.K * 4}, {bias, (size_t)h.D * 4},
                        {lens, (size_t)B * 4}};
    if (any_overlap(outs, 3, ins, 5))
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: the gradients must not overlap another argument", fn);
    ConvArgs a = {};
    a.x = x; a.weight = weight; a.bias = bias; a.lens = lens; a.dout = dout; a.dx = dx; a.dweight = dweight;
    a.dbias = dbias; a.B = B; a.L = L; a.silu = silu != 0;
    std::lock_guard<std::mutex> lk(h.enqueue);
    return conv_backward(h, a, reinterpret_cast<cudaStream_t>(stream));
}

static favor_status scan_call(const char* fn, favor_ssm hd, const ScanArgs& a, bool step, void* stream) {
    favor_status st = check_call(fn, hd, a.B, a.L);
    if (st != FAVOR_OK) return st;
    const SsmHandle& h = *reinterpret_cast<const SsmHandle*>(hd);
    if (!a.u || !a.dt || !a.A || !a.Bm || !a.Cm || !a.out)
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: null pointer", fn);
    const size_t es = esize(h), page = (size_t)h.D * h.N * 4, n = (size_t)a.B * a.L * h.D * es;
    const size_t nb = (size_t)a.B * a.L * h.G * h.N * es;
    st = check_pages(fn, a.state, a.pg.pages, a.pg.n_pages, a.B, page, step);
    if (st != FAVOR_OK) return st;
    if (a.state && !is_aligned16(a.state))
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: state must be 16-byte aligned", fn);
    if (!aligned(es, {a.u, a.dt, a.Bm, a.Cm, a.z, a.out}, {a.A, a.skip, a.dt_bias, a.pg.pages, a.lens}))
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: a pointer is not aligned to its element", fn);
    const Span outs[] = {{a.out, n}, {a.state, a.state ? page * a.pg.n_pages : 0}};
    const Span ins[] = {{a.u, n}, {a.dt, n}, {a.z, n}, {a.Bm, nb}, {a.Cm, nb}, {a.A, page},
                        {a.skip, (size_t)h.D * 4}, {a.dt_bias, (size_t)h.D * 4}, {a.pg.pages, (size_t)a.B * 4},
                        {a.lens, (size_t)a.B * 4}};
    if (any_overlap(outs, 2, ins, 10))
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: out and state must not overlap another argument", fn);
    if (step) return scan_step(h, a, reinterpret_cast<cudaStream_t>(stream));
    std::lock_guard<std::mutex> lk(h.enqueue);
    return scan_prompt(h, a, reinterpret_cast<cudaStream_t>(stream));
}

favor_status favor_ssm_scan(favor_ssm h, const void* u, const void* dt, const float* A, const void* Bm, const void* Cm,
                            const float* skip, const void* z, const float* dt_bias, float* state, const int* pages,
                            int n_pages, const int* lens, void* out, int B, int L, void* stream) {
    ScanArgs a = {};
    a.u = u; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.skip = skip; a.z = z; a.dt_bias = dt_bias; a.state = state;
    a.pg = {pages, n_pages}; a.lens = lens; a.out = out; a.B = B; a.L = L;
    return scan_call("favor_ssm_scan", h, a, false, stream);
}

favor_status favor_ssm_scan_step(favor_ssm h, const void* u, const void* dt, const float* A, const void* Bm,
                                 const void* Cm, const float* skip, const void* z, const float* dt_bias, float* state,
                                 const int* pages, int n_pages, void* out, int B, void* stream) {
    ScanArgs a = {};
    a.u = u; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.skip = skip; a.z = z; a.dt_bias = dt_bias; a.state = state;
    a.pg = {pages, n_pages}; a.out = out; a.B = B; a.L = 1;
    return scan_call("favor_ssm_scan_step", h, a, true, stream);
}

favor_status favor_ssm_scan_backward(favor_ssm hd, const void* u, const void* dt, const float* A, const void* Bm,
                                     const void* Cm, const float* skip, const void* z, const float* dt_bias,
                                     const int* lens, const void* dout, void* du, void* ddt, float* dA, void* dB,
                                     void* dC, float* dskip, void* dz, float* ddt_bias, int B, int L, void* stream) {
    const char* fn = "favor_ssm_scan_backward";
    favor_status st = check_call(fn, hd, B, L);
    if (st != FAVOR_OK) return st;
    const SsmHandle& h = *reinterpret_cast<const SsmHandle*>(hd);
    if (!u || !dt || !A || !Bm || !Cm || !dout || !du || !ddt || !dA || !dB || !dC)
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!skip != !dskip || !z != !dz || !dt_bias != !ddt_bias)
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: dskip, dz and ddt_bias go with skip, z and dt_bias", fn);
    if (!h.training) return set_error(FAVOR_ERR_UNSUPPORTED, "%s: the handle was created without training", fn);
    const size_t es = esize(h), n = (size_t)B * L * h.D * es, nb = (size_t)B * L * h.G * h.N * es;
    const size_t pa = (size_t)h.D * h.N * 4, pd = (size_t)h.D * 4;
    const Span outs[] = {{du, n}, {ddt, n}, {dz, n}, {dB, nb}, {dC, nb}, {dA, pa}, {dskip, pd}, {ddt_bias, pd}};
    const Span ins[] = {{u, n}, {dt, n}, {z, n}, {dout, n}, {Bm, nb}, {Cm, nb}, {A, pa}, {skip, pd}, {dt_bias, pd},
                        {lens, (size_t)B * 4}};
    if (!aligned(es, {u, dt, z, dout, Bm, Cm, du, ddt, dz, dB, dC}, {A, skip, dt_bias, lens, dA, dskip, ddt_bias}))
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: a pointer is not aligned to its element", fn);
    if (any_overlap(outs, 8, ins, 10))
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: the gradients must not overlap another argument", fn);
    ScanArgs a = {};
    a.u = u; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.skip = skip; a.z = z; a.dt_bias = dt_bias; a.lens = lens;
    a.dout = dout; a.du = du; a.ddt = ddt; a.dA = dA; a.dB = dB; a.dC = dC; a.dskip = dskip; a.dz = dz;
    a.ddt_bias = ddt_bias; a.B = B; a.L = L;
    std::lock_guard<std::mutex> lk(h.enqueue);
    return scan_backward(h, a, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
