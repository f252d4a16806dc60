// Host side of the gated linear recurrence: argument checks, handle lifetime,
// workspace.  Every check runs before anything is enqueued.
#include <mutex>
#include <new>

#include "call_checks.h"
#include "recur_internal.h"

using namespace favor;

namespace {

size_t esize(const RecurHandle& h) { return h.dtype == FAVOR_DTYPE_F32 ? 4 : 2; }

// Channels that an access to a row takes: 4 or 2 where D and every tensor allow it.
int row_width(const RecurHandle& h, std::initializer_list<const void*> tensors) {
    uintptr_t bits = (uintptr_t)h.D * esize(h);
    for (const void* p : tensors) bits |= reinterpret_cast<uintptr_t>(p);
    return bits % (4 * esize(h)) == 0 ? 4 : bits % (2 * esize(h)) == 0 ? 2 : 1;
}

favor_status check_gates(const char* fn, const RecurArgs& a) {
    if (!a.x || !a.r) return set_error(FAVOR_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (a.i_bias && !a.i) return set_error(FAVOR_ERR_INVALID_ARG, "%s: i_bias without i", fn);
    return FAVOR_OK;
}

favor_status scan_call(const char* fn, favor_recur hd, RecurArgs& a, bool step, void* stream) {
    favor_status st = check_handle_call(fn, reinterpret_cast<const RecurHandle*>(hd), a.B, a.L);
    if (st != FAVOR_OK) return st;
    const RecurHandle& h = *reinterpret_cast<const RecurHandle*>(hd);
    st = check_gates(fn, a);
    if (st != FAVOR_OK) return st;
    if (!a.out) return set_error(FAVOR_ERR_INVALID_ARG, "%s: null pointer", fn);
    const size_t es = esize(h), n = (size_t)a.B * a.L * h.D * es, page = (size_t)h.D * 4, rows = (size_t)a.B * 4;
    st = check_pages(fn, a.state, a.pg.pages, a.pg.n_pages, a.B, page, step);
    if (st != FAVOR_OK) return st;
    if (!aligned(es, {a.x, a.r, a.i, a.z, a.out}, {a.state, a.rate, a.r_bias, a.i_bias, a.pg.pages, a.lens}))
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: a pointer is not aligned to its element", fn);
    const Span outs[] = {{a.out, n}, {a.state, a.state ? page * a.pg.n_pages : 0}};
    const Span ins[] = {{a.x, n}, {a.r, n}, {a.i, n}, {a.z, n}, {a.rate, page}, {a.r_bias, page}, {a.i_bias, page},
                        {a.pg.pages, rows}, {a.lens, rows}};
    if (any_overlap(outs, 2, ins, 9))
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: out and state must not overlap another argument", fn);
    a.width = row_width(h, {a.x, a.r, a.i, a.z, a.out});
    if (step) return recur_step(h, a, reinterpret_cast<cudaStream_t>(stream));
    std::lock_guard<std::mutex> lk(h.enqueue);
    return recur_scan(h, a, reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

favor_status favor_recur_create(favor_recur* out, int D, favor_recur_scale scale, favor_dtype dtype, int max_B,
                                int max_L, int training) {
    const char* fn = "favor_recur_create";
    set_error(FAVOR_OK, "%s", "");
    if (!out) return set_error(FAVOR_ERR_INVALID_ARG, "%s: out is NULL", fn);
    *out = nullptr;
    if (D < 1 || max_B < 1 || max_L < 1)
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: sizes must be >= 1 (D=%d max_B=%d max_L=%d)", fn, D, max_B, max_L);
    if (dtype != FAVOR_DTYPE_F32 && dtype != FAVOR_DTYPE_BF16)
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
    if (scale != FAVOR_RECUR_PLAIN && scale != FAVOR_RECUR_MEAN && scale != FAVOR_RECUR_UNIT)
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: unknown scale %d", fn, (int)scale);
    if (D > (1 << 20) || (long long)max_B * max_L > (1LL << 30) || (long long)max_B * max_L > (1LL << 36) / D ||
        (long long)max_B * D > (1LL << 30))
        return set_error(FAVOR_ERR_UNSUPPORTED, "%s: D, max_B*max_L, max_B*D or max_B*max_L*D too large", fn);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return set_error(FAVOR_ERR_CUDA, "%s: no usable CUDA device", fn);
    }
    RecurHandle* h = new (std::nothrow) RecurHandle();
    if (!h) return set_error(FAVOR_ERR_NOMEM, "%s: host allocation failed", fn);
    h->D = D; h->scale = scale; h->dtype = dtype; h->max_B = max_B; h->max_L = max_L; h->training = training != 0;
    h->device = dev;
    cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, dev);
    if (h->num_sms < 1) h->num_sms = 1;
    h->ws_floats = recur_scan_ws(*h);
    if (h->training && recur_backward_ws(*h) > h->ws_floats) h->ws_floats = recur_backward_ws(*h);
    h->ws = nullptr;
    const cudaError_t e = h->ws_floats ? cudaMalloc(&h->ws, h->ws_floats * sizeof(float)) : cudaSuccess;
    if (e != cudaSuccess) {
        const favor_status st = e == cudaErrorMemoryAllocation ? FAVOR_ERR_NOMEM : FAVOR_ERR_CUDA;
        set_error(st, "%s: cudaMalloc of %zu bytes: %s", fn, h->ws_floats * sizeof(float), cudaGetErrorString(e));
        cudaGetLastError();
        delete h;
        return st;
    }
    *out = reinterpret_cast<favor_recur>(h);
    return FAVOR_OK;
}

favor_status favor_recur_destroy(favor_recur hd) {
    if (!hd) return FAVOR_OK;
    RecurHandle* h = reinterpret_cast<RecurHandle*>(hd);
    int cur = 0;
    cudaGetDevice(&cur);
    if (cur != h->device) cudaSetDevice(h->device);
    cudaDeviceSynchronize();
    if (h->ws) cudaFree(h->ws);
    if (cur != h->device) cudaSetDevice(cur);
    delete h;
    cudaGetLastError();
    return FAVOR_OK;
}

favor_status favor_recur_scan(favor_recur h, const void* x, const void* r, const void* i, const float* rate,
                              const float* r_bias, const float* i_bias, const void* z, float* state, const int* pages,
                              int n_pages, const int* lens, int clear, void* out, int B, int L, void* stream) {
    RecurArgs a = {};
    a.clear = clear != 0;
    a.x = x; a.r = r; a.i = i; a.rate = rate; a.r_bias = r_bias; a.i_bias = i_bias; a.z = z; a.state = state;
    a.pg = {pages, n_pages}; a.lens = lens; a.out = out; a.B = B; a.L = L;
    return scan_call("favor_recur_scan", h, a, false, stream);
}

favor_status favor_recur_step(favor_recur h, const void* x, const void* r, const void* i, const float* rate,
                              const float* r_bias, const float* i_bias, const void* z, float* state, const int* pages,
                              int n_pages, void* out, int B, void* stream) {
    RecurArgs a = {};
    a.x = x; a.r = r; a.i = i; a.rate = rate; a.r_bias = r_bias; a.i_bias = i_bias; a.z = z; a.state = state;
    a.pg = {pages, n_pages}; a.out = out; a.B = B; a.L = 1;
    return scan_call("favor_recur_step", h, a, true, stream);
}

favor_status favor_recur_backward(favor_recur hd, const void* x, const void* r, const void* i, const float* rate,
                                  const float* r_bias, const float* i_bias, const void* z, const int* lens,
                                  const void* dout, void* dx, void* dr, void* di, float* drate, float* dr_bias,
                                  float* di_bias, void* dz, int B, int L, void* stream) {
    const char* fn = "favor_recur_backward";
    favor_status st = check_handle_call(fn, reinterpret_cast<const RecurHandle*>(hd), B, L);
    if (st != FAVOR_OK) return st;
    const RecurHandle& h = *reinterpret_cast<const RecurHandle*>(hd);
    RecurArgs a = {};
    a.x = x; a.r = r; a.i = i; a.rate = rate; a.r_bias = r_bias; a.i_bias = i_bias; a.z = z; a.lens = lens;
    a.dout = dout; a.dx = dx; a.dr = dr; a.di = di; a.drate = drate; a.dr_bias = dr_bias; a.di_bias = di_bias;
    a.dz = dz; a.B = B; a.L = L;
    st = check_gates(fn, a);
    if (st != FAVOR_OK) return st;
    if (!dout || !dx || !dr) return set_error(FAVOR_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!i != !di || !rate != !drate || !r_bias != !dr_bias || !i_bias != !di_bias || !z != !dz)
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: di, drate, dr_bias, di_bias and dz go with their inputs", fn);
    if (!h.training) return set_error(FAVOR_ERR_UNSUPPORTED, "%s: the handle was created without training", fn);
    const size_t es = esize(h), n = (size_t)B * L * h.D * es, pd = (size_t)h.D * 4;
    if (!aligned(es, {x, r, i, z, dout, dx, dr, di, dz}, {rate, r_bias, i_bias, lens, drate, dr_bias, di_bias}))
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: a pointer is not aligned to its element", fn);
    const Span outs[] = {{dx, n}, {dr, n}, {di, n}, {dz, n}, {drate, pd}, {dr_bias, pd}, {di_bias, pd}};
    const Span ins[] = {{x, n}, {r, n}, {i, n}, {z, n}, {dout, n}, {rate, pd}, {r_bias, pd}, {i_bias, pd},
                        {lens, (size_t)B * 4}};
    if (any_overlap(outs, 7, ins, 9))
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: the gradients must not overlap another argument", fn);
    a.width = row_width(h, {x, r, i, z, dout, dx, dr, di, dz});
    std::lock_guard<std::mutex> lk(h.enqueue);
    return recur_backward(h, a, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
