// Internal declarations of the gated linear recurrence: the handle, the launch
// arguments, and the device code that the scan and its gradients share.
#pragma once

#include "pairs.cuh"

namespace favor {

struct RecurHandle {
    int D;
    favor_recur_scale scale;
    favor_dtype dtype;
    int max_B, max_L;
    bool training;          // the gradients' workspace exists
    int device, num_sms;
    float* ws;
    size_t ws_floats;
    // Held while a call that uses ws is enqueued: it is several launches.
    mutable std::mutex enqueue;
};

struct RecurArgs {
    const void *x, *r, *i, *z;                  // [B][L][D]; i, z may be null
    const float *rate, *r_bias, *i_bias;        // [D] or null
    float* state;                               // [n_pages][D] or null (zero start, end not kept)
    PageArgs pg;
    const int* lens;
    void* out;
    bool clear;                                 // zeros in out behind a row's end
    const void* dout;                           // gradients
    void *dx, *dr, *di, *dz;                    // di, dz null where i, z are
    float *drate, *dr_bias, *di_bias;           // null where the parameter is
    int B, L;
    int width;                                  // channels that an access to a row takes: 4, 2 or 1
};

favor_status recur_scan(const RecurHandle& h, const RecurArgs& a, cudaStream_t st);
favor_status recur_step(const RecurHandle& h, const RecurArgs& a, cudaStream_t st);
favor_status recur_backward(const RecurHandle& h, const RecurArgs& a, cudaStream_t st);
// Workspace (floats) the calls of a handle with these sizes can need.
size_t recur_scan_ws(const RecurHandle& h);
size_t recur_backward_ws(const RecurHandle& h);

// A row of tokens is cut into chunks, a block each, and a chunk into kRecWarps runs, a warp each; a warp walks its run
// rec_group tokens at a time.  A lane has 4 channels, a warp a slab of 128.
constexpr int kRecWarps = 8, kRecThreads = 32 * kRecWarps, kRecSlab = 128;
template <typename T>
__host__ __device__ constexpr int rec_group() { return sizeof(T) == 2 ? 4 : 2; }
constexpr int kRecGroupMax = 4, kRecRunMin = 8, kRecChunksMax = 64;

struct RecurPlan {
    int slabs;      // of channels
    int run;        // tokens of a run, a multiple of kRecGroupMax
    int chunks;     // of a row
};

// ------------------------------------------------------------------ the gates
// A lane's parameters.  `slow`: all rates of the warp are in [0, kSlowRate), and so is every y = rate s.
constexpr float kSlowRate = 0.125f;
struct RecurChan {
    F2 rate, r_bias, i_bias;        // the biases as sigmoid_bias gives them
    bool slow;
};

// A token's decay a is kept as d: where 0 <= 1 - a < 1/2, d = -(1 - a), and a h + b is h + (d h + b); else d = a
// (+0 or more), and it is d h + b.  d's sign bit tells them apart, so a token that loses nothing has -0.  Next to 1,
// fp32 holds 1 - a to many more digits than a, which would be 2^-25 off at every token, 2^-25 / (1 - a) of a state
// that lives 1 / (1 - a) tokens.  SLOW: the first kind alone.
template <bool SLOW>
__device__ __forceinline__ F2 recur_next(F2 d, F2 h, F2 b) {
    const F2 t = fma2(d, h, b);
    if (SLOW) return h + t;
    const float x = h.x(), y = h.y();
    return t + F2(__float_as_int(d.x()) < 0 ? x : 0.f, __float_as_int(d.y()) < 0 ? y : 0.f);
}
// a h.
template <bool SLOW>
__device__ __forceinline__ F2 recur_scale(F2 d, F2 h) {
    if (SLOW) return fma2(d, h, h);
    const float x = h.x(), y = h.y();
    return fma2(d, h, F2(__float_as_int(d.x()) < 0 ? x : 0.f, __float_as_int(d.y()) < 0 ? y : 0.f));
}
constexpr float kKeep = -0.f;       // d of a token that changes nothing

struct RecurGate {
    F2 d, w;            // the decay, the input's weight
    F2 s, sn;           // sigmoid(r'); gradients: sigmoid(-r')
    F2 a, rw;           // gradients: the decay itself, 1 / w (0 where w is)
};

// c = 1 - e^-y, d and a of one value of y.  Below 0.35 the series y - y^2/2 + .. + y^7/7!, the rest of which is
// under 0.35^7 / 8! = 2e-8 of it.
__device__ __forceinline__ void any_decay(float y, float& c, float& d, float& a) {
    float p = fmaf(y, 1.f / 5040, -1.f / 720);
    p = fmaf(y, p, 1.f / 120);
    p = fmaf(y, p, -1.f / 24);
    p = fmaf(y, p, 1.f / 6);
    p = fmaf(y, p, -1.f / 2);
    p = fmaf(y, p, 1.f);
    const float e = ex2_approx(-y * kLog2e);
    c = fabsf(y) < 0.35f ? y * p : 1.f - e;
    const bool near = c >= 0.f && c < 0.5f;
    d = near ? -fabsf(c) : e;      // a rate of -0, or one below 0 under a closed gate, makes c a -0
    a = near ? 1.f - c : e;
}

template <typename T, bool RATE, int SCALE, bool SLOW, bool GRAD>
__device__ __forceinline__ RecurGate recur_gate(F2 r, const RecurChan& p) {
    RecurGate g;
    if (!RATE || GRAD) sigmoids2<T, true>(r, p.r_bias, g.s, g.sn);
    else g.s = sigmoid2<T>(r, p.r_bias);
    if (SLOW) {
        // -c by the series to y^5/5!, the rest of which is under 0.125^5 / 6! = 4e-8 of it
        const F2 y = p.rate * g.s;
        F2 q = fma2(y, both(-1.f / 120), both(1.f / 24));
        q = fma2(y, q, both(-1.f / 6));
        q = fma2(y, q, both(1.f / 2));
        q = fma2(y, q, both(-1.f));
        g.d = y * q;
        if (GRAD) g.a = g.d + both(1.f);
        if (SCALE == FAVOR_RECUR_MEAN) g.w = g.d * both(-1.f);
        if (SCALE == FAVOR_RECUR_UNIT) {    // 1 - a^2 = c (2 - c) = -(d + d + d d)
            const F2 m = fma2(g.d, g.d, g.d + g.d);
            if (GRAD) {
                g.rw = each(m, [](float v) { return -v < 1.1754944e-38f ? 0.f : rsqrt_approx(-v); });
                g.w = m * both(-1.f) * g.rw;
            } else {
                g.w = each(m, [](float v) { return sqrt_approx(-v); });
            }
        }
        return g;
    }
    float c[2], d[2], a[2];
    if (RATE) {
        const F2 y = p.rate * g.s;
        any_decay(y.x(), c[0], d[0], a[0]);
        any_decay(y.y(), c[1], d[1], a[1]);
    } else {
        c[0] = g.sn.x(), c[1] = g.sn.y();
        a[0] = g.s.x(), a[1] = g.s.y();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            d[k] = c[k] < 0.5f ? -c[k] : a[k];
            a[k] = c[k] < 0.5f ? 1.f - c[k] : a[k];
        }
    }
    g.d = F2(d[0], d[1]);
    g.a = F2(a[0], a[1]);
    if (SCALE == FAVOR_RECUR_MEAN) g.w = F2(c[0], c[1]);
    if (SCALE == FAVOR_RECUR_UNIT) {        // 0 where 1 - a^2 is not positive, or flushed to 0
        float w[2], rw[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float q = c[k] * (2.f - c[k]);
            rw[k] = q < 1.1754944e-38f ? 0.f : rsqrt_approx(q);
            w[k] = q * rw[k];
        }
        g.w = F2(w[0], w[1]);
        g.rw = F2(rw[0], rw[1]);
    }
    return g;
}

// ------------------------------------------------------------------ a warp's rows
// Two pairs of channels.
struct F4 {
    F2 a, b;
};
// Four channels as they are stored.
template <typename T>
struct Raw4;
template <>
struct Raw4<__nv_bfloat16> {
    typedef uint2 V;
    typedef uint32_t H;     // two of them
};
template <>
struct Raw4<float> {
    typedef float4 V;
    typedef float2 H;
};
__device__ __forceinline__ F4 to_f4(uint2 u) { return {to_f2(u.x), to_f2(u.y)}; }
__device__ __forceinline__ F4 to_f4(float4 u) { return {F2(u.x, u.y), F2(u.z, u.w)}; }
__device__ __forceinline__ F2 to_f2(uint2 u, int half) { return to_f2(half ? u.y : u.x); }
__device__ __forceinline__ F2 to_f2(float4 u, int half) { return half ? F2(u.z, u.w) : F2(u.x, u.y); }
__device__ __forceinline__ uint2 raw_of(uint32_t a, uint32_t b) { return make_uint2(a, b); }
__device__ __forceinline__ float4 raw_of(float2 a, float2 b) { return make_float4(a.x, a.y, b.x, b.y); }
template <typename T>
__device__ __forceinline__ typename Raw4<T>::V from_f4(const F4& x) {
    return raw_of(from_f2(x.a, T()), from_f2(x.b, T()));
}
// What a lane needs to walk rows: its four channels, which are neighbours where rows are moved 4 channels at a time,
// else two pairs 64 channels apart, or 32 channels apart one by one, so that a warp's accesses stay whole; those
// that are not there (at D and behind) count for nothing.  [4, 4096, 1001] bf16 123 us (neighbours read one by one,
// each in a branch of its own, 256 at the time), gradients 335 (642); [4, 4096, 1024] 62 and 154.
struct RecurLane {
    int D, width, c;    // c: the first channel
    bool quads;
    int at;             // quads: c, or 0 for a lane without channels
    __device__ __forceinline__ RecurLane(const RecurArgs& a, int D_, int slab) : D(D_), width(a.width) {
        c = slab * kRecSlab + (threadIdx.x & 31) * width;
        quads = width == 4;
        at = c < D ? c : 0;
    }
    __device__ __forceinline__ int chan(int k) const {
        return c + (k >> 1) * (quads ? 2 : 64) + (k & 1) * (width == 1 ? 32 : 1);
    }
    __device__ __forceinline__ bool has(int k) const { return chan(k) < D; }
    // chan(k), or the place of the row's last n channels
    __device__ __forceinline__ int last(int k, int n) const { return min(chan(k), D - n); }
};
// A row's channels where they are not quads; p is the row.  Without a branch, so that a group's loads are on their way
// together: for a channel that is not there the row's last one is read.
__device__ __forceinline__ uint2 raw_part(const __nv_bfloat16* p, const RecurLane& l) {
    if (l.width == 2)
        return make_uint2(*reinterpret_cast<const uint32_t*>(p + l.last(0, 2)),
                          *reinterpret_cast<const uint32_t*>(p + l.last(2, 2)));
    const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
    const uint32_t a = q[l.last(0, 1)], b = q[l.last(1, 1)], c = q[l.last(2, 1)], d = q[l.last(3, 1)];
    return make_uint2(a | b << 16, c | d << 16);
}
__device__ __forceinline__ float4 raw_part(const float* p, const RecurLane& l) {
    return make_float4(p[l.last(0, 1)], p[l.last(1, 1)], p[l.last(2, 1)], p[l.last(3, 1)]);
}
__device__ __forceinline__ void raw_store(__nv_bfloat16* p, const RecurLane& l, uint2 u) {
    if (l.width == 2) {
        if (l.has(0)) *reinterpret_cast<uint32_t*>(p + l.chan(0)) = u.x;
        if (l.has(2)) *reinterpret_cast<uint32_t*>(p + l.chan(2)) = u.y;
        return;
    }
    unsigned short* q = reinterpret_cast<unsigned short*>(p);
    const uint32_t v[4] = {u.x & 0xffff, u.x >> 16, u.y & 0xffff, u.y >> 16};
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (l.has(k)) q[l.chan(k)] = (unsigned short)v[k];
}
__device__ __forceinline__ void raw_store(float* p, const RecurLane& l, float4 u) {
    const float v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (l.has(k)) p[l.chan(k)] = v[k];
}

template <typename T>
struct RecurRows {
    typename Raw4<T>::V v[rec_group<T>()];
    __device__ __forceinline__ F4 operator()(int s) const { return to_f4(v[s]); }
    __device__ __forceinline__ F2 operator()(int s, int half) const { return to_f2(v[s], half); }
};
// Rows [t, t + rec_group) of a tensor's batch row, the lane's channels.  AGAIN: they will be read once more.
// WHOLE: all are in front of `end`, and of quads (a lane without channels reads the row's first ones).  Else
// the last row in front of `end` stands for those at `end` and behind (t itself is in front).
template <typename T, bool AGAIN, bool WHOLE, int N = rec_group<T>()>
__device__ __forceinline__ void load_rows(const T* row0, const RecurLane& l, int t, int end, RecurRows<T>& r) {
    typedef typename Raw4<T>::V V;
    const T* p = row0 + (size_t)t * l.D + (WHOLE ? l.at : 0);
#pragma unroll
    for (int s = 0; s < N; ++s) {
        if (!WHOLE) r.v[s] = raw_part(p, l);
        else r.v[s] = AGAIN ? __ldg(reinterpret_cast<const V*>(p)) : __ldcs(reinterpret_cast<const V*>(p));
        if (WHOLE || t + s + 1 < end) p += l.D;
    }
}
template <typename T, bool WHOLE>
__device__ __forceinline__ void write_raw(T* row0, const RecurLane& l, int t, typename Raw4<T>::V u) {
    T* p = row0 + (size_t)t * l.D;
    if (!WHOLE) raw_store(p, l, u);
    else if (l.c < l.D) __stcs(reinterpret_cast<typename Raw4<T>::V*>(p + l.c), u);
}
template <typename T, bool WHOLE>
__device__ __forceinline__ void write_row(T* row0, const RecurLane& l, int t, const F4& x) {
    write_raw<T, WHOLE>(row0, l, t, from_f4<T>(x));
}
template <typename T>
__device__ __forceinline__ void clear_rows(T* row0, const RecurLane& l, int t, int end) {
    const F4 none = {both(0.f), both(0.f)};
    for (; t < end; ++t) {
        if (l.quads) write_row<T, true>(row0, l, t, none);
        else write_row<T, false>(row0, l, t, none);
    }
}
// 4 floats a lane of a [D] vector.
__device__ __forceinline__ F4 load_vec(const float* p, const RecurLane& l) {
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = p && l.has(k) ? p[l.chan(k)] : 0.f;
    return {F2(v[0], v[1]), F2(v[2], v[3])};
}
__device__ __forceinline__ void store_vec(float* p, const RecurLane& l, const F4& x) {
    const float v[4] = {x.a.x(), x.a.y(), x.b.x(), x.b.y()};
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (l.has(k)) p[l.chan(k)] = v[k];
}

struct RecurChan4 {
    RecurChan a, b;
};
template <typename T>
__device__ __forceinline__ RecurChan4 load_chans(const RecurArgs& a, const RecurLane& l) {
    const F4 rate = load_vec(a.rate, l), rb = load_vec(a.r_bias, l), ib = load_vec(a.i_bias, l);
    RecurChan4 p;
    p.a = {rate.a, sigmoid_bias<T>(rb.a), sigmoid_bias<T>(ib.a), false};
    p.b = {rate.b, sigmoid_bias<T>(rb.b), sigmoid_bias<T>(ib.b), false};
    auto slow = [](float v) { return v >= 0.f && v < kSlowRate; };
    const bool mine = slow(rate.a.x()) && slow(rate.a.y()) && slow(rate.b.x()) && slow(rate.b.y());
    p.a.slow = p.b.slow = a.rate && __all_sync(~0u, mine);
    return p;
}

// A group's decays and inputs from its rows; those at `end` and behind change nothing.
template <typename T>
struct RecurMaps {
    F4 d[rec_group<T>()], in[rec_group<T>()];
};
template <typename T, bool RATE, int SCALE, bool SLOW, bool WHOLE, typename X, typename R, typename I>
__device__ __forceinline__ void group_gates(X x, R r, I gi, bool has_i, const RecurChan4& par, int t, int end,
                                            RecurMaps<T>& m) {
#pragma unroll
    for (int s = 0; s < rec_group<T>(); ++s) {
        const F4 vr = r(s), vx = x(s);
        const RecurGate g0 = recur_gate<T, RATE, SCALE, SLOW, false>(vr.a, par.a);
        const RecurGate g1 = recur_gate<T, RATE, SCALE, SLOW, false>(vr.b, par.b);
        m.d[s] = {g0.d, g1.d};
        m.in[s] = SCALE == FAVOR_RECUR_PLAIN ? vx : F4{g0.w * vx.a, g1.w * vx.b};
    }
    if (has_i) {
#pragma unroll
        for (int s = 0; s < rec_group<T>(); ++s) {
            const F4 v = gi(s);
            m.in[s].a = m.in[s].a * sigmoid2<T>(v.a, par.a.i_bias);
            m.in[s].b = m.in[s].b * sigmoid2<T>(v.b, par.b.i_bias);
        }
    }
    if (!WHOLE) {
#pragma unroll
        for (int s = 0; s < rec_group<T>(); ++s)
            if (t + s >= end) m.d[s] = {both(kKeep), both(kKeep)}, m.in[s] = {both(0.f), both(0.f)};
    }
}
template <bool SLOW>
__device__ __forceinline__ F4 next4(const F4& d, const F4& h, const F4& b) {
    return {recur_next<SLOW>(d.a, h.a, b.a), recur_next<SLOW>(d.b, h.b, b.b)};
}
template <bool SLOW>
__device__ __forceinline__ F4 scale4(const F4& d, const F4& h) {
    return {recur_scale<SLOW>(d.a, h.a), recur_scale<SLOW>(d.b, h.b)};
}

// A stretch of tokens maps the state in front of it to p * state + h.
struct alignas(16) RecurMap {
    F4 p, h;
};
__device__ __forceinline__ RecurMap no_map() {
    return {{both(1.f), both(1.f)}, {both(0.f), both(0.f)}};
}
__device__ __forceinline__ F4 apply(const RecurMap& m, const F4& x) {
    return {fma2(m.p.a, x.a, m.h.a), fma2(m.p.b, x.b, m.h.b)};
}
// first, then `then`.
__device__ __forceinline__ RecurMap join(const RecurMap& first, const RecurMap& then) {
    return {{first.p.a * then.p.a, first.p.b * then.p.b}, apply(then, first.h)};
}

// Products of decays.  Equal decays next to 1 (an open gate's) round the same way at every token: their product kept in
// one float drifts by half a step a token, 5e-5 of a state in runs of 1024 tokens.  So a group's is kept as its loss,
// p - 1 (SLOW), or in two floats, p + rest; a run's in two.
template <bool SLOW>
struct GroupDecay {
    F2 p, rest;
    __device__ __forceinline__ GroupDecay() : p(both(SLOW ? 0.f : 1.f)), rest(both(0.f)) {}
    __device__ __forceinline__ void token(F2 d) {
        if (SLOW) {
            p = p + fma2(d, p, d);
            return;
        }
        // the rest of a product with a decay next to 1; one below 1/2 halves the product, and keeps none
        const bool kx = __float_as_int(d.x()) < 0, ky = __float_as_int(d.y()) < 0;
        const F2 keep(kx ? p.x() : 0.f, ky ? p.y() : 0.f), next = fma2(d, p, keep);
        const F2 sum = rest + fma2(d, p, fma2(next, both(-1.f), keep));
        p = next;
        rest = F2(kx ? sum.x() : 0.f, ky ? sum.y() : 0.f);
    }
    // (the product) x + h
    __device__ __forceinline__ F2 apply(F2 x, F2 h) const {
        return SLOW ? x + fma2(p, x, h) : fma2(p, x, fma2(rest, x, h));
    }
};
struct RunDecay {
    F2 p, rest;
    __device__ __forceinline__ RunDecay() : p(both(1.f)), rest(both(0.f)) {}
    __device__ __forceinline__ F2 value() const { return p + rest; }
    __device__ __forceinline__ F2 apply(F2 x, F2 h) const { return fma2(p, x, fma2(rest, x, h)); }
    template <bool SLOW>
    __device__ __forceinline__ void join(const GroupDecay<SLOW>& g) {
        const F2 minus = both(-1.f), next = SLOW ? fma2(p, g.p, p) : p * g.p;
        const F2 err = fma2(p, g.p, SLOW ? fma2(next, minus, p) : next * minus);
        rest = SLOW ? fma2(rest, g.p, rest) + err : fma2(rest, g.p, fma2(p, g.rest, err));
        p = next;
    }
};

// The maps of a call's runs and chunks, in the workspace: [row][chunk][run][slab] and [row][chunk][slab] of a warp's
// lanes.
struct RecurMapsAt {
    RecurMap *run, *chunk;
    RecurPlan p;
    __device__ __forceinline__ RecurMap* run_at(int b, int chunk_, int w, int slab) const {
        return run + ((((size_t)b * p.chunks + chunk_) * kRecWarps + w) * p.slabs + slab) * 32 + (threadIdx.x & 31);
    }
    __device__ __forceinline__ RecurMap* chunk_at(int b, int chunk_, int slab) const {
        return chunk + (((size_t)b * p.chunks + chunk_) * p.slabs + slab) * 32 + (threadIdx.x & 31);
    }
};
constexpr size_t kRecMapFloats = 32 * (sizeof(RecurMap) / 4);     // of a warp's lanes
inline size_t recur_run_floats(const RecurPlan& p, int B) {
    return (size_t)B * p.chunks * kRecWarps * p.slabs * kRecMapFloats;
}
inline size_t recur_chunk_floats(const RecurPlan& p, int B) { return (size_t)B * p.chunks * p.slabs * kRecMapFloats; }

// For every warp of a block: the state in front of the warp's run, from `start` in front of the row.  REVERSE:
// chunks and runs come last first.  The warps share the chunks in front, so that none joins more than an
// eighth of them.
struct RecurPlaces {
    RecurMap chunk[kRecWarps][32], run[kRecWarps][32];
};
template <bool REVERSE>
__device__ __forceinline__ F4 run_start(const RecurMapsAt& at, int b, int chunk, int slab, F4 start, RecurPlaces& sm) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int before = REVERSE ? at.p.chunks - 1 - chunk : chunk, each = (before + kRecWarps - 1) / kRecWarps;
    const int last = min(before, (warp + 1) * each);
    sm.run[warp][lane] = *at.run_at(b, chunk, warp, slab);
    RecurMap m = no_map();
#pragma unroll 4
    for (int k = warp * each; k < last; ++k) m = join(m, *at.chunk_at(b, REVERSE ? at.p.chunks - 1 - k : k, slab));
    sm.chunk[warp][lane] = m;
    __syncthreads();
    if (before)
#pragma unroll
        for (int w = 0; w < kRecWarps; ++w) start = apply(sm.chunk[w][lane], start);
    for (int k = REVERSE ? kRecWarps - 1 : 0; k != warp; k += REVERSE ? -1 : 1) start = apply(sm.run[k][lane], start);
    return start;
}

// Chunks of a row: as many blocks as the device holds at once (`per_sm` an SM), but kRecChunksMax at most (see
// run_start) and no run under kRecRunMin tokens: 8, with which [3, 1000, 500] fp32 took 13.9 us on the GPU, and 17.4
// with 16 (the call is the host's 19).  One wave of blocks and no more: where B * slabs comes to just over half of it,
// or just over all of it, the rest stands idle ([8, 4096, 2048] 220 us, [8, 4096, 2560] 412, [8, 4096, 5120] 652).
inline RecurPlan recur_plan(int num_sms, int per_sm, int D, int B, int L) {
    RecurPlan p;
    p.slabs = (D + kRecSlab - 1) / kRecSlab;
    long long chunks = (long long)num_sms * per_sm / ((long long)B * p.slabs);
    chunks = chunks < 1 ? 1 : chunks > kRecChunksMax ? kRecChunksMax : chunks;
    const long long runs = chunks * kRecWarps;
    long long run = (L + runs - 1) / runs;
    if (run < kRecRunMin) run = kRecRunMin;
    p.run = (int)((run + kRecGroupMax - 1) / kRecGroupMax * kRecGroupMax);
    p.chunks = (int)((L + (long long)p.run * kRecWarps - 1) / ((long long)p.run * kRecWarps));
    return p;
}
// Chunks x slabs x rows of any call with at most these sizes: a chunk a row, or as many as recur_plan's quotient gives
// and a row of max_L tokens fills.
inline size_t recur_blocks_max(int num_sms, int per_sm, int D, int max_B, int max_L) {
    const size_t places = (size_t)num_sms * per_sm, columns = (size_t)max_B * ((D + kRecSlab - 1) / kRecSlab);
    const size_t filled = ((size_t)max_L + kRecWarps * kRecRunMin - 1) / (kRecWarps * kRecRunMin);
    const size_t most = columns * (filled < kRecChunksMax ? filled : kRecChunksMax);
    return columns > places ? columns : places < most ? places : most;
}

// f<T, RATE, SCALE>::go(args...) for the handle's storage and scale and the call's decay.
template <template <typename, bool, int> class F, typename... A>
inline void recur_dispatch(const RecurHandle& h, bool rate, A&&... args) {
#define FAVOR_REC_SCALE(T, RATE)                                                                  \
    do {                                                                                          \
        if (h.scale == FAVOR_RECUR_PLAIN) F<T, RATE, FAVOR_RECUR_PLAIN>::go(args...);             \
        else if (h.scale == FAVOR_RECUR_MEAN) F<T, RATE, FAVOR_RECUR_MEAN>::go(args...);          \
        else F<T, RATE, FAVOR_RECUR_UNIT>::go(args...);                                           \
    } while (0)
    if (h.dtype == FAVOR_DTYPE_F32) {
        if (rate) FAVOR_REC_SCALE(float, true);
        else FAVOR_REC_SCALE(float, false);
    } else {
        if (rate) FAVOR_REC_SCALE(__nv_bfloat16, true);
        else FAVOR_REC_SCALE(__nv_bfloat16, false);
    }
#undef FAVOR_REC_SCALE
}

}  // namespace favor
