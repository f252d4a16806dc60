// Group normalisation with an activation over channels-last tokens, and its gradients:
//     n = (x - mean) / sqrt(var + eps) over the C = D / G channels of a token's group (without
//     centring n = x / sqrt(mean of x^2 + eps)),  u = n weight + bias,  out = act(u) or u act(z)
// and, with du = dout act'(u) (dout act(z), dz = dout u act'(z)), dn = du weight,
//     dx = (dn - mean(dn) - n mean(dn n)) / sqrt(var + eps)   (no mean(dn) without centring),
//     dweight = sum du n,  dbias = sum du over the tokens.
// Nothing but bytes: every input is read once and every output written once, 25 instructions an element
// forwards (28 by heads) and 46 back.  A group lies in the registers of the threads that share it: 1 to 32 lanes of a
// warp (their sums by shuffles), or a whole block.  The mean comes before the squares of what is left,
// so that an offset of the channels costs no digits.  A thread keeps its channels from token to token:
// their parameters, and the sums of their gradients, stay in registers too, and the next token's
// rows are on their way while this one's are worked on.  [1, 65536, 1024] bf16 by heads of 64 with a gate: 77 us
// (5.2 TB/s, 77% of a copy's rate); gradients of [8, 4096, 1536] with a gate 113 us (4.5 TB/s).
#include <initializer_list>
#include <type_traits>

#include "norm_internal.h"

namespace favor {

// n / d for n < 2^31 by a product: m = floor(2^(31+k) / d) + 1 with 2^k >= d.
struct Divide {
    unsigned d, m, k;
    __device__ __forceinline__ unsigned operator()(unsigned n) const {
        return (unsigned)(((unsigned long long)n * m) >> (31 + k));
    }
};
static Divide make_divide(unsigned d) {
    unsigned k = 0;
    while ((1u << k) < d) ++k;
    return {d, (unsigned)((1ull << (31 + k)) / d + 1), k};
}

struct NormPlan {
    int threads;        // of a block
    int share;          // threads that share a group: a power of two up to 32, or the block
    int per_block;      // groups of a token in a block
    int tokens;         // tokens of a block at a time
    int gx, gy;         // blocks: over tokens, over groups
    Divide by_L;
    int centred, act;
    float eps, inv_c;
    int C, D, G;
};

// ------------------------------------------------------------------ the activation
constexpr float kGeluC = 0.7978845608028653559f;    // sqrt(2 / pi)
constexpr float kGeluK = 0.044715f;

// f(x), and with GRAD f'(x).  gelu_tanh: x (1 + tanh(y)) / 2 = x sigmoid(2 y), y = sqrt(2/pi) (x + 0.044715 x^3).
template <typename T, bool GRAD, int N>
__device__ __forceinline__ void activate(int act, const F2 (&x)[N], F2 (&f)[N], F2 (&df)[N]) {
    const F2 one = both(1.f), none = both(0.f);
    if (act == FAVOR_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (!GRAD) {
                f[i] = silu2<T>(x[i]);
                continue;
            }
            F2 s, sn;
            sigmoids2<T>(x[i], none, s, sn);
            f[i] = x[i] * s;
            df[i] = s * fma2(x[i], sn, one);
        }
    } else if (act == FAVOR_ACT_GELU_TANH) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const F2 xx = x[i] * x[i], y = x[i] * fma2(xx, both(2.f * kGeluC * kGeluK), both(2.f * kGeluC));
            F2 s, sn;
            if (GRAD) sigmoids2<T>(y, none, s, sn);
            else s = sigmoid2<T>(y, none);
            f[i] = x[i] * s;
            if (GRAD) {     // an x^2 past all bounds meets a sn (x > 0) or an s of 0
                const F2 q = each(xx, [](float v) { return fminf(v, 1e30f); });
                df[i] = fma2(f[i] * sn, fma2(q, both(6.f * kGeluC * kGeluK), both(2.f * kGeluC)), s);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = x[i], df[i] = one;
    }
}

// ------------------------------------------------------------------ sums over a group
// WIDE: over the block; two sets of places in turn, so that one barrier a sum is enough.
struct GroupSum {
    float s[2][2][32];
};
// The sum of K values of every thread of a group.
template <bool WIDE, int K>
__device__ __forceinline__ void group_sum(float (&v)[K], int share, GroupSum& sm, int& turn) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (WIDE || o < share) {
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(~0u, v[k], o);
        }
    if (WIDE) {
        const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0) {
#pragma unroll
            for (int k = 0; k < K; ++k) sm.s[turn][k][threadIdx.x >> 5] = v[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = lane < warps ? sm.s[turn][k][lane] : 0.f;
        turn ^= 1;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(~0u, v[k], o);
    }
}

// ------------------------------------------------------------------ a thread's part of a group
// V channels as they are stored, and as pairs.
template <typename T, int V>
struct NormPack {
    static constexpr int kWords = V * (int)sizeof(T) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (kWords == 4) {
            const uint4 u = *reinterpret_cast<const uint4*>(p);
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        } else if constexpr (kWords == 2) {
            const uint2 u = *reinterpret_cast<const uint2*>(p);
            w[0] = u.x, w[1] = u.y;
        } else {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ F2 pair(int i) const {
        if constexpr (sizeof(T) == 2) return to_f2(w[i]);
        else return F2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
    __device__ __forceinline__ static void store(T* p, const F2* x) {
        if constexpr (kWords == 1) {
            *reinterpret_cast<uint32_t*>(p) = from_f2(x[0], T());
        } else if constexpr (kWords == 2) {
            *reinterpret_cast<float2*>(p) = make_float2(x[0].x(), x[0].y());
        } else if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint4*>(p) =
                make_uint4(from_f2(x[0], T()), from_f2(x[1], T()), from_f2(x[2], T()), from_f2(x[3], T()));
        } else {
            *reinterpret_cast<float4*>(p) = make_float4(x[0].x(), x[0].y(), x[1].x(), x[1].y());
        }
    }
};

// E packs of V channels: pack k of thread j of a group starts at channel (j + k share) V of it.  V is 16 bytes' worth,
// 2 or 1; N pairs of channels in all.
template <typename T, int V, int E, bool WIDE>
struct NormThread {
    static constexpr int N = V * E / 2;
    // A thread's channels of one token.
    struct Row {
        typename std::conditional<V == 1, T, NormPack<T, V == 1 ? 2 : V>>::type v[E];
        __device__ __forceinline__ F2 pair(int i) const {
            if constexpr (V == 1) return F2(to_f(v[2 * i]), to_f(v[2 * i + 1]));
            else return v[i / (V / 2)].pair(i % (V / 2));
        }
    };
    int j, g, tb;           // place in the group, group, place among the block's tokens
    bool on;                // has a group
    const NormPlan& p;
    __device__ __forceinline__ explicit NormThread(const NormPlan& pl) : p(pl) {
        const int slot = WIDE ? 0 : threadIdx.x / p.share;
        j = WIDE ? threadIdx.x : threadIdx.x % p.share;
        g = blockIdx.y * p.per_block + slot % p.per_block;
        tb = slot / p.per_block;
        on = tb < p.tokens && g < p.G;
    }
    __device__ __forceinline__ int chan(int k) const { return (j + k * p.share) * V; }
    __device__ __forceinline__ bool has(int k) const { return on && chan(k) < p.C; }
    // Token n of the call: whether it is there, and where the group starts in a token-major tensor and in x.
    __device__ __forceinline__ bool token(const NormArgs& a, unsigned n, size_t& at, size_t& atx) const {
        if (!on || n >= (unsigned)a.B * a.L) return false;
        at = (size_t)n * p.D + (size_t)g * p.C;
        atx = at;
        if (a.heads || a.lens) {
            const unsigned b = p.by_L(n), t = n - b * a.L;
            if (a.heads) atx = (((size_t)b * p.G + g) * a.L + t) * p.C;
            if (a.lens && (int)t >= row_len(a.lens, b, a.L)) return false;
        }
        return true;
    }
    __device__ __forceinline__ void load(const void* base, size_t at, bool ok, Row& r) const {
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const T* q = (const T*)base + at + chan(k);
            if constexpr (V == 1) {
                from_f(r.v[k], 0.f);
                if (ok && has(k)) r.v[k] = *q;
            } else {
                r.v[k].clear();
                if (ok && has(k)) r.v[k].load(q);
            }
        }
    }
    __device__ __forceinline__ void store(void* base, size_t at, const F2 (&x)[N]) const {
#pragma unroll
        for (int k = 0; k < E; ++k) {
            if (!has(k)) continue;
            T* q = (T*)base + at + chan(k);
            if constexpr (V == 1) from_f(*q, k % 2 ? x[k / 2].y() : x[k / 2].x());
            else NormPack<T, V>::store(q, x + k * (V / 2));
        }
    }
    __device__ __forceinline__ void params(const float* q, float otherwise, F2 (&v)[N]) const {
        float f[2 * N];
#pragma unroll
        for (int k = 0; k < E; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e)
                f[k * V + e] = q && has(k) ? q[(size_t)g * p.C + chan(k) + e] : otherwise;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = F2(f[2 * i], f[2 * i + 1]);
    }
    // n of the group in place of x; gives 1 / sqrt(var + eps).
    __device__ __forceinline__ float normalise(const Row& x, F2 (&n)[N], GroupSum& sm, int& turn) const {
        F2 s = both(0.f);
        float v[1];
#pragma unroll
        for (int i = 0; i < N; ++i) n[i] = x.pair(i);
        if (p.centred) {
#pragma unroll
            for (int i = 0; i < N; ++i) s = s + n[i];
            v[0] = s.x() + s.y();
            group_sum<WIDE>(v, p.share, sm, turn);
            const float mean = v[0] * p.inv_c;
#pragma unroll
            for (int i = 0; i < N; ++i)     // the pairs behind the group's end stay 0
                n[i] = n[i] + F2(has(2 * i / V) ? -mean : 0.f, has((2 * i + 1) / V) ? -mean : 0.f);
            s = both(0.f);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) s = fma2(n[i], n[i], s);
        v[0] = s.x() + s.y();
        group_sum<WIDE>(v, p.share, sm, turn);
        const float rstd = rsqrtf(fmaf(v[0], p.inv_c, p.eps));
#pragma unroll
        for (int i = 0; i < N; ++i) n[i] = n[i] * both(rstd);
        return rstd;
    }
};

// Threads of a block at most.  1024 leave a thread 64 registers, whatever the call's block has: the instances of 16
// channels a thread (bf16 groups above 4096 channels, fp32 above 2048) spill, forwards 190 to 810 bytes a thread, back
// 1000 to 1600 ([4, 4096, 5120] bf16 in one gated group 163 and 770 us, [4, 4096, 4096] 114 and 203).
template <int V, int E, bool WIDE>
__host__ __device__ constexpr int norm_threads() { return !WIDE ? 256 : V * E <= 8 ? 512 : 1024; }

template <typename T, int V, int E, bool WIDE>
__global__ void __launch_bounds__((norm_threads<V, E, WIDE>()), !WIDE && V * E <= 8 ? 4 : 1)
k_norm(NormArgs a, NormPlan p) {
    __shared__ GroupSum sm;
    typedef NormThread<T, V, E, WIDE> Thread;
    constexpr int N = Thread::N;
    const Thread th(p);
    F2 w[N], bias[N];
    th.params(a.weight, 1.f, w);
    th.params(a.bias, 0.f, bias);
    const unsigned step = p.gx * p.tokens, total = (unsigned)a.B * a.L;
    unsigned n = blockIdx.x * p.tokens + th.tb;
    size_t at = 0, atx = 0;
    bool ok = th.token(a, n, at, atx);
    typename Thread::Row x, z;
    th.load(a.x, atx, ok, x);
    th.load(a.z, at, ok && a.z, z);
    int turn = 0;
#pragma unroll 2
    for (unsigned first = blockIdx.x * p.tokens; first < total; first += step, n += step) {
        typename Thread::Row nx, nz;
        size_t nat = 0, natx = 0;
        const bool nok = th.token(a, n + step, nat, natx);
        th.load(a.x, natx, nok, nx);
        th.load(a.z, nat, nok && a.z, nz);
        F2 u[N], f[N], df[N];
        th.normalise(x, u, sm, turn);
#pragma unroll
        for (int i = 0; i < N; ++i) u[i] = fma2(u[i], w[i], bias[i]);
        if (a.z) {
            F2 v[N];
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = z.pair(i);
            activate<T, false, N>(p.act, v, f, df);
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = u[i] * f[i];
        } else {
            activate<T, false, N>(p.act, u, f, df);
        }
        if (!ok) {
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = both(0.f);
        }
        if (ok || (a.clear && th.on && n < total)) th.store(a.out, at, f);
        x = nx;
        z = nz;
        ok = nok;
        at = nat;
    }
}

template <typename T, int V, int E, bool WIDE>
__global__ void __launch_bounds__((norm_threads<V, E, WIDE>()), !WIDE && V * E <= 8 ? 2 : 1)
k_norm_bwd(NormArgs a, NormPlan p, float* part) {
    __shared__ GroupSum sm;
    extern __shared__ float sums[];     // [E * V][threads]
    typedef NormThread<T, V, E, WIDE> Thread;
    constexpr int N = Thread::N;
    const Thread th(p);
    F2 w[N], bias[N], dw[N], db[N];
    th.params(a.weight, 1.f, w);
    th.params(a.bias, 0.f, bias);
#pragma unroll
    for (int i = 0; i < N; ++i) dw[i] = db[i] = both(0.f);
    const unsigned step = p.gx * p.tokens, total = (unsigned)a.B * a.L;
    unsigned n = blockIdx.x * p.tokens + th.tb;
    size_t at = 0, atx = 0;
    bool ok = th.token(a, n, at, atx);
    typename Thread::Row x, z, g;
    th.load(a.x, atx, ok, x);
    th.load(a.z, at, ok && a.z, z);
    th.load(a.dout, at, ok, g);
    int turn = 0;
    for (unsigned first = blockIdx.x * p.tokens; first < total; first += step, n += step) {
        typename Thread::Row nx, nz, ng;
        size_t nat = 0, natx = 0;
        const bool nok = th.token(a, n + step, nat, natx);
        th.load(a.x, natx, nok, nx);
        th.load(a.z, nat, nok && a.z, nz);
        th.load(a.dout, nat, nok, ng);
        F2 nm[N], u[N], du[N], dz[N];
        const float rstd = th.normalise(x, nm, sm, turn);
#pragma unroll
        for (int i = 0; i < N; ++i) u[i] = fma2(nm[i], w[i], bias[i]);
        {
            F2 f[N], df[N];
            if (a.z) {
#pragma unroll
                for (int i = 0; i < N; ++i) du[i] = z.pair(i);
                activate<T, true, N>(p.act, du, f, df);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const F2 up = g.pair(i);
                    dz[i] = up * u[i] * df[i];
                    du[i] = up * f[i];
                }
            } else {
                activate<T, true, N>(p.act, u, f, df);
#pragma unroll
                for (int i = 0; i < N; ++i) du[i] = g.pair(i) * df[i];
            }
        }
        if (!ok) {      // whatever the parameters make of nothing
#pragma unroll
            for (int i = 0; i < N; ++i) du[i] = dz[i] = both(0.f);
        }
        F2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            dw[i] = fma2(du[i], nm[i], dw[i]);
            db[i] = db[i] + du[i];
            du[i] = du[i] * w[i];       // the gradient of n
            s1 = s1 + du[i];
            s2 = fma2(du[i], nm[i], s2);
        }
        float s[2] = {s1.x() + s1.y(), s2.x() + s2.y()};
        group_sum<WIDE>(s, p.share, sm, turn);
        const F2 m1 = both(p.centred ? -rstd * (s[0] * p.inv_c) : 0.f), m2 = both(-rstd * (s[1] * p.inv_c));
        if (th.on && n < total) {       // behind a row's end too: zeros
#pragma unroll
            for (int i = 0; i < N; ++i) du[i] = ok ? fma2(nm[i], m2, fma2(du[i], both(rstd), m1)) : both(0.f);
            th.store(a.dx, atx, du);
            if (a.z) th.store(a.dz, at, dz);
        }
        x = nx;
        z = nz;
        g = ng;
        ok = nok;
        at = nat;
        atx = natx;
    }
    // the block's tokens: their threads' sums, added in order by the first token's
#pragma unroll
    for (int what = 0; what < 2; ++what) {
        float* to = part + ((size_t)blockIdx.x * 2 + what) * p.D + (size_t)th.g * p.C;
        float v[2 * N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[2 * i] = (what ? db : dw)[i].x();
            v[2 * i + 1] = (what ? db : dw)[i].y();
        }
        if (p.tokens > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 2 * N; ++i) sums[i * blockDim.x + threadIdx.x] = v[i];
            __syncthreads();
            if (th.tb == 0)
                for (int t = 1; t < p.tokens; ++t)
#pragma unroll
                    for (int i = 0; i < 2 * N; ++i)
                        v[i] += sums[i * blockDim.x + threadIdx.x + t * p.per_block * p.share];
        }
        if (th.tb == 0) {
#pragma unroll
            for (int k = 0; k < E; ++k)
                if (th.has(k)) {
#pragma unroll
                    for (int e = 0; e < V; ++e) to[th.chan(k) + e] = v[k * V + e];
                }
        }
    }
}

// part [rows][2][D] summed over rows in a fixed order: 32 columns a block, a warp every 32nd row, 8 of them at a time.
__global__ void __launch_bounds__(1024)
k_norm_reduce(const float* part, int rows, int D, float* dweight, float* dbias) {
    __shared__ float s[32][33];
    const int n = 2 * D, lane = threadIdx.x & 31, y = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
    float sum = 0.f;
    if (i < n)
        for (int row = y; row < rows; row += 32 * 8) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = row + 32 * k < rows ? part[(size_t)(row + 32 * k) * n + i] : 0.f;
            sum += sum_two_by_two<8>(v);
        }
    s[y][lane] = sum;
    __syncthreads();
    sum = s[lane][y];       // column y's sums, one a lane
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    const int c = blockIdx.x * 32 + y;
    if (lane == 0 && c < n) {
        float* to = c < D ? dweight : dbias;
        if (to) to[c < D ? c : c - D] = sum;
    }
}

// ------------------------------------------------------------------ host
// Blocks an SM at most: what fits at 64 registers (6 or 8 leave a part wave: by heads 88 and 78 us instead of 77; the
// narrow instances that read less than 16 bytes at a time, and fp32's of 8 channels a thread, spill 28 to 250 bytes
// at it), and for gradients two waves of the two that fit (three at 80 registers spill: 137 us instead of 113; 6
// waves 145).
constexpr int kNormPerSm = 4, kNormBwdPerSm = 4;

static NormPlan norm_plan(const NormHandle& h, int B, int L, int V, int E, bool wide, int per_sm) {
    NormPlan p = {};
    p.C = h.D / h.G;
    p.D = h.D;
    p.G = h.G;
    const int need = (p.C + V * E - 1) / (V * E);
    if (wide) {
        p.threads = p.share = (need + 31) / 32 * 32;
        p.per_block = p.tokens = 1;
    } else {
        p.share = 1;
        while (p.share < need) p.share *= 2;
        // the block size that leaves the fewest threads idle, near 256 ones first
        int best = -1;
        for (int th : {256, 224, 192, 160, 128}) {
            const int places = th / p.share, per = places < h.G ? places : h.G, tok = places / per;
            const int gy = (h.G + per - 1) / per;
            const int used = (int)(1000LL * h.G * tok * p.share / ((long long)gy * th));
            if (used > best) {
                best = used;
                p.threads = th;
                p.per_block = per;
                p.tokens = tok;
            }
        }
    }
    p.gy = (h.G + p.per_block - 1) / p.per_block;
    const long long most = (long long)h.num_sms * per_sm, tiles = ((long long)B * L + p.tokens - 1) / p.tokens;
    const long long gx = (most + p.gy - 1) / p.gy;
    p.gx = (int)(gx < tiles ? gx : tiles);
    p.by_L = make_divide(L);
    p.centred = h.centred;
    p.act = h.act;
    p.eps = h.eps;
    p.inv_c = (float)(1.0 / p.C);
    return p;
}

// Whether the groups and tensors start on `bytes` bytes.
static bool norm_packs(const NormHandle& h, const NormArgs& a, int bytes) {
    uintptr_t bits = (uintptr_t)(h.D / h.G) * (h.dtype == FAVOR_DTYPE_F32 ? 4 : 2);
    for (const void* p : {a.x, a.z, (const void*)a.out, a.dout, (const void*)a.dx, (const void*)a.dz})
        bits |= reinterpret_cast<uintptr_t>(p);
    return bits % bytes == 0;
}

template <typename T, int V, int E, bool WIDE>
struct NormForward {
    static void go(const NormHandle& h, const NormArgs& a, cudaStream_t st) {
        const NormPlan p = norm_plan(h, a.B, a.L, V, E, WIDE, kNormPerSm);
        k_norm<T, V, E, WIDE><<<dim3(p.gx, p.gy), p.threads, 0, st>>>(a, p);
    }
};
template <typename T, int V, int E, bool WIDE>
struct NormBackward {
    static void go(const NormHandle& h, const NormArgs& a, cudaStream_t st) {
        const NormPlan p = norm_plan(h, a.B, a.L, V, E, WIDE, kNormBwdPerSm);
        const size_t smem = p.tokens > 1 ? (size_t)p.threads * V * E * 4 : 0;
        k_norm_bwd<T, V, E, WIDE><<<dim3(p.gx, p.gy), p.threads, smem, st>>>(a, p, h.ws);
        count_launch();
        if (a.dweight || a.dbias) {
            k_norm_reduce<<<(2 * h.D + 31) / 32, 1024, 0, st>>>(h.ws, p.gx, h.D, a.dweight, a.dbias);
            count_launch();
        }
    }
};

// F<T, V, E, WIDE>::go(...): E1 or 2 E1 packs a thread where a warp holds a group with them, else a block, of up to
// 512 threads or (E2 packs) 1024.
template <template <typename, int, int, bool> class F, typename T, int V, int E1, int E2>
static void norm_sizes(const NormHandle& h, const NormArgs& a, cudaStream_t st) {
    const int C = h.D / h.G;
    if (C <= 32 * V * E1) F<T, V, E1, false>::go(h, a, st);
    else if (C <= 64 * V * E1) F<T, V, 2 * E1, false>::go(h, a, st);
    else if (C <= 512 * V * E1) F<T, V, E1, true>::go(h, a, st);
    else F<T, V, E2, true>::go(h, a, st);
}
template <template <typename, int, int, bool> class F>
static void norm_dispatch(const NormHandle& h, const NormArgs& a, cudaStream_t st) {
    if (h.dtype == FAVOR_DTYPE_F32) {
        if (norm_packs(h, a, 16)) norm_sizes<F, float, 4, 1, 4>(h, a, st);
        else if (norm_packs(h, a, 8)) norm_sizes<F, float, 2, 2, 8>(h, a, st);
        else norm_sizes<F, float, 1, 4, 16>(h, a, st);
    } else {
        if (norm_packs(h, a, 16)) norm_sizes<F, __nv_bfloat16, 8, 1, 2>(h, a, st);
        else if (norm_packs(h, a, 4)) norm_sizes<F, __nv_bfloat16, 2, 4, 8>(h, a, st);
        else norm_sizes<F, __nv_bfloat16, 1, 4, 16>(h, a, st);
    }
}

// A row of sums a block over tokens: (most + gy - 1) / gy of them, gy = 1 at least.
size_t norm_backward_ws(const NormHandle& h) {
    const size_t tokens = (size_t)h.max_B * h.max_L, most = (size_t)h.num_sms * kNormBwdPerSm;
    return (tokens < most ? tokens : most) * 2 * h.D;
}

favor_status norm_forward(const NormHandle& h, const NormArgs& a, cudaStream_t st) {
    norm_dispatch<NormForward>(h, a, st);
    count_launch();
    return check_launch("favor_group_norm");
}

favor_status norm_backward(const NormHandle& h, const NormArgs& a, cudaStream_t st) {
    norm_dispatch<NormBackward>(h, a, st);
    return check_launch("favor_group_norm_backward");
}

}  // namespace favor
