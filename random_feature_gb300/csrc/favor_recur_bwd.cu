// Gradients of the gated linear recurrence.  With g = dout silu(z), lambda_t the gradient of h_t:
//     lambda_t = g_t + a_{t+1} lambda_{t+1},
//     dx = lambda w si,  di = lambda w x si (1 - si),  dz = dout h silu'(z),
//     q = lambda (h_{t-1} - v k),  v = si x,  k = 0, 1 or a / w (what -dw / da is),
//     dr = -a q rate s (1 - s), drate = -sum a q s  (dr = q a (1 - a) without a rate).
// What a token hands back, mu = a lambda, is a map of what it is handed, mu -> a mu + a g, as its state is
// of the one in front.  k_recur_bwd_maps joins both for every run of tokens (everything is read), and keeps
// the forward map from the run's start to every group of tokens; k_recur_bwd walks each run from its
// end, with the state in front of each group from that map.  So five tensors are read twice and four
// written: 14 elements for the 9 that are the least, and as much as 2 more for the groups' maps.
// [4, 8192, 1024] bf16: 271 us (2.2 TB/s of the 9), 41 and 90 instructions an element (318 in the general form of
// rates, 264 without rates); [2, 777, 500] fp32 20 us on the GPU (the call is the host's 37).
#include <type_traits>

#include "recur_internal.h"

namespace favor {

// Chunks for two blocks an SM, which the maps fill: 128 registers, and in bf16 12 to 100 bytes of spills.  k_recur_bwd
// takes 255 in bf16, with up to 56 bytes of spills (239 at most and none in fp32), so one block at a time (capped at
// 128 it took 312 us instead of 263; its rows through shared memory then 261; chunks for one block an SM 277).
constexpr int kRecBwdPerSm = 2;

// The maps from a run's start to its groups: [row][group of the row][slab] of a warp's lanes.
struct GroupMapsAt {
    RecurMap* at;
    int groups;     // of a row
    __device__ __forceinline__ RecurMap* operator()(const RecurPlan& p, int b, int g, int slab) const {
        return at + (((size_t)b * groups + g) * p.slabs + slab) * 32 + (threadIdx.x & 31);
    }
};

template <typename T, bool RATE, int SCALE>
__global__ void __launch_bounds__(kRecThreads, kRecBwdPerSm)
k_recur_bwd_maps(RecurArgs a, int D, RecurMapsAt fwd, RecurMapsAt rev, GroupMapsAt groups) {
    constexpr int G = rec_group<T>();
    __shared__ RecurMap runs[2][kRecWarps][32];
    const RecurPlan& p = fwd.p;
    const int slab = blockIdx.x % p.slabs, rest = blockIdx.x / p.slabs;
    const int chunk = rest % p.chunks, b = rest / p.chunks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const RecurLane l(a, D, slab);
    const int len = row_len(a.lens, b, a.L);
    const int t0 = (chunk * kRecWarps + warp) * p.run, end = min(len, t0 + p.run);
    const F4 none = {both(0.f), both(0.f)};
    F4 mh = none, back = none;      // the run's maps: the decays' product serves both
    RunDecay ma, mb;
    if (t0 < end) {
        const size_t row0 = (size_t)b * a.L * D;
        const T *x = (const T*)a.x + row0, *r = (const T*)a.r + row0, *gi = (const T*)a.i + row0;
        const T *z = (const T*)a.z + row0, *dout = (const T*)a.dout + row0;
        const RecurChan4 par = load_chans<T>(a, l);
        auto group = [&](auto slow, auto whole, int t, auto vx, auto vr, auto vi, auto vz, auto vg) {
            constexpr bool SLOW = decltype(slow)::value;
            RecurMaps<T> q;
            group_gates<T, RATE, SCALE, SLOW, decltype(whole)::value>(vx, vr, vi, a.i, par, t, end, q);
            const F4 before = {ma.value(), mb.value()};
            *groups(p, b, t / G, slab) = {before, mh};
            F4 h = none, hb = none;
            GroupDecay<SLOW> ga, gb;
#pragma unroll
            for (int s = 0; s < G; ++s) {
                h = next4<SLOW>(q.d[s], h, q.in[s]);
                ga.token(q.d[s].a);
                gb.token(q.d[s].b);
            }
            F4 up[G];
#pragma unroll
            for (int s = 0; s < G; ++s) up[s] = vg(s);
            if (a.z) {
#pragma unroll
                for (int s = 0; s < G; ++s) {
                    const F4 vs = vz(s);
                    up[s] = {up[s].a * silu2<T>(vs.a), up[s].b * silu2<T>(vs.b)};
                }
            }
#pragma unroll
            for (int s = G - 1; s >= 0; --s) {
                if (!decltype(whole)::value && t + s >= end) continue;
                hb = scale4<SLOW>(q.d[s], {hb.a + up[s].a, hb.b + up[s].b});
            }
            mh = {ga.apply(mh.a, h.a), gb.apply(mh.b, h.b)};
            back = {fma2(before.a, hb.a, back.a), fma2(before.b, hb.b, back.b)};
            ma.join(ga);
            mb.join(gb);
        };
        int t = t0;
        const int whole = l.quads ? t0 + (end - t0) / G * G : t0;
        auto walk = [&](auto slow) {
            RecurRows<T> nx, nr, ni, nz, ng;
            auto load = [&](int t) {
                load_rows<T, true, true>(x, l, t, end, nx);
                load_rows<T, true, true>(r, l, t, end, nr);
                if (a.i) load_rows<T, true, true>(gi, l, t, end, ni);
                if (a.z) load_rows<T, true, true>(z, l, t, end, nz);
                load_rows<T, true, true>(dout, l, t, end, ng);
            };
            load(t);
            for (; t < whole; t += G) {
                const RecurRows<T> vx = nx, vr = nr, vi = ni, vz = nz, vg = ng;
                if (t + G < whole) load(t + G);
                group(slow, std::true_type(), t, vx, vr, vi, vz, vg);
            }
        };
        if (t < whole) {
            if (RATE && par.a.slow) walk(std::integral_constant<bool, RATE>());
            else walk(std::false_type());
        }
        for (; t < end; t += G) {
            RecurRows<T> vx, vr, vi, vz, vg;
            load_rows<T, true, false>(x, l, t, end, vx);
            load_rows<T, true, false>(r, l, t, end, vr);
            if (a.i) load_rows<T, true, false>(gi, l, t, end, vi);
            if (a.z) load_rows<T, true, false>(z, l, t, end, vz);
            load_rows<T, true, false>(dout, l, t, end, vg);
            group(std::false_type(), std::false_type(), t, vx, vr, vi, vz, vg);
        }
    }
    const F4 product = {ma.value(), mb.value()};
    RecurMap m = {product, mh};
    const RecurMap handed = {product, back};
    *fwd.run_at(b, chunk, warp, slab) = m;
    *rev.run_at(b, chunk, warp, slab) = handed;
    runs[0][warp][lane] = m;
    runs[1][warp][lane] = handed;
    __syncthreads();
    if (warp == 0) {
        m = runs[0][0][lane];
#pragma unroll
        for (int w = 1; w < kRecWarps; ++w) m = join(m, runs[0][w][lane]);
        *fwd.chunk_at(b, chunk, slab) = m;
    }
    if (warp == 1) {
        m = runs[1][kRecWarps - 1][lane];
#pragma unroll
        for (int w = kRecWarps - 2; w >= 0; --w) m = join(m, runs[1][w][lane]);
        *rev.chunk_at(b, chunk, slab) = m;
    }
}

// part [row and chunk][3][D]: each block's sums of drate, dr and di.
template <typename T, bool RATE, int SCALE>
__global__ void __launch_bounds__(kRecThreads, 1)
k_recur_bwd(RecurArgs a, int D, RecurMapsAt fwd, RecurMapsAt rev, GroupMapsAt groups, float* part) {
    constexpr int G = rec_group<T>();
    __shared__ RecurPlaces places;
    __shared__ F4 sums[kRecWarps][3][32];
    const RecurPlan& p = fwd.p;
    const int slab = blockIdx.x % p.slabs, rest = blockIdx.x / p.slabs;
    const int chunk = rest % p.chunks, b = rest / p.chunks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const RecurLane l(a, D, slab);
    const int len = row_len(a.lens, b, a.L);
    const F4 none = {both(0.f), both(0.f)};
    const int t0 = (chunk * kRecWarps + warp) * p.run, end = min(len, t0 + p.run);
    const size_t row0 = (size_t)b * a.L * D;
    const T *x = (const T*)a.x + row0, *r = (const T*)a.r + row0, *gi = (const T*)a.i + row0, *z = (const T*)a.z + row0;
    const T* dout = (const T*)a.dout + row0;
    const F4 start = run_start<false>(fwd, b, chunk, slab, none, places);
    __syncthreads();
    F4 mu = run_start<true>(rev, b, chunk, slab, none, places);
    T *dx = (T*)a.dx + row0, *dr = (T*)a.dr + row0, *di = (T*)a.di + row0, *dz = (T*)a.dz + row0;
    const int from = max(t0, end), to = min(a.L, t0 + p.run);       // behind the row's end
    clear_rows(dx, l, from, to);
    clear_rows(dr, l, from, to);
    if (a.i) clear_rows(di, l, from, to);
    if (a.z) clear_rows(dz, l, from, to);
    F4 sum[3] = {none, none, none};     // of drate, dr, di
    if (t0 < end) {
        const RecurChan4 par = load_chans<T>(a, l);
        auto group = [&](auto slow, auto whole, int t, auto vx, auto vr, auto vi, auto vz, auto vg) {
            constexpr bool SLOW = decltype(slow)::value, WHOLE = decltype(whole)::value;
            const F4 h0 = apply(*groups(p, b, t / G, slab), start);
            typedef typename Raw4<T>::H H;
            H ox[2][G], orr[2][G], oi[2][G], oz[2][G];
            // one pair of channels after the other: even so this takes all the registers that a thread can have
            auto half = [&](int k, F2 h, const RecurChan& c, F2& m, F2& srate, F2& sr, F2& ss) {
                F2 hs[G + 1];       // the states in front of the group's tokens, and behind it
                hs[0] = h;
#pragma unroll
                for (int s = 0; s < G; ++s) {
                    const RecurGate q = recur_gate<T, RATE, SCALE, SLOW, false>(vr(s, k), c);
                    F2 v = vx(s, k);
                    if (a.i) v = v * sigmoid2<T>(vi(s, k), c.i_bias);
                    hs[s + 1] = recur_next<SLOW>(q.d, hs[s], SCALE == FAVOR_RECUR_PLAIN ? v : q.w * v);
                    if (!WHOLE && t + s >= end) hs[s + 1] = hs[s];
                }
                F2 some[3] = {both(0.f), both(0.f), both(0.f)};    // of these tokens, before they meet the whole sum
#pragma unroll
                for (int s = G - 1; s >= 0; --s) {
                    if (!WHOLE && t + s >= end) continue;
                    const RecurGate q = recur_gate<T, RATE, SCALE, SLOW, true>(vr(s, k), c);
                    F2 si, sn, v = vx(s, k), up = vg(s, k);
                    if (a.i) {
                        sigmoids2<T>(vi(s, k), c.i_bias, si, sn);
                        v = v * si;
                    }
                    if (a.z) {
                        const F2 xz = vz(s, k);
                        F2 zs, zn;
                        sigmoids2<T>(xz, both(0.f), zs, zn);
                        oz[k][s] = from_f2(up * hs[s + 1] * (zs * fma2(xz, zn, both(1.f))), T());
                        up = up * (xz * zs);
                    }
                    const F2 lam = up + m, lw = SCALE == FAVOR_RECUR_PLAIN ? lam : lam * q.w;
                    m = recur_scale<SLOW>(q.d, lam);
                    ox[k][s] = from_f2(a.i ? lw * si : lw, T());
                    if (a.i) {
                        const F2 y = lw * v * sn;
                        oi[k][s] = from_f2(y, T());
                        some[2] = some[2] + y;
                    }
                    F2 e = hs[s];
                    if (SCALE == FAVOR_RECUR_MEAN) e = fma2(v, both(-1.f), e);
                    if (SCALE == FAVOR_RECUR_UNIT) e = fma2(v * both(-1.f), q.a * q.rw, e);
                    const F2 aq = q.a * (lam * e);
                    F2 y;
                    if (RATE) {
                        const F2 as = aq * q.s * both(-1.f);
                        some[0] = some[0] + as;
                        y = as * (c.rate * q.sn);
                    } else {
                        y = aq * q.sn;
                    }
                    orr[k][s] = from_f2(y, T());
                    some[1] = some[1] + y;
                }
                srate = srate + some[0];
                sr = sr + some[1];
                ss = ss + some[2];
            };
            half(0, h0.a, par.a, mu.a, sum[0].a, sum[1].a, sum[2].a);
            half(1, h0.b, par.b, mu.b, sum[0].b, sum[1].b, sum[2].b);
#pragma unroll
            for (int s = G - 1; s >= 0; --s) {
                if (!WHOLE && t + s >= end) continue;
                write_raw<T, WHOLE>(dx, l, t + s, raw_of(ox[0][s], ox[1][s]));
                write_raw<T, WHOLE>(dr, l, t + s, raw_of(orr[0][s], orr[1][s]));
                if (a.i) write_raw<T, WHOLE>(di, l, t + s, raw_of(oi[0][s], oi[1][s]));
                if (a.z) write_raw<T, WHOLE>(dz, l, t + s, raw_of(oz[0][s], oz[1][s]));
            }
        };
        int t = t0 + (end - 1 - t0) / G * G;
        const int whole = l.quads ? (end - t0) / G * G : 0;     // tokens of whole groups, read 4 channels at a time
        for (; t >= t0 + whole; t -= G) {
            RecurRows<T> vx, vr, vi, vz, vg;
            load_rows<T, false, false>(x, l, t, end, vx);
            load_rows<T, false, false>(r, l, t, end, vr);
            if (a.i) load_rows<T, false, false>(gi, l, t, end, vi);
            if (a.z) load_rows<T, false, false>(z, l, t, end, vz);
            load_rows<T, false, false>(dout, l, t, end, vg);
            group(std::false_type(), std::false_type(), t, vx, vr, vi, vz, vg);
        }
        auto walk = [&](auto slow) {
            RecurRows<T> nx, nr, ni, nz, ng;        // the next group's rows are on their way
            auto load = [&](int t) {
                load_rows<T, false, true>(x, l, t, end, nx);
                load_rows<T, false, true>(r, l, t, end, nr);
                if (a.i) load_rows<T, false, true>(gi, l, t, end, ni);
                if (a.z) load_rows<T, false, true>(z, l, t, end, nz);
                load_rows<T, false, true>(dout, l, t, end, ng);
            };
            load(t);
            for (; t >= t0; t -= G) {
                const RecurRows<T> vx = nx, vr = nr, vi = ni, vz = nz, vg = ng;
                if (t > t0) load(t - G);
                group(slow, std::true_type(), t, vx, vr, vi, vz, vg);
            }
        };
        if (t >= t0) {
            if (RATE && par.a.slow) walk(std::integral_constant<bool, RATE>());
            else walk(std::false_type());
        }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) sums[warp][k][lane] = sum[k];
    __syncthreads();
    if (warp < 3) {
        F4 v[kRecWarps];
#pragma unroll
        for (int w = 0; w < kRecWarps; ++w) v[w] = sums[w][warp][lane];
#pragma unroll
        for (int n = kRecWarps / 2; n > 0; n >>= 1)
#pragma unroll
            for (int w = 0; w < n; ++w) v[w] = {v[w].a + v[w + n].a, v[w].b + v[w + n].b};
        store_vec(part + (((size_t)b * p.chunks + chunk) * 3 + warp) * D, l, v[0]);
    }
}

// part [rows][3][D] summed over rows in a fixed order.
__global__ void __launch_bounds__(256) k_recur_reduce(const float* part, int rows, int D, float* drate, float* dr_bias,
                                                      float* di_bias) {
    const int n = 3 * D, i = blockIdx.x * 32 + (threadIdx.x & 31);
    const float sum = block_column_sum(i < n ? part + i : nullptr, n, rows);
    if (threadIdx.x < 32 && i < n) {
        float* to = i < D ? drate : i < 2 * D ? dr_bias : di_bias;
        if (to) to[i % D] = sum;
    }
}

// ------------------------------------------------------------------ host
static int recur_groups(int L, int group) { return L / group + (L % group != 0); }

template <typename T, bool RATE, int SCALE>
struct RecurBwd {
    static void go(const RecurHandle& h, const RecurArgs& a, cudaStream_t st) {
        RecurMapsAt fwd = {}, rev = {};
        fwd.p = rev.p = recur_plan(h.num_sms, kRecBwdPerSm, h.D, a.B, a.L);
        float* ws = h.ws;
        auto take = [&](size_t floats) {
            float* at = ws;
            ws += floats;
            return reinterpret_cast<RecurMap*>(at);
        };
        const size_t run = recur_run_floats(fwd.p, a.B), chunk = recur_chunk_floats(fwd.p, a.B);
        fwd.run = take(run);
        rev.run = take(run);
        fwd.chunk = take(chunk);
        rev.chunk = take(chunk);
        GroupMapsAt groups;
        groups.groups = recur_groups(a.L, rec_group<T>());
        groups.at = take((size_t)a.B * groups.groups * fwd.p.slabs * kRecMapFloats);
        const int rows = a.B * fwd.p.chunks;
        const unsigned blocks = (unsigned)rows * fwd.p.slabs;
        k_recur_bwd_maps<T, RATE, SCALE><<<blocks, kRecThreads, 0, st>>>(a, h.D, fwd, rev, groups);
        k_recur_bwd<T, RATE, SCALE><<<blocks, kRecThreads, 0, st>>>(a, h.D, fwd, rev, groups, ws);
        count_launch(2);
        if (a.drate || a.dr_bias || a.di_bias) {
            k_recur_reduce<<<(3 * h.D + 31) / 32, 256, 0, st>>>(ws, rows, h.D, a.drate, a.dr_bias, a.di_bias);
            count_launch();
        }
    }
};

// Two sets of maps, three sums a channel for every chunk of a row, and a map for every group.
size_t recur_backward_ws(const RecurHandle& h) {
    const size_t blocks = recur_blocks_max(h.num_sms, kRecBwdPerSm, h.D, h.max_B, h.max_L);
    const int group = h.dtype == FAVOR_DTYPE_F32 ? rec_group<float>() : rec_group<__nv_bfloat16>();
    const size_t slabs = (h.D + kRecSlab - 1) / kRecSlab;
    return blocks * 2 * (kRecWarps + 1) * kRecMapFloats + blocks * 3 * kRecSlab +
           (size_t)h.max_B * recur_groups(h.max_L, group) * slabs * kRecMapFloats;
}

favor_status recur_backward(const RecurHandle& h, const RecurArgs& a, cudaStream_t st) {
    recur_dispatch<RecurBwd>(h, a.rate != nullptr, h, a, st);
    return check_launch("favor_recur_backward");
}

}  // namespace favor
