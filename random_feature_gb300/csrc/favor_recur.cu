// Gated linear recurrence over tokens, one state a channel:
//     s = sigmoid(r + r_bias),  a = e^(-rate s) (a = s without a rate),
//     w = 1, 1 - a or sqrt(1 - a^2),  h <- a h + w sigmoid(i + i_bias) x,  out = h or h z sigmoid(z)
// A token's map h -> a h + b is known without the state, and maps compose: every row is cut into runs of
// tokens, one a warp, as many as keep the device full.  k_recur_maps joins the maps of each run (x, r, i
// are read); k_recur_scan takes each run's start from the maps in front of it and walks it again, now
// writing the output.  No warp waits for another but at a block's start, and sums have one order.
// 25 and 36 instructions an element, 12 of the slow kind (4 clocks of a quarter SM each) and some 45 packed or
// single multiply-adds (1.45 clocks with three register operands); 8 elements are moved for the 5 that are
// the least (x, r, i twice).  [8, 4096, 1536] bf16: 156 us (3.2 TB/s of the 5; 5.2 of the 8), [1, 65536, 1024] 196
// us, and 129 and 170 when first measured with no arithmetic but the maps'.  That is where all rates of 128
// neighbouring channels are below 0.125; the general form takes 192 and 239, that without rates 146 of the first.
// In one pass, with blocks of a cluster that hand the state on in step, these took 135 and 354 us (an exchange cost
// 0.7 us a step for two blocks, 1.4 for eight), and gradients 328 instead of 263; rows of a call in groups
// of L2's size between the two kernels were no faster (46 us for a quarter of the first case).  The maps walk a run
// from its end to its start, where the scan begins.
#include <type_traits>

#include "recur_internal.h"

namespace favor {

// Blocks an SM: 16 warps of 128 registers.  Three blocks of 80 spill (209 us instead of 157), two channels a lane or
// two tokens a group in their place 177; without the next group's rows on their way 169.
constexpr int kRecPerSm = 2;

// Grid: rows x chunks x slabs.
template <typename T, bool RATE, int SCALE>
__global__ void __launch_bounds__(kRecThreads, kRecPerSm) k_recur_maps(RecurArgs a, int D, RecurMapsAt at, F4* first) {
    constexpr int G = rec_group<T>();
    __shared__ RecurMap runs[kRecWarps][32];
    const int slab = blockIdx.x % at.p.slabs, rest = blockIdx.x / at.p.slabs;
    const int chunk = rest % at.p.chunks, b = rest / at.p.chunks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const RecurLane l(a, D, slab);
    const int len = row_len(a.lens, b, a.L);
    if (a.state && chunk == 0) {    // the state in front of the row, which the scan's last run will overwrite
        const int page = block_page(a.pg, b);
        if (warp == 0 && page >= 0)
            first[((size_t)b * at.p.slabs + slab) * 32 + lane] = load_vec(a.state + (size_t)page * D, l);
    }
    const int t0 = (chunk * kRecWarps + warp) * at.p.run, end = min(len, t0 + at.p.run);
    F4 mh = {both(0.f), both(0.f)};     // the run's map: its decays' product, and its state from an empty start
    RunDecay ma, mb;
    if (t0 < end) {
        const size_t row0 = (size_t)b * a.L * D;
        const T *x = (const T*)a.x + row0, *r = (const T*)a.r + row0, *gi = (const T*)a.i + row0;
        const RecurChan4 par = load_chans<T>(a, l);
        auto group = [&](auto slow, auto whole, int t, auto vx, auto vr, auto vi) {
            constexpr bool SLOW = decltype(slow)::value;
            RecurMaps<T> q;
            group_gates<T, RATE, SCALE, SLOW, decltype(whole)::value>(vx, vr, vi, a.i, par, t, end, q);
            F4 h = {both(0.f), both(0.f)};
            GroupDecay<SLOW> ga, gb;
#pragma unroll
            for (int s = 0; s < G; ++s) {
                h = next4<SLOW>(q.d[s], h, q.in[s]);
                ga.token(q.d[s].a);
                gb.token(q.d[s].b);
            }
            mh = {ma.apply(h.a, mh.a), mb.apply(h.b, mh.b)};
            ma.join(ga);
            mb.join(gb);
        };
        int t = t0 + (end - 1 - t0) / G * G;
        const int whole = l.quads ? (end - t0) / G * G : 0;     // tokens of whole groups, read 4 channels at a time
        for (; t >= t0 + whole; t -= G) {
            RecurRows<T> vx, vr, vi;
            load_rows<T, true, false>(x, l, t, end, vx);
            load_rows<T, true, false>(r, l, t, end, vr);
            if (a.i) load_rows<T, true, false>(gi, l, t, end, vi);
            group(std::false_type(), std::false_type(), t, vx, vr, vi);
        }
        auto walk = [&](auto slow) {
            RecurRows<T> nx, nr, ni;        // the next group's rows are on their way
            auto load = [&](int t) {
                load_rows<T, true, true>(x, l, t, end, nx);
                load_rows<T, true, true>(r, l, t, end, nr);
                if (a.i) load_rows<T, true, true>(gi, l, t, end, ni);
            };
            load(t);
            for (; t >= t0; t -= G) {
                const RecurRows<T> vx = nx, vr = nr, vi = ni;
                if (t > t0) load(t - G);
                group(slow, std::true_type(), t, vx, vr, vi);
            }
        };
        if (t >= t0) {
            if (RATE && par.a.slow) walk(std::integral_constant<bool, RATE>());
            else walk(std::false_type());
        }
    }
    RecurMap m = {{ma.value(), mb.value()}, mh};
    *at.run_at(b, chunk, warp, slab) = m;
    runs[warp][lane] = m;
    __syncthreads();
    if (warp == 0) {
#pragma unroll
        for (int w = 1; w < kRecWarps; ++w) m = join(m, runs[w][lane]);
        *at.chunk_at(b, chunk, slab) = m;
    }
}

template <typename T, bool RATE, int SCALE>
__global__ void __launch_bounds__(kRecThreads, kRecPerSm)
k_recur_scan(RecurArgs a, int D, RecurMapsAt at, const F4* first, bool one_run) {
    constexpr int G = rec_group<T>();
    __shared__ RecurPlaces places;
    const int slab = blockIdx.x % at.p.slabs, rest = blockIdx.x / at.p.slabs;
    const int chunk = rest % at.p.chunks, b = rest / at.p.chunks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const RecurLane l(a, D, slab);
    const int len = row_len(a.lens, b, a.L);
    const int page = a.state ? block_page(a.pg, b) : 0;
    const int t0 = (chunk * kRecWarps + warp) * at.p.run, end = page < 0 ? t0 : min(len, t0 + at.p.run);
    const size_t row0 = (size_t)b * a.L * D;
    const T *x = (const T*)a.x + row0, *r = (const T*)a.r + row0, *gi = (const T*)a.i + row0, *z = (const T*)a.z + row0;
    T* out = (T*)a.out + row0;
    float* state = a.state && page >= 0 ? a.state + (size_t)page * D : nullptr;
    F4 h = {both(0.f), both(0.f)};
    if (state) h = one_run ? load_vec(state, l) : first[((size_t)b * at.p.slabs + slab) * 32 + lane];
    if (!one_run) h = run_start<false>(at, b, chunk, slab, h, places);
    // zeros where the row takes no part, and behind its end if they are wanted
    clear_rows(out, l, max(t0, end), min(a.clear ? a.L : len, t0 + at.p.run));
    if (t0 >= end) return;
    const RecurChan4 par = load_chans<T>(a, l);
    auto group = [&](auto slow, auto whole, int t, auto vx, auto vr, auto vi, auto vz) {
        constexpr bool SLOW = decltype(slow)::value, WHOLE = decltype(whole)::value;
        RecurMaps<T> q;
        group_gates<T, RATE, SCALE, SLOW, WHOLE>(vx, vr, vi, a.i, par, t, end, q);
#pragma unroll
        for (int s = 0; s < G; ++s) q.in[s] = h = next4<SLOW>(q.d[s], h, q.in[s]);
        if (a.z) {
#pragma unroll
            for (int s = 0; s < G; ++s) {
                const F4 g = vz(s);
                q.in[s] = {q.in[s].a * silu2<T>(g.a), q.in[s].b * silu2<T>(g.b)};
            }
        }
#pragma unroll
        for (int s = 0; s < G; ++s)
            if (WHOLE || t + s < end) write_row<T, WHOLE>(out, l, t + s, q.in[s]);
    };
    int t = t0;
    const int whole = l.quads ? t0 + (end - t0) / G * G : t0;   // behind the whole groups
    auto walk = [&](auto slow) {
        RecurRows<T> nx, nr, ni, nz;
        auto load = [&](int t) {
            load_rows<T, false, true>(x, l, t, end, nx);
            load_rows<T, false, true>(r, l, t, end, nr);
            if (a.i) load_rows<T, false, true>(gi, l, t, end, ni);
            if (a.z) load_rows<T, false, true>(z, l, t, end, nz);
        };
        load(t);
        for (; t < whole; t += G) {
            const RecurRows<T> vx = nx, vr = nr, vi = ni, vz = nz;
            if (t + G < whole) load(t + G);
            group(slow, std::true_type(), t, vx, vr, vi, vz);
        }
    };
    if (t < whole) {
        if (RATE && par.a.slow) walk(std::integral_constant<bool, RATE>());
        else walk(std::false_type());
    }
    for (; t < end; t += G) {
        RecurRows<T> vx, vr, vi, vz;
        load_rows<T, false, false>(x, l, t, end, vx);
        load_rows<T, false, false>(r, l, t, end, vr);
        if (a.i) load_rows<T, false, false>(gi, l, t, end, vi);
        if (a.z) load_rows<T, false, false>(z, l, t, end, vz);
        group(std::false_type(), std::false_type(), t, vx, vr, vi, vz);
    }
    if (state && end == len) store_vec(state, l, h);
}

// One token a row; grid: rows x channel blocks.
constexpr int kRecStepThreads = 128;

template <typename T, bool RATE, int SCALE>
__global__ void __launch_bounds__(kRecStepThreads) k_recur_step(RecurArgs a, int D, int blocks) {
    const int b = blockIdx.x / blocks, slab = (blockIdx.x % blocks) * (kRecStepThreads / 32) + (threadIdx.x >> 5);
    const int page = block_page(a.pg, b);
    const RecurLane l(a, D, slab);
    const RecurChan4 par = load_chans<T>(a, l);
    F4 y = {both(0.f), both(0.f)};
    T* out = (T*)a.out + (size_t)b * D;
    if (page >= 0) {
        float* state = a.state + (size_t)page * D;
        const F4 h = load_vec(state, l);
        auto load = [&](const void* p) {
            RecurRows<T> v;
            const T* q = (const T*)p + (size_t)b * D;
            if (l.quads) load_rows<T, false, true, 1>(q, l, 0, 1, v);
            else load_rows<T, false, false, 1>(q, l, 0, 1, v);
            return to_f4(v.v[0]);
        };
        F4 v = load(a.x), gi, vz;
        const F4 r = load(a.r);
        if (a.i) gi = load(a.i);
        if (a.z) vz = load(a.z);
        const RecurGate g0 = recur_gate<T, RATE, SCALE, false, false>(r.a, par.a);
        const RecurGate g1 = recur_gate<T, RATE, SCALE, false, false>(r.b, par.b);
        if (a.i) v = {v.a * sigmoid2<T>(gi.a, par.a.i_bias), v.b * sigmoid2<T>(gi.b, par.b.i_bias)};
        if (SCALE != FAVOR_RECUR_PLAIN) v = {g0.w * v.a, g1.w * v.b};
        y = next4<false>(F4{g0.d, g1.d}, h, v);
        store_vec(state, l, y);
        if (a.z) y = {y.a * silu2<T>(vz.a), y.b * silu2<T>(vz.b)};
    }
    if (l.quads) write_row<T, true>(out, l, 0, y);
    else write_row<T, false>(out, l, 0, y);
}

// ------------------------------------------------------------------ host
template <typename T, bool RATE, int SCALE>
struct RecurScan {
    static void go(const RecurHandle& h, const RecurArgs& a, cudaStream_t st) {
        RecurMapsAt at = {};
        at.p = recur_plan(h.num_sms, kRecPerSm, h.D, a.B, a.L);
        at.run = reinterpret_cast<RecurMap*>(h.ws);
        at.chunk = reinterpret_cast<RecurMap*>(h.ws + recur_run_floats(at.p, a.B));
        F4* first = reinterpret_cast<F4*>(h.ws + recur_run_floats(at.p, a.B) + recur_chunk_floats(at.p, a.B));
        const unsigned blocks = (unsigned)a.B * at.p.chunks * at.p.slabs;
        const bool one_run = a.L <= at.p.run;
        if (!one_run) {
            k_recur_maps<T, RATE, SCALE><<<blocks, kRecThreads, 0, st>>>(a, h.D, at, first);
            count_launch();
        }
        k_recur_scan<T, RATE, SCALE><<<blocks, one_run ? 32 : kRecThreads, 0, st>>>(a, h.D, at, first, one_run);
        count_launch();
    }
};
template <typename T, bool RATE, int SCALE>
struct RecurStep {
    static void go(const RecurHandle& h, const RecurArgs& a, cudaStream_t st) {
        const int per = kRecStepThreads * 4, blocks = (h.D + per - 1) / per;
        k_recur_step<T, RATE, SCALE><<<(unsigned)a.B * blocks, kRecStepThreads, 0, st>>>(a, h.D, blocks);
        count_launch();
    }
};

// The maps of runs and chunks, and the rows' starts; nothing where every row is one run.
size_t recur_scan_ws(const RecurHandle& h) {
    if (h.max_L <= kRecRunMin) return 0;
    return recur_blocks_max(h.num_sms, kRecPerSm, h.D, h.max_B, h.max_L) * (kRecWarps + 1) * kRecMapFloats +
           (size_t)h.max_B * ((h.D + kRecSlab - 1) / kRecSlab) * 32 * (sizeof(F4) / 4);
}

favor_status recur_scan(const RecurHandle& h, const RecurArgs& a, cudaStream_t st) {
    recur_dispatch<RecurScan>(h, a.rate != nullptr, h, a, st);
    return check_launch("favor_recur_scan");
}

favor_status recur_step(const RecurHandle& h, const RecurArgs& a, cudaStream_t st) {
    recur_dispatch<RecurStep>(h, a.rate != nullptr, h, a, st);
    return check_launch("favor_recur_step");
}

}  // namespace favor
