// Pages of a cache of recurrent states: a pool is n_pages blocks of page_bytes
// bytes.  Copying (forking), clearing and compacting move or write whole pages;
// each is bound by the bytes it moves.
#include "ssm_internal.h"

namespace favor {

// Bytes of a page that one block moves: 256 threads x 8 accesses of 16 bytes, so
// that a thread has 8 independent loads in flight (48 pages of 0.8 MB: 12.6 us, 6.1
// TB/s).
constexpr int kPageThreads = 256;
constexpr int kPageUnroll = 8;

template <typename W>
__device__ __forceinline__ void copy_slice(W* dst, const W* src, size_t n, size_t first) {
    W r[kPageUnroll];
#pragma unroll
    for (int i = 0; i < kPageUnroll; ++i) {
        const size_t at = first + (size_t)i * kPageThreads + threadIdx.x;
        if (at < n) r[i] = src[at];
    }
#pragma unroll
    for (int i = 0; i < kPageUnroll; ++i) {
        const size_t at = first + (size_t)i * kPageThreads + threadIdx.x;
        if (at < n) dst[at] = r[i];
    }
}

// Block = one slice of one pair.  The block decides for itself whether its pair
// is carried out, by the same rule in every block of the pair: both pages exist,
// no earlier pair names the destination, and (one pool) no pair reads it.
template <typename W>
__global__ void __launch_bounds__(kPageThreads)
k_pages_copy(W* dst_pool, int n_dst, const W* src_pool, int n_src, size_t words, int slices, const int* src,
             const int* dst, int n, int* done) {
    const int i = blockIdx.x / slices, sl = blockIdx.x % slices;
    const int s = src[i], d = dst[i];
    const bool one = (const void*)dst_pool == (const void*)src_pool;
    const bool self = one && s == d;
    int bad = s < 0 || s >= n_src || d < 0 || d >= n_dst;
    for (int j = threadIdx.x; j < n; j += kPageThreads) {
        if (j < i) bad |= dst[j] == d;
        if (one && !self) bad |= src[j] == d;
    }
    bad = __syncthreads_or(bad);
    if (done && sl == 0 && threadIdx.x == 0) done[i] = !bad;
    if (bad || self) return;
    copy_slice(dst_pool + (size_t)d * words, src_pool + (size_t)s * words, words,
               (size_t)sl * kPageThreads * kPageUnroll);
}

template <typename W>
__global__ void __launch_bounds__(kPageThreads)
k_pages_clear(W* pool, int n_pages, size_t words, int slices, const int* pages) {
    const int i = blockIdx.x / slices, sl = blockIdx.x % slices;
    const int p = pages[i];
    if (p < 0 || p >= n_pages) return;
    W zero;
    memset(&zero, 0, sizeof(W));
    W* d = pool + (size_t)p * words;
#pragma unroll
    for (int k = 0; k < kPageUnroll; ++k) {
        const size_t at = ((size_t)sl * kPageUnroll + k) * kPageThreads + threadIdx.x;
        if (at < words) d[at] = zero;
    }
}

// ---- compacting
// U live pages (named by the table) end in pages 0..U-1: those below U stay, the
// k-th live page at or above U (in order) goes to the k-th free page below U.
// Every block makes the same plan from the table in shared memory (a bit per
// page and the running count of each 32-page word), so that one launch does both
// the plan and the moves; sources are >= U and destinations < U, so no move
// touches another's page.
constexpr int kMaxPages = 1 << 17;

struct PagePlan {
    const uint32_t* bits;   // live pages
    const int* before;      // live pages in earlier words
    int n_pages;
    int live;               // U
    int low_live;           // live pages below U
    __device__ int live_before(int p) const {
        return before[p >> 5] + __popc(bits[p >> 5] & ((1u << (p & 31)) - 1u));
    }
    __device__ bool is_live(int p) const { return bits[p >> 5] >> (p & 31) & 1u; }
    // The page with k free pages before it: the last word whose free count is <= k.
    __device__ int kth_free(int k) const {
        int lo = 0, hi = ((live + 31) >> 5) - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (mid * 32 - before[mid] <= k) lo = mid;
            else hi = mid - 1;
        }
        uint32_t w = ~bits[lo];
        for (int r = k - (lo * 32 - before[lo]); r > 0; --r) w &= w - 1;
        return lo * 32 + __ffs(w) - 1;
    }
    // Where page p is after the compaction (-1: it is free).
    __device__ int target(int p) const {
        if (!is_live(p)) return -1;
        return p < live ? p : kth_free(live_before(p) - low_live);
    }
};

template <typename W>
__global__ void __launch_bounds__(kPageThreads)
k_pages_compact(W* pool, int n_pages, size_t words, int slices, const int* table, int S, int* new_table,
                int* page_map, int* n_live) {
    extern __shared__ uint32_t sm[];
    const int nw = (n_pages + 31) >> 5;
    uint32_t* bits = sm;
    int* before = reinterpret_cast<int*>(sm + nw);
    __shared__ int part[kPageThreads], total;
    for (int i = threadIdx.x; i < nw; i += kPageThreads) bits[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < S; i += kPageThreads) {
        const int p = table[i];
        if (p >= 0 && p < n_pages) atomicOr(&bits[p >> 5], 1u << (p & 31));
    }
    __syncthreads();
    // exclusive running count: a run of words per thread, then the runs
    const int per = (nw + kPageThreads - 1) / kPageThreads;
    const int w0 = threadIdx.x * per, w1 = min(nw, w0 + per);
    int sum = 0;
    for (int i = w0; i < w1; ++i) sum += __popc(bits[i]);
    part[threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.x < 32) {
        int run[kPageThreads / 32], mine = 0;
#pragma unroll
        for (int k = 0; k < kPageThreads / 32; ++k) {
            run[k] = part[threadIdx.x * (kPageThreads / 32) + k];
            mine += run[k];
        }
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if ((int)threadIdx.x >= o) inc += v;
        }
        int ex = inc - mine;
#pragma unroll
        for (int k = 0; k < kPageThreads / 32; ++k) {
            part[threadIdx.x * (kPageThreads / 32) + k] = ex;
            ex += run[k];
        }
        if (threadIdx.x == 31) total = inc;
    }
    __syncthreads();
    sum = part[threadIdx.x];
    for (int i = w0; i < w1; ++i) {
        before[i] = sum;
        sum += __popc(bits[i]);
    }
    __syncthreads();
    PagePlan plan{bits, before, n_pages, total, 0};
    plan.low_live = total < n_pages ? plan.live_before(total) : total;
    const int grid_threads = gridDim.x * kPageThreads, gt = blockIdx.x * kPageThreads + threadIdx.x;
    for (int i = gt; i < S; i += grid_threads) {
        const int p = table[i];
        new_table[i] = p >= 0 && p < n_pages ? plan.target(p) : -1;
    }
    if (page_map)
        for (int p = gt; p < n_pages; p += grid_threads) page_map[p] = plan.target(p);
    if (gt == 0) *n_live = total;
    // The moves, slice by slice: move m is (k-th live page >= U) -> (k-th free page < U), k = m.
    const int moves = total - plan.low_live;
    const long long items = (long long)moves * slices;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int k = (int)(it / slices), sl = (int)(it % slices);
        // k-th live page at or above U: the last word with at most low_live + k live pages before it
        const int want = plan.low_live + k;
        int lo = 0, hi = nw - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (before[mid] <= want) lo = mid;
            else hi = mid - 1;
        }
        uint32_t w = bits[lo];
        for (int r = want - before[lo]; r > 0; --r) w &= w - 1;
        const int s = lo * 32 + __ffs(w) - 1, d = plan.kth_free(k);
        copy_slice(pool + (size_t)d * words, pool + (size_t)s * words, words,
                   (size_t)sl * kPageThreads * kPageUnroll);
    }
}

// A further pool moved by the map of a compaction: page p goes to page_map[p],
// which has to be a page that the map calls free.
template <typename W>
__global__ void __launch_bounds__(kPageThreads)
k_pages_move(W* pool, int n_pages, size_t words, int slices, const int* page_map) {
    const int p = blockIdx.x / slices, sl = blockIdx.x % slices;
    const int d = page_map[p];
    if (d == p || d < 0 || d >= n_pages || page_map[d] >= 0) return;
    copy_slice(pool + (size_t)d * words, pool + (size_t)p * words, words, (size_t)sl * kPageThreads * kPageUnroll);
}

// Widest access that every page of the pools starts on and is a multiple of.
static int word_bytes(const void* a, const void* b, size_t page_bytes) {
    const uintptr_t m = reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) | page_bytes;
    return m % 16 == 0 ? 16 : m % 4 == 0 ? 4 : m % 2 == 0 ? 2 : 1;
}

static bool ranges_overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

static bool int_aligned(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

static favor_status check_pool(const char* fn, const void* pool, int n_pages, size_t page_bytes) {
    if (!pool) return set_error(FAVOR_ERR_INVALID_ARG, "%s: null pool", fn);
    if (n_pages < 1 || page_bytes < 1)
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: n_pages=%d page_bytes=%zu must be >= 1", fn, n_pages, page_bytes);
    if (page_bytes > ((size_t)1 << 40) / (size_t)n_pages)
        return set_error(FAVOR_ERR_UNSUPPORTED, "%s: pool of more than 2^40 bytes", fn);
    return FAVOR_OK;
}

// Blocks of an n-page call; 0 if the grid would be too large.
static unsigned page_grid(long long n, size_t words, int* slices) {
    const size_t per = (size_t)kPageThreads * kPageUnroll, s = (words + per - 1) / per;
    if (s > 0x7fffffff || (long long)s > 0x7fffffffLL / n) return 0;
    *slices = (int)s;
    return (unsigned)(n * (long long)s);
}

}  // namespace favor

using namespace favor;

#define FAVOR_BY_WORD(wb, CALL)                          \
    do {                                                 \
        if (wb == 16) { using W = uint4; CALL; }         \
        else if (wb == 4) { using W = uint32_t; CALL; }  \
        else if (wb == 2) { using W = uint16_t; CALL; }  \
        else { using W = uint8_t; CALL; }                \
    } while (0)

extern "C" {

favor_status favor_pages_copy(void* dst_pool, int n_dst, const void* src_pool, int n_src, size_t page_bytes,
                              const int* src, const int* dst, int n, int* done, void* stream) {
    const char* fn = "favor_pages_copy";
    set_error(FAVOR_OK, "%s", "");
    favor_status st = check_pool(fn, dst_pool, n_dst, page_bytes);
    if (st == FAVOR_OK) st = check_pool(fn, src_pool, n_src, page_bytes);
    if (st != FAVOR_OK) return st;
    if (!src || !dst) return set_error(FAVOR_ERR_INVALID_ARG, "%s: null index pointer", fn);
    if (n < 1) return set_error(FAVOR_ERR_INVALID_ARG, "%s: n=%d must be >= 1", fn, n);
    if (!int_aligned(src) || !int_aligned(dst) || !int_aligned(done))
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: an index pointer is not aligned", fn);
    const size_t ib = (size_t)n * 4, db = (size_t)n_dst * page_bytes;
    if (ranges_overlap(src, ib, dst_pool, db) || ranges_overlap(dst, ib, dst_pool, db) ||
        (done && (ranges_overlap(done, ib, dst_pool, db) || ranges_overlap(done, ib, src, ib) ||
                  ranges_overlap(done, ib, dst, ib) || ranges_overlap(done, ib, src_pool, (size_t)n_src * page_bytes))))
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: the indices, done and the pools must not overlap", fn);
    if (dst_pool != src_pool &&
        ranges_overlap(dst_pool, (size_t)n_dst * page_bytes, src_pool, (size_t)n_src * page_bytes))
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: the pools overlap without being the same", fn);
    const int wb = word_bytes(dst_pool, src_pool, page_bytes);
    int slices = 0;
    const unsigned grid = page_grid(n, page_bytes / wb, &slices);
    if (!grid) return set_error(FAVOR_ERR_UNSUPPORTED, "%s: n * page_bytes too large", fn);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    FAVOR_BY_WORD(wb, (k_pages_copy<W><<<grid, kPageThreads, 0, s>>>((W*)dst_pool, n_dst, (const W*)src_pool, n_src,
                                                                     page_bytes / wb, slices, src, dst, n, done)));
    count_launch();
    return check_launch(fn);
}

favor_status favor_pages_clear(void* pool, int n_pages, size_t page_bytes, const int* pages, int n, void* stream) {
    const char* fn = "favor_pages_clear";
    set_error(FAVOR_OK, "%s", "");
    favor_status st = check_pool(fn, pool, n_pages, page_bytes);
    if (st != FAVOR_OK) return st;
    if (!pages) return set_error(FAVOR_ERR_INVALID_ARG, "%s: null index pointer", fn);
    if (n < 1) return set_error(FAVOR_ERR_INVALID_ARG, "%s: n=%d must be >= 1", fn, n);
    if (!int_aligned(pages)) return set_error(FAVOR_ERR_INVALID_ARG, "%s: an index pointer is not aligned", fn);
    if (ranges_overlap(pages, (size_t)n * 4, pool, (size_t)n_pages * page_bytes))
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: the indices and the pool must not overlap", fn);
    const int wb = word_bytes(pool, pool, page_bytes);
    int slices = 0;
    const unsigned grid = page_grid(n, page_bytes / wb, &slices);
    if (!grid) return set_error(FAVOR_ERR_UNSUPPORTED, "%s: n * page_bytes too large", fn);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    FAVOR_BY_WORD(wb, (k_pages_clear<W><<<grid, kPageThreads, 0, s>>>((W*)pool, n_pages, page_bytes / wb, slices,
                                                                      pages)));
    count_launch();
    return check_launch(fn);
}

favor_status favor_pages_compact(void* pool, int n_pages, size_t page_bytes, const int* table, int S, int* new_table,
                                 int* page_map, int* n_live, void* stream) {
    const char* fn = "favor_pages_compact";
    set_error(FAVOR_OK, "%s", "");
    favor_status st = check_pool(fn, pool, n_pages, page_bytes);
    if (st != FAVOR_OK) return st;
    if (!table || !new_table || !n_live) return set_error(FAVOR_ERR_INVALID_ARG, "%s: null table pointer", fn);
    if (S < 1) return set_error(FAVOR_ERR_INVALID_ARG, "%s: S=%d must be >= 1", fn, S);
    if (n_pages > kMaxPages)
        return set_error(FAVOR_ERR_UNSUPPORTED, "%s: n_pages=%d (at most %d)", fn, n_pages, kMaxPages);
    if (!int_aligned(table) || !int_aligned(new_table) || !int_aligned(page_map) || !int_aligned(n_live))
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: an index pointer is not aligned", fn);
    const size_t tb = (size_t)S * 4, pb = (size_t)n_pages * page_bytes;
    if (ranges_overlap(table, tb, pool, pb) || ranges_overlap(new_table, tb, pool, pb) ||
        ranges_overlap(n_live, 4, pool, pb) || (page_map && ranges_overlap(page_map, (size_t)n_pages * 4, pool, pb)))
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: the tables and the pool must not overlap", fn);
    if (ranges_overlap(table, tb, new_table, tb) || ranges_overlap(table, tb, n_live, 4) ||
        ranges_overlap(new_table, tb, n_live, 4) ||
        (page_map && (ranges_overlap(table, tb, page_map, (size_t)n_pages * 4) ||
                      ranges_overlap(new_table, tb, page_map, (size_t)n_pages * 4) ||
                      ranges_overlap(n_live, 4, page_map, (size_t)n_pages * 4))))
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: table, new_table, page_map and n_live must not overlap", fn);
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return set_error(FAVOR_ERR_CUDA, "%s: no usable CUDA device", fn);
    }
    const int wb = word_bytes(pool, pool, page_bytes);
    int slices = 0;
    const unsigned most = page_grid((n_pages + 1) / 2, page_bytes / wb, &slices);   // at most half the pages move
    if (!most) return set_error(FAVOR_ERR_UNSUPPORTED, "%s: n_pages * page_bytes too large", fn);
    // every block repeats the plan, so no more blocks than run at once
    const unsigned grid = most < (unsigned)sms * 8 ? most : (unsigned)sms * 8;
    const size_t smem = (size_t)((n_pages + 31) / 32) * 8;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    FAVOR_BY_WORD(wb, (k_pages_compact<W><<<grid, kPageThreads, smem, s>>>((W*)pool, n_pages, page_bytes / wb, slices,
                                                                           table, S, new_table, page_map, n_live)));
    count_launch();
    return check_launch(fn);
}

favor_status favor_pages_move(void* pool, int n_pages, size_t page_bytes, const int* page_map, void* stream) {
    const char* fn = "favor_pages_move";
    set_error(FAVOR_OK, "%s", "");
    favor_status st = check_pool(fn, pool, n_pages, page_bytes);
    if (st != FAVOR_OK) return st;
    if (!page_map) return set_error(FAVOR_ERR_INVALID_ARG, "%s: null page_map", fn);
    if (!int_aligned(page_map)) return set_error(FAVOR_ERR_INVALID_ARG, "%s: an index pointer is not aligned", fn);
    if (ranges_overlap(page_map, (size_t)n_pages * 4, pool, (size_t)n_pages * page_bytes))
        return set_error(FAVOR_ERR_INVALID_ARG, "%s: the map and the pool must not overlap", fn);
    const int wb = word_bytes(pool, pool, page_bytes);
    int slices = 0;
    const unsigned grid = page_grid(n_pages, page_bytes / wb, &slices);
    if (!grid) return set_error(FAVOR_ERR_UNSUPPORTED, "%s: n_pages * page_bytes too large", fn);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    FAVOR_BY_WORD(wb, (k_pages_move<W><<<grid, kPageThreads, 0, s>>>((W*)pool, n_pages, page_bytes / wb, slices,
                                                                     page_map)));
    count_launch();
    return check_launch(fn);
}

}  // extern "C"
