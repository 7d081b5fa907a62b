// row_select.cuh -- the k largest of a row of keys, by one CTA or a cluster.
//
// A row is one K/V head's keys: its attention weights (evict.cuh), cut into
// consecutive segments, one per CTA of a thread-block cluster, or held by one CTA
// where they are few; or its block scores (select_blocks.cuh), which one CTA
// holds. The k-th largest key is closed in on: each round every CTA counts its
// keys in 1024 equal bins over the range that is left, the counts are added up
// over the cluster through distributed shared memory, and the bin that holds the
// k-th largest is the next range -- ten bits a round, from the bits in which the
// row's keys differ at all, and done as soon as the bin is taken whole. Every CTA
// adds up the same counts, so all of them agree on the cut without a second
// exchange, and nothing depends on timing.
// Of the keys equal to the cut the ones of lowest index are taken. The taken
// items are handed out in ascending order of index: an item's place is the
// number of taken items before it, from per-CTA counts and a scan inside the
// CTA.
#pragma once

#include <cooperative_groups.h>

#include "pa_device.cuh"

namespace pa {

// The CTAs that share a row: a thread-block cluster, or one CTA alone.
struct CtaCluster {
    cooperative_groups::cluster_group g = cooperative_groups::this_cluster();
    __device__ __forceinline__ int ranks() const { return (int)g.num_blocks(); }
    __device__ __forceinline__ int rank() const { return (int)g.block_rank(); }
    __device__ __forceinline__ void sync() const { g.sync(); }
    template <typename T>
    __device__ __forceinline__ T *at(T *p, int r) const {  // p in CTA r's shared memory
        return g.map_shared_rank(p, r);
    }
};
struct OneCta {
    __device__ __forceinline__ int ranks() const { return 1; }
    __device__ __forceinline__ int rank() const { return 0; }
    __device__ __forceinline__ void sync() const { __syncthreads(); }
    template <typename T>
    __device__ __forceinline__ T *at(T *p, int) const {
        return p;
    }
};

constexpr int kSelItems = 4;      // consecutive items per thread in the scan
constexpr int kSelMaxWarps = 32;
constexpr int kMaxCluster = 8;    // portable cluster size

// Unsigned keys in the order of the values; -0 equals +0 and a NaN, of either
// sign, is above every number. Key 0 is below every value's key.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0xffffffffu;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t order_key(double x) {
    if (x != x) return ~0ull;
    const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
    return (u >> 63) ? ~u : u | (1ull << 63);
}

constexpr int kCutBins = 1024;

struct RowSelectSmem {
    alignas(16) uint32_t bins[2][kCutBins];
    unsigned long long lo, hi;        // range of this CTA's keys
    uint32_t border, above, in_border;
    uint32_t count[2];                // this CTA's items above the cut, equal to it
    uint32_t warp_count[kSelMaxWarps];
};

// Items with a key above `key`, and the first `ties` (in order of index) of
// those equal to it.
template <typename Key>
struct Cut {
    Key key;
    uint32_t ties;
};

// Sum of `mine` over the threads before this one, and over all in `all`.
template <int THREADS>
__device__ __forceinline__ uint32_t block_before(RowSelectSmem &sm, uint32_t mine, uint32_t &all) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    if (lane == 31) sm.warp_count[warp] = upto;
    __syncthreads();
    uint32_t before = upto - mine;
    all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        const uint32_t c = sm.warp_count[w];
        if (w < warp) before += c;
        all += c;
    }
    __syncthreads();  // before the next use of warp_count
    return before;
}

// Bits of a key that can differ within a range.
__device__ __forceinline__ int bit_width(uint32_t x) { return 32 - __clz(x); }
__device__ __forceinline__ int bit_width(uint64_t x) { return 64 - __clzll((long long)x); }

// The cut that takes `need` items of the cluster's row; key_at(i), i < n, are
// this CTA's keys. 1 <= need <= items of the row. Called by every thread of
// every CTA of the cluster; a cluster barrier must come between two calls.
template <int THREADS, typename Key, typename Row, typename KeyAt>
__device__ __forceinline__ Cut<Key> cluster_cut(const Row &cluster, RowSelectSmem &sm,
                                                const KeyAt &key_at, int n, uint32_t need) {
    constexpr int PER = kCutBins / THREADS;  // bins of a thread, from the top down
    const int tid = threadIdx.x;
    const int ranks = cluster.ranks();
    if (tid == 0) {
        sm.lo = ~0ull;
        sm.hi = 0;
    }
    __syncthreads();
    Key lo = ~(Key)0, hi = 0;
#pragma unroll 4
    for (int i = tid; i < n; i += THREADS) {
        const Key k = key_at(i);
        lo = min(lo, k);
        hi = max(hi, k);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    if ((tid & 31) == 0) {
        atomicMin(&sm.lo, (unsigned long long)lo);
        atomicMax(&sm.hi, (unsigned long long)hi);
    }
    cluster.sync();
    for (int r = 0; r < ranks; ++r) {
        const RowSelectSmem *o = cluster.at(&sm, r);
        const Key l = (Key)o->lo, u = (Key)o->hi;  // (a CTA without keys: the widest lo, 0)
        lo = r == 0 ? l : min(lo, l);
        hi = r == 0 ? u : max(hi, u);
    }
    for (int round = 0;; ++round) {
        const int shift = max(0, bit_width((Key)(hi - lo)) - 10);
        // the other CTAs last read this half two rounds ago, before the
        // cluster barrier of the round in between
        uint32_t *bins = sm.bins[round & 1];
        for (int t = tid; t < kCutBins; t += THREADS) bins[t] = 0;
        __syncthreads();
#pragma unroll 4
        for (int i = tid; i < n; i += THREADS) {
            const Key k = key_at(i);
            if (k >= lo && k <= hi) atomicAdd(bins + (uint32_t)((k - lo) >> shift), 1u);
        }
        cluster.sync();
        uint32_t c[PER] = {};
        for (int r = 0; r < ranks; ++r) {
            const uint32_t *p = cluster.at(bins, r) + kCutBins - (tid + 1) * PER;
#pragma unroll
            for (int j = 0; j < PER; ++j) c[PER - 1 - j] += p[j];
        }
        uint32_t mine = 0, all;
#pragma unroll
        for (int j = 0; j < PER; ++j) mine += c[j];
        uint32_t above = block_before<THREADS>(sm, mine, all);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            if (above < need && need <= above + c[j]) {
                sm.border = kCutBins - 1 - tid * PER - j;
                sm.above = above;
                sm.in_border = c[j];
            }
            above += c[j];
        }
        __syncthreads();
        need -= sm.above;
        lo += (Key)sm.border << shift;
        // a bin that is taken whole needs no closer look
        if (sm.in_border == need) return {lo, 0xffffffffu};
        if (shift == 0) return {lo, need};
        hi = lo + min((Key)(hi - lo), (Key)(((Key)1 << shift) - 1));
        __syncthreads();  // before border and above are written again
    }
}

// emit(place, i) for every item i < n of this CTA with taken(i), place
// ascending with i from 0. A warp owns a run of items, counts and then emits
// the taken ones by ballots: one barrier.
template <int THREADS, typename Taken, typename Emit>
__device__ __forceinline__ void block_emit(RowSelectSmem &sm, int n, const Taken &taken,
                                           const Emit &emit) {
    constexpr int W = THREADS / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int run = (n + THREADS - 1) / THREADS * 32;
    const int begin = min(warp * run, n), end = min(begin + run, n);
    uint32_t mine = 0;
#pragma unroll 4
    for (int i = begin + lane; i < end; i += 32) mine += taken(i);
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) sm.warp_count[warp] = mine;
    __syncthreads();
    uint32_t place = __reduce_add_sync(0xffffffffu,
                                       lane < W && lane < warp ? sm.warp_count[lane] : 0u);
    for (int i0 = begin; i0 < end; i0 += 32) {
        const bool in = i0 + lane < end && taken(i0 + lane);
        const uint32_t who = __ballot_sync(0xffffffffu, in);
        if (in) emit((int)(place + __popc(who & ((1u << lane) - 1))), i0 + lane);
        place += __popc(who);
    }
}

// emit(place, i) for every taken item i of this CTA, place ascending with i
// from the cluster's first item on. sm.count holds this CTA's items above the
// cut and equal to it, written before the cluster last met; items(i0, k) fetches
// the ITEMS keys from i0 on, 0 (below every cut) past the end. Every thread of
// the cluster calls it; a cluster barrier must follow before a CTA exits or
// reuses `sm`.
template <int THREADS, int ITEMS, typename Key, typename Row, typename Items, typename Emit>
__device__ __forceinline__ void cluster_place(const Row &cluster, RowSelectSmem &sm,
                                              const Items &items, int n, const Cut<Key> &cut,
                                              const Emit &emit) {
    uint32_t gt_base = 0, eq_base = 0;
    for (int r = 0; r < cluster.rank(); ++r) {
        const uint32_t *c = cluster.at(sm.count, r);
        gt_base += c[0];
        eq_base += c[1];
    }
    for (int t0 = 0; t0 < n; t0 += THREADS * ITEMS) {
        const int i0 = t0 + (int)threadIdx.x * ITEMS;
        uint32_t is_gt = 0, is_eq = 0;
        Key k[ITEMS];
        items(i0, k);
#pragma unroll
        for (int u = 0; u < ITEMS; ++u) {
            is_gt |= (uint32_t)(k[u] > cut.key) << u;
            is_eq |= (uint32_t)(k[u] == cut.key) << u;
        }
        // counts before this thread's items: above in the low half, equal in
        // the high half (a tile has THREADS * ITEMS < 65536 items)
        const uint32_t mine = __popc(is_gt) | (__popc(is_eq) << 16);
        uint32_t all;
        const uint32_t before = block_before<THREADS>(sm, mine, all);
        uint32_t g = gt_base + (before & 0xffffu), e = eq_base + (before >> 16);
#pragma unroll
        for (int u = 0; u < ITEMS; ++u) {
            const bool ug = (is_gt >> u) & 1u, ue = (is_eq >> u) & 1u;
            if (ug || (ue && e < cut.ties)) emit((int)(g + min(e, cut.ties)), i0 + u);
            g += ug;
            e += ue;
        }
        gt_base += all & 0xffffu;
        eq_base += all >> 16;
    }
}

// Adds a thread's counts of items above the cut and equal to it to its CTA's.
__device__ __forceinline__ void add_counts(RowSelectSmem &sm, uint32_t gt, uint32_t eq) {
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if ((threadIdx.x & 31) == 0) {
        atomicAdd(&sm.count[0], gt);
        atomicAdd(&sm.count[1], eq);
    }
}

// The same from the cut alone; cut.key > 0.
template <int THREADS, typename Key, typename Row, typename KeyAt, typename Emit>
__device__ __forceinline__ void cluster_emit(const Row &cluster, RowSelectSmem &sm,
                                             const KeyAt &key_at, int n, const Cut<Key> &cut,
                                             const Emit &emit) {
    if (threadIdx.x < 2) sm.count[threadIdx.x] = 0;
    __syncthreads();
    uint32_t gt = 0, eq = 0;
    for (int i = threadIdx.x; i < n; i += THREADS) {
        const Key k = key_at(i);
        gt += k > cut.key;
        eq += k == cut.key;
    }
    add_counts(sm, gt, eq);
    cluster.sync();
    cluster_place<THREADS, kSelItems>(
        cluster, sm,
        [&](int i0, Key(&k)[kSelItems]) {
#pragma unroll
            for (int u = 0; u < kSelItems; ++u) k[u] = i0 + u < n ? key_at(i0 + u) : 0;
        },
        n, cut, emit);
}

}  // namespace pa
