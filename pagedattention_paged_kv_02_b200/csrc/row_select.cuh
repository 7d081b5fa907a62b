// row_select.cuh -- the k largest of a row of keys, by a cluster of CTAs.
//
// A row (block scores of one K/V head, attention weights of one K/V head) is
// cut into consecutive segments, one per CTA of a thread-block cluster. The
// k-th largest key is found digit by digit from the top (radix selection):
// each round every CTA counts the next 8-bit digit of its keys that share the
// digits found so far, the counts are added up over the cluster through
// distributed shared memory, and the digit that holds the k-th largest is the
// next one of the cut. Every CTA adds up the same counts, so all of them
// agree on the cut without a second exchange, and nothing depends on timing.
// Of the keys equal to the cut the ones of lowest index are taken. The taken
// items are handed out in ascending order of index: an item's place is the
// number of taken items before it, from per-CTA counts and a scan inside the
// CTA.
#pragma once

#include <cooperative_groups.h>

#include "pa_device.cuh"

namespace pa {

namespace cg = cooperative_groups;

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

struct RowSelectSmem {
    uint32_t hist[2][256];
    uint32_t total[256];
    uint32_t digit, above, in_digit;
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

// The cut that takes `need` items of the cluster's row; key_at(i), i < n, are
// this CTA's keys. 1 <= need <= items of the row. Called by every thread of
// every CTA of the cluster.
template <int THREADS, typename Key, typename KeyAt>
__device__ __forceinline__ Cut<Key> cluster_cut(cg::cluster_group &cluster, RowSelectSmem &sm,
                                                const KeyAt &key_at, int n, uint32_t need) {
    const int tid = threadIdx.x;
    const int ranks = (int)cluster.num_blocks();
    Key prefix = 0;
#pragma unroll 1
    for (int round = 0; round < (int)sizeof(Key); ++round) {
        const int shift = 8 * ((int)sizeof(Key) - 1 - round);
        // the other CTAs last read this half two rounds ago, before the
        // cluster barrier of the round in between
        uint32_t *h = sm.hist[round & 1];
        for (int t = tid; t < 256; t += THREADS) h[t] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += THREADS) {
            const Key k = key_at(i);
            if (round == 0 || (Key)(k >> shift >> 8) == prefix)
                atomicAdd(h + ((uint32_t)(k >> shift) & 255u), 1u);
        }
        cluster.sync();
        for (int t = tid; t < 256; t += THREADS) {
            uint32_t c = 0;
            for (int r = 0; r < ranks; ++r) c += cluster.map_shared_rank(h, r)[t];
            sm.total[t] = c;
        }
        __syncthreads();
        if (tid < 32) {  // lane l owns digits 255 - 8l .. 248 - 8l
            uint32_t mine = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) mine += sm.total[255 - 8 * tid - j];
            uint32_t upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
                if (tid >= o) upto += y;
            }
            uint32_t above = upto - mine;
            if (above < need && need <= upto) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t c = sm.total[255 - 8 * tid - j];
                    if (above < need && need <= above + c) {
                        sm.digit = 255 - 8 * tid - j;
                        sm.above = above;
                        sm.in_digit = c;
                        break;
                    }
                    above += c;
                }
            }
        }
        __syncthreads();
        prefix = (Key)(prefix << 8) | (Key)sm.digit;
        need -= sm.above;
        // all keys that share these digits are taken: the rest of the digits
        // cannot matter
        if (sm.in_digit == need) return {(Key)(prefix << shift), 0xffffffffu};
    }
    return {prefix, need};
}

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

// emit(place, i) for every item i < n of this CTA with taken(i), place
// ascending with i from `place`.
template <int THREADS, typename Taken, typename Emit>
__device__ __forceinline__ void block_emit(RowSelectSmem &sm, int n, uint32_t place,
                                           const Taken &taken, const Emit &emit) {
    for (int t0 = 0; t0 < n; t0 += THREADS * kSelItems) {
        const int i0 = t0 + (int)threadIdx.x * kSelItems;
        uint32_t in = 0;
#pragma unroll
        for (int u = 0; u < kSelItems; ++u)
            if (i0 + u < n) in |= (uint32_t)taken(i0 + u) << u;
        uint32_t all;
        uint32_t at = place + block_before<THREADS>(sm, __popc(in), all);
#pragma unroll
        for (int u = 0; u < kSelItems; ++u)
            if ((in >> u) & 1u) emit((int)at++, i0 + u);
        place += all;
    }
}

// emit(place, i) for every taken item i of this CTA, place ascending with i
// from the cluster's first item on. Every thread of the cluster calls it; a
// cluster barrier must follow before a CTA exits or reuses `sm`.
template <int THREADS, typename Key, typename KeyAt, typename Emit>
__device__ __forceinline__ void cluster_emit(cg::cluster_group &cluster, RowSelectSmem &sm,
                                             const KeyAt &key_at, int n, const Cut<Key> &cut,
                                             const Emit &emit) {
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid < 2) sm.count[tid] = 0;
    __syncthreads();
    uint32_t gt = 0, eq = 0;
    for (int i = tid; i < n; i += THREADS) {
        const Key k = key_at(i);
        gt += k > cut.key;
        eq += k == cut.key;
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
        atomicAdd(&sm.count[0], gt);
        atomicAdd(&sm.count[1], eq);
    }
    cluster.sync();
    uint32_t gt_base = 0, eq_base = 0;
    for (int r = 0; r < (int)cluster.block_rank(); ++r) {
        const uint32_t *c = cluster.map_shared_rank(sm.count, r);
        gt_base += c[0];
        eq_base += c[1];
    }
    for (int t0 = 0; t0 < n; t0 += THREADS * kSelItems) {
        const int i0 = t0 + tid * kSelItems;
        uint32_t is_gt = 0, is_eq = 0;
#pragma unroll
        for (int u = 0; u < kSelItems; ++u) {
            if (i0 + u < n) {
                const Key k = key_at(i0 + u);
                is_gt |= (uint32_t)(k > cut.key) << u;
                is_eq |= (uint32_t)(k == cut.key) << u;
            }
        }
        // counts before this thread's items: above in the low half, equal in
        // the high half (a tile has THREADS * kSelItems < 65536 items)
        const uint32_t mine = __popc(is_gt) | (__popc(is_eq) << 16);
        uint32_t all;
        const uint32_t before = block_before<THREADS>(sm, mine, all);
        uint32_t g = gt_base + (before & 0xffffu), e = eq_base + (before >> 16);
#pragma unroll
        for (int u = 0; u < kSelItems; ++u) {
            const bool ug = (is_gt >> u) & 1u, ue = (is_eq >> u) & 1u;
            if (ug || (ue && e < cut.ties)) emit((int)(g + min(e, cut.ties)), i0 + u);
            g += ug;
            e += ue;
        }
        gt_base += all & 0xffffu;
        eq_base += all >> 16;
    }
}

}  // namespace pa
