// select_blocks.cuh -- the blocks each query is worth attending to.
//
// For row b and K/V head h, block j of the row's table (n = ceil(ctx / bs)
// blocks) has the score
//     s_j = max over the query heads g of the group of
//           sum_d max(q_gd, 0) hi_jd + min(q_gd, 0) lo_jd
// (lo, hi: key_bounds.cuh), an upper bound of q_g . K over the block's keys.
// The first and the last blocks of the row are always taken (attention sinks
// and the local context), the rest by largest score, ties to the lowest
// index; a NaN score ranks above every number.
//
// A block is in or out by its place in the order, so scores are computed in
// 64 bits: a product of two bf16 values has 16 significand bits, and the sum
// of 2 D of them is exact in 53 bits unless their exponents span more than
// 29 bits; rounding can then only reorder blocks whose scores agree to about
// 2^-45.
//
// One cluster of CTAs per (row, K/V head): each CTA scores a segment of the
// row's blocks (a warp per block, lanes over the dimensions) and keeps the
// keys in shared memory; the cluster then selects (row_select.cuh). One
// launch, no workspace. Bound by the bounds' bytes: n * 2 * D elements per
// (row, K/V head).
#pragma once

#include "row_select.cuh"

namespace pa {

struct SelectArgs {
    int32_t *selected;  // [B][H_kv][K], ascending, -1 past the last
    const void *q;
    const void *key_bounds;
    const int32_t *block_tables;
    const int32_t *context_lens;
    int H_q, H_kv, group, bs, bs_shift, NB, MB, max_ctx;
    int K, first, last;
};

template <int VEC, typename T>
__device__ __forceinline__ void load_vec(const T *p, T (&x)[VEC]) {
    constexpr int BYTES = VEC * (int)sizeof(T);
    static_assert(BYTES == 4 || BYTES == 8 || BYTES == 16, "vector load");
    if constexpr (BYTES == 16)
        *reinterpret_cast<uint4 *>(x) = __ldg(reinterpret_cast<const uint4 *>(p));
    else if constexpr (BYTES == 8)
        *reinterpret_cast<uint2 *>(x) = __ldg(reinterpret_cast<const uint2 *>(p));
    else
        *reinterpret_cast<uint32_t *>(x) = __ldg(reinterpret_cast<const uint32_t *>(p));
}

// Key of a block's score, computed by a whole warp in 64 bits.
template <int D, typename T>
__device__ __forceinline__ uint64_t score_key(const SelectArgs &a, const T *q, int id, int h,
                                              int lane) {
    constexpr int VEC = D / 32;
    const T *lo_p = reinterpret_cast<const T *>(a.key_bounds) +
                    ((size_t)id * a.H_kv + h) * 2 * D + lane * VEC;
    alignas(16) T lo[VEC], hi[VEC], qv[VEC];
    load_vec<VEC>(lo_p, lo);
    load_vec<VEC>(lo_p + D, hi);
    uint64_t best = 0;
    for (int g = 0; g < a.group; ++g) {
        load_vec<VEC>(q + (size_t)g * D + lane * VEC, qv);
        double s = 0.0;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float x = (float)qv[v];
            s = fma((double)fmaxf(x, 0.f), (double)(float)hi[v], s);
            s = fma((double)fminf(x, 0.f), (double)(float)lo[v], s);
            if (x != x) s += (double)x;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        best = max(best, order_key(s));
    }
    return best;
}

template <int D, typename T>
__global__ void __launch_bounds__(kSelThreads)
    select_blocks_kernel(const __grid_constant__ SelectArgs a) {
    extern __shared__ uint64_t keys[];
    __shared__ RowSelectSmem sm;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int h = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t *dst = a.selected + ((size_t)b * a.H_kv + h) * a.K;

    int ctx = __ldg(a.context_lens + b);
    if (ctx < 0 || ctx > a.max_ctx) {
        if (rank == 0 && h == 0 && threadIdx.x == 0) flag_error(PA_ERR_BAD_TABLE);
        ctx = ctx < 0 ? 0 : a.max_ctx;
    }
    const int n = (int)(((long long)ctx + a.bs - 1) >> a.bs_shift);
    if (n <= a.K) {  // every block is taken (the whole cluster returns here)
        if (rank == 0)
            for (int i = threadIdx.x; i < a.K; i += kSelThreads) dst[i] = i < n ? i : -1;
        return;
    }
    if (rank == 0) {
        for (int i = threadIdx.x; i < a.first; i += kSelThreads) dst[i] = i;
        for (int i = threadIdx.x; i < a.last; i += kSelThreads)
            dst[a.K - a.last + i] = n - a.last + i;
    }
    const int need = a.K - a.first - a.last;
    if (need == 0) return;
    const int middle = n - a.first - a.last;  // more than need
    const int seg = (middle + ranks - 1) / ranks;
    const int s0 = min(rank * seg, middle);
    const int count = min(seg, middle - s0);

    const T *q = reinterpret_cast<const T *>(a.q) + ((size_t)b * a.H_q + (size_t)h * a.group) * D;
    const int32_t *row = a.block_tables + (size_t)b * a.MB + a.first + s0;
    for (int i = warp; i < count; i += kSelWarps) {
        const int id = __ldg(row + i);
        uint64_t k = 0;  // a block outside the pool ranks below every score
        if (id >= 0 && id < a.NB)
            k = score_key<D, T>(a, q, id, h, lane);
        else if (lane == 0)
            flag_error(PA_ERR_BAD_TABLE);
        if (lane == 0) keys[i] = k;
    }
    __syncthreads();
    auto key_at = [&](int i) { return keys[i]; };
    const Cut<uint64_t> cut = cluster_cut<uint64_t>(cluster, sm, key_at, count, (uint32_t)need);
    cluster_emit<uint64_t>(cluster, sm, key_at, count, cut, [&](int place, int i) {
        dst[a.first + place] = a.first + s0 + i;
    });
    cluster.sync();  // no CTA exits while another may read its shared memory
}

}  // namespace pa
