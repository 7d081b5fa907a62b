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
// A block is in or out by its place in the order, so the order is that of
// scores in 64 bits: a product of two bf16 values has 16 significand bits, and
// the sum of 2 D of them is exact in 53 bits unless their exponents span more
// than 29 bits; rounding can then only reorder blocks whose scores agree to
// about 2^-45. Computing every score so is bound by the 64-bit sums (0.56 TB/s
// over 98K blocks of 8 heads; the bounds' bytes would allow 6.5 TB/s), so bf16
// rows are scored in 32 bits first and only the blocks near the border again:
//   - the score is a product of the block's 2 D bounds with the vector
//     [min(q, 0), max(q, 0)], for all heads of the group: a warp-level
//     tensor-core product of 16 blocks x 8 heads x 2 D. The bounds go from
//     global memory straight into the A fragments, 16 bytes a load; a dot
//     product does not depend on the order of its terms, so the fragments'
//     k slots take the dimensions in the order those loads bring them. A
//     second product of the absolute values gives A = sum |terms|;
//   - its error: a k = 16 step adds 16 exact products to the accumulator, each
//     of the 17 cut at no less than 2^-23 of the largest, and rounds: at most
//     18 * 2^-23 A_i for accumulator i's share of A. Four accumulators take
//     D / 32 steps each (4 at D = 128): 72 * 2^-23 A, plus three additions:
//     below 2^-16 A. Products that underflow add less than 2^-100;
//   - with e the largest error bound of the row and t the border of the 32-bit
//     scores (at least `need` are >= t, fewer are above it, or exactly `need`
//     are >= t), a block above t + 2e is in and one below t - 2e is out. If
//     the blocks between are more than the places left, their scores are
//     computed in 64 bits: a few blocks are then ranked by comparing all pairs,
//     many (equal blocks, an infinite or NaN score in the row) by a second
//     selection.
//
// One cluster of CTAs per (row, K/V head): each CTA scores a segment of the
// row's blocks and keeps the keys in shared memory; the cluster then selects
// (row_select.cuh). One launch, no workspace. Bound by the bounds' bytes:
// n * 2 * D elements per (row, K/V head).
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

constexpr int kTensorHeads = 64;   // largest group scored on the tensor cores
constexpr int kFewBlocks = 256;    // blocks near the border ranked by pairs

struct SelectSmem {
    RowSelectSmem row;
    uint32_t err;                  // bits of this CTA's largest error bound
    uint32_t count[2];             // blocks above the border zone, in it
    uint32_t listed;               // rank 0: blocks in `zone_key`
    uint64_t zone_key[kFewBlocks];
    int zone_at[kFewBlocks];
};

// Bytes of a head's [min(q, 0), max(q, 0)] row: rows 16 banks apart, so that
// the 8 lanes of a 16-byte load phase (two rows, 64 bytes each) do not meet.
template <int D>
constexpr int kQRow = 2 * D * 2 + 64;

// The group's rows, zero past its last head up to a multiple of 8.
template <int D>
__device__ __forceinline__ void load_signed_queries(const __nv_bfloat16 *q, int group,
                                                    uint8_t *dst) {
    const int rows = (group + 7) / 8 * 8;
    for (int i = threadIdx.x; i < rows * D; i += kSelThreads) {
        const int g = i / D, d = i % D;
        const float x = g < group ? __bfloat162float(q[(size_t)g * D + d]) : 0.f;
        __nv_bfloat16 *r = reinterpret_cast<__nv_bfloat16 *>(dst + g * kQRow<D>);
        // a NaN goes into both, as it does into the sum
        r[d] = __float2bfloat16(x > 0.f ? 0.f : x);
        r[D + d] = __float2bfloat16(x < 0.f ? 0.f : x);
    }
}

// Scores of blocks [0, count) of this CTA into the high halves of keys; returns
// this thread's largest error bound, +inf where a score is not finite.
template <int D>
__device__ __forceinline__ float score_segment(const SelectArgs &a, const uint8_t *qs,
                                               const int32_t *table, int h, int count,
                                               uint64_t *keys) {
    constexpr int CH = D / 16;  // 64-byte pieces of a block's 2 D bounds
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, tig = lane & 3;
    const int tiles = (a.group + 7) / 8;
    float err = 0.f;
    for (int i0 = warp * 16; i0 < count; i0 += kSelWarps * 16) {
        uint4 x[2][CH];
        bool ok[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int i = i0 + g + 8 * r;
            const int id = i < count ? __ldg(table + i) : -1;
            ok[r] = id >= 0 && id < a.NB;
            if (i < count && !ok[r] && tig == 0) flag_error(PA_ERR_BAD_TABLE);
            const uint4 *p = reinterpret_cast<const uint4 *>(a.key_bounds) +
                             ((size_t)(ok[r] ? id : 0) * a.H_kv + h) * (D / 4) + tig;
#pragma unroll
            for (int j = 0; j < CH; ++j) x[r][j] = ok[r] ? __ldg(p + 4 * j) : make_uint4(0, 0, 0, 0);
        }
        float best[2] = {-INFINITY, -INFINITY}, size[2] = {0.f, 0.f};
        bool odd[2] = {false, false};  // some head's score is not finite
        for (int n = 0; n < tiles; ++n) {
            const uint32_t qr = smem_u32(qs) + (n * 8 + g) * kQRow<D> + tig * 16;
            float s[4][4] = {}, m[4] = {};
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                uint4 y;  // read again for every tile: registers hold the bounds
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w)
                             : "r"(qr + 64 * j));
                const uint32_t a0[4] = {x[0][j].x, x[1][j].x, x[0][j].y, x[1][j].y};
                const uint32_t a1[4] = {x[0][j].z, x[1][j].z, x[0][j].w, x[1][j].w};
                mma_bf16_16816(s[(2 * j) % 4], a0, y.x, y.y);
                mma_bf16_16816(s[(2 * j + 1) % 4], a1, y.z, y.w);
                constexpr uint32_t kAbs = 0x7fff7fffu;
                const uint32_t b0[4] = {a0[0] & kAbs, a0[1] & kAbs, a0[2] & kAbs, a0[3] & kAbs};
                const uint32_t b1[4] = {a1[0] & kAbs, a1[1] & kAbs, a1[2] & kAbs, a1[3] & kAbs};
                mma_bf16_16816(m, b0, y.x & kAbs, y.y & kAbs);
                mma_bf16_16816(m, b1, y.z & kAbs, y.w & kAbs);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (n * 8 + 2 * tig + (e & 1) >= a.group) continue;
                const float v = (s[0][e] + s[1][e]) + (s[2][e] + s[3][e]);
                best[e >> 1] = fmaxf(best[e >> 1], v);
                size[e >> 1] = fmaxf(size[e >> 1], m[e]);
                odd[e >> 1] |= !(fabsf(v) < INFINITY) || !(m[e] < INFINITY);
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float z = odd[r] ? INFINITY : fmaf(size[r], 0x1p-16f, 0x1p-100f);
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], o));
                z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, o));
            }
            const int i = i0 + g + 8 * r;
            if (ok[r]) err = fmaxf(err, z);
            // the lowest key is that of a block outside the pool
            if (tig == 0 && i < count) keys[i] = ok[r] ? (uint64_t)order_key(best[r]) << 32 : 1ull;
        }
    }
    return err;
}

__device__ __forceinline__ float key_value(uint32_t k) {  // the float of an order_key
    return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k);
}

// The cut of the cluster's row, by 32-bit scores where they decide and 64-bit
// ones where they do not. keys: order keys of the 32-bit scores in the high
// halves; on return such that the cut applies to them.
template <int D, typename T>
__device__ __forceinline__ Cut<uint64_t> refined_cut(const SelectArgs &a,
                                                     cg::cluster_group &cluster, SelectSmem &sm,
                                                     const T *q, const int32_t *table, int h,
                                                     int s0, int count, uint32_t need,
                                                     uint64_t *keys) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ranks = (int)cluster.num_blocks();
    const Cut<uint32_t> coarse = cluster_cut<uint32_t>(
        cluster, sm.row, [&](int i) { return (uint32_t)(keys[i] >> 32); }, count, need);
    // not enough blocks inside the pool: all of them, then the lowest others
    if (coarse.key == 0) return {1ull, coarse.ties};
    float e = 0.f;
    for (int r = 0; r < ranks; ++r)
        e = fmaxf(e, __uint_as_float(*cluster.map_shared_rank(&sm.err, r)));
    // order keys of the border zone's ends; the whole row without a bound
    uint32_t lo = 1, hi = 0xffffffffu;
    if (e < INFINITY) {
        const float t = key_value(coarse.key);
        lo = order_key(__fsub_rd(t, 2.f * e));
        hi = order_key(__fadd_ru(t, 2.f * e));
    }
    uint32_t above = 0, zone = 0;
    for (int i = tid; i < count; i += kSelThreads) {
        const uint32_t k = (uint32_t)(keys[i] >> 32);
        above += k > hi;
        zone += k >= lo && k <= hi;
    }
    above = __reduce_add_sync(0xffffffffu, above);
    zone = __reduce_add_sync(0xffffffffu, zone);
    if (lane == 0) {
        atomicAdd(&sm.count[0], above);
        atomicAdd(&sm.count[1], zone);
    }
    cluster.sync();
    above = zone = 0;
    for (int r = 0; r < ranks; ++r) {
        const uint32_t *c = cluster.map_shared_rank(sm.count, r);
        above += c[0];
        zone += c[1];
    }
    if (above + zone == need) return {((uint64_t)lo << 32) - 1, 0};

    constexpr uint64_t kIn = ~(uint64_t)0;  // above every score, a NaN's included
    if (zone <= kFewBlocks) {
        SelectSmem *lead = cluster.map_shared_rank(&sm, 0);
        for (int i = warp; i < count; i += kSelWarps) {
            const uint32_t k = (uint32_t)(keys[i] >> 32);
            if (k < lo || k > hi) continue;
            const uint64_t s = score_key<D, T>(a, q, __ldg(table + i), h, lane);
            if (lane == 0) {
                const uint32_t at = atomicAdd(&lead->listed, 1u);
                lead->zone_key[at] = s;
                lead->zone_at[at] = s0 + i;
            }
        }
        cluster.sync();
        // a block of the zone is in when fewer than the places left rank
        // before it: a larger score, or an equal one at a lower index
        for (int j = warp; j < (int)zone; j += kSelWarps) {
            const int at = lead->zone_at[j] - s0;
            if (at < 0 || at >= count) continue;  // another CTA's
            const uint64_t s = lead->zone_key[j];
            uint32_t before = 0;
            for (int o = lane; o < (int)zone; o += 32) {
                const uint64_t other = lead->zone_key[o];
                before += other > s || (other == s && lead->zone_at[o] - s0 < at);
            }
            before = __reduce_add_sync(0xffffffffu, before);
            if (lane == 0) keys[at] = before < need - above ? kIn : 0;
        }
        __syncthreads();
        // what is left in the zone's range of keys is out or set above
        return {hi == 0xffffffffu ? kIn - 1 : ((uint64_t)hi << 32) | 0xffffffffu, 0};
    }
    for (int i = warp; i < count; i += kSelWarps) {
        const uint32_t k = (uint32_t)(keys[i] >> 32);
        uint64_t s = k > hi ? kIn : 0;
        if (k >= lo && k <= hi)
            s = max((uint64_t)2, min(score_key<D, T>(a, q, __ldg(table + i), h, lane), kIn - 1));
        if (k == 0) s = 1;  // outside the pool
        __syncwarp();
        if (lane == 0) keys[i] = s;
    }
    __syncthreads();
    return cluster_cut<uint64_t>(
        cluster, sm.row, [&](int i) { return keys[i]; }, count, need);
}

// TENSOR: bf16 and a group of at most kTensorHeads; else every score is
// computed in 64 bits.
template <int D, typename T, bool TENSOR>
__global__ void __launch_bounds__(kSelThreads)
    select_blocks_kernel(const __grid_constant__ SelectArgs a) {
    extern __shared__ __align__(16) uint8_t select_smem[];
    __shared__ SelectSmem sm;
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
    const int32_t *table = a.block_tables + (size_t)b * a.MB + a.first + s0;
    Cut<uint64_t> cut;
    uint64_t *keys;
    if constexpr (TENSOR) {
        const int heads = (a.group + 7) / 8 * 8;
        keys = reinterpret_cast<uint64_t *>(select_smem + heads * kQRow<D>);
        load_signed_queries<D>(q, a.group, select_smem);
        if (threadIdx.x == 0) sm.err = sm.listed = sm.count[0] = sm.count[1] = 0;
        __syncthreads();
        float err = score_segment<D>(a, select_smem, table, h, count, keys);
        const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(err));  // err >= 0
        if (lane == 0) atomicMax(&sm.err, bits);
        __syncthreads();
        cut = refined_cut<D, T>(a, cluster, sm, q, table, h, s0, count, (uint32_t)need, keys);
    } else {
        keys = reinterpret_cast<uint64_t *>(select_smem);
        for (int i = warp; i < count; i += kSelWarps) {
            const int id = __ldg(table + i);
            uint64_t k = 0;  // a block outside the pool ranks below every score
            if (id >= 0 && id < a.NB)
                k = score_key<D, T>(a, q, id, h, lane);
            else if (lane == 0)
                flag_error(PA_ERR_BAD_TABLE);
            if (lane == 0) keys[i] = k;
        }
        __syncthreads();
        cut = cluster_cut<uint64_t>(
            cluster, sm.row, [&](int i) { return keys[i]; }, count, (uint32_t)need);
    }
    cluster_emit<uint64_t>(
        cluster, sm.row, [&](int i) { return keys[i]; }, count, cut, [&](int place, int i) {
            dst[a.first + place] = a.first + s0 + i;
        });
    cluster.sync();  // no CTA exits while another may read its shared memory
}

}  // namespace pa
