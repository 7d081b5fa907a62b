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
// over 98K blocks of 8 heads, where the bounds' bytes would allow 6.5 TB/s), so
// every block is scored in 32 bits with an error bound, and only the blocks
// near the border between in and out are scored again in 64.
//
// score_blocks: a warp per 16 blocks of a (row, K/V head).
//   - bf16: the score is a product of the block's 2 D bounds with the vector
//     [min(q, 0), max(q, 0)], for all heads of the group: a warp-level
//     tensor-core product of 16 blocks x 8 heads x 2 D. Bounds and queries go
//     from global memory straight into fragments, 16 bytes a load (8 KB in
//     flight per warp, no shared memory, no barrier): a dot product does not
//     depend on the order of its terms, so the k slots take the dimensions in
//     the order those loads bring them. A second product of the absolute
//     values gives A = sum |terms|.
//     Error: a k = 16 step adds 16 exact products to the accumulator, each of
//     the 17 cut at no less than 2^-23 of the largest, and rounds: at most
//     18 * 2^-23 A_i for accumulator i's share of A. Four accumulators take
//     D / 32 steps each (4 at D = 128): 72 * 2^-23 A, plus three additions:
//     below 2^-16 A. Products that underflow add less than 2^-100. (How a step
//     cuts its terms is not published. Over cancelling, widely spread, subnormal
//     and barely kept terms the largest error was 0.02 of the bound, in fp32
//     0.12 of its own; the tests hold both to 1.)
//   - fp32: lanes over the dimensions, fused multiply-adds and a shuffle sum:
//     2 D / 32 + 5 roundings of at most 2^-24 A, below 2^-19 A.
//   A score and its error bound go to the workspace, 8 bytes per block beside
//   the 4 D read.
//
// select_blocks: a CTA per (row, K/V head), a programmatic dependent.
//   - The border is first found to one of 1024 equal bins over the row's range
//     of 32-bit scores. With e the row's largest error bound, a block whose
//     score less 2e is in a bin above the border's is in (what scores better in
//     64 bits lies above that bin too, and that is fewer blocks than there are
//     places), and one whose score plus 2e is in a bin below it is out. The few
//     blocks between are ranked by comparing all pairs, those of them whose
//     32-bit scores are within 2e of each other at the border by scores in 64
//     bits.
//   - Where that does not narrow them down (a score far out, equal blocks, an
//     infinite or NaN score in the row, one within 2e of the largest number),
//     the border is found exactly (row_select.cuh), and all blocks within 2e of
//     it are scored and selected in 64 bits.
//
// Scoring and selecting in one kernel (a cluster of CTAs per row, scores in
// shared memory, no workspace) was built first and measured slower: 123 us on
// 16 rows of 64K to 128K tokens, its CTAs' shares of a row being uneven and the
// selection's barriers leaving the memory idle.
// Bound by the bounds' bytes: n * 2 * D elements per (row, K/V head).
#pragma once

#include "decode.cuh"
#include "row_select.cuh"

namespace pa {

constexpr int kScoreWarps = 4;
constexpr int kScoreRows = 16;     // blocks per warp and step, bf16
constexpr int kScoreRowsF32 = 4;   // fp32
constexpr int kBins = kCutBins;
constexpr int kFewBlocks = 256;    // blocks near the border ranked by pairs

struct SelectArgs {
    int32_t *selected;  // [B][H_kv][K], ascending, -1 past the last
    const void *q;
    const void *key_bounds;
    const int32_t *block_tables;
    const int32_t *context_lens;
    uint64_t *scores;   // [B][H_kv][max_blocks]: order key of the score << 32 | error bound
    int H_q, H_kv, group, bs, bs_shift, NB, MB, max_ctx;
    int K, first, last, max_blocks;
    int tiles;          // tiles of a row (16 or 4 blocks) that are scored at once
    int stage;          // blocks whose scores fit the selecting CTA's shared memory
};

// The value of an order key (a NaN for a NaN's).
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k);
}

// Blocks of a row, and those between its first and last ones that compete for
// `need` places (none when every block is taken).
struct Contest {
    int n, middle, need;
};
__device__ __forceinline__ Contest contest(const SelectArgs &a, int b, bool report) {
    int ctx = __ldg(a.context_lens + b);
    if (ctx < 0 || ctx > a.max_ctx) {
        if (report) flag_error(PA_ERR_BAD_TABLE);
        ctx = ctx < 0 ? 0 : a.max_ctx;
    }
    Contest c;
    c.n = (int)(((long long)ctx + a.bs - 1) >> a.bs_shift);
    c.need = a.K - a.first - a.last;
    c.middle = c.n > a.K && c.need > 0 ? c.n - a.first - a.last : 0;
    return c;
}

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

// Order key of a block's score, computed by a whole warp in 64 bits.
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
#pragma unroll 4
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

__device__ __forceinline__ uint64_t score_entry(float score, float err) {
    return (uint64_t)order_key(score) << 32 | __float_as_uint(err);
}

template <bool MAX>
__device__ __forceinline__ uint32_t signed_part(uint32_t q) {
    const __nv_bfloat162 z = __floats2bfloat162_rn(0.f, 0.f);
    const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162 *>(&q);
    const __nv_bfloat162 r = MAX ? __hmax2_nan(x, z) : __hmin2_nan(x, z);  // a NaN stays one
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Warp w of a row's scoring warps takes 16-block tile w / H_kv of K/V head
// w % H_kv -- the heads' bounds of a block lie together -- and every
// `tiles`-th tile behind it. Grid: (the row's warps / kScoreWarps, row).
template <int D>
__global__ void __launch_bounds__(kScoreWarps * 32, 4)
    score_blocks_bf16(const __grid_constant__ SelectArgs a) {
    constexpr int CH = D / 32;  // 64-byte pieces of a row of D
    allow_dependent_launch();
    const int b = blockIdx.y, lane = threadIdx.x & 31;
    const int g = lane >> 2, tig = lane & 3;
    const int w = (int)blockIdx.x * kScoreWarps + (threadIdx.x >> 5);
    const int first_tile = w / a.H_kv, h = w - first_tile * a.H_kv;
    if (first_tile >= a.tiles) return;
    const int middle = contest(a, b, false).middle;
    const int32_t *table = a.block_tables + (size_t)b * a.MB + a.first;
    uint64_t *out = a.scores + ((size_t)b * a.H_kv + h) * a.max_blocks;
    const __nv_bfloat16 *q =
        reinterpret_cast<const __nv_bfloat16 *>(a.q) + ((size_t)b * a.H_q + (size_t)h * a.group) * D;

    const int stride = a.tiles * kScoreRows;
    int i0 = first_tile * kScoreRows;
    int ids[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int i = i0 + g + 8 * r;
        ids[r] = i < middle ? __ldg(table + i) : -1;
    }
    for (; i0 < middle; i0 += stride) {
        uint4 x[2][2 * CH];
        bool ok[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            ok[r] = ids[r] >= 0 && ids[r] < a.NB;
            if (i0 + g + 8 * r < middle && !ok[r] && tig == 0) flag_error(PA_ERR_BAD_TABLE);
            const uint4 *p = reinterpret_cast<const uint4 *>(a.key_bounds) +
                             ((size_t)(ok[r] ? ids[r] : 0) * a.H_kv + h) * (D / 4) + tig;
#pragma unroll
            for (int j = 0; j < 2 * CH; ++j)
                x[r][j] = ok[r] ? __ldg(p + 4 * j) : make_uint4(0, 0, 0, 0);
            // the next step's ids, while these loads are in flight
            const long long i = (long long)i0 + stride + g + 8 * r;
            ids[r] = i < middle ? __ldg(table + i) : -1;
        }
        float best[2] = {-INFINITY, -INFINITY}, size[2] = {0.f, 0.f};
#pragma unroll 1
        for (int g0 = 0; g0 < a.group; g0 += 8) {
            const uint4 *qp = reinterpret_cast<const uint4 *>(q + (size_t)(g0 + g) * D) + tig;
            const bool live = g0 + g < a.group;
            uint4 y[CH];
#pragma unroll
            for (int j = 0; j < CH; ++j) y[j] = live ? __ldg(qp + 4 * j) : make_uint4(0, 0, 0, 0);
            float s[4][4] = {}, m[4] = {};
            constexpr uint32_t kAbs = 0x7fff7fffu;
#pragma unroll
            for (int j = 0; j < 2 * CH; ++j) {
                const uint4 w = y[j % CH];
                const uint32_t w0 = j < CH ? signed_part<false>(w.x) : signed_part<true>(w.x);
                const uint32_t w1 = j < CH ? signed_part<false>(w.y) : signed_part<true>(w.y);
                const uint32_t w2 = j < CH ? signed_part<false>(w.z) : signed_part<true>(w.z);
                const uint32_t w3 = j < CH ? signed_part<false>(w.w) : signed_part<true>(w.w);
                const uint32_t a0[4] = {x[0][j].x, x[1][j].x, x[0][j].y, x[1][j].y};
                const uint32_t a1[4] = {x[0][j].z, x[1][j].z, x[0][j].w, x[1][j].w};
                mma_bf16_16816(s[(2 * j) % 4], a0, w0, w1);
                mma_bf16_16816(s[(2 * j + 1) % 4], a1, w2, w3);
                const uint32_t b0[4] = {a0[0] & kAbs, a0[1] & kAbs, a0[2] & kAbs, a0[3] & kAbs};
                const uint32_t b1[4] = {a1[0] & kAbs, a1[1] & kAbs, a1[2] & kAbs, a1[3] & kAbs};
                mma_bf16_16816(m, b0, w0 & kAbs, w1 & kAbs);
                mma_bf16_16816(m, b1, w2 & kAbs, w3 & kAbs);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (g0 + 2 * tig + (e & 1) >= a.group) continue;
                const float v = (s[0][e] + s[1][e]) + (s[2][e] + s[3][e]);
                best[e >> 1] = fmaxf(best[e >> 1], v);
                // no bound on a score that is not finite (m is NaN only if v is)
                size[e >> 1] = fmaxf(size[e >> 1], fabsf(v) < INFINITY ? m[e] : INFINITY);
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float e = fmaf(size[r], 0x1p-16f, 0x1p-100f);
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], o));
                e = fmaxf(e, __shfl_xor_sync(0xffffffffu, e, o));
            }
            const int i = i0 + g + 8 * r;
            // entry 0, below every score: a block outside the pool
            if (tig == 0 && i < middle) out[i] = ok[r] ? score_entry(best[r], e) : 0;
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kScoreWarps * 32)
    score_blocks_f32(const __grid_constant__ SelectArgs a) {
    constexpr int VEC = D / 32;
    allow_dependent_launch();
    const int b = blockIdx.y, lane = threadIdx.x & 31;
    const int w = (int)blockIdx.x * kScoreWarps + (threadIdx.x >> 5);
    const int first_tile = w / a.H_kv, h = w - first_tile * a.H_kv;
    if (first_tile >= a.tiles) return;
    const int middle = contest(a, b, false).middle;
    const int32_t *table = a.block_tables + (size_t)b * a.MB + a.first;
    uint64_t *out = a.scores + ((size_t)b * a.H_kv + h) * a.max_blocks;
    const float *q =
        reinterpret_cast<const float *>(a.q) + ((size_t)b * a.H_q + (size_t)h * a.group) * D;
    for (int i0 = first_tile * kScoreRowsF32; i0 < middle; i0 += a.tiles * kScoreRowsF32) {
        const int end = min(middle, i0 + kScoreRowsF32);
#pragma unroll 2
        for (int i = i0; i < end; ++i) {
            const int id = __ldg(table + i);
            if (id < 0 || id >= a.NB) {
                if (lane == 0) {
                    flag_error(PA_ERR_BAD_TABLE);
                    out[i] = 0;
                }
                continue;
            }
            const float *p = reinterpret_cast<const float *>(a.key_bounds) +
                             ((size_t)id * a.H_kv + h) * 2 * D + lane * VEC;
            alignas(16) float lo[VEC], hi[VEC], x[VEC];
            load_vec<VEC>(p, lo);
            load_vec<VEC>(p + D, hi);
            float best = -INFINITY, size = 0.f;
#pragma unroll 4
            for (int g = 0; g < a.group; ++g) {
                load_vec<VEC>(q + (size_t)g * D + lane * VEC, x);
                float s = 0.f, m = 0.f;
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const float up = x[v] < 0.f ? 0.f : x[v], down = x[v] > 0.f ? 0.f : x[v];
                    s = fmaf(up, hi[v], s);
                    s = fmaf(down, lo[v], s);
                    m = fmaf(fabsf(up), fabsf(hi[v]), m);
                    m = fmaf(fabsf(down), fabsf(lo[v]), m);
                }
                s = warp_sum(s);
                m = warp_sum(m);
                best = fmaxf(best, s);
                size = fmaxf(size, fabsf(s) < INFINITY ? m : INFINITY);
            }
            if (lane == 0)
                out[i] = score_entry(best, fmaf(size, 0x1p-19f, 0x1p-100f));
        }
    }
}

struct SelectSmem {
    RowSelectSmem row;
    uint32_t lo, hi, err;     // order keys of the least and largest score, bits of the largest
                              // error bound
    int border;               // the bin that holds the border, kBins if there is none
    uint32_t above, zone;     // blocks above the border zone, in it
    uint32_t sure, close;     // blocks of the zone that are in, that 32 bits do not decide
    int zone_at[kFewBlocks];
    int close_at[kFewBlocks];
    uint64_t close_key[kFewBlocks];
};

// 32-bit scores of a row as bins.
struct Bins {
    float lo, scale, err;
    __device__ __forceinline__ int at(float s) const {  // ascending with s
        return max(0, (int)fminf((s - lo) * scale, (float)(kBins - 1)));
    }
};

// Selects and emits where a bin of 32-bit scores narrows the border down;
// false (for every thread) where it does not, with the keys' high halves as
// they were.
template <int THREADS, int D, typename T, typename Emit>
__device__ __forceinline__ bool select_by_bins(const SelectArgs &a, SelectSmem &sm, const T *q,
                                               const int32_t *table, int h, int count,
                                               uint32_t need, uint64_t *keys, const Emit &emit) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Bins bins;
    bins.err = __uint_as_float(sm.err);
    if (sm.lo > sm.hi || !(bins.err < INFINITY)) return false;
    bins.lo = key_value(sm.lo);
    const float top = key_value(sm.hi), width = top - bins.lo;
    bins.scale = width > 0.f ? (float)kBins / width : 0.f;
    if (!(width < INFINITY) || !(bins.scale < INFINITY)) return false;
    // a score less or plus 2e must not leave the range: equal scores have a scale
    // of 0, and 0 times an infinity no bin
    if (!(__fsub_rd(bins.lo, 2.f * bins.err) > -INFINITY) ||
        !(__fadd_ru(top, 2.f * bins.err) < INFINITY))
        return false;

    for (int i = tid; i < count; i += THREADS) {
        const uint32_t k = (uint32_t)(keys[i] >> 32);
        if (k != 0) atomicAdd(&sm.row.bins[0][bins.at(key_value(k))], 1u);
    }
    __syncthreads();
    {  // thread t owns the bins from kBins - 1 - t * PER down
        constexpr int PER = kBins / THREADS;
        uint32_t c[PER], mine = 0, all;
#pragma unroll
        for (int j = 0; j < PER; ++j) mine += c[j] = sm.row.bins[0][kBins - 1 - tid * PER - j];
        uint32_t above = block_before<THREADS>(sm.row, mine, all);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            if (above < need && need <= above + c[j]) sm.border = kBins - 1 - tid * PER - j;
            above += c[j];
        }
    }
    __syncthreads();
    const int border = sm.border;
    if (border == kBins) return false;  // fewer blocks inside the pool than places

    // the low half of a key: 2 in, 1 in the zone, 0 out
    uint32_t above = 0;
    for (int i = tid; i < count; i += THREADS) {
        const uint32_t k = (uint32_t)(keys[i] >> 32);
        uint32_t mark = 0;
        if (k != 0) {
            const float s = key_value(k);
            if (bins.at(__fsub_rd(s, 2.f * bins.err)) > border) {
                mark = 2;
                ++above;
            } else if (bins.at(__fadd_ru(s, 2.f * bins.err)) >= border) {
                mark = 1;
                const uint32_t at = atomicAdd(&sm.zone, 1u);
                if (at < kFewBlocks) sm.zone_at[at] = i;
            }
        }
        keys[i] = (uint64_t)k << 32 | mark;
    }
    above = __reduce_add_sync(0xffffffffu, above);
    if (lane == 0) atomicAdd(&sm.above, above);
    __syncthreads();
    // fewer than `need` blocks lie above the border's bin; had more been marked,
    // they would not fit the list (a test of each place as it is written instead:
    // 27.5 against 26.7 us for 128 ragged rows of up to 256 blocks and 8 heads)
    if (sm.above >= need) return false;
    const uint32_t zone = sm.zone, places = need - sm.above;
    uint32_t least = 1;  // the mark of a block that is in
    if (zone != places) {
        if (zone > kFewBlocks) return false;
        least = 2;
        const uint32_t *high = reinterpret_cast<const uint32_t *>(keys) + 1;
        for (int j = tid; j < (int)zone; j += THREADS) {
            const int at = sm.zone_at[j];
            const float s = key_value(high[2 * at]);
            const float up = __fadd_ru(s, 2.f * bins.err), down = __fsub_rd(s, 2.f * bins.err);
            uint32_t better = 0, not_worse = 0;
            for (int o = 0; o < (int)zone; ++o) {
                const float other = key_value(high[2 * sm.zone_at[o]]);
                better += other > up;
                not_worse += other >= down;
            }
            if (not_worse <= places) {
                *reinterpret_cast<uint32_t *>(keys + at) = 2;  // the low half
                atomicAdd(&sm.sure, 1u);
            } else if (better < places) {
                sm.close_at[atomicAdd(&sm.close, 1u)] = at;
            }
        }
        __syncthreads();
        const uint32_t close = sm.close, left = places - sm.sure;
        if (close != left) {
            for (int j = warp; j < (int)close; j += THREADS / 32) {
                const uint64_t s = score_key<D, T>(a, q, __ldg(table + sm.close_at[j]), h, lane);
                if (lane == 0) sm.close_key[j] = s;
            }
            __syncthreads();
        }
        // one of these is in when fewer than the places left rank before it: a
        // larger score, or an equal one at a lower index
        for (int j = tid; j < (int)close; j += THREADS) {
            const int at = sm.close_at[j];
            uint32_t before = 0;
            if (close != left) {
                const uint64_t s = sm.close_key[j];
                for (int o = 0; o < (int)close; ++o) {
                    const uint64_t other = sm.close_key[o];
                    before += other > s || (other == s && sm.close_at[o] < at);
                }
            }
            if (before < left) keys[at] = 2;
        }
        __syncthreads();
    }
    block_emit<THREADS>(
        sm.row, count, [&](int i) { return (uint32_t)keys[i] >= least; }, emit);
    return true;
}

// The cut of the row, by 32-bit scores where they decide and 64-bit ones where
// they do not. keys: order keys of the 32-bit scores in the high halves; on
// return such that the cut applies to them.
template <int THREADS, int D, typename T>
__device__ __noinline__ Cut<uint64_t> exact_cut(const SelectArgs &a, SelectSmem &sm, const T *q,
                                                const int32_t *table, int h, int count,
                                                uint32_t need, uint64_t *keys) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const OneCta cluster;
    const Cut<uint32_t> coarse = cluster_cut<THREADS, uint32_t>(
        cluster, sm.row, [&](int i) { return (uint32_t)(keys[i] >> 32); }, count, need);
    const float e = __uint_as_float(sm.err);
    // order keys of the border zone's ends; the whole row without a bound, or
    // without enough blocks inside the pool
    uint32_t lo = 1, hi = 0xffffffffu;
    if (e < INFINITY && coarse.key != 0) {
        const float t = key_value(coarse.key);
        lo = order_key(__fsub_rd(t, 2.f * e));
        hi = order_key(__fadd_ru(t, 2.f * e));
    }
    constexpr uint64_t kIn = ~(uint64_t)0;  // above every score, a NaN's included
    for (int i = warp; i < count; i += THREADS / 32) {
        const uint32_t k = (uint32_t)(keys[i] >> 32);
        uint64_t s = k > hi ? kIn : k == 0 ? 1 : 0;
        // what is sure to be out ranks below what is outside the pool; no place
        // is left for either
        if (k >= lo && k <= hi)
            s = max((uint64_t)2, min(score_key<D, T>(a, q, __ldg(table + i), h, lane), kIn - 1));
        __syncwarp();
        if (lane == 0) keys[i] = s;
    }
    cluster.sync();
    return cluster_cut<THREADS, uint64_t>(
        cluster, sm.row, [&](int i) { return keys[i]; }, count, need);
}

// Grid: (K/V head, row). A programmatic dependent of the scoring kernel, which
// began after everything before it had ended: only the scores are waited for.
template <int THREADS, int D, typename T>
__global__ void __launch_bounds__(THREADS)
    select_blocks_kernel(const __grid_constant__ SelectArgs a) {
    extern __shared__ __align__(16) uint64_t staged[];
    __shared__ SelectSmem sm;
    const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
    int32_t *dst = a.selected + ((size_t)b * a.H_kv + h) * a.K;
    const Contest c = contest(a, b, h == 0 && tid == 0);
    if (c.n <= a.K) {  // every block is taken
        for (int i = tid; i < a.K; i += THREADS) dst[i] = i < c.n ? i : -1;
    } else {
        for (int i = tid; i < a.first; i += THREADS) dst[i] = i;
        for (int i = tid; i < a.last; i += THREADS) dst[a.K - a.last + i] = c.n - a.last + i;
    }
    for (int i = tid; i < kBins; i += THREADS) sm.row.bins[0][i] = 0;
    if (tid == 0) {
        sm.lo = 0xffffffffu;
        sm.hi = sm.err = sm.above = sm.zone = sm.sure = sm.close = 0;
        sm.border = kBins;
    }
    wait_for_primary_grid();
    if (c.middle == 0) return;
    __syncthreads();

    // the row's scores into shared memory where they fit
    const int count = c.middle;
    uint64_t *row = a.scores + ((size_t)b * a.H_kv + h) * a.max_blocks;
    uint64_t *keys = count <= a.stage ? staged : row;
    uint32_t lo = 0xffffffffu, hi = 0, err = 0;
#pragma unroll 4
    for (int i = tid; i < count; i += THREADS) {
        const uint64_t x = __ldcg(row + i);
        const uint32_t k = (uint32_t)(x >> 32);
        if (k != 0) {
            lo = min(lo, k);
            hi = max(hi, k);
            err = max(err, (uint32_t)x);  // bits of values >= 0 order as the values
        }
        if (keys == staged) staged[i] = x;
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    err = __reduce_max_sync(0xffffffffu, err);
    if (lane == 0) {
        atomicMin(&sm.lo, lo);
        atomicMax(&sm.hi, hi);
        atomicMax(&sm.err, err);
    }
    __syncthreads();
    const T *q = reinterpret_cast<const T *>(a.q) + ((size_t)b * a.H_q + (size_t)h * a.group) * D;
    const int32_t *table = a.block_tables + (size_t)b * a.MB + a.first;
    auto emit = [&](int place, int i) { dst[a.first + place] = a.first + i; };
    if (!select_by_bins<THREADS, D, T>(a, sm, q, table, h, count, (uint32_t)c.need, keys, emit)) {
        const Cut<uint64_t> cut =
            exact_cut<THREADS, D, T>(a, sm, q, table, h, count, (uint32_t)c.need, keys);
        const OneCta cluster;
        cluster_emit<THREADS, uint64_t>(
            cluster, sm.row, [&](int i) { return keys[i]; }, count, cut, emit);
    }
}

}  // namespace pa
