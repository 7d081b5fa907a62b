// key_bounds.cuh -- elementwise minimum and maximum of the keys of a block.
//
// For physical block p, K/V head h and dimension d, over the block's valid
// tokens j:
//     lo[p][h][d] = min_j K_j[d],   hi[p][h][d] = max_j K_j[d].
// A query's largest possible product with any key of the block is then
//     sum_d max(q_d, 0) hi_d + min(q_d, 0) lo_d,
// the score select_blocks.cuh ranks blocks by (page "字节跳动 AI Infra (2)",
// algorithm-level table, sparse attention row: attend only where it matters).
// Minimum and maximum of stored values are stored values: nothing is rounded,
// and the result does not depend on the order of the tokens. A NaN key makes
// its dimension's bounds NaN.
//
// A step's appends touch the blocks from the one holding the first new token
// to the last one; those are summarised afresh from the cache, so that no
// state is carried from step to step and a repeated call changes nothing.
//
// One warp per (row, touched block, K/V head): a page of block_size rows of
// D elements is contiguous, so every load instruction of the warp reads 512
// consecutive bytes, eight of them in flight per lane. Memory-bound: the
// touched blocks' valid keys once, two rows of D per page written.
#pragma once

#include "pa_device.cuh"

namespace pa {

constexpr int kBoundsWarps = 8;

struct BoundsArgs {
    void *key_bounds;  // [NB][H_kv][2][D]: minima, then maxima
    const void *k_cache;
    const int32_t *block_tables;
    const int32_t *context_lens;
    const int32_t *new_lens;
    int H_kv, bs, bs_shift, NB, MB, max_new;
};

// Elementwise minimum / maximum of 16 bytes; a NaN operand gives NaN.
template <bool MAX>
__device__ __forceinline__ uint32_t extreme(uint32_t x, uint32_t y, __nv_bfloat16) {
    const __nv_bfloat162 a = *reinterpret_cast<const __nv_bfloat162 *>(&x);
    const __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162 *>(&y);
    const __nv_bfloat162 r = MAX ? __hmax2_nan(a, b) : __hmin2_nan(a, b);
    return *reinterpret_cast<const uint32_t *>(&r);
}
template <bool MAX>
__device__ __forceinline__ uint32_t extreme(uint32_t x, uint32_t y, float) {
    float r;
    if constexpr (MAX)
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(x)), "f"(__uint_as_float(y)));
    else
        asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(x)), "f"(__uint_as_float(y)));
    return __float_as_uint(r);
}

template <int D, typename T>
__global__ void __launch_bounds__(kBoundsWarps * 32)
    key_bounds_kernel(const __grid_constant__ BoundsArgs a) {
    constexpr int VPR = D * (int)sizeof(T) / 16;  // 16-byte vectors per row: 8, 16 or 32
    constexpr int RPI = 32 / VPR;                 // rows a warp reads per instruction
    const int b = blockIdx.y;
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * kBoundsWarps + (threadIdx.x >> 5);
    const int i = (int)(w / a.H_kv), h = (int)(w - (long long)i * a.H_kv);

    // lengths outside their range are clamped and recorded
    const long long cap = (long long)a.MB * a.bs;
    int ctx = __ldg(a.context_lens + b), fresh = __ldg(a.new_lens + b);
    const bool bad = ctx < 0 || ctx > cap || fresh < 0 || fresh > a.max_new || fresh > ctx;
    if (bad && w == 0 && lane == 0) flag_error(PA_ERR_BAD_TABLE);
    ctx = ctx < 0 ? 0 : (int)min((long long)ctx, cap);
    fresh = max(0, min(fresh, min(ctx, a.max_new)));
    if (fresh == 0) return;
    const int lb = ((ctx - fresh) >> a.bs_shift) + i;
    if (lb >= (ctx + a.bs - 1) >> a.bs_shift) return;
    const int id = __ldg(a.block_tables + (size_t)b * a.MB + lb);
    if (id < 0 || id >= a.NB) {
        if (lane == 0) flag_error(PA_ERR_BAD_TABLE);
        return;
    }
    const int n = min(a.bs, ctx - (lb << a.bs_shift));  // valid tokens, at least one
    const int r0 = lane / VPR, u = lane % VPR;
    const uint4 *page = reinterpret_cast<const uint4 *>(a.k_cache) +
                        ((size_t)id * a.H_kv + h) * a.bs * VPR + u;

    // lanes whose first row is past the end repeat row 0
    uint4 lo = __ldg(page + (size_t)(r0 < n ? r0 : 0) * VPR), hi = lo;
#pragma unroll 8
    for (int r = r0 + RPI; r < n; r += RPI) {
        const uint4 x = __ldg(page + (size_t)r * VPR);
        lo.x = extreme<false>(lo.x, x.x, T()), hi.x = extreme<true>(hi.x, x.x, T());
        lo.y = extreme<false>(lo.y, x.y, T()), hi.y = extreme<true>(hi.y, x.y, T());
        lo.z = extreme<false>(lo.z, x.z, T()), hi.z = extreme<true>(hi.z, x.z, T());
        lo.w = extreme<false>(lo.w, x.w, T()), hi.w = extreme<true>(hi.w, x.w, T());
    }
#pragma unroll
    for (int o = VPR; o < 32; o <<= 1) {
        lo.x = extreme<false>(lo.x, __shfl_xor_sync(0xffffffffu, lo.x, o), T());
        lo.y = extreme<false>(lo.y, __shfl_xor_sync(0xffffffffu, lo.y, o), T());
        lo.z = extreme<false>(lo.z, __shfl_xor_sync(0xffffffffu, lo.z, o), T());
        lo.w = extreme<false>(lo.w, __shfl_xor_sync(0xffffffffu, lo.w, o), T());
        hi.x = extreme<true>(hi.x, __shfl_xor_sync(0xffffffffu, hi.x, o), T());
        hi.y = extreme<true>(hi.y, __shfl_xor_sync(0xffffffffu, hi.y, o), T());
        hi.z = extreme<true>(hi.z, __shfl_xor_sync(0xffffffffu, hi.z, o), T());
        hi.w = extreme<true>(hi.w, __shfl_xor_sync(0xffffffffu, hi.w, o), T());
    }
    uint4 *dst = reinterpret_cast<uint4 *>(a.key_bounds) + ((size_t)id * a.H_kv + h) * 2 * VPR;
    if (lane < VPR) dst[u] = lo;
    if (r0 == RPI - 1) dst[VPR + u] = hi;
}

}  // namespace pa
