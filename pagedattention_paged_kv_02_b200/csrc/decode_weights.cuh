// decode_weights.cuh -- attention weights of a decode step, added up per
// position: the second kernel of the decode that accumulates weights.
//
// The split kernel (decode.cuh, Span::kWeighted) left every query head's
// scaled base-2 scores s_j and, per partition, the maximum m and the sum u of
// 2^(s_j - m) in 32 bits. Over the partitions of a head
//     M = max m,   U = sum u 2^(m - M),
// and a position's weight is p_j = 2^(s_j - M) / U. For each K/V head h
//     weights_out[b][h][j] = weights_in[b][h][j] + sum over the group of p_j
// (page "字节跳动 AI Infra (2)", KV table, H2O row: the tokens to keep are the
// ones attended to most). M and U are kept apart rather than as a logarithm:
// s_j - M is then the difference of two scores, whose rounding does not grow
// with log U.
//
// Where a row is one partition and its K/V head one tile of query heads, the
// split CTA has all it needs and finishes the weights itself (weights_here):
// no second kernel, 12.3 -> 8.2 us for four short rows.
//
// Otherwise: one CTA per (tile of 1024 positions, K/V head, row), four positions
// per thread, after its warps have put the statistics of the head's group
// together; the merge of the outputs (decode_merge.cuh) is a launch behind it.
// (Both in one launch, which depends on the split kernel alone, measured slower:
// 207 against 195 us on the Llama-shaped batch.) Reads 4 bytes per query head
// and 4 per K/V head and position (the scores mostly from L2), writes 4. Heads
// are added in order: the result does not depend on timing.
#pragma once

#include "decode.cuh"

namespace pa {

constexpr int kWeightThreads = 256;
constexpr int kWeightTile = 4 * kWeightThreads;
constexpr int kWeightHeads = 64;  // heads whose statistics a CTA holds at a time

__global__ void __launch_bounds__(kWeightThreads)
    decode_weights_kernel(const __grid_constant__ DecodeArgs a) {
    __shared__ float top[kWeightHeads], inv[kWeightHeads];
    // every CTA waits: nothing behind this grid can run before the split
    // kernel has finished
    wait_for_primary_grid();
    const int h = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ctx = clamped_ctx(a, b, false);
    const int t0 = blockIdx.x * kWeightTile;
    if (t0 >= ctx) return;
    const int n_splits = (ctx + a.P - 1) / a.P;
    const int t = t0 + 4 * threadIdx.x;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int g0 = 0; g0 < a.group; g0 += kWeightHeads) {
        const int n = min(kWeightHeads, a.group - g0);
        const size_t head = (size_t)b * a.H_q + (size_t)h * a.group + g0;
        __syncthreads();  // the previous heads' statistics have been used
        for (int g = warp; g < n; g += kWeightThreads / 32) {
            const float *pm = a.part_m + (head + g) * a.S_max;
            const float *pl = a.part_l + (head + g) * a.S_max;
            float M = -INFINITY, U = 0.f;
            for (int s = lane; s < n_splits; s += 32) M = fmaxf(M, pm[s]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
            for (int s = lane; s < n_splits; s += 32)  // (without a maximum: 0, or NaN)
                U += M == -INFINITY ? pl[s] : pl[s] * exp2f(pm[s] - M);
            U = warp_sum(U);
            if (lane == 0) {
                top[g] = M;
                inv[g] = U == 0.f ? 0.f : 1.f / U;  // no usable token: no weight
            }
        }
        __syncthreads();
        if (t < ctx) add_weights(a, a.scores + head * a.score_stride + t, n, top, inv, sum);
    }
    if (t < ctx) write_weights(a, b, h, t, ctx, sum);
}

}  // namespace pa
