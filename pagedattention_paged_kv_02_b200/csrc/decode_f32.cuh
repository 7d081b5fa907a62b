// decode_f32.cuh -- fp32 decode over listed blocks, and fp32 decode that
// leaves its scores (Span::kListed and Span::kWeighted of decode.cuh, same
// decomposition, table slices, epilogues).
//
// No tensor core takes fp32 without rounding it, so the products are fused
// multiply-adds; what matters is how few instructions go with them. A warp
// works on 16-token chunks:
//   scores: lane l takes token l % 16 and half the dimensions, for all query
//     heads of the tile; it walks its row in 16-byte steps from a place of its
//     own (step i reads vector i + token), so that neither the rows, 128 bytes
//     apart in the banks, nor the queries meet in a bank. One shuffle joins
//     the halves. Per token and head that is D / 32 fused multiply-adds a lane
//     and no reduction tree (a dot product across the lanes takes five
//     shuffles for D / 32 of them).
//   weights: a maximum over 16 lanes and one exponential per token and head;
//     the sums stay with the lanes until the end.
//   output: lanes over the dimensions; a token's weights for all heads come
//     from shared memory as one or two broadcast vectors.
// One 16-token stage per warp: 64 KB of shared memory for four warps at D =
// 128, so that three CTAs share an SM and overlap copies and arithmetic.
// Against the kernel of decode_split_f32 (a dot product across the warp per
// token and head), one row in partitions of 1024: 16 query heads on each of 8
// K/V heads over 1192 tokens, 363 -> 72 us; 16 on each of 2 over 675, 251 -> 50.
#pragma once

#include "decode.cuh"

namespace pa {

constexpr int kF32Warps = 4;

template <int D, int HT>
struct F32Smem {
    static constexpr int NW = kF32Warps;
    static constexpr int kStage = 2 * kChunk * D * 4;  // K rows, then V rows
    static constexpr int kRing = NW * kStage;
    static constexpr int kMerge = NW * HT * (D + 4) * 4 + 2 * NW * HT * 4;
    static constexpr int kOwn = (2 * HT + HT * D) * 4;  // cluster_epilogue's
    static constexpr int kStages =
        ((kRing > kMerge + kOwn ? kRing : kMerge + kOwn) + 1023) / 1024 * 1024;
    static constexpr int kQ = kStages;
    static constexpr int kP = kQ + HT * D * 4;
    static constexpr int kBars = kP + (NW * kChunk * HT * 4 + 15) / 16 * 16;
    static constexpr int kTable = kBars + NW * 8;
};

// N floats in shared memory, aligned to their size or 16 bytes.
template <int N>
__device__ __forceinline__ void read_vec(const float *p, float (&x)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const float4 y = reinterpret_cast<const float4 *>(p)[i];
            x[4 * i] = y.x, x[4 * i + 1] = y.y, x[4 * i + 2] = y.z, x[4 * i + 3] = y.w;
        }
    } else if constexpr (N == 2) {
        const float2 y = *reinterpret_cast<const float2 *>(p);
        x[0] = y.x, x[1] = y.y;
    } else {
        x[0] = p[0];
    }
}
template <int N>
__device__ __forceinline__ void store_vec(float *p, const float (&x)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            reinterpret_cast<float4 *>(p)[i] =
                make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = x[i];
    }
}

template <int D, int HT, Span SPAN>
__global__ void __launch_bounds__(kF32Warps * 32)
    decode_rows_f32(const __grid_constant__ DecodeArgs a) {
    static_assert(SPAN == Span::kListed || SPAN == Span::kWeighted, "see decode_split_f32");
    constexpr bool LISTED = SPAN == Span::kListed;
    constexpr bool WEIGHTED = SPAN == Span::kWeighted;
    using L = F32Smem<D, HT>;
    constexpr int NW = kF32Warps;
    constexpr int VEC = D / 32;  // output dims per lane
    constexpr int HV = D / 8;    // 16-byte vectors of half a row

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    int32_t *tbl = reinterpret_cast<int32_t *>(smem + L::kTable);
    float *qs = reinterpret_cast<float *>(smem + L::kQ);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = blockIdx.x;
    const int kvh = blockIdx.y / a.n_htiles, ht = blockIdx.y - kvh * a.n_htiles;
    const int b = blockIdx.z;
    const int h0 = kvh * a.group + ht * kHeadsF32;
    const int nh = min(HT, a.group - ht * kHeadsF32);

    allow_dependent_launch();
    const int ctx = clamped_ctx(a, b, s == 0 && blockIdx.y == 0 && threadIdx.x == 0);
    const int n_splits = LISTED ? a.S_max : (ctx + a.P - 1) / a.P;
    if (!LISTED) {
        if (s >= (n_splits > 0 ? n_splits : 1)) return;
        if (ctx == 0) {
            write_zero_rows<D, float>(a, b, h0, nh);
            return;
        }
    }
    const int tok0 = s * a.P;
    const int tok1 = min(tok0 + a.P, LISTED ? a.n_listed << a.bs_shift : ctx);
    const int n_chunks = (tok1 - tok0 + kChunk - 1) / kChunk;
    const int lb0 = tok0 >> a.bs_shift;
    const int n_tbl = ((tok1 - 1) >> a.bs_shift) - lb0 + 1;
    if constexpr (LISTED)
        load_listed(a, b, kvh, ctx, lb0, n_tbl, tbl);
    else
        load_table(a, b, lb0, n_tbl, tbl);
    const uint32_t bar = sbase + L::kBars + warp * 8;
    if (lane == 0) {
        mbar_init(bar, 1);
        fence_mbar_init();
    }
    {
        const float *q = reinterpret_cast<const float *>(a.q) + ((size_t)b * a.H_q + h0) * D;
        for (int i = threadIdx.x; i < HT * D; i += NW * 32) qs[i] = i < nh * D ? __ldg(q + i) : 0.f;
    }
    __syncthreads();

    const int my_n = n_chunks > warp ? (n_chunks - warp + NW - 1) / NW : 0;
    const float *ks = reinterpret_cast<const float *>(smem + warp * L::kStage);
    const float *vs = ks + kChunk * D;
    float *ps = reinterpret_cast<float *>(smem + L::kP) + warp * kChunk * HT;
    auto position = [&](int i) { return tok0 + (warp + i * NW) * kChunk; };
    auto issue = [&](int i) {  // lane 0
        const int t = position(i);
        const int id = block_of_chunk<LISTED>(a, tbl, lb0, t);
        if (id < 0) {
            mbar_arrive(bar);  // nothing to load; the chunk is skipped
            return;
        }
        mbar_arrive_expect_tx(bar, L::kStage);
        const size_t page = (((size_t)id * a.H_kv + kvh) * a.bs + (t & (a.bs - 1))) * D;
        const uint32_t dst = sbase + warp * L::kStage;
        bulk_load(dst, reinterpret_cast<const float *>(a.k_cache) + page, L::kStage / 2, bar);
        bulk_load(dst + L::kStage / 2, reinterpret_cast<const float *>(a.v_cache) + page,
                  L::kStage / 2, bar);
    };
    if (lane == 0 && my_n > 0) issue(0);

    float acc[HT][VEC], m[HT], l[HT];
#pragma unroll
    for (int g = 0; g < HT; ++g) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) acc[g][v] = 0.f;
        m[g] = -INFINITY;
        l[g] = 0.f;
    }
    float *scores = nullptr;
    if constexpr (WEIGHTED) scores = a.scores + ((size_t)b * a.H_q + h0) * a.score_stride;
    const int tok = lane & 15, half = lane >> 4;
    bool failed = false;
    int i = 0;
    for (; i < my_n; ++i) {
        const bool ok = mbar_wait(bar, i & 1, a.timeout_ns);
        if (!__all_sync(0xffffffffu, ok)) {
            failed = true;
            break;
        }
        const int t = position(i);
        if (block_of_chunk<LISTED>(a, tbl, lb0, t) >= 0) {
            const int valid = valid_of_chunk<LISTED>(a, tbl, lb0, t, tok1);
            float sc[HT];
#pragma unroll
            for (int g = 0; g < HT; ++g) sc[g] = 0.f;
            const float4 *k4 = reinterpret_cast<const float4 *>(ks) + tok * (D / 4) + half * HV;
            const float4 *q4 = reinterpret_cast<const float4 *>(qs) + half * HV;
#pragma unroll 4
            for (int v = 0; v < HV; ++v) {
                const int at = (v + tok) % HV;
                const float4 k = k4[at];
#pragma unroll
                for (int g = 0; g < HT; ++g) {
                    const float4 q = q4[g * (D / 4) + at];
                    sc[g] = fmaf(q.x, k.x, sc[g]);
                    sc[g] = fmaf(q.y, k.y, sc[g]);
                    sc[g] = fmaf(q.z, k.z, sc[g]);
                    sc[g] = fmaf(q.w, k.w, sc[g]);
                }
            }
            bool moved = false;
            float c[HT];
#pragma unroll
            for (int g = 0; g < HT; ++g) {
                sc[g] += __shfl_xor_sync(0xffffffffu, sc[g], 16);
                sc[g] = tok < valid ? sc[g] * a.scale_log2 : -INFINITY;
                if (WEIGHTED && half == 0 && g < nh)
                    scores[(size_t)g * a.score_stride + t + tok] = sc[g];
                float mx = sc[g];
#pragma unroll
                for (int o = 8; o > 0; o >>= 1)
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float mn = fmaxf(m[g], mx);
                c[g] = exp2f(m[g] - mn);
                m[g] = mn;
                moved |= c[g] != 1.f;
                sc[g] = exp2f(sc[g] - mn);
                l[g] = l[g] * c[g] + (half == 0 ? sc[g] : 0.f);
            }
            if (half == 0) store_vec<HT>(ps + tok * HT, sc);
            if (moved) {  // the same for every lane
#pragma unroll
                for (int g = 0; g < HT; ++g)
#pragma unroll
                    for (int v = 0; v < VEC; ++v) acc[g][v] *= c[g];
            }
            __syncwarp();
#pragma unroll 4
            for (int j = 0; j < valid; ++j) {  // tokens past the end are never touched
                float x[VEC], p[HT];
                read_vec<VEC>(vs + j * D + lane * VEC, x);
                read_vec<HT>(ps + j * HT, p);
#pragma unroll
                for (int g = 0; g < HT; ++g)
#pragma unroll
                    for (int v = 0; v < VEC; ++v) acc[g][v] = fmaf(p[g], x[v], acc[g][v]);
            }
        } else if constexpr (WEIGHTED) {
            clear_scores(a, scores, t, nh, lane);
        }
        __syncwarp();
        if (lane == 0 && i + 1 < my_n) {
            fence_proxy_async_smem();  // order this warp's reads before the refill
            issue(i + 1);
        }
    }
    if (failed) {
        flag_error(PA_ERR_TIMEOUT);
        mbar_wait(bar, i & 1, a.timeout_ns);  // let the copy in flight land (bounded)
    }
#pragma unroll
    for (int g = 0; g < HT; ++g) l[g] = warp_sum(l[g]);

    __syncthreads();  // every warp is done with its stage: reuse them
    constexpr int OS = D + 4;
    float *red_o = reinterpret_cast<float *>(smem);
    float *red_m = reinterpret_cast<float *>(smem + NW * HT * OS * 4);
    float *red_l = red_m + NW * HT;
#pragma unroll
    for (int g = 0; g < HT; ++g) {
        if (lane == 0) {
            red_m[warp * HT + g] = m[g];
            red_l[warp * HT + g] = l[g];
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) red_o[(warp * HT + g) * OS + lane * VEC + v] = acc[g][v];
    }
    __syncthreads();
    if (LISTED && a.cluster) {
        cluster_epilogue<D, NW, HT, float>(a, red_o, red_m, red_l,
                                           reinterpret_cast<float *>(smem + L::kMerge), b, h0, nh);
        return;
    }
    decode_epilogue<D, NW, HT, float>(a, red_o, red_m, red_l, b, h0, nh, s, n_splits);
    if constexpr (WEIGHTED) write_statistics<NW, HT>(a, red_m, red_l, b, h0, nh, s, kvh, ctx);
}

}  // namespace pa
