// evict.cuh -- cutting a paged cache back to the tokens attended to most.
//
// Page "字节跳动 AI Infra (2)", KV table, H2O row: keep the important tokens
// only. Of a row's n cached positions, each K/V head keeps `budget`: the
// first and the last ones (attention sinks and the local context) and, of
// those between, the ones of largest accumulated weight (decode_weights.cuh),
// ties to the lowest position; a NaN weight ranks above every number. The
// kept tokens' K and V move, in order, to positions 0 .. budget - 1 of the
// row's destination table, their weights likewise.
//
// Two kernels. evict_select: one cluster of CTAs per (row, K/V head) finds
// the kept positions (row_select.cuh) straight from the weights in global
// memory. evict_move: moves the rows.
//
// A destination block may be the row's own block at the same place (the cache
// is then compacted in place) or a block no row reads. In place, the token
// kept i-th sits at a position p_i >= i, and it may be written over position
// i only once whatever sits there has been read. So one CTA takes a column of
// the rows -- `width` bytes of K or of V, for one (row, K/V head) -- through
// the kept tokens in order, a chunk of them at a time: every load of a chunk
// comes before a barrier, every store after it. Tokens of later chunks have
// positions p_i >= i, which no earlier chunk has written. Columns are
// independent, which is where the parallelism of a small batch comes from.
// Tokens that stay where they are are neither read nor written.
//
// Bound by the bytes: the weights twice, the moved tokens' rows read and
// written once.
#pragma once

#include "row_select.cuh"

namespace pa {

constexpr int kEvictThreads = 512;

struct EvictArgs {
    char *k_cache, *v_cache;
    float *weights_out;
    const float *weights_in;  // may be weights_out
    int32_t *kept;            // [B][H_kv][budget], ascending, -1 past the last
    int32_t *new_lens;        // [B]
    const int32_t *block_tables;
    const int32_t *dst_tables;
    const int32_t *context_lens;
    long long stride;         // positions per (row, K/V head) of the weights
    int H_kv, bs, bs_shift, NB, MB, dst_MB, max_ctx;
    int budget, first, last;
    int row_bytes;            // D * element size
    int columns;              // of K, and of V
};

__device__ __forceinline__ int evict_len(const EvictArgs &a, int b, bool report) {
    int n = __ldg(a.context_lens + b);
    if (n < 0 || n > a.max_ctx) {
        if (report) flag_error(PA_ERR_BAD_TABLE);
        n = n < 0 ? 0 : a.max_ctx;
    }
    return n;
}

__global__ void __launch_bounds__(kEvictThreads)
    evict_select_kernel(const __grid_constant__ EvictArgs a) {
    __shared__ RowSelectSmem sm;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int h = blockIdx.y, b = blockIdx.z;
    int32_t *dst = a.kept + (size_t)((long long)b * a.H_kv + h) * a.budget;
    const bool lead = rank == 0 && h == 0 && threadIdx.x == 0;
    const int n = evict_len(a, b, lead);
    if (lead) a.new_lens[b] = min(n, a.budget);
    const int t = rank * kEvictThreads + threadIdx.x, threads = ranks * kEvictThreads;
    if (n <= a.budget) {  // nothing to evict (the whole cluster returns here)
        for (int i = t; i < a.budget; i += threads) dst[i] = i < n ? i : -1;
        return;
    }
    for (int i = t; i < a.first; i += threads) dst[i] = i;
    for (int i = t; i < a.last; i += threads) dst[a.budget - a.last + i] = n - a.last + i;
    const int need = a.budget - a.first - a.last;
    if (need == 0) return;
    const int middle = n - a.first - a.last;  // more than need
    const int seg = (middle + ranks - 1) / ranks;
    const int s0 = min(rank * seg, middle);
    const int count = min(seg, middle - s0);
    const float *w = a.weights_in + (size_t)((long long)b * a.H_kv + h) * a.stride + a.first + s0;
    auto key_at = [&](int i) { return order_key(w[i]); };
    const Cut<uint32_t> cut = cluster_cut<kEvictThreads, uint32_t>(cluster, sm, key_at, count, (uint32_t)need);
    cluster_emit<kEvictThreads, uint32_t>(cluster, sm, key_at, count, cut, [&](int place, int i) {
        dst[a.first + place] = a.first + s0 + i;
    });
    cluster.sync();  // no CTA exits while another may read its shared memory
}

constexpr int kMoveThreads = 256;
constexpr int kMoveLoads = 8;  // 16-byte loads a thread has in flight

__device__ __forceinline__ uint4 load_row(const char *p) {
    uint4 x;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                 : "l"(p)
                 : "memory");
    return x;
}

// Grid: (columns of K, columns of V, weights; K/V head; row).
__global__ void __launch_bounds__(kMoveThreads)
    evict_move_kernel(const __grid_constant__ EvictArgs a) {
    constexpr int U = kMoveLoads;
    constexpr int kMaxChunk = kMoveThreads / 4 * U;  // columns are at least 64 bytes wide
    __shared__ long long from[2][kMaxChunk], to[2][kMaxChunk];
    const int h = blockIdx.y, b = blockIdx.z;
    const int n = evict_len(a, b, false);
    const int kept = min(n, a.budget);
    const int32_t *pos = a.kept + (size_t)((long long)b * a.H_kv + h) * a.budget;

    if ((int)blockIdx.x == 2 * a.columns) {  // the weights' column
        const size_t row = (size_t)((long long)b * a.H_kv + h) * a.stride;
        const float *in = a.weights_in + row;
        float *out = a.weights_out + row;
        for (int c0 = 0; c0 < kept; c0 += kMoveThreads * U) {
            float x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = c0 + u * kMoveThreads + threadIdx.x;
                if (i < kept) x[u] = in[pos[i]];
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = c0 + u * kMoveThreads + threadIdx.x;
                if (i < kept) out[i] = x[u];
            }
        }
        for (int i = kept + threadIdx.x; i < n; i += kMoveThreads) out[i] = 0.f;
        return;
    }

    const bool is_v = (int)blockIdx.x >= a.columns;
    const int width = a.row_bytes / a.columns;
    const int per_row = width >> 4;                // threads on one token, a power of two
    const int chunk = kMoveThreads / per_row * U;  // tokens
    const int r0 = threadIdx.x / per_row;
    const int rows = kMoveThreads / per_row;
    char *cache = (is_v ? a.v_cache : a.k_cache) +
                  (size_t)((int)blockIdx.x - (is_v ? a.columns : 0)) * width +
                  (size_t)(threadIdx.x % per_row) * 16;
    const int32_t *src_row = a.block_tables + (size_t)b * a.MB;
    const int32_t *dst_row = a.dst_tables + (size_t)b * a.dst_MB;
    // cache rows the chunk's tokens come from and go to, -1 for one that stays
    auto locate = [&](int c0, int half) {
        for (int i = threadIdx.x; i < chunk; i += kMoveThreads) {
            long long s = -1, d = -1;
            if (c0 + i < kept) {
                const int p = pos[c0 + i], q = c0 + i;
                const int sb = __ldg(src_row + (p >> a.bs_shift));
                const int db = __ldg(dst_row + (q >> a.bs_shift));
                if (sb < 0 || sb >= a.NB || db < 0 || db >= a.NB) {
                    flag_error(PA_ERR_BAD_TABLE);
                } else if (sb != db || p != q) {
                    s = (((long long)sb * a.H_kv + h) << a.bs_shift) + (p & (a.bs - 1));
                    d = (((long long)db * a.H_kv + h) << a.bs_shift) + (q & (a.bs - 1));
                }
            }
            from[half][i] = s;
            to[half][i] = d;
        }
    };
    locate(0, 0);
    __syncthreads();
    int half = 0;
    for (int c0 = 0; c0 < kept; c0 += chunk, half ^= 1) {
        uint4 x[U];
        long long d[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = u * rows + r0;
            const long long s = from[half][i];
            d[u] = to[half][i];
            if (s >= 0) x[u] = load_row(cache + s * a.row_bytes);
        }
        locate(c0 + chunk, half ^ 1);
        __syncthreads();  // every load of the chunk before any of its stores
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (d[u] >= 0) *reinterpret_cast<uint4 *>(cache + d[u] * a.row_bytes) = x[u];
    }
}

}  // namespace pa
