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
// the kept positions (row_select.cuh), the order keys of its weights in shared
// memory where they fit. evict_move, a programmatic dependent: moves the rows.
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
// Tokens that stay where they are are neither read nor written. A row that
// moves into other blocks throughout has no such order: there a CTA takes a run
// of whole tokens instead, 256 bytes at a time (512 MB, four rows of 16K kept
// tokens of 8 heads: 90 us, and 112 by 64-byte columns). In place few rows make
// few columns and the move takes longer, selection included 150 us against 129
// for those four rows and 117 against 57 for one of them; 64 rows make enough
// (113 either way).
//
// Bound by the bytes: the weights twice, the moved tokens' rows read and
// written once.
#pragma once

#include "decode.cuh"
#include "row_select.cuh"

namespace pa {

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
    int parts;                // CTAs that share a (row, K/V head)'s K, and its V
    int columns;              // of them, those that take columns where order matters
    int weight_parts;         // CTAs that share its weights
    int stage;                // weights of a segment that fit shared memory
};

__device__ __forceinline__ int evict_len(const EvictArgs &a, int b, bool report) {
    int n = __ldg(a.context_lens + b);
    if (n < 0 || n > a.max_ctx) {
        if (report) flag_error(PA_ERR_BAD_TABLE);
        n = n < 0 ? 0 : a.max_ctx;
    }
    return n;
}

constexpr int kCandidates = 2048;  // of a row, in the bin that holds the border
// Up to this many of them are ranked one against the others (512 rows of 1.5K to
// 4K weights: 114.1 -> 112.6 us with the move), which grows with their square
// (256: the same; 512: four rows of up to 128K weights 128 -> 138 us).
constexpr int kFewCandidates = 128;

struct EvictSmem {
    RowSelectSmem row;
    uint32_t lo, hi;               // range of this CTA's keys
    alignas(16) uint32_t bins[kCutBins];
    uint32_t border, above, in_border;
    uint32_t candidates;           // of this CTA
    uint32_t own[kCandidates];     // its candidates
    alignas(16) uint32_t all[kCandidates];  // the row's
};

// The cut of the cluster's row with the keys of a CTA's segment in shared
// memory (0 from n up to a multiple of 8), and the counts cluster_place needs.
// The time goes into passes over the keys and into meetings of the cluster. So
// there are three passes, four keys to a read -- one adds the keys to 1024 bins
// over the row's range, one counts what is above the border's bin and sets aside
// what is in it, the last one (cluster_place) hands the kept items out -- and
// every CTA closes in on the border among the row's candidates by itself.
// False, for the whole cluster, when there are too many candidates.
template <int T, typename Row>
__device__ __forceinline__ bool staged_cut(const Row &cluster, EvictSmem &sm, const uint32_t *keys,
                                           int n, uint32_t need, Cut<uint32_t> &cut) {
    constexpr int PER = kCutBins / T;
    const int tid = threadIdx.x, ranks = cluster.ranks();
    uint32_t lo = 0xffffffffu, hi = 0;
    for (int r = 0; r < ranks; ++r) {
        const uint32_t *p = cluster.at(&sm.lo, r);  // lo, hi
        lo = min(lo, p[0]);
        hi = max(hi, p[1]);
    }
    // the bins cover the 32 octaves below the largest weight, the lowest one all
    // that is smaller (a zero would stretch them over every exponent)
    const uint32_t low = hi - min(hi - lo, (1u << 28) - 1);
    const int shift = max(0, bit_width(hi - low) - 10);
    auto count_key = [&](uint32_t k) {
        if (k != 0) atomicAdd(sm.bins + ((max(k, low) - low) >> shift), 1u);
    };
    const uint4 *quads = reinterpret_cast<const uint4 *>(keys);
    const int n_quads = (n + 3) / 4;
#pragma unroll 2
    for (int i = tid; i < n_quads; i += T) {
        const uint4 x = quads[i];
        count_key(x.x), count_key(x.y), count_key(x.z), count_key(x.w);
    }
    cluster.sync();
    uint32_t c[PER] = {}, mine = 0, all;  // from bin kCutBins - 1 - tid * PER down
#pragma unroll 8
    for (int r = 0; r < ranks; ++r) {
        const uint32_t *p = cluster.at(sm.bins, r) + kCutBins - (tid + 1) * PER;
        if constexpr (PER == 2) {
            const uint2 x = *reinterpret_cast<const uint2 *>(p);
            c[0] += x.y, c[1] += x.x;
        } else {
            static_assert(PER == 4, "one wide read");
            const uint4 x = *reinterpret_cast<const uint4 *>(p);
            c[0] += x.w, c[1] += x.z, c[2] += x.y, c[3] += x.x;
        }
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) mine += c[j];
    uint32_t above = block_before<T>(sm.row, mine, all);
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
    // the bin's lowest key (above 0, the padding) and the width of its range
    const uint32_t first = sm.border == 0 ? lo : low + (sm.border << shift);
    const uint32_t span = low + (sm.border << shift) + ((1u << shift) - 1) - first;
    uint32_t gt = 0;
#pragma unroll 2
    for (int i = tid; i < n_quads; i += T) {
        const uint4 q = quads[i];
        const uint32_t x[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (x[u] < first) continue;
            if (x[u] - first > span) {
                ++gt;
            } else {
                const uint32_t at = atomicAdd(&sm.candidates, 1u);
                if (at < kCandidates) sm.own[at] = x[u];
            }
        }
    }
    cluster.sync();
    const uint32_t inside = sm.candidates;
    const bool whole = sm.in_border == need;
    if (whole || span == 0) {  // the bin is taken whole, or is one value
        cut = whole ? Cut<uint32_t>{first - 1, 0} : Cut<uint32_t>{first, need};
        add_counts(sm.row, gt, 0);
        if (tid == 0) atomicAdd(&sm.row.count[whole ? 0 : 1], inside);
        cluster.sync();
        return true;
    }
    if (sm.in_border > kCandidates) return false;
    uint32_t rows = 0;
    for (int r = 0; r < ranks; ++r) {
        const uint32_t m = *cluster.at(&sm.candidates, r), *p = cluster.at(sm.own, r);
        for (int i = tid; i < (int)m; i += T) sm.all[rows + i] = p[i];
        rows += m;
    }
    if (rows <= kFewCandidates) {  // a thread each, the cut where `need` is reached
        if (tid < 4 && rows + tid < (rows + 3) / 4 * 4) sm.all[rows + tid] = 0;
        __syncthreads();
        if (tid < (int)rows) {
            const uint32_t k = sm.all[tid];
            uint32_t before = 0, same = 0;
            const uint4 *others = reinterpret_cast<const uint4 *>(sm.all);
#pragma unroll 4
            for (int i = 0; i < ((int)rows + 3) / 4; ++i) {
                const uint4 x = others[i];
                before += (x.x > k) + (x.y > k) + (x.z > k) + (x.w > k);
                same += (x.x == k) + (x.y == k) + (x.z == k) + (x.w == k);
            }
            if (before < need && need <= before + same) {
                sm.border = k;  // (every thread that writes writes the same)
                sm.above = need - before;
            }
        }
        __syncthreads();
        cut = Cut<uint32_t>{sm.border, sm.above};
    } else {
        __syncthreads();
        cut = cluster_cut<T, uint32_t>(
            OneCta(), sm.row, [&](int i) { return sm.all[i]; }, (int)rows, need);
    }
    uint32_t eq = 0;
    for (int i = tid; i < (int)inside; i += T) {
        gt += sm.own[i] > cut.key;
        eq += sm.own[i] == cut.key;
    }
    add_counts(sm.row, gt, eq);
    cluster.sync();
    return true;
}

template <int T, typename Row>
__global__ void __launch_bounds__(T)
    evict_select_kernel(const __grid_constant__ EvictArgs a) {
    extern __shared__ __align__(16) uint32_t evict_keys[];
    __shared__ EvictSmem sm;
    const Row cluster;
    const int rank = cluster.rank(), ranks = cluster.ranks();
    const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    int32_t *dst = a.kept + (size_t)((long long)b * a.H_kv + h) * a.budget;
    const bool lead = rank == 0 && h == 0 && tid == 0;
    const int n = evict_len(a, b, lead);
    if (lead) a.new_lens[b] = min(n, a.budget);
    const int t = rank * T + tid, threads = ranks * T;
    if (n <= a.budget) {  // nothing to evict (the whole cluster returns here)
        for (int i = t; i < a.budget; i += threads) dst[i] = i < n ? i : -1;
        return;
    }
    for (int i = t; i < a.first; i += threads) dst[i] = i;
    for (int i = t; i < a.last; i += threads) dst[a.budget - a.last + i] = n - a.last + i;
    const uint32_t need = (uint32_t)(a.budget - a.first - a.last);
    if (need == 0) return;
    const int middle = n - a.first - a.last;  // more than need
    const int seg = (middle + ranks - 1) / ranks;
    const int s0 = min(rank * seg, middle);
    const int count = min(seg, middle - s0);
    const float *w = a.weights_in + (size_t)((long long)b * a.H_kv + h) * a.stride + a.first + s0;
    auto emit = [&](int place, int i) { dst[a.first + place] = a.first + s0 + i; };
    const bool staged = seg <= a.stage;
    Cut<uint32_t> cut;
    bool done = false;
    if (staged) {
        for (int i = tid; i < kCutBins; i += T) sm.bins[i] = 0;
        if (tid == 0) {
            sm.lo = 0xffffffffu;
            sm.hi = sm.candidates = sm.row.count[0] = sm.row.count[1] = 0;
        }
        __syncthreads();
        uint32_t lo = 0xffffffffu, hi = 0;
#pragma unroll 8
        for (int i = tid; i < count; i += T) {
            const uint32_t k = order_key(__ldg(w + i));
            evict_keys[i] = k;
            lo = min(lo, k);
            hi = max(hi, k);
        }
        if (tid < 8 && count + tid < (count + 7) / 8 * 8) evict_keys[count + tid] = 0;
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if ((tid & 31) == 0) {
            atomicMin(&sm.lo, lo);
            atomicMax(&sm.hi, hi);
        }
        cluster.sync();
        if (ranks == 1 && count <= T) {
            // few weights: a thread each, in when fewer than `need` rank before
            // it (larger, or equal and earlier)
            const uint32_t k = tid < count ? evict_keys[tid] : 0;
            uint32_t before = 0;
            const uint4 *quads = reinterpret_cast<const uint4 *>(evict_keys);
            for (int i = 0; i < (count + 3) / 4; ++i) {  // (0 past the end ranks last)
                const uint4 x = quads[i];
                before += x.x > k || (x.x == k && 4 * i < tid);
                before += x.y > k || (x.y == k && 4 * i + 1 < tid);
                before += x.z > k || (x.z == k && 4 * i + 2 < tid);
                before += x.w > k || (x.w == k && 4 * i + 3 < tid);
            }
            const bool in = tid < count && before < need;
            uint32_t all;
            const uint32_t place = block_before<T>(sm.row, in, all);
            if (in) emit((int)place, tid);
            return;
        }
        done = staged_cut<T>(cluster, sm, evict_keys, count, need, cut);
    }
    if (done) {
        cluster_place<T, 8>(
            cluster, sm.row,
            [&](int i0, uint32_t(&k)[8]) {
                const uint4 *p = reinterpret_cast<const uint4 *>(evict_keys + i0);
                const uint4 none = make_uint4(0, 0, 0, 0);
                const uint4 x = i0 < count ? p[0] : none, y = i0 < count ? p[1] : none;
                k[0] = x.x, k[1] = x.y, k[2] = x.z, k[3] = x.w;
                k[4] = y.x, k[5] = y.y, k[6] = y.z, k[7] = y.w;
            },
            count, cut, emit);
    } else {  // a long segment, or many nearly equal weights
        auto key_at = [&](int i) { return staged ? evict_keys[i] : order_key(__ldg(w + i)); };
        cluster.sync();
        cut = cluster_cut<T, uint32_t>(cluster, sm.row, key_at, count, need);
        cluster_emit<T, uint32_t>(cluster, sm.row, key_at, count, cut, emit);
    }
    // the move may be placed once every row is done; not before, or its waiting
    // CTAs would be in the way of rows yet to start
    allow_dependent_launch();
    cluster.sync();  // no CTA exits while another may read its shared memory
}


__device__ __forceinline__ uint4 load_row(const char *p) {
    uint4 x;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                 : "l"(p)
                 : "memory");
    return x;
}

// Grid: (parts of K, parts of V, parts of the weights; K/V head; row). A chunk is
// U 16-byte loads of each of T threads.
template <int T, int U>
__global__ void __launch_bounds__(T)
    evict_move_kernel(const __grid_constant__ EvictArgs a) {
    constexpr int kMaxChunk = T / 4 * U;  // a token's part has 64 bytes or more
    __shared__ long long from[2][kMaxChunk], to[2][kMaxChunk];
    const int h = blockIdx.y, b = blockIdx.z;
    const int n = evict_len(a, b, false);
    const int kept = min(n, a.budget);
    wait_for_primary_grid();
    const int32_t *pos = a.kept + (size_t)((long long)b * a.H_kv + h) * a.budget;

    if ((int)blockIdx.x >= 2 * a.parts) {  // the weights
        constexpr int W = 8;               // of a chunk, per thread
        const size_t row = (size_t)((long long)b * a.H_kv + h) * a.stride;
        const float *in = a.weights_in + row;
        float *out = a.weights_out + row;
        // in place there is an order, as for the columns: one CTA keeps it
        const int part = (int)blockIdx.x - 2 * a.parts;
        const int parts = a.weights_in == a.weights_out ? 1 : a.weight_parts;
        if (part >= parts) return;
        const int run = (n + parts - 1) / parts;
        const int begin = min(part * run, n), end = min(begin + run, n);
        const int moved = min(end, kept);
        for (int c0 = begin; c0 < moved; c0 += T * W) {
            float x[W];
#pragma unroll
            for (int u = 0; u < W; ++u) {
                const int i = c0 + u * T + threadIdx.x;
                if (i < moved) x[u] = in[pos[i]];
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < W; ++u) {
                const int i = c0 + u * T + threadIdx.x;
                if (i < moved) out[i] = x[u];
            }
        }
        for (int i = max(begin, kept) + threadIdx.x; i < end; i += T) out[i] = 0.f;
        return;
    }

    const int32_t *src_row = a.block_tables + (size_t)b * a.MB;
    const int32_t *dst_row = a.dst_tables + (size_t)b * a.dst_MB;
    const bool is_v = (int)blockIdx.x >= a.parts;
    const int part = (int)blockIdx.x - (is_v ? a.parts : 0);
    bool stays = false;  // some block is its own destination
    for (int i = threadIdx.x; i < (kept + a.bs - 1) >> a.bs_shift; i += T)
        stays |= __ldg(src_row + i) == __ldg(dst_row + i);
    const bool columns = __syncthreads_or(stays) != 0;
    const int parts = columns ? a.columns : a.parts;
    if (part >= parts) return;
    const int width = columns ? a.row_bytes / parts : a.row_bytes;
    const int per_row = width >> 4;                // threads on one token, a power of two
    const int rows = T / per_row;
    const int chunk = rows * U;                    // tokens
    const int r0 = threadIdx.x / per_row;
    const int run = columns ? kept : (kept + parts - 1) / parts;
    const int begin = columns ? 0 : min(part * run, kept), end = min(begin + run, kept);
    char *cache = (is_v ? a.v_cache : a.k_cache) + (columns ? (size_t)part * width : 0) +
                  (size_t)(threadIdx.x % per_row) * 16;
    // cache rows the chunk's tokens come from and go to, -1 for one that stays
    auto locate = [&](int c0, int half) {
        for (int i = threadIdx.x; i < chunk; i += T) {
            long long s = -1, d = -1;
            if (c0 + i < end) {
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
    uint4 x0[U], x1[U];
    long long d0[U], d1[U];
    auto load = [&](uint4(&x)[U], long long(&d)[U], int half) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = u * rows + r0;
            const long long s = from[half][i];
            d[u] = to[half][i];
            if (s >= 0) x[u] = load_row(cache + s * a.row_bytes);
        }
    };
    auto store = [&](const uint4(&x)[U], const long long(&d)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (d[u] >= 0) *reinterpret_cast<uint4 *>(cache + d[u] * a.row_bytes) = x[u];
    };
    if (begin >= end) return;
    locate(begin, 0);
    __syncthreads();
    load(x0, d0, 0);
    locate(begin + chunk, 1);
    for (int c0 = begin; c0 < end; c0 += 2 * chunk) {
        __syncthreads();  // every load of chunk c0 before any of its stores
        load(x1, d1, 1);
        locate(c0 + 2 * chunk, 0);
        store(x0, d0);
        __syncthreads();  // the same for the chunk behind it
        load(x0, d0, 0);
        locate(c0 + 3 * chunk, 1);
        store(x1, d1);
    }
}

}  // namespace pa
