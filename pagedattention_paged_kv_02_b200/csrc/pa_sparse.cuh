// pa_sparse.cuh -- host entry points of the operators that decode over part
// of a paged cache (declared in include/pa.h): argument checks and launch
// configuration. Included by pa_lib.cu, whose helpers it uses.
#pragma once

namespace {

// Checks shared by these entry points; PA_OK means "go on".
pa_status check_cache_shape(int num_seqs, int num_kv_heads, int head_dim, int block_size,
                            int num_blocks, int max_blocks_per_seq, pa_dtype dtype) {
    if (num_seqs < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
        num_blocks <= 0 || max_blocks_per_seq <= 0)
        return PA_ERR_INVALID_ARG;
    if (dtype != PA_F32 && dtype != PA_BF16) return PA_ERR_INVALID_ARG;
    if (!head_dim_ok(head_dim) || !block_size_ok(block_size)) return PA_ERR_UNSUPPORTED;
    if (num_seqs > 65535 || num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
    if ((long long)max_blocks_per_seq * block_size > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

// Of a row's weights or listed tokens, and entries of its lists: sums of two stay
// in an int.
constexpr int kMaxPositions = 1 << 30;

constexpr int kSelectStage = 24576;  // scores a selecting CTA keeps in shared memory, at most

constexpr int kEvictStage = 40960;   // weights a selecting CTA keeps in shared memory, at most
constexpr size_t evict_stage_bytes(int weights) { return ((size_t)weights + 8) * 4; }

// A programmatic dependent of the launch before it: its CTAs may be placed
// while that grid finishes, and wait for it before they use its results.
template <typename K, typename... A>
pa_status launch_dependent(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t st,
                           const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = st;
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
        cudaGetLastError();
        return PA_ERR_CUDA;
    }
    return launch_status();
}

// CTAs of a row's cluster: enough for every SM when there are few rows, as
// long as a CTA keeps `grain` items of the longest row or more.
int cluster_size(long long rows, long long items, int grain) {
    int cs = 1;
    while (cs < kMaxCluster && rows * cs < 148 && items > (long long)cs * grain) cs *= 2;
    return cs;
}

// KV tokens per partition of these decodes over `total` tokens a row, or -1.
// Automatic: up to 1024 tokens, halved while the grid has fewer than two CTAs
// per SM and a partition keeps more than 128 tokens (a partition's tokens are a
// chain of 64 per step of its four warps: 1024 of them take about 20 us).
int spread_partition(long long total, long long rows, int partition_size) {
    if (total <= 0 || total > kMaxPositions) return -1;
    if (partition_size > 0)
        return partition_size % kChunk != 0 || partition_size > kMaxPartition ? -1 : partition_size;
    const int whole = round16((int)total);
    if (partition_size < 0) return whole <= kMaxPartition ? whole : -1;
    int P = std::min(whole, 1024);
    while (rows * ((total + P - 1) / P) < 2 * 148 && P > 128) P = round16(P / 2);
    return P;
}
int listed_partition(int n_listed, int bs, long long rows, int partition_size) {
    return spread_partition((long long)n_listed * bs, rows, partition_size);
}

// (Row, K/V head, tile of query heads) triples of a grid.
long long listed_rows(int num_seqs, int num_q_heads, int num_kv_heads) {
    const int group = num_q_heads / num_kv_heads;
    return (long long)num_seqs * num_kv_heads * ((group + kHeadsBf16 - 1) / kHeadsBf16);
}

// Whether a row's partitions are launched as a cluster that merges them: where
// a portable cluster holds them and the grid is at most two CTAs per SM. 64
// blocks of 16 tokens, 8 K/V heads, cluster against second kernel: 6.6 / 8.7 us
// for one row, 8.4 / 10.1 for four, but 16.8 / 14.8 for eight (512 CTAs), where
// a cluster's CTAs wait for room together.
bool listed_in_cluster(long long rows, long long S) {
    return S > 1 && S <= kMaxCluster && rows * S <= 2 * 148;
}

// Partials of S partitions for every (row, query head): outputs, then lse.
size_t partial_bytes(int B, int H_q, int D, long long S) {
    if (S <= 1) return 0;
    const size_t o = (size_t)B * H_q * S * D * sizeof(float);
    const size_t l = (size_t)B * H_q * S * sizeof(float);
    return (o + 255) / 256 * 256 + (l + 255) / 256 * 256;
}

// What the weight-accumulating decode adds to pa_decode's partials: two
// statistics per partition, then the scores.
size_t statistics_bytes(int B, int H_q, long long S) {
    return ((size_t)B * H_q * S * sizeof(float) + 255) / 256 * 256;
}
size_t score_bytes(int B, int H_q, int max_ctx) {
    return ((size_t)B * H_q * round16(max_ctx) * sizeof(float) + 255) / 256 * 256;
}

// Fills what every decode form shares and launches the split kernel.
struct DecodeShape {
    int num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, max_blocks_per_seq;
    pa_dtype dtype;
};

void fill_decode(DecodeArgs &a, const DecodeShape &s, void *out, const void *q,
                 const void *k_cache, const void *v_cache, const int32_t *block_tables,
                 const int32_t *context_lens, float scale, int P, long long S, void *workspace) {
    std::memset(&a, 0, sizeof(a));
    a.out = out;
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    if (S > 1) {
        a.part_o = static_cast<float *>(workspace);
        a.part_lse = reinterpret_cast<float *>(
            static_cast<char *>(workspace) +
            ((size_t)s.num_seqs * s.num_q_heads * S * s.head_dim * 4 + 255) / 256 * 256);
    }
    a.num_seqs = s.num_seqs;
    a.H_q = s.num_q_heads;
    a.H_kv = s.num_kv_heads;
    a.group = s.num_q_heads / s.num_kv_heads;
    a.bs = s.block_size;
    a.bs_shift = __builtin_ctz((unsigned)s.block_size);
    a.NB = s.num_blocks;
    a.MB = s.max_blocks_per_seq;
    a.P = P;
    a.S_max = (int)S;
    const int ht = s.dtype == PA_BF16 ? kHeadsBf16 : kHeadsF32;
    a.n_htiles = (a.group + ht - 1) / ht;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.timeout_ns = kWaitTimeoutNs;
}

template <int D, int HT, Span SPAN>
pa_status launch_rows_f32_tile(const DecodeArgs &a, dim3 grid, cudaStream_t st) {
    constexpr size_t fixed = 1024 + F32Smem<D, HT>::kTable;
    const size_t smem = fixed + slice_bytes(a.P, a.bs, slice_arrays(SPAN));
    auto k = decode_rows_f32<D, HT, SPAN>;
    if (allow_smem(k, fixed + kMaxSlice * slice_arrays(SPAN)) != cudaSuccess) return PA_ERR_CUDA;
    if (a.cluster) return launch_clusters(k, grid, kF32Warps * 32, (int)grid.x, smem, st, a);
    k<<<grid, kF32Warps * 32, smem, st>>>(a);
    return launch_status();
}

// A tile of 1, 4 or 8 query heads, whichever wastes the least of it.
template <int D, Span SPAN>
pa_status launch_rows_f32(const DecodeArgs &a, dim3 grid, cudaStream_t st) {
    return a.group == 1   ? launch_rows_f32_tile<D, 1, SPAN>(a, grid, st)
           : a.group <= 4 ? launch_rows_f32_tile<D, 4, SPAN>(a, grid, st)
                          : launch_rows_f32_tile<D, 8, SPAN>(a, grid, st);
}

template <Span SPAN>
pa_status launch_split(const DecodeArgs &a, const DecodeShape &s, cudaStream_t stream) {
    const dim3 grid((unsigned)a.S_max, (unsigned)(a.H_kv * a.n_htiles), (unsigned)a.num_seqs);
    if (s.dtype == PA_BF16) {
        CUtensorMap mk, mv;
        if (!encode_cache_map(&mk, a.k_cache, a.NB, a.H_kv, a.bs, s.head_dim, kChunk) ||
            !encode_cache_map(&mv, a.v_cache, a.NB, a.H_kv, a.bs, s.head_dim, kChunk))
            return PA_ERR_CUDA;
        return s.head_dim == 128
                   ? launch_decode_bf16<128, kDecodeWarps, kDecodeStages, SPAN>(a, mk, mv, grid,
                                                                                stream)
                   : launch_decode_bf16<64, kDecodeWarps, kDecodeStages, SPAN>(a, mk, mv, grid,
                                                                               stream);
    }
    return s.head_dim == 128 ? launch_rows_f32<128, SPAN>(a, grid, stream)
                             : launch_rows_f32<64, SPAN>(a, grid, stream);
}

// Checks of the arguments that both decode forms below share, in pa_decode's
// order; num_seqs == 0 has been dealt with.
bool decode_pointers_ok(const void *out, const void *q, const void *k_cache, const void *v_cache,
                        const void *block_tables, const void *context_lens) {
    return out && q && k_cache && v_cache && block_tables && context_lens && aligned(out, 16) &&
           aligned(q, 16) && aligned(k_cache, 16) && aligned(v_cache, 16) &&
           aligned(block_tables, 4) && aligned(context_lens, 4);
}

}  // namespace

extern "C" {

pa_status pa_update_key_bounds(void *key_bounds, const void *k_cache, const int32_t *block_tables,
                               const int32_t *context_lens, const int32_t *new_lens, int num_seqs,
                               int max_new_len, int num_kv_heads, int head_dim, int block_size,
                               int num_blocks, int max_blocks_per_seq, pa_dtype dtype,
                               cudaStream_t stream) {
    const pa_status st = check_cache_shape(num_seqs, num_kv_heads, head_dim, block_size,
                                           num_blocks, max_blocks_per_seq, dtype);
    if (st != PA_OK) return st;
    if (max_new_len < 0 || (long long)max_new_len > (long long)max_blocks_per_seq * block_size)
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || max_new_len == 0) return PA_OK;
    if (!key_bounds || !k_cache || !block_tables || !context_lens || !new_lens)
        return PA_ERR_INVALID_ARG;
    if (!aligned(key_bounds, 16) || !aligned(k_cache, 16) || !aligned(block_tables, 4) ||
        !aligned(context_lens, 4) || !aligned(new_lens, 4))
        return PA_ERR_INVALID_ARG;
    BoundsArgs a;
    a.key_bounds = key_bounds;
    a.k_cache = k_cache;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.new_lens = new_lens;
    a.H_kv = num_kv_heads;
    a.bs = block_size;
    a.bs_shift = __builtin_ctz((unsigned)block_size);
    a.NB = num_blocks;
    a.MB = max_blocks_per_seq;
    a.max_new = max_new_len;
    // max_new_len tokens touch at most this many blocks
    const long long blocks = std::min<long long>(
        ((long long)max_new_len + block_size - 2) / block_size + 1, max_blocks_per_seq);
    const long long gx = (blocks * num_kv_heads + kBoundsWarps - 1) / kBoundsWarps;
    if (gx > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)gx, (unsigned)num_seqs);
    constexpr int threads = kBoundsWarps * 32;
    if (dtype == PA_BF16) {
        if (head_dim == 128)
            key_bounds_kernel<128, __nv_bfloat16><<<grid, threads, 0, stream>>>(a);
        else
            key_bounds_kernel<64, __nv_bfloat16><<<grid, threads, 0, stream>>>(a);
    } else {
        if (head_dim == 128)
            key_bounds_kernel<128, float><<<grid, threads, 0, stream>>>(a);
        else
            key_bounds_kernel<64, float><<<grid, threads, 0, stream>>>(a);
    }
    return launch_status();
}

size_t pa_select_blocks_workspace_size(int num_seqs, int num_kv_heads, int block_size,
                                       int max_context_len) {
    if (num_seqs <= 0 || num_kv_heads <= 0 || block_size <= 0 || max_context_len <= 0) return 0;
    return (size_t)num_seqs * num_kv_heads *
           (((size_t)max_context_len + block_size - 1) / block_size) * sizeof(uint64_t);
}

pa_status pa_select_blocks(int32_t *selected, const void *q, const void *key_bounds,
                           const int32_t *block_tables, const int32_t *context_lens,
                           int max_selected, int num_first, int num_last, int num_seqs,
                           int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                           int num_blocks, int max_blocks_per_seq, int max_context_len,
                           void *workspace, size_t workspace_bytes_given, pa_dtype dtype,
                           cudaStream_t stream) {
    const pa_status st = check_cache_shape(num_seqs, num_kv_heads, head_dim, block_size,
                                           num_blocks, max_blocks_per_seq, dtype);
    if (st != PA_OK) return st;
    if (num_q_heads <= 0 || max_context_len < 0 || max_selected <= 0 || num_first < 0 ||
        num_last < 0 || (long long)num_first + num_last > max_selected)
        return PA_ERR_INVALID_ARG;
    if (num_q_heads % num_kv_heads != 0) return PA_ERR_UNSUPPORTED;
    if ((long long)max_context_len > (long long)max_blocks_per_seq * block_size)
        return PA_ERR_INVALID_ARG;
    if (max_selected > kMaxPositions) return PA_ERR_UNSUPPORTED;
    const long long blocks = ((long long)max_context_len + block_size - 1) / block_size;
    if (num_seqs == 0) return PA_OK;
    if (!selected || !q || !key_bounds || !block_tables || !context_lens)
        return PA_ERR_INVALID_ARG;
    if (!aligned(selected, 4) || !aligned(q, 16) || !aligned(key_bounds, 16) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4))
        return PA_ERR_INVALID_ARG;
    SelectArgs a;
    a.selected = selected;
    a.q = q;
    a.key_bounds = key_bounds;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.H_q = num_q_heads;
    a.H_kv = num_kv_heads;
    a.group = num_q_heads / num_kv_heads;
    a.bs = block_size;
    a.bs_shift = __builtin_ctz((unsigned)block_size);
    a.NB = num_blocks;
    a.MB = max_blocks_per_seq;
    a.max_ctx = max_context_len;
    a.K = max_selected;
    a.first = num_first;
    a.last = num_last;
    a.max_blocks = (int)blocks;
    a.scores = static_cast<uint64_t *>(workspace);
    a.stage = (int)std::min<long long>(blocks, kSelectStage);
    const size_t need =
        pa_select_blocks_workspace_size(num_seqs, num_kv_heads, block_size, max_context_len);
    if (need > 0 && (!workspace || workspace_bytes_given < need || !aligned(workspace, 256)))
        return PA_ERR_WORKSPACE;
    // several tiles to a warp once the grid fills the GPU several times over
    const int tile = dtype == PA_BF16 ? kScoreRows : kScoreRowsF32;
    const long long all_tiles = (blocks + tile - 1) / tile;
    int steps = 1;
    while (steps < 4 && (long long)num_seqs * num_kv_heads * all_tiles >
                            8LL * 148 * 4 * kScoreWarps * steps)
        steps *= 2;
    a.tiles = (int)((all_tiles + steps - 1) / steps);
    const long long gx = ((long long)a.tiles * num_kv_heads + kScoreWarps - 1) / kScoreWarps;
    if (gx > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    const bool contested = blocks > max_selected && max_selected > num_first + num_last;
    if (contested) {
        const dim3 grid((unsigned)gx, (unsigned)num_seqs);
        if (dtype == PA_BF16) {
            if (head_dim == 128)
                score_blocks_bf16<128><<<grid, kScoreWarps * 32, 0, stream>>>(a);
            else
                score_blocks_bf16<64><<<grid, kScoreWarps * 32, 0, stream>>>(a);
        } else {
            if (head_dim == 128)
                score_blocks_f32<128><<<grid, kScoreWarps * 32, 0, stream>>>(a);
            else
                score_blocks_f32<64><<<grid, kScoreWarps * 32, 0, stream>>>(a);
        }
        const pa_status scored = launch_status();
        if (scored != PA_OK) return scored;
    } else {
        a.stage = 0;  // no row is scored
    }
    auto launch = [&](auto kernel, int threads) {
        const dim3 grid((unsigned)num_kv_heads, (unsigned)num_seqs);
        const size_t smem = (size_t)a.stage * sizeof(uint64_t);
        if (allow_smem(kernel, kSelectStage * sizeof(uint64_t)) != cudaSuccess) return PA_ERR_CUDA;
        if (contested) return launch_dependent(kernel, grid, threads, smem, stream, a);
        // without the scoring kernel in between, the launch before may still
        // read what this one writes
        kernel<<<grid, threads, smem, stream>>>(a);
        return launch_status();
    };
    // Threads: many for long rows, where a pass over the scores is what counts;
    // few for short ones, where barriers are, and fewer still where there are
    // rows enough to fill the GPU with them (1024 rows of up to 256 blocks:
    // 26.7 us with 128, 28.7 with 256; 8 rows of 512: 10.6 and 9.6)
    auto pick = [&](auto many, auto some, auto few) {
        if (blocks > 2048) return launch(many, 1024);
        if (blocks <= 512 && (long long)num_seqs * num_kv_heads > 4 * 148) return launch(few, 128);
        return launch(some, 256);
    };
    if (dtype == PA_BF16) {
        using T = __nv_bfloat16;
        return head_dim == 128
                   ? pick(select_blocks_kernel<1024, 128, T>, select_blocks_kernel<256, 128, T>,
                          select_blocks_kernel<128, 128, T>)
                   : pick(select_blocks_kernel<1024, 64, T>, select_blocks_kernel<256, 64, T>,
                          select_blocks_kernel<128, 64, T>);
    }
    using T = float;
    return head_dim == 128
               ? pick(select_blocks_kernel<1024, 128, T>, select_blocks_kernel<256, 128, T>,
                      select_blocks_kernel<128, 128, T>)
               : pick(select_blocks_kernel<1024, 64, T>, select_blocks_kernel<256, 64, T>,
                      select_blocks_kernel<128, 64, T>);
}

size_t pa_decode_selected_blocks_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads,
                                                int head_dim, int block_size, int max_selected,
                                                int partition_size) {
    if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        num_q_heads % num_kv_heads != 0 || block_size <= 0 || max_selected <= 0)
        return 0;
    const int P = listed_partition(max_selected, block_size,
                                   listed_rows(num_seqs, num_q_heads, num_kv_heads),
                                   partition_size);
    if (P <= 0) return 0;
    const long long S = ((long long)max_selected * block_size + P - 1) / P;
    if (listed_in_cluster(listed_rows(num_seqs, num_q_heads, num_kv_heads), S)) return 0;
    return partial_bytes(num_seqs, num_q_heads, head_dim, S);
}

pa_status pa_decode_selected_blocks(void *out, const void *q, const void *k_cache,
                                    const void *v_cache, const int32_t *block_tables,
                                    const int32_t *context_lens, const int32_t *selected,
                                    int max_selected, int num_seqs, int num_q_heads,
                                    int num_kv_heads, int head_dim, int block_size,
                                    int num_blocks, int max_blocks_per_seq, float scale,
                                    int partition_size, void *workspace,
                                    size_t workspace_bytes_given, pa_dtype dtype,
                                    cudaStream_t stream) {
    pa_status st = check_cache_shape(num_seqs, num_kv_heads, head_dim, block_size, num_blocks,
                                     max_blocks_per_seq, dtype);
    if (st != PA_OK) return st;
    if (num_q_heads <= 0 || max_selected <= 0 || !std::isfinite(scale)) return PA_ERR_INVALID_ARG;
    if (num_q_heads % num_kv_heads != 0) return PA_ERR_UNSUPPORTED;
    if ((long long)max_selected * block_size > kMaxPositions) return PA_ERR_UNSUPPORTED;
    const int P = listed_partition(max_selected, block_size,
                                   listed_rows(num_seqs, num_q_heads, num_kv_heads),
                                   partition_size);
    if (P <= 0) return partition_size > 0 ? PA_ERR_INVALID_ARG : PA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PA_OK;
    if (!decode_pointers_ok(out, q, k_cache, v_cache, block_tables, context_lens) || !selected ||
        !aligned(selected, 4))
        return PA_ERR_INVALID_ARG;
    const long long S = ((long long)max_selected * block_size + P - 1) / P;
    const size_t need = pa_decode_selected_blocks_workspace_size(
        num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_selected, partition_size);
    if (need > 0 && (!workspace || workspace_bytes_given < need || !aligned(workspace, 256)))
        return PA_ERR_WORKSPACE;
    const DecodeShape shape{num_seqs,   num_q_heads, num_kv_heads,       head_dim,
                            block_size, num_blocks,  max_blocks_per_seq, dtype};
    DecodeArgs a;
    fill_decode(a, shape, out, q, k_cache, v_cache, block_tables, context_lens, scale, P, S,
                workspace);
    if ((long long)num_kv_heads * a.n_htiles > 65535) return PA_ERR_UNSUPPORTED;
    a.max_ctx = max_blocks_per_seq * block_size;
    a.selected = selected;
    a.n_listed = max_selected;
    a.cluster = listed_in_cluster(listed_rows(num_seqs, num_q_heads, num_kv_heads), S);
    st = launch_split<Span::kListed>(a, shape, stream);
    if (st != PA_OK || S <= 1 || a.cluster) return st;
    if (dtype == PA_BF16)
        return head_dim == 128 ? launch_reduce<128, __nv_bfloat16, true>(a, stream)
                               : launch_reduce<64, __nv_bfloat16, true>(a, stream);
    return head_dim == 128 ? launch_reduce<128, float, true>(a, stream)
                           : launch_reduce<64, float, true>(a, stream);
}

size_t pa_decode_accumulate_weights_workspace_size(int num_seqs, int num_q_heads, int head_dim,
                                                   int max_context_len, int partition_size) {
    if (num_seqs <= 0 || num_q_heads <= 0 || head_dim <= 0 || max_context_len <= 0 ||
        max_context_len > kMaxPositions)
        return 0;
    // the fewest rows that these query heads can make, and so the most partitions
    const long long rows = (long long)num_seqs * ((num_q_heads + kHeadsBf16 - 1) / kHeadsBf16);
    const int P = spread_partition(max_context_len, rows, partition_size);
    if (P <= 0) return 0;
    const long long S = ((long long)max_context_len + P - 1) / P;
    return partial_bytes(num_seqs, num_q_heads, head_dim, S) +
           2 * statistics_bytes(num_seqs, num_q_heads, S) +
           score_bytes(num_seqs, num_q_heads, max_context_len);
}

pa_status pa_decode_accumulate_weights(void *out, float *weights_out, const float *weights_in,
                                       const void *q, const void *k_cache, const void *v_cache,
                                       const int32_t *block_tables, const int32_t *context_lens,
                                       int num_seqs, int num_q_heads, int num_kv_heads,
                                       int head_dim, int block_size, int num_blocks,
                                       int max_blocks_per_seq, int max_context_len,
                                       int weights_stride, float scale, int partition_size,
                                       void *workspace, size_t workspace_bytes_given,
                                       pa_dtype dtype, cudaStream_t stream) {
    pa_status st = check_cache_shape(num_seqs, num_kv_heads, head_dim, block_size, num_blocks,
                                     max_blocks_per_seq, dtype);
    if (st != PA_OK) return st;
    if (num_q_heads <= 0 || max_context_len < 0 || !std::isfinite(scale)) return PA_ERR_INVALID_ARG;
    if (num_q_heads % num_kv_heads != 0) return PA_ERR_UNSUPPORTED;
    if ((long long)max_context_len > (long long)max_blocks_per_seq * block_size ||
        weights_stride < max_context_len)
        return PA_ERR_INVALID_ARG;
    if (max_context_len > kMaxPositions) return PA_ERR_UNSUPPORTED;
    const int P = spread_partition(std::max(max_context_len, 1),
                                   listed_rows(num_seqs, num_q_heads, num_kv_heads),
                                   partition_size);
    if (P <= 0) return partition_size > 0 ? PA_ERR_INVALID_ARG : PA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PA_OK;
    if (!decode_pointers_ok(out, q, k_cache, v_cache, block_tables, context_lens) ||
        !weights_out || !aligned(weights_out, 4) || !aligned(weights_in, 4))
        return PA_ERR_INVALID_ARG;
    // the new weights go over the old ones, or elsewhere; never half over them
    const size_t span = (size_t)num_seqs * num_kv_heads * weights_stride;
    if (weights_in && weights_in != weights_out && weights_in < weights_out + span &&
        weights_out < weights_in + span)
        return PA_ERR_INVALID_ARG;
    const size_t need = pa_decode_accumulate_weights_workspace_size(
        num_seqs, num_q_heads, head_dim, max_context_len, partition_size);
    if (need > 0 && (!workspace || workspace_bytes_given < need || !aligned(workspace, 256)))
        return PA_ERR_WORKSPACE;
    const long long S = std::max<long long>(1, ((long long)max_context_len + P - 1) / P);
    const DecodeShape shape{num_seqs,   num_q_heads, num_kv_heads,       head_dim,
                            block_size, num_blocks,  max_blocks_per_seq, dtype};
    DecodeArgs a;
    fill_decode(a, shape, out, q, k_cache, v_cache, block_tables, context_lens, scale, P, S,
                workspace);
    if ((long long)num_kv_heads * a.n_htiles > 65535) return PA_ERR_UNSUPPORTED;
    a.max_ctx = max_context_len;
    char *ws = static_cast<char *>(workspace) + partial_bytes(num_seqs, num_q_heads, head_dim, S);
    a.part_m = reinterpret_cast<float *>(ws);
    a.part_l = reinterpret_cast<float *>(ws + statistics_bytes(num_seqs, num_q_heads, S));
    a.scores = reinterpret_cast<float *>(ws + 2 * statistics_bytes(num_seqs, num_q_heads, S));
    a.score_stride = round16(max_context_len);
    a.weights_out = weights_out;
    a.weights_in = weights_in;
    a.weight_stride = weights_stride;
    a.weight_vec = weights_stride % 4 == 0 && aligned(weights_out, 16) && aligned(weights_in, 16);
    a.weights_here = S == 1 && a.n_htiles == 1;
    st = launch_split<Span::kWeighted>(a, shape, stream);
    if (st != PA_OK || a.weights_here || max_context_len == 0) return st;

    st = launch_dependent(decode_weights_kernel,
                          dim3((unsigned)((max_context_len + kWeightTile - 1) / kWeightTile),
                               (unsigned)num_kv_heads, (unsigned)num_seqs),
                          kWeightThreads, 0, stream, a);
    if (st != PA_OK || S <= 1) return st;
    if (dtype == PA_BF16)
        return head_dim == 128 ? launch_reduce<128, __nv_bfloat16>(a, stream)
                               : launch_reduce<64, __nv_bfloat16>(a, stream);
    return head_dim == 128 ? launch_reduce<128, float>(a, stream)
                           : launch_reduce<64, float>(a, stream);
}

pa_status pa_evict_tokens(void *k_cache, void *v_cache, float *weights_out,
                          const float *weights_in, int32_t *kept_positions,
                          int32_t *new_context_lens, const int32_t *block_tables,
                          const int32_t *dst_block_tables, const int32_t *context_lens,
                          int budget, int num_first, int num_last, int num_seqs,
                          int num_kv_heads, int head_dim, int block_size, int num_blocks,
                          int max_blocks_per_seq, int dst_max_blocks_per_seq,
                          int max_context_len, int weights_stride, pa_dtype dtype,
                          cudaStream_t stream) {
    const pa_status st = check_cache_shape(num_seqs, num_kv_heads, head_dim, block_size,
                                           num_blocks, max_blocks_per_seq, dtype);
    if (st != PA_OK) return st;
    if (budget <= 0 || num_first < 0 || num_last < 0 ||
        (long long)num_first + num_last > budget || dst_max_blocks_per_seq <= 0 ||
        max_context_len < 0 || weights_stride < max_context_len)
        return PA_ERR_INVALID_ARG;
    if ((long long)max_context_len > (long long)max_blocks_per_seq * block_size ||
        std::min(budget, max_context_len) > (long long)dst_max_blocks_per_seq * block_size)
        return PA_ERR_INVALID_ARG;
    if (max_context_len > kMaxPositions || budget > kMaxPositions) return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PA_OK;
    if (!k_cache || !v_cache || !weights_out || !weights_in || !kept_positions ||
        !new_context_lens || !block_tables || !dst_block_tables || !context_lens)
        return PA_ERR_INVALID_ARG;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(weights_out, 4) ||
        !aligned(weights_in, 4) || !aligned(kept_positions, 4) || !aligned(new_context_lens, 4) ||
        !aligned(block_tables, 4) || !aligned(dst_block_tables, 4) || !aligned(context_lens, 4))
        return PA_ERR_INVALID_ARG;
    // both kernels read the old lengths while the first writes the new ones
    if (new_context_lens < context_lens + num_seqs && context_lens < new_context_lens + num_seqs)
        return PA_ERR_INVALID_ARG;
    const size_t span = (size_t)num_seqs * num_kv_heads * weights_stride;
    if (weights_in != weights_out && weights_in < weights_out + span &&
        weights_out < weights_in + span)
        return PA_ERR_INVALID_ARG;
    EvictArgs a;
    a.k_cache = static_cast<char *>(k_cache);
    a.v_cache = static_cast<char *>(v_cache);
    a.weights_out = weights_out;
    a.weights_in = weights_in;
    a.kept = kept_positions;
    a.new_lens = new_context_lens;
    a.block_tables = block_tables;
    a.dst_tables = dst_block_tables;
    a.context_lens = context_lens;
    a.stride = weights_stride;
    a.H_kv = num_kv_heads;
    a.bs = block_size;
    a.bs_shift = __builtin_ctz((unsigned)block_size);
    a.NB = num_blocks;
    a.MB = max_blocks_per_seq;
    a.dst_MB = dst_max_blocks_per_seq;
    a.max_ctx = max_context_len;
    a.budget = budget;
    a.first = num_first;
    a.last = num_last;
    a.row_bytes = head_dim * (dtype == PA_BF16 ? 2 : 4);
    const long long rows = (long long)num_seqs * num_kv_heads;
    const int cs = cluster_size(rows, max_context_len, 4096);
    a.stage = std::min((max_context_len + cs - 1) / cs, kEvictStage);
    const dim3 grid((unsigned)cs, (unsigned)num_kv_heads, (unsigned)num_seqs);
    const size_t smem = evict_stage_bytes(a.stage), limit = evict_stage_bytes(kEvictStage);
    // a row to a CTA of its own where there are rows enough, or they are short
    pa_status r = PA_OK;
    if (cs > 1) {
        auto k = evict_select_kernel<512, CtaCluster>;
        if (allow_smem(k, limit) != cudaSuccess) return PA_ERR_CUDA;
        r = launch_clusters(k, grid, 512, cs, smem, stream, a);
    } else if (max_context_len > 16384) {
        auto k = evict_select_kernel<512, OneCta>;
        if (allow_smem(k, limit) != cudaSuccess) return PA_ERR_CUDA;
        k<<<grid, 512, smem, stream>>>(a);
        r = launch_status();
    } else {
        auto k = evict_select_kernel<256, OneCta>;
        if (allow_smem(k, limit) != cudaSuccess) return PA_ERR_CUDA;
        k<<<grid, 256, smem, stream>>>(a);
        r = launch_status();
    }
    if (r != PA_OK) return r;
    // CTAs of a (row, K/V head)'s K and of its V: as many as the GPU holds at a
    // time (two per SM; four 16K-token rows of 8 heads: 130 us, 138 with four
    // times as many) and as have 64 tokens, or a column of 64 bytes; then of its
    // weights, in runs of 8192 or more
    const int most = std::min(budget, max_context_len);
    a.columns = a.row_bytes / 64;
    a.parts = 1;
    while (4 * rows * a.parts <= 2 * 148 && a.parts < std::max(a.columns, most / 64)) a.parts *= 2;
    a.columns = std::min(a.columns, a.parts);
    a.weight_parts = 1;
    while (2 * rows * (a.parts + a.weight_parts) <= 2 * 148 &&
           a.weight_parts * 8192LL < max_context_len)
        a.weight_parts *= 2;
    const dim3 move_grid((unsigned)(2 * a.parts + a.weight_parts), (unsigned)num_kv_heads,
                         (unsigned)num_seqs);
    // small CTAs, and more of them on an SM, where a CTA has little to move
    if ((long long)most * (a.row_bytes / 16) <= 1024)
        return launch_dependent(evict_move_kernel<64, 4>, move_grid, 64, 0, stream, a);
    return launch_dependent(evict_move_kernel<256, 8>, move_grid, 256, 0, stream, a);
}

}  // extern "C"
