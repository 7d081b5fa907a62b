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

// A launch as clusters of `cs` consecutive CTAs along x.
template <typename K, typename A>
pa_status launch_cluster(K kernel, const A &args, dim3 grid, int threads, int cs, size_t smem,
                         cudaStream_t st) {
    if (set_smem(kernel, smem) != cudaSuccess) return PA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cs;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = st;
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    if (cudaLaunchKernelEx(&cfg, kernel, args) != cudaSuccess) {
        cudaGetLastError();
        return PA_ERR_CUDA;
    }
    return launch_status();
}

constexpr int kSelectSegment = 24576;  // blocks one CTA of a cluster can score

// CTAs of a row's cluster: enough for every SM when there are few rows, as
// long as a CTA keeps `grain` items of the longest row or more.
int cluster_size(long long rows, long long items, int grain) {
    int cs = 1;
    while (cs < kMaxCluster && rows * cs < 148 && items > (long long)cs * grain) cs *= 2;
    return cs;
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

pa_status pa_select_blocks(int32_t *selected, const void *q, const void *key_bounds,
                           const int32_t *block_tables, const int32_t *context_lens,
                           int max_selected, int num_first, int num_last, int num_seqs,
                           int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                           int num_blocks, int max_blocks_per_seq, int max_context_len,
                           pa_dtype dtype, cudaStream_t stream) {
    const pa_status st = check_cache_shape(num_seqs, num_kv_heads, head_dim, block_size,
                                           num_blocks, max_blocks_per_seq, dtype);
    if (st != PA_OK) return st;
    if (num_q_heads <= 0 || max_context_len < 0 || max_selected <= 0 || num_first < 0 ||
        num_last < 0 || (long long)num_first + num_last > max_selected)
        return PA_ERR_INVALID_ARG;
    if (num_q_heads % num_kv_heads != 0) return PA_ERR_UNSUPPORTED;
    if ((long long)max_context_len > (long long)max_blocks_per_seq * block_size)
        return PA_ERR_INVALID_ARG;
    const long long blocks = ((long long)max_context_len + block_size - 1) / block_size;
    if (blocks > (long long)kMaxCluster * kSelectSegment) return PA_ERR_UNSUPPORTED;
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
    int cs = cluster_size((long long)num_seqs * num_kv_heads, blocks, 64);
    while (blocks > (long long)cs * kSelectSegment) cs *= 2;
    const size_t smem = (size_t)(blocks + cs - 1) / cs * 8 + 8;
    const dim3 grid((unsigned)cs, (unsigned)num_kv_heads, (unsigned)num_seqs);
    if (dtype == PA_BF16)
        return head_dim == 128 ? launch_cluster(select_blocks_kernel<128, __nv_bfloat16>, a, grid,
                                                kSelThreads, cs, smem, stream)
                               : launch_cluster(select_blocks_kernel<64, __nv_bfloat16>, a, grid,
                                                kSelThreads, cs, smem, stream);
    return head_dim == 128 ? launch_cluster(select_blocks_kernel<128, float>, a, grid, kSelThreads,
                                            cs, smem, stream)
                           : launch_cluster(select_blocks_kernel<64, float>, a, grid, kSelThreads,
                                            cs, smem, stream);
}

}  // extern "C"
