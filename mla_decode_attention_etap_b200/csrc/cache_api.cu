// C ABI of the steps around the decode (declared in include/mla_decode.h): mla_cache_extend,
// mla_cache_append(_fp8) and mla_cache_accept.  Arguments are validated on the host before anything is
// launched; no call allocates memory or synchronises the host.
#include <cuda_runtime.h>

#include <cmath>

#include "mla_decode.h"
#include "api_common.h"
#include "cache_kernels.cuh"

namespace {

using mla::is_aligned;

int launched(cudaError_t e, const char *what) {
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? MLA_OK : mla::record_cuda_error(e, what);
}

// Sizes of a cache and its table, shared by the calls that walk one.
int check_cache(const int32_t *block_table, int batch, int64_t kv_rows, int max_blocks) {
    if (kv_rows < 1) return MLA_ERR_INVALID_ARG;
    if (block_table) {
        if (kv_rows % MLA_PAGE_SIZE != 0 || max_blocks < 1) return MLA_ERR_INVALID_ARG;
        if (kv_rows > INT32_MAX || (int64_t)max_blocks * MLA_PAGE_SIZE > INT32_MAX) return MLA_ERR_UNSUPPORTED;
    } else if ((int64_t)batch * kv_rows > INT32_MAX) {
        return MLA_ERR_UNSUPPORTED;
    }
    return MLA_OK;
}

// Tokens per CTA of the extend kernel's cluster before the next CTA is added.
constexpr int64_t kExtendTokensPerCta = 4096;
// More tokens than the largest cluster has threads: four a thread instead of one.
constexpr int64_t kExtendManyTokens = 8 * mla::kCacheThreads;
// Warps that the largest accept cluster (8 CTAs, one of them for the pages) has for rows.
constexpr int kAcceptClusterWarps = 7 * mla::kCacheThreads / 32;

int append(const void *latent, int64_t latent_stride, const void *norm_weight, float eps, const float *rope_table,
           int max_pos, int interleaved, const int32_t *positions, const int32_t *slots, int tokens, void *kv,
           uint8_t *kv8, float *kv_scale, int64_t cache_rows, const void *q_rope, int64_t q_token_stride,
           int64_t q_head_stride, int num_heads, void *q, int32_t *status, void *stream) {
    const bool fp8 = kv8 != nullptr;
    if (tokens < 0 || max_pos < 1 || cache_rows < 1) return MLA_ERR_INVALID_ARG;
    if (tokens > 0 && (!latent || !positions || !slots)) return MLA_ERR_INVALID_ARG;
    if (!rope_table || !status) return MLA_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return MLA_ERR_INVALID_ARG;
    if (interleaved != 0 && interleaved != 1) return MLA_ERR_INVALID_ARG;
    if (latent_stride < MLA_D_QK && tokens > 1) return MLA_ERR_INVALID_ARG;
    if (tokens > 0 && (q_rope == nullptr) != (q == nullptr)) return MLA_ERR_INVALID_ARG;
    if (q && (num_heads < 1 || q_token_stride < 0 || q_head_stride < 0)) return MLA_ERR_INVALID_ARG;
    if (cache_rows > INT32_MAX || (q && num_heads > MLA_MAX_COLUMNS)) return MLA_ERR_UNSUPPORTED;
    if (latent_stride % 8 != 0 || !is_aligned(latent, 16) || !is_aligned(norm_weight, 16) ||
        !is_aligned(rope_table, 16) || !is_aligned(kv, 16) || !is_aligned(kv8, 16) || !is_aligned(kv_scale, 4) ||
        !is_aligned(positions, 4) || !is_aligned(slots, 4) || !is_aligned(status, 4))
        return MLA_ERR_ALIGNMENT;
    if (q && (q_token_stride % 8 != 0 || q_head_stride % 8 != 0 || !is_aligned(q_rope, 16) || !is_aligned(q, 16)))
        return MLA_ERR_ALIGNMENT;
    if (tokens == 0) return MLA_OK;
    mla::AppendParams p{};
    p.latent = reinterpret_cast<const __nv_bfloat16 *>(latent);
    p.norm_weight = reinterpret_cast<const __nv_bfloat16 *>(norm_weight);
    p.rope_table = rope_table;
    p.positions = positions;
    p.slots = slots;
    p.kv = reinterpret_cast<__nv_bfloat16 *>(kv);
    p.kv8 = kv8;
    p.kv_scale = kv_scale;
    p.q_rope = reinterpret_cast<const __nv_bfloat16 *>(q_rope);
    p.q = reinterpret_cast<__nv_bfloat16 *>(q);
    p.status = status;
    p.row_stride = latent_stride;
    p.q_token_stride = q_token_stride;
    p.q_head_stride = q_head_stride;
    p.cache_rows = cache_rows;
    p.tokens = tokens;
    p.heads = q ? num_heads : 0;
    p.max_pos = max_pos;
    p.eps = eps;
    const int64_t warps = mla::kAppendThreads / 32;
    const int64_t groups = (p.heads + mla::kQueryHeads - 1) / mla::kQueryHeads;
    const int64_t rows = ((int64_t)tokens + warps - 1) / warps;
    const int64_t blocks = rows + ((int64_t)tokens * groups * 4 + mla::kAppendThreads - 1) / mla::kAppendThreads;
    if (blocks > INT32_MAX) return MLA_ERR_UNSUPPORTED;
    p.key_blocks = (int)rows;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto kernel = fp8 ? (interleaved ? mla::append_kernel<true, true> : mla::append_kernel<true, false>)
                      : (interleaved ? mla::append_kernel<false, true> : mla::append_kernel<false, false>);
    kernel<<<(unsigned)blocks, mla::kAppendThreads, 0, s>>>(p);
    return launched(cudaSuccess, "append_kernel launch");
}

}  // namespace

extern "C" {

int mla_cache_extend(const int32_t *seqlens, const int32_t *new_lens, const int32_t *parents, int batch, int q_len,
                     int32_t *block_table, int max_blocks, const int32_t *free_pages, int free_capacity,
                     const int32_t *num_free, int64_t kv_rows, int32_t *slots, int32_t *positions, int32_t *tree_mask,
                     int32_t *seqlens_out, int32_t *num_free_out, int32_t *status, void *stream) {
    if (batch < 1 || batch > MLA_MAX_BATCH || q_len < 1) return MLA_ERR_INVALID_ARG;
    if (!seqlens || !slots || !positions || !seqlens_out || !status) return MLA_ERR_INVALID_ARG;
    if ((parents == nullptr) != (tree_mask == nullptr)) return MLA_ERR_INVALID_ARG;
    if ((int64_t)batch * q_len > INT32_MAX || (parents && q_len > MLA_MAX_COLUMNS)) return MLA_ERR_UNSUPPORTED;
    const int st = check_cache(block_table, batch, kv_rows, max_blocks);
    if (st != MLA_OK) return st;
    if (block_table && ((!free_pages && free_capacity != 0) || !num_free || !num_free_out || free_capacity < 0))
        return MLA_ERR_INVALID_ARG;
    if (!is_aligned(seqlens, 4) || !is_aligned(new_lens, 4) || !is_aligned(parents, 4) || !is_aligned(block_table, 4) ||
        !is_aligned(free_pages, 4) || !is_aligned(num_free, 4) || !is_aligned(slots, 4) || !is_aligned(positions, 4) ||
        !is_aligned(tree_mask, 4) || !is_aligned(seqlens_out, 4) || !is_aligned(num_free_out, 4) ||
        !is_aligned(status, 4))
        return MLA_ERR_ALIGNMENT;
    mla::ExtendParams p{};
    p.seqlens = seqlens;
    p.new_lens = new_lens;
    p.parents = parents;
    p.block_table = block_table;
    p.free_pages = free_pages;
    p.num_free = num_free;
    p.slots = slots;
    p.positions = positions;
    p.tree_mask = tree_mask;
    p.seqlens_out = seqlens_out;
    p.num_free_out = num_free_out;
    p.status = status;
    p.kv_rows = kv_rows;
    p.batch = batch;
    p.q_len = q_len;
    p.max_blocks = max_blocks;
    p.free_capacity = free_capacity;
    p.tree_words = (q_len + 31) / 32;
    p.vector_out = q_len % 4 == 0 && is_aligned(slots, 16) && is_aligned(positions, 16);
    int ctas = 1;
    while (ctas < 8 && (int64_t)batch * q_len > ctas * kExtendTokensPerCta) ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, 1, 1);
    cfg.blockDim = dim3(mla::kCacheThreads, 1, 1);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const bool many = (int64_t)batch * q_len > kExtendManyTokens;
    return launched(cudaLaunchKernelEx(&cfg, many ? mla::extend_kernel<4> : mla::extend_kernel<1>, p),
                    "extend_kernel launch");
}

int mla_cache_append(const void *latent, int64_t latent_stride, const void *norm_weight, float eps,
                     const float *rope_table, int max_pos, int interleaved, const int32_t *positions,
                     const int32_t *slots, int tokens, void *kv, int64_t cache_rows, const void *q_rope,
                     int64_t q_token_stride, int64_t q_head_stride, int num_heads, void *q, int32_t *status,
                     void *stream) {
    if (!kv) return MLA_ERR_INVALID_ARG;
    return append(latent, latent_stride, norm_weight, eps, rope_table, max_pos, interleaved, positions, slots, tokens,
                  kv, nullptr, nullptr, cache_rows, q_rope, q_token_stride, q_head_stride, num_heads, q, status,
                  stream);
}

int mla_cache_append_fp8(const void *latent, int64_t latent_stride, const void *norm_weight, float eps,
                         const float *rope_table, int max_pos, int interleaved, const int32_t *positions,
                         const int32_t *slots, int tokens, void *kv8, float *kv_scale, int64_t cache_rows,
                         const void *q_rope, int64_t q_token_stride, int64_t q_head_stride, int num_heads, void *q,
                         int32_t *status, void *stream) {
    if (!kv8 || !kv_scale) return MLA_ERR_INVALID_ARG;
    return append(latent, latent_stride, norm_weight, eps, rope_table, max_pos, interleaved, positions, slots, tokens,
                  nullptr, reinterpret_cast<uint8_t *>(kv8), kv_scale, cache_rows, q_rope, q_token_stride,
                  q_head_stride, num_heads, q, status, stream);
}

int mla_cache_accept(void *kv, float *kv_scale, const int32_t *seqlens, const int32_t *new_lens, const int32_t *path,
                     const int32_t *path_lens, int batch, int q_len, int max_path, const int32_t *block_table,
                     int max_blocks, int32_t *free_pages, int free_capacity, const int32_t *num_free, int64_t kv_rows,
                     int32_t *seqlens_out, int32_t *num_free_out, int32_t *status, void *stream) {
    if (batch < 1 || batch > MLA_MAX_BATCH || q_len < 1 || max_path < 1) return MLA_ERR_INVALID_ARG;
    if (!kv || !seqlens || !new_lens || !path || !path_lens || !seqlens_out || !status) return MLA_ERR_INVALID_ARG;
    const int st = check_cache(block_table, batch, kv_rows, max_blocks);
    if (st != MLA_OK) return st;
    if (block_table && ((!free_pages && free_capacity != 0) || !num_free || !num_free_out || free_capacity < 0))
        return MLA_ERR_INVALID_ARG;
    if (!is_aligned(kv, 16) || !is_aligned(kv_scale, 4) || !is_aligned(seqlens, 4) || !is_aligned(new_lens, 4) ||
        !is_aligned(path, 4) || !is_aligned(path_lens, 4) || !is_aligned(block_table, 4) ||
        !is_aligned(free_pages, 4) || !is_aligned(num_free, 4) || !is_aligned(seqlens_out, 4) ||
        !is_aligned(num_free_out, 4) || !is_aligned(status, 4))
        return MLA_ERR_ALIGNMENT;
    mla::AcceptParams p{};
    p.kv = kv;
    p.kv_scale = kv_scale;
    p.seqlens = seqlens;
    p.new_lens = new_lens;
    p.path = path;
    p.path_lens = path_lens;
    p.block_table = block_table;
    p.free_pages = free_pages;
    p.num_free = num_free;
    p.seqlens_out = seqlens_out;
    p.num_free_out = num_free_out;
    p.status = status;
    p.kv_rows = kv_rows;
    p.batch = batch;
    p.q_len = q_len;
    p.max_path = max_path;
    p.max_blocks = max_blocks;
    p.free_capacity = free_capacity;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool fp8 = kv_scale != nullptr;
    const int items = batch * (fp8 ? mla::kAcceptSlices<true> : mla::kAcceptSlices<false>);
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(mla::kCacheThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (items <= kAcceptClusterWarps) {
        int ctas = 2;
        while ((ctas - 1) * (mla::kCacheThreads / 32) < items) ctas *= 2;
        cfg.gridDim = dim3(ctas, 1, 1);
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = ctas;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        return launched(cudaLaunchKernelEx(&cfg, fp8 ? mla::accept_kernel<true> : mla::accept_kernel<false>, p),
                        "accept_kernel launch");
    }
    const unsigned blocks = (items + mla::kAcceptThreads / 32 - 1) / (mla::kAcceptThreads / 32);
    if (fp8)
        mla::accept_rows_kernel<true><<<blocks, mla::kAcceptThreads, 0, s>>>(p);
    else
        mla::accept_rows_kernel<false><<<blocks, mla::kAcceptThreads, 0, s>>>(p);
    const int rc = launched(cudaSuccess, "accept_rows_kernel launch");
    if (rc != MLA_OK) return rc;
    cfg.gridDim = dim3(1, 1, 1);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    return launched(cudaLaunchKernelEx(&cfg, mla::accept_pages_kernel, p), "accept_pages_kernel launch");
}

}  // extern "C"
