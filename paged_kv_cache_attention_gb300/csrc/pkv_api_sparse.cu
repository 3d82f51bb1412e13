// pkv_api_sparse.cu -- the C ABI of the sparse decode step: host-side validation,
// tensor maps and kernel dispatch.  Nothing here touches device memory from the
// host or synchronises a stream.
#include <cmath>
#include <cstring>

#include "pkv_sparse.h"

namespace pkv {

namespace {

constexpr int kMaxBatch = 16384;      // prefix sums of all requests in shared memory
constexpr int kMaxTopK = 16384;
constexpr int64_t kMaxLen = 1 << 30;  // positions are 32-bit
constexpr int64_t kMaxPages = 262144;  // scores of a row in a cluster's shared memory

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

pkv_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return PKV_OK;
    return e == cudaErrorNotSupported ? PKV_ERR_UNSUPPORTED : PKV_ERR_CUDA;
}

// Pages, heads and head size that the calls of the step take.
pkv_status check_shape(int64_t num_blocks, int block_size, int num_kv_heads, int head_dim) {
    if (num_blocks <= 0 || block_size <= 0 || num_kv_heads <= 0 || head_dim <= 0)
        return PKV_ERR_INVALID_ARG;
    if (block_size != 16 && block_size != 32) return PKV_ERR_UNSUPPORTED;
    if (!head_dim_ok(head_dim)) return PKV_ERR_UNSUPPORTED;
    if (num_blocks >= (int64_t(1) << 31) / block_size ||
        num_blocks >= (int64_t(1) << 31) / num_kv_heads)
        return PKV_ERR_UNSUPPORTED;
    if ((int64_t)num_kv_heads * head_dim > (1 << 24)) return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

// Rows, requests and lists of select_pages and paged_sparse_attention.
pkv_status check_rows(const int32_t *cu_q, int batch, int rows, int num_qo_heads,
                      int num_kv_heads, int max_blocks_per_seq, int top_k) {
    if (batch < 0 || rows < 0 || num_qo_heads <= 0 || max_blocks_per_seq < 0 || top_k <= 0)
        return PKV_ERR_INVALID_ARG;
    if (num_qo_heads % num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
    if (!cu_q && rows != batch) return PKV_ERR_INVALID_ARG;
    if (num_qo_heads / num_kv_heads > 16 || top_k > kMaxTopK || rows > (1 << 24))
        return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

RowParams row_params(const int32_t *cu_q, const int32_t *seqlens, const int32_t *block_table,
                     int32_t *dev_error, int64_t num_blocks, int batch, int rows,
                     int max_blocks_per_seq, int max_seqlen, int num_qo_heads, int num_kv_heads,
                     int head_dim) {
    RowParams r;
    r.cu_q = cu_q;
    r.seqlens = seqlens;
    r.block_table = block_table;
    r.dev_error = dev_error;
    r.num_blocks = num_blocks;
    r.batch = batch;
    r.rows = rows;
    r.max_blocks_per_seq = max_blocks_per_seq;
    r.max_seqlen = max_seqlen;
    r.num_kv_heads = num_kv_heads;
    r.group = num_qo_heads / num_kv_heads;
    r.head_dim = head_dim;
    return r;
}

}  // namespace

}  // namespace pkv

using namespace pkv;

extern "C" {

pkv_status pkv_update_block_tables(int32_t *block_table, int max_blocks_per_seq,
                                   const int32_t *old_seqlens, const int32_t *new_seqlens,
                                   int batch, int32_t *free_blocks, int64_t num_blocks,
                                   int32_t *num_free, int block_size, int64_t *slot_mapping,
                                   int64_t *positions, int num_rows, int32_t *cu_seq_lens_q,
                                   int32_t *cu_seq_lens_k, int32_t *dev_error, void *stream) {
    if (batch < 0 || max_blocks_per_seq < 0 || num_blocks <= 0 || num_rows < 0 || block_size <= 0)
        return PKV_ERR_INVALID_ARG;
    if (block_size != 16 && block_size != 32) return PKV_ERR_UNSUPPORTED;
    if (batch > kMaxBatch || (int64_t)max_blocks_per_seq * block_size > kMaxLen ||
        num_blocks >= (int64_t(1) << 31) / block_size || num_rows > (1 << 30))
        return PKV_ERR_UNSUPPORTED;
    if (!free_blocks || !num_free || !cu_seq_lens_q || !cu_seq_lens_k ||
        (batch > 0 && (!old_seqlens || !new_seqlens)) ||
        (batch > 0 && max_blocks_per_seq > 0 && !block_table) ||
        (num_rows > 0 && (!slot_mapping || !positions)))
        return PKV_ERR_INVALID_ARG;
    if (!aligned(block_table, 4) || !aligned(old_seqlens, 4) || !aligned(new_seqlens, 4) ||
        !aligned(free_blocks, 4) || !aligned(num_free, 4) || !aligned(slot_mapping, 8) ||
        !aligned(positions, 8) || !aligned(cu_seq_lens_q, 4) || !aligned(cu_seq_lens_k, 4))
        return PKV_ERR_INVALID_ARG;
    TableParams p;
    p.block_table = block_table;
    p.old_len = old_seqlens;
    p.new_len = new_seqlens;
    p.free_blocks = free_blocks;
    p.num_free = num_free;
    p.slots = slot_mapping;
    p.positions = positions;
    p.cu_q = cu_seq_lens_q;
    p.cu_k = cu_seq_lens_k;
    p.dev_error = dev_error;
    p.num_blocks = num_blocks;
    p.batch = batch;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.block_size = block_size;
    p.bs_shift = block_size == 16 ? 4 : 5;
    p.rows = num_rows;
    p.rows_here = 0;
    return from_cuda(launch_block_tables(p, static_cast<cudaStream_t>(stream)));
}

pkv_status pkv_update_page_bounds(const void *k_cache, const uint8_t *k_scale,
                                  pkv_cache_desc cache, int8_t *page_bounds,
                                  uint8_t *bounds_scale, const int64_t *slot_mapping,
                                  int64_t num_tokens, int32_t *dev_error, void *stream) {
    const pkv_status st =
        check_shape(cache.num_blocks, cache.block_size, cache.num_kv_heads, cache.head_dim);
    if (st != PKV_OK) return st;
    if (cache.dtype != PKV_BF16 && cache.dtype != PKV_E4M3) return PKV_ERR_UNSUPPORTED;
    if (cache.layout != PKV_NHD && cache.layout != PKV_HND) return PKV_ERR_UNSUPPORTED;
    if (num_tokens < 0) return PKV_ERR_INVALID_ARG;
    if (num_tokens > (1 << 22)) return PKV_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PKV_OK;
    const bool fp8 = cache.dtype == PKV_E4M3;
    if (!k_cache || !page_bounds || !bounds_scale || !slot_mapping || (fp8 && !k_scale))
        return PKV_ERR_INVALID_ARG;
    if (!aligned(k_cache, 16) || !aligned(page_bounds, 16) || !aligned(slot_mapping, 8))
        return PKV_ERR_INVALID_ARG;
    BoundsParams p;
    p.k = k_cache;
    p.k_scale = fp8 ? k_scale : nullptr;
    p.bounds = page_bounds;
    p.bounds_scale = bounds_scale;
    p.slots = slot_mapping;
    p.num_tokens = num_tokens;
    p.capacity = cache.num_blocks * (int64_t)cache.block_size;
    p.dev_error = dev_error;
    p.num_kv_heads = cache.num_kv_heads;
    p.head_dim = cache.head_dim;
    p.block_size = cache.block_size;
    p.bs_shift = cache.block_size == 16 ? 4 : 5;
    p.hnd = cache.layout == PKV_HND ? 1 : 0;
    p.tokens_per_warp = p.heads_per_warp = 0;
    return from_cuda(launch_page_bounds(p, static_cast<cudaStream_t>(stream)));
}

pkv_status pkv_select_pages(int32_t *pages, int top_k, const void *q, const int8_t *page_bounds,
                            const uint8_t *bounds_scale, int64_t num_blocks, int block_size,
                            int num_kv_heads, int head_dim, const int32_t *block_table,
                            int max_blocks_per_seq, const int32_t *cache_seqlens, int max_seqlen,
                            const int32_t *cu_seq_lens_q, int batch, int total_q,
                            int num_qo_heads, int num_first, int num_recent, int32_t *dev_error,
                            void *stream) {
    pkv_status st = check_shape(num_blocks, block_size, num_kv_heads, head_dim);
    if (st != PKV_OK) return st;
    st = check_rows(cu_seq_lens_q, batch, total_q, num_qo_heads, num_kv_heads, max_blocks_per_seq,
                    top_k);
    if (st != PKV_OK) return st;
    if (max_seqlen < 0 || num_first < 0 || num_recent < 1 ||
        (int64_t)num_first + num_recent > top_k)
        return PKV_ERR_INVALID_ARG;
    if (max_seqlen > kMaxPages * (int64_t)block_size) return PKV_ERR_UNSUPPORTED;
    if (batch == 0 || total_q == 0) return PKV_OK;
    if (max_blocks_per_seq == 0) return PKV_ERR_INVALID_ARG;
    if (!pages || !q || !page_bounds || !bounds_scale || !block_table || !cache_seqlens)
        return PKV_ERR_INVALID_ARG;
    if (!aligned(pages, 4) || !aligned(q, 16) || !aligned(page_bounds, 16) ||
        !aligned(block_table, 4) || !aligned(cache_seqlens, 4) || !aligned(cu_seq_lens_q, 4))
        return PKV_ERR_INVALID_ARG;
    SelectParams p;
    p.r = row_params(cu_seq_lens_q, cache_seqlens, block_table, dev_error, num_blocks, batch,
                     total_q, max_blocks_per_seq, max_seqlen, num_qo_heads, num_kv_heads,
                     head_dim);
    p.q = q;
    p.bounds = page_bounds;
    p.bounds_scale = bounds_scale;
    p.pages = pages;
    p.top_k = top_k;
    p.num_first = num_first;
    p.num_recent = num_recent;
    p.block_size = block_size;
    p.bs_shift = block_size == 16 ? 4 : 5;
    p.cluster = p.cap = 0;
    return from_cuda(launch_select_pages(p, static_cast<cudaStream_t>(stream)));
}

pkv_status pkv_paged_sparse_attention(void *out, const void *q, const void *k_cache,
                                      const void *v_cache, const uint8_t *k_scale,
                                      const uint8_t *v_scale, pkv_cache_desc cache,
                                      const int32_t *block_table, int max_blocks_per_seq,
                                      const int32_t *cache_seqlens,
                                      const int32_t *cu_seq_lens_q, int batch, int total_q,
                                      const int32_t *pages, int top_k, const float *sink,
                                      int num_qo_heads, float sm_scale, float *lse_out,
                                      int32_t *dev_error, void *stream) {
    pkv_status st =
        check_shape(cache.num_blocks, cache.block_size, cache.num_kv_heads, cache.head_dim);
    if (st != PKV_OK) return st;
    if (cache.dtype != PKV_BF16 && cache.dtype != PKV_E4M3) return PKV_ERR_UNSUPPORTED;
    if (cache.layout != PKV_NHD && cache.layout != PKV_HND) return PKV_ERR_UNSUPPORTED;
    st = check_rows(cu_seq_lens_q, batch, total_q, num_qo_heads, cache.num_kv_heads,
                    max_blocks_per_seq, top_k);
    if (st != PKV_OK) return st;
    if (!std::isfinite(sm_scale)) return PKV_ERR_INVALID_ARG;
    if (batch == 0 || total_q == 0) return PKV_OK;
    if (max_blocks_per_seq == 0) return PKV_ERR_INVALID_ARG;
    const bool fp8 = cache.dtype == PKV_E4M3;
    if (!out || !q || !k_cache || !v_cache || !block_table || !cache_seqlens || !pages ||
        (fp8 && (!k_scale || !v_scale)))
        return PKV_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(block_table, 4) || !aligned(cache_seqlens, 4) || !aligned(cu_seq_lens_q, 4) ||
        !aligned(pages, 4) || !aligned(sink, 4) || !aligned(lse_out, 4) ||
        (fp8 && (!aligned(k_scale, 16) || !aligned(v_scale, 16))))
        return PKV_ERR_INVALID_ARG;
    SparseParams p;
    std::memset(&p, 0, sizeof p);
    p.r = row_params(cu_seq_lens_q, cache_seqlens, block_table, dev_error, cache.num_blocks,
                     batch, total_q, max_blocks_per_seq, (int)kMaxLen, num_qo_heads,
                     cache.num_kv_heads, cache.head_dim);
    p.q = q;
    p.out = out;
    p.pages = pages;
    p.sink = sink;
    p.lse_out = lse_out;
    p.k_scale = fp8 ? k_scale : nullptr;
    p.v_scale = fp8 ? v_scale : nullptr;
    p.top_k = top_k;
    p.hnd = cache.layout == PKV_HND ? 1 : 0;
    p.scale_log2 = sm_scale * 1.4426950408889634f;
    // As many CTAs per row and kv head as run at once, of at least 128 keys (8 kv heads,
    // 1024 keys: 8 rows 27.7 us in one CTA each, 9.7 in eight; 16 rows 28 and 14.5 in
    // four; 64 rows 46 and 61 in eight).
    const int64_t units = (int64_t)total_q * cache.num_kv_heads;
    int c = 1;
    while (c < 8 && units * c < 3LL * device_sm_count() &&
           (int64_t)top_k * cache.block_size / c >= 256)
        c *= 2;
    p.cluster = c;
    p.cap = (top_k + c - 1) / c;
    alignas(64) CUtensorMap tk, tv;
    const int rows = fp8 ? decode_fp8_box_rows(cache.head_dim, cache.block_size) : cache.block_size;
    if ((st = pool_map(&tk, k_cache, cache, rows)) != PKV_OK) return st;
    if ((st = pool_map(&tv, v_cache, cache, rows)) != PKV_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    // Chunks: tiles of 128 rows, where requests have 8 queries and fill a quarter of a tile on
    // average and rows would take all SMs a few rounds.  In tiles and row by row, 8 kv heads,
    // 1024 keys a query and no two lists alike (the less they differ, the better tiles
    // do): 16 requests, groups of 4 heads, 4 queries 52 and 32 us, 8 69 and 62, 16 84 and
    // 94, 64 117 and 289; groups of one, 32 queries 101 and 154; 1 request, 64 queries 67
    // and 30, 128 68 and 61, 256 68 and 92.  That was over 32K tokens and less: beyond, the
    // lists differ more and their windows are more, which the rule does not know (256 queries
    // of one request, 8 kv heads, 64 pages a query, groups of 4 and of one: 32K tokens 97 and
    // 170 us in tiles, 256K 196 and 539, 1M 363 and 1441; 115 to 118 row by row in all).
    if (!fp8 && cu_seq_lens_q && total_q >= 8LL * batch &&
        (int64_t)total_q * p.r.group >= 32LL * batch && units > 12LL * device_sm_count()) {
        bool fits = false;
        const cudaError_t e =
            launch_sparse_tile(p, fits, cache.block_size, k_cache, v_cache, &tk, &tv, s);
        if (fits) return from_cuda(e);
    }
    return from_cuda(fp8 ? launch_sparse_fp8(p, cache.block_size, &tk, &tv, s)
                         : launch_sparse(p, cache.block_size, &tk, &tv, s));
}

}  // extern "C"
