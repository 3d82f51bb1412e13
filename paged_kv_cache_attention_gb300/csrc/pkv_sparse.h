// pkv_sparse.h -- parameter blocks and launchers of the sparse decode step (block
// tables from lengths, page bounds, page selection, attention over lists of
// pages), shared by pkv_api_sparse.cu and the kernels.
#pragma once

#include "pkv_fp8.h"

namespace pkv {

struct TableParams {
    int32_t *block_table;          // [B, max_blocks_per_seq], in and out
    const int32_t *old_len, *new_len;  // [B]
    int32_t *free_blocks;          // [num_blocks] a stack, in and out
    int32_t *num_free;             // its height, in and out
    int64_t *slots, *positions;    // [rows]
    int32_t *cu_q, *cu_k;          // [B + 1]
    int32_t *dev_error;
    int64_t num_blocks;
    int batch, max_blocks_per_seq, block_size, bs_shift;
    int rows;
    int rows_here;                 // the table kernel writes the rows itself
};

struct BoundsParams {
    const void *k;                 // the pool
    const uint8_t *k_scale;        // nullptr: bf16
    int8_t *bounds;                // [num_blocks, Hkv, 2, D]
    uint8_t *bounds_scale;         // [num_blocks, Hkv]
    const int64_t *slots;          // [T]
    int64_t num_tokens, capacity;
    int32_t *dev_error;
    int num_kv_heads, head_dim, block_size, bs_shift, hnd;
    int tokens_per_warp, heads_per_warp;
};

// What the calls with a row per query share: which request and how many keys a
// row has (pkv_sparse.cuh).
struct RowParams {
    const int32_t *cu_q;           // [B + 1], or nullptr: row = request
    const int32_t *seqlens;        // [B]
    const int32_t *block_table;    // [B, max_blocks_per_seq]
    int32_t *dev_error;
    int64_t num_blocks;
    int batch, rows, max_blocks_per_seq, max_seqlen;
    int num_kv_heads, group, head_dim;
};

// Tiles of `queries` rows that cover all rows (tile_rows).
constexpr int kTiledRequests = 256;
inline int64_t row_tiles(const RowParams &r, int queries) {
    const int64_t tiles = ((int64_t)r.rows + queries - 1) / queries;
    return r.batch > kTiledRequests ? tiles : tiles + (r.batch < r.rows ? r.batch : r.rows);
}

struct SelectParams {
    RowParams r;
    const void *q;                 // [rows, Hq, D] bf16
    const int8_t *bounds;
    const uint8_t *bounds_scale;
    int32_t *pages;                // [rows, Hkv, top_k]
    int top_k, num_first, num_recent, block_size, bs_shift;
    int cluster;                   // CTAs per tile of queries and kv head
    int cap;                       // pages a CTA has room for
};

struct SparseParams {
    RowParams r;
    const void *q;                 // [rows, Hq, D] bf16
    void *out;
    const int32_t *pages;          // [rows, Hkv, top_k]
    const float *sink;             // [Hq] or nullptr
    float *lse_out;                // [rows, Hq] or nullptr
    const uint8_t *k_scale, *v_scale;
    int top_k, hnd;
    int cluster;                   // CTAs per row and kv head
    int cap;                       // list entries a CTA has room for
    int words, group_shift;        // tiles of queries: see sparse_tile.cu
    float scale_log2;
};

cudaError_t launch_block_tables(const TableParams &p, cudaStream_t stream);
cudaError_t launch_page_bounds(const BoundsParams &p, cudaStream_t stream);
cudaError_t launch_select_pages(const SelectParams &p, cudaStream_t stream);
cudaError_t launch_sparse(const SparseParams &p, int block_size, const CUtensorMap *tmap_k,
                          const CUtensorMap *tmap_v, cudaStream_t stream);
// Tiles of queries; fits: whether there is a kernel for the shape (else nothing is done).
cudaError_t launch_sparse_tile(const SparseParams &p, bool &fits, int block_size,
                               const void *k_cache, const void *v_cache, const CUtensorMap *tmap_k,
                               const CUtensorMap *tmap_v, cudaStream_t stream);
cudaError_t launch_sparse_fp8(const SparseParams &p, int block_size, const CUtensorMap *tmap_k,
                              const CUtensorMap *tmap_v, cudaStream_t stream);

// Lets `kernel` be launched with clusters of up to 16 CTAs on the current device,
// once per (kernel, device).
cudaError_t ensure_wide_clusters(const void *kernel);

// Launch with clusters of `cluster` CTAs along x (and launch_pdl's attribute).
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), unsigned grid, int cluster, unsigned block,
                           size_t smem, cudaStream_t stream, Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args &&>(args)...);
}

}  // namespace pkv
