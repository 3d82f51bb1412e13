// pkv_fp8.h -- parameter blocks and launchers of the 8-bit cache, the tree
// attention and the fused q/k norm, shared by pkv_api_fp8.cu and the kernels.
#pragma once

#include "pkv_internal.h"

namespace pkv {

// The two pools of a cache write or read-back.  k_scale == nullptr: pools of
// the rows' own dtype; otherwise e4m3 codes with one E8M0 byte per (token, kv
// head), [num_blocks, Hkv, block_size].
struct PoolArgs {
    void *k, *v;
    uint8_t *k_scale, *v_scale;
    int64_t capacity;    // num_blocks * block_size
    int num_kv_heads, head_dim, block_size;
    int bs_shift;        // log2(block_size)
    int hnd;
};

struct QuantWriteParams {
    const void *key, *value;       // [T, Hkv, D], rows of a token contiguous
    int64_t key_stride, value_stride;  // elements between tokens
    const int64_t *slot_mapping;   // [T]
    int64_t num_tokens;
    int32_t *dev_error;
    PoolArgs pool;
};

struct GatherParams {
    void *key, *value;             // [total_k, Hkv, D] bf16
    const int32_t *block_table;    // [B, max_blocks_per_seq]
    const int32_t *cu_k;           // [B + 1]
    int32_t *dev_error;
    int64_t num_blocks;
    int batch, max_blocks_per_seq, total_k;
    PoolArgs pool;
};

struct NormRopeParams {
    const void *query, *key, *value;
    void *query_out, *key_out;
    int64_t q_stride, k_stride, v_stride, qo_stride, ko_stride;  // elements between tokens
    const void *q_weight, *k_weight;   // [D]
    int weight_f32;                    // weights are fp32 (else the rows' dtype)
    const int64_t *positions, *slot_mapping;
    const float2 *cos_sin;
    int64_t num_tokens, max_position;
    int num_qo_heads, rotary_dim, neox;
    float eps;
    int32_t *dev_error;
    PoolArgs pool;
};

// decode over e4m3 pools: the fields of the bf16 decode, plus the scales
struct DecodeFp8Params {
    DecodeParams d;
    const uint8_t *k_scale, *v_scale;
};

// Attention of up to 256 drafted tokens per request over the pools.
struct TreeParams {
    const void *q;                 // [total_q, Hq, D] bf16
    void *out;
    const int32_t *block_table;    // [B, max_blocks_per_seq]
    const int32_t *cu_q;           // [B + 1]
    const int32_t *seqlens;        // [B]: context and drafted tokens
    const int64_t *mask;           // [total_q, mask_words]
    const int32_t *depth;          // [total_q] or nullptr
    const float *sink, *alibi;
    float *lse_out;                // [total_q, Hq] or nullptr
    long long *line;               // [B + 1] the requests' places on the line of work,
                                   // and a CTA group's share of it (tree.cu)
    float *part_lse;               // [2 * groups, Hkv, rows of a row group] (log2 units)
    float *part_o;                 // the same with [D / 4, rows, 4]
    int32_t *dev_error;
    const uint8_t *k_scale, *v_scale;
    int64_t num_blocks;
    int batch, num_qo_heads, num_kv_heads, group;
    int max_blocks_per_seq, max_seqlen, max_seqlen_q, total_q;
    int mask_words, window_left, head_dim, hnd, block_size;
    int groups;                    // CTA groups of num_kv_heads CTAs
    int min_tiles;                 // least key tiles of a group's share
    int row_tiles;                 // 128-row tiles of the largest request
    float scale_log2;
};

// cuTensorMapEncodeTiled of a 3-D view (pkv_api.cu).
pkv_status encode_map_3d(CUtensorMap *map, CUtensorMapDataType type, const void *base,
                         const cuuint64_t (&dims)[3], const cuuint64_t (&strides)[2],
                         const cuuint32_t (&box)[3], CUtensorMapSwizzle swizzle);

// The head sizes of the 8-bit cache and of the calls over both kinds of pools.
bool head_dim_ok(int d);

// Tensor map of a pool (bf16 or e4m3) with boxes of 128 bytes (64 for the codes of a
// 64-dim head) of box_rows tokens of one (page, kv head) (pkv_api_fp8.cu).
pkv_status pool_map(CUtensorMap *map, const void *base, const pkv_cache_desc &c, int box_rows);

cudaError_t launch_quant_write(const QuantWriteParams &p, int dtype, cudaStream_t stream);
cudaError_t launch_gather(const GatherParams &p, cudaStream_t stream);
cudaError_t launch_norm_rope(const NormRopeParams &p, int dtype, cudaStream_t stream);
// Tokens of a page that one box of the decode's tensor maps holds.
int decode_fp8_box_rows(int head_dim, int block_size);
cudaError_t launch_decode_fp8(const DecodeFp8Params &p, const pkv_cache_desc &cache,
                              const CUtensorMap *tmap_k, const CUtensorMap *tmap_v,
                              cudaStream_t stream);
cudaError_t launch_tree(const TreeParams &p, const CUtensorMap *tmap_k,
                        const CUtensorMap *tmap_v, cudaStream_t stream);

}  // namespace pkv
