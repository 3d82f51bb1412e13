// pkv_api_fp8.cu -- the C ABI of the 8-bit cache, the tree attention and the
// fused q/k norm: host-side validation, workspace sizing, tensor maps and
// kernel dispatch.  Nothing here touches device memory from the host or
// synchronises a stream.
#include <cmath>
#include <cstring>

#include "pkv_fp8.h"

namespace pkv {

bool head_dim_ok(int d) {
    return d == 64 || d == 80 || d == 96 || d == 112 || d == 128 || d == 256;
}

// TMA view of one pool whose box is 128 bytes (64 for the codes of a 64-dim
// head) of box_rows tokens of one (page, kv head): NHD {D, Hkv, num_blocks *
// bs}, HND {D, bs, num_blocks * Hkv}.
pkv_status pool_map(CUtensorMap *map, const void *base, const pkv_cache_desc &c, int box_rows) {
    const bool fp8 = c.dtype == PKV_E4M3;
    const cuuint64_t e = fp8 ? 1 : 2, D = (cuuint64_t)c.head_dim;
    const cuuint32_t bs = (cuuint32_t)box_rows;
    const bool nhd = c.layout == PKV_NHD;
    const cuuint64_t mid = nhd ? c.num_kv_heads : c.block_size;
    const cuuint64_t rows = (cuuint64_t)c.num_blocks * (nhd ? c.block_size : c.num_kv_heads);
    const cuuint64_t dims[3] = {D, mid, rows};
    const cuuint64_t strides[2] = {D * e, D * e * mid};
    const cuuint32_t w = fp8 ? (D == 64 ? 64 : 128) : 64;
    const cuuint32_t box[3] = {w, nhd ? 1u : bs, nhd ? bs : 1u};
    return encode_map_3d(map,
                         fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                         base, dims, strides, box,
                         w * e == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

namespace {

constexpr int kDefaultPartition = 512;
constexpr int kMaxPartition = 16384;
constexpr int kMaxAutoPartition = 1536;
// CTAs of the 8-bit decode that run at once: 6 per SM with heads up to 128 and up to
// 8 of them per kv head, which the rule below was measured with (else 3 to 5)
constexpr int kDecodeSlots = 912;

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

pkv_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return PKV_OK;
    return e == cudaErrorNotSupported ? PKV_ERR_UNSUPPORTED : PKV_ERR_CUDA;
}

// The shape of a pool and its dtype (one of the two given).
pkv_status check_pool(const pkv_cache_desc &c, bool fp8, bool same) {
    if (c.num_blocks <= 0 || c.block_size <= 0 || c.num_kv_heads <= 0 || c.head_dim <= 0)
        return PKV_ERR_INVALID_ARG;
    if (!((fp8 && c.dtype == PKV_E4M3) ||
          (same && (c.dtype == PKV_BF16 || c.dtype == PKV_F32))))
        return PKV_ERR_UNSUPPORTED;
    if (c.layout != PKV_NHD && c.layout != PKV_HND) return PKV_ERR_UNSUPPORTED;
    if (!head_dim_ok(c.head_dim)) return PKV_ERR_UNSUPPORTED;
    if (c.block_size != 16 && c.block_size != 32) return PKV_ERR_UNSUPPORTED;
    if (c.num_blocks >= (int64_t(1) << 31) / c.block_size ||
        c.num_blocks >= (int64_t(1) << 31) / c.num_kv_heads)
        return PKV_ERR_UNSUPPORTED;
    if ((int64_t)c.num_kv_heads * c.head_dim > (1 << 24)) return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

PoolArgs pool_args(const pkv_cache_desc &c, const void *k, const void *v, const void *ks,
                   const void *vs) {
    PoolArgs a;
    a.k = const_cast<void *>(k);
    a.v = const_cast<void *>(v);
    a.k_scale = static_cast<uint8_t *>(const_cast<void *>(ks));
    a.v_scale = static_cast<uint8_t *>(const_cast<void *>(vs));
    a.capacity = c.num_blocks * (int64_t)c.block_size;
    a.num_kv_heads = c.num_kv_heads;
    a.head_dim = c.head_dim;
    a.block_size = c.block_size;
    a.bs_shift = c.block_size == 16 ? 4 : 5;
    a.hnd = c.layout == PKV_HND ? 1 : 0;
    return a;
}

// Workspace of the tree attention: the line of work, and two partials per CTA.
// CTAs: groups of one per kv head on kTreeSms SMs.  A fixed count, so that the
// workspace of a problem does not depend on the device.
constexpr int kTreeTile = 128, kMaxDraft = 256, kTreeSms = 152;

struct TreeSplit {
    int groups, row_tiles;
    size_t line_bytes, lse_bytes, total;
};

TreeSplit tree_split(int batch, int Hq, int Hkv, int D, int max_q) {
    TreeSplit s;
    const int64_t rows = (int64_t)max_q * (Hq / Hkv);
    s.row_tiles = (int)((rows + kTreeTile - 1) / kTreeTile);
    if (s.row_tiles < 1) s.row_tiles = 1;
    s.groups = kTreeSms / Hkv > 0 ? kTreeSms / Hkv : 1;
    // rows of a row group: two tiles where the CTA takes two
    const size_t grow = kTreeTile * (D <= 128 && s.row_tiles > 1 ? 2 : 1);
    const size_t units = (size_t)2 * s.groups * Hkv * grow;
    s.line_bytes = (((size_t)batch + 1) * 8 + 255) / 256 * 256;
    s.lse_bytes = (units * sizeof(float) + 255) / 256 * 256;
    s.total = s.line_bytes + s.lse_bytes + units * D * sizeof(float);
    return s;
}

}  // namespace

}  // namespace pkv

using namespace pkv;

extern "C" {

pkv_status pkv_reshape_and_cache_fp8(const void *key, const void *value, int64_t key_stride,
                                     int64_t value_stride, int dtype, void *k_cache,
                                     void *v_cache, uint8_t *k_scale, uint8_t *v_scale,
                                     const int64_t *slot_mapping, int64_t num_tokens,
                                     pkv_cache_desc cache, int32_t *dev_error, void *stream) {
    const pkv_status st = check_pool(cache, true, false);
    if (st != PKV_OK) return st;
    if (num_tokens < 0) return PKV_ERR_INVALID_ARG;
    if (dtype != PKV_BF16 && dtype != PKV_F32) return PKV_ERR_UNSUPPORTED;
    const int64_t row = (int64_t)cache.num_kv_heads * cache.head_dim;
    const int vec = dtype == PKV_F32 ? 4 : 8;
    if (num_tokens == 0) return PKV_OK;
    if (key_stride < row || value_stride < row || key_stride % vec || value_stride % vec)
        return PKV_ERR_INVALID_ARG;
    if (!key || !value || !k_cache || !v_cache || !k_scale || !v_scale || !slot_mapping)
        return PKV_ERR_INVALID_ARG;
    if (!aligned(key, 16) || !aligned(value, 16) || !aligned(k_cache, 16) ||
        !aligned(v_cache, 16) || !aligned(slot_mapping, 8))
        return PKV_ERR_INVALID_ARG;
    QuantWriteParams p;
    p.key = key;
    p.value = value;
    p.key_stride = key_stride;
    p.value_stride = value_stride;
    p.slot_mapping = slot_mapping;
    p.num_tokens = num_tokens;
    p.dev_error = dev_error;
    p.pool = pool_args(cache, k_cache, v_cache, k_scale, v_scale);
    return from_cuda(launch_quant_write(p, dtype, static_cast<cudaStream_t>(stream)));
}

pkv_status pkv_gather_cache_fp8(void *key, void *value, const void *k_cache, const void *v_cache,
                                const uint8_t *k_scale, const uint8_t *v_scale,
                                pkv_cache_desc cache, const int32_t *block_table,
                                int max_blocks_per_seq, const int32_t *cu_seq_lens_k, int batch,
                                int64_t total_k, int32_t *dev_error, void *stream) {
    const pkv_status st = check_pool(cache, true, false);
    if (st != PKV_OK) return st;
    if (batch < 0 || total_k < 0 || max_blocks_per_seq < 0) return PKV_ERR_INVALID_ARG;
    if (total_k > (int64_t(1) << 30)) return PKV_ERR_UNSUPPORTED;
    if (batch == 0 || total_k == 0) return PKV_OK;  // (a table without columns has no rows)
    if (max_blocks_per_seq == 0) return PKV_ERR_INVALID_ARG;
    if (!key || !value || !k_cache || !v_cache || !k_scale || !v_scale || !block_table ||
        !cu_seq_lens_k)
        return PKV_ERR_INVALID_ARG;
    if (!aligned(key, 16) || !aligned(value, 16) || !aligned(k_cache, 16) ||
        !aligned(v_cache, 16) || !aligned(block_table, 4) || !aligned(cu_seq_lens_k, 4))
        return PKV_ERR_INVALID_ARG;
    GatherParams p;
    p.key = key;
    p.value = value;
    p.block_table = block_table;
    p.cu_k = cu_seq_lens_k;
    p.dev_error = dev_error;
    p.num_blocks = cache.num_blocks;
    p.batch = batch;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.total_k = (int)total_k;
    p.pool = pool_args(cache, k_cache, v_cache, k_scale, v_scale);
    return from_cuda(launch_gather(p, static_cast<cudaStream_t>(stream)));
}

pkv_status pkv_paged_decode_fp8(void *out, const void *q, const void *k_cache,
                                const void *v_cache, const uint8_t *k_scale,
                                const uint8_t *v_scale, pkv_cache_desc cache,
                                const int32_t *block_table, int max_blocks_per_seq,
                                const int32_t *cache_seqlens, int max_seqlen, const float *sink,
                                const float *alibi_slopes, int batch, int num_qo_heads,
                                int window_left, float sm_scale, int partition_size,
                                float *lse_out, void *workspace, size_t workspace_bytes,
                                int32_t *dev_error, void *stream) {
    pkv_status st = check_pool(cache, true, false);
    if (st != PKV_OK) return st;
    if (batch < 0 || batch > 65535 || num_qo_heads <= 0 || max_seqlen < 0 ||
        max_blocks_per_seq <= 0 || window_left < -1 || !std::isfinite(sm_scale))
        return PKV_ERR_INVALID_ARG;
    if (num_qo_heads % cache.num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
    const int G = num_qo_heads / cache.num_kv_heads;
    // (positions and partition bounds are 32-bit)
    if (G > 16 || max_seqlen > (1 << 30)) return PKV_ERR_UNSUPPORTED;
    int P = partition_size;
    if (P == 0) {
        // Longer ones while the SMs have more than eight full rounds of CTAs and the
        // longest sequence keeps eight partitions of the keys it attends (a window leaves
        // the last ones).  Share of a copy's rate with 512, 1024 and 1536, over five
        // draws: 8 of 32K..128K tokens 82, 87 and 89 % (heads of 64: 66, 77
        // and 80), 16 of 4K..32K 75, 79 and 70; fewer than eight, 128 of 0.5K..8K:
        // 85, 87 and 84.  16 of 32K..128K with a window of 4K: 51, 58 and 45.
        const int64_t span = window_left >= 0 && window_left < max_seqlen
                                 ? (int64_t)window_left + 1
                                 : max_seqlen;
        P = kDefaultPartition;
        while (P < kMaxAutoPartition &&
               (int64_t)batch * cache.num_kv_heads * (span / P) > 8 * kDecodeSlots &&
               span / (P + kDefaultPartition) >= 8)
            P += kDefaultPartition;
    }
    if (P < 0 || P % cache.block_size != 0 || P > kMaxPartition) return PKV_ERR_INVALID_ARG;
    if (batch == 0) return PKV_OK;
    if (!out || !q || !k_cache || !v_cache || !k_scale || !v_scale || !block_table ||
        !cache_seqlens)
        return PKV_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(k_scale, 16) || !aligned(v_scale, 16) || !aligned(block_table, 4) ||
        !aligned(cache_seqlens, 4))
        return PKV_ERR_INVALID_ARG;
    int64_t np = ((int64_t)max_seqlen + P - 1) / P;
    if (window_left >= 0) {
        const int64_t w = ((int64_t)window_left + 1 + P - 1) / P + 1;
        if (w < np) np = w;
    }
    if (np < 1) np = 1;
    if (np > 65535) return PKV_ERR_UNSUPPORTED;  // grid.y limit
    const size_t units = (size_t)batch * num_qo_heads * (size_t)np;
    // the layout of the workspace is paged_decode's: lse, then outputs; one
    // partition writes the output itself
    const size_t need = pkv_paged_decode_workspace_size(batch, num_qo_heads, cache.head_dim,
                                                        max_seqlen, P, window_left);
    if (np > 1 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need))
        return PKV_ERR_WORKSPACE;

    DecodeFp8Params pp;
    std::memset(&pp, 0, sizeof pp);
    DecodeParams &p = pp.d;
    p.q = q;
    p.out = out;
    p.block_table = block_table;
    p.seqlens = cache_seqlens;
    p.sink = sink;
    p.alibi = alibi_slopes;
    p.lse_out = lse_out;
    p.part_lse = static_cast<float *>(workspace);
    p.part_o = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                         (units * sizeof(float) + 255) / 256 * 256);
    p.dev_error = dev_error;
    p.num_blocks = cache.num_blocks;
    p.batch = batch;
    p.num_qo_heads = num_qo_heads;
    p.num_kv_heads = cache.num_kv_heads;
    p.group = G;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.max_seqlen = max_seqlen;
    p.window_left = window_left;
    p.head_dim = cache.head_dim;
    p.hnd = cache.layout == PKV_HND ? 1 : 0;
    p.partition_size = P;
    p.num_parts = (int)np;
    p.scale_log2 = sm_scale * 1.4426950408889634f;
    pp.k_scale = k_scale;
    pp.v_scale = v_scale;

    alignas(64) CUtensorMap tk, tv;
    const int rows = decode_fp8_box_rows(cache.head_dim, cache.block_size);
    if ((st = pool_map(&tk, k_cache, cache, rows)) != PKV_OK) return st;
    if ((st = pool_map(&tv, v_cache, cache, rows)) != PKV_OK) return st;
    return from_cuda(launch_decode_fp8(pp, cache, &tk, &tv, static_cast<cudaStream_t>(stream)));
}

pkv_status pkv_qk_norm_rope_reshape_and_cache(
    const void *query, const void *key, const void *value, int64_t query_stride,
    int64_t key_stride, int64_t value_stride, int dtype, void *query_out, void *key_out,
    int64_t query_out_stride, int64_t key_out_stride, void *k_cache, void *v_cache,
    uint8_t *k_scale, uint8_t *v_scale, const int64_t *positions, const int64_t *slot_mapping,
    int64_t num_tokens, int num_qo_heads, pkv_cache_desc cache, const void *q_weight,
    const void *k_weight, int weight_f32, float eps, const float *cos_sin, int max_position,
    int rotary_dim, int is_neox_style, int32_t *dev_error, void *stream) {
    const pkv_status st = check_pool(cache, true, true);
    if (st != PKV_OK) return st;
    if (num_tokens < 0 || num_qo_heads < 0 || max_position <= 0 || !std::isfinite(eps) ||
        eps < 0.f)
        return PKV_ERR_INVALID_ARG;
    if (dtype != PKV_BF16 && dtype != PKV_F32) return PKV_ERR_UNSUPPORTED;
    const bool fp8 = cache.dtype == PKV_E4M3;
    if (!fp8 && cache.dtype != dtype) return PKV_ERR_INVALID_ARG;
    if (rotary_dim <= 0 || rotary_dim > cache.head_dim || rotary_dim % 2 != 0)
        return PKV_ERR_INVALID_ARG;
    if (rotary_dim % 16 != 0) return PKV_ERR_UNSUPPORTED;
    const int64_t qrow = (int64_t)num_qo_heads * cache.head_dim;
    const int64_t krow = (int64_t)cache.num_kv_heads * cache.head_dim;
    if (qrow > (1 << 24)) return PKV_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PKV_OK;
    const int vec = dtype == PKV_F32 ? 4 : 8;
    const int64_t strides[5] = {query_stride, query_out_stride, key_stride, value_stride,
                                key_out_stride};
    for (int i = num_qo_heads > 0 ? 0 : 2; i < 5; ++i)
        if (strides[i] < (i < 2 ? qrow : krow) || strides[i] % vec != 0)
            return PKV_ERR_INVALID_ARG;
    if (!key || !value || !key_out || !k_cache || !v_cache || !positions || !slot_mapping ||
        !cos_sin || !k_weight || (num_qo_heads > 0 && (!query || !query_out || !q_weight)) ||
        (fp8 && (!k_scale || !v_scale)))
        return PKV_ERR_INVALID_ARG;
    if (num_qo_heads > 0 &&
        (!aligned(query, 16) || !aligned(query_out, 16) || !aligned(q_weight, 16)))
        return PKV_ERR_INVALID_ARG;
    if (!aligned(key, 16) || !aligned(value, 16) || !aligned(key_out, 16) ||
        !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(cos_sin, 16) ||
        !aligned(k_weight, 16) || !aligned(positions, 8) || !aligned(slot_mapping, 8))
        return PKV_ERR_INVALID_ARG;
    NormRopeParams p;
    p.query = query;
    p.key = key;
    p.value = value;
    p.query_out = query_out;
    p.key_out = key_out;
    p.q_stride = query_stride;
    p.k_stride = key_stride;
    p.v_stride = value_stride;
    p.qo_stride = query_out_stride;
    p.ko_stride = key_out_stride;
    p.q_weight = q_weight;
    p.k_weight = k_weight;
    p.weight_f32 = weight_f32 != 0 || dtype == PKV_F32;
    p.positions = positions;
    p.slot_mapping = slot_mapping;
    p.cos_sin = reinterpret_cast<const float2 *>(cos_sin);
    p.num_tokens = num_tokens;
    p.max_position = max_position;
    p.num_qo_heads = num_qo_heads;
    p.rotary_dim = rotary_dim;
    p.neox = is_neox_style != 0;
    p.eps = eps;
    p.dev_error = dev_error;
    p.pool = pool_args(cache, k_cache, v_cache, fp8 ? k_scale : nullptr,
                       fp8 ? v_scale : nullptr);
    return from_cuda(launch_norm_rope(p, dtype, static_cast<cudaStream_t>(stream)));
}

size_t pkv_paged_tree_attention_workspace_size(int batch, int num_qo_heads, int num_kv_heads,
                                               int head_dim, int max_seqlen_q) {
    if (batch <= 0 || num_kv_heads <= 0 || num_qo_heads < num_kv_heads || head_dim <= 0 ||
        max_seqlen_q < 0)
        return 256;
    return tree_split(batch, num_qo_heads, num_kv_heads, head_dim, max_seqlen_q).total;
}

pkv_status pkv_paged_tree_attention(
    void *out, const void *q, const void *k_cache, const void *v_cache, const uint8_t *k_scale,
    const uint8_t *v_scale, pkv_cache_desc cache, const int32_t *block_table,
    int max_blocks_per_seq, const int32_t *cu_seq_lens_q, const int32_t *cache_seqlens,
    int max_seqlen_q, int max_seqlen, int total_q, const int64_t *tree_mask, int mask_words,
    const int32_t *tree_depth, const float *sink, const float *alibi_slopes, int batch,
    int num_qo_heads, int window_left, float sm_scale, int partition_size, float *lse_out,
    void *workspace, size_t workspace_bytes, int32_t *dev_error, void *stream) {
    pkv_status st = check_pool(cache, true, true);
    if (st != PKV_OK) return st;
    if (cache.dtype == PKV_F32) return PKV_ERR_UNSUPPORTED;
    const bool fp8 = cache.dtype == PKV_E4M3;
    if (batch < 0 || batch > 65535 || num_qo_heads <= 0 || max_seqlen < 0 || max_seqlen_q < 0 ||
        total_q < 0 || max_blocks_per_seq <= 0 || window_left < -1 || !std::isfinite(sm_scale) ||
        partition_size < 0 || partition_size % kTreeTile != 0)
        return PKV_ERR_INVALID_ARG;
    if (num_qo_heads % cache.num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
    const int G = num_qo_heads / cache.num_kv_heads;
    if (G > 16 || max_seqlen_q > kMaxDraft || max_seqlen > (1 << 30) || total_q > (1 << 24))
        return PKV_ERR_UNSUPPORTED;
    if (mask_words * (int64_t)64 < max_seqlen_q) return PKV_ERR_INVALID_ARG;
    // positions of drafts come from their depths
    if ((window_left >= 0 || alibi_slopes) && !tree_depth) return PKV_ERR_INVALID_ARG;
    if (batch == 0 || total_q == 0 || max_seqlen_q == 0) return PKV_OK;
    if (!out || !q || !k_cache || !v_cache || !block_table || !cu_seq_lens_q || !cache_seqlens ||
        !tree_mask || (fp8 && (!k_scale || !v_scale)))
        return PKV_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(block_table, 4) || !aligned(cu_seq_lens_q, 4) || !aligned(cache_seqlens, 4) ||
        !aligned(tree_mask, 8) || (fp8 && (!aligned(k_scale, 16) || !aligned(v_scale, 16))))
        return PKV_ERR_INVALID_ARG;
    const TreeSplit s =
        tree_split(batch, num_qo_heads, cache.num_kv_heads, cache.head_dim, max_seqlen_q);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < s.total)
        return PKV_ERR_WORKSPACE;

    TreeParams p;
    std::memset(&p, 0, sizeof p);
    p.q = q;
    p.out = out;
    p.block_table = block_table;
    p.cu_q = cu_seq_lens_q;
    p.seqlens = cache_seqlens;
    p.mask = tree_mask;
    p.depth = tree_depth;
    p.sink = sink;
    p.alibi = alibi_slopes;
    p.lse_out = lse_out;
    char *ws = static_cast<char *>(workspace);
    p.line = reinterpret_cast<long long *>(ws);
    p.part_lse = reinterpret_cast<float *>(ws + s.line_bytes);
    p.part_o = reinterpret_cast<float *>(ws + s.line_bytes + s.lse_bytes);
    p.dev_error = dev_error;
    p.k_scale = fp8 ? k_scale : nullptr;
    p.v_scale = fp8 ? v_scale : nullptr;
    p.num_blocks = cache.num_blocks;
    p.batch = batch;
    p.num_qo_heads = num_qo_heads;
    p.num_kv_heads = cache.num_kv_heads;
    p.group = G;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.max_seqlen = max_seqlen;
    p.max_seqlen_q = max_seqlen_q;
    p.total_q = total_q;
    p.mask_words = mask_words;
    p.window_left = window_left;
    p.head_dim = cache.head_dim;
    p.hnd = cache.layout == PKV_HND ? 1 : 0;
    p.block_size = cache.block_size;
    p.groups = s.groups;
    p.min_tiles = partition_size > 0 ? partition_size / kTreeTile : 1;
    p.row_tiles = s.row_tiles;
    p.scale_log2 = sm_scale * 1.4426950408889634f;

    alignas(64) CUtensorMap tk, tv;
    if ((st = pool_map(&tk, k_cache, cache, cache.block_size)) != PKV_OK) return st;
    if ((st = pool_map(&tv, v_cache, cache, cache.block_size)) != PKV_OK) return st;
    return from_cuda(launch_tree(p, &tk, &tv, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
