// pkv_sparse.cuh -- device helpers of the sparse decode step: clusters and their
// shared memory, a row's request and length.
#pragma once

#include "pkv_fp8.cuh"
#include "pkv_sparse.h"

namespace pkv {

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Every thread of every CTA of the cluster; writes before it (shared memory of
// the cluster, global memory) are seen after it by the whole cluster.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}

// The address of a shared-memory word of this CTA in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ uint32_t cluster_ld32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float4 cluster_ld128(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Row t's request r, the number L of keys up to and with its own (0 and less: the row
// attends nothing) and the request's rows from t on, of those that exist: its last one is
// at its last position.  False: a row of no request.  Taken by a whole warp, which looks
// at 32 offsets at a time.
__device__ __forceinline__ bool row_request(const RowParams &p, int t, int block_size,
                                            bool report, int &r, int &L, int &count) {
    const int lane = threadIdx.x & 31;
    count = 1;
    r = t;
    if (p.cu_q) {
        int lo = 0, hi = p.batch;
        while (true) {
            const int step = (hi - lo + 31) / 32, at = lo + lane * step;
            const uint32_t m = __ballot_sync(0xffffffffu, at < hi && p.cu_q[at] <= t);
            const int c = __ffs(~m) - 1;  // leading offsets that are not above t
            const int below = m == 0xffffffffu ? 32 : c;
            if (below == 0) return false;
            lo += (below - 1) * step;
            hi = min(hi, lo + step);
            if (step == 1) break;
        }
        r = lo;
        const int end = min(p.cu_q[r + 1], p.rows);  // (more: check_offsets)
        if (t >= end) return false;
        count = end - t;
    }
    int n = p.seqlens[r];
    const int64_t table = (int64_t)p.max_blocks_per_seq * block_size;
    const int cap = table < p.max_seqlen ? (int)table : p.max_seqlen;
    if (n < 0 || n > cap) {
        if (report) flag_error(p.dev_error, PKV_DEVERR_SEQLEN);
        n = min(max(n, 0), cap);
    }
    L = n - (count - 1);
    return true;
}

// Offsets that decrease or leave the rows are flagged: each is looked at by one of the
// `step` threads of a launch that call this with `first` from 0 on, also those of requests
// that no row belongs to.  (Off the path to a CTA's first load.)
__device__ __forceinline__ void check_offsets(const RowParams &p, int64_t first, int64_t step) {
    if (!p.cu_q) return;
    for (int64_t i = first; i <= p.batch; i += step) {
        const int a = p.cu_q[i];
        if (a > p.rows || a < (i > 0 ? p.cu_q[i - 1] : 0))
            flag_error(p.dev_error, PKV_DEVERR_SEQLEN);
    }
}

// The rows [t0, t_end) of a tile of `queries` rows.  With few requests a tile holds rows
// of one request only, and the tiles are numbered request by request (one that holds
// the end of one request and the beginning of the next would take twice as long);
// else every `queries` rows.  Taken by a whole warp.
__device__ __forceinline__ void tile_rows(const RowParams &p, int tile, int queries, int &t0,
                                          int &t_end) {
    t0 = t_end = 0;
    if (p.batch > kTiledRequests) {
        const int64_t t = (int64_t)tile * queries;
        t0 = (int)min(t, (int64_t)p.rows);
        t_end = (int)min(t + queries, (int64_t)p.rows);
        return;
    }
    const int lane = threadIdx.x & 31;
    for (int r0 = 0; r0 < p.batch; r0 += 32) {
        const int r = r0 + lane;
        int a = 0, b = 0;
        if (r < p.batch) {
            a = min(max(p.cu_q[r], 0), p.rows);
            b = min(max(p.cu_q[r + 1], a), p.rows);
        }
        const int own = (b - a + queries - 1) / queries;
        int sum = own;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off) sum += o;
        }
        const uint32_t over = __ballot_sync(0xffffffffu, sum > tile);
        if (over) {
            const int w = __ffs(over) - 1;
            const int k = tile - __shfl_sync(0xffffffffu, sum - own, w);
            t0 = __shfl_sync(0xffffffffu, a, w) + k * queries;
            t_end = min(t0 + queries, __shfl_sync(0xffffffffu, b, w));
            return;
        }
        tile -= __shfl_sync(0xffffffffu, sum, 31);
    }
}

// The list of a row: strictly ascending pages below npages.  It ends at the first
// entry that is negative, not above the one before it or not a page of the row (the
// last two are errors).  Returns the entries before that; all threads of the CTA.
template <int THREADS>
__device__ __forceinline__ int list_length(const int32_t *list, int top_k, int npages,
                                           int32_t *dev_error, bool report, int *s_min) {
    int end = top_k;
    for (int i = threadIdx.x; i < top_k; i += THREADS) {
        const int e = list[i], before = i > 0 ? list[i - 1] : -1;
        if (e <= before || e >= npages) {
            end = i;
            break;
        }
    }
    end = __reduce_min_sync(0xffffffffu, end);
    if ((threadIdx.x & 31) == 0) s_min[threadIdx.x >> 5] = end;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) end = min(end, s_min[w]);
    if (report && threadIdx.x == 0 && end < top_k && list[end] >= 0)
        flag_error(dev_error, PKV_DEVERR_BLOCK_ID);
    return end;
}

// Join the cluster's parts of a row's heads and store them.  s_out [group][stride]
// holds this CTA's normalised outputs (zeros without keys), s_lse [group] their
// log-sum-exp in log2 units (-inf without keys, NaN stays):
//   o = sum_c 2^(lse_c - T) o_c / (sum_c 2^(lse_c - T) + 2^(sink - T))
template <int THREADS>
__device__ __forceinline__ void join_and_store(const SparseParams &p, int t, int g, int rank,
                                               const float *s_out, int stride,
                                               const float *s_lse) {
    const int C = p.cluster, G = p.r.group, D = p.r.head_dim;
    if (C > 1)
        cluster_sync();
    else
        __syncthreads();
    const uint32_t out = smem_u32(s_out), lse = smem_u32(s_lse);
    const int vecs = D / 4;
    for (int i = rank * THREADS + threadIdx.x; i < G * vecs; i += C * THREADS) {
        const int h = i / vecs, d = (i - h * vecs) * 4;
        const int hq = g * G + h;
        const float sink = p.sink ? p.sink[hq] * kLog2e : -INFINITY;
        float T = sink;
        for (int c = 0; c < C; ++c)
            T = fmaxf(T, C > 1 ? __uint_as_float(cluster_ld32(cluster_addr(lse + 4 * h, c)))
                               : s_lse[h]);
        const float Ts = T == -INFINITY ? 0.f : T;
        float sum = exp2f(sink - Ts);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < C; ++c) {
            float l;
            float4 v;
            if (C > 1) {
                l = __uint_as_float(cluster_ld32(cluster_addr(lse + 4 * h, c)));
                v = cluster_ld128(cluster_addr(out + 4 * (h * stride + d), c));
            } else {
                l = s_lse[h];
                v = *reinterpret_cast<const float4 *>(s_out + h * stride + d);
            }
            const float w = exp2f(l - Ts);
            sum += w;
            acc.x = fmaf(w, v.x, acc.x);
            acc.y = fmaf(w, v.y, acc.y);
            acc.z = fmaf(w, v.z, acc.z);
            acc.w = fmaf(w, v.w, acc.w);
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int64_t unit = (int64_t)t * p.r.num_kv_heads * G + hq;
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + unit * D + d) =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
        if (p.lse_out && d == 0)
            p.lse_out[unit] = sum == 0.f ? -INFINITY : (Ts + log2f(sum)) * kLn2;
    }
    if (C > 1) cluster_sync();  // the others may still read this CTA's part
}

}  // namespace pkv
