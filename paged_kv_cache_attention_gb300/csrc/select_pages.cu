// select_pages.cu -- for every query and kv head, the pages whose bounds allow the
// largest scores (an upper bound per page from its channels' least and largest
// keys, as in query-aware page selection, and the highest top_k of them).
//
// Query head h of a group: 2^E <= max_d |q_d| < 2^(E+1), e_h = max(E, -112) - 7,
//   c_d = rint(q_d * 2^-e_h), |c_d| <= 255
//   I_h = sum_d max(c_d, 0) * hi_d + min(c_d, 0) * lo_d     (codes of page_bounds.cu)
//   score = max over the group's heads of float(I_h * 2^(e_h + byte - 127))
// All factors are small integers and powers of two: |I_h| < 2^23 is exact in fp32
// whatever the order of the sum, so the lists do not depend on the launch.  (A sum of
// rounded products would swap pages that are nearly alike.)  A page with byte 255
// scores +inf; a head whose q is not finite has no say.  The first num_first and
// the last num_recent pages of the row are always taken; equal scores: the lower
// page first.
//
// I_h is a product [pages, 2 D] x [2 D, heads]: mma.sync m16n8k16 in f16 (integers
// up to 2048 are exact there), 16 pages as rows and up to 8 heads as columns.  The
// order of the summands is free, so a lane loads 16 codes in one go and uses them
// as the fragments of four steps, and the columns are laid out to match.  A code
// becomes an f16 by putting it into the mantissa of 1024 (a byte permutation) and
// taking 1152 off: 2.5 instructions for a pair.
//
// A cluster of CTAs shares the pages of a (query, kv head); each keeps its pages'
// scores in its own shared memory, as integers that sort like the scores.  The
// top_k-th largest is found digit by digit (8 bits at a time, histograms summed over the
// cluster), then the pages above it, and as many of those equal to it as there is
// room for, are written in ascending order.  One launch, no workspace.
//
// HBM bound: (2 D + 1) bytes per page and kv head, each read once in a decode step.
#include <cuda_fp16.h>

#include "pkv_sparse.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr uint32_t kForced = 0xffffffffu;  // above every score
constexpr int kNoVote = -100000;           // exponent of a head that has no say

// An unsigned integer that sorts like x (no NaN; -0 was made 0).
__device__ __forceinline__ uint32_t sortable(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// Four int8 codes of a word as f16 pairs (bytes 0 and 1, bytes 2 and 3), exact.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const uint32_t u = w ^ 0x80808080u;  // code + 128
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const uint32_t off = 0x64806480u;    // 1152, twice
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(off));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(off));
}

__device__ __forceinline__ void block_sync(bool cluster) {
    if (cluster)
        cluster_sync();
    else
        __syncthreads();
}

// NCH: 64-byte pieces of a page's codes; NT: 8-head column tiles.
template <int NCH, int NT>
__global__ void __launch_bounds__(kThreads) select_pages_kernel(const SelectParams p) {
    extern __shared__ uint32_t s_key[];          // [cap]
    __shared__ uint4 s_q[NT][NCH][2][32];        // column fragments: [..][steps 0-1, 2-3][lane]
    __shared__ int s_exp[16];
    __shared__ uint32_t s_hist[4][256];
    __shared__ uint32_t s_pick[2];               // digit, pages above it
    __shared__ int s_cnt[kWarps][2], s_total[2]; // above, equal: per warp, of the CTA

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int C = p.cluster, rank = C > 1 ? (int)cluster_rank() : 0;
    const int64_t unit = blockIdx.x / (unsigned)C;
    const int t = (int)(unit / p.r.num_kv_heads), g = (int)(unit % p.r.num_kv_heads);
    const int D = p.r.head_dim, G = p.r.group;

    pdl_wait();
    int r, L;
    if (!row_request(p.r, t, p.block_size, g == 0 && rank == 0 && threadIdx.x == 0, r, L)) return;
    const int n = (L + p.block_size - 1) / p.block_size;
    int32_t *out = p.pages + unit * p.top_k;
    if (n <= p.top_k) {  // all of them
        for (int i = rank * kThreads + threadIdx.x; i < p.top_k; i += C * kThreads)
            out[i] = i < n ? i : -1;
        return;
    }
    const int per = ((n + C - 1) / C + 15) / 16 * 16;
    const int base = rank * per, nl = min(max(n - base, 0), per);

    // the group's queries as column fragments
    for (int i = threadIdx.x; i < 4 * 256; i += kThreads) (&s_hist[0][0])[i] = 0;
    for (int i = threadIdx.x; i < NT * NCH * 64; i += kThreads)
        (&s_q[0][0][0][0])[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) +
                             ((int64_t)t * p.r.num_kv_heads + g) * G * D;
    for (int h = warp; h < G; h += kWarps) {
        uint32_t amax = 0;
        for (int d = lane; d < D; d += 32)
            amax = max(amax, (uint32_t)__bfloat16_as_ushort(q[h * D + d]) & 0x7fffu);
        amax = __reduce_max_sync(0xffffffffu, amax);
        const bool ok = amax < 0x7f80u;
        const int e = max((int)(amax >> 7) - 127, -112) - 7;
        if (lane == 0) s_exp[h] = ok ? e : kNoVote;
        const float f = ok ? __uint_as_float((uint32_t)(127 - e) << 23) : 0.f;
        for (int d = lane; d < D; d += 32) {
            const float c = ok ? rintf(__bfloat162float(q[h * D + d]) * f) : 0.f;
#pragma unroll
            for (int part = 0; part < 2; ++part) {  // against the lower, the upper bounds
                const int k = part * D + d;
                const int piece = k >> 6, tq = (k >> 4) & 3, step = (k >> 2) & 3, w = k & 3;
                // column h % 8, its lane's word 2 * (step % 2) + w / 2, half w % 2
                __half *dst = reinterpret_cast<__half *>(
                    &s_q[h >> 3][piece][step >> 1][(h & 7) * 4 + tq]);
                dst[4 * (step & 1) + w] = __float2half(part ? fmaxf(c, 0.f) : fminf(c, 0.f));
            }
        }
    }
    for (int h = G + threadIdx.x; h < 16; h += kThreads) s_exp[h] = kNoVote;
    __syncthreads();
    int top_e = kNoVote, low_e = 100000;
    for (int h = 0; h < G; ++h)
        if (s_exp[h] != kNoVote) {
            top_e = max(top_e, s_exp[h]);
            low_e = min(low_e, s_exp[h]);
        }
    // the heads' factors are exact relative to the largest, but for exponents further
    // apart than a float's (then each score is scaled by itself)
    const bool apart = top_e != kNoVote && top_e - low_e > 126;
    const int gq = lane >> 2, tq = lane & 3;
    int ex[NT][2];
    float fac[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            ex[nt][i] = s_exp[nt * 8 + 2 * tq + i];
            fac[nt][i] = ex[nt][i] == kNoVote ? 0.f
                                              : __uint_as_float((uint32_t)(127 + max(ex[nt][i] - top_e, -126)) << 23);
        }

    // scores of 16 pages at a time
    const int32_t *bt = p.r.block_table + (int64_t)r * p.r.max_blocks_per_seq;
    for (int i0 = warp * 16; i0 < nl; i0 += kWarps * 16) {
        uint4 w[2][NCH];
        uint32_t byte[2];
        bool live[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int i = i0 + gq + 8 * j, page = base + i;
            int id = -1;
            live[j] = false;
            if (i < nl) {
                id = __ldg(bt + page);
                live[j] = id >= 0 && id < p.r.num_blocks;
                if (!live[j] && tq == 0) flag_error(p.r.dev_error, PKV_DEVERR_BLOCK_ID);
            }
            const int64_t at = (int64_t)(live[j] ? id : 0) * p.r.num_kv_heads + g;
            byte[j] = live[j] ? p.bounds_scale[at] : 0u;
            const int8_t *b = p.bounds + at * 2 * D;
#pragma unroll
            for (int c = 0; c < NCH; ++c) {
                const int o = c * 64 + tq * 16;
                w[j][c] = live[j] && o < 2 * D ? *reinterpret_cast<const uint4 *>(b + o)
                                               : make_uint4(0u, 0u, 0u, 0u);
            }
        }
        float acc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const uint32_t w0[4] = {w[0][c].x, w[0][c].y, w[0][c].z, w[0][c].w};
            const uint32_t w1[4] = {w[1][c].x, w[1][c].y, w[1][c].z, w[1][c].w};
#pragma unroll
            for (int s2 = 0; s2 < 2; ++s2) {
                uint32_t a[2][4];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    codes_to_f16(w0[2 * s2 + s], a[s][0], a[s][2]);
                    codes_to_f16(w1[2 * s2 + s], a[s][1], a[s][3]);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint4 b = s_q[nt][c][s2][lane];
                    mma_f16_16816(acc[nt], a[0][0], a[0][1], a[0][2], a[0][3], b.x, b.y);
                    mma_f16_16816(acc[nt], a[1][0], a[1][1], a[1][2], a[1][3], b.z, b.w);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int be = (int)byte[j] - 127;
            float m = -INFINITY;
            if (!apart) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (ex[nt][i] != kNoVote) m = fmaxf(m, acc[nt][2 * j + i] * fac[nt][i]);
            } else {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (ex[nt][i] != kNoVote)
                            m = fmaxf(m, ldexpf(acc[nt][2 * j + i], ex[nt][i] + be));
            }
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const int i = i0 + gq + 8 * j, page = base + i;
            if (tq == j && i < nl) {
                if (!apart && top_e != kNoVote) m = ldexpf(m, top_e + be);
                if (byte[j] == kScaleNaN) m = INFINITY;
                uint32_t key = live[j] ? sortable(m + 0.f) : 0u;
                if (page < p.num_first || page >= n - p.num_recent) key = kForced;
                s_key[i] = key;
            }
        }
    }
    __syncthreads();

    // the top_k-th largest, 8 bits at a time
    uint32_t prefix = 0;
    int need = p.top_k;
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        for (int i = threadIdx.x; i < nl; i += kThreads) {
            const uint32_t key = s_key[i];
            if (pass == 0 || (key >> (shift + 8)) == (prefix >> (shift + 8)))
                atomicAdd(&s_hist[pass][(key >> shift) & 255u], 1u);
        }
        block_sync(C > 1);
        // thread b: bin 255 - b, so that a prefix sum counts from the largest down
        uint32_t v = 0;
        const uint32_t at = smem_u32(&s_hist[pass][255 - threadIdx.x]);
        if (C > 1)
            for (int c = 0; c < C; ++c) v += cluster_ld32(cluster_addr(at, c));
        else
            v = s_hist[pass][255 - threadIdx.x];
        uint32_t sum = v;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off) sum += o;
        }
        if (lane == 31) s_cnt[warp][0] = (int)sum;
        __syncthreads();
        for (int w = 0; w < warp; ++w) sum += (uint32_t)s_cnt[w][0];
        if (sum >= (uint32_t)need && sum - v < (uint32_t)need) {
            s_pick[0] = 255u - threadIdx.x;
            s_pick[1] = sum - v;
        }
        __syncthreads();
        prefix |= s_pick[0] << shift;
        need -= (int)s_pick[1];
        __syncthreads();  // s_pick and s_cnt are used again
    }

    // pages above it, and the first `need` of those equal to it, in ascending order
    const int seg = ((nl + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int lo = min(warp * seg, nl), hi = min(lo + seg, nl);
    int above = 0, equal = 0;
    for (int i = lo; i < hi; i += 32) {
        const uint32_t key = i + lane < hi ? s_key[i + lane] : 0u;
        const bool in = i + lane < hi;
        above += __popc(__ballot_sync(0xffffffffu, in && key > prefix));
        equal += __popc(__ballot_sync(0xffffffffu, in && key == prefix));
    }
    if (lane == 0) {
        s_cnt[warp][0] = above;
        s_cnt[warp][1] = equal;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        int s = 0;
        for (int w = 0; w < kWarps; ++w) s += s_cnt[w][threadIdx.x];
        s_total[threadIdx.x] = s;
    }
    block_sync(C > 1);
    int n_above = 0, n_equal = 0;  // before this warp's pages
    for (int c = 0; c < rank; ++c) {
        n_above += (int)cluster_ld32(cluster_addr(smem_u32(&s_total[0]), c));
        n_equal += (int)cluster_ld32(cluster_addr(smem_u32(&s_total[1]), c));
    }
    for (int w = 0; w < warp; ++w) {
        n_above += s_cnt[w][0];
        n_equal += s_cnt[w][1];
    }
    const uint32_t below = (1u << lane) - 1u;
    for (int i = lo; i < hi; i += 32) {
        const bool in = i + lane < hi;
        const uint32_t key = in ? s_key[i + lane] : 0u;
        const uint32_t ma = __ballot_sync(0xffffffffu, in && key > prefix);
        const uint32_t me = __ballot_sync(0xffffffffu, in && key == prefix);
        const int a = n_above + __popc(ma & below), e = n_equal + __popc(me & below);
        if (in && (key > prefix || (key == prefix && e < need))) out[a + min(e, need)] = base + i + lane;
        n_above += __popc(ma);
        n_equal += __popc(me);
    }
    if (C > 1) cluster_sync();  // the others may still read this CTA's counts
}

template <int NCH>
cudaError_t launch_n(const SelectParams &p, cudaStream_t stream) {
    auto kern = p.r.group <= 8 ? select_pages_kernel<NCH, 1> : select_pages_kernel<NCH, 2>;
    const int smem = p.cap * 4;
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kern), smem);
    if (e != cudaSuccess) return e;
    const int64_t grid = (int64_t)p.r.rows * p.r.num_kv_heads * p.cluster;
    if (grid > 0x7fffffff) return cudaErrorNotSupported;
    return launch_cluster(kern, (unsigned)grid, p.cluster, kThreads, (size_t)smem, stream, p);
}

}  // namespace

cudaError_t launch_select_pages(const SelectParams &p0, cudaStream_t stream) {
    SelectParams p = p0;
    const int64_t units = (int64_t)p.r.rows * p.r.num_kv_heads;
    const int n = (p.r.max_seqlen + p.block_size - 1) / p.block_size;
    // as many CTAs per row as there is room for at once, of at least 128 pages, and
    // more if the scores would not fit
    int c = 1;
    while (c < 8 && ((units * c < 2LL * device_sm_count() && n / c >= 256) || n / c > 32768)) c *= 2;
    p.cluster = c;
    p.cap = ((n + c - 1) / c + 15) / 16 * 16;
    if (p.cap > 49152) return cudaErrorNotSupported;
    switch ((2 * p.r.head_dim + 63) / 64) {
    case 2: return launch_n<2>(p, stream);
    case 3: return launch_n<3>(p, stream);
    case 4: return launch_n<4>(p, stream);
    case 8: return launch_n<8>(p, stream);
    default: return cudaErrorNotSupported;
    }
}

}  // namespace pkv
