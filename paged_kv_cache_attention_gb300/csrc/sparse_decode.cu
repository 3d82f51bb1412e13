// sparse_decode.cu -- attention of every query over its list of pages (bf16 pools).
//
// Row t attends, per kv head g, the keys of the pages pages[t, g, :] of its
// request, up to and with its own position:
//   s_j = sm_scale <q, k_j>,  o = sum_j p_j v_j / (sum_j p_j + exp(sink))
// with the softmax, the sink and the lse of decode.cu.  The list is strictly
// ascending, so only its last page can end inside (at the row's own key): the
// pages of a list are taken as a sequence of their own, with one end.
//
// A cluster of CTAs shares a row's list of a kv head evenly; every CTA of two warps
// streams its pages through rings of two pages per warp by TMA, as in the dense
// decode, with the products on mma.sync (heads as rows of S = Q K^T, as columns of
// O^T += V^T P^T).  The parts of a cluster meet in distributed shared memory:
// each CTA adds up its share of the outputs' columns.  One launch, no workspace.
//
// A weight rounds to bf16 for its product with V (at most 2^-8 of it, as in the dense
// decode: the products are of bf16 pairs); the sum of the weights takes it unrounded.
//
// HBM bound in a decode step (4 D bytes per key and kv head): 64 rows of 1024 keys, 8 kv
// heads of 128: 44.5 us, 89% of HBM's rate; 3 rows of 256 keys 5.4 us, the latency of
// the list, the pages and the join.
#include "pkv_sparse.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 2;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxGroup = 16;
constexpr float kNegInf = -INFINITY;

__device__ __forceinline__ uint32_t ld_b32(const __nv_bfloat16 *p) {
    return *reinterpret_cast<const uint32_t *>(p);
}

template <int D, int BS>
struct Shape {
    static constexpr int NST = 2;                            // pages in flight per warp
    static constexpr int HALVES = D / 64;
    static constexpr int HALF_BYTES = BS * 128;              // one 64-dim half of a page
    static constexpr int PAGE_BYTES = HALVES * HALF_BYTES;   // K (or V) of one page
    static constexpr int STAGE_BYTES = 2 * PAGE_BYTES;
    static constexpr int RING = kWarps * NST * STAGE_BYTES;
    static constexpr int ROW = D + 4;                        // floats of a row of the parts below
    // the ring is used again: [warp][8 heads][ROW] parts, then [16 heads][ROW] outputs
    static constexpr int OUT_OFF = kWarps * 8 * ROW * 4;
    static constexpr int BAR_OFF = RING > OUT_OFF + kMaxGroup * ROW * 4
                                       ? RING
                                       : OUT_OFF + kMaxGroup * ROW * 4;
    static constexpr int M_OFF = BAR_OFF + kWarps * NST * 8;
    static constexpr int L_OFF = M_OFF + kWarps * kMaxGroup * 4;
    static constexpr int LSE_OFF = L_OFF + kWarps * kMaxGroup * 4;
    static constexpr int MIN_OFF = LSE_OFF + kMaxGroup * 4;
    static constexpr int BLK_OFF = MIN_OFF + kWarps * 4;
    static constexpr int SMEM_FIXED = 1024 + BLK_OFF;        // + the CTA's page ids
};

template <int D, int BS, int NHT, bool HND>
__global__ void __launch_bounds__(kThreads)
sparse_decode_kernel(const SparseParams p, const __grid_constant__ CUtensorMap tmk,
                     const __grid_constant__ CUtensorMap tmv) {
    using C = Shape<D, BS>;
    constexpr int NST = C::NST;
    constexpr int NT = BS / 8;   // 8-token column tiles of S per page
    constexpr int KS = BS / 16;  // 16-token k-steps of PV per page
    constexpr int DK = D / 16;   // 16-dim k-steps of QK / m-tiles of PV

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);  // 1024-aligned
    int *s_blk = reinterpret_cast<int *>(smem + C::BLK_OFF);
    float *s_m = reinterpret_cast<float *>(smem + C::M_OFF);
    float *s_l = reinterpret_cast<float *>(smem + C::L_OFF);
    float *s_lse = reinterpret_cast<float *>(smem + C::LSE_OFF);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = p.cluster > 1 ? (int)cluster_rank() : 0;
    const int64_t unit = blockIdx.x / (unsigned)p.cluster;
    const int t = (int)(unit / p.r.num_kv_heads), g = (int)(unit % p.r.num_kv_heads);
    const int G = p.r.group, Dh = p.r.head_dim;

    const uint32_t ring = smem_u32(smem);
    const uint32_t bars = ring + C::BAR_OFF;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kWarps * NST; ++i) mbar_init(bars + 8 * i, 1);
        fence_barrier_init();
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    pdl_wait();
    const bool first = g == 0 && rank == 0;
    int r, L, count;
    const bool live = row_request(p.r, t, BS, first && threadIdx.x == 0, r, L, count);
    auto check = [&] {
        if (first)
            check_offsets(p.r, t + (int64_t)threadIdx.x * p.r.rows, (int64_t)kThreads * p.r.rows);
    };
    if (!live) return check();
    L = max(L, 0);
    const int npages = (L + BS - 1) / BS;
    const int32_t *list = p.pages + unit * p.top_k;
    const int n = list_length<kThreads>(list, p.top_k, npages, p.r.dev_error, rank == 0,
                                        reinterpret_cast<int *>(smem + C::MIN_OFF));
    const int per = (n + p.cluster - 1) / p.cluster;
    const int lo = min(rank * per, n), mine = min(per, n - lo);  // this CTA's entries
    const int32_t *bt = p.r.block_table + (int64_t)r * p.r.max_blocks_per_seq;
    int rows = mine * BS;  // keys, but for the end of the row's last page
    if (mine > 0 && list[lo + mine - 1] == npages - 1) rows -= npages * BS - L;
    for (int i = threadIdx.x; i < mine; i += kThreads) {
        int id = bt[list[lo + i]];
        if (id < 0 || id >= p.r.num_blocks) {
            flag_error(p.r.dev_error, PKV_DEVERR_BLOCK_ID);
            id = -1;
        }
        s_blk[i] = id;
    }
    __syncthreads();

    // pages of this warp: i = warp + j * kWarps
    const int nmine = mine > warp ? (mine - warp + kWarps - 1) / kWarps : 0;
    const uint32_t wring = ring + warp * NST * C::STAGE_BYTES;
    const uint32_t wbars = bars + warp * NST * 8;
    const uint64_t policy = l2_policy_evict_first();
    auto issue = [&](int j) {
        const int s = j % NST;
        const uint32_t bar = wbars + 8 * s;
        const int blk = s_blk[warp + j * kWarps];
        if (blk < 0) {  // invalid page: complete the phase without data
            mbar_arrive(bar);
            return;
        }
        mbar_arrive_expect_tx(bar, C::STAGE_BYTES);
        const uint32_t dst = wring + s * C::STAGE_BYTES;
        const int cy = HND ? 0 : g;
        const int cz = HND ? blk * p.r.num_kv_heads + g : blk * BS;
#pragma unroll
        for (int h = 0; h < C::HALVES; ++h) {
            tma_load_3d_hint(dst + h * C::HALF_BYTES, &tmk, bar, h * 64, cy, cz, policy);
            tma_load_3d_hint(dst + C::PAGE_BYTES + h * C::HALF_BYTES, &tmv, bar, h * 64, cy, cz,
                             policy);
        }
    };
    if (elect_one())
        for (int j = 0; j < NST && j < nmine; ++j) issue(j);
    check();

    // Q as the A operand (rows = query heads, zero-padded to 16; dims past the head
    // size are zeros, as the boxes' columns past it)
    const int gq = lane >> 2, tq = lane & 3;
    const __nv_bfloat16 *qb =
        static_cast<const __nv_bfloat16 *>(p.q) + ((int64_t)t * p.r.num_kv_heads + g) * G * Dh;
    uint32_t qa[DK][4];
#pragma unroll
    for (int kk = 0; kk < DK; ++kk) {
        const int d0 = kk * 16 + 2 * tq;
        const bool in = kk * 16 < Dh;
        const bool h0 = in && gq < G, h1 = in && NHT > 1 && gq + 8 < G;
        qa[kk][0] = h0 ? ld_b32(qb + gq * Dh + d0) : 0u;
        qa[kk][1] = h1 ? ld_b32(qb + (gq + 8) * Dh + d0) : 0u;
        qa[kk][2] = h0 ? ld_b32(qb + gq * Dh + d0 + 8) : 0u;
        qa[kk][3] = h1 ? ld_b32(qb + (gq + 8) * Dh + d0 + 8) : 0u;
    }

    float oacc[NHT][DK][4];
    float m_run[NHT], l_run[NHT];
#pragma unroll
    for (int ht = 0; ht < NHT; ++ht) {
        m_run[ht] = kNegInf;
        l_run[ht] = 0.f;
#pragma unroll
        for (int mt = 0; mt < DK; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) oacc[ht][mt][e] = 0.f;
    }

    int consumed = 0;
    for (int j = 0; j < nmine; ++j) {
        const int i = warp + j * kWarps;
        const int s = j % NST;
        if (!warp_wait_bounded(wbars + 8 * s, (j / NST) & 1, p.r.dev_error)) break;
        consumed = j + 1;
        if (s_blk[i] >= 0) {
            const uint32_t kb = wring + s * C::STAGE_BYTES;
            const uint32_t vb = kb + C::PAGE_BYTES;
            const int held = rows - i * BS;  // keys of this page (BS and more: all)
            // rows past the end may hold any bits: zero their V, so that a zero
            // weight never meets a non-finite value
            if (held < BS) {
                for (int e = lane; e < C::HALVES * BS * 8; e += 32) {
                    const int h = e / (BS * 8), rr = (e / 8) % BS, c = e % 8;
                    if (rr >= held) st_shared_zero16(vb + h * C::HALF_BYTES + sw128(rr, c));
                }
                __syncwarp();
            }
            // S = Q K^T  (rows: heads; columns: 8 tokens per tile)
            float sacc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) sacc[nt][e] = 0.f;
#pragma unroll
                for (int kp = 0; kp < D / 32; ++kp) {
                    const int c = kp * 4 + (lane >> 3);
                    const int rr = nt * 8 + (lane & 7);
                    uint32_t b0, b1, b2, b3;
                    ldsm_x4(kb + (c >> 3) * C::HALF_BYTES + sw128(rr, c & 7), b0, b1, b2, b3);
                    mma_bf16_16816(sacc[nt], qa[2 * kp][0], qa[2 * kp][1], qa[2 * kp][2],
                                   qa[2 * kp][3], b0, b1);
                    mma_bf16_16816(sacc[nt], qa[2 * kp + 1][0], qa[2 * kp + 1][1],
                                   qa[2 * kp + 1][2], qa[2 * kp + 1][3], b2, b3);
                }
            }
            // online softmax (log2 units), one head row per lane quad
#pragma unroll
            for (int ht = 0; ht < NHT; ++ht) {
                float mx = kNegInf;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float sv = nt * 8 + 2 * tq + e < held
                                             ? sacc[nt][2 * ht + e] * p.scale_log2
                                             : kNegInf;
                        sacc[nt][2 * ht + e] = sv;
                        mx = fmaxf(mx, sv);
                    }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float m_new = fmaxf(m_run[ht], mx);
                const float msub = m_new == kNegInf ? 0.f : m_new;
                const float alpha = fast_exp2(m_run[ht] - msub);
                float psum = 0.f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float pv = fast_exp2(sacc[nt][2 * ht + e] - msub);
                        sacc[nt][2 * ht + e] = pv;
                        psum += pv;
                    }
                l_run[ht] = l_run[ht] * alpha + psum;
                m_run[ht] = m_new;
                // O^T columns of this lane are heads ht*8 + 2tq and +1
                const float a0 = __shfl_sync(0xffffffffu, alpha, 8 * tq);
                const float a1 = __shfl_sync(0xffffffffu, alpha, 8 * tq + 4);
#pragma unroll
                for (int mt = 0; mt < DK; ++mt) {
                    oacc[ht][mt][0] *= a0;
                    oacc[ht][mt][1] *= a1;
                    oacc[ht][mt][2] *= a0;
                    oacc[ht][mt][3] *= a1;
                }
            }
            // O^T += V^T P^T
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t pb0[NHT], pb1[NHT];
#pragma unroll
                for (int ht = 0; ht < NHT; ++ht) {
                    pb0[ht] = pack_bf16(sacc[2 * ks][2 * ht], sacc[2 * ks][2 * ht + 1]);
                    pb1[ht] = pack_bf16(sacc[2 * ks + 1][2 * ht], sacc[2 * ks + 1][2 * ht + 1]);
                }
                const int jm = lane >> 3;
                const int rr = ks * 16 + ((jm >> 1) << 3) + (lane & 7);
#pragma unroll
                for (int mt = 0; mt < DK; ++mt) {
                    const int c = mt * 2 + (jm & 1);
                    uint32_t a0, a1, a2, a3;
                    ldsm_x4_t(vb + (c >> 3) * C::HALF_BYTES + sw128(rr, c & 7), a0, a1, a2, a3);
#pragma unroll
                    for (int ht = 0; ht < NHT; ++ht)
                        mma_bf16_16816(oacc[ht][mt], a0, a1, a2, a3, pb0[ht], pb1[ht]);
                }
            }
        }
        __syncwarp();
        if (j + NST < nmine && elect_one()) {
            fence_proxy_async_smem();
            issue(j + NST);
        }
    }
    if (consumed < nmine) {  // a wait gave up: let the copies in flight land
        const int last = min(nmine, consumed + NST);
        for (int j = consumed + 1; j < last; ++j)
            mbar_wait_bounded(wbars + 8 * (j % NST), (j / NST) & 1, p.r.dev_error);
    }

#pragma unroll
    for (int ht = 0; ht < NHT; ++ht) {
        l_run[ht] += __shfl_xor_sync(0xffffffffu, l_run[ht], 1);
        l_run[ht] += __shfl_xor_sync(0xffffffffu, l_run[ht], 2);
        if (tq == 0) {
            s_m[warp * kMaxGroup + ht * 8 + gq] = m_run[ht];
            s_l[warp * kMaxGroup + ht * 8 + gq] = l_run[ht];
        }
    }
    float *s_o = reinterpret_cast<float *>(smem);  // [warp][8 heads][ROW]
    float *s_out = reinterpret_cast<float *>(smem + C::OUT_OFF);
#pragma unroll
    for (int ht = 0; ht < NHT; ++ht) {
        __syncthreads();  // the ring is free (ht 0); the last heads are joined (ht 1)
#pragma unroll
        for (int mt = 0; mt < DK; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s_o[(warp * 8 + 2 * tq + (e & 1)) * C::ROW + mt * 16 + gq + (e >> 1) * 8] =
                    oacc[ht][mt][e];
        __syncthreads();
        const int heads = min(8, G - ht * 8);
        for (int i = threadIdx.x; i < heads * (Dh / 4); i += kThreads) {
            const int h = i / (Dh / 4), d = (i - h * (Dh / 4)) * 4, hh = ht * 8 + h;
            const float m0 = s_m[hh], m1 = s_m[kMaxGroup + hh];
            const float M = fmaxf(m0, m1), Ms = M == kNegInf ? 0.f : M;
            const float l0 = s_l[hh], l1 = s_l[kMaxGroup + hh];
            const float f0 = exp2f(m0 - Ms), f1 = exp2f(m1 - Ms);
            // a NaN sum keeps its maximum at -inf: do not lose it to a factor 0
            const float l = (l0 != l0 ? l0 : f0 * l0) + (l1 != l1 ? l1 : f1 * l1);
            const float inv = l == 0.f ? 0.f : 1.f / l;
            if (d == 0) s_lse[hh] = l == 0.f ? kNegInf : Ms + log2f(l);
            const float4 a = *reinterpret_cast<const float4 *>(s_o + h * C::ROW + d);
            const float4 b = *reinterpret_cast<const float4 *>(s_o + (8 + h) * C::ROW + d);
            *reinterpret_cast<float4 *>(s_out + hh * C::ROW + d) =
                make_float4((a.x * f0 + b.x * f1) * inv, (a.y * f0 + b.y * f1) * inv,
                            (a.z * f0 + b.z * f1) * inv, (a.w * f0 + b.w * f1) * inv);
        }
    }
    join_and_store<kThreads>(p, t, g, rank, s_out, C::ROW, s_lse);
}

template <int D, int BS, int NHT>
cudaError_t launch_one(const SparseParams &p, const CUtensorMap *tk, const CUtensorMap *tv,
                       cudaStream_t stream) {
    auto kern = p.hnd ? sparse_decode_kernel<D, BS, NHT, true>
                      : sparse_decode_kernel<D, BS, NHT, false>;
    const int smem = Shape<D, BS>::SMEM_FIXED + p.cap * 4;
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kern), smem);
    if (e != cudaSuccess) return e;
    const int64_t grid = (int64_t)p.r.rows * p.r.num_kv_heads * p.cluster;
    if (grid > 0x7fffffff) return cudaErrorNotSupported;
    return launch_cluster(kern, (unsigned)grid, p.cluster, kThreads, (size_t)smem, stream, p, *tk,
                          *tv);
}

template <int D>
cudaError_t launch_d(const SparseParams &p, int BS, const CUtensorMap *tk, const CUtensorMap *tv,
                     cudaStream_t stream) {
    if (BS == 16)
        return p.r.group <= 8 ? launch_one<D, 16, 1>(p, tk, tv, stream)
                              : launch_one<D, 16, 2>(p, tk, tv, stream);
    return p.r.group <= 8 ? launch_one<D, 32, 1>(p, tk, tv, stream)
                          : launch_one<D, 32, 2>(p, tk, tv, stream);
}

}  // namespace

cudaError_t launch_sparse(const SparseParams &p, int block_size, const CUtensorMap *tmap_k,
                          const CUtensorMap *tmap_v, cudaStream_t stream) {
    const int D = p.r.head_dim;
    if (D <= 64) return launch_d<64>(p, block_size, tmap_k, tmap_v, stream);
    if (D <= 128) return launch_d<128>(p, block_size, tmap_k, tmap_v, stream);
    return launch_d<256>(p, block_size, tmap_k, tmap_v, stream);
}

}  // namespace pkv
