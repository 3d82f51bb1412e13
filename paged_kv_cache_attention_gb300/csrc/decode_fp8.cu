// decode_fp8.cu -- split-KV decode over the 8-bit cache.
//
// The attention of decode.cu (same masks, sink, ALiBi and partitions; see
// there) with key j of a kv head stored as e4m3 codes kc_j and a byte:
//   s_j = sm_scale * 2^ek_j * <q, kc_j> + bias,   o = sum_j p_j 2^ev_j vc_j / l.
//
// HBM bound: 2*(D + 1) bytes per key and kv head, half of the bf16 cache.
// At 6.8 TB/s an SM receives 23 codes per clock, so the instructions spent on a
// code decide whether the kernel keeps up.  A 32-bit word of four codes becomes
// two f16 pairs in two conversions (three with V's byte shuffle), both scales
// stay out of the codes, and the softmax's bookkeeping is skipped while no
// row's maximum grows:
//   * K: the byte, as 2^ek, multiplies the fp32 score of its key;
//   * V: the weight that rounds to f16 is p_j 2^ev_j, as 2^(s_j + ev_j - r) with a
//     reference r of the row's own: the largest s_j + ev_j, less 6.  What a key
//     adds counts, not its scale: a huge V row of hardly any weight costs the others
//     nothing.  f16 keeps 11 bits of every weighted scale down to 2^-20 of the
//     row's largest (an error of 2^-31 of that one below it).  The sum of the p_j
//     alone has the row's largest score as its reference, so each score takes two
//     exponentials;
//   * both references move only when they are exceeded by 9 log2 units (weights
//     stay below 2^15).
// q is scaled per head by a power of two to at most 2^15 and held in f16,
// which is exact for every bf16 value within 2^-28 of the row's largest (and
// off by less than 2^-39 of the largest below that).
//
// The mma fragments follow the bytes: a 32-bit word of an ldmatrix row holds
// four consecutive dims of a key, two pairs, so a k-step of Q K^T takes 16 dims
// in that order (q's fragment is loaded to match); a transposed ldmatrix word
// holds two consecutive dims of two consecutive keys: one byte shuffle and it is
// one even-dim and one odd-dim fragment of O^T += V^T P^T.
//
// CTAs of two warps, each streaming every other stage of the partition (32
// tokens, 64 of a 64-dim head) through its own ring of two stages: K and V by
// TMA (one box per page and 128 dims), the scale bytes by 16-byte cp.async on
// the same barrier.
//
// Measured (GB300): 64 sequences of 512..4096 tokens (uniform), 32/8 heads of 128: 59 us,
// 5.1 TB/s, 76 % of a copy's rate (the bf16 cache takes 108 us), 68 % over five
// log-uniform draws, whose partitions are less even; one draw of 8 of 32K..128K, 64/8
// heads of 64: 120 us, 82 %.  Half as long stages (twice the
// warps) take 69 and 138 us, three or four of them in the ring 71 and 143, twice
// as long ones 72 and 152; partitions of 1024 tokens 65 and 120.  What is
// left is latency between dependent instructions at 2.5 warps per scheduler
// (issue slots 41 % used, tensor pipe 22 %).
#include <cstring>
#include <type_traits>

#include "pkv_sparse.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 2;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxGroup = 16;
constexpr float kWeightExp = 6.f;  // weights are at most 2^kWeightExp * 2^kLazy
constexpr float kLazy = 9.f;     // log2 units a score may exceed its row's reference
constexpr float kNegInf = -INFINITY;

__device__ __forceinline__ int clipped_len(const DecodeParams &p, int b, int block_size,
                                           bool report) {
    const long long cap_blocks = (long long)p.max_blocks_per_seq * block_size;
    const int cap = cap_blocks < p.max_seqlen ? (int)cap_blocks : p.max_seqlen;
    const int L = p.seqlens[b];
    if ((L < 0 || L > cap) && report) flag_error(p.dev_error, PKV_DEVERR_SEQLEN);
    return min(max(L, 0), cap);
}

__device__ __forceinline__ int first_kept(int L, int window_left) {
    return window_left < 0 ? 0 : max(L - 1 - window_left, 0);
}

// Byte offset of 16-byte chunk c of row r in a tile of W-byte rows (W = 64 or
// 128) that TMA wrote with W-byte swizzling.
template <int W>
__device__ __forceinline__ uint32_t swz(uint32_t r, uint32_t c) {
    return W == 128 ? sw128(r, c) : r * 64u + ((c ^ ((r >> 1) & 3u)) << 4);
}

// What a row's slices are multiplied by, for the sum l of its weights relative to
// 2^M; with it the row's lse is stored.  One partition: the output's factor, with
// the sink; else the partial's.
__device__ __forceinline__ float finish_row(const DecodeParams &p, int64_t unit, int hq, float M,
                                            float l, bool first) {
    if (p.num_parts > 1) {
        if (first)
            p.part_lse[unit * p.num_parts + blockIdx.y] = l == 0.f ? kNegInf : M + log2f(l);
        return l == 0.f ? 0.f : 1.f / l;  // NaN stays
    }
    const float sink = p.sink ? p.sink[hq] * kLog2e : kNegInf;
    const float T = fmaxf(M, sink), Ts = T == kNegInf ? 0.f : T;
    const float f = exp2f(M - Ts);
    const float lam = (l != l ? l : l * f) + exp2f(sink - Ts);
    if (first && p.lse_out) p.lse_out[unit] = lam == 0.f ? kNegInf : (Ts + log2f(lam)) * kLn2;
    return lam == 0.f ? 0.f : f / lam;
}

// Store four finished columns: of the output itself when there is one partition,
// else of the partition's partial.
__device__ __forceinline__ void store_row4(const DecodeParams &p, int64_t unit, int d, float4 o) {
    if (p.num_parts > 1)
        *reinterpret_cast<float4 *>(p.part_o + (unit * p.num_parts + blockIdx.y) * p.head_dim +
                                    d) = o;
    else
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + unit * p.head_dim + d) =
            make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
}

template <int D>
struct Shape {
    static constexpr int TOK = D == 64 ? 64 : 32;            // tokens per stage
    static constexpr int NST = 2;                            // stages per warp
    static constexpr int ROWB = D < 128 ? D : 128;           // bytes of a box row
    static constexpr int PARTS = D / ROWB;                   // boxes across the head size
    static constexpr int PART_BYTES = TOK * ROWB;
    static constexpr int KV_BYTES = PARTS * PART_BYTES;      // K (or V) of one stage
    static constexpr int RING = kWarps * NST * 2 * KV_BYTES;
    static constexpr int SCALE_OFF = RING;                   // [warp][stage][K, V][TOK] bytes
    static constexpr int FACT_OFF = SCALE_OFF + kWarps * NST * 2 * TOK;  // [warp][K, V][TOK] f32
    static constexpr int BAR_OFF = FACT_OFF + kWarps * 2 * TOK * 4;
    static constexpr int M_OFF = BAR_OFF + kWarps * NST * 8;
    static constexpr int L_OFF = M_OFF + kWarps * kMaxGroup * 4;
    static constexpr int R_OFF = L_OFF + kWarps * kMaxGroup * 4;
    static constexpr int BLK_OFF = R_OFF + kWarps * kMaxGroup * 4;
    static constexpr int SMEM_FIXED = 1024 + BLK_OFF;        // + the partition's block ids
    static_assert(kWarps * 8 * D * 4 <= RING, "merge scratch must fit in the ring");
    static_assert((kWarps * 8 + kMaxGroup) * D * 4 <= RING, "and the outputs behind it");
};

// The same attention over lists of pages (sparse_decode.cu): the keys are the rows
// of the pages that a CTA of a cluster takes of a row's list, one after another.
// Measured: 8 rows of 256 pages of 16, 8 kv heads of 64: 14.3 us (clusters of 8; 70 us in
// one CTA per row and kv head), 35 % of a copy's rate; 16 pages a warp, four stages, are
// too few to hide the list, the first loads and the join.
struct SparseFp8Params {
    DecodeFp8Params dense;  // what both have: q, pools, tables, shapes (no window, no ALiBi)
    SparseParams s;
};

__device__ __forceinline__ const DecodeFp8Params &dense_params(const DecodeFp8Params &p) {
    return p;
}
__device__ __forceinline__ const DecodeFp8Params &dense_params(const SparseFp8Params &p) {
    return p.dense;
}

template <int D, int BS, int NHT, bool HND, typename P>
__global__ void __launch_bounds__(kThreads)
decode_fp8_kernel(const P params, const __grid_constant__ CUtensorMap tmk,
                  const __grid_constant__ CUtensorMap tmv) {
    constexpr bool SPARSE = std::is_same<P, SparseFp8Params>::value;
    using C = Shape<D>;
    constexpr int NST = C::NST, TOK = C::TOK;
    constexpr int BR = BS < TOK ? BS : TOK;  // tokens per box: a page, or a stage's part of one
    constexpr int NC = D / 16;      // 16-dim chunks
    constexpr int NT = TOK / 8;     // 8-token tiles
    constexpr int NCP = TOK / 16;   // 16-byte pieces of a stage's K (or V) scale bytes
    const DecodeFp8Params &pp = dense_params(params);
    const DecodeParams &p = pp.d;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);  // 1024-aligned
    int *s_blk = reinterpret_cast<int *>(smem + C::BLK_OFF);
    float *s_m = reinterpret_cast<float *>(smem + C::M_OFF);
    float *s_l = reinterpret_cast<float *>(smem + C::L_OFF);
    float *s_r = reinterpret_cast<float *>(smem + C::R_OFF);

    // no early trigger: merge CTAs that wait on the SMs cost more (2 %) than
    // their launch latency
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.group, Dh = p.head_dim;
    int g = blockIdx.x, b = blockIdx.z;  // kv head; sequence, or row
    int rank = 0, L = 0, tok_lo = 0, tok_hi = 0;
    const int32_t *list = nullptr;       // SPARSE: this CTA's entries
    const int32_t *bt = nullptr;
    auto check = [&] {
        if constexpr (SPARSE) {
            const RowParams &r = params.s.r;
            if (g == 0 && rank == 0)
                check_offsets(r, b + (int64_t)threadIdx.x * r.rows, (int64_t)kThreads * r.rows);
        }
    };
    if constexpr (SPARSE) {
        const SparseParams &sp = params.s;
        rank = sp.cluster > 1 ? (int)cluster_rank() : 0;
        const int64_t unit = blockIdx.x / (unsigned)sp.cluster;
        b = (int)(unit / p.num_kv_heads);
        g = (int)(unit % p.num_kv_heads);
        int r, keys, count;
        if (!row_request(sp.r, b, BS, g == 0 && rank == 0 && threadIdx.x == 0, r, keys, count))
            return check();
        keys = max(keys, 0);
        const int npages = (keys + BS - 1) / BS;
        list = sp.pages + unit * sp.top_k;
        const int n = list_length<kThreads>(list, sp.top_k, npages, p.dev_error, rank == 0,
                                            reinterpret_cast<int *>(s_m));
        // pages of whole stages, so that every CTA's first stage starts with one of its own
        constexpr int U = TOK > BS ? TOK / BS : 1;
        const int per = ((n + sp.cluster - 1) / sp.cluster + U - 1) / U * U;
        const int lo = min(rank * per, n), mine = min(per, n - lo);
        list += lo;
        tok_hi = mine * BS;
        if (mine > 0 && list[mine - 1] == npages - 1) tok_hi -= npages * BS - keys;
        bt = p.block_table + (int64_t)r * p.max_blocks_per_seq;
    } else {
        L = clipped_len(p, b, BS, blockIdx.y == 0 && g == 0 && threadIdx.x == 0);
        const int start = first_kept(L, p.window_left);
        const int part = start / p.partition_size + blockIdx.y;
        tok_lo = max(part * p.partition_size, start);
        tok_hi = min((part + 1) * p.partition_size, L);
        bt = p.block_table + (int64_t)b * p.max_blocks_per_seq;
    }
    const int64_t unit0 = (int64_t)b * p.num_qo_heads + g * G;
    if (!SPARSE && tok_lo >= tok_hi) {  // this slot holds no attended key
        if (p.num_parts == 1)
            for (int i = threadIdx.x; i < G * (Dh / 4); i += kThreads) {
                const int h = i / (Dh / 4), d = (i - h * (Dh / 4)) * 4;
                finish_row(p, unit0 + h, g * G + h, kNegInf, 0.f, d == 0);
                store_row4(p, unit0 + h, d, make_float4(0.f, 0.f, 0.f, 0.f));
            }
        return;
    }

    // stages start at multiples of TOK; pages of the range
    const int st_lo = tok_lo / TOK;
    const int nst = SPARSE ? (tok_hi + TOK - 1) / TOK : (tok_hi - 1) / TOK - st_lo + 1;
    const int pg_lo = st_lo * TOK / BS, pg_first = tok_lo / BS;
    const int pg_last = SPARSE && tok_hi == 0 ? -1 : (tok_hi - 1) / BS;

    const uint32_t ring = smem_u32(smem);
    const uint32_t bars = ring + C::BAR_OFF;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kWarps * NST; ++i) mbar_init(bars + 8 * i, 1 + 2 * NCP);
        fence_barrier_init();
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    const int pg_end = ((st_lo + nst) * TOK - 1) / BS;  // the last stage's last page
    for (int page = pg_lo + threadIdx.x; page <= pg_end; page += kThreads) {
        int id = -1;
        if (page >= pg_first && page <= pg_last) {  // else: no attended key, not read
            id = bt[SPARSE ? list[page] : page];
            if (id < 0 || id >= p.num_blocks) {
                flag_error(p.dev_error, PKV_DEVERR_BLOCK_ID);
                id = -1;
            }
        }
        s_blk[page - pg_lo] = id;
    }
    __syncthreads();

    const int nmine = nst > warp ? (nst - warp + kWarps - 1) / kWarps : 0;
    const uint32_t wring = ring + warp * NST * 2 * C::KV_BYTES;
    const uint32_t wbars = bars + warp * NST * 8;
    const uint32_t wscale = ring + C::SCALE_OFF + warp * NST * 2 * TOK;
    float *wfact = reinterpret_cast<float *>(smem + C::FACT_OFF) + warp * 2 * TOK;
    const uint64_t policy = l2_policy_evict_first();

    // Stage j of this warp: lane 0 asks TMA for the boxes, the first lanes copy
    // the scale bytes, 16 K or V bytes each.
    auto issue = [&](int j) {
        const int s = j % NST;
        const uint32_t bar = wbars + 8 * s;
        const int first = (st_lo + warp + j * kWarps) * TOK;  // the stage's first token
        if (elect_one()) {
            int id[TOK / BR];
            uint32_t bytes = 0;
#pragma unroll
            for (int q = 0; q < TOK / BR; ++q) {
                id[q] = s_blk[(first + q * BR) / BS - pg_lo];
                if (id[q] >= 0) bytes += 2 * C::PARTS * BR * C::ROWB;
            }
            mbar_arrive_expect_tx(bar, bytes);
            const uint32_t dst = wring + s * 2 * C::KV_BYTES;
#pragma unroll
            for (int q = 0; q < TOK / BR; ++q) {
                if (id[q] < 0) continue;
                const int off = (first + q * BR) % BS;
                const int cy = HND ? off : g;
                const int cz = HND ? id[q] * p.num_kv_heads + g : id[q] * BS + off;
#pragma unroll
                for (int h = 0; h < C::PARTS; ++h) {
                    const uint32_t o = dst + h * C::PART_BYTES + q * BR * C::ROWB;
                    tma_load_3d_hint(o, &tmk, bar, h * 128, cy, cz, policy);
                    tma_load_3d_hint(o + C::KV_BYTES, &tmv, bar, h * 128, cy, cz, policy);
                }
            }
        }
        if (lane < 2 * NCP) {
            const int isv = lane / NCP, t = first + (lane % NCP) * 16;
            const int id = s_blk[t / BS - pg_lo];
            if (id >= 0)
                cp_async16(wscale + s * 2 * TOK + isv * TOK + (lane % NCP) * 16,
                           (isv ? pp.v_scale : pp.k_scale) +
                               ((int64_t)id * p.num_kv_heads + g) * BS + t % BS);
            cp_async_arrive(bar);
        }
    };
    for (int j = 0; j < NST && j < nmine; ++j) issue(j);
    check();

    // q as the A operand: row = head, 16 dims per k-step in the byte order.  A
    // negative sm_scale goes into q, so that scores grow with the products.
    const int gq = lane >> 2, tq = lane & 3;
    const __nv_bfloat16 *qb = static_cast<const __nv_bfloat16 *>(p.q) + unit0 * Dh;
    uint32_t qa[NHT][NC][2];
    float rowf[NHT];
#pragma unroll
    for (int ht = 0; ht < NHT; ++ht) {
        const int h = ht * 8 + gq;
        uint2 w[NC];
        uint32_t amax = 0;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            w[c] = make_uint2(0u, 0u);
            if (h < G && c * 16 < Dh)
                w[c] = *reinterpret_cast<const uint2 *>(qb + h * Dh + c * 16 + 4 * tq);
            const uint32_t v[2] = {w[c].x, w[c].y};
#pragma unroll
            for (int i = 0; i < 2; ++i)
                amax = max(amax, max(v[i] & 0x7fffu, (v[i] >> 16) & 0x7fffu));
        }
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // largest magnitude 2^E..2^(E+1): times 2^(14 - E)
        const int E = max((int)(amax >> 7) - 127, -100);
        const uint32_t neg = p.scale_log2 < 0.f ? 0x80000000u : 0u;
        const float f = __uint_as_float(((uint32_t)(127 + 14 - E) << 23) | neg);
        rowf[ht] = fabsf(p.scale_log2) * __uint_as_float((uint32_t)(127 + E - 14) << 23);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            qa[ht][c][0] = pack_f16(__uint_as_float(w[c].x << 16) * f,
                                    __uint_as_float(w[c].x & 0xffff0000u) * f);
            qa[ht][c][1] = pack_f16(__uint_as_float(w[c].y << 16) * f,
                                    __uint_as_float(w[c].y & 0xffff0000u) * f);
        }
    }

    float oacc[NHT][NC][4];
    float m_ref[NHT], r_ref[NHT], l_run[NHT], al2[NHT];
    bool head_ok[NHT];
#pragma unroll
    for (int ht = 0; ht < NHT; ++ht) {
        m_ref[ht] = r_ref[ht] = kNegInf;
        l_run[ht] = 0.f;
        head_ok[ht] = ht * 8 + gq < G;
        al2[ht] = (p.alibi && head_ok[ht]) ? p.alibi[g * G + ht * 8 + gq] * kLog2e : 0.f;
#pragma unroll
        for (int mt = 0; mt < NC; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) oacc[ht][mt][e] = 0.f;
    }
    const int qpos = L - 1;

    int consumed = 0;
    for (int j = 0; j < nmine; ++j) {
        const int i = warp + j * kWarps;
        const int s = j % NST;
        if (!warp_wait_bounded(wbars + 8 * s, (j / NST) & 1, p.dev_error)) break;
        consumed = j + 1;
        const uint32_t kb = wring + s * 2 * C::KV_BYTES, vb = kb + C::KV_BYTES;
        const uint8_t *sc = smem + C::SCALE_OFF + (warp * NST + s) * 2 * TOK;
        const int tok0 = (st_lo + i) * TOK;
        // lane = token (and token + 32): is it attended, its factors
        constexpr int NW = (TOK + 31) / 32;
        uint32_t okm[NW];
        bool full = true;
#pragma unroll
        for (int h = 0; h < NW; ++h) {
            const int t = tok0 + h * 32 + lane;
            const bool ok = h * 32 + lane < TOK && t >= tok_lo && t < tok_hi &&
                            s_blk[t / BS - pg_lo] >= 0;
            okm[h] = __ballot_sync(0xffffffffu, ok);
            full = full && okm[h] == (TOK < 32 ? (1u << (TOK % 32)) - 1u : 0xffffffffu);
        }
#pragma unroll
        for (int h = 0; h < NW; ++h) {
            const int t = h * 32 + lane;
            if (TOK < 32 && t >= TOK) break;
            const uint32_t vbyte = sc[TOK + t];
            wfact[t] = scale_value(sc[t]);
            // an unattended row's byte may be anything, but finite here: it meets a
            // score of -inf
            wfact[TOK + t] = vbyte == kScaleNaN && ((okm[h] >> lane) & 1u)
                                 ? __uint_as_float(0x7fffffffu)
                                 : (float)((int)vbyte - 127);
        }
        if (!full) {
            // unattended V rows may hold any bits: zero them, so that a zero
            // weight never meets a NaN code
            for (int e = lane; e < C::PARTS * TOK * (C::ROWB / 16); e += 32) {
                const int h = e / (TOK * (C::ROWB / 16)), r = (e / (C::ROWB / 16)) % TOK;
                const int c = e % (C::ROWB / 16);
                if (!((okm[r / 32] >> (r % 32)) & 1u))
                    st_shared_zero16(vb + h * C::PART_BYTES + swz<C::ROWB>(r, c));
            }
        }
        __syncwarp();

        float sacc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) sacc[nt][e] = 0.f;
#pragma unroll
            for (int c4 = 0; c4 < NC / 4; ++c4) {
                const int c = c4 * 4 + (lane >> 3);
                const int r = nt * 8 + (lane & 7);
                uint32_t w[4];
                ldsm_x4(kb + (c >> 3) * C::PART_BYTES + swz<C::ROWB>(r, c & 7), w[0], w[1], w[2],
                        w[3]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t b0, b1;
                    e4m3_to_f16(w[k], b0, b1);
                    mma_f16_16816(sacc[nt], qa[0][c4 * 4 + k][0],
                                  NHT > 1 ? qa[NHT - 1][c4 * 4 + k][0] : 0u,
                                  qa[0][c4 * 4 + k][1],
                                  NHT > 1 ? qa[NHT - 1][c4 * 4 + k][1] : 0u, b0, b1);
                }
            }
        }
        // online softmax (log2 units), one head row per lane quad
        float ao[NHT];
        bool moved = false;
#pragma unroll
        for (int ht = 0; ht < NHT; ++ht) {
            float rf = rowf[ht];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float2 kf = *reinterpret_cast<const float2 *>(wfact + nt * 8 + 2 * tq);
                sacc[nt][2 * ht] *= kf.x;
                sacc[nt][2 * ht + 1] *= kf.y;
            }
            if (!full || (!SPARSE && p.alibi)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int t = nt * 8 + 2 * tq + e;
                        const bool ok = (okm[t / 32] >> (t % 32)) & 1u;
                        sacc[nt][2 * ht + e] =
                            ok ? fmaf(sacc[nt][2 * ht + e], rf,
                                      al2[ht] * (float)(tok0 + t - qpos))
                               : kNegInf;
                    }
                rf = 1.f;  // the scores are complete
            }
            float mx = kNegInf, rx = kNegInf;  // the largest score, and score + V exponent
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float2 ev = *reinterpret_cast<const float2 *>(wfact + TOK + nt * 8 + 2 * tq);
                mx = fmax3(mx, sacc[nt][2 * ht], sacc[nt][2 * ht + 1]);
                rx = fmax3(rx, fmaf(sacc[nt][2 * ht], rf, ev.x),
                           fmaf(sacc[nt][2 * ht + 1], rf, ev.y));
            }
            mx *= rf;
            rx -= kWeightExp;
            if (!head_ok[ht]) mx = rx = kNegInf;
            ao[ht] = 1.f;
            if (__any_sync(0xffffffffu, mx > m_ref[ht] + kLazy || rx > r_ref[ht] + kLazy)) {
#pragma unroll
                for (int off = 1; off < 4; off <<= 1) {
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                    rx = fmaxf(rx, __shfl_xor_sync(0xffffffffu, rx, off));
                }
                const float m_new = fmaxf(m_ref[ht], mx), r_new = fmaxf(r_ref[ht], rx);
                ao[ht] = r_new == kNegInf ? 1.f : fast_exp2(r_ref[ht] - r_new);
                l_run[ht] *= m_new == kNegInf ? 1.f : fast_exp2(m_ref[ht] - m_new);
                m_ref[ht] = m_new;
                r_ref[ht] = r_new;
                moved = true;
            }
            const float msub = m_ref[ht] == kNegInf ? 0.f : m_ref[ht];
            const float rsub = r_ref[ht] == kNegInf ? 0.f : r_ref[ht];
            float p0 = 0.f, p1 = 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float2 ev = *reinterpret_cast<const float2 *>(wfact + TOK + nt * 8 + 2 * tq);
                const float x = sacc[nt][2 * ht], y = sacc[nt][2 * ht + 1];
                p0 += fast_exp2(fmaf(x, rf, -msub));
                p1 += fast_exp2(fmaf(y, rf, -msub));
                sacc[nt][2 * ht] = fast_exp2(fmaf(x, rf, ev.x) - rsub);
                sacc[nt][2 * ht + 1] = fast_exp2(fmaf(y, rf, ev.y) - rsub);
            }
            l_run[ht] += p0 + p1;
        }
        if (moved) {  // O^T columns of this lane are heads ht*8 + 2tq and +1
#pragma unroll
            for (int ht = 0; ht < NHT; ++ht) {
                const float a0 = __shfl_sync(0xffffffffu, ao[ht], 8 * tq);
                const float a1 = __shfl_sync(0xffffffffu, ao[ht], 8 * tq + 4);
#pragma unroll
                for (int mt = 0; mt < NC; ++mt) {
                    oacc[ht][mt][0] *= a0;
                    oacc[ht][mt][1] *= a1;
                    oacc[ht][mt][2] *= a0;
                    oacc[ht][mt][3] *= a1;
                }
            }
        }
        // O^T += V^T P^T
#pragma unroll
        for (int ks = 0; ks < NT / 2; ++ks) {
            uint32_t pb0[NHT], pb1[NHT];
#pragma unroll
            for (int ht = 0; ht < NHT; ++ht) {
                pb0[ht] = pack_f16(sacc[2 * ks][2 * ht], sacc[2 * ks][2 * ht + 1]);
                pb1[ht] = pack_f16(sacc[2 * ks + 1][2 * ht], sacc[2 * ks + 1][2 * ht + 1]);
            }
            const int jm = lane >> 3;
            const int r = ks * 16 + ((jm & 1) << 3) + (lane & 7);
#pragma unroll
            for (int c2 = 0; c2 < NC / 2; ++c2) {
                const int c = c2 * 2 + (jm >> 1);
                uint32_t w[4];  // (keys 0-7, 8-15) of chunk 2*c2, then of 2*c2 + 1
                ldsm_x4_t(vb + (c >> 3) * C::PART_BYTES + swz<C::ROWB>(r, c & 7), w[0], w[1],
                          w[2], w[3]);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t a0, a1, a2, a3;  // even dims, odd dims of keys 0-7 and 8-15
                    e4m3_to_f16(__byte_perm(w[2 * k], 0u, 0x3120), a0, a1);
                    e4m3_to_f16(__byte_perm(w[2 * k + 1], 0u, 0x3120), a2, a3);
#pragma unroll
                    for (int ht = 0; ht < NHT; ++ht)
                        mma_f16_16816(oacc[ht][c2 * 2 + k], a0, a1, a2, a3, pb0[ht], pb1[ht]);
                }
            }
        }
        __syncwarp();
        if (j + NST < nmine) {
            fence_proxy_async_smem();
            issue(j + NST);
        }
    }
    if (consumed < nmine) {  // a wait gave up: let the copies in flight land
        const int last = min(nmine, consumed + NST);
        for (int j = consumed + 1; j < last; ++j)
            mbar_wait_bounded(wbars + 8 * (j % NST), (j / NST) & 1, p.dev_error);
    }

#pragma unroll
    for (int ht = 0; ht < NHT; ++ht) {
        l_run[ht] += __shfl_xor_sync(0xffffffffu, l_run[ht], 1);
        l_run[ht] += __shfl_xor_sync(0xffffffffu, l_run[ht], 2);
        if (tq == 0) {
            s_m[warp * kMaxGroup + ht * 8 + gq] = m_ref[ht];
            s_l[warp * kMaxGroup + ht * 8 + gq] = l_run[ht];
            s_r[warp * kMaxGroup + ht * 8 + gq] = r_ref[ht];
        }
    }
    float *s_o = reinterpret_cast<float *>(smem);  // [warp][8 heads][D]
    // SPARSE: the CTA's outputs [16 heads][D] behind it, and its heads' lse (the stages'
    // scale bytes are free)
    float *s_out = s_o + kWarps * 8 * D;
    float *s_lse = reinterpret_cast<float *>(smem + C::FACT_OFF);
#pragma unroll
    for (int ht = 0; ht < NHT; ++ht) {
        __syncthreads();  // the ring is free (ht 0); the last heads are written (ht 1)
#pragma unroll
        for (int mt = 0; mt < NC; ++mt)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                *reinterpret_cast<float2 *>(s_o + (warp * 8 + 2 * tq + c) * D + mt * 16 +
                                            2 * gq) =
                    make_float2(oacc[ht][mt][c], oacc[ht][mt][2 + c]);
        __syncthreads();
        const int heads = min(8, G - ht * 8);
        for (int i = threadIdx.x; i < heads * (Dh / 4); i += kThreads) {
            const int h = i / (Dh / 4), d = (i - h * (Dh / 4)) * 4, hh = ht * 8 + h;
            const float m0 = s_m[hh], m1 = s_m[kMaxGroup + hh];
            const float M = fmaxf(m0, m1), Ms = M == kNegInf ? 0.f : M;
            const float l0 = s_l[hh], l1 = s_l[kMaxGroup + hh];
            // a NaN sum keeps its reference at -inf: do not lose it to a factor 0
            const float l = (l0 != l0 ? l0 : exp2f(m0 - Ms) * l0) +
                            (l1 != l1 ? l1 : exp2f(m1 - Ms) * l1);
            float mul;
            if constexpr (SPARSE) {
                mul = l == 0.f ? 0.f : 1.f / l;  // NaN stays
                if (d == 0) s_lse[hh] = l == 0.f ? kNegInf : M + log2f(l);
            } else {
                mul = finish_row(p, unit0 + hh, g * G + hh, M, l, d == 0);
            }
            // O is relative to 2^r: 2^(r - M) in two halves, because r holds V's
            // exponent and the whole may leave fp32's range where the result does not
            const float h0 = exp2f(0.5f * (s_r[hh] - Ms));
            const float h1 = exp2f(0.5f * (s_r[kMaxGroup + hh] - Ms));
            const float4 a = *reinterpret_cast<const float4 *>(s_o + h * D + d);
            const float4 c = *reinterpret_cast<const float4 *>(s_o + (8 + h) * D + d);
            auto join = [&](float x, float y) {
                return x * mul * h0 * h0 + y * mul * h1 * h1;
            };
            const float4 o = make_float4(join(a.x, c.x), join(a.y, c.y), join(a.z, c.z),
                                         join(a.w, c.w));
            if constexpr (SPARSE)
                *reinterpret_cast<float4 *>(s_out + hh * D + d) = o;
            else
                store_row4(p, unit0 + hh, d, o);
        }
    }
    if constexpr (SPARSE) join_and_store<kThreads>(params.s, b, g, rank, s_out, D, s_lse);
}

// ---------------------------------------------------------------------------
// merge of the partitions, sink, cast: one warp per (sequence, query head)
// ---------------------------------------------------------------------------
constexpr int kMergeThreads = 128;

// out = sum_i 2^(lse_i - M) o_i / (sum_i 2^(lse_i - M) + 2^(sink - M)).
// SPLIT warps share a row's partitions (long sequences of few heads).
template <int SPLIT>
__global__ void __launch_bounds__(kMergeThreads)
merge_fp8_kernel(const DecodeParams p, int D, int block_size) {
    constexpr int kUnits = kMergeThreads / 32 / SPLIT;
    __shared__ float s_acc[SPLIT > 1 ? kMergeThreads / 32 : 1][256];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t unit = (int64_t)blockIdx.x * kUnits + warp / SPLIT;
    const bool live = unit < (int64_t)p.batch * p.num_qo_heads;
    if (SPLIT == 1 && !live) return;
    const int b = live ? (int)(unit / p.num_qo_heads) : 0;
    const int h = live ? (int)(unit % p.num_qo_heads) : 0;
    const int L = clipped_len(p, b, block_size, false);
    const int P = p.partition_size, start = first_kept(L, p.window_left);
    const int n = live && L > 0 ? (L - 1) / P - start / P + 1 : 0;
    const int64_t base = ((int64_t)b * p.num_qo_heads + h) * p.num_parts;
    const float *lp = p.part_lse + base;
    const float sink = p.sink ? p.sink[h] * kLog2e : kNegInf;
    float M = sink;
    for (int i = lane; i < n; i += 32) M = fmaxf(M, lp[i]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    const float Ms = M == kNegInf ? 0.f : M;
    float sum = 0.f;
    for (int i = lane; i < n; i += 32) sum += exp2f(lp[i] - Ms);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    const float lam = sum + exp2f(sink - Ms);
    const float inv = lam > 0.f ? 1.f / lam : (lam == 0.f ? 0.f : lam);
    // lane l sums columns 4l .. 4l+3 (and 128 + 4l .. for D = 256)
    float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    const int c0 = 4 * lane;
    const float *po = p.part_o + base * D;
#pragma unroll 4
    for (int i = warp % SPLIT; i < n; i += SPLIT) {
        const float w = exp2f(lp[i] - Ms) * inv;
        const float *row = po + (int64_t)i * D;
        if (c0 < D) {
            const float4 v = *reinterpret_cast<const float4 *>(row + c0);
            acc[0].x = fmaf(w, v.x, acc[0].x);
            acc[0].y = fmaf(w, v.y, acc[0].y);
            acc[0].z = fmaf(w, v.z, acc[0].z);
            acc[0].w = fmaf(w, v.w, acc[0].w);
        }
        if (c0 + 128 < D) {
            const float4 v = *reinterpret_cast<const float4 *>(row + 128 + c0);
            acc[1].x = fmaf(w, v.x, acc[1].x);
            acc[1].y = fmaf(w, v.y, acc[1].y);
            acc[1].z = fmaf(w, v.z, acc[1].z);
            acc[1].w = fmaf(w, v.w, acc[1].w);
        }
    }
    if (SPLIT > 1) {
        *reinterpret_cast<float4 *>(&s_acc[warp][c0]) = acc[0];
        *reinterpret_cast<float4 *>(&s_acc[warp][128 + c0]) = acc[1];
        __syncthreads();
        if (warp % SPLIT != 0 || !live) return;
#pragma unroll
        for (int w = 1; w < SPLIT; ++w)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float4 v =
                    *reinterpret_cast<const float4 *>(&s_acc[warp + w][k * 128 + c0]);
                acc[k].x += v.x;
                acc[k].y += v.y;
                acc[k].z += v.z;
                acc[k].w += v.w;
            }
    }
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + unit * D;
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (c0 + k * 128 < D)
            *reinterpret_cast<uint2 *>(out + k * 128 + c0) =
                make_uint2(pack_bf16(acc[k].x, acc[k].y), pack_bf16(acc[k].z, acc[k].w));
    if (p.lse_out && lane == 0)
        p.lse_out[unit] = lam == 0.f ? kNegInf : (Ms + log2f(lam)) * kLn2;
}

cudaError_t launch_merge_fp8(const DecodeParams &p, int D, int BS, cudaStream_t stream) {
    const int64_t units = (int64_t)p.batch * p.num_qo_heads;
    if (p.num_parts > 16) {
        return launch_pdl(merge_fp8_kernel<4>, dim3((unsigned)units), dim3(kMergeThreads), 0,
                          stream, p, D, BS);
    }
    constexpr int kUnits = kMergeThreads / 32;
    return launch_pdl(merge_fp8_kernel<1>, dim3((unsigned)((units + kUnits - 1) / kUnits)),
                      dim3(kMergeThreads), 0, stream, p, D, BS);
}

template <int D, int BS, int NHT>
cudaError_t launch_one(const DecodeFp8Params &p, const CUtensorMap *tk, const CUtensorMap *tv,
                       cudaStream_t stream) {
    using C = Shape<D>;
    auto kern = p.d.hnd ? decode_fp8_kernel<D, BS, NHT, true, DecodeFp8Params>
                        : decode_fp8_kernel<D, BS, NHT, false, DecodeFp8Params>;
    // the pages of a partition, and those beside it in its first and last stage
    const int smem = C::SMEM_FIXED + (p.d.partition_size / BS + 6) * 4;
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kern), smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(p.d.num_kv_heads, p.d.num_parts, p.d.batch), dim3(kThreads),
                      (size_t)smem, stream, p, *tk, *tv);
}

template <int D, int BS, int NHT>
cudaError_t launch_one(const SparseFp8Params &p, const CUtensorMap *tk, const CUtensorMap *tv,
                       cudaStream_t stream) {
    using C = Shape<D>;
    auto kern = p.s.hnd ? decode_fp8_kernel<D, BS, NHT, true, SparseFp8Params>
                        : decode_fp8_kernel<D, BS, NHT, false, SparseFp8Params>;
    // the CTA's entries, rounded up to a stage
    const int smem = C::SMEM_FIXED + (p.s.cap + 8) * 4;
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kern), smem);
    if (e != cudaSuccess) return e;
    const int64_t grid = (int64_t)p.s.r.rows * p.s.r.num_kv_heads * p.s.cluster;
    if (grid > 0x7fffffff) return cudaErrorNotSupported;
    return launch_cluster(kern, (unsigned)grid, p.s.cluster, kThreads, (size_t)smem, stream, p,
                          *tk, *tv);
}

template <int D, typename P>
cudaError_t launch_d(const P &p, int group, int BS, const CUtensorMap *tk, const CUtensorMap *tv,
                     cudaStream_t stream) {
    if (BS == 16)
        return group <= 8 ? launch_one<D, 16, 1>(p, tk, tv, stream)
                          : launch_one<D, 16, 2>(p, tk, tv, stream);
    return group <= 8 ? launch_one<D, 32, 1>(p, tk, tv, stream)
                      : launch_one<D, 32, 2>(p, tk, tv, stream);
}

template <typename P>
cudaError_t launch_any(const P &p, int D, int group, int BS, const CUtensorMap *tk,
                       const CUtensorMap *tv, cudaStream_t stream) {
    if (D <= 64) return launch_d<64>(p, group, BS, tk, tv, stream);
    if (D <= 128) return launch_d<128>(p, group, BS, tk, tv, stream);
    return launch_d<256>(p, group, BS, tk, tv, stream);
}

}  // namespace

// Tokens per TMA box: see Shape.
int decode_fp8_box_rows(int head_dim, int block_size) {
    const int tok = head_dim <= 64 ? Shape<64>::TOK : Shape<128>::TOK;
    static_assert(Shape<128>::TOK == Shape<256>::TOK, "one rule for both");
    return block_size < tok ? block_size : tok;
}

cudaError_t launch_decode_fp8(const DecodeFp8Params &p, const pkv_cache_desc &cache,
                              const CUtensorMap *tmap_k, const CUtensorMap *tmap_v,
                              cudaStream_t stream) {
    const int D = cache.head_dim, BS = cache.block_size;
    const cudaError_t e = launch_any(p, D, p.d.group, BS, tmap_k, tmap_v, stream);
    if (e != cudaSuccess || p.d.num_parts == 1) return e;
    return launch_merge_fp8(p.d, D, BS, stream);
}

cudaError_t launch_sparse_fp8(const SparseParams &s, int block_size, const CUtensorMap *tmap_k,
                              const CUtensorMap *tmap_v, cudaStream_t stream) {
    SparseFp8Params p;
    std::memset(&p, 0, sizeof p);
    p.s = s;
    DecodeParams &d = p.dense.d;
    d.q = s.q;
    d.block_table = s.r.block_table;
    d.dev_error = s.r.dev_error;
    d.num_blocks = s.r.num_blocks;
    d.num_kv_heads = s.r.num_kv_heads;
    d.group = s.r.group;
    d.num_qo_heads = s.r.num_kv_heads * s.r.group;
    d.max_blocks_per_seq = s.r.max_blocks_per_seq;
    d.head_dim = s.r.head_dim;
    d.window_left = -1;
    d.num_parts = 1;
    d.scale_log2 = s.scale_log2;
    p.dense.k_scale = s.k_scale;
    p.dense.v_scale = s.v_scale;
    return launch_any(p, s.r.head_dim, s.r.group, block_size, tmap_k, tmap_v, stream);
}

}  // namespace pkv
