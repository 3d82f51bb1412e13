// tree.cu -- attention of a tree of drafted tokens over the paged cache.
//
// Request r has q_len drafted tokens, already written to its pages as the
// last q_len of its L positions; ctx = L - q_len.  Draft i sees context key
// j < ctx, and draft key ctx + n iff bit n of its mask is set:
//   pos(j) = j for a context key, ctx + depth[n] for draft key n
//   keep key j iff visible and (window_left < 0 or pos(j) >= qpos - window_left),
//   qpos = ctx + depth[i]
//   s = sm_scale * <q, k_j> + alibi[h] * (pos(j) - qpos);  o = softmax(s, sink) V.
//
// What bounds it: a decode step with q_len queries reads K and V once, so up
// to about 128 rows (drafts x heads of a group) per kv head it is HBM bound;
// beyond that the tensor cores are.  mma.sync would be the limit from 64 rows
// on, so the products run on tcgen05: the (draft, head) rows of one kv head are
// packed into tiles of 128 rows (M = 128), and because a 128-key step costs
// the tensor core about half the time its 64 KB of bf16 K and V take from HBM,
// the padding of small trees is free.
//
// Over 8-bit pools the codes become f16 tiles as they are; K's scale multiplies
// its column of S and V's scale its column of P, both in fp32, and q is scaled
// per row by a power of two into f16 (decode_fp8.cu gives the error bounds).
//
// One CTA per (kv head, row tile, partition, request): split-KV over
// partitions of a multiple of 128 keys and a merge kernel, or one partition and
// a direct store.  Warps 0-3: softmax, one row per thread; warp 4: TMA; warp 5:
// MMA issue; with 8-bit pools four more warps turn codes into f16 tiles.
//   S = Q K^T -> TMEM; the softmax takes its row into registers, writes P (16
//   bits) over S; O += P V with P from TMEM.  O is rescaled only when a row's
//   maximum grows by more than 2^4.  bf16 pools up to D = 128 run two CTAs
//   per SM (256 TMEM columns, 97 KB each) that cover each other's softmax;
//   the others run one CTA with two S buffers.
// Tiles that hold anything a row does not see (the drafts, the window's edge,
// the ends of the partition) take a general path with 128 visibility bits per
// row; V rows behind the end are zeroed, and a V row with a non-finite value
// is zeroed too and reaches, as NaN, only the rows that see it.
#include "pkv_fp8.cuh"
#include "pkv_tcgen05.cuh"

namespace pkv {

namespace {

constexpr int kTile = 128;      // rows and keys per tile
constexpr int kMaxDraft = 256;
constexpr float kNegInf = -INFINITY;
constexpr float kLazy = 4.f;    // log2 units a maximum may grow before O is rescaled
constexpr int kWeightExp = 10;  // f16 weights stay below 2^(kWeightExp + kLazy)

template <int T, bool KV8>
struct Cfg {
    static constexpr int HALVES = T / 64;
    static constexpr int HALF = kTile * 128;         // 128 rows of 64 dims
    static constexpr int TILE = HALVES * HALF;
    static constexpr int CTAS = (!KV8 && T <= 128) ? 2 : 1;
    static constexpr int NS = CTAS == 2 ? 1 : 2;     // S buffers
    static constexpr int KB = (T == 64 || (KV8 && T == 128)) ? 2 : 1;  // K and V buffers
    static constexpr int RU = !KV8 ? 0 : T == 256 ? 1 : T == 128 ? 3 : 8;  // raw tiles
    static constexpr int RAW = T * kTile;
    static constexpr int ROWB = T < 128 ? T : 128;   // bytes of a raw box row (8-bit pools)
    static constexpr int THREADS = KV8 ? 320 : 192;
    static constexpr int TMEM = NS * 128 + T <= 256 ? 256 : 512;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = TILE;
    static constexpr int OFF_V = OFF_K + KB * TILE;
    static constexpr int OFF_RAW = OFF_V + KB * TILE;
    static constexpr int OFF_SCALE = OFF_RAW + RU * RAW;
    static constexpr int OFF_FACT = OFF_SCALE + RU * kTile;  // [KB][K, V][128] float
    static constexpr int OFF_DEPTH = OFF_FACT + (KV8 ? KB * 2 * kTile * 4 : 0);
    static constexpr int OFF_BAR = OFF_DEPTH + kMaxDraft * 2;
    // barriers
    static constexpr int B_KFULL = 0, B_KEMPTY = B_KFULL + KB, B_VFULL = B_KEMPTY + KB,
                         B_VEMPTY = B_VFULL + KB, B_SFULL = B_VEMPTY + KB,
                         B_PFULL = B_SFULL + NS, B_O = B_PFULL + NS, B_LAND = B_O + 1,
                         B_POISON = B_LAND + 1, B_FACT = B_POISON + 2, B_RFULL = B_FACT + KB,
                         B_REMPTY = B_RFULL + RU, NBAR = B_REMPTY + RU;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;  // tmem, abort, maxdepth, poison[2][4]
    static constexpr int SMEM = 1024 + OFF_MISC + 48;
};

__device__ __forceinline__ uint8_t *align1024(uint8_t *p) {
    const uintptr_t a = (reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023);
    return reinterpret_cast<uint8_t *>(a);
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                            uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// What a request attends.  Lengths and offsets live on the device and are
// checked here: nothing outside [0, total_q) rows or the block table is used.
struct Req {
    int q_start, q_len, L, ctx, start;  // start: the first key any draft may see
};

__device__ __forceinline__ Req request(const TreeParams &p, int b, bool report) {
    Req r;
    const int a = p.cu_q[b], e = p.cu_q[b + 1];
    bool bad = a < 0 || a > p.total_q;
    r.q_start = min(max(a, 0), p.total_q);
    long long n = (long long)e - a;
    if (n < 0 || n > p.max_seqlen_q || n > p.total_q - r.q_start) bad = true;
    n = n < 0 ? 0 : n;
    r.q_len = (int)min(n, (long long)min(p.max_seqlen_q, p.total_q - r.q_start));
    const long long cap_blocks = (long long)p.max_blocks_per_seq * p.block_size;
    const int cap = cap_blocks < p.max_seqlen ? (int)cap_blocks : p.max_seqlen;
    const int L = p.seqlens[b];
    if (L < 0 || L > cap) bad = true;
    r.L = min(max(L, 0), cap);
    if (r.L < r.q_len) {  // the drafts are not all in the cache: nothing is attended
        bad = true;
        r.L = 0;
    }
    if (bad && report) flag_error(p.dev_error, PKV_DEVERR_SEQLEN);
    r.ctx = max(r.L - r.q_len, 0);
    r.start = p.window_left < 0 ? 0 : max(r.ctx - p.window_left, 0);
    return r;
}

// Bits n0 .. n0+31 of a draft's mask of nw 64-bit words (n0 may be negative).
__device__ __forceinline__ uint32_t mask_bits(const int64_t *m, int nw, int n0) {
    if (n0 <= -32 || n0 >= nw * 64) return 0u;
    const uint32_t *w = reinterpret_cast<const uint32_t *>(m);
    if (n0 < 0) return w[0] << (-n0);
    const int i = n0 >> 5, s = n0 & 31;
    const uint32_t lo = w[i], hi = i + 1 < 2 * nw ? w[i + 1] : 0u;
    return __funnelshift_r(lo, hi, s);
}

// Bits [lo, hi) of a 32-bit word, for any lo and hi.
__device__ __forceinline__ uint32_t range_bits(int lo, int hi) {
    lo = max(lo, 0);
    hi = min(hi, 32);
    if (lo >= hi) return 0u;
    const uint32_t top = hi == 32 ? 0xffffffffu : (1u << hi) - 1u;
    return top & ~((1u << lo) - 1u);
}

template <int T, bool KV8>
__global__ void __launch_bounds__(Cfg<T, KV8>::THREADS, Cfg<T, KV8>::CTAS)
tree_kernel(const TreeParams p, const __grid_constant__ CUtensorMap tmk,
            const __grid_constant__ CUtensorMap tmv) {
    using C = Cfg<T, KV8>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align1024(smem_raw);
    const uint32_t base = smem_u32(smem);
    uint16_t *s_depth = reinterpret_cast<uint16_t *>(smem + C::OFF_DEPTH);
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    int32_t *s_abort = reinterpret_cast<int32_t *>(misc + 1);
    int *s_maxdepth = reinterpret_cast<int *>(misc + 2);
    uint32_t *s_poison = misc + 4;  // [2][4]
    auto bar = [&](int i) { return base + C::OFF_BAR + 8 * i; };

    pdl_trigger();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.z;
    const int g = blockIdx.x / p.row_tiles, rt = blockIdx.x - g * p.row_tiles;
    const Req rq = request(p, b, blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0);
    const int G = p.group, Dh = p.head_dim;
    const int nrows = min(rq.q_len * G - rt * kTile, kTile);  // rows of this tile
    if (nrows <= 0) return;
    const int P = p.partition_size;
    const int part = rq.start / P + blockIdx.y;
    const int tok_lo = max(part * P, rq.start);
    const int tok_hi = (int)min((long long)(part + 1) * P, (long long)rq.L);
    const int kt0 = tok_lo / kTile;
    const int ntiles = tok_hi > tok_lo ? (tok_hi - 1) / kTile - kt0 + 1 : 0;
    if (ntiles == 0 && p.num_parts > 1) return;
    // (draft, head) of a row, and its index in q, out and lse
    auto row_unit = [&](int r) {
        const int i = rt * kTile + r, t = i / G;
        return (int64_t)(rq.q_start + t) * p.num_qo_heads + g * G + (i - t * G);
    };
    if (ntiles == 0) {  // no key at all: zeros, and the sink alone
        for (int i = threadIdx.x; i < nrows * (Dh / 8); i += C::THREADS) {
            const int r = i / (Dh / 8), c = i - r * (Dh / 8);
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + row_unit(r) * Dh +
                                       c * 8) = make_uint4(0u, 0u, 0u, 0u);
        }
        if (p.lse_out)
            for (int r = threadIdx.x; r < nrows; r += C::THREADS)
                p.lse_out[row_unit(r)] =
                    p.sink ? p.sink[g * G + (rt * kTile + r) % G] : kNegInf;
        return;
    }

    // ---- set-up: barriers, TMEM, Q tile, depths
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::KB; ++i) {
            mbar_init(bar(C::B_KFULL + i), KV8 ? 4 : 1);
            mbar_init(bar(C::B_KEMPTY + i), 1);
            mbar_init(bar(C::B_VFULL + i), KV8 ? 4 : 1);
            mbar_init(bar(C::B_VEMPTY + i), 1);
        }
        for (int i = 0; i < C::NS; ++i) {
            mbar_init(bar(C::B_SFULL + i), 1);
            mbar_init(bar(C::B_PFULL + i), 4);
        }
        mbar_init(bar(C::B_O), 1);
        mbar_init(bar(C::B_LAND), 1);
        for (int i = 0; i < 2; ++i) mbar_init(bar(C::B_POISON + i), 1);
        for (int i = 0; i < C::KB; ++i) mbar_init(bar(C::B_FACT + i), 4);
        for (int i = 0; i < C::RU; ++i) {
            mbar_init(bar(C::B_RFULL + i), 1 + 8);
            mbar_init(bar(C::B_REMPTY + i), 4);
        }
        fence_barrier_init();
        *s_abort = 0;
        *s_maxdepth = 0;
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    if (warp == 5) {
        tc::tmem_alloc(base + C::OFF_MISC, C::TMEM);
        tc::tmem_relinquish();
    }
    float rowf = fabsf(p.scale_log2);  // score = S * rowf
    if constexpr (!KV8) {
        for (int i = threadIdx.x; i < kTile * (T / 8); i += C::THREADS) {
            const int r = i / (T / 8), c = i - r * (T / 8);
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (r < nrows && c * 8 < Dh)
                v = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.q) +
                                                          row_unit(r) * Dh + c * 8));
            if (p.scale_log2 < 0.f) {  // the scale's sign goes into q
                v.x ^= 0x80008000u;
                v.y ^= 0x80008000u;
                v.z ^= 0x80008000u;
                v.w ^= 0x80008000u;
            }
            st_shared16(base + C::OFF_Q + (c >> 3) * C::HALF + sw128(r, c & 7), v.x, v.y, v.z,
                        v.w);
        }
    } else if (threadIdx.x < kTile) {
        // row r of thread r, in f16: times a power of two that brings its largest
        // value to 2^14..2^15 (exact down to 2^-28 of it)
        const int r = threadIdx.x;
        const uint4 *src = reinterpret_cast<const uint4 *>(
            static_cast<const __nv_bfloat16 *>(p.q) + (r < nrows ? row_unit(r) : 0) * Dh);
        const int nc = r < nrows ? Dh / 8 : 0;
        uint32_t amax = 0;
        for (int c = 0; c < nc; ++c) {
            const uint4 v = __ldg(src + c);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                amax = max(amax, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
        }
        const int E = max((int)(amax >> 7) - 127, -100);
        const uint32_t neg = p.scale_log2 < 0.f ? 0x80000000u : 0u;
        const float f = __uint_as_float(((uint32_t)(127 + 14 - E) << 23) | neg);
        rowf *= __uint_as_float((uint32_t)(127 + E - 14) << 23);
        for (int c = 0; c < T / 8; ++c) {
            uint32_t x[4] = {0u, 0u, 0u, 0u};
            if (c < nc) {
                const uint4 v = __ldg(src + c);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[e] = pack_f16(__uint_as_float(w[e] << 16) * f,
                                    __uint_as_float(w[e] & 0xffff0000u) * f);
            }
            st_shared16(base + C::OFF_Q + (c >> 3) * C::HALF + sw128(r, c & 7), x[0], x[1], x[2],
                        x[3]);
        }
    }
    fence_proxy_async_smem();
    __syncthreads();  // s_maxdepth is zero
    for (int i = threadIdx.x; i < rq.q_len; i += C::THREADS) {
        const int d = p.depth ? min(max(p.depth[rq.q_start + i], 0), 65535) : 0;
        s_depth[i] = (uint16_t)d;
        atomicMax(s_maxdepth, d);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = misc[0];
    const uint32_t t_o = tmem + C::NS * 128;

    const int BS = p.block_size, npg = kTile / BS;
    const int32_t *bt = p.block_table + (int64_t)b * p.max_blocks_per_seq;
    const int pg_first = tok_lo / BS, pg_last = (tok_hi - 1) / BS;
    // every row sees keys [wfull, ctx)
    const int wfull = p.window_left < 0
                          ? 0
                          : (int)max((long long)rq.ctx + *s_maxdepth - p.window_left, 0LL);
    auto partial = [&](int i) {  // some row does not see some key of tile i
        const int k0 = (kt0 + i) * kTile;
        return k0 < tok_lo || k0 < wfull || k0 + kTile > tok_hi || k0 + kTile > rq.ctx;
    };

    if (warp == 4) {
        // ------------------------------------------------------------ producer
        // box coordinates of (page, kv head); one past the pool reads zeros
        const int oob = p.hnd ? (int)(p.num_blocks * p.num_kv_heads)
                              : (int)(p.num_blocks * BS);
        const int cy = p.hnd ? 0 : g;
        auto page_id = [&](int i) {  // lane l < npg: page l of tile i, -1: not attended
            const int pg = (kt0 + i) * npg + lane;
            return lane < npg && pg >= pg_first && pg <= pg_last ? bt[pg] : -1;
        };
        int id = page_id(0);
        bool alive = true;
        int nk = 0, nv = 0, nfix = 0;
        for (int i = 0; i < ntiles && alive; ++i) {
            const int pg = (kt0 + i) * npg + lane;
            int row = oob;
            if (lane < npg && pg >= pg_first && pg <= pg_last) {
                if (id < 0 || id >= p.num_blocks) {
                    flag_error(p.dev_error, PKV_DEVERR_BLOCK_ID);
                    id = -1;
                } else {
                    row = p.hnd ? id * p.num_kv_heads + g : id * BS;
                }
            }
            const int id_now = id;
            if (i + 1 < ntiles) id = page_id(i + 1);
            if constexpr (!KV8) {
                const int s = i % C::KB;
                const uint32_t ph = (uint32_t)(i / C::KB) & 1u;
                // lane -> (page, 64-dim half)
                const int lp = lane / C::HALVES, lh = lane % C::HALVES;
                const int brow = __shfl_sync(0xffffffffu, row, lp);
                alive = warp_wait_bounded(bar(C::B_KEMPTY + s), ph ^ 1u, p.dev_error, s_abort);
                if (!alive) break;
                if (lane == 0) mbar_arrive_expect_tx(bar(C::B_KFULL + s), C::TILE);
                __syncwarp();
                if (lp < npg)
                    tma_load_3d(base + C::OFF_K + s * C::TILE + lh * C::HALF + lp * BS * 128,
                                &tmk, bar(C::B_KFULL + s), lh * 64, cy, brow);
                ++nk;
                alive = warp_wait_bounded(bar(C::B_VEMPTY + s), ph ^ 1u, p.dev_error, s_abort);
                if (!alive) break;
                const bool fix = partial(i);
                const uint32_t vbar = fix ? bar(C::B_LAND) : bar(C::B_VFULL + s);
                const uint32_t vb = base + C::OFF_V + s * C::TILE;
                if (lane == 0) mbar_arrive_expect_tx(vbar, C::TILE);
                __syncwarp();
                if (lp < npg)
                    tma_load_3d(vb + lh * C::HALF + lp * BS * 128, &tmv, vbar, lh * 64, cy,
                                brow);
                ++nv;
                if (fix) {
                    alive = warp_wait_bounded(bar(C::B_LAND), (uint32_t)nfix & 1u, p.dev_error,
                                              s_abort);
                    ++nfix;
                    if (!alive) break;
                    // lane owns rows lane, lane + 32, ..: rows outside the range
                    // are zeroed, and rows with an infinity or a NaN, noted
                    uint32_t *pois = s_poison + ((nfix - 1) & 1) * 4;
                    const int k0 = (kt0 + i) * kTile;
#pragma unroll 1
                    for (int w = 0; w < 4; ++w) {
                        const int r = w * 32 + lane, key = k0 + r;
                        const bool in = key >= tok_lo && key < tok_hi;
                        bool bad = false;
                        if (in) {
#pragma unroll 4
                            for (int c = 0; c < T / 8; ++c) {
                                const uint4 v =
                                    ld_shared16(vb + (c >> 3) * C::HALF + sw128(r, c & 7));
                                const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    bad |= (x[e] & 0x7f80u) == 0x7f80u ||
                                           (x[e] & 0x7f800000u) == 0x7f800000u;
                            }
                        }
                        if (!in || bad)
                            for (int c = 0; c < T / 8; ++c)
                                st_shared_zero16(vb + (c >> 3) * C::HALF + sw128(r, c & 7));
                        const uint32_t m = __ballot_sync(0xffffffffu, in && bad);
                        if (lane == 0) pois[w] = m;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar(C::B_POISON + ((nfix - 1) & 1)));
                        mbar_arrive(bar(C::B_VFULL + s));
                    }
                }
            } else {
                constexpr int PARTS = T / C::ROWB;  // boxes across the head size
                const int lp = lane / PARTS, lh = lane % PARTS;
                const int brow = __shfl_sync(0xffffffffu, row, lp);
                // scale bytes: lane l < 8 copies bytes 16 l .. of the tile
                const int sid = __shfl_sync(0xffffffffu, id_now, (lane * 16 / BS) & 31);
                for (int v = 0; v < 2 && alive; ++v) {
                    const int u = 2 * i + v, s = u % C::RU;
                    const uint32_t full = bar(C::B_RFULL + s);
                    alive = warp_wait_bounded(bar(C::B_REMPTY + s),
                                              ((uint32_t)(u / C::RU) & 1u) ^ 1u, p.dev_error,
                                              s_abort);
                    if (!alive) break;
                    if (lane == 0) mbar_arrive_expect_tx(full, C::RAW);
                    __syncwarp();
                    if (lp < npg)
                        tma_load_3d(base + C::OFF_RAW + s * C::RAW +
                                        lh * (kTile * C::ROWB) + lp * BS * C::ROWB,
                                    v ? &tmv : &tmk, full, lh * 128, cy, brow);
                    if (lane < 8) {
                        if (sid >= 0)
                            cp_async16(base + C::OFF_SCALE + s * kTile + lane * 16,
                                       (v ? p.v_scale : p.k_scale) +
                                           ((int64_t)sid * p.num_kv_heads + g) * BS +
                                           (lane * 16) % BS);
                        cp_async_arrive(full);
                    }
                    ++nk;
                }
            }
        }
        if (!alive) {  // a wait gave up: let the copies in flight land (bounded)
            if constexpr (!KV8) {
                for (int i = max(0, nk - C::KB); i < nk; ++i)
                    warp_wait_bounded(bar(C::B_KFULL + i % C::KB), (uint32_t)(i / C::KB) & 1u,
                                      p.dev_error);
                for (int i = max(0, nv - C::KB); i < nv; ++i)
                    if (!partial(i))
                        warp_wait_bounded(bar(C::B_VFULL + i % C::KB),
                                          (uint32_t)(i / C::KB) & 1u, p.dev_error);
                if (nv > 0 && partial(nv - 1) && nfix > 0)
                    warp_wait_bounded(bar(C::B_LAND), (uint32_t)(nfix - 1) & 1u, p.dev_error);
            } else {
                for (int u = max(0, nk - C::RU); u < nk; ++u)
                    warp_wait_bounded(bar(C::B_RFULL + u % C::RU), (uint32_t)(u / C::RU) & 1u,
                                      p.dev_error);
            }
        }
    } else if (warp == 5) {
        // ------------------------------------------------------------ MMA issuer
        // f16 operands over 8-bit pools, bf16 otherwise (A and B alike; the
        // format fields are bits 7 and 10)
        constexpr uint32_t fmt = KV8 ? (1u << 7 | 1u << 10) : 0u;
        constexpr uint32_t idS = tc::idesc_bf16_f32(128, 128, 0, 0) & ~fmt;
        constexpr uint32_t idO = tc::idesc_bf16_f32(128, T, 0, 1) & ~fmt;
        const uint64_t dq = tc::smem_desc_sw128(base + C::OFF_Q, 16, 1024);
        const uint64_t dk0 = tc::smem_desc_sw128(base + C::OFF_K, 16, 1024);
        const uint64_t dv0 = tc::smem_desc_sw128(base + C::OFF_V, C::HALF, 1024);
        bool alive = true;
        auto issue_s = [&](int i) {
            const int s = i % C::KB;
            alive = warp_wait_bounded(bar(C::B_KFULL + s), (uint32_t)(i / C::KB) & 1u,
                                      p.dev_error, s_abort);
            if (!alive) return;
            tc::fence_after_sync();
            if (lane == 0) {
                const uint64_t dk = dk0 + (uint64_t)((s * C::TILE) >> 4);
                const uint32_t d = tmem + (i % C::NS) * 128;
#pragma unroll
                for (int h = 0; h < C::HALVES; ++h)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t off = (h * C::HALF + k * 32) >> 4;
                        tc::mma_ss(d, dq + off, dk + off, idS, h + k > 0 ? 1u : 0u);
                    }
                tc::commit(bar(C::B_SFULL + i % C::NS));
                tc::commit(bar(C::B_KEMPTY + s));
            }
            __syncwarp();
        };
        issue_s(0);
        for (int i = 0; i < ntiles && alive; ++i) {
            if (C::NS == 2 && i + 1 < ntiles) issue_s(i + 1);
            if (!alive) break;
            const int s = i % C::KB;
            alive = warp_wait_bounded(bar(C::B_PFULL + i % C::NS), (uint32_t)(i / C::NS) & 1u,
                                      p.dev_error, s_abort) &&
                    warp_wait_bounded(bar(C::B_VFULL + s), (uint32_t)(i / C::KB) & 1u,
                                      p.dev_error, s_abort);
            if (!alive) break;
            tc::fence_after_sync();
            if (lane == 0) {
                const uint64_t dv = dv0 + (uint64_t)((s * C::TILE) >> 4);
                tc::mma_ts8(t_o, tmem + (i % C::NS) * 128, dv, idO, i > 0 ? 1u : 0u);
                tc::commit(bar(C::B_VEMPTY + s));
                if (i + 1 == ntiles) tc::commit(bar(C::B_O));
            }
            __syncwarp();
            if (C::NS == 1 && i + 1 < ntiles) issue_s(i + 1);
        }
        if (!alive) {  // let the products in flight finish (bounded) before TMEM goes
            if (lane == 0) tc::commit(bar(C::B_O));
            __syncwarp();
            warp_wait_bounded(bar(C::B_O), 0, p.dev_error);
        }
    } else if (warp < 4) {
        // ------------------------------------------------------------ softmax
        const int r = threadIdx.x;           // row = TMEM lane
        const bool warp_on = warp * 32 < nrows;
        const bool row_on = r < nrows;
        const int64_t unit = row_on ? row_unit(r) : 0;
        const int node = row_on ? (rt * kTile + r) / G : 0;
        const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
        const int head = row_on ? g * G + (rt * kTile + r) % G : 0;
        // weights are 2^(s - m_ref), and over 8-bit pools times the key's V scale:
        // m_ref follows the row's largest score, plus there the tile's largest
        // scale over 2^10, so that f16 holds the product; both sums share it
        float m_ref = kNegInf, l = 0.f;
        bool alive = true;
        int nfix = 0;
        auto page_id = [&](int i) {
            const int pg = (kt0 + i) * npg + lane;
            return lane < npg && pg >= pg_first && pg <= pg_last ? bt[pg] : 0;
        };
        int id = warp_on ? page_id(0) : 0;
        for (int i = 0; i < ntiles; ++i) {
            const uint32_t t_s = tmem + (i % C::NS) * 128 + lane_base;
            const bool fix = partial(i);
            const uint32_t badpg =
                __ballot_sync(0xffffffffu, id < 0 || (int64_t)id >= p.num_blocks);
            if (warp_on && i + 1 < ntiles) id = page_id(i + 1);
            const bool general = fix || badpg != 0 || p.alibi != nullptr;
            alive = warp_wait_bounded(bar(C::B_SFULL + i % C::NS), (uint32_t)(i / C::NS) & 1u,
                                      p.dev_error, s_abort);
            if (KV8 && alive)
                alive = warp_wait_bounded(bar(C::B_FACT + i % C::KB),
                                          (uint32_t)(i / C::KB) & 1u, p.dev_error, s_abort);
            if (!KV8 && fix && alive) {
                alive = warp_wait_bounded(bar(C::B_POISON + (nfix & 1)),
                                          (uint32_t)(nfix >> 1) & 1u, p.dev_error, s_abort);
                ++nfix;
            }
            if (!alive) break;
            if (warp_on) {
                const float4 *kf =
                    reinterpret_cast<const float4 *>(smem + C::OFF_FACT) + (i % C::KB) * 64;
                const float4 *vf = kf + 32;
                tc::fence_after_sync();
                const int k0 = (kt0 + i) * kTile;
                const float rf = general ? 1.f : rowf;
                // Chunk c (32 keys) of S as loaded -> scores: over 8-bit pools times
                // the K scales; in a general tile complete, with bias, -inf for what
                // the row does not see, NaN for a key whose V row is not finite.
                auto to_scores = [&](int c, uint32_t (&v)[32], uint32_t &hide) {
                    if constexpr (KV8) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 f = kf[c * 8 + e / 4];
                            v[e] = __float_as_uint(__uint_as_float(v[e]) * f.x);
                            v[e + 1] = __float_as_uint(__uint_as_float(v[e + 1]) * f.y);
                            v[e + 2] = __float_as_uint(__uint_as_float(v[e + 2]) * f.z);
                            v[e + 3] = __float_as_uint(__uint_as_float(v[e + 3]) * f.w);
                        }
                    }
                    hide = 0u;
                    if (!general) return;
                    const int depth = s_depth[node], qpos = rq.ctx + depth;
                    const int wlo = p.window_left < 0 ? 0 : max(qpos - p.window_left, 0);
                    const int kc = k0 + 32 * c;
                    uint32_t vis = range_bits(max(wlo, tok_lo) - kc, min(rq.ctx, tok_hi) - kc);
                    const int n0 = kc - rq.ctx;  // draft node of the chunk's first key
                    if (n0 > -32 && n0 < rq.q_len && row_on) {
                        const int64_t *mrow =
                            p.mask + (int64_t)(rq.q_start + node) * p.mask_words;
                        uint32_t d = mask_bits(mrow, p.mask_words, n0) &
                                     range_bits(max(tok_lo, rq.ctx) - kc, tok_hi - kc);
                        if (p.window_left >= 0) {
                            for (uint32_t m = d; m; m &= m - 1) {
                                const int e = __ffs(m) - 1;
                                if (s_depth[n0 + e] < depth - p.window_left) d &= ~(1u << e);
                            }
                        }
                        vis |= d;
                    }
                    for (int q = 0; q < 32 / BS; ++q)
                        if ((badpg >> (c * 32 / BS + q)) & 1u)
                            vis &= ~range_bits(q * BS, q * BS + BS);
                    const uint32_t pois =
                        !KV8 && fix ? *reinterpret_cast<volatile uint32_t *>(
                                          s_poison + ((nfix - 1) & 1) * 4 + c)
                                    : 0u;
                    hide = ~vis;
                    const float slope = p.alibi && row_on ? p.alibi[head] * kLog2e : 0.f;
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        float x = __uint_as_float(v[e]) * rowf;
                        if (p.alibi) {
                            const int k = kc + e;
                            const int n = min(max(k - rq.ctx, 0), rq.q_len - 1);
                            const int kpos = k < rq.ctx ? k : rq.ctx + s_depth[n];
                            x = fmaf(slope, (float)(kpos - qpos), x);
                        }
                        if ((pois >> e) & 1u) x = __uint_as_float(0x7fffffffu);
                        v[e] = __float_as_uint((vis >> e) & 1u ? x : kNegInf);
                    }
                };
                float a0 = kNegInf, a1 = kNegInf;
                auto maximum = [&](const uint32_t (&v)[32]) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        a0 = fmax3(a0, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
                        a1 = fmax3(a1, __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
                    }
                };
                // bf16 pools hold the whole row in registers; over 8-bit pools,
                // whose scales need them too, S is read from TMEM a second time
                uint32_t v[KV8 ? 2 : 4][32], hide[KV8 ? 2 : 4];
                float shift = 0.f;
                if constexpr (!KV8) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) tc::ld_32x32b_x32(t_s + 32 * c, v[c]);
                    tc::wait_ld();
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        to_scores(c, v[c], hide[c]);
                        maximum(v[c]);
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        tc::ld_32x32b_x32(t_s + 64 * h, v[0]);
                        tc::ld_32x32b_x32(t_s + 64 * h + 32, v[1]);
                        tc::wait_ld();
                        to_scores(2 * h, v[0], hide[0]);
                        maximum(v[0]);
                        to_scores(2 * h + 1, v[1], hide[1]);
                        maximum(v[1]);
                    }
                    // the tile's largest V scale (NaN rows aside), not below 2^-90:
                    // weights without the scale stay finite
                    const uint4 w = reinterpret_cast<const uint4 *>(vf)[lane];
                    uint32_t mxb = 0;
                    mxb = w.x < 0x7f800000u ? max(mxb, w.x) : mxb;
                    mxb = w.y < 0x7f800000u ? max(mxb, w.y) : mxb;
                    mxb = w.z < 0x7f800000u ? max(mxb, w.z) : mxb;
                    mxb = w.w < 0x7f800000u ? max(mxb, w.w) : mxb;
                    mxb = __reduce_max_sync(0xffffffffu, mxb);
                    shift = (float)(max((int)(mxb >> 23), 37) - 127 - kWeightExp);
                }
                const float mt = fmaxf(a0, a1) * rf + shift;
                if (i == 0) {
                    m_ref = mt;
                } else {
                    const bool grow = mt > m_ref + kLazy || (m_ref == kNegInf && mt > kNegInf);
                    if (__any_sync(0xffffffffu, grow)) {
                        if (C::NS == 2) {  // O must be at rest: the last PV is done
                            alive = warp_wait_bounded(bar(C::B_VEMPTY + (i - 1) % C::KB),
                                                      (uint32_t)((i - 1) / C::KB) & 1u,
                                                      p.dev_error, s_abort);
                            if (!alive) break;
                            tc::fence_after_sync();
                        }
                        const float f = grow ? fast_exp2(m_ref - mt) : 1.f;
                        if (grow) m_ref = mt;
                        l *= f;
#pragma unroll 1
                        for (int c = 0; c < T / 16; ++c) {
                            uint32_t o[16];
                            tc::ld_32x32b_x16(t_o + lane_base + 16 * c, o);
                            tc::wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tc::st_32x32b_x16(t_o + lane_base + 16 * c, o);
                        }
                    }
                }
                const float msub = m_ref == kNegInf ? 0.f : m_ref;
                float s0 = 0.f, s1 = 0.f;
                // weights of chunk c: their sum, and 16 columns of P over S columns
                // that have been read
                auto to_weights = [&](int c, const uint32_t (&v)[32], uint32_t hide) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        float x[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            x[k] = fast_exp2(fmaf(__uint_as_float(v[e + k]), rf, -msub));
                        s0 += x[0];
                        s1 += x[1];
                        s0 += x[2];
                        s1 += x[3];
                        if constexpr (KV8) {
                            const float4 f = vf[c * 8 + e / 4];
                            x[0] *= f.x;
                            x[1] *= f.y;
                            x[2] *= f.z;
                            x[3] *= f.w;
                            if (general) {  // a hidden key's scale may be NaN
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    if ((hide >> (e + k)) & 1u) x[k] = 0.f;
                            }
                            w[e / 2] = pack_f16(x[0], x[1]);
                            w[e / 2 + 1] = pack_f16(x[2], x[3]);
                        } else {
                            w[e / 2] = pack_bf16(x[0], x[1]);
                            w[e / 2 + 1] = pack_bf16(x[2], x[3]);
                        }
                    }
                    tc::st_32x32b_x16(t_s + 16 * c, w);
                };
                if constexpr (!KV8) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) to_weights(c, v[c], hide[c]);
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        tc::ld_32x32b_x32(t_s + 64 * h, v[0]);
                        tc::ld_32x32b_x32(t_s + 64 * h + 32, v[1]);
                        tc::wait_ld();
                        to_scores(2 * h, v[0], hide[0]);
                        to_weights(2 * h, v[0], hide[0]);
                        to_scores(2 * h + 1, v[1], hide[1]);
                        to_weights(2 * h + 1, v[1], hide[1]);
                    }
                }
                l += s0 + s1;
                tc::wait_st();
                tc::fence_before_sync();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_PFULL + i % C::NS));
        }
        // ---- epilogue
        if (alive) alive = warp_wait_bounded(bar(C::B_O), 0, p.dev_error, s_abort);
        if (alive && warp_on) {
            tc::fence_after_sync();
            float mul, lse;
            if (p.num_parts > 1) {
                mul = l == 0.f ? 0.f : 1.f / l;
                lse = l == 0.f ? kNegInf : m_ref + log2f(l);
            } else {
                const float sink = p.sink ? p.sink[head] * kLog2e : kNegInf;
                const float M = fmaxf(m_ref, sink);
                const float Ms = M == kNegInf ? 0.f : M;
                const float f = exp2f(m_ref - Ms);
                const float lam = l * f + exp2f(sink - Ms);
                mul = lam == 0.f ? 0.f : f / lam;
                lse = lam == 0.f ? kNegInf : (Ms + log2f(lam)) * kLn2;
                // a NaN weight leaves m_ref as it was: keep the NaN
                if (l != l) mul = lse = l;
            }
            const int64_t pidx = unit * p.num_parts + blockIdx.y;
#pragma unroll 1
            for (int c = 0; c < T / 32; ++c) {
                uint32_t v[32];
                tc::ld_32x32b_x32(t_o + lane_base + 32 * c, v);
                tc::wait_ld();
                if (row_on && p.num_parts > 1) {
                    float *dst = p.part_o + pidx * Dh + 32 * c;
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        if (32 * c + e < Dh)
                            *reinterpret_cast<float4 *>(dst + e) = make_float4(
                                __uint_as_float(v[e]) * mul, __uint_as_float(v[e + 1]) * mul,
                                __uint_as_float(v[e + 2]) * mul,
                                __uint_as_float(v[e + 3]) * mul);
                } else if (row_on) {
                    __nv_bfloat16 *dst =
                        static_cast<__nv_bfloat16 *>(p.out) + unit * Dh + 32 * c;
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        if (32 * c + e >= Dh) continue;
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            w[k] = pack_bf16(__uint_as_float(v[e + 2 * k]) * mul,
                                             __uint_as_float(v[e + 2 * k + 1]) * mul);
                        *reinterpret_cast<uint4 *>(dst + e) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                __syncwarp();  // the next load is warp-wide
            }
            if (row_on) {
                if (p.num_parts > 1)
                    p.part_lse[pidx] = lse;
                else if (p.lse_out)
                    p.lse_out[unit] = lse;
            }
        }
    } else if constexpr (KV8) {
        // ------------------------------------------------------------ codes -> f16 tiles
        // warps 6-9, 32 rows of every K and V tile each; a lane takes 16 codes
        // of a row at a time, and holds the row's scale bytes
        constexpr int CH = T / 16, RPI = 32 / CH;  // chunks per row, rows per round
        const int w = warp - 6;
        bool alive = true;
        auto row_id = [&](int i) {  // lane = row: its page if the row is in the range
            const int key = (kt0 + i) * kTile + w * 32 + lane;
            return key >= tok_lo && key < tok_hi ? bt[key / BS] : -1;
        };
        int id = row_id(0);
        for (int i = 0; i < ntiles && alive; ++i) {
            const uint32_t ok =
                __ballot_sync(0xffffffffu, id >= 0 && (int64_t)id < p.num_blocks);
            if (i + 1 < ntiles) id = row_id(i + 1);
            const int s = i % C::KB;
            const uint32_t free_ph = ((uint32_t)(i / C::KB) & 1u) ^ 1u;
            float *fact = reinterpret_cast<float *>(smem + C::OFF_FACT) + s * 256 + w * 32 + lane;
            float kscale = 0.f;
#pragma unroll 1
            for (int isv = 0; isv < 2; ++isv) {
                const int u = 2 * i + isv, rs = u % C::RU;
                alive = warp_wait_bounded(bar(C::B_RFULL + rs), (uint32_t)(u / C::RU) & 1u,
                                          p.dev_error, s_abort) &&
                        warp_wait_bounded(bar((isv ? C::B_VEMPTY : C::B_KEMPTY) + s), free_ph,
                                          p.dev_error, s_abort);
                if (!alive) break;
                const uint32_t raw = base + C::OFF_RAW + rs * C::RAW;
                const uint32_t byte = smem[C::OFF_SCALE + rs * kTile + w * 32 + lane];
                if (!isv) {
                    kscale = scale_value(byte);
                } else {
                    // both factors of this row: V's buffer is free, so the softmax of
                    // the tile that last used this slot is done
                    fact[0] = kscale;
                    fact[128] = (ok >> lane) & 1u ? scale_value(byte) : 0.f;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::B_FACT + s));
                }
                // V rows that are not attended may hold any codes, and a row of NaN
                // reaches who sees it through its factor: zero both
                const uint32_t nan_rows = __ballot_sync(0xffffffffu, byte == kScaleNaN);
                const uint32_t zero = isv ? ~ok | nan_rows : 0u;
                const uint32_t buf = base + (isv ? C::OFF_V : C::OFF_K) + s * C::TILE;
#pragma unroll 4
                for (int it = 0; it < 32 / RPI; ++it) {
                    const int rr = it * RPI + lane / CH, c = lane % CH, r = w * 32 + rr;
                    const int part_c = (c * 16) / C::ROWB, cc = c - part_c * (C::ROWB / 16);
                    const uint32_t ra = raw + part_c * (kTile * C::ROWB) +
                                        (C::ROWB == 128 ? sw128(r, cc)
                                                        : r * 64u + ((cc ^ ((r >> 1) & 3)) << 4));
                    uint4 code = ld_shared16(ra);
                    if ((zero >> rr) & 1u) code = make_uint4(0u, 0u, 0u, 0u);
                    uint32_t x[8];
                    e4m3_to_f16(code.x, x[0], x[1]);
                    e4m3_to_f16(code.y, x[2], x[3]);
                    e4m3_to_f16(code.z, x[4], x[5]);
                    e4m3_to_f16(code.w, x[6], x[7]);
                    const uint32_t dst = buf + (c >> 2) * C::HALF;
                    const int ch = (2 * c) & 7;
                    st_shared16(dst + sw128(r, ch), x[0], x[1], x[2], x[3]);
                    st_shared16(dst + sw128(r, ch + 1), x[4], x[5], x[6], x[7]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar((isv ? C::B_VFULL : C::B_KFULL) + s));
                    mbar_arrive(bar(C::B_REMPTY + rs));
                }
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 5) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, C::TMEM);
    }
}

// ---------------------------------------------------------------------------
// merge of the partitions, sink, cast: one warp per (draft, query head)
// ---------------------------------------------------------------------------
constexpr int kMergeThreads = 128;

__global__ void __launch_bounds__(kMergeThreads)
tree_merge_kernel(const TreeParams p) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int b = blockIdx.z, t = blockIdx.y;
    const int h = blockIdx.x * (kMergeThreads / 32) + (threadIdx.x >> 5);
    const Req rq = request(p, b, false);
    if (t >= rq.q_len || h >= p.num_qo_heads) return;
    const int P = p.partition_size, D = p.head_dim;
    const int n = rq.L > rq.start ? (rq.L - 1) / P - rq.start / P + 1 : 0;
    const int64_t unit = (int64_t)(rq.q_start + t) * p.num_qo_heads + h;
    const float *lp = p.part_lse + unit * p.num_parts;
    const float *po = p.part_o + unit * p.num_parts * D;
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
    const float inv = lam == 0.f ? 0.f : 1.f / lam;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + unit * D;
    for (int c = 4 * lane; c < D; c += 128) {
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const float w = exp2f(lp[i] - Ms);
            const float4 v = *reinterpret_cast<const float4 *>(po + (int64_t)i * D + c);
            acc.x = fmaf(w, v.x, acc.x);
            acc.y = fmaf(w, v.y, acc.y);
            acc.z = fmaf(w, v.z, acc.z);
            acc.w = fmaf(w, v.w, acc.w);
        }
        *reinterpret_cast<uint2 *>(out + c) =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    }
    if (p.lse_out && lane == 0) p.lse_out[unit] = lam == 0.f ? kNegInf : (Ms + log2f(lam)) * kLn2;
}

template <int T, bool KV8>
cudaError_t launch_one(const TreeParams &p, const CUtensorMap *tk, const CUtensorMap *tv,
                       cudaStream_t stream) {
    using C = Cfg<T, KV8>;
    static_assert(C::SMEM * C::CTAS + (C::CTAS - 1) * 1024 <= 232448, "shared memory");
    auto kern = tree_kernel<T, KV8>;
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kern), C::SMEM);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(p.num_kv_heads * p.row_tiles, p.num_parts, p.batch),
                      dim3(C::THREADS), (size_t)C::SMEM, stream, p, *tk, *tv);
}

}  // namespace

cudaError_t launch_tree(const TreeParams &p, const CUtensorMap *tmap_k,
                        const CUtensorMap *tmap_v, cudaStream_t stream) {
    const bool kv8 = p.k_scale != nullptr;
    cudaError_t e;
    if (p.head_dim <= 64)
        e = kv8 ? launch_one<64, true>(p, tmap_k, tmap_v, stream)
                : launch_one<64, false>(p, tmap_k, tmap_v, stream);
    else if (p.head_dim <= 128)
        e = kv8 ? launch_one<128, true>(p, tmap_k, tmap_v, stream)
                : launch_one<128, false>(p, tmap_k, tmap_v, stream);
    else
        e = kv8 ? launch_one<256, true>(p, tmap_k, tmap_v, stream)
                : launch_one<256, false>(p, tmap_k, tmap_v, stream);
    if (e != cudaSuccess || p.num_parts == 1) return e;
    constexpr int kHeads = kMergeThreads / 32;
    return launch_pdl(tree_merge_kernel,
                      dim3((p.num_qo_heads + kHeads - 1) / kHeads, p.max_seqlen_q, p.batch),
                      dim3(kMergeThreads), 0, stream, p);
}

}  // namespace pkv
