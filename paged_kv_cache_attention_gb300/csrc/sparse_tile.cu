// sparse_tile.cu -- attention over lists of pages for chunks of queries (bf16 pools).
//
// The attention of sparse_decode.cu where requests have several queries.  There, every
// (query, kv head) reads its own pages: a chunk reads the pages that its queries agree
// on once for each of them, and a product of 16 rows has the heads of one query.  Here a
// CTA takes 128 rows, (query, head) pairs of consecutive queries of one request and kv
// head (32 queries of 4 heads), and the union of their lists:
//   * every query's list becomes a bitmap of the request's pages, a window of a few
//     thousand pages at a time (what two CTAs have room for, however wide the tables
//     are); the union's pages are numbered in ascending order and taken 128 keys at a
//     time;
//   * S = Q K^T and O += P V are tcgen05 products of 128 x 128 x 128 with S, O and P
//     (bf16, in place of S) in tensor memory, K and V by TMA, page by page;
//   * thread = row in the softmax: a page that is not the row's weighs nothing, one that
//     is no row's of the warp is not looked at.  O is rescaled only when a row's
//     maximum grows by more than 2^8.
// Values that are not finite: a zero weight times such a value is NaN, also for a row
// that does not keep the key.  A warp looks through every tile of V: rows that no query
// keeps (behind the sequence or the union: they may hold anything) are zeroed, and if
// another has such a value the tile of queries is taken again, row by row.
//
// Two CTAs share an SM, so that one's softmax runs beside the other's products and loads.
// Eight softmax warps, of two halves of the keys: 181 us where four took 318 (890 queries
// of 1024 keys each, 8 kv heads of 4, D = 128).  Now 116 us, row by row 255.  A step takes
// 5000 clocks, 2950 with two CTAs: 2600 of softmax, the rest the way from products to
// softmax and back.  A tile's union has 275 pages where a list has 64 (neighbours share 31
// on average): 4.7 times the products that count, 37 us of the tensor pipe's time at
// cuBLAS's rate for 7.9.  So most of the time is hand-overs, and SMs that run one tile where
// others run two (240 tiles of 35 steps on 152 SMs; spread evenly they would take some
// 81 us).  Tiles are of one request each (rows counted on over requests, beyond
// kTiledRequests: 165 us).
//
// A weight rounds to bf16 for its product with V (at most 2^-8 of it, as in the dense
// calls: the products are of bf16 pairs); the sum of the weights takes it unrounded.
#include "pkv_sparse.cuh"
#include "pkv_tcgen05.cuh"

namespace pkv {

namespace {

constexpr int kRows = 128;             // rows of a tile: TMEM lanes
constexpr int kKeys = 128;             // keys of a step
constexpr int kD = 128;                // head size, padded
constexpr int kSoft = 8;               // softmax warps; then one that loads, one that issues
constexpr int kLoad = kSoft, kIssue = kSoft + 1, kCheck = kSoft + 2;  // and one that looks at V
constexpr int kThreads = (kSoft + 3) * 32;
constexpr int kHalf = 128 * 128;       // bytes of 128 rows of 64 dims
constexpr int kTile = 2 * kHalf;
constexpr float kNegInf = -INFINITY;
constexpr float kGrow = 8.f;           // log2 units a score may exceed its row's reference
constexpr uint32_t kCols = 256;        // O, then S
static_assert(kKeys == kRows && kD == kRows, "one tile size for Q, K and V");

// Barriers, each of one tile: the phases count the steps.
enum { kKFull, kKEmpty, kVFull, kVReady, kVEmpty, kSFull, kPFull, kODone, kDrain, kBars };

constexpr int kOffQ = 0, kOffK = kTile, kOffV = 2 * kTile, kOffBar = 3 * kTile;
constexpr int kOffTmem = kOffBar + kBars * 8;
constexpr int kOffList = kOffTmem + 8;
// then of a window: pages [32 words + PP] u16, bitmaps of the queries [queries][words], of the
// union [words] and its prefix counts [words + 1]
constexpr int kListBytes = 14000;

// 0 * x + sum of bf16 pairs.
__device__ __forceinline__ uint32_t zero_times(uint32_t x, uint32_t sum) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(sum));
    return r;
}

// Row (query, head h) by itself: plain sums.
__device__ __noinline__ void lone_row(const SparseParams &p, const void *k_cache,
                                      const void *v_cache, int t, int g, int h, int r, int L,
                                      int block_size) {
    const int lane = threadIdx.x & 31, D = p.r.head_dim, Hkv = p.r.num_kv_heads;
    const int hq = g * p.r.group + h;
    const int64_t unit = (int64_t)t * Hkv * p.r.group + hq;
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + unit * D;
    float x[4], o[4], m = kNegInf, l = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = lane + 32 * i < D ? __bfloat162float(q[lane + 32 * i]) : 0.f;
        o[i] = 0.f;
    }
    const int npages = (L + block_size - 1) / block_size;
    const int32_t *list = p.pages + ((int64_t)t * Hkv + g) * p.top_k;
    int before = -1;
    for (int e = 0; e < p.top_k; ++e) {
        const int page = list[e];
        if (page <= before || page >= npages) break;
        before = page;
        const int id = p.r.block_table[(int64_t)r * p.r.max_blocks_per_seq + page];
        if (id < 0 || id >= p.r.num_blocks) continue;
        for (int s = 0; s < block_size && page * block_size + s < L; ++s) {
            const int64_t row = p.hnd ? ((int64_t)id * Hkv + g) * block_size + s
                                      : ((int64_t)id * block_size + s) * Hkv + g;
            const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(k_cache) + row * D;
            const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(v_cache) + row * D;
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (lane + 32 * i < D) dot = fmaf(x[i], __bfloat162float(k[lane + 32 * i]), dot);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
            dot *= p.scale_log2;
            const float top = fmaxf(m, dot), ref = top == kNegInf ? 0.f : top;
            const float a = fast_exp2(m - ref), w = fast_exp2(dot - ref);
            l = l * a + w;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (lane + 32 * i < D) o[i] = fmaf(w, __bfloat162float(v[lane + 32 * i]), o[i] * a);
            m = top;
        }
    }
    const float sink = p.sink ? p.sink[hq] * kLog2e : kNegInf;
    const float T = fmaxf(m, sink), Ts = T == kNegInf ? 0.f : T;
    const float f = exp2f(m - Ts), lam = l * f + exp2f(sink - Ts);
    const float mul = lam == 0.f ? 0.f : f / lam;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + unit * D;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < D) out[lane + 32 * i] = __float2bfloat16_rn(o[i] * mul);
    if (p.lse_out && lane == 0) p.lse_out[unit] = lam == 0.f ? kNegInf : (Ts + log2f(lam)) * kLn2;
}

template <int BS>
__global__ void __launch_bounds__(kThreads, 2)
sparse_tile_kernel(const SparseParams p, const void *k_cache, const void *v_cache,
                   const __grid_constant__ CUtensorMap tmk,
                   const __grid_constant__ CUtensorMap tmv) {
    constexpr int PP = kKeys / BS;  // pages of a step
    constexpr int SHIFT = BS == 16 ? 4 : 5;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);  // 1024-aligned
    const uint32_t base = smem_u32(smem), bars = base + kOffBar;
    uint16_t *s_page = reinterpret_cast<uint16_t *>(smem + kOffList);
    uint32_t *s_own = reinterpret_cast<uint32_t *>(s_page + p.words * 32 + PP);
    __shared__ int s_end[kRows];       // where the queries' lists end
    __shared__ float s_max[2][kRows];  // the rows' largest scores (in the end: sums) by halves
    __shared__ int s_dead;  // a wait gave up: all others do
    __shared__ int s_bad;   // a value that is not finite
    auto bar = [&](int i) { return bars + 8 * i; };
    auto wait = [&](int i, uint32_t parity) {
        return mbar_wait_bounded(bar(i), parity, p.r.dev_error, &s_dead);
    };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = p.r.group, Dh = p.r.head_dim, Hkv = p.r.num_kv_heads;
    const int queries = kRows >> p.group_shift;
    const int g = blockIdx.x % Hkv;
    uint32_t *s_bits = s_own + queries * p.words;            // the union's
    int *s_before = reinterpret_cast<int *>(s_bits + p.words);

    if (threadIdx.x == 0) {
        for (int i = 0; i < kBars; ++i)
            mbar_init(bar(i), i == kPFull ? kSoft : 1);
        fence_barrier_init();
        s_dead = s_bad = 0;
    }
    if (warp == kIssue) {
        tc::tmem_alloc(base + kOffTmem, kCols);
        tc::tmem_relinquish();
    }
    pdl_wait();
    int t0, t_end;
    tile_rows(p.r, (int)(blockIdx.x / Hkv), queries, t0, t_end);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + kOffTmem);
    const uint32_t colO = tmem, colS = tmem + kD;

    int done = 0;  // steps of the requests before
    // the tile's rows, request by request (one, but where requests meet)
    for (int t = t0; t < t_end && !*static_cast<volatile int *>(&s_dead);) {
        int r, L, count;
        if (!row_request(p.r, t, BS, g == 0 && threadIdx.x == 0, r, L, count)) {
            ++t;
            continue;
        }
        const int first = t, nq = min(count, t_end - t);
        t += nq;
        const int keys = L + count - 1;  // of the request
        const int all_words = ((max(L + nq - 1, 0) + BS - 1) >> SHIFT) / 32 + 1;
        const int32_t *table = p.r.block_table + (int64_t)r * p.r.max_blocks_per_seq;

        if (threadIdx.x < nq) s_end[threadIdx.x] = p.top_k;
        // Q: row = query << group_shift | head, 128-byte swizzle; zeros in rows that are none.
        // A negative scale goes into Q, so that scores grow with the products, and one of 0 too
        // (0 times a value that is not finite: NaN).
        const uint32_t sign = p.scale_log2 < 0.f ? 0x80008000u : 0u;
#pragma unroll 4
        for (int i = threadIdx.x; i < kRows * 16; i += kThreads) {
            const int row = i >> 4, c = i & 15;
            const int j = row >> p.group_shift, h = row & ((1 << p.group_shift) - 1);
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (j < nq && h < G && c * 8 < Dh)
                v = *reinterpret_cast<const uint4 *>(
                    static_cast<const __nv_bfloat16 *>(p.q) +
                    (((int64_t)(first + j) * Hkv + g) * G + h) * Dh + c * 8);
            *reinterpret_cast<uint4 *>(smem + kOffQ + (c >> 3) * kHalf + sw128(row, c & 7)) =
                p.scale_log2 == 0.f ? make_uint4(zero_times(v.x, 0u), zero_times(v.y, 0u),
                                                 zero_times(v.z, 0u), zero_times(v.w, 0u))
                                    : make_uint4(v.x ^ sign, v.y ^ sign, v.z ^ sign, v.w ^ sign);
        }
        __syncthreads();
        // where each list ends
        const int64_t list_step = (int64_t)Hkv * p.top_k;
        const int32_t *lists = p.pages + ((int64_t)first * Hkv + g) * p.top_k;
        const int entries = nq * p.top_k;
#pragma unroll 4
        for (int i = threadIdx.x; i < entries; i += kThreads) {
            const int j = i / p.top_k, x = i - j * p.top_k;
            const int32_t *list = lists + j * list_step;
            const int e = list[x], before = x > 0 ? list[x - 1] : -1;
            if (e <= before || e >= (max(L + j, 0) + BS - 1) >> SHIFT) atomicMin(&s_end[j], x);
        }
        // Two softmax warps have the same rows (a warp reaches its quarter of the TMEM lanes
        // only): each takes half of a step's keys and of O's columns.
        const int quarter = warp & 3, half = warp >> 2;
        const int row = quarter * 32 + lane;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        // (whether x holds in either: a warp that gave up leaves together with its partner)
        auto pair_any = [&](bool x) {
            uint32_t r;
            asm volatile(
                "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
                "bar.red.or.pred p, %2, 64, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(r)
                : "r"((uint32_t)x), "r"(quarter + 1)
                : "memory");
            return r != 0;
        };
        const int j0 = row >> p.group_shift, h = row & ((1 << p.group_shift) - 1);
        const bool live = j0 < nq && h < G;
        float ref = kNegInf, l = 0.f;
        bool ok = true;

        int before = 0;  // steps of the windows before
        // the pages in windows of p.words * 32
        for (int w0 = 0; w0 < all_words && !*static_cast<volatile int *>(&s_dead); w0 += p.words) {
            const int words = min(p.words, all_words - w0), page0 = w0 * 32;
            const int32_t *bt = table + page0;
            const int total = keys - page0 * BS;
            // ------------------------------------------------ the lists as bitmaps
            for (int i = threadIdx.x; i < (nq + 1) * words; i += kThreads) {
                const int j = i / words, w = i - j * words;
                (j < nq ? s_own + j * p.words : s_bits)[w] = 0;
            }
            __syncthreads();
#pragma unroll 4
            for (int i = threadIdx.x; i < entries; i += kThreads) {
                const int j = i / p.top_k, x = i - j * p.top_k;
                const int e = lists[j * list_step + x] - page0;
                if (x < s_end[j] && (uint32_t)e < (uint32_t)words * 32u) {
                    const int id = bt[e];
                    if (id >= 0 && id < p.r.num_blocks) {
                        atomicOr(&s_own[j * p.words + (e >> 5)], 1u << (e & 31));
                        atomicOr(&s_bits[e >> 5], 1u << (e & 31));
                    } else {
                        flag_error(p.r.dev_error, PKV_DEVERR_BLOCK_ID);
                    }
                } else if (x == s_end[j] && e >= 0 && page0 == 0) {
                    flag_error(p.r.dev_error, PKV_DEVERR_BLOCK_ID);
                }
            }
            fence_proxy_async_smem();
            __syncthreads();
            if (warp == 0) {
                int sum = 0;
#pragma unroll 1
                for (int w0 = 0; w0 < words; w0 += 32) {
                    const int own = w0 + lane < words ? __popc(s_bits[w0 + lane]) : 0;
                    int in = own;
#pragma unroll
                    for (int off = 1; off < 32; off <<= 1) {
                        const int o = __shfl_up_sync(0xffffffffu, in, off);
                        if (lane >= off) in += o;
                    }
                    if (w0 + lane < words) s_before[w0 + lane] = sum + in - own;
                    sum += __shfl_sync(0xffffffffu, in, 31);
                }
                if (lane == 0) s_before[words] = sum;
            }
            __syncthreads();
            const int n = s_before[words], steps = (n + PP - 1) / PP;
            for (int w = threadIdx.x; w < words; w += kThreads) {
                int at = s_before[w];
                for (uint32_t b = s_bits[w]; b; b &= b - 1) s_page[at++] = (uint16_t)(w * 32 + __ffs(b) - 1);
            }
            if (threadIdx.x < PP) s_page[n + threadIdx.x] = 0;  // up to the last step's end
            __syncthreads();

            if (warp == kLoad) {
                // ------------------------------------------------ pages by TMA
                int id = lane < min(PP, n) ? bt[s_page[lane]] : 0;
                int j = 0;
                for (; j < steps; ++j) {
                    const int k = done + j, m = min(PP, n - j * PP);
                    const int next = lane < min(PP, n - (j + 1) * PP) ? bt[s_page[(j + 1) * PP + lane]] : 0;
                    const int cy = p.hnd ? 0 : g, cz = p.hnd ? id * Hkv + g : id * BS;
                    bool ok = true;
#pragma unroll 1
                    for (int v = 0; v < 2 && ok; ++v) {  // K, then V
                        if (k > 0) ok = __all_sync(0xffffffffu, wait(v ? kVEmpty : kKEmpty, (k - 1) & 1));
                        if (!ok) break;
                        const uint32_t full = bar(v ? kVFull : kKFull);
                        const bool one = elect_one();
                        if (one) mbar_arrive_expect_tx(full, m * BS * 256);
#pragma unroll
                        for (int i = 0; i < PP; ++i) {
                            const int z = __shfl_sync(0xffffffffu, cz, i);
                            if (i < m && one)
#pragma unroll
                                for (int h = 0; h < 2; ++h)
                                    tma_load_3d(base + (v ? kOffV : kOffK) + h * kHalf + i * BS * 128,
                                                v ? &tmv : &tmk, full, h * 64, cy, z);
                        }
                    }
                    if (!ok) break;
                    id = next;
                }
                if (j < steps) {  // a wait gave up: let the copies in flight land
                    for (int b = 0; b < 2; ++b)
                        for (int par = 0; par < 2; ++par)
                            mbar_wait_bounded(bar(b ? kVFull : kKFull), par, p.r.dev_error);
                }
            } else if (warp == kIssue) {
                // ------------------------------------------------ products
                bool ok = true;
                if (elect_one()) {
                    constexpr uint32_t idS = tc::idesc_bf16_f32(kRows, kKeys, 0, 0);
                    constexpr uint32_t idO = tc::idesc_bf16_f32(kRows, kD, 0, 1);
                    const uint64_t dq = tc::smem_desc_sw128(base + kOffQ, 16, 1024);
                    const uint64_t dk = tc::smem_desc_sw128(base + kOffK, 16, 1024);
                    const uint64_t dv = tc::smem_desc_sw128(base + kOffV, kHalf, 1024);
#pragma unroll 1
                    for (int j = 0; j < steps && ok; ++j) {
                        const int k = done + j;
                        // S goes where P was: the product with it must be done
                        ok = wait(kKFull, k & 1) && (k == 0 || wait(kODone, (k - 1) & 1));
                        if (!ok) break;
                        tc::fence_after_sync();
                        tc::mma_ss8<kHalf>(colS, dq, dk, idS, 0u);
                        tc::commit(bar(kSFull));
                        tc::commit(bar(kKEmpty));
                        ok = wait(kPFull, k & 1) && wait(kVReady, k & 1);
                        if (!ok) break;
                        tc::fence_after_sync();
                        // P: 16 keys in 8 columns, the second half's where its S was
#pragma unroll
                        for (int i = 0; i < kKeys / 16; ++i)
                            tc::mma_ts(colO, colS + (i / 4) * 64 + (i % 4) * 8, dv + i * 128, idO,
                                       before + j > 0 || i > 0 ? 1u : 0u);
                        tc::commit(bar(kODone));
                        tc::commit(bar(kVEmpty));
                    }
                    if (!ok) {  // the products in flight
                        tc::commit(bar(kDrain));
                        mbar_wait_bounded(bar(kDrain), 0, p.r.dev_error);
                    }
                }
                __syncwarp();
            } else if (warp == kCheck) {
                // ------------------------------------------------ V: tails zeroed, all finite?
                uint32_t sum[4] = {0u, 0u, 0u, 0u};  // of 0 * v: NaN if v is not finite
#pragma unroll 1
                for (int j = 0; j < steps; ++j) {
                    const int k = done + j, m = min(PP, n - j * PP);
                    if (!__all_sync(0xffffffffu, wait(kVFull, k & 1))) break;
                    // keys of the step that the request has (only its last page can end inside)
                    const int end = (m - 1) * BS + min(BS, total - (int)s_page[j * PP + m - 1] * BS);
                    uint4 *v = reinterpret_cast<uint4 *>(smem + kOffV) + lane;
                    if (end < kKeys) {
#pragma unroll 1
                        for (int i = lane; i < kKeys * 16; i += 32)  // (8 chunks a row, two halves)
                            if (((i >> 3) & (kKeys - 1)) >= end) v[i - lane] = make_uint4(0u, 0u, 0u, 0u);
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
#pragma unroll 1
                    for (int i0 = 0; i0 < kKeys * 16; i0 += 8 * 32) {
                        uint4 x[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] = v[i0 + 32 * i];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            sum[0] = zero_times(x[i].x, sum[0]);
                            sum[1] = zero_times(x[i].y, sum[1]);
                            sum[2] = zero_times(x[i].z, sum[2]);
                            sum[3] = zero_times(x[i].w, sum[3]);
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kVReady));
                }
                if ((sum[0] | sum[1] | sum[2] | sum[3]) & 0x7fff7fffu) s_bad = 1;
            } else {
                // ------------------------------------------------ softmax, thread = row
                constexpr int HP = PP / 2;  // pages of a half
                const int limit = live ? L + j0 - page0 * BS : 0;
                const uint32_t *own = s_own + (live ? j0 : 0) * p.words;
                const float scale = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);
#pragma unroll 1
                for (int j = 0; j < steps; ++j) {
                    const int k = done + j;
                    // keys of each page that the row keeps; pages that some row of the warp does
                    uint32_t held = 0, any = 0;  // 8 bits a page
                    const int i0 = j * PP + half * HP;
                    const uint32_t *two = reinterpret_cast<const uint32_t *>(s_page + i0);
#pragma unroll
                    for (int g2 = 0; g2 < HP; ++g2) {  // (entries past the last: page 0)
                        const int page = (two[g2 / 2] >> (g2 % 2 * 16)) & 0xffff;
                        const bool mine = live && i0 + g2 < n && (own[page >> 5] >> (page & 31)) & 1;
                        const int keep = mine ? min(max(limit - page * BS, 0), BS) : 0;
                        held |= (uint32_t)keep << (8 * g2);
                        any |= (keep > 0 ? 1u << g2 : 0u) | (keep > 0 && keep < BS ? 256u : 0u);
                    }
                    any = __reduce_or_sync(0xffffffffu, any);
                    const bool part = any & 256u;
                    ok = ok && __all_sync(0xffffffffu, wait(kSFull, k & 1));
                    tc::fence_after_sync();
                    // 16 keys at a time, those of pages that some row of the warp keeps.  (Rolled
                    // loops: code that is not in the instruction cache costs more than they do.)
                    constexpr int KP = BS / 16;
                    const uint32_t colH = colS + lanes + half * 64;
                    auto load_scores = [&](int c, uint32_t (&s)[16]) {
                        tc::ld_32x32b_x16(colH + c * 16, s);
                        const int keep = (int)((held >> (8 * (c / KP))) & 255u) - c % KP * 16;
                        tc::wait_ld();
                        if (part)
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (e >= keep) s[e] = 0xff800000u;
                        return keep > 0;
                    };
                    float mx = kNegInf;
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        if (!ok || !((any >> (c / KP)) & 1u)) continue;
                        uint32_t s[16];
                        const bool mine = load_scores(c, s);
                        float top = kNegInf;
#pragma unroll
                        for (int e = 0; e < 16; e += 2)
                            top = fmax3(top, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                        if (mine) mx = fmaxf(mx, top);
                    }
                    mx *= scale;
                    s_max[half][row] = mx;
                    if (pair_any(!ok)) {
                        ok = false;
                        break;
                    }
                    mx = fmaxf(mx, s_max[half ^ 1][row]);
                    if (__any_sync(0xffffffffu, mx > ref + kGrow || (ref == kNegInf && mx > kNegInf))) {
                        const float next = fmaxf(ref, mx);
                        const float a = next == kNegInf ? 1.f : fast_exp2(ref - next);
                        l *= a;
                        if (before + j > 0) {  // (ok: the next product is issued after this warp's P)
                            ok = __all_sync(0xffffffffu, wait(kODone, (k - 1) & 1));
                            tc::fence_after_sync();
#pragma unroll 1
                            for (int c = half * 64; ok && c < half * 64 + 64; c += 32) {
                                uint32_t o[32];
                                tc::ld_32x32b_x32(colO + lanes + c, o);
                                tc::wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
                                tc::st_32x32b_x32(colO + lanes + c, o);
                            }
                            tc::wait_st();
                        }
                        ref = next;
                    }
                    const float sub = ref == kNegInf ? 0.f : ref;
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t w[8];
                        if ((any >> (c / KP)) & 1u) {
                            uint32_t s[16];
                            const bool mine = load_scores(c, s);
                            float sum[2] = {0.f, 0.f};
                            const uint32_t all = mine ? 0xffffffffu : 0u;
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                const float x = fast_exp2(fmaf(__uint_as_float(s[e]), scale, -sub));
                                const float y = fast_exp2(fmaf(__uint_as_float(s[e + 1]), scale, -sub));
                                sum[0] += x;
                                sum[1] += y;
                                w[e / 2] = pack_bf16(x, y) & all;
                            }
                            if (mine) l += sum[0] + sum[1];
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e) w[e] = 0u;
                        }
                        tc::st_32x32b_x8(colH + c * 8, w);
                    }
                    tc::wait_st();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kPFull));
                }
            }
            before += steps;
            done += steps;
            tc::fence_before_sync();
            __syncthreads();
            tc::fence_after_sync();
        }
        if (warp < kSoft) {
            // ------------------------------------------------ the row's output
            if (before > 0 && ok) ok = __all_sync(0xffffffffu, wait(kODone, (done - 1) & 1));
            tc::fence_after_sync();
            s_max[half][row] = l;
            pair_any(false);
            l += s_max[half ^ 1][row];
            const float sink = p.sink && live ? p.sink[g * G + h] * kLog2e : kNegInf;
            const float T = fmaxf(ref, sink), Ts = T == kNegInf ? 0.f : T;
            const float f = exp2f(ref - Ts), lam = l * f + exp2f(sink - Ts);
            const float mul = lam == 0.f ? 0.f : f / lam;
            const int64_t unit = ((int64_t)(first + (live ? j0 : 0)) * Hkv + g) * G + (live ? h : 0);
            if (live && half == 0 && p.lse_out) p.lse_out[unit] = lam == 0.f ? kNegInf : (Ts + log2f(lam)) * kLn2;
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + unit * Dh;
#pragma unroll 1
            for (int c = half * 64; c < min(Dh, half * 64 + 64); c += 16) {
                uint32_t o[16];
                if (before > 0) {
                    tc::ld_32x32b_x16(colO + lanes + c, o);
                    tc::wait_ld();
                }
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    w[e] = before > 0 ? pack_bf16(__uint_as_float(o[2 * e]) * mul,
                                                 __uint_as_float(o[2 * e + 1]) * mul)
                                     : 0u;
                if (live) {
                    *reinterpret_cast<uint4 *>(out + c) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4 *>(out + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                }
            }
            tc::fence_before_sync();
        }
        __syncthreads();
        tc::fence_after_sync();
        if (s_bad && !s_dead) {  // all rows again, by themselves
#pragma unroll 1
            for (int x = warp; x < nq * G; x += kThreads / 32)
                lone_row(p, k_cache, v_cache, first + x / G, g, x % G, r, max(L + x / G, 0), BS);
            __syncthreads();
            if (threadIdx.x == 0) s_bad = 0;
        }
        __syncthreads();
    }
    if (warp == kIssue) tc::tmem_dealloc(tmem, kCols);
    if (g == 0) {
        const int64_t all = gridDim.x / (unsigned)Hkv;  // tiles
        check_offsets(p.r, blockIdx.x / Hkv + threadIdx.x * all, kThreads * all);
    }
}

template <int BS>
cudaError_t launch_bs(SparseParams p, bool &fits, const void *k, const void *v,
                      const CUtensorMap *tk, const CUtensorMap *tv, cudaStream_t stream) {
    const int queries = kRows >> p.group_shift;
    // Words of the bitmaps, 32 pages each, of a window that leaves room for two CTAs: for
    // 32 queries 70 words, 2240 pages (of a table of 4096: 185 us in one CTA per SM and
    // one window, 117 so).
    const int a_word = (queries + 2) * 4 + 32 * 2;
    p.words = min(p.r.max_blocks_per_seq / 32 + 1, kListBytes / a_word);
    const int64_t smem = 1024 + kOffList + (kKeys / BS + 2) * 2 + 4 + (int64_t)p.words * a_word;
    const int64_t grid = row_tiles(p.r, (int)queries) * p.r.num_kv_heads;
    fits = grid <= 0x7fffffff;
    if (!fits) return cudaErrorNotSupported;
    auto kern = sparse_tile_kernel<BS>;
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kern), (int)smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3((unsigned)grid), dim3(kThreads), (size_t)smem, stream, p, k, v, *tk,
                      *tv);
}

}  // namespace

cudaError_t launch_sparse_tile(const SparseParams &p0, bool &fits, int block_size, const void *k_cache,
                               const void *v_cache, const CUtensorMap *tmap_k,
                               const CUtensorMap *tmap_v, cudaStream_t stream) {
    SparseParams p = p0;
    fits = p.r.head_dim <= kD;
    if (!fits) return cudaErrorNotSupported;
    p.group_shift = 0;
    while ((1 << p.group_shift) < p.r.group) ++p.group_shift;
    return block_size == 16 ? launch_bs<16>(p, fits, k_cache, v_cache, tmap_k, tmap_v, stream)
                            : launch_bs<32>(p, fits, k_cache, v_cache, tmap_k, tmap_v, stream);
}

}  // namespace pkv
