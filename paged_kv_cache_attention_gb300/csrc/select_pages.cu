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
// up to 2048 are exact there), 16 pages as rows and heads of one or more queries as
// columns.  The order of the summands is free, so a lane loads 16 codes in one go
// and uses them as the fragments of four steps, and the columns are laid out to
// match.  A code becomes an f16 by putting it into the mantissa of 1024 (a byte
// permutation) and taking 1152 off: 2.5 instructions for a pair.
//
// A cluster of CTAs shares the pages of a tile of queries of one request and kv
// head; each keeps its pages' scores in its own shared memory, as integers that sort
// like the scores.  The top_k-th largest is found digit by digit (8 bits at a time,
// histograms summed over the cluster, until few are left), then the pages above it,
// and as many of those equal to it as there is room for, are written in ascending
// order.  One launch, no workspace.
//
// In a decode step (one query per tile) HBM bound: (2 D + 1) bytes per page and kv
// head, each read once; every lane copies the pieces it will use itself (cp.async, a
// tile ahead; three ahead leave room for fewer CTAs: 62 us for 48), so that nothing
// waits but on its own loads.  64 queries of 20K tokens, 8 kv heads of 128: 42 us, 59% of
// HBM's rate; all CTAs read first and choose then.  One query of 1M tokens: 52 us, 36%: a
// cluster of 16 CTAs on 128 of 152 SMs, and barriers for each digit.
//
// In a chunk the queries of a tile share the pages' loads and conversions: 934 queries of
// 26K tokens, 8 kv heads of 4: 132 us (600 row by row).  There two CTAs of eight warps
// an SM run one's choice beside the other's scores (163 us in one of 16), and two page
// tiles share what is read of the columns (138 us with one).  The scores
// take half of the time; the 25 GFLOP alone are 44 us at the rate of mma.sync (a product
// every 8.6 clocks of a scheduler), 13 us at cuBLAS's.
#include <cuda_fp16.h>

#include "pkv_sparse.cuh"

namespace pkv {

namespace {

constexpr uint32_t kForced = 0xffffffffu;  // above every score
constexpr int kNoVote = -100000;           // exponent of a column that has no say
constexpr int kRank = 32;                  // scores ranked against one another

// An unsigned integer that sorts like x (no NaN; -0 was made 0).
__device__ __forceinline__ uint32_t sortable(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// Four int8 codes of a word as f16 pairs (bytes 0 and 1, bytes 2 and 3), exact; plus
// 1152 each unless EXACT.
template <bool EXACT>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const uint32_t u = w ^ 0x80808080u;  // code + 128
    lo = __byte_perm(u, 0x64646464u, 0x4140);  // 1024 + code + 128
    hi = __byte_perm(u, 0x64646464u, 0x4342);
    if (EXACT) {
        const uint32_t off = 0x64806480u;  // 1152, twice
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(off));
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(off));
    }
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}

__device__ __forceinline__ float pow2(int e) {  // -126 <= e <= 127
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// x * 2^e, rounded once: x whole, -252 <= e <= 254.  The first product is exact, or
// overflows as the whole does, or is so small that the whole is 0.
__device__ __forceinline__ float scaled(float x, int e) {
    const int last = min(max(e, -126), 127);
    return x * pow2(e - last) * pow2(last);
}

// Count one more in a word of shared memory, if on (no branch).
__device__ __forceinline__ void count_if(uint32_t addr, bool on) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                 "@p red.shared::cta.add.u32 [%0], 1;\n\t}" ::"r"(addr),
                 "r"((uint32_t)on)
                 : "memory");
}

__device__ __forceinline__ void block_sync(bool cluster) {
    if (cluster)
        cluster_sync();
    else
        __syncthreads();
}

// NCH: 64-byte pieces of a page's codes; NT: 8-column tiles; GP: columns of a query
// (its group's heads, rounded up to a power of two).
template <int NCH, int NT, int GP, int W>
struct Shape {
    static constexpr int QT = NT * 8 / GP;               // queries of a tile
    static constexpr int WARPS = W;
    // 16-page tiles of a step: two share what is read of the columns, where registers allow
    static constexpr int PT = QT > 1 && NT <= 4 ? 2 : 1;
    static constexpr int STEP = 16 * PT;                 // pages of a step
    static constexpr int NST = 2;                        // steps in the ring per warp
    // Few columns: 1152 is taken off the sums, not off each code.  Four sums for a
    // quarter of the channels each stay below 2^24 (32 channels * 255 * 1279).
    static constexpr bool OFFSET = QT == 1 && NCH <= 4;
    static constexpr int STAGE = NCH * 1024;
    // One query: the ring, histograms [2][256], columns [NT][NCH][2][32 lanes].  Several:
    // columns, and in their place histograms [2][QT][256] once the scores are there.
    static constexpr int HIST = QT * 2048, COLS = NT * NCH * 1024;
    static constexpr int HIST_OFF = QT > 1 ? 0 : WARPS * NST * STAGE;
    static constexpr int Q_OFF = QT > 1 ? 0 : HIST_OFF + HIST;
    static constexpr int KEY_OFF = QT > 1 && HIST > COLS ? HIST : Q_OFF + COLS;  // scores: [QT][cap]
    static constexpr int GROUP = WARPS / QT;            // warps that select for a query
};

template <int NCH, int NT, int GP, int W>
__global__ void __launch_bounds__(W * 32, 16 / W)
select_pages_kernel(const SelectParams p) {
    using S = Shape<NCH, NT, GP, W>;
    // sums that do not wait for one another
    constexpr int NA = S::OFFSET ? 4 : NT * S::PT <= 2 ? 2 : 1;
    constexpr int kWarps = S::WARPS, kThreads = kWarps * 32;
    constexpr int QT = S::QT, NST = S::NST, PT = S::PT, STEP = S::STEP, GS = S::GROUP * 32, BPT = 256 / GS;
    extern __shared__ uint4 s_dyn[];
    uint4 *s_q = s_dyn + S::Q_OFF / 16;
    uint32_t *s_key = reinterpret_cast<uint32_t *>(s_dyn + S::KEY_OFF / 16);
    auto s_hist = reinterpret_cast<uint32_t (*)[QT][256]>(s_dyn + S::HIST_OFF / 16);
    __shared__ int s_exp[NT * 8];
    __shared__ alignas(16) float2 s_col[NT * 8];  // the exponent as a factor; -inf if no say
    __shared__ alignas(16) int s_sum[NT * 8][4];             // OFFSET: a column's sums over d / 4 % 4
    __shared__ uint32_t s_pick[QT][3];           // digit, pages above it, pages with it
    __shared__ int s_scale[QT == 1 ? W : 1][S::NST][16];  // scale bytes of the steps in flight
    __shared__ uint32_t s_range[S::WARPS][2];    // least and largest score
    __shared__ uint32_t s_both[2];               // the same of the CTA
    __shared__ int s_left[QT];                   // scores in the list to be ranked
    __shared__ int s_cnt[kWarps][2];             // above, equal: per warp
    __shared__ int s_total[QT][2];               // of the CTA

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gq = lane >> 2, tq = lane & 3;
    const int C = p.cluster, rank = C > 1 ? (int)cluster_rank() : 0;
    const int64_t unit = blockIdx.x / (unsigned)C;
    const int tile = (int)(unit / p.r.num_kv_heads), g = (int)(unit % p.r.num_kv_heads);
    const int D = p.r.head_dim, G = p.r.group, shift = p.bs_shift;

    pdl_wait();
    int t0 = tile, t_end = tile + 1;
    if (QT > 1) tile_rows(p.r, tile, QT, t0, t_end);
    // the tile's rows, request by request (one, but where requests meet)
    for (int t = t0; t < t_end;) {
        int r, L, count;
        if (!row_request(p.r, t, p.block_size, g == 0 && rank == 0 && threadIdx.x == 0, r, L,
                         count)) {
            ++t;
            continue;
        }
        const int nq = min(count, t_end - t);
        const int first = t;
        t += nq;
        auto pages_of = [&](int j) { return (max(L + j, 0) + p.block_size - 1) >> shift; };
        auto out_of = [&](int j) {
            return p.pages + ((int64_t)(first + j) * p.r.num_kv_heads + g) * p.top_k;
        };
#pragma unroll 1
        for (int j = 0; j < nq; ++j) {  // rows that take all their pages
            const int n = pages_of(j);
            if (n <= p.top_k)
#pragma unroll 1
                for (int i = rank * kThreads + threadIdx.x; i < p.top_k; i += C * kThreads)
                    out_of(j)[i] = i < n ? i : -1;
        }
        const int n = pages_of(nq - 1);
        if (n <= p.top_k) continue;
        const int per = ((n + C - 1) / C + STEP - 1) / STEP * STEP;
        const int base = rank * per, nl = min(max(n - base, 0), per);

        // the queries as column fragments
        if (QT > 1) __syncthreads();  // (the tile's rows before are done)
        if (QT == 1)
#pragma unroll 1
            for (int i = threadIdx.x; i < 128; i += kThreads)
                reinterpret_cast<uint4 *>(&s_hist[0][0][0])[i] = make_uint4(0u, 0u, 0u, 0u);
        const int32_t *bt = p.r.block_table + (int64_t)r * p.r.max_blocks_per_seq + base;
        for (int i = threadIdx.x; i < nl; i += kThreads) s_key[i] = (uint32_t)__ldg(bt + i);
        if (threadIdx.x < QT) s_left[threadIdx.x] = 0;
#pragma unroll 1
        for (int i = threadIdx.x; i < NT * NCH * 64; i += kThreads) s_q[i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
        for (int i = threadIdx.x; i < NT * 8; i += kThreads) {
            s_exp[i] = kNoVote;
            s_col[i] = make_float2(0.f, -INFINITY);
            *reinterpret_cast<int4 *>(s_sum[i]) = make_int4(0, 0, 0, 0);
        }
        __syncthreads();
        const int tiles = (nl + STEP - 1) / STEP;
        const int mine = tiles > warp ? (tiles - warp + kWarps - 1) / kWarps : 0;
        // Rows of the bounds in step k, for the tiles' pages gq and gq + 8, and the scale
        // byte (-1: no page) of page `lane` of the step.  The page ids wait in the first
        // row of scores, where a step's are read before its scores are written.
        auto rows_of = [&](int k, uint32_t (&row)[2 * PT], int &byte) {
            const int i = (warp + k * kWarps) * STEP + (PT == 2 ? lane : lane & 15);
            const int id = i < nl ? (int)s_key[i] : -1;
            const bool live = id >= 0 && id < p.r.num_blocks;
            const uint32_t at = (uint32_t)(live ? id : 0) * p.r.num_kv_heads + g;  // < 2^31
            byte = live ? (int)p.bounds_scale[at] : -1;
            if (!live && i < nl) flag_error(p.r.dev_error, PKV_DEVERR_BLOCK_ID);
#pragma unroll
            for (int j = 0; j < 2 * PT; ++j) row[j] = __shfl_sync(0xffffffffu, at, gq + 8 * j);
        };
        auto source = [&](uint32_t row, int c) {  // this lane's 16 codes of piece c
            return p.bounds + (uint64_t)row * (uint32_t)(2 * D) + tq * 16 + c * 64;
        };
        // One query: step k goes to slot k % NST of a ring; its scale bytes follow a step
        // later.
        const uint32_t ring = smem_u32(s_dyn) + warp * NST * S::STAGE + lane * 16;
        int *scale = &s_scale[QT == 1 ? warp : 0][0][0];
        int byte_ahead = -1;
        auto issue = [&](int k) {
            const uint32_t dst = ring + (k % NST) * S::STAGE;
            uint32_t row[2 * PT];
            rows_of(k, row, byte_ahead);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int c = 0; c < NCH; ++c) {  // (pages out of the pool: scores not used)
                    if (c < NCH - 1)
                        cp_async16(dst + (j * NCH + c) * 512, source(row[j], c));
                    else
                        cp_async16_or_zero(dst + (j * NCH + c) * 512, source(row[j], c),
                                           c * 64 + tq * 16 < 2 * D);
                }
        };
        auto keep_byte = [&](int k) {
            if (lane < 16) scale[(k % NST) * 16 + lane] = byte_ahead;
        };
        // Several queries: into registers, a piece ahead.
        auto load = [&](uint4 (&x)[2 * PT], const uint32_t (&row)[2 * PT], int c) {
#pragma unroll
            for (int j = 0; j < 2 * PT; ++j) {
                x[j] = make_uint4(0u, 0u, 0u, 0u);
                if (c < NCH - 1 || c * 64 + tq * 16 < 2 * D)
                    x[j] = __ldg(reinterpret_cast<const uint4 *>(source(row[j], c)));
            }
        };
        uint32_t row[2 * PT];
        int byte = -1;
        uint4 x[2 * PT];
        if (QT == 1) {
            if (mine > 0) issue(0);
            asm volatile("cp.async.commit_group;" ::: "memory");
        } else if (mine > 0) {
            rows_of(0, row, byte);
            load(x, row, 0);
        }
        const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) +
                                 ((int64_t)first * p.r.num_kv_heads + g) * G * D;
#pragma unroll 1
        for (int i = warp; i < nq * G; i += kWarps) {
            const int j = i / G, h = i - j * G, col = j * GP + h;
            const __nv_bfloat16 *x = q + ((int64_t)j * p.r.num_kv_heads * G + h) * D;
            constexpr int VL = NCH > 4 ? 8 : NCH > 2 ? 4 : 2;  // values of a lane
            float v[VL];
            uint32_t amax = 0;
#pragma unroll
            for (int m = 0; m < VL; ++m) {
                const int d = lane + 32 * m;
                const uint32_t bits = d < D ? (uint32_t)__bfloat16_as_ushort(x[d]) : 0u;
                amax = max(amax, bits & 0x7fffu);
                v[m] = __uint_as_float(bits << 16);
            }
            amax = __reduce_max_sync(0xffffffffu, amax);
            if (amax >= 0x7f80u) continue;  // not finite
            const int e = max((int)(amax >> 7) - 127, -112) - 7;
            if (lane == 0) {
                s_exp[col] = e;
                s_col[col] = make_float2(pow2(max(min(e, 60), -60)), 0.f);
            }
            const float f = __uint_as_float((uint32_t)(127 - e) << 23);
            // channel d is code d against the lower bounds and D + d against the upper:
            // code k: piece k / 64, lane (col % 8, k / 16 % 4), step k / 4 % 4, its value k % 4
            const uint32_t at = ((col >> 3) * NCH * 64 + (col & 7) * 4) * 16;
            int sum = 0;
#pragma unroll
            for (int m = 0; m < VL; ++m) {
                const int d = lane + 32 * m;
                if (d >= D) break;
                const float c = rintf(v[m] * f);
                sum += (int)c;
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    const int k = part * D + d;
                    const uint32_t o = at + (k >> 6) * 1024 + (k >> 3 & 1) * 512 + (k >> 4 & 3) * 16 +
                                       (k & 7) * 2;
                    *reinterpret_cast<__half *>(reinterpret_cast<char *>(s_q) + o) =
                        __float2half(part ? fmaxf(c, 0.f) : fminf(c, 0.f));
                }
            }
            if (S::OFFSET) {  // of the lanes with the same lane / 4 % 4, and so d / 4 % 4
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                if ((lane & 19) == 0) s_sum[col][lane >> 2] = sum;
            }
        }
        __syncthreads();
        // With exponents within +-60 (and scale bytes near 127) all products are exact, and a
        // score is one of a few; else each score is scaled by itself.
        bool plain = true;
        for (int i = lane; i < NT * 8; i += 32)
            plain = plain && (s_exp[i] == kNoVote || (s_exp[i] >= -60 && s_exp[i] <= 60));
        plain = __all_sync(0xffffffffu, plain);
        constexpr bool HELD = NT == 1 && NCH <= 4;
        uint4 qf[HELD ? NCH : 1][2];  // a single tile's columns stay in registers
        if (HELD)
#pragma unroll
            for (int c = 0; c < (HELD ? NCH : 1); ++c)
#pragma unroll
                for (int s2 = 0; s2 < 2; ++s2) qf[c][s2] = s_q[(c * 2 + s2) * 32 + lane];
        float off[S::OFFSET ? NT : 1][2][4];  // 1152 times a column's sums, exact
        if (S::OFFSET)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    off[nt][i / 4][i % 4] = 1152.f * (float)s_sum[nt * 8 + 2 * tq + i / 4][i % 4];

        // (whole numbers: partial sums in any order give the same)
        float part[PT][NT][NA][4];
        auto multiply = [&](int c, const uint4 (&x)[2 * PT]) {  // piece c of a step's pages
#pragma unroll
            for (int s2 = 0; s2 < 2; ++s2) {
                uint32_t a[PT][2][4];
#pragma unroll
                for (int u = 0; u < PT; ++u) {
                    const uint4 x0 = x[2 * u], x1 = x[2 * u + 1];
                    const uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w};
                    const uint32_t w1[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        codes_to_f16<!S::OFFSET>(w0[2 * s2 + s], a[u][s][0], a[u][s][2]);
                        codes_to_f16<!S::OFFSET>(w1[2 * s2 + s], a[u][s][1], a[u][s][3]);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint4 b = HELD ? qf[HELD ? c : 0][s2]
                                            : s_q[((nt * NCH + c) * 2 + s2) * 32 + lane];
#pragma unroll
                    for (int u = 0; u < PT; ++u) {
                        mma_f16_16816(part[u][nt][2 * s2 % NA], a[u][0][0], a[u][0][1], a[u][0][2],
                                      a[u][0][3], b.x, b.y);
                        mma_f16_16816(part[u][nt][(2 * s2 + 1) % NA], a[u][1][0], a[u][1][1],
                                      a[u][1][2], a[u][1][3], b.z, b.w);
                    }
                }
            }
        };
        // the scores of a step, this warp's steps every kWarps-th
#pragma unroll 1
        for (int k = 0; k < mine; ++k) {
#pragma unroll
            for (int u = 0; u < PT; ++u)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4 * NA; ++e) part[u][nt][e / 4][e % 4] = 0.f;
            uint32_t row_next[2 * PT];
            int byte_next = -1;
            if constexpr (QT == 1) {
                keep_byte(k);
                if (k + 1 < mine) issue(k + 1);
                asm volatile("cp.async.commit_group;" ::: "memory");
                asm volatile("cp.async.wait_group 1;" ::: "memory");
                __syncwarp();
                const uint32_t slot = ring + (k % NST) * S::STAGE;
#pragma unroll
                for (int c = 0; c < NCH; ++c) {
                    const uint4 y[2] = {lds128(slot + c * 512), lds128(slot + (NCH + c) * 512)};
                    multiply(c, y);
                }
            } else {
                if (k + 1 < mine) {
                    rows_of(k + 1, row_next, byte_next);
                } else {
#pragma unroll
                    for (int j = 0; j < 2 * PT; ++j) row_next[j] = row[j];
                }
#pragma unroll
                for (int c = 0; c < NCH; ++c) {
                    uint4 y[2 * PT];
                    if (c + 1 < NCH)
                        load(y, row, c + 1);
                    else
                        load(y, row_next, 0);
                    multiply(c, x);
#pragma unroll
                    for (int j = 0; j < 2 * PT; ++j) x[j] = y[j];
                }
            }
#pragma unroll
            for (int u = 0; u < PT; ++u) {
                float acc[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        acc[nt][e] = 0.f;
#pragma unroll
                        for (int i = 0; i < NA; ++i)
                            acc[nt][e] += S::OFFSET ? part[u][nt][i][e] -
                                                          off[S::OFFSET ? nt : 0][e & 1][i]
                                                    : part[u][nt][i][e];
                    }
                // Scores: of this lane's columns, then the best of the lanes that hold the
                // query's other columns.
                const int i0 = (warp + k * kWarps) * STEP + u * 16 + gq;
                int byte2[2];
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    byte2[j] = QT == 1 ? scale[(k % NST) * 16 + gq + 8 * j]
                                       : __shfl_sync(0xffffffffu, byte, u * 16 + gq + 8 * j);
                const bool near = plain && (uint32_t)(byte2[0] - 67) <= 103u &&
                                  (uint32_t)(byte2[1] - 67) <= 103u;
                const bool fast = __all_sync(0xffffffffu, near);
                if (fast) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float4 f = *reinterpret_cast<const float4 *>(&s_col[nt * 8 + 2 * tq]);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc[nt][e] = e & 1 ? fmaf(acc[nt][e], f.z, f.w) : fmaf(acc[nt][e], f.x, f.y);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const int ex = s_exp[nt * 8 + 2 * tq + (e & 1)];
                            acc[nt][e] = ex == kNoVote ? -INFINITY
                                                       : scaled(acc[nt][e], ex + byte2[e >> 1] - 127);
                        }
                }
                auto store = [&](int query, float m, int i, int byte, bool here) {
                    if (fast)
                        m *= pow2(byte - 127);
                    else if (byte == (int)kScaleNaN)
                        m = INFINITY;
                    uint32_t key = byte >= 0 ? sortable(m + 0.f) : 0u;
                    const int page = base + i;
                    if (page < p.num_first || page >= pages_of(query) - p.num_recent) key = kForced;
                    if (here) s_key[query * p.cap + i] = key;
                };
                auto best = [&](int nt, int j) { return fmaxf(acc[nt][2 * j], acc[nt][2 * j + 1]); };
                if constexpr (GP >= 4) {
                    // a query's lanes have its score for both rows: even ones store the first
                    const int j = tq & 1, i = i0 + 8 * j, byte = j ? byte2[1] : byte2[0];
#pragma unroll
                    for (int nt = 0; nt < NT; nt += GP == 16 ? 2 : 1) {
                        float m[2];
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            m[r] = best(nt, r);
                            if (GP == 16) m[r] = fmaxf(m[r], best(nt + 1, r));
                            m[r] = fmaxf(m[r], __shfl_xor_sync(0xffffffffu, m[r], 1));
                            if (GP >= 8) m[r] = fmaxf(m[r], __shfl_xor_sync(0xffffffffu, m[r], 2));
                        }
                        store((nt * 8 + 2 * tq) / GP, j ? m[1] : m[0], i, byte,
                              GP == 4 || tq < 2);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int i = i0 + 8 * j, byte = byte2[j];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (GP == 2) {
                                store(nt * 4 + tq, best(nt, j), i, byte, true);
                            } else {
                                store(nt * 8 + 2 * tq, acc[nt][2 * j], i, byte, true);
                                store(nt * 8 + 2 * tq + 1, acc[nt][2 * j + 1], i, byte, true);
                            }
                        }
                    }
                }
            }
            if (QT > 1) {
                byte = byte_next;
#pragma unroll
                for (int j = 0; j < 2 * PT; ++j) row[j] = row_next[j];
            }
        }
        if (QT == 1) asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();

        // The top_k-th largest score; a group of warps for each query.  The digits begin
        // below the leading bits that all scores share, and end when few enough are left
        // to be ranked against one another.  (Tiles shared by a cluster take all 32 bits in
        // the same steps: their barriers are the whole cluster's.)
        const int mq = warp / S::GROUP, li = threadIdx.x - mq * GS;
        const int nrow = mq < nq ? pages_of(mq) : 0;
        const bool choose = nrow > p.top_k;
        // Whole tiles are looked through: what lies behind a row counts as forced.
        const int scan = choose ? tiles * STEP : 0;
        const uint32_t *key_row = s_key + mq * p.cap;
        const bool fixed = QT > 1 && C > 1;
        auto group_sync = [&] {
            if (S::GROUP == 1)
                __syncwarp();
            else
                asm volatile("bar.sync %0, %1;" ::"r"(mq + 1), "n"(GS) : "memory");
        };
        auto sync = [&] {
            if (C > 1)
                cluster_sync();
            else
                group_sync();
        };
        if (QT > 1) {
#pragma unroll
            for (int i = li; i < 128; i += GS)
                *reinterpret_cast<uint4 *>(&s_hist[i >> 6][mq][(i & 63) * 4]) = make_uint4(0u, 0u, 0u, 0u);
            group_sync();
        }
        uint32_t prefix = 0;  // of the scores that are left: the bits from `digit` up
        int need = p.top_k + (n + STEP - 1) / STEP * STEP - nrow, left = 0, digit = 32, pass = 0;
        if (!fixed) {
            need = p.top_k - p.num_first - p.num_recent;  // forced ones are above all others
            uint32_t lo = 0xffffffffu, hi = 0;
#pragma unroll 1
            for (int i = li * 4; i < scan; i += GS * 4) {
                const uint4 k4 = *reinterpret_cast<const uint4 *>(key_row + i);
                const uint32_t key[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    lo = min(lo, key[b]);
                    hi = max(hi, key[b] + 1u);  // (0 for forced ones)
                }
            }
            lo = __reduce_min_sync(0xffffffffu, lo);
            hi = __reduce_max_sync(0xffffffffu, hi);
            if (hi > 0) --hi;
            if (S::GROUP > 1) {
                if (lane == 0) {
                    s_range[warp][0] = lo;
                    s_range[warp][1] = hi;
                }
                group_sync();
#pragma unroll
                for (int w = 0; w < S::GROUP; ++w) {
                    lo = min(lo, s_range[mq * S::GROUP + w][0]);
                    hi = max(hi, s_range[mq * S::GROUP + w][1]);
                }
            }
            if (C > 1) {  // (one query: all warps have the same) lane c looks at CTA c
                if (threadIdx.x == 0) {
                    s_both[0] = lo;
                    s_both[1] = hi;
                }
                cluster_sync();
                if (lane < C) {
                    const uint32_t at = cluster_addr(smem_u32(s_both), lane);
                    lo = cluster_ld32(at);
                    hi = cluster_ld32(at + 4);
                }
                lo = __reduce_min_sync(0xffffffffu, lo);
                hi = __reduce_max_sync(0xffffffffu, hi);
            }
            if (need == 0) lo = hi = kForced - 1;  // none but the forced ones
            digit = lo < hi ? 32 - __clz(lo ^ hi) : 0;
            prefix = digit == 32 ? 0u : lo >> digit << digit;
        }
        // Of what is left: all keys less than this far above prefix (not forced ones, unless
        // all 32 bits are taken).
        auto limit_of = [&] {
            const uint32_t all = digit == 32 ? 0xffffffffu : (1u << digit) - 1u;
            return fixed ? all : min(all, kForced - 1 - prefix);
        };
        bool ranked = false;
        while (choose || fixed) {
            if (digit == 0) break;
            const int next = fixed ? digit - 8 : max(digit - 8, 0);
            const uint32_t limit = limit_of();
            uint32_t *hist = s_hist[pass & 1][mq], *other = s_hist[(pass + 1) & 1][mq];
            const uint32_t bins = smem_u32(hist);
#pragma unroll 1
            for (int i = li * 4; i < scan; i += GS * 4) {
                const uint4 k4 = *reinterpret_cast<const uint4 *>(key_row + i);
                const uint32_t key[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const uint32_t d = key[b] - prefix;
                    count_if(bins + (d >> next) * 4, d <= limit);
                }
            }
            sync();
            // thread li: bins 255 - li * BPT and below, so that a prefix sum counts from
            // the largest down
            uint32_t v[BPT], own = 0;
#pragma unroll
            for (int b = 0; b < BPT; ++b) v[b] = C > 1 ? 0u : hist[255 - li * BPT - b];
            if (C > 1)  // (C: 2, 4, 8 or 16; loads of four CTAs in flight)
#pragma unroll 1
                for (int c = 0; c < C; c += 4) {
                    uint32_t x[BPT][4];
#pragma unroll
                    for (int d = 0; d < 4; ++d)
#pragma unroll
                        for (int b = 0; b < BPT; ++b)
                            x[b][d] = c + d < C ? cluster_ld32(cluster_addr(bins + 4 * (255 - li * BPT - b), c + d))
                                                : 0u;
#pragma unroll
                    for (int b = 0; b < BPT; ++b) v[b] += x[b][0] + x[b][1] + x[b][2] + x[b][3];
                }
#pragma unroll
            for (int b = 0; b < BPT; ++b) own += v[b];
            uint32_t sum = own;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, sum, off);
                if (lane >= off) sum += o;
            }
            if (S::GROUP > 1) {
                if (lane == 31) s_cnt[warp][0] = (int)sum;
                group_sync();
#pragma unroll 1
                for (int w = mq * S::GROUP; w < warp; ++w) sum += (uint32_t)s_cnt[w][0];
            }
            if (choose && sum >= (uint32_t)need && sum - own < (uint32_t)need) {
                uint32_t before = sum - own;
#pragma unroll
                for (int b = 0; b < BPT; ++b) {
                    if (before < (uint32_t)need && before + v[b] >= (uint32_t)need) {
                        s_pick[mq][0] = (uint32_t)(255 - li * BPT - b);
                        s_pick[mq][1] = before;
                        s_pick[mq][2] = v[b];
                    }
                    before += v[b];
                }
            }
            // the other buffer: read before this pass's barrier, counted in after the next
            if (pass > 0)
#pragma unroll 1
                for (int i = li; i < 256; i += GS) other[i] = 0;
            group_sync();
            ++pass;
            digit = next;
            if (choose) {
                prefix |= s_pick[mq][0] << digit;
                need -= (int)s_pick[mq][1];
                left = (int)s_pick[mq][2];
            }
            group_sync();
            if (!fixed && digit > 0 && left <= kRank) {
                ranked = true;
                break;
            }
        }
        if (ranked) {
            // the scores left, with their pages: [kRank] keys, then [kRank] pages
            uint32_t *list = s_hist[pass & 1][mq], *all = list;  // (all zeros, read by no one)
            const uint32_t limit = limit_of();
#pragma unroll 1
            for (int i = li * 4; i < scan; i += GS * 4) {
                const uint4 k4 = *reinterpret_cast<const uint4 *>(key_row + i);
                const uint32_t key[4] = {k4.x, k4.y, k4.z, k4.w};
                const bool some = key[0] - prefix <= limit || key[1] - prefix <= limit ||
                                  key[2] - prefix <= limit || key[3] - prefix <= limit;
                if (some)
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    if (key[b] - prefix <= limit) {
                        const int at = atomicAdd(&s_left[mq], 1);
                        list[at] = key[b];
                        list[kRank + at] = (uint32_t)(base + i + b);
                    }
            }
            sync();
            if (C > 1) {  // of the whole cluster, in the buffer whose counts are read
                all = s_hist[(pass + 1) & 1][mq];
                if (warp == 0) {  // (one query, left <= 32) lane c: CTA c's count
                    const int m = lane < C ? (int)cluster_ld32(cluster_addr(smem_u32(s_left), lane)) : 0;
                    int c = 0, at = lane;
#pragma unroll 1
                    for (int d = 0; d < C - 1; ++d) {
                        const int md = __shfl_sync(0xffffffffu, m, d);
                        if (c == d && at >= md) {
                            at -= md;
                            ++c;
                        }
                    }
                    if (lane < left) {
                        all[lane] = cluster_ld32(cluster_addr(smem_u32(&list[at]), c));
                        all[kRank + lane] = cluster_ld32(cluster_addr(smem_u32(&list[kRank + at]), c));
                    }
                }
                sync();
            }
#pragma unroll 1
            for (int i = li; i < left; i += GS) {
                const uint32_t key = all[i], page = all[kRank + i];
                int above = 0, equal = 0;  // equal ones with lower pages
#pragma unroll 4
                for (int j = 0; j < left; ++j) {
                    above += all[j] > key;
                    equal += all[j] == key && all[kRank + j] < page;
                }
                if (above + equal == need - 1) {  // the last one that is taken
                    s_pick[mq][0] = key;
                    s_pick[mq][1] = (uint32_t)equal + 1;
                }
            }
            sync();
            prefix = s_pick[mq][0];
            need = (int)s_pick[mq][1];
        }
        __syncthreads();  // s_cnt is used again

        // pages above it, and the first `need` of those equal to it, in ascending order
        // (each warp a run of pages)
        const int nlr = choose ? min(max(nrow - base, 0), per) : 0;
        const int seg = ((nlr + S::GROUP - 1) / S::GROUP + 127) / 128 * 128;
        const int lo = min((warp - mq * S::GROUP) * seg, nlr), hi = min(lo + seg, nlr);
        int above = 0, equal = 0;
        if (S::GROUP > 1 || C > 1) {  // how many before this warp's?
#pragma unroll 1
            for (int i = lo + 4 * lane; i < hi; i += 128) {
                const uint4 k4 = *reinterpret_cast<const uint4 *>(key_row + i);
                const uint32_t key[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    above += i + b < hi && key[b] > prefix;
                    equal += i + b < hi && key[b] == prefix;
                }
            }
            above = __reduce_add_sync(0xffffffffu, above);
            equal = __reduce_add_sync(0xffffffffu, equal);
        }
        if (lane == 0) {
            s_cnt[warp][0] = above;
            s_cnt[warp][1] = equal;
        }
        __syncthreads();
        if (li < 2) {
            int s = 0;
#pragma unroll 1
            for (int w = 0; w < S::GROUP; ++w) s += s_cnt[mq * S::GROUP + w][li];
            s_total[mq][li] = s;
        }
        block_sync(C > 1);
        int n_above = 0, n_equal = 0;  // before this warp's pages
        if (C > 1) {  // lane c looks at CTA c
            n_above = lane < rank ? (int)cluster_ld32(cluster_addr(smem_u32(&s_total[mq][0]), lane)) : 0;
            n_equal = lane < rank ? (int)cluster_ld32(cluster_addr(smem_u32(&s_total[mq][1]), lane)) : 0;
            n_above = __reduce_add_sync(0xffffffffu, n_above);
            n_equal = __reduce_add_sync(0xffffffffu, n_equal);
        }
#pragma unroll 1
        for (int w = mq * S::GROUP; w < warp; ++w) {
            n_above += s_cnt[w][0];
            n_equal += s_cnt[w][1];
        }
        int32_t *out = out_of(mq);
#pragma unroll 1
        for (int i0 = lo; i0 < hi; i0 += 1024) {
            uint32_t up = 0, same = 0;  // lane w: of the 32 pages from i0 + 32 w on
#pragma unroll 1
            for (int w0 = 0; w0 < 32 && i0 + w0 * 32 < hi; w0 += 4)
#pragma unroll
                for (int w = w0; w < w0 + 4; ++w) {
                    const int i = i0 + w * 32 + lane;
                    const uint32_t key = i < hi ? key_row[i] : 0u;
                    const uint32_t u = __ballot_sync(0xffffffffu, i < hi && key > prefix);
                    const uint32_t e = __ballot_sync(0xffffffffu, i < hi && key == prefix);
                    if (lane == w) {
                        up = u;
                        same = e;
                    }
                }
            int sum = __popc(up) + (__popc(same) << 16);
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, sum, off);
                if (lane >= off) sum += o;
            }
            const int a = n_above + (sum & 0xffff) - __popc(up);
            const int e = n_equal + (sum >> 16) - __popc(same);
            const int room = max(need - e, 0);
            while (__popc(same) > room) same ^= 0x80000000u >> __clz(same);
            int32_t *o = out + a + min(e, need);
#pragma unroll 1
            for (uint32_t take = up | same; take; take &= take - 1)
                *o++ = base + i0 + lane * 32 + __ffs(take) - 1;
            sum = __shfl_sync(0xffffffffu, sum, 31);
            n_above += sum & 0xffff;
            n_equal += sum >> 16;
        }
        if (C > 1) cluster_sync();  // the others may still read this CTA's counts
    }
    if (g == 0 && rank == 0) {
        const int64_t all = gridDim.x / (unsigned)C / (unsigned)p.r.num_kv_heads;  // tiles
        check_offsets(p.r, tile + threadIdx.x * all, kThreads * all);
    }
}

template <typename S>
int smem_bytes(int cap) {
    return S::KEY_OFF + S::QT * cap * 4;
}

constexpr int kMaxSmem = 224 * 1024;  // beside at most 3 KB of the kernel's own
constexpr int kHalfSmem = 111 * 1024;  // the same of two CTAs per SM

template <int NCH, int NT, int GP, int W>
cudaError_t launch_as(SelectParams p, bool &fits, cudaStream_t stream) {
    using S = Shape<NCH, NT, GP, W>;
    auto kern = select_pages_kernel<NCH, NT, GP, W>;
    const int64_t units = (S::QT > 1 ? row_tiles(p.r, S::QT) : p.r.rows) * p.r.num_kv_heads;
    const int n = (p.r.max_seqlen + p.block_size - 1) >> p.bs_shift;
    // CTAs per tile: several if the scores do not fit; of one query while they have an SM
    // each (8 kv heads of 8 contexts of 100K tokens: 4 CTAs 26 us, 1 43, 8 39) and 512 pages
    // to share out.  (Of several queries the choice in a cluster costs more than it saves:
    // 64 queries of 32K tokens, 8 kv heads: 1 CTA 32 us, 2 33, 4 115.)
    int c = 1;
    auto cap = [&] { return ((n + c - 1) / c + S::STEP - 1) / S::STEP * S::STEP; };
    while (c < 16 && ((S::QT == 1 && units * c <= device_sm_count() && n / c >= 512) ||
                      smem_bytes<S>(cap()) > kMaxSmem))
        c *= 2;
    fits = smem_bytes<S>(cap()) <= kMaxSmem && units * c <= 0x7fffffff;
    if (!fits) return cudaErrorNotSupported;
    p.cluster = c;
    p.cap = cap();
    const int smem = smem_bytes<S>(p.cap);
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kern), smem);
    if (e == cudaSuccess && c > 8) e = ensure_wide_clusters(reinterpret_cast<const void *>(kern));
    if (e != cudaSuccess) return e;
    return launch_cluster(kern, (unsigned)(units * c), c, S::WARPS * 32, (size_t)smem, stream, p);
}

// Eight warps while two CTAs fit an SM, else 16 in one (934 queries of 26K tokens: 132 us
// and 163).
template <int NCH, int NT, int GP>
cudaError_t launch_tiles(const SelectParams &p, bool &fits, cudaStream_t stream) {
    const int n = (p.r.max_seqlen + p.block_size - 1) >> p.bs_shift;
    if (smem_bytes<Shape<NCH, NT, GP, 8>>((n + 31) / 32 * 32) <= kHalfSmem)
        return launch_as<NCH, NT, GP, 8>(p, fits, stream);
    return launch_as<NCH, NT, GP, 16>(p, fits, stream);
}

template <int NCH>
cudaError_t launch_n(const SelectParams &p, cudaStream_t stream) {
    bool fits = false;
    const int G = p.r.group;
    // Tiles of queries where requests have several, 4 on average, and one at a time would
    // take all SMs a few rounds (24K tokens, 8 kv heads of 4, 16 requests of 4 queries: 41 us,
    // 40 one at a time; of 8 44 and 65, of 64 140 and 411; 32K tokens, 1 request of 8 queries:
    // 32 and 16, of 32 32 and 29, of 64 32 and 43); long contexts whose scores do not fit go
    // on with one query at a time.
    if (p.r.cu_q && p.r.rows >= 4LL * p.r.batch &&
        (int64_t)p.r.rows * p.r.num_kv_heads > 3LL * device_sm_count()) {
        const cudaError_t e = G == 1   ? launch_tiles<NCH, 1, 1>(p, fits, stream)
                              : G == 2 ? launch_tiles<NCH, 2, 2>(p, fits, stream)
                              : G <= 4 ? launch_tiles<NCH, 4, 4>(p, fits, stream)
                              : G <= 8 ? launch_tiles<NCH, 8, 8>(p, fits, stream)
                                       : launch_tiles<NCH, 8, 16>(p, fits, stream);
        if (fits) return e;
    }
    // Small CTAs, of which all queries of a decode step have theirs at once (64 queries of
    // 8K tokens, 8 kv heads: 15 us, 20 in CTAs of eight warps); larger ones where a CTA has
    // an SM to itself (one of 400K tokens: 29 us, 33 in CTAs of four).
    if ((int64_t)p.r.rows * p.r.num_kv_heads <= device_sm_count())
        return G <= 8 ? launch_as<NCH, 1, 8, 8>(p, fits, stream)
                      : launch_as<NCH, 2, 16, 8>(p, fits, stream);
    return G <= 8 ? launch_as<NCH, 1, 8, 4>(p, fits, stream)
                  : launch_as<NCH, 2, 16, 4>(p, fits, stream);
}

}  // namespace

cudaError_t launch_select_pages(const SelectParams &p, cudaStream_t stream) {
    switch ((2 * p.r.head_dim + 63) / 64) {
    case 2: return launch_n<2>(p, stream);
    case 3: return launch_n<3>(p, stream);
    case 4: return launch_n<4>(p, stream);
    case 8: return launch_n<8>(p, stream);
    default: return cudaErrorNotSupported;
    }
}

}  // namespace pkv
