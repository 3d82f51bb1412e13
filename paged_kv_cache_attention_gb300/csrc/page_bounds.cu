// page_bounds.cu -- the least and the largest key of every page, per channel, in 8
// bits: what select_pages scores a page with, without reading its keys.
//
// For a (page, kv head) with rows 0 .. n - 1 written:
//   lo_d = min_r k[r, d],  hi_d = max_r k[r, d]       (exact: no sum, no order)
//   e    = the least exponent >= -126 with max_d max(|lo_d|, |hi_d|) <= 127 * 2^e
//   codes floor(lo_d * 2^-e) and ceil(hi_d * 2^-e), byte e + 127
// Rounding is outward, so the codes times 2^e still bound every key.  A page with
// a key that is not finite has byte 255 and codes 0.
//
// Which pages: the tokens of a step come in order, so the last token of a page
// among its neighbours in slot_mapping says that rows 0 .. slot % bs are there;
// the page is read again as a whole (what older steps wrote is not kept in 8 bits
// and merged: codes would depend on the steps, and errors would add up).
//
// HBM bound: n * D keys read, 2 D + 1 bytes written per page and kv head.  A warp
// works by itself: it looks through a window of up to 32 tokens and takes the pages
// that end there, for some or all kv heads.  Its lanes hold 16 bytes of a row each,
// all rows of a page are in flight at once, and the rows' lanes meet in shuffles.
// Least and largest are kept in the 16-bit type that is exact: bf16, or for 8-bit
// pools f16 relative to the page's largest row scale (codes times 2^0 .. 2^-15 are
// f16 values; pages whose scales lie further apart go by fp32).
//
// Measured (8 kv heads of 128): 64 tokens 2.9 us; 16K bf16 tokens in 8 prompts 7.0 us;
// 88K tokens of 8-bit pages in 13 prompts 23.9 us from HBM (97 MB, 14.4 at its rate), 21.6
// where L2 still holds some of them (24.4 with the two CTAs per SM that unbounded registers
// leave room for).  Issue at 50%, DRAM at 45%: a warp loads a page, then works on it.
#include <cuda_fp16.h>

#include "pkv_sparse.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
// Rounds of warps before a warp takes more kv heads (88K 8-bit tokens: 5 and 8 21.6 us, 12
// 25; 2, with two CTAs per SM, 33 where 8 took 24.4).
constexpr int kRounds = 8;

template <bool FP8>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {  // a NaN stays
    uint32_t r;
    if (FP8)
        asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <bool FP8>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    if (FP8)
        asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        r = bf16x2_max_nan(a, b);
    return r;
}

// The two values of a pair as floats; FP8: times f.
template <bool FP8>
__device__ __forceinline__ void unpack2(uint32_t w, float f, float &x, float &y) {
    if (FP8) {
        const float2 v = __half22float2(*reinterpret_cast<__half2 *>(&w));
        x = v.x * f;
        y = v.y * f;
    } else {
        x = __uint_as_float(w << 16);
        y = __uint_as_float(w & 0xffff0000u);
    }
}

// The code of x * inv rounded up, for a lower bound (x has its sign turned) with the sign
// turned back.  The product is exact, or below the smallest float: still not 0.
__device__ __forceinline__ uint32_t code_of(float x, float inv, bool upper) {
    const int c = max(__float2int_ru(x * inv), x > 0.f ? 1 : -127);
    return (uint32_t)(upper ? c : -c) & 0xffu;
}

// Least and largest of a page whose row scales lie far apart, in fp32; the channels
// 16 c .. of row r0, r0 + step, ..
__device__ __noinline__ void fp32_bounds(const char *rows, int64_t row_bytes, const uint8_t *scale,
                                         int n, int r0, int step, float (&lo)[16], float (&hi)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        lo[i] = INFINITY;
        hi[i] = -INFINITY;
    }
    for (int r = r0; r < n; r += step) {
        const uint4 w = *reinterpret_cast<const uint4 *>(rows + r * row_bytes);
        const float f = scale_value(scale[r]);
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t p[2];
            e4m3_to_f16(v[i], p[0], p[1]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float x, y;
                unpack2<true>(p[k], f, x, y);
                lo[4 * i + 2 * k] = fminf(lo[4 * i + 2 * k], x);
                hi[4 * i + 2 * k] = fmaxf(hi[4 * i + 2 * k], x);
                lo[4 * i + 2 * k + 1] = fminf(lo[4 * i + 2 * k + 1], y);
                hi[4 * i + 2 * k + 1] = fmaxf(hi[4 * i + 2 * k + 1], y);
            }
        }
    }
}

// SPAN: lanes of a row (16 bytes each), a power of two; the last ones may be idle.
template <bool FP8, int BS, int SPAN>
__global__ void __launch_bounds__(kThreads, 3) page_bounds_kernel(const BoundsParams p) {
    constexpr int V = FP8 ? 16 : 8;     // channels of a lane
    constexpr int P = V / 2;            // pairs
    constexpr int STEP = 32 / SPAN;     // rows side by side
    constexpr int ROWS = BS / STEP;     // rows of a lane
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t id = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int groups = (p.num_kv_heads + p.heads_per_warp - 1) / p.heads_per_warp;
    const int64_t window = id / groups;
    const int g0 = (int)(id - window * groups) * p.heads_per_warp;
    const int64_t t0 = window * p.tokens_per_warp;
    if (t0 >= p.num_tokens) return;

    // the tokens of the window that are the last of their page among the next 32
    auto slot_of = [&](int64_t t) {
        int64_t s = t < p.num_tokens ? p.slots[t] : -1;
        if (s >= p.capacity) {
            if (g0 == 0 && t < t0 + p.tokens_per_warp) flag_error(p.dev_error, PKV_DEVERR_SLOT);
            s = -1;
        }
        return s < 0 ? -1 : (int)s;  // (slots are below 2^31)
    };
    const int slot = slot_of(t0 + lane), next = slot_of(t0 + 32 + lane);
    const int page = slot < 0 ? -1 - lane : slot >> p.bs_shift;
    const int next_page = next < 0 ? -1 : next >> p.bs_shift;
    const uint32_t alike = __match_any_sync(0xffffffffu, page);
    const uint32_t upto = (2u << lane) - 1u;  // this lane and those before it
    uint32_t work = __ballot_sync(0xffffffffu,
                                  slot >= 0 && lane < p.tokens_per_warp && !(alike & ~upto));
    for (uint32_t rest = work; rest; rest &= rest - 1) {
        const int c = __ffs(rest) - 1;
        const int pc = __shfl_sync(0xffffffffu, page, c);
        if (__ballot_sync(0xffffffffu, next_page == pc) & ((2u << c) - 1u)) work &= ~(1u << c);
    }

    const int D = p.head_dim, E = FP8 ? 1 : 2;
    const int c = lane & (SPAN - 1), r0 = lane / SPAN;
    const bool in = c * V < D;
    const int64_t row_bytes = (int64_t)(p.hnd ? 1 : p.num_kv_heads) * D * E;
    const int heads = min(p.heads_per_warp, p.num_kv_heads - g0);
    for (; work; work &= work - 1) {
        const int s = __shfl_sync(0xffffffffu, slot, __ffs(work) - 1);
        const int64_t blk = s >> p.bs_shift;
        const int n = (s & (BS - 1)) + 1;
#pragma unroll 1
        for (int h = 0; h < heads; ++h) {
            const int g = g0 + h;
            const int64_t unit = blk * p.num_kv_heads + g;
            const char *rows = static_cast<const char *>(p.k) +
                               (p.hnd ? unit * BS * D * E
                                      : (blk * BS * p.num_kv_heads + g) * (int64_t)D * E) +
                               (in ? c * 16 : 0);
            uint4 raw[ROWS];  // (rows past the last: the last again)
#pragma unroll
            for (int i = 0; i < ROWS; ++i)
                raw[i] = *reinterpret_cast<const uint4 *>(rows + min(r0 + i * STEP, n - 1) * row_bytes);
            int byte = 0, top = 0;
            bool ok = true, near = true;
            if (FP8) {
                byte = p.k_scale[unit * BS + min(lane, n - 1)];  // lane = row
                ok = __all_sync(0xffffffffu, byte != (int)kScaleNaN);
                top = __reduce_max_sync(0xffffffffu, byte);
                near = __all_sync(0xffffffffu, byte >= top - 15);
            }
            uint32_t lo[P], hi[P];
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
                uint32_t v[P];
                if (FP8) {
                    // the row's scale relative to the largest, 2^0 .. 2^-15, as an f16 pair
                    const int d = __shfl_sync(0xffffffffu, byte, min(r0 + i * STEP, n - 1)) - top;
                    const uint32_t f1 = d >= -14 ? (uint32_t)(15 + d) << 10 : 0x200u;
                    const uint32_t f = f1 | (f1 << 16);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        e4m3_to_f16(w[k], v[2 * k % P], v[(2 * k + 1) % P]);
                        v[2 * k % P] = f16x2_mul(v[2 * k % P], f);
                        v[(2 * k + 1) % P] = f16x2_mul(v[(2 * k + 1) % P], f);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = w[k];
                }
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    lo[k] = i == 0 ? v[k] : min2<FP8>(lo[k], v[k]);
                    hi[k] = i == 0 ? v[k] : max2<FP8>(hi[k], v[k]);
                }
            }
            // The rows' lanes meet and share the channels out: lanes 16 apart keep the upper
            // bounds, or the lower ones with their signs turned (so that all are largest
            // values); lanes 8 and 4 apart keep half of their channels each.
            const bool up = STEP == 1 || (lane & 16);
            const float f = FP8 ? scale_value((uint32_t)top) : 1.f;
            constexpr int LEVELS = STEP == 8 ? 3 : STEP == 4 ? 2 : STEP == 2 ? 1 : 0;
            constexpr int N = LEVELS == 0 ? V : V >> (LEVELS - 1);  // values a lane keeps
            float x[N], y[LEVELS == 0 ? V : 1];  // y: the lower bounds of a row of 32 lanes
            int at = 0;                          // the first one's channel, of the lane's V
            if constexpr (LEVELS == 0) {
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    unpack2<FP8>(hi[k], f, x[2 * k], x[2 * k + 1]);
                    unpack2<FP8>(lo[k] ^ 0x80008000u, f, y[2 * k], y[2 * k + 1]);
                }
            } else {
                uint32_t v[P];
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    const uint32_t low = lo[k] ^ 0x80008000u;
                    v[k] = max2<FP8>(up ? hi[k] : low,
                                     __shfl_xor_sync(0xffffffffu, up ? low : hi[k], 16));
                }
#pragma unroll
                for (int level = 1; level < LEVELS; ++level) {
                    const int m = P >> level, off = 16 >> level;
                    const bool second = lane & off;
                    if (second) at += 2 * m;
#pragma unroll
                    for (int k = 0; k < m; ++k)
                        v[k] = max2<FP8>(second ? v[k + m] : v[k],
                                         __shfl_xor_sync(0xffffffffu, second ? v[k] : v[k + m], off));
                }
#pragma unroll
                for (int k = 0; k < N / 2; ++k) unpack2<FP8>(v[k], f, x[2 * k], x[2 * k + 1]);
            }
            if constexpr (FP8) {
                if (ok && !near) {  // rare
                    float a[V], b[V];
                    fp32_bounds(rows, row_bytes, p.k_scale + unit * BS, n, r0, STEP, a, b);
                    for (int off = SPAN; off < 32; off <<= 1)
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            a[i] = fminf(a[i], __shfl_xor_sync(0xffffffffu, a[i], off));
                            b[i] = fmaxf(b[i], __shfl_xor_sync(0xffffffffu, b[i], off));
                        }
#pragma unroll
                    for (int i = 0; i < V; ++i)
#pragma unroll
                        for (int k = 0; k < N; ++k)
                            if (i == at + k) x[k] = up ? b[i] : -a[i];
                }
            }
            uint32_t amax = 0;  // (the bits of a NaN are above an infinity's)
#pragma unroll
            for (int k = 0; k < N; ++k) amax = max(amax, __float_as_uint(fabsf(x[k])));
            if (LEVELS == 0)
#pragma unroll
                for (int k = 0; k < N; ++k) amax = max(amax, __float_as_uint(fabsf(y[k])));
            amax = __reduce_max_sync(0xffffffffu, in ? amax : 0u);
            ok = ok && amax < 0x7f800000u;
            // amax = m * 2^x with 1 <= m < 2 and 127 = 1.984375 * 2^6: e = x - 6, one more
            // above 1.984375 (a carry out of the mantissa)
            const int e = max((int)((amax + 0x1ffffu) >> 23) - 127 - 6, -126);
            const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
            int8_t *out = p.bounds + unit * 2 * D + c * V + at;
            auto store = [&](const float *z, bool upper) {
                uint32_t w[(N + 3) / 4] = {};
#pragma unroll
                for (int k = 0; k < N; ++k)
                    w[k / 4] |= code_of(z[k], inv, upper) << (8 * (k % 4));
#pragma unroll
                for (int k = 0; k < N / 4; ++k)
                    reinterpret_cast<uint32_t *>(out + (upper ? D : 0))[k] = ok ? w[k] : 0u;
            };
            if (in) {
                store(x, up);
                if (LEVELS == 0) store(y, false);
            }
            if (lane == 0) p.bounds_scale[unit] = ok ? (uint8_t)(e + 127) : (uint8_t)kScaleNaN;
        }
    }
}

template <bool FP8, int BS>
cudaError_t launch_span(const BoundsParams &p, unsigned grid, cudaStream_t stream) {
    constexpr int L = FP8 ? 4 : 8;  // lanes of a row of 64 channels
    auto kern = p.head_dim <= 64    ? page_bounds_kernel<FP8, BS, L>
                : p.head_dim <= 128 ? page_bounds_kernel<FP8, BS, 2 * L>
                                    : page_bounds_kernel<FP8, BS, 4 * L>;
    return launch_pdl(kern, dim3(grid), dim3(kThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_page_bounds(const BoundsParams &p0, cudaStream_t stream) {
    BoundsParams p = p0;
    // A warp per token and kv head while they all run at once (a decode step); then
    // windows of more tokens, then more kv heads per warp.  (64 tokens: windows of 1
    // token 2.9 us, 4 5.2, 32 26; 1000 tokens 8.0, 6.6, 27; 16K tokens 12.6, 8.3, 7.1.)
    const int64_t warps = 16LL * device_sm_count();
    p.tokens_per_warp = 1;
    p.heads_per_warp = 1;
    while (p.tokens_per_warp < 32 &&
           (p.num_tokens + p.tokens_per_warp - 1) / p.tokens_per_warp * p.num_kv_heads > warps)
        p.tokens_per_warp *= 2;
    const int64_t windows = (p.num_tokens + p.tokens_per_warp - 1) / p.tokens_per_warp;
    while (p.heads_per_warp < p.num_kv_heads &&
           windows * (p.num_kv_heads / p.heads_per_warp) > kRounds * warps)
        p.heads_per_warp *= 2;
    const int groups = (p.num_kv_heads + p.heads_per_warp - 1) / p.heads_per_warp;
    const unsigned grid = (unsigned)((windows * groups + kWarps - 1) / kWarps);
    if (p.k_scale)
        return p.block_size == 16 ? launch_span<true, 16>(p, grid, stream)
                                  : launch_span<true, 32>(p, grid, stream);
    return p.block_size == 16 ? launch_span<false, 16>(p, grid, stream)
                              : launch_span<false, 32>(p, grid, stream);
}

}  // namespace pkv
