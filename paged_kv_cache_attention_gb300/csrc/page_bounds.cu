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
// takes a page of a kv head: its lanes hold 16 bytes of a row each, all rows of a
// page are in flight at once, the rows' lanes meet in shuffles at the end.
#include <cuda_fp16.h>

#include "pkv_sparse.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxTokens = 128;  // of a CTA
constexpr int kAhead = 32;       // tokens looked at beyond one for its page

// bytes 0..3 of w: clamped codes of four floats times inv (rounded down, or up)
template <bool UP>
__device__ __forceinline__ uint32_t codes4(const float *x, float inv) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float y = x[i] * inv;  // exact, or less than the smallest float
        int c = UP ? (int)ceilf(y) : (int)floorf(y);
        if (UP && x[i] > 0.f) c = max(c, 1);
        if (!UP && x[i] < 0.f) c = min(c, -1);
        w |= ((uint32_t)c & 0xffu) << (8 * i);
    }
    return w;
}

// The 16 bytes of a row that a lane holds: 8 bf16 values, or 16 codes times f.
template <bool FP8>
__device__ __forceinline__ void load_row(const uint4 &w, float f, float (&x)[FP8 ? 16 : 8]) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (FP8) {
            uint32_t lo, hi;
            e4m3_to_f16(v[i], lo, hi);
            const float2 a = __half22float2(*reinterpret_cast<__half2 *>(&lo));
            const float2 b = __half22float2(*reinterpret_cast<__half2 *>(&hi));
            x[4 * i] = a.x * f;
            x[4 * i + 1] = a.y * f;
            x[4 * i + 2] = b.x * f;
            x[4 * i + 3] = b.y * f;
        } else {
            x[2 * i] = __uint_as_float(v[i] << 16);
            x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
        }
    }
}

template <bool FP8, int BS>
__global__ void __launch_bounds__(kThreads) page_bounds_kernel(const BoundsParams p) {
    constexpr int V = FP8 ? 16 : 8;
    __shared__ int64_t s_slot[kMaxTokens + kAhead];
    __shared__ int s_work[kMaxTokens];  // tokens that are the last of their page
    __shared__ int s_count;
    pdl_wait();
    const int g = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t0 = (int64_t)blockIdx.y * p.tokens_per_cta;
    const int nt = (int)min((int64_t)p.tokens_per_cta, p.num_tokens - t0);
    if (threadIdx.x == 0) s_count = 0;
    for (int i = threadIdx.x; i < nt + kAhead; i += kThreads) {
        int64_t s = t0 + i < p.num_tokens ? p.slots[t0 + i] : -1;
        if (s >= p.capacity) {
            if (i < nt) flag_error(p.dev_error, PKV_DEVERR_SLOT);
            s = -1;
        }
        s_slot[i] = s < 0 ? -1 : s;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nt; i += kThreads) {
        const int64_t s = s_slot[i];
        if (s < 0) continue;
        bool last = true;
        for (int j = 1; j <= kAhead && last; ++j) {
            const int64_t o = s_slot[i + j];
            last = o < 0 || (o >> p.bs_shift) != (s >> p.bs_shift);
        }
        if (last) s_work[atomicAdd(&s_count, 1)] = i;
    }
    __syncthreads();
    const int work = s_count, D = p.head_dim;
    const int lanes = D / V;             // lanes of a row: 4 .. 32
    const int span = lanes <= 4 ? 4 : lanes <= 8 ? 8 : lanes <= 16 ? 16 : 32;
    const int step = 32 / span;          // rows side by side
    const int c = lane & (span - 1), r0 = lane / span;
    const bool in = c < lanes;
    for (int w = warp; w < work; w += kWarps) {
        const int64_t slot = s_slot[s_work[w]];
        const int64_t blk = slot >> p.bs_shift;
        const int n = (int)(slot & (BS - 1)) + 1;
        const int64_t unit = blk * p.num_kv_heads + g;
        const int64_t row0 = p.hnd ? unit * BS : blk * BS * p.num_kv_heads + g;
        const int64_t rstep = p.hnd ? 1 : p.num_kv_heads;
        float lo[V], hi[V];
        bool ok = true;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            lo[i] = INFINITY;
            hi[i] = -INFINITY;
        }
#pragma unroll 8
        for (int r = r0; r < n; r += step) {
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            float f = 1.f;
            if (in)
                x = *reinterpret_cast<const uint4 *>(static_cast<const char *>(p.k) +
                                                     (row0 + r * rstep) * D * (FP8 ? 1 : 2) +
                                                     c * 16);
            if (FP8) {
                const uint32_t byte = p.k_scale[unit * BS + r];
                ok = ok && byte != kScaleNaN;
                f = scale_value(byte == kScaleNaN ? 127u : byte);
            }
            float y[V];
            load_row<FP8>(x, f, y);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                ok = ok && fabsf(y[i]) < INFINITY;  // false for a NaN too
                lo[i] = fminf(lo[i], y[i]);
                hi[i] = fmaxf(hi[i], y[i]);
            }
        }
        for (int off = span; off < 32; off <<= 1)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                lo[i] = fminf(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], off));
                hi[i] = fmaxf(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], off));
            }
        ok = __all_sync(0xffffffffu, ok);
        uint32_t amax = 0;
        if (in && ok)
#pragma unroll
            for (int i = 0; i < V; ++i)
                amax = max(amax, max(__float_as_uint(fabsf(lo[i])), __float_as_uint(fabsf(hi[i]))));
        amax = __reduce_max_sync(0xffffffffu, amax);
        // amax = m * 2^x with 1 <= m < 2 and 127 = 1.984375 * 2^6: e = x - 6, one more
        // above 1.984375 (a carry out of the mantissa)
        const int e = max((int)((amax + 0x1ffffu) >> 23) - 127 - 6, -126);
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        if (r0 == 0 && in) {
            int8_t *out = p.bounds + unit * 2 * D + c * V;
#pragma unroll
            for (int i = 0; i < V / 4; ++i) {
                *reinterpret_cast<uint32_t *>(out + 4 * i) = ok ? codes4<false>(lo + 4 * i, inv) : 0u;
                *reinterpret_cast<uint32_t *>(out + D + 4 * i) = ok ? codes4<true>(hi + 4 * i, inv) : 0u;
            }
            if (c == 0) p.bounds_scale[unit] = ok ? (uint8_t)(e + 127) : (uint8_t)kScaleNaN;
        }
    }
}

}  // namespace

cudaError_t launch_page_bounds(const BoundsParams &p0, cudaStream_t stream) {
    BoundsParams p = p0;
    // few tokens: a CTA each; prompts: as many as fill a CTA's warps with pages
    const int64_t fill = 4LL * device_sm_count();
    int per = 8;
    while (per < kMaxTokens && (p.num_tokens + per - 1) / per * p.num_kv_heads > fill) per *= 2;
    p.tokens_per_cta = per;
    const int64_t y = (p.num_tokens + per - 1) / per;
    if (y > 65535) return cudaErrorNotSupported;
    auto kern = p.k_scale ? (p.block_size == 16 ? page_bounds_kernel<true, 16>
                                                : page_bounds_kernel<true, 32>)
                          : (p.block_size == 16 ? page_bounds_kernel<false, 16>
                                                : page_bounds_kernel<false, 32>);
    return launch_pdl(kern, dim3(p.num_kv_heads, (unsigned)y), dim3(kThreads), 0, stream, p);
}

}  // namespace pkv
