// qk_norm_rope.cu -- RMS norm of every q and k head, the rotary embedding and
// the cache write in one pass over a step's new tokens.
//
// Per token t and q or k head row x (D values):
//   y_i = x_i / sqrt(mean_j x_j^2 + eps) * w_i
//   the pairs of the first rotary_dim dimensions turn by the table's angle at
//   positions[t], as in rope_reshape_and_cache; the result rounds once.
// The rotated key (as rounded) and the value go to the pools at the token's
// slot: copied, or quantised as in reshape_and_cache_fp8.
//
// HBM bound: q, k, v are read once, q_out, k_out and the pools written once.
// A head row is held by LPR = D/8 lanes (rounded up to a power of two) of a
// warp, eight values each, so the sum of squares and a neox pair's other half
// are shuffles and nothing is read twice.  A group of LPR lanes takes several
// heads of one token, with the token's cos/sin and the weights in registers.
#include <type_traits>

#include "pkv_fp8.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 128;
constexpr int kCtas = 7;  // resident per SM (bf16 pools)

// Eight values of a head row as they lie in memory.
template <typename T>
struct Raw8 {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = *(reinterpret_cast<const uint4 *>(p) + i);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        if constexpr (sizeof(T) == 2) {
            const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
                x[4 * i] = __uint_as_float(v[i].x);
                x[4 * i + 1] = __uint_as_float(v[i].y);
                x[4 * i + 2] = __uint_as_float(v[i].z);
                x[4 * i + 3] = __uint_as_float(v[i].w);
            }
        }
    }
};

template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&x)[8]) {
    Raw8<T> r;
    r.load(p);
    r.get(x);
}

template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&x)[8]) {
    if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                                   pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    } else {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *(reinterpret_cast<float4 *>(p) + 1) = make_float4(x[4], x[5], x[6], x[7]);
    }
}

// The value a store of T keeps.
template <typename T>
__device__ __forceinline__ float rounded(float x) {
    if constexpr (sizeof(T) == 2) return __bfloat162float(__float2bfloat16_rn(x));
    return x;
}

// The norm's weights of eight dimensions.
template <typename T>
__device__ __forceinline__ void load_weights(const NormRopeParams &p, const void *w, int d0,
                                             bool active, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (!active) return;
    if (p.weight_f32)
        load8<float>(static_cast<const float *>(w) + d0, x);
    else
        load8<T>(static_cast<const T *>(w) + d0, x);
}

// Norm and rotation of one head row, eight values per lane of LPR; every lane
// of the warp takes part.
template <typename T, int LPR, bool NEOX>
__device__ __forceinline__ void norm_rotate(const Raw8<T> &raw, const float (&w)[8],
                                            const float (&cs)[NEOX ? 8 : 4],
                                            const float (&sn)[NEOX ? 8 : 4], float inv_d,
                                            float eps, int src_lane, float (&y)[8]) {
    float x[8];
    raw.get(x);
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        s0 = fmaf(x[i], x[i], s0);
        s1 = fmaf(x[i + 1], x[i + 1], s1);
    }
    float ss = s0 + s1;
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float inv = rsqrtf(fmaf(ss, inv_d, eps));
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] * inv * w[i];
    if constexpr (NEOX) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float o = __shfl_sync(0xffffffffu, y[i], src_lane);
            y[i] = fmaf(o, sn[i], y[i] * cs[i]);  // not rotated: y * 1 + y * 0
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = y[2 * i], b = y[2 * i + 1];
            y[2 * i] = fmaf(-b, sn[i], a * cs[i]);
            y[2 * i + 1] = fmaf(a, sn[i], b * cs[i]);
        }
    }
}

// Store one row of a k or v head to the pools: a copy, or codes and scale.
// Every lane of the warp calls it (shuffles); `store` says whether this
// lane's group writes.
template <typename T, int LPR, bool FP8>
__device__ __forceinline__ void pool_store(const PoolArgs &p, const PoolSlot &s, bool store,
                                           int g, bool is_v, int sub, bool active,
                                           const float (&x)[8]) {
    if constexpr (FP8) {
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1)
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        if (!store) return;
        const uint32_t byte = scale_byte(amax);
        const float inv = scale_inverse(byte);
        const bool bad = byte == kScaleNaN;
        if (active)
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(is_v ? p.v : p.k) + s.row +
                                       (int64_t)g * s.row_step + sub * 8) =
                make_uint2(quant4(x, inv, bad), quant4(x + 4, inv, bad));
        if (sub == 0)
            (is_v ? p.v_scale : p.k_scale)[s.scale + g * p.block_size] = (uint8_t)byte;
    } else {
        if (store && active)
            store8<T>(static_cast<T *>(is_v ? p.v : p.k) + s.row + (int64_t)g * s.row_step +
                          sub * 8,
                      x);
    }
}

// gpt groups of LPR lanes share a token (gpt a power of two dividing the
// CTA's groups); group r0 takes the heads r0, r0 + gpt, ... of q, of k and of
// v.  The first rows of all three are asked for before anything else, so that
// one trip to memory covers them, the position, the slot and the weights.
// Measured on 8448 tokens of 32 + 2 * 8 heads of 128 into bf16 pools (GB300,
// 225 MB): 42 us, 79 % of a copy's rate.  Seven CTAs per SM and two q rows ahead
// (uncapped and four rows: 56 us; one row: 46 us; the cap costs the neox variant
// 20 bytes of spills at its 72 registers); two groups per token (each
// cos/sin row is loaded by fewer groups) take 42 us, four 44, eight 48.
template <typename T, int LPR, bool FP8, bool NEOX>
__global__ void __launch_bounds__(kThreads, sizeof(T) != 2 ? 4 : FP8 ? kCtas - 1 : kCtas)
norm_rope_kernel(const NormRopeParams p, int gpt) {
    pdl_trigger();
    pdl_wait();
    constexpr int kGroups = kThreads / LPR;
    constexpr int UQ = 2;  // q rows of a batch; the next batch is in flight meanwhile
    const int sub = threadIdx.x % LPR, grp = threadIdx.x / LPR;
    const int D = p.pool.head_dim, Hq = p.num_qo_heads, Hkv = p.pool.num_kv_heads;
    const bool active = sub * 8 < D;
    const int64_t t = (int64_t)blockIdx.x * (kGroups / gpt) + grp / gpt;
    const int r0 = grp & (gpt - 1);
    const bool live = t < p.num_tokens, loads = live && active;
    const int d0 = sub * 8;  // this lane's dimensions are d0 .. d0 + 7

    const T *q_in = static_cast<const T *>(p.query) + t * p.q_stride + d0;
    const T *k_in = static_cast<const T *>(p.key) + t * p.k_stride + d0;
    const T *v_in = static_cast<const T *>(p.value) + t * p.v_stride + d0;
    Raw8<T> rq[UQ], rk, rv;
#pragma unroll
    for (int u = 0; u < UQ; ++u) {
        rq[u].zero();
        if (loads && u * gpt + r0 < Hq) rq[u].load(q_in + (u * gpt + r0) * D);
    }
    rk.zero();
    rv.zero();
    if (loads && r0 < Hkv) {
        rk.load(k_in + r0 * D);
        rv.load(v_in + r0 * D);
    }

    int64_t pos = -1, slot = -1;
    if (live) {
        pos = __ldg(p.positions + t);
        slot = __ldg(p.slot_mapping + t);
        if (pos < 0 || pos >= p.max_position) {
            if (sub == 0 && r0 == 0) flag_error(p.dev_error, PKV_DEVERR_POSITION);
            pos = -1;  // the token is left as it is
        } else if (slot >= p.pool.capacity) {
            if (sub == 0 && r0 == 0) flag_error(p.dev_error, PKV_DEVERR_SLOT);
            slot = -1;
        }
    }
    const bool on = live && pos >= 0, cached = on && slot >= 0;
    const PoolSlot ps = pool_slot(p.pool, cached ? (uint32_t)slot : 0u);

    // neox: lane sub < half_l holds the first member of its pairs and lane
    // sub + half_l the second
    const int rd = p.rotary_dim, half_l = rd / 16;
    const bool rot = active && d0 < rd;
    constexpr int NF = NEOX ? 8 : 4;  // frequencies per lane
    float cs[NF], sn[NF], w[8];
#pragma unroll
    for (int i = 0; i < NF; ++i) {
        cs[i] = 1.f;
        sn[i] = 0.f;
    }
    load_weights<T>(p, p.q_weight, d0, active && Hq > 0, w);
    if (on && rot) {
        const int f0 = NEOX ? 8 * (sub < half_l ? sub : sub - half_l) : 4 * sub;
        const float4 *row = reinterpret_cast<const float4 *>(p.cos_sin + pos * (rd / 2) + f0);
#pragma unroll
        for (int i = 0; i < NF; i += 2) {
            const float4 v = __ldg(row + i / 2);
            cs[i] = v.x;
            sn[i] = v.y;
            cs[i + 1] = v.z;
            sn[i + 1] = v.w;
        }
        if (NEOX && sub < half_l)  // x_a' = x_a c - x_b s
#pragma unroll
            for (int i = 0; i < NF; ++i) sn[i] = -sn[i];
    }
    const int partner = NEOX && rot ? (sub < half_l ? sub + half_l : sub - half_l) : sub;
    const int src_lane = (threadIdx.x & 31) - sub + partner;
    const float inv_d = 1.f / (float)D;

    // every lane of the CTA makes the same rounds
    T *q_out = static_cast<T *>(p.query_out) + t * p.qo_stride + d0;
    for (int base = 0; base < Hq; base += gpt * UQ) {
        Raw8<T> next[UQ];  // asked for before this batch is worked on
#pragma unroll
        for (int u = 0; u < UQ; ++u) {
            const int h = base + (UQ + u) * gpt + r0;
            next[u].zero();
            if (loads && h < Hq) next[u].load(q_in + h * D);
        }
#pragma unroll
        for (int u = 0; u < UQ; ++u) {
            if (base + u * gpt >= Hq) break;
            const int h = base + u * gpt + r0;
            float y[8];
            norm_rotate<T, LPR, NEOX>(rq[u], w, cs, sn, inv_d, p.eps, src_lane, y);
            if (on && active && h < Hq) store8<T>(q_out + h * D, y);
            rq[u] = next[u];
        }
    }
    load_weights<T>(p, p.k_weight, d0, active, w);
    T *k_out = static_cast<T *>(p.key_out) + t * p.ko_stride + d0;
    for (int base = 0; base < Hkv; base += gpt) {
        const int g = base + r0;
        if (base > 0 && loads && g < Hkv) {
            rk.load(k_in + g * D);
            rv.load(v_in + g * D);
        }
        float y[8];
        norm_rotate<T, LPR, NEOX>(rk, w, cs, sn, inv_d, p.eps, src_lane, y);
        if (on && active && g < Hkv) store8<T>(k_out + g * D, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = rounded<T>(y[i]);
        pool_store<T, LPR, FP8>(p.pool, ps, cached && g < Hkv, g, false, sub, active, y);
        rv.get(y);
        pool_store<T, LPR, FP8>(p.pool, ps, cached && g < Hkv, g, true, sub, active, y);
    }
}

template <typename T, int LPR, bool FP8>
cudaError_t launch_lpr(const NormRopeParams &p, cudaStream_t stream) {
    constexpr int kGroups = kThreads / LPR;
    const int rows = p.num_qo_heads + p.pool.num_kv_heads;
    int gpt = 1;
    while (gpt * 2 <= kGroups && gpt * 2 <= rows) gpt *= 2;
    // few tokens: as many groups as help one token; many: two, while the CTAs
    // still fill the SMs twice
    while (gpt > 2 && p.num_tokens * gpt / kGroups > (int64_t)device_sm_count() * kCtas * 2)
        gpt /= 2;
    const int64_t per_cta = kGroups / gpt;
    const int64_t blocks = (p.num_tokens + per_cta - 1) / per_cta;
    if (blocks > 0x7fffffffLL) return cudaErrorNotSupported;
    auto kern = p.neox ? norm_rope_kernel<T, LPR, FP8, true> : norm_rope_kernel<T, LPR, FP8, false>;
    return launch_pdl(kern, dim3((unsigned)blocks), dim3(kThreads), 0, stream, p, gpt);
}

template <typename T, bool FP8>
cudaError_t launch_t(const NormRopeParams &p, cudaStream_t stream) {
    const int D = p.pool.head_dim;
    if (D <= 64) return launch_lpr<T, 8, FP8>(p, stream);
    if (D <= 128) return launch_lpr<T, 16, FP8>(p, stream);
    return launch_lpr<T, 32, FP8>(p, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams &p, int dtype, cudaStream_t stream) {
    if (p.num_tokens == 0) return cudaSuccess;
    if (p.pool.k_scale)
        return dtype == PKV_F32 ? launch_t<float, true>(p, stream)
                                : launch_t<__nv_bfloat16, true>(p, stream);
    return dtype == PKV_F32 ? launch_t<float, false>(p, stream)
                            : launch_t<__nv_bfloat16, false>(p, stream);
}

}  // namespace pkv
