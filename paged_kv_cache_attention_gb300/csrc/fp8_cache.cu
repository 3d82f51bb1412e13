// fp8_cache.cu -- the 8-bit cache: quantising rows as they are written
// (reshape_and_cache_fp8) and reading them back (gather_cache_fp8).
//
// Per head row x of a new token (D values of one kv head):
//   a = max |x_i|;  e = ceil(log2(a / 448)) in [-126, 119];
//   code_i = e4m3(x_i * 2^-e)  (nearest even, saturating);  byte = e + 127.
// Reading back is code_i * 2^e, exact in bf16.  A row with a NaN or an
// infinity has byte 255 and reads back as NaN throughout.
//
// Both are bound by HBM: the write moves D*(2 + 1) + 1 bytes per head row
// (bf16), the read-back the same backwards.  A head row is taken by D/16
// lanes of a warp (rounded up to a power of two), 16 values each: 16-byte
// code vectors, the maximum in two to four shuffles, no shared memory.  Several
// rows per thread are in flight at once; no address needs a division.
#include "pkv_fp8.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;

// 16 values of a head row as they lie in memory, and what the write asks of
// them.
template <typename T>
struct Row16;

template <>
struct Row16<__nv_bfloat16> {
    uint32_t w[8];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p));
        const uint4 b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 0u;
    }
    // fp32 bits of the largest magnitude (at or above infinity's: not finite)
    __device__ __forceinline__ uint32_t amax() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = bf16x2_max_nan(m, w[i] & 0x7fff7fffu);
        return max(m << 16, m & 0xffff0000u);
    }
    __device__ __forceinline__ float at(int i) const {
        return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
};

template <>
struct Row16<float> {
    float x[16];
    __device__ __forceinline__ void load(const float *p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = __ldg(reinterpret_cast<const float4 *>(p) + i);
            x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = 0.f;
    }
    __device__ __forceinline__ uint32_t amax() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
        return m;
    }
    __device__ __forceinline__ float at(int i) const { return x[i]; }
};

// gpt groups of LPR lanes share a token (gpt a power of two dividing the
// CTA's groups); group r0 takes the head rows r0, r0 + gpt, .. of the 2 H rows
// of k and v, for UNR tokens at a time.
// Registers are capped for six CTAs per SM: on 66001 tokens of 8 heads of 128
// (GB300) that takes 66 us, 91 % of a copy's rate; five CTAs 75, uncapped with
// four tokens in flight 98, one token 87.
template <typename T, int LPR, int UNR>
__global__ void __launch_bounds__(kThreads, 6)
quant_write_kernel(const QuantWriteParams p, int gpt) {
    pdl_trigger();
    pdl_wait();
    const int sub = threadIdx.x % LPR, grp = threadIdx.x / LPR;
    const int H = p.pool.num_kv_heads, D = p.pool.head_dim;
    const bool active = sub * 16 < D;
    const int tpb = kThreads / LPR / gpt;  // tokens per CTA and step
    const int r0 = grp & (gpt - 1);
    const int64_t step = (int64_t)gridDim.x * tpb;
    for (int64_t base = (int64_t)blockIdx.x * tpb; base < p.num_tokens; base += step * UNR) {
        const int64_t t0 = base + grp / gpt;
        int64_t slot[UNR];
#pragma unroll
        for (int k = 0; k < UNR; ++k) {
            const int64_t t = t0 + k * step;
            slot[k] = t < p.num_tokens ? __ldg(p.slot_mapping + t) : -1;
        }
        // every lane of the CTA makes the same rounds (shuffles inside)
        for (int rr = 0; rr < 2 * H; rr += gpt) {
            const int r = rr + r0;
            const bool is_v = r >= H;
            const int g = is_v ? r - H : r;
            Row16<T> x[UNR];
#pragma unroll
            for (int k = 0; k < UNR; ++k) {
                const int64_t t = t0 + k * step;
                x[k].zero();
                if (active && r < 2 * H && t < p.num_tokens)
                    x[k].load((is_v ? static_cast<const T *>(p.value) + t * p.value_stride
                                    : static_cast<const T *>(p.key) + t * p.key_stride) +
                              g * D + sub * 16);
            }
#pragma unroll
            for (int k = 0; k < UNR; ++k) {
                uint32_t amax = x[k].amax();
#pragma unroll
                for (int off = LPR / 2; off > 0; off >>= 1)
                    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, off));
                if (slot[k] < 0 || r >= 2 * H) continue;
                if (slot[k] >= p.pool.capacity) {
                    if (sub == 0 && r == 0) flag_error(p.dev_error, PKV_DEVERR_SLOT);
                    continue;
                }
                const uint32_t byte = scale_byte(amax);
                const float inv = scale_inverse(byte);
                const PoolSlot s = pool_slot(p.pool, (uint32_t)slot[k]);
                if (active) {
                    uint32_t c[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float v[4] = {x[k].at(4 * i), x[k].at(4 * i + 1),
                                            x[k].at(4 * i + 2), x[k].at(4 * i + 3)};
                        c[i] = quant4(v, inv, byte == kScaleNaN);
                    }
                    uint8_t *dst = static_cast<uint8_t *>(is_v ? p.pool.v : p.pool.k) + s.row +
                                   (int64_t)g * s.row_step;
                    *reinterpret_cast<uint4 *>(dst + sub * 16) = make_uint4(c[0], c[1], c[2], c[3]);
                }
                if (sub == 0)
                    (is_v ? p.pool.v_scale : p.pool.k_scale)[s.scale + g * p.pool.block_size] =
                        (uint8_t)byte;
            }
        }
    }
}

template <typename T, int LPR>
cudaError_t launch_write_lpr(const QuantWriteParams &p, cudaStream_t stream) {
    constexpr int kGroups = kThreads / LPR;
    constexpr int UNR = sizeof(T) == 2 ? 2 : 1;
    int gpt = 1;
    while (gpt * 2 <= kGroups && gpt < 2 * p.pool.num_kv_heads) gpt *= 2;
    const int64_t tpb = kGroups / gpt;
    int64_t blocks = (p.num_tokens + tpb - 1) / tpb;
    if (blocks > (int64_t)device_sm_count() * 8)  // enough to fill the SMs: UNR tokens each
        blocks = (blocks + UNR - 1) / UNR;
    if (blocks > (int64_t)1 << 30) blocks = (int64_t)1 << 30;
    return launch_pdl(quant_write_kernel<T, LPR, UNR>, dim3((unsigned)blocks), dim3(kThreads), 0,
                      stream, p, gpt);
}

template <typename T>
cudaError_t launch_write(const QuantWriteParams &p, cudaStream_t stream) {
    const int D = p.pool.head_dim;
    if (D <= 64) return launch_write_lpr<T, 4>(p, stream);
    if (D <= 128) return launch_write_lpr<T, 8>(p, stream);
    return launch_write_lpr<T, 16>(p, stream);
}

// ---------------------------------------------------------------------------
// read-back
// ---------------------------------------------------------------------------
// A CTA takes `rows` consecutive output rows: its first threads find each
// row's request (binary search in cu_k) and slot, then all threads stream the
// (row, K or V, head, 16-code vector) space, several vectors in flight.  66K rows
// of 8 heads of 128 (GB300): 67 us, 92 % of a copy's rate; a call of 300 rows
// takes 2.8 us, launch and one chain of loads.
constexpr int kMaxGatherRows = 64;
constexpr int kGatherUnroll = 4;

__global__ void __launch_bounds__(kThreads)
gather_kernel(const GatherParams p, int rows) {
    __shared__ int32_t s_slot[kMaxGatherRows];
    pdl_trigger();
    pdl_wait();
    const int row0 = blockIdx.x * rows;
    if (blockIdx.x == 0) {  // the offsets themselves: non-decreasing, inside the output
        for (int i = threadIdx.x; i <= p.batch; i += kThreads) {
            const int a = p.cu_k[i];
            if (a < 0 || a > p.total_k || (i > 0 && a < p.cu_k[i - 1]))
                flag_error(p.dev_error, PKV_DEVERR_SEQLEN);
        }
    }
    for (int i = threadIdx.x; i < rows; i += kThreads) {
        const int row = row0 + i;
        int slot = -1;
        if (row < p.total_k) {
            int lo = 0, hi = p.batch;  // the last request whose first row is <= row
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (p.cu_k[mid] <= row)
                    lo = mid;
                else
                    hi = mid;
            }
            const int first = p.cu_k[lo];
            if (first >= 0 && first <= row && row < p.cu_k[lo + 1]) {
                const int pos = row - first, page = pos >> p.pool.bs_shift;
                if (page >= p.max_blocks_per_seq) {
                    flag_error(p.dev_error, PKV_DEVERR_SEQLEN);
                } else {
                    const int blk = p.block_table[(int64_t)lo * p.max_blocks_per_seq + page];
                    if (blk < 0 || blk >= p.num_blocks)
                        flag_error(p.dev_error, PKV_DEVERR_BLOCK_ID);
                    else
                        slot = (blk << p.pool.bs_shift) + (pos & (p.pool.block_size - 1));
                }
            }
        }
        s_slot[i] = slot;
    }
    __syncthreads();
    const int H = p.pool.num_kv_heads, D = p.pool.head_dim, V = D / 16;
    const int HV = H * V, per_row = 2 * HV;
    // this thread's first (row, vector), and the step of kThreads vectors
    const int step_r = kThreads / per_row, step_c = kThreads - step_r * per_row;
    int r = threadIdx.x / per_row, c = threadIdx.x - r * per_row;
    const uint32_t inv_v = 65536 / V + 1;  // x / V = x * inv_v >> 16 for x < 2^12 (V <= 16)
    while (r < rows) {
        uint4 code[kGatherUnroll];
        uint32_t byte[kGatherUnroll];
        __nv_bfloat16 *dst[kGatherUnroll];
#pragma unroll
        for (int u = 0; u < kGatherUnroll; ++u) {
            dst[u] = nullptr;
            const int slot = r < rows ? s_slot[r] : -1;
            if (slot >= 0) {  // else: no such row, or a bad page: left as it was
                const bool is_v = c >= HV;
                const int cc = is_v ? c - HV : c;
                const int g = HV < 4096 ? (int)(((uint32_t)cc * inv_v) >> 16) : cc / V;
                const int v = cc - g * V;
                const PoolSlot s = pool_slot(p.pool, (uint32_t)slot);
                code[u] = __ldg(reinterpret_cast<const uint4 *>(
                                    static_cast<const uint8_t *>(is_v ? p.pool.v : p.pool.k) +
                                    s.row + (int64_t)g * s.row_step) +
                                v);
                byte[u] = __ldg((is_v ? p.pool.v_scale : p.pool.k_scale) + s.scale +
                                g * p.pool.block_size);
                dst[u] = static_cast<__nv_bfloat16 *>(is_v ? p.value : p.key) +
                         ((int64_t)(row0 + r) * H + g) * D + v * 16;
            }
            r += step_r;
            c += step_c;
            if (c >= per_row) {
                c -= per_row;
                ++r;
            }
        }
#pragma unroll
        for (int u = 0; u < kGatherUnroll; ++u) {
            if (!dst[u]) continue;
            uint32_t x[8];
            dequant16_bf16(code[u], byte[u], x);
            uint4 *d = reinterpret_cast<uint4 *>(dst[u]);
            d[0] = make_uint4(x[0], x[1], x[2], x[3]);
            d[1] = make_uint4(x[4], x[5], x[6], x[7]);
        }
    }
}

}  // namespace

cudaError_t launch_quant_write(const QuantWriteParams &p, int dtype, cudaStream_t stream) {
    if (p.num_tokens == 0) return cudaSuccess;
    return dtype == PKV_F32 ? launch_write<float>(p, stream)
                            : launch_write<__nv_bfloat16>(p, stream);
}

cudaError_t launch_gather(const GatherParams &p, cudaStream_t stream) {
    if (p.total_k == 0 || p.batch == 0) return cudaSuccess;
    // rows per CTA: two rounds of the unrolled loop, fewer while that leaves
    // SMs idle
    const int per_row = 2 * p.pool.num_kv_heads * (p.pool.head_dim / 16);
    int rows = (2 * kGatherUnroll * kThreads + per_row - 1) / per_row;
    if (rows > kMaxGatherRows) rows = kMaxGatherRows;
    const int fill = (p.total_k + 2 * device_sm_count() - 1) / (2 * device_sm_count());
    if (rows > fill) rows = fill;
    if (rows < 1) rows = 1;
    return launch_pdl(gather_kernel, dim3((unsigned)((p.total_k + rows - 1) / rows)),
                      dim3(kThreads), 0, stream, p, rows);
}

}  // namespace pkv
