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
// code vectors, the maximum in two to four shuffles, no shared memory.
#include "pkv_fp8.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;

// 16 values of a head row as floats.
template <typename T>
__device__ __forceinline__ void load16(const T *p, float (&x)[16]);

template <>
__device__ __forceinline__ void load16<__nv_bfloat16>(const __nv_bfloat16 *p, float (&x)[16]) {
    const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p));
    const uint4 b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

template <>
__device__ __forceinline__ void load16<float>(const float *p, float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(p) + i);
        x[4 * i] = v.x;
        x[4 * i + 1] = v.y;
        x[4 * i + 2] = v.z;
        x[4 * i + 3] = v.w;
    }
}

// A unit is (token, K or V, kv head), heads fastest; LPR lanes take one unit,
// UNR units apart by one grid.
template <typename T, int LPR, int UNR>
__global__ void __launch_bounds__(kThreads)
quant_write_kernel(const QuantWriteParams p) {
    pdl_trigger();
    pdl_wait();
    const int sub = threadIdx.x % LPR;
    const int H = p.pool.num_kv_heads, D = p.pool.head_dim;
    const bool active = sub * 16 < D;
    const int64_t units = p.num_tokens * 2 * H;
    const int64_t stride = (int64_t)gridDim.x * (kThreads / LPR);
    const int64_t u0 = (int64_t)blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR;
    // every lane of a warp makes the same number of rounds (shuffles inside)
    const int64_t first = (int64_t)blockIdx.x * (kThreads / LPR) + (threadIdx.x & ~31) / LPR;
    for (int64_t base = 0; first + base < units; base += stride * UNR) {
        float x[UNR][16];
        int64_t slot[UNR];
        int head[UNR];
        bool is_v[UNR];
#pragma unroll
        for (int k = 0; k < UNR; ++k) {
            const int64_t u = u0 + base + k * stride;
            slot[k] = -1;
            head[k] = 0;
            is_v[k] = false;
#pragma unroll
            for (int i = 0; i < 16; ++i) x[k][i] = 0.f;
            if (u >= units) continue;
            const int64_t t = u / (2 * H);
            const int r = (int)(u - t * (2 * H));
            is_v[k] = r >= H;
            head[k] = is_v[k] ? r - H : r;
            slot[k] = __ldg(p.slot_mapping + t);
            if (active) {
                const T *src = is_v[k] ? static_cast<const T *>(p.value) + t * p.value_stride
                                       : static_cast<const T *>(p.key) + t * p.key_stride;
                load16<T>(src + head[k] * D + sub * 16, x[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < UNR; ++k) {
            uint32_t amax = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                amax = max(amax, __float_as_uint(x[k][i]) & 0x7fffffffu);
#pragma unroll
            for (int off = LPR / 2; off > 0; off >>= 1)
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, off));
            if (slot[k] < 0) continue;
            if (slot[k] >= p.pool.capacity) {
                if (sub == 0) flag_error(p.dev_error, PKV_DEVERR_SLOT);
                continue;
            }
            const uint32_t byte = scale_byte(amax);
            const float inv = scale_inverse(byte);
            const bool bad = byte == kScaleNaN;
            const PoolSlot s = pool_slot(p.pool, slot[k], head[k]);
            if (active) {
                const uint4 c = make_uint4(quant4(x[k], inv, bad), quant4(x[k] + 4, inv, bad),
                                           quant4(x[k] + 8, inv, bad),
                                           quant4(x[k] + 12, inv, bad));
                uint8_t *dst = static_cast<uint8_t *>(is_v[k] ? p.pool.v : p.pool.k) + s.row;
                *reinterpret_cast<uint4 *>(dst + sub * 16) = c;
            }
            if (sub == 0) (is_v[k] ? p.pool.v_scale : p.pool.k_scale)[s.scale] = (uint8_t)byte;
        }
    }
}

template <typename T, int LPR>
cudaError_t launch_write_lpr(const QuantWriteParams &p, cudaStream_t stream) {
    const int64_t units = p.num_tokens * 2 * p.pool.num_kv_heads;
    constexpr int kUnits = kThreads / LPR;
    constexpr int UNR = sizeof(T) == 2 ? 2 : 1;
    const int64_t cap = (int64_t)device_sm_count() * 64;
    int64_t blocks = (units + kUnits - 1) / kUnits;
    if (blocks > (int64_t)device_sm_count() * 8)  // enough to fill the SMs: several units each
        blocks = (blocks + UNR - 1) / UNR;
    if (blocks > cap) blocks = cap;
    return launch_pdl(quant_write_kernel<T, LPR, UNR>, dim3((unsigned)blocks), dim3(kThreads), 0,
                      stream, p);
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
// (row, K or V, head, 16-code vector) space.
constexpr int kMaxGatherRows = 64;

__global__ void __launch_bounds__(kThreads)
gather_kernel(const GatherParams p, int rows) {
    __shared__ int64_t s_slot[kMaxGatherRows];
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
        int64_t slot = -1;
        if (row < p.total_k) {
            int lo = 0, hi = p.batch;  // the last request whose first row is <= row
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (p.cu_k[mid] <= row)
                    lo = mid;
                else
                    hi = mid;
            }
            const int64_t first = p.cu_k[lo];
            if (first >= 0 && first <= row && row < p.cu_k[lo + 1]) {
                const int64_t pos = row - first;
                const int64_t page = pos / p.pool.block_size;
                if (page >= p.max_blocks_per_seq) {
                    flag_error(p.dev_error, PKV_DEVERR_SEQLEN);
                } else {
                    const int blk = p.block_table[(int64_t)lo * p.max_blocks_per_seq + page];
                    if (blk < 0 || blk >= p.num_blocks)
                        flag_error(p.dev_error, PKV_DEVERR_BLOCK_ID);
                    else
                        slot = (int64_t)blk * p.pool.block_size + pos % p.pool.block_size;
                }
            }
        }
        s_slot[i] = slot;
    }
    __syncthreads();
    const int H = p.pool.num_kv_heads, D = p.pool.head_dim, V = D / 16;
    const int per_row = 2 * H * V;
    const int total = rows * per_row;
    for (int i = threadIdx.x; i < total; i += kThreads) {
        const int r = i / per_row;
        int c = i - r * per_row;
        const int64_t slot = s_slot[r];
        if (slot < 0) continue;  // no such row, or a bad page: left as it was
        const bool is_v = c >= H * V;
        if (is_v) c -= H * V;
        const int g = c / V, v = c - g * V;
        const PoolSlot s = pool_slot(p.pool, slot, g);
        const uint8_t *src = static_cast<const uint8_t *>(is_v ? p.pool.v : p.pool.k) + s.row;
        const uint4 code = __ldg(reinterpret_cast<const uint4 *>(src) + v);
        const uint32_t byte = __ldg((is_v ? p.pool.v_scale : p.pool.k_scale) + s.scale);
        uint32_t x[8];
        dequant16_bf16(code, byte, x);
        uint4 *dst = reinterpret_cast<uint4 *>(
            static_cast<__nv_bfloat16 *>(is_v ? p.value : p.key) +
            ((int64_t)(row0 + r) * H + g) * D + v * 16);
        dst[0] = make_uint4(x[0], x[1], x[2], x[3]);
        dst[1] = make_uint4(x[4], x[5], x[6], x[7]);
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
    // rows per CTA: about four vectors per thread, fewer while that leaves SMs idle
    const int per_row = 2 * p.pool.num_kv_heads * (p.pool.head_dim / 16);
    int rows = (4 * kThreads + per_row - 1) / per_row;
    if (rows > kMaxGatherRows) rows = kMaxGatherRows;
    const int fill = (p.total_k + 2 * device_sm_count() - 1) / (2 * device_sm_count());
    if (rows > fill) rows = fill;
    if (rows < 1) rows = 1;
    return launch_pdl(gather_kernel, dim3((unsigned)((p.total_k + rows - 1) / rows)),
                      dim3(kThreads), 0, stream, p, rows);
}

}  // namespace pkv
