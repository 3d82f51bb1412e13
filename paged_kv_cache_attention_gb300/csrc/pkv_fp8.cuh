// pkv_fp8.cuh -- device helpers of the 8-bit cache.
//
// A cached row (one token, one kv head) is D e4m3 codes and one E8M0 byte b:
// value_i = code_i * 2^(b - 127).  The scale is a power of two, so
//   * the value has e4m3's 4 significant bits and is exact in bf16,
//   * writing rounds once (x * 2^-e is exact in fp32), and
//   * the attention kernels can move the scale into exponents.
// e4m3's relative step does not depend on the scale: rounding max|x| / 448 up
// to a power of two costs nothing but up to one binade of the smallest
// (subnormal) codes.
#pragma once

#include "pkv_device.cuh"
#include "pkv_fp8.h"

namespace pkv {

constexpr uint32_t kScaleNaN = 255u;  // a row that holds a NaN or an infinity

// E8M0 byte of a row whose largest magnitude has the fp32 bits `amax` (sign
// cleared): e = ceil(log2(amax / 448)), clamped to [-126, 119].  amax =
// m * 2^x with 1 <= m < 2 and 448 = 1.75 * 2^8, so e = x - 8 when m <= 1.75
// and x - 7 above: the carry of adding 2^21 - 1 to the bits decides.  119:
// 448 * 2^119 is the largest code value that a float holds.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    if (amax >= 0x7f800000u) return kScaleNaN;
    const int e = (int)((amax + 0x1fffffu) >> 23) - 135;
    return (uint32_t)(min(max(e, -126), 119) + 127);
}

// 2^-(byte - 127) as a float, for bytes written by scale_byte.
__device__ __forceinline__ float scale_inverse(uint32_t byte) {
    return byte == kScaleNaN ? 0.f : __uint_as_float((254u - byte) << 23);
}

// 2^(byte - 127); 255 is NaN.  (2^-127, byte 0, is a subnormal float.)
__device__ __forceinline__ float scale_value(uint32_t byte) {
    if (byte == kScaleNaN) return __uint_as_float(0x7fffffffu);
    return byte == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The larger of two bf16 pairs, NaN if either is (as 0x7fff).
__device__ __forceinline__ uint32_t bf16x2_max_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Two floats -> two e4m3 codes, nearest even, saturating at 448; lo in the low byte.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Four codes from four floats times `inv` (a row of scale byte 255 stores 0).
__device__ __forceinline__ uint32_t quant4(const float *x, float inv, bool bad) {
    const uint64_t f = f2_pack(inv, inv);
    float a, b, c, d;
    f2_unpack(f2_mul(f2_pack(x[0], x[1]), f), a, b);
    f2_unpack(f2_mul(f2_pack(x[2], x[3]), f), c, d);
    const uint32_t r = cvt_e4m3x2(a, b) | (cvt_e4m3x2(c, d) << 16);
    return bad ? 0u : r;
}

// Four e4m3 codes of a word as f16 pairs: bytes 0 and 1 in lo, 2 and 3 in hi
// (exact; the NaN codes give NaN).
__device__ __forceinline__ void e4m3_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// 16-byte asynchronous copies, completing on an mbarrier.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// The same, or 16 zeros (src is then not read).
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, bool copy) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(copy ? 16 : 0)
                 : "memory");
}

// One lane of a converged warp, always the same.  The compiler knows that only one
// thread goes on, and keeps descriptors and coordinates in uniform registers: a
// group of 8 products takes 160 cycles to issue, against 460 under lane == 0.
__device__ __forceinline__ bool elect_one() {
    uint32_t on;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(on)
        :
        : "memory");
    return on != 0;
}

__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void st_shared_zero16(uint32_t addr) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0) : "memory");
}

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1,
                                              uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
        "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Product of two f16 pairs.
__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Two fp32 -> packed f16x2 (nearest even); lo in the low half.
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 16 e4m3 codes (one 16-byte vector) times 2^(byte-127) as 16 bf16: exact.
// A code's fields moved to the top of bf16's low exponent bits are
// code * 2^-120; the two factors bring 2^120 and the scale.  One product with
// 2^(120 + e) would leave bf16's range for e > 7, so the exponent is split.
__device__ __forceinline__ void dequant16_bf16(const uint4 &c, uint32_t byte, uint32_t (&r)[8]) {
    const int e = (int)byte - 127;
    // 2^(120 + e1) * 2^e2, e1 + e2 = e, both factors normal
    const int e1 = min(e, 0) > -120 ? min(e, 0) : -120, e2 = e - e1;
    const uint32_t f1 = (uint32_t)(e1 + 120 + 127) << 7;
    const uint32_t f2 = byte == kScaleNaN ? 0x7fffu : (uint32_t)(e2 + 127) << 7;
    __nv_bfloat162 m1, m2;
    *reinterpret_cast<uint32_t *>(&m1) = f1 | (f1 << 16);
    *reinterpret_cast<uint32_t *>(&m2) = f2 | (f2 << 16);
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // bytes (0, 1) and (2, 3) side by side, each in the top byte of a half
        const uint32_t p0 = __byte_perm(w[i], 0u, 0x1404), p1 = __byte_perm(w[i], 0u, 0x3424);
        const uint32_t h0 = (p0 & 0x80008000u) | ((p0 >> 4) & 0x07f007f0u);
        const uint32_t h1 = (p1 & 0x80008000u) | ((p1 >> 4) & 0x07f007f0u);
        __nv_bfloat162 a0, a1;
        *reinterpret_cast<uint32_t *>(&a0) = h0;
        *reinterpret_cast<uint32_t *>(&a1) = h1;
        a0 = __hmul2(a0, m1);
        a1 = __hmul2(a1, m1);
        if (e2 != 0) {  // rare: values above 448, or below 2^-120
            a0 = __hmul2(a0, m2);
            a1 = __hmul2(a1, m2);
        }
        r[2 * i] = *reinterpret_cast<uint32_t *>(&a0);
        r[2 * i + 1] = *reinterpret_cast<uint32_t *>(&a1);
    }
}

// Where a slot's rows are in a pool: kv head g's row starts at element row +
// g * row_step, its E8M0 byte is scale + g * block_size.  slot is in [0,
// capacity), which is below 2^31.
struct PoolSlot {
    int64_t row, scale;
    int row_step;
};

__device__ __forceinline__ PoolSlot pool_slot(const PoolArgs &p, uint32_t slot) {
    const uint32_t blk = slot >> p.bs_shift, off = slot & (p.block_size - 1);
    PoolSlot s;
    s.scale = (int64_t)blk * (p.num_kv_heads * p.block_size) + off;
    s.row = (p.hnd ? s.scale : (int64_t)slot * p.num_kv_heads) * p.head_dim;
    s.row_step = p.hnd ? p.block_size * p.head_dim : p.head_dim;
    return s;
}

}  // namespace pkv
