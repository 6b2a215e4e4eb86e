// quant.cuh -- the 8-bit cache's format: e4m3 codes and the byte of a block's power of two; and
// what the tensor cores take of it.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "tc.cuh"

namespace ddt {

// 2^(byte - 127); 0 for byte 0
__device__ __forceinline__ float scale_of(int byte) { return __int_as_float(byte << 23); }

// the byte of the smallest e in [-100, 120] with m <= 448 * 2^e (448 = 1.75 * 2^8); 0 for m = 0
__device__ __forceinline__ int scale_byte(float m) {
    const int bits = __float_as_int(m), e = (bits >> 23) - 135 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
    return m > 0.f ? min(max(e, -100), 120) + 127 : 0;
}

// two codes, `lo` in the low byte: to nearest, ties to even, past 448 to 448, NaN to NaN
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// two codes' values (every e4m3 value is an fp16 value)
__device__ __forceinline__ float2 e4m3_values(uint32_t codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ void values8(uint2 c, float* v) {
    const uint32_t w[4] = {c.x & 0xffffu, c.x >> 16, c.y & 0xffffu, c.y >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = e4m3_values(w[i]);
        v[2 * i] = x.x;
        v[2 * i + 1] = x.y;
    }
}

// four codes in a word, and their values as fp16
__device__ __forceinline__ uint32_t e4m3x4(float x0, float x1, float x2, float x3) {
    uint32_t r;
    asm("{\n .reg .b16 a, b;\n cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n mov.b32 %0, {a, b};\n}"
        : "=r"(r)
        : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x4(__half2 x, __half2 y) {
    uint32_t r;
    asm("{\n .reg .b16 a, b;\n cvt.rn.satfinite.e4m3x2.f16x2 a, %1;\n cvt.rn.satfinite.e4m3x2.f16x2 b, %2;\n mov.b32 %0, {a, b};\n}"
        : "=r"(r)
        : "r"(*reinterpret_cast<const uint32_t*>(&x)), "r"(*reinterpret_cast<const uint32_t*>(&y)));
    return r;
}
__device__ __forceinline__ void e4m3x4_values(uint32_t c, __half2& x, __half2& y) {
    uint32_t a, b;
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}" : "=r"(a), "=r"(b) : "r"(c));
    x = *reinterpret_cast<const __half2*>(&a);
    y = *reinterpret_cast<const __half2*>(&b);
}

// Two fp32 in a 64-bit register: one instruction for both.
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float x, float y) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 f2_get(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator-(F2 a, F2 b) {
    F2 r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

namespace tc {

// Matrix descriptor as desc_sw128, for swizzled rows of 128, 64 or 32 bytes (modes 2, 4 and 6).
__device__ __forceinline__ uint64_t desc_sw(int row_bytes, uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    const uint64_t mode = row_bytes == 128 ? 2 : (row_bytes == 64 ? 4 : 6);
    return (desc_sw128(saddr, lbo, sbo) & ~(static_cast<uint64_t>(7) << 61)) | mode << 61;
}
// The byte of a tile of such rows that holds its byte `off`: bits 7.. of an address turn over bits 4..
template <int ROW_BYTES>
__device__ __forceinline__ uint32_t swizzled(uint32_t off) {
    return off ^ (off >> 3 & (ROW_BYTES - 1u) & 0x70u);
}
// kind::f8f6f4 with e4m3 A and B (format 0) and an fp32 accumulator; an MMA takes 32 bytes of K
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool a_mn, bool b_mn) { return idesc_f16(M, N, a_mn, b_mn); }
// D[tmem] (+)= A[smem desc] * B[smem desc]  (kind::f8f6f4, one CTA)
__device__ __forceinline__ void mma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

}  // namespace tc
}  // namespace ddt
