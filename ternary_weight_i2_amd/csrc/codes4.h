// codes4.h -- 4-bit codes as operands of the fp16 16x16x32 matrix instruction.
#pragma once

#include "common.h"

namespace bitnet {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef uint16_t us2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ us2 as_us2(uint32_t w) { return __builtin_bit_cast(us2, w); }
__device__ __forceinline__ h2 as_h2(uint32_t w) { return __builtin_bit_cast(h2, w); }
__device__ __forceinline__ h8 join(h2 a, h2 b, h2 c, h2 d) {
    return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// 1024 = 0x6400 twice, in a vector register: with the mask in a scalar one a
// nibble then takes its exponent in a single v_and_or_b32.
__device__ __forceinline__ uint32_t ones_1024() {
    uint32_t w;
    asm("v_mov_b32 %0, 0x64006400" : "=v"(w));
    return w;
}
// The eight codes of a word in the order 0 4, 1 5, 2 6, 3 7.  RAW: as fp16
// subnormals code * 2^-24, the second and fourth pair 16 times as large.  Else
// code - 8: a nibble in the low mantissa bits of 1024 makes 1024 + code (or 1024
// + 16 code one place up), and one packed operation the rest, exactly.
template <bool RAW>
__device__ __forceinline__ void codes8(uint32_t w, uint32_t one, h2 (&c)[4]) {
    const uint32_t w8 = w >> 8;
    if constexpr (RAW) {
        c[0] = as_h2(w & 0x000f000fu);
        c[1] = as_h2(w & 0x00f000f0u);
        c[2] = as_h2(w8 & 0x000f000fu);
        c[3] = as_h2(w8 & 0x00f000f0u);
    } else {
        const h2 s = {(_Float16)0.0625f, (_Float16)0.0625f};
        c[0] = as_h2((w & 0x000f000fu) | one) - (_Float16)1032.0f;
        c[1] = as_h2((w & 0x00f000f0u) | one) * s - (_Float16)72.0f;
        c[2] = as_h2((w8 & 0x000f000fu) | one) - (_Float16)1032.0f;
        c[3] = as_h2((w8 & 0x00f000f0u) | one) * s - (_Float16)72.0f;
    }
}
__device__ __forceinline__ f4 mfma(h8 a, h8 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Over the four lanes that hold a row (l, l ^ 16, l ^ 32, l ^ 48): the swaps
// hand every lane its own and its partner's value.
__device__ __forceinline__ void partners16(float v, float &a, float &b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                    false);
    a = __uint_as_float(r[0]);
    b = __uint_as_float(r[1]);
}
__device__ __forceinline__ void partners32(float v, float &a, float &b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                    false);
    a = __uint_as_float(r[0]);
    b = __uint_as_float(r[1]);
}
__device__ __forceinline__ float quad_max(float v) {
    float a, b;
    partners16(v, a, b);
    partners32(fmaxf(a, b), a, b);
    return fmaxf(a, b);
}
__device__ __forceinline__ float quad_sum(float v) {
    float a, b;
    partners16(v, a, b);
    partners32(a + b, a, b);
    return a + b;
}

template <int N>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&w)[N]) {
    static_assert(N == 2 || N == 4 || N == 8, "8, 16 or 32 bytes");
    if constexpr (N == 2) {
        const uint2 a = *reinterpret_cast<const uint2 *>(p);
        w[0] = a.x; w[1] = a.y;
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 a = reinterpret_cast<const uint4 *>(p)[i];
            w[4 * i] = a.x; w[4 * i + 1] = a.y; w[4 * i + 2] = a.z; w[4 * i + 3] = a.w;
        }
    }
}

}  // namespace bitnet
