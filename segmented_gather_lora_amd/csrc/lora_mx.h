// lora_mx.h -- microscaled 4-bit numbers: sizes and conversions shared by the kernels
// that read or write them.  A row is blocks of 32 numbers: 16 bytes of E2M1 codes (two a
// byte, the first in the low half) and one byte, the exponent of their common power
// of two plus 127.
#pragma once

#include "lora_gemm.h"

namespace lora {

constexpr int kMxBlock = 32;
inline int64_t mx_blocks(int64_t cols) { return (cols + kMxBlock - 1) / kMxBlock; }
inline int64_t mx_code_bytes(int64_t cols) { return 16 * mx_blocks(cols); }
inline int64_t mx_scale_bytes(int64_t cols) { return (mx_blocks(cols) + 3) / 4 * 4; }

// The scale byte (the power's exponent plus 127) of a block whose largest magnitude
// has these bits: floor(log2) - 2, 2 being E2M1's largest exponent; 255 (not a
// number) for a block that is not finite.
__device__ __forceinline__ int mx_scale_of(uint32_t top) {
    const int e = (int)(top >> 23);
    return e == 255 ? 255 : e > 2 ? e - 2 : 0;
}
// 8 codes: v over the power (exact, but for what is far below half of the smallest
// code), to the nearest, ties to even, held at 6.
__device__ __forceinline__ uint32_t mx_codes_of(const float v[8], int scale) {
    if (scale == 255) return 0u;
    const float inv = __uint_as_float((uint32_t)(254 - scale) << 23);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0] * inv, v[1] * inv, 1.f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2] * inv, v[3] * inv, 1.f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4] * inv, v[5] * inv, 1.f, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6] * inv, v[7] * inv, 1.f, 3);
    return c;
}

// A block of 32 bf16 numbers in one lane: its codes, and its scale byte.
__device__ __forceinline__ int mx_block_codes(const u32x4 (&x)[4], u32x4 &codes) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(max(top, x[j][e] << 16 & 0x7fff0000u), x[j][e] & 0x7fff0000u);
    const int scale = mx_scale_of(top);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) unpack_bf16(x[j][e], v[2 * e], v[2 * e + 1]);
        codes[j] = mx_codes_of(v, scale);
    }
    return scale;
}
// 8 codes (a dword) times their power as bf16, exact.  The conversion reads the
// exponent alone: 0 gives 2^-127, 255 NaN.
__device__ __forceinline__ u32x4 mx_numbers(uint32_t codes, uint32_t scale) {
    const float s = __uint_as_float(scale << 23);
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 0)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 1)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 2)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 3))};
}

}  // namespace lora
