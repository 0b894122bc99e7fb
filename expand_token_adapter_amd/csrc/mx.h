// mx.h -- the microscaled 4-bit form of rows and weights (gfx950).
//
// value = code * 2^(scale - 127): e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
// negatives), two a byte, and one exponent byte for each 32 columns of a row.  The
// scale of a block is the smallest power of two, 2^-127 at the least, that brings
// its largest magnitude to 6, the largest e2m1 value, or less.
//
// Why 6 and not a rule on the exponent alone (the largest magnitude's exponent
// minus 2): with that one, magnitudes from 6 to 8 times the scale would be cut to
// 6, up to a quarter of the largest value lost; here the largest is off by at most
// a fifth (5 is stored as 4), for one binade less at the small end of such blocks.  A
// power of two, because the matrix instruction takes exponent bytes for exactly such
// blocks (a lane's 32 codes of one row), so they cost a product no arithmetic.
//
// There is no 4-bit NaN: a block with a value that is not finite has the scale
// byte 255, and all of its values are NaN.
#pragma once

#include "device_common.h"
#include "host_checks.h"
#include "quant.h"

namespace lora {

constexpr int kMxBlock = LORA_MX_BLOCK;  // columns of a scale
constexpr int kMxPad = LORA_MX_PAD;      // rows are stored in whole multiples of this many columns
constexpr uint32_t kMxNan = 255;

// Exponent byte of a block whose largest finite magnitude has the fp32 bits
// `top` (127 for a block of zeros).  6 = 1.5 * 2^2: for a magnitude m * 2^E the
// exponent is E - 2 where m <= 1.5, else E - 1.  (A subnormal's E is below 2^-126,
// its byte 0.)
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
    const int e = (int)(top >> 23) - 2 + ((top & 0x7fffffu) > 0x400000u ? 1 : 0);
    return top == 0u ? 127u : (uint32_t)max(e, 0);
}

// 8 codes (a word) times a scale (exact in bf16 and fp32; magnitudes from 2^128 up,
// scale bytes 253 and 254, are infinite; checked for every code and byte).
template <int DT>
__device__ __forceinline__ Frag<DT> mx_decode8(uint32_t w, float s);
template <>
__device__ __forceinline__ Frag<LORA_BF16> mx_decode8<LORA_BF16>(uint32_t w, float s) {
    return Frag<LORA_BF16>{u32x4_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0)),
                                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1)),
                                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2)),
                                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3))}};
}
template <>
__device__ __forceinline__ Frag<LORA_F32> mx_decode8<LORA_F32>(uint32_t w, float s) {
    return Frag<LORA_F32>{
        __builtin_bit_cast(u32x4_t, __builtin_shufflevector(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0),
                                                            __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1), 0, 1, 2, 3)),
        __builtin_bit_cast(u32x4_t, __builtin_shufflevector(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2),
                                                            __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3), 0, 1, 2, 3))};
}

// Codes of 8 values with |value| <= 6 * 2^(scale - 127), the first in the low bits
// (rounded to nearest even, checked for every bf16 number and 4.8e7 pairs of
// values and scales).
__device__ __forceinline__ uint32_t mx_encode8(const Frag<LORA_BF16>& f, float s) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    const uint32_t a = f.q[0], b = f.q[1], c = f.q[2], d = f.q[3];  // (a bit cast of a vector's element takes its first)
    uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(0u, __builtin_bit_cast(bf16x2_t, a), s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, b), s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, c), s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, d), s, 3);
}
__device__ __forceinline__ uint32_t mx_encode8(const Frag<LORA_F32>& f, float s) {
    uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, f.get(0), f.get(1), s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f.get(2), f.get(3), s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f.get(4), f.get(5), s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f.get(6), f.get(7), s, 3);
}

// ------------------------------------------------------------------ host checks

// One 4-bit matrix argument with rows of `cols` values.
inline int check_mx(const lora_quant& q, int64_t cols) {
    if (!q.codes || !q.scales || !aligned16(q.codes) || ((uintptr_t)q.scales & 7u)) return LORA_ERR_INVALID_ARG;
    const int64_t full = round_up(cols, kMxPad);
    if (cols < 1 || q.ld < full / 2 || q.lds < full / kMxBlock) return LORA_ERR_INVALID_ARG;
    if (cols % 8 != 0 || q.ld % (kMxPad / 2) != 0 || q.lds % (kMxPad / kMxBlock) != 0) return LORA_ERR_UNSUPPORTED;
    return LORA_OK;
}

}  // namespace lora
