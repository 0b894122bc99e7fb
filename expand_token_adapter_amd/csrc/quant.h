// quant.h -- the 8-bit form of rows and weights (gfx950).
//
// value = code * 2^(scale - 127): e4m3 codes and one exponent byte for each
// block of 128 (rows: 1 x 128 elements; weights: 128 x 128).  The scale of a
// block is the smallest power of two, 2^-127 at the least, that brings its
// largest finite magnitude to 448, the largest e4m3 value, or less.
//
// Why a power of two and not amax / 448: dividing by it is exact, so a code is
// a plain rounding of x (to 4 significant bits, as with any other scale), x's
// restored value has 4 significant bits and is a bf16 number, and the matrix
// instruction applies it (v_mfma_scale_f32_16x16x128_f8f6f4 takes exponent
// bytes), so a product needs no vector work per block.  The price is at most
// one binade of the codes' range, at its small end.
#pragma once

#include "device_common.h"
#include "host_checks.h"

namespace lora {

constexpr int kQBlock = LORA_QUANT_BLOCK;

// ------------------------------------------------------------------ scales

// Exponent byte of a block whose largest finite magnitude has the fp32 bits
// `top` (127 for a block of zeros).  448 = 1.75 * 2^8: for a magnitude
// m * 2^E the exponent is E - 8 where m <= 1.75, else E - 7.
__device__ __forceinline__ uint32_t quant_scale_byte(uint32_t top) {
    const int e = (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    return top == 0u ? 127u : (uint32_t)max(e, 0);
}
// The scale operand of gfx950's v_cvt_scalef32_* conversions: they take the
// exponent field alone, so field 0 is 2^-127 and 255 is NaN, as the bytes are
// (checked for every byte and code).
__device__ __forceinline__ float quant_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// ------------------------------------------------------------------ codes

// 8 codes times a scale, as an operand fragment (bf16: exact for scale bytes
// from 3 to 246, else rounded to nearest even).
template <int DT>
__device__ __forceinline__ Frag<DT> dequant8(uint32_t w0, uint32_t w1, float s);
template <>
__device__ __forceinline__ Frag<LORA_BF16> dequant8<LORA_BF16>(uint32_t w0, uint32_t w1, float s) {
    return Frag<LORA_BF16>{
        u32x4_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w0, s, false)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w0, s, true)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w1, s, false)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w1, s, true))}};
}
template <>
__device__ __forceinline__ Frag<LORA_F32> dequant8<LORA_F32>(uint32_t w0, uint32_t w1, float s) {
    return Frag<LORA_F32>{
        __builtin_bit_cast(u32x4_t, __builtin_shufflevector(__builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)w0, s, false),
                                                            __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)w0, s, true),
                                                            0, 1, 2, 3)),
        __builtin_bit_cast(u32x4_t, __builtin_shufflevector(__builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)w1, s, false),
                                                            __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)w1, s, true),
                                                            0, 1, 2, 3))};
}
// Write a fragment's 8 values (16-byte aligned).
__device__ __forceinline__ void store_frag(void* p, const Frag<LORA_BF16>& f) {
    *gptr(reinterpret_cast<u32x4_t*>(p)) = f.q;
}
__device__ __forceinline__ void store_frag(void* p, const Frag<LORA_F32>& f) {
    LORA_GLOBAL u32x4_t* d = gptr(reinterpret_cast<u32x4_t*>(p));
    d[0] = f.q0;
    d[1] = f.q1;
}

// ------------------------------------------------------------------ rows in a backward

// 8 codes of one row and their scale byte, as loaded; decoded where they are
// used so that the loads stay in flight.
struct QuantRaw {
    u32x2_t codes;
    uint32_t scale;
    __device__ __forceinline__ static QuantRaw load(const uint8_t* code_row, const uint8_t* scale_row, int col) {
        QuantRaw r;
        const LORA_GLOBAL uint32_t* c = gptr(reinterpret_cast<const uint32_t*>(code_row + col));
        r.codes = u32x2_t{c[0], c[1]};
        r.scale = gptr(scale_row)[col / kQBlock];
        return r;
    }
    template <int DT>
    __device__ __forceinline__ Frag<DT> frag() const {
        return dequant8<DT>(codes[0], codes[1], quant_scale(scale));
    }
};

// ------------------------------------------------------------------ host checks

// One 8-bit matrix argument with rows of `cols` values.
inline int check_quant(const lora_quant& q, int64_t cols) {
    if (!q.codes || !q.scales || !aligned16(q.codes) || ((uintptr_t)q.scales & 3u)) return LORA_ERR_INVALID_ARG;
    if (cols < 1 || q.ld < round_up(cols, kQBlock) || q.lds < (cols + kQBlock - 1) / kQBlock) return LORA_ERR_INVALID_ARG;
    if (cols % 8 != 0 || q.ld % kQBlock != 0 || q.lds % 4 != 0) return LORA_ERR_UNSUPPORTED;
    return LORA_OK;
}

}  // namespace lora
