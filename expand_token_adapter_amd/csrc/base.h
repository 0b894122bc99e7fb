// base.h -- the frozen base product from 8-bit rows and an 8-bit weight (gfx950).
//
//   y_t (+)= sum_k x_tk W_nk
//
// with x and W as codes times power-of-two block scales (quant.h).
//
// bf16 y: one v_mfma_scale_f32_16x16x128_f8f6f4 takes exactly one block of 128
// along k for 16 outputs and 16 rows: its operands are codes as stored, its two
// exponent bytes a lane are the scales of the lane's weight row and activation
// row, and its sums stay in fp32 registers from the first block to the last.
// The instruction cuts each product of a group of 8 (k-consecutive codes of a
// lane) at 2^-13 of the power of two of the group's largest, and adds groups in
// fp32 (measured on the device: products 2^16 and 2^3 in a group give both, 2^16
// and 2^2 only the first; 14 counts as 8 there; in different groups 2^-7 is
// kept).  On normal data that is 1.5e-5 of the result, with outliers in 1% of
// the codes 5e-5: a hundredth of y's rounding to bf16 (1.7e-3), for twice the
// rate of the bf16 instruction.
//
// fp32 y: the codes times their scales are bf16 numbers, and
// v_mfma_f32_16x16x32_bf16 sums their exact products in fp32.
//
// A operand = weight rows (n), B operand = activation rows (t), so a lane ends
// with four consecutive n of one row t.  The order of the 128 products inside
// a block is free (both operands take the same one): lane group g = lane / 16
// takes the 16-byte units g and g + 4 of each 128-byte block row.
#pragma once

#include "quant.h"

namespace lora {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

struct BaseParams {
    const uint8_t* x;
    int64_t ldx;
    const uint8_t* xs;
    int64_t ldxs;
    const uint8_t* w;
    int64_t ldw;
    const uint8_t* ws;
    int64_t ldws;
    char* y;
    int64_t ldy;
    int32_t T, N, nkb;  // rows, outputs, blocks of 128 along k
    int32_t accumulate;
    int32_t tiles_n, tiles_t;
};

// One operand row's block of 128: this lane's 32 codes and the row's scale
// byte (bits 7:0 of scale; the others do not count).
template <int DT>
struct QuantFrag;
template <>
struct QuantFrag<LORA_BF16> {
    i32x8_t codes;
    int scale;
    __device__ __forceinline__ static QuantFrag make(u32x4_t u0, u32x4_t u1, uint32_t scale) {
        return QuantFrag{i32x8_t{(int)u0[0], (int)u0[1], (int)u0[2], (int)u0[3], (int)u1[0], (int)u1[1], (int)u1[2],
                                 (int)u1[3]},
                         (int)scale};
    }
    __device__ __forceinline__ f32x4_t mma(const QuantFrag& b, f32x4_t c) const {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(codes, b.codes, c, 0, 0, 0, scale, 0, b.scale);
    }
};
template <>
struct QuantFrag<LORA_F32> {
    Frag<LORA_BF16> q[4];
    __device__ __forceinline__ static QuantFrag make(u32x4_t u0, u32x4_t u1, uint32_t scale) {
        const float s = quant_scale(scale & 255u);
        return QuantFrag{{dequant8<LORA_BF16>(u0[0], u0[1], s), dequant8<LORA_BF16>(u0[2], u0[3], s),
                          dequant8<LORA_BF16>(u1[0], u1[1], s), dequant8<LORA_BF16>(u1[2], u1[3], s)}};
    }
    __device__ __forceinline__ f32x4_t mma(const QuantFrag& b, f32x4_t c) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) c = lora::mma(q[i], b.q[i], c);
        return c;
    }
};

// Four consecutive outputs of one row: added to what is there (accumulate) in
// fp32, rounded once.
template <int DT>
__device__ __forceinline__ void base_store4(const BaseParams& p, int t, int n, f32x4_t v) {
    if (t >= p.T || n >= p.N) return;  // (N is a multiple of 8: the four are in or out together)
    if constexpr (DT == LORA_BF16) {
        LORA_GLOBAL u32x2_t* d = gptr(reinterpret_cast<u32x2_t*>(p.y + ((int64_t)t * p.ldy + n) * 2));
        if (p.accumulate) {
            const u32x2_t o = *d;
            v += f32x4_t{__uint_as_float(o[0] << 16), __uint_as_float(o[0] & 0xffff0000u), __uint_as_float(o[1] << 16),
                         __uint_as_float(o[1] & 0xffff0000u)};
        }
        *d = u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    } else {
        LORA_GLOBAL f32x4_t* d = gptr(reinterpret_cast<f32x4_t*>(p.y + ((int64_t)t * p.ldy + n) * 4));
        if (p.accumulate) v += *d;
        *d = v;
    }
}

// ------------------------------------------------------------------ tiles through LDS
//
// A workgroup of WN x WT waves computes BN outputs x BT rows.  A step is one
// block of 128 along k: BN + BT block rows of 128 bytes go from memory straight
// into LDS, ST stages in a ring, the loads of step i + ST - 1 issued while step
// i is multiplied.  Unit c (16 bytes) of row r lies at position c ^ (r % 8) of
// the row, so that the 16 rows of an operand read fall on different banks.
// The scales of up to kBaseGroups * 4 blocks lie in LDS too, four blocks' bytes
// of one row in a word; a longer k is taken in pieces.

constexpr int kBaseGroups = 30;

template <int BN, int BT, int ST>
struct BaseLds {
    static constexpr int kStage = (BN + BT) * kQBlock;
    static constexpr int kScales = kBaseGroups * (BT + BN / 16) * 4;
    static constexpr int kBytes = ST * kStage + kScales;
};

template <int BN, int BT, int WN, int WT, int ST, int DT>
__global__ __launch_bounds__(WN* WT* kWave) void base_kernel(BaseParams p) {
    constexpr int NW = WN * WT;
    constexpr int FN = BN / WN / 16, FT = BT / WT / 16;  // 16 x 16 blocks of a wave
    constexpr int UN = BN / 8, UT = BT / 8;              // 1 KB loads of a stage
    constexpr int PW = (UN + UT) / NW;                   // loads of a wave and stage
    constexpr int NB = BN / 16;                          // weight scale words per group, one for each 16 outputs
    static_assert(UN % NW == 0 && UT % NW == 0, "every wave loads the same number of rows");
    using L = BaseLds<BN, BT, ST>;
    __shared__ __attribute__((aligned(16))) char s_lds[L::kBytes];
    uint32_t* s_xs = reinterpret_cast<uint32_t*>(s_lds + ST * L::kStage);  // [group][BT]
    uint32_t* s_ws = s_xs + kBaseGroups * BT;                              // [group][NB]

    const int wave = wave_id();
    const int lane = threadIdx.x & (kWave - 1);
    const int lr = lane & 15, lg = lane >> 4;
    // Workgroups of one XCD take neighbouring tiles.
    const int ntile = p.tiles_n * p.tiles_t;
    const int per = (ntile + kNumXcd - 1) / kNumXcd;
    const int tile = (int)(blockIdx.x % kNumXcd) * per + (int)(blockIdx.x / kNumXcd);
    if ((int)(blockIdx.x / kNumXcd) >= per || tile >= ntile) return;
    const int n0 = (tile % p.tiles_n) * BN, t0 = (tile / p.tiles_n) * BT;
    const int wn = (wave % WN) * (BN / WN), wt = (wave / WN) * (BT / WT);

    // Loads: wave w takes the 8-row units w, w + NW, ...; rows past the matrix
    // repeat its last row (their outputs are not stored).
    const int nrows = min(BN, p.N - n0), trows = min(BT, p.T - t0);
    const buf_rsrc_t rw = make_rsrc(p.w + (int64_t)n0 * p.ldw, (uint32_t)((nrows - 1) * p.ldw + (int64_t)p.nkb * kQBlock));
    const buf_rsrc_t rx = make_rsrc(p.x + (int64_t)t0 * p.ldx, (uint32_t)((trows - 1) * p.ldx + (int64_t)p.nkb * kQBlock));
    uint32_t voff[PW];
#pragma unroll
    for (int j = 0; j < PW; ++j) {
        const int r8 = lane >> 3;
        const int row = 8 * (wave + NW * j) + r8;  // of the stage: BN weight rows, then BT activation rows
        const uint32_t unit = (uint32_t)((lane & 7) ^ r8) * 16u;
        voff[j] = NW * j < UN ? (uint32_t)(min(row, nrows - 1) * p.ldw) + unit
                              : (uint32_t)(min(row - BN, trows - 1) * p.ldx) + unit;
    }
    auto issue = [&](int slot, int kb) {
        char* at = s_lds + slot * L::kStage + wave * 1024;
#pragma unroll
        for (int j = 0; j < PW; ++j)
            dma_lds(NW * j < UN ? rw : rx, voff[j], (uint32_t)kb * kQBlock, at + NW * j * 1024, 16);
    };

    f32x4_t acc[FN][FT];
#pragma unroll
    for (int a = 0; a < FN; ++a)
#pragma unroll
        for (int b = 0; b < FT; ++b) acc[a][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    // This lane's operand bytes of a block row: units lg and lg + 4.
    const int lrow = lr * kQBlock + ((lg ^ (lr & 7)) * 16);

    for (int k0 = 0; k0 < p.nkb; k0 += 4 * kBaseGroups) {
        const int k1 = min(p.nkb, k0 + 4 * kBaseGroups);
        const int ng = (k1 - k0 + 3) / 4;
        if (k0 > 0) {
            wait_vmcnt_le<0>();
            lds_barrier();  // the last piece's stages and scales are no longer read
        }
        for (int i = threadIdx.x; i < ng * BT; i += NW * kWave) {
            const int g = i % ng, t = min(i / ng, trows - 1);
            s_xs[g * BT + i / ng] = *gptr(reinterpret_cast<const uint32_t*>(p.xs + (int64_t)(t0 + t) * p.ldxs + k0 + 4 * g));
        }
        for (int i = threadIdx.x; i < ng * NB; i += NW * kWave) {
            const int g = i / NB, b = i % NB;
            const int nblk = min(n0 + 16 * b, p.N - 1) / kQBlock;
            s_ws[i] = *gptr(reinterpret_cast<const uint32_t*>(p.ws + (int64_t)nblk * p.ldws + k0 + 4 * g));
        }
        // (loads past the piece repeat its last block: every step waits for the same number)
#pragma unroll
        for (int s = 0; s < ST - 1; ++s) issue(s, min(k0 + s, k1 - 1));
        int slot = 0;
        for (int kb = k0; kb < k1; ++kb) {
            wait_vmcnt_le<PW*(ST - 2)>();
            lds_barrier();
            issue(slot == 0 ? ST - 1 : slot - 1, min(kb + ST - 1, k1 - 1));
            const char* sw = s_lds + slot * L::kStage + wn * kQBlock;
            const char* sx = s_lds + slot * L::kStage + (BN + wt) * kQBlock;
            const int g = (kb - k0) >> 2, sh = 8 * ((kb - k0) & 3);
            QuantFrag<DT> b[FT];
#pragma unroll
            for (int f = 0; f < FT; ++f)
                b[f] = QuantFrag<DT>::make(*reinterpret_cast<const u32x4_t*>(sx + f * 16 * kQBlock + lrow),
                                           *reinterpret_cast<const u32x4_t*>(sx + f * 16 * kQBlock + (lrow ^ 64)),
                                           s_xs[g * BT + wt + 16 * f + lr] >> sh);
#pragma unroll
            for (int f = 0; f < FN; ++f) {
                const QuantFrag<DT> a =
                    QuantFrag<DT>::make(*reinterpret_cast<const u32x4_t*>(sw + f * 16 * kQBlock + lrow),
                                        *reinterpret_cast<const u32x4_t*>(sw + f * 16 * kQBlock + (lrow ^ 64)),
                                        s_ws[g * NB + wn / 16 + f] >> sh);
#pragma unroll
                for (int h = 0; h < FT; ++h) acc[f][h] = a.mma(b[h], acc[f][h]);
            }
            slot = slot + 1 == ST ? 0 : slot + 1;
        }
    }
    wait_vmcnt_le<0>();  // nothing may land in LDS after the workgroup has ended
#pragma unroll
    for (int f = 0; f < FN; ++f)
#pragma unroll
        for (int h = 0; h < FT; ++h) base_store4<DT>(p, t0 + wt + 16 * h + lr, n0 + wn + 16 * f + 4 * lg, acc[f][h]);
}

}  // namespace lora
