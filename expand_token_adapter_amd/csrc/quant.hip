// quant.hip -- lora_quant_rows, lora_dequant_rows and lora_quant_weight.
//
// The activation checkpoint of the fine-tuning rows in 8 bits and the frozen
// weight's 8-bit form (quant.h states the form).  Streams over HBM: each value
// is read once and written once.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "quant.h"

using namespace lora;

namespace {

constexpr int kThreads = 256;

// max over the 16 lanes of a DPP row, in every lane (magnitudes as bits).
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x128, 0xf, 0xf, true));  // rotate by 8 lanes
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x124, 0xf, 0xf, true));
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x122, 0xf, 0xf, true));
    return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x121, 0xf, 0xf, true));
}

// fp32 bits of the largest magnitude of 8 values, at or above kNotFinite if one
// of them is not finite.
constexpr uint32_t kNotFinite = 0x7f800000u;
__device__ __forceinline__ uint32_t max8(const Frag<LORA_BF16>& f) {
    typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
    u16x2_t top{0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2_t, f.q[i] & 0x7fff7fffu));
    return (uint32_t)max(top[0], top[1]) << 16;
}
__device__ __forceinline__ uint32_t max8(const Frag<LORA_F32>& f) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, max(f.q0[i] & 0x7fffffffu, f.q1[i] & 0x7fffffffu));
    return top;
}

// The 8 values with zeros (nan false) or NaN in place of those that are not finite.
template <int DT>
__device__ Frag<DT> finite8(const Frag<DT>& f, bool nan) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[e] = f.get(e);
        if ((__float_as_uint(v[e]) & kNotFinite) == kNotFinite) v[e] = nan ? __uint_as_float(0x7fc00000u) : 0.f;
    }
    return Frag<DT>::from_f32(v);
}

// Codes of 8 values with |value| <= 448 * 2^(scale - 127), or NaN.
__device__ __forceinline__ u32x2_t encode8(const Frag<LORA_BF16>& f, uint32_t scale) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    typedef short i16x2_t __attribute__((ext_vector_type(2)));
    const float s = quant_scale(scale);
    u32x2_t c;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = f.q[2 * i], hi = f.q[2 * i + 1];  // (a bit cast of a vector's element takes its first)
        i16x2_t w{0, 0};
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, __builtin_bit_cast(bf16x2_t, lo), s, false);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, __builtin_bit_cast(bf16x2_t, hi), s, true);
        c[i] = __builtin_bit_cast(uint32_t, w);
    }
    return c;
}
__device__ __forceinline__ u32x2_t encode8(const Frag<LORA_F32>& f, uint32_t scale) {
    typedef short i16x2_t __attribute__((ext_vector_type(2)));
    const float s = quant_scale(scale);
    u32x2_t c;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        i16x2_t w{0, 0};
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, f.get(4 * i), f.get(4 * i + 1), s, false);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, f.get(4 * i + 2), f.get(4 * i + 3), s, true);
        c[i] = __builtin_bit_cast(uint32_t, w);
    }
    return c;
}

struct RowsParams {
    const char* x;
    char* xo;
    int64_t ldx;
    uint8_t* codes;
    int64_t ld;
    uint8_t* scales;
    int64_t lds;
    int32_t T, d, nb;  // nb: blocks of a row
};

// 16 lanes take one block of 128, 8 values (16 bytes of bf16, 8 codes) a lane:
// a wave's load is 1 KB of bf16 and its store 512 bytes of codes.  Each takes a
// few blocks, all loads in flight at once.  Streams: 4096 x 5120 bf16 rows are
// saved in 10.5 us (with 1 and 4 blocks 11.3 and 11.0) and restored in 9.9 (with 1
// and 2 blocks 11.1 and 10.2) with part of the data in the last-level cache, in
// 14.5 and 14.2 us (4.4 TB/s) from HBM, fp32 rows in 21.0 and 27.1; a large copy
// runs at 5.1 TB/s.  What bounds the save beside memory is vector work: the magnitudes
// are compared as packed 16-bit integers and the conversion divides by the scale
// (with fp32 arithmetic for both: 11.6 us).
constexpr int kSaveUnits = 2, kRestoreUnits = 4;

// Unit (row, block) i of this lane's 16; on: it exists.
struct RowUnit {
    int64_t row;
    uint32_t blk;
    int col;
    bool on;
};
template <int U>
__device__ __forceinline__ RowUnit row_unit(const RowsParams& p, int i) {
    const uint32_t units = (uint32_t)p.T * (uint32_t)p.nb;
    const uint32_t u = blockIdx.x * (uint32_t)(kThreads / 16 * U) + (uint32_t)(kThreads / 16 * i) + threadIdx.x / 16;
    const uint32_t uc = u < units ? u : units - 1;
    const uint32_t row = uc / (uint32_t)p.nb, blk = uc - row * (uint32_t)p.nb;
    return RowUnit{(int64_t)row, blk, (int)blk * kQBlock + 8 * (int)(threadIdx.x & 15), u < units};
}

// (columns past d are zeros)
template <int DT>
__global__ __launch_bounds__(kThreads) void quant_rows_kernel(RowsParams p) {
    constexpr int EB = Frag<DT>::kBytes;
    RowUnit r[kSaveUnits];
    Frag<DT> f[kSaveUnits];
#pragma unroll
    for (int i = 0; i < kSaveUnits; ++i) {
        r[i] = row_unit<kSaveUnits>(p, i);
        f[i] = Frag<DT>::load(p.x + (r[i].row * p.ldx + (r[i].col < p.d ? r[i].col : 0)) * EB);
    }
#pragma unroll
    for (int i = 0; i < kSaveUnits; ++i) {
        f[i] = f[i].masked(r[i].col < p.d);
        uint32_t top = row16_max(max8(f[i]));
        if (__ballot(top >= kNotFinite)) {
            // (rare: a block of this wave holds infinities or NaN)
            top = row16_max(max8(finite8<DT>(f[i], false)));
            f[i] = finite8<DT>(f[i], true);
        }
        const uint32_t scale = quant_scale_byte(top);
        if (r[i].on) {
            *gptr(reinterpret_cast<u32x2_t*>(p.codes + r[i].row * p.ld + r[i].col)) = encode8(f[i], scale);
            if ((threadIdx.x & 15) == 0) gptr(p.scales)[r[i].row * p.lds + r[i].blk] = (uint8_t)scale;
        }
    }
}

template <int DT>
__global__ __launch_bounds__(kThreads) void dequant_rows_kernel(RowsParams p) {
    constexpr int EB = Frag<DT>::kBytes;
    RowUnit r[kRestoreUnits];
    u32x2_t c[kRestoreUnits];
    uint32_t s[kRestoreUnits];
#pragma unroll
    for (int i = 0; i < kRestoreUnits; ++i) {
        r[i] = row_unit<kRestoreUnits>(p, i);
        c[i] = *gptr(reinterpret_cast<const u32x2_t*>(p.codes + r[i].row * p.ld + r[i].col));
        s[i] = gptr(p.scales)[r[i].row * p.lds + r[i].blk];
    }
#pragma unroll
    for (int i = 0; i < kRestoreUnits; ++i)
        if (r[i].on && r[i].col < p.d)
            store_frag(p.xo + (r[i].row * p.ldx + r[i].col) * EB, dequant8<DT>(c[i][0], c[i][1], quant_scale(s[i])));
}

struct WeightParams {
    const char* w;
    int64_t ldw;
    uint8_t* codes;
    int64_t ld;
    uint8_t* scales;
    int64_t lds;
    int32_t n, k;
};

// One workgroup per 128 x 128 block: 16 lanes x 8 values a row, 16 rows a
// pass.  A stream over HBM: 14336 x 4096 bf16 in 34.4 us (5.1 TB/s), transposed
// 37.4; fp32 53.7 and 56.5.  TR: the block's codes go through LDS and out as columns, so the
// codes and scales are those of the transposed weight (a block's largest
// magnitude is the same either way).
constexpr int kTrPitch = kQBlock + 4;
template <int DT, bool TR>
__global__ __launch_bounds__(kThreads) void quant_weight_kernel(WeightParams p) {
    constexpr int EB = Frag<DT>::kBytes;
    __shared__ uint32_t s_top[kThreads / kWave];
    __shared__ __attribute__((aligned(16))) uint8_t s_t[TR ? kQBlock * kTrPitch : 16];
    const int sub = threadIdx.x & 15;
    const int r0 = threadIdx.x / 16;
    const int kb = blockIdx.x, nb = blockIdx.y;
    const int col = kb * kQBlock + 8 * sub;
    Frag<DT> f[8];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = nb * kQBlock + 16 * i + r0;
        f[i] = Frag<DT>::zero();
        if (row < p.n && col < p.k) f[i] = Frag<DT>::load(p.w + ((int64_t)row * p.ldw + col) * EB);
        top = max(top, max8(finite8<DT>(f[i], false)));
    }
    top = row16_max(top);
    top = max(top, (uint32_t)__shfl_xor((int)top, 16, kWave));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32, kWave));
    if ((threadIdx.x & (kWave - 1)) == 0) s_top[threadIdx.x / kWave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / kWave; ++w) top = max(top, s_top[w]);
    const uint32_t scale = quant_scale_byte(top);
    if (threadIdx.x == 0) gptr(p.scales)[(int64_t)(TR ? kb : nb) * p.lds + (TR ? nb : kb)] = (uint8_t)scale;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = nb * kQBlock + 16 * i + r0;
        const u32x2_t c = encode8(finite8<DT>(f[i], true), scale);
        if constexpr (TR) {
            uint8_t* t = s_t + 8 * sub * kTrPitch + 16 * i + r0;
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e * kTrPitch] = (uint8_t)((e < 4 ? c[0] : c[1]) >> (8 * (e & 3)));
        } else if (row < p.n) {
            *gptr(reinterpret_cast<u32x2_t*>(p.codes + (int64_t)row * p.ld + col)) = c;
        }
    }
    if constexpr (TR) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = kb * kQBlock + 16 * i + r0;  // a row of the transposed weight
            const uint32_t* t = reinterpret_cast<const uint32_t*>(s_t + (16 * i + r0) * kTrPitch + 8 * sub);
            if (row < p.k)
                *gptr(reinterpret_cast<u32x2_t*>(p.codes + (int64_t)row * p.ld + nb * kQBlock + 8 * sub)) = u32x2_t{t[0], t[1]};
        }
    }
}

// Workgroups for T rows of d values, `units` blocks a lane.
int64_t rows_grid(int32_t T, int32_t d, int units) {
    const int64_t per = kThreads / 16 * units;
    return ((int64_t)T * ((d + (int64_t)kQBlock - 1) / kQBlock) + per - 1) / per;
}

int check_rows(int dtype, const void* x, int64_t ldx, int32_t T, int32_t d, const lora_quant& q, int units) {
    if (!valid_dtype(dtype) || T < 0 || d < 1) return LORA_ERR_INVALID_ARG;
    if (T == 0) return LORA_OK;
    int rc = check_matrix(x, d, ldx);
    if (rc == LORA_OK) rc = check_quant(q, d);
    if (rc != LORA_OK) return rc;
    return grid_fits(rows_grid(T, d, units), kThreads) ? LORA_OK : LORA_ERR_UNSUPPORTED;
}
static_assert(kSaveUnits <= 8 && kRestoreUnits <= 8, "blocks are numbered in 32 bits");

RowsParams rows_params(int64_t ldx, int32_t T, int32_t d, const lora_quant& q) {
    return RowsParams{nullptr, nullptr, ldx, q.codes, q.ld, q.scales, q.lds, T, d,
                      (int32_t)(((int64_t)d + kQBlock - 1) / kQBlock)};
}

}  // namespace

extern "C" int lora_quant_rows(int dtype, const void* x, int64_t ldx, int32_t T, int32_t d, lora_quant q, void* stream) {
    const int rc = check_rows(dtype, x, ldx, T, d, q, kSaveUnits);
    if (rc != LORA_OK || T == 0) return rc;
    RowsParams p = rows_params(ldx, T, d, q);
    p.x = static_cast<const char*>(x);
    const dim3 grid((unsigned)rows_grid(T, d, kSaveUnits)), block(kThreads);
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (dtype == LORA_BF16)
        hipLaunchKernelGGL(quant_rows_kernel<LORA_BF16>, grid, block, 0, st, p);
    else
        hipLaunchKernelGGL(quant_rows_kernel<LORA_F32>, grid, block, 0, st, p);
    return hipGetLastError() == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

extern "C" int lora_dequant_rows(int dtype, lora_quant q, int32_t T, int32_t d, void* x, int64_t ldx, void* stream) {
    const int rc = check_rows(dtype, x, ldx, T, d, q, kRestoreUnits);
    if (rc != LORA_OK || T == 0) return rc;
    RowsParams p = rows_params(ldx, T, d, q);
    p.xo = static_cast<char*>(x);
    const dim3 grid((unsigned)rows_grid(T, d, kRestoreUnits)), block(kThreads);
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (dtype == LORA_BF16)
        hipLaunchKernelGGL(dequant_rows_kernel<LORA_BF16>, grid, block, 0, st, p);
    else
        hipLaunchKernelGGL(dequant_rows_kernel<LORA_F32>, grid, block, 0, st, p);
    return hipGetLastError() == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

extern "C" int lora_quant_weight(int dtype, const void* w, int64_t ldw, int32_t d_out, int32_t d_in, int32_t transpose,
                                 lora_quant q, void* stream) {
    if (!valid_dtype(dtype) || d_out < 1 || d_in < 1 || (transpose != 0 && transpose != 1)) return LORA_ERR_INVALID_ARG;
    int rc = check_matrix(w, d_in, ldw);
    if (rc == LORA_OK) rc = check_quant(q, transpose ? d_out : d_in);
    if (rc != LORA_OK) return rc;
    if (d_out % 8 != 0) return LORA_ERR_UNSUPPORTED;
    const WeightParams p{static_cast<const char*>(w), ldw, q.codes, q.ld, q.scales, q.lds, d_out, d_in};
    const int64_t nbs = ((int64_t)d_out + kQBlock - 1) / kQBlock, kbs = ((int64_t)d_in + kQBlock - 1) / kQBlock;
    if (nbs > 65535 || !grid_fits(kbs, kThreads)) return LORA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)kbs, (unsigned)nbs), block(kThreads);
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (dtype == LORA_BF16 && transpose)
        hipLaunchKernelGGL((quant_weight_kernel<LORA_BF16, true>), grid, block, 0, st, p);
    else if (dtype == LORA_BF16)
        hipLaunchKernelGGL((quant_weight_kernel<LORA_BF16, false>), grid, block, 0, st, p);
    else if (transpose)
        hipLaunchKernelGGL((quant_weight_kernel<LORA_F32, true>), grid, block, 0, st, p);
    else
        hipLaunchKernelGGL((quant_weight_kernel<LORA_F32, false>), grid, block, 0, st, p);
    return hipGetLastError() == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}
