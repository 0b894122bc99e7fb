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

// Bits of the largest finite magnitude of 8 values.
__device__ __forceinline__ uint32_t finite_max8(const float* f) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t m = __float_as_uint(f[e]) & 0x7fffffffu;
        top = max(top, m < 0x7f800000u ? m : 0u);
    }
    return top;
}

// Codes of 8 values; what is not finite becomes NaN.
__device__ __forceinline__ u32x2_t encode8(const float* f, uint32_t scale) {
    const float inv = quant_inv_scale(scale);
    float z[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        z[e] = (__float_as_uint(f[e]) & 0x7f800000u) == 0x7f800000u ? __uint_as_float(0x7fc00000u) : f[e] * inv;
    return u32x2_t{quant_codes4(z[0], z[1], z[2], z[3]), quant_codes4(z[4], z[5], z[6], z[7])};
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

// 16 lanes take one block of 128: 8 values (16 bytes of bf16) a lane, so a
// wave reads 1 KB of bf16 in one load.  Columns past d are zeros.
template <int DT>
__global__ __launch_bounds__(kThreads) void quant_rows_kernel(RowsParams p) {
    constexpr int EB = Frag<DT>::kBytes;
    const int64_t units = (int64_t)p.T * p.nb;
    const int64_t step = (int64_t)gridDim.x * (kThreads / 16);
    const int sub = threadIdx.x & 15;
    for (int64_t u0 = (int64_t)blockIdx.x * (kThreads / 16); u0 < units; u0 += step) {
        const int64_t u = u0 + threadIdx.x / 16;
        const bool on = u < units;  // (whole 16-lane rows go on or off together)
        const int64_t row = (on ? u : 0) / p.nb;
        const int blk = (int)((on ? u : 0) - row * p.nb);
        const int col = blk * kQBlock + 8 * sub;
        float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (on && col < p.d) Elem<DT>::load8(p.x + (row * p.ldx + col) * EB, f);
        const uint32_t scale = quant_scale_byte(row16_max(finite_max8(f)));
        const u32x2_t c = encode8(f, scale);
        if (on) {
            *gptr(reinterpret_cast<u32x2_t*>(p.codes + row * p.ld + col)) = c;
            if (sub == 0) gptr(p.scales)[row * p.lds + blk] = (uint8_t)scale;
        }
    }
}

// 16 lanes take one block of 128, 8 values a lane.
template <int DT>
__global__ __launch_bounds__(kThreads) void dequant_rows_kernel(RowsParams p) {
    constexpr int EB = Frag<DT>::kBytes;
    const int64_t units = (int64_t)p.T * p.nb;
    const int64_t step = (int64_t)gridDim.x * (kThreads / 16);
    const int sub = threadIdx.x & 15;
    for (int64_t u = (int64_t)blockIdx.x * (kThreads / 16) + threadIdx.x / 16; u < units; u += step) {
        const int64_t row = u / p.nb;
        const int blk = (int)(u - row * p.nb);
        const int col = blk * kQBlock + 8 * sub;
        if (col >= p.d) continue;
        const u32x2_t c = *gptr(reinterpret_cast<const u32x2_t*>(p.codes + row * p.ld + col));
        store_frag(p.xo + (row * p.ldx + col) * EB, dequant8<DT>(c[0], c[1], quant_scale(gptr(p.scales)[row * p.lds + blk])));
    }
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
// pass.  TR: the block's codes go through LDS and out as columns, so the
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
    float f[8][8];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = nb * kQBlock + 16 * i + r0;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[i][e] = 0.f;
        if (row < p.n && col < p.k) Elem<DT>::load8(p.w + ((int64_t)row * p.ldw + col) * EB, f[i]);
        top = max(top, finite_max8(f[i]));
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
        const u32x2_t c = encode8(f[i], scale);
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

unsigned rows_grid(int64_t units) {
    return (unsigned)std::max<int64_t>(1, std::min<int64_t>((units + kThreads / 16 - 1) / (kThreads / 16), 256 * 32));
}

int check_rows(int dtype, const void* x, int64_t ldx, int32_t T, int32_t d, const lora_quant& q) {
    if (!valid_dtype(dtype) || T < 0 || d < 1) return LORA_ERR_INVALID_ARG;
    if (T == 0) return LORA_OK;
    const int rc = check_matrix(x, d, ldx);
    return rc != LORA_OK ? rc : check_quant(q, d);
}

RowsParams rows_params(int64_t ldx, int32_t T, int32_t d, const lora_quant& q) {
    return RowsParams{nullptr, nullptr, ldx, q.codes, q.ld, q.scales, q.lds, T, d, (d + kQBlock - 1) / kQBlock};
}

}  // namespace

extern "C" int lora_quant_rows(int dtype, const void* x, int64_t ldx, int32_t T, int32_t d, lora_quant q, void* stream) {
    const int rc = check_rows(dtype, x, ldx, T, d, q);
    if (rc != LORA_OK || T == 0) return rc;
    RowsParams p = rows_params(ldx, T, d, q);
    p.x = static_cast<const char*>(x);
    const dim3 grid(rows_grid((int64_t)T * p.nb)), block(kThreads);
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (dtype == LORA_BF16)
        hipLaunchKernelGGL(quant_rows_kernel<LORA_BF16>, grid, block, 0, st, p);
    else
        hipLaunchKernelGGL(quant_rows_kernel<LORA_F32>, grid, block, 0, st, p);
    return hipGetLastError() == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

extern "C" int lora_dequant_rows(int dtype, lora_quant q, int32_t T, int32_t d, void* x, int64_t ldx, void* stream) {
    const int rc = check_rows(dtype, x, ldx, T, d, q);
    if (rc != LORA_OK || T == 0) return rc;
    RowsParams p = rows_params(ldx, T, d, q);
    p.xo = static_cast<char*>(x);
    const dim3 grid(rows_grid((int64_t)T * p.nb)), block(kThreads);
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
    const int64_t nbs = ((int64_t)d_out + kQBlock - 1) / kQBlock;
    if (nbs > 65535) return LORA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)(((int64_t)d_in + kQBlock - 1) / kQBlock), (unsigned)nbs), block(kThreads);
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
