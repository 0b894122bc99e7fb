// mx.hip -- lora_quant_rows_mx, lora_dequant_rows_mx and lora_quant_weight_mx.
//
// Rows and frozen weights into the microscaled 4-bit form (mx.h states it) and
// back.  Streams over HBM: each value is read once and written once.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "mx.h"

using namespace lora;

namespace {

constexpr int kThreads = 256;
constexpr int kUnitLanes = kMxPad / 8;  // lanes of a unit: 8 columns each
constexpr int kUnitsWg = kThreads / kUnitLanes;

// max over the 4 lanes of a block, in each of them.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xb1, 0xf, 0xf, true));  // lanes 1 0 3 2
    return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4e, 0xf, 0xf, true));  // lanes 2 3 0 1
}

struct MxRowsParams {
    const char* x;
    char* xo;
    int64_t ldx;
    uint8_t* codes;
    int64_t ld;
    uint8_t* scales;
    int64_t lds;
    int32_t T, d, nc;  // nc: units of a row
};

// A unit is 256 columns of a row (padding included), 32 lanes with 8 columns each;
// four lanes share a scale.
constexpr int kSaveUnits = 4, kRestoreUnits = 4;

struct MxUnit {
    int64_t row;
    int col;
    bool on;
};
template <int U>
__device__ __forceinline__ MxUnit mx_unit(const MxRowsParams& p, int i) {
    const uint32_t units = (uint32_t)p.T * (uint32_t)p.nc;
    const uint32_t u = blockIdx.x * (uint32_t)(kUnitsWg * U) + (uint32_t)(kUnitsWg * i) + threadIdx.x / kUnitLanes;
    const uint32_t uc = u < units ? u : units - 1;
    const uint32_t row = uc / (uint32_t)p.nc;
    return MxUnit{(int64_t)row, (int)(uc - row * (uint32_t)p.nc) * kMxPad + 8 * (int)(threadIdx.x & (kUnitLanes - 1)), u < units};
}

// (columns past d are zeros, and the scales of blocks without a column 1)
template <int DT>
__global__ __launch_bounds__(kThreads) void mx_rows_kernel(MxRowsParams p) {
    constexpr int EB = Frag<DT>::kBytes;
    MxUnit r[kSaveUnits];
    Frag<DT> f[kSaveUnits];
#pragma unroll
    for (int i = 0; i < kSaveUnits; ++i) {
        r[i] = mx_unit<kSaveUnits>(p, i);
        f[i] = Frag<DT>::load(p.x + (r[i].row * p.ldx + (r[i].col < p.d ? r[i].col : 0)) * EB);
    }
#pragma unroll
    for (int i = 0; i < kSaveUnits; ++i) {
        f[i] = f[i].masked(r[i].col < p.d);
        const uint32_t top = quad_max(max8(f[i]));
        const bool nan = top >= kNotFinite;
        const uint32_t scale = nan ? kMxNan : mx_scale_byte(top);
        const uint32_t w = nan ? 0u : mx_encode8(f[i], quant_scale(scale));
        if (r[i].on) {
            *gptr(reinterpret_cast<uint32_t*>(p.codes + r[i].row * p.ld + r[i].col / 2)) = w;
            if ((threadIdx.x & 3) == 0) gptr(p.scales)[r[i].row * p.lds + r[i].col / kMxBlock] = (uint8_t)scale;
        }
    }
}

template <int DT>
__global__ __launch_bounds__(kThreads) void mx_restore_kernel(MxRowsParams p) {
    constexpr int EB = Frag<DT>::kBytes;
    MxUnit r[kRestoreUnits];
    uint32_t c[kRestoreUnits], s[kRestoreUnits];
#pragma unroll
    for (int i = 0; i < kRestoreUnits; ++i) {
        r[i] = mx_unit<kRestoreUnits>(p, i);
        c[i] = *gptr(reinterpret_cast<const uint32_t*>(p.codes + r[i].row * p.ld + r[i].col / 2));
        s[i] = gptr(p.scales)[r[i].row * p.lds + r[i].col / kMxBlock];
    }
#pragma unroll
    for (int i = 0; i < kRestoreUnits; ++i)
        if (r[i].on && r[i].col < p.d) store_frag(p.xo + (r[i].row * p.ldx + r[i].col) * EB, mx_decode8<DT>(c[i], quant_scale(s[i])));
}

struct MxWeightParams {
    const char* w;
    int64_t ldw;
    uint8_t* codes;
    int64_t ld;
    uint8_t* scales;
    int64_t lds;
    int32_t n, k;
};

// A workgroup takes R rows x C columns of w: C / 8 lanes a row, kThreads * 8 / C rows
// a pass, and whole 32 x 32 blocks, whose largest magnitudes meet in LDS.  As it
// is: 32 rows x 256 columns (128 bytes of codes of a row at a time).  Transposed:
// 256 rows x 64 columns, so that 128 bytes of bf16 of a row are read and 128 bytes
// of codes of a transposed row written at a time; codes go through LDS, a byte each.
constexpr int kTrPitch = 256 + 8;
template <int DT, bool TR>
__global__ __launch_bounds__(kThreads) void mx_weight_kernel(MxWeightParams p) {
    constexpr int EB = Frag<DT>::kBytes;
    constexpr int R = TR ? 256 : 32, C = TR ? 64 : 256;
    constexpr int LR = C / 8, RP = kThreads / LR, NP = R / RP;  // lanes of a row, rows of a pass, passes
    constexpr int NBR = R / 32, NBC = C / 32;
    constexpr int PB = 32 / RP;  // passes of a 32-row block (at least 1)
    static_assert(RP <= 32 && 32 % RP == 0, "a pass lies in one row of blocks");
    __shared__ uint32_t s_top[NBR * NBC][kThreads / kWave];
    __shared__ __attribute__((aligned(16))) uint8_t s_t[TR ? C * kTrPitch : 16];
    const int sub = threadIdx.x % LR, r0 = threadIdx.x / LR;
    const int wave = threadIdx.x / kWave;
    const int64_t row0 = (int64_t)(TR ? blockIdx.x : blockIdx.y) * R;
    const int64_t col = (int64_t)(TR ? blockIdx.y : blockIdx.x) * C + 8 * sub;
    Frag<DT> f[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int64_t row = row0 + RP * i + r0;
        f[i] = Frag<DT>::zero();
        if (row < p.n && col < p.k) f[i] = Frag<DT>::load(p.w + (row * p.ldw + col) * EB);
    }
    // The 32 x 32 blocks' largest magnitudes: over this lane's passes, the 4 lanes of a
    // block's row, the wave's rows, and the waves.
#pragma unroll
    for (int b = 0; b < NBR; ++b) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < PB; ++i) top = max(top, max8(f[b * PB + i]));
        top = quad_max(top);
#pragma unroll
        for (int d = LR; d < kWave; d *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, d, kWave));
        if ((threadIdx.x & (kWave - 1)) < LR && (sub & 3) == 0) s_top[b * NBC + sub / 4][wave] = top;
    }
    __syncthreads();
    uint32_t scale[NBR];
#pragma unroll
    for (int b = 0; b < NBR; ++b) {
        uint32_t top = 0;
#pragma unroll
        for (int w = 0; w < kThreads / kWave; ++w) top = max(top, s_top[b * NBC + sub / 4][w]);
        scale[b] = top >= kNotFinite ? kMxNan : mx_scale_byte(top);
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const uint32_t s = scale[i / PB];
        const uint32_t w = s == kMxNan ? 0u : mx_encode8(f[i], quant_scale(s));
        const int row = RP * i + r0;
        if constexpr (TR) {
#pragma unroll
            for (int e = 0; e < 8; ++e) s_t[(8 * sub + e) * kTrPitch + row] = (uint8_t)((w >> (4 * e)) & 15u);
        } else if (row0 + row < p.n) {
            *gptr(reinterpret_cast<uint32_t*>(p.codes + (row0 + row) * p.ld + col / 2)) = w;
            if ((sub & 3) == 0) gptr(p.scales)[(row0 + row) * p.lds + col / kMxBlock] = (uint8_t)s;
        }
    }
    if constexpr (TR) {
        __syncthreads();
        // a transposed row: 32 lanes with 8 codes each
        const int sub8 = threadIdx.x % 32, c0 = threadIdx.x / 32;
#pragma unroll
        for (int c = c0; c < C; c += kThreads / 32) {
            const int64_t q = (int64_t)blockIdx.y * C + c;
            if (q >= p.k) break;
            const u32x2_t t = *reinterpret_cast<const u32x2_t*>(s_t + c * kTrPitch + 8 * sub8);
            // bytes 0 .. 7 -> nibbles 0 .. 7
            const uint32_t lo = t[0] | t[0] >> 4, hi = t[1] | t[1] >> 4;
            const uint32_t w = (lo & 0xffu) | (lo >> 8 & 0xff00u) | ((hi & 0xffu) << 16) | ((hi >> 8 & 0xff00u) << 16);
            *gptr(reinterpret_cast<uint32_t*>(p.codes + q * p.ld + row0 / 2 + 4 * sub8)) = w;
            if ((sub8 & 3) == 0) {
                uint32_t top = 0;
#pragma unroll
                for (int v = 0; v < kThreads / kWave; ++v) top = max(top, s_top[sub8 / 4 * NBC + c / 32][v]);
                gptr(p.scales)[q * p.lds + row0 / kMxBlock + sub8 / 4] = (uint8_t)(top >= kNotFinite ? kMxNan : mx_scale_byte(top));
            }
        }
    }
}

int32_t units_of(int32_t d) { return (int32_t)(((int64_t)d + kMxPad - 1) / kMxPad); }
// Workgroups for T rows of d values, `units` units a lane.
int64_t rows_grid(int32_t T, int32_t d, int units) {
    const int64_t per = (int64_t)kUnitsWg * units;
    return ((int64_t)T * units_of(d) + per - 1) / per;
}

int check_rows(int dtype, const void* x, int64_t ldx, int32_t T, int32_t d, const lora_quant& q, int units) {
    if (!valid_dtype(dtype) || T < 0 || d < 1) return LORA_ERR_INVALID_ARG;
    if (T == 0) return LORA_OK;
    int rc = check_matrix(x, d, ldx);
    if (rc == LORA_OK) rc = check_mx(q, d);
    if (rc != LORA_OK) return rc;
    return grid_fits(rows_grid(T, d, units), kThreads) ? LORA_OK : LORA_ERR_UNSUPPORTED;
}
static_assert(kSaveUnits <= 16 && kRestoreUnits <= 16, "units are numbered in 32 bits");

MxRowsParams rows_params(int64_t ldx, int32_t T, int32_t d, const lora_quant& q) {
    return MxRowsParams{nullptr, nullptr, ldx, q.codes, q.ld, q.scales, q.lds, T, d, units_of(d)};
}

}  // namespace

extern "C" int lora_quant_rows_mx(int dtype, const void* x, int64_t ldx, int32_t T, int32_t d, lora_quant q, void* stream) {
    const int rc = check_rows(dtype, x, ldx, T, d, q, kSaveUnits);
    if (rc != LORA_OK || T == 0) return rc;
    MxRowsParams p = rows_params(ldx, T, d, q);
    p.x = static_cast<const char*>(x);
    const dim3 grid((unsigned)rows_grid(T, d, kSaveUnits)), block(kThreads);
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (dtype == LORA_BF16)
        hipLaunchKernelGGL(mx_rows_kernel<LORA_BF16>, grid, block, 0, st, p);
    else
        hipLaunchKernelGGL(mx_rows_kernel<LORA_F32>, grid, block, 0, st, p);
    return hipGetLastError() == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

extern "C" int lora_dequant_rows_mx(int dtype, lora_quant q, int32_t T, int32_t d, void* x, int64_t ldx, void* stream) {
    const int rc = check_rows(dtype, x, ldx, T, d, q, kRestoreUnits);
    if (rc != LORA_OK || T == 0) return rc;
    MxRowsParams p = rows_params(ldx, T, d, q);
    p.xo = static_cast<char*>(x);
    const dim3 grid((unsigned)rows_grid(T, d, kRestoreUnits)), block(kThreads);
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (dtype == LORA_BF16)
        hipLaunchKernelGGL(mx_restore_kernel<LORA_BF16>, grid, block, 0, st, p);
    else
        hipLaunchKernelGGL(mx_restore_kernel<LORA_F32>, grid, block, 0, st, p);
    return hipGetLastError() == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

extern "C" int lora_quant_weight_mx(int dtype, const void* w, int64_t ldw, int32_t d_out, int32_t d_in, int32_t transpose,
                                    lora_quant q, void* stream) {
    if (!valid_dtype(dtype) || d_out < 1 || d_in < 1 || (transpose != 0 && transpose != 1)) return LORA_ERR_INVALID_ARG;
    int rc = check_matrix(w, d_in, ldw);
    if (rc == LORA_OK) rc = check_mx(q, transpose ? d_out : d_in);
    if (rc != LORA_OK) return rc;
    if (d_out % 8 != 0) return LORA_ERR_UNSUPPORTED;
    const MxWeightParams p{static_cast<const char*>(w), ldw, q.codes, q.ld, q.scales, q.lds, d_out, d_in};
    // along x the stored rows' columns (whole units), along y their rows
    const int64_t gx = units_of(transpose ? d_out : d_in);
    const int64_t gy = transpose ? ((int64_t)d_in + 63) / 64 : ((int64_t)d_out + 31) / 32;
    if (gy > 65535 || !grid_fits(gx, kThreads)) return LORA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)gx, (unsigned)gy), block(kThreads);
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (dtype == LORA_BF16 && transpose)
        hipLaunchKernelGGL((mx_weight_kernel<LORA_BF16, true>), grid, block, 0, st, p);
    else if (dtype == LORA_BF16)
        hipLaunchKernelGGL((mx_weight_kernel<LORA_BF16, false>), grid, block, 0, st, p);
    else if (transpose)
        hipLaunchKernelGGL((mx_weight_kernel<LORA_F32, true>), grid, block, 0, st, p);
    else
        hipLaunchKernelGGL((mx_weight_kernel<LORA_F32, false>), grid, block, 0, st, p);
    return hipGetLastError() == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}
