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

// A unit is 256 columns of a row (padding included), 32 lanes with 8 columns each; four
// lanes share a scale.  Streams: 16384 x 4096 bf16 rows are saved in 33 us and restored in
// 32 from HBM (5.1 and 5.4 TB/s, as a large copy), fp32 rows in 60 and 55; 4096 x 5120 bf16
// in 13.5 and 13.1.
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

// A lane restores 16 bytes: 8 bf16 or 4 fp32 values, of a word or half a word of codes, so
// that a wave writes 1 KB in one piece (16384 x 4096 fp32 rows with 8 values a lane: 75 us
// in place of 55).
template <int DT>
__global__ __launch_bounds__(kThreads) void mx_restore_kernel(MxRowsParams p) {
    constexpr int EB = Frag<DT>::kBytes, V = 16 / EB;
    constexpr int kLanes = kMxPad / V;  // of a unit
    const uint32_t units = (uint32_t)p.T * (uint32_t)p.nc;
    const int lane = threadIdx.x % kLanes;
    int64_t row[kRestoreUnits];
    int col[kRestoreUnits];
    uint32_t c[kRestoreUnits], s[kRestoreUnits];
    bool on[kRestoreUnits];
#pragma unroll
    for (int i = 0; i < kRestoreUnits; ++i) {
        const uint32_t u = (blockIdx.x * (uint32_t)kRestoreUnits + (uint32_t)i) * (uint32_t)(kThreads / kLanes) + threadIdx.x / kLanes;
        const uint32_t uc = u < units ? u : units - 1, r = uc / (uint32_t)p.nc;
        row[i] = r;
        col[i] = (int)(uc - r * (uint32_t)p.nc) * kMxPad + V * lane;
        on[i] = u < units && col[i] < p.d;
        const uint8_t* at = p.codes + row[i] * p.ld + col[i] / 2;
        if constexpr (DT == LORA_BF16)
            c[i] = *gptr(reinterpret_cast<const uint32_t*>(at));
        else
            c[i] = *gptr(reinterpret_cast<const uint16_t*>(at));
        s[i] = gptr(p.scales)[row[i] * p.lds + col[i] / kMxBlock];
    }
#pragma unroll
    for (int i = 0; i < kRestoreUnits; ++i) {
        const Frag<DT> f = mx_decode8<DT>(c[i], quant_scale(s[i]));
        u32x4_t v;
        if constexpr (DT == LORA_BF16)
            v = f.q;
        else
            v = f.q0;
        if (on[i]) *gptr(reinterpret_cast<u32x4_t*>(p.xo + (row[i] * p.ldx + col[i]) * EB)) = v;
    }
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

// The largest of a value of each lane over the 4 lanes of a block's row and the lanes
// LANES, 2 LANES, ... apart, up to those END lanes apart.
template <int LANES, int END = kWave>
__device__ __forceinline__ uint32_t block_max(uint32_t v) {
    v = quad_max(v);
#pragma unroll
    for (int d = LANES; d < END; d *= 2) v = max(v, (uint32_t)__shfl_xor((int)v, d, kWave));
    return v;
}

// A weight as it is: a wave takes 32 rows x 256 columns, 32 lanes a row and 16 rows of its
// own a lane, so that a row's 512 bytes are read and 128 bytes of codes written at a time;
// a workgroup's waves lie one below the other.  (14336 x 4096 bf16: 35 us, 4.2 TB/s; with 64
// columns a wave 38.)
template <int DT>
__global__ __launch_bounds__(kThreads) void mx_weight_kernel(MxWeightParams p) {
    constexpr int EB = Frag<DT>::kBytes, NR = 16;
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t row0 = ((int64_t)blockIdx.y * (kThreads / kWave) + threadIdx.x / kWave) * 32 + lane / kUnitLanes;
    const int64_t col = (int64_t)blockIdx.x * kMxPad + 8 * (lane & (kUnitLanes - 1));
    Frag<DT> f[NR];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        f[i] = Frag<DT>::zero();
        if (row0 + 2 * i < p.n && col < p.k) f[i] = Frag<DT>::load(p.w + ((row0 + 2 * i) * p.ldw + col) * EB);
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) top = max(top, max8(f[i]));
    top = block_max<32>(top);
    const bool nan = top >= kNotFinite;
    const uint32_t scale = nan ? kMxNan : mx_scale_byte(top);
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int64_t row = row0 + 2 * i;
        if (row >= p.n) continue;
        *gptr(reinterpret_cast<uint32_t*>(p.codes + row * p.ld + col / 2)) = nan ? 0u : mx_encode8(f[i], quant_scale(scale));
        if ((lane & 3) == 0) gptr(p.scales)[row * p.lds + col / kMxBlock] = (uint8_t)scale;
    }
}

// Codes of 8 values of one column, of the fragments of 8 rows.
__device__ __forceinline__ uint32_t mx_encode_column(const Frag<LORA_BF16>* f, int e, float s) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    // (the halves e & 1 of two rows' words, the first row's low)
    const uint32_t sel = (e & 1) ? 0x07060302u : 0x05040100u;
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __builtin_amdgcn_perm(f[2 * i + 1].q[e >> 1], f[2 * i].q[e >> 1], sel);
    uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(0u, __builtin_bit_cast(bf16x2_t, v[0]), s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, v[1]), s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, v[2]), s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, v[3]), s, 3);
}
__device__ __forceinline__ uint32_t mx_encode_column(const Frag<LORA_F32>* f, int e, float s) {
    uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, f[0].get(e), f[1].get(e), s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[2].get(e), f[3].get(e), s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[4].get(e), f[5].get(e), s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[6].get(e), f[7].get(e), s, 3);
}

// Its transpose: a workgroup takes 256 rows x kTrCols columns, a lane 8 x 8 values, whose
// codes it makes column by column, a word of 8 rows each; a column's 256 codes, put
// together in LDS, are written 128 bytes at a time.  (14336 x 4096 bf16: 38.7 us, with
// 128 columns 40.4, with codes put into LDS a byte each 48.4.)
constexpr int kTrCols = 64, kTrLanes = kTrCols / 8, kTrThreads = 32 * kTrLanes;
constexpr int kTrPitch = 33;  // words: 8 columns of 8 rows fall on different banks
template <int DT>
__global__ __launch_bounds__(kTrThreads) void mx_weight_t_kernel(MxWeightParams p) {
    constexpr int EB = Frag<DT>::kBytes;
    __shared__ uint32_t s_t[kTrCols * kTrPitch];
    __shared__ __attribute__((aligned(8))) uint8_t s_scale[kTrCols / 32][8];
    const int sub = threadIdx.x % kTrLanes, rg = threadIdx.x / kTrLanes;  // rg: of 8 rows
    const int64_t row0 = (int64_t)blockIdx.x * kMxPad;
    const int64_t col = (int64_t)blockIdx.y * kTrCols + 8 * sub;
    Frag<DT> f[8];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = row0 + 8 * rg + i;
        f[i] = Frag<DT>::zero();
        if (row < p.n && col < p.k) f[i] = Frag<DT>::load(p.w + (row * p.ldw + col) * EB);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, max8(f[i]));
    static_assert(kTrLanes * 4 <= kWave, "a block's 4 groups of 8 rows are a wave's");
    top = block_max<kTrLanes, 4 * kTrLanes>(top);
    const bool nan = top >= kNotFinite;
    const uint32_t scale = nan ? kMxNan : mx_scale_byte(top);
#pragma unroll
    for (int e = 0; e < 8; ++e) s_t[(8 * sub + e) * kTrPitch + rg] = nan ? 0u : mx_encode_column(f, e, quant_scale(scale));
    if ((sub & 3) == 0 && (rg & 3) == 0) s_scale[sub / 4][rg / 4] = (uint8_t)scale;
    __syncthreads();
    // a transposed row: 32 lanes with 8 codes each
    const int at = threadIdx.x % 32;
#pragma unroll
    for (int c = threadIdx.x / 32; c < kTrCols; c += kTrThreads / 32) {
        const int64_t q = (int64_t)blockIdx.y * kTrCols + c;
        if (q >= p.k) break;
        *gptr(reinterpret_cast<uint32_t*>(p.codes + q * p.ld + row0 / 2 + 4 * at)) = s_t[c * kTrPitch + at];
        if (at == 0)
            *gptr(reinterpret_cast<u32x2_t*>(p.scales + q * p.lds + row0 / kMxBlock)) = *reinterpret_cast<const u32x2_t*>(s_scale[c / 32]);
    }
}

int32_t units_of(int32_t d) { return (int32_t)(((int64_t)d + kMxPad - 1) / kMxPad); }
// Workgroups for T rows of d values, `units` units of a workgroup.
int64_t rows_grid(int32_t T, int32_t d, int units) { return ((int64_t)T * units_of(d) + units - 1) / units; }
constexpr int kSaveWg = kUnitsWg * kSaveUnits;
int restore_wg(int dtype) { return kRestoreUnits * (dtype == LORA_BF16 ? kUnitsWg : kUnitsWg / 2); }

int check_rows(int dtype, const void* x, int64_t ldx, int32_t T, int32_t d, const lora_quant& q, int units) {
    if (!valid_dtype(dtype) || T < 0 || d < 1) return LORA_ERR_INVALID_ARG;
    if (T == 0) return LORA_OK;
    int rc = check_matrix(x, d, ldx);
    if (rc == LORA_OK) rc = check_mx(q, d);
    if (rc != LORA_OK) return rc;
    return grid_fits(rows_grid(T, d, units), kThreads) ? LORA_OK : LORA_ERR_UNSUPPORTED;
}
static_assert(kSaveWg <= kThreads && kRestoreUnits * kUnitsWg <= kThreads, "units are numbered in 32 bits");

MxRowsParams rows_params(int64_t ldx, int32_t T, int32_t d, const lora_quant& q) {
    return MxRowsParams{nullptr, nullptr, ldx, q.codes, q.ld, q.scales, q.lds, T, d, units_of(d)};
}

}  // namespace

extern "C" int lora_quant_rows_mx(int dtype, const void* x, int64_t ldx, int32_t T, int32_t d, lora_quant q, void* stream) {
    const int rc = check_rows(dtype, x, ldx, T, d, q, kSaveWg);
    if (rc != LORA_OK || T == 0) return rc;
    MxRowsParams p = rows_params(ldx, T, d, q);
    p.x = static_cast<const char*>(x);
    const dim3 grid((unsigned)rows_grid(T, d, kSaveWg)), block(kThreads);
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (dtype == LORA_BF16)
        hipLaunchKernelGGL(mx_rows_kernel<LORA_BF16>, grid, block, 0, st, p);
    else
        hipLaunchKernelGGL(mx_rows_kernel<LORA_F32>, grid, block, 0, st, p);
    return hipGetLastError() == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

extern "C" int lora_dequant_rows_mx(int dtype, lora_quant q, int32_t T, int32_t d, void* x, int64_t ldx, void* stream) {
    const int rc = check_rows(dtype, x, ldx, T, d, q, restore_wg(dtype));
    if (rc != LORA_OK || T == 0) return rc;
    MxRowsParams p = rows_params(ldx, T, d, q);
    p.xo = static_cast<char*>(x);
    const dim3 grid((unsigned)rows_grid(T, d, restore_wg(dtype))), block(kThreads);
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
    const int64_t gy = transpose ? ((int64_t)d_in + kTrCols - 1) / kTrCols : ((int64_t)d_out + 127) / 128;
    if (gy > 65535 || !grid_fits(gx, kTrThreads)) return LORA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)gx, (unsigned)gy), block(transpose ? kTrThreads : kThreads);
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (dtype == LORA_BF16 && transpose)
        hipLaunchKernelGGL(mx_weight_t_kernel<LORA_BF16>, grid, block, 0, st, p);
    else if (dtype == LORA_BF16)
        hipLaunchKernelGGL(mx_weight_kernel<LORA_BF16>, grid, block, 0, st, p);
    else if (transpose)
        hipLaunchKernelGGL(mx_weight_t_kernel<LORA_F32>, grid, block, 0, st, p);
    else
        hipLaunchKernelGGL(mx_weight_kernel<LORA_F32>, grid, block, 0, st, p);
    return hipGetLastError() == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}
