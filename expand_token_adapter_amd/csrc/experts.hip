// experts.hip -- rows to the experts of a mixture and back, and the gradients of both.
//
// Choice j of token t (number t k + j) has the place pos[t k + j] among the rows
// sorted by expert, or none (lora_expert_segments).  Everything here goes token by
// token: a token's row is read or written once, its k rows at the experts once each,
// and no two choices share a place, so there are no atomics and every sum runs over
// j (and the columns) in a fixed order.  All of it is bound by memory (us; a copy of as
// many bytes at 5.16 TB/s):
//   gather     6783 tokens, 2 of 8 experts, 4096 bf16                 32.0  (32.3)
//   gradients of combine, 4096 tokens, 4 of 32 experts, 4096 bf16    56.2  (58.6, the
//              last-level cache holds a part)
//   combine    8 tokens, 8 of 64 experts, 4096 bf16: 3.8, a launch and its two dependent
//              loads, the place and the row
#include <hip/hip_runtime.h>

#include <algorithm>

#include "device_common.h"
#include "host_checks.h"

using namespace lora;

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // choices of a token whose loads are in flight together

struct ExpertParams {
    const char* x;  // token rows read [T]: x or dy
    int64_t ldx;
    const char* o;  // expert rows read [T k]
    int64_t ldo;
    char* y;        // rows written: expert rows (gather, combine's gradient) or token rows
    int64_t ldy;
    const int32_t* pos;
    const float* w;
    float* dw;
    int32_t T, d, k, accumulate;
};

// The place of choice c, or -1.
__device__ __forceinline__ int place(const ExpertParams& p, int64_t c) {
    const int at = gptr(p.pos)[c];
    return (uint32_t)at < (uint32_t)p.T * (uint32_t)p.k ? at : -1;
}

// A thread takes 8 columns of a token: y[pos] = x.  (Token by token, not place by place:
// x is read once in place of k times.)
template <int DT>
__global__ __launch_bounds__(kThreads) void expert_gather_kernel(ExpertParams p) {
    constexpr int EB = Frag<DT>::kBytes;
    const uint32_t units = (uint32_t)p.d / 8;
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x, row = i / units;
    const int64_t t = row;
    if (t >= p.T) return;
    const int col = (int)(i - row * units) * 8;
    const Frag<DT> f = Frag<DT>::load(p.x + (t * p.ldx + col) * EB);
    for (int j0 = 0; j0 < p.k; j0 += kAhead) {
        int at[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) at[j] = j0 + j < p.k ? place(p, t * p.k + j0 + j) : -1;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (at[j] < 0) continue;
            char* to = p.y + (at[j] * p.ldy + col) * EB;
            if constexpr (DT == LORA_BF16) {
                *gptr(reinterpret_cast<u32x4_t*>(to)) = f.q;
            } else {
                LORA_GLOBAL u32x4_t* q = gptr(reinterpret_cast<u32x4_t*>(to));
                q[0] = f.q0;
                q[1] = f.q1;
            }
        }
    }
}

// A thread takes 8 columns of a token: y (+)= sum_j w_j o[pos_j], or without weights
// the plain sum (the gradient of the gather).
template <int DT, bool WEIGHTED>
__global__ __launch_bounds__(kThreads) void expert_combine_kernel(ExpertParams p) {
    constexpr int EB = Frag<DT>::kBytes;
    const uint32_t units = (uint32_t)p.d / 8;
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x, row = i / units;
    const int64_t t = row;
    if (t >= p.T) return;
    const int col = (int)(i - row * units) * 8;
    char* to = p.y + (t * p.ldy + col) * EB;
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < p.k; j0 += kAhead) {
        int at[kAhead];
        float w[kAhead];
        Frag<DT> f[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            at[j] = j0 + j < p.k ? place(p, t * p.k + j0 + j) : -1;
            if constexpr (WEIGHTED) w[j] = j0 + j < p.k ? gptr(p.w)[t * p.k + j0 + j] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (at[j] >= 0) f[j] = Frag<DT>::load(p.o + (at[j] * p.ldo + col) * EB);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (at[j] < 0) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] = WEIGHTED ? fmaf(w[j], f[j].get(e), sum[e]) : sum[e] + f[j].get(e);
        }
    }
    if (p.accumulate) {
        float old[8];
        Elem<DT>::load8(to, old);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += old[e];
    }
    Elem<DT>::store8(to, sum);
}

// W waves take a token: d_o[pos_j] = w_j dy and dw_j = <dy, o[pos_j]>, kDots choices at
// a time; lane sums over its columns in order, then over the wave's lanes and the waves.
// Both in one pass, so that dy is read once.  A wave a token where there are tokens for
// the chip and rows of less than 2048 columns, else four (us, four waves / one wave):
//   columns                        64        512       1024        2048        4096
//     32 tokens, 8 experts, bf16  5.0/6.4   5.1/5.4   5.2/6.4     5.3/8.5    6.4/12.6
//   1024 tokens, 2 experts, bf16  3.8/3.7   3.9/3.7   4.4/4.7
//                           fp32  5.4/3.8   6.0/4.5   8.1/6.9
//   2048 tokens, 2 experts, bf16  5.8/3.9   6.4/4.4   8.1/6.3
//   4096 tokens, 4 experts, bf16   13/5.6    16/9.3    20/14       32/35       69/69
//  16384 tokens, 2 experts, bf16   35/12     41/17     58/36       71/73      127/158
constexpr int kDots = 8;
template <int DT, int W>
__global__ __launch_bounds__(kThreads) void expert_combine_backward_kernel(ExpertParams p) {
    constexpr int EB = Frag<DT>::kBytes;
    constexpr int PER = kThreads / kWave / W;  // tokens of a workgroup
    __shared__ float s_dot[kThreads / kWave][kDots];
    const int wave = wave_id();
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t t = (int64_t)blockIdx.x * PER + wave / W;
    const int first = (wave % W) * kWave + lane;
    if (W == 1 && t >= p.T) return;  // (W > 1: a workgroup has one token, and every one exists)
    for (int j0 = 0; j0 < p.k; j0 += kDots) {
        int at[kDots];
        float w[kDots], dot[kDots];
#pragma unroll
        for (int j = 0; j < kDots; ++j) {
            at[j] = j0 + j < p.k ? place(p, t * p.k + j0 + j) : -1;
            w[j] = j0 + j < p.k ? gptr(p.w)[t * p.k + j0 + j] : 0.f;
            dot[j] = 0.f;
        }
        for (int c = first; c < p.d / 8; c += W * kWave) {
            const int col = 8 * c;
            Frag<DT> o[kDots];
            float dy[8];
            const Frag<DT> f = Frag<DT>::load(p.x + (t * p.ldx + col) * EB);
            if (p.dw) {
#pragma unroll
                for (int j = 0; j < kDots; ++j)
                    if (at[j] >= 0) o[j] = Frag<DT>::load(p.o + (at[j] * p.ldo + col) * EB);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) dy[e] = f.get(e);
#pragma unroll
            for (int j = 0; j < kDots; ++j) {
                if (at[j] < 0) continue;
                if (p.dw) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) dot[j] = fmaf(dy[e], o[j].get(e), dot[j]);
                }
                if (p.y) {
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = w[j] * dy[e];
                    Elem<DT>::store8(p.y + (at[j] * p.ldy + col) * EB, v);
                }
            }
        }
        if (!p.dw) continue;
#pragma unroll
        for (int j = 0; j < kDots; ++j) {
            if (j0 + j >= p.k) continue;
#pragma unroll
            for (int m = kWave / 2; m >= 1; m >>= 1) dot[j] += __shfl_xor(dot[j], m, kWave);
            if (lane == 0) s_dot[wave][j] = dot[j];
        }
        if constexpr (W > 1)
            __syncthreads();
        else
            __builtin_amdgcn_wave_barrier();
        if (wave % W == 0 && lane < kDots && j0 + lane < p.k) {
            float sum = s_dot[wave][lane];
#pragma unroll
            for (int v = 1; v < W; ++v) sum += s_dot[wave + v][lane];
            gptr(p.dw)[t * p.k + j0 + lane] = sum;
        }
        if constexpr (W > 1) __syncthreads();
    }
}

// What every call checks before its matrices.
int check_expert(int dtype, int32_t T, int32_t d, int32_t k, const int32_t* pos) {
    if (!valid_dtype(dtype) || T < 0 || d < 1 || k < 1) return LORA_ERR_INVALID_ARG;
    if (T == 0) return LORA_OK;
    if ((int64_t)T * k > INT32_MAX || !pos || ((uintptr_t)pos & 3u)) return LORA_ERR_INVALID_ARG;
    return LORA_OK;
}
bool valid_f32(const float* p) { return p && ((uintptr_t)p & 3u) == 0; }

// Rows of d values, and an array of 4-byte numbers of the choices.
RowSpan rows_span(int dtype, const void* p, int64_t rows, int32_t d, int64_t ld) {
    const int64_t eb = dtype == LORA_BF16 ? 2 : 4;
    return RowSpan::matrix(p, rows, d * eb, ld, eb);
}
RowSpan choices_span(const void* p, int32_t T, int32_t k) { return RowSpan::array(p, (int64_t)T * k * 4); }

// Workgroups for 8 columns a thread.
int64_t columns_grid(int32_t T, int32_t d) { return ((int64_t)T * (d / 8) + kThreads - 1) / kThreads; }

template <bool WEIGHTED>
int launch_combine(int dtype, const ExpertParams& p, hipStream_t st) {
    const dim3 grid((unsigned)columns_grid(p.T, p.d)), block(kThreads);
    if (dtype == LORA_BF16)
        hipLaunchKernelGGL((expert_combine_kernel<LORA_BF16, WEIGHTED>), grid, block, 0, st, p);
    else
        hipLaunchKernelGGL((expert_combine_kernel<LORA_F32, WEIGHTED>), grid, block, 0, st, p);
    return hipGetLastError() == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

// Waves that take a token of the combine's gradient (the kernel has the figures), and
// workgroups for all of them.
int backward_waves(int32_t T, int32_t d) { return T < 1024 || d >= 2048 ? 4 : 1; }
int64_t backward_grid(int32_t T, int32_t d) {
    const int per = kThreads / kWave / backward_waves(T, d);
    return ((int64_t)T + per - 1) / per;
}
template <int DT>
void launch_backward(const ExpertParams& p, hipStream_t st) {
    const dim3 grid((unsigned)backward_grid(p.T, p.d)), block(kThreads);
    if (backward_waves(p.T, p.d) == 4)
        hipLaunchKernelGGL((expert_combine_backward_kernel<DT, 4>), grid, block, 0, st, p);
    else
        hipLaunchKernelGGL((expert_combine_backward_kernel<DT, 1>), grid, block, 0, st, p);
}

}  // namespace

extern "C" int lora_expert_gather(int dtype, const void* x, int64_t ldx, int32_t T, int32_t d, int32_t k, const int32_t* pos, void* y,
                                  int64_t ldy, void* stream) {
    int rc = check_expert(dtype, T, d, k, pos);
    if (rc != LORA_OK || T == 0) return rc;
    rc = check_matrix(x, d, ldx);
    if (rc == LORA_OK) rc = check_matrix(y, d, ldy);
    if (rc != LORA_OK) return rc;
    if (!grid_fits(columns_grid(T, d), kThreads)) return LORA_ERR_UNSUPPORTED;
    const RowSpan out = rows_span(dtype, y, (int64_t)T * k, d, ldy);
    if (shares_memory(out, rows_span(dtype, x, T, d, ldx)) || shares_memory(out, choices_span(pos, T, k))) return LORA_ERR_INVALID_ARG;
    ExpertParams p{};
    p.x = static_cast<const char*>(x);
    p.ldx = ldx;
    p.y = static_cast<char*>(y);
    p.ldy = ldy;
    p.pos = pos;
    p.T = T;
    p.d = d;
    p.k = k;
    const dim3 grid((unsigned)columns_grid(T, d)), block(kThreads);
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (dtype == LORA_BF16)
        hipLaunchKernelGGL(expert_gather_kernel<LORA_BF16>, grid, block, 0, st, p);
    else
        hipLaunchKernelGGL(expert_gather_kernel<LORA_F32>, grid, block, 0, st, p);
    return hipGetLastError() == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

namespace {
int combine(int dtype, const void* o, int64_t ldo, int32_t T, int32_t d, int32_t k, const int32_t* pos, const float* w, bool weighted,
            void* y, int64_t ldy, int32_t accumulate, void* stream) {
    int rc = check_expert(dtype, T, d, k, pos);
    if (rc == LORA_OK && accumulate != 0 && accumulate != 1) rc = LORA_ERR_INVALID_ARG;
    if (rc != LORA_OK || T == 0) return rc;
    if (weighted && !valid_f32(w)) return LORA_ERR_INVALID_ARG;
    rc = check_matrix(o, d, ldo);
    if (rc == LORA_OK) rc = check_matrix(y, d, ldy);
    if (rc != LORA_OK) return rc;
    if (!grid_fits(columns_grid(T, d), kThreads)) return LORA_ERR_UNSUPPORTED;
    const RowSpan out = rows_span(dtype, y, T, d, ldy);
    if (shares_memory(out, rows_span(dtype, o, (int64_t)T * k, d, ldo)) || shares_memory(out, choices_span(pos, T, k)) ||
        (weighted && shares_memory(out, choices_span(w, T, k))))
        return LORA_ERR_INVALID_ARG;
    ExpertParams p{};
    p.o = static_cast<const char*>(o);
    p.ldo = ldo;
    p.y = static_cast<char*>(y);
    p.ldy = ldy;
    p.pos = pos;
    p.w = w;
    p.T = T;
    p.d = d;
    p.k = k;
    p.accumulate = accumulate;
    hipStream_t st = static_cast<hipStream_t>(stream);
    return weighted ? launch_combine<true>(dtype, p, st) : launch_combine<false>(dtype, p, st);
}
}  // namespace

extern "C" int lora_expert_gather_backward(int dtype, const void* dy, int64_t lddy, int32_t T, int32_t d, int32_t k, const int32_t* pos,
                                           void* dx, int64_t lddx, int32_t accumulate, void* stream) {
    return combine(dtype, dy, lddy, T, d, k, pos, nullptr, false, dx, lddx, accumulate, stream);
}

extern "C" int lora_expert_combine(int dtype, const void* o, int64_t ldo, int32_t T, int32_t d, int32_t k, const int32_t* pos,
                                   const float* w, void* y, int64_t ldy, int32_t accumulate, void* stream) {
    return combine(dtype, o, ldo, T, d, k, pos, w, true, y, ldy, accumulate, stream);
}

extern "C" int lora_expert_combine_backward(int dtype, const void* dy, int64_t lddy, const void* o, int64_t ldo, int32_t T, int32_t d,
                                            int32_t k, const int32_t* pos, const float* w, void* d_o, int64_t lddo, float* dw,
                                            void* stream) {
    int rc = check_expert(dtype, T, d, k, pos);
    if (rc != LORA_OK || T == 0) return rc;
    if (!valid_f32(w) || (dw && !valid_f32(dw)) || (!d_o && !dw)) return LORA_ERR_INVALID_ARG;
    rc = check_matrix(dy, d, lddy);
    if (rc == LORA_OK && dw) rc = check_matrix(o, d, ldo);
    if (rc == LORA_OK && d_o) rc = check_matrix(d_o, d, lddo);
    if (rc != LORA_OK) return rc;
    if (!grid_fits(backward_grid(T, d), kThreads)) return LORA_ERR_UNSUPPORTED;
    const RowSpan in_dy = rows_span(dtype, dy, T, d, lddy), in_o = rows_span(dtype, o, (int64_t)T * k, d, ldo);
    const RowSpan in_w = choices_span(w, T, k), in_pos = choices_span(pos, T, k);
    const RowSpan out_o = rows_span(dtype, d_o, (int64_t)T * k, d, lddo), out_w = choices_span(dw, T, k);
    // (rows in place are read before they are written, if they are the same rows)
    const bool in_place = d_o == o && (lddo == ldo || (int64_t)T * k == 1);
    if (d_o && (shares_memory(out_o, in_dy) || shares_memory(out_o, in_w) || shares_memory(out_o, in_pos) ||
                (dw && !in_place && shares_memory(out_o, in_o)) || (dw && shares_memory(out_o, out_w))))
        return LORA_ERR_INVALID_ARG;
    if (dw && (shares_memory(out_w, in_dy) || shares_memory(out_w, in_o) || shares_memory(out_w, in_w) || shares_memory(out_w, in_pos)))
        return LORA_ERR_INVALID_ARG;
    ExpertParams p{};
    p.x = static_cast<const char*>(dy);
    p.ldx = lddy;
    p.o = static_cast<const char*>(o);
    p.ldo = ldo;
    p.y = static_cast<char*>(d_o);
    p.ldy = lddo;
    p.pos = pos;
    p.w = w;
    p.dw = dw;
    p.T = T;
    p.d = d;
    p.k = k;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (dtype == LORA_BF16)
        launch_backward<LORA_BF16>(p, st);
    else
        launch_backward<LORA_F32>(p, st);
    return hipGetLastError() == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}
