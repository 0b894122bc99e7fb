// base.hip -- lora_base_product entry point (base_plan.h chooses the kernel).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "base.h"

using namespace lora;

namespace {

// WN x WT waves a workgroup
template <int DT, int KIND, int WN, int WT>
void launch_tiles(const BaseParams& p, unsigned grid, hipStream_t st) {
    constexpr BaseTile c = kTiles[KIND];
    static_assert(WN * WT * kWave <= c.threads, "the plan's bound on the launch");
    hipLaunchKernelGGL((base_kernel<c.bn, c.bt, WN, WT, c.stages, DT>), dim3(grid), dim3(WN * WT * kWave), 0, st, p);
}

template <int DT>
int launch_base(BaseParams p, const BasePlan& b, hipStream_t st) {
    p.splits = b.splits;
    if (b.kind == kStream) {
        hipLaunchKernelGGL((base_stream_kernel<kStreamWaves, DT>), dim3((unsigned)((p.N + 15) / 16)),
                           dim3(kStreamWaves * kWave), 0, st, p);
        return hipGetLastError() == hipSuccess ? LORA_OK : LORA_ERR_HIP;
    }
    const BaseTile& c = kTiles[b.kind];
    p.tiles_n = (p.N + c.bn - 1) / c.bn;
    p.tiles_t = (p.T + c.bt - 1) / c.bt;
    const unsigned grid = (unsigned)round_up((int64_t)p.tiles_n * p.tiles_t * p.splits, kNumXcd);
    switch (b.kind) {
        case kTile32x64: launch_tiles<DT, kTile32x64, 1, 4>(p, grid, st); break;
        case kTile64x64: launch_tiles<DT, kTile64x64, 2, 2>(p, grid, st); break;
        case kTile64x128: launch_tiles<DT, kTile64x128, 2, 2>(p, grid, st); break;
        case kTile128x128: launch_tiles<DT, kTile128x128, 2, 2>(p, grid, st); break;
        case kTile256x128: launch_tiles<DT, kTile256x128, 2, 2>(p, grid, st); break;
        // eight waves, or for fp32 y four (6783 x 4096 x 14336: 307 against 320 us, fp32 588 against 610)
        default: launch_tiles<DT, kTile256x256, 2, DT == LORA_BF16 ? 4 : 2>(p, grid, st); break;
    }
    if (hipGetLastError() != hipSuccess) return LORA_ERR_HIP;
    if (p.splits > 1) {
        const int64_t q = (int64_t)p.T * (p.N / 4);
        const unsigned sum_grid = (unsigned)std::min<int64_t>((q + kSumThreads - 1) / kSumThreads, kCus * 8);
        hipLaunchKernelGGL(base_sum_kernel<DT>, dim3(sum_grid), dim3(kSumThreads), 0, st, p);
    }
    return hipGetLastError() == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

}  // namespace

extern "C" size_t lora_base_product_workspace_bytes(int32_t T, int32_t d_in, int32_t d_out) {
    if (T < 0 || d_in < 1 || d_out < 1) return 0;
    if (T == 0) return 16;
    return std::max(base_workspace_bytes(base_plan(LORA_BF16, T, d_in, d_out), T, d_out),
                    base_workspace_bytes(base_plan(LORA_F32, T, d_in, d_out), T, d_out));
}

extern "C" int lora_base_product(int dtype, lora_quant x, int32_t T, int32_t d_in, lora_quant w, int32_t d_out, void* y,
                                 int64_t ldy, int32_t accumulate, void* ws, size_t ws_bytes, void* stream) {
    if (!valid_dtype(dtype) || T < 0 || d_in < 1 || d_out < 1 || (accumulate != 0 && accumulate != 1))
        return LORA_ERR_INVALID_ARG;
    if (T == 0) return LORA_OK;
    int rc = check_quant(x, d_in);
    if (rc == LORA_OK) rc = check_quant(w, d_in);
    if (rc == LORA_OK) rc = check_matrix(y, d_out, ldy);
    if (rc != LORA_OK) return rc;
    // a tile's 256 rows are addressed with 32-bit byte offsets, rows and outputs numbered in 32 bits
    if (x.ld > LORA_QUANT_MAX_LD || w.ld > LORA_QUANT_MAX_LD || T > INT32_MAX - 256 || d_out > INT32_MAX - 256)
        return LORA_ERR_UNSUPPORTED;
    const BasePlan b = base_plan(dtype, T, d_in, d_out);
    if (b.kind == kKinds) return LORA_ERR_UNSUPPORTED;
    if (!ws || !aligned16(ws) || ws_bytes < base_workspace_bytes(b, T, d_out)) return LORA_ERR_WORKSPACE;
    BaseParams p{};
    p.x = x.codes;
    p.ldx = x.ld;
    p.xs = x.scales;
    p.ldxs = x.lds;
    p.w = w.codes;
    p.ldw = w.ld;
    p.ws = w.scales;
    p.ldws = w.lds;
    p.y = static_cast<char*>(y);
    p.ldy = ldy;
    p.T = T;
    p.N = d_out;
    p.nkb = (d_in + kQBlock - 1) / kQBlock;
    p.accumulate = accumulate;
    p.part = static_cast<float*>(ws);
    hipStream_t st = static_cast<hipStream_t>(stream);
    return dtype == LORA_BF16 ? launch_base<LORA_BF16>(p, b, st) : launch_base<LORA_F32>(p, b, st);
}
