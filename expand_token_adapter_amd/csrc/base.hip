// base.hip -- lora_base_product entry point.
#include <hip/hip_runtime.h>

#include "base.h"

using namespace lora;

namespace {

template <int BN, int BT, int WN, int WT, int ST>
int launch_base(int dtype, BaseParams p, hipStream_t st) {
    p.tiles_n = (p.N + BN - 1) / BN;
    p.tiles_t = (p.T + BT - 1) / BT;
    const int64_t tiles = (int64_t)p.tiles_n * p.tiles_t;
    if (tiles > INT32_MAX - 8) return LORA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)round_up(tiles, kNumXcd)), block(WN * WT * kWave);
    if (dtype == LORA_BF16)
        hipLaunchKernelGGL((base_kernel<BN, BT, WN, WT, ST, LORA_BF16>), grid, block, 0, st, p);
    else
        hipLaunchKernelGGL((base_kernel<BN, BT, WN, WT, ST, LORA_F32>), grid, block, 0, st, p);
    return hipGetLastError() == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

}  // namespace

extern "C" size_t lora_base_product_workspace_bytes(int32_t T, int32_t d_in, int32_t d_out) {
    if (T < 0 || d_in < 1 || d_out < 1) return 0;
    return 16;
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
    // a tile's 256 rows are addressed with 32-bit byte offsets
    if (x.ld > LORA_QUANT_MAX_LD || w.ld > LORA_QUANT_MAX_LD) return LORA_ERR_UNSUPPORTED;
    if (!ws || !aligned16(ws) || ws_bytes < lora_base_product_workspace_bytes(T, d_in, d_out)) return LORA_ERR_WORKSPACE;
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
    return launch_base<64, 64, 2, 2, 4>(dtype, p, static_cast<hipStream_t>(stream));
}
