// mx_base.hip -- lora_base_product_mx and lora_expert_product_mx (mx_plan.h chooses the
// kernel).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "mx_base.h"

using namespace lora;

namespace {

// WN x WT waves a workgroup
template <int XB, int DT, bool HALVES, int KIND, int WN, int WT>
void launch_tiles(const MxParams& p, unsigned grid, hipStream_t st) {
    constexpr MxTile c = kMxTiles[KIND];
    static_assert(WN * WT == mx_waves(KIND, XB, mx_sums(XB, DT, !HALVES)), "the plan's bound on the launch");
    hipLaunchKernelGGL((mx_kernel<c.bn, c.bt, WN, WT, XB == 4 ? c.stages4 : c.stages8, XB, DT, HALVES>), dim3(grid),
                       dim3(WN * WT * kWave), 0, st, p);
}
template <int XB, int DT, bool HALVES, int KIND>
void launch_stream(const MxParams& p, unsigned grid, hipStream_t st) {
    constexpr MxTile c = kMxTiles[KIND];
    hipLaunchKernelGGL((mx_stream_kernel<c.waves, c.bn / 16, c.bt / 16, XB, DT, HALVES>), dim3(grid),
                       dim3(c.waves * kWave), 0, st, p);
}

// tiles_t: tiles along t of all weights, at most
template <int XB, int DT, bool HALVES>
int launch_mx(MxParams p, const BasePlan& b, int64_t tiles_t, hipStream_t st) {
    p.splits = b.splits;
    const MxTile& c = kMxTiles[b.kind];
    p.tiles_n = (p.N + c.bn - 1) / c.bn;
    p.tiles_t = (int32_t)tiles_t;
    const unsigned grid = (unsigned)round_up(p.tiles_n * tiles_t * p.splits, kNumXcd);
    // Rows in halves: in the 64 x 64 tile no two waves share an activation row, whose codes
    // each would take apart (256 x 4096 x 4096 16.1 us in place of 18.7; in one piece 10.0
    // against 9.7; in the 64 x 32 tile 317 x 5128 x 1032 14.1 with two that share, 15.1
    // without); the larger ones have two waves on a SIMD, one to take codes apart while
    // the other multiplies (128 x 128 outputs x rows a tile: 256 x 4096 x 4096 30.3 -> 26.5 us,
    // 2048 x 14336 x 4096 204 -> 195; 256 x 128: 49.7 -> 44.2, 184 -> 175; in one piece
    // 119 -> 122, 103 -> 108).
    switch (b.kind) {
        case kMx64x32: launch_tiles<XB, DT, HALVES, kMx64x32, 2, 2>(p, grid, st); break;
        case kMx64x64: launch_tiles<XB, DT, HALVES, kMx64x64, HALVES ? 1 : 2, HALVES ? 4 : 2>(p, grid, st); break;
        case kMx128x128: launch_tiles<XB, DT, HALVES, kMx128x128, 2, HALVES ? 4 : 2>(p, grid, st); break;
        case kMx256x128: launch_tiles<XB, DT, HALVES, kMx256x128, 2, HALVES ? 4 : 2>(p, grid, st); break;
        case kMx256x256:
            if constexpr (mx_kind_on(kMx256x256, XB, mx_sums(XB, DT, !HALVES))) launch_tiles<XB, DT, HALVES, kMx256x256, 2, 4>(p, grid, st);
            break;
        case kMx16x16: launch_stream<XB, DT, HALVES, kMx16x16>(p, grid, st); break;
        default: launch_stream<XB, DT, HALVES, kMx32x16>(p, grid, st); break;
    }
    if (hipGetLastError() != hipSuccess) return LORA_ERR_HIP;
    if (p.splits > 1) {
        BaseParams q{};
        q.y = p.y;
        q.ldy = p.ldy;
        q.T = p.T;
        q.N = p.N;
        q.accumulate = p.accumulate;
        q.splits = p.splits;
        q.part = p.part;
        const int64_t n = (int64_t)p.T * (p.N / 4);
        const unsigned sum_grid = (unsigned)std::min<int64_t>((n + kSumThreads - 1) / kSumThreads, kCus * 8);
        hipLaunchKernelGGL(base_sum_kernel<DT>, dim3(sum_grid), dim3(kSumThreads), 0, st, q);
    }
    return hipGetLastError() == hipSuccess ? LORA_OK : LORA_ERR_HIP;
}

// The rows of a call: their bits, and whether products of 8-bit rows may be cut.
struct MxRowsArg {
    int bits;
    bool cut;
};
MxRowsArg rows_arg(int32_t x_bits) { return MxRowsArg{x_bits & ~LORA_MX_CUT, (x_bits & LORA_MX_CUT) != 0}; }

int launch(const MxParams& p, MxRowsArg x, int dtype, const BasePlan& b, int64_t tiles_t, void* stream) {
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (x.bits == 4)
        return dtype == LORA_BF16 ? launch_mx<4, LORA_BF16, false>(p, b, tiles_t, st) : launch_mx<4, LORA_F32, false>(p, b, tiles_t, st);
    if (x.cut) return launch_mx<8, LORA_BF16, false>(p, b, tiles_t, st);
    return dtype == LORA_BF16 ? launch_mx<8, LORA_BF16, true>(p, b, tiles_t, st) : launch_mx<8, LORA_F32, true>(p, b, tiles_t, st);
}

// What both products check; d_out: of one weight.
int check_product(int dtype, int32_t bits, const lora_quant& x, int32_t T, int32_t d_in, const lora_quant& w, int32_t d_out, const void* y,
                  int64_t ldy) {
    int rc = bits == 4 ? check_mx(x, d_in) : check_quant(x, d_in);
    if (rc == LORA_OK) rc = check_mx(w, d_in);
    if (rc == LORA_OK) rc = check_matrix(y, d_out, ldy);
    if (rc != LORA_OK) return rc;
    // a tile's 256 rows are addressed with 32-bit byte offsets, rows and outputs numbered in 32 bits
    if (x.ld > LORA_QUANT_MAX_LD || w.ld > LORA_QUANT_MAX_LD || x.lds > LORA_QUANT_MAX_LD || w.lds > LORA_QUANT_MAX_LD ||
        T > INT32_MAX - 256 || d_out > INT32_MAX - 256)
        return LORA_ERR_UNSUPPORTED;
    return LORA_OK;
}
bool valid_product(int dtype, MxRowsArg x, int32_t T, int32_t d_in, int32_t d_out, int32_t accumulate) {
    const bool rows = x.bits == 4 ? !x.cut : x.bits == 8 && (!x.cut || dtype == LORA_BF16);
    return valid_dtype(dtype) && rows && T >= 0 && d_in >= 1 && d_out >= 1 && (accumulate == 0 || accumulate == 1);
}
MxParams product_params(int32_t bits, const lora_quant& x, int32_t T, int32_t d_in, const lora_quant& w, int32_t d_out, void* y,
                        int64_t ldy, int32_t accumulate) {
    MxParams p{};
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
    p.steps = (int32_t)(((int64_t)d_in + mx_step(bits) - 1) / mx_step(bits));
    p.accumulate = accumulate;
    return p;
}

}  // namespace

extern "C" size_t lora_base_product_mx_workspace_bytes(int32_t T, int32_t d_in, int32_t d_out) {
    if (T < 0 || d_in < 1 || d_out < 1) return 0;
    if (T == 0) return 16;
    size_t most = 0;
    for (const int bits : {4, 8})
        for (const int dtype : {LORA_BF16, LORA_F32})
            most = std::max(most, base_workspace_bytes(mx_plan(bits, dtype, T, d_in, d_out), T, d_out));
    return most;
}

extern "C" int lora_base_product_mx(int dtype, int32_t x_bits, lora_quant x, int32_t T, int32_t d_in, lora_quant w, int32_t d_out, void* y,
                                    int64_t ldy, int32_t accumulate, void* ws, size_t ws_bytes, void* stream) {
    const MxRowsArg xa = rows_arg(x_bits);
    if (!valid_product(dtype, xa, T, d_in, d_out, accumulate)) return LORA_ERR_INVALID_ARG;
    if (T == 0) return LORA_OK;
    const int rc = check_product(dtype, xa.bits, x, T, d_in, w, d_out, y, ldy);
    if (rc != LORA_OK) return rc;
    const BasePlan b = mx_plan(xa.bits, mx_sums(xa.bits, dtype, xa.cut), T, d_in, d_out);
    if (b.kind == kMxKinds) return LORA_ERR_UNSUPPORTED;
    if (!ws || !aligned16(ws) || ws_bytes < base_workspace_bytes(b, T, d_out)) return LORA_ERR_WORKSPACE;
    MxParams p = product_params(xa.bits, x, T, d_in, w, d_out, y, ldy, accumulate);
    p.part = static_cast<float*>(ws);
    return launch(p, xa, dtype, b, (T + kMxTiles[b.kind].bt - 1) / kMxTiles[b.kind].bt, stream);
}

extern "C" int lora_expert_product_mx(int dtype, int32_t x_bits, lora_quant x, int32_t T, int32_t d_in, lora_quant w, int32_t num_experts,
                                      int32_t d_out, lora_segments seg, void* y, int64_t ldy, int32_t accumulate, void* stream) {
    const MxRowsArg xa = rows_arg(x_bits);
    if (!valid_product(dtype, xa, T, d_in, d_out, accumulate) || num_experts < 1) return LORA_ERR_INVALID_ARG;
    if (T == 0) return LORA_OK;
    if (!seg.offsets) return LORA_ERR_INVALID_ARG;
    const int rc = check_product(dtype, xa.bits, x, T, d_in, w, d_out, y, ldy);
    if (rc != LORA_OK) return rc;
    int64_t tiles_t = 0;
    const BasePlan b = mx_expert_plan(xa.bits, mx_sums(xa.bits, dtype, xa.cut), T, d_in, d_out, num_experts, &tiles_t);
    if (b.kind == kMxKinds) return LORA_ERR_UNSUPPORTED;
    const int64_t eb = dtype == LORA_BF16 ? 2 : 4, rows_w = (int64_t)num_experts * d_out;
    const int64_t col_x = xa.bits == 4 ? round_up(d_in, kMxPad) / 2 : round_up(d_in, kQBlock), col_w = round_up(d_in, kMxPad) / 2;
    const int64_t col_xs = xa.bits == 4 ? round_up(d_in, kMxPad) / kMxBlock : round_up(d_in, kQBlock) / kQBlock;
    const RowSpan out = RowSpan::matrix(y, T, d_out * eb, ldy, eb);
    if (shares_memory(out, RowSpan::matrix(x.codes, T, col_x, x.ld, 1)) || shares_memory(out, RowSpan::matrix(x.scales, T, col_xs, x.lds, 1)) ||
        shares_memory(out, RowSpan::matrix(w.codes, rows_w, col_w, w.ld, 1)) ||
        shares_memory(out, RowSpan::matrix(w.scales, rows_w, round_up(d_in, kMxPad) / kMxBlock, w.lds, 1)) ||
        shares_memory(out, RowSpan::array(seg.offsets, ((int64_t)num_experts + 1) * 4)))
        return LORA_ERR_INVALID_ARG;
    MxParams p = product_params(xa.bits, x, T, d_in, w, d_out, y, ldy, accumulate);
    p.offsets = seg.offsets;
    p.experts = num_experts;
    return launch(p, xa, dtype, b, tiles_t, stream);
}
