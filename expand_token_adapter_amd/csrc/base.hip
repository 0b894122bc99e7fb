// base.hip -- lora_base_product entry point.
//
// Which kernel, tile and split of k a call takes goes by a model of its time.
// A tile kernel's workgroups take rounds of one per CU, a round its steps along
// k; small tiles fill the chip, large ones load less per product.  Measured
// (us, bf16 y; rows x k x outputs):
//                     32x64  64x64  64x128 128x128 256x128 256x256
//    256 x  4096 x 4096  13.5    9.1    11.4    15.3    23.4    40.1
//   1024 x  4096 x 4096  49.2   27.3    23.8    18.5    24.1    41.5
//   2048 x  4096 x 4096  98.1   51.9    45.5    34.3    29.8    42.3
//   6783 x 4096 x 14336  1132    607     540     415     354     307
// Small tiles are bound by the loads into LDS (64x64: 16 KB a step in 0.17 us,
// 95 GB/s a CU), 256x256 by the matrix cores at the clock that they leave (2.6
// PFLOP/s; the library's product with one scale for each whole operand takes 291 us).
// Where the tiles leave CUs without work, k is split, for a second kernel that
// adds the parts: 16 x 14336 x 4096, 64x64: 31.6 us in one part, 16.9 in four.
// Up to 16 rows may take the weight as a stream instead: 1 x 4096 x 4096 5.8 us
// against 8.1 for the best tiles, but 1 x 12232 x 352 11.0 against 6.8 and
// 16 x 14336 x 4096 23 against 16.9.
// The model's numbers are those that lost least against the best choice for 667
// random shapes (1 to 6783 rows, k to 14336, 256 to 4096 outputs, both types): 1.1%
// in the mean.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "base.h"

using namespace lora;

namespace {

constexpr int kCus = 256;
enum { kStream = 0, kTile32x64, kTile64x64, kTile64x128, kTile128x128, kTile256x128, kTile256x256, kKinds };
struct BaseTile {
    int32_t bn, bt;
    float start, step, step_f32;  // us of a workgroup: its start and end, a step along k (bf16, fp32 y)
};
constexpr BaseTile kTiles[kKinds] = {{0, 0, 0.f, 0.f, 0.f},          {32, 64, 0.5f, 0.151f, 0.289f},
                                     {64, 64, 0.85f, 0.198f, 0.306f},  {64, 128, 1.2f, 0.351f, 0.58f},
                                     {128, 128, 2.4f, 0.45f, 0.81f},  {256, 128, 3.5f, 0.677f, 1.518f},
                                     {256, 256, 3.1f, 1.122f, 2.93f}};
constexpr int32_t kSplits[] = {1, 2, 3, 4, 6, 8, 13, 16, 25, 32};
constexpr int kStreamRows = 16;
constexpr int kStreamWaves = 8;

struct BasePlan {
    int kind;
    int32_t splits;
};

BasePlan base_plan(int dtype, int64_t T, int64_t k, int64_t N) {
    const int32_t nkb = (int32_t)((k + kQBlock - 1) / kQBlock), groups = (nkb + 3) / 4;
    const float outputs = (float)T * (float)N;
    BasePlan best{kTile64x64, 1};
    float least = 0.f;
    for (int kind = kTile32x64; kind < kKinds; ++kind) {
        const BaseTile& c = kTiles[kind];
        const float step = dtype == LORA_BF16 ? c.step : c.step_f32;
        const int64_t tiles = (int64_t)(((uint32_t)N + c.bn - 1) / c.bn) * (((uint32_t)T + c.bt - 1) / c.bt);
        for (const int32_t s : kSplits) {
            if (s > 1 && (s > groups || tiles * s > 2 * kCus)) break;
            const float rounds = (float)((uint64_t)(tiles * s + kCus - 1) / kCus);
            float us = rounds * (c.start + (float)std::min(4 * ((groups + s - 1) / s), nkb) * step);
            if (s > 1) us += 2.5f + (float)s * (0.14f + outputs * 0.97e-6f);
            if (least == 0.f || us < least) {
                least = us;
                best = BasePlan{kind, s};
            }
        }
    }
    if (T <= kStreamRows && (float)nkb * (0.14f + 0.0017f * (float)(T - 1)) + (float)N * (float)k / 29e6f - 0.7f < least)
        best = BasePlan{kStream, 1};
    return best;
}

// (a split k has no more than 2 kCus workgroups, of 256 x 256 sums at most)
static_assert(LORA_BASE_PRODUCT_MAX_WORKSPACE >= 2 * kCus * 256 * 256 * (int)sizeof(float), "every plan fits");
size_t workspace_bytes(const BasePlan& b, int64_t T, int64_t N) {
    return b.splits > 1 ? (size_t)b.splits * (size_t)T * (size_t)N * sizeof(float) : 16;
}

template <int DT, int BN, int BT, int WN, int WT, int ST>
void launch_tiles(const BaseParams& p, unsigned grid, hipStream_t st) {
    hipLaunchKernelGGL((base_kernel<BN, BT, WN, WT, ST, DT>), dim3(grid), dim3(WN * WT * kWave), 0, st, p);
}

template <int DT>
int launch_base(BaseParams p, const BasePlan& b, hipStream_t st) {
    p.splits = b.splits;
    if (b.kind == kStream) {
        hipLaunchKernelGGL((base_stream_kernel<kStreamRows / 16, kStreamWaves, DT>), dim3((unsigned)((p.N + 15) / 16)),
                           dim3(kStreamWaves * kWave), 0, st, p);
        return hipGetLastError() == hipSuccess ? LORA_OK : LORA_ERR_HIP;
    }
    const BaseTile& c = kTiles[b.kind];
    p.tiles_n = (p.N + c.bn - 1) / c.bn;
    p.tiles_t = (p.T + c.bt - 1) / c.bt;
    const int64_t tasks = (int64_t)p.tiles_n * p.tiles_t * p.splits;
    if (tasks > INT32_MAX - kNumXcd * kBand) return LORA_ERR_UNSUPPORTED;
    const unsigned grid = (unsigned)round_up(tasks, kNumXcd);
    switch (b.kind) {
        case kTile32x64: launch_tiles<DT, 32, 64, 1, 4, 6>(p, grid, st); break;
        case kTile64x64: launch_tiles<DT, 64, 64, 2, 2, 4>(p, grid, st); break;
        case kTile64x128: launch_tiles<DT, 64, 128, 2, 2, 4>(p, grid, st); break;
        case kTile128x128: launch_tiles<DT, 128, 128, 2, 2, 3>(p, grid, st); break;
        case kTile256x128: launch_tiles<DT, 256, 128, 2, 2, 2>(p, grid, st); break;
        // eight waves, or for fp32 y four (6783 x 4096 x 14336: 307 against 320 us, fp32 588 against 610)
        default: launch_tiles<DT, 256, 256, 2, DT == LORA_BF16 ? 4 : 2, 2>(p, grid, st); break;
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
    return std::max(workspace_bytes(base_plan(LORA_BF16, T, d_in, d_out), T, d_out),
                    workspace_bytes(base_plan(LORA_F32, T, d_in, d_out), T, d_out));
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
    if (!ws || !aligned16(ws) || ws_bytes < workspace_bytes(b, T, d_out)) return LORA_ERR_WORKSPACE;
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
