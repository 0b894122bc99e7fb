// base_plan.h -- which kernel, tile and split of k a lora_base_product takes, and
// the LDS of a tile (host and device, no HIP).
//
// The choice goes by a model of the call's time.  A tile kernel's workgroups take
// rounds of one per CU, a round its steps along k; small tiles fill the chip, large
// ones load less per product.  Measured (us, bf16 y; rows x k x outputs):
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
// random shapes (1 to 6755 rows, k 256 to 14336, 256 to 4096 outputs, both types):
// 1.1% in the mean, 1.2% with 298 more.  They rank choices; the times of the largest
// products are too low (2048 x 14336 x 4096 79 us for 107, 6783 x 4096 x 14336 234
// for 307).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "host_checks.h"

namespace lora {

constexpr int kLdsBytes = 160 * 1024;  // of a CU

template <int BN, int BT, int ST>
struct BaseLds {
    static constexpr int kStage = (BN + BT) * LORA_QUANT_BLOCK;
    static constexpr int kNB = BN > LORA_QUANT_BLOCK ? BN / LORA_QUANT_BLOCK : 1;  // 128-row blocks of the weight tile
    static constexpr int kWeight = kNB * 64 * 4;                 // bytes of the weight's scale words
    static constexpr int kFit = (kLdsBytes - ST * kStage - kWeight) / (BT * 4);
    static constexpr int kGroups = kFit < 32 ? kFit : 32;
    static constexpr int kBytes = ST * kStage + kWeight + kGroups * BT * 4;
    static_assert(kGroups >= 8, "room for the scales of 4096 columns");
};

constexpr int kCus = 256;
enum { kStream = 0, kTile32x64, kTile64x64, kTile64x128, kTile128x128, kTile256x128, kTile256x256, kKinds };
struct BaseTile {
    int32_t bn, bt, stages;       // outputs, rows, stages of the ring in LDS
    int32_t threads;              // of a workgroup, at most
    float start, step, step_f32;  // us of a workgroup: its start and end, a step along k (bf16, fp32 y)
};
constexpr BaseTile kTiles[kKinds] = {{0, 0, 0, 0, 0.f, 0.f, 0.f},             {32, 64, 6, 256, 0.5f, 0.151f, 0.289f},
                                     {64, 64, 4, 256, 0.85f, 0.198f, 0.306f},  {64, 128, 4, 256, 1.2f, 0.351f, 0.58f},
                                     {128, 128, 3, 256, 2.4f, 0.45f, 0.81f},  {256, 128, 2, 256, 3.5f, 0.677f, 1.518f},
                                     {256, 256, 2, 512, 3.1f, 1.122f, 2.93f}};
// Parts of k, from 2 on no more than 1.63 apart.  Mean loss over the 965 shapes 1.2%;
// with powers of two alone 1.9%, with 5, 10 and 20 too 1.0%.
constexpr int32_t kSplits[] = {1, 2, 3, 4, 6, 8, 13, 16, 25, 32};
constexpr int kStreamRows = 16;  // one operand's rows
constexpr int kStreamWaves = 8;

struct BasePlan {
    int kind;
    int32_t splits;
};

// kind: kKinds if no kernel's launch holds the call.
inline BasePlan base_plan(int dtype, int64_t T, int64_t k, int64_t N) {
    const int32_t nkb = (int32_t)((k + LORA_QUANT_BLOCK - 1) / LORA_QUANT_BLOCK), groups = (nkb + 3) / 4;
    const float outputs = (float)T * (float)N;
    BasePlan best{kKinds, 1};
    float least = 0.f;
    for (int kind = kTile32x64; kind < kKinds; ++kind) {
        const BaseTile& c = kTiles[kind];
        const float step = dtype == LORA_BF16 ? c.step : c.step_f32;
        const int64_t tiles = (int64_t)(((uint32_t)N + c.bn - 1) / c.bn) * (((uint32_t)T + c.bt - 1) / c.bt);
        for (const int32_t s : kSplits) {
            if (s > 1 && (s > groups || tiles * s > 2 * kCus)) break;
            if (!grid_fits(tiles * s + 8, c.threads)) break;  // (rounded up to the XCDs)
            const float rounds = (float)((uint64_t)(tiles * s + kCus - 1) / kCus);
            float us = rounds * (c.start + (float)std::min(4 * ((groups + s - 1) / s), nkb) * step);
            if (s > 1) us += 2.5f + (float)s * (0.14f + outputs * 0.97e-6f);
            if (least == 0.f || us < least) {
                least = us;
                best = BasePlan{kind, s};
            }
        }
    }
    if (T <= kStreamRows && grid_fits((N + 15) / 16, kStreamWaves * 64) &&
        (float)nkb * (0.14f + 0.0017f * (float)(T - 1)) + (float)N * (float)k / 29e6f - 0.7f < least)
        best = BasePlan{kStream, 1};
    return best;
}

// (a split k has no more than 2 kCus workgroups, of 256 x 256 sums at most)
static_assert(LORA_BASE_PRODUCT_MAX_WORKSPACE >= 2 * kCus * 256 * 256 * (int)sizeof(float), "every plan fits");
inline size_t base_workspace_bytes(const BasePlan& b, int64_t T, int64_t N) {
    return b.splits > 1 ? (size_t)b.splits * (size_t)T * (size_t)N * sizeof(float) : 16;
}

}  // namespace lora
