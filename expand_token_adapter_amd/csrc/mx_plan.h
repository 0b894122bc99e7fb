// mx_plan.h -- which kernel, tile and split of k a product with a 4-bit weight takes,
// and the LDS of a tile (host and device, no HIP).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "base_plan.h"

namespace lora {

// A step along k of a tile kernel, by the bits of the activation rows: 128 bytes of
// an activation row.
constexpr int mx_step(int bits) { return bits == 4 ? 256 : 128; }

template <int BN, int BT, int ST, int XB>
struct MxLds {
    static constexpr int kStep = mx_step(XB);
    static constexpr int kRowW = kStep / 2, kRowX = 128;           // bytes of a row's step
    static constexpr int kWordsW = kStep / 128;                    // words of scales of a weight row's step
    static constexpr int kWordsX = XB == 4 ? 2 : 1;
    static constexpr int kStage = BN * kRowW + BT * kRowX;
    static constexpr int kChunksW = (BN * kWordsW + 63) / 64, kChunksX = (BT * kWordsX + 63) / 64;  // loads of 64 words
    static constexpr int kScales = (kChunksW + kChunksX) * 256;
    static constexpr int kBytes = ST * kStage + (ST + 1) * kScales;
    static_assert(kBytes <= kLdsBytes, "a CU's LDS");
};

enum { kMxStream = 0, kMx32x64, kMx64x64, kMx64x128, kMx128x128, kMx256x128, kMx256x256, kMxKinds };
struct MxTile {
    int32_t bn, bt;
    int32_t stages4, stages8;  // of the ring in LDS, for 4-bit and 8-bit rows
    int32_t threads;           // of a workgroup, at most
    // us of a workgroup: its start and end, 256 columns of k for 4-bit rows, for 8-bit rows with bf16 y and fp32 y
    float start, step4, step8, step8_f32;
};
constexpr MxTile kMxTiles[kMxKinds] = {{0, 0, 0, 0, 0, 0.f, 0.f, 0.f, 0.f},
                                       {32, 64, 6, 6, 256, 0.5f, 0.151f, 0.25f, 0.5f},
                                       {64, 64, 4, 6, 256, 0.85f, 0.198f, 0.35f, 0.55f},
                                       {64, 128, 4, 4, 256, 1.2f, 0.351f, 0.60f, 1.1f},
                                       {128, 128, 3, 4, 256, 2.4f, 0.45f, 0.75f, 1.6f},
                                       {256, 128, 3, 4, 256, 3.5f, 0.677f, 1.2f, 3.f},
                                       {256, 256, 2, 3, 512, 3.1f, 1.122f, 2.1f, 5.8f}};
constexpr int kMxStreamWaves = 8;

// bits: of the activation rows.  kind: kMxKinds if no kernel's launch holds the call.
inline BasePlan mx_plan(int bits, int dtype, int64_t T, int64_t k, int64_t N) {
    const int32_t steps = (int32_t)((k + 255) / 256);
    const float outputs = (float)T * (float)N;
    BasePlan best{kMxKinds, 1};
    float least = 0.f;
    for (int kind = kMx32x64; kind < kMxKinds; ++kind) {
        const MxTile& c = kMxTiles[kind];
        const float step = bits == 4 ? c.step4 : dtype == LORA_BF16 ? c.step8 : c.step8_f32;
        const int64_t tiles = (int64_t)(((uint32_t)N + c.bn - 1) / c.bn) * (((uint32_t)T + c.bt - 1) / c.bt);
        for (const int32_t s : kSplits) {
            if (s > 1 && (s > steps || tiles * s > 2 * kCus)) break;
            if (!grid_fits(tiles * s + 8, c.threads)) break;  // (rounded up to the XCDs)
            const float rounds = (float)((uint64_t)(tiles * s + kCus - 1) / kCus);
            float us = rounds * (c.start + (float)((steps + s - 1) / s) * step);
            if (s > 1) us += 2.5f + (float)s * (0.14f + outputs * 0.97e-6f);
            if (least == 0.f || us < least) {
                least = us;
                best = BasePlan{kind, s};
            }
        }
    }
    if (T <= kStreamRows && grid_fits((N + 15) / 16, kMxStreamWaves * 64) &&
        (float)steps * (0.2f + 0.003f * (float)(T - 1)) + (float)N * (float)k / 50e6f < least)
        best = BasePlan{kMxStream, 1};
    return best;
}

// Rows of a tile kind (the stream's tiles hold one operand's rows).
constexpr int32_t mx_tile_rows(int kind) { return kind == kMxStream ? kStreamRows : kMxTiles[kind].bt; }

// The experts' product of T rows over `experts` weights: how many rows each has is known
// on the device only, so the choice goes by the mean.  *tiles_t: tiles along t, at most.
inline BasePlan mx_expert_plan(int bits, int dtype, int64_t T, int64_t k, int64_t N, int64_t experts, int64_t* tiles_t) {
    const int32_t steps = (int32_t)((k + 255) / 256);
    const int64_t used = std::min(T, experts), mean = (T + used - 1) / used;
    BasePlan best{kMxKinds, 1};
    float least = 0.f;
    for (int kind = kMxStream; kind < kMxKinds; ++kind) {
        const MxTile& c = kMxTiles[kind];
        const int32_t bt = mx_tile_rows(kind);
        const int64_t most = T / bt + used, tiles_n = (N + (kind == kMxStream ? 16 : c.bn) - 1) / (kind == kMxStream ? 16 : c.bn);
        if (!grid_fits(most * tiles_n + 8, kind == kMxStream ? kMxStreamWaves * 64 : c.threads)) continue;
        float us;
        if (kind == kMxStream) {
            us = (float)(tiles_n * used * ((mean + bt - 1) / bt)) / (float)(kCus * 2) * (1.f + 0.12f * (float)steps);
        } else {
            const float step = bits == 4 ? c.step4 : dtype == LORA_BF16 ? c.step8 : c.step8_f32;
            const int64_t tiles = tiles_n * used * ((mean + bt - 1) / bt);
            us = (float)((tiles + kCus - 1) / kCus) * (c.start + (float)steps * step);
        }
        if (best.kind == kMxKinds || us < least) {
            least = us;
            best = BasePlan{kind, 1};
            *tiles_t = most;
        }
    }
    return best;
}

}  // namespace lora
