// mx_plan.h -- which kernel, tile and split of k a product with a 4-bit weight takes,
// and the LDS of a tile (host and device, no HIP).
//
// Measured (us, bf16 y, 4-bit rows / 8-bit rows with products cut; rows x k x outputs; the
// last two kernels read the weight straight into registers):
//                          64x32      64x64     128x128    256x128    256x256    16x16      32x16
//     1 x  4096 x  4096  5.4/6.9    6.4/7.9                                    3.4/3.7    4.6/4.8
//    16 x 14336 x  4096   13/19      15/20                                     9.7/12.8    13/16
//    32 x  4096 x  4096  5.6/7.2    6.6/8.2                                    6.7/8.7    5.7/6.8
//   128 x  4096 x  4096  6.2/8.3    7.2/9.3
//   256 x  4096 x  4096  9.1/13     7.9/9.8    13/16      19/26      28/40
//  1024 x  4096 x  4096   31/41      22/29     16/19      20/27      29/41
//  2048 x 14336 x  4096             121/189    77/104     64/89      88/120
//  6783 x  4096 x 14336             487/631   354/409    278/347    223/294
// (8-bit rows in two halves, fp32 y: 317 x 5128 x 1032 14.1 us with 64x32, 18 with
// 64x64, 256 x 4096 x 4096 16.1 with 64x64, 2048 x 14336 x 4096 174 and 6783 x 4096 x 14336
// 655 with 256x128.)
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "base_plan.h"

namespace lora {

// A step along k of a tile kernel, by the bits of the activation rows: 128 bytes of
// an activation row.
constexpr int mx_step(int bits) { return bits == 4 ? 256 : 128; }

// A row's scales are loaded for several steps at a time, since a load fetches a whole
// line of memory for each row however little of it is wanted: the words of kSpan steps,
// for a kSpan-th of the rows in each step.  They lie in a ring of three such spans: one
// that is read, one whose loads may be outstanding, and the one that the step ST later
// loads into.
template <int BN, int BT, int ST, int XB>
struct MxLds {
    static constexpr int kStep = mx_step(XB);
    static constexpr int kRowW = kStep / 2, kRowX = 128;  // bytes of a row's step
    static constexpr int kStage = BN * kRowW + BT * kRowX;
    static constexpr int kSlots = 3;
    static constexpr bool fits(int span) {
        return ST * kStage + kSlots * (BN * span * kStep / 128 + BT * (XB == 4 ? span * 2 : span / 4)) * 4 <= kLdsBytes;
    }
    static constexpr int kSpan = XB == 8 ? (fits(8) ? 8 : 4) : fits(4) ? 4 : 2;  // 1024 columns, or 512
    static_assert(ST <= kSpan, "a slot was last read before its first loads go out");
    static constexpr int kWordsW = kSpan * kStep / 128, kWordsX = XB == 4 ? kWordsW : kSpan / 4;  // of a row's span
    static constexpr int kAllW = BN * kWordsW / 64, kAllX = BT * kWordsX / 64;                  // loads of a span, 64 words each
    static constexpr int kLoadsW = kAllW / kSpan, kLoadsX = kAllX > kSpan ? kAllX / kSpan : 1;  // of a step
    static_assert(kAllW % kSpan == 0 && (kAllX % kSpan == 0 || kSpan % kAllX == 0), "the loads divide evenly");
    static constexpr int kScales = (kAllW + kAllX) * 256;
    static constexpr int kBytes = ST * kStage + kSlots * kScales;
    static_assert(kBytes <= kLdsBytes, "a CU's LDS");
};

// Kernels: tiles through LDS, and (from kMx16x16 on) tiles of waves side by side along k.
enum { kMx64x32 = 0, kMx64x64, kMx128x128, kMx256x128, kMx256x256, kMx16x16, kMx32x16, kMxKinds };
struct MxTile {
    int32_t bn, bt;            // outputs, rows
    int32_t stages4, stages8;  // of the ring in LDS, for 4-bit and 8-bit rows
    int32_t waves;             // of a workgroup (mx_waves)
    // us: a call's start and end, a workgroup's; a step of 256 columns (a piece of 512 of
    // every wave) for 4-bit rows, 8-bit rows with products cut, in halves; a step where several
    // workgroups share the CU (of all of them, or of each for the last two kernels)
    float start, tile, step[3], shared[3];
};
constexpr MxTile kMxTiles[kMxKinds] = {
    {64, 32, 4, 4, 4, 2.891f, 0.978f, {0.158f, 0.241f, 0.476f}, {0.437f, 0.402f, 0.746f}},
    {64, 64, 4, 4, 4, 2.496f, 1.365f, {0.217f, 0.315f, 0.749f}, {0.49f, 0.784f, 0.985f}},
    {128, 128, 4, 4, 4, 1.77f, 3.46f, {0.471f, 0.653f, 1.287f}, {0.f, 0.f, 0.f}},
    {256, 128, 2, 4, 4, 2.59f, 4.4f, {0.777f, 1.213f, 2.254f}, {0.f, 0.f, 0.f}},
    {256, 256, 2, 2, 8, 1.22f, 5.24f, {1.307f, 1.98f, 0.f}, {0.f, 0.f, 0.f}},
    {16, 16, 1, 1, 4, 2.312f, 0.278f, {0.639f, 0.545f, 0.991f}, {0.092f, 0.13f, 0.16f}},
    {32, 16, 1, 1, 4, 1.812f, 0.829f, {0.774f, 1.005f, 1.403f}, {0.156f, 0.182f, 0.223f}}};
// (8-bit rows in halves: the 256 x 256 tile's would not fit the registers)
constexpr bool mx_kind_on(int kind, int bits, int dtype) { return kind != kMx256x256 || bits == 4 || dtype == LORA_BF16; }
// What a choice goes by beside the rows' bits, `dtype` below: the type of y, for 8-bit rows
// that of a call that sums as this one does: LORA_F32 with the codes in halves, LORA_BF16
// with products that may be cut.
constexpr int mx_sums(int bits, int dtype, bool cut) { return bits == 4 ? dtype : cut ? LORA_BF16 : LORA_F32; }
// Waves of a workgroup: 8-bit rows in halves have two on a SIMD in the larger tiles
// (launch_mx has the figures).
constexpr int mx_waves(int kind, int bits, int dtype) {
    return bits == 8 && dtype == LORA_F32 && (kind == kMx128x128 || kind == kMx256x128) ? 8 : kMxTiles[kind].waves;
}

// Estimated us of a call of `tiles` tiles (not counting parts of k), `steps` steps of 256
// columns and s parts, after measurements of 1200 products and 800 experts' products of
// random sizes (1 to 6783 rows, k 256 to 14336, 256 to 14336 outputs, each kernel and
// split), and for the small kernels 900 and 500 more and 400 products of up to 64 rows: on
// those that the numbers were not fitted to, the choice is 0.4% slower than the best in the
// mean (few rows 0.6%; experts' products, whose rows are spread as the router likes, 2.4%;
// without the 64 x 32 tile 3.6% and experts' 7.7%).  The times rank choices; those of the
// largest products are too low (6783 x 4096 x 14336 158 us for 216, from 8-bit rows with
// products cut 223 for 282, in halves 488 for 578).
inline float mx_time(int kind, int bits, int dtype, int64_t tiles, int32_t steps, int32_t s, float outputs) {
    const MxTile& c = kMxTiles[kind];
    const int f = bits == 4 ? 0 : dtype == LORA_BF16 ? 1 : 2;
    const int64_t n = tiles * s;
    const float st = (float)(s == 1 ? steps : 4 * (((steps + 3) / 4 + s - 1) / s));
    float us = c.start;
    if (kind >= kMx16x16) {
        // (one workgroup's way through its k, or that of all that a CU has)
        const float alone = (float)(((steps + 1) / 2 + c.waves - 1) / c.waves) * c.step[f] + c.tile;
        us += std::max(alone, (float)((n + kCus - 1) / kCus) * (c.tile + st * c.shared[f]));
    } else if (kind <= kMx64x64) {  // two on a CU, or more
        const int64_t full = n / (2 * kCus), rest = n - full * 2 * kCus;
        us += (float)full * (c.tile + st * c.shared[f]);
        if (rest > 0) us += c.tile + st * (rest <= kCus ? c.step[f] : c.shared[f]);
    } else {
        us += (float)((n + kCus - 1) / kCus) * (c.tile + st * c.step[f]);
    }
    return s > 1 ? us + 2.03f + (float)s * (0.056f + outputs * 2.0e-6f) : us;
}

// bits: of the activation rows.  kind: kMxKinds if no kernel's launch holds the call.
inline BasePlan mx_plan(int bits, int dtype, int64_t T, int64_t k, int64_t N) {
    const int32_t steps = (int32_t)((k + 255) / 256);
    BasePlan best{kMxKinds, 1};
    float least = 0.f;
    for (int kind = 0; kind < kMxKinds; ++kind) {
        if (!mx_kind_on(kind, bits, dtype)) continue;
        const MxTile& c = kMxTiles[kind];
        const int64_t tiles = ((N + c.bn - 1) / c.bn) * ((T + c.bt - 1) / c.bt);
        for (const int32_t s : kSplits) {
            // (parts are of whole spans of scales, up to 1024 columns)
            if (s > 1 && (s > (steps + 3) / 4 || tiles * s > 2 * kCus || kind >= kMx16x16)) break;
            if (!grid_fits(tiles * s + 8, mx_waves(kind, bits, dtype) * 64)) break;  // (rounded up to the XCDs)
            const float us = mx_time(kind, bits, dtype, tiles, steps, s, (float)T * (float)N);
            if (best.kind == kMxKinds || us < least) {
                least = us;
                best = BasePlan{kind, s};
            }
        }
    }
    return best;
}

// The experts' product of T rows over `experts` weights: how many rows each has is known
// on the device only, so the choice goes by the mean, and half a tile more for each
// expert.  *tiles_t: tiles along t, at most.
inline BasePlan mx_expert_plan(int bits, int dtype, int64_t T, int64_t k, int64_t N, int64_t experts, int64_t* tiles_t) {
    const int32_t steps = (int32_t)((k + 255) / 256);
    const int64_t used = std::min(T, experts);
    BasePlan best{kMxKinds, 1};
    float least = 0.f;
    for (int kind = 0; kind < kMxKinds; ++kind) {
        if (!mx_kind_on(kind, bits, dtype)) continue;
        const MxTile& c = kMxTiles[kind];
        const int64_t most = T / c.bt + used, tiles_n = (N + c.bn - 1) / c.bn;
        if (!grid_fits(most * tiles_n + 8, mx_waves(kind, bits, dtype) * 64)) continue;
        const float each = std::max(1.f, (float)T / (float)(used * c.bt) + 0.5f);
        const float us = mx_time(kind, bits, dtype, (int64_t)((float)(tiles_n * used) * each), steps, 1, 0.f);
        if (best.kind == kMxKinds || us < least) {
            least = us;
            best = BasePlan{kind, 1};
            *tiles_t = most;
        }
    }
    return best;
}

// (a split k has no more than 2 kCus workgroups, of 256 x 256 sums at most)
static_assert(LORA_BASE_PRODUCT_MAX_WORKSPACE >= 2 * kCus * 256 * 256 * (int)sizeof(float), "every plan fits");

}  // namespace lora
