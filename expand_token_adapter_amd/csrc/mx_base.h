// mx_base.h -- products with a frozen 4-bit weight (gfx950).
//
//   y_t (+)= sum_k x_tk W_nk
//
// with W in the 4-bit form of mx.h and x in it or in the 8-bit form of quant.h; for
// a mixture of experts with a weight for each group of rows.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes 128 columns of 16 weight rows and 16
// activation rows.  Lane group g = lane / 16 of an operand in 4 bits holds columns
// 32 g .. 32 g + 31, one block with one scale; in 8 bits 16 g .. + 15 and 64 + 16 g
// .. + 15 (measured with one-hot operands; the scale of lane group g is that of
// columns 32 g .. 32 g + 31 in both, and 8-bit rows have the same for all of them).
//
// 4-bit rows: every product of two codes is a multiple of 1/4 up to 36, so the
// instruction, which keeps a group of 8 products down to 2^-13 of the largest one's
// power of two, cuts nothing, and its fp32 sums serve bf16 and fp32 y alike.  It
// runs at twice the rate of 8-bit operands.
// 8-bit rows: products of a group of 8 columns are cut as in base.h (measured: beside
// 4 * 256, 2^-3 is kept and 2^-4 lost, also in sevens; 0.5 * 256 counts as 1 * 256,
// as a subnormal 8-bit code counts as 2^-6).  bf16 y takes it: 1.5e-5 of a result on
// normal data.  fp32 y takes exact products of the values as bf16 numbers, as base.h
// does.
//
// A operand = weight rows (n), B operand = activation rows (t), blocks of weight rows
// in pairs so that a lane ends with eight consecutive n of one t, as in base.h.
#pragma once

#include "base.h"
#include "mx.h"
#include "mx_plan.h"

namespace lora {

struct MxParams {
    const uint8_t* x;
    int64_t ldx;
    const uint8_t* xs;
    int64_t ldxs;
    const uint8_t* w;
    int64_t ldw;
    const uint8_t* ws;
    int64_t ldws;
    char* y;
    int64_t ldy;
    int32_t T, N, steps;        // rows, outputs (of an expert), steps along k
    int32_t accumulate;
    int32_t tiles_n, tiles_t;   // (tiles_t: of one weight)
    int32_t splits;             // parts of k, each a workgroup's; more than one: fp32 sums to part
    float* part;                // [splits][T][N]
    const int32_t* offsets;     // experts' first rows [experts + 1], or NULL: one weight for all rows
    int32_t experts;
};

// ------------------------------------------------------------------ experts' tiles

// Rows lie sorted by expert, expert e's at offsets[e] .. offsets[e + 1] - 1, tiles of
// BT rows begin anew with each expert.  Every wave finds its tile from the offsets
// by itself: 64 experts at a time, a lane each.  (The offsets are read as they are
// on the device, so nothing waits for them on the host; rows outside [0, T) that bad
// offsets would name are left out.)
struct MxGroup {
    int first, rows;  // of the tile
    int expert;
};
// Tiles of this lane's expert e, and where its rows begin and end.
template <int BT>
__device__ __forceinline__ int mx_tiles_of(const MxParams& p, int e, int& begin, int& end) {
    begin = end = 0;
    if (e < p.experts) {
        begin = min(max(gptr(p.offsets)[e], 0), p.T);
        end = min(max(gptr(p.offsets)[e + 1], begin), p.T);
    }
    return (end - begin + BT - 1) / BT;
}
__device__ __forceinline__ int mx_scan(int v, int lane) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int o = __shfl_up(v, d, kWave);
        if (lane >= d) v += o;
    }
    return v;
}
template <int BT>
__device__ __forceinline__ int mx_total_tiles(const MxParams& p, int lane) {
    int total = 0;
    for (int e0 = 0; e0 < p.experts; e0 += kWave) {
        int b, e;
        total += __builtin_amdgcn_readlane(mx_scan(mx_tiles_of<BT>(p, e0 + lane, b, e), lane), kWave - 1);
    }
    return total;
}
// (tile below the total)
template <int BT>
__device__ __forceinline__ MxGroup mx_find_tile(const MxParams& p, int tile, int lane) {
    int before = 0;
    for (int e0 = 0; e0 < p.experts; e0 += kWave) {
        int b, e;
        const int n = mx_tiles_of<BT>(p, e0 + lane, b, e);
        const int incl = mx_scan(n, lane);
        const uint64_t past = __ballot(before + incl > tile);
        if (past) {
            const int at = __ffsll((long long)past) - 1;
            const int in = tile - before - __builtin_amdgcn_readlane(incl - n, at);
            const int begin = __builtin_amdgcn_readlane(b, at) + in * BT;
            return MxGroup{begin, min(BT, __builtin_amdgcn_readlane(e, at) - begin), e0 + at};
        }
        before += __builtin_amdgcn_readlane(incl, kWave - 1);
    }
    return MxGroup{0, 0, 0};
}

// ------------------------------------------------------------------ operands

// Whether a product's codes are decoded to bf16 numbers (XB: bits of the activation
// rows, DT: type of y).
template <int XB, int DT>
constexpr bool kMxDecode = XB == 8 && DT == LORA_F32;

// 32 4-bit codes as the matrix instruction's operand.
__device__ __forceinline__ i32x8_t mx_operand(u32x4_t q) { return i32x8_t{(int)q[0], (int)q[1], (int)q[2], (int)q[3], 0, 0, 0, 0}; }

// ------------------------------------------------------------------ tiles through LDS
//
// A workgroup of WN x WT waves computes BN outputs x BT rows.  A step is 256 columns
// of 4-bit rows or 128 of 8-bit rows, 128 bytes of an activation row; BN weight and
// BT activation rows' steps go from memory straight into LDS, ST stages in a ring,
// the step's scales into a ring of ST + 1.  The pieces of a step are handed over as
// in base.h: the weight blocks are taken two or four at a time, and after the barrier at the
// start of such a group its place is free for the step ST later, whose loads go out
// between the products.  Scales go out first: their slot was last read a step ago.
//
// 16-byte unit c of a row lies at position c ^ s of it: s is the operand row modulo 8
// for rows of 128 bytes, half of it modulo 4 for rows of 64 bytes, so that 8 lanes
// that a read takes together fall on different banks.
template <int BN, int BT, int WN, int WT, int ST, int XB, int DT>
__global__ __launch_bounds__(WN* WT* kWave) void mx_kernel(MxParams p) {
    using L = MxLds<BN, BT, ST, XB>;
    constexpr bool kDecode = kMxDecode<XB, DT>;
    constexpr int NW = WN * WT;
    constexpr int FN = BN / WN / 16, FT = BT / WT / 16;  // 16 x 16 blocks of a wave
    constexpr int SUB = XB == 4 ? 2 : 1;                 // instructions of a step and block
    constexpr int RW = 1024 / L::kRowW, RX = 1024 / L::kRowX;  // rows of a load
    // weight blocks of a group (so many that every wave has a load of its own), groups
    constexpr int GA = 32 * WN / RW < NW && FN % 4 == 0 ? 4 : 2, NG = FN / GA;
    // loads of a wave: for a weight group, for the activations, for the scales
    constexpr int GR = GA * 16 * WN;                     // weight rows of a group
    constexpr int WU = GR / RW >= NW ? GR / RW / NW : 1, XU = BT / RX / NW;
    constexpr int SU = (L::kChunksW + L::kChunksX + NW - 1) / NW;
    constexpr int PW = SU + NG * WU + XU;
    static_assert(FN % 2 == 0 && NG <= 4 && BT % (RX * NW) == 0, "the loads divide evenly");
    static_assert(GR / RW >= NW ? GR % (RW * NW) == 0 : NW % (GR / RW) == 0, "the weight's loads divide evenly");
    __shared__ __attribute__((aligned(16))) char s_lds[L::kBytes];
    char* s_sc = s_lds + ST * L::kStage;

    const int wave = wave_id();
    const int lane = threadIdx.x & (kWave - 1);
    const int lr = lane & 15, lg = lane >> 4;
    // Workgroups of one XCD take neighbouring tiles.
    const int tiles_t = p.offsets ? mx_total_tiles<BT>(p, lane) : p.tiles_t;
    const int ntile = p.tiles_n * tiles_t * p.splits;
    const int per = (ntile + kNumXcd - 1) / kNumXcd;
    const int task = (int)(blockIdx.x % kNumXcd) * per + (int)(blockIdx.x / kNumXcd);
    if ((int)(blockIdx.x / kNumXcd) >= per || task >= ntile) return;
    const int tile = task / p.splits, part = task - tile * p.splits;
    const int k0 = (int)((int64_t)p.steps * part / p.splits), k1 = (int)((int64_t)p.steps * (part + 1) / p.splits);
    // Order of the tiles: bands of up to kBand tiles along t, walked along n (base.h).
    const int band = tile / (kBand * p.tiles_n), in = tile - band * kBand * p.tiles_n;
    const int bt = min(kBand, tiles_t - band * kBand);
    const int n0 = in / bt * BN, tt = band * kBand + in % bt;
    MxGroup grp{tt * BT, 0, 0};
    if (p.offsets)
        grp = mx_find_tile<BT>(p, tt, lane);
    else
        grp.rows = min(BT, p.T - grp.first);
    const int t0 = grp.first, trows = grp.rows, nrows = min(BN, p.N - n0);
    const int wn = (wave % WN) * (BN / WN), wt = (wave / WN) * (BT / WT);

    // Rows past the tile lie past their buffer: nothing is fetched for them, and their
    // outputs are not stored.
    const int64_t wrow = (int64_t)grp.expert * p.N + n0;
    const buf_rsrc_t rw = make_rsrc(p.w + wrow * p.ldw, (uint32_t)((nrows - 1) * p.ldw + (int64_t)p.steps * L::kRowW));
    const buf_rsrc_t rx = make_rsrc(p.x + (int64_t)t0 * p.ldx, (uint32_t)((trows - 1) * p.ldx + (int64_t)p.steps * L::kRowX));
    const buf_rsrc_t rws = make_rsrc(p.ws + wrow * p.ldws, (uint32_t)((nrows - 1) * p.ldws + (int64_t)p.steps * L::kWordsW * 4));
    const buf_rsrc_t rxs = make_rsrc(p.xs + (int64_t)t0 * p.ldxs,
                                     (uint32_t)((trows - 1) * p.ldxs + (XB == 4 ? (int64_t)p.steps * 8 : (p.steps + 3) / 4 * 4)));
    // Load j of weight group g: row group (RW rows) c of the group's GR rows, in the
    // order wave column, row: rows 16 GA g .. 16 GA (g + 1) - 1 of every wave column.
    constexpr int LWR = 64 / RW;  // lanes of a weight row's step
    const int wr = lane / LWR;
    const int w_key = L::kRowW == 128 ? (wr & 3) : 2 * ((wr >> 3) & 1) + ((wr >> 1) & 1);
    const int x_r8 = lane >> 3;
    const uint32_t vx = (uint32_t)((8 * wave + x_r8) * p.ldx) + (uint32_t)((lane & 7) ^ x_r8) * 16u;
    auto issue_w = [&](int g, int j, int slot, int kb) {
        constexpr int CPG = 16 * GA / RW;                  // loads of a wave column's group
        const int c = (wave + NW * j) % (CPG * WN);        // (a wave without one repeats another's)
        const int row = c / CPG * (BN / WN) + 16 * GA * g + c % CPG * RW;
        // (rows of 128 bytes: a load is 8 rows, and the next 8 have the other half of the keys)
        const int key = L::kRowW == 128 ? w_key ^ ((c & 1) * 4) : w_key;
        const uint32_t v = (uint32_t)((row + wr) * p.ldw) + (uint32_t)((lane % LWR) ^ key) * 16u;
        dma_lds(rw, v, (uint32_t)kb * L::kRowW, s_lds + slot * L::kStage + row * L::kRowW, 16);
    };
    auto issue_x = [&](int j, int slot, int kb) {
        dma_lds(rx, vx + (uint32_t)(8 * NW * j * p.ldx), (uint32_t)kb * L::kRowX,
                s_lds + slot * L::kStage + BN * L::kRowW + (8 * wave + 8 * NW * j) * L::kRowX, 16);
    };
    auto issue_s = [&](int j, int sslot, int kb) {
        const int c = (wave + NW * j) % (L::kChunksW + L::kChunksX);
        char* at = s_sc + sslot * L::kScales + c * 256;
        if (c < L::kChunksW) {
            const int word = 64 * c + lane;
            dma_lds(rws, (uint32_t)((word / L::kWordsW) * p.ldws) + (uint32_t)(word % L::kWordsW) * 4u,
                    (uint32_t)kb * (L::kWordsW * 4), at, 4);
        } else {
            const int word = 64 * (c - L::kChunksW) + lane;
            dma_lds(rxs, (uint32_t)((word / L::kWordsX) * p.ldxs) + (uint32_t)(word % L::kWordsX) * 4u,
                    XB == 4 ? (uint32_t)kb * 8u : (uint32_t)kb & ~3u, at, 4);
        }
    };
    // Load o of a step: scales, weight group 0, activations, weight groups 1, 2, ...
    auto issue = [&](int o, int slot, int sslot, int kb) {
        if (o < SU)
            issue_s(o, sslot, kb);
        else if (o < SU + WU)
            issue_w(0, o - SU, slot, kb);
        else if (o < SU + WU + XU)
            issue_x(o - SU - WU, slot, kb);
        else
            issue_w((o - SU - XU) / WU, (o - SU - XU) % WU, slot, kb);
    };

    f32x4_t acc[FN][FT];
#pragma unroll
    for (int a = 0; a < FN; ++a)
#pragma unroll
        for (int b = 0; b < FT; ++b) acc[a][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // This lane's units of an operand row.  Weight row of operand row lr: 8 (lr / 4) +
    // lr % 4 of the pair of blocks, + 4 for its second block.
    const int lrow_w = (8 * (lr >> 2) + (lr & 3)) * L::kRowW + (L::kRowW == 128 ? (lg ^ (lr & 7)) * 16 : (lg ^ ((lr >> 1) & 3)) * 16);
    // 8-bit rows: units lg and lg + 4 (the instruction's columns), or 2 lg and 2 lg + 1
    // where the codes are decoded (the weight's columns); 4-bit rows: lg and lg + 4
    const int lrow_x = lr * L::kRowX + (((kDecode ? 2 * lg : lg) ^ (lr & 7)) * 16);
    constexpr int kOther = kDecode ? 16 : 64;
    u32x4_t a[2][GA][SUB], b[FT][2];
    uint32_t wsc[2][GA][SUB], xsc[FT][L::kWordsX];
    auto read_a = [&](int buf, int f, int u, int slot, int g) {
        const int blk = GA * g + f;
        const char* at = s_lds + slot * L::kStage + (wn + 32 * (blk / 2) + 4 * (blk & 1)) * L::kRowW;
        a[buf][f][u] = *reinterpret_cast<const u32x4_t*>(at + (u ? lrow_w ^ 64 : lrow_w));
    };
    auto read_ws = [&](int buf, int f, int sslot, int g) {
        const int blk = GA * g + f;
        const int row = wn + 32 * (blk / 2) + 4 * (blk & 1) + 8 * (lr >> 2) + (lr & 3);
        const uint32_t* at = reinterpret_cast<const uint32_t*>(s_sc + sslot * L::kScales) + row * L::kWordsW;
#pragma unroll
        for (int u = 0; u < SUB; ++u) wsc[buf][f][u] = at[u];
    };
    auto read_b = [&](int h, int u, int slot) {
        b[h][u] = *reinterpret_cast<const u32x4_t*>(s_lds + slot * L::kStage + BN * L::kRowW + (wt + 16 * h) * L::kRowX +
                                                    (u ? lrow_x ^ kOther : lrow_x));
    };
    auto read_xs = [&](int h, int sslot) {
        const uint32_t* at =
            reinterpret_cast<const uint32_t*>(s_sc + sslot * L::kScales + L::kChunksW * 256) + (wt + 16 * h + lr) * L::kWordsX;
#pragma unroll
        for (int u = 0; u < L::kWordsX; ++u) xsc[h][u] = at[u];
    };
    // The byte of lane group lg of the words of a step's 128-column parts, in bytes 0 and 1.
    const uint32_t sel = 0x0c0c0400u + (uint32_t)lg * 0x0101u;
    auto pick = [&](const uint32_t* w) {
        if constexpr (SUB == 2)
            return __builtin_amdgcn_perm(w[1], w[0], sel);
        else
            return w[0] >> (8 * lg);
    };

    const int nk = k1 - k0;
#pragma unroll
    for (int s = 0; s < ST; ++s)
#pragma unroll
        for (int o = 0; o < PW; ++o) issue(o, s, s, k0 + min(s, nk - 1));
    wait_vmcnt_le<PW*(ST - 1)>();
    lds_barrier();
#pragma unroll
    for (int f = 0; f < GA; ++f) {
#pragma unroll
        for (int u = 0; u < SUB; ++u) read_a(0, f, u, 0, 0);
        read_ws(0, f, 0, 0);
    }
#pragma unroll
    for (int h = 0; h < FT; ++h) {
        read_b(h, 0, 0);
        read_b(h, 1, 0);
        read_xs(h, 0);
    }
    int slot = 0, sslot = 0;
    constexpr auto before = [](int g) { return PW * g / NG; };  // loads of a step that go out before its group g
    static_assert(before(1) <= SU + WU + XU, "a group's place is free when its loads go out");
    auto step = [&](auto parity, int i) {
        constexpr int P = decltype(parity)::value;  // (an odd number of groups: the buffers of a change places each step)
        const int next = slot + 1 == ST ? 0 : slot + 1;
        const int snext = sslot + 1 == ST + 1 ? 0 : sslot + 1;
        const int sold = sslot == 0 ? ST : sslot - 1;  // the slot of the step before, for the step ST later
        const int kn = k0 + min(i + ST, nk - 1);
        auto group = [&](auto gc) {
            constexpr int g = decltype(gc)::value;
            constexpr bool last = g + 1 == NG;
            constexpr int cur = (P * NG + g) & 1, nxt = cur ^ 1;
            // What is read now has to be there: the loads issued after it may be outstanding.
            wait_vmcnt_le<last ? (NG - 1) * WU + (ST - 2) * PW + before(NG - 1)
                               : (NG - 2 - g) * WU + (ST - 1) * PW + before(g)>();
            lds_barrier();
            uint32_t as[GA];
#pragma unroll
            for (int f = 0; f < GA; ++f) as[f] = pick(wsc[cur][f]);
            Frag<LORA_BF16> aq[kDecode ? GA : 1][4];
            if constexpr (kDecode) {
#pragma unroll
                for (int f = 0; f < GA; ++f) {
                    const float s = quant_scale(as[f] & 255u);
#pragma unroll
                    for (int c = 0; c < 4; ++c) aq[f][c] = mx_decode8<LORA_BF16>(a[cur][f][0][c], s);
                }
            }
#pragma unroll
            for (int h = 0; h < FT; ++h) {
                if constexpr (XB == 4) {
                    const uint32_t bs = pick(xsc[h]);
#pragma unroll
                    for (int f = 0; f < GA; ++f) {
                        f32x4_t& c = acc[GA * g + f][h];
                        c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(a[cur][f][0]), mx_operand(b[h][0]), c, 4, 4,
                                                                             0, (int)as[f], 0, (int)bs);
                    }
#pragma unroll
                    for (int f = 0; f < GA; ++f) {
                        f32x4_t& c = acc[GA * g + f][h];
                        c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(a[cur][f][SUB - 1]), mx_operand(b[h][1]), c, 4, 4,
                                                                             1, (int)as[f], 1, (int)bs);
                    }
                } else {
                    const uint32_t bs = xsc[h][0] >> (8 * ((k0 + min(i, nk - 1)) & 3));
                    if constexpr (kDecode) {
                        const float s = quant_scale(bs & 255u);
                        const Frag<LORA_BF16> bq[4] = {dequant8<LORA_BF16>(b[h][0][0], b[h][0][1], s),
                                                       dequant8<LORA_BF16>(b[h][0][2], b[h][0][3], s),
                                                       dequant8<LORA_BF16>(b[h][1][0], b[h][1][1], s),
                                                       dequant8<LORA_BF16>(b[h][1][2], b[h][1][3], s)};
#pragma unroll
                        for (int f = 0; f < GA; ++f)
#pragma unroll
                            for (int c = 0; c < 4; ++c) acc[GA * g + f][h] = mma(aq[f][c], bq[c], acc[GA * g + f][h]);
                    } else {
                        const i32x8_t bo = __builtin_bit_cast(
                            i32x8_t, __builtin_shufflevector(b[h][0], b[h][1], 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
                        for (int f = 0; f < GA; ++f) {
                            f32x4_t& c = acc[GA * g + f][h];
                            c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(a[cur][f][0]), bo, c, 4, 0, 0,
                                                                                 (int)as[f], 0, (int)bs);
                        }
                    }
                }
                // reads of the next group (with the last group the next step's first and its
                // activations) and loads, a few at a time between the products
                constexpr int NR = GA * (SUB + 1);
#pragma unroll
                for (int r = h * NR / FT; r < (h + 1) * NR / FT; ++r) {
                    const int f = r / (SUB + 1), u = r % (SUB + 1);
                    if (u < SUB)
                        read_a(nxt, f, u, last ? next : slot, last ? 0 : g + 1);
                    else
                        read_ws(nxt, f, last ? snext : sslot, last ? 0 : g + 1);
                }
                if (last) {
                    read_b(h, 0, next);
                    read_b(h, 1, next);
                    read_xs(h, snext);
                }
                constexpr int o0 = before(g), n = before(g + 1) - o0;
#pragma unroll
                for (int o = o0 + h * n / FT; o < o0 + (h + 1) * n / FT; ++o) issue(o, slot, sold, kn);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        group(std::integral_constant<int, 0>{});
        if constexpr (NG > 1) group(std::integral_constant<int, 1 % NG>{});
        if constexpr (NG > 2) group(std::integral_constant<int, 2 % NG>{});
        if constexpr (NG > 3) group(std::integral_constant<int, 3 % NG>{});
        slot = next;
        sslot = snext;
    };
    for (int i = 0; i < nk; i += 2) {
        step(std::integral_constant<int, 0>{}, i);
        if (i + 1 < nk) step(std::integral_constant<int, NG & 1>{}, i + 1);
    }
    wait_vmcnt_le<0>();  // nothing may land in LDS after the workgroup has ended
#pragma unroll
    for (int h = 0; h < FT; ++h) {
        const int tl = wt + 16 * h + lr;
        const bool t_in = tl < trows;
        const int64_t t = t0 + (t_in ? tl : 0);
        if (p.splits > 1) {
            float* row = p.part + ((int64_t)part * p.T + t) * p.N;
#pragma unroll
            for (int f = 0; f < FN; f += 2) {
                const int n = n0 + wn + 16 * f + 8 * lg;
                if (t_in && n < p.N) {
                    LORA_GLOBAL f32x4_t* d = gptr(reinterpret_cast<f32x4_t*>(row + n));
                    d[0] = acc[f][h];
                    d[1] = acc[f + 1][h];
                }
            }
            continue;
        }
        // Eight outputs at a time, added to what is there in fp32 and rounded once; the old
        // values of a row are loaded together (outputs past the matrix load its first ones).
        char* row = p.y + t * p.ldy * Frag<DT>::kBytes;
        float old[FN / 2][8];
        if (p.accumulate) {
#pragma unroll
            for (int f = 0; f < FN; f += 2) {
                const int n = n0 + wn + 16 * f + 8 * lg;
                Elem<DT>::load8(row + (int64_t)(n < p.N ? n : 0) * Frag<DT>::kBytes, old[f / 2]);
            }
        }
#pragma unroll
        for (int f = 0; f < FN; f += 2) {
            const int n = n0 + wn + 16 * f + 8 * lg;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = acc[f + e / 4][h][e & 3] + (p.accumulate ? old[f / 2][e] : 0.f);
            if (t_in && n < p.N) Elem<DT>::store8(row + (int64_t)n * Frag<DT>::kBytes, v);
        }
    }
}

// ------------------------------------------------------------------ few rows: the weight as a stream
//
// Up to 16 rows a tile: the weight is read straight into operand registers and nothing
// of it is shared between waves.  A workgroup of NW waves computes 16 outputs of a
// tile's rows; wave w takes the steps w, w + NW, ... of 256 columns (128 bytes of a
// weight row), kMxU of them in flight, and the waves' sums are added in wave order
// through LDS.
constexpr int kMxU = 2;

template <int NW, int XB, int DT>
__global__ __launch_bounds__(NW* kWave) void mx_stream_kernel(MxParams p) {
    constexpr bool kDecode = kMxDecode<XB, DT>;
    __shared__ f32x4_t s_acc[NW][kWave];
    const int wave = wave_id();
    const int lane = threadIdx.x & (kWave - 1);
    const int lr = lane & 15, lg = lane >> 4;
    int n0 = blockIdx.x * 16;
    MxGroup grp{0, p.T, 0};
    if (p.offsets) {
        const int tiles = mx_total_tiles<16>(p, lane);
        const int tile = blockIdx.x / p.tiles_n;
        if (tile >= tiles) return;
        n0 = (blockIdx.x - tile * p.tiles_n) * 16;
        grp = mx_find_tile<16>(p, tile, lane);
    }
    const int64_t wrow = (int64_t)grp.expert * p.N + min(n0 + lr, p.N - 1);
    const LORA_GLOBAL uint8_t* w = gptr(p.w + wrow * p.ldw + 16 * lg);
    const LORA_GLOBAL uint8_t* ws = gptr(p.ws + wrow * p.ldws);
    const int64_t row = grp.first + min(lr, grp.rows - 1);
    const LORA_GLOBAL uint8_t* x = gptr(p.x + row * p.ldx + (kDecode ? 32 : 16) * lg);
    const LORA_GLOBAL uint8_t* xs = gptr(p.xs + row * p.ldxs);
    const uint32_t sel = 0x0c0c0400u + (uint32_t)lg * 0x0101u;
    f32x4_t acc{0.f, 0.f, 0.f, 0.f};
    // p.steps: of 128 columns for 8-bit rows (an odd number leaves the last step's second
    // half without a column), of 256 for 4-bit rows
    const int steps = XB == 4 ? p.steps : (p.steps + 1) / 2;
    for (int k0 = wave; k0 < steps; k0 += NW * kMxU) {
        u32x4_t a[kMxU][2], b[kMxU][XB == 4 ? 2 : 4];
        u32x2_t as[kMxU], bs[kMxU];
#pragma unroll
        for (int u = 0; u < kMxU; ++u) {
            const int kb = min(k0 + NW * u, steps - 1);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                a[u][i] = __builtin_nontemporal_load(reinterpret_cast<const LORA_GLOBAL u32x4_t*>(w + kb * 128 + 64 * i));
            as[u] = *reinterpret_cast<const LORA_GLOBAL u32x2_t*>(ws + kb * 8);
            if constexpr (XB == 4) {
#pragma unroll
                for (int i = 0; i < 2; ++i) b[u][i] = *reinterpret_cast<const LORA_GLOBAL u32x4_t*>(x + kb * 128 + 64 * i);
                bs[u] = *reinterpret_cast<const LORA_GLOBAL u32x2_t*>(xs + kb * 8);
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int kx = min(2 * kb + i, p.steps - 1);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        b[u][2 * i + h] = *reinterpret_cast<const LORA_GLOBAL u32x4_t*>(x + kx * 128 + (kDecode ? 16 : 64) * h);
                    bs[u][i] = xs[kx];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kMxU; ++u) {
            const int kb = k0 + NW * u;
            if (kb >= steps) break;
            const uint32_t sa = __builtin_amdgcn_perm(as[u][1], as[u][0], sel);
            if constexpr (XB == 4) {
                const uint32_t sb = __builtin_amdgcn_perm(bs[u][1], bs[u][0], sel);
                acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(a[u][0]), mx_operand(b[u][0]), acc, 4, 4, 0, (int)sa,
                                                                       0, (int)sb);
                acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(a[u][1]), mx_operand(b[u][1]), acc, 4, 4, 1, (int)sa,
                                                                       1, (int)sb);
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (2 * kb + i >= p.steps) break;
                    if constexpr (kDecode) {
                        const float fa = quant_scale((sa >> (8 * i)) & 255u), fb = quant_scale(bs[u][i]);
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            acc = mma(mx_decode8<LORA_BF16>(a[u][i][c], fa),
                                      dequant8<LORA_BF16>(b[u][2 * i + c / 2][2 * (c & 1)], b[u][2 * i + c / 2][2 * (c & 1) + 1], fb), acc);
                    } else {
                        const i32x8_t bo = __builtin_bit_cast(
                            i32x8_t, __builtin_shufflevector(b[u][2 * i], b[u][2 * i + 1], 0, 1, 2, 3, 4, 5, 6, 7));
                        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(a[u][i]), bo, acc, 4, 0, 0,
                                                                               (int)(sa >> (8 * i)), 0, (int)bs[u][i]);
                    }
                }
            }
        }
    }
    s_acc[wave][lane] = acc;
    __syncthreads();
    if (wave == 0) {
        f32x4_t sum = s_acc[0][lane];
#pragma unroll
        for (int v = 1; v < NW; ++v) sum += s_acc[v][lane];
        const int n = n0 + 4 * lg;
        if (lr < grp.rows && n < p.N) {  // (N is a multiple of 8: the four are in or out together)
            char* at = p.y + ((grp.first + lr) * p.ldy + n) * Frag<DT>::kBytes;
            if (p.accumulate) {
                if constexpr (DT == LORA_BF16) {
                    const u32x2_t o = *gptr(reinterpret_cast<const u32x2_t*>(at));
                    sum += f32x4_t{__uint_as_float(o[0] << 16), __uint_as_float(o[0] & 0xffff0000u), __uint_as_float(o[1] << 16),
                                   __uint_as_float(o[1] & 0xffff0000u)};
                } else {
                    sum += *gptr(reinterpret_cast<const f32x4_t*>(at));
                }
            }
            if constexpr (DT == LORA_BF16)
                *gptr(reinterpret_cast<u32x2_t*>(at)) = u32x2_t{pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3])};
            else
                *gptr(reinterpret_cast<f32x4_t*>(at)) = sum;
        }
    }
}

}  // namespace lora
