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
// as a subnormal 8-bit code counts as 2^-6).  So the rows' codes are taken in two halves,
// those of 2 and more and the smaller ones, and nothing is cut: the products of the first
// are multiples of 2^-2 * 0.5 and their powers of two up to 2^(8 + 2), of which 2^-13 is
// 2^-3; those of the second multiples of 2^-9 * 0.5, with up to 2^(0 + 2), of which 2^-13
// is 2^-11.  A code's half is its bit 6.  Each product is made twice; a caller of bf16 y
// who accepts the cut (LORA_MX_CUT: 1.5e-5 of a result on normal data, more where large
// products cancel) has them once.  (Codes decoded to
// bf16 numbers, for that instruction, cost as much of the matrix cores and more vector
// work: 2048 x 14336 x 4096, fp32 y, 175 us against 162, in 256 x 128 tiles of four waves.)
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
// Inclusive sum over the wave's lanes (in registers: 1, 2, 4, 8 lanes up within 16, then
// the sums of 16 and of 32 lanes to those behind them).
__device__ __forceinline__ int mx_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);
    return v + __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
}
template <int BT>
struct MxExperts {
    int begin, end, incl;  // of this lane's expert: its rows, the tiles of the experts up to it
    __device__ __forceinline__ static MxExperts load(const MxParams& p, int e) {
        MxExperts x{0, 0, 0};
        if (e < p.experts) {
            x.begin = min(max(gptr(p.offsets)[e], 0), p.T);
            x.end = min(max(gptr(p.offsets)[e + 1], x.begin), p.T);
        }
        x.incl = mx_scan(x.tiles());
        return x;
    }
    __device__ __forceinline__ int tiles() const { return (end - begin + BT - 1) / BT; }
    __device__ __forceinline__ int total() const { return __builtin_amdgcn_readlane(incl, kWave - 1); }
};
// The number of tiles; first: experts 0 .. 63.
template <int BT>
__device__ __forceinline__ int mx_total_tiles(const MxParams& p, int lane, const MxExperts<BT>& first) {
    int total = first.total();
    for (int e0 = kWave; e0 < p.experts; e0 += kWave) total += MxExperts<BT>::load(p, e0 + lane).total();
    return total;
}
// (tile below the total)
template <int BT>
__device__ __forceinline__ MxGroup mx_find_tile(const MxParams& p, int tile, int lane, MxExperts<BT> x) {
    for (int e0 = 0;;) {
        const uint64_t past = __ballot(x.incl > tile);
        if (past) {
            const int at = __ffsll((long long)past) - 1;
            const int in = tile - __builtin_amdgcn_readlane(x.incl - x.tiles(), at);
            const int begin = __builtin_amdgcn_readlane(x.begin, at) + in * BT;
            return MxGroup{begin, min(BT, __builtin_amdgcn_readlane(x.end, at) - begin), e0 + at};
        }
        tile -= x.total();
        e0 += kWave;
        if (e0 >= p.experts) return MxGroup{0, 0, 0};
        x = MxExperts<BT>::load(p, e0 + lane);
    }
}

// ------------------------------------------------------------------ operands

// Four 8-bit codes' upper half: the codes of magnitude 2 and more, zeros for the others.
__device__ __forceinline__ uint32_t mx_upper(uint32_t w) {
    // (bit 6 of every byte spread over it: the selectors 8 to 11 give the signs of bytes 1
    // and 3 of the second and the first operand)
    return w & __builtin_amdgcn_perm(w << 1, w << 9, 0x0b090a08u);
}
__device__ __forceinline__ u32x4_t mx_upper(u32x4_t q) { return u32x4_t{mx_upper(q[0]), mx_upper(q[1]), mx_upper(q[2]), mx_upper(q[3])}; }

// 32 4-bit codes as the matrix instruction's operand.
__device__ __forceinline__ i32x8_t mx_operand(u32x4_t q) { return i32x8_t{(int)q[0], (int)q[1], (int)q[2], (int)q[3], 0, 0, 0, 0}; }
// 32 8-bit codes.
__device__ __forceinline__ i32x8_t mx_operand(u32x4_t a, u32x4_t b) {
    return __builtin_bit_cast(i32x8_t, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// ------------------------------------------------------------------ tiles through LDS
//
// A workgroup of WN x WT waves computes BN outputs x BT rows.  A step is 256 columns
// of 4-bit rows or 128 of 8-bit rows, 128 bytes of an activation row; BN weight and
// BT activation rows' steps go from memory straight into LDS, ST stages in a ring,
// the scales a span of steps at a time (MxLds).  The pieces of a step are handed over as
// in base.h: the weight blocks are taken two or four at a time, and after the barrier at the
// start of such a group its place is free for the step ST later, whose loads go out
// between the products.
//
// 16-byte unit c of a row lies at position c ^ s of it: s is the operand row modulo 8
// for rows of 128 bytes, half of it modulo 4 for rows of 64 bytes, so that 8 lanes
// that a read takes together fall on different banks.
// XB: bits of the activation rows, DT: type of y, HALVES: the rows' codes in two halves.
template <int BN, int BT, int WN, int WT, int ST, int XB, int DT, bool HALVES>
__global__ __launch_bounds__(WN* WT* kWave) void mx_kernel(MxParams p) {
    using L = MxLds<BN, BT, ST, XB>;
    static_assert(XB == 8 || !HALVES, "4-bit rows' products are exact as they are");
    constexpr int NW = WN * WT;
    constexpr int FN = BN / WN / 16, FT = BT / WT / 16;  // 16 x 16 blocks of a wave
    constexpr int SUB = XB == 4 ? 2 : 1;                 // instructions of a step and block
    constexpr int RW = 1024 / L::kRowW, RX = 1024 / L::kRowX;  // rows of a load
    // weight blocks of a group (so many that every wave has a load of its own), groups
    constexpr int GA = 32 * WN / RW < NW && FN % 4 == 0 ? 4 : 2, NG = FN / GA;
    // loads of a wave: for a weight group, for the activations, for the scales
    constexpr int GR = GA * 16 * WN;                     // weight rows of a group
    constexpr int WU = GR / RW >= NW ? GR / RW / NW : 1, XU = BT / RX / NW;
    constexpr int SU = (L::kLoadsW + L::kLoadsX + NW - 1) / NW;
    constexpr int PW = SU + NG * WU + XU;
    static_assert(FN % 2 == 0 && NG <= 4 && BT % (RX * NW) == 0, "the loads divide evenly");
    static_assert(GR / RW >= NW ? GR % (RW * NW) == 0 : NW % (GR / RW) == 0, "the weight's loads divide evenly");
    __shared__ __attribute__((aligned(16))) char s_lds[L::kBytes];
    char* s_sc = s_lds + ST * L::kStage;

    const int wave = wave_id();
    const int lane = threadIdx.x & (kWave - 1);
    const int lr = lane & 15, lg = lane >> 4;
    // Workgroups of one XCD take neighbouring tiles.
    MxExperts<BT> ex{0, 0, 0};
    int tiles_t = p.tiles_t;
    if (p.offsets) {
        ex = MxExperts<BT>::load(p, lane);
        tiles_t = mx_total_tiles<BT>(p, lane, ex);
    }
    const int ntile = p.tiles_n * tiles_t * p.splits;
    const int per = (ntile + kNumXcd - 1) / kNumXcd;
    const int task = (int)(blockIdx.x % kNumXcd) * per + (int)(blockIdx.x / kNumXcd);
    if ((int)(blockIdx.x / kNumXcd) >= per || task >= ntile) return;
    const int tile = task / p.splits, kpart = task - tile * p.splits;
    // this workgroup's steps: whole spans of scales
    const int spans = (p.steps + L::kSpan - 1) / L::kSpan;
    const int k0 = L::kSpan * (int)((int64_t)spans * kpart / p.splits);
    const int k1 = min(p.steps, L::kSpan * (int)((int64_t)spans * (kpart + 1) / p.splits));
    // Order of the tiles: bands of up to kBand tiles along t, walked along n (base.h).
    const int band = tile / (kBand * p.tiles_n), in = tile - band * kBand * p.tiles_n;
    const int bt = min(kBand, tiles_t - band * kBand);
    const int n0 = in / bt * BN, tt = band * kBand + in % bt;
    MxGroup grp{tt * BT, 0, 0};
    if (p.offsets)
        grp = mx_find_tile<BT>(p, tt, lane, ex);
    else
        grp.rows = min(BT, p.T - grp.first);
    const int t0 = grp.first, trows = grp.rows, nrows = min(BN, p.N - n0);
    const int wn = (wave % WN) * (BN / WN), wt = (wave / WN) * (BT / WT);

    // Rows past the tile lie past their buffer: nothing is fetched for them, and their
    // outputs are not stored.
    const int64_t wrow = (int64_t)grp.expert * p.N + n0;
    const buf_rsrc_t rw = make_rsrc(p.w + wrow * p.ldw, (uint32_t)((nrows - 1) * p.ldw + (int64_t)p.steps * L::kRowW));
    const buf_rsrc_t rx = make_rsrc(p.x + (int64_t)t0 * p.ldx, (uint32_t)((trows - 1) * p.ldx + (int64_t)p.steps * L::kRowX));
    // The loads of a step, with what of their addresses stays the same (a row goes into the
    // part of the address that is checked, the column into the other).
    // Weights: load j of group g is RW rows, in the order wave column, row (rows 16 GA g ..
    // 16 GA (g + 1) - 1 of every wave column); a wave without one repeats another's.
    constexpr int CPG = 16 * GA / RW;  // loads of a wave column's group
    constexpr int LWR = 64 / RW;       // lanes of a weight row's step
    const int wr = lane / LWR;
    // (rows of 128 bytes: a load is 8 rows, and the next 8 have the other half of the keys)
    const int w_key = L::kRowW == 128 ? (wr & 3) ^ ((wave & 1) * 4) : 2 * ((wr >> 3) & 1) + ((wr >> 1) & 1);
    static_assert(CPG * WN % 2 == 0 && NW % 2 == 0, "a wave's loads have one parity");
    uint32_t vw[NG][WU], vx[XU];
    int lds_w[NG][WU], lds_x[XU];
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int j = 0; j < WU; ++j) {
            const int c = (wave + NW * j) % (CPG * WN);
            const int row = c / CPG * (BN / WN) + 16 * GA * g + c % CPG * RW;
            vw[g][j] = (uint32_t)((row + wr) * p.ldw) + (uint32_t)((lane % LWR) ^ w_key) * 16u;
            lds_w[g][j] = row * L::kRowW;
        }
#pragma unroll
    for (int j = 0; j < XU; ++j) {
        const int row = 8 * (wave + NW * j);
        vx[j] = (uint32_t)((row + (lane >> 3)) * p.ldx) + (uint32_t)((lane & 7) ^ (lane >> 3)) * 16u;
        lds_x[j] = BN * L::kRowW + row * L::kRowX;
    }
    // Scales: load j of this wave is 64 words of weight or of activation rows; those that go
    // out for place q of a span are of the next span, their part q of its rows.  8 words of
    // a row are exchanged by the row (4: by half as much), so that the rows that a read takes
    // together fall on different banks.
    constexpr int kKeyW = L::kWordsW == 8 ? 3 : 1, kKeyX = L::kWordsX == 8 ? 1 : 0;
    uint32_t vs[SU][L::kSpan];
    int lds_s[SU][L::kSpan], s_step[SU], s_left[SU];
    const uint8_t* s_base[SU];
#pragma unroll
    for (int j = 0; j < SU; ++j) {
        const int c = (wave + NW * j) % (L::kLoadsW + L::kLoadsX);
        const bool of_w = c < L::kLoadsW;
        const int words = of_w ? L::kWordsW : L::kWordsX;
        const uint32_t ld = (uint32_t)(of_w ? p.ldws : p.ldxs);
        s_step[j] = words * 4;
        s_base[j] = (of_w ? p.ws + wrow * p.ldws : p.xs + (int64_t)t0 * p.ldxs) + k0 / L::kSpan * s_step[j];
        s_left[j] = (int)(of_w ? (nrows - 1) * p.ldws + (int64_t)p.steps * (L::kRowW / 16)
                               : (trows - 1) * p.ldxs + (XB == 4 ? (int64_t)p.steps * 8 : (p.steps + 3) / 4 * 4)) -
                    k0 / L::kSpan * s_step[j];
#pragma unroll
        for (int q = 0; q < L::kSpan; ++q) {
            const int m = of_w ? (q * L::kLoadsW + c) % L::kAllW : (q * L::kLoadsX + c - L::kLoadsW) % L::kAllX;
            vs[j][q] = (uint32_t)(m * (64 / words) + lane / words) * ld +
                       ((uint32_t)(lane % words) * 4u ^ (uint32_t)((m & (of_w ? kKeyW : kKeyX)) * 8));
            lds_s[j][q] = (of_w ? 0 : L::kAllW * 256) + m * 256;
        }
    }
    buf_rsrc_t rs[SU];
    auto span_rsrc = [&]() {
#pragma unroll
        for (int j = 0; j < SU; ++j) rs[j] = make_rsrc(s_base[j], (uint32_t)max(s_left[j], 0));
    };
    auto next_span = [&]() {  // the scales' loads that follow are of the next span
#pragma unroll
        for (int j = 0; j < SU; ++j) {
            s_base[j] += s_step[j];
            s_left[j] -= s_step[j];
        }
        span_rsrc();
    };
    // Load o of a step: scales, weight group 0, activations, weight groups 1, 2, ...
    // slot, kb: the step's place in the ring and along k; q, to: its place in the span, and
    // where the scales go
    auto issue = [&](int o, int slot, int kb, int q, int to) {
        char* at = s_lds + slot * L::kStage;
        if (o < SU)
            dma_lds(rs[o], vs[o][q], 0u, s_sc + to + lds_s[o][q], 4);
        else if (o < SU + WU)
            dma_lds(rw, vw[0][o - SU], (uint32_t)kb * L::kRowW, at + lds_w[0][o - SU], 16);
        else if (o < SU + WU + XU)
            dma_lds(rx, vx[o - SU - WU], (uint32_t)kb * L::kRowX, at + lds_x[o - SU - WU], 16);
        else
            dma_lds(rw, vw[(o - SU - XU) / WU][(o - SU - XU) % WU], (uint32_t)kb * L::kRowW,
                    at + lds_w[(o - SU - XU) / WU][(o - SU - XU) % WU], 16);
    };

    // (Zeros that the compiler does not see as one constant: with that it copies every sum
    // to the loop's registers and back in each step: 2048 x 4096 x 4096 from 8-bit rows,
    // 256 x 128 tiles, 44.6 us in place of 30.)
    f32x4_t acc[FN][FT];
#pragma unroll
    for (int a = 0; a < FN; ++a)
#pragma unroll
        for (int b = 0; b < FT; ++b) {
            acc[a][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            asm volatile("" : "+v"(acc[a][b]));
        }

    // This lane's units of an operand row.  Weight row of operand row lr: 8 (lr / 4) +
    // lr % 4 of the pair of blocks, + 4 for its second block.
    const int lrow_w = (8 * (lr >> 2) + (lr & 3)) * L::kRowW + (L::kRowW == 128 ? (lg ^ (lr & 7)) * 16 : (lg ^ ((lr >> 1) & 3)) * 16);
    const int lrow_x = lr * L::kRowX + ((lg ^ (lr & 7)) * 16);  // (and 64 bytes on)
    u32x4_t a[2][GA][SUB], b[FT][2], upper[HALVES ? FT : 1][2];
    constexpr int SX = XB == 4 ? 2 : 1;
    uint32_t wsc[2][GA][SUB], xsc[FT][SX];
    auto read_a = [&](int buf, int f, int u, int slot, int g) {
        const int blk = GA * g + f;
        const char* at = s_lds + slot * L::kStage + (wn + 32 * (blk / 2) + 4 * (blk & 1)) * L::kRowW;
        a[buf][f][u] = *reinterpret_cast<const u32x4_t*>(at + (u ? lrow_w ^ 64 : lrow_w));
    };
    // scales of a step: its place in the span, exchanged as the row's words are
    constexpr int kPartW = L::kRowW / 16;  // bytes of a weight row's step
    const int srow_w = (8 * (lr >> 2) + (lr & 3)) * L::kWordsW * 4 + (L::kWordsW == 8 ? lr >> 2 : lr >> 3) * 8;
    const int srow_x = L::kAllW * 256 + lr * L::kWordsX * 4 + (L::kWordsX == 8 ? (lr >> 3) * 8 : 0);
    auto read_ws = [&](int buf, int f, const char* at, int part, int g) {
        const int blk = GA * g + f;
        const uint32_t* w = reinterpret_cast<const uint32_t*>(at + (wn + 32 * (blk / 2) + 4 * (blk & 1)) * L::kWordsW * 4 +
                                                              (srow_w ^ (part * kPartW)));
#pragma unroll
        for (int u = 0; u < SUB; ++u) wsc[buf][f][u] = w[u];
    };
    auto read_b = [&](int h, int u, int slot) {
        b[h][u] = *reinterpret_cast<const u32x4_t*>(s_lds + slot * L::kStage + BN * L::kRowW + (wt + 16 * h) * L::kRowX +
                                                    (u ? lrow_x ^ 64 : lrow_x));
    };
    auto read_xs = [&](int h, const char* at, int part) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(at + (wt + 16 * h) * L::kWordsX * 4 +
                                                              (XB == 4 ? srow_x ^ (part * 8) : srow_x + (part >> 2) * 4));
#pragma unroll
        for (int u = 0; u < SX; ++u) xsc[h][u] = w[u];
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
    // the first span's scales, then the first steps (and with them the second span's)
    span_rsrc();
#pragma unroll
    for (int q = 0; q < L::kSpan; ++q)
#pragma unroll
        for (int o = 0; o < SU; ++o) issue(o, 0, 0, q, 0);
    next_span();
#pragma unroll
    for (int s = 0; s < ST; ++s)
#pragma unroll
        for (int o = 0; o < PW; ++o) issue(o, s, k0 + min(s, nk - 1), s % L::kSpan, L::kScales);
    wait_vmcnt_le<PW*(ST - 1)>();
    lds_barrier();
#pragma unroll
    for (int f = 0; f < GA; ++f) {
#pragma unroll
        for (int u = 0; u < SUB; ++u) read_a(0, f, u, 0, 0);
        read_ws(0, f, s_sc, 0, 0);
    }
#pragma unroll
    for (int h = 0; h < FT; ++h) {
        read_b(h, 0, 0);
        read_b(h, 1, 0);
        read_xs(h, s_sc, 0);
    }
    // loads of a step that go out before its group g
    constexpr auto before = [](int g) { return PW * g / NG; };
    static_assert(before(1) <= SU + WU + XU, "a group's place is free when its loads go out");
    // where the scales lie of the span that is read, and those are loaded that go out now
    int read_at = 0, load_at = L::kScales;
    auto after_slot = [](int at) { return at == (L::kSlots - 1) * L::kScales ? 0 : at + L::kScales; };
    // Step i, place q modulo its span's steps: places in the rings are known when the code is made (half
    // of a step's instructions were their arithmetic, and a wave alone on its SIMD takes a
    // few cycles for each: 256 x 4096 x 4096 from 8-bit rows 14.0 us,
    // and 10.8 as it is).
    auto step = [&](auto place, int i) {
        constexpr int q = decltype(place)::value, slot = q % ST, next = (q + 1) % ST;
        constexpr int part = q % L::kSpan, npart = (q + 1) % L::kSpan, lpart = (q + ST) % L::kSpan;
        constexpr int P = q & 1;  // (an odd number of groups: the buffers of a change places each step)
        const int kn = k0 + min(i + ST, nk - 1);
        if constexpr (lpart == 0) {
            next_span();
            load_at = after_slot(load_at);
        }
        const char* sc = s_sc + read_at;
        if constexpr (npart == 0) read_at = after_slot(read_at);
        const char* nsc = s_sc + read_at;
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
                    const uint32_t bs = xsc[h][0] >> (8 * (part & 3));
                    if constexpr (HALVES) {
                        if constexpr (g == 0) {
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                upper[h][u] = mx_upper(b[h][u]);
                                b[h][u] ^= upper[h][u];
                                // (both now: else the compiler makes the lower half in the upper's
                                // registers, once the products that read them are done)
                                asm volatile("" : "+v"(upper[h][u]), "+v"(b[h][u]));
                            }
                        }
                        const i32x8_t bu = mx_operand(upper[h][0], upper[h][1]);
#pragma unroll
                        for (int f = 0; f < GA; ++f) {
                            f32x4_t& c = acc[GA * g + f][h];
                            c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(a[cur][f][0]), bu, c, 4, 0, 0,
                                                                                 (int)as[f], 0, (int)bs);
                        }
                    }
                    const i32x8_t bo = mx_operand(b[h][0], b[h][1]);
#pragma unroll
                    for (int f = 0; f < GA; ++f) {
                        f32x4_t& c = acc[GA * g + f][h];
                        c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(a[cur][f][0]), bo, c, 4, 0, 0, (int)as[f], 0,
                                                                             (int)bs);
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
                        read_ws(nxt, f, last ? nsc : sc, last ? npart : part, last ? 0 : g + 1);
                }
                if (last) {
                    read_b(h, 0, next);
                    read_b(h, 1, next);
                    read_xs(h, nsc, npart);
                }
                constexpr int o0 = before(g), n = before(g + 1) - o0;
#pragma unroll
                for (int o = o0 + h * n / FT; o < o0 + (h + 1) * n / FT; ++o) issue(o, slot, kn, lpart, load_at);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        group(std::integral_constant<int, 0>{});
        if constexpr (NG > 1) group(std::integral_constant<int, 1 % NG>{});
        if constexpr (NG > 2) group(std::integral_constant<int, 2 % NG>{});
        if constexpr (NG > 3) group(std::integral_constant<int, 3 % NG>{});
    };
    constexpr int U = L::kSpan < 4 ? 4 : L::kSpan;
    static_assert(U <= 8 && U % L::kSpan == 0 && U % ST == 0, "a span's steps take whole rounds of the ring");
    for (int i = 0; i < nk; i += U) {
        step(std::integral_constant<int, 0>{}, i);
        if (i + 1 < nk) step(std::integral_constant<int, 1>{}, i + 1);
        if (i + 2 < nk) step(std::integral_constant<int, 2>{}, i + 2);
        if (i + 3 < nk) step(std::integral_constant<int, 3>{}, i + 3);
        if constexpr (U > 4) {
            if (i + 4 < nk) step(std::integral_constant<int, 4 % U>{}, i + 4);
            if (i + 5 < nk) step(std::integral_constant<int, 5 % U>{}, i + 5);
            if (i + 6 < nk) step(std::integral_constant<int, 6 % U>{}, i + 6);
            if (i + 7 < nk) step(std::integral_constant<int, 7 % U>{}, i + 7);
        }
    }
    wait_vmcnt_le<0>();  // nothing may land in LDS after the workgroup has ended
#pragma unroll
    for (int h = 0; h < FT; ++h) {
        const int tl = wt + 16 * h + lr;
        const bool t_in = tl < trows;
        const int64_t t = t0 + (t_in ? tl : 0);
        if (p.splits > 1) {
            float* row = p.part + ((int64_t)kpart * p.T + t) * p.N;
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

// ------------------------------------------------------------------ few rows: waves side by side along k
//
// A workgroup of NW waves computes 16 FN outputs x 16 FT rows; wave w takes the pieces
// w, w + NW, ... of 512 columns (256 bytes of a weight row, 16 of its scales) for the whole
// tile, so no byte of the operands is wanted by two of its waves: they go from memory
// straight into operand registers, a piece ahead, without LDS and without a barrier until
// the waves' sums are added, in wave order, through LDS.  Rows that do not exist and
// columns past the end lie past their buffer: nothing is fetched for them.
template <int NW, int FN, int FT, int XB, int DT, bool HALVES>
__global__ __launch_bounds__(NW* kWave) void mx_stream_kernel(MxParams p) {
    static_assert(XB == 8 || !HALVES, "4-bit rows' products are exact as they are");
    constexpr int XH = XB == 4 ? 1 : 2;  // 16-byte units of a lane for 128 columns of an activation row
    __shared__ f32x4_t s_acc[NW][FN * FT][kWave];
    const int wave = wave_id();
    const int lane = threadIdx.x & (kWave - 1);
    const int lr = lane & 15, lg = lane >> 4;
    // Workgroups of one XCD take neighbouring tiles: of one weight block's rows, or of one
    // expert's tile of rows.
    MxExperts<16 * FT> ex{0, 0, 0};
    int tiles_t = p.tiles_t;
    if (p.offsets) {
        ex = MxExperts<16 * FT>::load(p, lane);
        tiles_t = mx_total_tiles<16 * FT>(p, lane, ex);
    }
    const int ntile = p.tiles_n * tiles_t;
    const int per = (ntile + kNumXcd - 1) / kNumXcd;
    const int tile = (int)(blockIdx.x % kNumXcd) * per + (int)(blockIdx.x / kNumXcd);
    if ((int)(blockIdx.x / kNumXcd) >= per || tile >= ntile) return;
    int n0, tt;
    if (p.offsets) {
        tt = tile / p.tiles_n;
        n0 = (tile - tt * p.tiles_n) * 16 * FN;
    } else {
        n0 = tile / tiles_t * 16 * FN;
        tt = tile % tiles_t;
    }
    MxGroup grp{tt * 16 * FT, min(16 * FT, p.T - tt * 16 * FT), 0};
    if (p.offsets) grp = mx_find_tile<16 * FT>(p, tt, lane, ex);
    const int nrows = min(16 * FN, p.N - n0);
    const int64_t wrow = (int64_t)grp.expert * p.N + n0;
    const int blocks = XB == 4 ? 2 * p.steps : p.steps;  // of 128 columns
    const int pieces = (blocks + 3) / 4;
    const uint32_t bytes_w = (uint32_t)((nrows - 1) * p.ldw + (int64_t)blocks * 64);
    const uint32_t bytes_ws = (uint32_t)((nrows - 1) * p.ldws + (int64_t)blocks * 4);
    const uint32_t bytes_x = (uint32_t)((grp.rows - 1) * p.ldx + (int64_t)blocks * (XB * 16));
    const uint32_t bytes_xs = (uint32_t)((grp.rows - 1) * p.ldxs + (XB == 4 ? (int64_t)blocks * 4 : (blocks + 3) / 4 * 4));
    const uint8_t *w0 = p.w + wrow * p.ldw, *ws0 = p.ws + wrow * p.ldws;
    const uint8_t *x0 = p.x + grp.first * p.ldx, *xs0 = p.xs + grp.first * p.ldxs;
    uint32_t vw[FN], vws[FN], vx[FT], vxs[FT];
#pragma unroll
    for (int f = 0; f < FN; ++f) {
        vw[f] = (uint32_t)((16 * f + lr) * p.ldw) + 16u * lg;
        vws[f] = (uint32_t)((16 * f + lr) * p.ldws);
    }
#pragma unroll
    for (int h = 0; h < FT; ++h) {
        vx[h] = (uint32_t)((16 * h + lr) * p.ldx) + 16u * lg;
        vxs[h] = (uint32_t)((16 * h + lr) * p.ldxs);
    }
    f32x4_t acc[FN][FT];
#pragma unroll
    for (int f = 0; f < FN; ++f)
#pragma unroll
        for (int h = 0; h < FT; ++h) {
            acc[f][h] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            asm volatile("" : "+v"(acc[f][h]));  // (as in mx_kernel)
        }
    struct Piece {
        u32x4_t a[FN][4], b[FT][4 * XH];
        u32x4_t as[FN], bs[FT];  // scales of the four blocks of 128 columns: words (8-bit rows: the bytes of a word)
    };
    // (a piece's columns come with the base, which is the same for all lanes, and the buffer
    // ends where the last row's columns do)
    auto load = [&](Piece& r, int k) {
        const int64_t cw = (int64_t)k * 256, cx = (int64_t)k * (XB * 64), cs = (int64_t)k * 16, csx = XB == 4 ? cs : (int64_t)k * 4;
        const buf_rsrc_t rw = make_rsrc(w0 + cw, bytes_w - (uint32_t)cw), rws = make_rsrc(ws0 + cs, bytes_ws - (uint32_t)cs);
        const buf_rsrc_t rx = make_rsrc(x0 + cx, bytes_x - (uint32_t)cx), rxs = make_rsrc(xs0 + csx, bytes_xs - (uint32_t)csx);
#pragma unroll
        for (int f = 0; f < FN; ++f) {
#pragma unroll
            for (int i = 0; i < 4; ++i) r.a[f][i] = buf_load16(rw, vw[f] + 64u * i, 0u);
            r.as[f] = buf_load16(rws, vws[f], 0u);
        }
#pragma unroll
        for (int h = 0; h < FT; ++h) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int u = 0; u < XH; ++u)
                    r.b[h][XH * i + u] = buf_load16(rx, vx[h] + (uint32_t)(XB * 16 * i + 64 * u), 0u);
            if constexpr (XB == 4)
                r.bs[h] = buf_load16(rxs, vxs[h], 0u);
            else
                r.bs[h][0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rxs, (int)vxs[h], 0, 0);
        }
    };
    auto multiply = [&](const Piece& r, int k) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (4 * k + i >= blocks) break;
            uint32_t as[FN], bs[FT];
#pragma unroll
            for (int f = 0; f < FN; ++f) as[f] = r.as[f][i] >> (8 * lg);
#pragma unroll
            for (int h = 0; h < FT; ++h) bs[h] = XB == 4 ? r.bs[h][i] >> (8 * lg) : r.bs[h][0] >> (8 * i);
#pragma unroll
            for (int h = 0; h < FT; ++h) {
                i32x8_t bo, bu;
                if constexpr (XB == 4) {
                    bo = mx_operand(r.b[h][i]);
                } else {
                    const u32x4_t q0 = r.b[h][XH * i], q1 = r.b[h][XH * i + XH - 1];
                    if constexpr (HALVES) {
                        u32x4_t u0 = mx_upper(q0), u1 = mx_upper(q1), l0 = q0 ^ u0, l1 = q1 ^ u1;
                        asm volatile("" : "+v"(u0), "+v"(u1), "+v"(l0), "+v"(l1));  // (as in mx_kernel)
                        bu = mx_operand(u0, u1);
                        bo = mx_operand(l0, l1);
                    } else {
                        bo = mx_operand(q0, q1);
                    }
                }
#pragma unroll
                for (int f = 0; f < FN; ++f) {
                    constexpr int kFormat = XB == 4 ? 4 : 0;
                    if constexpr (HALVES)
                        acc[f][h] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(r.a[f][i]), bu, acc[f][h], 4, kFormat, 0,
                                                                                     (int)as[f], 0, (int)bs[h]);
                    acc[f][h] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(r.a[f][i]), bo, acc[f][h], 4, kFormat, 0,
                                                                                 (int)as[f], 0, (int)bs[h]);
                }
            }
        }
    };
    Piece r0, r1;
    if (wave < pieces) {
        load(r0, wave);
        for (int k = wave;; k += 2 * NW) {
            if (k + NW >= pieces) {
                multiply(r0, k);
                break;
            }
            load(r1, k + NW);
            multiply(r0, k);
            if (k + 2 * NW >= pieces) {
                multiply(r1, k + NW);
                break;
            }
            load(r0, k + 2 * NW);
            multiply(r1, k + NW);
        }
    }
#pragma unroll
    for (int f = 0; f < FN; ++f)
#pragma unroll
        for (int h = 0; h < FT; ++h) s_acc[wave][f * FT + h][lane] = acc[f][h];
    __syncthreads();
    for (int blk = wave; blk < FN * FT; blk += NW) {
        f32x4_t sum = s_acc[0][blk][lane];
#pragma unroll
        for (int v = 1; v < NW; ++v) sum += s_acc[v][blk][lane];
        const int n = n0 + 16 * (blk / FT) + 4 * lg, t = 16 * (blk % FT) + lr;
        if (t < grp.rows && n < p.N) {  // (N is a multiple of 8: the four are in or out together)
            char* at = p.y + ((grp.first + t) * p.ldy + n) * Frag<DT>::kBytes;
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
