// base.h -- the frozen base product from 8-bit rows and an 8-bit weight (gfx950).
//
//   y_t (+)= sum_k x_tk W_nk
//
// with x and W as codes times power-of-two block scales (quant.h).
//
// bf16 y: one v_mfma_scale_f32_16x16x128_f8f6f4 takes exactly one block of 128
// along k for 16 outputs and 16 rows: its operands are codes as stored, its two
// exponent bytes a lane are the scales of the lane's weight row and activation
// row, and its sums stay in fp32 registers from the first block to the last.
// The instruction cuts each product of a group of 8 (k-consecutive codes of a
// lane) at 2^-13 of the power of two of the group's largest, and adds groups in
// fp32 (measured on the device: products 2^16 and 2^3 in a group give both, 2^16
// and 2^2 only the first; 14 counts as 8 there; in different groups 2^-7 is
// kept).  The power of two is the sum of the factors' exponents, and a subnormal
// code's is that of 2^-6: beside 2^-9 * 256 products down to 2^-10 of it are kept,
// beside 1 * 256 down to 2^-13 (a zero does not count).  On normal data the cut is
// 1.5e-5 of the result, with outliers in 1% of the codes 5e-5: a hundredth of y's
// rounding to bf16 (1.7e-3), for twice the rate of the bf16 instruction.
//
// fp32 y: the codes times their scales are bf16 numbers, and
// v_mfma_f32_16x16x32_bf16 sums their exact products in fp32.
//
// A operand = weight rows (n), B operand = activation rows (t), so a lane ends
// with four operand rows of one t.  Which weight row is which operand row is
// free as well: blocks are taken in pairs of 32 rows, operand row 4 g + i of
// block b of the pair is row 8 g + 4 b + i, so a lane's two times four outputs
// are eight consecutive n (one 16-byte store of bf16).  The order of the 128 products inside
// a block is free (both operands take the same one): lane group g = lane / 16
// takes the 16-byte units g and g + 4 of each 128-byte block row.
#pragma once

#include <type_traits>

#include "base_plan.h"
#include "quant.h"

namespace lora {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

struct BaseParams {
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
    int32_t T, N, nkb;  // rows, outputs, blocks of 128 along k
    int32_t accumulate;
    int32_t tiles_n, tiles_t;
    int32_t splits;  // parts of k, each a workgroup's; more than one: fp32 sums to part
    float* part;     // [splits][T][N]
};

// One operand row's block of 128: this lane's 32 codes.
struct QuantOperand {
    u32x4_t u[2];
};
// The same as an operand of the matrix instruction.  The scale comes as a word
// of four blocks' bytes and the place Q of this block's byte in it.
template <int DT>
struct QuantFrag;
template <>
struct QuantFrag<LORA_BF16> {
    i32x8_t codes;
    int scale;
    template <int Q>
    __device__ __forceinline__ static QuantFrag make(const QuantOperand& o, uint32_t scale) {
        return QuantFrag{__builtin_bit_cast(i32x8_t, __builtin_shufflevector(o.u[0], o.u[1], 0, 1, 2, 3, 4, 5, 6, 7)),
                         (int)scale};
    }
    template <int Q>
    __device__ __forceinline__ f32x4_t mma(const QuantFrag& b, f32x4_t c) const {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(codes, b.codes, c, 0, 0, Q, scale, Q, b.scale);
    }
};
template <>
struct QuantFrag<LORA_F32> {
    Frag<LORA_BF16> q[4];
    template <int Q>
    __device__ __forceinline__ static QuantFrag make(const QuantOperand& o, uint32_t scale) {
        const float s = quant_scale((scale >> (8 * Q)) & 255u);
        return QuantFrag{{dequant8<LORA_BF16>(o.u[0][0], o.u[0][1], s), dequant8<LORA_BF16>(o.u[0][2], o.u[0][3], s),
                          dequant8<LORA_BF16>(o.u[1][0], o.u[1][1], s), dequant8<LORA_BF16>(o.u[1][2], o.u[1][3], s)}};
    }
    template <int Q>
    __device__ __forceinline__ f32x4_t mma(const QuantFrag& b, f32x4_t c) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) c = lora::mma(q[i], b.q[i], c);
        return c;
    }
};

// Four consecutive outputs of one row: what is there, and its sum with v (in
// fp32, rounded once) stored.
template <int DT>
__device__ __forceinline__ f32x4_t base_load4(const BaseParams& p, int64_t t, int n) {
    const char* at = p.y + (t * p.ldy + n) * Frag<DT>::kBytes;
    if constexpr (DT == LORA_BF16) {
        const u32x2_t o = *gptr(reinterpret_cast<const u32x2_t*>(at));
        return f32x4_t{__uint_as_float(o[0] << 16), __uint_as_float(o[0] & 0xffff0000u), __uint_as_float(o[1] << 16),
                       __uint_as_float(o[1] & 0xffff0000u)};
    } else {
        return *gptr(reinterpret_cast<const f32x4_t*>(at));
    }
}
template <int DT>
__device__ __forceinline__ void base_store4(const BaseParams& p, int64_t t, int n, f32x4_t v, f32x4_t old) {
    char* at = p.y + (t * p.ldy + n) * Frag<DT>::kBytes;
    if (p.accumulate) v += old;
    if constexpr (DT == LORA_BF16)
        *gptr(reinterpret_cast<u32x2_t*>(at)) = u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    else
        *gptr(reinterpret_cast<f32x4_t*>(at)) = v;
}

// ------------------------------------------------------------------ tiles through LDS
//
// A workgroup of WN x WT waves computes BN outputs x BT rows.  A step is one
// block of 128 along k: BN + BT block rows of 128 bytes go from memory straight
// into LDS, ST stages in a ring, the loads of step i + ST - 1 issued while step
// i is multiplied.  Unit c (16 bytes) of a row lies at position c ^ s of the
// row, s the operand row modulo 8 that the row becomes, so that the rows that a
// read takes together fall on different banks.
// The scales of up to BaseLds::kGroups * 4 blocks lie in LDS too, four blocks'
// bytes of one row in a word; a longer k is taken in pieces.

constexpr int kBand = 4;

template <int BN, int BT, int WN, int WT, int ST, int DT>
__global__ __launch_bounds__(WN* WT* kWave) void base_kernel(BaseParams p) {
    using L = BaseLds<BN, BT, ST>;
    constexpr int NW = WN * WT;
    constexpr int FN = BN / WN / 16, FT = BT / WT / 16;  // 16 x 16 blocks of a wave
    constexpr int GA = 2, NG = FN / GA;         // weight blocks of a group, groups
    constexpr int WU = 4 / WT, XU = BT / 8 / NW;  // loads of a wave per weight group, for the activations
    constexpr int PW = NG * WU + XU;            // of a step
    constexpr int NB = L::kNB;                  // 128-row blocks of the weight tile
    static_assert(FN % 2 == 0 && NW % 4 == 0 && 4 % WT == 0 && BT % (8 * NW) == 0, "the loads divide evenly");
    static_assert(BN / WN <= kQBlock, "a wave's outputs lie in one block of 128 weight rows");
    __shared__ __attribute__((aligned(16))) char s_lds[L::kBytes];
    uint32_t* s_xs = reinterpret_cast<uint32_t*>(s_lds + ST * L::kStage);  // [group][BT]
    uint32_t* s_ws = s_xs + L::kGroups * BT;                              // [128-row block][64 groups]

    const int wave = wave_id();
    const int lane = threadIdx.x & (kWave - 1);
    const int lr = lane & 15, lg = lane >> 4;
    // Workgroups of one XCD take neighbouring tiles.
    const int ntile = p.tiles_n * p.tiles_t * p.splits;
    const int per = (ntile + kNumXcd - 1) / kNumXcd;
    const int task = (int)(blockIdx.x % kNumXcd) * per + (int)(blockIdx.x / kNumXcd);
    if ((int)(blockIdx.x / kNumXcd) >= per || task >= ntile) return;
    const int tile = task / p.splits, part = task - tile * p.splits;
    // this workgroup's blocks along k: whole words of scales
    const int ngr = (p.nkb + 3) / 4;
    const int kb0 = 4 * (int)((int64_t)ngr * part / p.splits);
    const int kb1 = min(p.nkb, 4 * (int)((int64_t)ngr * (part + 1) / p.splits));
    // Order of the tiles: bands of up to kBand tiles along t, walked along n, so
    // that the 32 tiles in flight on an XCD share few weight and activation rows.
    const int band = tile / (kBand * p.tiles_n), in = tile - band * kBand * p.tiles_n;
    const int bt = min(kBand, p.tiles_t - band * kBand);
    const int n0 = in / bt * BN, t0 = (band * kBand + in % bt) * BT;
    const int wn = (wave % WN) * (BN / WN), wt = (wave / WN) * (BT / WT);

    // The loads of a stage, 8 rows each: WU a wave for the weight rows that the
    // waves read as group g (rows 32 g .. + 31 of every wave column), XU for the
    // activation rows.  Rows past the matrix lie past their buffer: nothing is
    // fetched for them, and their outputs are not stored.
    const int nrows = min(BN, p.N - n0), trows = min(BT, p.T - t0);
    const buf_rsrc_t rw = make_rsrc(p.w + (int64_t)n0 * p.ldw, (uint32_t)((nrows - 1) * p.ldw + (int64_t)p.nkb * kQBlock));
    const buf_rsrc_t rx = make_rsrc(p.x + (int64_t)t0 * p.ldx, (uint32_t)((trows - 1) * p.ldx + (int64_t)p.nkb * kQBlock));
    const int w_row = wave / 4 * (BN / WN) + 8 * (wave & 3), x_row = 8 * wave, r8 = lane >> 3;
    const uint32_t vw = (uint32_t)((w_row + r8) * p.ldw) + (uint32_t)((lane & 7) ^ (r8 & 3) ^ (wave & 1) * 4) * 16u;
    const uint32_t vx = (uint32_t)((x_row + r8) * p.ldx) + (uint32_t)((lane & 7) ^ r8) * 16u;
    // Load o of a stage: those of weight group 0, of the activations, of weight groups 1, 2, ...
    auto issue = [&](int o, int slot, int kb) {
        const bool w = o < WU || o >= WU + XU;
        const int ow = o < WU ? o : o - XU;
        const int row = w ? 32 * (ow / WU) + NW / 4 * (ow % WU) * (BN / WN) : 8 * NW * (o - WU);
        char* at = s_lds + slot * L::kStage + (w ? w_row + row : BN + x_row + row) * kQBlock;
        if (w)
            dma_lds(rw, vw + (uint32_t)(row * p.ldw), (uint32_t)kb * kQBlock, at, 16);
        else
            dma_lds(rx, vx + (uint32_t)(row * p.ldx), (uint32_t)kb * kQBlock, at, 16);
    };

    f32x4_t acc[FN][FT];
#pragma unroll
    for (int a = 0; a < FN; ++a)
#pragma unroll
        for (int b = 0; b < FT; ++b) acc[a][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    // This lane's operand bytes of a block row: units lg and lg + 4.
    const int lrow = lr * kQBlock + ((lg ^ (lr & 7)) * 16);
    const int lrow_w = (8 * (lr >> 2) + (lr & 3)) * kQBlock + ((lg ^ (lr & 7)) * 16);
    QuantOperand b[FT], a[2][GA];
    uint32_t xs[FT], ws;  // scale words
    // half u of a block row: unit lg (u = 0) or lg + 4 (u = 1)
    auto read_b = [&](int f, int u, int slot) {
        b[f].u[u] = *reinterpret_cast<const u32x4_t*>(s_lds + slot * L::kStage + (BN + wt + 16 * f) * kQBlock +
                                                      (u ? lrow ^ 64 : lrow));
    };
    auto read_a = [&](QuantOperand* q, int f, int u, int slot, int grp) {
        const int blk = GA * grp + f;
        q[f].u[u] = *reinterpret_cast<const u32x4_t*>(s_lds + slot * L::kStage + (wn + 32 * (blk / 2) + 4 * (blk & 1)) * kQBlock +
                                                      (u ? lrow_w ^ 64 : lrow_w));
    };
    auto read_xs = [&](int f, int grp) { xs[f] = s_xs[grp * BT + wt + 16 * f + lr]; };
    auto read_ws = [&](uint32_t& to, int grp) { to = s_ws[wn / kQBlock * kWave + grp]; };

    for (int k0 = kb0; k0 < kb1; k0 += 4 * L::kGroups) {
        const int nk = min(kb1 - k0, 4 * L::kGroups);  // steps of this piece
        const int ng = (nk + 3) / 4;
        if (k0 > kb0) {
            wait_vmcnt_le<0>();
            lds_barrier();  // the last piece's stages and scales are no longer read
        }
        // scale words, a load for 64 rows of one group (activations) or for the
        // groups of one 128-row block (weight); past the matrix: the last row's
        for (int c = wave; c < ng * (BT / kWave); c += NW) {
            const int g = c / (BT / kWave), t = c % (BT / kWave) * kWave;
            lds_dma4_async(p.xs + (int64_t)(t0 + min(t + lane, trows - 1)) * p.ldxs + k0 + 4 * g, s_xs + g * BT + t);
        }
        if (wave < NB) {
            const int nblk = min(n0 + kQBlock * wave, p.N - 1) / kQBlock;
            lds_dma4_async(p.ws + (int64_t)nblk * p.ldws + k0 + 4 * min(lane, ng - 1), s_ws + wave * kWave);
        }
        // (loads past the piece repeat its last block: every step waits for the same number)
#pragma unroll
        for (int s = 0; s < ST; ++s)
#pragma unroll
            for (int o = 0; o < PW; ++o) issue(o, s, k0 + min(s, nk - 1));
        wait_vmcnt_le<PW*(ST - 1)>();
        lds_barrier();
#pragma unroll
        for (int f = 0; f < GA; ++f)
#pragma unroll
            for (int u = 0; u < 2; ++u) read_a(a[0], f, u, 0, 0);
#pragma unroll
        for (int f = 0; f < FT; ++f) {
            read_b(f, 0, 0);
            read_b(f, 1, 0);
            read_xs(f, 0);
        }
        read_ws(ws, 0);
        int slot = 0;
        // One step (Q: its number modulo 4).  The weight blocks are taken GA at a
        // time; while a group is multiplied the next one is read, and with the
        // last group the next step's first group and activations.  After the
        // barrier at the start of group g every wave has that group in registers,
        // so its place in the stage is free (with group 0 the activations' too) and
        // the loads of step i + ST can go there, spread over the groups: they have
        // nearly ST steps to land, not ST - 1 as with one barrier and all loads at
        // the step's end (4096 rows, 14336 -> 4096: 166 against 188 us).
        // Reads and loads go between products, a few at a time: a burst after the
        // barrier would leave the matrix cores without work meanwhile.
        // the loads of a step that go out before its group g
        constexpr auto before = [](int g) { return PW * g / NG; };
        auto step = [&](auto quarter, int i) {
            constexpr int Q = decltype(quarter)::value;
            const int next = slot + 1 == ST ? 0 : slot + 1;
            const int kn = k0 + min(i + ST, nk - 1);
            uint32_t ws_next = ws;
            auto group = [&](auto gc) {
                constexpr int g = decltype(gc)::value;
                constexpr bool last = g + 1 == NG;
                QuantOperand* cur = a[(Q * NG + g) & 1];
                QuantOperand* nxt = a[(Q * NG + g + 1) & 1];
                // What is read now has to be there: the loads issued after it may be
                // outstanding.
                wait_vmcnt_le<last ? (NG - 1) * WU + (ST - 2) * PW + before(NG - 1)
                                   : (NG - 2 - g) * WU + (ST - 1) * PW + before(g)>();
                lds_barrier();
                QuantFrag<DT> af[GA];
#pragma unroll
                for (int f = 0; f < GA; ++f) af[f] = QuantFrag<DT>::template make<Q>(cur[f], ws);
#pragma unroll
                for (int h = 0; h < FT; ++h) {
                    const QuantFrag<DT> bf = QuantFrag<DT>::template make<Q>(b[h], xs[h]);
#pragma unroll
                    for (int f = 0; f < GA; ++f)
                        acc[GA * g + f][h] = af[f].template mma<Q>(bf, acc[GA * g + f][h]);
#pragma unroll
                    for (int r = h * 2 * GA / FT; r < (h + 1) * 2 * GA / FT; ++r)
                        read_a(nxt, r >> 1, r & 1, last ? next : slot, last ? 0 : g + 1);
                    if (last) {
                        read_b(h, 0, next);
                        read_b(h, 1, next);
                        if (Q == 3) read_xs(h, min(i + 1, nk - 1) >> 2);
                        if (Q == 3 && h == 0) read_ws(ws_next, min(i + 1, nk - 1) >> 2);
                    }
                    constexpr int o0 = before(g), n = before(g + 1) - o0;
#pragma unroll
                    for (int o = o0 + h * n / FT; o < o0 + (h + 1) * n / FT; ++o) issue(o, slot, kn);
                    __builtin_amdgcn_sched_barrier(0);
                }
            };
            group(std::integral_constant<int, 0>{});
            if constexpr (NG > 1) group(std::integral_constant<int, 1 % NG>{});
            if constexpr (NG > 2) group(std::integral_constant<int, 2 % NG>{});
            if constexpr (NG > 3) group(std::integral_constant<int, 3 % NG>{});
            static_assert(NG <= 4, "groups");
            ws = ws_next;
            slot = next;
        };
        for (int i = 0; i < nk; i += 4) {
            step(std::integral_constant<int, 0>{}, i);
            if (i + 1 < nk) step(std::integral_constant<int, 1>{}, i + 1);
            if (i + 2 < nk) step(std::integral_constant<int, 2>{}, i + 2);
            if (i + 3 < nk) step(std::integral_constant<int, 3>{}, i + 3);
        }
    }
    wait_vmcnt_le<0>();  // nothing may land in LDS after the workgroup has ended
#pragma unroll
    for (int h = 0; h < FT; ++h) {
        const int t = t0 + wt + 16 * h + lr;
        const bool t_in = t < p.T;
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
        // Eight outputs at a time, added to what is there in fp32 and rounded once;
        // the old values of a row are loaded together (outputs past the matrix load
        // its first ones).
        char* row = p.y + (t_in ? t : 0) * p.ldy * Frag<DT>::kBytes;
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
            for (int e = 0; e < 8; ++e)
                v[e] = acc[f + e / 4][h][e & 3] + (p.accumulate ? old[f / 2][e] : 0.f);
            if (t_in && n < p.N) Elem<DT>::store8(row + (int64_t)n * Frag<DT>::kBytes, v);
        }
    }
}

// The sum of the parts of a split k, in order, as base_kernel stores it: a
// thread takes four outputs of a row, kParts parts in flight (the last again past
// the end; with a load at a time a product of 45 x 12992 x 472, then in 17 parts,
// took 14.6 us in place of 8.6; in 13 parts, as it is split now, 9.2).
constexpr int kSumThreads = 256, kParts = 8;
template <int DT>
__global__ __launch_bounds__(kSumThreads) void base_sum_kernel(BaseParams p) {
    const int64_t q = (int64_t)p.T * (p.N / 4);
    for (int64_t i = (int64_t)blockIdx.x * kSumThreads + threadIdx.x; i < q; i += (int64_t)gridDim.x * kSumThreads) {
        const LORA_GLOBAL f32x4_t* src = gptr(reinterpret_cast<const f32x4_t*>(p.part)) + i;
        const int64_t t = i / (p.N / 4);
        const int n = 4 * (int)(i - t * (p.N / 4));
        const f32x4_t old = p.accumulate ? base_load4<DT>(p, t, n) : f32x4_t{0.f, 0.f, 0.f, 0.f};
        f32x4_t sum = src[0];
        for (int s0 = 1; s0 < p.splits; s0 += kParts) {
            f32x4_t v[kParts];
#pragma unroll
            for (int j = 0; j < kParts; ++j) v[j] = src[min(s0 + j, p.splits - 1) * q];
#pragma unroll
            for (int j = 0; j < kParts; ++j)
                if (s0 + j < p.splits) sum += v[j];
        }
        base_store4<DT>(p, t, n, sum, old);
    }
}

// ------------------------------------------------------------------ few rows: the weight as a stream
//
// Up to kStreamRows = 16 rows: the weight is read once, straight into operand registers,
// and nothing of it is shared between waves.  A workgroup of NW waves computes
// 16 outputs of every row; wave w takes the blocks w, w + NW, ... along k (a
// workgroup reads NW * 128 consecutive bytes of each of its 16 weight rows at a
// time) and the waves' sums are added in wave order through LDS.  kU blocks a
// wave are in flight at once (the next kU asked for before these are multiplied:
// 1 x 12232 x 352 11.0 us as without, 1 x 4096 x 14336 17.1 against 14.7).
constexpr int kU = 4;

template <int NW, int DT>
__global__ __launch_bounds__(NW* kWave) void base_stream_kernel(BaseParams p) {
    __shared__ f32x4_t s_acc[NW][kWave];
    const int wave = wave_id();
    const int lane = threadIdx.x & (kWave - 1);
    const int lr = lane & 15, lg = lane >> 4;
    const int n0 = blockIdx.x * 16;
    const LORA_GLOBAL uint8_t* w = gptr(p.w + (int64_t)min(n0 + lr, p.N - 1) * p.ldw + 16 * lg);
    const uint8_t* ws = p.ws + (int64_t)(n0 / kQBlock) * p.ldws;
    const int64_t row = min(lr, p.T - 1);
    const LORA_GLOBAL uint8_t* x = gptr(p.x + row * p.ldx + 16 * lg);
    const LORA_GLOBAL uint8_t* xs = gptr(p.xs + row * p.ldxs);
    f32x4_t acc{0.f, 0.f, 0.f, 0.f};
    for (int k0 = wave; k0 < p.nkb; k0 += NW * kU) {
        QuantOperand a[kU], b[kU];
        uint32_t as[kU], bs[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int kb = min(k0 + NW * u, p.nkb - 1);
            const int off = kb * kQBlock;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                a[u].u[i] = __builtin_nontemporal_load(reinterpret_cast<const LORA_GLOBAL u32x4_t*>(w + off + 64 * i));
            as[u] = cptr(ws)[kb];
#pragma unroll
            for (int i = 0; i < 2; ++i) b[u].u[i] = *reinterpret_cast<const LORA_GLOBAL u32x4_t*>(x + off + 64 * i);
            bs[u] = xs[kb];
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (k0 + NW * u < p.nkb) {
                const QuantFrag<DT> af = QuantFrag<DT>::template make<0>(a[u], as[u]);
                acc = af.template mma<0>(QuantFrag<DT>::template make<0>(b[u], bs[u]), acc);
            }
        }
    }
    s_acc[wave][lane] = acc;
    __syncthreads();
    if (wave == 0) {
        f32x4_t sum = s_acc[0][lane];
#pragma unroll
        for (int v = 1; v < NW; ++v) sum += s_acc[v][lane];
        const int t = lr, n = n0 + 4 * lg;
        if (t < p.T && n < p.N)  // (N is a multiple of 8: the four are in or out together)
            base_store4<DT>(p, t, n, sum, p.accumulate ? base_load4<DT>(p, t, n) : f32x4_t{0.f, 0.f, 0.f, 0.f});
    }
}

}  // namespace lora
