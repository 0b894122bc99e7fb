// contract_wide.h -- token contraction of the backward from saved 8-bit rows
// for adapters of rank above 16 (gfx950).
//
// The sums of contract.h,
//   dA_a[k][c] += s_a * sum_rows g[row][k] * x[row][c]      (c < d_in)
//   dB_a[c][k] += s_a * sum_rows dy[row][c] * v[row][k]     (c < d_out)
// with a tile of 256 columns x up to 16 MB ranks (MB = 2 or 4).  contract.h's
// tile is 64 columns x 16 ranks and its waves split the rows, so a rank-64
// adapter reads its dY and x windows four times and its g and v windows once
// for every 64 columns.  Here each of the four waves owns 64 columns and all walk
// the same windows: x and dY are read once, and the g / v windows once per 256
// columns: wave mb loads rank block mb of them, makes it an operand and leaves it
// in LDS for the others (one barrier a window).  No sum crosses waves.  The price
// is larger partial tiles where workgroup ranges cut a tile.
//
// A window of an adapter with more rank blocks takes longer: the split of the
// work into equal ranges counts 2 + blocks for each.
#pragma once

#include "contract.h"

namespace lora {

constexpr int kWideCols = 256;

template <int DT, int MB>
struct WideLds {
    static constexpr int kTiles = ContractLds<DT, 4>::kTransBytes;
    static constexpr int kOp = sizeof(F32Full<DT>) / 16;  // 16-byte parts of an operand
    static constexpr int kBytes = kTiles + 2 * MB * kOp * kWave * 16;
};

constexpr int wide_fix_floats(int mb) { return 4 * mb * 4 * kWave * 4; }  // a partial tile

// One active adapter's units: rank groups x 256-column blocks x 32-row windows
// x a window's weight.
struct WideAct {
    int a, rgroups, nwin, lo, hi, weight;
    int64_t units;
};
template <int MB>
__device__ __forceinline__ WideAct wide_act(const ContractParams& p, int i, int ncb) {
    const ContractAct c = contract_act(p, i, ncb);  // (counts groups of 16 ranks)
    WideAct w{c.a, (c.rgroups + MB - 1) / MB, c.nwin, c.lo, c.hi, 2 + min(MB, c.rgroups), 0};
    w.units = (int64_t)w.rgroups * ncb * w.nwin * w.weight;
    return w;
}

// The columns of wave tile wt of column block cb_all.
struct WideCols {
    bool is_dA;
    int c0, N;
};
__device__ __forceinline__ WideCols wide_cols(const ContractParams& p, int cb_all, int wt) {
    WideCols w;
    w.is_dA = cb_all < p.ncb_in;
    w.N = w.is_dA ? p.d_in : p.d_out;
    w.c0 = (w.is_dA ? cb_all : cb_all - p.ncb_in) * kWideCols + 64 * wt;
    return w;
}

// One 16-rank x 16-column block of dA / dB (lane: 4 ranks, 1 column): where it
// lies and what is there.
struct WideOld {
    float* dst[4];
    bool ok[4], vec;  // vec: the lane's four ranks are 16 consecutive bytes of dB
    f32x4_t old;
    __device__ __forceinline__ void load(const WideCols& w, const lora_adapter& ad, const lora_adapter_grad& gr, int rank,
                                         int nb, int lr, int lg, int d_in) {
        const int col = w.c0 + 16 * nb + lr;
        const int r = ad.rank;
        vec = !w.is_dA && (r & 3) == 0 && ((uintptr_t)gr.dB & 15u) == 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int rk = rank + 4 * lg + i;
            ok[i] = col < w.N && rk < r;
            const int rk_ = ok[i] ? rk : 0, col_ = ok[i] ? col : 0;
            dst[i] = w.is_dA ? gr.dA + (int64_t)rk_ * d_in + col_ : gr.dB + (int64_t)col_ * r + rk_;
        }
        if (vec) {
            old = *gptr(reinterpret_cast<const f32x4_t*>(dst[0]));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) old[i] = *gptr(dst[i]);
        }
    }
    // s * sum is added to it
    __device__ __forceinline__ void add(float s, f32x4_t sum) const {
        if (vec) {
            if (ok[0]) *gptr(reinterpret_cast<f32x4_t*>(dst[0])) = old + s * sum;
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (ok[i]) *gptr(dst[i]) = old[i] + s * sum[i];
    }
};

// Body of workgroup blk of G (four waves); p.ncb_in / ncb_out count 256-column
// blocks and p.fix holds wide_fix_floats(MB) a slot.  s_mem: WideLds<DT, MB>.
template <int DT, int MB>
__device__ __forceinline__ void contract_wide_body(const ContractParams& p, int blk, int G, char* s_mem) {
    if (p.stop && *p.stop) return;
    const int wave = wave_id();
    const int lane = threadIdx.x & (kWave - 1);
    const int lr = lane & 15;
    const int lg = lane >> 4;
    const int ncb = p.ncb_in + p.ncb_out;
    const int n_act = p.sched[2];
    const int vg = (blk % kNumXcd) * (G / kNumXcd) + blk / kNumXcd;
    int32_t* meta = p.fix_meta + (int64_t)vg * 2 * kFixMeta;
    if (threadIdx.x == 0) {
        meta[0] = -1;
        meta[kFixMeta] = -1;
    }
    // Total units; workgroup 0 counts the bad entries.
    int64_t U = 0;
    for (int b = 0; b < n_act; b += kWave) {
        const int i = b + lane;
        WideAct c{};
        if (i < n_act) c = wide_act<MB>(p, i, ncb);
        U += uniform64(wave_sum64(c.units));
        if (blk == 0 && wave == 0 && i < n_act && c.rgroups == 0) atomicAdd(p.err, 1);
    }
    const int64_t begin = U * vg / G;
    const int64_t end = U * (vg + 1) / G;
    if (begin >= end) {
        if (threadIdx.x == 0) meta[0] = -2;
        return;
    }
    // The active adapter holding unit `begin` and the units before it.
    int act = 0;
    int64_t abase = 0;
    for (int b = 0; b < n_act; b += kWave) {
        const int i = b + lane;
        const int64_t un = i < n_act ? wide_act<MB>(p, i, ncb).units : 0;
        int64_t incl = un;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const int64_t o = __shfl_up(incl, d, kWave);
            if (lane >= d) incl += o;
        }
        const uint64_t hit = __ballot(i < n_act && abase + incl - un <= begin && begin < abase + incl);
        if (hit) {
            const int l = __ffsll((long long)hit) - 1;
            act = b + l;
            abase += uniform64(__shfl(incl - un, l, kWave));
            break;
        }
        abase += uniform64(__shfl(incl, kWave - 1, kWave));
    }

    using OP = F32Full<DT>;
    constexpr int kOp = WideLds<DT, MB>::kOp;
    char* tile0 = s_mem + 2 * wave * ContractLds<DT, 4>::kTileBytes;
    u32x4_t* s_op = reinterpret_cast<u32x4_t*>(s_mem + WideLds<DT, MB>::kTiles);  // [2][MB][kOp][lane]
    const int lrow = 4 * (lane >> 3);
    const int lcol = 8 * (lane & 7);
    auto act_uniform = [&](int i) {
        WideAct c = wide_act<MB>(p, i, ncb);
        c.a = __builtin_amdgcn_readfirstlane(c.a);
        c.rgroups = __builtin_amdgcn_readfirstlane(c.rgroups);
        c.nwin = __builtin_amdgcn_readfirstlane(c.nwin);
        c.lo = __builtin_amdgcn_readfirstlane(c.lo);
        c.hi = __builtin_amdgcn_readfirstlane(c.hi);
        c.weight = __builtin_amdgcn_readfirstlane(c.weight);
        c.units = uniform64(c.units);
        return c;
    };

    WideAct c = act_uniform(act);
    int slot = 0;
    for (int64_t u = begin; u < end;) {
        if (u >= abase + c.units) {  // next adapter
            abase += c.units;
            if (abase >= end) break;
            c = act_uniform(++act);
            continue;
        }
        // The windows of this tile that begin in [u, end): a window belongs to the
        // workgroup whose range holds its first unit.
        const int64_t local = u - abase;
        const int64_t tile_units = (int64_t)c.nwin * c.weight;
        const int tile_in = (int)(local / tile_units);  // rank group major, then column block
        const int64_t tile_u = abase + tile_in * tile_units;
        const int w0 = (int)((u - tile_u + c.weight - 1) / c.weight);
        const int w1 = (int)min((int64_t)c.nwin, (end - tile_u + c.weight - 1) / c.weight);
        u = min(end, tile_u + tile_units);
        if (w0 >= w1) continue;
        const int rg = tile_in / ncb;
        const int cb_all = tile_in - rg * ncb;
        const lora_adapter ad = load_adapter(p.adapters, c.a);
        const lora_adapter_grad gr = load_grad(p.grads, c.a);
        const WideCols wc = wide_cols(p, cb_all, wave);
        const int r = ad.rank;
        const int rank0 = rg * 16 * MB;
        const int nmb = min(MB, (r - rank0 + 15) / 16);
        const char* q = static_cast<const char*>(wc.is_dA ? p.x : p.dy);
        const int64_t ldq = wc.is_dA ? p.ldx : p.lddy;
        // this wave's rank block of g / v (ranks past r: discarded rows)
        const float* prow = (wc.is_dA ? p.gT : p.vT) + (int64_t)min(rank0 + 16 * min(wave, nmb - 1) + lr, r - 1) * p.ldT;
        // Columns past N (N is a multiple of 8) read column block 0 of the row; never written back.
        const int col = wc.c0 + lcol < wc.N ? wc.c0 + lcol : 0;
        const int lo = c.lo;
        const int hi = c.hi;
        const int wa = (lo & ~31) + 32 * w0;
        const int nw = w1 - w0;

        f32x4_t acc[MB][4];
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int nb = 0; nb < 4; ++nb) acc[mb][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        // Two windows in flight, row indices two further ahead; past the range the
        // last window again (loaded, never multiplied).
        auto windows = [&](auto q8) {
            constexpr bool Q8 = decltype(q8)::value;
            constexpr bool NT = !Q8 && DT == LORA_BF16;
            struct Win {
                std::conditional_t<Q8, QuantRaw, Frag<DT>> q[4];
                f32x4_t pv[2];
            };
            auto win_at = [&](int i) { return wa + 32 * (i < nw ? i : nw - 1); };
            auto load = [&](Win& W, const int32_t* rows, int i) {
                contract_load_q<DT, NT, Q8>(W.q, q, ldq, p.xs, p.ldxs, rows, col);
                const LORA_GLOBAL f32x4_t* src = gptr(reinterpret_cast<const f32x4_t*>(prow + win_at(i) + 8 * lg));
                W.pv[0] = src[0];
                W.pv[1] = src[1];
            };
            // Window i from W, its tile and operands in buffer half; then W takes window i + 2.
            auto window = [&](Win& W, int32_t* rows, int half, int i) {
                char* tile = tile0 + half * ContractLds<DT, 4>::kTileBytes;
                u32x4_t* ops = s_op + half * MB * kOp * kWave;
                contract_tile_write<DT, Q8>(W.q, tile, lcol, lrow);
                if (wave < nmb) {
                    const int pp = win_at(i) + 8 * lg;
                    float f[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = (pp + e >= lo && pp + e < hi) ? W.pv[e >> 2][e & 3] : 0.f;
                    const OP po = OP::make(f);
#pragma unroll
                    for (int k = 0; k < kOp; ++k)
                        ops[(wave * kOp + k) * kWave + lane] = reinterpret_cast<const u32x4_t*>(&po)[k];
                }
                load(W, rows, i + 2);
                contract_rows(rows, p.perm, win_at(i + 4), lo, hi, lrow);
                // (the other half's operands are read before the next barrier, and
                // written again after it)
                lds_barrier();
                Frag<DT> qf[4];
                contract_tile_read<DT>(qf, tile, lane);
#pragma unroll
                for (int mb = 0; mb < MB; ++mb) {
                    if (mb < nmb) {
                        OP po;
#pragma unroll
                        for (int k = 0; k < kOp; ++k)
                            reinterpret_cast<u32x4_t*>(&po)[k] = ops[(mb * kOp + k) * kWave + lane];
#pragma unroll
                        for (int nb = 0; nb < 4; ++nb) acc[mb][nb] = po.mma_left(qf[nb], acc[mb][nb]);
                    }
                }
            };
            int32_t rowsA[4], rowsB[4];
            Win WA, WB;
            // (in the loop's order: loads in another order would make the loop wait
            // for all of them, every time, before it can use its row indices)
            contract_rows(rowsA, p.perm, win_at(0), lo, hi, lrow);
            contract_rows(rowsB, p.perm, win_at(1), lo, hi, lrow);
            __builtin_amdgcn_sched_barrier(0);
            load(WA, rowsA, 0);
            __builtin_amdgcn_sched_barrier(0);
            contract_rows(rowsA, p.perm, win_at(2), lo, hi, lrow);
            __builtin_amdgcn_sched_barrier(0);
            load(WB, rowsB, 1);
            __builtin_amdgcn_sched_barrier(0);
            contract_rows(rowsB, p.perm, win_at(3), lo, hi, lrow);
            __builtin_amdgcn_sched_barrier(0);
            int i = 0;
            for (; i + 1 < nw; i += 2) {
                window(WA, rowsA, 0, i);
                window(WB, rowsB, 1, i + 1);
            }
            if (i < nw) window(WA, rowsA, 0, i);
        };
        if (wc.is_dA)
            windows(std::true_type{});
        else
            windows(std::false_type{});
        lds_barrier();  // the next tile writes the buffers from half 0 again

        const bool whole = w0 == 0 && w1 == c.nwin;
        f32x4_t* f = reinterpret_cast<f32x4_t*>(p.fix + ((int64_t)vg * 2 + slot) * wide_fix_floats(MB));
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            if (mb < nmb) {
                if (whole) {
                    WideOld old[4];
#pragma unroll
                    for (int nb = 0; nb < 4; ++nb) old[nb].load(wc, ad, gr, rank0 + 16 * mb, nb, lr, lg, p.d_in);
#pragma unroll
                    for (int nb = 0; nb < 4; ++nb) old[nb].add(ad.scale, acc[mb][nb]);
                } else {
#pragma unroll
                    for (int nb = 0; nb < 4; ++nb) *gptr(f + ((wave * MB + mb) * 4 + nb) * kWave + lane) = acc[mb][nb];
                }
            }
        }
        if (!whole && threadIdx.x == 0) {
            int32_t* m = meta + slot * kFixMeta;
            m[0] = (int32_t)(tile_u & 0x7fffffff);  // the tile's first unit: its id
            m[1] = (int32_t)(tile_u >> 31);
            m[2] = c.a;
            m[3] = rg;
            m[4] = cb_all;
            m[5] = w0 == 0 ? nmb : 0;  // owner: holds the tile's first window, runs its fix-up
        }
        slot = 1;  // only a workgroup's first and last tiles can be cut
    }
    if (slot == 0 && threadIdx.x == 0) meta[0] = -2;  // a range without a window's first unit: the fix-up steps over it
}

// Adds the partial tiles of each cut tile in workgroup order, then s times the
// sum to dA / dB.  Workgroup (g, wave tile, rank block): the tile that g owns (one at most:
// a range that owns a cut tile ends in it), 64 of its columns and 16 of its
// ranks; wave nb takes 16 columns.  Latency-bound, so what does not need each other is loaded together:
// the records of g and the workgroups after it, then the partial tiles, the
// table entries and the old values (2048 rows of ranks 8 to 64, 4096 -> 14336:
// 8.9 us in place of 13.2).
template <int MB>
__global__ __launch_bounds__(4 * kWave) void contract_wide_fixup_kernel(ContractParams p, int G) {
    if (p.stop && *p.stop) return;
    const int g0 = blockIdx.x, wt = blockIdx.y, mb = blockIdx.z;
    const int nb = wave_id();
    const int lane = threadIdx.x & (kWave - 1);
    // Lane j: the record of workgroup g + j (its first slot); past the grid none.
    auto record = [&](int g, int32_t& m0, int32_t& m1) {
        const bool in = g + lane < G;
        const int32_t* mg = p.fix_meta + (int64_t)(in ? g + lane : g0) * 2 * kFixMeta;
        m0 = in ? mg[0] : -3;
        m1 = mg[1];
    };
    int32_t m0, m1;
    record(g0 + 1, m0, m1);
    const int32_t* m = p.fix_meta + (int64_t)g0 * 2 * kFixMeta;
    const int sl = m[0] >= 0 && m[5] ? 0 : 1;
    m += sl * kFixMeta;
    if (m[0] < 0 || mb >= m[5]) return;
    const int32_t id0 = m[0], id1 = m[1];
    const WideCols wc = wide_cols(p, m[4], wt);
    if (wc.c0 >= wc.N) return;
    auto part = [&](int slot) {
        const f32x4_t* f = reinterpret_cast<const f32x4_t*>(p.fix + (int64_t)slot * wide_fix_floats(MB));
        return *gptr(f + ((wt * MB + mb) * 4 + nb) * kWave + lane);
    };
    const lora_adapter ad = load_adapter(p.adapters, m[2]);
    const lora_adapter_grad gr = load_grad(p.grads, m[2]);
    f32x4_t sum = part(g0 * 2 + sl);
    WideOld old;
    old.load(wc, ad, gr, (m[3] * MB + mb) * 16, nb, lane & 15, lane >> 4, p.d_in);
    // The later workgroups holding the tile form a run after g0, those without
    // units (-2) among them; their partial tiles are loaded two at a time (past the
    // run the last one again) and added in workgroup order.
    for (int g = g0 + 1; g < G; g += kWave) {
        if (g > g0 + 1) record(g, m0, m1);
        const bool same = m0 == id0 && m1 == id1;
        const uint64_t same_mask = __ballot(same);
        const uint64_t end_mask = __ballot(!same && m0 != -2);  // another tile, or past the grid
        const int n = end_mask ? __ffsll((long long)end_mask) - 1 : kWave;
        for (int j0 = 0; j0 < n; j0 += 2) {
            f32x4_t pv[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) pv[j] = part((g + min(j0 + j, n - 1)) * 2);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (j0 + j < n && ((same_mask >> (j0 + j)) & 1)) sum += pv[j];
        }
        if (n < kWave) break;
    }
    old.add(ad.scale, sum);
}

}  // namespace lora
