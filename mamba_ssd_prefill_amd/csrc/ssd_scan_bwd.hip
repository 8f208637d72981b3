// ssd_scan_bwd.hip -- the gradients of the selective scan (ssd_selective_scan_backward in
// include/mamba_ssd.h).  With g[n] the gradient of the state h[n] after token t,
//
//     g[n]  = C[n] dy + (exp(d A[n]) g[n] of token t+1),      dy = dout silu(z)
//     dC[n] = sum_c dy h[n],   dB[n] = sum_c g[n] d x         (over the channels of the group)
//     q[n]  = g[n] exp(d A[n]) h[n] of token t-1
//     dx = D dy + d sum_n g[n] B[n],   dd = x sum_n g[n] B[n] + sum_n A[n] q[n],   dA[n] = sum_t d q[n]
//
// A tile of 8 tokens is taken at a time, from the last to the first: the states of the tile are computed again
// from the saved state that enters it and kept in registers with their decays, and then the gradients run
// back through them.  Tiles of 16 tokens (half the saved states) needed twice the registers and LDS, and with
// two waves a SIMD instead of three the vector ALU waited: 360 us against 278 us at 2 x 2048 x 5120, N = 16, bf16.
// Bound by the vector ALU, which issues in 95% of the cycles there: 26 slots a (token, channel, n), 6 for the states and y
// again, 8 for the gradients, 6 for the two sums over the channels (dB and dC), the rest what a (token, channel)
// needs once.
#include "ssd_scan_common.h"
#include "ssd_sum_rows.h"

namespace ssd {

// Sums V values (32 or 64) over the wave's 64 lanes so that each lane ends with one total.  Two values at a time,
// a lane keeps the half of the lanes' sum of one and hands its part of the other across: V - 1 exchanges
// and additions in all, where V sums by themselves would take 6 V.  Values come in order of their index; at
// most six sums wait for their partner.  Lane l ends with the value whose index is l's bits in the order
// 3, 2, 1, 0, 5, 4 (the exchanges within 16 lanes ride on the addition, so they come first); of 32
// values, lanes l and l ^ 16 hold the same.
template <int V> struct WaveSum {
    static_assert(V == 32 || V == 64, "five or six exchanges");
    float wait[6];
    template <int LEVEL> __device__ static inline float join(float x, float y) {
        const int lane = threadIdx.x & 63;
        if constexpr (LEVEL < 4) {
            const bool up = lane & (8 >> LEVEL);
            const float mine = up ? y : x, other = up ? x : y;
            // partners: lane ^ 8 (rotate 16 by 8), ^ 7 (mirror 8), ^ 2, ^ 1
            return mine + (LEVEL == 0 ? dpp<0x128>(other) : LEVEL == 1 ? dpp<0x141>(other)
                           : LEVEL == 2 ? dpp<0x4e>(other) : dpp<0xb1>(other));
        } else {
            // (the pair's elements are named before the casts: a cast of a vector's element takes its first)
            const uint32_t u = __builtin_bit_cast(uint32_t, x), v = __builtin_bit_cast(uint32_t, y);
            const auto r = LEVEL == 4 ? __builtin_amdgcn_permlane32_swap(u, v, false, false)
                                      : __builtin_amdgcn_permlane16_swap(u, v, false, false);
            const uint32_t r0 = r[0], r1 = r[1];
            return __builtin_bit_cast(float, r0) + __builtin_bit_cast(float, r1);
        }
    }
    // value `i` (a constant after unrolling)
    __device__ inline void push(int i, float v) {
        if (!(i & 1)) { wait[0] = v; return; }
        v = join<0>(wait[0], v);
        if (!(i & 2)) { wait[1] = v; return; }
        v = join<1>(wait[1], v);
        if (!(i & 4)) { wait[2] = v; return; }
        v = join<2>(wait[2], v);
        if (!(i & 8)) { wait[3] = v; return; }
        v = join<3>(wait[3], v);
        if (!(i & 16)) { wait[4] = v; return; }
        v = join<4>(wait[4], v);
        if (V == 64 && !(i & 32)) { wait[5] = v; return; }
        wait[0] = join<5>(V == 64 ? wait[5] : v, v);
    }
    __device__ inline float total() const { return wait[0]; }
    __device__ static inline int index(int lane) {
        return (lane >> 3 & 1) | (lane >> 2 & 1) << 1 | (lane >> 1 & 1) << 2 | (lane & 1) << 3 | (lane >> 5 & 1) << 4 |
               (V == 64 ? (lane >> 4 & 1) << 5 : 0);
    }
};

// The tokens of a tile that a wave prepares and finishes: raw inputs, loaded a tile ahead.
template <typename T, int TPW> struct BackTokens {
    T x[TPW], dt[TPW], z[TPW], g[TPW];
    __device__ inline void load(const ScanArgs& a, const ScanPlace& p, int t0, int w, int nw) {
        const uint32_t lo = (uint32_t)p.c * (uint32_t)sizeof(T);
        const TileRows<T, kScanPeriod> rx(a.x, a.xs, p.row0, t0, a.seqlen);
        const TileRows<T, kScanPeriod> rd(a.dt, a.dts, p.row0, t0, a.seqlen);
        const TileRows<T, kScanPeriod> rg(a.dout, a.channels, p.row0, t0, a.seqlen);
#pragma unroll
        for (int j = 0; j < TPW; ++j) {
            x[j] = rx.load(w + j * nw, lo);
            dt[j] = rd.load(w + j * nw, lo);
            g[j] = rg.load(w + j * nw, lo);
        }
        if (a.z) {
            const TileRows<T, kScanPeriod> rz(a.z, a.zs, p.row0, t0, a.seqlen);
#pragma unroll
            for (int j = 0; j < TPW; ++j) z[j] = rz.load(w + j * nw, lo);
        }
    }
};

template <typename T, int NW, int NS, bool VL>
__global__ __launch_bounds__(NW * 64, NS == 4 ? 3 : 2) void k_scan_backward(ScanArgs args) {
    const ScanArgs& a = args;
    constexpr int TB = kScanPeriod;  // tokens of a tile: a saved state enters each
    constexpr int TPW = TB / NW;  // tokens a wave prepares and finishes
    static_assert(TPW >= 1, "every wave has a token of each tile");
    constexpr int N = NW * NS;
    typedef ScalarRows<T, NS> Rows;
    constexpr int GT = Rows::GROUP;
    __shared__ f32x2 s_d[TB][64];  // (d, d x)
    __shared__ float s_g[TB][64];  // dy
    __shared__ float s_y[NW][TB][64], s_u[NW][TB][64], s_q[NW][TB][64];
    const ScanPlace p = scan_place(a);
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n0 = w * NS;

    float A2[NS], g[NS], dA[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        A2[i] = decay_rate(a.A[(int64_t)p.c * N + n0 + i]);
        g[i] = dA[i] = 0.f;
    }
    const float bias = a.dt_bias ? a.dt_bias[p.c] : 0.f, Dc = a.D ? a.D[p.c] : 0.f;
    float dD = 0.f, db = 0.f;
    const int64_t soff = (int64_t)p.c * N + n0, sstride = (int64_t)a.channels * N;
    const int tile0 = p.split * a.tiles_per_split, tile1 = min(tile0 + a.tiles_per_split, a.ntiles);
    if (p.split + 1 < a.nsplit) {
        // (the last split's own pass began with the final state's gradient)
        const float* st = a.split_state + (int64_t)p.b * a.nsplit * sstride + soff;
        const float* sum = a.split_sum + (int64_t)p.b * a.nsplit * a.channels + p.c;
        if (a.nsplit > kFoldSplits) {
            load_states<NS>(st, DT_F32, p.split * sstride, g);
        } else {
            load_states<NS>(st, DT_F32, (a.nsplit - 2) * sstride, g);
            fold_splits<NS>(A2, g, a.nsplit - 2 - p.split, [&](int k) { return sum[(int64_t)(a.nsplit - 2 - k) * a.channels]; },
                            [&](int k) { return st + (a.nsplit - 3 - k) * sstride; });
        }
    } else if (!VL && a.dfin) {
        load_states<NS>(a.dfin, a.state_dtype, p.b * sstride + soff, g);
    }
    // this wave's sums over the channels: lane l holds that of token `pk`, state `pi` of a tile
    typedef WaveSum<TB * NS> Sum;
    const int pidx = Sum::index(lane), pk = TB - 1 - pidx / NS, pi = pidx % NS;
    float* part = a.part_bc + (((int64_t)p.b * a.groups + p.g) * a.cblk + p.cblk) * a.seqlen * N + n0 + pi;
    const int64_t part_c = (int64_t)a.batch * a.groups * a.cblk * a.seqlen * N;

    BackTokens<T, TPW> next;
    next.load(a, p, (tile1 - 1) * TB, w, NW);
    float hnext[NS];
    load_states<NS>(a.saved, DT_F32, ((int64_t)p.b * a.ntiles + tile1 - 1) * sstride + soff, hnext);
    for (int tile = tile1 - 1; tile >= tile0; --tile) {
        const ScanArgs& a = args_again();
        const int t0 = tile * TB;
        BackTokens<T, TPW> cur = next;
        SeqMasks m{0, 0, 0};
        if (VL) {
            // padding counts as nothing, whatever it holds: no step, no inputs, no gradient of its outputs
            m = seq_masks<TB>(a, p.row0, t0);
#pragma unroll
            for (int j = 0; j < TPW; ++j)
                if (m.pad >> (w + j * NW) & 1) cur.x[j] = cur.dt[j] = cur.z[j] = cur.g[j] = (T)0.f;
        }
        const Rows rb((const T*)a.B + p.g * N + n0, a.Bs, p.row0, t0, a.seqlen);
        const Rows rc((const T*)a.C + p.g * N + n0, a.Cs, p.row0, t0, a.seqlen);
        typename Rows::Group gb[2], gc[2];
        gb[0].load(rb, 0);
        gc[0].load(rc, 0);
        float hin[NS];
#pragma unroll
        for (int i = 0; i < NS; ++i) hin[i] = hnext[i];
        float step[TPW], dyj[TPW];
        steps(a, cur.dt, bias, step);
#pragma unroll
        for (int j = 0; j < TPW; ++j) dyj[j] = f32of(cur.g[j]);
        if (a.z) {
#pragma unroll
            for (int j = 0; j < TPW; ++j) dyj[j] *= silu_f(f32of(cur.z[j]));
        }
#pragma unroll
        for (int j = 0; j < TPW; ++j) {
            const int k = w + j * NW;
            const bool in = t0 + k < a.seqlen && p.live && !(VL && (m.pad >> k & 1));
            const float d = in ? step[j] : 0.f;
            s_d[k][lane] = f32x2{d, d * f32of(cur.x[j])};
            s_g[k][lane] = in ? dyj[j] : 0.f;
        }
        __syncthreads();

        // the tile's states and decays again
        float h[TB][NS], e[TB][NS];
#pragma unroll
        for (int k = 0; k < TB; ++k) {
            if (k % GT == 0 && k + GT < TB) {
                gb[(k / GT + 1) & 1].load(rb, k + GT);
                gc[(k / GT + 1) & 1].load(rc, k + GT);
            }
            if (VL && (m.pad >> k & 1)) {
                gb[(k / GT) & 1].clear(k % GT);
                gc[(k / GT) & 1].clear(k % GT);
            }
            float Bv[NS], Cv[NS];
            gb[(k / GT) & 1].values(k % GT, Bv);
            gc[(k / GT) & 1].values(k % GT, Cv);
            float prev[NS];
#pragma unroll
            for (int i = 0; i < NS; ++i) prev[i] = k ? h[k ? k - 1 : 0][i] : hin[i];
            if (VL && (m.start >> k & 1)) {
                const int q = a.seq[p.row0 + t0 + k];
#pragma unroll
                for (int i = 0; i < NS; ++i) prev[i] = 0.f;
                if (a.h0 && state_number(a, q)) load_states<NS>(a.h0, a.state_dtype, q * sstride + soff, prev);
            }
            if (VL && (m.pad >> k & 1)) {
#pragma unroll
                for (int i = 0; i < NS; ++i) prev[i] = 0.f;
            }
            const f32x2 dv = s_d[k][lane];
            float y = 0.f;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                e[k][i] = __builtin_amdgcn_exp2f(dv[0] * A2[i]);
                h[k][i] = e[k][i] * prev[i] + dv[1] * Bv[i];
                y += h[k][i] * Cv[i];
            }
            s_y[w][k][lane] = y;
        }
        // and the gradients back through them
        Sum sb, sc;
        float dAt[NS];
#pragma unroll
        for (int i = 0; i < NS; ++i) dAt[i] = 0.f;
#pragma unroll
        for (int k = TB - 1; k >= 0; --k) {
            if (k == TB / 2 - 1) {  // half of the tile's states and decays are used up: room for the next tile's inputs
                const ScanArgs& a = args_again();
                next.load(a, p, t0 - TB, w, NW);
                load_states<NS>(a.saved, DT_F32, ((int64_t)p.b * a.ntiles + max(tile - 1, 0)) * sstride + soff, hnext);
            }
            if (k % GT == GT - 1 && k >= GT && k / GT < TB / GT - 1) {  // (the last two groups are still there)
                gb[(k / GT - 1) & 1].load(rb, k - 2 * GT + 1);
                gc[(k / GT - 1) & 1].load(rc, k - 2 * GT + 1);
            }
            if (VL && (m.pad >> k & 1)) {
                gb[(k / GT) & 1].clear(k % GT);
                gc[(k / GT) & 1].clear(k % GT);
            }
            float Bv[NS], Cv[NS], prev[NS];
            gb[(k / GT) & 1].values(k % GT, Bv);
            gc[(k / GT) & 1].values(k % GT, Cv);
#pragma unroll
            for (int i = 0; i < NS; ++i) prev[i] = k ? h[k ? k - 1 : 0][i] : hin[i];
            if (VL && (m.start >> k & 1)) {
                const int q = a.seq[p.row0 + t0 + k];
#pragma unroll
                for (int i = 0; i < NS; ++i) prev[i] = 0.f;
                if (a.h0 && state_number(a, q)) load_states<NS>(a.h0, a.state_dtype, q * sstride + soff, prev);
            }
            if (VL && (m.end >> k & 1)) {
                const int q = a.seq[p.row0 + t0 + k];
#pragma unroll
                for (int i = 0; i < NS; ++i) g[i] = 0.f;
                if (a.dfin && state_number(a, q)) load_states<NS>(a.dfin, a.state_dtype, q * sstride + soff, g);
            }
            if (VL && (m.pad >> k & 1)) {
#pragma unroll
                for (int i = 0; i < NS; ++i) prev[i] = g[i] = 0.f;
            }
            const f32x2 dv = s_d[k][lane];
            const float dy = s_g[k][lane];
            float u = 0.f, qa = 0.f;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                g[i] += dy * Cv[i];
                sc.push((TB - 1 - k) * NS + i, dy * h[k][i]);
                sb.push((TB - 1 - k) * NS + i, g[i] * dv[1]);
                u += g[i] * Bv[i];
                g[i] *= e[k][i];
                const float q = g[i] * prev[i];
                qa += q * A2[i];
                dAt[i] += q * dv[0];
            }
            s_u[w][k][lane] = u;
            s_q[w][k][lane] = qa;
            if (VL && (m.start >> k & 1)) {
                const int q = a.seq[p.row0 + t0 + k];
                if (a.dh0 && state_number(a, q) && p.live)
                    store_states<NS>(a.dh0, a.state_dtype, q * sstride + soff, g);
            }
        }
        // a tile's sums first, then the tiles': long sums keep their low bits
#pragma unroll
        for (int i = 0; i < NS; ++i) dA[i] += dAt[i];
        if (t0 + pk < a.seqlen && (TB * NS == 64 || !(lane & 16))) {
            part[(int64_t)(t0 + pk) * N] = sb.total();
            part[part_c + (int64_t)(t0 + pk) * N] = sc.total();
        }
        __syncthreads();
        float dDt = 0.f, dbt = 0.f;
        const ScanArgs& a2 = args_again();
        const TileRows<T, kScanPeriod> rx(a2.dx, a2.channels, p.row0, t0, a2.seqlen);
        const TileRows<T, kScanPeriod> rd(a2.ddt, a2.channels, p.row0, t0, a2.seqlen);
        const TileRows<T, kScanPeriod> rz(a2.dz, a2.channels, p.row0, t0, a2.seqlen);
        const uint32_t lo = p.live ? (uint32_t)p.c * (uint32_t)sizeof(T) : kNoLane;
        float y[TPW], u[TPW], ddt[TPW];
#pragma unroll
        for (int j = 0; j < TPW; ++j) {
            const int k = w + j * NW;
            const float x = f32of(cur.x[j]);
            float q = 0.f;
            y[j] = Dc * x;
            u[j] = 0.f;
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                y[j] += s_y[i][k][lane];
                u[j] += s_u[i][k][lane];
                q += s_q[i][k][lane];
            }
            ddt[j] = x * u[j] + q * (1.f / kLog2e);
        }
        if (a2.softplus) {
#pragma unroll
            for (int j = 0; j < TPW; ++j) ddt[j] *= sigmoid_f(f32of(cur.dt[j]) + bias);
        }
#pragma unroll
        for (int j = 0; j < TPW; ++j) {
            const int k = w + j * NW;
            const float d = s_d[k][lane][0], dy = s_g[k][lane];
            rx.store(k, lo, Dc * dy + d * u[j]);
            rd.store(k, lo, ddt[j]);
            dDt += dy * f32of(cur.x[j]);  // zero past the end, where x = dy = 0
            dbt += t0 + k < a2.seqlen ? ddt[j] : 0.f;
        }
        if (a2.z) {
#pragma unroll
            for (int j = 0; j < TPW; ++j) {
                const float z = f32of(cur.z[j]), sz = sigmoid_f(z);
                rz.store(w + j * NW, lo, f32of(cur.g[j]) * y[j] * (sz * (1.f + z * (1.f - sz))));
            }
        }
        dD += dDt;
        db += dbt;
        __syncthreads();
    }
    if (!VL && a.dh0 && p.split == 0 && p.live) store_states<NS>(a.dh0, a.state_dtype, p.b * sstride + soff, g);
    const int64_t prow = (int64_t)p.b * a.nsplit + p.split;
    if (p.live) store_states<NS>(a.part_a, DT_F32, prow * sstride + soff, dA);
    s_y[w][0][lane] = dD;
    s_u[w][0][lane] = db;
    __syncthreads();
    if (w == 0 && p.live) {
        float d = 0.f, b = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            d += s_y[i][0][lane];
            b += s_u[i][0][lane];
        }
        a.part_d[prow * a.channels + p.c] = d;
        a.part_d[((int64_t)a.batch * a.nsplit + prow) * a.channels + p.c] = b;
    }
}

// First pass over the time splits, from the last token to the first: the gradient of the state entering each
// split but the first, from a zero gradient behind it (into the split before's place), and the sum of its steps.
template <typename T, int NW, int NS, bool VL>
__global__ __launch_bounds__(NW * 64) void k_scan_backward_carry(ScanArgs a) {
    constexpr int TB = kScanPeriod, TPW = TB / NW, N = NW * NS;
    typedef ScalarRows<T, NS> Rows;
    constexpr int GT = Rows::GROUP;
    __shared__ f32x2 s_d[2][TB][64];  // (d, dy), one tile ahead
    ScanArgs grid = a;
    grid.nsplit = a.nsplit - 1;
    ScanPlace p = scan_place(grid);
    p.split += 1;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n0 = w * NS;
    float A2[NS], g[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        A2[i] = decay_rate(a.A[(int64_t)p.c * N + n0 + i]);
        g[i] = 0.f;
    }
    const float bias = a.dt_bias ? a.dt_bias[p.c] : 0.f;
    const int64_t soff = (int64_t)p.c * N + n0, sstride = (int64_t)a.channels * N;
    const int tile0 = p.split * a.tiles_per_split, tile1 = min(tile0 + a.tiles_per_split, a.ntiles);
    float sum = 0.f;
    bool fresh = false;
    if (!VL && a.dfin && p.split == a.nsplit - 1) load_states<NS>(a.dfin, a.state_dtype, p.b * sstride + soff, g);
    T dt[TPW], z[TPW], go[TPW];
    auto load = [&](int t0) {
        const uint32_t lo = (uint32_t)p.c * (uint32_t)sizeof(T);
        const TileRows<T, kScanPeriod> rd(a.dt, a.dts, p.row0, t0, a.seqlen);
        const TileRows<T, kScanPeriod> rg(a.dout, a.channels, p.row0, t0, a.seqlen);
#pragma unroll
        for (int j = 0; j < TPW; ++j) {
            dt[j] = rd.load(w + j * NW, lo);
            go[j] = rg.load(w + j * NW, lo);
        }
        if (a.z) {
            const TileRows<T, kScanPeriod> rz(a.z, a.zs, p.row0, t0, a.seqlen);
#pragma unroll
            for (int j = 0; j < TPW; ++j) z[j] = rz.load(w + j * NW, lo);
        }
    };
    auto prepare = [&](int buf, int t0) {
        float step[TPW], dy[TPW];
        steps(a, dt, bias, step);
#pragma unroll
        for (int j = 0; j < TPW; ++j) dy[j] = f32of(go[j]);
        if (a.z) {
#pragma unroll
            for (int j = 0; j < TPW; ++j) dy[j] *= silu_f(f32of(z[j]));
        }
#pragma unroll
        for (int j = 0; j < TPW; ++j) {
            const bool in = t0 + w + j * NW < a.seqlen;
            s_d[buf][w + j * NW][lane] = f32x2{in ? step[j] : 0.f, in ? dy[j] : 0.f};
        }
    };
    load((tile1 - 1) * TB);
    prepare(0, (tile1 - 1) * TB);
    for (int tile = tile1 - 1; tile >= tile0; --tile) {
        const int t0 = tile * TB, buf = (tile1 - 1 - tile) & 1;
        const Rows rc((const T*)a.C + p.g * N + n0, a.Cs, p.row0, t0, a.seqlen);
        typename Rows::Group gc[2];
        gc[(TB / GT - 1) & 1].load(rc, TB - GT);
        load(t0 - TB);
        SeqMasks m{0, 0, 0};
        if (VL) m = seq_masks<TB>(a, p.row0, t0);
        __syncthreads();
        float part = 0.f;
#pragma unroll
        for (int k = TB - 1; k >= 0; --k) {
            if (k % GT == GT - 1 && k >= GT) gc[(k / GT - 1) & 1].load(rc, k - 2 * GT + 1);
            float Cv[NS];
            gc[(k / GT) & 1].values(k % GT, Cv);
            if (VL && (m.end >> k & 1)) {
                const int q = a.seq[p.row0 + t0 + k];
                fresh = true;
#pragma unroll
                for (int i = 0; i < NS; ++i) g[i] = 0.f;
                if (a.dfin && state_number(a, q)) load_states<NS>(a.dfin, a.state_dtype, q * sstride + soff, g);
            }
            const f32x2 dv = s_d[buf][k][lane];
            part += dv[0];
#pragma unroll
            for (int i = 0; i < NS; ++i) g[i] = __builtin_amdgcn_exp2f(dv[0] * A2[i]) * (g[i] + dv[1] * Cv[i]);
        }
        sum += part;
        prepare(buf ^ 1, t0 - TB);  // the other buffer's readers passed this tile's barrier
    }
    if (!p.live) return;
    store_states<NS>(a.split_state, DT_F32, ((int64_t)p.b * a.nsplit + p.split - 1) * sstride + soff, g);
    if (w == 0) a.split_sum[((int64_t)p.b * a.nsplit + p.split) * a.channels + p.c] = fresh ? __builtin_inff() : sum;
}

// Joins the splits where there are many, from the last to the first: the gradient entering each from behind.
__global__ __launch_bounds__(256) void k_scan_backward_join(ScanArgs a) {
    const int64_t per = (int64_t)a.channels * a.dstate, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= a.batch * per) return;
    const int b = (int)(i / per);
    const int64_t cn = i % per;
    const int c = (int)(cn / a.dstate);
    float* st = a.split_state + (int64_t)b * a.nsplit * per + cn;
    const float* sum = a.split_sum + (int64_t)b * a.nsplit * a.channels + c;
    // the last split's own pass began with the final state's gradient
    join_splits(decay_rate(a.A[cn]), st[(a.nsplit - 2) * per], a.nsplit - 2,
                [&](int k) { return sum[(int64_t)(a.nsplit - 2 - k) * a.channels]; },
                [&](int k) { return st + (a.nsplit - 3 - k) * per; });
}

// The results from the partial sums.  The first `nbc` workgroups: dB and dC from the channel blocks' sums
// (out[b][t][g][n] = sum over cblk blocks), 64 runs of 4 values each; the others: dA, dD and ddt_bias from the rows
// of (batch row, split).
template <typename T>
__global__ __launch_bounds__(256) void k_scan_sums(ScanArgs a, int nbc, T* dB, T* dC, float* dA, float* dD, float* db) {
    __shared__ f32x4 lds[256];
    const int lane = threadIdx.x & 63;
    const int N = a.dstate;
    if ((int)blockIdx.x < nbc) {
        const int64_t total = (int64_t)a.batch * a.seqlen * a.groups * N;
        int64_t i = ((int64_t)blockIdx.x * 64 + lane) * 4;
        const bool live = i < 2 * total, second = i >= total;
        if (second) i -= total;
        if (!live) i = 0;
        const int n = (int)(i % N);
        const int64_t r = i / N, row = r / a.groups, b = row / a.seqlen;
        const int g = (int)(r % a.groups), t = (int)(row % a.seqlen);
        const int64_t stride = (int64_t)a.seqlen * N;
        const float* src = a.part_bc + (second ? (int64_t)a.batch * a.groups * a.cblk * stride : 0) +
                           (b * a.groups + g) * a.cblk * stride + (int64_t)t * N + n;
        const f32x4 s = sum_rows<f32x4>(src, stride, a.cblk, lds, live);
        if (live && threadIdx.x < 64) *(typename TT<T>::v4*)((second ? dC : dB) + i) = cvt4<T>(s);
        return;
    }
    const int64_t na = (int64_t)a.channels * N, i = (int64_t)(blockIdx.x - nbc) * 64 + lane;
    const int rows = a.batch * a.nsplit;
    const bool live = i < na + 2 * a.channels, second = i >= na + a.channels;
    const float* src = a.part_a + i;
    float* dst = dA + i;
    int64_t stride = na;
    if (i >= na) {
        const int64_t c = i - na - (second ? a.channels : 0);
        src = a.part_d + (second ? (int64_t)rows * a.channels : 0) + c;
        dst = (second ? db : dD) ? (second ? db : dD) + c : nullptr;
        stride = a.channels;
    }
    const float s = sum_rows<float>(src, stride, rows, (float*)lds, live);
    if (live && dst && threadIdx.x < 64) *dst = s;
}

template <typename T, int NW, int NS>
hipError_t launch_scan_backward_n(ScanArgs& a, T* dB, T* dC, float* dA, float* dD, float* db, hipStream_t st) {
    void* args[] = {&a};
    hipError_t e = hipSuccess;
    const unsigned blocks = (unsigned)(a.batch * a.groups * a.cblk);
    if (a.nsplit > 1) {
        const void* fn = a.seq ? (const void*)&k_scan_backward_carry<T, NW, NS, true>
                               : (const void*)&k_scan_backward_carry<T, NW, NS, false>;
        e = hipLaunchKernel(fn, dim3(blocks * (a.nsplit - 1)), dim3(NW * 64), args, 0, st);
        if (e != hipSuccess) return e;
        if (a.nsplit > kFoldSplits) {
            const int64_t lanes = (int64_t)a.batch * a.channels * a.dstate;
            e = hipLaunchKernel((const void*)&k_scan_backward_join, dim3((unsigned)((lanes + 255) / 256)), dim3(256), args, 0, st);
            if (e != hipSuccess) return e;
        }
    }
    const void* fn = a.seq ? (const void*)&k_scan_backward<T, NW, NS, true> : (const void*)&k_scan_backward<T, NW, NS, false>;
    e = hipLaunchKernel(fn, dim3(blocks * a.nsplit), dim3(NW * 64), args, 0, st);
    if (e != hipSuccess) return e;
    // both tensors, 64 runs of 4 values a workgroup; 64 parameters a workgroup
    int nbc = (int)(((int64_t)a.batch * a.seqlen * a.groups * a.dstate / 2 + 63) / 64);
    const int np = (int)(((int64_t)a.channels * (a.dstate + 2) + 63) / 64);
    void* sargs[] = {&a, &nbc, &dB, &dC, &dA, &dD, &db};
    return hipLaunchKernel((const void*)&k_scan_sums<T>, dim3((unsigned)(nbc + np)), dim3(256), sargs, 0, st);
}

template <typename T>
hipError_t launch_scan_backward_t(ScanArgs& a, void* dB, void* dC, float* dA, float* dD, float* db, hipStream_t st) {
    switch (a.dstate) {
    case 8: return launch_scan_backward_n<T, 2, 4>(a, (T*)dB, (T*)dC, dA, dD, db, st);
    case 16: return launch_scan_backward_n<T, 4, 4>(a, (T*)dB, (T*)dC, dA, dD, db, st);
    case 32: return launch_scan_backward_n<T, 8, 4>(a, (T*)dB, (T*)dC, dA, dD, db, st);
    case 64: return launch_scan_backward_n<T, 8, 8>(a, (T*)dB, (T*)dC, dA, dD, db, st);
    default: return hipErrorNotSupported;
    }
}

hipError_t launch_scan_backward(ScanArgs& a, int in_dtype, void* dB, void* dC, float* dA, float* dD, float* db,
                                hipStream_t st) {
    switch (in_dtype) {
    case DT_F32: return launch_scan_backward_t<float>(a, dB, dC, dA, dD, db, st);
    case DT_F16: return launch_scan_backward_t<_Float16>(a, dB, dC, dA, dD, db, st);
    case DT_BF16: return launch_scan_backward_t<__bf16>(a, dB, dC, dA, dD, db, st);
    default: return hipErrorNotSupported;
    }
}

}  // namespace ssd
