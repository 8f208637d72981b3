// ssd_scan.hip -- the selective scan forward and its single-token step (ssd_selective_scan and
// ssd_selective_scan_step in include/mamba_ssd.h).
//
//     d = softplus(dt + bias),  h[n] = exp(d A[n]) h[n] + d x B[n],  y = sum_n C[n] h[n] + D x,  out = y silu(z)
//
// Each (token, channel, n) costs one exponential (two issue slots of the vector ALU, measured) and four products and
// sums, against 8 bytes of 16-bit input and output a (token, channel): the prompt scan is bound by the vector
// ALU, the step by the state's traffic.  Decays and products run as exp2 of d (A log2 e).
#include <algorithm>

#include "ssd_scan_common.h"

namespace ssd {

constexpr int kTile = 16;  // tokens of a tile

// The tokens of a tile that a wave prepares: raw inputs, loaded a tile ahead.
template <typename T, int TPW, bool Z> struct ScanTokens {
    T x[TPW], dt[TPW], z[Z ? TPW : 1];
    __device__ inline void load(const ScanArgs& a, const ScanPlace& p, int t0, int w, int nw) {
        const uint32_t lo = (uint32_t)p.c * (uint32_t)sizeof(T);
        const TileRows<T, kTile> rx(a.x, a.xs, p.row0, t0, a.seqlen);
        const TileRows<T, kTile> rd(a.dt, a.dts, p.row0, t0, a.seqlen);
#pragma unroll
        for (int j = 0; j < TPW; ++j) {
            x[j] = rx.load(w + j * nw, lo);
            dt[j] = rd.load(w + j * nw, lo);
        }
        if (Z && a.z) {
            const TileRows<T, kTile> rz(a.z, a.zs, p.row0, t0, a.seqlen);
#pragma unroll
            for (int j = 0; j < TPW; ++j) z[j] = rz.load(w + j * nw, lo);
        }
    }
};

// A workgroup runs its split's tokens a tile at a time: every wave prepares its tokens' (d, d x) in LDS, runs the
// recurrence of its NS states through the tile, leaves its share of y in LDS, and finishes its tokens.  Four states a
// lane (N = 64: eight) is what leaves a wave's part of the sums over n small and the waves many.  At 2 x 8192 x 5120, N = 16,
// bf16: 339 us, the vector ALU issuing in 96% of the cycles (some 2.0 GHz under this load) with 8.1 slots a (token,
// channel, n), 6 of them the recurrence's.
template <typename T, int NW, int NS, bool VL>
__global__ __launch_bounds__(NW * 64) void k_scan(ScanArgs a) {
    constexpr int TPW = kTile / NW;    // tokens a wave prepares and finishes
    constexpr int N = NW * NS, PERIOD = kScanPeriod;
    typedef ScalarRows<T, NS> Rows;
    constexpr int GT = Rows::GROUP;
    __shared__ f32x2 s_d[kTile][64];   // (d, d x)
    __shared__ float s_y[NW][kTile][64];
    const ScanPlace p = scan_place(a);
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n0 = w * NS;

    float A2[NS], h[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        A2[i] = decay_rate(a.A[(int64_t)p.c * N + n0 + i]);
        h[i] = 0.f;
    }
    const float bias = a.dt_bias ? a.dt_bias[p.c] : 0.f, Dc = a.D ? a.D[p.c] : 0.f;
    const int64_t soff = (int64_t)p.c * N + n0, sstride = (int64_t)a.channels * N;
    const int tile0 = p.split * a.tiles_per_split, tile1 = min(tile0 + a.tiles_per_split, (a.seqlen + kTile - 1) / kTile);
    if (p.split && a.nsplit > kFoldSplits) {
        load_states<NS>(a.split_state, DT_F32, ((int64_t)p.b * a.nsplit + p.split) * sstride + soff, h);
    } else {
        if (!VL && a.h0) load_states<NS>(a.h0, a.state_dtype, p.b * sstride + soff, h);
        const float* st = a.split_state + (int64_t)p.b * a.nsplit * sstride + soff;
        const float* sum = a.split_sum + (int64_t)p.b * a.nsplit * a.channels + p.c;
        fold_splits<NS>(A2, h, p.split, [&](int k) { return sum[(int64_t)k * a.channels]; },
                        [&](int k) { return st + (k + 1) * sstride; });
    }
    ScanTokens<T, TPW, true> next;
    next.load(a, p, tile0 * kTile, w, NW);
    for (int tile = tile0; tile < tile1; ++tile) {
        const int t0 = tile * kTile;
        const ScanTokens<T, TPW, true> cur = next;
        const Rows rb((const T*)a.B + p.g * N + n0, a.Bs, p.row0, t0, a.seqlen);
        const Rows rc((const T*)a.C + p.g * N + n0, a.Cs, p.row0, t0, a.seqlen);
        typename Rows::Group gb[2], gc[2];
        gb[0].load(rb, 0);
        gc[0].load(rc, 0);
        float step[TPW];
        steps(a, cur.dt, bias, step);
#pragma unroll
        for (int j = 0; j < TPW; ++j) {
            const int k = w + j * NW;
            const float d = t0 + k < a.seqlen ? step[j] : 0.f;  // (no step past the end: the state stays as it is)
            s_d[k][lane] = f32x2{d, d * f32of(cur.x[j])};
        }
        SeqMasks m{0, 0, 0};
        if (VL) m = seq_masks<kTile>(a, p.row0, t0);
        __syncthreads();
        next.load(a, p, t0 + kTile, w, NW);
#pragma unroll
        for (int k = 0; k < kTile; ++k) {
            if (k % GT == 0 && k + GT < kTile) {
                gb[(k / GT + 1) & 1].load(rb, k + GT);
                gc[(k / GT + 1) & 1].load(rc, k + GT);
            }
            float Bv[NS], Cv[NS];
            gb[(k / GT) & 1].values(k % GT, Bv);
            gc[(k / GT) & 1].values(k % GT, Cv);
            if (k % PERIOD == 0 && a.saved && t0 + k < a.seqlen && p.live) {
                float* sv = a.saved + ((int64_t)p.b * a.ntiles + (t0 + k) / PERIOD) * sstride + soff;
                store_states<NS>(sv, DT_F32, 0, h);
            }
            if (VL && (m.start >> k & 1)) {
                const int q = a.seq[p.row0 + t0 + k];
#pragma unroll
                for (int i = 0; i < NS; ++i) h[i] = 0.f;
                if (a.h0 && state_number(a, q)) load_states<NS>(a.h0, a.state_dtype, q * sstride + soff, h);
            }
            const f32x2 dv = s_d[k][lane];
            float y = 0.f;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                h[i] = __builtin_amdgcn_exp2f(dv[0] * A2[i]) * h[i] + dv[1] * Bv[i];
                y += h[i] * Cv[i];
            }
            s_y[w][k][lane] = y;
            if (VL && (m.end >> k & 1) && a.fin && p.live) {
                const int q = a.seq[p.row0 + t0 + k];
                if (state_number(a, q)) store_states<NS>(a.fin, a.state_dtype, q * sstride + soff, h);
            }
        }
        __syncthreads();
        const TileRows<T, kTile> ro(a.out, a.channels, p.row0, t0, a.seqlen);
        const uint32_t lo = p.live ? (uint32_t)p.c * (uint32_t)sizeof(T) : kNoLane;
        float y[TPW];
#pragma unroll
        for (int j = 0; j < TPW; ++j) {
            y[j] = Dc * f32of(cur.x[j]);
#pragma unroll
            for (int i = 0; i < NW; ++i) y[j] += s_y[i][w + j * NW][lane];
        }
        if (a.z) {
#pragma unroll
            for (int j = 0; j < TPW; ++j) y[j] *= silu_f(f32of(cur.z[j]));
        }
#pragma unroll
        for (int j = 0; j < TPW; ++j) ro.store(w + j * NW, lo, y[j]);
    }
    if (!VL && a.fin && tile1 * kTile >= a.seqlen && p.live)
        store_states<NS>(a.fin, a.state_dtype, p.b * sstride + soff, h);
}

// First pass over the time splits: the state at the end of each split but the last, from a zero state at
// its start (into the next split's place), and the sum of its steps, by which the state entering it decays
// (infinite where a sequence starts inside: nothing passes).  One barrier a tile: the next tile's (d, d x) go to the other
// buffer.  At 2 x 8192 x 5120, N = 16, bf16: 244 us, the vector ALU issuing in all cycles with 6.1 slots a (token,
// channel, n), 5 of them the recurrence's.
template <typename T, int NW, int NS, bool VL>
__global__ __launch_bounds__(NW * 64) void k_scan_carry(ScanArgs a) {
    constexpr int TPW = kTile / NW, N = NW * NS;
    typedef ScalarRows<T, NS> Rows;
    constexpr int GT = Rows::GROUP;
    __shared__ f32x2 s_d[2][kTile][64];  // (d, d x), one tile ahead
    ScanArgs grid = a;
    grid.nsplit = a.nsplit - 1;
    const ScanPlace p = scan_place(grid);
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n0 = w * NS;
    float A2[NS], h[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        A2[i] = decay_rate(a.A[(int64_t)p.c * N + n0 + i]);
        h[i] = 0.f;
    }
    const float bias = a.dt_bias ? a.dt_bias[p.c] : 0.f;
    const int64_t soff = (int64_t)p.c * N + n0, sstride = (int64_t)a.channels * N;
    const int tile0 = p.split * a.tiles_per_split, tile1 = tile0 + a.tiles_per_split;  // never the last split
    float sum = 0.f;
    bool fresh = false;
    ScanTokens<T, TPW, false> next;
    auto prepare = [&](int buf) {
        float step[TPW];
        steps(a, next.dt, bias, step);
#pragma unroll
        for (int j = 0; j < TPW; ++j) s_d[buf][w + j * NW][lane] = f32x2{step[j], step[j] * f32of(next.x[j])};
    };
    next.load(a, p, tile0 * kTile, w, NW);
    prepare(0);
    for (int tile = tile0; tile < tile1; ++tile) {
        const int t0 = tile * kTile, buf = (tile - tile0) & 1;
        const Rows rb((const T*)a.B + p.g * N + n0, a.Bs, p.row0, t0, a.seqlen);
        typename Rows::Group gb[2];
        gb[0].load(rb, 0);
        next.load(a, p, t0 + kTile, w, NW);
        SeqMasks m{0, 0, 0};
        if (VL) m = seq_masks<kTile>(a, p.row0, t0);
        __syncthreads();
        float part = 0.f;
#pragma unroll
        for (int k = 0; k < kTile; ++k) {
            if (k % GT == 0 && k + GT < kTile) gb[(k / GT + 1) & 1].load(rb, k + GT);
            float Bv[NS];
            gb[(k / GT) & 1].values(k % GT, Bv);
            if (VL && (m.start >> k & 1)) {
                const int q = a.seq[p.row0 + t0 + k];
                fresh = true;
#pragma unroll
                for (int i = 0; i < NS; ++i) h[i] = 0.f;
                if (a.h0 && state_number(a, q)) load_states<NS>(a.h0, a.state_dtype, q * sstride + soff, h);
            }
            const f32x2 dv = s_d[buf][k][lane];
            part += dv[0];
#pragma unroll
            for (int i = 0; i < NS; ++i) h[i] = __builtin_amdgcn_exp2f(dv[0] * A2[i]) * h[i] + dv[1] * Bv[i];
        }
        sum += part;
        prepare(buf ^ 1);  // the other buffer's readers passed this tile's barrier
    }
    if (!p.live) return;
    store_states<NS>(a.split_state, DT_F32, ((int64_t)p.b * a.nsplit + p.split + 1) * sstride + soff, h);
    if (w == 0) a.split_sum[((int64_t)p.b * a.nsplit + p.split) * a.channels + p.c] = fresh ? __builtin_inff() : sum;
}

// Joins the splits where there are many: the state entering each, from the states that k_scan_carry left.  A lane owns one (channel, n).
__global__ __launch_bounds__(256) void k_scan_join(ScanArgs a) {
    const int64_t per = (int64_t)a.channels * a.dstate, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= a.batch * per) return;
    const int b = (int)(i / per);
    const int64_t cn = i % per;
    const int c = (int)(cn / a.dstate);
    const float A2 = decay_rate(a.A[cn]);
    float h = 0.f;
    if (!a.seq && a.h0) {
        const int64_t o = b * per + cn;
        h = a.state_dtype == DT_F32   ? ((const float*)a.h0)[o]
            : a.state_dtype == DT_F16 ? (float)((const _Float16*)a.h0)[o]
                                      : (float)((const __bf16*)a.h0)[o];
    }
    float* st = a.split_state + (int64_t)b * a.nsplit * per + cn;
    const float* sum = a.split_sum + (int64_t)b * a.nsplit * a.channels + c;
    join_splits(A2, h, a.nsplit - 1, [&](int k) { return sum[(int64_t)k * a.channels]; },
                [&](int k) { return st + (k + 1) * per; });
}

// Four values of a row that starts on a multiple of four bytes.
template <typename T> __device__ inline void load_four(const T* p, float (&v)[4]) {
    typedef uint32_t words __attribute__((ext_vector_type(sizeof(T)), aligned(4)));
    const words u = *(const words*)p;
    typename TT<T>::v4 r;
    __builtin_memcpy(&r, &u, 4 * sizeof(T));
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = f32of(r[j]);
}

// One token: N / 4 lanes hold a channel's states, four each, and share the sum over n.  A lane takes its channel for R
// batch rows, so that A and the channel's parameters are read once for them and their states are on their way
// together.  Bound by the states' traffic: 179 MB in 38.3 us at 256 x 5120, N = 16, fp32 states (4.7 TB/s, where a large
// copy reaches 5.0); one row of 1536 channels takes 3.4 us, the time of a launch.
template <typename T, typename S, int N, int R> __global__ __launch_bounds__(256) void k_scan_step(ScanArgs a) {
    constexpr int LPC = N / 4, CPB = 256 / LPC;  // lanes per channel, channels per workgroup
    constexpr int SD = sizeof(S) == 4 ? DT_F32 : __is_same(S, __bf16) ? DT_BF16 : DT_F16;
    const uint32_t nb = (uint32_t)(a.channels + CPB - 1) / CPB;
    const int b0 = (int)(blockIdx.x / nb) * R, c = (int)(blockIdx.x % nb) * CPB + (int)threadIdx.x / LPC;
    const int n0 = (int)(threadIdx.x % LPC) * 4;
    if (c >= a.channels) return;  // whole channels: a channel's lanes stay together
    const int g = a.groups == 1 ? 0 : c / a.dg;
    float h[R][4], x[R], dt[R], z[R], B[R][4], C[R][4];
    int64_t at[R];
    bool have[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int b = min(b0 + r, a.batch - 1);
        const int slot = a.slots ? a.slots[b] : b;
        have[r] = slot >= 0 && slot < a.nseq;
        at[r] = ((int64_t)(have[r] ? slot : 0) * a.channels + c) * N + n0;
        load_states<4>(a.pool, SD, at[r], h[r]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int b = min(b0 + r, a.batch - 1);
        x[r] = f32of(((const T*)a.x)[b * a.xs + c]);
        dt[r] = f32of(((const T*)a.dt)[b * a.dts + c]);
        z[r] = a.z ? f32of(((const T*)a.z)[b * a.zs + c]) : 0.f;
        load_four((const T*)a.B + b * a.Bs + g * N + n0, B[r]);
        load_four((const T*)a.C + b * a.Cs + g * N + n0, C[r]);
    }
    const f32x4 A = *(const f32x4*)(a.A + (int64_t)c * N + n0);
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, Dc = a.D ? a.D[c] : 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (b0 + r >= a.batch) break;
        const float v = dt[r] + bias, d = a.softplus ? step_f(v) : v, u = d * x[r];
        float y = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            h[r][j] = __builtin_amdgcn_exp2f(d * decay_rate(A[j])) * h[r][j] + u * B[r][j];
            y += h[r][j] * C[r][j];
        }
        if (have[r]) store_states<4>(a.pool, SD, at[r], h[r]);
        y += dpp<0xb1>(y);  // lanes ^ 1
        if (LPC >= 4) y += dpp<0x4e>(y);    // ^ 2
        if (LPC >= 8) y += dpp<0x141>(y);   // the other half of 8
        if (LPC >= 16) y += dpp<0x140>(y);  // the other half of 16
        if (n0 == 0) {
            y += Dc * x[r];
            if (a.z) y *= silu_f(z[r]);
            ((T*)a.out)[(int64_t)(b0 + r) * a.channels + c] = (T)(have[r] ? y : 0.f);
        }
    }
}

// Rows a lane takes where that leaves kStepBlocks workgroups, four a CU: 256 x 5120, N = 16 takes 41.0, 38.3, 41.1 and 44 us
// with 1, 2, 4 and 8; small batches want every workgroup that one row a lane gives.
constexpr int kStepRows = 2, kStepBlocks = 1024;

// Time splits.  A split gives the chip more waves and costs a second pass over its tokens, without the outputs.  A tile
// takes a wave a time that its latency or, with many waves on a SIMD, their issue slots decide; the split that
// takes the least time by that is chosen.  The constants (us, for w waves a SIMD of 4 states a lane) were fitted on
// MI355X to 11 numbers of splits of 9 shapes from 1 x 131 x 1536 to 32 x 256 x 5120 (within 15% of the measured times
// near the best split).  Measured, forward, no split / the split taken: 1 x 131 x 1536 23.8 / 12.2 us, 1 x 4096 x 5120
// 711 / 143 us; 32 x 256 x 5120 151 us with none, 216 us with two.
struct TileTime {
    double latency, per_wave, issue;  // max(latency + per_wave * w, issue * w)
    int resident;                     // waves a SIMD holds; more come in rounds, the last of them partly filled
    double round(double w) const { return w > 0 ? std::max(latency + per_wave * w, issue * w) : 0; }
    double at(double w) const {
        if (w <= resident) return round(w);
        const int full = (int)(w / resident);
        const double even = round(resident) * w / resident, stepped = full * round(resident) + round(w - full * resident);
        return even + 0.3 * (stepped - even);
    }
};
int scan_splits(int64_t batch, int64_t seqlen, int64_t channels, int groups, int dstate, bool backward) {
    const TileTime main_pass = backward ? TileTime{2.9, 0.95, 1.64, 3} : TileTime{2.4, 0.6, 0.94, 6};
    const TileTime carry = backward ? TileTime{1.4, 0.25, 0.39, 8} : TileTime{1.9, 0.45, 0.65, 7};
    // the passes' own launches, and each split's part in the join (its states written and read twice at 5 MB a us)
    const double launches = backward ? 7 : 5, each = 0.05 + (double)batch * channels * dstate * 8 / 5e6;
    const int64_t dg = channels / groups, blocks = batch * groups * ((dg + 63) / 64);
    const int64_t tile = backward ? kScanPeriod : kTile, tiles = (seqlen + tile - 1) / tile;
    const int waves = dstate == 8 ? 2 : dstate == 16 ? 4 : 8;  // of a workgroup
    const double width = dstate == 64 ? 2 : 1;                 // quads of states a lane holds
    const double w1 = (double)blocks * waves / 1024;
    const int64_t most = std::min<int64_t>(tiles, 128);
    int64_t best = 1;
    double least = 0;
    for (int64_t want = 1; want <= most; want += want < 4 ? 1 : want / 2) {  // 1, 2, 3, 4, 6, 9, 13, 19, 28, 42, 63, 94
        const int64_t per = (tiles + want - 1) / want, s = (tiles + per - 1) / per;
        const double w = w1 * (double)s, again = s > 1 ? (double)(s - 1) / (double)s : 0;
        const double edges = 0.7 / std::max(1.0, w / main_pass.resident);  // a split's beginning and end, in tiles
        const double t = ((double)per + edges) * width * (main_pass.at(w) + again * carry.at(w)) +
                         (s > 1 ? launches + each * (double)s : 0);
        if (want == 1 || t < least) {
            least = t;
            best = s;
        }
    }
    return (int)best;
}

template <typename T, int NW, int NS> hipError_t launch_scan_n(ScanArgs& a, hipStream_t st) {
    void* args[] = {&a};
    const unsigned blocks = (unsigned)(a.batch * a.groups * a.cblk);
    if (a.nsplit > 1) {
        const void* fn = a.seq ? (const void*)&k_scan_carry<T, NW, NS, true> : (const void*)&k_scan_carry<T, NW, NS, false>;
        hipError_t e = hipLaunchKernel(fn, dim3(blocks * (a.nsplit - 1)), dim3(NW * 64), args, 0, st);
        if (e != hipSuccess) return e;
        if (a.nsplit > kFoldSplits) {
            const int64_t lanes = (int64_t)a.batch * a.channels * a.dstate;
            e = hipLaunchKernel((const void*)&k_scan_join, dim3((unsigned)((lanes + 255) / 256)), dim3(256), args, 0, st);
            if (e != hipSuccess) return e;
        }
    }
    const void* fn = a.seq ? (const void*)&k_scan<T, NW, NS, true> : (const void*)&k_scan<T, NW, NS, false>;
    return hipLaunchKernel(fn, dim3(blocks * a.nsplit), dim3(NW * 64), args, 0, st);
}

template <typename T> hipError_t launch_scan_t(ScanArgs& a, hipStream_t st) {
    switch (a.dstate) {
    case 8: return launch_scan_n<T, 2, 4>(a, st);
    case 16: return launch_scan_n<T, 4, 4>(a, st);
    case 32: return launch_scan_n<T, 8, 4>(a, st);
    case 64: return launch_scan_n<T, 8, 8>(a, st);
    default: return hipErrorNotSupported;
    }
}

hipError_t launch_scan(ScanArgs& a, int in_dtype, hipStream_t st) {
    switch (in_dtype) {
    case DT_F32: return launch_scan_t<float>(a, st);
    case DT_F16: return launch_scan_t<_Float16>(a, st);
    case DT_BF16: return launch_scan_t<__bf16>(a, st);
    default: return hipErrorNotSupported;
    }
}

template <typename T, typename S, int N> hipError_t launch_scan_step_n(ScanArgs& a, hipStream_t st) {
    const int64_t per_row = (a.channels + 1024 / N - 1) / (1024 / N);  // workgroups
    const bool many = per_row * (a.batch / kStepRows) >= kStepBlocks;
    const int64_t blocks = per_row * (many ? (a.batch + kStepRows - 1) / kStepRows : a.batch);
    void* args[] = {&a};
    return hipLaunchKernel(many ? (const void*)&k_scan_step<T, S, N, kStepRows> : (const void*)&k_scan_step<T, S, N, 1>,
                           dim3((unsigned)blocks), dim3(256), args, 0, st);
}

template <typename T, typename S> hipError_t launch_scan_step_ts(ScanArgs& a, hipStream_t st) {
    switch (a.dstate) {
    case 8: return launch_scan_step_n<T, S, 8>(a, st);
    case 16: return launch_scan_step_n<T, S, 16>(a, st);
    case 32: return launch_scan_step_n<T, S, 32>(a, st);
    case 64: return launch_scan_step_n<T, S, 64>(a, st);
    default: return hipErrorNotSupported;
    }
}

template <typename T> hipError_t launch_scan_step_t(ScanArgs& a, hipStream_t st) {
    switch (a.state_dtype) {
    case DT_F32: return launch_scan_step_ts<T, float>(a, st);
    case DT_F16: return launch_scan_step_ts<T, _Float16>(a, st);
    case DT_BF16: return launch_scan_step_ts<T, __bf16>(a, st);
    default: return hipErrorNotSupported;
    }
}

hipError_t launch_scan_step(ScanArgs& a, int in_dtype, hipStream_t st) {
    switch (in_dtype) {
    case DT_F32: return launch_scan_step_t<float>(a, st);
    case DT_F16: return launch_scan_step_t<_Float16>(a, st);
    case DT_BF16: return launch_scan_step_t<__bf16>(a, st);
    default: return hipErrorNotSupported;
    }
}

}  // namespace ssd
