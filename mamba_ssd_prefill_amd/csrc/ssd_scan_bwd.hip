// ssd_scan_bwd.hip -- the gradients of the selective scan (ssd_selective_scan_backward in
// include/mamba_ssd.h).  With g[n] the gradient of the state h[n] after token t,
//
//     g[n]  = C[n] dy + (exp(d A[n]) g[n] of token t+1),      dy = dout silu(z)
//     dC[n] = sum_c dy h[n],   dB[n] = sum_c g[n] d x         (over the channels of the group)
//     q[n]  = g[n] exp(d A[n]) h[n] of token t-1
//     dx = D dy + d sum_n g[n] B[n],   dd = x sum_n g[n] B[n] + sum_n A[n] q[n],   dA[n] = sum_t d q[n]
//
// A tile of 64 / NS tokens is taken at a time, from the last to the first: the states of the tile are
// computed again from the saved state that enters it and kept in registers with their decays (64 of each a
// lane), and then the gradients run back through them.  The tile's dB and dC are 64 values a wave, each
// a sum over its 64 lanes, so that after the sums lane l holds one value of each.
#include "ssd_scan_common.h"

namespace ssd {

// Sums v over the wave's 64 lanes, for 64 values v: lane l returns the sum of the value with index l.
// fn(i) gives value i.
__device__ inline float wave_sum64(const float (&v)[64]) {
    const int lane = threadIdx.x & 63;
    float r = 0.f;
#pragma unroll
    for (int i = 0; i < 64; ++i) {
        float s = v[i];
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1) s += __shfl_xor(s, m, 64);
        if (lane == i) r = s;
    }
    return r;
}

template <typename T, int NW, int NS, bool VL>
__global__ __launch_bounds__(NW * 64) void k_scan_backward(ScanArgs a) {
    constexpr int TB = 64 / NS;   // tokens of a tile
    constexpr int TPW = TB / NW;  // tokens a wave prepares and finishes
    static_assert(TPW >= 1, "every wave has a token of each tile");
    constexpr int N = NW * NS;
    __shared__ f32x2 s_d[TB][64];  // (d, d x)
    __shared__ float s_g[TB][64];  // dy
    __shared__ float s_y[NW][TB][64], s_u[NW][TB][64], s_q[NW][TB][64];
    const ScanPlace p = scan_place(a);
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n0 = w * NS;

    float A[NS], g[NS], dA[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        A[i] = a.A[(int64_t)p.c * N + n0 + i];
        g[i] = dA[i] = 0.f;
    }
    const float bias = a.dt_bias ? a.dt_bias[p.c] : 0.f, Dc = a.D ? a.D[p.c] : 0.f;
    float dD = 0.f, db = 0.f;
    const int64_t soff = (int64_t)p.c * N + n0, sstride = (int64_t)a.channels * N;
    const int tile0 = p.split * a.tiles_per_split, tile1 = min(tile0 + a.tiles_per_split, a.ntiles);
    if (p.split + 1 < a.nsplit) {
#pragma unroll
        for (int i = 0; i < NS; ++i) g[i] = a.split_state[((int64_t)p.b * a.nsplit + p.split) * sstride + soff + i];
    } else if (!VL && a.dfin) {
        load_states<NS>(a.dfin, a.state_dtype, p.b * sstride + soff, g);
    }
    float* part = a.part_bc + (((int64_t)p.b * a.groups + p.g) * a.cblk + p.cblk) * a.seqlen * N;
    const int64_t part_c = (int64_t)a.batch * a.groups * a.cblk * a.seqlen * N;

    for (int tile = tile1 - 1; tile >= tile0; --tile) {
        const int t0 = tile * TB;
        float xv[TPW], zv[TPW], gv[TPW], sg[TPW], dv_[TPW], dyv[TPW];
#pragma unroll
        for (int j = 0; j < TPW; ++j) {
            const int k = w + j * NW, t = t0 + k;
            const bool in = t < a.seqlen && p.live;
            const int64_t r = p.row0 + min(t, a.seqlen - 1);
            xv[j] = f32of(((const T*)a.x)[r * a.xs + p.c]);
            const float v = f32of(((const T*)a.dt)[r * a.dts + p.c]) + bias;
            gv[j] = in ? f32of(((const T*)a.dout)[r * a.channels + p.c]) : 0.f;
            zv[j] = a.z ? f32of(((const T*)a.z)[r * a.zs + p.c]) : 0.f;
            dv_[j] = in ? (a.softplus ? softplus_f(v) : v) : 0.f;
            sg[j] = a.softplus ? sigmoid_f(v) : 1.f;
            dyv[j] = a.z ? gv[j] * silu_f(zv[j]) : gv[j];
            s_d[k][lane] = f32x2{dv_[j], dv_[j] * xv[j]};
            s_g[k][lane] = dyv[j];
        }
        SeqMasks m{0, 0};
        if (VL) m = seq_masks<TB>(a, p.row0, t0);
        float hin[NS];
        load_states<NS>(a.saved, DT_F32, ((int64_t)p.b * a.ntiles + tile) * sstride + soff, hin);
        __syncthreads();

        // the tile's states and decays again
        float h[TB][NS], e[TB][NS];
#pragma unroll
        for (int k = 0; k < TB; ++k) {
            const int64_t r = p.row0 + min(t0 + k, a.seqlen - 1);
            float Bv[NS], Cv[NS];
            scalar_row<T, NS>((const T*)a.B + r * a.Bs + p.g * N + n0, Bv);
            scalar_row<T, NS>((const T*)a.C + r * a.Cs + p.g * N + n0, Cv);
            float prev[NS];
#pragma unroll
            for (int i = 0; i < NS; ++i) prev[i] = k ? h[k ? k - 1 : 0][i] : hin[i];
            if (VL && (m.start >> k & 1)) {
                const int q = a.seq[r];
#pragma unroll
                for (int i = 0; i < NS; ++i) prev[i] = 0.f;
                if (a.h0 && state_number(a, q)) load_states<NS>(a.h0, a.state_dtype, q * sstride + soff, prev);
            }
            const f32x2 dv = s_d[k][lane];
            float y = 0.f;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                e[k][i] = __builtin_amdgcn_exp2f(dv[0] * (A[i] * kLog2e));
                h[k][i] = e[k][i] * prev[i] + dv[1] * Bv[i];
                y += h[k][i] * Cv[i];
            }
            s_y[w][k][lane] = y;
        }
        // and the gradients back through them
        float vB[64], vC[64], dAt[NS];
#pragma unroll
        for (int i = 0; i < NS; ++i) dAt[i] = 0.f;
#pragma unroll
        for (int k = TB - 1; k >= 0; --k) {
            const int64_t r = p.row0 + min(t0 + k, a.seqlen - 1);
            float Bv[NS], Cv[NS], prev[NS];
            scalar_row<T, NS>((const T*)a.B + r * a.Bs + p.g * N + n0, Bv);
            scalar_row<T, NS>((const T*)a.C + r * a.Cs + p.g * N + n0, Cv);
#pragma unroll
            for (int i = 0; i < NS; ++i) prev[i] = k ? h[k ? k - 1 : 0][i] : hin[i];
            if (VL && (m.start >> k & 1)) {
                const int q = a.seq[r];
#pragma unroll
                for (int i = 0; i < NS; ++i) prev[i] = 0.f;
                if (a.h0 && state_number(a, q)) load_states<NS>(a.h0, a.state_dtype, q * sstride + soff, prev);
            }
            if (VL && (m.end >> k & 1)) {
                const int q = a.seq[r];
#pragma unroll
                for (int i = 0; i < NS; ++i) g[i] = 0.f;
                if (a.dfin && state_number(a, q)) load_states<NS>(a.dfin, a.state_dtype, q * sstride + soff, g);
            }
            const f32x2 dv = s_d[k][lane];
            const float dy = s_g[k][lane];
            float u = 0.f, qa = 0.f;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                g[i] += dy * Cv[i];
                vC[k * NS + i] = dy * h[k][i];
                vB[k * NS + i] = g[i] * dv[1];
                u += g[i] * Bv[i];
                g[i] *= e[k][i];
                const float q = g[i] * prev[i];
                qa += q * A[i];
                dAt[i] += q * dv[0];
            }
            s_u[w][k][lane] = u;
            s_q[w][k][lane] = qa;
            if (VL && (m.start >> k & 1)) {
                const int q = a.seq[r];
                if (a.dh0 && state_number(a, q) && p.live)
                    store_states<NS>(a.dh0, a.state_dtype, q * sstride + soff, g);
            }
        }
#pragma unroll
        for (int i = 0; i < NS; ++i) dA[i] += dAt[i];
        {
            const float sb = wave_sum64(vB), sc = wave_sum64(vC);
            const int k = lane / NS, i = lane % NS;
            if (t0 + k < a.seqlen) {
                part[(int64_t)(t0 + k) * N + n0 + i] = sb;
                part[part_c + (int64_t)(t0 + k) * N + n0 + i] = sc;
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < TPW; ++j) {
            const int k = w + j * NW, t = t0 + k;
            float y = Dc * xv[j], u = 0.f, q = 0.f;
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                y += s_y[i][k][lane];
                u += s_u[i][k][lane];
                q += s_q[i][k][lane];
            }
            const float ddt = (xv[j] * u + q) * sg[j];
            if (t < a.seqlen && p.live) {
                const int64_t o = (p.row0 + t) * a.channels + p.c;
                ((T*)a.dx)[o] = (T)(Dc * dyv[j] + dv_[j] * u);
                ((T*)a.ddt)[o] = (T)ddt;
                if (a.z) {
                    const float sz = sigmoid_f(zv[j]);
                    ((T*)a.dz)[o] = (T)(gv[j] * y * (sz * (1.f + zv[j] * (1.f - sz))));
                }
                dD += dyv[j] * xv[j];
                db += ddt;
            }
        }
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

// dB and dC from the channel blocks' sums: out[b][t][g][n] = sum over cblk blocks.
template <typename T>
__global__ __launch_bounds__(256) void k_scan_sum_bc(const float* part, int batch, int seqlen, int groups, int cblk, int N,
                                                     T* dB, T* dC) {
    const int64_t total = (int64_t)batch * seqlen * groups * N;
    int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= 2 * total) return;
    const bool c = i >= total;
    if (c) i -= total;
    const int n = (int)(i % N);
    const int64_t r = i / N;
    const int g = (int)(r % groups);
    const int64_t row = r / groups;
    const int t = (int)(row % seqlen);
    const int64_t b = row / seqlen;
    const int64_t stride = (int64_t)seqlen * N;
    const float* src = part + (c ? (int64_t)batch * groups * cblk * stride : 0) + (b * groups + g) * cblk * stride +
                       (int64_t)t * N + n;
    f32x4 s = *(const f32x4*)src;
    for (int k = 1; k < cblk; ++k) s += *(const f32x4*)(src + k * stride);
    *(typename TT<T>::v4*)((c ? dC : dB) + i) = cvt4<T>(s);
}

// dA, dD and ddt_bias from the rows of the partial sums.
__global__ __launch_bounds__(256) void k_scan_sum_params(const float* part_a, const float* part_d, int rows, int channels,
                                                         int N, float* dA, float* dD, float* db) {
    const int64_t na = (int64_t)channels * N, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const float* src;
    float* dst;
    int64_t stride;
    if (i < na) {
        src = part_a + i;
        dst = dA + i;
        stride = na;
    } else {
        const int64_t j = i - na;
        if (j >= 2 * (int64_t)channels) return;
        const bool second = j >= channels;
        const int64_t c = second ? j - channels : j;
        float* out = second ? db : dD;
        if (!out) return;
        src = part_d + (second ? (int64_t)rows * channels : 0) + c;
        dst = out + c;
        stride = channels;
    }
    float s = 0.f;
    for (int r = 0; r < rows; ++r) s += src[r * stride];
    *dst = s;
}

template <typename T, int NW, int NS>
hipError_t launch_scan_backward_n(ScanArgs& a, T* dB, T* dC, float* dA, float* dD, float* db, hipStream_t st) {
    void* args[] = {&a};
    const void* fn = a.seq ? (const void*)&k_scan_backward<T, NW, NS, true> : (const void*)&k_scan_backward<T, NW, NS, false>;
    hipError_t e = hipLaunchKernel(fn, dim3((unsigned)(a.batch * a.nsplit * a.groups * a.cblk)), dim3(NW * 64), args, 0, st);
    if (e != hipSuccess) return e;
    const int64_t quads = (int64_t)a.batch * a.seqlen * a.groups * a.dstate / 2;  // both tensors, 4 values a lane
    void* bargs[] = {&a.part_bc, &a.batch, &a.seqlen, &a.groups, &a.cblk, &a.dstate, &dB, &dC};
    e = hipLaunchKernel((const void*)&k_scan_sum_bc<T>, dim3((unsigned)((quads + 255) / 256)), dim3(256), bargs, 0, st);
    if (e != hipSuccess) return e;
    int rows = a.batch * a.nsplit;
    const int64_t items = (int64_t)a.channels * (a.dstate + 2);
    void* pargs[] = {&a.part_a, &a.part_d, &rows, &a.channels, &a.dstate, &dA, &dD, &db};
    return hipLaunchKernel((const void*)&k_scan_sum_params, dim3((unsigned)((items + 255) / 256)), dim3(256), pargs, 0, st);
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
