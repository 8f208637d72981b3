// ssd_recur.hip -- what stands around the gated recurrence's tiles (ssd_recur.h): the words they meet by, the sums of the
// parameters' gradients, and single tokens on a pool of states (ssd_gated_recurrence_step in include/mamba_ssd.h).
#include "ssd_recur.h"
#include "ssd_sum_rows.h"

namespace ssd {

const void* rec_kernel_f32(const RecurArgs&, bool backward);
const void* rec_kernel_f16(const RecurArgs&, bool backward);
const void* rec_kernel_bf16(const RecurArgs&, bool backward);

__global__ __launch_bounds__(256) void k_recur_clear(uint64_t* hops, int64_t n, uint32_t* tickets, int64_t chains) {
    const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    for (int64_t i = i0; i < chains; i += step) tickets[i * kTicketWords] = 0;
    for (int64_t i = i0; i < n; i += step) hops[i] = kNoHop;
}

// dA, dgate_bias, din_bias from the tiles' sums: 64 columns of [3][channels] a workgroup.
__global__ __launch_bounds__(256) void k_recur_sums(const float* part, int parts, int channels, float* dA, float* dgb, float* dib) {
    __shared__ float lds[256];
    const int64_t n = 3 * (int64_t)channels, i = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
    const bool live = i < n;
    const float s = sum_rows<float>(part + (live ? i : 0), n, parts, lds, live);
    if (!live || threadIdx.x >= 64) return;
    const int e = (int)(i / channels), c = (int)(i % channels);
    float* to = e == 0 ? dA : e == 1 ? dgb : dib;
    if (to) to[c] = s;
}

// One token a row: a lane takes V channels of up to ROWS rows, whose parameters it reads once.
template <typename T, int V> __device__ inline void step_load(const T* p, float (&v)[V]) {
    typedef T Raw __attribute__((ext_vector_type(V), aligned(sizeof(T))));
    if constexpr (V == 1) {
        v[0] = (float)*p;
    } else {
        const Raw r = *(const Raw*)p;
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = (float)r[e];
    }
}
template <typename T, int V> __device__ inline void step_store(T* p, const float (&v)[V]) {
    typedef T Raw __attribute__((ext_vector_type(V), aligned(sizeof(T))));
    if constexpr (V == 1) {
        *p = (T)v[0];
    } else {
        Raw r;
#pragma unroll
        for (int e = 0; e < V; ++e) r[e] = (T)v[e];
        *(Raw*)p = r;
    }
}
template <int V> __device__ inline void state_load(const void* p, int dtype, int64_t i, float (&v)[V]) {
    if (dtype == DT_F32)
        step_load<float, V>((const float*)p + i, v);
    else if (dtype == DT_F16)
        step_load<_Float16, V>((const _Float16*)p + i, v);
    else
        step_load<__bf16, V>((const __bf16*)p + i, v);
}
template <int V> __device__ inline void state_store(void* p, int dtype, int64_t i, const float (&v)[V]) {
    if (dtype == DT_F32)
        step_store<float, V>((float*)p + i, v);
    else if (dtype == DT_F16)
        step_store<_Float16, V>((_Float16*)p + i, v);
    else
        step_store<__bf16, V>((__bf16*)p + i, v);
}
template <typename T, int V, int ROWS> __global__ __launch_bounds__(256) void k_recur_step(RecurArgs a) {
    const uint32_t per = (uint32_t)a.channels / V;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int c = (int)(i % per) * V, b0 = (int)(i / per) * ROWS;
    if (b0 >= a.batch) return;
    float x[ROWS][V], g[ROWS][V], ig[ROWS][V], h[ROWS][V];
    int slot[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        const int b = min(b0 + k, a.batch - 1);
        slot[k] = a.slots ? a.slots[b] : b;
    }
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        const int64_t b = min(b0 + k, a.batch - 1);
        step_load<T, V>((const T*)a.x + b * a.xs + c, x[k]);
        step_load<T, V>((const T*)a.gate + b * a.gs + c, g[k]);
        if (a.ig) step_load<T, V>((const T*)a.ig + b * a.is + c, ig[k]);
    }
#pragma unroll
    for (int k = 0; k < ROWS; ++k)
        if (slot[k] >= 0 && slot[k] < a.nseq) state_load<V>(a.pool, a.state_dtype, (int64_t)slot[k] * a.channels + c, h[k]);
    RecParams p[V];
#pragma unroll
    for (int e = 0; e < V; ++e) p[e] = rec_params(a, c + e, true);
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        if (b0 + k >= a.batch) break;
        T* out = (T*)a.out + (int64_t)(b0 + k) * a.channels + c;
        if (slot[k] < 0 || slot[k] >= a.nseq) {
#pragma unroll
            for (int e = 0; e < V; ++e) out[e] = (T)0.f;
            continue;
        }
        float r[V], u[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            r[e] = gate_of(g[k][e], p[e].gb);
            u[e] = x[k][e];
        }
        if (a.ig) {
#pragma unroll
            for (int e = 0; e < V; ++e) u[e] *= gate_of(ig[k][e], p[e].ib);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float d = __builtin_amdgcn_exp2f(p[e].A2 * r[e]);
            if (a.normalize) u[e] *= beta_of(p[e].Am * r[e], d);
            h[k][e] = __builtin_fmaf(d, h[k][e], u[e]);
        }
        state_store<V>(a.pool, a.state_dtype, (int64_t)slot[k] * a.channels + c, h[k]);
        step_store<T, V>(out, h[k]);
    }
}

int64_t recur_tiles(int64_t seqlen, bool backward) {
    const int tile = backward ? RecBwd::TILE : RecFwd::TILE;
    return (seqlen + tile - 1) / tile;
}
int64_t recur_blocks(int64_t channels, int in_dtype) {
    const int64_t ch = in_dtype == DT_F32 ? RecGeo<float, RecFwd>::CH : RecGeo<_Float16, RecFwd>::CH;
    return (channels + ch - 1) / ch;
}

static hipError_t launch_rec_any(RecurArgs& a, int in_dtype, bool backward, hipStream_t st) {
    const int64_t chains = recur_blocks(a.channels, in_dtype) * a.batch;
    if (a.ntiles > 1) {
        int64_t n = (int64_t)a.batch * a.ntiles * a.channels, c = chains;
        void* args[] = {&a.hops, &n, &a.tickets, &c};
        const int64_t grid = (n + 1023) / 1024;
        const hipError_t e =
            hipLaunchKernel((const void*)&k_recur_clear, dim3((unsigned)(grid < 2048 ? grid : 2048)), dim3(256), args, 0, st);
        if (e != hipSuccess) return e;
    }
    const void* fn = in_dtype == DT_F32 ? rec_kernel_f32(a, backward)
                   : in_dtype == DT_F16 ? rec_kernel_f16(a, backward) : rec_kernel_bf16(a, backward);
    void* args[] = {&a};
    return hipLaunchKernel(fn, dim3((unsigned)(chains * a.ntiles)), dim3(64 * (backward ? RecBwd::W : RecFwd::W)), args, 0, st);
}

hipError_t launch_recur(RecurArgs& a, int in_dtype, hipStream_t st) { return launch_rec_any(a, in_dtype, false, st); }

hipError_t launch_recur_backward(RecurArgs& a, int in_dtype, float* dA, float* dgb, float* dib, hipStream_t st) {
    const hipError_t e = launch_rec_any(a, in_dtype, true, st);
    if (e != hipSuccess) return e;
    int parts = a.batch * a.ntiles;
    void* args[] = {&a.part, &parts, &a.channels, &dA, &dgb, &dib};
    return hipLaunchKernel((const void*)&k_recur_sums, dim3((unsigned)((3 * (int64_t)a.channels + 63) / 64)), dim3(256), args, 0,
                           st);
}

// HBM-bound: 256 x 5120, bf16 with fp32 states, 21 MB, 7.9 us with the launch.  Two channels a lane where their number is even, and
// four rows where that leaves 512 workgroups (one row 8.2 us, four channels 9.2 us).
template <typename T> static hipError_t launch_step_t(RecurArgs& a, hipStream_t st) {
    const int v = a.channels % 2 ? 1 : 2;
    const int64_t lanes = (int64_t)a.batch * (a.channels / v);
    const bool four = lanes / 4 >= 512 * 256;
    const void* fn = v == 2 ? (four ? (const void*)&k_recur_step<T, 2, 4> : (const void*)&k_recur_step<T, 2, 1>)
                            : (four ? (const void*)&k_recur_step<T, 1, 4> : (const void*)&k_recur_step<T, 1, 1>);
    const int64_t n = (four ? ((int64_t)a.batch + 3) / 4 : a.batch) * (int64_t)(a.channels / v);
    void* args[] = {&a};
    return hipLaunchKernel(fn, dim3((unsigned)((n + 255) / 256)), dim3(256), args, 0, st);
}
hipError_t launch_recur_step(RecurArgs& a, int in_dtype, hipStream_t st) {
    switch (in_dtype) {
    case DT_F32: return launch_step_t<float>(a, st);
    case DT_F16: return launch_step_t<_Float16>(a, st);
    case DT_BF16: return launch_step_t<__bf16>(a, st);
    default: return hipErrorNotSupported;
    }
}

}  // namespace ssd
