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

// One token a row: a lane a (row, channel).
template <typename T> __global__ __launch_bounds__(256) void k_recur_step(RecurArgs a) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)a.batch * a.channels) return;
    const int b = (int)(i / a.channels), c = (int)(i % a.channels);
    const int slot = a.slots ? a.slots[b] : b;
    T* out = (T*)a.out + i;
    if (slot < 0 || slot >= a.nseq) {
        *out = (T)0.f;
        return;
    }
    const float x = (float)((const T*)a.x)[b * a.xs + c], g = (float)((const T*)a.gate)[b * a.gs + c];
    const float ig = a.ig ? (float)((const T*)a.ig)[b * a.is + c] : 0.f;
    const int64_t at = (int64_t)slot * a.channels + c;
    const RecParams p = rec_params(a, c, true);
    const float r = gate_of(g, p.gb), d = __builtin_amdgcn_exp2f(p.A2 * r);
    float u = a.ig ? x * gate_of(ig, p.ib) : x;
    if (a.normalize) u *= beta_of(p.Am * r, d);
    const float h = __builtin_fmaf(d, state_at(a.pool, a.state_dtype, at), u);
    state_to(a.pool, a.state_dtype, at, h);
    *out = (T)h;
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
        const hipError_t e = hipLaunchKernel((const void*)&k_recur_clear, dim3((unsigned)(grid < 2048 ? grid : 2048)), dim3(256), args, 0, st);
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
    return hipLaunchKernel((const void*)&k_recur_sums, dim3((unsigned)((3 * (int64_t)a.channels + 63) / 64)), dim3(256), args, 0, st);
}

hipError_t launch_recur_step(RecurArgs& a, int in_dtype, hipStream_t st) {
    const int64_t n = (int64_t)a.batch * a.channels;
    const void* fn = in_dtype == DT_F32 ? (const void*)&k_recur_step<float>
                   : in_dtype == DT_F16 ? (const void*)&k_recur_step<_Float16> : (const void*)&k_recur_step<__bf16>;
    void* args[] = {&a};
    return hipLaunchKernel(fn, dim3((unsigned)((n + 255) / 256)), dim3(256), args, 0, st);
}

}  // namespace ssd
