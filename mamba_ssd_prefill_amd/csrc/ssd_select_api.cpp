// ssd_select_api.cpp -- the C ABI of the causal convolution, the selective scan and the 8-bit state
// cache (include/mamba_ssd.h): argument checks (host only, before any HIP call), workspaces and dispatch.
#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

#include "../../include/mamba_ssd.h"
#include "ssd_select.h"

#define SSD_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

constexpr size_t kAlign = 256;  // workspace region alignment
constexpr int64_t kMaxIndex = (int64_t)1 << 31;
constexpr int64_t kMaxLanes = (int64_t)1 << 32;  // of a launch

size_t elem_size(int dt) { return dt == SSD_F32 ? 4 : 2; }
size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool dtype_ok(int dt) { return dt >= SSD_F32 && dt <= SSD_BF16; }
bool flag_ok(int f) { return f == 0 || f == 1; }

ssd_status_t hip_status(hipError_t e) {
    if (e == hipSuccess) return SSD_OK;
    return e == hipErrorNotSupported ? SSD_ERR_UNSUPPORTED : SSD_ERR_HIP;
}

// Whether two arrays of states, `bytes` each, have bytes in common (NULL: not given).
bool overlap(const void* a, const void* b, size_t bytes) {
    const uintptr_t u = (uintptr_t)a, v = (uintptr_t)b;
    return a && b && (u < v ? v - u : u - v) < bytes;
}

// A row stride field: 0 (contiguous) or at least the row's length.
bool stride_ok(int64_t s, int64_t row) { return s == 0 || (s >= row && s < kMaxIndex); }

}  // namespace

// ---- causal convolution ------------------------------------------------------------------------

namespace {

ssd_status_t validate_conv(const ssd_conv_params_t* p, bool step) {
    if (!p) return SSD_ERR_NULL_POINTER;
    if (p->struct_size < sizeof(ssd_conv_params_t)) return SSD_ERR_INVALID_ARGUMENT;
    if (!dtype_ok(p->in_dtype) || !flag_ok(p->silu)) return SSD_ERR_INVALID_ARGUMENT;
    if (p->batch < 1 || p->seqlen < 1 || p->channels < 1) return SSD_ERR_INVALID_SHAPE;
    if (step && (p->seqlen != 1 || p->nseq < 1)) return SSD_ERR_INVALID_SHAPE;
    if (p->split_a < 0 || p->split_b < p->split_a || p->channels < p->split_b) return SSD_ERR_INVALID_SHAPE;
    if (!stride_ok(p->x_stride, p->channels)) return SSD_ERR_INVALID_SHAPE;
    if (p->width < 2 || p->width > 4) return SSD_ERR_UNSUPPORTED;
    // tokens have to fit 32-bit row indexes and lanes a grid (runs are of 32 tokens where there are that many)
    if ((int64_t)p->batch * p->seqlen >= kMaxIndex) return SSD_ERR_INVALID_SHAPE;
    const int64_t runs = (int64_t)p->batch * (((int64_t)p->seqlen + 31) / 32) + 3;
    if (((int64_t)p->channels + 63) / 64 * runs >= kMaxLanes / 64) return SSD_ERR_INVALID_SHAPE;
    return SSD_OK;
}

// The backward's sums take four lanes for each value of dw and dbias.
ssd_status_t validate_conv_backward(const ssd_conv_params_t* p) {
    const ssd_status_t s = validate_conv(p, false);
    if (s != SSD_OK) return s;
    if (((int64_t)p->channels * (p->width + 1) + 63) / 64 >= kMaxLanes / 256) return SSD_ERR_INVALID_SHAPE;
    return SSD_OK;
}

ssd::CausalConvArgs conv_args(const ssd_conv_params_t* p, const void* x, const float* w, const float* bias) {
    ssd::CausalConvArgs a{};
    a.x = x;
    a.w = w;
    a.bias = bias;
    a.batch = p->batch;
    a.seqlen = p->seqlen;
    a.channels = p->channels;
    a.width = p->width;
    a.silu = p->silu;
    a.nseq = p->nseq;
    a.split_a = p->split_a;
    a.split_b = p->split_b;
    a.xs = p->x_stride ? p->x_stride : p->channels;
    return a;
}

// The three channel ranges' tensors: each present and aligned where it has channels.
ssd_status_t check_ranges(const ssd_conv_params_t* p, const void* t0, const void* t1, const void* t2, size_t es) {
    const void* t[3] = {t0, t1, t2};
    const int n[3] = {p->split_a, p->split_b - p->split_a, p->channels - p->split_b};
    for (int i = 0; i < 3; ++i)
        if (n[i] && !t[i]) return SSD_ERR_NULL_POINTER;
    for (int i = 0; i < 3; ++i)
        if (n[i] && !aligned(t[i], es)) return SSD_ERR_MISALIGNED;
    return SSD_OK;
}

size_t conv_part_bytes(const ssd_conv_params_t* p) {
    const int64_t rows = ssd::conv_backward_rows(p->batch, p->seqlen, p->channels);
    const int64_t nseg = (p->seqlen + rows - 1) / rows;
    return align_up((size_t)((p->batch * nseg + 3) / 4) * p->channels * (p->width + 1) * 4);  // four runs a workgroup
}

}  // namespace

SSD_EXPORT ssd_status_t ssd_causal_conv(const ssd_conv_params_t* p, const void* x, const float* w, const float* bias,
                                        const int32_t* seq_idx, const void* initial_state, void* out0, void* out1,
                                        void* out2, void* final_state, void* stream) {
    ssd_status_t s = validate_conv(p, false);
    if (s != SSD_OK) return s;
    if (!x || !w) return SSD_ERR_NULL_POINTER;
    const size_t es = elem_size(p->in_dtype);
    s = check_ranges(p, out0, out1, out2, es);
    if (s != SSD_OK) return s;
    if (seq_idx && p->nseq < 1) return SSD_ERR_INVALID_SHAPE;
    if (!aligned(x, es) || !aligned(w, 4) || !aligned(bias, 4) || !aligned(seq_idx, 4) ||
        !aligned(initial_state, es) || !aligned(final_state, es))
        return SSD_ERR_MISALIGNED;
    const int64_t states = seq_idx ? p->nseq : p->batch;
    if (overlap(initial_state, final_state, states * p->channels * (p->width - 1) * es)) return SSD_ERR_INVALID_ARGUMENT;
    ssd::CausalConvArgs a = conv_args(p, x, w, bias);
    a.seq = seq_idx;
    a.h0 = initial_state;
    a.out[0] = out0;
    a.out[1] = out1;
    a.out[2] = out2;
    a.fin = final_state;
    return hip_status(ssd::launch_causal_conv(a, p->in_dtype, (hipStream_t)stream));
}

SSD_EXPORT size_t ssd_causal_conv_backward_workspace_size(const ssd_conv_params_t* p) {
    if (validate_conv_backward(p) != SSD_OK) return 0;
    return conv_part_bytes(p);
}

SSD_EXPORT ssd_status_t ssd_causal_conv_backward(const ssd_conv_params_t* p, const void* dout0, const void* dout1,
                                                 const void* dout2, const void* dfinal_state, const void* x,
                                                 const float* w, const float* bias, const int32_t* seq_idx,
                                                 const void* initial_state, void* dx, float* dw, float* dbias,
                                                 void* dinitial_state, void* workspace, size_t workspace_bytes,
                                                 void* stream) {
    ssd_status_t s = validate_conv_backward(p);
    if (s != SSD_OK) return s;
    if (!x || !w || !dx || !dw || !workspace) return SSD_ERR_NULL_POINTER;
    const size_t es = elem_size(p->in_dtype);
    s = check_ranges(p, dout0, dout1, dout2, es);
    if (s != SSD_OK) return s;
    if (seq_idx && p->nseq < 1) return SSD_ERR_INVALID_SHAPE;
    if (!aligned(x, es) || !aligned(w, 4) || !aligned(bias, 4) || !aligned(seq_idx, 4) ||
        !aligned(initial_state, es) || !aligned(dfinal_state, es) || !aligned(dx, es) || !aligned(dw, 4) ||
        !aligned(dbias, 4) || !aligned(dinitial_state, es) || !aligned(workspace, kAlign))
        return SSD_ERR_MISALIGNED;
    if (workspace_bytes < conv_part_bytes(p)) return SSD_ERR_WORKSPACE_TOO_SMALL;
    ssd::CausalConvArgs a = conv_args(p, x, w, bias);
    a.seq = seq_idx;
    a.h0 = initial_state;
    a.dout[0] = dout0;
    a.dout[1] = dout1;
    a.dout[2] = dout2;
    a.dfin = dfinal_state;
    a.dx = dx;
    a.dh0 = dinitial_state;
    a.part = (float*)workspace;
    return hip_status(ssd::launch_causal_conv_backward(a, p->in_dtype, dw, dbias, (hipStream_t)stream));
}

SSD_EXPORT ssd_status_t ssd_causal_conv_step(const ssd_conv_params_t* p, const void* x, const float* w,
                                             const float* bias, void* state, const int32_t* slots, void* out0,
                                             void* out1, void* out2, void* stream) {
    ssd_status_t s = validate_conv(p, true);
    if (s != SSD_OK) return s;
    if (!slots && p->nseq != p->batch) return SSD_ERR_INVALID_SHAPE;
    if (!x || !w || !state) return SSD_ERR_NULL_POINTER;
    const size_t es = elem_size(p->in_dtype);
    s = check_ranges(p, out0, out1, out2, es);
    if (s != SSD_OK) return s;
    if (!aligned(x, es) || !aligned(w, 4) || !aligned(bias, 4) || !aligned(state, es) || !aligned(slots, 4))
        return SSD_ERR_MISALIGNED;
    ssd::CausalConvArgs a = conv_args(p, x, w, bias);
    a.pool = state;
    a.slots = slots;
    a.out[0] = out0;
    a.out[1] = out1;
    a.out[2] = out2;
    return hip_status(ssd::launch_causal_conv_step(a, p->in_dtype, (hipStream_t)stream));
}

// ---- selective scan ------------------------------------------------------------------------------

namespace {

constexpr int kScanTile = 16;  // tokens of a forward tile
constexpr int64_t kMaxSeqlen = kMaxIndex - 64;  // a tile, and the 64 tokens whose numbers it looks at, end below 2^31
constexpr int64_t kMaxRow = (int64_t)1 << 24;  // elements between rows

ssd_status_t validate_scan(const ssd_scan_params_t* p, bool step) {
    if (!p) return SSD_ERR_NULL_POINTER;
    if (p->struct_size < sizeof(ssd_scan_params_t)) return SSD_ERR_INVALID_ARGUMENT;
    if (!dtype_ok(p->in_dtype) || !dtype_ok(p->state_dtype) || !flag_ok(p->dt_softplus)) return SSD_ERR_INVALID_ARGUMENT;
    if (p->batch < 1 || p->seqlen < 1 || p->channels < 1 || p->dstate < 1 || p->ngroups < 1)
        return SSD_ERR_INVALID_SHAPE;
    if (step && (p->seqlen != 1 || p->nseq < 1)) return SSD_ERR_INVALID_SHAPE;
    if (p->channels % p->ngroups) return SSD_ERR_INVALID_SHAPE;
    const int N = p->dstate;
    if (N != 8 && N != 16 && N != 32 && N != 64) return SSD_ERR_UNSUPPORTED;
    const int64_t gn = (int64_t)p->ngroups * N;
    if (!stride_ok(p->x_stride, p->channels) || !stride_ok(p->dt_stride, p->channels) ||
        !stride_ok(p->z_stride, p->channels) || !stride_ok(p->B_stride, gn) || !stride_ok(p->C_stride, gn))
        return SSD_ERR_INVALID_SHAPE;
    // a tile's rows are accessed at 32-bit offsets (a step's at 64-bit ones), those of B and C four bytes at a time
    if (p->channels >= kMaxRow || gn >= kMaxRow) return SSD_ERR_INVALID_SHAPE;
    if (!step && (p->x_stride >= kMaxRow || p->dt_stride >= kMaxRow || p->z_stride >= kMaxRow ||
                  p->B_stride >= kMaxRow || p->C_stride >= kMaxRow))
        return SSD_ERR_INVALID_SHAPE;
    if (p->in_dtype != SSD_F32 && (p->B_stride % 2 || p->C_stride % 2)) return SSD_ERR_MISALIGNED;
    // rows, tokens behind a row's end, channels and workgroups have to fit 32-bit indexes
    if (p->seqlen > kMaxSeqlen) return SSD_ERR_INVALID_SHAPE;
    if ((int64_t)p->batch * p->seqlen >= kMaxIndex || (int64_t)p->channels * N >= kMaxIndex)
        return SSD_ERR_INVALID_SHAPE;
    const int64_t blocks = (int64_t)p->batch * p->ngroups * ((p->channels / p->ngroups + 63) / 64);
    if (blocks >= kMaxLanes / 512) return SSD_ERR_INVALID_SHAPE;
    if (step && p->batch * (((int64_t)p->channels * (N / 4) + 255) / 256) >= kMaxLanes / 256) return SSD_ERR_INVALID_SHAPE;
    return SSD_OK;
}

int64_t scan_tiles(const ssd_scan_params_t* p, int tile) { return ((int64_t)p->seqlen + tile - 1) / tile; }

// The backward's sums take a lane for four values of dB or dC and for one of the parameters' gradients, by four waves.
ssd_status_t validate_scan_backward(const ssd_scan_params_t* p) {
    const ssd_status_t s = validate_scan(p, false);
    if (s != SSD_OK) return s;
    const int64_t runs = ((int64_t)p->batch * p->seqlen * (p->dstate / 2) + 63) / 64;
    if (runs >= kMaxLanes / 256 / p->ngroups) return SSD_ERR_INVALID_SHAPE;
    if (runs * p->ngroups + ((int64_t)p->channels * (p->dstate + 2) + 63) / 64 >= kMaxLanes / 256)
        return SSD_ERR_INVALID_SHAPE;
    return SSD_OK;
}

ssd::ScanArgs scan_args(const ssd_scan_params_t* p, const void* x, const void* dt, const float* A, const void* B,
                        const void* C, const float* D, const float* dt_bias, const void* z) {
    ssd::ScanArgs a{};
    a.x = x;
    a.dt = dt;
    a.A = A;
    a.B = B;
    a.C = C;
    a.D = D;
    a.dt_bias = dt_bias;
    a.z = z;
    a.batch = p->batch;
    a.seqlen = p->seqlen;
    a.channels = p->channels;
    a.dstate = p->dstate;
    a.groups = p->ngroups;
    a.dg = p->channels / p->ngroups;
    a.cblk = (a.dg + 63) / 64;
    a.nseq = p->nseq;
    a.state_dtype = p->state_dtype;
    a.softplus = p->dt_softplus;
    const int64_t D_ = p->channels, gn = (int64_t)p->ngroups * p->dstate;
    a.xs = p->x_stride ? p->x_stride : D_;
    a.dts = p->dt_stride ? p->dt_stride : D_;
    a.zs = p->z_stride ? p->z_stride : D_;
    a.Bs = p->B_stride ? p->B_stride : gn;
    a.Cs = p->C_stride ? p->C_stride : gn;
    a.ntiles = (int)scan_tiles(p, ssd::kScanPeriod);
    return a;
}

// Workspaces.  Forward: the states (and sums of steps) of the time splits.  Backward: those, then the partial sums.
struct ScanLayout {
    int nsplit;
    size_t state_off, sum_off, bc_off, a_off, d_off, total;
};

ScanLayout scan_layout(const ssd_scan_params_t* p, bool backward) {
    ScanLayout l{};
    const size_t B = p->batch, L = p->seqlen, D = p->channels, N = p->dstate, G = p->ngroups;
    const size_t cblk = (D / G + 63) / 64;
    l.nsplit = ssd::scan_splits(p->batch, p->seqlen, p->channels, p->ngroups, p->dstate, backward);
    const size_t S = l.nsplit;
    size_t off = 0;
    l.state_off = off;
    if (S > 1) off = align_up(off + B * S * D * N * 4);
    l.sum_off = off;
    if (S > 1) off = align_up(off + B * S * D * 4);
    if (backward) {
        l.bc_off = off;
        off = align_up(off + 2 * B * G * cblk * L * N * 4);
        l.a_off = off;
        off = align_up(off + B * S * D * N * 4);
        l.d_off = off;
        off = align_up(off + 2 * B * S * D * 4);
    }
    l.total = off ? off : kAlign;
    return l;
}

ssd_status_t check_scan_inputs(const ssd_scan_params_t* p, const void* x, const void* dt, const float* A, const void* B,
                               const void* C, const float* D, const float* dt_bias, const void* z) {
    if (!x || !dt || !A || !B || !C) return SSD_ERR_NULL_POINTER;
    const size_t es = elem_size(p->in_dtype);
    if (!aligned(x, es) || !aligned(dt, es) || !aligned(z, es) || !aligned(A, 16) || !aligned(B, 4) || !aligned(C, 4) ||
        !aligned(D, 4) || !aligned(dt_bias, 4))
        return SSD_ERR_MISALIGNED;
    return SSD_OK;
}

}  // namespace

SSD_EXPORT size_t ssd_selective_scan_workspace_size(const ssd_scan_params_t* p) {
    if (validate_scan(p, false) != SSD_OK) return 0;
    return scan_layout(p, false).total;
}

SSD_EXPORT size_t ssd_selective_scan_backward_workspace_size(const ssd_scan_params_t* p) {
    if (validate_scan_backward(p) != SSD_OK) return 0;
    return scan_layout(p, true).total;
}

SSD_EXPORT size_t ssd_selective_scan_saved_size(const ssd_scan_params_t* p) {
    if (validate_scan(p, false) != SSD_OK) return 0;
    return (size_t)p->batch * scan_tiles(p, ssd::kScanPeriod) * p->channels * p->dstate * 4;
}

SSD_EXPORT ssd_status_t ssd_selective_scan(const ssd_scan_params_t* p, const void* x, const void* dt, const float* A,
                                           const void* B, const void* C, const float* D, const float* dt_bias,
                                           const void* z, const int32_t* seq_idx, const void* initial_state, void* out,
                                           void* final_state, void* saved, void* workspace, size_t workspace_bytes,
                                           void* stream) {
    ssd_status_t s = validate_scan(p, false);
    if (s == SSD_OK) s = check_scan_inputs(p, x, dt, A, B, C, D, dt_bias, z);
    if (s != SSD_OK) return s;
    if (!out || !workspace) return SSD_ERR_NULL_POINTER;
    if (seq_idx && p->nseq < 1) return SSD_ERR_INVALID_SHAPE;
    if (!aligned(out, elem_size(p->in_dtype)) || !aligned(seq_idx, 4) || !aligned(initial_state, 16) ||
        !aligned(final_state, 16) || !aligned(saved, 16) || !aligned(workspace, kAlign))
        return SSD_ERR_MISALIGNED;
    const int64_t states = seq_idx ? p->nseq : p->batch;
    if (overlap(initial_state, final_state, states * p->channels * p->dstate * elem_size(p->state_dtype)))
        return SSD_ERR_INVALID_ARGUMENT;
    const ScanLayout l = scan_layout(p, false);
    if (workspace_bytes < l.total) return SSD_ERR_WORKSPACE_TOO_SMALL;
    ssd::ScanArgs a = scan_args(p, x, dt, A, B, C, D, dt_bias, z);
    a.seq = seq_idx;
    a.h0 = initial_state;
    a.out = out;
    a.fin = final_state;
    a.saved = (float*)saved;
    a.nsplit = l.nsplit;
    a.tiles_per_split = (int)((scan_tiles(p, kScanTile) + l.nsplit - 1) / l.nsplit);
    a.split_state = (float*)((char*)workspace + l.state_off);
    a.split_sum = (float*)((char*)workspace + l.sum_off);
    return hip_status(ssd::launch_scan(a, p->in_dtype, (hipStream_t)stream));
}

SSD_EXPORT ssd_status_t ssd_selective_scan_backward(const ssd_scan_params_t* p, const void* dout,
                                                    const void* dfinal_state, const void* x, const void* dt,
                                                    const float* A, const void* B, const void* C, const float* D,
                                                    const float* dt_bias, const void* z, const int32_t* seq_idx,
                                                    const void* initial_state, const void* saved, void* dx, void* ddt,
                                                    float* dA, void* dB, void* dC, float* dD, float* ddt_bias, void* dz,
                                                    void* dinitial_state, void* workspace, size_t workspace_bytes,
                                                    void* stream) {
    ssd_status_t s = validate_scan_backward(p);
    if (s == SSD_OK) s = check_scan_inputs(p, x, dt, A, B, C, D, dt_bias, z);
    if (s != SSD_OK) return s;
    if (!dout || !saved || !dx || !ddt || !dA || !dB || !dC || (z && !dz) || !workspace) return SSD_ERR_NULL_POINTER;
    if (dz && !z) return SSD_ERR_INVALID_ARGUMENT;
    if (seq_idx && p->nseq < 1) return SSD_ERR_INVALID_SHAPE;
    const size_t es = elem_size(p->in_dtype);
    if (!aligned(dout, es) || !aligned(dx, es) || !aligned(ddt, es) || !aligned(dz, es) || !aligned(dA, 4) ||
        !aligned(dB, 16) || !aligned(dC, 16) || !aligned(dD, 4) || !aligned(ddt_bias, 4) || !aligned(seq_idx, 4) ||
        !aligned(initial_state, 16) || !aligned(dfinal_state, 16) || !aligned(dinitial_state, 16) ||
        !aligned(saved, 16) || !aligned(workspace, kAlign))
        return SSD_ERR_MISALIGNED;
    const ScanLayout l = scan_layout(p, true);
    if (workspace_bytes < l.total) return SSD_ERR_WORKSPACE_TOO_SMALL;
    ssd::ScanArgs a = scan_args(p, x, dt, A, B, C, D, dt_bias, z);
    char* ws = (char*)workspace;
    a.seq = seq_idx;
    a.h0 = initial_state;
    a.saved = (float*)const_cast<void*>(saved);
    a.dout = dout;
    a.dfin = dfinal_state;
    a.dx = dx;
    a.ddt = ddt;
    a.dz = dz;
    a.dh0 = dinitial_state;
    a.nsplit = l.nsplit;
    a.tiles_per_split = (a.ntiles + l.nsplit - 1) / l.nsplit;
    a.split_state = (float*)(ws + l.state_off);
    a.split_sum = (float*)(ws + l.sum_off);
    a.part_bc = (float*)(ws + l.bc_off);
    a.part_a = (float*)(ws + l.a_off);
    a.part_d = (float*)(ws + l.d_off);
    return hip_status(ssd::launch_scan_backward(a, p->in_dtype, dB, dC, dA, dD, ddt_bias, (hipStream_t)stream));
}

SSD_EXPORT ssd_status_t ssd_selective_scan_step(const ssd_scan_params_t* p, const void* x, const void* dt,
                                                const float* A, const void* B, const void* C, const float* D,
                                                const float* dt_bias, const void* z, void* state,
                                                const int32_t* slots, void* out, void* stream) {
    ssd_status_t s = validate_scan(p, true);
    if (s == SSD_OK && !slots && p->nseq != p->batch) s = SSD_ERR_INVALID_SHAPE;
    if (s == SSD_OK) s = check_scan_inputs(p, x, dt, A, B, C, D, dt_bias, z);
    if (s != SSD_OK) return s;
    if (!state || !out) return SSD_ERR_NULL_POINTER;
    if (!aligned(state, 16) || !aligned(out, elem_size(p->in_dtype)) || !aligned(slots, 4)) return SSD_ERR_MISALIGNED;
    ssd::ScanArgs a = scan_args(p, x, dt, A, B, C, D, dt_bias, z);
    a.pool = state;
    a.slots = slots;
    a.out = out;
    return hip_status(ssd::launch_scan_step(a, p->in_dtype, (hipStream_t)stream));
}

// ---- 8-bit state cache ------------------------------------------------------------------------------

namespace {

ssd_status_t check_cache(const ssd_cache_params_t* p, const void* state, const int32_t* slots, const void* codes,
                         const float* scales) {
    if (!p) return SSD_ERR_NULL_POINTER;
    if (p->struct_size < sizeof(ssd_cache_params_t)) return SSD_ERR_INVALID_ARGUMENT;
    if (!dtype_ok(p->state_dtype) || (p->format != SSD_CACHE_INT8 && p->format != SSD_CACHE_E4M3))
        return SSD_ERR_INVALID_ARGUMENT;
    if (p->batch < 1 || p->nslots < 1 || p->elems < 1 || p->group < 1) return SSD_ERR_INVALID_SHAPE;
    if (p->group != 16 && p->group != 32 && p->group != 64 && p->group != 128) return SSD_ERR_UNSUPPORTED;
    if (p->elems % p->group || p->elems >= (int64_t)1 << 40) return SSD_ERR_INVALID_SHAPE;
    if (p->batch * ((p->elems + 2047) / 2048) >= kMaxLanes / 256) return SSD_ERR_INVALID_SHAPE;  // 8 values a lane
    if (!slots && p->nslots < p->batch) return SSD_ERR_INVALID_SHAPE;
    if (!state || !codes || !scales) return SSD_ERR_NULL_POINTER;
    if (!aligned(state, 16) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(slots, 4))
        return SSD_ERR_MISALIGNED;
    return SSD_OK;
}

ssd::CacheArgs cache_args(const ssd_cache_params_t* p, const int32_t* slots, const void* codes, const float* scales) {
    ssd::CacheArgs a{};
    a.slots = slots;
    a.codes = (uint8_t*)const_cast<void*>(codes);
    a.scales = const_cast<float*>(scales);
    a.elems = p->elems;
    a.batch = p->batch;
    a.nslots = p->nslots;
    a.group = p->group;
    a.format = p->format;
    a.state_dtype = p->state_dtype;
    return a;
}

}  // namespace

SSD_EXPORT ssd_status_t ssd_state_cache_write(const ssd_cache_params_t* p, const void* state, const int32_t* slots,
                                              void* codes, float* scales, void* stream) {
    const ssd_status_t s = check_cache(p, state, slots, codes, scales);
    if (s != SSD_OK) return s;
    ssd::CacheArgs a = cache_args(p, slots, codes, scales);
    a.state_in = state;
    return hip_status(ssd::launch_cache_write(a, (hipStream_t)stream));
}

SSD_EXPORT ssd_status_t ssd_state_cache_read(const ssd_cache_params_t* p, const void* codes, const float* scales,
                                             const int32_t* slots, void* state, void* stream) {
    const ssd_status_t s = check_cache(p, state, slots, codes, scales);
    if (s != SSD_OK) return s;
    ssd::CacheArgs a = cache_args(p, slots, codes, scales);
    a.state_out = state;
    return hip_status(ssd::launch_cache_read(a, (hipStream_t)stream));
}
