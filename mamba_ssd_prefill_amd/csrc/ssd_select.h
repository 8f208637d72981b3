// ssd_select.h -- argument blocks and launchers of the selective scan, the causal convolution and
// the 8-bit state cache (kernels in ssd_scan.hip, ssd_scan_bwd.hip, ssd_conv.hip, ssd_cache.hip; checks in
// ssd_select_api.cpp).  Layouts are described in include/mamba_ssd.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssd {

// ---- causal convolution ----------------------------------------------------------------------
// out[0..2] (or dout): channel ranges [0, split_a), [split_a, split_b), [split_b, channels).
struct CausalConvArgs {
    const void* x;
    const float* w;
    const float* bias;
    const int32_t* seq;
    const void* h0;
    void* out[3];
    void* fin;
    // backward
    const void* dout[3];
    const void* dfin;
    void* dx;
    float* part;  // [ceil(batch * nseg / 4)][width + 1][channels]: sums of dw, then dbias, over four segments
    void* dh0;
    // step
    void* pool;
    const int32_t* slots;
    int batch, seqlen, channels, width, silu, nseq, split_a, split_b;
    int rows, nseg;  // tokens per lane and segments per batch row
    int64_t xs;
};

// Tokens per lane of the backward (the rows of `part` that the workspace has to hold).
int conv_backward_rows(int64_t batch, int64_t seqlen, int64_t channels);

hipError_t launch_causal_conv(CausalConvArgs& a, int in_dtype, hipStream_t st);
hipError_t launch_causal_conv_backward(CausalConvArgs& a, int in_dtype, float* dw, float* db, hipStream_t st);
hipError_t launch_causal_conv_step(CausalConvArgs& a, int in_dtype, hipStream_t st);

// ---- selective scan ---------------------------------------------------------------------------
struct ScanArgs {
    const void* x;
    const void* dt;
    const float* A;
    const void* B;
    const void* C;
    const float* D;
    const float* dt_bias;
    const void* z;
    const int32_t* seq;
    const void* h0;
    void* out;
    void* fin;
    float* saved;  // [batch][tiles][channels][dstate]: the state entering each tile of kScanPeriod tokens
    // backward
    const void* dout;
    const void* dfin;
    void* dx;
    void* ddt;
    void* dz;
    void* dh0;
    float* part_bc;  // [2][batch][groups * cblk][seqlen][dstate]: dB and dC summed over a channel block
    float* part_a;   // [batch * nsplit][channels][dstate]
    float* part_d;   // [2][batch * nsplit][channels]: dD, ddt_bias
    // time splits: state (or, backward, gradient) entering each split, and each split's sum of steps
    float* split_state;  // [batch][nsplit][channels][dstate]
    float* split_sum;    // [batch][nsplit][channels]
    // step
    void* pool;
    const int32_t* slots;
    int batch, seqlen, channels, dstate, groups, dg, cblk, nseq, state_dtype, softplus;
    int nsplit, tiles_per_split, ntiles;
    int64_t xs, dts, zs, Bs, Cs;
};

// Tokens between two saved states.
constexpr int kScanPeriod = 8;

// Time splits of the forward and the backward: a function of the sizes alone, so that workspaces
// can be sized without a device.
int scan_splits(int64_t batch, int64_t seqlen, int64_t channels, int groups, int dstate, bool backward);

hipError_t launch_scan(ScanArgs& a, int in_dtype, hipStream_t st);
hipError_t launch_scan_backward(ScanArgs& a, int in_dtype, void* dB, void* dC, float* dA, float* dD, float* db,
                                hipStream_t st);
hipError_t launch_scan_step(ScanArgs& a, int in_dtype, hipStream_t st);

// ---- 8-bit state cache --------------------------------------------------------------------------
struct CacheArgs {
    const void* state_in;
    void* state_out;
    const int32_t* slots;
    uint8_t* codes;
    float* scales;
    int64_t elems;
    int batch, nslots, group, format, state_dtype;
};
hipError_t launch_cache_write(CacheArgs& a, hipStream_t st);
hipError_t launch_cache_read(CacheArgs& a, hipStream_t st);

}  // namespace ssd
