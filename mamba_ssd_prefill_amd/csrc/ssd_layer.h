// ssd_layer.h -- argument blocks and launchers of the residual norm, the matrix product with its epilogue and the gated
// recurrence (kernels in ssd_norm.hip, ssd_linear*.hip, ssd_recur.hip; checks in ssd_layer_api.cpp).  Layouts are
// described in include/mamba_ssd.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssd_linear_plan.h"

namespace ssd {

// ---- residual norm ----------------------------------------------------------------------------
struct RmsArgs {
    const void* x;  // the backward's: the sum
    const void* res;
    const float* w;
    void* out;  // values or codes
    float* scales;
    void* sum;
    // backward
    const void* dout;
    const void* dsum;
    void* dx;
    void* dres;
    float* part;  // [parts][width]: sums of dw over the rows of a workgroup
    int64_t rows, xs, rs;
    int width, res_dtype, format;  // format -1: values
    int parts;
    float eps;
};
constexpr int kNormMaxWidth = 16384;
constexpr int kNormParts = 1024;  // workgroups of the backward at most
int norm_parts(int64_t rows, int width, int in_dtype);

hipError_t launch_rms_norm(RmsArgs& a, int in_dtype, hipStream_t st);
hipError_t launch_rms_norm_backward(RmsArgs& a, int in_dtype, float* dw, hipStream_t st);

// ---- matrix product ---------------------------------------------------------------------------
struct LinearArgs {
    const void* x;  // [M] rows of kbytes, xs bytes apart
    const void* w;  // [N] rows of kbytes, ws bytes apart
    const float* bias;
    const void* res;  // [M][N] out type, rows rs elements apart
    const float* sx;  // [M] or NULL
    const float* sw;  // [N] or NULL
    void* out;        // [M][N]
    void* pre;        // [M][N] or NULL
    float* part;      // [splits][M][N] fp32 where the contraction is split
    int64_t xs, ws, rs;
    int M, N, kbytes, act, out_dtype;
    int splits, steps_per_split;
};
// b: a second product in the same launch (by linear_plan_two), or NULL
hipError_t launch_linear(LinearArgs& a, LinearArgs* b, int type, const LinearPlan& p, hipStream_t st);

// Rows copied into ones that the product takes: kp values a row, those behind the source's zero.
struct PackArgs {
    const void* src;  // [rows] of cols values, stride elements apart
    void* dst;        // [rows][kp], or transposed: [cols][kp] with kp >= rows
    int64_t rows, cols, stride, kp;
};
// Two operands' in one launch (dst NULL: none).
hipError_t launch_pack(PackArgs& a, PackArgs& b, int elem_bytes, hipStream_t st);

// dpre = dout act'(pre), as rows of np >= N values and transposed with rows of mp >= M (either NULL: not wanted), and its
// sums over stretches of 64 rows.
struct DpreArgs {
    const void* dout;
    const void* pre;
    void* rows;
    void* cols;
    float* part;  // [ceil(M / 64)][N]
    int64_t M, N, np, mp;
    int act;
};
// That (where one of rows, cols and part is wanted), two operands transposed (dst NULL: none), and the sums of `part` (dbias NULL:
// not wanted).
hipError_t launch_linear_before(DpreArgs& a, PackArgs& p, PackArgs& q, int dtype, float* dbias, hipStream_t st);

// ---- gated recurrence -------------------------------------------------------------------------
struct RecurArgs {
    const void* x;
    const void* gate;
    const void* ig;
    const float* A;
    const float* gb;
    const float* ib;
    const int32_t* seq;
    const void* h0;
    void* out;
    void* fin;
    float* saved;  // [batch][kept][channels]: the state entering every kRecurSaved tokens
    // backward
    const void* dout;
    const void* dfin;
    void* dx;
    void* dgate;
    void* dig;
    void* dh0;
    float* part;  // [batch][tiles][3][channels]: dA, dgate_bias, din_bias
    // with more than one tile: what each does to the state (or its gradient), and how many workgroups of each chain of
    // tiles have started
    uint64_t* hops;     // [batch][tiles][channels]
    uint32_t* tickets;  // [batch][blocks][kTicketWords]
    // step
    void* pool;
    const int32_t* slots;
    int batch, seqlen, channels, nseq, state_dtype, normalize;
    int ntiles;
    int64_t xs, gs, is;
};
constexpr int kTicketWords = 32;  // counters on lines of their own
constexpr int kRecurWaves = 4;   // of a workgroup
constexpr int kRecurTile = 128;  // tokens of a tile of the forward pass
constexpr int kRecurSaved = 64;  // tokens between two kept states: a tile of the backward pass
constexpr int64_t recur_kept(int64_t seqlen) { return (seqlen + kRecurSaved - 1) / kRecurSaved; }
int64_t recur_tiles(int64_t seqlen, bool backward);
int64_t recur_blocks(int64_t channels, int in_dtype);  // workgroups of a tile of one batch row

hipError_t launch_recur(RecurArgs& a, int in_dtype, hipStream_t st);
hipError_t launch_recur_backward(RecurArgs& a, int in_dtype, float* dA, float* dgb, float* dib, hipStream_t st);
hipError_t launch_recur_step(RecurArgs& a, int in_dtype, hipStream_t st);

}  // namespace ssd
