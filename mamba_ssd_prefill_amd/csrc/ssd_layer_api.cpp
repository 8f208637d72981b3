// ssd_layer_api.cpp -- the C ABI of the residual norm, the matrix product with its epilogue and the gated recurrence
// (include/mamba_ssd.h): argument checks (host only, before any HIP call), workspaces and dispatch.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/mamba_ssd.h"
#include "ssd_layer.h"

#define SSD_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

constexpr size_t kAlign = 256;  // workspace region alignment
constexpr int64_t kMaxIndex = (int64_t)1 << 31;
constexpr int64_t kMaxLanes = (int64_t)1 << 32;  // of a launch

size_t elem_size(int dt) { return dt == SSD_F32 ? 4 : dt == SSD_F16 || dt == SSD_BF16 ? 2 : 1; }
size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool dtype_ok(int dt) { return dt >= SSD_F32 && dt <= SSD_BF16; }
bool flag_ok(int f) { return f == 0 || f == 1; }
bool stride_ok(int64_t s, int64_t row) { return s == 0 || (s >= row && s < kMaxIndex); }

ssd_status_t hip_status(hipError_t e) {
    if (e == hipSuccess) return SSD_OK;
    return e == hipErrorNotSupported ? SSD_ERR_UNSUPPORTED : SSD_ERR_HIP;
}

// Whether [a, a + na) and [b, b + nb) have bytes in common (NULL: not given).
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t u = (uintptr_t)a, v = (uintptr_t)b;
    return a && b && (u < v ? v - u < na : u - v < nb);
}

// Regions of a workspace, one behind the other.
struct Regions {
    size_t total = 0;
    size_t add(size_t bytes) {
        const size_t at = total;
        total += align_up(bytes);
        return at;
    }
    size_t size() const { return total ? total : kAlign; }
};

}  // namespace

// ---- residual norm -----------------------------------------------------------------------------

namespace {

ssd_status_t validate_norm(const ssd_norm_params_t* p, bool backward) {
    if (!p) return SSD_ERR_NULL_POINTER;
    if (p->struct_size < sizeof(ssd_norm_params_t)) return SSD_ERR_INVALID_ARGUMENT;
    if (!dtype_ok(p->in_dtype) || (p->sum_dtype != p->in_dtype && p->sum_dtype != SSD_F32)) return SSD_ERR_INVALID_ARGUMENT;
    if (p->format != -1 && (backward || (p->format != SSD_CACHE_INT8 && p->format != SSD_CACHE_E4M3)))
        return SSD_ERR_INVALID_ARGUMENT;
    if (!(p->eps >= 0.f) || !isfinite(p->eps)) return SSD_ERR_INVALID_ARGUMENT;
    if (p->rows < 1 || p->width < 1 || p->rows >= kMaxIndex) return SSD_ERR_INVALID_SHAPE;
    if (p->width > ssd::kNormMaxWidth) return SSD_ERR_UNSUPPORTED;
    if (!stride_ok(p->x_stride, p->width) || !stride_ok(p->residual_stride, p->width)) return SSD_ERR_INVALID_SHAPE;
    return SSD_OK;
}

ssd::RmsArgs norm_args(const ssd_norm_params_t* p, const void* x, const float* w) {
    ssd::RmsArgs a{};
    a.x = x;
    a.w = w;
    a.rows = p->rows;
    a.width = p->width;
    a.res_dtype = p->sum_dtype;
    a.format = p->format;
    a.eps = p->eps;
    a.xs = p->x_stride ? p->x_stride : p->width;
    a.rs = p->residual_stride ? p->residual_stride : p->width;
    return a;
}

}  // namespace

SSD_EXPORT ssd_status_t ssd_rms_norm(const ssd_norm_params_t* p, const void* x, const float* w, const void* residual,
                                     void* out, float* scales, void* sum, void* stream) {
    const ssd_status_t s = validate_norm(p, false);
    if (s != SSD_OK) return s;
    if (!x || !w || !out || (p->format >= 0 && !scales) || (residual && !sum)) return SSD_ERR_NULL_POINTER;
    if ((p->format < 0 && scales) || (!residual && sum)) return SSD_ERR_INVALID_ARGUMENT;
    const size_t es = elem_size(p->in_dtype), rs = elem_size(p->sum_dtype);
    if (!aligned(x, es) || !aligned(w, 4) || !aligned(residual, rs) || (p->format < 0 && !aligned(out, es)) ||
        !aligned(scales, 4) || !aligned(sum, rs))
        return SSD_ERR_MISALIGNED;
    ssd::RmsArgs a = norm_args(p, x, w);
    // in place, each value is read before its lane writes it; anywhere else another lane's may not have been
    if (residual && !(sum == residual && a.rs == p->width) &&
        overlap(residual, (size_t)((p->rows - 1) * a.rs + p->width) * rs, sum, (size_t)p->rows * p->width * rs))
        return SSD_ERR_INVALID_ARGUMENT;
    a.res = residual;
    a.out = out;
    a.scales = scales;
    a.sum = sum;
    return hip_status(ssd::launch_rms_norm(a, p->in_dtype, (hipStream_t)stream));
}

SSD_EXPORT size_t ssd_rms_norm_backward_workspace_size(const ssd_norm_params_t* p) {
    if (validate_norm(p, true) != SSD_OK) return 0;
    return align_up((size_t)ssd::norm_parts(p->rows, p->width, p->in_dtype) * p->width * 4);
}

SSD_EXPORT ssd_status_t ssd_rms_norm_backward(const ssd_norm_params_t* p, const void* dout, const void* s_, const float* w,
                                              const void* dsum, void* dx, void* dresidual, float* dw, void* workspace,
                                              size_t workspace_bytes, void* stream) {
    const ssd_status_t s = validate_norm(p, true);
    if (s != SSD_OK) return s;
    if (!dout || !s_ || !w || (!dx && !dresidual) || !workspace) return SSD_ERR_NULL_POINTER;
    const size_t es = elem_size(p->in_dtype), rs = elem_size(p->sum_dtype);
    if (!aligned(dout, es) || !aligned(s_, rs) || !aligned(w, 4) || !aligned(dsum, rs) || !aligned(dx, es) ||
        !aligned(dresidual, rs) || !aligned(dw, 4) || !aligned(workspace, kAlign))
        return SSD_ERR_MISALIGNED;
    const size_t n = (size_t)p->rows * p->width;
    if (dresidual != dsum && overlap(dsum, n * rs, dresidual, n * rs)) return SSD_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < ssd_rms_norm_backward_workspace_size(p)) return SSD_ERR_WORKSPACE_TOO_SMALL;
    ssd::RmsArgs a = norm_args(p, s_, w);
    a.dout = dout;
    a.dsum = dsum;
    a.dx = dx;
    a.dres = dresidual;
    a.part = (float*)workspace;
    a.parts = ssd::norm_parts(p->rows, p->width, p->in_dtype);
    return hip_status(ssd::launch_rms_norm_backward(a, p->in_dtype, dw, (hipStream_t)stream));
}

// ---- matrix product ----------------------------------------------------------------------------

namespace {

constexpr int kMaxInt8Width = 131071;               // 128 * 128 * K stays below 2^31

ssd_status_t validate_linear(const ssd_linear_params_t* p, bool backward) {
    if (!p) return SSD_ERR_NULL_POINTER;
    if (p->struct_size < sizeof(ssd_linear_params_t)) return SSD_ERR_INVALID_ARGUMENT;
    if (p->in_dtype < SSD_F32 || p->in_dtype > (backward ? (int)SSD_BF16 : (int)SSD_IN_E4M3) || !dtype_ok(p->out_dtype) ||
        (backward && p->out_dtype != p->in_dtype) || p->act < SSD_ACT_NONE || p->act > SSD_ACT_GELU)
        return SSD_ERR_INVALID_ARGUMENT;
    if (p->rows < 1 || p->width < 1 || p->outs < 1) return SSD_ERR_INVALID_SHAPE;
    if (!stride_ok(p->x_stride, p->width) || !stride_ok(p->residual_stride, p->outs)) return SSD_ERR_INVALID_SHAPE;
    const size_t es = elem_size(p->in_dtype);
    const int64_t M = p->rows, K = p->width, N = p->outs;
    if (ssd::padded(K, es) * (int64_t)es >= ssd::kMaxRowBytes) return SSD_ERR_INVALID_SHAPE;
    if (p->in_dtype == SSD_IN_INT8 && K > kMaxInt8Width) return SSD_ERR_UNSUPPORTED;
    // lanes of the product (512 for 256 x 256 outputs) and of the operands' copies (one for 16 bytes of either, in one launch); of
    // the gradient behind the activation with the transposed copies (256 for 64 x 64 of any)
    const int64_t most = kMaxLanes / 256, mb = (M + 63) / 64, nb = (N + 63) / 64, kb = (K + 63) / 64 + 1;
    if (mb * nb >= most || mb * kb >= most || nb * kb >= most || (mb + nb) * kb >= most) return SSD_ERR_INVALID_SHAPE;
    if ((M + N) * (ssd::padded(K, es) * (int64_t)es / 16) >= kMaxLanes - 256) return SSD_ERR_INVALID_SHAPE;
    if (backward && mb * nb + (mb + nb) * kb >= most) return SSD_ERR_INVALID_SHAPE;
    if (backward && ssd::padded(M > N ? M : N, es) * (int64_t)es >= ssd::kMaxRowBytes)
        return SSD_ERR_INVALID_SHAPE;
    return SSD_OK;
}

// Where weight has to start so that rows cut out of one that starts on 16 bytes are taken: loaded as they are, or copied.
size_t weight_align(int64_t row_bytes, size_t es) { return row_bytes % 16 == 0 ? 16 : row_bytes % 4 == 0 ? 4 : es; }

// The workspace of a product: copies of the operands where their rows do not fit, and the sums of the splits.
struct LinearLayout : ssd::LinearForm {
    size_t x_off, w_off, part_off, total;
};

LinearLayout linear_layout(const ssd_linear_params_t* p) {
    const size_t es = elem_size(p->in_dtype);
    LinearLayout l{ssd::linear_form(p->rows, p->width, p->outs, p->x_stride, p->in_dtype, es)};
    Regions r;
    l.x_off = l.may_pack_x ? r.add((size_t)p->rows * l.kp * es) : 0;
    l.w_off = l.pack_w ? r.add((size_t)p->outs * l.kp * es) : 0;
    l.part_off = l.plan.splits > 1 ? r.add((size_t)l.plan.splits * p->rows * p->outs * 4) : 0;
    l.total = r.size();
    return l;
}

}  // namespace

SSD_EXPORT size_t ssd_linear_workspace_size(const ssd_linear_params_t* p) {
    if (validate_linear(p, false) != SSD_OK) return 0;
    return linear_layout(p).total;
}

SSD_EXPORT ssd_status_t ssd_linear(const ssd_linear_params_t* p, const void* x, const void* weight, const float* bias,
                                   const void* residual, const float* x_scale, const float* weight_scale, void* pre,
                                   void* out, void* workspace, size_t workspace_bytes, void* stream) {
    const ssd_status_t s = validate_linear(p, false);
    if (s != SSD_OK) return s;
    if (!x || !weight || !out || !workspace) return SSD_ERR_NULL_POINTER;
    if ((x_scale || weight_scale) && p->in_dtype < SSD_IN_INT8) return SSD_ERR_INVALID_ARGUMENT;
    const size_t es = elem_size(p->in_dtype), os = elem_size(p->out_dtype);
    LinearLayout l = linear_layout(p);
    if (!aligned(x, l.may_pack_x ? es : 16) || !aligned(weight, weight_align(p->width * (int64_t)es, es)) ||
        !aligned(bias, 4) || !aligned(residual, os) || !aligned(x_scale, 4) || !aligned(weight_scale, 4) ||
        !aligned(pre, os) || !aligned(out, os) || !aligned(workspace, kAlign))
        return SSD_ERR_MISALIGNED;
    // in place, each value is read by the lane that writes it; anywhere else another lane may still read
    const int64_t rs = p->residual_stride ? p->residual_stride : p->outs;
    if (residual && !(out == residual && rs == p->outs) &&
        overlap(residual, (size_t)((p->rows - 1) * rs + p->outs) * os, out, (size_t)p->rows * p->outs * os))
        return SSD_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < l.total) return SSD_ERR_WORKSPACE_TOO_SMALL;
    const hipStream_t st = (hipStream_t)stream;
    char* ws = (char*)workspace;
    const int64_t K = p->width;
    int64_t xs = p->x_stride ? p->x_stride : K, wstr = K;
    ssd::PackArgs px{}, pw{};
    if (l.pack_x || !aligned(x, l.plan.narrow ? 4 : 16)) {
        px = ssd::PackArgs{x, ws + l.x_off, p->rows, p->width, xs, l.kp};
        x = px.dst;
        xs = l.kp;
    }
    if (l.pack_w) {
        pw = ssd::PackArgs{weight, ws + l.w_off, p->outs, p->width, p->width, l.kp};
        weight = pw.dst;
        wstr = l.kp;
    }
    if (px.dst || pw.dst) {
        const hipError_t e = ssd::launch_pack(px, pw, (int)es, st);
        if (e != hipSuccess) return hip_status(e);
    }
    ssd::LinearArgs a{};
    a.x = x;
    a.w = weight;
    a.bias = bias;
    a.res = residual;
    a.sx = x_scale;
    a.sw = weight_scale;
    a.out = out;
    a.pre = pre;
    a.part = (float*)(ws + l.part_off);
    a.xs = xs * es;
    a.ws = wstr * es;
    a.rs = rs;
    a.M = p->rows;
    a.N = p->outs;
    a.kbytes = (int)((l.plan.narrow ? K : l.kp) * es);
    a.act = p->act;
    a.out_dtype = p->out_dtype;
    return hip_status(ssd::launch_linear(a, nullptr, p->in_dtype, l.plan, st));
}

namespace {

// The backward's workspace.
struct LinearBackLayout : ssd::LinearBackForm {
    bool rows;  // dpre as rows of its own (else dout serves)
    size_t rows_off, cols_off, wt_off, xt_off, part_off, bias_off, total;
};

LinearBackLayout linear_back_layout(const ssd_linear_params_t* p) {
    const size_t es = elem_size(p->in_dtype);
    const size_t M = p->rows, K = p->width, N = p->outs;
    LinearBackLayout l{ssd::linear_back_form(p->rows, p->width, p->outs, p->in_dtype, es)};
    l.rows = p->act || l.np != p->outs;
    Regions r;
    l.rows_off = l.rows ? r.add(M * l.np * es) : 0;
    l.cols_off = r.add(N * l.mp * es);
    l.wt_off = r.add(K * l.np * es);
    l.xt_off = r.add(K * l.mp * es);
    size_t part = 0;
    if (l.dx_plan.splits > 1) part = l.dx_plan.splits * M * K * 4;
    if (l.dw_plan.splits > 1 && l.dw_plan.splits * N * K * 4 > part) part = l.dw_plan.splits * N * K * 4;
    l.part_off = part ? r.add(part) : 0;
    l.bias_off = r.add((M + 63) / 64 * N * 4);
    l.total = r.size();
    return l;
}

}  // namespace

SSD_EXPORT size_t ssd_linear_backward_workspace_size(const ssd_linear_params_t* p) {
    if (validate_linear(p, true) != SSD_OK) return 0;
    return linear_back_layout(p).total;
}

SSD_EXPORT ssd_status_t ssd_linear_backward(const ssd_linear_params_t* p, const void* dout, const void* x, const void* weight,
                                            const void* pre, void* dx, void* dweight, float* dbias, void* workspace,
                                            size_t workspace_bytes, void* stream) {
    const ssd_status_t s = validate_linear(p, true);
    if (s != SSD_OK) return s;
    if (!dout || !x || !weight || (!dx && !dweight && !dbias) || (p->act && !pre) || !workspace) return SSD_ERR_NULL_POINTER;
    if (!p->act && pre) return SSD_ERR_INVALID_ARGUMENT;
    const size_t es = elem_size(p->in_dtype);
    const LinearBackLayout l = linear_back_layout(p);
    const bool rows = l.rows && dx;  // (else dx comes from dout itself)
    if (!aligned(dout, dx && !rows ? 16 : es) || !aligned(x, es) || !aligned(weight, es) || !aligned(pre, es) || !aligned(dx, es) ||
        !aligned(dweight, es) || !aligned(dbias, 4) || !aligned(workspace, kAlign))
        return SSD_ERR_MISALIGNED;
    if (workspace_bytes < l.total) return SSD_ERR_WORKSPACE_TOO_SMALL;
    const hipStream_t st = (hipStream_t)stream;
    char* ws = (char*)workspace;
    const int64_t M = p->rows, K = p->width, N = p->outs;
    ssd::DpreArgs d{};
    d.dout = dout;
    d.pre = pre;
    d.rows = rows ? ws + l.rows_off : nullptr;
    d.cols = dweight ? ws + l.cols_off : nullptr;
    d.part = dbias ? (float*)(ws + l.bias_off) : nullptr;
    d.M = M;
    d.N = N;
    d.np = l.np;
    d.mp = l.mp;
    d.act = p->act;
    ssd::PackArgs wt{}, xt{};
    if (dx) wt = ssd::PackArgs{weight, ws + l.wt_off, N, K, K, l.np};
    if (dweight) xt = ssd::PackArgs{x, ws + l.xt_off, M, K, p->x_stride ? p->x_stride : K, l.mp};
    const hipError_t before = ssd::launch_linear_before(d, wt, xt, p->in_dtype, dbias, st);
    if (before != hipSuccess) return hip_status(before);
    const auto product = [&](const void* xr, const void* wr, int64_t rows, int64_t row_bytes, void* out) {
        ssd::LinearArgs a{};
        a.x = xr;
        a.w = wr;
        a.xs = a.ws = row_bytes;
        a.kbytes = (int)row_bytes;
        a.M = (int)rows;
        a.N = p->width;
        a.rs = K;
        a.out = out;
        a.out_dtype = p->in_dtype;
        a.part = (float*)(ws + l.part_off);
        return a;
    };
    ssd::LinearArgs x_args = product(rows ? ws + l.rows_off : dout, wt.dst, M, l.np * es, dx);
    ssd::LinearArgs w_args = product(ws + l.cols_off, xt.dst, N, l.mp * es, dweight);
    if (dx && dweight && l.both_plan.splits) {  // (the longer contraction's workgroups first)
        ssd::LinearArgs &first = N > M ? x_args : w_args, &then = N > M ? w_args : x_args;
        return hip_status(ssd::launch_linear(first, &then, p->in_dtype, l.both_plan, st));
    }
    if (dx) {
        const hipError_t e = ssd::launch_linear(x_args, nullptr, p->in_dtype, l.dx_plan, st);
        if (e != hipSuccess) return hip_status(e);
    }
    if (dweight) {
        const hipError_t e = ssd::launch_linear(w_args, nullptr, p->in_dtype, l.dw_plan, st);
        if (e != hipSuccess) return hip_status(e);
    }
    return SSD_OK;
}

// ---- gated recurrence ----------------------------------------------------------------------------

namespace {

constexpr int64_t kMaxRecRow = (int64_t)1 << 21;  // elements between rows: a tile's 128 rows have 31-bit offsets

ssd_status_t validate_recurrence(const ssd_recurrence_params_t* p, bool step) {
    if (!p) return SSD_ERR_NULL_POINTER;
    if (p->struct_size < sizeof(ssd_recurrence_params_t)) return SSD_ERR_INVALID_ARGUMENT;
    if (!dtype_ok(p->in_dtype) || !dtype_ok(p->state_dtype) || !flag_ok(p->normalize)) return SSD_ERR_INVALID_ARGUMENT;
    if (p->batch < 1 || p->seqlen < 1 || p->channels < 1) return SSD_ERR_INVALID_SHAPE;
    if (step && (p->seqlen != 1 || p->nseq < 1)) return SSD_ERR_INVALID_SHAPE;
    const int64_t D = p->channels;
    if (D >= kMaxRecRow || (int64_t)p->batch * p->seqlen >= kMaxIndex) return SSD_ERR_INVALID_SHAPE;
    if (!stride_ok(p->x_stride, D) || !stride_ok(p->gate_stride, D) || !stride_ok(p->in_stride, D))
        return SSD_ERR_INVALID_SHAPE;
    if (!step && (p->x_stride >= kMaxRecRow || p->gate_stride >= kMaxRecRow || p->in_stride >= kMaxRecRow))
        return SSD_ERR_INVALID_SHAPE;
    if (step) return (int64_t)p->batch * D >= kMaxLanes ? SSD_ERR_INVALID_SHAPE : SSD_OK;
    const int64_t groups = ssd::recur_blocks(D, p->in_dtype) * p->batch * ssd::recur_tiles(p->seqlen, true);
    return groups >= kMaxLanes / (64 * ssd::kRecurWaves) ? SSD_ERR_INVALID_SHAPE : SSD_OK;
}

struct RecLayout {
    size_t hops_off, ticket_off, part_off, total;
};

RecLayout rec_layout(const ssd_recurrence_params_t* p, bool backward) {
    RecLayout l{};
    const size_t tiles = ssd::recur_tiles(p->seqlen, backward), n = p->batch * tiles * p->channels;
    Regions r;
    if (tiles > 1) {
        l.hops_off = r.add(n * 8);
        l.ticket_off = r.add((size_t)p->batch * ssd::recur_blocks(p->channels, p->in_dtype) * ssd::kTicketWords * 4);
    }
    if (backward) l.part_off = r.add(3 * n * 4);
    l.total = r.size();
    return l;
}

ssd::RecurArgs rec_args(const ssd_recurrence_params_t* p, const void* x, const void* gate, const float* A, const void* in_gate,
                        const float* gate_bias, const float* in_bias) {
    ssd::RecurArgs a{};
    a.x = x;
    a.gate = gate;
    a.ig = in_gate;
    a.A = A;
    a.gb = gate_bias;
    a.ib = in_bias;
    a.batch = p->batch;
    a.seqlen = p->seqlen;
    a.channels = p->channels;
    a.nseq = p->nseq;
    a.state_dtype = p->state_dtype;
    a.normalize = p->normalize;
    a.xs = p->x_stride ? p->x_stride : p->channels;
    a.gs = p->gate_stride ? p->gate_stride : p->channels;
    a.is = p->in_stride ? p->in_stride : p->channels;
    return a;
}

void rec_space(ssd::RecurArgs& a, const ssd_recurrence_params_t* p, const RecLayout& l, char* ws, bool backward) {
    a.ntiles = (int)ssd::recur_tiles(p->seqlen, backward);
    a.hops = (uint64_t*)(ws + l.hops_off);
    a.tickets = (uint32_t*)(ws + l.ticket_off);
    a.part = (float*)(ws + l.part_off);
}

ssd_status_t check_rec_inputs(const ssd_recurrence_params_t* p, const void* x, const void* gate, const float* A,
                              const void* in_gate, const float* gate_bias, const float* in_bias) {
    if (!x || !gate || !A) return SSD_ERR_NULL_POINTER;
    if (in_bias && !in_gate) return SSD_ERR_INVALID_ARGUMENT;
    const size_t es = elem_size(p->in_dtype);
    if (!aligned(x, es) || !aligned(gate, es) || !aligned(in_gate, es) || !aligned(A, 4) || !aligned(gate_bias, 4) ||
        !aligned(in_bias, 4))
        return SSD_ERR_MISALIGNED;
    return SSD_OK;
}

}  // namespace

SSD_EXPORT size_t ssd_gated_recurrence_workspace_size(const ssd_recurrence_params_t* p) {
    if (validate_recurrence(p, false) != SSD_OK) return 0;
    return rec_layout(p, false).total;
}

SSD_EXPORT size_t ssd_gated_recurrence_backward_workspace_size(const ssd_recurrence_params_t* p) {
    if (validate_recurrence(p, false) != SSD_OK) return 0;
    return rec_layout(p, true).total;
}

SSD_EXPORT size_t ssd_gated_recurrence_saved_size(const ssd_recurrence_params_t* p) {
    if (validate_recurrence(p, false) != SSD_OK) return 0;
    return (size_t)p->batch * ssd::recur_kept(p->seqlen) * p->channels * 4;
}

SSD_EXPORT ssd_status_t ssd_gated_recurrence(const ssd_recurrence_params_t* p, const void* x, const void* gate, const float* A,
                                             const void* in_gate, const float* gate_bias, const float* in_bias,
                                             const int32_t* seq_idx, const void* initial_state, void* out,
                                             void* final_state, void* saved, void* workspace, size_t workspace_bytes,
                                             void* stream) {
    ssd_status_t s = validate_recurrence(p, false);
    if (s == SSD_OK) s = check_rec_inputs(p, x, gate, A, in_gate, gate_bias, in_bias);
    if (s != SSD_OK) return s;
    if (!out || !workspace) return SSD_ERR_NULL_POINTER;
    if (seq_idx && p->nseq < 1) return SSD_ERR_INVALID_SHAPE;
    const size_t es = elem_size(p->in_dtype), ss = elem_size(p->state_dtype);
    if (!aligned(out, es) || !aligned(seq_idx, 4) || !aligned(initial_state, ss) || !aligned(final_state, ss) ||
        !aligned(saved, 4) || !aligned(workspace, kAlign))
        return SSD_ERR_MISALIGNED;
    const size_t states = (size_t)(seq_idx ? p->nseq : p->batch) * p->channels * ss;
    if (overlap(initial_state, states, final_state, states)) return SSD_ERR_INVALID_ARGUMENT;
    const RecLayout l = rec_layout(p, false);
    if (workspace_bytes < l.total) return SSD_ERR_WORKSPACE_TOO_SMALL;
    ssd::RecurArgs a = rec_args(p, x, gate, A, in_gate, gate_bias, in_bias);
    rec_space(a, p, l, (char*)workspace, false);
    a.seq = seq_idx;
    a.h0 = initial_state;
    a.out = out;
    a.fin = final_state;
    a.saved = (float*)saved;
    return hip_status(ssd::launch_recur(a, p->in_dtype, (hipStream_t)stream));
}

SSD_EXPORT ssd_status_t ssd_gated_recurrence_backward(
    const ssd_recurrence_params_t* p, const void* dout, const void* dfinal_state, const void* x, const void* gate, const float* A,
    const void* in_gate, const float* gate_bias, const float* in_bias, const int32_t* seq_idx, const void* initial_state,
    const void* saved, void* dx, void* dgate, float* dA, void* din_gate, float* dgate_bias, float* din_bias,
    void* dinitial_state, void* workspace, size_t workspace_bytes, void* stream) {
    ssd_status_t s = validate_recurrence(p, false);
    if (s == SSD_OK) s = check_rec_inputs(p, x, gate, A, in_gate, gate_bias, in_bias);
    if (s != SSD_OK) return s;
    if (!dout || !saved || !dx || !dgate || !dA || (in_gate && !din_gate) || !workspace) return SSD_ERR_NULL_POINTER;
    if ((din_gate || din_bias) && !in_gate) return SSD_ERR_INVALID_ARGUMENT;
    if (seq_idx && p->nseq < 1) return SSD_ERR_INVALID_SHAPE;
    const size_t es = elem_size(p->in_dtype), ss = elem_size(p->state_dtype);
    if (!aligned(dout, es) || !aligned(dx, es) || !aligned(dgate, es) || !aligned(din_gate, es) || !aligned(dA, 4) ||
        !aligned(dgate_bias, 4) || !aligned(din_bias, 4) || !aligned(seq_idx, 4) || !aligned(initial_state, ss) ||
        !aligned(dfinal_state, ss) || !aligned(dinitial_state, ss) || !aligned(saved, 4) || !aligned(workspace, kAlign))
        return SSD_ERR_MISALIGNED;
    const size_t states = (size_t)(seq_idx ? p->nseq : p->batch) * p->channels * ss;
    if (overlap(dfinal_state, states, dinitial_state, states)) return SSD_ERR_INVALID_ARGUMENT;
    const RecLayout l = rec_layout(p, true);
    if (workspace_bytes < l.total) return SSD_ERR_WORKSPACE_TOO_SMALL;
    ssd::RecurArgs a = rec_args(p, x, gate, A, in_gate, gate_bias, in_bias);
    rec_space(a, p, l, (char*)workspace, true);
    a.seq = seq_idx;
    a.h0 = initial_state;
    a.saved = (float*)const_cast<void*>(saved);
    a.dout = dout;
    a.dfin = dfinal_state;
    a.dx = dx;
    a.dgate = dgate;
    a.dig = din_gate;
    a.dh0 = dinitial_state;
    return hip_status(ssd::launch_recur_backward(a, p->in_dtype, dA, dgate_bias, din_bias, (hipStream_t)stream));
}

SSD_EXPORT ssd_status_t ssd_gated_recurrence_step(const ssd_recurrence_params_t* p, const void* x, const void* gate,
                                                  const float* A, const void* in_gate, const float* gate_bias,
                                                  const float* in_bias, void* state, const int32_t* slots, void* out,
                                                  void* stream) {
    ssd_status_t s = validate_recurrence(p, true);
    if (s == SSD_OK && !slots && p->nseq != p->batch) s = SSD_ERR_INVALID_SHAPE;
    if (s == SSD_OK) s = check_rec_inputs(p, x, gate, A, in_gate, gate_bias, in_bias);
    if (s != SSD_OK) return s;
    if (!state || !out) return SSD_ERR_NULL_POINTER;
    if (!aligned(state, elem_size(p->state_dtype)) || !aligned(out, elem_size(p->in_dtype)) || !aligned(slots, 4))
        return SSD_ERR_MISALIGNED;
    ssd::RecurArgs a = rec_args(p, x, gate, A, in_gate, gate_bias, in_bias);
    a.pool = state;
    a.slots = slots;
    a.out = out;
    return hip_status(ssd::launch_recur_step(a, p->in_dtype, (hipStream_t)stream));
}
