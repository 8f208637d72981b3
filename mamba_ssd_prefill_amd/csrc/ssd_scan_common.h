// ssd_scan_common.h -- device code shared by the forward and the backward of the selective scan.
//
// A workgroup holds 64 channels of one batch row, one a lane; its NW waves hold NS states each
// of the N = NW * NS.  So B and C of a token are the same for a whole wave and are read as scalars, each
// wave's part of the recurrence needs no other, and only the sums over n (y, and two sums of the
// backward) cross waves, through LDS.  What a (token, channel) needs once -- the step d, d * x, the gate
// -- is computed by one of the waves, tokens dealt round robin.
#pragma once

#include "ssd_device.h"
#include "ssd_select.h"

namespace ssd {

constexpr float kLog2e = 1.44269504088896340736f;

// A log2(e), the decay's exponent for a step of 1, kept finite: no step (a token behind the end, padding) times an infinite A
// would be NaN, where the state has to stay as it is.  (A NaN stays one.)
__device__ inline float decay_rate(float A) {
    const float r = A * kLog2e;
    return r < -__FLT_MAX__ ? -__FLT_MAX__ : r;
}

// The rows of B (or C) of a tile for one wave, NS values each, read through the scalar cache (the data is written
// before the launch) a group of GROUP tokens at a time, so that a group can be on its way while the one
// before is used.  One base address a tile and 32-bit offsets: scalar instructions issue at the rate of vector
// ones, and 64-bit addresses for every token took more of them than the recurrence itself.
typedef const __attribute__((address_space(4))) char* ScalarPtr;
template <typename T, int NS> struct ScalarRows {
    static constexpr int WORDS = NS * (int)sizeof(T) / 4;  // 4-byte words of a row
    static constexpr int GROUP = WORDS <= 2 ? 4 : WORDS <= 4 ? 2 : 1;
    ScalarPtr base;
    uint32_t stride;
    int last;  // rows past the end read the last one
    __device__ inline ScalarRows(const T* rows, int64_t row_stride, int64_t row0, int t0, int seqlen) {
        stride = (uint32_t)row_stride * (uint32_t)sizeof(T);
        base = (ScalarPtr)((uintptr_t)rows + (uint64_t)(uint32_t)(row0 + t0) * stride);
        last = seqlen - 1 - t0;
    }
    struct Group {
        uint32_t w[GROUP][WORDS];
        __device__ inline void load(const ScalarRows& r, int k0) {
#pragma unroll
            for (int j = 0; j < GROUP; ++j) {
                const uint32_t off = (uint32_t)min(k0 + j, r.last) * r.stride;
                typedef const __attribute__((address_space(4))) uint32_t* Words;
#pragma unroll
                for (int i = 0; i < WORDS; ++i) w[j][i] = ((Words)(r.base + off))[i];
            }
        }
        __device__ inline void clear(int j) {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) w[j][i] = 0;
        }
        // token k0 + j as fp32
        __device__ inline void values(int j, float (&v)[NS]) const {
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int i = 0; i < NS; ++i) v[i] = __builtin_bit_cast(float, w[j][i]);
            } else {
#pragma unroll
                for (int i = 0; i < NS / 2; ++i) {
                    const uint32_t u = w[j][i];
                    if constexpr (__is_same(T, __bf16)) {
                        v[2 * i] = __builtin_bit_cast(float, u << 16);
                        v[2 * i + 1] = __builtin_bit_cast(float, u & 0xffff0000u);
                    } else {
                        const f16x2 h = __builtin_bit_cast(f16x2, u);
                        v[2 * i] = (float)h[0];
                        v[2 * i + 1] = (float)h[1];
                    }
                }
            }
        }
    };
};

// The rows of one tensor for a tile of tokens, as a buffer that ends with the batch row: loads of tokens past
// the end give zeros, stores to them (and from lanes without a channel) are dropped, and an access
// takes one 32-bit offset.  Rows are below 2^24 elements apart and there are below 2^31 of them, so a tile's
// offsets stay below 2^31 and its start is one 32 x 32 bit product.
template <typename T, int TOKENS> struct TileRows {
    __amdgpu_buffer_rsrc_t rsrc;
    uint32_t stride;
    // TOKENS rows from token t0 of a batch row (t0 < 0: none)
    __device__ inline TileRows(const void* base, int64_t row_stride, int64_t row0, int t0, int seqlen) {
        stride = (uint32_t)row_stride * (uint32_t)sizeof(T);
        int n = min(seqlen - t0, TOKENS);
        asm("" : "+s"(n));  // (else the two bounds become one vector instruction, with quarter-rate products behind it)
        n = t0 < 0 ? 0 : max(n, 0);
        rsrc = make_rsrc((const char*)base + (uint64_t)(uint32_t)(row0 + max(t0, 0)) * stride, (uint32_t)n * stride);
    }
    __device__ inline T load(int k, uint32_t lane_off) const {
        const int off = (int)(lane_off + (uint32_t)k * stride);
        if constexpr (sizeof(T) == 4) {
            const uint32_t u = __builtin_amdgcn_raw_buffer_load_b32(rsrc, off, 0, 0);
            return __builtin_bit_cast(T, u);
        } else {
            const uint16_t u = __builtin_amdgcn_raw_buffer_load_b16(rsrc, off, 0, 0);
            return __builtin_bit_cast(T, u);
        }
    }
    __device__ inline void store(int k, uint32_t lane_off, float v) const {
        const int off = (int)(lane_off + (uint32_t)k * stride);
        const T o = (T)v;
        if constexpr (sizeof(T) == 4)
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, o), rsrc, off, 0, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, o), rsrc, off, 0, 0);
    }
};
constexpr uint32_t kNoLane = 0x80000000u;  // a store offset past every buffer

// NS states at element offset `off`.
template <int NS> __device__ inline void load_states(const void* base, int dtype, int64_t off, float (&h)[NS]) {
#pragma unroll
    for (int i = 0; i < NS; i += 4) {
        f32x4 v;
        if (dtype == DT_F32) {
            v = *(const f32x4*)((const float*)base + off + i);
        } else if (dtype == DT_F16) {
            const f16x4 r = *(const f16x4*)((const _Float16*)base + off + i);
            v = f32x4{(float)r[0], (float)r[1], (float)r[2], (float)r[3]};
        } else {
            const bf16x4 r = *(const bf16x4*)((const __bf16*)base + off + i);
            v = f32x4{(float)r[0], (float)r[1], (float)r[2], (float)r[3]};
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) h[i + j] = v[j];
    }
}
template <int NS> __device__ inline void store_states(void* base, int dtype, int64_t off, const float (&h)[NS]) {
#pragma unroll
    for (int i = 0; i < NS; i += 4) {
        const f32x4 v = {h[i], h[i + 1], h[i + 2], h[i + 3]};
        if (dtype == DT_F32)
            *(f32x4*)((float*)base + off + i) = v;
        else if (dtype == DT_F16)
            *(f16x4*)((_Float16*)base + off + i) = cvt4<_Float16>(v);
        else
            *(bf16x4*)((__bf16*)base + off + i) = cvt4<__bf16>(v);
    }
}

// A lane exchange within 16 lanes that rides on the instruction using it.
template <int CTRL> __device__ inline float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

// softplus(v) = max(v, 0) + log1p(u), u = exp(-|v|).  log1p(u) = log(s) + (u - (s - 1)) / s to first order in
// what rounding s = 1 + u loses; s - 1 is exact, and the division is left out: where s is not next to 1 the
// term is below a step of the result.  The hardware logarithm is relative to its result near 1 too, so small
// steps keep their relative precision.
__device__ inline float step_f(float v) {
    const float u = __builtin_amdgcn_exp2f(-fabsf(v) * kLog2e), s = 1.f + u;
    return fmaxf(v, 0.f) + (__builtin_amdgcn_logf(s) * 0.693147180559945309417f + (u - (s - 1.f)));
}

// The steps of a wave's tokens.  (All of them behind one branch: a branch for each token keeps their chains of dependent
// instructions from running side by side.)
template <typename T, int K> __device__ inline void steps(const ScanArgs& a, const T (&dt)[K], float bias, float (&d)[K]) {
#pragma unroll
    for (int j = 0; j < K; ++j) d[j] = f32of(dt[j]) + bias;
    if (a.softplus) {
#pragma unroll
        for (int j = 0; j < K; ++j) d[j] = step_f(d[j]);
    }
}

// softplus'(v)
__device__ inline float sigmoid_f(float v) { return __builtin_amdgcn_rcpf(1.f + __expf(-v)); }

// The kernel's own arguments, read again from the kernarg segment (scalar loads that hit the cache).  Within a
// tile loop this keeps the two dozen pointers and strides from being held in scalar registers all along, which
// costs more in spills to vector lanes than the loads do.
__device__ inline const ScanArgs& args_again() {
    typedef const __attribute__((address_space(4))) ScanArgs* Ptr;
    Ptr p = (Ptr)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const ScanArgs*)p;
}

// Where a workgroup stands.
struct ScanPlace {
    int b, split, g, cblk;
    int c;        // this lane's channel
    bool live;    // false for lanes behind the group's last channel (they repeat it and store nothing)
    int64_t row0; // b * seqlen
};
__device__ inline ScanPlace scan_place(const ScanArgs& a) {
    ScanPlace p;
    int i = blockIdx.x;
    p.cblk = i % a.cblk;
    i /= a.cblk;
    p.g = i % a.groups;
    i /= a.groups;
    p.split = i % a.nsplit;
    p.b = i / a.nsplit;
    const int k = p.cblk * 64 + (int)(threadIdx.x & 63);
    p.live = k < a.dg;
    p.c = p.g * a.dg + (p.live ? k : a.dg - 1);
    p.row0 = (int64_t)p.b * a.seqlen;
    return p;
}

__device__ inline bool state_number(const ScanArgs& a, int q) { return q >= 0 && q < a.nseq; }

// Sequence starts and ends and padding among the T tokens from t0 (those past the end are padding): bit k for token t0 + k.
struct SeqMasks {
    uint32_t start, end, pad;
};
template <int T> __device__ inline SeqMasks seq_masks(const ScanArgs& a, int64_t row0, int t0) {
    const int k = threadIdx.x & 63, t = t0 + k;
    bool s = false, e = false, p = true;
    if (k < T && t < a.seqlen) {
        const int32_t q = a.seq[row0 + t];
        p = !state_number(a, q);
        s = t == 0 || a.seq[row0 + t - 1] != q;
        e = t == a.seqlen - 1 || a.seq[row0 + t + 1] != q;
    }
    return SeqMasks{(uint32_t)__ballot(s), (uint32_t)__ballot(e), (uint32_t)__ballot(p)};
}

// The state v behind a split whose steps sum to d (infinite: nothing passes), `own` its state from a zero start.  (A
// zero state passes nothing either, also where negative steps make the decay's product infinite.)
__device__ inline float join_one(float A2, float v, float d, float own) {
    return d == __builtin_inff() || v == 0.f ? own : __builtin_amdgcn_exp2f(d * A2) * v + own;
}

// Carries v through `n` time splits in order, v = decay(k) v + *place(k), and leaves it in their places.  step(k) is
// the sum of steps that v decays by on the way (infinite: nothing passes).  Eight splits' values are
// loaded together, so that the chain waits for one load in eight.
template <typename Step, typename Place>
__device__ inline void join_splits(float A2, float v, int n, Step step, Place place) {
    for (int k0 = 0; k0 < n; k0 += 8) {
        float own[8], d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int k = min(k0 + j, n - 1);
            own[j] = *place(k);
            d[j] = step(k);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (k0 + j >= n) break;
            v = join_one(A2, v, d[j], own[j]);
            *place(k0 + j) = v;
        }
    }
}

// The same inside a pass over the splits, for a wave's own NS states of up to kFoldSplits splits: h after n splits,
// without the join's launch.  With more splits every workgroup's own walk takes longer than that launch: 1 x 131 x 1536 in 9
// splits takes 16.4 us a call so and 19.1 with the launch, but the main pass of 2 x 2048 x 5120 in 19 splits 119.8 us
// against 109.5 + 7.5, the backward of 2 x 500 x 1536 in some 30 splits 38.6 against 28.0 + 6.1.
constexpr int kFoldSplits = 16;
template <int NS, typename Step, typename Place>
__device__ inline void fold_splits(const float (&A2)[NS], float (&h)[NS], int n, Step step, Place place) {
    for (int k0 = 0; k0 < n; k0 += 4) {
        float own[4][NS], d[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = min(k0 + j, n - 1);
            load_states<NS>(place(k), DT_F32, 0, own[j]);
            d[j] = step(k);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (k0 + j >= n) break;
#pragma unroll
            for (int i = 0; i < NS; ++i)
                h[i] = join_one(A2[i], h[i], d[j], own[j][i]);
        }
    }
}

}  // namespace ssd
