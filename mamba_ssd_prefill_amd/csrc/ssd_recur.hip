// ssd_recur.hip -- the gated linear recurrence over prompts, its gradients, and single tokens on a pool of states
// (ssd_gated_recurrence / _backward / _step in include/mamba_ssd.h).
//
//     r = sigmoid(gate + gate_bias),  i = sigmoid(in_gate + in_bias) (or 1),  a = exp(A r),  beta = sqrt(1 - a^2) (or 1)
//     h = a h + beta i x
//     g = dout + (a g of t+1),  dl = a g h of t-1 - (a^2 / beta) g i x     (l = A r)
//     dx = g beta i,  din_gate = g beta x i (1 - i),  dgate = dl A r (1 - r),  dA = sum dl r
//
// Both passes are HBM-bound (8 and 14 bytes a token and channel of 16 bits), so each reads its inputs once: a workgroup
// walks 32 channels of a batch row through time in tiles of kRecurTile tokens.  A lane holds two channels over a
// run of T tokens; the runs of a tile are joined by what each lets through (the product of its decays) and what it
// adds, over the four runs of a wave by lane exchanges and over waves through LDS.  The next tile's rows are on
// their way meanwhile.  Prompts of few channels are cut in time: a first pass finds what each split lets
// through and adds, and the main pass starts from the splits before it.
#include "ssd_layer.h"
#include "ssd_scan_common.h"

namespace ssd {

constexpr int kRecWaves = 8, kRecT = kRecurTile / (4 * kRecWaves), kRecThreads = 64 * kRecWaves;
static_assert(kRecT * 4 * kRecWaves == kRecurTile, "runs of a tile");
constexpr int kRecCh = 32;  // channels of a workgroup

// Two channels of a token.
struct Two {
    float c[2];
};

// The rows of one tensor for a tile as a buffer that ends with the batch row: tokens behind the end read as 0 and are not
// written; the same for lanes without a channel, by an offset past every buffer.
template <typename T, bool PAIRED> struct RecRows {
    __amdgpu_buffer_rsrc_t rsrc;
    uint32_t stride;
    __device__ inline RecRows(const void* base, int64_t row_stride, int64_t row, int ntok) {
        stride = (uint32_t)row_stride * (uint32_t)sizeof(T);
        rsrc = make_rsrc((const char*)base + row * (int64_t)stride, (uint32_t)max(ntok, 0) * stride);
    }
    typedef uint32_t Raw __attribute__((ext_vector_type(sizeof(T) == 4 ? 2 : 1)));
    struct Held {
        uint32_t w[sizeof(T) == 4 ? 2 : 1];
    };
    __device__ inline Held load(uint32_t tok, const uint32_t (&ch)[2]) const {
        Held h;
        const uint32_t o = tok * stride;
        if constexpr (sizeof(T) == 4) {
            if constexpr (PAIRED) {
                const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(rsrc, (int)(o + ch[0]), 0, 0);
                h.w[0] = v[0];
                h.w[1] = v[1];
            } else {
                h.w[0] = __builtin_amdgcn_raw_buffer_load_b32(rsrc, (int)(o + ch[0]), 0, 0);
                h.w[1] = __builtin_amdgcn_raw_buffer_load_b32(rsrc, (int)(o + ch[1]), 0, 0);
            }
        } else if constexpr (PAIRED) {
            h.w[0] = __builtin_amdgcn_raw_buffer_load_b32(rsrc, (int)(o + ch[0]), 0, 0);
        } else {
            const uint32_t lo = __builtin_amdgcn_raw_buffer_load_b16(rsrc, (int)(o + ch[0]), 0, 0);
            const uint32_t hi = __builtin_amdgcn_raw_buffer_load_b16(rsrc, (int)(o + ch[1]), 0, 0);
            h.w[0] = (lo & 0xffffu) | hi << 16;
        }
        return h;
    }
    __device__ static inline Two values(const Held& h) {
        if constexpr (sizeof(T) == 4) {
            return Two{{__builtin_bit_cast(float, h.w[0]), __builtin_bit_cast(float, h.w[1])}};
        } else if constexpr (__is_same(T, __bf16)) {
            return Two{{__builtin_bit_cast(float, h.w[0] << 16), __builtin_bit_cast(float, h.w[0] & 0xffff0000u)}};
        } else {
            const f16x2 v = __builtin_bit_cast(f16x2, h.w[0]);
            return Two{{(float)v[0], (float)v[1]}};
        }
    }
    __device__ inline void store(uint32_t tok, const uint32_t (&ch)[2], float v0, float v1) const {
        const uint32_t o = tok * stride;
        if constexpr (sizeof(T) == 4) {
            if constexpr (PAIRED) {
                __builtin_amdgcn_raw_buffer_store_b64(u32x2{__builtin_bit_cast(uint32_t, v0), __builtin_bit_cast(uint32_t, v1)},
                                                      rsrc, (int)(o + ch[0]), 0, 0);
            } else {
                __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v0), rsrc, (int)(o + ch[0]), 0, 0);
                __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v1), rsrc, (int)(o + ch[1]), 0, 0);
            }
        } else {
            const uint16_t a = __builtin_bit_cast(uint16_t, (T)v0), b = __builtin_bit_cast(uint16_t, (T)v1);
            if constexpr (PAIRED) {
                __builtin_amdgcn_raw_buffer_store_b32((uint32_t)a | (uint32_t)b << 16, rsrc, (int)(o + ch[0]), 0, 0);
            } else {
                __builtin_amdgcn_raw_buffer_store_b16(a, rsrc, (int)(o + ch[0]), 0, 0);
                __builtin_amdgcn_raw_buffer_store_b16(b, rsrc, (int)(o + ch[1]), 0, 0);
            }
        }
    }
};

__device__ inline float state_at(const void* p, int dtype, int64_t i) {
    return dtype == DT_F32 ? ((const float*)p)[i] : dtype == DT_F16 ? (float)((const _Float16*)p)[i] : (float)((const __bf16*)p)[i];
}
__device__ inline void state_to(void* p, int dtype, int64_t i, float v) {
    if (dtype == DT_F32)
        ((float*)p)[i] = v;
    else if (dtype == DT_F16)
        ((_Float16*)p)[i] = (_Float16)v;
    else
        ((__bf16*)p)[i] = (__bf16)v;
}

// sigmoid(v) = 1 / (1 + e), e = exp(-v), and 1 - sigmoid(v) = e / (1 + e), each right relative to itself (a gate closed
// so far that e is infinite is 0, and the other 1).
struct Gate {
    float s, c;
};
__device__ inline Gate gate_of(float v) {
    const float t = -v * kLog2e, e = __builtin_amdgcn_exp2f(t), s = __builtin_amdgcn_rcpf(1.f + e);
    return Gate{s, t > 126.f ? 1.f : e * s};
}

// sqrt(1 - exp(2 l)), l <= 0, a = exp(l).  Near 0 the difference loses what a was rounded by, so 1 - exp(y) comes
// from its series there: 8 terms are right to 2^-26 down to y = -1/2.
__device__ inline float beta_of(float l, float a) {
    const float y = 2.f * l;
    float p = __builtin_fmaf(y, 1.f / 40320.f, 1.f / 5040.f);
    p = __builtin_fmaf(y, p, 1.f / 720.f);
    p = __builtin_fmaf(y, p, 1.f / 120.f);
    p = __builtin_fmaf(y, p, 1.f / 24.f);
    p = __builtin_fmaf(y, p, 1.f / 6.f);
    p = __builtin_fmaf(y, p, 0.5f);
    p = __builtin_fmaf(y, p, 1.f);
    const float b2 = y > -0.5f ? -y * p : __builtin_fmaf(-a, a, 1.f);
    return __builtin_amdgcn_sqrtf(b2);
}

// A channel's parameters.  A is kept finite, so that a closed gate times an infinite A is not NaN.
struct RecParams {
    float A, A2, gb, ib;
};
__device__ inline RecParams rec_params(const RecurArgs& a, int c, bool live) {
    RecParams p{0.f, 0.f, 0.f, 0.f};
    if (live) {
        const float A = a.A[c];
        p.A = A < -0x1p100f ? -0x1p100f : A;
        p.A2 = p.A * kLog2e;
        p.gb = a.gb ? a.gb[c] : 0.f;
        p.ib = a.ib ? a.ib[c] : 0.f;
    }
    return p;
}

// What a run of tokens does to the state before it: h -> p h + q.  p = -1: nothing passes (a sequence starts in it).
struct Hop {
    float p, q;
};
__device__ inline Hop then(Hop f, Hop s) {  // f first
    if (s.p < 0.f) return s;
    return Hop{f.p < 0.f ? f.p : f.p * s.p, __builtin_fmaf(s.p, f.q, s.q)};
}
__device__ inline float after(Hop s, float h) { return s.p < 0.f ? s.q : __builtin_fmaf(s.p, h, s.q); }

__device__ inline Hop shift_hop(Hop v, int lanes) { return Hop{__shfl_up(v.p, lanes, 64), __shfl_up(v.q, lanes, 64)}; }
__device__ inline Hop shift_hop_down(Hop v, int lanes) { return Hop{__shfl_down(v.p, lanes, 64), __shfl_down(v.q, lanes, 64)}; }

// The state entering each lane's run, from the runs' hops and the state `carry` entering the tile, which becomes the one
// leaving it.  `lds` [waves][32]: a tile's own place (two used in turn).  REV: time runs backwards, from the
// last run to the first.
template <bool REV> __device__ inline float join_runs(Hop own, float& carry, Hop* lds, int slot) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), run = lane >> 4;
    Hop inc = own;
#pragma unroll
    for (int d = 1; d < 4; d *= 2) {
        const Hop o = REV ? shift_hop_down(inc, 16 * d) : shift_hop(inc, 16 * d);
        if (REV ? run + d < 4 : run >= d) inc = then(o, inc);
    }
    if (run == (REV ? 0 : 3)) lds[wave * kRecCh + slot] = inc;
    const Hop before = REV ? shift_hop_down(inc, 16) : shift_hop(inc, 16);  // of the wave's runs before this one
    __syncthreads();
    float h = carry, mine = 0.f;
#pragma unroll
    for (int k = 0; k < kRecWaves; ++k) {
        const int w = REV ? kRecWaves - 1 - k : k;
        if (w == wave) mine = h;
        h = after(lds[w * kRecCh + slot], h);
    }
    carry = h;
    return run == (REV ? 3 : 0) ? mine : after(before, mine);
}

// Where a workgroup stands.  Neighbouring channel blocks go to one XCD (workgroups are dealt to eight in turn), whose L2
// then holds the 128-byte lines that two of them share.
struct RecPlace {
    int b, split, c0, tok;     // first of this lane's channels, first token of its run in a tile
    bool live[2];
    int64_t row0;
};
__device__ inline RecPlace rec_place(const RecurArgs& a) {
    RecPlace p;
    const int nblk = (a.channels + kRecCh - 1) / kRecCh;
    uint32_t i = blockIdx.x;
    const uint32_t n = gridDim.x, whole = n / 8 * 8;
    if (i < whole) i = (i & 7) * (whole / 8) + i / 8;
    const int blk = (int)(i % (uint32_t)nblk);
    i /= (uint32_t)nblk;
    p.split = (int)(i % (uint32_t)a.nsplit);
    p.b = (int)(i / (uint32_t)a.nsplit);
    const int lane = threadIdx.x & 63;
    p.c0 = blk * kRecCh + (lane & 15) * 2;
    p.live[0] = p.c0 < a.channels;
    p.live[1] = p.c0 + 1 < a.channels;
    p.tok = ((int)(threadIdx.x >> 6) * 4 + (lane >> 4)) * kRecT;
    p.row0 = (int64_t)p.b * a.seqlen;
    return p;
}

// Of a lane's T tokens from t: which start a sequence, end one, and are padding (those behind the row's end are neither
// start nor end); their numbers.
struct RecSeq {
    uint32_t start, end, pad;
    int32_t q[kRecT];
};
__device__ inline RecSeq rec_seq(const RecurArgs& a, int64_t row0, int t) {
    RecSeq s{0, 0, 0, {}};
    const int32_t* seq = a.seq + row0;
    int32_t before = 0;
    if (t > 0 && t < a.seqlen) before = seq[t - 1];
#pragma unroll
    for (int j = 0; j < kRecT; ++j) {
        s.q[j] = -1;
        if (t + j < a.seqlen) {
            const int32_t q = seq[t + j];
            s.q[j] = q;
            if (t + j == 0 || before != q) s.start |= 1u << j;
            if (t + j == a.seqlen - 1 || seq[t + j + 1] != q) s.end |= 1u << j;
            if (q < 0 || q >= a.nseq) s.pad |= 1u << j;
            before = q;
        }
    }
    return s;
}

// Decays and additions of a lane's tokens.  Tokens behind the row's end leave the state as it is.
template <typename T, bool PAIRED, bool PACKED> struct RecTile {
    typedef RecRows<T, PAIRED> Rows;
    typename Rows::Held x[kRecT], g[kRecT], i[kRecT];
    __device__ inline void load(const RecurArgs& a, const RecPlace& p, const uint32_t (&ch)[2], int t0) {
        const int n = min(a.seqlen - t0, kRecurTile);
        const Rows rx(a.x, a.xs, p.row0 + min(t0, a.seqlen - 1), n), rg(a.gate, a.gs, p.row0 + min(t0, a.seqlen - 1), n);
#pragma unroll
        for (int j = 0; j < kRecT; ++j) {
            x[j] = rx.load(p.tok + j, ch);
            g[j] = rg.load(p.tok + j, ch);
        }
        if (a.ig) {
            const Rows ri(a.ig, a.is, p.row0 + min(t0, a.seqlen - 1), n);
#pragma unroll
            for (int j = 0; j < kRecT; ++j) i[j] = ri.load(p.tok + j, ch);
        }
    }
};

// The tile's decay and addition of token j, channel k.
struct RecStep {
    float a, u;
};
__device__ inline RecStep rec_step_of(const RecurArgs& a, const RecParams& p, float x, float g, float i) {
    const float r = gate_of(g + p.gb).s;
    const float d = __builtin_amdgcn_exp2f(p.A2 * r);
    float u = a.ig ? x * gate_of(i + p.ib).s : x;
    if (a.normalize) u *= beta_of(p.A * r, d);
    return RecStep{d, u};
}

// MAIN: outputs; else only what the split lets through and adds.
template <typename T, bool PAIRED, bool PACKED, bool MAIN> __global__ __launch_bounds__(kRecThreads) void k_recur(RecurArgs a) {
    typedef RecTile<T, PAIRED, PACKED> Tile;
    typedef typename Tile::Rows Rows;
    __shared__ Hop lds[2][2][kRecWaves * kRecCh];
    const RecPlace p = rec_place(a);
    const int slot = (threadIdx.x & 15) * 2;
    uint32_t ch[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) ch[k] = p.live[k] ? (uint32_t)(p.c0 + k) * (uint32_t)sizeof(T) : kNoLane;
    RecParams prm[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) prm[k] = rec_params(a, p.c0 + k, p.live[k]);
    const int first = p.split * a.tiles_per_split, last = min(first + a.tiles_per_split, a.ntiles);
    float carry[2] = {0.f, 0.f};
    Hop whole[2] = {{1.f, 0.f}, {1.f, 0.f}};
    if constexpr (MAIN) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (!p.live[k]) continue;
            if (!PACKED && a.h0) carry[k] = state_at(a.h0, a.state_dtype, (int64_t)p.b * a.channels + p.c0 + k);
            for (int s = 0; s < p.split; ++s) {
                const int64_t o = ((int64_t)p.b * a.nsplit + s) * a.channels + p.c0 + k;
                carry[k] = after(Hop{a.split_decay[o], a.split_state[o]}, carry[k]);
            }
        }
    }
    Tile next;
    if (first < last) next.load(a, p, ch, first * kRecurTile);
    for (int tile = first; tile < last; ++tile) {
        const int t0 = tile * kRecurTile;
        Tile now = next;
        if (tile + 1 < last) next.load(a, p, ch, t0 + kRecurTile);
        RecSeq sq;
        if constexpr (PACKED) sq = rec_seq(a, p.row0, t0 + p.tok);
        if (MAIN && a.saved && threadIdx.x < 16) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (p.live[k]) a.saved[((int64_t)p.b * a.ntiles + tile) * a.channels + p.c0 + k] = carry[k];
        }
        float d[kRecT][2], u[kRecT][2];
        Hop own[2] = {{1.f, 0.f}, {1.f, 0.f}};
#pragma unroll
        for (int j = 0; j < kRecT; ++j) {
            const Two x = Rows::values(now.x[j]), g = Rows::values(now.g[j]);
            Two i{{0.f, 0.f}};
            if (a.ig) i = Rows::values(now.i[j]);
            const bool in = t0 + p.tok + j < a.seqlen;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                RecStep s = rec_step_of(a, prm[k], x.c[k], g.c[k], i.c[k]);
                if (!in) s = RecStep{1.f, 0.f};
                if constexpr (PACKED) {
                    if (sq.start >> j & 1) {
                        const bool pad = sq.pad >> j & 1;
                        const float h0 = pad || !a.h0 || !p.live[k] ? 0.f
                            : state_at(a.h0, a.state_dtype, (int64_t)sq.q[j] * a.channels + p.c0 + k);
                        s = RecStep{-1.f, __builtin_fmaf(s.a, h0, s.u)};
                    }
                }
                d[j][k] = s.a;
                u[j][k] = s.u;
                own[k] = PACKED ? then(own[k], Hop{s.a, s.u}) : Hop{own[k].p * s.a, __builtin_fmaf(s.a, own[k].q, s.u)};
            }
        }
        float h[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if constexpr (MAIN) {
                h[k] = join_runs<false>(own[k], carry[k], lds[tile & 1][k], slot / 2);
            } else {
                // the split's hop: its runs' hops in order
                const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, run = lane >> 4;
                Hop inc = own[k];
#pragma unroll
                for (int e = 1; e < 4; e *= 2) {
                    const Hop o = shift_hop(inc, 16 * e);
                    if (run >= e) inc = then(o, inc);
                }
                if (run == 3) lds[tile & 1][k][wave * kRecCh + slot / 2] = inc;
                __syncthreads();
                for (int w = 0; w < kRecWaves; ++w) whole[k] = then(whole[k], lds[tile & 1][k][w * kRecCh + slot / 2]);
            }
        }
        if constexpr (MAIN) {
            const Rows ro(a.out, a.channels, p.row0 + t0, min(a.seqlen - t0, kRecurTile));
#pragma unroll
            for (int j = 0; j < kRecT; ++j) {
#pragma unroll
                for (int k = 0; k < 2; ++k) h[k] = after(Hop{d[j][k], u[j][k]}, h[k]);
                ro.store(p.tok + j, ch, h[0], h[1]);
                if constexpr (PACKED) {
                    if (a.fin && (sq.end & ~sq.pad) >> j & 1) {
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            if (p.live[k]) state_to(a.fin, a.state_dtype, (int64_t)sq.q[j] * a.channels + p.c0 + k, h[k]);
                    }
                }
            }
        }
    }
    if (threadIdx.x < 16) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (!p.live[k]) continue;
            if constexpr (!MAIN) {
                const int64_t o = ((int64_t)p.b * a.nsplit + p.split) * a.channels + p.c0 + k;
                a.split_decay[o] = whole[k].p;
                a.split_state[o] = whole[k].q;
            } else if (!PACKED && a.fin && last == a.ntiles) {
                state_to(a.fin, a.state_dtype, (int64_t)p.b * a.channels + p.c0 + k, carry[k]);
            }
        }
    }
}

// Gradients.  The tiles run from the last to the first.  MAIN false: what a split passes on to the tokens before it of
// the gradient behind it, and what it adds.
template <typename T, bool PAIRED, bool PACKED, bool MAIN>
__global__ __launch_bounds__(kRecThreads) void k_recur_backward(RecurArgs a) {
    typedef RecTile<T, PAIRED, PACKED> Tile;
    typedef typename Tile::Rows Rows;
    __shared__ Hop lds[2][2][2][kRecWaves * kRecCh];
    const RecPlace p = rec_place(a);
    const int slot = (threadIdx.x & 15) * 2;
    uint32_t ch[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) ch[k] = p.live[k] ? (uint32_t)(p.c0 + k) * (uint32_t)sizeof(T) : kNoLane;
    RecParams prm[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) prm[k] = rec_params(a, p.c0 + k, p.live[k]);
    const int first = p.split * a.tiles_per_split, last = min(first + a.tiles_per_split, a.ntiles);
    float carry[2] = {0.f, 0.f};
    float sA[2] = {0.f, 0.f}, sg[2] = {0.f, 0.f}, si[2] = {0.f, 0.f};
    Hop whole[2] = {{1.f, 0.f}, {1.f, 0.f}};
    if constexpr (MAIN) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (!p.live[k]) continue;
            if (!PACKED && a.dfin) carry[k] = state_at(a.dfin, a.state_dtype, (int64_t)p.b * a.channels + p.c0 + k);
            for (int s = a.nsplit - 1; s > p.split; --s) {
                const int64_t o = ((int64_t)p.b * a.nsplit + s) * a.channels + p.c0 + k;
                carry[k] = after(Hop{a.split_decay[o], a.split_state[o]}, carry[k]);
            }
        }
    }
    for (int tile = last - 1; tile >= first; --tile) {
        const int t0 = tile * kRecurTile, n = min(a.seqlen - t0, kRecurTile);
        Tile now;
        now.load(a, p, ch, t0);
        typename Rows::Held dout[kRecT];
        const Rows rd(a.dout, a.channels, p.row0 + t0, n);
#pragma unroll
        for (int j = 0; j < kRecT; ++j) dout[j] = rd.load(p.tok + j, ch);
        RecSeq sq;
        if constexpr (PACKED) sq = rec_seq(a, p.row0, t0 + p.tok);
        Gate r[kRecT][2], i[kRecT][2];
        float d[kRecT][2], be[kRecT][2];
        Hop own[2] = {{1.f, 0.f}, {1.f, 0.f}};
#pragma unroll
        for (int j = 0; j < kRecT; ++j) {
            const Two x = Rows::values(now.x[j]), g = Rows::values(now.g[j]);
            Two iv{{0.f, 0.f}};
            if (a.ig) iv = Rows::values(now.i[j]);
            const bool in = t0 + p.tok + j < a.seqlen;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                r[j][k] = gate_of(g.c[k] + prm[k].gb);
                i[j][k] = a.ig ? gate_of(iv.c[k] + prm[k].ib) : Gate{1.f, 0.f};
                d[j][k] = __builtin_amdgcn_exp2f(prm[k].A2 * r[j][k].s);
                be[j][k] = a.normalize ? beta_of(prm[k].A * r[j][k].s, d[j][k]) : 1.f;
                Hop s{d[j][k], x.c[k] * i[j][k].s * be[j][k]};
                if (!in) s = Hop{1.f, 0.f};
                if constexpr (PACKED) {
                    if (sq.start >> j & 1) {
                        const bool pad = sq.pad >> j & 1;
                        const float h0 = pad || !a.h0 || !p.live[k] ? 0.f
                            : state_at(a.h0, a.state_dtype, (int64_t)sq.q[j] * a.channels + p.c0 + k);
                        s = Hop{-1.f, __builtin_fmaf(s.p, h0, s.q)};
                    }
                    own[k] = then(own[k], s);
                } else {
                    own[k] = Hop{own[k].p * s.p, __builtin_fmaf(s.p, own[k].q, s.q)};
                }
            }
        }
        // the state entering the run, and then what each token passes on of the gradient behind it
        float before[kRecT][2];
        Hop back[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if constexpr (MAIN) {
                float c = p.live[k] ? a.saved[((int64_t)p.b * a.ntiles + tile) * a.channels + p.c0 + k] : 0.f;
                float h = join_runs<false>(own[k], c, lds[tile & 1][0][k], slot / 2);
#pragma unroll
                for (int j = 0; j < kRecT; ++j) {
                    if constexpr (PACKED) {
                        if (sq.start >> j & 1)
                            h = sq.pad >> j & 1 || !a.h0 || !p.live[k] ? 0.f
                                : state_at(a.h0, a.state_dtype, (int64_t)sq.q[j] * a.channels + p.c0 + k);
                    }
                    before[j][k] = h;
                    h = __builtin_fmaf(d[j][k], h, Rows::values(now.x[j]).c[k] * i[j][k].s * be[j][k]);
                }
            }
            back[k] = Hop{1.f, 0.f};
#pragma unroll
            for (int j = kRecT - 1; j >= 0; --j) {
                const bool in = t0 + p.tok + j < a.seqlen;
                float o = Rows::values(dout[j]).c[k];
                Hop s{d[j][k], d[j][k] * o};  // v -> a (dout + v)
                if constexpr (PACKED) {
                    const bool pad = sq.pad >> j & 1;
                    if (sq.end >> j & 1) {  // behind a sequence's end: the gradient of its final state
                        const float v = pad || !a.dfin || !p.live[k] ? 0.f
                            : state_at(a.dfin, a.state_dtype, (int64_t)sq.q[j] * a.channels + p.c0 + k);
                        s = Hop{-1.f, d[j][k] * (o + v)};
                    }
                    if (sq.start >> j & 1 || pad) s = Hop{-1.f, 0.f};
                }
                if (!in) s = Hop{1.f, 0.f};
                back[k] = PACKED ? then(back[k], s) : Hop{back[k].p * s.p, __builtin_fmaf(s.p, back[k].q, s.q)};
            }
        }
        if constexpr (!MAIN) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, run = lane >> 4;
                Hop inc = back[k];
#pragma unroll
                for (int e = 1; e < 4; e *= 2) {
                    const Hop o = shift_hop_down(inc, 16 * e);
                    if (run + e < 4) inc = then(o, inc);
                }
                if (run == 0) lds[tile & 1][1][k][wave * kRecCh + slot / 2] = inc;
                __syncthreads();
                for (int w = kRecWaves - 1; w >= 0; --w) whole[k] = then(whole[k], lds[tile & 1][1][k][w * kRecCh + slot / 2]);
            }
        } else {
            float v[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) v[k] = join_runs<true>(back[k], carry[k], lds[tile & 1][1][k], slot / 2);
            const Rows rx(a.dx, a.channels, p.row0 + t0, n), rg(a.dgate, a.channels, p.row0 + t0, n);
            const Rows ri(a.ig ? a.dig : a.dgate, a.channels, p.row0 + t0, a.ig ? n : 0);
#pragma unroll
            for (int j = kRecT - 1; j >= 0; --j) {
                const bool in = t0 + p.tok + j < a.seqlen;
                const Two x = Rows::values(now.x[j]), o = Rows::values(dout[j]);
                float dx[2], dg[2], di[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    bool pad = !in;
                    if constexpr (PACKED) {
                        pad = pad || (sq.pad >> j & 1);
                        if (sq.end >> j & 1)
                            v[k] = pad || !a.dfin || !p.live[k] ? 0.f
                                : state_at(a.dfin, a.state_dtype, (int64_t)sq.q[j] * a.channels + p.c0 + k);
                    }
                    const float g = o.c[k] + v[k];
                    const float gx = g * x.c[k], gi = gx * i[j][k].s;
                    float dl = d[j][k] * g * before[j][k];
                    // (beta = 0, a closed gate: the product with r (1 - r) goes to 0)
                    if (a.normalize && be[j][k] != 0.f) dl -= d[j][k] * d[j][k] / be[j][k] * gi;
                    const float dr = dl * prm[k].A;
                    dx[k] = pad ? 0.f : g * be[j][k] * i[j][k].s;
                    dg[k] = pad ? 0.f : dr * r[j][k].s * r[j][k].c;
                    di[k] = pad ? 0.f : gi * be[j][k] * i[j][k].c;
                    sA[k] += pad ? 0.f : dl * r[j][k].s;
                    sg[k] += dg[k];
                    si[k] += di[k];
                    if (in) v[k] = d[j][k] * g;
                    if constexpr (PACKED) {
                        if (sq.start >> j & 1) {
                            if (a.dh0 && !pad && p.live[k])
                                state_to(a.dh0, a.state_dtype, (int64_t)sq.q[j] * a.channels + p.c0 + k, v[k]);
                        }
                        if (pad) v[k] = 0.f;
                    }
                }
                rx.store(p.tok + j, ch, dx[0], dx[1]);
                rg.store(p.tok + j, ch, dg[0], dg[1]);
                if (a.ig) ri.store(p.tok + j, ch, di[0], di[1]);
            }
        }
    }
    if constexpr (!MAIN) {
        if (threadIdx.x < 16) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (!p.live[k]) continue;
                const int64_t o = ((int64_t)p.b * a.nsplit + p.split) * a.channels + p.c0 + k;
                a.split_decay[o] = whole[k].p;
                a.split_state[o] = whole[k].q;
            }
        }
    } else {
        if (!PACKED && a.dh0 && first == 0 && threadIdx.x < 16) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (p.live[k]) state_to(a.dh0, a.state_dtype, (int64_t)p.b * a.channels + p.c0 + k, carry[k]);
        }
        // the sums over the workgroup's tokens: over a wave's four runs, then over waves
        __shared__ float sums[3][2][kRecWaves * kRecCh];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float s[3] = {sA[k], sg[k], si[k]};
#pragma unroll
            for (int e = 0; e < 3; ++e) {
                s[e] += __shfl_xor(s[e], 16, 64);
                s[e] += __shfl_xor(s[e], 32, 64);
                if ((threadIdx.x & 63) < 16) sums[e][k][(threadIdx.x >> 6) * kRecCh + slot / 2] = s[e];
            }
        }
        __syncthreads();
        if (threadIdx.x < 16) {
            const int64_t part = (int64_t)p.b * a.nsplit + p.split;
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int e = 0; e < 3; ++e) {
                    float s = 0.f;
                    for (int w = 0; w < kRecWaves; ++w) s += sums[e][k][w * kRecCh + slot / 2];
                    if (p.live[k]) a.part[(part * 3 + e) * a.channels + p.c0 + k] = s;
                }
        }
    }
}

// dA, dgate_bias, din_bias from the workgroups' sums.
__global__ __launch_bounds__(256) void k_recur_sums(const float* part, int parts, int channels, float* dA, float* dgb, float* dib) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= channels) return;
    float s[3] = {0.f, 0.f, 0.f};
    for (int k = 0; k < parts; ++k)
#pragma unroll
        for (int e = 0; e < 3; ++e) s[e] += part[((int64_t)k * 3 + e) * channels + c];
    if (dA) dA[c] = s[0];
    if (dgb) dgb[c] = s[1];
    if (dib) dib[c] = s[2];
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
    const RecStep s = rec_step_of(a, rec_params(a, c, true), x, g, ig);
    const float h = __builtin_fmaf(s.a, state_at(a.pool, a.state_dtype, at), s.u);
    state_to(a.pool, a.state_dtype, at, h);
    *out = (T)h;
}

int recur_splits(int64_t batch, int64_t seqlen, int64_t channels) {
    const int64_t blocks = batch * ((channels + kRecCh - 1) / kRecCh), tiles = (seqlen + kRecurTile - 1) / kRecurTile;
    int64_t s = blocks >= 256 ? 1 : (512 + blocks - 1) / blocks;
    if (s > tiles) s = tiles;
    if (s > 32) s = 32;
    const int64_t per = (tiles + s - 1) / s;
    return (int)((tiles + per - 1) / per);  // none without a tile
}

namespace {
template <typename T, bool PAIRED, bool PACKED> hipError_t launch_rec_t(RecurArgs& a, bool backward, hipStream_t st) {
    const unsigned blocks = (unsigned)((a.channels + kRecCh - 1) / kRecCh) * (unsigned)a.nsplit * (unsigned)a.batch;
    void* args[] = {&a};
    if (a.nsplit > 1) {
        const hipError_t e = hipLaunchKernel(backward ? (const void*)&k_recur_backward<T, PAIRED, PACKED, false>
                                                      : (const void*)&k_recur<T, PAIRED, PACKED, false>,
                                             dim3(blocks), dim3(kRecThreads), args, 0, st);
        if (e != hipSuccess) return e;
    }
    return hipLaunchKernel(backward ? (const void*)&k_recur_backward<T, PAIRED, PACKED, true>
                                    : (const void*)&k_recur<T, PAIRED, PACKED, true>,
                           dim3(blocks), dim3(kRecThreads), args, 0, st);
}
// Whether the two channels of a lane can be accessed together: every row starts on a multiple of that.
template <typename T> bool paired(const RecurArgs& a) {
    if (a.channels & 1) return false;
    if (sizeof(T) == 4) return true;
    if ((a.xs | a.gs | (a.ig ? a.is : 0)) & 1) return false;
    const void* p[] = {a.x, a.gate, a.ig, a.out, a.dout, a.dx, a.dgate, a.dig};
    for (const void* q : p)
        if ((uintptr_t)q & 3) return false;
    return true;
}
template <typename T> hipError_t launch_rec(RecurArgs& a, bool backward, hipStream_t st) {
    if (paired<T>(a))
        return a.seq ? launch_rec_t<T, true, true>(a, backward, st) : launch_rec_t<T, true, false>(a, backward, st);
    return a.seq ? launch_rec_t<T, false, true>(a, backward, st) : launch_rec_t<T, false, false>(a, backward, st);
}
hipError_t launch_rec_any(RecurArgs& a, int in_dtype, bool backward, hipStream_t st) {
    switch (in_dtype) {
    case DT_F32: return launch_rec<float>(a, backward, st);
    case DT_F16: return launch_rec<_Float16>(a, backward, st);
    case DT_BF16: return launch_rec<__bf16>(a, backward, st);
    default: return hipErrorNotSupported;
    }
}
}  // namespace

hipError_t launch_recur(RecurArgs& a, int in_dtype, hipStream_t st) { return launch_rec_any(a, in_dtype, false, st); }

hipError_t launch_recur_backward(RecurArgs& a, int in_dtype, float* dA, float* dgb, float* dib, hipStream_t st) {
    const hipError_t e = launch_rec_any(a, in_dtype, true, st);
    if (e != hipSuccess) return e;
    int parts = a.batch * a.nsplit;
    void* args[] = {&a.part, &parts, &a.channels, &dA, &dgb, &dib};
    return hipLaunchKernel((const void*)&k_recur_sums, dim3((unsigned)((a.channels + 255) / 256)), dim3(256), args, 0, st);
}

hipError_t launch_recur_step(RecurArgs& a, int in_dtype, hipStream_t st) {
    const int64_t n = (int64_t)a.batch * a.channels;
    const void* fn = in_dtype == DT_F32 ? (const void*)&k_recur_step<float>
                   : in_dtype == DT_F16 ? (const void*)&k_recur_step<_Float16> : (const void*)&k_recur_step<__bf16>;
    void* args[] = {&a};
    return hipLaunchKernel(fn, dim3((unsigned)((n + 255) / 256)), dim3(256), args, 0, st);
}

}  // namespace ssd
