// ssd_conv.hip -- the causal depthwise convolution of width W in {2, 3, 4} with an optional SiLU: prompts,
// their gradients, and one token on a pool of states (ssd_causal_conv* in include/mamba_ssd.h).
//
//     pre[t] = bias + sum_k w[k] in[t - (W-1) + k],     out = silu(pre) or pre
//     dpre[t] = dout[t] silu'(pre[t]),   dx[s] = sum_i w[W-1-i] dpre[s+i],   dw[k] = sum_t dpre[t] in[t-(W-1)+k]
//
// All three are HBM-bound streams: at 2 x 4096 x 5376, W = 4, bf16 the forward moves 176 MB in 36.5 us (4.8 TB/s, where a
// large copy reaches 5.0), the backward 264 MB in 60 us (4.4) and 5 us for its sums; a step of one row takes the 2.8 us of
// a launch.  A lane owns CW neighbouring channels of a run of tokens and slides a
// window of W-1 inputs down them, so each input is read once a run plus a halo of W-1 rows;
// consecutive lanes take consecutive channels.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "ssd_device.h"
#include "ssd_select.h"
#include "ssd_sum_rows.h"

namespace ssd {

// CW elements in one access.  Rows are kept as loaded until they are used: converting a row that is still on its way
// would wait for it.
template <typename T, int CW> struct ConvPiece { typedef T type __attribute__((ext_vector_type(CW))); };
template <typename T> struct ConvPiece<T, 1> { struct type { T v; __device__ T operator[](int) const { return v; } }; };
template <typename T, int CW> __device__ inline typename ConvPiece<T, CW>::type load_raw(const T* p) {
    return *(const typename ConvPiece<T, CW>::type*)p;
}
template <typename T, int CW> __device__ inline void load_cw(const T* p, float (&v)[CW]) {
    const auto r = load_raw<T, CW>(p);
#pragma unroll
    for (int e = 0; e < CW; ++e) v[e] = (float)r[e];
}
template <typename T, int CW> __device__ inline void store_cw(T* p, const float (&v)[CW]) {
    if constexpr (CW > 1) {
        typename ConvPiece<T, CW>::type r;
#pragma unroll
        for (int e = 0; e < CW; ++e) r[e] = (T)v[e];
        *(typename ConvPiece<T, CW>::type*)p = r;
    } else {
        *p = (T)v[0];
    }
}

// A run of rows, loaded AHEAD rows before they are used.  The address moves on by a row a step and stays at the last
// one: a product for each row's address took more slots than the convolution's own.
template <typename T, int CW, int AHEAD> struct RowStream {
    typename ConvPiece<T, CW>::type r[AHEAD];
    const T* at;
    int64_t stride;
    int left;  // rows behind the one last asked for
    __device__ inline RowStream(const T* first, int64_t stride_, int rows) : at(first), stride(stride_), left(rows - 1) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            r[i] = load_raw<T, CW>(at);
            advance();
        }
    }
    __device__ inline void advance() {
        at += left > 0 ? stride : 0;
        --left;
    }
    __device__ inline void take(float (&v)[CW]) {
#pragma unroll
        for (int e = 0; e < CW; ++e) v[e] = (float)r[0][e];
#pragma unroll
        for (int i = 0; i + 1 < AHEAD; ++i) r[i] = r[i + 1];
        r[AHEAD - 1] = load_raw<T, CW>(at);
        advance();
    }
};

// Row `row` of channel c0 in a tensor split by channel ranges.
template <typename T> __device__ inline T* split_ptr(void* const* base, int sa, int sb, int ch, int c0, int64_t row) {
    if (c0 < sa) return (T*)base[0] + row * sa + c0;
    if (c0 < sb) return (T*)base[1] + row * (sb - sa) + (c0 - sa);
    return (T*)base[2] + row * (ch - sb) + (c0 - sb);
}

// The lane's item: a piece of CW channels and a run of a.rows tokens.  A wave takes 64 pieces of one run, so that
// tokens, sequence numbers and the branches on them are scalar; a workgroup takes four runs that follow one another:
// the rows that two runs both read then come from its own XCD's L2 (2 x 4096 x 5376 forward 47 us with 256
// pieces of one run, 39 us so).
struct ConvItem {
    int b, c0, t0, t1;
};
template <int CW> __device__ inline bool conv_item(const CausalConvArgs& a, ConvItem* it) {
    const int npc = a.channels / CW;
    const uint32_t pblocks = (uint32_t)(npc + 63) / 64;
    const int pc = (int)(blockIdx.x % pblocks) * 64 + (int)(threadIdx.x & 63);
    const uint32_t r = (blockIdx.x / pblocks) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (pc >= npc || r >= (uint32_t)a.batch * (uint32_t)a.nseg) return false;
    it->c0 = pc * CW;
    it->t0 = (int)(r % (uint32_t)a.nseg) * a.rows;
    it->b = (int)(r / (uint32_t)a.nseg);
    it->t1 = min(it->t0 + a.rows, a.seqlen);
    return true;
}

template <int W, int CW> struct ConvW {
    float w[W][CW], bias[CW];
    __device__ inline void load(const CausalConvArgs& a, int c0) {
#pragma unroll
        for (int e = 0; e < CW; ++e) {
            struct __attribute__((packed, aligned(4))) Taps { float v[W]; };  // one access, on any multiple of 4 bytes
            const Taps t = *(const Taps*)(a.w + (int64_t)(c0 + e) * W);
#pragma unroll
            for (int k = 0; k < W; ++k) w[k][e] = t.v[k];
            bias[e] = a.bias ? a.bias[c0 + e] : 0.f;
        }
    }
};

// Walks one sequence after another down a batch row: the number of the sequence holding the
// current token, its place in it (counted up to W-1), and the W-1 inputs before it.
template <typename T, int W, int CW, bool VL> struct ConvWalk {
    const CausalConvArgs& a;
    const int b, c0;
    typedef const __attribute__((address_space(4))) int32_t* Numbers;  // read through the scalar cache
    Numbers seq;
    int q, place, qn, qnn;  // qn, qnn: the numbers of the next token and of the one after it
    float win[W - 1][CW];

    __device__ inline ConvWalk(const CausalConvArgs& a_, int b_, int c0_) : a(a_), b(b_), c0(c0_) {
        seq = VL ? (Numbers)(uintptr_t)(a.seq + (int64_t)b * a.seqlen) : (Numbers)0;
    }
    __device__ inline const T* row(int t) const { return (const T*)a.x + ((int64_t)b * a.seqlen + t) * a.xs + c0; }
    __device__ inline bool has_state(int n) const { return n >= 0 && n < (VL ? a.nseq : a.batch); }
    // the window before a sequence's first token, shifted by `done` inputs already taken
    __device__ inline void load_state(int done) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            if (j + done > W - 2) continue;  // an input of the sequence itself
#pragma unroll
            for (int e = 0; e < CW; ++e)
                win[j][e] = a.h0 && has_state(q)
                                ? (float)((const T*)a.h0)[((int64_t)q * a.channels + c0 + e) * (W - 1) + j + done]
                                : 0.f;
        }
    }
    // stand before token t: the loads first, all at once (rows before the batch row's first are its first)
    __device__ inline void start(int t) {
        typename ConvPiece<T, CW>::type before[W - 1];
        int number[W];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) before[j] = load_raw<T, CW>(row(max(t - (W - 1) + j, 0)));
        if constexpr (VL) {
#pragma unroll
            for (int j = 0; j < W; ++j) number[j] = seq[max(t - j, 0)];
            qnn = seq[min(t + 1, a.seqlen - 1)];
            q = qn = number[0];
        } else {
            q = b;
        }
        place = 0;
#pragma unroll
        for (int j = 1; j < W; ++j)
            if (place == j - 1 && t >= j && (!VL || number[j] == q)) place = j;
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int e = 0; e < CW; ++e) win[j][e] = (float)before[j][e];
        if (place < W - 1) load_state(place);
    }
    // begin with token t, coming from t - 1 (or from start(t))
    __device__ inline void step_to(int t) {
        if constexpr (VL) {
            if (qn != q) {
                q = qn;
                place = 0;
                load_state(0);
            }
            qn = qnn;
            qnn = seq[min(t + 2, a.seqlen - 1)];  // loaded two tokens ahead, like the inputs
        }
    }
    __device__ inline void taps(const ConvW<W, CW>& k, const float (&cur)[CW], float (&pre)[CW]) const {
#pragma unroll
        for (int e = 0; e < CW; ++e) {
            float s = k.bias[e];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) s += k.w[j][e] * win[j][e];
            pre[e] = s + k.w[W - 1][e] * cur[e];
        }
    }
    __device__ inline void push(const float (&cur)[CW]) {
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j)
#pragma unroll
            for (int e = 0; e < CW; ++e) win[j][e] = win[j + 1][e];
#pragma unroll
        for (int e = 0; e < CW; ++e) win[W - 2][e] = cur[e];
        if (place < W) ++place;
    }
    // the window holds inputs (or the initial state) as they were, so this rounds nothing
    __device__ inline void store_state() const {
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int e = 0; e < CW; ++e)
                ((T*)a.fin)[((int64_t)q * a.channels + c0 + e) * (W - 1) + j] = (T)win[j][e];
    }
    __device__ inline bool last(int t) const { return t == a.seqlen - 1 || (VL && qn != q); }
};

// Rows on their way while one is used (2 and 4 measured alike forward; backward 70.0, 68.2, 67.7 us with 1, 2, 3 in
// runs of 32 tokens and 66.7, 71.4 with 2, 3 in runs of 16, at 2 x 4096 x 5376).
constexpr int kConvAhead = 2, kConvAheadBackward = 2;

template <typename T, int W, int CW, bool VL> __global__ __launch_bounds__(256) void k_causal_conv(CausalConvArgs a) {
    ConvItem it;
    if (!conv_item<CW>(a, &it)) return;
    ConvW<W, CW> k;
    k.load(a, it.c0);
    ConvWalk<T, W, CW, VL> s(a, it.b, it.c0);
    s.start(it.t0);
    T* out = split_ptr<T>(a.out, a.split_a, a.split_b, a.channels, it.c0, (int64_t)it.b * a.seqlen + it.t0);
    const int os = it.c0 < a.split_a ? a.split_a : it.c0 < a.split_b ? a.split_b - a.split_a : a.channels - a.split_b;
    RowStream<T, CW, kConvAhead> rows(s.row(it.t0), a.xs, it.t1 - it.t0);
#pragma unroll 4
    for (int t = it.t0; t < it.t1; ++t, out += os) {
        float cur[CW], pre[CW];
        rows.take(cur);
        s.step_to(t);
        s.taps(k, cur, pre);
        if (a.silu) {
#pragma unroll
            for (int e = 0; e < CW; ++e) pre[e] = silu_f(pre[e]);
        }
        store_cw<T, CW>(out, pre);
        s.push(cur);
        if (VL && a.fin && s.last(t) && s.has_state(s.q)) s.store_state();
    }
    // (outside the loop where it can be: a store that may or may not have been made makes the next row's wait one
    // for everything)
    if (!VL && a.fin && it.t1 == a.seqlen) s.store_state();
}

// silu'(v) = p (1 + v (1 - p)), p the sigmoid of v
__device__ inline float dsilu_f(float v) {
    const float p = __builtin_amdgcn_rcpf(1.f + __expf(-v));
    return p * (1.f + v * (1.f - p));
}

// One pass over a run of tokens and the W-1 tokens behind it: dpre of a token completes dx of the token
// W-1 before it.  dw and db: the lane's sums over its own tokens.
template <typename T, int W, int CW, bool VL, bool ST>
__device__ inline void conv_backward_run(const CausalConvArgs& a, const ConvItem& it, float (&dw)[W][CW], float (&db)[CW]) {
    ConvW<W, CW> k;
    k.load(a, it.c0);
    ConvWalk<T, W, CW, VL> s(a, it.b, it.c0);
    s.start(it.t0);
    const int64_t row0 = (int64_t)it.b * a.seqlen;
    const T* dout = split_ptr<T>((void* const*)a.dout, a.split_a, a.split_b, a.channels, it.c0, row0 + it.t0);
    const int os = it.c0 < a.split_a ? a.split_a : it.c0 < a.split_b ? a.split_b - a.split_a : a.channels - a.split_b;
    // dx of the W-1 tokens before the current one, still short of later tokens' terms
    float acc[W - 1][CW] = {};
    // gradients of the initial state, at a sequence's first tokens
    float dh[W - 1][CW] = {};
    const int end = min(it.t1 + W - 1, a.seqlen);
    // what the states add at token t, place `place` of its sequence
    auto states = [&](int t, int place, const float (&g)[CW], float (&here)[CW]) {
        const bool last = s.last(t);
        // the initial state: tap j of the token at place p reads its column p + j while that is below W-1;
        // the lane that holds the sequence's first token sums and stores it
        const bool head = a.dh0 && place <= W - 2 && t - place >= it.t0 && t - place < it.t1 && s.has_state(s.q);
        if (head) {
#pragma unroll
            for (int c = 0; c < W - 1; ++c) {
#pragma unroll
                for (int j = 0; j <= c; ++j) {
                    if (place + j != c) continue;
                    // the sequence's first token (place 0) begins every column
#pragma unroll
                    for (int e = 0; e < CW; ++e) dh[c][e] = (place ? dh[c][e] : 0.f) + k.w[j][e] * g[e];
                }
            }
        }
        if (a.dfin && last && s.has_state(s.q)) {
            // column j of the final state is the input of token t - (W-2) + j, if it is in the sequence
            const T* df = (const T*)a.dfin + ((int64_t)s.q * a.channels + it.c0) * (W - 1);
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                if (W - 2 - j > place) continue;
#pragma unroll
                for (int e = 0; e < CW; ++e) {
                    const float v = (float)df[e * (W - 1) + j];
                    if (j == W - 2)
                        here[e] += v;
                    else
                        acc[j + 1][e] += v;
                }
            }
            // a sequence shorter than the state keeps part of its initial state: column place + 1 + j
            if (head) {
#pragma unroll
                for (int c = 1; c < W - 1; ++c)
#pragma unroll
                    for (int j = 0; j < c; ++j) {
                        if (place + 1 + j != c) continue;
#pragma unroll
                        for (int e = 0; e < CW; ++e) dh[c][e] += (float)df[e * (W - 1) + j];
                    }
            }
        }
        if (head && (last || place == W - 2)) {
#pragma unroll
            for (int c = 0; c < W - 1; ++c)
#pragma unroll
                for (int e = 0; e < CW; ++e)
                    ((T*)a.dh0)[((int64_t)s.q * a.channels + it.c0 + e) * (W - 1) + c] = (T)dh[c][e];
        }
    };
    RowStream<T, CW, kConvAheadBackward> xrows(s.row(it.t0), a.xs, end - it.t0), grows(dout, os, end - it.t0);
    T* dx = (T*)a.dx + (row0 + it.t0) * a.channels + it.c0;
    // One token.  INNER: it is one of the run's own with W-1 of them before it, so that nothing here branches by lane
    // (a load or store that may or may not have been made makes the next row's wait one for everything).
    auto token = [&](auto inner, int t) {
        constexpr bool INNER = decltype(inner)::value;
        float here[CW] = {};
        if (INNER || t < end) {
            float cur[CW], pre[CW], g[CW];
            xrows.take(cur);
            grows.take(g);
            s.step_to(t);
            if (VL && !s.has_state(s.q)) {  // padding counts as nothing, whatever it holds
#pragma unroll
                for (int e = 0; e < CW; ++e) {
                    cur[e] = g[e] = 0.f;
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) s.win[j][e] = 0.f;
                }
            }
            s.taps(k, cur, pre);
            if (a.silu) {
#pragma unroll
                for (int e = 0; e < CW; ++e) g[e] *= dsilu_f(pre[e]);
            }
            const int place = s.place;  // of t in its sequence, up to W
            if (INNER || t < it.t1) {
#pragma unroll
                for (int e = 0; e < CW; ++e) {
                    db[e] += g[e];
                    dw[W - 1][e] += g[e] * cur[e];
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) dw[j][e] += g[e] * s.win[j][e];
                }
            }
#pragma unroll
            for (int e = 0; e < CW; ++e) here[e] = k.w[W - 1][e] * g[e];
            // acc[j] belongs to token t - (W-1) + j, which tap j of t reads if it is in t's sequence
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
                if (!VL || W - 1 - j <= place) {
#pragma unroll
                    for (int e = 0; e < CW; ++e) acc[j][e] += k.w[j][e] * g[e];
                }
            s.push(cur);
            if constexpr (ST) states(t, place, g, here);
        }
        if (INNER || t - (W - 1) >= it.t0) {
            store_cw<T, CW>(dx, acc[0]);
            dx += a.channels;
        }
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j)
#pragma unroll
            for (int e = 0; e < CW; ++e) acc[j][e] = acc[j + 1][e];
#pragma unroll
        for (int e = 0; e < CW; ++e) acc[W - 2][e] = here[e];
    };
    int t = it.t0;
    for (; t < it.t0 + W - 1; ++t) token(std::false_type{}, t);
    for (; t < it.t1; ++t) token(std::true_type{}, t);
    for (; t < it.t1 + W - 1; ++t) token(std::false_type{}, t);
}

// The sums of a workgroup's four runs meet in LDS and go to its row of `part` ([W + 1][channels], dw then dbias), summed
// by k_conv_sums in a fixed order.  (A row for every run, 28 MB of them at 2 x 4096 x 5376, cost 78.6 us in all against 74.5.)
template <typename T, int W, int CW, bool VL, bool ST>
__global__ __launch_bounds__(256) void k_causal_conv_backward(CausalConvArgs a) {
    __shared__ float s_part[4][W + 1][CW][64];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    float dw[W][CW] = {}, db[CW] = {};
    ConvItem it;
    const bool mine = conv_item<CW>(a, &it);
    if (mine) conv_backward_run<T, W, CW, VL, ST>(a, it, dw, db);
#pragma unroll
    for (int e = 0; e < CW; ++e) {
#pragma unroll
        for (int j = 0; j < W; ++j) s_part[w][j][e][lane] = dw[j][e];
        s_part[w][W][e][lane] = db[e];
    }
    __syncthreads();
    const uint32_t pblocks = (uint32_t)(a.channels / CW + 63) / 64;
    const int c0 = ((int)(blockIdx.x % pblocks) * 64 + lane) * CW;
    if (c0 >= a.channels) return;
    float* part = a.part + (int64_t)(blockIdx.x / pblocks) * (W + 1) * a.channels + c0;
    for (int j = w; j <= W; j += 4)
#pragma unroll
        for (int e = 0; e < CW; ++e)
            part[(int64_t)j * a.channels + e] = (s_part[0][j][e][lane] + s_part[1][j][e][lane]) + (s_part[2][j][e][lane] + s_part[3][j][e][lane]);
}

// dw [channels][W] and dbias [channels] from the rows of `part`, 64 values a workgroup.
template <int W> __global__ __launch_bounds__(256) void k_conv_sums(const float* part, int nrows, int channels,
                                                                     float* dw, float* db) {
    __shared__ float lds[256];
    const int64_t n = (int64_t)channels * (W + 1), i = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
    const float s = sum_rows<float>(part + i, n, nrows, lds, i < n);
    if (i >= n || threadIdx.x >= 64) return;
    const int c = (int)(i % channels), j = (int)(i / channels);
    if (j < W)
        dw[(int64_t)c * W + j] = s;
    else if (db)
        db[c] = s;
}

// One token: a lane owns a channel, reads the W-1 inputs of its slot, writes the output and moves the
// state on by one input.
template <typename T, int W> __global__ __launch_bounds__(256) void k_causal_conv_step(CausalConvArgs a) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)a.batch * a.channels) return;
    const int c = (int)(i % a.channels), b = (int)(i / a.channels);
    const int slot = a.slots ? a.slots[b] : b;
    T* out = split_ptr<T>(a.out, a.split_a, a.split_b, a.channels, c, b);
    if (slot < 0 || slot >= a.nseq) {
        *out = (T)0.f;
        return;
    }
    T* st = (T*)a.pool + ((int64_t)slot * a.channels + c) * (W - 1);
    const T cur = ((const T*)a.x)[b * a.xs + c];
    float s = a.bias ? a.bias[c] : 0.f;
    T win[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        win[j] = st[j];
        s += a.w[(int64_t)c * W + j] * (float)win[j];
    }
    s += a.w[(int64_t)c * W + W - 1] * (float)cur;
    *out = (T)(a.silu ? silu_f(s) : s);
#pragma unroll
    for (int j = 0; j + 1 < W - 1; ++j) st[j] = win[j + 1];
    st[W - 2] = cur;
}

// Tokens of a run, up to `most`.  Long runs read fewer rows twice; and the workgroups, 2048 of which the chip holds at a
// time, should come in full rounds, for in a round that is partly filled too few loads are on their way.  Both as a
// cost relative to one pass over the rows, fitted to the times (us) of runs of 8, 16, 24, 32, 48 and 64 tokens:
// 2 x 4096 x 5376 forward 35.3 34.0 33.0 35.2 33.1 35.8, backward 75 66 64 65 61 66;
// 8 x 2048 x 5376 forward 73 73 72 72 74 77 (so 32 at most forward), backward 146 131 127 123 123 132;
// 1 x 4096 x 1792 forward 8.1 8.2 9.0 10.1 12.5 14.4, backward 17.3 16.8 18.8 19.0 25.1 28.3.
static int conv_rows(int64_t batch, int64_t seqlen, int64_t pieces, int most) {
    const int64_t pblocks = (pieces + 63) / 64;
    int best = 8;
    double least = 0;
    for (int rows = 8; rows <= most; rows += 4) {
        const int64_t runs = batch * ((seqlen + rows - 1) / rows), rounds = pblocks * ((runs + 3) / 4);
        const double full = (double)rounds / 2048, cost = (1 + 3.0 / rows) * std::cbrt(std::ceil(full) / full);
        if (rows == 8 || cost < least) {
            least = cost;
            best = rows;
        }
    }
    return best;
}
// Channels a lane takes where rows allow it (4: forward 36.7 us against 36.8 with 2 at 2 x 4096 x 5376 and 11.3 against 9.6 at
// 1 x 4096 x 1792, packed; backward 79 against 70 at 2 x 4096 x 5376).
constexpr int kConvWide = 2;
constexpr int kConvMost = 32, kConvBackwardMost = 64;

int conv_backward_rows(int64_t batch, int64_t seqlen, int64_t channels) {
    return conv_rows(batch, seqlen, (channels + kConvWide - 1) / kConvWide, kConvBackwardMost);
}

// Whether lanes can take kConvWide channels with one access: every row they touch starts on a multiple of as many elements.
static bool conv_wide(const CausalConvArgs& a, size_t es, const void* const* tens, int ntens) {
    if (a.channels % kConvWide || a.split_a % kConvWide || a.split_b % kConvWide || a.xs % kConvWide) return false;
    if ((uintptr_t)a.x % (kConvWide * es)) return false;
    for (int i = 0; i < ntens; ++i)
        if ((uintptr_t)tens[i] % (kConvWide * es)) return false;
    return true;
}

static unsigned conv_blocks(const CausalConvArgs& a, int cw) {
    const int64_t pblocks = (a.channels / cw + 63) / 64, runs = (int64_t)a.batch * a.nseg;
    return (unsigned)(pblocks * ((runs + 3) / 4));
}

template <typename T, int W> hipError_t launch_conv_tw(CausalConvArgs& a, hipStream_t st) {
    const bool wide = conv_wide(a, sizeof(T), a.out, 3);
    a.rows = conv_rows(a.batch, a.seqlen, a.channels / (wide ? kConvWide : 1), kConvMost);
    a.nseg = (a.seqlen + a.rows - 1) / a.rows;
    void* args[] = {&a};
    const void* fn = a.seq ? (wide ? (const void*)&k_causal_conv<T, W, kConvWide, true> : (const void*)&k_causal_conv<T, W, 1, true>)
                           : (wide ? (const void*)&k_causal_conv<T, W, kConvWide, false> : (const void*)&k_causal_conv<T, W, 1, false>);
    return hipLaunchKernel(fn, dim3(conv_blocks(a, wide ? kConvWide : 1)), dim3(256), args, 0, st);
}

template <typename T, int W, int CW> const void* conv_backward_kernel(bool packed, bool states) {
    if (packed) return (const void*)&k_causal_conv_backward<T, W, CW, true, true>;
    return states ? (const void*)&k_causal_conv_backward<T, W, CW, false, true>
                  : (const void*)&k_causal_conv_backward<T, W, CW, false, false>;
}

template <typename T, int W> hipError_t launch_conv_back_tw(CausalConvArgs& a, float* dw, float* db, hipStream_t st) {
    a.rows = conv_backward_rows(a.batch, a.seqlen, a.channels);
    a.nseg = (a.seqlen + a.rows - 1) / a.rows;
    const void* tens[4] = {a.dout[0], a.dout[1], a.dout[2], a.dx};
    const bool wide = conv_wide(a, sizeof(T), tens, 4);
    void* args[] = {&a};
    const bool states = a.dh0 || a.dfin;
    const void* fn = wide ? conv_backward_kernel<T, W, kConvWide>(a.seq, states)
                        : conv_backward_kernel<T, W, 1>(a.seq, states);
    hipError_t e = hipLaunchKernel(fn, dim3(conv_blocks(a, wide ? kConvWide : 1)), dim3(256), args, 0, st);
    if (e != hipSuccess) return e;
    int nrows = (int)(((int64_t)a.batch * a.nseg + 3) / 4);
    const int64_t n = (int64_t)a.channels * (W + 1);
    void* sargs[] = {&a.part, &nrows, &a.channels, &dw, &db};
    return hipLaunchKernel((const void*)&k_conv_sums<W>, dim3((unsigned)((n + 63) / 64)), dim3(256), sargs, 0, st);
}

template <typename T, int W> hipError_t launch_conv_step_tw(CausalConvArgs& a, hipStream_t st) {
    const int64_t items = (int64_t)a.batch * a.channels;
    void* args[] = {&a};
    return hipLaunchKernel((const void*)&k_causal_conv_step<T, W>, dim3((unsigned)((items + 255) / 256)), dim3(256),
                           args, 0, st);
}

#define SSD_CONV_BY_TYPE(fn, ...)                                              \
    switch (in_dtype * 8 + a.width) {                                          \
    case DT_F32 * 8 + 2: return fn<float, 2>(__VA_ARGS__);                     \
    case DT_F32 * 8 + 3: return fn<float, 3>(__VA_ARGS__);                     \
    case DT_F32 * 8 + 4: return fn<float, 4>(__VA_ARGS__);                     \
    case DT_F16 * 8 + 2: return fn<_Float16, 2>(__VA_ARGS__);                  \
    case DT_F16 * 8 + 3: return fn<_Float16, 3>(__VA_ARGS__);                  \
    case DT_F16 * 8 + 4: return fn<_Float16, 4>(__VA_ARGS__);                  \
    case DT_BF16 * 8 + 2: return fn<__bf16, 2>(__VA_ARGS__);                   \
    case DT_BF16 * 8 + 3: return fn<__bf16, 3>(__VA_ARGS__);                   \
    case DT_BF16 * 8 + 4: return fn<__bf16, 4>(__VA_ARGS__);                   \
    default: return hipErrorNotSupported;                                      \
    }

hipError_t launch_causal_conv(CausalConvArgs& a, int in_dtype, hipStream_t st) {
    SSD_CONV_BY_TYPE(launch_conv_tw, a, st)
}
hipError_t launch_causal_conv_backward(CausalConvArgs& a, int in_dtype, float* dw, float* db, hipStream_t st) {
    SSD_CONV_BY_TYPE(launch_conv_back_tw, a, dw, db, st)
}
hipError_t launch_causal_conv_step(CausalConvArgs& a, int in_dtype, hipStream_t st) {
    SSD_CONV_BY_TYPE(launch_conv_step_tw, a, st)
}

}  // namespace ssd
