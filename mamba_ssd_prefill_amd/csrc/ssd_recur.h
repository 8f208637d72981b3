// ssd_recur.h -- kernels of the gated linear recurrence over prompts and of its gradients (ssd_gated_recurrence / _backward
// in include/mamba_ssd.h).
//
//     r = sigmoid(gate + gate_bias),  i = sigmoid(in_gate + in_bias) (or 1),  a = exp(A r),  beta = sqrt(1 - a^2) (or 1)
//     h = a h + beta i x
//     g = dout + (a g of t+1),  dl = a g h of t-1 - (a^2 / beta) g i x     (l = A r)
//     dx = g beta i,  din_gate = g beta x i (1 - i),  dgate = dl A r (1 - r),  dA = sum dl r
//
// Both passes read each input once and write each output once: 8 and 14 bytes a token and channel of 16 bits.  A workgroup takes
// a tile of 128 bytes of channels and kRecurTile tokens, all tiles of a time before those of the next; a lane holds two
// channels over a run of TOK tokens.  What a run of tokens does to the state is a hop h -> p h + q.  The runs of a wave are
// joined by lane exchanges, the waves through LDS, and the tiles through memory: a tile publishes its hop as soon as it has
// it, finds the state that enters it by looking back over the hops before it, and publishes the state that leaves it, so
// that those behind need not look further.
//
// Rows of 128 bytes are what the memory wants: reading three tensors of 2 x 8192 x 5120 by walking 32-byte columns of them
// reached 2.0 TB/s, 64 bytes 2.4, 128 bytes 3.8 on 160 CUs alone (one workgroup a column, a forward pass of 250 us).
//
// Measured, bf16 with both gates: forward 169 us at 2 x 8192 x 5120 (671 MB: 4.0 TB/s, a large copy reaches 5.1), 92 us at 2 x
// 4096 x 5120, whose backward pass takes 162 us.  The vector ALU issues for some 100 of the 169 us, HBM would need 133: what
// holds the time is a tile's chain of ticket, loads, hop and look-back, which three waves a SIMD do not cover wholly.
#pragma once

#include "ssd_layer.h"
#include "ssd_scan_common.h"

namespace ssd {

// Waves of a workgroup, tokens of a tile, waves that a SIMD is to hold (which bounds the registers; the backward's forms
// for packed rows and odd channels need more of them).  Measured at 2 x 4096 x 5120, bf16: tiles of 64, 128, 256 tokens
// forward 270, 183, 177 us at 2 x 8192; backward with 2 and 3 waves a SIMD 210 and 172 us.
struct RecFwd {
    static constexpr int W = kRecurWaves, TILE = kRecurTile, EU = 3, FAR = 8;
};
struct RecBwd {
    static constexpr int W = kRecurWaves, TILE = kRecurSaved, EU = 3, FAR = 4;
};
// Lanes of a row of 128 bytes, runs of a wave, tokens of a run, by the element size.
template <typename T, typename D> struct RecGeo {
    static constexpr int LN = 64 / (int)sizeof(T), CH = 2 * LN, RUNS = 64 / LN, W = D::W, TILE = D::TILE;
    static constexpr int TOK = TILE / (RUNS * W), THREADS = 64 * W, FAR = sizeof(T) == 4 ? 1 : D::FAR;
    static_assert(RUNS * W * TOK == TILE, "a tile");
    static_assert(kRecurSaved % TOK == 0, "states are kept where a run starts");
};

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
    // keeps the compiler from holding on to what it unpacked before
    __device__ static inline void pin(Held& h) {
        asm volatile("" : "+v"(h.w[0]));
        if constexpr (sizeof(T) == 4) asm volatile("" : "+v"(h.w[1]));
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

// A channel's parameters, scaled for the exponentials: A log2(e), -2 A, and the biases times -log2(e).  A is kept finite, so
// that a closed gate times an infinite A is not NaN.
struct RecParams {
    float A, A2, Am, gb, ib;
};
__device__ inline RecParams rec_params(const RecurArgs& a, int c, bool live) {
    RecParams p{0.f, 0.f, 0.f, 0.f, 0.f};
    if (live) {
        const float A = a.A[c];
        p.A = A < -0x1p100f ? -0x1p100f : A;
        p.A2 = p.A * kLog2e;
        p.Am = -2.f * p.A;
        p.gb = a.gb ? -kLog2e * a.gb[c] : 0.f;
        p.ib = a.ib ? -kLog2e * a.ib[c] : 0.f;
    }
    return p;
}

// sigmoid(v) = 1 / (1 + e), e = exp(-v - bias), and 1 - sigmoid = e / (1 + e), each right relative to itself (a gate closed
// so far that e is infinite is 0, and the other 1).
__device__ inline float gate_of(float v, float bias) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(__builtin_fmaf(v, -kLog2e, bias)));
}
struct Gate {
    float s, c;
};
__device__ inline Gate gates_of(float v, float bias) {
    const float t = __builtin_fmaf(v, -kLog2e, bias), e = __builtin_amdgcn_exp2f(t), s = __builtin_amdgcn_rcpf(1.f + e);
    return Gate{s, t > 126.f ? 1.f : e * s};
}

// sqrt(1 - exp(-z)), z = -2 A r >= 0, a = exp(-z / 2).  Near 0 the difference loses what a was rounded by, so up to
// z = 1/2 it is z times the minimax polynomial of (1 - exp(-z)) / z there (right to 0.12 * 2^-24).
__device__ inline float beta_of(float z, float a) {
    float p = __builtin_fmaf(z, -0.0011216349666938186f, 0.008187386207282543f);
    p = __builtin_fmaf(z, p, -0.041629090905189514f);
    p = __builtin_fmaf(z, p, 0.16666224598884583f);
    p = __builtin_fmaf(z, p, -0.4999998211860657f);
    p = __builtin_fmaf(z, p, 1.f) * z;
    float q = __builtin_fmaf(-a, a, 1.f);
    asm("" : "+v"(p), "+v"(q));  // (both at hand: else a branch for every value, which keeps them from running side by side)
    return __builtin_amdgcn_sqrtf(z < 0.5f ? p : q);
}

// What a run of tokens does to the state before it: h -> p h + q.  PACKED: p = -1 lets nothing through (a sequence starts
// in it), not even a NaN.
struct Hop {
    float p, q;
};
template <bool PACKED> __device__ inline Hop then(Hop f, Hop s) {  // f first
    if (PACKED && s.p < 0.f) return s;
    return Hop{PACKED && f.p < 0.f ? f.p : f.p * s.p, __builtin_fmaf(s.p, f.q, s.q)};
}
template <bool PACKED> __device__ inline float after(Hop s, float h) {
    return PACKED && s.p < 0.f ? s.q : __builtin_fmaf(s.p, h, s.q);
}

__device__ inline uint32_t bits(float v) { return __builtin_bit_cast(uint32_t, v); }
__device__ inline float unbits(uint32_t v) { return __builtin_bit_cast(float, v); }
// The runs of a wave (of LN lanes each) joined in pairs: rows of 16 lanes, then half waves.  At each level every lane gets
// the hop of the pair's first in time (REV: time runs backwards), and `own` becomes that of the whole pair.
template <int LN, bool REV, bool PACKED> struct WaveHops {
    Hop first[2];
    template <int LEVEL> __device__ inline void level(Hop& own) {
        Hop lo, hi;
        if constexpr (LEVEL == 0) {
            const auto p = __builtin_amdgcn_permlane16_swap(bits(own.p), bits(own.p), false, false);
            const auto q = __builtin_amdgcn_permlane16_swap(bits(own.q), bits(own.q), false, false);
            lo = Hop{unbits(p[0]), unbits(q[0])};
            hi = Hop{unbits(p[1]), unbits(q[1])};
        } else {
            const auto p = __builtin_amdgcn_permlane32_swap(bits(own.p), bits(own.p), false, false);
            const auto q = __builtin_amdgcn_permlane32_swap(bits(own.q), bits(own.q), false, false);
            lo = Hop{unbits(p[0]), unbits(q[0])};
            hi = Hop{unbits(p[1]), unbits(q[1])};
        }
        first[LEVEL] = REV ? hi : lo;
        own = then<PACKED>(first[LEVEL], REV ? lo : hi);
    }
    __device__ inline Hop join(Hop own) {
        if constexpr (LN == 16) level<0>(own);
        level<1>(own);
        return own;
    }
    // the state entering this lane's run, from the one entering the wave
    __device__ inline float enter(float h) const {
        const bool late16 = ((threadIdx.x & 16) != 0) != REV, late32 = ((threadIdx.x & 32) != 0) != REV;
        h = late32 ? after<PACKED>(first[1], h) : h;
        if constexpr (LN == 16) h = late16 ? after<PACKED>(first[0], h) : h;
        return h;
    }
};

// (p, q) of two channels a lane.
typedef f32x4 HopPair;

// The runs of a tile: put() leaves the waves' hops in LDS ([W][LN]); behind a barrier fold() gives the tile's, and
// enter() the state entering a run from the one entering the tile.
template <int W, int LN, bool REV, bool PACKED> struct TileHops {
    WaveHops<LN, REV, PACKED> waves[2];
    Hop tile[2], before[2];  // of the whole tile, of the waves before this one
    __device__ inline void put(const Hop (&own)[2], HopPair* lds) {
        const Hop a = waves[0].join(own[0]), b = waves[1].join(own[1]);
        const int lane = threadIdx.x & 63;
        if (lane < LN) lds[(threadIdx.x >> 6) * LN + lane] = HopPair{a.p, a.q, b.p, b.q};
    }
    __device__ inline void fold(const HopPair* lds) {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        tile[0] = tile[1] = before[0] = before[1] = Hop{1.f, 0.f};
#pragma unroll 2
        for (int i = 0; i < W; ++i) {
            const int w = REV ? W - 1 - i : i;
            const HopPair o = lds[w * LN + (threadIdx.x & (LN - 1))];
            if (w == wave) {
                before[0] = tile[0];
                before[1] = tile[1];
            }
            tile[0] = then<PACKED>(tile[0], Hop{o[0], o[1]});
            tile[1] = then<PACKED>(tile[1], Hop{o[2], o[3]});
        }
    }
    __device__ inline float enter(int k, float h) const { return waves[k].enter(after<PACKED>(before[k], h)); }
};

// ---- tiles through memory ---------------------------------------------------------------------------
// A tile's word for a channel: its hop (p, q), or (-1, the state that leaves it), which lets nothing before it through.
// A word is written and read whole, by atomics that the whole device sees, and says by itself whether it is there yet.
constexpr uint64_t kNoHop = ~(uint64_t)0;
// Looks (of a microsecond or so) at a word that is not there before a lane gives up, and its states become NaN.  Workgroups
// take a chain's tiles in the order of their start, so a tile that is waited for is always running and its word microseconds
// away: this ends only waits that a second call running on the same workspace made endless.
constexpr int kMaxLooks = 1 << 16;

__device__ inline float no_nan(float v) { return v != v ? __builtin_nanf("") : v; }  // (all ones would be kNoHop)
__device__ inline void publish(uint64_t* at, Hop h) {
    const uint64_t v = (uint64_t)bits(no_nan(h.p)) << 32 | bits(no_nan(h.q));
    __hip_atomic_store(at, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The state entering tile `tile` (REV: the gradient behind it) for this lane's two channels.  The words of W tiles (fp32:
// twice as many) before it are read at a time, one a wave; if none of them lets nothing through, those of FAR times as many
// are, again until one does.  From there on the hops are applied one by one.  So the result is that of tiles one behind the
// other to the bit, whichever words were there at which time.  (2 x 8192 x 5120 bf16: the near windows alone 174 us, eight times as
// many where they do not do 169, 16 and 32 tiles at every look 177 and 180; training at 2 x 4096 x 5120 262 and 258 us.
// fp32, 1 x 3001 x 1110: 24.5 us, 25.7 with a far window of 32 tiles.)
// c0: the workgroup's first channel; `init`: what enters the first tile.  `lds`: [32 * W * FAR].
template <int W, int LN, bool REV, int FAR> struct LookBack {
    static constexpr int CH = 2 * LN, PER = 64 / CH, WIN = W * PER;
    const uint64_t* base;
    HopPair* lds;
    Hop init;
    int tile, tiles, stride, c, place, looks;
    bool live;
    __device__ inline LookBack(const RecurArgs& a, int b, int tile_, int c0, const void* first, HopPair* lds_)
        : lds(lds_), init{-1.f, 0.f}, tile(tile_), tiles(a.ntiles), stride(a.channels), looks(0) {
        const int lane = threadIdx.x & 63;
        place = (int)(threadIdx.x >> 6) * PER + lane / CH;
        c = c0 + lane % CH;
        live = c < a.channels;
        base = a.hops + (int64_t)b * a.ntiles * a.channels + (live ? c : 0);
        if (live && first) init.q = state_at(first, a.state_dtype, (int64_t)b * a.channels + c);
    }
    // Whether the words of N windows tell it all, and the state if so.
    template <int N> __device__ inline bool look(float (&h)[2]) {
        const int lane = threadIdx.x & 63;
        uint64_t v[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int t = REV ? tile + 1 + place + n * WIN : tile - 1 - place - n * WIN;
            v[n] = 0;
            if (live && t >= 0 && t < tiles)
                v[n] = __hip_atomic_load(base + (int64_t)t * stride, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int t = REV ? tile + 1 + place + n * WIN : tile - 1 - place - n * WIN;
            Hop r = init;
            if (live && t >= 0 && t < tiles) {
                while (v[n] == kNoHop && looks < kMaxLooks) {
                    __builtin_amdgcn_s_sleep(1);
                    v[n] = __hip_atomic_load(base + (int64_t)t * stride, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                    ++looks;
                }
                r = v[n] == kNoHop ? Hop{-1.f, __builtin_nanf("")} : Hop{unbits((uint32_t)(v[n] >> 32)), unbits((uint32_t)v[n])};
            }
            ((f32x2*)lds)[(n * WIN + place) * CH + lane % CH] = f32x2{r.p, r.q};
        }
        __syncthreads();
        bool found[2] = {false, false};
        h[0] = h[1] = 0.f;
#pragma unroll 2
        for (int i = N * WIN - 1; i >= 0; --i) {
            const HopPair o = lds[i * LN + (lane & (LN - 1))];
            found[0] = found[0] || o[0] < 0.f;
            found[1] = found[1] || o[2] < 0.f;
            h[0] = after<true>(Hop{o[0], o[1]}, h[0]);
            h[1] = after<true>(Hop{o[2], o[3]}, h[1]);
        }
        return __all(found[0] && found[1]);  // (the same in every wave)
    }
    __device__ inline void run(float (&h)[2]) {
        if (look<1>(h)) return;
        for (int round = 0; round < kMaxLooks; ++round) {
            __syncthreads();
            if (look<FAR>(h)) return;
        }
        h[0] = h[1] = __builtin_nanf("");
    }
};

// A workgroup's tile.  The workgroups are dealt to the chains (a block of channels of a batch row) in turn, and a chain's
// take its tiles in the order that they start (REV: from the last), by a counter a chain.  (Neighbouring chains
// go to one XCD, workgroups being dealt to eight in turn: 195 -> 184 us.)  So the tile before one that
// is being worked on is done or being worked on too, whatever the order of a launch's workgroups.  (One counter for all of
// them was the bottleneck: 10240 workgroups took 183 us.)
struct RecPlace {
    int b, tile, block0, c0, tok;  // first channel of the workgroup, of this lane; first token of its run in the tile
    bool live[2];
    int64_t row0;
};
template <typename G, bool REV> __device__ inline RecPlace rec_place(const RecurArgs& a) {
    __shared__ uint32_t mine;
    const uint32_t nblk = ((uint32_t)a.channels + G::CH - 1) / G::CH, chains = nblk * (uint32_t)a.batch;
    const uint32_t turn = blockIdx.x % chains, whole = chains / 8 * 8;
    const uint32_t chain = turn < whole ? (turn & 7) * (whole / 8) + turn / 8 : turn;
    RecPlace p;
    p.tile = 0;
    if (a.ntiles > 1) {
        if (threadIdx.x == 0)
            mine = __hip_atomic_fetch_add(a.tickets + (size_t)chain * kTicketWords, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        p.tile = __builtin_amdgcn_readfirstlane((int)mine);
        p.tile = min(max(p.tile, 0), a.ntiles - 1);  // (never, but for a second call on the same workspace)
        if (REV) p.tile = a.ntiles - 1 - p.tile;
    }
    p.block0 = (int)(chain % nblk) * G::CH;
    p.b = (int)(chain / nblk);
    const int lane = threadIdx.x & 63;
    p.c0 = p.block0 + (lane & (G::LN - 1)) * 2;
    p.live[0] = p.c0 < a.channels;
    p.live[1] = p.c0 + 1 < a.channels;
    p.tok = ((int)(threadIdx.x >> 6) * G::RUNS + lane / G::LN) * G::TOK;
    p.row0 = (int64_t)p.b * a.seqlen;
    return p;
}

// A lane's inputs of a tile, as loaded.  seq: the sequence numbers of its tokens, and of the ones before and behind.
template <typename T, bool PAIRED, bool PACKED, typename G, typename F> struct RecTile {
    static constexpr int TOK = G::TOK;
    typedef RecRows<T, PAIRED> Rows;
    typename Rows::Held x[TOK], g[TOK], i[F::ig ? TOK : 1];
    int32_t seq[PACKED ? TOK + 2 : 1];
    __device__ inline void load(const RecurArgs& a, const RecPlace& p, const uint32_t (&ch)[2], int t0) {
        const int n = min(a.seqlen - t0, G::TILE);
        const Rows rx(a.x, a.xs, p.row0 + t0, n), rg(a.gate, a.gs, p.row0 + t0, n);
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
            x[j] = rx.load(p.tok + j, ch);
            g[j] = rg.load(p.tok + j, ch);
        }
        if constexpr (F::ig) {
            const Rows ri(a.ig, a.is, p.row0 + t0, n);
#pragma unroll
            for (int j = 0; j < TOK; ++j) i[j] = ri.load(p.tok + j, ch);
        }
        if constexpr (PACKED) {
#pragma unroll
            for (int j = 0; j < TOK + 2; ++j) {
                const int t = min(max(t0 + p.tok + j - 1, 0), a.seqlen - 1);
                seq[j] = a.seq[p.row0 + t];
            }
        }
    }
};

// Of a lane's tokens from t: which start a sequence, end one, and are padding (those behind the row's end are neither
// start nor end).
struct RecSeq {
    uint32_t start, end, pad;
};
template <int TOK> __device__ inline RecSeq rec_seq(const RecurArgs& a, const int32_t (&q)[TOK + 2], int t) {
    RecSeq s{0, 0, 0};
#pragma unroll
    for (int j = 0; j < TOK; ++j) {
        if (t + j < a.seqlen) {
            if (t + j == 0 || q[j] != q[j + 1]) s.start |= 1u << j;
            if (t + j == a.seqlen - 1 || q[j + 2] != q[j + 1]) s.end |= 1u << j;
            if (q[j + 1] < 0 || q[j + 1] >= a.nseq) s.pad |= 1u << j;
        }
    }
    return s;
}
// The state (or its gradient) of sequence q for this lane's channel k, 0 where there is none.
__device__ inline float seq_state(const RecurArgs& a, const RecPlace& p, const void* states, int32_t q, bool pad, int k) {
    return pad || !states || !p.live[k] ? 0.f : state_at(states, a.state_dtype, (int64_t)q * a.channels + p.c0 + k);
}

// What a call has besides x and gate, as compile-time flags: a branch for every value keeps the values' chains of dependent
// instructions from running side by side.
template <bool IG, bool NORM> struct RecForm {
    static constexpr bool ig = IG, norm = NORM;
};

// Decay and addition of a token.
struct RecStep {
    float a, u;
};

template <typename T, bool PAIRED, bool PACKED, typename F>
__global__ __launch_bounds__(64 * RecFwd::W, RecFwd::EU) void k_recur(RecurArgs a) {
    typedef RecGeo<T, RecFwd> G;
    constexpr int TOK = G::TOK, LN = G::LN, W = G::W;
    typedef RecTile<T, PAIRED, PACKED, G, F> Tile;
    typedef typename Tile::Rows Rows;
    __shared__ HopPair waves[W * LN];
    __shared__ HopPair looked[W * 32 * G::FAR];
    const RecPlace p = rec_place<G, false>(a);
    const int t0 = p.tile * G::TILE;
    uint32_t ch[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) ch[k] = p.live[k] ? (uint32_t)(p.c0 + k) * (uint32_t)sizeof(T) : kNoLane;
    Tile now;
    now.load(a, p, ch, t0);
    RecParams prm[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) prm[k] = rec_params(a, p.c0 + k, p.live[k]);
    RecSeq sq{0, 0, 0};
    if constexpr (PACKED) sq = rec_seq<TOK>(a, now.seq, t0 + p.tok);
    RecStep st[TOK][2];
#pragma unroll
    for (int j = 0; j < TOK; ++j) {
        const Two x = Rows::values(now.x[j]), g = Rows::values(now.g[j]);
        Two i{};
        if constexpr (F::ig) i = Rows::values(now.i[j]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float r = gate_of(g.c[k], prm[k].gb), d = __builtin_amdgcn_exp2f(prm[k].A2 * r);
            float u = x.c[k];
            if constexpr (F::ig) u *= gate_of(i.c[k], prm[k].ib);
            if constexpr (F::norm) u *= beta_of(prm[k].Am * r, d);
            st[j][k] = RecStep{d, u};
        }
    }
    if (t0 + G::TILE > a.seqlen) {  // tokens behind the row's end leave the state as it is
#pragma unroll
        for (int j = 0; j < TOK; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (t0 + p.tok + j >= a.seqlen) st[j][k] = RecStep{1.f, 0.f};
    }
    if constexpr (PACKED) {
        if (sq.start) {
#pragma unroll
            for (int j = 0; j < TOK; ++j)
                if (sq.start >> j & 1) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float h0 = seq_state(a, p, a.h0, now.seq[j + 1], sq.pad >> j & 1, k);
                        st[j][k] = RecStep{-1.f, __builtin_fmaf(st[j][k].a, h0, st[j][k].u)};
                    }
                }
        }
    }
    Hop own[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        own[k] = Hop{st[0][k].a, st[0][k].u};
#pragma unroll
        for (int j = 1; j < TOK; ++j) own[k] = then<PACKED>(own[k], Hop{st[j][k].a, st[j][k].u});
    }
    TileHops<W, LN, false, PACKED> hops;
    hops.put(own, waves);
    __syncthreads();
    hops.fold(waves);
    const bool writer = threadIdx.x < LN;
    uint64_t* const word = a.hops + ((int64_t)p.b * a.ntiles + p.tile) * a.channels + p.c0;
    if (writer && p.tile > 0 && p.tile + 1 < a.ntiles) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (p.live[k]) publish(word + k, hops.tile[k]);
    }
    float h[2];
    if (p.tile > 0) {
        LookBack<W, LN, false, G::FAR>(a, p.b, p.tile, p.block0, PACKED ? nullptr : a.h0, looked).run(h);
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            h[k] = !PACKED && a.h0 && p.live[k] ? state_at(a.h0, a.state_dtype, (int64_t)p.b * a.channels + p.c0 + k) : 0.f;
    }
    if (writer) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (!p.live[k]) continue;
            const float end = after<PACKED>(hops.tile[k], h[k]);
            if (p.tile + 1 < a.ntiles) publish(word + k, Hop{-1.f, end});
            if (!PACKED && a.fin && p.tile + 1 == a.ntiles)
                state_to(a.fin, a.state_dtype, (int64_t)p.b * a.channels + p.c0 + k, end);
        }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) h[k] = hops.enter(k, h[k]);
    if (a.saved && p.tok % kRecurSaved == 0 && t0 + p.tok < a.seqlen) {
        const int64_t at = ((int64_t)p.b * recur_kept(a.seqlen) + (t0 + p.tok) / kRecurSaved) * a.channels + p.c0;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (p.live[k]) a.saved[at + k] = h[k];
    }
    const Rows ro(a.out, a.channels, p.row0 + t0, min(a.seqlen - t0, G::TILE));
#pragma unroll
    for (int j = 0; j < TOK; ++j) {
#pragma unroll
        for (int k = 0; k < 2; ++k) h[k] = after<PACKED>(Hop{st[j][k].a, st[j][k].u}, h[k]);
        ro.store(p.tok + j, ch, h[0], h[1]);
        if constexpr (PACKED) {
            if (a.fin && (sq.end & ~sq.pad) >> j & 1) {
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (p.live[k]) state_to(a.fin, a.state_dtype, (int64_t)now.seq[j + 1] * a.channels + p.c0 + k, h[k]);
            }
        }
    }
}

// Gradients.  The state entering the tile is the one that the forward pass kept; the gradient behind it comes by looking
// back over the tiles after it.
template <typename T, bool PAIRED, bool PACKED, typename F>
__global__ __launch_bounds__(64 * RecBwd::W, PAIRED && !PACKED ? RecBwd::EU : 2) void k_recur_backward(RecurArgs a) {
    typedef RecGeo<T, RecBwd> G;
    constexpr int TOK = G::TOK, LN = G::LN, W = G::W;
    typedef RecTile<T, PAIRED, PACKED, G, F> Tile;
    typedef typename Tile::Rows Rows;
    __shared__ HopPair waves[2][W * LN];
    __shared__ HopPair looked[W * 32 * G::FAR];
    __shared__ f32x4 parked[TOK][64 * W];  // r and A (1 - r) of a lane's tokens, which are not needed before the gradients
    const RecPlace p = rec_place<G, true>(a);
    const int t0 = p.tile * G::TILE, n = min(a.seqlen - t0, G::TILE);
    uint32_t ch[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) ch[k] = p.live[k] ? (uint32_t)(p.c0 + k) * (uint32_t)sizeof(T) : kNoLane;
    Tile now;
    typename Rows::Held dout[TOK];
    now.load(a, p, ch, t0);
    const Rows rd(a.dout, a.channels, p.row0 + t0, n);
#pragma unroll
    for (int j = 0; j < TOK; ++j) dout[j] = rd.load(p.tok + j, ch);
    float start[2] = {0.f, 0.f};
    RecParams prm[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (p.live[k]) start[k] = a.saved[((int64_t)p.b * a.ntiles + p.tile) * a.channels + p.c0 + k];
        prm[k] = rec_params(a, p.c0 + k, p.live[k]);
    }
    RecSeq sq{0, 0, 0};
    if constexpr (PACKED) sq = rec_seq<TOK>(a, now.seq, t0 + p.tok);
    // of each token: the decay, r and A (1 - r), beta i and 1 - i, and the part of the decay's gradient that goes by
    // beta: dl = a g (h - a i x / beta), h the state before it
    float d[TOK][2], bi[TOK][2], ic[TOK][2], w[TOK][2];
#pragma unroll
    for (int j = 0; j < TOK; ++j) {
        const Two x = Rows::values(now.x[j]), g = Rows::values(now.g[j]);
        Two iv{};
        if constexpr (F::ig) iv = Rows::values(now.i[j]);
        f32x4 park;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const Gate r = gates_of(g.c[k], prm[k].gb);
            park[k] = r.s;
            park[2 + k] = prm[k].A * r.c;
            d[j][k] = __builtin_amdgcn_exp2f(prm[k].A2 * r.s);
            float xi = x.c[k];
            bi[j][k] = 1.f;
            if constexpr (F::ig) {
                const Gate i = gates_of(iv.c[k], prm[k].ib);
                bi[j][k] = i.s;
                ic[j][k] = i.c;
                xi *= i.s;
            }
            if constexpr (F::norm) {
                const float be = beta_of(prm[k].Am * r.s, d[j][k]);
                bi[j][k] *= be;
                // (beta = 0, a closed gate: the product with r (1 - r) goes to 0)
                w[j][k] = be != 0.f ? d[j][k] * xi * __builtin_amdgcn_rcpf(be) : 0.f;
            }
        }
        parked[j][threadIdx.x] = park;
    }
    // Tokens that count as nothing, so that no mask is needed behind this: those behind the row's end pass on what they get,
    // and padding (whatever it holds) nothing.
    if (t0 + G::TILE > a.seqlen || (PACKED && sq.pad)) {
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
            const bool out = t0 + p.tok + j >= a.seqlen, pad = PACKED && (sq.pad >> j & 1);
            if (out || pad) {
                now.x[j] = dout[j] = typename Rows::Held{};
                parked[j][threadIdx.x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    d[j][k] = out ? 1.f : 0.f;
                    bi[j][k] = w[j][k] = ic[j][k] = 0.f;
                }
            }
        }
    }
    // (x and dout stay packed between their uses: unpacked ones of all tokens cost 32 registers)
#pragma unroll
    for (int j = 0; j < TOK; ++j) Rows::pin(now.x[j]);
    // The hops of the states (tokens behind the row's end come after all others here), and of the gradients: what each
    // token passes on of the gradient v behind it, v -> a (dout + v).
    Hop own[2], back[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
            Hop s{d[j][k], Rows::values(now.x[j]).c[k] * bi[j][k]};
            if constexpr (PACKED) {
                if (sq.start >> j & 1)
                    s = Hop{-1.f, __builtin_fmaf(s.p, seq_state(a, p, a.h0, now.seq[j + 1], sq.pad >> j & 1, k), s.q)};
                if (sq.pad >> j & 1) s = Hop{-1.f, 0.f};  // (the forward pass may have carried a NaN here)
            }
            own[k] = j ? then<PACKED>(own[k], s) : s;
        }
#pragma unroll
        for (int j = TOK - 1; j >= 0; --j) {
            const float o = Rows::values(dout[j]).c[k];
            Hop s{d[j][k], d[j][k] * o};
            if constexpr (PACKED) {
                const bool pad = sq.pad >> j & 1;
                // behind a sequence's end: the gradient of its final state
                if (sq.end >> j & 1) s = Hop{-1.f, d[j][k] * (o + seq_state(a, p, a.dfin, now.seq[j + 1], pad, k))};
                if (sq.start >> j & 1 || pad) s = Hop{-1.f, 0.f};
            }
            back[k] = j == TOK - 1 ? s : then<PACKED>(back[k], s);
        }
    }
    TileHops<W, LN, false, PACKED> fwd;
    TileHops<W, LN, true, PACKED> rev;
    fwd.put(own, waves[0]);
    rev.put(back, waves[1]);
    __syncthreads();
    rev.fold(waves[1]);
    const bool writer = threadIdx.x < LN;
    uint64_t* const word = a.hops + ((int64_t)p.b * a.ntiles + p.tile) * a.channels + p.c0;
    if (writer && p.tile > 0 && p.tile + 1 < a.ntiles) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (p.live[k]) publish(word + k, rev.tile[k]);
    }
    fwd.fold(waves[0]);
#pragma unroll
    for (int j = 0; j < TOK; ++j) Rows::pin(now.x[j]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float h = fwd.enter(k, start[k]);
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
            if constexpr (PACKED) {
                if (sq.start >> j & 1) h = seq_state(a, p, a.h0, now.seq[j + 1], sq.pad >> j & 1, k);
                if (sq.pad >> j & 1) h = 0.f;
            }
            w[j][k] = F::norm ? h - w[j][k] : h;
            h = __builtin_fmaf(d[j][k], h, Rows::values(now.x[j]).c[k] * bi[j][k]);
        }
    }
    float v[2];
    if (p.tile + 1 < a.ntiles) {
        LookBack<W, LN, true, G::FAR>(a, p.b, p.tile, p.block0, PACKED ? nullptr : a.dfin, looked).run(v);
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            v[k] = !PACKED && a.dfin && p.live[k] ? state_at(a.dfin, a.state_dtype, (int64_t)p.b * a.channels + p.c0 + k) : 0.f;
    }
    if (writer) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (!p.live[k]) continue;
            const float end = after<PACKED>(rev.tile[k], v[k]);
            if (p.tile > 0) publish(word + k, Hop{-1.f, end});
            if (!PACKED && a.dh0 && p.tile == 0) state_to(a.dh0, a.state_dtype, (int64_t)p.b * a.channels + p.c0 + k, end);
        }
    }
    float sum[3][2] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};  // dA, dgate_bias, din_bias
#pragma unroll
    for (int j = 0; j < TOK; ++j) {
        Rows::pin(now.x[j]);
        Rows::pin(dout[j]);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) v[k] = rev.enter(k, v[k]);
    const Rows rx(a.dx, a.channels, p.row0 + t0, n), rg(a.dgate, a.channels, p.row0 + t0, n);
    const Rows ri(F::ig ? a.dig : a.dgate, a.channels, p.row0 + t0, F::ig ? n : 0);
#pragma unroll
    for (int j = TOK - 1; j >= 0; --j) {
        const Two x = Rows::values(now.x[j]), o = Rows::values(dout[j]);
        const f32x4 park = parked[j][threadIdx.x];
        float dx[2], dg[2], di[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const bool pad = PACKED && (sq.pad >> j & 1);
            if constexpr (PACKED) {
                if (sq.end >> j & 1) v[k] = seq_state(a, p, a.dfin, now.seq[j + 1], pad, k);
            }
            const float g = o.c[k] + v[k], ag = d[j][k] * g;
            const float dA = ag * w[j][k] * park[k];
            dx[k] = g * bi[j][k];
            dg[k] = dA * park[2 + k];
            di[k] = 0.f;
            if constexpr (F::ig) di[k] = dx[k] * x.c[k] * ic[j][k];
            sum[0][k] += dA;
            sum[1][k] += dg[k];
            if constexpr (F::ig) sum[2][k] += di[k];
            v[k] = ag;
            if constexpr (PACKED) {
                if (sq.start >> j & 1 && a.dh0 && !pad && p.live[k])
                    state_to(a.dh0, a.state_dtype, (int64_t)now.seq[j + 1] * a.channels + p.c0 + k, ag);
                if (pad) v[k] = 0.f;
            }
        }
        rx.store(p.tok + j, ch, dx[0], dx[1]);
        rg.store(p.tok + j, ch, dg[0], dg[1]);
        if constexpr (F::ig) ri.store(p.tok + j, ch, di[0], di[1]);
    }
    // the sums over the tile's tokens: over a wave's runs, then over waves
    __shared__ float sums[3][2][W * LN];
#pragma unroll
    for (int e = 0; e < 3; ++e)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float s = sum[e][k];
#pragma unroll
            for (int m = LN; m < 64; m *= 2) s += __shfl_xor(s, m, 64);
            if ((threadIdx.x & 63) < LN) sums[e][k][(threadIdx.x >> 6) * LN + (threadIdx.x & 63)] = s;
        }
    __syncthreads();
    if (writer) {
        const int64_t part = (int64_t)p.b * a.ntiles + p.tile;
#pragma unroll
        for (int e = 0; e < 3; ++e)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < W; ++w) s += sums[e][k][w * LN + threadIdx.x];
                if (p.live[k]) a.part[(part * 3 + e) * a.channels + p.c0 + k] = s;
            }
    }
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
template <typename T, bool PAIRED, bool PACKED, typename F> const void* rec_kernel_f(bool backward) {
    return backward ? (const void*)&k_recur_backward<T, PAIRED, PACKED, F> : (const void*)&k_recur<T, PAIRED, PACKED, F>;
}
template <typename T, bool PAIRED, bool PACKED> const void* rec_kernel_p(const RecurArgs& a, bool backward) {
    if (a.ig)
        return a.normalize ? rec_kernel_f<T, PAIRED, PACKED, RecForm<true, true>>(backward)
                           : rec_kernel_f<T, PAIRED, PACKED, RecForm<true, false>>(backward);
    return a.normalize ? rec_kernel_f<T, PAIRED, PACKED, RecForm<false, true>>(backward)
                       : rec_kernel_f<T, PAIRED, PACKED, RecForm<false, false>>(backward);
}
template <typename T> const void* rec_kernel(const RecurArgs& a, bool backward) {
    if (paired<T>(a)) return a.seq ? rec_kernel_p<T, true, true>(a, backward) : rec_kernel_p<T, true, false>(a, backward);
    return a.seq ? rec_kernel_p<T, false, true>(a, backward) : rec_kernel_p<T, false, false>(a, backward);
}

}  // namespace ssd
