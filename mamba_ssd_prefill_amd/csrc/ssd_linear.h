// ssd_linear.h -- the matrix product out[m][n] = act(sum_k x[m][k] w[n][k] sx[m] sw[n] + bias[n]) + res[m][n] in tiles.
//
// Both operands have the contraction's values one behind the other, so a tile of either is rows of 128 bytes (32 fp32,
// 64 16-bit or 128 8-bit values), and everything up to the matrix instruction is the same for all types.  A
// workgroup brings BM rows of x and BN of w into LDS by steps of 128 bytes, S of them in LDS or on their way
// (direct loads to LDS, 16 bytes a lane; pieces behind a row's end are read past the buffer, as zeros).  Two steps are
// enough where one takes a microsecond; short ones, of small tiles, are loads' latency, and take 6 or 8.
//
// w is the matrix instruction's first operand, so a lane's four accumulators are four consecutive n of one m; the rows
// of w that the 16 lanes of a block take are chosen so that the NB blocks of a wave leave 4 NB consecutive n in a lane,
// which the epilogue reads and writes 16 bytes at a time.
//
// LDS rows are 128 bytes, two to a line of 64 banks; piece c of row r lies at c ^ swz(r), chosen so that the 16
// rows that a read takes at one c fall on 16 different places of a line (no bank conflicts by the counter).
//
// Large products are bound by the matrix instructions and how well they are fed, smaller ones by their number of workgroups
// and a step's latency, single rows by the weights' bytes.  Measured, bf16: 8192 x 8192 x 8192 865 us, 1.27 PFLOP/s (a
// library's product 1.42); 4096 x 4096 x 1024 36 us (library 40), 4096 x 1024 x 4096 34 us (35); one row of 2560 x
// 10576, 54 MB of weights, 10 us.  e4m3 to bf16: 8192 x 8192 x 8192 426 to 444 us, 2.5 PFLOP/s (library 2.8 to 3.0);
// 2048 x 2560 x 10576 61 to 67 us (74).  int8: 69 us there, 8192 x 5120 x 2560 115 us.
// fp32: 2048 x 2048 x 2048 132 us, 130 TFLOP/s (library, at 4096^3, 136).
#pragma once

#include "ssd_device.h"
#include "ssd_layer.h"

#define SSD_LDS_PTR(T, p) ((__attribute__((address_space(3))) T*)(p))

namespace ssd {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// One 16-byte piece of each operand (two for e4m3) multiplied onto a 16 x 16 block.  ISSUES: its
// instructions.
template <int TYPE> struct Mul;
template <> struct Mul<LT_BF16> {
    typedef f32x4 Acc;
    static constexpr int PIECES = 1, ISSUES = 1;
    __device__ static inline void run(const u32x4 (&w)[1], const u32x4 (&x)[1], Acc& c) {
        c = TT<__bf16>::mma(__builtin_bit_cast(bf16x8, w[0]), __builtin_bit_cast(bf16x8, x[0]), c);
    }
};
template <> struct Mul<LT_F16> {
    typedef f32x4 Acc;
    static constexpr int PIECES = 1, ISSUES = 1;
    __device__ static inline void run(const u32x4 (&w)[1], const u32x4 (&x)[1], Acc& c) {
        c = TT<_Float16>::mma(__builtin_bit_cast(f16x8, w[0]), __builtin_bit_cast(f16x8, x[0]), c);
    }
};
template <> struct Mul<LT_F32> {
    typedef f32x4 Acc;
    static constexpr int PIECES = 1, ISSUES = 4;
    // one of a piece's four values
    __device__ static inline void run_one(const u32x4 (&w)[1], const u32x4 (&x)[1], Acc& c, int e) {
        c = TT<float>::mma(__builtin_bit_cast(f32x4, w[0])[e], __builtin_bit_cast(f32x4, x[0])[e], c);
    }
};
template <> struct Mul<LT_I8> {
    typedef i32x4 Acc;
    static constexpr int PIECES = 1, ISSUES = 1;
    __device__ static inline void run(const u32x4 (&w)[1], const u32x4 (&x)[1], Acc& c) {
        c = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w[0]), __builtin_bit_cast(i32x4, x[0]), c, 0, 0, 0);
    }
};
// e4m3 for outputs of 16 bits.  The instruction adds eight products of a lane at a time, each cut to 13 bits below the largest
// one's leading bit (found by single products: 256 * 256 + 15 gives 65544; the other e4m3 instructions do the same).  Of
// 2048 x 2560 x 10576 normal values the sums are off by 1.5e-5 in the 2-norm, where rounding to bf16 takes 1.7e-3 and to fp16
// 2.1e-4; so outputs of 32 bits, which would show it, come by LT_E4M3_F32.
template <> struct Mul<LT_E4M3> {
    typedef f32x4 Acc;
    static constexpr int PIECES = 2, ISSUES = 1;
    __device__ static inline void run(const u32x4 (&w)[2], const u32x4 (&x)[2], Acc& c) {
        const i32x8 a = __builtin_shufflevector(__builtin_bit_cast(i32x4, w[0]), __builtin_bit_cast(i32x4, w[1]), 0, 1, 2, 3, 4, 5, 6, 7);
        const i32x8 b = __builtin_shufflevector(__builtin_bit_cast(i32x4, x[0]), __builtin_bit_cast(i32x4, x[1]), 0, 1, 2, 3, 4, 5, 6, 7);
        // (both scales 2^0: the rows' own come in the epilogue)
        c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0x7f7f7f7f, 0, 0x7f7f7f7f);
    }
};
// e4m3 with sums in fp32: the codes become fp16, which holds them all, on their way to the matrix instruction (6.5e-8 off, as
// fp16 operands are; 2048 x 2560 x 10576 114 us, 65 by the instruction for codes, 64 rows of it 11.7 and 9.0).
template <> struct Mul<LT_E4M3_F32> {
    typedef f32x4 Acc;
    static constexpr int PIECES = 1, ISSUES = 2;
    // eight of a piece's 16 codes
    __device__ static inline f16x8 half_of(const u32x4& p, int h) {
        f16x8 v;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const f16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)p[2 * h + i], 1.f, false);
            const f16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)p[2 * h + i], 1.f, true);
            v[4 * i] = lo[0];
            v[4 * i + 1] = lo[1];
            v[4 * i + 2] = hi[0];
            v[4 * i + 3] = hi[1];
        }
        return v;
    }
};

// ---- epilogue -----------------------------------------------------------------------------------
// gelu(v) = v (1 + erf(v / sqrt(2))) / 2
__device__ inline float gelu_f(float v) { return 0.5f * v * (1.f + erff(v * 0.70710678118654752440f)); }
__device__ inline float gelu_d(float v) {
    return 0.5f * (1.f + erff(v * 0.70710678118654752440f)) + v * __expf(-0.5f * v * v) * 0.39894228040143267794f;
}
__device__ inline float sigm_f(float v) { return __builtin_amdgcn_rcpf(1.f + __expf(-v)); }
__device__ inline float act_f(float v, int act) {
    // (v times a sigmoid of 0: -infinity gives 0 in the limit)
    return act == 1 ? (v == -__builtin_inff() ? 0.f : v * sigm_f(v)) : act == 2 ? (v == -__builtin_inff() ? 0.f : gelu_f(v)) : v;
}
__device__ inline float act_d(float v, int act) {
    if (act == 1) {
        const float s = sigm_f(v), c = 1.f - s;
        return c == 0.f ? 1.f : s == 0.f ? 0.f : s * __builtin_fmaf(v, c, 1.f);
    }
    return act == 2 ? (fabsf(v) > 1e4f ? (v > 0.f ? 1.f : 0.f) : gelu_d(v)) : 1.f;
}

// C consecutive values of one row at element offset `off`, n of them existing; the type is a run-time one.
template <int C, typename T> constexpr int piece_of() { return C % (16 / (int)sizeof(T)) == 0 ? 16 / (int)sizeof(T) : 4; }
template <int C, typename T> __device__ inline void row_load_t(const void* p, int64_t off, int n, float (&v)[C]) {
    constexpr int ONE = piece_of<C, T>();
    typedef T Raw __attribute__((ext_vector_type(ONE), aligned(sizeof(T))));
    const T* q = (const T*)p + off;
#pragma unroll
    for (int i = 0; i < C; i += ONE) {
        if (i + ONE <= n) {
            const Raw r = *(const Raw*)(q + i);
#pragma unroll
            for (int e = 0; e < ONE; ++e) v[i + e] = (float)r[e];
        } else {
#pragma unroll
            for (int e = 0; e < ONE; ++e) v[i + e] = i + e < n ? (float)q[i + e] : 0.f;
        }
    }
}
template <int C, typename T> __device__ inline void row_store_t(void* p, int64_t off, int n, const float (&v)[C]) {
    constexpr int ONE = piece_of<C, T>();
    typedef T Raw __attribute__((ext_vector_type(ONE), aligned(sizeof(T))));
    T* q = (T*)p + off;
#pragma unroll
    for (int i = 0; i < C; i += ONE) {
        if (i + ONE <= n) {
            Raw r;
#pragma unroll
            for (int e = 0; e < ONE; ++e) r[e] = (T)v[i + e];
            *(Raw*)(q + i) = r;
        } else {
#pragma unroll
            for (int e = 0; e < ONE; ++e)
                if (i + e < n) q[i + e] = (T)v[i + e];
        }
    }
}
template <int C> __device__ inline void row_load(const void* p, int dt, int64_t off, int n, float (&v)[C]) {
    if (dt == DT_F32)
        row_load_t<C, float>(p, off, n, v);
    else if (dt == DT_F16)
        row_load_t<C, _Float16>(p, off, n, v);
    else
        row_load_t<C, __bf16>(p, off, n, v);
}
template <int C> __device__ inline void row_store(void* p, int dt, int64_t off, int n, const float (&v)[C]) {
    if (dt == DT_F32)
        row_store_t<C, float>(p, off, n, v);
    else if (dt == DT_F16)
        row_store_t<C, _Float16>(p, off, n, v);
    else
        row_store_t<C, __bf16>(p, off, n, v);
}

// What C consecutive columns from n take besides the product.
template <int C> struct Columns {
    float bias[C], scale[C];
    int n, live;
    __device__ inline Columns(const LinearArgs& a, int n0) : n(n0), live(a.N - n0) {
        if (a.bias) row_load_t<C, float>(a.bias, n, live, bias);
        if (a.sw) row_load_t<C, float>(a.sw, n, live, scale);
    }
    // the outputs of row m from its sums
    __device__ inline void finish(const LinearArgs& a, int m, float (&v)[C]) const {
        if (live <= 0) return;
        const int64_t o = (int64_t)m * a.N + n;
        if (a.sx) {
            const float s = a.sx[m];
#pragma unroll
            for (int e = 0; e < C; ++e) v[e] *= s;
        }
        if (a.sw) {
#pragma unroll
            for (int e = 0; e < C; ++e) v[e] *= scale[e];
        }
        if (a.bias) {
#pragma unroll
            for (int e = 0; e < C; ++e) v[e] += bias[e];
        }
        if (a.pre) row_store<C>(a.pre, a.out_dtype, o, live, v);
        if (a.act) {
#pragma unroll
            for (int e = 0; e < C; ++e) v[e] = act_f(v[e], a.act);
        }
        if (a.res) {
            float r[C];
            row_load<C>(a.res, a.out_dtype, (int64_t)m * a.rs + n, live, r);
#pragma unroll
            for (int e = 0; e < C; ++e) v[e] += r[e];
        }
        row_store<C>(a.out, a.out_dtype, o, live, v);
    }
};

// At most N of this wave's memory accesses on their way (bits 3:0 and 15:14 of the instruction's operand; the other counters
// unwatched).
template <int N> __device__ inline void wait_loads() {
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x0f70);
}

// This wave's reads of LDS are done.
__device__ inline void wait_reads() { __builtin_amdgcn_s_waitcnt(0xc07f); }
// A barrier that waits for nothing else (__syncthreads waits for all loads).
__device__ inline void barrier_only() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// ---- tiles ----------------------------------------------------------------------------------------
constexpr uint32_t kNoPiece = 0x80000000u;  // an offset past every operand's buffer: reads as zeros

// BM x BN outputs a workgroup, WVM x WVN waves, S steps in LDS, W bytes a lane and load: 16, or 4 for rows that start
// anywhere on 4 bytes.
template <int TYPE, int BM, int BN, int WVM, int WVN, int S, int W> struct LinearTile {
    static constexpr int NW = WVM * WVN, THREADS = 64 * NW, MB = BM / WVM / 16, NB = BN / WVN / 16;
    static constexpr int STEP = 128, WIDE = W;  // bytes of a row, of a load
    static constexpr int LPR = STEP / W, RPL = 64 / LPR;  // lanes of a row, rows of a wave's load
    static constexpr int RPI = RPL * NW;                  // rows that one load of every lane brings
    static constexpr int IX = (BM + RPI - 1) / RPI, IW = (BN + RPI - 1) / RPI;  // (the last one by some waves, which others repeat)
    static constexpr int LOADS = IX + IW;  // of a lane for a step
    static constexpr int STAGE = (BM + BN) * STEP, LDS = S * STAGE;
    static_assert((S - 1) * LOADS < 64, "loads on their way are counted in six bits");
    static_assert(BM % (16 * WVM) == 0 && BN % (16 * WVN) == 0 && LDS <= 160 * 1024, "blocks of a wave");
    // the first of the RPL rows that a wave brings with load j of a tile's ROWS
    template <int ROWS> __device__ static inline int load_row(int j, int wave) {
        return (j + 1) * RPI <= ROWS ? j * RPI + wave * RPL : j * RPI + wave % ((ROWS - j * RPI) / RPL) * RPL;
    }
    // where in its row the W bytes are that a lane brings to its place
    __device__ static inline uint32_t bytes_at(int lane, int swz) {
        const int at = lane % LPR * W;
        return (uint32_t)((at >> 4 ^ swz) << 4 | (at & 15));
    }
    __device__ static inline int swz_x(int row) { return (row >> 1) & 7; }
    __device__ static inline int swz_w(int row) { return (row >> 1 & 1) | (row / (4 * NB) & 3) << 1; }
};

// Where a lane's pieces come from and go to: rows behind the last one repeat it.
template <typename G, int BM, int BN> struct Loads {
    __amdgpu_buffer_rsrc_t rx, rw;
    char* lds;
    uint32_t kbytes, ox[G::IX], ow[G::IW], cx[G::IX], cw[G::IW];
    int tx[G::IX], tw[G::IW];  // where a wave's rows go
    __device__ inline Loads(const LinearArgs& a, char* to, int m0, int n0, int wave, int lane) {
        rx = make_rsrc((const char*)a.x + (int64_t)m0 * a.xs, 0x7fffffffu);
        rw = make_rsrc((const char*)a.w + (int64_t)n0 * a.ws, 0x7fffffffu);
        lds = to;
        kbytes = (uint32_t)a.kbytes;
#pragma unroll
        for (int j = 0; j < G::IX; ++j) {
            tx[j] = G::template load_row<BM>(j, wave) * G::STEP;
            const int row = G::template load_row<BM>(j, wave) + lane / G::LPR;
            cx[j] = G::bytes_at(lane, G::swz_x(row));
            ox[j] = (uint32_t)min(row, a.M - 1 - m0) * (uint32_t)a.xs + cx[j];
        }
#pragma unroll
        for (int j = 0; j < G::IW; ++j) {
            tw[j] = (BM + G::template load_row<BN>(j, wave)) * G::STEP;
            const int row = G::template load_row<BN>(j, wave) + lane / G::LPR;
            cw[j] = G::bytes_at(lane, G::swz_w(row));
            ow[j] = (uint32_t)min(row, a.N - 1 - n0) * (uint32_t)a.ws + cw[j];
        }
    }
    __device__ inline void issue(int step, int place) const {
        const uint32_t k = (uint32_t)step * G::STEP, left = kbytes - k;
        char* to = lds + place * G::STAGE;
#pragma unroll
        for (int j = 0; j < G::IX; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, SSD_LDS_PTR(void, to + tx[j]), G::WIDE,
                                                     cx[j] < left ? ox[j] + k : kNoPiece, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < G::IW; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, SSD_LDS_PTR(void, to + tw[j]), G::WIDE,
                                                     cw[j] < left ? ow[j] + k : kNoPiece, 0, 0, 0);
    }
};

// The order of a stretch of instructions: READS reads of LDS spread over the first MULS matrix instructions; the same with
// LOADS loads to LDS before them.  (As written, all of them would be issued before the first matrix instruction, by every
// wave of a SIMD at the same time.)
template <int READS, int MULS> __device__ inline void reads_among() {
    constexpr int PER = MULS / READS > 0 ? MULS / READS : 1;
#pragma unroll
    for (int i = 0; i < READS; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, PER, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, MULS, 0);
}
template <int LOADS, int READS, int MULS> __device__ inline void loads_among() {
    constexpr int PER = MULS / (READS + LOADS) > 0 ? MULS / (READS + LOADS) : 1;
#pragma unroll
    for (int i = 0; i < READS; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, PER, 0);
    }
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, PER, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, MULS, 0);
}

// A half step's fragments of a wave's blocks, or a whole step's where an instruction takes two pieces.
template <typename G, typename M> struct Frags {
    u32x4 x[G::MB][M::PIECES], w[G::NB][M::PIECES];
    __device__ inline void read(const char* px, const char* pw, int xrow, int wrow, int half, int q) {
#pragma unroll
        for (int p = 0; p < M::PIECES; ++p) {
            const int c = (M::PIECES == 2 ? p : half) * 4 + q;
#pragma unroll
            for (int i = 0; i < G::NB; ++i) w[i][p] = *(const u32x4*)(pw + i * 4 * G::STEP + (c ^ G::swz_w(wrow + i * 4)) * 16);
#pragma unroll
            for (int j = 0; j < G::MB; ++j) x[j][p] = *(const u32x4*)(px + j * 16 * G::STEP + (c ^ G::swz_x(xrow + j * 16)) * 16);
        }
    }
    __device__ inline void multiply(typename M::Acc (&acc)[G::NB][G::MB]) const {
        if constexpr (M::ISSUES == 4) {  // (fp32: the four instructions of a block depend on each other)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < G::NB; ++i)
#pragma unroll
                    for (int j = 0; j < G::MB; ++j) M::run_one(w[i], x[j], acc[i][j], e);
        } else if constexpr (M::ISSUES == 2) {  // (codes that become fp16: each once)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f16x8 v[G::MB];
#pragma unroll
                for (int j = 0; j < G::MB; ++j) v[j] = M::half_of(x[j][0], h);
#pragma unroll
                for (int i = 0; i < G::NB; ++i) {
                    const f16x8 u = M::half_of(w[i][0], h);
#pragma unroll
                    for (int j = 0; j < G::MB; ++j) acc[i][j] = TT<_Float16>::mma(u, v[j], acc[i][j]);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < G::NB; ++i)
#pragma unroll
                for (int j = 0; j < G::MB; ++j) M::run(w[i], x[j], acc[i][j]);
        }
    }
};

// One product, or two of like size in one launch (`other`'s workgroups from `count` on).
template <int TYPE, int BM, int BN, int WVM, int WVN, int S, int W>
__global__ __launch_bounds__(64 * WVM * WVN, 2) void k_linear(LinearArgs one, LinearArgs other, uint32_t count) {
    typedef LinearTile<TYPE, BM, BN, WVM, WVN, S, W> G;
    typedef Mul<TYPE> M;
    extern __shared__ __align__(1024) char lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool second = blockIdx.x >= count;
    const LinearArgs& a = second ? other : one;
    const int tm = (a.M + BM - 1) / BM, tn = (a.N + BN - 1) / BN;
    // Neighbouring tiles go to one XCD (workgroups are dealt to eight in turn), in groups of 8 rows of tiles, so that
    // the rows they share come from its L2.
    uint32_t id = second ? blockIdx.x - count : blockIdx.x;
    const uint32_t whole = (second ? gridDim.x - count : count) / 8 * 8;
    if (id < whole) id = (id & 7) * (whole / 8) + id / 8;
    const int split = (int)(id % (uint32_t)a.splits);
    id /= (uint32_t)a.splits;
    const int grp = 8 * tn, g0 = (int)id / grp * 8, gm = min(8, tm - g0);
    const int m0 = (g0 + (int)(id % (uint32_t)grp) % gm) * BM, n0 = (int)(id % (uint32_t)grp) / gm * BN;
    const int steps = (a.kbytes + G::STEP - 1) / G::STEP;
    const int s0 = split * a.steps_per_split, s1 = min(s0 + a.steps_per_split, steps);

    const Loads<G, BM, BN> loads(a, lds, m0, n0, wave, lane);
    typename M::Acc acc[G::NB][G::MB];
#pragma unroll
    for (int i = 0; i < G::NB; ++i)
#pragma unroll
        for (int j = 0; j < G::MB; ++j) acc[i][j] = vzero<typename M::Acc>();
    const int wm = wave % WVM, wn = wave / WVM, l16 = lane & 15, q = lane >> 4;
    // this lane's row of its wave's first block, and the piece it starts with
    const int xrow = wm * G::MB * 16 + l16, wrow = wn * G::NB * 16 + (l16 >> 2) * 4 * G::NB + (l16 & 3);
    const char* const px = lds + xrow * G::STEP;
    const char* const pw = lds + (BM + wrow) * G::STEP;
    if constexpr (M::PIECES == 2 || S == 2) {
        // One set of fragments: e4m3, whose step is one instruction a block, and large tiles in two places, whose waves
        // multiply for long enough to cover another's waits (8192^3 bf16, 256 x 256: 865 us so, 887 with the loop below; 128 x
        // 128 by four waves 1000 and 1020; but 256 x 160 in three places 1093 and 972, 256 x 128 1041 and 932).
#pragma unroll
        for (int i = 0; i < S - 1; ++i)
            if (s0 + i < s1) loads.issue(s0 + i, i);
        for (int step = s0, place = 0; step < s1; ++step) {
            if (S > 2 && step + S - 2 < s1)
                wait_loads<(S - 2) * G::LOADS>();
            else
                wait_loads<0>();
            barrier_only();
            if (step + S - 1 < s1) loads.issue(step + S - 1, place == 0 ? S - 1 : place - 1);
            const char *tx = px + place * G::STAGE, *tw = pw + place * G::STAGE;
#pragma unroll
            for (int h = 0; h < 2 / M::PIECES; ++h) {
                Frags<G, M> f;
                f.read(tx, tw, xrow, wrow, h, q);
                f.multiply(acc);
            }
            wait_reads();  // (the place is written again behind the next barrier)
            place = place == S - 1 ? 0 : place + 1;
        }
    } else {
#pragma unroll
        for (int i = 0; i < S; ++i)
            if (s0 + i < s1) loads.issue(s0 + i, i);
        // Two sets: half a step is read while the one before is multiplied (16 x 5120 x 2560 in tiles of 16 x 64: 13.5 us
        // so, 19.5 with the loop above).
        Frags<G, M> f0, f1;
        int step = s0, place = 0;
        if (s0 + S <= s1) {
            wait_loads<(S - 1) * G::LOADS>();
            barrier_only();
            f0.read(px, pw, xrow, wrow, 0, q);
            for (; step + S < s1; ++step) {
                const int at = place * G::STAGE, next = place == S - 1 ? 0 : place + 1;
                f1.read(px + at, pw + at, xrow, wrow, 1, q);
                f0.multiply(acc);
                reads_among<G::MB + G::NB, G::MB * G::NB * M::ISSUES>();
                // this wave has read all of the step, and its loads of the next one are there (those of the S - 2 behind it may be
                // on their way): behind the barrier the same holds for every wave, and the step's place is free
                wait_reads();
                wait_loads<(S - 2) * G::LOADS>();
                barrier_only();
                loads.issue(step + S, place);
                place = next;
                f0.read(px + place * G::STAGE, pw + place * G::STAGE, xrow, wrow, 0, q);
                f1.multiply(acc);
                loads_among<G::LOADS, G::MB + G::NB, G::MB * G::NB * M::ISSUES>();
                // (fp32: the compiler reuses a block's registers one wait state early across the loop's end)
                if constexpr (M::ISSUES == 4) {
                    __builtin_amdgcn_sched_barrier(0);
                    asm volatile("s_nop 1");
                }
            }
        }
        // the last S steps, or what there is
        wait_loads<0>();
        barrier_only();
        for (; step < s1; ++step) {
            const int at = place * G::STAGE;
            f0.read(px + at, pw + at, xrow, wrow, 0, q);
            f1.read(px + at, pw + at, xrow, wrow, 1, q);
            f0.multiply(acc);
            f1.multiply(acc);
            place = place == S - 1 ? 0 : place + 1;
        }
    }
    constexpr int C = 4 * G::NB;
    const int n = n0 + wn * G::NB * 16 + q * C;
    if (a.splits > 1) {
#pragma unroll
        for (int j = 0; j < G::MB; ++j) {
            const int m = m0 + xrow + j * 16;
            if (m >= a.M || n >= a.N) continue;
            float v[C];
#pragma unroll
            for (int i = 0; i < G::NB; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const auto t = acc[i][j][e];
                    v[i * 4 + e] = __builtin_bit_cast(float, t);
                }
            row_store_t<C, float>(a.part, ((int64_t)split * a.M + m) * a.N + n, a.N - n, v);
        }
        return;
    }
    const Columns<C> cols(a, n);
#pragma unroll
    for (int j = 0; j < G::MB; ++j) {
        const int m = m0 + xrow + j * 16;
        if (m >= a.M) continue;
        float v[C];
#pragma unroll
        for (int i = 0; i < G::NB; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[i * 4 + e] = (float)acc[i][j][e];
        cols.finish(a, m, v);
    }
}

// The sums over the splits of the contraction, and what stands behind the product: four outputs a lane.
template <typename V> __global__ __launch_bounds__(256) void k_linear_join(LinearArgs a) {
    const int per = (a.N + 3) / 4;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int m = (int)(i / per), n = (int)(i % per) * 4;
    if (m >= a.M) return;
    V s[4] = {0, 0, 0, 0};
    const int64_t o = (int64_t)m * a.N + n;
    for (int k = 0; k < a.splits; ++k) {
        float v[4];
        row_load_t<4, float>(a.part, (int64_t)k * a.M * a.N + o, a.N - n, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += __builtin_bit_cast(V, v[e]);
    }
    const Columns<4> cols(a, n);
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)s[e];
    cols.finish(a, m, v);
}

template <int TYPE, int BM, int BN, int WVM, int WVN, int S = 2, int W = 16>
hipError_t launch_tile(LinearArgs& a, LinearArgs* b, hipStream_t st) {
    typedef LinearTile<TYPE, BM, BN, WVM, WVN, S, W> G;
    const auto groups = [](const LinearArgs& l) {
        return (uint32_t)((int64_t)((l.M + BM - 1) / BM) * ((l.N + BN - 1) / BN) * l.splits);
    };
    uint32_t count = groups(a);
    void* args[] = {&a, b ? b : &a, &count};
    const void* fn = (const void*)&k_linear<TYPE, BM, BN, WVM, WVN, S, W>;
    return hipLaunchKernel(fn, dim3(b ? count + groups(*b) : count), dim3(G::THREADS), args, G::LDS, st);
}

constexpr int kNarrowTiles = 16;
// (b: a second product in the same launch, neither being split, or NULL)
template <int TYPE> hipError_t launch_linear_type(LinearArgs& a, LinearArgs* b, const LinearPlan& p, hipStream_t st) {
    hipError_t e;
    // (kTiles in ssd_linear.hip; what each takes of the 160 KB of LDS decides how many share a CU)
    switch (p.narrow ? kNarrowTiles + p.tile : p.tile) {
    case 0: e = launch_tile<TYPE, 128, 128, 2, 2>(a, b, st); break;
    case 1: e = launch_tile<TYPE, 256, 256, 2, 4>(a, b, st); break;
    case 2: e = launch_tile<TYPE, 128, 192, 2, 2>(a, b, st); break;
    case 3: e = launch_tile<TYPE, 256, 160, 4, 2, TYPE == LT_E4M3 ? 2 : 3>(a, b, st); break;
    case 4: e = launch_tile<TYPE, 256, 128, 4, 2, TYPE == LT_E4M3 ? 2 : 3>(a, b, st); break;
    case 5: e = launch_tile<TYPE, 64, 128, 1, 4, 3>(a, b, st); break;
    case 6: e = launch_tile<TYPE, 32, 64, 1, 4, 6>(a, b, st); break;
    case 7: e = launch_tile<TYPE, 16, 64, 1, 4, 8>(a, b, st); break;
    case kNarrowTiles + 5: e = launch_tile<TYPE, 64, 128, 1, 4, 3, 4>(a, b, st); break;
    case kNarrowTiles + 6: e = launch_tile<TYPE, 32, 64, 1, 4, 6, 4>(a, b, st); break;
    case kNarrowTiles + 7: e = launch_tile<TYPE, 16, 64, 1, 4, 7, 4>(a, b, st); break;
    case 8:
        // (fp32 has none: its tiles go by their area, by which 128 x 128 with two workgroups a CU is never behind)
        if constexpr (TYPE != LT_F32) {
            e = launch_tile<TYPE, 128, 128, 4, 2, TYPE == LT_E4M3 ? 2 : 4>(a, b, st);
            break;
        }
        [[fallthrough]];
    default: return hipErrorNotSupported;
    }
    if (e != hipSuccess || a.splits == 1) return e;
    const int64_t lanes = (int64_t)a.M * ((a.N + 3) / 4);
    void* args[] = {&a};
    const void* fn = TYPE == LT_I8 ? (const void*)&k_linear_join<int> : (const void*)&k_linear_join<float>;
    return hipLaunchKernel(fn, dim3((unsigned)((lanes + 255) / 256)), dim3(256), args, 0, st);
}

}  // namespace ssd
