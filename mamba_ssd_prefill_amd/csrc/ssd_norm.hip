// ssd_norm.hip -- root-mean-square norm of a residual stream's rows with the addition before it, its output as values or
// in 8 bits, and its gradients (ssd_rms_norm / _backward in include/mamba_ssd.h).
//
//     s = x + residual,  r = 1 / sqrt(mean(s^2) + eps),  y = s r w
//     n = s r,  g = dout w,  ds = r (g - n mean(g n)) + dsum,  dw = sum_rows dout n
//
// Both are HBM-bound streams: a row is read once, stays in registers (fp32) over the sums of the row, and is written
// once: 8192 x 2560 of bf16 onto an fp32 residual, 252 MB, 51 us forward (5.0 TB/s, a large copy's rate), and 336 MB, 70 us
// backward (4.8 TB/s).  A lane takes pieces of 16 bytes (of 16-bit values; 16 of fp32), a row's lanes being one wave, four
// or sixteen by its width.  Rows and pieces need no alignment beyond their elements': wide accesses take any address on this
// chip, and only the last piece of an odd row goes value by value.
#include "ssd_code8.h"
#include "ssd_layer.h"
#include "ssd_sum_rows.h"

namespace ssd {

// VEC values at p of which n exist (the others read as 0 and are not written), 16 bytes an access.
template <typename T, int VEC> __device__ inline void load_piece(const T* p, int n, float (&v)[VEC]) {
    constexpr int ONE = 16 / (int)sizeof(T) < VEC ? 16 / (int)sizeof(T) : VEC;
    typedef T Raw __attribute__((ext_vector_type(ONE), aligned(sizeof(T))));
    if (n >= VEC) {
#pragma unroll
        for (int i = 0; i < VEC; i += ONE) {
            const Raw r = *(const Raw*)(p + i);
#pragma unroll
            for (int e = 0; e < ONE; ++e) v[i + e] = (float)r[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = e < n ? (float)p[e] : 0.f;
    }
}
template <typename T, int VEC> __device__ inline void store_piece(T* p, int n, const float (&v)[VEC]) {
    constexpr int ONE = 16 / (int)sizeof(T) < VEC ? 16 / (int)sizeof(T) : VEC;
    typedef T Raw __attribute__((ext_vector_type(ONE), aligned(sizeof(T))));
    if (n >= VEC) {
#pragma unroll
        for (int i = 0; i < VEC; i += ONE) {
            Raw r;
#pragma unroll
            for (int e = 0; e < ONE; ++e) r[e] = (T)v[i + e];
            *(Raw*)(p + i) = r;
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (e < n) p[e] = (T)v[e];
    }
}
// The same for a type known at run time: in_dtype T, or fp32.
template <typename T, int VEC>
__device__ inline void load_piece_as(const void* p, int64_t off, bool f32, int n, float (&v)[VEC]) {
    if (f32)
        load_piece<float, VEC>((const float*)p + off, n, v);
    else
        load_piece<T, VEC>((const T*)p + off, n, v);
}
template <typename T, int VEC>
__device__ inline void store_piece_as(void* p, int64_t off, bool f32, int n, const float (&v)[VEC]) {
    if (f32)
        store_piece<float, VEC>((float*)p + off, n, v);
    else
        store_piece<T, VEC>((T*)p + off, n, v);
}

__device__ inline float wave_sum(float v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
    return v;
}

// Sums over the W waves of a row, in one order for every lane.  `lds`: W values of its own.
template <int W> __device__ inline float row_sum(float v, float* lds) {
    v = wave_sum(v);
    if constexpr (W > 1) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) lds[wave] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) v += lds[i];
    }
    return v;
}
template <int W> __device__ inline void row_sums(float& v, float& u, float* lds) {
    v = wave_sum(v);
    u = wave_sum(u);
    if constexpr (W > 1) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            lds[wave] = v;
            lds[W + wave] = u;
        }
        __syncthreads();
        v = u = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            v += lds[i];
            u += lds[W + i];
        }
    }
}
// 1 / sqrt(v).  (The instruction takes a subnormal v for 0: rows of tiny values, or of zeros, with a subnormal eps.)
__device__ inline float inverse_root(float v) {
    const bool tiny = v < 0x1p-100f;
    return __builtin_amdgcn_rsqf(tiny ? v * 0x1p60f : v) * (tiny ? 0x1p30f : 1.f);
}

// In 64 bits: the sum of v, and the largest of u (neither negative).
template <int W> __device__ inline void row_sum_max(double& v, double& u, double* lds) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) {
        v += __shfl_xor(v, m, 64);
        u = __builtin_fmax(u, __shfl_xor(u, m, 64));
    }
    if constexpr (W > 1) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            lds[wave] = v;
            lds[W + wave] = u;
        }
        __syncthreads();
        v = u = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            v += lds[i];
            u = __builtin_fmax(u, lds[W + i]);
        }
    }
}

// 1 / v and 1 / sqrt(v) by Newton's steps from the instructions' 23 bits or so, some 2^-45 and 2^-52 off (NaN for 0 and the
// infinities, whose rows have no codes).
__device__ inline double inverse(double v) {
    const double q = __builtin_amdgcn_rcp(v);
    return __builtin_fma(__builtin_fma(-v, q, 1.0), q, q);
}
__device__ inline double inverse_root(double v) {
    double q = __builtin_amdgcn_rsq(v);
#pragma unroll
    for (int i = 0; i < 2; ++i) q = __builtin_fma(__builtin_fma(-v * q, q, 1.0), 0.5 * q, q);
    return q;
}

// The codes of the quotients t scale, right to two steps of 64 bits: cut to 21 bits with the last one set where something was cut
// ("rounded to odd"), a quotient rounds to the code that all of it does, which the conversion instruction does for e4m3,
// ties to even.
template <int VEC> __device__ inline void codes_of(const double (&t)[VEC], double scale, int format, uint8_t (&c)[VEC]) {
    float q[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const uint64_t u = __builtin_bit_cast(uint64_t, t[e] * scale);
        const uint32_t high = (uint32_t)(u >> 32) | min((uint32_t)u, 1u);
        q[e] = (float)__builtin_bit_cast(double, (uint64_t)high << 32);
    }
    if (format == 0) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) c[e] = (uint8_t)code_int8(q[e]);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = fminf(fmaxf(q[e + i], -448.f), 448.f);
            int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
            w = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], w, true);
#pragma unroll
            for (int i = 0; i < 4; ++i) c[e + i] = (uint8_t)((uint32_t)w >> 8 * i);
        }
    }
}

// W waves a row (a workgroup is four rows of one wave, or one row), NP pieces a lane at most.  CODES: behind s everything is in
// 64 bits, since a value next to a border of two codes has to fall on its own side: with y and the scale in 32 bits some ten
// of 2048 x 2560 values took their neighbour's code.  (Such values of bf16 onto bf16 to e4m3, from the caches: 11.9 us, 12.5
// in 32 bits with a second exchange for the largest |y|; 8192 x 2560 onto fp32 48.4 and 45.8, by the 96 registers.)
template <typename T, int W, int NP, bool CODES>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void k_rms_norm(RmsArgs a) {
    constexpr int VEC = 16 / (int)sizeof(T), LANES = 64 * W, ROWS = W == 1 ? 4 : 1;
    __shared__ double lds[4 * W];
    const int lane = W == 1 ? (int)(threadIdx.x & 63) : (int)threadIdx.x;
    const int D = a.width;
    const bool res32 = a.res_dtype == DT_F32;
    int turn = 0;  // (places for the sums are used in turn: a wave may be a row ahead of another's reads, never two)
    for (int64_t row = (int64_t)blockIdx.x * ROWS + (W == 1 ? (int)(threadIdx.x >> 6) : 0); row < a.rows;
         row += (int64_t)gridDim.x * ROWS, ++turn) {
        float v[NP][VEC];
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const int e0 = (lane + LANES * k) * VEC;
            if (e0 < D) load_piece<T, VEC>((const T*)a.x + row * a.xs + e0, D - e0, v[k]);
        }
        if (a.res) {
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const int e0 = (lane + LANES * k) * VEC;
                if (e0 < D) {
                    float r[VEC];
                    load_piece_as<T, VEC>(a.res, row * a.rs + e0, res32, D - e0, r);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) v[k][e] += r[e];
                }
            }
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const int e0 = (lane + LANES * k) * VEC;
                if (e0 < D) store_piece_as<T, VEC>(a.sum, row * D + e0, res32, D - e0, v[k]);
            }
        }
        double* const sums = lds + (turn & 1) * 2 * W;
        if constexpr (!CODES) {
            float ss = 0.f;
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const int e0 = (lane + LANES * k) * VEC;
                if (e0 < D) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) ss = __builtin_fmaf(v[k][e], v[k][e], ss);
                }
            }
            const float r = inverse_root(row_sum<W>(ss, (float*)sums) / (float)D + a.eps);
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const int e0 = (lane + LANES * k) * VEC;
                if (e0 < D) {
                    float w[VEC];
                    load_piece<float, VEC>(a.w + e0, D - e0, w);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) v[k][e] = v[k][e] * r * w[e];
                    store_piece<T, VEC>((T*)a.out + row * D + e0, D - e0, v[k]);
                }
            }
        } else {
            // y = t r, t = s w (exact in 64 bits), so the largest |y| is r times the largest |t|, and both come by one exchange;
            // `odd` is NaN where a weight is none or infinite, as is r where a value of the row is
            double ss = 0, t[NP][VEC], most = 0;
            float odd = 0.f;
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const int e0 = (lane + LANES * k) * VEC;
                if (e0 < D) {
                    float w[VEC];
                    load_piece<float, VEC>(a.w + e0, D - e0, w);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const double d = v[k][e];
                        ss = __builtin_fma(d, d, ss);
                        t[k][e] = d * (double)w[e];
                        most = __builtin_fmax(most, __builtin_fabs(t[k][e]));
                        odd = __builtin_fmaf(w[e], 0.f, odd);
                    }
                }
            }
            if (odd != odd) most = (double)__builtin_inff();
            row_sum_max<W>(ss, most, sums);
            const double r = inverse_root(ss / (double)D + (double)a.eps);
            float s = (float)(most * r * (a.format == 0 ? 1.0 / 127.0 : 1.0 / 448.0));
            const bool out = !(s < __builtin_inff());  // (an infinity or NaN in the row, or a scale past fp32)
            const bool none = out || s < kMinScale;
            if (none) s = out ? __builtin_nanf("") : 0.f;
            const double c0 = r * inverse((double)s);
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const int e0 = (lane + LANES * k) * VEC;
                if (e0 < D) {
                    uint8_t c[VEC];
                    codes_of<VEC>(t[k], c0, a.format, c);
                    if (none) __builtin_memset(c, 0, VEC);
                    uint8_t* p = (uint8_t*)a.out + row * D + e0;
                    if (e0 + VEC <= D) {
                        __builtin_memcpy(p, c, VEC);
                    } else {
#pragma unroll
                        for (int e = 0; e < VEC; ++e)
                            if (e0 + e < D) p[e] = c[e];
                    }
                }
            }
            if (lane == 0) a.scales[row] = s;
        }
    }
}

// Gradients.  A workgroup takes every parts-th row (W = 1: four rows at a time), and its lanes keep the sums over
// these rows of their pieces of dw.
template <typename T, int W, int NP>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void k_rms_norm_backward(RmsArgs a) {
    constexpr int VEC = 16 / (int)sizeof(T), LANES = 64 * W, ROWS = W == 1 ? 4 : 1;
    __shared__ float lds[4 * W];
    __shared__ float meet[W == 1 ? 4 * 64 * NP * VEC : 1];
    const int lane = W == 1 ? (int)(threadIdx.x & 63) : (int)threadIdx.x, sub = W == 1 ? (int)(threadIdx.x >> 6) : 0;
    const int D = a.width;
    const bool res32 = a.res_dtype == DT_F32;
    float dw[NP][VEC];
#pragma unroll
    for (int k = 0; k < NP; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) dw[k][e] = 0.f;
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * ROWS + sub; row < a.rows; row += (int64_t)gridDim.x * ROWS) {
        float s[NP][VEC], g[NP][VEC], ss = 0.f, gs = 0.f;
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const int e0 = (lane + LANES * k) * VEC;
            if (e0 < D) {
                load_piece_as<T, VEC>(a.x, row * a.xs + e0, res32, D - e0, s[k]);
                load_piece<T, VEC>((const T*)a.dout + row * D + e0, D - e0, g[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const int e0 = (lane + LANES * k) * VEC;
            if (e0 < D) {
                float w[VEC];
                load_piece<float, VEC>(a.w + e0, D - e0, w);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    ss = __builtin_fmaf(s[k][e], s[k][e], ss);
                    gs = __builtin_fmaf(g[k][e] * w[e], s[k][e], gs);
                }
            }
        }
        // (two places for the sums, used in turn: a wave may be a row ahead of another's reads, never two)
        row_sums<W>(ss, gs, lds + (turn & 1) * 2 * W);
        ++turn;
        const float r = inverse_root(ss / (float)D + a.eps);
        const float c = gs / (float)D * r * r;  // ds = r (g - s c) + dsum
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const int e0 = (lane + LANES * k) * VEC;
            if (e0 < D) {
                float w[VEC], d[VEC];
                load_piece<float, VEC>(a.w + e0, D - e0, w);
                if (a.dsum) load_piece_as<T, VEC>(a.dsum, row * D + e0, res32, D - e0, d);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    dw[k][e] = __builtin_fmaf(g[k][e], s[k][e] * r, dw[k][e]);
                    const float v = r * __builtin_fmaf(-s[k][e], c, g[k][e] * w[e]);
                    d[e] = a.dsum ? v + d[e] : v;
                }
                if (a.dx) store_piece<T, VEC>((T*)a.dx + row * D + e0, D - e0, d);
                if (a.dres) store_piece_as<T, VEC>(a.dres, row * D + e0, res32, D - e0, d);
            }
        }
    }
    if constexpr (W == 1) {  // the four rows' sums meet in LDS
#pragma unroll
        for (int k = 0; k < NP; ++k)
#pragma unroll
            for (int e = 0; e < VEC; ++e) meet[((sub * NP + k) * VEC + e) * 64 + lane] = dw[k][e];
        __syncthreads();
        if (sub) return;
#pragma unroll
        for (int k = 0; k < NP; ++k)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int i = (k * VEC + e) * 64 + lane;
                dw[k][e] = (meet[i] + meet[NP * VEC * 64 + i]) + (meet[2 * NP * VEC * 64 + i] + meet[3 * NP * VEC * 64 + i]);
            }
    }
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const int e0 = (lane + LANES * k) * VEC;
        if (e0 < D) store_piece<float, VEC>(a.part + (int64_t)blockIdx.x * D + e0, D - e0, dw[k]);
    }
}

// dw from the workgroups' sums: 64 columns a workgroup.  (With 4 waves instead of 16, 1024 x 2560 sums took 14 us.)
__global__ __launch_bounds__(1024) void k_norm_dw(const float* part, float* dw, int parts, int width) {
    __shared__ float lds[1024];
    const int c = blockIdx.x * 64 + (threadIdx.x & 63);
    const bool live = c < width;
    const float s = sum_many_rows<float>(part + (live ? c : 0), width, parts, lds, live);
    if (live && threadIdx.x < 64) dw[c] = s;
}

namespace {
template <typename T, bool CODES> const void* forward_kernel(int pieces, bool few, int& W) {
    if (!few) {
        W = 1;
        if (pieces <= 64) return (const void*)&k_rms_norm<T, 1, 1, CODES>;
        if (pieces <= 128) return (const void*)&k_rms_norm<T, 1, 2, CODES>;
    }
    W = 4;
    if (pieces <= 256) return (const void*)&k_rms_norm<T, 4, 1, CODES>;
    if (pieces <= 512) return (const void*)&k_rms_norm<T, 4, 2, CODES>;
    if (pieces <= 1024) return (const void*)&k_rms_norm<T, 4, 4, CODES>;
    W = 16;
    if constexpr (sizeof(T) == 4)  // (16384 values are 2048 pieces of 16 bits)
        if (pieces > 2048) return (const void*)&k_rms_norm<T, 16, 4, CODES>;
    return (const void*)&k_rms_norm<T, 16, 2, CODES>;
}
template <typename T> const void* backward_kernel(int pieces, int& W) {
    W = 1;
    if (pieces <= 64) return (const void*)&k_rms_norm_backward<T, 1, 1>;
    if (pieces <= 128) return (const void*)&k_rms_norm_backward<T, 1, 2>;
    W = 4;
    if (pieces <= 256) return (const void*)&k_rms_norm_backward<T, 4, 1>;
    if (pieces <= 512) return (const void*)&k_rms_norm_backward<T, 4, 2>;
    if (pieces <= 1024) return (const void*)&k_rms_norm_backward<T, 4, 4>;
    W = 16;
    if constexpr (sizeof(T) == 4)  // (16384 values are 2048 pieces of 16 bits)
        if (pieces > 2048) return (const void*)&k_rms_norm_backward<T, 16, 4>;
    return (const void*)&k_rms_norm_backward<T, 16, 2>;
}
int pieces_of(int width, int in_dtype) {
    const int vec = in_dtype == DT_F32 ? 4 : 8;
    return (width + vec - 1) / vec;
}
template <typename F> hipError_t by_type(int in_dtype, F f) {
    switch (in_dtype) {
    case DT_F32: return f((float*)nullptr);
    case DT_F16: return f((_Float16*)nullptr);
    case DT_BF16: return f((__bf16*)nullptr);
    default: return hipErrorNotSupported;
    }
}
}  // namespace

// Rows of up to 128 pieces by one wave each instead of four: 8192 x 1024 bf16 21.3 us against 22.7, in e4m3 22.9 against 27.6;
// 2048 x 1024 8.0 against 8.1, in e4m3 8.9 against 9.7.  Of fewer rows a wave more is a shorter way for each.  (Wider rows do not
// gain: 8192 x 2560 52.6 by one wave, 50.6 by four, 1024 x 2560 11.7 and 8.6.)
constexpr int64_t kFewRows = 2048;
constexpr int64_t kNormBlocks = 1 << 20;  // more rows are taken in turns

int norm_parts(int64_t rows, int width, int in_dtype) {
    const int64_t groups = pieces_of(width, in_dtype) <= 128 ? (rows + 3) / 4 : rows;
    return (int)(groups < kNormParts ? groups : kNormParts);
}

hipError_t launch_rms_norm(RmsArgs& a, int in_dtype, hipStream_t st) {
    return by_type(in_dtype, [&](auto* t) {
        typedef __remove_pointer(decltype(t)) T;
        int W;
        const void* fn = a.format < 0 ? forward_kernel<T, false>(pieces_of(a.width, in_dtype), a.rows < kFewRows, W)
                                        : forward_kernel<T, true>(pieces_of(a.width, in_dtype), a.rows < kFewRows, W);
        int64_t grid = W == 1 ? (a.rows + 3) / 4 : a.rows;
        if (grid > kNormBlocks) grid = kNormBlocks;
        void* args[] = {&a};
        return hipLaunchKernel(fn, dim3((unsigned)grid), dim3(W == 1 ? 256 : 64 * W), args, 0, st);
    });
}

hipError_t launch_rms_norm_backward(RmsArgs& a, int in_dtype, float* dw, hipStream_t st) {
    const hipError_t e = by_type(in_dtype, [&](auto* t) {
        typedef __remove_pointer(decltype(t)) T;
        int W;
        const void* fn = backward_kernel<T>(pieces_of(a.width, in_dtype), W);
        void* args[] = {&a};
        return hipLaunchKernel(fn, dim3((unsigned)a.parts), dim3(W == 1 ? 256 : 64 * W), args, 0, st);
    });
    if (e != hipSuccess || !dw) return e;
    void* args[] = {&a.part, &dw, &a.parts, &a.width};
    return hipLaunchKernel((const void*)&k_norm_dw, dim3((unsigned)((a.width + 63) / 64)), dim3(1024), args, 0, st);
}

}  // namespace ssd
