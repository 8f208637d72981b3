// ssd_linear.hip -- what stands around the matrix product: rows that it cannot take as they are copied into ones that it can,
// and dout act'(pre) for its gradients (ssd_linear / _backward in include/mamba_ssd.h).
#include <math.h>

#include "ssd_linear.h"
#include "ssd_sum_rows.h"

namespace ssd {

hipError_t launch_linear_f32(LinearArgs&, LinearArgs*, const LinearPlan&, hipStream_t);
hipError_t launch_linear_f16(LinearArgs&, LinearArgs*, const LinearPlan&, hipStream_t);
hipError_t launch_linear_bf16(LinearArgs&, LinearArgs*, const LinearPlan&, hipStream_t);
hipError_t launch_linear_i8(LinearArgs&, LinearArgs*, const LinearPlan&, hipStream_t);
hipError_t launch_linear_e4m3(LinearArgs&, LinearArgs*, const LinearPlan&, hipStream_t);
hipError_t launch_linear_e4m3_f32(LinearArgs&, LinearArgs*, const LinearPlan&, hipStream_t);

hipError_t launch_linear(LinearArgs& a, LinearArgs* b, int type, const LinearPlan& p, hipStream_t st) {
    for (LinearArgs* l : {&a, b}) {
        if (!l) continue;
        l->splits = p.splits;
        const int steps = (l->kbytes + 127) / 128;
        l->steps_per_split = (steps + p.splits - 1) / p.splits;
    }
    switch (type) {
    case LT_F32: return launch_linear_f32(a, b, p, st);
    case LT_F16: return launch_linear_f16(a, b, p, st);
    case LT_BF16: return launch_linear_bf16(a, b, p, st);
    case LT_I8: return launch_linear_i8(a, b, p, st);
    case LT_E4M3: return a.out_dtype == DT_F32 ? launch_linear_e4m3_f32(a, b, p, st) : launch_linear_e4m3(a, b, p, st);
    default: return hipErrorNotSupported;
    }
}

// ---- rows of another pitch, or transposed --------------------------------------------------------------
// V values of T as loaded (as integers of its size: nothing is computed with them).
template <typename T> struct Piece {
    static constexpr int V = 16 / (int)sizeof(T);
    T v[V];
    // n of them exist at p, the others are 0
    __device__ inline void load(const T* p, int64_t n) {
        typedef T Raw __attribute__((ext_vector_type(V), aligned(sizeof(T))));
        if (n >= V) {
            const Raw r = *(const Raw*)p;
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = r[e];
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = e < n ? p[e] : (T)0;
        }
    }
    __device__ inline void store(T* p) const {  // 16-byte aligned
        typedef T Raw __attribute__((ext_vector_type(V)));
        Raw r;
#pragma unroll
        for (int e = 0; e < V; ++e) r[e] = v[e];
        *(Raw*)p = r;
    }
};

// Both operands' rows in one launch, a piece a lane.  (fp32, 333 and 771 rows of 1110: 7 us, of which a launch takes 3; the
// product after it 18.)
template <typename T> __global__ __launch_bounds__(256) void k_pack_rows(PackArgs a, PackArgs b, uint32_t na) {
    uint32_t i = blockIdx.x * 256 + threadIdx.x;  // (a launch's lanes fit)
    const bool second = i >= na;
    if (second) i -= na;
    const PackArgs& p = second ? b : a;
    const uint32_t per = (uint32_t)(p.kp / Piece<T>::V);
    const int64_t r = i / per, c = i % per * Piece<T>::V;
    if (r >= p.rows) return;
    Piece<T> v;
    v.load((const T*)p.src + r * p.stride + c, p.cols - c);
    v.store((T*)p.dst + r * p.kp + c);
}

// 64 x 64 values on their way to rows of the transposed.
template <typename T> struct Square {
    static constexpr int V = Piece<T>::V, LPR = 64 / V, RPP = 256 / LPR, PASSES = 64 / RPP, PITCH = 64 + 4 / (int)sizeof(T);
    T t[64][PITCH];
    // rows r0.. of the transposed: this lane's pieces of columns c0.. of `rows` rows of kp values
    __device__ inline void store_columns(T* dst, int64_t kp, int64_t c0, int64_t cols, int64_t r0) const {
        const int x = (int)(threadIdx.x % LPR) * V, y = threadIdx.x / LPR;
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            const int64_t c = c0 + y + i * RPP;
            if (c >= cols || r0 + x >= kp) continue;
            Piece<T> p;
#pragma unroll
            for (int e = 0; e < V; ++e) p.v[e] = t[x + e][y + i * RPP];
            p.store(dst + c * kp + r0 + x);
        }
    }
};

hipError_t launch_pack(PackArgs& a, PackArgs& b, int elem_bytes, hipStream_t st) {
    auto lanes = [&](const PackArgs& p) { return p.dst ? p.rows * (p.kp / (16 / elem_bytes)) : 0; };
    uint32_t na = (uint32_t)lanes(a);
    const void* fn = elem_bytes == 4 ? (const void*)&k_pack_rows<uint32_t>
                   : elem_bytes == 2 ? (const void*)&k_pack_rows<uint16_t> : (const void*)&k_pack_rows<uint8_t>;
    void* args[] = {&a, &b, &na};
    return hipLaunchKernel(fn, dim3((unsigned)((na + lanes(b) + 255) / 256)), dim3(256), args, 0, st);
}

// ---- before the gradients' products -----------------------------------------------------------------------
// 64 x 64 values a workgroup, through LDS: dout act'(pre), written as rows and as columns, since the two products take their
// contraction's values one behind the other, with its column sums, from the values before they are rounded; and the
// transposed weight and input.  HBM-bound: dout and pre of 4096 x 4096 f16, a weight and an input of
// 4096 x 1024, 168 MB, 31.6 us, 5.3 TB/s (in two launches 29.4 and 7.8).
// dpre is rounded to the operands' type for the products, which take no wider one (fp16: values below 2^-14 lose bits, as
// those of dout have).  Of 4096 x 1024 x 4096 normal values in fp16 the gradients are 2.9e-4 off in the 2-norm, 2.1e-4 of it by
// their own rounding; in two parts, the rounded value and the rest, they would be 2.1e-4 off, and the products, of
// twice the contraction, take 140 us instead of 76 (one by one).  Without an activation dpre is dout, and nothing is rounded.
template <typename T> struct Dpre {
    static constexpr int V = Square<T>::V;
    Square<T> sq;
    float sums[Square<T>::RPP][64], quarters[256];
    __device__ inline void run(const DpreArgs& a, uint32_t block) {
        typedef Square<T> S;
        const uint32_t cb = (uint32_t)((a.N + 63) / 64);
        const int64_t r0 = (int64_t)(block / cb) * 64, c0 = (int64_t)(block % cb) * 64;
        const int x = (int)(threadIdx.x % S::LPR) * V, y = threadIdx.x / S::LPR;
        const int64_t c = c0 + x;
        float s[V];
#pragma unroll
        for (int e = 0; e < V; ++e) s[e] = 0.f;
#pragma unroll
        for (int k = 0; k < S::PASSES; ++k) {
            const int64_t r = r0 + y + k * S::RPP;
            float v[V];
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = 0.f;
            if (r < a.M && c < a.N) {
                const int n = (int)min(a.N - c, (int64_t)V);
                row_load_t<V, T>(a.dout, r * a.N + c, n, v);
                if (a.act) {
                    float p[V];
                    row_load_t<V, T>(a.pre, r * a.N + c, n, p);
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (e < n) v[e] *= act_d(p[e], a.act);
                }
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                s[e] += v[e];
                if (a.cols) sq.t[y + k * S::RPP][x + e] = (T)v[e];
            }
            // (a padded pitch is the next multiple of a piece)
            if (a.rows && r < a.M && c < a.np) row_store_t<V, T>(a.rows, r * a.np + c, V, v);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) sums[y][x + e] = s[e];
        __syncthreads();
        if (a.cols) sq.store_columns((T*)a.cols, a.mp, c0, a.N, r0);
        if (a.part) {
            const int col = threadIdx.x & 63, part = threadIdx.x >> 6;
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < S::RPP / 4; ++i) t += sums[part * (S::RPP / 4) + i][col];
            quarters[threadIdx.x] = t;
            __syncthreads();
            if (threadIdx.x < 64 && c0 + col < a.N)
                a.part[(r0 / 64) * a.N + c0 + col] = (quarters[col] + quarters[64 + col]) + (quarters[128 + col] + quarters[192 + col]);
        }
    }
    __device__ inline void transpose(const PackArgs& p, uint32_t block) {
        typedef Square<T> S;
        const uint32_t cb = (uint32_t)((p.cols + 63) / 64);
        const int64_t r0 = (int64_t)(block / cb) * 64, c0 = (int64_t)(block % cb) * 64;
        const int x = (int)(threadIdx.x % S::LPR) * V, y = threadIdx.x / S::LPR;
#pragma unroll
        for (int k = 0; k < S::PASSES; ++k) {
            const int64_t r = r0 + y + k * S::RPP, c = c0 + x;
            Piece<T> v{};
            if (r < p.rows && c < p.cols) v.load((const T*)p.src + r * p.stride + c, p.cols - c);
#pragma unroll
            for (int e = 0; e < V; ++e) sq.t[y + k * S::RPP][x + e] = v.v[e];
        }
        __syncthreads();
        sq.store_columns((T*)p.dst, p.kp, c0, p.cols, r0);
    }
};
// The first `nd` workgroups dout act'(pre), then `np` transposing p, the others q.
template <typename T>
__global__ __launch_bounds__(256) void k_linear_before(DpreArgs a, PackArgs p, PackArgs q, uint32_t nd, uint32_t np) {
    __shared__ Dpre<T> d;
    if (blockIdx.x < nd) {
        d.run(a, blockIdx.x);
    } else {
        const uint32_t i = blockIdx.x - nd;
        const bool second = i >= np;
        d.transpose(second ? q : p, second ? i - np : i);
    }
}

__global__ __launch_bounds__(1024) void k_dbias(const float* part, float* db, int parts, int64_t N) {
    __shared__ float lds[1024];
    const int64_t c = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
    const bool live = c < N;
    const float s = sum_many_rows<float>(part + (live ? c : 0), N, parts, lds, live);
    if (live && threadIdx.x < 64) db[c] = s;
}

hipError_t launch_linear_before(DpreArgs& a, PackArgs& p, PackArgs& q, int dtype, float* dbias, hipStream_t st) {
    // (padded columns behind N and padded rows behind M lie in the last blocks of 64)
    auto blocks = [](const PackArgs& t) { return t.dst ? (t.kp + 63) / 64 * ((t.cols + 63) / 64) : 0; };
    uint32_t nd = a.rows || a.cols || a.part ? (uint32_t)(((a.M + 63) / 64) * ((a.N + 63) / 64)) : 0, np = (uint32_t)blocks(p);
    const void* fn = dtype == DT_F32 ? (const void*)&k_linear_before<float>
                   : dtype == DT_F16 ? (const void*)&k_linear_before<_Float16> : (const void*)&k_linear_before<__bf16>;
    void* args[] = {&a, &p, &q, &nd, &np};
    const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)(nd + np + blocks(q))), dim3(256), args, 0, st);
    if (e != hipSuccess || !dbias) return e;
    int parts = (int)((a.M + 63) / 64);
    void* sum_args[] = {&a.part, &dbias, &parts, &a.N};
    return hipLaunchKernel((const void*)&k_dbias, dim3((unsigned)((a.N + 63) / 64)), dim3(1024), sum_args, 0, st);
}

}  // namespace ssd
