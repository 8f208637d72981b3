// ssd_linear.hip -- what stands around the matrix product: the choice of tiles, rows that it cannot take as they are
// copied into ones that it can, and dout act'(pre) for its gradients (ssd_linear / _backward in include/mamba_ssd.h).
#include "ssd_linear.h"
#include "ssd_sum_rows.h"

namespace ssd {

hipError_t launch_linear_f32(LinearArgs&, const LinearPlan&, hipStream_t);
hipError_t launch_linear_f16(LinearArgs&, const LinearPlan&, hipStream_t);
hipError_t launch_linear_bf16(LinearArgs&, const LinearPlan&, hipStream_t);
hipError_t launch_linear_i8(LinearArgs&, const LinearPlan&, hipStream_t);
hipError_t launch_linear_e4m3(LinearArgs&, const LinearPlan&, hipStream_t);

LinearPlan linear_plan(int64_t M, int64_t N, int64_t kbytes, int type) {
    const int64_t tiles = ((M + 127) / 128) * ((N + 127) / 128), steps = (kbytes + 127) / 128;
    int64_t s = tiles >= 256 ? 1 : 512 / tiles;
    if (s > steps / 4) s = steps / 4;
    if (s > 32) s = 32;
    if (s < 1) s = 1;
    const int64_t per = (steps + s - 1) / s;
    return LinearPlan{0, (int)((steps + per - 1) / per)};  // none without a step
}

hipError_t launch_linear(LinearArgs& a, int type, const LinearPlan& p, hipStream_t st) {
    a.splits = p.splits;
    const int steps = (a.kbytes + 127) / 128;
    a.steps_per_split = (steps + p.splits - 1) / p.splits;
    switch (type) {
    case LT_F32: return launch_linear_f32(a, p, st);
    case LT_F16: return launch_linear_f16(a, p, st);
    case LT_BF16: return launch_linear_bf16(a, p, st);
    case LT_I8: return launch_linear_i8(a, p, st);
    case LT_E4M3: return launch_linear_e4m3(a, p, st);
    default: return hipErrorNotSupported;
    }
}

// ---- rows of another pitch, or transposed --------------------------------------------------------------
// 64 x 64 values a workgroup.
template <typename T, bool TRANSPOSED> __global__ __launch_bounds__(256) void k_pack(PackArgs a) {
    __shared__ T tile[TRANSPOSED ? 64 : 1][TRANSPOSED ? 64 + 4 / (int)sizeof(T) : 1];
    const int64_t cb = TRANSPOSED ? (a.cols + 63) / 64 : (a.kp + 63) / 64;
    const int64_t r0 = (int64_t)(blockIdx.x / (uint32_t)cb) * 64, c0 = (int64_t)(blockIdx.x % (uint32_t)cb) * 64;
    const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
    if constexpr (!TRANSPOSED) {
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
            const int64_t r = r0 + y + i, c = c0 + x;
            if (r < a.rows && c < a.kp) ((T*)a.dst)[r * a.kp + c] = c < a.cols ? ((const T*)a.src)[r * a.stride + c] : (T)0;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
            const int64_t r = r0 + y + i, c = c0 + x;
            tile[y + i][x] = r < a.rows && c < a.cols ? ((const T*)a.src)[r * a.stride + c] : (T)0;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
            const int64_t c = c0 + y + i, r = r0 + x;
            if (c < a.cols && r < a.kp) ((T*)a.dst)[c * a.kp + r] = tile[x][y + i];
        }
    }
}

hipError_t launch_pack(PackArgs& a, int elem_bytes, bool transposed, hipStream_t st) {
    const int64_t blocks = transposed ? ((a.kp + 63) / 64) * ((a.cols + 63) / 64) : ((a.rows + 63) / 64) * ((a.kp + 63) / 64);
    const void* fn = elem_bytes == 4 ? (transposed ? (const void*)&k_pack<uint32_t, true> : (const void*)&k_pack<uint32_t, false>)
                   : elem_bytes == 2 ? (transposed ? (const void*)&k_pack<uint16_t, true> : (const void*)&k_pack<uint16_t, false>)
                                     : (transposed ? (const void*)&k_pack<uint8_t, true> : (const void*)&k_pack<uint8_t, false>);
    void* args[] = {&a};
    return hipLaunchKernel(fn, dim3((unsigned)blocks), dim3(256), args, 0, st);
}

// ---- dout act'(pre) -------------------------------------------------------------------------------------
// 64 x 64 values a workgroup; the column sums come from the values before they are rounded.
template <typename T> __global__ __launch_bounds__(256) void k_dpre(DpreArgs a) {
    __shared__ T tile[64][64 + 4 / (int)sizeof(T)];
    __shared__ float sums[256];
    const int64_t cb = (a.N + 63) / 64;
    const int64_t r0 = (int64_t)(blockIdx.x / (uint32_t)cb) * 64, c0 = (int64_t)(blockIdx.x % (uint32_t)cb) * 64;
    const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
    const int64_t c = c0 + x;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 64; i += 4) {
        const int64_t r = r0 + y + i;
        float v = 0.f;
        if (r < a.M && c < a.N) {
            v = (float)((const T*)a.dout)[r * a.N + c];
            if (a.act) v *= act_d((float)((const T*)a.pre)[r * a.N + c], a.act);
        }
        s += v;
        const T o = (T)v;
        if (a.rows && r < a.M && c < a.np) ((T*)a.rows)[r * a.np + c] = o;
        if (a.cols) tile[y + i][x] = o;
    }
    sums[threadIdx.x] = s;
    __syncthreads();
    if (a.part && threadIdx.x < 64 && c < a.N)
        a.part[(r0 / 64) * a.N + c] = (sums[x] + sums[64 + x]) + (sums[128 + x] + sums[192 + x]);
    if (a.cols) {
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
            const int64_t n = c0 + y + i, m = r0 + x;
            if (n < a.N && m < a.mp) ((T*)a.cols)[n * a.mp + m] = tile[x][y + i];
        }
    }
}

__global__ __launch_bounds__(256) void k_dbias(const float* part, float* db, int parts, int64_t N) {
    __shared__ float lds[256];
    const int64_t c = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
    const bool live = c < N;
    const float s = sum_rows<float>(part + (live ? c : 0), N, parts, lds, live);
    if (live && threadIdx.x < 64) db[c] = s;
}

hipError_t launch_dpre(DpreArgs& a, int dtype, float* dbias, hipStream_t st) {
    // (a padded column behind N lies in the last block of 64, a padded row behind M likewise: both pitches are the next
    // multiple of at most 8)
    const int64_t blocks = ((a.M + 63) / 64) * ((a.N + 63) / 64);
    const void* fn = dtype == DT_F32 ? (const void*)&k_dpre<float>
                   : dtype == DT_F16 ? (const void*)&k_dpre<_Float16> : (const void*)&k_dpre<__bf16>;
    void* args[] = {&a};
    const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)blocks), dim3(256), args, 0, st);
    if (e != hipSuccess || !dbias) return e;
    int parts = (int)((a.M + 63) / 64);
    void* sum_args[] = {&a.part, &dbias, &parts, &a.N};
    return hipLaunchKernel((const void*)&k_dbias, dim3((unsigned)((a.N + 63) / 64)), dim3(256), sum_args, 0, st);
}

}  // namespace ssd
