// ssd_cache.hip -- states held in 8 bits: written with one fp32 scale per group of consecutive values, and
// read back (ssd_state_cache_write / _read in include/mamba_ssd.h).
//
//     scale = max|v| / M,  code = round(v / scale),  v' = code * scale        M = 127 (int8) or 448 (e4m3)
//
// Both directions are HBM-bound streams.  A lane takes 4 consecutive values (16 or 8 bytes of state, 4 bytes of
// codes); the group / 4 lanes of a group share their maximum by cross-lane shuffles.
#include "ssd_device.h"
#include "ssd_select.h"

namespace ssd {

constexpr float kMinScale = 0x1p-80f;  // below it the remainder of a quotient next to a border could leave the fp32 range

// v / s for a rounding to fewer bits: the fp32 quotient whose last bit is set when it is not exact, cut
// towards zero ("rounded to odd").  Rounding it again to 8 bits or fewer gives the exact quotient's nearest
// code; rounding a quotient that was itself rounded to nearest could fall on a border between two codes
// that the exact quotient only comes close to.  The remainder v - q s is exact in one fma.
__device__ inline float quotient_to_odd(float v, float s) {
    const float q = v / s;
    const float r = __builtin_fmaf(-q, s, v);
    uint32_t u = __builtin_bit_cast(uint32_t, q);
    if (r != 0.f) {
        if ((r < 0.f) != (q < 0.f)) u -= 1;  // |q| is above the exact quotient: step back
        u |= 1u;
    }
    return __builtin_bit_cast(float, u);
}

__device__ inline uint32_t code_int8(float q) {
    return (uint32_t)(int)rintf(fminf(fmaxf(q, -127.f), 127.f)) & 0xffu;
}

// e4m3 of a clamped quotient: the nearest multiple of the step at its magnitude, ties to even.
__device__ inline uint32_t code_e4m3(float q) {
    const uint32_t sign = __builtin_bit_cast(uint32_t, q) >> 31 << 7;
    const float m = fminf(fabsf(q), 448.f);
    int e = (int)(__builtin_bit_cast(uint32_t, m) >> 23) - 127;
    e = e < -6 ? -6 : e;
    // m / 2^(e-3) is below 16, so adding 1.5 * 2^23 rounds it to an integer, ties to even
    const float k = m * __builtin_bit_cast(float, (uint32_t)(127 + 3 - e) << 23) + 12582912.f;
    const int n = (int)(__builtin_bit_cast(uint32_t, k) & 0x3fffffu);  // 0 .. 16, in steps of 2^(e-3)
    // n = 8 + mantissa in the binade e (0 .. 7: the subnormal one); 16 carries into the next binade
    return sign | (uint32_t)((e + 6) * 8 + n);
}

__device__ inline float value_e4m3(uint32_t c) {
    const int e = (c >> 3) & 15, m = c & 7;
    if (e == 15 && m == 7) return __builtin_nanf("");
    const float v = e ? __builtin_bit_cast(float, (uint32_t)(e + 120) << 23 | (uint32_t)m << 20) : (float)m * 0x1p-9f;
    return c & 0x80u ? -v : v;
}

template <typename S> __device__ inline f32x4 cache_load4(const S* p) {
    if constexpr (sizeof(S) == 4) {
        return *(const f32x4*)p;
    } else {
        const typename TT<S>::v4 v = *(const typename TT<S>::v4*)p;
        return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
    }
}

constexpr int kCacheIter = 4;  // pieces of 4 values a lane takes (1024 values apart)

// Block (row, run of 4096 values); groups never straddle a wave's 256 consecutive values.
template <typename S> __global__ __launch_bounds__(256) void k_cache_write(CacheArgs a) {
    const int64_t nrun = (a.elems + 1024 * kCacheIter - 1) / (1024 * kCacheIter);
    const int b = (int)(blockIdx.x / nrun);
    const int64_t e0 = (int64_t)(blockIdx.x % nrun) * 1024 * kCacheIter + threadIdx.x * 4;
    const int slot = a.slots ? a.slots[b] : b;
    if (slot < 0 || slot >= a.nslots) return;
    const S* src = (const S*)a.state_in + (int64_t)b * a.elems;
    uint8_t* codes = a.codes + (int64_t)slot * a.elems;
    float* scales = a.scales + (int64_t)slot * (a.elems / a.group);
    f32x4 v[kCacheIter];
#pragma unroll
    for (int i = 0; i < kCacheIter; ++i) {
        v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        const int64_t e = e0 + i * 1024;
        if (e < a.elems) v[i] = cache_load4<S>(src + e);
    }
    const float most = a.format == 0 ? 127.f : 448.f;
#pragma unroll
    for (int i = 0; i < kCacheIter; ++i) {
        const int64_t e = e0 + i * 1024;
        float m = 0.f;
        bool bad = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            m = fmaxf(m, fabsf(v[i][j]));
            bad |= !(fabsf(v[i][j]) <= 3.402823466e38f);
        }
        if (bad) m = __builtin_inff();  // an infinity or a NaN in the group
        for (int d = a.group / 8; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
        float s = m / most;
        uint32_t code = 0;
        if (!(m <= 3.402823466e38f)) {
            s = __builtin_nanf("");
        } else if (s < kMinScale) {
            s = 0.f;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float q = quotient_to_odd(v[i][j], s);
                code |= (a.format == 0 ? code_int8(q) : code_e4m3(q)) << (8 * j);
            }
        }
        if (e < a.elems) {
            *(uint32_t*)(codes + e) = code;
            if (e % a.group == 0) scales[e / a.group] = s;
        }
    }
}

template <typename S> __global__ __launch_bounds__(256) void k_cache_read(CacheArgs a) {
    const int64_t nrun = (a.elems + 1024 * kCacheIter - 1) / (1024 * kCacheIter);
    const int b = (int)(blockIdx.x / nrun);
    const int64_t e0 = (int64_t)(blockIdx.x % nrun) * 1024 * kCacheIter + threadIdx.x * 4;
    const int slot = a.slots ? a.slots[b] : b;
    const bool have = slot >= 0 && slot < a.nslots;
    const uint8_t* codes = a.codes + (have ? slot : 0) * a.elems;
    const float* scales = a.scales + (have ? slot : 0) * (a.elems / a.group);
    S* dst = (S*)a.state_out + (int64_t)b * a.elems;
    uint32_t c[kCacheIter];
    float s[kCacheIter];
#pragma unroll
    for (int i = 0; i < kCacheIter; ++i) {
        const int64_t e = e0 + i * 1024;
        c[i] = 0;
        s[i] = 0.f;
        if (have && e < a.elems) {
            c[i] = *(const uint32_t*)(codes + e);
            s[i] = scales[e / a.group];
        }
    }
#pragma unroll
    for (int i = 0; i < kCacheIter; ++i) {
        const int64_t e = e0 + i * 1024;
        if (e >= a.elems) continue;
        f32x4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t k = (c[i] >> (8 * j)) & 0xffu;
            v[j] = (a.format == 0 ? (float)(int8_t)k : value_e4m3(k)) * s[i];
        }
        if constexpr (sizeof(S) == 4) {
            *(f32x4*)(dst + e) = v;
        } else {
            *(typename TT<S>::v4*)(dst + e) = cvt4<S>(v);
        }
    }
}

template <typename S> hipError_t launch_cache_s(CacheArgs& a, bool write, hipStream_t st) {
    const int64_t nrun = (a.elems + 1024 * kCacheIter - 1) / (1024 * kCacheIter);
    void* args[] = {&a};
    return hipLaunchKernel(write ? (const void*)&k_cache_write<S> : (const void*)&k_cache_read<S>,
                           dim3((unsigned)(nrun * a.batch)), dim3(256), args, 0, st);
}

static hipError_t launch_cache(CacheArgs& a, bool write, hipStream_t st) {
    switch (a.state_dtype) {
    case DT_F32: return launch_cache_s<float>(a, write, st);
    case DT_F16: return launch_cache_s<_Float16>(a, write, st);
    case DT_BF16: return launch_cache_s<__bf16>(a, write, st);
    default: return hipErrorNotSupported;
    }
}
hipError_t launch_cache_write(CacheArgs& a, hipStream_t st) { return launch_cache(a, true, st); }
hipError_t launch_cache_read(CacheArgs& a, hipStream_t st) { return launch_cache(a, false, st); }

}  // namespace ssd
