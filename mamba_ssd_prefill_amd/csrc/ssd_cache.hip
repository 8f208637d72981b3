// ssd_cache.hip -- states held in 8 bits: written with one fp32 scale per group of consecutive values, and
// read back (ssd_state_cache_write / _read in include/mamba_ssd.h).
//
//     scale = max|v| / M,  code = round(v / scale),  v' = code * scale        M = 127 (int8) or 448 (e4m3)
//
// Both directions are HBM-bound streams: 52 MB each at 16 x 655360 fp32 values in 12.7 us written and 9.4 us read
// (4.1 and 5.6 TB/s; a large copy reaches 5.0, and part of this comes from the last-level cache).  A lane takes 4
// consecutive values (16 or 8 bytes of state, 4 bytes of codes); the group / 4 lanes of a group share their
// maximum by lane exchanges.
#include "ssd_code8.h"
#include "ssd_select.h"

namespace ssd {

template <typename S> __device__ inline f32x4 cache_load4(const S* p) {
    if constexpr (sizeof(S) == 4) {
        return *(const f32x4*)p;
    } else {
        const typename TT<S>::v4 v = *(const typename TT<S>::v4*)p;
        return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
    }
}

// The largest m over the group / 4 neighbouring lanes of a group (4, 8, 16 or 32).
template <int CTRL> __device__ inline uint32_t max_dpp(uint32_t m) {
    return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, CTRL, 0xf, 0xf, true));
}
__device__ inline uint32_t group_max(uint32_t m, int group) {
    m = max_dpp<0x4e>(max_dpp<0xb1>(m));    // lanes ^ 1, ^ 2
    if (group >= 32) m = max_dpp<0x141>(m);  // the other half of 8
    if (group >= 64) m = max_dpp<0x140>(m);  // the other half of 16
    if (group >= 128) {
        const auto r = __builtin_amdgcn_permlane16_swap(m, m, false, false);
        const uint32_t r0 = r[0], r1 = r[1];
        m = max(r0, r1);
    }
    return m;
}

// Pieces of 4 values a lane takes, 1024 values apart.  Measured at 16 x 655360 fp32 values (42 MB, 10 MB of codes): write
// 15.8, 14.5, 17.4, 28.8 us with 1, 2, 4, 8 pieces (a workgroup computes when all its loads are there, so
// small ones overlap better), read 12.4, 10.3, 9.7, 10.1 us.
constexpr int kWriteIter = 2, kReadIter = 4;

// Block (row, run of values); groups never straddle a wave's 256 consecutive values.
template <typename S> __global__ __launch_bounds__(256) void k_cache_write(CacheArgs a) {
    const uint32_t nrun = (uint32_t)((a.elems + 1024 * kWriteIter - 1) / (1024 * kWriteIter));
    const int b = (int)(blockIdx.x / nrun), gbits = __builtin_ctz(a.group);
    const int64_t e0 = (int64_t)(blockIdx.x % nrun) * 1024 * kWriteIter + threadIdx.x * 4;
    const int slot = a.slots ? a.slots[b] : b;
    if (slot < 0 || slot >= a.nslots) return;
    const S* src = (const S*)a.state_in + (int64_t)b * a.elems;
    uint8_t* codes = a.codes + (int64_t)slot * a.elems;
    float* scales = a.scales + (int64_t)slot * (a.elems >> gbits);
    f32x4 v[kWriteIter];
#pragma unroll
    for (int i = 0; i < kWriteIter; ++i) {
        v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        const int64_t e = e0 + i * 1024;
        if (e < a.elems) v[i] = cache_load4<S>(src + e);
    }
    const float most = a.format == 0 ? 127.f : 448.f;
#pragma unroll
    for (int i = 0; i < kWriteIter; ++i) {
        const int64_t e = e0 + i * 1024;
        // as integers the magnitudes keep their order, with the infinities and NaN above every number
        uint32_t mu = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float x = v[i][j];
            mu = max(mu, __builtin_bit_cast(uint32_t, x) & 0x7fffffffu);
        }
        mu = group_max(mu, a.group);
        float s = __builtin_bit_cast(float, mu) / most;
        uint32_t code = 0;
        if (mu >= 0x7f800000u) {
            s = __builtin_nanf("");
        } else if (s < kMinScale) {
            s = 0.f;
        } else {
            const float inv = 1.f / s;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float q = quotient_to_odd(v[i][j], s, inv);
                code |= (a.format == 0 ? code_int8(q) : code_e4m3(q)) << (8 * j);
            }
        }
        if (e < a.elems) {
            *(uint32_t*)(codes + e) = code;
            if (!(e & (a.group - 1))) scales[e >> gbits] = s;
        }
    }
}

template <typename S> __global__ __launch_bounds__(256) void k_cache_read(CacheArgs a) {
    const uint32_t nrun = (uint32_t)((a.elems + 1024 * kReadIter - 1) / (1024 * kReadIter));
    const int b = (int)(blockIdx.x / nrun), gbits = __builtin_ctz(a.group);
    const int64_t e0 = (int64_t)(blockIdx.x % nrun) * 1024 * kReadIter + threadIdx.x * 4;
    const int slot = a.slots ? a.slots[b] : b;
    const bool have = slot >= 0 && slot < a.nslots;
    const uint8_t* codes = a.codes + (have ? slot : 0) * a.elems;
    const float* scales = a.scales + (have ? slot : 0) * (a.elems >> gbits);
    S* dst = (S*)a.state_out + (int64_t)b * a.elems;
    uint32_t c[kReadIter];
    float s[kReadIter];
#pragma unroll
    for (int i = 0; i < kReadIter; ++i) {
        const int64_t e = e0 + i * 1024;
        c[i] = 0;
        s[i] = 0.f;
        if (have && e < a.elems) {
            c[i] = *(const uint32_t*)(codes + e);
            s[i] = scales[e >> gbits];
        }
    }
#pragma unroll
    for (int i = 0; i < kReadIter; ++i) {
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
    const int64_t run = 1024 * (write ? kWriteIter : kReadIter), nrun = (a.elems + run - 1) / run;
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
