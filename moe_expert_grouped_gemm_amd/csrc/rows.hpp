// rows.hpp -- pieces shared by the kernels that hold rows of a matrix in
// registers (norms, the block's norms and gate, the experts' weighted sum):
// reductions over a wave or a row's team of waves, bf16 and E4M3 packing,
// 16-byte loads and stores that may go past the caches.
#pragma once
#include "common.hpp"

namespace ptgg {
namespace {

// Sum over the wave, in every lane: four DPP steps inside each 16 lanes, then
// the four rows' sums by readlane.
__device__ __forceinline__ float wave_sum(float x)
{
    x += bits_f32(__builtin_amdgcn_update_dpp(0, (int)f32_bits(x), 0xB1, 0xF, 0xF, false));    // lanes ^ 1
    x += bits_f32(__builtin_amdgcn_update_dpp(0, (int)f32_bits(x), 0x4E, 0xF, 0xF, false));    // lanes ^ 2
    x += bits_f32(__builtin_amdgcn_update_dpp(0, (int)f32_bits(x), 0x141, 0xF, 0xF, false));   // mirror of 8
    x += bits_f32(__builtin_amdgcn_update_dpp(0, (int)f32_bits(x), 0x140, 0xF, 0xF, false));   // mirror of 16
    const int i = (int)f32_bits(x);
    return (bits_f32(__builtin_amdgcn_readlane(i, 0)) + bits_f32(__builtin_amdgcn_readlane(i, 16))) +
           (bits_f32(__builtin_amdgcn_readlane(i, 32)) + bits_f32(__builtin_amdgcn_readlane(i, 48)));
}

__device__ __forceinline__ uint32_t quad_max_u32(uint32_t x)
{
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, false));
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, false));
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t x)
{
    x = quad_max_u32(x);
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xF, 0xF, false));
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x140, 0xF, 0xF, false));
    return max(max((uint32_t)__builtin_amdgcn_readlane((int)x, 0), (uint32_t)__builtin_amdgcn_readlane((int)x, 16)),
               max((uint32_t)__builtin_amdgcn_readlane((int)x, 32), (uint32_t)__builtin_amdgcn_readlane((int)x, 48)));
}

// Across the W waves of a row's team (the whole workgroup where W > 1), in a
// fixed order; s holds W words that no other reduction in flight uses.
template <int W>
__device__ __forceinline__ float team_sum(float x, float *s)
{
    x = wave_sum(x);
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
        __syncthreads();
        x = s[0];
#pragma unroll
        for (int w = 1; w < W; ++w) x += s[w];
    }
    return x;
}

template <int W>
__device__ __forceinline__ uint32_t team_max_u32(uint32_t x, uint32_t *s)
{
    x = wave_max_u32(x);
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
        __syncthreads();
        x = s[0];
#pragma unroll
        for (int w = 1; w < W; ++w) x = max(x, s[w]);
    }
    return x;
}

__device__ __forceinline__ void unpack8(const uintx4 v, float (&f)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bits_f32(v[i] << 16);
        f[2 * i + 1] = bits_f32(v[i] & 0xFFFF0000u);
    }
}

// bf16 to nearest even; a NaN stays a (quiet) NaN.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)lo, (__bf16)hi});
}

__device__ __forceinline__ uintx4 pack8(const float (&f)[8])
{
    return uintx4{bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7])};
}

// E4M3 within +-448; NaN stays NaN.
__device__ __forceinline__ float clamp448(float v)
{
    const float c = __builtin_fminf(__builtin_fmaxf(v, -448.0f), 448.0f);
    return v != v ? v : c;
}

__device__ __forceinline__ uintx2 codes8(const float (&f)[8])
{
    int w0 = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(f[0]), clamp448(f[1]), 0, false);
    w0 = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(f[2]), clamp448(f[3]), w0, true);
    int w1 = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(f[4]), clamp448(f[5]), 0, false);
    w1 = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(f[6]), clamp448(f[7]), w1, true);
    return uintx2{(uint32_t)w0, (uint32_t)w1};
}

__device__ __forceinline__ uint32_t amax8(const float (&f)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, f32_bits(f[i]) & 0x7FFFFFFFu);
    return m;
}

// Loads and stores, past the caches with NT -- where a lane's 16 bytes are all
// that it reads there: of 8 fp32 values two instructions read half a line each,
// and the second must find it in the caches.
template <bool NT, class T>
__device__ __forceinline__ T load_as(const void *p)
{
    return NT ? __builtin_nontemporal_load((const T *)p) : *(const T *)p;
}
template <bool NT, class T>
__device__ __forceinline__ void store_as(void *p, T v)
{
    if (NT) __builtin_nontemporal_store(v, (T *)p);
    else *(T *)p = v;
}

// Eight values of the residual stream from element e.
template <bool F32, bool NT>
__device__ __forceinline__ void load_stream(const void *p, int64_t e, float (&f)[8])
{
    if constexpr (F32) {
        const floatx4 a = *(const floatx4 *)((const float *)p + e), b = *(const floatx4 *)((const float *)p + e + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = a[i], f[4 + i] = b[i];
    } else {
        unpack8(load_as<NT, uintx4>((const uint16_t *)p + e), f);
    }
}

template <bool F32, bool NT>
__device__ __forceinline__ void store_stream(void *p, int64_t e, const float (&f)[8])
{
    if constexpr (F32) {
        *(floatx4 *)((float *)p + e) = floatx4{f[0], f[1], f[2], f[3]};
        *(floatx4 *)((float *)p + e + 4) = floatx4{f[4], f[5], f[6], f[7]};
    } else {
        store_as<NT>((uint16_t *)p + e, pack8(f));
    }
}

}  // namespace
}  // namespace ptgg
