// route_device.hpp -- device pieces of the router, shared by the router's own
// kernels and the few-token layer.
//
// LANES consecutive lanes hold one token's logits, EPL consecutive experts
// each, so a tie between lanes falls to the lowest lane.
#pragma once
#include "common.hpp"
#include "layer.hpp"

namespace ptgg {

// Logits e0 .. e0 + EPL - 1 of a token (-inf past E).  vec: rows start on
// 16-byte (fp32) or 8-byte (bf16) boundaries.
template <int EPL>
__device__ __forceinline__ void load_logits(const void *logits, int bf16, int64_t row, int E, int e0, float (&z)[EPL])
{
    const float ninf = -__builtin_huge_valf();
    const bool vec = (E & 3) == 0;
#pragma unroll
    for (int i = 0; i < EPL; i += 4) {
        const int e = e0 + i;
        if (vec) {
            if (e < E) {
                if (bf16) {
                    const uintx2 v = *(const uintx2 *)((const uint16_t *)logits + row * E + e);
                    z[i] = bits_f32(v[0] << 16), z[i + 1] = bits_f32(v[0] & 0xFFFF0000u);
                    z[i + 2] = bits_f32(v[1] << 16), z[i + 3] = bits_f32(v[1] & 0xFFFF0000u);
                } else {
                    const floatx4 v = *(const floatx4 *)((const float *)logits + row * E + e);
                    z[i] = v[0], z[i + 1] = v[1], z[i + 2] = v[2], z[i + 3] = v[3];
                }
            } else {
                z[i] = z[i + 1] = z[i + 2] = z[i + 3] = ninf;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                z[i + j] = ninf;
                if (e + j < E)
                    z[i + j] = bf16 ? bf16_to_f32(((const uint16_t *)logits)[row * E + e + j])
                                    : ((const float *)logits)[row * E + e + j];
            }
        }
    }
}

// Order-preserving unsigned key of a score; 0 for what is never chosen
// (-inf and NaN).
__device__ __forceinline__ uint32_t score_key(float s)
{
    if (!(s > -__builtin_huge_valf())) return 0u;
    if (s == 0.0f) s = 0.0f;                       // -0 and +0 are equal scores
    const uint32_t u = f32_bits(s);
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

// Reductions over LANES lanes (a power of two; every lane of the group active).
template <int LANES>
__device__ __forceinline__ float group_sum(float x)
{
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) x += __shfl_xor(x, d, 64);
    return x;
}
template <int LANES>
__device__ __forceinline__ double group_sum(double x)
{
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) x += __shfl_xor(x, d, 64);
    return x;
}
template <int LANES>
__device__ __forceinline__ float group_max(float x)
{
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) x = __builtin_fmaxf(x, __shfl_xor(x, d, 64));
    return x;
}
template <int LANES>
__device__ __forceinline__ uint32_t group_max_u32(uint32_t x)
{
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) x = max(x, (uint32_t)__shfl_xor((int)x, d, 64));
    return x;
}

// The sigmoid in 64 bits: scores that differ by less than fp32 can tell apart
// would otherwise be ordered by the rounding of exp, and a token whose logits
// all lie far below zero would have no shares left.
__device__ __forceinline__ double sigmoid64(float z) { return 1.0 / (1.0 + exp(-(double)z)); }

// Choose the k experts with the largest scores (ties to the lowest index) and
// their weights.  Lane j < k of the group returns the j-th expert (-1: none
// left that can be chosen) and its weight.  nan: a NaN among the scores.
template <int LANES, int EPL>
__device__ __forceinline__ void choose(const RouteParams &p, const float (&z)[EPL], int &id, float &weight, bool &nan)
{
    const int sub = threadIdx.x & (LANES - 1), e0 = sub * EPL;
    uint32_t key[EPL];
    nan = false;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        float s = z[i];
        if (p.sigmoid && z[i] > -__builtin_huge_valf()) {
            const float b = p.bias && e0 + i < p.E ? p.bias[e0 + i] : 0.0f;
            s = (float)(sigmoid64(z[i]) + (double)b);
        }
        nan |= s != s;
        key[i] = score_key(s);
    }
    id = -1;
    float mine = -__builtin_huge_valf();
    const uint64_t group = LANES == 64 ? ~0ull : ((1ull << (LANES & 63)) - 1) << ((threadIdx.x & 63) & ~(LANES - 1));
    for (int j = 0; j < p.k; ++j) {
        uint32_t best = 0;
        int at = 0;
        float bz = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (key[i] > best) best = key[i], at = i, bz = z[i];
        const uint32_t top = group_max_u32<LANES>(best);
        const uint64_t have = __ballot(best == top) & group;
        const int lane = __builtin_ctzll(have);                    // the group is never empty
        const int e = __shfl(e0 + at, lane, 64);
        const float ez = __shfl(bz, lane, 64);
        if (top != 0) {
            if (sub == j) id = e, mine = ez;
            if ((int)(threadIdx.x & 63) == lane) {
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (i == at) key[i] = 0;
            }
        }
    }
    if (p.sigmoid) {
        double v = id >= 0 ? sigmoid64(mine) : 0.0;
        if (p.renorm) {
            const double total = group_sum<LANES>(v);
            v = total > 0.0 ? v / total : 0.0;
        }
        weight = (float)(v * (double)p.scale);
    } else {
        // largest logit first: softmax over the chosen (renorm) or over all
        float m = mine;
        if (!p.renorm) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) m = __builtin_fmaxf(m, z[i]);
        }
        m = group_max<LANES>(m);
        const float e = id >= 0 ? expf(mine - m) : 0.0f;
        float total = e;
        if (!p.renorm) {
            total = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) total += z[i] > -__builtin_huge_valf() ? expf(z[i] - m) : 0.0f;
        }
        total = group_sum<LANES>(total);
        weight = id >= 0 ? e / total * p.scale : 0.0f;
    }
}

}  // namespace ptgg
