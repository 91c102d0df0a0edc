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

// One step of a reduction over 2, 4, ... 64 lanes: op(x, its value in the other
// half of each 2 D lanes), the smaller groups being uniform already.  All on
// the vector ALU: DPP within 16 lanes, the row swaps above.
template <int D, class Op>
__device__ __forceinline__ uint32_t step_u32(uint32_t x, Op op)
{
    if constexpr (D <= 8) {
        constexpr int ctrl = D == 1 ? 0xB1 : D == 2 ? 0x4E : D == 4 ? 0x141 : 0x140;
        return op(x, (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, ctrl, 0xF, 0xF, false));
    } else if constexpr (D == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        return op(r[0], r[1]);
    } else {
        const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        return op(r[0], r[1]);
    }
}

// Reductions over LANES lanes (a power of two; every lane of the group
// active): all lanes get the result, the same bits in each.
template <int LANES, class Op>
__device__ __forceinline__ uint32_t group_reduce(uint32_t x, Op op)
{
    if constexpr (LANES > 1) x = step_u32<1>(x, op);
    if constexpr (LANES > 2) x = step_u32<2>(x, op);
    if constexpr (LANES > 4) x = step_u32<4>(x, op);
    if constexpr (LANES > 8) x = step_u32<8>(x, op);
    if constexpr (LANES > 16) x = step_u32<16>(x, op);
    if constexpr (LANES > 32) x = step_u32<32>(x, op);
    return x;
}
template <int LANES>
__device__ __forceinline__ float group_sum(float x)
{
    return bits_f32(group_reduce<LANES>(f32_bits(x), [](uint32_t a, uint32_t b) { return f32_bits(bits_f32(a) + bits_f32(b)); }));
}
// Sum of a lane's f(0) .. f(EPL - 1): fours one after another, then pairs of them, as four to a lane are joined across
// lanes, so that the bits are the same however many a lane holds.
template <int EPL, class F>
__device__ __forceinline__ float fours_sum(F f)
{
    float s[EPL / 4];
#pragma unroll
    for (int i = 0; i < EPL / 4; ++i) s[i] = ((f(4 * i) + f(4 * i + 1)) + f(4 * i + 2)) + f(4 * i + 3);
#pragma unroll
    for (int n = 1; n < EPL / 4; n *= 2)
#pragma unroll
        for (int i = 0; i + n < EPL / 4; i += 2 * n) s[i] += s[i + n];
    return s[0];
}
// x of the group's lane j, in every lane.
template <int LANES>
__device__ __forceinline__ uint32_t group_lane(uint32_t x, int j)
{
    if constexpr (LANES == 64) return (uint32_t)__builtin_amdgcn_readlane((int)x, j);
    return (uint32_t)__shfl((int)x, ((threadIdx.x & 63) & ~(LANES - 1)) + j, 64);
}
// Over the slots of a token, which lie in the group's first 16 lanes at most
// and are zero elsewhere; valid in those lanes.
template <int LANES>
__device__ __forceinline__ float slots_sum(float x)
{
    return group_sum<LANES < 16 ? LANES : 16>(x);
}
template <int D>
__device__ __forceinline__ double add_step(double x)
{
    constexpr int ctrl = D == 1 ? 0xB1 : D == 2 ? 0x4E : D == 4 ? 0x141 : 0x140;
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t l = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, ctrl, 0xF, 0xF, false);
    const uint32_t h = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), ctrl, 0xF, 0xF, false);
    return x + __builtin_bit_cast(double, (uint64_t)h << 32 | l);
}
template <int LANES>
__device__ __forceinline__ double slots_sum(double x)
{
    x = add_step<4>(add_step<2>(add_step<1>(x)));
    if constexpr (LANES > 8) x = add_step<8>(x);
    return x;
}
template <int LANES>
__device__ __forceinline__ float group_max(float x)
{
    return bits_f32(group_reduce<LANES>(f32_bits(x), [](uint32_t a, uint32_t b) {
        return f32_bits(__builtin_fmaxf(bits_f32(a), bits_f32(b)));
    }));
}
template <int LANES>
__device__ __forceinline__ uint32_t group_max_u32(uint32_t x)
{
    return group_reduce<LANES>(x, [](uint32_t a, uint32_t b) { return max(a, b); });
}

// The sigmoid in 64 bits: scores that differ by less than fp32 can tell apart
// would otherwise be ordered by the rounding of exp, and a token whose logits
// all lie far below zero would have no shares left.
__device__ __forceinline__ double sigmoid64(float z) { return 1.0 / (1.0 + exp(-(double)z)); }

// The score's inverse for keys that are not 0.
__device__ __forceinline__ float key_score(uint32_t k) { return bits_f32(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu)); }

// One logit, as load_logits gives it.
__device__ __forceinline__ float logit_at(const void *logits, int bf16, int64_t i)
{
    return bf16 ? bf16_to_f32(((const uint16_t *)logits)[i]) : ((const float *)logits)[i];
}

// The least 32-bit score that may belong among the chosen once scores are exact, given the k-th one's.  A sigmoid is off
// by less than 2^-22 (|z| v (1 - v) < 1/4 bounds the exponent's rounding, and three more roundings of 2^-24), the sum
// with the bias by a rounding: less than half of the margin.  Never -inf, which is what a score has that must not be
// chosen, also where the k-th is next to fp32's lowest value (experts masked by their bias).
__host__ __device__ __forceinline__ float candidate_floor(float kth)
{
    return __builtin_fmaxf(kth - 0x1p-20f * (1.0f + __builtin_fabsf(kth)), -3.40282346638528859812e+38f);
}

// What a slot's lane knows of its expert.
struct Slot {
    int id;                   // -1: none
    uint32_t key;
};

// The k largest keys of the group, ties to the lowest expert; lane j < k gets
// the j-th one (id -1 where all the rest are 0).  Taken keys become 0.
template <int LANES, int EPL>
__device__ __forceinline__ Slot take_largest(int k, uint32_t (&key)[EPL])
{
    const int sub = threadIdx.x & (LANES - 1), e0 = sub * EPL;
    Slot s = {-1, 0};
    for (int j = 0; j < k; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) best = max(best, key[i]);
        const uint32_t top = group_max_u32<LANES>(best);
        // the lowest expert that has it: in its lane, then over the lanes
        int at = 0;
#pragma unroll
        for (int i = EPL - 1; i > 0; --i) {
            at = key[i] == top ? i : at;
            // all the comparisons at once would overflow the scalar registers that hold their outcomes
            if (EPL > 4 && i % 4 == 0) __builtin_amdgcn_sched_barrier(0);
        }
        at = key[0] == top ? 0 : at;
        uint32_t e;
        if constexpr (LANES == 64) {
            e = group_lane<64>((uint32_t)(e0 + at), __builtin_ctzll(__ballot(best == top)));   // some lane has it
        } else {
            e = ~group_max_u32<LANES>(best == top ? ~(uint32_t)(e0 + at) : 0u);
        }
        if (sub == j && top != 0) s = {(int)e, top};
        // (where nothing is left this clears a 0)
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            key[i] = (int)e - e0 == i ? 0u : key[i];
            if (EPL > 4 && i % 4 == 3) __builtin_amdgcn_sched_barrier(0);
        }
    }
    return s;
}

// Choose the k experts with the largest scores (ties to the lowest index) and
// their weights.  z, bias: the lane's experts' (0 without a bias).  Lane j < k of
// the group returns the j-th expert (-1: none left that can be chosen) and its
// weight.  nan: a NaN among the scores.
//
// Sigmoid scores are ordered as 64 bits rounded to 32 give them, which is dear
// for every expert.  Scores in 32 bits name the candidates; where exactly k of
// them reach the k-th one's neighbourhood (candidate_floor), only those are
// computed in 64 bits and put in order, else all that do.
template <int LANES, int EPL>
__device__ __forceinline__ void choose(const RouteParams &p, int64_t t, const float (&z)[EPL], const float (&bias)[EPL],
                                       int &id, float &weight, bool &nan)
{
    const int sub = threadIdx.x & (LANES - 1);
    const float ninf = -__builtin_huge_valf();
    uint32_t key[EPL];
    nan = false;
    if (!p.sigmoid) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            nan |= z[i] != z[i];
            key[i] = score_key(z[i]);
        }
        const Slot s = take_largest<LANES, EPL>(p.k, key);
        id = s.id;
        const float mine = key_score(s.key);
        // the largest logit of all is the first slot's
        const float m = bits_f32(group_lane<LANES>(f32_bits(mine), 0));
        const float e = id >= 0 ? expf(mine - m) : 0.0f;
        float total;
        if (p.renorm) {
            total = slots_sum<LANES>(e);
        } else {
            total = group_sum<LANES>(fours_sum<EPL>([&](int i) { return z[i] > ninf ? expf(z[i] - m) : 0.0f; }));
        }
        weight = id >= 0 ? e / total * p.scale : 0.0f;
        return;
    }
    float near[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        near[i] = z[i] > ninf ? __builtin_amdgcn_rcpf(1.0f + __expf(-z[i])) + bias[i] : z[i];
        nan |= near[i] != near[i];
        key[i] = score_key(near[i]);
    }
    Slot s = take_largest<LANES, EPL>(p.k, key);
    const uint32_t kth = group_max_u32<LANES>(sub == p.k - 1 ? s.key : 0u);
    const float floor = candidate_floor(key_score(kth));
    bool close = false;
#pragma unroll
    for (int i = 0; i < EPL; ++i) close |= kth != 0 && key[i] != 0 && near[i] >= floor;
    double v;
    if (group_max_u32<LANES>(close ? 1u : 0u)) {               // one that was not taken is near
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            key[i] = 0;                                        // the others lie lower for certain
            if (near[i] >= floor) key[i] = score_key((float)(sigmoid64(z[i]) + (double)bias[i]));
        }
        s = take_largest<LANES, EPL>(p.k, key);
        id = s.id;
        v = id >= 0 ? sigmoid64(logit_at(p.logits, p.bf16, t * p.E + id)) : 0.0;
    } else {
        // the chosen ones in the order of their exact scores; lanes without one stay where they are, behind
        v = 0.0;
        uint32_t exact = 0;
        if (s.id >= 0) {
            v = sigmoid64(logit_at(p.logits, p.bf16, t * p.E + s.id));
            exact = score_key((float)(v + (double)(p.bias ? p.bias[s.id] : 0.0f)));
        }
        int rank = 0;
        for (int j = 0; j < p.k; ++j) {
            const uint32_t other = group_lane<LANES>(exact, j);
            const int oid = (int)group_lane<LANES>((uint32_t)s.id, j);
            rank += oid >= 0 && (other > exact || (other == exact && oid < s.id)) ? 1 : 0;
        }
        const int to = 4 * (((threadIdx.x & 63) & ~(LANES - 1)) + (s.id >= 0 ? rank : sub));
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        id = __builtin_amdgcn_ds_permute(to, s.id);
        const uint32_t l = (uint32_t)__builtin_amdgcn_ds_permute(to, (int)(uint32_t)u);
        const uint32_t h = (uint32_t)__builtin_amdgcn_ds_permute(to, (int)(uint32_t)(u >> 32));
        v = __builtin_bit_cast(double, (uint64_t)h << 32 | l);
    }
    if (p.renorm) {
        const double total = slots_sum<LANES>(v);
        v = total > 0.0 ? v / total : 0.0;
    }
    weight = (float)(v * (double)p.scale);
}

}  // namespace ptgg
