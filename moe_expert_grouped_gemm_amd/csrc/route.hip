// route.hip -- the MoE router: top-k experts of each token, their weights, the
// order of the chosen rows by expert, and the gradient of the logits.
//
// Order.  The row of pair (token t, slot j) with expert e is the number of
// rows of earlier experts plus the number of earlier tokens that chose e (a
// token chooses an expert once).  Tokens go in chunks of 64: a chunk keeps one
// 64-bit word per expert in LDS, bit t set where token t of the chunk chose
// it, so a rank is the population count of the bits below t -- no sort and no
// atomic whose order shows.  With several workgroups (parts of consecutive
// chunks) a second kernel adds the counts of the parts before.
//
// What bounds it: launch and wave-reduction latency; the logits of 16384
// tokens are 16 MB at most.
#include "route_device.hpp"

namespace ptgg {

namespace {

constexpr int kRouteThreads = 512;

// Exclusive scan of n values v[0..n) in LDS by a kRouteThreads workgroup, n <=
// 1024; returns the total.
__device__ __forceinline__ int scan_lds(int *v, int n, int *s_wave)
{
    constexpr int PER = kRouteMaxExperts / kRouteThreads;
    const int i0 = threadIdx.x * PER;
    int own[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        own[i] = i0 + i < n ? v[i0 + i] : 0;
        sum += own[i];
    }
    int total;
    int at = block_exclusive_scan<kRouteThreads>(sum, s_wave, &total);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (i0 + i < n) v[i0 + i] = at;
        at += own[i];
    }
    __syncthreads();
    return total;
}

// One part: chunks of 64 tokens in a row.  ONE: the only part, which finishes
// the order itself; otherwise row_of receives ranks within the part and
// counts the part's totals.
template <int LANES, int EPL, bool ONE>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteParams p, int chunks_per_part, RoutePlan plan)
{
    constexpr int GROUPS = kRouteThreads / LANES;
    __shared__ uint64_t s_mask[kRouteMaxExperts];
    __shared__ int s_count[kRouteMaxExperts];      // tokens of earlier chunks; with ONE, finally the first rows
    __shared__ int s_ids[kRouteChunk * kRouteMaxTopk];
    __shared__ int s_wave[kRouteThreads / 64];
    const int tid = threadIdx.x, sub = tid & (LANES - 1);
    const int64_t t_first = (int64_t)blockIdx.x * chunks_per_part * kRouteChunk;
    const int64_t t_last = min(p.T, t_first + (int64_t)chunks_per_part * kRouteChunk);
    for (int e = tid; e < p.E; e += kRouteThreads) s_count[e] = 0;
    bool any_nan = false;
    for (int64_t t0 = t_first; t0 < t_last; t0 += kRouteChunk) {
        const int n = (int)min((int64_t)kRouteChunk, t_last - t0);
        for (int e = tid; e < p.E; e += kRouteThreads) s_mask[e] = 0;
        __syncthreads();
        for (int i = tid / LANES; i < n; i += GROUPS) {       // a whole group of lanes per token
            float z[EPL];
            load_logits<EPL>(p.logits, p.bf16, t0 + i, p.E, sub * EPL, z);
            int id;
            float w;
            bool nan;
            choose<LANES, EPL>(p, z, id, w, nan);
            any_nan |= nan;
            if (sub < p.k) {
                p.topk_ids[(t0 + i) * p.k + sub] = id;
                p.topk_weights[(t0 + i) * p.k + sub] = w;
                s_ids[i * p.k + sub] = id;
                if (id >= 0) atomicOr((unsigned long long *)&s_mask[id], 1ull << i);
            }
        }
        __syncthreads();
        for (int i = tid; i < n * p.k; i += kRouteThreads) {
            const int id = s_ids[i], t = i / p.k;
            const int rank = id < 0 ? -1 : s_count[id] + __builtin_popcountll(s_mask[id] & ((1ull << t) - 1));
            if (ONE) s_ids[i] = rank;                          // one part of one chunk
            else p.row_of[t0 * p.k + i] = rank;
        }
        __syncthreads();
        for (int e = tid; e < p.E; e += kRouteThreads) s_count[e] += __builtin_popcountll(s_mask[e]);
        __syncthreads();
    }
    if (any_nan && p.err) atomicOr(p.err, kErrNanLogit);
    if (!ONE) {
        for (int e = tid; e < p.E; e += kRouteThreads) p.counts[(int64_t)blockIdx.x * p.E + e] = (uint16_t)s_count[e];
        return;
    }
    __shared__ int s_blocks[kRouteMaxExperts];
    for (int e = tid; e < p.E; e += kRouteThreads) {
        p.lens[e] = s_count[e];
        if (plan.plan) s_blocks[e] = (s_count[e] + plan.cap - 1) / plan.cap;
    }
    __syncthreads();
    const int total = scan_lds(s_count, p.E, s_wave);
    if (plan.plan) {
        const int blocks = scan_lds(s_blocks, p.E, s_wave);
        if (tid == 0) plan.plan[0] = blocks;
        for (int e = tid; e < p.E; e += kRouteThreads) {
            const int first = s_count[e], end = e + 1 < p.E ? s_count[e + 1] : total;
            FewBlock *b = (FewBlock *)(plan.plan + 4) + s_blocks[e];
            uint64_t left = s_mask[e];
            for (int r = first; r < end; r += plan.cap, ++b) {
                const int n = min(plan.cap, end - r);
                FewBlock v = {e, r, n, 0, {}};
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (i < n) {
                        v.token[i] = (uint8_t)__builtin_ctzll(left);
                        left &= left - 1;
                    }
                *b = v;
            }
        }
    }
    const int pairs = (int)p.T * p.k;
    for (int i = tid; i < pairs; i += kRouteThreads) {
        const int rank = s_ids[i];
        int row = -1;
        if (rank >= 0) {
            row = s_count[p.topk_ids[i]] + rank;               // written by this workgroup before its barriers
            p.token_of[row] = i / p.k;
        }
        p.row_of[i] = row;
        if (i >= total) p.token_of[i] = -1;
    }
}

// Second kernel of several parts: the part's first row of each expert is the
// rows of earlier experts plus those of earlier parts.
__global__ __launch_bounds__(kRouteThreads) void route_rows_kernel(RouteParams p, int parts, int chunks_per_part)
{
    __shared__ int s_before[kRouteMaxExperts], s_total[kRouteMaxExperts];
    __shared__ int s_wave[kRouteThreads / 64];
    const int tid = threadIdx.x, part = blockIdx.x;
    for (int e = tid; e < p.E; e += kRouteThreads) s_before[e] = s_total[e] = 0;
    __syncthreads();
    // E columns, and as many rows of counts side by side as the workgroup has
    const int side = max(1, kRouteThreads / p.E);
    for (int i = tid; i < side * p.E; i += kRouteThreads) {
        const int e = i % p.E;
        int before = 0, total = 0;
        for (int b = i / p.E; b < parts; b += side) {
            const int c = p.counts[(int64_t)b * p.E + e];
            total += c;
            before += b < part ? c : 0;
        }
        atomicAdd(&s_before[e], before);                       // integers: their order does not show
        atomicAdd(&s_total[e], total);
    }
    __syncthreads();
    if (part == 0)
        for (int e = tid; e < p.E; e += kRouteThreads) p.lens[e] = s_total[e];
    __syncthreads();
    const int total = scan_lds(s_total, p.E, s_wave);
    const int64_t i0 = (int64_t)part * chunks_per_part * kRouteChunk * p.k;
    const int64_t i1 = min(p.T * p.k, i0 + (int64_t)chunks_per_part * kRouteChunk * p.k);
    for (int64_t i = i0 + tid; i < i1; i += kRouteThreads) {
        const int id = p.topk_ids[i];
        if (id >= 0) {
            const int row = s_total[id] + s_before[id] + p.row_of[i];
            p.row_of[i] = row;
            p.token_of[row] = (int)(i / p.k);
        }
        if (i >= total) p.token_of[i] = -1;
    }
}

// dlogits[t, :].  With g = scale dweights and p the softmax over all experts:
//   softmax           p_e (g_e - sum_j p_j g_j)          (g_e = 0 where e was not chosen)
//   softmax, renorm   the same over the chosen alone
//   sigmoid           g v (1 - v);  renorm: (g - sum_j w_j g_j) / total first
// v (1 - v) is taken as q / (1 + q)^2 with q = e^-|z|, which keeps its digits
// where v rounds to 1.
template <int LANES, int EPL>
__global__ __launch_bounds__(kThreads) void route_bwd_kernel(RouteBwdParams p)
{
    const int sub = threadIdx.x & (LANES - 1), e0 = sub * EPL;
    const int64_t t = (int64_t)blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
    if (t >= p.T) return;                                      // whole groups
    const float ninf = -__builtin_huge_valf();
    float z[EPL], d[EPL];
    load_logits<EPL>(p.logits, p.bf16, t, p.E, e0, z);
    int id = -1;
    float g = 0.0f;
    if (sub < p.k) {
        id = p.topk_ids[t * p.k + sub];
        if (id < 0 || id >= p.E) id = -1;
        else g = p.dweights[t * p.k + sub] * p.scale;
    }
    // the chosen expert's logit, from the lane that holds it
    float mine = ninf;
    for (int j = 0; j < p.k; ++j) {
        const int e = __shfl(id, ((threadIdx.x & 63) & ~(LANES - 1)) + j, 64);
        float v = ninf;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (e == e0 + i) v = z[i];
        v = group_max<LANES>(v);
        if (sub == j) mine = v;
    }
    if (!(mine > ninf)) id = -1, g = 0.0f;
    float dc = 0.0f;                                           // gradient of the chosen logit by this lane's slot
    float m = 0.0f, inv = 0.0f, dot = 0.0f;
    if (!p.sigmoid) {
        m = mine;
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
            for (int i = 0; i < EPL; ++i) total += z[i] > ninf ? expf(z[i] - m) : 0.0f;
        }
        total = group_sum<LANES>(total);
        inv = total > 0.0f ? 1.0f / total : 0.0f;
        dot = group_sum<LANES>(e * inv * g);
        dc = p.renorm ? e * inv * (g - dot) : e * inv * g;
    } else if (p.renorm) {
        // shares in 64 bits, as the forward takes them
        const double v = id >= 0 ? sigmoid64(mine) : 0.0;
        const double total = group_sum<LANES>(v);
        const double share = total > 0.0 ? v / total : 0.0;
        const double mean = group_sum<LANES>(share * g);
        // v (1 - v) / total = share (1 - v)
        dc = id >= 0 ? (float)(share * sigmoid64(-mine) * (g - mean)) : 0.0f;
    } else if (id >= 0) {
        const float q = expf(-__builtin_fabsf(mine));
        dc = g * (q / ((1.0f + q) * (1.0f + q)));
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        d[i] = (!p.sigmoid && !p.renorm && z[i] > ninf) ? -expf(z[i] - m) * inv * dot : 0.0f;
    for (int j = 0; j < p.k; ++j) {
        const int src = ((threadIdx.x & 63) & ~(LANES - 1)) + j;
        const int e = __shfl(id, src, 64);
        const float v = __shfl(dc, src, 64);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (e == e0 + i) d[i] += v;
    }
    const bool vec = (p.E & 3) == 0;
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int i = 0; i < EPL; i += 4) {
        const int e = e0 + i;
        if (vec) {
            if (e < p.E) {
                if (p.bf16)
                    *(bf16x4 *)((__bf16 *)p.dlogits + t * p.E + e) =
                        bf16x4{(__bf16)d[i], (__bf16)d[i + 1], (__bf16)d[i + 2], (__bf16)d[i + 3]};
                else
                    *(floatx4 *)((float *)p.dlogits + t * p.E + e) = floatx4{d[i], d[i + 1], d[i + 2], d[i + 3]};
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (e + j < p.E) {
                    if (p.bf16) ((__bf16 *)p.dlogits)[t * p.E + e + j] = (__bf16)d[i + j];
                    else ((float *)p.dlogits)[t * p.E + e + j] = d[i + j];
                }
        }
    }
}

// Lanes per token: four experts a lane, at least as many lanes as slots.
template <class Run>
hipError_t by_width(int E, int k, Run run)
{
    if (E <= 32 && k <= 8) run.template operator()<8, 4>();
    else if (E <= 64) run.template operator()<16, 4>();
    else if (E <= 128) run.template operator()<32, 4>();
    else if (E <= 256) run.template operator()<64, 4>();
    else if (E <= 512) run.template operator()<64, 8>();
    else run.template operator()<64, 16>();
    return hipGetLastError();
}

struct RunRoute {
    const RouteParams &p;
    int parts, chunks;
    RoutePlan plan;
    hipStream_t s;
    template <int LANES, int EPL>
    void operator()() const
    {
        if (p.T <= kRouteChunk)
            hipLaunchKernelGGL((route_kernel<LANES, EPL, true>), dim3(1), dim3(kRouteThreads), 0, s, p, 1,
                               plan);
        else
            hipLaunchKernelGGL((route_kernel<LANES, EPL, false>), dim3((unsigned)parts), dim3(kRouteThreads), 0, s, p,
                               chunks, plan);
    }
};

struct RunRouteBwd {
    const RouteBwdParams &p;
    hipStream_t s;
    template <int LANES, int EPL>
    void operator()() const
    {
        constexpr int PER = kThreads / LANES;
        hipLaunchKernelGGL((route_bwd_kernel<LANES, EPL>), dim3((unsigned)((p.T + PER - 1) / PER)), dim3(kThreads), 0,
                           s, p);
    }
};

int64_t chunks_per_part(int64_t T)
{
    const int64_t chunks = (T + kRouteChunk - 1) / kRouteChunk;
    return (chunks + kRouteMaxParts - 1) / kRouteMaxParts;
}

}  // namespace

int route_parts(int64_t T)
{
    const int64_t per = chunks_per_part(T) * kRouteChunk;
    return T > 0 ? (int)((T + per - 1) / per) : 0;
}

hipError_t launch_moe_route(const RouteParams &p, hipStream_t s)
{
    const int parts = route_parts(p.T), chunks = (int)chunks_per_part(p.T);
    hipError_t e = by_width(p.E, p.k, RunRoute{p, parts, chunks, RoutePlan{nullptr, 1}, s});
    if (e == hipSuccess && p.T > kRouteChunk) {
        hipLaunchKernelGGL(route_rows_kernel, dim3((unsigned)parts), dim3(kRouteThreads), 0, s, p, parts, chunks);
        e = hipGetLastError();
    }
    return e;
}

hipError_t launch_moe_route_plan(const RouteParams &p, const RoutePlan &plan, hipStream_t s)
{
    return by_width(p.E, p.k, RunRoute{p, 1, 1, plan, s});
}

hipError_t launch_moe_route_bwd(const RouteBwdParams &p, hipStream_t s)
{
    return by_width(p.E, p.k, RunRouteBwd{p, s});
}

}  // namespace ptgg
