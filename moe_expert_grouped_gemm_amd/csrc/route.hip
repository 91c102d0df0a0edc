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

// Threads of a chunk's workgroup: as many as the registers of a lane's experts
// allow, since 64 tokens of 16 lanes and more take several turns.
__host__ __device__ constexpr int chunk_threads(int epl) { return epl <= 8 ? 1024 : 512; }

// A chunk's tokens: their experts and weights to memory, the experts also to
// s_ids and, as bit t of s_mask[expert], the tokens.  s_mask is zero before.
// Returns whether this thread saw a NaN.
template <int LANES, int EPL, int NT>
__device__ __forceinline__ bool choose_chunk(const RouteParams &p, int64_t t0, int n, uint64_t *s_mask, int *s_ids)
{
    const int tid = threadIdx.x, sub = tid & (LANES - 1);
    bool any_nan = false;
    float next[EPL], bias[EPL] = {};
    if (p.bias && tid / LANES < n) {
        load_logits<EPL>(p.bias, 0, 0, p.E, sub * EPL, bias);  // a row like any other, but its end is 0
#pragma unroll
        for (int j = 0; j < EPL; ++j) bias[j] = sub * EPL + j < p.E ? bias[j] : 0.0f;
    }
    if (tid / LANES < n) load_logits<EPL>(p.logits, p.bf16, t0 + tid / LANES, p.E, sub * EPL, next);
    for (int i = tid / LANES; i < n; i += NT / LANES) {       // a whole group of lanes per token
        float z[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) z[j] = next[j];
        if (i + NT / LANES < n) load_logits<EPL>(p.logits, p.bf16, t0 + i + NT / LANES, p.E, sub * EPL, next);
        int id;
        float w;
        bool nan;
        choose<LANES, EPL>(p, t0 + i, z, bias, id, w, nan);
        any_nan |= nan;
        if (sub < p.k) {
            p.topk_ids[(t0 + i) * p.k + sub] = id;
            p.topk_weights[(t0 + i) * p.k + sub] = w;
            s_ids[i * p.k + sub] = id;
            if (id >= 0) atomicOr((unsigned long long *)&s_mask[id], 1ull << i);
        }
    }
    return any_nan;
}

// Exclusive prefix over the workgroup of one value a thread; s_wave: a word per
// wave.  The caller's barriers separate two calls.
template <int NT>
__device__ __forceinline__ int scan_threads(int v, int *s_wave, int *total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int x = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int y = __shfl_up(x, d, 64);
        if (lane >= d) x += y;
    }
    if (lane == 63) s_wave[wave] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
        const int s = s_wave[w];
        before += w < wave ? s : 0;
        all += s;
    }
    *total = all;
    return before + x - v;
}

// At most 64 tokens: one workgroup chooses, counts and orders.
template <int LANES, int EPL>
__global__ __launch_bounds__(chunk_threads(EPL)) void route_one_kernel(RouteParams p, RoutePlan plan)
{
    constexpr int NT = chunk_threads(EPL), PER = kRouteMaxExperts / NT;
    __shared__ uint64_t s_mask[kRouteMaxExperts];
    __shared__ int s_first[kRouteMaxExperts];      // each expert's first row
    __shared__ int s_ids[kRouteChunk * kRouteMaxTopk];
    __shared__ int s_wave[NT / 64];
    const int tid = threadIdx.x;
    for (int e = tid; e < p.E; e += NT) s_mask[e] = 0;
    __syncthreads();
    if (choose_chunk<LANES, EPL, NT>(p, 0, (int)p.T, s_mask, s_ids) && p.err) atomicOr(p.err, kErrNanLogit);
    __syncthreads();
    // rows in the low half of a word, the plan's blocks in the high one: at most 1024 of either
    int count[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = tid * PER + i, c = e < p.E ? __builtin_popcountll(s_mask[e]) : 0;
        count[i] = c | (plan.plan ? (c + plan.cap - 1) / plan.cap << 16 : 0);
        sum += count[i];
    }
    int total;
    int at = scan_threads<NT>(sum, s_wave, &total);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = tid * PER + i;
        if (e < p.E) {
            const int first = at & 0xFFFF, end = first + (count[i] & 0xFFFF);
            s_first[e] = first;
            p.lens[e] = end - first;
            if (plan.plan) {
                FewBlock *b = (FewBlock *)(plan.plan + 4) + (at >> 16);
                uint64_t left = s_mask[e];
                for (int r = first; r < end; r += plan.cap, ++b) {
                    const int n = min(plan.cap, end - r);
                    FewBlock v = {e, r, n, (uint16_t)(at >> 16), (uint16_t)(count[i] >> 16), {}};
#pragma unroll
                    for (int t = 0; t < 16; ++t)
                        if (t < n) {
                            v.token[t] = (uint8_t)__builtin_ctzll(left);
                            left &= left - 1;
                        }
                    *b = v;
                }
            }
        }
        at += count[i];
    }
    if (plan.plan && tid == 0) plan.plan[0] = total >> 16;
    __syncthreads();
    const int pairs = (int)p.T * p.k;
    for (int i = tid; i < pairs; i += NT) {
        const int id = s_ids[i], t = i / p.k;
        int row = -1;
        if (id >= 0) {
            row = s_first[id] + __builtin_popcountll(s_mask[id] & ((1ull << t) - 1));
            p.token_of[row] = t;
        }
        p.row_of[i] = row;
        if (i >= (total & 0xFFFF)) p.token_of[i] = -1;
    }
}

// One part of many tokens: chunks of 64 in a row.  row_of receives the ranks
// within the part, counts its totals.
template <int LANES, int EPL>
__global__ __launch_bounds__(chunk_threads(EPL)) void route_kernel(RouteParams p, int chunks_per_part)
{
    constexpr int NT = chunk_threads(EPL);
    __shared__ uint64_t s_mask[kRouteMaxExperts];
    __shared__ int s_count[kRouteMaxExperts];      // tokens of earlier chunks
    __shared__ int s_ids[kRouteChunk * kRouteMaxTopk];
    const int tid = threadIdx.x;
    const int64_t t_first = (int64_t)blockIdx.x * chunks_per_part * kRouteChunk;
    const int64_t t_last = min(p.T, t_first + (int64_t)chunks_per_part * kRouteChunk);
    for (int e = tid; e < p.E; e += NT) s_count[e] = 0, s_mask[e] = 0;
    __syncthreads();
    bool any_nan = false;
    for (int64_t t0 = t_first; t0 < t_last; t0 += kRouteChunk) {
        const int n = (int)min((int64_t)kRouteChunk, t_last - t0);
        any_nan |= choose_chunk<LANES, EPL, NT>(p, t0, n, s_mask, s_ids);
        __syncthreads();
        for (int i = tid; i < n * p.k; i += NT) {
            const int id = s_ids[i], t = i / p.k;
            p.row_of[t0 * p.k + i] =
                id < 0 ? -1 : s_count[id] + __builtin_popcountll(s_mask[id] & ((1ull << t) - 1));
        }
        __syncthreads();
        for (int e = tid; e < p.E; e += NT) {
            s_count[e] += __builtin_popcountll(s_mask[e]);
            s_mask[e] = 0;
        }
        __syncthreads();
    }
    if (any_nan && p.err) atomicOr(p.err, kErrNanLogit);
    const int pitch = route_pitch(p.E);
    for (int e = tid; e < pitch; e += NT)
        p.counts[(int64_t)blockIdx.x * pitch + e] = e < p.E ? (uint16_t)s_count[e] : (uint16_t)0;
}

// Second kernel of several parts: the part's first row of each expert is the
// rows of earlier experts plus those of earlier parts.  Every workgroup reads
// all counts, 8 experts of a part a load: thread t takes column t / side of
// them and parts t % side, t % side + side, ....
__global__ __launch_bounds__(kRouteThreads) void route_rows_kernel(RouteParams p, int parts, int chunks_per_part)
{
    __shared__ int s_before[kRouteMaxExperts], s_total[kRouteMaxExperts];
    __shared__ int s_wave[kRouteThreads / 64];
    const int tid = threadIdx.x, part = blockIdx.x;
    const int pitch = route_pitch(p.E), columns = pitch / 8;
    const int64_t i0 = (int64_t)part * chunks_per_part * kRouteChunk * p.k;
    const int64_t i1 = min(p.T * p.k, i0 + (int64_t)chunks_per_part * kRouteChunk * p.k);
    // this thread's first pair is on its way meanwhile
    const int64_t mine = min(i0 + tid, i1 - 1);
    const int first_id = p.topk_ids[mine], first_rank = p.row_of[mine];
    for (int e = tid; e < p.E; e += kRouteThreads) s_before[e] = s_total[e] = 0;
    __syncthreads();
    // a power of two, so that a column's threads are lanes of one wave or whole waves
    const int side = 1 << (31 - __builtin_clz(kRouteThreads / columns));
    const int column = tid / side, lanes = min(side, 64);
    uint32_t before[8] = {}, total8[8] = {};
    if (column < columns) {
#pragma unroll 8
        for (int b = tid % side; b < parts; b += side) {
            const uintx4 v = *(const uintx4 *)(p.counts + (int64_t)b * pitch + column * 8);
            const uint32_t mask = b < part ? ~0u : 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                total8[2 * i] += v[i] & 0xFFFFu;
                total8[2 * i + 1] += v[i] >> 16;
                before[2 * i] += v[i] & 0xFFFFu & mask;
                before[2 * i + 1] += v[i] >> 16 & mask;
            }
        }
    }
    const auto add = [](uint32_t a, uint32_t b) { return a + b; };
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (lanes > 1) before[i] = step_u32<1>(before[i], add), total8[i] = step_u32<1>(total8[i], add);
        if (lanes > 2) before[i] = step_u32<2>(before[i], add), total8[i] = step_u32<2>(total8[i], add);
        if (lanes > 4) before[i] = step_u32<4>(before[i], add), total8[i] = step_u32<4>(total8[i], add);
        if (lanes > 8) before[i] = step_u32<8>(before[i], add), total8[i] = step_u32<8>(total8[i], add);
        if (lanes > 16) before[i] = step_u32<16>(before[i], add), total8[i] = step_u32<16>(total8[i], add);
        if (lanes > 32) before[i] = step_u32<32>(before[i], add), total8[i] = step_u32<32>(total8[i], add);
    }
    if (column < columns && tid % lanes == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (column * 8 + i < p.E) {
                atomicAdd(&s_before[column * 8 + i], (int)before[i]);      // integers: their order does not show
                atomicAdd(&s_total[column * 8 + i], (int)total8[i]);
            }
    }
    __syncthreads();
    constexpr int PER = kRouteMaxExperts / kRouteThreads;
    int count[PER], sum = 0, total;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        count[i] = tid * PER + i < p.E ? s_total[tid * PER + i] : 0;
        sum += count[i];
    }
    int at = scan_threads<kRouteThreads>(sum, s_wave, &total);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = tid * PER + i;
        if (e < p.E) {
            s_before[e] += at;                                 // now the part's first row of the expert
            if (part == 0) p.lens[e] = count[i];
        }
        at += count[i];
    }
    __syncthreads();
    for (int64_t i = i0 + tid; i < i1; i += kRouteThreads) {
        const bool own = i == i0 + tid;
        const int id = own ? first_id : p.topk_ids[i];
        if (id >= 0) {
            const int row = s_before[id] + (own ? first_rank : p.row_of[i]);
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
    // the chosen expert's logit: the row is on its way to this wave already
    float mine = ninf;
    if (id >= 0)
        mine = p.bf16 ? bf16_to_f32(((const uint16_t *)p.logits)[t * p.E + id]) : ((const float *)p.logits)[t * p.E + id];
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
        const double total = slots_sum<LANES>(v);
        const double share = total > 0.0 ? v / total : 0.0;
        const double mean = slots_sum<LANES>(share * g);
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
        const int e = (int)group_lane<LANES>((uint32_t)id, j);
        const float v = bits_f32(group_lane<LANES>(f32_bits(dc), j));
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

// Lanes per token, at least as many as slots.  For few tokens four experts a
// lane: the shortest way through one token.  For many eight: a round of the
// choice costs a wave about as much whether it holds one token or two (5000
// tokens, 128 experts, softmax: 17.5 us with 32 lanes each, 8.0 with 16; 16384 of
// 256, sigmoid: 20.8 with 64, 18.1 with 32).
template <class Run>
hipError_t by_width(int64_t T, int E, int k, Run run)
{
    const bool few = T <= 16;
    if (E <= 32 && k <= 8) run.template operator()<8, 4>();
    else if (E <= 64 && (few || k > 8)) run.template operator()<16, 4>();
    else if (E <= 64) run.template operator()<8, 8>();
    else if (E <= 128) few ? run.template operator()<32, 4>() : run.template operator()<16, 8>();
    else if (E <= 256) few ? run.template operator()<64, 4>() : run.template operator()<32, 8>();
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
            hipLaunchKernelGGL((route_one_kernel<LANES, EPL>), dim3(1), dim3(chunk_threads(EPL)), 0, s, p, plan);
        else
            hipLaunchKernelGGL((route_kernel<LANES, EPL>), dim3((unsigned)parts), dim3(chunk_threads(EPL)), 0, s, p,
                               chunks);
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
    hipError_t e = by_width(p.T, p.E, p.k, RunRoute{p, parts, chunks, RoutePlan{nullptr, 1}, s});
    if (e == hipSuccess && p.T > kRouteChunk) {
        hipLaunchKernelGGL(route_rows_kernel, dim3((unsigned)parts), dim3(kRouteThreads), 0, s, p, parts, chunks);
        e = hipGetLastError();
    }
    return e;
}

hipError_t launch_moe_route_plan(const RouteParams &p, const RoutePlan &plan, hipStream_t s)
{
    return by_width(p.T, p.E, p.k, RunRoute{p, 1, 1, plan, s});
}

hipError_t launch_moe_route_bwd(const RouteBwdParams &p, hipStream_t s)
{
    return by_width(0, p.E, p.k, RunRouteBwd{p, s});      // its loads and stores want whole lines of a token
}

}  // namespace ptgg
