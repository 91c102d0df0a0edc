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
// What bounds it: launch and wave-reduction latency -- a token's choice is a
// thousand vector instructions of a wave, so it is spread over the CUs; the
// logits of 16384 tokens on 256 experts in fp32 are 16 MB.
#include "route_device.hpp"

namespace ptgg {

namespace {

constexpr int kRouteThreads = 512;
constexpr int kOrderThreads = 1024;       // a pair each

// Threads of a chunk's workgroup: as many as the registers of a lane's experts
// allow, since 64 tokens of 16 lanes and more take several turns.
__host__ __device__ constexpr int chunk_threads(int epl) { return epl <= 8 ? 1024 : 512; }

// The bias of experts e0 .. e0 + EPL - 1: a row like any other, but its end is 0.
template <int EPL>
__device__ __forceinline__ void load_bias(const RouteParams &p, int e0, float (&bias)[EPL])
{
    load_logits<EPL>(p.bias, 0, 0, p.E, e0, bias);
#pragma unroll
    for (int j = 0; j < EPL; ++j) bias[j] = e0 + j < p.E ? bias[j] : 0.0f;
}

// A chunk's tokens: their experts and weights to memory, the experts also to
// s_ids and, as bit t of s_mask[expert], the tokens.  s_mask is zero before.
// Returns whether this thread saw a NaN.
template <int LANES, int EPL, int NT>
__device__ __forceinline__ bool choose_chunk(const RouteParams &p, int64_t t0, int n, uint64_t *s_mask, int *s_ids)
{
    const int tid = threadIdx.x, sub = tid & (LANES - 1);
    bool any_nan = false;
    float next[EPL], bias[EPL] = {};
    if (p.bias && tid / LANES < n) load_bias<EPL>(p, sub * EPL, bias);
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

// Counts, orders and plans what at most 64 tokens chose, in one workgroup.  Of
// their choices s_ids has the experts and s_mask, as bit t of s_mask[expert], the
// tokens.
template <int NT>
__device__ __forceinline__ void order_chunk(const RouteParams &p, const RoutePlan &plan, const uint64_t *s_mask,
                                            const int *s_ids, int *s_first, int *s_wave)
{
    constexpr int PER = kRouteMaxExperts / NT;
    const int tid = threadIdx.x;
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

// At most 64 tokens: one workgroup chooses, counts and orders.
template <int LANES, int EPL>
__global__ __launch_bounds__(chunk_threads(EPL)) void route_one_kernel(RouteParams p, RoutePlan plan)
{
    constexpr int NT = chunk_threads(EPL);
    __shared__ uint64_t s_mask[kRouteMaxExperts];
    __shared__ int s_first[kRouteMaxExperts];      // each expert's first row
    __shared__ int s_ids[kRouteChunk * kRouteMaxTopk];
    __shared__ int s_wave[NT / 64];
    const int tid = threadIdx.x;
    for (int e = tid; e < p.E; e += NT) s_mask[e] = 0;
    __syncthreads();
    if (choose_chunk<LANES, EPL, NT>(p, 0, (int)p.T, s_mask, s_ids) && p.err) atomicOr(p.err, kErrNanLogit);
    __syncthreads();
    order_chunk<NT>(p, plan, s_mask, s_ids, s_first, s_wave);
}

// The same where one workgroup would take long over the choice: that by a
// workgroup for every few tokens, then the order by one.
template <int LANES, int EPL>
__global__ __launch_bounds__(kThreads) void route_choose_kernel(RouteParams p)
{
    const int sub = threadIdx.x & (LANES - 1);
    const int64_t t = (int64_t)blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
    if (t >= p.T) return;                                      // whole groups
    float z[EPL], bias[EPL] = {};
    load_logits<EPL>(p.logits, p.bf16, t, p.E, sub * EPL, z);
    if (p.bias) load_bias<EPL>(p, sub * EPL, bias);
    int id;
    float w;
    bool nan;
    choose<LANES, EPL>(p, t, z, bias, id, w, nan);
    if (nan && p.err) atomicOr(p.err, kErrNanLogit);
    if (sub < p.k) {
        p.topk_ids[t * p.k + sub] = id;
        p.topk_weights[t * p.k + sub] = w;
    }
}

__global__ __launch_bounds__(kOrderThreads) void route_order_kernel(RouteParams p, RoutePlan plan)
{
    __shared__ uint64_t s_mask[kRouteMaxExperts];
    __shared__ int s_first[kRouteMaxExperts], s_ids[kRouteChunk * kRouteMaxTopk], s_wave[kOrderThreads / 64];
    const int tid = threadIdx.x, pairs = (int)p.T * p.k;
    const int id = tid < pairs ? p.topk_ids[tid] : -1;         // 1024 pairs at most
    for (int e = tid; e < p.E; e += kOrderThreads) s_mask[e] = 0;
    __syncthreads();
    if (tid < pairs) s_ids[tid] = id;
    if (id >= 0) atomicOr((unsigned long long *)&s_mask[id], 1ull << (tid / p.k));
    __syncthreads();
    order_chunk<kOrderThreads>(p, plan, s_mask, s_ids, s_first, s_wave);
}

// One part of many tokens: chunks of 64 in a row.  row_of receives the ranks
// within the part, counts its totals.
template <int LANES, int EPL>
__global__ __launch_bounds__(chunk_threads(EPL)) void route_kernel(RouteParams p, int part_tokens)
{
    constexpr int NT = chunk_threads(EPL);
    __shared__ uint64_t s_mask[kRouteMaxExperts];
    __shared__ int s_count[kRouteMaxExperts];      // tokens of earlier chunks
    __shared__ int s_ids[kRouteChunk * kRouteMaxTopk];
    const int tid = threadIdx.x;
    const int64_t t_first = (int64_t)blockIdx.x * part_tokens;
    const int64_t t_last = min(p.T, t_first + part_tokens);
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
__global__ __launch_bounds__(kRouteThreads) void route_rows_kernel(RouteParams p, int parts, int part_tokens)
{
    __shared__ int s_before[kRouteMaxExperts], s_total[kRouteMaxExperts];
    __shared__ int s_wave[kRouteThreads / 64];
    const int tid = threadIdx.x, part = blockIdx.x;
    const int pitch = route_pitch(p.E), columns = pitch / 8;
    const int64_t i0 = (int64_t)part * part_tokens * p.k;
    const int64_t i1 = min(p.T * p.k, i0 + (int64_t)part_tokens * p.k);
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

// Whether at most 64 tokens' experts are chosen by several workgroups before one orders them, which costs 0.9 us and
// saves the time of a CU's share: 64 tokens, sigmoid, 8 of 60: 7.3 us alone, 8.0 with several; of 128: 10.0, 7.7; of 256:
// 17.6, 7.6; of 1024: 52.6, 10.4; 16 tokens, 8 of 128: 6.5, 7.4; of 256: 8.3, 7.3.
bool two_kernels(int64_t T, int E) { return T > 8 && T * E > 4096; }

// Lanes per token, at least as many as slots.  Where tokens are few for the CUs at work, four experts a lane: the
// shortest way through one token.  Otherwise eight: a round of the choice costs a wave about as much whether it holds
// one token or two (5000 tokens, 128 experts, softmax: 17.5 us with 32 lanes each, 8.0 with 16; 16384 of 256, sigmoid:
// 20.8 with 64, 18.1 with 32).
bool few_lanes(const RouteParams &p) { return p.T <= 16 || (p.T <= kRouteChunk && two_kernels(p.T, p.E)); }
template <class Run>
hipError_t by_width(bool few, int E, int k, Run run)
{
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
    int parts, part_tokens;
    RoutePlan plan;
    hipStream_t s;
    template <int LANES, int EPL>
    void operator()() const
    {
        constexpr int PER = kThreads / LANES;
        if (p.T > kRouteChunk) {
            hipLaunchKernelGGL((route_kernel<LANES, EPL>), dim3((unsigned)parts), dim3(chunk_threads(EPL)), 0, s, p,
                               part_tokens);
        } else if (!two_kernels(p.T, p.E)) {
            hipLaunchKernelGGL((route_one_kernel<LANES, EPL>), dim3(1), dim3(chunk_threads(EPL)), 0, s, p, plan);
        } else {
            hipLaunchKernelGGL((route_choose_kernel<LANES, EPL>), dim3((unsigned)((p.T + PER - 1) / PER)), dim3(kThreads),
                               0, s, p);
            hipLaunchKernelGGL(route_order_kernel, dim3(1), dim3(kOrderThreads), 0, s, p, plan);
        }
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

// Tokens of a part: few keep the choice short, but every part reads all parts' counts (8 of 256, sigmoid, with 64, 32
// and 16 to a part: 1040 tokens 22.6 us, 16.0 and 13.6; 4100 tokens 26.6, 19.0 and 20.5).
int part_tokens_of(int64_t T)
{
    const int64_t per = (T + kRouteMaxParts - 1) / kRouteMaxParts;
    if (per > kRouteChunk) return (int)((per + kRouteChunk - 1) / kRouteChunk) * kRouteChunk;
    return T <= 160 * 16 ? 16 : T <= 160 * 32 ? 32 : kRouteChunk;
}

}  // namespace

int route_parts(int64_t T) { return (int)((T + part_tokens_of(T) - 1) / part_tokens_of(T)); }

hipError_t launch_moe_route(const RouteParams &p, hipStream_t s)
{
    const int parts = route_parts(p.T), part_tokens = part_tokens_of(p.T);
    hipError_t e = by_width(few_lanes(p), p.E, p.k, RunRoute{p, parts, part_tokens, RoutePlan{nullptr, 1}, s});
    if (e == hipSuccess && p.T > kRouteChunk) {
        hipLaunchKernelGGL(route_rows_kernel, dim3((unsigned)parts), dim3(kRouteThreads), 0, s, p, parts, part_tokens);
        e = hipGetLastError();
    }
    return e;
}

hipError_t launch_moe_route_plan(const RouteParams &p, const RoutePlan &plan, hipStream_t s)
{
    return by_width(few_lanes(p), p.E, p.k, RunRoute{p, 1, 0, plan, s});
}

hipError_t launch_moe_route_bwd(const RouteBwdParams &p, hipStream_t s)
{
    return by_width(true, p.E, p.k, RunRouteBwd{p, s});   // its loads and stores want whole lines of a token
}

}  // namespace ptgg
