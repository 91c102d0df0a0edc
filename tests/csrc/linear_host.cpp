// Host build of the dense product's planner (plan_linear of the library's
// linear_plan.hpp).  Compiled by tests/test_linear_plan.py with `hipcc -x hip
// --offload-host-only`; nothing here runs on a GPU.
#include "../../moe_expert_grouped_gemm_amd/csrc/linear_plan.hpp"

// op 0, 1, 2: forward, dgrad, wgrad; rows, columns and reduction of the product
// that it computes.
extern "C" void ptgg_host_linear_plan(int op, int64_t M, int64_t N, int64_t K, int64_t out[11])
{
    const ptgg::LinearPlan p = ptgg::plan_linear(op, M, N, K);
    const ptgg::WideCut &c = p.cut;
    const int64_t v[11] = {p.tile, p.splits, p.part, c.whole, c.rest, c.parts, c.tails, c.cuts, c.main, c.cut, p.partial_bytes};
    for (int i = 0; i < 11; ++i) out[i] = v[i];
}
