// Host build of the router's threshold between certain and possible choices
// (candidate_floor of the library's route_device.hpp).  Compiled by
// tests/test_route_host.py with `hipcc -x hip --offload-host-only`; nothing
// here runs on a GPU.
#include "../../moe_expert_grouped_gemm_amd/csrc/route_device.hpp"

extern "C" float ptgg_host_candidate_floor(float kth) { return ptgg::candidate_floor(kth); }
