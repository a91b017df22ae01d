// Split-KV kernels over an 8-bit cache, bf16 q and out.
#include <algorithm>

#include "q8_launch.cuh"

namespace pa {

int launch_q8_bf16(const Args& a, const SplitPlan& plan, void* workspace, unsigned int* err, char* msg, size_t msg_len) {
    return launch_q8_t<__nv_bfloat16>(a, plan, workspace, err, msg, msg_len);
}

int q8_occupancy_bf16(const SplitPlan& plan) { return q8_occupancy_t<__nv_bfloat16>(plan); }

}  // namespace pa
