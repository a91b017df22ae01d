// Split-KV kernels over an 8-bit cache, f16 q and out.
#include <algorithm>

#include "q8_launch.cuh"

namespace pa {

int launch_q8_f16(const Args& a, const SplitPlan& plan, void* workspace, unsigned int* err, char* msg, size_t msg_len) {
    return launch_q8_t<__half>(a, plan, workspace, err, msg, msg_len);
}

int q8_occupancy_f16(const SplitPlan& plan) { return q8_occupancy_t<__half>(plan); }

}  // namespace pa
