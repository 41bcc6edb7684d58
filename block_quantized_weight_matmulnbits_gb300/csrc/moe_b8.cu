// mnb_moe with 8-bit codes (kernels in moe.cuh).
#include "moe.cuh"

namespace mnb {
namespace moe {

cudaError_t launch_b8(const Params& gate_up, const Params& down, int act_bf16, cudaStream_t s) {
    return launch_bits<8>(gate_up, down, act_bf16, s);
}

}  // namespace moe
}  // namespace mnb
