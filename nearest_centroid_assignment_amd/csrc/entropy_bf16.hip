// entropy_bf16.hip - the kernels of entropy.h for bfloat16 operands.
#include "entropy.h"

namespace kx {

template <>
hipError_t launch_entropy_t<bf16>(const EntropyProblem &pr, bool dz, hipStream_t s) {
    return pick_entropy<bf16>(pr, dz, s);
}
template <>
hipError_t launch_entropy_dx_t<bf16>(const EntropyGrad &e, hipStream_t s) {
    return pick_dx<bf16>(e, s);
}
template <>
hipError_t launch_entropy_dw_t<bf16>(const EntropyGrad &e, hipStream_t s) {
    return pick_dw<bf16>(e, s);
}
template <>
hipError_t launch_entropy_both_t<bf16>(const EntropyGrad &e, hipStream_t s) {
    return pick_entropy_both<bf16>(e, s);
}

}  // namespace kx
