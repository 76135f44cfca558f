// entropy_f32.hip - the kernels of entropy.h for float32 operands.
#include "entropy.h"

namespace kx {

template <>
hipError_t launch_entropy_t<float>(const EntropyProblem &pr, bool dz, hipStream_t s) {
    return pick_entropy<float>(pr, dz, s);
}
template <>
hipError_t launch_entropy_dx_t<float>(const EntropyGrad &e, hipStream_t s) {
    return pick_dx<float>(e, s);
}
template <>
hipError_t launch_entropy_dw_t<float>(const EntropyGrad &e, hipStream_t s) {
    return pick_dw<float>(e, s);
}
template <>
hipError_t launch_entropy_both_t<float>(const EntropyGrad &e, hipStream_t s) {
    return pick_entropy_both<float>(e, s);
}

}  // namespace kx
