// entropy_f16.hip - the kernels of entropy.h for float16 operands.
#include "entropy.h"

namespace kx {

template <>
hipError_t launch_entropy_t<f16>(const EntropyProblem &pr, bool dz, hipStream_t s) {
    return pick_entropy<f16>(pr, dz, s);
}
template <>
hipError_t launch_entropy_dx_t<f16>(const EntropyGrad &e, hipStream_t s) {
    return pick_dx<f16>(e, s);
}
template <>
hipError_t launch_entropy_dw_t<f16>(const EntropyGrad &e, hipStream_t s) {
    return pick_dw<f16>(e, s);
}
template <>
hipError_t launch_entropy_both_t<f16>(const EntropyGrad &e, hipStream_t s) {
    return pick_entropy_both<f16>(e, s);
}

}  // namespace kx
