// linear_f16.hip - the tiled products of linear.h for f16 operands, which the
// caller has laid on 16-byte boundaries.
#include "linear.h"

namespace kx {

template <>
hipError_t launch_rows_t<f16>(const RowsProblem &pr, hipStream_t s) {
    return pr.p_rows ? pick_rows<f16, true, 16>(pr, s) : pick_rows<f16, false, 16>(pr, s);
}
template <>
hipError_t launch_grad_t<f16>(const GradProblem &pr, hipStream_t s) {
    return pick_grad<f16, 16>(pr, s);
}

}  // namespace kx
