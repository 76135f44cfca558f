// linear_f32.hip - the products of linear.h for float32 operands.
#include "linear.h"

namespace kx {

template <>
hipError_t launch_rows_t<float>(const RowsProblem &pr, hipStream_t s) {
    return pr.p_rows ? pick_rows<float, true>(pr, s) : pick_rows<float, false>(pr, s);
}
template <>
hipError_t launch_thin_t<float>(const RowsProblem &pr, hipStream_t s) {
    return pick_thin<float>(pr, s);
}
template <>
hipError_t launch_grad_t<float>(const GradProblem &pr, hipStream_t s) {
    return pick_grad<float>(pr, s);
}
template <>
hipError_t launch_both_t<float>(const RowsProblem &r, const GradProblem &g, const SlopeSum &sum,
                                hipStream_t s) {
    return pick_both<float>(r, g, sum, s);
}

}  // namespace kx
