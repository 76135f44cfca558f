// linear_f16.hip - the products of linear.h for f16 operands, whose rows the caller has laid on
// 4-byte boundaries (thin products take any).
#include "linear.h"

namespace kx {

template <>
hipError_t launch_rows_t<f16>(const RowsProblem &pr, hipStream_t s) {
    return pr.p_rows ? pick_rows<f16, true>(pr, s) : pick_rows<f16, false>(pr, s);
}
template <>
hipError_t launch_thin_t<f16>(const RowsProblem &pr, hipStream_t s) {
    return pick_thin<f16>(pr, s);
}
template <>
hipError_t launch_grad_t<f16>(const GradProblem &pr, hipStream_t s) {
    return pick_grad<f16>(pr, s);
}
template <>
hipError_t launch_both_t<f16>(const RowsProblem &r, const GradProblem &g, const SlopeSum &sum,
                              hipStream_t s) {
    return pick_both<f16>(r, g, sum, s);
}

}  // namespace kx
