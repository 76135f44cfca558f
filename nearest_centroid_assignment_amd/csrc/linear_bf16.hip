// linear_bf16.hip - the products of linear.h for bf16 operands, whose rows the caller has laid on
// 4-byte boundaries (thin products take any).
#include "linear.h"

namespace kx {

template <>
hipError_t launch_rows_t<bf16>(const RowsProblem &pr, hipStream_t s) {
    return pr.p_rows ? pick_rows<bf16, true>(pr, s) : pick_rows<bf16, false>(pr, s);
}
template <>
hipError_t launch_thin_t<bf16>(const RowsProblem &pr, hipStream_t s) {
    return pick_thin<bf16>(pr, s);
}
template <>
hipError_t launch_grad_t<bf16>(const GradProblem &pr, hipStream_t s) {
    return pick_grad<bf16>(pr, s);
}
template <>
hipError_t launch_both_t<bf16>(const RowsProblem &r, const GradProblem &g, const SlopeSum &sum,
                               hipStream_t s) {
    return pick_both<bf16>(r, g, sum, s);
}

}  // namespace kx
