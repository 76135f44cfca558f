// linear_f32.hip - the tiled products of linear.h for float32 operands. Rows on
// 16-byte boundaries move 16 bytes a lane into LDS, any others 4: the float32
// matrix instructions take 16 times as long per byte as the 16-bit ones and
// hide the four times as many moves.
#include "linear.h"

namespace kx {

template <>
hipError_t launch_rows_t<float>(const RowsProblem &pr, hipStream_t s) {
    const bool wide = on_chunk(pr.q, pr.ldq, pr.depth, 4) &&
                      on_chunk(pr.p, pr.ldp, pr.p_rows ? pr.p_cols : pr.depth, 4);
    if (pr.p_rows) return wide ? pick_rows<float, true, 16>(pr, s) : pick_rows<float, true, 4>(pr, s);
    return wide ? pick_rows<float, false, 16>(pr, s) : pick_rows<float, false, 4>(pr, s);
}
template <>
hipError_t launch_grad_t<float>(const GradProblem &pr, hipStream_t s) {
    const bool wide = on_chunk(pr.x, pr.ldx, pr.x_cols, 4) && on_chunk(pr.dz, pr.lddz, pr.dz_cols, 4);
    return wide ? pick_grad<float, 16>(pr, s) : pick_grad<float, 4>(pr, s);
}

}  // namespace kx
