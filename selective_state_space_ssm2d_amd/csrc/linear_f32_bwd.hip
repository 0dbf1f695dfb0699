// libssm2d: both gradients of projections of float32 tensors in one launch.
#include "linear.h"

namespace ssm2d_impl {
namespace gemm {

template <>
int run_pair<float>(GemmParams dx, const GemmPlan &gx, GemmParams dw, const GemmPlan &gw, bool x_maps, bool y_maps, void *ws, hipStream_t s)
{
    return run_pair_of<float>(dx, gx, dw, gw, x_maps, y_maps, ws, s);
}

}  // namespace gemm
}  // namespace ssm2d_impl
