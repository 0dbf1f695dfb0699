// libssm2d: matrix products of float32 tensors.
#include "linear.h"

namespace ssm2d_impl {
namespace gemm {

template <>
int run_gemm<float>(GemmParams p, const GemmPlan &g, bool a_kc, bool b_kc, void *ws, hipStream_t s)
{
    return run_gemm_of<float>(p, g, a_kc, b_kc, ws, s);
}

}  // namespace gemm
}  // namespace ssm2d_impl
