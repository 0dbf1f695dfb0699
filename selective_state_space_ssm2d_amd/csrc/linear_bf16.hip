// libssm2d: matrix products of bf16 tensors.
#include "linear.h"

namespace ssm2d_impl {
namespace gemm {

template <>
int run_gemm<uint16_t>(GemmParams p, const GemmPlan &g, bool a_kc, bool b_kc, void *ws, hipStream_t s)
{
    return run_gemm_of<uint16_t>(p, g, a_kc, b_kc, ws, s);
}

}  // namespace gemm
}  // namespace ssm2d_impl
