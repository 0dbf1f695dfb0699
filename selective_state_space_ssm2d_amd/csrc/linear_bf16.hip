// libssm2d: matrix products of bf16 tensors.
#include "linear.h"

namespace ssm2d_impl {
namespace gemm {

SSM2D_DEFINE_RUN_GEMM(uint16_t)

}  // namespace gemm
}  // namespace ssm2d_impl
