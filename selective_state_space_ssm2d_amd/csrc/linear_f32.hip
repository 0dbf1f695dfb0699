// libssm2d: matrix products of float32 tensors.
#include "linear.h"

namespace ssm2d_impl {
namespace gemm {

SSM2D_DEFINE_RUN_GEMM(float)

}  // namespace gemm
}  // namespace ssm2d_impl
