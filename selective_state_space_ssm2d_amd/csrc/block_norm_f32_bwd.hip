// libssm2d: the block norm, backward, float32.
#include "block_norm.h"

namespace ssm2d_impl {
namespace norm {

template int launch_norm<float, float, true>(NormParams, float *, float *, float *, hipStream_t);

}  // namespace norm
}  // namespace ssm2d_impl
