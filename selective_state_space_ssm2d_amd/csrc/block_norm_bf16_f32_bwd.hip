// libssm2d: the block norm, backward, bf16 with a residual in float32.
#include "block_norm.h"

namespace ssm2d_impl {
namespace norm {

template int launch_norm<uint16_t, float, true>(NormParams, float *, float *, float *, hipStream_t);

}  // namespace norm
}  // namespace ssm2d_impl
