// libssm2d: the gated delta rule in chunks, fp32 inputs: forward.
#include "delta_chunk.h"

namespace ssm2d_impl {

template <>
int delta_chunk_fwd<float>(const DeltaArgs &a)
{
    return chunk_kd<float, false>(a);
}

}  // namespace ssm2d_impl
