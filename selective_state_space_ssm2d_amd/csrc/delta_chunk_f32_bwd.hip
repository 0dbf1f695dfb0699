// libssm2d: the gated delta rule in chunks, fp32 inputs: backward.
#include "delta_chunk.h"

namespace ssm2d_impl {

template <>
int delta_chunk_bwd<float>(const DeltaArgs &a)
{
    return chunk_kd<float, true>(a);
}

}  // namespace ssm2d_impl
