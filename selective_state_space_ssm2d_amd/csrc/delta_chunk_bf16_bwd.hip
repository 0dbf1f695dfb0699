// libssm2d: the gated delta rule in chunks, bf16 inputs: backward.
#include "delta_chunk.h"

namespace ssm2d_impl {

template <>
int delta_chunk_bwd<uint16_t>(const DeltaArgs &a)
{
    return chunk_kd<uint16_t, true>(a);
}

}  // namespace ssm2d_impl
