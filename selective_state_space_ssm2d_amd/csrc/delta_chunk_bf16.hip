// libssm2d: the gated delta rule in chunks, bf16 inputs: forward.
#include "delta_chunk.h"

namespace ssm2d_impl {

template <>
int delta_chunk_fwd<uint16_t>(const DeltaArgs &a)
{
    return chunk_kd<uint16_t, false>(a);
}

}  // namespace ssm2d_impl
