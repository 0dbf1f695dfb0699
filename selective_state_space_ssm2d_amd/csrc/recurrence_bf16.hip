// libssm2d: the gated linear recurrence, forward, bf16.
#include "recurrence.h"

namespace ssm2d_impl {

template int rec_run<uint16_t, false>(const RecParams &, const RecPlan &, long, bool, hipStream_t);

}  // namespace ssm2d_impl
