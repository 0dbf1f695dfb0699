// libssm2d: the gated linear recurrence, forward, float32.
#include "recurrence.h"

namespace ssm2d_impl {

template int rec_run<float, false>(const RecParams &, const RecPlan &, long, bool, hipStream_t);

}  // namespace ssm2d_impl
