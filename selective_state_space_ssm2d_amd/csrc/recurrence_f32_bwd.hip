// libssm2d: the gated linear recurrence, backward, float32.
#include "recurrence.h"

namespace ssm2d_impl {

template int rec_run<float, true>(const RecParams &, const RecPlan &, long, bool, hipStream_t);

}  // namespace ssm2d_impl
