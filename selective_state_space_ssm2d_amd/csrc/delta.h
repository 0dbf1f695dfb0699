// libssm2d: the gated delta rule (include/ssm2d_ops.h has the recurrence):
// what its translation units share on the host.
#pragma once

#include "ops_common.h"

namespace ssm2d_impl {

// One call's tensors and sizes, checked (delta.hip). Element strides.
struct DeltaArgs {
    const void *q, *k, *v, *dout;
    const float *g, *beta, *h_init, *dh_last;
    const int *cu;
    void *o, *dq, *dk, *dv;
    float *h_last, *dg, *dbeta, *dh_init;
    long batch, tokens, n_seq;  // n_seq > 0: packed
    int hk, h, dk_, dv_;
    long qs[3], ks[3], vs[3], os[3], gs[3], bs[3];
    float scale;
    int dev;
    void *stream;
};

// The recurrence token by token (delta_step.hip): state h_init (NULL: zeros)
// to h_last (NULL: dropped; may be h_init).
template <typename T>
int delta_step(const DeltaArgs &a);

// In chunks of 64 tokens (delta_chunk.h).
template <typename T>
int delta_chunk_fwd(const DeltaArgs &a);
template <typename T>
int delta_chunk_bwd(const DeltaArgs &a);
template <>
int delta_chunk_fwd<float>(const DeltaArgs &a);
template <>
int delta_chunk_fwd<uint16_t>(const DeltaArgs &a);
template <>
int delta_chunk_bwd<float>(const DeltaArgs &a);
template <>
int delta_chunk_bwd<uint16_t>(const DeltaArgs &a);

}  // namespace ssm2d_impl
