// libssm2d: C entries of the gated delta rule: argument checks and the choice
// of the kernels.
#include "delta.h"

#include <cstring>

namespace ssm2d_impl {
namespace {

// Up to so many tokens the recurrence itself, in one launch and no workspace,
// is faster than the chunks, whose cost does not fall below 64 tokens'. For 8 x
// 8 heads of 128 x 128 it takes 14 us of 8 tokens and 25 of 16 (bf16; fp32 13
// and 23), the chunks 21 (fp32 32); for 64 x 16 of 64 x 64 23 and 42, and 37
// (fp32 69).
template <typename T>
constexpr long kFewTokens = sizeof(T) == 2 ? 8 : 16;

int fill(DeltaArgs *a, const ssm2d_delta_shape *sh, float scale, void *stream, bool *work)
{
    *work = false;
    if (!sh) return SSM2D_ERR_NULLPTR;
    if (sh->batch < 0 || sh->tokens < 0 || sh->n_seq < 0 || sh->heads_qk < 0 || sh->heads < 0 || sh->d_k < 0 || sh->d_v < 0)
        return SSM2D_ERR_BAD_DIM;
    if (sh->n_seq > 0 && sh->batch != 1) return SSM2D_ERR_BAD_DIM;
    if (sh->heads_qk > 0 ? sh->heads % sh->heads_qk != 0 : sh->heads != 0) return SSM2D_ERR_BAD_DIM;
    const int64_t seqs = sh->n_seq > 0 ? sh->n_seq : sh->batch;
    if (sh->d_k > SSM2D_DELTA_MAX_DK || sh->d_v > SSM2D_DELTA_MAX_DV || sh->tokens >= (int64_t{1} << 31) - 64 ||
        sh->heads >= (1 << 15) || seqs >= (1 << 24) || seqs * std::max<int64_t>(sh->heads, 1) >= (1 << 24))
        return SSM2D_ERR_UNSUPPORTED;
    a->batch = sh->batch, a->tokens = sh->tokens, a->n_seq = sh->n_seq;
    a->hk = static_cast<int>(sh->heads_qk), a->h = static_cast<int>(sh->heads);
    a->dk_ = static_cast<int>(sh->d_k), a->dv_ = static_cast<int>(sh->d_v);
    for (int i = 0; i < 3; ++i) {
        a->qs[i] = sh->q_stride[i], a->ks[i] = sh->k_stride[i], a->vs[i] = sh->v_stride[i], a->os[i] = sh->do_stride[i];
        a->gs[i] = sh->g_stride[i], a->bs[i] = sh->beta_stride[i];
    }
    a->scale = scale;
    a->stream = stream;
    *work = seqs > 0 && sh->heads > 0 && sh->d_k > 0 && sh->d_v > 0;  // (without tokens the states still pass on)
    return SSM2D_OK;
}

__global__ void pass_states(const float *in, float *out, long n)
{
    const long step = static_cast<long>(gridDim.x) * blockDim.x;
    for (long i = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += step) out[i] = in ? in[i] : 0.0f;
}

// Workgroups of 256 for n elements (any number beyond these takes more turns).
unsigned blocks_of(long n) { return static_cast<unsigned>(std::min<long>((n + 255) / 256, 1 << 20)); }

int pass_states_on(const DeltaArgs &a, const float *in, float *out)
{
    const long n = (a.n_seq > 0 ? a.n_seq : a.batch) * a.h * a.dk_ * a.dv_;
    if (!out || out == in || n == 0) return SSM2D_OK;
    pass_states<<<dim3(blocks_of(n)), dim3(256), 0, static_cast<hipStream_t>(a.stream)>>>(in, out, n);
    return launched();
}

// Heads without keys or values leave nothing to sum: outputs that are not
// empty themselves are zeros.
template <typename T>
__global__ void fill_zeros(T *out, long n)
{
    const long step = static_cast<long>(gridDim.x) * blockDim.x;
    for (long i = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += step) out[i] = 0;
}

template <typename T>
int zeros(T *out, int64_t rows, int64_t d, void *stream)
{
    if (rows <= 0 || d <= 0) return SSM2D_OK;
    if (rows > (int64_t{1} << 45) / d) return SSM2D_ERR_UNSUPPORTED;  // (far beyond memory; rows are below 2^55)
    if (!out) return SSM2D_ERR_NULLPTR;
    if (off_by(out, sizeof(T))) return SSM2D_ERR_MISALIGNED;
    fill_zeros<<<dim3(blocks_of(rows * d)), dim3(256), 0, static_cast<hipStream_t>(stream)>>>(out, rows * d);
    return launched();
}

template <typename T>
bool misaligned_in(const DeltaArgs &a)
{
    return off_by(a.q, sizeof(T)) || off_by(a.k, sizeof(T)) || off_by(a.v, sizeof(T)) || off_by(a.dout, sizeof(T)) ||
           off_by(a.o, sizeof(T)) || off_by(a.dq, sizeof(T)) || off_by(a.dk, sizeof(T)) || off_by(a.dv, sizeof(T)) || off_by(a.g, 4) ||
           off_by(a.beta, 4) || off_by(a.h_init, 4) || off_by(a.h_last, 4) || off_by(a.dh_last, 4) || off_by(a.dh_init, 4) ||
           off_by(a.dg, 4) || off_by(a.dbeta, 4) || off_by(a.cu, 4);
}

template <typename F>
int run(DeltaArgs &a, F &&f)
{
    return guarded([&]() -> int {
        const hipError_t e = hipGetDevice(&a.dev);
        if (e != hipSuccess) return hip_fail(e);
        std::lock_guard<std::recursive_mutex> lock(g_mutex);
        return f();
    });
}

template <typename T>
int fwd_entry(const T *q, const T *k, const T *v, const float *g, const float *beta, const float *h_init, const int32_t *cu, T *o,
              float *h_last, const ssm2d_delta_shape *sh, float scale, void *stream)
{
    DeltaArgs a{};
    bool work = false;
    const int st = fill(&a, sh, scale, stream, &work);
    if (st != SSM2D_OK) return st;
    if (!work) return sh->d_k == 0 ? zeros(o, a.batch * a.tokens * a.h, a.dv_, stream) : SSM2D_OK;
    a.q = q, a.k = k, a.v = v, a.g = g, a.beta = beta, a.h_init = h_init, a.cu = a.n_seq > 0 ? cu : nullptr, a.o = o, a.h_last = h_last;
    if (a.tokens > 0 && (!q || !k || !v || !g || !beta || !o || (a.n_seq > 0 && !cu))) return SSM2D_ERR_NULLPTR;
    if (misaligned_in<T>(a)) return SSM2D_ERR_MISALIGNED;
    return run(a, [&]() -> int {
        if (a.tokens == 0) return pass_states_on(a, h_init, h_last);
        if (a.n_seq == 0 && a.tokens <= kFewTokens<T>) return delta_step<T>(a);
        return delta_chunk_fwd<T>(a);
    });
}

template <typename T>
int bwd_entry(const T *q, const T *k, const T *v, const float *g, const float *beta, const float *h_init, const int32_t *cu, const T *dout,
              const float *dh_last, T *dq, T *dk, T *dv, float *dg, float *dbeta, float *dh_init, const ssm2d_delta_shape *sh, float scale,
              void *stream)
{
    DeltaArgs a{};
    bool work = false;
    const int st = fill(&a, sh, scale, stream, &work);
    if (st != SSM2D_OK) return st;
    if (!work) {
        const int64_t rows = a.batch * a.tokens;
        int z = SSM2D_OK;
        for (T *out : {dq, dk})
            if (z == SSM2D_OK) z = zeros(out, rows * a.hk, a.dk_, stream);
        if (z == SSM2D_OK) z = zeros(dv, rows * a.h, a.dv_, stream);
        for (float *out : {dg, dbeta})
            if (z == SSM2D_OK) z = zeros(out, rows * a.h, 1, stream);
        return z;
    }
    a.q = q, a.k = k, a.v = v, a.g = g, a.beta = beta, a.h_init = h_init, a.cu = a.n_seq > 0 ? cu : nullptr, a.dout = dout, a.dh_last = dh_last;
    a.dq = dq, a.dk = dk, a.dv = dv, a.dg = dg, a.dbeta = dbeta, a.dh_init = dh_init;
    if (a.tokens > 0 && (!q || !k || !v || !g || !beta || !dout || !dq || !dk || !dv || !dg || !dbeta || (a.n_seq > 0 && !cu)))
        return SSM2D_ERR_NULLPTR;
    if (misaligned_in<T>(a)) return SSM2D_ERR_MISALIGNED;
    return run(a, [&]() -> int {
        if (a.tokens == 0) return pass_states_on(a, dh_last, dh_init);
        return delta_chunk_bwd<T>(a);
    });
}

template <typename T>
int step_entry(const T *q, const T *k, const T *v, const float *g, const float *beta, float *state, T *o, const ssm2d_delta_shape *sh,
               float scale, void *stream)
{
    DeltaArgs a{};
    bool work = false;
    if (sh && sh->n_seq != 0) return SSM2D_ERR_BAD_FLAGS;
    const int st = fill(&a, sh, scale, stream, &work);
    if (st != SSM2D_OK || a.tokens == 0) return st;
    if (!work) return sh->d_k == 0 ? zeros(o, a.batch * a.tokens * a.h, a.dv_, stream) : SSM2D_OK;
    a.q = q, a.k = k, a.v = v, a.g = g, a.beta = beta, a.h_init = state, a.h_last = state, a.o = o;
    if (!q || !k || !v || !g || !beta || !state || !o) return SSM2D_ERR_NULLPTR;
    if (misaligned_in<T>(a)) return SSM2D_ERR_MISALIGNED;
    return run(a, [&] { return delta_step<T>(a); });
}

}  // namespace
}  // namespace ssm2d_impl

extern "C" {

int ssm2d_gated_delta_fwd(const float *q, const float *k, const float *v, const float *g, const float *beta, const float *h_init,
                          const int32_t *cu_seqlens, float *o, float *h_last, const ssm2d_delta_shape *shape, float scale, void *stream)
{
    return ssm2d_impl::fwd_entry<float>(q, k, v, g, beta, h_init, cu_seqlens, o, h_last, shape, scale, stream);
}

int ssm2d_gated_delta_fwd_bf16(const uint16_t *q, const uint16_t *k, const uint16_t *v, const float *g, const float *beta,
                               const float *h_init, const int32_t *cu_seqlens, uint16_t *o, float *h_last,
                               const ssm2d_delta_shape *shape, float scale, void *stream)
{
    return ssm2d_impl::fwd_entry<uint16_t>(q, k, v, g, beta, h_init, cu_seqlens, o, h_last, shape, scale, stream);
}

int ssm2d_gated_delta_bwd(const float *q, const float *k, const float *v, const float *g, const float *beta, const float *h_init,
                          const int32_t *cu_seqlens, const float *dout, const float *dh_last, float *dq, float *dk, float *dv, float *dg,
                          float *dbeta, float *dh_init, const ssm2d_delta_shape *shape, float scale, void *stream)
{
    return ssm2d_impl::bwd_entry<float>(q, k, v, g, beta, h_init, cu_seqlens, dout, dh_last, dq, dk, dv, dg, dbeta, dh_init, shape, scale,
                                        stream);
}

int ssm2d_gated_delta_bwd_bf16(const uint16_t *q, const uint16_t *k, const uint16_t *v, const float *g, const float *beta,
                               const float *h_init, const int32_t *cu_seqlens, const uint16_t *dout, const float *dh_last, uint16_t *dq,
                               uint16_t *dk, uint16_t *dv, float *dg, float *dbeta, float *dh_init, const ssm2d_delta_shape *shape,
                               float scale, void *stream)
{
    return ssm2d_impl::bwd_entry<uint16_t>(q, k, v, g, beta, h_init, cu_seqlens, dout, dh_last, dq, dk, dv, dg, dbeta, dh_init, shape,
                                           scale, stream);
}

int ssm2d_gated_delta_step(const float *q, const float *k, const float *v, const float *g, const float *beta, float *state, float *o,
                           const ssm2d_delta_shape *shape, float scale, void *stream)
{
    return ssm2d_impl::step_entry<float>(q, k, v, g, beta, state, o, shape, scale, stream);
}

int ssm2d_gated_delta_step_bf16(const uint16_t *q, const uint16_t *k, const uint16_t *v, const float *g, const float *beta,
                                float *state, uint16_t *o, const ssm2d_delta_shape *shape, float scale, void *stream)
{
    return ssm2d_impl::step_entry<uint16_t>(q, k, v, g, beta, state, o, shape, scale, stream);
}

}  // extern "C"
