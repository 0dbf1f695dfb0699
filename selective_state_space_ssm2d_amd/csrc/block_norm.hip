// libssm2d: the block norm's entries and their checks (block_norm.h has the kernels).
#include "block_norm.h"

namespace ssm2d_impl {
namespace norm {

extern template int launch_norm<float, float, false>(NormParams, float *, float *, float *, hipStream_t);
extern template int launch_norm<float, float, true>(NormParams, float *, float *, float *, hipStream_t);
extern template int launch_norm<uint16_t, uint16_t, false>(NormParams, float *, float *, float *, hipStream_t);
extern template int launch_norm<uint16_t, uint16_t, true>(NormParams, float *, float *, float *, hipStream_t);
extern template int launch_norm<uint16_t, float, false>(NormParams, float *, float *, float *, hipStream_t);
extern template int launch_norm<uint16_t, float, true>(NormParams, float *, float *, float *, hipStream_t);

}  // namespace norm

namespace {

using namespace norm;

constexpr uint32_t kNormFlags = SSM2D_NORM_ON | SSM2D_NORM_GATE_SIGMOID | SSM2D_NORM_GATE_FIRST | SSM2D_NORM_RESIDUAL_F32;

// SSM2D_OK and *work, or what is wrong with the shape.
int check_norm(const ssm2d_block_norm_shape *a, uint32_t flags, bool *work)
{
    *work = false;
    if (flags & ~kNormFlags) return SSM2D_ERR_BAD_FLAGS;
    if (!a) return SSM2D_ERR_NULLPTR;
    if (a->rows < 0 || a->n < 0 || a->groups < 1 || a->n % a->groups != 0) return SSM2D_ERR_BAD_DIM;
    if (a->n > SSM2D_NORM_MAX_N) return SSM2D_ERR_UNSUPPORTED;
    if (a->rows > (int64_t{1} << 50) / std::max<int64_t>(a->n, 1)) return SSM2D_ERR_UNSUPPORTED;
    for (const int64_t st : {a->x_stride, a->gate_stride, a->res_stride, a->dout_stride, a->dy_stride})
        if (st < 0) return SSM2D_ERR_BAD_DIM;
    *work = a->rows > 0 && a->n > 0;
    return SSM2D_OK;
}

NormParams norm_params(const ssm2d_block_norm_shape &a, float eps, uint32_t flags)
{
    NormParams p{};
    p.rows = a.rows, p.n = static_cast<int>(a.n), p.groups = static_cast<int>(a.groups);
    p.ldx = a.x_stride, p.ldg = a.gate_stride, p.ldr = a.res_stride, p.ldo = a.dout_stride, p.ldy = a.dy_stride;
    p.eps = eps, p.inv_n = 1.0f / static_cast<float>(a.n), p.inv_g = 1.0f / static_cast<float>(a.n / a.groups);
    p.on = (flags & SSM2D_NORM_ON) != 0, p.first = (flags & SSM2D_NORM_GATE_FIRST) != 0;
    p.sigmoid = (flags & SSM2D_NORM_GATE_SIGMOID) != 0;
    return p;
}

template <typename T>
int norm_fwd(const T *x, const T *gate, const void *res, const float *weight, const float *scale, const float *next, void *out, T *y,
             const ssm2d_block_norm_shape *a, float eps, uint32_t flags, void *stream)
{
    bool work = false;
    const int st = check_norm(a, flags, &work);
    if (st != SSM2D_OK || !work) return st;
    if (!x || !out) return SSM2D_ERR_NULLPTR;
    const bool f32 = sizeof(T) == 4 || (flags & SSM2D_NORM_RESIDUAL_F32);
    const size_t tr = f32 ? 4 : 2;
    if (off_by(x, sizeof(T)) || off_by(gate, sizeof(T)) || off_by(y, sizeof(T)) || off_by(res, tr) || off_by(out, tr) || off_by(weight, 4) ||
        off_by(scale, 4) || off_by(next, 4))
        return SSM2D_ERR_MISALIGNED;
    NormParams p = norm_params(*a, eps, flags);
    p.x = x, p.gate = gate, p.res = res, p.weight = p.on ? weight : nullptr, p.scale = scale, p.next = next, p.out = out, p.y = y;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return f32 ? launch_norm<T, float, false>(p, nullptr, nullptr, nullptr, s) : launch_norm<T, T, false>(p, nullptr, nullptr, nullptr, s);
}

int64_t norm_workspace(const ssm2d_block_norm_shape *a, uint32_t flags)
{
    bool work = false;
    const int st = check_norm(a, flags, &work);
    if (st != SSM2D_OK) return -st;
    return work ? std::min<int64_t>(a->rows, kMaxParts) * 3 * a->n * 4 : 0;
}

template <typename T>
int norm_bwd(const T *x, const T *gate, const void *res, const float *weight, const float *scale, const float *next, const void *dout,
             const T *dy, T *dx, T *dgate, void *dres, float *dweight, float *dscale, float *dnext, const ssm2d_block_norm_shape *a, float eps,
             uint32_t flags, void *ws, int64_t ws_bytes, void *stream)
{
    bool work = false;
    const int st = check_norm(a, flags, &work);
    if (st != SSM2D_OK) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (off_by(dweight, 4) || off_by(dscale, 4) || off_by(dnext, 4)) return SSM2D_ERR_MISALIGNED;
    auto clear = [&](float *d) {
        if (!d || a->n == 0) return static_cast<int>(SSM2D_OK);
        clear_floats<<<dim3(static_cast<unsigned>((a->n + 255) / 256)), dim3(256), 0, s>>>(d, a->n);
        return launched();
    };
    if (!work) {  // (sums over no rows)
        for (float *d : {dweight, dscale, dnext}) {
            const int e = clear(d);
            if (e != SSM2D_OK) return e;
        }
        return SSM2D_OK;
    }
    if (!x) return SSM2D_ERR_NULLPTR;
    const bool f32 = sizeof(T) == 4 || (flags & SSM2D_NORM_RESIDUAL_F32);
    const size_t tr = f32 ? 4 : 2;
    if (off_by(x, sizeof(T)) || off_by(gate, sizeof(T)) || off_by(dy, sizeof(T)) || off_by(dx, sizeof(T)) || off_by(dgate, sizeof(T)) ||
        off_by(res, tr) || off_by(dout, tr) || off_by(dres, tr) || off_by(weight, 4) || off_by(scale, 4) || off_by(next, 4) || off_by(ws, 16))
        return SSM2D_ERR_MISALIGNED;
    NormParams p = norm_params(*a, eps, flags);
    p.x = x, p.gate = gate, p.res = res, p.weight = p.on ? weight : nullptr, p.scale = scale, p.next = next, p.dout = dout, p.dy = dy;
    p.dx = dx, p.dgate = dgate, p.dres = dres, p.sums = dweight || dscale || dnext;
    if (p.sums && (!ws || ws_bytes < norm_workspace(a, flags))) return SSM2D_ERR_NOMEM;
    if (!p.on) {  // (a weight that is left out has no gradient)
        const int e = clear(dweight);
        if (e != SSM2D_OK) return e;
        dweight = nullptr, p.sums = dscale || dnext;
    }
    p.part = static_cast<float *>(ws);
    return f32 ? launch_norm<T, float, true>(p, dweight, dscale, dnext, s) : launch_norm<T, T, true>(p, dweight, dscale, dnext, s);
}

}  // namespace
}  // namespace ssm2d_impl

extern "C" {

int ssm2d_block_norm_fwd(const float *x, const float *gate, const void *residual, const float *weight, const float *scale,
                         const float *next_weight, void *out, float *y, const ssm2d_block_norm_shape *shape, float eps, uint32_t flags,
                         void *stream)
{
    return ssm2d_impl::norm_fwd<float>(x, gate, residual, weight, scale, next_weight, out, y, shape, eps, flags, stream);
}

int ssm2d_block_norm_fwd_bf16(const uint16_t *x, const uint16_t *gate, const void *residual, const float *weight, const float *scale,
                              const float *next_weight, void *out, uint16_t *y, const ssm2d_block_norm_shape *shape, float eps,
                              uint32_t flags, void *stream)
{
    return ssm2d_impl::norm_fwd<uint16_t>(x, gate, residual, weight, scale, next_weight, out, y, shape, eps, flags, stream);
}

int64_t ssm2d_block_norm_bwd_workspace(const ssm2d_block_norm_shape *shape, uint32_t flags)
{
    return ssm2d_impl::norm_workspace(shape, flags);
}

int ssm2d_block_norm_bwd(const float *x, const float *gate, const void *residual, const float *weight, const float *scale,
                         const float *next_weight, const void *dout, const float *dy, float *dx, float *dgate, void *dresidual,
                         float *dweight, float *dscale, float *dnext_weight, const ssm2d_block_norm_shape *shape, float eps, uint32_t flags,
                         void *workspace, int64_t workspace_bytes, void *stream)
{
    return ssm2d_impl::norm_bwd<float>(x, gate, residual, weight, scale, next_weight, dout, dy, dx, dgate, dresidual, dweight, dscale,
                                       dnext_weight, shape, eps, flags, workspace, workspace_bytes, stream);
}

int ssm2d_block_norm_bwd_bf16(const uint16_t *x, const uint16_t *gate, const void *residual, const float *weight, const float *scale,
                              const float *next_weight, const void *dout, const uint16_t *dy, uint16_t *dx, uint16_t *dgate, void *dresidual,
                              float *dweight, float *dscale, float *dnext_weight, const ssm2d_block_norm_shape *shape, float eps,
                              uint32_t flags, void *workspace, int64_t workspace_bytes, void *stream)
{
    return ssm2d_impl::norm_bwd<uint16_t>(x, gate, residual, weight, scale, next_weight, dout, dy, dx, dgate, dresidual, dweight, dscale,
                                          dnext_weight, shape, eps, flags, workspace, workspace_bytes, stream);
}

}  // extern "C"
