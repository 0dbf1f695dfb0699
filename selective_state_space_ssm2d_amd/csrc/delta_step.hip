// libssm2d: the gated delta rule token by token, for serving and for
// sequences of a few tokens.
//
// Memory-bound: a token costs 6 d_k d_v operations a head and one read and
// write of the state's 4 d_k d_v bytes. A workgroup holds VS columns of one
// head's state in registers (columns are independent: k and q mix rows only),
// a thread VEC neighbouring columns of every KR-th row. One pass over the
// state gives both S'^T k and S'^T q; the output needs no second one, since
//   S^T q = S'^T q + (k . q) u.
// Measured: 128 streams of 16 heads of 128 x 128 (bf16) take 46 us, 59 with the
// states in memory rather than cache (4.6 TB/s); one stream takes 4.6 us, a launch
// and a read's latency.
// Nothing is rounded but the output: q, k and v are widened, the state and all
// sums are fp32.
#include "delta.h"

namespace ssm2d_impl {
namespace {

struct StepParams {
    const void *q, *k, *v;
    const float *g, *beta, *h_init;
    float *h_last;
    void *o;
    long tokens, first;  // first: the launch's first head of all batch entries'
    int hk, h, dk, dv, slices;
    long qs[3], ks[3], vs[3], gs[3], bs[3];
    float scale;
};

// Sum of a row's lanes VL, 2 VL .. apart (VL = 4: by two rotations of the row).
template <int VL>
__device__ __forceinline__ float row_turn(float v)
{
    static_assert(VL == 4, "rotations");
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x128, 0xf, 0xf, true));  // row_ror:8
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x124, 0xf, 0xf, true));  // row_ror:4
    return v;
}

template <typename T, int VS, int VEC>
__global__ __launch_bounds__(256) void delta_step_kernel(StepParams p)
{
    constexpr int VL = VS / VEC, KR = 256 / VL, RPT = SSM2D_DELTA_MAX_DK / KR, RW = 64 / VL;  // RW: row groups a wave
    __shared__ float sk[SSM2D_DELTA_MAX_DK], sq[SSM2D_DELTA_MAX_DK];
    __shared__ float part[4][VS][2];
    const int tid = threadIdx.x, vl = tid % VL, kr = tid / VL, wave = tid / 64;
    const unsigned own = blockIdx.x / static_cast<unsigned>(p.slices);
    const int slice = static_cast<int>(blockIdx.x - own * p.slices);
    const long bh = p.first + own;
    const long b = bh / p.h;
    const int h = static_cast<int>(bh - b * p.h), hq = h / (p.h / p.hk);
    const int col = slice * VS + vl * VEC;
    const bool live = col < p.dv;
    const long base = bh * p.dk * p.dv + col;
    float S[RPT][VEC];
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        const int row = r * KR + kr;
        Raw<float, VEC> t;
        if (p.h_init && live && row < p.dk) t.load(p.h_init + base + static_cast<long>(row) * p.dv);
        else t.clear();
#pragma unroll
        for (int j = 0; j < VEC; ++j) S[r][j] = t.get(j);
    }
    const T *qp = static_cast<const T *>(p.q) + b * p.qs[0] + hq * p.qs[2], *kp = static_cast<const T *>(p.k) + b * p.ks[0] + hq * p.ks[2];
    const T *vp = static_cast<const T *>(p.v) + b * p.vs[0] + h * p.vs[2];
    T *op = static_cast<T *>(p.o) + (b * p.tokens * p.h + h) * p.dv;
    for (long t = 0; t < p.tokens; ++t) {
        if (tid < SSM2D_DELTA_MAX_DK) sk[tid] = tid < p.dk ? widen1(kp[t * p.ks[1] + tid]) : 0.0f;
        else sq[tid - SSM2D_DELTA_MAX_DK] = tid - SSM2D_DELTA_MAX_DK < p.dk ? widen1(qp[t * p.qs[1] + tid - SSM2D_DELTA_MAX_DK]) : 0.0f;
        const float alpha = expf(p.g[b * p.gs[0] + t * p.gs[1] + h * p.gs[2]]);
        const float beta = p.beta[b * p.bs[0] + t * p.bs[1] + h * p.bs[2]];
        float v[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = live ? widen1(vp[t * p.vs[1] + col + j]) : 0.0f;
        __syncthreads();
        float ak[VEC], aq[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) ak[j] = aq[j] = 0.0f;
#pragma unroll
        for (int r = 0; r < RPT; ++r) {
            const float kk = sk[r * KR + kr], qq = sq[r * KR + kr];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                S[r][j] *= alpha;
                ak[j] = fmaf(kk, S[r][j], ak[j]);
                aq[j] = fmaf(qq, S[r][j], aq[j]);
            }
        }
        // k . q, by every wave; the columns' sums over its row groups, then over the waves
        const float kq = lane_sum<64>(sk[tid % 64] * sq[tid % 64] + sk[64 + tid % 64] * sq[64 + tid % 64]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            // (rows of 16 lanes hold 16 / VL row groups of the same columns; mirror
            // images would mix columns, so within them a rotation by VL)
            if constexpr (VL == 4) ak[j] = row_turn<4>(ak[j]), aq[j] = row_turn<4>(aq[j]);
            if constexpr (VL <= 16) ak[j] = pair_sum<16>(ak[j]), aq[j] = pair_sum<16>(aq[j]);
            if constexpr (VL <= 32) ak[j] = pair_sum<32>(ak[j]), aq[j] = pair_sum<32>(aq[j]);
            if (kr % RW == 0) {
                part[wave][vl * VEC + j][0] = ak[j];
                part[wave][vl * VEC + j][1] = aq[j];
            }
        }
        __syncthreads();
        float u[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int c = vl * VEC + j;
            const float ks = (part[0][c][0] + part[1][c][0]) + (part[2][c][0] + part[3][c][0]);
            const float qs = (part[0][c][1] + part[1][c][1]) + (part[2][c][1] + part[3][c][1]);
            u[j] = beta * (v[j] - ks);
            if (live && kr == 0) store1(op + t * p.h * p.dv + col + j, p.scale * (qs + kq * u[j]));
        }
#pragma unroll
        for (int r = 0; r < RPT; ++r)
#pragma unroll
            for (int j = 0; j < VEC; ++j) S[r][j] = fmaf(sk[r * KR + kr], u[j], S[r][j]);
        __syncthreads();  // (sk, sq and part are read before the next token's are written)
    }
    if (!p.h_last || !live) return;
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        const int row = r * KR + kr;
        if (row >= p.dk) continue;
        Raw<float, VEC> t;
        t.set(S[r]);
        t.store(p.h_last + base + static_cast<long>(row) * p.dv);
    }
}

}  // namespace

template <typename T>
int delta_step(const DeltaArgs &a)
{
    StepParams p{};
    p.q = a.q, p.k = a.k, p.v = a.v, p.g = a.g, p.beta = a.beta, p.h_init = a.h_init, p.h_last = a.h_last, p.o = a.o;
    p.tokens = a.tokens, p.hk = a.hk, p.h = a.h, p.dk = a.dk_, p.dv = a.dv_, p.scale = a.scale;
    for (int i = 0; i < 3; ++i) {
        p.qs[i] = a.qs[i], p.ks[i] = a.ks[i], p.vs[i] = a.vs[i], p.gs[i] = a.gs[i], p.bs[i] = a.bs[i];
    }
    const hipStream_t s = static_cast<hipStream_t>(a.stream);
    const long heads = a.batch * a.h;
    auto go = [&](auto vs, auto vec) -> int {
        constexpr int VS = decltype(vs)::value, VEC = decltype(vec)::value;
        p.slices = (a.dv_ + VS - 1) / VS;
        const long most = most_groups(256) / p.slices;
        for (p.first = 0; p.first < heads; p.first += most) {
            delta_step_kernel<T, VS, VEC><<<dim3(static_cast<unsigned>(std::min(heads - p.first, most) * p.slices)), dim3(256), 0, s>>>(p);
            const int st = launched();
            if (st != SSM2D_OK) return st;
        }
        return SSM2D_OK;
    };
    using std::integral_constant;
    if (a.dv_ % 4 != 0 || off_by(a.h_init, 16) || off_by(a.h_last, 16))
        return go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    // Narrow slices while they are what fills the chip: of one token of 16 heads of
    // 128 x 128, bf16, 16 and 64 columns take 4.6 and 5.9 us for one stream, 5.0
    // and 5.8 for 2, 6.4 and 6.2 for 4, 10.3 and 6.9 for 8, 77 and 46 for 128.
    if (heads * ((a.dv_ + 63) / 64) >= 128) return go(integral_constant<int, 64>{}, integral_constant<int, 4>{});
    return go(integral_constant<int, 16>{}, integral_constant<int, 4>{});
}

template int delta_step<float>(const DeltaArgs &);
template int delta_step<uint16_t>(const DeltaArgs &);

}  // namespace ssm2d_impl
