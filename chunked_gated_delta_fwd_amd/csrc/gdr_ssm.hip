// Selective state space scan with one decay per head.  Per sequence and head,
// with the state S as [n][p]:
//
//   dt_t = softplus(dt_raw_t + dt_bias),  a_t = exp(dt_t A)
//   S_t = a_t S_{t-1} + dt_t b_t x_t^T,   y_t = S_t^T c_t + D x_t
//
// b and c are shared by the H / G heads of a group.
#include "gdr_device.h"
#include "gdr_mixer.h"

namespace gdr {
namespace {

// log(1 + e^v) without overflow; log1p keeps the small values' bits
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))); }

__device__ __forceinline__ float time_step(const SsmArgs &a, float raw, int h) {
    return softplus(raw + (a.dt_bias ? a.dt_bias[h] : 0.f));
}

// --- one token ------------------------------------------------------------------
// HBM bound: the state is read and written once, 8 n p bytes a head.  A block
// owns one (sequence, head) with the whole state in registers, 16 bytes a
// lane, so all of its loads are in flight at once; y is summed over the rows
// each thread holds, then over row groups through LDS.
template <int N, int P, bool BF16>
__global__ void __launch_bounds__(256) gdr_ssm_step_kernel(SsmArgs a) {
    constexpr int CG = P / 4, RG = 256 / CG, RPT = N / RG;
    __shared__ float s_b[N], s_c[N], s_part[RG][P];
    const int64_t seq = blockIdx.x / a.heads;
    const int h = static_cast<int>(blockIdx.x % a.heads);
    const int g = h / (a.heads / a.groups);
    const int t = threadIdx.x, cg = t % CG, rg = t / CG;
    const int j0 = 4 * cg, i0 = RPT * rg;
    float *hp = a.ht + (seq * a.heads + h) * N * P;
    f32x4 S[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) S[i] = *reinterpret_cast<const f32x4 *>(hp + (i0 + i) * P + j0);
    if (t < N) s_b[t] = load_scalar<BF16>(a.b, seq * a.ldb + g * N + t);
    else if (t < 2 * N) s_c[t - N] = load_scalar<BF16>(a.c, seq * a.ldc + g * N + t - N);
    const float raw = a.gate_bf16 ? load_scalar<true>(a.dt, seq * a.lddt + h) : load_scalar<false>(a.dt, seq * a.lddt + h);
    const float dt = time_step(a, raw, h);
    const float decay = expf(dt * a.A[h]);
    f32x4 x;
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = load_scalar<BF16>(a.x, seq * a.ldx + h * P + j0 + c);
    __syncthreads();
    f32x4 y = zero4();
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        S[i] = S[i] * decay + x * (dt * s_b[i0 + i]);
        *reinterpret_cast<f32x4 *>(hp + (i0 + i) * P + j0) = S[i];
        y = y + S[i] * s_c[i0 + i];
    }
    *reinterpret_cast<f32x4 *>(&s_part[rg][j0]) = y;
    __syncthreads();
    if (rg == 0) {
        f32x4 o = x * (a.D ? a.D[h] : 0.f);
#pragma unroll
        for (int r = 0; r < RG; ++r) o = o + *reinterpret_cast<const f32x4 *>(&s_part[r][j0]);
        const int64_t to = (seq * a.heads + h) * P + j0;
        if constexpr (BF16) *reinterpret_cast<bf16x4 *>(reinterpret_cast<uint16_t *>(a.y) + to) = cvt4(o);
        else *reinterpret_cast<f32x4 *>(reinterpret_cast<float *>(a.y) + to) = o;
    }
}

template <class F>
hipError_t by_ssm(const SsmArgs &a, F f) {
    auto type = [&]<int N, int P>() {
        return a.bf16 ? f.template operator()<N, P, true>() : f.template operator()<N, P, false>();
    };
    if (a.n == 64) return a.p == 64 ? type.template operator()<64, 64>() : type.template operator()<64, 128>();
    return a.p == 64 ? type.template operator()<128, 64>() : type.template operator()<128, 128>();
}

}  // namespace

hipError_t launch_ssm_step(const SsmArgs &a, hipStream_t stream) {
    return by_ssm(a, [&]<int N, int P, bool BF16>() {
        hipLaunchKernelGGL((gdr_ssm_step_kernel<N, P, BF16>), dim3(static_cast<uint32_t>(a.n_seq * a.heads)), dim3(256), 0,
                           stream, a);
        return hipGetLastError();
    });
}

}  // namespace gdr
