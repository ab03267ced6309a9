// Norm of every query and key head row with the position rotation in the same
// pass, forward and backward:
//
//   n = x / sqrt(s + eps) * w,  s = sum x^2 (L2) or its mean (RMS)
//   (a, b) -> (a cos - b sin, a sin + b cos) on the first `rot` channels
//
// pairs (i, i + rot/2) or, interleaved, (2i, 2i + 1), angle i of the token's
// row of the tables.  HBM bound: every value is read and written once.
//
// Layout: a head row of d = 64, 128 or 256 channels lies on d / 8 lanes, 8
// channels each (16 bytes of bf16, 32 of f32), so a wave holds 8, 4 or 2 rows,
// the sum of squares is 3 to 5 lane exchanges, and a rotation pair's other
// half is a lane exchange (or the same lane's neighbour channel).  A lane
// group keeps one token and walks its heads, so cos and sin are read once per
// token and slice of heads.  All arithmetic is fp32; outputs are rounded once.
#include "gdr_device.h"
#include "gdr_mixer.h"

namespace gdr {
namespace {

constexpr int kThreads = 256;

template <bool BF16>
__device__ __forceinline__ void ld8f(const void *base, int64_t i, float (&o)[8]) {
    if constexpr (BF16) {
        const v4u32 u = *reinterpret_cast<const v4u32 *>(reinterpret_cast<const uint16_t *>(base) + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            o[2 * e] = __uint_as_float(u[e] << 16);
            o[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
        }
    } else {
        const f32x4 *p = reinterpret_cast<const f32x4 *>(reinterpret_cast<const float *>(base) + i);
        const f32x4 u = p[0], v = p[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            o[e] = u[e];
            o[4 + e] = v[e];
        }
    }
}
template <bool BF16>
__device__ __forceinline__ void st8f(void *base, int64_t i, const float (&o)[8]) {
    if constexpr (BF16) {
        v4u32 u;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            u[e] = bf16_bits(o[2 * e]) | (static_cast<uint32_t>(bf16_bits(o[2 * e + 1])) << 16);
        *reinterpret_cast<v4u32 *>(reinterpret_cast<uint16_t *>(base) + i) = u;
    } else {
        f32x4 *p = reinterpret_cast<f32x4 *>(reinterpret_cast<float *>(base) + i);
        p[0] = f32x4{o[0], o[1], o[2], o[3]};
        p[1] = f32x4{o[4], o[5], o[6], o[7]};
    }
}

// sum over the lanes of a row (a power of two of neighbouring lanes)
template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int m = 1; m < LANES; m *= 2) x += __shfl_xor(x, m);
    return x;
}

// A lane's part of its token's rotation: y = x * c + partner(x) * s
struct Turn {
    float c[8], s[8];
    int partner;   // lane that holds the other halves (this lane: not exchanged)
    bool on;
};

// position of a token, clamped into the tables whatever `pos` holds
__device__ __forceinline__ int64_t position(const NormArgs &a, int64_t token) {
    const int64_t p = a.pos ? a.pos[token] : token % a.seq_len;
    return p < 0 ? 0 : p >= a.table ? a.table - 1 : p;
}

template <int LANES>
__device__ __forceinline__ void load_turn(const NormArgs &a, int64_t token, int l, Turn &t) {
    const int half = a.rot / 2;
    t.on = 8 * l < a.rot;
    t.partner = threadIdx.x % 64;
    if (!t.on) return;
    const int64_t row = position(a, token) * half;
    if (a.interleaved) {
        const f32x4 c = *reinterpret_cast<const f32x4 *>(a.cos + row + 4 * l);
        const f32x4 s = *reinterpret_cast<const f32x4 *>(a.sin + row + 4 * l);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            t.c[e] = c[e / 2];
            t.s[e] = (e & 1) ? s[e / 2] : -s[e / 2];
        }
    } else {
        const bool low = 8 * l < half;
        const int at = low ? 8 * l : 8 * l - half;
        const f32x4 *c = reinterpret_cast<const f32x4 *>(a.cos + row + at);
        const f32x4 *s = reinterpret_cast<const f32x4 *>(a.sin + row + at);
        const f32x4 c0 = c[0], c1 = c[1], s0 = s[0], s1 = s[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            t.c[e] = c0[e];
            t.c[4 + e] = c1[e];
            t.s[e] = low ? -s0[e] : s0[e];
            t.s[4 + e] = low ? -s1[e] : s1[e];
        }
        t.partner += low ? half / 8 : -half / 8;
    }
}

// Rotates a lane's 8 channels (back: the transposed rotation).  Every lane of
// the wave takes part: the partner's values come through a lane exchange.
__device__ __forceinline__ void rotate(const NormArgs &a, const Turn &t, bool back, float (&x)[8]) {
    float o[8];
    if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = x[e ^ 1];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = __shfl(x[e], t.partner);
    }
    if (t.on) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * t.c[e] + (back ? -o[e] : o[e]) * t.s[e];
    }
}

// A work item: one token and `per` of its q heads or of its k heads.
struct Item {
    int64_t token;
    int first, end;
    bool is_k;
};
__device__ __forceinline__ Item item_of(const NormArgs &a, int64_t i, int per, int slices_q, int slices) {
    Item r;
    r.token = i / slices;
    int s = static_cast<int>(i - r.token * slices);
    r.is_k = s >= slices_q;
    if (r.is_k) s -= slices_q;
    const int heads = r.is_k ? a.hk : a.hq;
    r.first = s * per;
    r.end = r.first + per < heads ? r.first + per : heads;
    return r;
}

template <bool BF16, int D>
__global__ void __launch_bounds__(kThreads) gdr_norm_fwd_kernel(NormArgs a, int64_t items, int per, int slices_q,
                                                                 int slices) {
    constexpr int LANES = D / 8, ROWS = kThreads / LANES;
    const int l = threadIdx.x % LANES;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / LANES;
    const bool live = i < items;
    const Item it = item_of(a, live ? i : items - 1, per, slices_q, slices);
    const void *in = it.is_k ? a.k : a.q, *wp = it.is_k ? a.wk : a.wq;
    void *out = it.is_k ? a.ok : a.oq;
    const int64_t at = it.token * (it.is_k ? a.ldk : a.ldq) + 8 * l;
    const int64_t to = it.token * (it.is_k ? a.hk : a.hq) * D + 8 * l;
    const float inv_m = a.rms ? 1.f / D : 1.f;
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.f;
    if (wp) ld8f<BF16>(wp, 8 * l, w);
    Turn t;
    if (a.rot) load_turn<LANES>(a, it.token, l, t);
    constexpr int U = 4;
    // every lane of a wave runs the same number of rows (the exchanges need
    // them all): `per` of them, those past the slice read and store nothing
    for (int h0 = 0; h0 < per; h0 += U) {
        float x[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = it.first + h0 + u;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[u][e] = 0.f;
            if (h0 + u < per && h < it.end) ld8f<BF16>(in, at + static_cast<int64_t>(h) * D, x[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = it.first + h0 + u;
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s += x[u][e] * x[u][e];
            const float inv = 1.f / sqrtf(row_sum<LANES>(s) * inv_m + a.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[u][e] *= inv * w[e];
            if (a.rot) rotate(a, t, false, x[u]);
            if (live && h0 + u < per && h < it.end) st8f<BF16>(out, to + static_cast<int64_t>(h) * D, x[u]);
        }
    }
}

// Backward.  With g = R^T do (the rotation undone) and r = 1 / sqrt(s + eps):
//   dw = sum over rows of g x r,   dx = r (g w) - x r^3 (sum g w x) [/ d]
// A block walks several items; dw is summed in registers, then over the
// block's rows in a fixed order, then over blocks by a second kernel.
template <bool BF16, int D>
__global__ void __launch_bounds__(kThreads) gdr_norm_bwd_kernel(NormArgs a, int64_t items, int per, int slices_q,
                                                                 int slices) {
    constexpr int LANES = D / 8, ROWS = kThreads / LANES;
    const int l = threadIdx.x % LANES, sub = threadIdx.x / LANES;
    const float inv_m = a.rms ? 1.f / D : 1.f;
    float aq[8], ak[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) aq[e] = ak[e] = 0.f;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * ROWS;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * ROWS; base < items; base += stride) {
        const int64_t i = base + sub;
        const bool live = i < items;
        const Item it = item_of(a, live ? i : items - 1, per, slices_q, slices);
        const void *in = it.is_k ? a.k : a.q, *gin = it.is_k ? a.dok : a.doq, *wp = it.is_k ? a.wk : a.wq;
        void *out = it.is_k ? a.dk : a.dq;
        const int64_t at = it.token * (it.is_k ? a.ldk : a.ldq) + 8 * l;
        const int64_t gat = it.token * (it.is_k ? a.lddok : a.lddoq) + 8 * l;
        const int64_t to = it.token * (it.is_k ? a.hk : a.hq) * D + 8 * l;
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.f;
        if (wp) ld8f<BF16>(wp, 8 * l, w);
        Turn t;
        if (a.rot) load_turn<LANES>(a, it.token, l, t);
        constexpr int U = 2;
        for (int h0 = 0; h0 < per; h0 += U) {
            float x[U][8], g[U][8];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = it.first + h0 + u;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[u][e] = g[u][e] = 0.f;
                if (live && h0 + u < per && h < it.end) {
                    ld8f<BF16>(in, at + static_cast<int64_t>(h) * D, x[u]);
                    ld8f<BF16>(gin, gat + static_cast<int64_t>(h) * D, g[u]);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = it.first + h0 + u;
                if (a.rot) rotate(a, t, true, g[u]);
                float s = 0.f, d = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    s += x[u][e] * x[u][e];
                    d += g[u][e] * w[e] * x[u][e];
                }
                const float inv = 1.f / sqrtf(row_sum<LANES>(s) * inv_m + a.eps);
                const float back = row_sum<LANES>(d) * inv_m * inv * inv * inv;
                if (live && h0 + u < per && h < it.end) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float dw = g[u][e] * (x[u][e] * inv);
                        aq[e] += it.is_k ? 0.f : dw;
                        ak[e] += it.is_k ? dw : 0.f;
                        x[u][e] = inv * (g[u][e] * w[e]) - x[u][e] * back;
                    }
                    st8f<BF16>(out, to + static_cast<int64_t>(h) * D, x[u]);
                }
            }
        }
    }
    if (!a.part) return;
    __shared__ float sum[ROWS][2][D];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        sum[sub][0][8 * l + e] = aq[e];
        sum[sub][1][8 * l + e] = ak[e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
        float s = 0.f;
        for (int r = 0; r < ROWS; ++r) s += sum[r][i / D][i % D];
        a.part[static_cast<int64_t>(blockIdx.x) * 2 * D + i] = s;
    }
}

// dwq and dwk: 16 columns a block, the rows of partial sums on 64 threads each
__global__ void __launch_bounds__(1024) gdr_norm_wsum_kernel(NormArgs a, int64_t rows) {
    __shared__ float sum[64][17];
    const int col = threadIdx.x % 16, sub = threadIdx.x / 16;
    const int i = blockIdx.x * 16 + col;
    float s = 0.f;
    for (int64_t r = sub; r < rows; r += 64) s += a.part[r * 2 * a.d + i];
    sum[sub][col] = s;
    __syncthreads();
    if (threadIdx.x < 16) {
        float v = 0.f;
        for (int k = 0; k < 64; ++k) v += sum[k][threadIdx.x];
        if (i < a.d) {
            if (a.dwq) a.dwq[i] = v;
        } else if (a.dwk) {
            a.dwk[i - a.d] = v;
        }
    }
}

template <class F>
hipError_t by_norm(const NormArgs &a, F f) {
    auto dim = [&]<bool BF16>() {
        switch (a.d) {
        case 64: return f.template operator()<BF16, 64>();
        case 128: return f.template operator()<BF16, 128>();
        default: return f.template operator()<BF16, 256>();
        }
    };
    return a.bf16 ? dim.template operator()<true>() : dim.template operator()<false>();
}

struct Split {
    int per, slices_q, slices;
    int64_t items;
};
// Heads of an item: up to 16, so that the tables are read once for them; fewer
// when there would be less than 4 waves a CU otherwise.
Split split_of(const NormArgs &a) {
    Split s;
    s.per = a.hq > a.hk ? a.hq : a.hk;
    if (s.per > 16) s.per = 16;
    auto count = [&] {
        s.slices_q = (a.hq + s.per - 1) / s.per;
        s.slices = s.slices_q + (a.hk + s.per - 1) / s.per;
        s.items = a.tokens * s.slices;
    };
    count();
    while (s.per > 1 && s.items * (a.d / 8) < 256 * 4 * 64) {
        s.per = (s.per + 1) / 2;
        count();
    }
    return s;
}

}  // namespace

hipError_t launch_norm_fwd(const NormArgs &a, hipStream_t stream) {
    const Split s = split_of(a);
    return by_norm(a, [&]<bool BF16, int D>() {
        constexpr int ROWS = kThreads / (D / 8);
        const int64_t blocks = (s.items + ROWS - 1) / ROWS;
        if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
        hipLaunchKernelGGL((gdr_norm_fwd_kernel<BF16, D>), dim3(static_cast<uint32_t>(blocks)), dim3(kThreads), 0, stream, a,
                           s.items, s.per, s.slices_q, s.slices);
        return hipGetLastError();
    });
}

int64_t norm_bwd_blocks(const NormArgs &a) {
    const int64_t rows = kThreads / (a.d / 8);
    const int64_t blocks = (split_of(a).items + rows - 1) / rows;
    return blocks < 2048 ? blocks : 2048;
}

hipError_t launch_norm_bwd(const NormArgs &a, hipStream_t stream) {
    const Split s = split_of(a);
    const int64_t blocks = norm_bwd_blocks(a);
    return by_norm(a, [&]<bool BF16, int D>() {
        if (blocks > 0)
            hipLaunchKernelGGL((gdr_norm_bwd_kernel<BF16, D>), dim3(static_cast<uint32_t>(blocks)), dim3(kThreads), 0, stream,
                               a, s.items, s.per, s.slices_q, s.slices);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess || !a.part) return e;
        hipLaunchKernelGGL(gdr_norm_wsum_kernel, dim3(2 * D / 16), dim3(1024), 0, stream, a, blocks);
        return hipGetLastError();
    });
}

}  // namespace gdr
