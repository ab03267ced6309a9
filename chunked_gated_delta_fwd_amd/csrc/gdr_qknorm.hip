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
#include "gdr_lanes.h"
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
__device__ __forceinline__ void st8f(void *base, int64_t i, const float (&o)[8], bool past) {
    if constexpr (BF16) {
        v4u32 u;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            u[e] = bf16_bits(o[2 * e]) | (static_cast<uint32_t>(bf16_bits(o[2 * e + 1])) << 16);
        store_piece(reinterpret_cast<v4u32 *>(reinterpret_cast<uint16_t *>(base) + i), u, past);
    } else {
        f32x4 *p = reinterpret_cast<f32x4 *>(reinterpret_cast<float *>(base) + i);
        store_piece(p, f32x4{o[0], o[1], o[2], o[3]}, past);
        store_piece(p + 1, f32x4{o[4], o[5], o[6], o[7]}, past);
    }
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

// The q or the k side of a call: a block works on one of them, on items of a
// token and `per` of its heads.
struct Side {
    int heads, per, slices;
    int64_t items;
};
__host__ __device__ inline Side side_of(int64_t tokens, int heads, int most) {
    Side s;
    s.heads = heads;
    s.per = heads < most ? heads : most;
    s.slices = (heads + s.per - 1) / s.per;
    s.items = tokens * s.slices;
    return s;
}

// Of `blocks` blocks, blocks_k work on k, evenly spread among q's: a token's q
// and k are then read at about the same time (in two runs one after the other
// the forward pass took 230 us where it takes 213, at 65536 tokens of 16 and 16
// heads of 128).  The block's number on its side is left in `mine`.
__device__ __forceinline__ bool side_of_block(int64_t blocks_k, int64_t blocks, int64_t &mine) {
    const int64_t b = blockIdx.x, k = b * blocks_k / blocks;
    const bool is_k = (b + 1) * blocks_k / blocks != k;
    mine = is_k ? k : b - k;
    return is_k;
}

// 65536 tokens of 16 + 16 bf16 heads of 128: 216 to 219 us without rotation,
// 4.9 TB/s of the 1.07 GB, 231 us with (a large copy reaches 5.2 TB/s).
template <bool BF16, int D>
__global__ void __launch_bounds__(kThreads) gdr_norm_fwd_kernel(NormArgs a, int most, int64_t blocks_k) {
    constexpr int LANES = D / 8, ROWS = kThreads / LANES;
    const int l = threadIdx.x % LANES;
    int64_t mine;
    const bool is_k = side_of_block(blocks_k, gridDim.x, mine);
    const Side sd = side_of(a.tokens, is_k ? a.hk : a.hq, most);
    const int64_t i0 = mine * ROWS + threadIdx.x / LANES;
    const bool live = i0 < sd.items;
    const int64_t i = live ? i0 : sd.items - 1;
    const int64_t token = sd.slices == 1 ? i : i / sd.slices;
    const int first = static_cast<int>(i - token * sd.slices) * sd.per;
    const int count = !live ? 0 : first + sd.per < sd.heads ? sd.per : sd.heads - first;
    const void *in = is_k ? a.k : a.q, *wp = is_k ? a.wk : a.wq;
    void *out = is_k ? a.ok : a.oq;
    const int64_t at = token * (is_k ? a.ldk : a.ldq) + static_cast<int64_t>(first) * D + 8 * l;
    const int64_t to = (token * sd.heads + first) * D + 8 * l;
    const float inv_m = a.rms ? 1.f / D : 1.f;
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.f;
    if (wp) ld8f<BF16>(wp, 8 * l, w);
    Turn t;
    if (a.rot) load_turn<LANES>(a, token, l, t);
    const bool past = past_caches(a.tokens * (a.hq + a.hk) * D * (BF16 ? 2 : 4));
    constexpr int U = 4;
    // every lane of a wave runs the same number of rows (the exchanges need
    // them all): those past the item's heads read and store nothing
    for (int h0 = 0; h0 < sd.per; h0 += U) {
        float x[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[u][e] = 0.f;
            if (h0 + u < count) ld8f<BF16>(in, at + static_cast<int64_t>(h0 + u) * D, x[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s += x[u][e] * x[u][e];
            const float inv = 1.f / sqrtf(lane_sum<LANES>(s) * inv_m + a.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[u][e] *= inv * w[e];
            if (a.rot) rotate(a, t, false, x[u]);
            if (h0 + u < count) st8f<BF16>(out, to + static_cast<int64_t>(h0 + u) * D, x[u], past);
        }
    }
}

// Backward.  With g = R^T do (the rotation undone) and r = 1 / sqrt(s + eps):
//   dw = sum over rows of g x r,   dx = r (g w) - x r^3 (sum g w x) [/ d]
// A block walks several items, all of q or all of k; dw is summed in registers,
// then over the block's rows in a fixed order, then over blocks (q's rows of
// partial sums first) by a second kernel.  16384 tokens of 32 + 4 bf16 heads of
// 128: 102 us and 5 for the sums, 4.4 TB/s of the 453 MB.
template <bool BF16, int D>
__global__ void __launch_bounds__(kThreads) gdr_norm_bwd_kernel(NormArgs a, int most, int64_t blocks_k) {
    constexpr int LANES = D / 8, ROWS = kThreads / LANES;
    const int l = threadIdx.x % LANES, sub = threadIdx.x / LANES;
    int64_t mine;
    const bool is_k = side_of_block(blocks_k, gridDim.x, mine);
    const void *in = is_k ? a.k : a.q, *gin = is_k ? a.dok : a.doq, *wp = is_k ? a.wk : a.wq;
    void *out = is_k ? a.dk : a.dq;
    const int64_t ld = is_k ? a.ldk : a.ldq, ldg = is_k ? a.lddok : a.lddoq;
    const Side sd = side_of(a.tokens, is_k ? a.hk : a.hq, most);
    const int heads = sd.heads, per = sd.per;
    const int64_t items = sd.items;
    const int64_t stride = (is_k ? blocks_k : gridDim.x - blocks_k) * ROWS;
    const float inv_m = a.rms ? 1.f / D : 1.f;
    float w[8], acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        w[e] = 1.f;
        acc[e] = 0.f;
    }
    if (wp) ld8f<BF16>(wp, 8 * l, w);
    const bool past = past_caches(a.tokens * (a.hq + a.hk) * D * (BF16 ? 2 : 4));
    for (int64_t base = mine * ROWS; base < items; base += stride) {
        const bool live = base + sub < items;
        const int64_t i = live ? base + sub : items - 1;
        const int64_t token = sd.slices == 1 ? i : i / sd.slices;
        const int first = static_cast<int>(i - token * sd.slices) * per;
        const int count = !live ? 0 : first + per < heads ? per : heads - first;
        const int64_t at = token * ld + static_cast<int64_t>(first) * D + 8 * l;
        const int64_t gat = token * ldg + static_cast<int64_t>(first) * D + 8 * l;
        const int64_t to = (token * heads + first) * D + 8 * l;
        Turn t;
        if (a.rot) load_turn<LANES>(a, token, l, t);
        constexpr int U = 4;
        // every lane of a wave runs the same number of rows, for the exchanges
        for (int h0 = 0; h0 < per; h0 += U) {
            float x[U][8], g[U][8];
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[u][e] = g[u][e] = 0.f;
                if (h0 + u < count) {
                    ld8f<BF16>(in, at + static_cast<int64_t>(h0 + u) * D, x[u]);
                    ld8f<BF16>(gin, gat + static_cast<int64_t>(h0 + u) * D, g[u]);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (a.rot) rotate(a, t, true, g[u]);
                float s = 0.f, d = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    s += x[u][e] * x[u][e];
                    d += g[u][e] * w[e] * x[u][e];
                }
                const float inv = 1.f / sqrtf(lane_sum<LANES>(s) * inv_m + a.eps);
                const float back = lane_sum<LANES>(d) * inv_m * inv * inv * inv;
                if (h0 + u < count) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        acc[e] += g[u][e] * (x[u][e] * inv);
                        x[u][e] = inv * (g[u][e] * w[e]) - x[u][e] * back;
                    }
                    st8f<BF16>(out, to + static_cast<int64_t>(h0 + u) * D, x[u], past);
                }
            }
        }
    }
    if (!a.part) return;
    __shared__ float sum[ROWS][D];
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[sub][8 * l + e] = acc[e];
    __syncthreads();
    if (threadIdx.x < D) {
        float s = 0.f;
        for (int r = 0; r < ROWS; ++r) s += sum[r][threadIdx.x];
        a.part[((is_k ? gridDim.x - blocks_k : 0) + mine) * D + threadIdx.x] = s;
    }
}

// dwq (blockIdx.y 0, from the first blocks_q rows of partial sums) and dwk: 16
// columns a block, the rows on 64 threads each, 4 loads of a thread in flight
__global__ void __launch_bounds__(1024) gdr_norm_wsum_kernel(NormArgs a, int64_t blocks_q, int64_t blocks) {
    __shared__ float sum[64][17];
    const int col = threadIdx.x % 16, sub = threadIdx.x / 16;
    const int i = blockIdx.x * 16 + col;
    const int64_t first = blockIdx.y ? blocks_q : 0, end = blockIdx.y ? blocks : blocks_q;
    float s[4] = {};
    int64_t r = first + sub;
    for (; r + 3 * 64 < end; r += 4 * 64)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k] += a.part[(r + 64 * k) * a.d + i];
    for (; r < end; r += 64) s[0] += a.part[r * a.d + i];
    sum[sub][col] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    if (threadIdx.x < 16) {
        float v = 0.f;
        for (int k = 0; k < 64; ++k) v += sum[k][threadIdx.x];
        float *to = blockIdx.y ? a.dwk : a.dwq;
        if (to) to[i] = v;
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

// Heads of an item at most: 16, so that the tables are read once for them;
// fewer when there would be less than 4 waves a CU otherwise.  16 + 16 bf16
// heads of 128, rotated, 64 tokens: 5.4 us with one head an item, 10.5 with 16;
// 65536 tokens: 428 and 231.
int most_heads(const NormArgs &a) {
    int most = 16;
    while (most > 1 && (side_of(a.tokens, a.hq, most).items + side_of(a.tokens, a.hk, most).items) * (a.d / 8) < 256 * 4 * 64)
        most /= 2;
    return most;
}
int64_t blocks_of(const Side &s, int d) {
    const int64_t rows = kThreads / (d / 8);
    return (s.items + rows - 1) / rows;
}

}  // namespace

hipError_t launch_norm_fwd(const NormArgs &a, hipStream_t stream) {
    const int most = most_heads(a);
    const int64_t blocks_q = blocks_of(side_of(a.tokens, a.hq, most), a.d);
    const int64_t blocks = blocks_q + blocks_of(side_of(a.tokens, a.hk, most), a.d);
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
    return by_norm(a, [&]<bool BF16, int D>() {
        hipLaunchKernelGGL((gdr_norm_fwd_kernel<BF16, D>), dim3(static_cast<uint32_t>(blocks)), dim3(kThreads), 0, stream, a,
                           most, blocks - blocks_q);
        return hipGetLastError();
    });
}

namespace {
struct BwdSplit {
    int per;
    int64_t blocks_q, blocks;
};
// 8 blocks a CU at most, shared between q and k by their heads: each leaves a
// row of partial sums (16384 tokens, 32 + 4 heads of 128: 4 blocks a CU 127 us,
// 8 110, and with half the rows in flight 115 and 120)
BwdSplit bwd_split(const NormArgs &a) {
    BwdSplit s;
    s.per = most_heads(a);
    const int64_t nq = blocks_of(side_of(a.tokens, a.hq, s.per), a.d), nk = blocks_of(side_of(a.tokens, a.hk, s.per), a.d);
    const int64_t heads = static_cast<int64_t>(a.hq) + a.hk, most_q = (2048 * static_cast<int64_t>(a.hq) + heads - 1) / heads;
    s.blocks_q = nq < most_q ? nq : most_q;
    const int64_t most_k = 2048 - most_q > 0 ? 2048 - most_q : 1;
    s.blocks = s.blocks_q + (nk < most_k ? nk : most_k);
    return s;
}
}  // namespace

int64_t norm_bwd_blocks(const NormArgs &a) { return bwd_split(a).blocks; }

hipError_t launch_norm_bwd(const NormArgs &a, hipStream_t stream) {
    const BwdSplit s = bwd_split(a);
    return by_norm(a, [&]<bool BF16, int D>() {
        if (s.blocks > 0)
            hipLaunchKernelGGL((gdr_norm_bwd_kernel<BF16, D>), dim3(static_cast<uint32_t>(s.blocks)), dim3(kThreads), 0, stream,
                               a, s.per, s.blocks - s.blocks_q);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess || !a.part) return e;
        hipLaunchKernelGGL(gdr_norm_wsum_kernel, dim3(D / 16, 2), dim3(1024), 0, stream, a, s.blocks_q, s.blocks);
        return hipGetLastError();
    });
}

}  // namespace gdr
