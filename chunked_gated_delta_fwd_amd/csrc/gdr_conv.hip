// Short causal depthwise convolution of a token mixer, W = 2, 3 or 4 taps:
//
//   z[t, c] = bias[c] + sum_j w[c, j] x[t - (W-1) + j, c],   y = z or z sigmoid(z)
//
// where positions before a sequence's first token are its state s0 (W - 1
// rows) and the final state is the last W - 1 rows of [s0, x].  Forward,
// backward and the single-token step.  The arithmetic (2 W + 4 operations a
// value) is far below what the bytes allow, so everything here is about
// reading and writing each value once in 16-byte pieces.
//
// Layout: a thread owns one 16-byte piece of the channels (8 bf16, 4 f32; one
// channel when sizes or addresses do not allow pieces) and walks a strip of
// tokens with the last W - 1 rows in registers, so a row is read once per
// strip and the W - 1 rows before a strip come from L2 (xcd_run puts
// neighbouring strips on one XCD).  Sums are fp32, y is rounded once.
#include "gdr_device.h"
#include "gdr_mixer.h"

namespace gdr {
namespace {

constexpr int kThreads = 256;

// VEC consecutive elements at p as floats
template <bool BF16, int VEC>
__device__ __forceinline__ void ldv(const void *base, int64_t i, float (&o)[VEC]) {
    if constexpr (VEC == 1) {
        o[0] = load_scalar<BF16>(base, i);
    } else if constexpr (BF16) {
        typedef unsigned int Piece __attribute__((ext_vector_type(VEC / 2)));
        const Piece u = *reinterpret_cast<const Piece *>(reinterpret_cast<const uint16_t *>(base) + i);
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
            o[2 * e] = __uint_as_float(u[e] << 16);
            o[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
        }
    } else {
        const f32x4 u = *reinterpret_cast<const f32x4 *>(reinterpret_cast<const float *>(base) + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = u[e];
    }
}
template <bool BF16, int VEC, bool PAST = false>
__device__ __forceinline__ void stv(void *base, int64_t i, const float (&o)[VEC]) {
    if constexpr (VEC == 1) {
        if constexpr (BF16) reinterpret_cast<uint16_t *>(base)[i] = bf16_bits(o[0]);
        else reinterpret_cast<float *>(base)[i] = o[0];
    } else if constexpr (BF16) {
        typedef unsigned int Piece __attribute__((ext_vector_type(VEC / 2)));
        Piece u;
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e)
            u[e] = bf16_bits(o[2 * e]) | (static_cast<uint32_t>(bf16_bits(o[2 * e + 1])) << 16);
        Piece *const to = reinterpret_cast<Piece *>(reinterpret_cast<uint16_t *>(base) + i);
        if constexpr (PAST) __builtin_nontemporal_store(u, to);
        else *to = u;
    } else {
        f32x4 u;
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = o[e];
        f32x4 *const to = reinterpret_cast<f32x4 *>(reinterpret_cast<float *>(base) + i);
        if constexpr (PAST) __builtin_nontemporal_store(u, to);
        else *to = u;
    }
}

// sigmoid(z); bf16 outputs take the hardware's exp2 and reciprocal (1 ulp of
// fp32 each, far below a bf16 step), f32 outputs the library's exp and divide.
template <bool BF16>
__device__ __forceinline__ float sigmoid(float z) {
    if constexpr (BF16) return __builtin_amdgcn_rcpf(1.f + fast_exp2(-kLog2e * z));
    else return 1.f / (1.f + expf(-z));
}

// The W taps of VEC channels: w[c][j], contiguous.
template <bool BF16, int W, int VEC>
__device__ __forceinline__ void load_taps(const void *w, int64_t c, float (&o)[VEC][W]) {
    if constexpr (VEC == 1) {
#pragma unroll
        for (int j = 0; j < W; ++j) o[0][j] = load_scalar<BF16>(w, c * W + j);
    } else {
        float f[W][VEC];
#pragma unroll
        for (int j = 0; j < W; ++j) ldv<BF16, VEC>(w, c * W + j * VEC, f[j]);
#pragma unroll
        for (int v = 0; v < VEC; ++v)
#pragma unroll
            for (int j = 0; j < W; ++j) o[v][j] = f[(v * W + j) / VEC][(v * W + j) % VEC];
    }
}

// Sequence n's tokens [s, e), clamped to the tensor whatever cu holds.
__device__ __forceinline__ void seq_range(const ConvArgs &a, int64_t n, int64_t &s, int64_t &e) {
    if (a.cu) {
        s = a.cu[n];
        e = a.cu[n + 1];
        s = s < 0 ? 0 : s > a.total ? a.total : s;
        e = e < s ? s : e > a.total ? a.total : e;
    } else {
        s = n * a.seq_len;
        e = s + a.seq_len;
    }
}
// The sequence that holds token t (length-0 sequences hold none): the last n with cu[n] <= t.
__device__ __forceinline__ int64_t seq_of(const ConvArgs &a, int64_t t) {
    if (!a.cu) return t / a.seq_len;
    int64_t lo = 0, hi = a.n_seq;   // cu[lo] <= t < cu[hi] for valid content
    while (hi - lo > 1) {
        const int64_t m = (lo + hi) / 2;
        if (a.cu[m] <= t) lo = m;
        else hi = m;
    }
    return lo;
}

// Row at position pos of sequence n that starts at s; the state before it.
template <bool BF16, int W, int VEC>
__device__ __forceinline__ void load_past(const ConvArgs &a, int64_t pos, int64_t n, int64_t s, int64_t c,
                                          float (&o)[VEC]) {
    if (pos >= s) {
        ldv<BF16, VEC>(a.x, pos * a.ldx + c, o);
    } else if (a.s0) {
        ldv<BF16, VEC>(a.s0, (n * (W - 1) + (W - 1) + (pos - s)) * a.ch + c, o);
    } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) o[v] = 0.f;
    }
}

constexpr int kBatch = 4;   // rows in flight per thread (2, 4, 8: 446, 395, 414 us forward, 133, 115, 118 backward at the sizes below)

// 65536 tokens of 8192 bf16 channels, 4 taps: 383 us, 5.6 TB/s of the 2.15 GB
// read and written once (a large copy reaches 5.2): HBM bound.

// PAST: y is stored past the caches (compiled apart: a branch at each store
// takes 24 us).
template <bool BF16, int W, int VEC, bool PAST>
__global__ void __launch_bounds__(kThreads) gdr_conv_fwd_kernel(ConvArgs a, int64_t strip, int64_t n_strips,
                                                                 int64_t blocks) {
    const int64_t nvec = a.ch / VEC;
    const int64_t idx = xcd_run(blockIdx.x, blocks) * kThreads + threadIdx.x;
    const int64_t row = idx / nvec;
    const int64_t c = (idx - row * nvec) * VEC;
    if (row >= n_strips) {
        // the final state of sequence row - n_strips
        const int64_t n = row - n_strips;
        if (!a.st || n >= a.n_seq) return;
        int64_t s, e;
        seq_range(a, n, s, e);
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            float v[VEC];
            load_past<BF16, W, VEC>(a, e - (W - 1) + i, n, s, c, v);
            stv<BF16, VEC>(a.st, (n * (W - 1) + i) * a.ch + c, v);
        }
        return;
    }
    float w[VEC][W], bias[VEC];
    load_taps<BF16, W, VEC>(a.w, c, w);
#pragma unroll
    for (int v = 0; v < VEC; ++v) bias[v] = 0.f;
    if (a.bias) ldv<BF16, VEC>(a.bias, c, bias);
    const bool silu = a.silu != 0;

    const int64_t t0 = row * strip, t1 = t0 + strip < a.total ? t0 + strip : a.total;
    float win[W - 1][VEC];
    auto token = [&](int64_t t, const float (&x)[VEC]) {
        float o[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            float z = bias[v];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) z += w[v][j] * win[j][v];
            z += w[v][W - 1] * x[v];
            o[v] = silu ? z * sigmoid<BF16>(z) : z;
#pragma unroll
            for (int j = 0; j + 1 < W - 1; ++j) win[j][v] = win[j + 1][v];
            win[W - 2][v] = x[v];
        }
        stv<BF16, VEC, PAST>(a.y, t * a.ch + c, o);
    };
    for (int64_t t = t0; t < t1;) {
        const int64_t n = seq_of(a, t);
        int64_t s, e;
        seq_range(a, n, s, e);
        if (t < s || t >= e) {   // outside every sequence: not written
            ++t;
            continue;
        }
        const int64_t end = e < t1 ? e : t1;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) load_past<BF16, W, VEC>(a, t - (W - 1) + j, n, s, c, win[j]);
        for (; t + kBatch <= end; t += kBatch) {
            float x[kBatch][VEC];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) ldv<BF16, VEC>(a.x, (t + u) * a.ldx + c, x[u]);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) token(t + u, x[u]);
        }
        for (; t < end; ++t) {
            float x[VEC];
            ldv<BF16, VEC>(a.x, t * a.ldx + c, x);
            token(t, x);
        }
    }
}

// One token a sequence: a thread reads its piece of the W - 1 state rows and x,
// writes y and the shifted rows.  256 sequences of 8192 bf16 channels: 7.0 us
// for 34 MB, most of it the time of any launch.
template <bool BF16, int W, int VEC>
__global__ void __launch_bounds__(kThreads) gdr_conv_step_kernel(ConvArgs a) {
    const int64_t nvec = a.ch / VEC;
    const int64_t idx = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t n = idx / nvec;
    if (n >= a.n_seq) return;
    const int64_t c = (idx - n * nvec) * VEC;
    float x[W][VEC], w[VEC][W], o[VEC], bias[VEC];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) ldv<BF16, VEC>(a.st, (n * (W - 1) + j) * a.ch + c, x[j]);
    ldv<BF16, VEC>(a.x, n * a.ldx + c, x[W - 1]);
    load_taps<BF16, W, VEC>(a.w, c, w);
#pragma unroll
    for (int v = 0; v < VEC; ++v) bias[v] = 0.f;
    if (a.bias) ldv<BF16, VEC>(a.bias, c, bias);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        float z = bias[v];
#pragma unroll
        for (int j = 0; j < W; ++j) z += w[v][j] * x[j][v];
        o[v] = a.silu ? z * sigmoid<BF16>(z) : z;
    }
    stv<BF16, VEC>(a.y, n * a.ch + c, o);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) stv<BF16, VEC>(a.st, (n * (W - 1) + j) * a.ch + c, x[j + 1]);
}

// --- backward -------------------------------------------------------------------
// With dz = dy act'(z):
//   dx[p] = sum_j w[j] dz[p + (W-1) - j]  (+ dst where p is a row of the final state)
//   dw[j] = sum_t dz[t] x[t - (W-1) + j],   db = sum_t dz[t],
//   ds0 likewise for the positions before the sequence.
// z is recomputed.  A thread walks its strip and W - 1 tokens past it (their
// dz belong to its dx) with x and dz windows in registers.  dw and db: sums
// over the strip in registers, over the block's strips through LDS in a fixed
// order, over blocks by a second kernel (no atomics: the same bits every run).
// 16384 tokens of 4608 bf16 channels, 4 taps: 109 us and 4 for the sums, 4.2
// TB/s of the 453 MB; bound by HBM and by the strips' overlap.

// lanes of a block along the channels: a power of two up to 64
__host__ __device__ inline int conv_bwd_lanes(int64_t nvec) {
    int c = 1;
    while (c < 64 && c < nvec) c *= 2;
    return c;
}

template <bool BF16>
__device__ __forceinline__ float act_grad(float z, float dy, bool silu) {
    if (!silu) return dy;
    const float s = sigmoid<BF16>(z);
    return dy * s * (1.f + z * (1.f - s));
}

template <bool BF16, int W, int VEC>
__global__ void __launch_bounds__(kThreads) gdr_conv_bwd_kernel(ConvArgs a, int64_t strip, int64_t main_blocks,
                                                                 int64_t row_blocks) {
    const int64_t nvec = a.ch / VEC;
    float w[VEC][W], bias[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) bias[v] = 0.f;
    const bool silu = a.silu != 0;

    if (blockIdx.x >= main_blocks) {   // ds0 of one (sequence, piece)
        const int64_t idx = (blockIdx.x - main_blocks) * kThreads + threadIdx.x;
        const int64_t n = idx / nvec;
        if (n >= a.n_seq) return;
        const int64_t c = (idx - n * nvec) * VEC;
        load_taps<BF16, W, VEC>(a.w, c, w);
        if (a.bias) ldv<BF16, VEC>(a.bias, c, bias);
        int64_t s, e;
        seq_range(a, n, s, e);
        float line[2 * W - 2][VEC];   // positions s - (W-1) .. s + W - 2
#pragma unroll
        for (int i = 0; i < 2 * W - 2; ++i) {
            const int64_t pos = s - (W - 1) + i;
            if (pos < e) load_past<BF16, W, VEC>(a, pos, n, s, c, line[i]);
            else {
#pragma unroll
                for (int v = 0; v < VEC; ++v) line[i][v] = 0.f;
            }
        }
        float g[W - 1][VEC];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            if (a.dst && i >= e - s) ldv<BF16, VEC>(a.dst, (n * (W - 1) + i - (e - s)) * a.ch + c, g[i]);
            else {
#pragma unroll
                for (int v = 0; v < VEC; ++v) g[i][v] = 0.f;
            }
        }
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {   // token s + k reaches rows k .. W-2 of the state with taps 0 ..
            if (s + k >= e) break;
            float dy[VEC];
            ldv<BF16, VEC>(a.dy, (s + k) * a.lddy + c, dy);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                float z = bias[v];
#pragma unroll
                for (int j = 0; j < W; ++j) z += w[v][j] * line[k + j][v];
                const float dz = act_grad<BF16>(z, dy[v], silu);
#pragma unroll
                for (int j = 0; j + k < W - 1; ++j) g[k + j][v] += dz * w[v][j];
            }
        }
#pragma unroll
        for (int i = 0; i < W - 1; ++i) stv<BF16, VEC>(a.ds0, (n * (W - 1) + i) * a.ch + c, g[i]);
        return;
    }

    const int lanes = conv_bwd_lanes(nvec), strips = kThreads / lanes;
    const int lane = threadIdx.x % lanes, sub = threadIdx.x / lanes;
    const int64_t item = xcd_run(blockIdx.x, main_blocks);
    const int64_t cb = item / row_blocks, rb = item - cb * row_blocks;
    const int64_t cv = cb * lanes + lane;
    const bool live = cv < nvec;
    const int64_t c = live ? cv * VEC : 0;
    load_taps<BF16, W, VEC>(a.w, c, w);
    if (a.bias) ldv<BF16, VEC>(a.bias, c, bias);
    float acc[VEC][W + 1];
#pragma unroll
    for (int v = 0; v < VEC; ++v)
#pragma unroll
        for (int j = 0; j <= W; ++j) acc[v][j] = 0.f;

    const int64_t t0 = (rb * strips + sub) * strip;
    const int64_t t1 = t0 + strip < a.total ? t0 + strip : a.total;
    for (int64_t t = live ? t0 : t1; t < t1;) {
        const int64_t n = seq_of(a, t);
        int64_t s, e;
        seq_range(a, n, s, e);
        if (t < s || t >= e) {
            ++t;
            continue;
        }
        const int64_t first = t, end = e < t1 ? e : t1;
        float xw[W - 1][VEC], dzw[W - 1][VEC];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            load_past<BF16, W, VEC>(a, t - (W - 1) + j, n, s, c, xw[j]);
#pragma unroll
            for (int v = 0; v < VEC; ++v) dzw[j][v] = 0.f;
        }
        // token u: its dz (0 past the sequence), its part of dw, and dx of u - (W-1)
        auto token = [&](int64_t u, const float (&x)[VEC], const float (&dy)[VEC], bool mine, bool write,
                         const float (&more)[VEC]) {
            float o[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                float z = bias[v];
#pragma unroll
                for (int j = 0; j < W - 1; ++j) z += w[v][j] * xw[j][v];
                z += w[v][W - 1] * x[v];
                const float dz = act_grad<BF16>(z, dy[v], silu);
                if (mine) {
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) acc[v][j] += dz * xw[j][v];
                    acc[v][W - 1] += dz * x[v];
                    acc[v][W] += dz;
                }
                float g = more[v] + w[v][0] * dz;
#pragma unroll
                for (int j = 1; j < W; ++j) g += w[v][j] * dzw[W - 1 - j][v];
                o[v] = g;
#pragma unroll
                for (int j = 0; j + 1 < W - 1; ++j) {
                    xw[j][v] = xw[j + 1][v];
                    dzw[j][v] = dzw[j + 1][v];
                }
                xw[W - 2][v] = x[v];
                dzw[W - 2][v] = dz;
            }
            if (write) stv<BF16, VEC>(a.dx, (u - (W - 1)) * a.ch + c, o);
        };
        float none[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) none[v] = 0.f;
        int64_t u = first;
        for (; u < end && u < first + (W - 1); ++u) {
            float x[VEC], dy[VEC];
            ldv<BF16, VEC>(a.x, u * a.ldx + c, x);
            ldv<BF16, VEC>(a.dy, u * a.lddy + c, dy);
            token(u, x, dy, true, false, none);
        }
        for (; u + kBatch <= end; u += kBatch) {
            float x[kBatch][VEC], dy[kBatch][VEC];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                ldv<BF16, VEC>(a.x, (u + i) * a.ldx + c, x[i]);
                ldv<BF16, VEC>(a.dy, (u + i) * a.lddy + c, dy[i]);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) token(u + i, x[i], dy[i], true, true, none);
        }
        for (; u < end + (W - 1); ++u) {
            float x[VEC], dy[VEC], more[VEC];
            const int64_t p = u - (W - 1), place = p - (e - (W - 1));
#pragma unroll
            for (int v = 0; v < VEC; ++v) x[v] = dy[v] = more[v] = 0.f;
            if (u < e) {
                ldv<BF16, VEC>(a.x, u * a.ldx + c, x);
                ldv<BF16, VEC>(a.dy, u * a.lddy + c, dy);
            }
            if (a.dst && p >= first && place >= 0)
                ldv<BF16, VEC>(a.dst, (n * (W - 1) + place) * a.ch + c, more);
            token(u, x, dy, u < end, p >= first, more);
        }
        t = end;
    }

    // dw and db over the block's strips, in their order
    constexpr int kVals = VEC * (W + 1);
    __shared__ float sum[64][kVals + 1];
    for (int k = 0; k < strips; ++k) {
        if (sub == k) {
#pragma unroll
            for (int v = 0; v < VEC; ++v)
#pragma unroll
                for (int j = 0; j <= W; ++j) {
                    float &d = sum[lane][v * (W + 1) + j];
                    d = k ? d + acc[v][j] : acc[v][j];
                }
        }
        __syncthreads();
    }
    float *to = a.part + rb * a.ch * (W + 1);
    for (int i = threadIdx.x; i < lanes * kVals; i += kThreads) {
        const int64_t at = cb * lanes * kVals + i;
        if (at < static_cast<int64_t>(a.ch) * (W + 1)) to[at] = sum[i / kVals][i % kVals];
    }
}

// dw[c][j] and db[c]: the rows of partial sums, added in order
template <int W>
__global__ void __launch_bounds__(64) gdr_conv_wsum_kernel(ConvArgs a, int64_t rows) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
    const int64_t cols = static_cast<int64_t>(a.ch) * (W + 1);
    if (i >= cols) return;
    float s[8] = {};
    int64_t r = 0;
    for (; r + 8 <= rows; r += 8)
#pragma unroll
        for (int k = 0; k < 8; ++k) s[k] += a.part[(r + k) * cols + i];
    for (; r < rows; ++r) s[0] += a.part[r * cols + i];
    const float v = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
    const int64_t c = i / (W + 1);
    const int j = static_cast<int>(i % (W + 1));
    if (j < W) a.dw[c * W + j] = v;
    else if (a.db) a.db[c] = v;
}

// Calls f.template operator()<BF16, W, VEC>() for the call's type, taps and
// piece; VECB: channels of a bf16 piece.
template <int VECB, class F>
hipError_t by_conv(const ConvArgs &a, F f) {
    auto width = [&]<bool BF16, int VEC>() {
        switch (a.width) {
        case 2: return f.template operator()<BF16, 2, VEC>();
        case 3: return f.template operator()<BF16, 3, VEC>();
        default: return f.template operator()<BF16, 4, VEC>();
        }
    };
    if (a.bf16) return a.vec ? width.template operator()<true, VECB>() : width.template operator()<true, 1>();
    return a.vec ? width.template operator()<false, 4>() : width.template operator()<false, 1>();
}

int64_t pieces(int32_t ch, int32_t bf16, int32_t vec, int vecb) { return vec ? ch / (bf16 ? vecb : 4) : ch; }

// Channels of a bf16 piece in the backward pass: its windows and sums for 8
// take over 200 registers, 2 waves a SIMD, and 131 us where 4 take 113 (16384
// tokens of 4608 channels).
constexpr int kBwdVec = 4;

}  // namespace

hipError_t launch_conv_fwd(const ConvArgs &a, hipStream_t stream) {
    const int64_t nvec = pieces(a.ch, a.bf16, a.vec, 8);
    // Strips of 64 tokens re-read 3 rows in 67; shorter ones when there would
    // be fewer than 8 waves a CU otherwise.  256 tokens of 4096 bf16 channels:
    // 4.2 us in strips of 4, 18.7 in strips of 64; 65536 of 8192: 575 and 389.
    // Pieces against single channels (a count or address that is no multiple
    // of 16 bytes): 16384 tokens of 4608 and 4607 channels, 61 and 70 us.
    int64_t strip = 64;
    while (strip > kBatch && (a.total + strip - 1) / strip * nvec < 256 * 8 * 64) strip /= 2;
    const int64_t n_strips = (a.total + strip - 1) / strip;
    const int64_t blocks = ((n_strips + (a.st ? a.n_seq : 0)) * nvec + kThreads - 1) / kThreads;
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
    return by_conv<8>(a, [&]<bool BF16, int W, int VEC>() {
        const dim3 grid(static_cast<uint32_t>(blocks));
        if (VEC > 1 && past_caches(a.total * a.ch * (BF16 ? 2 : 4)))
            hipLaunchKernelGGL((gdr_conv_fwd_kernel<BF16, W, VEC, (VEC > 1)>), grid, dim3(kThreads), 0, stream, a, strip,
                               n_strips, blocks);
        else
            hipLaunchKernelGGL((gdr_conv_fwd_kernel<BF16, W, VEC, false>), grid, dim3(kThreads), 0, stream, a, strip, n_strips,
                               blocks);
        return hipGetLastError();
    });
}

hipError_t launch_conv_step(const ConvArgs &a, hipStream_t stream) {
    const int64_t blocks = (pieces(a.ch, a.bf16, a.vec, 8) * a.n_seq + kThreads - 1) / kThreads;
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
    return by_conv<8>(a, [&]<bool BF16, int W, int VEC>() {
        hipLaunchKernelGGL((gdr_conv_step_kernel<BF16, W, VEC>), dim3(static_cast<uint32_t>(blocks)), dim3(kThreads), 0,
                           stream, a);
        return hipGetLastError();
    });
}

// Strips of 64 tokens (3 rows re-read on either side, one row of sums stored
// for the block's strips); shorter ones while there are less than 4 blocks a CU.
// 256 tokens of 4096 bf16 channels: 14.5 us in strips of 8, 29.5 in strips of
// 64; 16384 of 4608: 214 and 112.
struct BwdSplit {
    int64_t strip, rows, blocks;
};
static BwdSplit bwd_split(int64_t total, int32_t ch, int32_t bf16, int32_t vec) {
    const int64_t nvec = pieces(ch, bf16, vec, kBwdVec);
    const int lanes = conv_bwd_lanes(nvec);
    BwdSplit s;
    s.strip = 128;
    do {
        s.strip /= 2;
        const int64_t per = kThreads / lanes * s.strip;
        s.rows = (total + per - 1) / per;
        s.blocks = s.rows * ((nvec + lanes - 1) / lanes);
    } while (s.strip > 8 && s.blocks < 1024);
    return s;
}

int64_t conv_bwd_rows(int64_t total, int32_t ch, int32_t bf16, int32_t vec) { return bwd_split(total, ch, bf16, vec).rows; }

hipError_t launch_conv_bwd(const ConvArgs &a, hipStream_t stream) {
    const int64_t nvec = pieces(a.ch, a.bf16, a.vec, kBwdVec);
    const BwdSplit s = bwd_split(a.total, a.ch, a.bf16, a.vec);
    const int64_t blocks = s.blocks + (a.ds0 ? (a.n_seq * nvec + kThreads - 1) / kThreads : 0);
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
    return by_conv<kBwdVec>(a, [&]<bool BF16, int W, int VEC>() {
        if (blocks > 0)
            hipLaunchKernelGGL((gdr_conv_bwd_kernel<BF16, W, VEC>), dim3(static_cast<uint32_t>(blocks)), dim3(kThreads), 0,
                               stream, a, s.strip, s.blocks, s.rows);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        const int64_t cols = static_cast<int64_t>(a.ch) * (W + 1);
        hipLaunchKernelGGL((gdr_conv_wsum_kernel<W>), dim3(static_cast<uint32_t>((cols + 63) / 64)), dim3(64), 0, stream,
                           a, s.rows);
        return hipGetLastError();
    });
}

}  // namespace gdr
