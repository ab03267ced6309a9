// Device code shared by the state space scan's kernels (gdr_ssm.hip, gdr_ssm_bwd.hip).
#pragma once

#include <cfloat>

#include "gdr_device.h"
#include "gdr_lanes.h"
#include "gdr_mixer.h"

namespace gdr {
namespace {

// Matrix operands.  A product runs over 32 contraction indices k at a time,
// as two blocks of 16: lane (l16, lq) supplies row (or column) l16 with
// k = 4 lq + r of the first block and 16 + 4 lq + r of the second, r = 0..3,
// the order in which result tiles hold their rows.  bf16 operands take one
// 16x16x32 instruction, f32 operands eight 16x16x4 ones (fp32 products, no
// rounding of the inputs).
struct BfT {
    typedef uint16_t E;
    typedef bf16x8 F8;
    typedef bf16x4 F4;
    static __device__ __forceinline__ F4 raw4(const E *p) { return ld4(p); }
    static __device__ __forceinline__ f32x4 up(F4 a) { return up4(a); }
    static constexpr bool kBf16 = true;
    static constexpr int kParts = 3;   // operands that a split fp32 value takes
    static __device__ __forceinline__ f32x4 mma(F8 a, F8 b, f32x4 c) { return mfma32(a, b, c); }
    // LDS rows are an odd multiple of 8 banks apart: measured per wave, an
    // operand read then takes 2.7 units where 4 banks apart take 4.0, and a
    // transposed one 1.6 instead of 2.4.  Permuted (KP): columns in kpos order,
    // so that an operand with k along a row is one 16-byte read (two 8-byte
    // ones take 16 units; a transposed read costs 2.4 for it).  Plain: for
    // arrays that are only read across their rows.
    static constexpr int pitch(int cols, bool) { return cols + 16; }
    template <bool KP>
    static __device__ __forceinline__ int col(int x) { return KP ? kpos(x) : x; }   // of 4 columns from x, x % 4 == 0
    // k along a row: columns 32 q ..
    template <bool KP>
    static __device__ __forceinline__ F8 kfrag(const E *row, int q, int lq) {
        if constexpr (KP) return ld8(row + 32 * q + 8 * lq);
        else return cat(ld4(row + 32 * q + 4 * lq), ld4(row + 32 * q + 16 + 4 * lq));
    }
    // k along the rows of an LDS array: rows j0 .. j0 + 31, column x0 + l16
    template <bool KP>
    static __device__ __forceinline__ F8 tr(const E *m, int pitch, int j0, int x0, int l16, int lq) {
        const E *p = m + (j0 + 4 * lq + l16 / 4) * pitch +
                     (KP ? (x0 & ~31) + ((x0 >> 2) & 4) + 8 * (l16 % 4) : x0 + 4 * (l16 % 4));
        return cat(ld4_tr(p), ld4_tr(p + 16 * pitch));
    }
    static __device__ __forceinline__ f32x4 lo(F8 a) { return up4(__builtin_shufflevector(a, a, 0, 1, 2, 3)); }
    static __device__ __forceinline__ f32x4 hi(F8 a) { return up4(__builtin_shufflevector(a, a, 4, 5, 6, 7)); }
    static __device__ __forceinline__ f32x4 load4(const E *p) { return up4(ld4(p)); }
    static __device__ __forceinline__ void store4(E *p, f32x4 v) { st4(p, cvt4(v)); }
    // 0 in every lane, or NaN in some where a value of the wave's is not finite
    static __device__ __forceinline__ float probe(F8 a, F8 b) {
        const f32x4 d = mma(b, F8{}, mma(a, F8{}, zero4()));
        return (d[0] + d[1]) + (d[2] + d[3]);
    }
    // A part that is taken off a value.  INF: what is left of an infinite one is
    // infinite too, not NaN; only where that can be told apart in a result, the
    // state and a score with one x (65536 tokens take 847 us without, 878 with it
    // everywhere).
    template <bool INF>
    static __device__ __forceinline__ float part(uint32_t bits) {
        const float t = __uint_as_float(bits);
        return INF ? __builtin_amdgcn_fmed3f(t, -FLT_MAX, FLT_MAX) : t;
    }
    // An fp32 value as two bf16 ones: its top 8 bits and the rest, rounded.  The
    // sum is within 2^-15 of the value, so an operand that only reaches a bf16
    // output leaves that output its own rounding (2^-8) alone; one bf16 operand
    // added as much again (y of 600 tokens in 37 sequences was 2.2e-3 off and is
    // 1.7e-3 so, which is y's rounding; 65536 tokens take 830 us for 760, 55 of
    // them for the state's second part).
    static constexpr int kOutParts = 2;
    template <bool INF>
    static __device__ __forceinline__ void two(f32x4 a, F4 (&o)[2]) {
        v2u32 top;
        f32x4 rest;
#pragma unroll
        for (int e = 0; e < 2; ++e)
            top[e] = __builtin_amdgcn_perm(__float_as_uint(a[2 * e + 1]), __float_as_uint(a[2 * e]), 0x07060302u);
#pragma unroll
        for (int e = 0; e < 4; ++e) rest[e] = a[e] - part<INF>(__float_as_uint(a[e]) & 0xFFFF0000u);
        o[0] = __builtin_bit_cast(F4, top);
        o[1] = cvt4(rest);
    }
    static __device__ __forceinline__ void two(f32x4 a, f32x4 b, F8 (&o)[2]) {
        F4 x[2], y[2];
        two<false>(a, x);
        two<false>(b, y);
#pragma unroll
        for (int k = 0; k < 2; ++k) o[k] = cat(x[k], y[k]);
    }
    static __device__ __forceinline__ void store_two(E *top, E *rest, f32x4 v) {
        F4 o[2];
        two<true>(v, o);
        st4(top, o[0]);
        st4(rest, o[1]);
    }
    // An fp32 value as a sum of three bf16 ones: each takes the top 8 bits of
    // what is left, so the sum is the value exactly (a bf16 product keeps all
    // 16 bits of its operands' product in fp32).  This keeps the states, and
    // everything a gradient sums from them, at fp32 accuracy at three times
    // the matrix work; one rounded operand would leave 2^-8.
    template <bool INF>
    static __device__ __forceinline__ void split(f32x4 a, f32x4 b, F8 (&o)[3]) {
        typedef unsigned int u8v __attribute__((ext_vector_type(4)));
        u8v w[3];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float x = e < 2 ? a[2 * e] : b[2 * e - 4], y = e < 2 ? a[2 * e + 1] : b[2 * e - 3];
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const uint32_t xb = __float_as_uint(x), yb = __float_as_uint(y);
                w[k][e] = __builtin_amdgcn_perm(yb, xb, 0x07060302u);   // top halves of x (low) and y (high)
                if (k < 2) {
                    x -= part<INF>(xb & 0xFFFF0000u);
                    y -= part<INF>(yb & 0xFFFF0000u);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) o[k] = __builtin_bit_cast(F8, w[k]);
    }
};

struct FpT {
    typedef float E;
    struct F8 {
        f32x4 a, b;
    };
    typedef f32x4 F4;
    static __device__ __forceinline__ F4 raw4(const E *p) { return *reinterpret_cast<const f32x4 *>(p); }
    static __device__ __forceinline__ f32x4 up(F4 a) { return a; }
    static constexpr bool kBf16 = false;
    static constexpr int kParts = 1;
    static constexpr int pitch(int cols, bool) { return cols + 4; }
    template <bool KP>
    static __device__ __forceinline__ int col(int x) { return x; }
    static __device__ __forceinline__ f32x4 mma(F8 a, F8 b, f32x4 c) {
#pragma unroll
        for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.a[r], b.a[r], c, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.b[r], b.b[r], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ f32x4 load4(const E *p) { return *reinterpret_cast<const f32x4 *>(p); }
    static __device__ __forceinline__ void store4(E *p, f32x4 v) { *reinterpret_cast<f32x4 *>(p) = v; }
    template <bool KP>
    static __device__ __forceinline__ F8 kfrag(const E *row, int q, int lq) {
        return {load4(row + 32 * q + 4 * lq), load4(row + 32 * q + 16 + 4 * lq)};
    }
    template <bool KP>
    static __device__ __forceinline__ F8 tr(const E *m, int pitch, int j0, int x0, int l16, int lq) {
        F8 o;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            o.a[r] = m[(j0 + 4 * lq + r) * pitch + x0 + l16];
            o.b[r] = m[(j0 + 16 + 4 * lq + r) * pitch + x0 + l16];
        }
        return o;
    }
    static __device__ __forceinline__ f32x4 lo(F8 a) { return a.a; }
    static __device__ __forceinline__ f32x4 hi(F8 a) { return a.b; }
    static __device__ __forceinline__ float probe(F8 a, F8 b) {
        float t = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) t = fmaf(a.a[r], 0.f, fmaf(a.b[r], 0.f, fmaf(b.a[r], 0.f, fmaf(b.b[r], 0.f, t))));
        return t;
    }
    static constexpr int kOutParts = 1;
    static __device__ __forceinline__ void two(f32x4 a, f32x4 b, F8 (&o)[1]) { o[0] = {a, b}; }
    static __device__ __forceinline__ void store_two(E *top, E *, f32x4 v) { store4(top, v); }
    template <bool INF>
    static __device__ __forceinline__ void split(f32x4 a, f32x4 b, F8 (&o)[1]) { o[0] = {a, b}; }
};

constexpr int kSsmThreads = 256;

// A 64-row tile of COLS columns on its way from HBM to LDS through registers.
template <class T, int COLS, bool KP, int THREADS = kSsmThreads>
struct Tile {
    static constexpr int kPitch = T::pitch(COLS, KP);
    static constexpr int kPiece = 16 / sizeof(typename T::E);       // elements of 16 bytes
    static constexpr int kPerRow = COLS / kPiece;
    static constexpr int kN = 64 * kPerRow / THREADS;
    static constexpr int kStep = THREADS / kPerRow;                 // rows between a thread's pieces
    v4u32 r[kN];
    // rows `ld` bytes apart; rows past the resource's end read as zeros
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rsrc, uint32_t ld) {
        uint32_t tid = threadIdx.x;
        asm volatile("" : "+v"(tid));   // offsets are cheap: made anew for each tile, not kept in registers
        const uint32_t at = (tid / kPerRow) * ld + (tid % kPerRow) * 16;
#pragma unroll
        for (int k = 0; k < kN; ++k) r[k] = __builtin_bit_cast(v4u32, buf_load<16>(rsrc, at + k * (kStep * ld)));
    }
    __device__ __forceinline__ void store(typename T::E *m) const {
        uint32_t tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        const uint32_t x = (tid % kPerRow) * kPiece;
        typename T::E *const row = m + (tid / kPerRow) * kPitch;
        constexpr bool kPermuted = T::kBf16 && KP;
        typename T::E *const to = row + (kPermuted ? kpos(x) : x), *const to4 = row + (kPermuted ? kpos(x + 4) : x);
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            if constexpr (kPermuted) {
                *reinterpret_cast<v2u32 *>(to + k * (kStep * kPitch)) = v2u32{r[k][0], r[k][1]};
                *reinterpret_cast<v2u32 *>(to4 + k * (kStep * kPitch)) = v2u32{r[k][2], r[k][3]};
            } else {
                *reinterpret_cast<v4u32 *>(to + k * (kStep * kPitch)) = r[k];
            }
        }
    }
};

// log(1 + e^v) without overflow; log1p keeps the small values' bits
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))); }

// The raw dt of a token as it lies in memory, in a float's upper half for bf16
// once bits() has put it there.  Kept apart from the load, so that a prefetched
// one is not waited for (and with it every load before it) where it is issued.
struct RawDt {
    uint32_t word = 0;
    __device__ __forceinline__ void load(const SsmArgs &a, int64_t token, int h) {
        if (a.gate_bf16) word = static_cast<const uint16_t *>(a.dt)[token * a.lddt + h];
        else word = static_cast<const uint32_t *>(a.dt)[token * a.lddt + h];
    }
    __device__ __forceinline__ float value(const SsmArgs &a) const {
        return __uint_as_float(a.gate_bf16 ? word << 16 : word);
    }
};
__device__ __forceinline__ float dt_raw(const SsmArgs &a, int64_t token, int h) {
    RawDt r;
    r.load(a, token, h);
    return r.value(a);
}
__device__ __forceinline__ float head_bias(const SsmArgs &a, int h) { return a.dt_bias ? a.dt_bias[h] : 0.f; }

// Per-token scalars of a 64-token chunk, G the running sum of dt A from the
// chunk's start.  The sum is taken in fp64 and kept as two floats, because
// e^(G_i - G_j) of near tokens has to be right where both are large.
struct Gates {
    float dt[64], ghi[64], glo[64];
    float eg[64];      // e^G_i: what the chunk's incoming state has decayed to
    float ew[64];      // e^(G_end - G_j): what token j's write has decayed to at the end
    float w[64];       // dt_j times that
    float decay;       // e^G_end
};

// One wave, lane = token.  Tokens past the end have dt = 0 and write nothing.
__device__ __forceinline__ void chunk_gates(float raw, float bias, float A, bool valid, Gates &s) {
    const int l = threadIdx.x % 64;
    const float dt = valid ? softplus(raw + bias) : 0.f;
    double g = static_cast<double>(dt) * static_cast<double>(A);
    g = dpp_add64<0x111, 0xF>(g);   // inclusive scan, as wave_inclusive_scan
    g = dpp_add64<0x112, 0xF>(g);
    g = dpp_add64<0x114, 0xF>(g);
    g = dpp_add64<0x118, 0xF>(g);
    g = dpp_add64<0x142, 0xA>(g);
    g = dpp_add64<0x143, 0xC>(g);
    const uint64_t b = __builtin_bit_cast(uint64_t, g);
    const uint64_t end_lo = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<uint32_t>(b), 63));
    const uint64_t end_hi = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<uint32_t>(b >> 32), 63));
    const double end = __builtin_bit_cast(double, end_hi << 32 | end_lo);
    const float hi = static_cast<float>(g);
    const float ew = __expf(static_cast<float>(end - g));
    s.dt[l] = dt;
    s.ghi[l] = hi;
    s.glo[l] = static_cast<float>(g - hi);
    s.eg[l] = __expf(hi);
    s.ew[l] = ew;
    s.w[l] = dt * ew;
    if (l == 63) s.decay = __expf(static_cast<float>(end));
}

// Gates that a pass of its own has made (SsmArgs::gates), on their way to LDS.
template <int THREADS>
struct GateTile {
    static constexpr int kFloats = sizeof(Gates) / 4, kN = (kFloats + THREADS - 1) / THREADS;
    static_assert(kFloats <= kGateRow);
    float r[kN];
    __device__ __forceinline__ void load(const SsmArgs &a, int64_t row, int h) {
        const __amdgpu_buffer_rsrc_t from = chunk_rsrc(a.gates + (row * a.heads + h) * kGateRow, kGateRow * 4);
#pragma unroll
        for (int k = 0; k < kN; ++k) r[k] = __builtin_bit_cast(float, buf_load<4>(from, (threadIdx.x + k * THREADS) * 4));
    }
    __device__ __forceinline__ void store(Gates &s) const {
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            const int i = threadIdx.x + k * THREADS;
            if (i < kFloats) reinterpret_cast<float *>(&s)[i] = r[k];
        }
    }
};

// A span: consecutive whole chunks of one sequence (its last may be ragged),
// walked by one block per head.  Without a table each sequence is one span.
struct Span {
    int64_t t0;      // first token
    int64_t len;
    int64_t seq;
    int64_t row0;    // the sequence's chunk rows start here, plus the span's place in it
    bool first, last;
};
__device__ __forceinline__ Span span_of_block(const SsmArgs &a, uint32_t s) {
    Span r;
    if (a.spans) {
        const int4 v = a.spans[s];
        r.t0 = v.x;
        r.len = v.y;
        r.seq = static_cast<uint32_t>(v.z) >> 2;
        r.first = v.z & 1;
        r.last = v.z & 2;
        r.row0 = v.w;
    } else if (a.cu) {
        int64_t b = a.cu[s], e = a.cu[s + 1];
        b = b < 0 ? 0 : b > a.total ? a.total : b;
        e = e < b ? b : e > a.total ? a.total : e;
        r.seq = s;
        r.t0 = b;
        r.len = e - b;
        r.row0 = 0;
        r.first = r.last = true;
    } else {   // rows of seq_len tokens, row_spans spans each
        const uint32_t seq = s / a.row_spans, k = s - seq * a.row_spans;
        const int64_t at = k * a.span_len, left = a.seq_len - at;
        r.seq = seq;
        r.t0 = seq * a.seq_len + at;
        r.len = left < a.span_len ? left : a.span_len;
        r.row0 = seq * a.row_chunks + at / 64;
        r.first = k == 0;
        r.last = k + 1 == a.row_spans;
    }
    return r;
}
// First token and number of tokens (none: rows <= 0) of a chunk row.
__device__ __forceinline__ void chunk_of_row(const SsmArgs &a, int64_t row, int64_t &t0, int &rows) {
    if (a.chunks) {
        const int4 v = a.chunks[row];
        t0 = v.x;
        rows = v.y;
    } else {
        const uint32_t seq = static_cast<uint32_t>(row) / static_cast<uint32_t>(a.row_chunks);
        const int64_t at = 64 * (row - static_cast<int64_t>(seq) * a.row_chunks), left = a.seq_len - at;
        t0 = seq * a.seq_len + at;
        rows = static_cast<int>(left < 64 ? left : 64);
    }
}

// A sequence's first span and their number.
__device__ __forceinline__ void spans_of_seq(const SsmArgs &a, uint32_t seq, int64_t &first, int &count) {
    if (a.spans) {
        first = a.span_first[seq];
        count = a.span_first[seq + 1] - static_cast<int>(first);
    } else {
        first = static_cast<int64_t>(seq) * a.row_spans;
        count = a.row_spans;
    }
}

// Work item of a block, as gqa_xcd_item but in 32 bits: heads that share b and
// c follow each other on one XCD.
__device__ __forceinline__ uint32_t shared_item(uint32_t item, uint32_t grid, uint32_t heads, uint32_t groups) {
    const uint32_t r = heads / groups, span = 8 * r;
    if (r > 1) {
        const uint32_t w = item % span;
        if (item - w + span <= grid) item = (item - w) + (w % 8) * r + w / 8;
    }
    return item;
}

// Element of a [n][p] state that a lane's register r of tile (nt, pt) holds:
// OB false: rows n = 4 lq + r, column p = l16; OB true: row n = l16, p = 4 lq + r.
// Work buffers keep states as tiles, nt * (P / 16) + pt, of 64 lanes x 4 values.
template <int P, bool OB>
__device__ __forceinline__ f32x4 load_state_tile(const float *m, int nt, int pt, int l16, int lq) {
    if constexpr (OB) {
        return *reinterpret_cast<const f32x4 *>(m + (16 * nt + l16) * P + 16 * pt + 4 * lq);
    } else {
        f32x4 v;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = m[(16 * nt + 4 * lq + r) * P + 16 * pt + l16];
        return v;
    }
}
template <int P, bool OB>
__device__ __forceinline__ void store_state_tile(float *m, int nt, int pt, int l16, int lq, f32x4 v) {
    if constexpr (OB) {
        *reinterpret_cast<f32x4 *>(m + (16 * nt + l16) * P + 16 * pt + 4 * lq) = v;
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) m[(16 * nt + 4 * lq + r) * P + 16 * pt + l16] = v[r];
    }
}

// A state in a work buffer: tile `tile`, 16 bytes a lane (voff = 16 lane).
__device__ __forceinline__ f32x4 load_tile(__amdgpu_buffer_rsrc_t r, uint32_t voff, int tile) {
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, voff, tile * 1024, 0));
}
template <int AUX = 0>   // 2: past the caches
__device__ __forceinline__ void store_tile(__amdgpu_buffer_rsrc_t r, uint32_t voff, int tile, f32x4 v) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u32, v), r, voff, tile * 1024, AUX);
}

// Walks of the state over the chunks of a span, one block per (span, head):
//   kLocal   the state that the span's own tokens make from zero, and its decay
//   kStates  the state before each chunk, stored for the gradients
//   kOut     the outputs y, and the final state
// Backward in time (rev; not kOut) the same walk makes the gradient E of the
// state: E <- e^G_end E + sum_i e^G_i c_i dy_i^T, stored at each chunk's end.
//
// 65536 tokens in 15 sequences, 32 heads on 16 groups, n = p = 128, bf16:
// kLocal 170 to 200 us, kOut 580 to 650 us, which is 2.7 TB/s of x, y, b, c and
// gates.  kOut issues 103 matrix, 555 vector and 102 LDS instructions a wave and
// chunk (counted; 78, 413 and 96, and 500 to 550 us, with y's operands in one
// bf16 part).  At 2.4 GHz the vector unit is busy for 230 us of it, LDS for 205
// and 58 more of bank conflicts, the matrix unit for 170, and a chunk has three
// barriers: no single one of them bounds it, and HBM does not (with one part and
// no loads from HBM 487 us).  16384 tokens, 32 heads, n = 128, p = 64: kLocal 80
// us, kStates 145 us for both directions, 272 MB of states each.
enum WalkMode { kLocal, kStates, kOut };

// Waves of a block: one per 16 columns p, so that its part of the state stays
// in registers.  32 columns a wave halve the LDS reads but leave 2 waves a SIMD
// in blocks of 67 KB, two to a CU: kOut took 545 us at best instead of 517 (65536
// tokens of 32 heads, n = p = 128, y's operands in one part; smaller blocks, three
// to a CU, were not measured).
constexpr int walk_threads(int p) { return 4 * p; }
constexpr int walk_waves(bool bf16, int p) { return p == 128 ? (bf16 ? 4 : 2) : (bf16 ? 2 : 1); }   // a SIMD's, at least

// PRE: the gates come from memory (a.gates); else the last wave makes each
// chunk's while the others are at work on the one before (calls that are not
// split: a row of 64 tokens, 8 heads, n = 128, p = 64, 7 us so and 13 with the
// pass, of 448 tokens 25 and 30; 32 sequences in 16384 tokens, 32 heads, n = p =
// 128, 216 us so and 211 with the pass and the table; y's operands in one part).
template <class T, int N, int P, int MODE, bool OB, bool PRE>
__global__ void __launch_bounds__(walk_threads(P), walk_waves(T::kBf16, P)) gdr_ssm_walk_kernel(SsmArgs a) {
    typedef typename T::E E;
    typedef typename T::F8 F8;
    constexpr int NT = N / 16, PT = P / 16, TH = walk_threads(P), WAVES = TH / 64;   // a wave owns a column tile
    constexpr bool kY = MODE == kOut;
    constexpr bool KU = kY;   // the scores read U along its rows, the state update across them
    typedef Tile<T, N, KU, TH> TileU;
    typedef Tile<T, N, true, TH> TileC;
    typedef Tile<T, P, false, TH> TileV;
    constexpr int PU = TileU::kPitch, PC = TileC::kPitch, PV = TileV::kPitch, PS = T::pitch(64, true);
    // The scores wait in registers until x and c have been read, and take their
    // places, where that lets one block more onto a CU (with a place of their own
    // 592 blocks of 600 tokens took 15.3 us instead of 13.6, 65536 tokens of 32
    // heads 545 instead of 514; a block alone on its CU 31.6 instead of 33.2).
    constexpr bool kInV = kY && T::kBf16 && P == 64;
    static_assert(!kInV || (PS <= PV && PS <= PC));
    __shared__ __attribute__((aligned(16))) E sU[64 * PU], sV[64 * PV], sC[kY ? 64 * PC : 16];
    __shared__ __attribute__((aligned(16))) E sOwnP[kY && !kInV ? T::kOutParts * 64 * PS : 16];
    E *const sP = kInV ? sV : sOwnP, *const sP2 = kInV ? sC : sOwnP + (T::kOutParts - 1) * 64 * PS;   // the scores' parts
    __shared__ __attribute__((aligned(16))) Gates sg[PRE ? 1 : 2];

    const uint32_t heads = a.heads, groups = a.groups;
    const uint32_t item = shared_item(blockIdx.x, gridDim.x, heads, groups);
    const uint32_t si = item / heads;
    const int h = static_cast<int>(item - si * heads);
    const int g = h / static_cast<int>(heads / groups);
    const bool rev = MODE != kOut && blockIdx.y == 1;
    const Span sp = span_of_block(a, si);
    if (a.spans && sp.len < 0) return;                              // surplus entry
    if (MODE == kLocal && (rev ? sp.first : sp.last)) return;       // nothing follows it
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / 64);   // the same in every lane
    const int l = tid % 64, lane16 = l % 16, lane4 = l / 16;
    int l16 = lane16, lq = lane4;
    const int64_t hb = (static_cast<int64_t>(rev ? 1 : 0) * a.n_spans + si) * a.heads + h;   // slot in the span buffers

    f32x4 Z[NT];
    const float *init = rev ? a.dht : a.h0;
    const bool split = MODE != kLocal && a.span_state;
    const __amdgpu_buffer_rsrc_t mine = chunk_rsrc(a.span_state + hb * (N * P), N * P * 4);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        Z[nt] = zero4();
        if (MODE == kLocal) continue;
        if (split) Z[nt] = load_tile(mine, 16 * l, nt * PT + wave);
        else if (init) Z[nt] = load_state_tile<P, OB>(init + (sp.seq * a.heads + h) * (N * P), nt, wave, l16, lq);
    }

    // The states of both directions go past the caches from 256 MiB (32 heads,
    // n = p = 128, a gradient of 2048 tokens, 134 MB: 132 us, 139 so; 4096: 220 and
    // 217; 8192: 399 and 375).
    const bool past = MODE == kStates && past_caches(a.n_chunks * a.heads * (N * P * 4));
    const int chunks = static_cast<int>((sp.len + 63) / 64);
    const int64_t ldu = rev ? a.ldc : a.ldb, ldv = rev ? a.lddy : a.ldx;
    const E *ub = static_cast<const E *>(rev ? a.c : a.b) + g * N;
    const E *vb = static_cast<const E *>(rev ? a.dy : a.x) + h * P;
    const E *cb = static_cast<const E *>(a.c) + g * N;
    TileU tu;
    TileC tc;
    TileV tv;
    GateTile<TH> tg;
    RawDt raw;   // not PRE, the last wave: dt of the chunk after the prefetched one
    const float bias = PRE ? 0.f : head_bias(a, h), A = PRE ? 0.f : a.A[h];
    auto chunk_at = [&](int k) { return rev ? chunks - 1 - k : k; };
    auto rows_of = [&](int c) {
        const int64_t left = sp.len - 64 * static_cast<int64_t>(c);
        return static_cast<int>(left < 64 ? left : 64);
    };
    auto load_tiles = [&](int k) {
        const int c = chunk_at(k), rows = rows_of(c);
        const int64_t t = sp.t0 + 64 * static_cast<int64_t>(c);
        constexpr int es = sizeof(E);
        const uint32_t u = static_cast<uint32_t>(((rows - 1) * ldu + N) * es), v = static_cast<uint32_t>(((rows - 1) * ldv + P) * es);
        tu.load(chunk_rsrc(ub + t * ldu, u), static_cast<uint32_t>(ldu * es));
        tv.load(chunk_rsrc(vb + t * ldv, v), static_cast<uint32_t>(ldv * es));
        if constexpr (kY) {
            const uint32_t w = static_cast<uint32_t>(((rows - 1) * a.ldc + N) * es);
            tc.load(chunk_rsrc(cb + t * a.ldc, w), static_cast<uint32_t>(a.ldc * es));
        }
        if constexpr (PRE) {
            const int64_t row = sp.row0 + c;   // within the table, whatever cu_seqlens holds
            tg.load(a, row < a.n_chunks ? row : a.n_chunks - 1, h);
        }
    };
    auto load_raw = [&](int k) {
        const int c = chunk_at(k);
        if (l < rows_of(c)) raw.load(a, sp.t0 + 64 * static_cast<int64_t>(c) + l, h);
    };
    auto store_tiles = [&] {
        tu.store(sU);
        tv.store(sV);
        if constexpr (kY) tc.store(sC);
        if constexpr (PRE) tg.store(sg[0]);
    };
    if (chunks > 0) {
        load_tiles(0);
        if (!PRE && wave == WAVES - 1) {
            load_raw(0);
            chunk_gates(raw.value(a), bias, A, l < rows_of(chunk_at(0)), sg[0]);
            if (chunks > 1) load_raw(1);
        }
        store_tiles();
    }
    auto store_zeros = [&] {   // tiles above the diagonal that the products' pairs of tiles reach
        if (wave == 0 || wave == 2) {
            const int at = (16 * wave + l16) * PS + T::template col<true>(16 * (wave + 1) + 4 * lq);
            T::store_two(sP + at, sP2 + at, zero4());
        }
    };
    if (kY && !kInV) store_zeros();
    const float dh = kY && a.D ? a.D[h] : 0.f;
    float total = 0.f;   // kLocal: log of the span's decay
    // all loads so far have arrived: otherwise the compiler would wait for the
    // initial state inside the loop, and with it for each chunk's prefetch
    __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
    for (int k = 0; k < chunks; ++k) {
        const int c = chunk_at(k), rows = rows_of(c);
        const int64_t t = sp.t0 + 64 * static_cast<int64_t>(c);
        const Gates &s = sg[PRE ? 0 : k & 1];
        if (MODE == kStates && sp.row0 + c < a.n_chunks) {   // always, unless cu_seqlens breaks its preconditions
            const __amdgpu_buffer_rsrc_t to = chunk_rsrc(
                a.chunk_state + ((static_cast<int64_t>(rev ? 1 : 0) * a.n_chunks + sp.row0 + c) * a.heads + h) * (N * P), N * P * 4);
            if (past) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) store_tile<2>(to, 16 * l, nt * PT + wave, Z[nt]);
            } else {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) store_tile(to, 16 * l, nt * PT + wave, Z[nt]);
            }
        }
        __syncthreads();   // this chunk's tiles and gates are in LDS
        if (k + 1 < chunks) load_tiles(k + 1);

        // The lane's coordinates are opaque to the compiler in each phase: LDS
        // addresses are made there, not kept over the whole loop, where they
        // would take the registers that 4 waves a SIMD need
        asm volatile("" : "+v"(l16), "+v"(lq));
        constexpr int kScores = (10 + WAVES - 1) / WAVES;
        f32x4 scores[kScores];
        auto score_tile = [&](int m, int &it, int &jt) {   // a wave takes tiles wave, wave + WAVES, .. of the ten
            const int idx = wave + WAVES * m;
            it = idx >= 6 ? 3 : idx >= 3 ? 2 : idx >= 1 ? 1 : 0;
            jt = idx - it * (it + 1) / 2;
            return idx < 10;
        };
        auto store_score = [&](int m, int it, int jt) {
            const int at = (16 * it + l16) * PS + T::template col<true>(16 * jt + 4 * lq);
            T::store_two(sP + at, sP2 + at, scores[m]);
        };
        if constexpr (kY) {
            // scores, transposed: tile (j, i) of B C^T
#pragma unroll
            for (int m = 0; m < kScores; ++m) {
                int it, jt;
                if (!score_tile(m, it, jt)) break;
                f32x4 acc = zero4();
#pragma unroll
                for (int q = 0; q < N / 32; ++q)
                    acc = T::mma(T::template kfrag<KU>(sU + (16 * jt + l16) * PU, q, lq),
                                 T::template kfrag<true>(sC + (16 * it + l16) * PC, q, lq), acc);
                const int i = 16 * it + l16, j0 = 16 * jt + 4 * lq;
                const float gi = s.ghi[i], gil = s.glo[i];
                const f32x4 gj = *reinterpret_cast<const f32x4 *>(&s.ghi[j0]), gl = *reinterpret_cast<const f32x4 *>(&s.glo[j0]);
                const f32x4 dj = *reinterpret_cast<const f32x4 *>(&s.dt[j0]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float v = acc[r] * __expf((gi - gj[r]) + (gil - gl[r])) * dj[r];
                    scores[m][r] = j0 + r <= i ? v : 0.f;
                }
                if constexpr (!kInV) store_score(m, it, jt);
            }
        }
        if (!PRE && wave == WAVES - 1 && k + 1 < chunks) {   // the next chunk's gates (the first two waves have one score tile more)
            chunk_gates(raw.value(a), bias, A, l < rows_of(chunk_at(k + 1)), sg[(k + 1) & 1]);
            if (k + 2 < chunks) load_raw(k + 2);
        }
        asm volatile("" : "+v"(l16), "+v"(lq));
        F8 v[2];   // x (or dy) with tokens as k
#pragma unroll
        for (int q = 0; q < 2; ++q) v[q] = T::template tr<false>(sV, PV, 32 * q, 16 * wave, l16, lq);
        if constexpr (kY) {
            // y^T = e^G (S^T C^T) + D x^T + X^T P^T for this wave's columns
            f32x4 Y[4];
#pragma unroll
            for (int it = 0; it < 4; ++it) Y[it] = zero4();
#pragma unroll
            for (int q = 0; q < N / 32; ++q) {
                F8 cf[4];
#pragma unroll
                for (int it = 0; it < 4; ++it) cf[it] = T::template kfrag<true>(sC + (16 * it + l16) * PC, q, lq);
                F8 z[T::kOutParts];
                T::two(Z[2 * q], Z[2 * q + 1], z);
#pragma unroll
                for (int e = T::kOutParts - 1; e >= 0; --e)
#pragma unroll
                    for (int it = 0; it < 4; ++it) Y[it] = T::mma(z[e], cf[it], Y[it]);
            }
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const float eg = s.eg[16 * it + l16];
                Y[it] = Y[it] * eg + T::load4(sV + (16 * it + l16) * PV + 16 * wave + 4 * lq) * dh;
            }
            if constexpr (kInV) {
                __syncthreads();   // x and c have been read
                asm volatile("" : "+v"(l16), "+v"(lq));
#pragma unroll
                for (int m = 0; m < kScores; ++m) {
                    int it, jt;
                    if (score_tile(m, it, jt)) store_score(m, it, jt);
                }
                store_zeros();
            }
            __syncthreads();   // the scores are in LDS
            asm volatile("" : "+v"(l16), "+v"(lq));
            uint32_t ldy = static_cast<uint32_t>(a.heads * P * sizeof(E));
            asm volatile("" : "+s"(ldy));   // as for the tiles' offsets
            const uint32_t y0 = l16 * ldy + (16 * wave + 4 * lq) * sizeof(E);
            E *yb = static_cast<E *>(a.y) + (t * a.heads + h) * P;
            const __amdgpu_buffer_rsrc_t ry = chunk_rsrc(yb, static_cast<uint32_t>((rows - 1) * ldy + P * sizeof(E)));
            // An x that is not finite must not meet the zeros of earlier tokens'
            // scores: such a chunk is summed one token at a time, up to its own
            if (__builtin_expect(__builtin_amdgcn_ballot_w64(!(T::probe(v[0], v[1]) == 0.f)) != 0, 0)) {
#pragma unroll
                for (int it = 0; it < 4; ++it)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int i = 16 * it + l16;
                        float sum = 0.f;
#pragma unroll 1
                        for (int j = 0; j <= i && j < rows; ++j) {
                            const int at = i * PS + T::template col<true>(j & ~3) + (j & 3);
                            float score = load_scalar<T::kBf16>(sP, at);
                            if constexpr (T::kOutParts > 1) score += load_scalar<T::kBf16>(sP2, at);
                            sum += score * load_scalar<T::kBf16>(vb, (t + j) * ldv + 16 * wave + 4 * lq + r);
                        }
                        Y[it][r] += sum;
                    }
            } else {
#pragma unroll
                for (int it = 0; it < 4; ++it)
#pragma unroll
                    for (int e = T::kOutParts - 1; e >= 0; --e)
#pragma unroll
                        for (int q = 0; q <= it / 2; ++q)
                            Y[it] = T::mma(v[q], T::template kfrag<true>((e ? sP2 : sP) + (16 * it + l16) * PS, q, lq), Y[it]);
            }
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const uint32_t off = y0 + it * (16 * ldy);
                if constexpr (T::kBf16) __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(v2u32, cvt4(Y[it])), ry, off, 0, 0);
                else __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u32, Y[it]), ry, off, 0, 0);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" : "+v"(l16), "+v"(lq));
        // Z <- decay Z + U^T (w V)
        const float decay = s.decay;
        if (MODE == kLocal) total += s.ghi[63] + s.glo[63];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) Z[nt] = Z[nt] * decay;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const float *w = rev ? s.eg : s.w;
            const f32x4 wa = *reinterpret_cast<const f32x4 *>(w + 32 * q + 4 * lq);
            const f32x4 wb = *reinterpret_cast<const f32x4 *>(w + 32 * q + 16 + 4 * lq);
            F8 vs[T::kParts];
            T::template split<!OB>(T::lo(v[q]) * wa, T::hi(v[q]) * wb, vs);
#pragma unroll
            for (int nt = 0; nt < NT; nt += 2) {   // two tiles at a time: products on one sum do not follow each other
                F8 u[2];
#pragma unroll
                for (int k2 = 0; k2 < 2; ++k2) u[k2] = T::template tr<KU>(sU, PU, 32 * q, 16 * (nt + k2), l16, lq);
#pragma unroll
                for (int e = T::kParts - 1; e >= 0; --e)
#pragma unroll
                    for (int k2 = 0; k2 < 2; ++k2)
                        Z[nt + k2] = OB ? T::mma(vs[e], u[k2], Z[nt + k2]) : T::mma(u[k2], vs[e], Z[nt + k2]);
            }
        }
        __syncthreads();   // the chunk's tiles have been read
        if (k + 1 < chunks) store_tiles();
    }

    l16 = lane16;
    lq = lane4;
    asm volatile("" : "+v"(l16), "+v"(lq));
    float *out = nullptr;
    if (MODE == kLocal) out = a.span_state;
    else if (MODE == kOut && sp.last && a.ht) out = a.ht + (sp.seq * a.heads + h) * (N * P);
    else if (MODE == kStates && rev && sp.first && a.dh0) out = a.dh0 + (sp.seq * a.heads + h) * (N * P);
    if (out) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (MODE == kLocal) store_tile(mine, 16 * l, nt * PT + wave, Z[nt]);
            else store_state_tile<P, OB>(out, nt, wave, l16, lq, Z[nt]);
        }
    }
    if (MODE == kLocal && tid == 0) a.span_decay[hb] = expf(total);
}

// States at the spans' starts (rev: their gradients at the spans' ends) from
// the spans' own: s <- decay s + local along each sequence, in place, 4 values
// a thread.  grid.x: (sequence, head, 1024 values), grid.y: direction.  HBM
// bound: 28 us for about 100 MB of states at 65536 tokens and 32 heads.
template <int N, int P, bool OB>
__global__ void __launch_bounds__(kSsmThreads) gdr_ssm_join_kernel(SsmArgs a) {
    constexpr uint32_t kParts = N * P / (4 * kSsmThreads);
    const uint32_t item = blockIdx.x / kParts, heads = a.heads;
    const int piece = static_cast<int>(blockIdx.x % kParts) * kSsmThreads + threadIdx.x;   // (tile, lane)
    const uint32_t seq = item / heads, h = item - seq * heads;
    const bool rev = blockIdx.y == 1;
    int64_t first;
    int count;
    spans_of_seq(a, seq, first, count);
    const int tile = piece / 64, l16 = piece % 16, lq = (piece % 64) / 16;
    const float *init = rev ? a.dht : a.h0;
    f32x4 s = zero4();
    if (init) s = load_state_tile<P, OB>(init + (static_cast<int64_t>(seq) * heads + h) * (N * P), tile / (P / 16), tile % (P / 16), l16, lq);
    const int64_t base = (rev ? a.n_spans : 0) + first;
    constexpr int U = 8;   // spans in flight
    for (int k0 = 0; k0 < count; k0 += U) {
        f32x4 v[U];
        float d[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + u;
            v[u] = zero4();
            d[u] = 0.f;
            if (k + 1 < count) {   // the last one's own state leads nowhere
                const int64_t slot = (base + (rev ? count - 1 - k : k)) * heads + h;
                v[u] = *reinterpret_cast<const f32x4 *>(a.span_state + slot * (N * P) + piece * 4);
                d[u] = a.span_decay[slot];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + u;
            if (k >= count) break;
            const int64_t slot = (base + (rev ? count - 1 - k : k)) * heads + h;
            *reinterpret_cast<f32x4 *>(a.span_state + slot * (N * P) + piece * 4) = s;
            s = s * d[u] + v[u];
        }
    }
}

}  // namespace
}  // namespace gdr
