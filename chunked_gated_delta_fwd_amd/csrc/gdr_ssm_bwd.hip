// Gradients of the state space scan (gdr_ssm.hip), in chunks of 64 tokens.
// With S the state before a chunk, E the gradient of the state after it, G
// the running sum of dt A inside it, and for i >= j
//
//   L_ij = e^(G_i - G_j),  K_ij = c_i . b_j,  M_ij = dy_i . x_j,  W = L K M:
//
//   dx_j = D dy_j + dt_j (sum_i L_ij K_ij dy_i + e^(G_end - G_j) E^T b_j)
//   db_j = sum_i L_ij M_ij dt_j c_i + dt_j e^(G_end - G_j) E x_j    (over the group's heads)
//   dc_i = sum_j L_ij M_ij dt_j b_j + e^G_i S dy_i                  (likewise)
//   v_j  = sum_i W_ij + e^(G_end - G_j) b_j^T E x_j                 (dt's own part)
//   l_t  = l_{t+1} + sum_{j<t} W_tj dt_j + e^G_t c_t^T S dy_t
//          - dt_t (sum_{i>t} W_it + e^(G_end - G_t) b_t^T E x_t),   l_{end+1} = <E, S_end>
//   ddt  = (v + A l) sigmoid(raw),  dA = sum dt l,  dbias = sum ddt,  dD = sum dy . x
//
// l is the gradient of dt A.  Its recursion starts anew in every chunk from
// the inner product of E and the state after the chunk, so its rounding does
// not grow with the sequence; the diagonal of W is left out of it because it
// would cancel, and what does cancel, W's sums along rows and columns, is
// summed in fp64 (51 tokens of 2 heads: dA is off by 4.3e-7 of itself, 1.3e-6
// with sums in fp32, the geometric mean of ten draws; it costs 1.5 % of a call).
// W's sums use fp32 products of exact bf16 inputs, the states enter c^T S dy
// and b^T E x as exact sums of bf16 parts, so ddt, dA and dbias are
// fp32-accurate also for bf16 inputs; operands that only reach dx (L K, E),
// which is bf16 itself, are taken as two bf16 parts.
//
// S and E of every chunk come from the walks of gdr_ssm_device.h.
#include <type_traits>

#include "gdr_ssm_device.h"

namespace gdr {
namespace {

// The units of work are (chunk, group, head), in that order; a block takes an
// equal run of them, so that one round of blocks does all, and where a run ends
// inside a (chunk, group) the parts of db and dc meet in memory.
struct GradSplit {
    uint32_t items, len, per_group;   // len: of a block's run
    // the block that starts a (chunk, group), and how many blocks share it
    __device__ __forceinline__ uint32_t first(uint32_t unit) const { return unit * per_group / len; }
    __device__ __forceinline__ int parts(uint32_t unit) const {
        return static_cast<int>(((unit + 1) * per_group - 1) / len - first(unit)) + 1;
    }
};
// Of the chunks that there are, not of the table's entries; but not shorter
// runs than the room for the parts allows (a.grad_least), whatever cu_seqlens holds.
__device__ __forceinline__ GradSplit grad_split(const SsmArgs &a) {
    GradSplit s;
    const uint32_t used = a.chunks ? static_cast<uint32_t>(*a.chunks_used) : static_cast<uint32_t>(a.n_chunks);
    const uint32_t blocks = static_cast<uint32_t>(a.grad_blocks), least = static_cast<uint32_t>(a.grad_least);
    s.per_group = static_cast<uint32_t>(a.heads / a.groups);
    s.items = used * static_cast<uint32_t>(a.heads);
    const uint32_t len = (s.items + blocks - 1) / blocks;
    s.len = len < least ? least : len;
    return s;
}

// Blocks of 8 waves; a wave owns one or two of the (i, j) tiles of the lower
// triangle, one tile of rows n of db and dc (of half the tokens when n is 64)
// and one tile of rows p of dx (likewise).  db and dc are summed over a
// group's heads in registers; their L M parts as one matrix, multiplied once.
// 8 waves, because with 4 the sums and states of a wave take over 256
// registers and spill.
//
// 16384 tokens in 4 sequences, 32 heads on one b and c, n = 128, p = 64, bf16:
// 235 to 250 us; 540 MB of states and 200 MB of x, dy, dx, gates and sums, 3
// TB/s.  A head takes some 6 us of a block (88 KB a CU in that time: near what
// HBM gives), and what surrounds a group's heads 8 us.
constexpr int kGradThreads = 512;

template <class T, int N, int P>
__global__ void __launch_bounds__(kGradThreads) gdr_ssm_grad_kernel(SsmArgs a) {
    typedef typename T::E E;
    typedef typename T::F8 F8;
    constexpr int NT = N / 16, PT = P / 16, IW = NT / 2, JW = PT / 2;   // i tiles of db, dc and j tiles of dx per wave
    typedef Tile<T, N, true, kGradThreads> TileN;
    typedef Tile<T, P, true, kGradThreads> TileP;
    constexpr int PN = TileN::kPitch, PP = TileP::kPitch, PS = T::pitch(64, true), PE = T::pitch(P, false);
    constexpr int kXY = 2 * 64 * PP > 64 * PN ? 2 * 64 * PP : 64 * PN;   // x and dy; c before and after the heads
    constexpr int kE = T::kBf16 ? (N * PE > 64 * PS ? N * PE : 64 * PS) : 64 * PS;
    __shared__ __attribute__((aligned(16))) E sB[64 * PN], sXY[kXY], sE[kE], sPd[64 * PS];
    // the second parts of what only reaches dx (E and L K)
    __shared__ __attribute__((aligned(16))) E sE2[T::kBf16 ? N * PE : 16], sPd2[T::kBf16 ? 64 * PS : 16];
    __shared__ __attribute__((aligned(16))) Gates sg;
    __shared__ __attribute__((aligned(16))) float s_s[NT][64], s_e[NT][64], s_w[64], s_m[64], s_es[8];
    __shared__ double s_row[4][64], s_col[4][64];
    E *const sX = sXY, *const sY = sXY + 64 * PP, *const sC = sXY;

    const uint32_t per_group = static_cast<uint32_t>(a.heads / a.groups), groups = a.groups;
    const GradSplit split = grad_split(a);
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / 64);   // the same in every lane
    const int l = tid % 64;
    int l16 = l % 16, lq = l / 16;
    const int nt = wave % NT, it0 = wave / NT * IW;     // db, dc: rows 16 nt .., tokens 16 it0 ..
    const int pt = wave % PT, jt0 = wave / PT * JW;     // dx: rows 16 pt .., tokens 16 jt0 ..
    const bool first_n = wave < NT;
    constexpr int es = sizeof(E);
    uint32_t item = blockIdx.x * split.len;
    const uint32_t end = item + split.len < split.items ? item + split.len : split.items;
    while (item < end) {
        const uint32_t unit = item / per_group;
        const int64_t row = unit / groups;
        const int g = static_cast<int>(unit - static_cast<uint32_t>(row) * groups);
        const int h0 = static_cast<int>(g * per_group + (item - unit * per_group));
        item = (unit + 1) * per_group < end ? (unit + 1) * per_group : end;
        const int h1 = static_cast<int>(g * per_group + (item - unit * per_group));
        int rows;
        int64_t t0;
        chunk_of_row(a, row, t0, rows);
        if (rows <= 0) continue;   // a length-0 sequence's row
        auto tile_rsrc = [&](const void *base, int64_t ld, int64_t col, int cols) {
            return chunk_rsrc(static_cast<const E *>(base) + t0 * ld + col, static_cast<uint32_t>(((rows - 1) * ld + cols) * es));
        };
        TileP tx, ty;
        GateTile<kGradThreads> tg;
        float d_next;
        auto load_xy = [&](int h) {
            tx.load(tile_rsrc(a.x, a.ldx, static_cast<int64_t>(h) * P, P), static_cast<uint32_t>(a.ldx * es));
            ty.load(tile_rsrc(a.dy, a.lddy, static_cast<int64_t>(h) * P, P), static_cast<uint32_t>(a.lddy * es));
            tg.load(a, row, h);
            d_next = a.D ? a.D[h] : 0.f;
        };
        const float *const Sbase = a.chunk_state, *const Ebase = a.chunk_state + a.n_chunks * a.heads * (N * P);
        f32x4 Sv[PT], Ev[PT];   // this wave's rows n of S and E
        auto load_states = [&](int h) {
            const int64_t at = (row * a.heads + h) * (N * P) + (nt * PT * 64 + l) * 4;
#pragma unroll
            for (int k = 0; k < PT; ++k) {
                Sv[k] = *reinterpret_cast<const f32x4 *>(Sbase + at + k * 256);
                Ev[k] = *reinterpret_cast<const f32x4 *>(Ebase + at + k * 256);
            }
        };
        {
            TileN tb, tc;
            tb.load(tile_rsrc(a.b, a.ldb, static_cast<int64_t>(g) * N, N), static_cast<uint32_t>(a.ldb * es));
            tc.load(tile_rsrc(a.c, a.ldc, static_cast<int64_t>(g) * N, N), static_cast<uint32_t>(a.ldc * es));
            tb.store(sB);
            tc.store(sC);
        }
        load_xy(h0);
        load_states(h0);
        __syncthreads();

        // this wave's tiles of the lower triangle's ten: number wave, and wave + 8
        int ti[2], tj[2];
        f32x4 K[2], R[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int idx = wave + 8 * k;
            ti[k] = idx >= 6 ? 3 : idx >= 3 ? 2 : idx >= 1 ? 1 : 0;
            tj[k] = idx - ti[k] * (ti[k] + 1) / 2;
            K[k] = R[k] = zero4();
            if (idx < 10) {
#pragma unroll
                for (int q = 0; q < N / 32; ++q)
                    K[k] = T::mma(T::template kfrag<true>(sC + (16 * ti[k] + l16) * PN, q, lq),
                                  T::template kfrag<true>(sB + (16 * tj[k] + l16) * PN, q, lq), K[k]);
            }
        }
        // the values of c beside this wave's rows n of dc (c leaves LDS for x and dy)
        typename T::F4 cd[IW];
#pragma unroll
        for (int i = 0; i < IW; ++i) cd[i] = T::raw4(sC + (16 * (it0 + i) + l16) * PN + T::template col<true>(16 * nt + 4 * lq));
        // tiles above the diagonal that pairs of tiles reach
        if (wave == 1 || wave == 3) {
            const int at = (16 * wave + l16) * PS + T::template col<true>(16 * (wave - 1) + 4 * lq);
            T::store_two(sPd + at, sPd2 + at, zero4());
        }
        f32x4 dc[IW], db[IW];
#pragma unroll
        for (int i = 0; i < IW; ++i) dc[i] = db[i] = zero4();
        __syncthreads();

        for (int h = h0; h < h1; ++h) {
            const Gates &s = sg;
            tx.store(sX);
            ty.store(sY);
            tg.store(sg);
            __syncthreads();
            // Unconditional (the last head's own once more), so that a later wait
            // for the states can count these as still on their way
            const float dh = d_next;
            load_xy(h + 1 < h1 ? h + 1 : h);
            // opaque coordinates, as in the walks: addresses are made in each phase
            asm volatile("" : "+v"(l16), "+v"(lq));
            // M, W and what they give
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (wave + 8 * k >= 10) continue;
                f32x4 m = zero4();
#pragma unroll
                for (int q = 0; q < P / 32; ++q)
                    m = T::mma(T::template kfrag<true>(sY + (16 * ti[k] + l16) * PP, q, lq),
                               T::template kfrag<true>(sX + (16 * tj[k] + l16) * PP, q, lq), m);
                const int i0 = 16 * ti[k] + 4 * lq, j = 16 * tj[k] + l16;
                const f32x4 gi = *reinterpret_cast<const f32x4 *>(&s.ghi[i0]), gil = *reinterpret_cast<const f32x4 *>(&s.glo[i0]);
                const float gj = s.ghi[j], gjl = s.glo[j], dtj = s.dt[j];
                f32x4 pd;
                double rs[4];
                double col = 0.;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const bool below = i0 + r > j, on = i0 + r == j;
                    const float e = __expf((gi[r] - gj) + (gil[r] - gjl));
                    const float lk = below || on ? e * K[k][r] : 0.f;
                    const float lm = below || on ? e * m[r] : 0.f;
                    const float w = lk * m[r];
                    pd[r] = lk;
                    R[k][r] += lm * dtj;
                    rs[r] = below ? static_cast<double>(w) * dtj : 0.;
                    col += below ? w : 0.f;   // in fp64, as rs: their difference counts
                    if (on) {
                        s_w[j] = w;
                        s_m[j] = m[r];
                    }
                }
                T::store_two(sPd + j * PS + T::template col<true>(i0), sPd2 + j * PS + T::template col<true>(i0), pd);
#pragma unroll
                for (int r = 0; r < 4; ++r) rs[r] = row_sum64(rs[r]);
                if (l16 == 0) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) s_row[tj[k]][i0 + r] = rs[r];
                }
                col = sum_rows64(col);
                if (lq == 0) s_col[ti[k]][j] = col;
            }
            asm volatile("" : "+v"(l16), "+v"(lq));
            // S dy^T and E x^T for this wave's rows n
            if (first_n) {
                float es_sum = 0.f;
#pragma unroll
                for (int k = 0; k < PT; ++k) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) es_sum += Ev[k][r] * Sv[k][r];
                    const int at = (16 * nt + l16) * PE + 16 * k + 4 * lq;
                    if constexpr (T::kBf16) T::store_two(sE + at, sE2 + at, Ev[k]);
                }
                es_sum = lane_sum<64>(es_sum);
                if (l == 0) s_es[wave] = es_sum;
            }
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                f32x4 acc[IW];
#pragma unroll
                for (int i = 0; i < IW; ++i) acc[i] = zero4();
#pragma unroll
                for (int q = 0; q < P / 32; ++q) {
                    F8 st[T::kParts], f[IW];
#pragma unroll
                    for (int i = 0; i < IW; ++i) f[i] = T::template kfrag<true>((side ? sX : sY) + (16 * (it0 + i) + l16) * PP, q, lq);
                    T::template split<false>(side ? Ev[2 * q] : Sv[2 * q], side ? Ev[2 * q + 1] : Sv[2 * q + 1], st);
                    if constexpr (T::kBf16) __builtin_amdgcn_sched_barrier(0);   // the reads together, ahead of the products
#pragma unroll
                    for (int e = T::kParts - 1; e >= 0; --e)
#pragma unroll
                        for (int i = 0; i < IW; ++i) acc[i] = T::mma(st[e], f[i], acc[i]);
                }
#pragma unroll
                for (int i = 0; i < IW; ++i) {
                    const int at = 16 * (it0 + i) + l16;
                    const float f = side ? s.w[at] : s.eg[at];
                    const f32x4 o = side ? T::load4(sB + at * PN + T::template col<true>(16 * nt + 4 * lq)) : T::up(cd[i]);
                    float d = 0.f;
#pragma unroll
                    for (int r = 0; r < 4; ++r) d += acc[i][r] * o[r];
                    if (side) db[i] = db[i] + acc[i] * f;
                    else dc[i] = dc[i] + acc[i] * f;
                    d = sum_rows(d);
                    if (lq == 0) (side ? s_e : s_s)[nt][at] = d;
                }
            }
            __syncthreads();
            load_states(h + 1 < h1 ? h + 1 : h);

            asm volatile("" : "+v"(l16), "+v"(lq));
            // dx for this wave's rows p
            {
                f32x4 X[JW], V[JW];
#pragma unroll
                for (int j = 0; j < JW; ++j) X[j] = V[j] = zero4();
                const float *Ep = Ebase + (row * a.heads + h) * (N * P);
#pragma unroll
                for (int q = 0; q < N / 32; ++q) {
                    F8 e[T::kOutParts];
                    if constexpr (T::kBf16) {
                        e[0] = T::template tr<false>(sE, PE, 32 * q, 16 * pt, l16, lq);
                        e[1] = T::template tr<false>(sE2, PE, 32 * q, 16 * pt, l16, lq);
                    } else {
                        // lane p = l16 of E's tile holds p = 4 (lane / 16) + r: gather the four rows n
                        f32x4 v[2];
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                v[b][r] = Ep[(((2 * q + b) * PT + pt) * 64 + 16 * (l16 / 4) + 4 * lq + r) * 4 + l16 % 4];
                        T::two(v[0], v[1], e);
                    }
                    F8 f[JW];
#pragma unroll
                    for (int j = 0; j < JW; ++j) f[j] = T::template kfrag<true>(sB + (16 * (jt0 + j) + l16) * PN, q, lq);
#pragma unroll
                    for (int k = T::kOutParts - 1; k >= 0; --k)
#pragma unroll
                        for (int j = 0; j < JW; ++j) V[j] = T::mma(e[k], f[j], V[j]);
                }
                const uint32_t ldx = static_cast<uint32_t>(a.heads * P * es);
                const __amdgpu_buffer_rsrc_t rx = chunk_rsrc(static_cast<E *>(a.dx) + (t0 * a.heads + h) * P,
                                                             static_cast<uint32_t>((rows - 1) * ldx + P * es));
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const F8 y = T::template tr<true>(sY, PP, 32 * q, 16 * pt, l16, lq);
#pragma unroll
                    for (int k = T::kOutParts - 1; k >= 0; --k)
#pragma unroll
                        for (int j = 0; j < JW; ++j)
                            if (q >= (jt0 + j) / 2)
                                X[j] = T::mma(y, T::template kfrag<true>((k ? sPd2 : sPd) + (16 * (jt0 + j) + l16) * PS, q, lq), X[j]);
                }
#pragma unroll
                for (int j = 0; j < JW; ++j) {
                    const int at = 16 * (jt0 + j) + l16, p0 = 16 * pt + 4 * lq;
                    const f32x4 v = (X[j] + V[j] * s.ew[at]) * s.dt[at] + T::load4(sY + at * PP + T::template col<true>(p0)) * dh;
                    const uint32_t off = at * ldx + p0 * es;
                    if constexpr (T::kBf16) __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(v2u32, cvt4(v)), rx, off, 0, 0);
                    else __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u32, v), rx, off, 0, 0);
                }
            }
            if (wave == 7) {   // lane = token: the sums of this head's parts, for gdr_ssm_finish_kernel
                const int tile = l / 16;
                double rw = 0., cl = 0.;
                float st = 0.f, et = 0.f, es_sum = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (k <= tile) rw += s_row[k][l];
                    if (k >= tile) cl += s_col[k][l];
                }
#pragma unroll
                for (int k = 0; k < NT; ++k) {
                    st += s_s[k][l];
                    et += s_e[k][l];
                    es_sum += s_es[k];
                }
                float *to = a.token_part + (row * a.heads + h) * kTokenPart + l;
                to[0] = static_cast<float>(rw - s.dt[l] * cl);
                to[64] = static_cast<float>(cl);
                to[128] = s_w[l];
                to[192] = s_m[l];
                to[256] = st;
                to[320] = et;
                if (l == 0) to[384] = es_sum;
            }
            __syncthreads();
        }

        asm volatile("" : "+v"(l16), "+v"(lq));
        // the heads' L M dt parts: dc += R B, db += R^T C, with R (once for all
        // heads) as two bf16 parts: one would add a rounding to db's and dc's own
        TileN tc;
        tc.load(tile_rsrc(a.c, a.ldc, static_cast<int64_t>(g) * N, N), static_cast<uint32_t>(a.ldc * es));
        if (wave == 0 || wave == 2) T::store4(sE + (16 * wave + l16) * PS + T::template col<true>(16 * (wave + 1) + 4 * lq), zero4());
        tc.store(sC);
#pragma unroll
        for (int part = 0; part < (T::kBf16 ? 2 : 1); ++part) {
            if (part) __syncthreads();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (wave + 8 * k >= 10) continue;
                f32x4 v = R[k];
                if constexpr (T::kBf16) v = up4(cvt4(v));
                R[k] = R[k] - v;
                T::store4(sPd + (16 * tj[k] + l16) * PS + T::template col<true>(16 * ti[k] + 4 * lq), v);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int at = (16 * ti[k] + 4 * lq + r) * PS + T::template col<true>(16 * tj[k] + (l16 & 12)) + (l16 & 3);
                    if constexpr (T::kBf16) sE[at] = bf16_bits(v[r]);
                    else sE[at] = v[r];
                }
            }
            __syncthreads();
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const F8 bt = T::template tr<true>(sB, PN, 32 * q, 16 * nt, l16, lq), ct = T::template tr<true>(sC, PN, 32 * q, 16 * nt, l16, lq);
#pragma unroll
                for (int i = 0; i < IW; ++i) {
                    const int it = it0 + i;
                    if (q <= it / 2) dc[i] = T::mma(bt, T::template kfrag<true>(sE + (16 * it + l16) * PS, q, lq), dc[i]);
                    if (q >= it / 2) db[i] = T::mma(ct, T::template kfrag<true>(sPd + (16 * it + l16) * PS, q, lq), db[i]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < IW; ++i) {
            const int t = 16 * (it0 + i) + l16;
            if (t >= rows) continue;
            const int64_t to = ((t0 + t) * a.groups + g) * N + 16 * nt + 4 * lq;
            if (split.parts(unit) > 1) {
                const int64_t plane = a.total * a.groups * N;
                const int part = static_cast<int>(blockIdx.x - split.first(unit));
                *reinterpret_cast<f32x4 *>(a.bc_part + (2 * part) * plane + to) = db[i];
                *reinterpret_cast<f32x4 *>(a.bc_part + (2 * part + 1) * plane + to) = dc[i];
            } else {
                T::store4(static_cast<E *>(a.db) + to, db[i]);
                T::store4(static_cast<E *>(a.dc) + to, dc[i]);
            }
        }
        __syncthreads();   // the tiles have been read
    }
}

// The gradient of dt, and each chunk's part of dA, dD and dbias, from the
// token sums of gdr_ssm_grad_kernel: a wave per (chunk, head), lane = token.
__device__ __forceinline__ void finish_dt(const SsmArgs &a, uint32_t block) {
    const int l = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int64_t item = static_cast<int64_t>(block) * (kSsmThreads / 64) + wave;
    if (item >= a.n_chunks * a.heads) return;
    const int64_t row = static_cast<uint32_t>(item) / static_cast<uint32_t>(a.heads);
    const int h = static_cast<int>(item - row * a.heads);
    int rows;
    int64_t t0;
    chunk_of_row(a, row, t0, rows);
    float *const part = a.head_part + item * 3;
    if (rows <= 0) {
        if (l < 3) part[l] = 0.f;
        return;
    }
    const bool valid = l < rows;
    const float raw = valid ? dt_raw(a, t0 + l, h) : 0.f, bias = head_bias(a, h), A = a.A[h];
    const Gates &s = *reinterpret_cast<const Gates *>(a.gates + item * kGateRow);
    const float *in = a.token_part + item * kTokenPart;
    const float diff = in[l], cl = in[64 + l], diag = in[128 + l], m = in[192 + l], st = in[256 + l], et = in[320 + l];
    const float es_sum = in[384];
    const float dt = s.dt[l], v = cl + diag + s.ew[l] * et;
    const double write = static_cast<double>(s.w[l]) * et;
    double u = diff + static_cast<double>(s.eg[l]) * st - write;
#pragma unroll
    for (int k = 1; k < 64; k *= 2) {
        const double o = __shfl_down(u, k);
        if (l + k < 64) u += o;
    }
    const double dl = static_cast<double>(s.decay) * es_sum + sum_rows64(row_sum64(write)) + u;
    double draw = 0.;
    if (valid) {
        draw = (v + A * dl) / (1.f + expf(-(raw + bias)));
        const int64_t to = (t0 + l) * a.heads + h;
        if (a.gate_bf16) static_cast<uint16_t *>(a.ddt)[to] = bf16_bits(static_cast<float>(draw));
        else static_cast<float *>(a.ddt)[to] = static_cast<float>(draw);
    }
    auto sum = [](double x) { return static_cast<float>(sum_rows64(row_sum64(x))); };
    const float da = sum(valid ? dt * dl : 0.), dd = sum(valid ? m : 0.), dbias = sum(draw);
    if (l == 0) {
        part[0] = da;
        part[1] = dd;
        part[2] = dbias;
    }
}

// db and dc of the (chunk, group)s that blocks shared: the parts, added in order
template <class T, int N>
__device__ __forceinline__ void finish_bc(const SsmArgs &a, uint32_t block) {
    const GradSplit split = grad_split(a);
    constexpr uint32_t kPieces = N / 16;
    const uint32_t unit = block / (2 * kPieces), groups = a.groups;
    if (unit >= split.items / split.per_group) return;
    const int parts = split.parts(unit), side = block / kPieces % 2;
    if (parts == 1) return;
    const int64_t row = unit / groups, plane = a.total * a.groups * N;
    const int g = static_cast<int>(unit - static_cast<uint32_t>(row) * groups);
    int rows;
    int64_t t0;
    chunk_of_row(a, row, t0, rows);
    const float *const from = a.bc_part + side * plane;
    const int i = block % kPieces * kSsmThreads + threadIdx.x, t = i / (N / 4);
    if (t >= rows) return;
    const int64_t to = ((t0 + t) * a.groups + g) * N + 4 * (i % (N / 4));
    f32x4 s = zero4();
#pragma unroll 4
    for (int k = 0; k < parts; ++k) s = s + *reinterpret_cast<const f32x4 *>(from + 2 * k * plane + to);
    T::store4(static_cast<typename T::E *>(side ? a.dc : a.db) + to, s);
}

// What the gradient's blocks left: dt_blocks blocks of the first kind, the others
// of the second.  One launch for both, whose loads wait beside each other: with
// one each the gradient took 486 us where it took 481 so (16384 tokens, 32 heads, n =
// 128, p = 64).
template <class T, int N>
__global__ void __launch_bounds__(kSsmThreads) gdr_ssm_finish_kernel(SsmArgs a, uint32_t dt_blocks) {
    if (blockIdx.x < dt_blocks) finish_dt(a, blockIdx.x);
    else finish_bc<T, N>(a, blockIdx.x - dt_blocks);
}

// dA, dD and dbias of a head from its chunks
__global__ void __launch_bounds__(kSsmThreads) gdr_ssm_heads_kernel(SsmArgs a) {
    __shared__ float sum[3][4];
    const int h = blockIdx.x;
    float s[3] = {};
    for (int64_t r = threadIdx.x; r < a.n_chunks; r += kSsmThreads)
#pragma unroll
        for (int k = 0; k < 3; ++k) s[k] += a.head_part[(r * a.heads + h) * 3 + k];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        s[k] = lane_sum<64>(s[k]);
        if (threadIdx.x % 64 == 0) sum[k][threadIdx.x / 64] = s[k];
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        float *const to[3] = {a.dA, a.dD, a.dbias};
        for (int k = 0; k < 3; ++k)
            if (to[k]) to[k][h] = (sum[k][0] + sum[k][1]) + (sum[k][2] + sum[k][3]);
    }
}

}  // namespace

int ssm_grad_parts(SsmArgs &a) {
    // one block a CU (its registers allow no second one): 16384 tokens, 32 heads,
    // n = 128, p = 64, 256, 512 and 1024 blocks: 461, 481, 526 us a whole gradient
    const int64_t items = a.n_chunks * a.heads, per_group = a.heads / a.groups;
    a.grad_blocks = static_cast<int32_t>(items < 256 ? items : 256);
    const int64_t sure = (a.cu ? (a.total + 63) / 64 : a.n_chunks) * a.heads;   // fewer only where cu_seqlens leaves tokens out
    a.grad_least = a.grad_blocks ? static_cast<int32_t>((sure + a.grad_blocks - 1) / a.grad_blocks) : 1;
    if (a.grad_least < 1) a.grad_least = 1;
    if (per_group == 1) return 1;
    const int64_t parts = (per_group - 2) / a.grad_least + 2;
    return static_cast<int>(parts < per_group ? parts : per_group);
}

hipError_t launch_ssm_bwd(const SsmArgs &a, hipStream_t stream) {
    const dim3 block(kSsmThreads);
    auto run = [&]<class T, int N, int P>() {
        const int64_t walks = a.n_spans * a.heads;
        if (walks > 0x7FFFFFFF || a.n_chunks * a.heads > 0x7FFFFFFF ||
             a.n_seq * a.heads * (N * P / 1024) > 0x7FFFFFFF)
            return hipErrorInvalidValue;
        const dim3 grid(static_cast<uint32_t>(walks), 2), walk(walk_threads(P));
        if (walks > 0) {
            if (a.span_state) {
                hipLaunchKernelGGL((gdr_ssm_walk_kernel<T, N, P, kLocal, true, true>), grid, walk, 0, stream, a);
                hipLaunchKernelGGL((gdr_ssm_join_kernel<N, P, true>),
                                   dim3(static_cast<uint32_t>(a.n_seq * a.heads * (N * P / 1024)), 2), block, 0, stream, a);
            }
            hipLaunchKernelGGL((gdr_ssm_walk_kernel<T, N, P, kStates, true, true>), grid, walk, 0, stream, a);
            hipLaunchKernelGGL((gdr_ssm_grad_kernel<T, N, P>), dim3(a.grad_blocks), dim3(kGradThreads), 0, stream, a);
        }
        if (walks > 0) {
            const int64_t dt_blocks = (a.n_chunks * a.heads + 3) / 4;
            const int64_t blocks = dt_blocks + (a.bc_part ? a.n_chunks * a.groups * (N / 8) : 0);
            if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
            hipLaunchKernelGGL((gdr_ssm_finish_kernel<T, N>), dim3(static_cast<uint32_t>(blocks)), block, 0, stream, a,
                               static_cast<uint32_t>(dt_blocks));
        }
        hipLaunchKernelGGL(gdr_ssm_heads_kernel, dim3(a.heads), block, 0, stream, a);
        return hipGetLastError();
    };
    auto dims = [&]<class T>() {
        if (a.n == 64) return a.p == 64 ? run.template operator()<T, 64, 64>() : run.template operator()<T, 64, 128>();
        return a.p == 64 ? run.template operator()<T, 128, 64>() : run.template operator()<T, 128, 128>();
    };
    return a.bf16 ? dims.template operator()<BfT>() : dims.template operator()<FpT>();
}

}  // namespace gdr
