// Softmax attention, backward.  With the forward's lse the probabilities are
// made again, p_ij = e^{s_ij - lse_i}, and with delta_i = do_i . o_i
//
//     dv_j = sum_i p_ij do_i,   ds_ij = p_ij (do_i . v_j - delta_i),
//     dq_i = scale sum_j ds_ij k_j,   dk_j = scale sum_i ds_ij q_i,
//
// dk and dv over every query head that shares the key head.  Two passes, one
// that holds query rows and walks the keys (dq, delta), one that holds key rows
// and walks the queries (dk, dv): scores and do . v are made twice, seven
// products for five, so that every sum stays in registers in a fixed order.
//
// 4 x 4096 tokens, 32 heads on 4, d 128, causal, bf16: 1.83 to 1.92 ms a call. In
// a traced run of 1.94: the first pass 0.80 (3 products, 1030 TFLOP/s), the second
// 1.11 (4 products, 990), the join of dk and dv of a group's halves 0.027.
#include "gdr_attn_device.h"

namespace gdr {
namespace {

// dq: a block takes 128 query rows of one head, 32 a wave, as the forward does,
// and is bound as it is, with no maximum to keep: 3 products a pair and head.
template <class T, int D>
struct AttnDq {
    typedef typename T::E E;
    typedef typename T::F8 F8;
    static constexpr int kKeys = T::kBf16 ? 64 : 32;
    typedef AttnTile<T, D, kKeys> Tile;
    static constexpr int kSteps = D / 16, kParts = D / 32, kSub = kKeys / 32;
    struct Lds {
        alignas(16) char k[2][Tile::kBytes];
        alignas(16) char v[2][Tile::kBytes];
    };
    struct Row {
        F8 q[kSteps], dout[kSteps];
        f32x16 dq[kParts];   // transposed: channels x queries
        float lse, delta;    // lse in powers of two
    };

    // CAREFUL as in the forward: a key that is not finite reaches the rows that see it and no other.
    // SUMS: in place of dq, the sum of each row's ds (this lane's half) in delta.
    template <bool CAREFUL, bool SUMS>
    static __device__ __forceinline__ void walk(Row &w, const AttnSight &sight, float c, int32_t i0, int32_t i1,
                                                int32_t begin, int32_t end, const E *k, const E *v, uint32_t step_k,
                                                uint32_t step_v, int32_t lk, Lds &lds, int wave, int lane) {
        const int col = lane & 31, h = lane >> 5;
        const typename Tile::From fk = Tile::from(wave, lane, step_k), fv = Tile::from(wave, lane, step_v);
        const int32_t lo = i0 + 32 * wave, at = sight.at(lo + col);
#pragma unroll
        for (int t = 0; t < kParts; ++t) w.dq[t] = zero16();
        float rest = 0.f;
        const typename Tile::Lane places = Tile::lane_places(lane);
        auto load = [&](int32_t j, int b) {
            Tile::load(fk, reinterpret_cast<const E *>(reinterpret_cast<const char *>(k) + static_cast<int64_t>(j) * step_k),
                       step_k, lk - j, lds.k[b], wave);
            Tile::load(fv, reinterpret_cast<const E *>(reinterpret_cast<const char *>(v) + static_cast<int64_t>(j) * step_v),
                       step_v, lk - j, lds.v[b], wave);
        };
        if (begin < end) load(begin, 0);
        const auto tile = [&](auto which, int32_t j) {
            constexpr int buf = decltype(which)::value;
            const typename Tile::Lane l = attn_here(places);
            loads_landed();
            __syncthreads();
            if (j + kKeys < end) load(j + kKeys, buf ^ 1);
            const int32_t hi = lo + 31 < i1 ? lo + 31 : i1;
            if (lo > i1) return;
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
                const int32_t ju = j + 32 * u;
                if (!sight.any(lo, hi, ju, 32)) continue;
                f32x16 s = zero16(), dp = zero16();
#pragma unroll
                for (int ks = 0; ks < kSteps; ++ks) s = T::mma(Tile::rows(lds.k[buf], l, 32 * u, ks), w.q[ks], s);
#pragma unroll
                for (int ks = 0; ks < kSteps; ++ks) dp = T::mma(Tile::rows(lds.v[buf], l, 32 * u, ks), w.dout[ks], dp);
                attn_ahead<T, 2 * kSteps>();
                const bool whole = sight.all(lo, hi, ju, 32);
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = fast_exp2(__builtin_fmaf(s[r], c, -w.lse)) * (dp[r] - w.delta);
                if (!whole) {
                    const int32_t d0 = attn_here(at - ju - 4 * h);
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (!sight.sees(d0, 8 * (r / 4) + r % 4)) s[r] = 0.f;
                }
                if constexpr (SUMS) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) rest += s[r];
                    continue;
                }
                // bf16: ds is rounded to nearest for the product with the keys
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    const F8 ds = T::part(s, kb);
                    if (!CAREFUL || whole) {
#pragma unroll
                        for (int t = 0; t < kParts; ++t)
                            w.dq[t] = T::mma(Tile::across(lds.k[buf], l, 32 * u + 16 * kb, t), ds, w.dq[t]);
                    } else {
                        for (int key = 0; key < 16; ++key) {
                            const int slot = (key >> 2 & 1) == h ? (key & 3) + (key >> 1 & 4) : -1;
                            const bool seen = sight.sees(at, ju + 16 * kb + key);
#pragma unroll
                            for (int t = 0; t < kParts; ++t) {
                                const f32x16 x =
                                    T::mma(T::only(Tile::across(lds.k[buf], l, 32 * u + 16 * kb, t), slot),
                                           T::only(ds, slot), zero16());
#pragma unroll
                                for (int r = 0; r < 16; ++r) w.dq[t][r] += seen ? x[r] : 0.f;
                            }
                        }
                    }
                }
            }
        };
        for (int32_t j = begin; j < end; j += 2 * kKeys) {
            tile(IntC<0>{}, j);
            if (j + kKeys < end) tile(IntC<1>{}, j + kKeys);
        }
        if (SUMS) w.delta = rest;
    }
};

// delta cancels against do . v, and made from a bf16 o it carries o's rounding:
// in dq and dk, relative to that of ds, about n^-1/2 of it where n keys share a
// row's weight.  A row's ds sum to zero with the delta that belongs to them, so
// where a block's rows see at most kFewKeys keys a walk of its own takes the sum
// (errors of dq and dk in 2-norm: rows of 2 keys 3.4e-3 without, 2.4e-3 with it,
// of 30 keys 2.6e-3 and 2.4e-3; one rounding of the result is 1.7e-3).
constexpr int32_t kFewKeys = 192;

// The share of begin .. end - 1 that run `part` of `parts` takes, in steps of STEP; it may be empty.
template <int STEP>
__device__ __forceinline__ void attn_share(int32_t &begin, int32_t &end, int32_t part, int32_t parts) {
    const int32_t steps = begin < end ? (end - begin + STEP - 1) / STEP : 0, share = (steps + parts - 1) / parts * STEP;
    begin += part * share;
    end = begin + share < end ? begin + share : end;
}

template <class T, int D>
__device__ __attribute__((noinline)) float attn_dq_delta(AttnArgsAt at, uint32_t tiles, __attribute__((address_space(3))) typename AttnDq<T, D>::Lds *lds);

template <class T, int D, bool CAREFUL, bool SUMS>
__device__ __forceinline__ bool attn_dq_block(AttnArgsAt args, const AttnArgs &a, uint32_t tiles,
                                              typename AttnDq<T, D>::Lds &lds, float &sum) {
    typedef AttnDq<T, D> F;
    typedef typename T::E E;
    typedef typename T::F8 F8;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 31, h = lane >> 5;
    const int group = a.hq / a.hk;
    const uint32_t pairs = static_cast<uint32_t>(a.cu ? 1 : a.n_seq) * a.hk;
    AttnItem item = attn_item(blockIdx.x, pairs, tiles, group * a.runs_q);
    if (item.tile < 0) return false;
    const int32_t part = item.way / group;
    item.way %= group;
    const int32_t n = a.cu ? attn_find(a.cu, static_cast<int32_t>(a.n_seq), a.total_q, item.tile, lane) : item.pair / a.hk;
    const int hk = item.pair % a.hk, hq = hk * group + item.way;
    const AttnSeq seq = attn_seq(a, n);
    const int64_t tile = a.cu ? item.tile - (attn_clamp(a.cu[n], 0, a.total_q) / kAttnRows + n) : item.tile;
    if (tile < 0 || tile * kAttnRows >= seq.lq) return false;
    const AttnSight sight(a, seq);
    const int32_t i0 = static_cast<int32_t>(tile * kAttnRows);
    const int32_t i1 = i0 + kAttnRows < seq.lq ? i0 + kAttnRows - 1 : seq.lq - 1;
    const int64_t back = static_cast<int64_t>(sight.at(i0)) - sight.back + 1;
    const int32_t first = back > 0 ? static_cast<int32_t>(back) : 0;
    int32_t begin = first / F::kKeys * F::kKeys;
    int32_t end = sight.at(i1) + 1 < seq.lk ? sight.at(i1) + 1 : seq.lk;
    const bool few = T::kBf16 && !SUMS && end - first <= kFewKeys;
    if (!SUMS && a.runs_q > 1) attn_share<F::kKeys>(begin, end, part, a.runs_q);
    if (few) sum = attn_dq_delta<T, D>(args, tiles, attn_lds(lds));

    typename F::Row w;
    {
        const int32_t i = i0 + 32 * wave + col < seq.lq ? i0 + 32 * wave + col : seq.lq - 1;
        const int64_t row = seq.q0 + i, head = static_cast<int64_t>(hq) * D + 8 * h;
        const E *q = static_cast<const E *>(a.q) + row * a.ldq + head;
        const E *o = static_cast<const E *>(a.o) + row * a.ldo + head;
        const E *dout = static_cast<const E *>(a.dout) + row * a.lddo + head;
        float dot = 0.f;
#pragma unroll
        for (int ks = 0; ks < F::kSteps; ++ks) {
            w.q[ks] = T::load(q + 16 * ks);
            w.dout[ks] = T::load(dout + 16 * ks);
            const F8 x = T::load(o + 16 * ks);
#pragma unroll
            for (int s = 0; s < 8; ++s) dot = __builtin_fmaf(T::up(w.dout[ks], s), T::up(x, s), dot);
        }
        w.delta = few ? sum : half_sum(dot);
        // a row that sees no key, or whose scores are all -inf: +inf makes its probabilities 0, where -inf would take
        // -inf from -inf
        const float lse = a.lse[row * a.hq + hq];
        w.lse = lse == -__builtin_inff() ? __builtin_inff() : lse * kLog2e;
        if (!SUMS && part == 0 && i0 + 32 * wave + col < seq.lq && h == 0) {
            float *stat = a.stat + static_cast<int64_t>(hq) * a.total_q + row;
            stat[0] = w.lse;
            stat[a.hq * a.total_q] = w.delta;
        }
    }
    const float c = a.scale * kLog2e;
    const E *k = static_cast<const E *>(a.k) + seq.k0 * a.ldk + static_cast<int64_t>(hk) * D;
    const E *v = static_cast<const E *>(a.v) + seq.k0 * a.ldv + static_cast<int64_t>(hk) * D;
    const uint32_t step_k = static_cast<uint32_t>(a.ldk * sizeof(E)), step_v = static_cast<uint32_t>(a.ldv * sizeof(E));
    if constexpr (SUMS) {
        const float before = w.delta;
        F::template walk<CAREFUL, true>(w, sight, c, i0, i1, begin, end, k, v, step_k, step_v, seq.lk, lds, wave, lane);
        sum = before + half_sum(w.delta);
        __syncthreads();   // the tiles are read: other ones may take their place
        return false;
    }
    F::template walk<CAREFUL, false>(w, sight, c, i0, i1, begin, end, k, v, step_k, step_v, seq.lk, lds, wave, lane);
    float x = 0.f;   // 0, or NaN where a gradient is not finite
#pragma unroll
    for (int t = 0; t < F::kParts; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) x = __builtin_fmaf(w.dq[t][r], 0.f, x);
    if (!CAREFUL && __syncthreads_or(x != 0.f)) return true;
    const int32_t i = i0 + 32 * wave + col;
    if (i < seq.lq) {
        const int64_t at = ((seq.q0 + i) * a.hq + hq) * D;
        if (a.part_q) {
            float *dq = a.part_q + part * a.total_q * a.hq * D + at;
#pragma unroll
            for (int t = 0; t < F::kParts; ++t) attn_store<AttnF32>(dq + 32 * t, w.dq[t], a.scale, h);
        } else {
            E *dq = static_cast<E *>(a.dq) + at;
#pragma unroll
            for (int t = 0; t < F::kParts; ++t) attn_store<T>(dq + 32 * t, w.dq[t], a.scale, h);
        }
    }
    return false;
}

template <class T, int D>
__device__ __attribute__((noinline)) void attn_dq_careful(AttnArgsAt at, uint32_t tiles, __attribute__((address_space(3))) typename AttnDq<T, D>::Lds *lds) {
    float sum;
    at = attn_scalar(at);
    (void)attn_dq_block<T, D, true, false>(at, attn_args(at), __builtin_amdgcn_readfirstlane(tiles), attn_scalar(lds), sum);
}
template <class T, int D>
__device__ __attribute__((noinline)) float attn_dq_delta(AttnArgsAt at, uint32_t tiles, __attribute__((address_space(3))) typename AttnDq<T, D>::Lds *lds) {
    float sum;
    at = attn_scalar(at);
    (void)attn_dq_block<T, D, false, true>(at, attn_args(at), __builtin_amdgcn_readfirstlane(tiles), attn_scalar(lds), sum);
    return sum;
}

template <class T, int D>
__global__ __launch_bounds__(256, T::kBf16 ? (D == 64 ? 3 : 2) : 1) void gdr_attn_dq_kernel(AttnArgs a, uint32_t tiles) {
    __shared__ typename AttnDq<T, D>::Lds lds;
    float sum;
    if (attn_dq_block<T, D, false, false>(attn_args_at(), a, tiles, lds, sum)) attn_dq_careful<T, D>(attn_args_at(), tiles, attn_lds(lds));
}

// dk and dv: a block takes 128 key rows of one key head, 32 a wave, and walks
// the query rows that see them, head after head of its part of the group.  Keys
// and both sums fill the registers (256 at d 128), so the block's values lie in
// LDS and are read again each tile: 4 products a pair and head, bound by them
// and LDS reads (five operands for four products).
template <class T, int D>
struct AttnDkv {
    typedef typename T::E E;
    typedef typename T::F8 F8;
    static constexpr int kQueries = T::kBf16 && D == 64 ? 64 : 32, kSub = kQueries / 32;   // a tile
    typedef AttnTile<T, D, kQueries> Tile;
    static constexpr int kSteps = D / 16, kParts = D / 32;
    typedef AttnTile<T, D, kAttnRows> Values;
    struct Lds {
        alignas(16) float lse[2][64], delta[2][64];   // a load of a wave each
        alignas(16) char q[2][Tile::kBytes];
        alignas(16) char dout[2][Tile::kBytes];
        alignas(16) char v[Values::kBytes];           // the block's values, which registers have no room for
    };
    struct Row {
        F8 k[kSteps];
        f32x16 dk[kParts], dv[kParts];   // transposed: channels x keys
    };
    struct Where {
        const E *q, *dout;               // first row of the sequence, first head of the part
        const E *v;                      // the block's first key
        const float *lse, *delta;
        int64_t total;                   // between two heads' lse
        uint32_t step_q, step_do, step_v;
        int32_t heads, lq, keys;          // keys: from the block's first to the sequence's last
    };

    // CAREFUL: a query or output gradient that is not finite reaches the keys that its row sees and no other.
    template <bool CAREFUL>
    static __device__ __forceinline__ void walk(Row &w, const Where &from, const AttnSight &sight, float c, int32_t j0,
                                                int32_t j1, int32_t begin, int32_t end, Lds &lds, int wave, int lane) {
        const int col = lane & 31, h = lane >> 5;
        const typename Tile::From fq = Tile::from(wave, lane, from.step_q), fo = Tile::from(wave, lane, from.step_do);
        const int32_t lo = j0 + 32 * wave, j = lo + col;
#pragma unroll
        for (int t = 0; t < kParts; ++t) w.dk[t] = w.dv[t] = zero16();
        if (begin >= end) return;
        Values::load(Values::from(wave, lane, from.step_v), from.v, from.step_v, from.keys, lds.v, wave);
        auto load = [&](int head, int32_t i, int b) {
            const int32_t rows = from.lq - i;
            Tile::load(fq, reinterpret_cast<const E *>(reinterpret_cast<const char *>(from.q + head * D) +
                                                       static_cast<int64_t>(i) * from.step_q), from.step_q, rows, lds.q[b], wave);
            Tile::load(fo, reinterpret_cast<const E *>(reinterpret_cast<const char *>(from.dout + head * D) +
                                                       static_cast<int64_t>(i) * from.step_do), from.step_do, rows, lds.dout[b], wave);
            if (wave < 2) {
                const float *x = (wave == 0 ? from.lse : from.delta) + head * from.total + i;
                lds_load4(uniform_rsrc(x, 4 * (rows < kQueries ? rows : kQueries)), 4 * lane, lds_address(wave == 0 ? lds.lse[b] : lds.delta[b]));
            }
        };
        load(0, begin, 0);
        const typename Tile::Lane places = Tile::lane_places(lane);
        const typename Tile::Lane own{places.along + 32 * wave * Tile::kRow, 4 * h * 4u};   // values; statistics
        int32_t i = begin, head = 0;
        // one tile of queries; returns whether there is a next one
        const auto tile = [&](auto which) {
            constexpr int buf = decltype(which)::value;
            const typename Tile::Lane l = attn_here(places), mine = attn_here(own);
            int32_t next = i + kQueries, nhead = head;
            if (next >= end) next = begin, ++nhead;
            loads_landed();
            __syncthreads();
            if (nhead < from.heads) load(nhead, next, buf ^ 1);
            const int32_t last = i + kQueries - 1 < from.lq ? i + kQueries - 1 : from.lq - 1;
            if (lo <= j1 && sight.any(i, last, lo, 32)) {
                f32x16 p[kSub], dp[kSub];
#pragma unroll
                for (int u = 0; u < kSub; ++u) {
                    p[u] = dp[u] = zero16();
#pragma unroll
                    for (int ks = 0; ks < kSteps; ++ks) p[u] = T::mma(Tile::rows(lds.q[buf], l, 32 * u, ks), w.k[ks], p[u]);
#pragma unroll
                    for (int ks = 0; ks < kSteps; ++ks)
                        dp[u] = T::mma(Tile::rows(lds.dout[buf], l, 32 * u, ks), Tile::rows(lds.v, mine, 0, ks), dp[u]);
                }
                const bool whole = last == i + kQueries - 1 && sight.all(i, last, lo, 32);
                __builtin_amdgcn_sched_barrier(0);   // rows' statistics wait: earlier they cost spilled operands
                const char *stats = reinterpret_cast<const char *>(lds.lse[buf]) + mine.across;
#pragma unroll
                for (int x = 0; x < 4 * kSub; ++x) {
                    const f32x4 lse = *reinterpret_cast<const f32x4 *>(stats + 32 * x);
                    const f32x4 delta = *reinterpret_cast<const f32x4 *>(stats + 32 * x + sizeof(lds.lse));
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int u = x / 4, r = 4 * (x % 4) + q;
                        p[u][r] = fast_exp2(__builtin_fmaf(p[u][r], c, -lse[q]));
                        dp[u][r] = p[u][r] * (dp[u][r] - delta[q]);
                    }
                }
                if (!whole) {
                    // rows behind the last are zeros, but a zero times a key that is not finite is not
                    const int32_t i4 = attn_here(i + 4 * h), rows = from.lq - i4;
#pragma unroll
                    for (int u = 0; u < kSub; ++u)
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            const int x = 32 * u + 8 * (r / 4) + r % 4;
                            if (x >= rows || !sight.sees(sight.at(i4 + x), j)) p[u][r] = dp[u][r] = 0.f;
                        }
                }
                // bf16: p and ds are rounded to nearest for the products over the queries
#pragma unroll
                for (int kb = 0; kb < 2 * kSub; ++kb) {
                    const F8 pp = T::part(p[kb / 2], kb % 2), ds = T::part(dp[kb / 2], kb % 2);
                    if (!CAREFUL || whole) {
#pragma unroll
                        for (int t = 0; t < kParts; ++t) {
                            w.dv[t] = T::mma(Tile::across(lds.dout[buf], l, 16 * kb, t), pp, w.dv[t]);
                            w.dk[t] = T::mma(Tile::across(lds.q[buf], l, 16 * kb, t), ds, w.dk[t]);
                        }
                    } else {
                        for (int row = 0; row < 16; ++row) {
                            const int slot = (row >> 2 & 1) == h ? (row & 3) + (row >> 1 & 4) : -1;
                            const bool seen = i + 16 * kb + row < from.lq && sight.sees(sight.at(i + 16 * kb + row), j);
#pragma unroll
                            for (int t = 0; t < kParts; ++t) {
                                const f32x16 x = T::mma(T::only(Tile::across(lds.dout[buf], l, 16 * kb, t), slot),
                                                        T::only(pp, slot), zero16());
                                const f32x16 y = T::mma(T::only(Tile::across(lds.q[buf], l, 16 * kb, t), slot),
                                                        T::only(ds, slot), zero16());
#pragma unroll
                                for (int r = 0; r < 16; ++r) {
                                    w.dv[t][r] += seen ? x[r] : 0.f;
                                    w.dk[t][r] += seen ? y[r] : 0.f;
                                }
                            }
                        }
                    }
                }
            }
            i = next;
            head = nhead;
            return head < from.heads;
        };
        while (tile(IntC<0>{}) && tile(IntC<1>{})) {
        }
    }
};

template <class T, int D, bool CAREFUL>
__device__ __forceinline__ bool attn_dkv_block(const AttnArgs &a, uint32_t tiles, typename AttnDkv<T, D>::Lds &lds) {
    typedef AttnDkv<T, D> F;
    typedef typename T::E E;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 31, h = lane >> 5;
    const int group = a.hq / a.hk;
    const uint32_t pairs = static_cast<uint32_t>(a.cu ? 1 : a.n_seq) * a.hk;
    const AttnItem item = attn_item(blockIdx.x, pairs, tiles, a.parts);
    if (item.tile < 0) return false;
    const int32_t *cuk = a.cuk ? a.cuk : a.cu;
    const int32_t n = a.cu ? attn_find(cuk, static_cast<int32_t>(a.n_seq), a.total_k, item.tile, lane) : item.pair / a.hk;
    const int hk = item.pair % a.hk;
    const AttnSeq seq = attn_seq(a, n);
    int64_t tile = a.cu ? item.tile - (attn_clamp(cuk[n], 0, a.total_k) / kAttnRows + n) : item.tile;
    if (tile < 0 || tile * kAttnRows >= seq.lk) return false;
    tile = (seq.lk - 1) / kAttnRows - tile;   // early keys first: causal ones are seen by the most queries
    const AttnSight sight(a, seq);
    const int32_t j0 = static_cast<int32_t>(tile * kAttnRows);
    const int32_t j1 = j0 + kAttnRows < seq.lk ? j0 + kAttnRows - 1 : seq.lk - 1;
    // queries of which some sees a key of the block: at(i) >= j0 and at(i) - j1 < back
    int64_t begin = 0, end = seq.lq;
    if (sight.slope) {
        begin = static_cast<int64_t>(j0) - sight.first;
        if (begin < 0) begin = 0;
        const int64_t e = static_cast<int64_t>(j1) + sight.back - sight.first;
        if (e < end) end = e;
    }
    begin = begin / F::kQueries * F::kQueries;

    const int teams = a.parts / a.runs, team = item.way % teams;
    const int head0 = group * team / teams, heads = group * (team + 1) / teams - head0;
    const int64_t hq = static_cast<int64_t>(hk) * group + head0;
    typename F::Where from;
    from.q = static_cast<const E *>(a.q) + seq.q0 * a.ldq + hq * D;
    from.dout = static_cast<const E *>(a.dout) + seq.q0 * a.lddo + hq * D;
    from.lse = a.stat + hq * a.total_q + seq.q0;
    from.delta = from.lse + a.hq * a.total_q;
    from.total = a.total_q;
    from.step_q = static_cast<uint32_t>(a.ldq * sizeof(E));
    from.step_do = static_cast<uint32_t>(a.lddo * sizeof(E));
    from.v = static_cast<const E *>(a.v) + (seq.k0 + j0) * a.ldv + static_cast<int64_t>(hk) * D;
    from.step_v = static_cast<uint32_t>(a.ldv * sizeof(E));
    from.heads = heads;
    from.lq = seq.lq;
    from.keys = seq.lk - j0;
    typename F::Row w;
    {
        const int64_t row = seq.k0 + (j0 + 32 * wave + col < seq.lk ? j0 + 32 * wave + col : seq.lk - 1);
        const int64_t head = static_cast<int64_t>(hk) * D + 8 * h;
        const E *k = static_cast<const E *>(a.k) + row * a.ldk + head;
#pragma unroll
        for (int ks = 0; ks < F::kSteps; ++ks) w.k[ks] = T::load(k + 16 * ks);
    }
    const float c = a.scale * kLog2e;
    int32_t b = static_cast<int32_t>(begin), e = static_cast<int32_t>(end);
    if (a.runs > 1) attn_share<F::kQueries>(b, e, item.way / teams, a.runs);
    F::template walk<CAREFUL>(w, from, sight, c, j0, j1, b, e, lds, wave, lane);
    float x = 0.f;
#pragma unroll
    for (int t = 0; t < F::kParts; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) x = __builtin_fmaf(w.dk[t][r], 0.f, __builtin_fmaf(w.dv[t][r], 0.f, x));
    if (!CAREFUL && __syncthreads_or(x != 0.f)) return true;
    const int32_t j = j0 + 32 * wave + col;
    if (j >= seq.lk) return false;
    const int64_t at = ((seq.k0 + j) * a.hk + hk) * D;
    if (a.part) {
        const int64_t all = a.total_k * a.hk * D;
        float *part = a.part + 2 * item.way * all + at;
#pragma unroll
        for (int t = 0; t < F::kParts; ++t) {
            attn_store<AttnF32>(part + 32 * t, w.dk[t], a.scale, h);
            attn_store<AttnF32>(part + all + 32 * t, w.dv[t], 1.f, h);
        }
    } else {
#pragma unroll
        for (int t = 0; t < F::kParts; ++t) {
            attn_store<T>(static_cast<E *>(a.dk) + at + 32 * t, w.dk[t], a.scale, h);
            attn_store<T>(static_cast<E *>(a.dv) + at + 32 * t, w.dv[t], 1.f, h);
        }
    }
    return false;
}

template <class T, int D>
__device__ __attribute__((noinline)) void attn_dkv_careful(AttnArgsAt at, uint32_t tiles, __attribute__((address_space(3))) typename AttnDkv<T, D>::Lds *lds) {
    (void)attn_dkv_block<T, D, true>(attn_args(attn_scalar(at)), __builtin_amdgcn_readfirstlane(tiles), attn_scalar(lds));
}

template <class T, int D>
__global__ __launch_bounds__(256, T::kBf16 ? 2 : 1) void gdr_attn_dkv_kernel(AttnArgs a, uint32_t tiles) {
    __shared__ typename AttnDkv<T, D>::Lds lds;
    if (attn_dkv_block<T, D, false>(a, tiles, lds)) attn_dkv_careful<T, D>(attn_args_at(), tiles, attn_lds(lds));
}

// Sums the parts of dk and dv (QUERIES: of dq) in order, for the rows of one
// tile's sequence; bound by their loads from the caches (16384 keys, 4 heads, two
// parts of 128 channels: 27 us).
template <class T, bool QUERIES>
__global__ __launch_bounds__(256) void gdr_attn_join_kernel(AttnArgs a, uint32_t tiles) {
    const int lane = threadIdx.x & 63;
    const int32_t slot = blockIdx.x % tiles, which = blockIdx.x / tiles;
    const int32_t *cu = QUERIES || !a.cuk ? a.cu : a.cuk;
    const int64_t total = QUERIES ? a.total_q : a.total_k;
    const int32_t n = a.cu ? attn_find(cu, static_cast<int32_t>(a.n_seq), total, slot, lane) : which;
    const AttnSeq seq = attn_seq(a, n);
    const int32_t length = QUERIES ? seq.lq : seq.lk;
    const int64_t tile = a.cu ? slot - (attn_clamp(cu[n], 0, total) / kAttnRows + n) : slot;
    if (tile < 0 || tile * kAttnRows >= length) return;
    const int64_t row = static_cast<int64_t>(QUERIES ? a.hq : a.hk) * a.d, all = total * row;
    const int64_t j0 = tile * kAttnRows, rows = length - j0 < kAttnRows ? length - j0 : kAttnRows;
    const int64_t from = ((QUERIES ? seq.q0 : seq.k0) + j0) * row, count = rows * row;
    const int32_t parts = QUERIES ? a.runs_q : a.parts;
    constexpr int kSums = QUERIES ? 1 : 2;
    for (int64_t x = threadIdx.x * 4 + blockIdx.y * 1024; x < count; x += gridDim.y * 1024)
#pragma unroll
        for (int what = 0; what < kSums; ++what) {
            const float *part = (QUERIES ? a.part_q : a.part) + what * all + from + x;
            f32x4 sum = zero4();
#pragma unroll 4
            for (int p = 0; p < parts; ++p) sum += *reinterpret_cast<const f32x4 *>(part + p * kSums * all);
            typename T::E *to = static_cast<typename T::E *>(QUERIES ? a.dq : what ? a.dv : a.dk) + from + x;
            if constexpr (T::kBf16) *reinterpret_cast<bf16x4 *>(to) = cvt4(sum);
            else *reinterpret_cast<f32x4 *>(to) = sum;
        }
}

template <class T, int D>
hipError_t run(const AttnArgs &a, hipStream_t stream) {
    const int64_t pairs = (a.cu ? 1 : a.n_seq) * a.hk, rows = a.cu ? 1 : a.n_seq;
    const int64_t tiles_q = attn_tiles(a.cu != nullptr, a.n_seq, a.seq_q, a.total_q);
    const int64_t tiles_k = attn_tiles(a.cu != nullptr, a.n_seq, a.seq_k, a.total_k);
    const int64_t grid_q = attn_grid(pairs, tiles_q, static_cast<int64_t>(a.hq / a.hk) * a.runs_q), grid_k = attn_grid(pairs, tiles_k, a.parts);
    if (a.total_q > 0) {
        gdr_attn_dq_kernel<T, D><<<dim3(static_cast<unsigned>(grid_q)), 256, 0, stream>>>(a, static_cast<uint32_t>(tiles_q));
        if (a.part_q)
            gdr_attn_join_kernel<T, true><<<dim3(static_cast<unsigned>(tiles_q * rows), 32), 256, 0, stream>>>(a, static_cast<uint32_t>(tiles_q));
    }
    if (a.total_k > 0) {
        gdr_attn_dkv_kernel<T, D><<<dim3(static_cast<unsigned>(grid_k)), 256, 0, stream>>>(a, static_cast<uint32_t>(tiles_k));
        if (a.part)
            gdr_attn_join_kernel<T, false><<<dim3(static_cast<unsigned>(tiles_k * rows), 32), 256, 0, stream>>>(a, static_cast<uint32_t>(tiles_k));
    }
    return hipGetLastError();
}

}  // namespace

// What costs least by attn_time; a step is 32 queries (dq: a tile of keys), as
// measured on large calls.  Sums go through the caches at 8 TB/s, and joining
// them takes 5 us more.  Without and with runs, causal, us a call: bf16, d 128,
// 2048 tokens, 8 heads on 2, 160 and 102, 4096, 8 on 1, 296 and 197; d 64, 8192, 4
// on 1, 320 and 171; f32, d 128, 700, 2 on 1, 323 and 110.  They have to promise
// 15 %: 2048, 32 on 8, 197 and 208.
void attn_bwd_split(AttnArgs &a) {
    const AttnCost keys = a.bf16 ? (a.d == 64 ? AttnCost{512, 1.1, 1.0} : AttnCost{512, 2.2, 1.45})
                                 : (a.d == 64 ? AttnCost{256, 5.5, 5.5} : AttnCost{256, 11.0, 11.0});
    const AttnCost queries = a.bf16 ? (a.d == 64 ? AttnCost{768, 2.6, 1.3} : AttnCost{512, 3.0, 1.9})
                                    : (a.d == 64 ? AttnCost{256, 3.5, 3.5} : AttnCost{256, 7.0, 7.0});
    const int32_t group = a.hq / a.hk;
    const double seqs = a.n_seq > 0 ? static_cast<double>(a.n_seq) : 1.0;
    const double lq = a.cu ? a.total_q / seqs : a.seq_q, lk = a.cu ? a.total_k / seqs : a.seq_k;
    // rows of the other side that a block works on, at most and on average; packed sequences have other lengths
    // than the mean
    const auto least = [&](const AttnCost &cost, double blocks, double own, double other, int32_t step, int32_t most_teams,
                           int32_t &teams, int32_t &runs, double bytes) {
        double most = a.cu ? 2.5 * other : other, mean = a.causal ? other - (own < other ? own : other) / 2 : other;
        if (a.window > 0 && a.window + kAttnRows < most) most = a.window + kAttnRows;
        if (mean > most) mean = most;
        const double steps = mean / step + 1, longest = most / step + 1;
        double best = 0;
        teams = runs = 1;
        const auto consider = [&](int32_t t, int32_t r) {
            const double heads = static_cast<double>(most_teams) / t / r;
            double time = attn_time(cost, blocks * t * r, steps * heads, longest * heads);
            if (t * r > 1) time += 5 + bytes * t * r / 8e6;
            if (t * r == 1 || time < (r > 1 ? 0.85 : 0.95) * best) {
                best = time;
                teams = t;
                runs = r;
            }
        };
        for (int32_t t = 1; t <= most_teams; t = t < most_teams && 2 * t > most_teams ? most_teams : 2 * t) consider(t, 1);
        for (int32_t r = 2; r <= 16 && longest / r >= 4; r += r < 4 ? 1 : 4) consider(most_teams, r);
    };
    int32_t teams, one;
    least(keys, a.hk * attn_blocks(a.cu != nullptr, seqs, lk), lk, lq, 32, group, teams, a.runs, 16.0 * a.total_k * a.hk * a.d);
    a.parts = teams * a.runs;
    least(queries, a.hq * attn_blocks(a.cu != nullptr, seqs, lq), lq, lk, a.bf16 ? 64 : 32, 1, one, a.runs_q,
          8.0 * a.total_q * a.hq * a.d);
}

int64_t attn_bwd_grid(const AttnArgs &a) {
    const int64_t pairs = (a.cu ? 1 : a.n_seq) * a.hk;
    const int64_t q = attn_grid(pairs, attn_tiles(a.cu != nullptr, a.n_seq, a.seq_q, a.total_q), static_cast<int64_t>(a.hq / a.hk) * a.runs_q);
    const int64_t k = attn_grid(pairs, attn_tiles(a.cu != nullptr, a.n_seq, a.seq_k, a.total_k), a.parts);
    return q > k ? q : k;
}

hipError_t launch_attn_bwd(const AttnArgs &a, hipStream_t stream) {
    if (a.bf16) return a.d == 64 ? run<AttnBf, 64>(a, stream) : run<AttnBf, 128>(a, stream);
    return a.d == 64 ? run<AttnF32, 64>(a, stream) : run<AttnF32, 128>(a, stream);
}

}  // namespace gdr
