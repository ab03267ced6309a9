// Softmax attention over packed or equal rows, forward.  Per sequence and head,
// over the keys j that query i sees,
//
//     s_ij = scale q_i . k_j,   lse_i = log sum_j e^{s_ij},   o_i = sum_j e^{s_ij - lse_i} v_j.
//
// One pass over the keys with the running maximum and sum of each row.
#include "gdr_attn_device.h"

namespace gdr {
namespace {

// A block takes 128 query rows of one head, 32 a wave, and walks the keys in
// tiles.  Scores are made transposed (keys x queries), so that a lane holds one
// query's scores and the maximum and sum cross lanes once a tile, and the
// result registers are the next product's operand.  The next tile's keys and
// values load to LDS while this one is worked on.
//
// Bound by the matrix unit and the exponentials between its two products, which
// the second wave of a SIMD fills in part.  2 x 8192 tokens, 32 heads on 4,
// causal, bf16: d 128 1.00 to 1.05 ms, 1050 to 1100 TFLOP/s of the 1251 of a
// large matrix product; d 64 860 (twice the exponentials a product).  f32, 2 x
// 4096, 16 heads on 4: d 128 116 of 153, d 64 105: one wave a SIMD, whose
// exponentials nothing overlaps.
template <class T, int D>
struct AttnFwd {
    typedef typename T::E E;
    typedef typename T::F8 F8;
    static constexpr int kKeys = T::kBf16 ? 64 : 32;   // a tile
    typedef AttnTile<T, D, kKeys> Tile;
    static constexpr int kSteps = D / 16, kParts = D / 32, kSub = kKeys / 32;
    struct Lds {
        alignas(16) char k[2][Tile::kBytes];
        alignas(16) char v[2][Tile::kBytes];
    };
    // A row's scores may pass its reference value by so many powers of two
    // before sums and outputs are rescaled to a new one.
    static constexpr float kSlack = 8.f;

    struct Row {
        F8 q[kSteps];
        f32x16 o[kParts];   // transposed: channels x queries
        float ref, sum;     // ref: in powers of two; sum: of this lane's half
    };

    // CAREFUL: a value that is not finite reaches the rows that see its key and no other.  A product
    // gives every row of a tile each of its keys, zero times those it does not see, which a value that
    // is not finite would turn into NaN; there one key after another is added to the rows that see it.
    template <bool CAREFUL>
    static __device__ __forceinline__ void walk(Row &w, const AttnSight &sight, float c, int32_t i0, int32_t i1,
                                                int32_t begin, int32_t end, const E *k, const E *v, uint32_t step_k,
                                                uint32_t step_v, int32_t lk, Lds &lds, int wave, int lane) {
        const int col = lane & 31, h = lane >> 5;
        const typename Tile::From fk = Tile::from(wave, lane, step_k), fv = Tile::from(wave, lane, step_v);
        const int32_t lo = i0 + 32 * wave, at = sight.at(lo + col);
#pragma unroll
        for (int t = 0; t < kParts; ++t) w.o[t] = zero16();
        w.ref = -__builtin_inff();
        w.sum = 0.f;
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
            if (lo > i1 || !sight.any(lo, hi, j, kKeys)) return;
            f32x16 s[kSub];
#pragma unroll
            for (int t = 0; t < kSub; ++t) {
                s[t] = zero16();
#pragma unroll
                for (int ks = 0; ks < kSteps; ++ks) s[t] = T::mma(Tile::rows(lds.k[buf], l, 32 * t, ks), w.q[ks], s[t]);
            }
            attn_ahead<T, kSub * kSteps>();
            const bool whole = sight.all(lo, hi, j, kKeys);
            if (!whole) {
                const int32_t d0 = attn_here(at - j - 4 * h);
#pragma unroll
                for (int t = 0; t < kSub; ++t)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (!sight.sees(d0, 32 * t + 8 * (r / 4) + r % 4)) s[t][r] = -__builtin_inff();
            }
            float top = s[0][0];
#pragma unroll
            for (int t = 0; t < kSub; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) top = fmaxf(top, s[t][r]);
            top = half_max(top) * c;
            if (__builtin_amdgcn_ballot_w64(top > w.ref + kSlack)) {
                // a row that has seen no key keeps -inf, and a factor of 1 for its zeros
                const float now = fmaxf(top, w.ref), f = now == w.ref ? 1.f : fast_exp2(w.ref - now);
                w.ref = now;
                w.sum *= f;
#pragma unroll
                for (int t = 0; t < kParts; ++t) w.o[t] *= f;
            }
            const float ref = w.ref == -__builtin_inff() ? 0.f : w.ref;
            float sums[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int t = 0; t < kSub; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) {   // -inf gives 0: c is above zero
                    s[t][r] = fast_exp2(__builtin_fmaf(s[t][r], c, -ref));
                    sums[r % 4] += s[t][r];
                }
            w.sum += (sums[0] + sums[1]) + (sums[2] + sums[3]);
            // bf16: probabilities are rounded to nearest for the product with the values (2^-8 of each at most, of
            // independent signs); their sum is not
#pragma unroll
            for (int kb = 0; kb < 2 * kSub; ++kb) {
                const F8 p = T::part(s[kb / 2], kb % 2);
                if (!CAREFUL || whole) {
#pragma unroll
                    for (int t = 0; t < kParts; ++t)
                        w.o[t] = T::mma(Tile::across(lds.v[buf], l, 16 * kb, t), p, w.o[t]);
                } else {
                    for (int key = 0; key < 16; ++key) {   // slot s of half h holds key 4 h + s % 4 + 2 (s & 4)
                        const int slot = (key >> 2 & 1) == h ? (key & 3) + (key >> 1 & 4) : -1;
                        const bool seen = sight.sees(at, j + 16 * kb + key);
#pragma unroll
                        for (int t = 0; t < kParts; ++t) {
                            const f32x16 x = T::mma(T::only(Tile::across(lds.v[buf], l, 16 * kb, t), slot),
                                                    T::only(p, slot), zero16());
#pragma unroll
                            for (int r = 0; r < 16; ++r) w.o[t][r] += seen ? x[r] : 0.f;
                        }
                    }
                }
            }
        };
        for (int32_t j = begin; j < end; j += 2 * kKeys) {
            tile(IntC<0>{}, j);
            if (j + kKeys < end) tile(IntC<1>{}, j + kKeys);
        }
    }
};

__device__ __forceinline__ float attn_lse(float ref, float sum) {
    return sum == 0.f ? -__builtin_inff() : (ref + __builtin_log2f(sum)) * 0.69314718055994530942f;
}

// The block that this launched one is a split of: an XCD takes the first split
// of a team of blocks, then the second, and so on.
__device__ __forceinline__ uint32_t attn_cut(const AttnArgs &a, uint32_t &split) {
    const uint32_t at = (blockIdx.x - static_cast<uint32_t>(a.whole)) / 8, runs = a.team * a.splits;
    split = __builtin_amdgcn_readfirstlane(at % runs / a.team);
    return __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a.whole) + 8 * (at / runs * a.team + at % a.team) + blockIdx.x % 8);
}
// The run of key tiles that one of a block's splits walks, of `count` in all.
struct AttnRun {
    int32_t first, last, count;   // tiles first .. last - 1; count: runs that hold any
};
__device__ __forceinline__ AttnRun attn_run(const AttnArgs &a, int32_t tiles, int32_t split) {
    const int32_t even = (tiles + a.splits - 1) / a.splits, share = even > a.least ? even : a.least;
    AttnRun r;
    r.count = tiles > share ? (tiles + share - 1) / share : 1;
    r.first = split * share;
    r.last = r.first + share < tiles ? r.first + share : tiles;
    return r;
}

// A block's rows, and which keys some of them sees, from a whole tile on.
struct AttnBlock {
    AttnSeq seq;
    int32_t hk, hq, i0, i1, begin, end;   // rows i0 .. i1
};
template <int KEYS>
__device__ __forceinline__ bool attn_block(const AttnArgs &a, const AttnItem &item, int lane, AttnBlock &b) {
    if (item.tile < 0) return false;
    const int32_t n = a.cu ? attn_find(a.cu, static_cast<int32_t>(a.n_seq), a.total_q, item.tile, lane) : item.pair / a.hk;
    b.hk = item.pair % a.hk;
    b.hq = b.hk * (a.hq / a.hk) + item.way;
    b.seq = attn_seq(a, n);
    const int64_t tile = a.cu ? item.tile - (attn_clamp(a.cu[n], 0, a.total_q) / kAttnRows + n) : item.tile;
    if (tile < 0 || tile * kAttnRows >= b.seq.lq) return false;
    const AttnSight sight(a, b.seq);
    b.i0 = static_cast<int32_t>(tile * kAttnRows);
    b.i1 = b.i0 + kAttnRows < b.seq.lq ? b.i0 + kAttnRows - 1 : b.seq.lq - 1;
    const int64_t first = static_cast<int64_t>(sight.at(b.i0)) - sight.back + 1;
    b.begin = first > 0 ? static_cast<int32_t>(first) / KEYS * KEYS : 0;
    b.end = sight.at(b.i1) + 1 < b.seq.lk ? sight.at(b.i1) + 1 : b.seq.lk;
    return true;
}

// A block's rows.  Returns, for every wave alike, whether some output is not
// finite and the rows have to be done again with care.
template <class T, int D, bool CAREFUL>
__device__ __forceinline__ bool attn_fwd_block(const AttnArgs &a, uint32_t tiles, typename AttnFwd<T, D>::Lds &lds) {
    typedef AttnFwd<T, D> F;
    typedef typename T::E E;
    typedef typename T::F8 F8;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 31, h = lane >> 5;
    const uint32_t pairs = static_cast<uint32_t>(a.cu ? 1 : a.n_seq) * a.hk, group = a.hq / a.hk;
    const bool cut = a.splits > 1 && blockIdx.x >= static_cast<uint32_t>(a.whole);
    uint32_t block = blockIdx.x, split = 0;
    if (cut) block = attn_cut(a, split);
    AttnBlock b;
    if (!attn_block<F::kKeys>(a, attn_item(block, pairs, tiles, group), lane, b)) return false;
    const AttnSeq &seq = b.seq;
    const AttnSight sight(a, seq);
    const int32_t i0 = b.i0, i1 = b.i1, hk = b.hk, hq = b.hq;
    int32_t begin = b.begin, end = b.end;
    bool alone = true;
    if (cut) {
        const AttnRun run = attn_run(a, begin < end ? (end - begin + F::kKeys - 1) / F::kKeys : 0, static_cast<int32_t>(split));
        if (static_cast<int32_t>(split) >= run.count) return false;
        alone = run.count == 1;
        end = begin + run.last * F::kKeys < end ? begin + run.last * F::kKeys : end;
        begin += run.first * F::kKeys;
    }

    const float c = a.scale * kLog2e;
    typename F::Row w;
    {
        const int32_t i = i0 + 32 * wave + col < seq.lq ? i0 + 32 * wave + col : seq.lq - 1;
        const E *q = static_cast<const E *>(a.q) + (seq.q0 + i) * a.ldq + static_cast<int64_t>(hq) * D + 8 * h;
#pragma unroll
        for (int ks = 0; ks < F::kSteps; ++ks) {
            const F8 x = T::load(q + 16 * ks);
            w.q[ks] = c < 0.f ? T::flip(x) : x;
        }
    }
    const E *k = static_cast<const E *>(a.k) + seq.k0 * a.ldk + static_cast<int64_t>(hk) * D;
    const E *v = static_cast<const E *>(a.v) + seq.k0 * a.ldv + static_cast<int64_t>(hk) * D;
    const uint32_t step_k = static_cast<uint32_t>(a.ldk * sizeof(E)), step_v = static_cast<uint32_t>(a.ldv * sizeof(E));
    F::template walk<CAREFUL>(w, sight, attn_positive(c), i0, i1, begin, end, k, v, step_k, step_v, seq.lk, lds, wave, lane);
    float x = 0.f;   // 0, or NaN where an output is not finite
#pragma unroll
    for (int t = 0; t < F::kParts; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) x = __builtin_fmaf(w.o[t][r], 0.f, x);
    if (!CAREFUL && __syncthreads_or(x != 0.f)) return true;
    const int32_t i = i0 + 32 * wave + col;
    const float sum = half_sum(w.sum);
    if (i >= seq.lq) return false;
    if (alone) {
        const int64_t row = (seq.q0 + i) * a.hq + hq;
        // no key seen (or scores of -inf alone): 0, and NaN stays NaN
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int t = 0; t < F::kParts; ++t) attn_store<T>(static_cast<E *>(a.o) + row * D + 32 * t, w.o[t], inv, h);
        if (a.lse && h == 0) a.lse[row] = attn_lse(w.ref, sum);
    } else {
        const int64_t at = (blockIdx.x - a.whole) * a.run_rows + i - i0;
#pragma unroll
        for (int t = 0; t < F::kParts; ++t) attn_store<AttnF32>(a.run_o + at * D + 32 * t, w.o[t], 1.f, h);
        if (h == 0) {
            a.run_stat[2 * at] = w.ref;
            a.run_stat[2 * at + 1] = sum;
        }
    }
    return false;
}

// A function of its own: inside the kernel it would cost the other walk registers.
template <class T, int D>
__device__ __attribute__((noinline)) void attn_fwd_careful(AttnArgsAt at, uint32_t tiles, __attribute__((address_space(3))) typename AttnFwd<T, D>::Lds *lds) {
    (void)attn_fwd_block<T, D, true>(attn_args(attn_scalar(at)), __builtin_amdgcn_readfirstlane(tiles), attn_scalar(lds));
}

template <class T, int D>
__global__ __launch_bounds__(256, T::kBf16 ? (D == 64 ? 3 : 2) : 1) void gdr_attn_fwd_kernel(AttnArgs a, uint32_t tiles) {
    __shared__ typename AttnFwd<T, D>::Lds lds;
    if (attn_fwd_block<T, D, false>(a, tiles, lds)) attn_fwd_careful<T, D>(attn_args_at(), tiles, attn_lds(lds));
}

// Joins a block's runs, bound by their loads and a launch (8 pieces of 512
// queries: 9 us beside the runs' 200): 4 channels a thread, 8 rows (d 64: 16) at a time, the
// rows shared by the launch's blocks along y.
template <class T, int D>
__global__ __launch_bounds__(256) void gdr_attn_runs_kernel(AttnArgs a, uint32_t tiles) {
    typedef typename T::E E;
    constexpr int kThreads = D / 4;
    const uint32_t pairs = static_cast<uint32_t>(a.cu ? 1 : a.n_seq) * a.hk, group = a.hq / a.hk;
    AttnBlock b;
    if (!attn_block<AttnFwd<T, D>::kKeys>(a, attn_item(static_cast<uint32_t>(a.whole) + blockIdx.x, pairs, tiles, group), threadIdx.x & 63, b)) return;
    constexpr int kKeys = AttnFwd<T, D>::kKeys;
    const int32_t count = attn_run(a, b.begin < b.end ? (b.end - b.begin + kKeys - 1) / kKeys : 0, 0).count;
    if (count == 1) return;
    const int channel = threadIdx.x % kThreads * 4;
    // launched blocks of the runs: attn_cut's inverse
    const uint32_t place = blockIdx.x / 8;
    const int64_t slab = (static_cast<int64_t>(place / a.team) * a.splits * a.team + place % a.team) * 8 + blockIdx.x % 8;
    const int64_t step = 8 * static_cast<int64_t>(a.team) * a.run_rows;
    for (int32_t i = b.i0 + (blockIdx.y * 256 + threadIdx.x) / kThreads; i <= b.i1; i += gridDim.y * 256 / kThreads) {
        const int64_t row = (b.seq.q0 + i) * a.hq + b.hq, at = slab * a.run_rows + i - b.i0;
        const float *stat = a.run_stat + 2 * at, *out = a.run_o + at * D + channel;
        float top = -__builtin_inff();
#pragma unroll 4
        for (int32_t s = 0; s < count; ++s) top = fmaxf(top, stat[2 * s * step]);
        const float base = top == -__builtin_inff() ? 0.f : top;
        float total = 0.f;
        f32x4 x = zero4();
#pragma unroll 4
        for (int32_t s = 0; s < count; ++s) {
            const float f = fast_exp2(stat[2 * s * step] - base);
            total = __builtin_fmaf(f, stat[2 * s * step + 1], total);
            x += f * *reinterpret_cast<const f32x4 *>(out + s * step * D);
        }
        x *= total == 0.f ? 0.f : 1.f / total;
        E *o = static_cast<E *>(a.o) + row * D + channel;
        if constexpr (T::kBf16) *reinterpret_cast<bf16x4 *>(o) = cvt4(x);
        else *reinterpret_cast<f32x4 *>(o) = x;
        if (a.lse && channel == 0) a.lse[row] = attn_lse(top, total);
    }
}

template <class T, int D>
hipError_t run(const AttnArgs &a, hipStream_t stream) {
    const int64_t tiles = attn_tiles(a.cu != nullptr, a.n_seq, a.seq_q, a.total_q);
    gdr_attn_fwd_kernel<T, D><<<dim3(static_cast<unsigned>(attn_fwd_grid(a))), 256, 0, stream>>>(a, static_cast<uint32_t>(tiles));
    if (a.splits > 1)
        gdr_attn_runs_kernel<T, D><<<dim3(static_cast<unsigned>(attn_cut_blocks(a)), D / 8), 256, 0, stream>>>(a, static_cast<uint32_t>(tiles));
    return hipGetLastError();
}

}  // namespace

namespace {
int64_t all_blocks(const AttnArgs &a) {
    return attn_grid((a.cu ? 1 : a.n_seq) * a.hk, attn_tiles(a.cu != nullptr, a.n_seq, a.seq_q, a.total_q), a.hq / a.hk);
}
}  // namespace

// The runs that cost least by attn_time, of all blocks' keys or, where blocks of
// one length fill the chip some times, of those that are left for a last round;
// a tile of keys as measured on large calls.  Runs' outputs go through the
// caches at 6 TB/s, the second launch takes 5 us.  About 512 queries in each of 8
// sequences, 4000 keys before them, 16 heads on 2, d 128 (about 580 blocks, 512
// at a time): 222 us with all blocks' keys whole or all split, 188 with the last
// blocks' split.
// Packed sequences are taken to be alike: 64 queries over 32768 keys are split by
// themselves (78 us) and walked whole beside 63 sequences of 500 keys (590).
void attn_split(AttnArgs &a) {
    const int32_t keys = a.bf16 ? 64 : 32;
    const AttnCost cost = a.bf16 ? (a.d == 64 ? AttnCost{768, 1.95, 0.9} : AttnCost{512, 2.2, 1.35})
                                 : (a.d == 64 ? AttnCost{256, 2.5, 2.5} : AttnCost{256, 5.0, 5.0});
    const double seqs = a.n_seq > 0 ? static_cast<double>(a.n_seq) : 1.0;
    const double lq = a.cu ? a.total_q / seqs : a.seq_q, lk = a.cu ? a.total_k / seqs : a.seq_k;
    const double blocks = a.hq * attn_blocks(a.cu != nullptr, seqs, lq);
    // keys that a block sees, at most and on average
    double most = lk, mean = a.causal ? lk - (lq < lk ? lq : lk) / 2 : lk;
    if (a.window > 0 && a.window + kAttnRows < most) most = a.window + kAttnRows;
    if (mean > most) mean = most;
    const double tiles = most / keys + 1, steps = mean / keys + 1;
    const double rounds = mean > 0.9 * most ? static_cast<double>(static_cast<int64_t>(blocks / cost.slots)) : 0;
    double best = attn_time(cost, blocks, steps, tiles);
    a.splits = a.least = 1;
    a.whole = 0;
    // teams share their keys; where attn_item deals pairs to XCDs, whole ones end at its last block
    const int64_t pairs = (a.cu ? 1 : a.n_seq) * a.hk, group = a.hq / a.hk;
    a.team = static_cast<int32_t>(pairs % 8 == 0 ? group : pairs * group > 8 ? pairs * group / 8 : 1);
    const int64_t team = 8 * static_cast<int64_t>(a.team);
    for (int last = 0; last < (rounds > 0 ? 2 : 1); ++last) {
        const double before = last ? rounds * cost.slots : 0, rest = blocks - before;
        for (int32_t s = 2; s <= 64 && tiles / s >= 4 && rest > 0.5; s += s < 4 ? 1 : s < 16 ? 2 : 8) {
            const double t = before / cost.slots * cost.full * steps + attn_time(cost, rest * s, steps / s, tiles / s) + 5 +
                             8.0 * a.total_q * a.hq * a.d * s * (rest / blocks) / 6e6;
            if (t < 0.95 * best) {
                best = t;
                a.splits = s;
                a.least = static_cast<int32_t>(tiles / s + 0.999);
                a.whole = static_cast<int64_t>(all_blocks(a) * (before / blocks)) / team * team;
            }
        }
    }
    const int64_t rows = a.cu ? a.total_q : a.seq_q;
    a.run_rows = static_cast<int32_t>(rows < kAttnRows ? rows : kAttnRows);
}

int64_t attn_cut_blocks(const AttnArgs &a) {
    if (a.splits == 1) return 0;
    const int64_t team = 8 * static_cast<int64_t>(a.team);
    return (all_blocks(a) - a.whole + team - 1) / team * team;
}

int64_t attn_fwd_grid(const AttnArgs &a) { return a.splits == 1 ? all_blocks(a) : a.whole + attn_cut_blocks(a) * a.splits; }

hipError_t launch_attn_fwd(const AttnArgs &a, hipStream_t stream) {
    if (a.bf16) return a.d == 64 ? run<AttnBf, 64>(a, stream) : run<AttnBf, 128>(a, stream);
    return a.d == 64 ? run<AttnF32, 64>(a, stream) : run<AttnF32, 128>(a, stream);
}

}  // namespace gdr
