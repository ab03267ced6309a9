// A key-value cache in pages: attention of one new token of every sequence over
// it, the store of new keys and values, and the tables and slots of new tokens.
#include "gdr_attn_device.h"

namespace gdr {
namespace {

// --- one token over the cache ---------------------------------------------------------

// A block takes a chunk of one sequence's keys and one key head with its group
// of query heads (32 at most), a quarter a wave, in tiles of 32 keys.  Keys go
// from memory to the matrix operand, values through 32 rows of LDS of the
// wave's own that are read transposed.  The next tile's loads start once this
// one's keys are multiplied and its values are in LDS.  The waves' sums are
// joined in LDS, the blocks' by a second kernel.  Bound by HBM: 64 sequences of
// 4096 to 8192 keys, 32 heads on 4, d 128: 167 us, 4.8 TB/s (a large copy: 5.1);
// one of 131072, 16 heads on 2: 29.2 us, 4.6 TB/s, and 4.6 for the join.
template <class T, int D>
__global__ __launch_bounds__(256, T::kBf16 ? 2 : 1) void gdr_paged_step_kernel(PagedArgs a) {
    typedef typename T::E E;
    typedef typename T::F8 F8;
    typedef AttnTile<T, D, 32> Tile;
    constexpr int kSteps = D / 16, kParts = D / 32, kRow = D * sizeof(E), kLoads = 32 * kRow / 1024;
    __shared__ union {
        alignas(16) char vals[4][32 * kRow];
        float o[4][kParts][16][64];
    } lds;
    __shared__ float refs[4][32], sums[4][32];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 31, h = lane >> 5;
    char *vals = lds.vals[wave];
    const uint32_t group = a.hq / a.hk, blocks = (group + 31) / 32, splits = static_cast<uint32_t>(a.splits);
    uint32_t item = blockIdx.x;
    const int64_t split = item % splits;
    item /= splits;
    const uint32_t head0 = item % blocks * 32;
    item /= blocks;
    const int hk = item % a.hk;
    const int64_t n = item / a.hk;

    int64_t len = a.lens[n];
    len = len < 0 ? 0 : len > a.width * a.page ? a.width * a.page : len;
    const int64_t first = a.window > 0 && len > a.window ? len - a.window : 0;
    const int64_t begin64 = first + split * a.chunk, end64 = begin64 + a.chunk < len ? begin64 + a.chunk : len;
    if (begin64 >= end64 && split > 0) return;   // the first chunk of no keys writes zeros
    const int32_t share = begin64 < end64 ? static_cast<int32_t>((end64 - begin64 + 127) / 128 * 32) : 0;
    const int32_t begin = static_cast<int32_t>(begin64) + wave * share;
    const int32_t end = begin + share < end64 ? begin + share : static_cast<int32_t>(end64);

    const uint32_t head = head0 + col < group ? head0 + col : group - 1;
    const float c0 = a.scale * kLog2e, c = __builtin_fabsf(c0);
    F8 q[kSteps];
    {
        const E *x = static_cast<const E *>(a.q) + n * a.ldq + (static_cast<int64_t>(hk) * group + head) * D + 8 * h;
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks) {
            q[ks] = T::load(x + 16 * ks);
            if (c0 < 0.f) q[ks] = T::flip(q[ks]);
        }
    }
    const int32_t *table = a.table + n * a.width;
    const int64_t row_step = static_cast<int64_t>(a.hk) * kRow;
    const char *kbase = static_cast<const char *>(a.k) + static_cast<int64_t>(hk) * kRow;
    const char *vbase = static_cast<const char *>(a.v) + static_cast<int64_t>(hk) * kRow;
    // The cache row of this lane's key of the tile at j, -1 where there is none.
    auto entry = [&](int32_t j, int32_t &in_page) {
        const int32_t key = j + col < end ? j + col : end - 1;
        const uint32_t p = static_cast<uint32_t>((static_cast<uint64_t>(key) * a.magic) >> a.shift);
        in_page = j + col < end ? key - static_cast<int32_t>(p) * a.page : -1;
        return table[p];
    };
    auto row_of = [&](int32_t page, int32_t in_page) {
        return in_page >= 0 && page >= 0 && page < a.pages ? page * a.page + in_page : -1;
    };
    F8 kreg[kSteps];
    v4u32 vreg[kLoads];
    auto load = [&](int32_t row) {
        const char *k = kbase + (row < 0 ? 0 : row) * row_step + h * 8 * sizeof(E);
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks) kreg[ks] = T::load(reinterpret_cast<const E *>(k + ks * 16 * sizeof(E)));
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int at = i * 1024 + lane * 16;
            const int32_t r = __shfl(row, at / kRow);
            vreg[i] = v4u32{0, 0, 0, 0};   // a row that is not there: zeros, whatever the memory holds
            if (r >= 0) vreg[i] = *reinterpret_cast<const v4u32 *>(vbase + r * row_step + at % kRow);
        }
    };
    const typename Tile::Lane places = Tile::lane_places(lane);
    f32x16 o[kParts];
#pragma unroll
    for (int t = 0; t < kParts; ++t) o[t] = zero16();
    float ref = -__builtin_inff(), sum = 0.f;
    if (begin < end) {
        int32_t in_page, next_in = -1, next_page = -1;
        const int32_t page = entry(begin, in_page);
        int32_t row = row_of(page, in_page);
        if (begin + 32 < end) next_page = entry(begin + 32, next_in);
        load(row);
        for (int32_t j = begin; j < end; j += 32) {
            f32x16 s = zero16();
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks) s = T::mma(kreg[ks], q[ks], s);
            // LDS of one wave: its accesses stay in order
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int at = i * 1024 + lane * 16;
                *reinterpret_cast<v4u32 *>(vals + Tile::place(at / kRow, at % kRow / 16)) = vreg[i];
            }
            const uint64_t there = __builtin_amdgcn_ballot_w64(row >= 0);   // bit k: key j + k
            if (j + 32 < end) {
                row = row_of(next_page, next_in);
                if (j + 64 < end) next_page = entry(j + 64, next_in);
                load(row);
            }
            const uint32_t mine = static_cast<uint32_t>(there) >> (4 * h);
            float top = -__builtin_inff();
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                if (!(mine >> (8 * (r / 4) + r % 4) & 1)) s[r] = -__builtin_inff();
                top = fmaxf(top, s[r]);
            }
            top = half_max(top) * c;
            if (__builtin_amdgcn_ballot_w64(top > ref + 8.f)) {
                const float now = fmaxf(top, ref), f = now == ref ? 1.f : fast_exp2(ref - now);
                ref = now;
                sum *= f;
#pragma unroll
                for (int t = 0; t < kParts; ++t) o[t] *= f;
            }
            const float base = ref == -__builtin_inff() ? 0.f : ref;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float p = fast_exp2(__builtin_fmaf(s[r], c, -base));
                s[r] = mine >> (8 * (r / 4) + r % 4) & 1 ? p : 0.f;
                sum += s[r];
            }
            // bf16: the probabilities stand in two parts, within 2^-15 of them, since memory is waited for and not
            // products (64 sequences of 4096 to 8192 keys: 169.6 us with one part, 166.7 with two; one of 131072:
            // 36.6 and 36.9)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                F8 p, rest;
                if constexpr (T::kBf16) T::parts(s, kb, p, rest);
                else p = T::part(s, kb);
#pragma unroll
                for (int t = 0; t < kParts; ++t) {
                    const F8 x = Tile::across(vals, places, 16 * kb, t);
                    o[t] = T::mma(x, p, o[t]);
                    if constexpr (T::kBf16) o[t] = T::mma(x, rest, o[t]);
                }
            }
        }
    }
    sum = half_sum(sum);
    if (h == 0) {
        refs[wave][col] = ref;
        sums[wave][col] = sum;
    }
    __syncthreads();   // every wave is done with its values too: o takes their place
    const float top = fmaxf(fmaxf(refs[0][col], refs[1][col]), fmaxf(refs[2][col], refs[3][col]));
    const float base = top == -__builtin_inff() ? 0.f : top;
    float total = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) total = __builtin_fmaf(fast_exp2(refs[w][col] - base), sums[w][col], total);
    const float f = fast_exp2(ref - base);
#pragma unroll
    for (int t = 0; t < kParts; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) lds.o[wave][t][r][lane] = o[t][r] * f;
    __syncthreads();
    if (wave >= kParts || head0 + col >= group) return;
    f32x16 x;
#pragma unroll
    for (int r = 0; r < 16; ++r)
        x[r] = (lds.o[0][wave][r][lane] + lds.o[1][wave][r][lane]) + (lds.o[2][wave][r][lane] + lds.o[3][wave][r][lane]);
    const int64_t out = n * a.hq + static_cast<int64_t>(hk) * group + head;
    if (splits == 1) {
        attn_store<T>(static_cast<E *>(a.o) + out * D + 32 * wave, x, total == 0.f ? 0.f : 1.f / total, h);
    } else {
        const int64_t at = out * splits + split;
        attn_store<AttnF32>(a.part + at * D + 32 * wave, x, 1.f, h);
        if (h == 0 && wave == 0) {
            a.stat[2 * at] = top;
            a.stat[2 * at + 1] = total;
        }
    }
}

// Joins the chunks of a query head: 4 channels a thread, ROWS chunks at a time.
// Each row of threads keeps a reference of its own, so that nothing waits for
// the largest before the outputs are loaded.
template <class T, int D, int ROWS>
__global__ __launch_bounds__(ROWS * D / 4) void gdr_paged_join_kernel(PagedArgs a) {
    constexpr int kThreads = D / 4;
    __shared__ f32x4 outs[ROWS][kThreads];
    __shared__ float refs[ROWS], totals[ROWS];
    const int x = threadIdx.x % kThreads, y = threadIdx.x / kThreads;
    const int64_t out = blockIdx.x, n = out / a.hq;
    int64_t len = a.lens[n];
    len = len < 0 ? 0 : len > a.width * a.page ? a.width * a.page : len;
    if (a.window > 0 && len > a.window) len = a.window;
    const int32_t count = len > 0 ? static_cast<int32_t>((len + a.chunk - 1) / a.chunk) : 1;
    const float *stat = a.stat + out * a.splits * 2;
    const float *part = a.part + out * a.splits * D + 4 * x;
    float top = -__builtin_inff(), total = 0.f;
    f32x4 sum = zero4();
#pragma unroll 4
    for (int32_t s = y; s < count; s += ROWS) {
        const float ref = stat[2 * s], more = stat[2 * s + 1];
        const f32x4 o = *reinterpret_cast<const f32x4 *>(part + static_cast<int64_t>(s) * D);
        const float now = fmaxf(top, ref), base = now == -__builtin_inff() ? 0.f : now;
        const float f = fast_exp2(top - base), g = fast_exp2(ref - base);
        top = now;
        total = __builtin_fmaf(total, f, more * g);
        sum = sum * f + o * g;
    }
    outs[y][x] = sum;
    if (x == 0) {
        refs[y] = top;
        totals[y] = total;
    }
    __syncthreads();
    if (y) return;
    for (int i = 1; i < ROWS; ++i) top = fmaxf(top, refs[i]);
    const float base = top == -__builtin_inff() ? 0.f : top;
    total = 0.f;
    sum = zero4();
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const float f = fast_exp2(refs[i] - base);
        total = __builtin_fmaf(totals[i], f, total);
        sum += outs[i][x] * f;
    }
    sum *= total == 0.f ? 0.f : 1.f / total;
    typename T::E *o = static_cast<typename T::E *>(a.o) + out * D + 4 * x;
    if constexpr (T::kBf16) *reinterpret_cast<bf16x4 *>(o) = cvt4(sum);
    else *reinterpret_cast<f32x4 *>(o) = sum;
}

template <class T, int D>
hipError_t run_step(const PagedArgs &a, hipStream_t stream) {
    const int64_t join = a.n_seq * a.hq;
    gdr_paged_step_kernel<T, D><<<dim3(static_cast<unsigned>(a.n_seq * a.hk * ((a.hq / a.hk + 31) / 32) * a.splits)), 256, 0, stream>>>(a);
    if (a.splits > 16) gdr_paged_join_kernel<T, D, 32><<<dim3(static_cast<unsigned>(join)), 8 * D, 0, stream>>>(a);
    else if (a.splits > 1) gdr_paged_join_kernel<T, D, 4><<<dim3(static_cast<unsigned>(join)), D, 0, stream>>>(a);
    return hipGetLastError();
}

// --- store ------------------------------------------------------------------------------

// 16 bytes a thread.  Bound by HBM: 16384 tokens of 8 heads of 128, bf16, 26.1 us
// (5.1 TB/s, as a large copy); a few tokens by the launch.
__global__ __launch_bounds__(256) void gdr_page_store_kernel(StoreArgs a) {
    const int64_t pieces = a.row_bytes / 16, count = 2 * a.tokens * pieces;
    const int64_t i = blockIdx.x * static_cast<int64_t>(256) + threadIdx.x;
    if (i >= count) return;
    const bool v = i >= a.tokens * pieces;
    const int64_t at = v ? i - a.tokens * pieces : i, t = at / pieces, piece = at % pieces * 16;
    const int32_t slot = a.slots[t];
    if (slot < 0 || slot >= a.rows) return;
    const char *from = v ? static_cast<const char *>(a.v) + t * a.ldv : static_cast<const char *>(a.k) + t * a.ldk;
    char *to = static_cast<char *>(v ? a.vp : a.kp) + slot * a.row_bytes;
    *reinterpret_cast<v4u32 *>(to + piece) = *reinterpret_cast<const v4u32 *>(from + piece);
}

// --- plan -------------------------------------------------------------------------------

struct PlanSeq {
    uint32_t past, fresh, held, need;   // sums of two stay below 2^32
};
__device__ __forceinline__ PlanSeq plan_seq(const PlanArgs &a, int64_t n) {
    PlanSeq s;
    const uint32_t page = a.page;
    s.past = a.past[n] > 0 ? a.past[n] : 0;
    s.fresh = a.fresh[n] > 0 ? a.fresh[n] : 0;
    s.held = s.past / page + (s.past % page != 0);
    const uint32_t len = s.past + s.fresh;
    s.need = len / page + (len % page != 0) - s.held;
    return s;
}
__device__ __forceinline__ int32_t plan_int(int64_t x) { return x > 0x7FFFFFFF ? 0x7FFFFFFF : static_cast<int32_t>(x); }

// Each block has a run of sequences (and the place behind the last one, which
// stands for the totals).  The tokens and pages before its run are sums over the
// lengths, which every block makes for itself, N values from the caches, so that
// one launch does.  Blocks along y share a sequence's tokens.  Bound by latency:
// 5.5 us for 256 requests, 12 of them prompts of up to 4096 tokens; 3.6 for 8
// tokens, where a call's host time is 5.1.
__global__ __launch_bounds__(256) void gdr_page_plan_kernel(PlanArgs a, int64_t run) {
    __shared__ int64_t sums[2][4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t start = blockIdx.x * run, stop = start + run < a.n_seq + 1 ? start + run : a.n_seq + 1;
    const int64_t i0 = blockIdx.y * static_cast<int64_t>(256) + threadIdx.x, hop = gridDim.y * static_cast<int64_t>(256);
    int64_t tokens = 0, pages = 0;
    for (int64_t m = threadIdx.x; m < start && m < a.n_seq; m += 256) {
        const PlanSeq s = plan_seq(a, m);
        tokens += s.fresh;
        pages += s.need;
    }
    for (int m = 1; m < 64; m *= 2) {
        tokens += __shfl_xor(tokens, m);
        pages += __shfl_xor(pages, m);
    }
    if (lane == 0) {
        sums[0][wave] = tokens;
        sums[1][wave] = pages;
    }
    __syncthreads();
    tokens = sums[0][0] + sums[0][1] + sums[0][2] + sums[0][3];
    pages = sums[1][0] + sums[1][1] + sums[1][2] + sums[1][3];
    for (int64_t n = start; n < stop; ++n) {
        if (i0 == 0) a.cu[n] = plan_int(tokens < a.tokens ? tokens : a.tokens);
        if (n == a.n_seq) {
            if (i0 == 0) {
                a.used[0] = plan_int(tokens);
                a.used[1] = plan_int(pages);
            }
            for (int64_t t = tokens + i0; t < a.tokens; t += hop) {
                a.positions[t] = 0;
                a.slots[t] = -1;
            }
            return;
        }
        const PlanSeq s = plan_seq(a, n);
        if (i0 == 0) a.lens[n] = plan_int(static_cast<int64_t>(s.past) + s.fresh);
        int32_t *row = a.table + n * a.width;
        const auto taken = [&](int64_t i) { return pages + i < a.pool_size ? a.pool[pages + i] : -1; };
        for (int64_t i = i0; i < s.need && s.held + i < a.width; i += hop) row[s.held + i] = taken(i);
        for (int64_t i = i0; i < s.fresh && tokens + i < a.tokens; i += hop) {
            const uint32_t at = s.past + static_cast<uint32_t>(i), p = at / static_cast<uint32_t>(a.page);
            // a page taken now comes from the pool again: the row may not be written yet
            const int64_t page = p >= a.width ? -1 : p >= s.held ? taken(p - s.held) : row[p];
            const int64_t slot = page * a.page + at % static_cast<uint32_t>(a.page);
            a.positions[tokens + i] = plan_int(at);
            a.slots[tokens + i] = page < 0 || slot > 0x7FFFFFFF ? -1 : static_cast<int32_t>(slot);
        }
        tokens += s.fresh;
        pages += s.need;
    }
}

}  // namespace

// The chunk (a multiple of 128 keys) that costs least by a model of the launch,
// in us: a step of 128 keys takes a block 1.25 (64 channels 0.7, f32 7 and 2.9)
// and the chip holds 512 blocks; the cache is read at 5.1 TB/s where all CUs
// have a block; a second kernel takes 5.5, 0.02 more a chunk of a sequence, and
// the traffic of the chunks' outputs.  Measured against 512 and 1024 keys:
// 64 x 1024 keys, 4 key heads, 30.4 and (one chunk, no second kernel) 23.8 us;
// 1 x 16384, 2 key heads, 16.9 and 21.9.  At most about 1024 blocks at the
// longest: more would only split further what fills the chip already.  All
// sequences are taken to be as long as the table holds: one of 131072 keys
// beside 63 of 1000 in such a table is one chunk, 1910 us for 78 us of bytes.
void paged_split(PagedArgs &a) {
    int64_t keys = a.width * a.page;
    if (a.window > 0 && keys > a.window) keys = a.window;
    if (keys < 1) keys = 1;
    const int64_t blocks32 = (a.hq / a.hk + 31) / 32, rows = a.n_seq * a.hk * blocks32;
    const double step = a.bf16 ? (a.d == 64 ? 0.7 : 1.25) : (a.d == 64 ? 2.9 : 7.0);
    const double bytes = static_cast<double>(rows / blocks32) * keys * a.d * (a.bf16 ? 4 : 8);
    int64_t most = (keys + 127) / 128 * 128, least = (rows * keys / 1024 + 127) / 128 * 128;
    if (most > 1 << 20) most = 1 << 20;
    if (least < 128) least = 128;
    double best = 0;
    a.splits = 0;
    for (int64_t chunk = most; chunk >= least || a.splits == 0; chunk = (chunk / 2 + 127) / 128 * 128) {
        const int64_t splits = (keys + chunk - 1) / chunk;
        const double blocks = static_cast<double>(rows) * splits, rounds = blocks > 512 ? blocks / 512 : 1;
        double t = 4.3 + chunk / 128 * step * rounds;
        const double read = bytes / 5.1e6 * (blocks < 256 ? 256 / (blocks > 1 ? blocks : 1) : 1);
        if (read > t) t = read;
        if (splits > 1) t += 5.5 + 0.02 * splits + static_cast<double>(a.n_seq) * a.hq * splits * a.d * 8 / 4e6;
        if (a.splits == 0 || t < 0.97 * best) {
            best = t;
            a.chunk = static_cast<int32_t>(chunk);
            a.splits = splits;
        }
        if (chunk == 128) break;
    }
}

int64_t paged_grid(const PagedArgs &a) {
    const int64_t step = a.n_seq * a.hk * ((a.hq / a.hk + 31) / 32) * a.splits, join = a.splits > 1 ? a.n_seq * a.hq : 0;
    const int64_t threads = a.splits > 16 ? 8 * a.d : a.d;   // of a block that joins
    return step > (join * threads + 255) / 256 ? step : (join * threads + 255) / 256;
}

hipError_t launch_paged_step(const PagedArgs &a, hipStream_t stream) {
    if (a.bf16) return a.d == 64 ? run_step<AttnBf, 64>(a, stream) : run_step<AttnBf, 128>(a, stream);
    return a.d == 64 ? run_step<AttnF32, 64>(a, stream) : run_step<AttnF32, 128>(a, stream);
}

int64_t page_store_grid(const StoreArgs &a) { return (2 * a.tokens * (a.row_bytes / 16) + 255) / 256; }

hipError_t launch_page_store(const StoreArgs &a, hipStream_t stream) {
    gdr_page_store_kernel<<<dim3(static_cast<unsigned>(page_store_grid(a))), 256, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_page_plan(const PlanArgs &a, hipStream_t stream) {
    const int64_t run = (a.n_seq + 1024) / 1024, blocks = (a.n_seq + run) / run;   // places 0 .. n_seq
    const int64_t share = (a.tokens + 8191) / 8192;
    const unsigned y = share < 1 ? 1 : share > 16 ? 16 : static_cast<unsigned>(share);
    gdr_page_plan_kernel<<<dim3(static_cast<unsigned>(blocks), y), 256, 0, stream>>>(a, run);
    return hipGetLastError();
}

}  // namespace gdr
