// Selective state space scan with one decay per head.  Per sequence and head,
// with the state S as [n][p]:
//
//   dt_t = softplus(dt_raw_t + dt_bias),  a_t = exp(dt_t A)
//   S_t = a_t S_{t-1} + dt_t b_t x_t^T,   y_t = S_t^T c_t + D x_t
//
// b and c are shared by the H / G heads of a group.
//
// Prompts run in chunks of 64 tokens.  With G the running sum of dt A inside
// a chunk and S the state before it,
//
//   y_i = e^G_i S^T c_i + sum_{j <= i} e^(G_i - G_j) dt_j (c_i . b_j) x_j + D x_i
//   S'  = e^G_end S + sum_j e^(G_end - G_j) dt_j b_j x_j^T
//
// are four matrix products.  The state stays in registers over a walk of
// chunks; long sequences are cut into spans that are walked at once: first
// each span's own state from zero, then a pass that joins them along the
// sequence, then the outputs.
#include <type_traits>

#include "gdr_ssm_device.h"

namespace gdr {
namespace {

// --- one token ------------------------------------------------------------------
// HBM bound: the state is read and written once, 8 n p bytes a head.  A block
// owns one (sequence, head) with the whole state in registers, 16 bytes a
// lane, so all of its loads are in flight at once; y is summed over the rows
// each thread holds, then over row groups through LDS.  256 sequences of 32
// heads of 128 x 128: 180 us, 6.0 TB/s of 1.08 GB (a large copy reaches 5.2).
// PAST: the state goes past the caches both ways.
template <int N, int P, bool BF16, bool PAST>
__global__ void __launch_bounds__(256) gdr_ssm_step_kernel(SsmArgs a) {
    constexpr int CG = P / 4, RG = 256 / CG, RPT = N / RG;
    __shared__ float s_b[N], s_c[N], s_part[RG][P];
    const uint32_t seq32 = blockIdx.x / static_cast<uint32_t>(a.heads);
    const int64_t seq = seq32;
    const int h = static_cast<int>(blockIdx.x - seq32 * a.heads);
    const int g = h / (a.heads / a.groups);
    const int t = threadIdx.x, cg = t % CG, rg = t / CG;
    const int j0 = 4 * cg, i0 = RPT * rg;
    float *hp = a.ht + (seq * a.heads + h) * N * P;
    f32x4 S[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const f32x4 *from = reinterpret_cast<const f32x4 *>(hp + (i0 + i) * P + j0);
        if constexpr (PAST) S[i] = __builtin_nontemporal_load(from);
        else S[i] = *from;
    }
    if (t < N) s_b[t] = load_scalar<BF16>(a.b, seq * a.ldb + g * N + t);
    else if (t < 2 * N) s_c[t - N] = load_scalar<BF16>(a.c, seq * a.ldc + g * N + t - N);
    const float dt = softplus(dt_raw(a, seq, h) + head_bias(a, h));
    const float decay = expf(dt * a.A[h]);
    f32x4 x;
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = load_scalar<BF16>(a.x, seq * a.ldx + h * P + j0 + c);
    __syncthreads();
    f32x4 y = zero4();
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        S[i] = S[i] * decay + x * (dt * s_b[i0 + i]);
        f32x4 *const to = reinterpret_cast<f32x4 *>(hp + (i0 + i) * P + j0);
        if constexpr (PAST) __builtin_nontemporal_store(S[i], to);
        else *to = S[i];
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

// --- tables ---------------------------------------------------------------------
constexpr int kTableThreads = 1024;

// One block: prefix sums of every sequence's numbers of spans and chunks (at
// least one, so that a length-0 sequence has a walk that hands its state on),
// then the entries, each of which finds its sequence by bisection.  Here the
// lengths are known: nothing is split when no sequence is longer than a.whole.
// 17 sequences in 65536 tokens: 10 us, one block's latency.
__global__ void __launch_bounds__(kTableThreads) gdr_ssm_table_kernel(SsmArgs a, SsmTables t) {
    // 64 bits: sequences that cu_seqlens makes overlap can sum to any number
    __shared__ int64_t s_span[kTableThreads], s_chunk[kTableThreads];
    __shared__ int32_t s_longest;
    const int tid = threadIdx.x;
    auto range = [&](int64_t n, int64_t &b, int64_t &e) {
        b = a.cu[n];
        e = a.cu[n + 1];
        b = b < 0 ? 0 : b > a.total ? a.total : b;
        e = e < b ? b : e > a.total ? a.total : e;
    };
    auto clamp = [](int64_t v, int64_t most) { return static_cast<int32_t>(v < most ? v : most); };
    if (tid == 0) s_longest = 0;
    __syncthreads();
    int32_t longest = 0;
    for (int64_t n = tid; n < a.n_seq; n += kTableThreads) {
        int64_t b, e;
        range(n, b, e);
        longest = e - b > longest ? static_cast<int32_t>(e - b) : longest;
    }
    atomicMax(&s_longest, longest);
    __syncthreads();
    const int64_t span_len = s_longest > a.whole ? a.span_len : a.whole;
    int64_t spans = 0, chunks = 0;
    for (int64_t base = 0; base < a.n_seq; base += kTableThreads) {
        int64_t ms = 0, mc = 0;
        if (base + tid < a.n_seq) {
            int64_t b, e;
            range(base + tid, b, e);
            ms = (e - b + span_len - 1) / span_len;
            mc = (e - b + 63) / 64;
            ms = ms < 1 ? 1 : ms;
            mc = mc < 1 ? 1 : mc;
        }
        s_span[tid] = ms;
        s_chunk[tid] = mc;
        __syncthreads();
        const int live = static_cast<int>(a.n_seq - base < kTableThreads ? a.n_seq - base : kTableThreads);
        for (int m = 1; m < live; m *= 2) {
            const int64_t os = tid >= m ? s_span[tid - m] : 0, oc = tid >= m ? s_chunk[tid - m] : 0;
            __syncthreads();
            s_span[tid] += os;
            s_chunk[tid] += oc;
            __syncthreads();
        }
        if (base + tid < a.n_seq) {
            t.span_first[base + tid] = clamp(spans + s_span[tid] - ms, a.n_spans);
            t.chunk_first[base + tid] = clamp(chunks + s_chunk[tid] - mc, a.n_chunks);
        }
        spans += s_span[live - 1];
        chunks += s_chunk[live - 1];
        __syncthreads();
    }
    if (tid == 0) {
        t.span_first[a.n_seq] = clamp(spans, a.n_spans);
        t.chunk_first[a.n_seq] = clamp(chunks, a.n_chunks);
    }
    __threadfence_block();
    __syncthreads();
    auto fill = [&](const int32_t *first, int64_t unit, int64_t count, int4 *table) {
        const int64_t used = first[a.n_seq];
        for (int64_t i = tid; i < count; i += kTableThreads) {
            int4 v = make_int4(0, -1, 0, 0);
            if (i < used) {
                int64_t lo = 0, hi = a.n_seq;
                while (hi - lo > 1) {
                    const int64_t m = (lo + hi) / 2;
                    if (first[m] <= i) lo = m;
                    else hi = m;
                }
                int64_t b, e;
                range(lo, b, e);
                const int64_t at = (i - first[lo]) * unit;
                const int64_t left = e - b - at;
                v.x = static_cast<int32_t>(b + at);
                v.y = static_cast<int32_t>(left < 0 ? 0 : left < unit ? left : unit);
                v.z = static_cast<int32_t>((static_cast<uint32_t>(lo) << 2) | (i + 1 == first[lo + 1] ? 2u : 0u) |
                                           (i == first[lo] ? 1u : 0u));
                v.w = static_cast<int32_t>(t.chunk_first[lo] + at / 64);
            }
            table[i] = v;
        }
    };
    fill(t.span_first, span_len, a.n_spans, t.spans);
    fill(t.chunk_first, 64, a.n_chunks, t.chunks);
}

// The gates of every chunk and head, a wave each: 24 us for the 1041 chunks of
// 65536 tokens and 32 heads (51 MB written), where every walk that needs them
// would make them anew, in fp64, beside its products.
__global__ void __launch_bounds__(kSsmThreads) gdr_ssm_gates_kernel(SsmArgs a) {
    __shared__ __attribute__((aligned(16))) Gates sg[kSsmThreads / 64];
    const int l = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const uint32_t item = blockIdx.x * (kSsmThreads / 64) + wave;
    if (item >= a.n_chunks * a.heads) return;
    const uint32_t row = item / static_cast<uint32_t>(a.heads);
    const int h = static_cast<int>(item - row * a.heads);
    int rows;
    int64_t t0;
    chunk_of_row(a, row, t0, rows);
    if (rows <= 0) return;   // no chunk: never read
    const bool valid = l < rows;
    Gates &s = sg[wave];
    chunk_gates(valid ? dt_raw(a, t0 + l, h) : 0.f, head_bias(a, h), a.A[h], valid, s);
    lds_wait();
    float *to = a.gates + static_cast<int64_t>(item) * kGateRow;
    const float *from = reinterpret_cast<const float *>(&s);
#pragma unroll
    for (int k = 0; k < 6; ++k) to[64 * k + l] = from[64 * k + l];
    if (l == 0) to[384] = s.decay;
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

// 512 walks at 8 waves each fill the chip.  Equal rows take that many; in the
// backward pass, where the walk from the end runs beside the one from the
// start, half of it (one row of 16384 tokens, 32 heads, n = 128: forward, p =
// 64, 128, 256, 512, 1024, 2048 walks: 333, 184, 140, 136, 143 us; backward,
// 256 and 512: 417 and 411, p = 128: 777 and 787).  Packed sequences make walks
// of all lengths and take twice as many (15 in 65536 tokens, p = 128, 512 and
// 1024: 834 to 1172 and 778 to 792 us; backward of 4 to 16 in 16384, p = 64,
// 256 and 512: 464 to 482 and 461 to 464).
//
// Not split when that takes fewer steps than its extra launches and its second
// pass over the tokens cost: no sequence longer than `whole` (32 heads, p =
// 64, 16384 tokens, whole = 2048, packed sequences of up to 1930: 141 us whole,
// 188 split; of up to 2489: 163 and 155, 3529: 265 and 161), or none longer
// than `few` (8 and 32 heads, p = 64 and 128; forward bf16, 320 tokens: 23 to 26
// us whole, 22 to 32 split, 512: 35 to 39 and 23 to 45, 1024: 65 to 74 and 26 to
// 46; f32, 192: 30 and 29 to 32, 320: 47 and 30 to 35; backward bf16, 512: 46 to
// 69 and 46 to 82, 768: 54 to 86 and 50 to 91, 1024: 62 to 100 and 50 to 104;
// f32, 384: 64 to 71 and 57 to 70, 512: 71 to 77 and 60 to 75).
// The longest of packed sequences is taken for four times their average, and
// for a third of all tokens at least, so that one long among many short ones
// costs no more than 3 x few steps (37 sequences in 600 tokens: 14 us whole,
// 45 split).
void ssm_spans(SsmArgs &a, bool bwd) {
    int64_t longest = a.seq_len;
    if (a.cu) {   // not known here
        const int64_t four = a.n_seq ? 4 * a.total / a.n_seq : 0;
        longest = four > a.total ? a.total : four > a.total / 3 ? four : a.total / 3;
    }
    const int64_t few = bwd ? (a.bf16 ? 768 : 448) : (a.bf16 ? 512 : 192);
    const int64_t len = (a.total * a.heads / ((bwd ? 256 : 512) * (a.cu ? 2 : 1)) + 63) / 64 * 64;
    a.span_len = len < 64 ? 64 : len;
    a.whole = (a.cu && !bwd ? 4 : 2) * a.span_len;
    if (longest <= few || (a.cu ? a.total : longest) <= a.whole) a.span_len = 0;
}

hipError_t launch_ssm_table(const SsmArgs &a, const SsmTables &t, hipStream_t stream) {
    hipLaunchKernelGGL(gdr_ssm_table_kernel, dim3(1), dim3(kTableThreads), 0, stream, a, t);
    return hipGetLastError();
}

hipError_t launch_ssm_gates(const SsmArgs &a, hipStream_t stream) {
    const int64_t items = a.n_chunks * a.heads;
    if (items > 0x7FFFFFFF) return hipErrorInvalidValue;
    hipLaunchKernelGGL(gdr_ssm_gates_kernel, dim3(static_cast<uint32_t>((items + 3) / 4)), dim3(kSsmThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_ssm_fwd(const SsmArgs &a, hipStream_t stream) {
    return by_ssm(a, [&]<int N, int P, bool BF16>() {
        typedef std::conditional_t<BF16, BfT, FpT> T;
        const dim3 block(kSsmThreads);
        const int64_t walks = (a.span_state ? a.n_spans : a.n_seq) * a.heads;
        if (walks > 0x7FFFFFFF || a.n_seq * a.heads * (N * P / 1024) > 0x7FFFFFFF) return hipErrorInvalidValue;
        const dim3 grid(static_cast<uint32_t>(walks));
        const dim3 out(walk_threads(P));
        if (a.span_state) {
            hipLaunchKernelGGL((gdr_ssm_walk_kernel<T, N, P, kLocal, false, true>), grid, dim3(walk_threads(P)), 0, stream, a);
            hipLaunchKernelGGL((gdr_ssm_join_kernel<N, P, false>), dim3(static_cast<uint32_t>(a.n_seq * a.heads * (N * P / 1024))),
                               block, 0, stream, a);
            hipLaunchKernelGGL((gdr_ssm_walk_kernel<T, N, P, kOut, false, true>), grid, out, 0, stream, a);
        } else {
            hipLaunchKernelGGL((gdr_ssm_walk_kernel<T, N, P, kOut, false, false>), grid, out, 0, stream, a);
        }
        return hipGetLastError();
    });
}

hipError_t launch_ssm_step(const SsmArgs &a, hipStream_t stream) {
    return by_ssm(a, [&]<int N, int P, bool BF16>() {
        const dim3 grid(static_cast<uint32_t>(a.n_seq * a.heads)), block(256);
        // A layer's state comes round again after every other layer's, and is
        // in no cache then.  States of 2, 17, 67, 134, 268 and 537 MB in turn with
        // others, us kept in the caches and past them: 4.1 and 4.6, 9.7 and 7.8, 30
        // and 22, 55 and 46, 104 and 90, 209 and 180.  (The same state over and
        // over: 6.1 and 6.0, 20 and 20, 40 and 45, 79 and 90 from 17 to 268 MB.)
        if (a.n_seq * a.heads * (N * P * 4) >= (1 << 24))
            hipLaunchKernelGGL((gdr_ssm_step_kernel<N, P, BF16, true>), grid, block, 0, stream, a);
        else
            hipLaunchKernelGGL((gdr_ssm_step_kernel<N, P, BF16, false>), grid, block, 0, stream, a);
        return hipGetLastError();
    });
}

}  // namespace gdr
