// Device code shared by the attention kernels (gdr_attn.hip, gdr_attn_bwd.hip,
// gdr_paged.hip): the 32x32 matrix products, tiles in LDS, and which block
// works on what.
//
// Matrix operands.  A product contracts 16 indices k: lane (c, h), c = lane %
// 32, h = lane / 32, supplies row (or column) c with eight values of k.
//   natural order:  k = 8 h + s, s = 0..7              (two operands along rows)
//   result order:   k = 4 h + s, s < 4;  8 + 4 h + s - 4, s >= 4
// A result tile holds, in lane (c, h), column c and rows 8 (r / 4) + 4 h + r % 4
// for its registers r = 0..15: registers 0..7 and 8..15 are operands in result
// order of a product over its rows, so scores feed the next product without
// leaving their lane.  bf16 takes one 32x32x16 instruction, f32 eight 32x32x2.
#pragma once

#include "gdr_attn.h"
#include "gdr_device.h"

namespace gdr {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x16 zero16() {
    f32x16 z;
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = 0.f;
    return z;
}

// Both halves' values of a lane pair (c, 0), (c, 1).
__device__ __forceinline__ float half_max(float x) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float half_sum(float x) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// What scores are multiplied by, in powers of two: one operand of the scores
// takes a negative factor's sign, and 0 becomes a factor that leaves nothing of
// a finite score, so that the -inf of a hidden one stays it.
__device__ __forceinline__ float attn_positive(float c) { return fmaxf(__builtin_fabsf(c), 1e-37f); }

struct AttnBf {
    typedef uint16_t E;
    typedef bf16x8 F8;
    static constexpr bool kBf16 = true;
    static __device__ __forceinline__ f32x16 mma(F8 a, F8 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ F8 load(const E *p) { return *reinterpret_cast<const F8 *>(p); }
    static __device__ __forceinline__ float up(F8 x, int i) { return (float)x[i]; }
    static __device__ __forceinline__ F8 flip(F8 x) {   // -x, exact
        return __builtin_bit_cast(F8, __builtin_bit_cast(v4u32, x) ^ 0x80008000u);
    }
    // registers 8 kb .. 8 kb + 7, rounded to nearest even
    static __device__ __forceinline__ F8 part(const f32x16 &x, int kb) {
        F8 r;
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = (__bf16)x[8 * kb + i];
        return r;
    }
    // registers 8 kb .. as the sum of two parts: cut to bf16, and what is left, rounded, 2^-15 of it away at most.  Both are
    // above zero where it is (2^-120 at least, or as much again of something smaller), so that an infinite factor stays one.
    static __device__ __forceinline__ void parts(const f32x16 &x, int kb, F8 &high, F8 &low) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float y = x[8 * kb + i], z = __uint_as_float(__float_as_uint(y) & 0xFFFF0000u);
            high[i] = __builtin_bit_cast(__bf16, static_cast<uint16_t>(__float_as_uint(y) >> 16));
            low[i] = (__bf16)fmaxf(y - z, fminf(z, 0x1p-120f));
        }
    }
    static __device__ __forceinline__ F8 only(F8 x, int i) {   // element i, zeros elsewhere (i at run time)
        F8 r;
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = j == i ? x[j] : (__bf16)0.f;
        return r;
    }
};

struct AttnF32 {
    typedef float E;
    typedef f32x8 F8;
    static constexpr bool kBf16 = false;
    static __device__ __forceinline__ f32x16 mma(F8 a, F8 b, f32x16 c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ F8 load(const E *p) {
        return __builtin_shufflevector(*reinterpret_cast<const f32x4 *>(p), *reinterpret_cast<const f32x4 *>(p + 4), 0, 1, 2, 3,
                                       4, 5, 6, 7);
    }
    static __device__ __forceinline__ float up(F8 x, int i) { return x[i]; }
    static __device__ __forceinline__ F8 flip(F8 x) { return -x; }
    static __device__ __forceinline__ F8 part(const f32x16 &x, int kb) {
        F8 r;
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = x[8 * kb + i];
        return r;
    }
    static __device__ __forceinline__ F8 only(F8 x, int i) {
        F8 r;
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = j == i ? x[j] : 0.f;
        return r;
    }
};

// --- tiles in LDS ------------------------------------------------------------------

// Loads to LDS past the registers: lane l's 16 (4) bytes land at `lds` + 16 l (4 l).
// Not the builtin: the compiler waits for such loads before every LDS read that
// follows, and a tile is loaded while another one is read.  A load past the
// buffer's end stores zeros.  The wait states are this code's own affair: a
// scalar register of the descriptor that a vector instruction wrote (a first
// lane read, a spilled one read back) may be read by a load five states later,
// m0 one; the compiler does not see that there is a load in here.  m0 is named
// as written, so that none of the compiler's own uses is carried across; that
// it may not be preserved, which the warning for reserved registers says, is
// what is meant.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void lds_load16(v4u32 rsrc, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 : : "s"(lds), "v"(off), "s"(rsrc) : "m0", "memory");
}
__device__ __forceinline__ void lds_load4(v4u32 rsrc, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 : : "s"(lds), "v"(off), "s"(rsrc) : "m0", "memory");
}
#pragma clang diagnostic pop
__device__ __forceinline__ void loads_landed() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

__device__ __forceinline__ v4u32 uniform_rsrc(const void *base, uint32_t bytes) {
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    v4u32 r;
    r[0] = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(p));
    r[1] = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(p >> 32) & 0xFFFFu);
    r[2] = __builtin_amdgcn_readfirstlane(bytes);
    r[3] = 0x00020000u;
    return r;
}
__device__ __forceinline__ uint32_t lds_address(const void *p) {
    return __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(
        reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void *)p)));
}

// ROWS rows of D elements, compact, in 16-byte pieces.  Piece c of row r lies
// at place c ^ turn(r): 16 rows' reads of one piece, and 4 rows' reads of 4
// neighbouring pieces (transposed reads), each touch all 64 banks once.
template <class T, int D, int ROWS>
struct AttnTile {
    typedef typename T::E E;
    typedef typename T::F8 F8;
    static constexpr int kRow = D * sizeof(E), kPieces = kRow / 16, kBytes = ROWS * kRow, kWaves = 4;
    static constexpr int kLoads = kBytes / 1024 / kWaves;    // of a wave
    static constexpr int kWays = kRow == 512 ? 2 : 1;        // places that a lane's pieces alternate between
    static_assert(kBytes % (1024 * kWaves) == 0);

    static __device__ __forceinline__ int turn(int r) {
        if constexpr (kPieces == 8) return (r << 1 & 4) | (r >> 2 & 3);
        else return (r << 2 & 12) | (r >> 2 & 3);
    }
    // Byte offset of a piece in the tile.
    static __device__ __forceinline__ int place(int row, int piece) { return row * kRow + ((piece ^ turn(row)) << 4); }

    // Where lane `lane` of wave `wave` loads from, for rows `step` bytes apart.
    struct From {
        uint32_t off[kWays];
        uint32_t hop;                                        // from one load of a wave to the next
    };
    static __device__ __forceinline__ From from(int wave, int lane, uint32_t step) {
        From f;
#pragma unroll
        for (int w = 0; w < kWays; ++w) {
            const int at = (wave + w * kWaves) * 1024 + lane * 16, row = at / kRow, piece = at % kRow / 16;
            f.off[w] = (wave * 1024 + lane * 16) / kRow * step + ((piece ^ turn(row)) << 4);
        }
        f.hop = kWaves * 1024 / kRow * step;
        return f;
    }
    // Starts loading the tile at `base`, of which `rows` rows are there.
    static __device__ __forceinline__ void load(const From &f, const E *base, uint32_t step, int rows, const void *lds,
                                                int wave) {
        const int there = rows < ROWS ? rows : ROWS;
        const v4u32 rsrc = uniform_rsrc(base, there > 0 ? (there - 1) * step + kRow : 0);
        const uint32_t to = lds_address(lds) + wave * 1024;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) lds_load16(rsrc, f.off[i % kWays] + i * f.hop, to + i * kWaves * 1024);
    }
    // Places that a lane reads, from which those of other steps differ by an exclusive or: kept apart from
    // the loop over the tiles (attn_here), so that registers hold these two and not all of them.
    struct Lane {
        uint32_t along, across;
    };
    static __device__ __forceinline__ Lane lane_places(int lane) {
        const int c = lane & 31, h = lane >> 5;
        Lane l;
        if constexpr (T::kBf16) {
            const int j = lane & 15, r = 4 * h + (j >> 2);
            l.along = place(c, h);
            l.across = place(r, (lane >> 3 & 2) | (j >> 1 & 1)) + (j & 1) * 8;
        } else {
            l.along = place(c, 2 * h);
            l.across = place(4 * h, c >> 2) + (c & 3) * 4;
        }
        return l;
    }
    // Operand along rows: row r0 + c (r0 a multiple of 32), elements 16 ks + 8 h .., natural order.
    static __device__ __forceinline__ F8 rows(const char *tile, const Lane &l, int r0, int ks) {
        if constexpr (T::kBf16) {
            return *reinterpret_cast<const F8 *>(tile + (l.along ^ (ks * 32)) + r0 * kRow);
        } else {
            const f32x4 a = *reinterpret_cast<const f32x4 *>(tile + (l.along ^ (ks * 64)) + r0 * kRow);
            const f32x4 b = *reinterpret_cast<const f32x4 *>(tile + (l.along ^ (ks * 64 + 16)) + r0 * kRow);
            return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
    // Operand across rows: element 32 t + c of the rows r0 .. r0 + 15 (r0 a multiple of 16), result order.
    static __device__ __forceinline__ F8 across(const char *tile, const Lane &l, int r0, int t) {
        if constexpr (T::kBf16) {
            // turn(r + 8) is turn(r) ^ 2
            return cat(ld4_tr(reinterpret_cast<const uint16_t *>(tile + (l.across ^ (t * 64)) + r0 * kRow)),
                       ld4_tr(reinterpret_cast<const uint16_t *>(tile + (l.across ^ (t * 64 + 32)) + (r0 + 8) * kRow)));
        } else {
            static_assert(T::kBf16 || kPieces >= 16);
            F8 v;
#pragma unroll
            for (int s = 0; s < 8; ++s)   // row 4 h + s % 4 + 2 (s & 4)
                v[s] = *reinterpret_cast<const float *>(tile + (l.across ^ (t * 128) ^ ((s & 3) * 64 + (s >> 2) * 32)) +
                                                        (r0 + (s & 3) + 2 * (s & 4)) * kRow);
            return v;
        }
    }
};

// The same value, which the compiler takes for a new one: what is made of it stays where it is used.
__device__ __forceinline__ int32_t attn_here(int32_t x) {
    asm volatile("" : "+v"(x));
    return x;
}
template <class L>
__device__ __forceinline__ L attn_here(L l) {
    asm volatile("" : "+v"(l.along), "+v"(l.across));
    return l;
}

// Orders what stands before it in the block: operand reads run four ahead of the
// N products that take one each (left alone, each product waits for a read that
// starts behind the one before; forward of 2 x 8192, 1045 and 1017 us).
template <class T, int N>
__device__ __forceinline__ void attn_ahead() {
    if constexpr (T::kBf16) {
        constexpr int kAhead = 4;
        __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);   // LDS reads
#pragma unroll
        for (int i = 0; i < N - kAhead; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);    // products
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, kAhead, 0);
    }
}

// 32 channels of a lane's row (a transposed result tile), scaled by f, to
// `row`: bf16 in 16-byte pieces, for which the halves swap a register pair.
// Every lane of a pair (c, 0), (c, 1) calls it or neither does.
template <class T>
__device__ __forceinline__ void attn_store(typename T::E *row, const f32x16 &x, float f, int h) {
    if constexpr (T::kBf16) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            v2u32 y[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                f32x4 z;
#pragma unroll
                for (int r = 0; r < 4; ++r) z[r] = x[8 * p + 4 * q + r] * f;
                y[q] = __builtin_bit_cast(v2u32, cvt4(z));
            }
            const auto a = __builtin_amdgcn_permlane32_swap(y[0][0], y[1][0], false, false);
            const auto b = __builtin_amdgcn_permlane32_swap(y[0][1], y[1][1], false, false);
            *reinterpret_cast<v4u32 *>(row + 16 * p + 8 * h) = v4u32{a[0], b[0], a[1], b[1]};
        }
    } else {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            f32x4 z;
#pragma unroll
            for (int r = 0; r < 4; ++r) z[r] = x[4 * p + r] * f;
            *reinterpret_cast<f32x4 *>(row + 8 * p + 4 * h) = z;
        }
    }
}

// --- sequences and blocks -----------------------------------------------------------

struct AttnSeq {
    int64_t q0, k0;   // first rows
    int32_t lq, lk;
};
__device__ __forceinline__ int64_t attn_clamp(int64_t x, int64_t lo, int64_t hi) { return x < lo ? lo : x > hi ? hi : x; }
// Sequence n, whatever cu_seqlens holds within the tensors.
__device__ __forceinline__ AttnSeq attn_seq(const AttnArgs &a, int64_t n) {
    AttnSeq s;
    if (!a.cu) {
        s.q0 = n * a.seq_q;
        s.k0 = n * a.seq_k;
        s.lq = static_cast<int32_t>(a.seq_q);
        s.lk = static_cast<int32_t>(a.seq_k);
        return s;
    }
    const int32_t *ck = a.cuk ? a.cuk : a.cu;
    s.q0 = attn_clamp(a.cu[n], 0, a.total_q);
    s.lq = static_cast<int32_t>(attn_clamp(a.cu[n + 1], s.q0, a.total_q) - s.q0);
    s.k0 = attn_clamp(ck[n], 0, a.total_k);
    s.lk = static_cast<int32_t>(attn_clamp(ck[n + 1], s.k0, a.total_k) - s.k0);
    return s;
}

// Tiles of kAttnRows rows.  Packed sequences start at tile cu[n] / kAttnRows +
// n: at least one tile later than the last of sequence n - 1, so no table is
// needed, and some tiles are empty.
__host__ __device__ inline int64_t attn_tiles(bool packed, int64_t n_seq, int64_t seq, int64_t total) {
    return packed ? total / kAttnRows + n_seq : (seq + kAttnRows - 1) / kAttnRows;
}
// Last sequence that starts at or before `tile`: a wave narrows 64 sequences at a time.
__device__ __forceinline__ int32_t attn_find(const int32_t *cu, int32_t n_seq, int64_t total, int32_t tile, int lane) {
    int32_t lo = 0, hi = n_seq;
    while (hi - lo > 1) {
        const int32_t step = (hi - lo + 63) / 64, at = lo + lane * step;
        const bool before = at < hi && attn_clamp(cu[at], 0, total) / kAttnRows + at <= tile;
        const int count = __builtin_popcountll(__builtin_amdgcn_ballot_w64(before));
        lo += (count > 0 ? count - 1 : 0) * step;
        hi = hi < lo + step ? hi : lo + step;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// Blocks b, b + 8, .. run on one XCD (with an L2 of its own): they work on the
// same key head (of the same row of the batch), where the counts divide.  Late
// tiles first: causal ones see the most keys.
struct AttnItem {
    int32_t pair, tile;   // (row, key head), tile of the row (packed: of all)
    int32_t way;          // query head of the group, or part of it
};
__host__ __device__ inline int64_t attn_grid(int64_t pairs, int64_t tiles, int64_t ways) {
    return pairs == 0 ? 0 : pairs < 8 && 8 % pairs == 0 ? 8 * ((tiles * ways * pairs + 7) / 8) : pairs * tiles * ways;
}
// All counts are below 2^31, as the grid is.
__device__ __forceinline__ AttnItem attn_item(uint32_t block, uint32_t pairs, uint32_t tiles, uint32_t ways) {
    AttnItem t;
    uint32_t tile;
    if (pairs % 8 == 0) {
        const uint32_t at = block / 8, head = at / ways;
        t.way = at % ways;
        tile = head % tiles;
        t.pair = head / tiles * 8 + block % 8;
    } else if (8 % pairs == 0) {
        const uint32_t x = block % 8, at = block / 8 * (8 / pairs) + x / pairs;   // the XCDs of a pair in turn
        t.pair = x % pairs;
        t.way = at % ways;
        tile = at / ways;
    } else {
        const uint32_t at = block / pairs;
        t.pair = block % pairs;
        t.way = at % ways;
        tile = at / ways;
    }
    t.tile = static_cast<int32_t>(tiles) - 1 - static_cast<int32_t>(tile);   // negative: none
    return t;
}

// The arguments where the kernel was given them, for functions that are not
// inlined: a reference to the kernel's own copy would put it on the stack.
// attn_args_at is for kernels: a function has no such place and takes the pointer.
typedef __attribute__((address_space(4))) const AttnArgs *AttnArgsAt;
__device__ __forceinline__ AttnArgsAt attn_args_at() { return (AttnArgsAt)__builtin_amdgcn_kernarg_segment_ptr(); }
// Functions get their parameters in vector registers: the first lane's make
// what hangs on them scalar again.
__device__ __forceinline__ AttnArgsAt attn_scalar(AttnArgsAt at) {
    const uint64_t p = reinterpret_cast<uint64_t>(at);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(p));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(p >> 32));
    return reinterpret_cast<AttnArgsAt>(static_cast<uint64_t>(hi) << 32 | lo);
}
template <class L>
__device__ __forceinline__ __attribute__((address_space(3))) L *attn_lds(L &lds) {
    return (__attribute__((address_space(3))) L *)&lds;
}
template <class L>
__device__ __forceinline__ L &attn_scalar(__attribute__((address_space(3))) L *lds) {
    const uint32_t p = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds)));
    return *(L *)reinterpret_cast<__attribute__((address_space(3))) L *>(static_cast<uintptr_t>(p));
}
__device__ __forceinline__ AttnArgs attn_args(AttnArgsAt at) {
    AttnArgs a;
    __builtin_memcpy(&a, (const AttnArgs *)at, sizeof(a));
    return a;
}

// Which keys a query sees.  Query i stands behind key at(i) (causal: the last
// one it sees, i + lk - lq; else the sequence's last key), and sees key j where
// 0 <= at(i) - j < back, one unsigned comparison that also ends the sequence.
struct AttnSight {
    int32_t first, slope;
    uint32_t back;
    __device__ __forceinline__ AttnSight(const AttnArgs &a, const AttnSeq &s)
        : first(a.causal ? s.lk - s.lq : s.lk - 1), slope(a.causal ? 1 : 0),
          back(a.window ? static_cast<uint32_t>(a.window) : 0x7FFFFFFFu) {}
    __device__ __forceinline__ int32_t at(int32_t i) const { return first + slope * i; }
    __device__ __forceinline__ bool sees(int32_t at, int32_t j) const { return static_cast<uint32_t>(at - j) < back; }
    // Queries lo .. hi and keys j .. j + n - 1: all pairs seen, any pair seen.
    __device__ __forceinline__ bool all(int32_t lo, int32_t hi, int32_t j, int32_t n) const {
        return at(lo) - (j + n - 1) >= 0 && static_cast<int64_t>(at(hi)) - j < back;
    }
    __device__ __forceinline__ bool any(int32_t lo, int32_t hi, int32_t j, int32_t n) const {
        return at(hi) - j >= 0 && static_cast<int64_t>(at(lo)) - (j + n - 1) < back;
    }
};

}  // namespace
}  // namespace gdr
