// Internal interface between the host API (gdr_mixer_api.cpp) and the kernels
// of the operators around the recurrence: the short causal convolution
// (gdr_conv.hip), the query/key norm with rotation (gdr_qknorm.hip) and the
// state space scan (gdr_ssm.hip).  Not installed; not part of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdr {

// Blocks are dispatched round-robin over the 8 XCDs; this renumbering gives
// each XCD one contiguous run of the `count` blocks, so that neighbours share
// an L2 (a bijection on 0 .. count-1 for any count).
__device__ __forceinline__ int64_t xcd_run(int64_t block, int64_t count) {
    const int64_t q = count / 8, r = count % 8, x = block % 8;
    return x * q + (x < r ? x : r) + block / 8;
}

// Whether an output of so many bytes is stored past the caches.  A convolution
// of 4096 channels and the norm that reads it, us with plain and with such
// stores: 32 MB 31 and 35, 64 MB 48 and 52, 128 MB 112 and 107, 512 MB 464 and
// 439; a norm gradient of 151 MB alone 109 and 106.  (Not the convolution's
// gradient, 114.8 and 114.4.)
__host__ __device__ inline bool past_caches(int64_t bytes) { return bytes >= (int64_t{1} << 27); }
// Stores a piece of 8 or 16 bytes.
template <class V>
__device__ __forceinline__ void store_piece(V *to, V v, bool past) {
    if (past) {
        asm volatile("");   // otherwise the compiler joins the two stores into a plain one
        __builtin_nontemporal_store(v, to);
        asm volatile("");
    } else {
        *to = v;
    }
}

// Short causal depthwise convolution; rows of x and dy are ld* elements apart.
struct ConvArgs {
    const void *x, *w, *bias;   // bias NULL: none
    const int32_t *cu;          // NULL: n_seq rows of seq_len tokens
    const void *s0;             // [N, W-1, ch], NULL: zeros
    void *y, *st;               // st NULL: not written
    int64_t ldx, n_seq, seq_len, total;
    int32_t ch, width, bf16, silu, vec;   // vec: 16-byte pieces of the channels
    // backward
    const void *dy, *dst;       // dst NULL: zeros
    void *dx, *ds0;             // ds0 NULL: not written
    float *dw, *db;             // db NULL: not written
    float *part;                // [conv_bwd_rows][ch][W + 1]
    int64_t lddy;
};
hipError_t launch_conv_fwd(const ConvArgs &a, hipStream_t stream);
// Rows of per-block partial sums of dw and db that a backward call stores.
int64_t conv_bwd_rows(int64_t total, int32_t ch, int32_t bf16, int32_t vec);
hipError_t launch_conv_bwd(const ConvArgs &a, hipStream_t stream);
// One token for each of n_seq sequences: x rows ldx apart, st read and updated in place.
hipError_t launch_conv_step(const ConvArgs &a, hipStream_t stream);

// Norm of each head row of q and k, rotated by position.
struct NormArgs {
    const void *q, *k, *wq, *wk;          // weights [d], NULL: ones
    const float *cos, *sin;               // [table, rot/2]
    const int32_t *pos;                   // [tokens], NULL: the token's index in its row
    void *oq, *ok;
    int64_t tokens, seq_len, table, ldq, ldk;
    int32_t hq, hk, d, rot, bf16, rms, interleaved;
    float eps;
    // backward
    const void *doq, *dok;
    void *dq, *dk;
    float *dwq, *dwk;                     // [d], NULL: no weights
    float *part;                          // [norm_bwd_blocks][d]
    int64_t lddoq, lddok;
};
hipError_t launch_norm_fwd(const NormArgs &a, hipStream_t stream);
int64_t norm_bwd_blocks(const NormArgs &a);
hipError_t launch_norm_bwd(const NormArgs &a, hipStream_t stream);

// Selective state space scan.
constexpr int kGateRow = 6 * 64 + 4;     // floats of a (chunk, head) in gates
constexpr int kTokenPart = 6 * 64 + 4;   // floats of a (chunk, head) in token_part
struct SsmArgs {
    const void *x, *dt, *b, *c;
    const float *A, *D, *dt_bias;         // [H]; D, dt_bias NULL: zeros
    const int32_t *cu;                    // NULL: n_seq rows of seq_len tokens
    const float *h0;                      // [N, H, n, p], NULL: zeros
    void *y;
    float *ht;                            // NULL: not written (step: the state, in place)
    int64_t n_seq, seq_len, total;
    int64_t ldx, lddt, ldb, ldc;
    int32_t heads, groups, n, p, bf16, gate_bf16;
    // Spans of span_len tokens (a multiple of 64) that are walked in parallel.
    // With cu, from a table, or (NULL) one per sequence: {first token, length
    // (< 0: surplus entry), sequence << 2 | last << 1 | first, chunk row of its
    // first chunk}.  Without, row_spans and row_chunks (64 tokens) a sequence.
    const int4 *spans;
    int32_t row_spans, row_chunks;
    const int32_t *span_first;            // [N + 1] first span of each sequence
    int64_t n_spans;                      // entries: an upper bound on the spans
    int64_t span_len;
    int64_t whole;                        // spans are this long when no sequence is longer (a multiple of span_len)
    float *gates;                         // [n_chunks][H][kGateRow]; NULL: made inside the walks (not split)
    float *span_state;                    // [directions][n_spans][H][n p]; NULL: not split
    float *span_decay;                    // [directions][n_spans][H]
    // backward
    const void *dy;
    const float *dht;                     // [N, H, n, p], NULL: zeros
    int64_t lddy;
    float *chunk_state;                   // [2][n_chunks][H][n p]: states before chunks, gradients after them
    int64_t n_chunks;                     // entries: an upper bound on the 64-token chunks
    const int4 *chunks;                   // as spans, span_len 64; NULL without cu
    void *dx, *ddt, *db, *dc;
    float *dA, *dD, *dbias, *dh0;         // dD, dbias, dh0 NULL: not written
    const int32_t *chunks_used;           // entries of chunks in use
    int32_t grad_blocks, grad_least;      // blocks of the gradient, and the least (chunk, head)s of one
    float *bc_part;                       // [parts][db, dc][total][G][n]; NULL: one block sums a group
    float *token_part;                    // [n_chunks][H][kTokenPart]: per-token sums
    float *head_part;                     // [n_chunks][H]{dA, dD, dbias}
};
hipError_t launch_ssm_step(const SsmArgs &a, hipStream_t stream);
// Sets span_len (0: each sequence is walked by one block) and whole.
void ssm_spans(SsmArgs &a, bool bwd);
// Tables of spans and of 64-token chunks from the content of cu_seqlens:
// first spans [N + 1], chunks [N + 1]; tables [n_spans], [n_chunks].
struct SsmTables {
    int32_t *span_first, *chunk_first;
    int4 *spans, *chunks;
};
hipError_t launch_ssm_table(const SsmArgs &a, const SsmTables &t, hipStream_t stream);
// The gates of every (chunk, head).
hipError_t launch_ssm_gates(const SsmArgs &a, hipStream_t stream);
hipError_t launch_ssm_fwd(const SsmArgs &a, hipStream_t stream);
// Sets grad_blocks and grad_least (a.n_chunks set): how many blocks at most sum one group's db and dc.
int ssm_grad_parts(SsmArgs &a);
hipError_t launch_ssm_bwd(const SsmArgs &a, hipStream_t stream);

}  // namespace gdr
