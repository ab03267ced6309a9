// Host side of the operators around the recurrence (include/gdr.h): the short
// causal convolution, the query/key norm with rotation and the state space
// scan.  Validation, workspace and launches; the same rules as gdr_api.cpp,
// except that inputs named there may have rows further apart than compact.
#include "gdr.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "gdr_entry.h"
#include "gdr_internal.h"
#include "gdr_mixer.h"

namespace {

using namespace gdr::host;

// --- short convolution ----------------------------------------------------------

struct ConvIn {
    const gdr_tensor *x, *w, *bias, *cu, *s0;
    int activation;
    Span sx, sw, sbias, scu, ss0;
    int64_t B, T, N;
};

// Checks what forward, backward and step share and fills the arguments.
// x is [B, T, ch], or [B, ch] for a step (lead = 1).
int plan_conv(ConvIn &c, int lead, gdr::ConvArgs &a) {
    std::memset(&a, 0, sizeof(a));
    int64_t n;
    int rc;
    if (!c.x) return fail(GDR_EINVAL, "x: descriptor is NULL");
    if (!is_float(c.x)) return fail(GDR_EDTYPE, "x: dtype must be bf16 or f32, got %s", dtype_name(c.x->dtype));
    const size_t e = dtype_size(c.x->dtype);
    if ((rc = check_rows(c.x, "x", lead + 1, lead, e, &a.ldx, &c.sx))) return rc;
    if ((rc = check_tensor(c.w, "w", 2, &n, e))) return rc;
    c.sw = span_of(c.w, n);
    if (c.bias) {
        if ((rc = check_tensor(c.bias, "bias", 1, &n, e))) return rc;
        c.sbias = span_of(c.bias, n);
    }
    if (c.cu) {
        if ((rc = check_tensor(c.cu, "cu_seqlens", 1, &n, 4))) return rc;
        c.scu = span_of(c.cu, n);
    }
    if (c.s0) {
        if ((rc = check_tensor(c.s0, "s0", 3, &n, e))) return rc;
        c.ss0 = span_of(c.s0, n);
    }
    const int64_t ch = c.x->shape[lead], W = c.w->shape[1];
    c.B = c.x->shape[0];
    c.T = lead == 2 ? c.x->shape[1] : 1;
    if ((rc = sequences(c.cu, c.B, c.T, &c.N))) return rc;
    if (W < 2 || W > 4) return fail(GDR_ESHAPE, "w: 2, 3 or 4 taps are supported, got %lld", (long long)W);
    if (ch < 1 || ch > (1 << 24)) return fail(GDR_ESHAPE, "x: between 1 and 2^24 channels are supported, got %lld", (long long)ch);
    if ((rc = want_dtype(c.w, "w", c.x->dtype)) || (rc = want_dtype(c.bias, "bias", c.x->dtype)) ||
        (rc = want_dtype(c.s0, "s0", c.x->dtype)))
        return rc;
    if ((rc = want_shape(c.w, "w", {ch, W}, "[channels, W]")) || (rc = want_shape(c.bias, "bias", {ch}, "[channels]")) ||
        (rc = want_shape(c.s0, "s0", {c.N, W - 1, ch}, "[N, W - 1, channels]")))
        return rc;
    if (c.activation != GDR_ACT_NONE && c.activation != GDR_ACT_SILU)
        return fail(GDR_EINVAL, "activation: unknown value %d", c.activation);
    a.x = c.x->data;
    a.w = c.w->data;
    a.bias = c.bias ? c.bias->data : nullptr;
    a.cu = c.cu ? static_cast<const int32_t *>(c.cu->data) : nullptr;
    a.s0 = c.s0 ? c.s0->data : nullptr;
    a.n_seq = c.N;
    a.seq_len = c.T;
    a.total = live_tokens(c.N, c.B, c.T);
    a.ch = static_cast<int32_t>(ch);
    a.width = static_cast<int32_t>(W);
    a.bf16 = c.x->dtype == GDR_BF16;
    a.silu = c.activation == GDR_ACT_SILU;
    // 16-byte pieces where every row of every tensor starts on one
    a.vec = (ch * static_cast<int64_t>(e)) % 16 == 0 && (a.ldx * static_cast<int64_t>(e)) % 16 == 0 && aligned16(c.x) &&
            aligned16(c.w) && aligned16(c.bias) && aligned16(c.s0);
    return GDR_OK;
}

// --- query/key norm ---------------------------------------------------------------

struct NormIn {
    const gdr_tensor *q, *k, *wq, *wk, *cos, *sin, *pos;
    int norm;
    float eps;
    int interleaved;
    Span sq, sk, swq, swk, scos, ssin, spos;
    int64_t B, T;
};

int plan_norm(NormIn &c, gdr::NormArgs &a) {
    std::memset(&a, 0, sizeof(a));
    int64_t n;
    int rc;
    if (!c.q) return fail(GDR_EINVAL, "q: descriptor is NULL");
    if (!is_float(c.q)) return fail(GDR_EDTYPE, "q: dtype must be bf16 or f32, got %s", dtype_name(c.q->dtype));
    if ((rc = check_rows(c.q, "q", 4, 2, 16, &a.ldq, &c.sq))) return rc;
    if ((rc = check_rows(c.k, "k", 4, 2, 16, &a.ldk, &c.sk))) return rc;
    struct Opt {
        const gdr_tensor *t;
        const char *name;
        int ndim;
        size_t align;
        Span *span;
    } opts[] = {{c.wq, "wq", 1, 16, &c.swq}, {c.wk, "wk", 1, 16, &c.swk},       {c.cos, "cos", 2, 16, &c.scos},
                {c.sin, "sin", 2, 16, &c.ssin}, {c.pos, "positions", 2, 4, &c.spos}};
    for (const Opt &o : opts) {
        if (!o.t) continue;
        if ((rc = check_tensor(o.t, o.name, o.ndim, &n, o.align))) return rc;
        *o.span = span_of(o.t, n);
    }
    c.B = c.q->shape[0];
    c.T = c.q->shape[1];
    const int64_t hq = c.q->shape[2], hk = c.k->shape[2], d = c.q->shape[3];
    if (c.B > 0 && c.T > 0x7FFFFFFFLL / c.B) return fail(GDR_ESHAPE, "B * T exceeds 2^31 - 1 tokens");
    if (d != 64 && d != 128 && d != 256) return fail(GDR_ESHAPE, "q: head dim must be 64, 128 or 256, got %lld", (long long)d);
    if (hq < 1 || hk < 1 || hq > 65536 || hk > 65536) return fail(GDR_ESHAPE, "head counts must be between 1 and 65536");
    if ((rc = want_dtype(c.k, "k", c.q->dtype)) || (rc = want_dtype(c.wq, "wq", c.q->dtype)) ||
        (rc = want_dtype(c.wk, "wk", c.q->dtype)) || (rc = want_dtype(c.cos, "cos", GDR_F32)) ||
        (rc = want_dtype(c.sin, "sin", GDR_F32)) || (rc = want_dtype(c.pos, "positions", GDR_I32)))
        return rc;
    if ((rc = want_shape(c.k, "k", {c.B, c.T, hk, d}, "[B, T, Hk, d] with q's B, T and d")) ||
        (rc = want_shape(c.wq, "wq", {d}, "[d]")) || (rc = want_shape(c.wk, "wk", {d}, "[d]")) ||
        (rc = want_shape(c.pos, "positions", {c.B, c.T}, "[B, T]")))
        return rc;
    if (!c.cos != !c.sin) return fail(GDR_EINVAL, "cos and sin: both tables or neither");
    if (c.pos && !c.cos) return fail(GDR_EINVAL, "positions without cos and sin");
    if (c.norm != GDR_NORM_L2 && c.norm != GDR_NORM_RMS) return fail(GDR_EINVAL, "norm: unknown value %d", c.norm);
    if (!std::isfinite(c.eps) || c.eps < 0) return fail(GDR_EINVAL, "eps must be finite and not negative");
    int64_t rot = 0, table = 0;
    if (c.cos) {
        table = c.cos->shape[0];
        rot = 2 * c.cos->shape[1];
        if ((rc = want_shape(c.sin, "sin", {table, rot / 2}, "cos's shape"))) return rc;
        if (rot < 16 || rot > d || rot % 16)
            return fail(GDR_ESHAPE, "cos: [table, rot / 2] with rot a multiple of 16 up to the head dim, got rot = %lld",
                        (long long)rot);
        if (table < 1 || table > 0x7FFFFFFF) return fail(GDR_ESHAPE, "cos: the table needs between 1 and 2^31 - 1 rows");
        if (!c.pos && c.T > table)
            return fail(GDR_ESHAPE, "cos: %lld rows for %lld tokens", (long long)table, (long long)c.T);
    }
    a.q = c.q->data;
    a.k = c.k->data;
    a.wq = c.wq ? c.wq->data : nullptr;
    a.wk = c.wk ? c.wk->data : nullptr;
    a.cos = c.cos ? static_cast<const float *>(c.cos->data) : nullptr;
    a.sin = c.sin ? static_cast<const float *>(c.sin->data) : nullptr;
    a.pos = c.pos ? static_cast<const int32_t *>(c.pos->data) : nullptr;
    a.tokens = c.B * c.T;
    a.seq_len = c.T;
    a.table = table;
    a.hq = static_cast<int32_t>(hq);
    a.hk = static_cast<int32_t>(hk);
    a.d = static_cast<int32_t>(d);
    a.rot = static_cast<int32_t>(rot);
    a.bf16 = c.q->dtype == GDR_BF16;
    a.rms = c.norm == GDR_NORM_RMS;
    a.interleaved = c.interleaved != 0;
    a.eps = c.eps;
    return GDR_OK;
}

// --- state space scan ---------------------------------------------------------------

// The scan's chunk tiles are addressed with 32-bit byte offsets over 64 rows.
constexpr int64_t kMaxRow = 1 << 25;

struct SsmIn {
    const gdr_tensor *x, *dt, *A, *b, *c, *D, *dt_bias, *cu, *h0;
    Span sx, sdt, sA, sb, sc, sD, sbias, scu, sh0;
    int64_t B, T, N;
};

// x [B, T, H, p], dt [B, T, H], b and c [B, T, G, n]; without T for a step (lead = 1).
int plan_ssm(SsmIn &s, int lead, gdr::SsmArgs &a) {
    std::memset(&a, 0, sizeof(a));
    int64_t n;
    int rc;
    if (!s.x) return fail(GDR_EINVAL, "x: descriptor is NULL");
    if (!is_float(s.x)) return fail(GDR_EDTYPE, "x: dtype must be bf16 or f32, got %s", dtype_name(s.x->dtype));
    if ((rc = check_rows(s.x, "x", lead + 2, lead, 16, &a.ldx, &s.sx))) return rc;
    if (s.dt && !is_float(s.dt)) return fail(GDR_EDTYPE, "dt: dtype must be bf16 or f32, got %s", dtype_name(s.dt->dtype));
    if ((rc = check_rows(s.dt, "dt", lead + 1, lead, s.dt ? dtype_size(s.dt->dtype) : 4, &a.lddt, &s.sdt))) return rc;
    if ((rc = check_rows(s.b, "b", lead + 2, lead, 16, &a.ldb, &s.sb))) return rc;
    if ((rc = check_rows(s.c, "c", lead + 2, lead, 16, &a.ldc, &s.sc))) return rc;
    struct Opt {
        const gdr_tensor *t;
        const char *name;
        int ndim;
        size_t align;
        Span *span;
        bool needed;
    } opts[] = {{s.A, "A", 1, 4, &s.sA, true},          {s.D, "D", 1, 4, &s.sD, false},
                {s.dt_bias, "dt_bias", 1, 4, &s.sbias, false}, {s.cu, "cu_seqlens", 1, 4, &s.scu, false},
                {s.h0, "h0", 4, 16, &s.sh0, false}};
    for (const Opt &o : opts) {
        if (!o.t && !o.needed) continue;
        if ((rc = check_tensor(o.t, o.name, o.ndim, &n, o.align))) return rc;
        *o.span = span_of(o.t, n);
    }
    s.B = s.x->shape[0];
    s.T = lead == 2 ? s.x->shape[1] : 1;
    if ((rc = sequences(s.cu, s.B, s.T, &s.N))) return rc;
    const int64_t H = s.x->shape[lead], p = s.x->shape[lead + 1], G = s.b->shape[lead], nn = s.b->shape[lead + 1];
    if ((rc = want_dtype(s.b, "b", s.x->dtype)) || (rc = want_dtype(s.c, "c", s.x->dtype)) ||
        (rc = want_dtype(s.A, "A", GDR_F32)) || (rc = want_dtype(s.D, "D", GDR_F32)) ||
        (rc = want_dtype(s.dt_bias, "dt_bias", GDR_F32)) || (rc = want_dtype(s.h0, "h0", GDR_F32)))
        return rc;
    if (p != 64 && p != 128) return fail(GDR_ESHAPE, "x: p must be 64 or 128, got %lld", (long long)p);
    if (nn != 64 && nn != 128) return fail(GDR_ESHAPE, "b: n must be 64 or 128, got %lld", (long long)nn);
    if (H < 1 || G < 1 || H > 65536) return fail(GDR_ESHAPE, "head and group counts must be between 1 and 65536");
    if (H % G != 0) return fail(GDR_ESHAPE, "H (%lld) must be a multiple of G (%lld)", (long long)H, (long long)G);
    const bool step = lead == 1;
    if (step) {
        if ((rc = want_shape(s.dt, "dt", {s.B, H}, "[B, H]")) || (rc = want_shape(s.b, "b", {s.B, G, nn}, "[B, G, n]")) ||
            (rc = want_shape(s.c, "c", {s.B, G, nn}, "[B, G, n]")))
            return rc;
    } else {
        if ((rc = want_shape(s.dt, "dt", {s.B, s.T, H}, "[B, T, H]")) ||
            (rc = want_shape(s.b, "b", {s.B, s.T, G, nn}, "[B, T, G, n]")) ||
            (rc = want_shape(s.c, "c", {s.B, s.T, G, nn}, "[B, T, G, n]")))
            return rc;
    }
    if ((rc = want_shape(s.A, "A", {H}, "[H]")) || (rc = want_shape(s.D, "D", {H}, "[H]")) ||
        (rc = want_shape(s.dt_bias, "dt_bias", {H}, "[H]")) ||
        (rc = want_shape(s.h0, "h0", {s.N, H, nn, p}, "[N, H, n, p]")))
        return rc;
    if (s.N * H > 0x3FFFFFFFLL) return fail(GDR_ESHAPE, "N * H exceeds the launch grid limit");
    const int64_t e = static_cast<int64_t>(dtype_size(s.x->dtype));
    if (!step && (a.ldx * e > kMaxRow || a.ldb * e > kMaxRow || a.ldc * e > kMaxRow))
        return fail(GDR_ESTRIDE, "x, b and c: rows may be at most %lld bytes apart", (long long)kMaxRow);
    a.x = s.x->data;
    a.dt = s.dt->data;
    a.b = s.b->data;
    a.c = s.c->data;
    a.A = static_cast<const float *>(s.A->data);
    a.D = s.D ? static_cast<const float *>(s.D->data) : nullptr;
    a.dt_bias = s.dt_bias ? static_cast<const float *>(s.dt_bias->data) : nullptr;
    a.cu = s.cu ? static_cast<const int32_t *>(s.cu->data) : nullptr;
    a.h0 = s.h0 ? static_cast<const float *>(s.h0->data) : nullptr;
    a.n_seq = s.N;
    a.seq_len = s.T;
    a.total = live_tokens(s.N, s.B, s.T);
    a.heads = static_cast<int32_t>(H);
    a.groups = static_cast<int32_t>(G);
    a.n = static_cast<int32_t>(nn);
    a.p = static_cast<int32_t>(p);
    a.bf16 = s.x->dtype == GDR_BF16;
    a.gate_bf16 = s.dt->dtype == GDR_BF16;
    return GDR_OK;
}

// Parts of a call's workspace; also sets the counts that the launches need.
// The entries of a table bound the spans: each sequence has at least one and
// at most its length / span + 1.
void carve_ssm(gdr::SsmArgs &a, bool bwd, Carve &c, gdr::SsmTables &t) {
    std::memset(&t, 0, sizeof(t));
    const int64_t state = static_cast<int64_t>(a.n) * a.p, H = a.heads;
    auto entries = [&](int64_t span) {
        if (a.cu) return a.total / span + a.n_seq;
        const int64_t each = (a.seq_len + span - 1) / span;
        return a.n_seq * (each < 1 ? 1 : each);
    };
    gdr::ssm_spans(a, bwd);
    const bool split = a.span_len > 0;
    if (!split) a.span_len = a.whole = ((a.cu ? a.total : a.seq_len) / 64 + 1) * 64;
    a.n_spans = split ? entries(a.span_len) : a.n_seq;
    a.row_spans = static_cast<int32_t>((a.seq_len + a.span_len - 1) / a.span_len);
    if (a.row_spans < 1) a.row_spans = 1;
    a.row_chunks = static_cast<int32_t>((a.seq_len + 63) / 64);
    if (a.row_chunks < 1) a.row_chunks = 1;
    if (!split && !bwd) return;
    const int64_t ways = bwd ? 2 : 1;
    a.n_chunks = entries(64);
    if (a.cu) {
        t.span_first = c.take<int32_t>(a.n_seq + 1);
        t.chunk_first = c.take<int32_t>(a.n_seq + 1);
        t.spans = c.take<int4>(a.n_spans);
        t.chunks = c.take<int4>(a.n_chunks);
    }
    a.gates = c.take<float>(a.n_chunks * H * gdr::kGateRow);
    if (split) {
        a.span_state = c.take<float>(ways * a.n_spans * H * state);
        a.span_decay = c.take<float>(ways * a.n_spans * H);
    }
    if (bwd) {
        a.chunk_state = c.take<float>(2 * a.n_chunks * H * state);
        a.token_part = c.take<float>(a.n_chunks * H * gdr::kTokenPart);
        a.head_part = c.take<float>(a.n_chunks * H * 3);
        const int64_t parts = gdr::ssm_grad_parts(a);
        if (parts > 1) a.bc_part = c.take<float>(2 * parts * a.total * a.groups * a.n);
    }
}

// Tables and gates, then the walks.
hipError_t run_ssm(gdr::SsmArgs &a, const gdr::SsmTables &t, bool bwd, hipStream_t stream) {
    hipError_t e = hipSuccess;
    if (a.gates && a.n_seq > 0) {
        if (a.cu) {
            e = gdr::launch_ssm_table(a, t, stream);
            a.spans = t.spans;
            a.span_first = t.span_first;
            a.chunks = t.chunks;
            a.chunks_used = t.chunk_first + a.n_seq;
        }
        if (e == hipSuccess) e = gdr::launch_ssm_gates(a, stream);
        if (e != hipSuccess) return e;
    }
    return bwd ? gdr::launch_ssm_bwd(a, stream) : gdr::launch_ssm_fwd(a, stream);
}

}  // namespace

extern "C" {

int gdr_short_conv_fwd(const gdr_tensor *x, const gdr_tensor *w, const gdr_tensor *bias, const gdr_tensor *cu_seqlens,
                       const gdr_tensor *s0, const gdr_tensor *y, const gdr_tensor *st, int activation,
                       hipStream_t stream) {
    return entry([&]() -> int {
        ConvIn c{x, w, bias, cu_seqlens, s0, activation};
        gdr::ConvArgs a;
        int64_t ny, nst = 0;
        int rc;
        if ((rc = plan_conv(c, 2, a))) return rc;
        const size_t e = dtype_size(x->dtype);
        if ((rc = check_tensor(y, "y", 3, &ny, e))) return rc;
        if (st && (rc = check_tensor(st, "st", 3, &nst, e))) return rc;
        if ((rc = want_dtype(y, "y", x->dtype)) || (rc = want_dtype(st, "st", x->dtype))) return rc;
        if ((rc = want_shape(y, "y", {c.B, c.T, a.ch}, "x's shape")) ||
            (rc = want_shape(st, "st", {c.N, a.width - 1, a.ch}, "[N, W - 1, channels]")))
            return rc;
        if ((rc = check_overlaps({{"x", c.sx}, {"w", c.sw}, {"bias", c.sbias}, {"cu_seqlens", c.scu}, {"s0", c.ss0}},
                                 {{"y", span_of(y, ny)}, {"st", span_of(st, nst)}})))
            return rc;
        if ((rc = check_device())) return rc;
        if ((rc = check_cu(cu_seqlens, a.n_seq, c.B * c.T, stream))) return rc;
        if (a.n_seq == 0 || (a.total == 0 && !st)) return ok();
        a.y = y->data;
        a.st = st ? st->data : nullptr;
        a.vec = a.vec && aligned16(y) && aligned16(st);
        return launch([&] { return gdr::launch_conv_fwd(a, stream); }, "short convolution kernel");
    });
}

int gdr_short_conv_bwd(const gdr_tensor *x, const gdr_tensor *w, const gdr_tensor *bias, const gdr_tensor *cu_seqlens,
                       const gdr_tensor *s0, const gdr_tensor *dy, const gdr_tensor *dst, const gdr_tensor *dx,
                       const gdr_tensor *dw, const gdr_tensor *db, const gdr_tensor *ds0, int activation,
                       void *workspace, int64_t *workspace_bytes, hipStream_t stream) {
    return entry([&]() -> int {
        ConvIn c{x, w, bias, cu_seqlens, s0, activation};
        gdr::ConvArgs a;
        int64_t ndst = 0, ndx, ndw, ndb = 0, nds0 = 0;
        Span sdy;
        int rc;
        if ((rc = plan_conv(c, 2, a))) return rc;
        const size_t e = dtype_size(x->dtype);
        if ((rc = check_rows(dy, "dy", 3, 2, e, &a.lddy, &sdy))) return rc;
        if (dst && (rc = check_tensor(dst, "dst", 3, &ndst, e))) return rc;
        if ((rc = check_tensor(dx, "dx", 3, &ndx, e)) || (rc = check_tensor(dw, "dw", 2, &ndw, 4))) return rc;
        if (db && (rc = check_tensor(db, "db", 1, &ndb, 4))) return rc;
        if (ds0 && (rc = check_tensor(ds0, "ds0", 3, &nds0, e))) return rc;
        if ((rc = want_dtype(dy, "dy", x->dtype)) || (rc = want_dtype(dst, "dst", x->dtype)) ||
            (rc = want_dtype(dx, "dx", x->dtype)) || (rc = want_dtype(dw, "dw", GDR_F32)) ||
            (rc = want_dtype(db, "db", GDR_F32)) || (rc = want_dtype(ds0, "ds0", x->dtype)))
            return rc;
        const int64_t W = a.width, ch = a.ch;
        if ((rc = want_shape(dy, "dy", {c.B, c.T, ch}, "x's shape")) || (rc = want_shape(dx, "dx", {c.B, c.T, ch}, "x's shape")) ||
            (rc = want_shape(dst, "dst", {c.N, W - 1, ch}, "[N, W - 1, channels]")) ||
            (rc = want_shape(ds0, "ds0", {c.N, W - 1, ch}, "[N, W - 1, channels]")) ||
            (rc = want_shape(dw, "dw", {ch, W}, "[channels, W]")) || (rc = want_shape(db, "db", {ch}, "[channels]")))
            return rc;
        if ((rc = check_overlaps({{"x", c.sx}, {"w", c.sw}, {"bias", c.sbias}, {"cu_seqlens", c.scu}, {"s0", c.ss0},
                                  {"dy", sdy}, {"dst", span_of(dst, ndst)}},
                                 {{"dx", span_of(dx, ndx)}, {"dw", span_of(dw, ndw)}, {"db", span_of(db, ndb)},
                                  {"ds0", span_of(ds0, nds0)}})))
            return rc;
        a.dy = dy->data;
        a.dst = dst ? dst->data : nullptr;
        a.dx = dx->data;
        a.dw = static_cast<float *>(dw->data);
        a.db = db ? static_cast<float *>(db->data) : nullptr;
        a.ds0 = ds0 ? ds0->data : nullptr;
        a.vec = a.vec && (a.lddy * static_cast<int64_t>(e)) % 16 == 0 && aligned16(dy) && aligned16(dst) && aligned16(dx) &&
                aligned16(ds0);
        const size_t need = static_cast<size_t>(gdr::conv_bwd_rows(a.total, a.ch, a.bf16, a.vec)) *
                            static_cast<size_t>(ch * (W + 1)) * 4;
        if ((rc = Workspace::check(need, workspace, workspace_bytes))) return rc == 1 ? ok() : rc;
        if ((rc = check_device())) return rc;
        if ((rc = check_cu(cu_seqlens, a.n_seq, c.B * c.T, stream))) return rc;
        Workspace ws;
        void *p;
        if ((rc = ws.get(need, workspace, stream, &p))) return rc;
        a.part = static_cast<float *>(p);
        rc = launch([&] { return gdr::launch_conv_bwd(a, stream); }, "short convolution backward kernels");
        const int rr = ws.release();
        return rc ? rc : rr;
    });
}

int gdr_short_conv_step(const gdr_tensor *x, const gdr_tensor *state, const gdr_tensor *w, const gdr_tensor *bias,
                        const gdr_tensor *y, int activation, hipStream_t stream) {
    return entry([&]() -> int {
        ConvIn c{x, w, bias, nullptr, nullptr, activation};
        gdr::ConvArgs a;
        int64_t ny, nst;
        int rc;
        if ((rc = plan_conv(c, 1, a))) return rc;
        const size_t e = dtype_size(x->dtype);
        if ((rc = check_tensor(state, "state", 3, &nst, e)) || (rc = check_tensor(y, "y", 2, &ny, e))) return rc;
        if ((rc = want_dtype(state, "state", x->dtype)) || (rc = want_dtype(y, "y", x->dtype))) return rc;
        if ((rc = want_shape(state, "state", {c.B, a.width - 1, a.ch}, "[B, W - 1, channels]")) ||
            (rc = want_shape(y, "y", {c.B, a.ch}, "x's shape")))
            return rc;
        if ((rc = check_overlaps({{"x", c.sx}, {"w", c.sw}, {"bias", c.sbias}},
                                 {{"y", span_of(y, ny)}, {"state", span_of(state, nst)}})))
            return rc;
        if ((rc = check_device())) return rc;
        if (c.B == 0) return ok();
        a.y = y->data;
        a.st = state->data;
        a.vec = a.vec && aligned16(y) && aligned16(state);
        return launch([&] { return gdr::launch_conv_step(a, stream); }, "short convolution step kernel");
    });
}

int gdr_qk_norm_rope_fwd(const gdr_tensor *q, const gdr_tensor *k, const gdr_tensor *wq, const gdr_tensor *wk,
                         const gdr_tensor *cos, const gdr_tensor *sin, const gdr_tensor *positions,
                         const gdr_tensor *oq, const gdr_tensor *ok_, int norm, float eps, int interleaved,
                         hipStream_t stream) {
    return entry([&]() -> int {
        NormIn c{q, k, wq, wk, cos, sin, positions, norm, eps, interleaved};
        gdr::NormArgs a;
        int64_t noq, nok;
        int rc;
        if ((rc = plan_norm(c, a))) return rc;
        if ((rc = check_tensor(oq, "oq", 4, &noq, 16)) || (rc = check_tensor(ok_, "ok", 4, &nok, 16))) return rc;
        if ((rc = want_dtype(oq, "oq", q->dtype)) || (rc = want_dtype(ok_, "ok", q->dtype))) return rc;
        if ((rc = want_shape(oq, "oq", {c.B, c.T, a.hq, a.d}, "q's shape")) ||
            (rc = want_shape(ok_, "ok", {c.B, c.T, a.hk, a.d}, "k's shape")))
            return rc;
        if ((rc = check_overlaps({{"q", c.sq}, {"k", c.sk}, {"wq", c.swq}, {"wk", c.swk}, {"cos", c.scos}, {"sin", c.ssin},
                                  {"positions", c.spos}},
                                 {{"oq", span_of(oq, noq)}, {"ok", span_of(ok_, nok)}})))
            return rc;
        if ((rc = check_device())) return rc;
        if (a.tokens == 0) return ok();
        a.oq = oq->data;
        a.ok = ok_->data;
        return launch([&] { return gdr::launch_norm_fwd(a, stream); }, "query/key norm kernel");
    });
}

int gdr_qk_norm_rope_bwd(const gdr_tensor *q, const gdr_tensor *k, const gdr_tensor *wq, const gdr_tensor *wk,
                         const gdr_tensor *cos, const gdr_tensor *sin, const gdr_tensor *positions,
                         const gdr_tensor *doq, const gdr_tensor *dok, const gdr_tensor *dq, const gdr_tensor *dk,
                         const gdr_tensor *dwq, const gdr_tensor *dwk, int norm, float eps, int interleaved,
                         void *workspace, int64_t *workspace_bytes, hipStream_t stream) {
    return entry([&]() -> int {
        NormIn c{q, k, wq, wk, cos, sin, positions, norm, eps, interleaved};
        gdr::NormArgs a;
        int64_t ndq, ndk, ndwq = 0, ndwk = 0;
        Span sdoq, sdok;
        int rc;
        if ((rc = plan_norm(c, a))) return rc;
        if ((rc = check_rows(doq, "doq", 4, 2, 16, &a.lddoq, &sdoq)) || (rc = check_rows(dok, "dok", 4, 2, 16, &a.lddok, &sdok)))
            return rc;
        if ((rc = check_tensor(dq, "dq", 4, &ndq, 16)) || (rc = check_tensor(dk, "dk", 4, &ndk, 16))) return rc;
        if (dwq && (rc = check_tensor(dwq, "dwq", 1, &ndwq, 4))) return rc;
        if (dwk && (rc = check_tensor(dwk, "dwk", 1, &ndwk, 4))) return rc;
        if ((rc = want_dtype(doq, "doq", q->dtype)) || (rc = want_dtype(dok, "dok", q->dtype)) ||
            (rc = want_dtype(dq, "dq", q->dtype)) || (rc = want_dtype(dk, "dk", q->dtype)) ||
            (rc = want_dtype(dwq, "dwq", GDR_F32)) || (rc = want_dtype(dwk, "dwk", GDR_F32)))
            return rc;
        const int64_t d = a.d;
        if ((rc = want_shape(doq, "doq", {c.B, c.T, a.hq, d}, "q's shape")) ||
            (rc = want_shape(dok, "dok", {c.B, c.T, a.hk, d}, "k's shape")) ||
            (rc = want_shape(dq, "dq", {c.B, c.T, a.hq, d}, "q's shape")) ||
            (rc = want_shape(dk, "dk", {c.B, c.T, a.hk, d}, "k's shape")) || (rc = want_shape(dwq, "dwq", {d}, "[d]")) ||
            (rc = want_shape(dwk, "dwk", {d}, "[d]")))
            return rc;
        if ((rc = check_overlaps({{"q", c.sq}, {"k", c.sk}, {"wq", c.swq}, {"wk", c.swk}, {"cos", c.scos}, {"sin", c.ssin},
                                  {"positions", c.spos}, {"doq", sdoq}, {"dok", sdok}},
                                 {{"dq", span_of(dq, ndq)}, {"dk", span_of(dk, ndk)}, {"dwq", span_of(dwq, ndwq)},
                                  {"dwk", span_of(dwk, ndwk)}})))
            return rc;
        a.doq = doq->data;
        a.dok = dok->data;
        a.dq = dq->data;
        a.dk = dk->data;
        a.dwq = dwq ? static_cast<float *>(dwq->data) : nullptr;
        a.dwk = dwk ? static_cast<float *>(dwk->data) : nullptr;
        const bool sums = a.dwq || a.dwk;
        const size_t need = sums ? static_cast<size_t>(gdr::norm_bwd_blocks(a)) * static_cast<size_t>(d) * 4 : 0;
        if ((rc = Workspace::check(need, workspace, workspace_bytes))) return rc == 1 ? ok() : rc;
        if ((rc = check_device())) return rc;
        Workspace ws;
        void *p;
        if ((rc = ws.get(need, workspace, stream, &p))) return rc;
        // without tokens the sums are zero: the second kernel reads no partial row
        a.part = sums ? static_cast<float *>(p ? p : static_cast<void *>(dwq ? dwq->data : dwk->data)) : nullptr;
        if (a.tokens == 0 && !sums) return ok();
        rc = launch([&] { return gdr::launch_norm_bwd(a, stream); }, "query/key norm backward kernels");
        const int rr = ws.release();
        return rc ? rc : rr;
    });
}

int gdr_ssm_step(const gdr_tensor *x, const gdr_tensor *dt, const gdr_tensor *A, const gdr_tensor *b, const gdr_tensor *c,
                 const gdr_tensor *D, const gdr_tensor *dt_bias, const gdr_tensor *h, const gdr_tensor *y,
                 hipStream_t stream) {
    return entry([&]() -> int {
        SsmIn s{x, dt, A, b, c, D, dt_bias, nullptr, nullptr};
        gdr::SsmArgs a;
        int64_t nh, ny;
        int rc;
        if ((rc = plan_ssm(s, 1, a))) return rc;
        if ((rc = check_tensor(h, "h", 4, &nh, 16)) || (rc = check_tensor(y, "y", 3, &ny, 16))) return rc;
        if ((rc = want_dtype(h, "h", GDR_F32)) || (rc = want_dtype(y, "y", x->dtype))) return rc;
        if ((rc = want_shape(h, "h", {s.B, a.heads, a.n, a.p}, "[B, H, n, p]")) ||
            (rc = want_shape(y, "y", {s.B, a.heads, a.p}, "x's shape")))
            return rc;
        if ((rc = check_overlaps({{"x", s.sx}, {"dt", s.sdt}, {"A", s.sA}, {"b", s.sb}, {"c", s.sc}, {"D", s.sD}, {"dt_bias", s.sbias}},
                                 {{"y", span_of(y, ny)}, {"h", span_of(h, nh)}})))
            return rc;
        if ((rc = check_device())) return rc;
        if (s.B == 0) return ok();
        a.ht = static_cast<float *>(h->data);
        a.y = y->data;
        return launch([&] { return gdr::launch_ssm_step(a, stream); }, "state space step kernel");
    });
}

int gdr_ssm_scan_fwd(const gdr_tensor *x, const gdr_tensor *dt, const gdr_tensor *A, const gdr_tensor *b,
                     const gdr_tensor *c, const gdr_tensor *D, const gdr_tensor *dt_bias, const gdr_tensor *cu_seqlens,
                     const gdr_tensor *h0, const gdr_tensor *y, const gdr_tensor *ht, void *workspace,
                     int64_t *workspace_bytes, hipStream_t stream) {
    return entry([&]() -> int {
        SsmIn s{x, dt, A, b, c, D, dt_bias, cu_seqlens, h0};
        gdr::SsmArgs a;
        int64_t ny, nht = 0;
        int rc;
        if ((rc = plan_ssm(s, 2, a))) return rc;
        if ((rc = check_tensor(y, "y", 4, &ny, 16))) return rc;
        if (ht && (rc = check_tensor(ht, "ht", 4, &nht, 16))) return rc;
        if ((rc = want_dtype(y, "y", x->dtype)) || (rc = want_dtype(ht, "ht", GDR_F32))) return rc;
        if ((rc = want_shape(y, "y", {s.B, s.T, a.heads, a.p}, "x's shape")) ||
            (rc = want_shape(ht, "ht", {s.N, a.heads, a.n, a.p}, "[N, H, n, p]")))
            return rc;
        if ((rc = check_overlaps({{"x", s.sx}, {"dt", s.sdt}, {"A", s.sA}, {"b", s.sb}, {"c", s.sc}, {"D", s.sD},
                                  {"dt_bias", s.sbias}, {"cu_seqlens", s.scu}, {"h0", s.sh0}},
                                 {{"y", span_of(y, ny)}, {"ht", span_of(ht, nht)}})))
            return rc;
        a.y = y->data;
        a.ht = ht ? static_cast<float *>(ht->data) : nullptr;
        Carve size{nullptr};
        gdr::SsmTables t;
        carve_ssm(a, false, size, t);
        if ((rc = Workspace::check(size.used, workspace, workspace_bytes))) return rc == 1 ? ok() : rc;
        if ((rc = check_device())) return rc;
        if ((rc = check_cu(cu_seqlens, a.n_seq, s.B * s.T, stream))) return rc;
        Workspace ws;
        void *p;
        if ((rc = ws.get(size.used, workspace, stream, &p))) return rc;
        if (a.n_seq == 0 || (a.total == 0 && !ht)) return ok();
        Carve parts{static_cast<unsigned char *>(p)};
        carve_ssm(a, false, parts, t);
        rc = launch([&] { return run_ssm(a, t, false, stream); }, "state space scan kernels");
        const int rr = ws.release();
        return rc ? rc : rr;
    });
}

int gdr_ssm_scan_bwd(const gdr_tensor *x, const gdr_tensor *dt, const gdr_tensor *A, const gdr_tensor *b,
                     const gdr_tensor *c, const gdr_tensor *D, const gdr_tensor *dt_bias, const gdr_tensor *cu_seqlens,
                     const gdr_tensor *h0, const gdr_tensor *dy, const gdr_tensor *dht, const gdr_tensor *dx,
                     const gdr_tensor *ddt, const gdr_tensor *dA, const gdr_tensor *db, const gdr_tensor *dc,
                     const gdr_tensor *dD, const gdr_tensor *ddt_bias, const gdr_tensor *dh0, void *workspace,
                     int64_t *workspace_bytes, hipStream_t stream) {
    return entry([&]() -> int {
        SsmIn s{x, dt, A, b, c, D, dt_bias, cu_seqlens, h0};
        gdr::SsmArgs a;
        int64_t ndht = 0;
        Span sdy;
        int rc;
        if ((rc = plan_ssm(s, 2, a))) return rc;
        if ((rc = check_rows(dy, "dy", 4, 2, 16, &a.lddy, &sdy))) return rc;
        if (dht && (rc = check_tensor(dht, "dht", 4, &ndht, 16))) return rc;
        struct Out {
            const gdr_tensor *t;
            const char *name;
            int ndim;
            size_t align;
            int32_t dtype;
            bool needed;
            int64_t n;
        } outs[] = {{dx, "dx", 4, 16, x->dtype, true, 0},   {ddt, "ddt", 3, 4, dt->dtype, true, 0},
                    {dA, "dA", 1, 4, GDR_F32, true, 0},     {db, "db", 4, 16, x->dtype, true, 0},
                    {dc, "dc", 4, 16, x->dtype, true, 0},   {dD, "dD", 1, 4, GDR_F32, false, 0},
                    {ddt_bias, "ddt_bias", 1, 4, GDR_F32, false, 0}, {dh0, "dh0", 4, 16, GDR_F32, false, 0}};
        for (Out &o : outs) {
            if (!o.t && !o.needed) continue;
            if ((rc = check_tensor(o.t, o.name, o.ndim, &o.n, o.align))) return rc;
            if ((rc = want_dtype(o.t, o.name, o.dtype))) return rc;
        }
        if ((rc = want_dtype(dy, "dy", x->dtype)) || (rc = want_dtype(dht, "dht", GDR_F32))) return rc;
        const int64_t H = a.heads, G = a.groups;
        if ((rc = want_shape(dy, "dy", {s.B, s.T, H, a.p}, "x's shape")) ||
            (rc = want_shape(dht, "dht", {s.N, H, a.n, a.p}, "[N, H, n, p]")) ||
            (rc = want_shape(dx, "dx", {s.B, s.T, H, a.p}, "x's shape")) ||
            (rc = want_shape(ddt, "ddt", {s.B, s.T, H}, "dt's shape")) || (rc = want_shape(dA, "dA", {H}, "[H]")) ||
            (rc = want_shape(db, "db", {s.B, s.T, G, a.n}, "b's shape")) ||
            (rc = want_shape(dc, "dc", {s.B, s.T, G, a.n}, "c's shape")) || (rc = want_shape(dD, "dD", {H}, "[H]")) ||
            (rc = want_shape(ddt_bias, "ddt_bias", {H}, "[H]")) ||
            (rc = want_shape(dh0, "dh0", {s.N, H, a.n, a.p}, "[N, H, n, p]")))
            return rc;
        if (a.lddy * static_cast<int64_t>(dtype_size(x->dtype)) > kMaxRow)
            return fail(GDR_ESTRIDE, "dy: rows may be at most %lld bytes apart", (long long)kMaxRow);
        if ((rc = check_overlaps({{"x", s.sx}, {"dt", s.sdt}, {"A", s.sA}, {"b", s.sb}, {"c", s.sc}, {"D", s.sD},
                                  {"dt_bias", s.sbias}, {"cu_seqlens", s.scu}, {"h0", s.sh0}, {"dy", sdy},
                                  {"dht", span_of(dht, ndht)}},
                                 {{"dx", span_of(dx, outs[0].n)}, {"ddt", span_of(ddt, outs[1].n)},
                                  {"dA", span_of(dA, outs[2].n)}, {"db", span_of(db, outs[3].n)},
                                  {"dc", span_of(dc, outs[4].n)}, {"dD", span_of(dD, outs[5].n)},
                                  {"ddt_bias", span_of(ddt_bias, outs[6].n)}, {"dh0", span_of(dh0, outs[7].n)}})))
            return rc;
        auto f32 = [](const gdr_tensor *t) { return t ? static_cast<float *>(t->data) : nullptr; };
        a.dy = dy->data;
        a.dht = f32(dht);
        a.dx = dx->data;
        a.ddt = ddt->data;
        a.db = db->data;
        a.dc = dc->data;
        a.dA = f32(dA);
        a.dD = f32(dD);
        a.dbias = f32(ddt_bias);
        a.dh0 = f32(dh0);
        Carve size{nullptr};
        gdr::SsmTables t;
        carve_ssm(a, true, size, t);
        if ((rc = Workspace::check(size.used, workspace, workspace_bytes))) return rc == 1 ? ok() : rc;
        if ((rc = check_device())) return rc;
        if ((rc = check_cu(cu_seqlens, a.n_seq, s.B * s.T, stream))) return rc;
        Workspace ws;
        void *p;
        if ((rc = ws.get(size.used, workspace, stream, &p))) return rc;
        Carve parts{static_cast<unsigned char *>(p)};
        carve_ssm(a, true, parts, t);
        rc = launch([&] { return run_ssm(a, t, true, stream); }, "state space scan backward kernels");
        const int rr = ws.release();
        return rc ? rc : rr;
    });
}

}  // extern "C"
