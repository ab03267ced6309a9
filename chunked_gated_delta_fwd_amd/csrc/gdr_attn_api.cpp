// Host side of softmax attention and its paged cache (include/gdr.h):
// validation, workspace and launches, by the rules of gdr_mixer_api.cpp.
#include "gdr.h"

#include <hip/hip_runtime.h>

#include "gdr_attn.h"
#include "gdr_entry.h"

namespace {

using namespace gdr::host;

constexpr int64_t kMostRows = 1 << 30;          // tokens of a call, so that differences of places fit 32 bits
constexpr int64_t kMostApart = 1 << 25;         // bytes between rows, so that offsets in a tile do
constexpr int64_t kMostHeads = 65536;

int close_rows(const gdr_tensor *t, const char *name, int64_t ld) {
    if (ld * static_cast<int64_t>(dtype_size(t->dtype)) > kMostApart)
        return fail(GDR_ESTRIDE, "%s: rows may be at most 32 MiB apart (they are %lld elements)", name, (long long)ld);
    return GDR_OK;
}

struct AttnIn {
    const gdr_tensor *q, *k, *v, *cu, *cuk;
    int causal;
    int64_t window;
    float scale;
    Span sq, sk, sv, scu, scuk;
    int64_t B, Tq, Tk;
};

int plan_attn(AttnIn &c, gdr::AttnArgs &a) {
    std::memset(&a, 0, sizeof(a));
    int64_t n;
    int rc;
    if (!c.q) return fail(GDR_EINVAL, "q: descriptor is NULL");
    if (!is_float(c.q)) return fail(GDR_EDTYPE, "q: dtype must be bf16 or f32, got %s", dtype_name(c.q->dtype));
    if ((rc = check_rows(c.q, "q", 4, 2, 16, &a.ldq, &c.sq)) || (rc = check_rows(c.k, "k", 4, 2, 16, &a.ldk, &c.sk)) ||
        (rc = check_rows(c.v, "v", 4, 2, 16, &a.ldv, &c.sv)))
        return rc;
    if (c.cu) {
        if ((rc = check_tensor(c.cu, "cu_seqlens", 1, &n, 4))) return rc;
        c.scu = span_of(c.cu, n);
    }
    if (c.cuk) {
        if (!c.cu) return fail(GDR_EINVAL, "cu_seqlens_k without cu_seqlens");
        if ((rc = check_tensor(c.cuk, "cu_seqlens_k", 1, &n, 4))) return rc;
        c.scuk = span_of(c.cuk, n);
    }
    c.B = c.q->shape[0];
    c.Tq = c.q->shape[1];
    c.Tk = c.k->shape[1];
    const int64_t hq = c.q->shape[2], hk = c.k->shape[2], d = c.q->shape[3];
    int64_t N;
    if ((rc = sequences(c.cu, c.B, c.Tq > c.Tk ? c.Tq : c.Tk, &N))) return rc;
    if (c.B * c.Tq > kMostRows || c.B * c.Tk > kMostRows) return fail(GDR_ESHAPE, "B * T exceeds 2^30 tokens");
    if ((rc = want_dtype(c.k, "k", c.q->dtype)) || (rc = want_dtype(c.v, "v", c.q->dtype)) ||
        (rc = want_dtype(c.cuk, "cu_seqlens_k", GDR_I32)))
        return rc;
    if (d != 64 && d != 128) return fail(GDR_ESHAPE, "q: head dim must be 64 or 128, got %lld", (long long)d);
    if (hq < 1 || hk < 1 || hq > kMostHeads || hk > kMostHeads)
        return fail(GDR_ESHAPE, "head counts must be between 1 and 65536");
    if (hq % hk) return fail(GDR_ESHAPE, "Hq = %lld must be a multiple of Hk = %lld", (long long)hq, (long long)hk);
    if ((rc = want_shape(c.k, "k", {c.B, c.Tk, hk, d}, "[B, Tk, Hk, d] with q's B and d")) ||
        (rc = want_shape(c.v, "v", {c.B, c.Tk, hk, d}, "k's shape")))
        return rc;
    if (c.cu && !c.cuk && c.Tk != c.Tq)
        return fail(GDR_ESHAPE, "k: %lld tokens for q's %lld need cu_seqlens_k", (long long)c.Tk, (long long)c.Tq);
    if (c.cuk && (rc = want_shape(c.cuk, "cu_seqlens_k", {N + 1}, "[N + 1]"))) return rc;
    if ((rc = close_rows(c.q, "q", a.ldq)) || (rc = close_rows(c.k, "k", a.ldk)) || (rc = close_rows(c.v, "v", a.ldv))) return rc;
    if (c.window < 0) return fail(GDR_EINVAL, "window must not be negative");
    if (c.window > 0 && !c.causal) return fail(GDR_EINVAL, "window needs causal");
    if (!std::isfinite(c.scale)) return fail(GDR_EINVAL, "scale must be finite");
    a.q = c.q->data;
    a.k = c.k->data;
    a.v = c.v->data;
    a.cu = c.cu ? static_cast<const int32_t *>(c.cu->data) : nullptr;
    a.cuk = c.cuk ? static_cast<const int32_t *>(c.cuk->data) : nullptr;
    a.n_seq = N;
    a.seq_q = c.Tq;
    a.seq_k = c.Tk;
    a.total_q = live_tokens(N, c.B, c.Tq);
    a.total_k = live_tokens(N, c.B, c.Tk);
    a.hq = static_cast<int32_t>(hq);
    a.hk = static_cast<int32_t>(hk);
    a.d = static_cast<int32_t>(d);
    a.bf16 = c.q->dtype == GDR_BF16;
    a.causal = c.causal != 0;
    a.window = c.window < kMostRows ? c.window : 0;
    a.scale = c.scale;
    return GDR_OK;
}

// A launch holds fewer than 2^32 threads along x.
int fits(int64_t blocks) {
    if (blocks >= 1 << 24)
        return fail(GDR_ESHAPE, "the call would take %lld blocks of 256 threads, more than the 2^24 - 1 of a launch", (long long)blocks);
    return GDR_OK;
}

// Dimensions of a tensor with a number a token: [tokens], or rows of a batch.
int token_dims(const gdr_tensor *t) { return t && t->ndim == 1 ? 1 : 2; }

// Both offsets' contents, with the opt-in check on.
int check_offsets(const AttnIn &c, const gdr::AttnArgs &a, hipStream_t stream) {
    const int rc = check_cu(c.cu, a.n_seq, c.B * c.Tq, stream);
    return rc ? rc : check_cu(c.cuk, a.n_seq, c.B * c.Tk, stream);
}

}  // namespace

extern "C" {

int gdr_attn_fwd(const gdr_tensor *q, const gdr_tensor *k, const gdr_tensor *v, const gdr_tensor *cu_seqlens,
                 const gdr_tensor *cu_seqlens_k, const gdr_tensor *o, const gdr_tensor *lse, int causal, int64_t window,
                 float scale, void *workspace, int64_t *workspace_bytes, hipStream_t stream) {
    return entry([&]() -> int {
        AttnIn c{q, k, v, cu_seqlens, cu_seqlens_k, causal, window, scale};
        gdr::AttnArgs a;
        int64_t no, nl = 0;
        int rc;
        if ((rc = plan_attn(c, a))) return rc;
        if ((rc = check_tensor(o, "o", 4, &no, 16))) return rc;
        if (lse && (rc = check_tensor(lse, "lse", 3, &nl, 4))) return rc;
        if ((rc = want_dtype(o, "o", q->dtype)) || (rc = want_dtype(lse, "lse", GDR_F32)) ||
            (rc = want_shape(o, "o", {c.B, c.Tq, a.hq, a.d}, "q's shape")) ||
            (rc = want_shape(lse, "lse", {c.B, c.Tq, a.hq}, "[B, T, Hq]")))
            return rc;
        if ((rc = check_overlaps({{"q", c.sq}, {"k", c.sk}, {"v", c.sv}, {"cu_seqlens", c.scu}, {"cu_seqlens_k", c.scuk}},
                                 {{"o", span_of(o, no)}, {"lse", span_of(lse, nl)}})))
            return rc;
        a.o = o->data;
        a.lse = lse ? static_cast<float *>(lse->data) : nullptr;
        gdr::attn_split(a);
        if ((rc = fits(gdr::attn_fwd_grid(a)))) return rc;
        Carve sizes{nullptr};
        const auto carve = [&](Carve &w) {
            const int64_t runs = gdr::attn_cut_blocks(a) * a.splits * a.run_rows;
            a.run_o = w.take<float>(runs * a.d);
            a.run_stat = w.take<float>(runs * 2);
        };
        carve(sizes);
        if ((rc = Workspace::check(sizes.used, workspace, workspace_bytes))) return rc == 1 ? ok() : rc;
        if ((rc = check_device())) return rc;
        if ((rc = check_offsets(c, a, stream))) return rc;
        if (a.total_q == 0) return ok();
        Workspace ws;
        void *p;
        if ((rc = ws.get(sizes.used, workspace, stream, &p))) return rc;
        Carve parts{static_cast<unsigned char *>(p)};
        carve(parts);
        rc = launch([&] { return gdr::launch_attn_fwd(a, stream); }, "attention kernels");
        const int rr = ws.release();
        return rc ? rc : rr;
    });
}

int gdr_attn_bwd(const gdr_tensor *q, const gdr_tensor *k, const gdr_tensor *v, const gdr_tensor *cu_seqlens,
                 const gdr_tensor *cu_seqlens_k, const gdr_tensor *o, const gdr_tensor *lse, const gdr_tensor *dout,
                 const gdr_tensor *dq, const gdr_tensor *dk, const gdr_tensor *dv, int causal, int64_t window,
                 float scale, void *workspace, int64_t *workspace_bytes, hipStream_t stream) {
    return entry([&]() -> int {
        AttnIn c{q, k, v, cu_seqlens, cu_seqlens_k, causal, window, scale};
        gdr::AttnArgs a;
        Span so, sdo;
        int64_t nl, ndq, ndk, ndv;
        int rc;
        if ((rc = plan_attn(c, a))) return rc;
        if ((rc = check_rows(o, "o", 4, 2, 16, &a.ldo, &so)) || (rc = check_tensor(lse, "lse", 3, &nl, 4)) ||
            (rc = check_rows(dout, "do", 4, 2, 16, &a.lddo, &sdo)) || (rc = check_tensor(dq, "dq", 4, &ndq, 16)) ||
            (rc = check_tensor(dk, "dk", 4, &ndk, 16)) || (rc = check_tensor(dv, "dv", 4, &ndv, 16)))
            return rc;
        const int32_t dt = q->dtype;
        if ((rc = want_dtype(o, "o", dt)) || (rc = want_dtype(lse, "lse", GDR_F32)) || (rc = want_dtype(dout, "do", dt)) ||
            (rc = want_dtype(dq, "dq", dt)) || (rc = want_dtype(dk, "dk", dt)) || (rc = want_dtype(dv, "dv", dt)))
            return rc;
        if ((rc = want_shape(o, "o", {c.B, c.Tq, a.hq, a.d}, "q's shape")) ||
            (rc = want_shape(lse, "lse", {c.B, c.Tq, a.hq}, "[B, T, Hq]")) ||
            (rc = want_shape(dout, "do", {c.B, c.Tq, a.hq, a.d}, "q's shape")) ||
            (rc = want_shape(dq, "dq", {c.B, c.Tq, a.hq, a.d}, "q's shape")) ||
            (rc = want_shape(dk, "dk", {c.B, c.Tk, a.hk, a.d}, "k's shape")) ||
            (rc = want_shape(dv, "dv", {c.B, c.Tk, a.hk, a.d}, "k's shape")))
            return rc;
        if ((rc = close_rows(o, "o", a.ldo)) || (rc = close_rows(dout, "do", a.lddo))) return rc;
        if ((rc = check_overlaps({{"q", c.sq}, {"k", c.sk}, {"v", c.sv}, {"cu_seqlens", c.scu}, {"cu_seqlens_k", c.scuk},
                                  {"o", so}, {"lse", span_of(lse, nl)}, {"do", sdo}},
                                 {{"dq", span_of(dq, ndq)}, {"dk", span_of(dk, ndk)}, {"dv", span_of(dv, ndv)}})))
            return rc;
        a.o = o->data;
        a.lse = static_cast<float *>(lse->data);
        a.dout = dout->data;
        a.dq = dq->data;
        a.dk = dk->data;
        a.dv = dv->data;
        gdr::attn_bwd_split(a);
        if ((rc = fits(gdr::attn_bwd_grid(a)))) return rc;
        Carve sizes{nullptr};
        const auto carve = [&](Carve &w) {
            a.stat = w.take<float>(2 * static_cast<int64_t>(a.hq) * a.total_q);
            a.part = a.parts > 1 ? w.take<float>(2 * static_cast<int64_t>(a.parts) * a.total_k * a.hk * a.d) : nullptr;
            a.part_q = a.runs_q > 1 ? w.take<float>(static_cast<int64_t>(a.runs_q) * a.total_q * a.hq * a.d) : nullptr;
        };
        carve(sizes);
        if ((rc = Workspace::check(sizes.used, workspace, workspace_bytes))) return rc == 1 ? ok() : rc;
        if ((rc = check_device())) return rc;
        if ((rc = check_offsets(c, a, stream))) return rc;
        if (a.total_q == 0 && a.total_k == 0) return ok();
        Workspace ws;
        void *p;
        if ((rc = ws.get(sizes.used, workspace, stream, &p))) return rc;
        Carve parts{static_cast<unsigned char *>(p)};
        carve(parts);
        rc = launch([&] { return gdr::launch_attn_bwd(a, stream); }, "attention backward kernels");
        const int rr = ws.release();
        return rc ? rc : rr;
    });
}

int gdr_attn_paged_step(const gdr_tensor *q, const gdr_tensor *k_pages, const gdr_tensor *v_pages,
                        const gdr_tensor *block_table, const gdr_tensor *lens, const gdr_tensor *o, int64_t window,
                        float scale, void *workspace, int64_t *workspace_bytes, hipStream_t stream) {
    return entry([&]() -> int {
        gdr::PagedArgs a;
        std::memset(&a, 0, sizeof(a));
        Span sq;
        int64_t nk, nv, nt, nl, no;
        int rc;
        if (!q) return fail(GDR_EINVAL, "q: descriptor is NULL");
        if (!is_float(q)) return fail(GDR_EDTYPE, "q: dtype must be bf16 or f32, got %s", dtype_name(q->dtype));
        if ((rc = check_rows(q, "q", 3, 1, 16, &a.ldq, &sq)) || (rc = check_tensor(k_pages, "k_pages", 4, &nk, 16)) ||
            (rc = check_tensor(v_pages, "v_pages", 4, &nv, 16)) || (rc = check_tensor(block_table, "block_table", 2, &nt, 4)) ||
            (rc = check_tensor(lens, "lens", 1, &nl, 4)) || (rc = check_tensor(o, "o", 3, &no, 16)))
            return rc;
        if ((rc = want_dtype(k_pages, "k_pages", q->dtype)) || (rc = want_dtype(v_pages, "v_pages", q->dtype)) ||
            (rc = want_dtype(block_table, "block_table", GDR_I32)) || (rc = want_dtype(lens, "lens", GDR_I32)) ||
            (rc = want_dtype(o, "o", q->dtype)))
            return rc;
        const int64_t N = q->shape[0], hq = q->shape[1], d = q->shape[2];
        const int64_t P = k_pages->shape[0], page = k_pages->shape[1], hk = k_pages->shape[2], M = block_table->shape[1];
        if (d != 64 && d != 128) return fail(GDR_ESHAPE, "q: head dim must be 64 or 128, got %lld", (long long)d);
        if (hq < 1 || hk < 1 || hq > kMostHeads || hk > kMostHeads)
            return fail(GDR_ESHAPE, "head counts must be between 1 and 65536");
        if (hq % hk) return fail(GDR_ESHAPE, "Hq = %lld must be a multiple of Hk = %lld", (long long)hq, (long long)hk);
        if (N > kMostRows) return fail(GDR_ESHAPE, "q: at most 2^30 sequences are supported");
        if (page < 1 || page > 65536) return fail(GDR_ESHAPE, "k_pages: pages of 1 to 65536 tokens are supported, got %lld", (long long)page);
        if (P > 0x7FFFFFFF / page) return fail(GDR_ESHAPE, "k_pages: more than 2^31 - 1 tokens in all pages");
        if (M > kMostRows / page) return fail(GDR_ESHAPE, "block_table: more than 2^30 tokens a sequence");
        if ((rc = want_shape(k_pages, "k_pages", {P, page, hk, d}, "[pages, page, Hk, d] with q's d")) ||
            (rc = want_shape(v_pages, "v_pages", {P, page, hk, d}, "k_pages' shape")) ||
            (rc = want_shape(block_table, "block_table", {N, M}, "[N, pages of a sequence]")) ||
            (rc = want_shape(lens, "lens", {N}, "[N]")) || (rc = want_shape(o, "o", {N, hq, d}, "q's shape")))
            return rc;
        if (window < 0) return fail(GDR_EINVAL, "window must not be negative");
        if (!std::isfinite(scale)) return fail(GDR_EINVAL, "scale must be finite");
        if ((rc = check_overlaps({{"q", sq}, {"k_pages", span_of(k_pages, nk)}, {"v_pages", span_of(v_pages, nv)},
                                  {"block_table", span_of(block_table, nt)}, {"lens", span_of(lens, nl)}},
                                 {{"o", span_of(o, no)}})))
            return rc;
        a.q = q->data;
        a.k = k_pages->data;
        a.v = v_pages->data;
        a.table = static_cast<const int32_t *>(block_table->data);
        a.lens = static_cast<const int32_t *>(lens->data);
        a.o = o->data;
        a.n_seq = N;
        a.pages = P;
        a.width = P > 0 ? M : 0;   // without a page there is no key
        a.window = window < kMostRows ? window : 0;
        a.page = static_cast<int32_t>(page);
        a.hq = static_cast<int32_t>(hq);
        a.hk = static_cast<int32_t>(hk);
        a.d = static_cast<int32_t>(d);
        a.bf16 = q->dtype == GDR_BF16;
        a.scale = scale;
        // ceil(2^shift / page) with 2^(shift - 32) < page <= 2^(shift - 31): its excess times j stays below
        // 2^shift for j < 2^31
        int shift = 31;
        while ((int64_t{1} << (shift - 31)) < page) ++shift;
        a.magic = static_cast<uint32_t>(((int64_t{1} << shift) + page - 1) / page);
        a.shift = shift;
        gdr::paged_split(a);
        if ((rc = fits(gdr::paged_grid(a)))) return rc;
        Carve sizes{nullptr};
        const auto carve = [&](Carve &w) {
            const int64_t chunks = a.splits > 1 ? N * hq * a.splits : 0;
            a.part = w.take<float>(chunks * d);
            a.stat = w.take<float>(chunks * 2);
        };
        carve(sizes);
        if ((rc = Workspace::check(sizes.used, workspace, workspace_bytes))) return rc == 1 ? ok() : rc;
        if ((rc = check_device())) return rc;
        if (N == 0) return ok();
        Workspace ws;
        void *p;
        if ((rc = ws.get(sizes.used, workspace, stream, &p))) return rc;
        Carve parts{static_cast<unsigned char *>(p)};
        carve(parts);
        rc = launch([&] { return gdr::launch_paged_step(a, stream); }, "paged attention kernels");
        const int rr = ws.release();
        return rc ? rc : rr;
    });
}

int gdr_page_store(const gdr_tensor *k, const gdr_tensor *v, const gdr_tensor *slots, const gdr_tensor *k_pages,
                   const gdr_tensor *v_pages, hipStream_t stream) {
    return entry([&]() -> int {
        gdr::StoreArgs a;
        std::memset(&a, 0, sizeof(a));
        Span sk, sv;
        int64_t ns, nk, nv;
        int rc;
        if (!k) return fail(GDR_EINVAL, "k: descriptor is NULL");
        if (!is_float(k)) return fail(GDR_EDTYPE, "k: dtype must be bf16 or f32, got %s", dtype_name(k->dtype));
        if ((rc = check_rows(k, "k", 4, 2, 16, &a.ldk, &sk)) || (rc = check_rows(v, "v", 4, 2, 16, &a.ldv, &sv)) ||
            (rc = check_tensor(slots, "slots", token_dims(slots), &ns, 4)) || (rc = check_tensor(k_pages, "k_pages", 4, &nk, 16)) ||
            (rc = check_tensor(v_pages, "v_pages", 4, &nv, 16)))
            return rc;
        if ((rc = want_dtype(v, "v", k->dtype)) || (rc = want_dtype(slots, "slots", GDR_I32)) ||
            (rc = want_dtype(k_pages, "k_pages", k->dtype)) || (rc = want_dtype(v_pages, "v_pages", k->dtype)))
            return rc;
        const int64_t B = k->shape[0], T = k->shape[1], hk = k->shape[2], d = k->shape[3];
        const int64_t P = k_pages->shape[0], page = k_pages->shape[1];
        const int64_t e = static_cast<int64_t>(dtype_size(k->dtype));
        if (B > 0 && T > kMostRows / B) return fail(GDR_ESHAPE, "B * T exceeds 2^30 tokens");
        if (hk < 1 || hk > kMostHeads || d < 1 || d > kMostHeads || (hk * d * e) % 16)
            return fail(GDR_ESHAPE, "k: Hk * d must be a positive multiple of 16 bytes, got %lld * %lld elements", (long long)hk,
                        (long long)d);
        if (page < 1 || page > 65536) return fail(GDR_ESHAPE, "k_pages: pages of 1 to 65536 tokens are supported, got %lld", (long long)page);
        if (P > 0x7FFFFFFF / page) return fail(GDR_ESHAPE, "k_pages: more than 2^31 - 1 tokens in all pages");
        if ((rc = want_shape(v, "v", {B, T, hk, d}, "k's shape")) ||
            (rc = slots->ndim == 1 ? want_shape(slots, "slots", {B * T}, "[B * T]") : want_shape(slots, "slots", {B, T}, "[B, T]")) ||
            (rc = want_shape(k_pages, "k_pages", {P, page, hk, d}, "[pages, page, Hk, d] with k's Hk and d")) ||
            (rc = want_shape(v_pages, "v_pages", {P, page, hk, d}, "k_pages' shape")))
            return rc;
        if ((rc = check_overlaps({{"k", sk}, {"v", sv}, {"slots", span_of(slots, ns)}},
                                 {{"k_pages", span_of(k_pages, nk)}, {"v_pages", span_of(v_pages, nv)}})))
            return rc;
        a.k = k->data;
        a.v = v->data;
        a.slots = static_cast<const int32_t *>(slots->data);
        a.kp = k_pages->data;
        a.vp = v_pages->data;
        a.tokens = B * T;
        a.rows = P * page;
        a.row_bytes = hk * d * e;
        a.ldk = a.ldk * e;
        a.ldv = a.ldv * e;
        if ((rc = fits(gdr::page_store_grid(a)))) return rc;
        if ((rc = check_device())) return rc;
        if (a.tokens == 0 || a.rows == 0) return ok();
        return launch([&] { return gdr::launch_page_store(a, stream); }, "page store kernel");
    });
}

int gdr_page_plan(const gdr_tensor *past, const gdr_tensor *fresh, const gdr_tensor *free_pages,
                  const gdr_tensor *block_table, const gdr_tensor *cu_seqlens, const gdr_tensor *lens,
                  const gdr_tensor *positions, const gdr_tensor *slots, const gdr_tensor *used, int32_t page,
                  hipStream_t stream) {
    return entry([&]() -> int {
        gdr::PlanArgs a;
        std::memset(&a, 0, sizeof(a));
        struct Arg {
            const gdr_tensor *t;
            const char *name;
            int ndim;
            Span span;
        } args[] = {{past, "past", 1, {}},         {fresh, "new", 1, {}},   {free_pages, "free_pages", 1, {}},
                    {block_table, "block_table", 2, {}}, {cu_seqlens, "cu_seqlens", 1, {}}, {lens, "lens", 1, {}},
                    {positions, "positions", token_dims(positions), {}}, {slots, "slots", token_dims(slots), {}}, {used, "used", 1, {}}};
        int rc;
        for (Arg &x : args) {
            int64_t n;
            if ((rc = check_tensor(x.t, x.name, x.ndim, &n, 4)) || (rc = want_dtype(x.t, x.name, GDR_I32))) return rc;
            x.span = span_of(x.t, n);
        }
        const int64_t N = past->shape[0], M = block_table->shape[1], T = positions->shape[positions->ndim - 1];
        if (N > kMostRows) return fail(GDR_ESHAPE, "past: at most 2^30 sequences are supported");
        if (T > kMostRows) return fail(GDR_ESHAPE, "positions: at most 2^30 tokens are supported");
        if (page < 1 || page > 65536) return fail(GDR_ESHAPE, "page: 1 to 65536 tokens are supported, got %d", page);
        if (M > kMostRows / page) return fail(GDR_ESHAPE, "block_table: more than 2^30 tokens a sequence");
        if ((rc = want_shape(fresh, "new", {N}, "[N]")) || (rc = want_shape(block_table, "block_table", {N, M}, "[N, pages of a sequence]")) ||
            (rc = want_shape(cu_seqlens, "cu_seqlens", {N + 1}, "[N + 1]")) || (rc = want_shape(lens, "lens", {N}, "[N]")) ||
            (rc = positions->ndim == 1 ? GDR_OK : want_shape(positions, "positions", {1, T}, "[1, tokens]")) ||
            (rc = slots->ndim == 1 ? want_shape(slots, "slots", {T}, "[tokens] of positions")
                                   : want_shape(slots, "slots", {1, T}, "[1, tokens] of positions")) ||
            (rc = want_shape(used, "used", {2}, "[2]")))
            return rc;
        if ((rc = check_overlaps({{"past", args[0].span}, {"new", args[1].span}, {"free_pages", args[2].span}},
                                 {{"block_table", args[3].span}, {"cu_seqlens", args[4].span}, {"lens", args[5].span},
                                  {"positions", args[6].span}, {"slots", args[7].span}, {"used", args[8].span}})))
            return rc;
        if ((rc = check_device())) return rc;
        const auto ints = [](const gdr_tensor *t) { return static_cast<int32_t *>(t->data); };
        a.past = ints(past);
        a.fresh = ints(fresh);
        a.pool = ints(free_pages);
        a.table = ints(block_table);
        a.cu = ints(cu_seqlens);
        a.lens = ints(lens);
        a.positions = ints(positions);
        a.slots = ints(slots);
        a.used = ints(used);
        a.n_seq = N;
        a.pool_size = free_pages->shape[0];
        a.width = M;
        a.tokens = T;
        a.page = page;
        return launch([&] { return gdr::launch_page_plan(a, stream); }, "page plan kernel");
    });
}

}  // extern "C"
