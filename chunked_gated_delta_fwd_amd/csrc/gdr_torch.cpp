// Python calls of the operators in mixer.py and attention.py: torch tensors in, the C ABI of
// include/gdr.h called on torch's current stream, torch tensors out.  These
// operators run once per layer and token while decoding, in a few
// microseconds, so the marshalling is compiled.  No arithmetic here.
#include <torch/extension.h>

// torch's ROCm devices and streams carry the device type "cuda": these headers name them so
#include <ATen/hip/impl/HIPStreamMasqueradingAsCUDA.h>
#include <c10/core/DeviceGuard.h>
#include <hip/hip_runtime.h>

#include <cmath>
#include <optional>
#include <string>

#include "gdr.h"

namespace {

typedef std::optional<at::Tensor> Opt;

py::object &error_class() {
    static py::object *cls = new py::object();   // never destroyed: the interpreter may be gone by then
    return *cls;
}
[[noreturn]] void raise(int status, const std::string &text) {
    py::object e = error_class()(status, text);
    PyErr_SetObject(error_class().ptr(), e.ptr());
    throw py::error_already_set();
}
void check(int status) {
    if (status != 0) raise(status, gdr_last_error());
}

// The device of a call, from its first tensor; all others have to be there.
struct Call {
    c10::Device device;
    c10::DeviceGuard guard;
    explicit Call(const at::Tensor &x) : device(on_gpu(x)), guard(device) {}
    static c10::Device on_gpu(const at::Tensor &x) {
        if (!x.is_cuda()) raise(GDR_EDEVICE, "every tensor has to be on one GPU (one is on " + x.device().str() + ")");
        return x.device();
    }
    hipStream_t stream() const { return c10::hip::getCurrentHIPStreamMasqueradingAsCUDA(device.index()).stream(); }
};

// A descriptor that points at the tensor's own shape and strides.
struct Desc {
    gdr_tensor t;
    bool there = true;
    Desc(const at::Tensor &x, const Call &c) {
        switch (x.scalar_type()) {
        case at::kFloat: t.dtype = GDR_F32; break;
        case at::kBFloat16: t.dtype = GDR_BF16; break;
        case at::kInt: t.dtype = GDR_I32; break;
        default: raise(GDR_EDTYPE, std::string("unsupported dtype ") + c10::toString(x.scalar_type()));
        }
        if (x.device() != c.device) raise(GDR_EDEVICE, "every tensor has to be on one GPU (one is on " + x.device().str() + ")");
        t.data = x.data_ptr();
        t.ndim = static_cast<int32_t>(x.dim());
        t.shape = x.sizes().data();
        t.strides = x.strides().data();
    }
    Desc(const Opt &x, const Call &c) : Desc(x && x->defined() ? Desc(*x, c) : Desc()) {}
    const gdr_tensor *p() const { return there ? &t : nullptr; }

  private:
    Desc() : t{}, there(false) {}
};

at::Tensor empty(at::IntArrayRef shape, const at::Tensor &like, at::ScalarType type) {
    return at::empty(shape, like.options().dtype(type));
}
at::Tensor given_or(const Opt &given, at::IntArrayRef shape, const at::Tensor &like, at::ScalarType type) {
    return given ? *given : empty(shape, like, type);
}
void want_dims(const at::Tensor &t, int64_t n, const char *name) {
    if (t.dim() != n)
        raise(GDR_ESHAPE, std::string(name) + ": expected " + std::to_string(n) + " dimensions, got " + std::to_string(t.dim()));
}
// for the shape of a state that the call makes; a cu_seqlens without an offset is refused by the library
int64_t sequences(const at::Tensor &x, const Opt &cu) {
    if (!cu) return x.size(0);
    want_dims(*cu, 1, "cu_seqlens");
    return cu->size(0) > 0 ? cu->size(0) - 1 : 0;
}

at::Tensor conv_state(const at::Tensor &x, const at::Tensor &w, const Opt &cu) {
    return empty({sequences(x, cu), w.size(1) > 0 ? w.size(1) - 1 : 0, x.size(2)}, x, x.scalar_type());
}

// f(workspace, workspace_bytes) with the library's workspace, or in a stream
// capture with one from torch's allocator, which belongs to the graph then.
template <class F>
void with_workspace(const Call &c, F f) {
    hipStreamCaptureStatus st = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing(c.stream(), &st) != hipSuccess || st == hipStreamCaptureStatusNone) {
        check(f(nullptr, nullptr));
        return;
    }
    int64_t bytes = 0;
    check(f(nullptr, &bytes));
    bytes = bytes < 16 ? 16 : bytes;
    at::Tensor ws = at::empty({bytes}, at::TensorOptions().dtype(at::kByte).device(c.device));
    check(f(ws.data_ptr(), &bytes));
}

std::tuple<at::Tensor, Opt> short_conv_fwd(const at::Tensor &x, const at::Tensor &w, const Opt &bias, const Opt &cu,
                                           const Opt &s0, int act, bool want_st, const Opt &y_, const Opt &st_) {
    want_dims(x, 3, "x");
    want_dims(w, 2, "w");
    Call c(x);
    at::Tensor y = given_or(y_, x.sizes(), x, x.scalar_type());
    Opt st = st_;
    if (!st && want_st) st = conv_state(x, w, cu);
    check(gdr_short_conv_fwd(Desc(x, c).p(), Desc(w, c).p(), Desc(bias, c).p(), Desc(cu, c).p(), Desc(s0, c).p(),
                             Desc(y, c).p(), Desc(st, c).p(), act, c.stream()));
    return {y, st};
}

std::tuple<at::Tensor, at::Tensor, Opt, Opt> short_conv_bwd(const at::Tensor &x, const at::Tensor &w, const at::Tensor &dy,
                                                            const Opt &bias, const Opt &cu, const Opt &s0, const Opt &dst,
                                                            int act, const Opt &dx_, const Opt &dw_, const Opt &db_,
                                                            const Opt &ds0_, bool want_ds0) {
    want_dims(x, 3, "x");
    want_dims(w, 2, "w");
    Call c(x);
    at::Tensor dx = given_or(dx_, x.sizes(), x, x.scalar_type()), dw = given_or(dw_, w.sizes(), x, at::kFloat);
    Opt db = db_, ds0 = ds0_;
    if (!db && bias) db = empty(bias->sizes(), x, at::kFloat);
    if (!ds0 && want_ds0) ds0 = conv_state(x, w, cu);
    const Desc d[] = {Desc(x, c),  Desc(w, c),   Desc(bias, c), Desc(cu, c), Desc(s0, c), Desc(dy, c),
                      Desc(dst, c), Desc(dx, c), Desc(dw, c),   Desc(db, c), Desc(ds0, c)};
    with_workspace(c, [&](void *ws, int64_t *bytes) {
        return gdr_short_conv_bwd(d[0].p(), d[1].p(), d[2].p(), d[3].p(), d[4].p(), d[5].p(), d[6].p(), d[7].p(), d[8].p(),
                                  d[9].p(), d[10].p(), act, ws, bytes, c.stream());
    });
    return {dx, dw, db, ds0};
}

at::Tensor short_conv_step(const at::Tensor &x, const at::Tensor &state, const at::Tensor &w, const Opt &bias, int act,
                           const Opt &y_) {
    Call c(x);
    at::Tensor y = given_or(y_, x.sizes(), x, x.scalar_type());
    check(gdr_short_conv_step(Desc(x, c).p(), Desc(state, c).p(), Desc(w, c).p(), Desc(bias, c).p(), Desc(y, c).p(), act,
                              c.stream()));
    return y;
}

std::tuple<at::Tensor, at::Tensor> qk_norm_rope_fwd(const at::Tensor &q, const at::Tensor &k, const Opt &wq, const Opt &wk,
                                                    const Opt &cos, const Opt &sin, const Opt &pos, int norm, double eps,
                                                    bool interleaved, const Opt &oq_, const Opt &ok_) {
    Call c(q);
    at::Tensor oq = given_or(oq_, q.sizes(), q, q.scalar_type()), ok = given_or(ok_, k.sizes(), q, k.scalar_type());
    check(gdr_qk_norm_rope_fwd(Desc(q, c).p(), Desc(k, c).p(), Desc(wq, c).p(), Desc(wk, c).p(), Desc(cos, c).p(),
                               Desc(sin, c).p(), Desc(pos, c).p(), Desc(oq, c).p(), Desc(ok, c).p(), norm,
                               static_cast<float>(eps), interleaved, c.stream()));
    return {oq, ok};
}

std::tuple<at::Tensor, at::Tensor, Opt, Opt> qk_norm_rope_bwd(const at::Tensor &q, const at::Tensor &k, const at::Tensor &doq,
                                                              const at::Tensor &dok, const Opt &wq, const Opt &wk,
                                                              const Opt &cos, const Opt &sin, const Opt &pos, int norm,
                                                              double eps, bool interleaved, const Opt &dq_, const Opt &dk_,
                                                              const Opt &dwq_, const Opt &dwk_) {
    Call c(q);
    at::Tensor dq = given_or(dq_, q.sizes(), q, q.scalar_type()), dk = given_or(dk_, k.sizes(), q, k.scalar_type());
    Opt dwq = dwq_, dwk = dwk_;
    if (!dwq && wq) dwq = empty(wq->sizes(), q, at::kFloat);
    if (!dwk && wk) dwk = empty(wk->sizes(), q, at::kFloat);
    const Desc d[] = {Desc(q, c),   Desc(k, c),   Desc(wq, c), Desc(wk, c), Desc(cos, c), Desc(sin, c), Desc(pos, c),
                      Desc(doq, c), Desc(dok, c), Desc(dq, c), Desc(dk, c), Desc(dwq, c), Desc(dwk, c)};
    with_workspace(c, [&](void *ws, int64_t *bytes) {
        return gdr_qk_norm_rope_bwd(d[0].p(), d[1].p(), d[2].p(), d[3].p(), d[4].p(), d[5].p(), d[6].p(), d[7].p(), d[8].p(),
                                    d[9].p(), d[10].p(), d[11].p(), d[12].p(), norm, static_cast<float>(eps), interleaved,
                                    ws, bytes, c.stream());
    });
    return {dq, dk, dwq, dwk};
}

std::tuple<at::Tensor, Opt> ssm_scan_fwd(const at::Tensor &x, const at::Tensor &dt, const at::Tensor &A, const at::Tensor &b,
                                         const at::Tensor &cc, const Opt &D, const Opt &bias, const Opt &cu, const Opt &h0,
                                         bool want_ht, const Opt &y_, const Opt &ht_) {
    want_dims(x, 4, "x");
    want_dims(b, 4, "b");
    Call c(x);
    at::Tensor y = given_or(y_, x.sizes(), x, x.scalar_type());
    Opt ht = ht_;
    if (!ht && want_ht) ht = empty({sequences(x, cu), x.size(2), b.size(3), x.size(3)}, x, at::kFloat);
    const Desc d[] = {Desc(x, c), Desc(dt, c),   Desc(A, c),  Desc(b, c),  Desc(cc, c), Desc(D, c),
                      Desc(bias, c), Desc(cu, c), Desc(h0, c), Desc(y, c), Desc(ht, c)};
    with_workspace(c, [&](void *ws, int64_t *bytes) {
        return gdr_ssm_scan_fwd(d[0].p(), d[1].p(), d[2].p(), d[3].p(), d[4].p(), d[5].p(), d[6].p(), d[7].p(), d[8].p(),
                                d[9].p(), d[10].p(), ws, bytes, c.stream());
    });
    return {y, ht};
}

py::tuple ssm_scan_bwd(const at::Tensor &x, const at::Tensor &dt, const at::Tensor &A, const at::Tensor &b,
                       const at::Tensor &cc, const at::Tensor &dy, const Opt &D, const Opt &bias, const Opt &cu, const Opt &h0,
                       const Opt &dht, bool want_dh0, const Opt &dx_, const Opt &ddt_, const Opt &dA_, const Opt &db_,
                       const Opt &dc_, const Opt &dD_, const Opt &dbias_, const Opt &dh0_) {
    want_dims(x, 4, "x");
    want_dims(b, 4, "b");
    Call c(x);
    at::Tensor dx = given_or(dx_, x.sizes(), x, x.scalar_type()), ddt = given_or(ddt_, dt.sizes(), x, dt.scalar_type());
    at::Tensor dA = given_or(dA_, A.sizes(), x, at::kFloat), db = given_or(db_, b.sizes(), x, b.scalar_type());
    at::Tensor dc = given_or(dc_, cc.sizes(), x, cc.scalar_type());
    Opt dD = dD_, dbias = dbias_, dh0 = dh0_;
    if (!dD && D) dD = empty(D->sizes(), x, at::kFloat);
    if (!dbias && bias) dbias = empty(bias->sizes(), x, at::kFloat);
    if (!dh0 && want_dh0) dh0 = empty({sequences(x, cu), x.size(2), b.size(3), x.size(3)}, x, at::kFloat);
    const Desc d[] = {Desc(x, c),  Desc(dt, c),  Desc(A, c),  Desc(b, c),  Desc(cc, c), Desc(D, c),  Desc(bias, c),
                      Desc(cu, c), Desc(h0, c),  Desc(dy, c), Desc(dht, c), Desc(dx, c), Desc(ddt, c), Desc(dA, c),
                      Desc(db, c), Desc(dc, c),  Desc(dD, c), Desc(dbias, c), Desc(dh0, c)};
    with_workspace(c, [&](void *ws, int64_t *bytes) {
        return gdr_ssm_scan_bwd(d[0].p(), d[1].p(), d[2].p(), d[3].p(), d[4].p(), d[5].p(), d[6].p(), d[7].p(), d[8].p(),
                                d[9].p(), d[10].p(), d[11].p(), d[12].p(), d[13].p(), d[14].p(), d[15].p(), d[16].p(),
                                d[17].p(), d[18].p(), ws, bytes, c.stream());
    });
    return py::make_tuple(dx, ddt, dA, db, dc, dD, dbias, dh0);
}

at::Tensor ssm_step(const at::Tensor &x, const at::Tensor &dt, const at::Tensor &A, const at::Tensor &b, const at::Tensor &cc,
                    const at::Tensor &h, const Opt &D, const Opt &bias, const Opt &y_) {
    Call c(x);
    at::Tensor y = given_or(y_, x.sizes(), x, x.scalar_type());
    check(gdr_ssm_step(Desc(x, c).p(), Desc(dt, c).p(), Desc(A, c).p(), Desc(b, c).p(), Desc(cc, c).p(), Desc(D, c).p(),
                       Desc(bias, c).p(), Desc(h, c).p(), Desc(y, c).p(), c.stream()));
    return y;
}

// The calls below make tensors only to fill them: no gradient of theirs is recorded.
typedef at::AutoDispatchBelowADInplaceOrView Unrecorded;

float scale_or(const std::optional<double> &scale, const at::Tensor &q) {
    const int64_t d = q.size(-1);
    return scale ? static_cast<float>(*scale) : 1.f / std::sqrt(static_cast<float>(d > 0 ? d : 1));
}

std::tuple<at::Tensor, Opt> attn_fwd(const at::Tensor &q, const at::Tensor &k, const at::Tensor &v, const Opt &cu,
                                     const Opt &cuk, bool causal, int64_t window, const std::optional<double> &scale,
                                     bool want_lse, const Opt &o_, const Opt &lse_) {
    Unrecorded guard;
    want_dims(q, 4, "q");
    Call c(q);
    at::Tensor o = given_or(o_, q.sizes(), q, q.scalar_type());
    Opt lse = lse_;
    if (!lse && want_lse) lse = empty({q.size(0), q.size(1), q.size(2)}, q, at::kFloat);
    const Desc d[] = {Desc(q, c), Desc(k, c), Desc(v, c), Desc(cu, c), Desc(cuk, c), Desc(o, c), Desc(lse, c)};
    with_workspace(c, [&](void *ws, int64_t *bytes) {
        return gdr_attn_fwd(d[0].p(), d[1].p(), d[2].p(), d[3].p(), d[4].p(), d[5].p(), d[6].p(), causal, window,
                            scale_or(scale, q), ws, bytes, c.stream());
    });
    return {o, lse};
}

std::tuple<at::Tensor, at::Tensor, at::Tensor> attn_bwd(const at::Tensor &q, const at::Tensor &k, const at::Tensor &v,
                                                        const at::Tensor &o, const at::Tensor &lse, const at::Tensor &dout,
                                                        const Opt &cu, const Opt &cuk, bool causal, int64_t window,
                                                        const std::optional<double> &scale, const Opt &dq_, const Opt &dk_,
                                                        const Opt &dv_) {
    Unrecorded guard;
    want_dims(q, 4, "q");
    Call c(q);
    at::Tensor dq = given_or(dq_, q.sizes(), q, q.scalar_type()), dk = given_or(dk_, k.sizes(), q, k.scalar_type());
    at::Tensor dv = given_or(dv_, v.sizes(), q, v.scalar_type());
    const Desc d[] = {Desc(q, c), Desc(k, c),   Desc(v, c),    Desc(cu, c), Desc(cuk, c), Desc(o, c),
                      Desc(lse, c), Desc(dout, c), Desc(dq, c), Desc(dk, c), Desc(dv, c)};
    with_workspace(c, [&](void *ws, int64_t *bytes) {
        return gdr_attn_bwd(d[0].p(), d[1].p(), d[2].p(), d[3].p(), d[4].p(), d[5].p(), d[6].p(), d[7].p(), d[8].p(), d[9].p(),
                            d[10].p(), causal, window, scale_or(scale, q), ws, bytes, c.stream());
    });
    return {dq, dk, dv};
}

at::Tensor attn_paged_step(const at::Tensor &q, const at::Tensor &kp, const at::Tensor &vp, const at::Tensor &table,
                           const at::Tensor &lens, int64_t window, const std::optional<double> &scale, const Opt &o_) {
    Unrecorded guard;
    want_dims(q, 3, "q");
    Call c(q);
    at::Tensor o = given_or(o_, q.sizes(), q, q.scalar_type());
    const Desc d[] = {Desc(q, c), Desc(kp, c), Desc(vp, c), Desc(table, c), Desc(lens, c), Desc(o, c)};
    with_workspace(c, [&](void *ws, int64_t *bytes) {
        return gdr_attn_paged_step(d[0].p(), d[1].p(), d[2].p(), d[3].p(), d[4].p(), d[5].p(), window, scale_or(scale, q), ws,
                                   bytes, c.stream());
    });
    return o;
}

py::tuple page_plan(const at::Tensor &past, const at::Tensor &fresh, const at::Tensor &pool, const at::Tensor &table,
                    int64_t page, int64_t tokens, const Opt &cu_, const Opt &lens_, const Opt &positions_, const Opt &slots_,
                    const Opt &used_) {
    Unrecorded guard;
    want_dims(past, 1, "past");
    if (tokens < 0 || tokens > int64_t{1} << 30) raise(GDR_EINVAL, "tokens must be between 0 and 2^30, got " + std::to_string(tokens));
    if (page < 1 || page > 65536) raise(GDR_ESHAPE, "page: 1 to 65536 tokens are supported, got " + std::to_string(page));
    Call c(past);
    const int64_t n = past.size(0);
    // one allocation for what is not given, cut in pieces: a call takes 5.5 us, and 6.7 with five
    int64_t at = 0;
    const auto room = [&](const Opt &given, int64_t count) { return given ? 0 : (count + 3) / 4 * 4; };
    const int64_t all = room(cu_, n + 1) + room(lens_, n) + room(used_, 2) + room(positions_, tokens) + room(slots_, tokens);
    const at::Tensor whole = empty({all}, past, at::kInt);
    const auto cut = [&](const Opt &given, at::IntArrayRef shape, at::IntArrayRef strides, int64_t count) {
        if (given) return *given;
        const at::Tensor t = whole.as_strided(shape, strides, at);
        at += room(given, count);
        return t;
    };
    const at::Tensor cu = cut(cu_, {n + 1}, {1}, n + 1), lens = cut(lens_, {n}, {1}, n), used = cut(used_, {2}, {1}, 2);
    const at::Tensor positions = cut(positions_, {1, tokens}, {tokens, 1}, tokens);
    const at::Tensor slots = cut(slots_, {1, tokens}, {tokens, 1}, tokens);
    check(gdr_page_plan(Desc(past, c).p(), Desc(fresh, c).p(), Desc(pool, c).p(), Desc(table, c).p(), Desc(cu, c).p(),
                        Desc(lens, c).p(), Desc(positions, c).p(), Desc(slots, c).p(), Desc(used, c).p(),
                        static_cast<int32_t>(page), c.stream()));
    return py::make_tuple(cu, lens, positions, slots, used);
}

void page_store(const at::Tensor &k, const at::Tensor &v, const at::Tensor &slots, const at::Tensor &kp, const at::Tensor &vp) {
    Unrecorded guard;
    Call c(k);
    check(gdr_page_store(Desc(k, c).p(), Desc(v, c).p(), Desc(slots, c).p(), Desc(kp, c).p(), Desc(vp, c).p(), c.stream()));
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
    m.def("set_error", [](py::object cls) { error_class() = cls; });
    m.def("short_conv_fwd", &short_conv_fwd);
    m.def("short_conv_bwd", &short_conv_bwd);
    m.def("short_conv_step", &short_conv_step);
    m.def("qk_norm_rope_fwd", &qk_norm_rope_fwd);
    m.def("qk_norm_rope_bwd", &qk_norm_rope_bwd);
    m.def("ssm_scan_fwd", &ssm_scan_fwd);
    m.def("ssm_scan_bwd", &ssm_scan_bwd);
    m.def("ssm_step", &ssm_step);
    m.def("attn_fwd", &attn_fwd);
    m.def("attn_bwd", &attn_bwd);
    m.def("attn_paged_step", &attn_paged_step);
    m.def("page_plan", &page_plan);
    m.def("page_store", &page_store);
}
