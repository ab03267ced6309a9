// Host-side pieces of the entries that take rows of wider projections and a
// caller's workspace (gdr_mixer_api.cpp, gdr_attn_api.cpp): the checks of
// arguments, the workspace of a call and its launches.  Not installed; not
// part of the C ABI.
#pragma once

#include <cmath>
#include <cstdint>
#include <cstring>
#include <exception>
#include <initializer_list>
#include <string>

#include "gdr_host.h"

namespace gdr {
namespace host {

// No C++ exception leaves a C entry.
template <class F>
inline int entry(F f) noexcept {
    try {
        return f();
    } catch (const std::exception &e) {
        try {
            return fail(GDR_ENOMEM, "out of host resources: %s", e.what());
        } catch (...) {
            return GDR_ENOMEM;
        }
    }
}

// Like check_tensor for an input whose last dimensions are compact and whose
// rows (the first `lead` dimensions) are `ld` >= a row's elements apart: a
// slice of the columns of a wider projection.
inline int check_rows(const gdr_tensor *t, const char *name, int ndim, int lead, size_t align, int64_t *ld, Span *span) {
    if (!t) return fail(GDR_EINVAL, "%s: descriptor is NULL", name);
    gdr_tensor plain = *t;
    plain.strides = nullptr;
    int64_t n;
    int rc;
    if ((rc = check_tensor(&plain, name, ndim, &n, align))) return rc;
    int64_t inner = 1, rows = 1;
    for (int i = lead; i < ndim; ++i) inner *= t->shape[i];
    for (int i = 0; i < lead; ++i) rows *= t->shape[i];
    *ld = inner;
    *span = Span{};
    if (n == 0) return GDR_OK;
    if (t->strides) {
        int64_t expect = 1;
        for (int i = ndim - 1; i >= lead; --i) {
            if (t->shape[i] != 1 && t->strides[i] != expect)
                return fail(GDR_ESTRIDE, "%s: a row must be compact (dimension %d has stride %lld, expected %lld)", name, i,
                            (long long)t->strides[i], (long long)expect);
            expect *= t->shape[i];
        }
        bool seen = false;
        int64_t step = 0;   // stride that dimension i has to have
        for (int i = lead - 1; i >= 0; --i) {
            if (t->shape[i] == 1) continue;
            if (!seen) {
                if (t->strides[i] < inner || t->strides[i] > INT64_MAX / 64 / rows)
                    return fail(GDR_ESTRIDE, "%s: rows of %lld elements are %lld apart", name, (long long)inner,
                                (long long)t->strides[i]);
                *ld = t->strides[i];
                seen = true;
            } else if (t->strides[i] != step) {
                return fail(GDR_ESTRIDE, "%s: rows must be evenly spaced (dimension %d has stride %lld, expected %lld)",
                            name, i, (long long)t->strides[i], (long long)step);
            }
            step = *ld * (i == lead - 1 ? t->shape[i] : rows);
        }
    }
    const size_t e = dtype_size(t->dtype);
    if (rows > 1 && (static_cast<size_t>(*ld) * e) % align != 0)
        return fail(GDR_ESTRIDE, "%s: rows must start at multiples of %zu bytes (they are %lld elements apart)", name,
                    align, (long long)*ld);
    span->lo = reinterpret_cast<uintptr_t>(t->data);
    span->hi = span->lo + static_cast<uintptr_t>((rows - 1) * *ld + inner) * e;
    return GDR_OK;
}

struct Named {
    const char *name;
    Span span;
};
// No output may overlap an input or another output.
inline int check_overlaps(std::initializer_list<Named> ins, std::initializer_list<Named> outs) {
    for (const Named *o = outs.begin(); o != outs.end(); ++o) {
        for (const Named &i : ins)
            if (overlap(o->span, i.span)) return fail(GDR_EALIAS, "%s overlaps %s", o->name, i.name);
        for (const Named *p = outs.begin(); p != o; ++p)
            if (overlap(o->span, p->span)) return fail(GDR_EALIAS, "%s overlaps %s", o->name, p->name);
    }
    return GDR_OK;
}

inline bool is_float(const gdr_tensor *t) { return t->dtype == GDR_BF16 || t->dtype == GDR_F32; }

inline int want_dtype(const gdr_tensor *t, const char *name, int32_t dtype) {
    if (t && t->dtype != dtype) return fail(GDR_EDTYPE, "%s: dtype must be %s, got %s", name, dtype_name(dtype), dtype_name(t->dtype));
    return GDR_OK;
}
inline int want_shape(const gdr_tensor *t, const char *name, std::initializer_list<int64_t> s, const char *text) {
    if (t && !shape_is(t, s)) {
        std::string want;
        for (int64_t e : s) want += (want.empty() ? "" : ", ") + std::to_string(static_cast<long long>(e));
        return fail(GDR_ESHAPE, "%s: shape %s must be %s = [%s]", name, shape_str(t).c_str(), text, want.c_str());
    }
    return GDR_OK;
}
inline bool aligned16(const gdr_tensor *t) { return !t || reinterpret_cast<uintptr_t>(t->data) % 16 == 0; }

// Number of sequences of a call: cu_seqlens' (B must be 1), or B.
inline int sequences(const gdr_tensor *cu, int64_t B, int64_t T, int64_t *N) {
    if (B > 0 && T > 0x7FFFFFFFLL / B) return fail(GDR_ESHAPE, "B * T exceeds 2^31 - 1 tokens");
    if (!cu) {
        *N = B;
        return GDR_OK;
    }
    int rc;
    if ((rc = want_dtype(cu, "cu_seqlens", GDR_I32))) return rc;
    if (B != 1) return fail(GDR_ESHAPE, "cu_seqlens requires B == 1 (got B = %lld)", (long long)B);
    if (cu->shape[0] < 1) return fail(GDR_ESHAPE, "cu_seqlens must hold at least one offset");
    *N = cu->shape[0] - 1;
    return GDR_OK;
}
// Tokens that the kernels look at.  Without a sequence there are none, whatever
// T is: cu_seqlens has no second offset that a token could be looked up in.
inline int64_t live_tokens(int64_t N, int64_t B, int64_t T) { return N == 0 ? 0 : B * T; }

// A call's workspace: the caller's, or the library's (the ring, or the large
// buffer over 1 MiB).  `check` comes before the device is touched and returns 1
// when the call only asked for the size.
class Workspace {
  public:
    static int check(size_t need, const void *given, int64_t *given_bytes) {
        if (!given && given_bytes) {
            *given_bytes = static_cast<int64_t>(need);
            return 1;
        }
        if (!given) return GDR_OK;
        if (!given_bytes) return fail(GDR_EINVAL, "workspace: its size is missing");
        if (*given_bytes < static_cast<int64_t>(need))
            return fail(GDR_EINVAL, "workspace: %lld bytes given, %zu needed", (long long)*given_bytes, need);
        if (reinterpret_cast<uintptr_t>(given) % 16) return fail(GDR_EINVAL, "workspace: must be 16-byte aligned");
        return GDR_OK;
    }
    int get(size_t need, void *given, hipStream_t stream, void **out) {
        *out = given;
        if (given) return GDR_OK;
        if (need == 0) return GDR_OK;
        hipStreamCaptureStatus st = hipStreamCaptureStatusNone;
        if (hipStreamIsCapturing(stream, &st) == hipSuccess && st != hipStreamCaptureStatusNone)
            return fail(GDR_EINVAL, "workspace: the library's own buffers cannot be used in a stream capture; give one of %zu bytes",
                        need);
        return lease_.acquire(need, need > kRingSlot, stream, out);
    }
    int release() { return lease_.release(); }

  private:
    WsLease lease_;
};

// The opt-in check of the content of cu_seqlens, on a small workspace of its own.
inline int check_cu(const gdr_tensor *cu, int64_t N, int64_t total, hipStream_t stream) {
    if (!cu || !g_check_cu.load(std::memory_order_relaxed)) return GDR_OK;
    WsLease lease;
    void *ws = nullptr;
    int rc;
    if ((rc = lease.acquire(16, false, stream, &ws))) return rc;
    return check_cu_content(static_cast<const int32_t *>(cu->data), N, total, static_cast<int32_t *>(ws), stream);
}

template <class F>
inline int launch(F f, const char *what) {
    const hipError_t e = forced_failure() ? hipErrorLaunchFailure : f();
    return e == hipSuccess ? ok() : launch_error(e, what);
}

// Carves a workspace into 256-byte aligned parts: one pass with a NULL base
// sums the size, a second one hands out the addresses.
struct Carve {
    unsigned char *base;
    size_t used = 0;
    template <class T>
    T *take(int64_t count) {
        T *p = base ? reinterpret_cast<T *>(base + used) : nullptr;
        used += (static_cast<size_t>(count) * sizeof(T) + 255) & ~static_cast<size_t>(255);
        return p;
    }
};

}  // namespace host
}  // namespace gdr
