// Host-side pieces shared by the library's C ABI sources (gdr_api.cpp,
// gdr_mixer_api.cpp, gdr_attn_api.cpp): error text, descriptor checks, the device check, the
// workspace ring and the debug options.  One copy of each for the library
// (inline variables).  Not installed; not part of the C ABI.
#pragma once

#include "gdr.h"

#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdlib>
#include <cstdio>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <string>

#include "gdr_internal.h"

namespace gdr {
namespace host {

inline thread_local std::string g_last_error;

inline int fail(int code, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return code;
}

inline int ok() {
    g_last_error.clear();
    return GDR_OK;
}

inline size_t dtype_size(int32_t dt) { return dt == GDR_F32 ? 4 : dt == GDR_BF16 ? 2 : dt == GDR_I32 ? 4 : 0; }

inline const char *dtype_name(int32_t dt) {
    return dt == GDR_F32 ? "f32" : dt == GDR_BF16 ? "bf16" : dt == GDR_I32 ? "i32" : "?";
}

struct Span {
    uintptr_t lo = 0, hi = 0;   // [lo, hi) bytes; empty when lo == hi
};

// Checks rank, non-negative extents, compact strides and the data pointer.
inline int check_tensor(const gdr_tensor *t, const char *name, int ndim, int64_t *numel, size_t align) {
    if (!t) return fail(GDR_EINVAL, "%s: descriptor is NULL", name);
    if (t->ndim != ndim) return fail(GDR_ESHAPE, "%s: expected %d dimensions, got %d", name, ndim, t->ndim);
    if (ndim > 0 && !t->shape) return fail(GDR_EINVAL, "%s: shape pointer is NULL", name);
    if (dtype_size(t->dtype) == 0) return fail(GDR_EDTYPE, "%s: unknown dtype %d", name, t->dtype);
    int64_t n = 1;
    for (int i = 0; i < ndim; ++i) {
        if (t->shape[i] < 0) return fail(GDR_ESHAPE, "%s: negative extent in dimension %d", name, i);
        if (t->shape[i] > 0 && n > (INT64_MAX / 16) / t->shape[i])
            return fail(GDR_ESHAPE, "%s: too many elements", name);
        n *= t->shape[i];
    }
    if (t->strides && n > 0) {   // no element is at any place in an empty one
        int64_t expect = 1;
        for (int i = ndim - 1; i >= 0; --i) {
            if (t->shape[i] != 1 && t->strides[i] != expect)
                return fail(GDR_ESTRIDE,
                            "%s: strides must be compact row-major (dimension %d has stride %lld, expected %lld)",
                            name, i, (long long)t->strides[i], (long long)expect);
            expect *= t->shape[i];
        }
    }
    if (n > 0 && !t->data) return fail(GDR_EINVAL, "%s: data pointer is NULL", name);
    if (n > 0 && (reinterpret_cast<uintptr_t>(t->data) % align) != 0)
        return fail(GDR_EINVAL, "%s: data pointer must be %zu-byte aligned", name, align);
    *numel = n;
    return GDR_OK;
}

inline Span span_of(const gdr_tensor *t, int64_t numel) {
    Span s;
    if (t && t->data && numel > 0) {
        s.lo = reinterpret_cast<uintptr_t>(t->data);
        s.hi = s.lo + static_cast<uintptr_t>(numel) * dtype_size(t->dtype);
    }
    return s;
}

inline bool overlap(const Span &a, const Span &b) {
    return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}

inline bool shape_is(const gdr_tensor *t, std::initializer_list<int64_t> s) {
    int i = 0;
    for (int64_t e : s)
        if (t->shape[i++] != e) return false;
    return true;
}

inline std::string shape_str(const gdr_tensor *t) {
    std::string s = "[";
    for (int i = 0; i < t->ndim; ++i) {
        if (i) s += ", ";
        s += std::to_string(static_cast<long long>(t->shape[i]));
    }
    return s + "]";
}

// gfx950 check for the current device, remembered per device ordinal.
inline int check_device() {
    static int state[64];   // 0 unknown, 1 gfx950, -1 other
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return fail(GDR_EDEVICE, "hipGetDevice failed");
    if (dev >= 0 && dev < 64 && state[dev] == 1) return GDR_OK;
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess)
        return fail(GDR_EDEVICE, "hipGetDeviceProperties failed for device %d", dev);
    const bool good = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    if (dev >= 0 && dev < 64) state[dev] = good ? 1 : -1;
    if (!good) return fail(GDR_EDEVICE, "device %d is %s; this library is built for gfx950", dev, prop.gcnArchName);
    return GDR_OK;
}

// Library-owned device workspaces, reused across calls.  On this runtime
// freeing a stream-ordered allocation (hipFreeAsync) blocks the calling
// thread until the stream has caught up, which serialised the host with the
// GPU at every call.  Instead each device keeps a ring of buffers that are
// never freed while in use: a call takes the next slot of the ring (or the
// one large slot, for the backward's multi-GB workspace), makes its stream
// wait on the GPU for the slot's previous user (an event recorded after that
// user's last kernel, so reuse is ordered across streams without a host
// wait), and records the event again after its own kernels.  Slots are
// indexed by a counter, never by stream or tensor identity.
//
// The whole ring is created by the first call on a device: one allocation
// holding all slots (at least kRingSlot bytes each) and all events, so later
// calls allocate nothing.  A request larger than a slot regrows the whole ring
// once (every slot's previous user is waited for first).  Everything is kept
// until gdr_free_workspaces or the end of the process.
inline int launch_error(hipError_t e, const char *what) {
    return fail(GDR_ELAUNCH, "%s: %s", what, hipGetErrorString(e));
}

inline constexpr int kRing = 8;
inline constexpr size_t kRingSlot = 1u << 20;
inline constexpr int kMaxDevices = 64;
struct WsSlot {
    std::mutex mu;
    hipEvent_t ev = nullptr;
    bool used = false;
};
struct WsDevice {
    // mu guards next, block and cap; a regrow also holds every slot's lock,
    // so a thread holding one slot's lock reads block and cap unchanged.
    std::mutex mu;
    unsigned next = 0;
    unsigned char *block = nullptr;   // kRing slots of cap bytes
    size_t cap = 0;
    WsSlot ring[kRing];
    WsSlot big;
    void *big_ptr = nullptr;
    size_t big_cap = 0;
};
inline WsDevice g_ws[kMaxDevices];

inline size_t round_mib(size_t x) { return (x + 0xFFFFF) & ~static_cast<size_t>(0xFFFFF); }

// (Re)creates the ring of device D with slots of at least `bytes`; the caller
// holds D.mu and no slot lock.
inline int ring_grow(WsDevice &D, size_t bytes) {
    std::unique_lock<std::mutex> locks[kRing];
    for (int i = 0; i < kRing; ++i) locks[i] = std::unique_lock<std::mutex>(D.ring[i].mu);
    for (WsSlot &s : D.ring)
        if (s.used) {
            (void)hipEventSynchronize(s.ev);
            s.used = false;
        }
    if (D.block) (void)hipFree(D.block);
    D.block = nullptr;
    D.cap = 0;
    const size_t cap = round_mib(bytes > kRingSlot ? bytes : kRingSlot);
    void *p = nullptr;
    const hipError_t e = hipMalloc(&p, cap * kRing);
    if (e != hipSuccess) return fail(GDR_ENOMEM, "workspace ring of %zu bytes: %s", cap * kRing, hipGetErrorString(e));
    for (WsSlot &s : D.ring)
        if (!s.ev && hipEventCreateWithFlags(&s.ev, hipEventDisableTiming) != hipSuccess) {
            s.ev = nullptr;
            (void)hipFree(p);
            return fail(GDR_ENOMEM, "workspace event could not be created");
        }
    D.block = static_cast<unsigned char *>(p);
    D.cap = cap;
    return GDR_OK;
}

// Holds one slot from acquire() to release(); the slot's lock is kept in
// between so that its event is recorded before anyone else can take it.
class WsLease {
  public:
    int acquire(size_t bytes, bool big, hipStream_t stream, void **out) {
        int dev = 0;
        if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices)
            return fail(GDR_EDEVICE, "no current device");
        WsDevice &D = g_ws[dev];
        WsSlot *s;
        void *ptr;
        if (big) {
            s = &D.big;
            lock_ = std::unique_lock<std::mutex>(s->mu);
            if (!s->ev && hipEventCreateWithFlags(&s->ev, hipEventDisableTiming) != hipSuccess) {
                s->ev = nullptr;
                return fail(GDR_ENOMEM, "workspace event could not be created");
            }
            if (D.big_cap < bytes) {
                if (D.big_ptr) {
                    if (s->used) (void)hipEventSynchronize(s->ev);
                    (void)hipFree(D.big_ptr);
                    D.big_ptr = nullptr;
                    D.big_cap = 0;
                    s->used = false;
                }
                const size_t want = round_mib(bytes > 65536 ? bytes : 65536);
                const hipError_t e = hipMalloc(&D.big_ptr, want);
                if (e != hipSuccess) {
                    D.big_ptr = nullptr;
                    return fail(GDR_ENOMEM, "workspace of %zu bytes: %s", want, hipGetErrorString(e));
                }
                D.big_cap = want;
            }
            ptr = D.big_ptr;
        } else {
            unsigned idx;
            {
                std::lock_guard<std::mutex> g(D.mu);
                if (!D.block || D.cap < bytes) {
                    const int rc = ring_grow(D, bytes);
                    if (rc) return rc;
                }
                idx = D.next++ % kRing;
            }
            s = &D.ring[idx];
            lock_ = std::unique_lock<std::mutex>(s->mu);
            ptr = D.block + static_cast<size_t>(idx) * D.cap;
        }
        if (s->used && hipEventQuery(s->ev) != hipSuccess) {
            const hipError_t e = hipStreamWaitEvent(stream, s->ev, 0);
            if (e != hipSuccess) return launch_error(e, "workspace wait");
        }
        slot_ = s;
        stream_ = stream;
        *out = ptr;
        return GDR_OK;
    }
    // After the call's last kernel that touches the workspace (also on error
    // paths: whatever was enqueued is then ordered before the next user).
    int release() {
        if (!slot_) return GDR_OK;
        const hipError_t e = hipEventRecord(slot_->ev, stream_);
        if (e == hipSuccess) slot_->used = true;
        slot_ = nullptr;
        lock_.unlock();
        return e == hipSuccess ? GDR_OK : launch_error(e, "workspace release");
    }
    ~WsLease() { (void)release(); }

  private:
    WsSlot *slot_ = nullptr;
    hipStream_t stream_ = nullptr;
    std::unique_lock<std::mutex> lock_;
};

// Debug and test options (gdr_debug_set).  The cu_seqlens content check can
// also be switched on for the whole process with GDR_DEBUG_CHECK_CU=1.
inline std::atomic<int> g_check_cu{[] {
    const char *e = std::getenv("GDR_DEBUG_CHECK_CU");
    return (e && *e && std::strcmp(e, "0") != 0) ? 1 : 0;
}()};
inline std::atomic<int64_t> g_fail_launches{0};
inline std::atomic<int32_t> g_spin_max{gdr::kSpinDefault};

// True when the test hook says this launch is to fail (consumes one).
inline bool forced_failure() {
    int64_t n = g_fail_launches.load(std::memory_order_relaxed);
    while (n > 0)
        if (g_fail_launches.compare_exchange_weak(n, n - 1, std::memory_order_relaxed)) return true;
    return false;
}
// With the cu_seqlens check on: checks the content on the device, waits for
// the stream and reports the first violated precondition (GDR_EINVAL).
// `result` is 16 bytes of device workspace owned by the call.
inline int check_cu_content(const int32_t *cu, int64_t n_seq, int64_t total, int32_t *result, hipStream_t stream) {
    if (!g_check_cu.load(std::memory_order_relaxed)) return GDR_OK;
    hipError_t e = gdr::launch_check_cu(cu, n_seq, total, result, stream);
    if (e != hipSuccess) return launch_error(e, "cu_seqlens check kernel");
    int32_t r[4];
    if ((e = hipMemcpyAsync(r, result, sizeof(r), hipMemcpyDeviceToHost, stream)) != hipSuccess ||
        (e = hipStreamSynchronize(stream)) != hipSuccess)
        return launch_error(e, "cu_seqlens check");
    switch (r[0]) {
    case 0: return GDR_OK;
    case 1: return fail(GDR_EINVAL, "cu_seqlens: cu[0] must be 0, got %d", r[2]);
    case 2: return fail(GDR_EINVAL, "cu_seqlens: offsets must not decrease (cu[%d] = %d > cu[%d] = %d)", r[1], r[2],
                        r[1] + 1, r[3]);
    default: return fail(GDR_EINVAL, "cu_seqlens: cu[N] = cu[%d] = %d must equal the %d tokens", r[1], r[2], r[3]);
    }
}

}  // namespace host
}  // namespace gdr
