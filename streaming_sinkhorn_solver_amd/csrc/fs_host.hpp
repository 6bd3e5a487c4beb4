// fs_host.hpp -- host-side pieces shared by the entry points of attention,
// layers and losses: errors, the device check, views and their extents, the
// workspace.  Nothing here allocates, synchronises or throws.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "fs_attention.h"
#include "fs_attn_args.h"
#include "fs_internal.h"

namespace fs {

constexpr size_t kAlign = 256;
constexpr int kCus = 256;  // compute units of the MI355X
inline size_t up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline fs_status fail(fs_status s, const char* fmt, ...) {
    char buf[320];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return report(s, buf);
}

// The current device is a gfx950 (its properties are read once per device).
inline fs_status check_gpu() {
    constexpr int kMax = 64;
    static std::atomic<int> known[kMax];  // 0 unknown, 1 gfx950, 2 another
    int count = 0, dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) {
        (void)hipGetLastError();
        return fail(FS_ERR_DEVICE, "no HIP device available");
    }
    int k = dev < kMax ? known[dev].load(std::memory_order_relaxed) : 0;
    if (k == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceCount(&count) != hipSuccess || count < 1 ||
            hipGetDeviceProperties(&prop, dev) != hipSuccess) {
            (void)hipGetLastError();
            return fail(FS_ERR_DEVICE, "no HIP device available");
        }
        k = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
        if (dev < kMax) known[dev].store(k, std::memory_order_relaxed);
    }
    if (k != 1)
        return fail(FS_ERR_DEVICE, "device %d is not a gfx950, for which this library is built",
                    dev);
    return FS_OK;
}

inline int elem_size(int dtype) { return dtype == FS_DTYPE_F32 ? 4 : 2; }
inline int op_of(int dtype) {
    return dtype == FS_DTYPE_F32 ? OP_F32 : dtype == FS_DTYPE_BF16 ? OP_BF16 : OP_F16;
}

struct Extent {
    uintptr_t lo = 0, hi = 0;
    bool overlaps(const Extent& o) const { return lo < o.hi && o.lo < hi; }
};

// Checks a view of [b][r][h] rows of w elements and turns it into the
// kernels' form.  written: it may not overlap itself.
inline fs_status take_view(const char* name, const fs_rows& t, int64_t b, int64_t r, int64_t h, int64_t w,
                    int es, bool written, AttnView& v, Extent& e) {
    v = AttnView{(char*)t.data, t.stride_batch, t.stride_row, t.stride_head, 0};
    e = Extent{};
    if (b == 0 || r == 0 || h == 0) return FS_OK;
    if (!t.data) return fail(FS_ERR_INVALID_ARG, "%s must be non-NULL", name);
    if ((uintptr_t)t.data % es)
        return fail(FS_ERR_INVALID_ARG, "%s is not aligned to its element type", name);
    // the stride of an axis of one entry means nothing
    if (b == 1) v.sb = 0;
    if (r == 1) v.sr = 0;
    if (h == 1) v.sh = 0;
    constexpr int64_t kMaxStride = (int64_t)1 << 40;
    if (v.sb < 0 || v.sr < 0 || v.sh < 0 || v.sb > kMaxStride || v.sr > kMaxStride ||
        v.sh > kMaxStride)
        return fail(FS_ERR_INVALID_ARG, "%s has a stride outside 0..2^40", name);
    struct Axis {
        int64_t n, s;
    } ax[3] = {{b, v.sb}, {r, v.sr}, {h, v.sh}};
    std::sort(ax, ax + 3, [](const Axis& x, const Axis& y) { return x.s < y.s; });
    int64_t span = w;  // elements from the first to behind the last
    for (const Axis& x : ax) {
        if (x.n == 1) continue;
        if (written && x.s < span)
            return fail(FS_ERR_INVALID_ARG, "%s is written and its strides overlap", name);
        if (x.s > 0 && x.n > ((int64_t)1 << 46) / x.s)
            return fail(FS_ERR_INVALID_ARG, "%s spans too much memory", name);
        span += (x.n - 1) * x.s;
    }
    e.lo = (uintptr_t)t.data;
    e.hi = e.lo + (uintptr_t)span * es;
    const auto whole = [&](int64_t x) { return x * es % 16 == 0; };
    v.vec = (uintptr_t)t.data % 16 == 0 && whole(v.sb) && whole(v.sr) && whole(v.sh) && whole(w);
    return FS_OK;
}

inline Extent flat(const void* p, size_t bytes) {
    return p ? Extent{(uintptr_t)p, (uintptr_t)p + bytes} : Extent{};
}

inline fs_status check_workspace(const void* ws, size_t have, size_t need) {
    if (!ws || (uintptr_t)ws % kAlign)
        return fail(FS_ERR_WORKSPACE, "workspace must be non-NULL and %zu-byte aligned", kAlign);
    if (have < need)
        return fail(FS_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", have, need);
    return FS_OK;
}

inline fs_status hip_status(hipError_t e, const char* where) {
    if (e == hipSuccess) return FS_OK;
    return fail(FS_ERR_DEVICE, "%s: HIP error %d (%s)", where, (int)e, hipGetErrorString(e));
}

#define FS_TRY(x)                        \
    do {                                 \
        const fs_status st_ = (x);       \
        if (st_ != FS_OK) return st_;    \
    } while (0)

// An output against every input (and the workspace).
inline fs_status check_apart(const char* name, const Extent& out, const Extent* in, int n_in) {
    for (int i = 0; i < n_in; ++i)
        if (out.overlaps(in[i]))
            return fail(FS_ERR_INVALID_ARG, "%s overlaps an input or the workspace", name);
    return FS_OK;
}

}  // namespace fs
