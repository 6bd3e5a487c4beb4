// fs_distill.hip -- distillation of a teacher's top logits into rows of a
// student's logits x over many classes:
//   p = softmax(x / T), tau = the teacher's weights of a row's few entries, W
//   their sum: loss = T^2 sum tau (log tau - log p[id]),
//   dx_c = dloss T (W p_c - sum_{id = c} tau).
// Bound by memory: a row's log-sum-exp is formed in one pass with a running
// maximum, the gradient in a second one over the row that comes from the caches
// (a workgroup's row was read a moment ago).  Where rows are few, several
// workgroups share one and meet in a second launch.
#include "fs_layers_args.h"
#include "fs_rowops.hpp"

#include <algorithm>

namespace fs {

namespace {

// What a launch does: a row at once (loss, and the gradient where wanted); the
// ranges' maxima and sums; loss and gradient from those; the gradient from lse.
enum { WHOLE, PARTS, JOIN, BACK };

// A running sum of 2^((x - m) c) under the largest x so far.
struct Running {
    float m = -INFINITY, s = 0.f;
    template <typename T>
    __device__ __forceinline__ void add(const T (&v)[8], float c) {
        float x[8], top = m;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = (float)v[e];
            top = fmaxf(top, x[e]);
        }
        if (top > m) {
            s *= ex2((m - top) * c);
            m = top;
        }
        if (m == -INFINITY) {  // nothing but -inf so far, or a NaN, which stays
#pragma unroll
            for (int e = 0; e < 8; ++e) s = x[e] == x[e] ? s : x[e];
            return;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) s += ex2((x[e] - m) * c);
    }
};

template <int NT>
__device__ __forceinline__ float block_fold(float x, bool sum, float* buf) {
    x = sum ? lanes_sum<64>(x) : lanes_max<64>(x);
    if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = x;
    __syncthreads();
    x = buf[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) x = sum ? x + buf[w] : fmaxf(x, buf[w]);
    __syncthreads();
    return x;
}

// The sum over threads, ranges, of (m, s) under their common maximum.
template <int NT>
__device__ __forceinline__ float2 block_running(Running r, float c, float* buf) {
    const float top = block_fold<NT>(r.m, false, buf);
    const float s = r.m == -INFINITY ? r.s : r.s * ex2((r.m - top) * c);
    return make_float2(top, block_fold<NT>(s, true, buf));
}

template <int OP, int NT, bool WIDE, int MODE>
__global__ __launch_bounds__(NT) void distill_kernel(const DistillArgs a, int sections) {
    using T = typename El<OP>::T;
    constexpr int U = 4, kStep = 8 * NT;
    __shared__ float buf[NT / 64];
    __shared__ int ids[kDistillMaxTop];
    __shared__ float tau[kDistillMaxTop];
    const int64_t block = flat_block();
    const int64_t row = block / sections;
    const int sec = (int)(block - row * sections), tid = threadIdx.x;
    if (row >= a.rows) return;
    const int lo = sec * a.split_cols, hi = min(a.classes, lo + a.split_cols);
    const T* x = (const T*)a.x + row * a.sx;
    T* gx = (T*)a.gx + row * a.sgx;
    const float c = kLog2e / a.T, inv_t = 1.f / a.T;
    const bool on = !a.active || a.active[row];

    const auto load = [&](int at, T(&v)[8]) {
        if constexpr (WIDE) {
            if (at < hi)
                __builtin_memcpy(v, __builtin_assume_aligned(x + at, 16), sizeof(v));
            else
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = (T)-INFINITY;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = at + e * NT < hi ? x[at + e * NT] : (T)-INFINITY;
        }
    };
    const auto store = [&](int at, const T(&v)[8]) {
        if constexpr (WIDE) {
            if (at < hi) __builtin_memcpy(__builtin_assume_aligned(gx + at, 16), v, sizeof(v));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (at + e * NT < hi) gx[at + e * NT] = v[e];
        }
    };
    const int first = lo + (WIDE ? tid * 8 : tid);

    // the row's (or the range's) maximum and sum
    float2 ms = make_float2(-INFINITY, 0.f);
    if constexpr (MODE == WHOLE || MODE == PARTS) {
        if (on) {
            Running r;
            for (int at = first; at < hi; at += U * kStep) {
                T v[U][8];
#pragma unroll
                for (int u = 0; u < U; ++u) load(at + u * kStep, v[u]);
#pragma unroll
                for (int u = 0; u < U; ++u) r.add(v[u], c);
            }
            ms = block_running<NT>(r, c, buf);
        }
        if constexpr (MODE == PARTS) {
            if (tid == 0) a.part[row * a.split + sec] = ms;
            return;
        }
    }
    if constexpr (MODE == JOIN) {
        Running r;
        if (on && tid < a.split) {
            const float2 p = a.part[row * a.split + tid];
            r.m = p.x, r.s = p.y;
        }
        ms = block_running<NT>(r, c, buf);
    }
    const float lse = MODE == BACK ? (on ? a.lse[row] : 0.f)
                                   : ms.y == 0.f ? -INFINITY : fmaf(ms.x, inv_t, logf(ms.y));
    const float g = a.gx ? a.gloss[row] : 0.f;
    bool some = on && lse != -INFINITY && (MODE != BACK || g != 0.f);

    // the teacher's weights: (log tau, then tau) of each entry, NaN ones too
    float weight = 0.f;
    if (some) {
        float top = -INFINITY;
        for (int k = tid; k < a.k; k += NT) {
            int id = a.ids[row * a.k + k];
            float t = -INFINITY;
            if (id >= 0 && id < a.classes) t = a.teacher[row * a.k + k] * inv_t;
            if (t == -INFINITY) id = -1;
            ids[k] = id;
            tau[k] = t;
            top = fmaxf(top, t);
        }
        float ref;  // log of the weights' divisor
        if (a.teacher_lse) {
            ref = a.teacher_lse[row];
        } else {
            top = block_fold<NT>(top, false, buf);
            float s = 0.f;
            for (int k = tid; k < a.k; k += NT)
                if (ids[k] >= 0) s += ex2((tau[k] - top) * kLog2e);
            s = block_fold<NT>(s, true, buf);
            ref = top + logf(s);
        }
        float sum = 0.f, all = 0.f;
        for (int k = tid; k < a.k; k += NT) {
            if (ids[k] < 0) continue;
            const float lt = tau[k] - ref, w = ex2(lt * kLog2e);
            tau[k] = w;
            all += w;
            if (MODE != BACK && sec == 0 && w != 0.f)
                sum = fmaf(w, lt - fmaf((float)x[ids[k]], inv_t, -lse), sum);
        }
        weight = block_fold<NT>(all, true, buf);
        some = weight != 0.f;
        if (MODE != BACK && sec == 0) {
            sum = block_fold<NT>(sum, true, buf);
            if (tid == 0) a.loss[row] = some ? a.T * a.T * sum : 0.f;
        }
    } else if (MODE != BACK && sec == 0 && tid == 0) {
        a.loss[row] = 0.f;
    }
    if (MODE != BACK && sec == 0 && tid == 0) a.lse[row] = on ? lse : 0.f;
    if (!a.gx) return;

    if (!some || g == 0.f) {
        const T zero[8] = {};
        for (int at = first; at < hi; at += kStep) store(at, zero);
        return;
    }
    // p_c = p1 2^((f x_c - f0) f2)
    const float f = MODE == BACK ? inv_t : 1.f, f0 = MODE == BACK ? lse : ms.x;
    const float f2 = MODE == BACK ? kLog2e : c, p1 = MODE == BACK ? 1.f : 1.f / ms.y;
    const float gt = g * a.T, gp = gt * weight * p1;
    for (int at = first; at < hi; at += U * kStep) {
        T v[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) load(at + u * kStep, v[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[u][e] = (T)(gp * ex2(fmaf((float)v[u][e], f, -f0) * f2));
            store(at + u * kStep, v[u]);
        }
    }
    // the classes that the teacher names, over what was written: once the stores
    // in front of the barrier are through
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    for (int k = tid; k < a.k; k += NT) {
        const int id = ids[k];
        if (id < lo || id >= hi) continue;
        float t = 0.f;
        bool again = false;  // an earlier entry of this class does it
        for (int o = 0; o < a.k; ++o)
            if (ids[o] == id) {
                again |= o < k;
                t += tau[o];
            }
        if (again) continue;
        gx[id] = (T)fmaf(gp, ex2(fmaf((float)x[id], f, -f0) * f2), -gt * t);
    }
}

template <int OP, int NT, bool WIDE, int MODE>
hipError_t go(const DistillArgs& a, int sections, hipStream_t s) {
    distill_kernel<OP, NT, WIDE, MODE>
        <<<flat_grid((int64_t)a.rows * sections), NT, 0, s>>>(a, sections);
    return hipGetLastError();
}
template <int OP, int NT, bool WIDE>
hipError_t launch(const DistillArgs& a, hipStream_t s) {
    if (!a.loss) return go<OP, NT, WIDE, BACK>(a, a.split, s);
    if (a.split == 1) return go<OP, NT, WIDE, WHOLE>(a, 1, s);
    const hipError_t e = go<OP, NT, WIDE, PARTS>(a, a.split, s);
    if (e != hipSuccess) return e;
    return go<OP, NT, WIDE, JOIN>(a, a.gx ? a.split : 1, s);
}
template <int OP>
hipError_t launch(const DistillArgs& a, hipStream_t s) {
    return a.wide ? launch<OP, 256, true>(a, s) : launch<OP, 256, false>(a, s);
}

}  // namespace

int distill_split(int rows, int classes, int* split_cols) {
    int64_t s = rows > 0 ? (1024 + rows - 1) / rows : 1;
    s = std::max<int64_t>(1, std::min<int64_t>({s, (int64_t)kDistillMaxSplit, classes / 4096}));
    *split_cols = (int)(((classes + s - 1) / s + 7) / 8 * 8);
    return (classes + *split_cols - 1) / *split_cols;
}

hipError_t launch_distill(const DistillArgs& a, hipStream_t s) {
    return a.op == OP_BF16 ? launch<OP_BF16>(a, s)
           : a.op == OP_F16 ? launch<OP_F16>(a, s)
                            : launch<OP_F32>(a, s);
}

}  // namespace fs
