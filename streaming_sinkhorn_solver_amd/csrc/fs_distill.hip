// fs_distill.hip -- distillation of a teacher's top logits into rows of a
// student's logits x over many classes:
//   p = softmax(x / T), tau = the teacher's weights of a row's few entries, W
//   their sum: loss = T^2 sum tau (log tau - log p[id]),
//   dx_c = dloss T (W p_c - sum_{id = c} tau).
// Bound by memory.  A workgroup reads its row (or its range of one) once and keeps
// it in registers over the row's maximum, sum and gradient; rows that are too long
// for that are read a second time, in part, for the gradient.  Where rows are few,
// several workgroups share one and meet in a second launch.  (Loss and gradient of
// 4096 x 131072, bf16: 463 us for 2.15 GB of logits read and gradient written, 4.6
// TB/s, half of each row read twice; 4096 x 65536: 210 us.  With nothing kept it took
// 668 us: the rows of eight workgroups a CU push one another out of the caches.  With
// all of a row kept it took 799: one workgroup a CU, whose reads, exponentials and
// writes take turns.)
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
    __device__ __forceinline__ float under(float top, float c) const {
        return m == -INFINITY ? s : s * ex2((m - top) * c);
    }
};

__host__ __device__ constexpr int padded(int k) { return (k + 3) / 4 * 4; }

template <int NT>
__device__ __forceinline__ float block_max(float x, float* buf) {
    x = lanes_max<64>(x);
    if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = x;
    stage_barrier();
    x = buf[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) x = fmaxf(x, buf[w]);
    return x;
}
template <int NT>
__device__ __forceinline__ float block_sum(float x, float* buf) {
    x = lanes_sum<64>(x);
    if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = x;
    stage_barrier();
    x = buf[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) x += buf[w];
    return x;
}

// From here on the compiler knows nothing of v any more: what is kept over a
// barrier are the logits as they were read, not their fp32 forms (twice the
// registers).
template <typename T>
__device__ __forceinline__ void forget(T (&v)[8]) {
    constexpr int N = 8 * sizeof(T) / 4;
    uint32_t w[N];
    __builtin_memcpy(w, v, sizeof(w));
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+v"(w[i]));
    __builtin_memcpy(v, w, sizeof(w));
}

// NT threads, of which each keeps the first CH groups of 8 of its range in
// registers; REST: there may be more, which are read once more for the gradient.
// (Rows of 1024 threads: 64 registers, so that two fit a CU and one's reads and
// writes run beside the other's exponentials.)
template <int OP, int NT, int CH, bool REST, bool WIDE, int MODE>
__global__ __launch_bounds__(NT, NT == 1024 ? 8 : 1) void distill_kernel(const DistillArgs a,
                                                                         int sections) {
    using T = typename El<OP>::T;
    constexpr int U = 2, kStep = 8 * NT;
    __shared__ float buf[2][NT / 64];
    extern __shared__ __align__(16) int ids[];  // ids and tau of whole groups of four
    float* const tau = (float*)(ids + padded(a.k));
    __shared__ float mass;  // of the teacher's weights
    const int64_t block = flat_block();
    const int64_t row = block / sections;
    const int sec = (int)(block - row * sections), tid = threadIdx.x;
    if (row >= a.rows) return;
    const int lo = sec * a.split_cols, hi = min(a.classes, lo + a.split_cols);
    const T* x = (const T*)a.x + row * a.sx;
    T* gx = (T*)a.gx + row * a.sgx;
    const float c = kLog2e / a.T, inv_t = 1.f / a.T;
    const bool on = !a.active || a.active[row];

    // this thread's eight of the 8 NT columns from lo + `col` on; -inf behind the end
    constexpr uint32_t ES = sizeof(T);
    const uint32_t size = (uint32_t)(hi - lo), off = WIDE ? tid * 8 : tid;
    const RowBuffer from(x + lo, size * ES), to(gx + lo, a.gx ? size * ES : 0);
    const auto load = [&](uint32_t col, T(&v)[8]) {
        if constexpr (WIDE) {
            const uint32_t at = col + off;
            u32x4 w[ES / 2];
#pragma unroll
            for (uint32_t i = 0; i < ES / 2; ++i) {
                w[i] = from.read16(at * ES + 16 * i);
                constexpr uint32_t none = OP == OP_F32    ? 0xff800000u
                                          : OP == OP_BF16 ? 0xff80ff80u
                                                          : 0xfc00fc00u;
#pragma unroll
                for (int e = 0; e < 4; ++e) w[i][e] = at < size ? w[i][e] : none;
            }
            __builtin_memcpy(v, w, sizeof(v));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t at = col + off + e * NT;
                const T t = from.read<T>(at * ES);
                v[e] = at < size ? t : (T)-INFINITY;
            }
        }
    };
    const auto store = [&](uint32_t col, const T(&v)[8]) {
        if constexpr (WIDE) {
            u32x4 w[ES / 2];
            __builtin_memcpy(w, v, sizeof(v));
#pragma unroll
            for (uint32_t i = 0; i < ES / 2; ++i) to.write16((col + off) * ES + 16 * i, w[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) to.write<T>((col + off + e * NT) * ES, v[e]);
        }
    };

    // the first reads of the range, under way while the teacher's entries are worked on
    T v[CH > 0 ? CH : 1][8];
    constexpr uint32_t rest = CH * kStep;
    if (CH > 0 && on && (MODE == WHOLE || MODE == PARTS || a.gx)) {
#pragma unroll
        for (int u = 0; u < CH; ++u) load(u * kStep, v[u]);
    }

    // The teacher's weights, by the first wave: id (-1: none) and tau of each entry, and
    // a lane's sum of tau log tau, all that the loss needs of its logarithms.  These are
    // formed from differences of logits as they stand: the digits that a quotient by T or
    // a log-sum-exp of it lacks would count |logit| / T times.
    float own = 0.f, weight = 0.f;
    if (MODE != PARTS && tid < 64) {
        float most = -INFINITY, ref;
        for (int k = tid; k < a.k; k += 64) {
            int id = -1;
            float t = -INFINITY;
            if (on) {
                id = a.ids[row * a.k + k];
                if (id >= 0 && id < a.classes) t = a.teacher[row * a.k + k];
                if (t == -INFINITY) id = -1;
            }
            ids[k] = id;
            tau[k] = t;
            most = fmaxf(most, t);
        }
        if (a.k + tid < padded(a.k)) ids[a.k + tid] = -1, tau[a.k + tid] = 0.f;
        if (a.teacher_lse) {
            ref = on ? a.teacher_lse[row] : 0.f;
        } else {
            most = lanes_max<64>(most);
            float s = 0.f;
            for (int k = tid; k < a.k; k += 64)
                if (ids[k] >= 0) s += ex2((tau[k] - most) * c);
            ref = logf(lanes_sum<64>(s));
        }
        for (int k = tid; k < a.k; k += 64) {
            const float t = tau[k];
            float lt = fmaf(t - most, inv_t, -ref);
            if (a.teacher_lse) {
                // the quotient in two parts; what is too small for one is -inf, too large NaN
                const float q = t * inv_t;
                lt = q == -INFINITY ? q : (q - ref) + fmaf(-q, a.T, t) * inv_t;
            }
            const float w = ids[k] >= 0 ? ex2(lt * kLog2e) : 0.f;
            tau[k] = w;
            weight += w;
            own += w == 0.f ? 0.f : w * lt;
        }
        weight = lanes_sum<64>(weight);
        if (tid == 0) mass = weight;
    }

    // the row's (or the range's) maximum and sum
    float2 ms = make_float2(-INFINITY, 0.f);
    if constexpr (MODE == WHOLE || MODE == PARTS) {
        Running r;
        if (on) {
#pragma unroll
            for (int u = 0; u < CH; ++u) {
                forget(v[u]);
                r.add(v[u], c);
                forget(v[u]);
            }
            if constexpr (REST)
                for (uint32_t at = rest; at < size; at += U * kStep) {
                    T w[U][8];
#pragma unroll
                    for (int u = 0; u < U; ++u) load(at + u * kStep, w[u]);
#pragma unroll
                    for (int u = 0; u < U; ++u) r.add(w[u], c);
                }
        }
        ms.x = block_max<NT>(r.m, buf[0]);
        ms.y = block_sum<NT>(r.under(ms.x, c), buf[1]);
        if constexpr (MODE == PARTS) {
            if (tid == 0) a.part[row * a.split + sec] = ms;
            return;
        }
    }
    if constexpr (MODE == JOIN) {  // every wave for itself: at most 64 ranges
        Running r;
        const int lane = tid & 63;
        if (lane < a.split) {
            const float2 p = a.part[row * a.split + lane];
            r.m = p.x, r.s = p.y;
        }
        ms.x = lanes_max<64>(r.m);
        ms.y = lanes_sum<64>(r.under(ms.x, c));
    }
    const float log_sum = MODE == BACK ? 0.f : logf(ms.y);
    const float lse = MODE == BACK ? (on ? a.lse[row] : 0.f)
                                   : ms.y == 0.f ? -INFINITY : fmaf(ms.x, inv_t, log_sum);
    const float f1 = MODE == BACK && a.lse_rest ? a.lse_rest[row] * kLog2e : 0.f;
    if (MODE != BACK && sec == 0 && tid < 64) {
        float sum = 0.f;
        const bool some = lse != -INFINITY && weight != 0.f;
        if (some) {
            sum = own;
            for (int k = tid; k < a.k; k += 64) {
                const int id = ids[k];
                const float w = tau[k];
                if (id < 0 || w == 0.f) continue;
                sum = fmaf(-w, fmaf((float)x[id] - ms.x, inv_t, -log_sum), sum);
            }
            sum = lanes_sum<64>(sum);
        }
        if (tid == 0) {
            a.loss[row] = some ? a.T * a.T * sum : 0.f;
            a.lse[row] = on ? lse : 0.f;
            if (a.lse_rest)
                a.lse_rest[row] = on && fabsf(lse) < INFINITY ? fmaf(ms.x, inv_t, -lse) + log_sum : 0.f;
        }
    }
    if (!a.gx) return;

    stage_barrier();
    weight = mass;
    const float g = a.gloss[row];
    if (!on || lse == -INFINITY || weight == 0.f || g == 0.f) {
        const T zero[8] = {};
        for (uint32_t at = 0; at < size; at += kStep) store(at, zero);
        return;
    }
    // p_c = p1 2^((f x_c - f0) f2 - f1)
    const float f = MODE == BACK ? inv_t : 1.f, f0 = MODE == BACK ? lse : ms.x;
    const float f2 = MODE == BACK ? kLog2e : c, p1 = MODE == BACK ? 1.f : 1.f / ms.y;
    const float gt = g * a.T, gp = gt * weight * p1;
    const auto grad = [&](float xc) {
        const float z = fmaf(xc, f, -f0);
        return gp * ex2(MODE == BACK ? fmaf(z, f2, -f1) : z * f2);
    };
#pragma unroll
    for (int u = 0; u < CH; ++u) {
        forget(v[u]);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[u][e] = (T)grad((float)v[u][e]);
        store(u * kStep, v[u]);
    }
    if constexpr (REST)
        for (uint32_t at = rest; at < size; at += U * kStep) {
            T w[U][8];
#pragma unroll
            for (int u = 0; u < U; ++u) load(at + u * kStep, w[u]);
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int e = 0; e < 8; ++e) w[u][e] = (T)grad((float)w[u][e]);
                store(at + u * kStep, w[u]);
            }
        }
    // the classes that the teacher names, over what was written: once the stores
    // in front of the barrier are through
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    for (int k = tid; k < a.k; k += NT) {
        const int id = ids[k];
        if (id < lo || id >= hi) continue;
        const float xc = (float)x[id];
        float t = 0.f;
        bool again = false;  // an earlier entry of this class does it
        for (int o = 0; o < a.k; o += 4) {
            typedef __attribute__((ext_vector_type(4))) int i32x4;
            const i32x4 other = *(const i32x4*)(ids + o);
            const f32x4 w = *(const f32x4*)(tau + o);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (other[e] == id) {
                    again |= o + e < k;
                    t += w[e];
                }
        }
        if (!again) gx[id] = (T)(grad(xc) - gt * t);
    }
}

template <int OP, int NT, int CH, bool REST, bool WIDE, int MODE>
hipError_t go(const DistillArgs& a, int sections, hipStream_t s) {
    distill_kernel<OP, NT, CH, REST, WIDE, MODE>
        <<<flat_grid((int64_t)a.rows * sections), NT, 8 * padded(a.k), s>>>(a, sections);
    return hipGetLastError();
}

// The smallest shape that keeps `cols` columns in registers, or part of them.
template <int OP, bool WIDE, int MODE>
hipError_t held(const DistillArgs& a, int cols, int sections, hipStream_t s) {
    if constexpr (MODE == BACK) return go<OP, 256, 0, true, WIDE, MODE>(a, sections, s);
    if (cols <= 512) return go<OP, 64, 1, false, WIDE, MODE>(a, sections, s);
    if (cols <= 2048) return go<OP, 64, 4, false, WIDE, MODE>(a, sections, s);
    if (cols <= 4096) return go<OP, 128, 4, false, WIDE, MODE>(a, sections, s);
    if (cols <= 8192) return go<OP, 256, 4, false, WIDE, MODE>(a, sections, s);
    if constexpr (MODE == WHOLE) {
        // Many rows go better with smaller workgroups, which read a rest again: without a
        // gradient, and with one where the rest is small; in fp32 while all of the logits
        // are small, too (us, 256 threads and a rest / 512; rows x classes):
        //                         bf16                           fp32
        //                 loss alone   and gradient    loss alone    and gradient
        //    512 x 8200   6.1 / 6.1     9.8 / 9.7      7.8 / 7.4     13.4 / 12.2
        //   1024 x 10007  9.2 / 10.5   15.1 / 17.0    10.9 / 12.6    21.0 / 23.7
        //   1024 x 10000  8.7 / 8.6    13.8 / 14.2    10.7 / 10.6    22.0 / 21.1
        //   1500 x 10007 11.6 / 13.0   18.8 / 21.8    13.8 / 15.6    30.7 / 31.7
        //   2048 x 8200  12.0 / 14.2   20.0 / 23.3    15.6 / 17.7    31.5 / 34.2
        //   2048 x 10000 12.2 / 15.2   24.2 / 27.1    17.7 / 19.9    43.8 / 40.6
        //   4096 x 8200  19.8 / 24.3   38.7 / 43.5    27.4 / 31.6    63.0 / 58.2
        //   4096 x 10000 22.0 / 27.1   43.0 / 46.3    31.4 / 34.3    80.6 / 69.1
        //   4096 x 16384 28.0 / 32.6   65.5 / 56.9    48.2 / 48.4   127.1 / 113.5
        const bool small =
            cols <= 10240 && (OP != OP_F32 || (int64_t)a.rows * cols * 4 <= 70 << 20);
        if (cols <= 16384 && a.rows >= 1024 && (small || !a.gx))
            return go<OP, 256, 4, true, WIDE, MODE>(a, sections, s);
        if (cols <= 16384) return go<OP, 512, 4, false, WIDE, MODE>(a, sections, s);
        if (cols <= 32768) return go<OP, 1024, 4, false, WIDE, MODE>(a, sections, s);
        // (single elements of 16 bits come in registers of their own first)
        if constexpr (OP == OP_F32 || !WIDE)
            return go<OP, 1024, 4, true, WIDE, MODE>(a, sections, s);
        else if (cols <= 65536)
            return go<OP, 1024, 8, false, WIDE, MODE>(a, sections, s);
        else
            return go<OP, 1024, 8, true, WIDE, MODE>(a, sections, s);
    }
    return go<OP, 256, 4, true, WIDE, MODE>(a, sections, s);
}
template <int OP, bool WIDE>
hipError_t launch(const DistillArgs& a, hipStream_t s) {
    if (!a.loss) return held<OP, WIDE, BACK>(a, a.split_cols, a.split, s);
    if (a.split == 1) return held<OP, WIDE, WHOLE>(a, a.classes, 1, s);
    const hipError_t e = held<OP, WIDE, PARTS>(a, a.split_cols, a.split, s);
    if (e != hipSuccess) return e;
    return held<OP, WIDE, JOIN>(a, a.split_cols, a.gx ? a.split : 1, s);
}
template <int OP>
hipError_t launch(const DistillArgs& a, hipStream_t s) {
    return a.wide ? launch<OP, true>(a, s) : launch<OP, false>(a, s);
}

}  // namespace

// The loss: one workgroup a row, but where rows are long and few, whose ranges' parts
// a second launch joins (us, bf16, loss and gradient, one workgroup a row / ranges):
//   rows              1           32          64          128         256
//   32000 classes     7.6 / 8.2   8.2 / 9.1   8.5 / 10.2  9.1 / 12.7  10.7 / 14.2
//   65536 classes    10.8 / 8.0  11.7 / 9.2  12.3 / 11.1 14.2 / 14.5  17.6 / 21.2
//   131072 classes   18.2 / 8.0  19.7 / 10.9 20.9 / 14.5 23.0 / 21.0  32.9 / 37.8
// (fp32: 32000 classes 8.2 / 8.5, 9.0 / 9.6, 9.9 / 11.3; 131072 classes 23.0 / 8.1,
// 25.5 / 14.4, 28.3 / 21.2, 34.0 / 36.3, 59.3 / 65.7.)  The gradient alone needs
// nothing of the rest of its row: ranges for 1024 workgroups.
int distill_split(int rows, int classes, bool backward, int* split_cols) {
    int64_t s = 1;
    if (rows > 0 && (backward || (classes > 32768 && rows < 128)))
        s = std::min<int64_t>((1024 + rows - 1) / rows, classes / 4096);
    s = std::max<int64_t>(1, std::min<int64_t>(s, kDistillMaxSplit));
    *split_cols = (int)(((classes + s - 1) / s + 7) / 8 * 8);
    return (classes + *split_cols - 1) / *split_cols;
}

hipError_t launch_distill(const DistillArgs& a, hipStream_t s) {
    return a.op == OP_BF16 ? launch<OP_BF16>(a, s)
           : a.op == OP_F16 ? launch<OP_F16>(a, s)
                            : launch<OP_F32>(a, s);
}

}  // namespace fs
