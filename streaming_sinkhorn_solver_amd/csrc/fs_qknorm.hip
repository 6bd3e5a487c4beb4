// fs_qknorm.hip -- the norm of every head's row of queries and keys and the
// rotation by its position, in one pass, and the pass's gradients:
//   r = 1 / sqrt(mean(x^2) + eps),  z = w x r,  y = R z  (R a rotation of pairs)
//   g = R^T dy,  dw = sum over rows of x r g,  dx = r (w g - x r^2 mean(x w g)).
// Bound by memory: a row of d elements is read once and written once, the
// angles' cosines and sines are shared by the heads of a token.  A lane holds
// four pairs (8 elements), d / 8 lanes (rounded up to a power of two) a row,
// so a row's sums are butterflies within those lanes.  (4 x 4096 tokens, 32 + 8
// heads of 128, bf16: forward 73 us for 335 MB, 4.6 TB/s; backward 102 us for
// 503 MB, 4.9 TB/s, and 5 us for the weights' sums.  Lanes of 16-byte loads,
// half as many a row, were slower, 122 and 172 us against 93 and 137 at the time.)
#include "fs_attn.hpp"

#include <type_traits>

namespace fs {

namespace {

// Element (0 or 1) of pair p.
__device__ __forceinline__ int pair_at(const NormArgs& a, int p, int which) {
    if (2 * p >= a.rot || a.interleaved) return 2 * p + which;
    return p + which * (a.rot / 2);
}

// Four elements at x0.
template <typename T>
__device__ __forceinline__ void load4(const T* row, int x0, float (&out)[4]) {
    T v[4];
    __builtin_memcpy(v, __builtin_assume_aligned(row + x0, sizeof(v)), sizeof(v));
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = (float)v[i];
}
template <typename T>
__device__ __forceinline__ void store4v(T* row, int x0, const float (&in)[4]) {
    T v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (T)in[i];
    __builtin_memcpy(__builtin_assume_aligned(row + x0, sizeof(v)), v, sizeof(v));
}

// A lane's pairs p0 .. p0 + 3 of a row: u = first, v = second elements.
// wide: whole groups of four pairs lie on one side of rot and rows are aligned.
template <typename T>
__device__ __forceinline__ void load_pairs(const NormArgs& a, const T* row, int p0, bool wide,
                                           float (&u)[4], float (&v)[4]) {
    if (wide) {
        if (2 * p0 >= a.rot || a.interleaved) {
            float lo[4], hi[4];
            load4(row, 2 * p0, lo);
            load4(row, 2 * p0 + 4, hi);
            u[0] = lo[0], v[0] = lo[1], u[1] = lo[2], v[1] = lo[3];
            u[2] = hi[0], v[2] = hi[1], u[3] = hi[2], v[3] = hi[3];
        } else {
            load4(row, p0, u);
            load4(row, p0 + a.rot / 2, v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = p0 + i < a.d / 2;
            u[i] = in ? (float)row[pair_at(a, p0 + i, 0)] : 0.f;
            v[i] = in ? (float)row[pair_at(a, p0 + i, 1)] : 0.f;
        }
    }
}
template <typename T>
__device__ __forceinline__ void store_pairs(const NormArgs& a, T* row, int p0, bool wide,
                                            const float (&u)[4], const float (&v)[4]) {
    if (wide) {
        if (2 * p0 >= a.rot || a.interleaved) {
            const float lo[4] = {u[0], v[0], u[1], v[1]}, hi[4] = {u[2], v[2], u[3], v[3]};
            store4v(row, 2 * p0, lo);
            store4v(row, 2 * p0 + 4, hi);
        } else {
            store4v(row, p0, u);
            store4v(row, p0 + a.rot / 2, v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (p0 + i < a.d / 2) {
                row[pair_at(a, p0 + i, 0)] = (T)u[i];
                row[pair_at(a, p0 + i, 1)] = (T)v[i];
            }
    }
}
// Cosines and sines of a token's pairs (1, 0 where nothing turns).
__device__ __forceinline__ void load_angles(const NormArgs& a, int b, int i, int p0, float (&c)[4],
                                            float (&s)[4]) {
    const int half = a.rot / 2;
#pragma unroll
    for (int x = 0; x < 4; ++x) c[x] = 1.f, s[x] = 0.f;
    if (p0 >= half) return;
    const int64_t given = a.positions ? a.positions[b * a.pos_stride + i] : (int64_t)a.offset + i;
    const int64_t pos = min(max(given, (int64_t)0), (int64_t)a.n_pos - 1);
    const float* ct = a.cos_t + pos * half + p0;
    const float* st = a.sin_t + pos * half + p0;
    if (a.table_vec) {
        load4(ct, 0, c);
        load4(st, 0, s);
        return;
    }
#pragma unroll
    for (int x = 0; x < 4; ++x)
        if (p0 + x < half) c[x] = ct[x], s[x] = st[x];
}

// A lane's two groups of four elements of U rows of whole, aligned groups.
// The loads ask nothing first (a lane without pairs reads the row's first ones,
// a head behind the last the last one's), so that all are in flight before the
// first is waited for; what was read in another's place counts as zero.
template <typename T, int U>
struct WideRows {
    T lo[U][4], hi[U][4];
    __device__ __forceinline__ void load(const NormArgs& a, const T* x, int64_t sh, int h0, int step,
                                         int heads, int p0) {
        const bool next = 2 * p0 >= a.rot || a.interleaved;  // the pairs' elements are neighbours
        const int at = p0 < a.d / 2 ? p0 : 0;
        const int xl = at == p0 && next ? 2 * at : at;
        const int xh = at != p0 ? 4 : next ? xl + 4 : at + a.rot / 2;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int head = h0 + k * step;
            const T* row = x + (head < heads ? head : heads - 1) * sh;
            __builtin_memcpy(lo[k], __builtin_assume_aligned(row + xl, sizeof(lo[k])), sizeof(lo[k]));
            __builtin_memcpy(hi[k], __builtin_assume_aligned(row + xh, sizeof(hi[k])), sizeof(hi[k]));
        }
    }
    __device__ __forceinline__ void pairs(const NormArgs& a, int k, bool in, int p0, float (&u)[4],
                                          float (&v)[4]) const {
        const bool next = 2 * p0 >= a.rot || a.interleaved;
        float l[4], h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            l[e] = in ? (float)lo[k][e] : 0.f;
            h[e] = in ? (float)hi[k][e] : 0.f;
        }
        u[0] = l[0], v[0] = next ? l[1] : h[0];
        u[1] = next ? l[2] : l[1], v[1] = next ? l[3] : h[1];
        u[2] = next ? h[0] : l[2], v[2] = next ? h[1] : h[2];
        u[3] = next ? h[2] : l[3], v[3] = h[3];
    }
};

// Weights of a lane's pairs.
__device__ __forceinline__ void load_weights(const NormArgs& a, const float* w, int p0,
                                             float (&u)[4], float (&v)[4]) {
    if (w && (uintptr_t)w % 16 == 0 && a.rot % 8 == 0 && a.d % 8 == 0 && p0 < a.d / 2) {
        load_pairs(a, w, p0, true, u, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool in = p0 + i < a.d / 2;
        u[i] = !in ? 0.f : w ? w[pair_at(a, p0 + i, 0)] : 1.f;
        v[i] = !in ? 0.f : w ? w[pair_at(a, p0 + i, 1)] : 1.f;
    }
}
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = LPR / 2; o >= 1; o >>= 1) x += __shfl_xor(x, o, 64);
    return x;
}

// A wave takes U rows a lane group, heads h0, h0 + 64 / LPR, ... of one token:
// the angles, the weights and the token's place are formed once, and U rows'
// loads are in flight together.
template <int LPR, int U>
struct NormItem {
    static constexpr int kGroups = 64 / LPR, kHeads = kGroups * U;
    int b, i, h0;
    bool any;
    __device__ __forceinline__ NormItem(const NormArgs& a, int heads, uint32_t item) {
        const uint32_t per = (uint32_t)(heads + kHeads - 1) / kHeads;  // items of a token
        const uint32_t tok = item / per;
        any = tok < (uint32_t)a.B * a.n;
        b = (int)(tok / a.n), i = (int)(tok - b * (uint32_t)a.n);
        h0 = (int)(item - tok * per) * kHeads + (threadIdx.x & 63) / LPR;
    }
};

template <int OP, int LPR, int U>
__global__ __launch_bounds__(256) void norm_rotate_kernel(const NormArgs a) {
    using T = typename El<OP>::T;
    using Item = NormItem<LPR, U>;
    const NormRows& R = a.r[blockIdx.y];
    if (R.heads == 0) return;
    const Item it(a, R.heads, (blockIdx.z * gridDim.x + blockIdx.x) * 4 + wave_id());
    if (!it.any) return;
    const int p0 = 4 * (threadIdx.x % LPR);
    const bool wide = R.x.vec && R.y.vec && a.rot % 8 == 0 && a.d % 8 == 0;
    const bool in = p0 < a.d / 2;
    const T* x = (const T*)R.x.p + it.b * R.x.sb + (int64_t)it.i * R.x.sr;
    const auto work = [&](auto form) {
        constexpr bool WIDE = decltype(form)::value;
        float u[U][4], v[U][4];
        WideRows<T, U> rows;
        if constexpr (WIDE) rows.load(a, x, R.x.sh, it.h0, Item::kGroups, R.heads, p0);
        float c[4], s[4], wu[4], wv[4];
        load_angles(a, it.b, it.i, p0, c, s);
        load_weights(a, R.w, p0, wu, wv);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int head = it.h0 + k * Item::kGroups;
            const bool live = in && head < R.heads;
            if constexpr (WIDE) {
                rows.pairs(a, k, live, p0, u[k], v[k]);
                continue;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) u[k][e] = v[k][e] = 0.f;
            if (live) load_pairs(a, x + head * R.x.sh, p0, false, u[k], v[k]);
        }
        T* y = (T*)R.y.p + it.b * R.y.sb + (int64_t)it.i * R.y.sr;
        const float dinv = 1.f / (float)a.d;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            float q = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) q = fmaf(u[k][e], u[k][e], fmaf(v[k][e], v[k][e], q));
            q = row_sum<LPR>(q);
            const float inv = 1.f / sqrtf(fmaf(q, dinv, a.eps));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float zu = u[k][e] * inv * wu[e], zv = v[k][e] * inv * wv[e];
                u[k][e] = fmaf(zu, c[e], -zv * s[e]);
                v[k][e] = fmaf(zv, c[e], zu * s[e]);
            }
            const int head = it.h0 + k * Item::kGroups;
            if (in && head < R.heads) store_pairs(a, y + head * R.y.sh, p0, WIDE, u[k], v[k]);
        }
    };
    if (wide)
        work(std::true_type{});
    else
        work(std::false_type{});
}

// Backward: a workgroup takes items blockIdx.x * 4 + wave, in steps of the grid;
// a lane's pairs are the same in every row, so the weights' gradient is summed
// in registers, over the workgroup in LDS and over workgroups by
// norm_weight_kernel, in a fixed order.
template <int OP, int LPR, int U>
__global__ __launch_bounds__(256) void norm_rotate_bwd_kernel(const NormArgs a) {
    using T = typename El<OP>::T;
    using Item = NormItem<LPR, U>;
    constexpr int GRP = 256 / LPR;
    __shared__ float red[GRP][8 * LPR];
    const NormRows& R = a.r[blockIdx.y];
    if (R.heads == 0) return;
    const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR, p0 = 4 * lane;
    const bool wide = R.x.vec && R.y.vec && R.g.vec && a.rot % 8 == 0 && a.d % 8 == 0;
    const bool in = p0 < a.d / 2;
    float wu[4], wv[4], du[4] = {0, 0, 0, 0}, dv[4] = {0, 0, 0, 0};
    load_weights(a, R.w, p0, wu, wv);
    const float dinv = 1.f / (float)a.d;
    // Two loops, so that the usual one does not hold the other's registers (150
    // for one with both, three waves a SIMD, 129 us; 108, four, 102 us).
    const auto work = [&](auto form) {
        constexpr bool WIDE = decltype(form)::value;
        for (uint32_t item = blockIdx.x * 4 + wave_id();; item += gridDim.x * 4) {
            const Item it(a, R.heads, item);
            if (!it.any) break;
            const T* x = (const T*)R.x.p + it.b * R.x.sb + (int64_t)it.i * R.x.sr;
            const T* g = (const T*)R.g.p + it.b * R.g.sb + (int64_t)it.i * R.g.sr;
            T* y = (T*)R.y.p + it.b * R.y.sb + (int64_t)it.i * R.y.sr;
            float u[U][4], v[U][4], gu[U][4], gv[U][4];
            WideRows<T, U> xs, gs;
            if constexpr (WIDE) {
                xs.load(a, x, R.x.sh, it.h0, Item::kGroups, R.heads, p0);
                gs.load(a, g, R.g.sh, it.h0, Item::kGroups, R.heads, p0);
            }
            float c[4], s[4];
            load_angles(a, it.b, it.i, p0, c, s);
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int head = it.h0 + k * Item::kGroups;
                const bool live = in && head < R.heads;
                if constexpr (WIDE) {
                    xs.pairs(a, k, live, p0, u[k], v[k]);
                    gs.pairs(a, k, live, p0, gu[k], gv[k]);
                    continue;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) u[k][e] = v[k][e] = gu[k][e] = gv[k][e] = 0.f;
                if (live) {
                    load_pairs(a, x + head * R.x.sh, p0, false, u[k], v[k]);
                    load_pairs(a, g + head * R.g.sh, p0, false, gu[k], gv[k]);
                }
            }
#pragma unroll
            for (int k = 0; k < U; ++k) {
                float q = 0.f, m = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float tu = fmaf(gu[k][e], c[e], gv[k][e] * s[e]);
                    const float tv = fmaf(gv[k][e], c[e], -gu[k][e] * s[e]);
                    gu[k][e] = tu;
                    gv[k][e] = tv;
                    q = fmaf(u[k][e], u[k][e], fmaf(v[k][e], v[k][e], q));
                    m = fmaf(u[k][e] * wu[e], tu, fmaf(v[k][e] * wv[e], tv, m));
                }
                q = row_sum<LPR>(q);
                m = row_sum<LPR>(m);
                // (lanes without a head hold zeros: with eps = 0 their 1 / 0 would
                // reach the weights' sums)
                const int head = it.h0 + k * Item::kGroups;
                const float inv = head < R.heads ? 1.f / sqrtf(fmaf(q, dinv, a.eps)) : 0.f;
                const float k2 = inv * inv * m * dinv;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    du[e] = fmaf(u[k][e] * inv, gu[k][e], du[e]);
                    dv[e] = fmaf(v[k][e] * inv, gv[k][e], dv[e]);
                    u[k][e] = inv * fmaf(wu[e], gu[k][e], -u[k][e] * k2);
                    v[k][e] = inv * fmaf(wv[e], gv[k][e], -v[k][e] * k2);
                }
                if (in && head < R.heads) store_pairs(a, y + head * R.y.sh, p0, WIDE, u[k], v[k]);
            }
        }
    };
    if (wide)
        work(std::true_type{});
    else
        work(std::false_type{});
    if (!R.gw) return;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        red[grp][8 * lane + k] = du[k];
        red[grp][8 * lane + 4 + k] = dv[k];
    }
    __syncthreads();
    for (int x = threadIdx.x; x < 8 * LPR; x += 256) {
        const int p = 4 * (x >> 3) + (x & 3);
        if (p >= a.d / 2) continue;
        float t = 0.f;
#pragma unroll
        for (int y = 0; y < GRP; ++y) t += red[y][x];
        a.part[((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * a.d + pair_at(a, p, (x >> 2) & 1)] = t;
    }
}

// dw[x]: the workgroups' parts, in 64 bits and a fixed order; 8 elements a
// workgroup, 32 lanes an element.
__global__ __launch_bounds__(256) void norm_weight_kernel(const NormArgs a, int blocks) {
    __shared__ double red[32][8];
    const NormRows& R = a.r[blockIdx.y];
    if (!R.gw) return;
    const int e = threadIdx.x & 7, x = blockIdx.x * 8 + e, y = threadIdx.x >> 3;
    double s = 0.0;
    if (x < a.d && R.heads > 0) {
#pragma unroll 8
        for (int k = y; k < blocks; k += 32)
            s += (double)a.part[((int64_t)blockIdx.y * blocks + k) * a.d + x];
    }
    red[y][e] = s;
    __syncthreads();
    for (int o = 16; o >= 1; o >>= 1) {
        if (y < o) red[y][e] += red[y + o][e];
        __syncthreads();
    }
    if (y == 0 && x < a.d) R.gw[x] = (float)red[0][e];
}

// Rows a lane group: four (backward: two) where that still leaves every SIMD
// several waves, else one (the latency of a single token's rows is then one
// load's).  Several / one, us, 40 heads of 128 in bf16: 40960 rows, forward 9.8 /
// 9.2, backward 15.0 / 14.9; 81920, 11.9 / 13.4, 19.5 / 20.5; 131072, 17.0 / 18.5,
// 25.1 / 26.5; 327680, 33.7 / 40.3, 48.6 / 51.0.  Few heads leave lanes of a wave
// of several rows without any (2 heads, 131072 rows, 43.9 / 31.4, 49.2 / 38.0).
constexpr int64_t kManyRows = 131072;
int64_t items(const NormArgs& a, int lpr, int u) {
    const int per = 64 / lpr * u;
    const int64_t q = (a.r[0].heads + per - 1) / per, k = (a.r[1].heads + per - 1) / per;
    return (int64_t)a.B * a.n * (q > k ? q : k);
}

template <int OP, int LPR>
hipError_t fwd(const NormArgs& a, hipStream_t s) {
    const bool many = (int64_t)a.B * a.n * (a.r[0].heads + a.r[1].heads) >= kManyRows;
    const int64_t n = items(a, LPR, many ? 4 : 1);
    if (n == 0) return hipSuccess;
    const dim3 f = flat_grid((n + 3) / 4), g(f.x, 2, f.y);
    if (many)
        norm_rotate_kernel<OP, LPR, 4><<<g, 256, 0, s>>>(a);
    else
        norm_rotate_kernel<OP, LPR, 1><<<g, 256, 0, s>>>(a);
    return hipGetLastError();
}

template <int OP, int LPR>
hipError_t bwd(const NormArgs& a, hipStream_t s) {
    const bool many = (int64_t)a.B * a.n * (a.r[0].heads + a.r[1].heads) >= kManyRows;
    const dim3 g((unsigned)a.blocks, 2);
    if (many)
        norm_rotate_bwd_kernel<OP, LPR, 2><<<g, 256, 0, s>>>(a);
    else
        norm_rotate_bwd_kernel<OP, LPR, 1><<<g, 256, 0, s>>>(a);
    return hipGetLastError();
}

template <int OP>
hipError_t launch(const NormArgs& a, bool back, hipStream_t s) {
    if (a.d <= 64) return back ? bwd<OP, 8>(a, s) : fwd<OP, 8>(a, s);
    if (a.d <= 128) return back ? bwd<OP, 16>(a, s) : fwd<OP, 16>(a, s);
    return back ? bwd<OP, 32>(a, s) : fwd<OP, 32>(a, s);
}
hipError_t launch(const NormArgs& a, bool back, hipStream_t s) {
    return a.op == OP_BF16 ? launch<OP_BF16>(a, back, s)
           : a.op == OP_F16 ? launch<OP_F16>(a, back, s)
                            : launch<OP_F32>(a, back, s);
}

}  // namespace

int norm_bwd_blocks(int64_t rows) {
    const int64_t b = (rows + 31) / 32;
    return b < 1 ? 1 : b > 1024 ? 1024 : (int)b;
}

hipError_t launch_norm_rotate(const NormArgs& a, hipStream_t s) { return launch(a, false, s); }

hipError_t launch_norm_rotate_bwd(const NormArgs& a, hipStream_t s) {
    const bool any = (int64_t)a.B * a.n > 0;  // else the weights' sums are empty
    const hipError_t e = any ? launch(a, true, s) : hipSuccess;
    if (e != hipSuccess || (!a.r[0].gw && !a.r[1].gw)) return e;
    norm_weight_kernel<<<dim3((unsigned)((a.d + 7) / 8), 2), 256, 0, s>>>(a, any ? a.blocks : 0);
    return hipGetLastError();
}

}  // namespace fs
