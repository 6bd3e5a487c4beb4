// fs_qknorm.hip -- the norm of every head's row of queries and keys and the
// rotation by its position, in one pass, and the pass's gradients:
//   r = 1 / sqrt(mean(x^2) + eps),  z = w x r,  y = R z  (R a rotation of pairs)
//   g = R^T dy,  dw = sum over rows of x r g,  dx = r (w g - x r^2 mean(x w g)).
// Bound by memory: a row of d elements is read once and written once, the
// angles' cosines and sines are shared by the heads of a token.  A lane holds
// four pairs (8 elements), d / 8 lanes (rounded up to a power of two) a row,
// so a row's sums are butterflies within those lanes.
#include "fs_attn.hpp"

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
#pragma unroll
    for (int x = 0; x < 4; ++x)
        if (p0 + x < half) c[x] = ct[x], s[x] = st[x];
}
// Weights of a lane's pairs.
__device__ __forceinline__ void load_weights(const NormArgs& a, const float* w, int p0,
                                             float (&u)[4], float (&v)[4]) {
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

template <int OP, int LPR>
__global__ __launch_bounds__(256) void norm_rotate_kernel(const NormArgs a) {
    using T = typename El<OP>::T;
    const NormRows& R = a.r[blockIdx.y];
    const uint32_t rows = (uint32_t)a.B * a.n * R.heads;
    const uint32_t r = blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
    const int p0 = 4 * (threadIdx.x % LPR);
    if (r >= rows) return;
    const uint32_t tok = r / R.heads;
    const int head = (int)(r - tok * R.heads), b = (int)(tok / a.n), i = (int)(tok - b * (uint32_t)a.n);
    const bool wide = R.x.vec && R.y.vec && a.rot % 8 == 0 && a.d % 8 == 0;
    const bool in = p0 < a.d / 2;
    const T* x = (const T*)R.x.p + b * R.x.sb + (int64_t)i * R.x.sr + head * R.x.sh;
    float u[4] = {0, 0, 0, 0}, v[4] = {0, 0, 0, 0};
    if (in) load_pairs(a, x, p0, wide, u, v);
    float c[4], s[4], wu[4], wv[4];
    load_angles(a, b, i, p0, c, s);
    load_weights(a, R.w, p0, wu, wv);
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) q = fmaf(u[k], u[k], fmaf(v[k], v[k], q));
    q = row_sum<LPR>(q);
    const float inv = 1.f / sqrtf(q / (float)a.d + a.eps);
    if (!in) return;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float zu = u[k] * inv * wu[k], zv = v[k] * inv * wv[k];
        u[k] = fmaf(zu, c[k], -zv * s[k]);
        v[k] = fmaf(zv, c[k], zu * s[k]);
    }
    store_pairs(a, (T*)R.y.p + b * R.y.sb + (int64_t)i * R.y.sr + head * R.y.sh, p0, wide, u, v);
}

// Backward: a workgroup takes rows blockIdx.x, + gridDim.x, ... in groups of
// 256 / LPR; a lane's pairs are the same in every row, so the weights'
// gradient is summed in registers, over the workgroup in LDS and over
// workgroups by norm_weight_kernel, in a fixed order.
template <int OP, int LPR>
__global__ __launch_bounds__(256) void norm_rotate_bwd_kernel(const NormArgs a) {
    using T = typename El<OP>::T;
    constexpr int RPB = 256 / LPR;
    __shared__ float red[RPB][8 * LPR];
    const NormRows& R = a.r[blockIdx.y];
    const uint32_t rows = (uint32_t)a.B * a.n * R.heads;
    const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR, p0 = 4 * lane;
    const bool wide = R.x.vec && R.y.vec && R.g.vec && a.rot % 8 == 0 && a.d % 8 == 0;
    const bool in = p0 < a.d / 2;
    float wu[4], wv[4], du[4] = {0, 0, 0, 0}, dv[4] = {0, 0, 0, 0};
    load_weights(a, R.w, p0, wu, wv);
    const float dinv = 1.f / (float)a.d;
    for (uint32_t r = blockIdx.x * RPB + grp; r < rows; r += gridDim.x * RPB) {
        const uint32_t tok = r / R.heads;
        const int head = (int)(r - tok * R.heads), b = (int)(tok / a.n),
                  i = (int)(tok - b * (uint32_t)a.n);
        const T* x = (const T*)R.x.p + b * R.x.sb + (int64_t)i * R.x.sr + head * R.x.sh;
        const T* g = (const T*)R.g.p + b * R.g.sb + (int64_t)i * R.g.sr + head * R.g.sh;
        float u[4] = {0, 0, 0, 0}, v[4] = {0, 0, 0, 0}, gu[4] = {0, 0, 0, 0}, gv[4] = {0, 0, 0, 0};
        if (in) {
            load_pairs(a, x, p0, wide, u, v);
            load_pairs(a, g, p0, wide, gu, gv);
        }
        float c[4], s[4];
        load_angles(a, b, i, p0, c, s);
        float q = 0.f, m = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float tu = fmaf(gu[k], c[k], gv[k] * s[k]), tv = fmaf(gv[k], c[k], -gu[k] * s[k]);
            gu[k] = tu;
            gv[k] = tv;
            q = fmaf(u[k], u[k], fmaf(v[k], v[k], q));
            m = fmaf(u[k] * wu[k], tu, fmaf(v[k] * wv[k], tv, m));
        }
        q = row_sum<LPR>(q);
        m = row_sum<LPR>(m);
        const float inv = 1.f / sqrtf(q * dinv + a.eps);
        const float k2 = inv * inv * m * dinv;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            du[k] = fmaf(u[k] * inv, gu[k], du[k]);
            dv[k] = fmaf(v[k] * inv, gv[k], dv[k]);
            u[k] = inv * fmaf(wu[k], gu[k], -u[k] * k2);
            v[k] = inv * fmaf(wv[k], gv[k], -v[k] * k2);
        }
        if (in)
            store_pairs(a, (T*)R.y.p + b * R.y.sb + (int64_t)i * R.y.sr + head * R.y.sh, p0, wide, u,
                        v);
    }
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
        for (int y = 0; y < RPB; ++y) t += red[y][x];
        a.part[((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * a.d + pair_at(a, p, (x >> 2) & 1)] = t;
    }
}

// dw[x]: the workgroups' parts, in 64 bits and a fixed order; 32 elements a
// workgroup, 8 lanes an element.
__global__ __launch_bounds__(256) void norm_weight_kernel(const NormArgs a, int blocks) {
    __shared__ double red[8][32];
    const NormRows& R = a.r[blockIdx.y];
    if (!R.gw) return;
    const int x = blockIdx.x * 32 + (threadIdx.x & 31), y = threadIdx.x >> 5;
    double s = 0.0;
    if (x < a.d && R.heads > 0)
        for (int k = y; k < blocks; k += 8)
            s += (double)a.part[((int64_t)blockIdx.y * blocks + k) * a.d + x];
    red[y][threadIdx.x & 31] = s;
    __syncthreads();
    if (y == 0 && x < a.d) {
        for (int k = 1; k < 8; ++k) s += red[k][threadIdx.x & 31];
        R.gw[x] = (float)s;
    }
}

int64_t most_rows(const NormArgs& a) {
    const int h = a.r[0].heads > a.r[1].heads ? a.r[0].heads : a.r[1].heads;
    return (int64_t)a.B * a.n * h;
}

template <int OP>
hipError_t fwd(const NormArgs& a, hipStream_t s) {
    const int64_t rows = most_rows(a);
    if (rows == 0) return hipSuccess;
    if (a.d <= 64)
        norm_rotate_kernel<OP, 8><<<dim3((unsigned)((rows + 31) / 32), 2), 256, 0, s>>>(a);
    else if (a.d <= 128)
        norm_rotate_kernel<OP, 16><<<dim3((unsigned)((rows + 15) / 16), 2), 256, 0, s>>>(a);
    else
        norm_rotate_kernel<OP, 32><<<dim3((unsigned)((rows + 7) / 8), 2), 256, 0, s>>>(a);
    return hipGetLastError();
}

template <int OP>
hipError_t bwd(const NormArgs& a, hipStream_t s) {
    const dim3 g((unsigned)a.blocks, 2);
    if (a.d <= 64)
        norm_rotate_bwd_kernel<OP, 8><<<g, 256, 0, s>>>(a);
    else if (a.d <= 128)
        norm_rotate_bwd_kernel<OP, 16><<<g, 256, 0, s>>>(a);
    else
        norm_rotate_bwd_kernel<OP, 32><<<g, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

int norm_bwd_blocks(int64_t rows) {
    const int64_t b = (rows + 31) / 32;
    return b < 1 ? 1 : b > 1024 ? 1024 : (int)b;
}

hipError_t launch_norm_rotate(const NormArgs& a, hipStream_t s) {
    return a.op == OP_BF16 ? fwd<OP_BF16>(a, s) : a.op == OP_F16 ? fwd<OP_F16>(a, s)
                                                                : fwd<OP_F32>(a, s);
}

hipError_t launch_norm_rotate_bwd(const NormArgs& a, hipStream_t s) {
    hipError_t e = a.op == OP_BF16 ? bwd<OP_BF16>(a, s) : a.op == OP_F16 ? bwd<OP_F16>(a, s)
                                                                        : bwd<OP_F32>(a, s);
    if (e != hipSuccess || (!a.r[0].gw && !a.r[1].gw)) return e;
    norm_weight_kernel<<<dim3((unsigned)((a.d + 31) / 32), 2), 256, 0, s>>>(a, a.blocks);
    return hipGetLastError();
}

}  // namespace fs
