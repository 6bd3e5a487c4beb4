// fs_layernorm.hip -- the layer norm of rows with the residual sum in front of
// it, and its gradients:
//   z = x + r,  h = (z - mean z) rstd,  y = w h + b;
//   u = w g,  dx = rstd (u - mean u - h mean(u h)) + dz,  dw = sum g h,  db = sum g.
// Bound by memory: a row is read once and stays in registers over both sums of
// its statistics (the second is of squared distances from the mean, so that a
// large mean costs the variance no digits; the mean itself is an fp32 number).  Up to 1024 elements a row lies with 8 to 64 lanes
// of a wave, whose sums need no barrier, beyond with a workgroup.  (16384 rows of
// 4096, bf16, with the residual: forward 90 us for 537 MB, 6.0 TB/s; backward 116
// us for 537 MB, 4.6 TB/s, and 5 us for the weights' sums; a large copy reaches
// 4.9 TB/s.  32 rows of 4096: 3.7 us.)
#include "fs_layers_args.h"
#include "fs_rowops.hpp"

#include <type_traits>

namespace fs {

namespace {

__device__ __forceinline__ void place(const LayerNormArgs& a, int64_t row, int& b, int& i) {
    b = a.B == 1 ? 0 : (int)((uint32_t)row / (uint32_t)a.n);
    i = (int)(row - (int64_t)b * a.n);
}
__device__ __forceinline__ bool row_on(const LayerNormArgs& a, int b, int i) {
    return !a.lengths || i < a.lengths[b];
}

// LPR threads a row, CH groups of 8 elements a thread.
template <int LPR, int CH, ShareForm FORM>
__device__ __forceinline__ void load_weight(const float* w, int lane, int width, float fill,
                                            float (&out)[CH][8]) {
    if (w) {
        Share<float, LPR, CH, FORM> s;
        s.load(w, lane, width, true);
        __builtin_memcpy(out, s.v, sizeof(out));
        return;
    }
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) out[j][e] = fill;
}

template <int OP, int LPR, int CH, ShareForm FORM>
__global__ __launch_bounds__(threads_of<LPR>()) void layer_norm_kernel(const LayerNormArgs a) {
    using T = typename El<OP>::T;
    constexpr int GRP = threads_of<LPR>() / LPR;
    __shared__ float2 buf[2 * RowFold<LPR>::kWaves];
    RowFold<LPR> fold(buf);
    const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR, W = a.width;
    float w[CH][8], bias[CH][8];
    load_weight<LPR, CH, FORM>(a.w, lane, W, 1.f, w);
    load_weight<LPR, CH, FORM>(a.b, lane, W, 0.f, bias);
    const float inv_w = 1.f / (float)W;
    const int64_t rows = (int64_t)a.B * a.n;
    // (the groups of a workgroup leave the loop together: its sums have barriers)
    for (int64_t first = (int64_t)blockIdx.x * GRP; first < rows; first += (int64_t)gridDim.x * GRP) {
        const int64_t row = first + grp;
        if (LPR <= 64 && row >= rows) break;
        int b, i;
        place(a, row, b, i);
        const bool on = row_on(a, b, i);
        Share<T, LPR, CH, FORM> x, r;
        x.load((const T*)a.x.p + b * a.x.sb + i * a.x.sr, lane, W, on);
        float z[CH][8];
        if (a.r.p) {
            r.load((const T*)a.r.p + b * a.r.sb + i * a.r.sr, lane, W, on);
#pragma unroll
            for (int j = 0; j < CH; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) x.v[j][e] = (T)((float)x.v[j][e] + (float)r.v[j][e]);
            x.store((T*)a.z.p + b * a.z.sb + i * a.z.sr, lane, W);
        }
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < CH; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) s += z[j][e] = (float)x.v[j][e];
        const float mean = fold.sum(s) * inv_w;
        float q = 0.f;
#pragma unroll
        for (int j = 0; j < CH; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                z[j][e] = share_at<LPR, FORM>(lane, j, e) < W ? z[j][e] - mean : 0.f;
                q = fmaf(z[j][e], z[j][e], q);
            }
        q = fold.sum(q);
        const float rstd = 1.f / sqrtf(fmaf(q, inv_w, a.eps));
#pragma unroll
        for (int j = 0; j < CH; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x.v[j][e] = (T)(on ? fmaf(z[j][e] * rstd, w[j][e], bias[j][e]) : 0.f);
        x.store((T*)a.y.p + b * a.y.sb + i * a.y.sr, lane, W);
        if (lane == 0 && a.mean) a.mean[row] = on ? mean : 0.f;
        if (lane == 0 && a.rstd) a.rstd[row] = on ? rstd : 0.f;
    }
}

// Backward: a workgroup takes rows in steps of the grid; a thread's columns are
// the same in every row, so the weights' gradients are summed in its registers,
// over the workgroup's rows in LDS, and over workgroups by layer_norm_sum_kernel.
template <int OP, int LPR, int CH, ShareForm FORM>
__global__ __launch_bounds__(threads_of<LPR>()) void layer_norm_bwd_kernel(const LayerNormArgs a) {
    using T = typename El<OP>::T;
    constexpr int GRP = threads_of<LPR>() / LPR;
    __shared__ float2 buf[2 * RowFold<LPR>::kWaves];
    __shared__ float red[GRP > 1 ? 2 * GRP * LPR * CH * 8 : 1];
    RowFold<LPR> fold(buf);
    const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR, W = a.width;
    float w[CH][8], dw[CH][8], db[CH][8];
    load_weight<LPR, CH, FORM>(a.w, lane, W, 1.f, w);
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[j][e] = db[j][e] = 0.f;
    const float inv_w = 1.f / (float)W;
    const int64_t rows = (int64_t)a.B * a.n, step = (int64_t)gridDim.x * GRP;
    // A row's three reads are issued while the row in front of it is worked on: two
    // workgroups a CU (whose parts of the sums are few then) would leave memory idle
    // over each row's latency (16384 rows of 4096, bf16: 179 us without, 116 with).
    struct Row {
        Share<T, LPR, CH, FORM> z, g, t;
        float mean, rstd;
        int b, i;
        bool on;
    };
    const auto fetch = [&](int64_t row, Row& r) {
        place(a, row, r.b, r.i);
        r.on = row_on(a, r.b, r.i);
        r.z.load((const T*)a.x.p + r.b * a.x.sb + r.i * a.x.sr, lane, W, r.on);
        r.g.load((const T*)a.g.p + r.b * a.g.sb + r.i * a.g.sr, lane, W, r.on);
        if (a.gz.p) r.t.load((const T*)a.gz.p + r.b * a.gz.sb + r.i * a.gz.sr, lane, W, r.on);
        r.mean = r.on ? a.mean[row] : 0.f;
        r.rstd = r.on ? a.rstd[row] : 0.f;
    };
    // (1024 threads a row have no registers for it: single elements in bf16 and fp32 and
    // fp32 from whole dwords on keep one or two of 128 in memory as it is)
    constexpr bool AHEAD = LPR <= 256;
    Row next;
    int64_t first = (int64_t)blockIdx.x * GRP;
    if (AHEAD && first + grp < rows) fetch(first + grp, next);
    for (; first < rows; first += step) {
        const int64_t row = first + grp;
        if (LPR <= 64 && row >= rows) break;
        Row r;
        if constexpr (AHEAD) {
            r = next;
            if (row + step < rows) fetch(row + step, next);
        } else {
            fetch(row, r);
        }
        float h[CH][8], s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int j = 0; j < CH; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float ge = (float)r.g.v[j][e];  // 0 behind the row's end
                h[j][e] = ((float)r.z.v[j][e] - r.mean) * r.rstd;
                dw[j][e] = fmaf(ge, h[j][e], dw[j][e]);
                db[j][e] += ge;
                const float u = ge * w[j][e];
                s1 += u;
                s2 = fmaf(u, h[j][e], s2);
            }
        const float2 s = fold.sum2(s1, s2);
        const float m1 = s.x * inv_w, m2 = s.y * inv_w;
#pragma unroll
        for (int j = 0; j < CH; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float d = r.rstd * (fmaf((float)r.g.v[j][e], w[j][e], -m1) - h[j][e] * m2);
                if (a.gz.p) d += (float)r.t.v[j][e];
                r.z.v[j][e] = (T)(r.on ? d : 0.f);
            }
        r.z.store((T*)a.gx.p + r.b * a.gx.sb + r.i * a.gx.sr, lane, W);
    }
    if (!a.part) return;
    float* part = a.part + (int64_t)blockIdx.x * 2 * W;
    if constexpr (GRP == 1) {
#pragma unroll
        for (int j = 0; j < CH; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int at = share_at<LPR, FORM>(lane, j, e);
                if (at < W) part[at] = dw[j][e], part[W + at] = db[j][e];
            }
    } else {
        constexpr int C = LPR * CH * 8;
#pragma unroll
        for (int j = 0; j < CH; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int at = share_at<LPR, FORM>(lane, j, e);
                red[grp * C + at] = dw[j][e];
                red[(GRP + grp) * C + at] = db[j][e];
            }
        __syncthreads();
        for (int x = threadIdx.x; x < W; x += threads_of<LPR>()) {
            float sw = 0.f, sb = 0.f;
#pragma unroll
            for (int y = 0; y < GRP; ++y) sw += red[y * C + x], sb += red[(GRP + y) * C + x];
            part[x] = sw;
            part[W + x] = sb;
        }
    }
}

// dw and db: the workgroups' parts in 64 bits and a fixed order; 32 columns a
// workgroup, 32 lanes a column.
__global__ __launch_bounds__(1024) void layer_norm_sum_kernel(const LayerNormArgs a, int blocks) {
    __shared__ double red[32][33];
    const int c = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t x = (int64_t)blockIdx.x * 32 + c;  // of 2 width
    double s = 0.0;
    if (x < 2 * a.width) {
#pragma unroll 8
        for (int k = y; k < blocks; k += 32) s += (double)a.part[(int64_t)k * 2 * a.width + x];
    }
    red[y][c] = s;
    __syncthreads();
    for (int o = 16; o >= 1; o >>= 1) {
        if (y < o) red[y][c] += red[y + o][c];
        __syncthreads();
    }
    if (y || x >= 2 * a.width) return;
    s = red[0][c];
    if (x < a.width) {
        if (a.gw) a.gw[x] = (float)s;
    } else if (a.gb) {
        a.gb[x - a.width] = (float)s;
    }
}

template <int OP, int LPR, int CH, ShareForm FORM>
hipError_t launch(const LayerNormArgs& a, bool back, hipStream_t s) {
    constexpr int GRP = threads_of<LPR>() / LPR;
    const int64_t groups = ((int64_t)a.B * a.n + GRP - 1) / GRP;
    if (back)
        layer_norm_bwd_kernel<OP, LPR, CH, FORM><<<(unsigned)a.blocks, threads_of<LPR>(), 0, s>>>(a);
    else
        layer_norm_kernel<OP, LPR, CH, FORM>
            <<<(unsigned)(groups < 4096 ? groups : 4096), threads_of<LPR>(), 0, s>>>(a);
    return hipGetLastError();
}
template <int OP, int LPR, int CH>
hipError_t launch(const LayerNormArgs& a, bool back, hipStream_t s) {
    return a.form == WIDE     ? launch<OP, LPR, CH, WIDE>(a, back, s)
           : a.form == DWORDS ? launch<OP, LPR, CH, DWORDS>(a, back, s)
                              : launch<OP, LPR, CH, SINGLE>(a, back, s);
}
template <int OP>
hipError_t launch(const LayerNormArgs& a, bool back, hipStream_t s) {
    if (a.width <= 64) return launch<OP, 8, 1>(a, back, s);
    if (a.width <= 128) return launch<OP, 16, 1>(a, back, s);
    if (a.width <= 256) return launch<OP, 32, 1>(a, back, s);
    if (a.width <= 512) return launch<OP, 64, 1>(a, back, s);
    if (a.width <= 1024) return launch<OP, 64, 2>(a, back, s);
    if (a.width <= 2048) return launch<OP, 256, 1>(a, back, s);
    if (a.width <= 4096) return launch<OP, 256, 2>(a, back, s);
    if (a.width <= 8192) return launch<OP, 512, 2>(a, back, s);
    return launch<OP, 1024, 2>(a, back, s);
}
hipError_t launch(const LayerNormArgs& a, bool back, hipStream_t s) {
    return a.op == OP_BF16 ? launch<OP_BF16>(a, back, s)
           : a.op == OP_F16 ? launch<OP_F16>(a, back, s)
                            : launch<OP_F32>(a, back, s);
}

}  // namespace

// Workgroups of the backward pass: two a CU (of 1024 threads one), each of which
// leaves 2 x width sums to add up (us, 256 / 512 workgroups: 4096 rows of 16384, bf16,
// 137 / 155; 16384 rows of 4096, 151 / 119).
int layer_norm_bwd_blocks(int64_t rows, int width) {
    const int grp = width <= 64 ? 32 : width <= 128 ? 16 : width <= 256 ? 8 : width <= 1024 ? 4 : 1;
    const int64_t b = (rows + grp - 1) / grp;
    const int most = width > 8192 ? 256 : 512;
    return b < 1 ? 1 : b > most ? most : (int)b;
}

hipError_t launch_layer_norm(const LayerNormArgs& a, hipStream_t s) { return launch(a, false, s); }

hipError_t launch_layer_norm_bwd(const LayerNormArgs& a, hipStream_t s) {
    const bool any = (int64_t)a.B * a.n > 0;  // else the weights' sums are empty
    const hipError_t e = any ? launch(a, true, s) : hipSuccess;
    if (e != hipSuccess || !a.part) return e;
    layer_norm_sum_kernel<<<(unsigned)((2 * a.width + 31) / 32), 1024, 0, s>>>(a, any ? a.blocks : 0);
    return hipGetLastError();
}

}  // namespace fs
