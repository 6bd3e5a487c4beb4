// fs_quant.hip -- rows held in 8-bit integers with a scale each, and the product
// of two such sets:
//   a = max |x|, q = 127 x / a to the nearest whole number, scale = a / 127;
//   y_ij = scale_i scale'_j sum_k q_ik q'_jk + b_j, the sum exact in 32 bits.
#include "fs_layers_args.h"
#include "fs_rowops.hpp"

#include <algorithm>

namespace fs {

namespace {

typedef __attribute__((__vector_size__(4 * sizeof(int)))) int i32x4;
typedef __attribute__((__vector_size__(16 * sizeof(int)))) int i32x16;

// ---- quantisation -----------------------------------------------------------

// The whole number nearest to 127 x / a, |x| <= a.  In fp32 the quotient is off by
// less than 127 * 2^-22 < 1e-4; nearer than that to a half (and where 127 / a is
// no fp32 number) the products 254 x and (2 q +- 1) a, exact in 64 bits, decide.
__device__ __forceinline__ int quantized(float x, float a, float inv) {
    const float r = x * inv, q = rintf(r);
    if (fabsf(r - q) < 0.4999f) return (int)q;
    if (a == 0.f) return 0;
    const double p = 254.0 * (double)x, top = (double)a;
    int n = (int)(p * (0.5 / top));  // off by less than one and a half
#pragma unroll
    for (int step = 0; step < 2; ++step) {
        const double hi = (2 * n + 1) * top, lo = (2 * n - 1) * top;
        if (p > hi || (p == hi && (n & 1)))
            ++n;
        else if (p < lo || (p == lo && (n & 1)))
            --n;
    }
    return n;
}

template <int LPR>
constexpr int threads_of() {
    return LPR > 256 ? LPR : 256;
}

// Bound by memory: a row is read once and stays in registers over its maximum.
template <int OP, int LPR, int CH, bool WIDE>
__global__ __launch_bounds__(threads_of<LPR>()) void quantize_kernel(const QuantArgs a) {
    using T = typename El<OP>::T;
    constexpr int GRP = threads_of<LPR>() / LPR;
    __shared__ float2 buf[2 * RowFold<LPR>::kWaves];
    RowFold<LPR> fold(buf);
    const int lane = threadIdx.x % LPR, W = a.width;
    const int64_t row = flat_block() * GRP + threadIdx.x / LPR;
    if (row >= a.rows) return;  // (LPR > 64: the whole workgroup)
    Share<T, LPR, CH, WIDE> x;
    x.load((const T*)a.x + row * a.sx, lane, W, true);
    // magnitudes compare as their bits do, NaN above infinity
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            top = max(top, __float_as_uint((float)x.v[j][e]) & 0x7fffffffu);
    top = fold.max_bits(top);
    const bool finite = top < 0x7f800000u;
    const float amax = __uint_as_float(top), inv = 127.f / amax;
    int8_t* q = a.q + row * a.sq;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        int8_t out[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            out[e] = finite ? (int8_t)quantized((float)x.v[j][e], amax, inv) : (int8_t)0;
        if constexpr (WIDE) {
            const int at = share_at<LPR, true>(lane, j, 0);
            if (at < W) __builtin_memcpy(__builtin_assume_aligned(q + at, 8), out, 8);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int at = share_at<LPR, false>(lane, j, e);
                if (at < W) q[at] = out[e];
            }
        }
    }
    if (lane == 0) a.scale[row] = finite ? amax / 127.f : NAN;
}

template <int OP, int LPR, int CH>
hipError_t quantize(const QuantArgs& a, hipStream_t s) {
    constexpr int GRP = threads_of<LPR>() / LPR;
    const dim3 grid = flat_grid(((int64_t)a.rows + GRP - 1) / GRP);
    if (a.wide)
        quantize_kernel<OP, LPR, CH, true><<<grid, threads_of<LPR>(), 0, s>>>(a);
    else
        quantize_kernel<OP, LPR, CH, false><<<grid, threads_of<LPR>(), 0, s>>>(a);
    return hipGetLastError();
}
template <int OP>
hipError_t quantize(const QuantArgs& a, hipStream_t s) {
    if (a.width <= 128) return quantize<OP, 16, 1>(a, s);
    if (a.width <= 512) return quantize<OP, 64, 1>(a, s);
    if (a.width <= 2048) return quantize<OP, 256, 1>(a, s);
    if (a.width <= 8192) return quantize<OP, 256, 4>(a, s);
    return quantize<OP, 1024, 8>(a, s);
}

// ---- product ----------------------------------------------------------------

// Sixteen bytes of a row from k on; zeros from k = end on.
__device__ __forceinline__ i32x4 load_chunk(const int8_t* row, int k, int end) {
    i32x4 v = {0, 0, 0, 0};
    if (k + 16 <= end) {
        __builtin_memcpy(&v, row + k, 16);
    } else {
        int8_t t[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) t[i] = k + i < end ? row[k + i] : (int8_t)0;
        __builtin_memcpy(&v, t, 16);
    }
    return v;
}

template <int OP>
__device__ __forceinline__ void put(const ProductArgs& a, int i, int j, int sum, float sw, float bias) {
    using T = typename El<OP>::T;
    ((T*)a.y)[i * a.sy + j] = (T)fmaf((float)sum * a.scale_x[i], sw, bias);
}

// Few rows: a workgroup takes 16 columns and all rows (RB blocks of 16), its
// waves divide k.  Bound by the read of the columns' bytes.
template <int OP, int RB>
__global__ __launch_bounds__(256) void product_rows_kernel(const ProductArgs a) {
    __shared__ int red[4][RB * 256];
    const int lane = threadIdx.x & 63, wave = wave_id(), r = lane & 15, c = lane >> 4;
    const int j0 = blockIdx.x * 16;
    const int8_t* w = a.w + (int64_t)min(j0 + r, a.n - 1) * a.sw;
    const int8_t* x[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) x[b] = a.x + (int64_t)min(16 * b + r, a.m - 1) * a.sx;
    i32x4 acc[RB] = {};
    const int steps = (a.k + 63) / 64;
    for (int t = wave; t < steps; t += 4) {
        const int k = t * 64 + c * 16;
        const i32x4 wv = load_chunk(w, k, a.k);
#pragma unroll
        for (int b = 0; b < RB; ++b)
            acc[b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(load_chunk(x[b], k, a.k), wv, acc[b], 0, 0, 0);
    }
    // a lane holds column r, rows 4 c .. 4 c + 3 of each block
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) red[wave][b * 256 + (4 * c + e) * 16 + r] = acc[b][e];
    __syncthreads();
    for (int p = threadIdx.x; p < RB * 256; p += 256) {
        const int i = p / 16, j = j0 + p % 16;
        if (i < a.m && j < a.n)
            put<OP>(a, i, j, red[0][p] + red[1][p] + red[2][p] + red[3][p], a.scale_w[j],
                    a.bias ? a.bias[j] : 0.f);
    }
}

// Tiles of BM x BN outputs over steps of 128 k, in two buffers of LDS: while the
// matrix units work on one, the next step's rows come into the other.  The 16-byte
// chunks of a row of 128 bytes stand in an order that depends on its number, so
// that 16 lanes reading one chunk of 16 rows use all banks.  WM x WN waves.
template <int BM, int BN, int WM, int WN>
struct Tile {
    static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
    static constexpr int MI = BM / WM / 32, NI = BN / WN / 32;
    static constexpr int kStage = (BM + BN) * 128;
};
__device__ __forceinline__ uint32_t chunk_at(int row, int chunk) {
    return row * 128 + ((chunk ^ (row >> 1)) & 7) * 16;
}

template <int OP, int BM, int BN, int WM, int WN, bool ALIGNED>
__global__ __launch_bounds__(64 * WM * WN) void product_kernel(const ProductArgs a) {
    using L = Tile<BM, BN, WM, WN>;
    constexpr int MI = L::MI, NI = L::NI;
    extern __shared__ __align__(16) char lds[];
    const uint32_t base = lds_addr(lds);
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int rows = (a.m + BM - 1) / BM, cols = (a.n + BN - 1) / BN;
    // tiles that an XCD works on at one time share operands: eight row blocks of
    // one column block after the other
    int bi, bj;
    {
        const int total = rows * cols, id = blockIdx.x;
        const int xcd = id & 7, q = total >> 3, rem = total & 7;
        const int at = xcd * q + min(xcd, rem) + (id >> 3);
        const int band = at / (8 * cols), first = band * 8, high = min(8, rows - first);
        bi = first + (at - band * 8 * cols) % high;
        bj = (at - band * 8 * cols) / high;
    }
    const int i0 = bi * BM, j0 = bj * BN;
    const int k0 = blockIdx.y * a.split_k, k1 = min(a.k, k0 + a.split_k);
    const int steps = (k1 - k0 + 127) / 128;
    constexpr int kCopies = (BM + BN) * 8 / L::kThreads;  // 16-byte chunks of a thread
    // chunk c of a wave's copies covers 8 rows of the tiles, x's first
    const auto source = [&](int c, int& row, int& chunk) -> const int8_t* {
        const int t = (wave * kCopies + c) * 8 + (lane >> 3);
        row = t;
        chunk = (lane ^ (t >> 1)) & 7;
        return t < BM ? a.x + (int64_t)min(i0 + t, a.m - 1) * a.sx
                      : a.w + (int64_t)min(j0 + t - BM, a.n - 1) * a.sw;
    };
    uint32_t voff[kCopies];
    i32x4 held[kCopies];
    if constexpr (ALIGNED) {
#pragma unroll
        for (int c = 0; c < kCopies; ++c) {
            int row, chunk;
            const int8_t* p = source(c, row, chunk);
            const bool left = (wave * kCopies + c) * 8 < BM;
            voff[c] = (uint32_t)(p - (left ? a.x + (int64_t)i0 * a.sx : a.w + (int64_t)j0 * a.sw)) + chunk * 16;
        }
    }
    const auto fetch = [&](int t) {
        if constexpr (ALIGNED) {
            const int k = k0 + t * 128;
#pragma unroll
            for (int c = 0; c < kCopies; ++c) {
                const bool left = (wave * kCopies + c) * 8 < BM;
                const int8_t* from = (left ? a.x + (int64_t)i0 * a.sx : a.w + (int64_t)j0 * a.sw) + k;
                // chunks behind the end: the row's first ones, which the products leave out
                const uint32_t chunk = (lane ^ (((wave * kCopies + c) * 8 + (lane >> 3)) >> 1)) & 7;
                const uint32_t back = k + (int)chunk * 16 < k1 ? 0 : chunk * 16;
                dma_to_lds16((const char*)from, voff[c] - back,
                             lds + (t & 1) * L::kStage + (wave * kCopies + c) * 1024);
            }
        } else {
#pragma unroll
            for (int c = 0; c < kCopies; ++c) {
                int row, chunk;
                const int8_t* p = source(c, row, chunk);
                held[c] = load_chunk(p, k0 + t * 128 + chunk * 16, k1);
            }
        }
    };
    const auto keep = [&](int t) {
        if constexpr (!ALIGNED) {
#pragma unroll
            for (int c = 0; c < kCopies; ++c)
                lds_write<i32x4>(base + (t & 1) * L::kStage + (wave * kCopies + c) * 1024 + lane * 16,
                                 held[c]);
        }
    };
    const int wm = wave / WN, wn = wave % WN;
    const int ra = wm * MI * 32 + (lane & 31), rb = BM + wn * NI * 32 + (lane & 31);
    i32x16 acc[MI][NI] = {};
    const auto work = [&](int t, bool tail) {
        const uint32_t at = base + (t & 1) * L::kStage;
        const int left = k1 - k0 - t * 128;
        // operands of the next 32 k are read while this one's products run
        i32x4 x[2][MI], w[2][NI];
        const auto read = [&](int kk) {
            const int chunk = 2 * kk + (lane >> 5);
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                x[kk & 1][i] = lds_read<i32x4>(at + chunk_at(ra + 32 * i, chunk));
                if (ALIGNED && tail && chunk * 16 >= left) x[kk & 1][i] = i32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int j = 0; j < NI; ++j)
                w[kk & 1][j] = lds_read<i32x4>(at + chunk_at(rb + 32 * j, chunk));
        };
        read(0);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            if (kk < 3) read(kk + 1);
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(x[kk & 1][i], w[kk & 1][j],
                                                                      acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    const int whole = ALIGNED ? (k1 - k0) / 128 : steps;
    if (steps > 0) {
        fetch(0);
        keep(0);
    }
    for (int t = 0; t < whole; ++t) {
        // this step's rows are there, and nobody reads the other buffer any more
        if constexpr (ALIGNED) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        stage_barrier();
        if (t + 1 < steps) fetch(t + 1);
        work(t, false);
        if (t + 1 < steps) keep(t + 1);
    }
    if (whole < steps) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        stage_barrier();
        work(whole, true);
    }
    const int h = lane >> 5;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
        const int col = j0 + wn * NI * 32 + 32 * j + (lane & 31);
        if (col >= a.n) continue;
        const float sw = a.scale_w[col], bias = a.bias ? a.bias[col] : 0.f;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            __builtin_amdgcn_sched_barrier(0);  // (64 rows' places at a time would not fit)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = i0 + wm * MI * 32 + 32 * i + 8 * (r >> 2) + 4 * h + (r & 3);
                if (row >= a.m) continue;
                if (a.split > 1)
                    a.part[((int64_t)blockIdx.y * a.m + row) * a.n + col] = acc[i][j][r];
                else
                    put<OP>(a, row, col, acc[i][j][r], sw, bias);
            }
        }
    }
}

// The ranges' sums of a split product.
template <int OP>
__global__ __launch_bounds__(256) void product_join_kernel(const ProductArgs a) {
    const int64_t at = flat_block() * 256 + threadIdx.x, size = (int64_t)a.m * a.n;
    if (at >= size) return;
    int sum = 0;
    for (int s = 0; s < a.split; ++s) sum += a.part[s * size + at];
    const int i = (int)(at / a.n), j = (int)(at - (int64_t)i * a.n);
    put<OP>(a, i, j, sum, a.scale_w[j], a.bias ? a.bias[j] : 0.f);
}

template <int OP, int BM, int BN, int WM, int WN>
hipError_t tiles(const ProductArgs& a, hipStream_t s) {
    using L = Tile<BM, BN, WM, WN>;
    const int64_t count = ((int64_t)a.m + BM - 1) / BM * (((int64_t)a.n + BN - 1) / BN);
    const dim3 grid((unsigned)count, (unsigned)a.split);
    if (a.aligned)
        product_kernel<OP, BM, BN, WM, WN, true><<<grid, L::kThreads, 2 * L::kStage, s>>>(a);
    else if constexpr (BM <= 128)
        product_kernel<OP, BM, BN, WM, WN, false><<<grid, L::kThreads, 2 * L::kStage, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.split == 1) return e;
    product_join_kernel<OP><<<flat_grid(((int64_t)a.m * a.n + 255) / 256), 256, 0, s>>>(a);
    return hipGetLastError();
}

constexpr int kFewRows = 64;

int tile_of(int m, int n) {
    const auto count = [&](int64_t b) { return (m + b - 1) / b * ((n + b - 1) / b); };
    if (count(256) >= 192) return 256;
    if (count(128) >= 192) return 128;
    return 64;
}

template <int OP>
hipError_t product(const ProductArgs& a, hipStream_t s) {
    if (a.m <= kFewRows) {
        const unsigned g = (unsigned)((a.n + 15) / 16);
        if (a.m <= 16)
            product_rows_kernel<OP, 1><<<g, 256, 0, s>>>(a);
        else if (a.m <= 32)
            product_rows_kernel<OP, 2><<<g, 256, 0, s>>>(a);
        else
            product_rows_kernel<OP, 4><<<g, 256, 0, s>>>(a);
        return hipGetLastError();
    }
    const int t = tile_of(a.m, a.n);
    if (t == 256 && a.aligned) return tiles<OP, 256, 256, 2, 4>(a, s);
    if (t >= 128) return tiles<OP, 128, 128, 2, 2>(a, s);
    return tiles<OP, 64, 64, 2, 2>(a, s);
}

}  // namespace

int product_split(int m, int n, int k, int* split_k) {
    *split_k = k > 0 ? k : 1;
    if (m <= kFewRows || n <= 0) return 1;
    const int64_t t = tile_of(m, n), count = (m + t - 1) / t * ((n + t - 1) / t);
    if (t > 64 || count >= 128) return 1;
    const int64_t s = std::min<int64_t>(std::min<int64_t>(256 / count, k / 1024), 16);
    if (s <= 1) return 1;
    *split_k = (int)(((k + s - 1) / s + 127) / 128 * 128);
    return (k + *split_k - 1) / *split_k;
}

hipError_t launch_quantize(const QuantArgs& a, hipStream_t s) {
    return a.op == OP_BF16 ? quantize<OP_BF16>(a, s)
           : a.op == OP_F16 ? quantize<OP_F16>(a, s)
                            : quantize<OP_F32>(a, s);
}

hipError_t launch_product(const ProductArgs& a, hipStream_t s) {
    return a.op == OP_BF16 ? product<OP_BF16>(a, s)
           : a.op == OP_F16 ? product<OP_F16>(a, s)
                            : product<OP_F32>(a, s);
}

}  // namespace fs
