// fs_quant.hip -- rows held in 8-bit integers with a scale each, and the product
// of two such sets:
//   a = max |x|, q = 127 x / a to the nearest whole number, scale = a / 127;
//   y_ij = scale_i scale'_j sum_k q_ik q'_jk + b_j, the sum exact in 32 bits.
// (8192 rows of 8192, bf16: 45 to 50 us for 201 MB, 4.0 to 4.5 TB/s; the product of two
// such sets 503 to 547 us, 2010 to 2190 TOP/s, where the library's 8-bit product took 515
// to 547 on the same cards; 8 rows against 8192 of 4096, 9 us for 34 MB.)
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

// Bound by memory: a row is read once and stays in registers over its maximum.
template <int OP, int LPR, int CH, bool WIDE_ROWS>
__global__ __launch_bounds__(threads_of<LPR>()) void quantize_kernel(const QuantArgs a) {
    using T = typename El<OP>::T;
    constexpr int GRP = threads_of<LPR>() / LPR;
    __shared__ float2 buf[2 * RowFold<LPR>::kWaves];
    RowFold<LPR> fold(buf);
    const int lane = threadIdx.x % LPR, W = a.width;
    const int64_t row = flat_block() * GRP + threadIdx.x / LPR;
    if (row >= a.rows) return;  // (LPR > 64: the whole workgroup)
    Share<T, LPR, CH, WIDE_ROWS ? WIDE : SINGLE> x;
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
        if constexpr (WIDE_ROWS) {
            const int at = share_at<LPR, WIDE>(lane, j, 0);
            if (at < W) __builtin_memcpy(__builtin_assume_aligned(q + at, 8), out, 8);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int at = share_at<LPR, SINGLE>(lane, j, e);
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

template <int OP>
__device__ __forceinline__ void put(const ProductArgs& a, int i, int j, int sum, float sw, float bias) {
    using T = typename El<OP>::T;
    ((T*)a.y)[i * a.sy + j] = (T)fmaf((float)sum * a.scale_x[i], sw, bias);
}

// Sixteen bytes of a row from k on.  Rows that start at a whole dword (DWORDS) are
// read as they stand; else five dwords are read from the one on that holds the
// first byte, and shifted (16-byte loads of any address take four times as long).
// A dword that is read holds a byte of the row.
template <bool DWORDS>
struct Bytes {
    const int8_t* p;
    uint32_t shift;  // bytes, 0..3
    __device__ __forceinline__ Bytes(const int8_t* row) : p(row), shift(0) {
        if constexpr (!DWORDS) {
            shift = (uint32_t)(uintptr_t)row & 3;
            p = row - shift;
        }
    }
    struct Raw {
        uint32_t w[DWORDS ? 4 : 5];
    };
    __device__ __forceinline__ void read(int k, Raw& r) const {
        __builtin_memcpy(r.w, __builtin_assume_aligned(p + k, 4), 16);
        if constexpr (!DWORDS)
            __builtin_memcpy(r.w + 4, __builtin_assume_aligned(p + k + (shift ? 16 : 12), 4), 4);
    }
    __device__ __forceinline__ i32x4 value(const Raw& r) const {
        i32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = DWORDS ? (int)r.w[i] : (int)__builtin_amdgcn_alignbyte(r.w[i + 1], r.w[i], shift);
        return v;
    }
    // from k on, zeros from `end` on
    __device__ __forceinline__ i32x4 tail(int k, int end) const {
        int8_t t[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) t[i] = k + i < end ? p[shift + k + i] : (int8_t)0;
        i32x4 v;
        __builtin_memcpy(&v, t, 16);
        return v;
    }
};

// Few rows: a workgroup takes 16 CB columns and all rows (RB blocks of 16), its
// eight waves divide k.  Bound by the read of the columns' bytes.
constexpr int kRowWaves = 8;
template <int OP, int RB, int CB, bool DWORDS>
__global__ __launch_bounds__(64 * kRowWaves) void product_rows_kernel(const ProductArgs a) {
    constexpr int N = RB * CB * 256;
    __shared__ int red[kRowWaves][N];
    const int lane = threadIdx.x & 63, wave = wave_id(), r = lane & 15, c = lane >> 4;
    const int j0 = blockIdx.x * 16 * CB;
    using Row = Bytes<DWORDS>;
    const auto column = [&](int b) { return Row(a.w + (int64_t)min(j0 + 16 * b + r, a.n - 1) * a.sw); };
    const auto state = [&](int b) { return Row(a.x + (int64_t)min(16 * b + r, a.m - 1) * a.sx); };
    i32x4 acc[CB][RB] = {};
    // whole steps of 64 k: reads that ask nothing, U of them under way together
    constexpr int U = RB * CB <= 2 ? 8 : 2;
    const int whole = a.k / 64;
    int t = wave;
    for (; t + kRowWaves * (U - 1) < whole; t += kRowWaves * U) {
        typename Row::Raw wv[U][CB], xv[U][RB];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (t + kRowWaves * u) * 64 + c * 16;
#pragma unroll
            for (int b = 0; b < CB; ++b) column(b).read(k, wv[u][b]);
#pragma unroll
            for (int b = 0; b < RB; ++b) state(b).read(k, xv[u][b]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int q = 0; q < CB; ++q)
#pragma unroll
                for (int b = 0; b < RB; ++b)
                    acc[q][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                        state(b).value(xv[u][b]), column(q).value(wv[u][q]), acc[q][b], 0, 0, 0);
    }
    for (; t < (a.k + 63) / 64; t += kRowWaves) {
        const int k = t * 64 + c * 16;
        i32x4 wv[CB], xv[RB];
        if (t < whole) {
            typename Row::Raw raw;
#pragma unroll
            for (int b = 0; b < CB; ++b) column(b).read(k, raw), wv[b] = column(b).value(raw);
#pragma unroll
            for (int b = 0; b < RB; ++b) state(b).read(k, raw), xv[b] = state(b).value(raw);
        } else {
#pragma unroll
            for (int b = 0; b < CB; ++b) wv[b] = column(b).tail(k, a.k);
#pragma unroll
            for (int b = 0; b < RB; ++b) xv[b] = state(b).tail(k, a.k);
        }
#pragma unroll
        for (int q = 0; q < CB; ++q)
#pragma unroll
            for (int b = 0; b < RB; ++b)
                acc[q][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(xv[b], wv[q], acc[q][b], 0, 0, 0);
    }
    // a lane holds column r, rows 4 c .. 4 c + 3 of each block
#pragma unroll
    for (int q = 0; q < CB; ++q)
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                red[wave][((b * 16 + 4 * c + e) * CB + q) * 16 + r] = acc[q][b][e];
    __syncthreads();
    for (int p = threadIdx.x; p < N; p += 64 * kRowWaves) {
        const int i = p / (16 * CB), j = j0 + p % (16 * CB);
        int sum = 0;
#pragma unroll
        for (int w = 0; w < kRowWaves; ++w) sum += red[w][p];
        if (i < a.m && j < a.n) put<OP>(a, i, j, sum, a.scale_w[j], a.bias ? a.bias[j] : 0.f);
    }
}

// Rows that the tiles cannot copy as they are, laid out with a stride of whole 16
// bytes and zeros behind their end: a thread writes 16 bytes (blockIdx.z: x, w).
__global__ __launch_bounds__(256) void product_pack_kernel(const ProductArgs a) {
    const bool left = blockIdx.z == 0;
    int8_t* to = left ? a.pack_x : a.pack_w;
    if (!to) return;
    const int chunks = (a.k + 15) / 16;
    const int64_t at = flat_block() * 256 + threadIdx.x;
    const int64_t row = at / chunks;
    if (row >= (left ? a.m : a.n)) return;
    const int c = (int)(at - row * chunks) * 16;
    const Bytes<false> src(left ? a.x + row * a.sx : a.w + row * a.sw);
    i32x4 v;
    if (c + 16 <= a.k) {
        Bytes<false>::Raw raw;
        src.read(c, raw);
        v = src.value(raw);
    } else {
        v = src.tail(c, a.k);
    }
    *(i32x4*)(to + at * 16) = v;
}

// Tiles of BM x BN outputs over steps of 128 k, in STAGES buffers of LDS (2 for tiles of
// 256, 2 or 4 for 128, 5 for 64): while the matrix units work on one, the rows of the next
// STAGES - 1 steps are on their way.
// The 16-byte chunks of a row of 128 bytes stand in an order that depends on its
// number, so that 16 lanes reading one chunk of 16 rows use all banks.  WM x WN
// waves.  Bound, for tiles of 256, by the matrix units at the clock that is left: at
// 8192^3 their pipes are busy in half of the cycles, at 1.9 GHz, and LDS serves its
// 128 bytes a cycle for nearly as long (eight waves of 128 x 64 read 192 KB a step of
// 2048 cycles and 64 KB come in; four of 128 x 128, which read 128 KB, have nobody to
// hide their waits: 577 us against 524).
template <int BM, int BN, int WM, int WN, int STAGES>
struct Tile {
    static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
    static constexpr int MI = BM / WM / 32, NI = BN / WN / 32;
    static constexpr int kStage = (BM + BN) * 128;
    static constexpr int kStages = STAGES;
};
__device__ __forceinline__ uint32_t chunk_at(int row, int chunk) {
    return row * 128 + ((chunk ^ (row >> 1)) & 7) * 16;
}

template <int OP, int BM, int BN, int WM, int WN, int STAGES>
__global__ __launch_bounds__(64 * WM * WN) void product_kernel(const ProductArgs a) {
    using L = Tile<BM, BN, WM, WN, STAGES>;
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
    // chunk c of a wave's copies covers 8 rows of the tiles, x's first; rows behind
    // the last are the last one once more
    uint32_t voff[kCopies];
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
        const int t = (wave * kCopies + c) * 8 + (lane >> 3);
        const uint32_t row = t < BM ? min(t, a.m - 1 - i0) : min(t - BM, a.n - 1 - j0);
        voff[c] = row * (uint32_t)(t < BM ? a.sx : a.sw) + ((lane ^ (t >> 1)) & 7) * 16;
    }
    // a quarter of a step's copies
    const auto copy = [&](int t, int buffer, int quarter) {
        const int k = k0 + t * 128;
#pragma unroll
        for (int c = quarter * (kCopies / 4); c < (quarter + 1) * (kCopies / 4); ++c) {
            const bool left = (wave * kCopies + c) * 8 < BM;
            const int8_t* from = (left ? a.x + (int64_t)i0 * a.sx : a.w + (int64_t)j0 * a.sw) + k;
            uint32_t at = voff[c];
            if (k + 128 > k1) {
                // chunks behind the end: the row's first ones, which the products leave out
                const uint32_t chunk = (lane ^ (((wave * kCopies + c) * 8 + (lane >> 3)) >> 1)) & 7;
                at -= k + (int)chunk * 16 < k1 ? 0 : chunk * 16;
            }
            dma_to_lds16((const char*)from, at,
                         lds + buffer * L::kStage + (wave * kCopies + c) * 1024);
        }
    };
    const int wm = wave / WN, wn = wave % WN;
    const int ra = wm * MI * 32 + (lane & 31), rb = BM + wn * NI * 32 + (lane & 31);
    i32x16 acc[MI][NI] = {};
    constexpr int AHEAD = L::kStages - 1;
    const auto work = [&](int t, int buffer, bool tail) {
        const uint32_t at = base + buffer * L::kStage;
        const int left = k1 - k0 - t * 128, next = buffer == 0 ? AHEAD : buffer - 1;
        // operands of the next 32 k are read, and a quarter of a later step's rows
        // sent for, while this one's products run
        i32x4 x[2][MI], w[2][NI];
        const auto read = [&](int kk) {
            const int chunk = 2 * kk + (lane >> 5);
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                x[kk & 1][i] = lds_read<i32x4>(at + chunk_at(ra + 32 * i, chunk));
                if (tail && chunk * 16 >= left) x[kk & 1][i] = i32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int j = 0; j < NI; ++j)
                w[kk & 1][j] = lds_read<i32x4>(at + chunk_at(rb + 32 * j, chunk));
        };
        read(0);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            if (kk < 3) read(kk + 1);
            if (!tail && t + AHEAD < steps) copy(t + AHEAD, next, kk);
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(x[kk & 1][i], w[kk & 1][j],
                                                                      acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    const int whole = (k1 - k0) / 128;
    for (int t = 0; t < AHEAD && t < steps; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) copy(t, t, q);
    int buffer = 0;
    const auto ready = [&](int t) {
        // this step's rows are there, and nobody reads the buffer before it any more
        if (AHEAD > 1 && t + AHEAD - 1 < steps)
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"((AHEAD - 1) * kCopies) : "memory");
        else
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        stage_barrier();
    };
    for (int t = 0; t < whole; ++t) {
        ready(t);
        work(t, buffer, false);
        buffer = buffer == AHEAD ? 0 : buffer + 1;
    }
    if (whole < steps) {
        ready(whole);
        work(whole, buffer, true);
    }
    constexpr int NC = NI * 32, PITCH = NC + 4, LANES = NC / 8, ROWS = 64 / LANES;
    static_assert(L::kWaves * 32 * PITCH * 4 <= L::kStages * L::kStage, "the sums' LDS");
    const uint32_t mine = base + wave * 32 * PITCH * 4;
    const int h = lane >> 5;
    if (!a.y_wide || a.split > 1) {
        // ranges' sums and rows of any width: single elements, neighbours by lane
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            const int col = j0 + wn * NC + 32 * j + (lane & 31);
            if (col >= a.n) continue;
            const float sw = a.scale_w[col], bias = a.bias ? a.bias[col] : 0.f;
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                __builtin_amdgcn_sched_barrier(0);  // (64 rows' places at a time would not fit)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int row = i0 + (wm * MI + i) * 32 + 8 * (r >> 2) + 4 * h + (r & 3);
                    if (row >= a.m) continue;
                    if (a.split > 1)
                        a.part[((int64_t)blockIdx.y * a.m + row) * a.n + col] = acc[i][j][r];
                    else
                        put<OP>(a, row, col, acc[i][j][r], sw, bias);
                }
            }
        }
        return;
    }
    // The sums, 32 rows of the wave's columns at a time, go through LDS, so that a lane
    // has eight neighbours of one row (a 16-byte store of a 16-bit type; single
    // elements took as long as eight steps of k).
    stage_barrier();  // the last step's operands are read
    const int c8 = lane % LANES * 8, col = j0 + wn * NC + c8;
    float sw[8], bias[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int j = min(col + e, a.n - 1);
        sw[e] = a.scale_w[j];
        bias[e] = a.bias ? a.bias[j] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                lds_write<int>(mine + ((8 * (r >> 2) + 4 * h + (r & 3)) * PITCH + 32 * j + (lane & 31)) * 4,
                               acc[i][j][r]);
        asm volatile("" ::: "memory");  // (a wave's LDS operations run in order)
#pragma unroll
        for (int q = 0; q < 32; q += ROWS) {
            using T = typename El<OP>::T;
            const int at = q + lane / LANES, row = i0 + (wm * MI + i) * 32 + at;
            i32x4 v[2];
            v[0] = lds_read<i32x4>(mine + (at * PITCH + c8) * 4);
            v[1] = lds_read<i32x4>(mine + (at * PITCH + c8 + 4) * 4);
            if (row >= a.m || col >= a.n) continue;
            const float sx = a.scale_x[row];
            T out[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) out[e] = (T)fmaf((float)v[e >> 2][e & 3] * sx, sw[e], bias[e]);
            __builtin_memcpy(__builtin_assume_aligned((T*)a.y + row * a.sy + col, 16), out, sizeof(out));
        }
        asm volatile("" ::: "memory");
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

template <int OP, int BM, int BN, int WM, int WN, int STAGES>
hipError_t tiles(const ProductArgs& a, hipStream_t s) {
    using L = Tile<BM, BN, WM, WN, STAGES>;
    const int64_t count = ((int64_t)a.m + BM - 1) / BM * (((int64_t)a.n + BN - 1) / BN);
    const dim3 grid((unsigned)count, (unsigned)a.split);
    product_kernel<OP, BM, BN, WM, WN, STAGES><<<grid, L::kThreads, L::kStages * L::kStage, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.split == 1) return e;
    product_join_kernel<OP><<<flat_grid(((int64_t)a.m * a.n + 255) / 256), 256, 0, s>>>(a);
    return hipGetLastError();
}

constexpr int kFewRows = 32;

int64_t tiles_of(int m, int n, int64_t b) { return (m + b - 1) / b * ((n + b - 1) / b); }

// The largest tiles (fewest bytes through LDS for a product) that still fill the
// chip: 4096 x 4096 x 4096 in tiles of 256 / 128, us, 68 / 83; 2048 x 4096 x 4096, 128
// workgroups of tiles of 256, 62 / 48.
int tile_of(int m, int n) {
    return tiles_of(m, n, 256) >= 192 ? 256 : tiles_of(m, n, 128) >= 192 ? 128 : 64;
}

// Two blocks of columns a workgroup where that leaves 256 workgroups: the rows' bytes,
// which each of them reads anew from L2, count as the columns' do (us, one / two: 16
// x 8192 x 4096, 10.9 / 9.9; 8 x 32768 x 4096, 34.9 / 32.5; 32 x 32768 x 4096, 53.9 /
// 42.1; but 1 x 32768 x 4096, 29.9 / 31.7, 8 x 4096 x 16384, 17.8 / 25.0, and 32 x 4096 x
// 4096, 8.7 / 9.8).
template <int OP, bool DWORDS>
hipError_t rows(const ProductArgs& a, hipStream_t s) {
    constexpr int T = 64 * kRowWaves;
    const unsigned one = (unsigned)((a.n + 15) / 16), two = (unsigned)((a.n + 31) / 32);
    const bool wide = a.n >= 8192 && a.m > 4;
    if (a.m <= 16 && wide)
        product_rows_kernel<OP, 1, 2, DWORDS><<<two, T, 0, s>>>(a);
    else if (a.m <= 16)
        product_rows_kernel<OP, 1, 1, DWORDS><<<one, T, 0, s>>>(a);
    else if (wide)
        product_rows_kernel<OP, 2, 2, DWORDS><<<two, T, 0, s>>>(a);
    else
        product_rows_kernel<OP, 2, 1, DWORDS><<<one, T, 0, s>>>(a);
    return hipGetLastError();
}

template <int OP>
hipError_t product(const ProductArgs& a, hipStream_t s) {
    if (a.m <= kFewRows) return a.dwords ? rows<OP, true>(a, s) : rows<OP, false>(a, s);
    ProductArgs b = a;
    if (a.pack_x || a.pack_w) {
        const int chunks = (a.k + 15) / 16;
        const int most = std::max(a.pack_x ? a.m : 0, a.pack_w ? a.n : 0);
        dim3 grid = flat_grid(((int64_t)most * chunks + 255) / 256);
        grid.z = a.pack_w ? 2 : 1;
        product_pack_kernel<<<grid, 256, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        if (a.pack_x) b.x = a.pack_x, b.sx = 16 * chunks;
        if (a.pack_w) b.w = a.pack_w, b.sw = 16 * chunks;
        b.k = 16 * chunks;  // (k is whole chunks, or both are packed with zeros)
    }
    const int t = tile_of(a.m, a.n);
    if (t == 256) return tiles<OP, 256, 256, 2, 4, 2>(b, s);
    // one workgroup a CU has all of LDS for rows on their way (1024 x 4096 x 4096: 27 us
    // with four buffers, 32 with two; with more workgroups two of them share a CU: 2048
    // x 4096 x 4096, 55 / 48)
    if (t == 128 && tiles_of(a.m, a.n, 128) <= 256) return tiles<OP, 128, 128, 2, 4, 4>(b, s);
    if (t == 128) return tiles<OP, 128, 128, 2, 4, 2>(b, s);
    return tiles<OP, 64, 64, 2, 2, 5>(b, s);
}

}  // namespace

bool product_few(int m) { return m <= kFewRows; }

int product_split(int m, int n, int k, int* split_k) {
    k = (k + 15) / 16 * 16;
    *split_k = k > 0 ? k : 1;
    if (m <= kFewRows || n <= 0) return 1;
    const int64_t count = tiles_of(m, n, 64);
    if (tile_of(m, n) > 64 || count >= 128) return 1;
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
