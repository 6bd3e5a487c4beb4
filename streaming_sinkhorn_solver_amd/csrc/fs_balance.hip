// fs_balance.hip -- the k largest columns of each row of logits, how often each
// column is chosen, the balance loss and its gradient:
//   p = softmax(x), f_e = c_e / (k N), P_e = mean p_e:
//   L0 = E sum f P, L1 = mean lse^2, gates = p of the chosen (over their sum S);
//   dp_e = dL0 E f_e / N + sum_{id = e} (dgate - (sum dgate gate)) / S,
//   dx = p (dp - sum p dp + dL1 2 lse / N).
// A row's columns lie with LPT lanes, neighbours with one lane, so that the lowest
// of equal columns is the first of the lowest lane.  Sums over columns run in the
// lanes' registers over a workgroup's rows, then over workgroups in a second
// launch (in 64 bits, in a fixed order).
#include "fs_layers_args.h"
#include "fs_rowops.hpp"

#include <algorithm>

namespace fs {

namespace {

constexpr int kThreads = 256;

// Order of floats as that of whole numbers; NaN counts as -inf, -0 as 0.  No
// float's key is 0, which stands for a column that is chosen already.
__device__ __forceinline__ uint32_t key_of(float x) {
    x = x == x ? x + 0.f : -INFINITY;
    const uint32_t b = __float_as_uint(x);
    return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key ^ (key & 0x80000000u ? 0x80000000u : 0xffffffffu));
}

template <typename T, int EPL, bool WIDE>
__device__ __forceinline__ void load_columns(const T* row, int e0, int E, bool on, T (&v)[EPL]) {
    if constexpr (WIDE) {
#pragma unroll
        for (int j = 0; j < EPL; j += 8) {
            if (on && e0 + j < E)
                __builtin_memcpy(v + j, __builtin_assume_aligned(row + e0 + j, 16), 8 * sizeof(T));
            else
#pragma unroll
                for (int e = 0; e < 8; ++e) v[j + e] = (T)-INFINITY;
        }
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) v[j] = on && e0 + j < E ? row[e0 + j] : (T)-INFINITY;
    }
}

// Totals of a batch entry -> loss, from columns' sums of p and counts that the
// workgroup's threads each give for their columns.
struct LossSum {
    double terms, squares, rows;
    __device__ __forceinline__ void write(const BalanceArgs& a, int b) const {
        const double n = rows;
        a.loss[2 * b] = n > 0 ? (float)(a.E * terms / (a.k * n * n)) : 0.f;
        a.loss[2 * b + 1] = n > 0 ? (float)(squares / n) : 0.f;
    }
};

template <int OP, int LPT, int EPL, int KMAX, bool WIDE>
__global__ __launch_bounds__(kThreads) void balance_kernel(const BalanceArgs a) {
    using T = typename El<OP>::T;
    constexpr int GRP = kThreads / LPT, COLS = LPT * EPL;
    __shared__ float red_p[4][COLS];
    __shared__ int red_c[4][COLS];
    __shared__ float2 red_s[4];
    __shared__ double red_t[4];
    const int lane = threadIdx.x & 63, part = lane % LPT, e0 = part * EPL, b = blockIdx.y, E = a.E;
    const int size = a.lengths ? max(0, min(a.n, a.lengths[b])) : a.n;
    float sum_p[EPL] = {}, squares = 0.f, count = 0.f;
    int hits[EPL] = {};
    for (int64_t first = (int64_t)blockIdx.x * GRP; first < a.n; first += (int64_t)gridDim.x * GRP) {
        const int64_t i = first + threadIdx.x / LPT;
        if (i >= a.n) break;
        const int64_t row = (int64_t)b * a.n + i;
        T v[EPL];
        load_columns<T, EPL, WIDE>((const T*)a.x.p + b * a.x.sb + i * a.x.sr, e0, E, i < size, v);
        uint32_t key[EPL];
        float x[EPL], top = -INFINITY;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            x[j] = (float)v[j];
            key[j] = e0 + j < E ? key_of(x[j]) : 0u;
            top = fmaxf(top, x[j]);
        }
        top = lanes_max<LPT>(top);
        const bool on = top != -INFINITY;
        const float ref = on ? top : 0.f;
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) s += x[j] = on ? ex2((x[j] - ref) * kLog2e) : 0.f;
        s = lanes_sum<LPT>(s);
        const float inv = on ? 1.f / s : 0.f, lse = on ? ref + logf(s) : 0.f;
        // the largest that is left, k times
        int ids[KMAX];
        float gate[KMAX], all = 0.f;
#pragma unroll
        for (int t = 0; t < KMAX; ++t) {
            ids[t] = -1;
            gate[t] = 0.f;
            if (t >= a.k) continue;
            uint32_t best = 0;
#pragma unroll
            for (int j = 0; j < EPL; ++j) best = max(best, key[j]);
            const uint32_t most = lanes_max<LPT>(best);
            const uint64_t have = __ballot(best == most) >> (lane - part);
            const int from = __builtin_ctzll(have);
            int at = 0;
#pragma unroll
            for (int j = EPL - 1; j >= 0; --j) at = key[j] == most ? j : at;
            if (part == from && on) {
#pragma unroll
                for (int j = 0; j < EPL; ++j)
                    if (j == at) key[j] = 0u, hits[j] += 1;
            }
            const int id = __shfl(e0 + at, lane - part + from, 64);
            gate[t] = on ? ex2((value_of(most) - ref) * kLog2e) * inv : 0.f;
            ids[t] = on ? id : -1;
            all += gate[t];
        }
        const float scale = a.normalize && on ? 1.f / all : 1.f;
#pragma unroll
        for (int t = 0; t < KMAX; ++t)
            if (t < a.k && t % LPT == part) {
                a.ids[row * a.k + t] = ids[t];
                a.gates[row * a.k + t] = gate[t] * scale;
            }
        if (part == 0) {
            a.lse[row] = lse;
            squares = fmaf(lse, lse, squares);
            count += on ? 1.f : 0.f;
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j) sum_p[j] = fmaf(x[j], inv, sum_p[j]);
    }
    // over the rows of a wave, then of the workgroup
#pragma unroll
    for (int o = LPT; o < 64; o <<= 1) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            sum_p[j] += __shfl_xor(sum_p[j], o, 64);
            hits[j] += __shfl_xor(hits[j], o, 64);
        }
        squares += __shfl_xor(squares, o, 64);
        count += __shfl_xor(count, o, 64);
    }
    const int wave = threadIdx.x >> 6;
    if (lane < LPT) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) red_p[wave][e0 + j] = sum_p[j], red_c[wave][e0 + j] = hits[j];
    }
    if (lane == 0) red_s[wave] = make_float2(squares, count);
    __syncthreads();
    const int64_t at = (int64_t)b * a.blocks + blockIdx.x;
    double terms = 0.0;
    for (int e = threadIdx.x; e < E; e += kThreads) {
        const float p = red_p[0][e] + red_p[1][e] + red_p[2][e] + red_p[3][e];
        const int c = red_c[0][e] + red_c[1][e] + red_c[2][e] + red_c[3][e];
        if (a.blocks == 1) {
            a.counts[(int64_t)b * E + e] = c;
            terms += (double)c * p;
        } else {
            a.part_p[at * E + e] = p;
            a.part_c[at * E + e] = c;
        }
    }
    const float sq = red_s[0].x + red_s[1].x + red_s[2].x + red_s[3].x;
    const float rows = red_s[0].y + red_s[1].y + red_s[2].y + red_s[3].y;
    if (a.blocks > 1) {
        if (threadIdx.x == 0) a.part_s[at] = make_float2(sq, rows);
        return;
    }
    for (int o = 32; o >= 1; o >>= 1) terms += __shfl_xor(terms, o, 64);
    if (lane == 0) red_t[wave] = terms;
    __syncthreads();
    if (threadIdx.x == 0)
        LossSum{red_t[0] + red_t[1] + red_t[2] + red_t[3], sq, rows}.write(a, b);
}

// The workgroups' sums of one batch entry: 64 columns at a time, 16 lanes each.
__global__ __launch_bounds__(1024) void balance_join_kernel(const BalanceArgs a) {
    __shared__ double red_p[16][64];
    __shared__ int red_c[16][64];
    const int b = blockIdx.x, c = threadIdx.x & 63, y = threadIdx.x >> 6;
    double terms = 0.0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
        double p = 0.0;
        int n = 0;
        if (e0 + c < a.E) {
#pragma unroll 4
            for (int k = y; k < a.blocks; k += 16) {
                const int64_t at = ((int64_t)b * a.blocks + k) * a.E + e0 + c;
                p += (double)a.part_p[at];
                n += a.part_c[at];
            }
        }
        red_p[y][c] = p;
        red_c[y][c] = n;
        __syncthreads();
        if (y == 0) {
#pragma unroll
            for (int k = 1; k < 16; ++k) p += red_p[k][c], n += red_c[k][c];
            if (e0 + c < a.E) a.counts[(int64_t)b * a.E + e0 + c] = n;
            terms += (double)n * p;
        }
        __syncthreads();
    }
    if (y) return;
    double squares = 0.0, rows = 0.0;
    for (int k = c; k < a.blocks; k += 64) {
        const float2 s = a.part_s[(int64_t)b * a.blocks + k];
        squares += (double)s.x;
        rows += (double)s.y;
    }
    for (int o = 32; o >= 1; o >>= 1) {
        terms += __shfl_xor(terms, o, 64);
        squares += __shfl_xor(squares, o, 64);
        rows += __shfl_xor(rows, o, 64);
    }
    if (c == 0) LossSum{terms, squares, rows}.write(a, b);
}

template <int OP, int LPT, int EPL, bool WIDE>
__global__ __launch_bounds__(kThreads) void balance_bwd_kernel(const BalanceArgs a) {
    using T = typename El<OP>::T;
    constexpr int GRP = kThreads / LPT;
    const int lane = threadIdx.x & 63, part = lane % LPT, e0 = part * EPL, b = blockIdx.y, E = a.E;
    const int size = a.lengths ? max(0, min(a.n, a.lengths[b])) : a.n;
    // what every row's probabilities are worth to the balance: E c_e / (k N^2)
    float even[EPL];
    uint32_t sum = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int c = e0 + j < E ? a.counts[(int64_t)b * E + e0 + j] : 0;
        even[j] = (float)c;
        sum += (uint32_t)c;
    }
    sum = lanes_fold<LPT>(sum, [](uint32_t x, uint32_t y) { return x + y; });
    const float n = (float)sum / (float)a.k, inv_n = sum ? 1.f / n : 0.f;
    const float balance = a.gloss[2 * b] * (float)E * inv_n * inv_n / (float)a.k;
    const float square = 2.f * a.gloss[2 * b + 1] * inv_n;
#pragma unroll
    for (int j = 0; j < EPL; ++j) even[j] *= balance;
    for (int64_t first = (int64_t)blockIdx.x * GRP; first < a.n; first += (int64_t)gridDim.x * GRP) {
        const int64_t i = first + threadIdx.x / LPT;
        if (i >= a.n) break;
        const int64_t row = (int64_t)b * a.n + i;
        const int* ids = a.ids + row * a.k;
        const bool on = i < size && ids[0] >= 0;
        const float lse = on ? a.lse[row] : 0.f;
        T v[EPL];
        load_columns<T, EPL, WIDE>((const T*)a.x.p + b * a.x.sb + i * a.x.sr, e0, E, on, v);
        float p[EPL], dp[EPL], chosen = 0.f, worth = 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            p[j] = ex2(((float)v[j] - lse) * kLog2e);
            dp[j] = even[j];
        }
        if (a.ggates && on) {
            float dg[EPL] = {}, times[EPL] = {};
            for (int t = 0; t < a.k; ++t) {
                const int at = ids[t] - e0;
                const float g = a.ggates[row * a.k + t];
#pragma unroll
                for (int j = 0; j < EPL; ++j)
                    if (at == j) dg[j] += g, times[j] += 1.f;
            }
            float shift = 0.f, scale = 1.f;
            if (a.normalize) {
#pragma unroll
                for (int j = 0; j < EPL; ++j) {
                    chosen = fmaf(p[j], times[j], chosen);
                    worth = fmaf(p[j], dg[j], worth);
                }
                chosen = lanes_sum<LPT>(chosen);
                worth = lanes_sum<LPT>(worth);
                scale = chosen > 0.f ? 1.f / chosen : 0.f;
                shift = worth * scale;
            }
#pragma unroll
            for (int j = 0; j < EPL; ++j) dp[j] = fmaf(dg[j] - times[j] * shift, scale, dp[j]);
        }
        float mean = 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) mean = fmaf(p[j], dp[j], mean);
        mean = lanes_sum<LPT>(mean) - square * lse;
        T* gx = (T*)a.gx.p + b * a.gx.sb + i * a.gx.sr;
#pragma unroll
        for (int j = 0; j < EPL; ++j) v[j] = (T)(on ? p[j] * (dp[j] - mean) : 0.f);
        if constexpr (WIDE) {
#pragma unroll
            for (int j = 0; j < EPL; j += 8)
                if (e0 + j < E)
                    __builtin_memcpy(__builtin_assume_aligned(gx + e0 + j, 16), v + j, 8 * sizeof(T));
        } else {
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                if (e0 + j < E) gx[e0 + j] = v[j];
        }
    }
}

template <int OP, int LPT, int EPL, bool WIDE>
hipError_t go(const BalanceArgs& a, bool back, hipStream_t s) {
    const dim3 grid((unsigned)a.blocks, (unsigned)a.B);
    if (back)
        balance_bwd_kernel<OP, LPT, EPL, WIDE><<<grid, kThreads, 0, s>>>(a);
    else if (a.k <= 8)
        balance_kernel<OP, LPT, EPL, 8, WIDE><<<grid, kThreads, 0, s>>>(a);
    else
        balance_kernel<OP, LPT, EPL, kBalanceMaxTop, WIDE><<<grid, kThreads, 0, s>>>(a);
    return hipGetLastError();
}
template <int OP, int LPT, int EPL>
hipError_t go(const BalanceArgs& a, bool back, hipStream_t s) {
    return a.wide ? go<OP, LPT, EPL, true>(a, back, s) : go<OP, LPT, EPL, false>(a, back, s);
}
template <int OP>
hipError_t go(const BalanceArgs& a, bool back, hipStream_t s) {
    if (a.E <= 8) return go<OP, 1, 8>(a, back, s);
    if (a.E <= 16) return go<OP, 2, 8>(a, back, s);
    if (a.E <= 32) return go<OP, 4, 8>(a, back, s);
    if (a.E <= 64) return go<OP, 8, 8>(a, back, s);
    if (a.E <= 128) return go<OP, 16, 8>(a, back, s);
    if (a.E <= 256) return go<OP, 32, 8>(a, back, s);
    if (a.E <= 512) return go<OP, 64, 8>(a, back, s);
    return go<OP, 64, 16>(a, back, s);
}
hipError_t go(const BalanceArgs& a, bool back, hipStream_t s) {
    return a.op == OP_BF16 ? go<OP_BF16>(a, back, s)
           : a.op == OP_F16 ? go<OP_F16>(a, back, s)
                            : go<OP_F32>(a, back, s);
}

int rows_at_once(int E) {
    int lanes = 1;
    while (lanes < 64 && lanes * 8 < E) lanes *= 2;
    return kThreads / lanes;
}

}  // namespace

// Workgroups of a batch entry: two turns of rows each, 512 in all at most.
int balance_blocks(int B, int n, int E) {
    const int64_t turns = ((int64_t)n + rows_at_once(E) - 1) / rows_at_once(E);
    const int64_t most = std::max<int64_t>(1, 512 / std::max(B, 1));
    return (int)std::max<int64_t>(1, std::min<int64_t>((turns + 1) / 2, most));
}

hipError_t launch_balance(const BalanceArgs& a, hipStream_t s) {
    const hipError_t e = go(a, false, s);
    if (e != hipSuccess || a.blocks == 1) return e;
    balance_join_kernel<<<(unsigned)a.B, 1024, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_balance_bwd(const BalanceArgs& a, hipStream_t s) { return go(a, true, s); }

}  // namespace fs
