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
#include <type_traits>

namespace fs {

namespace {

constexpr int kThreads = 256;

// A column's place in the order of a row's logits as a whole number: the logit's
// order (NaN counts as -inf, -0 as 0), below it the column's number from behind, so
// that no two are alike and the lowest of equal columns is the largest.  A 16-bit
// logit and its column fit 32 bits.  0 stands for none (a real one is above it).
template <int OP>
struct Place {
    using Key = uint32_t;
    static __device__ __forceinline__ Key of(float x, int col) {
        x = x == x ? x + 0.f : -INFINITY;
        uint32_t b;
        if constexpr (OP == OP_BF16) {
            b = __float_as_uint(x) >> 16;
        } else {
            const _Float16 h = (_Float16)x;
            uint16_t t;
            __builtin_memcpy(&t, &h, 2);
            b = t;
        }
        b ^= b & 0x8000u ? 0xffffu : 0x8000u;
        return b << 16 | (0xffffu - (uint32_t)col);
    }
    static __device__ __forceinline__ int column(Key k) { return 0xffff - (int)(k & 0xffffu); }
    static __device__ __forceinline__ float value(Key k) {
        uint32_t b = k >> 16;
        b ^= b & 0x8000u ? 0x8000u : 0xffffu;
        if constexpr (OP == OP_BF16) return __uint_as_float(b << 16);
        const uint16_t t = (uint16_t)b;
        _Float16 h;
        __builtin_memcpy(&h, &t, 2);
        return (float)h;
    }
    template <int LPT>
    static __device__ __forceinline__ Key most(Key k) {
        return lanes_max<LPT>(k);
    }
};
template <>
struct Place<OP_F32> {
    using Key = uint64_t;
    static __device__ __forceinline__ Key of(float x, int col) {
        x = x == x ? x + 0.f : -INFINITY;
        uint32_t b = __float_as_uint(x);
        b ^= b & 0x80000000u ? 0xffffffffu : 0x80000000u;
        return (Key)b << 32 | (0xffffffffu - (uint32_t)col);
    }
    static __device__ __forceinline__ int column(Key k) { return (int)(0xffffffffu - (uint32_t)k); }
    static __device__ __forceinline__ float value(Key k) {
        const uint32_t b = (uint32_t)(k >> 32);
        return __uint_as_float(b ^ (b & 0x80000000u ? 0x80000000u : 0xffffffffu));
    }
    template <int LPT>
    static __device__ __forceinline__ Key most(Key k) {
        const auto larger = [](Key a, Key b) { return a > b ? a : b; };
        const auto step = [&](auto o) {
            constexpr int O = decltype(o)::value;
            if constexpr (LPT > O)
                k = larger(k, (Key)lane_other<O>((uint32_t)(k >> 32)) << 32 | lane_other<O>((uint32_t)k));
        };
        step(std::integral_constant<int, 1>{});
        step(std::integral_constant<int, 2>{});
        step(std::integral_constant<int, 4>{});
        step(std::integral_constant<int, 8>{});
        step(std::integral_constant<int, 16>{});
        step(std::integral_constant<int, 32>{});
        return k;
    }
};

// Eight keys in descending order (Batcher's odd-even merge: 19 exchanges).
template <typename Key>
__device__ __forceinline__ void sort8(Key (&k)[8]) {
    const auto order = [&](int i, int j) {
        const Key a = k[i], b = k[j];
        k[i] = a > b ? a : b;
        k[j] = a > b ? b : a;
    };
    order(0, 1), order(2, 3), order(4, 5), order(6, 7);
    order(0, 2), order(1, 3), order(4, 6), order(5, 7);
    order(1, 2), order(5, 6);
    order(0, 4), order(1, 5), order(2, 6), order(3, 7);
    order(2, 4), order(3, 5);
    order(1, 2), order(3, 4), order(5, 6);
}

// A lane's columns e0 .. e0 + EPL - 1 of a row; -inf behind the last and in rows
// that take no part.  A lane without a column reads the row's first and leaves it.
template <typename T, int EPL, bool WIDE>
__device__ __forceinline__ void load_columns(const T* row, int e0, int E, bool on, T (&v)[EPL]) {
    if constexpr (WIDE) {
#pragma unroll
        for (int j = 0; j < EPL; j += 8) {
            const bool in = on && e0 + j < E;
            T t[8];
            __builtin_memcpy(t, __builtin_assume_aligned(row + (in ? e0 + j : 0), 16), sizeof(t));
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j + e] = in ? t[e] : (T)-INFINITY;
        }
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const bool in = on && e0 + j < E;
            const T t = row[in ? e0 + j : 0];
            v[j] = in ? t : (T)-INFINITY;
        }
    }
}

// Losses from a batch entry's sums: of c_e sum_i p_ie, of lse^2, of rows.
__device__ __forceinline__ void write_loss(const BalanceArgs& a, int b, double terms,
                                           double squares, double n) {
    a.loss[2 * b] = n > 0 ? (float)(a.E * terms / (a.k * n * n)) : 0.f;
    a.loss[2 * b + 1] = n > 0 ? (float)(squares / n) : 0.f;
}

// A lane sorts its eight columns (two lists of eight, of 16), and k times the
// largest head of the lists is taken: a maximum over the lanes, and the list that
// it came from moves up.
template <int OP, int LPT, int EPL, int KMAX, bool WIDE>
__global__ __launch_bounds__(kThreads) void balance_kernel(const BalanceArgs a) {
    using T = typename El<OP>::T;
    using P = Place<OP>;
    using Key = typename P::Key;
    constexpr int GRP = kThreads / LPT, COLS = LPT * EPL, LISTS = EPL / 8;
    constexpr int SLOTS = (KMAX + LPT - 1) / LPT;  // of the chosen, a lane's
    __shared__ float red_p[4][COLS];
    __shared__ uint32_t hits[COLS];
    __shared__ float2 red_s[4];
    __shared__ double red_t[4];
    const int lane = threadIdx.x & 63, part = lane % LPT, e0 = part * EPL, b = blockIdx.y, E = a.E;
    const int size = a.lengths ? max(0, min(a.n, a.lengths[b])) : a.n;
    for (int e = threadIdx.x; e < COLS; e += kThreads) hits[e] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.blocks > 1) a.arrived[b] = 0;
    __syncthreads();
    float sum_p[EPL] = {}, squares = 0.f, count = 0.f;
    const int step = gridDim.x * GRP;
    const auto fetch = [&](int64_t i, T(&v)[EPL]) {
        load_columns<T, EPL, WIDE>((const T*)a.x.p + b * a.x.sb + i * a.x.sr, e0, E, i < size, v);
    };
    int64_t i = (int64_t)blockIdx.x * GRP + threadIdx.x / LPT;
    T next[EPL];
    if (i < a.n) fetch(i, next);
    for (; i < a.n; i += step) {
        const int64_t row = (int64_t)b * a.n + i;
        T v[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) v[j] = next[j];
        if (i + step < a.n) fetch(i + step, next);
        Key key[LISTS][8];
        float x[EPL], top = -INFINITY;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            x[j] = (float)v[j];
            key[j / 8][j % 8] = e0 + j < E ? P::of(x[j], e0 + j) : (Key)0;
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
#pragma unroll
        for (int l = 0; l < LISTS; ++l) sort8(key[l]);
        Key mine[SLOTS] = {};
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) {
            const int turns = min(LPT, a.k - q * LPT);
            for (int u = 0; u < turns; ++u) {
                Key head = key[0][0];
                if constexpr (LISTS > 1) head = head > key[1][0] ? head : key[1][0];
                const Key most = P::template most<LPT>(head);
#pragma unroll
                for (int l = 0; l < LISTS; ++l) {
                    const bool taken = key[l][0] == most;
#pragma unroll
                    for (int j = 0; j < 7; ++j) key[l][j] = taken ? key[l][j + 1] : key[l][j];
                    key[l][7] = taken ? (Key)0 : key[l][7];
                }
                mine[q] = part == u ? most : mine[q];
            }
        }
        float gate[SLOTS], all = 0.f;
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) {
            const bool have = on && q * LPT + part < a.k;
            gate[q] = have ? ex2((P::value(mine[q]) - ref) * kLog2e) * inv : 0.f;
            all += gate[q];
        }
        const float scale = a.normalize && on ? 1.f / lanes_sum<LPT>(all) : 1.f;
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) {
            const int t = q * LPT + part;
            if (t >= a.k) continue;
            const int id = on ? P::column(mine[q]) : -1;
            a.ids[row * a.k + t] = id;
            a.gates[row * a.k + t] = gate[q] * scale;
            if (on) atomicAdd(&hits[id], 1u);  // whole numbers: the order does not matter
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
        for (int j = 0; j < EPL; ++j) sum_p[j] += __shfl_xor(sum_p[j], o, 64);
        squares += __shfl_xor(squares, o, 64);
        count += __shfl_xor(count, o, 64);
    }
    const int wave = threadIdx.x >> 6;
    if (lane < LPT) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) red_p[wave][e0 + j] = sum_p[j];
    }
    if (lane == 0) red_s[wave] = make_float2(squares, count);
    __syncthreads();
    const int64_t at = (int64_t)b * a.blocks + blockIdx.x;
    double terms = 0.0;
    for (int e = threadIdx.x; e < E; e += kThreads) {
        const float p = red_p[0][e] + red_p[1][e] + red_p[2][e] + red_p[3][e];
        const int c = (int)hits[e];
        if (a.blocks == 1) {
            a.counts[(int64_t)b * E + e] = c;
            terms += (double)c * p;
        } else {
            a.part[at * E + e] = make_float2(p, __int_as_float(c));
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
    if (threadIdx.x == 0) write_loss(a, b, red_t[0] + red_t[1] + red_t[2] + red_t[3], sq, rows);
}

// The workgroups' sums of a batch entry, 16 columns a workgroup, 64 lanes each, in
// 64 bits and a fixed order.  The last of the entry's workgroups to arrive adds
// their terms (in their order) to the loss; the counter was cleared by the launch
// before.
__global__ __launch_bounds__(1024) void balance_join_kernel(const BalanceArgs a) {
    __shared__ double red_p[64][17];
    __shared__ int red_c[64][17];
    __shared__ int last;
    const int b = blockIdx.y, c = threadIdx.x & 15, y = threadIdx.x >> 4, e = blockIdx.x * 16 + c;
    double p = 0.0;
    int n = 0;
    if (e < a.E) {
#pragma unroll 4
        for (int k = y; k < a.blocks; k += 64) {
            const float2 v = a.part[((int64_t)b * a.blocks + k) * a.E + e];
            p += (double)v.x;
            n += __float_as_int(v.y);
        }
    }
    red_p[y][c] = p;
    red_c[y][c] = n;
    __syncthreads();
    for (int o = 32; o >= 1; o >>= 1) {
        if (y < o) red_p[y][c] += red_p[y + o][c], red_c[y][c] += red_c[y + o][c];
        __syncthreads();
    }
    double* terms = a.terms + (int64_t)b * gridDim.x;
    if (threadIdx.x < 64) {
        double t = 0.0;
        if (y == 0) {
            if (e < a.E) a.counts[(int64_t)b * a.E + e] = red_c[0][c];
            t = (double)red_c[0][c] * red_p[0][c];
        }
        for (int o = 8; o >= 1; o >>= 1) t += __shfl_xor(t, o, 64);
        if (threadIdx.x == 0) {
            __hip_atomic_store(terms + blockIdx.x, t, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            last = __hip_atomic_fetch_add(a.arrived + b, 1, __ATOMIC_ACQ_REL,
                                          __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!last || threadIdx.x >= 64) return;
    double sum = 0.0, squares = 0.0, rows = 0.0;
    for (int k = threadIdx.x; k < (int)gridDim.x; k += 64)
        sum += __hip_atomic_load(terms + k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    for (int k = threadIdx.x; k < a.blocks; k += 64) {
        const float2 s = a.part_s[(int64_t)b * a.blocks + k];
        squares += (double)s.x;
        rows += (double)s.y;
    }
    for (int o = 32; o >= 1; o >>= 1) {
        sum += __shfl_xor(sum, o, 64);
        squares += __shfl_xor(squares, o, 64);
        rows += __shfl_xor(rows, o, 64);
    }
    if (threadIdx.x == 0) write_loss(a, b, sum, squares, rows);
}

// Backward.  A lane takes up to SLOTS of a row's chosen columns; what each is worth
// goes to the lane that has the column through LDS, within a wave (whose LDS
// operations run in order).  Columns that are named twice are added one after the
// other.
template <int OP, int LPT, int EPL, int KMAX, bool WIDE>
__global__ __launch_bounds__(kThreads) void balance_bwd_kernel(const BalanceArgs a) {
    using T = typename El<OP>::T;
    constexpr int GRP = kThreads / LPT, SLOTS = (KMAX + LPT - 1) / LPT, COLS = LPT * EPL;
    __shared__ __align__(16) float worth_of[GRP][COLS];
    __shared__ __align__(16) int named_by[GRP][COLS];
    const int lane = threadIdx.x & 63, part = lane % LPT, e0 = part * EPL, b = blockIdx.y, E = a.E;
    const int size = a.lengths ? max(0, min(a.n, a.lengths[b])) : a.n;
    const uint32_t worth = lds_addr(worth_of[threadIdx.x / LPT]);
    const uint32_t named = lds_addr(named_by[threadIdx.x / LPT]);
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
    struct Row {
        T v[EPL];
        int id[SLOTS];  // of this lane's chosen columns, -1: none
        float g[SLOTS], x[SLOTS], lse;
        bool on;
    };
    const auto fetch = [&](int64_t i, Row& r) {
        const int64_t row = (int64_t)b * a.n + i;
        const T* x = (const T*)a.x.p + b * a.x.sb + i * a.x.sr;
        const int* ids = a.ids + row * a.k;
        r.on = i < size && ids[0] >= 0;
        r.lse = r.on ? a.lse[row] : 0.f;
        load_columns<T, EPL, WIDE>(x, e0, E, r.on, r.v);
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) {
            const int t = q * LPT + part;
            r.id[q] = -1;
            r.g[q] = r.x[q] = 0.f;
            if (!a.ggates || !r.on || t >= a.k) continue;
            const int id = ids[t];
            if (id < 0 || id >= E) continue;
            r.id[q] = id;
            r.g[q] = a.ggates[row * a.k + t];
            if (a.normalize) r.x[q] = (float)x[id];
        }
    };
    const int step = gridDim.x * GRP;
    for (int64_t i = (int64_t)blockIdx.x * GRP + threadIdx.x / LPT; i < a.n; i += step) {
        Row r;
        fetch(i, r);
        float p[EPL], dp[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) p[j] = ex2(((float)r.v[j] - r.lse) * kLog2e);
        if (a.ggates) {
            if (a.normalize) {
                float chosen = 0.f, mid = 0.f;
#pragma unroll
                for (int q = 0; q < SLOTS; ++q) {
                    const float pq = r.id[q] >= 0 ? ex2((r.x[q] - r.lse) * kLog2e) : 0.f;
                    chosen += pq;
                    mid = fmaf(pq, r.g[q], mid);
                }
                chosen = lanes_sum<LPT>(chosen);
                mid = lanes_sum<LPT>(mid);
                // (a choice from elsewhere may have no probability at all)
                const float scale = chosen != 0.f ? 1.f / chosen : 0.f, shift = mid * scale;
#pragma unroll
                for (int q = 0; q < SLOTS; ++q) r.g[q] = (r.g[q] - shift) * scale;
            }
#pragma unroll
            for (int j = 0; j < EPL; j += 4) lds_write<f32x4>(worth + 4 * (e0 + j), f32x4{0, 0, 0, 0});
#pragma unroll
            for (int q = 0; q < SLOTS; ++q)
                if (r.id[q] >= 0) lds_write<int>(named + 4 * r.id[q], q * LPT + part);
            asm volatile("" ::: "memory");
            bool twice = false;
#pragma unroll
            for (int q = 0; q < SLOTS; ++q)
                if (r.id[q] >= 0) {
                    twice |= lds_read<int>(named + 4 * r.id[q]) != q * LPT + part;
                    lds_write<float>(worth + 4 * r.id[q], r.g[q]);
                }
            asm volatile("" ::: "memory");
            if (__ballot(twice)) {
#pragma unroll
                for (int j = 0; j < EPL; j += 4)
                    lds_write<f32x4>(worth + 4 * (e0 + j), f32x4{0, 0, 0, 0});
                asm volatile("" ::: "memory");
#pragma unroll
                for (int q = 0; q < SLOTS; ++q)
                    for (int t = 0; t < LPT; ++t) {
                        if (part == t && r.id[q] >= 0) {
                            const uint32_t at = worth + 4 * r.id[q];
                            lds_write<float>(at, lds_read<float>(at) + r.g[q]);
                        }
                        asm volatile("" ::: "memory");
                    }
            }
#pragma unroll
            for (int j = 0; j < EPL; j += 4) {
                const f32x4 w = lds_read<f32x4>(worth + 4 * (e0 + j));
#pragma unroll
                for (int e = 0; e < 4; ++e) dp[j + e] = even[j + e] + w[e];
            }
            asm volatile("" ::: "memory");
        } else {
#pragma unroll
            for (int j = 0; j < EPL; ++j) dp[j] = even[j];
        }
        float mean = 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) mean = fmaf(p[j], dp[j], mean);
        mean = lanes_sum<LPT>(mean) - square * r.lse;
        T* gx = (T*)a.gx.p + b * a.gx.sb + i * a.gx.sr;
#pragma unroll
        for (int j = 0; j < EPL; ++j) r.v[j] = (T)(r.on ? p[j] * (dp[j] - mean) : 0.f);
        if constexpr (WIDE) {
#pragma unroll
            for (int j = 0; j < EPL; j += 8)
                if (e0 + j < E)
                    __builtin_memcpy(__builtin_assume_aligned(gx + e0 + j, 16), r.v + j, 8 * sizeof(T));
        } else {
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                if (e0 + j < E) gx[e0 + j] = r.v[j];
        }
    }
}

template <int OP, int LPT, int EPL, int KMAX, bool WIDE>
hipError_t go(const BalanceArgs& a, bool back, hipStream_t s) {
    if (back) {
        // no sums over rows: enough workgroups for every CU's waves
        const int64_t turns = ((int64_t)a.n + kThreads / LPT - 1) / (kThreads / LPT);
        const dim3 grid((unsigned)std::min<int64_t>(turns, std::max(1, 4096 / a.B)), (unsigned)a.B);
        balance_bwd_kernel<OP, LPT, EPL, KMAX, WIDE><<<grid, kThreads, 0, s>>>(a);
    } else {
        const dim3 grid((unsigned)a.blocks, (unsigned)a.B);
        balance_kernel<OP, LPT, EPL, KMAX, WIDE><<<grid, kThreads, 0, s>>>(a);
    }
    return hipGetLastError();
}
template <int OP, int LPT, int EPL, bool WIDE>
hipError_t go(const BalanceArgs& a, bool back, hipStream_t s) {
    constexpr int COLS = LPT * EPL, MOST = COLS < kBalanceMaxTop ? COLS : kBalanceMaxTop;
    return a.k <= 8 ? go<OP, LPT, EPL, 8, WIDE>(a, back, s) : go<OP, LPT, EPL, MOST, WIDE>(a, back, s);
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

// Workgroups of a batch entry: two turns of rows each, 1024 in all at most.
int balance_blocks(int B, int n, int E) {
    const int64_t turns = ((int64_t)n + rows_at_once(E) - 1) / rows_at_once(E);
    const int64_t most = std::max<int64_t>(1, 1024 / std::max(B, 1));
    return (int)std::max<int64_t>(1, std::min<int64_t>((turns + 1) / 2, most));
}

hipError_t launch_balance(const BalanceArgs& a, hipStream_t s) {
    const hipError_t e = go(a, false, s);
    if (e != hipSuccess || a.blocks == 1) return e;
    balance_join_kernel<<<dim3((unsigned)((a.E + 15) / 16), (unsigned)a.B), 1024, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_balance_bwd(const BalanceArgs& a, hipStream_t s) { return go(a, true, s); }

}  // namespace fs
