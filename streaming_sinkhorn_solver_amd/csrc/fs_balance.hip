// fs_balance.hip -- the k largest columns of each row of logits, how often each
// column is chosen, the balance loss and its gradient:
//   p = softmax(x), f_e = c_e / (k N), P_e = mean p_e:
//   L0 = E sum f P, L1 = mean lse^2, gates = p of the chosen (over their sum S);
//   dp_e = dL0 E f_e / N + sum_{id = e} (dgate - (sum dgate gate)) / S,
//   dx = p (dp - sum p dp + dL1 2 lse / N).
// A row's columns lie with LPT lanes.  Sums over rows run in the lanes' registers over
// a workgroup's rows (fp32: four rows a lane at 65536 x 256), then over workgroups in a
// second launch (in 64 bits, in a fixed order).  (65536 rows of 256 columns, 8 chosen,
// bf16: forward 20.2 us for 38 MB and 6.4 for the join, backward 24.6 us for 71 MB;
// bound by the vector unit: 564 instructions for four rows forward, 421 backward, which
// issue in 15 and 11 us.)
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
// logit has ten zeros at the end of its fp32 form, which hold the column's number.  0
// stands for none (a real one is above it).
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(fmaxf(x + 0.f, -INFINITY));
    return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float ordered(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
template <int OP>
struct Place {
    using Key = uint32_t;
    static constexpr uint32_t kLow = kBalanceMaxExperts - 1;
    static __device__ __forceinline__ Key of(float x, int col, bool in) {
        const Key k = (order_of(x) & ~kLow) | (kLow - (uint32_t)col);
        return k & (in ? ~0u : 0u);
    }
    static __device__ __forceinline__ int column(Key k) { return (int)(kLow - (k & kLow)); }
    static __device__ __forceinline__ float value(Key k) {
        return ordered(k & 0x80000000u ? k & ~kLow : k | kLow);
    }
    template <int LPT>
    static __device__ __forceinline__ Key most(Key k) {
        return lanes_max<LPT>(k);
    }
};
static_assert(kBalanceMaxExperts == 1 << 10, "a column's number has ten bits");
template <>
struct Place<OP_F32> {
    using Key = uint64_t;
    static __device__ __forceinline__ Key of(float x, int col, bool in) {
        return in ? (Key)order_of(x) << 32 | (0xffffffffu - (uint32_t)col) : (Key)0;
    }
    static __device__ __forceinline__ int column(Key k) { return (int)(0xffffffffu - (uint32_t)k); }
    static __device__ __forceinline__ float value(Key k) { return ordered((uint32_t)(k >> 32)); }
    template <int LPT>
    static __device__ __forceinline__ Key most(Key k) {
        const auto step = [&](auto o) {
            constexpr int O = decltype(o)::value;
            if constexpr (LPT > O) {
                const Key other =
                    (Key)lane_other<O>((uint32_t)(k >> 32)) << 32 | lane_other<O>((uint32_t)k);
                k = k > other ? k : other;
            }
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

template <typename Key>
__device__ __forceinline__ void exchange(Key& a, Key& b) {
    const Key x = a, y = b;
    a = x > y ? x : y;
    b = x > y ? y : x;
}
// Eight keys in descending order (Batcher's odd-even merge: 19 exchanges).
template <typename Key>
__device__ __forceinline__ void sort8(Key (&k)[8]) {
    const auto order = [&](int i, int j) { exchange(k[i], k[j]); };
    order(0, 1), order(2, 3), order(4, 5), order(6, 7);
    order(0, 2), order(1, 3), order(4, 6), order(5, 7);
    order(1, 2), order(5, 6);
    order(0, 4), order(1, 5), order(2, 6), order(3, 7);
    order(2, 4), order(3, 5);
    order(1, 2), order(3, 4), order(5, 6);
}
// a: the eight largest of two descending lists (one list against the other from
// behind leaves them, rising and falling once, which twelve exchanges sort).
template <typename Key>
__device__ __forceinline__ void merge8(Key (&a)[8], const Key (&b)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = a[j] > b[7 - j] ? a[j] : b[7 - j];
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if ((j & o) == 0) exchange(a[j], a[j + o]);
}

// The column that is a lane's j-th of a row's LPT lanes.  WIDE: groups of eight
// neighbours, groups side by side with neighbouring lanes; else single ones, so that
// a wave's reads and writes are of neighbours either way.
template <int LPT, bool WIDE>
__device__ __forceinline__ int column_of(int part, int j) {
    return WIDE ? (j / 8 * LPT + part) * 8 + j % 8 : j * LPT + part;
}
// A lane's columns of a row; -inf behind the last and in rows that take no part.  A
// lane without a column reads the row's first and leaves it.
template <typename T, int LPT, int EPL, bool WIDE>
__device__ __forceinline__ void load_columns(const T* row, int part, int E, bool on, T (&v)[EPL]) {
    if constexpr (WIDE) {
#pragma unroll
        for (int j = 0; j < EPL; j += 8) {
            const int col = column_of<LPT, WIDE>(part, j);
            const bool in = on && col < E;
            T t[8];
            __builtin_memcpy(t, __builtin_assume_aligned(row + (in ? col : 0), 16), sizeof(t));
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j + e] = in ? t[e] : (T)-INFINITY;
        }
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int col = column_of<LPT, WIDE>(part, j);
            const bool in = on && col < E;
            const T t = row[in ? col : 0];
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

// A lane sorts its columns (16 of them in two lists of eight, merged to the largest
// eight where no more are chosen), and k times the largest head of the lists is
// taken: a maximum over the lanes, and the list that it came from moves up.  Bound by
// the vector unit's instructions, of which a lane of 16 columns needs fewer a row
// than two of eight.
template <int OP, int LPT, int EPL, int KMAX, bool WIDE>
__global__ __launch_bounds__(kThreads) void balance_kernel(const BalanceArgs a) {
    using T = typename El<OP>::T;
    using P = Place<OP>;
    using Key = typename P::Key;
    constexpr int GRP = kThreads / LPT, COLS = LPT * EPL;
    constexpr int SORTED = EPL / 8, LISTS = KMAX <= 8 ? 1 : SORTED;
    constexpr int SLOTS = (KMAX + LPT - 1) / LPT;  // of the chosen, a lane's
    __shared__ float red_p[4][COLS];
    __shared__ uint32_t hits[COLS];
    __shared__ float2 red_s[4];
    __shared__ double red_t[4];
    const int lane = threadIdx.x & 63, part = lane % LPT, b = blockIdx.y, E = a.E;
    const int size = a.lengths ? max(0, min(a.n, a.lengths[b])) : a.n;
    for (int e = threadIdx.x; e < COLS; e += kThreads) hits[e] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.blocks > 1) a.arrived[b] = 0;
    __syncthreads();
    float sum_p[EPL] = {}, squares = 0.f, count = 0.f;
    const int step = gridDim.x * GRP;
    const auto fetch = [&](int64_t i, T(&v)[EPL]) {
        load_columns<T, LPT, EPL, WIDE>((const T*)a.x.p + b * a.x.sb + i * a.x.sr, part, E, i < size, v);
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
        Key key[SORTED][8];
        float x[EPL], top = -INFINITY;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            x[j] = (float)v[j];
            const int col = column_of<LPT, WIDE>(part, j);
            key[j / 8][j % 8] = P::of(x[j], col, (WIDE ? col - j % 8 : col) < E);
            top = fmaxf(top, x[j]);
        }
        top = lanes_max<LPT>(top);
        const float ref = top == -INFINITY ? 0.f : top;
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) s += x[j] = ex2((x[j] - ref) * kLog2e);
        s = lanes_sum<LPT>(s);
        // 0 for a row of -inf alone, which takes no part; the maximum passes over a NaN, the
        // sum is one, also where a row holds nothing else
        const bool on = s != 0.f;
        const float inv = on ? __builtin_amdgcn_rcpf(s) : 0.f, lse = on ? fmaf(lg2(s), kLn2, ref) : 0.f;
#pragma unroll
        for (int l = 0; l < SORTED; ++l) sort8(key[l]);
        if constexpr (SORTED > LISTS) merge8(key[0], key[1]);
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
        const float scale = a.normalize && on ? __builtin_amdgcn_rcpf(lanes_sum<LPT>(all)) : 1.f;
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
        for (int j = 0; j < EPL; ++j) red_p[wave][column_of<LPT, WIDE>(part, j)] = sum_p[j];
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
            a.part[at * (E + 1) + e] = make_float2(p, __int_as_float(c));
        }
    }
    const float sq = red_s[0].x + red_s[1].x + red_s[2].x + red_s[3].x;
    const float rows = red_s[0].y + red_s[1].y + red_s[2].y + red_s[3].y;
    if (a.blocks > 1) {
        if (threadIdx.x == 0) a.part[at * (E + 1) + E] = make_float2(sq, __int_as_float((int)rows));
        return;
    }
    for (int o = 32; o >= 1; o >>= 1) terms += __shfl_xor(terms, o, 64);
    if (lane == 0) red_t[wave] = terms;
    __syncthreads();
    if (threadIdx.x == 0) write_loss(a, b, red_t[0] + red_t[1] + red_t[2] + red_t[3], sq, rows);
}

// The workgroups' sums of a batch entry (behind the columns' those of lse^2 and of
// rows that take part), 8 columns a workgroup, 128 lanes each, in 64 bits and a fixed
// order.  The last of the entry's workgroups to arrive adds their terms (in their
// order) to the loss; the counter was cleared by the launch before.
__global__ __launch_bounds__(1024) void balance_join_kernel(const BalanceArgs a) {
    __shared__ double red_p[128][9];
    __shared__ int red_c[128][9];
    __shared__ int last;
    const int b = blockIdx.y, c = threadIdx.x & 7, y = threadIdx.x >> 3, e = blockIdx.x * 8 + c;
    double p = 0.0;
    int n = 0;
    if (e <= a.E) {
#pragma unroll 8
        for (int k = y; k < a.blocks; k += 128) {
            const float2 v = a.part[((int64_t)b * a.blocks + k) * (a.E + 1) + e];
            p += (double)v.x;
            n += __float_as_int(v.y);
        }
    }
    red_p[y][c] = p;
    red_c[y][c] = n;
    __syncthreads();
    for (int o = 64; o >= 1; o >>= 1) {
        if (y < o) red_p[y][c] += red_p[y + o][c], red_c[y][c] += red_c[y + o][c];
        __syncthreads();
    }
    // [gridDim.x] terms, then the sums of squares and rows
    double* terms = a.terms + (int64_t)b * (gridDim.x + 2);
    const auto put = [&](int at, double v) {
        __hip_atomic_store(terms + at, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    };
    if (threadIdx.x < 64) {
        double t = 0.0;
        if (y == 0 && e < a.E) {
            a.counts[(int64_t)b * a.E + e] = red_c[0][c];
            t = (double)red_c[0][c] * red_p[0][c];
        }
        if (y == 0 && e == a.E) put(gridDim.x, red_p[0][c]), put(gridDim.x + 1, (double)red_c[0][c]);
        for (int o = 4; o >= 1; o >>= 1) t += __shfl_xor(t, o, 64);
        if (threadIdx.x == 0) put(blockIdx.x, t);
        __threadfence();
        if (threadIdx.x == 0)
            last = __hip_atomic_fetch_add(a.arrived + b, 1, __ATOMIC_ACQ_REL,
                                          __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
    }
    __syncthreads();
    if (!last || threadIdx.x >= 64) return;
    const auto get = [&](int at) {
        return __hip_atomic_load(terms + at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    };
    double sum = 0.0;
    for (int k = threadIdx.x; k < (int)gridDim.x; k += 64) sum += get(k);
    for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, 64);
    if (threadIdx.x == 0) write_loss(a, b, sum, get(gridDim.x), get(gridDim.x + 1));
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
    __shared__ __align__(16) float named_by[GRP][COLS];
    const int lane = threadIdx.x & 63, part = lane % LPT, b = blockIdx.y, E = a.E;
    const int size = a.lengths ? max(0, min(a.n, a.lengths[b])) : a.n;
    const uint32_t worth = lds_addr(worth_of[threadIdx.x / LPT]);
    const uint32_t named = lds_addr(named_by[threadIdx.x / LPT]);
    // a lane's columns by fours, the fours of a row's lanes side by side
    const auto fours = [&](int j) { return (uint32_t)(j / 4 * LPT + part) * 16; };
    const auto place = [](int col) {
        const int p = WIDE ? col / 8 % LPT : col % LPT;
        const int j = WIDE ? col / (8 * LPT) * 8 + col % 8 : col / LPT;
        return (uint32_t)((j / 4 * LPT + p) * 4 + j % 4) * 4;
    };
#pragma unroll
    for (int j = 0; j < EPL; j += 4) {
        lds_write<f32x4>(worth + fours(j), f32x4{0, 0, 0, 0});
        lds_write<f32x4>(named + fours(j), f32x4{0, 0, 0, 0});
    }
    asm volatile("" ::: "memory");
    // what every row's probabilities are worth to the balance: E c_e / (k N^2)
    float even[EPL];
    uint32_t sum = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int col = column_of<LPT, WIDE>(part, j);
        const int c = col < E ? a.counts[(int64_t)b * E + col] : 0;
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
        int id[SLOTS], first;  // this lane's chosen columns, the row's first
        float g[SLOTS], lse;
    };
    // (every read of a row is under way before the first is waited for)
    const auto fetch = [&](int64_t i, Row& r) {
        const int64_t row = (int64_t)b * a.n + i;
        const bool in = i < size;
        const int* ids = a.ids + row * a.k;
        load_columns<T, LPT, EPL, WIDE>((const T*)a.x.p + b * a.x.sb + i * a.x.sr, part, E, in, r.v);
        r.first = ids[0];
        r.lse = a.lse[row];
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) {
            const int t = q * LPT + part;
            r.id[q] = ids[t < a.k ? t : 0];
            r.g[q] = a.ggates ? a.ggates[row * a.k + (t < a.k ? t : 0)] : 0.f;
            if (t >= a.k || !a.ggates) r.id[q] = -1;
        }
        if (!in) r.first = -1;
    };
    const int step = gridDim.x * GRP;
    int64_t i = (int64_t)blockIdx.x * GRP + threadIdx.x / LPT;
    Row next;
    if (i < a.n) fetch(i, next);
    for (; i < a.n; i += step) {
        Row r = next;
        if (i + step < a.n) fetch(i + step, next);
        const bool on = r.first >= 0;
        // p by the row's own sum: lse as fp32 holds it is off by up to 2^-24 of it, a factor of
        // all of the row (6e-5 at logits of 1000), which falls out
        float p[EPL], dp[EPL], all = 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            all += p[j] = on ? ex2(((float)r.v[j] - r.lse) * kLog2e) : 0.f;
            dp[j] = even[j];
        }
        all = lanes_sum<LPT>(all);
        const float inv = all != 0.f ? __builtin_amdgcn_rcpf(all) : 0.f;  // of p as it stands
        if (a.ggates) {
            bool have[SLOTS], twice = false;
            uint32_t at[SLOTS];
#pragma unroll
            for (int q = 0; q < SLOTS; ++q) {
                have[q] = on && r.id[q] >= 0 && r.id[q] < E;
                at[q] = have[q] ? place(r.id[q]) : 0;
                if (have[q]) lds_write<int>(named + at[q], 1 + q * LPT + part);
            }
            asm volatile("" ::: "memory");
#pragma unroll
            for (int q = 0; q < SLOTS; ++q)
                if (have[q]) twice |= lds_read<int>(named + at[q]) != 1 + q * LPT + part;
            asm volatile("" ::: "memory");
            if (!__ballot(twice)) {
#pragma unroll
                for (int q = 0; q < SLOTS; ++q)
                    if (have[q]) {
                        lds_write<float>(worth + at[q], r.g[q]);
                        lds_write<float>(named + at[q], 1.f);
                    }
            } else {
#pragma unroll
                for (int q = 0; q < SLOTS; ++q)
                    if (have[q]) lds_write<float>(named + at[q], 0.f);
                asm volatile("" ::: "memory");
#pragma unroll
                for (int q = 0; q < SLOTS; ++q)
                    for (int t = 0; t < LPT; ++t) {
                        if (part == t && have[q]) {
                            lds_write<float>(worth + at[q], lds_read<float>(worth + at[q]) + r.g[q]);
                            lds_write<float>(named + at[q], lds_read<float>(named + at[q]) + 1.f);
                        }
                        asm volatile("" ::: "memory");
                    }
            }
            asm volatile("" ::: "memory");
            float dg[EPL], times[EPL], scale = 1.f, shift = 0.f;
#pragma unroll
            for (int j = 0; j < EPL; j += 4) {
                const f32x4 x = lds_read<f32x4>(worth + fours(j));
                const f32x4 y = lds_read<f32x4>(named + fours(j));
#pragma unroll
                for (int e = 0; e < 4; ++e) dg[j + e] = x[e], times[j + e] = y[e];
            }
            asm volatile("" ::: "memory");
            // zeros again for the next row
#pragma unroll
            for (int q = 0; q < SLOTS; ++q)
                if (have[q]) {
                    lds_write<float>(worth + at[q], 0.f);
                    lds_write<float>(named + at[q], 0.f);
                }
            asm volatile("" ::: "memory");
            if (a.normalize) {
                float chosen = 0.f, mid = 0.f;
#pragma unroll
                for (int j = 0; j < EPL; ++j) {
                    chosen = fmaf(p[j], times[j], chosen);
                    mid = fmaf(p[j], dg[j], mid);
                }
                chosen = lanes_sum<LPT>(chosen);
                mid = lanes_sum<LPT>(mid);
                // (a choice from elsewhere may have no probability at all)
                const float over = chosen != 0.f ? 1.f / chosen : 0.f;
                scale = all * over;
                shift = mid * over;
            }
#pragma unroll
            for (int j = 0; j < EPL; ++j) dp[j] = fmaf(fmaf(-times[j], shift, dg[j]), scale, dp[j]);
        }
        float mean = 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) mean = fmaf(p[j], dp[j], mean);
        mean = (lanes_sum<LPT>(mean) * inv - (on ? square * r.lse : 0.f)) * inv;
        T* gx = (T*)a.gx.p + b * a.gx.sb + i * a.gx.sr;
#pragma unroll
        for (int j = 0; j < EPL; ++j) r.v[j] = (T)(on ? p[j] * fmaf(dp[j], inv, -mean) : 0.f);
        if constexpr (WIDE) {
#pragma unroll
            for (int j = 0; j < EPL; j += 8) {
                const int col = column_of<LPT, WIDE>(part, j);
                if (col < E)
                    __builtin_memcpy(__builtin_assume_aligned(gx + col, 16), r.v + j, 8 * sizeof(T));
            }
        } else {
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                const int col = column_of<LPT, WIDE>(part, j);
                if (col < E) gx[col] = r.v[j];
            }
        }
    }
}

template <int OP, int LPT, int EPL, int KMAX, bool WIDE>
hipError_t go(const BalanceArgs& a, bool back, hipStream_t s) {
    if (back) {
        // four workgroups a CU, which read a row ahead
        const int64_t turns = ((int64_t)a.n + kThreads / LPT - 1) / (kThreads / LPT);
        const dim3 grid((unsigned)std::min<int64_t>(turns, std::max(1, 1024 / a.B)), (unsigned)a.B);
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
    if (a.E <= 128) return go<OP, 8, 16>(a, back, s);
    if (a.E <= 256) return go<OP, 16, 16>(a, back, s);
    if (a.E <= 512) return go<OP, 32, 16>(a, back, s);
    return go<OP, 64, 16>(a, back, s);
}
hipError_t go(const BalanceArgs& a, bool back, hipStream_t s) {
    return a.op == OP_BF16 ? go<OP_BF16>(a, back, s)
           : a.op == OP_F16 ? go<OP_F16>(a, back, s)
                            : go<OP_F32>(a, back, s);
}

int rows_at_once(int E) {
    int lanes = 1;
    while (lanes < 64 && lanes * (E <= 64 ? 8 : 16) < E) lanes *= 2;
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
    balance_join_kernel<<<dim3((unsigned)(a.E / 8 + 1), (unsigned)a.B), 1024, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_balance_bwd(const BalanceArgs& a, hipStream_t s) { return go(a, true, s); }

}  // namespace fs
