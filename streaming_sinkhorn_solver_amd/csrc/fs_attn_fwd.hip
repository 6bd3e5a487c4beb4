// fs_attn_fwd.hip -- attention between two sets of states, forward:
//   s_ij = scale q_i.k_j + T[bucket(j - i - offset), head],
//   L_i = log sum_j exp s_ij,   O_i = sum_j exp(s_ij - L_i) v_j
// over the visible keys.  One pass over the keys with a running reference M
// and sum, in base 2 (s2 = s log2 e): a row's weights are 2^(s2 - M), and M
// moves up only when a score exceeds it by more than kSlack, so that the sums
// are rescaled a few times per row, not once per tile.
#include "fs_attn.hpp"

namespace fs {

namespace {

// The weights go into the second product in the element type.  M lies kShift
// below the largest score seen when it was set: fp16 keeps weights down to
// 2^-24, so its weights are lifted by 2^6 (at most 2^14), which leaves a row's
// lost mass below 2^-31 per key.  bf16 and fp32 have the exponents of fp32.
constexpr float kSlack = 8.f;
template <int OP>
constexpr float kShift = OP == OP_F16 ? 6.f : 0.f;

// Running state of a lane's column (a query row; the two halves of a wave
// hold the same reference and each its own part of the sum).
struct Run {
    float ref = -INFINITY;
    float sum = 0.f;
};

// Moves the reference up to mx - shift where some row needs it; acc and the
// sum follow.
template <int OP, int ND>
__device__ __forceinline__ void raise_ref(Run& st, float mx, f32x16 (&acc)[ND]) {
    if (!__any(mx > st.ref + (kSlack + kShift<OP>))) return;
    const float to = fmaxf(st.ref, mx - kShift<OP>);
    const float f = to == st.ref ? 1.f : ex2(st.ref - to);
    st.ref = to;
    st.sum *= f;
#pragma unroll
    for (int x = 0; x < ND; ++x)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[x][r] *= f;
}

// s <- 2^(s cm + ca - ref); returns the sum of the sixteen.  A row that has
// seen no key yet (ref = -inf, all its scores -inf) gets zeros.
__device__ __forceinline__ float weights(f32x16& s, float cm, float ca, const Run& st) {
    const float sub = ca - (st.ref == -INFINITY ? 0.f : st.ref);
    float t = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        s[r] = ex2(fmaf(s[r], cm, sub));
        t += s[r];
    }
    return t;
}

// Four results of a lane as four elements of a row (x0 a multiple of 4).
template <int OP>
__device__ __forceinline__ void store4(typename El<OP>::T* row, int x0, int d, bool vec, float a,
                                       float b, float c, float e) {
    using T = typename El<OP>::T;
    const float y[4] = {a, b, c, e};
    T o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (T)y[i];
    if (vec) {
        if (x0 < d) __builtin_memcpy(__builtin_assume_aligned(row + x0, sizeof(o)), o, sizeof(o));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (x0 + i < d) row[x0 + i] = o[i];
    }
}

// ---- many query rows ------------------------------------------------------
// A workgroup of four waves takes 128 query rows of one head, 32 a wave, and
// a range of keys in tiles of KT staged through LDS and shared by the waves.
// Scores are formed with keys in the rows (S^T = K Q^T), so a lane holds
// scores of one query row: maximum and sum need one exchange, between the
// halves of the wave, and the weights are operands of O^T = V^T P^T as they
// are.
template <int OP, int DP>
constexpr int kTileKeys = DP * (int)sizeof(typename El<OP>::T) <= 256 ? 64 : 32;

template <int OP, int DP, bool BIAS>
__global__ __launch_bounds__(256, DP * sizeof(typename El<OP>::T) <= 256 ? 2 : 1)
void attn_fwd_kernel(const AttnArgs a) {
    using E = El<OP>;
    using T = typename E::T;
    using L = Tile<OP, DP>;
    constexpr int KT = kTileKeys<OP, DP>, NB = KT / 32, ND = DP / 32, NK = DP / 16;
    __shared__ __attribute__((aligned(256))) char kt[KT * L::kRow];
    __shared__ __attribute__((aligned(256))) char vt[KT * L::kRow];
    __shared__ float line[BIAS ? 2 * kAttnMaxEdge + 1 : 1];

    const int t = threadIdx.x, lane = t & 63, wid = t >> 6, h = lane >> 5;
    const int nqb = (a.n + kAttnRows - 1) / kAttnRows;
    int w = xcd_item(blockIdx.x, gridDim.x);
    const int qb = w % nqb;
    w /= nqb;
    const int split = w % a.n_split;
    w /= a.n_split;
    const int head = w % a.H, b = w / a.H, kvh = head / a.G;

    const int off = attn_offset(a, b);
    const int i0 = qb * kAttnRows + wid * 32, i = i0 + (lane & 31);
    const bool row_ok = i < attn_q_len(a, b);
    int len = attn_kv_len(a, b);
    if (a.causal) len = min(len, max(0, min(qb * kAttnRows + kAttnRows, a.n) + off));
    const int jb = split * a.split_keys;
    const int je = a.n_split == 1 ? len : min(len, jb + a.split_keys);

    if (BIAS) load_line(a, head, line, t, 256);

    typename E::Frag qf[NK];
    load_row_frags<OP, DP>((const T*)a.q.p + b * a.q.sb + (int64_t)i * a.q.sr + head * a.q.sh,
                           row_ok, a.d, a.q.vec, lane, qf);
    f32x16 acc[ND];
#pragma unroll
    for (int x = 0; x < ND; ++x)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[x][r] = 0.f;
    Run st;

    const T* kbase = (const T*)a.k.p + b * a.k.sb + kvh * a.k.sh;
    const T* vbase = (const T*)a.v.p + b * a.v.sb + kvh * a.v.sh;
    Stage<OP, DP, KT, 256> ks, vs;
    uint64_t next = 0;
    if (jb < je) {
        next = seen_keys(a, b, je, jb, lane);
        ks.load(kbase + (int64_t)jb * a.k.sr, a.k.sr, next, a.d, a.k.vec, t);
        vs.load(vbase + (int64_t)jb * a.v.sr, a.v.sr, next, a.dv, a.v.vec, t);
    }
    for (int j0 = jb; j0 < je; j0 += KT) {
        const uint64_t seen = next;
        __syncthreads();
        ks.store(kt, t);
        vs.store(vt, t);
        __syncthreads();
        if (j0 + KT < je) {
            next = seen_keys(a, b, je, j0 + KT, lane);
            ks.load(kbase + (int64_t)(j0 + KT) * a.k.sr, a.k.sr, next, a.d, a.k.vec, t);
            vs.load(vbase + (int64_t)(j0 + KT) * a.v.sr, a.v.sr, next, a.dv, a.v.vec, t);
        }
        f32x16 s[NB];
        uint32_t vis[NB];
        bool all = true;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            vis[nb] = (uint32_t)(seen >> (32 * nb));
            if (a.causal) vis[nb] &= bits_upto(i + off - (j0 + 32 * nb));
            all = all && vis[nb] == ~0u;
            vis[nb] >>= 4 * h;
        }
        all = __all(all);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int r = 0; r < 16; ++r) s[nb][r] = 0.f;
#pragma unroll
            for (int kk = 0; kk < NK; ++kk)
                s[nb] = E::mfma(L::frag_rows(kt, 32 * nb, kk, lane), qf[kk], s[nb]);
        }
        float cm = a.c, ca = 0.f;
        if (BIAS) {
            const int lo = j0 - i0 - 31 - off, hi = j0 + KT - 1 - i0 - off;
            if (hi <= -a.r0) {
                ca = line[0];
            } else if (lo >= a.rp) {
                ca = line[a.r0 + a.rp];
            } else {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        s[nb][r] = fmaf(s[nb][r], a.c,
                                        line[line_index(a, j0 + 32 * nb + 8 * (r >> 2) + 4 * h +
                                                               (r & 3) - i - off)]);
                cm = 1.f;
            }
        }
        if (!all) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int r = 0; r < 16; ++r) s[nb][r] = flag(vis[nb], r) ? s[nb][r] : -INFINITY;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[nb][r]);
        mx = half_max(mx);
        mx = fmaf(mx, cm, ca);
        raise_ref<OP, ND>(st, mx, acc);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            st.sum += weights(s[nb], cm, ca, st);
#pragma unroll
            for (int rc = 0; rc < 2; ++rc) {
                const typename E::Frag pf = L::pack(s[nb], rc);
#pragma unroll
                for (int cb = 0; cb < ND; ++cb)
                    acc[cb] = E::mfma(L::frag_cols(vt, 32 * nb + 16 * rc, cb, lane), pf, acc[cb]);
            }
        }
    }

    st.sum = half_sum(st.sum);
    if (i >= a.n) return;
    if (!row_ok) st.sum = 0.f;
    if (a.n_split > 1) {
        const int64_t row = (int64_t)(b * a.H + head) * a.n + i;
        const int64_t rows = (int64_t)a.B * a.H * a.n;
        if (h == 0) a.part_ml[split * rows + row] = make_float2(st.sum > 0.f || st.sum != st.sum ? st.ref : -INFINITY, st.sum);
        float* po = a.part_o + (split * rows + row) * a.dv;
#pragma unroll
        for (int cb = 0; cb < ND; ++cb)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int x = 32 * cb + 8 * (r >> 2) + 4 * h + (r & 3);
                if (x < a.dv) po[x] = row_ok ? acc[cb][r] : 0.f;
            }
        return;
    }
    const bool some = !(st.sum == 0.f);
    const float inv = some ? 1.f / st.sum : 0.f;
    T* o = (T*)a.o.p + b * a.o.sb + (int64_t)i * a.o.sr + head * a.o.sh;
#pragma unroll
    for (int cb = 0; cb < ND; ++cb)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float y[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) y[r] = some ? acc[cb][4 * q + r] * inv : 0.f;
            store4<OP>(o, 32 * cb + 8 * q + 4 * h, a.dv, a.o.vec, y[0], y[1], y[2], y[3]);
        }
    if (a.lse && h == 0)
        a.lse[(int64_t)(b * a.H + head) * a.n + i] =
            some ? (st.ref + lg2(st.sum)) * kLn2 : -INFINITY;
}

// ---- few query rows -------------------------------------------------------
// For single tokens and a few rows per head the keys are the whole cost.  The
// query rows of all heads of a key head are packed into blocks of 32; the
// four waves of a workgroup take key tiles of 32 in turn, each staged in the
// wave's own part of LDS with the next tile's loads in flight, without
// barriers, and their four results are joined at the end.  Long key ranges
// are split over workgroups and joined by a second kernel.
template <int OP, int DP, bool BIAS>
__global__ __launch_bounds__(256, DP * sizeof(typename El<OP>::T) <= 256 ? 2 : 1)
void attn_rows_kernel(const AttnArgs a) {
    using E = El<OP>;
    using T = typename E::T;
    using L = Tile<OP, DP>;
    constexpr int KT = 32, ND = DP / 32, NK = DP / 16;
    __shared__ __attribute__((aligned(256))) char tiles[4][2][KT * L::kRow];
    static_assert(sizeof(tiles) >= 4 * 32 * DP * 4, "the four results fit the tiles' memory");
    __shared__ short bucket[BIAS ? 2 * kAttnMaxEdge + 1 : 1];
    __shared__ float wref[4][32], wsum[4][32];

    const int t = threadIdx.x, lane = t & 63, wid = t >> 6, h = lane >> 5;
    const int rows = a.G * a.n;
    const int nrb = (rows + 31) / 32;
    int w = xcd_item(blockIdx.x, gridDim.x);
    const int rb = w % nrb;
    w /= nrb;
    const int split = w % a.n_split;
    w /= a.n_split;
    const int kvh = w % a.K, b = w / a.K;

    const int off = attn_offset(a, b);
    const int rho = rb * 32 + (lane & 31);
    const int g = min(rho, rows - 1) / a.n, i = min(rho, rows - 1) - g * a.n;
    const int head = kvh * a.G + g;
    const bool row_ok = rho < rows && i < attn_q_len(a, b);
    int len = attn_kv_len(a, b);
    if (a.causal) len = min(len, max(0, a.n + off));
    const int jb = split * a.split_keys;
    const int je = a.n_split == 1 ? len : min(len, jb + a.split_keys);

    float bias_lo = 0.f, bias_hi = 0.f;
    if (BIAS) {
        for (int x = t; x < a.r0 + a.rp + 1; x += 256) bucket[x] = (short)bucket_of(a, x - a.r0);
        __syncthreads();
        bias_lo = bias2(a.bias[(int64_t)bucket[0] * a.H + head]);
        bias_hi = bias2(a.bias[(int64_t)bucket[a.r0 + a.rp] * a.H + head]);
    }

    typename E::Frag qf[NK];
    load_row_frags<OP, DP>((const T*)a.q.p + b * a.q.sb + (int64_t)i * a.q.sr + head * a.q.sh,
                           row_ok, a.d, a.q.vec, lane, qf);
    f32x16 acc[ND];
#pragma unroll
    for (int x = 0; x < ND; ++x)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[x][r] = 0.f;
    Run st;

    const T* kbase = (const T*)a.k.p + b * a.k.sb + kvh * a.k.sh;
    const T* vbase = (const T*)a.v.p + b * a.v.sb + kvh * a.v.sh;
    char* kt = tiles[wid][0];
    char* vt = tiles[wid][1];
    Stage<OP, DP, KT, 64> ks, vs;
    const int j_first = jb + wid * KT;
    uint32_t next = 0;
    if (j_first < je) {
        next = (uint32_t)seen_keys(a, b, je, j_first, lane);
        ks.load(kbase + (int64_t)j_first * a.k.sr, a.k.sr, next, a.d, a.k.vec, lane);
        vs.load(vbase + (int64_t)j_first * a.v.sr, a.v.sr, next, a.dv, a.v.vec, lane);
    }
    for (int j0 = j_first; j0 < je; j0 += 4 * KT) {
        const uint32_t seen = next;
        // the wave's own LDS: its reads of the last tile are in registers by now
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        ks.store(kt, lane);
        vs.store(vt, lane);
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        if (j0 + 4 * KT < je) {
            const int jn = j0 + 4 * KT;
            next = (uint32_t)seen_keys(a, b, je, jn, lane);
            ks.load(kbase + (int64_t)jn * a.k.sr, a.k.sr, next, a.d, a.k.vec, lane);
            vs.load(vbase + (int64_t)jn * a.v.sr, a.v.sr, next, a.dv, a.v.vec, lane);
        }
        uint32_t vis = seen;
        if (a.causal) vis &= bits_upto(i + off - j0);
        const bool all = __all(vis == ~0u);
        vis >>= 4 * h;
        f32x16 s;
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = 0.f;
#pragma unroll
        for (int kk = 0; kk < NK; ++kk) s = E::mfma(L::frag_rows(kt, 0, kk, lane), qf[kk], s);
        float cm = a.c, ca = 0.f;
        if (BIAS) {
            const int lo = j0 - (a.n - 1) - off, hi = j0 + KT - 1 - off;
            if (hi <= -a.r0) {
                ca = bias_lo;
            } else if (lo >= a.rp) {
                ca = bias_hi;
            } else {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int c = bucket[line_index(a, j0 + 8 * (r >> 2) + 4 * h + (r & 3) - i - off)];
                    s[r] = fmaf(s[r], a.c, bias2(a.bias[(int64_t)c * a.H + head]));
                }
                cm = 1.f;
            }
        }
        if (!all) {
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = flag(vis, r) ? s[r] : -INFINITY;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[r]);
        mx = fmaf(half_max(mx), cm, ca);
        raise_ref<OP, ND>(st, mx, acc);
        st.sum += weights(s, cm, ca, st);
#pragma unroll
        for (int rc = 0; rc < 2; ++rc) {
            const typename E::Frag pf = L::pack(s, rc);
#pragma unroll
            for (int cb = 0; cb < ND; ++cb)
                acc[cb] = E::mfma(L::frag_cols(vt, 16 * rc, cb, lane), pf, acc[cb]);
        }
    }

    // join the four waves' results: [wave][element][row] in the tiles' memory
    st.sum = half_sum(st.sum);
    __syncthreads();
    float* buf = (float*)&tiles[0][0][0];
#pragma unroll
    for (int cb = 0; cb < ND; ++cb)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            buf[(wid * DP + 32 * cb + 8 * (r >> 2) + 4 * h + (r & 3)) * 32 + (lane & 31)] = acc[cb][r];
    if (h == 0) {
        wref[wid][lane] = st.ref;
        wsum[wid][lane] = st.sum;
    }
    __syncthreads();
    const int q = t & 31;
    const int orho = rb * 32 + q;
    if (orho >= rows) return;
    const int og = orho / a.n, oi = orho - og * a.n, ohead = kvh * a.G + og;
    const bool ok = oi < attn_q_len(a, b);
    float ref = -INFINITY;
#pragma unroll
    for (int x = 0; x < 4; ++x) ref = fmaxf(ref, wref[x][q]);
    float f[4], sum = 0.f;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        f[x] = wref[x][q] == -INFINITY ? 0.f : ex2(wref[x][q] - ref);
        sum += wref[x][q] == -INFINITY ? 0.f : wsum[x][q] * f[x];
    }
    if (!ok) sum = 0.f;
    const bool some = !(sum == 0.f);
    const bool last = a.n_split == 1;
    const float inv = !some ? 0.f : last ? 1.f / sum : 1.f;
    const int64_t prow = (int64_t)(b * a.H + ohead) * a.n + oi;
    const int64_t prows = (int64_t)a.B * a.H * a.n;
    T* o = (T*)a.o.p + b * a.o.sb + (int64_t)oi * a.o.sr + ohead * a.o.sh;
    float* po = a.part_o + (split * prows + prow) * a.dv;
    for (int x = (t >> 5) * 4; x < a.dv; x += 32) {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y[e] = 0.f;
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (wref[v][q] != -INFINITY) y[e] = fmaf(buf[(v * DP + x + e) * 32 + q], f[v], y[e]);
            y[e] = some ? y[e] * inv : 0.f;
        }
        if (last) {
            store4<OP>(o, x, a.dv, a.o.vec, y[0], y[1], y[2], y[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (x + e < a.dv) po[x + e] = y[e];
        }
    }
    if (t < 32) {
        if (!last)
            a.part_ml[split * prows + prow] = make_float2(some ? ref : -INFINITY, sum);
        else if (a.lse)
            a.lse[prow] = some ? (ref + lg2(sum)) * kLn2 : -INFINITY;
    }
}

// Joins the key ranges' results of one row (32 lanes a row, a fixed order).
template <int OP>
__global__ __launch_bounds__(256) void attn_merge_kernel(const AttnArgs a) {
    using T = typename El<OP>::T;
    const int64_t rows = (int64_t)a.B * a.H * a.n;
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    float ref = -INFINITY;
    for (int s = 0; s < a.n_split; ++s) ref = fmaxf(ref, a.part_ml[s * rows + row].x);
    float sum = 0.f;
    for (int s = 0; s < a.n_split; ++s) {
        const float2 ml = a.part_ml[s * rows + row];
        if (ml.x != -INFINITY) sum = fmaf(ml.y, ex2(ml.x - ref), sum);
    }
    const bool some = !(sum == 0.f);
    const float inv = some ? 1.f / sum : 0.f;
    const int i = (int)(row % a.n);
    const int64_t bh = row / a.n;
    const int head = (int)(bh % a.H), b = (int)(bh / a.H);
    T* o = (T*)a.o.p + b * a.o.sb + (int64_t)i * a.o.sr + head * a.o.sh;
    for (int x = lane; x < a.dv; x += 32) {
        float y = 0.f;
        for (int s = 0; s < a.n_split; ++s) {
            const float2 ml = a.part_ml[s * rows + row];
            if (ml.x != -INFINITY)
                y = fmaf(a.part_o[(s * rows + row) * a.dv + x], ex2(ml.x - ref), y);
        }
        o[x] = (T)(some ? y * inv : 0.f);
    }
    if (a.lse && lane == 0) a.lse[row] = some ? (ref + lg2(sum)) * kLn2 : -INFINITY;
}

template <int OP, int DP>
hipError_t fwd(const AttnArgs& a, bool few, hipStream_t s) {
    if (few) {
        const int64_t g = (int64_t)a.B * a.K * a.n_split * (((int64_t)a.G * a.n + 31) / 32);
        if (a.bias)
            attn_rows_kernel<OP, DP, true><<<(unsigned)g, 256, 0, s>>>(a);
        else
            attn_rows_kernel<OP, DP, false><<<(unsigned)g, 256, 0, s>>>(a);
    } else {
        const int64_t g = (int64_t)a.B * a.H * a.n_split * ((a.n + kAttnRows - 1) / kAttnRows);
        if (a.bias)
            attn_fwd_kernel<OP, DP, true><<<(unsigned)g, 256, 0, s>>>(a);
        else
            attn_fwd_kernel<OP, DP, false><<<(unsigned)g, 256, 0, s>>>(a);
    }
    return hipGetLastError();
}

hipError_t dispatch(const AttnArgs& a, bool few, hipStream_t s) {
    const int w = a.d > a.dv ? a.d : a.dv;
    switch (a.op) {
        case OP_BF16:
            return w <= 64    ? fwd<OP_BF16, 64>(a, few, s)
                   : w <= 128 ? fwd<OP_BF16, 128>(a, few, s)
                              : fwd<OP_BF16, 256>(a, few, s);
        case OP_F16:
            return w <= 64    ? fwd<OP_F16, 64>(a, few, s)
                   : w <= 128 ? fwd<OP_F16, 128>(a, few, s)
                              : fwd<OP_F16, 256>(a, few, s);
        default:
            return w <= 64 ? fwd<OP_F32, 64>(a, few, s) : fwd<OP_F32, 128>(a, few, s);
    }
}

}  // namespace

hipError_t launch_attn_fwd(const AttnArgs& a, hipStream_t s) { return dispatch(a, false, s); }
hipError_t launch_attn_rows(const AttnArgs& a, hipStream_t s) { return dispatch(a, true, s); }

hipError_t launch_attn_merge(const AttnArgs& a, hipStream_t s) {
    const int64_t rows = (int64_t)a.B * a.H * a.n;
    const unsigned g = (unsigned)((rows + 7) / 8);
    if (a.op == OP_BF16)
        attn_merge_kernel<OP_BF16><<<g, 256, 0, s>>>(a);
    else if (a.op == OP_F16)
        attn_merge_kernel<OP_F16><<<g, 256, 0, s>>>(a);
    else
        attn_merge_kernel<OP_F32><<<g, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace fs
