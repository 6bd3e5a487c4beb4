// fs_attn_bwd.hip -- gradients of the attention of fs_attn_fwd.hip.  With
// P_ij = exp(s_ij - L_i) formed again from the scores and the stored L,
//   delta_i = do_i.o_i - dL_i,     dS_ij = P_ij (do_i.v_j - delta_i),
//   dV_j = sum_i P_ij do_i,        dK_j = scale sum_i dS_ij q_i,
//   dQ_i = scale sum_j dS_ij k_j,  dT[c] = sum of dS over the pairs of bucket c.
// Two passes, one over queries for a resident block of keys (dK, dV) and one
// over keys for a resident block of queries (dQ, dT): seven products instead
// of five, but every sum is formed in one place in a fixed order, so equal
// calls give equal bits.
#include "fs_attn.hpp"

namespace fs {

namespace {

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

// ---- delta ----------------------------------------------------------------
// 16 lanes a row.
template <int OP>
__global__ __launch_bounds__(256) void attn_delta_kernel(const AttnArgs a) {
    using T = typename El<OP>::T;
    constexpr int EPC = 16 / sizeof(T);
    const int64_t rows = (int64_t)a.B * a.n * a.H;
    const int64_t r = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
    const int lane = threadIdx.x & 15;
    if (r >= rows) return;
    const int head = (int)(r % a.H);
    const int64_t bi = r / a.H;
    const int i = (int)(bi % a.n), b = (int)(bi / a.n);
    const T* o = (const T*)a.o.p + b * a.o.sb + (int64_t)i * a.o.sr + head * a.o.sh;
    const T* g = (const T*)a.go.p + b * a.go.sb + (int64_t)i * a.go.sr + head * a.go.sh;
    const bool ok = i < attn_q_len(a, b);
    float s = 0.f;
    if (ok)
        for (int x = lane * EPC; x < a.dv; x += 16 * EPC) {
            T p[EPC], q[EPC];
            load_elems<OP, EPC>(o, x, a.dv, a.o.vec, p);
            load_elems<OP, EPC>(g, x, a.dv, a.go.vec, q);
#pragma unroll
            for (int e = 0; e < EPC; ++e) s = fmaf((float)p[e], (float)q[e], s);
        }
#pragma unroll
    for (int m = 8; m >= 1; m >>= 1) s += __shfl_xor(s, m, 64);
    if (lane == 0) {
        const int64_t at = ((int64_t)b * a.H + head) * a.n + i;
        a.delta[at] = ok ? s - (a.glse ? a.glse[at] : 0.f) : 0.f;
    }
}

// ---- rounding of dS -------------------------------------------------------
// dS goes into its product in the element type.  Its size follows the
// gradient's, which fp16's exponents need not hold, so for fp16 every column
// (a lane pair) carries a power of two that keeps its largest value so far
// between 2^6 and 2^15, and the sums are divided by it at the end.  P is at
// most 1 and is lifted by 2^14 (fp16).
template <int OP>
constexpr float kLiftP = OP == OP_F16 ? 16384.f : 1.f;

template <int OP, int ND>
struct DsScale {
    float f = 1.f;
    bool set = false;
    __device__ __forceinline__ void apply(f32x16& ds, f32x16 (&acc)[ND]) {
        if constexpr (OP == OP_F16) {
            float mx = 0.f;
#pragma unroll
            for (int r = 0; r < 16; ++r) mx = fmaxf(mx, fabsf(ds[r]));
            mx = half_max(mx);
            const bool low = !set && mx > 0.f && mx < INFINITY;
            const bool high = mx * f > 32768.f && mx < INFINITY;
            if (__any(low || high)) {
                // the power of two that puts mx at 2^10 .. 2^11
                const float to =
                    low || high ? ldexpf(1.f, min(10 - ilogbf(mx), 100)) : f;
                const float k = to / f;
                if (low || high) {
                    if (set) {
#pragma unroll
                        for (int x = 0; x < ND; ++x)
#pragma unroll
                            for (int r = 0; r < 16; ++r) acc[x][r] *= k;
                    }
                    f = to;
                    set = true;
                }
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) ds[r] *= f;
        }
    }
    __device__ __forceinline__ float undo() const { return 1.f / f; }
};

template <int OP, int DP>
constexpr int kBwdTile = DP * (int)sizeof(typename El<OP>::T) <= 256 ? 64 : 32;

// ---- dK, dV ---------------------------------------------------------------
// A workgroup holds 128 keys of one key head, 32 a wave, as operands, and
// passes over the queries of every head of the group in tiles staged in LDS.
// Scores are formed with queries in the rows, so a lane holds one key's
// column: a key that is masked out spoils nothing but its own column, which
// is written as zero, and needs no test in the loop.
template <int OP, int DP, bool BIAS>
__global__ __launch_bounds__(256, 1) void attn_bwd_kv_kernel(const AttnArgs a) {
    using E = El<OP>;
    using T = typename E::T;
    using L = Tile<OP, DP>;
    constexpr int QT = 32, ND = DP / 32, NK = DP / 16;
    __shared__ __attribute__((aligned(256))) char qt[QT * L::kRow];
    __shared__ __attribute__((aligned(256))) char gt[QT * L::kRow];
    __shared__ __attribute__((aligned(16))) float row_l[QT], row_d[QT];
    __shared__ float line[BIAS ? 2 * kAttnMaxEdge + 1 : 1];

    const int t = threadIdx.x, lane = t & 63, wid = t >> 6, h = lane >> 5;
    const int nkb = (a.m + kAttnRows - 1) / kAttnRows;
    int w = xcd_item(blockIdx.x, gridDim.x);
    const int kb = w % nkb;
    w /= nkb;
    const int split = w % a.q_split;
    w /= a.q_split;
    const int kvh = w % a.K, b = w / a.K;

    const int off = attn_offset(a, b);
    const int len = attn_kv_len(a, b);
    const int qlen = attn_q_len(a, b);
    const int j0 = kb * kAttnRows + wid * 32, j = j0 + (lane & 31);
    bool key_ok = j < len;
    if (key_ok && a.key_mask) key_ok = a.key_mask[b * a.mask_stride + j] != 0;

    typename E::Frag kf[NK], vf[NK];
    load_row_frags<OP, DP>((const T*)a.k.p + b * a.k.sb + (int64_t)j * a.k.sr + kvh * a.k.sh,
                           key_ok, a.d, a.k.vec, lane, kf);
    load_row_frags<OP, DP>((const T*)a.v.p + b * a.v.sb + (int64_t)j * a.v.sr + kvh * a.v.sh,
                           key_ok, a.dv, a.v.vec, lane, vf);
    f32x16 dk[ND], dvv[ND];
#pragma unroll
    for (int x = 0; x < ND; ++x)
#pragma unroll
        for (int r = 0; r < 16; ++r) dk[x][r] = dvv[x][r] = 0.f;
    DsScale<OP, ND> dss;

    // the first query that sees a key of this block
    int first = split * a.split_rows;
    const int end = a.q_split == 1 ? qlen : min(qlen, first + a.split_rows);
    if (a.causal) first = max(first, (max(0, kb * kAttnRows - off) / QT) * QT);
    if (kb * kAttnRows >= len) first = end;

    for (int g = 0; g < a.G; ++g) {
        const int head = kvh * a.G + g;
        const T* qbase = (const T*)a.q.p + b * a.q.sb + head * a.q.sh;
        const T* gbase = (const T*)a.go.p + b * a.go.sb + head * a.go.sh;
        const int64_t lrow = ((int64_t)b * a.H + head) * a.n;
        if (BIAS) {
            __syncthreads();
            load_line(a, head, line, t, 256);
        }
        Stage<OP, DP, QT, 256> qs, gs;
        float nl = 0.f, nd = 0.f;
        auto fetch = [&](int i0) {
            const uint64_t seen = bits_upto(end - 1 - i0);
            qs.load(qbase + (int64_t)i0 * a.q.sr, a.q.sr, seen, a.d, a.q.vec, t);
            gs.load(gbase + (int64_t)i0 * a.go.sr, a.go.sr, seen, a.dv, a.go.vec, t);
            if (t < QT) {
                const bool ok = i0 + t < end;
                nl = ok ? a.lse[lrow + i0 + t] : -INFINITY;
                nd = ok ? a.delta[lrow + i0 + t] : 0.f;
            }
        };
        if (first < end) fetch(first);
        for (int i0 = first; i0 < end; i0 += QT) {
            __syncthreads();
            qs.store(qt, t);
            gs.store(gt, t);
            if (t < QT) {
                // a row without keys gives no weight: 2^(s - inf) = 0
                row_l[t] = nl == -INFINITY ? -INFINITY : -nl * kLog2e;
                row_d[t] = nd;
            }
            __syncthreads();
            if (i0 + QT < end) fetch(i0 + QT);

            f32x16 s, dp;
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.f;
#pragma unroll
            for (int kk = 0; kk < NK; ++kk) s = E::mfma(L::frag_rows(qt, 0, kk, lane), kf[kk], s);
#pragma unroll
            for (int kk = 0; kk < NK; ++kk) dp = E::mfma(L::frag_rows(gt, 0, kk, lane), vf[kk], dp);
            float rl[16], rd[16];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x4 x = *(const f32x4*)&row_l[8 * q + 4 * h];
                const f32x4 y = *(const f32x4*)&row_d[8 * q + 4 * h];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    rl[4 * q + r] = x[r];
                    rd[4 * q + r] = y[r];
                }
            }
            if (BIAS) {
                const int lo = j0 - i0 - (QT - 1) - off, hi = j0 + 31 - i0 - off;
                if (hi <= -a.r0) {
                    const float ca = line[0];
#pragma unroll
                    for (int r = 0; r < 16; ++r) rl[r] += ca;
                } else if (lo >= a.rp) {
                    const float ca = line[a.r0 + a.rp];
#pragma unroll
                    for (int r = 0; r < 16; ++r) rl[r] += ca;
                } else {
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        rl[r] += line[line_index(a, j - (i0 + 8 * (r >> 2) + 4 * h + (r & 3)) - off)];
                }
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = ex2(fmaf(s[r], a.c, rl[r]));
            if (a.causal) {
                // queries from j - off on see key j
                const uint32_t vis = ~bits_upto(j - off - i0 - 1) >> (4 * h);
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = flag(vis, r) ? s[r] : 0.f;
            }
            f32x16 ds;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                ds[r] = s[r] * (dp[r] - rd[r]);
                s[r] *= kLiftP<OP>;
            }
            dss.apply(ds, dk);
#pragma unroll
            for (int rc = 0; rc < 2; ++rc) {
                const typename E::Frag pf = L::pack(s, rc), df = L::pack(ds, rc);
#pragma unroll
                for (int cb = 0; cb < ND; ++cb) {
                    dvv[cb] = E::mfma(L::frag_cols(gt, 16 * rc, cb, lane), pf, dvv[cb]);
                    dk[cb] = E::mfma(L::frag_cols(qt, 16 * rc, cb, lane), df, dk[cb]);
                }
            }
        }
    }

    if (j >= a.m) return;
    const float fk = a.scale * dss.undo(), fv = 1.f / kLiftP<OP>;
    if (a.q_split > 1) {
        const int64_t row = ((int64_t)b * a.K + kvh) * a.m + j;
        const int64_t rows = (int64_t)a.B * a.K * a.m;
        float* pk = a.part_k + (split * rows + row) * a.d;
        float* pv = a.part_v + (split * rows + row) * a.dv;
#pragma unroll
        for (int cb = 0; cb < ND; ++cb)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int x = 32 * cb + 8 * (r >> 2) + 4 * h + (r & 3);
                if (x < a.d) pk[x] = key_ok ? dk[cb][r] * fk : 0.f;
                if (x < a.dv) pv[x] = key_ok ? dvv[cb][r] * fv : 0.f;
            }
        return;
    }
    T* ok = (T*)a.gk.p + b * a.gk.sb + (int64_t)j * a.gk.sr + kvh * a.gk.sh;
    T* ov = (T*)a.gv.p + b * a.gv.sb + (int64_t)j * a.gv.sr + kvh * a.gv.sh;
#pragma unroll
    for (int cb = 0; cb < ND; ++cb)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float y[4], z[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                y[r] = key_ok ? dk[cb][4 * q + r] * fk : 0.f;
                z[r] = key_ok ? dvv[cb][4 * q + r] * fv : 0.f;
            }
            if (a.gk.p) store4<OP>(ok, 32 * cb + 8 * q + 4 * h, a.d, a.gk.vec, y[0], y[1], y[2], y[3]);
            if (a.gv.p) store4<OP>(ov, 32 * cb + 8 * q + 4 * h, a.dv, a.gv.vec, z[0], z[1], z[2], z[3]);
        }
}

// Sums the query ranges' parts of dK and dV (a fixed order).
template <int OP>
__global__ __launch_bounds__(256) void attn_kv_merge_kernel(const AttnArgs a) {
    using T = typename El<OP>::T;
    const int64_t rows = (int64_t)a.B * a.K * a.m;
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    const int j = (int)(row % a.m);
    const int64_t bk = row / a.m;
    const int kvh = (int)(bk % a.K), b = (int)(bk / a.K);
    if (a.gk.p) {
        T* o = (T*)a.gk.p + b * a.gk.sb + (int64_t)j * a.gk.sr + kvh * a.gk.sh;
        for (int x = lane; x < a.d; x += 32) {
            float y = 0.f;
            for (int s = 0; s < a.q_split; ++s) y += a.part_k[(s * rows + row) * a.d + x];
            o[x] = (T)y;
        }
    }
    if (a.gv.p) {
        T* o = (T*)a.gv.p + b * a.gv.sb + (int64_t)j * a.gv.sr + kvh * a.gv.sh;
        for (int x = lane; x < a.dv; x += 32) {
            float y = 0.f;
            for (int s = 0; s < a.q_split; ++s) y += a.part_v[(s * rows + row) * a.dv + x];
            o[x] = (T)y;
        }
    }
}

// ---- dQ, dT ---------------------------------------------------------------
// The mirror image: 128 query rows of a head, 32 a wave, keys in tiles, keys
// in the rows of the scores.  Here a masked key does enter sums over keys, so
// its weight is set to zero.
//
// Bias gradient: dS summed over the pairs of every relative position r, and
// those sums over each bucket by attn_bias_sum_kernel.  A tile whose pairs all
// lie beyond the last edge goes into one of two running sums of the lane.  In
// a tile near the diagonal a wave writes each 32 x 32 block to its own LDS
// with query x's row moved by x, so that a relative position is a column, and
// 63 lanes sum a column each; positions between the last edges are added to
// the wave's line in LDS (one lane a position), those beyond to the lane's
// running sums.
constexpr int kDiag = 64;
template <int OP, int DP, bool BIAS>
__global__ __launch_bounds__(256, 1) void attn_bwd_q_kernel(const AttnArgs a) {
    using E = El<OP>;
    using T = typename E::T;
    using L = Tile<OP, DP>;
    constexpr int KT = kBwdTile<OP, DP>, NB = KT / 32, ND = DP / 32, NK = DP / 16;
    constexpr int kLine = 2 * kAttnMaxEdge + 1;
    __shared__ __attribute__((aligned(256))) char kt[KT * L::kRow];
    __shared__ __attribute__((aligned(256))) char vt[KT * L::kRow];
    __shared__ float line[BIAS ? kLine : 1];
    __shared__ float diag[BIAS ? 4 : 1][BIAS ? 32 * kDiag : 1];
    __shared__ float gline[BIAS ? 4 : 1][BIAS ? kLine : 1];

    const int t = threadIdx.x, lane = t & 63, wid = t >> 6, h = lane >> 5;
    const int nqb = (a.n + kAttnRows - 1) / kAttnRows;
    int w = xcd_item(blockIdx.x, gridDim.x);
    const int qb = w % nqb;
    w /= nqb;
    const int head = w % a.H, b = w / a.H, kvh = head / a.G;
    const int n_line = a.r0 + a.rp + 1;

    const int off = attn_offset(a, b);
    const int i0 = qb * kAttnRows + wid * 32, i = i0 + (lane & 31);
    const bool row_ok = i < attn_q_len(a, b);
    int len = attn_kv_len(a, b);
    if (a.causal) len = min(len, max(0, min(qb * kAttnRows + kAttnRows, a.n) + off));

    if (BIAS) {
        load_line(a, head, line, t, 256);
        if (a.gbias) {
            for (int x = lane; x < n_line; x += 64) gline[wid][x] = 0.f;
            for (int x = lane; x < 32 * kDiag; x += 64) diag[wid][x] = 0.f;
        }
    }
    typename E::Frag qf[NK], gf[NK];
    load_row_frags<OP, DP>((const T*)a.q.p + b * a.q.sb + (int64_t)i * a.q.sr + head * a.q.sh,
                           row_ok, a.d, a.q.vec, lane, qf);
    load_row_frags<OP, DP>((const T*)a.go.p + b * a.go.sb + (int64_t)i * a.go.sr + head * a.go.sh,
                           row_ok, a.dv, a.go.vec, lane, gf);
    const int64_t lrow = ((int64_t)b * a.H + head) * a.n;
    const float lse = row_ok ? a.lse[lrow + i] : -INFINITY;
    const float rl = lse == -INFINITY ? -INFINITY : -lse * kLog2e;
    const float rd = row_ok ? a.delta[lrow + i] : 0.f;
    f32x16 acc[ND];
#pragma unroll
    for (int x = 0; x < ND; ++x)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[x][r] = 0.f;
    DsScale<OP, ND> dss;
    float sum_lo = 0.f, sum_hi = 0.f;

    const T* kbase = (const T*)a.k.p + b * a.k.sb + kvh * a.k.sh;
    const T* vbase = (const T*)a.v.p + b * a.v.sb + kvh * a.v.sh;
    Stage<OP, DP, KT, 256> ks, vs;
    uint64_t next = 0;
    auto fetch = [&](int j0) {
        next = seen_keys(a, b, len, j0, lane);
        ks.load(kbase + (int64_t)j0 * a.k.sr, a.k.sr, next, a.d, a.k.vec, t);
        vs.load(vbase + (int64_t)j0 * a.v.sr, a.v.sr, next, a.dv, a.v.vec, t);
    };
    if (len > 0) fetch(0);
    for (int j0 = 0; j0 < len; j0 += KT) {
        const uint64_t seen = next;
        __syncthreads();
        ks.store(kt, t);
        vs.store(vt, t);
        __syncthreads();
        if (j0 + KT < len) fetch(j0 + KT);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int jb = j0 + 32 * nb;
            uint32_t vis = (uint32_t)(seen >> (32 * nb));
            if (a.causal) vis &= bits_upto(i + off - jb);
            const bool all = __all(vis == ~0u);
            vis >>= 4 * h;
            f32x16 s, dp;
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.f;
#pragma unroll
            for (int kk = 0; kk < NK; ++kk) s = E::mfma(L::frag_rows(kt, 32 * nb, kk, lane), qf[kk], s);
#pragma unroll
            for (int kk = 0; kk < NK; ++kk) dp = E::mfma(L::frag_rows(vt, 32 * nb, kk, lane), gf[kk], dp);
            bool lo_far = false, hi_far = false;
            if (BIAS) {
                const int lo = jb - i0 - 31 - off, hi = jb + 31 - i0 - off;
                lo_far = hi <= -a.r0;
                hi_far = !lo_far && lo >= a.rp;
            }
            if (BIAS && !lo_far && !hi_far) {
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    s[r] = ex2(fmaf(s[r], a.c,
                                    rl + line[line_index(a, jb + 8 * (r >> 2) + 4 * h + (r & 3) - i - off)]));
            } else {
                const float ca = rl + (BIAS ? line[lo_far ? 0 : n_line - 1] : 0.f);
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = ex2(fmaf(s[r], a.c, ca));
            }
            f32x16 ds;
#pragma unroll
            for (int r = 0; r < 16; ++r) ds[r] = s[r] * (dp[r] - rd);
            if (!all) {
#pragma unroll
                for (int r = 0; r < 16; ++r) ds[r] = flag(vis, r) ? ds[r] : 0.f;
            }
            if (BIAS && a.gbias) {
                if (lo_far || hi_far) {
                    float x = 0.f;
#pragma unroll
                    for (int r = 0; r < 16; ++r) x += ds[r];
                    if (lo_far) sum_lo += x;
                    else sum_hi += x;
                } else {
                    float* dg = diag[wid];
                    const int q = lane & 31;
                    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        dg[q * kDiag + 8 * (r >> 2) + 4 * h + (r & 3) - q + 31] = ds[r];
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                    float x = 0.f;
#pragma unroll
                    for (int y = 0; y < 32; ++y) x += dg[y * kDiag + lane];
                    const int r = jb - i0 - 31 - off + lane;  // lane 63: no pair, x = 0
                    if (r <= -a.r0) sum_lo += x;
                    else if (r >= a.rp) sum_hi += x;
                    else gline[wid][r + a.r0] += x;
                    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                }
            }
            dss.apply(ds, acc);
#pragma unroll
            for (int rc = 0; rc < 2; ++rc) {
                const typename E::Frag df = L::pack(ds, rc);
#pragma unroll
                for (int cb = 0; cb < ND; ++cb)
                    acc[cb] = E::mfma(L::frag_cols(kt, 32 * nb + 16 * rc, cb, lane), df, acc[cb]);
            }
        }
    }

    if (BIAS && a.gbias) {
        sum_lo = wave_sum(sum_lo);
        sum_hi = wave_sum(sum_hi);
        if (lane == 0) {
            // both ends are one bucket each; with no edges they are one entry
            gline[wid][0] += sum_lo;
            gline[wid][n_line - 1] += sum_hi;
        }
        __syncthreads();
        float* part = a.line_part + ((int64_t)head * a.B * nqb + (int64_t)b * nqb + qb) * n_line;
        for (int x = t; x < n_line; x += 256)
            part[x] = (gline[0][x] + gline[1][x]) + (gline[2][x] + gline[3][x]);
    }
    if (i >= a.n || !a.gq.p) return;
    const float f = a.scale * dss.undo();
    T* o = (T*)a.gq.p + b * a.gq.sb + (int64_t)i * a.gq.sr + head * a.gq.sh;
#pragma unroll
    for (int cb = 0; cb < ND; ++cb)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float y[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) y[r] = row_ok ? acc[cb][4 * q + r] * f : 0.f;
            store4<OP>(o, 32 * cb + 8 * q + 4 * h, a.d, a.gq.vec, y[0], y[1], y[2], y[3]);
        }
}

// dT[bucket, head]: the bucket's positions of every part's line, in 64 bits
// and a fixed order.  One workgroup per entry.
__global__ __launch_bounds__(256) void attn_bias_sum_kernel(const AttnArgs a) {
    __shared__ double red[256];
    const int bucket = blockIdx.x, head = blockIdx.y, t = threadIdx.x;
    const int n_line = a.r0 + a.rp + 1;
    const int parts = a.B * ((a.n + kAttnRows - 1) / kAttnRows);
    // the line positions of this bucket: distances [from, to), on one side
    const int E1 = a.n_edges + 1;
    const bool after = a.two_sided && bucket >= E1;
    const int c = after ? bucket - E1 : bucket;
    const int from = c == 0 ? 0 : (int)a.edges[c - 1];
    const int to = c == a.n_edges ? a.r0 + 1 : (int)a.edges[c];  // the line ends at r0
    int lo, hi;  // line indices [lo, hi)
    if (after) {
        lo = a.r0 + max(from, 1);
        hi = a.r0 + to;
        if (c == a.n_edges) hi = n_line;
    } else {
        lo = a.r0 - to + 1;
        hi = a.r0 - from + 1;
    }
    lo = max(lo, 0);
    hi = min(hi, n_line);
    double s = 0.0;
    const float* base = a.line_part + (int64_t)head * parts * n_line;
    for (int x = lo + (t & 31); x < hi; x += 32)
        for (int p = t >> 5; p < parts; p += 8) s += (double)base[(int64_t)p * n_line + x];
    red[t] = s;
    __syncthreads();
    for (int o = 128; o >= 1; o >>= 1) {
        if (t < o) red[t] += red[t + o];
        __syncthreads();
    }
    if (t == 0) a.gbias[(int64_t)bucket * a.H + head] = (float)red[0];
}

template <int OP, int DP>
hipError_t bwd_kv(const AttnArgs& a, hipStream_t s) {
    const int64_t g = (int64_t)a.B * a.K * a.q_split * ((a.m + kAttnRows - 1) / kAttnRows);
    if (a.bias)
        attn_bwd_kv_kernel<OP, DP, true><<<(unsigned)g, 256, 0, s>>>(a);
    else
        attn_bwd_kv_kernel<OP, DP, false><<<(unsigned)g, 256, 0, s>>>(a);
    return hipGetLastError();
}

template <int OP, int DP>
hipError_t bwd_q(const AttnArgs& a, hipStream_t s) {
    const int64_t g = (int64_t)a.B * a.H * ((a.n + kAttnRows - 1) / kAttnRows);
    if (a.bias)
        attn_bwd_q_kernel<OP, DP, true><<<(unsigned)g, 256, 0, s>>>(a);
    else
        attn_bwd_q_kernel<OP, DP, false><<<(unsigned)g, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

#define FS_ATTN_DISPATCH(FN)                                                              \
    const int w = a.d > a.dv ? a.d : a.dv;                                                \
    switch (a.op) {                                                                       \
        case OP_BF16:                                                                     \
            return w <= 64    ? FN<OP_BF16, 64>(a, s)                                     \
                   : w <= 128 ? FN<OP_BF16, 128>(a, s)                                    \
                              : FN<OP_BF16, 256>(a, s);                                   \
        case OP_F16:                                                                      \
            return w <= 64    ? FN<OP_F16, 64>(a, s)                                      \
                   : w <= 128 ? FN<OP_F16, 128>(a, s)                                     \
                              : FN<OP_F16, 256>(a, s);                                    \
        default:                                                                          \
            return w <= 64 ? FN<OP_F32, 64>(a, s) : FN<OP_F32, 128>(a, s);                \
    }

hipError_t launch_attn_bwd_kv(const AttnArgs& a, hipStream_t s) { FS_ATTN_DISPATCH(bwd_kv) }
hipError_t launch_attn_bwd_q(const AttnArgs& a, hipStream_t s) { FS_ATTN_DISPATCH(bwd_q) }

hipError_t launch_attn_delta(const AttnArgs& a, hipStream_t s) {
    const int64_t rows = (int64_t)a.B * a.n * a.H;
    const unsigned g = (unsigned)((rows + 15) / 16);
    if (a.op == OP_BF16)
        attn_delta_kernel<OP_BF16><<<g, 256, 0, s>>>(a);
    else if (a.op == OP_F16)
        attn_delta_kernel<OP_F16><<<g, 256, 0, s>>>(a);
    else
        attn_delta_kernel<OP_F32><<<g, 256, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_attn_kv_merge(const AttnArgs& a, hipStream_t s) {
    const int64_t rows = (int64_t)a.B * a.K * a.m;
    const unsigned g = (unsigned)((rows + 7) / 8);
    if (a.op == OP_BF16)
        attn_kv_merge_kernel<OP_BF16><<<g, 256, 0, s>>>(a);
    else if (a.op == OP_F16)
        attn_kv_merge_kernel<OP_F16><<<g, 256, 0, s>>>(a);
    else
        attn_kv_merge_kernel<OP_F32><<<g, 256, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_attn_bias_sum(const AttnArgs& a, hipStream_t s) {
    const unsigned buckets = (unsigned)((a.n_edges + 1) * (a.two_sided ? 2 : 1));
    attn_bias_sum_kernel<<<dim3(buckets, (unsigned)a.H), 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace fs
