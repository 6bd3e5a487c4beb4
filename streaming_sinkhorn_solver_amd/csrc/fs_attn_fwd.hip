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

// ---- many query rows ------------------------------------------------------
// A workgroup of four waves takes 128 query rows of one head, 32 a wave, and
// a range of keys in tiles of KT staged through LDS and shared by the waves.
// Scores are formed with keys in the rows (S^T = K Q^T), so a lane holds
// scores of one query row: maximum and sum need one exchange, between the
// halves of the wave, and the weights are operands of O^T = V^T P^T as they
// are.
//
// What the two forms below share: a lane's query row, its range of keys, the
// scores made ready and the output.
template <int OP, int DP, bool BIAS>
struct FwdPass {
    using E = El<OP>;
    using T = typename E::T;
    using L = Tile<OP, DP>;
    static constexpr int ND = DP / 32, NK = DP / 16;
    int lane, wid, h, split, head, b, kvh, off, i0, i, jb, je;
    bool row_ok;
    LdsFloats line;

    __device__ __forceinline__ FwdPass(const AttnArgs& a, float* line_mem) {
        lane = threadIdx.x & 63, wid = wave_id(), h = lane >> 5;
        const int nqb = (a.n + kAttnRows - 1) / kAttnRows;
        int w = xcd_item(blockIdx.x, gridDim.x, a.G * a.n_split * nqb);
        const int qb = w % nqb;
        w /= nqb;
        split = w % a.n_split;
        w /= a.n_split;
        head = w % a.H, b = w / a.H, kvh = head / a.G;
        line.a = lds_addr(line_mem);
        off = attn_offset(a, b);
        i0 = qb * kAttnRows + wid * 32, i = i0 + (lane & 31);
        const int qlen = attn_q_len(a, b);
        row_ok = i < qlen;
        int len = attn_kv_len(a, b);
        // (keys that only rows behind qlen would see are not read)
        if (a.causal) len = min(len, max(0, min(qb * kAttnRows + kAttnRows, qlen) + off));
        jb = split * a.split_keys;
        je = a.n_split == 1 ? len : min(len, jb + a.split_keys);
    }
    // NB blocks of 32 scores from key j0 on, ready for s cm + ca: the bias in,
    // hidden keys at -inf.
    template <int NB>
    __device__ __forceinline__ void prepare(const AttnArgs& a, int j0, uint64_t word, f32x16 (&s)[NB],
                                            float& cm, float& ca) const {
        uint32_t vis[NB];
        bool all = true;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            vis[nb] = (uint32_t)(word >> (32 * nb));
            if (a.causal) vis[nb] &= bits_upto(i + off - (j0 + 32 * nb));
            all = all && vis[nb] == ~0u;
            vis[nb] >>= 4 * h;
        }
        all = __all(all);
        cm = a.c, ca = 0.f;
        if (BIAS) {
            const int lo = j0 - i0 - 31 - off, hi = j0 + 32 * NB - 1 - i0 - off;
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
            asm volatile("");  // a branch: most tiles need none of it
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int r = 0; r < 16; ++r) s[nb][r] = flag(vis[nb], r) ? s[nb][r] : -INFINITY;
        }
    }
    // Moves the reference up to the scores' maximum where it has to.
    template <int NB>
    __device__ __forceinline__ void raise(const f32x16 (&s)[NB], float cm, float ca, Run& st,
                                          f32x16 (&acc)[ND]) const {
        float mx = -INFINITY;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[nb][r]);
        mx = fmaf(half_max(mx), cm, ca);
        raise_ref<OP, ND>(st, mx, acc);
    }
    __device__ __forceinline__ void store(const AttnArgs& a, Run st, const f32x16 (&acc)[ND]) const {
        st.sum = half_sum(st.sum);
        if (i >= a.n) return;
        if (!row_ok) st.sum = 0.f;
        if (a.n_split > 1) {
            const int64_t row = (int64_t)(b * a.H + head) * a.n + i;
            const int64_t rows = (int64_t)a.B * a.H * a.n;
            if (h == 0) a.part_ml[split * rows + row] = make_float2(st.sum == 0.f ? -INFINITY : st.ref, st.sum);
            float* po = a.part_o + (split * rows + row) * a.dv_pad;
#pragma unroll
            for (int cb = 0; cb < ND; ++cb)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int x = 32 * cb + 8 * q + 4 * h;
                    if (x < a.dv)
                        *(f32x4*)(po + x) = f32x4{acc[cb][4 * q], acc[cb][4 * q + 1], acc[cb][4 * q + 2],
                                                  acc[cb][4 * q + 3]};
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
};

// Tiles of 128 keys (rows of 128 bytes), worked on 64 at a time, the next tile
// fetched meanwhile.  Few registers leave two waves a SIMD, and with little
// work per key one barrier for 128 keys costs less than the pipelining of the
// form below gains (2048 x 2048, 16 heads of 64, batch 4, with a bias: 116
// against 132 us).
constexpr int kNarrowAhead = 8;
template <int OP, int DP, bool BIAS>
__global__ __launch_bounds__(256, 2) void attn_fwd_narrow_kernel(const AttnArgs a) {
    using P = FwdPass<OP, DP, BIAS>;
    using E = typename P::E;
    using T = typename P::T;
    using L = typename P::L;
    constexpr int TK = 128, KT = 64, NB = 2, ND = P::ND, NK = P::NK, kBytes = TK * L::kRow;
    using Load = Loader<OP, DP, KT, 256>;
    __shared__ __attribute__((aligned(256))) char tiles[2][2][kBytes];  // keys, values
    __shared__ uint64_t words[128];
    __shared__ float line_mem[BIAS ? 2 * kAttnMaxEdge + 1 : 1];
    const P p(a, line_mem);
    const int t = threadIdx.x, lane = p.lane;
    const T* kbase = (const T*)a.k.p + p.b * a.k.sb + p.kvh * a.k.sh;
    const T* vbase = (const T*)a.v.p + p.b * a.v.sb + p.kvh * a.v.sh;
    const uint32_t tile0 = lds_addr(tiles);
    const SeenKeys<KT, 4> seen{a.key_mask ? a.key_mask + p.b * a.mask_stride : nullptr, lds_addr(words),
                               p.jb, KT, p.je};
    const auto fetch = [&](int jt, int buf) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int64_t j = jt + x * KT;
            const uint64_t word = seen((jt - p.jb) / KT + x);
            const uint32_t lds = tile0 + 2 * buf * kBytes + x * KT * L::kRow;
            Load::fill(lds, kbase + j * a.k.sr, a.k.sr, word, a.d, a.k.vec, t);
            Load::fill(lds + kBytes, vbase + j * a.v.sr, a.v.sr, word, a.dv, a.v.vec, t);
        }
    };
    if (p.jb < p.je) {
        seen.fill(0, lane, p.wid);
        if (a.key_mask) __syncthreads();
        fetch(p.jb, 0);
    }
    if (BIAS) load_line(a, p.head, p.line, t, 256);
    typename E::Frag qf[NK];
    load_row_frags<OP, DP>((const T*)a.q.p + p.b * a.q.sb + (int64_t)p.i * a.q.sr + p.head * a.q.sh,
                           p.row_ok, a.d, a.q.vec, lane, qf);
    f32x16 acc[ND];
#pragma unroll
    for (int x = 0; x < ND; ++x)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[x][r] = 0.f;
    Run st;
    const typename L::Lanes lanes(tile0, lane);
    int cur = 0;
    for (int jt = p.jb; jt < p.je; jt += TK) {
        dma_wait();
        __builtin_amdgcn_s_barrier();
        const int u = (jt - p.jb) / KT;
        if (u % 64 == 0) seen.fill(u + 64, lane, p.wid);
        const typename L::Lanes now(lanes, cur * 2 * kBytes);
        cur ^= 1;
        if (jt + TK < p.je) fetch(jt + TK, cur);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int j0 = jt + x * KT, o = x * KT * L::kRow;
            f32x16 s[NB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int r = 0; r < 16; ++r) s[nb][r] = 0.f;
            constexpr int kScores = NB * NK, kValues = 2 * NB * ND;
            auto prod = products<kNarrowAhead, kScores, kValues, typename E::Frag>([&](int y) {
                if (y < kScores) return L::frag_rows(now, o + 32 * (y % NB) * L::kRow, y / NB);
                y -= kScores;
                return L::frag_cols(now, kBytes + o + 16 * (y / ND) * L::kRow, y % ND);
            });
            prod.first([&](int y, typename E::Frag op) { s[y % NB] = E::mfma(op, qf[y / NB], s[y % NB]); });
            float cm, ca;
            p.prepare(a, j0, seen(u + x), s, cm, ca);
            p.raise(s, cm, ca, st, acc);
            typename E::Frag pf[2 * NB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                st.sum += weights(s[nb], cm, ca, st);
                pf[2 * nb] = L::pack(s[nb], 0);
                pf[2 * nb + 1] = L::pack(s[nb], 1);
            }
            prod.second([&](int y, typename E::Frag op) { acc[y % ND] = E::mfma(op, pf[y / ND], acc[y % ND]); });
        }
    }
    p.store(a, st, acc);
}

// Rows of 256 and 512 bytes: tiles of KT keys, and the steps are pipelined by
// one: the scores of tile u + 1 are issued to the
// matrix cores among the exponentials of tile u, so that both units have work
// of the same wave.  Keys and values stand in rings of R tiles.  At the barrier
// of step u every wave has formed the scores of u and used the values of u - 1,
// so the keys of u + R and the values of u + R - 1 are fetched into those
// places; behind the last tile the fetches go on, of zeros, so that the number
// of copies in flight is always the same.  (4096 x 8192, 32 heads of 128 over 8,
// batch 2: 1125 us, 977 TFLOP/s; 1220 with the products' operands loaded where
// the compiler puts them.)
template <int OP, int DP>
constexpr int kStepKeys = Tile<OP, DP>::kRow <= 256 ? 64 : 32;

template <int OP, int DP, bool BIAS>
__global__ __launch_bounds__(256, (Tile<OP, DP>::kRow <= 256 ? 2 : 1))
void attn_fwd_kernel(const AttnArgs a) {
    using P = FwdPass<OP, DP, BIAS>;
    using E = typename P::E;
    using T = typename P::T;
    using L = typename P::L;
    constexpr int KT = kStepKeys<OP, DP>, NB = KT / 32, ND = P::ND, NK = P::NK;
    using Load = Loader<OP, DP, KT, 256>;
    constexpr int R = 2, kTileBytes = KT * L::kRow;
    __shared__ __attribute__((aligned(256))) char tiles[2 * R][kTileBytes];  // keys, values
    __shared__ uint64_t words[128];
    __shared__ float line_mem[BIAS ? 2 * kAttnMaxEdge + 1 : 1];
    const P p(a, line_mem);
    const int t = threadIdx.x, lane = p.lane, jb = p.jb, je = p.je;
    const T* kbase = (const T*)a.k.p + p.b * a.k.sb + p.kvh * a.k.sh;
    const T* vbase = (const T*)a.v.p + p.b * a.v.sb + p.kvh * a.v.sh;
    const uint32_t tile0 = lds_addr(tiles);
    const SeenKeys<KT, 4> seen{a.key_mask ? a.key_mask + p.b * a.mask_stride : nullptr, lds_addr(words),
                               jb, KT, je};
    const int n_tiles = jb < je ? (je - jb + KT - 1) / KT : 0;
    const auto fetch_k = [&](int u, int place) {
        Load::fill(tile0 + place * kTileBytes, kbase + (jb + (int64_t)u * KT) * a.k.sr, a.k.sr,
                   seen(u), a.d, a.k.vec, t);
    };
    const auto fetch_v = [&](int u, int place) {
        Load::fill(tile0 + (R + place) * kTileBytes, vbase + (jb + (int64_t)u * KT) * a.v.sr, a.v.sr,
                   seen(u), a.dv, a.v.vec, t);
    };
    if (n_tiles) {
        seen.fill(0, lane, p.wid);
        seen.fill(64, lane, p.wid);
        if (a.key_mask) __syncthreads();
        fetch_k(0, 0);
#pragma unroll
        for (int u = 0; u < R - 1; ++u) {
            fetch_v(u, u);
            fetch_k(u + 1, u + 1);
        }
    }
    if (BIAS) load_line(a, p.head, p.line, t, 256);
    typename E::Frag qf[NK];
    load_row_frags<OP, DP>((const T*)a.q.p + p.b * a.q.sb + (int64_t)p.i * a.q.sr + p.head * a.q.sh,
                           p.row_ok, a.d, a.q.vec, lane, qf);
    f32x16 acc[ND];
#pragma unroll
    for (int x = 0; x < ND; ++x)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[x][r] = 0.f;
    Run st;

    const typename L::Lanes lanes(tile0, lane);
    // one tile: s its scores, sn those of the next tile; place: its place
    const auto step = [&](int u, f32x16 (&s)[NB], f32x16 (&sn)[NB], int place) {
        const int j0 = jb + u * KT;
        float cm, ca;
        p.prepare(a, j0, seen(u), s, cm, ca);
        p.raise(s, cm, ca, st, acc);

        dma_wait_but<(R - 2) * 2 * Load::kN>();
        __builtin_amdgcn_s_barrier();
        if (a.key_mask && u % 64 == 0 && u > 0) seen.fill(u + 64, lane, p.wid);
        fetch_v(u + R - 1, (place + R - 1) % R);
        fetch_k(u + R, place);
        // The next tile's scores (behind the last tile: scores that no one
        // uses), this tile's weights and their products with the values, in an
        // order that is written out: operands are read kAhead products ahead,
        // and the sixteen weights of an operand pair are formed between the
        // products, two at a time, each in time for its own.
        const int kt = (place + 1) % R * kTileBytes, vt = (R + place) * kTileBytes;
        constexpr int kAhead = BIAS && DP > 64 ? 2 : 4, kScores = NB * NK, kAll = kScores + 2 * NB * ND, kPairs = 8 * NB;
        typename E::Frag f[kAhead], pf[2 * NB];
        const float sub = ca - (st.ref == -INFINITY ? 0.f : st.ref);
        float part[2] = {0.f, 0.f};
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int r = 0; r < 16; ++r) sn[nb][r] = 0.f;
        const auto operand = [&](int x) {
            if (x < kScores) return L::frag_rows(lanes, kt + 32 * (x % NB) * L::kRow, x / NB);
            const int y = x - kScores;
            return L::frag_cols(lanes, vt + 16 * (y / ND) * L::kRow, y % ND);
        };
#pragma unroll
        for (int x = 0; x < kAhead; ++x) f[x] = operand(x);
#pragma unroll
        for (int x = 0; x < kAll; ++x) {
            __builtin_amdgcn_sched_barrier(0);
            const typename E::Frag op = f[x % kAhead];
            if (x + kAhead < kAll) f[x % kAhead] = operand(x + kAhead);
            if (x < kScores)
                sn[x % NB] = E::mfma(op, qf[x / NB], sn[x % NB]);
            else
                acc[(x - kScores) % ND] = E::mfma(op, pf[(x - kScores) / ND], acc[(x - kScores) % ND]);
#pragma unroll
            for (int y = 0; y < kPairs; ++y)
                if (y * (kAll - ND) / kPairs == x) {
                    const int nb = y / 8, r = 2 * (y % 8);
                    const float u = ex2(fmaf(s[nb][r], cm, sub)), v = ex2(fmaf(s[nb][r + 1], cm, sub));
                    part[0] += u;
                    part[1] += v;
                    pf[y / 4][r % 8] = (T)u;
                    pf[y / 4][r % 8 + 1] = (T)v;
                }
        }
        st.sum += part[0] + part[1];
    };
    if (n_tiles) {
        f32x16 sa[NB], sb[NB];
        dma_wait();
        __syncthreads();
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int r = 0; r < 16; ++r) sa[nb][r] = 0.f;
#pragma unroll
            for (int kk = 0; kk < NK; ++kk)
                sa[nb] = E::mfma(L::frag_rows(lanes, 32 * nb * L::kRow, kk), qf[kk], sa[nb]);
        }
        for (int u = 0;;) {
            step(u, sa, sb, 0);
            if (++u == n_tiles) break;
            step(u, sb, sa, 1);
            if (++u == n_tiles) break;
        }
        dma_wait();
    }

    p.store(a, st, acc);
}

// ---- few query rows -------------------------------------------------------
// For single tokens and a few rows per head the keys are the whole cost.  The
// query rows of all heads of a key head are packed into blocks of 32; the
// four waves of a workgroup take key tiles of 32 in turn, each staged in the
// wave's own part of LDS with the next tile's loads in flight, without
// barriers, and their four results are joined at the end.  Long key ranges
// are split over workgroups and joined by a second kernel.  Bound by memory:
// one token for each of 8 sequences of up to 32768 keys, 32 heads of 128 over
// 8, 839 MB of keys and values in 172 us (4.9 TB/s), 5 us more to join; the
// smallest calls (4 sequences of 512 keys, 8 heads of 64: 11 us) by the launch
// and the chain of a tile's loads, products and the joins.
template <int OP, int DP>
struct RowsShape {
    static constexpr int kRow = Tile<OP, DP>::kRow;
    static constexpr int kWaves = kRow <= 128 ? 8 : 4;
    static constexpr int kBufs = kRow <= 256 ? 2 : 1;
};
template <int OP, int DP, bool BIAS>
__global__ __launch_bounds__((64 * RowsShape<OP, DP>::kWaves), (RowsShape<OP, DP>::kWaves / 4))
void attn_rows_kernel(const AttnArgs a) {
    using E = El<OP>;
    using T = typename E::T;
    using L = Tile<OP, DP>;
    constexpr int KT = 32, ND = DP / 32, NK = DP / 16;
    constexpr int NW = RowsShape<OP, DP>::kWaves, NB = RowsShape<OP, DP>::kBufs;
    using Load = Loader<OP, DP, KT, 64>;
    __shared__ __attribute__((aligned(256))) char tiles[NW][NB][2][KT * L::kRow];
    static_assert(sizeof(tiles) >= NW * 32 * DP * 4, "the waves' results fit the tiles' memory");
    __shared__ short bucket[BIAS ? 2 * kAttnMaxEdge + 1 : 1];
    __shared__ float wref[NW][32], wsum[NW][32];
    __shared__ uint64_t words[NW][128];

    const int t = threadIdx.x, lane = t & 63, wid = wave_id(), h = lane >> 5;
    const int rows = a.G * a.n;
    const int nrb = (rows + 31) / 32;
    int w = xcd_item(blockIdx.x, gridDim.x, a.n_split * nrb);
    const int rb = w % nrb;
    w /= nrb;
    const int split = w % a.n_split;
    w /= a.n_split;
    const int kvh = w % a.K, b = w / a.K;

    const int off = attn_offset(a, b);
    const int rho = rb * 32 + (lane & 31);
    const int g = min(rho, rows - 1) / a.n, i = min(rho, rows - 1) - g * a.n;
    const int head = kvh * a.G + g;
    const int qlen = attn_q_len(a, b);
    const bool row_ok = rho < rows && i < qlen;
    int len = attn_kv_len(a, b);
    if (a.causal) len = min(len, max(0, qlen + off));
    const int jb = split * a.split_keys;
    const int je = a.n_split == 1 ? len : min(len, jb + a.split_keys);

    const T* kbase = (const T*)a.k.p + b * a.k.sb + kvh * a.k.sh;
    const T* vbase = (const T*)a.v.p + b * a.v.sb + kvh * a.v.sh;
    const int j_first = jb + wid * KT;
    const SeenKeys<KT, 1> keys{a.key_mask ? a.key_mask + b * a.mask_stride : nullptr,
                               lds_addr(words[wid]), j_first, NW * KT, je};
    const int n_tiles = j_first < je ? (je - j_first + NW * KT - 1) / (NW * KT) : 0;
    constexpr int kTileBytes = KT * L::kRow;
    const uint32_t tile0 = lds_addr(tiles[wid]);
    const auto fetch = [&](int u, int buf) {
        const int64_t j0 = j_first + (int64_t)u * NW * KT;
        const uint64_t seen = keys(u);
        Load::fill(tile0 + 2 * buf * kTileBytes, kbase + j0 * a.k.sr, a.k.sr, seen, a.d, a.k.vec, lane);
        Load::fill(tile0 + (2 * buf + 1) * kTileBytes, vbase + j0 * a.v.sr, a.v.sr, seen, a.dv,
                   a.v.vec, lane);
    };
    if (n_tiles) {
        keys.fill(0, lane, 0);
        wave_fence();
        fetch(0, 0);
    }
    const typename L::Lanes lanes(tile0, lane);
    float bias_lo = 0.f, bias_hi = 0.f;
    if (BIAS) {
        for (int x = t; x < a.r0 + a.rp + 1; x += 64 * NW) bucket[x] = (short)bucket_of(a, x - a.r0);
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

    int cur = 0;
    for (int u = 0; u < n_tiles; ++u) {
        const int j0 = j_first + u * NW * KT;
        uint32_t vis = (uint32_t)keys(u);
        // the wave's own buffers: no barrier
        dma_wait();
        wave_fence();
        const typename L::Lanes now(lanes, cur * 2 * kTileBytes);
        if (u % 64 == 0) keys.fill(u + 64, lane, 0);
        wave_fence();
        if (NB == 2) {
            cur ^= 1;
            if (u + 1 < n_tiles) fetch(u + 1, cur);
        }
        if (a.causal) vis &= bits_upto(i + off - j0);
        const bool all = __all(vis == ~0u);
        vis >>= 4 * h;
        f32x16 s;
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = 0.f;
        auto prod = products<4, NK, 2 * ND, typename E::Frag>([&](int y) {
            if (y < NK) return L::frag_rows(now, 0, y);
            y -= NK;
            return L::frag_cols(now, kTileBytes + 16 * (y / ND) * L::kRow, y % ND);
        });
        prod.first([&](int y, typename E::Frag op) { s = E::mfma(op, qf[y], s); });
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
            asm volatile("");  // a branch: most tiles need none of it
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = flag(vis, r) ? s[r] : -INFINITY;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[r]);
        mx = fmaf(half_max(mx), cm, ca);
        raise_ref<OP, ND>(st, mx, acc);
        st.sum += weights(s, cm, ca, st);
        const typename E::Frag pf[2] = {L::pack(s, 0), L::pack(s, 1)};
        prod.second([&](int y, typename E::Frag op) { acc[y % ND] = E::mfma(op, pf[y / ND], acc[y % ND]); });
        if (NB == 1 && u + 1 < n_tiles) {
            dma_wait();
            wave_fence();
            fetch(u + 1, 0);
        }
    }

    // join the waves' results: [wave][element][row] in the tiles' memory
    st.sum = half_sum(st.sum);
    __syncthreads();
    const LdsFloats buf{lds_addr(tiles)};
#pragma unroll
    for (int cb = 0; cb < ND; ++cb)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            buf.set((wid * DP + 32 * cb + 8 * (r >> 2) + 4 * h + (r & 3)) * 32 + (lane & 31), acc[cb][r]);
    if (h == 0) {
        wref[wid][lane] = st.ref;
        wsum[wid][lane] = st.sum;
    }
    __syncthreads();
    const int q = t & 31;
    const int orho = rb * 32 + q;
    if (orho >= rows) return;
    const int og = orho / a.n, oi = orho - og * a.n, ohead = kvh * a.G + og;
    const bool ok = oi < qlen;
    float ref = -INFINITY;
#pragma unroll
    for (int x = 0; x < NW; ++x) ref = fmaxf(ref, wref[x][q]);
    float f[NW], sum = 0.f;
#pragma unroll
    for (int x = 0; x < NW; ++x) {
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
    float* po = a.part_o + (split * prows + prow) * a.dv_pad;
    for (int x = (t >> 5) * 4; x < a.dv; x += 8 * NW) {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y[e] = 0.f;
#pragma unroll
            for (int v = 0; v < NW; ++v)
                if (wref[v][q] != -INFINITY) y[e] = fmaf(buf[(v * DP + x + e) * 32 + q], f[v], y[e]);
            y[e] = some ? y[e] * inv : 0.f;
        }
        if (last) {
            store4<OP>(o, x, a.dv, a.o.vec, y[0], y[1], y[2], y[3]);
        } else {
            *(f32x4*)(po + x) = f32x4{y[0], y[1], y[2], y[3]};
        }
    }
    if (t < 32) {
        if (!last)
            a.part_ml[split * prows + prow] = make_float2(some ? ref : -INFINITY, sum);
        else if (a.lse)
            a.lse[prow] = some ? (ref + lg2(sum)) * kLn2 : -INFINITY;
    }
}

// Joins the key ranges' results, in a fixed order: 32 lanes a row, four
// elements a lane at a time.  4 to 5 us, most of it the launch.
template <int OP>
__global__ __launch_bounds__(256) void attn_merge_kernel(const AttnArgs a) {
    using T = typename El<OP>::T;
    __shared__ float weight[8][kAttnMaxSplit];
    const int64_t rows = (int64_t)a.B * a.H * a.n;
    const int grp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = flat_block() * 8 + grp;
    if (row >= rows) return;
    // lane s, s + 32: the ranges' references and sums
    float2 ml[kAttnMaxSplit / 32];
    float ref = -INFINITY;
#pragma unroll
    for (int x = 0; x < kAttnMaxSplit / 32; ++x) {
        const int s = lane + 32 * x;
        ml[x] = s < a.n_split ? a.part_ml[s * rows + row] : make_float2(-INFINITY, 0.f);
        ref = fmaxf(ref, ml[x].x);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) ref = fmaxf(ref, __shfl_xor(ref, o, 64));
    float sum = 0.f;
#pragma unroll
    for (int x = 0; x < kAttnMaxSplit / 32; ++x) {
        const float f = ml[x].x == -INFINITY ? 0.f : ex2(ml[x].x - ref);
        weight[grp][lane + 32 * x] = f;
        sum = fmaf(ml[x].x == -INFINITY ? 0.f : ml[x].y, f, sum);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, 64);
    wave_fence();
    const bool some = !(sum == 0.f);
    const float inv = some ? 1.f / sum : 0.f;
    const int i = (int)(row % a.n);
    const int64_t bh = row / a.n;
    const int head = (int)(bh % a.H), b = (int)(bh / a.H);
    T* o = (T*)a.o.p + b * a.o.sb + (int64_t)i * a.o.sr + head * a.o.sh;
    const float* po = a.part_o + row * a.dv_pad;
    const int64_t next = rows * a.dv_pad;
    for (int x = 4 * lane; x < a.dv; x += 128) {
        f32x4 y = {0.f, 0.f, 0.f, 0.f};
        for (int s0 = 0; s0 < a.n_split; s0 += 8) {
            f32x4 p[8];
#pragma unroll
            for (int s = 0; s < 8; ++s)
                p[s] = *(const f32x4*)(po + min(s0 + s, a.n_split - 1) * next + x);
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const float f = s0 + s < a.n_split ? weight[grp][s0 + s] : 0.f;
                // a range without keys holds nothing
                y += f == 0.f ? f32x4{0.f, 0.f, 0.f, 0.f} : p[s] * f;
            }
        }
        y = some ? y * inv : f32x4{0.f, 0.f, 0.f, 0.f};
        store4<OP>(o, x, a.dv, a.o.vec, y[0], y[1], y[2], y[3]);
    }
    if (a.lse && lane == 0) a.lse[row] = some ? (ref + lg2(sum)) * kLn2 : -INFINITY;
}

template <int OP, int DP>
hipError_t fwd(const AttnArgs& a, bool few, hipStream_t s) {
    if (few) {
        const int64_t g = (int64_t)a.B * a.K * a.n_split * (((int64_t)a.G * a.n + 31) / 32);
        constexpr int nt = 64 * RowsShape<OP, DP>::kWaves;
        if (a.bias)
            attn_rows_kernel<OP, DP, true><<<(unsigned)g, nt, 0, s>>>(a);
        else
            attn_rows_kernel<OP, DP, false><<<(unsigned)g, nt, 0, s>>>(a);
    } else {
        const int64_t g = (int64_t)a.B * a.H * a.n_split * ((a.n + kAttnRows - 1) / kAttnRows);
        if constexpr (Tile<OP, DP>::kRow <= 128) {
            if (a.bias)
                attn_fwd_narrow_kernel<OP, DP, true><<<(unsigned)g, 256, 0, s>>>(a);
            else
                attn_fwd_narrow_kernel<OP, DP, false><<<(unsigned)g, 256, 0, s>>>(a);
        } else {
            if (a.bias)
                attn_fwd_kernel<OP, DP, true><<<(unsigned)g, 256, 0, s>>>(a);
            else
                attn_fwd_kernel<OP, DP, false><<<(unsigned)g, 256, 0, s>>>(a);
        }
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
    const dim3 g = flat_grid((rows + 7) / 8);
    if (a.op == OP_BF16)
        attn_merge_kernel<OP_BF16><<<g, 256, 0, s>>>(a);
    else if (a.op == OP_F16)
        attn_merge_kernel<OP_F16><<<g, 256, 0, s>>>(a);
    else
        attn_merge_kernel<OP_F32><<<g, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace fs
