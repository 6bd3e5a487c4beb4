// fs_attn_bwd.hip -- gradients of the attention of fs_attn_fwd.hip.  With
// P_ij = exp(s_ij - L_i) formed again from the scores and the stored L,
//   delta_i = do_i.o_i - dL_i,     dS_ij = P_ij (do_i.v_j - delta_i),
//   dV_j = sum_i P_ij do_i,        dK_j = scale sum_i dS_ij q_i,
//   dQ_i = scale sum_j dS_ij k_j,  dT[c] = sum of dS over the pairs of bucket c.
// Two passes, one over keys for a resident block of queries (dQ, delta made
// exact) and then one over queries for a resident block of keys (dK, dV, dT):
// seven products instead of five, but every sum is formed in one place in a
// fixed order, so equal calls give equal bits.
#include "fs_attn.hpp"

namespace fs {

namespace {

// ---- row terms ------------------------------------------------------------
// Per query row, for the two passes: -L in base 2 (-inf for a row that takes
// no part: 2^(s - inf) = 0) and delta from the stored o.  Rows are padded to
// whole tiles with the values of a row that takes no part.  16 lanes a row.
// Bound by memory and by its launch (14 us for the 67 MB of o and do at 2048
// rows, 32 heads of 128, batch 2).
template <int OP>
__global__ __launch_bounds__(256) void attn_delta_kernel(const AttnArgs a) {
    using T = typename El<OP>::T;
    constexpr int EPC = 16 / sizeof(T);
    const int64_t rows = (int64_t)a.B * a.n_pad * a.H;
    const int64_t r = flat_block() * 16 + (threadIdx.x >> 4);
    const int lane = threadIdx.x & 15;
    if (r >= rows) return;
    const int head = (int)(r % a.H);
    const int64_t bi = r / a.H;
    const int i = (int)(bi % a.n_pad), b = (int)(bi / a.n_pad);
    const bool ok = i < row_len(a.q_len, b, a.n);
    float s = 0.f;
    if (ok) {
        const T* o = (const T*)a.o.p + b * a.o.sb + (int64_t)i * a.o.sr + head * a.o.sh;
        const T* g = (const T*)a.go.p + b * a.go.sb + (int64_t)i * a.go.sr + head * a.go.sh;
        for (int x = lane * EPC; x < a.dv; x += 16 * EPC) {
            T p[EPC], q[EPC];
            load_elems<OP, EPC>(o, x, a.dv, a.o.vec, p);
            load_elems<OP, EPC>(g, x, a.dv, a.go.vec, q);
#pragma unroll
            for (int e = 0; e < EPC; ++e) s = fmaf((float)p[e], (float)q[e], s);
        }
    }
#pragma unroll
    for (int m = 8; m >= 1; m >>= 1) s += __shfl_xor(s, m, 64);
    if (lane == 0) {
        const int64_t at = ((int64_t)b * a.H + head) * a.n + i;
        const float l = ok ? a.lse[at] : -INFINITY;
        const bool part = l != -INFINITY;
        const int64_t to = ((int64_t)b * a.H + head) * a.n_pad + i;
        a.nl2[to] = part ? -l * kLog2e : -INFINITY;
        a.delta[to] = part ? s - (a.glse ? a.glse[at] : 0.f) : 0.f;
    }
}

// ---- rounding of dS -------------------------------------------------------
// dS goes into its product in the element type.  Its size follows the
// gradient's, which fp16's exponents need not hold, so for fp16 every column
// (a lane pair) carries a power of two, set by its first values to bring the
// largest to 2^10 and lowered when one passes 2^15 (fp16 ends at 2^16), and
// the sums are divided by it at the end.  P is at most 1 and is lifted by 2^14.
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

// Two forms of each pass.  Shared: the four waves of a workgroup hold 32 rows
// each and pass over the same tiles, fetched once for all.  Alone, for few rows
// in all: the waves hold the same 32 rows, each passes over every fourth tile,
// fetched for itself, and their sums are joined at the end -- four times the
// workgroups and a quarter of the steps for four times the fetches.  (Rows of
// 512 bytes leave no LDS for tiles of four waves: always shared.)
//
// A tile is worked on 32 rows at a time.  Where LDS allows, the next tile is
// fetched into a second buffer meanwhile; where registers allow, two waves
// share a SIMD, and one's products run under the other's exponentials.
// Measured against forms whose steps are pipelined within a wave (the products
// of the next 32 rows among the exponentials of these): those need the second
// wave's registers, and took 659 us against 390 (queries) and 763 against 650
// (keys) for 2048 x 4096, 32 heads of 128 over 8, batch 2.
constexpr int kAhead = 4;  // products ahead of which operands are read
template <int OP, int DP, bool ALONE, int MOST>
struct BwdShape {
    static constexpr int kRow = Tile<OP, DP>::kRow;
    static constexpr int kTile = ALONE || kRow > 256 ? 32 : kRow > 128 || MOST < 128 ? 64 : 128;
    static constexpr int kBufs = ALONE && kRow > 128 ? 1 : 2;
    static constexpr int kSets = ALONE ? 4 : 1;
    static constexpr int kRows = ALONE ? 32 : kAttnRows;  // rows a workgroup holds
    static constexpr int kNt = ALONE ? 64 : 256;          // threads that fetch a tile
};

// Joins one lane-held 32-column result of four waves: adds waves 1..3 to wave 0
// through LDS (buf: 3 * DP * 32 floats), in order.
template <int DP, int ND>
__device__ __forceinline__ void join_waves(f32x16 (&x)[ND], LdsFloats buf, int wid, int lane) {
    const int h = lane >> 5;
    __syncthreads();
    if (wid > 0) {
#pragma unroll
        for (int cb = 0; cb < ND; ++cb)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                buf.set(((wid - 1) * DP + 32 * cb + 8 * (r >> 2) + 4 * h + (r & 3)) * 32 + (lane & 31),
                        x[cb][r]);
    }
    __syncthreads();
    if (wid == 0) {
#pragma unroll
        for (int w = 0; w < 3; ++w)
#pragma unroll
            for (int cb = 0; cb < ND; ++cb)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    x[cb][r] += buf[(w * DP + 32 * cb + 8 * (r >> 2) + 4 * h + (r & 3)) * 32 + (lane & 31)];
    }
}

// ---- dK, dV, dT -----------------------------------------------------------
// A workgroup holds keys of one key head, 32 a wave, as operands, and passes
// over the queries of every head of the group in tiles staged in LDS.  Scores
// are formed with queries in the rows, so a lane holds one key's column: a key
// that is masked out spoils nothing but its own column, which is written as
// zero, and needs no test in the loop (but for the bias, whose sums run over
// columns).
//
// Bias gradient: dS summed over the pairs of every relative position r, and
// those sums over each bucket by attn_bias_sum_kernel.  A block whose pairs all
// lie beyond the last edge goes into one of two running sums of the lane.  For
// a block near the diagonal a wave writes the 32 x 32 values to its own LDS
// with key x's row moved by x, so that a relative position is a column, and 63
// lanes sum a column each; positions between the last edges are added to the
// wave's line in LDS (one lane a position), those beyond to the lane's sums.
constexpr int kDiag = 64;

// What the two forms share of the pass over queries: a lane's key, the range of
// queries, the bias's sums and the output.
template <int OP, int DP, bool BIAS, bool ALONE>
struct KvPass {
    using S = BwdShape<OP, DP, ALONE, 64>;
    static constexpr int ROWS = S::kRows, QT = S::kTile;
    using E = El<OP>;
    using T = typename E::T;
    using L = Tile<OP, DP>;
    static constexpr int ND = DP / 32, NK = DP / 16;
    int lane, wid, h, kb, split, kvh, b, n_line, off, j0, j, first, end, n_tiles;
    bool key_ok;
    LdsFloats line, gline, dg;
    float sum_lo, sum_hi;

    __device__ __forceinline__ KvPass(const AttnArgs& a, float* lines, float* diag) {
        const int t = threadIdx.x;
        lane = t & 63, wid = wave_id(), h = lane >> 5;
        const int nkb = (a.m + ROWS - 1) / ROWS;
        int w = xcd_item(blockIdx.x, gridDim.x, a.q_split * nkb);
        kb = w % nkb;
        w /= nkb;
        split = w % a.q_split;
        w /= a.q_split;
        kvh = w % a.K, b = w / a.K;
        n_line = a.r0 + a.rp + 1;
        line.a = lds_addr(lines);
        gline.a = line.a + 4 * (1 + wid) * n_line;
        dg.a = lds_addr(diag) + (BIAS ? wid * 32 * kDiag * 4 : 0);
        off = attn_offset(a, b);
        const int len = attn_kv_len(a, b), qlen = attn_q_len(a, b);
        j0 = kb * ROWS + (ALONE ? 0 : wid * 32), j = j0 + (lane & 31);
        key_ok = j < len;
        if (a.causal) key_ok = key_ok && j < qlen + off;  // some row sees it
        if (key_ok && a.key_mask) key_ok = a.key_mask[b * a.mask_stride + j] != 0;
        // tiles of this workgroup's query range, from the first that sees a key
        // of this block on
        first = split * a.split_rows;
        end = a.q_split == 1 ? qlen : min(qlen, first + a.split_rows);
        if (a.causal) first = max(first, (max(0, kb * ROWS - off) / QT) * QT);
        if (kb * ROWS >= len) first = end;
        n_tiles = first < end ? (end - first + QT - 1) / QT : 0;
        if (BIAS && a.gbias)
            for (int x = lane; x < 32 * kDiag; x += 64) dg.set(x, 0.f);
    }

    // Tile u of head g of the group.
    struct Place {
        int g, u;
    };
    // `step` tiles on; without a bias the tiles of all heads are one sequence.
    __device__ __forceinline__ Place advance(Place x, int step) const {
        x.u += step;
        if (!BIAS && n_tiles > 0)
            while (x.u >= n_tiles) x.u -= n_tiles, ++x.g;
        return x;
    }
    // -L of the lane's row of a tile (rows are padded to whole tiles), read a tile
    // before the tile's fetch asks which rows take part.  A row that takes none
    // has -inf and weight 0; it is fetched as zeros, or what it holds (the loss of
    // an empty row may well have no derivative) would enter sums as 0 * NaN.
    __device__ __forceinline__ float row_term(const AttnArgs& a, Place x) const {
        const int64_t lrow = ((int64_t)b * a.H + kvh * a.G + x.g) * a.n_pad + first + x.u * QT;
        return lane < QT ? a.nl2[lrow + lane] : -INFINITY;
    }
    static __device__ __forceinline__ uint64_t live(float term) { return __ballot(term != -INFINITY); }
    // A tile's rows in `seen`: q and do to LDS (lds: a tile each), and the row
    // terms, 64 floats for every 32 rows, to terms (these first: an address that
    // had to be put into memory is read again, and that waits for the copies
    // before it).
    __device__ __forceinline__ void fetch(const AttnArgs& a, Place x, uint64_t seen, uint32_t lds,
                                          uint32_t terms) const {
        // Measured on forward and backward together, all places kept / those of the
        // wide path / none: 2048 x 4096, 32 heads of 128 over 8, batch 2, 1267 / 1251
        // / 1265 us; with a bias, whose sums take more registers, 2048 x 2048, 16
        // heads of 64, batch 4, 508 / 504 / 494 us.
        using Load = Loader<OP, DP, QT, S::kNt, BIAS ? PLACES_ANEW : PLACES_KEPT_WIDE>;
        const int i0 = first + x.u * QT, head = kvh * a.G + x.g;
        const int part = ALONE ? 0 : wid;  // 32 rows a wave
        if (part < QT / 32) {
            const int64_t lrow = ((int64_t)b * a.H + head) * a.n_pad + i0 + 32 * part;
            const float* src = (lane < 32 ? a.nl2 : a.delta) + lrow + (lane & 31);
            dma_lane4((const char*)src, terms + 256 * part);
        }
        const int t = ALONE ? lane : (int)threadIdx.x;
        Load::fill(lds, (const T*)a.q.p + b * a.q.sb + head * a.q.sh + (int64_t)i0 * a.q.sr, a.q.sr,
                   seen, a.d, a.q.vec, t);
        Load::fill(lds + QT * L::kRow,
                   (const T*)a.go.p + b * a.go.sb + head * a.go.sh + (int64_t)i0 * a.go.sr, a.go.sr,
                   seen, a.dv, a.go.vec, t);
    }

    __device__ __forceinline__ void start_head(const AttnArgs& a, int g) {
        sum_lo = sum_hi = 0.f;
        if (!BIAS) return;
        __syncthreads();
        load_line(a, kvh * a.G + g, line, threadIdx.x, 256);
        if (a.gbias)
            for (int x = lane; x < n_line; x += 64) gline.set(x, 0.f);
        __syncthreads();
    }

    // Row terms of a block as the lane needs them: rl = -L (+ bias), rd = delta.
    // Where lo or hi is set, the block lies wholly behind or before the edges.
    __device__ __forceinline__ void row_terms(const AttnArgs& a, int i0, uint32_t terms, float (&rl)[16],
                                              float (&rd)[16], bool& lo_far, bool& hi_far) const {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const f32x4 x = lds_read<f32x4>(terms + 4 * (8 * q + 4 * h));
            const f32x4 y = lds_read<f32x4>(terms + 4 * (32 + 8 * q + 4 * h));
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                rl[4 * q + r] = x[r];
                rd[4 * q + r] = y[r];
            }
        }
        lo_far = hi_far = false;
        if (BIAS) {
            lo_far = j0 + 31 - i0 - off <= -a.r0;
            hi_far = !lo_far && j0 - i0 - 31 - off >= a.rp;
            if (lo_far || hi_far) {
                const float ca = line[lo_far ? 0 : n_line - 1];
#pragma unroll
                for (int r = 0; r < 16; ++r) rl[r] += ca;
            } else {
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    rl[r] += line[line_index(a, j - (i0 + 8 * (r >> 2) + 4 * h + (r & 3)) - off)];
            }
        }
    }
    // Scores of queries before j - off do not see key j.
    __device__ __forceinline__ void hide(const AttnArgs& a, int i0, f32x16& s) const {
        if (a.causal && j0 + 31 - off > i0) {
            asm volatile("");  // a branch: most tiles need none of it
            const uint32_t vis = ~bits_upto(j - off - i0 - 1) >> (4 * h);
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = flag(vis, r) ? s[r] : -INFINITY;
        }
    }
    // Adds a block's dS to the sums of its relative positions.
    __device__ __forceinline__ void add_bias(const AttnArgs& a, int i0, const f32x16& ds, bool lo_far,
                                             bool hi_far) {
        if (!BIAS || !a.gbias) return;
        if (lo_far || hi_far) {
            float x = 0.f;
#pragma unroll
            for (int r = 0; r < 16; ++r) x += ds[r];
            x = key_ok ? x : 0.f;
            if (lo_far) sum_lo += x;
            else sum_hi += x;
            return;
        }
        const int k = lane & 31;
        wave_fence();
#pragma unroll
        for (int r = 0; r < 16; ++r)
            dg.set(k * kDiag + k - (8 * (r >> 2) + 4 * h + (r & 3)) + 31, key_ok ? ds[r] : 0.f);
        wave_fence();
        float x = 0.f;
#pragma unroll
        for (int y = 0; y < 32; ++y) x += dg[y * kDiag + lane];
        const int r = j0 - i0 - 31 - off + lane;  // lane 63: no pair, x = 0
        if (r <= -a.r0) sum_lo += x;
        else if (r >= a.rp) sum_hi += x;
        else gline.set(r + a.r0, gline[r + a.r0] + x);
        wave_fence();
    }
    __device__ __forceinline__ void end_head(const AttnArgs& a, int g) {
        if (!BIAS || !a.gbias) return;
        sum_lo = wave_sum(sum_lo);
        sum_hi = wave_sum(sum_hi);
        if (lane == 0) {
            gline.set(0, gline[0] + sum_lo);
            gline.set(n_line - 1, gline[n_line - 1] + sum_hi);
        }
        __syncthreads();
        const int nkb = (a.m + ROWS - 1) / ROWS;
        float* part = a.line_part + ((int64_t)(kvh * a.G + g) * a.B * a.line_blocks +
                                     (int64_t)b * a.line_blocks + split * nkb + kb) * n_line;
        for (int x = threadIdx.x; x < n_line; x += 256)
            part[x] = (line[n_line + x] + line[2 * n_line + x]) + (line[3 * n_line + x] + line[4 * n_line + x]);
    }

    template <bool DK, bool DV>
    __device__ __forceinline__ void store(const AttnArgs& a, const f32x16 (&dk)[ND],
                                          const f32x16 (&dv)[ND]) const {
        if (j >= a.m) return;
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
                    if (DK && x < a.d) pk[x] = key_ok ? dk[cb][r] : 0.f;
                    if (DV && x < a.dv) pv[x] = key_ok ? dv[cb][r] : 0.f;
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
                    y[r] = DK && key_ok ? dk[cb][4 * q + r] : 0.f;
                    z[r] = DV && key_ok ? dv[cb][4 * q + r] : 0.f;
                }
                if (DK && a.gk.p) store4<OP>(ok, 32 * cb + 8 * q + 4 * h, a.d, a.gk.vec, y[0], y[1], y[2], y[3]);
                if (DV && a.gv.p) store4<OP>(ov, 32 * cb + 8 * q + 4 * h, a.dv, a.gv.vec, z[0], z[1], z[2], z[3]);
            }
    }
};

// PART: which sums this launch forms.  Both, as a rule; rows of 512 bytes leave
// no registers for both, and they are formed by two launches.  Rows of 256
// bytes have the registers (dK, dV, and the keys and values themselves: 256
// numbers a lane) for one wave a SIMD, which bounds them: the products wait for
// the exponentials (597 us for 2048 x 4096, 32 heads of 128 over 8, batch 2, 920
// TFLOP/s, the matrix pipes busy 40% of the cycles; held to two waves, 186
// registers go to memory and it takes 1150 and more).
// fp16 at 512 bytes keeps 76 registers in memory in the launch for dK (146 with
// a bias): 196 to 209 us against 133 in bf16 for 1024 x 2048, 16 heads of 256,
// batch 2.
enum KvPart : int { PART_BOTH = 0, PART_DV = 1, PART_DK = 2 };
template <int OP, int DP, bool BIAS, bool ALONE, int PART>
__global__ __launch_bounds__(256, (Tile<OP, DP>::kRow <= 128 && !(BIAS && ALONE) ? 2 : 1))
void attn_bwd_kv_kernel(const AttnArgs a) {
    using P = KvPass<OP, DP, BIAS, ALONE>;
    using S = typename P::S;
    using E = typename P::E;
    using T = typename P::T;
    using L = typename P::L;
    constexpr bool DK = PART != PART_DV, DV = PART != PART_DK;
    constexpr int ND = P::ND, NK = P::NK, QT = P::QT, kBytes = QT * L::kRow;
    __shared__ __attribute__((aligned(256))) char tiles[S::kSets][S::kBufs][2][kBytes];
    __shared__ __attribute__((aligned(16))) float terms[S::kSets][S::kBufs][2 * QT];
    __shared__ float diag[BIAS ? 4 * 32 * kDiag : 1];
    extern __shared__ float lines[];  // BIAS: [1 + 4][n_line], the bias and the waves' sums
    static_assert(!ALONE || sizeof(tiles) >= 3 * 32 * DP * 4, "the waves' sums fit the tiles' memory");
    P p(a, lines, diag);
    const int lane = p.lane, wid = p.wid, set = ALONE ? wid : 0;

    // With a bias the heads are taken one after the other (each has its line);
    // else the tiles of all heads are one sequence.
    const int step = ALONE ? 4 : 1, u_first = ALONE ? wid : 0;
    const int n_all = BIAS ? p.n_tiles : p.n_tiles * a.G;
    typename P::Place here{0, 0};
    float term = -INFINITY;
    if (u_first < n_all) {
        here = p.advance(here, u_first);
        term = p.row_term(a, here);
    }

    typename E::Frag kf[NK], vf[NK];
    load_row_frags<OP, DP>((const T*)a.k.p + p.b * a.k.sb + (int64_t)p.j * a.k.sr + p.kvh * a.k.sh,
                           p.key_ok, a.d, a.k.vec, lane, kf);
    if (DK)
        load_row_frags<OP, DP>((const T*)a.v.p + p.b * a.v.sb + (int64_t)p.j * a.v.sr + p.kvh * a.v.sh,
                               p.key_ok, a.dv, a.v.vec, lane, vf);
    f32x16 dk[ND], dv[ND];
#pragma unroll
    for (int x = 0; x < ND; ++x)
#pragma unroll
        for (int r = 0; r < 16; ++r) dk[x][r] = dv[x][r] = 0.f;
    DsScale<OP, ND> dss;
    const uint32_t tile0 = lds_addr(tiles[set]), term0 = lds_addr(terms[set]);
    typename L::Lanes now(tile0, lane);
    int cur = 0;

    for (int g0 = 0; g0 < (BIAS ? a.G : 1); ++g0) {
        int u = u_first;
        if (g0 > 0) here = {g0, u}, term = u < n_all ? p.row_term(a, here) : -INFINITY;
        p.start_head(a, g0);
        const auto fetch = [&](typename P::Place x, uint64_t seen, int buf) {
            p.fetch(a, x, seen, tile0 + 2 * buf * kBytes, term0 + 8 * QT * buf);
        };
        typename P::Place next = p.advance(here, step);
        if (u < n_all) {
            fetch(here, P::live(term), cur);
            if (u + step < n_all) term = p.row_term(a, next);
        }
        for (; u < n_all; u += step) {
            dma_wait();
            if (ALONE)
                wave_fence();
            else
                __builtin_amdgcn_s_barrier();
            const uint32_t term_lds = term0 + 8 * QT * cur;
            const uint64_t seen = P::live(term);
            if (S::kBufs == 2) {
                cur ^= 1;
                if (u + step < n_all) fetch(next, seen, cur);
            }
            const typename P::Place after = p.advance(next, step);
            if (u + 2 * step < n_all) term = p.row_term(a, after);
            const int i00 = p.first + here.u * QT;
#pragma unroll
            for (int qb = 0; qb < QT / 32; ++qb) {
                const int i0 = i00 + 32 * qb, o = 32 * qb * L::kRow;
                f32x16 s, dp;
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.f;
                // q and do rows in turn, then their columns (rc, cb; dV, dK)
                constexpr int kFirst = DK ? 2 * NK : NK, kSecond = DK && DV ? 4 * ND : 2 * ND;
                auto prod = products<kAhead, kFirst, kSecond, typename E::Frag>([&](int y) {
                    if (y < kFirst)
                        return DK ? L::frag_rows(now, y % 2 * kBytes + o, y / 2) : L::frag_rows(now, o, y);
                    y -= kFirst;
                    const int of = DK && DV ? (y % 2 ? 0 : kBytes) : DK ? 0 : kBytes;
                    if (DK && DV) y /= 2;
                    return L::frag_cols(now, of + o + 16 * (y / ND) * L::kRow, y % ND);
                });
                prod.first([&](int y, typename E::Frag op) {
                    if (DK && y % 2)
                        dp = E::mfma(op, vf[y / 2], dp);
                    else
                        s = E::mfma(op, kf[DK ? y / 2 : y], s);
                });
                float rl[16], rd[16];
                bool lo_far, hi_far;
                p.row_terms(a, i0, term_lds + 256 * qb, rl, rd, lo_far, hi_far);
                p.hide(a, i0, s);
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const float w = ex2(fmaf(s[r], a.c, rl[r]));
                    dp[r] = w * (dp[r] - rd[r]);
                    s[r] = w * kLiftP<OP>;
                }
                if (DK) {
                    p.add_bias(a, i0, dp, lo_far, hi_far);
                    dss.apply(dp, dk);
                }
                const typename E::Frag pf[2] = {L::pack(s, 0), L::pack(s, 1)};
                const typename E::Frag df[2] = {L::pack(dp, 0), L::pack(dp, 1)};
                prod.second([&](int y, typename E::Frag op) {
                    const bool k = DK && (!DV || y % 2);
                    if (DK && DV) y /= 2;
                    if (k)
                        dk[y % ND] = E::mfma(op, df[y / ND], dk[y % ND]);
                    else
                        dv[y % ND] = E::mfma(op, pf[y / ND], dv[y % ND]);
                });
            }
            if (S::kBufs == 1 && u + step < n_all) {
                dma_wait();
                wave_fence();
                fetch(next, seen, 0);
            }
            here = next;
            next = after;
            if (S::kBufs == 2) now.move(cur ? 2 * kBytes : -2 * kBytes);
        }
        if (DK) p.end_head(a, g0);
    }

    const float fk = a.scale * dss.undo(), fv = 1.f / kLiftP<OP>;
#pragma unroll
    for (int cb = 0; cb < ND; ++cb)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            if (DK) dk[cb][r] *= fk;
            if (DV) dv[cb][r] *= fv;
        }
    if (ALONE) {
        const LdsFloats buf{lds_addr(tiles)};
        join_waves<DP, ND>(dk, buf, wid, lane);
        join_waves<DP, ND>(dv, buf, wid, lane);
        if (wid > 0) return;
    }
    p.template store<DK, DV>(a, dk, dv);
}

// Sums the query ranges' parts of dK and dV (a fixed order).  Bound by memory:
// the parts are read once.
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

// ---- dQ -------------------------------------------------------------------
// The mirror image: query rows of a head, keys in tiles, keys in the rows of
// the scores.  Here a masked key does enter sums over keys, so its weight is
// set to zero.
//
// The stored o is rounded, and with it delta: enough for a gradient that is
// rounded as well, but not for the bias's, an fp32 sum over many rows.  Since
// sum_j P_ij = 1, sum_j dS_ij is what delta lacks of sum_j P_ij do_i.v_j (and
// dL_i); the pass adds it, and the pass over the queries after it uses the
// result.
//
// Bound by the matrix unit and the exponentials between its products: two
// waves a SIMD, 379 to 395 us for 2048 x 4096, 32 heads of 128 over 8, batch 2
// (1040 to 1090 TFLOP/s, the matrix pipes busy 56% of the cycles; 580 with one
// wave).
template <int OP, int DP, bool BIAS, bool ALONE>
struct QPass {
    using S = BwdShape<OP, DP, ALONE, 128>;
    static constexpr int ROWS = S::kRows;
    using E = El<OP>;
    using T = typename E::T;
    using L = Tile<OP, DP>;
    static constexpr int ND = DP / 32, NK = DP / 16;
    int lane, wid, h, head, b, kvh, n_line, off, i0, i, len;
    bool row_ok, in;
    int64_t lrow;
    float rl, rd;
    LdsFloats line;

    __device__ __forceinline__ QPass(const AttnArgs& a, float* line_mem) {
        const int t = threadIdx.x;
        lane = t & 63, wid = wave_id(), h = lane >> 5;
        const int nqb = (a.n + ROWS - 1) / ROWS;
        int w = xcd_item(blockIdx.x, gridDim.x, a.G * nqb);
        const int qb = w % nqb;
        w /= nqb;
        head = w % a.H, b = w / a.H, kvh = head / a.G;
        n_line = a.r0 + a.rp + 1;
        line.a = lds_addr(line_mem);
        off = attn_offset(a, b);
        i0 = qb * ROWS + (ALONE ? 0 : wid * 32), i = i0 + (lane & 31);
        const int qlen = attn_q_len(a, b);
        row_ok = i < qlen;
        in = i < a.n;
        len = attn_kv_len(a, b);
        if (a.causal) len = min(len, max(0, min((qb + 1) * ROWS, qlen) + off));
        lrow = ((int64_t)b * a.H + head) * a.n_pad + i;
        rl = in ? a.nl2[lrow] : -INFINITY;
        rd = in ? a.delta[lrow] : 0.f;
    }
    // A block's scores ready for s cm + ca: masked keys at -inf, the bias in.
    __device__ __forceinline__ void prepare(const AttnArgs& a, int j0, uint32_t vis, f32x16& s, float& cm,
                                            float& ca) const {
        if (a.causal) vis &= bits_upto(i + off - j0);
        const bool all = __all(vis == ~0u);
        vis >>= 4 * h;
        cm = a.c, ca = rl;
        if (BIAS) {
            if (j0 + 31 - i0 - off <= -a.r0) {
                ca += line[0];
            } else if (j0 - i0 - 31 - off >= a.rp) {
                ca += line[n_line - 1];
            } else {
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    s[r] = fmaf(s[r], a.c, line[line_index(a, j0 + 8 * (r >> 2) + 4 * h + (r & 3) - i - off)]);
                cm = 1.f;
            }
        }
        if (!all) {
            asm volatile("");  // a branch: most tiles need none of it
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = flag(vis, r) ? s[r] : -INFINITY;
        }
    }
    // delta made exact; dQ (zero for a row that takes no part).  rest: the row's
    // sum of dS.
    __device__ __forceinline__ void store(const AttnArgs& a, const f32x16 (&acc)[ND], float rest) const {
        if (!in) return;
        const bool part = row_ok && rl != -INFINITY;
        if (h == 0 && part)
            a.delta[lrow] = rd + rest - (a.glse ? a.glse[((int64_t)b * a.H + head) * a.n + i] : 0.f);
        if (!a.gq.p) return;
        T* o = (T*)a.gq.p + b * a.gq.sb + (int64_t)i * a.gq.sr + head * a.gq.sh;
#pragma unroll
        for (int cb = 0; cb < ND; ++cb)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                store4<OP>(o, 32 * cb + 8 * q + 4 * h, a.d, a.gq.vec, part ? acc[cb][4 * q] : 0.f,
                           part ? acc[cb][4 * q + 1] : 0.f, part ? acc[cb][4 * q + 2] : 0.f,
                           part ? acc[cb][4 * q + 3] : 0.f);
    }
};

template <int OP, int DP, bool BIAS, bool ALONE>
__global__ __launch_bounds__(256, (Tile<OP, DP>::kRow <= 256 ? 2 : 1))
void attn_bwd_q_kernel(const AttnArgs a) {
    using P = QPass<OP, DP, BIAS, ALONE>;
    using S = typename P::S;
    using E = typename P::E;
    using T = typename P::T;
    using L = typename P::L;
    constexpr int ND = P::ND, NK = P::NK, KT = S::kTile, kBytes = KT * L::kRow;
    constexpr int kPart = KT < 64 ? KT : 64, kParts = KT / kPart;  // keys of a word of flags
    using Load = Loader<OP, DP, kPart, S::kNt>;
    __shared__ __attribute__((aligned(256))) char tiles[S::kSets][S::kBufs][2][kBytes];
    __shared__ float line_mem[BIAS ? 2 * kAttnMaxEdge + 1 : 1];
    __shared__ float wsum[4][32];
    __shared__ uint64_t words[S::kSets][128];
    P p(a, line_mem);
    const int lane = p.lane, wid = p.wid, set = ALONE ? wid : 0;
    if (BIAS) {
        load_line(a, p.head, p.line, threadIdx.x, 256);
        __syncthreads();
    }
    typename E::Frag qf[NK], gf[NK];
    load_row_frags<OP, DP>((const T*)a.q.p + p.b * a.q.sb + (int64_t)p.i * a.q.sr + p.head * a.q.sh,
                           p.row_ok, a.d, a.q.vec, lane, qf);
    load_row_frags<OP, DP>((const T*)a.go.p + p.b * a.go.sb + (int64_t)p.i * a.go.sr + p.head * a.go.sh,
                           p.row_ok, a.dv, a.go.vec, lane, gf);
    f32x16 acc[ND];
#pragma unroll
    for (int x = 0; x < ND; ++x)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[x][r] = 0.f;
    DsScale<OP, ND> dss;
    float rest = 0.f;  // sum of dS
    const T* kbase = (const T*)a.k.p + p.b * a.k.sb + p.kvh * a.k.sh;
    const T* vbase = (const T*)a.v.p + p.b * a.v.sb + p.kvh * a.v.sh;
    const uint32_t tile0 = lds_addr(tiles[set]);
    const typename L::Lanes lanes(tile0, lane);
    // tiles u of this wave (or workgroup) start at key j_first + u stride
    const int j_first = ALONE ? wid * KT : 0, stride = ALONE ? 4 * KT : KT;
    const SeenKeys<kPart, ALONE ? 1 : 4> keys{a.key_mask ? a.key_mask + p.b * a.mask_stride : nullptr,
                                              lds_addr(words[set]), j_first, stride / kParts, p.len};
    const int n_tiles = p.len > j_first ? (p.len - j_first + stride - 1) / stride : 0;
    const auto fetch = [&](int u, int buf) {
        const int t = ALONE ? lane : (int)threadIdx.x;
#pragma unroll
        for (int x = 0; x < kParts; ++x) {
            const int64_t j0 = j_first + (int64_t)u * stride + x * kPart;
            const uint64_t seen = keys(u * kParts + x);
            const uint32_t lds = tile0 + 2 * buf * kBytes + x * kPart * L::kRow;
            Load::fill(lds, kbase + j0 * a.k.sr, a.k.sr, seen, a.d, a.k.vec, t);
            Load::fill(lds + kBytes, vbase + j0 * a.v.sr, a.v.sr, seen, a.dv, a.v.vec, t);
        }
    };
    if (n_tiles) {
        keys.fill(0, lane, ALONE ? 0 : wid);
        if (ALONE)
            wave_fence();
        else if (a.key_mask)
            __syncthreads();
        fetch(0, 0);
    }
    int cur = 0;
    for (int u = 0; u < n_tiles; ++u) {
        dma_wait();
        if (ALONE)
            wave_fence();
        else
            __builtin_amdgcn_s_barrier();
        // the words of the 64 after these (the next fetch needs them at the earliest)
        if (u * kParts % 64 == 0) {
            keys.fill(u * kParts + 64, lane, ALONE ? 0 : wid);
            wave_fence();
        }
        const typename L::Lanes now(lanes, cur * 2 * kBytes);
        if (S::kBufs == 2) {
            cur ^= 1;
            if (u + 1 < n_tiles) fetch(u + 1, cur);
        }
#pragma unroll 2
        for (int nb = 0; nb < KT / 32; ++nb) {
            const int j0 = j_first + u * stride + 32 * nb, o = 32 * nb * L::kRow;
            const uint32_t vis = (uint32_t)(keys(u * kParts + nb / 2) >> (32 * (nb & 1)));
            f32x16 s, dp;
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.f;
            auto prod = products<L::kRow == 256 ? 3 : kAhead, 2 * NK, 2 * ND, typename E::Frag>([&](int y) {
                if (y < 2 * NK) return L::frag_rows(now, y % 2 * kBytes + o, y / 2);
                y -= 2 * NK;
                return L::frag_cols(now, o + 16 * (y / ND) * L::kRow, y % ND);
            });
            prod.first([&](int y, typename E::Frag op) {
                if (y % 2)
                    dp = E::mfma(op, gf[y / 2], dp);
                else
                    s = E::mfma(op, qf[y / 2], s);
            });
            float cm, ca, x = 0.f;
            p.prepare(a, j0, vis, s, cm, ca);
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                dp[r] = ex2(fmaf(s[r], cm, ca)) * (dp[r] - p.rd);
                x += dp[r];
            }
            rest += x;
            dss.apply(dp, acc);
            const typename E::Frag df[2] = {L::pack(dp, 0), L::pack(dp, 1)};
            prod.second([&](int y, typename E::Frag op) { acc[y % ND] = E::mfma(op, df[y / ND], acc[y % ND]); });
        }
        if (S::kBufs == 1 && u + 1 < n_tiles) {
            dma_wait();
            wave_fence();
            fetch(u + 1, 0);
        }
    }
    rest = half_sum(rest);
    const float f = a.scale * dss.undo();
#pragma unroll
    for (int cb = 0; cb < ND; ++cb)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[cb][r] *= f;
    if (ALONE) {
        if (p.h == 0) wsum[wid][lane] = rest;
        join_waves<DP, ND>(acc, LdsFloats{lds_addr(tiles)}, wid, lane);
        if (wid > 0) return;
        rest = (wsum[0][lane & 31] + wsum[1][lane & 31]) + (wsum[2][lane & 31] + wsum[3][lane & 31]);
    }
    p.store(a, acc, rest);
}

// dT[bucket, head]: the bucket's positions of every part's line, in 64 bits
// and a fixed order.  One workgroup per entry (5 us for 32 buckets, 16 heads).
__global__ __launch_bounds__(256) void attn_bias_sum_kernel(const AttnArgs a) {
    __shared__ double red[256];
    const int bucket = blockIdx.x, head = blockIdx.y, t = threadIdx.x;
    const int n_line = a.r0 + a.rp + 1;
    const int parts = a.B * a.line_blocks;
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

template <int OP, int DP, bool ALONE>
hipError_t bwd_kv_as(const AttnArgs& a, hipStream_t s) {
    constexpr int rows = BwdShape<OP, DP, ALONE, 64>::kRows;
    const unsigned g = (unsigned)((int64_t)a.B * a.K * a.q_split * ((a.m + rows - 1) / rows));
    const size_t lds = a.bias ? (size_t)5 * (a.r0 + a.rp + 1) * sizeof(float) : 0;
    constexpr int one = Tile<OP, DP>::kRow <= 256 ? PART_BOTH : PART_DK;
    if (a.bias)
        attn_bwd_kv_kernel<OP, DP, true, ALONE, one><<<g, 256, lds, s>>>(a);
    else
        attn_bwd_kv_kernel<OP, DP, false, ALONE, one><<<g, 256, lds, s>>>(a);
    if constexpr (one == PART_DK) {
        if (a.bias)
            attn_bwd_kv_kernel<OP, DP, true, ALONE, PART_DV><<<g, 256, lds, s>>>(a);
        else
            attn_bwd_kv_kernel<OP, DP, false, ALONE, PART_DV><<<g, 256, lds, s>>>(a);
    }
    return hipGetLastError();
}
template <int OP, int DP>
hipError_t bwd_kv(const AttnArgs& a, hipStream_t s) {
    if constexpr (Tile<OP, DP>::kRow <= 256)
        if (a.alone_k) return bwd_kv_as<OP, DP, true>(a, s);
    return bwd_kv_as<OP, DP, false>(a, s);
}

template <int OP, int DP, bool ALONE>
hipError_t bwd_q_as(const AttnArgs& a, hipStream_t s) {
    constexpr int rows = BwdShape<OP, DP, ALONE, 128>::kRows;
    const unsigned g = (unsigned)((int64_t)a.B * a.H * ((a.n + rows - 1) / rows));
    if (a.bias)
        attn_bwd_q_kernel<OP, DP, true, ALONE><<<g, 256, 0, s>>>(a);
    else
        attn_bwd_q_kernel<OP, DP, false, ALONE><<<g, 256, 0, s>>>(a);
    return hipGetLastError();
}
template <int OP, int DP>
hipError_t bwd_q(const AttnArgs& a, hipStream_t s) {
    if constexpr (Tile<OP, DP>::kRow <= 256)
        if (a.alone_q) return bwd_q_as<OP, DP, true>(a, s);
    return bwd_q_as<OP, DP, false>(a, s);
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
    const int64_t rows = (int64_t)a.B * a.n_pad * a.H;
    const dim3 g = flat_grid((rows + 15) / 16);
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
