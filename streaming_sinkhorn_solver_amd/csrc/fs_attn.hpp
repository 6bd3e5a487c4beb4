// fs_attn.hpp -- device-side pieces shared by the attention kernels: element
// types on the 32x32 matrix instructions, staged tiles in LDS read along rows
// and across them, the visible keys of a tile and the bucket bias.
//
// Every product of these kernels is a sum of v_mfma_f32_32x32 blocks.  Lane l
// holds, of an A (or B) operand block, row (or column) l & 31 at eight
// contraction indices that belong to its half h = l >> 5; of the 32x32 result
// it holds column l & 31 at rows 8 (r >> 2) + 4 h + (r & 3), r = 0..15.  Scores
// are formed with the index that the next product sums over in the rows, so
// that a lane's sixteen results, rounded, are two operands of that product as
// they stand: operand rc, element e is result 8 rc + e, which is contraction
// index 16 rc + 8 (e >> 2) + 4 h + (e & 3).  The other operand is gathered
// from LDS in the same order (frag_cols).
#pragma once

#include "fs_attn_args.h"
#include "fs_device.hpp"

namespace fs {

// Element types.  Frag: eight contraction elements of a lane.
template <int OP>
struct El;

template <>
struct El<OP_BF16> {
    using T = __bf16;
    using Frag = bf16x8;
    static __device__ __forceinline__ f32x16 mfma(Frag a, Frag b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};

template <>
struct El<OP_F16> {
    using T = _Float16;
    using Frag = f16x8;
    static __device__ __forceinline__ f32x16 mfma(Frag a, Frag b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};

// fp32: the same sixteen contraction indices as eight 32x32x2 products (the
// order of a sum's terms is free, so element e of both halves makes one).
template <>
struct El<OP_F32> {
    using T = float;
    typedef __attribute__((__vector_size__(32))) float Frag;
    static __device__ __forceinline__ f32x16 mfma(Frag a, Frag b, f32x16 c) {
#pragma unroll
        for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], c, 0, 0, 0);
        return c;
    }
};

// The wave's number in its workgroup, known to the compiler to be one for all
// its lanes.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Shared memory by its LDS address (the low half of a shared object's generic
// address): loads and stores of a known address space whatever the pointer
// went through.
__device__ __forceinline__ uint32_t lds_addr(const void* p) { return (uint32_t)(uintptr_t)p; }
template <typename V>
__device__ __forceinline__ V lds_read(uint32_t a) {
    typedef __attribute__((address_space(3))) V lds_v;
    return *(const lds_v*)(uintptr_t)a;
}
template <typename V>
__device__ __forceinline__ void lds_write(uint32_t a, const V& v) {
    typedef __attribute__((address_space(3))) V lds_v;
    *(lds_v*)(uintptr_t)a = v;
}
struct LdsFloats {
    uint32_t a;
    __device__ __forceinline__ float operator[](int i) const { return lds_read<float>(a + 4 * i); }
    __device__ __forceinline__ void set(int i, float x) const { lds_write<float>(a + 4 * i, x); }
};

// The other half's value of the same column (lane l ^ 32).
__device__ __forceinline__ float half_max(float x) {
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// A tile of rows of DP elements in LDS, in 16-byte chunks.  Chunk c of row r
// is stored at chunk c ^ swz(r).  Sixteen successive rows read at one c (the
// row operands, 256 bytes a clock) then fall on the 64 banks once each, and so
// do four successive rows read at two neighbouring c (the column operands).
// Measured with four waves, cycles a wave's load: 2.9 against 4.0 for a
// swizzle over eight rows (2.7 for addresses in order).
template <int OP, int DP>
struct Tile {
    using E = El<OP>;
    using T = typename E::T;
    using Frag = typename E::Frag;
    static constexpr int kEpc = 16 / sizeof(T);          // elements per chunk
    static constexpr int kCh = DP * (int)sizeof(T) / 16;  // chunks per row
    static constexpr int kRow = DP * (int)sizeof(T);      // bytes per row

    // rows of 128 bytes: two rows lie side by side in the banks
    static __device__ __forceinline__ int swz(int r) {
        return kRow == 128 ? (r & 2) | ((r >> 2) & 1) | ((r >> 1) & 4)
                           : ((r & 3) << 1) | ((r >> 2) & 1) | (r & 8);
    }
    static __device__ __forceinline__ int at(int r, int c) { return r * kRow + ((c ^ swz(r)) << 4); }

    // The swizzle moves chunks within groups of sixteen (eight), so an operand's
    // address is one of a few values of the lane plus a constant, which the
    // load instruction holds (the values are kept opaque, or the compiler would
    // form each address anew).
    static constexpr int kGroup = kRow == 128 ? 8 : 16;           // chunks of a group
    static constexpr int kRowAddrs = kGroup / 2;                  // (kk, half) of a group
    static constexpr int kColAddrs = sizeof(T) == 2 ? kGroup / 4 : 8;
    struct Lanes {
        uint32_t rows[kRowAddrs], cols[kColAddrs];
        __device__ __forceinline__ Lanes(uint32_t t, int lane) {
            const int r = lane & 31, h = lane >> 5, i = lane & 15;
#pragma unroll
            for (int x = 0; x < kRowAddrs; ++x) {
                rows[x] = t + (sizeof(T) == 2 ? at(r, 2 * x + h) : at(r, 4 * (x >> 1) + 2 * h + (x & 1)));
                asm volatile("" : "+v"(rows[x]));
            }
#pragma unroll
            for (int x = 0; x < kColAddrs; ++x) {
                cols[x] = t + (sizeof(T) == 2 ? at(4 * h + (i >> 2), x * 4 + ((lane >> 4) & 1) * 2 + ((i & 3) >> 1)) + (i & 1) * 8
                                              : at(4 * h + (x & 3), (x >> 2) * 8 + (r >> 2)) + (r & 3) * 4);
                asm volatile("" : "+v"(cols[x]));
            }
        }
        // the same in another buffer
        __device__ __forceinline__ Lanes(const Lanes& l, uint32_t offset) {
#pragma unroll
            for (int x = 0; x < kRowAddrs; ++x) rows[x] = l.rows[x] + offset;
#pragma unroll
            for (int x = 0; x < kColAddrs; ++x) cols[x] = l.cols[x] + offset;
        }
        // the same, in place of these: half the registers where they are scarce
        __device__ __forceinline__ void move(uint32_t offset) {
#pragma unroll
            for (int x = 0; x < kRowAddrs; ++x) rows[x] += offset;
#pragma unroll
            for (int x = 0; x < kColAddrs; ++x) cols[x] += offset;
        }
    };

    // Operand whose rows (or columns) are the tile's rows r0 + (lane & 31),
    // contraction over elements 16 kk + 8 h + 0..7.  o: the tile's offset plus
    // r0 * kRow, r0 a multiple of 16.
    static __device__ __forceinline__ Frag frag_rows(const Lanes& l, int o, int kk) {
        if constexpr (sizeof(T) == 2) {
            return lds_read<Frag>(l.rows[kk % kRowAddrs] + o + kk / kRowAddrs * (16 * kGroup));
        } else {
            const int c = 2 * kk % kRowAddrs;
            o += 2 * kk / kRowAddrs * (16 * kGroup);
            const f32x4 lo = lds_read<f32x4>(l.rows[c] + o);
            const f32x4 hi = lds_read<f32x4>(l.rows[c + 1] + o);
            return Frag{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        }
    }

    // Operand whose rows are the tile's elements 32 cb + (lane & 31),
    // contraction over the tile's rows r0 + 8 (e >> 2) + 4 h + (e & 3); o as
    // above.  16-bit types: ds_read_b64_tr_b16 hands lane i of 16 the i-th
    // column of the 4 x 16 block whose row i >> 2, columns 4 (i & 3) + 0..3 it
    // addresses.  Rows eight further on have their chunks exchanged between the
    // halves of a group.
    static __device__ __forceinline__ Frag frag_cols(const Lanes& l, int o, int cb) {
        if constexpr (sizeof(T) == 2) {
            typedef __attribute__((__vector_size__(8))) short s16x4;
            typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
            const int c = cb % kColAddrs;
            o += cb / kColAddrs * (16 * kGroup);
            union {
                s16x4 q[2];
                Frag f;
            } u;
            u.q[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)(l.cols[c] + o));
            u.q[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4*)(uintptr_t)(l.cols[c ^ (kColAddrs / 2)] + o + 8 * kRow));
            return u.f;
        } else {
            Frag f;
            o += cb / 2 * 256;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[e] = lds_read<float>(l.cols[(e & 3) + 4 * ((cb & 1) ^ (e >> 2))] + o + 8 * (e >> 2) * kRow);
            return f;
        }
    }

    // Eight results of a lane (registers 8 rc .. 8 rc + 7) as an operand.
    static __device__ __forceinline__ Frag pack(const f32x16& x, int rc) {
        Frag f;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = (T)x[8 * rc + e];
        return f;
    }
};

// Two runs of products whose operands come from LDS, with vector work between
// them.  Operands are read A products ahead, across the gap (the order is
// pinned: left to itself the compiler reads each operand right before its
// product and waits out the latency of LDS every time).
template <int A, int N1, int N2, typename Frag, typename Operand>
struct Products {
    Frag f[A];
    Operand operand;
    __device__ __forceinline__ Products(Operand o) : operand(o) {
#pragma unroll
        for (int x = 0; x < A; ++x)
            if (x < N1 + N2) f[x] = operand(x);
    }
    template <int FROM, int TO, typename Product>
    __device__ __forceinline__ void run(Product product) {
#pragma unroll
        for (int x = FROM; x < TO; ++x) {
            __builtin_amdgcn_sched_barrier(0);
            const Frag op = f[x % A];
            if (x + A < N1 + N2) f[x % A] = operand(x + A);
            product(x - FROM, op);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    template <typename Product>
    __device__ __forceinline__ void first(Product product) { run<0, N1>(product); }
    template <typename Product>
    __device__ __forceinline__ void second(Product product) { run<N1, N1 + N2>(product); }
};
template <int A, int N1, int N2, typename Frag, typename Operand>
__device__ __forceinline__ Products<A, N1, N2, Frag, Operand> products(Operand o) {
    return Products<A, N1, N2, Frag, Operand>(o);
}

// Eight elements of a row in global memory from element x0 on, zero behind
// width d.  vec: the row is 16-byte aligned and d a multiple of a chunk.
template <int OP, int N>
__device__ __forceinline__ void load_elems(const typename El<OP>::T* row, int x0, int d, bool vec,
                                           typename El<OP>::T (&out)[N]) {
    using T = typename El<OP>::T;
    constexpr int kEpc = 16 / sizeof(T);
    static_assert(N % kEpc == 0, "whole chunks");
    if (vec) {
#pragma unroll
        for (int c = 0; c < N / kEpc; ++c) {
            u32x4 v = {0, 0, 0, 0};
            if (x0 + c * kEpc < d) v = *(const u32x4*)(row + x0 + c * kEpc);
            __builtin_memcpy(&out[c * kEpc], &v, 16);
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) out[e] = x0 + e < d ? row[x0 + e] : (T)0.f;
    }
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

// Operand fragments of one row held for a whole kernel: elements 16 kk + 8 h.
template <int OP, int DP>
__device__ __forceinline__ void load_row_frags(const typename El<OP>::T* row, bool valid, int d,
                                               bool vec, int lane,
                                               typename El<OP>::Frag (&f)[DP / 16]) {
    using T = typename El<OP>::T;
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
        T x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (T)0.f;
        if (valid) load_elems<OP, 8>(row, 16 * kk + 8 * (lane >> 5), d, vec, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[kk][e] = x[e];
    }
}

// Sixteen bytes that no one writes: the source of rows that do not exist.
static __device__ __attribute__((aligned(16))) const uint32_t attn_zeros[4] = {0, 0, 0, 0};

// One wave-wide 16-byte-per-lane copy to LDS: lane i's bytes at src_i land at
// lds + 16 i (lds wave-uniform).  Not modelled by the compiler: the
// caller waits (dma_wait) before it reads, and before a barrier publishes it.
__device__ __forceinline__ void dma_lane16(const char* src, uint32_t lds) {
    uint32_t saved;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %1\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %2, off\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(src)
        : "memory");
}
// The same with 4 bytes a lane.
__device__ __forceinline__ void dma_lane4(const char* src, uint32_t lds) {
    uint32_t saved;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %1\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dword %2, off\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(src)
        : "memory");
}
// The wave's copies have landed and its own LDS reads are done (so the buffer
// they came from may be filled again).
__device__ __forceinline__ void dma_wait() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
}
// The same but for the wave's last N copies (loads complete in order).
template <int N>
__device__ __forceinline__ void dma_wait_but() {
    static_assert(N < 64, "a six-bit counter");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// Fills a tile of ROWS rows in LDS from global memory, by NT threads (whole
// waves; t counts within them).  Chunk positions in LDS are dealt out in
// order, so a lane fetches the chunk that belongs at its position.  Rows whose
// bit in `seen` is clear are filled with zeros and never read: what stands
// there (NaN in padding, memory behind the tensor) cannot enter a product.
// Aligned rows (vec) go straight to LDS and are complete after dma_wait();
// others are loaded element by element and stored at once.  A thread's places in a
// tile are the same at every fill and the compiler would keep them; for kernels
// without the registers they are formed anew: those of the element path only, or
// of both (kept in memory, they are read again between the copies, and each read
// waits for the copies before it).
enum Places { PLACES_KEPT, PLACES_KEPT_WIDE, PLACES_ANEW };
template <int OP, int DP, int ROWS, int NT, Places PLACES = PLACES_KEPT>
struct Loader {
    using L = Tile<OP, DP>;
    using T = typename El<OP>::T;
    static constexpr int kN = ROWS * L::kCh / NT, kStep = NT / L::kCh;
    static_assert(ROWS * L::kCh % NT == 0 && NT % L::kCh == 0 && ROWS <= 64,
                  "whole rows per step, a flag each");
    static constexpr uint64_t kAll = ROWS >= 64 ? ~0ull : (1ull << ROWS) - 1;

    static __device__ __forceinline__ void fill(uint32_t lds, const T* base, int64_t stride,
                                                uint64_t seen, int w, bool vec, int t) {
        if (PLACES == PLACES_ANEW) asm volatile("" : "+v"(t));
        int c0 = t % L::kCh, r0 = t / L::kCh;
        const uint32_t dst = lds + (NT == 64 ? 0 : wave_id() * 1024);
        if (vec) {
            const char* src = (const char*)(base + r0 * stride);
            const int64_t step = kStep * stride * (int64_t)sizeof(T);
            if (w == DP && (seen & kAll) == kAll) {
#pragma unroll
                for (int s = 0; s < kN; ++s, src += step)
                    dma_lane16(src + ((c0 ^ L::swz(r0 + s * kStep)) << 4), dst + s * NT * 16);
            } else {
#pragma unroll
                for (int s = 0; s < kN; ++s, src += step) {
                    const int r = r0 + s * kStep, c = c0 ^ L::swz(r);
                    const bool ok = ((seen >> r) & 1) && c * L::kEpc < w;
                    dma_lane16(ok ? src + (c << 4) : (const char*)attn_zeros, dst + s * NT * 16);
                }
            }
        } else {
            if (PLACES == PLACES_KEPT_WIDE) {
                asm volatile("" : "+v"(t));
                c0 = t % L::kCh, r0 = t / L::kCh;
            }
#pragma unroll
            for (int s = 0; s < kN; ++s) {
                const int r = r0 + s * kStep, c = c0 ^ L::swz(r);
                T x[L::kEpc];
#pragma unroll
                for (int e = 0; e < L::kEpc; ++e) x[e] = (T)0.f;
                if (((seen >> r) & 1)) load_elems<OP, L::kEpc>(base + r * stride, c * L::kEpc, w, false, x);
                u32x4 v;
                __builtin_memcpy(&v, x, 16);
                lds_write<u32x4>(lds + (s * NT + t) * 16, v);
            }
        }
    }
};

// Order between a wave's own LDS stores and loads (issued in order; the fence
// keeps the compiler from exchanging them).
__device__ __forceinline__ void wave_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// The keys and queries of a batch entry that exist, and the position of query
// row 0.  The entry is the whole wave's: said so, what follows from them stays
// in scalar registers, and with it the tiles' addresses.
__device__ __forceinline__ int row_len(const int* len, int b, int n) {
    return len ? min(max(len[b], 0), n) : n;
}
__device__ __forceinline__ int attn_kv_len(const AttnArgs& a, int b) {
    return __builtin_amdgcn_readfirstlane(row_len(a.kv_len, b, a.m));
}
__device__ __forceinline__ int attn_q_len(const AttnArgs& a, int b) {
    return __builtin_amdgcn_readfirstlane(row_len(a.q_len, b, a.n));
}
__device__ __forceinline__ int attn_offset(const AttnArgs& a, int b) {
    const int o = a.offsets ? a.offsets[b] : a.offset;
    return __builtin_amdgcn_readfirstlane(min(max(o, -kAttnMaxOffset), kAttnMaxOffset));
}

// Which of the keys of a tile of KT (at most 64) exist and are not masked out:
// bit x of tile u's word for key j_first + u stride + x < je.  Without a mask
// the word follows from je; with one, words are formed 64 tiles at a time and
// kept in LDS (one wave's work, W waves sharing it), so that no tile's fetch
// waits for a mask byte.
template <int KT, int W>
struct SeenKeys {
    const uint8_t* mask;  // of this batch entry, or NULL
    uint32_t words;       // LDS address of 128 words
    int j_first, stride, je;

    // words of tiles u .. u + 63 (all lanes of the wave; part wid of W), eight
    // loads at a time
    __device__ __forceinline__ void fill(int u, int lane, int wid) const {
        if (!mask) return;
#pragma unroll 1
        for (int v = u + wid * 8; v < u + 64 && j_first + (int64_t)v * stride < je; v += 8 * W) {
            bool ok[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const int64_t j = j_first + (int64_t)(v + x) * stride + lane;
                ok[x] = lane < KT && j < je && mask[j] != 0;
            }
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const uint64_t w = __ballot(ok[x]);
                if (lane == 0) lds_write<uint64_t>(words + 8 * ((v + x) & 127), w);
            }
        }
    }
    __device__ __forceinline__ uint64_t operator()(int u) const {
        const int64_t left = je - (j_first + (int64_t)u * stride);
        if (left <= 0) return 0;
        if (mask) {
            const uint64_t w = lds_read<uint64_t>(words + 8 * (u & 127));
            const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(w >> 32));
            const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)w);
            return ((uint64_t)hi << 32) | lo;
        }
        return left >= KT ? (KT == 64 ? ~0ull : (1ull << (KT & 63)) - 1) : (1ull << left) - 1;
    }
};
// Bits 0 .. x (none for x < 0).
__device__ __forceinline__ uint32_t bits_upto(int x) {
    return x < 0 ? 0u : x >= 31 ? ~0u : (2u << x) - 1u;
}
// result register r of a lane stands for index 8 (r >> 2) + 4 h + (r & 3);
// w is the word of 32 flags shifted right by 4 h
__device__ __forceinline__ bool flag(uint32_t w, int r) {
    return (w >> (8 * (r >> 2) + (r & 3))) & 1u;
}

// ---- bucket bias ----------------------------------------------------------
// The bias depends on r = j - i - offset alone and is constant below -R0 and
// above RP (R0 the last edge; RP = R0 two-sided, else 0), so a head's bias is
// a line of R0 + RP + 1 values, kept in LDS in base-2 units.
__device__ __forceinline__ int line_index(const AttnArgs& a, int r) {
    return min(max(r, -a.r0), a.rp) + a.r0;
}
__device__ __forceinline__ int bucket_of(const AttnArgs& a, int r) {
    const int dist = a.two_sided ? abs(r) : max(-r, 0);
    int c = 0;
    for (int e = 0; e < a.n_edges; ++e) c += dist >= (int)a.edges[e];
    return c + (a.two_sided && r > 0 ? a.n_edges + 1 : 0);
}
// A value of -1e6 or less stands for a mask and is taken as -inf, no weight.  Next
// to any other key it has none in fp32 either; in a row that has no other the
// scores would be lost beside it, and with them L's last digits: exp(s - L) of the
// backward pass would be off by 2^(half a step of L in base 2), 4% at -1e6 but 2^64
// at -1e9 (gradients of 1e37).  The lowest values would leave the range in base 2.
constexpr float kNoWeight = -1e6f;
__device__ __forceinline__ float bias2(float x) { return x <= kNoWeight ? -INFINITY : x * kLog2e; }
__device__ __forceinline__ void load_line(const AttnArgs& a, int head, LdsFloats line, int t, int nt) {
    for (int i = t; i < a.r0 + a.rp + 1; i += nt)
        line.set(i, bias2(a.bias[(int64_t)bucket_of(a, i - a.r0) * a.H + head]));
}

// Work item of a 1-D grid whose items come in groups of `group` that read the
// same keys.  Workgroups go to the 8 XCDs round-robin and each XCD has its own
// L2, so a group's items are given to one XCD, and the groups to the XCDs in
// turn (sequences of unequal length then spread over them); where the groups
// are not a multiple of 8, each XCD takes an equal run of items instead.
__device__ __forceinline__ int xcd_item(int id, int total, int group) {
    const int x = id & 7, k = id >> 3;
    if (total / group % 8 == 0) return (k / group * 8 + x) * group + k % group;
    const int q = total >> 3, r = total & 7;
    return x * q + min(x, r) + k;
}

}  // namespace fs
