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
// is stored at chunk c ^ swz(r): eight successive rows read at one c (the row
// operands) and four successive rows read at two neighbouring c (the column
// operands) then fall on different banks.
template <int OP, int DP>
struct Tile {
    using E = El<OP>;
    using T = typename E::T;
    using Frag = typename E::Frag;
    static constexpr int kEpc = 16 / sizeof(T);          // elements per chunk
    static constexpr int kCh = DP * (int)sizeof(T) / 16;  // chunks per row
    static constexpr int kRow = DP * (int)sizeof(T);      // bytes per row

    static __device__ __forceinline__ int swz(int r) {
        return (((r & 3) << 1) | ((r >> 2) & 1)) & (kCh - 1);
    }
    static __device__ __forceinline__ int at(int r, int c) { return r * kRow + ((c ^ swz(r)) << 4); }

    // Operand whose rows (or columns) are the tile's rows r0 + (lane & 31),
    // contraction over elements 16 kk + 8 h + 0..7.
    static __device__ __forceinline__ Frag frag_rows(uint32_t t, int r0, int kk, int lane) {
        const int r = r0 + (lane & 31), h = lane >> 5;
        if constexpr (sizeof(T) == 2) {
            return lds_read<Frag>(t + at(r, 2 * kk + h));
        } else {
            const f32x4 lo = lds_read<f32x4>(t + at(r, 4 * kk + 2 * h));
            const f32x4 hi = lds_read<f32x4>(t + at(r, 4 * kk + 2 * h + 1));
            return Frag{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        }
    }

    // Operand whose rows are the tile's elements 32 cb + (lane & 31),
    // contraction over the tile's rows r0 + 8 (e >> 2) + 4 h + (e & 3).
    // 16-bit types: ds_read_b64_tr_b16 hands lane i of 16 the i-th column of
    // the 4 x 16 block whose row i >> 2, columns 4 (i & 3) + 0..3 it addresses.
    static __device__ __forceinline__ Frag frag_cols(uint32_t t, int r0, int cb, int lane) {
        const int h = lane >> 5;
        if constexpr (sizeof(T) == 2) {
            typedef __attribute__((__vector_size__(8))) short s16x4;
            typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
            const int i = lane & 15;
            const int r = r0 + 4 * h + (i >> 2);
            const int c = cb * 4 + ((lane >> 4) & 1) * 2 + ((i & 3) >> 1);
            const uint32_t p = t + at(r, c) + (i & 1) * 8;
            union {
                s16x4 q[2];
                Frag f;
            } u;
            u.q[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)p);
            u.q[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)(p + 8 * kRow));
            return u.f;
        } else {
            Frag f;
            const int x = cb * 32 + (lane & 31);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int r = r0 + 8 * (e >> 2) + 4 * h + (e & 3);
                f[e] = lds_read<float>(t + at(r, x >> 2) + (x & 3) * 4);
            }
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

// Fills a tile of ROWS rows in LDS from global memory, by NT threads (whole
// waves; t counts within them).  Chunk positions in LDS are dealt out in
// order, so a lane fetches the chunk that belongs at its position.  Rows whose
// bit in `seen` is clear are filled with zeros and never read: what stands
// there (NaN in padding, memory behind the tensor) cannot enter a product.
// Aligned rows (vec) go straight to LDS and are complete after dma_wait();
// others are loaded element by element and stored at once.
template <int OP, int DP, int ROWS, int NT>
struct Loader {
    using L = Tile<OP, DP>;
    using T = typename El<OP>::T;
    static constexpr int kN = ROWS * L::kCh / NT, kStep = NT / L::kCh;
    static_assert(ROWS * L::kCh % NT == 0 && NT % L::kCh == 0, "whole rows per step");
    static constexpr uint64_t kAll = ROWS == 64 ? ~0ull : (1ull << ROWS) - 1;

    static __device__ __forceinline__ void fill(uint32_t lds, const T* base, int64_t stride,
                                                uint64_t seen, int w, bool vec, int t) {
        const int c0 = t % L::kCh, r0 = t / L::kCh;
        const uint32_t dst = lds + (t & ~63) * 16;
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
#pragma unroll
            for (int s = 0; s < kN; ++s) {
                const int r = r0 + s * kStep, c = c0 ^ L::swz(r);
                T x[L::kEpc];
#pragma unroll
                for (int e = 0; e < L::kEpc; ++e) x[e] = (T)0.f;
                if ((seen >> r) & 1) load_elems<OP, L::kEpc>(base + r * stride, c * L::kEpc, w, false, x);
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

// The keys of a batch entry that exist, and the position of query row 0.
__device__ __forceinline__ int attn_kv_len(const AttnArgs& a, int b) {
    return a.kv_len ? min(max(a.kv_len[b], 0), a.m) : a.m;
}
__device__ __forceinline__ int attn_q_len(const AttnArgs& a, int b) {
    return a.q_len ? min(max(a.q_len[b], 0), a.n) : a.n;
}
__device__ __forceinline__ int attn_offset(const AttnArgs& a, int b) {
    const int o = a.offsets ? a.offsets[b] : a.offset;
    return min(max(o, -kAttnMaxOffset), kAttnMaxOffset);
}

// Bit x: key j0 + x (x < 64) exists and is not masked out.
__device__ __forceinline__ uint64_t seen_keys(const AttnArgs& a, int b, int len, int j0, int lane) {
    bool s = j0 + lane < len;
    if (a.key_mask && s) s = a.key_mask[b * a.mask_stride + j0 + lane] != 0;
    return __ballot(s);
}
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
// A value of -1e30 or less (the type's lowest among them) is taken as -inf, no
// weight: in base 2 the lowest would leave the range, and next to it scores
// would be lost in rounding anyway.
__device__ __forceinline__ float bias2(float x) { return x <= -1e30f ? -INFINITY : x * kLog2e; }
__device__ __forceinline__ void load_line(const AttnArgs& a, int head, LdsFloats line, int t, int nt) {
    for (int i = t; i < a.r0 + a.rp + 1; i += nt)
        line.set(i, bias2(a.bias[(int64_t)bucket_of(a, i - a.r0) * a.H + head]));
}

// Work item of a 1-D grid, consecutive ones on the same XCD: workgroups go to
// the 8 XCDs round-robin, and those that read the same keys then share an L2.
__device__ __forceinline__ int xcd_item(int id, int total) {
    const int x = id & 7, q = total >> 3, r = total & 7;
    return x * q + min(x, r) + (id >> 3);
}

}  // namespace fs
