// fs_rowops.hpp -- device-side pieces of the kernels that work on whole rows:
// sums and maxima over a row's lanes, and a lane's share of a row's elements.
#pragma once

#include "fs_attn.hpp"
#include "fs_layers_args.h"

namespace fs {

// Lane l's value at lane l ^ O (O < 16: of a mirror image, for which the lanes
// below O agree already; 16, 32: of the other row or half).
template <int O>
__device__ __forceinline__ uint32_t lane_other(uint32_t x) {
    if constexpr (O == 1) return __builtin_amdgcn_update_dpp(0u, x, 0xB1, 0xF, 0xF, true);
    if constexpr (O == 2) return __builtin_amdgcn_update_dpp(0u, x, 0x4E, 0xF, 0xF, true);
    if constexpr (O == 4) return __builtin_amdgcn_update_dpp(0u, x, 0x141, 0xF, 0xF, true);
    if constexpr (O == 8) return __builtin_amdgcn_update_dpp(0u, x, 0x140, 0xF, 0xF, true);
    const bool upper = threadIdx.x & O;
    if constexpr (O == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        return upper ? r[0] : r[1];
    }
    if constexpr (O == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        return upper ? r[0] : r[1];
    }
}
template <int O>
__device__ __forceinline__ float lane_other(float x) {
    return __uint_as_float(lane_other<O>(__float_as_uint(x)));
}

// f over the LPR lanes (a power of two, up to 64) of a lane group; all lanes get
// the result, and the same bits.
template <int LPR, typename V, typename F>
__device__ __forceinline__ V lanes_fold(V x, F f) {
    if constexpr (LPR > 1) x = f(x, lane_other<1>(x));
    if constexpr (LPR > 2) x = f(x, lane_other<2>(x));
    if constexpr (LPR > 4) x = f(x, lane_other<4>(x));
    if constexpr (LPR > 8) x = f(x, lane_other<8>(x));
    if constexpr (LPR > 16) x = f(x, lane_other<16>(x));
    if constexpr (LPR > 32) x = f(x, lane_other<32>(x));
    return x;
}
template <int LPR>
__device__ __forceinline__ float lanes_sum(float x) {
    return lanes_fold<LPR>(x, [](float a, float b) { return a + b; });
}
template <int LPR>
__device__ __forceinline__ float lanes_max(float x) {
    return lanes_fold<LPR>(x, [](float a, float b) { return fmaxf(a, b); });
}
template <int LPR>
__device__ __forceinline__ uint32_t lanes_max(uint32_t x) {
    return lanes_fold<LPR>(x, [](uint32_t a, uint32_t b) { return max(a, b); });
}

// Threads of a workgroup whose rows lie with LPR threads each.
template <int LPR>
constexpr int threads_of() {
    return LPR > 256 ? LPR : 256;
}

// Sums over the LPR threads of a row, of whole waves if more than 64: the waves'
// sums meet in LDS.  Two buffers in turn, so that one barrier a sum is enough: a
// buffer is written again only behind the next sum's barrier, in front of which
// everyone has read it.
template <int LPR>
struct RowFold {
    static constexpr int kWaves = LPR > 64 ? LPR / 64 : 1;
    float2* buf;  // [2 kWaves] in LDS
    int turn = 0;
    __device__ __forceinline__ explicit RowFold(float2* b) : buf(b) {}
    __device__ __forceinline__ float2 sum2(float a, float b) {
        constexpr int L = LPR > 64 ? 64 : LPR;
        a = lanes_sum<L>(a);
        b = lanes_sum<L>(b);
        if constexpr (LPR > 64) {
            float2* at = buf + turn * kWaves;
            if ((threadIdx.x & 63) == 0) at[threadIdx.x >> 6] = make_float2(a, b);
            stage_barrier();  // (the rows' loads that are under way are not waited for)
            a = b = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) a += at[w].x, b += at[w].y;
            turn ^= 1;
        }
        return make_float2(a, b);
    }
    __device__ __forceinline__ float sum(float a) {
        constexpr int L = LPR > 64 ? 64 : LPR;
        a = lanes_sum<L>(a);
        if constexpr (LPR > 64) {
            float2* at = buf + turn * kWaves;
            if ((threadIdx.x & 63) == 0) at[threadIdx.x >> 6].x = a;
            stage_barrier();  // (the rows' loads that are under way are not waited for)
            a = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) a += at[w].x;
            turn ^= 1;
        }
        return a;
    }
    __device__ __forceinline__ uint32_t max_bits(uint32_t a) {
        constexpr int L = LPR > 64 ? 64 : LPR;
        a = lanes_max<L>(a);
        if constexpr (LPR > 64) {
            float2* at = buf + turn * kWaves;
            if ((threadIdx.x & 63) == 0) at[threadIdx.x >> 6].x = __uint_as_float(a);
            stage_barrier();  // (the rows' loads that are under way are not waited for)
            a = 0;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) a = max(a, __float_as_uint(at[w].x));
            turn ^= 1;
        }
        return a;
    }
};

// A lane's share of a row of `width` elements: CH groups of 8.  WIDE: groups of
// neighbours, read with 16 bytes a lane (rows are whole, aligned groups).  DWORDS: the
// same of rows that only start at whole dwords, which 16-byte accesses may; the last
// group may be a part.  SINGLE: single elements, LPR apart, so that a wave reads
// neighbours.
template <int LPR, ShareForm FORM>
__device__ __forceinline__ int share_at(int lane, int j, int e) {
    return FORM != SINGLE ? (lane + j * LPR) * 8 + e : (j * 8 + e) * LPR + lane;
}

template <typename T, int LPR, int CH, ShareForm FORM>
struct Share {
    T v[CH][8];
    // on: the row takes part; zeros stand for one that does not.  A lane without an
    // element (of a whole group) reads the row's first and leaves it: loads that ask
    // nothing are all under way before the first is waited for.
    __device__ __forceinline__ void load(const T* row, int lane, int width, bool on) {
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            if constexpr (FORM != SINGLE) {
                constexpr int N = 2 * sizeof(T);
                const int at = share_at<LPR, FORM>(lane, j, 0);
                const bool in = on && (FORM == WIDE ? at < width : at + 8 <= width);
                uint32_t w[N];
                __builtin_memcpy(w, __builtin_assume_aligned(row + (in ? at : 0), FORM == WIDE ? 16 : 4),
                                 sizeof(w));
#pragma unroll
                for (int i = 0; i < N; ++i) w[i] = in ? w[i] : 0u;
                __builtin_memcpy(v[j], w, sizeof(w));
                if (FORM == DWORDS && on && !in && at < width) {
#pragma unroll
                    for (int e = 0; e < 7; ++e)
                        if (at + e < width) v[j][e] = row[at + e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int at = share_at<LPR, FORM>(lane, j, e);
                    const bool in = on && at < width;
                    const T t = row[in ? at : 0];
                    v[j][e] = in ? t : (T)0.f;
                }
            }
        }
    }
    __device__ __forceinline__ void store(T* row, int lane, int width) const {
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            if constexpr (FORM != SINGLE) {
                const int at = share_at<LPR, FORM>(lane, j, 0);
                if (FORM == WIDE ? at < width : at + 8 <= width) {
                    __builtin_memcpy(__builtin_assume_aligned(row + at, FORM == WIDE ? 16 : 4), v[j],
                                     sizeof(v[j]));
                } else if (FORM == DWORDS && at < width) {
#pragma unroll
                    for (int e = 0; e < 7; ++e)
                        if (at + e < width) row[at + e] = v[j][e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int at = share_at<LPR, FORM>(lane, j, e);
                    if (at < width) row[at] = v[j][e];
                }
            }
        }
    }
};

// A range of memory behind a buffer descriptor: reads behind its end give zeros,
// writes there are dropped, without a branch.  The range's start and size are one
// for all lanes, at most 2^31 bytes; an access is in it or behind it as a whole.
struct RowBuffer {
    __amdgpu_buffer_rsrc_t r;
    __device__ __forceinline__ RowBuffer(const void* p, uint32_t bytes)
        : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00027000)) {}
    __device__ __forceinline__ u32x4 read16(uint32_t at) const {
        return __builtin_amdgcn_raw_buffer_load_b128(r, (int)at, 0, 0);
    }
    __device__ __forceinline__ void write16(uint32_t at, u32x4 v) const {
        __builtin_amdgcn_raw_buffer_store_b128(v, r, (int)at, 0, 0);
    }
    template <typename T>
    __device__ __forceinline__ T read(uint32_t at) const {
        T v;
        if constexpr (sizeof(T) == 4) {
            const uint32_t w = __builtin_amdgcn_raw_buffer_load_b32(r, (int)at, 0, 0);
            __builtin_memcpy(&v, &w, 4);
        } else {
            const uint16_t w = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)at, 0, 0);
            __builtin_memcpy(&v, &w, 2);
        }
        return v;
    }
    template <typename T>
    __device__ __forceinline__ void write(uint32_t at, T v) const {
        if constexpr (sizeof(T) == 4) {
            uint32_t w;
            __builtin_memcpy(&w, &v, 4);
            __builtin_amdgcn_raw_buffer_store_b32(w, r, (int)at, 0, 0);
        } else {
            uint16_t w;
            __builtin_memcpy(&w, &v, 2);
            __builtin_amdgcn_raw_buffer_store_b16(w, r, (int)at, 0, 0);
        }
    }
};

}  // namespace fs
