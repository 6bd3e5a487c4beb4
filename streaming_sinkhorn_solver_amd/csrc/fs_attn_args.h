// fs_attn_args.h -- argument blocks and launchers of the attention kernels,
// shared by the host library and the kernel translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fs_device.hpp"

namespace fs {

constexpr int kAttnMaxEdges = 255;     // edges of one side (the block is a kernel argument)
constexpr int kAttnMaxEdge = 1024;     // the largest edge (a bias line stays within 8 KB of LDS)
constexpr int kAttnMaxOffset = 1 << 29;  // j - i - offset stays a 32-bit number
constexpr int kAttnMaxSplit = 64;
constexpr int kAttnRows = 128;         // query (or key) rows of a workgroup of four waves
constexpr int kAttnRowPad = 128;      // row terms are padded to whole query tiles
constexpr int kAttnFewRows = 32;       // packed rows of a workgroup of the few-row kernel

// Strides are in elements: batch, row, head.
struct AttnView {
    char* p;
    int64_t sb, sr, sh;
    int vec;  // rows 16-byte aligned, their width whole 16-byte chunks
};

struct AttnArgs {
    AttnView q, k, v, o;
    AttnView go, gq, gk, gv;  // backward: gradients of o, q, k, v
    float* lse;               // [B][H][n]
    const float* glse;        // gradient of lse or NULL
    int n_pad;                // n rounded up to kAttnRowPad
    float* nl2;               // backward workspace: [B][H][n_pad] -lse in base 2, and
    float* delta;             //   do.o - glse, refined by the pass over the keys
    int alone_q, alone_k;     // backward passes with 32 rows a workgroup (see BwdShape)
    int line_blocks;          // parts of a batch entry in line_part
    int op;                   // ScoreOp
    int B, n, m, H, K, G, d, dv;
    float scale, c;           // c = scale log2(e)
    int causal, offset;
    const int* q_len;
    const int* kv_len;
    const int* offsets;
    const uint8_t* key_mask;
    int64_t mask_stride;
    const float* bias;  // [buckets][H] or NULL
    int n_edges, two_sided, r0, rp;
    uint16_t edges[kAttnMaxEdges + 1];
    int n_split, split_keys;  // key ranges of the forward pass
    int dv_pad;               // dv rounded up to whole 16-byte chunks of fp32
    float* part_o;            // [n_split][B H n][dv_pad]
    float2* part_ml;          // [n_split][B H n]: reference and sum
    int q_split, split_rows;  // query ranges of the key gradients
    float* part_k;            // [q_split][B K m][d]
    float* part_v;            // [q_split][B K m][dv]
    float* line_part;         // bias gradient: [H][B line_blocks][r0 + rp + 1]
    float* gbias;             // [buckets][H]
};

// Grid of `blocks` workgroups over two dimensions: a launch may have fewer than
// 2^32 threads along each (flat_block gives the workgroup's number).
inline dim3 flat_grid(int64_t blocks) {
    constexpr int64_t kRow = 1 << 20;
    return blocks <= kRow ? dim3((unsigned)blocks)
                          : dim3((unsigned)kRow, (unsigned)((blocks + kRow - 1) / kRow));
}
__device__ __forceinline__ int64_t flat_block() {
    return (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
}

hipError_t launch_attn_fwd(const AttnArgs& a, hipStream_t s);
hipError_t launch_attn_rows(const AttnArgs& a, hipStream_t s);
hipError_t launch_attn_merge(const AttnArgs& a, hipStream_t s);
hipError_t launch_attn_delta(const AttnArgs& a, hipStream_t s);
hipError_t launch_attn_bwd_kv(const AttnArgs& a, hipStream_t s);
hipError_t launch_attn_bwd_q(const AttnArgs& a, hipStream_t s);
hipError_t launch_attn_kv_merge(const AttnArgs& a, hipStream_t s);
hipError_t launch_attn_bias_sum(const AttnArgs& a, hipStream_t s);

// One row set of the norm + rotation pass (queries, or keys).
struct NormRows {
    AttnView x, y;      // forward: in, out; backward: x in, y = gradient of x (out)
    AttnView g;         // backward: gradient of the output
    const float* w;     // [d] or NULL (ones)
    float* gw;          // backward: [d] or NULL
    int heads;
};
struct NormArgs {
    NormRows r[2];
    int op, B, n, d, rot, interleaved;
    float eps;
    const float* cos_t;
    const float* sin_t;  // [positions][rot / 2]
    int n_pos;
    int table_vec;         // tables 16-byte aligned, their rows whole 16-byte chunks
    const int* positions;  // [B][n] (row stride pos_stride) or NULL
    int64_t pos_stride;
    int offset;
    float* part;        // backward: [2][blocks][d] weight-gradient partials
    int blocks;
};
hipError_t launch_norm_rotate(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_rotate_bwd(const NormArgs& a, hipStream_t s);
int norm_bwd_blocks(int64_t rows);

}  // namespace fs
