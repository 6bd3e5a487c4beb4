// fs_layers_args.h -- argument blocks and launchers of the kernels behind
// include/fs_layers.h, shared by the host library and the kernel translation
// units.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fs_attn_args.h"

namespace fs {

constexpr int kNormMaxWidth = 16384;
constexpr int kQuantMaxWidth = 65536;  // 128 * 128 * 65536 fits 32 bits
constexpr int kDistillMaxTop = 1024;
constexpr int kDistillMaxSplit = 64;
constexpr int kBalanceMaxExperts = 1024;
constexpr int kBalanceMaxTop = 32;

// How a row's elements are read and written (Share in fs_rowops.hpp).
enum ShareForm : int { SINGLE, WIDE, DWORDS };

// Layer norm.  Where nothing tells the batch's entries apart they are one.
struct LayerNormArgs {
    int op, B, n, width;
    int form;  // ShareForm: how all of its rows may be read
    float eps;
    const int* lengths;
    AttnView x, r, z, y;     // forward: in, residual, their sum, out (r, z: p NULL for none)
    AttnView g, gz, gx;      // backward (x holds z): gradients of y and of z, of x
    const float* w;          // [width] or NULL
    const float* b;
    float* mean;             // [B][n] (forward: or NULL)
    float* rstd;
    float* gw;               // [width] or NULL
    float* gb;
    float* part;             // [blocks][2][width]
    int blocks;
};
hipError_t launch_layer_norm(const LayerNormArgs& a, hipStream_t s);
hipError_t launch_layer_norm_bwd(const LayerNormArgs& a, hipStream_t s);
int layer_norm_bwd_blocks(int64_t rows, int width);

struct QuantArgs {
    int op, rows, width, wide;
    const char* x;
    int64_t sx;
    int8_t* q;
    int64_t sq;
    float* scale;
};
hipError_t launch_quantize(const QuantArgs& a, hipStream_t s);

struct ProductArgs {
    int op, m, n, k;
    int dwords;  // both operands' rows start at whole dwords
    const int8_t* x;
    int64_t sx;
    const float* scale_x;
    const int8_t* w;
    int64_t sw;
    const float* scale_w;
    const float* bias;
    char* y;
    int64_t sy;
    int y_wide;          // rows of y 16-byte aligned, n whole groups of eight
    int split, split_k;  // ranges of k, each of split_k
    int* part;           // [split][m][n]
    // [rows][k rounded up to 16]: where an operand whose rows are not whole, aligned
    // 16-byte chunks is laid out first; NULL for one that is, and for few rows
    int8_t* pack_x;
    int8_t* pack_w;
};
hipError_t launch_product(const ProductArgs& a, hipStream_t s);
// Few rows: no ranges, nothing laid out.
bool product_few(int m);
// Ranges of k of a product of this size (1: no parts).
int product_split(int m, int n, int k, int* split_k);

struct DistillArgs {
    int op, rows, classes, k, wide;
    float T;
    const int* ids;
    const float* teacher;
    const float* teacher_lse;
    const uint8_t* active;
    const char* x;
    int64_t sx;
    char* gx;         // or NULL
    int64_t sgx;
    float* loss;      // NULL: backward alone
    float* lse;
    float* lse_rest;  // or NULL
    const float* gloss;
    int split, split_cols;  // ranges of a row's classes
    float2* part;           // [rows][split]: reference and sum
};
hipError_t launch_distill(const DistillArgs& a, hipStream_t s);
// Ranges of a row's classes that a call on `rows` rows works on apart.
int distill_split(int rows, int classes, bool backward, int* split_cols);

struct BalanceArgs {
    int op, B, n, E, k, normalize, wide;
    const int* lengths;
    AttnView x, gx;
    int* ids;
    float* gates;
    int* counts;
    float* loss;
    float* lse;
    const float* gloss;
    const float* ggates;
    int blocks;        // workgroups of a batch entry
    float2* part;      // [B][blocks][E + 1] sum of p, count (as bits); of lse^2, rows
    double* terms;     // [B][E / 8 + 1 + 2] the columns' terms of the loss; the last sums
    int* arrived;      // [B] workgroups whose term is there
};
hipError_t launch_balance(const BalanceArgs& a, hipStream_t s);
hipError_t launch_balance_bwd(const BalanceArgs& a, hipStream_t s);
int balance_blocks(int B, int n, int E);

}  // namespace fs
