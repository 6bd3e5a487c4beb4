// fs_attn_api.cpp -- host side of include/fs_attention.h: argument checks,
// workspace layout and the choice of kernel and split.  Nothing here
// allocates, synchronises or throws.
#include "fs_host.hpp"

using namespace fs;

namespace {

// ---- attention ------------------------------------------------------------

// Bytes of a tile's row in LDS.
int tile_row(const fs_attention_desc& d) {
    const int width = std::max(d.d, d.dv);
    return (width <= 64 ? 64 : width <= 128 ? 128 : 256) * elem_size(d.dtype);
}

// The few-row kernel packs the rows of a key head's queries into blocks of 32,
// its waves divide the keys; the other reads the keys once per head for 128
// rows, its waves divide the rows.  The first for single tokens, and for more
// rows if they are narrow and fill few workgroups of the other (measured, us,
// few-row against the other: 8 x 1024 rows of 64, 1024 keys, 11.6 / 16.8; 2 x 8
// x 500 fp32 rows of 48, 700 keys, 25.7 / 48.5; but 8 x 4 x 512 rows of 128,
// 2048 keys, 62.5 / 38.4 and 16 x 48 rows of 128, 8192 keys, 35.0 / 22.3).  The
// border, at 512 rows of 64 a head by the other's workgroups (few-row / other):
//   workgroups        32           64          128          256          512
//   bf16, 700 keys    16.5 / 17.8  11.5 / 19.4 20.3 / 22.8  37.8 / 18.8  73.5 / 25.2
//   bf16, 2048 keys   17.1 / 17.4  16.6 / 21.6 31.2 / 31.0  61.3 / 41.7   120 / 54.4
//   fp32 (48), 700    20.9 / 47.8  27.6 / 49.0 50.5 / 52.5   103 / 59.7   203 / 106
bool few_rows(const fs_attention_desc& d) {
    if (d.n <= kAttnFewRows) return true;
    return d.d <= 64 && d.dv <= 64 && (int64_t)d.batch * d.heads * cdiv(d.n, kAttnRows) <= 64;
}

int buckets_of(const fs_attention_desc& d) { return (d.n_edges + 1) * (d.two_sided ? 2 : 1); }

// Everything that does not need the tensors; fills a.
fs_status take_desc(const fs_attention_desc* p, AttnArgs& a) {
    if (!p) return fail(FS_ERR_INVALID_ARG, "desc must be non-NULL");
    const fs_attention_desc& d = *p;
    if (d.dtype < FS_DTYPE_F32 || d.dtype > FS_DTYPE_F16)
        return fail(FS_ERR_INVALID_ARG, "unknown fs_dtype %d", d.dtype);
    if (d.batch < 0 || d.n < 0 || d.m < 0 || d.n > (1 << 28) || d.m > (1 << 28))
        return fail(FS_ERR_INVALID_ARG, "batch, n and m must be >= 0 and n, m <= 2^28 (got %d, %d, %d)",
                    d.batch, d.n, d.m);
    if (d.heads < 1 || d.kv_heads < 1 || d.heads % d.kv_heads)
        return fail(FS_ERR_INVALID_ARG,
                    "heads must be a positive multiple of kv_heads (got %d, %d)", d.heads,
                    d.kv_heads);
    const int wmax = d.dtype == FS_DTYPE_F32 ? 128 : 256;
    if (d.d < 1 || d.d > wmax || d.dv < 1 || d.dv > wmax)
        return fail(FS_ERR_INVALID_ARG, "d and dv must be in [1, %d] for this type (got %d, %d)",
                    wmax, d.d, d.dv);
    constexpr float kLog2E = 1.4426950408889634f;  // scores are kept in base 2
    if (!(d.scale > 0.f) || !std::isfinite(d.scale * kLog2E))
        return fail(FS_ERR_INVALID_ARG, "scale must be positive and at most 2e38");
    if (d.offset < -kAttnMaxOffset || d.offset > kAttnMaxOffset)
        return fail(FS_ERR_INVALID_ARG, "offset must be within +-2^29 (got %d)", d.offset);
    if (d.key_mask && d.key_mask_stride < 0)
        return fail(FS_ERR_INVALID_ARG, "key_mask_stride must be >= 0");
    if (d.batch > 1 && d.key_mask && d.key_mask_stride > 0 && d.key_mask_stride < d.m)
        return fail(FS_ERR_INVALID_ARG, "key_mask_stride must be 0 or at least m");
    a.op = op_of(d.dtype);
    a.B = d.batch;
    a.n = d.n;
    a.m = d.m;
    a.H = d.heads;
    a.K = d.kv_heads;
    a.G = d.heads / d.kv_heads;
    a.d = d.d;
    a.dv = d.dv;
    a.n_pad = (int)(cdiv(d.n, kAttnRowPad) * kAttnRowPad);
    a.dv_pad = (d.dv + 3) / 4 * 4;
    a.scale = d.scale;
    a.c = d.scale * kLog2E;
    a.causal = d.causal != 0;
    a.offset = d.offset;
    a.q_len = d.q_len;
    a.kv_len = d.kv_len;
    a.offsets = d.offsets;
    a.key_mask = d.key_mask;
    a.mask_stride = d.key_mask_stride;
    a.bias = d.bias;
    if (d.bias) {
        if (d.n_edges < 0 || d.n_edges > kAttnMaxEdges || (d.n_edges > 0 && !d.edges))
            return fail(FS_ERR_INVALID_ARG, "n_edges must be in [0, %d] with edges given (got %d)",
                        kAttnMaxEdges, d.n_edges);
        int last = 1;
        for (int i = 0; i < d.n_edges; ++i) {
            if (d.edges[i] < last || d.edges[i] > kAttnMaxEdge)
                return fail(FS_ERR_INVALID_ARG, "edges must ascend within [1, %d] (edge %d is %d)",
                            kAttnMaxEdge, i, d.edges[i]);
            last = d.edges[i];
            a.edges[i] = (uint16_t)last;
        }
        a.n_edges = d.n_edges;
        a.two_sided = d.two_sided != 0;
        a.r0 = last;
        a.rp = a.two_sided ? last : 0;
    }
    // launch grids and row counts stay 32-bit numbers
    const int64_t rows = (int64_t)d.batch * d.heads * d.n;
    const int64_t krows = (int64_t)d.batch * d.kv_heads * d.m;
    if ((int64_t)d.batch * d.heads > (1 << 24) || d.heads > 65535 || rows > ((int64_t)1 << 31) ||
        krows > ((int64_t)1 << 31) || (int64_t)a.G * d.n > (1 << 30))
        return fail(FS_ERR_INVALID_ARG, "batch * heads * rows is beyond 2^31");

    // Key ranges.  Few rows: enough workgroups for the chip, at least one tile
    // for every wave, at most 32 tiles (ranges of unequal sequences then even
    // out).  Many rows: only where whole sequences leave CUs idle.
    const int row = tile_row(d);
    const bool few = few_rows(d);
    const int64_t items = few ? (int64_t)d.batch * d.kv_heads * cdiv((int64_t)a.G * d.n, 32)
                              : (int64_t)d.batch * d.heads * cdiv(d.n, kAttnRows);
    const int64_t turn = few ? (row <= 128 ? 8 : 4) * 32 : 256;  // keys of one turn of a workgroup
    a.n_split = 1;
    a.split_keys = d.m;
    if (items > 0 && d.m > 0) {
        int64_t s = cdiv(kCus, items);
        if (few) s = std::max(s, cdiv(d.m, 32 * turn));
        if (few && d.m <= 2 * turn) s = 1;  // the second launch costs more than two tiles
        s = std::max<int64_t>(1, std::min({s, (int64_t)kAttnMaxSplit, d.m / turn}));
        a.split_keys = (int)(cdiv(cdiv(d.m, s), turn) * turn);
        a.n_split = (int)cdiv(d.m, a.split_keys);
    }
    // Backward passes: 128 rows a workgroup where that fills the chip, else 32
    // (with the waves dividing the other side), and then the queries in ranges
    // if there are few keys.  The gradients of keys in rows of 256 bytes have one
    // buffer a wave and pay only where 128 rows leave most CUs idle (us, 32 /
    // 128 rows: 2 x 2 x 1024 keys of 128, 256 queries, 30.5 / 48.2, but 8 x 2048
    // keys, 128 queries, 29.3 / 16.6; 4 x 8 x 2048 keys, 512 queries, 151 / 64).
    // The borders (us, 32 / 128 rows, row terms included) by workgroups of 128 rows,
    // the queries' pass at 512 rows and 700 keys a head, the keys' at 512 rows:
    //   queries     64          128         256         512
    //   bf16, 64    16.1/24.1   17.8/24.5   30.4/26.4   55.6/39.7
    //   fp32, 48    34.0/79.1   53.5/81.8   99.3/85.3    188/151
    //   bf16, 128   21.0/28.4   28.0/29.0   48.6/34.5   86.2/54.7
    //   keys        48          96          128         192         256         384
    //   bf16, 64    17.0/27.4   17.4/30.9   17.6/36.2   25.7/22.2   29.3/23.6   41.1/29.5
    //   fp32, 48    31.8/52.5   58.1/56.3               86.9/79.8                169/153
    //   bf16, 128   23.8/43.3   41.7/45.9   42.6/51.8   61.3/32.7   79.4/35.3    118/59.5
    // (between 64 and 256 workgroups of keys the other form is up to a fifth
    // faster than the one taken.)
    const bool can = row <= 256;
    a.alone_q = can && (int64_t)d.batch * d.heads * cdiv(d.n, kAttnRows) < kCus;
    a.alone_k = can && (int64_t)d.batch * d.kv_heads * cdiv(d.m, kAttnRows) <
                           (row <= 128 || d.dtype == FS_DTYPE_F32 ? kCus : kCus / 4);
    const int64_t kblocks = cdiv(d.m, a.alone_k ? 32 : kAttnRows);
    const int64_t kitems = (int64_t)d.batch * d.kv_heads * kblocks;
    a.q_split = 1;
    a.split_rows = d.n;
    if (kitems > 0 && d.n > 0) {
        const int64_t want = kCus / kitems;
        const int64_t most = std::min<int64_t>(16, d.n / 256);
        const int64_t s = std::max<int64_t>(1, std::min(want, most));
        a.split_rows = (int)(cdiv(cdiv(d.n, s), 128) * 128);
        a.q_split = (int)cdiv(d.n, a.split_rows);
    }
    a.line_blocks = (int)(a.q_split * kblocks);
    // The traversals number their workgroups along one dimension, where a launch
    // has fewer than 2^32 threads (the largest takes one workgroup for every 32
    // rows of a key head at least, 128 of a head, or 32 keys).
    const int64_t fwd = items * a.n_split * (few && row <= 128 ? 512 : 256);
    const int64_t bwd_q = (int64_t)d.batch * d.heads * cdiv(d.n, a.alone_q ? 32 : kAttnRows) * 256;
    const int64_t bwd_k = kitems * a.q_split * 256;
    if (std::max({fwd, bwd_q, bwd_k}) >= (int64_t)1 << 32)
        return fail(FS_ERR_INVALID_ARG, "batch * heads is too large: a launch has fewer than 2^32 threads");
    return FS_OK;
}

struct FwdLayout {
    size_t ml = 0, o = 0, total = kAlign;
};
FwdLayout fwd_layout(const AttnArgs& a) {
    FwdLayout l;
    if (a.n_split > 1) {
        const size_t rows = (size_t)a.B * a.H * a.n;
        l.ml = 0;
        l.o = up((size_t)a.n_split * rows * sizeof(float2));
        l.total = l.o + up((size_t)a.n_split * rows * a.dv_pad * 4);
    }
    return l;
}

struct BwdLayout {
    size_t nl2 = 0, delta = 0, pk = 0, pv = 0, line = 0, total = kAlign;
};
BwdLayout bwd_layout(const AttnArgs& a) {
    BwdLayout l;
    const size_t terms = up((size_t)a.B * a.H * a.n_pad * 4);
    l.delta = terms;
    size_t at = 2 * terms;
    if (a.q_split > 1) {
        const size_t rows = (size_t)a.B * a.K * a.m;
        l.pk = at;
        at += up((size_t)a.q_split * rows * a.d * 4);
        l.pv = at;
        at += up((size_t)a.q_split * rows * a.dv * 4);
    }
    if (a.bias) {
        l.line = at;
        at += up((size_t)a.H * a.B * a.line_blocks * (a.r0 + a.rp + 1) * 4);
    }
    l.total = std::max(at, kAlign);
    return l;
}

// Device arrays of the description, as extents.
int desc_extents(const fs_attention_desc& d, Extent* e) {
    int n = 0;
    e[n++] = flat(d.q_len, 4 * (size_t)d.batch);
    e[n++] = flat(d.kv_len, 4 * (size_t)d.batch);
    e[n++] = flat(d.offsets, 4 * (size_t)d.batch);
    e[n++] = d.batch && d.m ? flat(d.key_mask, (size_t)(d.batch - 1) * d.key_mask_stride + d.m)
                            : Extent{};
    if (d.bias) e[n++] = flat(d.bias, 4 * (size_t)buckets_of(d) * d.heads);
    return n;
}

}  // namespace

extern "C" {

fs_status fs_bucket_edges(int32_t side_buckets, int32_t max_distance, int32_t* edges) {
    if (!edges) return fail(FS_ERR_INVALID_ARG, "edges must be non-NULL");
    if (side_buckets < 2 || side_buckets > 64 || max_distance <= side_buckets / 2 ||
        max_distance > kAttnMaxEdge)
        return fail(FS_ERR_INVALID_ARG,
                    "needs 2 <= side_buckets <= 64 and side_buckets / 2 < max_distance <= %d "
                    "(got %d, %d)",
                    kAttnMaxEdge, side_buckets, max_distance);
    const int first = side_buckets / 2, rest = side_buckets - first;
    // edge u > first: the smallest x with x^rest >= first^(rest - k) max^k,
    // k = u - first.  The numbers have at most 32 * 10 bits.
    struct Big {
        uint32_t w[12] = {1};
        void mul(uint32_t f) {
            uint64_t c = 0;
            for (uint32_t& x : w) {
                c += (uint64_t)x * f;
                x = (uint32_t)c;
                c >>= 32;
            }
        }
        bool below(const Big& o) const {
            for (int i = 11; i >= 0; --i)
                if (w[i] != o.w[i]) return w[i] < o.w[i];
            return false;
        }
    };
    for (int u = 1; u < side_buckets; ++u) {
        int x = u;
        if (u > first) {
            Big bound;
            for (int i = 0; i < rest; ++i)
                bound.mul((uint32_t)(i < u - first ? max_distance : first));
            for (x = first; x < max_distance; ++x) {
                Big p;
                for (int i = 0; i < rest; ++i) p.mul((uint32_t)x);
                if (!p.below(bound)) break;
            }
        }
        edges[u - 1] = x;
    }
    return FS_OK;
}

size_t fs_attention_workspace_bytes(const fs_attention_desc* desc, int32_t backward) {
    AttnArgs a{};
    if (take_desc(desc, a) != FS_OK) return 0;
    return backward ? bwd_layout(a).total : fwd_layout(a).total;
}

fs_status fs_attention_forward(const fs_attention_desc* desc, fs_rows q, fs_rows k, fs_rows v,
                               fs_rows o, float* lse, void* workspace, size_t workspace_bytes,
                               void* stream) {
    AttnArgs a{};
    FS_TRY(take_desc(desc, a));
    const int es = elem_size(desc->dtype);
    Extent in[10], out;
    FS_TRY(take_view("q", q, a.B, a.n, a.H, a.d, es, false, a.q, in[0]));
    FS_TRY(take_view("k", k, a.B, a.m, a.K, a.d, es, false, a.k, in[1]));
    FS_TRY(take_view("v", v, a.B, a.m, a.K, a.dv, es, false, a.v, in[2]));
    FS_TRY(take_view("o", o, a.B, a.n, a.H, a.dv, es, true, a.o, out));
    const FwdLayout l = fwd_layout(a);
    FS_TRY(check_workspace(workspace, workspace_bytes, l.total));
    in[3] = flat(workspace, l.total);
    const int n_in = 4 + desc_extents(*desc, in + 4);
    const Extent le = flat(lse, 4 * (size_t)a.B * a.H * a.n);
    FS_TRY(check_apart("o", out, in, n_in));
    FS_TRY(check_apart("lse", le, in, n_in));
    if (le.overlaps(out)) return fail(FS_ERR_INVALID_ARG, "lse overlaps o");
    FS_TRY(check_gpu());
    if (a.B == 0 || a.n == 0) return FS_OK;
    a.lse = lse;
    a.part_ml = (float2*)((char*)workspace + l.ml);
    a.part_o = (float*)((char*)workspace + l.o);
    const hipStream_t s = (hipStream_t)stream;
    hipError_t e = few_rows(*desc) ? launch_attn_rows(a, s) : launch_attn_fwd(a, s);
    if (e == hipSuccess && a.n_split > 1) e = launch_attn_merge(a, s);
    return hip_status(e, "fs_attention_forward");
}

fs_status fs_attention_backward(const fs_attention_desc* desc, fs_rows q, fs_rows k, fs_rows v,
                                fs_rows o, const float* lse, fs_rows d_o, const float* d_lse,
                                fs_rows d_q, fs_rows d_k, fs_rows d_v, float* d_bias,
                                void* workspace, size_t workspace_bytes, void* stream) {
    AttnArgs a{};
    FS_TRY(take_desc(desc, a));
    const int es = elem_size(desc->dtype);
    Extent in[16], out[4];
    FS_TRY(take_view("q", q, a.B, a.n, a.H, a.d, es, false, a.q, in[0]));
    FS_TRY(take_view("k", k, a.B, a.m, a.K, a.d, es, false, a.k, in[1]));
    FS_TRY(take_view("v", v, a.B, a.m, a.K, a.dv, es, false, a.v, in[2]));
    FS_TRY(take_view("o", o, a.B, a.n, a.H, a.dv, es, false, a.o, in[3]));
    FS_TRY(take_view("d_o", d_o, a.B, a.n, a.H, a.dv, es, false, a.go, in[4]));
    if (a.B && a.n && !lse) return fail(FS_ERR_INVALID_ARG, "lse must be non-NULL");
    if (d_bias && !a.bias) return fail(FS_ERR_INVALID_ARG, "d_bias needs a bias");
    int n_out = 0;
    const char* names[4] = {"d_q", "d_k", "d_v", "d_bias"};
    AttnView* views[3] = {&a.gq, &a.gk, &a.gv};
    const fs_rows* given[3] = {&d_q, &d_k, &d_v};
    for (int i = 0; i < 3; ++i, ++n_out) {
        *views[i] = AttnView{};
        if (!given[i]->data) continue;
        FS_TRY(take_view(names[i], *given[i], a.B, i ? a.m : a.n, i ? a.K : a.H, i == 2 ? a.dv : a.d,
                         es, true, *views[i], out[i]));
    }
    out[n_out++] = flat(d_bias, d_bias ? 4 * (size_t)buckets_of(*desc) * a.H : 0);
    const BwdLayout l = bwd_layout(a);
    FS_TRY(check_workspace(workspace, workspace_bytes, l.total));
    in[5] = flat(workspace, l.total);
    in[6] = flat(lse, 4 * (size_t)a.B * a.H * a.n);
    in[7] = flat(d_lse, 4 * (size_t)a.B * a.H * a.n);
    const int n_in = 8 + desc_extents(*desc, in + 8);
    for (int i = 0; i < n_out; ++i) FS_TRY(check_apart(names[i], out[i], in, n_in));
    for (int i = 0; i < 3; ++i)
        if (out[3].overlaps(out[i])) return fail(FS_ERR_INVALID_ARG, "d_bias overlaps %s", names[i]);
    for (int i = 0; i < 3; ++i)
        for (int x = 0; x < i; ++x)
            if (given[i]->data && given[i]->data == given[x]->data)
                return fail(FS_ERR_INVALID_ARG, "%s and %s are the same memory", names[x], names[i]);
    FS_TRY(check_gpu());
    a.lse = const_cast<float*>(lse);
    a.glse = d_lse;
    a.gbias = d_bias;
    a.nl2 = (float*)((char*)workspace + l.nl2);
    a.delta = (float*)((char*)workspace + l.delta);
    a.part_k = (float*)((char*)workspace + l.pk);
    a.part_v = (float*)((char*)workspace + l.pv);
    a.line_part = (float*)((char*)workspace + l.line);
    const hipStream_t s = (hipStream_t)stream;
    const char* where = "fs_attention_backward";
    const bool rows = a.B > 0 && a.n > 0, keys = a.B > 0 && a.m > 0;
    if (rows) FS_TRY(hip_status(launch_attn_delta(a, s), where));
    if (rows && (a.gq.p || a.gbias)) FS_TRY(hip_status(launch_attn_bwd_q(a, s), where));
    if (keys && (a.gk.p || a.gv.p || a.gbias)) {
        FS_TRY(hip_status(launch_attn_bwd_kv(a, s), where));
        if (a.q_split > 1) FS_TRY(hip_status(launch_attn_kv_merge(a, s), where));
    }
    if (a.gbias) FS_TRY(hip_status(launch_attn_bias_sum(a, s), where));
    return FS_OK;
}

}  // extern "C"

namespace {

// ---- norm + rotation ------------------------------------------------------

fs_status take_norm_desc(const fs_qk_norm_desc* p, NormArgs& a) {
    if (!p) return fail(FS_ERR_INVALID_ARG, "desc must be non-NULL");
    const fs_qk_norm_desc& d = *p;
    if (d.dtype < FS_DTYPE_F32 || d.dtype > FS_DTYPE_F16)
        return fail(FS_ERR_INVALID_ARG, "unknown fs_dtype %d", d.dtype);
    if (d.batch < 0 || d.n < 0 || d.heads_q < 0 || d.heads_k < 0)
        return fail(FS_ERR_INVALID_ARG, "batch, n, heads_q and heads_k must be >= 0");
    if (d.d < 2 || d.d > 256 || d.d % 2)
        return fail(FS_ERR_INVALID_ARG, "d must be even and in [2, 256] (got %d)", d.d);
    if (d.rot < 0 || d.rot > d.d || d.rot % 2)
        return fail(FS_ERR_INVALID_ARG, "rot must be even and in [0, d] (got %d)", d.rot);
    if (!(d.eps >= 0.f) || !std::isfinite(d.eps))
        return fail(FS_ERR_INVALID_ARG, "eps must be >= 0 and finite");
    if (d.rot > 0 && (!d.cos_table || !d.sin_table || d.n_pos < 1))
        return fail(FS_ERR_INVALID_ARG, "the rotation needs both tables and n_pos >= 1");
    if (d.positions && (d.positions_stride < 0 ||
                        (d.batch > 1 && d.positions_stride > 0 && d.positions_stride < d.n)))
        return fail(FS_ERR_INVALID_ARG, "positions_stride must be 0 or at least n");
    // an item is a token's heads, or part of them: their number and the tokens' in
    // 32 bits
    if ((int64_t)d.batch * d.n > 1 << 26 ||
        (int64_t)d.batch * d.n * ((int64_t)d.heads_q + d.heads_k) > ((int64_t)1 << 31))
        return fail(FS_ERR_INVALID_ARG, "batch * n is beyond 2^26, or with the heads beyond 2^31");
    a.op = op_of(d.dtype);
    a.B = d.batch;
    a.n = d.n;
    a.d = d.d;
    a.rot = d.rot;
    a.interleaved = d.interleaved != 0;
    a.eps = d.eps;
    a.cos_t = d.cos_table;
    a.sin_t = d.sin_table;
    a.n_pos = d.n_pos;
    a.table_vec = d.rot % 8 == 0 && (uintptr_t)d.cos_table % 16 == 0 && (uintptr_t)d.sin_table % 16 == 0;
    a.positions = d.positions;
    a.pos_stride = d.positions_stride;
    a.offset = d.offset;
    a.r[0].heads = d.heads_q;
    a.r[1].heads = d.heads_k;
    a.blocks = norm_bwd_blocks((int64_t)d.batch * d.n * (d.heads_q + d.heads_k));
    return FS_OK;
}

size_t norm_workspace(const NormArgs& a) { return up((size_t)2 * a.blocks * a.d * 4); }

int norm_extents(const fs_qk_norm_desc& d, const float* qw, const float* kw, Extent* e) {
    int n = 0;
    e[n++] = flat(qw, 4 * (size_t)d.d);
    e[n++] = flat(kw, 4 * (size_t)d.d);
    if (d.rot > 0) {
        e[n++] = flat(d.cos_table, (size_t)d.n_pos * (d.rot / 2) * 4);
        e[n++] = flat(d.sin_table, (size_t)d.n_pos * (d.rot / 2) * 4);
    }
    if (d.batch && d.n)
        e[n++] = flat(d.positions, 4 * ((size_t)(d.batch - 1) * d.positions_stride + d.n));
    return n;
}

}  // namespace

extern "C" {

size_t fs_qk_norm_workspace_bytes(const fs_qk_norm_desc* desc) {
    NormArgs a{};
    if (take_norm_desc(desc, a) != FS_OK) return 0;
    return std::max(norm_workspace(a), kAlign);
}

fs_status fs_qk_norm_rotate(const fs_qk_norm_desc* desc, fs_rows q, fs_rows k,
                            const float* q_weight, const float* k_weight, fs_rows q_out,
                            fs_rows k_out, void* stream) {
    NormArgs a{};
    FS_TRY(take_norm_desc(desc, a));
    const int es = elem_size(desc->dtype);
    Extent in[8], out[2];
    FS_TRY(take_view("q", q, a.B, a.n, a.r[0].heads, a.d, es, false, a.r[0].x, in[0]));
    FS_TRY(take_view("k", k, a.B, a.n, a.r[1].heads, a.d, es, false, a.r[1].x, in[1]));
    FS_TRY(take_view("q_out", q_out, a.B, a.n, a.r[0].heads, a.d, es, true, a.r[0].y, out[0]));
    FS_TRY(take_view("k_out", k_out, a.B, a.n, a.r[1].heads, a.d, es, true, a.r[1].y, out[1]));
    const int n_in = 2 + norm_extents(*desc, q_weight, k_weight, in + 2);
    FS_TRY(check_apart("q_out", out[0], in, n_in));
    FS_TRY(check_apart("k_out", out[1], in, n_in));
    if (out[0].hi && q_out.data == k_out.data && out[1].hi)
        return fail(FS_ERR_INVALID_ARG, "q_out and k_out are the same memory");
    FS_TRY(check_gpu());
    a.r[0].w = q_weight;
    a.r[1].w = k_weight;
    return hip_status(launch_norm_rotate(a, (hipStream_t)stream), "fs_qk_norm_rotate");
}

fs_status fs_qk_norm_rotate_backward(const fs_qk_norm_desc* desc, fs_rows q, fs_rows k,
                                     const float* q_weight, const float* k_weight,
                                     fs_rows d_q_out, fs_rows d_k_out, fs_rows d_q, fs_rows d_k,
                                     float* d_q_weight, float* d_k_weight, void* workspace,
                                     size_t workspace_bytes, void* stream) {
    NormArgs a{};
    FS_TRY(take_norm_desc(desc, a));
    const int es = elem_size(desc->dtype);
    Extent in[11], out[4];
    FS_TRY(take_view("q", q, a.B, a.n, a.r[0].heads, a.d, es, false, a.r[0].x, in[0]));
    FS_TRY(take_view("k", k, a.B, a.n, a.r[1].heads, a.d, es, false, a.r[1].x, in[1]));
    FS_TRY(take_view("d_q_out", d_q_out, a.B, a.n, a.r[0].heads, a.d, es, false, a.r[0].g, in[2]));
    FS_TRY(take_view("d_k_out", d_k_out, a.B, a.n, a.r[1].heads, a.d, es, false, a.r[1].g, in[3]));
    FS_TRY(take_view("d_q", d_q, a.B, a.n, a.r[0].heads, a.d, es, true, a.r[0].y, out[0]));
    FS_TRY(take_view("d_k", d_k, a.B, a.n, a.r[1].heads, a.d, es, true, a.r[1].y, out[1]));
    const size_t need = std::max(norm_workspace(a), kAlign);
    FS_TRY(check_workspace(workspace, workspace_bytes, need));
    in[4] = flat(workspace, need);
    const int n_in = 5 + norm_extents(*desc, q_weight, k_weight, in + 5);
    out[2] = flat(d_q_weight, 4 * (size_t)a.d);
    out[3] = flat(d_k_weight, 4 * (size_t)a.d);
    const char* names[4] = {"d_q", "d_k", "d_q_weight", "d_k_weight"};
    for (int i = 0; i < 4; ++i) FS_TRY(check_apart(names[i], out[i], in, n_in));
    if (out[2].overlaps(out[3]) || out[2].overlaps(out[0]) || out[2].overlaps(out[1]) ||
        out[3].overlaps(out[0]) || out[3].overlaps(out[1]))
        return fail(FS_ERR_INVALID_ARG, "a weight's gradient overlaps another output");
    if (out[0].hi && d_q.data == d_k.data && out[1].hi)
        return fail(FS_ERR_INVALID_ARG, "d_q and d_k are the same memory");
    FS_TRY(check_gpu());
    a.r[0].w = q_weight;
    a.r[1].w = k_weight;
    a.r[0].gw = d_q_weight;
    a.r[1].gw = d_k_weight;
    a.part = (float*)workspace;
    return hip_status(launch_norm_rotate_bwd(a, (hipStream_t)stream),
                      "fs_qk_norm_rotate_backward");
}

}  // extern "C"
