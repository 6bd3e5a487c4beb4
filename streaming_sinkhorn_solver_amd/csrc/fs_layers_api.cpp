// fs_layers_api.cpp -- host side of include/fs_layers.h: argument checks,
// workspace layout and the choice of splits.  Nothing here allocates,
// synchronises or throws.
#include "fs_layers.h"

#include <cstdlib>
#include <utility>

#include "fs_host.hpp"
#include "fs_layers_args.h"

using namespace fs;

namespace {

fs_status check_dtype(int32_t dtype) {
    if (dtype < FS_DTYPE_F32 || dtype > FS_DTYPE_F16)
        return fail(FS_ERR_INVALID_ARG, "unknown fs_dtype %d", dtype);
    return FS_OK;
}

bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

// An array of `count` elements of `size` bytes that the call needs.
fs_status take_flat(const char* name, const void* p, int64_t count, size_t size, Extent& e) {
    e = Extent{};
    if (count == 0) return FS_OK;
    if (!p) return fail(FS_ERR_INVALID_ARG, "%s must be non-NULL", name);
    if ((uintptr_t)p % size)
        return fail(FS_ERR_INVALID_ARG, "%s is not aligned to its element type", name);
    e = flat(p, (size_t)count * size);
    return FS_OK;
}

// Whether two views of b x r rows of w elements, neither of which overlaps itself, share
// one.  Of equal strides: whether their offset d comes nearer than w to a difference of
// two rows' places, i L + j S with |i| < the longer stride's rows and |j| < the shorter's;
// a block of the shorter's rows ends before the longer stride does, so that only the i
// next to -d / L can do it, and of those the j next to the rest.  Other strides: taken to.
bool views_meet(const AttnView& x, const AttnView& y, int64_t b, int64_t r, int64_t w, int es) {
    if (x.sb != y.sb || x.sr != y.sr) return true;
    int64_t L = x.sb, nl = b, S = x.sr, ns = r;
    if (L < S) std::swap(L, S), std::swap(nl, ns);
    const auto near = [](int64_t d, int64_t s, int64_t n) { return n > 1 ? -d / s : 0; };
    const int64_t d = (y.p - x.p) / es, i0 = near(d, L, nl);
    for (int64_t i = i0 - 1; i <= i0 + 1; ++i) {
        if (i <= -nl || i >= nl) continue;
        const int64_t rest = d + i * L, j0 = near(rest, S, ns);
        for (int64_t j = j0 - 1; j <= j0 + 1; ++j)
            if (j > -ns && j < ns && std::abs(rest + j * S) < w) return true;
    }
    return false;
}

// Outputs against the inputs and against one another.  Two views (of b x r rows of w
// elements) may be slices of one buffer side by side.
struct Outputs {
    Extent e[8];
    const char* name[8];
    const AttnView* view[8];
    int n = 0;
    int64_t b = 0, r = 0, w = 0;
    int es = 1;
    void add(const char* what, const Extent& x, const AttnView* v = nullptr) {
        if (x.hi > x.lo) e[n] = x, view[n] = v, name[n++] = what;
    }
    fs_status check(const Extent* in, int n_in) const {
        for (int i = 0; i < n; ++i) {
            FS_TRY(check_apart(name[i], e[i], in, n_in));
            for (int j = 0; j < i; ++j)
                if (e[i].overlaps(e[j]) &&
                    (!view[i] || !view[j] || views_meet(*view[i], *view[j], b, r, w, es)))
                    return fail(FS_ERR_INVALID_ARG, "%s overlaps %s", name[i], name[j]);
        }
        return FS_OK;
    }
};

// ---- layer norm -------------------------------------------------------------

fs_status take_norm(const fs_layer_norm_desc* p, LayerNormArgs& a) {
    if (!p) return fail(FS_ERR_INVALID_ARG, "desc must be non-NULL");
    const fs_layer_norm_desc& d = *p;
    FS_TRY(check_dtype(d.dtype));
    if (d.batch < 0 || d.n < 0 || (int64_t)d.batch * d.n > 0x7fffffff)
        return fail(FS_ERR_INVALID_ARG,
                    "batch and n must be >= 0 and their product below 2^31 (got %d, %d)", d.batch,
                    d.n);
    if (d.width < 1 || d.width > kNormMaxWidth)
        return fail(FS_ERR_INVALID_ARG, "width must be in [1, %d] (got %d)", kNormMaxWidth, d.width);
    if (!(d.eps >= 0.f) || !std::isfinite(d.eps))
        return fail(FS_ERR_INVALID_ARG, "eps must be >= 0 and finite");
    a.op = op_of(d.dtype);
    a.B = d.batch;
    a.n = d.n;
    a.width = d.width;
    a.eps = d.eps;
    a.lengths = d.lengths;
    a.blocks = layer_norm_bwd_blocks((int64_t)d.batch * d.n, d.width);
    return FS_OK;
}

size_t norm_workspace(const LayerNormArgs& a) {
    return std::max(kAlign, up((size_t)a.blocks * 2 * a.width * 4));
}

// The widest accesses that all views allow: 16 bytes of aligned rows of whole groups of
// eight, 16 bytes of rows that start at whole dwords (5331 rows of 777, fp32, against
// single elements: forward 9.5 / 10.0 us, backward 17.2 / 19.7), single elements.
int row_form(AttnView* const* views, int count, int width, int es, bool weights) {
    bool wide = weights && width % 8 == 0, dwords = width >= 8;
    for (int i = 0; i < count; ++i) {
        const AttnView& v = *views[i];
        if (!v.p) continue;
        wide &= v.vec != 0;
        dwords &= (((uintptr_t)v.p | (uintptr_t)(v.sb * es) | (uintptr_t)(v.sr * es)) & 3) == 0;
    }
    return wide ? WIDE : dwords ? DWORDS : SINGLE;
}

// Where no length tells the batch's entries apart and they follow one another
// like their rows, they are one.
void fold_batch(LayerNormArgs& a, AttnView* const* views, int count) {
    if (a.lengths || a.B <= 1) return;
    for (int i = 0; i < count; ++i)
        if (views[i]->p && a.n > 1 && views[i]->sb != a.n * views[i]->sr) return;
    for (int i = 0; i < count; ++i)
        if (a.n == 1) views[i]->sr = views[i]->sb;
    a.n *= a.B;
    a.B = 1;
}

}  // namespace

extern "C" {

size_t fs_layer_norm_workspace_bytes(const fs_layer_norm_desc* desc) {
    LayerNormArgs a{};
    if (take_norm(desc, a) != FS_OK) return 0;
    return norm_workspace(a);
}

fs_status fs_layer_norm(const fs_layer_norm_desc* desc, fs_rows x, fs_rows residual,
                        const float* weight, const float* bias, fs_rows total, fs_rows y,
                        float* mean, float* rstd, void* stream) {
    LayerNormArgs a{};
    FS_TRY(take_norm(desc, a));
    const int es = elem_size(desc->dtype);
    const int64_t rows = (int64_t)a.B * a.n;
    Extent in[5], out[4];
    if (rows > 0 && !residual.data != !total.data)
        return fail(FS_ERR_INVALID_ARG, "residual and total are given both or neither");
    FS_TRY(take_view("x", x, a.B, a.n, 1, a.width, es, false, a.x, in[0]));
    if (residual.data) {
        FS_TRY(take_view("residual", residual, a.B, a.n, 1, a.width, es, false, a.r, in[1]));
        FS_TRY(take_view("total", total, a.B, a.n, 1, a.width, es, true, a.z, out[1]));
    }
    FS_TRY(take_view("y", y, a.B, a.n, 1, a.width, es, true, a.y, out[0]));
    if (weight) FS_TRY(take_flat("weight", weight, a.width, 4, in[2]));
    if (bias) FS_TRY(take_flat("bias", bias, a.width, 4, in[3]));
    if (a.lengths) FS_TRY(take_flat("lengths", a.lengths, a.B, 4, in[4]));
    if (mean) FS_TRY(take_flat("mean", mean, rows, 4, out[2]));
    if (rstd) FS_TRY(take_flat("rstd", rstd, rows, 4, out[3]));
    Outputs o;
    o.b = a.B, o.r = a.n, o.w = a.width, o.es = es;
    o.add("y", out[0], &a.y);
    o.add("total", out[1], &a.z);
    o.add("mean", out[2]);
    o.add("rstd", out[3]);
    FS_TRY(o.check(in, 5));
    FS_TRY(check_gpu());
    if (rows == 0) return FS_OK;
    a.w = weight;
    a.b = bias;
    a.mean = mean;
    a.rstd = rstd;
    AttnView* const views[4] = {&a.x, &a.r, &a.z, &a.y};
    a.form = row_form(views, 4, a.width, es, aligned16(weight) && aligned16(bias));
    fold_batch(a, views, 4);
    return hip_status(launch_layer_norm(a, (hipStream_t)stream), "fs_layer_norm");
}

fs_status fs_layer_norm_backward(const fs_layer_norm_desc* desc, fs_rows z, const float* weight,
                                 const float* mean, const float* rstd, fs_rows d_y,
                                 fs_rows d_total, fs_rows d_x, float* d_weight, float* d_bias,
                                 void* workspace, size_t workspace_bytes, void* stream) {
    LayerNormArgs a{};
    FS_TRY(take_norm(desc, a));
    const int es = elem_size(desc->dtype);
    const int64_t rows = (int64_t)a.B * a.n;
    Extent in[8], out[3];
    FS_TRY(take_view("z", z, a.B, a.n, 1, a.width, es, false, a.x, in[0]));
    FS_TRY(take_view("d_y", d_y, a.B, a.n, 1, a.width, es, false, a.g, in[1]));
    if (d_total.data)
        FS_TRY(take_view("d_total", d_total, a.B, a.n, 1, a.width, es, false, a.gz, in[2]));
    FS_TRY(take_view("d_x", d_x, a.B, a.n, 1, a.width, es, true, a.gx, out[0]));
    FS_TRY(take_flat("mean", mean, rows, 4, in[3]));
    FS_TRY(take_flat("rstd", rstd, rows, 4, in[4]));
    if (weight) FS_TRY(take_flat("weight", weight, a.width, 4, in[5]));
    if (a.lengths) FS_TRY(take_flat("lengths", a.lengths, a.B, 4, in[6]));
    if (d_weight) FS_TRY(take_flat("d_weight", d_weight, a.width, 4, out[1]));
    if (d_bias) FS_TRY(take_flat("d_bias", d_bias, a.width, 4, out[2]));
    const size_t need = norm_workspace(a);
    FS_TRY(check_workspace(workspace, workspace_bytes, need));
    in[7] = flat(workspace, need);
    Outputs o;
    const char* names[3] = {"d_x", "d_weight", "d_bias"};
    for (int i = 0; i < 3; ++i) o.add(names[i], out[i]);
    FS_TRY(o.check(in, 8));
    FS_TRY(check_gpu());
    a.w = weight;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.gw = d_weight;
    a.gb = d_bias;
    a.part = d_weight || d_bias ? (float*)workspace : nullptr;
    AttnView* const views[4] = {&a.x, &a.g, &a.gz, &a.gx};
    a.form = row_form(views, 4, a.width, es, aligned16(weight));
    fold_batch(a, views, 4);
    return hip_status(launch_layer_norm_bwd(a, (hipStream_t)stream), "fs_layer_norm_backward");
}

}  // extern "C"

namespace {

// ---- rows in 8-bit integers ---------------------------------------------------

// A matrix of int8 (or other) rows as a view.
fs_status take_matrix(const char* name, const void* p, int64_t rows, int64_t stride, int64_t width,
                      int es, bool written, Extent& e) {
    AttnView v;
    return take_view(name, fs_rows{const_cast<void*>(p), 0, stride, 0}, 1, width ? rows : 0, 1,
                     width, es, written, v, e);
}

constexpr int kProductMaxRows = 1 << 24;

bool product_sizes(int32_t m, int32_t n, int32_t k) {
    return m >= 0 && n >= 0 && k >= 0 && m <= kProductMaxRows && n <= kProductMaxRows &&
           (int64_t)m * n <= (int64_t)1 << 36 && k <= kQuantMaxWidth;
}
// (offsets within a tile of 256 rows stay 32-bit numbers; an operand that is not there
// yet may come to stand anywhere)
bool ready_for_tiles(const int8_t* q, int64_t rows, int64_t stride, int32_t k) {
    return k % 16 == 0 && q && aligned16(q) && (rows <= 1 || (stride % 16 == 0 && stride <= 1 << 22));
}
struct ProductLayout {
    int split = 1, split_k = 1;
    bool pack_x = false, pack_w = false;
    size_t x = 0, w = 0, total = kAlign;
};
ProductLayout product_layout(const fs_quantized_product_desc& d) {
    ProductLayout l;
    if (d.m == 0 || d.n == 0) return l;
    l.split = product_split(d.m, d.n, d.k, &l.split_k);
    size_t at = l.split > 1 ? up((size_t)l.split * d.m * d.n * 4) : 0;
    if (!product_few(d.m) && d.k > 0) {
        const size_t row = (size_t)cdiv(d.k, 16) * 16;
        l.pack_x = !ready_for_tiles(d.q_x, d.m, d.q_x_stride, d.k);
        l.pack_w = !ready_for_tiles(d.q_w, d.n, d.q_w_stride, d.k);
        l.x = at;
        if (l.pack_x) at += up(row * d.m);
        l.w = at;
        if (l.pack_w) at += up(row * d.n);
    }
    l.total = std::max(at, kAlign);
    return l;
}

}  // namespace

extern "C" {

fs_status fs_quantize_rows(int32_t dtype, int32_t rows, int32_t width, const void* x,
                           int64_t x_stride, int8_t* q, int64_t q_stride, float* scale,
                           void* stream) {
    FS_TRY(check_dtype(dtype));
    if (rows < 0 || width < 1 || width > kQuantMaxWidth)
        return fail(FS_ERR_INVALID_ARG, "needs rows >= 0 and 1 <= width <= %d (got %d, %d)",
                    kQuantMaxWidth, rows, width);
    QuantArgs a{};
    Extent in, out[2];
    FS_TRY(take_matrix("x", x, rows, x_stride, width, elem_size(dtype), false, in));
    FS_TRY(take_matrix("q", q, rows, q_stride, width, 1, true, out[0]));
    FS_TRY(take_flat("scale", scale, rows, 4, out[1]));
    Outputs o;
    o.add("q", out[0]);
    o.add("scale", out[1]);
    FS_TRY(o.check(&in, 1));
    FS_TRY(check_gpu());
    if (rows == 0) return FS_OK;
    a.op = op_of(dtype);
    a.rows = rows;
    a.width = width;
    a.x = (const char*)x;
    a.sx = rows > 1 ? x_stride : 0;
    a.q = q;
    a.sq = rows > 1 ? q_stride : 0;
    a.scale = scale;
    a.wide = width % 8 == 0 && aligned16(x) && a.sx * elem_size(dtype) % 16 == 0 &&
             (uintptr_t)q % 8 == 0 && a.sq % 8 == 0;
    return hip_status(launch_quantize(a, (hipStream_t)stream), "fs_quantize_rows");
}

size_t fs_quantized_product_workspace_bytes(const fs_quantized_product_desc* desc) {
    if (!desc || !product_sizes(desc->m, desc->n, desc->k)) {
        (void)fail(FS_ERR_INVALID_ARG, "desc is NULL or m, n or k out of range");
        return 0;
    }
    return product_layout(*desc).total;
}

fs_status fs_quantized_product(const fs_quantized_product_desc* desc, void* workspace,
                               size_t workspace_bytes, void* stream) {
    if (!desc) return fail(FS_ERR_INVALID_ARG, "desc must be non-NULL");
    const fs_quantized_product_desc& d = *desc;
    FS_TRY(check_dtype(d.dtype));
    if (!product_sizes(d.m, d.n, d.k))
        return fail(FS_ERR_INVALID_ARG,
                    "needs 0 <= m, n <= 2^24, m n <= 2^36 and 0 <= k <= %d (got %d, %d, %d)",
                    kQuantMaxWidth, d.m, d.n, d.k);
    Extent in[6], out;
    const bool any = d.m > 0 && d.n > 0;
    const int m = any ? d.m : 0, n = any ? d.n : 0;
    FS_TRY(take_matrix("q_x", d.q_x, m, d.q_x_stride, d.k, 1, false, in[0]));
    FS_TRY(take_matrix("q_w", d.q_w, n, d.q_w_stride, d.k, 1, false, in[1]));
    FS_TRY(take_flat("scale_x", d.scale_x, m, 4, in[2]));
    FS_TRY(take_flat("scale_w", d.scale_w, n, 4, in[3]));
    if (d.bias) FS_TRY(take_flat("bias", d.bias, n, 4, in[4]));
    FS_TRY(take_matrix("y", d.y, m, d.y_stride, n, elem_size(d.dtype), true, out));
    ProductArgs a{};
    const ProductLayout l = product_layout(d);
    const size_t need = l.total;
    FS_TRY(check_workspace(workspace, workspace_bytes, need));
    in[5] = flat(workspace, need);
    FS_TRY(check_apart("y", out, in, 6));
    FS_TRY(check_gpu());
    if (!any) return FS_OK;
    a.op = op_of(d.dtype);
    a.m = m;
    a.n = n;
    a.k = d.k;
    a.x = d.q_x;
    a.sx = m > 1 ? d.q_x_stride : 0;
    a.scale_x = d.scale_x;
    a.w = d.q_w;
    a.sw = n > 1 ? d.q_w_stride : 0;
    a.scale_w = d.scale_w;
    a.bias = d.bias;
    a.y = (char*)d.y;
    a.sy = m > 1 ? d.y_stride : 0;
    a.y_wide = n % 8 == 0 && aligned16(d.y) && a.sy * elem_size(d.dtype) % 16 == 0;
    a.dwords = ((uintptr_t)d.q_x | (uintptr_t)d.q_w | (uintptr_t)a.sx | (uintptr_t)a.sw) % 4 == 0;
    a.split = l.split;
    a.split_k = l.split_k;
    a.part = (int*)workspace;
    a.pack_x = l.pack_x ? (int8_t*)workspace + l.x : nullptr;
    a.pack_w = l.pack_w ? (int8_t*)workspace + l.w : nullptr;
    return hip_status(launch_product(a, (hipStream_t)stream), "fs_quantized_product");
}

}  // extern "C"

namespace {

// ---- distillation --------------------------------------------------------------

fs_status take_distill(const fs_distill_desc* p, bool backward, DistillArgs& a) {
    if (!p) return fail(FS_ERR_INVALID_ARG, "desc must be non-NULL");
    const fs_distill_desc& d = *p;
    FS_TRY(check_dtype(d.dtype));
    if (d.rows < 0 || d.classes < 1 || d.classes > 1 << 24)
        return fail(FS_ERR_INVALID_ARG, "needs rows >= 0 and 1 <= classes <= 2^24 (got %d, %d)",
                    d.rows, d.classes);
    if (d.k < 1 || d.k > kDistillMaxTop)
        return fail(FS_ERR_INVALID_ARG, "k must be in [1, %d] (got %d)", kDistillMaxTop, d.k);
    if (!(d.temperature >= 0x1p-20f && d.temperature <= 0x1p20f))
        return fail(FS_ERR_INVALID_ARG, "temperature must be in [2^-20, 2^20]");
    // (logits of 16 have an lse of 2^14 there, of whose rounding 2^-10 of p is left)
    if (backward && d.temperature < 0x1p-10f && !d.lse_rest)
        return fail(FS_ERR_INVALID_ARG, "a temperature below 2^-10 needs lse_rest");
    a.op = op_of(d.dtype);
    a.rows = d.rows;
    a.classes = d.classes;
    a.k = d.k;
    a.T = d.temperature;
    a.ids = d.ids;
    a.teacher = d.teacher;
    a.teacher_lse = d.teacher_lse;
    a.active = d.active;
    a.lse_rest = d.lse_rest;
    a.split = distill_split(d.rows, d.classes, backward, &a.split_cols);
    return FS_OK;
}

size_t distill_workspace(const DistillArgs& a) {
    return a.split > 1 ? up((size_t)a.rows * a.split * sizeof(float2)) : kAlign;
}

// The logits, the teacher and the row mask; four extents.
fs_status distill_inputs(const fs_distill_desc& d, fs_rows logits, DistillArgs& a, bool& vec,
                         Extent* in) {
    AttnView v;
    FS_TRY(take_view("logits", logits, 1, a.rows, 1, a.classes, elem_size(d.dtype), false, v, in[0]));
    FS_TRY(take_flat("ids", d.ids, (int64_t)a.rows * a.k, 4, in[1]));
    FS_TRY(take_flat("teacher", d.teacher, (int64_t)a.rows * a.k, 4, in[2]));
    in[3] = in[4] = Extent{};
    if (d.teacher_lse) FS_TRY(take_flat("teacher_lse", d.teacher_lse, a.rows, 4, in[3]));
    if (d.active) FS_TRY(take_flat("active", d.active, a.rows, 1, in[4]));
    a.x = v.p;
    a.sx = v.sr;
    vec = v.vec;
    return FS_OK;
}

}  // namespace

extern "C" {

size_t fs_distill_workspace_bytes(const fs_distill_desc* desc) {
    DistillArgs a{};
    if (take_distill(desc, false, a) != FS_OK) return 0;
    return distill_workspace(a);
}

fs_status fs_distill_loss(const fs_distill_desc* desc, fs_rows logits, float* loss, float* lse,
                          const float* d_loss, fs_rows d_logits, void* workspace,
                          size_t workspace_bytes, void* stream) {
    DistillArgs a{};
    FS_TRY(take_distill(desc, false, a));
    Extent in[7], out[4];
    bool vec = false;
    FS_TRY(distill_inputs(*desc, logits, a, vec, in));
    FS_TRY(take_flat("loss", loss, a.rows, 4, out[0]));
    FS_TRY(take_flat("lse", lse, a.rows, 4, out[1]));
    if (a.lse_rest) FS_TRY(take_flat("lse_rest", a.lse_rest, a.rows, 4, out[3]));
    if (a.rows > 0 && !d_loss != !d_logits.data)
        return fail(FS_ERR_INVALID_ARG, "d_loss and d_logits are given both or neither");
    AttnView g{};
    if (d_logits.data) {
        FS_TRY(take_flat("d_loss", d_loss, a.rows, 4, in[5]));
        FS_TRY(take_view("d_logits", d_logits, 1, a.rows, 1, a.classes, elem_size(desc->dtype), true,
                         g, out[2]));
    }
    const size_t need = distill_workspace(a);
    FS_TRY(check_workspace(workspace, workspace_bytes, need));
    in[6] = flat(workspace, need);
    Outputs o;
    const char* names[4] = {"loss", "lse", "d_logits", "lse_rest"};
    for (int i = 0; i < 4; ++i) o.add(names[i], out[i]);
    FS_TRY(o.check(in, 7));
    FS_TRY(check_gpu());
    if (a.rows == 0) return FS_OK;
    a.gx = g.p;
    a.sgx = g.sr;
    a.wide = vec && (!g.p || g.vec) && a.classes % 8 == 0;
    a.loss = loss;
    a.lse = lse;
    a.gloss = d_loss;
    a.part = (float2*)workspace;
    return hip_status(launch_distill(a, (hipStream_t)stream), "fs_distill_loss");
}

fs_status fs_distill_loss_backward(const fs_distill_desc* desc, fs_rows logits, const float* lse,
                                   const float* d_loss, fs_rows d_logits, void* stream) {
    DistillArgs a{};
    FS_TRY(take_distill(desc, true, a));
    Extent in[8], out;
    bool vec = false;
    FS_TRY(distill_inputs(*desc, logits, a, vec, in));
    FS_TRY(take_flat("lse", lse, a.rows, 4, in[5]));
    FS_TRY(take_flat("d_loss", d_loss, a.rows, 4, in[6]));
    if (a.lse_rest) FS_TRY(take_flat("lse_rest", a.lse_rest, a.rows, 4, in[7]));
    AttnView g{};
    FS_TRY(take_view("d_logits", d_logits, 1, a.rows, 1, a.classes, elem_size(desc->dtype), true, g,
                     out));
    FS_TRY(check_apart("d_logits", out, in, 8));
    FS_TRY(check_gpu());
    if (a.rows == 0) return FS_OK;
    a.gx = g.p;
    a.sgx = g.sr;
    a.wide = vec && g.vec && a.classes % 8 == 0;
    a.lse = const_cast<float*>(lse);
    a.gloss = d_loss;
    return hip_status(launch_distill(a, (hipStream_t)stream), "fs_distill_loss_backward");
}

}  // extern "C"

namespace {

// ---- balanced use of the columns -----------------------------------------------

fs_status take_balance(const fs_balance_desc* p, BalanceArgs& a) {
    if (!p) return fail(FS_ERR_INVALID_ARG, "desc must be non-NULL");
    const fs_balance_desc& d = *p;
    FS_TRY(check_dtype(d.dtype));
    if (d.batch < 0 || d.n < 0 || d.batch > 65535 || (int64_t)d.batch * d.n > 0x7fffffff)
        return fail(FS_ERR_INVALID_ARG,
                    "needs 0 <= batch <= 65535, n >= 0 and batch * n below 2^31 (got %d, %d)",
                    d.batch, d.n);
    if (d.experts < 1 || d.experts > kBalanceMaxExperts)
        return fail(FS_ERR_INVALID_ARG, "experts must be in [1, %d] (got %d)", kBalanceMaxExperts,
                    d.experts);
    if (d.k < 1 || d.k > std::min(kBalanceMaxTop, d.experts))
        return fail(FS_ERR_INVALID_ARG, "k must be in [1, min(%d, experts)] (got %d)",
                    kBalanceMaxTop, d.k);
    if ((int64_t)d.n * d.k > 0x7fffffff)
        return fail(FS_ERR_INVALID_ARG, "n * k must be below 2^31 (got %d, %d)", d.n, d.k);
    a.op = op_of(d.dtype);
    a.B = d.batch;
    a.n = d.n;
    a.E = d.experts;
    a.k = d.k;
    a.normalize = d.normalize != 0;
    a.lengths = d.lengths;
    a.blocks = balance_blocks(d.batch, d.n, d.experts);
    return FS_OK;
}

struct BalanceLayout {
    size_t terms = 0, arrived = 0, total = kAlign;
};
BalanceLayout balance_layout(const BalanceArgs& a) {
    BalanceLayout l;
    if (a.blocks > 1) {
        l.terms = up((size_t)a.B * a.blocks * (a.E + 1) * sizeof(float2));
        l.arrived = l.terms + up((size_t)a.B * (a.E / 8 + 3) * sizeof(double));
        l.total = l.arrived + up((size_t)a.B * sizeof(int));
    }
    return l;
}

}  // namespace

extern "C" {

size_t fs_balance_workspace_bytes(const fs_balance_desc* desc) {
    BalanceArgs a{};
    if (take_balance(desc, a) != FS_OK) return 0;
    return balance_layout(a).total;
}

fs_status fs_balance_loss(const fs_balance_desc* desc, fs_rows logits, int32_t* ids, float* gates,
                          int32_t* counts, float* loss, float* lse, void* workspace,
                          size_t workspace_bytes, void* stream) {
    BalanceArgs a{};
    FS_TRY(take_balance(desc, a));
    const int64_t rows = (int64_t)a.B * a.n;
    Extent in[3], out[5];
    FS_TRY(take_view("logits", logits, a.B, a.n, 1, a.E, elem_size(desc->dtype), false, a.x, in[0]));
    if (a.lengths) FS_TRY(take_flat("lengths", a.lengths, a.B, 4, in[1]));
    FS_TRY(take_flat("ids", ids, rows * a.k, 4, out[0]));
    FS_TRY(take_flat("gates", gates, rows * a.k, 4, out[1]));
    FS_TRY(take_flat("counts", counts, (int64_t)a.B * a.E, 4, out[2]));
    FS_TRY(take_flat("loss", loss, 2 * (int64_t)a.B, 4, out[3]));
    FS_TRY(take_flat("lse", lse, rows, 4, out[4]));
    const BalanceLayout l = balance_layout(a);
    FS_TRY(check_workspace(workspace, workspace_bytes, l.total));
    in[2] = flat(workspace, l.total);
    Outputs o;
    const char* names[5] = {"ids", "gates", "counts", "loss", "lse"};
    for (int i = 0; i < 5; ++i) o.add(names[i], out[i]);
    FS_TRY(o.check(in, 3));
    FS_TRY(check_gpu());
    if (a.B == 0) return FS_OK;
    a.wide = a.x.vec && a.E % 8 == 0;
    a.ids = ids;
    a.gates = gates;
    a.counts = counts;
    a.loss = loss;
    a.lse = lse;
    a.part = (float2*)workspace;
    a.terms = (double*)((char*)workspace + l.terms);
    a.arrived = (int*)((char*)workspace + l.arrived);
    return hip_status(launch_balance(a, (hipStream_t)stream), "fs_balance_loss");
}

fs_status fs_balance_loss_backward(const fs_balance_desc* desc, fs_rows logits, const int32_t* ids,
                                   const int32_t* counts, const float* lse, const float* d_loss,
                                   const float* d_gates, fs_rows d_logits, void* stream) {
    BalanceArgs a{};
    FS_TRY(take_balance(desc, a));
    const int64_t rows = (int64_t)a.B * a.n;
    Extent in[7], out;
    FS_TRY(take_view("logits", logits, a.B, a.n, 1, a.E, elem_size(desc->dtype), false, a.x, in[0]));
    if (a.lengths) FS_TRY(take_flat("lengths", a.lengths, a.B, 4, in[1]));
    FS_TRY(take_flat("ids", ids, rows * a.k, 4, in[2]));
    FS_TRY(take_flat("counts", counts, (int64_t)a.B * a.E, 4, in[3]));
    FS_TRY(take_flat("lse", lse, rows, 4, in[4]));
    FS_TRY(take_flat("d_loss", d_loss, 2 * (int64_t)a.B, 4, in[5]));
    if (d_gates) FS_TRY(take_flat("d_gates", d_gates, rows * a.k, 4, in[6]));
    FS_TRY(take_view("d_logits", d_logits, a.B, a.n, 1, a.E, elem_size(desc->dtype), true, a.gx, out));
    FS_TRY(check_apart("d_logits", out, in, 7));
    FS_TRY(check_gpu());
    if (rows == 0) return FS_OK;
    a.wide = a.x.vec && a.gx.vec && a.E % 8 == 0;
    a.ids = const_cast<int32_t*>(ids);
    a.counts = const_cast<int32_t*>(counts);
    a.lse = const_cast<float*>(lse);
    a.gloss = d_loss;
    a.ggates = d_gates;
    return hip_status(launch_balance_bwd(a, (hipStream_t)stream), "fs_balance_loss_backward");
}

}  // extern "C"
