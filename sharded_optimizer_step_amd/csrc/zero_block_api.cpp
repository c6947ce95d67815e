// zero_block_api.cpp -- the C ABI of the calls around a training block: 8-bit
// activation checkpoints, the weight gradient taken from one, the norms with
// gate and residual scale, the layer norm and the gated feed-forward block.
// Argument checks and launches; the kernels are in zero_act8.hip,
// zero_wgrad.hip, zero_block_norm.hip, zero_layer_norm.hip, zero_ffn.hip and
// zero_ffn_act.hip.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "zero_block.h"
#include "zero_internal.h"
#include "zero_step.h"

using namespace zero;

namespace {

constexpr int64_t kMaxSize = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxCols = int64_t{1} << 30;
constexpr size_t kPtrAlign = 16;  // of act8 buffers and workspaces

int hip_status(hipError_t e) { return e == hipSuccess ? ZERO_OK : ZERO_ERR_HIP; }

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool format_ok(int32_t f) { return f == ZERO_ACT8_E4M3 || f == ZERO_ACT8_INT8; }

bool buffer_ok(const void* p) { return p != nullptr && aligned(p, kPtrAlign); }

bool given(const zero_rows& r) { return r.data != nullptr; }

// A given row-major operand of `cols` columns; type 0: either.
bool rows_ok(const zero_rows& r, int64_t cols, int32_t type, bool vector = false)
{
    if (r.data == nullptr || r.reserved != 0) return false;
    if (r.dtype != ZERO_BF16 && r.dtype != ZERO_F32) return false;
    if (type != 0 && r.dtype != type) return false;
    if (!aligned(r.data, r.dtype == ZERO_F32 ? 4 : 2)) return false;
    return vector || r.ld >= cols;
}

bool optional_ok(const zero_rows& r, int64_t cols, int32_t type, bool vector = false)
{
    return !given(r) || rows_ok(r, cols, type, vector);
}

// Two outputs of one call at the same address.
bool same(const void* a, const void* b) { return a != nullptr && a == b; }

Rows view(const zero_rows& r) { return Rows{r.data, r.ld, r.dtype == ZERO_F32}; }

// The vectors of 8 columns that a launch over rows x cols visits have to fit a grid.
bool list_ok(int64_t rows, int64_t cols)
{
    return rows >= 0 && rows <= kMaxSize && cols >= 0 && cols <= kMaxCols &&
           static_cast<double>(rows) * static_cast<double>(act8_pitch(cols)) < 0x1p36;
}

bool product_ok(int64_t rows, int64_t outs, int64_t cols)
{
    return rows >= 0 && rows <= kMaxSize && outs >= 0 && outs <= kMaxSize && cols >= 0 && cols <= kMaxCols &&
           // a workgroup of 256 threads for every 64 x 64 of dw, at the most: a grid counts fewer than 2^32 threads
           ((outs + 127) / 128) * ((cols + 127) / 128) < (int64_t{1} << 20);
}

bool norm_sizes_ok(int64_t rows, int64_t cols)
{
    return rows >= 0 && rows <= kMaxSize && cols >= 0 && cols <= ZERO_BLOCK_NORM_MAX_COLS;
}

bool activation_ok(int32_t act) { return act == ZERO_FFN_SILU || act == ZERO_FFN_GELU || act == ZERO_FFN_GELU_TANH; }

bool ffn_sizes_ok(int64_t rows, int64_t cols, int64_t hidden)
{
    return product_ok(cols, rows, hidden) && product_ok(hidden, rows, cols) && product_ok(rows, hidden, cols) &&
           hidden <= kMaxCols && list_ok(rows, hidden) && list_ok(rows, cols);
}

// Whether two of n outputs lie at one address.
template <class... P>
bool any_same(P... p)
{
    const void* v[] = {p...};
    const int n = static_cast<int>(sizeof...(p));
    for (int i = 0; i < n; ++i)
        for (int j = i + 1; j < n; ++j)
            if (same(v[i], v[j])) return true;
    return false;
}

// The largest of the workspaces of a feed-forward block's products, which run one after the other.
size_t ffn_grad_bytes(int64_t rows, int64_t cols, int64_t hidden)
{
    const size_t input = ffn_workspace_bytes(kFfnInput, rows, cols, hidden), weight = ffn_workspace_bytes(kFfnWeight, rows, cols, hidden);
    const size_t coded = wgrad_plan(rows, hidden, cols).bytes;
    const size_t most = input > weight ? input : weight;
    return most > coded ? most : coded;
}

}  // namespace

extern "C" {

size_t zero_act8_bytes(int64_t rows, int64_t cols)
{
    if (!list_ok(rows, cols)) return 0;
    const int64_t pitch = act8_pitch(cols);
    return static_cast<size_t>(rows * pitch + rows * (pitch / kActBlock));
}

int zero_act8_save(const zero_rows* x, int64_t rows, int64_t cols, int32_t format, void* ckpt, hipStream_t stream)
{
    if (!list_ok(rows, cols) || !format_ok(format) || x == nullptr) return ZERO_ERR_INVALID_ARGUMENT;
    if (rows == 0 || cols == 0) return ZERO_OK;
    if (!rows_ok(*x, cols, 0) || !buffer_ok(ckpt)) return ZERO_ERR_INVALID_ARGUMENT;
    return hip_status(launch_act8_save(view(*x), rows, cols, format, static_cast<uint8_t*>(ckpt), stream));
}

int zero_act8_load(const void* ckpt, int64_t rows, int64_t cols, int32_t format, const zero_rows* out, hipStream_t stream)
{
    if (!list_ok(rows, cols) || !format_ok(format) || out == nullptr) return ZERO_ERR_INVALID_ARGUMENT;
    if (rows == 0 || cols == 0) return ZERO_OK;
    if (!rows_ok(*out, cols, 0) || !buffer_ok(ckpt)) return ZERO_ERR_INVALID_ARGUMENT;
    return hip_status(launch_act8_load(static_cast<const uint8_t*>(ckpt), rows, cols, format, view(*out), stream));
}

size_t zero_act8_wgrad_workspace_bytes(int64_t rows, int64_t outs, int64_t cols)
{
    return product_ok(rows, outs, cols) ? wgrad_plan(rows, outs, cols).bytes : 0;
}

int zero_act8_wgrad(const zero_rows* dy, const void* ckpt, int64_t rows, int64_t outs, int64_t cols, int32_t format,
                    const zero_rows* col_scale, const zero_rows* dw, int32_t flags, void* ws, size_t ws_bytes,
                    hipStream_t stream)
{
    if (!product_ok(rows, outs, cols) || !format_ok(format) || dy == nullptr || dw == nullptr)
        return ZERO_ERR_INVALID_ARGUMENT;
    if ((flags & ~ZERO_GRAD_ACCUMULATE) != 0) return ZERO_ERR_INVALID_ARGUMENT;
    const bool accumulate = (flags & ZERO_GRAD_ACCUMULATE) != 0;
    if (outs == 0 || cols == 0 || (rows == 0 && accumulate)) return ZERO_OK;
    if (!rows_ok(*dw, cols, accumulate ? ZERO_F32 : 0)) return ZERO_ERR_INVALID_ARGUMENT;
    if (rows > 0 && (!rows_ok(*dy, outs, ZERO_BF16) || !buffer_ok(ckpt))) return ZERO_ERR_INVALID_ARGUMENT;
    WgradArgs a{};
    if (col_scale != nullptr) {
        if (!rows_ok(*col_scale, cols, 0, true)) return ZERO_ERR_INVALID_ARGUMENT;
        if (rows > 0) a.col_scale = view(*col_scale);  // an empty sum is 0 whatever its scale
    }
    const WgradPlan plan = wgrad_plan(rows, outs, cols);
    if (plan.bytes > 0) {
        if (!buffer_ok(ws)) return ZERO_ERR_INVALID_ARGUMENT;
        if (ws_bytes < plan.bytes) return ZERO_ERR_WORKSPACE_TOO_SMALL;
        forget_plans(ws, plan.bytes);
    }
    a.dy = static_cast<const uint16_t*>(dy->data);
    a.ld_dy = dy->ld;
    a.pitch = act8_pitch(cols);
    a.codes = static_cast<const uint8_t*>(ckpt);
    a.scales = a.codes + rows * a.pitch;
    a.rows = rows;
    a.outs = outs;
    a.cols = cols;
    a.dw = view(*dw);
    a.accumulate = accumulate;
    a.part = static_cast<float*>(ws);
    return hip_status(launch_wgrad(a, plan, format, stream));
}

int zero_block_norm(const zero_block_norm_args* g, hipStream_t stream)
{
    if (g == nullptr || g->reserved != 0 || !norm_sizes_ok(g->rows, g->cols)) return ZERO_ERR_INVALID_ARGUMENT;
    const float alpha = static_cast<float>(g->residual_scale), eps = static_cast<float>(g->eps);
    if (!std::isfinite(alpha) || !std::isfinite(eps) || !(g->eps >= 0.0)) return ZERO_ERR_INVALID_ARGUMENT;
    const bool saves = g->ckpt_post != nullptr || g->ckpt_pre != nullptr;
    if (saves && !format_ok(g->format)) return ZERO_ERR_INVALID_ARGUMENT;
    if (g->rows == 0 || g->cols == 0) return ZERO_OK;
    if (!rows_ok(g->x, g->cols, 0)) return ZERO_ERR_INVALID_ARGUMENT;
    if (given(g->y)) {
        if (!rows_ok(g->y, g->cols, ZERO_BF16) || !rows_ok(g->x_out, g->cols, g->x.dtype)) return ZERO_ERR_INVALID_ARGUMENT;
        if (!optional_ok(g->w_post, g->cols, 0, true)) return ZERO_ERR_INVALID_ARGUMENT;
        if (given(g->gate) && (g->gate_rows < 1 || !rows_ok(g->gate, g->cols, 0))) return ZERO_ERR_INVALID_ARGUMENT;
    } else if (given(g->w_post) || given(g->gate) || given(g->x_out) || g->ckpt_post != nullptr) {
        return ZERO_ERR_INVALID_ARGUMENT;
    }
    if (g->rstd_post != nullptr && !given(g->w_post)) return ZERO_ERR_INVALID_ARGUMENT;
    if (given(g->w_pre)) {
        if (!rows_ok(g->w_pre, g->cols, 0, true) || !rows_ok(g->h, g->cols, ZERO_BF16)) return ZERO_ERR_INVALID_ARGUMENT;
    } else if (given(g->h) || g->rstd_pre != nullptr || g->ckpt_pre != nullptr) {
        return ZERO_ERR_INVALID_ARGUMENT;
    }
    if (!given(g->y) && !given(g->w_pre)) return ZERO_ERR_INVALID_ARGUMENT;  // nothing to compute
    if ((g->ckpt_post != nullptr && !aligned(g->ckpt_post, kPtrAlign)) ||
        (g->ckpt_pre != nullptr && !aligned(g->ckpt_pre, kPtrAlign)) ||
        !aligned(g->rstd_post, 4) || !aligned(g->rstd_pre, 4))
        return ZERO_ERR_INVALID_ARGUMENT;
    if (same(g->x_out.data, g->h.data) || same(g->rstd_post, g->rstd_pre) || same(g->ckpt_post, g->ckpt_pre))
        return ZERO_ERR_INVALID_ARGUMENT;
    NormArgs a{};
    a.rows = g->rows;
    a.cols = static_cast<int32_t>(g->cols);
    a.alpha = alpha;
    a.eps = eps;
    a.x = view(g->x);
    a.y = view(g->y);
    a.w_post = view(g->w_post);
    a.gate = view(g->gate);
    a.w_pre = view(g->w_pre);
    a.x_out = view(g->x_out);
    a.h = view(g->h);
    if (given(g->gate)) a.gate_div = fast_div(static_cast<uint32_t>(g->gate_rows < g->rows ? g->gate_rows : g->rows));
    a.rstd_post = g->rstd_post;
    a.rstd_pre = g->rstd_pre;
    a.ckpt_post = static_cast<uint8_t*>(g->ckpt_post);
    a.ckpt_pre = static_cast<uint8_t*>(g->ckpt_pre);
    a.format = g->format;
    return hip_status(launch_block_norm(a, stream));
}

size_t zero_block_norm_grad_workspace_bytes(int64_t rows, int64_t cols, int64_t gate_rows)
{
    if (!norm_sizes_ok(rows, cols) || gate_rows < 0) return 0;
    return norm_grad_plan(rows, cols, gate_rows).bytes;
}

int zero_block_norm_grad(const zero_block_norm_grad_args* g, void* ws, size_t ws_bytes, hipStream_t stream)
{
    if (g == nullptr || !norm_sizes_ok(g->rows, g->cols)) return ZERO_ERR_INVALID_ARGUMENT;
    const float alpha = static_cast<float>(g->residual_scale);
    if (!std::isfinite(alpha) || (g->flags & ~ZERO_GRAD_ACCUMULATE) != 0) return ZERO_ERR_INVALID_ARGUMENT;
    const bool accumulate = (g->flags & ZERO_GRAD_ACCUMULATE) != 0;
    if ((g->ckpt_pre != nullptr || g->ckpt_post != nullptr) && !format_ok(g->format)) return ZERO_ERR_INVALID_ARGUMENT;
    if (given(g->gate) && g->gate_rows < 1) return ZERO_ERR_INVALID_ARGUMENT;
    if (g->cols == 0) return ZERO_OK;
    if (!optional_ok(g->w_post, g->cols, 0, true) || !optional_ok(g->gate, g->cols, 0) ||
        (given(g->dw_post) && !given(g->w_post)) || (given(g->dgate) && !given(g->gate)))
        return ZERO_ERR_INVALID_ARGUMENT;
    const int32_t grad_type = accumulate ? ZERO_F32 : 0;
    if (!optional_ok(g->dw_pre, g->cols, grad_type, true) || !optional_ok(g->dw_post, g->cols, grad_type, true) ||
        !optional_ok(g->dgate, g->cols, grad_type))
        return ZERO_ERR_INVALID_ARGUMENT;
    if (same(g->dw_pre.data, g->dw_post.data) || same(g->dw_pre.data, g->dgate.data) ||
        same(g->dw_post.data, g->dgate.data) || same(g->dx.data, g->dy.data))
        return ZERO_ERR_INVALID_ARGUMENT;
    if (g->rows > 0) {
        if (!rows_ok(g->dx, g->cols, 0) || !optional_ok(g->dx_out, g->cols, g->dx.dtype)) return ZERO_ERR_INVALID_ARGUMENT;
        if (given(g->dh)) {
            if (!rows_ok(g->dh, g->cols, ZERO_BF16) || !rows_ok(g->w_pre, g->cols, 0, true)) return ZERO_ERR_INVALID_ARGUMENT;
            if (g->rstd_pre == nullptr || !aligned(g->rstd_pre, 4)) return ZERO_ERR_INVALID_ARGUMENT;
            if (g->ckpt_pre != nullptr ? !aligned(g->ckpt_pre, kPtrAlign) : !rows_ok(g->x_out, g->cols, g->dx.dtype))
                return ZERO_ERR_INVALID_ARGUMENT;
        } else if (given(g->w_pre) || given(g->dw_pre) || !given(g->dx_out)) {
            return ZERO_ERR_INVALID_ARGUMENT;
        }
        const bool from_y = given(g->dy) || given(g->dw_post) || given(g->dgate);
        if (!optional_ok(g->dy, g->cols, ZERO_BF16)) return ZERO_ERR_INVALID_ARGUMENT;
        if (given(g->w_post) && (g->rstd_post == nullptr || !aligned(g->rstd_post, 4))) return ZERO_ERR_INVALID_ARGUMENT;
        if (from_y && (given(g->w_post) || given(g->dgate))) {
            if (g->ckpt_post != nullptr ? !aligned(g->ckpt_post, kPtrAlign) : !rows_ok(g->y, g->cols, ZERO_BF16))
                return ZERO_ERR_INVALID_ARGUMENT;
        }
    }
    NormGradArgs a{};
    a.rows = g->rows;
    a.cols = static_cast<int32_t>(g->cols);
    a.alpha = alpha;
    a.plan = norm_grad_plan(g->rows, g->cols, given(g->gate) ? g->gate_rows : 0);
    if (a.plan.bytes > 0) {
        if (!buffer_ok(ws)) return ZERO_ERR_INVALID_ARGUMENT;
        if (ws_bytes < a.plan.bytes) return ZERO_ERR_WORKSPACE_TOO_SMALL;
        forget_plans(ws, a.plan.bytes);
    }
    a.dh = view(g->dh);
    a.dx_out = view(g->dx_out);
    a.w_post = view(g->w_post);
    a.gate = view(g->gate);
    a.w_pre = view(g->w_pre);
    if (g->ckpt_pre == nullptr && given(g->dh)) a.x_out = view(g->x_out);
    if (g->ckpt_post == nullptr) a.y = view(g->y);
    a.dx = view(g->dx);
    a.dy = view(g->dy);
    a.dw_pre = view(g->dw_pre);
    a.dw_post = view(g->dw_post);
    a.dgate = view(g->dgate);
    a.ckpt_pre = static_cast<const uint8_t*>(g->ckpt_pre);
    a.ckpt_post = static_cast<const uint8_t*>(g->ckpt_post);
    a.rstd_pre = g->rstd_pre;
    a.rstd_post = g->rstd_post;
    a.format = g->format;
    a.accumulate = accumulate;
    a.gate_div = fast_div(static_cast<uint32_t>(a.plan.gate_rows));
    // Only the sums that this call makes, one after the other from the start of
    // ws: what it overwrites of a step's plan there then always includes the
    // plan's signature, by which a step captured earlier knows that its table is gone.
    const int64_t sums = a.plan.units * a.cols;
    a.sum_pre = static_cast<float*>(ws);
    a.sum_post = a.sum_pre + (given(g->dw_pre) ? sums : 0);
    a.row_sums = a.sum_post + (given(g->dw_post) || (given(g->dgate) && a.plan.per_gate > 0) ? sums : 0);
    return hip_status(launch_block_norm_grad(a, stream));
}

int zero_layer_norm(const zero_layer_norm_args* g, hipStream_t stream)
{
    if (g == nullptr || g->reserved != 0 || !norm_sizes_ok(g->rows, g->cols)) return ZERO_ERR_INVALID_ARGUMENT;
    const float eps = static_cast<float>(g->eps);
    if (!std::isfinite(eps) || !(g->eps >= 0.0)) return ZERO_ERR_INVALID_ARGUMENT;
    if ((g->ckpt_xn != nullptr || g->ckpt_h != nullptr) && !format_ok(g->format)) return ZERO_ERR_INVALID_ARGUMENT;
    if (g->rows == 0 || g->cols == 0) return ZERO_OK;
    if (!rows_ok(g->x, g->cols, 0) || !rows_ok(g->h, g->cols, ZERO_BF16)) return ZERO_ERR_INVALID_ARGUMENT;
    if (given(g->y) ? !rows_ok(g->y, g->cols, ZERO_BF16) || !rows_ok(g->x_out, g->cols, g->x.dtype) : given(g->x_out))
        return ZERO_ERR_INVALID_ARGUMENT;
    if (!optional_ok(g->w, g->cols, 0, true) || !optional_ok(g->b, g->cols, 0, true)) return ZERO_ERR_INVALID_ARGUMENT;
    if (!aligned(g->ckpt_xn, kPtrAlign) || !aligned(g->ckpt_h, kPtrAlign) || !aligned(g->mean, 4) || !aligned(g->rstd, 4))
        return ZERO_ERR_INVALID_ARGUMENT;
    if (any_same(g->x_out.data, g->h.data, static_cast<const void*>(g->mean), static_cast<const void*>(g->rstd), g->ckpt_xn, g->ckpt_h))
        return ZERO_ERR_INVALID_ARGUMENT;
    LayerNormArgs a{};
    a.rows = g->rows;
    a.cols = static_cast<int32_t>(g->cols);
    a.eps = eps;
    a.x = view(g->x);
    a.y = view(g->y);
    a.w = view(g->w);
    a.b = view(g->b);
    a.x_out = view(g->x_out);
    a.h = view(g->h);
    a.mean = g->mean;
    a.rstd = g->rstd;
    a.ckpt_xn = static_cast<uint8_t*>(g->ckpt_xn);
    a.ckpt_h = static_cast<uint8_t*>(g->ckpt_h);
    a.format = g->format;
    return hip_status(launch_layer_norm(a, stream));
}

size_t zero_layer_norm_grad_workspace_bytes(int64_t rows, int64_t cols)
{
    return norm_sizes_ok(rows, cols) ? layer_norm_grad_plan(rows, cols).bytes : 0;
}

int zero_layer_norm_grad(const zero_layer_norm_grad_args* g, void* ws, size_t ws_bytes, hipStream_t stream)
{
    if (g == nullptr || !norm_sizes_ok(g->rows, g->cols) || (g->flags & ~ZERO_GRAD_ACCUMULATE) != 0) return ZERO_ERR_INVALID_ARGUMENT;
    const bool accumulate = (g->flags & ZERO_GRAD_ACCUMULATE) != 0;
    if (g->ckpt_xn != nullptr && !format_ok(g->format)) return ZERO_ERR_INVALID_ARGUMENT;
    if (g->cols == 0) return ZERO_OK;
    const int32_t grad_type = accumulate ? ZERO_F32 : 0;
    if (!optional_ok(g->w, g->cols, 0, true) || !optional_ok(g->dw, g->cols, grad_type, true) ||
        !optional_ok(g->db, g->cols, grad_type, true))
        return ZERO_ERR_INVALID_ARGUMENT;
    if (any_same(g->dx.data, g->dy.data, g->dw.data, g->db.data)) return ZERO_ERR_INVALID_ARGUMENT;
    if (g->rows > 0) {
        if (!rows_ok(g->dx, g->cols, 0) || !rows_ok(g->dh, g->cols, ZERO_BF16) || !optional_ok(g->dx_out, g->cols, g->dx.dtype) ||
            !optional_ok(g->dy, g->cols, ZERO_BF16))
            return ZERO_ERR_INVALID_ARGUMENT;
        if (g->rstd == nullptr || !aligned(g->rstd, 4)) return ZERO_ERR_INVALID_ARGUMENT;
        if (g->ckpt_xn != nullptr ? !aligned(g->ckpt_xn, kPtrAlign)
                                  : !rows_ok(g->x_out, g->cols, g->dx.dtype) || g->mean == nullptr || !aligned(g->mean, 4))
            return ZERO_ERR_INVALID_ARGUMENT;
    }
    LayerNormGradArgs a{};
    a.plan = layer_norm_grad_plan(g->rows, g->cols);
    if (a.plan.bytes > 0) {
        if (!buffer_ok(ws)) return ZERO_ERR_INVALID_ARGUMENT;
        if (ws_bytes < a.plan.bytes) return ZERO_ERR_WORKSPACE_TOO_SMALL;
        forget_plans(ws, a.plan.bytes);
    }
    a.rows = g->rows;
    a.cols = static_cast<int32_t>(g->cols);
    a.dh = view(g->dh);
    a.dx_out = view(g->dx_out);
    a.w = view(g->w);
    a.x_out = view(g->x_out);
    a.dx = view(g->dx);
    a.dy = view(g->dy);
    a.dw = view(g->dw);
    a.db = view(g->db);
    a.ckpt_xn = static_cast<const uint8_t*>(g->ckpt_xn);
    a.mean = g->mean;
    a.rstd = g->rstd;
    a.format = g->format;
    a.accumulate = accumulate;
    // Only what this call makes, one after the other from the start of ws: what
    // it overwrites of a step's plan there then always includes the plan's signature.
    const int64_t sums = a.plan.units * a.cols;
    a.row_means = static_cast<float*>(ws);
    a.sum_w = a.row_means + (a.plan.strips ? 2 * g->rows : 0);
    a.sum_b = a.sum_w + (given(g->dw) ? sums : 0);
    return hip_status(launch_layer_norm_grad(a, stream));
}

size_t zero_block_ffn_workspace_bytes(int64_t rows, int64_t cols, int64_t hidden)
{
    return ffn_sizes_ok(rows, cols, hidden) ? ffn_workspace_bytes(kFfnForward, rows, cols, hidden) : 0;
}

int zero_block_ffn(const zero_block_ffn_args* g, void* ws, size_t ws_bytes, hipStream_t stream)
{
    if (g == nullptr || !ffn_sizes_ok(g->rows, g->cols, g->hidden) || !activation_ok(g->act)) return ZERO_ERR_INVALID_ARGUMENT;
    if ((g->ckpt_gate != nullptr || g->ckpt_up != nullptr) && !format_ok(g->format)) return ZERO_ERR_INVALID_ARGUMENT;
    if (g->rows == 0 || g->hidden == 0) return ZERO_OK;
    if (g->cols > 0 && (!rows_ok(g->h, g->cols, ZERO_BF16) || !rows_ok(g->w_gate, g->cols, ZERO_BF16) || !rows_ok(g->w_up, g->cols, ZERO_BF16)))
        return ZERO_ERR_INVALID_ARGUMENT;
    if (!rows_ok(g->a, g->hidden, ZERO_BF16) || !optional_ok(g->gate, g->hidden, ZERO_BF16) || !optional_ok(g->up, g->hidden, ZERO_BF16))
        return ZERO_ERR_INVALID_ARGUMENT;
    if (!aligned(g->ckpt_gate, kPtrAlign) || !aligned(g->ckpt_up, kPtrAlign)) return ZERO_ERR_INVALID_ARGUMENT;
    if (any_same(g->a.data, g->gate.data, g->up.data, g->ckpt_gate, g->ckpt_up)) return ZERO_ERR_INVALID_ARGUMENT;
    const size_t bytes = ffn_workspace_bytes(kFfnForward, g->rows, g->cols, g->hidden);
    if (bytes > 0) {
        if (!buffer_ok(ws)) return ZERO_ERR_INVALID_ARGUMENT;
        if (ws_bytes < bytes) return ZERO_ERR_WORKSPACE_TOO_SMALL;
        forget_plans(ws, bytes);
    }
    FfnArgs a{};
    a.rows = g->rows;
    a.cols = g->cols;
    a.hidden = g->hidden;
    a.h = static_cast<const uint16_t*>(g->h.data);
    a.ld_h = g->h.ld;
    a.w[0] = static_cast<const uint16_t*>(g->w_gate.data);
    a.w[1] = static_cast<const uint16_t*>(g->w_up.data);
    a.ld_w[0] = g->w_gate.ld;
    a.ld_w[1] = g->w_up.ld;
    a.out[0] = view(g->gate);
    a.out[1] = view(g->up);
    a.a = view(g->a);
    a.ckpt[0] = static_cast<uint8_t*>(g->ckpt_gate);
    a.ckpt[1] = static_cast<uint8_t*>(g->ckpt_up);
    a.format = g->format;
    a.act = g->act;
    a.part = static_cast<float*>(ws);
    return hip_status(launch_ffn(kFfnForward, a, stream));
}

size_t zero_block_ffn_grad_workspace_bytes(int64_t rows, int64_t cols, int64_t hidden)
{
    return ffn_sizes_ok(rows, cols, hidden) ? ffn_grad_bytes(rows, cols, hidden) : 0;
}

int zero_block_ffn_grad(const zero_block_ffn_grad_args* g, void* ws, size_t ws_bytes, hipStream_t stream)
{
    if (g == nullptr || g->reserved != 0 || !ffn_sizes_ok(g->rows, g->cols, g->hidden) || !activation_ok(g->act) ||
        (g->flags & ~ZERO_GRAD_ACCUMULATE) != 0)
        return ZERO_ERR_INVALID_ARGUMENT;
    const bool accumulate = (g->flags & ZERO_GRAD_ACCUMULATE) != 0, coded = g->ckpt_gate != nullptr;
    if ((coded || g->ckpt_h != nullptr || g->ckpt_a != nullptr) && !format_ok(g->format)) return ZERO_ERR_INVALID_ARGUMENT;
    if (coded != (g->ckpt_up != nullptr)) return ZERO_ERR_INVALID_ARGUMENT;
    const bool weights = given(g->dw_gate) || given(g->dw_up);
    if (g->rows > 0 && g->hidden > 0 && g->cols > 0) {  // an empty operand may have no address
        if (!weights && (given(g->h) || g->ckpt_h != nullptr || given(g->col_scale))) return ZERO_ERR_INVALID_ARGUMENT;
        if (given(g->col_scale) && g->ckpt_h == nullptr) return ZERO_ERR_INVALID_ARGUMENT;
        if (!given(g->dh) && (given(g->w_gate) || given(g->w_up))) return ZERO_ERR_INVALID_ARGUMENT;
    }
    const int32_t grad_type = accumulate ? ZERO_F32 : 0;
    if (!optional_ok(g->dw_gate, g->cols, grad_type) || !optional_ok(g->dw_up, g->cols, grad_type) ||
        !optional_ok(g->col_scale, g->cols, 0, true) || !optional_ok(g->dh, g->cols, ZERO_BF16))
        return ZERO_ERR_INVALID_ARGUMENT;
    if (g->rows > 0 && g->hidden > 0) {
        if (!rows_ok(g->da, g->hidden, ZERO_BF16) || !rows_ok(g->dgate, g->hidden, ZERO_BF16) || !rows_ok(g->dup, g->hidden, ZERO_BF16))
            return ZERO_ERR_INVALID_ARGUMENT;
        if (!coded && (!rows_ok(g->gate, g->hidden, ZERO_BF16) || !rows_ok(g->up, g->hidden, ZERO_BF16))) return ZERO_ERR_INVALID_ARGUMENT;
        if (given(g->dh) && g->cols > 0 && (!rows_ok(g->w_gate, g->cols, ZERO_BF16) || !rows_ok(g->w_up, g->cols, ZERO_BF16)))
            return ZERO_ERR_INVALID_ARGUMENT;
        if (weights && g->cols > 0 && g->ckpt_h == nullptr && !rows_ok(g->h, g->cols, ZERO_BF16)) return ZERO_ERR_INVALID_ARGUMENT;
    }
    if (!aligned(g->ckpt_gate, kPtrAlign) || !aligned(g->ckpt_up, kPtrAlign) || !aligned(g->ckpt_h, kPtrAlign) || !aligned(g->ckpt_a, kPtrAlign))
        return ZERO_ERR_INVALID_ARGUMENT;
    if (any_same(g->dgate.data, g->dup.data, g->dh.data, g->dw_gate.data, g->dw_up.data, g->ckpt_a)) return ZERO_ERR_INVALID_ARGUMENT;
    const size_t bytes = ffn_grad_bytes(g->rows, g->cols, g->hidden);
    if (bytes > 0) {
        if (!buffer_ok(ws)) return ZERO_ERR_INVALID_ARGUMENT;
        if (ws_bytes < bytes) return ZERO_ERR_WORKSPACE_TOO_SMALL;
        forget_plans(ws, bytes);
    }
    FfnArgs a{};
    a.rows = g->rows;
    a.cols = g->cols;
    a.hidden = g->hidden;
    a.d[0] = static_cast<const uint16_t*>(g->dgate.data);
    a.d[1] = static_cast<const uint16_t*>(g->dup.data);
    a.ld_d[0] = g->dgate.ld;
    a.ld_d[1] = g->dup.ld;
    a.accumulate = accumulate;
    a.part = static_cast<float*>(ws);
    if (g->rows > 0 && g->hidden > 0) {
        FfnActArgs f{};
        f.rows = g->rows;
        f.hidden = g->hidden;
        f.da = view(g->da);
        f.saved[0] = view(g->gate);
        f.saved[1] = view(g->up);
        f.d[0] = view(g->dgate);
        f.d[1] = view(g->dup);
        f.ckpt[0] = static_cast<const uint8_t*>(g->ckpt_gate);
        f.ckpt[1] = static_cast<const uint8_t*>(g->ckpt_up);
        f.ckpt_a = static_cast<uint8_t*>(g->ckpt_a);
        f.format = g->format;
        f.act = g->act;
        const hipError_t e = launch_ffn_act_grad(f, stream);
        if (e != hipSuccess) return ZERO_ERR_HIP;
    }
    if (given(g->dh) && g->rows > 0 && g->cols > 0) {
        a.w[0] = static_cast<const uint16_t*>(g->w_gate.data);
        a.w[1] = static_cast<const uint16_t*>(g->w_up.data);
        a.ld_w[0] = g->w_gate.ld;
        a.ld_w[1] = g->w_up.ld;
        a.out[0] = view(g->dh);
        const hipError_t e = launch_ffn(kFfnInput, a, stream);
        if (e != hipSuccess) return ZERO_ERR_HIP;
    }
    if (!weights || g->hidden == 0 || g->cols == 0 || (g->rows == 0 && accumulate)) return ZERO_OK;
    if (g->ckpt_h == nullptr) {
        a.h = static_cast<const uint16_t*>(g->h.data);
        a.ld_h = g->h.ld;
        a.out[0] = view(g->dw_gate);
        a.out[1] = view(g->dw_up);
        if (!given(g->dw_gate)) {  // one gradient is the first
            a.d[0] = a.d[1];
            a.ld_d[0] = a.ld_d[1];
            a.out[0] = a.out[1];
            a.out[1] = Rows{};
        }
        return hip_status(launch_ffn(kFfnWeight, a, stream));
    }
    for (const bool up : {false, true}) {
        const zero_rows& dw = up ? g->dw_up : g->dw_gate;
        if (!given(dw)) continue;
        const int st = zero_act8_wgrad(up ? &g->dup : &g->dgate, g->ckpt_h, g->rows, g->hidden, g->cols, g->format,
                                       given(g->col_scale) ? &g->col_scale : nullptr, &dw, g->flags, ws, ws_bytes, stream);
        if (st != ZERO_OK) return st;
    }
    return ZERO_OK;
}

}  // extern "C"
