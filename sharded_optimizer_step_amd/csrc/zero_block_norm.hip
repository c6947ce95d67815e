// zero_block_norm.hip -- the norm after a block, its gate, the residual scale
// and add, and the norm before the next block, in one pass over the rows, and
// the backward pass of the same, gfx950.
//
// A row stays in the registers of L lanes, V vectors of 8 columns a lane, so
// every operand is read once and every result written once. Both are streams:
// with bf16 rows and both act8 buffers, 10.06 bytes a column forwards and as
// many backwards.
#include "zero_act8_device.h"

namespace zero {
namespace {

// Sums over the L lanes of a row of N values at once, in every lane, in a fixed
// order. Rows wider than a wave meet in LDS: `red` alternates between two
// halves, so one barrier a call is enough.
template <int L, int N>
__device__ __forceinline__ void row_sum(float (&x)[N], float (*red)[N][16], int& half)
{
#pragma unroll
    for (int n = 0; n < N; ++n) x[n] = wave_sum(x[n]);
    if constexpr (L > 64) {
        constexpr int W = L / 64;
        const int wave = threadIdx.x / 64;
        if (threadIdx.x % 64 == 0) {
#pragma unroll
            for (int n = 0; n < N; ++n) red[half][n][wave] = x[n];
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float s = red[half][n][0];
#pragma unroll
            for (int w = 1; w < W; ++w) s += red[half][n][w];
            x[n] = s;
        }
        half ^= 1;
    }
}

__device__ __forceinline__ void save8(uint8_t* ckpt, int64_t rows, int64_t pitch, int format, int64_t row, int v,
                                      const float (&f)[8])
{
    const Code8 c = format == ZERO_ACT8_E4M3 ? encode8<ZERO_ACT8_E4M3>(f) : encode8<ZERO_ACT8_INT8>(f);
    *(ZERO_G u32x2*)(ckpt + code_at(row, pitch, v)) = c.codes;
    if ((v & 3) == 0) *(ZERO_G uint8_t*)(ckpt + rows * pitch + scale_at(row, pitch, v)) = static_cast<uint8_t>(c.scale);
}

constexpr int threads_of(int L) { return L < 256 ? 256 : L; }

template <int L, int V, bool F32>
__global__ __launch_bounds__(threads_of(L)) void block_norm_kernel(NormArgs a)
{
    constexpr int NT = threads_of(L);
    constexpr int R = NT / L;  // rows of a workgroup
    __shared__ float red[2][1][16];
    int half = 0;
    const int lane = threadIdx.x % L;
    const int nv = static_cast<int>(act8_pitch(a.cols) / 8);
    const int64_t pitch = 8 * static_cast<int64_t>(nv);
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    const bool has_y = a.y.p != nullptr, has_post = a.w_post.p != nullptr, has_pre = a.w_pre.p != nullptr;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * R; base < a.rows; base += static_cast<int64_t>(gridDim.x) * R) {
        // a wave past the last row has nothing to do and, at R > 1, no barrier to meet
        const int64_t row = R > 1 ? base + __builtin_amdgcn_readfirstlane(threadIdx.x / L) : base;
        if (R > 1 && row >= a.rows) break;
        Raw8<F32> rx[V];
        Raw8<false> ry[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int v = lane + j * L, n = v < nv ? a.cols - 8 * v : 0;
            rx[j] = load8<F32>(a.x, row, 8 * v, n);
            ry[j] = has_y ? load8<false>(a.y, row, 8 * v, n) : Raw8<false>{};
        }
        float x[V][8];
#pragma unroll
        for (int j = 0; j < V; ++j) unpack<F32>(rx[j], x[j]);
        if (has_y) {
            float y[V][8], rstd = 1.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) unpack<false>(ry[j], y[j]);
            if (has_post) {
                float s[1] = {0.0f};
#pragma unroll
                for (int j = 0; j < V; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[0] = fmaf(y[j][i], y[j][i], s[0]);
                row_sum<L, 1>(s, red, half);
                rstd = 1.0f / sqrtf(s[0] * inv_cols + a.eps);
                if (a.rstd_post != nullptr && lane == 0) ((ZERO_G float*)a.rstd_post)[row] = rstd;
            }
            const int64_t g = a.gate.p != nullptr ? div_by(static_cast<uint32_t>(row), a.gate_div) : 0;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int v = lane + j * L, n = a.cols - 8 * v;
                if (v >= nv) continue;
                float t[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[j][i] *= rstd;
                if (a.ckpt_post != nullptr) save8(a.ckpt_post, a.rows, pitch, a.format, row, v, y[j]);
                if (has_post) {
                    load8_any(a.w_post, 0, 8 * v, n, t);
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[j][i] *= t[i];
                }
                if (a.gate.p != nullptr) {
                    load8_any(a.gate, g, 8 * v, n, t);
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[j][i] *= a.alpha * t[i];
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[j][i] *= a.alpha;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) x[j][i] += y[j][i];
                store8<F32>(a.x_out, row, 8 * v, n, x[j]);
                // the norm below is that of the residual stream as stored
                if constexpr (!F32) unpack<false>(Raw8<false>{pack8(x[j])}, x[j]);
            }
        }
        if (has_pre) {
            float s[1] = {0.0f};
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) s[0] = fmaf(x[j][i], x[j][i], s[0]);
            row_sum<L, 1>(s, red, half);
            const float rstd = 1.0f / sqrtf(s[0] * inv_cols + a.eps);
            if (a.rstd_pre != nullptr && lane == 0) ((ZERO_G float*)a.rstd_pre)[row] = rstd;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int v = lane + j * L, n = a.cols - 8 * v;
                if (v >= nv) continue;
                float w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[j][i] *= rstd;
                if (a.ckpt_pre != nullptr) save8(a.ckpt_pre, a.rows, pitch, a.format, row, v, x[j]);
                load8_any(a.w_pre, 0, 8 * v, n, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] *= x[j][i];
                store8<false>(a.h, row, 8 * v, n, w);
            }
        }
    }
}

// ------------------------------------------------------------------ backward

// Adds to or overwrites 8 columns of a gradient.
__device__ __forceinline__ void grad8(const Rows& m, int64_t row, int col, int n, bool accumulate, float (&f)[8])
{
    if (m.f32) {
        if (accumulate) {
            float old[8];
            unpack<true>(load8<true>(m, row, col, n), old);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] += old[i];
        }
        store8<true>(m, row, col, n, f);
    } else {
        store8<false>(m, row, col, n, f);
    }
}

// What a lane holds of one vector of a row between its two passes over it.
// CODED: both saved rows are act8 buffers; otherwise either may be the rows
// themselves.
template <bool F32, bool CODED>
struct GradRow {
    Raw8<F32> d;
    Raw8<false> h;
    Raw8<F32> x;
    Raw8<false> y;
    u32x2 cx, cy;
    uint32_t sx, sy;
};

// Which operands a call has; all of it is uniform.
struct GradHas {
    bool dx_out, pre, post, gate, yn, y;
};

template <bool F32, bool CODED>
__device__ __forceinline__ GradRow<F32, CODED> load_row(const NormGradArgs& a, const GradHas& has, int64_t pitch, int64_t row,
                                                        int v, int n)
{
    GradRow<F32, CODED> r{};
    if (has.dx_out) r.d = load8<F32>(a.dx_out, row, 8 * v, n);
    if (has.pre) {
        r.h = load8<false>(a.dh, row, 8 * v, n);
        if (CODED || a.ckpt_pre != nullptr) {
            if (n > 0) {
                r.cx = ld_codes(a.ckpt_pre + code_at(row, pitch, v));
                r.sx = ld_scale(a.ckpt_pre + a.rows * pitch + scale_at(row, pitch, v));
            }
        } else {
            r.x = load8<F32>(a.x_out, row, 8 * v, n);
        }
    }
    if (has.yn) {
        if (CODED || a.ckpt_post != nullptr) {
            if (n > 0) {
                r.cy = ld_codes(a.ckpt_post + code_at(row, pitch, v));
                r.sy = ld_scale(a.ckpt_post + a.rows * pitch + scale_at(row, pitch, v));
            }
        } else {
            r.y = load8<false>(a.y, row, 8 * v, n);
        }
    }
    return r;
}

template <bool F32, bool CODED>
__device__ __forceinline__ void keep_raw(GradRow<F32, CODED>& r)
{
    asm volatile("" : "+v"(r.d.v[0]), "+v"(r.h.v[0]), "+v"(r.cx), "+v"(r.cy), "+v"(r.sx), "+v"(r.sy));
    if constexpr (F32) asm volatile("" : "+v"(r.d.v[1]));
    if constexpr (!CODED) {
        asm volatile("" : "+v"(r.x.v[0]), "+v"(r.y.v[0]));
        if constexpr (F32) asm volatile("" : "+v"(r.x.v[1]));
    }
}

template <bool F32>
__device__ __forceinline__ void saved8(bool coded, int format, u32x2 codes, uint32_t scale, const Raw8<F32>& raw, float rstd,
                                       float (&f)[8])
{
    if (!coded) {
        unpack<F32>(raw, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= rstd;
    } else if (format == ZERO_ACT8_E4M3) {
        decode8<ZERO_ACT8_E4M3>(codes, scale, f);
    } else {
        decode8<ZERO_ACT8_INT8>(codes, scale, f);
    }
}

__device__ __forceinline__ GradHas grad_has(const NormGradArgs& a)
{
    GradHas has;
    has.dx_out = a.dx_out.p != nullptr;
    has.pre = a.dh.p != nullptr;
    has.post = a.w_post.p != nullptr;
    has.gate = a.gate.p != nullptr;
    has.y = a.dy.p != nullptr || a.dw_post.p != nullptr || a.dgate.p != nullptr;
    has.yn = has.y && (has.post || a.dgate.p != nullptr);
    return has;
}

// e = gain * w_post of 8 columns, gain = alpha * gate
__device__ __forceinline__ void load_e(const NormGradArgs& a, const GradHas& has, int64_t gate_row, int v, int n, float (&e)[8])
{
    float t[8];
    if (has.gate) load8_any(a.gate, gate_row, 8 * v, n, e);
    if (has.post) load8_any(a.w_post, 0, 8 * v, n, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        e[i] = has.gate ? a.alpha * e[i] : a.alpha;
        if (has.post) e[i] *= t[i];
    }
}

__device__ __forceinline__ void add_to(float (&sum)[8], const float (&x)[8], const float (&y)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = fmaf(x[i], y[i], sum[i]);
}

// With v = w_pre dh, the two row means that the formulas need, mean(v xn) and
// mean(e d yn) with d = dx_out + rstd (v - xn mean(v xn)), come from three
// sums that do not wait for each other: sum v xn, sum e yn (dx_out + rstd v)
// and sum e yn xn. One exchange between the waves a row, not two. This adds 8
// columns to the three sums.
template <bool F32, bool CODED>
__device__ __forceinline__ void add_row_sums(const NormGradArgs& a, const GradHas& has, int64_t gate_row, int v, int n,
                                             const GradRow<F32, CODED>& raw, float rstd_pre, float rstd_post, float (&s)[3])
{
    float d[8], xn[8], w[8], t[8];
    unpack<F32>(raw.d, d);
    if (has.pre) {
        saved8<F32>(CODED || a.ckpt_pre != nullptr, a.format, raw.cx, raw.sx, raw.x, rstd_pre, xn);
        unpack<false>(raw.h, t);
        load8_any(a.w_pre, 0, 8 * v, n, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            t[i] *= w[i];
            s[0] = fmaf(t[i], xn[i], s[0]);
            d[i] = fmaf(rstd_pre, t[i], d[i]);
        }
    }
    if (has.post && has.yn) {
        saved8<false>(CODED || a.ckpt_post != nullptr, a.format, raw.cy, raw.sy, raw.y, rstd_post, t);
        load_e(a, has, gate_row, v, n, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float ey = w[i] * t[i];
            s[1] = fmaf(ey, d[i], s[1]);
            if (has.pre) s[2] = fmaf(ey, xn[i], s[2]);
        }
    }
}

// rstd_pre mean(v xn) and mean(e d yn) of a row
struct Along {
    float x, y;
};
__device__ __forceinline__ Along along(const GradHas& has, const float (&s)[3], float rstd_pre, float inv_cols)
{
    const float x = has.pre ? rstd_pre * (s[0] * inv_cols) : 0.0f;
    return Along{x, (s[1] - x * s[2]) * inv_cols};
}

// The row sums alone, for rows too wide for one workgroup's registers.
template <bool F32, bool CODED>
__global__ __launch_bounds__(1024) void block_norm_along_kernel(NormGradArgs a)
{
    __shared__ float red[2][3][16];
    int half = 0;
    const GradHas has = grad_has(a);
    const int nv = static_cast<int>(act8_pitch(a.cols) / 8);
    const int64_t pitch = 8 * static_cast<int64_t>(nv);
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float rstd_pre = has.pre ? ((const ZERO_G float*)a.rstd_pre)[row] : 1.0f;
        const float rstd_post = has.post ? ((const ZERO_G float*)a.rstd_post)[row] : 1.0f;
        const int64_t gate_row = has.gate ? div_by(static_cast<uint32_t>(row), a.gate_div) : 0;
        float s[3] = {0.0f, 0.0f, 0.0f};
        for (int v = threadIdx.x; v < nv; v += 1024) {
            const int n = a.cols - 8 * v;
            const GradRow<F32, CODED> raw = load_row<F32, CODED>(a, has, pitch, row, v, n);
            add_row_sums<F32, CODED>(a, has, gate_row, v, n, raw, rstd_pre, rstd_post, s);
        }
        row_sum<1024, 3>(s, red, half);
        if (threadIdx.x == 0) {
            const Along r = along(has, s, rstd_pre, inv_cols);
            ((ZERO_G float*)a.row_sums)[2 * row] = r.x;
            ((ZERO_G float*)a.row_sums)[2 * row + 1] = r.y;
        }
    }
}

// MANY: a unit takes many whole gate rows; dgate is written as each of them
// ends. Otherwise a unit lies in one gate row and its sums of d yn go to the
// workspace, from which the join takes both dgate and dw_post.
//
// A lane keeps its part of a row as loaded, not as fp32, from the sums to the
// results, and unpacks it a second time there: the column sums need the
// registers (keep_raw hides from the compiler that it could keep the fp32).
//
// STRIP: the row sums come from block_norm_along_kernel, and a workgroup takes
// one strip (blockIdx.y) of L * V vectors of its unit's rows.
template <int L, int V, bool F32, bool CODED, bool MANY, bool STRIP>
__global__ __launch_bounds__(threads_of(L)) void block_norm_grad_kernel(NormGradArgs a)
{
    constexpr int NT = threads_of(L);
    constexpr int R = NT / L;
    __shared__ float red[2][3][16];
    int half = 0;
    const int lane = threadIdx.x % L + (STRIP ? static_cast<int>(blockIdx.y) * L * V : 0);
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * R + (R > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / L) : 0);
    if (unit >= a.plan.units) return;  // whole waves at R > 1, no one at R == 1
    const int nv = static_cast<int>(act8_pitch(a.cols) / 8);
    const int64_t pitch = 8 * static_cast<int64_t>(nv);
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    const GradHas has = grad_has(a);
    int64_t gate_row, row, end;
    if constexpr (MANY) {
        gate_row = unit * a.plan.unit_gates;
        row = gate_row * a.plan.gate_rows;
        end = min(a.rows, (gate_row + a.plan.unit_gates) * a.plan.gate_rows);
    } else {
        gate_row = unit / a.plan.per_gate;
        row = gate_row * a.plan.gate_rows + (unit - gate_row * a.plan.per_gate) * a.plan.unit_rows;
        end = min(min(a.rows, (gate_row + 1) * a.plan.gate_rows), row + a.plan.unit_rows);
    }
    float sum_pre[V][8] = {}, sum_yn[V][8] = {}, sum_post[MANY ? V : 1][8] = {};
    while (row < end) {
        // the rows of this unit that share one gate row
        const int64_t stop = MANY ? min(end, (gate_row + 1) * a.plan.gate_rows) : end;
        for (; row < stop; ++row) {
            const float rstd_pre = has.pre ? ((const ZERO_G float*)a.rstd_pre)[row] : 1.0f;
            const float rstd_post = has.post ? ((const ZERO_G float*)a.rstd_post)[row] : 1.0f;
            GradRow<F32, CODED> raw[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int v = lane + j * L, n = v < nv ? a.cols - 8 * v : 0;
                raw[j] = load_row<F32, CODED>(a, has, pitch, row, v, n);
            }
            Along m;
            if constexpr (STRIP) {
                m = Along{((const ZERO_G float*)a.row_sums)[2 * row], ((const ZERO_G float*)a.row_sums)[2 * row + 1]};
            } else {
                float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const int v = lane + j * L, n = v < nv ? a.cols - 8 * v : 0;
                    add_row_sums<F32, CODED>(a, has, gate_row, v, n, raw[j], rstd_pre, rstd_post, s);
                    keep_raw(raw[j]);
                }
                if (has.pre || (has.post && has.yn)) row_sum<L, 3>(s, red, half);
                m = along(has, s, rstd_pre, inv_cols);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int v = lane + j * L, n = a.cols - 8 * v;
                if (v >= nv) continue;
                float d[8], t[8], w[8];
                unpack<F32>(raw[j].d, d);
                if (has.pre) {
                    float xn[8];
                    saved8<F32>(CODED || a.ckpt_pre != nullptr, a.format, raw[j].cx, raw[j].sx, raw[j].x, rstd_pre, xn);
                    unpack<false>(raw[j].h, t);
                    add_to(sum_pre[j], t, xn);
                    load8_any(a.w_pre, 0, 8 * v, n, w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) d[i] = fmaf(-m.x, xn[i], fmaf(rstd_pre, t[i] * w[i], d[i]));
                }
                store8<F32>(a.dx, row, 8 * v, n, d);
                if (!has.y) continue;
                load_e(a, has, gate_row, v, n, w);
                if (has.yn) {
                    saved8<false>(CODED || a.ckpt_post != nullptr, a.format, raw[j].cy, raw[j].sy, raw[j].y, rstd_post, t);
                    add_to(sum_yn[j], d, t);
                }
                if (a.dy.p == nullptr) continue;
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = has.post ? rstd_post * fmaf(-m.y, t[i], w[i] * d[i]) : w[i] * d[i];
                store8<false>(a.dy, row, 8 * v, n, w);
            }
        }
        if constexpr (MANY) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int v = lane + j * L, n = a.cols - 8 * v;
                if (v >= nv) continue;
                float t[8];
                load8_any(a.gate, gate_row, 8 * v, n, t);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum_yn[j][i] *= a.alpha;
                add_to(sum_post[j], t, sum_yn[j]);
                if (a.dgate.p != nullptr) {
                    if (has.post) {
                        load8_any(a.w_post, 0, 8 * v, n, t);
#pragma unroll
                        for (int i = 0; i < 8; ++i) sum_yn[j][i] *= t[i];
                    }
                    grad8(a.dgate, gate_row, 8 * v, n, a.accumulate, sum_yn[j]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) sum_yn[j][i] = 0.0f;
            }
            ++gate_row;
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int v = lane + j * L, n = a.cols - 8 * v;
        if (v >= nv) continue;
        const Rows pre{a.sum_pre, a.cols, 1}, post{a.sum_post, a.cols, 1};
        if (a.dw_pre.p != nullptr) store8<true>(pre, unit, 8 * v, n, sum_pre[j]);
        if (a.dw_post.p != nullptr || (!MANY && a.dgate.p != nullptr))
            store8<true>(post, unit, 8 * v, n, MANY ? sum_post[j] : sum_yn[j]);
    }
}

// The units' sums joined in order: 64 columns a workgroup, its 16 waves each
// a sixteenth of the units that are summed together.
constexpr int kJoinWaves = 16;

// The sum over the waves of a workgroup, lane by lane.
__device__ __forceinline__ float across_waves(float s, float* lds)
{
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    __syncthreads();
    lds[wave * 64 + lane] = s;
    __syncthreads();
    s = lds[lane];
#pragma unroll
    for (int w = 1; w < kJoinWaves; ++w) s += lds[w * 64 + lane];
    return s;
}

__device__ __forceinline__ float join_sum(const float* part, int64_t first, int64_t count, int cols, int col, float* lds)
{
    const int wave = threadIdx.x / 64;
    const int64_t each = (count + kJoinWaves - 1) / kJoinWaves;
    const int64_t from = first + wave * each, to = min(first + count, from + each);
    float s = 0.0f;
    if (col < cols) {
        for (int64_t u = from; u < to; ++u) s += ((const ZERO_G float*)part)[u * cols + col];
    }
    return across_waves(s, lds);
}

__device__ __forceinline__ float one(const Rows& m, int64_t row, int col)
{
    if (m.f32) return ((const ZERO_G float*)m.p)[row * m.ld + col];
    return __uint_as_float(static_cast<uint32_t>(((const ZERO_G uint16_t*)m.p)[row * m.ld + col]) << 16);
}
__device__ __forceinline__ void grad1(const Rows& m, int64_t row, int col, bool accumulate, float f)
{
    if (m.f32) {
        ZERO_G float* p = (ZERO_G float*)m.p + row * m.ld + col;
        *p = accumulate ? *p + f : f;
    } else {
        ((ZERO_G uint16_t*)m.p)[row * m.ld + col] = static_cast<uint16_t>(pack_bf16(f, 0.0f));
    }
}

__global__ __launch_bounds__(64 * kJoinWaves) void block_norm_join_kernel(NormGradArgs a)
{
    __shared__ float lds[64 * kJoinWaves];
    const int col = blockIdx.x * 64 + threadIdx.x % 64;
    const bool writes = threadIdx.x < 64 && col < a.cols;
    if (a.dw_pre.p != nullptr) {
        const float s = join_sum(a.sum_pre, 0, a.plan.units, a.cols, col, lds);
        if (writes) grad1(a.dw_pre, 0, col, a.accumulate, s);
    }
    if (a.plan.per_gate == 0) {
        if (a.dw_post.p != nullptr) {
            const float s = join_sum(a.sum_post, 0, a.plan.units, a.cols, col, lds);
            if (writes) grad1(a.dw_post, 0, col, a.accumulate, s);
        }
    } else if (a.dw_post.p != nullptr || a.dgate.p != nullptr) {
        const int64_t gates = a.plan.gates, per_gate = a.plan.per_gate;
        const bool reads = col < a.cols && gates > 0;
        const float w = reads && a.w_post.p != nullptr ? one(a.w_post, 0, col) : 1.0f;
        float total = 0.0f;
        if (gates < kJoinWaves) {
            for (int64_t g = 0; g < gates; ++g) {
                const float s = join_sum(a.sum_post, g * per_gate, per_gate, a.cols, col, lds);
                if (!writes) continue;
                total += (a.gate.p != nullptr ? one(a.gate, g, col) : 1.0f) * s;
                if (a.dgate.p != nullptr) grad1(a.dgate, g, col, a.accumulate, a.alpha * w * s);
            }
        } else {
            // a gate row a wave
            const int64_t each = (gates + kJoinWaves - 1) / kJoinWaves, wave = threadIdx.x / 64;
            if (reads) {
                for (int64_t g = wave * each; g < min(gates, (wave + 1) * each); ++g) {
                    float s = 0.0f;
                    for (int64_t u = 0; u < per_gate; ++u) s += ((const ZERO_G float*)a.sum_post)[(g * per_gate + u) * a.cols + col];
                    total += one(a.gate, g, col) * s;
                    if (a.dgate.p != nullptr) grad1(a.dgate, g, col, a.accumulate, a.alpha * w * s);
                }
            }
            total = across_waves(total, lds);
        }
        if (writes && a.dw_post.p != nullptr) grad1(a.dw_post, 0, col, a.accumulate, a.alpha * total);
    }
}

}  // namespace

template <int L, int V>
static void norm_shape(const NormArgs& a, hipStream_t s)
{
    const int64_t groups = (a.rows + threads_of(L) / L - 1) / (threads_of(L) / L);
    const unsigned grid = static_cast<unsigned>(groups < (1 << 20) ? groups : 1 << 20);
    if (a.x.f32) block_norm_kernel<L, V, true><<<grid, threads_of(L), 0, s>>>(a);
    else block_norm_kernel<L, V, false><<<grid, threads_of(L), 0, s>>>(a);
}

hipError_t launch_block_norm(const NormArgs& a, hipStream_t s)
{
    const int nv = static_cast<int>(act8_pitch(a.cols) / 8);
    if (nv <= 64) norm_shape<64, 1>(a, s);
    else if (nv <= 128) norm_shape<64, 2>(a, s);
    else if (nv <= 256) norm_shape<256, 1>(a, s);
    else if (nv <= 512) norm_shape<256, 2>(a, s);
    else if (nv <= 1024) norm_shape<512, 2>(a, s);
    else norm_shape<1024, 2>(a, s);
    return hipGetLastError();
}

// ------------------------------------------------------------------ the backward pass's plan

// A workgroup's registers hold rows of 8192 columns with their column sums;
// wider rows go in strips of 4096.
constexpr int kGradMaxVecs = 1024;
constexpr int kStripLanes = 512;

static int grad_lanes(int64_t cols)
{
    const int64_t nv = act8_pitch(cols) / 8;
    return nv <= 128 ? 64 : nv <= 256 ? 256 : 512;
}

NormGradPlan norm_grad_plan(int64_t rows, int64_t cols, int64_t gate_rows)
{
    NormGradPlan p{};
    const int64_t nv = act8_pitch(cols) / 8;
    p.strips = nv <= kGradMaxVecs ? 0 : (nv + kStripLanes - 1) / kStripLanes;
    p.gate_rows = gate_rows > 0 && gate_rows < rows ? gate_rows : (rows > 0 ? rows : 1);
    p.gates = (rows + p.gate_rows - 1) / p.gate_rows;
    // 16 waves a compute unit: enough rows in flight, and as few partial rows as that takes
    int64_t target = static_cast<int64_t>(kComputeUnits) * 16 * 64 / grad_lanes(cols);
    if (p.strips > 0) target /= p.strips;
    if (p.gates >= target) {
        p.unit_gates = (p.gates + target - 1) / target;
        p.units = (p.gates + p.unit_gates - 1) / p.unit_gates;
    } else if (p.gates > 0) {
        p.per_gate = target / p.gates;
        if (p.per_gate > p.gate_rows) p.per_gate = p.gate_rows;
        p.unit_rows = (p.gate_rows + p.per_gate - 1) / p.per_gate;
        p.per_gate = (p.gate_rows + p.unit_rows - 1) / p.unit_rows;
        // the last gate row may be short: its units past the end sum nothing
        p.units = p.gates * p.per_gate;
    } else {
        p.per_gate = 1;
    }
    p.bytes = 2 * sizeof(float) * static_cast<size_t>(p.units * cols + (p.strips > 0 ? rows : 0));
    return p;
}

template <int L, int V, bool STRIP, bool F32, bool CODED>
static void grad_split(const NormGradArgs& a, hipStream_t s)
{
    constexpr int R = threads_of(L) / L;
    const dim3 grid(static_cast<unsigned>((a.plan.units + R - 1) / R), STRIP ? static_cast<unsigned>(a.plan.strips) : 1);
    if constexpr (STRIP) {
        const unsigned rows = static_cast<unsigned>(a.rows < (1 << 20) ? a.rows : 1 << 20);
        block_norm_along_kernel<F32, CODED><<<rows, 1024, 0, s>>>(a);
    }
    if (a.plan.per_gate == 0) block_norm_grad_kernel<L, V, F32, CODED, true, STRIP><<<grid, threads_of(L), 0, s>>>(a);
    else block_norm_grad_kernel<L, V, F32, CODED, false, STRIP><<<grid, threads_of(L), 0, s>>>(a);
}

template <int L, int V, bool STRIP>
static void grad_shape(const NormGradArgs& a, hipStream_t s)
{
    // rows that are not needed are neither coded nor read
    const bool coded = (a.ckpt_pre != nullptr || a.x_out.p == nullptr) && (a.ckpt_post != nullptr || a.y.p == nullptr);
    if (a.dx.f32 && coded) grad_split<L, V, STRIP, true, true>(a, s);
    else if (a.dx.f32) grad_split<L, V, STRIP, true, false>(a, s);
    else if (coded) grad_split<L, V, STRIP, false, true>(a, s);
    else grad_split<L, V, STRIP, false, false>(a, s);
}

hipError_t launch_block_norm_grad(const NormGradArgs& a, hipStream_t s)
{
    if (a.plan.units > 0) {
        const int nv = static_cast<int>(act8_pitch(a.cols) / 8);
        if (nv <= 64) grad_shape<64, 1, false>(a, s);
        else if (nv <= 128) grad_shape<64, 2, false>(a, s);
        else if (nv <= 256) grad_shape<256, 1, false>(a, s);
        else if (nv <= 512) grad_shape<512, 1, false>(a, s);
        else if (nv <= kGradMaxVecs) grad_shape<512, 2, false>(a, s);
        else grad_shape<kStripLanes, 1, true>(a, s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.dw_pre.p == nullptr && a.dw_post.p == nullptr && (a.dgate.p == nullptr || a.plan.per_gate == 0))
        return hipSuccess;
    block_norm_join_kernel<<<static_cast<unsigned>((a.cols + 63) / 64), 64 * kJoinWaves, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace zero
