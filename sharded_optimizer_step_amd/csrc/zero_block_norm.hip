// zero_block_norm.hip -- the norm after a block, its gate, the residual scale
// and add, and the norm before the next block, in one pass over the rows, and
// the backward pass of the same, gfx950.
//
// A row stays in the registers of L lanes, V vectors of 8 columns a lane, so
// every operand is read once and every result written once (backwards, rows too
// wide for that are read twice, see below). Both are streams, bound by HBM: with
// bf16 rows and both act8 buffers, 10.06 bytes a column forwards and as many
// backwards. 16384 x 4096: forwards 123 to 147 us (4.6 to 5.5 TB/s, where copies
// run at 4.8 to 5.4), backwards 143 and 5 to join its sums (4.7). 3001 x 5003
// with fp32 rows: forwards 60 us (14.06 bytes a column and 4 of a gate for every
// row, 4.5 TB/s), backwards 76 and 9 from rows as they are (18 bytes, 3.6 TB/s);
// their rows start anywhere in a line, and ten waves a workgroup leave room for
// one on a compute unit. 128 x 768: 5.6, and 6.4 and 3.4, the latency of a few
// rows in turn.
#include "zero_act8_device.h"

namespace zero {
namespace {

// Rows of up to 512 columns take a wave each, four to a workgroup; wider ones
// a workgroup of as many waves as they have 512 columns.
constexpr int kWaveVecs = 64;
constexpr int kMaxLanes = 1024;
constexpr int kRoomWaves = 16;  // of a compute unit, for rows that stay in registers

// Sums of N values at once over the lanes of a row, in every lane, in a fixed
// order. The waves of a workgroup meet in LDS: `red` alternates between two
// halves, so one barrier a call is enough.
template <bool WAVE, int N>
__device__ __forceinline__ void row_sum(float (&x)[N], float (*red)[N][kMaxLanes / 64], int& half)
{
#pragma unroll
    for (int n = 0; n < N; ++n) x[n] = wave_sum(x[n]);
    if constexpr (!WAVE) {
        const int waves = blockDim.x / 64;
        if (threadIdx.x % 64 == 0) {
#pragma unroll
            for (int n = 0; n < N; ++n) red[half][n][threadIdx.x / 64] = x[n];
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) x[n] = 0.0f;
        for (int w = 0; w < waves; w += 2) {  // in pairs: half the roundings
#pragma unroll
            for (int n = 0; n < N; ++n) x[n] += red[half][n][w] + (w + 1 < waves ? red[half][n][w + 1] : 0.0f);
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

// A lane's first vector and the distance to its next one, and the row of its
// wave or workgroup.
template <bool WAVE>
__device__ __forceinline__ int row_lane() { return WAVE ? threadIdx.x % 64 : threadIdx.x; }
template <bool WAVE>
__device__ __forceinline__ int row_lanes() { return WAVE ? 64 : blockDim.x; }
template <bool WAVE>
__device__ __forceinline__ int64_t row_slot()
{
    return WAVE ? static_cast<int64_t>(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64) : blockIdx.x;
}

// The sum of squares of a row: in fp32 over two waves, in fp64 over those.
template <bool WAVE>
__device__ __forceinline__ double row_squares(float x, float (*red)[kMaxLanes / 64], int& half)
{
    x = wave_sum(x);
    double s = x;
    if constexpr (!WAVE) {
        const int waves = blockDim.x / 64;
        if (threadIdx.x % 64 == 0) red[half][threadIdx.x / 64] = x;
        __syncthreads();
        s = 0.0;
        for (int w = 0; w < waves; w += 2) s += red[half][w] + (w + 1 < waves ? red[half][w + 1] : 0.0f);
        half ^= 1;
    }
    return s;
}

// 1 / sqrt(sum / cols + eps) in two parts: an fp32 root corrected by its
// residual in fp64.
struct Rstd {
    float hi, lo;
};
__device__ __forceinline__ Rstd row_rstd(double sum, double inv_cols, float eps)
{
    const double a = fma(sum, inv_cols, static_cast<double>(eps));
    if (!(a > 0x1p-100 && a < 0x1p100)) return Rstd{1.0f / sqrtf(static_cast<float>(a)), 0.0f};
    const double r = __builtin_amdgcn_rsqf(static_cast<float>(a));
    const double root = fma(0.5 * r, fma(-a * r, r, 1.0), r);
    const float hi = static_cast<float>(root);
    return Rstd{hi, static_cast<float>(root - hi)};
}

// x / sqrt(..) of 8 columns. A code and the middle of two codes have 8
// significant bits at most, so the code of the fp32 product is that of the
// exact one unless the product ends in 16 zeros: those few, one in 65536, go
// one step towards the exact value. (Also where no checkpoint is written: what
// a call computes does not depend on what it saves.)
__device__ __forceinline__ void normalise(float (&x)[8], Rstd r)
{
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = x[i] * r.hi;
    const auto tails = [&](int i) {
        return __builtin_bit_cast(u16x2, __builtin_amdgcn_perm(__float_as_uint(v[i + 1]), __float_as_uint(v[i]), 0x05040100u));
    };
    const u16x2 least = __builtin_elementwise_min(__builtin_elementwise_min(tails(0), tails(2)),
                                                  __builtin_elementwise_min(tails(4), tails(6)));
    if (least.x == 0 || least.y == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t bits = __float_as_uint(v[i]);
            const float off = fmaf(x[i], r.lo, fmaf(x[i], r.hi, -v[i])) * v[i];
            const uint32_t step = off > 0.0f ? 1u : off < 0.0f ? ~0u : 0u;  // none for a NaN, and for what is exact
            if ((bits & 0xFFFFu) == 0) v[i] = __uint_as_float(bits + step);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v[i];
}

__device__ __forceinline__ void add_squares(float& s, const float (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
}

// 8 columns of e = alpha * gate * w_post, what the normalised block output is
// multiplied with; absent operands are ones.
__device__ __forceinline__ void load_gain(const Rows& gate, const Rows& w_post, float alpha, int64_t gate_row, int v, int n, float (&e)[8])
{
    const bool has_gate = gate.p != nullptr, has_post = w_post.p != nullptr;
    float t[8];
    if (has_gate) load8_any(gate, gate_row, 8 * v, n, e);
    if (has_post) load8_any(w_post, 0, 8 * v, n, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        e[i] = has_gate ? alpha * e[i] : alpha;
        if (has_post) e[i] *= t[i];
    }
}

// A workgroup (or wave) takes neighbouring rows, V vectors of 8 columns a
// lane. At V == 1 a lane keeps its columns' gain and weight in registers, and
// the next row's loads are started before this row's sums, so that they are in
// flight across its two barriers; the gain is read again where the gate's row
// changes. (16 waves of rows a compute unit; 20, 32 and 48 are level with it on
// large calls, and 1000 x 4096 takes 15.5 us in 32 instead of 12.9.)
template <bool WAVE, int V, bool F32>
__global__ __launch_bounds__(WAVE ? 256 : kMaxLanes) void block_norm_kernel(NormArgs a)
{
    constexpr bool kEarly = V == 1;
    __shared__ float red[2][kMaxLanes / 64];
    int half = 0;
    const int lane = row_lane<WAVE>(), lanes = row_lanes<WAVE>();
    const int nv = static_cast<int>(act8_pitch(a.cols) / 8);
    const int64_t pitch = 8 * static_cast<int64_t>(nv);
    const double inv_cols = 1.0 / a.cols;
    const bool has_y = a.y.p != nullptr, has_post = a.w_post.p != nullptr, has_pre = a.w_pre.p != nullptr;
    int64_t row = row_slot<WAVE>() * a.unit_rows;
    const int64_t end = min(a.rows, row + a.unit_rows);
    if (row >= end) return;  // whole waves, and none where there are barriers
    Raw8<F32> next_x[V];
    Raw8<false> next_y[V];
    const auto load = [&](int64_t r) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int v = lane + j * lanes, n = v < nv ? a.cols - 8 * v : 0;
            next_y[j] = {};
            if (a.stream != 0) {
                if (has_y) next_y[j] = load8<false, true>(a.y, r, 8 * v, n);
                next_x[j] = load8<F32, true>(a.x, r, 8 * v, n);
            } else {
                if (has_y) next_y[j] = load8<false>(a.y, r, 8 * v, n);
                next_x[j] = load8<F32>(a.x, r, 8 * v, n);
            }
        }
    };
    int64_t gate_row = -1;
    float e[8], w[8];
    if (kEarly) {
        load(row);
        if (has_pre) load8_any(a.w_pre, 0, 8 * lane, lane < nv ? a.cols - 8 * lane : 0, w);
    }
    for (; row < end; ++row) {
        const int64_t g = a.gate.p != nullptr ? div_by(static_cast<uint32_t>(row), a.gate_div) : 0;
        if (kEarly && has_y && g != gate_row) load_gain(a.gate, a.w_post, a.alpha, g, lane, lane < nv ? a.cols - 8 * lane : 0, e);
        gate_row = g;
        if (!kEarly) load(row);
        float x[V][8], y[V][8];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int v = lane + j * lanes, n = v < nv ? a.cols - 8 * v : 0;
            unpack<F32>(next_x[j], 8 * v, n, x[j]);
            unpack<false>(next_y[j], 8 * v, n, y[j]);
        }
        if (kEarly && row + 1 < end) load(row + 1);
        if (has_y) {
            Rstd rstd{1.0f, 0.0f};
            if (has_post) {
                float s = 0.0f;
#pragma unroll
                for (int j = 0; j < V; ++j) add_squares(s, y[j]);
                rstd = row_rstd(row_squares<WAVE>(s, red, half), inv_cols, a.eps);
                if (a.rstd_post != nullptr && lane == 0) ((ZERO_G float*)a.rstd_post)[row] = rstd.hi;
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int v = lane + j * lanes, n = a.cols - 8 * v;
                if (v >= nv) continue;
                if (!kEarly) load_gain(a.gate, a.w_post, a.alpha, g, v, n, e);
                if (has_post) normalise(y[j], rstd);
                if (a.ckpt_post != nullptr) save8(a.ckpt_post, a.rows, pitch, a.format, row, v, y[j]);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[j][i] = fmaf(e[i], y[j][i], x[j][i]);
                store8<F32, true>(a.x_out, row, 8 * v, n, x[j]);
                // the norm below is that of the residual stream as stored
                if constexpr (!F32) round_bf16(x[j]);
            }
        }
        if (has_pre) {
            float s = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) add_squares(s, x[j]);
            const Rstd rstd = row_rstd(row_squares<WAVE>(s, red, half), inv_cols, a.eps);
            if (a.rstd_pre != nullptr && lane == 0) ((ZERO_G float*)a.rstd_pre)[row] = rstd.hi;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int v = lane + j * lanes, n = a.cols - 8 * v;
                if (v >= nv) continue;
                if (!kEarly) load8_any(a.w_pre, 0, 8 * v, n, w);
                normalise(x[j], rstd);
                if (a.ckpt_pre != nullptr) save8(a.ckpt_pre, a.rows, pitch, a.format, row, v, x[j]);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[j][i] = x[j][i] * w[i];
                store8<false, true>(a.h, row, 8 * v, n, y[j]);
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
            unpack<true>(load8<true>(m, row, col, n), col, n, old);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] += old[i];
        }
        store8<true>(m, row, col, n, f);
    } else {
        store8<false>(m, row, col, n, f);
    }
}

// What a lane reads of a row.
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
    float rstd_pre, rstd_post;
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
    r.rstd_pre = has.pre ? ((const ZERO_G float*)a.rstd_pre)[row] : 1.0f;
    r.rstd_post = has.post ? ((const ZERO_G float*)a.rstd_post)[row] : 1.0f;
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

template <bool F32>
__device__ __forceinline__ void saved8(bool coded, int format, u32x2 codes, uint32_t scale, const Raw8<F32>& raw, int v, int n,
                                       float rstd, float (&f)[8])
{
    if (!coded) {
        unpack<F32>(raw, 8 * v, n, f);
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

// 8 columns of a row as both passes over it need them.
struct GradCols {
    float d[8];   // dx_out + rstd_pre v, v = w_pre dh
    float xn[8], yn[8];
};

// With v = w_pre dh, the two row means that the formulas need, mean(v xn) and
// mean(e d yn) with d = dx_out + rstd (v - xn mean(v xn)), come from three
// sums that do not wait for each other: sum v xn, sum e yn (dx_out + rstd v)
// and sum e yn xn. One exchange between the waves a row, not two. This adds 8
// columns to the three sums, and dh xn to sum_pre.
template <bool F32, bool CODED>
__device__ __forceinline__ void add_row_sums(const NormGradArgs& a, const GradHas& has, const GradRow<F32, CODED>& raw,
                                             int v, int n, const float (&w_pre)[8], const float (&e)[8], GradCols& c, float (&s)[3],
                                             float (&sum_pre)[8])
{
    unpack<F32>(raw.d, 8 * v, n, c.d);
    if (has.pre) {
        float h[8];
        saved8<F32>(CODED || a.ckpt_pre != nullptr, a.format, raw.cx, raw.sx, raw.x, v, n, raw.rstd_pre, c.xn);
        unpack<false>(raw.h, 8 * v, n, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sum_pre[i] = fmaf(h[i], c.xn[i], sum_pre[i]);
            const float t = h[i] * w_pre[i];
            s[0] = fmaf(t, c.xn[i], s[0]);
            c.d[i] = fmaf(raw.rstd_pre, t, c.d[i]);
        }
    }
    if (has.yn) {
        saved8<false>(CODED || a.ckpt_post != nullptr, a.format, raw.cy, raw.sy, raw.y, v, n, raw.rstd_post, c.yn);
        if (has.post) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float ey = e[i] * c.yn[i];
                s[1] = fmaf(ey, c.d[i], s[1]);
                if (has.pre) s[2] = fmaf(ey, c.xn[i], s[2]);
            }
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

// The row sums alone, for rows too wide for one workgroup's registers: they
// are then read twice.
template <bool F32, bool CODED>
__global__ __launch_bounds__(kMaxLanes) void block_norm_along_kernel(NormGradArgs a)
{
    __shared__ float red[2][3][kMaxLanes / 64];
    int half = 0;
    const GradHas has = grad_has(a);
    const int nv = static_cast<int>(act8_pitch(a.cols) / 8);
    const int64_t pitch = 8 * static_cast<int64_t>(nv);
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t gate_row = has.gate ? div_by(static_cast<uint32_t>(row), a.gate_div) : 0;
        float s[3] = {0.0f, 0.0f, 0.0f}, unused[8] = {}, rstd_pre = 1.0f;
        for (int v = threadIdx.x; v < nv; v += kMaxLanes) {
            const int n = a.cols - 8 * v;
            const GradRow<F32, CODED> raw = load_row<F32, CODED>(a, has, pitch, row, v, n);
            float w[8] = {}, e[8];
            if (has.pre) load8_any(a.w_pre, 0, 8 * v, n, w);
            load_gain(a.gate, a.w_post, a.alpha, gate_row, v, n, e);
            GradCols c;
            add_row_sums<F32, CODED>(a, has, raw, v, n, w, e, c, s, unused);
            rstd_pre = raw.rstd_pre;
        }
        row_sum<false, 3>(s, red, half);
        if (threadIdx.x == 0) {
            const Along r = along(has, s, rstd_pre, inv_cols);
            ((ZERO_G float*)a.row_sums)[2 * row] = r.x;
            ((ZERO_G float*)a.row_sums)[2 * row + 1] = r.y;
        }
    }
}

// A lane keeps 8 columns: their weights and their column sums in registers
// over all rows of its unit. The next row's loads are started before this
// row's sums, so they are in flight across its barrier.
//
// MANY: a unit takes many whole gate rows; dgate is written as each of them
// ends. Otherwise a unit lies in one gate row and its sums of d yn go to the
// workspace, from which the join takes both dgate and dw_post.
//
// STRIP: the row sums come from block_norm_along_kernel, and a workgroup takes
// one strip (blockIdx.y) of its unit's columns.
//
// MAX: the most threads of a workgroup. Those of 1024 have 128 registers each,
// and those of 768 have 168: some of them do without the early loads.
template <bool WAVE, int MAX, bool F32, bool CODED, bool MANY, bool STRIP>
__global__ __launch_bounds__(MAX) void block_norm_grad_kernel(NormGradArgs a)
{
    __shared__ float red[2][3][kMaxLanes / 64];
    int half = 0;
    const int v = row_lane<WAVE>() + (STRIP ? static_cast<int>(blockIdx.y * blockDim.x) : 0);
    const int64_t unit = row_slot<WAVE>();
    if (unit >= a.plan.units) return;  // whole waves, and none where there are barriers
    const int nv = static_cast<int>(act8_pitch(a.cols) / 8);
    const int64_t pitch = 8 * static_cast<int64_t>(nv);
    const int n = v < nv ? a.cols - 8 * v : 0;
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
    constexpr bool kEarly = MAX < 768 || (MAX == 768 && (CODED || !MANY));
    float sum_pre[8] = {}, sum_yn[8] = {}, sum_post[8] = {};
    float w_pre[8] = {}, e[8];
    if (has.pre) load8_any(a.w_pre, 0, 8 * v, n, w_pre);
    load_gain(a.gate, a.w_post, a.alpha, gate_row, v, n, e);
    GradRow<F32, CODED> next{};
    if (kEarly && row < end) next = load_row<F32, CODED>(a, has, pitch, row, v, n);
    int64_t gate_end = (gate_row + 1) * a.plan.gate_rows;
    for (; row < end; ++row) {
        const GradRow<F32, CODED> raw = kEarly ? next : load_row<F32, CODED>(a, has, pitch, row, v, n);
        if (kEarly && row + 1 < end) next = load_row<F32, CODED>(a, has, pitch, row + 1, v, n);
        Along m;
        if constexpr (STRIP) m = Along{((const ZERO_G float*)a.row_sums)[2 * row], ((const ZERO_G float*)a.row_sums)[2 * row + 1]};
        GradCols c;
        float s[3] = {0.0f, 0.0f, 0.0f};
        add_row_sums<F32, CODED>(a, has, raw, v, n, w_pre, e, c, s, sum_pre);
        if constexpr (!STRIP) {
            if (has.pre || (has.post && has.yn)) row_sum<WAVE, 3>(s, red, half);
            m = along(has, s, raw.rstd_pre, inv_cols);
        }
        if (v < nv) {
            if (has.pre) {
#pragma unroll
                for (int i = 0; i < 8; ++i) c.d[i] = fmaf(-m.x, c.xn[i], c.d[i]);
            }
            if (a.stream != 0) store8<F32, true>(a.dx, row, 8 * v, n, c.d);
            else store8<F32>(a.dx, row, 8 * v, n, c.d);
            if (has.yn) {
#pragma unroll
                for (int i = 0; i < 8; ++i) sum_yn[i] = fmaf(c.d[i], c.yn[i], sum_yn[i]);
            }
            if (a.dy.p != nullptr) {
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o[i] = has.post ? raw.rstd_post * fmaf(-m.y, c.yn[i], e[i] * c.d[i]) : e[i] * c.d[i];
                if (a.stream != 0) store8<false, true>(a.dy, row, 8 * v, n, o);
                else store8<false>(a.dy, row, 8 * v, n, o);
            }
        }
        if constexpr (MANY) {
            if (row + 1 == gate_end || row + 1 == end) {
                float t[8];
                load8_any(a.gate, gate_row, 8 * v, n, t);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    sum_yn[i] *= a.alpha;
                    sum_post[i] = fmaf(t[i], sum_yn[i], sum_post[i]);
                }
                if (a.dgate.p != nullptr) {
                    if (has.post) {
                        load8_any(a.w_post, 0, 8 * v, n, t);
#pragma unroll
                        for (int i = 0; i < 8; ++i) sum_yn[i] *= t[i];
                    }
                    grad8(a.dgate, gate_row, 8 * v, n, a.accumulate, sum_yn);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) sum_yn[i] = 0.0f;
                ++gate_row;
                gate_end += a.plan.gate_rows;
                if (row + 1 < end) load_gain(a.gate, a.w_post, a.alpha, gate_row, v, n, e);
            }
        }
    }
    if (v >= nv) return;
    const Rows pre{a.sum_pre, a.cols, 1}, post{a.sum_post, a.cols, 1};
    if (a.dw_pre.p != nullptr) store8<true>(pre, unit, 8 * v, n, sum_pre);
    if (a.dw_post.p != nullptr || (!MANY && a.dgate.p != nullptr)) store8<true>(post, unit, 8 * v, n, MANY ? sum_post : sum_yn);
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

// The units' sums joined in order: 64 columns a workgroup, its 16 waves each a
// sixteenth of the units. blockIdx.y 0 makes dw_pre, 1 dw_post (each unit's
// sum of d yn times its gate row, or with many gate rows the units' own
// sums), 2 and on dgate, one gate row a workgroup, or one a wave where there
// are many. 512 units of 4096 columns take 5.3 us, 295 of 5003 8.8: latency of
// the loads, a sixteenth of the units after each other.
constexpr int kJoinWaves = 16;

// How many gate rows a workgroup of the join takes.
__host__ __device__ inline int64_t join_gates(const NormGradPlan& p) { return p.gates < kJoinWaves ? 1 : kJoinWaves; }

// The sum over the waves of a workgroup, lane by lane.
__device__ __forceinline__ float across_waves(float s, float* lds)
{
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    lds[wave * 64 + lane] = s;
    __syncthreads();
    s = lds[lane];
#pragma unroll
    for (int w = 1; w < kJoinWaves; ++w) s += lds[w * 64 + lane];
    return s;
}

// The sum of column col over `count` rows of part, in order, eight loads at a time.
__device__ __forceinline__ float column_sum(const float* part, int64_t first, int64_t count, int cols, int col)
{
    const ZERO_G float* p = (const ZERO_G float*)part + first * cols + col;
    float s = 0.0f;
    int64_t u = 0;
    for (; u + 8 <= count; u += 8) {
        float t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = p[static_cast<int64_t>(i) * cols];
#pragma unroll
        for (int i = 0; i < 8; ++i) s += t[i];
        p += 8 * static_cast<int64_t>(cols);
    }
    for (; u < count; ++u, p += cols) s += *p;
    return s;
}

__global__ __launch_bounds__(64 * kJoinWaves) void block_norm_join_kernel(NormGradArgs a)
{
    __shared__ float lds[64 * kJoinWaves];
    const int col = blockIdx.x * 64 + threadIdx.x % 64;
    const int64_t wave = threadIdx.x / 64;
    const bool reads = col < a.cols, writes = reads && wave == 0;
    const int64_t per_gate = a.plan.per_gate;
    if (blockIdx.y >= 2) {
        const int64_t step = join_gates(a.plan), g0 = (blockIdx.y - 2) * step;
        float s = 0.0f;
        if (step > 1) {
            const int64_t g = g0 + wave;
            if (!reads || g >= a.plan.gates) return;
            s = column_sum(a.sum_post, g * per_gate, per_gate, a.cols, col);
            if (a.w_post.p != nullptr) s *= one(a.w_post, 0, col);
            grad1(a.dgate, g, col, a.accumulate, a.alpha * s);
            return;
        }
        const int64_t each = (per_gate + kJoinWaves - 1) / kJoinWaves, from = min(per_gate, wave * each);
        if (reads) s = column_sum(a.sum_post, g0 * per_gate + from, min(each, per_gate - from), a.cols, col);
        s = across_waves(s, lds);
        if (!writes) return;
        if (a.w_post.p != nullptr) s *= one(a.w_post, 0, col);
        grad1(a.dgate, g0, col, a.accumulate, a.alpha * s);
        return;
    }
    const Rows& dw = blockIdx.y == 0 ? a.dw_pre : a.dw_post;
    if (dw.p == nullptr) return;
    const int64_t each = (a.plan.units + kJoinWaves - 1) / kJoinWaves;
    int64_t u = min(a.plan.units, wave * each);
    const int64_t to = min(a.plan.units, u + each);
    float s = 0.0f;
    if (reads) {
        if (blockIdx.y == 0 || per_gate == 0) {
            s = column_sum(blockIdx.y == 0 ? a.sum_pre : a.sum_post, u, to - u, a.cols, col);
        } else {
            while (u < to) {  // the part of a gate row's units that is this wave's
                const int64_t g = u / per_gate, stop = min(to, (g + 1) * per_gate);
                const float t = column_sum(a.sum_post, u, stop - u, a.cols, col);
                s = fmaf(a.gate.p != nullptr ? a.alpha * one(a.gate, g, col) : a.alpha, t, s);
                u = stop;
            }
        }
    }
    s = across_waves(s, lds);
    if (writes) grad1(dw, 0, col, a.accumulate, s);
}

}  // namespace

// Threads of a workgroup that takes a row of nv vectors, V of them a lane.
static unsigned block_threads(int64_t nv, int per_lane) { return static_cast<unsigned>((nv + 64 * per_lane - 1) / (64 * per_lane) * 64); }

// Rows of one unit, so that all units together fill the chip once: as many
// workgroups of `waves` waves a compute unit as `room` waves of it allow.
static int64_t rows_a_unit(int64_t rows, int64_t waves, int64_t room)
{
    const int64_t units = kComputeUnits * (room > waves ? room / waves : 1);
    return (rows + units - 1) / units;
}

template <bool WAVE, int V>
static void norm_shape(NormArgs a, int64_t nv, hipStream_t s)
{
    const unsigned threads = WAVE ? 256 : block_threads(nv, V);
    a.unit_rows = rows_a_unit(a.rows, WAVE ? 1 : threads / 64, kRoomWaves);
    const int64_t units = (a.rows + a.unit_rows - 1) / a.unit_rows;
    const unsigned grid = static_cast<unsigned>(WAVE ? (units + 3) / 4 : units);
    if (a.x.f32) block_norm_kernel<WAVE, V, true><<<grid, threads, 0, s>>>(a);
    else block_norm_kernel<WAVE, V, false><<<grid, threads, 0, s>>>(a);
}

// The outputs go past the caches at any size: 16384 x 4096 and the decoding of
// its checkpoints 197 us instead of 223, 2048 x 4096 28.4 instead of 31.8, and
// never slower. x and y do when what a call moves is more than the 256 MiB
// Infinity Cache holds and their rows lie on 16 bytes. Read past the caches and
// through them, the decoding included: 16384 x 4096 197 us and 212, 8192 x 4096
// 94 and 103, 6144 x 4096 72 and 76, about what the cache holds; below that 4096
// x 4096 53 and 52 to 56, 2048 x 4096 32 and 30. 6000 x 5003, whose neighbouring
// loads share lines, 151 and 154 on one machine, 158 and 146 on another.
constexpr int64_t kInfinityCache = int64_t{256} << 20;

static bool streams_inputs(const NormArgs& a)
{
    const int64_t x = a.x.f32 ? 4 : 2;
    const int64_t column = x + (a.y.p != nullptr ? 2 + x : 0) + (a.h.p != nullptr ? 2 : 0) + (a.ckpt_post != nullptr) + (a.ckpt_pre != nullptr);
    return a.rows * a.cols * column > kInfinityCache && rows_on_16(a.x) && rows_on_16(a.y);
}

hipError_t launch_block_norm(const NormArgs& args, hipStream_t s)
{
    NormArgs a = args;
    a.stream = streams_inputs(a);
    const int64_t nv = act8_pitch(a.cols) / 8;
    // One vector a lane as long as a workgroup has the lanes: 8192 x 8192 with
    // both reads 213 us, 231 with two; 3001 x 5003 81 and 102. Wider rows have
    // nothing in flight across their sums: 8192 x 8192 146 us (4.6 TB/s),
    // 4096 x 12288 148 (3.4), 2048 x 16384 93 (3.6).
    if (nv <= kWaveVecs) norm_shape<true, 1>(a, nv, s);
    else if (nv <= kMaxLanes) norm_shape<false, 1>(a, nv, s);
    else norm_shape<false, 2>(a, nv, s);
    return hipGetLastError();
}

// ------------------------------------------------------------------ the backward pass's plan

// Rows wider than 6144 columns go in strips of 4096, in two passes over them;
// up to 8192 they still fit one workgroup if they come from 8 bits and there
// are few gate rows (otherwise its registers do not hold what it needs). The
// units are the same either way. From 8 bits and from rows as they are, in
// TB/s of what has to be read and written once: 16384 x 4096 152 and 233 us (4.4
// and 3.5), 8192 x 8192 162 and 422 (4.2 and 1.9), 4096 x 12288 215 and 310 (2.4
// and 2.0).
constexpr int kWideVecs = 768;
constexpr int kStripLanes = 512;

NormGradPlan norm_grad_plan(int64_t rows, int64_t cols, int64_t gate_rows)
{
    NormGradPlan p{};
    const int64_t nv = act8_pitch(cols) / 8;
    p.gate_rows = gate_rows > 0 && gate_rows < rows ? gate_rows : (rows > 0 ? rows : 1);
    p.gates = (rows + p.gate_rows - 1) / p.gate_rows;
    // Units of 16 waves a compute unit, of one workgroup of wide rows. Most of
    // the kernels have 129 to 168 registers, which let 12 waves run at once (more
    // registers 8, and 128 or fewer 16), so a large call goes in up to two rounds.
    // Planned for 16, 12 and 8 waves, from 8 bits: 16384 x 4096 145, 142 and 141
    // us, 65536 x 768 150, 118 and 142, 131072 x 512 166, 166 and 135, 3001 x 4096
    // in gates of 700 43, 38 and 38.
    const int64_t waves = (nv + 63) / 64;
    int64_t target = kComputeUnits * (waves > 8 ? 1 : waves > 0 ? 16 / waves : 16);
    if (nv > kWideVecs) {
        p.strips = (nv + kStripLanes - 1) / kStripLanes;
        target = kComputeUnits * 2 / p.strips;
    }
    // Whole gate rows a unit where they are more than the units: a little more
    // than target of them leave nearly half the units without rows. 16384 x 4096
    // from 8 bits: gates of 32 rows (512 units) 149 us, of 31 (265) 259, of 24
    // (342) 212, of 16 (512) 153; 3001 x 5003 gates of 12 rows (251) 70 us, of 11
    // (137) 95. Gates of one row 281 us, which read and write a gate for each.
    if (p.gates >= target) {
        p.unit_gates = (p.gates + target - 1) / target;
        p.units = (p.gates + p.unit_gates - 1) / p.unit_gates;
    } else if (p.gates > 0) {
        // The fewest rows a unit with which the units that have rows run at
        // once (more rows a unit never make more units): 9000 x 4096 in gates
        // of 2048 86 us, 95 with each gate row cut alike whatever the last has.
        const int64_t last = rows - (p.gates - 1) * p.gate_rows;
        int64_t least = (rows + target - 1) / target, most = p.gate_rows;
        while (least < most) {
            const int64_t r = least + (most - least) / 2;
            const int64_t units = (p.gates - 1) * ((p.gate_rows + r - 1) / r) + (last + r - 1) / r;
            if (units <= target) most = r;
            else least = r + 1;
        }
        p.unit_rows = most;
        p.per_gate = (p.gate_rows + p.unit_rows - 1) / p.unit_rows;
        // The last gate row may be short: its units past the end sum nothing.
        p.units = p.gates * p.per_gate;
    } else {
        p.per_gate = 1;
    }
    p.bytes = 2 * sizeof(float) * static_cast<size_t>(p.units * cols + (p.strips > 0 ? rows : 0));
    return p;
}

template <bool WAVE, int MAX, bool STRIP, bool F32, bool CODED>
static void grad_split(const NormGradArgs& a, int64_t nv, hipStream_t s)
{
    const unsigned groups = static_cast<unsigned>(WAVE ? (a.plan.units + 3) / 4 : a.plan.units);
    const dim3 grid(groups, STRIP ? static_cast<unsigned>(a.plan.strips) : 1);
    const unsigned threads = WAVE ? 256 : STRIP ? kStripLanes : block_threads(nv, 1);
    if constexpr (STRIP) {
        const unsigned rows = static_cast<unsigned>(a.rows < (1 << 20) ? a.rows : 1 << 20);
        block_norm_along_kernel<F32, CODED><<<rows, kMaxLanes, 0, s>>>(a);
    }
    if constexpr (MAX < kMaxLanes) {
        if (a.plan.per_gate == 0) {
            block_norm_grad_kernel<WAVE, MAX, F32, CODED, true, STRIP><<<grid, threads, 0, s>>>(a);
            return;
        }
    }
    block_norm_grad_kernel<WAVE, MAX, F32, CODED, false, STRIP><<<grid, threads, 0, s>>>(a);
}

template <bool WAVE, int MAX, bool STRIP>
static void grad_shape(const NormGradArgs& a, bool coded, int64_t nv, hipStream_t s)
{
    if constexpr (MAX < kMaxLanes) {
        if (!coded) {
            if (a.dx.f32) grad_split<WAVE, MAX, STRIP, true, false>(a, nv, s);
            else grad_split<WAVE, MAX, STRIP, false, false>(a, nv, s);
            return;
        }
    }
    if (a.dx.f32) grad_split<WAVE, MAX, STRIP, true, true>(a, nv, s);
    else grad_split<WAVE, MAX, STRIP, false, true>(a, nv, s);
}

hipError_t launch_block_norm_grad(const NormGradArgs& args, hipStream_t s)
{
    NormGradArgs a = args;
    a.stream = rows_on_16(a.dx) && rows_on_16(a.dy);
    if (a.plan.units > 0) {
        const int64_t nv = act8_pitch(a.cols) / 8;
        // rows that are not needed are neither coded nor read
        const bool coded = (a.ckpt_pre != nullptr || a.x_out.p == nullptr) && (a.ckpt_post != nullptr || a.y.p == nullptr);
        if (nv <= kWaveVecs) grad_shape<true, 256, false>(a, coded, nv, s);
        else if (nv <= 512) grad_shape<false, 512, false>(a, coded, nv, s);
        else if (nv <= kWideVecs) grad_shape<false, 768, false>(a, coded, nv, s);
        else if (nv <= kMaxLanes && coded && a.plan.per_gate > 0) grad_shape<false, kMaxLanes, false>(a, coded, nv, s);
        else grad_shape<false, kStripLanes, true>(a, coded, nv, s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.dw_pre.p == nullptr && a.dw_post.p == nullptr && (a.dgate.p == nullptr || a.plan.per_gate == 0))
        return hipSuccess;
    const int64_t step = join_gates(a.plan);
    const int64_t gates = a.dgate.p != nullptr && a.plan.per_gate > 0 ? (a.plan.gates + step - 1) / step : 0;
    const dim3 grid(static_cast<unsigned>((a.cols + 63) / 64), static_cast<unsigned>(2 + gates));
    block_norm_join_kernel<<<grid, 64 * kJoinWaves, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace zero
