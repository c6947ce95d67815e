// zero_layer_norm.hip -- the layer norm with the residual add before it, in one
// pass over the rows, and its backward pass, gfx950.
//
// A row stays in the registers of L lanes, V vectors of 8 columns a lane, so
// every operand is read once and every result written once. Both passes are
// streams, bound by HBM. Medians of nine launches and the least of them: 16384 x
// 4096 forward with x_out and 8 bits saved 114 and 108 us (606 MB, 5.3 and 5.6
// TB/s), backward from 8 bits 94 and 92 us (472 MB, 5.0 and 5.1 TB/s) and 5 to join
// the column sums; unaligned fp32 rows of 5003, backward, 58 and 56 us (240 MB, 4.1
// and 4.3 TB/s). Rows of more than 8192 columns have nothing in flight across a
// row's sums forward, and are read twice backward: 6000 x 11008 bf16 154 us a call
// (3.4 TB/s), backward 165 from 8 bits and 181 from rows (2.9). A short call is
// bound by its launch: 128 x 768 5.0 and 4.8 us.
#include "zero_norm_device.h"

namespace zero {
namespace {

// How many columns lie in the row from vector v on.
__device__ __forceinline__ int columns(int cols, int v, int nv) { return v < nv ? cols - 8 * v : 0; }

// A row's mean and its reciprocal root, in two parts each.
struct Moments {
    float mean, lo;
    Rstd rstd;
};

// The sum over the 16 lanes of a row of lanes, in all of them.
template <int CTRL>
__device__ __forceinline__ double add_moved(double x)
{
    const uint64_t bits = __builtin_bit_cast(uint64_t, x);
    const uint64_t moved = dpp<CTRL>(static_cast<uint32_t>(bits)) | static_cast<uint64_t>(dpp<CTRL>(static_cast<uint32_t>(bits >> 32))) << 32;
    return x + __builtin_bit_cast(double, moved);
}
__device__ __forceinline__ double sum_of_16(double x)
{
    static_assert(kMaxLanes / 64 <= 16, "a lane for every wave");
    return add_moved<kMirror>(add_moved<kHalfMirror>(add_moved<kQuadXor2>(add_moved<kQuadXor1>(x))));
}

// The moments of a row from what its lanes hold. A wave takes a first mean m of
// its own columns, and then, about m, the sum r (what m is off by) and the
// squares q of its columns. With the difference d of each m to the first
// wave's, a row's mean is m_0 + D / C, D = sum (count d + r), and its squares
// about that are sum q + 2 e r + count e^2, e = d - D / C: no step subtracts
// large sums, so a row of values far from 0 keeps its variance in fp32, and the
// waves meet once.
//
// Differences of bf16 values, which are coarse, to one m are all rounded the
// same way, and so is their sum. There m has 16 bits, whose multiples a lane's
// own sum (of few values: exact, but for values far below others) is compared
// with almost always exactly, and m itself is off by 2^-16, which adds little to
// the squares: bf16 rows of unequal values vary by 2^-15 of their mean and more.
// With that, the join of the waves in fp64 (a lane for each wave: no slower than
// one after the other in fp32) and ties settled, 0 to 4 of 67108864 values saved
// in e4m3 have another code than in 64 bits; 32 to 44 without.
template <bool WAVE, int V, bool F32>
__device__ __forceinline__ Moments moments(float (&x)[V][8], int lane, int lanes, int cols, int nv, double inv_cols, float eps,
                                           f32x4 (*red)[kMaxLanes / 64], int& half)
{
    float own = 0.0f;
    int own_count = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        own += ((x[j][0] + x[j][1]) + (x[j][2] + x[j][3])) + ((x[j][4] + x[j][5]) + (x[j][6] + x[j][7]));
        own_count += min(max(columns(cols, lane + j * lanes, nv), 0), 8);
    }
    const float s = wave_sum(own);
    const int wave = WAVE ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const auto count_of = [&](int w) {
        int count = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) count += min(max(cols - 8 * (w * 64 + j * lanes), 0), 512);
        return static_cast<float>(count);
    };
    float m = s * __builtin_amdgcn_rcpf(count_of(wave));  // of at least one column
    if constexpr (!F32) m = __uint_as_float(__float_as_uint(m) & 0xFFFFFF00u);
    float r = F32 ? 0.0f : fmaf(-static_cast<float>(own_count), m, own), q = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int n = columns(cols, lane + j * lanes, nv);
        if (n < 8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[j][i] = i < n ? x[j][i] : m;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float c = x[j][i] - m;
            if constexpr (F32) r += c;
            q = fmaf(c, c, q);
        }
    }
    r = wave_sum(r);
    q = wave_sum(q);
    // Joined in fp64: D is a small sum of terms as large as the waves' means lie apart. (Each d itself is an fp32
    // difference, off by 2^-24 of how far the two waves lie apart: no more than the squares about it bear.)
    float first = m;
    double step, squares;
    if constexpr (WAVE) {
        step = r * inv_cols;
        squares = fma(-step, static_cast<double>(r), static_cast<double>(q));
    } else {
        if (threadIdx.x % 64 == 0) red[half][wave] = f32x4{m, r, q, 0.0f};
        __syncthreads();
        first = red[half][0].x;
        const int w = threadIdx.x % 16;  // each lane takes a wave's part
        const bool there = w < static_cast<int>(blockDim.x / 64);
        const f32x4 t = red[half][there ? w : 0];
        const double count = there ? count_of(w) : 0.0f, off = t.x - first, rest = t.y;
        step = sum_of_16(there ? fma(count, off, rest) : 0.0) * inv_cols;
        const double e = off - step;
        squares = sum_of_16(there ? fma(e, fma(count, e, 2.0 * rest), static_cast<double>(t.z)) : 0.0);
        half ^= 1;
    }
    Moments out;
    const double mean = first + step;
    out.mean = static_cast<float>(mean);
    out.lo = static_cast<float>(mean - out.mean);
    // all columns alike may leave less than nothing
    out.rstd = row_rstd(squares < 0.0 ? 0.0 : squares, inv_cols, eps);
    return out;
}

// A workgroup (or wave) takes neighbouring rows. At V == 1 a lane keeps its
// columns' weight and bias in registers, and the next row's loads are started
// before this row's sums.
template <bool WAVE, int V, bool F32>
__global__ __launch_bounds__(WAVE ? 256 : kMaxLanes) void layer_norm_kernel(LayerNormArgs a)
{
    constexpr bool kEarly = V == 1;
    __shared__ f32x4 red[2][kMaxLanes / 64];
    int half = 0;
    const int lane = row_lane<WAVE>(), lanes = row_lanes<WAVE>();
    const int nv = static_cast<int>(act8_pitch(a.cols) / 8);
    const int64_t pitch = 8 * static_cast<int64_t>(nv);
    const double inv_cols = 1.0 / a.cols;
    const bool has_y = a.y.p != nullptr;
    int64_t row = row_slot<WAVE>() * a.unit_rows;
    const int64_t end = min(a.rows, row + a.unit_rows);
    if (row >= end) return;  // whole waves, and none where there are barriers
    Raw8<F32> next_x[V];
    Raw8<false> next_y[V];
    const auto load = [&](int64_t r) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int v = lane + j * lanes, n = columns(a.cols, v, nv);
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
    float w[8], b[8];
    const auto affine = [&](int v, int n) {
        if (a.w.p != nullptr) load8_any(a.w, 0, 8 * v, n, w);
        if (a.b.p != nullptr) load8_any(a.b, 0, 8 * v, n, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (a.w.p == nullptr) w[i] = 1.0f;
            if (a.b.p == nullptr) b[i] = 0.0f;
        }
    };
    if (kEarly) {
        load(row);
        affine(lane, columns(a.cols, lane, nv));
    }
    for (; row < end; ++row) {
        if (!kEarly) load(row);
        float x[V][8];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int v = lane + j * lanes, n = columns(a.cols, v, nv);
            unpack<F32>(next_x[j], 8 * v, n, x[j]);
            if (has_y) {
                float y[8];
                unpack<false>(next_y[j], 8 * v, n, y);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[j][i] += y[i];
                if (n > 0) store8<F32, true>(a.x_out, row, 8 * v, n, x[j]);
                // the norm below is that of the residual stream as stored
                if constexpr (!F32) round_bf16(x[j]);
            }
        }
        if (kEarly && row + 1 < end) load(row + 1);
        const Moments m = moments<WAVE, V, F32>(x, lane, lanes, a.cols, nv, inv_cols, a.eps, red, half);
        if (lane == 0) {
            if (a.mean != nullptr) ((ZERO_G float*)a.mean)[row] = m.mean;
            if (a.rstd != nullptr) ((ZERO_G float*)a.rstd)[row] = m.rstd.hi;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int v = lane + j * lanes, n = a.cols - 8 * v;
            if (v >= nv) continue;
            if (!kEarly) affine(v, n);
            float xn[8], h[8];
            // the difference and the root in two parts: rounded once, so that its 8-bit code is seldom another
            const auto small = [&](int i, float c) { return fmaf(c, m.rstd.lo, (((x[j][i] - c) - m.mean) - m.lo) * m.rstd.hi); };
            uint32_t least = ~0u;  // of the values' last 16 bits
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float c = x[j][i] - m.mean;
                xn[i] = i < n ? fmaf(c, m.rstd.hi, small(i, c)) : 0.0f;
                least = min(least, __float_as_uint(xn[i]) & 0xFFFFu);
            }
            if (least == 0) {
                // What was rounded to the middle between two codes goes to the side that it came from. (Also where no
                // codes are saved: what a call computes does not depend on what it saves.)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t bits = __float_as_uint(xn[i]);
                    const float c = x[j][i] - m.mean, off = (fmaf(c, m.rstd.hi, -xn[i]) + small(i, c)) * xn[i];
                    const uint32_t step = off > 0.0f ? 1u : off < 0.0f ? ~0u : 0u;  // none for a NaN, and for what is exact
                    if ((bits & 0xFFFFu) == 0) xn[i] = __uint_as_float(bits + step);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = fmaf(w[i], xn[i], b[i]);
            if (a.ckpt_xn != nullptr) save8(a.ckpt_xn, a.rows, pitch, a.format, row, v, xn);
            if (a.ckpt_h != nullptr) save8(a.ckpt_h, a.rows, pitch, a.format, row, v, h);
            store8<false, true>(a.h, row, 8 * v, n, h);
        }
    }
}

// ------------------------------------------------------------------ backward

// What a lane reads of a row.
template <bool F32, bool CODED>
struct NormRow {
    Raw8<false> dh;
    Raw8<F32> x;  // unless CODED
    u32x2 codes;
    uint32_t scale;
    float mean, rstd;
};

template <bool F32, bool CODED>
__device__ __forceinline__ NormRow<F32, CODED> load_row(const LayerNormGradArgs& a, int64_t pitch, int64_t row, int v, int n)
{
    NormRow<F32, CODED> r{};
    r.rstd = ((const ZERO_G float*)a.rstd)[row];
    if constexpr (!CODED) r.mean = ((const ZERO_G float*)a.mean)[row];
    r.dh = load8<false>(a.dh, row, 8 * v, n);
    if constexpr (CODED) {
        if (n > 0) {
            r.codes = ld_codes(a.ckpt_xn + code_at(row, pitch, v));
            r.scale = ld_scale(a.ckpt_xn + a.rows * pitch + scale_at(row, pitch, v));
        }
    } else {
        r.x = load8<F32>(a.x_out, row, 8 * v, n);
    }
    return r;
}
// xn of 8 columns, 0 from column n on.
template <bool F32, bool CODED>
__device__ __forceinline__ void saved_xn(const NormRow<F32, CODED>& r, int format, int v, int n, float (&xn)[8])
{
    if constexpr (CODED) {
        if (format == ZERO_ACT8_E4M3) decode8<ZERO_ACT8_E4M3>(r.codes, r.scale, xn);
        else decode8<ZERO_ACT8_INT8>(r.codes, r.scale, xn);
        if (n < 8) {  // a block of NaN has them beyond the row too
#pragma unroll
            for (int i = 0; i < 8; ++i) xn[i] = i < n ? xn[i] : 0.0f;
        }
    } else {
        unpack<F32>(r.x, 8 * v, n, xn);
#pragma unroll
        for (int i = 0; i < 8; ++i) xn[i] = i < n ? (xn[i] - r.mean) * r.rstd : 0.0f;
    }
}

// mean(t) and mean(t xn) of a row, t = w dh, from sums that do not wait for each other.
template <bool F32, bool CODED>
__device__ __forceinline__ void add_row(const NormRow<F32, CODED>& r, int format, int v, int n, const float (&w)[8], float (&t)[8],
                                        float (&xn)[8], float (&s)[2], float (&sum_w)[8], float (&sum_b)[8])
{
    saved_xn<F32, CODED>(r, format, v, n, xn);
    unpack<false>(r.dh, 8 * v, n, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        sum_w[i] = fmaf(t[i], xn[i], sum_w[i]);
        sum_b[i] += t[i];
        t[i] *= w[i];
        s[0] += t[i];
        s[1] = fmaf(t[i], xn[i], s[1]);
    }
}

__device__ __forceinline__ void load_weights(const Rows& m, int v, int n, float (&w)[8])
{
    if (m.p != nullptr) {
        load8_any(m, 0, 8 * v, n, w);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.0f;
}

// The two means of each row alone, for rows too wide for one workgroup's
// registers: they are then read twice.
template <bool F32, bool CODED>
__global__ __launch_bounds__(kMaxLanes) void layer_norm_along_kernel(LayerNormGradArgs a)
{
    __shared__ float red[2][2][kMaxLanes / 64];
    int half = 0;
    const int nv = static_cast<int>(act8_pitch(a.cols) / 8);
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float s[2] = {0.0f, 0.0f}, unused[8] = {}, w[8], t[8], xn[8];
        for (int v = threadIdx.x; v < nv; v += kMaxLanes) {
            const int n = a.cols - 8 * v;
            load_weights(a.w, v, n, w);
            add_row(load_row<F32, CODED>(a, 8 * static_cast<int64_t>(nv), row, v, n), a.format, v, n, w, t, xn, s, unused, unused);
        }
        row_sum<false, 2>(s, red, half);
        if (threadIdx.x == 0) *(ZERO_G f32x2*)(a.row_means + 2 * row) = f32x2{s[0] * inv_cols, s[1] * inv_cols};
    }
}

// A lane keeps 8 columns: their weights and their column sums in registers
// over all rows of its unit. The next row's loads are started before this
// row's sums, so that they are in flight across its barrier.
//
// STRIP: the means come from layer_norm_along_kernel, and a workgroup takes
// one strip (blockIdx.y) of its unit's columns.
template <bool WAVE, int MAX, bool F32, bool CODED, bool STRIP>
__global__ __launch_bounds__(MAX) void layer_norm_grad_kernel(LayerNormGradArgs a)
{
    __shared__ float red[2][2][kMaxLanes / 64];
    int half = 0;
    const int v = row_lane<WAVE>() + (STRIP ? static_cast<int>(blockIdx.y * blockDim.x) : 0);
    const int64_t unit = row_slot<WAVE>();
    if (unit >= a.plan.units) return;  // whole waves, and none where there are barriers
    const int nv = static_cast<int>(act8_pitch(a.cols) / 8);
    const int64_t pitch = 8 * static_cast<int64_t>(nv);
    const int n = columns(a.cols, v, nv);
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    int64_t row = unit * a.plan.unit_rows;
    const int64_t end = min(a.rows, row + a.plan.unit_rows);
    float sum_w[8] = {}, sum_b[8] = {}, w[8];
    load_weights(a.w, v, n, w);
    NormRow<F32, CODED> next{};
    Raw8<F32> next_d{};
    f32x2 next_means{};
    const auto load = [&](int64_t r) {
        next = load_row<F32, CODED>(a, pitch, r, v, n);
        if (a.dx_out.p != nullptr) next_d = load8<F32>(a.dx_out, r, 8 * v, n);
        if constexpr (STRIP) next_means = *(const ZERO_G f32x2*)(a.row_means + 2 * r);
    };
    if (row < end) load(row);
    for (; row < end; ++row) {
        float t[8], xn[8], d[8], s[2] = {0.0f, 0.0f};
        const float rstd = next.rstd;
        const f32x2 means = next_means;
        add_row(next, a.format, v, n, w, t, xn, s, sum_w, sum_b);
        unpack<F32>(next_d, 8 * v, n, d);
        if (row + 1 < end) load(row + 1);
        float mean = means.x, along = means.y;
        if constexpr (!STRIP) {
            row_sum<WAVE, 2>(s, red, half);
            mean = s[0] * inv_cols;
            along = s[1] * inv_cols;
        }
        if (v >= nv) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = fmaf(rstd, fmaf(-along, xn[i], t[i] - mean), d[i]);
        if (a.stream != 0) store8<F32, true>(a.dx, row, 8 * v, n, d);
        else store8<F32>(a.dx, row, 8 * v, n, d);
        if (a.dy.p != nullptr) {
            if (a.stream != 0) store8<false, true>(a.dy, row, 8 * v, n, d);
            else store8<false>(a.dy, row, 8 * v, n, d);
        }
    }
    if (v >= nv) return;
    const Rows to_w{a.sum_w, a.cols, 1}, to_b{a.sum_b, a.cols, 1};
    if (a.dw.p != nullptr) store8<true>(to_w, unit, 8 * v, n, sum_w);
    if (a.db.p != nullptr) store8<true>(to_b, unit, 8 * v, n, sum_b);
}

// The units' sums joined in order: 64 columns a workgroup, its 16 waves each a
// sixteenth of the units; blockIdx.y 0 makes dw, 1 db.
__global__ __launch_bounds__(64 * kJoinWaves) void layer_norm_join_kernel(LayerNormGradArgs a)
{
    __shared__ float lds[64 * kJoinWaves];
    const int col = blockIdx.x * 64 + threadIdx.x % 64;
    const int64_t wave = threadIdx.x / 64;
    const Rows& to = blockIdx.y == 0 ? a.dw : a.db;
    if (to.p == nullptr) return;
    const int64_t each = (a.plan.units + kJoinWaves - 1) / kJoinWaves;
    const int64_t from = min(a.plan.units, wave * each), until = min(a.plan.units, from + each);
    float s = 0.0f;
    if (col < a.cols) s = column_sum(blockIdx.y == 0 ? a.sum_w : a.sum_b, from, until - from, a.cols, col);
    s = across_waves(s, lds);
    if (col < a.cols && wave == 0) grad1(to, 0, col, a.accumulate, s);
}

template <bool WAVE, int V>
void norm_shape(LayerNormArgs a, int64_t nv, hipStream_t s)
{
    const unsigned threads = WAVE ? 256 : block_threads(nv, V);
    a.unit_rows = rows_a_unit(a.rows, WAVE ? 1 : threads / 64, kRoomWaves);
    const int64_t units = (a.rows + a.unit_rows - 1) / a.unit_rows;
    const unsigned grid = static_cast<unsigned>(WAVE ? (units + 3) / 4 : units);
    if (a.x.f32) layer_norm_kernel<WAVE, V, true><<<grid, threads, 0, s>>>(a);
    else layer_norm_kernel<WAVE, V, false><<<grid, threads, 0, s>>>(a);
}

template <bool WAVE, int MAX, bool STRIP, bool F32, bool CODED>
void grad_rows(const LayerNormGradArgs& a, int64_t nv, hipStream_t s)
{
    const unsigned groups = static_cast<unsigned>(WAVE ? (a.plan.units + 3) / 4 : a.plan.units);
    const dim3 grid(groups, STRIP ? static_cast<unsigned>((nv + MAX - 1) / MAX) : 1);
    if constexpr (STRIP) {
        const unsigned rows = static_cast<unsigned>(a.rows < (1 << 20) ? a.rows : 1 << 20);
        layer_norm_along_kernel<F32, CODED><<<rows, kMaxLanes, 0, s>>>(a);
    }
    layer_norm_grad_kernel<WAVE, MAX, F32, CODED, STRIP><<<grid, WAVE || STRIP ? MAX : block_threads(nv, 1), 0, s>>>(a);
}

template <bool WAVE, int MAX, bool STRIP>
void grad_shape(const LayerNormGradArgs& a, int64_t nv, hipStream_t s)
{
    if (a.ckpt_xn != nullptr) {
        if (a.dx.f32) grad_rows<WAVE, MAX, STRIP, true, true>(a, nv, s);
        else grad_rows<WAVE, MAX, STRIP, false, true>(a, nv, s);
    } else {
        if (a.dx.f32) grad_rows<WAVE, MAX, STRIP, true, false>(a, nv, s);
        else grad_rows<WAVE, MAX, STRIP, false, false>(a, nv, s);
    }
}

// Inputs are read past the caches when a call moves more than the Infinity
// Cache holds and their rows lie on 16 bytes.
bool streams_inputs(const LayerNormArgs& a)
{
    const int64_t x = a.x.f32 ? 4 : 2;
    const int64_t column = x + (a.y.p != nullptr ? 2 + x : 0) + 2 + (a.ckpt_xn != nullptr) + (a.ckpt_h != nullptr);
    return a.rows * a.cols * column > kInfinityCache && rows_on_16(a.x) && rows_on_16(a.y);
}

}  // namespace

hipError_t launch_layer_norm(const LayerNormArgs& args, hipStream_t s)
{
    LayerNormArgs a = args;
    a.stream = streams_inputs(a);
    const int64_t nv = act8_pitch(a.cols) / 8;
    if (nv <= kWaveVecs) norm_shape<true, 1>(a, nv, s);
    else if (nv <= kMaxLanes) norm_shape<false, 1>(a, nv, s);
    else norm_shape<false, 2>(a, nv, s);
    return hipGetLastError();
}

// Rows wider than 8192 columns go in strips of 4096, in two passes over them.
constexpr int kStripLanes = 512;

LayerNormGradPlan layer_norm_grad_plan(int64_t rows, int64_t cols)
{
    LayerNormGradPlan p{};
    const int64_t nv = act8_pitch(cols) / 8;
    p.strips = nv > kMaxLanes;
    const int64_t waves = p.strips ? (nv + kStripLanes - 1) / kStripLanes * (kStripLanes / 64) : (nv + 63) / 64;
    p.unit_rows = rows_a_unit(rows, waves > 0 ? waves : 1, kRoomWaves);
    p.units = p.unit_rows > 0 ? (rows + p.unit_rows - 1) / p.unit_rows : 0;
    p.bytes = 2 * sizeof(float) * static_cast<size_t>(p.units * cols + (p.strips ? rows : 0));
    return p;
}

hipError_t launch_layer_norm_grad(const LayerNormGradArgs& args, hipStream_t s)
{
    LayerNormGradArgs a = args;
    a.stream = rows_on_16(a.dx) && rows_on_16(a.dy);
    if (a.plan.units > 0) {
        const int64_t nv = act8_pitch(a.cols) / 8;
        if (nv <= kWaveVecs) grad_shape<true, 256, false>(a, nv, s);
        else if (nv <= 512) grad_shape<false, 512, false>(a, nv, s);
        else if (nv <= kMaxLanes) grad_shape<false, kMaxLanes, false>(a, nv, s);
        else grad_shape<false, kStripLanes, true>(a, nv, s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.dw.p == nullptr && a.db.p == nullptr) return hipSuccess;
    layer_norm_join_kernel<<<dim3(static_cast<unsigned>((a.cols + 63) / 64), 2), 64 * kJoinWaves, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace zero
