// zero_norm_device.h -- what the kernels of the norms share: rows in the
// registers of a wave or workgroup, their sums, gradients written or added to,
// and column sums joined over units.
#pragma once

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

// The waves of a join's workgroup.
constexpr int kJoinWaves = 16;

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

// Threads of a workgroup that takes a row of nv vectors, V of them a lane.
inline unsigned block_threads(int64_t nv, int per_lane) { return static_cast<unsigned>((nv + 64 * per_lane - 1) / (64 * per_lane) * 64); }

// Rows of one unit, so that all units together fill the chip once: as many
// workgroups of `waves` waves a compute unit as `room` waves of it allow.
inline int64_t rows_a_unit(int64_t rows, int64_t waves, int64_t room)
{
    const int64_t units = kComputeUnits * (room > waves ? room / waves : 1);
    return (rows + units - 1) / units;
}

// What a call may move before its lines push each other out of the Infinity Cache.
constexpr int64_t kInfinityCache = int64_t{256} << 20;

}  // namespace
}  // namespace zero
