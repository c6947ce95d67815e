// zero_act8_device.h -- device helpers shared by the kernels around a training
// block: 8-element loads and stores at any alignment, reductions, and the
// 8-bit form of 32 columns (four neighbouring lanes, 8 columns each).
#pragma once

#include <hip/hip_runtime.h>

#include "zero_block.h"

namespace zero {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Operands are device memory: global_* instructions, which do not wait on
// the LDS counter. The types carry the element alignment only; gfx950 takes a
// 16-byte access at any 2-byte address.
#define ZERO_G __attribute__((address_space(1)))
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));

// STREAM: a line that this kernel does not touch again should not displace
// others from the caches.
template <bool STREAM, class T>
__device__ __forceinline__ u32x4 ld16_as(const void* p)
{
    if constexpr (STREAM) return __builtin_nontemporal_load((const ZERO_G T*)p);
    else return *(const ZERO_G T*)p;
}
template <bool STREAM, class T>
__device__ __forceinline__ void st16_as(void* p, u32x4 v)
{
    if constexpr (STREAM) __builtin_nontemporal_store(v, (ZERO_G T*)p);
    else *(ZERO_G T*)p = v;
}
template <bool STREAM = false>
__device__ __forceinline__ u32x4 ld16_a2(const void* p) { return ld16_as<STREAM, u32x4_a2>(p); }
template <bool STREAM = false>
__device__ __forceinline__ u32x4 ld16_a4(const void* p) { return ld16_as<STREAM, u32x4_a4>(p); }
template <bool STREAM = false>
__device__ __forceinline__ void st16_a2(void* p, u32x4 v) { st16_as<STREAM, u32x4_a2>(p, v); }
template <bool STREAM = false>
__device__ __forceinline__ void st16_a4(void* p, u32x4 v) { st16_as<STREAM, u32x4_a4>(p, v); }

// Eight values as loaded: bf16 in one 16-byte load, fp32 in two.
template <bool F32>
struct Raw8 {
    u32x4 v[F32 ? 2 : 1];
};

// Where column `col` of a row lies: what all lanes of a row share, and a 32-bit
// offset (cols < 2^30), which together are one addressing mode.
template <bool F32>
__device__ __forceinline__ char* row_at(const Rows& m, int64_t row, int col)
{
    constexpr int kSize = F32 ? 4 : 2;
    return static_cast<char*>(m.p) + row * m.ld * kSize + static_cast<uint32_t>(col) * kSize;
}

// A row's last vector may have only n < 8 elements. It is read as the 8
// elements that end with the row, so that its load is like the others and
// waits for nothing, and moved into place when it is unpacked.
__device__ __forceinline__ int back(int col, int n) { return n > 0 && n < 8 && col > 0 ? 8 - n : 0; }

// Eight elements of a row from column col, to be unpacked with the same col
// and n; elements from `n` on are not read.
template <bool F32, bool STREAM = false>
__device__ __forceinline__ Raw8<F32> load8(const Rows& m, int64_t row, int col, int n)
{
    Raw8<F32> r{};
    const char* p = row_at<F32>(m, row, col - back(col, n));
    if (n >= 8 || (n > 0 && col > 0)) {
        if constexpr (F32) {
            r.v[0] = ld16_a4<STREAM>(p);
            r.v[1] = ld16_a4<STREAM>(p + 16);
        } else {
            r.v[0] = ld16_a2<STREAM>(p);
        }
    } else if (n > 0) {  // the row has fewer than 8 columns
#pragma unroll
        for (int i = 0; i < 7; ++i) {
            if (i >= n) continue;
            if constexpr (F32) r.v[i / 4][i % 4] = ((const ZERO_G uint32_t*)p)[i];
            else r.v[0][i / 2] |= static_cast<uint32_t>(((const ZERO_G uint16_t*)p)[i]) << (16 * (i % 2));
        }
    }
    return r;
}

// What load8 read, as fp32; zeros from element `n` on.
template <bool F32>
__device__ __forceinline__ void unpack(const Raw8<F32>& r, int col, int n, float (&f)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (F32) f[i] = __uint_as_float(r.v[i / 4][i % 4]);
        else f[i] = __uint_as_float(i % 2 ? r.v[0][i / 2] & 0xFFFF0000u : r.v[0][i / 2] << 16);
    }
    for (int k = back(col, n); k > 0; --k) {  // one lane of a row at most
#pragma unroll
        for (int i = 0; i < 7; ++i) f[i] = f[i + 1];
        f[7] = 0.0f;
    }
}

// Eight elements of a vector or gate row of either type, as fp32.
__device__ __forceinline__ void load8_any(const Rows& m, int64_t row, int col, int n, float (&f)[8])
{
    if (m.f32) unpack<true>(load8<true>(m, row, col, n), col, n, f);
    else unpack<false>(load8<false>(m, row, col, n), col, n, f);
}

// Two fp32 values to bf16, nearest even (one instruction on gfx950).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const bf16x2 v = __builtin_convertvector(f32x2{lo, hi}, bf16x2);
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ u32x4 pack8(const float (&f)[8])
{
    return u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
}

// Eight values rounded to bf16, as fp32.
__device__ __forceinline__ void round_bf16(float (&f)[8])
{
    const u32x4 v = pack8(f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(i % 2 ? v[i / 2] & 0xFFFF0000u : v[i / 2] << 16);
}

// The first n of eight values to p, rounded to bf16 or as they are.
template <bool F32, bool STREAM = false>
__device__ __forceinline__ void store8(const Rows& m, int64_t row, int col, int n, const float (&f)[8])
{
    if constexpr (F32) {
        char* p = row_at<true>(m, row, col);
        if (n >= 8) {
            st16_a4<STREAM>(p, __builtin_bit_cast(u32x4, f32x4{f[0], f[1], f[2], f[3]}));
            st16_a4<STREAM>(p + 16, __builtin_bit_cast(u32x4, f32x4{f[4], f[5], f[6], f[7]}));
        } else {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < n) ((ZERO_G float*)p)[i] = f[i];
        }
    } else {
        char* p = row_at<false>(m, row, col);
        const u32x4 v = pack8(f);
        if (n >= 8) {
            st16_a2<STREAM>(p, v);
        } else {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < n) ((ZERO_G uint16_t*)p)[i] = static_cast<uint16_t>(v[i / 2] >> (16 * (i & 1)));
        }
    }
}

// ------------------------------------------------------------------ reductions

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x)
{
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), CTRL, 0xF, 0xF, true));
}
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

// The sum over a wave, in every lane, always in the same order.
__device__ __forceinline__ float wave_sum(float x)
{
    x += __uint_as_float(dpp<kQuadXor1>(__float_as_uint(x)));
    x += __uint_as_float(dpp<kQuadXor2>(__float_as_uint(x)));
    x += __uint_as_float(dpp<kHalfMirror>(__float_as_uint(x)));
    x += __uint_as_float(dpp<kMirror>(__float_as_uint(x)));
    x += __shfl_xor(x, 16);
    x += __shfl_xor(x, 32);
    return x;
}

// The largest of the four lanes of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t x)
{
    x = max(x, dpp<kQuadXor1>(x));
    return max(x, dpp<kQuadXor2>(x));
}

// ------------------------------------------------------------------ the 8-bit form

struct Code8 {
    u32x2 codes;
    uint32_t scale;  // k + 127, or 255
};

// This lane's 8 of a block of 32 values held by a quad. The bit patterns of
// |x| order like their values, with inf and NaN above every finite one, so one
// integer maximum finds both the largest value and whether the block is
// finite; its exponent field, carried over when its mantissa is above F's,
// gives the smallest k with max <= F * 2^k without a logarithm. A block that
// is not finite gets codes 0 and the scale that makes NaN of any code.
template <int FMT>
__device__ __forceinline__ Code8 encode8(const float (&x)[8])
{
    constexpr uint32_t kOver = FMT == ZERO_ACT8_E4M3 ? 0x1FFFFF : 0x01FFFF;  // 2^23 - 1 - mantissa(F)
    constexpr int kTop = FMT == ZERO_ACT8_E4M3 ? 8 : 6;                      // exponent of F
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    top = quad_max(top);
    const bool fine = top < 0x7F800000u;
    const int k = max(static_cast<int>((top + kOver) >> 23) - (127 + kTop), kActMinExp);
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = x[i] * inv;
    Code8 r;
    if constexpr (FMT == ZERO_ACT8_E4M3) {
        int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
        int hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
        r.codes = u32x2{static_cast<uint32_t>(lo), static_cast<uint32_t>(hi)};
    } else {
        // adding 1.5 * 2^23 rounds to an integer, nearest even, and leaves its
        // two's complement in the low bits
        uint32_t b[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(v[i] + 12582912.0f);
        const auto bytes = [&](int i) {
            const uint32_t p = __builtin_amdgcn_perm(b[i + 1], b[i], 0x0C0C0400u);
            const uint32_t q = __builtin_amdgcn_perm(b[i + 3], b[i + 2], 0x0C0C0400u);
            return p | (q << 16);
        };
        r.codes = u32x2{bytes(0), bytes(4)};
    }
    if (!fine) r.codes = u32x2{0, 0};
    r.scale = fine ? static_cast<uint32_t>(k + 127) : 255u;
    return r;
}

// 2^k of a scale byte as fp32; 255 is NaN.
__device__ __forceinline__ float act8_unit(uint32_t scale)
{
    return __uint_as_float(scale == 255u ? 0x7FC00000u : scale << 23);
}

template <int FMT>
__device__ __forceinline__ void decode8(u32x2 codes, uint32_t scale, float (&f)[8])
{
    const float unit = act8_unit(scale);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if constexpr (FMT == ZERO_ACT8_E4M3) {
            // two codes and their scale an instruction; a NaN scale gives NaN
            const f32x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes[h], unit, false);
            const f32x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes[h], unit, true);
            f[4 * h + 0] = lo.x;
            f[4 * h + 1] = lo.y;
            f[4 * h + 2] = hi.x;
            f[4 * h + 3] = hi.y;
        } else {
            const int w = static_cast<int>(codes[h]);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[4 * h + i] = static_cast<float>((w << (24 - 8 * i)) >> 24) * unit;
        }
    }
}

// Where the 8 columns of vector v (columns 8v ..) of a row lie in an act8 buffer.
__device__ __forceinline__ int64_t code_at(int64_t row, int64_t pitch, int v) { return row * pitch + static_cast<uint32_t>(8 * v); }
__device__ __forceinline__ int64_t scale_at(int64_t row, int64_t pitch, int v) { return row * (pitch / kActBlock) + static_cast<uint32_t>(v) / 4; }

__device__ __forceinline__ u32x2 ld_codes(const uint8_t* p) { return *(const ZERO_G u32x2*)p; }
__device__ __forceinline__ uint32_t ld_scale(const uint8_t* p) { return *(const ZERO_G uint8_t*)p; }

__device__ __forceinline__ uint32_t div_by(uint32_t n, FastDiv d) { return (__umulhi(n, d.mul) + n) >> d.shift; }

}  // namespace
}  // namespace zero
