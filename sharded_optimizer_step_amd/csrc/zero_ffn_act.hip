// zero_ffn_act.hip -- the activation of the gated feed-forward block backwards:
// dgate = da up act'(gate) and dup = da act(gate) from the saved gate and up, and
// act(gate) up again in 8 bits, gfx950.
//
// A stream, 8 columns a lane, visited as one list of vectors like the 8-bit
// rows. What is summed from dgate and dup later is held in fp32, where one of
// them that is rounded to the wrong bf16 neighbour counts for 2^-8. So they are
// the nearest bf16 values of the formulas: each is computed in fp32 with a
// bound on its error, and where the bf16 value is not the same on both sides
// of that, in fp64. One in about a thousand is.
//
// Bound by HBM and the fp32 form together: 8192 x 11008 from 8 bits 168 us in the
// median and 160 at the least, 727 MB at 4.3 and 4.5 TB/s (219 with one kernel for
// all activations and the two gradients' roundings checked one after the other);
// the error function's form 28.1 and 27.6 us for 2011 x 2731 (44 MB), where erfcf's
// instructions take most of the time.
#include "zero_act8_device.h"

namespace zero {
namespace {

constexpr int kThreads = 256;
constexpr float kUnit = 0x1p-24f;  // half a step of fp32, relative

// act(g) = g p and act'(g) in fp32, within slack_f of itself and slack_d.
struct Terms {
    float f, d, slack_f, slack_d;
    bool sure;  // the bounds hold
};

// The bounds count units of 2^-24: one for an operation, two for the
// instructions of the exponential and the reciprocal, and what the rounding of
// the exponent's argument adds, its size.
template <int ACT>
__device__ __forceinline__ Terms terms(float g)
{
    const float size = fabsf(g);
    Terms t;
    if constexpr (ACT == ZERO_FFN_GELU) {
        // p = erfc(-g / sqrt 2) / 2, within 32 units and 1.5 g^2 of its argument's
        const float p = 0.5f * erfcf(g * -0.70710678f), bell = 0.39894228f * __builtin_amdgcn_exp2f(g * g * -0.72134752f);
        t.f = g * p;
        t.d = fmaf(g, bell, p);
        t.slack_f = fmaf(g * g, 2.0f * kUnit, 40.0f * kUnit);
        t.slack_d = fmaf(size, bell, p) * fmaf(g * g, 2.0f * kUnit, 44.0f * kUnit);
        t.sure = size < 12.0f;
        return t;
    }
    float z = g, steep = g;  // act(g) = g logistic(z), steep = g z'
    if constexpr (ACT == ZERO_FFN_GELU_TANH) {
        z = 1.59576912f * fmaf(0.044715f * g * g, g, g);
        steep = g * fmaf(0.214064449f * g, g, 1.59576912f);
    }
    const float e = __builtin_amdgcn_exp2f(z * -1.44269504f), p = __builtin_amdgcn_rcpf(1.0f + e);
    const float pull = steep * (e * p);
    t.f = g * p;
    t.d = fmaf(p, pull, p);
    // (z itself is within 5 units of the exact one)
    constexpr float kOfZ = ACT == ZERO_FFN_SILU ? 1.5f * kUnit : 7.0f * kUnit;
    t.slack_f = fmaf(fabsf(z), kOfZ, 8.0f * kUnit);
    t.slack_d = fmaf(p, fabsf(pull), p) * fmaf(fabsf(z), 3.0f * kOfZ, 24.0f * kUnit);
    t.sure = fabsf(z) < 80.0f;
    return t;
}

// The same in fp64.
template <int ACT>
__device__ __forceinline__ void terms64(double g, double& f, double& d)
{
    if constexpr (ACT == ZERO_FFN_GELU) {
        const double p = 0.5 * erfc(g * -0.70710678118654752);
        f = g * p;
        d = fma(g, 0.39894228040143268 * exp(-0.5 * g * g), p);
        return;
    }
    double z = g, steep = g;
    if constexpr (ACT == ZERO_FFN_GELU_TANH) {
        z = 1.5957691216057308 * (g + 0.044715 * g * g * g);
        steep = 1.5957691216057308 * g * (1.0 + 0.134145 * g * g);
    }
    // p = 1 / (1 + e) and q = 1 - p = e / (1 + e) of e = exp(-|z|), or the other way round
    const double e = exp(-fabs(z)), big = 1.0 / (1.0 + e), small = e * big;
    const double p = z < 0.0 ? small : big, q = z < 0.0 ? big : small;
    f = g * p;
    d = fma(p, steep * q, p);
}

// The fp32 value whose rounding to bf16 is that of x.
__device__ __forceinline__ float for_bf16(double x)
{
    const float f = static_cast<float>(x);
    const uint32_t bits = __float_as_uint(f);
    if ((bits & 0xFFFFu) != 0x8000u || static_cast<double>(f) == x) return f;
    return __uint_as_float(fabs(static_cast<double>(f)) > fabs(x) ? bits - 1 : bits + 1);
}

template <int ACT, bool CODED>
__global__ __launch_bounds__(kThreads) void ffn_act_grad_kernel(FfnActArgs a, int64_t total, uint32_t nv, FastDiv by_nv)
{
    // a workgroup's vectors from its first row on: 32 bits are enough
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads, row0 = first / nv;
    const uint32_t at = static_cast<uint32_t>(first - row0 * nv) + threadIdx.x, q = div_by(at, by_nv);
    const int64_t row = row0 + q, pitch = 8 * static_cast<int64_t>(nv);
    const int v = static_cast<int>(at - q * nv), n = static_cast<int>(min(a.hidden - 8 * static_cast<int64_t>(v), int64_t{8}));
    if (first + threadIdx.x >= total) return;  // whole quads
    float g[8], u[8], da[8];
    const Raw8<false> raw_da = load8<false, true>(a.da, row, 8 * v, n);
    if constexpr (CODED) {
        u32x2 c[2];
        uint32_t s[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            c[k] = ld_codes(a.ckpt[k] + code_at(row, pitch, v));
            s[k] = ld_scale(a.ckpt[k] + a.rows * pitch + scale_at(row, pitch, v));
        }
        if (a.format == ZERO_ACT8_E4M3) {
            decode8<ZERO_ACT8_E4M3>(c[0], s[0], g);
            decode8<ZERO_ACT8_E4M3>(c[1], s[1], u);
        } else {
            decode8<ZERO_ACT8_INT8>(c[0], s[0], g);
            decode8<ZERO_ACT8_INT8>(c[1], s[1], u);
        }
    } else {
        const Raw8<false> raw_g = load8<false, true>(a.saved[0], row, 8 * v, n), raw_u = load8<false, true>(a.saved[1], row, 8 * v, n);
        unpack<false>(raw_g, 8 * v, n, g);
        unpack<false>(raw_u, 8 * v, n, u);
    }
    unpack<false>(raw_da, 8 * v, n, da);
    float dg[8], du[8], again[8];
    uint32_t unsure = 0, least = ~0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const Terms t = terms<ACT>(g[i]);
        const float both = da[i] * u[i];
        dg[i] = both * t.d;
        du[i] = da[i] * t.f;
        again[i] = t.f * u[i];
        // both rounded from either end of what they may be (a zero has no slack: it is exact)
        const float sg = fabsf(both) * t.slack_d, su = fabsf(du[i]) * t.slack_f;
        const bool apart = pack_bf16(dg[i] - sg, du[i] - su) != pack_bf16(dg[i] + sg, du[i] + su);
        unsure |= apart || !t.sure ? 1u << i : 0u;
        // twice the bits without the sign, less one: zeros come last
        least = min(least, min((__float_as_uint(dg[i]) << 1) - 1, (__float_as_uint(du[i]) << 1) - 1));
    }
    // Beside values of so little size fp32's smallest steps count: below 2^-100.
    if (least < 27u << 24) unsure = 0xFF;
    unsure &= (1u << max(n, 0)) - 1;
    while (unsure != 0) {  // of each lane the first one that is left
        const int i = __builtin_ctz(unsure);
        unsure &= unsure - 1;
        float gi = g[0], ui = u[0], di = da[0];
#pragma unroll
        for (int k = 1; k < 8; ++k) {
            gi = i == k ? g[k] : gi;
            ui = i == k ? u[k] : ui;
            di = i == k ? da[k] : di;
        }
        double f, d;
        terms64<ACT>(gi, f, d);
        const float x = for_bf16(static_cast<double>(di) * ui * d), y = for_bf16(di * f);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            dg[k] = i == k ? x : dg[k];
            du[k] = i == k ? y : du[k];
        }
    }
    if (a.ckpt_a != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) again[i] = i < n ? again[i] : 0.0f;
        const Code8 c = a.format == ZERO_ACT8_E4M3 ? encode8<ZERO_ACT8_E4M3>(again) : encode8<ZERO_ACT8_INT8>(again);
        *(ZERO_G u32x2*)(a.ckpt_a + code_at(row, pitch, v)) = c.codes;
        if ((v & 3) == 0) *(ZERO_G uint8_t*)(a.ckpt_a + a.rows * pitch + scale_at(row, pitch, v)) = static_cast<uint8_t>(c.scale);
    }
    store8<false>(a.d[0], row, 8 * v, n, dg);
    store8<false>(a.d[1], row, 8 * v, n, du);
}

}  // namespace

template <int ACT>
static void launch_act(const FfnActArgs& a, hipStream_t s)
{
    const uint32_t nv = static_cast<uint32_t>(act8_pitch(a.hidden) / 8);
    const int64_t total = a.rows * nv;
    const unsigned grid = static_cast<unsigned>((total + kThreads - 1) / kThreads);
    if (a.ckpt[0] != nullptr) ffn_act_grad_kernel<ACT, true><<<grid, kThreads, 0, s>>>(a, total, nv, fast_div(nv));
    else ffn_act_grad_kernel<ACT, false><<<grid, kThreads, 0, s>>>(a, total, nv, fast_div(nv));
}

hipError_t launch_ffn_act_grad(const FfnActArgs& a, hipStream_t s)
{
    if (a.act == ZERO_FFN_SILU) launch_act<ZERO_FFN_SILU>(a, s);
    else if (a.act == ZERO_FFN_GELU) launch_act<ZERO_FFN_GELU>(a, s);
    else launch_act<ZERO_FFN_GELU_TANH>(a, s);
    return hipGetLastError();
}

}  // namespace zero
