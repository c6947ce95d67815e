// zero_block.h -- host types and launch wrappers of the calls around a
// training block (8-bit activation checkpoints, the weight gradient taken
// from one, the norms with gate and residual scale, the layer norm, the gated
// feed-forward block). Not part of the public C ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "zero_step.h"

namespace zero {

constexpr int kActBlock = 32;    // columns that share one power of two
constexpr int kActMinExp = -117; // smallest k: e4m3's smallest code times 2^k is still a normal fp32 number
constexpr int kComputeUnits = 256;  // of an MI355X: the split rules below must not depend on a device

__host__ __device__ inline int64_t act8_pitch(int64_t cols) { return (cols + kActBlock - 1) / kActBlock * kActBlock; }

// Division of n < 2^31 by a fixed d in [1, 2^31): n / d = (mulhi(n, mul) + n) >> shift.
struct FastDiv {
    uint32_t mul;
    uint32_t shift;
};
inline FastDiv fast_div(uint32_t d)
{
    uint32_t shift = 0;
    while ((1ull << shift) < d) ++shift;
    return FastDiv{static_cast<uint32_t>((((1ull << shift) - d) << 32) / d + 1), shift};
}

// A row-major operand as the kernels see it.
struct Rows {
    void* p;
    int64_t ld;
    int32_t f32;  // fp32, else bf16
};

// Every row of m starts on 16 bytes (so does an absent operand's).
inline bool rows_on_16(const Rows& m)
{
    return (reinterpret_cast<uintptr_t>(m.p) | static_cast<uint64_t>(m.ld) * (m.f32 ? 4 : 2)) % 16 == 0;
}

hipError_t launch_act8_save(const Rows& x, int64_t rows, int64_t cols, int format, uint8_t* ckpt, hipStream_t s);
hipError_t launch_act8_load(const uint8_t* ckpt, int64_t rows, int64_t cols, int format, const Rows& out,
                            hipStream_t s);

// The weight gradient: tiles of dw. The first `whole` tiles are summed over all
// rows by one workgroup; each of the others over `split` ranges of them, whose
// sums go to the workspace (a tile's ranges next to each other), and a second
// launch adds them in order.
struct WgradPlan {
    int tile;       // index of the tile shape
    int64_t whole;
    int split;      // ranges of rows
    int64_t chunk;  // rows of a range (the last may be shorter)
    size_t bytes;   // workspace
};
WgradPlan wgrad_plan(int64_t rows, int64_t outs, int64_t cols);

struct WgradArgs {
    const uint16_t* dy;
    int64_t ld_dy;
    const uint8_t* codes;
    const uint8_t* scales;
    int64_t pitch;  // bytes of a row of codes; a row of scales has pitch / 32
    int64_t rows, outs, cols;
    Rows col_scale;  // p null: ones
    Rows dw;
    int accumulate;
    float* part;
};
hipError_t launch_wgrad(const WgradArgs& a, const WgradPlan& plan, int format, hipStream_t s);

struct NormArgs {
    int64_t rows;
    int64_t unit_rows;  // rows that a workgroup (or wave) takes, set at the launch
    int32_t cols;
    float alpha, eps;
    int32_t stream;  // read x and y past the caches, set at the launch
    Rows x, y, w_post, gate, w_pre, x_out, h;
    FastDiv gate_div;
    float* rstd_post;
    float* rstd_pre;
    uint8_t* ckpt_post;
    uint8_t* ckpt_pre;
    int format;
};
hipError_t launch_block_norm(const NormArgs& a, hipStream_t s);

// How the rows of a norm's backward pass are dealt out. A unit is what one
// workgroup (or one wave, for short rows) sums over. With few gate rows
// (per_gate >= 1) each gate row is cut into per_gate units of unit_rows rows;
// with many (per_gate == 0) a unit takes unit_gates whole gate rows.
struct NormGradPlan {
    int64_t gates;       // rows of the gate (1 without one)
    int64_t gate_rows;   // rows that share one
    int64_t per_gate;
    int64_t unit_rows;
    int64_t unit_gates;
    int64_t units;
    int64_t strips;      // strips of columns, where rows may be too wide for one workgroup; else 0
    size_t bytes;        // workspace: two fp32 rows of cols per unit; with strips, two fp32 values per row
};
NormGradPlan norm_grad_plan(int64_t rows, int64_t cols, int64_t gate_rows);

struct NormGradArgs {
    int64_t rows;
    int32_t cols;
    float alpha;
    Rows dh, dx_out, w_post, gate, w_pre, x_out, y, dx, dy, dw_pre, dw_post, dgate;
    const uint8_t* ckpt_pre;
    const uint8_t* ckpt_post;
    const float* rstd_pre;
    const float* rstd_post;
    int format;
    int accumulate;
    int stream;  // write dx and dy past the caches, set at the launch
    NormGradPlan plan;
    FastDiv gate_div;
    float* sum_pre;   // [units][cols]: sums of dh * xn, for dw_pre
    float* sum_post;  // [units][cols]: sums of d * yn (few gate rows, for dw_post and dgate), or of gate * d * yn (many, for dw_post)
    float* row_sums;  // [rows][2] with strips
};
hipError_t launch_block_norm_grad(const NormGradArgs& a, hipStream_t s);

struct LayerNormArgs {
    int64_t rows;
    int64_t unit_rows;  // rows that a workgroup (or wave) takes, set at the launch
    int32_t cols;
    float eps;
    int32_t stream;  // read x and y past the caches, set at the launch
    Rows x, y, w, b, x_out, h;
    float* mean;
    float* rstd;
    uint8_t* ckpt_xn;
    uint8_t* ckpt_h;
    int format;
};
hipError_t launch_layer_norm(const LayerNormArgs& a, hipStream_t s);

// The rows of the backward pass: `units` of unit_rows rows, each of which a
// workgroup (or wave) sums over; a second launch joins their sums.
struct LayerNormGradPlan {
    int64_t unit_rows;
    int64_t units;
    bool strips;   // rows too wide for one workgroup
    size_t bytes;  // workspace: two fp32 rows of cols per unit, and for rows in strips two fp32 values per row
};
LayerNormGradPlan layer_norm_grad_plan(int64_t rows, int64_t cols);

struct LayerNormGradArgs {
    int64_t rows;
    int32_t cols;
    Rows dh, dx_out, w, x_out, dx, dy, dw, db;
    const uint8_t* ckpt_xn;
    const float* mean;
    const float* rstd;
    int format;
    int accumulate;
    int stream;  // write dx and dy past the caches, set at the launch
    LayerNormGradPlan plan;
    float* sum_w;  // [units][cols]: sums of dh * xn
    float* sum_b;  // [units][cols]: sums of dh
    float* row_means;  // [rows][2] with strips
};
hipError_t launch_layer_norm_grad(const LayerNormGradArgs& a, hipStream_t s);

// The three products of the gated feed-forward block.
enum FfnKind {
    kFfnForward,  // [gate | up] = h [w_gate | w_up]^T, with the activation
    kFfnInput,    // dh = dgate w_gate + dup w_up
    kFfnWeight,   // dw_gate = dgate^T h and dw_up = dup^T h
};

// Workspace of a product: aligned copies of operands whose columns are not a
// multiple of 8, and the parts of tiles that are split over the summed index,
// whatever the operands' alignment, and whether one or both weight gradients
// are made.
size_t ffn_workspace_bytes(FfnKind kind, int64_t rows, int64_t cols, int64_t hidden);

struct FfnArgs {
    int64_t rows, cols, hidden;
    const uint16_t* h;
    int64_t ld_h;
    const uint16_t* w[2];  // w_gate, w_up
    int64_t ld_w[2];
    const uint16_t* d[2];  // dgate, dup; for one weight gradient the first is what it is taken from
    int64_t ld_d[2];
    Rows out[2];           // gate and up (p null: not wanted), or dh, or one or two weight gradients
    Rows a;
    uint8_t* ckpt[2];      // of gate and up, or null
    int format;
    int act;
    int accumulate;
    float* part;
    // set at the launch
    int outputs;    // weight gradients made at once
    int plain;      // whole steps of unaligned operands are read at 32-bit offsets
    int64_t chunk;  // steps of a range of a split tile
    int split;
};
hipError_t launch_ffn(FfnKind kind, const FfnArgs& a, hipStream_t s);

// dgate, dup and a in 8 bits from da and the saved gate and up.
struct FfnActArgs {
    int64_t rows, hidden;
    Rows da, saved[2], d[2];
    const uint8_t* ckpt[2];  // null: from saved
    uint8_t* ckpt_a;
    int format;
    int act;
};
hipError_t launch_ffn_act_grad(const FfnActArgs& a, hipStream_t s);

}  // namespace zero
