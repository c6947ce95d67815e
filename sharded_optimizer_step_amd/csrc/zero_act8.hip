// zero_act8.hip -- activation rows to and from their 8-bit form, gfx950.
//
// Both are streams: 8 columns (one 16-byte bf16 load) a thread, four threads
// to a block of 32 columns, whose largest value they find with two quad
// permutes. The rows are visited as one list of 8-column vectors, so narrow
// and odd rows fill a wave like wide ones. HBM bounds both: 16384 x 4096 bf16
// (3.03 bytes a value) is saved in 40 us and read back in 30, 5.1 and 6.8 TB/s
// (part of it from the Infinity Cache), where a copy of 2 GiB runs at 4.9; a
// call of 129 x 771 takes 4.5 us, a launch's latency.
#include "zero_act8_device.h"

namespace zero {
namespace {

constexpr int kActThreads = 256;
constexpr int kActVecs = 4;  // vectors of a thread: their loads are all in flight together

// Vector `i` of the tile that starts at vector `first` of the list: its row and its place in the row.
struct Place {
    int64_t row;
    int v;
};
__device__ __forceinline__ Place place(int64_t row0, uint32_t rest, uint32_t i, uint32_t nv, FastDiv by_nv)
{
    const uint32_t n = rest + i;
    const uint32_t q = div_by(n, by_nv);
    return Place{row0 + q, static_cast<int>(n - q * nv)};
}

template <bool F32, int FMT>
__global__ __launch_bounds__(kActThreads) void act8_save_kernel(Rows x, int64_t total, int cols, uint32_t nv,
                                                                FastDiv by_nv, uint8_t* codes, uint8_t* scales)
{
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (kActThreads * kActVecs);
    const int64_t row0 = first / nv;
    const uint32_t rest = static_cast<uint32_t>(first - row0 * nv);
    const int64_t pitch = 8 * static_cast<int64_t>(nv);
    Raw8<F32> raw[kActVecs];
    Place at[kActVecs];
#pragma unroll
    for (int u = 0; u < kActVecs; ++u) {
        const uint32_t i = u * kActThreads + threadIdx.x;
        if (first + i >= total) continue;  // whole quads: the list is a multiple of four vectors
        at[u] = place(row0, rest, i, nv, by_nv);
        raw[u] = load8<F32>(x, at[u].row, 8 * at[u].v, cols - 8 * at[u].v);
    }
#pragma unroll
    for (int u = 0; u < kActVecs; ++u) {
        const uint32_t i = u * kActThreads + threadIdx.x;
        if (first + i >= total) continue;
        float f[8];
        unpack<F32>(raw[u], 8 * at[u].v, cols - 8 * at[u].v, f);
        const Code8 c = encode8<FMT>(f);
        *(ZERO_G u32x2*)(codes + code_at(at[u].row, pitch, at[u].v)) = c.codes;
        if ((at[u].v & 3) == 0) *(ZERO_G uint8_t*)(scales + scale_at(at[u].row, pitch, at[u].v)) = static_cast<uint8_t>(c.scale);
    }
}

template <bool F32, int FMT>
__global__ __launch_bounds__(kActThreads) void act8_load_kernel(const uint8_t* codes, const uint8_t* scales, int64_t total,
                                                                int cols, uint32_t nv, FastDiv by_nv, Rows out)
{
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (kActThreads * kActVecs);
    const int64_t row0 = first / nv;
    const uint32_t rest = static_cast<uint32_t>(first - row0 * nv);
    const int64_t pitch = 8 * static_cast<int64_t>(nv);
    u32x2 c[kActVecs];
    uint32_t s[kActVecs];
    Place at[kActVecs];
#pragma unroll
    for (int u = 0; u < kActVecs; ++u) {
        const uint32_t i = u * kActThreads + threadIdx.x;
        if (first + i >= total) continue;
        at[u] = place(row0, rest, i, nv, by_nv);
        c[u] = ld_codes(codes + code_at(at[u].row, pitch, at[u].v));
        s[u] = ld_scale(scales + scale_at(at[u].row, pitch, at[u].v));
    }
#pragma unroll
    for (int u = 0; u < kActVecs; ++u) {
        const uint32_t i = u * kActThreads + threadIdx.x;
        if (first + i >= total) continue;
        float f[8];
        decode8<FMT>(c[u], s[u], f);
        store8<F32, true>(out, at[u].row, 8 * at[u].v, cols - 8 * at[u].v, f);
    }
}

int64_t tiles(int64_t vectors) { return (vectors + kActThreads * kActVecs - 1) / (kActThreads * kActVecs); }

}  // namespace

hipError_t launch_act8_save(const Rows& x, int64_t rows, int64_t cols, int format, uint8_t* ckpt, hipStream_t s)
{
    const int64_t pitch = act8_pitch(cols);
    const uint32_t nv = static_cast<uint32_t>(pitch / 8);
    const int64_t total = rows * nv;
    const unsigned grid = static_cast<unsigned>(tiles(total));
    uint8_t* scales = ckpt + rows * pitch;
    const FastDiv d = fast_div(nv);
    const int c = static_cast<int>(cols);
    const bool e4m3 = format == ZERO_ACT8_E4M3;
    if (x.f32 && e4m3) act8_save_kernel<true, ZERO_ACT8_E4M3><<<grid, kActThreads, 0, s>>>(x, total, c, nv, d, ckpt, scales);
    else if (x.f32) act8_save_kernel<true, ZERO_ACT8_INT8><<<grid, kActThreads, 0, s>>>(x, total, c, nv, d, ckpt, scales);
    else if (e4m3) act8_save_kernel<false, ZERO_ACT8_E4M3><<<grid, kActThreads, 0, s>>>(x, total, c, nv, d, ckpt, scales);
    else act8_save_kernel<false, ZERO_ACT8_INT8><<<grid, kActThreads, 0, s>>>(x, total, c, nv, d, ckpt, scales);
    return hipGetLastError();
}

hipError_t launch_act8_load(const uint8_t* ckpt, int64_t rows, int64_t cols, int format, const Rows& out, hipStream_t s)
{
    const int64_t pitch = act8_pitch(cols);
    const uint32_t nv = static_cast<uint32_t>(pitch / 8);
    const int64_t total = rows * nv;
    const unsigned grid = static_cast<unsigned>(tiles(total));
    const uint8_t* scales = ckpt + rows * pitch;
    const FastDiv d = fast_div(nv);
    const int c = static_cast<int>(cols);
    const bool e4m3 = format == ZERO_ACT8_E4M3;
    if (out.f32 && e4m3) act8_load_kernel<true, ZERO_ACT8_E4M3><<<grid, kActThreads, 0, s>>>(ckpt, scales, total, c, nv, d, out);
    else if (out.f32) act8_load_kernel<true, ZERO_ACT8_INT8><<<grid, kActThreads, 0, s>>>(ckpt, scales, total, c, nv, d, out);
    else if (e4m3) act8_load_kernel<false, ZERO_ACT8_E4M3><<<grid, kActThreads, 0, s>>>(ckpt, scales, total, c, nv, d, out);
    else act8_load_kernel<false, ZERO_ACT8_INT8><<<grid, kActThreads, 0, s>>>(ckpt, scales, total, c, nv, d, out);
    return hipGetLastError();
}

}  // namespace zero
