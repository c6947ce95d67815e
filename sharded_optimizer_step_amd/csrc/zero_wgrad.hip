// zero_wgrad.hip -- the weight gradient dW = dY^T X of a linear layer whose
// input X was saved in 8 bits, gfx950.
//
// Both factors have the summed index (the token) as their slow one, so both
// lie in LDS as they lie in memory, a row of a tile per token, and the
// transposing LDS reads turn 4 tokens x 16 columns into the operand layout of
// the matrix instructions. The 8-bit codes are decoded to bf16 on their way
// from memory to LDS: a power-of-two scale makes that exact, so the product
// is the bf16 one, with half the reads of X.
#include "zero_act8_device.h"

namespace zero {
namespace {

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// 16 codes with one scale, as bf16.
template <int FMT>
__device__ __forceinline__ void decode16(u32x4 codes, uint32_t scale, u32x4 (&out)[2])
{
    const float unit = act8_unit(scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = codes[i];
        uint32_t lo, hi;
        if constexpr (FMT == ZERO_ACT8_E4M3) {
            lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, unit, false));
            hi = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, unit, true));
        } else {
            float f[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) f[b] = static_cast<float>(static_cast<int>(w << (24 - 8 * b)) >> 24) * unit;
            lo = pack_bf16(f[0], f[1]);
            hi = pack_bf16(f[2], f[3]);
        }
        out[i / 2][2 * (i % 2)] = lo;
        out[i / 2][2 * (i % 2) + 1] = hi;
    }
}

// Eight consecutive tokens of this lane's column, from a tile in LDS whose
// rows are tokens: `at` is the lane's own place, see tr_place.
template <int STRIDE>
__device__ __forceinline__ bf16x8 read_tr(const uint16_t* at)
{
    typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
    const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)at);
    const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(at + 4 * STRIDE));
    typedef short i16x8 __attribute__((ext_vector_type(8)));
    return __builtin_bit_cast(bf16x8, (i16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// BM x BN tile of dW, BK tokens at a time, WM x WN waves.
template <int BM_, int BN_, int BK_, int WM_, int WN_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, BK = BK_, WM = WM_, WN = WN_;
    static constexpr int NT = 64 * WM * WN;
    static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;  // 16 x 16 pieces of a wave
    // 32 bytes over the row keep the four rows that a transposing read touches on different banks
    static constexpr int SA = BM + 16, SB = BN + 16;
    static constexpr int VA = BK * BM / 8 / NT, VB = BK * BN / 16 / NT;
};

template <class T, int FMT>
__global__ __launch_bounds__(T::NT) void wgrad_kernel(WgradArgs a, int tiles_m, int tiles_n, int split, int64_t chunk)
{
    __shared__ __align__(16) uint16_t sa[2][T::BK * T::SA];
    __shared__ __align__(16) uint16_t sb[2][T::BK * T::SB];
    // Consecutive workgroups go to the eight XCDs in turn: each XCD gets a run
    // of neighbouring tiles, which share their factors in its L2.
    const int tiles = tiles_m * tiles_n;
    const int total = tiles * split;
    const int each = (total + 7) / 8;
    const int id = (blockIdx.x % 8) * each + blockIdx.x / 8;
    if (id >= total || static_cast<int>(blockIdx.x / 8) >= each) return;
    const int part = id / tiles;
    const int in_part = id - part * tiles;
    // a run of tiles goes down 8 rows of tiles before it moves a tile to the right
    constexpr int kDown = 8;
    const int band = in_part / (kDown * tiles_n);
    const int rows_in_band = min(kDown, tiles_m - band * kDown);
    const int in_band = in_part - band * kDown * tiles_n;
    const int64_t m0 = static_cast<int64_t>(band * kDown + in_band % rows_in_band) * T::BM;
    const int64_t n0 = static_cast<int64_t>(in_band / rows_in_band) * T::BN;
    const int64_t begin = part * chunk, end = min(a.rows, begin + chunk);
    const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
    const bool inside = m0 + T::BM <= a.outs;

    u32x4 ra[T::VA], rb[T::VB];
    uint32_t rs[T::VB];
    const auto fetch = [&](int64_t k0) {
#pragma unroll
        for (int i = 0; i < T::VA; ++i) {
            const int id = tid + i * T::NT, r = id / (T::BM / 8), c = id % (T::BM / 8) * 8;
            const int64_t t = k0 + r, left = a.outs - (m0 + c);
            const Rows dy{const_cast<uint16_t*>(a.dy + m0), a.ld_dy, 0};
            if (inside) ra[i] = t < end ? ld16_a2(a.dy + t * a.ld_dy + m0 + c) : u32x4{};
            else ra[i] = t < end && left > 0 ? load8<false>(dy, t, c, left < 8 ? static_cast<int>(left) : 8).v[0] : u32x4{};
        }
#pragma unroll
        for (int i = 0; i < T::VB; ++i) {
            const int id = tid + i * T::NT, r = id / (T::BN / 16), c = id % (T::BN / 16) * 16;
            const int64_t t = k0 + r;
            if (t < end && n0 + c < a.pitch) {
                rb[i] = *(const ZERO_G u32x4*)(a.codes + t * a.pitch + n0 + c);
                rs[i] = ld_scale(a.scales + t * (a.pitch / kActBlock) + (n0 + c) / kActBlock);
            } else {
                rb[i] = u32x4{};
                rs[i] = 127;
            }
        }
    };
    const auto stage = [&](int buf) {
#pragma unroll
        for (int i = 0; i < T::VA; ++i) {
            const int id = tid + i * T::NT, r = id / (T::BM / 8), c = id % (T::BM / 8) * 8;
            *reinterpret_cast<u32x4*>(&sa[buf][r * T::SA + c]) = ra[i];
        }
#pragma unroll
        for (int i = 0; i < T::VB; ++i) {
            const int id = tid + i * T::NT, r = id / (T::BN / 16), c = id % (T::BN / 16) * 16;
            u32x4 w[2];
            decode16<FMT>(rb[i], rs[i], w);
            *reinterpret_cast<u32x4*>(&sb[buf][r * T::SB + c]) = w[0];
            *reinterpret_cast<u32x4*>(&sb[buf][r * T::SB + c + 8]) = w[1];
        }
    };

    const int wm = wave / T::WN * (T::BM / T::WM), wn = wave % T::WN * (T::BN / T::WN);
    // In a transposing read 16 lanes take 4 tokens x 16 columns: lane i reads 4
    // columns of token i / 4 and gets column i of all four.
    const int tr_row = 8 * (lane / 16) + lane % 16 / 4, tr_col = lane % 4 * 4;
    f32x4 acc[T::TN][T::TM];
#pragma unroll
    for (int j = 0; j < T::TN; ++j)
#pragma unroll
        for (int i = 0; i < T::TM; ++i) acc[j][i] = f32x4{};

    int buf = 0;
    if (begin < end) {
        fetch(begin);
        stage(0);
        if (begin + T::BK < end) fetch(begin + T::BK);
        __syncthreads();
    }
    for (int64_t k0 = begin; k0 < end; k0 += T::BK) {
        // the next tile, fetched an iteration ago, goes to the other buffer; the
        // barrier at the end of the last iteration was after its last read
        if (k0 + T::BK < end) stage(buf ^ 1);
        if (k0 + 2 * T::BK < end) fetch(k0 + 2 * T::BK);
#pragma unroll
        for (int k = 0; k < T::BK; k += 32) {
            bf16x8 fa[T::TM], fb[T::TN];
#pragma unroll
            for (int i = 0; i < T::TM; ++i) fa[i] = read_tr<T::SA>(&sa[buf][(k + tr_row) * T::SA + wm + 16 * i + tr_col]);
#pragma unroll
            for (int j = 0; j < T::TN; ++j) fb[j] = read_tr<T::SB>(&sb[buf][(k + tr_row) * T::SB + wn + 16 * j + tr_col]);
#pragma unroll
            for (int j = 0; j < T::TN; ++j)
#pragma unroll
                for (int i = 0; i < T::TM; ++i)
                    acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], acc[j][i], 0, 0, 0);
        }
        __syncthreads();
        buf ^= 1;
    }

    // X is the first operand, so a lane holds four neighbouring columns of one row of dW
#pragma unroll
    for (int j = 0; j < T::TN; ++j) {
        const int64_t n = n0 + wn + 16 * j + lane / 16 * 4;
        const int left = n < a.cols ? static_cast<int>(a.cols - n < 4 ? a.cols - n : 4) : 0;
        float scale[4] = {1.0f, 1.0f, 1.0f, 1.0f};
        if (split == 1 && a.col_scale.p != nullptr) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (r < left) scale[r] = a.col_scale.f32 ? ((const ZERO_G float*)a.col_scale.p)[n + r]
                                                         : __uint_as_float(static_cast<uint32_t>(((const ZERO_G uint16_t*)a.col_scale.p)[n + r]) << 16);
        }
#pragma unroll
        for (int i = 0; i < T::TM; ++i) {
            const int64_t m = m0 + wm + 16 * i + lane % 16;
            if (m >= a.outs || left == 0) continue;
            f32x4 v = acc[j][i];
            if (split > 1) {
                float* p = a.part + (static_cast<int64_t>(part) * a.outs + m) * a.cols + n;
                if (left == 4) st16_a4(p, __builtin_bit_cast(u32x4, v));
                else
                    for (int r = 0; r < left; ++r) ((ZERO_G float*)p)[r] = v[r];
                continue;
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] *= scale[r];
            if (a.dw.f32) {
                float* p = static_cast<float*>(a.dw.p) + m * a.dw.ld + n;
                if (left == 4) {
                    if (a.accumulate) v += __builtin_bit_cast(f32x4, ld16_a4(p));
                    st16_a4(p, __builtin_bit_cast(u32x4, v));
                } else {
#pragma unroll
                    for (int r = 0; r < 3; ++r)
                        if (r < left) ((ZERO_G float*)p)[r] = a.accumulate ? ((ZERO_G float*)p)[r] + v[r] : v[r];
                }
            } else {
                uint16_t* p = static_cast<uint16_t*>(a.dw.p) + m * a.dw.ld + n;
                const u32x2 w{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
                typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
                if (left == 4) *(ZERO_G u32x2_a2*)p = w;
                else {
#pragma unroll
                    for (int r = 0; r < 3; ++r)
                        if (r < left) ((ZERO_G uint16_t*)p)[r] = static_cast<uint16_t>(w[r / 2] >> (16 * (r % 2)));
                }
            }
        }
    }
}

// The partial products of a split sum, added in the order of the tokens.
__global__ __launch_bounds__(256) void wgrad_join_kernel(WgradArgs a, int split, FastDiv by_cols)
{
    const int64_t size = a.outs * a.cols;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < size; i += static_cast<int64_t>(gridDim.x) * 256) {
        float s = ((const ZERO_G float*)a.part)[i];
        for (int p = 1; p < split; ++p) s += ((const ZERO_G float*)a.part)[p * size + i];
        const int64_t m = size < (1ll << 31) ? div_by(static_cast<uint32_t>(i), by_cols) : i / a.cols;
        const int64_t n = i - m * a.cols;
        if (a.col_scale.p != nullptr)
            s *= a.col_scale.f32 ? ((const ZERO_G float*)a.col_scale.p)[n]
                                 : __uint_as_float(static_cast<uint32_t>(((const ZERO_G uint16_t*)a.col_scale.p)[n]) << 16);
        if (a.dw.f32) {
            ZERO_G float* p = (ZERO_G float*)a.dw.p + m * a.dw.ld + n;
            *p = a.accumulate ? *p + s : s;
        } else {
            ((ZERO_G uint16_t*)a.dw.p)[m * a.dw.ld + n] = static_cast<uint16_t>(pack_bf16(s, 0.0f));
        }
    }
}

using Tile128 = Tile<128, 128, 64, 2, 2>;

template <class T>
hipError_t launch_tile(const WgradArgs& a, const WgradPlan& plan, int format, hipStream_t s)
{
    const int64_t tm = (a.outs + T::BM - 1) / T::BM, tn = (a.cols + T::BN - 1) / T::BN;
    const int64_t total = tm * tn * plan.split;
    const unsigned grid = static_cast<unsigned>((total + 7) / 8 * 8);
    const int m = static_cast<int>(tm), n = static_cast<int>(tn);
    if (format == ZERO_ACT8_E4M3) wgrad_kernel<T, ZERO_ACT8_E4M3><<<grid, T::NT, 0, s>>>(a, m, n, plan.split, plan.chunk);
    else wgrad_kernel<T, ZERO_ACT8_INT8><<<grid, T::NT, 0, s>>>(a, m, n, plan.split, plan.chunk);
    return hipGetLastError();
}

}  // namespace

// Tiles that fill the compute units are not split. Fewer of them are split
// over the tokens until two workgroups a unit are there, but not below 256
// tokens a part.
WgradPlan wgrad_plan(int64_t rows, int64_t outs, int64_t cols)
{
    WgradPlan p{};
    constexpr int64_t kSlots = 2 * kComputeUnits, kLeast = 256;
    const int64_t tiles = ((outs + 127) / 128) * ((cols + 127) / 128);
    int64_t split = 1;
    if (tiles > 0 && 2 * tiles <= kSlots) {
        split = kSlots / tiles;
        const int64_t most = (rows + kLeast - 1) / kLeast;
        if (split > most) split = most;
        if (split < 1) split = 1;
    }
    p.chunk = (rows + split - 1) / split;
    p.chunk = (p.chunk + 63) / 64 * 64;
    if (p.chunk < 64) p.chunk = 64;
    split = (rows + p.chunk - 1) / p.chunk;
    p.split = split < 1 ? 1 : static_cast<int>(split);
    p.bytes = p.split > 1 ? sizeof(float) * static_cast<size_t>(p.split) * static_cast<size_t>(outs * cols) : 0;
    return p;
}

hipError_t launch_wgrad(const WgradArgs& a, const WgradPlan& plan, int format, hipStream_t s)
{
    const hipError_t e = launch_tile<Tile128>(a, plan, format, s);
    if (e != hipSuccess || plan.split == 1) return e;
    const int64_t blocks = (a.outs * a.cols + 255) / 256;
    const unsigned grid = static_cast<unsigned>(blocks < 8 * kComputeUnits ? blocks : 8 * kComputeUnits);
    wgrad_join_kernel<<<grid, 256, 0, s>>>(a, plan.split, fast_div(static_cast<uint32_t>(a.cols)));
    return hipGetLastError();
}

}  // namespace zero
