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
//
// e4m3: one instruction for two codes and their scale. int8: the code with its
// sign bit turned over is u = code + 128 in 0 .. 255; under the byte 0x64 it is
// the half 1024 + u, and one mixed fma makes (1024 + u) unit - 1152 unit =
// code * unit, without a rounding: two and a quarter instructions a code
// instead of three and a half.
template <int FMT>
__device__ __forceinline__ void decode16(u32x4 codes, uint32_t scale, u32x4 (&out)[2])
{
    const float unit = act8_unit(scale);
    const float back = -1152.0f * unit;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t lo, hi;
        if constexpr (FMT == ZERO_ACT8_E4M3) {
            lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[i], unit, false));
            hi = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[i], unit, true));
        } else {
            typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
            const uint32_t u = codes[i] ^ 0x80808080u;
            const f16x2 a = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u));
            const f16x2 b = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u));
            lo = pack_bf16(fmaf(static_cast<float>(a.x), unit, back), fmaf(static_cast<float>(a.y), unit, back));
            hi = pack_bf16(fmaf(static_cast<float>(b.x), unit, back), fmaf(static_cast<float>(b.y), unit, back));
        }
        out[i / 2][2 * (i % 2)] = lo;
        out[i / 2][2 * (i % 2) + 1] = hi;
    }
}

// Eight tokens of this lane's column, from a tile in LDS whose rows are tokens;
// `at` is what the lane itself reads of the first four, see tr_row.
template <int STRIDE>
__device__ __forceinline__ bf16x8 read_tr(const uint16_t* at)
{
    typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
    const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)at);
    const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(at + 16 * STRIDE));
    typedef short i16x8 __attribute__((ext_vector_type(8)));
    return __builtin_bit_cast(bf16x8, (i16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// The column scales of columns n .. n + left - 1, at most four.
__device__ __forceinline__ f32x4 load_scale(const WgradArgs& a, int64_t n, int left)
{
    f32x4 s{1.0f, 1.0f, 1.0f, 1.0f};
    if (a.col_scale.p != nullptr) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (r < left)
                s[r] = a.col_scale.f32 ? ((const ZERO_G float*)a.col_scale.p)[n + r]
                                       : __uint_as_float(static_cast<uint32_t>(((const ZERO_G uint16_t*)a.col_scale.p)[n + r]) << 16);
    }
    return s;
}

// Columns n .. n + left - 1 of row m of dW: the sums v times their scales.
__device__ __forceinline__ void store_dw(const WgradArgs& a, int64_t m, int64_t n, int left, f32x4 v, f32x4 scale)
{
    v *= scale;
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

// BM x BN tile of dW, BK tokens at a time, WM x WN waves, SLOTS workgroups a
// compute unit (two waves a SIMD and LDS for that many).
template <int BM_, int BN_, int BK_, int WM_, int WN_, int SLOTS_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, BK = BK_, WM = WM_, WN = WN_, SLOTS = SLOTS_;
    static constexpr int NT = 64 * WM * WN;
    static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;  // 16 x 16 pieces of a wave
    // 32 bytes over the row keep the four rows that a transposing read touches on different banks
    static constexpr int SA = BM + 16, SB = BN + 16;
    // a thread fetches 8 columns of dY, 16 of X, of every RA-th and RB-th row
    static constexpr int CA = BM / 8, RA = NT / CA, VA = BK / RA;
    static constexpr int CB = BN / 16, RB = NT / CB, VB = BK / RB;
    static_assert(NT % CA == 0 && NT % CB == 0 && BK % RA == 0 && BK % RB == 0, "a thread keeps its columns");
};

template <class T, int FMT>
__global__ __launch_bounds__(T::NT, T::NT / 256 * T::SLOTS) void wgrad_kernel(WgradArgs a, int tiles_m, int tiles_n, int split, int64_t chunk)
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
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / 64), lane = tid % 64;

    // This thread's 8 columns of dY. Columns from `outs` on are not read: a
    // vector that would run over them is read further left and shifted, one
    // wholly beyond them is another valid one, whose products are not stored.
    const int ca = tid % T::CA * 8, row_a = tid / T::CA;
    const int64_t left_a = a.outs - (m0 + ca);
    const int shift = left_a > 0 && left_a < 8 && a.outs >= 8 ? static_cast<int>(8 - left_a) : 0;
    const int64_t col_a = left_a > 0 ? m0 + ca - shift : 0;
    const bool ragged = m0 + T::BM > a.outs && a.outs % 8 != 0;
    const int cb = tid % T::CB * 16, row_b = tid / T::CB;
    // 16 decoded columns are 32 bytes of LDS, written 16 at a time: every second
    // four lanes write their second half first, so that eight lanes in a row
    // touch different banks.
    const int first_b = tid / 4 % 2 * 8;
    const int64_t col_b = n0 + cb < a.pitch ? n0 + cb : 0;
    const int64_t pitch_s = a.pitch / kActBlock;
    // Whole tiles are read at a base that all threads share and 32-bit offsets.
    const bool plain = !ragged && a.outs >= 8 && a.ld_dy < (int64_t{1} << 24) && a.pitch < (int64_t{1} << 25);
    uint32_t off_a = static_cast<uint32_t>((row_a * a.ld_dy + col_a) * 2);
    uint32_t off_b = static_cast<uint32_t>(row_b * a.pitch + col_b);
    uint32_t off_s = static_cast<uint32_t>(row_b * pitch_s + col_b / kActBlock);

    u32x4 ra[T::VA], rb[T::VB];
    uint32_t rs[T::VB];
    // (a shared base and a 32-bit offset are one load instruction; left to
    // itself the compiler keeps a 64-bit address of each load in registers)
    const auto fetch_whole = [&](int64_t k0) {
        asm volatile("" : "+v"(off_a), "+v"(off_b), "+v"(off_s));
#pragma unroll
        for (int i = 0; i < T::VA; ++i)
            ra[i] = ld16_a2(reinterpret_cast<const char*>(a.dy + (k0 + i * T::RA) * a.ld_dy) + off_a);
#pragma unroll
        for (int i = 0; i < T::VB; ++i) {
            rb[i] = ld16_a4(a.codes + (k0 + i * T::RB) * a.pitch + off_b);
            rs[i] = ld_scale(a.scales + (k0 + i * T::RB) * pitch_s + off_s);
        }
    };
    const auto fetch = [&](int64_t k0) {
        if (plain && k0 + T::BK <= end) return fetch_whole(k0);
#pragma unroll
        for (int i = 0; i < T::VA; ++i) {
            const int64_t t = k0 + row_a + i * T::RA;
            const Rows dy{const_cast<uint16_t*>(a.dy + col_a), a.ld_dy, 0};
            ra[i] = u32x4{};
            if (t < end) ra[i] = load8<false>(dy, t, 0, a.outs >= 8 ? 8 : left_a > 0 ? static_cast<int>(left_a) : 0).v[0];
        }
#pragma unroll
        for (int i = 0; i < T::VB; ++i) {
            const int64_t t = k0 + row_b + i * T::RB;
            rb[i] = u32x4{};
            rs[i] = 127;
            if (t < end) {
                rb[i] = ld16_a4(a.codes + t * a.pitch + col_b);
                rs[i] = ld_scale(a.scales + t * pitch_s + col_b / kActBlock);
            }
        }
    };
    const auto shift_left = [&] {
        if (ragged && shift > 0) {
#pragma unroll
            for (int i = 0; i < T::VA; ++i) {
                for (int k = 0; k < shift; ++k) {  // one element to the left
                    ra[i].x = ra[i].x >> 16 | ra[i].y << 16;
                    ra[i].y = ra[i].y >> 16 | ra[i].z << 16;
                    ra[i].z = ra[i].z >> 16 | ra[i].w << 16;
                    ra[i].w >>= 16;
                }
            }
        }
    };
    const auto stage_whole = [&](int buf) {
#pragma unroll
        for (int i = 0; i < T::VA; ++i) *reinterpret_cast<u32x4*>(&sa[buf][(row_a + i * T::RA) * T::SA + ca]) = ra[i];
#pragma unroll
        for (int i = 0; i < T::VB; ++i) {
            u32x4 w[2];
            const u32x4 c = first_b != 0 ? u32x4{rb[i].z, rb[i].w, rb[i].x, rb[i].y} : rb[i];
            decode16<FMT>(c, rs[i], w);
            uint16_t* p = &sb[buf][(row_b + i * T::RB) * T::SB + cb];
            *reinterpret_cast<u32x4*>(p + first_b) = w[0];
            *reinterpret_cast<u32x4*>(p + 8 - first_b) = w[1];
        }
    };
    const auto stage = [&](int buf) {
        shift_left();
        stage_whole(buf);
    };

    const int wm = wave / T::WN * (T::BM / T::WM), wn = wave % T::WN * (T::BN / T::WN);
    // In a transposing read 16 lanes take 4 tokens x 16 columns: lane i reads 4
    // columns of token i / 4 and gets column i of all four. A wave's first read
    // takes tokens 0 .. 15 of 32 and its second the rest, for both factors, so
    // the 8 tokens of a sum's lane are 4 g .. 4 g + 3 and 16 more of each (which
    // 8 does not matter to the sum) and 32 lanes read 8 neighbouring rows, which
    // lie on different banks.
    const int tr_row = lane / 4, tr_col = lane % 4 * 4;
    f32x4 acc[T::TN][T::TM];
#pragma unroll
    for (int j = 0; j < T::TN; ++j)
#pragma unroll
        for (int i = 0; i < T::TM; ++i) acc[j][i] = f32x4{};

    const auto multiply = [&](int buf) {
#pragma unroll
        for (int k = 0; k < T::BK; k += 32) {
            bf16x8 fa[T::TM], fb[T::TN];
#pragma unroll
            for (int j = 0; j < T::TN; ++j) fb[j] = read_tr<T::SB>(&sb[buf][(k + tr_row) * T::SB + wn + 16 * j + tr_col]);
#pragma unroll
            for (int i = 0; i < T::TM; ++i) fa[i] = read_tr<T::SA>(&sa[buf][(k + tr_row) * T::SA + wm + 16 * i + tr_col]);
#pragma unroll
            for (int i = 0; i < T::TM; ++i)
#pragma unroll
                for (int j = 0; j < T::TN; ++j)
                    acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], acc[j][i], 0, 0, 0);
        }
    };
    // One tile from `buf` while the next, fetched a step ago, goes to the other
    // buffer (whose last reads were before the last barrier) and the one after
    // that is fetched.
    const auto step = [&](int64_t k0, int buf) {
        if (k0 + T::BK < end) stage(buf ^ 1);
        if (k0 + 2 * T::BK < end) fetch(k0 + 2 * T::BK);
        multiply(buf);
        __syncthreads();
    };
    const auto whole_step = [&](int64_t k0, int buf) {
        stage_whole(buf ^ 1);
        fetch_whole(k0 + 2 * T::BK);
        multiply(buf);
        __syncthreads();
    };
    if (begin < end) {
        fetch(begin);
        stage(0);
        if (begin + T::BK < end) fetch(begin + T::BK);
        __syncthreads();
    }
    int64_t k0 = begin;
    if (plain) {
        for (; k0 + 4 * T::BK <= end; k0 += 2 * T::BK) {
            whole_step(k0, 0);
            whole_step(k0 + T::BK, 1);
        }
    }
    for (; k0 < end; k0 += 2 * T::BK) {
        step(k0, 0);
        if (k0 + T::BK < end) step(k0 + T::BK, 1);
    }

    // X is the first operand, so a lane holds four neighbouring columns of one row
    // of dW, and four lanes 16. Sixteen rows at a time go through LDS (each wave
    // its own part of what the tiles lay in; the last barrier is behind every
    // read of them), so that a store, and a read of what is added to, covers
    // whole lines.
    constexpr int kWide = T::TN * 16, kLanes = kWide / 4, kPad = kWide + 4;
    static_assert(T::NT / 64 * 16 * kPad * sizeof(float) <= sizeof(sa), "the tiles' LDS holds 16 rows a wave");
    float* out = reinterpret_cast<float*>(&sa[0][0]) + wave * 16 * kPad;
    const int64_t n = n0 + wn + lane % kLanes * 4;
    const int left = n < a.cols ? static_cast<int>(min(a.cols - n, int64_t{4})) : 0;
    const f32x4 scale = split == 1 ? load_scale(a, n, left) : f32x4{};
#pragma unroll
    for (int i = 0; i < T::TM; ++i) {
#pragma unroll
        for (int j = 0; j < T::TN; ++j) *reinterpret_cast<f32x4*>(out + lane % 16 * kPad + 16 * j + lane / 16 * 4) = acc[j][i];
#pragma unroll
        for (int r = 0; r < 16; r += 64 / kLanes) {
            const int row = r + lane / kLanes;
            const int64_t m = m0 + wm + 16 * i + row;
            const f32x4 v = *reinterpret_cast<const f32x4*>(out + row * kPad + lane % kLanes * 4);
            if (m >= a.outs || left == 0) continue;
            if (split == 1) {
                store_dw(a, m, n, left, v, scale);
                continue;
            }
            float* p = a.part + (static_cast<int64_t>(part) * a.outs + m) * a.cols + n;
            if (left == 4) st16_a4(p, __builtin_bit_cast(u32x4, v));
            else {
#pragma unroll
                for (int c = 0; c < 3; ++c)
                    if (c < left) ((ZERO_G float*)p)[c] = v[c];
            }
        }
    }
}

// The partial products of a split sum, added in the order of the tokens. A
// workgroup's eight waves make 8 / waves sets; a set takes 64 vectors of four
// columns, each of its waves an equal share of the parts, four loads in
// flight.
constexpr int kJoinWaves = 8;

// Four parts a wave before a set gets more waves.
inline int join_waves(int split) { return split <= 4 ? 1 : split <= 8 ? 2 : split <= 16 ? 4 : kJoinWaves; }

__global__ __launch_bounds__(64 * kJoinWaves) void wgrad_join_kernel(WgradArgs a, int split, int waves, uint32_t per_row, FastDiv by_row)
{
    __shared__ f32x4 sums[kJoinWaves][64];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int set = wave / waves, member = wave % waves, sets = kJoinWaves / waves;
    const int64_t size = a.outs * a.cols, vectors = a.outs * per_row;
    const int each = (split + waves - 1) / waves;
    const int from = min(split, member * each), to = min(split, from + each);
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * sets * 64; first < vectors; first += static_cast<int64_t>(gridDim.x) * sets * 64) {
        const int64_t mine = first + set * 64 + lane, i = min(mine, vectors - 1);
        const int64_t m = vectors < (1ll << 31) ? div_by(static_cast<uint32_t>(i), by_row) : i / per_row;
        const int64_t n = (i - m * per_row) * 4;
        const int left = static_cast<int>(min(a.cols - n, int64_t{4}));
        const ZERO_G float* p = (const ZERO_G float*)a.part + from * size + m * a.cols + n;
        f32x4 s{};
        if (left == 4) {
            int k = from;
            for (; k + 4 <= to; k += 4, p += 4 * size) {
                f32x4 t[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) t[u] = __builtin_bit_cast(f32x4, ld16_a4((const float*)(p + u * size)));
#pragma unroll
                for (int u = 0; u < 4; ++u) s += t[u];
            }
            for (; k < to; ++k, p += size) s += __builtin_bit_cast(f32x4, ld16_a4((const float*)p));
        } else {
            for (int k = from; k < to; ++k, p += size)
#pragma unroll
                for (int r = 0; r < 3; ++r)
                    if (r < left) s[r] += p[r];
        }
        if (waves > 1) {
            sums[wave][lane] = s;
            __syncthreads();
            for (int w = 1; w < waves; ++w) s += sums[min(wave + w, kJoinWaves - 1)][lane];
            __syncthreads();
        }
        if (member == 0 && mine < vectors) store_dw(a, m, n, left, s, load_scale(a, n, left));
    }
}

using TileBig = Tile<256, 256, 32, 2, 4, 1>;
using TileMid = Tile<128, 128, 64, 2, 2, 2>;
using TileSmall = Tile<64, 64, 64, 2, 2, 3>;

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

// A tile shape and the time of one of its workgroups for BK tokens, alone on
// its compute unit and with the chip full of them.
struct Candidate {
    int tile, bm, bn, bk, slots;
    double alone, full;  // us
};
template <class T>
constexpr Candidate candidate(int tile, double alone, double full)
{
    return Candidate{tile, T::BM, T::BN, T::BK, T::SLOTS, alone, full};
}

}  // namespace

// The tile and the number of ranges that the tokens are cut into, by the time
// that they are expected to take: rounds of workgroups through the chip, each
// of them a start and its tokens, and for a split sum the partial products
// written, read and joined by a second launch. Measured: 8192 tokens and
// 4096 x 4096 take 211 us with 256 x 256 tiles, 290 with 128 x 128, 484 with
// 64 x 64; 1024 tokens and 768 x 768 23, 16 and 9.2 us; 30011 tokens and
// 200 x 333 unsplit 698, 420 and 218 us, split 30, 26 and 24 us.
WgradPlan wgrad_plan(int64_t rows, int64_t outs, int64_t cols)
{
    static const Candidate kTiles[] = {candidate<TileBig>(0, 0.80, 0.87), candidate<TileMid>(1, 0.95, 1.18),
                                       candidate<TileSmall>(2, 0.47, 0.76)};
    constexpr double kStart = 4.0, kJoin = 7.0, kBytes = 2e6;  // us a round, us a join, partial bytes written and read a us
    WgradPlan best{};
    double least = 0.0;
    for (const Candidate& c : kTiles) {
        const int64_t tiles = ((outs + c.bm - 1) / c.bm) * ((cols + c.bn - 1) / c.bn);
        const int64_t slots = static_cast<int64_t>(c.slots) * kComputeUnits;
        for (const int want : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64, 96, 128}) {
            if (want > 1 && rows < 128 * static_cast<int64_t>(want)) break;
            int64_t steps = ((rows + want - 1) / want + c.bk - 1) / c.bk;
            if (steps < 1) steps = 1;
            const int64_t chunk = steps * c.bk;
            const int64_t split = rows > 0 ? (rows + chunk - 1) / chunk : 1;
            const double fill = static_cast<double>(tiles * split) / static_cast<double>(slots);
            const double step = c.alone + (c.full - c.alone) * (fill < 1.0 ? fill : 1.0);
            const double bytes = split > 1 ? 4.0 * static_cast<double>(split) * static_cast<double>(outs) * static_cast<double>(cols) : 0.0;
            const double us = static_cast<double>((tiles * split + slots - 1) / slots) * (kStart + static_cast<double>(steps) * step) +
                              (split > 1 ? kJoin + bytes / kBytes : 0.0);
            if (least == 0.0 || us < least) {
                least = us;
                best = WgradPlan{c.tile, static_cast<int>(split), chunk, static_cast<size_t>(bytes)};
            }
        }
    }
    return best;
}

hipError_t launch_wgrad(const WgradArgs& a, const WgradPlan& plan, int format, hipStream_t s)
{
    const hipError_t e = plan.tile == 0   ? launch_tile<TileBig>(a, plan, format, s)
                         : plan.tile == 1 ? launch_tile<TileMid>(a, plan, format, s)
                                          : launch_tile<TileSmall>(a, plan, format, s);
    if (e != hipSuccess || plan.split == 1) return e;
    const uint32_t per_row = static_cast<uint32_t>((a.cols + 3) / 4);
    const int waves = join_waves(plan.split);
    const int64_t each = 64 * kJoinWaves / waves, blocks = (a.outs * per_row + each - 1) / each;
    const unsigned grid = static_cast<unsigned>(blocks < 8 * kComputeUnits ? blocks : 8 * kComputeUnits);
    wgrad_join_kernel<<<grid, 64 * kJoinWaves, 0, s>>>(a, plan.split, waves, per_row, fast_div(per_row));
    return hipGetLastError();
}

}  // namespace zero
