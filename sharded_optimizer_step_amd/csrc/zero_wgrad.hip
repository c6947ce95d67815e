// zero_wgrad.hip -- the weight gradient dW = dY^T X of a linear layer whose
// input X was saved in 8 bits, gfx950.
//
// Both factors have the summed index (the token) as their slow one, so both
// lie in LDS as they lie in memory, a row of a tile per token, and the
// transposing LDS reads turn 4 tokens x 16 columns into the operand layout of
// the matrix instructions. The 8-bit codes are decoded to bf16 on their way
// from memory to LDS: a power-of-two scale makes that exact, so the product
// is the bf16 one, with half the reads of X.
//
// Large products are bound by their matrix instructions (busy 56% of the
// cycles, LDS 36% with conflicts in 0.6%) and by what does not overlap with
// them: a wave decodes and stages a tile, then multiplies one, and the two
// waves of a SIMD do so nearly together; at the 2.0 to 2.1 GHz that the chip
// holds under this load. 8192 tokens: 11008 x 4096 from e4m3 to bf16 648 us
// (1.14 PFLOP/s; 2.7 rounds of tiles); 4096 x 4096 from int8, with inputs that do
// not lie in the caches, 248 us to bf16 (1.11), 255 to fp32 and 271 added to
// fp32 (1.01; 134 MB of dW read and written instead of 34 written). Small ones
// are bound by a tile's start and the latency of its steps: 192 tokens and
// 768 x 768 5.6 us.
#include "zero_act8_device.h"

namespace zero {
namespace {

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// 16 codes with one scale, as bf16.
//
// e4m3: one instruction for two codes and their scale. int8: the code with its
// sign bit turned over is u = code + 128 in 0 .. 255; under the byte 0x64 it is
// the half 1024 + u, less 1152 the code, and one mixed fma scales it, all
// without a rounding: two and three quarters instructions a code instead of
// three and a half. (One fma of 1024 + u with -1152 unit would save half of
// one, but 1152 unit overflows before the largest blocks do.)
template <int FMT>
__device__ __forceinline__ void decode16(u32x4 codes, uint32_t scale, u32x4 (&out)[2])
{
    const float unit = act8_unit(scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t lo, hi;
        if constexpr (FMT == ZERO_ACT8_E4M3) {
            lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[i], unit, false));
            hi = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[i], unit, true));
        } else {
            typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
            const uint32_t u = codes[i] ^ 0x80808080u;
            constexpr _Float16 kBack = -1152;
            const f16x2 a = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) + f16x2{kBack, kBack};
            const f16x2 b = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) + f16x2{kBack, kBack};
            lo = pack_bf16(fmaf(static_cast<float>(a.x), unit, 0.0f), fmaf(static_cast<float>(a.y), unit, 0.0f));
            hi = pack_bf16(fmaf(static_cast<float>(b.x), unit, 0.0f), fmaf(static_cast<float>(b.y), unit, 0.0f));
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
        if (left == 4) __builtin_nontemporal_store(w, (ZERO_G u32x2_a2*)p);
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

// Where tile `id` of a grid of tiles lies: it goes down 8 rows of tiles before
// it moves a tile to the right, so that neighbours share their factors.
struct TilePlace {
    int m, n;
};
__host__ __device__ inline TilePlace tile_place(int id, int tiles_m, int tiles_n)
{
    constexpr int kDown = 8;
    const int band = id / (kDown * tiles_n), in_band = id - band * kDown * tiles_n;
    const int left = tiles_m - band * kDown, rows = left < kDown ? left : kDown;
    return TilePlace{band * kDown + in_band % rows, in_band / rows};
}

template <class T, int FMT>
__global__ __launch_bounds__(T::NT, T::NT / 256 * T::SLOTS) void wgrad_kernel(WgradArgs a, int tiles_m, int tiles_n, int whole, int split,
                                                                             int64_t chunk)
{
    __shared__ __align__(16) uint16_t sa[2][T::BK * T::SA];
    __shared__ __align__(16) uint16_t sb[2][T::BK * T::SB];
    // The first `whole` workgroups take a tile each and all tokens; the tiles
    // after these are split over the tokens. Consecutive workgroups go to the
    // eight XCDs in turn: each XCD gets a run of neighbouring tiles, which share
    // their factors in its L2.
    const int rest = tiles_m * tiles_n - whole, whole_blocks = (whole + 7) / 8 * 8;
    const bool parted = static_cast<int>(blockIdx.x) >= whole_blocks;
    const int block = parted ? blockIdx.x - whole_blocks : blockIdx.x;
    const int total = parted ? rest * split : whole;
    const int each = (total + 7) / 8;
    const int id = block % 8 * each + block / 8;
    if (id >= total || block / 8 >= each) return;
    const int part = parted ? id / rest : 0;
    const int split_tile = id - part * rest;  // among the split ones
    const TilePlace place = tile_place(parted ? whole + split_tile : id, tiles_m, tiles_n);
    const int64_t m0 = static_cast<int64_t>(place.m) * T::BM, n0 = static_cast<int64_t>(place.n) * T::BN;
    const int64_t begin = parted ? part * chunk : 0, end = parted ? min(a.rows, begin + chunk) : a.rows;
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
    const bool plain = a.outs >= 8 && a.ld_dy < (int64_t{1} << 24) && a.pitch < (int64_t{1} << 25);
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
        if (shift == 0) return;
#pragma unroll
        for (int i = 0; i < T::VA; ++i) {
            uint64_t lo = ra[i].x | static_cast<uint64_t>(ra[i].y) << 32, hi = ra[i].z | static_cast<uint64_t>(ra[i].w) << 32;
            if (shift >= 4) {
                lo = hi >> (16 * (shift - 4));
                hi = 0;
            } else {
                lo = lo >> (16 * shift) | hi << (64 - 16 * shift);
                hi >>= 16 * shift;
            }
            ra[i] = u32x4{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi), static_cast<uint32_t>(hi >> 32)};
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
        if (ragged) shift_left();
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
        stage(buf ^ 1);
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
    // whole lines. The fences keep the compiler from moving a lane's reads over
    // its writes, which other lanes read; a wave's LDS accesses are in order.
    constexpr int kWide = T::TN * 16, kLanes = kWide / 4, kPad = kWide + 4;
    static_assert(T::NT / 64 * 16 * kPad * sizeof(float) <= sizeof(sa), "the tiles' LDS holds 16 rows a wave");
    float* out = reinterpret_cast<float*>(&sa[0][0]) + wave * 16 * kPad;
    const int64_t n = n0 + wn + lane % kLanes * 4;
    const int left = n < a.cols ? static_cast<int>(min(a.cols - n, int64_t{4})) : 0;
    const f32x4 scale = parted ? f32x4{} : load_scale(a, n, left);
    // a part of a split tile goes to the workspace whole
    float* to = a.part + (static_cast<int64_t>(split_tile) * split + part) * (T::BM * T::BN) + wm * T::BN + wn + lane % kLanes * 4;
#pragma unroll
    for (int i = 0; i < T::TM; ++i) {
#pragma unroll
        for (int j = 0; j < T::TN; ++j) *reinterpret_cast<f32x4*>(out + lane % 16 * kPad + 16 * j + lane / 16 * 4) = acc[j][i];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int r = 0; r < 16; r += 64 / kLanes) {
            const int row = r + lane / kLanes;
            const int64_t m = m0 + wm + 16 * i + row;
            const f32x4 v = *reinterpret_cast<const f32x4*>(out + row * kPad + lane % kLanes * 4);
            if (parted) *(ZERO_G f32x4*)(to + (16 * i + row) * T::BN) = v;
            else if (m < a.outs && left > 0) store_dw(a, m, n, left, v, scale);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// The parts of the split tiles, added in the order of the tokens. A
// workgroup's eight waves make 8 / waves sets; a set takes 64 vectors of four
// columns of a tile, each of its waves an equal share of the parts, four loads
// in flight. 24 tiles of 64 x 64 in 32 parts take 4.5 us, beside 21 for the
// parts themselves (30011 tokens, 200 x 333).
constexpr int kJoinWaves = 8;

// Four parts a wave before a set gets more waves.
inline int join_waves(int split) { return split <= 4 ? 1 : split <= 8 ? 2 : split <= 16 ? 4 : kJoinWaves; }

// BM x BN tiles, the first of them tile `whole` of the grid.
template <int BM, int BN>
__global__ __launch_bounds__(64 * kJoinWaves) void wgrad_join_kernel(WgradArgs a, int tiles_m, int tiles_n, int whole, int split, int waves)
{
    __shared__ f32x4 sums[kJoinWaves][64];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int set = wave / waves, member = wave % waves;
    const int tile = blockIdx.y, vector = (static_cast<int>(blockIdx.x) * (kJoinWaves / waves) + set) * 64 + lane;
    const int each = (split + waves - 1) / waves;
    const int from = min(split, member * each), to = min(split, from + each);
    const ZERO_G f32x4* p = (const ZERO_G f32x4*)a.part + (static_cast<int64_t>(tile) * split + from) * (BM * BN / 4) + vector;
    f32x4 s{};
    int k = from;
    for (; k + 4 <= to; k += 4, p += BM * BN) {
        f32x4 t[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) t[u] = p[u * (BM * BN / 4)];
#pragma unroll
        for (int u = 0; u < 4; ++u) s += t[u];
    }
    for (; k < to; ++k, p += BM * BN / 4) s += *p;
    if (waves > 1) {
        sums[wave][lane] = s;
        __syncthreads();
        if (member != 0) return;
        for (int w = 1; w < waves; ++w) s += sums[wave + w][lane];
    }
    const TilePlace place = tile_place(whole + tile, tiles_m, tiles_n);
    const int64_t m = static_cast<int64_t>(place.m) * BM + vector / (BN / 4), n = static_cast<int64_t>(place.n) * BN + vector % (BN / 4) * 4;
    if (m >= a.outs || n >= a.cols) return;
    const int left = static_cast<int>(min(a.cols - n, int64_t{4}));
    store_dw(a, m, n, left, s, load_scale(a, n, left));
}

using TileBig = Tile<256, 256, 32, 2, 4, 1>;
using TileMid = Tile<128, 128, 64, 2, 2, 2>;
using TileSmall = Tile<64, 64, 64, 2, 2, 3>;

template <class T>
hipError_t launch_tile(const WgradArgs& a, const WgradPlan& plan, int format, hipStream_t s)
{
    const int m = static_cast<int>((a.outs + T::BM - 1) / T::BM), n = static_cast<int>((a.cols + T::BN - 1) / T::BN);
    const int whole = static_cast<int>(plan.whole), rest = m * n - whole;
    const unsigned grid = static_cast<unsigned>((whole + 7) / 8 * 8 + (static_cast<int64_t>(rest) * plan.split + 7) / 8 * 8);
    if (format == ZERO_ACT8_E4M3) wgrad_kernel<T, ZERO_ACT8_E4M3><<<grid, T::NT, 0, s>>>(a, m, n, whole, plan.split, plan.chunk);
    else wgrad_kernel<T, ZERO_ACT8_INT8><<<grid, T::NT, 0, s>>>(a, m, n, whole, plan.split, plan.chunk);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || rest == 0 || plan.split == 1) return e;
    const int waves = join_waves(plan.split);
    const dim3 join(static_cast<unsigned>(T::BM * T::BN / 4 / 64 * waves / kJoinWaves), static_cast<unsigned>(rest));
    wgrad_join_kernel<T::BM, T::BN><<<join, 64 * kJoinWaves, 0, s>>>(a, m, n, whole, plan.split, waves);
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

// The tile shape, how many of its tiles are taken whole, and the number of
// ranges of tokens that the others are cut into, by the time that they are
// expected to take: rounds of workgroups through the chip, each of them a
// start and its tokens, and for split tiles their parts written, read and
// joined by a second launch. Either no tile is whole, or as many as fill whole
// rounds, or all. Measured: 8192 tokens and 4096 x 4096 take 240 us with
// 256 x 256 tiles, 307 with 128 x 128, 512 with 64 x 64; 1024 tokens and
// 768 x 768 33, 20 and 13 us; 30011 tokens and 200 x 333 unsplit 692, 393 and
// 254 us, split 31, 25 and 22 us; a million tokens and 64 x 64 106 us in 128
// ranges, 50 in 768.
//
// A step's times are differences of two lengths, e4m3 to bf16: one tile, and one
// as many as the chip holds. (Taken again, over 64 and 192 steps: 0.72 and 0.83,
// 0.89 and 1.10, 0.59 and 0.81 us.) The model knows nothing of the epilogue, nor
// of what the caches hold: it says 227 us of the 4096 x 4096 above and 29 of
// 30011 x 200 x 333, which take 240 and 22. It only has to order the candidates.
WgradPlan wgrad_plan(int64_t rows, int64_t outs, int64_t cols)
{
    static const Candidate kTiles[] = {candidate<TileBig>(0, 0.80, 0.87), candidate<TileMid>(1, 0.95, 1.18),
                                       candidate<TileSmall>(2, 0.47, 0.76)};
    constexpr double kStart = 4.0, kJoin = 7.0, kBytes = 2e6;  // us a round, us a join, bytes of parts written and read a us
    constexpr int64_t kMostParts = int64_t{1} << 16;  // tiles of one join (its grid's second size)
    WgradPlan best{};
    double least = -1.0;
    for (const Candidate& c : kTiles) {
        const int64_t tiles = ((outs + c.bm - 1) / c.bm) * ((cols + c.bn - 1) / c.bn);
        const int64_t slots = static_cast<int64_t>(c.slots) * kComputeUnits;
        const int64_t all_steps = rows > 0 ? (rows + c.bk - 1) / c.bk : 1;
        const auto rounds = [&](int64_t groups, int64_t steps) {
            const double fill = static_cast<double>(groups) / static_cast<double>(slots);
            const double step = c.alone + (c.full - c.alone) * (fill < 1.0 ? fill : 1.0);
            return static_cast<double>((groups + slots - 1) / slots) * (kStart + static_cast<double>(steps) * step);
        };
        const double unsplit = rounds(tiles, all_steps);
        if (least < 0.0 || unsplit < least) {
            least = unsplit;
            best = WgradPlan{c.tile, tiles, 1, all_steps * c.bk, 0};
        }
        const int64_t full_rounds = tiles / slots * slots;
        for (const int64_t whole : {int64_t{0}, full_rounds}) {
            const int64_t rest = tiles - whole;
            if (rest == 0 || rest >= kMostParts || (whole == 0 && rest > 2 * slots)) continue;
            for (const int want : {2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64, 96, 128, 192, 256, 384, 512, 768}) {
                if (rows < 128 * static_cast<int64_t>(want)) break;
                const int64_t steps = (all_steps + want - 1) / want;
                const int64_t split = (all_steps + steps - 1) / steps;
                const double bytes = 4.0 * static_cast<double>(rest * split) * c.bm * c.bn;
                const double us = (whole > 0 ? rounds(whole, all_steps) : 0.0) + rounds(rest * split, steps) + kJoin + bytes / kBytes;
                if (us < least) {
                    least = us;
                    best = WgradPlan{c.tile, whole, static_cast<int>(split), steps * c.bk, static_cast<size_t>(bytes)};
                }
            }
            if (full_rounds == 0) break;
        }
    }
    return best;
}

hipError_t launch_wgrad(const WgradArgs& a, const WgradPlan& plan, int format, hipStream_t s)
{
    return plan.tile == 0   ? launch_tile<TileBig>(a, plan, format, s)
           : plan.tile == 1 ? launch_tile<TileMid>(a, plan, format, s)
                            : launch_tile<TileSmall>(a, plan, format, s);
}

}  // namespace zero
