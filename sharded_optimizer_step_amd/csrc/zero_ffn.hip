// zero_ffn.hip -- the products of the gated feed-forward block, gfx950:
// forward both projections with the activation, backward the gradient of the
// input and those of the two weights.
//
// All three are sums of bf16 products over tiles in LDS, one kernel for each.
// Where the summed index is a factor's fast one (h and the weights forward,
// dgate and dup for dh) its tile has rows of 64 summed elements and a lane
// reads 8 of them at once; where it is the slow one (the weights for dh, both
// factors of the weight gradients) the tile lies as in memory and the
// transposing LDS reads turn it.
//
// Many rows are bound by the matrix instructions, and at 68 to 72% of their
// cycles by the chip's power. 8192 rows x 4096 x 11008 (1.48 TFLOP each), the
// median of nine profiled launches and their least: forward 1.38 and 1.22 ms
// (1.07 and 1.21 PFLOP/s; 1.17 to 1.21 ms a call in a row), dh 1.09 and 1.07 (1.35
// and 1.38), both weight gradients 1.20 and 1.16 (1.23 and 1.27); a library's plain
// products of these sizes reach 1.24 to 1.57. Few rows are bound by reading the
// weights: one row 44 and 40 us, 180 MB at 4.1 and 4.5 TB/s (reads reach 7.0): 172
// workgroups leave a third of the chip without one. Small products are bound by
// latency: 192 x 768 x 2048 forward 9.3 and 9.2 us.
#include <type_traits>
#include <utility>

#include "zero_act8_device.h"

namespace zero {
namespace {

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
#define ZERO_L __attribute__((address_space(3)))

constexpr int BK = 32;  // summed elements of a step

// ------------------------------------------------------------------ activations

// The forms of a kernel whose instructions all waves fetch: short, without
// branches. 1 / (1 + exp(-x)), within 3 units of its last place and |x| 2^-24 of itself
// (what is made of it is rounded to bf16 or 8 bits). For large |x| the
// exponential is infinite or 0, and the result the limit.
__device__ __forceinline__ float logistic(float x)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.44269504f));
}

// f = act(f) u for 8 values, all of them at once: their exponentials and
// reciprocals do not wait for each other.
__device__ __forceinline__ void gated(int act, float (&f)[8], const float (&u)[8])
{
    float p[8];
    if (act == ZERO_FFN_SILU) {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = logistic(f[i]);
    } else if (act == ZERO_FFN_GELU) {
        // erfc(x) for x >= 0 as exp(-x^2) times a polynomial of 1 / (1 + p x), within 1.5e-7 (Abramowitz and Stegun, 7.1.26)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = fabsf(f[i]) * 0.70710678f, t = __builtin_amdgcn_rcpf(fmaf(0.3275911f, x, 1.0f));
            const float poly = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f), -0.284496736f), 0.254829592f);
            const float half = 0.5f * poly * __builtin_amdgcn_exp2f(x * x * -1.44269504f);
            p[i] = f[i] > 0.0f ? 1.0f - half : half;
        }
    } else {  // (1 + tanh(z)) / 2 is the logistic function of 2 z
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = logistic(1.59576912f * fmaf(0.044715f * f[i] * f[i], f[i], f[i]));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = f[i] * p[i] * u[i];
}

// ------------------------------------------------------------------ tiles in LDS

// BM x BN tile of the output, WM x WN waves, DEPTH steps in LDS, SLOTS
// workgroups a compute unit.
template <int BM_, int BN_, int WM_, int WN_, int DEPTH_, int SLOTS_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, DEPTH = DEPTH_, SLOTS = SLOTS_;
    static constexpr int NT = 64 * WM * WN;
    static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;  // 16 x 16 pieces of a wave
    static constexpr int kWavesASimd = NT * SLOTS > 256 ? NT * SLOTS / 256 : 1;
};

// A tile of SIZE rows or columns of a factor and BK elements of the summed
// index. ALONG: the summed index runs along its rows, of 64 bytes; otherwise
// across them, of 2 SIZE bytes.
//
// Tiles go from memory to LDS without passing through registers, a wave's 64
// units of 16 bytes one after the other, so they cannot be padded. The units
// are permuted within their rows instead. ALONG: four rows are one span of the
// 64 banks, and a read is served in four parts of 16 lanes, lanes 0 .. 3, 12 ..
// 15 and 20 .. 27 of 32 or the others: with the rows' units permuted by 0, 2, 3,
// 1 for each four rows, and so 16 neighbouring lanes too, they lie apart. Across: 32 lanes of a transposing read take 32 bytes, two
// units, of rows 0 .. 3 and 8 .. 11 of 16 (or the others), whose pairs of units
// are permuted by eight different numbers.
template <bool ALONG, int SIZE, int NT>
struct Factor {
    static constexpr int kRowBytes = ALONG ? BK * 2 : SIZE * 2;
    static constexpr int kUnits = kRowBytes / 16;             // of a row
    static constexpr int kVecs = SIZE * BK * 2 / 16 / NT;     // units a thread loads
    static constexpr int kStep = NT / kUnits;                 // rows from one of them to the next
    static_assert(SIZE * BK * 2 / 16 % NT == 0 && NT % kUnits == 0, "every thread loads as many units, at one place of their rows");
    static_assert(ALONG || SIZE >= 128, "eight pairs of units");

    static __device__ __forceinline__ int place(int row, int unit)
    {
        return ALONG ? unit ^ ((row >> 2 ^ row >> 3) & 1) << 1 ^ (row >> 3 & 1) : unit ^ ((row & 3) << 1 | (row >> 3 & 1) << 3);
    }
};

// The elements from `shift` on, and zeros.
__device__ __forceinline__ u32x4 shift_unit(u32x4 v, int shift)
{
    uint64_t lo = v.x | static_cast<uint64_t>(v.y) << 32, hi = v.z | static_cast<uint64_t>(v.w) << 32;
    if (shift >= 4) {
        lo = hi >> (16 * (shift - 4));
        hi = 0;
    } else if (shift > 0) {
        lo = lo >> (16 * shift) | hi << (64 - 16 * shift);
        hi >>= 16 * shift;
    }
    return u32x4{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi), static_cast<uint32_t>(hi >> 32)};
}

// Elements col .. col + 7 of a row of `limit` elements, zeros beyond it.
__device__ __forceinline__ u32x4 load_unit(const uint16_t* row, int64_t col, int64_t limit)
{
    const int64_t left = limit - col;
    if (left >= 8) return ld16_a2(row + col);
    if (left <= 0) return u32x4{};
    if (limit >= 8) return shift_unit(ld16_a2(row + limit - 8), static_cast<int>(8 - left));
    u32x4 v{};
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < left) v[i / 2] |= static_cast<uint32_t>(((const ZERO_G uint16_t*)row)[col + i]) << (16 * (i % 2));
    return v;
}

// A raw buffer of 2 GiB from p on; loads from offsets beyond it give zeros.
__device__ __forceinline__ i32x4 buffer_at(const uint16_t* p)
{
    const uint64_t at = reinterpret_cast<uint64_t>(p);
    return i32x4{static_cast<int>(at), static_cast<int>(at >> 32 & 0xFFFF), static_cast<int>(0x80000000u), 0x00020000};
}
constexpr uint32_t kBeyond = 0xFFFFFF00u;

// 16 bytes a lane from `offset` of a buffer to LDS, a wave's 64 units one after
// the other from base + TO on. An instruction that the compiler does not look into:
// it would have every transposing read wait for all loads to LDS. The waits
// are those of the waves' meetings.
template <int TO>
__device__ __forceinline__ void load_to_lds(i32x4 buffer, uint32_t offset, uint32_t base)
{
    asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 : : "s"(base), "v"(offset), "s"(buffer), "n"(TO) : "memory", "scc", "m0");
}

// 8 summed elements for this lane's row or column of a piece of 16, from a tile
// in LDS; `at` is the lane's own place in it, see lane_place.
template <bool ALONG, int ROW_BYTES>
__device__ __forceinline__ i32x4 read_piece(const char* at)
{
    if constexpr (ALONG) {
        return *reinterpret_cast<const i32x4*>(at);
    } else {
        const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZERO_L i16x4*)at);
        const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZERO_L i16x4*)(at + 4 * ROW_BYTES));
        return __builtin_bit_cast(i32x4, (i16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
}

// sum += b a for a piece of 16 x 16, in place. The compiler's own form of the
// instruction may write its sum to other registers than it reads it from, and
// where its surroundings are held in an order, as below, it then moves and
// spills sums. It does not look into this one and so waits for nothing on its
// behalf: not for a vector instruction that wrote an operand within the two
// instructions before (there are none: operands come from LDS, a test of the
// assembly says so), nor for what reads the sums after the last one: settle().
__device__ __forceinline__ void add_product(f32x4& sum, i32x4 b, i32x4 a)
{
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(sum) : "v"(b), "v"(a));
}
template <int N>
__device__ __forceinline__ void settle(f32x4 (&sums)[N])
{
    asm volatile("s_nop 15\n\ts_nop 15");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+a"(sums[i]));
}

// f(0), f(1), .. f(N - 1) with numbers that are constants.
template <class F, int... I>
__device__ __forceinline__ void unrolled_of(F&& f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void unrolled(F&& f)
{
    unrolled_of(f, std::make_integer_sequence<int, N>{});
}

// Where tile `id` of a grid of tiles lies: it goes down 8 rows of tiles before
// it moves a tile to the right, so that neighbours share their factors.
struct TilePlace {
    int m, n;
};
__device__ __forceinline__ TilePlace tile_place(int id, int tiles_m, int tiles_n)
{
    constexpr int kDown = 8;
    const int band = id / (kDown * tiles_n), in_band = id - band * kDown * tiles_n;
    const int left = tiles_m - band * kDown, rows = left < kDown ? left : kDown;
    return TilePlace{band * kDown + in_band % rows, in_band / rows};
}

// ------------------------------------------------------------------ results

// 8 neighbouring values of a result row, columns n .. n + left - 1. Forward: f
// is gate and u up.
template <FfnKind KIND>
__device__ __forceinline__ void finish(const FfnArgs& a, int which, int64_t m, int64_t n, int left, float (&f)[8], float (&u)[8])
{
    if constexpr (KIND == kFfnForward) {
        if (a.ckpt[0] != nullptr || a.ckpt[1] != nullptr) {
            const int64_t pitch = act8_pitch(a.hidden);
#pragma unroll
            for (int i = 0; i < 8; ++i) {  // beyond the last column a tile holds other ones
                if (i >= left) f[i] = u[i] = 0.0f;
            }
            const auto save = [&](uint8_t* ckpt, const float (&x)[8]) {
                if (ckpt == nullptr) return;
                const Code8 c = a.format == ZERO_ACT8_E4M3 ? encode8<ZERO_ACT8_E4M3>(x) : encode8<ZERO_ACT8_INT8>(x);
                if (n >= pitch) return;
                *(ZERO_G u32x2*)(ckpt + m * pitch + n) = c.codes;
                if (n % kActBlock == 0) *(ZERO_G uint8_t*)(ckpt + a.rows * pitch + (m * pitch + n) / kActBlock) = static_cast<uint8_t>(c.scale);
            };
            save(a.ckpt[0], f);
            save(a.ckpt[1], u);
        }
        if (left <= 0) return;
        if (a.out[0].p != nullptr) store8<false, true>(a.out[0], m, n, left, f);
        if (a.out[1].p != nullptr) store8<false, true>(a.out[1], m, n, left, u);
        gated(a.act, f, u);
        store8<false, true>(a.a, m, n, left, f);
    } else {
        if (left <= 0) return;
        const Rows& to = a.out[which];
        if (!to.f32) {
            store8<false, true>(to, m, n, left, f);
            return;
        }
        if (a.accumulate) {
            float old[8];
            unpack<true>(load8<true, true>(to, m, n, left), n, left, old);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] += old[i];
        }
        store8<true, true>(to, m, n, left, f);
    }
}

// What a product sums: its output is m x n, its summed index `k` long, in
// `segments` one after the other (dh is the sum of two products). The weight
// gradients are two outputs, one under the other, whose rows of tiles do not
// meet.
template <class T, FfnKind KIND>
struct Shape {
    static constexpr int kCols = KIND == kFfnForward ? T::BN / 2 : T::BN;  // columns of a tile: forward, of gate and as many of up
    static __host__ __device__ int64_t m(const FfnArgs& a) { return KIND == kFfnWeight ? a.hidden : a.rows; }
    static __host__ __device__ int64_t n(const FfnArgs& a) { return KIND == kFfnForward ? a.hidden : a.cols; }
    static __host__ __device__ int64_t k(const FfnArgs& a) { return KIND == kFfnForward ? a.cols : KIND == kFfnInput ? a.hidden : a.rows; }
};

template <class T, FfnKind KIND, bool FAST>
__global__ __launch_bounds__(T::NT, T::kWavesASimd) void ffn_kernel(FfnArgs a, int tiles_m, int tiles_n, int whole)
{
    using S = Shape<T, KIND>;
    constexpr bool kAlongA = KIND != kFfnWeight, kAlongB = KIND == kFfnForward;
    using A = Factor<kAlongA, T::BM, T::NT>;
    using B = Factor<kAlongB, T::BN, T::NT>;
    constexpr int kDepth = T::DEPTH;
    __shared__ __align__(16) char tiles[kDepth][(T::BM + T::BN) * BK * 2];

    // The first `whole` workgroups take a tile each and all of the summed index;
    // the tiles after these are split over it. Consecutive workgroups go to the
    // eight XCDs in turn: each XCD gets a run of neighbouring tiles.
    const int rest = tiles_m * tiles_n - whole, whole_blocks = (whole + 7) / 8 * 8;
    const bool parted = static_cast<int>(blockIdx.x) >= whole_blocks;
    const int block = parted ? blockIdx.x - whole_blocks : blockIdx.x;
    const int total = parted ? rest * a.split : whole;
    const int each = (total + 7) / 8;
    const int id = block % 8 * each + block / 8;
    if (id >= total || block / 8 >= each) return;
    const int part = parted ? id / rest : 0;
    const int split_tile = id - part * rest;  // among the split ones
    const TilePlace place = tile_place(parted ? whole + split_tile : id, tiles_m, tiles_n);
    const int which = KIND == kFfnWeight && a.outputs == 2 && place.m >= tiles_m / 2 ? 1 : 0;
    const int64_t m0 = static_cast<int64_t>(place.m - which * (tiles_m / 2)) * T::BM, n0 = static_cast<int64_t>(place.n) * S::kCols;
    const int64_t m_end = S::m(a), n_end = S::n(a), k_end = S::k(a);
    const int64_t seg_steps = (k_end + BK - 1) / BK;
    const int64_t all_steps = KIND == kFfnInput ? 2 * seg_steps : seg_steps;
    const int64_t begin = parted ? part * a.chunk : 0, end = parted ? min(all_steps, begin + a.chunk) : all_steps;

    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / 64), lane = tid % 64;

    // The units that this thread loads: one place of a row, every kStep-th row.
    const int row_a = tid / A::kUnits, row_b = tid / B::kUnits;
    const auto unit_a = [&](int i) { return A::place(row_a + i * A::kStep, tid % A::kUnits); };
    const auto unit_b = [&](int i) { return B::place(row_b + i * B::kStep, tid % B::kUnits); };
    // forward the second half of B's rows are those of up
    constexpr int kHalfB = KIND == kFfnForward ? B::kVecs / 2 : B::kVecs;
    // Rows beyond the last one are read as the last one, columns as the last
    // eight (which is where a unit that ends beyond them lies, moved into place
    // by `shift` elements): products of what is beyond are not stored. Offsets
    // are from eight elements before a tile, so that none is negative. (An aligned
    // factor's rows hold whole units: what a copy has beyond its columns are zeros.)
    const auto held = [](int64_t columns) { return FAST ? (columns + 7) / 8 * 8 : columns; };
    uint32_t off_a[A::kVecs], off_b[B::kVecs];
#pragma unroll
    for (int i = 0; i < A::kVecs; ++i) {
        const int64_t ld = KIND == kFfnForward ? a.ld_h : a.ld_d[which];
        const int64_t row = kAlongA ? min(static_cast<int64_t>(row_a + i * A::kStep), m_end - 1 - m0) : row_a + i * A::kStep;
        const int64_t col = kAlongA ? unit_a(i) * 8 : min(static_cast<int64_t>(unit_a(i) * 8), held(m_end) - 8 - m0);
        off_a[i] = static_cast<uint32_t>((row * ld + col + 8) * 2);
    }
#pragma unroll
    for (int i = 0; i < B::kVecs; ++i) {
        const int64_t ld = KIND == kFfnWeight ? a.ld_h : a.ld_w[KIND == kFfnForward && i >= kHalfB ? 1 : 0];
        const int r = row_b + i % kHalfB * B::kStep;
        const int64_t row = kAlongB ? min(static_cast<int64_t>(r), n_end - 1 - n0) : r;
        const int64_t col = kAlongB ? unit_b(i) * 8 : min(static_cast<int64_t>(unit_b(i) * 8), held(n_end) - 8 - n0);
        off_b[i] = static_cast<uint32_t>((row * ld + col + 8) * 2);
    }
    const auto shift_of = [](int64_t over) { return over > 0 && over < 8 ? static_cast<int>(over) : 0; };
    // (read once: not in every step, whose waits would then wait for them)
    const uint16_t* const d_which = a.d[which];
    const int64_t ld_which = a.ld_d[which];
    struct Step {
        const uint16_t *a, *b0, *b1;
        int64_t left;  // summed elements from this step on
    };
    const auto step_at = [&](int64_t s) {
        const int seg = KIND == kFfnInput && s >= seg_steps ? 1 : 0;
        const int64_t k0 = (s - seg * seg_steps) * BK;
        Step t;
        t.left = k_end - k0;
        if constexpr (KIND == kFfnForward) {
            t.a = a.h + m0 * a.ld_h + k0;
            t.b0 = a.w[0] + n0 * a.ld_w[0] + k0;
            t.b1 = a.w[1] + n0 * a.ld_w[1] + k0;
        } else if constexpr (KIND == kFfnInput) {
            t.a = a.d[seg] + m0 * a.ld_d[seg] + k0;
            t.b0 = t.b1 = a.w[seg] + k0 * a.ld_w[seg] + n0;
        } else {
            t.a = d_which + k0 * ld_which + m0;
            t.b0 = t.b1 = a.h + k0 * a.ld_h + n0;
        }
        return t;
    };
    // The step whose tiles are sent next, straight to LDS. (In the last one of a
    // sum, elements beyond it are read from beyond the buffer: zeros.)
    constexpr int kLoads = A::kVecs + B::kVecs;
    struct Cursor {
        const uint16_t *a, *b0, *b1;
        int64_t left, to_switch;  // summed elements left in this sum; steps to the second sum
    } cursor;
    const int64_t step_a = kAlongA ? BK : BK * (KIND == kFfnWeight ? ld_which : a.ld_d[0]);
    const int64_t step_b = kAlongB ? BK : BK * (KIND == kFfnWeight ? a.ld_h : a.ld_w[0]);
    const auto point_at = [&](int64_t s) {
        const Step t = step_at(s);
        cursor = Cursor{t.a - 8, t.b0 - 8, t.b1 - 8, t.left, seg_steps - s};
    };
    const auto advance = [&] {
        cursor.a += step_a;
        cursor.b0 += step_b;
        cursor.b1 += step_b;
        cursor.left -= BK;
        if constexpr (KIND == kFfnInput) {
            if (--cursor.to_switch == 0) point_at(seg_steps);
        }
    };
    const uint32_t lds_base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((ZERO_L char*)&tiles[0][0])) + wave * 1024;
    // load L of a step to slot U of the ring; WHOLE: none of it is beyond the sum
    const auto send_one = [&](auto slot, auto number, auto whole_step) {
        constexpr int U = decltype(slot)::value, L = decltype(number)::value;
        constexpr bool WHOLE = decltype(whole_step)::value;
        constexpr int kSlot = U * (T::BM + T::BN) * BK * 2;
        if constexpr (L < A::kVecs) {
            const uint32_t off = WHOLE || (kAlongA ? unit_a(L) * 8 : row_a + L * A::kStep) < cursor.left ? off_a[L] : kBeyond;
            load_to_lds<kSlot + L * T::NT * 16>(buffer_at(cursor.a), off, lds_base);
        } else {
            constexpr int I = L - A::kVecs;
            const uint32_t off = WHOLE || (kAlongB ? unit_b(I) * 8 : row_b + I * B::kStep) < cursor.left ? off_b[I] : kBeyond;
            load_to_lds<kSlot + T::BM * BK * 2 + I * T::NT * 16>(buffer_at(I < kHalfB ? cursor.b0 : cursor.b1), off, lds_base);
        }
    };
    const auto send = [&](auto slot) {
        unrolled<kLoads>([&](auto l) { send_one(slot, l, std::false_type{}); });
        advance();
    };
    // Or through registers, where the rows of an operand do not all lie on 16
    // bytes: two steps' units, so that their loads are in flight as long.
    struct Units {
        u32x4 a[A::kVecs], b[B::kVecs];
    };
    // Steps that are whole go with their loads in flight over a step.
    const auto in_flight = [&](int64_t left) { return a.plain != 0 && left >= BK; };
    const auto fetch = [&](int64_t s, Units& v) {
        const Step t = step_at(s);
        if (!in_flight(t.left)) return;
        const char *pa = reinterpret_cast<const char*>(t.a - 8), *pb0 = reinterpret_cast<const char*>(t.b0 - 8), *pb1 = reinterpret_cast<const char*>(t.b1 - 8);
#pragma unroll
        for (int i = 0; i < A::kVecs; ++i) v.a[i] = ld16_a2(pa + off_a[i]);
#pragma unroll
        for (int i = 0; i < B::kVecs; ++i) v.b[i] = ld16_a2((i < kHalfB ? pb0 : pb1) + off_b[i]);
    };
    // What fetch(s) read, to its tiles; or the step's units one after the other, each no further than its row goes.
    const auto stage = [&](int64_t s, Units& v, char* to) {
        const Step t = step_at(s);
        char* to_b = to + T::BM * BK * 2;
        if (in_flight(t.left)) {
            if (!kAlongA && m0 + T::BM > m_end) {
#pragma unroll
                for (int i = 0; i < A::kVecs; ++i) v.a[i] = shift_unit(v.a[i], shift_of(unit_a(i) * 8 - (m_end - 8 - m0)));
            }
            if (!kAlongB && n0 + S::kCols > n_end) {
#pragma unroll
                for (int i = 0; i < B::kVecs; ++i) v.b[i] = shift_unit(v.b[i], shift_of(unit_b(i) * 8 - (n_end - 8 - n0)));
            }
#pragma unroll
            for (int i = 0; i < A::kVecs; ++i) *reinterpret_cast<u32x4*>(to + (i * T::NT + tid) * 16) = v.a[i];
#pragma unroll
            for (int i = 0; i < B::kVecs; ++i) *reinterpret_cast<u32x4*>(to_b + (i * T::NT + tid) * 16) = v.b[i];
            return;
        }
        const int seg = KIND == kFfnInput && s >= seg_steps ? 1 : 0;
#pragma unroll 1
        for (int i = 0; i < A::kVecs; ++i) {
            const int row = row_a + i * A::kStep;
            const int64_t ld = KIND == kFfnForward ? a.ld_h : a.ld_d[KIND == kFfnInput ? seg : which];
            u32x4 v{};
            if (row < (kAlongA ? m_end - m0 : t.left)) v = load_unit(t.a + row * ld, unit_a(i) * 8, kAlongA ? t.left : m_end - m0);
            *reinterpret_cast<u32x4*>(to + (i * T::NT + tid) * 16) = v;
        }
#pragma unroll 1
        for (int i = 0; i < B::kVecs; ++i) {
            const int up = i < kHalfB ? 0 : 1, row = row_b + (i - up * kHalfB) * B::kStep;
            const int64_t ld = KIND == kFfnWeight ? a.ld_h : a.ld_w[KIND == kFfnInput ? seg : up];
            u32x4 v{};
            if (row < (kAlongB ? n_end - n0 : t.left)) v = load_unit((up ? t.b1 : t.b0) + row * ld, unit_b(i) * 8, kAlongB ? t.left : n_end - n0);
            *reinterpret_cast<u32x4*>(to_b + (i * T::NT + tid) * 16) = v;
        }
    };

    // Where this lane reads. The four groups of 16 lanes take summed elements 8 g
    // .. 8 g + 7 of 32. ALONG, a lane reads them of row lane % 16 of a piece;
    // across, the 16 lanes of a group read 4 elements' rows, 4 columns a lane, and
    // get a column of all 4 each. There the lane's part of the address and the
    // piece's meet by exclusive or in the bits that are permuted.
    const int wm = wave / T::WN, wn = wave % T::WN, group = lane / 16, in_group = lane % 16;
    const int across_row = 8 * group + in_group / 4;
    constexpr int kColsB = S::kCols / T::WN;  // forward a wave's first pieces are of gate, the others of as many columns of up
    uint32_t at_a, at_b;  // of piece 0
    if constexpr (kAlongA) at_a = (wm * (T::BM / T::WM) + in_group) * A::kRowBytes + A::place(in_group, group) * 16;
    else at_a = across_row * A::kRowBytes + A::place(across_row, wm * (T::BM / T::WM) / 8) * 16 + in_group % 4 * 8;
    if constexpr (kAlongB) at_b = (wn * kColsB + in_group) * B::kRowBytes + B::place(in_group, group) * 16;
    else at_b = across_row * B::kRowBytes + B::place(across_row, wn * kColsB / 8) * 16 + in_group % 4 * 8;
    f32x4 acc[T::TN][T::TM];
#pragma unroll
    for (int j = 0; j < T::TN; ++j)
#pragma unroll
        for (int i = 0; i < T::TM; ++i) {
            acc[j][i] = f32x4{};
            asm volatile("" : "+a"(acc[j][i]));
        }
    // The pieces of the factor of which a wave has few are read first; those of
    // the other are multiplied with them one after the other, in the order in
    // which the next step's are read.
    constexpr bool kManyB = T::TN > T::TM;
    constexpr int kMany = kManyB ? T::TN : T::TM, kFew = kManyB ? T::TM : T::TN, kProducts = kMany * kFew;
    struct Pieces {
        i32x4 few[kFew], many[kMany];
    };
    const auto read_a = [&](const char* from, int i) {
        if constexpr (kAlongA) return read_piece<true, A::kRowBytes>(from + at_a + 16 * i * A::kRowBytes);
        else return read_piece<false, A::kRowBytes>(from + (at_a ^ i * 32));
    };
    const auto read_b = [&](const char* from, int j) {
        from += T::BM * BK * 2;
        if constexpr (kAlongB) {
            const int row = 16 * j + (KIND == kFfnForward && j >= T::TN / 2 ? T::BN / 2 - T::TN * 8 : 0);
            return read_piece<true, B::kRowBytes>(from + at_b + row * B::kRowBytes);
        } else return read_piece<false, B::kRowBytes>(from + (at_b ^ j * 32));
    };
    const auto read_one = [&](Pieces& h, const char* from, int q) {
        // (kept from the compiler where it would hold the address of every piece in a register that it lacks)
        if constexpr (T::kWavesASimd > 1) asm volatile("" : "+v"(at_a), "+v"(at_b));
        if (q < kFew) h.few[q] = kManyB ? read_a(from, q) : read_b(from, q);
        else h.many[q - kFew] = kManyB ? read_b(from, q - kFew) : read_a(from, q - kFew);
    };
    const auto read = [&](Pieces& h, const char* from) {
#pragma unroll
        for (int q = 0; q < kFew + kMany; ++q) read_one(h, from, q);
    };
    const auto multiply_one = [&](const Pieces& h, int t) {
        const int x = t / kFew, y = t % kFew;
        if (kManyB) add_product(acc[x][y], h.many[x], h.few[y]);
        else add_product(acc[y][x], h.few[y], h.many[x]);
    };
    const auto multiply = [&](const Pieces& h) { unrolled<kProducts>([&](auto t) { multiply_one(h, t); }); };
    // The waves meet: all reads of LDS are done, and writes, and all loads to LDS
    // but those of the last LATER steps that were sent.
    const auto meet = [&](auto later) {
        constexpr int kPending = FAST ? decltype(later)::value * kLoads : 63;
        static_assert(kPending < 64, "the counter has six bits");
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt vmcnt(%0)" : : "n"(kPending) : "memory");
        __builtin_amdgcn_s_waitcnt(15 | 7 << 4 | 3 << 14);  // lgkmcnt(0) alone
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    // A step, whose pieces are in registers or on their way there. Once they have
    // come, in every wave, the step's tiles are free for the step kDepth later,
    // and the next step's tiles have arrived: its pieces are read while this
    // step's are multiplied. A load to LDS is in flight for kDepth - 1 steps.
    // u: the step's number modulo kDepth and 2.
    Pieces p[2];
    Units v[2];
    constexpr int kUnroll = kDepth % 2 ? 2 * kDepth : kDepth;
    const auto step = [&](int64_t s, auto u) {
        if (s + kDepth <= end) meet(std::integral_constant<int, kDepth - 2>{});
        else meet(std::integral_constant<int, 0>{});
        if constexpr (FAST) {
            if (s + kDepth < end) send(std::integral_constant<int, u % kDepth>{});
        } else {
            if (s + 2 < end) stage(s + 2, v[u % 2], tiles[u % 2]);
            if (s + 4 < end) fetch(s + 4, v[u % 2]);
        }
        if (s + 1 < end) read(p[(u + 1) % 2], tiles[(u + 1) % kDepth]);
        multiply(p[u % 2]);
    };
    static_assert(FAST || kDepth == 2, "through registers two steps lie in LDS");
    if (begin < end) {
        if constexpr (FAST) {
            point_at(begin);
            unrolled<kDepth>([&](auto u) {
                if (begin + u < end) send(u);
            });
            if (begin + kDepth <= end) meet(std::integral_constant<int, kDepth - 1>{});
            else meet(std::integral_constant<int, 0>{});
        } else {
            fetch(begin, v[0]);
            stage(begin, v[0], tiles[0]);
            if (begin + 1 < end) {
                fetch(begin + 1, v[1]);
                stage(begin + 1, v[1], tiles[1]);
            }
            if (begin + 2 < end) fetch(begin + 2, v[0]);
            if (begin + 3 < end) fetch(begin + 3, v[1]);
            meet(std::integral_constant<int, 0>{});
        }
        read(p[0], tiles[0]);
    }
    // Before which product a piece of the next step is read: the few and the first
    // two of the many at once, each other one when an earlier one's products have
    // freed as many registers; and the loads are sent evenly among them. (Products are
    // in the order that they are written in, and reads and loads stay between
    // them. Left to itself the compiler reads as late as it can, to save
    // registers, and the waves then meet waiting.)
    constexpr int kFirst = kFew + 2;
    constexpr auto read_at = [](int q) { return q < kFirst ? q * 2 * kFew / kFirst : 2 * kFew + (q - kFirst) * (kFew > 1 ? kFew - 1 : 1); };
    constexpr auto send_at = [](int l) { return (2 * l + 1) * kProducts / (2 * kLoads); };
    int64_t s = begin;
    if constexpr (FAST) {
        // Steps in which nothing is asked, up to one that sends one that is not whole.
        const int64_t asked = k_end % BK == 0 ? end : KIND == kFfnInput ? min(end, seg_steps - 1) : min(end, all_steps - 1);
        for (; s + kUnroll + kDepth <= asked; s += kUnroll) {
            unrolled<kUnroll>([&](auto u) {
                meet(std::integral_constant<int, kDepth - 2>{});
                unrolled<kProducts>([&](auto t) {
                    unrolled<kFew + kMany>([&](auto q) {
                        if constexpr (read_at(q) == t) read_one(p[(u + 1) % 2], tiles[(u + 1) % kDepth], q);
                    });
                    unrolled<kLoads>([&](auto l) {
                        if constexpr (send_at(l) == t) send_one(std::integral_constant<int, u % kDepth>{}, l, std::true_type{});
                    });
                    multiply_one(p[u % 2], t);
                });
                advance();
            });
        }
    }
    for (; s < end; s += kUnroll) {
        unrolled<kUnroll>([&](auto u) {
            if (s + u < end) step(s + u, u);
        });
    }
    // the last step's tiles are read, in every wave, since its meeting
#pragma unroll
    for (int j = 0; j < T::TN; ++j) settle(acc[j]);

    // B is the first operand, so a lane holds four neighbouring columns of one
    // row of the output. Sixteen rows and more at a time go through LDS (each wave
    // its own part of what the tiles lay in; the last barrier is behind every read
    // of them), after which a lane has eight neighbouring columns, forward of gate
    // and of up, and eight lanes whole lines. The fences keep the compiler from
    // moving a lane's reads over its writes, which other lanes read; a wave's LDS
    // accesses are in order.
    //
    // The code of the results stands here once, in a loop, and the sums move up to
    // the pieces that it takes: written out for every piece it is run once a tile
    // and its instructions come from memory each time (25 us a tile instead of 7).
    constexpr int kWide = T::TN * 16, kOut = KIND == kFfnForward ? kWide / 2 : kWide, kLanes = kOut / 8, kPad = kWide + 4;
    constexpr int kRoom = sizeof(tiles) / (T::NT / 64) / (16 * kPad * 4);  // pieces of 16 rows
    constexpr int kAtOnce = kRoom >= T::TM ? T::TM : kRoom >= 2 && T::TM % 2 == 0 ? 2 : 1;
    static_assert(KIND != kFfnForward || kOut % kActBlock == 0, "a block of 32 columns lies in one wave");
    static_assert(kRoom >= 1, "LDS holds 16 rows of every wave");
    float* out = reinterpret_cast<float*>(&tiles[0][0]) + wave * kAtOnce * 16 * kPad;
    const int64_t n = n0 + wn * kOut + lane % kLanes * 8;
    const int left = static_cast<int>(min(n_end - n, int64_t{8}));
    const int part_col = wn * kOut + lane % kLanes * 8;
    float* const part_tile = a.part + (static_cast<int64_t>(split_tile) * a.split + part) * (T::BM * T::BN) + part_col;
#pragma unroll 1
    for (int first = wm * (T::BM / T::WM); first < (wm + 1) * (T::BM / T::WM); first += 16 * kAtOnce) {
        unrolled<kAtOnce>([&](auto i) {
            unrolled<T::TN>([&](auto j) {
                *reinterpret_cast<f32x4*>(out + (16 * i + in_group) * kPad + 16 * j + group * 4) = acc[j][i];
            });
        });
        unrolled<T::TM - kAtOnce>([&](auto i) { unrolled<T::TN>([&](auto j) { acc[j][i] = acc[j][i + kAtOnce]; }); });
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll 1
        for (int row = lane / kLanes; row < 16 * kAtOnce; row += 64 / kLanes) {
            const int64_t m = m0 + first + row;
            if (m >= m_end) break;  // whole rows
            float f[8], u[8] = {};
            const float* from = out + row * kPad + lane % kLanes * 8;
#pragma unroll
            for (int c = 0; c < 8; c += 4) {
                *reinterpret_cast<f32x4*>(f + c) = *reinterpret_cast<const f32x4*>(from + c);
                if constexpr (KIND == kFfnForward) *reinterpret_cast<f32x4*>(u + c) = *reinterpret_cast<const f32x4*>(from + kOut + c);
            }
            if (parted) {
                float* to = part_tile + (first + row) * T::BN;
#pragma unroll
                for (int c = 0; c < 8; c += 4) {
                    *(ZERO_G f32x4*)(to + c) = *reinterpret_cast<f32x4*>(f + c);
                    if constexpr (KIND == kFfnForward) *(ZERO_G f32x4*)(to + T::BN / 2 + c) = *reinterpret_cast<f32x4*>(u + c);
                }
            } else {
                finish<KIND>(a, which, m, n, left, f, u);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// The parts of the split tiles, added in order: a thread takes 8 columns of a
// row of a tile (forward of gate and of up), four parts in flight.
template <class T, FfnKind KIND>
__global__ __launch_bounds__(256) void ffn_join_kernel(FfnArgs a, int tiles_m, int tiles_n, int whole)
{
    using S = Shape<T, KIND>;
    constexpr int kVecs = S::kCols / 8;
    const int tile = blockIdx.y, vector = blockIdx.x * 256 + threadIdx.x;
    const TilePlace place = tile_place(whole + tile, tiles_m, tiles_n);
    const int which = KIND == kFfnWeight && a.outputs == 2 && place.m >= tiles_m / 2 ? 1 : 0;
    const int row = vector / kVecs, col = vector % kVecs * 8;
    const int64_t m = static_cast<int64_t>(place.m - which * (tiles_m / 2)) * T::BM + row, n = static_cast<int64_t>(place.n) * S::kCols + col;
    if (m >= S::m(a)) return;  // whole rows
    const float* p = a.part + static_cast<int64_t>(tile) * a.split * (T::BM * T::BN) + row * T::BN + col;
    f32x4 s[4] = {};
    for (int k = 0; k < a.split; k += 4) {
        f32x4 t[4][4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (k + x >= a.split) break;
            const float* q = p + static_cast<int64_t>(k + x) * (T::BM * T::BN);
            t[x][0] = *(const ZERO_G f32x4*)q;
            t[x][1] = *(const ZERO_G f32x4*)(q + 4);
            if constexpr (KIND == kFfnForward) {
                t[x][2] = *(const ZERO_G f32x4*)(q + T::BN / 2);
                t[x][3] = *(const ZERO_G f32x4*)(q + T::BN / 2 + 4);
            }
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (k + x >= a.split) break;
#pragma unroll
            for (int y = 0; y < (KIND == kFfnForward ? 4 : 2); ++y) s[y] += t[x][y];
        }
    }
    float f[8], u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        f[i] = s[i / 4][i % 4];
        u[i] = s[2 + i / 4][i % 4];
    }
    finish<KIND>(a, which, m, n, static_cast<int>(min(S::n(a) - n, int64_t{8})), f, u);
}

// Big, for whole rounds of the chip. Forward eight waves of 64 x 128 sums, so
// that a wave's columns of gate, and as many of up, are 64, a line of each, in a
// ring of three: 1261 us for 8192 x 4096 x 11008, 1292 in a ring of four (one
// workgroup a unit either way), 1314 with four waves of 128 x 128. Backward four
// waves of 128 x 128 sums, which read the fewest pieces: dh 1100 us, the weight
// gradients 1190; 1212 and 1235 with eight waves. The smaller ones where there
// are fewer sums than that: two, three or four workgroups a unit hide each
// other's latency and a split leaves less to join (see the plan's times).
template <FfnKind KIND>
using Big = Tile<256, 256, KIND == kFfnForward ? 4 : 2, 2, KIND == kFfnForward ? 3 : 4, 1>;
using Mid = Tile<128, 128, 2, 2, 4, 2>;
using Small = Tile<64, 128, 2, 2, 4, 3>;
using Flat = Tile<32, 128, 1, 2, 4, 4>;
using Slow = Tile<128, 128, 2, 2, 2, 2>;  // through registers: a step takes 0.95 us with the chip full, Mid's 0.52

// Whether 32-bit offsets reach over the 256 rows of a tile.
bool in_reach(int64_t ld) { return ld <= (int64_t{1} << 22); }

// Whether they do for all operands, the same ones in both segments, and what
// runs across the summed index has a whole unit.
template <FfnKind KIND>
bool plain(const FfnArgs& a)
{
    const bool h = in_reach(a.ld_h), w = in_reach(a.ld_w[0]) && in_reach(a.ld_w[1]);
    const bool d = in_reach(a.ld_d[0]) && ((KIND == kFfnWeight && a.outputs == 1) || in_reach(a.ld_d[1]));
    if (KIND == kFfnForward) return h && w;
    if (KIND == kFfnInput) return d && w && a.ld_d[0] == a.ld_d[1] && a.ld_w[0] == a.ld_w[1] && a.cols >= 8;
    return d && h && a.hidden >= 8 && a.cols >= 8;
}

// Every row of an operand starts on 16 bytes.
bool on_16(const uint16_t* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) | static_cast<uint64_t>(ld) * 2) % 16 == 0; }

// Whether every 16-byte unit that a product reads also lies on 16 bytes and inside its row.
template <FfnKind KIND>
bool fast(const FfnArgs& a)
{
    const bool h = on_16(a.h, a.ld_h), d = on_16(a.d[0], a.ld_d[0]) && ((KIND == kFfnWeight && a.outputs == 1) || on_16(a.d[1], a.ld_d[1]));
    const bool w = on_16(a.w[0], a.ld_w[0]) && on_16(a.w[1], a.ld_w[1]);
    if (!plain<KIND>(a) || a.cols % 8 != 0) return false;
    if (KIND == kFfnForward) return h && w;
    return a.hidden % 8 == 0 && d && (KIND == kFfnInput ? w : h);
}

// Tiles of the output, the first `whole` of them summed by one workgroup each,
// the others over `split` ranges of steps, whose sums go to the workspace (a
// tile's ranges next to each other), and a second launch adds them in order.
struct FfnPlan {
    int tile;
    int64_t whole;
    int split;
    int64_t chunk;  // steps of a range (the last may have fewer)
    size_t bytes;   // workspace
};

template <class T, FfnKind KIND, bool FAST>
hipError_t launch_tile(const FfnArgs& a, const FfnPlan& plan, hipStream_t s)
{
    using S = Shape<T, KIND>;
    const int m = static_cast<int>((S::m(a) + T::BM - 1) / T::BM) * a.outputs;
    const int n = static_cast<int>((S::n(a) + S::kCols - 1) / S::kCols);
    const int whole = static_cast<int>(plan.whole), rest = m * n - whole;
    const unsigned grid = static_cast<unsigned>((whole + 7) / 8 * 8 + (static_cast<int64_t>(rest) * plan.split + 7) / 8 * 8);
    ffn_kernel<T, KIND, FAST><<<grid, T::NT, 0, s>>>(a, m, n, whole);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || rest == 0) return e;
    ffn_join_kernel<T, KIND><<<dim3((T::BM * S::kCols / 8 + 255) / 256, static_cast<unsigned>(rest)), 256, 0, s>>>(a, m, n, whole);
    return hipGetLastError();
}

// A tile shape; the time of a step of one of its workgroups alone on its
// compute unit, of a step of as many as the chip holds at once, and of a round's
// start and results, us.
struct Candidate {
    int tile, bm, bn, slots;
    double alone, full, start;
};
template <class T>
constexpr Candidate candidate(int tile, double alone, double full, double start)
{
    return Candidate{tile, T::BM, T::BN, T::SLOTS, alone, full, start};
}
enum TileId { kBig, kMid, kSmall, kFlat, kSlow };

// f(plan, the time that it is expected to take) for every plan of a product.
template <class F>
void each_plan(FfnKind kind, bool aligned, int outputs, int64_t rows, int64_t cols, int64_t hidden, F&& f)
{
    static const Candidate kTiles[] = {candidate<Flat>(kFlat, 0.18, 0.52, 3.0), candidate<Small>(kSmall, 0.17, 0.60, 3.0),
                                       candidate<Mid>(kMid, 0.25, 0.52, 4.0), candidate<Big<kFfnForward>>(kBig, 0.60, 0.76, 9.0)};
    static const Candidate kSlowTile = candidate<Slow>(kSlow, 0.70, 0.95, 5.0);
    constexpr double kJoin = 4.0, kParts = 6e6, kMemory = 5.5e6;  // us a join; bytes a us of parts written and read, and of factors
    constexpr double kCaches = 64e6;                              // bytes of factors: twice the L2s
    constexpr int64_t kMostParts = int64_t{1} << 16;              // tiles of one join (its grid's second size)
    const int64_t m = kind == kFfnWeight ? hidden : rows, n = kind == kFfnForward ? 2 * hidden : cols;
    const int64_t k = kind == kFfnForward ? cols : kind == kFfnInput ? hidden : rows;
    const int64_t all_steps = (k + BK - 1) / BK * (kind == kFfnInput ? 2 : 1);
    // A workgroup alone waits longer for a step that comes from memory than for one that the L2s hold: with one
    // time for both, dh of 128 rows x 4096 x 11008 from memory took 84 us and now 63, or that of 4096 rows x 768 x
    // 2048 41 instead of 33.
    const double far = 2.0 * static_cast<double>(m + n) * static_cast<double>(k) * (kind == kFfnInput ? 2 : 1) > kCaches ? 1.5 : 1.0;
    const auto consider = [&](const Candidate& c) {
        const double alone = c.alone * far < c.full ? c.alone * far : c.alone < c.full ? c.full : c.alone;
        const int64_t tiles_m = (m + c.bm - 1) / c.bm * outputs, tiles_n = (n + c.bn - 1) / c.bn;
        const int64_t tiles = tiles_m * tiles_n, slots = static_cast<int64_t>(c.slots) * kComputeUnits;
        // What one workgroup's step brings from memory: of what it shares with each of its neighbours a third is there.
        const auto shared = [](int64_t tiles, int64_t most) { return 1.0 + 0.3 * static_cast<double>((tiles < most ? tiles : most) - 1); };
        const double bytes = 2.0 * BK * (c.bn / shared(tiles_m, 8) + c.bm / shared(tiles_n, 4));
        // the four waves of the largest backward tile take longer over their results
        const double start = c.tile == kBig && kind != kFfnForward ? 14.0 : c.start;
        const auto round = [&](int64_t groups, int64_t steps) {
            const double g = static_cast<double>(groups), full = g / static_cast<double>(slots) * c.full, memory = g * bytes / kMemory;
            const double step = full > memory ? full : memory;
            return start + static_cast<double>(steps) * (step > alone ? step : alone);
        };
        const auto rounds = [&](int64_t groups, int64_t steps) {
            return static_cast<double>(groups / slots) * round(slots, steps) + (groups % slots > 0 ? round(groups % slots, steps) : 0.0);
        };
        f(FfnPlan{c.tile, tiles, 1, all_steps, 0}, rounds(tiles, all_steps));
        const int64_t full_rounds = tiles / slots * slots;
        for (const int64_t whole : {int64_t{0}, full_rounds}) {
            const int64_t rest = tiles - whole;
            if (rest == 0 || rest >= kMostParts || (whole == 0 && rest > 2 * slots)) continue;
            for (const int want : {2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64}) {
                if (all_steps < 4 * want) break;
                const int64_t steps = (all_steps + want - 1) / want;
                const int64_t split = (all_steps + steps - 1) / steps;
                const double room = 4.0 * static_cast<double>(rest * split) * c.bm * c.bn;
                const double used = room * static_cast<double>(m < c.bm ? m : c.bm) / c.bm;  // rows beyond the last are not written
                f(FfnPlan{c.tile, whole, static_cast<int>(split), steps, static_cast<size_t>(room)},
                  (whole > 0 ? rounds(whole, all_steps) : 0.0) + rounds(rest * split, steps) + kJoin + used / kParts);
            }
            if (full_rounds == 0) break;
        }
    };
    if (!aligned) consider(kSlowTile);
    else
        for (const Candidate& c : kTiles)
            if (kind != kFfnWeight || c.bm >= 128) consider(c);
}

// The plan that is expected to take the least time: rounds of workgroups
// through the chip, each a start and its steps, and for split tiles their parts
// written, read and joined by a second launch. Either no tile is whole, or as
// many as fill whole rounds, or all. The model knows little of what the caches
// hold; it only has to order the plans.
struct TimedPlan {
    FfnPlan plan;
    double us;
};
TimedPlan plan_for(FfnKind kind, bool aligned, int outputs, int64_t rows, int64_t cols, int64_t hidden)
{
    FfnPlan best{};
    double least = -1.0;
    each_plan(kind, aligned, outputs, rows, cols, hidden, [&](const FfnPlan& p, double us) {
        if (least < 0.0 || us < least) {
            least = us;
            best = p;
        }
    });
    return TimedPlan{best, least};
}

// A factor of a product: rows and columns of an operand.
struct Operand {
    const uint16_t* p;
    int64_t ld, rows, cols;
};

// f(operand) for each of a product's factors.
template <class F>
void each_operand(FfnKind kind, FfnArgs& a, int outputs, F&& f)
{
    if (kind != kFfnForward) {
        f(a.d[0], a.ld_d[0], a.rows, a.hidden);
        if (kind == kFfnInput || outputs == 2) f(a.d[1], a.ld_d[1], a.rows, a.hidden);
    }
    if (kind != kFfnInput) f(a.h, a.ld_h, a.rows, a.cols);
    if (kind != kFfnWeight) {
        f(a.w[0], a.ld_w[0], a.hidden, a.cols);
        f(a.w[1], a.ld_w[1], a.hidden, a.cols);
    }
}

// Whether a product whose operands' rows do not all hold whole units of 16
// bytes, because there are not a multiple of 8 columns, copies them to the
// workspace first, zeros up to whole units, and then takes the tiles that go
// straight to LDS. Loads at odd addresses take more than twice as long as
// aligned ones, for every tile that they are part of; a copy reads each
// operand once. 2011 rows x 1003 x 2731: forward 72 -> 51 us, dh 61 -> 57, both
// weight gradients 64 -> 46; 4096 x 4091 x 4093: 462 -> 260, 408 -> 251 and 420 ->
// 225. A few rows do not repay their weights' copy: forward 16 x 1003 x 2731
// takes 14 us as they are and 18 from copies, 64 x 4091 x 11003 62 and 124. (Operands of a multiple of 8
// columns that lie at odd addresses or strides are read where they are: a
// caller can place them better, and the workspace of those who did is smaller.)
struct CopyPlan {
    TimedPlan timed;
    size_t bytes;  // of the copies; 0: none are made
};
CopyPlan plan_unaligned(FfnKind kind, int outputs, int64_t rows, int64_t cols, int64_t hidden)
{
    const CopyPlan here{plan_for(kind, false, outputs, rows, cols, hidden), 0};
    if ((cols % 8 == 0 && (kind == kFfnForward || hidden % 8 == 0)) || rows == 0 || cols < 8 || hidden < 8) return here;
    constexpr double kCopy = 3.0, kCopied = 6e6;  // us a launch; bytes read and written a us
    size_t bytes = 0;
    bool fits = true;
    FfnArgs none{};
    none.rows = rows;
    none.cols = cols;
    none.hidden = hidden;
    each_operand(kind, none, outputs, [&](const uint16_t*, int64_t, int64_t r, int64_t c) {
        const int64_t units = (c + 7) / 8;
        if (!in_reach(8 * units) || r > (int64_t{1} << 30) / units) fits = false;  // the latter: units in 32 bits
        else bytes += (static_cast<size_t>(r * units) * 16 + 255) / 256 * 256;
    });
    if (!fits) return here;
    TimedPlan copied = plan_for(kind, true, outputs, rows, cols, hidden);
    copied.us += kCopy + 2.0 * static_cast<double>(bytes) / kCopied;
    return copied.us < here.timed.us ? CopyPlan{copied, bytes} : here;
}

// Operands, and where their copies lie.
struct CopyArgs {
    Operand from[4];
    uint16_t* to[4];
    FastDiv units[4];  // of a row
};

// A thread copies a unit, 8 columns: a stream.
__global__ __launch_bounds__(256) void ffn_copy_kernel(CopyArgs c)
{
    const Operand& o = c.from[blockIdx.y];
    const uint32_t units = static_cast<uint32_t>((o.cols + 7) / 8), at = blockIdx.x * 256u + threadIdx.x;
    const uint32_t row = div_by(at, c.units[blockIdx.y]), unit = at - row * units;
    if (row >= o.rows) return;
    *(ZERO_G u32x4*)(c.to[blockIdx.y] + static_cast<int64_t>(at) * 8) = load_unit(o.p + row * o.ld, int64_t{unit} * 8, o.cols);
}

// The operands whose rows do not lie on 16 bytes, end inside a unit or lie too
// far apart, copied to the workspace, where they do not; the parts of split
// tiles come behind them. The two sums of dh are read at the same offsets: of its
// two gradients, and of its two weights, both stay where they are, at one stride,
// or both are copied.
hipError_t copy_operands(FfnKind kind, FfnArgs& a, size_t bytes, hipStream_t s)
{
    bool stays[4];
    int64_t strides[4];
    int count = 0;
    each_operand(kind, a, a.outputs, [&](const uint16_t*& p, int64_t& ld, int64_t, int64_t cols) {
        strides[count] = ld;
        stays[count++] = cols % 8 == 0 && on_16(p, ld) && in_reach(ld);
    });
    for (int i = 0; kind == kFfnInput && i < count; i += 2) stays[i] = stays[i + 1] = stays[i] && stays[i + 1] && strides[i] == strides[i + 1];
    CopyArgs c{};
    int n = 0, at = 0;
    int64_t most = 0;
    char* to = reinterpret_cast<char*>(a.part);
    a.part = reinterpret_cast<float*>(to + bytes);
    each_operand(kind, a, a.outputs, [&](const uint16_t*& p, int64_t& ld, int64_t rows, int64_t cols) {
        if (stays[at++]) return;
        const int64_t units = (cols + 7) / 8;
        c.from[n] = Operand{p, ld, rows, cols};
        c.to[n] = reinterpret_cast<uint16_t*>(to);
        c.units[n] = fast_div(static_cast<uint32_t>(units));
        ++n;
        p = reinterpret_cast<const uint16_t*>(to);
        ld = units * 8;
        to += (rows * units * 16 + 255) / 256 * 256;
        if (rows * units > most) most = rows * units;
    });
    ffn_copy_kernel<<<dim3(static_cast<unsigned>((most + 255) / 256), static_cast<unsigned>(n)), 256, 0, s>>>(c);
    return hipGetLastError();
}

template <FfnKind KIND>
hipError_t launch_kind(FfnArgs a, hipStream_t s)
{
    a.outputs = KIND == kFfnWeight && a.out[1].p != nullptr ? 2 : 1;
    a.plain = plain<KIND>(a);
    FfnPlan plan;
    if (fast<KIND>(a)) {
        plan = plan_for(KIND, true, a.outputs, a.rows, a.cols, a.hidden).plan;
    } else {
        const CopyPlan odd = plan_unaligned(KIND, a.outputs, a.rows, a.cols, a.hidden);
        plan = odd.timed.plan;
        if (odd.bytes > 0) {
            const hipError_t e = copy_operands(KIND, a, odd.bytes, s);
            if (e != hipSuccess) return e;
            if (!plain<KIND>(a)) return hipErrorInvalidValue;  // the tiles that are launched below go by it
        }
    }
    a.chunk = plan.chunk;
    a.split = plan.split;
    switch (plan.tile) {
    case kBig: return launch_tile<Big<KIND>, KIND, true>(a, plan, s);
    case kMid: return launch_tile<Mid, KIND, true>(a, plan, s);
    case kSlow: return launch_tile<Slow, KIND, false>(a, plan, s);
    default: break;
    }
    if constexpr (KIND != kFfnWeight) {  // its columns' tiles are 128 or more: their units are permuted by pairs of eight
        if (plan.tile == kSmall) return launch_tile<Small, KIND, true>(a, plan, s);
        return launch_tile<Flat, KIND, true>(a, plan, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace

size_t ffn_workspace_bytes(FfnKind kind, int64_t rows, int64_t cols, int64_t hidden)
{
    size_t most = 0;
    for (int outputs = 1; outputs <= (kind == kFfnWeight ? 2 : 1); ++outputs) {
        const CopyPlan odd = plan_unaligned(kind, outputs, rows, cols, hidden);
        for (const size_t bytes : {plan_for(kind, true, outputs, rows, cols, hidden).plan.bytes, odd.bytes + odd.timed.plan.bytes})
            if (bytes > most) most = bytes;
    }
    return most;
}

hipError_t launch_ffn(FfnKind kind, const FfnArgs& a, hipStream_t s)
{
    return kind == kFfnForward ? launch_kind<kFfnForward>(a, s) : kind == kFfnInput ? launch_kind<kFfnInput>(a, s) : launch_kind<kFfnWeight>(a, s);
}

}  // namespace zero
