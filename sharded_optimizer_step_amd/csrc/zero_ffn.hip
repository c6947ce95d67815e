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
#include "zero_act8_device.h"

namespace zero {
namespace {

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
#define ZERO_L __attribute__((address_space(3)))

constexpr int BK = 64;  // summed elements of a step

// ------------------------------------------------------------------ activations

// 1 / (1 + exp(-x)), within 3 units of its last place and |x| 2^-24 of itself
// (what is made of it is rounded to bf16 or 8 bits). For large |x| the
// exponential is infinite or 0, and the result the limit.
__device__ __forceinline__ float logistic(float x)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.44269504f));
}

__device__ __forceinline__ float activation(int act, float g)
{
    if (act == ZERO_FFN_SILU) return g * logistic(g);
    if (act == ZERO_FFN_GELU) return 0.5f * g * (1.0f + erff(g * 0.70710678f));
    return g * logistic(1.59576912f * fmaf(0.044715f * g * g, g, g));  // (1 + tanh(z)) / 2 is the logistic function of 2 z
}

// ------------------------------------------------------------------ tiles in LDS

// BM x BN tile of the output, WM x WN waves, SLOTS workgroups a compute unit.
template <int BM_, int BN_, int WM_, int WN_, int SLOTS_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, SLOTS = SLOTS_;
    static constexpr int NT = 64 * WM * WN;
    static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;  // 16 x 16 pieces of a wave
};

// A tile of SIZE rows or columns of a factor and BK elements of the summed
// index. ALONG: the summed index runs along its rows, of 128 bytes; otherwise
// across them, of 2 SIZE bytes.
//
// Tiles go from memory to LDS without passing through registers, a wave's 64
// units of 16 bytes one after the other, so they cannot be padded. The units
// are permuted within their rows instead. ALONG: 16 lanes read the same unit of
// 16 rows, and two rows are one span of the 64 banks, so unit u of row r lies
// at u ^ (r / 2 % 8). Across: 32 lanes of a transposing read take 32 bytes, two
// units, of rows 0 .. 3 and 8 .. 11 of 16 (or the others), whose pairs of units
// are permuted by eight different numbers.
template <bool ALONG, int SIZE, int NT>
struct Factor {
    static constexpr int kRowBytes = ALONG ? BK * 2 : SIZE * 2;
    static constexpr int kUnits = kRowBytes / 16;             // of a row
    static constexpr int kVecs = SIZE * BK * 2 / 16 / NT;     // units a thread loads
    static constexpr int kStep = NT / kUnits;                 // rows from one of them to the next
    static_assert(NT % kUnits == 0 && kStep % 16 == 0, "a thread's units lie at one place of their rows");
    static_assert(ALONG || SIZE >= 128, "eight pairs of units");

    static __device__ __forceinline__ int place(int row, int unit)
    {
        return ALONG ? unit ^ (row >> 1 & 7) : unit ^ ((row & 3) << 1 | (row >> 3 & 1) << 3);
    }
};

// Elements col .. col + 7 of a row of `limit` elements, zeros beyond it.
__device__ __forceinline__ u32x4 load_unit(const uint16_t* row, int64_t col, int64_t limit)
{
    const int64_t left = limit - col;
    if (left >= 8) return ld16_a2(row + col);
    if (left <= 0) return u32x4{};
    if (limit >= 8) {  // the last 8 of the row, moved into place
        const u32x4 v = ld16_a2(row + limit - 8);
        const int shift = static_cast<int>(8 - left);
        uint64_t lo = v.x | static_cast<uint64_t>(v.y) << 32, hi = v.z | static_cast<uint64_t>(v.w) << 32;
        if (shift >= 4) {
            lo = hi >> (16 * (shift - 4));
            hi = 0;
        } else {
            lo = lo >> (16 * shift) | hi << (64 - 16 * shift);
            hi >>= 16 * shift;
        }
        return u32x4{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi), static_cast<uint32_t>(hi >> 32)};
    }
    u32x4 v{};
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < left) v[i / 2] |= static_cast<uint32_t>(((const ZERO_G uint16_t*)row)[col + i]) << (16 * (i % 2));
    return v;
}

// A raw buffer of 2 GiB from p on; loads from offsets beyond it give zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const uint16_t* p)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p), 0, 0x80000000u, 0x00020000);
}
constexpr uint32_t kBeyond = 0xFFFFFF00u;

// 8 summed elements for this lane's row or column of a piece of 16, from a tile
// in LDS; `at` is the lane's own place in it, see lane_place.
template <bool ALONG, int ROW_BYTES>
__device__ __forceinline__ bf16x8 read_piece(const char* at)
{
    if constexpr (ALONG) {
        return *reinterpret_cast<const bf16x8*>(at);
    } else {
        const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZERO_L i16x4*)at);
        const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ZERO_L i16x4*)(at + 4 * ROW_BYTES));
        return __builtin_bit_cast(bf16x8, (i16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
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
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = activation(a.act, f[i]) * u[i];
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
__global__ __launch_bounds__(T::NT, T::NT / 256 * T::SLOTS) void ffn_kernel(FfnArgs a, int tiles_m, int tiles_n, int whole)
{
    using S = Shape<T, KIND>;
    constexpr bool kAlongA = KIND != kFfnWeight, kAlongB = KIND == kFfnForward;
    using A = Factor<kAlongA, T::BM, T::NT>;
    using B = Factor<kAlongB, T::BN, T::NT>;
    // arrays of their own, so that the compiler sees that a step's reads are not what the next one's loads write
    __shared__ __align__(16) char sa0[T::BM * BK * 2], sa1[T::BM * BK * 2], sb0[T::BN * BK * 2], sb1[T::BN * BK * 2];

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
    const int which = KIND == kFfnWeight && place.m >= tiles_m / 2 ? 1 : 0;
    if (KIND == kFfnWeight && a.out[which].p == nullptr) return;
    const int64_t m0 = static_cast<int64_t>(place.m - which * (tiles_m / 2)) * T::BM, n0 = static_cast<int64_t>(place.n) * S::kCols;
    const int64_t m_end = S::m(a), n_end = S::n(a), k_end = S::k(a);
    const int64_t seg_steps = (k_end + BK - 1) / BK;
    const int64_t all_steps = KIND == kFfnInput ? 2 * seg_steps : seg_steps;
    const int64_t begin = parted ? part * a.chunk : 0, end = parted ? min(all_steps, begin + a.chunk) : all_steps;

    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / 64), lane = tid % 64;

    // The units that this thread loads: one place of a row, every kStep-th row.
    const int row_a = tid / A::kUnits, unit_a = A::place(row_a, tid % A::kUnits);
    const int row_b = tid / B::kUnits, unit_b = B::place(row_b, tid % B::kUnits);
    // forward the second half of B's rows are those of up
    constexpr int kHalfB = KIND == kFfnForward ? B::kVecs / 2 : B::kVecs;
    uint32_t off_a[A::kVecs], off_b[B::kVecs];
    if constexpr (FAST) {
        // Rows and columns beyond the last one are read as the last one: their products are not stored.
#pragma unroll
        for (int i = 0; i < A::kVecs; ++i) {
            const int64_t ld = KIND == kFfnForward ? a.ld_h : a.ld_d[0];
            const int64_t row = kAlongA ? min(static_cast<int64_t>(row_a + i * A::kStep), m_end - 1 - m0) : row_a + i * A::kStep;
            const int64_t col = kAlongA ? unit_a * 8 : min(static_cast<int64_t>(unit_a * 8), m_end - 8 - m0);
            off_a[i] = static_cast<uint32_t>((row * ld + col) * 2);
        }
#pragma unroll
        for (int i = 0; i < B::kVecs; ++i) {
            const int64_t ld = KIND == kFfnWeight ? a.ld_h : a.ld_w[0];
            const int r = row_b + i % kHalfB * B::kStep;
            const int64_t row = kAlongB ? min(static_cast<int64_t>(r), n_end - 1 - n0) : r;
            const int64_t col = kAlongB ? unit_b * 8 : min(static_cast<int64_t>(unit_b * 8), n_end - 8 - n0);
            off_b[i] = static_cast<uint32_t>((row * ld + col) * 2);
        }
    }
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
            t.a = a.d[which] + k0 * a.ld_d[which] + m0;
            t.b0 = t.b1 = a.h + k0 * a.ld_h + n0;
        }
        return t;
    };
    // A step's tiles straight to LDS. (In the last one, elements beyond the sum are read from beyond the buffer: zeros.)
    const auto send = [&](int64_t s, char* sa, char* sb) {
        const Step t = step_at(s);
        const __amdgpu_buffer_rsrc_t ra = buffer_at(t.a), rb0 = buffer_at(t.b0), rb1 = buffer_at(t.b1);
        const bool full = t.left >= BK;
#pragma unroll
        for (int i = 0; i < A::kVecs; ++i) {
            uint32_t off = off_a[i];
            if (!full && (kAlongA ? unit_a * 8 : row_a + i * A::kStep) >= t.left) off = kBeyond;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (ZERO_L void*)(sa + (i * T::NT + wave * 64) * 16), 16, off, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < B::kVecs; ++i) {
            uint32_t off = off_b[i];
            if (!full && (kAlongB ? unit_b * 8 : row_b + i * B::kStep) >= t.left) off = kBeyond;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(i < kHalfB ? rb0 : rb1, (ZERO_L void*)(sb + (i * T::NT + wave * 64) * 16), 16, off, 0, 0, 0);
        }
    };
    // Or through registers, for operands whose rows do not all lie on 16 bytes.
    u32x4 va[A::kVecs], vb[B::kVecs];
    const auto fetch = [&](int64_t s) {
        const Step t = step_at(s);
        const int seg = KIND == kFfnInput && s >= seg_steps ? 1 : 0;
#pragma unroll
        for (int i = 0; i < A::kVecs; ++i) {
            const int row = row_a + i * A::kStep;
            const int64_t ld = KIND == kFfnForward ? a.ld_h : a.ld_d[KIND == kFfnInput ? seg : which];
            va[i] = u32x4{};
            if (row < (kAlongA ? m_end - m0 : t.left)) va[i] = load_unit(t.a + row * ld, unit_a * 8, kAlongA ? t.left : m_end - m0);
        }
#pragma unroll
        for (int i = 0; i < B::kVecs; ++i) {
            const int row = row_b + i % kHalfB * B::kStep;
            const int64_t ld = KIND == kFfnWeight ? a.ld_h : a.ld_w[KIND == kFfnInput ? seg : i < kHalfB ? 0 : 1];
            vb[i] = u32x4{};
            if (row < (kAlongB ? n_end - n0 : t.left))
                vb[i] = load_unit((i < kHalfB ? t.b0 : t.b1) + row * ld, unit_b * 8, kAlongB ? t.left : n_end - n0);
        }
    };
    const auto stage = [&](char* sa, char* sb) {
#pragma unroll
        for (int i = 0; i < A::kVecs; ++i) *reinterpret_cast<u32x4*>(sa + (i * T::NT + tid) * 16) = va[i];
#pragma unroll
        for (int i = 0; i < B::kVecs; ++i) *reinterpret_cast<u32x4*>(sb + (i * T::NT + tid) * 16) = vb[i];
    };

    // Where this lane reads. The four groups of 16 lanes take summed elements 8 g
    // .. 8 g + 7 of 32. ALONG, a lane reads them of row lane % 16 of a piece;
    // across, the 16 lanes of a group read 4 elements' rows, 4 columns a lane, and
    // get a column of all 4 each.
    const int wm = wave / T::WN, wn = wave % T::WN, group = lane / 16, in_group = lane % 16;
    const auto piece_a = [&](const char* sa, int i, int k) {
        if constexpr (kAlongA) return sa + (wm * (T::BM / T::WM) + 16 * i + in_group) * A::kRowBytes + A::place(in_group, k / 8 + group) * 16;
        else {
            const int row = 8 * group + in_group / 4, col = wm * (T::BM / T::WM) + 16 * i;
            return sa + (k + row) * A::kRowBytes + A::place(row, col / 8) * 16 + in_group % 4 * 8;
        }
    };
    // Forward a wave's first pieces are of gate, the others of up.
    const auto piece_b = [&](const char* sb, int j, int k) {
        const int col = KIND == kFfnForward ? (j < T::TN / 2 ? 0 : T::BN / 2 - T::TN * 8) + wn * (T::TN * 8) + 16 * j : wn * (T::BN / T::WN) + 16 * j;
        if constexpr (kAlongB) return sb + (col + in_group) * B::kRowBytes + B::place(in_group, k / 8 + group) * 16;
        else {
            const int row = 8 * group + in_group / 4;
            return sb + (k + row) * B::kRowBytes + B::place(row, col / 8) * 16 + in_group % 4 * 8;
        }
    };
    f32x4 acc[T::TN][T::TM];
#pragma unroll
    for (int j = 0; j < T::TN; ++j)
#pragma unroll
        for (int i = 0; i < T::TM; ++i) acc[j][i] = f32x4{};
    const auto multiply = [&](const char* sa, const char* sb) {
#pragma unroll
        for (int k = 0; k < BK; k += 32) {
            bf16x8 fa[T::TM], fb[T::TN];
#pragma unroll
            for (int j = 0; j < T::TN; ++j) fb[j] = read_piece<kAlongB, B::kRowBytes>(piece_b(sb, j, k));
#pragma unroll
            for (int i = 0; i < T::TM; ++i) fa[i] = read_piece<kAlongA, A::kRowBytes>(piece_a(sa, i, k));
#pragma unroll
            for (int i = 0; i < T::TM; ++i)
#pragma unroll
                for (int j = 0; j < T::TN; ++j)
                    acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], acc[j][i], 0, 0, 0);
        }
    };
    // All of this step's loads to LDS have arrived and all of its reads from it
    // are done, in every wave.
    const auto meet = [&] {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    // One step from its tiles while the next one's go to the other two, whose
    // last reads were before the last barrier.
    const auto step = [&](int64_t s, char* sa, char* sb, char* next_a, char* next_b) {
        if constexpr (FAST) {
            if (s + 1 < end) send(s + 1, next_a, next_b);
            multiply(sa, sb);
        } else {
            if (s + 1 < end) fetch(s + 1);
            multiply(sa, sb);
            if (s + 1 < end) stage(next_a, next_b);
        }
        meet();
    };
    if (begin < end) {
        if constexpr (FAST) send(begin, sa0, sb0);
        else {
            fetch(begin);
            stage(sa0, sb0);
        }
        meet();
    }
    for (int64_t s = begin; s < end; s += 2) {
        step(s, sa0, sb0, sa1, sb1);
        if (s + 1 < end) step(s + 1, sa1, sb1, sa0, sb0);
    }

    // B is the first operand, so a lane holds four neighbouring columns of one
    // row of the output. Sixteen rows at a time go through LDS (each wave its own
    // part of what the tiles lay in; the last barrier is behind every read of
    // them), after which a lane has eight neighbouring columns, forward of gate
    // and of up, and eight lanes whole lines. The fences keep the compiler from
    // moving a lane's reads over its writes, which other lanes read; a wave's LDS
    // accesses are in order.
    constexpr int kWide = T::TN * 16, kOut = KIND == kFfnForward ? kWide / 2 : kWide, kLanes = kOut / 8, kPad = kWide + 4;
    static_assert(T::NT / 256 * 16 * kPad * sizeof(float) <= sizeof(sa0) && T::BN >= T::BM, "each array holds 16 rows of a fourth of the waves");
    const int quarter = wave % 4;
    float* out = reinterpret_cast<float*>(quarter == 0 ? sa0 : quarter == 1 ? sa1 : quarter == 2 ? sb0 : sb1) + wave / 4 * 16 * kPad;
    const int64_t n = n0 + wn * kOut + lane % kLanes * 8;
    const int left = static_cast<int>(min(n_end - n, int64_t{8}));
#pragma unroll
    for (int i = 0; i < T::TM; ++i) {
#pragma unroll
        for (int j = 0; j < T::TN; ++j) *reinterpret_cast<f32x4*>(out + in_group * kPad + 16 * j + group * 4) = acc[j][i];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int r = 0; r < 16; r += 64 / kLanes) {
            const int row = r + lane / kLanes, tile_row = wm * (T::BM / T::WM) + 16 * i + row;
            const int64_t m = m0 + tile_row;
            float f[8], u[8] = {};
            const float* from = out + row * kPad + lane % kLanes * 8;
#pragma unroll
            for (int c = 0; c < 8; c += 4) {
                *reinterpret_cast<f32x4*>(f + c) = *reinterpret_cast<const f32x4*>(from + c);
                if constexpr (KIND == kFfnForward) *reinterpret_cast<f32x4*>(u + c) = *reinterpret_cast<const f32x4*>(from + kOut + c);
            }
            if (parted) {
                float* to = a.part + (static_cast<int64_t>(split_tile) * a.split + part) * (T::BM * T::BN) + tile_row * T::BN + wn * kOut + lane % kLanes * 8;
#pragma unroll
                for (int c = 0; c < 8; c += 4) {
                    *(ZERO_G f32x4*)(to + c) = *reinterpret_cast<f32x4*>(f + c);
                    if constexpr (KIND == kFfnForward) *(ZERO_G f32x4*)(to + T::BN / 2 + c) = *reinterpret_cast<f32x4*>(u + c);
                }
            } else if (m < m_end) {
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
    const int which = KIND == kFfnWeight && place.m >= tiles_m / 2 ? 1 : 0;
    const int row = vector / kVecs, col = vector % kVecs * 8;
    const int64_t m = static_cast<int64_t>(place.m - which * (tiles_m / 2)) * T::BM + row, n = static_cast<int64_t>(place.n) * S::kCols + col;
    if (m >= S::m(a)) return;  // whole rows
    if (KIND == kFfnWeight && a.out[which].p == nullptr) return;
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

using TileBigF = Tile<256, 256, 4, 2, 1>;  // forward: a wave's columns of gate and of up fill a line each
using TileBig = Tile<256, 256, 2, 4, 1>;
using TileMid = Tile<128, 128, 2, 2, 2>;

bool on_16(const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) | static_cast<uint64_t>(ld) * 2) % 16 == 0 && ld <= (int64_t{1} << 22); }

// Whether every 16-byte unit that a product reads lies on 16 bytes and inside
// its row, and 32-bit offsets reach over a tile.
template <FfnKind KIND>
bool fast(const FfnArgs& a)
{
    const bool h = on_16(a.h, a.ld_h), d = on_16(a.d[0], a.ld_d[0]) && on_16(a.d[1], a.ld_d[1]) && a.ld_d[0] == a.ld_d[1];
    const bool w = on_16(a.w[0], a.ld_w[0]) && on_16(a.w[1], a.ld_w[1]) && a.ld_w[0] == a.ld_w[1];
    if (KIND == kFfnForward) return h && w && a.cols % 8 == 0;
    if (KIND == kFfnInput) return d && w && a.cols % 8 == 0 && a.hidden % 8 == 0;
    return d && h && a.cols % 8 == 0 && a.hidden % 8 == 0;
}

template <class T, FfnKind KIND>
hipError_t launch_tile(const FfnArgs& a, const FfnPlan& plan, hipStream_t s)
{
    using S = Shape<T, KIND>;
    const int m = static_cast<int>((S::m(a) + T::BM - 1) / T::BM) * (KIND == kFfnWeight ? 2 : 1);
    const int n = static_cast<int>((S::n(a) + S::kCols - 1) / S::kCols);
    const int whole = static_cast<int>(plan.whole), rest = m * n - whole;
    const unsigned grid = static_cast<unsigned>((whole + 7) / 8 * 8 + (static_cast<int64_t>(rest) * plan.split + 7) / 8 * 8);
    if (fast<KIND>(a)) ffn_kernel<T, KIND, true><<<grid, T::NT, 0, s>>>(a, m, n, whole);
    else ffn_kernel<T, KIND, false><<<grid, T::NT, 0, s>>>(a, m, n, whole);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || rest == 0 || plan.split == 1) return e;
    ffn_join_kernel<T, KIND><<<dim3(T::BM * S::kCols / 8 / 256, static_cast<unsigned>(rest)), 256, 0, s>>>(a, m, n, whole);
    return hipGetLastError();
}

}  // namespace

FfnPlan ffn_plan(FfnKind kind, int64_t rows, int64_t cols, int64_t hidden)
{
    const int64_t m = kind == kFfnWeight ? hidden : rows, n = kind == kFfnForward ? 2 * hidden : cols;
    const int64_t k = kind == kFfnForward ? cols : kind == kFfnInput ? hidden : rows;
    const int64_t steps = (k + BK - 1) / BK * (kind == kFfnInput ? 2 : 1);
    const auto tiles = [&](int64_t bm, int64_t bn) { return (m + bm - 1) / bm * ((n + bn - 1) / bn) * (kind == kFfnWeight ? 2 : 1); };
    FfnPlan p{};
    p.tile = tiles(256, 256) >= kComputeUnits ? 0 : 1;
    p.whole = p.tile == 0 ? tiles(256, 256) : tiles(128, 128);
    p.split = 1;
    p.chunk = steps;
    return p;
}

hipError_t launch_ffn(FfnKind kind, const FfnArgs& args, const FfnPlan& plan, hipStream_t s)
{
    FfnArgs a = args;
    a.chunk = plan.chunk;
    a.split = plan.split;
    if (kind == kFfnForward) return plan.tile == 0 ? launch_tile<TileBigF, kFfnForward>(a, plan, s) : launch_tile<TileMid, kFfnForward>(a, plan, s);
    if (kind == kFfnInput) return plan.tile == 0 ? launch_tile<TileBig, kFfnInput>(a, plan, s) : launch_tile<TileMid, kFfnInput>(a, plan, s);
    return plan.tile == 0 ? launch_tile<TileBig, kFfnWeight>(a, plan, s) : launch_tile<TileMid, kFfnWeight>(a, plan, s);
}

}  // namespace zero
