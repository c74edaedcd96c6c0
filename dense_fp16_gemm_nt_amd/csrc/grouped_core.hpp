// Device building blocks of the grouped products (gfx950 / CDNA4 only).
//
// Every operator is a set of output tiles D[i][j] = sum_c X(i, c) Y(j, c), and
// differs in how X and Y lie in memory.  A side is either "by rows", where the
// contraction c is contiguous (rows of A, rows of B in A B^T), or "by columns",
// where i or j is (B in G B, both sides in G^T A).  Tiles go from memory to LDS
// directly, in the layout they have; sides by columns are transposed on the
// way out of LDS (ds_read_b64_tr_b16: 4 values of c for each of 16 columns).
//
// A buffer resource ends with the last row that belongs to a tile, so rows of
// other groups, or behind the last one, arrive as zeros whatever memory holds;
// 16-byte chunks behind a row's end get an offset past every buffer's end.  A
// zero meets a zero there: a value that is not finite never spreads to an
// output that it is not part of.
//
// Sums are held in fp32 by the matrix cores; an output is rounded once.
#pragma once

#include <type_traits>
#include <utility>

#include "attn_core.hpp"
#include "common.hpp"
#include "sched.hpp"

namespace g16 {
namespace grp {

using attn::BF16;
using attn::Div;
using attn::F16;
using attn::s16x4;

// An offset past the end of every buffer: they have less than 2^31 bytes (steps
// of 512 rows by columns up to 2^32: there it names rows of the same matrix, for
// columns that are not stored).
constexpr uint32_t kBeyond = 0x80000000u;

// Tile of BM rows of X by BN rows of Y, BK of the contraction at a time in a
// ring of STAGES; WM x WN waves over the tile, and WK along the contraction,
// whose sums are added at the end.
template <int BM_, int BN_, int BK_, int WM_, int WN_, int WK_, int STAGES_, int PER_CU_>
struct Cfg {
    static constexpr int BM = BM_, BN = BN_, BK = BK_, WM = WM_, WN = WN_, WK = WK_, STAGES = STAGES_, PER_CU = PER_CU_;
    static constexpr int WAVES = WM * WN * WK, THREADS = 64 * WAVES;
    // 32 x 32 blocks of a wave; a side of 16 is half a block, whose other half repeats it and is not stored
    static constexpr int FM = BM == 16 ? 1 : BM / WM / 32, FN = BN == 16 ? 1 : BN / WN / 32;
    static constexpr int KSUB = BK / 16 / WK;                    // products of a block and step
    static constexpr int X_BYTES = BM * BK * 2, Y_BYTES = BN * BK * 2, STAGE = X_BYTES + Y_BYTES;
    static constexpr int LDS = STAGES * STAGE;
    static constexpr int LOADS = STAGE / (THREADS * 16);         // of a wave and step
    static_assert(LDS * PER_CU <= 160 * 1024, "LDS budget");
    static_assert(X_BYTES % (THREADS * 16) == 0 && Y_BYTES % (THREADS * 16) == 0, "every wave loads as much of each side");
    static_assert((STAGES - 1) * LOADS < 64, "vmcnt is 6 bits");
    static_assert(FM >= 1 && FN >= 1 && KSUB >= 1, "a wave has a block and a product");
};

// ------------------------------------------------------------- LDS layouts
// By rows: EXT rows of BK elements; chunk c of row r at c ^ swz: the lanes of a
// fragment read rows at one chunk, and 16 rows in a row cover all 64 banks.
// By columns: BK rows of EXT elements.  A transposing read takes 4 rows of 64
// bytes for 32 lanes; four neighbouring rows are put into the four quarters of
// the 256-byte bank window.
template <bool COLS, int EXT, int BK>
struct Tile {
    static constexpr int CH = (COLS ? EXT : BK) / 8;   // chunks of a row
    static constexpr int PITCH = 16 * CH;
    static __device__ __forceinline__ int swz(int r)
    {
        if (COLS) return CH >= 16 ? (r & 3) << 2 : CH == 8 ? ((r >> 1) & 1) << 2 : 0;
        return CH >= 16 ? (r & 15) : CH == 8 ? ((r >> 1) & 7) : 0;
    }
};

// A side's loads, step by step along the contraction, by all threads.
template <class C, bool COLS, int EXT>
struct Side {
    using L = Tile<COLS, EXT, C::BK>;
    static constexpr int LOADS = EXT * C::BK * 2 / (C::THREADS * 16), ROWS = C::THREADS / L::CH;
    static_assert(C::THREADS % L::CH == 0, "a load of all threads covers whole rows");
    uint32_t off[LOADS];
    uint64_t at;       // the next step
    uint32_t ld;       // bytes from a row to the next
    int ext;           // rows, or columns, that there are

    static __device__ __forceinline__ int row(int i, int tid) { return i * ROWS + tid / L::CH; }
    static __device__ __forceinline__ int chunk(int i, int tid) { return (tid % L::CH) ^ L::swz(row(i, tid)); }

    __device__ __forceinline__ void start(const char* base, int64_t pitch, int extent, int tid)
    {
        at = (uint64_t)base;
        ld = (uint32_t)pitch;
        ext = extent < EXT ? extent : EXT;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int c = chunk(i, tid);
            off[i] = COLS && 8 * c >= ext ? kBeyond : (uint32_t)row(i, tid) * ld + 16u * (uint32_t)c;
        }
    }
    // leaves out the first steps
    __device__ __forceinline__ void skip(int steps) { at += (uint64_t)steps * (COLS ? (uint64_t)C::BK * ld : (uint64_t)(2 * C::BK)); }
    template <int... I>
    __device__ __forceinline__ void issue(u32x4 rs, uint32_t dst, const uint32_t (&o)[LOADS], std::integer_sequence<int, I...>)
    {
        (attn::load_to_lds<I * C::THREADS * 16>(rs, dst, o[I]), ...);
    }
    // the next step, of which `left` elements of the contraction are there, to
    // dst (the wave's first 1024 bytes of the side)
    __device__ __forceinline__ void next(uint32_t dst, int left, int tid)
    {
        const bool any = left > 0 && ext > 0;
        uint32_t bytes = 0;
        if (COLS)
            bytes = any ? (uint32_t)((left < C::BK ? left : C::BK) - 1) * ld + 2u * (uint32_t)ext : 0u;
        else
            bytes = any ? (uint32_t)(ext - 1) * ld + 2u * (uint32_t)(left < C::BK ? left : C::BK) : 0u;
        const u32x4 rs = {(uint32_t)at, (uint32_t)(at >> 32) & 0xffffu, bytes, 0x00020000u};
        if (!COLS && left < C::BK) {   // the last step: chunks behind the end of a row that is not the last
            uint32_t o[LOADS];
#pragma unroll
            for (int i = 0; i < LOADS; ++i) o[i] = 8 * chunk(i, tid) >= left ? kBeyond : off[i];
            issue(rs, dst, o, std::make_integer_sequence<int, LOADS>());
        } else {
            issue(rs, dst, off, std::make_integer_sequence<int, LOADS>());
        }
        at += COLS ? (uint64_t)C::BK * ld : (uint64_t)(2 * C::BK);
    }
};

// A lane's addresses of fragments (32 rows or columns by 16 of the
// contraction: lane l has row or column l % 32 and elements 8 (l / 32) .. + 7),
// for blocks of 32 and steps of 16.
template <class C, bool COLS, int EXT, int BLOCKS>
struct Frags {
    using L = Tile<COLS, EXT, C::BK>;
    static constexpr int N = COLS ? BLOCKS : C::KSUB;
    uint32_t a[N];

    // first: the wave's first row or column; k0: its first element of a step
    __device__ __forceinline__ void start(uint32_t lds, int first, int k0, int lane)
    {
        const int half = lane >> 5, i16 = lane & 15;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            if (COLS) {
                const int r = k0 + 8 * half + (i16 >> 2);   // k0 is a multiple of 16
                const int c = (first + 32 * n) / 8 + (EXT == 16 ? 0 : ((lane >> 4) & 1) << 1) + ((i16 & 3) >> 1);
                a[n] = lds + r * L::PITCH + ((c ^ L::swz(r)) << 4) + ((i16 & 1) << 3);
            } else {
                const int r = first + (lane & (EXT == 16 ? 15 : 31)), c = k0 / 8 + 2 * n + half;
                a[n] = lds + r * L::PITCH + ((c ^ L::swz(r)) << 4);
            }
        }
    }
    __device__ __forceinline__ u32x4 read(uint32_t stage, int block, int step) const
    {
        if (COLS) {   // rows + 4 and + 16 leave the swizzle as it is
            const uint32_t p = a[block] + stage + (uint32_t)(16 * step * L::PITCH);
            const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((G16_LDS s16x4*)(uintptr_t)p));
            const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((G16_LDS s16x4*)(uintptr_t)(p + 4 * L::PITCH)));
            return u32x4{lo[0], lo[1], hi[0], hi[1]};
        }
        return *reinterpret_cast<const G16_LDS u32x4*>((uintptr_t)(a[step] + stage + (uint32_t)(32 * block * L::PITCH)));
    }
};

// Waits until at most N of the wave's loads to LDS are in flight and its LDS
// reads are done, then for the other waves.
template <int N>
__device__ __forceinline__ void publish()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
    __builtin_amdgcn_sched_barrier(0);
}

template <class C>
using Acc = f32x16[C::FM][C::FN];

// One step of a stage.
template <typename T, class C, bool XC, bool YC>
__device__ __forceinline__ void multiply(const Frags<C, XC, C::BM, C::FM>& fx, const Frags<C, YC, C::BN, C::FN>& fy, uint32_t stage, Acc<C>& acc)
{
#pragma unroll
    for (int s = 0; s < C::KSUB; ++s) {
        u32x4 x[C::FM], y[C::FN];
#pragma unroll
        for (int i = 0; i < C::FM; ++i) x[i] = fx.read(stage, i, s);
#pragma unroll
        for (int j = 0; j < C::FN; ++j) y[j] = fy.read(stage, j, s);
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
            for (int j = 0; j < C::FN; ++j) acc[i][j] = T::mfma(y[j], x[i], acc[i][j]);
    }
}

// Between what lanes of a wave write to LDS and what others of it read: the wave
// does both in order, and the compiler has to keep that order.
__device__ __forceinline__ void wave_in_order()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Adds the sums of the waves along the contraction to those of the first.
template <class C>
__device__ __forceinline__ void add_waves(char* smem, int wk, int lane, Acc<C>& acc)
{
    if constexpr (C::WK > 1) {
        static_assert(C::WM == 1 && C::WN == 1, "the waves of one tile");
        static_assert((C::WK - 1) * C::FM * C::FN * 4096 <= C::LDS, "LDS budget");
        f32x4* to = reinterpret_cast<f32x4*>(smem) + lane;
        if (wk > 0) {
#pragma unroll
            for (int b = 0; b < C::FM * C::FN; ++b)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const f32x16& v = acc[b / C::FN][b % C::FN];
                    to[(((wk - 1) * C::FM * C::FN + b) * 4 + g) * 64] = f32x4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
                }
        }
        __syncthreads();
        if (wk == 0) {
#pragma unroll
            for (int w = 1; w < C::WK; ++w)
#pragma unroll
                for (int b = 0; b < C::FM * C::FN; ++b)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const f32x4 v = to[(((w - 1) * C::FM * C::FN + b) * 4 + g) * 64];
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[b / C::FN][b % C::FN][4 * g + e] += v[e];
                    }
        }
    }
}

// A 32-bit value as two operands of 16 bits: the upper one, and what it leaves,
// which T::pack rounds.  Off by at most 2^-16 of the value in bf16, by 2^-20 of
// it or 2^-25 in fp16, where they reach twice the type's largest value.  Both
// have the value's sign, and neither is zero unless the value is (in fp16: is
// below 2^-24), so that an infinite factor of theirs makes one infinity; of an
// infinite value the upper is the type's largest and the lower infinite.
template <typename T>
__device__ __forceinline__ float upper(float x)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    if constexpr (std::is_same<T, F16>::value) {
        // a step of 32 bits less, so that something is left, and 2^-24 less, so
        // that it is no less than that; of 0 the first is no number, and 0 is what is left
        const float least = __builtin_bit_cast(float, b - 1u) - __builtin_copysignf(0x1p-24f, x);
        return (float)__builtin_amdgcn_cvt_pkrtz(__builtin_amdgcn_fmed3f(least, 0.f, x), 0.f)[0];
    } else {
        return __builtin_bit_cast(float, (x != 0.f ? b - 1u : 0u) & 0xffff0000u);
    }
}
// Both terms of two values.
struct Terms {
    uint32_t upper, lower;
};
template <typename T>
__device__ __forceinline__ Terms terms(float x, float y)
{
    const float a = upper<T>(x), b = upper<T>(y);
    return {T::pack(a, b), T::pack(x - a, y - b)};
}

// Writes a wave's blocks, its first row and column at `d`: rounded (or as they
// are, F32), through LDS so that a store covers whole lines.  `rows` and `cols`
// say how many are there; columns come in eights.
template <typename T, class C, bool F32>
__device__ __forceinline__ void store(char* lds, char* d, int64_t ld, int rows, int cols, const Acc<C>& acc, int lane)
{
    constexpr int SIZE = F32 ? 4 : 2, PITCH = C::FN * 32 * SIZE, CH = PITCH / 16, PER = 64 / CH;
    static_assert(CH <= 64, "a store covers whole rows");
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
        const int r = lane & 31, half = lane >> 5;
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4 v = f32x4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
                if constexpr (F32) {
                    const int c = 8 * j + 2 * g + half;
                    *reinterpret_cast<f32x4*>(lds + r * PITCH + ((c ^ (r % CH)) << 4)) = v;
                } else {
                    const int c = 4 * j + g;
                    *reinterpret_cast<u32x2*>(lds + r * PITCH + ((c ^ (r % CH)) << 4) + 8 * half) = u32x2{T::pack(v[0], v[1]), T::pack(v[2], v[3])};
                }
            }
        wave_in_order();
#pragma unroll
        for (int q = 0; q < 32 / PER; ++q) {
            const int y = q * PER + lane / CH, c = lane % CH;
            const u32x4 v = *reinterpret_cast<const u32x4*>(lds + y * PITCH + ((c ^ (y % CH)) << 4));
            if ((C::BM > 16 || y < 16) && (C::BN > 16 || c * (16 / SIZE) < 16) && 32 * i + y < rows && c * (16 / SIZE) < cols)
                *reinterpret_cast<u32x4*>(d + (int64_t)(32 * i + y) * ld + 16 * c) = v;
        }
        wave_in_order();
    }
}

}  // namespace grp
}  // namespace g16
