// C-ABI boundary and kernels of the grouped products and of the product with
// low-rank adapters: argument validation (before any HIP call), device checks,
// plans and launches.  The contract of every entry point is in
// include/grouped.h, the shared device code in grouped_core.hpp.
#include "grouped.h"

#include <hip/hip_runtime.h>

#include <cmath>

#include "grouped_core.hpp"
#include "grouped_ring.hpp"
#include "host.hpp"

using namespace g16;
using namespace g16::host;

namespace {

using attn::Div;
using grp::Acc;
using grp::BF16;
using grp::Cfg;
using grp::F16;

// What a launch computes.  NT, NN and TN are the three products of a group;
// LOW the adapters' projections onto their rank, a product NT whose matrix a
// table chooses and whose result is scaled; ADAPT the shared projection, with
// the adapters' second products added to the same sums; EACH the same in large
// tiles, which have rows of one request each, for ranks up to 32, and EACH2 for
// ranks above.  LOW's results are operands of the second product, as two terms
// each (grp::upper): the matrix cores take 32-bit operands at a sixteenth of
// the rate, and one term of 16 bits shows in the outputs (bf16, rank 64: 1.4e-3
// of their norm off the 32-bit values; with two 8.6e-5, as sums in another
// order).  What that costs: requests of some ten rows and a rank of 16, 35.0 us
// for 34.1, of 128 58.3 for 49.8 (90 of them, 2304 x 2048); prompts of rank 64
// 177.6 for 177.0 (4096 x 4096, 6206 rows).
enum Mode { NT, NN, TN, LOW, ADAPT, EACH, EACH2 };
constexpr bool each_request(int mode) { return mode == EACH || mode == EACH2; }

struct Args {
    const char* x;
    const char* y;
    char* d;
    const int32_t* cu;
    int64_t x_ld, y_ld, y_mat, d_ld, d_mat;   // bytes
    int groups;          // or requests
    int rows;            // of the tensors that cu divides
    int cols;            // of D
    int x_cols;          // TN: rows of a group's D, which are columns of X
    int depth;           // the contraction, except for TN
    int low_rows;        // LOW: rows of `down`; columns behind them are zeros, whatever A holds
    int rank;            // EACH, EACH2
    Div col_tiles;
    Div per_group;       // TN: tiles of a group, padded to whole rounds of the XCDs
    uint32_t group_tiles;
    int sorted;          // TN: the longest groups first
    uint32_t row_tiles;  // of all groups, at most
    Div splits;          // parts of the contraction, whose sums a second launch joins
    float* parts;
    uint32_t walkers;    // workgroups of the launch of large tiles
    // adapters
    const int32_t* ids;
    const float* scales;
    const char* low;     // LOW's results, rows of `rank` (EACH, EACH2: of 128 bytes)
    int64_t low_rest;    // bytes from their upper to their lower terms
    const char* down;
    int64_t down_ld, down_mat;
    const char* up;
    int64_t up_ld, up_mat;
    int adapters;
    Div rank_chunks;
    Div term_chunks;     // twice as many: both terms
};

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

// A group's rows.  Offsets are clamped to the tensor, so that a table that
// decreases or runs past it still names rows that exist.
struct Rows {
    int first, count;
};
__device__ __forceinline__ Rows rows_of(const Args& g, int e)
{
    const int a = clampi(g.cu[e], 0, g.rows);
    return {a, clampi(g.cu[e + 1], a, g.rows) - a};
}

// Inclusive sum over the lanes.
__device__ __forceinline__ uint32_t wave_scan(uint32_t x)
{
    auto add = [&](auto ctrl, auto rows) {
        x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, decltype(ctrl)::value, decltype(rows)::value, 0xf, false);
    };
    using std::integral_constant;
    add(integral_constant<int, 0x111>(), integral_constant<int, 0xf>());   // 1, 2, 4 and 8 lanes up within 16
    add(integral_constant<int, 0x112>(), integral_constant<int, 0xf>());
    add(integral_constant<int, 0x114>(), integral_constant<int, 0xf>());
    add(integral_constant<int, 0x118>(), integral_constant<int, 0xf>());
    add(integral_constant<int, 0x142>(), integral_constant<int, 0xa>());   // lane 15 of a row of 16 to the next row,
    add(integral_constant<int, 0x143>(), integral_constant<int, 0xc>());   // lane 31 to the upper half
    return x;
}

// A workgroup's tile: the group, its first row, how many rows there are from
// the tile's first row on (TN: in the group), and the tile's first column.
struct Work {
    int group, row0, rows, tile0, col0;   // tile0: the tile's first row within the group (TN: of D)
    bool found;
};

constexpr uint32_t kGroupTiles = 4;   // row tiles that neighbours share columns over

// Row tiles of BM, those of all groups one after the other.  Each lane looks at
// one group, 64 at a time; with up to 64 groups it keeps what it saw.
template <int BM, int MODE>
struct Groups {
    Rows s;
    uint32_t tiles, upto, total;
    uint32_t place;   // TN: the lane's group among all, the longest first

    __device__ __forceinline__ void look(const Args& g, int e, int groups)
    {
        s = Rows{0, 0};
        if (e < groups) {
            if (MODE == ADAPT) {   // requests are neighbours: one run of rows
                const int a = clampi(g.cu[0], 0, g.rows);
                s = Rows{a, clampi(g.cu[g.groups], a, g.rows) - a};
            } else {
                s = rows_of(g, e);
                if (MODE == LOW && (uint32_t)g.ids[e] >= (uint32_t)g.adapters) s.count = 0;
            }
        }
        tiles = (uint32_t)(s.count + BM - 1) / BM;
        upto = wave_scan(tiles);
    }
    __device__ __forceinline__ void start(const Args& g)
    {
        const int groups = MODE == ADAPT ? 1 : g.groups, lane = threadIdx.x & 63;
        total = 0;
        for (int base = 0; base < groups; base += 64) {
            look(g, base + lane, groups);
            total += (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
        }
        // a table that decreases can name rows more than once: no more tiles
        // than the launch and the room for parts were made for
        if (total > g.row_tiles) total = g.row_tiles;
    }
    // TN: all groups have as many tiles, which take as long as their groups do.
    // Where the host says so the longest come first, so that what is left for
    // the end is short.
    __device__ __forceinline__ void order(const Args& g)
    {
        const int lane = threadIdx.x & 63;
        place = 0;
        if (!g.sorted) return;
        const int mine = lane < g.groups ? rows_of(g, lane).count : -1;
        for (int e = 0; e < g.groups; ++e) {
            const int other = __builtin_amdgcn_readlane(mine, e);
            place += other > mine || (other == mine && e < lane);
        }
    }
    __device__ __forceinline__ uint32_t at(const Args& g, uint32_t p) const
    {
        return !g.sorted ? p : (uint32_t)__builtin_ctzll(__builtin_amdgcn_ballot_w64(place == p));
    }
    // Tile t of `total`.
    __device__ __forceinline__ Work find(const Args& g, uint32_t t)
    {
        const int groups = MODE == ADAPT ? 1 : g.groups, lane = threadIdx.x & 63;
        uint32_t before = 0;
        for (int base = 0; base < groups; base += 64) {
            if (groups > 64) look(g, base + lane, groups);
            const uint64_t past = __builtin_amdgcn_ballot_w64(before + upto > t);
            if (past != 0) {
                const int w = __builtin_ctzll(past);
                const int first = __builtin_amdgcn_readlane(s.first, w), count = __builtin_amdgcn_readlane(s.count, w);
                const uint32_t start = before + (uint32_t)__builtin_amdgcn_readlane((int)upto, w) - (uint32_t)__builtin_amdgcn_readlane((int)tiles, w);
                const int tile0 = (int)(t - start) * BM;
                return Work{base + w, first + tile0, count - tile0, tile0, 0, true};
            }
            before += (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
        }
        return Work{0, 0, 0, 0, 0, false};
    }
};

// Tile `t` of all tiles in the order that the launches share.
template <int BM, int BN, int MODE>
__device__ __forceinline__ Work tile_at(const Args& g, Groups<BM, MODE>& groups, uint32_t t)
{
    uint32_t ti, tj;
    Work r;
    if (MODE == TN) {
        const uint32_t p = t / g.group_tiles, e = groups.at(g, p);
        grouped_tile_in<uint32_t>(t - p * g.group_tiles, g.group_tiles / g.col_tiles.d, g.col_tiles.d, kGroupTiles, &ti, &tj);
        const Rows s = rows_of(g, (int)e);
        r = Work{(int)e, s.first, s.count, (int)ti * BM, 0, true};
    } else {
        grouped_tile_in<uint32_t>(t, groups.total, g.col_tiles.d, kGroupTiles, &ti, &tj);
        r = groups.find(g, ti);
    }
    r.col0 = (int)tj * BN;
    return r;
}

// How many tiles there are.
template <int BM, int MODE>
__device__ __forceinline__ uint32_t all_tiles(const Args& g, Groups<BM, MODE>& groups)
{
    if (MODE == TN) {
        groups.order(g);
        return (uint32_t)g.groups * g.group_tiles;
    }
    groups.start(g);
    return groups.total * g.col_tiles.d;
}

// A workgroup's tile and part; `slot` is the place of its sums among the parts'.
template <int BM, int BN, int MODE, bool SPLIT>
__device__ __forceinline__ Work find_work(const Args& g, uint32_t index, uint32_t* part, uint32_t* slot)
{
    Groups<BM, MODE> groups;
    const uint32_t all = all_tiles<BM, MODE>(g, groups);
    uint32_t t;
    *part = 0;
    if (MODE == TN) {
        uint32_t i = index;
        if (SPLIT) {
            const uint32_t launch = g.per_group.d * (uint32_t)g.groups;
            *part = i / launch;
            i -= *part * launch;
        }
        const uint32_t e = g.per_group.of(i);
        i -= e * g.per_group.d;
        // whole rounds of the XCDs: each has a part of the group's tiles of its own
        t = g.per_group.d == g.group_tiles ? i : (uint32_t)xcd_slot(i, g.per_group.d);
        if (t >= g.group_tiles) return Work{0, 0, 0, 0, 0, false};
        t += e * g.group_tiles;
    } else {
        const uint32_t n = SPLIT ? all * g.splits.d : all;
        if (index >= n) return Work{0, 0, 0, 0, 0, false};
        // each XCD has a run of neighbouring tiles, whose rows and columns its L2 holds
        t = (uint32_t)xcd_slot(index, n);
        if (SPLIT) {
            *part = t / all;
            t -= *part * all;
        }
    }
    *slot = *part * all + t;
    return tile_at<BM, BN, MODE>(g, groups, t);
}

// How many tiles a part has.
template <int BM, int MODE>
__device__ __forceinline__ uint32_t slot_count(const Args& g)
{
    Groups<BM, MODE> groups;
    return all_tiles<BM, MODE>(g, groups);
}

// 16 zero bytes for chunks that belong to no request.
__device__ __attribute__((aligned(16))) uint32_t g_nothing[4] = {0, 0, 0, 0};

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"   // M0 is written inside, on purpose
template <int AT>
__device__ __forceinline__ void load_to_lds_from(const char* p, uint32_t dst)
{
    asm volatile("s_add_u32 m0, %0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"(dst), "v"(p), "n"(AT) : "memory", "m0", "scc");
}
#pragma clang diagnostic pop

template <int STEP, int... I>
__device__ __forceinline__ void load_all(const char* const* p, uint32_t dst, std::integer_sequence<int, I...>)
{
    (load_to_lds_from<I * STEP>(p[I], dst), ...);
}

// ADAPT: the adapters' second products are more of the contraction.  The
// requests with an adapter that a tile's rows belong to, one after the other,
// have twice `rank` elements of it each, the upper and the lower terms of what
// LOW left, in which a row meets its own request's part and zeros elsewhere.  A
// table in LDS says which they are.
struct alignas(8) Entry {
    int16_t first, end;   // rows of the tile
    int32_t id;
};

// Fills the table and returns how many requests there are; by one wave.
template <int BM>
__device__ __forceinline__ int fill_table(const Args& g, const Work& wk, Entry* table)
{
    const int lane = threadIdx.x & 63, end = wk.rows < BM ? wk.rows : BM;
    int count = 0;
    for (int base = 0; base < g.groups; base += 64) {
        const int b = base + lane;
        int lo = end, hi = end, id = -1;
        if (b < g.groups) {
            lo = clampi(g.cu[b] - wk.row0, 0, end);
            hi = clampi(g.cu[b + 1] - wk.row0, lo, end);
            id = g.ids[b];
        }
        const bool there = hi > lo && (uint32_t)id < (uint32_t)g.adapters;
        const uint64_t all = __builtin_amdgcn_ballot_w64(there);
        const int at = count + __builtin_popcountll(all & ((uint64_t(1) << lane) - 1));
        // a table of offsets that does not decrease has at most a request for each row
        if (there && at < BM) table[at] = Entry{(int16_t)lo, (int16_t)hi, id};
        count += __builtin_popcountll(all);
        if (__builtin_amdgcn_ballot_w64(b < g.groups && lo >= end) != 0) break;   // requests behind the tile
    }
    return count < BM ? count : BM;
}

// Whose a chunk of the requests' part of the contraction is, and which of its.
// Without a branch: loads of several chunks then look it up at once.
__device__ __forceinline__ Entry entry_of(const Args& g, const Entry* table, int count, int at, int* in)
{
    const int q = (int)g.term_chunks.of((uint32_t)at);
    *in = at - q * (int)g.term_chunks.d;
    Entry e = table[q < count ? q : count - 1];
    if (q >= count) {
        e.end = e.first;
        e.id = -1;
    }
    return e;
}

// The loads of step s of the requests' part of the contraction; `low` is the
// tile's first row.
template <class C>
__device__ __forceinline__ void load_requests(const Args& g, const Work& wk, const Entry* table, int count, const char* low, int s, uint32_t dst, int tid)
{
    using SX = grp::Side<C, false, C::BM>;
    using SY = grp::Side<C, false, C::BN>;
    const char* px[SX::LOADS];
    const char* py[SY::LOADS];
    const int chunks = (int)g.rank_chunks.d;
    auto where = [&](int chunk, int* in) {
        return entry_of(g, table, count, s * (C::BK / 8) + chunk, in);
    };
#pragma unroll
    for (int i = 0; i < SX::LOADS; ++i) {
        int in;
        const Entry e = where(SX::chunk(i, tid), &in);
        const int r = SX::row(i, tid);
        const char* p = low + (int64_t)r * (16 * chunks) + 16 * in + (in < chunks ? 0 : g.low_rest - 16 * chunks);
        px[i] = r >= e.first && r < e.end ? p : (const char*)g_nothing;
    }
#pragma unroll
    for (int i = 0; i < SY::LOADS; ++i) {
        int in;
        const Entry e = where(SY::chunk(i, tid), &in);
        const int r = wk.col0 + SY::row(i, tid);
        py[i] = e.id >= 0 && r < g.cols ? g.up + (int64_t)e.id * g.up_mat + (int64_t)r * g.up_ld + 16 * (in < chunks ? in : in - chunks) : (const char*)g_nothing;
    }
    load_all<C::THREADS * 16>(px, dst, std::make_integer_sequence<int, SX::LOADS>());
    load_all<C::THREADS * 16>(py, dst + C::X_BYTES, std::make_integer_sequence<int, SY::LOADS>());
}

// The values of each half of a register that are an infinity or a NaN: the
// sign's bit of the half is set.
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t v)
{
    constexpr uint32_t EXP = std::is_same<T, F16>::value ? 0x7c007c00u : 0x7f807f80u;   // all ones, plus one
    return ((v & EXP) + (0x80008000u - EXP)) & 0x80008000u;
}

// One step of the requests' part of the contraction.  The zeros that a row has
// for other requests keep their matrices out of its sums as long as these are
// finite, so what is not is left out here, and added by store_not_finite to the
// rows that it belongs to.  Returns whether there was any.
template <typename T, class C>
__device__ __forceinline__ bool multiply_requests(const grp::Frags<C, false, C::BM, C::FM>& fx, const grp::Frags<C, false, C::BN, C::FN>& fy, uint32_t stage,
                                                  Acc<C>& acc)
{
    bool any = false;
#pragma unroll
    for (int s = 0; s < C::KSUB; ++s) {
        u32x4 x[C::FM], y[C::FN];
#pragma unroll
        for (int i = 0; i < C::FM; ++i) x[i] = fx.read(stage, i, s);
        uint32_t bad = 0;
#pragma unroll
        for (int j = 0; j < C::FN; ++j) {
            y[j] = fy.read(stage, j, s);
#pragma unroll
            for (int e = 0; e < 4; ++e) bad |= not_finite<T>(y[j][e]);
        }
        if (__builtin_amdgcn_ballot_w64(bad != 0) != 0) {
            any = true;
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) y[j][e] &= ~((not_finite<T>(y[j][e]) >> 15) * 0xffffu);
        }
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
            for (int j = 0; j < C::FN; ++j) acc[i][j] = T::mfma(y[j], x[i], acc[i][j]);
    }
    return any;
}

// Writes a wave's blocks as grp::store does, one value at a time, and adds the
// products with what is not finite to them before they are rounded: a finite
// sum beyond fp16's largest value is no infinity here.  The blocks are the
// tile's rows from r0 on and D's columns from c0 on; `low` is the tile's first
// row.
template <typename T, class C, bool F32>
__device__ __forceinline__ void store_not_finite(const Args& g, const Entry* table, int count, const char* low, char* lds, char* d, int64_t ld, int r0, int c0,
                                                 int rows, int cols, const Acc<C>& acc, int lane)
{
    constexpr int W = 32 * C::FN, ROWS = C::BM == 16 ? 16 : 32, COLS = C::BN == 16 ? 16 : W;
    const int64_t low_ld = 16 * (int64_t)g.rank_chunks.d;
    float* to = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
#pragma unroll
        for (int b = 0; b < 4 * C::FN; ++b) {
            const f32x16& v = acc[i][b / 4];
            const int at = 4 * (b % 4);
            *reinterpret_cast<f32x4*>(to + (lane & 31) * W + 8 * b + 4 * (lane >> 5)) = f32x4{v[at], v[at + 1], v[at + 2], v[at + 3]};
        }
        grp::wave_in_order();
        for (int x = lane; x < 32 * W; x += 64) {
            const int r = x / W, c = x % W, row = r0 + 32 * i + r;
            if (r >= ROWS || c >= COLS || 32 * i + r >= rows || c >= cols) continue;
            float v = to[x];
            for (int q = 0; q < count; ++q) {
                const Entry e = table[q];
                if (row < e.first || row >= e.end) continue;
                const char* up = g.up + (int64_t)e.id * g.up_mat + (int64_t)(c0 + c) * g.up_ld;
                for (int p = 0; p < (int)low_ld; p += 4) {   // two ranks
                    const uint32_t u2 = *reinterpret_cast<const uint32_t*>(up + p), bad = not_finite<T>(u2);
                    if (bad == 0) continue;
                    const char* h2 = low + row * low_ld + p;
                    const attn::f32x2 u = T::unpack(u2), h = T::unpack(*reinterpret_cast<const uint32_t*>(h2)) +
                                                             T::unpack(*reinterpret_cast<const uint32_t*>(h2 + g.low_rest));
                    v += (bad & 0x8000u ? h[0] * u[0] : 0.f) + (bad & 0x80000000u ? h[1] * u[1] : 0.f);
                }
            }
            char* at = d + (int64_t)(32 * i + r) * ld + (F32 ? 4 : 2) * c;
            if constexpr (F32)
                *reinterpret_cast<float*>(at) = v;
            else
                *reinterpret_cast<uint16_t*>(at) = (uint16_t)T::pack(v, 0.f);
        }
        grp::wave_in_order();
    }
}

// What becomes of a tile's sums.  ROUNDED: they are outputs.  PART: of a part of
// the contraction, in fp32, tile by tile, for the launch that joins them.
// PLANE: the same as rows of a matrix like D, for finish_kernel.  HELD: as they
// lie in the lanes, for the launch of tiles that has them as FIRST sums, before
// the requests' part of the contraction, and no other.
enum Sums { ROUNDED, PART, PLANE, HELD, FIRST };

template <class C, int MODE>
constexpr int kTileLds = C::LDS + (MODE == ADAPT ? C::BM * (int)sizeof(Entry) + 16 : 0);

// A tile, or a part of its contraction: steps come to LDS, STAGES - 1 of them
// ahead, while the one that is there is multiplied.
//
// Few rows wait for the matrices' bytes, so tiles are small, for many
// workgroups, and their steps long: 96 KiB are on the way on each compute unit
// and four waves divide the step among them (512 rows over 64 matrices of 2048 x
// 4096: 194 us, 5.2 TB/s; 8 rows over 16 of 1024 x 2048: 8 us).  With 50 to some
// hundreds of rows for a matrix tiles grow, since LDS reads and loads from L2
// bound them: 64 x 128 by two workgroups on a compute unit have 775 TFLOP/s, 128
// x 128 some 1000.  Larger ones are ring_kernel's.
template <typename T, class C, int MODE, bool F32, Sums SUMS>
__device__ __forceinline__ void tile_body(const Args& g, char* smem, uint32_t index)
{
    constexpr bool XC = MODE == TN, YC = MODE == NN || MODE == TN, SPLIT = SUMS == PART || SUMS == PLANE || SUMS == HELD;
    uint32_t part, slot;
    const Work wk = find_work<C::BM, C::BN, MODE, SPLIT>(g, index, &part, &slot);
    if (!wk.found) return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int k = w % C::WK, wn = (w / C::WK) % C::WN, wm = w / C::WK / C::WN;

    grp::Side<C, XC, C::BM> x;
    grp::Side<C, YC, C::BN> y;
    int depth = g.depth;
    if (MODE == TN) {
        depth = wk.rows;
        x.start(g.x + (int64_t)wk.row0 * g.x_ld + 2 * (int64_t)wk.tile0, g.x_ld, g.x_cols - wk.tile0, tid);
        y.start(g.y + (int64_t)wk.row0 * g.y_ld + 2 * (int64_t)wk.col0, g.y_ld, g.cols - wk.col0, tid);
    } else {
        const int m = MODE == LOW ? g.ids[wk.group] : MODE == ADAPT ? 0 : wk.group;
        const char* mat = g.y + (int64_t)m * g.y_mat;
        x.start(g.x + (int64_t)wk.row0 * g.x_ld, g.x_ld, wk.rows, tid);
        if (MODE == NN)
            y.start(mat + 2 * (int64_t)wk.col0, g.y_ld, g.cols - wk.col0, tid);
        else
            y.start(mat + (int64_t)wk.col0 * g.y_ld, g.y_ld, (MODE == LOW ? g.low_rows : g.cols) - wk.col0, tid);
    }
    const uint32_t lds = attn::lds_address(smem), mine = lds + 1024u * (uint32_t)w;
    grp::Frags<C, XC, C::BM, C::FM> fx;
    grp::Frags<C, YC, C::BN, C::FN> fy;
    fx.start(lds, wm * C::FM * 32, k * (C::BK / C::WK), lane);
    fy.start(lds + C::X_BYTES, wn * C::FN * 32, k * (C::BK / C::WK), lane);

    Acc<C> acc;
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) acc[i][j] = f32x16{};

    // Step s is loaded into stage s % STAGES while the STAGES - 1 steps before
    // it are multiplied; steps behind the last load zeros, so that every wait
    // counts the same loads.
    int steps = (depth + C::BK - 1) / C::BK, left = depth;
    if (SPLIT) {
        const int per = (int)g.splits.of((uint32_t)steps + g.splits.d - 1), first = (int)part * per;
        steps = clampi(steps - first, 0, per);
        x.skip(first);
        y.skip(first);
        left = clampi(depth - first * C::BK, 0, steps * C::BK);
    }
    auto held = [&](uint32_t p, int block, int q) {   // a lane's four of the sums in part p
        return (f32x4*)g.parts + ((((int64_t)p * C::WAVES + w) * (C::FM * C::FN) + block) * 4 + q) * 64 + lane;
    };
    if constexpr (SUMS == FIRST) {
        static_assert(C::WK == 1, "every wave has sums");
        steps = left = 0;
        const uint32_t all = slot_count<C::BM, MODE>(g);
        for (uint32_t p = 0; p < g.splits.d; ++p)
#pragma unroll
            for (int b = 0; b < C::FM * C::FN; ++b)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x4 v = *held(p * all + slot, b, q);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[b / C::FN][b % C::FN][4 * q + e] += v[e];
                }
    }
    uint32_t fill = 0;
    auto load = [&] {
        x.next(mine + fill, left, tid);
        y.next(mine + fill + C::X_BYTES, left, tid);
        left -= C::BK;
        fill = fill == (C::STAGES - 1) * C::STAGE ? 0 : fill + C::STAGE;
    };
    Entry* table = reinterpret_cast<Entry*>(smem + C::LDS);
    int requests = 0, next = 0;   // ADAPT: of the tile; the next step of theirs
    const int shared = steps;     // the steps before theirs
    bool bad = false;             // whether their matrices hold what is not finite
    const char* low = MODE != ADAPT ? nullptr : g.low + (int64_t)wk.row0 * (16 * g.rank_chunks.d);
    auto load_more = [&] {
        if (MODE == ADAPT && left <= 0 && requests > 0) {
            load_requests<C>(g, wk, table, requests, low, next++, mine + fill, tid);
            fill = fill == (C::STAGES - 1) * C::STAGE ? 0 : fill + C::STAGE;
        } else {
            load();
        }
    };
    int* count = reinterpret_cast<int*>(table + C::BM);   // and, behind it, whether any wave found such values
    if (MODE == ADAPT && g.adapters > 0 && (!SPLIT || part + 1 == g.splits.d)) {   // the requests go with the last part
        const int own = steps < C::STAGES - 1 ? steps : C::STAGES - 1;
        for (int s = 0; s < own; ++s) load();
        if (w == 0) {
            const int n = fill_table<C::BM>(g, wk, table);
            if (lane == 0) {
                count[0] = n;
                count[1] = 0;
            }
        }
        __syncthreads();
        requests = __builtin_amdgcn_readfirstlane(*count);
        for (int s = own; s < C::STAGES - 1; ++s) load_more();
        steps += (requests * (int)g.term_chunks.d + C::BK / 8 - 1) / (C::BK / 8);
    } else {
        for (int s = 0; s < C::STAGES - 1; ++s) load();
    }
    const bool busy = MODE == TN || wk.rows > wm * C::FM * 32;   // the wave has rows
    uint32_t stage = 0;
    for (int s = 0; s < shared; ++s) {
        grp::publish<(C::STAGES - 2) * C::LOADS>();
        load_more();
        if (busy) grp::multiply<T, C>(fx, fy, stage, acc);
        stage = stage == (C::STAGES - 1) * C::STAGE ? 0 : stage + C::STAGE;
    }
    if constexpr (MODE == ADAPT) {
        for (int s = shared; s < steps; ++s) {
            grp::publish<(C::STAGES - 2) * C::LOADS>();
            load_more();
            if (busy) bad |= multiply_requests<T, C>(fx, fy, stage, acc);
            stage = stage == (C::STAGES - 1) * C::STAGE ? 0 : stage + C::STAGE;
        }
    }
    if (MODE == ADAPT && bad) count[1] = 1;
    grp::publish<0>();
    grp::add_waves<C>(smem, k, lane, acc);
    if (k > 0) return;
    bad = MODE == ADAPT && requests > 0 && __builtin_amdgcn_readfirstlane(count[1]) != 0;

    const int r0 = wm * C::FM * 32, c0 = wn * C::FN * 32, rows = (MODE == TN ? g.x_cols - wk.tile0 : wk.rows) - r0, cols = g.cols - wk.col0 - c0;
    constexpr bool WIDE = F32 || SPLIT || MODE == ADAPT;
    constexpr int STAGING = C::FN * 32 * 32 * (WIDE ? 4 : 2);
    constexpr int AFTER = (C::WK - 1) * C::FM * C::FN * 4096;   // the other waves' sums
    static_assert(AFTER + C::WM * C::WN * STAGING <= C::LDS, "LDS budget");
    char* staging = smem + AFTER + (wm * C::WN + wn) * STAGING;
    if constexpr (SUMS == HELD) {
#pragma unroll
        for (int b = 0; b < C::FM * C::FN; ++b)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x16& v = acc[b / C::FN][b % C::FN];
                *held(slot, b, q) = f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
            }
    } else if constexpr (SUMS == PLANE) {
        float* d = g.parts + ((int64_t)part * g.rows + wk.row0 + r0) * g.cols + wk.col0 + c0;
        grp::store<T, C, true>(staging, (char*)d, 4 * (int64_t)g.cols, rows, cols, acc, lane);
    } else if constexpr (SUMS == PART) {
        char* d = (char*)(g.parts + (int64_t)slot * (C::BM * C::BN) + r0 * C::BN + c0);
        if (MODE == ADAPT && bad)
            store_not_finite<T, C, true>(g, table, requests, low, staging, d, 4 * C::BN, r0, wk.col0 + c0, rows, cols, acc, lane);
        else
            grp::store<T, C, true>(staging, d, 4 * C::BN, rows, cols, acc, lane);
    } else {
        char* d = g.d + (MODE == TN ? (int64_t)wk.group * g.d_mat + (int64_t)(wk.tile0 + r0) * g.d_ld : (int64_t)(wk.row0 + r0) * g.d_ld) +
                  (int64_t)(wk.col0 + c0) * (F32 ? 4 : 2);
        if constexpr (MODE == LOW) {
            const float scale = g.scales != nullptr ? g.scales[g.ids[wk.group]] : 1.f;
            const int end = F32 ? C::BN : g.low_rows - wk.col0 - c0;   // the columns there are
            Acc<C> rest;   // the lower terms
#pragma unroll
            for (int i = 0; i < C::FM; ++i)
#pragma unroll
                for (int j = 0; j < C::FN; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float v = acc[i][j][e] * scale;
                        acc[i][j][e] = F32 ? v : grp::upper<T>(v);
                        rest[i][j][e] = v - acc[i][j][e];
                    }
            if (end < 32 * C::FN && end < cols) {
#pragma unroll
                for (int i = 0; i < C::FM; ++i)
#pragma unroll
                    for (int j = 0; j < C::FN; ++j)
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (32 * j + 8 * (e / 4) + 4 * (lane >> 5) >= end) acc[i][j][e] = rest[i][j][e] = 0.f;
            }
            grp::store<T, C, F32>(staging, d, g.d_ld, rows, cols, acc, lane);
            if constexpr (!F32) grp::store<T, C, false>(staging, d + g.low_rest, g.d_ld, rows, cols, rest, lane);
        } else if (MODE == ADAPT && bad) {
            store_not_finite<T, C, F32>(g, table, requests, low, staging, d, g.d_ld, r0, wk.col0 + c0, rows, cols, acc, lane);
        } else {
            grp::store<T, C, F32>(staging, d, g.d_ld, rows, cols, acc, lane);
        }
    }
}

// Up to 16 rows of few requests (some users' next tokens): the adapters'
// projections come with the shared one, as further columns of the same
// product, whose tile has 16 rows of the shared matrix and RB blocks of 16 rows
// of `down`, so many of each request.  Their sums are the second product's
// operand as they lie in the accumulators, two terms of each: the order of that
// contraction is free, and `up` is read to match.  What bounds it is the latency
// of a chain: arguments, the first loads, the bytes (120 KiB in flight on a
// compute unit, in stages of 24 or 40 KiB, of which 8 are the shared matrix's),
// the sums of four waves.  So the shared matrix is asked for before the requests'
// rows are known, which are read as scalars, by themselves.
template <typename T, int RB>
__global__ __launch_bounds__(256, 1) void single_kernel(const Args g)
{
    using C = Cfg<16, 16 + 16 * RB, 256, 1, 1, 4, RB == 1 ? 6 : 4, 1>;
    static_assert(RB == 1 || RB == 3, "whole blocks of 32 columns, and four stages of them");
    constexpr int FN = (RB + 1) / 2;
    using W = grp::Side<C, false, 16>;
    using X = grp::Side<C, false, 16>;
    using L = grp::Tile<false, 16, C::BK>;
    constexpr int LATE = (1 + RB) * X::LOADS, LOADS = W::LOADS + LATE;   // of a step
    __shared__ __attribute__((aligned(1024))) char smem[C::STAGES * C::STAGE];
    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t lds = attn::lds_address(smem), mine = lds + 1024u * (uint32_t)w;
    const int col0 = (int)xcd_slot(blockIdx.x, gridDim.x) * 16;

    // stage: 16 rows of the shared matrix, RB x 16 of `down`, 16 of A
    constexpr uint32_t PIECE = 16 * C::BK * 2;
    W y;
    y.start(g.y + (int64_t)col0 * g.y_ld, g.y_ld, g.cols - col0, tid);
    int y_left = g.depth;
#pragma unroll
    for (int s = 0; s < C::STAGES - 1; ++s, y_left -= C::BK) y.next(mine + s * C::STAGE, y_left, tid);

    typedef const __attribute__((address_space(4))) int32_t* Scalars;
    const Scalars cu = (Scalars)(uintptr_t)g.cu, ids = (Scalars)(uintptr_t)g.ids;
    const int row0 = clampi(cu[0], 0, g.rows), rows = clampi(cu[g.groups], row0, g.rows) - row0;
    const int rank = 8 * (int)g.rank_chunks.d, each = (rank + 15) / 16;   // blocks of a request
    X x, down[RB];
    x.start(g.x + (int64_t)row0 * g.x_ld, g.x_ld, rows, tid);
    int first[RB], end[RB];   // the rows of a block's request
    float scale[RB];
    u32x4 u[RB] = {};         // `up` for the lane's column, in the order of the accumulators
    const bool mine_up = w == 0 && (lane & 31) < 16 && col0 + (lane & 31) < g.cols;
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        const int q = b / each, part = b - q * each;
        const bool there = q < g.groups;
        first[b] = there ? cu[q] - row0 : 0;
        end[b] = there ? cu[q + 1] - row0 : 0;
        const int id = there ? ids[q] : -1;
        const bool adapted = (uint32_t)id < (uint32_t)g.adapters;
        if (!adapted) end[b] = first[b];
        const int64_t at = adapted ? id : 0;
        down[b].start(g.down + at * g.down_mat + (int64_t)(16 * part) * g.down_ld, g.down_ld, adapted ? rank - 16 * part : 0, tid);
        scale[b] = adapted && g.scales != nullptr ? ((const __attribute__((address_space(4))) float*)(uintptr_t)g.scales)[at] : 1.f;
        const char* up = g.up + at * g.up_mat + (int64_t)(col0 + (lane & 31)) * g.up_ld + 32 * part + 8 * half;
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (mine_up && adapted && 16 * part + 8 * e < rank) {
                const u32x2 v = *reinterpret_cast<const u32x2*>(up + 16 * e);
                u[b][2 * e] = v[0];
                u[b][2 * e + 1] = v[1];
            }
    }
    int left = g.depth;
    auto late = [&](uint32_t at) {
#pragma unroll
        for (int b = 0; b < RB; ++b) down[b].next(at + (1 + b) * PIECE, left, tid);
        x.next(at + (1 + RB) * PIECE, left, tid);
        left -= C::BK;
    };
#pragma unroll
    for (int s = 0; s < C::STAGES - 1; ++s) late(mine + s * C::STAGE);

    // fragments: rows l % 16 of A and l % 32 of the rest
    uint32_t fx[C::KSUB], fy[C::KSUB];
#pragma unroll
    for (int n = 0; n < C::KSUB; ++n) {
        const int c = w * (C::BK / C::WK / 8) + 2 * n + half, r = lane & 15;
        const uint32_t at = lds + (uint32_t)(r * L::PITCH + ((c ^ L::swz(r)) << 4));
        fx[n] = at + (1 + RB) * PIECE;
        fy[n] = at + (lane & 16 ? PIECE : 0);
    }
    f32x16 acc[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[j] = f32x16{};
    const int steps = (g.depth + C::BK - 1) / C::BK;
    uint32_t stage = 0, fill = (C::STAGES - 1) * C::STAGE;
    for (int s = 0; s < steps; ++s) {
        // the first stages' loads came in another order: of the later ones no
        // more than those of the stages behind may be in flight
        if (s < C::STAGES - 1)
            grp::publish<(C::STAGES - 2) * LATE>();
        else
            grp::publish<(C::STAGES - 2) * LOADS>();
        y.next(mine + fill, y_left, tid);
        y_left -= C::BK;
        late(mine + fill);
        fill = stage;
#pragma unroll
        for (int n = 0; n < C::KSUB; ++n) {
            const u32x4 a = *reinterpret_cast<const G16_LDS u32x4*>((uintptr_t)(fx[n] + stage));
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const u32x4 b = *reinterpret_cast<const G16_LDS u32x4*>((uintptr_t)(fy[n] + stage + 2 * j * PIECE));
                acc[j] = T::mfma(b, a, acc[j]);
            }
        }
        stage = stage == (C::STAGES - 1) * C::STAGE ? 0 : stage + C::STAGE;
    }
    grp::publish<0>();
    using A = Cfg<32, 32 * FN, 256, 1, 1, 4, 2, 1>;   // of whole blocks, for what follows
    static_assert(3 * FN * 4096 + 4096 <= (int)sizeof(smem), "LDS budget");
    Acc<A> sums;
#pragma unroll
    for (int j = 0; j < FN; ++j) sums[0][j] = acc[j];
    grp::add_waves<A>(smem, w, lane, sums);
    if (w > 0) return;
    f32x16 d = sums[0][0];
    const int m = lane & 31;
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        const f32x16& h = sums[0][(b + 1) / 2];
        const int at = (b + 1) % 2 * 8;
        u32x4 upper, lower;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const grp::Terms t = grp::terms<T>(h[at + 2 * i] * scale[b], h[at + 2 * i + 1] * scale[b]);
            // no row of `down` behind the rank: zeros, whatever A holds
            const bool there = 16 * (b % each) + 4 * (i & ~1) < rank;
            upper[i] = there ? t.upper : 0;
            lower[i] = there ? t.lower : 0;
        }
        const f32x16 sum = T::mfma(u[b], lower, T::mfma(u[b], upper, d));
        const bool own = m >= first[b] && m < end[b];   // a lane's sums are one row's
#pragma unroll
        for (int i = 0; i < 16; ++i) d[i] = own ? sum[i] : d[i];
    }
    using O = Cfg<16, 16, 512, 1, 1, 4, 4, 1>;
    Acc<O> out = {{d}};
    grp::store<T, O, false>(smem + 3 * FN * 4096, g.d + (int64_t)row0 * g.d_ld + 2 * (int64_t)col0, g.d_ld, rows, g.cols - col0, out, lane);
}

template <typename T, class C, int MODE, bool F32, Sums SUMS>
__global__ __launch_bounds__(C::THREADS, C::PER_CU * C::WAVES / 4) void tile_kernel(const Args g)
{
    __shared__ __attribute__((aligned(1024))) char smem[kTileLds<C, MODE>];
    tile_body<T, C, MODE, F32, SUMS>(g, smem, blockIdx.x);
}

// Few rows, or few tiles of a long contraction: the projections onto the rank,
// by the first workgroups, beside the shared product, whose sums the next launch
// puts together with the adapters' second products: finish_kernel, for which
// both are in fp32 (SUMS PLANE), or, where requests have many rows, tiles that
// have the sums as their FIRST (SUMS HELD).  64 rows, 14336 x 4096, rank 16: 23
// us, 5.2 TB/s; the call takes 39, and with the launches in turn 53.
struct PairArgs {
    Args low, base;
    uint32_t low_wgs;
};

template <typename T, class L, class C, Sums SUMS>
__global__ __launch_bounds__(256, 2) void pair_kernel(const PairArgs p)
{
    static_assert(L::THREADS == 256 && C::THREADS == 256, "one launch");
    __shared__ __attribute__((aligned(1024))) char smem[kTileLds<C, ADAPT> > kTileLds<L, LOW> ? kTileLds<C, ADAPT> : kTileLds<L, LOW>];
    if (blockIdx.x < p.low_wgs)
        tile_body<T, L, LOW, SUMS == PLANE, ROUNDED>(p.low, smem, blockIdx.x);
    else
        tile_body<T, C, ADAPT, false, SUMS>(p.base, smem, blockIdx.x - p.low_wgs);
}

// Sum over groups of L neighbouring lanes, by the lanes' own data paths.
template <int L>
__device__ __forceinline__ float sum_lanes(float x)
{
    auto add = [&](auto ctrl) {
        const int y = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), decltype(ctrl)::value, 0xf, 0xf, false);
        x += __builtin_bit_cast(float, y);
    };
    using std::integral_constant;
    if constexpr (L > 1) add(integral_constant<int, 0xb1>());    // lane ^ 1
    if constexpr (L > 2) add(integral_constant<int, 0x4e>());    // lane ^ 2
    if constexpr (L > 4) add(integral_constant<int, 0x141>());   // 7 - lane within 8: the other four
    if constexpr (L > 8) add(integral_constant<int, 0x140>());   // 15 - lane within 16: the other eight
    return x;
}

// A row and 512 columns for a workgroup: the shared product's parts, and the
// second product of the row's adapter, a dot
// product of `rank` for each column, in fp32.  L lanes, 8 ranks each, have a
// column, so that a load covers whole rows of `up` (with a lane to a column
// those of rank 64 took 3 times as long).  What bounds it is the bytes of `up`,
// read once for each row of its request (64 rows of 14336, rank 16: 6.8 us).
// Every workgroup looks for its row's request from the first on, 64 at a time,
// so that single tokens take longer than their number says (1024 x 1024, rank
// 16: 256 of them 13 us a call, 1000 41, 2000 101, 4096 318).
template <typename T, int L>
__global__ __launch_bounds__(256) void finish_kernel(const Args g)
{
    __shared__ float dots[512];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, c0 = (int)blockIdx.x * 512 + 128 * w;
    const int row0 = clampi(g.cu[0], 0, g.rows), row = row0 + (int)blockIdx.y;
    if (row >= clampi(g.cu[g.groups], row0, g.rows)) return;
    int id = -1;   // the adapter of the row's request
    for (int base = 0; base < g.groups; base += 64) {
        const int b = base + lane;
        const uint64_t mine = __builtin_amdgcn_ballot_w64(b < g.groups && g.cu[b] <= row && row < g.cu[b + 1]);
        if (mine != 0) {
            id = g.ids[base + __builtin_ctzll(mine)];
            break;
        }
    }
    const bool adapted = (uint32_t)id < (uint32_t)g.adapters;
    if (adapted) {
        const int chunk = lane % L, first = c0 + lane / L;
        const bool there = chunk < (int)g.rank_chunks.d;
        f32x4 h0 = {0.f, 0.f, 0.f, 0.f}, h1 = h0;
        if (there) {
            const f32x4* h = reinterpret_cast<const f32x4*>(g.low) + ((int64_t)row * g.rank_chunks.d + chunk) * 2;
            h0 = h[0];
            h1 = h[1];
        }
        // chunks that are not there are read as ones that are and cleared, so
        // that all loads are in flight together
        const char* up = g.up + (int64_t)id * g.up_mat + (there ? 16 * chunk : 0);
        const uint32_t keep = there ? 0xffffffffu : 0u;
        constexpr int N = 2 * L < 8 ? 2 * L : 8;
        for (int base = 0; base < 2 * L; base += N) {
            u32x4 a[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = first + (base + i) * (64 / L);
                a[i] = *reinterpret_cast<const u32x4*>(up + (int64_t)(c < g.cols ? c : g.cols - 1) * g.up_ld);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float x = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const attn::f32x2 u = T::unpack(a[i][j] & keep);
                    x = __builtin_fmaf(j < 2 ? h0[2 * j] : h1[2 * j - 4], u[0], x);
                    x = __builtin_fmaf(j < 2 ? h0[2 * j + 1] : h1[2 * j - 3], u[1], x);
                }
                x = sum_lanes<L>(x);
                if (chunk == 0) dots[128 * w + (base + i) * (64 / L) + lane / L] = x;
            }
        }
    }
    const int c = c0 + 2 * lane;
    if (c >= g.cols) return;
    const float* at = g.parts + (int64_t)row * g.cols + c;
    float x = 0.f, y = 0.f;
    for (uint32_t p = 0; p < g.splits.d; ++p, at += (int64_t)g.rows * g.cols) {
        const attn::f32x2 v = *reinterpret_cast<const attn::f32x2*>(at);
        x += v[0];
        y += v[1];
    }
    if (adapted) {   // a wave's own values
        grp::wave_in_order();
        x += dots[128 * w + 2 * lane];
        y += dots[128 * w + 2 * lane + 1];
    }
    *reinterpret_cast<uint32_t*>(g.d + (int64_t)row * g.d_ld + 2 * (int64_t)c) = T::pack(x, y);
}

template <typename T>
const void* finish(int64_t rank)
{
    return rank <= 8    ? (const void*)&finish_kernel<T, 1>
           : rank <= 16 ? (const void*)&finish_kernel<T, 2>
           : rank <= 32 ? (const void*)&finish_kernel<T, 4>
           : rank <= 64 ? (const void*)&finish_kernel<T, 8>
                        : (const void*)&finish_kernel<T, 16>;
}

// Eight columns of a row: the parts' sums added up in order.
__device__ __forceinline__ void join8(const float* at, int64_t step, int parts, float (&v)[8])
{
    f32x4 lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
    for (int p = 0; p < parts; ++p, at += step) {
        lo += *reinterpret_cast<const f32x4*>(at);
        hi += *reinterpret_cast<const f32x4*>(at + 4);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = lo[e];
        v[4 + e] = hi[e];
    }
}

// Writes them, rounded (or as they are, F32).
template <typename T, bool F32>
__device__ __forceinline__ void store8(char* d, const float (&v)[8])
{
    if constexpr (F32) {
        *reinterpret_cast<f32x4*>(d) = f32x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f32x4*>(d + 16) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
        *reinterpret_cast<u32x4*>(d) = u32x4{T::pack(v[0], v[1]), T::pack(v[2], v[3]), T::pack(v[4], v[5]), T::pack(v[6], v[7])};
    }
}

// Joins the parts of every tile; a workgroup has 2048 elements of one.  Bound by
// the parts' bytes, 6 TB/s (and where they are few by the launch, 4 us).
template <typename T, class C, int MODE, bool F32>
__global__ __launch_bounds__(256) void join_kernel(const Args g)
{
    constexpr uint32_t SUB = C::BM * C::BN / 2048;
    static_assert(C::BM * C::BN % 2048 == 0 && C::BN <= 2048, "whole rows for a workgroup");
    Groups<C::BM, MODE> groups;
    const uint32_t all = all_tiles<C::BM, MODE>(g, groups), t = blockIdx.x / SUB;
    if (t >= all) return;
    const Work wk = tile_at<C::BM, C::BN, MODE>(g, groups, t);
    if (!wk.found) return;
    const int x = (int)(blockIdx.x % SUB) * 2048 + (int)threadIdx.x * 8, r = x / C::BN, c = x % C::BN;
    const int rows = MODE == TN ? g.x_cols - wk.tile0 : wk.rows;
    if (r >= rows || wk.col0 + c >= g.cols) return;
    char* d = g.d + (MODE == TN ? (int64_t)wk.group * g.d_mat + (int64_t)(wk.tile0 + r) * g.d_ld : (int64_t)(wk.row0 + r) * g.d_ld) +
              (int64_t)(wk.col0 + c) * (F32 ? 4 : 2);
    float v[8];
    join8(g.parts + (int64_t)t * (C::BM * C::BN) + x, (int64_t)all * (C::BM * C::BN), (int)g.splits.d, v);
    if constexpr (MODE == LOW) {
        const float scale = g.scales != nullptr ? g.scales[g.ids[wk.group]] : 1.f;
        const bool there = wk.col0 + c < g.low_rows;
        float hi[8], lo[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            hi[e] = there ? grp::upper<T>(v[e] * scale) : 0.f;
            lo[e] = there ? v[e] * scale - hi[e] : 0.f;
        }
        store8<T, false>(d, hi);
        store8<T, false>(d + g.low_rest, lo);
    } else {
        store8<T, F32>(d, v);
    }
}

// Large tiles of NT, NN, TN, EACH and EACH2: a workgroup for each compute unit
// walks them.  Four waves of 128 x 128 outputs read a third less from LDS than
// eight of half of it, and the next tile's first loads are on the way while a tile's
// outputs are written.  The matrix cores are busy for 89 to 90 % of the time
// (by columns on both sides 71 %) and the board's power limits them: 16384 rows
// over 8 matrices of 14336 x 4096 1306 us, 1473 TFLOP/s; gradients of 8192 rows
// 686 us, 1402 TFLOP/s, and 749 us, 1284.  A tile costs some 5 us beside its
// products, for its operands and its 65536 outputs.
//
// The tiles that are left for the last round, where they are half a round or
// less, are divided along the contraction, so that all workgroups have a part;
// a second launch joins the parts.  (8192 rows over 6 matrices, 560 tiles of
// 224 steps: 2.19 rounds instead of 3.)
struct Walk {
    uint32_t total, full, rest, parts;   // tiles, those of whole rounds, the others, and the parts of each of these
    __device__ __forceinline__ void start(uint32_t tiles, uint32_t walkers, bool split)
    {
        total = tiles;
        rest = tiles % walkers;
        full = tiles - rest;
        parts = split && rest > 0 ? walkers / rest : 1;
    }
    // parts of a tile of so many steps
    __device__ __forceinline__ uint32_t of(uint32_t steps) const
    {
        const uint32_t most = steps / 4;   // of four steps or more
        return parts < most ? parts : most > 1 ? most : 1;
    }
};

// A tile's steps, and its place: tiles at the end of a side move back.
template <int MODE>
__device__ __forceinline__ uint32_t place_large(const Args& g, Work& wk)
{
    wk.col0 = (int)clamped_origin(wk.col0 / grp::kRingTile, grp::kRingTile, g.cols);
    int depth = g.depth;
    if (MODE == TN) {
        wk.tile0 = (int)clamped_origin(wk.tile0 / grp::kRingTile, grp::kRingTile, g.x_cols);
        depth = wk.rows;
    }
    uint32_t steps = (uint32_t)(depth + grp::kRingStep - 1) / grp::kRingStep;
    // the adapter's second product, both terms, is a step, or with EACH2 two
    if (each_request(MODE) && (uint32_t)g.ids[wk.group] < (uint32_t)g.adapters) steps += MODE == EACH2 ? 2 : 1;
    return steps < 2 ? 2 : steps;
}

template <typename T, int MODE, bool F32>
__global__ __launch_bounds__(256, 1) void ring_kernel(const Args g)
{
    constexpr bool XC = MODE == TN, YC = MODE == NN || MODE == TN;
    constexpr int TILE = grp::kRingTile, STEP = grp::kRingStep;
    __shared__ __attribute__((aligned(1024))) char smem[grp::kRingLds];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = w / 2 * 128, wn = w % 2 * 128;
    const uint32_t lds = attn::lds_address(smem), lb = lds + 8192u * (uint32_t)w;

    Groups<TILE, MODE> groups;
    Walk walk;
    walk.start(all_tiles<TILE, MODE>(g, groups), gridDim.x, g.parts != nullptr);
    const uint32_t items = walk.full + walk.rest * walk.parts;

    grp::RingSide<XC> a;
    grp::RingSide<YC> b;
    grp::RingStore out;
    a.start(lds, g.x_ld, wm, w, lane);
    b.start(lds + 65536, g.y_ld, wn, w, lane);
    constexpr int64_t PART_LD = 4 * TILE;
    out.start(lds, g.d_ld, F32 ? g.d_ld : PART_LD, w, lane);
    const uint32_t sta = (uint32_t)(STEP * g.x_ld), stb = (uint32_t)(STEP * g.y_ld);
    const int kr = 16 * w + lane / 32;
    uint32_t ha[2], hb[2];   // the adapter's steps: see gen_grouped_sched.py
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int r = 64 * w + lane / 8, c = (lane & 7) ^ grp::RingSide<false>::swz(8 * q + lane / 8);
        const int u = MODE == EACH ? c & 3 : c;   // EACH: `up` twice, for 32 upper terms and 32 lower ones
        ha[q] = (uint32_t)(r * 128 + 16 * c);
        hb[q] = each_request(MODE) && 8 * u < g.rank ? (uint32_t)(r * g.up_ld + 16 * u) : grp::kBeyond;
    }

    // One tile, or part of one: its operands, scalars all of them.
    struct Item {
        bool found;
        u32x4 rsa, rsb, rsd;
        uint32_t rem, wide, gstr, hk, ext;   // steps, ..., what the first step lacks, how many of the first are the adapter's
        Work wk;
    };
    // Sorted: the first round has the longest tiles, in order, and every second
    // round is dealt the other way round.
    const uint32_t own_slot = (uint32_t)xcd_slot(blockIdx.x, gridDim.x);
    bool back = false;
    auto prepare = [&](uint32_t base) {
        Item it = {};
        const uint32_t slot = base + (back ? gridDim.x - 1 - own_slot : own_slot);
        if (slot >= items) return it;
        uint32_t t = slot, part = 0;
        if (slot >= walk.full) {
            t = slot - walk.full;
            part = t / walk.rest;
            t = walk.full + t - part * walk.rest;
        }
        Work wk = tile_at<TILE, TILE, MODE>(g, groups, t);
        const uint32_t steps = place_large<MODE>(g, wk);
        // the contraction's first step is the partial one: see gen_grouped_sched.py
        int hk = MODE == TN ? 0 : (g.depth + STEP - 1) / STEP * STEP - g.depth;
        uint32_t ext = each_request(MODE) && (int)steps * STEP > g.depth + hk ? (MODE == EACH2 ? 2 : 1) : 0;
        const uint32_t parts = slot < walk.full ? 1 : walk.of(steps);
        if (part >= parts) return it;   // the last of the workgroup's anyway
        const uint32_t first = part * steps / parts;
        it.found = true;
        it.rem = grp::uniform((part + 1) * steps / parts - first);

        const char *x, *y, *d;
        int64_t x_bytes, y_bytes;
        int rows = 128;   // of the wave
        if (MODE == TN) {
            const int64_t n = wk.rows;
            x = g.x + wk.row0 * g.x_ld + 2 * (int64_t)wk.tile0;
            y = g.y + wk.row0 * g.y_ld + 2 * (int64_t)wk.col0;
            x_bytes = n == 0 ? 0 : (n - 1) * g.x_ld + 2 * TILE;
            y_bytes = n == 0 ? 0 : (n - 1) * g.y_ld + 2 * TILE;
            d = g.d + wk.group * g.d_mat + (int64_t)(wk.tile0 + wm) * g.d_ld;
        } else {
            const int64_t n = wk.rows < TILE ? wk.rows : TILE, length = g.depth + hk;
            x = g.x + wk.row0 * g.x_ld - 2 * hk;
            x_bytes = (n - 1) * g.x_ld + 2 * length;
            y = g.y + wk.group * g.y_mat + (MODE != NN ? wk.col0 * g.y_ld - 2 * hk : 2 * (int64_t)wk.col0 - hk * g.y_ld);
            y_bytes = MODE != NN ? (TILE - 1) * g.y_ld + 2 * length : (length - 1) * g.y_ld + 2 * TILE;
            rows = clampi((int)n - wm, 0, 128);
            d = g.d + (int64_t)(wk.row0 + wm) * g.d_ld;
        }
        if (first > 0) {   // a later part
            const int64_t skip = first - ext;
            const int64_t dx = skip * (XC ? STEP * g.x_ld : 2 * STEP), dy = skip * (YC ? STEP * g.y_ld : 2 * STEP);
            x += dx;
            y += dy;
            x_bytes -= dx < x_bytes ? dx : x_bytes;
            y_bytes -= dy < y_bytes ? dy : y_bytes;
            hk = 0;
            ext = 0;
        }
        int64_t d_ld = g.d_ld;
        d += (int64_t)(wk.col0 + wn) * (F32 ? 4 : 2);
        if (parts > 1) {
            d_ld = PART_LD;
            d = (const char*)(g.parts + (int64_t)(slot - walk.full) * (TILE * TILE) + wm * TILE + wn);
        }
        it.rsa = grp::ring_rsrc(x, x_bytes);
        it.rsb = grp::ring_rsrc(y, y_bytes);
        it.rsd = grp::ring_rsrc(d, rows == 0 ? 0 : (rows - 1) * d_ld + 128 * (F32 || parts > 1 ? 4 : 2));
        it.wide = F32 ? 1u + (parts > 1) : grp::uniform(parts) - 1u;   // not 0: outputs in 32 bits
        it.gstr = grp::uniform((uint32_t)(16 * d_ld));
        it.hk = grp::uniform((uint32_t)hk);
        it.ext = grp::uniform(ext);
        it.wk = wk;
        return it;
    };

    uint32_t base = 0, own = 1, par = 0;   // see gen_grouped_sched.py: first, par
    Item it = prepare(base);
    while (it.found) {
        base += gridDim.x;
        back = MODE == TN && g.sorted && !back;
        const Item then = prepare(base);
        // its step 0 by the same masks, and not an adapter's
        const bool carry = then.found && then.ext == 0 && then.hk == it.hk;
        const u32x4 none = {0, 0, 0, 0x00020000u};
        const u32x4 rsa = it.rsa, rsb = it.rsb, rsd = it.rsd, rsan = carry ? then.rsa : none, rsbn = carry ? then.rsb : none;
        uint32_t hm[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) hm[q] = 8 * ((lane & 7) ^ grp::RingSide<false>::swz(8 * q + lane / 8)) < (int)it.hk ? grp::kBeyond : 0u;
        if (F32 && it.wide > 1) out.sw = (uint32_t)((lane & 15) * PART_LD + 16 * (lane >> 4));   // a part: the last of the workgroup's items
        const uint32_t wide = it.wide, gstr = it.gstr, hk = it.hk, first = grp::uniform(own);
        uint32_t rem = grp::uniform(it.rem), koa = 0, kob = 0, kha, khb, sdo, ht;
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"   // M0 is written inside, on purpose
#define G16_GROUPED_BLOCK(LOOP, ...) \
    if constexpr (std::is_same<T, F16>::value) \
        asm volatile(LOOP("f16") : G16_GROUPED_STATE : G16_GROUPED_COMMON, __VA_ARGS__ : G16_GROUPED_CLOBBERS); \
    else \
        asm volatile(LOOP("bf16") : G16_GROUPED_STATE : G16_GROUPED_COMMON, __VA_ARGS__ : G16_GROUPED_CLOBBERS)
        if constexpr (MODE == NT || each_request(MODE)) {
            u32x4 rsa0 = rsa, rsb0 = rsb, rsa1 = rsa;
            if (each_request(MODE)) {
                const int64_t n = it.wk.rows < TILE ? it.wk.rows : TILE;
                rsa0 = grp::ring_rsrc(g.low + (int64_t)it.wk.row0 * 128, n * 128);
                rsa1 = grp::ring_rsrc(g.low + g.low_rest + (int64_t)it.wk.row0 * 128, n * 128);
                rsb0 = grp::ring_rsrc(g.up + (it.ext ? (int64_t)g.ids[it.wk.group] * g.up_mat : 0) + it.wk.col0 * g.up_ld, (TILE - 1) * g.up_ld + 2 * g.rank);
            }
            const uint32_t sb8 = grp::uniform((uint32_t)(8 * g.up_ld)), ext = it.ext;
            if constexpr (MODE == EACH2) {
                G16_GROUPED_BLOCK(G16_GROUPED_RR2, G16_GROUPED_A_ROWS, G16_GROUPED_B_ROWS, G16_GROUPED_EXT, [rsa1] "s"(rsa1));
            } else {
                G16_GROUPED_BLOCK(G16_GROUPED_RR, G16_GROUPED_A_ROWS, G16_GROUPED_B_ROWS, G16_GROUPED_EXT);
            }
        } else if constexpr (MODE == NN) {
            G16_GROUPED_BLOCK(G16_GROUPED_RC, G16_GROUPED_A_ROWS, G16_GROUPED_B_COLS, [hk] "s"(hk), [kr] "v"(kr));
        } else {
            G16_GROUPED_BLOCK(G16_GROUPED_CC, G16_GROUPED_A_COLS, G16_GROUPED_B_COLS);
        }
#pragma clang diagnostic pop
        wg_barrier();   // every wave is done reading the ring before the next tile's loads
        par = grp::uniform(carry ? (par + it.rem) & 1 : 0);
        own = grp::uniform(carry ? 0 : 1);
        it = then;
    }
    attn::landed<0>();   // loads from empty buffers
}

// Joins what ring_kernel divided; a workgroup takes 2048 elements of a tile at a time.
template <typename T, int MODE, bool F32>
__global__ __launch_bounds__(256) void ring_join_kernel(const Args g)
{
    constexpr int TILE = grp::kRingTile;
    constexpr uint32_t SUB = TILE * TILE / 2048;
    Groups<TILE, MODE> groups;
    Walk walk;
    walk.start(all_tiles<TILE, MODE>(g, groups), g.walkers, true);
    if (walk.parts < 2) return;
    for (uint32_t i = blockIdx.x; i < walk.rest * SUB; i += gridDim.x) {
        const uint32_t t = i / SUB;
        Work wk = tile_at<TILE, TILE, MODE>(g, groups, walk.full + t);
        const uint32_t parts = walk.of(place_large<MODE>(g, wk));
        const int x = (int)(i % SUB) * 2048 + (int)threadIdx.x * 8, r = x / TILE, c = x % TILE;
        if (parts < 2 || (MODE != TN && r >= wk.rows)) continue;
        char* d = g.d + (MODE == TN ? (int64_t)wk.group * g.d_mat + (int64_t)(wk.tile0 + r) * g.d_ld : (int64_t)(wk.row0 + r) * g.d_ld) +
                  (int64_t)(wk.col0 + c) * (F32 ? 4 : 2);
        float v[8];
        join8(g.parts + (int64_t)t * (TILE * TILE) + x, (int64_t)walk.rest * (TILE * TILE), (int)parts, v);
        store8<T, F32>(d, v);
    }
}

// ------------------------------------------------------------ validation
constexpr int64_t kMaxWidth = int64_t(1) << 22;       // elements of a row and its pitch: a tile of 256 rows spans less than 2^31 bytes
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1024;
constexpr int64_t kMaxGroups = int64_t(1) << 22;
constexpr int64_t kMaxTiles = int64_t(1) << 22;       // workgroups of a launch, at most 512 threads each: less than 2^32 threads

// Shapes of tiles: rows x columns x contraction, waves along these, stages,
// workgroups of a compute unit.
using Tiny = Cfg<16, 16, 512, 1, 1, 4, 4, 1>;
using Small = Cfg<32, 32, 256, 1, 1, 4, 4, 1>;
using Flat = Cfg<32, 128, 64, 1, 4, 1, 4, 2>;
using Tiny2 = Cfg<16, 16, 256, 1, 1, 4, 4, 2>;    // two for a compute unit, of projections beside shared products
using Small2 = Cfg<32, 32, 128, 1, 1, 4, 4, 2>;
using Square = Cfg<64, 64, 64, 2, 2, 1, 4, 2>;
using Oblong = Cfg<64, 128, 64, 2, 2, 1, 3, 2>;
using Middle = Cfg<128, 128, 64, 2, 2, 1, 2, 2>;
using Large = Cfg<256, 256, 64, 2, 4, 1, 2, 1>;

// What a shape takes: microseconds for 1024 of the contraction with one and
// with two workgroups on a compute unit, all of them busy, and the same where a
// row pitch is not a multiple of a cache line, so that rows of 128 bytes are
// parts of two lines (measured on MI355X, operands in L2).
struct Rate {
    double one, two, odd_one, odd_two;
};
constexpr Rate kTiny = {1.3, 1.3, 1.4, 1.4}, kSmall = {2.0, 2.0, 2.1, 2.1}, kFlat = {5.4, 7.8, 5.9, 10.3}, kSquare = {5.0, 6.4, 5.2, 8.9};
constexpr Rate kOblong = {6.8, 10.0, 7.0, 14.2}, kMiddle = {10.5, 16.8, 13.8, 19.8}, kLarge = {28., 28., 30., 30.}, kRing = {20.6, 20.6, 22.2, 22.2};
constexpr Rate kTiny2 = {1.6, 2.6, 1.8, 2.8}, kSmall2 = {2.4, 3.9, 2.5, 4.2};
bool odd_pitch(const Args& g) { return ((g.x_ld | g.y_ld) & 127) != 0; }

// A shape's kernels.
struct Form {
    int bm, bn, bk, threads, per_cu;
    Rate rate;
    const void *whole, *split, *join;
};

template <typename T, int MODE, bool F32, class C, bool PARTS>
Form form(const Rate& rate)
{
    Form f = {C::BM, C::BN, C::BK, C::THREADS, C::PER_CU, rate, (const void*)&tile_kernel<T, C, MODE, F32, ROUNDED>, nullptr, nullptr};
    if constexpr (PARTS) {
        f.split = (const void*)&tile_kernel<T, C, MODE, F32, PART>;
        f.join = (const void*)&join_kernel<T, C, MODE, F32>;
    }
    return f;
}

constexpr int kMaxForms = 7;
template <typename T, int MODE, bool F32>
struct Forms {
    Form f[kMaxForms];
    int n = 0;
    Forms()
    {
        if constexpr (MODE != TN && !each_request(MODE)) {
            f[n++] = form<T, MODE, F32, Tiny, false>(kTiny);
            f[n++] = form<T, MODE, F32, Small, false>(kSmall);
        }
        if constexpr (MODE == NT || MODE == NN) f[n++] = form<T, MODE, F32, Flat, false>(kFlat);
        if constexpr (!each_request(MODE)) f[n++] = form<T, MODE, F32, Square, true>(kSquare);
        if constexpr (MODE != TN && !each_request(MODE)) f[n++] = form<T, MODE, F32, Oblong, true>(kOblong);
        if constexpr (MODE != LOW && !each_request(MODE)) f[n++] = form<T, MODE, F32, Middle, true>(kMiddle);
        if constexpr (MODE == ADAPT) f[n++] = form<T, MODE, F32, Large, false>(kLarge);
        if constexpr (MODE == NT || MODE == NN || MODE == TN || each_request(MODE))
            f[n++] = Form{grp::kRingTile, grp::kRingTile, grp::kRingStep, 256, 0, kRing, (const void*)&ring_kernel<T, MODE, F32>, nullptr,
                          (const void*)&ring_join_kernel<T, MODE, F32>};
    }
};

// What the large tiles' kernel takes: see grouped_ring.hpp.
constexpr int64_t kRingPitch = int64_t(1) << 21;
bool ring_takes(int mode, const Args& g)
{
    const int64_t pitch = 2 * kRingPitch;
    if (g.cols < grp::kRingTile || g.x_ld >= pitch || g.y_ld >= pitch || g.d_ld >= 2 * pitch) return false;
    if (mode == TN) {
        const int64_t reach = (int64_t)g.rows + 3 * grp::kRingStep;
        return g.x_cols >= grp::kRingTile && reach * g.x_ld < (int64_t(1) << 32) && reach * g.y_ld < (int64_t(1) << 32);
    }
    return g.depth > grp::kRingStep && (mode != NN || ((int64_t)g.depth + 2 * grp::kRingStep) * g.y_ld < (int64_t(1) << 31));
}

struct Plan {
    const Form* form;
    int64_t wgs, splits, part_bytes;
    bool walks;
    double us;
};

constexpr int64_t kMaxSplits = 16;

// TN: whether the longest groups come first.  Large tiles' workgroups find the
// order once, the others for each tile, and with many rounds the order makes no
// difference.  (7901 rows over 8 matrices of 1024 x 4864, large tiles: 101 us in
// the groups' own order, 75 so; 9630 rows, 8 of 2048 x 1536, tiles of 128 x 128:
// 85 and 76; but 1500 rows, 64 of 2048 x 1024, 16 rounds of them: 102 and 136.
// Between 8 groups and 64 of the small tiles nothing was measured.)
bool sorts(bool walks, int64_t groups, int64_t tiles, int cus)
{
    return groups > 1 && groups <= (walks ? 64 : 16) && tiles <= (int64_t)(walks ? 8 : 16) * cus;
}

// The shape and the parts of the contraction that a model of the time finds
// best: rounds of the compute units, each with what starting a workgroup costs
// and the contraction's share, not less than the operands take from memory;
// and for parts their bytes and the second launch.  The number of tiles is the
// device's to know where there are several groups: half a tile for each group
// is taken as lost.
template <int MODE, bool F32>
Plan plan(const Form* forms, int n, const Args& g, int cus, int* status)
{
    const int64_t used = MODE == ADAPT ? 1 : g.groups < g.rows ? g.groups : g.rows;   // groups with rows, at most
    const double depth = MODE == TN ? (g.groups > 0 ? (double)g.rows / g.groups : 0.) : g.depth;
    // matrices, rows read and rows written, at 5.5 TB/s
    const double mats = MODE == TN ? (double)g.groups * g.x_cols * g.cols : (each_request(MODE) ? 1. : used) * g.cols * depth;
    const double rows = MODE == TN ? (double)g.rows * (g.x_cols + g.cols) : (double)g.rows * (depth + g.cols);
    const double memory = (mats * (MODE == TN && F32 ? 2 : 1) + rows) * 2 / 5.5e6;
    // TN: matrices are written when a workgroup ends, half of it beside others'
    // products; and a single round of workgroups takes as long as its longest
    // group, taken as 1.6 times the mean (of 8 groups whose likelihoods are even
    // from 0.2 to 1.8 it is 1.3 to 2.1 times that, mostly 1.6)
    const double written = MODE == TN ? mats * (F32 ? 4 : 2) / 5.5e6 / 2 : 0., longest = MODE == TN && g.groups > 1 ? 1.6 : 1.;
    const bool odd = odd_pitch(g);
    Plan best = {nullptr, 0, 1, 0, false, 1e300};
    for (int i = 0; i < n; ++i) {
        const Form& f = forms[i];
        const bool ring = f.per_cu == 0;
        const double one = odd ? f.rate.odd_one : f.rate.one, two = odd ? f.rate.odd_two : f.rate.two;
        if (ring && !ring_takes(MODE, g)) continue;
        const int64_t ct = ceil_div(g.cols, f.bn);
        int64_t most;    // tiles, at most
        double tiles;    // and as expected
        if (MODE == TN) {
            const int64_t t = ct * ceil_div(g.x_cols, f.bm);
            most = g.groups * (ring || t < 8 * kNumXcd ? t : ceil_div(t, kNumXcd) * kNumXcd);
            tiles = (double)g.groups * t;
        } else {
            most = (g.rows + used * (f.bm - 1)) / f.bm * ct;
            const double r = used == 1 ? ceil_div(g.rows, f.bm) : (double)g.rows / f.bm + 0.5 * used + 0.29 * std::sqrt((double)used);
            tiles = (r < used ? used : r) * ct;
        }
        if (most > kMaxTiles) continue;
        if (ring) {
            const double d = (depth < 128 ? 128 : depth) / 1024 * one + 6.0;
            const int64_t count = (int64_t)(tiles + 0.5), rest = count % cus;
            // whole tiles: in rounds; sorted ones of unequal length pack better
            double us = (count / cus) * d + (rest == 0 ? 0. : count < cus ? longest * d : d);
            if (MODE == TN && sorts(true, g.groups, count, cus)) {
                us = d * ((double)count / cus + 0.25);
                if (us < longest * d) us = longest * d;
            }
            // or the last round's in parts
            bool split = rest > 0 && rest <= cus / 2 && depth >= 512 && count < 16 * cus;
            if (split) {
                const double parts = cus / rest, in_parts = (count / cus) * d + d / parts + 8 + (double)rest * parts * f.bm * f.bn * 8 / 8e6;
                split = in_parts < us;
                if (split) us = in_parts;
            }
            us += written;
            if (us < memory + 3) us = memory + 3;
            if (us < best.us) {
                // where the device alone knows the tiles, parts are made
                // possible for it if its last round may be a small one
                const bool known = MODE == TN || used == 1, may = 20 * rest <= 11 * cus || 10 * rest >= 9 * cus;
                const bool parts = known ? split : may && depth >= 512 && count < 16 * cus;
                best = Plan{&f, parts || most > cus ? cus : most, 1, parts ? (int64_t)cus * f.bm * f.bn * 4 : 0, true, us};
            }
            continue;
        }
        const double slots = (double)cus * f.per_cu;
        double extra = 0;
        if (MODE == ADAPT && g.adapters > 0) {   // a tile's requests, twice `rank` of the contraction each
            const double requests = g.groups < g.rows ? g.groups : g.rows, mean = g.rows / requests, mine = f.bm / mean + 1;
            extra = (16. * g.rank_chunks.d * (mine < requests ? mine : requests) + 256) / 1024;
        }
        for (int64_t s = 1; s <= (f.split == nullptr ? 1 : kMaxSplits); s += s < 4 ? 1 : s / 2) {
            const int64_t steps = ceil_div((int64_t)depth, f.bk * s);
            if (s > 1 && (steps < 4 || most * s > kMaxTiles / 8)) break;   // a tile of the join has up to 8 workgroups
            const double d = (double)(steps * f.bk) / 1024 + extra / s, wgs = tiles * s;
            const double full = (double)(int64_t)(wgs / slots), rest = wgs - full * slots;
            double us = 1.5 + full * (2.3 + two * d) + written;
            if (rest > 0) us += 2.3 + (rest > cus ? two : one) * d * (full == 0 ? longest : 1.);
            if (us < memory + 3) us = memory + 3;
            if (s > 1) us += one * extra * (1 - 1. / s);   // they all go with the last part
            if (s > 1) us += 6 + wgs * f.bm * f.bn * 8 / 8e6;
            if (us < best.us) best = Plan{&f, most * s, s, s > 1 ? most * s * f.bm * f.bn * 4 : 0, false, us};
        }
    }
    *status = best.form == nullptr ? GEMM_F16_NT_UNSUPPORTED : GEMM_F16_NT_OK;
    return best;
}

template <int MODE, bool F32 = false>
Plan plan_for(int dtype, const Args& g, int cus, int* status)
{
    static const Forms<F16, MODE, F32> f16;
    static const Forms<BF16, MODE, F32> bf16;
    return dtype == GROUPED_F16 ? plan<MODE, F32>(f16.f, f16.n, g, cus, status) : plan<MODE, F32>(bf16.f, bf16.n, g, cus, status);
}

template <int MODE>
int run(const Plan& p, const Args& args, void* parts, int cus, hipStream_t s)
{
    Args g = args;
    const Form& f = *p.form;
    const int64_t ct = ceil_div(g.cols, f.bn);
    g.col_tiles = attn::div_by(ct);
    g.splits = attn::div_by(p.splits);
    g.parts = p.part_bytes > 0 ? (float*)parts : nullptr;
    g.walkers = (uint32_t)p.wgs;
    const int64_t used = MODE == ADAPT ? 1 : g.groups < g.rows ? g.groups : g.rows;   // groups with rows
    g.row_tiles = (uint32_t)((g.rows + used * (f.bm - 1)) / f.bm);
    if (MODE == TN) {
        const int64_t t = ct * ceil_div(g.x_cols, f.bm);
        g.group_tiles = (uint32_t)t;
        g.sorted = sorts(p.walks, g.groups, g.groups * t, cus);
        g.per_group = attn::div_by(p.walks || t < 8 * kNumXcd ? t : ceil_div(t, kNumXcd) * kNumXcd);
    }
    int st = launch(p.splits > 1 ? f.split : f.whole, p.wgs, f.threads, &g, s);
    if (st != GEMM_F16_NT_OK || g.parts == nullptr) return st;
    const int64_t pieces = p.walks ? 4 * cus : p.wgs / p.splits * (f.bm * f.bn / 2048);
    return launch(f.join, pieces, 256, &g, s);
}

bool widths_ok(int64_t n, int64_t k) { return n % 8 == 0 && k % 8 == 0 && n < kMaxWidth && k < kMaxWidth; }

enum Written { A_, B_, D_ };

struct Span {
    const void* p;
    int64_t bytes;
};

// GEMM_F16_NT_OK, 1 where a valid call has nothing to write, or an error.
int check_grouped(const grouped_desc* d, Written out, Span work = {nullptr, 0})
{
    if (d == nullptr) return GEMM_F16_NT_INVALID_ARG;
    if (d->dtype != GROUPED_F16 && d->dtype != GROUPED_BF16) return GEMM_F16_NT_INVALID_ARG;
    if (d->b_fp32 != 0 && d->b_fp32 != 1) return GEMM_F16_NT_INVALID_ARG;
    if (d->groups < 0 || d->rows < 0 || d->N < 0 || d->K < 0) return GEMM_F16_NT_INVALID_ARG;
    if (d->lda < d->K || d->ldb < d->K || d->ldd < d->N) return GEMM_F16_NT_INVALID_ARG;
    const int64_t ea = d->K == 0 ? 0 : extent(d->K, {{d->rows, d->lda}});
    const int64_t ed = d->N == 0 ? 0 : extent(d->N, {{d->rows, d->ldd}});
    int64_t eb = d->K == 0 ? 0 : extent(d->K, {{d->N, d->ldb}, {d->groups, d->stride_b}});
    if (ea < 0 || eb < 0 || ed < 0) return GEMM_F16_NT_INVALID_ARG;
    if (d->b_fp32) eb *= 2;
    const bool none = out == B_ ? eb == 0 : d->groups == 0 || (out == A_ ? ea : ed) == 0;   // nothing to write
    if (!none) {
        if (d->cu == nullptr) return GEMM_F16_NT_INVALID_ARG;
        if ((ea > 0 && d->A == nullptr) || (eb > 0 && d->B == nullptr) || (ed > 0 && d->D == nullptr)) return GEMM_F16_NT_INVALID_ARG;
        if (out == B_ && d->groups > 1 && d->stride_b < (d->N - 1) * d->ldb + d->K) return GEMM_F16_NT_INVALID_ARG;
        const Span all[] = {{d->A, ea}, {d->B, eb}, {d->D, ed}, {d->cu, d->groups < kMaxGroups ? 4 * (d->groups + 1) : 0}};
        for (int i = 0; i < 4; ++i)
            if ((i != (int)out && overlaps(all[out].p, all[out].bytes, all[i].p, all[i].bytes)) || overlaps(work.p, work.bytes, all[i].p, all[i].bytes))
                return GEMM_F16_NT_INVALID_ARG;
    }
    if (out != B_ && d->b_fp32) return GEMM_F16_NT_UNSUPPORTED;
    if (!widths_ok(d->N, d->K) || d->lda >= kMaxWidth || d->ldb >= kMaxWidth || d->ldd >= kMaxWidth) return GEMM_F16_NT_UNSUPPORTED;
    if (d->rows > kMaxRows || d->groups >= kMaxGroups) return GEMM_F16_NT_UNSUPPORTED;
    if (!aligned16(d->A, {d->lda}) || !aligned16(d->D, {d->ldd}) || !aligned16(d->B, {d->ldb, d->stride_b})) return GEMM_F16_NT_UNSUPPORTED;
    return ((uintptr_t)d->cu & 3) != 0 ? GEMM_F16_NT_UNSUPPORTED : none ? 1 : GEMM_F16_NT_OK;
}

int check_adapters(const adapter_desc* d, Span work = {nullptr, 0})
{
    if (d == nullptr) return GEMM_F16_NT_INVALID_ARG;
    if (d->dtype != GROUPED_F16 && d->dtype != GROUPED_BF16) return GEMM_F16_NT_INVALID_ARG;
    if (d->rows < 0 || d->N < 0 || d->K < 0 || d->rank < 0 || d->adapters < 0 || d->requests < 0) return GEMM_F16_NT_INVALID_ARG;
    if (d->lda < d->K || d->ldb < d->K || d->ldd < d->N || d->ld_down < d->K || d->ld_up < d->rank) return GEMM_F16_NT_INVALID_ARG;
    const int64_t ea = d->K == 0 ? 0 : extent(d->K, {{d->rows, d->lda}}), eb = d->K == 0 ? 0 : extent(d->K, {{d->N, d->ldb}});
    const int64_t ed = d->N == 0 ? 0 : extent(d->N, {{d->rows, d->ldd}});
    const int64_t edn = d->K == 0 ? 0 : extent(d->K, {{d->rank, d->ld_down}, {d->adapters, d->stride_down}});
    const int64_t eup = d->rank == 0 ? 0 : extent(d->rank, {{d->N, d->ld_up}, {d->adapters, d->stride_up}});
    if (ea < 0 || eb < 0 || ed < 0 || edn < 0 || eup < 0) return GEMM_F16_NT_INVALID_ARG;
    const bool none = ed == 0 || d->requests == 0;
    if (!none) {
        if (d->cu == nullptr || d->ids == nullptr || d->D == nullptr) return GEMM_F16_NT_INVALID_ARG;
        if ((ea > 0 && d->A == nullptr) || (eb > 0 && d->B == nullptr) || (edn > 0 && d->down == nullptr) || (eup > 0 && d->up == nullptr))
            return GEMM_F16_NT_INVALID_ARG;
        const int64_t few = d->requests < kMaxGroups ? d->requests : 0;
        const Span written[] = {{d->D, ed}, work};
        const Span read[] = {{d->A, ea}, {d->B, eb}, {d->down, edn}, {d->up, eup}, {d->cu, 4 * (few + 1)}, {d->ids, 4 * few},
                             {d->scales, d->scales != nullptr && d->adapters < kMaxGroups ? 4 * d->adapters : 0}};
        for (const Span& w : written)
            for (const Span& r : read)
                if (overlaps(w.p, w.bytes, r.p, r.bytes)) return GEMM_F16_NT_INVALID_ARG;
        if (overlaps(d->D, ed, work.p, work.bytes)) return GEMM_F16_NT_INVALID_ARG;
    }
    if (!widths_ok(d->N, d->K) || d->rank % 8 != 0 || d->rank > 128) return GEMM_F16_NT_UNSUPPORTED;
    if (d->lda >= kMaxWidth || d->ldb >= kMaxWidth || d->ldd >= kMaxWidth || d->ld_down >= kMaxWidth || d->ld_up >= kMaxWidth) return GEMM_F16_NT_UNSUPPORTED;
    if (d->rows > kMaxRows || d->requests >= kMaxGroups || d->adapters >= kMaxGroups) return GEMM_F16_NT_UNSUPPORTED;
    if (!aligned16(d->A, {d->lda}) || !aligned16(d->B, {d->ldb}) || !aligned16(d->D, {d->ldd}) ||
        !aligned16(d->down, {d->ld_down, d->stride_down}) || !aligned16(d->up, {d->ld_up, d->stride_up}))
        return GEMM_F16_NT_UNSUPPORTED;
    if (((uintptr_t)d->cu | (uintptr_t)d->ids | (uintptr_t)d->scales) & 3) return GEMM_F16_NT_UNSUPPORTED;
    return none ? 1 : GEMM_F16_NT_OK;
}

// Arguments of a call: written is D for NT, A for NN, B for TN.
Args grouped_args(const grouped_desc* d, int mode)
{
    Args g = {};
    g.cu = d->cu;
    g.groups = (int)d->groups;
    g.rows = (int)d->rows;
    g.x = (const char*)(mode == NT ? d->A : d->D);
    g.x_ld = 2 * (mode == NT ? d->lda : d->ldd);
    g.y = (const char*)(mode == TN ? d->A : d->B);
    g.y_ld = 2 * (mode == TN ? d->lda : d->ldb);
    g.y_mat = 2 * d->stride_b;
    const int64_t size = d->b_fp32 ? 4 : 2;
    g.d = (char*)(mode == NT ? d->D : mode == NN ? d->A : d->B);
    g.d_ld = mode == NT ? 2 * d->ldd : mode == NN ? 2 * d->lda : size * d->ldb;
    g.d_mat = size * d->stride_b;
    g.cols = (int)(mode == NT ? d->N : d->K);
    g.x_cols = (int)d->N;
    g.depth = (int)(mode == NT ? d->K : d->N);
    return g;
}

int plan_grouped(const grouped_desc* d, int mode, const Args& g, int cus, Plan* p)
{
    int st = GEMM_F16_NT_OK;
    *p = mode == NT ? plan_for<NT>(d->dtype, g, cus, &st) : mode == NN ? plan_for<NN>(d->dtype, g, cus, &st)
         : d->b_fp32 ? plan_for<TN, true>(d->dtype, g, cus, &st) : plan_for<TN>(d->dtype, g, cus, &st);
    return st;
}

template <int MODE>
int64_t grouped_bytes(const grouped_desc* d, Written out)
{
    int st = check_grouped(d, out), cus = 0;
    if (st != GEMM_F16_NT_OK) return st > 0 ? 0 : st;
    Plan p;
    if ((st = device_cus(&cus)) != GEMM_F16_NT_OK || (st = plan_grouped(d, MODE, grouped_args(d, MODE), cus, &p)) != GEMM_F16_NT_OK) return st;
    return p.part_bytes;
}

template <int MODE>
int grouped_run(const grouped_desc* d, Written out, void* workspace, int64_t workspace_bytes, void* stream)
{
    int st = check_grouped(d, out), cus = 0;
    if (st != GEMM_F16_NT_OK) return st > 0 ? GEMM_F16_NT_OK : st;
    const Args g = grouped_args(d, MODE);
    Plan p;
    if ((st = device_cus(&cus)) != GEMM_F16_NT_OK || (st = plan_grouped(d, MODE, g, cus, &p)) != GEMM_F16_NT_OK) return st;
    if ((st = check_workspace(workspace, workspace_bytes, p.part_bytes)) != GEMM_F16_NT_OK) return st;
    if ((st = check_grouped(d, out, {workspace, p.part_bytes})) != GEMM_F16_NT_OK) return st;
    return run<MODE>(p, g, workspace, cus, (hipStream_t)stream);
}

// The launches of adapter_nt: the projections onto the rank, to the workspace,
// and the rest, or both in one.  Parts of both lie behind the projections.
struct AdapterCall {
    Args low, rest;
    Plan low_plan, plan;
    bool adapted, each;
    const void* single;   // all in one launch
    const void* pair;     // projections and shared product in one
    const void* end;      // and what puts them together
    int bm, bn;           // the shared product's tile there
    bool dots;            // finish_kernel
    int64_t low_wgs;
    int cus;
    int64_t low_bytes, bytes;   // of the projections, and of all of the workspace
};

// The pairs of launches, by the shared product's tiles and what ends the call.
struct PairForm {
    int bm, bn, bk;
    Rate rate;
    const void *plane, *held, *first;
};

template <typename T>
struct PairForms {
    PairForm f[4] = {{16, 16, 256, kTiny2, (const void*)&pair_kernel<T, Tiny2, Tiny2, PLANE>, nullptr, nullptr},
                     {32, 32, 128, kSmall2, (const void*)&pair_kernel<T, Tiny2, Small2, PLANE>, nullptr, nullptr},
                     {64, 64, 64, kSquare, (const void*)&pair_kernel<T, Tiny2, Square, PLANE>, nullptr, nullptr},
                     {64, 128, 64, kOblong, (const void*)&pair_kernel<T, Tiny2, Oblong, PLANE>, (const void*)&pair_kernel<T, Tiny2, Oblong, HELD>,
                      (const void*)&tile_kernel<T, Oblong, ADAPT, false, FIRST>}};
};

// A pair of launches, where the model finds it faster than the projections by
// themselves and then the rest: for few rows, for requests of few rows, whose
// parts of the contraction would fill their tiles with zeros, and with a long
// contraction and few tiles, where the projections take as long as the rest.
// (bf16, 4096 x 4096, 256 requests of one row, rank 64: 65 us, and 117
// with the projections first; rank 16, one request of 195 rows, 2304 x 5376: 24 and,
// with the projections first, 32; seven of 1226, 3032 x 384: 20 and 17.)
void plan_pair(const adapter_desc* d, AdapterCall* c, int64_t* parts, double* two)
{
    static const PairForms<F16> f16;
    static const PairForms<BF16> bf16;
    const PairForm* forms = d->dtype == GROUPED_F16 ? f16.f : bf16.f;
    const int64_t used = d->requests < d->rows ? d->requests : d->rows;
    const bool odd = odd_pitch(c->rest);
    const double slots = 2. * c->cus, depth = (double)d->K / 1024, kinds = (double)(used < d->adapters ? used : d->adapters) * d->rank * 2;
    const double memory = 1.5 + ((double)(d->N + d->rows) * d->K * 2 + kinds * d->K) / 5.6e6;
    const int64_t low_wgs = (d->rows + used * 15) / 16 * ceil_div(d->rank, 16);   // at most
    const double low_rows = (double)d->rows / 16 + 0.5 * used, low_mean = (low_rows > used ? low_rows : (double)used) * ceil_div(d->rank, 16);
    const double low_one = odd ? kTiny2.odd_one : kTiny2.one, low_two = odd ? kTiny2.odd_two : kTiny2.two;
    // finish_kernel reads `up` for each row, more often from L2 than from memory,
    // and has 8 workgroups on a compute unit, each a chain of some 5 us.  It was
    // measured up to 4096 rows and is not taken beyond (1024 x 1024, rank 16, one
    // row a request: 318 us, and 361 for 4104 in tiles).
    double dots = (double)d->rows * d->N * d->rank * 2 / 1e7;
    if (dots < kinds * d->N / 5e6) dots = kinds * d->N / 5e6;
    if (dots < (double)d->rows * ceil_div(d->N, 512) * 2.5e-3) dots = (double)d->rows * ceil_div(d->N, 512) * 2.5e-3;
    dots = d->rows > 4096 ? 1e300 : dots + 4;
    double best = 1e300;
    const PairForm* form = nullptr;
    int64_t splits = 1;
    for (int i = d->rows <= 16 ? 0 : d->rows <= 32 ? 1 : 2; i < 4; ++i) {
        const PairForm& f = forms[i];
        const double one = odd ? f.rate.odd_one : f.rate.one, two = odd ? f.rate.odd_two : f.rate.two;
        const int64_t tiles = ceil_div(d->rows, f.bm) * ceil_div(d->N, f.bn);
        for (int64_t s = 1; s <= kMaxSplits; s += s < 4 ? 1 : s / 2) {
            const int64_t steps = ceil_div(d->K, f.bk * s);
            if (low_wgs + tiles * s > kMaxTiles || (s > 1 && steps < 4)) break;
            // the launch's rounds, the projections counted as so many of the others
            const double k = (double)(steps * f.bk) / 1024, each = 2.3 + two * k, wgs = (double)(tiles * s) + low_mean * (2.3 + low_two * depth) / each;
            const double full = (double)(int64_t)(wgs / slots), rest = wgs - full * slots;
            const bool alone = full == 0 ? (double)(tiles * s) + low_mean <= c->cus : rest <= c->cus;   // on a compute unit
            double us = full * each + (rest == 0 ? 0. : alone ? 2.3 + one * k : each);
            const double low = 2.3 + (low_mean > c->cus ? low_two : low_one) * depth;
            if (us < low) us = low;
            us += 1.5;
            if (us < memory) us = memory;
            const double by_dots = us + dots + (double)d->rows * d->N * s * 8 / 8e6;
            if (by_dots < best) {
                best = by_dots;
                form = &f;
                splits = s;
                c->dots = true;
            }
            if (f.held == nullptr) continue;
            // tiles with their requests' parts of the contraction as in plan()
            const double mine = (double)f.bm / d->rows * used + 1, length = (2. * d->rank * (mine < used ? mine : used) + 256) / 1024;
            const int64_t rounds = (int64_t)(tiles / slots);
            const double more = tiles - rounds * slots;
            us += 3.5 + rounds * (2.3 + two * length) + (more > c->cus ? 2.3 + two * length : more > 0 ? 2.3 + one * length : 0.) +
                  (double)tiles * s * f.bm * f.bn * 8 / 8e6;
            if (us < best) {
                best = us;
                form = &f;
                splits = s;
                c->dots = false;
            }
        }
    }
    if (form == nullptr || best >= *two) return;
    *two = best;
    const int64_t rt = ceil_div(d->rows, form->bm), ct = ceil_div(d->N, form->bn);
    c->pair = c->dots ? form->plane : form->held;
    c->bm = form->bm;
    c->bn = form->bn;
    c->end = !c->dots ? form->first : d->dtype == GROUPED_F16 ? finish<F16>(d->rank) : finish<BF16>(d->rank);
    c->each = false;
    c->low.d_ld = (c->dots ? 4 : 2) * d->rank;   // in fp32, or in two terms
    c->low.low_rest = c->rest.low_rest = 2 * d->rows * d->rank;
    c->low.cols = c->low.low_rows = d->rank;
    c->low.col_tiles = attn::div_by(ceil_div(d->rank, 16));
    c->low.row_tiles = (uint32_t)((d->rows + used * 15) / 16);
    c->low_wgs = low_wgs;
    c->rest.row_tiles = (uint32_t)rt;
    c->rest.col_tiles = attn::div_by(ct);
    c->rest.splits = attn::div_by(splits);
    c->plan.splits = splits;
    c->plan.wgs = rt * ct * splits;
    c->low_bytes = ceil_div(4 * d->rows * d->rank, 256) * 256;
    *parts = c->dots ? d->rows * d->N * splits * 4 : rt * ct * splits * form->bm * form->bn * 4;
}

int run_pair(const AdapterCall& c, void* workspace, hipStream_t s)
{
    PairArgs p;
    p.low = c.low;
    p.low.d = (char*)workspace;
    p.base = c.rest;
    p.base.adapters = 0;   // none in this launch
    p.base.parts = (float*)((char*)workspace + c.low_bytes);
    p.low_wgs = (uint32_t)c.low_wgs;
    int st = launch(c.pair, c.low_wgs + c.plan.wgs, 256, &p, s);
    if (st != GEMM_F16_NT_OK) return st;
    Args g = p.base;
    g.adapters = c.rest.adapters;
    g.low = (const char*)workspace;
    if (!c.dots) return launch(c.end, c.plan.wgs / c.plan.splits, 256, &g, s);
    void* a[] = {&g};
    const dim3 grid((unsigned)ceil_div(g.cols, 512), (unsigned)g.rows);
    return hipLaunchKernel(c.end, grid, dim3(256), a, 0, s) == hipSuccess ? GEMM_F16_NT_OK : GEMM_F16_NT_LAUNCH;
}

int plan_adapters(const adapter_desc* d, int cus, AdapterCall* c)
{
    int st = GEMM_F16_NT_OK;
    c->cus = cus;
    c->adapted = d->adapters > 0 && d->rank > 0;
    c->single = c->pair = c->end = nullptr;
    c->dots = false;
    Args g = {};
    g.x = (const char*)d->A;
    g.cu = d->cu;
    g.x_ld = 2 * d->lda;
    g.groups = (int)d->requests;
    g.rows = (int)d->rows;
    g.depth = (int)d->K;
    g.ids = d->ids;
    g.scales = d->scales;
    g.adapters = c->adapted ? (int)d->adapters : 0;
    g.rank_chunks = attn::div_by(c->adapted ? d->rank / 8 : 1);
    g.low_rest = 2 * d->rows * d->rank;
    g.term_chunks = attn::div_by(2 * g.rank_chunks.d);
    c->low_bytes = 0;
    int64_t parts = 0;
    if (c->adapted) {
        c->low = g;
        c->low.y = (const char*)d->down;
        c->low.y_ld = 2 * d->ld_down;
        c->low.y_mat = 2 * d->stride_down;
        c->low.d_ld = 2 * d->rank;
        c->low.cols = c->low.low_rows = d->rank;
        c->low_plan = plan_for<LOW>(d->dtype, c->low, c->cus, &st);
        if (st != GEMM_F16_NT_OK) return st;
        c->low_bytes = ceil_div(4 * d->rows * d->rank, 256) * 256;
        parts = c->low_plan.part_bytes;
    }
    g.down = (const char*)d->down;
    g.down_ld = 2 * d->ld_down;
    g.down_mat = 2 * d->stride_down;
    g.y = (const char*)d->B;
    g.y_ld = 2 * d->ldb;
    g.d = (char*)d->D;
    g.d_ld = 2 * d->ldd;
    g.cols = (int)d->N;
    g.up = (const char*)d->up;
    g.up_ld = 2 * d->ld_up;
    g.up_mat = 2 * d->stride_up;
    c->rest = g;
    c->each = false;
    c->plan = plan_for<ADAPT>(d->dtype, g, c->cus, &st);
    if (c->adapted && d->rank <= 64 && g.up_ld < 2 * kRingPitch) {   // large tiles, of one request each
        int each_st = GEMM_F16_NT_OK;
        const Plan each = d->rank <= 32 ? plan_for<EACH>(d->dtype, g, c->cus, &each_st) : plan_for<EACH2>(d->dtype, g, c->cus, &each_st);
        if (each_st == GEMM_F16_NT_OK && (st != GEMM_F16_NT_OK || each.us < c->plan.us)) {
            st = GEMM_F16_NT_OK;
            c->each = true;
            c->plan = each;
            c->rest.rank = d->rank;
            // rows of 64 elements: 32 upper and 32 lower terms, or 64 of one kind; zeros behind the rank
            const bool both = d->rank <= 32;
            c->low.cols = both ? 32 : 64;
            c->low.d_ld = 128;
            c->low.low_rest = c->rest.low_rest = both ? 64 : 128 * d->rows;
            c->low_bytes = (both ? 128 : 256) * d->rows;
            c->low_plan = plan_for<LOW>(d->dtype, c->low, c->cus, &st);
            parts = c->low_plan.part_bytes;
        }
    }
    if (st != GEMM_F16_NT_OK) return st;
    double two = c->plan.us + (c->adapted ? c->low_plan.us : 0.) + 1;   // what two launches take
    if (c->adapted) plan_pair(d, c, &parts, &two);
    const int64_t blocks = d->requests * ceil_div(d->rank, 16);
    if (c->adapted && d->rows <= 16 && blocks <= 3) {
        // rounds of the compute units, each with what starting a workgroup
        // costs and its tile's share of the contraction.  Measured on MI355X,
        // in one launch and in a pair: one request of rank 16, 4096 x 4096 10.3
        // and 13.0 us, 1024 x 1024 5.3 and 7.6, 4096 x 14336 23 and 29; three
        // 16.0 and 13.8, 8.0 and 7.5 (where the host's second launch counts),
        // 30 and 30.
        const double us = 1.5 + (double)ceil_div(ceil_div(d->N, 16), c->cus) * (2.0 + (blocks == 1 ? 1.65 : 3.0) * (double)d->K / 1024);
        if (us < two) {
            if (d->dtype == GROUPED_F16)
                c->single = blocks == 1 ? (const void*)&single_kernel<F16, 1> : (const void*)&single_kernel<F16, 3>;
            else
                c->single = blocks == 1 ? (const void*)&single_kernel<BF16, 1> : (const void*)&single_kernel<BF16, 3>;
            c->bytes = 0;
            return GEMM_F16_NT_OK;
        }
    }
    if (c->pair == nullptr && c->plan.part_bytes > parts) parts = c->plan.part_bytes;
    c->bytes = c->low_bytes + parts;
    return GEMM_F16_NT_OK;
}

}  // namespace

extern "C" {

int grouped_nt_check(const grouped_desc* d) { const int st = check_grouped(d, D_); return st > 0 ? GEMM_F16_NT_OK : st; }
int grouped_nn_check(const grouped_desc* d) { const int st = check_grouped(d, A_); return st > 0 ? GEMM_F16_NT_OK : st; }
int grouped_tn_check(const grouped_desc* d) { const int st = check_grouped(d, B_); return st > 0 ? GEMM_F16_NT_OK : st; }
int adapter_nt_check(const adapter_desc* d) { const int st = check_adapters(d); return st > 0 ? GEMM_F16_NT_OK : st; }

int64_t grouped_nt_workspace(const grouped_desc* d) { return grouped_bytes<NT>(d, D_); }
int64_t grouped_nn_workspace(const grouped_desc* d) { return grouped_bytes<NN>(d, A_); }
int64_t grouped_tn_workspace(const grouped_desc* d) { return grouped_bytes<TN>(d, B_); }

int grouped_nt(const grouped_desc* d, void* workspace, int64_t workspace_bytes, void* stream)
{
    return grouped_run<NT>(d, D_, workspace, workspace_bytes, stream);
}
int grouped_nn(const grouped_desc* d, void* workspace, int64_t workspace_bytes, void* stream)
{
    return grouped_run<NN>(d, A_, workspace, workspace_bytes, stream);
}
int grouped_tn(const grouped_desc* d, void* workspace, int64_t workspace_bytes, void* stream)
{
    return grouped_run<TN>(d, B_, workspace, workspace_bytes, stream);
}

int gemm_f16_nt_grouped_plan(const grouped_desc* d, int product, int cus, int tile[2], int64_t* parts)
{
    if (product < GROUPED_NT || product > GROUPED_TN || cus < 1 || tile == nullptr || parts == nullptr) return GEMM_F16_NT_INVALID_ARG;
    const int mode = product == GROUPED_NT ? NT : product == GROUPED_NN ? NN : TN;
    int st = check_grouped(d, mode == NT ? D_ : mode == NN ? A_ : B_);
    if (st < 0) return st;
    tile[0] = tile[1] = 0;
    *parts = 0;
    if (st > 0) return GEMM_F16_NT_OK;
    Plan p;
    if ((st = plan_grouped(d, mode, grouped_args(d, mode), cus, &p)) != GEMM_F16_NT_OK) return st;
    tile[0] = p.form->bm;
    tile[1] = p.form->bn;
    *parts = p.walks ? (p.part_bytes > 0 ? 0 : 1) : p.splits;
    return GEMM_F16_NT_OK;
}

int gemm_f16_nt_adapter_plan(const adapter_desc* d, int cus, int* way, int tile[2], int64_t* parts, int low_tile[2], int64_t* low_parts)
{
    if (cus < 1 || way == nullptr || tile == nullptr || parts == nullptr || low_tile == nullptr || low_parts == nullptr) return GEMM_F16_NT_INVALID_ARG;
    int st = check_adapters(d);
    if (st < 0) return st;
    *way = tile[0] = tile[1] = low_tile[0] = low_tile[1] = 0;
    *parts = *low_parts = 0;
    if (st > 0) return GEMM_F16_NT_OK;
    AdapterCall c;
    if ((st = plan_adapters(d, cus, &c)) != GEMM_F16_NT_OK) return st;
    if (c.single != nullptr) {
        *way = ADAPTER_ONE_LAUNCH;
        tile[0] = tile[1] = 16;
        *parts = 1;
        return GEMM_F16_NT_OK;
    }
    const bool pair = c.pair != nullptr;
    *way = pair ? (c.dots ? ADAPTER_DOTS : ADAPTER_SUMS) : c.each ? ADAPTER_EACH : ADAPTER_TILES;
    tile[0] = pair ? c.bm : c.plan.form->bm;
    tile[1] = pair ? c.bn : c.plan.form->bn;
    *parts = !pair && c.plan.walks ? (c.plan.part_bytes > 0 ? 0 : 1) : c.plan.splits;
    if (c.adapted) {
        low_tile[0] = pair ? 16 : c.low_plan.form->bm;
        low_tile[1] = pair ? 16 : c.low_plan.form->bn;
        *low_parts = pair ? 1 : c.low_plan.splits;
    }
    return GEMM_F16_NT_OK;
}

int64_t adapter_nt_workspace(const adapter_desc* d)
{
    int st = check_adapters(d), cus = 0;
    if (st != GEMM_F16_NT_OK) return st > 0 ? 0 : st;
    AdapterCall c;
    return (st = device_cus(&cus)) != GEMM_F16_NT_OK || (st = plan_adapters(d, cus, &c)) != GEMM_F16_NT_OK ? st : c.bytes;
}

int adapter_nt(const adapter_desc* d, void* workspace, int64_t workspace_bytes, void* stream)
{
    int st = check_adapters(d), cus = 0;
    if (st != GEMM_F16_NT_OK) return st > 0 ? GEMM_F16_NT_OK : st;
    AdapterCall c;
    if ((st = device_cus(&cus)) != GEMM_F16_NT_OK || (st = plan_adapters(d, cus, &c)) != GEMM_F16_NT_OK) return st;
    if ((st = check_workspace(workspace, workspace_bytes, c.bytes)) != GEMM_F16_NT_OK) return st;
    if ((st = check_adapters(d, {workspace, c.bytes})) != GEMM_F16_NT_OK) return st;
    if (c.single != nullptr) return launch(c.single, ceil_div(c.rest.cols, 16), 256, &c.rest, (hipStream_t)stream);
    if (c.pair != nullptr) return run_pair(c, workspace, (hipStream_t)stream);
    char* parts = (char*)workspace + c.low_bytes;
    if (c.adapted) {
        c.low.d = (char*)workspace;
        if ((st = run<LOW>(c.low_plan, c.low, parts, c.cus, (hipStream_t)stream)) != GEMM_F16_NT_OK) return st;
    }
    c.rest.low = (const char*)workspace;
    if (!c.each) return run<ADAPT>(c.plan, c.rest, parts, c.cus, (hipStream_t)stream);
    return d->rank <= 32 ? run<EACH>(c.plan, c.rest, parts, c.cus, (hipStream_t)stream) : run<EACH2>(c.plan, c.rest, parts, c.cus, (hipStream_t)stream);
}

}  // extern "C"
