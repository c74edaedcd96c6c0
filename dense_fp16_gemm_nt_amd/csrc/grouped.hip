// C-ABI boundary and kernels of the grouped products and of the product with
// low-rank adapters: argument validation (before any HIP call), device checks,
// plans and launches.  The contract of every entry point is in
// include/grouped.h, the shared device code in grouped_core.hpp.
#include "grouped.h"

#include <hip/hip_runtime.h>

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
// the adapters' second products added to the same sums.
enum Mode { NT, NN, TN, LOW, ADAPT };

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
    Div col_tiles;
    Div per_group;       // TN: tiles of a group, padded to whole rounds of the XCDs
    uint32_t group_tiles;
    // adapters
    const int32_t* ids;
    const float* scales;
    const char* low;     // LOW's results, rows of `rank`
    const char* up;
    int64_t up_ld, up_mat;
    int adapters;
    Div rank_chunks;
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

template <int BM, int BN, int MODE>
__device__ __forceinline__ Work find_work(const Args& g)
{
    uint32_t ti, tj;
    if (MODE == TN) {
        const uint32_t e = g.per_group.of(blockIdx.x), i = blockIdx.x - e * g.per_group.d;
        // whole rounds of the XCDs: each has a part of the group's tiles of its own
        const uint32_t t = g.per_group.d == g.group_tiles ? i : (uint32_t)xcd_slot(i, g.per_group.d);
        if (t >= g.group_tiles) return Work{0, 0, 0, 0, 0, false};
        grouped_tile_in<uint32_t>(t, g.group_tiles / g.col_tiles.d, g.col_tiles.d, kGroupTiles, &ti, &tj);
        const Rows s = rows_of(g, (int)e);
        return Work{(int)e, s.first, s.count, (int)ti * BM, (int)tj * BN, true};
    }
    Groups<BM, MODE> groups;
    groups.start(g);
    const uint32_t all = groups.total * g.col_tiles.d;
    if (blockIdx.x >= all) return Work{0, 0, 0, 0, 0, false};
    // each XCD has a run of neighbouring tiles, whose rows and columns its L2 holds
    const uint32_t t = (uint32_t)xcd_slot(blockIdx.x, all);
    grouped_tile_in<uint32_t>(t, groups.total, g.col_tiles.d, kGroupTiles, &ti, &tj);
    Work r = groups.find(g, ti);
    r.col0 = (int)tj * BN;
    return r;
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
// have `rank` elements of it each, in which a row meets its own request's part
// and zeros elsewhere.  A table in LDS says which they are.
struct Entry {
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

// The loads of step s of the requests' part of the contraction.
template <class C>
__device__ __forceinline__ void load_requests(const Args& g, const Work& wk, const Entry* table, int count, int s, uint32_t dst, int tid)
{
    using SX = grp::Side<C, false, C::BM>;
    using SY = grp::Side<C, false, C::BN>;
    const char* px[SX::LOADS];
    const char* py[SY::LOADS];
    auto where = [&](int chunk, int* in) {
        const int at = s * (C::BK / 8) + chunk, q = (int)g.rank_chunks.of((uint32_t)at);
        *in = at - q * (int)g.rank_chunks.d;
        return q < count ? table[q] : Entry{0, 0, -1};
    };
#pragma unroll
    for (int i = 0; i < SX::LOADS; ++i) {
        int in;
        const Entry e = where(SX::chunk(i, tid), &in);
        const int r = SX::row(i, tid);
        px[i] = r >= e.first && r < e.end ? g.low + ((int64_t)(wk.row0 + r) * g.rank_chunks.d + in) * 16 : (const char*)g_nothing;
    }
#pragma unroll
    for (int i = 0; i < SY::LOADS; ++i) {
        int in;
        const Entry e = where(SY::chunk(i, tid), &in);
        const int r = wk.col0 + SY::row(i, tid);
        py[i] = e.id >= 0 && r < g.cols ? g.up + (int64_t)e.id * g.up_mat + (int64_t)r * g.up_ld + 16 * in : (const char*)g_nothing;
    }
    load_all<C::THREADS * 16>(px, dst, std::make_integer_sequence<int, SX::LOADS>());
    load_all<C::THREADS * 16>(py, dst + C::X_BYTES, std::make_integer_sequence<int, SY::LOADS>());
}

template <typename T, class C, int MODE, bool F32>
__global__ __launch_bounds__(C::THREADS, C::PER_CU * C::WAVES / 4) void tile_kernel(const Args g)
{
    constexpr bool XC = MODE == TN, YC = MODE == NN || MODE == TN;
    __shared__ __attribute__((aligned(1024))) char smem[C::LDS + (MODE == ADAPT ? C::BM * sizeof(Entry) + 16 : 0)];
    const Work wk = find_work<C::BM, C::BN, MODE>(g);
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
            y.start(mat + (int64_t)wk.col0 * g.y_ld, g.y_ld, g.cols - wk.col0, tid);
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
    uint32_t fill = 0;
    auto load = [&] {
        x.next(mine + fill, left, tid);
        y.next(mine + fill + C::X_BYTES, left, tid);
        left -= C::BK;
        fill = fill == (C::STAGES - 1) * C::STAGE ? 0 : fill + C::STAGE;
    };
    Entry* table = reinterpret_cast<Entry*>(smem + C::LDS);
    int requests = 0, next = 0;   // ADAPT: of the tile; the next step of theirs
    auto load_more = [&] {
        if (MODE == ADAPT && left <= 0 && requests > 0) {
            load_requests<C>(g, wk, table, requests, next++, mine + fill, tid);
            fill = fill == (C::STAGES - 1) * C::STAGE ? 0 : fill + C::STAGE;
        } else {
            load();
        }
    };
    if constexpr (MODE == ADAPT) {
        const int own = steps < C::STAGES - 1 ? steps : C::STAGES - 1;
        for (int s = 0; s < own; ++s) load();
        int* count = reinterpret_cast<int*>(table + C::BM);
        if (w == 0) {
            const int n = fill_table<C::BM>(g, wk, table);
            if (lane == 0) *count = n;
        }
        __syncthreads();
        requests = __builtin_amdgcn_readfirstlane(*count);
        for (int s = own; s < C::STAGES - 1; ++s) load_more();
        steps += (requests * (int)g.rank_chunks.d + C::BK / 8 - 1) / (C::BK / 8);
    } else {
#pragma unroll
        for (int s = 0; s < C::STAGES - 1; ++s) load();
    }
    const bool busy = MODE == TN || wk.rows > wm * C::FM * 32;   // the wave has rows
    uint32_t stage = 0;
    for (int s = 0; s < steps; ++s) {
        grp::publish<(C::STAGES - 2) * C::LOADS>();
        load_more();
        if (busy) grp::multiply<T, C>(fx, fy, stage, acc);
        stage = stage == (C::STAGES - 1) * C::STAGE ? 0 : stage + C::STAGE;
    }
    grp::publish<0>();
    grp::add_waves<C>(smem, k, lane, acc);
    if (k > 0) return;

    float scale = 1.f;
    if (MODE == LOW && g.scales != nullptr) scale = g.scales[g.ids[wk.group]];
    const int r0 = wm * C::FM * 32, c0 = wn * C::FN * 32, rows = (MODE == TN ? g.x_cols - wk.tile0 : wk.rows) - r0, cols = g.cols - wk.col0 - c0;
    char* d = g.d + (MODE == TN ? (int64_t)wk.group * g.d_mat + (int64_t)(wk.tile0 + r0) * g.d_ld : (int64_t)(wk.row0 + r0) * g.d_ld) +
              (int64_t)(wk.col0 + c0) * (F32 ? 4 : 2);
    constexpr int STAGING = C::FN * 32 * 32 * (F32 ? 4 : 2);
    constexpr int AFTER = (C::WK - 1) * C::FM * C::FN * 4096;   // the other waves' sums
    static_assert(AFTER + C::WM * C::WN * STAGING <= C::LDS, "LDS budget");
    grp::store<T, C, F32>(smem + AFTER + (wm * C::WN + wn) * STAGING, d, g.d_ld, rows, cols, scale, acc, lane);
}

// Large tiles of NT, NN and TN: a workgroup for each compute unit walks them.
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
    uint32_t total;
    if (MODE == TN) {
        total = (uint32_t)g.groups * g.group_tiles;
    } else {
        groups.start(g);
        total = groups.total * g.col_tiles.d;
    }
    uint32_t slot = (uint32_t)xcd_slot(blockIdx.x, gridDim.x);
    if (slot >= total) return;

    grp::RingSide<XC> a;
    grp::RingSide<YC> b;
    grp::RingStore out;
    a.start(lds, g.x_ld, wm, w, lane);
    b.start(lds + 65536, g.y_ld, wn, w, lane);
    out.template start<F32>(lds, g.d_ld, w, lane);
    const uint32_t sta = (uint32_t)(STEP * g.x_ld), stb = (uint32_t)(STEP * g.y_ld);
    // the contraction's first step is the partial one: see gen_grouped_sched.py
    uint32_t kt = (uint32_t)(g.depth + STEP - 1) / STEP;
    const int hk = MODE == TN ? 0 : (int)kt * STEP - g.depth, kr = 16 * w + lane / 32;
    uint32_t hm[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) hm[q] = 8 * ((lane & 7) ^ grp::RingSide<false>::swz(8 * q + lane / 8)) < hk ? grp::kBeyond : 0u;

    for (; slot < total; slot += gridDim.x) {
        uint32_t ti, tj;
        Work wk;
        if (MODE == TN) {
            const uint32_t e = g.per_group.of(slot);
            grouped_tile_in<uint32_t>(slot - e * g.group_tiles, g.group_tiles / g.col_tiles.d, g.col_tiles.d, kGroupTiles, &ti, &tj);
            const Rows s = rows_of(g, (int)e);
            wk = Work{(int)e, s.first, s.count, (int)clamped_origin(ti, TILE, g.x_cols), 0, true};
            kt = (uint32_t)(s.count + STEP - 1) / STEP;
            if (kt < 2) kt = 2;
        } else {
            grouped_tile_in<uint32_t>(slot, groups.total, g.col_tiles.d, kGroupTiles, &ti, &tj);
            wk = groups.find(g, ti);
        }
        wk.col0 = (int)clamped_origin(tj, TILE, g.cols);

        u32x4 rsa, rsb;
        int rows = 128;   // of the wave
        const char* d;
        if (MODE == TN) {
            const int64_t n = wk.rows;
            rsa = grp::ring_rsrc(g.x + wk.row0 * g.x_ld + 2 * (int64_t)wk.tile0, n == 0 ? 0 : (n - 1) * g.x_ld + 2 * TILE);
            rsb = grp::ring_rsrc(g.y + wk.row0 * g.y_ld + 2 * (int64_t)wk.col0, n == 0 ? 0 : (n - 1) * g.y_ld + 2 * TILE);
            d = g.d + wk.group * g.d_mat + (int64_t)(wk.tile0 + wm) * g.d_ld;
        } else {
            const int64_t n = wk.rows < TILE ? wk.rows : TILE;
            const char* mat = g.y + wk.group * g.y_mat;
            rsa = grp::ring_rsrc(g.x + wk.row0 * g.x_ld - 2 * hk, (n - 1) * g.x_ld + 2 * (int64_t)(g.depth + hk));
            if (MODE == NT)
                rsb = grp::ring_rsrc(mat + wk.col0 * g.y_ld - 2 * hk, (TILE - 1) * g.y_ld + 2 * (int64_t)(g.depth + hk));
            else
                rsb = grp::ring_rsrc(mat + 2 * (int64_t)wk.col0 - hk * g.y_ld, (int64_t)(g.depth + hk - 1) * g.y_ld + 2 * TILE);
            rows = clampi((int)n - wm, 0, 128);
            d = g.d + (int64_t)(wk.row0 + wm) * g.d_ld;
        }
        const u32x4 rsd = grp::ring_rsrc(d + (int64_t)(wk.col0 + wn) * (F32 ? 4 : 2), rows == 0 ? 0 : (rows - 1) * g.d_ld + 128 * (F32 ? 4 : 2));
        uint32_t koa = 0, kob = 0, kha, khb, rem = kt, sdo;
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"   // M0 is written inside, on purpose
#define G16_GROUPED_BLOCK(LOOP, ...) \
    if constexpr (std::is_same<T, F16>::value) \
        asm volatile(LOOP("f16") : G16_GROUPED_STATE : G16_GROUPED_COMMON, __VA_ARGS__ : G16_GROUPED_CLOBBERS); \
    else \
        asm volatile(LOOP("bf16") : G16_GROUPED_STATE : G16_GROUPED_COMMON, __VA_ARGS__ : G16_GROUPED_CLOBBERS)
        if constexpr (MODE == NT) {
            G16_GROUPED_BLOCK(G16_GROUPED_RR, G16_GROUPED_STAGED, G16_GROUPED_A_ROWS, G16_GROUPED_B_ROWS);
        } else if constexpr (MODE == NN) {
            G16_GROUPED_BLOCK(G16_GROUPED_RC, G16_GROUPED_STAGED, G16_GROUPED_A_ROWS, G16_GROUPED_B_COLS, [hk] "s"(hk), [kr] "v"(kr));
        } else if constexpr (F32) {
            G16_GROUPED_BLOCK(G16_GROUPED_CC32, G16_GROUPED_A_COLS, G16_GROUPED_B_COLS);
        } else {
            G16_GROUPED_BLOCK(G16_GROUPED_CC, G16_GROUPED_STAGED, G16_GROUPED_A_COLS, G16_GROUPED_B_COLS);
        }
#pragma clang diagnostic pop
        wg_barrier();   // every wave is done reading the ring before the next tile's loads
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
using Low64 = Cfg<32, 64, 128, 1, 1, 4, 6, 1>;
using Low128 = Cfg<32, 128, 128, 1, 1, 4, 4, 1>;
using Square = Cfg<64, 64, 128, 2, 2, 1, 4, 1>;
using Middle = Cfg<128, 128, 64, 2, 2, 1, 2, 2>;
using Large = Cfg<256, 256, 64, 2, 4, 1, 2, 1>;

struct Shape {
    int bm, bn, threads;
    const void* f;
    bool walks;   // a workgroup for each compute unit at most
};

template <typename T, class C, int MODE, bool F32 = false>
Shape shape()
{
    return {C::BM, C::BN, C::THREADS, (const void*)&tile_kernel<T, C, MODE, F32>, false};
}
template <typename T, int MODE, bool F32 = false>
Shape ring_shape()
{
    return {grp::kRingTile, grp::kRingTile, 256, (const void*)&ring_kernel<T, MODE, F32>, true};
}

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
    return g.depth > grp::kRingStep && (mode == NT || ((int64_t)g.depth + 2 * grp::kRingStep) * g.y_ld < (int64_t(1) << 31));
}

// Tiles by the rows that a group has on average, and for few rows by the
// workgroups that they make.
template <typename T, int MODE>
Shape pick(const Args& g, int cus)
{
    const int64_t rows = g.rows, groups = MODE == ADAPT ? 1 : g.groups, cols = g.cols;
    const int64_t used = groups < rows ? groups : rows, mean = ceil_div(rows, used);
    if (mean <= 16 && used * ceil_div(cols, 32) < 2 * cus) return shape<T, Tiny, MODE>();
    const int64_t large = (rows + 255 * used) / 256 * ceil_div(cols, 256);
    if constexpr (MODE == ADAPT) {
        if (mean <= 32) return shape<T, Small, MODE>();
        if (mean <= 64) return shape<T, Square, MODE>();
        return mean > 160 && large >= cus ? shape<T, Large, MODE>() : shape<T, Middle, MODE>();
    } else {
        if (mean <= 48) return used * ceil_div(mean, 32) * ceil_div(cols, 128) < 2 * cus ? shape<T, Small, MODE>() : shape<T, Flat, MODE>();
        return mean > 160 && large >= cus && ring_takes(MODE, g) ? ring_shape<T, MODE>() : shape<T, Middle, MODE>();
    }
}

template <typename T>
Shape pick_low(int64_t rows, int64_t requests, int rank)
{
    const int64_t used = requests < rows ? requests : rows;
    if (ceil_div(rows, used) <= 16) return shape<T, Tiny, LOW>();
    return rank <= 32 ? shape<T, Small, LOW>() : rank <= 64 ? shape<T, Low64, LOW>() : shape<T, Low128, LOW>();
}

template <typename T, bool F32>
Shape pick_tn(const Args& g, int cus)
{
    const int64_t large = (int64_t)g.groups * ceil_div(g.x_cols, 256) * ceil_div(g.cols, 256);
    return g.rows > 192 * (int64_t)g.groups && large >= cus && ring_takes(TN, g) ? ring_shape<T, TN, F32>() : shape<T, Middle, TN, F32>();
}

template <int MODE>
int run(const Shape& c, const Args& args, int cus, hipStream_t s)
{
    Args g = args;
    const int64_t ct = ceil_div(g.cols, c.bn);
    g.col_tiles = attn::div_by(ct);
    int64_t wgs;
    if (MODE == TN) {
        const int64_t t = ct * ceil_div(g.x_cols, c.bm);
        const int64_t padded = c.walks || t < 8 * kNumXcd ? t : ceil_div(t, kNumXcd) * kNumXcd;
        g.group_tiles = (uint32_t)t;
        g.per_group = attn::div_by(padded);
        wgs = padded * g.groups;
    } else {
        const int64_t used = MODE == ADAPT ? 1 : g.groups < g.rows ? g.groups : g.rows;   // groups with rows
        wgs = (g.rows + used * (c.bm - 1)) / c.bm * ct;
    }
    if (wgs > kMaxTiles) return GEMM_F16_NT_UNSUPPORTED;
    if (c.walks && wgs > cus) wgs = cus;
    return launch(c.f, wgs, c.threads, &g, s);
}

bool widths_ok(int64_t n, int64_t k) { return n % 8 == 0 && k % 8 == 0 && n < kMaxWidth && k < kMaxWidth; }

enum Written { A_, B_, D_ };

int check_grouped(const grouped_desc* d, Written out)
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
        const void* w = out == A_ ? d->A : out == B_ ? d->B : d->D;
        const int64_t we = out == A_ ? ea : out == B_ ? eb : ed;
        if ((out != A_ && overlaps(w, we, d->A, ea)) || (out != B_ && overlaps(w, we, d->B, eb)) ||
            (out != D_ && overlaps(w, we, d->D, ed)) || (d->groups < kMaxGroups && overlaps(w, we, d->cu, 4 * (d->groups + 1))))
            return GEMM_F16_NT_INVALID_ARG;
    }
    if (out != B_ && d->b_fp32) return GEMM_F16_NT_UNSUPPORTED;
    if (!widths_ok(d->N, d->K) || d->lda >= kMaxWidth || d->ldb >= kMaxWidth || d->ldd >= kMaxWidth) return GEMM_F16_NT_UNSUPPORTED;
    if (d->rows > kMaxRows || d->groups >= kMaxGroups) return GEMM_F16_NT_UNSUPPORTED;
    if (!aligned16(d->A, {d->lda}) || !aligned16(d->D, {d->ldd}) || !aligned16(d->B, {d->ldb, d->stride_b})) return GEMM_F16_NT_UNSUPPORTED;
    return ((uintptr_t)d->cu & 3) != 0 ? GEMM_F16_NT_UNSUPPORTED : none ? 1 : GEMM_F16_NT_OK;
}

struct Span {
    const void* p;
    int64_t bytes;
};

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

int64_t low_bytes(const adapter_desc* d) { return d->adapters == 0 ? 0 : 2 * d->rows * d->rank; }

}  // namespace

extern "C" {

int grouped_nt_check(const grouped_desc* d) { const int st = check_grouped(d, D_); return st > 0 ? GEMM_F16_NT_OK : st; }
int grouped_nn_check(const grouped_desc* d) { const int st = check_grouped(d, A_); return st > 0 ? GEMM_F16_NT_OK : st; }
int grouped_tn_check(const grouped_desc* d) { const int st = check_grouped(d, B_); return st > 0 ? GEMM_F16_NT_OK : st; }
int adapter_nt_check(const adapter_desc* d) { const int st = check_adapters(d); return st > 0 ? GEMM_F16_NT_OK : st; }

int grouped_nt(const grouped_desc* d, void* stream)
{
    int st = check_grouped(d, D_);
    if (st != GEMM_F16_NT_OK) return st > 0 ? GEMM_F16_NT_OK : st;
    int cus = 0;
    if ((st = device_cus(&cus)) != GEMM_F16_NT_OK) return st;
    Args g = {};
    g.x = (const char*)d->A;
    g.y = (const char*)d->B;
    g.d = (char*)d->D;
    g.cu = d->cu;
    g.x_ld = 2 * d->lda;
    g.y_ld = 2 * d->ldb;
    g.y_mat = 2 * d->stride_b;
    g.d_ld = 2 * d->ldd;
    g.groups = (int)d->groups;
    g.rows = (int)d->rows;
    g.cols = (int)d->N;
    g.depth = (int)d->K;
    return run<NT>(d->dtype == GROUPED_F16 ? pick<F16, NT>(g, cus) : pick<BF16, NT>(g, cus), g, cus, (hipStream_t)stream);
}

int grouped_nn(const grouped_desc* d, void* stream)
{
    int st = check_grouped(d, A_);
    if (st != GEMM_F16_NT_OK) return st > 0 ? GEMM_F16_NT_OK : st;
    int cus = 0;
    if ((st = device_cus(&cus)) != GEMM_F16_NT_OK) return st;
    Args g = {};
    g.x = (const char*)d->D;
    g.y = (const char*)d->B;
    g.d = (char*)d->A;
    g.cu = d->cu;
    g.x_ld = 2 * d->ldd;
    g.y_ld = 2 * d->ldb;
    g.y_mat = 2 * d->stride_b;
    g.d_ld = 2 * d->lda;
    g.groups = (int)d->groups;
    g.rows = (int)d->rows;
    g.cols = (int)d->K;
    g.depth = (int)d->N;
    return run<NN>(d->dtype == GROUPED_F16 ? pick<F16, NN>(g, cus) : pick<BF16, NN>(g, cus), g, cus, (hipStream_t)stream);
}

int grouped_tn(const grouped_desc* d, void* stream)
{
    int st = check_grouped(d, B_);
    if (st != GEMM_F16_NT_OK) return st > 0 ? GEMM_F16_NT_OK : st;
    int cus = 0;
    if ((st = device_cus(&cus)) != GEMM_F16_NT_OK) return st;
    Args g = {};
    g.x = (const char*)d->D;
    g.y = (const char*)d->A;
    g.d = (char*)d->B;
    g.cu = d->cu;
    g.x_ld = 2 * d->ldd;
    g.y_ld = 2 * d->lda;
    const int64_t size = d->b_fp32 ? 4 : 2;
    g.d_ld = size * d->ldb;
    g.d_mat = size * d->stride_b;
    g.groups = (int)d->groups;
    g.rows = (int)d->rows;
    g.x_cols = (int)d->N;
    g.cols = (int)d->K;
    const bool f16 = d->dtype == GROUPED_F16;
    const Shape c = d->b_fp32 ? (f16 ? pick_tn<F16, true>(g, cus) : pick_tn<BF16, true>(g, cus))
                              : (f16 ? pick_tn<F16, false>(g, cus) : pick_tn<BF16, false>(g, cus));
    return run<TN>(c, g, cus, (hipStream_t)stream);
}

int64_t adapter_nt_workspace(const adapter_desc* d)
{
    const int st = check_adapters(d);
    return st < 0 ? st : st > 0 ? 0 : low_bytes(d);
}

int adapter_nt(const adapter_desc* d, void* workspace, int64_t workspace_bytes, void* stream)
{
    int st = check_adapters(d);
    if (st != GEMM_F16_NT_OK) return st > 0 ? GEMM_F16_NT_OK : st;
    if ((st = check_adapters(d, {workspace, low_bytes(d)})) != GEMM_F16_NT_OK) return st;
    if ((st = check_workspace(workspace, workspace_bytes, low_bytes(d))) != GEMM_F16_NT_OK) return st;
    int cus = 0;
    if ((st = device_cus(&cus)) != GEMM_F16_NT_OK) return st;
    const bool adapted = low_bytes(d) > 0, f16 = d->dtype == GROUPED_F16;
    Args g = {};
    g.x = (const char*)d->A;
    g.cu = d->cu;
    g.x_ld = 2 * d->lda;
    g.groups = (int)d->requests;
    g.rows = (int)d->rows;
    g.depth = (int)d->K;
    g.ids = d->ids;
    g.scales = d->scales;
    g.adapters = adapted ? (int)d->adapters : 0;
    g.rank_chunks = attn::div_by(adapted ? d->rank / 8 : 1);
    if (adapted) {
        Args l = g;
        l.y = (const char*)d->down;
        l.y_ld = 2 * d->ld_down;
        l.y_mat = 2 * d->stride_down;
        l.d = (char*)workspace;
        l.d_ld = 2 * d->rank;
        l.cols = (int)d->rank;
        const Shape c = f16 ? pick_low<F16>(d->rows, d->requests, d->rank) : pick_low<BF16>(d->rows, d->requests, d->rank);
        if ((st = run<LOW>(c, l, cus, (hipStream_t)stream)) != GEMM_F16_NT_OK) return st;
    }
    g.y = (const char*)d->B;
    g.y_ld = 2 * d->ldb;
    g.d = (char*)d->D;
    g.d_ld = 2 * d->ldd;
    g.cols = (int)d->N;
    g.low = (const char*)workspace;
    g.up = (const char*)d->up;
    g.up_ld = 2 * d->ld_up;
    g.up_mat = 2 * d->stride_up;
    return run<ADAPT>(f16 ? pick<F16, ADAPT>(g, cus) : pick<BF16, ADAPT>(g, cus), g, cus, (hipStream_t)stream);
}

}  // extern "C"
