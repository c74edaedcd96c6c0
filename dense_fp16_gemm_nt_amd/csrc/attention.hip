// C-ABI boundary and kernels of the attention operators: argument validation
// (before any HIP call), device checks, split plans and launches.  The
// contract of every entry point is in include/attention.h, the shared device
// code in attn_core.hpp.
#include "attention.h"

#include <hip/hip_runtime.h>

#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstring>
#include <initializer_list>

#include "attn_core.hpp"
#include "sched.hpp"

using namespace g16;

namespace {

using attn::BF16;
using attn::Div;
using attn::F16;
using attn::f32x2;
using attn::Job;
using attn::kThreads;
using attn::kTileKeys;
using attn::kTileRows;
using attn::Keys;
using attn::Parts;
using attn::Row;
using attn::State;

// ---------------------------------------------------------------- prompt
struct PromptArgs {
    const char* q;
    const char* k;
    const char* v;
    char* o;
    float* lse;
    const int32_t* cu_q;
    const int32_t* cu_k;
    int64_t q_row, q_head, k_row, k_head, v_row, v_head, o_row, o_head;   // bytes
    int batch, total_q, total_k, heads, kv_heads, d, causal;
    int careful;   // rows may meet keys that they do not read: see accumulate_careful
    Div group, splits, units;   // units: kv heads x splits, or an eighth of them (by_xcd)
    Div join_kv;                // kv heads
    int by_xcd;
    float c, slack;
    uint32_t flip;
    int zero;
    Parts parts;
};

// A row tile of the packed batch: sequence bounds and the tile's first row.
struct Tile {
    int q0, nq, k0, nk, row0;
    bool found;
};

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

// A sequence's bounds and its number of tiles.  Offsets are clamped to the
// tensors, so that a table that decreases or runs past them still names rows
// that exist.
struct Seq {
    int q0, nq, k0, nk;
    uint32_t tiles;
};

template <int ROWS>
__device__ __forceinline__ Seq sequence(const PromptArgs& g, int b)
{
    const int a0 = g.cu_q[b], a1 = g.cu_q[b + 1], b0 = g.cu_k[b], b1 = g.cu_k[b + 1];
    Seq s;
    s.q0 = clampi(a0, 0, g.total_q);
    s.nq = clampi(a1, s.q0, g.total_q) - s.q0;
    s.k0 = clampi(b0, 0, g.total_k);
    s.nk = clampi(b1, s.k0, g.total_k) - s.k0;
    s.tiles = ((uint32_t)s.nq * g.group.d + ROWS - 1) / ROWS;
    return s;
}

// Sum over this lane and those below it, by the lanes' own data paths (six
// instructions; the same through LDS took 0.5 us of a workgroup's time).
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

// Tile `t` of the sequences' tiles put one after the other; each lane looks at
// one sequence, 64 at a time.  Within a sequence the tiles come in falling
// order: under a causal mask those have the most keys, and the longest work
// starts first.  (The tiles of all sequences ordered by their keys took 131
// against 132 us on packed lengths of 1 to 2900 and 46 against 44 with heads of
// 96: neighbours then share no keys.)
template <int ROWS>
__device__ __forceinline__ Tile find_tile(const PromptArgs& g, uint32_t t)
{
    Tile r = {0, 0, 0, 0, 0, false};
    if (g.batch == 1) {
        const Seq s = sequence<ROWS>(g, 0);
        r = Tile{s.q0, s.nq, s.k0, s.nk, (int)((s.tiles - 1 - t) * ROWS), t < s.tiles};
        return r;
    }
    const int lane = threadIdx.x & 63;
    uint32_t before = 0;
    for (int base = 0; base < g.batch; base += 64) {
        Seq s = {0, 0, 0, 0, 0};
        if (base + lane < g.batch) s = sequence<ROWS>(g, base + lane);
        const uint32_t upto = before + wave_scan(s.tiles);
        const uint64_t past = __builtin_amdgcn_ballot_w64(upto > t);
        if (past != 0) {
            const int w = __builtin_ctzll(past);
            r.found = true;
            r.q0 = __builtin_amdgcn_readlane(s.q0, w);
            r.nq = __builtin_amdgcn_readlane(s.nq, w);
            r.k0 = __builtin_amdgcn_readlane(s.k0, w);
            r.nk = __builtin_amdgcn_readlane(s.nk, w);
            r.row0 = (__builtin_amdgcn_readlane((int)upto, w) - 1 - (int)t) * ROWS;
            return r;
        }
        before = (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
    }
    return r;
}

// Part `i` of n things split evenly: [first, last).
struct Range {
    int first, last;
};
__device__ __forceinline__ Range part_of(int n, const Div& splits, int i)
{
    const int per = (int)splits.of((uint32_t)n + splits.d - 1);
    const int first = i * per < n ? i * per : n;
    return {first, first + per < n ? first + per : n};
}

template <int ROWS>
__device__ __forceinline__ Job prompt_job(const PromptArgs& g, const Tile& t, int kv)
{
    Job j;
    j.q = g.q + (int64_t)t.q0 * g.q_row + (int64_t)kv * g.group.d * g.q_head;
    j.k = g.k + (int64_t)t.k0 * g.k_row + (int64_t)kv * g.k_head;
    j.v = g.v + (int64_t)t.k0 * g.v_row + (int64_t)kv * g.v_head;
    j.q_token = g.q_row;
    j.q_head = g.q_head;
    j.k_row = g.k_row;
    j.v_row = g.v_row;
    j.rows = t.nq * (int)g.group.d;
    j.row0 = t.row0;
    j.group = g.group;
    j.keys = t.nk;
    j.lead = g.causal ? t.nk - t.nq : INT32_MAX;
    j.d = g.d;
    j.c = g.c;
    j.slack = g.slack;
    j.flip = g.flip;
    j.zero = g.zero != 0;
    j.most = t.nk;
    if (g.causal) {
        const int last = (j.rows - t.row0 > ROWS ? t.row0 + ROWS : j.rows) - 1;
        j.most = clampi((int)g.group.of(last) + j.lead + 1, 0, t.nk);
    }
    return j;
}

// W waves of 32 rows (four, or eight for long workgroups: see plan_prompt).
// Heads of up to 64 elements leave registers for three waves on a SIMD.
template <typename T, int D, bool SPLIT, int W>
__global__ __launch_bounds__(64 * W, D == 64 && W == 4 ? 3 : 2) void prompt_kernel(const PromptArgs g)
{
    __shared__ __attribute__((aligned(256))) char smem[attn::lds_bytes<D>()];
    constexpr int ROWS = W * attn::kWaveRows;
    // a unit is a kv head and a split; consecutive workgroups go to the XCDs
    // in turn, and each XCD keeps to its own units, whose keys its L2 then
    // holds, with the tiles of the most keys first
    uint32_t i = blockIdx.x;
    if (g.by_xcd) i /= kNumXcd;
    const uint32_t t = g.units.of(i);
    uint32_t unit = i - t * g.units.d;
    if (g.by_xcd) unit += blockIdx.x % kNumXcd * g.units.d;
    const int kv = (int)g.splits.of(unit), split = SPLIT ? (int)(unit - kv * g.splits.d) : 0;
    const Tile tile = find_tile<ROWS>(g, t);
    if (!tile.found) return;
    Job j = prompt_job<ROWS>(g, tile, kv);
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    State<D> st;
    const int rows = j.rows - j.row0;
    if (rows <= attn::kWaveRows) {
        // the rows of one wave (a single token, a short chunk): four waves
        // take them and divide the keys
        const Row row = attn::row_of(j, j.row0 + (lane & 31));
        const Keys keys = {j.k, j.v, j.k_row, j.v_row, j.keys}, none = {};
        const int n = attn::key_blocks(j.most);
        const Range r = SPLIT ? part_of(n, g.splits, split) : Range{0, n};
        attn::run_blocks<T, D, 2, false, false>(j, keys, none, r.first, r.last, row, smem, st);
        if (g.careful && attn::spoilt<D>(st)) {
            attn::landed<0>();
            attn::run_blocks<T, D, 2, true>(j, keys, none, r.first, r.last, row, smem, st);
        }
        attn::merge_waves<D>(j, st, row.valid, rows, smem, [&](int y, int e, float m, float l, f32x4 o) {
            const int x = j.row0 + y, token_in = (int)g.group.of(x);
            const int64_t token = (int64_t)tile.q0 + token_in;
            const int head = kv * (int)g.group.d + x - token_in * (int)g.group.d;
            if constexpr (SPLIT)
                attn::store_part4(g.parts, split, token * g.heads + head, g.d, e, m, l, o);
            else
                attn::store_row4<T>(g.o + token * g.o_row + head * g.o_head,
                                    g.lse == nullptr ? nullptr : g.lse + token * g.heads + head, g.c, e, m, l, o);
        });
        return;
    }
    const int n = (int)(((uint32_t)j.most + kTileKeys - 1) / kTileKeys);
    const Range r = SPLIT ? part_of(n, g.splits, split) : Range{0, n};
    j.tile0 = r.first;
    j.tile1 = r.last;
    const Row row = attn::row_of(j, j.row0 + w * attn::kWaveRows + (lane & 31));
    attn::run_tiles<T, D, W>(j, row, smem, st);
    if (g.careful && attn::any_wave<W>(attn::spoilt<D>(st), smem)) {
        attn::init(st);
        attn::run_tiles_careful<T, D, W>(j, row, smem, st);
    }
    const int64_t token = (int64_t)tile.q0 + row.token;
    const int head = kv * (int)g.group.d + row.head;
    if constexpr (SPLIT)
        attn::store_part<D>(st, row.valid, g.d, g.parts, split, token * g.heads + head, half);
    else
        attn::store_row<T, D>(j, st, row.valid, g.o + token * g.o_row + head * g.o_head,
                              g.lse == nullptr ? nullptr : g.lse + token * g.heads + head, half);
}

// Joins the splits: 32 lanes of 4 elements and GROUPS groups of parts for a row.
template <int GROUPS>
constexpr int kJoinRows = kThreads / 32 / GROUPS;

template <typename T, int GROUPS>
__global__ __launch_bounds__(kThreads) void prompt_join_kernel(const PromptArgs g)
{
    constexpr uint32_t kSub = kTileRows / kJoinRows<GROUPS>;
    const uint32_t sub = blockIdx.x % kSub, x = blockIdx.x / kSub, t = g.join_kv.of(x);
    const int kv = (int)(x - t * g.join_kv.d);
    const Tile tile = find_tile<kTileRows>(g, t);
    if (!tile.found) return;
    const int r = tile.row0 + (int)sub * kJoinRows<GROUPS> + (int)(threadIdx.x >> 5) / GROUPS, e = (threadIdx.x & 31) * 4;
    const bool there = r < tile.nq * (int)g.group.d && e < g.d;
    const int token_in = (int)g.group.of(r);
    const int64_t token = (int64_t)tile.q0 + token_in;
    const int head = kv * (int)g.group.d + r - token_in * (int)g.group.d;
    attn::join_row<T, GROUPS>(g.parts, (int)g.splits.d, there, token * g.heads + head, g.c, g.d, e,
                              g.o + token * g.o_row + head * g.o_head,
                              g.lse == nullptr ? nullptr : g.lse + token * g.heads + head);
}

// --------------------------------------------------------- shared prefix
struct SharedArgs {
    const char* q;
    const char* kp;
    const char* vp;
    const char* ks;
    const char* vs;
    char* o;
    float* lse;
    const int32_t* lens;
    int64_t q_row, q_head, kp_row, kp_head, vp_row, vp_head;   // bytes
    int64_t ks_slot, ks_row, ks_head, vs_slot, vs_row, vs_head, o_row, o_head;
    int batch, prefix, slot_rows, heads, d;
    Div group, kv_heads, round, row_tiles, own_tiles, prefix_splits, own_splits;   // see SharedPlan
    int together;
    int parts_of_row;     // the prefix's, then those of the row's own keys, of
    int own_blocks;       // blocks of 32 keys each
    uint32_t prefix_wgs, own_wgs, round_prefix, round_own;
    int by_xcd;
    int rounded;          // the prefix goes through row tiles
    int solo;             // a wave takes what a workgroup would of the slots' own keys
    uint32_t own_jobs;    // of these
    float c, slack;
    uint32_t flip;
    int zero;
    Parts parts;
};

template <typename T, int D>
__global__ __launch_bounds__(kThreads, 2) void shared_kernel(const SharedArgs g)
{
    __shared__ __attribute__((aligned(256))) char smem[attn::lds_bytes<D>()];
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // Workgroups on the prefix (matrix products) and on the slots' own keys
    // (bytes from HBM) come in rounds: one on the prefix for each compute
    // unit, then a share of the others, so that a compute unit works on both
    // at once.
    uint32_t i = blockIdx.x;
    const uint32_t round = g.round.of(i);
    i -= round * g.round.d;
    const bool own = i >= g.round_prefix;
    i = own ? i - g.round_prefix + round * g.round_own : i + round * g.round_prefix;
    if (i >= (own ? g.own_wgs : g.prefix_wgs)) return;
    Job j;
    j.q_token = g.q_row;
    j.q_head = g.q_head;
    j.group = g.group;
    j.lead = INT32_MAX;
    j.d = g.d;
    j.c = g.c;
    j.slack = g.slack;
    j.flip = g.flip;
    j.zero = g.zero != 0;
    State<D> st;
    if (!own) {
        uint32_t unit, t;   // a kv head and a part of the prefix, and rows
        if (g.by_xcd) {     // the row tiles of a unit one after the other on one XCD: its L2 holds their keys
            const uint32_t x = i / kNumXcd;
            unit = g.row_tiles.of(x);
            t = x - unit * g.row_tiles.d;
            unit = unit * kNumXcd + i % kNumXcd;
        } else {
            unit = g.row_tiles.of(i);
            t = i - unit * g.row_tiles.d;
        }
        const int kv = (int)g.prefix_splits.of(unit), part = (int)(unit - kv * g.prefix_splits.d);
        j.q = g.q + (int64_t)kv * g.group.d * g.q_head;
        j.k = g.kp + kv * g.kp_head;
        j.v = g.vp + kv * g.vp_head;
        j.k_row = g.kp_row;
        j.v_row = g.vp_row;
        j.rows = g.batch * (int)g.group.d;
        j.row0 = (int)t * kTileRows;
        j.keys = g.prefix;
        if (j.rows <= attn::kWaveRows) {
            const Row row = attn::row_of(j, lane & 31);
            const Keys keys = {j.k, j.v, j.k_row, j.v_row, j.keys}, none = {};
            const Range r = part_of(attn::key_blocks(g.prefix), g.prefix_splits, part);
            attn::run_blocks<T, D, 2>(j, keys, none, r.first, r.last, row, smem, st);
            attn::merge_waves<D>(j, st, row.valid, j.rows, smem, [&](int r, int e, float m, float l, f32x4 o) {
                const int b = (int)g.group.of(r);
                const int64_t x = (int64_t)b * g.heads + kv * (int)g.group.d + r - b * (int)g.group.d;
                attn::store_part4(g.parts, part, x, g.d, e, m, l, o);
            });
            return;
        }
        const Range r = part_of((int)(((uint32_t)g.prefix + kTileKeys - 1) / kTileKeys), g.prefix_splits, part);
        j.tile0 = r.first;
        j.tile1 = r.last;
        const Row row = attn::row_of(j, j.row0 + w * attn::kWaveRows + (lane & 31));
        // a last tile whose end holds rows of V that are no keys goes by itself
        const int ragged = attn::overlap(j.v_row, j.d) && j.tile1 > j.tile0 && (int64_t)j.tile1 * kTileKeys > g.prefix;
        j.tile1 -= ragged;
        attn::run_tiles<T, D, attn::kWaves>(j, row, smem, st);
        if (ragged) {
            j.tile0 = j.tile1++;
            attn::run_tiles_careful<T, D, attn::kWaves>(j, row, smem, st);
        }
        attn::store_part<D>(st, row.valid, g.d, g.parts, part,
                            (int64_t)row.token * g.heads + kv * (int)g.group.d + row.head, half);
        return;
    }
    if (g.solo) {   // each wave a slot's rows and keys of its own
        i = i * attn::kWaves + w;
        if (i >= g.own_jobs) return;
    }
    uint32_t y = g.kv_heads.of(i);
    const int kv = (int)(i - y * g.kv_heads.d);
    const Div& splits = g.together ? g.prefix_splits : g.own_splits;
    uint32_t z = splits.of(y);
    const int split = (int)(y - z * splits.d);
    const int64_t slot = g.own_tiles.of(z);
    j.row0 = (int)(z - (uint32_t)slot * g.own_tiles.d) * attn::kWaveRows;
    const int len = g.lens[slot];
    if (len < 0) return;
    const Keys mine = {g.ks + slot * g.ks_slot + kv * g.ks_head, g.vs + slot * g.vs_slot + kv * g.vs_head, g.ks_row, g.vs_row,
                       len < g.slot_rows ? len : g.slot_rows};
    const Keys before = {g.kp + kv * g.kp_head, g.vp + kv * g.vp_head, g.kp_row, g.vp_row, g.together ? g.prefix : 0};
    j.q = g.q + slot * g.q_row + (int64_t)kv * g.group.d * g.q_head;
    j.rows = (int)g.group.d;
    j.keys = INT32_MAX;   // the runs end themselves
    const int rows = j.rows - j.row0 < attn::kWaveRows ? j.rows - j.row0 : attn::kWaveRows;
    const int own_n = attn::key_blocks(mine.keys);
    const int64_t x0 = slot * g.heads + kv * j.rows + j.row0;
    int part = split, block0, block1;
    if (g.together) {
        const Range r = part_of(attn::key_blocks(g.prefix) + own_n, splits, split);
        block0 = r.first;
        block1 = r.last;
    } else {
        part += (int)g.prefix_splits.d;
        block0 = split * g.own_blocks;
        block1 = block0 + g.own_blocks < own_n ? block0 + g.own_blocks : own_n;
        if (block0 >= block1) {   // the slot is not that long
            if (lane < rows)
                *reinterpret_cast<f32x2*>(g.parts.ml + 2 * (part * g.parts.n + x0 + lane)) =
                    f32x2{-__builtin_inff(), 0.f};
            return;
        }
    }
    const Row row = attn::row_of(j, j.row0 + (lane & 31));
    if (g.solo) {
        const int head = kv * j.rows + row.head;
        if (g.together)
            attn::run_blocks<T, D, 2, false, true, 1>(j, before, mine, block0, block1, row, smem, st);
        else
            attn::run_blocks<T, D, 1, false, true, 1>(j, before, mine, block0, block1, row, smem, st);
        attn::landed<0>();   // the loads past the last block
        if (g.together)
            attn::store_row<T, D>(j, st, row.valid, g.o + slot * g.o_row + (int64_t)head * g.o_head,
                                  g.lse == nullptr ? nullptr : g.lse + slot * g.heads + head, half);
        else
            attn::store_part<D>(st, row.valid, g.d, g.parts, part, slot * g.heads + head, half);
        return;
    }
    // beside a prefix whose weights are rounded once, so are these
    if (g.rounded)
        attn::run_blocks<T, D, 1>(j, before, mine, block0, block1, row, smem, st);
    else
        attn::run_blocks<T, D, 2>(j, before, mine, block0, block1, row, smem, st);
    attn::merge_waves<D>(j, st, row.valid, rows, smem, [&](int r, int e, float m, float l, f32x4 o) {
        if (g.parts_of_row == 1)
            attn::store_row4<T>(g.o + slot * g.o_row + (int64_t)(kv * j.rows + j.row0 + r) * g.o_head,
                                g.lse == nullptr ? nullptr : g.lse + x0 + r, g.c, e, m, l, o);
        else
            attn::store_part4(g.parts, part, x0 + r, g.d, e, m, l, o);
    });
}

template <typename T, int GROUPS>
__global__ __launch_bounds__(kThreads) void shared_join_kernel(const SharedArgs g)
{
    const int64_t x = (int64_t)blockIdx.x * kJoinRows<GROUPS> + (threadIdx.x >> 5) / GROUPS;
    const int e = (threadIdx.x & 31) * 4;
    const int64_t b = x / g.heads;
    const bool there = b < g.batch && e < g.d && g.lens[b] >= 0;
    const int64_t head = x - b * g.heads;
    attn::join_row<T, GROUPS>(g.parts, g.parts_of_row, there, x, g.c, g.d, e, g.o + b * g.o_row + head * g.o_head,
                              g.lse == nullptr ? nullptr : g.lse + x);
}

// --------------------------------------------------------------- devices
constexpr int kMaxDevices = 64;
std::atomic<int> g_cus[kMaxDevices];   // compute units; 0 unknown, -1 not gfx950

int device_cus(int* cus)
{
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return GEMM_F16_NT_DEVICE;
    int n = g_cus[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        hipDeviceProp_t prop;
        n = -1;
        if (hipGetDeviceProperties(&prop, dev) == hipSuccess && std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 &&
            prop.multiProcessorCount > 0)
            n = prop.multiProcessorCount;
        g_cus[dev].store(n, std::memory_order_relaxed);   // threads that ask at once store the same
    }
    if (n < 0) return GEMM_F16_NT_DEVICE;
    *cus = n;
    return GEMM_F16_NT_OK;
}

// ------------------------------------------------------------ validation
constexpr int64_t kMaxRowStride = int64_t(1) << 23;   // a tile of 64 rows spans less than 2^30 bytes
constexpr int64_t kMaxIndex = (int64_t(1) << 31) - 1024;
constexpr int64_t kMaxStride = int64_t(1) << 40;      // elements; keeps every offset inside 63 bits
constexpr int64_t kMaxBlocks = 64;   // of 32 keys, of a slot's part, so that long and short slots even out
// A launch holds less than 2^32 threads.  This many units of work (row tiles
// of 128 and slots' parts of 64 blocks of keys, times kv heads) keep every
// launch of a call, of workgroups of 512 threads, at half of that or less, and
// the joins at 4/5: 32 heads to a kv head and two parts are most, with
// 2^22 / (32 / 128 + 1) slots and kv heads of 32 rows, 8 rows to 256 threads.
constexpr int64_t kMaxUnits = int64_t(1) << 22;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool overlaps(const void* a, int64_t abytes, const void* b, int64_t bbytes)
{
    if (abytes <= 0 || bbytes <= 0) return false;
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + (uintptr_t)bbytes && b0 < a0 + (uintptr_t)abytes;
}

struct Axis {
    int64_t n, stride;
};

// Bytes from a tensor's first to its last element; 0 if it has none, -1 for
// a bad stride.
int64_t extent(int64_t d, std::initializer_list<Axis> axes)
{
    __int128 last = d - 1;
    for (const Axis& a : axes) {
        if (a.n == 0) return 0;
        if (a.stride < 0 || a.stride > kMaxStride) return -1;
        last += (__int128)(a.n - 1) * a.stride;
    }
    const __int128 bytes = 2 * (last + 1);
    return bytes < ((__int128)1 << 60) ? (int64_t)bytes : -1;
}

bool aligned16(const void* p, std::initializer_list<int64_t> strides)
{
    uint64_t all = (uintptr_t)p >> 1 | ((uintptr_t)p & 1);
    for (int64_t s : strides) all |= (uint64_t)s;
    return (all & 7) == 0;
}

// Heads, head size, type and scale.
int check_common(int dtype, int64_t heads, int64_t kv_heads, int64_t d, float scale)
{
    if (dtype != ATTN_F16 && dtype != ATTN_BF16) return GEMM_F16_NT_INVALID_ARG;
    if (heads < 1 || kv_heads < 1 || heads % kv_heads != 0 || d < 1) return GEMM_F16_NT_INVALID_ARG;
    if (!std::isfinite(scale) || !std::isfinite(scale * 1.4426950408889634f)) return GEMM_F16_NT_INVALID_ARG;
    if (d % 8 != 0 || d > 128 || heads > (1 << 20)) return GEMM_F16_NT_UNSUPPORTED;
    return GEMM_F16_NT_OK;
}

// O's rows and heads lie apart.
bool rows_apart(int64_t rows, int64_t row, int64_t heads, int64_t head, int64_t d)
{
    if (rows <= 1) return heads <= 1 || head >= d;
    if (heads <= 1) return row >= d;
    return (head >= d && row >= (heads - 1) * head + d) || (row >= d && head >= (rows - 1) * row + d);
}

struct Scale {
    float c, slack;
    uint32_t flip;
    int zero;
};

// scores = c * (q . k) in base 2 with c > 0: a negative scale flips Q's sign
// bits, which is exact; for scale 0 (or a c below fp32's normal numbers) every
// score is 0.
Scale scale_of(float scale)
{
    const float c = std::fabs(scale) * 1.4426950408889634f;
    if (c < FLT_MIN) return {1.f, attn::kSlack, 0u, 1};
    return {c, attn::kSlack / c, scale < 0.f ? 0x80008000u : 0u, 0};
}

int check_prompt(const attn_prompt_desc* d)
{
    if (d == nullptr) return GEMM_F16_NT_INVALID_ARG;
    const int st = check_common(d->dtype, d->heads, d->kv_heads, d->head_dim, d->scale);
    if (st != GEMM_F16_NT_OK) return st;
    if ((d->causal != 0 && d->causal != 1) || d->batch < 0 || d->total_q < 0 || d->total_k < 0) return GEMM_F16_NT_INVALID_ARG;
    const int64_t hd = d->head_dim;
    const int64_t eq = extent(hd, {{d->total_q, d->q_row}, {d->heads, d->q_head}});
    const int64_t eo = extent(hd, {{d->total_q, d->o_row}, {d->heads, d->o_head}});
    const int64_t ek = extent(hd, {{d->total_k, d->k_row}, {d->kv_heads, d->k_head}});
    const int64_t ev = extent(hd, {{d->total_k, d->v_row}, {d->kv_heads, d->v_head}});
    if (eq < 0 || eo < 0 || ek < 0 || ev < 0) return GEMM_F16_NT_INVALID_ARG;
    if (d->total_q == 0 || d->batch == 0) return GEMM_F16_NT_OK;
    if (d->Q == nullptr || d->O == nullptr || d->cu_q == nullptr || d->cu_k == nullptr) return GEMM_F16_NT_INVALID_ARG;
    if (d->total_k > 0 && (d->K == nullptr || d->V == nullptr)) return GEMM_F16_NT_INVALID_ARG;
    if (!rows_apart(d->total_q, d->o_row, d->heads, d->o_head, hd)) return GEMM_F16_NT_INVALID_ARG;
    const int64_t el = d->lse == nullptr ? 0 : d->total_q * d->heads * 4;
    if (overlaps(d->O, eo, d->Q, eq) || overlaps(d->O, eo, d->K, ek) || overlaps(d->O, eo, d->V, ev) ||
        overlaps(d->lse, el, d->O, eo) || overlaps(d->lse, el, d->Q, eq) || overlaps(d->lse, el, d->K, ek) ||
        overlaps(d->lse, el, d->V, ev))
        return GEMM_F16_NT_INVALID_ARG;
    if (!aligned16(d->Q, {d->q_row, d->q_head}) || !aligned16(d->O, {d->o_row, d->o_head}) ||
        !aligned16(d->K, {d->k_row, d->k_head}) || !aligned16(d->V, {d->v_row, d->v_head}))
        return GEMM_F16_NT_UNSUPPORTED;
    if (((uintptr_t)d->cu_q | (uintptr_t)d->cu_k | (uintptr_t)d->lse) & 3) return GEMM_F16_NT_UNSUPPORTED;
    if (d->k_row >= kMaxRowStride || d->v_row >= kMaxRowStride) return GEMM_F16_NT_UNSUPPORTED;
    const int64_t group = d->heads / d->kv_heads;
    if (d->batch > kMaxIndex || d->total_k > kMaxIndex || d->total_q > kMaxIndex / group) return GEMM_F16_NT_UNSUPPORTED;
    const int64_t seqs = d->batch < d->total_q ? d->batch : d->total_q;
    if (d->total_q * group / kTileRows + seqs > kMaxUnits / d->kv_heads) return GEMM_F16_NT_UNSUPPORTED;
    return GEMM_F16_NT_OK;
}

int check_shared(const attn_shared_prefix_desc* d)
{
    if (d == nullptr) return GEMM_F16_NT_INVALID_ARG;
    const int st = check_common(d->dtype, d->heads, d->kv_heads, d->head_dim, d->scale);
    if (st != GEMM_F16_NT_OK) return st;
    if (d->batch < 0 || d->prefix < 0 || d->slot_rows < 0) return GEMM_F16_NT_INVALID_ARG;
    const int64_t hd = d->head_dim, hk = d->kv_heads;
    const int64_t eq = extent(hd, {{d->batch, d->q_row}, {d->heads, d->q_head}});
    const int64_t eo = extent(hd, {{d->batch, d->o_row}, {d->heads, d->o_head}});
    const int64_t ekp = extent(hd, {{d->prefix, d->kp_row}, {hk, d->kp_head}});
    const int64_t evp = extent(hd, {{d->prefix, d->vp_row}, {hk, d->vp_head}});
    const int64_t eks = extent(hd, {{d->batch, d->ks_slot}, {d->slot_rows, d->ks_row}, {hk, d->ks_head}});
    const int64_t evs = extent(hd, {{d->batch, d->vs_slot}, {d->slot_rows, d->vs_row}, {hk, d->vs_head}});
    if (eq < 0 || eo < 0 || ekp < 0 || evp < 0 || eks < 0 || evs < 0) return GEMM_F16_NT_INVALID_ARG;
    if (d->batch == 0) return GEMM_F16_NT_OK;
    if (d->Q == nullptr || d->O == nullptr || d->lens == nullptr) return GEMM_F16_NT_INVALID_ARG;
    if (d->prefix > 0 && (d->Kp == nullptr || d->Vp == nullptr)) return GEMM_F16_NT_INVALID_ARG;
    if (d->slot_rows > 0 && (d->Ks == nullptr || d->Vs == nullptr)) return GEMM_F16_NT_INVALID_ARG;
    if (!rows_apart(d->batch, d->o_row, d->heads, d->o_head, hd)) return GEMM_F16_NT_INVALID_ARG;
    if (overlaps(d->O, eo, d->Q, eq) || overlaps(d->O, eo, d->Kp, ekp) || overlaps(d->O, eo, d->Vp, evp) ||
        overlaps(d->O, eo, d->Ks, eks) || overlaps(d->O, eo, d->Vs, evs))
        return GEMM_F16_NT_INVALID_ARG;
    const int64_t el = d->lse == nullptr ? 0 : d->batch * d->heads * 4;
    if (overlaps(d->lse, el, d->O, eo) || overlaps(d->lse, el, d->Q, eq) || overlaps(d->lse, el, d->Kp, ekp) ||
        overlaps(d->lse, el, d->Vp, evp) || overlaps(d->lse, el, d->Ks, eks) || overlaps(d->lse, el, d->Vs, evs))
        return GEMM_F16_NT_INVALID_ARG;
    if (!aligned16(d->Q, {d->q_row, d->q_head}) || !aligned16(d->O, {d->o_row, d->o_head}) ||
        !aligned16(d->Kp, {d->kp_row, d->kp_head}) || !aligned16(d->Vp, {d->vp_row, d->vp_head}) ||
        !aligned16(d->Ks, {d->ks_slot, d->ks_row, d->ks_head}) || !aligned16(d->Vs, {d->vs_slot, d->vs_row, d->vs_head}))
        return GEMM_F16_NT_UNSUPPORTED;
    if (((uintptr_t)d->lens | (uintptr_t)d->lse) & 3) return GEMM_F16_NT_UNSUPPORTED;
    if (d->kp_row >= kMaxRowStride || d->vp_row >= kMaxRowStride || d->ks_row >= kMaxRowStride ||
        d->vs_row >= kMaxRowStride)
        return GEMM_F16_NT_UNSUPPORTED;
    if (d->prefix > kMaxIndex || d->slot_rows > kMaxIndex || d->batch > kMaxIndex / d->heads) return GEMM_F16_NT_UNSUPPORTED;
    const int64_t group = d->heads / hk, parts = d->slot_rows / (kMaxBlocks * attn::kBlockKeys) + 1;
    if (ceil_div(d->batch * group, kTileRows) + d->batch * ceil_div(group, attn::kWaveRows) * parts > kMaxUnits / hk)
        return GEMM_F16_NT_UNSUPPORTED;
    return GEMM_F16_NT_OK;
}

// ----------------------------------------------------------------- plans
struct PromptPlan {
    int64_t waves, tiles, splits, part_bytes;
};

// Row tiles of one kv head: a packed batch has at most one ragged tile for
// each sequence (and one sequence no more than its rows fill).  Where all
// tiles of all kv heads leave compute units without work, the keys are split,
// at least 256 of them (of a sequence of the batch's mean length) to a part.
// Splitting uneven batches by the longest sequence they may hold, in parts of
// at least 256, was no faster: the join costs 5 us and the parts' bytes.
//
// Eight waves share a tile of K and V where workgroups are long: they read
// half as many bytes into LDS, but a compute unit then holds one workgroup,
// and nothing runs beside its beginning and end.  Measured on MI355X, eight
// against four: 16384 tokens 1941 against 2007 us, 4096 151 against 160, 512
// against 20000 keys 175 against 185; packed lengths of 333 to 1999 with
// heads of 96 (16 tiles of keys to a workgroup on average) 50.8 against 46.1,
// of 1 to 2900 138.7 against 138.3, heads of 64 elements (three workgroups of
// four waves to a compute unit) 155 against 153.  With one workgroup to a
// compute unit the last round has to be well filled too, 5/6 of all rounds'
// places: 32 query and 8 key/value heads, causal, 3500 tokens (86%) 98 against
// 108 us, 5000 (82%) 202 against 195; without a mask 2048 (100%) 64 against 68,
// 3000 (73%) 156 against 142, 2400 (59%) 128 against 112.
constexpr int64_t kLongTiles = 24;

PromptPlan plan_prompt(const attn_prompt_desc* d, int cus)
{
    PromptPlan p;
    const int64_t group = d->heads / d->kv_heads;
    const int64_t seqs = d->batch < d->total_q ? d->batch : d->total_q;   // with a query
    const int64_t keys = ceil_div(d->total_k, seqs), queries = ceil_div(d->total_q, seqs);
    auto plan = [&](int64_t waves) {
        p.waves = waves;
        const int64_t rows = waves * attn::kWaveRows;
        p.tiles = seqs == 1 ? ceil_div(d->total_q * group, rows) : d->total_q * group / rows + seqs;
        const int64_t wgs = p.tiles * d->kv_heads, slots = waves == attn::kWaves ? 2 * cus : cus;
        int64_t s = wgs >= cus ? 1 : slots / wgs;
        if (s > keys / (4 * kTileKeys)) s = keys / (4 * kTileKeys);
        p.splits = s < 1 ? 1 : s;
    };
    plan(2 * attn::kWaves);
    const int64_t seen = d->causal ? keys - (queries < keys ? queries : keys) / 2 : keys;   // of a row, about
    const int64_t wgs = p.tiles * d->kv_heads * p.splits;
    const bool full = 6 * wgs >= 5 * cus * ceil_div(wgs, cus);
    if (d->head_dim <= 64 || queries * group < 2 * kTileRows || !full || seen < kLongTiles * kTileKeys * p.splits)
        plan(attn::kWaves);
    p.part_bytes = p.splits > 1 ? p.splits * d->total_q * d->heads * (d->head_dim + 2) * 4 : 0;
    return p;
}

// A row's keys come in parts: of the prefix, which row tiles of all slots'
// rows (128, or up to 32 by the few-rows way) run through, and of its own
// slot.  Where that needs no split (splits == 1 below) a slot's rows take a
// short prefix and their own keys as one run instead, without a joining
// launch: 3 x 500 + 64 keys 10.1 against 12.8 us, 32 x 200 + 100 8.6 against
// 14.8, 64 x 500 + 500 20.6 against 22.5; with a split and for longer
// prefixes the other way was faster (8 x 1000 + 300 14.1 against 15.1,
// 4 x 8000 + 100 14.8 against 18.4).  One sequence alone has nobody to share
// with.
constexpr int64_t kMinBlocks = 16;      // of 32 keys, for a part
constexpr int64_t kTogetherBlocks = 16;

// Many short slots: a wave takes one's rows and keys, without the merging of
// four waves, and a quarter of the workgroups find their work.  125 x 32 kv
// heads of 80 with up to 25 own keys behind 1512 shared ones 21.4 against 42.1
// us; with up to 169 (6 blocks) 86.6 against 87.6, with up to 257 (9 blocks)
// 22.2 against 21.1.  Where a short prefix goes with the slot's own keys a
// workgroup's waves have to come in two rounds at least: 128 x 8 kv heads, 100
// and up to 30 keys, 10.6 against 15.0 us, 128 x 32, 200 and up to 25, 31.9
// against 55.2; but 64 x 8, 130 and up to 90, 13.0 against 10.6.
constexpr int64_t kSoloBlocks = 8;

struct SharedPlan {
    bool together;              // prefix and own keys as one run
    int64_t row_tiles;          // of the prefix: batch * group rows in tiles of 128, or of 32 where that is all
    int64_t own_tiles;          // of a slot: group rows in tiles of 32
    int64_t prefix_splits;      // parts of the prefix, or of the one run
    int64_t own_splits;         // parts of a slot, of own_blocks blocks of 32 keys each
    int64_t own_blocks;
    int64_t prefix_wgs, own_wgs, rounds, round_prefix, round_own;   // see shared_kernel
    bool solo;                  // a wave has a slot's part, not a workgroup
    int64_t own_jobs;
    int64_t part_bytes;
};

SharedPlan plan_shared(const attn_shared_prefix_desc* d, int cus)
{
    SharedPlan p = {};
    const int64_t group = d->heads / d->kv_heads, rows = d->batch * group;
    const int64_t prefix_blocks = ceil_div(d->prefix, attn::kBlockKeys), slot_blocks = ceil_div(d->slot_rows, attn::kBlockKeys);
    p.own_tiles = ceil_div(group, attn::kWaveRows);
    const int64_t jobs = d->batch * d->kv_heads * p.own_tiles;
    const int64_t run_want = 2 * cus / jobs, run_most = (prefix_blocks + slot_blocks) / kMinBlocks;
    const int64_t run_splits = run_want < run_most ? run_want : run_most;
    p.together = d->batch == 1 || prefix_blocks == 0 || (run_splits <= 1 && prefix_blocks <= kTogetherBlocks);
    if (p.together) {
        p.prefix_splits = run_splits < 1 ? 1 : run_splits;
        p.own_jobs = jobs * p.prefix_splits;
        p.solo = p.prefix_splits == 1 && prefix_blocks + slot_blocks <= kSoloBlocks && jobs >= 4 * cus;
    } else {
        const bool few = rows <= attn::kWaveRows;
        p.row_tiles = few ? 1 : ceil_div(rows, kTileRows);
        // a part of the prefix in row tiles takes about as long as the slots'
        // own keys do together, at some 0.8 us for 64 keys and 5.5 TB/s, but 4
        // to 16 tiles of keys: fewer parts are joined sooner
        const double own_us = (double)d->batch * d->slot_rows * d->kv_heads * d->head_dim * 4 / 5.5e6;
        const int64_t tiles = own_us < 4 ? 4 : own_us > 16 ? 16 : (int64_t)own_us;
        const int64_t want = ceil_div(2 * cus, p.row_tiles * d->kv_heads), most = ceil_div(prefix_blocks, few ? kMinBlocks : 2 * tiles);
        p.prefix_splits = want < most ? want : most;
        p.prefix_wgs = p.row_tiles * d->kv_heads * p.prefix_splits;
        const int64_t per = ceil_div(slot_blocks, ceil_div(2 * cus, jobs));
        p.own_blocks = per < kMinBlocks ? kMinBlocks : per > kMaxBlocks ? kMaxBlocks : per;
        p.own_splits = ceil_div(slot_blocks, p.own_blocks);
        p.own_jobs = jobs * p.own_splits;
        p.solo = !few && p.own_splits == 1 && slot_blocks <= kSoloBlocks && jobs >= 2 * cus;
    }
    p.own_wgs = p.solo ? ceil_div(p.own_jobs, attn::kWaves) : p.own_jobs;
    p.round_prefix = p.prefix_wgs < cus ? p.prefix_wgs : cus;
    p.rounds = p.prefix_wgs == 0 ? 1 : ceil_div(p.prefix_wgs, p.round_prefix);
    p.round_own = ceil_div(p.own_wgs, p.rounds);
    const int64_t parts = p.prefix_splits + p.own_splits;
    // one run in one part stores its rows itself; a prefix alone (slots without
    // rows) leaves them to the join even then, which knows the slots in use
    p.part_bytes = !p.together || parts > 1 ? parts * d->batch * d->heads * (d->head_dim + 2) * 4 : 0;
    return p;
}

// Parts in a workspace: m and l of every part, then the O's (16-byte aligned).
Parts parts_in(void* ws, int64_t splits, int64_t rows)
{
    Parts p;
    p.ml = (float*)ws;
    p.o = (float*)ws + ceil_div(2 * splits * rows, 4) * 4;
    p.n = rows;
    return p;
}
int64_t parts_total(int64_t part_bytes) { return part_bytes == 0 ? 0 : part_bytes + 16; }

int launch(const void* f, int64_t wgs, int threads, const void* args, hipStream_t s)
{
    void* a[] = {const_cast<void*>(args)};
    return hipLaunchKernel(f, dim3((unsigned)wgs), dim3(threads), a, 0, s) == hipSuccess ? GEMM_F16_NT_OK : GEMM_F16_NT_LAUNCH;
}

// The instantiation for a type and head size.
template <template <typename, int> class K>
const void* pick(int dtype, int64_t d)
{
    if (dtype == ATTN_F16) return d <= 64 ? K<F16, 64>::f() : d <= 96 ? K<F16, 96>::f() : K<F16, 128>::f();
    return d <= 64 ? K<BF16, 64>::f() : d <= 96 ? K<BF16, 96>::f() : K<BF16, 128>::f();
}
template <bool SPLIT>
struct Prompt {
    template <typename T, int D>
    struct Short {
        static const void* f() { return (const void*)&prompt_kernel<T, D, SPLIT, attn::kWaves>; }
    };
    template <typename T, int D>
    struct Long {   // heads of up to 64 elements have no eight-wave form
        static const void* f() { return (const void*)&prompt_kernel<T, D == 64 ? 96 : D, SPLIT, 2 * attn::kWaves>; }
    };
    static const void* f(const attn_prompt_desc* d, int64_t waves)
    {
        return waves == attn::kWaves ? pick<Short>(d->dtype, d->head_dim) : pick<Long>(d->dtype, d->head_dim);
    }
};
template <typename T, int D>
struct SharedParts {
    static const void* f() { return (const void*)&shared_kernel<T, D>; }
};

// The joining kernel: as many groups as leave each at most 4 parts, up to 8,
// since a group reads its parts one after the other.
template <template <typename, int> class K>
const void* pick_join(int dtype, int64_t parts, int64_t* rows)
{
    const int groups = parts <= 4 ? 1 : parts <= 8 ? 2 : parts <= 16 ? 4 : 8;
    *rows = kThreads / 32 / groups;
    if (dtype == ATTN_F16) return groups == 1 ? K<F16, 1>::f() : groups == 2 ? K<F16, 2>::f() : groups == 4 ? K<F16, 4>::f() : K<F16, 8>::f();
    return groups == 1 ? K<BF16, 1>::f() : groups == 2 ? K<BF16, 2>::f() : groups == 4 ? K<BF16, 4>::f() : K<BF16, 8>::f();
}
template <typename T, int GROUPS>
struct PromptJoin {
    static const void* f() { return (const void*)&prompt_join_kernel<T, GROUPS>; }
};
template <typename T, int GROUPS>
struct SharedJoin {
    static const void* f() { return (const void*)&shared_join_kernel<T, GROUPS>; }
};

int check_workspace(const void* ws, int64_t have, int64_t need)
{
    if (need == 0) return GEMM_F16_NT_OK;
    if (ws == nullptr || have < need) return GEMM_F16_NT_INVALID_ARG;
    return ((uintptr_t)ws & 15) != 0 ? GEMM_F16_NT_UNSUPPORTED : GEMM_F16_NT_OK;
}

}  // namespace

extern "C" {

int attn_prompt_check(const attn_prompt_desc* d) { return check_prompt(d); }

int64_t attn_prompt_workspace(const attn_prompt_desc* d)
{
    int st = check_prompt(d);
    if (st != GEMM_F16_NT_OK) return st;
    if (d->total_q == 0 || d->batch == 0) return 0;
    int cus = 0;
    if ((st = device_cus(&cus)) != GEMM_F16_NT_OK) return st;
    return parts_total(plan_prompt(d, cus).part_bytes);
}

int attn_prompt(const attn_prompt_desc* d, void* workspace, int64_t workspace_bytes, void* stream)
{
    int st = check_prompt(d);
    if (st != GEMM_F16_NT_OK || d->total_q == 0 || d->batch == 0) return st;
    int cus = 0;
    if ((st = device_cus(&cus)) != GEMM_F16_NT_OK) return st;
    const PromptPlan p = plan_prompt(d, cus);
    if ((st = check_workspace(workspace, workspace_bytes, parts_total(p.part_bytes))) != GEMM_F16_NT_OK) return st;
    const Scale sc = scale_of(d->scale);
    PromptArgs g;
    g.q = (const char*)d->Q;
    g.k = (const char*)d->K;
    g.v = (const char*)d->V;
    g.o = (char*)d->O;
    g.lse = d->lse;
    g.cu_q = d->cu_q;
    g.cu_k = d->cu_k;
    g.q_row = 2 * d->q_row;
    g.q_head = 2 * d->q_head;
    g.k_row = 2 * d->k_row;
    g.k_head = 2 * d->k_head;
    g.v_row = 2 * d->v_row;
    g.v_head = 2 * d->v_head;
    g.o_row = 2 * d->o_row;
    g.o_head = 2 * d->o_head;
    g.batch = d->batch;
    g.total_q = (int)d->total_q;
    g.total_k = (int)d->total_k;
    g.heads = d->heads;
    g.kv_heads = d->kv_heads;
    g.group = attn::div_by(d->heads / d->kv_heads);
    g.d = d->head_dim;
    g.causal = d->causal;
    g.careful = d->causal != 0 || d->v_row < d->head_dim;
    const int64_t units = d->kv_heads * p.splits;
    g.by_xcd = units % kNumXcd == 0;
    g.units = attn::div_by(g.by_xcd ? units / kNumXcd : units);
    g.splits = attn::div_by(p.splits);
    g.join_kv = attn::div_by(d->kv_heads);
    g.c = sc.c;
    g.slack = sc.slack;
    g.flip = sc.flip;
    g.zero = sc.zero;
    g.parts = parts_in(workspace, p.splits, d->total_q * d->heads);
    const int64_t wgs = p.tiles * units;
    const hipStream_t s = (hipStream_t)stream;
    const int threads = 64 * (int)p.waves;
    if (p.splits == 1) return launch(Prompt<false>::f(d, p.waves), wgs, threads, &g, s);
    if ((st = launch(Prompt<true>::f(d, p.waves), wgs, threads, &g, s)) != GEMM_F16_NT_OK) return st;
    int64_t join_rows = 0;
    const void* join = pick_join<PromptJoin>(d->dtype, p.splits, &join_rows);
    const int64_t seqs = d->batch < d->total_q ? d->batch : d->total_q;
    const int64_t join_tiles = d->total_q * g.group.d / kTileRows + seqs;
    return launch(join, join_tiles * d->kv_heads * (kTileRows / join_rows), kThreads, &g, s);
}

int attn_shared_prefix_check(const attn_shared_prefix_desc* d) { return check_shared(d); }

int64_t attn_shared_prefix_workspace(const attn_shared_prefix_desc* d)
{
    int st = check_shared(d);
    if (st != GEMM_F16_NT_OK) return st;
    if (d->batch == 0) return 0;
    int cus = 0;
    if ((st = device_cus(&cus)) != GEMM_F16_NT_OK) return st;
    return parts_total(plan_shared(d, cus).part_bytes);
}

int attn_shared_prefix(const attn_shared_prefix_desc* d, void* workspace, int64_t workspace_bytes, void* stream)
{
    int st = check_shared(d);
    if (st != GEMM_F16_NT_OK || d->batch == 0) return st;
    int cus = 0;
    if ((st = device_cus(&cus)) != GEMM_F16_NT_OK) return st;
    const SharedPlan p = plan_shared(d, cus);
    if ((st = check_workspace(workspace, workspace_bytes, parts_total(p.part_bytes))) != GEMM_F16_NT_OK) return st;
    const Scale sc = scale_of(d->scale);
    SharedArgs g;
    g.q = (const char*)d->Q;
    g.kp = (const char*)d->Kp;
    g.vp = (const char*)d->Vp;
    g.ks = (const char*)d->Ks;
    g.vs = (const char*)d->Vs;
    g.o = (char*)d->O;
    g.lse = d->lse;
    g.lens = d->lens;
    g.q_row = 2 * d->q_row;
    g.q_head = 2 * d->q_head;
    g.kp_row = 2 * d->kp_row;
    g.kp_head = 2 * d->kp_head;
    g.vp_row = 2 * d->vp_row;
    g.vp_head = 2 * d->vp_head;
    g.ks_slot = 2 * d->ks_slot;
    g.ks_row = 2 * d->ks_row;
    g.ks_head = 2 * d->ks_head;
    g.vs_slot = 2 * d->vs_slot;
    g.vs_row = 2 * d->vs_row;
    g.vs_head = 2 * d->vs_head;
    g.o_row = 2 * d->o_row;
    g.o_head = 2 * d->o_head;
    g.batch = (int)d->batch;
    g.prefix = (int)d->prefix;
    g.slot_rows = (int)d->slot_rows;
    g.heads = d->heads;
    g.d = d->head_dim;
    g.group = attn::div_by(d->heads / d->kv_heads);
    g.kv_heads = attn::div_by(d->kv_heads);
    g.together = (int)p.together;
    g.row_tiles = attn::div_by(p.row_tiles);
    g.own_tiles = attn::div_by(p.own_tiles);
    g.prefix_splits = attn::div_by(p.prefix_splits);
    g.own_splits = attn::div_by(p.own_splits);
    g.parts_of_row = (int)(p.prefix_splits + p.own_splits);
    g.own_blocks = (int)p.own_blocks;
    g.prefix_wgs = (uint32_t)p.prefix_wgs;
    g.own_wgs = (uint32_t)p.own_wgs;
    g.own_jobs = (uint32_t)p.own_jobs;
    g.solo = (int)p.solo;
    g.round_prefix = (uint32_t)p.round_prefix;
    g.round_own = (uint32_t)p.round_own;
    g.round = attn::div_by(p.round_prefix + p.round_own);
    g.by_xcd = d->kv_heads * p.prefix_splits % kNumXcd == 0;
    g.rounded = !p.together && d->batch * (d->heads / d->kv_heads) > attn::kWaveRows;
    g.c = sc.c;
    g.slack = sc.slack;
    g.flip = sc.flip;
    g.zero = sc.zero;
    g.parts = parts_in(workspace, p.prefix_splits + p.own_splits, d->batch * d->heads);
    const int64_t wgs = p.rounds * (p.round_prefix + p.round_own);
    const hipStream_t s = (hipStream_t)stream;
    st = launch(pick<SharedParts>(d->dtype, d->head_dim), wgs, kThreads, &g, s);
    if (st != GEMM_F16_NT_OK || p.part_bytes == 0) return st;
    int64_t join_rows = 0;
    const void* join = pick_join<SharedJoin>(d->dtype, p.prefix_splits + p.own_splits, &join_rows);
    return launch(join, ceil_div(d->batch * d->heads, join_rows), kThreads, &g, s);
}

}  // extern "C"
