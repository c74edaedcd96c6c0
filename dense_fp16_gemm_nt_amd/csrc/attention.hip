// C-ABI boundary and kernels of the attention operators: argument validation
// (before any HIP call), device checks, split plans and launches.  The
// contract of every entry point is in include/attention.h, the shared device
// code in attn_core.hpp.
#include "attention.h"

#include <hip/hip_runtime.h>

#include <atomic>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstring>

#include "attn_core.hpp"
#include "sched.hpp"
#ifndef NOFEW
#define NOFEW 0
#endif

using namespace g16;

namespace {

using attn::BF16;
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
    int batch, total_q, total_k, heads, kv_heads, group, d, causal;
    int tiles;    // row tiles of one kv head, at most
    int splits;
    float c;
    uint32_t flip;
    int zero_q;
    Parts parts;
};

// A row tile of the packed batch: sequence bounds and the tile's first row.
struct Tile {
    int q0, nq, k0, nk, row0;
    bool found;
};

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

// Tile `t` of the sequences' tiles put one after the other.  Each lane looks
// at one sequence, 64 at a time; offsets are clamped to the tensors, so that
// a table that decreases or runs past them still names rows that exist.
// Within a sequence the tiles come in falling order: under a causal mask
// those have the most keys, and the longest work starts first.
__device__ __forceinline__ Tile find_tile(const PromptArgs& g, int t)
{
    const int lane = threadIdx.x & 63;
    Tile r;
    r.found = false;
    r.q0 = r.nq = r.k0 = r.nk = r.row0 = 0;
    int64_t before = 0;
    for (int base = 0; base < g.batch; base += 64) {
        const int b = base + lane;
        int q0 = 0, q1 = 0;
        if (b < g.batch) {
            q0 = clampi(g.cu_q[b], 0, g.total_q);
            q1 = clampi(g.cu_q[b + 1], q0, g.total_q);
        }
        const int mine = (int)(((int64_t)(q1 - q0) * g.group + kTileRows - 1) / kTileRows);
        int64_t upto = mine;
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) {
            const int64_t y = __shfl_up(upto, s);
            if (lane >= s) upto += y;
        }
        const uint64_t past = __builtin_amdgcn_ballot_w64(before + upto > t);
        if (past != 0) {
            const int w = __builtin_ctzll(past);
            r.found = true;
            r.q0 = __builtin_amdgcn_readlane(q0, w);
            r.nq = __builtin_amdgcn_readlane(q1, w) - r.q0;
            const int n = __builtin_amdgcn_readlane(mine, w);
            const int64_t end = before + __shfl(upto, w);
            r.row0 = __builtin_amdgcn_readfirstlane((int)(end - 1 - t)) * kTileRows;
            (void)n;
            const int sb = base + w;
            r.k0 = clampi(g.cu_k[sb], 0, g.total_k);
            r.nk = clampi(g.cu_k[sb + 1], r.k0, g.total_k) - r.k0;
            return r;
        }
        before += __shfl(upto, 63);
    }
    return r;
}

__device__ __forceinline__ Job prompt_job(const PromptArgs& g, const Tile& t, int kv, int split)
{
    Job j;
    j.q = g.q + (int64_t)t.q0 * g.q_row + (int64_t)kv * g.group * g.q_head;
    j.k = g.k + (int64_t)t.k0 * g.k_row + (int64_t)kv * g.k_head;
    j.v = g.v + (int64_t)t.k0 * g.v_row + (int64_t)kv * g.v_head;
    j.q_token = g.q_row;
    j.q_head = g.q_head;
    j.k_row = g.k_row;
    j.v_row = g.v_row;
    j.rows = t.nq * g.group;
    j.row0 = t.row0;
    j.group = g.group;
    j.keys = t.nk;
    j.lead = g.causal ? t.nk - t.nq : INT32_MAX;
    j.d = g.d;
    j.c = g.c;
    j.flip = g.flip;
    j.zero_q = g.zero_q != 0;
    int most = t.nk;
    if (g.causal) {
        const int last = (t.row0 + kTileRows < j.rows ? t.row0 + kTileRows : j.rows) - 1;
        const int lim = last / g.group + j.lead + 1;
        most = lim < 0 ? 0 : lim < t.nk ? lim : t.nk;
    }
    j.most = most;
    const int n = (most + kTileKeys - 1) / kTileKeys;
    j.tile0 = (int)((int64_t)n * split / g.splits);
    j.tile1 = (int)((int64_t)n * (split + 1) / g.splits);
    return j;
}

#ifndef W64
#define W64 2
#endif
template <typename T, int D, bool SPLIT>
__global__ __launch_bounds__(kThreads, D == 64 ? W64 : 2) void prompt_kernel(const PromptArgs g)
{
    __shared__ __attribute__((aligned(256))) char smem[attn::lds_bytes<D>()];
    // a unit is a kv head and a split; consecutive workgroups go to the XCDs
    // in turn, and each XCD keeps to its own units, whose keys its L2 then
    // holds, with the tiles of the most keys first
    const uint32_t units = (uint32_t)g.kv_heads * (uint32_t)g.splits;
    uint32_t unit, t;
    if (units % kNumXcd == 0) {
        const uint32_t per = units / kNumXcd, i = blockIdx.x / kNumXcd;
        unit = blockIdx.x % kNumXcd * per + i % per;
        t = i / per;
    } else {
        unit = blockIdx.x % units;
        t = blockIdx.x / units;
    }
    const int kv = (int)(unit / (uint32_t)g.splits), split = (int)(unit % (uint32_t)g.splits);
    const Tile tile = find_tile(g, (int)t);
    if (!tile.found) return;
    const Job j = prompt_job(g, tile, kv, split);
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    State<D> st;
    const int rows = j.rows - j.row0;
    if (!NOFEW && rows <= attn::kWaveRows) {
        // the rows of one wave (a single token, a short chunk): all waves
        // take them and divide the keys
        const Row row = attn::row_of(j, j.row0 + (lane & 31));
        const Keys keys = {j.k, j.v, j.k_row, j.v_row, j.keys}, none = {};
        const int n = attn::key_blocks(j.most);
        attn::run_blocks<T, D>(j, keys, none, (int)((int64_t)n * split / g.splits), (int)((int64_t)n * (split + 1) / g.splits),
                               row, smem, st);
        attn::merge_waves<D>(st, row.valid, rows, g.d, smem, [&](int r, int e, float m, float l, f32x4 o) {
            const int x = j.row0 + r;
            const int64_t token = (int64_t)tile.q0 + x / g.group;
            const int head = kv * g.group + x % g.group;
            if constexpr (SPLIT)
                attn::store_part4(g.parts, split, token * g.heads + head, g.d, e, m, l, o);
            else
                attn::store_row4<T>(g.o + token * g.o_row + head * g.o_head,
                                    g.lse == nullptr ? nullptr : g.lse + token * g.heads + head, e, m, l, o);
        });
        return;
    }
    const Row row = attn::row_of(j, j.row0 + w * attn::kWaveRows + (lane & 31));
    attn::run_tiles<T, D>(j, row, smem, st);
    if (!row.valid) return;
    const int64_t token = (int64_t)tile.q0 + row.token;
    const int head = kv * g.group + row.head;
    if constexpr (SPLIT)
        attn::store_part<D>(st, g.d, g.parts, split, token * g.heads + head, half);
    else
        attn::store_row<T, D>(st, g.d, g.o + token * g.o_row + head * g.o_head,
                              g.lse == nullptr ? nullptr : g.lse + token * g.heads + head, half);
}

// Joins the splits: 32 lanes of 4 elements and GROUPS groups of parts for a row.
template <int GROUPS>
constexpr int kJoinRows = kThreads / 32 / GROUPS;

template <typename T, int GROUPS>
__global__ __launch_bounds__(kThreads) void prompt_join_kernel(const PromptArgs g)
{
    constexpr uint32_t kSub = kTileRows / kJoinRows<GROUPS>;
    const uint32_t sub = blockIdx.x % kSub, x = blockIdx.x / kSub;
    const int kv = (int)(x % (uint32_t)g.kv_heads);
    const Tile tile = find_tile(g, (int)(x / (uint32_t)g.kv_heads));
    if (!tile.found) return;
    const int r = tile.row0 + (int)sub * kJoinRows<GROUPS> + (int)(threadIdx.x >> 5) / GROUPS, e = (threadIdx.x & 31) * 4;
    const bool there = r < tile.nq * g.group && e < g.d;
    const int64_t token = (int64_t)tile.q0 + r / g.group;
    const int head = kv * g.group + r % g.group;
    attn::join_row<T, GROUPS>(g.parts, g.splits, there, token * g.heads + head, g.d, e,
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
    int batch, prefix, slot_rows, heads, kv_heads, group, d;
    int together;         // each slot's rows take prefix and own keys as one run (splits: prefix_splits)
    int row_tiles;        // of the prefix: batch * group rows in tiles of 128, or of 32 where that is all
    int own_tiles;        // of a slot: group rows in tiles of 32
    int prefix_splits;    // parts of a row that come from the prefix ...
    int own_splits;       // ... and from its own keys,
    int own_blocks;       // this many blocks of 32 keys each
    uint32_t prefix_wgs, own_wgs, round_prefix, round_own;
    float c;
    uint32_t flip;
    int zero_q;
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
    const uint32_t round = i / (g.round_prefix + g.round_own);
    i -= round * (g.round_prefix + g.round_own);
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
    j.flip = g.flip;
    j.zero_q = g.zero_q != 0;
    State<D> st;
    if (!own) {
        const uint32_t units = (uint32_t)g.kv_heads * (uint32_t)g.prefix_splits, tiles = (uint32_t)g.row_tiles;
        uint32_t unit, t;
        if (units % kNumXcd == 0) {   // the row tiles of a unit one after the other on one XCD: its L2 holds their keys
            unit = i / kNumXcd / tiles * kNumXcd + i % kNumXcd;
            t = i / kNumXcd % tiles;
        } else {
            unit = i / tiles;
            t = i % tiles;
        }
        const int kv = (int)(unit / (uint32_t)g.prefix_splits), part = (int)(unit % (uint32_t)g.prefix_splits);
        j.q = g.q + (int64_t)kv * g.group * g.q_head;
        j.k = g.kp + kv * g.kp_head;
        j.v = g.vp + kv * g.vp_head;
        j.k_row = g.kp_row;
        j.v_row = g.vp_row;
        j.rows = g.batch * g.group;
        j.row0 = (int)t * kTileRows;
        j.keys = g.prefix;
        if (j.rows <= attn::kWaveRows) {
            const Row row = attn::row_of(j, lane & 31);
            const Keys keys = {j.k, j.v, j.k_row, j.v_row, j.keys}, none = {};
            const int n = attn::key_blocks(g.prefix);
            attn::run_blocks<T, D>(j, keys, none, (int)((int64_t)n * part / g.prefix_splits),
                                   (int)((int64_t)n * (part + 1) / g.prefix_splits), row, smem, st);
            attn::merge_waves<D>(st, row.valid, j.rows, g.d, smem, [&](int r, int e, float m, float l, f32x4 o) {
                const int64_t x = (int64_t)(r / g.group) * g.heads + kv * g.group + r % g.group;
                attn::store_part4(g.parts, part, x, g.d, e, m, l, o);
            });
            return;
        }
        const int n = (int)(((int64_t)g.prefix + kTileKeys - 1) / kTileKeys);
        j.tile0 = (int)((int64_t)n * part / g.prefix_splits);
        j.tile1 = (int)((int64_t)n * (part + 1) / g.prefix_splits);
        const Row row = attn::row_of(j, j.row0 + w * attn::kWaveRows + (lane & 31));
        attn::run_tiles<T, D>(j, row, smem, st);
        if (row.valid) attn::store_part<D>(st, g.d, g.parts, part, (int64_t)row.token * g.heads + kv * g.group + row.head, half);
        return;
    }
    const int kv = (int)(i % (uint32_t)g.kv_heads);
    i /= (uint32_t)g.kv_heads;
    const uint32_t splits = (uint32_t)(g.together ? g.prefix_splits : g.own_splits);
    const int split = (int)(i % splits);
    i /= splits;
    j.row0 = (int)(i % (uint32_t)g.own_tiles) * attn::kWaveRows;
    const int64_t slot = i / (uint32_t)g.own_tiles;
    const int len = g.lens[slot];
    if (len < 0) return;
    const Keys mine = {g.ks + slot * g.ks_slot + kv * g.ks_head, g.vs + slot * g.vs_slot + kv * g.vs_head, g.ks_row, g.vs_row,
                       len < g.slot_rows ? len : g.slot_rows};
    const Keys before = {g.kp + kv * g.kp_head, g.vp + kv * g.vp_head, g.kp_row, g.vp_row, g.together ? g.prefix : 0};
    j.q = g.q + slot * g.q_row + (int64_t)kv * g.group * g.q_head;
    j.rows = g.group;
    j.keys = INT32_MAX;   // the runs end themselves
    const int rows = g.group - j.row0 < attn::kWaveRows ? g.group - j.row0 : attn::kWaveRows;
    const int own_n = attn::key_blocks(mine.keys);
    const int64_t x0 = slot * g.heads + kv * g.group + j.row0;
    int part = split, block0, block1;
    if (g.together) {
        const int n = attn::key_blocks(g.prefix) + own_n;
        block0 = (int)((int64_t)n * split / splits);
        block1 = (int)((int64_t)n * (split + 1) / splits);
    } else {
        part += g.prefix_splits;
        block0 = split * g.own_blocks;
        block1 = block0 + g.own_blocks < own_n ? block0 + g.own_blocks : own_n;
        if (block0 >= block1) {   // the slot is not that long
            if ((int)threadIdx.x < rows)
                *reinterpret_cast<f32x2*>(g.parts.ml + 2 * (part * g.parts.n + x0 + threadIdx.x)) =
                    f32x2{-__builtin_inff(), 0.f};
            return;
        }
    }
    const Row row = attn::row_of(j, j.row0 + (lane & 31));
    attn::run_blocks<T, D>(j, before, mine, block0, block1, row, smem, st);
    attn::merge_waves<D>(st, row.valid, rows, g.d, smem, [&](int r, int e, float m, float l, f32x4 o) {
        if (g.prefix_splits + g.own_splits == 1)
            attn::store_row4<T>(g.o + slot * g.o_row + (int64_t)(kv * g.group + j.row0 + r) * g.o_head,
                                g.lse == nullptr ? nullptr : g.lse + x0 + r, e, m, l, o);
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
    attn::join_row<T, GROUPS>(g.parts, g.prefix_splits + g.own_splits, there, x, g.d, e, g.o + b * g.o_row + head * g.o_head,
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
    float c;
    uint32_t flip;
    int zero;
};

// scores = c * (q . k) in base 2 with c > 0: a negative scale flips Q's sign
// bits, which is exact; for scale 0 (or a c below fp32's normal numbers) every
// score is 0.
Scale scale_of(float scale)
{
    const float c = std::fabs(scale) * 1.4426950408889634f;
    if (c < FLT_MIN) return {1.f, 0u, 1};
    return {c, scale < 0.f ? 0x80008000u : 0u, 0};
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
    if (overlaps(d->O, eo, d->Q, eq) || overlaps(d->O, eo, d->K, ek) || overlaps(d->O, eo, d->V, ev))
        return GEMM_F16_NT_INVALID_ARG;
    if (!aligned16(d->Q, {d->q_row, d->q_head}) || !aligned16(d->O, {d->o_row, d->o_head}) ||
        !aligned16(d->K, {d->k_row, d->k_head}) || !aligned16(d->V, {d->v_row, d->v_head}))
        return GEMM_F16_NT_UNSUPPORTED;
    if (((uintptr_t)d->cu_q | (uintptr_t)d->cu_k | (uintptr_t)d->lse) & 3) return GEMM_F16_NT_UNSUPPORTED;
    if (d->k_row >= kMaxRowStride || d->v_row >= kMaxRowStride) return GEMM_F16_NT_UNSUPPORTED;
    const int64_t group = d->heads / d->kv_heads;
    if (d->total_k > kMaxIndex || d->total_q > kMaxIndex / group) return GEMM_F16_NT_UNSUPPORTED;
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
    if (!aligned16(d->Q, {d->q_row, d->q_head}) || !aligned16(d->O, {d->o_row, d->o_head}) ||
        !aligned16(d->Kp, {d->kp_row, d->kp_head}) || !aligned16(d->Vp, {d->vp_row, d->vp_head}) ||
        !aligned16(d->Ks, {d->ks_slot, d->ks_row, d->ks_head}) || !aligned16(d->Vs, {d->vs_slot, d->vs_row, d->vs_head}))
        return GEMM_F16_NT_UNSUPPORTED;
    if (((uintptr_t)d->lens | (uintptr_t)d->lse) & 3) return GEMM_F16_NT_UNSUPPORTED;
    if (d->kp_row >= kMaxRowStride || d->vp_row >= kMaxRowStride || d->ks_row >= kMaxRowStride ||
        d->vs_row >= kMaxRowStride)
        return GEMM_F16_NT_UNSUPPORTED;
    if (d->prefix > kMaxIndex || d->slot_rows > kMaxIndex || d->batch > kMaxIndex / d->heads) return GEMM_F16_NT_UNSUPPORTED;
    return GEMM_F16_NT_OK;
}

// ----------------------------------------------------------------- plans
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

#ifndef PT
#define PT 32
#endif
#ifndef MINB
#define MINB 16
#define MAXB 64
#define TB 32
#define TN 8
#endif
constexpr int64_t kMinBlocks = MINB;
constexpr int64_t kMaxBlocks = MAXB;
constexpr int64_t kTogetherBlocks = TB, kTogetherBatch = TN;

struct PromptPlan {
    int64_t tiles, splits, part_bytes;
};

// Row tiles of one kv head: a packed batch has at most one ragged tile for
// each sequence.  Where all tiles of all kv heads leave compute units without
// work, the keys are split.
PromptPlan plan_prompt(const attn_prompt_desc* d, int cus)
{
    PromptPlan p;
    const int64_t group = d->heads / d->kv_heads;
    const int64_t seqs = d->batch < d->total_q ? d->batch : d->total_q;   // with a query
    p.tiles = d->total_q * group / kTileRows + seqs;
    const int64_t blocks = p.tiles * d->kv_heads;
    const int64_t key_tiles = ceil_div(ceil_div(d->total_k, seqs), kTileKeys);
    int64_t s = blocks >= cus ? 1 : 2 * cus / blocks;
    if (s > key_tiles / 4) s = key_tiles / 4;
    p.splits = s < 1 ? 1 : s;
    p.part_bytes = p.splits > 1 ? p.splits * d->total_q * d->heads * (d->head_dim + 2) * 4 : 0;
    return p;
}

struct SharedPlan {
    int64_t together, row_tiles, own_tiles, prefix_splits, own_splits, own_blocks, prefix_wgs, own_wgs, rounds, round_prefix, round_own,
        part_bytes;
};

SharedPlan plan_shared(const attn_shared_prefix_desc* d, int cus)
{
    SharedPlan p = {};
    const int64_t group = d->heads / d->kv_heads, rows = d->batch * group;
    const int64_t prefix_blocks = ceil_div(d->prefix, attn::kBlockKeys), slot_blocks = ceil_div(d->slot_rows, attn::kBlockKeys);
    p.own_tiles = ceil_div(group, attn::kWaveRows);
    const int64_t jobs = d->batch * d->kv_heads * p.own_tiles;
    p.together = d->batch == 1 || prefix_blocks == 0 || (prefix_blocks <= kTogetherBlocks && d->batch <= kTogetherBatch);
    if (p.together) {
        const int64_t n = prefix_blocks + slot_blocks, most = n / kMinBlocks;
        const int64_t want = 2 * cus / jobs;
        p.prefix_splits = want < most ? want : most;
        if (p.prefix_splits < 1) p.prefix_splits = 1;
        p.own_wgs = jobs * p.prefix_splits;
    } else {
        const bool few = rows <= attn::kWaveRows;
        p.row_tiles = few ? 1 : ceil_div(rows, kTileRows);
        const int64_t want = ceil_div(2 * cus, p.row_tiles * d->kv_heads), most = ceil_div(prefix_blocks, few ? kMinBlocks : PT);
        p.prefix_splits = want < most ? want : most;
        p.prefix_wgs = p.row_tiles * d->kv_heads * p.prefix_splits;
        const int64_t own_want = ceil_div(2 * cus, jobs);
        int64_t per = ceil_div(slot_blocks, own_want);   // blocks of a part
        per = per < kMinBlocks ? kMinBlocks : per > kMaxBlocks ? kMaxBlocks : per;
        p.own_blocks = per;
        p.own_splits = ceil_div(slot_blocks, per);
        p.own_wgs = jobs * p.own_splits;
    }
    p.round_prefix = p.prefix_wgs < cus ? p.prefix_wgs : cus;
    p.rounds = p.prefix_wgs == 0 ? 1 : ceil_div(p.prefix_wgs, p.round_prefix);
    p.round_own = ceil_div(p.own_wgs, p.rounds);
    const int64_t parts = p.prefix_splits + p.own_splits;
    p.part_bytes = parts > 1 ? parts * d->batch * d->heads * (d->head_dim + 2) * 4 : 0;
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

int launch(const void* f, int64_t blocks, const void* args, hipStream_t s)
{
    void* a[] = {const_cast<void*>(args)};
    return hipLaunchKernel(f, dim3((unsigned)blocks), dim3(kThreads), a, 0, s) == hipSuccess ? GEMM_F16_NT_OK : GEMM_F16_NT_LAUNCH;
}

// The instantiation for a type and head size.
template <template <typename, int> class K>
const void* pick(int dtype, int64_t d)
{
    if (dtype == ATTN_F16) return d <= 64 ? K<F16, 64>::f() : d <= 96 ? K<F16, 96>::f() : K<F16, 128>::f();
    return d <= 64 ? K<BF16, 64>::f() : d <= 96 ? K<BF16, 96>::f() : K<BF16, 128>::f();
}
template <typename T, int D>
struct PromptWhole {
    static const void* f() { return (const void*)&prompt_kernel<T, D, false>; }
};
template <typename T, int D>
struct PromptSplit {
    static const void* f() { return (const void*)&prompt_kernel<T, D, true>; }
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
    g.group = d->heads / d->kv_heads;
    g.d = d->head_dim;
    g.causal = d->causal;
    g.tiles = (int)p.tiles;
    g.splits = (int)p.splits;
    g.c = sc.c;
    g.flip = sc.flip;
    g.zero_q = sc.zero;
    g.parts = parts_in(workspace, p.splits, d->total_q * d->heads);
    const int64_t blocks = p.tiles * d->kv_heads * p.splits;
    int64_t join_rows = 0;
    const void* join = pick_join<PromptJoin>(d->dtype, p.splits, &join_rows);
    const int64_t join_wgs = p.tiles * d->kv_heads * (kTileRows / join_rows);
    if (blocks > INT_MAX || (p.splits > 1 && join_wgs > INT_MAX)) return GEMM_F16_NT_UNSUPPORTED;
    const hipStream_t s = (hipStream_t)stream;
    if (p.splits == 1) return launch(pick<PromptWhole>(d->dtype, d->head_dim), blocks, &g, s);
    if ((st = launch(pick<PromptSplit>(d->dtype, d->head_dim), blocks, &g, s)) != GEMM_F16_NT_OK) return st;
    return launch(join, join_wgs, &g, s);
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
    g.kv_heads = d->kv_heads;
    g.group = d->heads / d->kv_heads;
    g.d = d->head_dim;
    g.together = (int)p.together;
    g.row_tiles = (int)p.row_tiles;
    g.own_tiles = (int)p.own_tiles;
    g.prefix_splits = (int)p.prefix_splits;
    g.own_splits = (int)p.own_splits;
    g.own_blocks = (int)p.own_blocks;
    g.prefix_wgs = (uint32_t)p.prefix_wgs;
    g.own_wgs = (uint32_t)p.own_wgs;
    g.round_prefix = (uint32_t)p.round_prefix;
    g.round_own = (uint32_t)p.round_own;
    g.c = sc.c;
    g.flip = sc.flip;
    g.zero_q = sc.zero;
    g.parts = parts_in(workspace, p.prefix_splits + p.own_splits, d->batch * d->heads);
    const int64_t blocks = p.rounds * (p.round_prefix + p.round_own);
    if (blocks > INT_MAX) return GEMM_F16_NT_UNSUPPORTED;
    const hipStream_t s = (hipStream_t)stream;
    st = launch(pick<SharedParts>(d->dtype, d->head_dim), blocks, &g, s);
    if (st != GEMM_F16_NT_OK || p.part_bytes == 0) return st;
    int64_t join_rows = 0;
    const void* join = pick_join<SharedJoin>(d->dtype, p.prefix_splits + p.own_splits, &join_rows);
    return launch(join, ceil_div(d->batch * d->heads, join_rows), &g, s);
}

}  // extern "C"
