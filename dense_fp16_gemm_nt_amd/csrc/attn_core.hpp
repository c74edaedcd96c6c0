// Device building blocks of the attention kernels (gfx950 / CDNA4 only).
//
// One wave owns 32 query rows and walks keys in tiles of 64.  Scores are
// computed transposed, S^T = K Q^T, on the 32x32x16 MFMA: its output puts
// query column l % 32 on lane l, so a lane holds 16 scores of one row for
// each block of 32 keys (the other 16 sit on lane l +- 32), and the row's
// maximum, sum and rescaling need one exchange between two lanes and no
// broadcast.  The same registers, rounded to 16 bits, are the B operand of
// O^T += V^T P^T: the order of keys within a product is free, so P^T's
// accumulator order is taken as the order of the contraction and V^T is read
// to match (ds_read_b64_tr_b16 transposes 4 keys x 16 elements on the way
// out of LDS).  P therefore never passes through LDS.
//
// Softmax runs in base 2: p = 2^(c s - (m - kShift)), c = scale * log2 e,
// with m a running row maximum of c s.  m is raised only where a tile's
// maximum exceeds it by more than kSlack, so most tiles skip the rescaling of
// the accumulator (64 multiplications); p then reaches at most
// 2^(kShift + kSlack) = 2^15, inside fp16.  kShift = 7 keeps weights down to
// 2^-31 of the largest above fp16's smallest subnormal (2^-24).  Numerator
// and denominator carry the same factor.
//
// Rounding: scores, maxima, sums and the output accumulate in fp32.  P is
// rounded once to the operands' 16-bit type because the matrix cores take no
// wider operand at their full rate (relative error at most eps / 2 for each
// weight, as for V itself); the denominator adds the unrounded p.
#pragma once

#include "common.hpp"

namespace g16 {
namespace attn {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kTileKeys = 64;    // keys of one tile
constexpr int kWaveRows = 32;    // query rows of one wave
constexpr int kWaves = 4;        // waves of one workgroup
constexpr int kTileRows = kWaveRows * kWaves;
constexpr int kThreads = 64 * kWaves;
constexpr float kShift = 7.0f;
constexpr float kSlack = 8.0f;
constexpr float kLn2 = 0.693147180559945309f;

struct F16 {
    static __device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
    // two fp32 to fp16, nearest even
    static __device__ __forceinline__ uint32_t pack(float x, float y)
    {
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){x, y}, f16x2));
    }
};

struct BF16 {
    static __device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack(float x, float y)
    {
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){x, y}, bf16x2));
    }
};

// Head sizes are instantiated as 64, 96 and 128; others (multiples of 8)
// run on the next one with zeros in the missing elements.  LDS rows hold 64
// or 128 elements.
template <int D>
struct Shape {
    static_assert(D == 64 || D == 96 || D == 128, "instantiated head sizes");
    static constexpr int CHUNKS = D == 64 ? 8 : 16;      // 16-byte chunks of an LDS row
    static constexpr int PITCH = CHUNKS * 16;            // bytes of an LDS row
    static constexpr int TILE = kTileKeys * PITCH;       // bytes of a K or V tile
    static constexpr int KSTEPS = D / 16;                // products of a score block
    static constexpr int DBLOCKS = D / 32;               // 32-element blocks of the output
    static constexpr int LOADS = TILE / (kThreads * 16); // 16-byte loads of a thread for one tile
    static constexpr int LOAD_ROWS = kThreads / CHUNKS;  // rows that one load of all threads covers
};

// Chunk c of row r of a K tile sits at chunk c ^ swz_k(r): the 32 lanes of a
// fragment read 32 rows at one chunk, and any 16 rows in a row then cover
// all 64 banks (256 bytes: one row of 128 elements or two of 64).
template <int D>
__device__ __forceinline__ int swz_k(int r)
{
    return Shape<D>::CHUNKS == 16 ? (r & 15) : ((r >> 1) & 7);
}
// V tiles are read in 64-byte pieces of 4 + 4 rows (32 elements of 8 keys
// for each transposing read); four neighbouring rows are put into the four
// quarters of the 256-byte bank window.
template <int D>
__device__ __forceinline__ int swz_v(int r)
{
    return Shape<D>::CHUNKS == 16 ? ((r & 3) << 2) : (((r >> 1) & 1) << 2);
}

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float max3(float a, float b, float c) { return __builtin_fmaxf(__builtin_fmaxf(a, b), c); }

// Over lanes l and l ^ 32.
__device__ __forceinline__ float max_halves(float x)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __builtin_fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ __forceinline__ float sum_halves(float x)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}

// What a workgroup computes: kTileRows rows from row0 on of a sequence's
// `rows` = tokens * group rows for one kv head (row r: token r / group, query
// head r % group of the kv head), against keys [64 tile0, 64 tile1).
struct Job {
    const char* q;       // token 0, the kv head's first query head
    const char* k;       // key 0 of the kv head
    const char* v;
    int64_t q_token, q_head, k_row, v_row;   // strides in bytes
    int rows, row0, group;
    int keys;            // keys of the sequence
    int lead;            // causal: row's keys are [0, token + lead + 1); otherwise INT32_MAX
    int tile0, tile1;
    int d;               // head size
    float c;             // |scale| * log2 e
    uint32_t flip;       // sign bits flipped in Q (a negative scale)
    bool zero_q;         // scale = 0: every score is 0
};

// What a lane knows of its row.
struct Row {
    int token, head;     // head within the group
    int limit;           // keys it may read
    bool valid;
};

__device__ __forceinline__ Row row_of(const Job& j, int r)
{
    Row x;
    x.valid = r < j.rows;
    const int rr = x.valid ? r : 0;
    x.token = (int)((uint32_t)rr / (uint32_t)j.group);
    x.head = rr - x.token * j.group;
    // a row that is not there masks nothing; its output is not stored
    const int64_t lim = j.lead == INT32_MAX ? (int64_t)j.keys : (int64_t)x.token + j.lead + 1;
    x.limit = !x.valid ? INT32_MAX : (int)(lim < 0 ? 0 : lim < j.keys ? lim : j.keys);
    return x;
}

// The wave's Q fragments: lane l holds row l % 32, elements 16 s + 8 (l / 32) .. + 7.
template <int D>
__device__ __forceinline__ void load_q(const Job& j, const Row& row, int half, u32x4 (&q)[Shape<D>::KSTEPS])
{
    const char* p = j.q + (int64_t)row.token * j.q_token + (int64_t)row.head * j.q_head;
#pragma unroll
    for (int s = 0; s < Shape<D>::KSTEPS; ++s) {
        const int e = 16 * s + 8 * half;
        u32x4 x = {0, 0, 0, 0};
        if (row.valid && e < j.d && !j.zero_q) {
            x = *reinterpret_cast<const u32x4*>(p + 2 * e);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] ^= j.flip;
        }
        q[s] = x;
    }
}

// 16 bytes a lane from a buffer to LDS, lane i's at dst + 16 i.  Written as
// an instruction of its own, without registers that it could leave in
// flight, because the compiler puts a wait for every outstanding
// builtin load to LDS before each transposing read of LDS; the kernels wait
// for their tiles themselves (vmcnt before the barrier that publishes one).
__device__ __forceinline__ uint32_t lds_address(const char* p) { return (uint32_t)(uintptr_t)(const G16_LDS char*)p; }
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // M0 is written inside, on purpose
__device__ __forceinline__ void load_to_lds(u32x4 rs, uint32_t dst, uint32_t off)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(dst), "v"(off), "s"(rs)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// A thread's part of a tile's loads into LDS: its place in the first
// kThreads * 16 bytes of a tile, as a byte offset from the tile's first row.
// Elements behind the head size lie past the end of every buffer.
template <int D, bool IS_V>
__device__ __forceinline__ uint32_t tile_offset(int64_t row_bytes, int d, int tid)
{
    using S = Shape<D>;
    const int r = tid / S::CHUNKS, pc = tid % S::CHUNKS;
    const int lc = pc ^ (IS_V ? swz_v<D>(r) : swz_k<D>(r));   // both repeat every 16 rows
    return lc * 8 < d ? (uint32_t)r * (uint32_t)row_bytes + (uint32_t)lc * 16u : 0x80000000u;
}

// A tile's loads, by all threads of the workgroup.  The buffer starts at the
// tile's first row and ends with its last one inside the sequence, so rows
// behind it (another sequence's, or stale ones) arrive as zeros whatever
// memory holds; the base moves in 64 bits from tile to tile and offsets stay
// below 2^31 (0x80000000 for what is past the head size).
template <int D>
__device__ __forceinline__ void load_tile(const char* base, int64_t row_bytes, int keys, int tile, int d, uint32_t off,
                                          uint32_t dst)
{
    using S = Shape<D>;
    const int key0 = tile * kTileKeys;
    const int n = keys - key0 < kTileKeys ? keys - key0 : kTileKeys;
    const uint32_t bytes = n > 0 ? (uint32_t)(n - 1) * (uint32_t)row_bytes + 2u * (uint32_t)d : 0u;
    const uint64_t at = (uint64_t)(base + (int64_t)key0 * row_bytes);
    const u32x4 rs = {(uint32_t)at, (uint32_t)(at >> 32) & 0xffffu, bytes, 0x00020000u};
#pragma unroll
    for (int i = 0; i < S::LOADS; ++i)
        load_to_lds(rs, dst + i * (kThreads * 16), off + (uint32_t)(i * S::LOAD_ROWS) * (uint32_t)row_bytes);
}

// A lane's LDS addresses: of the fragments of a K tile's first 32 rows, and of
// the transposing reads of a V tile's first rows.  The steps add constants.
template <int D>
struct Reads {
    uint32_t k[Shape<D>::KSTEPS], v[Shape<D>::DBLOCKS];
};

template <int D>
__device__ __forceinline__ Reads<D> reads_of(uint32_t lds, int lane)
{
    using S = Shape<D>;
    Reads<D> x;
    const int r = lane & 31, half = lane >> 5, i16 = lane & 15;
    const int k = r * S::PITCH + ((half ^ swz_k<D>(r)) << 4);
#pragma unroll
    for (int i = 0; i < S::KSTEPS; ++i) x.k[i] = lds + (k ^ (i << 5));
    const int chunk = (((lane >> 4) & 1) << 1) | ((i16 & 3) >> 1);
    const int v = (4 * half + (i16 >> 2)) * S::PITCH + ((chunk ^ swz_v<D>(i16 >> 2)) << 4) + ((i16 & 1) << 3);
#pragma unroll
    for (int b = 0; b < S::DBLOCKS; ++b) x.v[b] = lds + (v ^ (b << 6));
    return x;
}

// S^T of one tile, whose K rows are at byte `at` of LDS: s[b] holds keys 32 b ..
// of row l % 32.
template <typename T, int D>
__device__ __forceinline__ void scores(const Reads<D>& x, uint32_t at, const u32x4 (&q)[Shape<D>::KSTEPS], f32x16 (&s)[2])
{
    using S = Shape<D>;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        f32x16 acc = {};
#pragma unroll
        for (int i = 0; i < S::KSTEPS; ++i)
            acc = T::mfma(*reinterpret_cast<const G16_LDS u32x4*>(x.k[i] + at + b * 32 * S::PITCH), q[i], acc);
        s[b] = acc;
    }
}

// Scores of keys past a row's limit become -inf, whatever they were.
__device__ __forceinline__ void mask(f32x16 (&s)[2], int limit, int key0, int half)
{
    const int n = limit - key0 - 4 * half;   // of the keys 32 b + 8 (i / 4) + i % 4
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            s[b][i] = (32 * b + 8 * (i / 4) + i % 4) < n ? s[b][i] : -__builtin_inff();
}

// One row's running state: m (base 2), the lane's part of the sum, O^T.
template <int D>
struct State {
    float m, l;
    f32x16 o[Shape<D>::DBLOCKS];
};

template <int D>
__device__ __forceinline__ void init(State<D>& st)
{
    st.m = -__builtin_inff();
    st.l = 0.f;
#pragma unroll
    for (int b = 0; b < Shape<D>::DBLOCKS; ++b) st.o[b] = f32x16{};
}

// The maximum of a row's scores in a tile, in the units of m.
__device__ __forceinline__ float top_score(const f32x16 (&s)[2], float c)
{
    float mx = __builtin_fmaxf(s[0][0], s[1][0]);
#pragma unroll
    for (int i = 1; i < 16; ++i) mx = max3(mx, s[0][i], s[1][i]);
    return max_halves(mx) * c;
}

// Raises a row's maximum where a tile's asks for it, and rescales what was
// summed so far.  Each row goes by its own maximum alone, so a row's bits do
// not depend on the rows that share its wave.
template <int D>
__device__ __forceinline__ void raise(float mx, State<D>& st)
{
    const float m = mx > st.m + kSlack ? mx : st.m;
    const float a = m == st.m ? 1.f : exp2_(st.m - m);
    st.m = m;
    st.l *= a;
#pragma unroll
    for (int b = 0; b < Shape<D>::DBLOCKS; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) st.o[b][i] *= a;
}

// Softmax weights of one tile: P^T as B operands p[kk] of the keys 16 kk ..
// 16 kk + 15, and their sum.
template <typename T, int D>
__device__ __forceinline__ void weights(const f32x16 (&s)[2], float c, State<D>& st, u32x4 (&p)[4])
{
    const float base = st.m == -__builtin_inff() ? 0.f : kShift - st.m;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = exp2_(__builtin_fmaf(s[b][8 * h + i], c, base));
            st.l += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
#pragma unroll
            for (int i = 0; i < 4; ++i) p[2 * b + h][i] = T::pack(e[2 * i], e[2 * i + 1]);
        }
}

// O^T += V^T P^T over one tile, whose V rows are at byte `at` of LDS.
template <typename T, int D>
__device__ __forceinline__ void accumulate(const Reads<D>& x, uint32_t at, const u32x4 (&p)[4], State<D>& st)
{
    using S = Shape<D>;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int b = 0; b < S::DBLOCKS; ++b) {
            const uint32_t a = x.v[b] + at + kk * 16 * S::PITCH;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((G16_LDS s16x4*)a);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((G16_LDS s16x4*)(a + 8 * S::PITCH));
            const u32x2 lo2 = __builtin_bit_cast(u32x2, lo), hi2 = __builtin_bit_cast(u32x2, hi);
            st.o[b] = T::mfma(u32x4{lo2[0], lo2[1], hi2[0], hi2[1]}, p[kk], st.o[b]);
        }
}

// LDS of a workgroup: two K tiles, then two V tiles.
template <int D>
constexpr int lds_bytes()
{
    return 4 * Shape<D>::TILE;
}

// All tiles of a job; the four waves share the K and V tiles.  Tile t + 1 of
// K and t of V are in LDS when iteration t begins; K t + 2 and V t + 1 are
// loaded while it runs.
template <typename T, int D>
__device__ __forceinline__ void run_tiles(const Job& j, const Row& row, char* smem, State<D>& st)
{
    using S = Shape<D>;
    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
    u32x4 q[S::KSTEPS];
    load_q<D>(j, row, half, q);
    init(st);
    if (j.tile0 >= j.tile1) return;
    const int first_limit = __builtin_amdgcn_readfirstlane(row.limit);   // the wave's smallest
    const uint32_t lds = lds_address(smem);
    const Reads<D> x = reads_of<D>(lds, lane);
    const uint32_t koff = tile_offset<D, false>(j.k_row, j.d, tid), voff = tile_offset<D, true>(j.v_row, j.d, tid);
    const uint32_t dst = lds + __builtin_amdgcn_readfirstlane(tid >> 6) * 1024;
    constexpr uint32_t K0 = 0, V0 = 2 * S::TILE;
    auto load_k = [&](int t, uint32_t par) { load_tile<D>(j.k, j.k_row, j.keys, t, j.d, koff, dst + K0 + par * S::TILE); };
    auto load_v = [&](int t, uint32_t par) { load_tile<D>(j.v, j.v_row, j.keys, t, j.d, voff, dst + V0 + par * S::TILE); };
    load_k(j.tile0, 0);
    load_v(j.tile0, 0);
    if (j.tile0 + 1 < j.tile1) load_k(j.tile0 + 1, 1);
    wait_vmcnt<0>();
    wg_barrier();
    f32x16 cur[2], next[2];
    scores<T, D>(x, K0, q, cur);
    auto step = [&](int t, uint32_t par, f32x16 (&a)[2], f32x16 (&b)[2]) {
        // this wave's reads of K t and V t - 1 are done and its loads of
        // K t + 1 and V t have landed; behind the barrier that holds for all
        wait_lgkmcnt0();
        wait_vmcnt<0>();
        wg_barrier();
        if (t + 2 < j.tile1) load_k(t + 2, par);
        if (t + 1 < j.tile1) {
            load_v(t + 1, 1 - par);
            scores<T, D>(x, K0 + (1 - par) * S::TILE, q, b);
        }
        if ((t + 1) * kTileKeys > first_limit) mask(a, row.limit, t * kTileKeys, half);
        const float mx = top_score(a, j.c);
        if (__builtin_amdgcn_ballot_w64(mx > st.m + kSlack) != 0) raise<D>(mx, st);
        u32x4 p[4];
        weights<T, D>(a, j.c, st, p);
        accumulate<T, D>(x, V0 + par * S::TILE, p, st);
    };
    int t = j.tile0;
    for (; t + 1 < j.tile1; t += 2) {
        step(t, 0, cur, next);
        step(t + 1, 1, next, cur);
    }
    if (t < j.tile1) step(t, 0, cur, next);
}

// Partial results of a split job: for row x (of n) and part s, m and l at
// ml[(s n + x) 2] and the unscaled O at o[(s n + x) d].
struct Parts {
    float* ml;
    float* o;
    int64_t n;
};

// The row's O, normalised and rounded, and its log-sum-exp.
template <typename T, int D>
__device__ __forceinline__ void store_row(const State<D>& st, int d, char* o, float* lse, int half)
{
    const float l = sum_halves(st.l);
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int b = 0; b < Shape<D>::DBLOCKS; ++b)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int e = 32 * b + 8 * g + 4 * half;
            if (e < d) {
                u32x2 x;
                x[0] = T::pack(st.o[b][4 * g] * inv, st.o[b][4 * g + 1] * inv);
                x[1] = T::pack(st.o[b][4 * g + 2] * inv, st.o[b][4 * g + 3] * inv);
                *reinterpret_cast<u32x2*>(o + 2 * e) = x;
            }
        }
    if (lse != nullptr && half == 0) *lse = l == 0.f ? -__builtin_inff() : (st.m - kShift + __builtin_log2f(l)) * kLn2;
}

template <int D>
__device__ __forceinline__ void store_part(const State<D>& st, int d, const Parts& w, int part, int64_t x, int half)
{
    const float l = sum_halves(st.l);
    const int64_t at = (int64_t)part * w.n + x;
    if (half == 0) *reinterpret_cast<f32x2*>(w.ml + 2 * at) = f32x2{st.m, l};
    if (l == 0.f) return;   // no key: nothing reads this part's O
    float* o = w.o + at * d;
#pragma unroll
    for (int b = 0; b < Shape<D>::DBLOCKS; ++b)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int e = 32 * b + 8 * g + 4 * half;
            if (e < d)
                *reinterpret_cast<f32x4*>(o + e) =
                    f32x4{st.o[b][4 * g], st.o[b][4 * g + 1], st.o[b][4 * g + 2], st.o[b][4 * g + 3]};
        }
}

// Joins `parts` partial results of row x and stores it; four elements from e on.
template <typename T>
__device__ __forceinline__ void join_row(const Parts& w, int parts, int64_t x, int d, int e, char* o, float* lse)
{
    float m = -__builtin_inff();
    for (int s = 0; s < parts; ++s) m = __builtin_fmaxf(m, w.ml[2 * ((int64_t)s * w.n + x)]);
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    float l = 0.f;
    for (int s = 0; s < parts; ++s) {
        const int64_t at = (int64_t)s * w.n + x;
        const f32x2 ml = *reinterpret_cast<const f32x2*>(w.ml + 2 * at);
        if (ml[1] == 0.f) continue;
        const float f = exp2_(ml[0] - m);
        l += f * ml[1];
        const f32x4 y = *reinterpret_cast<const f32x4*>(w.o + at * d + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += f * y[i];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    u32x2 r;
    r[0] = T::pack(acc[0] * inv, acc[1] * inv);
    r[1] = T::pack(acc[2] * inv, acc[3] * inv);
    *reinterpret_cast<u32x2*>(o + 2 * e) = r;
    if (lse != nullptr && e == 0) *lse = l == 0.f ? -__builtin_inff() : (m - kShift + __builtin_log2f(l)) * kLn2;
}

}  // namespace attn
}  // namespace g16
