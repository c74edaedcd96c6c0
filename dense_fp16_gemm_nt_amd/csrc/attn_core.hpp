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
// Softmax runs in base 2: p = 2^(c (s - m) + kShift), c = scale * log2 e,
// with m a running row maximum of the scores s = q . k.  m is raised only where
// a tile's maximum exceeds it by more than kSlack / c, so most tiles skip the
// rescaling of the accumulator (64 multiplications); p then reaches at most
// 2^(kShift + kSlack).  Numerator and denominator carry the same factor, and the
// type decides on it.  fp16 has little room below 1: kShift = 7 keeps p at 2^15
// or less and weights down to 2^-31 of the largest above the smallest subnormal
// (2^-24).  bf16 has fp32's exponents, and so has O, which is summed before it
// is divided: kShift = -16 keeps p at 2^-8 or less, so that O stays finite for V
// up to the type's largest value as long as a row's weights, the largest as 1,
// add up to 256 or less; and w v has 8 bits or more above fp32's smallest
// subnormal (2^-149) where it is 2^-125 or more.
//
// The exponent is one fused c s + (kShift - c m), whose second part is rounded
// once for a raised m.  That is off by half a step of c m, which for |c m| up to
// kFar is at most 2^-14.  Where a row's maximum is farther from 0 (a step of
// fp32 is 64 at 10^9, and a weight 2^64 times off) its scores are taken as
// s - m first.
//
// Rounding: scores, maxima, sums and the output accumulate in fp32.  P is
// rounded once to the operands' 16-bit type because the matrix cores take no
// wider operand at their full rate (relative error at most eps / 2 for each
// weight, as for V itself); the denominator adds the unrounded p.  Where no
// more than 32 rows meet the keys the matrix cores have time: P goes as two
// operands there, its rounding and the rest.
#pragma once

#include <utility>

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
constexpr float kSlack = 8.0f;
constexpr float kFar = 1024.0f;   // 2^10
constexpr float kLn2 = 0.693147180559945309f;

struct F16 {
    static constexpr float kShift = 7.0f;
    static __device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
    static constexpr uint32_t kInf = 0x7c00, kOne = 0x3c00, k128 = 0x5800, k16384 = 0x7400;
    // two fp32 to fp16, nearest even
    static __device__ __forceinline__ uint32_t pack(float x, float y)
    {
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){x, y}, f16x2));
    }
    static __device__ __forceinline__ f32x2 unpack(uint32_t p)
    {
        return __builtin_convertvector(__builtin_bit_cast(f16x2, p), f32x2);
    }
};

struct BF16 {
    static constexpr float kShift = -16.0f;
    static constexpr uint32_t kInf = 0x7f80, kOne = 0x3f80, k128 = 0x4300, k16384 = 0x4680;
    static __device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack(float x, float y)
    {
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){x, y}, bf16x2));
    }
    static __device__ __forceinline__ f32x2 unpack(uint32_t p)
    {
        return f32x2{__builtin_bit_cast(float, p << 16), __builtin_bit_cast(float, p & 0xffff0000u)};
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

// Division by a number that a launch knows (Granlund and Montgomery, "Division
// by invariant integers using multiplication", PLDI 1994): n / d for n < 2^31
// is the high half of n * mul, shifted.  A division of two registers costs
// some 40 instructions, and a short prompt's workgroup is mostly such work.
struct Div {
    uint32_t d, mul, shift;
    __host__ __device__ __forceinline__ uint32_t of(uint32_t n) const
    {
        return d < 2 ? n : (uint32_t)(((uint64_t)n * mul) >> 32) >> shift;
    }
};

inline Div div_by(int64_t by)
{
    Div x = {(uint32_t)by, 0, 0};
    if (x.d < 2) return x;
    uint32_t bits = 0;
    while ((uint64_t(1) << bits) < x.d) ++bits;   // 2^bits >= d
    x.mul = (uint32_t)((uint64_t(1) << (31 + bits)) / x.d + 1);
    x.shift = bits - 1;
    return x;
}

// What a workgroup computes: rows from row0 on of a sequence's
// `rows` = tokens * group rows for one kv head (row r: token r / group, query
// head r % group of the kv head), against keys [64 tile0, 64 tile1).
struct Job {
    const char* q;       // token 0, the kv head's first query head
    const char* k;       // key 0 of the kv head
    const char* v;
    int64_t q_token, q_head, k_row, v_row;   // strides in bytes
    int rows, row0;
    Div group;
    int keys;            // keys of the sequence
    int lead;            // causal: row's keys are [0, token + lead + 1); otherwise INT32_MAX
    int most;            // keys that the last row may read
    int tile0, tile1;
    int d;               // head size
    float c, slack;      // |scale| * log2 e, and kSlack / c
    uint32_t flip;       // sign bits flipped in Q (a negative scale)
    bool zero;           // scale = 0: every score is 0, so Q and K are taken as zeros
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
    x.token = (int)j.group.of(rr);
    x.head = rr - x.token * (int)j.group.d;
    // a row that is not there masks nothing; its output is not stored
    const int64_t lim = j.lead == INT32_MAX ? (int64_t)j.keys : (int64_t)x.token + j.lead + 1;
    x.limit = !x.valid ? INT32_MAX : (int)(lim < 0 ? 0 : lim < j.keys ? lim : j.keys);
    return x;
}

// The wave's Q fragments: lane l holds row l % 32, elements 16 s + 8 (l / 32)
// .. + 7.  Rows that are not there and elements behind the head size are read
// as ones that are and cleared, so that all loads are in flight together.
template <int D>
__device__ __forceinline__ void load_q(const Job& j, const Row& row, int half, u32x4 (&q)[Shape<D>::KSTEPS])
{
    const char* p = j.q + (int64_t)row.token * j.q_token + (int64_t)row.head * j.q_head;
#pragma unroll
    for (int s = 0; s < Shape<D>::KSTEPS; ++s) {
        const int e = 16 * s + 8 * half;
        q[s] = *reinterpret_cast<const u32x4*>(p + (e < j.d ? 2 * e : 0));
    }
#pragma unroll
    for (int s = 0; s < Shape<D>::KSTEPS; ++s) {
        const uint32_t keep = row.valid && 16 * s + 8 * half < j.d && !j.zero ? 0xffffffffu : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) q[s][i] = (q[s][i] & keep) ^ j.flip;
    }
}

// 16 bytes a lane from a buffer to LDS, lane i's at dst + AT + 16 i.  Written as
// an instruction of its own, without registers that it could leave in
// flight, because the compiler puts a wait for every outstanding
// builtin load to LDS before each transposing read of LDS; the kernels wait
// for their tiles themselves (vmcnt before the barrier that publishes one).
__device__ __forceinline__ uint32_t lds_address(const char* p) { return (uint32_t)(uintptr_t)(const G16_LDS char*)p; }
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // M0 is written inside, on purpose
template <int AT>
__device__ __forceinline__ void load_to_lds(u32x4 rs, uint32_t dst, uint32_t off)
{
    asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(dst), "v"(off), "s"(rs), "n"(AT)
                 : "memory", "m0", "scc");
}
#pragma clang diagnostic pop

// The loads of a K or V tile after tile, by all threads of a workgroup.  The
// buffer starts at a tile's first row and ends with its last one inside the
// sequence, so rows behind it (another sequence's, or stale ones) arrive as
// zeros whatever memory holds, and so do the elements behind the head size,
// whose offset lies past the end of every buffer.  The base moves in 64 bits
// from tile to tile; offsets stay below 2^31.
template <int D, int W>
struct Loader {
    using S = Shape<D>;
    static constexpr int THREADS = 64 * W, LOADS = S::TILE / (THREADS * 16), LOAD_ROWS = THREADS / S::CHUNKS;
    uint32_t off[LOADS];   // a thread's 16 bytes from the tile's first row on
    uint64_t at;              // the next tile
    int left;                 // keys from there on
    uint32_t row_bytes, last; // bytes from a row to the next, and of a row's head

    // The first tile to load; where `zero` all of them arrive as zeros.
    __device__ __forceinline__ void start(const char* base, int64_t pitch, int keys, int tile, int d, int tid, bool v, bool zero)
    {
        const int r = tid / S::CHUNKS, pc = tid % S::CHUNKS;
        const int lc = pc ^ (v ? swz_v<D>(r) : swz_k<D>(r));   // both repeat every 16 rows
        row_bytes = (uint32_t)pitch;
        last = 2u * (uint32_t)d;
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            off[i] = lc * 8 < d ? (uint32_t)(r + i * LOAD_ROWS) * row_bytes + (uint32_t)lc * 16u : 0x80000000u;
        at = (uint64_t)(base + (int64_t)tile * kTileKeys * pitch);
        left = zero ? 0 : keys - tile * kTileKeys;
    }
    template <int... I>
    __device__ __forceinline__ void issue(u32x4 rs, uint32_t dst, std::integer_sequence<int, I...>)
    {
        (load_to_lds<I * THREADS * 16>(rs, dst, off[I]), ...);
    }
    // the next tile into the buffer at dst (the wave's first 1024 bytes of it)
    __device__ __forceinline__ void next(uint32_t dst)
    {
        const int n = left < kTileKeys ? left : kTileKeys;
        const uint32_t bytes = n > 0 ? (uint32_t)(n - 1) * row_bytes + last : 0u;
        issue(u32x4{(uint32_t)at, (uint32_t)(at >> 32) & 0xffffu, bytes, 0x00020000u}, dst,
              std::make_integer_sequence<int, LOADS>());
        at += (uint64_t)kTileKeys * row_bytes;
        left -= kTileKeys;
    }
};

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

// Waits for everything the wave has in flight (loads to LDS, LDS reads) and
// for the other waves: what each of them loaded or wrote is then there for
// all, and what each of them read may be overwritten.
__device__ __forceinline__ void publish()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Waits until at most N of the wave's loads to LDS are in flight and its LDS
// reads are done.
template <int N>
__device__ __forceinline__ void landed()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// S^T of 32 keys, whose K rows are at byte `at` of LDS: keys 8 (i / 4) +
// 4 (l / 32) + i % 4 of row l % 32.
template <typename T, int D>
__device__ __forceinline__ f32x16 scores(const Reads<D>& x, uint32_t at, const u32x4 (&q)[Shape<D>::KSTEPS])
{
    f32x16 acc = {};
#pragma unroll
    for (int i = 0; i < Shape<D>::KSTEPS; ++i)
        acc = T::mfma(*reinterpret_cast<const G16_LDS u32x4*>(x.k[i] + at), q[i], acc);
    return acc;
}

// Scores of all but the first `keys` of 32 keys become -inf, whatever they were.
__device__ __forceinline__ void mask(f32x16& s, int keys, int half)
{
    const int n = keys - 4 * half;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = (8 * (i / 4) + i % 4) < n ? s[i] : -__builtin_inff();
}

// One row's running state: the maximum m of its scores, the score above which
// m is raised, kShift - c m, the lane's part of the sum, O^T.  A row whose m is
// far from 0 has `over` = -inf and `base` = kShift.
template <int D>
struct State {
    float m, over, base, l;
    f32x16 o[Shape<D>::DBLOCKS];
};

template <int D>
__device__ __forceinline__ void init(State<D>& st)
{
    st.m = st.over = -__builtin_inff();
    st.base = 0.f;   // until there is a key every score is -inf
    st.l = 0.f;
#pragma unroll
    for (int b = 0; b < Shape<D>::DBLOCKS; ++b) st.o[b] = f32x16{};
}

// The maximum of a row's scores (of 32 keys for each block).  A tree: a chain would wait for each instruction's result in turn.
template <int N>
__device__ __forceinline__ float top_score(const f32x16 (&s)[N])
{
    float a[5 * N], b = s[0][15];
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int k = 0; k < 5; ++k) a[5 * i + k] = max3(s[i][3 * k], s[i][3 * k + 1], s[i][3 * k + 2]);
        b = i == 0 ? b : __builtin_fmaxf(b, s[i][15]);
    }
    if constexpr (N == 1) {
        b = max3(b, max3(a[0], a[1], a[2]), __builtin_fmaxf(a[3], a[4]));
    } else {
        const float x = max3(a[0], a[1], a[2]), y = max3(a[3], a[4], a[5]), z = max3(a[6], a[7], a[8]);
        b = max3(b, a[9], max3(x, y, z));
    }
    return max_halves(b);
}

// Raises a row's maximum where a tile's asks for it, and rescales what was
// summed so far; the tile's scores of a row far from 0 become s - m.  Each row
// goes by its own maximum alone, so a row's bits do not depend on the rows that
// share its wave.
template <typename T, int D, int N>
__device__ __forceinline__ void raise(const Job& j, float mx, f32x16 (&s)[N], State<D>& st)
{
    const bool up = mx > st.over;
    const float m = up ? __builtin_fmaxf(mx, st.m) : st.m;
    const float a = m == st.m ? 1.f : exp2_((st.m - m) * j.c);
    const bool far = up && !(__builtin_fabsf(m * j.c) <= kFar);   // a row far from 0 has every tile with a key raise it
    if (up) {
        st.over = far ? -__builtin_inff() : m + j.slack;
        st.base = far ? T::kShift : __builtin_fmaf(-m, j.c, T::kShift);
    }
    st.m = m;
    st.l *= a;
    const float off = far ? m : 0.f;
#pragma unroll
    for (int b = 0; b < N; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[b][i] -= off;
#pragma unroll
    for (int b = 0; b < Shape<D>::DBLOCKS; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) st.o[b][i] *= a;
}

// What every tile of keys begins with.
template <typename T, int D, int N>
__device__ __forceinline__ void follow(const Job& j, f32x16 (&s)[N], State<D>& st)
{
    const float mx = top_score(s);
    if (__builtin_amdgcn_ballot_w64(mx > st.over) != 0) raise<T, D>(j, mx, s, st);
}

// Softmax weights of 32 keys: P^T as B operands p[kk] of the keys 16 kk ..
// 16 kk + 15, and their sum (of the weights before their rounding: the
// log-sum-exp has to hold in fp32).  LEAN takes them pair by pair, which costs
// a little time (16384 tokens, d 128: 1924 against 1877 us) and saves some 29
// registers, which lets three waves share a SIMD for d 64 (164 of the 168 that
// they may have; 4096 tokens, 32 heads: 154 against 159 us).
template <typename T, int D, bool LEAN = false>
__device__ __forceinline__ void weights(const f32x16& s, float c, State<D>& st, u32x4 (&p)[2])
{
    auto weight = [&](int i) { return exp2_(__builtin_fmaf(s[i], c, st.base)); };
    if constexpr (LEAN) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = weight(2 * i), y = weight(2 * i + 1);
            p[i / 4][i % 4] = T::pack(x, y);
            st.l += x + y;
            if (i % 2 == 1) asm volatile("" : "+v"(st.l));   // not put off
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = weight(8 * h + i);
            st.l += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
#pragma unroll
            for (int i = 0; i < 4; ++i) p[h][i] = T::pack(e[2 * i], e[2 * i + 1]);
        }
    }
}

// The same weights as two operands each, p[0] and what its rounding left,
// p[1]: for the few rows whose products are not what they wait for.
template <typename T, int D>
__device__ __forceinline__ void weights_whole(const f32x16& s, float c, State<D>& st, u32x4 (&p)[2][2])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = exp2_(__builtin_fmaf(s[2 * i], c, st.base)), y = exp2_(__builtin_fmaf(s[2 * i + 1], c, st.base));
        st.l += x + y;
        const uint32_t r = T::pack(x, y);
        const f32x2 z = T::unpack(r);
        p[0][i / 4][i % 4] = r;
        p[1][i / 4][i % 4] = T::pack(x - z[0], y - z[1]);
    }
}

// The fragment of V^T for keys 16 kk .. and elements 32 b .., whose rows are at
// byte `at` of LDS.
template <int D>
__device__ __forceinline__ u32x4 read_v(const Reads<D>& x, uint32_t at, int kk, int b)
{
    using S = Shape<D>;
    const uint32_t a = x.v[b] + at + kk * 16 * S::PITCH;
    const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((G16_LDS s16x4*)a));
    const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((G16_LDS s16x4*)(a + 8 * S::PITCH)));
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
}

// O^T += V^T P^T over 32 keys, whose V rows are at byte `at` of LDS; P as N
// operands.
template <typename T, int D, int N>
__device__ __forceinline__ void accumulate(const Reads<D>& x, uint32_t at, const u32x4 (&p)[N][2], State<D>& st)
{
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int b = 0; b < Shape<D>::DBLOCKS; ++b) {
            const u32x4 v = read_v<D>(x, at, kk, b);
#pragma unroll
            for (int n = 0; n < N; ++n) st.o[b] = T::mfma(v, p[n][kk], st.o[b]);
        }
}

// A product with V is not blind to a masked key: weight 0 times an infinity is
// NaN.  Keys that no row may read are not loaded, unless V's rows are closer than
// they are long (overlap): rows behind the last then begin before its end.
// Under a causal mask one row of a tile reads a key that another may not.  If
// such a key's V is not finite a sum is spoilt that it has no part in.  Such sums show at the end as O that is
// not finite; the job is then done again, careful: V's finite elements are
// multiplied as ever, and the others are counted for each row over the keys it
// may read (of the first `keys` of the 32), by kind (+inf, -inf, NaN as 1, 128
// and 16384: up to 32 of each stay apart in an fp32 sum), and added as they are.
template <typename T, int D, int N>
__device__ __forceinline__ void accumulate_careful(const Reads<D>& x, uint32_t at, const u32x4 (&p)[N][2], int keys, int half,
                                                   State<D>& st)
{
    u32x4 allowed[2];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int key = 16 * kk + 8 * (i / 2) + 4 * half + 2 * (i % 2);
            allowed[kk][i] = (key < keys ? T::kOne : 0u) | (key + 1 < keys ? T::kOne << 16 : 0u);
        }
#pragma unroll
    for (int b = 0; b < Shape<D>::DBLOCKS; ++b) {
        f32x16 count = {};
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            u32x4 v = read_v<D>(x, at, kk, b), odd = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t h = v[i / 2] >> (16 * (i % 2)) & 0xffffu, size = h & 0x7fffu;
                if (size >= T::kInf) {
                    v[i / 2] &= i % 2 == 0 ? 0xffff0000u : 0x0000ffffu;
                    odd[i / 2] |= (size > T::kInf ? T::k16384 : (h & 0x8000u) != 0 ? T::k128 : T::kOne) << (16 * (i % 2));
                }
            }
#pragma unroll
            for (int n = 0; n < N; ++n) st.o[b] = T::mfma(v, p[n][kk], st.o[b]);
            count = T::mfma(odd, allowed[kk], count);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int n = (int)count[i];
            if ((n & 127) != 0) st.o[b][i] += __builtin_inff();
            if ((n >> 7 & 127) != 0) st.o[b][i] -= __builtin_inff();
            if (n >> 14 != 0) st.o[b][i] = __builtin_nanf("");
        }
    }
}

// Whether V's rows, a stride of bytes apart, are closer than they are long.
__device__ __forceinline__ bool overlap(int64_t v_row, int d) { return v_row < 2 * d; }

// Whether some element of the wave's O is not finite.
template <int D>
__device__ __forceinline__ bool spoilt(const State<D>& st)
{
    float z = 0.f;
#pragma unroll
    for (int b = 0; b < Shape<D>::DBLOCKS; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) z = __builtin_fmaf(st.o[b][i], 0.f, z);
    return __builtin_amdgcn_ballot_w64(!(z == 0.f)) != 0;
}

// LDS of a workgroup: two K and two V tiles, or a K and a V block of 32 keys
// for each wave, or the waves' partial outputs.
constexpr int kMergePad = 4;   // floats between rows, so that 32 rows at one element spread over the banks
template <int D>
constexpr int lds_bytes()
{
    constexpr int tiles = 4 * Shape<D>::TILE, merge = kWaves * kWaveRows * (2 + D + kMergePad) * 4;
    return tiles > merge ? tiles : merge;
}

// ---------------------------------------------------------------- many rows
// All tiles of a job; the four waves share the K and V tiles.  Tile t + 1 of
// K and t of V are in LDS when iteration t begins; K t + 2 and V t + 1 are
// loaded while it runs.
template <typename T, int D, int W>
__device__ __forceinline__ void run_tiles(const Job& j, const Row& row, char* smem, State<D>& st)
{
    using S = Shape<D>;
    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
    init(st);
    if (j.tile0 >= j.tile1) return;
    const int first_limit = __builtin_amdgcn_readfirstlane(row.limit);   // the wave's smallest
    const uint32_t lds = lds_address(smem);
    const Reads<D> x = reads_of<D>(lds, lane);
    const uint32_t dst = lds + __builtin_amdgcn_readfirstlane(tid >> 6) * 1024;
    constexpr uint32_t K0 = 0, V0 = 2 * S::TILE, HALF = S::TILE / 2;
    Loader<D, W> k, v;
    k.start(j.k, j.k_row, j.keys, j.tile0, j.d, tid, false, j.zero);
    v.start(j.v, j.v_row, j.keys, j.tile0, j.d, tid, true, false);
    k.next(dst + K0);
    v.next(dst + V0);
    if (j.tile0 + 1 < j.tile1) k.next(dst + K0 + S::TILE);
    u32x4 q[S::KSTEPS];
    load_q<D>(j, row, half, q);
    publish();
    f32x16 cur[2], next[2];
    cur[0] = scores<T, D>(x, K0, q);
    cur[1] = scores<T, D>(x, K0 + HALF, q);
    auto step = [&](int t, uint32_t par, f32x16 (&a)[2], f32x16 (&b)[2]) {
        // K t + 1 and V t have landed; K t and V t - 1 have been read
        publish();
        if (t + 2 < j.tile1) k.next(dst + K0 + par * S::TILE);
        if (t + 1 < j.tile1) {
            v.next(dst + V0 + (1 - par) * S::TILE);
            b[0] = scores<T, D>(x, K0 + (1 - par) * S::TILE, q);
            b[1] = scores<T, D>(x, K0 + (1 - par) * S::TILE + HALF, q);
        }
        if ((t + 1) * kTileKeys > first_limit) {
            mask(a[0], row.limit - t * kTileKeys, half);
            mask(a[1], row.limit - t * kTileKeys - 32, half);
        }
        follow<T, D>(j, a, st);
        u32x4 p0[1][2], p1[1][2];
        weights<T, D, D == 64>(a[0], j.c, st, p0[0]);
        weights<T, D, D == 64>(a[1], j.c, st, p1[0]);
        accumulate<T, D>(x, V0 + par * S::TILE, p0, st);
        accumulate<T, D>(x, V0 + par * S::TILE + HALF, p1, st);
    };
    int t = j.tile0;
    for (; t + 1 < j.tile1; t += 2) {
        step(t, 0, cur, next);
        step(t + 1, 1, next, cur);
    }
    if (t < j.tile1) step(t, 0, cur, next);
}

// The same for a job whose V is not all finite, one tile after the other;
// begins with what `st` holds.
template <typename T, int D, int W>
__device__ __forceinline__ void run_tiles_careful(const Job& j, const Row& row, char* smem, State<D>& st)
{
    using S = Shape<D>;
    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
    const uint32_t lds = lds_address(smem);
    const Reads<D> x = reads_of<D>(lds, lane);
    const uint32_t dst = lds + __builtin_amdgcn_readfirstlane(tid >> 6) * 1024;
    Loader<D, W> k, v;
    k.start(j.k, j.k_row, j.keys, j.tile0, j.d, tid, false, j.zero);
    v.start(j.v, j.v_row, j.keys, j.tile0, j.d, tid, true, false);
    u32x4 q[S::KSTEPS];
    load_q<D>(j, row, half, q);
    for (int t = j.tile0; t < j.tile1; ++t) {
        publish();
        k.next(dst);
        v.next(dst + S::TILE);
        publish();
        for (int b = 0; b < 2; ++b) {
            const int keys = row.limit - t * kTileKeys - 32 * b;
            f32x16 s[1] = {scores<T, D>(x, b * (S::TILE / 2), q)};
            mask(s[0], keys, half);
            follow<T, D>(j, s, st);
            u32x4 p[1][2];
            weights<T, D>(s[0], j.c, st, p[0]);
            accumulate_careful<T, D>(x, S::TILE + b * (S::TILE / 2), p, keys, half, st);
        }
    }
}

// Whether `x` holds for some wave of the workgroup.
template <int W>
__device__ __forceinline__ bool any_wave(bool x, char* smem)
{
    int* flags = reinterpret_cast<int*>(smem);
    publish();
    if ((threadIdx.x & 63) == 0) flags[threadIdx.x >> 6] = x;
    publish();
    int any = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) any |= flags[i];
    return __builtin_amdgcn_readfirstlane(any) != 0;
}

// ----------------------------------------------------------------- few rows
// Up to 32 rows against many keys: the keys' bytes are the work, so all four
// waves take the same rows and deal blocks of 32 keys among them.  Each wave
// loads its blocks into LDS of its own and waits for its own loads alone, so
// a workgroup keeps 32 to 64 KiB in flight without a barrier in the loop.
// The keys are one run or two, one after the other (a shared prefix and a
// sequence's own keys).
struct Keys {
    const char* k;
    const char* v;
    int64_t k_row, v_row;   // bytes
    int keys;
};
constexpr int kBlockKeys = 32;
__device__ __forceinline__ int key_blocks(int keys) { return (int)(((int64_t)keys + kBlockKeys - 1) / kBlockKeys); }

// Blocks [block0, block1) of the runs' blocks; row.limit counts keys of the
// first run.  P goes as N operands (2: its rounding and the rest).  CAREFUL: as
// run_tiles_careful; without it V's rows may overlap where CLEAR.  DEAL: how
// many waves share the blocks (1: each wave has rows and blocks of its own).
template <typename T, int D, int N, bool CAREFUL = false, bool CLEAR = !CAREFUL, int DEAL = kWaves>
__device__ __forceinline__ void run_blocks(const Job& j, const Keys& one, const Keys& two, int block0, int block1,
                                           const Row& row, char* smem, State<D>& st)
{
    using S = Shape<D>;
    constexpr int ROWS = 64 / S::CHUNKS;        // rows of one load
    constexpr int NL = kBlockKeys / ROWS;       // loads of a block
    constexpr int COLS = S::CHUNKS == 16 ? 4 : 2;   // the swizzle of K differs from load to load, with this period
    constexpr uint32_t HALF = S::TILE / 2;
    const int lane = threadIdx.x & 63, half = lane >> 5, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    init(st);
    int at = DEAL == 1 ? block0 : w < DEAL ? block0 + w : block1;   // a larger workgroup's other waves take none
    if (at >= block1) return;
    const int first_limit = __builtin_amdgcn_readfirstlane(row.limit);
    const int blocks1 = key_blocks(one.keys);
    const uint32_t lds = lds_address(smem) + w * S::TILE;
    const Reads<D> x = reads_of<D>(lds, lane);
    const int r = lane / S::CHUNKS, pc = lane % S::CHUNKS;
    uint32_t kcol[COLS];
#pragma unroll
    for (int i = 0; i < COLS; ++i) {
        const int lc = pc ^ swz_k<D>(r + i * ROWS);
        kcol[i] = lc * 8 < j.d ? lc * 16 : 0x80000000u;
    }
    const int vc = pc ^ swz_v<D>(r);
    const uint32_t vcol = vc * 8 < j.d ? vc * 16 : 0x80000000u;
    // a block past the last is loaded as zeros: the counts of loads in flight stay the same
    auto load = [&](int blk, bool v) {
        const bool second = blk >= blocks1;
        const int key0 = (second ? blk - blocks1 : blk) * kBlockKeys;
        const int keys = second ? two.keys : one.keys;
        const int64_t row_bytes = v ? (second ? two.v_row : one.v_row) : (second ? two.k_row : one.k_row);
        const char* base = v ? (second ? two.v : one.v) : (second ? two.k : one.k);
        const int n = blk >= block1 || (j.zero && !v) ? 0 : keys - key0 < kBlockKeys ? keys - key0 : kBlockKeys;
        const uint32_t bytes = n > 0 ? (uint32_t)(n - 1) * (uint32_t)row_bytes + 2u * (uint32_t)j.d : 0u;
        const uint64_t a = (uint64_t)(base + (int64_t)key0 * row_bytes);
        const u32x4 rs = {(uint32_t)a, (uint32_t)(a >> 32) & 0xffffu, bytes, 0x00020000u};
        const uint32_t off = (uint32_t)r * (uint32_t)row_bytes;
#pragma unroll
        for (int i = 0; i < NL; ++i)
            load_to_lds<0>(rs, lds + (v ? HALF : 0) + i * 1024,
                           off + (uint32_t)(i * ROWS) * (uint32_t)row_bytes + (v ? vcol : kcol[i % COLS]));
    };
    u32x4 q[S::KSTEPS];
    load_q<D>(j, row, half, q);   // ahead of the blocks: the first wait is for these and K
    load(at, false);
    load(at, true);
    for (; at < block1; at += DEAL) {
        landed<NL>();   // K; V may be in flight
        f32x16 s[1] = {scores<T, D>(x, 0, q)};
        landed<NL>();   // K has been read
        load(at + DEAL, false);
        const bool second = at >= blocks1;
        const int key0 = (second ? at - blocks1 : at) * kBlockKeys;
        const int n = (second ? two.keys : one.keys) - key0, lim = row.limit - key0;
        const int readable = second || n < lim ? n : lim;
        if (n < kBlockKeys || (!second && key0 + kBlockKeys > first_limit)) mask(s[0], readable, half);
        follow<T, D>(j, s, st);
        u32x4 p[N][2];
        if constexpr (N == 2)
            weights_whole<T, D>(s[0], j.c, st, p);
        else
            weights<T, D>(s[0], j.c, st, p[0]);
        landed<NL>();   // V; the next K may be in flight
        if (CLEAR && n < kBlockKeys && overlap(second ? two.v_row : one.v_row, j.d))   // each lane what it loaded
            for (int i = r; i < kBlockKeys; i += ROWS)
                if (i >= n) *reinterpret_cast<G16_LDS u32x4*>(lds + HALF + i * S::PITCH + pc * 16) = u32x4{0, 0, 0, 0};
        if constexpr (CAREFUL)
            accumulate_careful<T, D>(x, HALF, p, readable, half, st);
        else
            accumulate<T, D>(x, HALF, p, st);
        landed<NL>();   // V has been read
        load(at + DEAL, true);
    }
}

// Partial results of a split job: for row x (of n) and part s, m (a score) and
// l at ml[(s n + x) 2] and the unscaled O at o[(s n + x) d].
struct Parts {
    float* ml;
    float* o;
    int64_t n;
};

// Four elements of a row's output.
template <typename T>
__device__ __forceinline__ void store4(char* o, int e, f32x4 x)
{
    *reinterpret_cast<u32x2*>(o + 2 * e) = u32x2{T::pack(x[0], x[1]), T::pack(x[2], x[3])};
}
__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }
template <typename T>
__device__ __forceinline__ float lse_of(float m, float l, float c)
{
    return l == 0.f ? -__builtin_inff() : __builtin_fmaf(m, c, __builtin_log2f(l) - T::kShift) * kLn2;
}

// Calls f(e, block, group) for a lane's groups of accumulator registers that
// lie inside the head size; e is group g's first element of the pair (g, g + STEP).
template <int D, int STEP, typename F>
__device__ __forceinline__ void each_group(int d, int half, F f)
{
    auto all = [&](auto whole) {
#pragma unroll
        for (int b = 0; b < Shape<D>::DBLOCKS; ++b)
#pragma unroll
            for (int g = 0; g < 4; g += STEP) {
                const int e = 32 * b + 8 * g + (STEP == 2 ? 8 : 4) * half;
                if (decltype(whole)::value || e < d) f(e, b, g);
            }
    };
    if (d == D)   // the usual case, without a branch for each group
        all(std::true_type());
    else
        all(std::false_type());
}

// The row's O, normalised and rounded, and its log-sum-exp.  Lanes l and
// l + 32 hold the two halves of each 8 elements; they exchange halves of two
// groups, so that each stores 16 bytes.
template <typename T, int D>
__device__ __forceinline__ void store_row(const Job& j, const State<D>& st, bool valid, char* o, float* lse, int half)
{
    const float l = sum_halves(st.l), inv = inverse(l);
    u32x4 x[Shape<D>::DBLOCKS][2];
#pragma unroll
    for (int b = 0; b < Shape<D>::DBLOCKS; ++b)
#pragma unroll
        for (int g = 0; g < 4; g += 2)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const f32x16& y = st.o[b];
                const auto z = __builtin_amdgcn_permlane32_swap(
                    T::pack(y[4 * g + 2 * i] * inv, y[4 * g + 2 * i + 1] * inv),
                    T::pack(y[4 * g + 4 + 2 * i] * inv, y[4 * g + 5 + 2 * i] * inv), false, false);
                x[b][g / 2][i] = z[0];
                x[b][g / 2][i + 2] = z[1];
            }
    if (!valid) return;
    each_group<D, 2>(j.d, half, [&](int e, int b, int g) { *reinterpret_cast<u32x4*>(o + 2 * e) = x[b][g / 2]; });
    if (lse != nullptr && half == 0) *lse = lse_of<T>(st.m, l, j.c);
}

template <int D>
__device__ __forceinline__ void store_part(const State<D>& st, bool valid, int d, const Parts& w, int part, int64_t x, int half)
{
    const float l = sum_halves(st.l);
    if (!valid) return;
    const int64_t at = (int64_t)part * w.n + x;
    if (half == 0) *reinterpret_cast<f32x2*>(w.ml + 2 * at) = f32x2{st.m, l};
    if (l == 0.f) return;   // no key: nothing reads this part's O
    float* o = w.o + at * d;
    each_group<D, 1>(d, half, [&](int e, int b, int g) {
        const f32x16& y = st.o[b];
        *reinterpret_cast<f32x4*>(o + e) = f32x4{y[4 * g], y[4 * g + 1], y[4 * g + 2], y[4 * g + 3]};
    });
}

// Four elements of a row whose sums are complete: the output, or a part.
template <typename T>
__device__ __forceinline__ void store_row4(char* o, float* lse, float c, int e, float m, float l, f32x4 x)
{
    const float inv = inverse(l);
    store4<T>(o, e, f32x4{x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv});
    if (lse != nullptr && e == 0) *lse = lse_of<T>(m, l, c);
}
__device__ __forceinline__ void store_part4(const Parts& w, int part, int64_t row, int d, int e, float m, float l, f32x4 x)
{
    const int64_t at = (int64_t)part * w.n + row;
    if (e == 0) *reinterpret_cast<f32x2*>(w.ml + 2 * at) = f32x2{m, l};
    *reinterpret_cast<f32x4*>(w.o + at * d + e) = x;
}

// Adds up what the four waves hold of the same rows and hands every four
// elements of a row that is there to store(r, e, m, l, o).
template <int D, typename F>
__device__ __forceinline__ void merge_waves(const Job& j, const State<D>& st, bool valid, int rows, char* smem, F store)
{
    constexpr int PITCH = D + kMergePad;
    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, r = lane & 31;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    f32x2* ml = reinterpret_cast<f32x2*>(smem);
    float* o = reinterpret_cast<float*>(smem) + kWaves * kWaveRows * 2;
    // a row's largest m of the waves that saw a key of it
    auto top = [&](int row) {
        float m = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            const f32x2 y = ml[i * kWaveRows + row];
            m = y[1] == 0.f ? m : __builtin_fmaxf(m, y[0]);
        }
        return m;
    };
    const float l = sum_halves(st.l);
    publish();   // the waves are done with their K and V blocks
    if (half == 0 && w < kWaves) ml[w * kWaveRows + r] = f32x2{st.m, l};
    publish();
    if (valid && w < kWaves) {
        const float f = exp2_((st.m - top(r)) * j.c);
        const bool some = l != 0.f;
        float* to = o + (w * kWaveRows + r) * PITCH;
#pragma unroll
        for (int b = 0; b < Shape<D>::DBLOCKS; ++b)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *reinterpret_cast<f32x4*>(to + 32 * b + 8 * g + 4 * half) =
                    some ? f32x4{st.o[b][4 * g] * f, st.o[b][4 * g + 1] * f, st.o[b][4 * g + 2] * f, st.o[b][4 * g + 3] * f}
                         : f32x4{0.f, 0.f, 0.f, 0.f};
    }
    publish();
    for (int i = tid; i < rows * (D / 4); i += blockDim.x) {
        const int row = i / (D / 4), e = i % (D / 4) * 4;
        if (e >= j.d) continue;
        const float m = top(row);
        float sum = 0.f;
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < kWaves; ++k) {
            const f32x2 y = ml[k * kWaveRows + row];
            sum += y[1] == 0.f ? 0.f : exp2_((y[0] - m) * j.c) * y[1];
            const f32x4 z = *reinterpret_cast<const f32x4*>(o + (k * kWaveRows + row) * PITCH + e);
#pragma unroll
            for (int c = 0; c < 4; ++c) x[c] += z[c];
        }
        store(row, e, m, sum, x);
    }
}

// Joins `parts` partial results of row x, four elements from e on: GROUPS
// groups of 32 lanes take every GROUPS-th part, their sums meet in LDS, and
// the first group stores.  All threads of the workgroup call it; `there` says
// whether the lane has a row and elements.
template <typename T, int GROUPS>
__device__ __forceinline__ void join_row(const Parts& w, int parts, bool there, int64_t x, float c, int d, int e, char* o, float* lse)
{
    const int tid = threadIdx.x, grp = (tid >> 5) % GROUPS;
    if (!there) {
        x = 0;
        e = 0;
    }
    float m = -__builtin_inff();
#pragma unroll 4
    for (int s = grp; s < parts; s += GROUPS) {
        const f32x2 ml = *reinterpret_cast<const f32x2*>(w.ml + 2 * ((int64_t)s * w.n + x));
        m = ml[1] == 0.f ? m : __builtin_fmaxf(m, ml[0]);
    }
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    float l = 0.f;
#pragma unroll 4
    for (int s = grp; s < parts; s += GROUPS) {
        const int64_t at = (int64_t)s * w.n + x;
        const f32x2 ml = *reinterpret_cast<const f32x2*>(w.ml + 2 * at);
        const f32x4 y = *reinterpret_cast<const f32x4*>(w.o + at * d + e);
        const bool some = ml[1] != 0.f;   // otherwise O holds whatever was there
        const float f = exp2_((ml[0] - m) * c);
        l += some ? f * ml[1] : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += some ? f * y[i] : 0.f;
    }
    if constexpr (GROUPS > 1) {
        __shared__ f32x4 sums[kThreads];
        __shared__ f32x2 mls[kThreads / 32];
        sums[tid] = acc;
        if ((tid & 31) == 0) mls[tid >> 5] = f32x2{m, l};
        __syncthreads();
        if (grp != 0) return;
        const int first = tid >> 5;
        m = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) m = mls[first + i][1] == 0.f ? m : __builtin_fmaxf(m, mls[first + i][0]);
        acc = f32x4{0.f, 0.f, 0.f, 0.f};
        l = 0.f;
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
            const f32x2 ml = mls[first + i];
            const float f = ml[1] == 0.f ? 0.f : exp2_((ml[0] - m) * c);
            l += f * ml[1];
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[k] += f * sums[tid + 32 * i][k];
        }
    }
    if (there) store_row4<T>(o, lse, c, e, m, l, acc);
}

}  // namespace attn
}  // namespace g16
