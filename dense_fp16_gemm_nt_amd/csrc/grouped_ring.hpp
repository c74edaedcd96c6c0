// The grouped products' large tiles: 256 x 256 outputs by four waves, whose k
// loop is one inline-assembly block (gen_grouped_sched.py, which describes it).
// This file supplies the block's operands and the walk over the tiles.
//
// One wave to a SIMD with a 128 x 128 accumulator reads two thirds of the LDS
// bytes of the eight-wave tile for the same products.  A workgroup for each
// compute unit walks the tiles, since starting one costs some 2 us.
//
// Takes: N and K of 256 or more (tiles at the end of a side of columns move
// back and overlap their neighbour, which computes the same values), at least
// two steps of the contraction by rows, row pitches under 2^21 elements, and
// extents along a contraction by columns that 32-bit offsets reach.
#pragma once

#include "grouped_core.hpp"
#include "grouped_sched.inc"

namespace g16 {
namespace grp {

constexpr int kRingTile = 256, kRingStep = 64;
constexpr int kRingLds = 160 * 1024;   // two stages of two sides of 32 KiB, and 8 KiB for each wave's epilogue

// A side's load offsets and fragment addresses in the layouts of the block.
template <bool COLS>
struct RingSide {
    uint32_t x[8];                // load q: rows 8 (8 w + q) .. + 7 of the side, or 2 (8 w + q), + 1 of the contraction
    uint32_t r[COLS ? 8 : 2];     // fragments of the wave's blocks (by columns) or of the sub-steps

    // Four neighbouring rows by columns, and four that lie 8 further on, go to
    // the eight 32-byte parts of the bank window: 32 lanes of a transposing
    // read take 32 bytes of each.
    static __device__ __forceinline__ int swz(int r) { return COLS ? ((r & 3) | ((r >> 1) & 4)) << 1 : (r >> 1) & 7; }

    __device__ __forceinline__ void start(uint32_t lds, int64_t pitch, int first, int w, int lane)
    {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int row = COLS ? 2 * (8 * w + q) + lane / 32 : 8 * (8 * w + q) + lane / 8;
            const int c = (COLS ? lane % 32 : lane % 8) ^ swz(row);
            x[q] = (uint32_t)(row * pitch + 16 * c) - 1024u * (q % 4);
        }
        const int g = lane >> 4, i = lane & 15;
#pragma unroll
        for (int n = 0; n < (COLS ? 8 : 2); ++n) {
            if (COLS) {
                const int row = 8 * g + (i >> 2), c = first / 8 + 2 * n + ((i & 3) >> 1);
                r[n] = lds + row * 512 + ((c ^ swz(row)) << 4) + ((i & 1) << 3);
            } else {
                const int row = first + i;
                r[n] = lds + row * 128 + (((4 * n + g) ^ swz(row)) << 4);
            }
        }
    }
};

// A value that is the same for all lanes, as an operand in scalar registers.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)x); }

__device__ __forceinline__ u32x4 ring_rsrc(const char* base, int64_t bytes)
{
    const uint64_t at = (uint64_t)base;
    return u32x4{uniform((uint32_t)at), uniform((uint32_t)(at >> 32) & 0xffffu), uniform((uint32_t)bytes), 0x00020000u};
}

// What a block needs beside its sides.
struct RingStore {
    uint32_t ew[8], er[4], so[4], sw;   // sw: of outputs in 32 bits

    __device__ __forceinline__ void start(uint32_t lds, int64_t pitch, int64_t wide_pitch, int w, int lane)
    {
        const uint32_t epi = lds + 131072u + 8192u * (uint32_t)w;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int r = lane & 15, n = 16 * j + 4 * (lane >> 4);
            ew[j] = epi + r * 256 + ((((n >> 3) ^ r) & 15) << 4) + ((n & 7) << 1);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int r = 4 * q + (lane >> 4), c = lane & 15;
            er[q] = epi + r * 256 + ((c ^ r) << 4);
            so[q] = (uint32_t)(r * pitch + 16 * c);
        }
        sw = (uint32_t)((lane & 15) * wide_pitch + 16 * (lane >> 4));
    }
};

// Operands of the blocks: common ones, and each side's fragment addresses.
#define G16_GROUPED_COMMON \
    [ax0] "v"(a.x[0]), [ax1] "v"(a.x[1]), [ax2] "v"(a.x[2]), [ax3] "v"(a.x[3]), [ax4] "v"(a.x[4]), [ax5] "v"(a.x[5]), [ax6] "v"(a.x[6]), \
    [ax7] "v"(a.x[7]), [bx0] "v"(b.x[0]), [bx1] "v"(b.x[1]), [bx2] "v"(b.x[2]), [bx3] "v"(b.x[3]), [bx4] "v"(b.x[4]), [bx5] "v"(b.x[5]), \
    [bx6] "v"(b.x[6]), [bx7] "v"(b.x[7]), [rsa] "s"(rsa), [rsb] "s"(rsb), [rsd] "s"(rsd), [lb] "s"(lb), [gstr] "s"(gstr), [wide] "s"(wide), \
    [rsan] "s"(rsan), [rsbn] "s"(rsbn), [first] "s"(first), [par] "s"(par), \
    [ew0] "v"(out.ew[0]), [ew1] "v"(out.ew[1]), [ew2] "v"(out.ew[2]), [ew3] "v"(out.ew[3]), [ew4] "v"(out.ew[4]), [ew5] "v"(out.ew[5]), \
    [ew6] "v"(out.ew[6]), [ew7] "v"(out.ew[7]), [er0] "v"(out.er[0]), [er1] "v"(out.er[1]), [er2] "v"(out.er[2]), [er3] "v"(out.er[3]), \
    [so0] "v"(out.so[0]), [so1] "v"(out.so[1]), [so2] "v"(out.so[2]), [so3] "v"(out.so[3]), [sw] "v"(out.sw)
#define G16_GROUPED_A_ROWS [ra0] "v"(a.r[0]), [ra1] "v"(a.r[1]), [hm0] "v"(hm[0]), [hm1] "v"(hm[1])
#define G16_GROUPED_B_ROWS [rb0] "v"(b.r[0]), [rb1] "v"(b.r[1])
#define G16_GROUPED_EXT \
    [ext] "s"(ext), [rsa0] "s"(rsa0), [rsb0] "s"(rsb0), [ha0] "v"(ha[0]), [ha1] "v"(ha[1]), [hb0] "v"(hb[0]), [hb1] "v"(hb[1]), [sb8] "s"(sb8)
#define G16_GROUPED_A_COLS \
    [ra0] "v"(a.r[0]), [ra1] "v"(a.r[1]), [ra2] "v"(a.r[2]), [ra3] "v"(a.r[3]), [ra4] "v"(a.r[4]), [ra5] "v"(a.r[5]), [ra6] "v"(a.r[6]), \
    [ra7] "v"(a.r[7]), [sta] "s"(sta)
#define G16_GROUPED_B_COLS \
    [rb0] "v"(b.r[0]), [rb1] "v"(b.r[1]), [rb2] "v"(b.r[2]), [rb3] "v"(b.r[3]), [rb4] "v"(b.r[4]), [rb5] "v"(b.r[5]), [rb6] "v"(b.r[6]), \
    [rb7] "v"(b.r[7]), [stb] "s"(stb)
#define G16_GROUPED_STATE \
    [koa] "+s"(koa), [kob] "+s"(kob), [kha] "=&s"(kha), [khb] "=&s"(khb), [rem] "+s"(rem), [sdo] "=&s"(sdo), \
    [ht] "=&v"(ht)

#define G16_GROUPED_CLOBBERS \
    "memory", "m0", "scc", "vcc", \
    "v64", "v65", "v66", "v67", "v68", "v69", "v70", "v71", "v72", "v73", "v74", "v75", "v76", "v77", "v78", "v79", "v80", "v81", "v82", "v83", \
    "v84", "v85", "v86", "v87", "v88", "v89", "v90", "v91", "v92", "v93", "v94", "v95", "v96", "v97", "v98", "v99", "v100", "v101", "v102", \
    "v103", "v104", "v105", "v106", "v107", "v108", "v109", "v110", "v111", "v112", "v113", "v114", "v115", "v116", "v117", "v118", "v119", \
    "v120", "v121", "v122", "v123", "v124", "v125", "v126", "v127", "v128", "v129", "v130", "v131", "v132", "v133", "v134", "v135", "v136", \
    "v137", "v138", "v139", "v140", "v141", "v142", "v143", "v144", "v145", "v146", "v147", "v148", "v149", "v150", "v151", "v152", "v153", \
    "v154", "v155", "v156", "v157", "v158", "v159", "v160", "v161", "v162", "v163", "v164", "v165", "v166", "v167", "v168", "v169", "v170", \
    "v171", "v172", "v173", "v174", "v175", "v176", "v177", "v178", "v179", "v180", "v181", "v182", "v183", "v184", "v185", "v186", "v187", \
    "v188", "v189", "v190", "v191", "v192", "v193", "v194", "v195", "v196", "v197", "v198", "v199", "v200", "v201", "v202", "v203", "v204", \
    "v205", "v206", "v207", "v208", "v209", "v210", "v211", "v212", "v213", "v214", "v215", "v216", "v217", "v218", "v219", "v220", "v221", \
    "v222", "v223", "v224", "v225", "v226", "v227", "v228", "v229", "v230", "v231", "v232", "v233", "v234", "v235", "v236", "v237", "v238", \
    "v239", "v240", "v241", "v242", "v243", "v244", "v245", "v246", "v247", "v248", "v249", "v250", "v251", "v252", "v253", "v254", "v255", \
    "a0", "a1", "a2", "a3", "a4", "a5", "a6", "a7", "a8", "a9", "a10", "a11", "a12", "a13", "a14", "a15", \
    "a16", "a17", "a18", "a19", "a20", "a21", "a22", "a23", "a24", "a25", "a26", "a27", "a28", "a29", "a30", "a31", \
    "a32", "a33", "a34", "a35", "a36", "a37", "a38", "a39", "a40", "a41", "a42", "a43", "a44", "a45", "a46", "a47", \
    "a48", "a49", "a50", "a51", "a52", "a53", "a54", "a55", "a56", "a57", "a58", "a59", "a60", "a61", "a62", "a63", \
    "a64", "a65", "a66", "a67", "a68", "a69", "a70", "a71", "a72", "a73", "a74", "a75", "a76", "a77", "a78", "a79", \
    "a80", "a81", "a82", "a83", "a84", "a85", "a86", "a87", "a88", "a89", "a90", "a91", "a92", "a93", "a94", "a95", \
    "a96", "a97", "a98", "a99", "a100", "a101", "a102", "a103", "a104", "a105", "a106", "a107", "a108", "a109", "a110", "a111", \
    "a112", "a113", "a114", "a115", "a116", "a117", "a118", "a119", "a120", "a121", "a122", "a123", "a124", "a125", "a126", "a127", \
    "a128", "a129", "a130", "a131", "a132", "a133", "a134", "a135", "a136", "a137", "a138", "a139", "a140", "a141", "a142", "a143", \
    "a144", "a145", "a146", "a147", "a148", "a149", "a150", "a151", "a152", "a153", "a154", "a155", "a156", "a157", "a158", "a159", \
    "a160", "a161", "a162", "a163", "a164", "a165", "a166", "a167", "a168", "a169", "a170", "a171", "a172", "a173", "a174", "a175", \
    "a176", "a177", "a178", "a179", "a180", "a181", "a182", "a183", "a184", "a185", "a186", "a187", "a188", "a189", "a190", "a191", \
    "a192", "a193", "a194", "a195", "a196", "a197", "a198", "a199", "a200", "a201", "a202", "a203", "a204", "a205", "a206", "a207", \
    "a208", "a209", "a210", "a211", "a212", "a213", "a214", "a215", "a216", "a217", "a218", "a219", "a220", "a221", "a222", "a223", \
    "a224", "a225", "a226", "a227", "a228", "a229", "a230", "a231", "a232", "a233", "a234", "a235", "a236", "a237", "a238", "a239", \
    "a240", "a241", "a242", "a243", "a244", "a245", "a246", "a247", "a248", "a249", "a250", "a251", "a252", "a253", "a254", "a255"

}  // namespace grp
}  // namespace g16
