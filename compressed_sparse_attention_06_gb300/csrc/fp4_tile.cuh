// FP4 (E2M1 + E4M3 per 16) cache rows into a swizzled bf16 operand tile, shared by the
// tensor-core kernels that read FP4 rows.
#pragma once

#include "sm100_ptx.cuh"

namespace {

__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// 128-dim block db (chunks 2db, 2db+1: dims 128db .. 128db+127) of an FP4 row into row
// r of the tile as bf16, by table lookup rather than per-value conversion.  Per 16-dim
// scale block, the eight E2M1 magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 are multiplied by
// the block's E4M3 scale as bf16 pairs (exact: an E2M1 value times an E4M3 scale has at
// most 6 significant bits), then split into a low-byte and a high-byte table; each
// code's 3 magnitude bits pick its two bytes with a byte permute, and its sign bit is
// XORed into the bf16 sign.  The squares (for the row's RMS) come from a byte table of
// 4 x magnitude^2 summed with dp4a, times scale^2 / 4 per scale block; the block's sum
// of squares is returned.  code[4]: the block's 64 code bytes (value 2k in the low
// nibble of byte k); sc0, sc1: the four scale bytes of each chunk.  The eight scale
// blocks are independent chains, unrolled together for the latency; not inlined: one
// copy of the code serves the four blocks, which keeps a CTA's single pass over a tile
// (decode) from stalling on instruction fetch.
template <int CHUNK>
__device__ __noinline__ float fp4_block_to_tile(uint4 k0, uint4 k1, uint4 k2, uint4 k3, uint32_t sc0, uint32_t sc1,
                                                uint8_t* sK, int db, int r) {
    const uint32_t cw[16] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w,
                             k2.x, k2.y, k2.z, k2.w, k3.x, k3.y, k3.z, k3.w};
    float ss[8];
#pragma unroll
    for (int sb = 0; sb < 8; ++sb) {                    // scale block: chunk sb / 4, 16 dims
        const uint32_t scw = sb < 4 ? sc0 : sc1;
        const float sc = e4m3_to_f32((scw >> (8 * (sb & 3))) & 0xFFu);
        const uint32_t s2 = __byte_perm(__float_as_uint(sc), 0u, 0x3232);     // (bf16 scale, bf16 scale)
        const uint32_t t01 = bf16x2_mul(0x3F000000u, s2);                     // (0, 0.5) x scale
        const uint32_t t23 = bf16x2_mul(0x3FC03F80u, s2);                     // (1, 1.5)
        const uint32_t t45 = bf16x2_mul(0x40404000u, s2);                     // (2, 3)
        const uint32_t t67 = bf16x2_mul(0x40C04080u, s2);                     // (4, 6)
        const uint32_t lo0 = __byte_perm(t01, t23, 0x6420), hi0 = __byte_perm(t01, t23, 0x7531);
        const uint32_t lo1 = __byte_perm(t45, t67, 0x6420), hi1 = __byte_perm(t45, t67, 0x7531);
        uint32_t q = 0u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int u = 2 * (sb & 3) + h;              // 16-byte unit of the chunk row: 8 values
            const uint32_t w = cw[2 * sb + h];
            const uint32_t m = w & 0x77777777u, mh = m >> 16, w4 = w << 4;
            uint32_t lo = __byte_perm(lo0, lo1, m), hi = __byte_perm(hi0, hi1, m);
            const uint32_t p0 = __byte_perm(lo, hi, 0x5140) ^ (__byte_perm(w4, w, 0x4000) & 0x80008000u);
            const uint32_t p1 = __byte_perm(lo, hi, 0x7362) ^ (__byte_perm(w4, w, 0x5010) & 0x80008000u);
            lo = __byte_perm(lo0, lo1, mh);
            hi = __byte_perm(hi0, hi1, mh);
            const uint32_t p2 = __byte_perm(lo, hi, 0x5140) ^ (__byte_perm(w4, w, 0x6020) & 0x80008000u);
            const uint32_t p3 = __byte_perm(lo, hi, 0x7362) ^ (__byte_perm(w4, w, 0x7030) & 0x80008000u);
            q = __dp4a(__byte_perm(0x09040100u, 0x90402410u, m), 0x01010101u, q);
            q = __dp4a(__byte_perm(0x09040100u, 0x90402410u, mh), 0x01010101u, q);
            *reinterpret_cast<uint4*>(sK + (2 * db + (sb >> 2)) * CHUNK + sm100::sw128_offset((uint32_t)r, (uint32_t)u)) =
                make_uint4(p0, p1, p2, p3);
        }
        ss[sb] = (float)q * 0.25f * (sc * sc);
    }
    return ((ss[0] + ss[1]) + (ss[2] + ss[3])) + ((ss[4] + ss[5]) + (ss[6] + ss[7]));
}

}  // namespace
