// MXFP8 quantisation of a 64 x 64 bf16 unit held in shared memory (128-byte
// rows, 128-byte swizzle) by one warp: row-wise blocks (lane = a row) and
// column-wise blocks (lane = two columns), shared by the quantisers.
#pragma once
#include <cstdint>

#include "e4m3.cuh"
#include "ptx.cuh"

namespace temx {

// E8M0 byte from |amax| as bf16 bits: exponent field - 8, floored at 0;
// 0xFF for NaN/inf.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
    const uint32_t ef = amax_bits >> 7;
    if (ef == 0xFFu) return 0xFFu;
    return ef > 8u ? ef - 8u : 0u;
}

// One row of a unit (64 bf16 at shared address `row_addr`, 128-byte swizzle
// phase `sw`): two row-wise blocks -> codes[2][8] words, scale bytes sb[2].
__device__ __forceinline__ void row_blocks(uint32_t row_addr, int sw, uint32_t (&codes)[2][8], uint32_t (&sb)[2]) {
    uint32_t w[32];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint4 v = lds128(row_addr + ((j ^ sw) << 4));
        w[4 * j + 0] = v.x; w[4 * j + 1] = v.y; w[4 * j + 2] = v.z; w[4 * j + 3] = v.w;
    }
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
        const uint32_t m2 = amax_words<16>(w + 16 * blk);
        sb[blk] = scale_byte(max(m2 & 0xFFFFu, m2 >> 16));
        const float m = inv_scale(sb[blk]);
#pragma unroll
        for (int i = 0; i < 8; ++i) codes[blk][i] = quant4(w[16 * blk + 2 * i], w[16 * blk + 2 * i + 1], m);
        if (sb[blk] == 0xFFu) {
#pragma unroll
            for (int i = 0; i < 8; ++i) codes[blk][i] = 0x7F7F7F7Fu;
        }
    }
}

// Columns 2l and 2l+1 over the 32 rows from `row0` (a multiple of 8):
// codes lo[8] / hi[8] (32 bytes each, rows in order) and their scale bytes.
__device__ __forceinline__ void col_blocks(uint32_t tile, int row0, int lane, uint32_t (&lo)[8], uint32_t (&hi)[8],
                                           uint32_t& s_lo, uint32_t& s_hi, float& sum_lo, float& sum_hi) {
    uint32_t w[32];
    const uint32_t base = tile + row0 * 128 + ((lane & 3) << 2);
    const int chunk = lane >> 2;
#pragma unroll
    for (int r = 0; r < 32; ++r) w[r] = lds32(base + r * 128 + ((chunk ^ (r & 7)) << 4));
#pragma unroll
    for (int r = 0; r < 32; ++r) {                  // column sums for the bias gradient (row order)
        sum_lo += bf16_lo(w[r]);
        sum_hi += bf16_hi(w[r]);
    }
    const uint32_t m2 = amax_words<32>(w);
    s_lo = scale_byte(m2 & 0xFFFFu);
    s_hi = scale_byte(m2 >> 16);
    const float m_lo = inv_scale(s_lo), m_hi = inv_scale(s_hi);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t a0 = w[4 * i], a1 = w[4 * i + 1], a2 = w[4 * i + 2], a3 = w[4 * i + 3];
        lo[i] = cvt_e4m3x2(__fmul_rn(bf16_lo(a0), m_lo), __fmul_rn(bf16_lo(a1), m_lo)) |
                (cvt_e4m3x2(__fmul_rn(bf16_lo(a2), m_lo), __fmul_rn(bf16_lo(a3), m_lo)) << 16);
        hi[i] = cvt_e4m3x2(__fmul_rn(bf16_hi(a0), m_hi), __fmul_rn(bf16_hi(a1), m_hi)) |
                (cvt_e4m3x2(__fmul_rn(bf16_hi(a2), m_hi), __fmul_rn(bf16_hi(a3), m_hi)) << 16);
    }
    if (s_lo == 0xFFu) {
#pragma unroll
        for (int i = 0; i < 8; ++i) lo[i] = 0x7F7F7F7Fu;
    }
    if (s_hi == 0xFFu) {
#pragma unroll
        for (int i = 0; i < 8; ++i) hi[i] = 0x7F7F7F7Fu;
    }
}

__device__ __forceinline__ void sts16(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.b16 [%0], %1;" :: "r"(addr), "h"(static_cast<uint16_t>(v)) : "memory");
}

// Barrier `id` over `n` threads (whole warps) of the CTA.
__device__ __forceinline__ void named_barrier_sync(uint32_t id, uint32_t n) {
    asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(n) : "memory");
}

// Byte offset of 16-byte chunk c of 64-byte row r in a 64-byte-swizzled tile.
__device__ __forceinline__ uint32_t sw64(int r, int c) { return uint32_t(r * 64 + ((c ^ ((r >> 1) & 3)) << 4)); }

}  // namespace temx
