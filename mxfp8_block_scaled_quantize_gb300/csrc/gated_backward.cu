// Backward pass of the gated feed-forward's activation and product: from the
// gradient dh of h = act(g) u and the pre-activations [g | u] that the forward
// GEMM kept,
//   dg = dh u act'(g),   du = dh act(g),
// each evaluated in fp32 and rounded once to bf16 (what the bias gradient, a
// plain copy and the quantised copies all see, so they belong together).  The
// bf16 matrix [dg | du] is written as it is, or MXFP8-quantised exactly as
// te_mx_quantize quantises it: row-wise (the operand of dX = [dg | du] W) and
// column-wise (the operand of dW = [dg | du]^T X), the tokens zero-padded to a
// multiple of 128 there, the granularity of a GEMM's K.
//
// Bound by HBM: 6 bytes read per element of dh, 4 written in bf16 or 4.1 as
// the two copies' codes and scales (2 bytes each).
//   dense:      16-byte loads and stores, a thread per 8 columns.
//   quantising: the MXFP8 quantiser's decomposition (mx_unit.cuh): units of 64
//               rows x 64 columns of dh, g and u per pair of warps, loaded by
//               TMA; the pair turns g and u into dg and du in place, in shared
//               memory, then one warp quantises dg and the other du; the CTA
//               walks strips of 8 units, so that a strip's row-wise scale bytes
//               leave as whole words.  Four warps write them a round later, so
//               that no pair waits for the others and the pairs' loads, arithmetic
//               and stores overlap.
// Measured (us; floor, here): dense 4096 x 4096 24.7, 26.7; both copies 8192 x
// 18432 225, 277 (391 with one warp per unit, 291 with the scale bytes written
// before the pair goes on); what is left is the arithmetic of two quantisations
// per element pair at 16 warps per SM.
#include <cuda_runtime.h>

#include "e4m3.cuh"
#include "f32x2.cuh"
#include "gated_act.cuh"
#include "mx_unit.cuh"
#include "ptx.cuh"
#include "temx_internal.h"
#include "units.cuh"

namespace temx {

namespace {

constexpr int kRows = 64;                    // unit height (two column-wise blocks)
constexpr int kCols = 64;                    // unit width in bf16 (= 128-byte swizzle row)
constexpr int kTileBytes = kRows * kCols * 2;
constexpr int kUnitBytes = 3 * kTileBytes;   // dh, gate, up
constexpr int kUnits = 8;                    // units per strip: 8 x 2 scale bytes = 16 per row
constexpr int kThreads = kUnits * 64;        // a pair of warps per unit
constexpr int kScaleSlots = 4;               // rounds whose row-wise scale bytes may be in use at a time
constexpr int kScaleWarps = 4;               // warps that write them
constexpr int kSmemBytes = kUnits * kUnitBytes + 1024;

struct GatedBwdParams {
    int64_t rows, F;
    int64_t col_units;       // ceil(F / 64)
    int64_t bands;           // 64-row bands (with a column-wise copy: of the padded rows)
    uint8_t* s_row;
    int64_t ld_s_row;
    uint8_t* s_col;
    int64_t ld_s_col;
    int32_t act;
    unsigned int* status;
};

__device__ __forceinline__ uint32_t pack_bf16(uint64_t v) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(f32x2::hi(v)), "f"(f32x2::lo(v)));
    return r;
}
__device__ __forceinline__ uint64_t bf16_pair(uint32_t w) { return f32x2::pack(bf16_lo(w), bf16_hi(w)); }

// Two elements (a word each of dh, gate and up) -> gate becomes dg, up du.
template <int kAct>
__device__ __forceinline__ void dgate2(uint32_t dh, uint32_t& gate, uint32_t& up) {
    uint64_t a, d;
    gated::act_and_grad2<kAct>(bf16_pair(gate), a, d);
    const uint64_t h = bf16_pair(dh);
    gate = pack_bf16(f32x2::mul(f32x2::mul(h, bf16_pair(up)), d));
    up = pack_bf16(f32x2::mul(h, a));
}

template <int kAct>
__device__ __forceinline__ void dgate8(const uint4& dh, uint4& gate, uint4& up) {
    dgate2<kAct>(dh.x, gate.x, up.x);
    dgate2<kAct>(dh.y, gate.y, up.y);
    dgate2<kAct>(dh.z, gate.z, up.z);
    dgate2<kAct>(dh.w, gate.w, up.w);
}

// ---------------------------------------------------------------- dense

constexpr int kDenseThreads = 256;

__global__ void __launch_bounds__(kDenseThreads)
gated_backward_kernel(const GatedBackwardArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t nv = a.F / 8, total = a.rows * nv;         // 16-byte vectors of a row, of dh
    const UnitWalk walk(int64_t(gridDim.x) * kDenseThreads, nv);
    int64_t i = int64_t(blockIdx.x) * kDenseThreads + threadIdx.x;
    if (i >= total) return;
    int32_t row, c;
    walk.start(i, row, c);
    gated::with(a.act, [&](auto act) {
        for (; i < total; i += int64_t(gridDim.x) * kDenseThreads, walk.step(row, c)) {
            const uint16_t* gu = static_cast<const uint16_t*>(a.gate_up) + row * a.ld_gate_up + 8 * c;
            const uint4 dh = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.dh) + row * a.ld_dh + 8 * c);
            uint4 g = *reinterpret_cast<const uint4*>(gu), u = *reinterpret_cast<const uint4*>(gu + a.F);
            dgate8<decltype(act)::value>(dh, g, u);
            uint16_t* d = static_cast<uint16_t*>(a.d_gate_up) + row * a.ld_d + 8 * c;
            st_global_v4(d, g.x, g.y, g.z, g.w);
            st_global_v4(d + a.F, u.x, u.y, u.z, u.w);
        }
    });
}

// ---------------------------------------------------------------- quantising

template <bool kDense, bool kRowwise, bool kColwise>
__global__ void __launch_bounds__(kThreads, 1)
gated_backward_quantize_kernel(const __grid_constant__ CUtensorMap dh_map, const __grid_constant__ CUtensorMap gu_map,
                               const __grid_constant__ CUtensorMap d_map, const __grid_constant__ CUtensorMap qrow_map,
                               const __grid_constant__ CUtensorMap qcol_map, const GatedBwdParams p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[kUnits];
    __shared__ __align__(8) uint64_t scales_full[kScaleSlots], scales_empty[kScaleSlots];
    // row-wise scale bytes of a strip: (gate, up) x 64 rows x 16 bytes
    __shared__ __align__(16) uint8_t row_scales[kScaleSlots][2][kRows][16];

    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pair = warp >> 1, half = warp & 1;             // the pair's unit of a strip; gate or up
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t strips_per_band = (p.col_units + kUnits - 1) / kUnits;
    const int64_t n_strips = p.bands * strips_per_band;
    if (int64_t(blockIdx.x) >= n_strips) return;                         // (uniform over the CTA)
    const int64_t n_mine = (n_strips - blockIdx.x + gridDim.x - 1) / gridDim.x;
    const uint32_t unit = smem_u32(smem + pair * kUnitBytes), tile = unit + (1 + half) * kTileBytes;
    const UnitWalk walk(gridDim.x, strips_per_band);
    int32_t band, strip;
    walk.start(blockIdx.x, band, strip);
    int32_t next_band = band, next_strip = strip;
    const uint32_t bar = smem_u32(&bars[pair]);              // three arrivals: dh (the even warp), gate, up (each its own)
    auto unit_col = [&](int32_t st) { return st * kUnits + pair; };
    // lane 0: load dh, or this warp's half of [gate | up], of the strip (b, st)
    // (past the rows' end: zeros; past the band's end: the arrival alone)
    auto load_dh = [&](int32_t b, int32_t st) {
        if (unit_col(st) < p.col_units) {
            mbar_arrive_expect_tx(bar, kTileBytes);
            tma_load_2d(unit, &dh_map, bar, unit_col(st) * kCols, b * kRows);
        } else {
            mbar_arrive(bar);
        }
    };
    auto load_half = [&](int32_t b, int32_t st) {
        if (unit_col(st) < p.col_units) {
            mbar_arrive_expect_tx(bar, kTileBytes);
            tma_load_3d(tile, &gu_map, bar, unit_col(st) * kCols, half, b * kRows);
        } else {
            mbar_arrive(bar);
        }
    };
    if (lane == 0 && half == 0) mbar_init(bar, 3);
    if (threadIdx.x == 0)
        for (int k = 0; k < kScaleSlots; ++k) {
            mbar_init(smem_u32(&scales_full[k]), kThreads / 32);
            mbar_init(smem_u32(&scales_empty[k]), kScaleWarps);
        }
    if (lane == 0) fence_mbarrier_init();
    __syncthreads();
    if (lane == 0) {
        if (half == 0) load_dh(band, strip);
        load_half(band, strip);
    }
    __syncwarp();

    bool ok = true;                      // false once a wait gave up: the warp then only keeps the barriers
    // (warps 0 .. kScaleWarps - 1) write the row-wise scale bytes of round i, of
    // the strip (b, st): lane = row of one half; 16 bytes, or single bytes where
    // the strip is cut by the end of F or the half does not start on a 16-byte boundary
    auto write_scales = [&](int64_t i, int32_t b, int32_t st) {
        const int slot = int(i % kScaleSlots), hs = warp >> 1, rl = (warp & 1) * 32 + lane;
        ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&scales_full[slot]), uint32_t(i / kScaleSlots) & 1u, p.status));
        const int64_t r = int64_t(b) * kRows + rl;
        const int64_t first = int64_t(st) * kUnits * 2;                // the strip's first scale byte
        const int64_t valid = p.F / 32 - first;                         // scale bytes of the half left
        if (ok && r < p.rows) {
            uint8_t* sp = p.s_row + r * p.ld_s_row + hs * (p.F / 32) + first;
            const uint4 v = lds128(smem_u32(&row_scales[slot][hs][rl][0]));
            if (valid >= 16 && (hs == 0 || p.F % 512 == 0)) {
                st_global_v4(sp, v.x, v.y, v.z, v.w);
            } else {
                const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    if (k < valid) st_global_u8(sp + k, (w4[k >> 2] >> (8 * (k & 3))) & 0xFFu);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&scales_empty[slot]));
    };
    int32_t last_band = 0, last_strip = 0;
    for (int64_t i = 0; i < n_mine; ++i) {
        const int32_t col = unit_col(strip);
        const int slot = int(i % kScaleSlots);
        const bool mine = col < p.col_units, more = i + 1 < n_mine;
        walk.step(next_band, next_strip);
        if (ok && !__all_sync(0xFFFFFFFFu, mbar_wait(bar, uint32_t(i & 1), p.status))) {
            ok = false;
            if (lane == 0) mbar_wait(bar, uint32_t(i & 1), p.status);   // gave up: let the loads in flight land
        }
        const int64_t r0 = int64_t(band) * kRows, c0 = int64_t(col) * kCols;
        if (ok && mine) {
            gated::with(p.act, [&](auto act) {
#pragma unroll 4
                for (int k = 0; k < 8; ++k) {                  // (every tile has the same swizzle)
                    const uint32_t off = uint32_t(k * 64 + half * 32 + lane) * 16;
                    uint4 g = lds128(unit + kTileBytes + off), u = lds128(unit + 2 * kTileBytes + off);
                    dgate8<decltype(act)::value>(lds128(unit + off), g, u);
                    sts128(unit + kTileBytes + off, g.x, g.y, g.z, g.w);
                    sts128(unit + 2 * kTileBytes + off, u.x, u.y, u.z, u.w);
                }
            });
            if (kDense) fence_proxy_async_smem();
        }
        named_barrier_sync(1 + pair, 64);         // both tiles of the unit hold the gradient, dh is read
        if (ok && more && lane == 0 && half == 0) load_dh(next_band, next_strip);
        // The slot's bytes of four rounds ago are written.  Every warp waits for that
        // before it arrives on scales_full, with a unit or without: an arrival counts
        // in the phase at hand, so a warp rounds ahead would complete it for the others.
        // (Warps with a unit wait as late as they can; all of them here: 323 us, not 310, for
        // 8192 x 18432 back to back.)
        auto wait_slot = [&]() {
            if (kRowwise && i >= kScaleSlots)
                ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&scales_empty[slot]), uint32_t(i / kScaleSlots - 1) & 1u,
                                                             p.status));
        };
        if (!mine) wait_slot();
        if (ok && mine) {
            if (kDense && lane == 0) {
                if (r0 < p.rows) tma_store_3d(&d_map, tile, int32_t(c0), half, int32_t(r0));
                bulk_commit();
            }
            uint32_t cc[2][2][8];                 // column codes [half of the rows][column 2l / 2l+1][words]
            uint32_t rc[2][2][8];                 // row codes [row l / l+32][block][words]
            if (kColwise) {
                uint32_t s_lo[2], s_hi[2];
                float unused = 0.0f;
                col_blocks(tile, 0, lane, cc[0][0], cc[0][1], s_lo[0], s_hi[0], unused, unused);
                col_blocks(tile, 32, lane, cc[1][0], cc[1][1], s_lo[1], s_hi[1], unused, unused);
                const int64_t c = c0 + 2 * lane;
                if (c < p.F) {                                 // F % 32 == 0: c + 1 valid too
                    uint8_t* sp = p.s_col + (half * p.F + c) * p.ld_s_col + (r0 >> 5);
                    st_global_u16(sp, s_lo[0] | (s_lo[1] << 8));
                    st_global_u16(sp + p.ld_s_col, s_hi[0] | (s_hi[1] << 8));
                }
            }
            if (kRowwise) {
                wait_slot();
#pragma unroll
                for (int rr = 0; rr < 2; ++rr) {
                    uint32_t sb[2];
                    row_blocks(tile + (lane + 32 * rr) * 128, lane & 7, rc[rr], sb);
                    sts16(smem_u32(&row_scales[slot][half][lane + 32 * rr][2 * pair]), sb[0] | (sb[1] << 8));
                }
            }
            if (kDense && lane == 0) bulk_wait_read_all();     // the copy out has read the tile
            __syncwarp();                         // every lane has read the tile: reuse it for the codes
            if (kRowwise) {
#pragma unroll
                for (int rr = 0; rr < 2; ++rr) {
                    const int r = lane + 32 * rr;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t* w = rc[rr][c >> 1] + 4 * (c & 1);
                        sts128(tile + sw64(r, c), w[0], w[1], w[2], w[3]);
                    }
                }
            }
            if (kColwise) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const uint32_t* w = cc[h][j] + 4 * t;
                            sts128(tile + 4096 + sw64(2 * lane + j, 2 * h + t), w[0], w[1], w[2], w[3]);
                        }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (kRowwise && r0 < p.rows) tma_store_3d(&qrow_map, tile, int32_t(c0), half, int32_t(r0));
                if (kColwise) tma_store_3d(&qcol_map, tile + 4096, int32_t(r0), int32_t(c0), half);
                bulk_commit();
            }
        }
        if (ok && more && lane == 0) {
            bulk_wait_read_all();                 // the stores have read the tile: refill it
            load_half(next_band, next_strip);
        }
        __syncwarp();
        if (kRowwise) {
            if (lane == 0) mbar_arrive(smem_u32(&scales_full[slot]));
            if (warp < kScaleWarps && i > 0) write_scales(i - 1, last_band, last_strip);
            last_band = band;
            last_strip = strip;
        }
        band = next_band;
        strip = next_strip;
    }
    if (kRowwise && warp < kScaleWarps) write_scales(n_mine - 1, last_band, last_strip);
    if (lane == 0) bulk_wait_all();
}

template <bool kDense, bool kRowwise, bool kColwise>
cudaError_t launch(const CUtensorMap (&m)[5], const GatedBwdParams& p, int sms, cudaStream_t stream) {
    auto kern = gated_backward_quantize_kernel<kDense, kRowwise, kColwise>;
    cudaError_t e = set_smem_attribute_once(reinterpret_cast<const void*>(kern), kSmemBytes);
    if (e != cudaSuccess) return e;
    const int64_t strips = p.bands * ((p.col_units + kUnits - 1) / kUnits);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(strips < sms ? strips : sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, m[0], m[1], m[2], m[3], m[4], p);
}

}  // namespace

te_mx_status gated_backward_launch(const GatedBackwardArgs& a, cudaStream_t stream) {
    int sms = 0;
    te_mx_status st = device_sm_count(&sms);
    if (st != TE_MX_OK) return st;
    const bool dense = a.d_gate_up != nullptr, rowwise = a.q_row != nullptr, colwise = a.q_col != nullptr;
    cudaError_t e;
    if (!rowwise && !colwise) {
        const int64_t blocks = (a.rows * (a.F / 8) + kDenseThreads - 1) / kDenseThreads, most = int64_t(sms) * 8;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(unsigned(blocks < most ? blocks : most));
        cfg.blockDim = dim3(kDenseThreads);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, gated_backward_kernel, a);
        return cuda_status(e, "gated backward kernel launch");
    }
    // The maps' middle dimension is the half (gate, up), so that boxes past
    // column F are clipped, not continued in the other half.
    const uint64_t F = uint64_t(a.F), rows = uint64_t(a.rows), padded = (rows + 127) / 128 * 128;
    CUtensorMap m[5];
    if ((st = encode_tensor_map_2d(&m[0], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.dh, F, rows, uint64_t(a.ld_dh) * 2, kCols, kRows,
                                   CU_TENSOR_MAP_SWIZZLE_128B)) != TE_MX_OK) return st;
    if ((st = encode_tensor_map_3d(&m[1], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.gate_up, F, 2, rows, F * 2,
                                   uint64_t(a.ld_gate_up) * 2, kCols, 1, kRows, CU_TENSOR_MAP_SWIZZLE_128B)) != TE_MX_OK)
        return st;
    m[2] = m[3] = m[4] = m[1];
    if (dense && (st = encode_tensor_map_3d(&m[2], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.d_gate_up, F, 2, rows, F * 2,
                                            uint64_t(a.ld_d) * 2, kCols, 1, kRows, CU_TENSOR_MAP_SWIZZLE_128B)) != TE_MX_OK)
        return st;
    if (rowwise && (st = encode_tensor_map_3d(&m[3], CU_TENSOR_MAP_DATA_TYPE_UINT8, a.q_row, F, 2, rows, F, 2 * F, kCols, 1,
                                              kRows, CU_TENSOR_MAP_SWIZZLE_64B)) != TE_MX_OK)
        return st;
    if (colwise && (st = encode_tensor_map_3d(&m[4], CU_TENSOR_MAP_DATA_TYPE_UINT8, a.q_col, padded, F, 2,
                                              uint64_t(a.ld_q_col), uint64_t(a.ld_q_col) * F, kRows, kCols, 1,
                                              CU_TENSOR_MAP_SWIZZLE_64B)) != TE_MX_OK)
        return st;
    GatedBwdParams p;
    p.rows = a.rows; p.F = a.F;
    p.col_units = (a.F + kCols - 1) / kCols;
    p.bands = (colwise ? int64_t(padded) : a.rows + kRows - 1) / kRows;
    p.s_row = a.s_row; p.ld_s_row = a.ld_s_row;
    p.s_col = a.s_col; p.ld_s_col = a.ld_s_col;
    p.act = a.act;
    if ((st = device_status_ptr(&p.status)) != TE_MX_OK) return st;
    if (dense) {
        if (rowwise && colwise) e = launch<true, true, true>(m, p, sms, stream);
        else if (rowwise) e = launch<true, true, false>(m, p, sms, stream);
        else e = launch<true, false, true>(m, p, sms, stream);
    } else {
        if (rowwise && colwise) e = launch<false, true, true>(m, p, sms, stream);
        else if (rowwise) e = launch<false, true, false>(m, p, sms, stream);
        else e = launch<false, false, true>(m, p, sms, stream);
    }
    return cuda_status(e, "gated backward kernel launch");
}

}  // namespace temx
