// Backward pass of the root-mean-square norm.  With xh = z rs and g = dy gamma, over
// each row of H elements:
//   dx = rs (g - xh c) + dz,  c = sum(g xh) / H  (the gradient of x and of the
//   residual; dz is the gradient that reaches z by the residual path),
//   dgamma = sum over the rows of dy xh.
// Everything between a load and a store is fp32; dx and dgamma are rounded once, when
// they are stored.  Each kernel adds in a fixed order.
#include <cuda_runtime.h>

#include "f32x2.cuh"
#include "ptx.cuh"
#include "row_ops.cuh"
#include "temx_internal.h"

namespace temx {

namespace {

// Rows on 16-byte boundaries: one pass over dy, z and dz, persistent.  A group of
// threads owns the same columns (kV vectors per thread) of every row that it takes,
// so the sums of dy xh over the rows stay in registers.  The rows come through a ring
// in shared memory, one bulk copy of each operand, and are read there twice: for the
// row's sum, and for its dx once the sum is known, so that no word waits in registers.
// A row's stage is filled again after the next row's barrier, which every warp reaches
// past its last read of the row.  HBM bounds it: 8192 x 7168 bf16 with dz 74.8 us (floor
// 69.4; with the words kept in registers, spilled, 147; two groups of 448 threads at 72
// registers 94; the next row's sum taken before this row's dx 81), 1111 x 8200 fp32
// without dz 25 (16.2), of which the join of the blocks' sums takes 5.
// The groups of a block are joined at the end, so that every block leaves one partial
// sum per column.
// kOnce: a ring of one stage, for rows of which two do not fit: words stay in
// registers from the sum to dx, and dz is loaded from global memory.
constexpr int kBwdMaxGroups = 15;                // (named barriers)
constexpr int kBwdMaxStages = 16;
constexpr int kBwdSmem = 200 * 1024;             // the ring

struct RmsBwdShape {
    int nvec;        // vectors of a row
    int group;       // threads per group
    int groups;      // groups per block
    int stages;      // rows of a group's ring
    int streams;     // operands in the ring: dy, z and perhaps dz
};

template <typename T, bool kP32, int kV, int kMost, bool kOnce>
__global__ void __launch_bounds__(kMost, 1)
rms_backward_vec_kernel(const RmsBackwardArgs a, const RmsBwdShape sh, unsigned int* status) {
    using V = Vec<T>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t full[kBwdMaxGroups][kBwdMaxStages];          // a row's operands landed
    __shared__ float warp_part[2][kMost / 32];             // by parity of the row

    const int group = threadIdx.x / sh.group, t = threadIdx.x % sh.group, lane = threadIdx.x & 31;
    const int gwarps = sh.group >> 5;
    const uint32_t bytes = uint32_t(sh.nvec) * 16, stage_bytes = uint32_t(sh.streams) * bytes;       // dy, z, dz
    const uint32_t ring = smem_u32(smem) + uint32_t(group * sh.stages) * stage_bytes;
    const int64_t first = int64_t(blockIdx.x) * sh.groups + group, step = int64_t(gridDim.x) * sh.groups;
    const int n_mine = first < a.rows ? int((a.rows - first + step - 1) / step) : 0;
    if (t == 0) {
        for (int i = 0; i < sh.stages; ++i) mbar_init(smem_u32(&full[group][i]), 1);
        fence_mbarrier_init();
    }
    grid_dependency_wait();
    grid_launch_dependents();
    __syncthreads();
    auto load = [&](int i, int s) {                        // row i of this group into stage s, by its thread 0
        const int64_t row = first + i * step;
        const uint32_t bar = smem_u32(&full[group][s]), dst = ring + uint32_t(s) * stage_bytes;
        mbar_arrive_expect_tx(bar, stage_bytes);
        bulk_load_row(dst, static_cast<const T*>(a.dy) + row * a.ld_dy, bytes, bar);
        bulk_load_row(dst + bytes, static_cast<const T*>(a.z) + row * a.ld_z, bytes, bar);
        if (sh.streams == 3) bulk_load_row(dst + 2 * bytes, static_cast<const T*>(a.dz) + row * a.ld_dz, bytes, bar);
    };
    if (t == 0)
        for (int i = 0; i < sh.stages && i < n_mine; ++i) load(i, i);

    ParamVec<T, kP32> ga[kV];
    uint64_t dga[kV][V::kPairs];
    bool live[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        const int j = t + v * sh.group;
        live[v] = j < sh.nvec;
        ga[v].load(a.gamma, live[v] ? j : 0);
#pragma unroll
        for (int k = 0; k < V::kPairs; ++k) dga[v][k] = 0;
    }
    const uint32_t at = ring + 16u * uint32_t(t), apart = 16u * uint32_t(sh.group);          // of its vectors
    constexpr bool kUnpackGamma = kV * V::kN > 16 || kMost > 512;      // (else it stays unpacked in registers)
    const float inv_h = 1.0f / float(a.hidden);
    bool ok = true;                                        // false once a wait gave up: no waits or copies from then on
    uint4 wd[kOnce ? kV : 1], wz[kOnce ? kV : 1];
    // a thread's part of a row's sum of g xh; its part of dgamma's
    auto sum_of = [&](uint32_t here, uint64_t rs2) {
        uint64_t s = 0;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            if (!live[v]) continue;
            uint4& d4 = wd[kOnce ? v : 0];
            uint4& z4 = wz[kOnce ? v : 0];
            d4 = lds128(at + here + v * apart);
            z4 = lds128(at + here + bytes + v * apart);
            if constexpr (kUnpackGamma)
#pragma unroll
                for (int q = 0; q < ParamVec<T, kP32>::kWords; ++q) unpack_again(ga[v].w[q]);
#pragma unroll
            for (int k = 0; k < V::kPairs; ++k) {
                const uint64_t d = V::pair(d4, k), xh = f32x2::mul(V::pair(z4, k), rs2);
                s = f32x2::fma(f32x2::mul(d, ga[v].pair(k)), xh, s);
                dga[v][k] = f32x2::fma(d, xh, dga[v][k]);
            }
        }
        return f32x2::lo(s) + f32x2::hi(s);
    };
    // over the group's warps, in order (a parity's slots are read before the next row's
    // barrier, and written again after it)
    auto across_group = [&](float s, int i) {
        if (gwarps == 1) {
            __syncwarp();
            return s;
        }
        float* part = &warp_part[i & 1][group * gwarps];
        if (lane == 0) part[t >> 5] = s;
        group_barrier(1 + group, sh.group);
        return warp_sum(lane < gwarps ? part[lane] : 0.0f);
    };
    // dx = rs (g - z (rs c)) + dz  (rs rs would be no number for rows near 0 with a tiny eps)
    auto dx_of = [&](int64_t row, uint32_t here, float r, float total) {
        const uint64_t rs2 = f32x2::both(r), k2 = f32x2::both(-r * (total * inv_h));
        const uint4* dz = a.dz ? reinterpret_cast<const uint4*>(static_cast<const T*>(a.dz) + row * a.ld_dz) + t : nullptr;
        uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(a.dx) + row * a.ld_dx) + t;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            if (!live[v]) continue;
            uint4& d4 = wd[kOnce ? v : 0];
            uint4& z4 = wz[kOnce ? v : 0];
            uint4 w = make_uint4(0, 0, 0, 0);
            if constexpr (kOnce) {
                unpack_again(d4);
                unpack_again(z4);
            } else {
                d4 = lds128(at + here + v * apart);
                z4 = lds128(at + here + bytes + v * apart);
            }
            if (!kOnce && sh.streams == 3) w = lds128(at + here + 2 * bytes + v * apart);
            else if (dz) w = dz[v * sh.group];
            if constexpr (kUnpackGamma)
#pragma unroll
                for (int q = 0; q < ParamVec<T, kP32>::kWords; ++q) unpack_again(ga[v].w[q]);
            uint64_t o[V::kPairs];
#pragma unroll
            for (int k = 0; k < V::kPairs; ++k) {
                const uint64_t q = f32x2::fma(V::pair(z4, k), k2, f32x2::mul(V::pair(d4, k), ga[v].pair(k)));
                o[k] = dz ? f32x2::fma(q, rs2, V::pair(w, k)) : f32x2::mul(q, rs2);
            }
            out[v * sh.group] = V::from_pairs(o);
        }
    };
    const float* rs_p = a.rsigma + first;
    if constexpr (kOnce) {
        for (int i = 0; i < n_mine; ++i) {
            const float r = __ldg(rs_p + i * step);
            ok = ok && mbar_wait(smem_u32(&full[group][0]), uint32_t(i & 1), status);
            const float total = across_group(warp_sum(sum_of(0, f32x2::both(r))), i);
            if (t == 0 && ok && i + 1 < n_mine) load(i + 1, 0);        // every warp has read the row
            if (a.dx) dx_of(first + i * step, 0, r, total);
        }
    } else {
        int stage = 0, before = 0;                         // of this row, of the row before
        uint32_t phase = 0;
        float rs = n_mine > 0 ? __ldg(rs_p) : 0.0f;
        for (int i = 0; i < n_mine; ++i) {
            const float r = rs;
            const uint32_t here = uint32_t(stage) * stage_bytes;
            if (i + 1 < n_mine) rs = __ldg(rs_p + (i + 1) * step);
            ok = ok && mbar_wait(smem_u32(&full[group][stage]), phase, status);
            const float total = across_group(warp_sum(sum_of(here, f32x2::both(r))), i);
            // (every warp is past the row before)
            if (t == 0 && ok && i > 0 && i - 1 + sh.stages < n_mine) load(i - 1 + sh.stages, before);
            if (a.dx) dx_of(first + i * step, here, r, total);
            before = stage;
            if (++stage == sh.stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
    }
    if (!ok && t == 0)                                     // gave up: let the copies in flight land
        for (int q = 0; q < sh.stages && q < n_mine; ++q)
            for (uint32_t p = 0; p < 2; ++p) mbar_wait(smem_u32(&full[group][q]), p, status, 1000000ull);
    __syncthreads();                                       // (every copy has landed and been read)
    if (!a.dgamma) return;
    // the groups' column sums meet in the ring and are added in group order
    float* sums = reinterpret_cast<float*>(smem);
    const int cols = sh.nvec * V::kN;
#pragma unroll
    for (int v = 0; v < kV; ++v)
        if (live[v]) {
#pragma unroll
            for (int k = 0; k < V::kPairs; ++k)
                *reinterpret_cast<uint64_t*>(sums + group * cols + (t + v * sh.group) * V::kN + 2 * k) = dga[v][k];
        }
    __syncthreads();
    for (int col = threadIdx.x; col < cols; col += blockDim.x) {
        float sg = 0.0f;
        for (int q = 0; q < sh.groups; ++q) sg += sums[q * cols + col];
        a.partial[int64_t(blockIdx.x) * a.hidden + col] = sg;
    }
}

// Few rows on 16-byte boundaries: one launch.  dgamma needs no sum over a row's
// elements (rs is given), so the first col_blocks blocks own 8 vectors of columns
// each and add them over all rows, while a block per row computes dx; dy and z come
// from L2 the second time.  (dx may not overlap dy or z here.)  Measured, with dz (us;
// this, the persistent kernel and the join of its blocks' sums): 1 x 7168 bf16 2.9, 6.5;
// 304 x 7168 5.5, 8.8; 512 x 7168 8.6, 11.5; 1000 x 7168 16.5, 17.5; 2000 x 7168 29, 26;
// 512 x 512 4.0, 4.9; 1000 x 512 6.0, 4.9; 512 x 16384 fp32 46, 53: so up to 512 rows.
constexpr int kFewThreads = 512;
constexpr int kFewRows = 512;
constexpr int kFewVectors = 8;                   // of columns per column block: 128 bytes of a row
template <typename T, bool kP32, int kV>
__global__ void __launch_bounds__(kFewThreads, kV <= 4 ? 2 : 1)
rms_backward_few_kernel(const RmsBackwardArgs a, int nvec, int col_blocks) {
    using V = Vec<T>;
    constexpr int kCols = kFewVectors * V::kN;
    __shared__ float cols[kFewThreads / 32][kCols];
    __shared__ float part[32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const uint4* dy = static_cast<const uint4*>(a.dy);
    const uint4* z = static_cast<const uint4*>(a.z);
    const int64_t pitch_dy = a.ld_dy * int64_t(sizeof(T)) / 16, pitch_z = a.ld_z * int64_t(sizeof(T)) / 16;
    if (int(blockIdx.x) < col_blocks) {
        const int vec = int(blockIdx.x) * kFewVectors + lane % kFewVectors, groups = blockDim.x / kFewVectors;
        uint64_t dga[V::kPairs];
#pragma unroll
        for (int k = 0; k < V::kPairs; ++k) dga[k] = 0;
        if (vec < nvec)
            for (int64_t r0 = threadIdx.x / kFewVectors; r0 < a.rows; r0 += 4 * groups) {       // four rows in flight
                uint4 wd[4], wz[4];
                float rs[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int64_t row = r0 + q * groups;
                    const bool live = row < a.rows;
                    wd[q] = live ? dy[row * pitch_dy + vec] : make_uint4(0, 0, 0, 0);
                    wz[q] = live ? z[row * pitch_z + vec] : make_uint4(0, 0, 0, 0);
                    rs[q] = live ? a.rsigma[row] : 0.0f;
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint64_t rs2 = f32x2::both(rs[q]);
#pragma unroll
                    for (int k = 0; k < V::kPairs; ++k)
                        dga[k] = f32x2::fma(V::pair(wd[q], k), f32x2::mul(V::pair(wz[q], k), rs2), dga[k]);
                }
            }
        // the warp's four rows, then the warps in order
#pragma unroll
        for (int k = 0; k < V::kN; ++k) {
            float v = k % 2 ? f32x2::hi(dga[k / 2]) : f32x2::lo(dga[k / 2]);
            v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
            v += __shfl_xor_sync(0xFFFFFFFFu, v, 16);
            if (lane < kFewVectors) cols[warp][lane * V::kN + k] = v;
        }
        __syncthreads();
        for (int c = threadIdx.x; c < kCols; c += blockDim.x) {
            const int64_t col = int64_t(blockIdx.x) * kCols + c;
            if (col >= a.hidden) continue;
            float s = cols[0][c];
            for (int w = 1; w < warps; ++w) s += cols[w][c];
            store_param(a.dgamma, a.param_dtype, col, s);
        }
        return;
    }
    const int64_t row = int(blockIdx.x) - col_blocks;
    const float rs = a.rsigma[row];
    const uint64_t rs2 = f32x2::both(rs);
    const uint4* dz = a.dz ? reinterpret_cast<const uint4*>(static_cast<const T*>(a.dz) + row * a.ld_dz) : nullptr;
    uint4 wd[kV], wz[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        const int i = threadIdx.x + v * blockDim.x;
        wd[v] = i < nvec ? dy[row * pitch_dy + i] : make_uint4(0, 0, 0, 0);
        wz[v] = i < nvec ? z[row * pitch_z + i] : make_uint4(0, 0, 0, 0);
    }
    uint64_t s = 0;
    ParamVec<T, kP32> g;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        const int i = threadIdx.x + v * blockDim.x;
        if (i < nvec) {
            g.load(a.gamma, i);
#pragma unroll
            for (int k = 0; k < V::kPairs; ++k)
                s = f32x2::fma(f32x2::mul(V::pair(wd[v], k), g.pair(k)), f32x2::mul(V::pair(wz[v], k), rs2), s);
        }
    }
    const float c = across_warps(warp_sum(f32x2::lo(s) + f32x2::hi(s)), part, warps, warp, lane) / float(a.hidden);
    const uint64_t k2 = f32x2::both(-rs * c);                // (as in the kernel above)
    uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(a.dx) + row * a.ld_dx);
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        const int i = threadIdx.x + v * blockDim.x;
        if (i < nvec) {
            g.load(a.gamma, i);
            uint4 w = make_uint4(0, 0, 0, 0);
            if (dz) w = dz[i];
            uint64_t o[V::kPairs];
#pragma unroll
            for (int k = 0; k < V::kPairs; ++k) {
                const uint64_t q = f32x2::fma(V::pair(wz[v], k), k2, f32x2::mul(V::pair(wd[v], k), g.pair(k)));
                o[k] = dz ? f32x2::fma(q, rs2, V::pair(w, k)) : f32x2::mul(q, rs2);
            }
            out[i] = V::from_pairs(o);
        }
    }
}

// Rows of up to 512 kE elements in any layout: persistent.  blockDim.x threads own
// the same columns (kE each, element by element) of every row that they take;
// blockDim.y such groups per block, joined at the end.  The next row is loaded before
// the sum of this one crosses the group.  Loads and stores of single elements bound it:
// 4097 x 1023 fp16 with dz 13.9 us (floor 5.0), 8192 x 7167 bf16 152 (69).
template <int kE> constexpr int kAnyBlocks = kE <= 8 ? 2 : 1;          // per SM
template <typename T, typename P, int kE>
__global__ void __launch_bounds__(kAnyThreads, kAnyBlocks<kE>)
rms_backward_any_kernel(const RmsBackwardArgs a) {
    __shared__ float part[2][kAnyThreads / 32];            // by parity of the row
    extern __shared__ float sums[];                        // [blockDim.y][blockDim.x * kE]
    grid_dependency_wait();
    grid_launch_dependents();
    const int hidden = int(a.hidden), t = int(threadIdx.x), tx = int(blockDim.x), group = int(threadIdx.y);
    const int lane = t & 31, gwarps = tx >> 5, gwarp0 = group * gwarps;
    const int64_t first = int64_t(blockIdx.x) * blockDim.y + group, step = int64_t(gridDim.x) * blockDim.y;
    const int n_mine = first < a.rows ? int((a.rows - first + step - 1) / step) : 0;
    float ga[kE], dga[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        const int i = t + e * tx;
        ga[e] = i < hidden ? load_param<P>(a.gamma, i) : 0.0f;
        dga[e] = 0.0f;
    }
    T d[kE], z[kE];
    float rs = 0.0f;
    auto load = [&](int64_t row) {                         // (past the row's end: zeros, so zeros in every sum)
        const T* dy = static_cast<const T*>(a.dy) + row * a.ld_dy + t;
        const T* pz = static_cast<const T*>(a.z) + row * a.ld_z + t;
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            const bool live = t + e * tx < hidden;
            d[e] = live ? dy[e * tx] : from_f32<T>(0.0f);
            z[e] = live ? pz[e * tx] : from_f32<T>(0.0f);
        }
        rs = a.rsigma[row];
    };
    if (n_mine > 0) load(first);
    const float inv_h = 1.0f / float(hidden);
    for (int i = 0; i < n_mine; ++i) {
        const int64_t row = first + i * step;
        const float r = rs;
        float g[kE], xh[kE], s = 0.0f;
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            const float v = to_f32(d[e]);
            xh[e] = to_f32(z[e]) * r;
            g[e] = v * ga[e];
            s = fmaf(g[e], xh[e], s);
            dga[e] = fmaf(v, xh[e], dga[e]);
        }
        T w[kE];
        if (a.dz) {
            const T* dz = static_cast<const T*>(a.dz) + row * a.ld_dz + t;
#pragma unroll
            for (int e = 0; e < kE; ++e) w[e] = t + e * tx < hidden ? dz[e * tx] : from_f32<T>(0.0f);
        }
        if (i + 1 < n_mine) load(row + step);
        float total = warp_sum(s);
        if (gwarps > 1) {
            float* slot = &part[i & 1][gwarp0];            // (read before the next row's barrier, written again after it)
            if (lane == 0) slot[t >> 5] = total;
            group_barrier(1 + group, tx);
            total = warp_sum(lane < gwarps ? slot[lane] : 0.0f);
        }
        const float c = total * inv_h;
        if (a.dx) {
            T* dx = static_cast<T*>(a.dx) + row * a.ld_dx + t;
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                float o = r * (g[e] - xh[e] * c);
                if (a.dz) o += to_f32(w[e]);
                if (t + e * tx < hidden) dx[e * tx] = from_f32<T>(o);
            }
        }
    }
    if (!a.dgamma) return;
    // the groups' column sums, added in group order
#pragma unroll
    for (int e = 0; e < kE; ++e) sums[group * tx * kE + t + e * tx] = dga[e];
    __syncthreads();
    for (int c = group * tx + t; c < hidden; c += tx * int(blockDim.y)) {
        float s = 0.0f;
        for (int q = 0; q < int(blockDim.y); ++q) s += sums[q * tx * kE + c];
        a.partial[int64_t(blockIdx.x) * hidden + c] = s;
    }
}

// Longer rows: a block per row for dx, which reads dy and z twice, and a pass for the
// columns' sums.  Loads of single elements, several in flight, bound them: 1749 x 12998 fp32
// with dz 112 us (floor 54; a load at a time 156), 3000 x 20001 bf16 190 (53; 278).
template <typename T, typename P>
__global__ void __launch_bounds__(kAnyThreads)
rms_backward_dx_kernel(const RmsBackwardArgs a) {
    __shared__ float part[32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t row = blockIdx.x;
    const T* z = static_cast<const T*>(a.z) + row * a.ld_z;
    const T* dy = static_cast<const T*>(a.dy) + row * a.ld_dy;
    const T* dz = a.dz ? static_cast<const T*>(a.dz) + row * a.ld_dz : nullptr;
    T* dx = static_cast<T*>(a.dx) + row * a.ld_dx;
    const float rs = a.rsigma[row];
    T d[kLongAhead], zs[kLongAhead], add[kLongAhead];
    float ga[kLongAhead];
    auto load = [&](int q, int64_t i) {
        d[q] = dy[i];
        zs[q] = z[i];
        ga[q] = load_param<P>(a.gamma, i);
    };
    const float s = long_sum(a.hidden, load, [&](int q, int64_t) { return to_f32(d[q]) * ga[q] * (to_f32(zs[q]) * rs); });
    const float c = across_warps(warp_sum(s), part, kAnyThreads / 32, threadIdx.x >> 5, threadIdx.x & 31) / float(a.hidden);
    for (int64_t i = threadIdx.x; i < a.hidden; i += kLongAhead * kAnyThreads)
        long_batch(i, a.hidden, [&](int q, int64_t at) {
            load(q, at);
            if (dz) add[q] = dz[at];
        }, [&](int q, int64_t at) {
            float o = rs * (to_f32(d[q]) * ga[q] - to_f32(zs[q]) * rs * c);
            if (dz) o += to_f32(add[q]);
            dx[at] = from_f32<T>(o);
        });
}

// Partial sums of dy xh over the rows blockIdx.y, blockIdx.y + parts, ...; a thread
// owns kColsEach columns, kColThreads apart.  Few parts (one, from 1.2 million columns on)
// have many rows each, so a sum is made of batches of kGammaBatch rows, and these of as many
// batches: chains of 64 + 64 + the rest.
constexpr int kColThreads = 256, kColsEach = 2, kGammaBatch = 64;
template <typename T>
__global__ void __launch_bounds__(kColThreads)
rms_backward_gamma_kernel(const RmsBackwardArgs a, int parts) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t c = int64_t(blockIdx.x) * (kColThreads * kColsEach) + threadIdx.x;
    const T* z = static_cast<const T*>(a.z) + c;
    const T* dy = static_cast<const T*>(a.dy) + c;
    float outer[kColsEach], total[kColsEach];
#pragma unroll
    for (int e = 0; e < kColsEach; ++e) outer[e] = total[e] = 0.0f;
    constexpr int kAhead = 4;                              // rows in flight
    int batches = 0;
    for (int64_t r0 = blockIdx.y; r0 < a.rows;) {
        float s[kColsEach];
#pragma unroll
        for (int e = 0; e < kColsEach; ++e) s[e] = 0.0f;
        const int64_t past = r0 + kGammaBatch * int64_t(parts), end = past < a.rows ? past : a.rows;
        for (; r0 < end; r0 += kAhead * int64_t(parts)) {
            T d[kAhead][kColsEach], v[kAhead][kColsEach];
            float rs[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int64_t r = r0 + k * int64_t(parts);
                rs[k] = r < a.rows ? a.rsigma[r] : 0.0f;
#pragma unroll
                for (int e = 0; e < kColsEach; ++e) {
                    const bool live = r < a.rows && c + e * kColThreads < a.hidden;
                    d[k][e] = live ? dy[r * a.ld_dy + e * kColThreads] : from_f32<T>(0.0f);
                    v[k][e] = live ? z[r * a.ld_z + e * kColThreads] : from_f32<T>(0.0f);
                }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
#pragma unroll
                for (int e = 0; e < kColsEach; ++e) s[e] = fmaf(to_f32(d[k][e]), to_f32(v[k][e]) * rs[k], s[e]);
        }
        const bool full = ++batches % kGammaBatch == 0;
#pragma unroll
        for (int e = 0; e < kColsEach; ++e) {
            outer[e] += s[e];
            if (full) {
                total[e] += outer[e];
                outer[e] = 0.0f;
            }
        }
    }
#pragma unroll
    for (int e = 0; e < kColsEach; ++e)
        if (c + e * kColThreads < a.hidden) a.partial[int64_t(blockIdx.y) * a.hidden + c + e * kColThreads] = total[e] + outer[e];
}

// dgamma from `parts` partial sums per column.  A block owns 32 columns (lane =
// column); warp w adds parts w, w + 32, ... in order, then the warps' sums are added
// in warp order.
constexpr int kReduceWarps = 32;
constexpr int kReduceLoads = 5;
__global__ void __launch_bounds__(kReduceWarps * 32)
rms_backward_reduce_kernel(const RmsBackwardArgs a, int parts) {
    __shared__ float sums[kReduceWarps][33];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c = int64_t(blockIdx.x) * 32 + lane;
    float s = 0.0f;
    if (c < a.hidden)
        for (int p0 = warp; p0 < parts; p0 += kReduceLoads * kReduceWarps) {
            float v[kReduceLoads];
#pragma unroll
            for (int k = 0; k < kReduceLoads; ++k) {
                const int64_t p = p0 + k * kReduceWarps;
                v[k] = p < parts ? a.partial[p * a.hidden + c] : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < kReduceLoads; ++k) s += v[k];
        }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < a.hidden) {
        for (int w = 1; w < kReduceWarps; ++w) s += sums[w][lane];
        store_param(a.dgamma, a.param_dtype, c, s);
    }
}

// ---------------------------------------------------------------- launches

template <typename T, bool kP32, int kV, int kMost, bool kOnce>
cudaError_t backward_vec_launch(const RmsBackwardArgs& a, int nvec, int streams, int sms, unsigned int* status, int* parts,
                                cudaStream_t stream) {
    auto kern = rms_backward_vec_kernel<T, kP32, kV, kMost, kOnce>;
    RmsBwdShape sh{};
    sh.nvec = nvec;
    sh.streams = streams;
    const int row_bytes = streams * nvec * 16;
    sh.group = row_threads(nvec, kV);
    sh.groups = kMost / sh.group;
    if (sh.groups > kBwdMaxGroups) sh.groups = kBwdMaxGroups;
    if (sh.groups > a.rows) sh.groups = int(a.rows);
    // (several groups hold 2048 vectors at most between them, so two rows each of three operands fit)
    sh.stages = kOnce ? 1 : kBwdSmem / (sh.groups * row_bytes);
    if (sh.stages > kBwdMaxStages) sh.stages = kBwdMaxStages;
    const int ring = sh.groups * sh.stages * row_bytes, sums = sh.groups * nvec * Vec<T>::kN * 4;
    cudaError_t e = set_smem_attribute_once(reinterpret_cast<const void*>(kern), kBwdSmem);
    if (e != cudaSuccess) return e;
    const int64_t want = (a.rows + sh.groups - 1) / sh.groups;
    int64_t most = sms;
    if (most > rms_backward_parts(a.rows)) most = rms_backward_parts(a.rows);      // (the workspace's rows)
    *parts = int(want < most ? want : most);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(*parts));
    cfg.blockDim = dim3(unsigned(sh.group * sh.groups));
    cfg.dynamicSmemBytes = size_t(ring > sums ? ring : sums);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a, sh, status);
}

// Vectors of a row that the ring kernel takes: kBwdV<T> in each of up to 896 threads, or
// twice as many in each of 512 (both hold their sums and gamma in registers); 128 KB of
// dy and z at most (64 KB of 16-bit elements, so three operands' rows fit twice).
template <typename T> constexpr int kBwdV = sizeof(T) == 4 ? 4 : 2;
template <typename T> constexpr int kBwdMostVectors = 2 * kBwdV<T> * 512;

template <typename T, bool kP32>
cudaError_t backward_vec(const RmsBackwardArgs& a, int sms, unsigned int* status, int* parts, cudaStream_t stream) {
    constexpr int kV = kBwdV<T>;
    const int nvec = int(a.hidden / Vec<T>::kN);
    // (dz in the ring too where two rows then fit)
    const int streams = a.dz && 2 * 3 * 16 * nvec <= kBwdSmem ? 3 : 2;
    if (nvec <= kV * 512) return backward_vec_launch<T, kP32, kV, 512, false>(a, nvec, streams, sms, status, parts, stream);
    if constexpr (sizeof(T) == 4) {
        // (from 3201 vectors on two rows of dy and z do not fit)
        if (2 * 2 * 16 * nvec <= kBwdSmem) return backward_vec_launch<T, kP32, kV, 896, false>(a, nvec, streams, sms, status, parts, stream);
        return backward_vec_launch<T, kP32, 2 * kV, 512, true>(a, nvec, 2, sms, status, parts, stream);
    } else {
        if (nvec <= kV * 896) return backward_vec_launch<T, kP32, kV, 896, false>(a, nvec, streams, sms, status, parts, stream);
        return backward_vec_launch<T, kP32, 2 * kV, 512, false>(a, nvec, streams, sms, status, parts, stream);
    }
}

// One launch for dx and dgamma: see rms_backward_few_kernel.  (Up to kBwdMostVectors: more
// than four per thread are rows of fp32.)
template <typename T, bool kP32>
cudaError_t backward_few(const RmsBackwardArgs& a, cudaStream_t stream) {
    const int nvec = int(a.hidden / Vec<T>::kN);
    const int v = nvec <= 512 ? 1 : nvec <= 1024 ? 2 : nvec <= 2048 ? 4 : 8;
    int threads = row_threads(nvec, v);
    if (threads < 256) threads = 256;                      // (row groups of the column blocks)
    const int col_blocks = a.dgamma ? (nvec + kFewVectors - 1) / kFewVectors : 0;
    const dim3 grid(unsigned(col_blocks + (a.dx ? a.rows : 0))), block{unsigned(threads)};
    if (v == 1) return launch_dependent(rms_backward_few_kernel<T, kP32, 1>, grid, block, stream, a, nvec, col_blocks);
    if (v == 2) return launch_dependent(rms_backward_few_kernel<T, kP32, 2>, grid, block, stream, a, nvec, col_blocks);
    if constexpr (sizeof(T) == 4)
        if (v == 8) return launch_dependent(rms_backward_few_kernel<T, kP32, 8>, grid, block, stream, a, nvec, col_blocks);
    return launch_dependent(rms_backward_few_kernel<T, kP32, 4>, grid, block, stream, a, nvec, col_blocks);
}

// dx shares memory with dy or z (then the columns' sums must not read after dx is written).
template <typename T>
bool dx_overlaps(const RmsBackwardArgs& a) {
    auto ends = [&](const void* p, int64_t ld) { return static_cast<const T*>(p) + (a.rows - 1) * ld + a.hidden; };
    auto meet = [&](const void* p, int64_t ld) { return p < ends(a.dx, a.ld_dx) && a.dx < ends(p, ld); };
    return a.dx && (meet(a.dy, a.ld_dy) || meet(a.z, a.ld_z));
}

template <typename T, typename P, int kE>
cudaError_t backward_any_launch(const RmsBackwardArgs& a, int sms, int* parts, cudaStream_t stream) {
    const int tx = row_threads(a.hidden, kE);
    int ty = kAnyThreads / tx;
    // (16 at most, a warp each, which need no named barrier; else 8 at most)
    if (ty > a.rows) ty = int(a.rows);
    const int64_t want = (a.rows + ty - 1) / ty;
    int64_t most = int64_t(kAnyBlocks<kE>) * sms;
    if (most > rms_backward_parts(a.rows)) most = rms_backward_parts(a.rows);
    *parts = int(want < most ? want : most);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(*parts));
    cfg.blockDim = dim3(unsigned(tx), unsigned(ty));
    cfg.dynamicSmemBytes = size_t(kE * tx * ty) * sizeof(float);       // (at most 32 KB)
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rms_backward_any_kernel<T, P, kE>, a);
}

template <typename T, typename P>
cudaError_t backward_any(const RmsBackwardArgs& a, int sms, int* parts, cudaStream_t stream) {
    if (a.hidden <= 4 * kAnyThreads) return backward_any_launch<T, P, 4>(a, sms, parts, stream);
    if (a.hidden <= 8 * kAnyThreads) return backward_any_launch<T, P, 8>(a, sms, parts, stream);
    return backward_any_launch<T, P, 16>(a, sms, parts, stream);
}

template <typename T>
cudaError_t backward(const RmsBackwardArgs& a, int sms, unsigned int* status, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    const dim3 reduce_grid(unsigned((a.hidden + 31) / 32));
    const int64_t nvec = a.hidden / Vec<T>::kN;
    auto fits = [&](const void* p, int64_t ld) { return !p || rows_on16(p, ld, a.rows, sizeof(T)); };
    int n = 0;
    if (a.rows > 0 && a.hidden % Vec<T>::kN == 0 && nvec <= kBwdMostVectors<T> && fits(a.z, a.ld_z) && fits(a.dy, a.ld_dy) &&
        fits(a.dz, a.ld_dz) && fits(a.dx, a.ld_dx) && on16(a.gamma)) {
        if (a.rows <= kFewRows && !dx_overlaps<T>(a)) {
            if constexpr (sizeof(T) == 2)
                if (a.param_dtype != TE_MX_FP32) return backward_few<T, false>(a, stream);
            return backward_few<T, true>(a, stream);
        }
        if constexpr (sizeof(T) == 2)
            e = a.param_dtype != TE_MX_FP32 ? backward_vec<T, false>(a, sms, status, &n, stream)
                                            : backward_vec<T, true>(a, sms, status, &n, stream);
        else e = backward_vec<T, true>(a, sms, status, &n, stream);
        if (e != cudaSuccess || !a.dgamma) return e;
        return launch_dependent(rms_backward_reduce_kernel, reduce_grid, dim3(kReduceWarps * 32), stream, a, n);
    }
    if (a.rows > 0 && a.hidden <= 16 * kAnyThreads) {
        e = a.param_dtype == a.dtype ? backward_any<T, T>(a, sms, &n, stream) : backward_any<T, float>(a, sms, &n, stream);
        if (e != cudaSuccess || !a.dgamma) return e;
        return launch_dependent(rms_backward_reduce_kernel, reduce_grid, dim3(kReduceWarps * 32), stream, a, n);
    }
    const unsigned cols = unsigned((a.hidden + kColThreads * kColsEach - 1) / (kColThreads * kColsEach));
    n = rms_backward_parts(a.rows);
    // (blocks for the whole GPU twice over; with as many parts as the workspace holds the
    // partial sums themselves, of 3000 x 20001, cost 20 us)
    if (n > 1 + 16 * sms / int(cols)) n = 1 + 16 * sms / int(cols);
    // (the columns' sums first: dx may overwrite dy or z)
    if (a.dgamma && n > 0) {
        e = launch_dependent(rms_backward_gamma_kernel<T>, dim3(cols, unsigned(n)), dim3(kColThreads), stream, a, n);
        if (e != cudaSuccess) return e;
    }
    if (a.dx && a.rows > 0) {
        const dim3 grid(unsigned(a.rows));
        e = a.param_dtype == a.dtype ? launch_dependent(rms_backward_dx_kernel<T, T>, grid, dim3(kAnyThreads), stream, a)
                                     : launch_dependent(rms_backward_dx_kernel<T, float>, grid, dim3(kAnyThreads), stream, a);
        if (e != cudaSuccess) return e;
    }
    if (!a.dgamma) return e;
    return launch_dependent(rms_backward_reduce_kernel, reduce_grid, dim3(kReduceWarps * 32), stream, a, n);
}

}  // namespace

// Rows of partial sums in the workspace.
int rms_backward_parts(int64_t rows) { return int(rows < kRmsMaxParts ? rows : kRmsMaxParts); }

te_mx_status rms_backward_launch(const RmsBackwardArgs& a, cudaStream_t stream) {
    int sms = 0;
    unsigned int* status = nullptr;
    te_mx_status st = device_sm_count(&sms);
    if (st != TE_MX_OK || (st = device_status_ptr(&status)) != TE_MX_OK) return st;
    cudaError_t e = a.dtype == TE_MX_FP32   ? backward<float>(a, sms, status, stream)
                    : a.dtype == TE_MX_FP16 ? backward<__half>(a, sms, status, stream)
                                            : backward<__nv_bfloat16>(a, sms, status, stream);
    return cuda_status(e, "rmsnorm backward kernel launch");
}

}  // namespace temx
