// Root-mean-square norm with the residual's addition, its output in the
// activations' type and / or MXFP8-quantised, and its backward pass.
//
// Forward, over each row of H elements:
//   z = x + residual, rounded to its type (z = x without a residual),
//   rs = 1 / sqrt(sum(z^2) / H + eps),  y = (z rs) gamma.
// Backward, with xh = z rs and g = dy gamma:
//   dx = rs (g - xh c) + dz,  c = sum(g xh) / H  (the gradient of x and of the
//   residual; dz is the gradient that reaches z by the residual path),
//   dgamma = sum over the rows of dy xh.
// Everything between a load and a store is fp32; z, y, dx and dgamma are rounded
// once, when they are stored.  The norm is that of the rounded z, which is what
// the next layer and the backward pass read.  Quantised copies are made of the
// unrounded y.  Each kernel adds in a fixed order.
#include <cuda_runtime.h>

#include "e4m3.cuh"
#include "f32x2.cuh"
#include "ptx.cuh"
#include "row_ops.cuh"
#include "temx_internal.h"

namespace temx {

namespace {

// Threads of a block, at most, where a thread holds kV vectors (two: 72 registers each
// for two blocks per SM).
constexpr int kThreads = 512;
template <int kV> constexpr int kMostThreads = kV == 1 ? 1024 : kV == 2 ? 448 : kThreads;

// Sum over the block's warps of a value that each warp has summed (the same value
// in each thread, in warp order).  `part`: a slot for each warp; one call between
// two barriers of the block.
__device__ __forceinline__ float across_warps(float v, float* part, int warps, int warp, int lane) {
    if (warps == 1) return v;
    if (lane == 0) part[warp] = v;
    __syncthreads();
    return warp_sum(lane < warps ? part[lane] : 0.0f);
}

// max(|a|, |b|) in magnitude (the sign bit is meaningless); NaN if either is NaN.
__device__ __forceinline__ float maxabs(float a, float b) {
    float d;
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// E8M0 byte of an MX block from its largest magnitude (exponent field - 8, floored
// at 0; 0xFF for NaN and infinities).
__device__ __forceinline__ uint32_t mx_scale_byte(float amax) {
    const uint32_t ef = (__float_as_uint(amax) & 0x7FFFFFFFu) >> 23;
    if (ef == 0xFFu) return 0xFFu;
    return ef > 8u ? ef - 8u : 0u;
}

// A pair, rounded to T and widened again.
template <typename T> __device__ __forceinline__ uint64_t rounded(uint64_t v) {
    return f32x2::pack(to_f32(from_f32<T>(f32x2::lo(v))), to_f32(from_f32<T>(f32x2::hi(v))));
}

// The compiler takes the words for new ones from here on: what it unpacked of them
// before is unpacked again rather than kept in registers.
__device__ __forceinline__ void unpack_again(uint4& w) { asm volatile("" : "+r"(w.x), "+r"(w.y), "+r"(w.z), "+r"(w.w)); }

// ---------------------------------------------------------------- forward

// Rows on 16-byte boundaries; persistent.  blockDim.x threads hold a row, kV vectors
// each, and later rows' words are in flight while this row's sum crosses the block: the
// next row's x and residual, or the next two rows' x where there is no residual (with
// one row ahead, 28 KB in flight per SM, 8192 x 7168 bf16 took 41.3 us); blockDim.y rows
// per block where a warp holds a row (then no warp waits for another).  The longest
// chain of a sum: 8 kV / 2 + 1 + 5 additions in a warp, 5 over the warps.
// kQuantise (T = bf16): four neighbouring lanes hold an MX block of 32 elements.
template <typename T, bool kP32, int kV, bool kQuantise, bool kResidual>
__global__ void __launch_bounds__(kMostThreads<kV>, kV == 2 ? 2 : 1)
rms_forward_vec_kernel(const RmsArgs a, int nvec) {
    using V = Vec<T>;
    __shared__ float part[2][32];                          // by parity of the row
    grid_dependency_wait();
    grid_launch_dependents();
    const int t = int(threadIdx.x), tx = int(blockDim.x), lane = t & 31, warp = t >> 5, warps = tx >> 5;
    const int64_t step = int64_t(gridDim.x) * blockDim.y;
    constexpr bool kKeep = kV <= 2;                        // gamma in registers (of more vectors it comes from L1)
    ParamVec<T, kP32> g[kKeep ? kV : 1];
    if constexpr (kKeep) {
#pragma unroll
        for (int v = 0; v < kV; ++v) g[v].load(a.gamma, t + v * tx < nvec ? t + v * tx : 0);
    }
    auto load = [&](uint4 (&w)[kV], const void* from, int64_t ld, int64_t row) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const T*>(from) + row * ld);
#pragma unroll
        for (int v = 0; v < kV; ++v) w[v] = t + v * tx < nvec ? __ldcs(p + t + v * tx) : make_uint4(0, 0, 0, 0);
    };
    // the row of words x (and residual r), which then hold those of row `next`
    auto one_row = [&](int64_t row, int64_t next, uint4 (&x)[kV], uint4 (&r)[kV], float* slots) {
        uint4 z[kV];
        uint64_t s = 0;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            z[v] = x[v];
            if constexpr (kResidual) {
                uint64_t o[V::kPairs];
#pragma unroll
                for (int k = 0; k < V::kPairs; ++k) o[k] = f32x2::add(V::pair(x[v], k), V::pair(r[v], k));
                z[v] = V::from_pairs(o);
                const int i = t + v * tx;
                if (i < nvec) reinterpret_cast<uint4*>(static_cast<T*>(a.z) + row * a.ld_z)[i] = z[v];
            }
#pragma unroll
            for (int k = 0; k < V::kPairs; ++k) {
                const uint64_t p = V::pair(z[v], k);
                s = f32x2::fma(p, p, s);
            }
        }
        if (next < a.rows) {
            load(x, a.x, a.ld_x, next);
            if constexpr (kResidual) load(r, a.residual, a.ld_residual, next);
        }
        const float total = across_warps(warp_sum(f32x2::lo(s) + f32x2::hi(s)), slots, warps, warp, lane);
        const float rs = 1.0f / sqrtf(total / float(a.hidden) + a.eps);
        if (t == 0 && a.rsigma) a.rsigma[row] = rs;
        const uint64_t rs2 = f32x2::both(rs);
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int i = t + v * tx;
            ParamVec<T, kP32>& gv = g[kKeep ? v : 0];
            if constexpr (!kKeep) gv.load(a.gamma, i < nvec ? i : 0);
            uint64_t o[V::kPairs];
#pragma unroll
            for (int k = 0; k < V::kPairs; ++k) o[k] = f32x2::mul(f32x2::mul(V::pair(z[v], k), rs2), gv.pair(k));
            if (a.y && i < nvec) reinterpret_cast<uint4*>(static_cast<T*>(a.y) + row * a.ld_y)[i] = V::from_pairs(o);
            if constexpr (kQuantise) {
                float m = maxabs(f32x2::lo(o[0]), f32x2::hi(o[0]));
#pragma unroll
                for (int k = 1; k < V::kPairs; ++k) m = maxabs(m, maxabs(f32x2::lo(o[k]), f32x2::hi(o[k])));
                m = maxabs(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
                m = maxabs(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
                const uint32_t sb = mx_scale_byte(m);
                const uint64_t inv = f32x2::both(inv_scale(sb));
                uint32_t c[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint64_t p = f32x2::mul(o[2 * k], inv), q = f32x2::mul(o[2 * k + 1], inv);
                    c[k] = cvt_e4m3x2(f32x2::lo(p), f32x2::hi(p)) | (cvt_e4m3x2(f32x2::lo(q), f32x2::hi(q)) << 16);
                    if (sb == 0xFFu) c[k] = 0x7F7F7F7Fu;
                }
                if (i < nvec) {
                    reinterpret_cast<uint2*>(a.q_row + row * a.hidden)[i] = make_uint2(c[0], c[1]);
                    if ((lane & 3) == 0) a.s_row[row * a.ld_s_row + (i >> 2)] = uint8_t(sb);
                }
            }
        }
    };
    uint4 x[kV], r[kV];                                    // (r: the residual, or the row after x's)
    int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    if (row < a.rows) load(x, a.x, a.ld_x, row);
    if constexpr (kResidual) {
        if (row < a.rows) load(r, a.residual, a.ld_residual, row);
        for (int parity = 0; row < a.rows; row += step, parity ^= 1) one_row(row, row + step, x, r, part[parity]);
    } else {
        if (row + step < a.rows) load(r, a.x, a.ld_x, row + step);
        for (; row < a.rows; row += 2 * step) {
            one_row(row, row + 2 * step, x, x, part[0]);
            if (row + step < a.rows) one_row(row + step, row + 3 * step, r, r, part[1]);
        }
    }
}

// Rows of up to 512 kE elements in any layout: persistent, element by element,
// gamma in registers.
constexpr int kAnyThreads = 512;
template <typename T, typename P, int kE>
__global__ void __launch_bounds__(kAnyThreads, kE <= 8 ? 2 : 1)
rms_forward_any_kernel(const RmsArgs a) {
    __shared__ float part[2][32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int hidden = int(a.hidden), t = int(threadIdx.x), tx = int(blockDim.x);
    const int lane = t & 31, warp = t >> 5, warps = tx >> 5;
    const int64_t first = int64_t(blockIdx.x) * blockDim.y + threadIdx.y, step = int64_t(gridDim.x) * blockDim.y;
    float ga[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) ga[e] = t + e * tx < hidden ? load_param<P>(a.gamma, t + e * tx) : 0.0f;
    T x[kE], r[kE];
    auto load = [&](int64_t row) {
        const T* px = static_cast<const T*>(a.x) + row * a.ld_x + t;
        const T* pr = static_cast<const T*>(a.residual) + row * a.ld_residual + t;
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            const bool live = t + e * tx < hidden;
            x[e] = live ? px[e * tx] : from_f32<T>(0.0f);
            r[e] = live && a.residual ? pr[e * tx] : from_f32<T>(0.0f);
        }
    };
    if (first < a.rows) load(first);
    int parity = 0;
    for (int64_t row = first; row < a.rows; row += step, parity ^= 1) {
        float z[kE], s = 0.0f;
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            z[e] = to_f32(x[e]);
            if (a.residual) {
                const T rounded_z = from_f32<T>(z[e] + to_f32(r[e]));
                z[e] = to_f32(rounded_z);
                if (t + e * tx < hidden) (static_cast<T*>(a.z) + row * a.ld_z)[t + e * tx] = rounded_z;
            }
            s = fmaf(z[e], z[e], s);
        }
        if (row + step < a.rows) load(row + step);
        const float total = across_warps(warp_sum(s), part[parity], warps, warp, lane);
        const float rs = 1.0f / sqrtf(total / float(hidden) + a.eps);
        T* y = static_cast<T*>(a.y) + row * a.ld_y + t;
#pragma unroll
        for (int e = 0; e < kE; ++e)
            if (t + e * tx < hidden) y[e * tx] = from_f32<T>(z[e] * rs * ga[e]);
        if (t == 0 && a.rsigma) a.rsigma[row] = rs;
    }
}

// A thread's sum of terms(i) over i = t, t + kAnyThreads, ...: up to 32768 of them
// (2^24 elements), 64 to a batch, the batches added 64 to a batch of batches, so that a
// chain has at most 64 + 64 + 8 additions.
template <typename F> __device__ __forceinline__ float long_sum(int64_t hidden, F&& term) {
    float total = 0.0f, outer = 0.0f;
    int batches = 0;
    for (int64_t i = threadIdx.x; i < hidden;) {
        float batch = 0.0f;
        for (int k = 0; k < 64 && i < hidden; ++k, i += kAnyThreads) batch += term(i);
        outer += batch;
        if (++batches == 64) {
            total += outer;
            outer = 0.0f;
            batches = 0;
        }
    }
    return total + outer;
}

// Longer rows: a block per row, which reads it twice, the second time from L1 or
// L2.  (y may be x, and z may be x or the residual: a thread has read an element
// the last time when it writes it.)
template <typename T, typename P>
__global__ void __launch_bounds__(kAnyThreads)
rms_forward_long_kernel(const RmsArgs a) {
    __shared__ float part[32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
    const T* r = a.residual ? static_cast<const T*>(a.residual) + row * a.ld_residual : nullptr;
    T* z = a.residual ? static_cast<T*>(a.z) + row * a.ld_z : nullptr;
    const float s = long_sum(a.hidden, [&](int64_t i) {
        float v = to_f32(x[i]);
        if (r) {
            const T rounded_z = from_f32<T>(v + to_f32(r[i]));
            z[i] = rounded_z;
            v = to_f32(rounded_z);
        }
        return v * v;
    });
    const float total = across_warps(warp_sum(s), part, kAnyThreads / 32, threadIdx.x >> 5, threadIdx.x & 31);
    const float rs = 1.0f / sqrtf(total / float(a.hidden) + a.eps);
    T* y = static_cast<T*>(a.y) + row * a.ld_y;
    const T* from = z ? z : x;
    for (int64_t i = threadIdx.x; i < a.hidden; i += kAnyThreads)
        y[i] = from_f32<T>(to_f32(from[i]) * rs * load_param<P>(a.gamma, i));
    if (threadIdx.x == 0 && a.rsigma) a.rsigma[row] = rs;
}

// ---------------------------------------------------------------- column-wise copy

// The column-wise MXFP8 copy of y = z rs gamma (z and rs from the kernel above; its
// programmatic dependent).  A warp takes 32 rows x 64 columns, a lane two columns,
// whose blocks are then its own; four warps stack 128 rows, so that a column's codes
// leave as up to 128 contiguous bytes through shared memory.  A block's largest |y| is
// fl(max fl(z rs) gamma): rounding keeps the order, so gamma enters after the maximum.
// Blocks go from the last rows to the first: what the kernel above wrote last is still
// in L2 (it reads x and the residual as data that is not read again).
constexpr int kColWarps = 4;
template <bool kP32>
__global__ void __launch_bounds__(kColWarps * 32, 4)
rms_colwise_kernel(const RmsArgs a, unsigned col_units) {
    __shared__ __align__(16) uint8_t codes[64][kColWarps * 32 + 16];     // (rows 16 bytes longer: fewer bank conflicts)
    __shared__ __align__(16) float2 rs[kColWarps * 32];    // twice each: a pair
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned block = gridDim.x - 1 - blockIdx.x;
    const int64_t c0 = int64_t(block % col_units) * 64, r00 = int64_t(block / col_units) * (kColWarps * 32);
    const int64_t r0 = r00 + warp * 32, c = c0 + 2 * lane;
    if (r0 < a.rows) {                                     // (rows and hidden are multiples of 32)
        const float mine = a.rsigma[r0 + lane];
        rs[threadIdx.x] = make_float2(mine, mine);
        __syncwarp();
        const bool live = c < a.hidden;
        const int64_t ld = a.residual ? a.ld_z : a.ld_x;
        const uint16_t* z = static_cast<const uint16_t*>(a.residual ? a.z : a.x) + r0 * ld + (live ? c : 0);
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = __ldcs(reinterpret_cast<const uint32_t*>(z + i * ld));
        using P = typename std::conditional<kP32, float, __nv_bfloat16>::type;
        const uint64_t g = live ? f32x2::pack(load_param<P>(a.gamma, c), load_param<P>(a.gamma, c + 1)) : 0;
        const uint32_t rs_at = smem_u32(rs + warp * 32);
        float lo = 0.0f, hi = 0.0f;
        uint64_t y[32];                                    // z rs
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            uint64_t rs_a, rs_b;
            asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(rs_a), "=l"(rs_b) : "r"(rs_at + 8u * i));
            y[i] = f32x2::mul(f32x2::pack(bf16_lo(w[i]), bf16_hi(w[i])), rs_a);
            y[i + 1] = f32x2::mul(f32x2::pack(bf16_lo(w[i + 1]), bf16_hi(w[i + 1])), rs_b);
            lo = maxabs(lo, maxabs(f32x2::lo(y[i]), f32x2::lo(y[i + 1])));
            hi = maxabs(hi, maxabs(f32x2::hi(y[i]), f32x2::hi(y[i + 1])));
        }
        const uint32_t s_lo = mx_scale_byte(lo * f32x2::lo(g)), s_hi = mx_scale_byte(hi * f32x2::hi(g));
        const uint64_t inv = f32x2::pack(inv_scale(s_lo), inv_scale(s_hi));
        uint32_t q_lo[8], q_hi[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint64_t p[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) p[k] = f32x2::mul(f32x2::mul(y[4 * i + k], g), inv);
            q_lo[i] = cvt_e4m3x2(f32x2::lo(p[0]), f32x2::lo(p[1])) | (cvt_e4m3x2(f32x2::lo(p[2]), f32x2::lo(p[3])) << 16);
            q_hi[i] = cvt_e4m3x2(f32x2::hi(p[0]), f32x2::hi(p[1])) | (cvt_e4m3x2(f32x2::hi(p[2]), f32x2::hi(p[3])) << 16);
        }
        if (__any_sync(0xFFFFFFFFu, s_lo == 0xFFu || s_hi == 0xFFu)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (s_lo == 0xFFu) q_lo[i] = 0x7F7F7F7Fu;
                if (s_hi == 0xFFu) q_hi[i] = 0x7F7F7F7Fu;
            }
        }
        uint4* to_lo = reinterpret_cast<uint4*>(&codes[2 * lane][warp * 32]);
        uint4* to_hi = reinterpret_cast<uint4*>(&codes[2 * lane + 1][warp * 32]);
        to_lo[0] = make_uint4(q_lo[0], q_lo[1], q_lo[2], q_lo[3]);
        to_lo[1] = make_uint4(q_lo[4], q_lo[5], q_lo[6], q_lo[7]);
        to_hi[0] = make_uint4(q_hi[0], q_hi[1], q_hi[2], q_hi[3]);
        to_hi[1] = make_uint4(q_hi[4], q_hi[5], q_hi[6], q_hi[7]);
        if (live) {
            uint8_t* s = a.s_col + c * a.ld_s_col + (r0 >> 5);
            s[0] = uint8_t(s_lo);
            s[a.ld_s_col] = uint8_t(s_hi);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 64 * kColWarps * 2; i += kColWarps * 32) {
        const int col = i / (kColWarps * 2), chunk = i % (kColWarps * 2);
        const int64_t r = r00 + 16 * chunk;
        if (c0 + col < a.hidden && r < a.rows)
            *reinterpret_cast<uint4*>(a.q_col + (c0 + col) * a.rows + r) = *reinterpret_cast<const uint4*>(&codes[col][16 * chunk]);
    }
}

// ---------------------------------------------------------------- backward

// Rows on 16-byte boundaries: one pass over dy, z and dz, persistent.  A group of
// threads owns the same columns (kV vectors per thread) of every row that it takes,
// so the sums of dy xh over the rows stay in registers.  The rows come through a ring
// in shared memory, one bulk copy of each operand, and are read there twice: for the
// row's sum, and for its dx once the sum is known, so that no word waits in registers.
// The sum of the next row is taken before the dx of this one, so that its way across
// the warp and the group is hidden behind that; a row's stage is filled again after
// the next row's barrier, which every warp reaches past its last read of the row.
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
    // dx = rs g - rs c xh + dz, xh = z rs
    auto dx_of = [&](int64_t row, uint32_t here, float r, float total) {
        const uint64_t rs2 = f32x2::both(r), k2 = f32x2::both(-r * r * (total * inv_h));
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
                o[k] = f32x2::fma(f32x2::mul(V::pair(d4, k), ga[v].pair(k)), rs2, f32x2::mul(V::pair(z4, k), k2));
                if (dz) o[k] = f32x2::add(o[k], V::pair(w, k));
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
// from L2 the second time.  (dx may not overlap dy or z here.)
constexpr int kFewThreads = 512;
constexpr int kFewRows = 304;
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
    const uint64_t k2 = f32x2::both(-rs * rs * c);
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
                o[k] = f32x2::fma(f32x2::mul(V::pair(wd[v], k), g.pair(k)), rs2, f32x2::mul(V::pair(wz[v], k), k2));
                if (dz) o[k] = f32x2::add(o[k], V::pair(w, k));
            }
            out[i] = V::from_pairs(o);
        }
    }
}

// Rows of up to 512 kE elements in any layout: persistent.  blockDim.x threads own
// the same columns (kE each, element by element) of every row that they take;
// blockDim.y such groups per block, joined at the end.  The next row is loaded before
// the sum of this one crosses the group.
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
// columns' sums.
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
    const float s = long_sum(a.hidden, [&](int64_t i) {
        return to_f32(dy[i]) * load_param<P>(a.gamma, i) * (to_f32(z[i]) * rs);
    });
    const float c = across_warps(warp_sum(s), part, kAnyThreads / 32, threadIdx.x >> 5, threadIdx.x & 31) / float(a.hidden);
    for (int64_t i = threadIdx.x; i < a.hidden; i += kAnyThreads) {
        float o = rs * (to_f32(dy[i]) * load_param<P>(a.gamma, i) - to_f32(z[i]) * rs * c);
        if (dz) o += to_f32(dz[i]);
        dx[i] = from_f32<T>(o);
    }
}

// Partial sums of dy xh over the rows blockIdx.y, blockIdx.y + parts, ...; a thread
// owns one column.
constexpr int kColThreads = 256;
template <typename T>
__global__ void __launch_bounds__(kColThreads)
rms_backward_gamma_kernel(const RmsBackwardArgs a, int parts) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t c = int64_t(blockIdx.x) * kColThreads + threadIdx.x;
    if (c >= a.hidden) return;
    const T* z = static_cast<const T*>(a.z) + c;
    const T* dy = static_cast<const T*>(a.dy) + c;
    float s = 0.0f;
    for (int64_t r0 = blockIdx.y; r0 < a.rows; r0 += 4 * int64_t(parts)) {         // four rows in flight
        float d[4], xh[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t r = r0 + k * int64_t(parts);
            const bool live = r < a.rows;
            d[k] = live ? to_f32(dy[r * a.ld_dy]) : 0.0f;
            xh[k] = live ? to_f32(z[r * a.ld_z]) * a.rsigma[r] : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) s = fmaf(d[k], xh[k], s);
    }
    a.partial[int64_t(blockIdx.y) * a.hidden + c] = s;
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

// Blocks of `threads` threads that an SM holds, if it holds `most` threads.
int resident(int threads, int most) { return threads > most ? 1 : most / threads > 32 ? 32 : most / threads; }

// Threads that hold a row of `n` pieces, `per` each.
int row_threads(int64_t n, int64_t per) { return int((n + 32 * per - 1) / (32 * per) * 32); }

template <typename T, bool kP32, int kV, bool kQuantise>
cudaError_t forward_vec_launch(const RmsArgs& a, int nvec, int sms, cudaStream_t stream) {
    const int tx = row_threads(nvec, kV), ty = tx == 32 ? 4 : 1;
    int64_t blocks = (a.rows + ty - 1) / ty;
    const int64_t most = int64_t(sms) * (kV > 2 ? (tx * 2 > kThreads ? 1 : 2) : resident(tx * ty, kV == 2 ? 896 : 1024));
    if (blocks > most) blocks = most;
    const dim3 grid{unsigned(blocks)}, block{unsigned(tx), unsigned(ty)};
    return a.residual ? launch_dependent(rms_forward_vec_kernel<T, kP32, kV, kQuantise, true>, grid, block, stream, a, nvec)
                      : launch_dependent(rms_forward_vec_kernel<T, kP32, kV, kQuantise, false>, grid, block, stream, a, nvec);
}

// Vectors per thread: one while there are too few rows to fill the GPU with smaller
// blocks, else two, four or eight as the row needs.
template <typename T, bool kP32, bool kQuantise>
cudaError_t forward_vec(const RmsArgs& a, int sms, cudaStream_t stream) {
    const int nvec = int(a.hidden / Vec<T>::kN);
    if (nvec <= 32 || (a.rows <= 2 * sms && nvec <= 1024)) return forward_vec_launch<T, kP32, 1, kQuantise>(a, nvec, sms, stream);
    if (nvec <= 2 * kMostThreads<2>) return forward_vec_launch<T, kP32, 2, kQuantise>(a, nvec, sms, stream);
    if (nvec <= 4 * kThreads) return forward_vec_launch<T, kP32, 4, kQuantise>(a, nvec, sms, stream);
    return forward_vec_launch<T, kP32, 8, kQuantise>(a, nvec, sms, stream);
}

template <typename T, typename P, int kE>
cudaError_t forward_any_launch(const RmsArgs& a, int sms, cudaStream_t stream) {
    const int tx = row_threads(a.hidden, kE), ty = tx == 32 ? 4 : 1;
    int64_t blocks = (a.rows + ty - 1) / ty;
    const int64_t most = int64_t(sms) * (kE > 8 ? 1 : resident(tx * ty, 1024));
    if (blocks > most) blocks = most;
    return launch_dependent(rms_forward_any_kernel<T, P, kE>, dim3(unsigned(blocks)), dim3(unsigned(tx), unsigned(ty)), stream, a);
}

template <typename T, typename P>
cudaError_t forward_any(const RmsArgs& a, int sms, cudaStream_t stream) {
    if (a.hidden <= 4 * kAnyThreads) return forward_any_launch<T, P, 4>(a, sms, stream);
    if (a.hidden <= 8 * kAnyThreads) return forward_any_launch<T, P, 8>(a, sms, stream);
    if (a.hidden <= 16 * kAnyThreads) return forward_any_launch<T, P, 16>(a, sms, stream);
    return launch_dependent(rms_forward_long_kernel<T, P>, dim3(unsigned(a.rows)), dim3(kAnyThreads), stream, a);
}

template <typename T>
cudaError_t forward(const RmsArgs& a, int sms, cudaStream_t stream) {
    const int64_t nvec = a.hidden / Vec<T>::kN;
    auto fits = [&](const void* p, int64_t ld) { return !p || rows_on16(p, ld, a.rows, sizeof(T)); };
    if (a.hidden % Vec<T>::kN == 0 && nvec <= 8 * kThreads && fits(a.x, a.ld_x) && fits(a.residual, a.ld_residual) &&
        fits(a.z, a.ld_z) && fits(a.y, a.ld_y) && on16(a.gamma)) {
        if constexpr (sizeof(T) == 2)
            if (a.param_dtype != TE_MX_FP32) return forward_vec<T, false, false>(a, sms, stream);
        return forward_vec<T, true, false>(a, sms, stream);
    }
    if (a.param_dtype == a.dtype) return forward_any<T, T>(a, sms, stream);
    return forward_any<T, float>(a, sms, stream);
}

template <typename T, bool kP32, int kV, int kMost, bool kOnce>
cudaError_t backward_vec_launch(const RmsBackwardArgs& a, int nvec, int streams, int sms, unsigned int* status, int* parts,
                                cudaStream_t stream) {
    auto kern = rms_backward_vec_kernel<T, kP32, kV, kMost, kOnce>;
    RmsBwdShape sh{};
    sh.nvec = nvec;
    sh.streams = streams;
    const int row_bytes = streams * nvec * 16, least = kOnce ? 1 : 2;
    sh.group = row_threads(nvec, kV);
    sh.groups = kMost / sh.group;
    if (sh.groups > kBwdMaxGroups) sh.groups = kBwdMaxGroups;
    if (sh.groups > a.rows) sh.groups = int(a.rows);
    while (sh.groups > 1 && least * sh.groups * row_bytes > kBwdSmem) --sh.groups;
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
// dy and z at most.
template <typename T> constexpr int kBwdV = sizeof(T) == 4 ? 4 : 2;
template <typename T> constexpr int kBwdMostVectors = 2 * kBwdV<T> * 512;

template <typename T, bool kP32>
cudaError_t backward_vec(const RmsBackwardArgs& a, int sms, unsigned int* status, int* parts, cudaStream_t stream) {
    constexpr int kV = kBwdV<T>;
    const int nvec = int(a.hidden / Vec<T>::kN);
    // (dz in the ring too where two rows then fit)
    const int streams = a.dz && 2 * 3 * 16 * nvec <= kBwdSmem ? 3 : 2;
    if (2 * streams * 16 * nvec > kBwdSmem) return backward_vec_launch<T, kP32, 2 * kV, 512, true>(a, nvec, 2, sms, status, parts, stream);
    if (nvec <= kV * 512) return backward_vec_launch<T, kP32, kV, 512, false>(a, nvec, streams, sms, status, parts, stream);
    if (nvec <= kV * 896) return backward_vec_launch<T, kP32, kV, 896, false>(a, nvec, streams, sms, status, parts, stream);
    return backward_vec_launch<T, kP32, 2 * kV, 512, false>(a, nvec, streams, sms, status, parts, stream);
}

// One launch for dx and dgamma: see rms_backward_few_kernel.
bool few_rows(int64_t rows, int64_t nvec) { return nvec <= 8 * kFewThreads && rows <= kFewRows; }

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
    if (v == 4) return launch_dependent(rms_backward_few_kernel<T, kP32, 4>, grid, block, stream, a, nvec, col_blocks);
    return launch_dependent(rms_backward_few_kernel<T, kP32, 8>, grid, block, stream, a, nvec, col_blocks);
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
    if (ty > 15) ty = tx == 32 ? 16 : 15;                  // (named barriers; a warp alone needs none)
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
        if (few_rows(a.rows, nvec) && !dx_overlaps<T>(a)) {
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
    n = rms_backward_parts(a.rows);
    // (the columns' sums first: dx may overwrite dy or z)
    if (a.dgamma && n > 0) {
        const unsigned cols = unsigned((a.hidden + kColThreads - 1) / kColThreads);
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

// Elements of a row that the quantising kernel holds.
int64_t rms_quantize_max_hidden() { return 8 * kThreads * Vec<__nv_bfloat16>::kN; }

te_mx_status rms_forward_launch(const RmsArgs& a, cudaStream_t stream) {
    int sms = 0;
    te_mx_status st = device_sm_count(&sms);
    if (st != TE_MX_OK) return st;
    cudaError_t e = a.dtype == TE_MX_FP32   ? forward<float>(a, sms, stream)
                    : a.dtype == TE_MX_FP16 ? forward<__half>(a, sms, stream)
                                            : forward<__nv_bfloat16>(a, sms, stream);
    return cuda_status(e, "rmsnorm kernel launch");
}

te_mx_status rms_quantize_launch(const RmsArgs& a, cudaStream_t stream) {
    int sms = 0;
    te_mx_status st = device_sm_count(&sms);
    if (st != TE_MX_OK) return st;
    const bool p32 = a.param_dtype == TE_MX_FP32;
    using B = __nv_bfloat16;
    cudaError_t e;
    if (a.q_row) e = p32 ? forward_vec<B, true, true>(a, sms, stream) : forward_vec<B, false, true>(a, sms, stream);
    else e = p32 ? forward_vec<B, true, false>(a, sms, stream) : forward_vec<B, false, false>(a, sms, stream);
    if (e != cudaSuccess || !a.q_col) return cuda_status(e, "rmsnorm quantize kernel launch");
    const unsigned col_units = unsigned((a.hidden + 63) / 64);
    const int64_t bands = (a.rows + 32 * kColWarps - 1) / (32 * kColWarps);
    const dim3 grid(unsigned(bands * col_units));
    e = p32 ? launch_dependent(rms_colwise_kernel<true>, grid, dim3(kColWarps * 32), stream, a, col_units)
            : launch_dependent(rms_colwise_kernel<false>, grid, dim3(kColWarps * 32), stream, a, col_units);
    return cuda_status(e, "rmsnorm column-wise kernel launch");
}

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
