// Root-mean-square norm with the residual's addition, its output in the
// activations' type and / or MXFP8-quantised.  Over each row of H elements:
//   z = x + residual, rounded to its type (z = x without a residual),
//   rs = 1 / sqrt(sum(z^2) / H + eps),  y = (z rs) gamma.
// Everything between a load and a store is fp32; z and y are rounded
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

// ---------------------------------------------------------------- forward

// Rows on 16-byte boundaries; persistent.  blockDim.x threads hold a row, kV vectors
// each, and later rows' words are in flight while this row's sum crosses the block: the
// next row's x and residual, or the next two rows' x where there is no residual (with
// one row ahead, 28 KB in flight per SM, 8192 x 7168 bf16 took 41.3 us); blockDim.y rows
// per block where a warp holds a row (then no warp waits for another).  The longest
// chain of a sum: 8 kV / 2 + 1 + 5 additions in a warp, 5 over the warps.
// HBM bounds it: 8192 x 7168 bf16 with a residual 74 us (floor 69.4), without 41 (34.7).
// kQuantise (T = bf16): four neighbouring lanes hold an MX block of 32 elements; with a
// residual 65 us (61), without, where instructions bound it, 43 (26).
// kShift: rows of 16-bit elements off 16-byte boundaries, as ShiftedRows (nvec is
// counted here); with a residual (us; this, element by element): 14676 x 4001 bf16 122,
// 208; 16384 x 769 31, 55; 16384 x 257 17, 23; 16384 x 101 9.1, 8.3.
template <typename T, bool kP32, int kV, bool kQuantise, bool kResidual, bool kShift>
__global__ void __launch_bounds__(kMostThreads<kV>, kV == 2 ? 2 : 1)
rms_forward_vec_kernel(const RmsArgs a, int nvec) {
    using V = Vec<T>;
    __shared__ float part[2][32];                          // by parity of the row
    grid_dependency_wait();
    grid_launch_dependents();
    const int t = int(threadIdx.x), tx = int(blockDim.x), lane = t & 31, warp = t >> 5, warps = tx >> 5;
    const int64_t step = int64_t(gridDim.x) * blockDim.y;
    ShiftedRow<T> sr{int(a.hidden), 0};
    if constexpr (kShift) {
        sr.shift = int((int64_t(blockIdx.x) * blockDim.y + threadIdx.y) * a.ld_x % V::kN);
        nvec = sr.vectors();
    }
    constexpr bool kKeep = kV <= 2 || kShift;              // gamma in registers (of more vectors it comes from L1)
    ParamVec<T, kP32> g[kKeep ? kV : 1];
    if constexpr (kKeep) {
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            if constexpr (kShift) sr.template load_params<kP32>(g[v], a.gamma, t + v * tx);
            else g[v].load(a.gamma, t + v * tx < nvec ? t + v * tx : 0);
        }
    }
    auto load = [&](uint4 (&w)[kV], const void* from, int64_t ld, int64_t row) {
        if constexpr (kShift) {
            const T* p = static_cast<const T*>(from) + row * ld;
#pragma unroll
            for (int v = 0; v < kV; ++v) w[v] = t + v * tx < nvec ? sr.load(p, t + v * tx) : make_uint4(0, 0, 0, 0);
        } else {
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const T*>(from) + row * ld);
#pragma unroll
            for (int v = 0; v < kV; ++v) w[v] = t + v * tx < nvec ? __ldcs(p + t + v * tx) : make_uint4(0, 0, 0, 0);
        }
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
                if constexpr (kShift) {
                    if (i < nvec) sr.store(static_cast<T*>(a.z) + row * a.ld_z, i, z[v]);
                } else {
                    if (i < nvec) reinterpret_cast<uint4*>(static_cast<T*>(a.z) + row * a.ld_z)[i] = z[v];
                }
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
            if constexpr (kQuantise && kResidual) unpack_again(z[v]);      // (8192 x 7168: 66.2 -> 65.2 us)
            if constexpr (!kKeep) gv.load(a.gamma, i < nvec ? i : 0);
            uint64_t o[V::kPairs];
#pragma unroll
            for (int k = 0; k < V::kPairs; ++k) o[k] = f32x2::mul(f32x2::mul(V::pair(z[v], k), rs2), gv.pair(k));
            if constexpr (kShift) {
                if (a.y && i < nvec) sr.store(static_cast<T*>(a.y) + row * a.ld_y, i, V::from_pairs(o));
            } else {
                if (a.y && i < nvec) reinterpret_cast<uint4*>(static_cast<T*>(a.y) + row * a.ld_y)[i] = V::from_pairs(o);
            }
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
// gamma in registers.  3001 x 1021 fp16 in pitch 1024, y in pitch 1021: 11.9 us (floor 3.6).
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

// Longer rows: a block per row, which reads it twice, the second time from L1 or
// L2.  (y may be x, and z may be x or the residual: a thread has read an element
// the last time when it writes it.)  1749 x 12998 fp32 with a residual 64 us (floor 54; a
// load at a time 96), 3000 x 20001 bf16 117 (71; 204).
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
    T xs[kLongAhead], res[kLongAhead];
    const float s = long_sum(a.hidden, [&](int q, int64_t i) {
        xs[q] = x[i];
        if (r) res[q] = r[i];
    }, [&](int q, int64_t i) {
        float v = to_f32(xs[q]);
        if (r) {
            const T rounded_z = from_f32<T>(v + to_f32(res[q]));
            z[i] = rounded_z;
            v = to_f32(rounded_z);
        }
        return v * v;
    });
    const float total = across_warps(warp_sum(s), part, kAnyThreads / 32, threadIdx.x >> 5, threadIdx.x & 31);
    const float rs = 1.0f / sqrtf(total / float(a.hidden) + a.eps);
    T* y = static_cast<T*>(a.y) + row * a.ld_y;
    const T* from = z ? z : x;
    float ga[kLongAhead];
    for (int64_t i = threadIdx.x; i < a.hidden; i += kLongAhead * kAnyThreads)
        long_batch(i, a.hidden, [&](int q, int64_t at) {
            xs[q] = from[at];
            ga[q] = load_param<P>(a.gamma, at);
        }, [&](int q, int64_t at) { y[at] = from_f32<T>(to_f32(xs[q]) * rs * ga[q]); });
    if (threadIdx.x == 0 && a.rsigma) a.rsigma[row] = rs;
}

// ---------------------------------------------------------------- column-wise copy

// The column-wise MXFP8 copy of y = z rs gamma (z and rs from the kernel above; its
// programmatic dependent).  A warp takes 32 rows x 64 columns, a lane two columns,
// whose blocks are then its own; four warps stack 128 rows, so that a column's codes
// leave as up to 128 contiguous bytes through shared memory, and its scale bytes four
// at a time (single bytes, a sector of L2 each, took 10 us more).  A block's largest |y| is
// fl(max fl(z rs) gamma): rounding keeps the order, so gamma enters after the maximum.
// Blocks go from the last rows to the first: what the kernel above wrote last is still
// in L2 (it reads x and the residual as data that is not read again).  8192 x 7168: 30.5 us
// (floor 26) with six blocks per SM, 80 registers each; with four, 100 registers, 34 (both
// kernels, six and four: 16384 x 1024 26.9, 27.7; 2048 x 4096 15.4, 15.0; 512 x 4096 7.7, 7.0;
// 160 x 7168 7.6, 7.4); with seven, spilled, 33; half the rows in each half of a warp, 48
// registers, 32.5; four columns x 16 rows per lane 33.  Tried, with four blocks and single
// bytes: persistent with the next tile's words in registers 40, TMA loads and stores in a ring
// per warp 40, both copies in one pass over z in the shared memory of clusters (three blocks of
// 256 threads per SM) 145 to 168 for all of it, against 104 with the two kernels.
constexpr int kColWarps = 4;
template <bool kP32>
__global__ void __launch_bounds__(kColWarps * 32, 6)
rms_colwise_kernel(const RmsArgs a, unsigned col_units) {
    __shared__ __align__(16) uint8_t codes[64][kColWarps * 32 + 16];     // (rows 16 bytes longer: fewer bank conflicts)
    __shared__ __align__(4) uint8_t scales[64][kColWarps];
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
        scales[2 * lane][warp] = uint8_t(s_lo);
        scales[2 * lane + 1][warp] = uint8_t(s_hi);
    }
    __syncthreads();
    if (threadIdx.x < 64 && c0 + threadIdx.x < a.hidden) {
        uint8_t* s = a.s_col + (c0 + threadIdx.x) * a.ld_s_col + (r00 >> 5);
        const int n = a.rows - r00 < kColWarps * 32 ? int(a.rows - r00) / 32 : kColWarps;
        if (n == 4 && (reinterpret_cast<uintptr_t>(s) & 3u) == 0)
            *reinterpret_cast<uint32_t*>(s) = *reinterpret_cast<const uint32_t*>(scales[threadIdx.x]);
        else
            for (int i = 0; i < n; ++i) s[i] = scales[threadIdx.x][i];
    }
    for (int i = threadIdx.x; i < 64 * kColWarps * 2; i += kColWarps * 32) {
        const int col = i / (kColWarps * 2), chunk = i % (kColWarps * 2);
        const int64_t r = r00 + 16 * chunk;
        if (c0 + col < a.hidden && r < a.rows)
            *reinterpret_cast<uint4*>(a.q_col + (c0 + col) * a.rows + r) = *reinterpret_cast<const uint4*>(&codes[col][16 * chunk]);
    }
}

// ---------------------------------------------------------------- launches

// Blocks of `threads` threads that an SM holds, if it holds `most` threads.
int resident(int threads, int most) { return threads > most ? 1 : most / threads > 32 ? 32 : most / threads; }

template <typename T, bool kP32, int kV, bool kQuantise, bool kShift>
cudaError_t forward_vec_launch(const RmsArgs& a, int nvec, int sms, cudaStream_t stream) {
    const int tx = row_threads(nvec, kV), ty = tx == 32 ? 4 : 1;
    int64_t blocks = (a.rows + ty - 1) / ty;
    const int64_t most = int64_t(sms) * (kV > 2 ? (tx * 2 > kThreads ? 1 : 2) : resident(tx * ty, kV == 2 ? 896 : 1024));
    if (blocks > most) blocks = most;
    if (kShift) blocks = blocks_for_shifts(blocks, ty, a.rows);
    const dim3 grid{unsigned(blocks)}, block{unsigned(tx), unsigned(ty)};
    return a.residual ? launch_dependent(rms_forward_vec_kernel<T, kP32, kV, kQuantise, true, kShift>, grid, block, stream, a, nvec)
                      : launch_dependent(rms_forward_vec_kernel<T, kP32, kV, kQuantise, false, kShift>, grid, block, stream, a, nvec);
}

// Vectors per thread: one while there are too few rows to fill the GPU with smaller
// blocks, else two, four or eight as the row needs (eight not with kShift).
template <typename T, bool kP32, bool kQuantise, bool kShift>
cudaError_t forward_vec(const RmsArgs& a, int sms, cudaStream_t stream) {
    // (a shifted row's elements can begin and end within vectors)
    const int nvec = int(kShift ? (a.hidden + 2 * (Vec<T>::kN - 1)) / Vec<T>::kN : a.hidden / Vec<T>::kN);
    if (nvec <= 32 || (a.rows <= 2 * sms && nvec <= 1024)) return forward_vec_launch<T, kP32, 1, kQuantise, kShift>(a, nvec, sms, stream);
    if (nvec <= 2 * kMostThreads<2>) return forward_vec_launch<T, kP32, 2, kQuantise, kShift>(a, nvec, sms, stream);
    if (kShift || nvec <= 4 * kThreads) return forward_vec_launch<T, kP32, 4, kQuantise, kShift>(a, nvec, sms, stream);
    if constexpr (!kShift) return forward_vec_launch<T, kP32, 8, kQuantise, false>(a, nvec, sms, stream);
    return cudaErrorInvalidValue;                          // (not reached)
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

// Elements of a row that four vectors in each of a block's threads hold, whatever its shift.
constexpr int64_t kMostShifted = 4 * kThreads * 8 - 14;
constexpr int64_t kLeastShifted = 192;          // (below, single elements are as fast)

template <typename T>
cudaError_t forward(const RmsArgs& a, int sms, cudaStream_t stream) {
    const int64_t nvec = a.hidden / Vec<T>::kN;
    auto fits = [&](const void* p, int64_t ld) { return !p || rows_on16(p, ld, a.rows, sizeof(T)); };
    if (a.hidden % Vec<T>::kN == 0 && nvec <= 8 * kThreads && fits(a.x, a.ld_x) && fits(a.residual, a.ld_residual) &&
        fits(a.z, a.ld_z) && fits(a.y, a.ld_y) && on16(a.gamma)) {
        if constexpr (sizeof(T) == 2)
            if (a.param_dtype != TE_MX_FP32) return forward_vec<T, false, false, false>(a, sms, stream);
        return forward_vec<T, true, false, false>(a, sms, stream);
    }
    if constexpr (sizeof(T) == 2)
        if (a.rows > 1 && a.hidden >= kLeastShifted && a.hidden <= kMostShifted && shifts_alike<T>(a.x, a.ld_x, a.ld_x) && shifts_alike<T>(a.residual, a.ld_residual, a.ld_x) &&
            shifts_alike<T>(a.z, a.ld_z, a.ld_x) && shifts_alike<T>(a.y, a.ld_y, a.ld_x))
            return a.param_dtype != TE_MX_FP32 ? forward_vec<T, false, false, true>(a, sms, stream)
                                               : forward_vec<T, true, false, true>(a, sms, stream);
    if (a.param_dtype == a.dtype) return forward_any<T, T>(a, sms, stream);
    return forward_any<T, float>(a, sms, stream);
}

}  // namespace

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
    if (a.q_row) e = p32 ? forward_vec<B, true, true, false>(a, sms, stream) : forward_vec<B, false, true, false>(a, sms, stream);
    else e = p32 ? forward_vec<B, true, false, false>(a, sms, stream) : forward_vec<B, false, false, false>(a, sms, stream);
    if (e != cudaSuccess || !a.q_col) return cuda_status(e, "rmsnorm quantize kernel launch");
    const unsigned col_units = unsigned((a.hidden + 63) / 64);
    const int64_t bands = (a.rows + 32 * kColWarps - 1) / (32 * kColWarps);
    const dim3 grid(unsigned(bands * col_units));
    e = p32 ? launch_dependent(rms_colwise_kernel<true>, grid, dim3(kColWarps * 32), stream, a, col_units)
            : launch_dependent(rms_colwise_kernel<false>, grid, dim3(kColWarps * 32), stream, a, col_units);
    return cuda_status(e, "rmsnorm column-wise kernel launch");
}

}  // namespace temx
