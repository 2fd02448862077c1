// LayerNorm whose output keeps the activation's type, and its backward pass
// with the gradients of the scale and the shift.
//
// Forward, over each row of H elements (te.LayerNorm as the drop-in of
// torch.nn.LayerNorm, leeroopedia "FP8 Training Quickstart"; parameters
// 'scale' and 'bias' and epsilon 1e-5, TE "Getting Started" JAX page):
//   mu = sum(x) / H,  var = sum((x - mu)^2) / H,  rs = 1 / sqrt(var + eps),
//   y = (x - mu) rs gamma + beta.
// Backward, with xh = (x - mu) rs and g = dy gamma:
//   dx = rs (g - c1 - xh c2),  c1 = sum(g) / H,  c2 = sum(g xh) / H,
//   dgamma = sum over the rows of dy xh,  dbeta = sum over the rows of dy.
// x, y, dy and dx are bf16, fp16 or fp32; gamma, beta, dgamma and dbeta have
// that type or fp32.  Everything between a load and a store is fp32; each
// result is rounded once, when it is stored.  Each kernel adds in a fixed order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "f32x2.cuh"
#include "ptx.cuh"
#include "temx_internal.h"

namespace temx {

namespace {

// ---------------------------------------------------------------- elements

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Element i of a parameter array of type P.
template <typename P> __device__ __forceinline__ float load_param(const void* p, int64_t i) {
    return to_f32(static_cast<const P*>(p)[i]);
}
__device__ __forceinline__ void store_param(void* p, int dt, int64_t i, float v) {
    if (dt == TE_MX_FP32) static_cast<float*>(p)[i] = v;
    else if (dt == TE_MX_FP16) static_cast<__half*>(p)[i] = from_f32<__half>(v);
    else static_cast<__nv_bfloat16*>(p)[i] = from_f32<__nv_bfloat16>(v);
}

// Warp sum in a fixed butterfly order (every lane gets the same value).
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sum over the blockDim.x threads of a row (the same value in each, a fixed
// order).  `red`: one float per warp, used once between block barriers.
__device__ __forceinline__ float row_sum(float v, float* red) {
    v = warp_sum(v);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < warps; ++w) s += red[w];
    return s;
}

constexpr int kRowThreads = 256;

// ---------------------------------------------------------------- 16-byte vectors

// A 16-byte vector of T as kPairs packed fp32 pairs, and back (one rounding).
template <typename T> struct Vec {
    static constexpr int kN = 16 / sizeof(T), kPairs = kN / 2;
    static __device__ __forceinline__ uint64_t pair(const uint4& v, int i) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        if constexpr (sizeof(T) == 4) {
            return f32x2::pack(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        } else if constexpr (std::is_same<T, __half>::value) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            return f32x2::pack(f.x, f.y);
        } else {
            return f32x2::pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
        }
    }
    static __device__ __forceinline__ uint4 from_pairs(const uint64_t (&p)[kPairs]) {
        uint32_t w[4];
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                w[2 * i] = uint32_t(p[i]);
                w[2 * i + 1] = uint32_t(p[i] >> 32);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (std::is_same<T, __half>::value)
                    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f32x2::hi(p[i])), "f"(f32x2::lo(p[i])));
                else
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f32x2::hi(p[i])), "f"(f32x2::lo(p[i])));
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// The parameters of the vector's elements: kWords 16-byte loads (two when the
// parameters are fp32 and the activations are not).
template <typename T, bool kP32> struct ParamVec {
    static constexpr int kWords = (kP32 && sizeof(T) == 2) ? 2 : 1;
    uint4 w[kWords];
    __device__ __forceinline__ void load(const void* p, int vec) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = __ldg(static_cast<const uint4*>(p) + vec * kWords + i);
    }
    __device__ __forceinline__ uint64_t pair(int i) const {
        if constexpr (kWords == 2) return Vec<float>::pair(w[i >> 1], i & 1);
        else return Vec<T>::pair(w[0], i);
    }
};

// Forward, rows on 16-byte boundaries.  blockDim.x threads hold a row in
// registers, kV vectors each, so x is read once; blockDim.y rows per block
// (one unless a warp holds a row).  The longest chain of a sum has 8 kV / 2 +
// 1 + 5 additions in a warp and 32 over the warps.
template <typename T, bool kP32, int kV>
__global__ void __launch_bounds__(1024)
ln_forward_vec_kernel(const LnArgs a, int nvec) {
    using V = Vec<T>;
    __shared__ float red[2][32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    if (row >= a.rows) return;                       // (blockDim.y > 1: a whole warp, no barriers follow)
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + row * a.ld_x);
    uint4 xr[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        const int i = threadIdx.x + v * blockDim.x;
        xr[v] = i < nvec ? x[i] : make_uint4(0, 0, 0, 0);
    }
    ParamVec<T, kP32> g, b;
    auto load_params = [&](int i) {
        g.load(a.gamma, i);
        if (a.beta) b.load(a.beta, i);
    };
    if constexpr (kV == 1)                           // (in flight during the sums; more would cost registers)
        if (threadIdx.x < nvec) load_params(threadIdx.x);
    uint64_t s = 0;
#pragma unroll
    for (int v = 0; v < kV; ++v)
#pragma unroll
        for (int i = 0; i < V::kPairs; ++i) s = f32x2::add(s, V::pair(xr[v], i));
    const float mu = row_sum(f32x2::lo(s) + f32x2::hi(s), red[0]) / float(a.hidden);
    const uint64_t mu2 = f32x2::both(mu);
    s = 0;
#pragma unroll
    for (int v = 0; v < kV; ++v)
        if (threadIdx.x + v * blockDim.x < nvec) {
#pragma unroll
            for (int i = 0; i < V::kPairs; ++i) {
                const uint64_t d = f32x2::sub(V::pair(xr[v], i), mu2);
                s = f32x2::fma(d, d, s);
            }
        }
    const float rs = 1.0f / sqrtf(row_sum(f32x2::lo(s) + f32x2::hi(s), red[1]) / float(a.hidden) + a.eps);
    const uint64_t rs2 = f32x2::both(rs);
    uint4* y = reinterpret_cast<uint4*>(static_cast<T*>(a.y) + row * a.ld_y);
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        const int i = threadIdx.x + v * blockDim.x;
        if (i < nvec) {
            if constexpr (kV > 1) load_params(i);
            uint64_t o[V::kPairs];
#pragma unroll
            for (int k = 0; k < V::kPairs; ++k) {
                const uint64_t xh = f32x2::mul(f32x2::sub(V::pair(xr[v], k), mu2), rs2);
                o[k] = a.beta ? f32x2::fma(xh, g.pair(k), b.pair(k)) : f32x2::mul(xh, g.pair(k));
            }
            y[i] = V::from_pairs(o);
        }
    }
    if (threadIdx.x == 0 && a.mu) {
        a.mu[row] = mu;
        a.rsigma[row] = rs;
    }
}

// ---------------------------------------------------------------- any layout

// Rows of more elements than the persistent kernels for any layout take (below),
// up to 1024 kE: one block per row, whose threads hold it in registers, kE
// elements each, so it is read once.
template <typename T, typename P, int kE>
__global__ void __launch_bounds__(1024)
ln_forward_kernel(const LnArgs a) {
    __shared__ float red[2][32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t row = blockIdx.x;
    const int hidden = int(a.hidden);
    const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
    float v[kE], s = 0.0f;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        const int i = threadIdx.x + e * blockDim.x;
        v[e] = i < hidden ? to_f32(x[i]) : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < kE; ++e) s += v[e];
    const float mu = row_sum(s, red[0]) / float(hidden);
    s = 0.0f;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        const float d = threadIdx.x + e * blockDim.x < hidden ? v[e] - mu : 0.0f;
        s = fmaf(d, d, s);
    }
    const float rs = 1.0f / sqrtf(row_sum(s, red[1]) / float(hidden) + a.eps);
    T* y = static_cast<T*>(a.y) + row * a.ld_y;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        const int i = threadIdx.x + e * blockDim.x;
        if (i < hidden) {
            const float b = a.beta ? load_param<P>(a.beta, i) : 0.0f;
            y[i] = from_f32<T>(fmaf((v[e] - mu) * rs, load_param<P>(a.gamma, i), b));
        }
    }
    if (threadIdx.x == 0 && a.mu) {
        a.mu[row] = mu;
        a.rsigma[row] = rs;
    }
}

template <typename T, typename P, int kE>
__global__ void __launch_bounds__(1024)
ln_backward_dx_kernel(const LnBackwardArgs a) {
    __shared__ float red[2][32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t row = blockIdx.x;
    const int hidden = int(a.hidden);
    const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
    const T* dy = static_cast<const T*>(a.dy) + row * a.ld_dy;
    const float mu = a.mu[row], rs = a.rsigma[row];
    float g[kE], xh[kE], s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        const int i = threadIdx.x + e * blockDim.x;
        const bool live = i < hidden;
        g[e] = live ? to_f32(dy[i]) * load_param<P>(a.gamma, i) : 0.0f;
        xh[e] = live ? (to_f32(x[i]) - mu) * rs : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        s1 += g[e];
        s2 = fmaf(g[e], xh[e], s2);
    }
    const float c1 = row_sum(s1, red[0]) / float(hidden), c2 = row_sum(s2, red[1]) / float(hidden);
    T* dx = static_cast<T*>(a.dx) + row * a.ld_dx;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        const int i = threadIdx.x + e * blockDim.x;
        if (i < hidden) dx[i] = from_f32<T>(rs * (g[e] - c1 - xh[e] * c2));
    }
}

// Rows past what a block's registers hold: the row read three times (forward)
// or twice, the later times from L1 / L2.  Up to 2^24 elements, 65536 in a
// thread: added one after another their sum could be off by 2^-8, so a thread
// adds eight in a tree, 64 trees to a batch, and the batches (at most 3 + 64 + 128
// additions in a chain, 2^-16).
template <int kN, typename F>
__device__ __forceinline__ void long_sums(int64_t hidden, float (&total)[kN], F&& terms) {
    int64_t i = threadIdx.x;
    auto tree = [&](float (&sum)[kN], auto&& live) {
        float v[8][kN];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
#pragma unroll
            for (int n = 0; n < kN; ++n) v[k][n] = 0.0f;
            if (live(k)) terms(i + k * kRowThreads, v[k]);
        }
#pragma unroll
        for (int n = 0; n < kN; ++n)
            sum[n] += ((v[0][n] + v[1][n]) + (v[2][n] + v[3][n])) + ((v[4][n] + v[5][n]) + (v[6][n] + v[7][n]));
        i += 8 * kRowThreads;
    };
#pragma unroll
    for (int n = 0; n < kN; ++n) total[n] = 0.0f;
    for (int64_t left = hidden / (8 * kRowThreads); left > 0; left -= 64) {       // whole trees
        float batch[kN] = {};
        for (int b = left < 64 ? int(left) : 64; b > 0; --b) tree(batch, [](int) { return true; });
#pragma unroll
        for (int n = 0; n < kN; ++n) total[n] += batch[n];
    }
    tree(total, [&](int k) { return i + k * kRowThreads < hidden; });
}

template <typename T, typename P>
__global__ void __launch_bounds__(kRowThreads)
ln_forward_long_kernel(const LnArgs a) {
    __shared__ float red[2][32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
    T* y = static_cast<T*>(a.y) + row * a.ld_y;
    float s[1];
    long_sums(a.hidden, s, [&](int64_t i, float (&v)[1]) { v[0] = to_f32(x[i]); });
    const float mu = row_sum(s[0], red[0]) / float(a.hidden);
    long_sums(a.hidden, s, [&](int64_t i, float (&v)[1]) {
        const float d = to_f32(x[i]) - mu;
        v[0] = d * d;
    });
    const float rs = 1.0f / sqrtf(row_sum(s[0], red[1]) / float(a.hidden) + a.eps);
    for (int64_t i = threadIdx.x; i < a.hidden; i += kRowThreads) {
        const float xh = (to_f32(x[i]) - mu) * rs;
        const float b = a.beta ? load_param<P>(a.beta, i) : 0.0f;
        y[i] = from_f32<T>(fmaf(xh, load_param<P>(a.gamma, i), b));
    }
    if (threadIdx.x == 0 && a.mu) {
        a.mu[row] = mu;
        a.rsigma[row] = rs;
    }
}

// (8 blocks per SM: 2000 x 70001 bf16 388 us, 455 with the 6 that its registers would leave)
template <typename T, typename P>
__global__ void __launch_bounds__(kRowThreads, 8)
ln_backward_dx_long_kernel(const LnBackwardArgs a) {
    __shared__ float red[2][32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
    const T* dy = static_cast<const T*>(a.dy) + row * a.ld_dy;
    T* dx = static_cast<T*>(a.dx) + row * a.ld_dx;
    const float mu = a.mu[row], rs = a.rsigma[row];
    float s[2];
    long_sums(a.hidden, s, [&](int64_t i, float (&v)[2]) {
        v[0] = to_f32(dy[i]) * load_param<P>(a.gamma, i);
        v[1] = v[0] * ((to_f32(x[i]) - mu) * rs);
    });
    const float c1 = row_sum(s[0], red[0]) / float(a.hidden), c2 = row_sum(s[1], red[1]) / float(a.hidden);
    for (int64_t i = threadIdx.x; i < a.hidden; i += kRowThreads) {
        const float g = to_f32(dy[i]) * load_param<P>(a.gamma, i);
        const float xh = (to_f32(x[i]) - mu) * rs;
        dx[i] = from_f32<T>(rs * (g - c1 - xh * c2));
    }
}

// Partial sums of dy xh and dy over the rows blockIdx.y, blockIdx.y + parts,
// ...; a thread owns one column.
template <typename T>
__global__ void __launch_bounds__(kRowThreads)
ln_backward_params_kernel(const LnBackwardArgs a, int parts) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t c = int64_t(blockIdx.x) * kRowThreads + threadIdx.x;
    if (c >= a.hidden) return;
    const T* x = static_cast<const T*>(a.x) + c;
    const T* dy = static_cast<const T*>(a.dy) + c;
    float sg = 0.0f, sb = 0.0f;
    for (int64_t r0 = blockIdx.y; r0 < a.rows; r0 += 4 * int64_t(parts)) {         // four rows in flight
        float d[4], xh[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t r = r0 + k * int64_t(parts);
            const bool live = r < a.rows;
            d[k] = live ? to_f32(dy[r * a.ld_dy]) : 0.0f;
            xh[k] = live ? (to_f32(x[r * a.ld_x]) - a.mu[r]) * a.rsigma[r] : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            sg = fmaf(d[k], xh[k], sg);
            sb += d[k];
        }
    }
    a.partial[(2 * int64_t(blockIdx.y)) * a.hidden + c] = sg;
    a.partial[(2 * int64_t(blockIdx.y) + 1) * a.hidden + c] = sb;
}

// dgamma / dbeta from `parts` partial sums per column.  A block owns 32
// columns (lane = column); warp w adds parts w, w + 32, ... in order, then the
// warps' sums are added in warp order.  The sums come from L2 and the loads'
// latency is what this costs: 32 warps with five loads in flight each hold the
// parts of a block per SM (the whole backward pass, 4096 x 4096 fp32: 37.3 us;
// four loads 37.9, ten 37.0 but 30.4 against 27.4 for 515 x 16384; 8 warps 41.7).
constexpr int kReduceWarps = 32;
constexpr int kReduceLoads = 5;
__global__ void __launch_bounds__(kReduceWarps * 32)
ln_backward_reduce_kernel(const LnBackwardArgs a, int parts) {
    __shared__ float sums[2][kReduceWarps][33];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c = int64_t(blockIdx.x) * 32 + lane;
    float sg = 0.0f, sb = 0.0f;
    if (c < a.hidden)
        for (int p0 = warp; p0 < parts; p0 += kReduceLoads * kReduceWarps) {
            float g[kReduceLoads], b[kReduceLoads];
#pragma unroll
            for (int k = 0; k < kReduceLoads; ++k) {
                const int64_t p = p0 + k * kReduceWarps;
                g[k] = p < parts ? a.partial[2 * p * a.hidden + c] : 0.0f;
                b[k] = p < parts ? a.partial[(2 * p + 1) * a.hidden + c] : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < kReduceLoads; ++k) {
                sg += g[k];
                sb += b[k];
            }
        }
    sums[0][warp][lane] = sg;
    sums[1][warp][lane] = sb;
    __syncthreads();
    if (warp < 2 && c < a.hidden) {
        float s = sums[warp][0][lane];
#pragma unroll
        for (int w = 1; w < kReduceWarps; ++w) s += sums[warp][w][lane];
        if (warp == 0) store_param(a.dgamma, a.param_dtype, c, s);
        else if (a.dbeta) store_param(a.dbeta, a.param_dtype, c, s);
    }
}

// Backward, rows on 16-byte boundaries: one pass over dy and x, persistent.  A
// group of threads owns the same columns (kV vectors per thread) of every row
// that it takes, so the sums of dy xh and dy over the rows stay in registers.
// dy and x come through a ring of rows in shared memory, one bulk copy each,
// and their words stay in registers from the row's sums to its dx.
// Rows past a block's threads are split over a cluster of blocks, which add
// each other's sums with remote stores.  Short rows: several groups per block,
// joined at the end, so that every block leaves one partial sum per column.
// Measured, 8192 x 7168 bf16 (floor 52 us; a plain copy of the bytes 58): 68 us,
// of which 7 go to the column sums' join.  A row's two sums cross the group in
// a dependent chain (shuffles, shared memory, a barrier) that 14 warps cannot
// hide; two rows at a time (78 us), dx a row later (84 us), rows' sums in warps
// of their own (113 us) and four vectors per thread in two groups (77 us) all
// cost more, in registers first: whatever spills misses the L1, which the ring
// leaves small.  fp32 rows take four vectors per thread, as many columns as two
// of 16 bits: 515 x 16384 28 us (two: 44 us, in clusters of four).
constexpr int kBwdMaxGroups = 16;
constexpr int kBwdMaxStages = 16;
constexpr int kBwdSmem = 200 * 1024;             // the ring
constexpr int kBwdMaxCluster = 8;
constexpr int kBwdThreads = 512;                 // 128 registers each
template <typename T> constexpr int kBwdVectors = sizeof(T) == 4 ? 4 : 2;        // per thread

struct LnBwdShape {
    int nvec;        // vectors of a row
    int cvec;        // vectors of a block's part of it
    int group;       // threads per group
    int groups;      // groups per block
    int stages;      // rows of a group's ring
    int cluster;     // blocks per row
};

__device__ __forceinline__ void bulk_load_row(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}
__device__ __forceinline__ uint32_t block_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t remote_smem(uint32_t addr, uint32_t rank) {
    uint32_t d;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(addr), "r"(rank));
    return d;
}
__device__ __forceinline__ void all_blocks_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 8 bytes to a block of the cluster, counted on that block's barrier.
__device__ __forceinline__ void remote_store(uint32_t addr, uint64_t v, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];"
                 :: "r"(addr), "l"(v), "r"(bar) : "memory");
}
__device__ __forceinline__ void group_barrier(int id, int threads) {
    asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(threads) : "memory");
}

// Sums over the warp of two values in one butterfly: lanes 0..15 add up the
// first, lanes 16..31 the second, and return it.
__device__ __forceinline__ float warp_sum2(float a, float b, int lane) {
    float half = (lane < 16 ? a : b) + __shfl_xor_sync(0xFFFFFFFFu, lane < 16 ? b : a, 16);
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) half += __shfl_xor_sync(0xFFFFFFFFu, half, o);
    return half;
}

template <typename T, bool kP32, bool kCluster>
__global__ void __launch_bounds__(kBwdThreads, 1)
ln_backward_vec_kernel(const LnBackwardArgs a, const LnBwdShape sh, unsigned int* status) {
    using V = Vec<T>;
    constexpr int kV = kBwdVectors<T>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t full[kBwdMaxGroups][kBwdMaxStages];          // a row's dy and x landed
    __shared__ __align__(8) uint64_t joined[2];                                   // every block's sums of a row are there
    __shared__ __align__(8) float warp_part[2][kBwdThreads / 32][2];              // by parity of the row
    __shared__ __align__(8) float block_part[2][kBwdMaxCluster][2];

    const int group = threadIdx.x / sh.group, t = threadIdx.x % sh.group, lane = threadIdx.x & 31;
    const int gwarps = sh.group >> 5, gwarp0 = group * gwarps;
    const uint32_t rank = kCluster ? block_rank() : 0u;
    const int unit = int(blockIdx.x) / sh.cluster, units = int(gridDim.x) / sh.cluster;
    const int vec0 = int(rank) * sh.cvec, mine = min(sh.cvec, sh.nvec - vec0);      // this block's vectors
    const uint32_t bytes = uint32_t(mine) * 16, stage_bytes = uint32_t(sh.cvec) * 32;     // dy, then x
    const uint32_t ring = smem_u32(smem) + uint32_t(group * sh.stages) * stage_bytes;
    // rows first, first + step, ... of this group (every block of a cluster: the same)
    const int64_t first = int64_t(unit) * sh.groups + group, step = int64_t(units) * sh.groups;
    const int n_mine = first < a.rows ? int((a.rows - first + step - 1) / step) : 0;
    if (t == 0)
        for (int i = 0; i < sh.stages; ++i) mbar_init(smem_u32(&full[group][i]), 1);
    if (kCluster && threadIdx.x == 0) {
        mbar_init(smem_u32(&joined[0]), 1);
        mbar_init(smem_u32(&joined[1]), 1);
    }
    if (t == 0) fence_mbarrier_init();
    grid_dependency_wait();
    grid_launch_dependents();
    if constexpr (kCluster) all_blocks_sync();             // the barriers are ready before any remote store
    else __syncthreads();

    auto load = [&](int i, int s) {                        // row i of this group into stage s, by its thread 0
        const int64_t row = first + i * step;
        const uint32_t bar = smem_u32(&full[group][s]), dst = ring + uint32_t(s) * stage_bytes;
        mbar_arrive_expect_tx(bar, 2 * bytes);
        bulk_load_row(dst, static_cast<const T*>(a.dy) + row * a.ld_dy + int64_t(vec0) * V::kN, bytes, bar);
        bulk_load_row(dst + stage_bytes / 2, static_cast<const T*>(a.x) + row * a.ld_x + int64_t(vec0) * V::kN, bytes, bar);
    };
    if (t == 0)
        for (int i = 0; i < sh.stages && i < n_mine; ++i) load(i, i);

    // (threads past the row's end work on its first vector with zeros in dy and
    // gamma, so that nothing below branches; only their stores are left out)
    uint64_t ga[kV][V::kPairs], dga[kV][V::kPairs], dbe[kV][V::kPairs];
    bool live[kV];
    uint32_t at[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        const int j = t + v * sh.group;
        live[v] = j < mine;
        at[v] = ring + 16u * uint32_t(live[v] ? j : 0);
        ParamVec<T, kP32> w;
        w.load(a.gamma, vec0 + (live[v] ? j : 0));
#pragma unroll
        for (int k = 0; k < V::kPairs; ++k) {
            ga[v][k] = live[v] ? w.pair(k) : 0;
            dga[v][k] = dbe[v][k] = 0;
        }
    }
    const float inv_h = 1.0f / float(a.hidden);
    uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(a.dx) + first * a.ld_dx) + vec0 + t;
    const int64_t out_step = step * a.ld_dx * int64_t(sizeof(T)) / 16;
    const float* mu_p = a.mu + first;
    const float* rs_p = a.rsigma + first;
    float mu = n_mine > 0 ? __ldg(mu_p) : 0.0f, rs = n_mine > 0 ? __ldg(rs_p) : 0.0f;
    bool ok = true;                                        // false once a wait gave up: no waits or copies from then on
    int stage = 0;
    uint32_t phase = 0;
    for (int i = 0; i < n_mine; ++i) {
        const float r = rs;
        const uint64_t mu2 = f32x2::both(mu), rs2 = f32x2::both(r);
        ok = ok && mbar_wait(smem_u32(&full[group][stage]), phase, status);
        uint4 wd[kV], wx[kV];
        uint64_t s1 = 0, s2 = 0;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            wd[v] = lds128(at[v] + uint32_t(stage) * stage_bytes);
            wx[v] = lds128(at[v] + uint32_t(stage) * stage_bytes + stage_bytes / 2);
            if (!live[v]) wd[v] = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int k = 0; k < V::kPairs; ++k) {
                const uint64_t d = V::pair(wd[v], k), xh = f32x2::mul(f32x2::sub(V::pair(wx[v], k), mu2), rs2);
                const uint64_t g = f32x2::mul(d, ga[v][k]);
                s1 = f32x2::add(s1, g);
                s2 = f32x2::fma(g, xh, s2);
                dga[v][k] = f32x2::fma(d, xh, dga[v][k]);
                dbe[v][k] = f32x2::add(dbe[v][k], d);
            }
        }
        mu_p += step;
        rs_p += step;
        if (i + 1 < n_mine) {                              // the next row's statistics, a row ahead
            mu = __ldg(mu_p);
            rs = __ldg(rs_p);
        }
        // the row's sums: over the warp, then over the group's warps (every warp
        // adds them up, lane = warp).  A parity's slots are read before the next
        // row's barrier, and written again after it.
        float total = warp_sum2(f32x2::lo(s1) + f32x2::hi(s1), f32x2::lo(s2) + f32x2::hi(s2), lane);
        if (gwarps > 1) {
            float(*part)[2] = &warp_part[i & 1][gwarp0];
            if (lane % 16 == 0) part[t >> 5][lane / 16] = total;
            group_barrier(1 + group, sh.group);
            const float2 f = lane < gwarps ? *reinterpret_cast<const float2*>(part[lane]) : make_float2(0.0f, 0.0f);
            total = warp_sum2(f.x, f.y, lane);
        } else {
            __syncwarp();                                  // every lane has read the stage
        }
        if (t == 0 && ok && i + sh.stages < n_mine) load(i + sh.stages, stage);      // (every warp has read it)
        if (++stage == sh.stages) {
            stage = 0;
            phase ^= 1u;
        }
        float c1 = __shfl_sync(0xFFFFFFFFu, total, 0), c2 = __shfl_sync(0xFFFFFFFFu, total, 16);
        if constexpr (kCluster) {
            // every block's sums to every block; block_part[parity] is written for
            // row i + 2 only by blocks that hold all sums of row i + 1, which every
            // block sent after its barrier of row i + 1, past its reads of row i
            const uint32_t bar = smem_u32(&joined[i & 1]);
            if (t == 0) mbar_arrive_expect_tx(bar, 8u * uint32_t(sh.cluster));
            if (t < sh.cluster)
                remote_store(remote_smem(smem_u32(&block_part[i & 1][rank][0]), uint32_t(t)), f32x2::pack(c1, c2),
                             remote_smem(bar, uint32_t(t)));
            ok = ok && mbar_wait(bar, uint32_t(i >> 1) & 1u, status);
            c1 = c2 = 0.0f;
            for (int b = 0; b < sh.cluster; ++b) {
                c1 += block_part[i & 1][b][0];
                c2 += block_part[i & 1][b][1];
            }
        }
        if (a.dx) {
            // dx = rs g - rs c2 xh - rs c1, xh = (x - mu) rs
            const uint64_t k1 = f32x2::both(-r * (c1 * inv_h)), k2 = f32x2::both(-r * r * (c2 * inv_h));
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                uint64_t o[V::kPairs];
#pragma unroll
                for (int k = 0; k < V::kPairs; ++k)
                    o[k] = f32x2::fma(f32x2::mul(V::pair(wd[v], k), ga[v][k]), rs2,
                                      f32x2::fma(f32x2::sub(V::pair(wx[v], k), mu2), k2, k1));
                if (live[v]) out[v * sh.group] = V::from_pairs(o);
            }
        }
        out += out_step;
    }
    if (!ok && t == 0)                                     // gave up: let the copies in flight land
        for (int s = 0; s < sh.stages && s < n_mine; ++s)
            for (uint32_t q = 0; q < 2; ++q) mbar_wait(smem_u32(&full[group][s]), q, status, 1000000ull);
    __syncthreads();                                       // (every copy has landed and been read)
    if (a.dgamma) {
        // the groups' column sums meet in the ring and are added in group order
        float* sums = reinterpret_cast<float*>(smem);
        const int cols = sh.cvec * V::kN;
#pragma unroll
        for (int v = 0; v < kV; ++v)
            if (live[v]) {
#pragma unroll
                for (int k = 0; k < V::kPairs; ++k) {
                    const int col = (t + v * sh.group) * V::kN + 2 * k;
                    *reinterpret_cast<uint64_t*>(sums + (2 * group) * cols + col) = dga[v][k];
                    *reinterpret_cast<uint64_t*>(sums + (2 * group + 1) * cols + col) = dbe[v][k];
                }
            }
        __syncthreads();
        for (int col = threadIdx.x; col < mine * V::kN; col += blockDim.x) {
            float sg = 0.0f, sb = 0.0f;
            for (int q = 0; q < sh.groups; ++q) {
                sg += sums[(2 * q) * cols + col];
                sb += sums[(2 * q + 1) * cols + col];
            }
            a.partial[(2 * int64_t(unit)) * a.hidden + vec0 * V::kN + col] = sg;
            a.partial[(2 * int64_t(unit) + 1) * a.hidden + vec0 * V::kN + col] = sb;
        }
    }
    if constexpr (kCluster) all_blocks_sync();             // no block leaves while another may still store to it
}

// Backward, few rows on 16-byte boundaries: one launch.  dgamma and dbeta need no
// sums over rows' elements (mu and rsigma are given), so the first col_blocks
// blocks own 8 vectors of columns each and add them over all rows, while a
// block per row computes dx; dy and x come from L2 the second time.  (dx may not
// overlap dy or x here.)  Measured (us; this, the persistent kernel and the join
// of its blocks' sums): 1 x 7168 bf16 2.4, 7.1; 512 x 7168 8.5, 15.2; 2048 x 7168
// 23.1, 27.8; 4096 x 7168 42.5, 42.3; 1000 x 2048 8.5, 10.8; 2000 x 2048 15.5,
// 14.1; 100 x 16384 fp32 12.4, 16.7; 515 x 16384 fp32 32, 28: so up to 304 rows,
// and up to four times the row's vectors where a thread holds at most four of
// them and L2 the rest (few_rows).
constexpr int kFewThreads = 512;
constexpr int kFewRows = 304;
constexpr int kFewVectors = 8;                   // of columns per column block: 128 bytes of a row
template <typename T, bool kP32, int kV>
__global__ void __launch_bounds__(kFewThreads, kV <= 4 ? 2 : 1)
ln_backward_few_kernel(const LnBackwardArgs a, int nvec, int col_blocks) {
    using V = Vec<T>;
    constexpr int kCols = kFewVectors * V::kN;
    __shared__ float cols[2][kFewThreads / 32][kCols];
    __shared__ __align__(8) float part[kFewThreads / 32][2];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const uint4* dy = static_cast<const uint4*>(a.dy);
    const uint4* x = static_cast<const uint4*>(a.x);
    const int64_t pitch_dy = a.ld_dy * int64_t(sizeof(T)) / 16, pitch_x = a.ld_x * int64_t(sizeof(T)) / 16;
    if (int(blockIdx.x) < col_blocks) {
        const int vec = int(blockIdx.x) * kFewVectors + lane % kFewVectors, groups = blockDim.x / kFewVectors;
        uint64_t dga[V::kPairs], dbe[V::kPairs];
#pragma unroll
        for (int k = 0; k < V::kPairs; ++k) dga[k] = dbe[k] = 0;
        if (vec < nvec)
            for (int64_t r0 = threadIdx.x / kFewVectors; r0 < a.rows; r0 += 4 * groups) {       // four rows in flight
                uint4 wd[4], wx[4];
                float mu[4], rs[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int64_t row = r0 + q * groups;
                    const bool live = row < a.rows;
                    wd[q] = live ? dy[row * pitch_dy + vec] : make_uint4(0, 0, 0, 0);
                    wx[q] = live ? x[row * pitch_x + vec] : make_uint4(0, 0, 0, 0);
                    mu[q] = live ? a.mu[row] : 0.0f;
                    rs[q] = live ? a.rsigma[row] : 0.0f;
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint64_t mu2 = f32x2::both(mu[q]), rs2 = f32x2::both(rs[q]);
#pragma unroll
                    for (int k = 0; k < V::kPairs; ++k) {
                        const uint64_t d = V::pair(wd[q], k);
                        dga[k] = f32x2::fma(d, f32x2::mul(f32x2::sub(V::pair(wx[q], k), mu2), rs2), dga[k]);
                        dbe[k] = f32x2::add(dbe[k], d);
                    }
                }
            }
        // the warp's four rows, then the warps in order
        float v[2][V::kN];
#pragma unroll
        for (int k = 0; k < V::kPairs; ++k) {
            v[0][2 * k] = f32x2::lo(dga[k]);
            v[0][2 * k + 1] = f32x2::hi(dga[k]);
            v[1][2 * k] = f32x2::lo(dbe[k]);
            v[1][2 * k + 1] = f32x2::hi(dbe[k]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < V::kN; ++k) {
                v[h][k] += __shfl_xor_sync(0xFFFFFFFFu, v[h][k], 8);
                v[h][k] += __shfl_xor_sync(0xFFFFFFFFu, v[h][k], 16);
                if (lane < kFewVectors) cols[h][warp][lane * V::kN + k] = v[h][k];
            }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * kCols; i += blockDim.x) {
            const int h = i / kCols, c = i % kCols;
            const int64_t col = int64_t(blockIdx.x) * kCols + c;
            if (col >= a.hidden) continue;
            float s = cols[h][0][c];
            for (int w = 1; w < warps; ++w) s += cols[h][w][c];
            if (h == 0) store_param(a.dgamma, a.param_dtype, col, s);
            else if (a.dbeta) store_param(a.dbeta, a.param_dtype, col, s);
        }
        return;
    }
    const int64_t row = int(blockIdx.x) - col_blocks;
    const float mu = a.mu[row], rs = a.rsigma[row];
    const uint64_t mu2 = f32x2::both(mu), rs2 = f32x2::both(rs);
    uint4 wd[kV], wx[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        const int i = threadIdx.x + v * blockDim.x;
        wd[v] = i < nvec ? dy[row * pitch_dy + i] : make_uint4(0, 0, 0, 0);
        wx[v] = i < nvec ? x[row * pitch_x + i] : make_uint4(0, 0, 0, 0);
    }
    uint64_t s1 = 0, s2 = 0;
    ParamVec<T, kP32> g;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        const int i = threadIdx.x + v * blockDim.x;
        if (i < nvec) {
            g.load(a.gamma, i);
#pragma unroll
            for (int k = 0; k < V::kPairs; ++k) {
                const uint64_t d = f32x2::mul(V::pair(wd[v], k), g.pair(k));
                s1 = f32x2::add(s1, d);
                s2 = f32x2::fma(d, f32x2::mul(f32x2::sub(V::pair(wx[v], k), mu2), rs2), s2);
            }
        }
    }
    float total = warp_sum2(f32x2::lo(s1) + f32x2::hi(s1), f32x2::lo(s2) + f32x2::hi(s2), lane);
    if (lane % 16 == 0) part[warp][lane / 16] = total;
    __syncthreads();
    const float2 f = lane < warps ? *reinterpret_cast<const float2*>(part[lane]) : make_float2(0.0f, 0.0f);
    total = warp_sum2(f.x, f.y, lane);
    const float inv_h = 1.0f / float(a.hidden);
    const float c1 = __shfl_sync(0xFFFFFFFFu, total, 0), c2 = __shfl_sync(0xFFFFFFFFu, total, 16);
    const uint64_t k1 = f32x2::both(-rs * (c1 * inv_h)), k2 = f32x2::both(-rs * rs * (c2 * inv_h));
    uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(a.dx) + row * a.ld_dx);
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        const int i = threadIdx.x + v * blockDim.x;
        if (i < nvec) {
            g.load(a.gamma, i);
            uint64_t o[V::kPairs];
#pragma unroll
            for (int k = 0; k < V::kPairs; ++k)
                o[k] = f32x2::fma(f32x2::mul(V::pair(wd[v], k), g.pair(k)), rs2,
                                  f32x2::fma(f32x2::sub(V::pair(wx[v], k), mu2), k2, k1));
            out[i] = V::from_pairs(o);
        }
    }
}

// Rows of up to 512 kE elements in any layout, backward: persistent.
// blockDim.x threads own the same columns (kE each, element by element) of every
// row that they take, so dy and x are read once and the columns' sums stay in
// registers; blockDim.y such groups per block, joined at the end.  The next row
// is loaded before the sums of this one cross the group.  Measured (us; this, a
// pass for dx and one for the columns' sums): 4097 x 1023 fp16 with fp32
// parameters 17.2, 30.5; 5000 x 3001 fp32 49, 141; 1000 x 7001 bf16 30, 56.
constexpr int kAnyThreads = 512;
template <int kE> constexpr int kAnyBlocks = kE <= 4 ? 2 : 1;          // per SM
template <int kE> constexpr bool kAhead = kE <= 8;                     // (more would not fit in the registers)
template <typename T, typename P, int kE>
__global__ void __launch_bounds__(kAnyThreads, kAnyBlocks<kE>)
ln_backward_any_kernel(const LnBackwardArgs a) {
    __shared__ float part[2][kAnyThreads / 32][2];         // by parity of the row
    extern __shared__ float sums[];                        // [2][blockDim.x * blockDim.y * kE]
    grid_dependency_wait();
    grid_launch_dependents();
    const int hidden = int(a.hidden), t = int(threadIdx.x), tx = int(blockDim.x), group = int(threadIdx.y);
    const int lane = t & 31, gwarps = tx >> 5, gwarp0 = group * gwarps;
    const int64_t first = int64_t(blockIdx.x) * blockDim.y + group, step = int64_t(gridDim.x) * blockDim.y;
    const int n_mine = first < a.rows ? int((a.rows - first + step - 1) / step) : 0;
    float ga[kE], dga[kE], dbe[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        const int i = t + e * tx;
        ga[e] = i < hidden ? load_param<P>(a.gamma, i) : 0.0f;
        dga[e] = dbe[e] = 0.0f;
    }
    T d[kE], x[kE];
    float mu = 0.0f, rs = 0.0f;
    auto load = [&](int64_t row) {                         // (past the row's end: zeros in dy, so zeros in every sum)
        const T* dy = static_cast<const T*>(a.dy) + row * a.ld_dy + t;
        const T* px = static_cast<const T*>(a.x) + row * a.ld_x + t;
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            const bool live = t + e * tx < hidden;
            d[e] = live ? dy[e * tx] : from_f32<T>(0.0f);
            x[e] = live ? px[e * tx] : from_f32<T>(0.0f);
        }
        mu = a.mu[row];
        rs = a.rsigma[row];
    };
    if (n_mine > 0) load(first);
    const float inv_h = 1.0f / float(hidden);
    for (int i = 0; i < n_mine; ++i) {
        const int64_t row = first + i * step;
        const float m = mu, r = rs;
        float g[kE], xh[kE], s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            const float v = to_f32(d[e]);
            xh[e] = t + e * tx < hidden ? (to_f32(x[e]) - m) * r : 0.0f;
            g[e] = v * ga[e];
            s1 += g[e];
            s2 = fmaf(g[e], xh[e], s2);
            dga[e] = fmaf(v, xh[e], dga[e]);
            dbe[e] += v;
        }
        if (kAhead<kE> && i + 1 < n_mine) load(row + step);
        float total = warp_sum2(s1, s2, lane);
        if (gwarps > 1) {
            float(*slot)[2] = &part[i & 1][gwarp0];        // (read before the next row's barrier, written again after it)
            if (lane % 16 == 0) slot[t >> 5][lane / 16] = total;
            group_barrier(1 + group, tx);
            const float2 f = lane < gwarps ? make_float2(slot[lane][0], slot[lane][1]) : make_float2(0.0f, 0.0f);
            total = warp_sum2(f.x, f.y, lane);
        }
        const float c1 = __shfl_sync(0xFFFFFFFFu, total, 0) * inv_h, c2 = __shfl_sync(0xFFFFFFFFu, total, 16) * inv_h;
        if (a.dx) {
            T* dx = static_cast<T*>(a.dx) + row * a.ld_dx + t;
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                if constexpr (!kAhead<kE>) {               // (from the words again, not kept)
                    g[e] = to_f32(d[e]) * ga[e];
                    xh[e] = (to_f32(x[e]) - m) * r;
                }
                if (t + e * tx < hidden) dx[e * tx] = from_f32<T>(r * (g[e] - c1 - xh[e] * c2));
            }
        }
        if (!kAhead<kE> && i + 1 < n_mine) load(row + step);
    }
    if (!a.dgamma) return;
    // the groups' column sums, added in group order
    float* sums_b = sums + int(blockDim.y) * tx * kE;
    float* mine = sums + group * tx * kE;
    float* mine_b = sums_b + group * tx * kE;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        mine[t + e * tx] = dga[e];
        mine_b[t + e * tx] = dbe[e];
    }
    __syncthreads();
    for (int c = group * tx + t; c < hidden; c += tx * int(blockDim.y)) {
        float sg = 0.0f, sb = 0.0f;
        for (int q = 0; q < int(blockDim.y); ++q) {
            sg += sums[q * tx * kE + c];
            sb += sums_b[q * tx * kE + c];
        }
        a.partial[2 * int64_t(blockIdx.x) * hidden + c] = sg;
        a.partial[(2 * int64_t(blockIdx.x) + 1) * hidden + c] = sb;
    }
}

// Forward, many long rows on 16-byte boundaries: persistent.  Groups of threads
// take rows in turn, kFwdVectors vectors per thread; rows come through a ring in
// shared memory, one bulk copy each, and gamma and beta stay in registers.
// Measured (us; ring, a block per row, floor): 8192 x 7168 bf16 40.9, 48.4, 34.6
// (a plain copy of the bytes: 38.9); with fp32 parameters 42.2, 57.8; 16384 x
// 3584 43.9, 52.6.  Rows of 256 vectors: 8192 x 2048 17.0, 15.4, so shorter rows
// stay with the block per row.
constexpr int kFwdVectors = 4;
constexpr int kFwdRingVectors = 384;             // vectors of a row from which the ring is used
constexpr int kFwdThreads = 512;
constexpr int kFwdMaxGroups = 16;
constexpr int kFwdMaxStages = 16;
constexpr int kFwdSmem = 200 * 1024;

struct LnFwdShape {
    int nvec;        // vectors of a row
    int group;       // threads per group
    int groups;      // groups per block
    int stages;      // rows of a group's ring
};

// Sum over the `warps` warps of a group (the same value in each thread, a fixed
// order); `part`: 16 slots, zero past the warps.
__device__ __forceinline__ float group_sum(float v, float* part, int warps, int gwarp, int lane, int id, int threads) {
    v = warp_sum(v);
    if (warps == 1) return v;
    if (lane == 0) part[gwarp] = v;
    group_barrier(id, threads);
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float4 f = *reinterpret_cast<const float4*>(part + 4 * k);
        s += (f.x + f.y) + (f.z + f.w);
    }
    return s;
}

template <typename T, bool kP32>
__global__ void __launch_bounds__(kFwdThreads, 1)
ln_forward_ring_kernel(const LnArgs a, const LnFwdShape sh, unsigned int* status) {
    using V = Vec<T>;
    constexpr int kV = kFwdVectors;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t full[kFwdMaxGroups][kFwdMaxStages];
    __shared__ __align__(16) float part[2][kFwdMaxGroups][16];         // of the mean, of the squares

    const int group = threadIdx.x / sh.group, t = threadIdx.x % sh.group, lane = threadIdx.x & 31;
    const int gwarps = sh.group >> 5, gwarp = t >> 5;
    const uint32_t bytes = uint32_t(sh.nvec) * 16;
    const uint32_t ring = smem_u32(smem) + uint32_t(group * sh.stages) * bytes;
    const int64_t first = int64_t(blockIdx.x) * sh.groups + group, step = int64_t(gridDim.x) * sh.groups;
    const int n_mine = first < a.rows ? int((a.rows - first + step - 1) / step) : 0;
    if (t == 0) {
        for (int i = 0; i < sh.stages; ++i) mbar_init(smem_u32(&full[group][i]), 1);
        fence_mbarrier_init();
    }
    if (threadIdx.x < kFwdMaxGroups * 16) (&part[0][0][0])[threadIdx.x] = (&part[1][0][0])[threadIdx.x] = 0.0f;
    grid_dependency_wait();
    grid_launch_dependents();
    __syncthreads();
    auto load = [&](int i, int s) {                        // row i of this group into stage s, by its thread 0
        const uint32_t bar = smem_u32(&full[group][s]);
        mbar_arrive_expect_tx(bar, bytes);
        bulk_load_row(ring + uint32_t(s) * bytes, static_cast<const T*>(a.x) + (first + i * step) * a.ld_x, bytes, bar);
    };
    if (t == 0)
        for (int i = 0; i < sh.stages && i < n_mine; ++i) load(i, i);

    // (threads past the row's end work on its first vector and leave it out of
    // the sums and the stores)
    ParamVec<T, kP32> g[kV], b[kV];
    bool live[kV];
    uint32_t at[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        const int j = t + v * sh.group;
        live[v] = j < sh.nvec;
        at[v] = ring + 16u * uint32_t(live[v] ? j : 0);
        g[v].load(a.gamma, live[v] ? j : 0);
        if (a.beta) b[v].load(a.beta, live[v] ? j : 0);
        else
#pragma unroll
            for (int k = 0; k < ParamVec<T, kP32>::kWords; ++k) b[v].w[k] = make_uint4(0, 0, 0, 0);
    }
    const float inv_h = 1.0f / float(a.hidden);
    uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(a.y) + first * a.ld_y) + t;
    const int64_t out_step = step * a.ld_y * int64_t(sizeof(T)) / 16;
    bool ok = true;                                        // false once a wait gave up: no waits or copies from then on
    int stage = 0;
    uint32_t phase = 0;
    for (int i = 0; i < n_mine; ++i) {
        ok = ok && mbar_wait(smem_u32(&full[group][stage]), phase, status);
        uint4 x[kV];
        uint64_t s[kV];
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            x[v] = lds128(at[v] + uint32_t(stage) * bytes);
            s[v] = 0;
#pragma unroll
            for (int k = 0; k < V::kPairs; ++k) s[v] = f32x2::add(s[v], V::pair(x[v], k));
            if (!live[v]) s[v] = 0;
        }
#pragma unroll
        for (int v = 1; v < kV; ++v) s[0] = f32x2::add(s[0], s[v]);
        const float mu = group_sum(f32x2::lo(s[0]) + f32x2::hi(s[0]), part[0][group], gwarps, gwarp, lane, 1 + group, sh.group) * inv_h;
        if (gwarps == 1) __syncwarp();
        if (t == 0 && ok && i + sh.stages < n_mine) load(i + sh.stages, stage);      // (every warp has read the stage)
        const uint64_t mu2 = f32x2::both(mu);
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            s[v] = 0;
#pragma unroll
            for (int k = 0; k < V::kPairs; ++k) {
                const uint64_t d = f32x2::sub(V::pair(x[v], k), mu2);
                s[v] = f32x2::fma(d, d, s[v]);
            }
            if (!live[v]) s[v] = 0;
        }
#pragma unroll
        for (int v = 1; v < kV; ++v) s[0] = f32x2::add(s[0], s[v]);
        const float var = group_sum(f32x2::lo(s[0]) + f32x2::hi(s[0]), part[1][group], gwarps, gwarp, lane, 1 + group, sh.group) * inv_h;
        const float rs = 1.0f / sqrtf(var + a.eps);
        const uint64_t rs2 = f32x2::both(rs);
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            uint64_t o[V::kPairs];
#pragma unroll
            for (int k = 0; k < V::kPairs; ++k)
                o[k] = f32x2::fma(f32x2::mul(f32x2::sub(V::pair(x[v], k), mu2), rs2), g[v].pair(k), b[v].pair(k));
            if (live[v]) out[v * sh.group] = V::from_pairs(o);
        }
        out += out_step;
        if (t == 0 && a.mu) {
            a.mu[first + i * step] = mu;
            a.rsigma[first + i * step] = rs;
        }
        if (++stage == sh.stages) {
            stage = 0;
            phase ^= 1u;
        }
    }
    if (!ok && t == 0)                                     // gave up: let the copies in flight land
        for (int q = 0; q < sh.stages && q < n_mine; ++q)
            for (uint32_t p = 0; p < 2; ++p) mbar_wait(smem_u32(&full[group][q]), p, status, 1000000ull);
}

// Rows of up to 512 kE elements in any layout, forward: persistent, as the
// backward pass, with gamma and beta in registers.  Bound by the loads and stores
// of single elements.  Measured (us; this, a block per row): 4097 x 1023 fp16 with
// fp32 parameters 11.1, 12.3; 5000 x 3001 fp32 40, 54; 1000 x 7001 bf16 23, 27;
// 16384 x 65 5.6, 17.4.
template <int kE> constexpr int kAnyFwdBlocks = kE <= 8 ? 2 : 1;       // per SM
template <typename T, typename P, int kE>
__global__ void __launch_bounds__(kAnyThreads, kAnyFwdBlocks<kE>)
ln_forward_any_kernel(const LnArgs a) {
    __shared__ __align__(16) float part[2][kAnyThreads / 32][16];      // of the mean, of the squares
    grid_dependency_wait();
    grid_launch_dependents();
    const int hidden = int(a.hidden), t = int(threadIdx.x), tx = int(blockDim.x), group = int(threadIdx.y);
    const int lane = t & 31, gwarps = tx >> 5, gwarp = t >> 5;
    const int64_t first = int64_t(blockIdx.x) * blockDim.y + group, step = int64_t(gridDim.x) * blockDim.y;
    if (t < 16) part[0][group][t] = part[1][group][t] = 0.0f;
    __syncthreads();
    float ga[kE], be[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        const int i = t + e * tx;
        ga[e] = i < hidden ? load_param<P>(a.gamma, i) : 0.0f;
        be[e] = i < hidden && a.beta ? load_param<P>(a.beta, i) : 0.0f;
    }
    T x[kE];
    auto load = [&](int64_t row) {
        const T* px = static_cast<const T*>(a.x) + row * a.ld_x + t;
#pragma unroll
        for (int e = 0; e < kE; ++e) x[e] = t + e * tx < hidden ? px[e * tx] : from_f32<T>(0.0f);
    };
    if (first < a.rows) load(first);
    for (int64_t row = first; row < a.rows; row += step) {
        float v[kE], s = 0.0f;
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            v[e] = to_f32(x[e]);
            s += v[e];
        }
        if (row + step < a.rows) load(row + step);
        const float mu = group_sum(s, part[0][group], gwarps, gwarp, lane, 1 + group, tx) / float(hidden);
        s = 0.0f;
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            const float d = t + e * tx < hidden ? v[e] - mu : 0.0f;
            s = fmaf(d, d, s);
        }
        const float rs = 1.0f / sqrtf(group_sum(s, part[1][group], gwarps, gwarp, lane, 1 + group, tx) / float(hidden) + a.eps);
        T* y = static_cast<T*>(a.y) + row * a.ld_y + t;
#pragma unroll
        for (int e = 0; e < kE; ++e)
            if (t + e * tx < hidden) y[e * tx] = from_f32<T>(fmaf((v[e] - mu) * rs, ga[e], be[e]));
        if (t == 0 && a.mu) {
            a.mu[row] = mu;
            a.rsigma[row] = rs;
        }
    }
}

// ---------------------------------------------------------------- launches

// Launch with programmatic stream serialisation: the blocks may start while
// the previous kernel in the stream finishes (every kernel here waits for it
// before its first access to global memory).
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kern)(P...), dim3 grid, dim3 block, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Threads that hold a row of `hidden` elements, `per` each.
dim3 row_block(int64_t hidden, int64_t per) { return dim3(unsigned((hidden + 32 * per - 1) / (32 * per) * 32)); }

bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
// Rows of a matrix of elements of `size` bytes start on 16-byte boundaries.
bool rows_on16(const void* p, int64_t ld, int64_t rows, size_t size) {
    return on16(p) && (rows == 1 || ld * int64_t(size) % 16 == 0);
}

template <typename T, bool kP32>
cudaError_t forward_ring(const LnArgs& a, const LnFwdShape& sh, int sms, unsigned int* status, cudaStream_t stream) {
    auto kern = ln_forward_ring_kernel<T, kP32>;
    cudaError_t e = set_smem_attribute_once(reinterpret_cast<const void*>(kern), kFwdSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    const int64_t want = (a.rows + sh.groups - 1) / sh.groups;
    cfg.gridDim = dim3(unsigned(want < sms ? want : sms));
    cfg.blockDim = dim3(unsigned(sh.group * sh.groups));
    cfg.dynamicSmemBytes = size_t(sh.groups * sh.stages * sh.nvec * 16);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a, sh, status);
}

template <typename T, bool kP32>
cudaError_t forward_vec(const LnArgs& a, int sms, unsigned int* status, cudaStream_t stream) {
    const int nvec = int(a.hidden / Vec<T>::kN);
    LnFwdShape sh{};
    sh.nvec = nvec;
    constexpr int kV = kFwdVectors;
    sh.group = ((nvec + kV - 1) / kV + 31) / 32 * 32;
    if (sh.group <= kFwdThreads && nvec >= kFwdRingVectors) {
        sh.groups = kFwdThreads / sh.group;
        sh.stages = kFwdSmem / (sh.groups * nvec * 16);
        if (sh.stages > kFwdMaxStages) sh.stages = kFwdMaxStages;
        if (a.rows >= 2 * int64_t(sms) * sh.groups) return forward_ring<T, kP32>(a, sh, sms, status, stream);
    }
    // Threads per row: one vector per thread while there are too few rows to
    // fill the GPU with smaller blocks, else up to four; eight for rows past 2048
    // vectors, so that two blocks fit on an SM (2000 x 16384 fp32: 45 us, four 67;
    // 515 x 16384: 17.9, 23.6), unless a block per SM is all there is (150 x
    // 16384: 9.2, four 7.8).
    const int v = a.rows <= 2 * sms && nvec <= 1024 ? 1 : nvec <= 64 ? 2 : nvec <= 2048 || (nvec <= 4096 && a.rows <= sms) ? 4 : 8;
    const int tx = ((nvec + v - 1) / v + 31) / 32 * 32, ty = tx == 32 ? 4 : 1;
    const dim3 grid(unsigned((a.rows + ty - 1) / ty)), block{unsigned(tx), unsigned(ty)};
    if (v == 1) return launch_dependent(ln_forward_vec_kernel<T, kP32, 1>, grid, block, stream, a, nvec);
    if (v == 2) return launch_dependent(ln_forward_vec_kernel<T, kP32, 2>, grid, block, stream, a, nvec);
    if (v == 4) return launch_dependent(ln_forward_vec_kernel<T, kP32, 4>, grid, block, stream, a, nvec);
    return launch_dependent(ln_forward_vec_kernel<T, kP32, 8>, grid, block, stream, a, nvec);
}

// (a block takes more rows than one at a time once every SM has a block)
template <typename T, typename P, int kE>
cudaError_t forward_any_launch(const LnArgs& a, int sms, cudaStream_t stream) {
    const unsigned tx = row_block(a.hidden, kE).x;
    int64_t ty = a.rows / sms;
    if (ty > kAnyThreads / int(tx)) ty = kAnyThreads / int(tx);
    if (ty < 1) ty = 1;
    int64_t blocks = (a.rows + ty - 1) / ty;
    if (blocks > int64_t(kAnyFwdBlocks<kE>) * sms) blocks = int64_t(kAnyFwdBlocks<kE>) * sms;
    return launch_dependent(ln_forward_any_kernel<T, P, kE>, dim3(unsigned(blocks)), dim3(tx, unsigned(ty)), stream, a);
}

template <typename T, typename P>
cudaError_t forward_any(const LnArgs& a, int sms, cudaStream_t stream) {
    if (a.hidden <= 4 * kAnyThreads) return forward_any_launch<T, P, 4>(a, sms, stream);
    if (a.hidden <= 8 * kAnyThreads) return forward_any_launch<T, P, 8>(a, sms, stream);
    if (a.hidden <= 16 * kAnyThreads) return forward_any_launch<T, P, 16>(a, sms, stream);
    const dim3 grid(unsigned(a.rows));
    if (a.hidden <= 16384) return launch_dependent(ln_forward_kernel<T, P, 16>, grid, row_block(a.hidden, 16), stream, a);
    return launch_dependent(ln_forward_long_kernel<T, P>, grid, dim3(kRowThreads), stream, a);
}

template <typename T>
cudaError_t forward(const LnArgs& a, int sms, unsigned int* status, cudaStream_t stream) {
    const int64_t nvec = a.hidden / Vec<T>::kN;
    if (a.hidden % Vec<T>::kN == 0 && nvec <= 8192 && rows_on16(a.x, a.ld_x, a.rows, sizeof(T)) &&
        rows_on16(a.y, a.ld_y, a.rows, sizeof(T)) && on16(a.gamma) && on16(a.beta)) {
        if constexpr (sizeof(T) == 2)
            if (a.param_dtype != TE_MX_FP32) return forward_vec<T, false>(a, sms, status, stream);
        return forward_vec<T, true>(a, sms, status, stream);
    }
    if (a.param_dtype == a.dtype) return forward_any<T, T>(a, sms, stream);
    return forward_any<T, float>(a, sms, stream);
}

template <typename T, bool kP32, bool kCluster>
cudaError_t backward_vec_launch(const LnBackwardArgs& a, const LnBwdShape& sh, int smem, int sms, unsigned int* status,
                                int* parts, cudaStream_t stream) {
    auto kern = ln_backward_vec_kernel<T, kP32, kCluster>;
    cudaError_t e = set_smem_attribute_once(reinterpret_cast<const void*>(kern), kBwdSmem);
    if (e != cudaSuccess) return e;
    const int64_t want = (a.rows + sh.groups - 1) / sh.groups;
    int64_t most = sms / sh.cluster;
    if (most > ln_backward_parts(a.rows)) most = ln_backward_parts(a.rows);        // (the workspace's rows)
    *parts = int(want < most ? want : most);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(*parts * sh.cluster));
    cfg.blockDim = dim3(unsigned(sh.group * sh.groups));
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(sh.cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kCluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a, sh, status);
}

template <typename T, bool kP32>
cudaError_t backward_vec(const LnBackwardArgs& a, int sms, unsigned int* status, int* parts, cudaStream_t stream) {
    constexpr int kV = kBwdVectors<T>;
    LnBwdShape sh{};
    sh.nvec = int(a.hidden / Vec<T>::kN);
    sh.cluster = 1;
    while (sh.nvec > kV * kBwdThreads * sh.cluster) sh.cluster *= 2;
    sh.cvec = (sh.nvec + sh.cluster - 1) / sh.cluster;
    sh.group = ((sh.cvec + kV - 1) / kV + 31) / 32 * 32;
    sh.groups = sh.cluster > 1 ? 1 : kBwdThreads / sh.group;
    if (sh.groups > kBwdMaxGroups - 1 && sh.group > 32) sh.groups = kBwdMaxGroups - 1;      // (named barriers)
    if (sh.groups > kBwdMaxGroups) sh.groups = kBwdMaxGroups;
    if (sh.groups > a.rows) sh.groups = int(a.rows);
    sh.stages = kBwdSmem / (sh.groups * sh.cvec * 32);
    if (sh.stages > kBwdMaxStages) sh.stages = kBwdMaxStages;
    const int ring = sh.groups * sh.stages * sh.cvec * 32, sums = sh.groups * sh.cvec * Vec<T>::kN * 8;
    const int smem = ring > sums ? ring : sums;
    if (sh.cluster == 1) return backward_vec_launch<T, kP32, false>(a, sh, smem, sms, status, parts, stream);
    return backward_vec_launch<T, kP32, true>(a, sh, smem, sms, status, parts, stream);
}

// One launch for dx and the parameters' gradients: see ln_backward_few_kernel.
bool few_rows(int64_t rows, int64_t nvec) {
    if (nvec > 8 * kFewThreads) return false;
    return rows <= kFewRows || (nvec <= 4 * kFewThreads && rows <= 4 * nvec && rows * nvec <= 3 << 20);
}

template <typename T, bool kP32>
cudaError_t backward_few(const LnBackwardArgs& a, cudaStream_t stream) {
    const int nvec = int(a.hidden / Vec<T>::kN);
    const int v = nvec <= 512 ? 1 : nvec <= 1024 ? 2 : nvec <= 2048 ? 4 : 8;
    int threads = ((nvec + v - 1) / v + 31) / 32 * 32;
    const int least = a.rows <= kFewRows ? 256 : kFewThreads;          // (row groups of the column blocks)
    if (threads < least) threads = least;
    const int col_blocks = a.dgamma ? (nvec + kFewVectors - 1) / kFewVectors : 0;
    const dim3 grid(unsigned(col_blocks + (a.dx ? a.rows : 0))), block{unsigned(threads)};
    if (v == 1) return launch_dependent(ln_backward_few_kernel<T, kP32, 1>, grid, block, stream, a, nvec, col_blocks);
    if (v == 2) return launch_dependent(ln_backward_few_kernel<T, kP32, 2>, grid, block, stream, a, nvec, col_blocks);
    if (v == 4) return launch_dependent(ln_backward_few_kernel<T, kP32, 4>, grid, block, stream, a, nvec, col_blocks);
    return launch_dependent(ln_backward_few_kernel<T, kP32, 8>, grid, block, stream, a, nvec, col_blocks);
}

// dx shares memory with dy or x (then the parameters' sums must not read after dx is written).
template <typename T>
bool dx_overlaps(const LnBackwardArgs& a) {
    auto ends = [&](const void* p, int64_t ld) { return static_cast<const T*>(p) + (a.rows - 1) * ld + a.hidden; };
    auto meet = [&](const void* p, int64_t ld) { return p < ends(a.dx, a.ld_dx) && a.dx < ends(p, ld); };
    return a.dx && (meet(a.dy, a.ld_dy) || meet(a.x, a.ld_x));
}

template <typename T, typename P, int kE>
cudaError_t backward_any_launch(const LnBackwardArgs& a, int sms, int* parts, cudaStream_t stream) {
    const unsigned tx = row_block(a.hidden, kE).x;
    unsigned ty = kAnyThreads / tx;
    if (ty > a.rows) ty = unsigned(a.rows);
    const int64_t want = (a.rows + ty - 1) / ty;
    int64_t most = int64_t(kAnyBlocks<kE>) * sms;
    if (most > ln_backward_parts(a.rows)) most = ln_backward_parts(a.rows);
    *parts = int(want < most ? want : most);
    const size_t smem = size_t(2) * kE * tx * ty * sizeof(float);
    cudaError_t e = set_smem_attribute_once(reinterpret_cast<const void*>(ln_backward_any_kernel<T, P, kE>), 8 * kE * kAnyThreads);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(*parts));
    cfg.blockDim = dim3(tx, ty);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, ln_backward_any_kernel<T, P, kE>, a);
}

template <typename T, typename P>
cudaError_t backward_any(const LnBackwardArgs& a, int sms, int* parts, cudaStream_t stream) {
    if (a.hidden <= 4 * kAnyThreads) return backward_any_launch<T, P, 4>(a, sms, parts, stream);
    if (a.hidden <= 8 * kAnyThreads) return backward_any_launch<T, P, 8>(a, sms, parts, stream);
    return backward_any_launch<T, P, 16>(a, sms, parts, stream);
}

// (longer rows)
template <typename T, typename P>
cudaError_t backward_dx_any(const LnBackwardArgs& a, cudaStream_t stream) {
    const dim3 grid(unsigned(a.rows));
    if (a.hidden <= 16384) return launch_dependent(ln_backward_dx_kernel<T, P, 16>, grid, row_block(a.hidden, 16), stream, a);
    return launch_dependent(ln_backward_dx_long_kernel<T, P>, grid, dim3(kRowThreads), stream, a);
}

template <typename T>
cudaError_t backward(const LnBackwardArgs& a, int sms, unsigned int* status, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    const dim3 reduce_grid(unsigned((a.hidden + 31) / 32));
    if (a.rows > 0 && a.hidden % Vec<T>::kN == 0 && a.hidden / Vec<T>::kN <= kBwdVectors<T> * kBwdThreads * kBwdMaxCluster &&
        rows_on16(a.x, a.ld_x, a.rows, sizeof(T)) && rows_on16(a.dy, a.ld_dy, a.rows, sizeof(T)) &&
        rows_on16(a.dx, a.ld_dx, a.rows, sizeof(T)) && on16(a.gamma)) {
        // (without the parameters' gradients there is nothing to join)
        if ((a.dgamma || a.rows <= kFewRows) && few_rows(a.rows, a.hidden / Vec<T>::kN) && !dx_overlaps<T>(a)) {
            if constexpr (sizeof(T) == 2)
                if (a.param_dtype != TE_MX_FP32) return backward_few<T, false>(a, stream);
            return backward_few<T, true>(a, stream);
        }
        int n = 0;
        if constexpr (sizeof(T) == 2)
            e = a.param_dtype != TE_MX_FP32 ? backward_vec<T, false>(a, sms, status, &n, stream)
                                            : backward_vec<T, true>(a, sms, status, &n, stream);
        else e = backward_vec<T, true>(a, sms, status, &n, stream);
        if (e != cudaSuccess || !a.dgamma) return e;
        return launch_dependent(ln_backward_reduce_kernel, reduce_grid, dim3(kReduceWarps * 32), stream, a, n);
    }
    if (a.rows > 0 && a.hidden <= 16 * kAnyThreads) {
        int n = 0;
        e = a.param_dtype == a.dtype ? backward_any<T, T>(a, sms, &n, stream) : backward_any<T, float>(a, sms, &n, stream);
        if (e != cudaSuccess || !a.dgamma) return e;
        return launch_dependent(ln_backward_reduce_kernel, reduce_grid, dim3(kReduceWarps * 32), stream, a, n);
    }
    const int parts = ln_backward_parts(a.rows);
    // (the parameters' sums first: dx may overwrite dy)
    if (a.dgamma && parts > 0) {
        const unsigned cols = unsigned((a.hidden + kRowThreads - 1) / kRowThreads);
        e = launch_dependent(ln_backward_params_kernel<T>, dim3(cols, unsigned(parts)), dim3(kRowThreads), stream, a, parts);
        if (e != cudaSuccess) return e;
    }
    if (a.dx && a.rows > 0) {
        e = a.param_dtype == a.dtype ? backward_dx_any<T, T>(a, stream) : backward_dx_any<T, float>(a, stream);
        if (e != cudaSuccess) return e;
    }
    if (!a.dgamma) return e;
    return launch_dependent(ln_backward_reduce_kernel, reduce_grid, dim3(kReduceWarps * 32), stream, a, parts);
}

}  // namespace

// Rows of partial sums in the workspace.
int ln_backward_parts(int64_t rows) { return int(rows < kLnMaxParts ? rows : kLnMaxParts); }

te_mx_status ln_forward_launch(const LnArgs& a, cudaStream_t stream) {
    int sms = 0;
    unsigned int* status = nullptr;
    te_mx_status st = device_sm_count(&sms);
    if (st != TE_MX_OK || (st = device_status_ptr(&status)) != TE_MX_OK) return st;
    cudaError_t e = a.dtype == TE_MX_FP32   ? forward<float>(a, sms, status, stream)
                    : a.dtype == TE_MX_FP16 ? forward<__half>(a, sms, status, stream)
                                            : forward<__nv_bfloat16>(a, sms, status, stream);
    return cuda_status(e, "layernorm kernel launch");
}

te_mx_status ln_backward_launch(const LnBackwardArgs& a, cudaStream_t stream) {
    int sms = 0;
    unsigned int* status = nullptr;
    te_mx_status st = device_sm_count(&sms);
    if (st != TE_MX_OK || (st = device_status_ptr(&status)) != TE_MX_OK) return st;
    cudaError_t e = a.dtype == TE_MX_FP32   ? backward<float>(a, sms, status, stream)
                    : a.dtype == TE_MX_FP16 ? backward<__half>(a, sms, status, stream)
                                            : backward<__nv_bfloat16>(a, sms, status, stream);
    return cuda_status(e, "layernorm backward kernel launch");
}

}  // namespace temx
