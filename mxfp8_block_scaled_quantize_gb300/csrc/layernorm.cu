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
// result is rounded once, when it is stored.  Sums are taken in a fixed order.
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

// Element i of a parameter array of runtime type `dt`.
__device__ __forceinline__ float load_param(const void* p, int dt, int64_t i) {
    if (dt == TE_MX_FP32) return __ldg(static_cast<const float*>(p) + i);
    if (dt == TE_MX_FP16) return to_f32(static_cast<const __half*>(p)[i]);
    return to_f32(static_cast<const __nv_bfloat16*>(p)[i]);
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

// Sum over the block's threads, the same value in each (`red`: one float per
// warp).  Ends with every thread past its reads of `red`.
__device__ __forceinline__ float block_sum(float v, float* red) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    v = warp_sum(v);
    if (lane == 0) red[warp] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < warps; ++w) s += red[w];
    __syncthreads();
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

// One block per row, element by element, the row read three times (the second
// and third time from L1 / L2).
template <typename T>
__global__ void __launch_bounds__(kRowThreads)
ln_forward_kernel(const LnArgs a) {
    __shared__ float red[kRowThreads / 32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
    T* y = static_cast<T*>(a.y) + row * a.ld_y;
    float s = 0.0f;
    for (int64_t i = threadIdx.x; i < a.hidden; i += kRowThreads) s += to_f32(x[i]);
    const float mu = block_sum(s, red) / float(a.hidden);
    s = 0.0f;
    for (int64_t i = threadIdx.x; i < a.hidden; i += kRowThreads) {
        const float d = to_f32(x[i]) - mu;
        s = fmaf(d, d, s);
    }
    const float rs = 1.0f / sqrtf(block_sum(s, red) / float(a.hidden) + a.eps);
    for (int64_t i = threadIdx.x; i < a.hidden; i += kRowThreads) {
        const float xh = (to_f32(x[i]) - mu) * rs;
        const float b = a.beta ? load_param(a.beta, a.param_dtype, i) : 0.0f;
        y[i] = from_f32<T>(fmaf(xh, load_param(a.gamma, a.param_dtype, i), b));
    }
    if (threadIdx.x == 0 && a.mu) {
        a.mu[row] = mu;
        a.rsigma[row] = rs;
    }
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads)
ln_backward_dx_kernel(const LnBackwardArgs a) {
    __shared__ float red[kRowThreads / 32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
    const T* dy = static_cast<const T*>(a.dy) + row * a.ld_dy;
    T* dx = static_cast<T*>(a.dx) + row * a.ld_dx;
    const float mu = a.mu[row], rs = a.rsigma[row];
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t i = threadIdx.x; i < a.hidden; i += kRowThreads) {
        const float g = to_f32(dy[i]) * load_param(a.gamma, a.param_dtype, i);
        s1 += g;
        s2 = fmaf(g, (to_f32(x[i]) - mu) * rs, s2);
    }
    const float c1 = block_sum(s1, red) / float(a.hidden), c2 = block_sum(s2, red) / float(a.hidden);
    for (int64_t i = threadIdx.x; i < a.hidden; i += kRowThreads) {
        const float g = to_f32(dy[i]) * load_param(a.gamma, a.param_dtype, i);
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
    for (int64_t r = blockIdx.y; r < a.rows; r += parts) {
        const float d = to_f32(dy[r * a.ld_dy]);
        sg = fmaf(d, (to_f32(x[r * a.ld_x]) - a.mu[r]) * a.rsigma[r], sg);
        sb += d;
    }
    a.partial[(2 * int64_t(blockIdx.y)) * a.hidden + c] = sg;
    a.partial[(2 * int64_t(blockIdx.y) + 1) * a.hidden + c] = sb;
}

// dgamma / dbeta from `parts` partial sums per column.  A block owns 32
// columns (lane = column); warp w adds parts w, w + 32, ... in order, loading
// four of them at a time (the sums come from L2 and the loads' latency is what
// this costs), then the warps' sums are added in warp order.
constexpr int kReduceWarps = 32;
__global__ void __launch_bounds__(kReduceWarps * 32)
ln_backward_reduce_kernel(const LnBackwardArgs a, int parts) {
    __shared__ float sums[2][kReduceWarps][33];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c = int64_t(blockIdx.x) * 32 + lane;
    float sg = 0.0f, sb = 0.0f;
    if (c < a.hidden)
        for (int p0 = warp; p0 < parts; p0 += 4 * kReduceWarps) {
            float g[4], b[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t p = p0 + k * kReduceWarps;
                g[k] = p < parts ? a.partial[2 * p * a.hidden + c] : 0.0f;
                b[k] = p < parts ? a.partial[(2 * p + 1) * a.hidden + c] : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
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

// Backward, rows on 16-byte boundaries, one pass over dy and x.  Persistent;
// a group of threads owns the same columns (two vectors per thread at most) of
// every row that it takes, so the columns' sums of dy xh and dy stay in its
// registers from row to row.  dy and x come through a ring of rows in shared
// memory, one bulk copy each, several rows ahead (a row's two sums are a
// dependent chain of loads, shuffles and a barrier, which the copies of the
// next rows cover); a row's g and xh stay in registers between its sums and
// dx.  Rows past 16 KB are split over a cluster of blocks: each adds its part
// of the two sums to every other's with one 8-byte remote store per row.
// Short rows: several groups per block, joined at the end, so that every block
// leaves one partial sum per column.
constexpr int kBwdThreads = 512;
constexpr int kBwdMaxStages = 8;
constexpr int kBwdRingBytes = 200 * 1024;
constexpr int kBwdMaxGroups = 16;
constexpr int kBwdMaxCluster = 8;

struct LnBwdShape {
    int nvec;        // vectors of a row
    int cvec;        // vectors of a block's part of it
    int group;       // threads per group
    int groups;      // groups per block
    int stages;
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
__device__ __forceinline__ void lds_pairs(uint32_t addr, uint64_t& a, uint64_t& b) {
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr) : "memory");
}
__device__ __forceinline__ void group_barrier(int id, int threads) {
    asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(threads) : "memory");
}

// The warps' sums of a row group meet in 16 slots (zero past its warps), which
// every thread adds in the same order, four independent chains of packed pairs.
constexpr int kPartWarps = 16, kPartGroups = 8;
__device__ __forceinline__ uint64_t sum_slots2(uint32_t addr) {          // 16 pairs (c1, c2)
    uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < kPartWarps / 2; ++j) {
        uint64_t u, v;
        lds_pairs(addr + 16 * j, u, v);
        acc[j & 1] = f32x2::add(acc[j & 1], u);
        acc[2 + (j & 1)] = f32x2::add(acc[2 + (j & 1)], v);
    }
    return f32x2::add(f32x2::add(acc[0], acc[2]), f32x2::add(acc[1], acc[3]));
}

template <typename T, bool kP32, int kV, bool kCluster>
__global__ void __launch_bounds__(kBwdThreads, 1)
ln_backward_vec_kernel(const LnBackwardArgs a, const LnBwdShape sh, unsigned int* status) {
    using V = Vec<T>;
    extern __shared__ __align__(128) uint8_t ring_raw[];
    __shared__ __align__(8) uint64_t full[kBwdMaxGroups][kBwdMaxStages];
    __shared__ __align__(8) uint64_t part_full[2];
    __shared__ __align__(16) float2 warp_part[2][kPartGroups][kPartWarps];     // by parity of the row count
    __shared__ __align__(16) float2 block_part[2][kBwdMaxCluster];

    const int group = threadIdx.x / sh.group, t = threadIdx.x % sh.group, lane = threadIdx.x & 31;
    const int gwarps = sh.group >> 5;
    const uint32_t rank = kCluster ? block_rank() : 0u;
    const int unit = int(blockIdx.x) / sh.cluster, units = int(gridDim.x) / sh.cluster;
    const int vec0 = int(rank) * sh.cvec, mine = min(sh.cvec, sh.nvec - vec0);      // this block's vectors
    const uint32_t stage_bytes = uint32_t(sh.cvec) * 32;                            // dy, then x
    const uint32_t ring = smem_u32(ring_raw) + uint32_t(group * sh.stages) * stage_bytes;
    const int64_t first = int64_t(unit) * sh.groups + group, step = int64_t(units) * sh.groups;
    const int64_t n_mine = first < a.rows ? (a.rows - first + step - 1) / step : 0;
    if (t == 0)
        for (int i = 0; i < sh.stages; ++i) mbar_init(smem_u32(&full[group][i]), 1);
    if (kCluster && threadIdx.x == 0) {
        mbar_init(smem_u32(&part_full[0]), 1);
        mbar_init(smem_u32(&part_full[1]), 1);
    }
    if (t == 0) fence_mbarrier_init();
    if (threadIdx.x < kPartGroups * kPartWarps) {        // (slots past a group's warps stay 0)
        (&warp_part[0][0][0])[threadIdx.x] = make_float2(0.0f, 0.0f);
        (&warp_part[1][0][0])[threadIdx.x] = make_float2(0.0f, 0.0f);
    }
    grid_dependency_wait();
    grid_launch_dependents();
    if constexpr (kCluster) all_blocks_sync();           // the barriers are ready before any remote store
    else __syncthreads();

    const uint32_t bytes = uint32_t(mine) * 16;
    auto load = [&](int64_t i) {                          // row i of this group, by its thread 0
        const int64_t row = first + i * step;
        const uint32_t bar = smem_u32(&full[group][i % sh.stages]), dst = ring + uint32_t(i % sh.stages) * stage_bytes;
        mbar_arrive_expect_tx(bar, 2 * bytes);
        bulk_load_row(dst, static_cast<const T*>(a.dy) + row * a.ld_dy + int64_t(vec0) * V::kN, bytes, bar);
        bulk_load_row(dst + stage_bytes / 2, static_cast<const T*>(a.x) + row * a.ld_x + int64_t(vec0) * V::kN, bytes, bar);
    };
    if (t == 0)
        for (int64_t i = 0; i < sh.stages && i < n_mine; ++i) load(i);

    uint64_t ga[kV][V::kPairs], dga[kV][V::kPairs], dbe[kV][V::kPairs];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        ParamVec<T, kP32> w;
        const bool live = t + v * sh.group < mine;
        if (live) w.load(a.gamma, vec0 + t + v * sh.group);
#pragma unroll
        for (int k = 0; k < V::kPairs; ++k) {
            ga[v][k] = live ? w.pair(k) : 0;
            dga[v][k] = dbe[v][k] = 0;
        }
    }
    const float inv_h = 1.0f / float(a.hidden);
    float mu = 0.0f, rs = 0.0f;
    if (n_mine > 0) {
        mu = __ldg(a.mu + first);
        rs = __ldg(a.rsigma + first);
    }
    bool ok = true;
    int stage = 0;
    uint32_t phase = 0;
    for (int64_t i = 0; i < n_mine; ++i) {
        const int64_t row = first + i * step;
        const uint64_t mu2 = f32x2::both(mu), rs2 = f32x2::both(rs);
        const float rs_now = rs;
        if (i + 1 < n_mine) {                            // the next row's statistics, a row ahead
            mu = __ldg(a.mu + row + step);
            rs = __ldg(a.rsigma + row + step);
        }
        if (ok && !mbar_wait(smem_u32(&full[group][stage]), phase, status)) {
            ok = false;                                  // gave up: let the copies in flight land
            if (t == 0)
                for (int64_t j = i; j < i + sh.stages && j < n_mine; ++j)
                    mbar_wait(smem_u32(&full[group][j % sh.stages]), uint32_t(j / sh.stages) & 1u, status);
        }
        const uint32_t src = ring + uint32_t(stage) * stage_bytes;
        uint64_t g[kV][V::kPairs], xh[kV][V::kPairs], s1 = 0, s2 = 0;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int j = t + v * sh.group;
            if (j < mine) {
                const uint4 wd = lds128(src + 16 * j), wx = lds128(src + stage_bytes / 2 + 16 * j);
#pragma unroll
                for (int k = 0; k < V::kPairs; ++k) {
                    const uint64_t d = V::pair(wd, k);
                    xh[v][k] = f32x2::mul(f32x2::sub(V::pair(wx, k), mu2), rs2);
                    g[v][k] = f32x2::mul(d, ga[v][k]);
                    s1 = f32x2::add(s1, g[v][k]);
                    s2 = f32x2::fma(g[v][k], xh[v][k], s2);
                    dga[v][k] = f32x2::fma(d, xh[v][k], dga[v][k]);
                    dbe[v][k] = f32x2::add(dbe[v][k], d);
                }
            }
        }
        // lanes 0..15 add up the first sum, lanes 16..31 the second
        float c1 = f32x2::lo(s1) + f32x2::hi(s1), c2 = f32x2::lo(s2) + f32x2::hi(s2);
        float half = (lane < 16 ? c1 : c2) + __shfl_xor_sync(0xFFFFFFFFu, lane < 16 ? c2 : c1, 16);
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) half += __shfl_xor_sync(0xFFFFFFFFu, half, o);
        if (gwarps > 1) {
            // (a parity's slots are read before the next row's barrier, and
            // written again after it)
            float* part = reinterpret_cast<float*>(warp_part[i & 1][group]);
            if ((lane & 15) == 0) part[2 * (t >> 5) + (lane >> 4)] = half;
            group_barrier(1 + group, sh.group);
            const uint64_t c = sum_slots2(smem_u32(part));
            c1 = f32x2::lo(c);
            c2 = f32x2::hi(c);
        } else {
            c1 = __shfl_sync(0xFFFFFFFFu, half, 0);      // (every lane has read the stage)
            c2 = __shfl_sync(0xFFFFFFFFu, half, 16);
        }
        if (t == 0 && ok && i + sh.stages < n_mine) load(i + sh.stages);
        if constexpr (kCluster) {
            // every block's sums to every block; block_part[parity] is written for
            // row i + 2 only by blocks that hold all sums of row i + 1, whose
            // senders had read those of row i
            const uint32_t bar = smem_u32(&part_full[i & 1]);
            if (t == 0) mbar_arrive_expect_tx(bar, 8u * uint32_t(sh.cluster));
            if (t < sh.cluster)
                remote_store(remote_smem(smem_u32(&block_part[i & 1][rank]), uint32_t(t)), f32x2::pack(c1, c2),
                             remote_smem(bar, uint32_t(t)));
            ok = ok && mbar_wait(bar, uint32_t(i >> 1) & 1u, status);
            c1 = c2 = 0.0f;
            for (int r = 0; r < sh.cluster; ++r) {
                const float2 f = block_part[i & 1][r];
                c1 += f.x;
                c2 += f.y;
            }
        }
        if (a.dx) {
            // dx = rs g - rs c2 xh - rs c1
            const uint64_t m2 = f32x2::both(-rs_now * (c2 * inv_h)), m1 = f32x2::both(-rs_now * (c1 * inv_h));
            uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(a.dx) + row * a.ld_dx) + vec0;
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                const int j = t + v * sh.group;
                if (j < mine) {
                    uint64_t o[V::kPairs];
#pragma unroll
                    for (int k = 0; k < V::kPairs; ++k) o[k] = f32x2::fma(g[v][k], rs2, f32x2::fma(xh[v][k], m2, m1));
                    out[j] = V::from_pairs(o);
                }
            }
        }
        if (++stage == sh.stages) {
            stage = 0;
            phase ^= 1u;
        }
    }
    if (a.dgamma) {
        // the groups' column sums meet in the ring (every copy has landed and
        // been read) and are added in group order
        float* sums = reinterpret_cast<float*>(ring_raw);
        const int cols = sh.cvec * V::kN;
        __syncthreads();
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int j = t + v * sh.group;
            if (j < mine) {
#pragma unroll
                for (int k = 0; k < V::kPairs; ++k) {
                    const int c = j * V::kN + 2 * k;
                    *reinterpret_cast<uint64_t*>(sums + (2 * group) * cols + c) = dga[v][k];
                    *reinterpret_cast<uint64_t*>(sums + (2 * group + 1) * cols + c) = dbe[v][k];
                }
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < mine * V::kN; c += blockDim.x) {
            float sg = 0.0f, sb = 0.0f;
            for (int q = 0; q < sh.groups; ++q) {
                sg += sums[(2 * q) * cols + c];
                sb += sums[(2 * q + 1) * cols + c];
            }
            a.partial[(2 * int64_t(unit)) * a.hidden + vec0 * V::kN + c] = sg;
            a.partial[(2 * int64_t(unit) + 1) * a.hidden + vec0 * V::kN + c] = sb;
        }
    }
    if constexpr (kCluster) all_blocks_sync();            // no block leaves while another may still store to it
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

bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
// Rows of a matrix of elements of `size` bytes start on 16-byte boundaries.
bool rows_on16(const void* p, int64_t ld, int64_t rows, size_t size) {
    return on16(p) && (rows == 1 || ld * int64_t(size) % 16 == 0);
}

template <typename T, bool kP32>
cudaError_t forward_vec(const LnArgs& a, cudaStream_t stream) {
    const int nvec = int(a.hidden / Vec<T>::kN);
    // Threads per row: one vector per thread while there are too few rows to
    // fill the GPU with smaller blocks, else up to four (eight for rows past
    // 4096 vectors).
    int v = a.rows <= 304 && nvec <= 1024 ? 1 : nvec <= 64 ? 2 : nvec <= 4096 ? 4 : 8;
    const int tx = ((nvec + v - 1) / v + 31) / 32 * 32, ty = tx == 32 ? 4 : 1;
    const dim3 grid(unsigned((a.rows + ty - 1) / ty)), block{unsigned(tx), unsigned(ty)};
    if (v == 1) return launch_dependent(ln_forward_vec_kernel<T, kP32, 1>, grid, block, stream, a, nvec);
    if (v == 2) return launch_dependent(ln_forward_vec_kernel<T, kP32, 2>, grid, block, stream, a, nvec);
    if (v == 4) return launch_dependent(ln_forward_vec_kernel<T, kP32, 4>, grid, block, stream, a, nvec);
    return launch_dependent(ln_forward_vec_kernel<T, kP32, 8>, grid, block, stream, a, nvec);
}

template <typename T>
cudaError_t forward(const LnArgs& a, cudaStream_t stream) {
    const int64_t nvec = a.hidden / Vec<T>::kN;
    if (a.hidden % Vec<T>::kN == 0 && nvec <= 8192 && rows_on16(a.x, a.ld_x, a.rows, sizeof(T)) &&
        rows_on16(a.y, a.ld_y, a.rows, sizeof(T)) && on16(a.gamma) && on16(a.beta)) {
        if constexpr (sizeof(T) == 2)
            if (a.param_dtype != TE_MX_FP32) return forward_vec<T, false>(a, stream);
        return forward_vec<T, true>(a, stream);
    }
    return launch_dependent(ln_forward_kernel<T>, dim3(unsigned(a.rows)), dim3(kRowThreads), stream, a);
}

template <typename T, bool kP32, int kV, bool kCluster>
cudaError_t backward_vec_launch(const LnBackwardArgs& a, const LnBwdShape& sh, int sms, unsigned int* status, int* parts,
                                cudaStream_t stream) {
    auto kern = ln_backward_vec_kernel<T, kP32, kV, kCluster>;
    const int ring = sh.groups * sh.stages * sh.cvec * 32, sums = sh.groups * sh.cvec * Vec<T>::kN * 8;
    const int smem = ring > sums ? ring : sums;
    cudaError_t e = set_smem_attribute_once(reinterpret_cast<const void*>(kern), kBwdRingBytes);
    if (e != cudaSuccess) return e;
    const int64_t want = (a.rows + sh.groups - 1) / sh.groups, most = sms / sh.cluster;
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
    LnBwdShape sh{};
    sh.nvec = int(a.hidden / Vec<T>::kN);
    sh.cluster = 1;
    while (sh.nvec > 1024 * sh.cluster) sh.cluster *= 2;                   // at most 16 KB of a row per block
    sh.cvec = (sh.nvec + sh.cluster - 1) / sh.cluster;
    const int v = sh.cvec > 32 ? 2 : 1;
    sh.group = ((sh.cvec + v - 1) / v + 31) / 32 * 32;
    // as many groups as the block's threads (and named barriers) allow
    sh.groups = sh.cluster > 1 ? 1 : kBwdThreads / sh.group;
    if (sh.groups > kBwdMaxGroups - 1 && sh.group > 32) sh.groups = kBwdMaxGroups - 1;
    if (sh.groups > a.rows) sh.groups = int(a.rows);
    sh.stages = kBwdRingBytes / (sh.groups * sh.cvec * 32);
    if (sh.stages > kBwdMaxStages) sh.stages = kBwdMaxStages;
    if (v == 1) return backward_vec_launch<T, kP32, 1, false>(a, sh, sms, status, parts, stream);
    if (sh.cluster == 1) return backward_vec_launch<T, kP32, 2, false>(a, sh, sms, status, parts, stream);
    return backward_vec_launch<T, kP32, 2, true>(a, sh, sms, status, parts, stream);
}

template <typename T>
cudaError_t backward(const LnBackwardArgs& a, int sms, unsigned int* status, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    const dim3 reduce_grid(unsigned((a.hidden + 31) / 32));
    if (a.rows > 0 && a.hidden % Vec<T>::kN == 0 && a.hidden / Vec<T>::kN <= 1024 * kBwdMaxCluster &&
        rows_on16(a.x, a.ld_x, a.rows, sizeof(T)) && rows_on16(a.dy, a.ld_dy, a.rows, sizeof(T)) &&
        rows_on16(a.dx, a.ld_dx, a.rows, sizeof(T)) && on16(a.gamma)) {
        int n = 0;
        if constexpr (sizeof(T) == 2)
            e = a.param_dtype != TE_MX_FP32 ? backward_vec<T, false>(a, sms, status, &n, stream)
                                            : backward_vec<T, true>(a, sms, status, &n, stream);
        else e = backward_vec<T, true>(a, sms, status, &n, stream);
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
        e = launch_dependent(ln_backward_dx_kernel<T>, dim3(unsigned(a.rows)), dim3(kRowThreads), stream, a);
        if (e != cudaSuccess) return e;
    }
    if (!a.dgamma) return e;
    return launch_dependent(ln_backward_reduce_kernel, reduce_grid, dim3(kReduceWarps * 32), stream, a, parts);
}

}  // namespace

// Rows of partial sums in the workspace.
int ln_backward_parts(int64_t rows) { return int(rows < kLnMaxParts ? rows : kLnMaxParts); }

te_mx_status ln_forward_launch(const LnArgs& a, cudaStream_t stream) {
    cudaError_t e = a.dtype == TE_MX_FP32   ? forward<float>(a, stream)
                    : a.dtype == TE_MX_FP16 ? forward<__half>(a, stream)
                                            : forward<__nv_bfloat16>(a, stream);
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
