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
// columns (lane = column); warp w adds parts w, w + 8, ... in order, then the
// warps' sums are added in warp order.
constexpr int kReduceWarps = 8;
__global__ void __launch_bounds__(kReduceWarps * 32)
ln_backward_reduce_kernel(const LnBackwardArgs a, int parts) {
    __shared__ float sums[2][kReduceWarps][32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c = int64_t(blockIdx.x) * 32 + lane;
    float sg = 0.0f, sb = 0.0f;
    if (c < a.hidden)
        for (int p = warp; p < parts; p += kReduceWarps) {
            sg += a.partial[2 * int64_t(p) * a.hidden + c];
            sb += a.partial[(2 * int64_t(p) + 1) * a.hidden + c];
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

// Launch with programmatic stream serialisation: the blocks may start while
// the previous kernel in the stream finishes (every kernel here waits for it
// before its first access to global memory).
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kern)(P...), dim3 grid, int threads, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads));
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename T>
cudaError_t forward(const LnArgs& a, cudaStream_t stream) {
    return launch_dependent(ln_forward_kernel<T>, dim3(unsigned(a.rows)), kRowThreads, stream, a);
}

template <typename T>
cudaError_t backward(const LnBackwardArgs& a, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    const int parts = ln_backward_parts(a.rows);
    // (the parameters' sums first: dx may overwrite dy)
    if (a.dgamma && parts > 0) {
        const unsigned cols = unsigned((a.hidden + kRowThreads - 1) / kRowThreads);
        e = launch_dependent(ln_backward_params_kernel<T>, dim3(cols, unsigned(parts)), kRowThreads, stream, a, parts);
        if (e != cudaSuccess) return e;
    }
    if (a.dx && a.rows > 0) {
        e = launch_dependent(ln_backward_dx_kernel<T>, dim3(unsigned(a.rows)), kRowThreads, stream, a);
        if (e != cudaSuccess) return e;
    }
    if (!a.dgamma) return e;
    return launch_dependent(ln_backward_reduce_kernel, dim3(unsigned((a.hidden + 31) / 32)), kReduceWarps * 32, stream, a,
                            parts);
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
    cudaError_t e = a.dtype == TE_MX_FP32   ? backward<float>(a, stream)
                    : a.dtype == TE_MX_FP16 ? backward<__half>(a, stream)
                                            : backward<__nv_bfloat16>(a, stream);
    return cuda_status(e, "layernorm backward kernel launch");
}

}  // namespace temx
