// What the row-wise kernels share: elements of bf16, fp16 and fp32 as fp32,
// 16-byte vectors of them as packed fp32 pairs, parameters, warp sums, and
// launches that overlap the end of the kernel before.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "f32x2.cuh"
#include "temx_internal.h"

namespace temx {

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

// ---------------------------------------------------------------- rows off 16-byte boundaries

// Rows of 16-bit elements whose pitch is no multiple of 8: the rows of a block that are
// multiples of 8 apart start equally far behind a 16-byte boundary (the base lies on
// one), so they are read and written in whole vectors all the same.  Vector i of a row
// that starts `shift` elements behind a boundary holds its elements 8 i - shift ..
// 8 i - shift + 7; of the first and the last vector, which reach into the neighbouring
// rows, only the row's own elements are touched, one by one.
template <typename T> struct ShiftedRow {
    static constexpr int kN = Vec<T>::kN;
    int hidden, shift;
    __device__ __forceinline__ int vectors() const { return (hidden + shift + kN - 1) / kN; }
    __device__ __forceinline__ bool whole(int i) const { return i * kN >= shift && i * kN - shift + kN <= hidden; }
    __device__ __forceinline__ bool has(int i, int k) const { return unsigned(i * kN - shift + k) < unsigned(hidden); }
    // The vector's elements, 0 outside the row.  `row`: its first element; read once.
    __device__ __forceinline__ uint4 load(const T* row, int i) const {
        if (whole(i)) return __ldcs(reinterpret_cast<const uint4*>(row - shift) + i);
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < kN; ++k)
            if (has(i, k)) w[k / 2] |= uint32_t(reinterpret_cast<const uint16_t*>(row)[i * kN - shift + k]) << (k % 2 * 16);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void store(T* row, int i, const uint4& v) const {
        if (whole(i)) {
            reinterpret_cast<uint4*>(row - shift)[i] = v;
            return;
        }
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < kN; ++k)
            if (has(i, k)) reinterpret_cast<uint16_t*>(row)[i * kN - shift + k] = uint16_t(w[k / 2] >> (k % 2 * 16));
    }
    // parameters of the vector's elements (0 outside the row)
    template <bool kP32> __device__ __forceinline__ void load_params(ParamVec<T, kP32>& p, const void* from, int i) const {
        float f[kN];
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            f[k] = 0.0f;
            if (has(i, k)) {
                if constexpr (kP32) f[k] = load_param<float>(from, i * kN - shift + k);
                else f[k] = load_param<T>(from, i * kN - shift + k);
            }
        }
        if constexpr (ParamVec<T, kP32>::kWords == 2) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
                p.w[q] = make_uint4(__float_as_uint(f[4 * q]), __float_as_uint(f[4 * q + 1]), __float_as_uint(f[4 * q + 2]),
                                    __float_as_uint(f[4 * q + 3]));
        } else {
            uint64_t o[kN / 2];
#pragma unroll
            for (int k = 0; k < kN / 2; ++k) o[k] = f32x2::pack(f[2 * k], f[2 * k + 1]);
            p.w[0] = Vec<T>::from_pairs(o);                // (exact)
        }
    }
};

// ---------------------------------------------------------------- blocks

// Sizes and both addresses are multiples of 16 bytes; counted on the mbarrier `bar`.
__device__ __forceinline__ void bulk_load_row(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}
// Barrier `id` over `threads` threads (whole warps) of the block.
__device__ __forceinline__ void group_barrier(int id, int threads) {
    asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(threads) : "memory");
}

// Sum over the block's warps of a value that each warp has summed (the same value
// in each thread, in warp order).  `part`: a slot for each warp; one call between
// two barriers of the block.
__device__ __forceinline__ float across_warps(float v, float* part, int warps, int warp, int lane) {
    if (warps == 1) return v;
    if (lane == 0) part[warp] = v;
    __syncthreads();
    return warp_sum(lane < warps ? part[lane] : 0.0f);
}

// The compiler takes the words for new ones from here on: what it unpacked of them
// before is unpacked again rather than kept in registers.
__device__ __forceinline__ void unpack_again(uint4& w) { asm volatile("" : "+r"(w.x), "+r"(w.y), "+r"(w.z), "+r"(w.w)); }

// What a thread takes of a long row, i = t, t + kAnyThreads, ... in a block of
// kAnyThreads, kLongAhead elements at a time: all loaded, load(q, i), before the first is
// used, use(q, i), which may write (the compiler moves no load past such a write).
constexpr int kAnyThreads = 512;                 // of the kernels for rows in any layout
constexpr int kLongAhead = 8;
template <typename L, typename U>
__device__ __forceinline__ void long_batch(int64_t i, int64_t hidden, L&& load, U&& use) {
#pragma unroll
    for (int q = 0; q < kLongAhead; ++q)
        if (i + q * kAnyThreads < hidden) load(q, i + q * kAnyThreads);
#pragma unroll
    for (int q = 0; q < kLongAhead; ++q)
        if (i + q * kAnyThreads < hidden) use(q, i + q * kAnyThreads);
}
// A thread's sum of the terms that use() returns: up to 32768 of them (rows of 2^24
// elements), 64 to a batch, the batches added 64 to a batch of batches, so that a chain has
// at most 64 + 64 + 8 additions.
template <typename L, typename U> __device__ __forceinline__ float long_sum(int64_t hidden, L&& load, U&& use) {
    float total = 0.0f, outer = 0.0f;
    int batches = 0;
    for (int64_t i = threadIdx.x; i < hidden;) {
        float batch = 0.0f;
        for (int k = 0; k < 64 && i < hidden; k += kLongAhead, i += kLongAhead * kAnyThreads)
            long_batch(i, hidden, load, [&](int q, int64_t at) { batch += use(q, at); });
        outer += batch;
        if (++batches == 64) {
            total += outer;
            outer = 0.0f;
            batches = 0;
        }
    }
    return total + outer;
}

// ---------------------------------------------------------------- launches

// Threads that hold a row of `n` pieces, `per` each.
inline int row_threads(int64_t n, int64_t per) { return int((n + 32 * per - 1) / (32 * per) * 32); }


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

// Whether a matrix's rows can be taken as ShiftedRows beside those of pitch `ld`.
template <typename T> inline bool shifts_alike(const void* p, int64_t ld_p, int64_t ld) {
    return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld_p - ld) % Vec<T>::kN == 0);
}
// Blocks, so that the rows of a block (rows_per_block at a time) are multiples of 8 apart.
inline int64_t blocks_for_shifts(int64_t blocks, int rows_per_block, int64_t rows) {
    if (blocks * rows_per_block >= rows) return blocks;    // (one row each)
    const int64_t unit = rows_per_block >= 8 ? 1 : 8 / rows_per_block;
    return blocks < unit ? unit : blocks / unit * unit;
}

inline bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
// Rows of a matrix of elements of `size` bytes start on 16-byte boundaries.
inline bool rows_on16(const void* p, int64_t ld, int64_t rows, size_t size) {
    return on16(p) && (rows == 1 || ld * int64_t(size) % 16 == 0);
}

}  // namespace temx
