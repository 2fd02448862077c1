// Activations of the gated feed-forward (te_mx_activation) and their
// derivatives, on packed fp32 pairs.
//
// With s the logistic function of x (SiLU) or of z = 2 sqrt(2/pi) (x +
// 0.044715 x^3) (the tanh form of GELU, 0.5 (1 + tanh(z / 2)) = s):
//   act(x) = x s,   act'(x) = s (1 + x (1 - s) dz/dx),
// s evaluated as 1 / (1 + 2^t), t = -log2(e) z, with the two MUFU operations
// per value (ex2, reciprocal) and the rest packed.  ReLU keeps NaN.  Where s is
// below the smallest normal number (x < -87.3 for SiLU) it is taken as 0, an
// error of act(x) of less than 1.1e-36.
#pragma once
#include <cstdint>

#include "../../include/temx.h"
#include "f32x2.cuh"

namespace temx {
namespace gated {

constexpr float kNegLog2e = -1.4426950408889634f;
constexpr float kZ1 = 2.0f * 0.7978845608028654f;        // z = kZ1 x + kZ3 x^3
constexpr float kZ3 = kZ1 * 0.044715f;

__device__ __forceinline__ uint64_t relu2(uint64_t x) {
    float a0, a1;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(a0) : "f"(f32x2::lo(x)));
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(a1) : "f"(f32x2::hi(x)));
    return f32x2::pack(a0, a1);
}

// 1 / (1 + 2^t)
__device__ __forceinline__ uint64_t logistic2(uint64_t t) {
    float e0, e1, s0, s1;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(f32x2::lo(t)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(f32x2::hi(t)));
    const uint64_t q = f32x2::add(f32x2::pack(e0, e1), f32x2::both(1.0f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s0) : "f"(f32x2::lo(q)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s1) : "f"(f32x2::hi(q)));
    return f32x2::pack(s0, s1);
}

// t of GELU; t -> -+inf where x^2 overflows, which gives x or -0 as it should.
__device__ __forceinline__ uint64_t gelu_t2(uint64_t x) {
    return f32x2::mul(x, f32x2::fma(f32x2::mul(x, x), f32x2::both(kNegLog2e * kZ3), f32x2::both(kNegLog2e * kZ1)));
}

// (The activation is a template argument: a branch between the pairs of an
// unrolled loop would leave each to the latency of its own MUFU chain.  `with`
// picks it once, outside the loop.)
template <int kAct>
__device__ __forceinline__ uint64_t act2(uint64_t x) {
    if constexpr (kAct == TE_MX_ACT_RELU) return relu2(x);
    else return f32x2::mul(x, logistic2(kAct == TE_MX_ACT_GELU ? gelu_t2(x) : f32x2::mul(x, f32x2::both(kNegLog2e))));
}

template <int kAct> struct Act { static constexpr int value = kAct; };
template <typename F>
__device__ __forceinline__ void with(int act, F&& f) {
    if (act == TE_MX_ACT_SILU) f(Act<TE_MX_ACT_SILU>{});
    else if (act == TE_MX_ACT_GELU) f(Act<TE_MX_ACT_GELU>{});
    else f(Act<TE_MX_ACT_RELU>{});
}

// a = act(x), d = act'(x).  (1 - s cancels where s is near 1; there act' is
// near 1 and the term's error is a few units of its last place.)
template <int kAct>
__device__ __forceinline__ void act_and_grad2(uint64_t x, uint64_t& a, uint64_t& d) {
    float x0 = f32x2::lo(x), x1 = f32x2::hi(x);
    if constexpr (kAct == TE_MX_ACT_RELU) {
        a = relu2(x);
        d = f32x2::pack(x0 > 0.0f ? 1.0f : 0.0f, x1 > 0.0f ? 1.0f : 0.0f);
        return;
    }
    uint64_t y = x, slope_y = x;                           // slope_y = y dz/dx
    if constexpr (kAct == TE_MX_ACT_GELU) {
        // (beyond +-30 act' is 0 or 1 to fp32; the clamp keeps x^2 finite and NaN a NaN)
        asm("max.NaN.f32 %0, %0, 0fC1F00000;" : "+f"(x0));
        asm("max.NaN.f32 %0, %0, 0fC1F00000;" : "+f"(x1));
        asm("min.NaN.f32 %0, %0, 0f41F00000;" : "+f"(x0));
        asm("min.NaN.f32 %0, %0, 0f41F00000;" : "+f"(x1));
        y = f32x2::pack(x0, x1);
        slope_y = f32x2::mul(y, f32x2::fma(f32x2::mul(y, y), f32x2::both(3.0f * kZ3), f32x2::both(kZ1)));
    }
    const uint64_t s = logistic2(kAct == TE_MX_ACT_GELU ? gelu_t2(y) : f32x2::mul(x, f32x2::both(kNegLog2e)));
    const uint64_t one = f32x2::both(1.0f);
    a = f32x2::mul(x, s);
    d = f32x2::mul(s, f32x2::fma(slope_y, f32x2::sub(one, s), one));
}

}  // namespace gated
}  // namespace temx
