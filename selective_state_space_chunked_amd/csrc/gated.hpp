// The gated linear recurrence, shared by its training and serving kernels:
//
//   rho = sigmoid(r + r_bias),  iota = sigmoid(i + i_bias),
//   q = power softplus(lam) rho,  a = e^-q = 2^-t,  beta = sqrt(1 - a^2),
//   h_t = a_t h_{t-1} + beta_t iota_t x_t.
#pragma once
#include "tokens.hpp"

namespace ssm {

// What a channel has once: what multiplies rho in the exponent of a = 2^-t, and the biases, times -log2(e) as exp2
// takes them.
struct GateChannel {
    float rate, rb, ib;
};
__device__ __forceinline__ GateChannel gate_channel(const float* lam, const float* rb, const float* ib, float power, int d) {
    return {power * softplus_t(lam[d]) * kLog2e, rb ? -kLog2e * rb[d] : 0.0f, ib ? -kLog2e * ib[d] : 0.0f};
}
// sigmoid(v + bias): below about v = -87 the exponential is infinite and the gate 0
__device__ __forceinline__ float gate_open(float v, float nb) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(fmaf(v, -kLog2e, nb)));
}
// Of an opened decay gate, t = q log2(e): a = 2^-t and 1 - a^2.  From q = 1 on the difference loses nothing (a^2 <=
// 0.14); below, where a slow channel's a is near 1 and the difference would keep few bits, 1 - e^-2q = 2 a sinh(q) by
// its series in t, whose first term left out is q^10 / 11! < 2^-25 of it.  rho is at most 1, so where a wave's channels
// all have rates below that point (SLOW) there is nothing to choose.
constexpr float kGateSlow = kLog2e;
template <bool SLOW>
__device__ __forceinline__ float gate_rest(float t, float& a) {
    constexpr float c = kLn2 * kLn2;
    a = __builtin_amdgcn_exp2f(-t);
    const float s = t * t;
    const float p = fmaf(s, fmaf(s, fmaf(s, fmaf(s, 2 * kLn2 * c * c * c * c / 362880, 2 * kLn2 * c * c * c / 5040),
                                         2 * kLn2 * c * c / 120), 2 * kLn2 * c / 6), 2 * kLn2);
    const float v = t * a * p;
    return SLOW || t < kGateSlow ? v : fmaf(-a, a, 1.0f);
}

}  // namespace ssm
