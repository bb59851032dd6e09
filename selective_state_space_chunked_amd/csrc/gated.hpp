// The gated linear recurrence, shared by its training and serving kernels:
//
//   rho = sigmoid(r + r_bias),  iota = sigmoid(i + i_bias),
//   q = power softplus(lam) rho,  a = e^-q,  beta = sqrt(1 - a^2),
//   h_t = a_t h_{t-1} + beta_t iota_t x_t.
#pragma once
#include "tokens.hpp"

namespace ssm {

// What a channel has once, the biases times -log2(e) as exp2 takes them.
struct GateChannel {
    float rate, rb, ib;
};
__device__ __forceinline__ GateChannel gate_channel(const float* lam, const float* rb, const float* ib, float power, int d) {
    return {power * softplus_t(lam[d]), rb ? -kLog2e * rb[d] : 0.0f, ib ? -kLog2e * ib[d] : 0.0f};
}
// sigmoid(v + bias): below about v = -87 the exponential is infinite and the gate 0
__device__ __forceinline__ float gate_open(float v, float nb) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(fmaf(v, -kLog2e, nb)));
}
__device__ __forceinline__ float gate_decay(float q) { return __builtin_amdgcn_exp2f(-kLog2e * q); }
// 1 - a^2 = 1 - e^-2q.  From q = 1/2 on the difference loses nothing (a^2 <= 0.37); below, where a slow channel's
// a is near 1 and the difference would keep few bits, 1 - e^-2q = 2 a sinh(q) by its series, whose first term left
// out is q^8 / 9! < 2^-26 of it.
__device__ __forceinline__ float gate_rest(float q, float a) {
    const float s = q * q;
    const float p = fmaf(s, fmaf(s, fmaf(s, 1.0f / 5040, 1.0f / 120), 1.0f / 6), 1.0f);
    return q < 0.5f ? 2.0f * q * a * p : fmaf(-a, a, 1.0f);
}

}  // namespace ssm
