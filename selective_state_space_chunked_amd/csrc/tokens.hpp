// Shared by the packed-row kernels: the rows and slots of a call's sequences,
// row accesses, activations.
#pragma once
#include "common.hpp"
#include "kernels.hpp"

namespace ssm {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float sigmoid_f(float v) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * kLog2e));
}
// log(1 + e^v) from the hardware exp2 and log2 (accurate to an ulp or two where
// the library function takes several times the instructions; it runs once a
// channel and row).  With e = e^v and w = 1 + e rounded, log(1 + e) is log(w) plus
// (e - (w - 1)) / w, which the rounding of the sum lost: below w = 2, where it
// matters against the result, 1 / w may be left out (at most u / 2 of an error
// of u), above it is below an ulp of log(w).  From 20 on the result is v (e^-20 is
// below half an ulp).
__device__ __forceinline__ float softplus_t(float v) {
    const float e = __builtin_amdgcn_exp2f(v * kLog2e);
    const float w = 1.0f + e;
    const float r = fmaf(__builtin_amdgcn_logf(w), kLn2, w < 2.0f ? e - (w - 1.0f) : 0.0f);
    return v > 20.0f ? v : r;
}
// float to the stream's type, to nearest even, by the conversion instruction
template <typename T> __device__ __forceinline__ T to_stream(float f);
template <> __device__ __forceinline__ float to_stream<float>(float f) { return f; }
template <> __device__ __forceinline__ bf16_t to_stream<bf16_t>(float f) {
    return __builtin_bit_cast(bf16_t, (__bf16)f);
}

// a value that is the same in all lanes of the wave, as a scalar
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The last sequence whose first row is at or before row t: -1 before the first
// one, S from the end of the last one on.  Called by whole waves with one t;
// each round the 64 lanes probe 64 entries of the ascending list.
__device__ __forceinline__ int find_seq(const int32_t* start, int S, int t) {
    int lo = 0, hi = S + 1;   // entries before lo are <= t, from hi on > t
    const int lane = lane_id();
    while (hi - lo > 64) {
        const int step = (hi - lo + 63) / 64;
        const int i = lo + lane * step;
        const int c = __popcll(__ballot(i < hi && start[i < hi ? i : lo] <= t));
        if (c == 0) return lo - 1;
        const int top = lo + c * step;
        lo += (c - 1) * step;
        hi = min(hi, top);
    }
    const int i = lo + lane;
    return lo + __popcll(__ballot(i < hi && start[i < hi ? i : lo] <= t)) - 1;
}

// The slot of sequence s, or -1 for an empty place: a slot outside the pool, or
// one that an earlier sequence of the call has.  Called by whole waves with one s.
__device__ __forceinline__ int slot_of(const Sequences& q, int s) {
    if (!q.slot) return s < q.slots ? s : -1;
    const int v = q.slot[s];
    if (v < 0 || v >= q.slots) return -1;
    bool taken = false;
    for (int i = lane_id(); i < s; i += 64) taken |= q.slot[i] == v;
    return __ballot(taken) ? -1 : v;
}

// V consecutive elements: one 16-byte access (V elements of T are 16 bytes), or one element
template <typename T, int V>
__device__ __forceinline__ void load_v(const T* p, float (&v)[V]) {
    if (V == 1) {
        v[0] = to_f32(p[0]);
    } else if (sizeof(T) == 4) {
        const float4 w = *reinterpret_cast<const float4*>(p);
        v[0] = w.x; v[1 % V] = w.y; v[2 % V] = w.z; v[3 % V] = w.w;
    } else {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[(2 * e) % V] = __uint_as_float(ws[e] << 16);
            v[(2 * e + 1) % V] = __uint_as_float(ws[e] & 0xffff0000u);
        }
    }
}
template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, const float (&v)[V]) {
    if (V == 1) {
        p[0] = from_f32<T>(v[0]);
    } else if (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1 % V], v[2 % V], v[3 % V]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = (uint32_t)from_f32<bf16_t>(v[(2 * e) % V]) | ((uint32_t)from_f32<bf16_t>(v[(2 * e + 1) % V]) << 16);
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

}  // namespace ssm
