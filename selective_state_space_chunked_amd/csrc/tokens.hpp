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

// The slot that sequence s names, or -1 where it is outside the pool.
__device__ __forceinline__ int slot_named(const Sequences& q, int s) {
    const int v = q.slot ? q.slot[s] : s;
    return v >= 0 && v < q.slots ? v : -1;
}
// Whether an earlier sequence of the call has the same slot.  Called by whole waves with one s.
__device__ __forceinline__ bool slot_taken(const Sequences& q, int s, int v) {
    if (!q.slot) return false;
    bool taken = false;
    for (int i = lane_id(); i < s; i += 256) {   // four probes under way
        int u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) u[k] = i + 64 * k < s ? q.slot[i + 64 * k] : -1;
#pragma unroll
        for (int k = 0; k < 4; ++k) taken |= u[k] == v;
    }
    return __ballot(taken) != 0;
}
// The slot of sequence s, or -1 for an empty place: a slot outside the pool, or
// one that an earlier sequence of the call has.  Called by whole waves with one s.
__device__ __forceinline__ int slot_of(const Sequences& q, int s) {
    const int v = uniform(slot_named(q, s));
    return v < 0 || slot_taken(q, s, v) ? -1 : v;
}

// A wave's view of the call's sequences.  Fewer than 64 of them (as a rule) lie in
// one register a list, so what a wave asks about them costs one trip to memory,
// under way while its first rows are loaded; otherwise each question reads the
// lists.  Every member is called by whole waves with scalar arguments.
struct SeqTable {
    const Sequences& q;
    const bool small;
    int start_, slot_, fresh_;
    __device__ __forceinline__ explicit SeqTable(const Sequences& q_) : q(q_), small(q_.S < 64) {
        start_ = slot_ = fresh_ = 0;
        if (small) {
            const int l = lane_id();
            start_ = q.start[min(l, q.S)];
            slot_ = q.slot ? q.slot[min(l, q.S - 1)] : l;
            fresh_ = q.fresh ? q.fresh[min(l, q.S - 1)] : 0;
        }
    }
    // the last sequence whose first row is at or before row t, as find_seq
    __device__ __forceinline__ int find(int t) const {
        if (!small) return uniform(find_seq(q.start, q.S, t));
        return __popcll(__ballot(lane_id() <= q.S && start_ <= t)) - 1;
    }
    __device__ __forceinline__ int first(int s) const {   // s <= S
        return small ? __builtin_amdgcn_readlane(start_, s) : uniform(q.start[s]);
    }
    __device__ __forceinline__ int end(int s) const { return min(first(s + 1), q.T); }
    __device__ __forceinline__ int slot(int s) const {   // as slot_of
        if (!small) return uniform(slot_of(q, s));
        const int v = __builtin_amdgcn_readlane(slot_, s);
        if (v < 0 || v >= q.slots) return -1;
        return __ballot(lane_id() < s && slot_ == v) ? -1 : v;
    }
    __device__ __forceinline__ bool fresh(int s) const {
        return small ? __builtin_amdgcn_readlane(fresh_, s) != 0 : q.fresh && q.fresh[s];
    }
};

// Four consecutive elements at any element's address (global memory takes
// unaligned accesses), as floats and back.  Eight bf16 elements a lane would be
// whole 16-byte accesses, but twice the registers: the packed convolution of 8192
// rows x 4096 channels took 33.6 us with four and 37.6 us with eight.
typedef uint32_t u32x2 __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4 __attribute__((ext_vector_type(4), aligned(4)));
template <typename T> struct Vec;
template <> struct Vec<float> {
    static constexpr int V = 4;
    f32x4 r;
    __device__ __forceinline__ void arrived() { __asm__ volatile("" : "+v"(r)); }   // its load is waited for here
    __device__ __forceinline__ void load(const float* p) { r = *reinterpret_cast<const f32x4*>(p); }
    __device__ __forceinline__ void load(const float* p, int n) {   // the first n, the others 0
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = e < n ? p[e] : 0.0f;
    }
    __device__ __forceinline__ void get(float (&v)[4]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = r[e];
    }
    __device__ __forceinline__ void set(const float (&v)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = v[e];
    }
    __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<f32x4*>(p) = r; }
    __device__ __forceinline__ void store(float* p, int n) const {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < n) p[e] = r[e];
    }
};
template <> struct Vec<bf16_t> {
    static constexpr int V = 4;
    u32x2 r;
    __device__ __forceinline__ void arrived() { __asm__ volatile("" : "+v"(r)); }
    __device__ __forceinline__ void load(const bf16_t* p) { r = *reinterpret_cast<const u32x2*>(p); }
    __device__ __forceinline__ void load(const bf16_t* p, int n) {
        r = u32x2(0);
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < n) r[e / 2] |= (uint32_t)p[e] << (16 * (e & 1));
    }
    __device__ __forceinline__ void get(float (&v)[V]) const {
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
            v[2 * e] = __uint_as_float(r[e] << 16);
            v[2 * e + 1] = __uint_as_float(r[e] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&v)[V]) {
#pragma unroll
        for (int e = 0; e < V / 2; ++e)
            r[e] = (uint32_t)to_stream<bf16_t>(v[2 * e]) | ((uint32_t)to_stream<bf16_t>(v[2 * e + 1]) << 16);
    }
    __device__ __forceinline__ void store(bf16_t* p) const { *reinterpret_cast<u32x2*>(p) = r; }
    __device__ __forceinline__ void store(bf16_t* p, int n) const {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < n) p[e] = (bf16_t)(r[e / 2] >> (16 * (e & 1)));
    }
};

}  // namespace ssm
