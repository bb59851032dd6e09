// The selective scan over packed rows, with its layer's skip and gate:
//
//   h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t,  y_t = (C_t . h_t + skip x_t) z_t sigmoid(z_t)
//
// Prompts.  A lane holds one channel with its N states; a wave walks 64
// channels down a range of rows, so the streams are read along the channels as
// the projections write them, and B_t, C_t are the same for the whole wave: they
// come as fp32 through the scalar cache and enter the products as scalar
// operands (one pass turns them into fp32 first).  Per state and row that leaves
// a multiply and an exp2 for the transition, a multiply and a multiply-add for
// the state and one multiply-add for y.  Few long sequences do not fill the GPU,
// so the rows are cut into ranges whatever the sequences' lengths: a first pass
// leaves, for the sequence that crosses the end of each range, its state there
// (from zero where it crosses the whole range) and the sum of its step sizes;
// the second pass composes those of the ranges before it,
//   h <- exp(A sum delta) h + S,
// and walks its rows.
//
// Single tokens.  Bound by the states' traffic: four states a lane, so a wave
// reads and writes the pool in whole lines.
#include <algorithm>

#include "tokens.hpp"

namespace ssm {
namespace {

typedef __attribute__((address_space(4))) const float sfloat;   // read through the scalar cache

// B_t, C_t of every row in fp32, row t at bc[t * 2N]: B then C
template <typename T>
__global__ __launch_bounds__(256) void tok_bc_kernel(TokScanParams p) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int N = p.N;
    if (i >= (int64_t)p.q.T * 2 * N) return;
    const int64_t t = i / (2 * N);
    const int n = (int)(i - t * 2 * N);
    p.bc[i] = n < N ? to_f32(((const T*)p.Bm)[t * p.sB + n]) : to_f32(((const T*)p.C)[t * p.sC + n - N]);
}

constexpr int kGrp = 4;   // rows loaded together

template <typename T, int N>
struct ScanLane {
    const T *delta, *x, *z;
    T* y;
    sfloat* bc;
    int64_t sdelta, sx, sz, sy;
    float a[N], h[N], bias, skip, dsum;
    int softplus;
    bool skips, gates;

    __device__ __forceinline__ ScanLane(const TokScanParams& p, int d) {
        delta = (const T*)p.delta + d;
        x = (const T*)p.x + d;
        gates = p.z != nullptr;
        z = gates ? (const T*)p.z + d : x;   // without a gate: read and not used
        y = (T*)p.y + d;
        bc = (sfloat*)(uintptr_t)p.bc;
        sdelta = p.sdelta; sx = p.sx; sz = gates ? p.sz : p.sx; sy = p.sy;
#pragma unroll
        for (int n = 0; n < N; ++n) a[n] = p.A[(int64_t)d * N + n] * kLog2e;
        bias = p.stepf.bias ? p.stepf.bias[d] : 0.0f;
        skip = p.skip ? p.skip[d] : 0.0f;
        skips = p.skip != nullptr;
        softplus = p.stepf.softplus;
    }
    template <bool OUT>
    __device__ __forceinline__ void row(int t, float d, float xv, float zv) {
        sfloat* r = bc + (int64_t)t * (2 * N);
        const float u = d * xv;
        float o = 0.0f;
        if (!OUT) dsum += d;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            h[n] = fmaf(__builtin_amdgcn_exp2f(a[n] * d), h[n], u * r[n]);
            if (OUT) o = fmaf(h[n], r[N + n], o);
        }
        if (OUT) {
            if (skips) o = fmaf(skip, xv, o);
            if (gates) o *= zv * sigmoid_f(zv);
            y[(int64_t)t * sy] = to_stream<T>(o);
        }
    }
    // rows [t0, t1), t0 < t1: the next group's loads are under way while a group is computed
    template <bool OUT>
    __device__ __forceinline__ void walk(int t0, int t1) {
        T rd[kGrp], rx[kGrp], rz[kGrp];
        auto load = [&](int t) {
#pragma unroll
            for (int g = 0; g < kGrp; ++g) {
                const int64_t r = min(t + g, t1 - 1);
                rd[g] = delta[r * sdelta];
                rx[g] = x[r * sx];
                if (OUT) rz[g] = z[r * sz];
            }
        };
        load(t0);
        for (int t = t0; t < t1; t += kGrp) {
            float dl[kGrp], xv[kGrp], zv[kGrp];
#pragma unroll
            for (int g = 0; g < kGrp; ++g) {
                dl[g] = to_f32(rd[g]) + bias;
                xv[g] = to_f32(rx[g]);
                zv[g] = OUT ? to_f32(rz[g]) : 0.0f;
            }
            load(min(t + kGrp, t1 - 1));
            if (softplus) {
#pragma unroll
                for (int g = 0; g < kGrp; ++g) dl[g] = softplus_t(dl[g]);
            }
            if (t + kGrp <= t1) {
#pragma unroll
                for (int g = 0; g < kGrp; ++g) row<OUT>(t + g, dl[g], xv[g], zv[g]);
            } else {
#pragma unroll
                for (int g = 0; g < kGrp - 1; ++g)
                    if (t + g < t1) row<OUT>(t + g, dl[g], xv[g], zv[g]);
            }
        }
    }
};
template <int N>
__device__ __forceinline__ void load_states(const float* p, float (&h)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n) h[n] = p[n];
}

// Range c's rows [r0, r1), and the workspace's per-range state at [c][n][d].
struct Range_ {
    int r0, r1;
};
__device__ __forceinline__ Range_ rows_of(const TokScanParams& p, int c) {
    const int r0 = c * p.rows;
    return {r0, min(r0 + p.rows, p.q.T)};
}

// First pass, ranges 0 .. nrange-2.
template <typename T, int N>
__global__ __launch_bounds__(256) void tok_scan_sum_kernel(TokScanParams p, int cblocks) {
    const int cb = blockIdx.x % cblocks;
    const int c = uniform((blockIdx.x / cblocks) * 4 + (threadIdx.x >> 6));
    if (c >= p.nrange - 1) return;
    const Range_ r = rows_of(p, c);
    const int s = uniform(find_seq(p.q.start, p.q.S, r.r1 - 1));
    if (s < 0 || s >= p.q.S) return;
    const int st = uniform(p.q.start[s]), en = uniform(min(p.q.start[s + 1], p.q.T));
    if (st < 0 || en <= r.r1) return;   // none crosses the end
    const int slot = uniform(slot_of(p.q, s));
    if (slot < 0) return;
    // lanes past the last channel repeat it: the same values to the same places, without a branch a row
    const int d = min(cb * 64 + lane_id(), p.D - 1);
    ScanLane<T, N> l(p, d);
    const int64_t at = (int64_t)c * N * p.D + d;
#pragma unroll
    for (int n = 0; n < N; ++n) l.h[n] = 0.0f;
    l.dsum = 0.0f;
    if (st >= r.r0) {   // it begins here: its first state, kept for the second pass (which may find it overwritten)
        if (!(p.q.fresh && p.q.fresh[s])) load_states<N>(p.pool + slot * p.spool + (int64_t)d * N, l.h);
#pragma unroll
        for (int n = 0; n < N; ++n) p.h0[at + (int64_t)n * p.D] = l.h[n];
    }
    l.template walk<false>(max(st, r.r0), r.r1);
#pragma unroll
    for (int n = 0; n < N; ++n) p.hsum[at + (int64_t)n * p.D] = l.h[n];
    p.dsum[(int64_t)c * p.D + d] = l.dsum;
}

// Second pass: every row's output and every sequence's last state.
template <typename T, int N>
__global__ __launch_bounds__(256) void tok_scan_kernel(TokScanParams p, int cblocks) {
    const int cb = blockIdx.x % cblocks;
    const int c = uniform((blockIdx.x / cblocks) * 4 + (threadIdx.x >> 6));
    if (c >= p.nrange) return;
    const Range_ r = rows_of(p, c);
    int s = uniform(find_seq(p.q.start, p.q.S, r.r0));
    if (s >= p.q.S) return;
    const int d = min(cb * 64 + lane_id(), p.D - 1);
    ScanLane<T, N> l(p, d);
    if (s < 0) s = 0;
    for (; s < p.q.S; ++s) {
        const int st = uniform(p.q.start[s]);
        if (st >= r.r1) break;
        const int en = uniform(min(p.q.start[s + 1], p.q.T));
        if (st < 0 || en <= max(st, r.r0)) continue;
        const int slot = uniform(slot_of(p.q, s));
        if (slot < 0) continue;
        float* pool = p.pool + slot * p.spool + (int64_t)d * N;
#pragma unroll
        for (int n = 0; n < N; ++n) l.h[n] = 0.0f;
        if (st < r.r0) {   // from the ranges before: the state that crosses into this one
            for (int k = st / p.rows; k < c; ++k) {
                const float ds = p.dsum[(int64_t)k * p.D + d];
                const float* S = p.hsum + (int64_t)k * N * p.D + d;
#pragma unroll
                for (int n = 0; n < N; ++n)
                    l.h[n] = fmaf(__builtin_amdgcn_exp2f(l.a[n] * ds), l.h[n], S[(int64_t)n * p.D]);
            }
        } else if (en > r.r1) {
            const float* S = p.h0 + (int64_t)c * N * p.D + d;
#pragma unroll
            for (int n = 0; n < N; ++n) l.h[n] = S[(int64_t)n * p.D];
        } else if (!(p.q.fresh && p.q.fresh[s])) {
            load_states<N>(pool, l.h);
        }
        l.template walk<true>(max(st, r.r0), min(en, r.r1));
        if (en <= r.r1) {
#pragma unroll
            for (int n = 0; n < N; ++n) pool[n] = l.h[n];
        }
    }
}

// One row a sequence.  Q lanes a channel, four states each (the last lane's may
// be fewer); VEC: the states of a lane are one 16-byte access.
template <typename T, int Q, bool VEC>
__global__ __launch_bounds__(256) void tok_step_kernel(TokScanParams p, int cblocks) {
    const int s = blockIdx.x / cblocks;
    const int i = (blockIdx.x % cblocks) * 256 + (int)threadIdx.x;
    const int d0 = i / Q, q = i % Q;
    const bool act = d0 < p.D;
    const int d = act ? d0 : 0, n0 = 4 * q, N = p.N;
    const bool four = n0 + 4 <= N;   // VEC: all of a lane's states or (N = 12) none
    const int slot = uniform(slot_of(p.q, s));
    if (slot < 0) return;
    const int64_t t = s;
    float* pool = p.pool + slot * p.spool + (int64_t)d * N + n0;
    const float* A = p.A + (int64_t)d * N + n0;
    const T* B = (const T*)p.Bm + t * p.sB + n0;
    const T* C = (const T*)p.C + t * p.sC + n0;
    const bool fresh = p.q.fresh && p.q.fresh[s];
    float h[4] = {}, a[4] = {}, b[4], c[4];
    if (VEC && four) {
        const float4 av = *reinterpret_cast<const float4*>(A);
        a[0] = av.x; a[1] = av.y; a[2] = av.z; a[3] = av.w;
        if (!fresh) {
            const float4 hv = *reinterpret_cast<const float4*>(pool);
            h[0] = hv.x; h[1] = hv.y; h[2] = hv.z; h[3] = hv.w;
        }
    } else if (!VEC) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (n0 + e < N) {
                a[e] = A[e];
                if (!fresh) h[e] = pool[e];
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        b[e] = n0 + e < N ? to_f32(B[e]) : 0.0f;
        c[e] = n0 + e < N ? to_f32(C[e]) : 0.0f;
    }
    float dl = to_f32(((const T*)p.delta)[t * p.sdelta + d]) + (p.stepf.bias ? p.stepf.bias[d] : 0.0f);
    if (p.stepf.softplus) dl = softplus_t(dl);
    const float x = to_f32(((const T*)p.x)[t * p.sx + d]);
    const float u = dl * x;
    float y = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (n0 + e < N) {
            h[e] = fmaf(__builtin_amdgcn_exp2f(a[e] * kLog2e * dl), h[e], u * b[e]);
            y = fmaf(h[e], c[e], y);
        }
    }
    if (Q > 1) y += dpp<SSM_DPP_QUAD(1, 0, 3, 2)>(0.0f, y);
    if (Q > 2) y += dpp<SSM_DPP_QUAD(2, 3, 0, 1)>(0.0f, y);
    if (!act) return;
    if (VEC) {
        if (four) *reinterpret_cast<float4*>(pool) = make_float4(h[0], h[1], h[2], h[3]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n0 + e < N) pool[e] = h[e];
    }
    if (q == 0) {
        if (p.skip) y = fmaf(p.skip[d], x, y);
        if (p.z) {
            const float z = to_f32(((const T*)p.z)[t * p.sz + d]);
            y *= z * sigmoid_f(z);
        }
        ((T*)p.y)[t * p.sy + d] = to_stream<T>(y);
    }
}

template <typename T>
hipError_t tok_step(const TokScanParams& p, hipStream_t st) {
    const int q = p.N <= 4 ? 1 : p.N <= 8 ? 2 : 4;
    const int64_t cblocks = ((int64_t)p.D * q + 255) / 256, blocks = cblocks * p.q.S;
    if (blocks >= (1LL << 31)) return hipErrorInvalidValue;
    const unsigned g = (unsigned)blocks;
    const int cb = (int)cblocks;
    if (p.vec) {   // N a multiple of 4: a lane has four states or none
        if (q == 1) tok_step_kernel<T, 1, true><<<g, 256, 0, st>>>(p, cb);
        else if (q == 2) tok_step_kernel<T, 2, true><<<g, 256, 0, st>>>(p, cb);
        else tok_step_kernel<T, 4, true><<<g, 256, 0, st>>>(p, cb);
    } else {
        if (q == 1) tok_step_kernel<T, 1, false><<<g, 256, 0, st>>>(p, cb);
        else if (q == 2) tok_step_kernel<T, 2, false><<<g, 256, 0, st>>>(p, cb);
        else tok_step_kernel<T, 4, false><<<g, 256, 0, st>>>(p, cb);
    }
    return hipGetLastError();
}

template <typename T, int N>
hipError_t tok_scan_n(const TokScanParams& p, bool sum, hipStream_t st) {
    const int64_t cblocks = ((int64_t)p.D + 63) / 64;
    const int64_t groups = ((int64_t)(sum ? p.nrange - 1 : p.nrange) + 3) / 4;
    if (cblocks * groups >= (1LL << 31)) return hipErrorInvalidValue;
    const unsigned g = (unsigned)(cblocks * groups);
    if (sum) tok_scan_sum_kernel<T, N><<<g, 256, 0, st>>>(p, (int)cblocks);
    else tok_scan_kernel<T, N><<<g, 256, 0, st>>>(p, (int)cblocks);
    return hipGetLastError();
}
template <typename T>
hipError_t tok_scan_t(const TokScanParams& p, bool sum, hipStream_t st) {
    switch (p.N) {
#define SSM_N(n) case n: return tok_scan_n<T, n>(p, sum, st);
        SSM_N(1) SSM_N(2) SSM_N(3) SSM_N(4) SSM_N(5) SSM_N(6) SSM_N(7) SSM_N(8)
        SSM_N(9) SSM_N(10) SSM_N(11) SSM_N(12) SSM_N(13) SSM_N(14) SSM_N(15) SSM_N(16)
#undef SSM_N
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_tok_step(const TokScanParams& p, int dtype, hipStream_t st) {
    return dtype == 1 ? tok_step<bf16_t>(p, st) : tok_step<float>(p, st);
}
hipError_t launch_tok_bc(const TokScanParams& p, int dtype, hipStream_t st) {
    const int64_t blocks = ((int64_t)p.q.T * 2 * p.N + 255) / 256;
    if (blocks >= (1LL << 31)) return hipErrorInvalidValue;
    if (dtype == 1) tok_bc_kernel<bf16_t><<<(unsigned)blocks, 256, 0, st>>>(p);
    else tok_bc_kernel<float><<<(unsigned)blocks, 256, 0, st>>>(p);
    return hipGetLastError();
}
hipError_t launch_tok_scan(const TokScanParams& p, int dtype, bool sum, hipStream_t st) {
    return dtype == 1 ? tok_scan_t<bf16_t>(p, sum, st) : tok_scan_t<float>(p, sum, st);
}

}  // namespace ssm
