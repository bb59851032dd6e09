// The short causal convolution and the selective scan over packed rows: the
// tokens of all sequences of a call are the rows of one matrix, lanes run along
// the channels, and each sequence's state comes from and returns to its slot of
// a pool.
#include <algorithm>

#include "common.hpp"
#include "kernels.hpp"

namespace ssm {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float sigmoid_f(float v) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * kLog2e));
}
__device__ __forceinline__ float softplus_t(float v) { return v > 20.0f ? v : log1pf(expf(v)); }

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

// ---------------------------------------------------------------------------
// convolution
// ---------------------------------------------------------------------------
// A wave takes 64 * V channels of a run of kTokRun rows.  A sequence's first
// W-1 rows and its new state belong to the run its first row lies in (which then
// reaches past its end where the sequence starts in its last rows), so only
// that wave reads and writes the slot.
constexpr int kTokRun = 16;

template <typename T, int W, int V>
struct ConvLane {
    const T* x; T* y; T* pool;
    int64_t sx, sy, spool;
    float w[V][W], bias[V];
    int silu;
    bool act;
    float win[W - 1][V];   // the W-1 inputs before the next row

    __device__ __forceinline__ void load_row(int t, float (&v)[V]) const { load_v<T, V>(x + t * sx, v); }
    __device__ __forceinline__ void step(int t) {
        float v[V], o[V];
        load_row(t, v);
#pragma unroll
        for (int c = 0; c < V; ++c) {
            float a = bias[c];
#pragma unroll
            for (int k = 0; k < W - 1; ++k) a = fmaf(w[c][k], win[k][c], a);
            a = fmaf(w[c][W - 1], v[c], a);
            o[c] = silu ? a * sigmoid_f(a) : a;
#pragma unroll
            for (int k = 0; k + 1 < W - 1; ++k) win[k][c] = win[k + 1][c];
            win[W - 2][c] = v[c];
        }
        if (act) store_v<T, V>(y + t * sy, o);
    }
    // the slot's inputs (or zeros), oldest first
    __device__ __forceinline__ void load_state(int slot, bool fresh, float (&h)[V * (W - 1)]) const {
#pragma unroll
        for (int i = 0; i < V * (W - 1); ++i) h[i] = 0.0f;
        if (fresh) return;
        const T* s = pool + slot * spool;
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            float v[V];
            load_v<T, V>(s + i * V, v);
#pragma unroll
            for (int c = 0; c < V; ++c) h[i * V + c] = v[c];
        }
    }
    __device__ __forceinline__ void store_state(int slot, const float (&h)[V * (W - 1)]) const {
        if (!act) return;
        T* s = pool + slot * spool;
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            float v[V];
#pragma unroll
            for (int c = 0; c < V; ++c) v[c] = h[i * V + c];
            store_v<T, V>(s + i * V, v);
        }
    }
};

template <typename T, int W, int V, bool STEP>
__global__ __launch_bounds__(256) void tok_conv_kernel(TokConvParams p, int cblocks) {
    const int cb = blockIdx.x % cblocks;
    const int64_t unit = (int64_t)(blockIdx.x / cblocks) * 4 + (threadIdx.x >> 6);   // run of rows, or sequence
    const int c0 = (cb * 64 + lane_id()) * V;
    ConvLane<T, W, V> l;
    l.act = c0 < p.D;
    const int c = l.act ? c0 : 0;
    l.x = (const T*)p.x + c; l.y = (T*)p.y + c; l.pool = (T*)p.pool + (int64_t)c * (W - 1);
    l.sx = p.sx; l.sy = p.sy; l.spool = p.spool; l.silu = p.silu;
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int k = 0; k < W; ++k) l.w[i][k] = p.w[(int64_t)(c + i) * W + k];
        l.bias[i] = p.bias ? p.bias[c + i] : 0.0f;
    }
    float h[V * (W - 1)];
    auto begin = [&](int s, int slot, int st, int len) {   // window and new state of a sequence
        l.load_state(slot, p.q.fresh && p.q.fresh[s], h);
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) l.win[i][e] = h[e * (W - 1) + i];
        float nh[V * (W - 1)];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            const int at = len - (W - 1) + i;   // place of the input in the sequence
            float v[V];
            if (at >= 0) {
                l.load_row(st + at, v);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    v[e] = 0.0f;
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) v[e] = k == len + i ? h[e * (W - 1) + k] : v[e];
                }
            }
#pragma unroll
            for (int e = 0; e < V; ++e) nh[e * (W - 1) + i] = v[e];
        }
        l.store_state(slot, nh);
    };
    if (STEP) {
        if (unit >= p.q.S) return;
        const int slot = slot_of(p.q, (int)unit);
        if (slot < 0) return;
        begin((int)unit, slot, (int)unit, 1);
        l.step((int)unit);
        return;
    }
    const int r0 = (int)min(unit * kTokRun, (int64_t)p.q.T), r1 = min(r0 + kTokRun, p.q.T);
    if (r0 >= r1) return;
    const int32_t* start = p.q.start;
    int s = find_seq(start, p.q.S, r0);
    if (s >= p.q.S) return;
    if (s >= 0) {   // the sequence that runs into this range
        const int st = start[s], en = min(start[s + 1], p.q.T);
        if (st >= 0 && st < r0) {
            const int t0 = max(r0, st + W - 1), t1 = min(en, r1);
            if (t0 < t1 && slot_of(p.q, s) >= 0) {
#pragma unroll
                for (int i = 0; i < W - 1; ++i) l.load_row(t0 - (W - 1) + i, l.win[i]);
                for (int t = t0; t < t1; ++t) l.step(t);
            }
        }
        if (st < r0) ++s;
    } else {
        s = 0;
    }
    for (; s < p.q.S; ++s) {   // sequences whose first row lies in this range
        const int st = start[s];
        if (st >= r1) break;
        const int en = min(start[s + 1], p.q.T);
        if (st < r0 || en <= st) continue;
        const int slot = slot_of(p.q, s);
        if (slot < 0) continue;
        begin(s, slot, st, en - st);
        const int t1 = min(en, max(r1, st + W - 1));
        for (int t = st; t < t1; ++t) l.step(t);
    }
}

template <typename T, int W>
hipError_t tok_conv_w(const TokConvParams& p, hipStream_t st) {
    constexpr int V = 16 / (int)sizeof(T);
    const int64_t v = p.vec ? V : 1;
    const int64_t cblocks = (p.D + 64 * v - 1) / (64 * v);
    const int64_t units = p.q.start ? ((int64_t)p.q.T + kTokRun - 1) / kTokRun : p.q.S;
    const int64_t blocks = cblocks * ((units + 3) / 4);
    if (blocks >= (1LL << 31)) return hipErrorInvalidValue;
    const unsigned g = (unsigned)blocks;
    if (p.vec) {
        if (p.q.start) tok_conv_kernel<T, W, V, false><<<g, 256, 0, st>>>(p, (int)cblocks);
        else tok_conv_kernel<T, W, V, true><<<g, 256, 0, st>>>(p, (int)cblocks);
    } else {
        if (p.q.start) tok_conv_kernel<T, W, 1, false><<<g, 256, 0, st>>>(p, (int)cblocks);
        else tok_conv_kernel<T, W, 1, true><<<g, 256, 0, st>>>(p, (int)cblocks);
    }
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// selective scan: a lane walks one channel of one sequence, its states in registers
// ---------------------------------------------------------------------------
template <typename T>
__global__ __launch_bounds__(64) void tok_scan_kernel(TokScanParams p, int cblocks) {
    constexpr int NM = 16;
    const int cb = blockIdx.x % cblocks, s = blockIdx.x / cblocks;
    int st = s, en = s + 1;
    if (p.q.start) {
        st = p.q.start[s];
        en = min(p.q.start[s + 1], p.q.T);
    }
    if (st < 0 || st >= en) return;
    const int slot = slot_of(p.q, s);
    if (slot < 0) return;
    const int d = cb * 64 + lane_id();
    if (d >= p.D) return;
    const int N = p.N;
    float* pool = p.pool + slot * p.spool + (int64_t)d * N;
    float h[NM], a[NM];
    const bool fresh = p.q.fresh && p.q.fresh[s];
#pragma unroll
    for (int n = 0; n < NM; ++n) {
        h[n] = n < N && !fresh ? pool[n] : 0.0f;
        a[n] = n < N ? p.A[(int64_t)d * N + n] * kLog2e : 0.0f;
    }
    const float bias = p.stepf.bias ? p.stepf.bias[d] : 0.0f, skip = p.skip ? p.skip[d] : 0.0f;
    for (int t = st; t < en; ++t) {
        float dl = to_f32(((const T*)p.delta)[t * p.sdelta + d]) + bias;
        if (p.stepf.softplus) dl = softplus_t(dl);
        const float x = to_f32(((const T*)p.x)[t * p.sx + d]);
        const T* B = (const T*)p.Bm + t * p.sB;
        const T* C = (const T*)p.C + t * p.sC;
        const float u = dl * x;
        float y = 0.0f;
#pragma unroll
        for (int n = 0; n < NM; ++n) {
            if (n < N) {
                h[n] = fmaf(__builtin_amdgcn_exp2f(a[n] * dl), h[n], u * to_f32(B[n]));
                y = fmaf(h[n], to_f32(C[n]), y);
            }
        }
        if (p.skip) y = fmaf(skip, x, y);
        if (p.z) {
            const float z = to_f32(((const T*)p.z)[t * p.sz + d]);
            y *= z * sigmoid_f(z);
        }
        ((T*)p.y)[t * p.sy + d] = from_f32<T>(y);
    }
#pragma unroll
    for (int n = 0; n < NM; ++n)
        if (n < N) pool[n] = h[n];
}

template <typename T>
hipError_t tok_scan_t(const TokScanParams& p, hipStream_t st) {
    const int64_t cblocks = (p.D + 63) / 64, blocks = cblocks * p.q.S;
    if (blocks >= (1LL << 31)) return hipErrorInvalidValue;
    tok_scan_kernel<T><<<(unsigned)blocks, 64, 0, st>>>(p, (int)cblocks);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_tok_conv(const TokConvParams& p, int dtype, hipStream_t st) {
    if (dtype == 1)
        return p.W == 2 ? tok_conv_w<bf16_t, 2>(p, st) : p.W == 3 ? tok_conv_w<bf16_t, 3>(p, st) : tok_conv_w<bf16_t, 4>(p, st);
    return p.W == 2 ? tok_conv_w<float, 2>(p, st) : p.W == 3 ? tok_conv_w<float, 3>(p, st) : tok_conv_w<float, 4>(p, st);
}
hipError_t launch_tok_scan(const TokScanParams& p, int dtype, hipStream_t st) {
    return dtype == 1 ? tok_scan_t<bf16_t>(p, st) : tok_scan_t<float>(p, st);
}

}  // namespace ssm
