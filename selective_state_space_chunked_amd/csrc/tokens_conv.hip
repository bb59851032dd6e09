// The short causal convolution over packed rows: the tokens of all sequences of
// a call are the rows of one matrix, lanes run along the channels, and each
// sequence's last W-1 inputs come from and return to its slot of a pool.
#include <algorithm>

#include "tokens.hpp"

namespace ssm {
namespace {

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

}  // namespace

hipError_t launch_tok_conv(const TokConvParams& p, int dtype, hipStream_t st) {
    if (dtype == 1)
        return p.W == 2 ? tok_conv_w<bf16_t, 2>(p, st) : p.W == 3 ? tok_conv_w<bf16_t, 3>(p, st) : tok_conv_w<bf16_t, 4>(p, st);
    return p.W == 2 ? tok_conv_w<float, 2>(p, st) : p.W == 3 ? tok_conv_w<float, 3>(p, st) : tok_conv_w<float, 4>(p, st);
}

}  // namespace ssm
