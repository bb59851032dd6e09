// The short causal convolution over packed rows: the tokens of all sequences of
// a call are the rows of one matrix, and each sequence's last W-1 inputs come
// from and return to its slot of a pool.
//
// A lane takes four neighbouring channels, so a wave reads and writes whole lines
// of a row, and keeps the W-1 inputs before its rows in registers while it walks
// down a run of them, four rows' loads under way at a time.  A few operations an
// element: bound by HBM (8192 rows x 4096 channels in bf16: 134 MB in 32 us),
// single tokens by the latency of their loads (64 x 2048: 2.8 us).
#include <algorithm>

#include "tokens.hpp"

namespace ssm {
namespace {

// A wave takes the runs of kTokRun rows.  A sequence's first W-1 rows and its new
// state belong to the run its first row lies in (which then reaches past its end
// where the sequence starts in its last rows), so only that wave reads and
// writes the slot.
constexpr int kTokRun = 16;
constexpr int kTokGrp = 4;   // rows whose loads are issued together

// FULL: every lane has all its channels.
template <typename T, int W, bool FULL>
struct ConvLane {
    static constexpr int V = Vec<T>::V, H = W - 1;
    const T* x;
    T *y, *pool;
    int64_t sx, sy, spool;
    float w[V][W], bias[V];
    int silu, cnt;     // channels of the lane, 0 past the last one
    float win[H][V];   // the inputs before the next row

    __device__ __forceinline__ ConvLane(const TokConvParams& p, int c0) {
        cnt = max(min(V, p.D - c0), 0);
        const int c = cnt > 0 ? c0 : 0;
        x = (const T*)p.x + c;
        y = (T*)p.y + c;
        pool = (T*)p.pool + (int64_t)c * H;
        sx = p.sx; sy = p.sy; spool = p.spool; silu = p.silu;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int ci = FULL || i < cnt ? c + i : c;
#pragma unroll
            for (int k = 0; k < W; ++k) w[i][k] = p.w[(int64_t)ci * W + k];
            bias[i] = p.bias ? p.bias[ci] : 0.0f;
        }
    }
    __device__ __forceinline__ void load_row(int t, Vec<T>& v) const {
        if (FULL) v.load(x + t * sx);
        else v.load(x + t * sx, cnt);
    }
    // rows t .. t+G-1, as loaded, of which the first n are there
    template <int G>
    __device__ __forceinline__ void rows(int t, const Vec<T>* r, int n) {
        float e[H + G][V];
#pragma unroll
        for (int i = 0; i < H; ++i)
#pragma unroll
            for (int c = 0; c < V; ++c) e[i][c] = win[i][c];
#pragma unroll
        for (int g = 0; g < G; ++g) r[g].get(e[H + g]);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (g > 0 && g >= n) continue;
            float o[V];
#pragma unroll
            for (int c = 0; c < V; ++c) {
                float a = bias[c];
#pragma unroll
                for (int k = 0; k < W; ++k) a = fmaf(w[c][k], e[g + k][c], a);
                o[c] = silu ? a * sigmoid_f(a) : a;
            }
            Vec<T> q;
            q.set(o);
            if (FULL) q.store(y + (t + g) * sy);
            else q.store(y + (t + g) * sy, cnt);
        }
#pragma unroll
        for (int i = 0; i < H; ++i)   // of a group with fewer rows the window is not used again
#pragma unroll
            for (int c = 0; c < V; ++c) win[i][c] = e[G + i][c];
    }
    __device__ __forceinline__ void window(const Vec<T>* r) {
#pragma unroll
        for (int i = 0; i < H; ++i) r[i].get(win[i]);
    }
    // rows [t0, t1): the next group's loads are under way while a group is computed
    __device__ __forceinline__ void walk(int t0, int t1) {
        Vec<T> r[kTokGrp];
        if (t0 >= t1) return;
#pragma unroll
        for (int g = 0; g < kTokGrp; ++g) load_row(min(t0 + g, t1 - 1), r[g]);
        walk(t0, t1, r);
    }
    // (whole groups apart: with the same loads and stores in every turn a wait is for a group's loads alone)
    __device__ __forceinline__ void walk(int t0, int t1, Vec<T> (&r)[kTokGrp]) {   // r: the first group
#pragma unroll
        for (int g = 0; g < kTokGrp; ++g) r[g].arrived();
        int t = t0;
        for (; t + kTokGrp <= t1; t += kTokGrp) {
            Vec<T> nx[kTokGrp];
#pragma unroll
            for (int g = 0; g < kTokGrp; ++g) load_row(min(t + kTokGrp + g, t1 - 1), nx[g]);
            rows<kTokGrp>(t, r, kTokGrp);
#pragma unroll
            for (int g = 0; g < kTokGrp; ++g) r[g] = nx[g];
        }
        if (t < t1) rows<kTokGrp>(t, r, t1 - t);
    }
    // the slot's inputs, [channel][oldest first]
    __device__ __forceinline__ void load_state(int slot, Vec<T> (&h)[H]) const {
        const T* s = pool + slot * spool;
#pragma unroll
        for (int i = 0; i < H; ++i) {
            if (FULL) h[i].load(s + i * V);
            else h[i].load(s + i * V, cnt * H - i * V);
        }
    }
    __device__ __forceinline__ void store_state(int slot, const float (&h)[V * H]) const {
        T* s = pool + slot * spool;
#pragma unroll
        for (int i = 0; i < H; ++i) {
            float v[V];
#pragma unroll
            for (int c = 0; c < V; ++c) v[c] = h[i * V + c];
            Vec<T> q;
            q.set(v);
            if (FULL) q.store(s + i * V);
            else q.store(s + i * V, cnt * H - i * V);
        }
    }
    // The window a sequence begins with and the state it leaves: its last H inputs, of the rows and, where it is
    // shorter, the state before.
    __device__ __forceinline__ void begin(const Vec<T> (&old)[H], bool fresh, int st, int len, float (&nh)[V * H]) {
        float h[V * H];
#pragma unroll
        for (int i = 0; i < H; ++i) {
            float v[V];
            old[i].get(v);
#pragma unroll
            for (int c = 0; c < V; ++c) h[i * V + c] = fresh ? 0.0f : v[c];
        }
#pragma unroll
        for (int i = 0; i < H; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) win[i][e] = h[e * H + i];
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const int at = len - H + i;   // place of the input in the sequence
            float v[V];
            if (at >= 0) {
                Vec<T> r;
                load_row(st + at, r);
                r.get(v);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    v[e] = 0.0f;
#pragma unroll
                    for (int k = 0; k < H; ++k) v[e] = k == len + i ? h[e * H + k] : v[e];
                }
            }
#pragma unroll
            for (int e = 0; e < V; ++e) nh[e * H + i] = v[e];
        }
    }
};

template <typename T, int W, bool FULL>
__device__ __forceinline__ void rows_of_wave(const TokConvParams& p, int c0, int64_t unit) {
    constexpr int H = W - 1, V = Vec<T>::V;
    const int r0 = (int)min(unit * kTokRun, (int64_t)p.q.T), r1 = min(r0 + kTokRun, p.q.T);
    if (r0 >= r1) return;
    const SeqTable q(p.q);
    ConvLane<T, W, FULL> l(p, c0);
    // what most waves begin with, whichever sequence the rows belong to: the first rows and those before them
    Vec<T> before[H], head[kTokGrp];
#pragma unroll
    for (int i = 0; i < H; ++i) l.load_row(max(r0 - H + i, 0), before[i]);
#pragma unroll
    for (int g = 0; g < kTokGrp; ++g) l.load_row(min(r0 + g, r1 - 1), head[g]);
    int s = q.find(r0);
    if (s >= p.q.S) return;
    if (s >= 0) {   // the sequence that runs into this range
        const int st = q.first(s), en = q.end(s);
        if (st >= 0 && st < r0) {
            const int t0 = max(r0, st + H), t1 = min(en, r1);
            if (t0 < t1 && q.slot(s) >= 0) {
                if (t0 == r0) {
                    l.window(before);
                    l.walk(t0, t1, head);
                } else {   // its first H rows are the wave's before
#pragma unroll
                    for (int i = 0; i < H; ++i) l.load_row(t0 - H + i, before[i]);
                    l.window(before);
                    l.walk(t0, t1);
                }
            }
        }
        if (st < r0) ++s;
    } else {
        s = 0;
    }
    for (; s < p.q.S; ++s) {   // sequences whose first row lies in this range
        const int st = q.first(s);
        if (st >= r1) break;
        const int en = q.end(s);
        if (st < r0 || en <= st) continue;
        const int slot = q.slot(s);
        if (slot < 0) continue;
        Vec<T> old[H];
        float nh[V * H];
        l.load_state(slot, old);
        l.begin(old, q.fresh(s), st, en - st, nh);
        l.store_state(slot, nh);
        l.walk(st, min(en, max(r1, st + H)));
    }
}
template <typename T, int W>
__global__ __launch_bounds__(256) void tok_conv_kernel(TokConvParams p, int cblocks) {
    constexpr int V = Vec<T>::V;
    const int cb = blockIdx.x % cblocks;
    const int64_t unit = (int64_t)(blockIdx.x / cblocks) * 4 + uniform(threadIdx.x >> 6);
    const int c0 = (cb * 64 + lane_id()) * V;
    if ((cb + 1) * 64 * V <= p.D) rows_of_wave<T, W, true>(p, c0, unit);
    else rows_of_wave<T, W, false>(p, c0, unit);
}

// One row a sequence: the state is loaded from the slot that is named, and what
// decides whether the sequence has it comes in meanwhile.
template <typename T, int W, bool FULL>
__device__ __forceinline__ void step_of_wave(const TokConvParams& p, int c0, int s) {
    constexpr int H = W - 1, V = Vec<T>::V;
    const int slot = uniform(slot_named(p.q, s));
    ConvLane<T, W, FULL> l(p, c0);
    Vec<T> old[H], r;
    l.load_row(s, r);
    if (slot < 0) return;
    l.load_state(slot, old);
    const bool fresh = p.q.fresh && p.q.fresh[s];
    if (slot_taken(p.q, s, slot)) return;
    float nh[V * H];
    l.begin(old, fresh, s, 1, nh);
    l.store_state(slot, nh);
    l.template rows<1>(s, &r, 1);
}
template <typename T, int W>
__global__ __launch_bounds__(64) void tok_conv_step_kernel(TokConvParams p, int cblocks) {
    constexpr int V = Vec<T>::V;
    const int cb = blockIdx.x % cblocks, s = blockIdx.x / cblocks;
    const int c0 = (cb * 64 + lane_id()) * V;
    if ((cb + 1) * 64 * V <= p.D) step_of_wave<T, W, true>(p, c0, s);
    else step_of_wave<T, W, false>(p, c0, s);
}

template <typename T, int W>
hipError_t tok_conv_w(const TokConvParams& p, hipStream_t st) {
    const int64_t wide = 64 * Vec<T>::V, cblocks = (p.D + wide - 1) / wide;
    const int64_t units = p.q.start ? (((int64_t)p.q.T + kTokRun - 1) / kTokRun + 3) / 4 : p.q.S;
    const int64_t blocks = cblocks * units;
    if (blocks >= (1LL << 31)) return hipErrorInvalidValue;
    if (p.q.start) tok_conv_kernel<T, W><<<(unsigned)blocks, 256, 0, st>>>(p, (int)cblocks);
    else tok_conv_step_kernel<T, W><<<(unsigned)blocks, 64, 0, st>>>(p, (int)cblocks);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_tok_conv(const TokConvParams& p, int dtype, hipStream_t st) {
    if (dtype == 1)
        return p.W == 2 ? tok_conv_w<bf16_t, 2>(p, st) : p.W == 3 ? tok_conv_w<bf16_t, 3>(p, st) : tok_conv_w<bf16_t, 4>(p, st);
    return p.W == 2 ? tok_conv_w<float, 2>(p, st) : p.W == 3 ? tok_conv_w<float, 3>(p, st) : tok_conv_w<float, 4>(p, st);
}

}  // namespace ssm
