// The selective scan over packed rows, with its layer's skip and gate:
//
//   h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t,  y_t = (C_t . h_t + skip x_t) z_t sigmoid(z_t)
//
// Prompts.  A lane holds one channel with its N states; a wave walks 64
// channels down a range of rows, so the streams are read along the channels as
// the projections write them.  B_t, C_t are the same for the whole wave: 16 rows
// of them at a time go to LDS as fp32 and come back as broadcast 16-byte reads.
// Per state and row that leaves a multiply and an exp2 for the transition, a
// multiply for the state, a quarter of a matrix instruction for the input term
// and one multiply-add for y.  Few long sequences do not fill the GPU, so the rows are cut into ranges whatever
// the sequences' lengths: a first pass leaves, for the sequence that crosses the
// end of each range, its state there (from zero where it runs through the whole
// range) and the sum of its step sizes; a small kernel composes them,
//   h <- exp(A sum delta) h + S,
// and the second pass walks every range from the state that enters it.
//
// The passes are bound by the issue of these instructions (an exp2 takes 8
// cycles, the others 2 to 3): the main loops hold 217 (first pass) and 314 vector
// instructions for four rows, 208 and 272 of them the state's own; loads by
// scalar addresses and B, C by way of LDS leave the rest that small.  8192 rows x
// 2048 channels x 16 states in bf16, 13 sequences: 46 us, 10 us between and 59 us
// (17000 x 1024, one sequence: 48, 10 and 58), where the streams alone are 28 us of
// memory traffic.  Of each pass about 10 us do not shrink with the rows: a wave's first loads follow one
// another (lists of sequences, A, states, rows).  Each sequence in a range is walked from its own first loads on, so
// many short ones among long ones cost more: 8 sequences of 1024 rows and 256 of one row take 338 us (in 9 sequences
// 117 us), 1024 of 8 rows 128 us, all at 2048 channels.
//
// Single tokens.  Bound by the states' traffic: four states a lane, so a wave
// reads and writes the pool in whole lines.  256 x 4096 x 16 with 32 places empty: 125 MB in 25 us,
// 5.0 TB/s; one sequence of 2048 channels: 3.5 us, the latency of its loads.
#include <algorithm>

#include "buffer.hpp"
#include "tokens.hpp"

namespace ssm {
namespace {

// The streams are read through buffers (kept as flat pointers the compiler spends two vector registers and a 64-bit
// vector addition on every access).
constexpr uint32_t kAll = 0xffffffffu;   // rows of a group: in bounds by their index, no limit wanted

typedef float f4 __attribute__((ext_vector_type(4)));
constexpr int kScanWaves = 4;   // of a workgroup: the same rows, neighbouring channels
constexpr int kTile = 16;   // rows of B and C in LDS
constexpr int kGrp = 4;   // rows loaded together

// FULL: step sizes by softplus, a skip and a gate, as a layer has them; otherwise each as the call says.
template <typename T, int N, bool FULL>
struct ScanLane {
    static constexpr int NQ = N <= 4 ? 4 : N <= 8 ? 8 : 16;   // places of B, then of C, in a row of LDS
    static constexpr int NV = (N + 3) / 4;
    static constexpr int kLds = kTile * 2 * NQ;               // floats of LDS a wave
    static constexpr int kStage = kTile * NQ / 64;            // loads of a lane for a tile of B, and of C
    const T *delta, *x, *z, *B, *C;
    T* y;
    int64_t sdelta, sx, sz, sy, sB, sC;
    uint32_t bd, bx, bz, by;  // bytes from one row to the next
    uint32_t row_bytes, db;   // of a row's channels; byte offset of the lane's
    int rows, r0, span;
    uint32_t ob, oc;          // byte offset of the lane's element of B and of C in a tile
    float *put, *putc, *lds, *lds_b;
    float a[N], bias, skip, dsum;
    f4 h[NV];                 // the channel's states; those past N stay what they are and go nowhere
    int softplus;
    bool skips, gates;

    // lane of channel d, in the range of rows [r0_, r1_)
    __device__ __forceinline__ ScanLane(const TokScanParams& p, int d, int r0_, int r1_, float* lds_) {
        r0 = r0_;
        span = r1_ - r0_;
        delta = (const T*)p.delta; x = (const T*)p.x; y = (T*)p.y; B = (const T*)p.Bm; C = (const T*)p.C;
        gates = p.z != nullptr;
        z = gates ? (const T*)p.z : x;   // without a gate: read and not used
        rows = p.q.T;
        db = (uint32_t)d * sizeof(T);
        sdelta = p.sdelta; sx = p.sx; sz = gates ? p.sz : p.sx; sy = p.sy; sB = p.sB; sC = p.sC;
        bd = (uint32_t)sdelta * sizeof(T); bx = (uint32_t)sx * sizeof(T);
        row_bytes = (uint32_t)p.D * sizeof(T);
        bz = (uint32_t)sz * sizeof(T); by = max((uint32_t)sy * (uint32_t)sizeof(T), row_bytes);
        const int lane = lane_id(), n = lane % NQ, r = lane / NQ;
        ob = n < N ? (uint32_t)(r * (int)sB + n) * sizeof(T) : 0x7fffffffu;   // places past the states: 0, or any element of rows far apart (they meet nothing)
        oc = n < N ? (uint32_t)(r * (int)sC + n) * sizeof(T) : 0x7fffffffu;
        lds = lds_;
        put = lds_ + r * 2 * NQ + (n % 4) * (NQ / 4) + n / 4;
        putc = lds_ + r * 2 * NQ + NQ + n;
        lds_b = lds_ + (lane % 4) * (NQ / 4);
#pragma unroll
        for (int n = 0; n < N; ++n) a[n] = p.A[(int64_t)d * N + n] * kLog2e;
        bias = p.stepf.bias ? p.stepf.bias[d] : 0.0f;
        skip = p.skip ? p.skip[d] : 0.0f;
        skips = p.skip != nullptr;
        softplus = p.stepf.softplus;
    }
    __device__ __forceinline__ void set(const float (&v)[N]) {
#pragma unroll
        for (int n = 0; n < 4 * NV; ++n) h[n / 4][n % 4] = n < N ? v[n] : 0.0f;
    }
    __device__ __forceinline__ void get(float (&v)[N]) const {
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] = h[n / 4][n % 4];
    }
    template <bool OUT>
    __device__ __forceinline__ void row(int i, buffer_t yg, uint32_t yo, float dl, float xv, float zv) {
        // Four states of the wave's 64 channels a matrix instruction: sixteen blocks of 4 x 4, h += b u with b the
        // rows (lane l: state l % 4 of the four) and u the columns (lane l: its channel), four states a lane.
        float b[NQ / 4];
        __builtin_memcpy(b, __builtin_assume_aligned(lds_b + i * 2 * NQ, NQ >= 16 ? 16 : NQ), sizeof(b));
        const f4* c = reinterpret_cast<const f4*>(lds + i * 2 * NQ + NQ);
        const float u = dl * xv;
        float o = 0.0f;
        if (!OUT) dsum += dl;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (4 * q + e < N) h[q][e] *= __builtin_amdgcn_exp2f(a[4 * q + e] * dl);
            h[q] = __builtin_amdgcn_mfma_f32_4x4x1f32(b[q], u, h[q], 0, 0, 0);
        }
        if (OUT) {
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const f4 w = c[q];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (4 * q + e < N) o = fmaf(h[q][e], w[e], o);
            }
        }
        if (OUT) {
            if (FULL || skips) o = fmaf(skip, xv, o);
            if (FULL || gates) o *= zv * sigmoid_f(zv);
            buffer_store(yg, yo, to_stream<T>(o));
        }
    }
    // A SIMD issues from its oldest wave first, so of four waves with the same work one would be done when another has
    // half of it left, alone and too few to fill the SIMD.  A wave behind the others goes first (8192 x 2048: 54 + 70 us
    // without, 50 + 65 us with it).
    __device__ __forceinline__ void yield(int t) const {
        const int64_t done = 4 * (int64_t)(t - r0);
        if (done < span) __builtin_amdgcn_s_setprio(3);
        else if (done < 2 * (int64_t)span) __builtin_amdgcn_s_setprio(2);
        else if (done < 3 * (int64_t)span) __builtin_amdgcn_s_setprio(1);
        else __builtin_amdgcn_s_setprio(0);
    }
    // rows [t0, t1), t0 < t1: the next group's streams and the next tile's B and C are under way
    // while a group is computed
    template <bool OUT>
    __device__ __forceinline__ void walk(int t0, int t1) {
        T rd[kGrp], rx[kGrp], rz[kGrp], rb[kStage], rc[kStage];
        const T *pd = delta + t0 * sdelta, *px = x + t0 * sx, *pz = z + t0 * sz;
        T* py = y + t0 * sy;
        int tl = t0;   // the row of pd, px, pz
        auto load = [&] {   // rows tl .. tl+3 (past the last row of all, the last one again)
            const buffer_t d_ = buffer_of(pd, kAll), x_ = buffer_of(px, kAll), z_ = buffer_of(pz, kAll);
#pragma unroll
            for (int g = 0; g < kGrp; ++g) {
                const uint32_t r = max(min(g, rows - 1 - tl), 0);
                rd[g] = buffer_load<T>(d_, db, r * bd);
                rx[g] = buffer_load<T>(x_, db, r * bx);
                if (OUT) rz[g] = buffer_load<T>(z_, db, r * bz);
            }
            const int64_t on = tl + kGrp < rows ? kGrp : 0;
            tl += (int)on;
            pd += on * sdelta; px += on * sx; pz += on * sz;
        };
        auto load_bc = [&](int t) {   // rows from t1 on are past the buffers' ends
            const int64_t left = t1 - 1 - t;
            const uint32_t eb = (uint32_t)(min(left, (int64_t)kTile - 1) * sB + N) * sizeof(T);
            const uint32_t ec = (uint32_t)(min(left, (int64_t)kTile - 1) * sC + N) * sizeof(T);
            const buffer_t bb = buffer_of(B + t * sB, eb), cb = buffer_of(C + t * sC, ec);
#pragma unroll
            for (int q = 0; q < kStage; ++q) {
                rb[q] = buffer_load<T>(bb, ob + (uint32_t)(q * (64 / NQ) * (int)sB) * sizeof(T));
                if (OUT) rc[q] = buffer_load<T>(cb, oc + (uint32_t)(q * (64 / NQ) * (int)sC) * sizeof(T));
            }
        };
        auto stage = [&] {   // a wave's own tile: its LDS accesses complete in order, nothing to wait for
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int q = 0; q < kStage; ++q) {
                put[q * (64 / NQ) * 2 * NQ] = to_f32(rb[q]);
                if (OUT) putc[q * (64 / NQ) * 2 * NQ] = to_f32(rc[q]);
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            __builtin_amdgcn_wave_barrier();
        };
        // Waits are for the loads of a group or tile before, with the next one's under way: for that the compiler has
        // to see the same loads on every way through the loops, and none pending from before them (57 + 75 us where it
        // did not, 53 + 72 us where it did).
        load_bc(t0);
        load();
#pragma unroll
        for (int g = 0; g < kGrp; ++g) {
            __asm__ volatile("" : "+v"(rd[g]), "+v"(rx[g]));
            if (OUT) __asm__ volatile("" : "+v"(rz[g]));
        }
        for (int tt = t0; tt < t1; tt += kTile) {
            yield(tt);
            stage();
            load_bc(min(tt + kTile, t1 - 1));   // (after the last tile: of no use)
            const int n = min(kTile, t1 - tt);
            int i = 0;
#pragma unroll 1
            do {
                // rows from t1 on are identity steps: step size and input 0, B and C read as 0, y past the
                // end of its buffer
                float dl[kGrp], xv[kGrp], zv[kGrp];
#pragma unroll
                for (int g = 0; g < kGrp; ++g) {
                    dl[g] = to_f32(rd[g]) + bias;
                    xv[g] = to_f32(rx[g]);
                    zv[g] = OUT ? to_f32(rz[g]) : 0.0f;
                }
                load();
#pragma unroll
                for (int g = 0; g < kGrp; ++g) {
                    if (FULL || softplus) dl[g] = softplus_t(dl[g]);
                }
                if (i + kGrp > n) {
#pragma unroll
                    for (int g = 0; g < kGrp; ++g) {
                        dl[g] = i + g < n ? dl[g] : 0.0f;
                        xv[g] = i + g < n ? xv[g] : 0.0f;
                    }
                }
                const buffer_t yg = buffer_of(py, (uint32_t)(min(kGrp, n - i) - 1) * by + row_bytes);
#pragma unroll
                for (int g = 0; g < kGrp; ++g) row<OUT>(i + g, yg, db + g * by, dl[g], xv[g], zv[g]);
                py += kGrp * sy;
                i += kGrp;
            } while (i < n);
        }
    }
};
// a range's states in the workspace, [n][d]
template <int N>
__device__ __forceinline__ void get_range(const float* base, int D, int d, float (&h)[N]) {
    const buffer_t b = buffer_of(base, kAll);
#pragma unroll
    for (int n = 0; n < N; ++n) h[n] = buffer_load<float>(b, (uint32_t)d * 4, (uint32_t)(n * D) * 4);
}
template <int N>
__device__ __forceinline__ void put_range(float* base, int D, int d, const float (&h)[N]) {
    const buffer_t b = buffer_of(base, kAll);
#pragma unroll
    for (int n = 0; n < N; ++n) buffer_store(b, (uint32_t)d * 4 + (uint32_t)(n * D) * 4, h[n]);
}
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

// First pass, ranges 0 .. nrange-2.  The states are kept apart from the second pass's by the sum of step sizes, not
// by a product of transitions: exp(A sum) costs one exp2 a state and range.
template <typename T, int N, bool FULL>
__global__ __launch_bounds__(64 * kScanWaves, 16 / kScanWaves) void tok_scan_sum_kernel(TokScanParams p, int gblocks) {
    const int cb = uniform((blockIdx.x % gblocks) * (blockDim.x >> 6) + (threadIdx.x >> 6));
    const int c = blockIdx.x / gblocks;
    if (cb * 64 >= p.D) return;
    const Range_ r = rows_of(p, c);
    const SeqTable q(p.q);
    const int s = q.find(r.r1 - 1);
    int st = 0, en = 0, slot = -1;
    if (s >= 0 && s < p.q.S) {
        st = q.first(s);
        en = q.end(s);
        if (st >= 0 && st < r.r1 && en > r.r1) slot = q.slot(s);   // st beyond: the list does not ascend
    }
    if (cb == 0 && lane_id() == 0) p.through[c] = slot >= 0 && st < r.r0;
    if (slot < 0) return;   // none crosses the end
    // lanes past the last channel repeat it: the same values to the same places, without a branch a row
    const int d = min(cb * 64 + lane_id(), p.D - 1);
    __shared__ __align__(16) float lds[kScanWaves * ScanLane<T, N, FULL>::kLds];
    ScanLane<T, N, FULL> l(p, d, r.r0, r.r1, lds + (threadIdx.x >> 6) * ScanLane<T, N, FULL>::kLds);
    const int64_t at = (int64_t)c * N * p.D;
    float h[N] = {};
    l.dsum = 0.0f;
    if (st >= r.r0) {   // it begins here: its first state, kept for the second pass (which may find it overwritten)
        if (!q.fresh(s)) load_states<N>(p.pool + slot * p.spool + (int64_t)d * N, h);
        put_range<N>(p.h0 + at, p.D, d, h);
    }
    l.set(h);
    l.template walk<false>(max(st, r.r0), r.r1);
    l.get(h);
    put_range<N>(p.hsum + at, p.D, d, h);
    p.dsum[(int64_t)c * p.D + d] = l.dsum;
}

// Between the passes: the states at the ranges' ends, from those that each range leaves alone,
//   h <- exp(A dsum) h + S where the sequence runs through the whole range, S where it begins there.
// A workgroup takes 64 channels of one state; its 16 waves take the ranges in runs of PER, compose
// each, then each composes the runs before its own and goes over its ranges again.  PER ranges stay in
// registers in between, so the states are read once and written once, which bounds it (127 ranges of
// 2048 x 16 states, 33 MB: 9.8 us); more than 16 * PER ranges are taken in turns of that many, with the state
// carried over.
constexpr int kRuns = 16;
template <int PER>
__global__ __launch_bounds__(64 * kRuns) void tok_scan_join_kernel(TokScanParams p) {
    __shared__ float end_[kRuns][64], decay_[kRuns][64];
    const int n = blockIdx.x % p.N, lane = lane_id(), w = uniform(threadIdx.x >> 6);
    const int d = min((int)(blockIdx.x / p.N) * 64 + lane, p.D - 1);
    const float a = p.A[(int64_t)d * p.N + n] * kLog2e;
    const int ends = p.nrange - 1;
    float* const S = p.hsum + (int64_t)n * p.D + d;
    const int64_t step = (int64_t)p.N * p.D;
    float carry = 0.0f;
    for (int base = 0; base < ends; base += kRuns * PER) {
        const int k0 = base + w * PER;
        float s[PER], e[PER];
        int f[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int j = min(k0 + i, ends - 1);
            s[i] = S[j * step];
            e[i] = p.dsum[(int64_t)j * p.D + d];
            f[i] = p.through[j];
        }
        // the run as a map: through a run with a beginning in it nothing comes (decay -1)
        float h = 0.0f, decay = 1.0f;
        bool all = true;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const bool has = k0 + i < ends;
            e[i] = __builtin_amdgcn_exp2f(a * e[i]);
            const float g = f[i] ? fmaf(e[i], h, s[i]) : s[i];
            h = has ? g : h;
            decay *= has ? e[i] : 1.0f;
            all = all && (f[i] || !has);
        }
        end_[w][lane] = h;
        decay_[w][lane] = all ? decay : -1.0f;
        __syncthreads();
        float in = carry;
        for (int i = 0; i < w; ++i) {
            const float q = decay_[i][lane];
            in = q < 0.0f ? end_[i][lane] : fmaf(q, in, end_[i][lane]);
        }
        h = in;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            h = f[i] ? fmaf(e[i], h, s[i]) : s[i];
            if (k0 + i < ends) S[(int64_t)(k0 + i) * step] = h;
        }
        for (int i = w; i < kRuns; ++i) {   // on to what the next turn begins with
            const float q = decay_[i][lane];
            in = q < 0.0f ? end_[i][lane] : fmaf(q, in, end_[i][lane]);
        }
        carry = in;
        __syncthreads();
    }
}

// Second pass: every row's output and every sequence's last state.  128 registers, four waves a SIMD.
template <typename T, int N, bool FULL>
__global__ __launch_bounds__(64 * kScanWaves, 16 / kScanWaves) void tok_scan_kernel(TokScanParams p, int gblocks) {
    const int cb = uniform((blockIdx.x % gblocks) * (blockDim.x >> 6) + (threadIdx.x >> 6));
    const int c = blockIdx.x / gblocks;
    if (cb * 64 >= p.D) return;
    const Range_ r = rows_of(p, c);
    const SeqTable q(p.q);
    int s = q.find(r.r0);
    if (s >= p.q.S) return;
    const int d = min(cb * 64 + lane_id(), p.D - 1);
    __shared__ __align__(16) float lds[kScanWaves * ScanLane<T, N, FULL>::kLds];
    ScanLane<T, N, FULL> l(p, d, r.r0, r.r1, lds + (threadIdx.x >> 6) * ScanLane<T, N, FULL>::kLds);
    if (s < 0) s = 0;
    for (; s < p.q.S; ++s) {
        const int st = q.first(s);
        if (st >= r.r1) break;
        const int en = q.end(s);
        if (st < 0 || en <= max(st, r.r0)) continue;
        const int slot = q.slot(s);
        if (slot < 0) continue;
        float* pool = p.pool + slot * p.spool + (int64_t)d * N;
        float h[N] = {};
        if (st < r.r0) {   // from the ranges before: the state that crosses into this one
            get_range<N>(p.hsum + (int64_t)(p.joined ? c - 1 : st / p.rows) * N * p.D, p.D, d, h);
            if (!p.joined) {
#pragma unroll 1
                for (int k = st / p.rows + 1; k < c; ++k) {
                    float S[N];
                    get_range<N>(p.hsum + (int64_t)k * N * p.D, p.D, d, S);
                    const float ds = p.dsum[(int64_t)k * p.D + d];
#pragma unroll
                    for (int n = 0; n < N; ++n) h[n] = fmaf(__builtin_amdgcn_exp2f(l.a[n] * ds), h[n], S[n]);
                }
            }
        } else if (en > r.r1) {
            get_range<N>(p.h0 + (int64_t)c * N * p.D, p.D, d, h);
        } else if (!q.fresh(s)) {
            load_states<N>(pool, h);
        }
        l.set(h);
        l.template walk<true>(max(st, r.r0), min(en, r.r1));
        if (en <= r.r1) {
            l.get(h);
#pragma unroll
            for (int n = 0; n < N; ++n) pool[n] = h[n];
        }
    }
}

// One row a sequence.  Q lanes share a channel, four states each (the last lane's may be fewer), and Q channels
// (units): the loads of all their states are under way together, and what a channel has once (step size, input,
// gate) lane q of the group reads and forms for unit q; the others take it by a lane move, and the units' sums
// over the states come back to it by a transpose.  VEC: the states of a lane are one 16-byte access.  Measured at
// 256 x 4096 x 16: one channel a lane group 41 us, four 31, what a channel has once formed by one lane 27.
template <int Q, int U>
__device__ __forceinline__ float of_unit(float v) {   // lane U of the group's value
    if (Q == 4) return dpp<SSM_DPP_QUAD(U, U, U, U)>(0.0f, v);
    if (Q == 2) return dpp<SSM_DPP_QUAD(U, U, 2 + U, 2 + U)>(0.0f, v);
    return v;
}
template <typename T, int Q, bool VEC>
__global__ __launch_bounds__(256) void tok_step_kernel(TokScanParams p, int cblocks) {
    constexpr int G = 256 / Q;   // groups of a workgroup; unit u's channel is c0 + u * G
    const int s = blockIdx.x / cblocks, q = threadIdx.x % Q;
    const int c0 = (blockIdx.x % cblocks) * 256 + (int)threadIdx.x / Q;
    const int n0 = 4 * q, N = p.N;
    const bool four = n0 + 4 <= N;   // VEC: all of a lane's states or (N = 12) none
    // the state is loaded from the slot that is named; whether the sequence has it comes in meanwhile
    const int slot = uniform(slot_named(p.q, s));
    if (slot < 0) return;
    const int64_t t = s;
    const bool fresh = p.q.fresh && p.q.fresh[s];
    float* const pool = p.pool + slot * p.spool + n0;
    const T* B = (const T*)p.Bm + t * p.sB + n0;
    const T* C = (const T*)p.C + t * p.sC + n0;
    // a lane's places in a channel's states and A, from the workgroup's first channel: 32 bits
    const int last = p.D - 1 - (int)(blockIdx.x % cblocks) * 256;
    float* const hb = pool + (int64_t)(p.D - 1 - last) * N;
    const float* const Ab = p.A + (int64_t)(p.D - 1 - last) * N + n0;
    float h[Q][4], a[Q][4], b[4], c[4];
#pragma unroll
    for (int u = 0; u < Q; ++u) {
        const int at = min((int)threadIdx.x / Q + u * G, last) * N;
        const float *A = Ab + at, *hp = hb + at;
#pragma unroll
        for (int e = 0; e < 4; ++e) h[u][e] = a[u][e] = 0.0f;
        if (VEC && four) {
            if (!fresh) {
                const float4 hv = *reinterpret_cast<const float4*>(hp);
                h[u][0] = hv.x; h[u][1] = hv.y; h[u][2] = hv.z; h[u][3] = hv.w;
            }
            const float4 av = *reinterpret_cast<const float4*>(A);
            a[u][0] = av.x; a[u][1] = av.y; a[u][2] = av.z; a[u][3] = av.w;
        } else if (!VEC) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (n0 + e < N) {
                    a[u][e] = A[e];
                    if (!fresh) h[u][e] = hp[e];
                }
            }
        }
    }
    const int dq = min(c0 + q * G, p.D - 1);   // the lane's own unit
    float step = to_f32(((const T*)p.delta)[t * p.sdelta + dq]);
    const float x = to_f32(((const T*)p.x)[t * p.sx + dq]);
    const float bias = p.stepf.bias ? p.stepf.bias[dq] : 0.0f, skip = p.skip ? p.skip[dq] : 0.0f;
    const float z = p.z ? to_f32(((const T*)p.z)[t * p.sz + dq]) : 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const bool has = VEC ? four : n0 + e < N;
        b[e] = has ? to_f32(B[e]) : 0.0f;
        c[e] = has ? to_f32(C[e]) : 0.0f;
    }
    if (slot_taken(p.q, s, slot)) return;
    step += bias;
    if (p.stepf.softplus) step = softplus_t(step);
    const float in = step * x, step2 = step * kLog2e;
    float y[Q];
    auto unit = [&](int u, float dl, float v) {
        y[u] = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {   // of a place past the states: not used, as v may be infinite
            h[u][e] = fmaf(__builtin_amdgcn_exp2f(a[u][e] * dl), h[u][e], v * b[e]);
            if (VEC) y[u] = fmaf(h[u][e], c[e], y[u]);
            else y[u] = n0 + e < N ? fmaf(h[u][e], c[e], y[u]) : y[u];
        }
        if (VEC && Q == 4) y[u] = four ? y[u] : 0.0f;
        if ((int)threadIdx.x / Q + u * G > last) return;
        float* hp = hb + ((int)threadIdx.x / Q + u * G) * N;
        if (VEC) {
            if (four) *reinterpret_cast<float4*>(hp) = make_float4(h[u][0], h[u][1], h[u][2], h[u][3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n0 + e < N) hp[e] = h[u][e];
        }
    };
    unit(0, of_unit<Q, 0>(step2), of_unit<Q, 0>(in));
    if (Q > 1) unit(1 % Q, of_unit<Q, 1 % Q>(step2), of_unit<Q, 1 % Q>(in));
    if (Q > 2) {
        unit(2 % Q, of_unit<Q, 2 % Q>(step2), of_unit<Q, 2 % Q>(in));
        unit(3 % Q, of_unit<Q, 3 % Q>(step2), of_unit<Q, 3 % Q>(in));
    }
    float o = y[0];   // lane q: unit q's sum over the group's lanes
    if (Q > 1) o = pair_level<SSM_DPP_QUAD(1, 0, 3, 2)>(y[0], y[1 % Q], (q & 1) != 0);
    if (Q > 2) {
        const float r = pair_level<SSM_DPP_QUAD(1, 0, 3, 2)>(y[2 % Q], y[3 % Q], (q & 1) != 0);
        o = pair_level<SSM_DPP_QUAD(2, 3, 0, 1)>(o, r, (q & 2) != 0);
    }
    if (c0 + q * G >= p.D) return;
    if (p.skip) o = fmaf(skip, x, o);
    if (p.z) o *= z * sigmoid_f(z);
    ((T*)p.y)[t * p.sy + dq] = to_stream<T>(o);
}

template <typename T, int Q>
hipError_t tok_step_q(const TokScanParams& p, hipStream_t st) {
    const int64_t cblocks = ((int64_t)p.D + 255) / 256, blocks = cblocks * p.q.S;
    if (blocks >= (1LL << 31)) return hipErrorInvalidValue;
    // VEC: N a multiple of 4, so a lane has four states or none
    if (p.vec) tok_step_kernel<T, Q, true><<<(unsigned)blocks, 256, 0, st>>>(p, (int)cblocks);
    else tok_step_kernel<T, Q, false><<<(unsigned)blocks, 256, 0, st>>>(p, (int)cblocks);
    return hipGetLastError();
}
template <typename T>
hipError_t tok_step(const TokScanParams& p, hipStream_t st) {
    return p.N <= 4 ? tok_step_q<T, 1>(p, st) : p.N <= 8 ? tok_step_q<T, 2>(p, st) : tok_step_q<T, 4>(p, st);
}

template <typename T, int N>
hipError_t tok_scan_n(const TokScanParams& p, bool sum, hipStream_t st) {
    const int64_t cblocks = ((int64_t)p.D + 63) / 64;
    const int64_t gblocks = (cblocks + kScanWaves - 1) / kScanWaves;   // workgroups along the channels
    const int waves = (int)((cblocks + gblocks - 1) / gblocks);
    const int64_t blocks = gblocks * (sum ? p.nrange - 1 : p.nrange);
    if (blocks >= (1LL << 31)) return hipErrorInvalidValue;
    const unsigned g = (unsigned)blocks, t = 64 * waves;
    const int gb = (int)gblocks;
    if (sum && p.stepf.softplus) tok_scan_sum_kernel<T, N, true><<<g, t, 0, st>>>(p, gb);
    else if (sum) tok_scan_sum_kernel<T, N, false><<<g, t, 0, st>>>(p, gb);
    else if (p.skip && p.z && p.stepf.softplus) tok_scan_kernel<T, N, true><<<g, t, 0, st>>>(p, gb);
    else tok_scan_kernel<T, N, false><<<g, t, 0, st>>>(p, gb);
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
hipError_t launch_tok_join(const TokScanParams& p, hipStream_t st) {
    const int64_t blocks = ((int64_t)p.D + 63) / 64 * p.N;
    if (p.nrange - 1 <= 8 * kRuns) tok_scan_join_kernel<8><<<(unsigned)blocks, 64 * kRuns, 0, st>>>(p);
    else tok_scan_join_kernel<16><<<(unsigned)blocks, 64 * kRuns, 0, st>>>(p);
    return hipGetLastError();
}
hipError_t launch_tok_scan(const TokScanParams& p, int dtype, bool sum, hipStream_t st) {
    return dtype == 1 ? tok_scan_t<bf16_t>(p, sum, st) : tok_scan_t<float>(p, sum, st);
}

}  // namespace ssm
