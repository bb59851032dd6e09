// The gated linear recurrence (gated.hpp) over packed rows, with a pool of states.
//
// Prompts.  A lane holds four channels, so a wave walks 256 channels down a range of rows and reads the streams
// along the channels, as the projections write them.  Few long sequences do not fill the GPU, so the rows are cut
// into ranges whatever the sequences' lengths: a first pass leaves, for the sequence that crosses the end of each
// range, its state there (from zero where it runs through the whole range) and the sum of its q; the states between
// ranges are composed, h <- e^(-sum q) h + S, and the second pass walks every range from the state that enters it.
// Single tokens: a row a sequence, four channels a lane.
#include <algorithm>

#include "gated.hpp"

namespace ssm {
namespace {

constexpr int kGrp = 4;   // rows loaded together
constexpr int kCh = 4;    // channels of a lane

// A lane's channels.  EVEN: all four are channels of the layer, or (past the last one, where D is a multiple of four)
// the last four again, whose results go nowhere; otherwise the first n, one by one.
template <typename T, bool EVEN>
struct GatedLane {
    const T *x, *r, *i;
    T* y;
    int64_t sx, sr, si, sy;
    int n;
    bool live;
    GateChannel c[kCh];
    float h[kCh], qsum[kCh];
    Vec<T> vx[kGrp], vr[kGrp], vi[kGrp];

    __device__ __forceinline__ GatedLane(const TokGatedParams& p, int d0) {
        live = d0 < p.D;
        n = max(0, min(kCh, p.D - d0));
        const int d = EVEN ? min(d0, p.D - kCh) : min(d0, p.D - 1);
        x = (const T*)p.x + d; r = (const T*)p.r + d; i = (const T*)p.i + d; y = (T*)p.y + d;
        sx = p.sx; sr = p.sr; si = p.si; sy = p.sy;
#pragma unroll
        for (int e = 0; e < kCh; ++e) {
            c[e] = gate_channel(p.lam, p.rb, p.ib, p.power, EVEN ? d + e : min(d + e, p.D - 1));
            h[e] = qsum[e] = 0.0f;
        }
    }
    __device__ __forceinline__ void get(const float* at) {   // the state, from its first channel's place
        Vec<float> v;
        if (EVEN) v.load(at); else v.load(at, n);
        v.get(h);
    }
    __device__ __forceinline__ void put(float* at, const float (&s)[kCh]) const {
        Vec<float> v;
        v.set(s);
        if (EVEN) {
            if (live) v.store(at);
        } else {
            v.store(at, n);
        }
    }
    __device__ __forceinline__ void load(int g, int t) {
        if (EVEN) {
            vx[g].load(x + t * sx);
            vr[g].load(r + t * sr);
            vi[g].load(i + t * si);
        } else {
            vx[g].load(x + t * sx, n);
            vr[g].load(r + t * sr, n);
            vi[g].load(i + t * si, n);
        }
    }
    template <bool OUT>
    __device__ __forceinline__ void row(const Vec<T>& wx, const Vec<T>& wr, const Vec<T>& wi, int t) {
        float xv[kCh], rv[kCh], iv[kCh];
        wx.get(xv);
        wr.get(rv);
        wi.get(iv);
#pragma unroll
        for (int e = 0; e < kCh; ++e) {
            const float q = c[e].rate * gate_open(rv[e], c[e].rb);
            const float a = gate_decay(q);
            const float b = __builtin_amdgcn_sqrtf(gate_rest(q, a)) * gate_open(iv[e], c[e].ib) * xv[e];
            h[e] = fmaf(a, h[e], b);
            if (!OUT) qsum[e] += q;
        }
        if (OUT) {
            Vec<T> o;
            o.set(h);
            if (EVEN) {
                if (live) o.store(y + t * sy);
            } else {
                o.store(y + t * sy, n);
            }
        }
    }
    // rows [t0, t1), t0 < t1, with the next group's loads under way
    template <bool OUT>
    __device__ __forceinline__ void walk(int t0, int t1) {
#pragma unroll
        for (int g = 0; g < kGrp; ++g) load(g, min(t0 + g, t1 - 1));
        for (int t = t0; t < t1; t += kGrp) {
            Vec<T> wx[kGrp], wr[kGrp], wi[kGrp];
#pragma unroll
            for (int g = 0; g < kGrp; ++g) {
                wx[g] = vx[g];
                wr[g] = vr[g];
                wi[g] = vi[g];
            }
#pragma unroll
            for (int g = 0; g < kGrp; ++g) load(g, min(t + kGrp + g, t1 - 1));
            if (t + kGrp <= t1) {
#pragma unroll
                for (int g = 0; g < kGrp; ++g) row<OUT>(wx[g], wr[g], wi[g], t + g);
            } else {
#pragma unroll
                for (int g = 0; g < kGrp; ++g)
                    if (t + g < t1) row<OUT>(wx[g], wr[g], wi[g], t + g);
            }
        }
    }
};

struct Rows {
    int r0, r1;
};
__device__ __forceinline__ Rows rows_of(const TokGatedParams& p, int c) {
    const int r0 = c * p.rows;
    return {r0, min(r0 + p.rows, p.q.T)};
}

// First pass, ranges 0 .. nrange-2: what the sequence that crosses the range's end does there.
template <typename T, bool EVEN>
__device__ __forceinline__ void sum_range(const TokGatedParams& p, int c, int d0, int s, int st, int slot, bool fresh) {
    const Rows r = rows_of(p, c);
    const int64_t at = (int64_t)c * p.D + d0;
    GatedLane<T, EVEN> l(p, d0);
    if (st >= r.r0) {   // it begins here: its first state, kept for the second pass (which may find it overwritten)
        if (!fresh) l.get(p.pool + slot * p.spool + (EVEN ? min(d0, p.D - kCh) : d0));
        l.put(p.h0 + at, l.h);
    }
    l.template walk<false>(max(st, r.r0), r.r1);
    l.put(p.hsum + at, l.h);
    l.put(p.dsum + at, l.qsum);
}
template <typename T>
__global__ __launch_bounds__(256) void tok_gated_sum_kernel(TokGatedParams p, int cblocks) {
    const int d0 = ((blockIdx.x % cblocks) * 4 + uniform(threadIdx.x >> 6)) * 64 * kCh;
    const int c = blockIdx.x / cblocks;
    if (d0 >= p.D) return;
    const Rows r = rows_of(p, c);
    const SeqTable q(p.q);
    const int s = q.find(r.r1 - 1);
    int st = 0, slot = -1;
    if (s >= 0 && s < p.q.S) {
        st = q.first(s);
        if (st >= 0 && st < r.r1 && q.end(s) > r.r1) slot = q.slot(s);   // st beyond: the list does not ascend
    }
    if (d0 == 0 && lane_id() == 0) p.through[c] = slot >= 0 && st < r.r0;
    if (slot < 0) return;   // none crosses the end
    const bool fresh = q.fresh(s);
    const int d = d0 + lane_id() * kCh;
    if (p.D % kCh == 0 || d0 + 64 * kCh <= p.D) sum_range<T, true>(p, c, d, s, st, slot, fresh);
    else sum_range<T, false>(p, c, d, s, st, slot, fresh);
}

// The states at the ranges' ends from what each range leaves alone, where there are more than kTokChain of them: a
// workgroup takes 64 channels, its 16 waves the ranges in runs of PER; each composes its run, then the runs before its
// own, and goes over its ranges again.
constexpr int kRuns = 16, PER = 16;
__global__ __launch_bounds__(64 * kRuns) void tok_gated_join_kernel(TokGatedParams p) {
    __shared__ float end_[kRuns][64], decay_[kRuns][64];
    const int lane = lane_id(), w = uniform(threadIdx.x >> 6);
    const int d = min((int)blockIdx.x * 64 + lane, p.D - 1);
    const int ends = p.nrange - 1;
    float* const S = p.hsum + d;
    float carry = 0.0f;
    for (int base = 0; base < ends; base += kRuns * PER) {
        const int k0 = base + w * PER;
        float s[PER], e[PER];
        int f[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int j = min(k0 + i, ends - 1);
            s[i] = S[(int64_t)j * p.D];
            e[i] = p.dsum[(int64_t)j * p.D + d];
            f[i] = p.through[j];
        }
        // the run as a map: through a run with a beginning in it nothing comes (decay -1)
        float h = 0.0f, decay = 1.0f;
        bool all = true;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const bool has = k0 + i < ends;
            e[i] = gate_decay(e[i]);
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
            if (k0 + i < ends) S[(int64_t)(k0 + i) * p.D] = h;
        }
        for (int i = w; i < kRuns; ++i) {   // on to what the next turn begins with
            const float q = decay_[i][lane];
            in = q < 0.0f ? end_[i][lane] : fmaf(q, in, end_[i][lane]);
        }
        carry = in;
        __syncthreads();
    }
}

// Second pass: every row's output and every sequence's last state.
template <typename T, bool EVEN>
__device__ __forceinline__ void walk_range(const TokGatedParams& p, const SeqTable& q, int c, int d0, int s) {
    const Rows r = rows_of(p, c);
    GatedLane<T, EVEN> l(p, d0);
    const int dc = EVEN ? min(d0, p.D - kCh) : d0;   // where the lane reads its states
    for (; s < p.q.S; ++s) {
        const int st = q.first(s);
        if (st >= r.r1) break;
        const int en = q.end(s);
        if (st < 0 || en <= max(st, r.r0)) continue;
        const int slot = q.slot(s);
        if (slot < 0) continue;
        float* const pool = p.pool + slot * p.spool;
#pragma unroll
        for (int e = 0; e < kCh; ++e) l.h[e] = 0.0f;
        if (st < r.r0) {   // from the ranges before: the state that crosses into this one
            const int k0 = p.joined ? c - 1 : st / p.rows;
            l.get(p.hsum + (int64_t)k0 * p.D + dc);
#pragma unroll 1
            for (int k = k0 + 1; k < c; ++k) {
                Vec<float> vs, vq;
                if (EVEN) {
                    vs.load(p.hsum + (int64_t)k * p.D + dc);
                    vq.load(p.dsum + (int64_t)k * p.D + dc);
                } else {
                    vs.load(p.hsum + (int64_t)k * p.D + dc, l.n);
                    vq.load(p.dsum + (int64_t)k * p.D + dc, l.n);
                }
                float S[kCh], Q[kCh];
                vs.get(S);
                vq.get(Q);
#pragma unroll
                for (int e = 0; e < kCh; ++e) l.h[e] = fmaf(gate_decay(Q[e]), l.h[e], S[e]);
            }
        } else if (en > r.r1) {
            l.get(p.h0 + (int64_t)c * p.D + dc);
        } else if (!q.fresh(s)) {
            l.get(pool + dc);
        }
        l.template walk<true>(max(st, r.r0), min(en, r.r1));
        if (en <= r.r1) l.put(pool + d0, l.h);
    }
}
template <typename T>
__global__ __launch_bounds__(256) void tok_gated_kernel(TokGatedParams p, int cblocks) {
    const int d0 = ((blockIdx.x % cblocks) * 4 + uniform(threadIdx.x >> 6)) * 64 * kCh;
    const int c = blockIdx.x / cblocks;
    if (d0 >= p.D) return;
    const Rows r = rows_of(p, c);
    const SeqTable q(p.q);
    const int s = q.find(r.r0);
    if (s >= p.q.S) return;
    const int d = d0 + lane_id() * kCh;
    if (p.D % kCh == 0 || d0 + 64 * kCh <= p.D) walk_range<T, true>(p, q, c, d, max(s, 0));
    else walk_range<T, false>(p, q, c, d, max(s, 0));
}

// One row a sequence.
template <typename T, bool EVEN>
__device__ __forceinline__ void step_row(const TokGatedParams& p, int s, int slot, int d0) {
    GatedLane<T, EVEN> l(p, d0);
    float* const pool = p.pool + slot * p.spool;
    l.load(0, s);
    if (!(p.q.fresh && p.q.fresh[s])) l.get(pool + (EVEN ? min(d0, p.D - kCh) : d0));
    if (slot_taken(p.q, s, slot)) return;
    l.template row<true>(l.vx[0], l.vr[0], l.vi[0], s);
    l.put(pool + d0, l.h);
}
template <typename T>
__global__ __launch_bounds__(256) void tok_gated_step_kernel(TokGatedParams p, int cblocks) {
    const int d0 = ((blockIdx.x % cblocks) * 4 + uniform(threadIdx.x >> 6)) * 64 * kCh;
    const int s = blockIdx.x / cblocks;
    if (d0 >= p.D) return;
    const int slot = uniform(slot_named(p.q, s));
    if (slot < 0) return;
    const int d = d0 + lane_id() * kCh;
    if (p.D % kCh == 0 || d0 + 64 * kCh <= p.D) step_row<T, true>(p, s, slot, d);
    else step_row<T, false>(p, s, slot, d);
}

}  // namespace

hipError_t launch_tok_gated(const TokGatedParams& p, int dtype, bool sum, hipStream_t st) {
    const int cblocks = (p.D + 256 * kCh - 1) / (256 * kCh);
    const unsigned blocks = (unsigned)cblocks * (unsigned)(sum ? p.nrange - 1 : p.nrange);
    if (sum) {
        if (dtype) tok_gated_sum_kernel<bf16_t><<<blocks, 256, 0, st>>>(p, cblocks);
        else tok_gated_sum_kernel<float><<<blocks, 256, 0, st>>>(p, cblocks);
    } else {
        if (dtype) tok_gated_kernel<bf16_t><<<blocks, 256, 0, st>>>(p, cblocks);
        else tok_gated_kernel<float><<<blocks, 256, 0, st>>>(p, cblocks);
    }
    return hipGetLastError();
}
hipError_t launch_tok_gated_join(const TokGatedParams& p, hipStream_t st) {
    tok_gated_join_kernel<<<(unsigned)((p.D + 63) / 64), 64 * kRuns, 0, st>>>(p);
    return hipGetLastError();
}
hipError_t launch_tok_gated_step(const TokGatedParams& p, int dtype, hipStream_t st) {
    const int cblocks = (p.D + 256 * kCh - 1) / (256 * kCh);
    const unsigned blocks = (unsigned)cblocks * (unsigned)p.q.S;
    if (dtype) tok_gated_step_kernel<bf16_t><<<blocks, 256, 0, st>>>(p, cblocks);
    else tok_gated_step_kernel<float><<<blocks, 256, 0, st>>>(p, cblocks);
    return hipGetLastError();
}

}  // namespace ssm
