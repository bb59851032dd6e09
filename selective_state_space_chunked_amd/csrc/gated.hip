// The gated linear recurrence over streams (B, D, L), forward and backward (gated.hpp has the step):
//
//   mu_t = gy_t + a_{t+1} mu_{t+1}  (the last one + gh_last),
//   E_t = mu_t (q_t / beta_t a_t^2 iota_t x_t - q_t a_t h_{t-1})      (q times the derivative by q),
//   gr = E (1 - rho),  glam = sigmoid(lam) / softplus(lam) sum E,
//   gx = mu beta iota,  gi = mu beta x iota (1 - iota),  gh0 = a_0 mu_0.
// The derivative of beta alone, a^2 / beta, has a pole where a gate closes; with q in front it goes to 0.
//
// A lane holds eight consecutive steps of a row (b, d): their maps h -> a h + b are composed in the lane, the lanes
// of 16 by a DPP scan, and beyond 16 through scalars (a wave) and LDS (a workgroup), so the streams are read once,
// in whole lines along the steps, and the state moves on from tile to tile.  The 16, 64, 256 or 1024 lanes of a row
// are chosen so that the rows fill the GPU (gated_lanes in api_gated.inc).  The forward leaves the state that every 16
// lanes enter with, once in 128 steps; from it the backward forms the states again while it walks the tiles from the
// last to the first, so it reads four streams and writes three and no state of the forward is rounded to the stream's
// type.
//
// Bound by HBM, with the vector unit issuing for 59 (forward) and 72 % (backward) of the time: an element is 35 and 67
// instructions.  B=8 D=2048 L=4096 bf16: forward 121 us (544 MB, 4.5 TB/s), backward 189 us (959 MB, 5.1 TB/s; 4 GiB are
// copied at 4.75); B=1 D=1024 L=128000 fp32: 433 and 734 us (2.1 and 3.7 GB, 4.8 and 5.0 TB/s).  A row of 517 steps a
// workgroup (B=2 D=195 fp32): 4.9 and 7.0 us, latency.
#include <algorithm>

#include "gated.hpp"

namespace ssm {
namespace {

constexpr int kRun = 8;   // steps of a lane

typedef uint32_t run_u4 __attribute__((ext_vector_type(4), aligned(2)));
typedef float run_f4 __attribute__((ext_vector_type(4), aligned(4)));

// Eight steps at any element's address.
template <typename T> struct Run;
template <> struct Run<bf16_t> {
    run_u4 r;
    __device__ __forceinline__ void load(const bf16_t* p) { r = *reinterpret_cast<const run_u4*>(p); }
    __device__ __forceinline__ void load_last(const bf16_t* p, int n) {   // the last n of the eight, the others 0
        r = run_u4(0);
#pragma unroll
        for (int j = 0; j < kRun; ++j)
            if (j >= kRun - n) r[j / 2] |= (uint32_t)p[j] << (16 * (j & 1));
    }
    __device__ __forceinline__ void get(float (&v)[kRun]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = __uint_as_float(r[e] << 16);
            v[2 * e + 1] = __uint_as_float(r[e] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ static void store(bf16_t* p, const float (&v)[kRun]) {
        run_u4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] = (uint32_t)to_stream<bf16_t>(v[2 * e]) | ((uint32_t)to_stream<bf16_t>(v[2 * e + 1]) << 16);
        *reinterpret_cast<run_u4*>(p) = o;
    }
};
template <> struct Run<float> {
    run_f4 r[2];
    __device__ __forceinline__ void load(const float* p) {
        r[0] = *reinterpret_cast<const run_f4*>(p);
        r[1] = *reinterpret_cast<const run_f4*>(p + 4);
    }
    __device__ __forceinline__ void load_last(const float* p, int n) {
#pragma unroll
        for (int j = 0; j < kRun; ++j) r[j / 4][j % 4] = j >= kRun - n ? p[j] : 0.0f;
    }
    __device__ __forceinline__ void get(float (&v)[kRun]) const {
#pragma unroll
        for (int j = 0; j < kRun; ++j) v[j] = r[j / 4][j % 4];
    }
    __device__ __forceinline__ static void store(float* p, const float (&v)[kRun]) {
        run_f4 a, b;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            a[e] = v[e];
            b[e] = v[4 + e];
        }
        *reinterpret_cast<run_f4*>(p) = a;
        *reinterpret_cast<run_f4*>(p + 4) = b;
    }
};

// A lane's place in its row.  Its run ends at step min(t + 8, L): where the row ends inside the run or before it, the
// eight steps read are the row's last ones (in bounds, by the same load), of which the run has the last n and the
// others are passed over.
struct Place {
    int at, n;   // first step read (negative in rows of fewer than eight), steps of the run
    __device__ __forceinline__ Place(int t, int L) : at(min(t, L - kRun)), n(max(0, min(kRun, L - t))) {}
};
template <typename T>
__device__ __forceinline__ void load_run_at(Run<T>& r, const T* row, Place pl, bool tiny) {
    if (tiny) r.load_last(row + pl.at, pl.at < 0 ? pl.n : 0);   // rows of fewer than eight steps: one by one
    else r.load(row + pl.at);
}
template <typename T>
__device__ __forceinline__ void store_run_at(T* row, const float (&v)[kRun], Place pl) {
    if (pl.n == kRun) {
        Run<T>::store(row + pl.at, v);
    } else if (pl.n > 0) {
#pragma unroll
        for (int j = 0; j < kRun; ++j)
            if (j >= kRun - pl.n) row[pl.at + j] = to_stream<T>(v[j]);
    }
}

__device__ __forceinline__ float lane_value(float v, int l) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}

// The wait states that a DPP read needs after the last write of a scan, which the compiler does not see.
__device__ __forceinline__ void settle(float& P, float& S) { asm volatile("s_nop 1" : "+v"(P), "+v"(S)); }

// The maps of the waves of a row, from wave to wave through LDS: one barrier a tile, two buffers in turn.
template <int NW> struct WaveMaps {
    float2 m[2][NW];
};

// Up the steps: in, the lanes' maps (P, S); out, the state each lane enters with; carry, the state before the tile,
// becomes the one after it; row_in is the state that the lane's 16 lanes enter with.
template <int LANES, int NW>
__device__ __forceinline__ float enter_up(float P, float S, float& carry, float& row_in, WaveMaps<NW>& lds, int buf) {
    row_scan_affine_up(P, S);
    settle(P, S);
    const float Pe = dpp<SSM_DPP_ROW_SHR(1)>(1.0f, P), Se = dpp<SSM_DPP_ROW_SHR(1)>(0.0f, S);
    if (LANES == 16) {
        row_in = carry;
        carry = fmaf(row_bcast<15>(P), carry, row_bcast<15>(S));
    } else {
        const float P0 = lane_value(P, 15), P1 = lane_value(P, 31), P2 = lane_value(P, 47), P3 = lane_value(P, 63);
        const float S0 = lane_value(S, 15), S1 = lane_value(S, 31), S2 = lane_value(S, 47), S3 = lane_value(S, 63);
        float c0 = carry;
        if (NW > 1) {
            const int w = uniform(threadIdx.x >> 6);
            if (lane_id() == 0) lds.m[buf][w] = make_float2(P0 * P1 * P2 * P3, fmaf(P3, fmaf(P2, fmaf(P1, S0, S1), S2), S3));
            __syncthreads();
            float c = carry;
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                if (i == w) c0 = c;
                const float2 m = lds.m[buf][i];
                c = fmaf(m.x, c, m.y);
            }
            carry = c;
        }
        const float c1 = fmaf(P0, c0, S0), c2 = fmaf(P1, c1, S1), c3 = fmaf(P2, c2, S2);
        const int k = lane_id() >> 4;
        row_in = k == 0 ? c0 : k == 1 ? c1 : k == 2 ? c2 : c3;
        if (NW == 1) carry = fmaf(P3, c3, S3);
    }
    return fmaf(Pe, row_in, Se);
}
// Down the steps: the same from the last lane to the first.
template <int LANES, int NW>
__device__ __forceinline__ float enter_down(float P, float S, float& carry, WaveMaps<NW>& lds, int buf) {
    // (P, S) scanned inclusively already
    const float Pe = dpp<SSM_DPP_ROW_SHL(1)>(1.0f, P), Se = dpp<SSM_DPP_ROW_SHL(1)>(0.0f, S);
    float row_in;
    if (LANES == 16) {
        row_in = carry;
        carry = fmaf(row_bcast<0>(P), carry, row_bcast<0>(S));
    } else {
        const float P0 = lane_value(P, 0), P1 = lane_value(P, 16), P2 = lane_value(P, 32), P3 = lane_value(P, 48);
        const float S0 = lane_value(S, 0), S1 = lane_value(S, 16), S2 = lane_value(S, 32), S3 = lane_value(S, 48);
        float c3 = carry;
        if (NW > 1) {
            const int w = uniform(threadIdx.x >> 6);
            if (lane_id() == 0) lds.m[buf][w] = make_float2(P0 * P1 * P2 * P3, fmaf(P0, fmaf(P1, fmaf(P2, S3, S2), S1), S0));
            __syncthreads();
            float c = carry;
#pragma unroll
            for (int i = NW - 1; i >= 0; --i) {
                if (i == w) c3 = c;
                const float2 m = lds.m[buf][i];
                c = fmaf(m.x, c, m.y);
            }
            carry = c;
        }
        const float c2 = fmaf(P3, c3, S3), c1 = fmaf(P2, c2, S2), c0 = fmaf(P1, c1, S1);
        const int k = lane_id() >> 4;
        row_in = k == 0 ? c0 : k == 1 ? c1 : k == 2 ? c2 : c3;
        if (NW == 1) carry = fmaf(P0, c0, S0);
    }
    return fmaf(Pe, row_in, Se);
}

constexpr int threads_of(int lanes) { return std::max(256, lanes); }

// The row of a lane: rows past the last one repeat it and write nothing.
template <int LANES> struct RowOf {
    int row, b, d, l;
    bool live;
    __device__ __forceinline__ RowOf(int B, int D) {
        constexpr int R = threads_of(LANES) / LANES;
        const int64_t k = (int64_t)blockIdx.x * R + threadIdx.x / LANES;
        live = k < (int64_t)B * D;
        row = live ? (int)k : B * D - 1;
        if (LANES >= 64) row = uniform(row);
        b = row / D;
        d = row % D;
        l = threadIdx.x % LANES;
    }
};

template <typename T, int LANES, bool SLOW, int NW>
__device__ __forceinline__ void gated_fwd(const GatedParams& p, const RowOf<LANES>& at, const GateChannel& c, WaveMaps<NW>& maps) {
    constexpr int TILE = LANES * kRun;
    const T* const x = (const T*)p.x + at.b * p.sx[0] + at.d * p.sx[1];
    const T* const r = (const T*)p.r + at.b * p.sr[0] + at.d * p.sr[1];
    const T* const g = (const T*)p.i + at.b * p.si[0] + at.d * p.si[1];
    T* const y = (T*)p.y + at.b * p.sy[0] + at.d * p.sy[1];
    float* const ck = p.ckpt_out + (int64_t)at.row * p.nchunk;
    const int L = p.L;
    const bool tiny = L < kRun;
    float carry = p.h0 ? p.h0[at.row] : 0.0f;
    Run<T> rx, rr, ri;
    Place pl(at.l * kRun, L);
    load_run_at(rx, x, pl, tiny);
    load_run_at(rr, r, pl, tiny);
    load_run_at(ri, g, pl, tiny);
    int buf = 0;
    for (int t0 = 0; t0 < L; t0 += TILE, buf ^= 1) {
        float xv[kRun], rv[kRun], iv[kRun], a[kRun], b[kRun];
        rx.get(xv);
        rr.get(rv);
        ri.get(iv);
        const Place next(t0 + TILE + at.l * kRun, L);   // past the row's end: its last steps, of no use
        load_run_at(rx, x, next, tiny);
        load_run_at(rr, r, next, tiny);
        load_run_at(ri, g, next, tiny);
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            const float t = c.rate * gate_open(rv[j], c.rb);
            const float v = SLOW ? gate_rest<true>(t, a[j]) : gate_rest<false>(t, a[j]);
            b[j] = __builtin_amdgcn_sqrtf(v) * (gate_open(iv[j], c.ib) * xv[j]);
        }
        if (t0 + TILE > L) {
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                const bool has = j >= kRun - pl.n;
                a[j] = has ? a[j] : 1.0f;
                b[j] = has ? b[j] : 0.0f;
            }
        }
        float P = a[0], S = b[0];
#pragma unroll
        for (int j = 1; j < kRun; ++j) {
            S = fmaf(a[j], S, b[j]);
            P *= a[j];
        }
        float row_in;
        float h = enter_up<LANES, NW>(P, S, carry, row_in, maps, buf);
        if (p.ckpt_out && (at.l & 15) == 0 && pl.n > 0 && at.live) ck[t0 / kGatedChunk + (at.l >> 4)] = row_in;
        if (p.y) {
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                h = fmaf(a[j], h, b[j]);
                xv[j] = h;
            }
            if (at.live) store_run_at(y, xv, pl);
        }
        pl = next;
    }
    if (p.h_last && at.l == 0 && at.live) p.h_last[at.row] = carry;
}

// a channel's sums to its parameters' gradients; sigmoid(lam) / softplus(lam) goes to 1 as lam falls
__device__ __forceinline__ void put_sums(const GatedParams& p, int d, float E, float r, float i) {
    if (p.grb) p.grb[d] = r;
    if (p.gib) p.gib[d] = i;
    if (p.glam) {
        const float lam = p.lam[d], sp = softplus_t(lam);
        p.glam[d] = E * (sp > 0.0f ? sigmoid_f(lam) / sp : 1.0f);
    }
}

template <typename T, int LANES, bool SLOW, int NW>
__device__ __forceinline__ void gated_bwd(const GatedParams& p, const RowOf<LANES>& at, const GateChannel& c, WaveMaps<NW>& maps) {
    constexpr int TILE = LANES * kRun;
    const T* const x = (const T*)p.x + at.b * p.sx[0] + at.d * p.sx[1];
    const T* const r = (const T*)p.r + at.b * p.sr[0] + at.d * p.sr[1];
    const T* const g = (const T*)p.i + at.b * p.si[0] + at.d * p.si[1];
    const T* const gy = (const T*)p.gy + at.b * p.sgy[0] + at.d * p.sgy[1];
    T* const gx = (T*)p.gx + at.b * p.sgx[0] + at.d * p.sgx[1];
    T* const gr = (T*)p.gr + at.b * p.sgr[0] + at.d * p.sgr[1];
    T* const gi = (T*)p.gi + at.b * p.sgi[0] + at.d * p.sgi[1];
    const float* const ck = p.ckpt + (int64_t)at.row * p.nchunk;
    const float rate = c.rate * kLn2;
    const int L = p.L;
    const bool tiny = L < kRun;
    float carry = p.gh_last ? p.gh_last[at.row] : 0.0f;   // a mu of the step after the tile's last
    float sumE = 0.0f, sumr = 0.0f, sumi = 0.0f;
    const int last = (L - 1) / TILE * TILE;
    Run<T> rx, rr, ri, rg;
    Place pl(last + at.l * kRun, L);
    load_run_at(rx, x, pl, tiny);
    load_run_at(rr, r, pl, tiny);
    load_run_at(ri, g, pl, tiny);
    load_run_at(rg, gy, pl, tiny);
    float h_row = ck[min(last / kGatedChunk + (at.l >> 4), p.nchunk - 1)];
    int buf = 0;
    for (int t0 = last; t0 >= 0; t0 -= TILE, buf ^= 1) {
        float xv[kRun], rho[kRun], iota[kRun], a[kRun], beta[kRun], rs[kRun], hp[kRun], gv[kRun];
        rx.get(xv);
        rr.get(rho);
        ri.get(iota);
        rg.get(gv);
        const float h_in = h_row;
        const int tn = max(t0 - TILE, 0);   // before the first tile: loaded again, of no use
        const Place next(tn + at.l * kRun, L);
        load_run_at(rx, x, next, tiny);
        load_run_at(rr, r, next, tiny);
        load_run_at(ri, g, next, tiny);
        load_run_at(rg, gy, next, tiny);
        h_row = ck[min(tn / kGatedChunk + (at.l >> 4), p.nchunk - 1)];
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            rho[j] = gate_open(rho[j], c.rb);
            iota[j] = gate_open(iota[j], c.ib);
            const float v = SLOW ? gate_rest<true>(c.rate * rho[j], a[j]) : gate_rest<false>(c.rate * rho[j], a[j]);
            rs[j] = __builtin_amdgcn_rsqf(fmaxf(v, 0x1p-126f));   // 1 / beta, finite where a gate is shut
            beta[j] = v * rs[j];
        }
        if (t0 + TILE > L) {   // a step that is passed over: a = 1 and no terms
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                const bool has = j >= kRun - pl.n;
                a[j] = has ? a[j] : 1.0f;
                beta[j] = has ? beta[j] : 0.0f;
                rho[j] = has ? rho[j] : 0.0f;
                iota[j] = has ? iota[j] : 0.0f;
                xv[j] = has ? xv[j] : 0.0f;
                gv[j] = has ? gv[j] : 0.0f;
            }
        }
        // the lane's maps, up for the states and down for mu: the product of a is the same
        float P = 1.0f, S = 0.0f, R = 0.0f;
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            hp[j] = beta[j] * iota[j] * xv[j];
            S = fmaf(a[j], S, hp[j]);
            P *= a[j];
        }
#pragma unroll
        for (int j = kRun - 1; j >= 0; --j) R = a[j] * (gv[j] + R);
        float Q = P;
        row_scan_affine_updown(P, S, Q, R);
        settle(P, S);
        settle(Q, R);
        const float Pe = dpp<SSM_DPP_ROW_SHR(1)>(1.0f, P), Se = dpp<SSM_DPP_ROW_SHR(1)>(0.0f, S);
        float h = fmaf(Pe, h_in, Se);
        float mu = enter_down<LANES, NW>(Q, R, carry, maps, buf);
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            const float b = hp[j];
            hp[j] = h;
            h = fmaf(a[j], h, b);
        }
        float gs = 0.0f, is = 0.0f, es = 0.0f;
#pragma unroll
        for (int j = kRun - 1; j >= 0; --j) {
            const float m = gv[j] + mu;
            mu = a[j] * m;
            const float u = iota[j] * xv[j], gu = m * beta[j];
            const float q = rate * rho[j];
            // E = m a (q / beta a u - q h); q / beta first, which stays below 1 + q where 1 / beta grows
            const float E = mu * fmaf(a[j] * u, q * rs[j], -q * hp[j]);
            const float er = E * (1.0f - rho[j]), ei = gu * u * (1.0f - iota[j]);
            es += E;
            gs += er;
            is += ei;
            gv[j] = gu * iota[j];
            rho[j] = er;
            iota[j] = ei;
        }
        sumE += es;
        sumr += gs;
        sumi += is;
        if (at.live) {
            if (p.gx) store_run_at(gx, gv, pl);
            if (p.gr) store_run_at(gr, rho, pl);
            if (p.gi) store_run_at(gi, iota, pl);
        }
        pl = next;
    }
    if (p.gh0 && at.l == 0 && at.live) p.gh0[at.row] = carry;
    if (!p.sums) return;
    sumE = row_sum(sumE);
    sumr = row_sum(sumr);
    sumi = row_sum(sumi);
    if (LANES >= 64) {
        sumE = (lane_value(sumE, 0) + lane_value(sumE, 16)) + (lane_value(sumE, 32) + lane_value(sumE, 48));
        sumr = (lane_value(sumr, 0) + lane_value(sumr, 16)) + (lane_value(sumr, 32) + lane_value(sumr, 48));
        sumi = (lane_value(sumi, 0) + lane_value(sumi, 16)) + (lane_value(sumi, 32) + lane_value(sumi, 48));
    }
    if (NW > 1) {
        __shared__ float part[3][NW];
        if (lane_id() == 0) {
            const int w = threadIdx.x >> 6;
            part[0][w] = sumE;
            part[1][w] = sumr;
            part[2][w] = sumi;
        }
        __syncthreads();
        sumE = sumr = sumi = 0.0f;
        for (int w = 0; w < NW; ++w) {
            sumE += part[0][w];
            sumr += part[1][w];
            sumi += part[2][w];
        }
    }
    if (at.l == 0 && at.live && p.B == 1) {   // nothing to add
        put_sums(p, at.d, sumE, sumr, sumi);
    } else if (at.l == 0 && at.live) {
        p.part[at.row] = sumE;
        p.part[(int64_t)p.B * p.D + at.row] = sumr;
        p.part[2 * (int64_t)p.B * p.D + at.row] = sumi;
    }
}

template <typename T, int LANES, bool BWD>
__global__ __launch_bounds__(threads_of(LANES)) void gated_kernel(GatedParams p) {
    constexpr int NW = LANES > 64 ? LANES / 64 : 1;
    __shared__ WaveMaps<NW> maps;
    const RowOf<LANES> at(p.B, p.D);
    if (LANES == 64 && !at.live) return;
    const GateChannel c = gate_channel(p.lam, p.rb, p.ib, p.power, at.d);
    // (a workgroup of several waves has one row, so its waves go the same way)
    const bool slow = __ballot(!(c.rate < kGateSlow)) == 0;
    if (BWD) {
        if (slow) gated_bwd<T, LANES, true, NW>(p, at, c, maps);
        else gated_bwd<T, LANES, false, NW>(p, at, c, maps);
    } else {
        if (slow) gated_fwd<T, LANES, true, NW>(p, at, c, maps);
        else gated_fwd<T, LANES, false, NW>(p, at, c, maps);
    }
}

// Sums of the rows' parts over the batch, in a fixed order: a workgroup has 64 channels, its waves the batch rows in
// turn.
constexpr int kSumWaves = 8;
__global__ __launch_bounds__(64 * kSumWaves) void gated_sum_kernel(GatedParams p) {
    __shared__ float part[kSumWaves][3][64];
    const int lane = lane_id(), w = threadIdx.x >> 6;
    const int d = blockIdx.x * 64 + lane;
    const int64_t n = (int64_t)p.B * p.D;
    float s[3] = {0.0f, 0.0f, 0.0f};
    if (d < p.D)
        for (int b = w; b < p.B; b += kSumWaves)
#pragma unroll
            for (int k = 0; k < 3; ++k) s[k] += p.part[k * n + (int64_t)b * p.D + d];
#pragma unroll
    for (int k = 0; k < 3; ++k) part[w][k][lane] = s[k];
    __syncthreads();
    if (w != 0 || d >= p.D) return;
#pragma unroll
    for (int i = 1; i < kSumWaves; ++i)
#pragma unroll
        for (int k = 0; k < 3; ++k) s[k] += part[i][k][lane];
    put_sums(p, d, s[0], s[1], s[2]);
}

template <typename T, int LANES>
hipError_t launch(const GatedParams& p, bool bwd, hipStream_t st) {
    constexpr int TH = threads_of(LANES);
    const unsigned blocks = (unsigned)(((int64_t)p.B * p.D + TH / LANES - 1) / (TH / LANES));
    if (bwd) gated_kernel<T, LANES, true><<<blocks, TH, 0, st>>>(p);
    else gated_kernel<T, LANES, false><<<blocks, TH, 0, st>>>(p);
    return hipGetLastError();
}
template <typename T>
hipError_t launch_lanes(const GatedParams& p, bool bwd, hipStream_t st) {
    switch (p.lanes) {
        case 16: return launch<T, 16>(p, bwd, st);
        case 64: return launch<T, 64>(p, bwd, st);
        case 256: return launch<T, 256>(p, bwd, st);
        default: return launch<T, 1024>(p, bwd, st);
    }
}

}  // namespace

hipError_t launch_gated(const GatedParams& p, bool bwd, int dtype, hipStream_t st) {
    return dtype ? launch_lanes<bf16_t>(p, bwd, st) : launch_lanes<float>(p, bwd, st);
}
hipError_t launch_gated_sum(const GatedParams& p, hipStream_t st) {
    gated_sum_kernel<<<(unsigned)((p.D + 63) / 64), 64 * kSumWaves, 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace ssm
