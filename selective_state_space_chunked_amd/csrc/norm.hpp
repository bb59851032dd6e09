// Shared by the group norm's kernels: how the channels of a group lie over lanes, sums over a group.
//
// A team -- a wave, or a workgroup of 256 or 1024 lanes where a group has more channels than a wave holds -- takes
// whole groups of one row: P lanes a group (a power of two, or the whole team), each with R vectors of V channels, P
// vectors apart.  So a row is in registers from its one load to its one store, the statistics come from there in two
// passes (the mean, then the squares around it), and the channels' weights stay in registers while the team goes on
// from row to row.  All teams together sweep the rows, so that what is read at a time lies together (each team its own run
// of rows: 52 and 78 us where these take 48 and 75, forward and backward of 16384 x 2048 in groups of 64, bf16 with a gate).
#pragma once
#include "tokens.hpp"

namespace ssm {

typedef uint32_t norm_u4 __attribute__((ext_vector_type(4), aligned(2)));
typedef float norm_f4 __attribute__((ext_vector_type(4), aligned(4)));

// V consecutive channels at any element's address: 16 bytes, or one element.
template <typename T, int V> struct Chan;
template <> struct Chan<bf16_t, 8> {
    norm_u4 r;
    __device__ __forceinline__ void load(const bf16_t* p) { r = *reinterpret_cast<const norm_u4*>(p); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = __uint_as_float(r[e] << 16);
            v[2 * e + 1] = __uint_as_float(r[e] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ static void store(bf16_t* p, const float (&v)[8]) {
        norm_u4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] = (uint32_t)to_stream<bf16_t>(v[2 * e]) | ((uint32_t)to_stream<bf16_t>(v[2 * e + 1]) << 16);
        *reinterpret_cast<norm_u4*>(p) = o;
    }
};
template <> struct Chan<float, 4> {
    norm_f4 r;
    __device__ __forceinline__ void load(const float* p) { r = *reinterpret_cast<const norm_f4*>(p); }
    __device__ __forceinline__ void get(float (&v)[4]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = r[e];
    }
    __device__ __forceinline__ static void store(float* p, const float (&v)[4]) {
        norm_f4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = v[e];
        *reinterpret_cast<norm_f4*>(p) = o;
    }
};
template <typename T> struct Chan<T, 1> {
    T r;
    __device__ __forceinline__ void load(const T* p) { r = *p; }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = to_f32(r); }
    __device__ __forceinline__ static void store(T* p, const float (&v)[1]) { *p = to_stream<T>(v[0]); }
};

constexpr int kNormWaves = 8;   // teams of a workgroup where a team is a wave
constexpr int norm_threads(int team) { return team == 64 ? 64 * kNormWaves : team; }
constexpr int norm_teams(int team) { return team == 64 ? kNormWaves : 1; }

// Sums of K values over the P lanes of a group, in all of them.
template <int TEAM, int K>
__device__ __forceinline__ void group_sums(float (&v)[K], int P, float (*lds)[16]) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (TEAM > 64 || P > 1) v[k] += dpp<SSM_DPP_QUAD(1, 0, 3, 2)>(0.0f, v[k]);
        if (TEAM > 64 || P > 2) v[k] += dpp<SSM_DPP_QUAD(2, 3, 0, 1)>(0.0f, v[k]);
        if (TEAM > 64 || P > 4) v[k] += dpp<SSM_DPP_ROW_HALF_MIRROR>(0.0f, v[k]);
        if (TEAM > 64 || P > 8) v[k] += dpp<SSM_DPP_ROW_MIRROR>(0.0f, v[k]);
        if (TEAM > 64 || P > 16) {
            const auto s = __builtin_amdgcn_permlane16_swap(__float_as_int(v[k]), __float_as_int(v[k]), false, false);
            v[k] = __int_as_float(s[0]) + __int_as_float(s[1]);
        }
        if (TEAM > 64 || P > 32) {
            const auto s = __builtin_amdgcn_permlane32_swap(__float_as_int(v[k]), __float_as_int(v[k]), false, false);
            v[k] = __int_as_float(s[0]) + __int_as_float(s[1]);
        }
    }
    if (TEAM > 64) {
        __syncthreads();   // what the sums before these read is done with
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (lane_id() == 0) lds[k][threadIdx.x >> 6] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            v[k] = 0.0f;
#pragma unroll
            for (int w = 0; w < TEAM / 64; ++w) v[k] += lds[k][w];
        }
    }
}

// A lane's share of its team's groups.
template <int TEAM, int V, int R>
struct Share {
    int at[R];      // first channel of each vector (0 for none)
    bool has[R];
    int row, step, end;   // the team's rows
    __device__ __forceinline__ Share(const NormParams& p) {
        const int l = TEAM == 64 ? lane_id() : (int)threadIdx.x;
        const int gb = blockIdx.x % p.gblocks, chunk = blockIdx.x / p.gblocks;
        const int g = TEAM == 64 ? gb * (64 / p.P) + l / p.P : gb;
        const int j = TEAM == 64 ? l % p.P : l;
        const int lanes = TEAM == 64 ? p.P : TEAM, nv = p.Cg / V;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            has[i] = g < p.G && j + i * lanes < nv;
            at[i] = has[i] ? g * p.Cg + (j + i * lanes) * V : 0;
        }
        // every so many rows: what all teams read at a time lies together
        row = chunk * norm_teams(TEAM) + (TEAM == 64 ? uniform(threadIdx.x >> 6) : 0);
        step = p.chunks * norm_teams(TEAM);
        end = p.T;
    }
};
// A row's normalised values in place of x (0 where the lane has none), and 1 / sqrt(var + eps).
template <int TEAM, int V, int R>
__device__ __forceinline__ float normalise(float (&x)[R][V], const bool (&has)[R], const NormParams& p, float (*lds)[16]) {
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) s[0] += has[i] ? x[i][e] : 0.0f;
    group_sums<TEAM, 1>(s, p.P, lds);
    const float mean = s[0] * p.inv;
    s[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            x[i][e] = has[i] ? x[i][e] - mean : 0.0f;
            s[0] = fmaf(x[i][e], x[i][e], s[0]);
        }
    group_sums<TEAM, 1>(s, p.P, lds);
    const float rstd = __builtin_amdgcn_rsqf(fmaf(s[0], p.inv, p.eps));
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) x[i][e] *= rstd;
    return rstd;
}

}  // namespace ssm
