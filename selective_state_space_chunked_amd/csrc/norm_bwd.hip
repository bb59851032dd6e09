// Group norm of rows with activation and gate, backward (norm.hpp has the layout, norm_fwd.hip the forward):
//
//   gz = gy u sigmoid(z) (1 + z (1 - sigmoid(z))),  gu = gy z sigmoid(z),
//   gv = gu or gu sigmoid(v) (1 + v (1 - sigmoid(v))),  gw = sum gv xh,  gbias = sum gv over the rows,
//   gx = (gv w - mean(gv w) - xh mean(gv w xh)) / sqrt(var + eps), means over the group.
// The statistics are formed again from x, which is in registers anyway: nothing is kept from the forward.  Each
// workgroup adds its rows' gw and gbias, a small kernel the workgroups' sums, both in a fixed order.
//
// Bound by HBM: 16384 x 2048 in groups of 64, bf16 with a gate, 338 MB in 70 to 75 us (4.5 to 4.9 TB/s), and 4.7 us
// for the sums.
#include "norm.hpp"

namespace ssm {
namespace {

template <typename T, int TEAM, int V, int R>
__global__ __launch_bounds__(norm_threads(TEAM)) void norm_bwd_kernel(NormParams p) {
    __shared__ float lds[2][16];
    const Share<TEAM, V, R> at(p);
    float w[R][V], b[R][V], gw[R][V], gb[R][V];
    // A lane without channels has read the first ones of the weights and of each row, which may be another group's and not
    // finite: what comes of them is chosen to be 0, not multiplied by it.
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            w[i][e] = p.w && at.has[i] ? p.w[at.at[i] + e] : 1.0f;
            b[i][e] = p.bias && at.has[i] ? p.bias[at.at[i] + e] : 0.0f;
            gw[i][e] = gb[i][e] = 0.0f;
        }
    const T* const x = (const T*)p.x;
    const T* const z = (const T*)p.z;
    const T* const gy = (const T*)p.gy;
    if (at.row < at.end) {
        Chan<T, V> cx[R], cz[R], cg[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            cx[i].load(x + at.row * p.sx + at.at[i]);
            cg[i].load(gy + at.row * p.sgy + at.at[i]);
            if (z) cz[i].load(z + at.row * p.sz + at.at[i]);
        }
        for (int row = at.row; row < at.end; row += at.step) {
            float xh[R][V], g[R][V], zv[R][V];
            const int next = min(row + at.step, at.end - 1);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                cx[i].get(xh[i]);
                cg[i].get(g[i]);
                if (z) cz[i].get(zv[i]);
                cx[i].load(x + next * p.sx + at.at[i]);
                cg[i].load(gy + next * p.sgy + at.at[i]);
                if (z) cz[i].load(z + next * p.sz + at.at[i]);
            }
            const float rstd = normalise<TEAM, V, R>(xh, at.has, p, lds);
            float m[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < R; ++i) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float v = fmaf(xh[i][e], w[i][e], b[i][e]);
                    float gv = g[i][e];
                    const float sv = p.silu ? sigmoid_f(v) : 1.0f;
                    if (z) {
                        const float zz = zv[i][e], sz = sigmoid_f(zz);
                        zv[i][e] = gv * v * sv * sz * fmaf(zz, 1.0f - sz, 1.0f);
                        gv *= zz * sz;
                    }
                    if (p.silu) gv *= sv * fmaf(v, 1.0f - sv, 1.0f);
                    gv = at.has[i] ? gv : 0.0f;
                    gw[i][e] = fmaf(gv, xh[i][e], gw[i][e]);
                    gb[i][e] += gv;
                    g[i][e] = gv * w[i][e];
                    m[0] += g[i][e];
                    m[1] = fmaf(g[i][e], xh[i][e], m[1]);
                }
                if (z && p.gz && at.has[i]) Chan<T, V>::store((T*)p.gz + row * p.sgz + at.at[i], zv[i]);
            }
            if (p.gx) {
                group_sums<TEAM, 2>(m, p.P, lds);
                const float m0 = m[0] * p.inv, m1 = m[1] * p.inv;
#pragma unroll
                for (int i = 0; i < R; ++i) {
#pragma unroll
                    for (int e = 0; e < V; ++e) g[i][e] = rstd * (fmaf(-xh[i][e], m1, g[i][e]) - m0);
                    if (at.has[i]) Chan<T, V>::store((T*)p.gx + row * p.sgx + at.at[i], g[i]);
                }
            }
        }
    }
    if (!p.sums) return;
    float* const pw = p.part + (int64_t)(blockIdx.x / p.gblocks) * 2 * p.C;
    float* const pb = pw + p.C;
    if (TEAM == 64) {   // the waves' sums, one after the other
        __shared__ float acc[2][R * V][64];
        const int l = lane_id(), me = threadIdx.x >> 6;
        for (int k = 0; k < kNormWaves; ++k) {
            if (me == k) {
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        if (k) {
                            gw[i][e] += acc[0][i * V + e][l];
                            gb[i][e] += acc[1][i * V + e][l];
                        }
                        acc[0][i * V + e][l] = gw[i][e];
                        acc[1][i * V + e][l] = gb[i][e];
                    }
            }
            __syncthreads();
        }
        if (me != kNormWaves - 1) return;
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (at.has[i])
#pragma unroll
            for (int e = 0; e < V; ++e) {
                pw[at.at[i] + e] = gw[i][e];
                pb[at.at[i] + e] = gb[i][e];
            }
}

constexpr int kSumWaves = 16;
__global__ __launch_bounds__(64 * kSumWaves) void norm_sum_kernel(NormParams p) {
    __shared__ float part[kSumWaves][64];
    const int k = blockIdx.y, lane = lane_id(), w = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (c < p.C)
#pragma unroll 4
        for (int n = w; n < p.chunks; n += kSumWaves) s += p.part[((int64_t)n * 2 + k) * p.C + c];
    part[w][lane] = s;
    __syncthreads();
    float* const out = k ? p.gbias : p.gw;
    if (w != 0 || c >= p.C || !out) return;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < kSumWaves; ++i) s += part[i][lane];
    out[c] = s;
}

template <typename T, int V, int R>
hipError_t launch(const NormParams& p, hipStream_t st) {
    const unsigned blocks = (unsigned)p.gblocks * (unsigned)p.chunks;
    if (p.team == 64) norm_bwd_kernel<T, 64, V, R><<<blocks, norm_threads(64), 0, st>>>(p);
    else if (p.team == 256) norm_bwd_kernel<T, 256, V, R><<<blocks, 256, 0, st>>>(p);
    else if constexpr (V * R <= 8)
        norm_bwd_kernel<T, 1024, V, R><<<blocks, 1024, 0, st>>>(p);
    else   // (a group has at most kNormMost channels: 1024 lanes of one vector of eight)
        return hipErrorInvalidValue;
    return hipGetLastError();
}
template <typename T, int V>
hipError_t launch_type(const NormParams& p, hipStream_t st) {
    if (p.V > 1) return p.R == 1 ? launch<T, V, 1>(p, st) : launch<T, V, 2>(p, st);
    if (p.R == 8) return launch<T, 1, 8>(p, st);
    norm_bwd_kernel<T, 64, 1, 2><<<(unsigned)p.gblocks * (unsigned)p.chunks, norm_threads(64), 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_bwd(const NormParams& p, int dtype, hipStream_t st) {
    return dtype ? launch_type<bf16_t, 8>(p, st) : launch_type<float, 4>(p, st);
}
hipError_t launch_norm_sum(const NormParams& p, hipStream_t st) {
    norm_sum_kernel<<<dim3((p.C + 63) / 64, 2), 64 * kSumWaves, 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace ssm
