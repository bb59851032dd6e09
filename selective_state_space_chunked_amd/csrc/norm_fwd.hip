// Group norm of rows with activation and gate, forward (norm.hpp has the layout):
//
//   xh = (x - mean) / sqrt(var + eps) over the channels of a group of one row,
//   v = xh w + bias,  u = v or v sigmoid(v),  y = u or u z sigmoid(z).
#include "norm.hpp"

namespace ssm {
namespace {

template <typename T, int TEAM, int V, int R>
__global__ __launch_bounds__(norm_threads(TEAM)) void norm_fwd_kernel(NormParams p) {
    __shared__ float lds[1][16];
    const Share<TEAM, V, R> at(p);
    float w[R][V], b[R][V];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            w[i][e] = p.w ? p.w[at.at[i] + e] : 1.0f;
            b[i][e] = p.bias ? p.bias[at.at[i] + e] : 0.0f;
        }
    if (at.row >= at.end) return;
    Chan<T, V> cx[R], cz[R];
    const T* const x = (const T*)p.x;
    const T* const z = (const T*)p.z;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        cx[i].load(x + at.row * p.sx + at.at[i]);
        if (z) cz[i].load(z + at.row * p.sz + at.at[i]);
    }
    for (int row = at.row; row < at.end; row += at.step) {
        float v[R][V], g[R][V];
        const int next = min(row + at.step, at.end - 1);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            cx[i].get(v[i]);
            if (z) cz[i].get(g[i]);
            cx[i].load(x + next * p.sx + at.at[i]);
            if (z) cz[i].load(z + next * p.sz + at.at[i]);
        }
        normalise<TEAM, V, R>(v, at.has, p, lds);
#pragma unroll
        for (int i = 0; i < R; ++i) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                v[i][e] = fmaf(v[i][e], w[i][e], b[i][e]);
                if (p.silu) v[i][e] *= sigmoid_f(v[i][e]);
                if (z) v[i][e] *= g[i][e] * sigmoid_f(g[i][e]);
            }
            if (at.has[i]) Chan<T, V>::store((T*)p.y + row * p.sy + at.at[i], v[i]);
        }
    }
}

template <typename T, int V, int R>
hipError_t launch(const NormParams& p, hipStream_t st) {
    const unsigned blocks = (unsigned)p.gblocks * (unsigned)p.chunks;
    if (p.team == 64) norm_fwd_kernel<T, 64, V, R><<<blocks, norm_threads(64), 0, st>>>(p);
    else if (p.team == 256) norm_fwd_kernel<T, 256, V, R><<<blocks, 256, 0, st>>>(p);
    else norm_fwd_kernel<T, 1024, V, R><<<blocks, 1024, 0, st>>>(p);
    return hipGetLastError();
}
template <typename T, int V>
hipError_t launch_type(const NormParams& p, hipStream_t st) {
    if (p.V > 1) return p.R == 1 ? launch<T, V, 1>(p, st) : launch<T, V, 2>(p, st);
    if (p.R == 8) return launch<T, 1, 8>(p, st);
    norm_fwd_kernel<T, 64, 1, 2><<<(unsigned)p.gblocks * (unsigned)p.chunks, norm_threads(64), 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_fwd(const NormParams& p, int dtype, hipStream_t st) {
    return dtype ? launch_type<bf16_t, 8>(p, st) : launch_type<float, 4>(p, st);
}

}  // namespace ssm
