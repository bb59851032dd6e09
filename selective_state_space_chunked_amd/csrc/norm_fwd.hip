// Group norm of rows with activation and gate, forward (norm.hpp has the layout):
//
//   xh = (x - mean) / sqrt(var + eps) over the channels of a group of one row,
//   v = xh w + bias,  u = v or v sigmoid(v),  y = u or u z sigmoid(z).
//
// Bound by HBM: 16384 x 2048 in groups of 64, bf16 with a gate, 201 MB in 48 us (4.2 TB/s; a copy of 4 GiB has 4.75).
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
    // The next row comes while one is worked on.  (Two rows at a time are no faster where a lane has one vector of each,
    // and slower where it has single elements: 16384 x 2080 in groups of 65, bf16, 60 us and 73.)
    auto load = [&](int row) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            cx[i].load(x + row * p.sx + at.at[i]);
            if (z) cz[i].load(z + row * p.sz + at.at[i]);
        }
    };
    load(at.row);
    for (int row = at.row; row < at.end; row += at.step) {
        float v[R][V], g[R][V];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            cx[i].get(v[i]);
            if (z) cz[i].get(g[i]);
        }
        load(min(row + at.step, at.end - 1));
        normalise<TEAM, V, R>(v, at.has, p, lds);
#pragma unroll
        for (int i = 0; i < R; ++i) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float u = fmaf(v[i][e], w[i][e], b[i][e]);
                if (p.silu) u *= sigmoid_f(u);
                if (z) u *= g[i][e] * sigmoid_f(g[i][e]);
                v[i][e] = u;
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
    else if constexpr (V * R <= 8)
        norm_fwd_kernel<T, 1024, V, R><<<blocks, 1024, 0, st>>>(p);
    else   // (a group has at most kNormMost channels: 1024 lanes of one vector of eight)
        return hipErrorInvalidValue;
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
