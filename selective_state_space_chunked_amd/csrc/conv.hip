// The short causal convolution in front of a selective scan, forward and
// backward, and the 8-bit checkpoints of its input.
//
//   p_t = bias + sum_{k<W} w_k e_{t+k},  e = (W-1 earlier inputs | x),  y = p or p sigmoid(p)
//   gp = gy act'(p),  ge_j = sum_k w_k gp_{j-k},  gw_k = sum gp_t e_{t+k},  gbias = sum gp
//
// W is 2 to 4, so a step takes a handful of operations on the 4 (bf16) to 8
// bytes it moves: the kernels are bound by HBM.  A lane takes 8 consecutive
// steps of a row.
#include <algorithm>

#include "common.hpp"
#include "kernels.hpp"

namespace ssm {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTiny8 = 7.888609052210118e-31f;   // 2^-100: blocks below it are held as zeros

__device__ __forceinline__ float sigmoid_f(float v) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * kLog2e));
}

// One row's input: the stream itself, or the values its 8-bit checkpoint stands for.
template <typename T, bool X8>
struct Row {
    const T* x;
    const int8_t* q;
    const float* s;
    const T* init;   // the W-1 inputs before step 0, or null
    int L, W;
    __device__ __forceinline__ float at(int t) const {   // t in [-(W-1), L)
        if (t < 0) return init ? to_f32(init[t + W - 1]) : 0.0f;
        if (X8) return (float)q[t] * s[t / kCkptBlock];
        return to_f32(x[t]);
    }
};
template <typename T, bool X8>
__device__ __forceinline__ Row<T, X8> row_of(const ConvParams& p, int b, int d) {
    const int64_t r = (int64_t)b * p.D + d;
    Row<T, X8> o;
    o.x = X8 ? nullptr : (const T*)p.x + b * p.sx[0] + d * p.sx[1];
    o.q = X8 ? p.x8 + r * p.L : nullptr;
    o.s = X8 ? p.x8_scale + r * p.nblk : nullptr;
    o.init = p.init ? (const T*)p.init + r * (p.W - 1) : nullptr;
    o.L = p.L;
    o.W = p.W;
    return o;
}
// steps t0 .. t0+7 of the row (steps past the end 0)
template <typename T, bool X8>
__device__ __forceinline__ void load_x(const Row<T, X8>& r, int t0, float (&v)[kConvRun], bool vec) {
    if (X8 || t0 + kConvRun > r.L) {
#pragma unroll
        for (int j = 0; j < kConvRun; ++j) v[j] = t0 + j < r.L ? r.at(t0 + j) : 0.0f;
    } else {
        load_run<kConvRun>(r.x + t0, v, vec);
    }
}

// max |x| of a checkpoint block as a bit pattern: of non-negative floats the
// integers order as the values do, infinity above all numbers and NaN above it.
__device__ __forceinline__ int block_max(int m) {   // over aligned groups of 8 lanes
    m = max(m, dpp_i<SSM_DPP_QUAD(1, 0, 3, 2)>(0, m));
    m = max(m, dpp_i<SSM_DPP_QUAD(2, 3, 0, 1)>(0, m));
    return max(m, dpp_i<SSM_DPP_ROW_HALF_MIRROR>(0, m));
}

// Forward: block (TX lanes along the row, 256 / TX rows).  With P8 the eight
// lanes of a 64-step block agree on its scale (TX >= 8).
template <typename T, int W, bool X8, bool P8>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvParams p, int segs) {
    const int64_t rb = blockIdx.x / segs;
    const int run = (int)(blockIdx.x % segs) * blockDim.x + threadIdx.x;
    const int64_t row = rb * blockDim.y + threadIdx.y;
    const bool act = row < (int64_t)p.B * p.D && run < p.nrun;
    if (!P8 && !act) return;
    const int b = act ? (int)(row / p.D) : 0, d = act ? (int)(row % p.D) : 0;
    const Row<T, X8> in = row_of<T, X8>(p, b, d);
    const int t0 = run * kConvRun;
    float e[kConvRun + W - 1];
    float v[kConvRun] = {};
    if (act) load_x(in, t0, v, p.vx);
    if (P8) {
        int m = 0;
#pragma unroll
        for (int j = 0; j < kConvRun; ++j) m = max(m, __float_as_int(v[j]) & 0x7fffffff);
        m = block_max(m);
        const float amax = __int_as_float(m);
        const bool bad = m >= 0x7f800000, zero = amax < kTiny8;
        const float scale = bad ? __int_as_float(0x7fc00000) : zero ? 0.0f : amax / 127.0f;
        const float inv = bad || zero ? 0.0f : 127.0f / amax;
        if (act) {
            int8_t* o = p.o8 + row * p.L + t0;
            uint32_t w0 = 0, w1 = 0;
#pragma unroll
            for (int j = 0; j < kConvRun; ++j) {
                const int q = bad ? 0 : (int)rintf(v[j] * inv);
                if (j < 4) w0 |= (uint32_t)(q & 255) << (8 * j);
                else w1 |= (uint32_t)(q & 255) << (8 * (j - 4));
            }
            if (p.v8) {
                *reinterpret_cast<uint2*>(o) = make_uint2(w0, w1);
            } else {
#pragma unroll
                for (int j = 0; j < kConvRun; ++j)
                    if (t0 + j < p.L) o[j] = (int8_t)((j < 4 ? w0 >> (8 * j) : w1 >> (8 * (j - 4))) & 255);
            }
            if ((run & 7) == 0) p.o8_scale[row * p.nblk + run / 8] = scale;
        }
    }
    if (!act) return;
    if (p.last && run == 0) {
        T* last = (T*)p.last + row * (W - 1);
        for (int i = 0; i < W - 1; ++i) last[i] = from_f32<T>(in.at(p.L - (W - 1) + i));
    }
    if (!p.y) return;
#pragma unroll
    for (int i = 0; i < W - 1; ++i) e[i] = in.at(t0 - (W - 1) + i);
#pragma unroll
    for (int j = 0; j < kConvRun; ++j) e[W - 1 + j] = v[j];
    float w[W];
#pragma unroll
    for (int k = 0; k < W; ++k) w[k] = p.w[(int64_t)d * W + k];
    const float bias = p.bias ? p.bias[d] : 0.0f;
    float o[kConvRun];
#pragma unroll
    for (int j = 0; j < kConvRun; ++j) {
        float a = bias;
#pragma unroll
        for (int k = 0; k < W; ++k) a = fmaf(w[k], e[j + k], a);
        o[j] = p.silu ? a * sigmoid_f(a) : a;
    }
    store_run<kConvRun>((T*)p.y + b * p.sy[0] + d * p.sy[1] + t0, o, p.vy, p.L - t0);
}

// Backward: a workgroup takes the items (batch row, run) [part * per_part, ..)
// of one channel and leaves its sums of gw and gbias: no atomics, one order.
template <typename T, int W, bool X8>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvParams p) {
    const int d = blockIdx.x / p.parts, part = blockIdx.x % p.parts;
    const int items = p.B * p.nrun;
    const int i0 = part * p.per_part, i1 = min(i0 + p.per_part, items);
    float w[W];
#pragma unroll
    for (int k = 0; k < W; ++k) w[k] = p.w[(int64_t)d * W + k];
    const float bias = p.bias ? p.bias[d] : 0.0f;
    constexpr int H = W - 1, R = kConvRun;
    float acc[W + 1] = {};
    for (int it = i0 + (int)threadIdx.x; it < i1; it += 256) {
        const int b = it / p.nrun, run = it % p.nrun, t0 = run * R;
        const Row<T, X8> in = row_of<T, X8>(p, b, d);
        const T* gy = (const T*)p.gy + b * p.sgy[0] + d * p.sgy[1];
        float v[R], g[R];
        load_x(in, t0, v, p.vx);
        const int n = p.L - t0;   // steps from t0 on
        if (n >= R) load_run<R>(gy + t0, g, p.vgy);
        else load_run_masked<T, R>(gy + t0, g, n);
        float e[R + 2 * H], gp[R + H];
#pragma unroll
        for (int i = 0; i < H; ++i) e[i] = in.at(t0 - H + i);
#pragma unroll
        for (int j = 0; j < R; ++j) e[H + j] = v[j];
#pragma unroll
        for (int i = 0; i < H; ++i) e[H + R + i] = R + i < n ? in.at(t0 + R + i) : 0.0f;
#pragma unroll
        for (int j = 0; j < R + H; ++j) {
            float a = bias;
#pragma unroll
            for (int k = 0; k < W; ++k) a = fmaf(w[k], e[j + k], a);
            const float go = j < R ? g[j < R ? j : 0] : (j < n ? to_f32(gy[t0 + j]) : 0.0f);
            float q = go;
            if (p.silu) {
                const float s = sigmoid_f(a);
                q = go * s * fmaf(a, 1.0f - s, 1.0f);
            }
            gp[j] = j < n ? q : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if (j < n) {   // steps past the end add nothing, whatever lies there
#pragma unroll
                for (int k = 0; k < W; ++k) acc[k] = fmaf(gp[j], e[j + k], acc[k]);
                acc[W] += gp[j];
            }
        }
        const int64_t row = (int64_t)b * p.D + d;
        const T* gl = p.glast ? (const T*)p.glast + row * H : nullptr;
        if (p.gx) {
            float o[R];
#pragma unroll
            for (int j = 0; j < R; ++j) {
                float a = 0.0f;
#pragma unroll
                for (int k = 0; k < W; ++k) a = fmaf(w[k], gp[j + H - k], a);
                if (gl && j < n && j + H >= n) a += to_f32(gl[j + H - n]);
                o[j] = a;
            }
            store_run<R>((T*)p.gx + b * p.sgx[0] + d * p.sgx[1] + t0, o, p.vgx, n);
        }
        if (p.ginit && run == 0) {
            T* gi = (T*)p.ginit + row * H;
#pragma unroll
            for (int j = 0; j < H; ++j) {
                float a = 0.0f;
#pragma unroll
                for (int k = 0; k <= j; ++k) a = fmaf(w[k], gp[j - k], a);
                if (gl && j >= n) a += to_f32(gl[j - n]);
                gi[j] = from_f32<T>(a);
            }
        }
    }
    if (!p.gw && !p.gbias) return;
    __shared__ float sum[4][W + 1];
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int k = 0; k <= W; ++k) {
        float a = acc[k];
        for (int m = 32; m; m >>= 1) a += __shfl_xor(a, m);
        if (lane == 0) sum[threadIdx.x >> 6][k] = a;
    }
    __syncthreads();
    if (threadIdx.x <= W) {
        const int k = threadIdx.x;
        const float a = (sum[0][k] + sum[1][k]) + (sum[2][k] + sum[3][k]);
        if (p.parts > 1) p.part[((int64_t)part * p.D + d) * (W + 1) + k] = a;
        else if (k < W) { if (p.gw) p.gw[(int64_t)d * W + k] = a; }
        else if (p.gbias) p.gbias[d] = a;
    }
}
// the parts of gw and gbias, added in order
__global__ __launch_bounds__(256) void conv_reduce_kernel(ConvParams p) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, n = (int64_t)p.D * (p.W + 1);
    if (i >= n) return;
    float a = 0.0f;
    for (int q = 0; q < p.parts; ++q) a += p.part[q * n + i];
    const int64_t d = i / (p.W + 1);
    const int k = (int)(i % (p.W + 1));
    if (k < p.W) { if (p.gw) p.gw[d * p.W + k] = a; }
    else if (p.gbias) p.gbias[d] = a;
}

template <typename T>
__global__ __launch_bounds__(256) void ckpt8_unpack_kernel(ConvParams p, int segs) {
    const int64_t rb = blockIdx.x / segs;
    const int run = (int)(blockIdx.x % segs) * blockDim.x + threadIdx.x;
    const int64_t row = rb * blockDim.y + threadIdx.y;
    if (row >= (int64_t)p.B * p.D || run >= p.nrun) return;
    const int b = (int)(row / p.D), d = (int)(row % p.D), t0 = run * kConvRun;
    const int8_t* q = p.x8 + row * p.L + t0;
    const float s = p.x8_scale[row * p.nblk + run / 8];
    const int n = p.L - t0;
    float v[kConvRun];
#pragma unroll
    for (int j = 0; j < kConvRun; ++j) v[j] = j < n ? (float)q[j] * s : 0.0f;
    store_run<kConvRun>((T*)p.y + b * p.sy[0] + d * p.sy[1] + t0, v, p.vy, n);
}

// lanes along the row and rows per workgroup; blocks along the row
struct RowGrid {
    dim3 block;
    int segs;
    unsigned grid;
};
bool row_grid(const ConvParams& p, RowGrid* g) {
    int tx = 8;   // the lanes of a checkpoint block stay together
    while (tx < 256 && tx < p.nrun) tx *= 2;
    g->block = dim3(tx, 256 / tx);
    g->segs = (p.nrun + tx - 1) / tx;
    const int64_t rows = (int64_t)p.B * p.D, per = 256 / tx;
    const int64_t blocks = (rows + per - 1) / per * g->segs;
    if (blocks <= 0 || blocks >= (1LL << 31)) return false;
    g->grid = (unsigned)blocks;
    return true;
}

template <typename T, int W>
hipError_t conv_fwd_w(const ConvParams& p, hipStream_t st) {
    RowGrid g;
    if (!row_grid(p, &g)) return hipErrorInvalidValue;
    if (p.o8) conv_fwd_kernel<T, W, false, true><<<g.grid, g.block, 0, st>>>(p, g.segs);
    else if (p.x8) conv_fwd_kernel<T, W, true, false><<<g.grid, g.block, 0, st>>>(p, g.segs);
    else conv_fwd_kernel<T, W, false, false><<<g.grid, g.block, 0, st>>>(p, g.segs);
    return hipGetLastError();
}
template <typename T, int W>
hipError_t conv_bwd_w(const ConvParams& p, hipStream_t st) {
    const int64_t blocks = (int64_t)p.D * p.parts;
    if (blocks >= (1LL << 31)) return hipErrorInvalidValue;
    if (p.x8) conv_bwd_kernel<T, W, true><<<(unsigned)blocks, 256, 0, st>>>(p);
    else conv_bwd_kernel<T, W, false><<<(unsigned)blocks, 256, 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_conv_fwd(const ConvParams& p, int dtype, hipStream_t st) {
    if (dtype == 1)
        return p.W == 2 ? conv_fwd_w<bf16_t, 2>(p, st) : p.W == 3 ? conv_fwd_w<bf16_t, 3>(p, st) : conv_fwd_w<bf16_t, 4>(p, st);
    return p.W == 2 ? conv_fwd_w<float, 2>(p, st) : p.W == 3 ? conv_fwd_w<float, 3>(p, st) : conv_fwd_w<float, 4>(p, st);
}
hipError_t launch_conv_bwd(const ConvParams& p, int dtype, hipStream_t st) {
    if (dtype == 1)
        return p.W == 2 ? conv_bwd_w<bf16_t, 2>(p, st) : p.W == 3 ? conv_bwd_w<bf16_t, 3>(p, st) : conv_bwd_w<bf16_t, 4>(p, st);
    return p.W == 2 ? conv_bwd_w<float, 2>(p, st) : p.W == 3 ? conv_bwd_w<float, 3>(p, st) : conv_bwd_w<float, 4>(p, st);
}
hipError_t launch_conv_reduce(const ConvParams& p, hipStream_t st) {
    const int64_t n = (int64_t)p.D * (p.W + 1);
    conv_reduce_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(p);
    return hipGetLastError();
}
hipError_t launch_ckpt8_unpack(const ConvParams& p, int dtype, hipStream_t st) {
    RowGrid g;
    if (!row_grid(p, &g)) return hipErrorInvalidValue;
    if (dtype == 1) ckpt8_unpack_kernel<bf16_t><<<g.grid, g.block, 0, st>>>(p, g.segs);
    else ckpt8_unpack_kernel<float><<<g.grid, g.block, 0, st>>>(p, g.segs);
    return hipGetLastError();
}

}  // namespace ssm
