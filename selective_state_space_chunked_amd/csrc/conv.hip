// The short causal convolution in front of a selective scan, forward and
// backward, and the 8-bit checkpoints of its input.
//
//   p_t = bias + sum_{k<W} w_k e_{t+k},  e = (W-1 earlier inputs | x),  y = p or p sigmoid(p)
//   gp = gy act'(p),  ge_j = sum_k w_k gp_{j-k},  gw_k = sum gp_t e_{t+k},  gbias = sum gp
//
// W is 2 to 4, so a step takes a handful of operations on the 4 (bf16) to 8
// bytes it moves: the kernels are bound by HBM.  A lane takes 8 consecutive
// steps of a row: one 16-byte access of bf16, and the W-1 steps it needs beside
// its own are a lane's away.
//
// Measured, kernel time and bytes moved (a copy of 256 MiB runs at 4.9 TB/s,
// read + written):
//   B=8 D=2048 L=4096 W=4 bf16   forward                63 us   4.4 TB/s
//                                forward + checkpoint   77 us   4.5 TB/s
//                                backward               77 us   5.3 TB/s
//                                backward from 8 bits   77 us   4.5 TB/s
//                                checkpoint to bf16     32 us   6.4 TB/s
//   B=1 D=1024 L=128000 f32      checkpoint            145 us   4.6 TB/s
//                                checkpoint to f32     124 us   5.4 TB/s
#include <algorithm>

#include "buffer.hpp"
#include "common.hpp"
#include "kernels.hpp"

namespace ssm {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTiny8 = 7.888609052210118e-31f;   // 2^-100: blocks below it are held as zeros
constexpr float kTop8 = 0x1.020406p+121f;          // the largest scale whose product with 127 is finite

__device__ __forceinline__ float sigmoid_f(float v) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * kLog2e));
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Accesses of 16 and 8 bytes at any element's address (global memory takes them unaligned): rows need not
// start at 16-byte units.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2), aligned(1)));
typedef float f32x4 __attribute__((ext_vector_type(4), aligned(4)));

// a run to a stream: float to bf16 by the conversion instruction, to nearest even
__device__ __forceinline__ void store_stream(float* p, const float (&v)[kConvRun], int n) {
    if (n >= kConvRun) {
        *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
    } else if (n > 0) {
#pragma unroll
        for (int j = 0; j < kConvRun; ++j)
            if (j < n) p[j] = v[j];
    }
}
__device__ __forceinline__ void store_stream(bf16_t* p, const float (&v)[kConvRun], int n) {
    uint32_t w[kConvRun / 2];
#pragma unroll
    for (int j = 0; j < kConvRun / 2; ++j)
        w[j] = (uint32_t)__builtin_bit_cast(bf16_t, (__bf16)v[2 * j]) |
               ((uint32_t)__builtin_bit_cast(bf16_t, (__bf16)v[2 * j + 1]) << 16);
    if (n >= kConvRun) {
        *reinterpret_cast<u32x4*>(p) = u32x4{w[0], w[1], w[2], w[3]};
    } else if (n > 0) {
#pragma unroll
        for (int j = 0; j < kConvRun; ++j)
            if (j < n) p[j] = (bf16_t)(w[j / 2] >> (16 * (j & 1)));
    }
}

// A lane's left and right neighbour in the wave (lane 0, lane 63: `edge`).
__device__ __forceinline__ float from_left(float v, float edge) {
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(edge), __float_as_int(v), 0x138, 0xf, 0xf, false));
}
__device__ __forceinline__ float from_right(float v, float edge) {
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(edge), __float_as_int(v), 0x130, 0xf, 0xf, false));
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
// max |x| of a checkpoint block as a bit pattern: of non-negative floats the
// integers order as the values do, infinity above all numbers and NaN above it.
__device__ __forceinline__ int block_max(int m) {   // over aligned groups of 8 lanes
    m = max(m, dpp_i<SSM_DPP_QUAD(1, 0, 3, 2)>(0, m));
    m = max(m, dpp_i<SSM_DPP_QUAD(2, 3, 0, 1)>(0, m));
    return max(m, dpp_i<SSM_DPP_ROW_HALF_MIRROR>(0, m));
}

// rint(v inv) in the low byte: the product rounded to fp32, then to a whole number by adding 1.5 * 2^23 (where
// the spacing of fp32 is 1), to nearest even both times
__device__ __forceinline__ uint32_t nearest_byte(float v, float inv) {
#pragma clang fp contract(off)
    const float q = v * inv;
    return __float_as_uint(q + 12582912.0f);
}
__device__ __forceinline__ uint32_t four_bytes(const uint32_t* k) {
    const uint32_t lo = __builtin_amdgcn_perm(k[1], k[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(k[3], k[2], 0x0c0c0400u);
    return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}

// gy silu'(p) of the step whose window is e[0..W-1]
template <int W>
__device__ __forceinline__ float grad_pre(const float* e, const float (&w)[W], float bias, float gy) {
    float a = bias;
#pragma unroll
    for (int k = 0; k < W; ++k) a = fmaf(w[k], e[k], a);
    const float s = sigmoid_f(a), gs = gy * s;   // gy s (1 + a (1 - s))
    return fmaf(gs, fmaf(-a, s, a), gs);
}

// A run of eight steps as loaded, turned into floats where it is used (so loads stay under way meanwhile).
template <typename T> struct Run;
template <> struct Run<bf16_t> {
    u32x4 r;
    __device__ __forceinline__ void load(const bf16_t* p) { r = *reinterpret_cast<const u32x4*>(p); }
    __device__ __forceinline__ void load(const bf16_t* p, int n) {   // the first n
        r = u32x4(0);
        if (n >= kConvRun) {
            load(p);
        } else if (n > 0) {
            uint32_t w[4] = {};
#pragma unroll
            for (int j = 0; j < kConvRun; ++j)
                if (j < n) w[j / 2] |= (uint32_t)p[j] << (16 * (j & 1));
            r = u32x4{w[0], w[1], w[2], w[3]};
        }
    }
    __device__ __forceinline__ void get(float (&v)[kConvRun]) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = __uint_as_float(w[e] << 16);
            v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
    }
};
template <> struct Run<float> {
    f32x4 r[2];
    __device__ __forceinline__ void load(const float* p) {
        r[0] = *reinterpret_cast<const f32x4*>(p);
        r[1] = *reinterpret_cast<const f32x4*>(p + 4);
    }
    __device__ __forceinline__ void load(const float* p, int n) {
        r[0] = r[1] = f32x4(0.0f);
        if (n >= kConvRun) {
            load(p);
        } else if (n > 0) {
            float v[kConvRun];
#pragma unroll
            for (int j = 0; j < kConvRun; ++j) v[j] = j < n ? p[j] : 0.0f;
            r[0] = f32x4{v[0], v[1], v[2], v[3]};
            r[1] = f32x4{v[4], v[5], v[6], v[7]};
        }
    }
    __device__ __forceinline__ void get(float (&v)[kConvRun]) const {
        v[0] = r[0].x; v[1] = r[0].y; v[2] = r[0].z; v[3] = r[0].w;
        v[4] = r[1].x; v[5] = r[1].y; v[6] = r[1].z; v[7] = r[1].w;
    }
};
struct Run8 {
    u32x2 r;
    float s;
    __device__ __forceinline__ void load(const int8_t* p, const float* sc) {
        r = *reinterpret_cast<const u32x2*>(p);
        s = *sc;
    }
    __device__ __forceinline__ void load(const int8_t* p, const float* sc, int n) {
        r = u32x2(0);
        s = 0.0f;
        if (n >= kConvRun) {
            load(p, sc);
        } else if (n > 0) {
            uint32_t w[2] = {};
            s = *sc;
#pragma unroll
            for (int j = 0; j < kConvRun; ++j)
                if (j < n) w[j / 4] |= (uint32_t)(uint8_t)p[j] << (8 * (j & 3));
            r = u32x2{w[0], w[1]};
        }
    }
    // q s as 2 ((q + 128) h - 128 h) with h = s / 2: the sum of unsigned bytes is one conversion, and the multiply-add
    // rounds the exact q h once.  128 s would overflow for blocks that reach to within 1/128 of the largest
    // float, 128 h does not; halving and doubling are exact.  B=8 D=2048 L=4096, backward to bf16 with the
    // sums over the parts: 86.6 us, by signed bytes and one product (more instructions) 92.1.
    __device__ __forceinline__ void get(float (&v)[kConvRun]) const {
        const uint32_t w[2] = {r.x ^ 0x80808080u, r.y ^ 0x80808080u};
        const float h = 0.5f * s, off = -128.0f * h;
#pragma unroll
        for (int j = 0; j < kConvRun; ++j) v[j] = 2.0f * fmaf((float)((w[j / 4] >> (8 * (j & 3))) & 255u), h, off);
    }
};

// Forward: a workgroup takes TX lanes' runs of TY rows (TX * TY = 256), UNITS neighbouring groups of rows, with all
// loads issued before the first is used; the grid runs along the steps first, so the workgroups under way sweep
// the streams in order (along the channels first it takes longer).  A lane's inputs before its own come from its left
// neighbour by a lane move, at a wave's first lane from memory (lanes 0 .. W-2 load them with the rest).  With P8 the
// eight lanes of a 64-step block agree on its scale (TX >= 8).
template <typename T, int W, bool X8, bool P8, int UNITS>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvParams p, int dblocks) {
    constexpr int H = W - 1, R = kConvRun;
    const int run = blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.z, t0 = run * R;
    // the W-1 steps before a lane's own are the left neighbour's last ones
    for (int db = blockIdx.y; db < dblocks; db += gridDim.y) {
        Run<T> x[UNITS];
        Run8 q[UNITS];
        float left[UNITS][H], w[UNITS][W], bias[UNITS], halo[UNITS];
        int n[UNITS];
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int d = (db * UNITS + u) * blockDim.y + threadIdx.y;
            n[u] = d < p.D && run < p.nrun ? p.L - t0 : 0;
            const Row<T, X8> in = row_of<T, X8>(p, b, n[u] > 0 ? d : 0);
            if (X8) {
                if (n[u] >= R) q[u].load(in.q + t0, in.s + t0 / kCkptBlock);
                else q[u].load(in.q + t0, in.s + t0 / kCkptBlock, n[u]);
            } else {
                if (n[u] >= R) x[u].load(in.x + t0);
                else x[u].load(in.x + t0, n[u]);
            }
            const int dw = n[u] > 0 && p.y ? d : 0;
#pragma unroll
            for (int k = 0; k < W; ++k) w[u][k] = p.y ? p.w[(int64_t)dw * W + k] : 0.0f;
            bias[u] = p.y && p.bias ? p.bias[dw] : 0.0f;
#pragma unroll
            for (int i = 0; i < H; ++i) left[u][i] = 0.0f;
            if (p.init && run == 0 && n[u] > 0) {
                const T* init = (const T*)p.init + ((int64_t)b * p.D + d) * H;
#pragma unroll
                for (int i = 0; i < H; ++i) left[u][i] = to_f32(init[i]);
            }
            // lane i < H: the input H - i steps before lane 0's run, where the wave begins inside a row
            const int th = uniform(t0) - H + lane_id(), n0 = uniform(n[u]), d0 = uniform(d);
            halo[u] = 0.0f;
            if (lane_id() < H && th >= 0 && n0 > 0 && p.y) halo[u] = row_of<T, X8>(p, b, d0).at(th);
        }
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int d = (db * UNITS + u) * blockDim.y + threadIdx.y;
            const int64_t row = (int64_t)b * p.D + d;
            float v[R], e[R + H];
            if (X8) q[u].get(v);
            else x[u].get(v);
            if (P8) {
                int m = 0;
#pragma unroll
                for (int j = 0; j < R; ++j) m = max(m, __float_as_int(v[j]) & 0x7fffffff);   // past the end: 0
                m = block_max(m);
                const float amax = __int_as_float(m);
                const bool bad = m >= 0x7f800000, zero = amax < kTiny8;
                const float scale = bad ? __int_as_float(0x7fc00000) : zero ? 0.0f : fminf(amax / 127.0f, kTop8);
                const float inv = bad || zero ? 0.0f : 127.0f / amax;
                if (n[u] > 0) {
                    int8_t* o = p.o8 + row * p.L + t0;
                    uint32_t k[R];
#pragma unroll
                    for (int j = 0; j < R; ++j) k[j] = nearest_byte(v[j], inv);
                    const uint32_t w0 = bad ? 0 : four_bytes(k), w1 = bad ? 0 : four_bytes(k + 4);
                    if (n[u] >= R) {
                        *reinterpret_cast<u32x2*>(o) = u32x2{w0, w1};
                    } else {
#pragma unroll
                        for (int j = 0; j < R; ++j)
                            if (j < n[u]) o[j] = (int8_t)((j < 4 ? w0 >> (8 * j) : w1 >> (8 * (j - 4))) & 255);
                    }
                    if ((run & 7) == 0) p.o8_scale[row * p.nblk + run / 8] = scale;
                }
            }
            if (p.last && run == 0 && n[u] > 0) {
                const Row<T, X8> in = row_of<T, X8>(p, b, d);
                T* last = (T*)p.last + row * H;
                for (int i = 0; i < H; ++i) last[i] = from_f32<T>(in.at(p.L - H + i));
            }
            if (!p.y) continue;
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const float edge = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(halo[u]), i));
                e[i] = from_left(v[R - H + i], edge);
                e[i] = run == 0 ? left[u][i] : e[i];
            }
#pragma unroll
            for (int j = 0; j < R; ++j) e[H + j] = v[j];
            if (n[u] <= 0) continue;
            float o[R];
#pragma unroll
            for (int j = 0; j < R; ++j) {
                float a = bias[u];
#pragma unroll
                for (int k = 0; k < W; ++k) a = fmaf(w[u][k], e[j + k], a);
                o[j] = p.silu ? a * sigmoid_f(a) : a;
            }
            store_stream((T*)p.y + b * p.sy[0] + d * p.sy[1] + t0, o, n[u]);
        }
    }
}

// What a lane has of its run, loaded a step ahead.
template <typename T, int W, bool X8>
struct BwdTile {
    static constexpr int H = W - 1, R = kConvRun;
    int b, run, n;      // n: steps from the run's first one on, 0 for a lane without an item
    bool full;          // every lane's run is whole
    Run<T> g, x;
    Run8 q;
    float halo;         // lane i < H: the input H - i steps before lane 0's run
    T* gx;
    __device__ __forceinline__ void get_x(float (&v)[R]) const {
        if (X8) q.get(v);
        else x.get(v);
    }
};
// A lane's item of one channel, batch row and run (item = row * runs + run), and the streams' pointers there.  It
// moves back by a workgroup's 256 items without a division or a product: q rows and r runs, and one more row where
// the runs underflow.
template <typename T, int W, bool X8>
struct BwdAt {
    static constexpr int H = W - 1, R = kConvRun;
    int item, b, run, q, r;
    const T *x, *gy;
    const int8_t* x8;
    const float* s;
    T* gx;
    int64_t mx, mg, mo;   // elements back for q rows and r runs

    __device__ __forceinline__ BwdAt(const ConvParams& p, int d, int i) {
        item = i;
        b = i / p.nrun;
        run = i - b * p.nrun;
        q = 256 / p.nrun;
        r = 256 - q * p.nrun;
        x = (const T*)p.x + b * p.sx[0] + d * p.sx[1] + run * R;
        gy = (const T*)p.gy + b * p.sgy[0] + d * p.sgy[1] + run * R;
        gx = (T*)p.gx + b * p.sgx[0] + d * p.sgx[1] + run * R;
        x8 = p.x8 + ((int64_t)b * p.D + d) * p.L + run * R;
        mx = X8 ? q * ((int64_t)p.D * p.L) + r * R : q * p.sx[0] + r * R;
        mg = q * p.sgy[0] + r * R;
        mo = q * p.sgx[0] + r * R;
    }
    __device__ __forceinline__ void back(const ConvParams& p) {
        item -= 256;
        b -= q;
        run -= r;
        const bool w = run < 0;
        b -= w ? 1 : 0;
        run += w ? p.nrun : 0;
        const int64_t row = (int64_t)p.nrun * R;
        if (X8) x8 -= mx + (w ? (int64_t)p.D * p.L - row : 0);
        else x -= mx + (w ? p.sx[0] - row : 0);
        gy -= mg + (w ? p.sgy[0] - row : 0);
        gx -= mo + (w ? p.sgx[0] - row : 0);
    }
    __device__ __forceinline__ void load(const ConvParams& p, int d, int end, BwdTile<T, W, X8>& t) const {
        const int lane = lane_id();
        const bool act = item < end;
        t.b = act ? b : 0;
        t.run = act ? run : 0;
        t.n = act ? p.L - run * R : 0;
        t.full = __all(t.n >= R);
        t.gx = gx;
        if (t.full) t.g.load(gy);
        else t.g.load(gy, t.n);
        if (X8) {
            const float* sc = p.x8_scale + ((int64_t)b * p.D + d) * p.nblk + run / (kCkptBlock / R);
            if (t.full) t.q.load(x8, sc);
            else t.q.load(x8, sc, t.n);
        } else {
            if (t.full) t.x.load(x);
            else t.x.load(x, t.n);
        }
        const int t0 = uniform(t.run) * R - H + lane;   // in lane 0's row
        t.halo = 0.0f;
        if (lane < H && t0 >= 0 && t0 < p.L) t.halo = row_of<T, X8>(p, uniform(t.b), d).at(t0);
    }
};

// gw and gbias of a run's steps
template <int W>
__device__ __forceinline__ void add_steps(float (&acc)[W + 1], const float* gp, const float* e) {
#pragma unroll
    for (int j = 0; j < kConvRun; ++j) {
#pragma unroll
        for (int q = 0; q < W; ++q) acc[q] = fmaf(gp[j], e[j + q], acc[q]);
        acc[W] += gp[j];
    }
}
// of the steps from `from` on and before `to`
template <int W>
__device__ __forceinline__ void add_steps(float (&acc)[W + 1], const float* gp, const float* e, int from, int to) {
    if (from <= 0 && to >= kConvRun) {
        add_steps<W>(acc, gp, e);
    } else if (from < kConvRun && to > 0) {
#pragma unroll
        for (int j = 0; j < kConvRun; ++j) {
            if (j >= from && j < to) {
#pragma unroll
                for (int q = 0; q < W; ++q) acc[q] = fmaf(gp[j], e[j + q], acc[q]);
                acc[W] += gp[j];
            }
        }
    }
}

// workgroup barrier that waits for LDS accesses only: loads and stores of global memory stay under way
__device__ __forceinline__ void lds_barrier() { __asm__ volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// a workgroup's sums of gw and gbias, of its lanes' acc
template <int W>
__device__ __forceinline__ void bwd_sums(const ConvParams& p, int d, int part, const float (&acc)[W + 1]) {
    const int lane = lane_id();
    if (!p.gw && !p.gbias) return;
    __shared__ float sum[4][W + 1];
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
// Backward: a workgroup takes the items (batch row, run) [part * per_part, ..)
// of one channel and leaves its sums of gw and gbias: no atomics, one order.
// Neighbouring lanes hold neighbouring items, so the inputs before a run and the
// gradients after it come from the lanes beside it, between waves through LDS.
// The items are taken 256 at a time from the last to the first, so the gradients
// after a group are those of the group before; the next group's loads are under
// way while one is computed.  For short rows (no whole tile of 512 steps, or over a
// third of the lanes idle in the kernel below): B=2 D=195 L=517 f32 5.4 us, of
// which a launch is 3.
template <typename T, int W, bool X8>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvParams p) {
    constexpr int H = W - 1, R = kConvRun;
    const int d = blockIdx.x % p.D, part = blockIdx.x / p.D;
    const int items = p.B * p.nrun;
    const int i0 = part * p.per_part, i1 = min(i0 + p.per_part, items);
    float w[W];
#pragma unroll
    for (int k = 0; k < W; ++k) w[k] = p.w[(int64_t)d * W + k];
    const float bias = p.bias ? p.bias[d] : 0.0f;
    const int lane = lane_id(), wave = uniform((int)threadIdx.x >> 6);
    __shared__ float begin[2][4][4];   // each wave's first H gradients, of this group and the last one
    float acc[W + 1] = {};
    const int groups = (i1 - i0 + 255) / 256;
    BwdTile<T, W, X8> c, nx;
    BwdAt<T, W, X8> at(p, d, i0 + (groups - 1) * 256 + (int)threadIdx.x);
    at.load(p, d, i1, c);
    float after[H] = {};   // wave 3: the first H gradients of the group to the right
    for (int k = groups - 1; k >= 0; --k) {
        if (k > 0) {
            at.back(p);
            at.load(p, d, i1, nx);
        }
        const int n = c.n, item = i0 + k * 256 + (int)threadIdx.x;
        float v[R], g[R], e[R + H], gp[R + H];
        c.get_x(v);
        c.g.get(g);
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const float edge = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(c.halo), i));
            e[i] = from_left(v[R - H + i], edge);
            e[i] = c.run == 0 ? 0.0f : e[i];
        }
        if (p.init && c.run == 0 && n > 0) {
            const T* init = (const T*)p.init + ((int64_t)c.b * p.D + d) * H;
#pragma unroll
            for (int i = 0; i < H; ++i) e[i] = to_f32(init[i]);
        }
#pragma unroll
        for (int j = 0; j < R; ++j) e[H + j] = v[j];
#pragma unroll
        for (int j = 0; j < R; ++j) gp[j] = g[j];
        if (p.silu) {   // one branch for the run: its steps' exp2 and reciprocals overlap
#pragma unroll
            for (int j = 0; j < R; ++j) gp[j] = grad_pre<W>(e + j, w, bias, g[j]);
        }
        if (!c.full) {
#pragma unroll
            for (int j = 0; j < R; ++j) gp[j] = j < n ? gp[j] : 0.0f;
        }
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < H; ++i) begin[k & 1][wave][i] = gp[i];
        }
        lds_barrier();
        float edge[H];
#pragma unroll
        for (int i = 0; i < H; ++i) {
            edge[i] = wave < 3 ? begin[k & 1][wave < 3 ? wave + 1 : 0][i] : after[i];
            after[i] = begin[k & 1][0][i];   // written again two barriers on
            gp[R + i] = from_right(gp[i], edge[i]);
        }
        if (k == groups - 1 && item + 1 == i1 && n > R) {   // the next item is another workgroup's: its first gradients again
            const Row<T, X8> in = row_of<T, X8>(p, c.b, d);
            const T* gy = (const T*)p.gy + c.b * p.sgy[0] + d * p.sgy[1];
            float f[2 * H], gr[H];
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const int t = c.run * R + R + i;
                f[i] = v[R - H + i];
                f[H + i] = t < p.L ? in.at(t) : 0.0f;
                gr[i] = t < p.L ? to_f32(gy[t]) : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < H; ++i) gp[R + i] = p.silu ? grad_pre<W>(f + i, w, bias, gr[i]) : gr[i];
        }
        if (n < R + H) {   // none after the row's last step
#pragma unroll
            for (int i = 0; i < H; ++i) gp[R + i] = R + i < n ? gp[R + i] : 0.0f;
        }
        if (c.full) {
            add_steps<W>(acc, gp, e);
        } else {
            add_steps<W>(acc, gp, e, 0, n);   // steps past the end add nothing, whatever lies there
        }
        const int64_t row = (int64_t)c.b * p.D + d;
        const T* gl = p.glast ? (const T*)p.glast + row * H : nullptr;
        if (p.gx) {
            float o[R];
#pragma unroll
            for (int j = 0; j < R; ++j) {
                float a = 0.0f;
#pragma unroll
                for (int q = 0; q < W; ++q) a = fmaf(w[q], gp[j + H - q], a);
                o[j] = a;
            }
            if (gl && n > 0 && n < R + H) {   // the last W-1 steps
#pragma unroll
                for (int j = 0; j < R; ++j)
                    if (j < n && j + H >= n) o[j] += to_f32(gl[j + H - n]);
            }
            if (c.full) store_stream(c.gx, o, R);
            else store_stream(c.gx, o, n);
        }
        if (p.ginit && c.run == 0 && n > 0) {
            T* gi = (T*)p.ginit + row * H;
#pragma unroll
            for (int j = 0; j < H; ++j) {
                float a = 0.0f;
#pragma unroll
                for (int q = 0; q <= j; ++q) a = fmaf(w[q], gp[j - q], a);
                if (gl && j >= n) a += to_f32(gl[j - n]);
                gi[j] = from_f32<T>(a);
            }
        }
        c = nx;
    }
    bwd_sums<W>(p, d, part, acc);
}

// Backward of rows of some length.  As above, but a wave takes tiles of 64 runs of one row each and forms the gradients
// after a tile again (one lane a step, from the inputs and gradients there), so waves wait for nothing of each other;
// a tile's row and place are scalar, and a lane's addresses are its fixed offset from them.  The loop issues the same
// loads and stores in every turn, so the wait for a tile's loads is one for these alone, with the next tile's loads
// and the last one's stores under way (with a branch around either the compiler has to wait for everything).  Bound by
// HBM, with half of the time in its 33 vector instructions a step (38 from 8 bits).  B=8 D=2048 L=4096 bf16, with the
// sums over the parts: 82 us, from 8 bits 81; the kernel above takes 94 and 92.
template <typename T, int W, bool X8>
struct RowTile {
    static constexpr int H = W - 1, R = kConvRun, N = 64 * R;   // steps of a tile
    Run<T> g, x;
    Run8 q;
    T ex;         // lane i < H: the input H - i steps before the tile; lane 32 + i, i < 2 H: i - H steps from its end
    int8_t exq;   // the same of a checkpoint
    float exs;
    T eg;         // lane 32 + i, i < H: gy i steps from the tile's end
    // a whole tile from step `first` on
    __device__ __forceinline__ void load(const ConvParams& p, int b, int d, int first) {
        const int at = lane_id() * R;
        const T* gy = (const T*)p.gy + b * p.sgy[0] + d * p.sgy[1] + first;
        const Row<T, X8> in = row_of<T, X8>(p, b, d);
        g.load(gy + at);
        if (X8) q.load(in.q + first + at, in.s + (first + at) / kCkptBlock);
        else x.load(in.x + first + at);
        edges(p, in, gy, first);
    }
    // a tile of the row's last `left` steps
    __device__ __forceinline__ void load(const ConvParams& p, int b, int d, int first, int left) {
        const int at = lane_id() * R;
        const T* gy = (const T*)p.gy + b * p.sgy[0] + d * p.sgy[1] + first;
        const Row<T, X8> in = row_of<T, X8>(p, b, d);
        g.load(gy + at, left - at);
        if (X8) q.load(in.q + first + at, in.s + (first + at) / kCkptBlock, left - at);
        else x.load(in.x + first + at, left - at);
        edges(p, in, gy, first);
    }
    __device__ __forceinline__ void edges(const ConvParams& p, const Row<T, X8>& in, const T* gy, int first) {
        const int lane = lane_id(), i = lane & 31, t = (lane < 32 ? 0 : N) - H + i;   // from the tile's first step
        const bool has = i < (lane < 32 ? H : 2 * H);
        const int lo = max(first - H, 0), some = min(p.L - lo, N + 2 * H);   // the first step in reach, and their number
        const uint32_t at = has ? (uint32_t)(first + t - lo) : 0x3fffffffu;     // before the row: past every end
        if (X8) {
            const int s0 = max(first / kCkptBlock - 1, 0);
            exq = buffer_load<int8_t>(buffer_of(in.q + lo, (uint32_t)some), at);
            exs = buffer_load<float>(buffer_of(in.s + s0, (uint32_t)min(p.nblk - s0, 16) * 4),
                                     has ? (uint32_t)(((first + t) >> 6) - s0) * 4 : 0x7fffffffu);
        } else {
            ex = buffer_load<T>(buffer_of(in.x + lo, (uint32_t)some * sizeof(T)), at * sizeof(T));
        }
        const int after = min(max(p.L - first - N, 0), H);
        eg = buffer_load<T>(buffer_of(gy + N, (uint32_t)after * sizeof(T)),
                            lane >= 32 ? (uint32_t)i * sizeof(T) : 0x7fffffffu);
    }
    __device__ __forceinline__ float edge() const { return X8 ? (float)exq * exs : to_f32(ex); }
};
template <typename T, int W, bool X8, bool GX, bool FULL>
__device__ __forceinline__ void bwd_tile(const ConvParams& p, const RowTile<T, W, X8>& c, int b, int d, int first, int cut,
                                         const float (&w)[W], float bias, float (&acc)[W + 1]) {
    constexpr int H = W - 1, R = kConvRun, N = 64 * R;
    const int lane = lane_id(), left = p.L - first, n = left - lane * R;   // steps from the tile's, the lane's first one on
    float v[R], e[R + H], gp[R + H], gr[R], ex = c.edge();
    if (X8) c.q.get(v);
    else c.x.get(v);
    c.g.get(gr);
    if (p.init && first < H) {
        if (lane < H - first) ex = to_f32(((const T*)p.init)[((int64_t)b * p.D + d) * H + first + lane]);
        __asm__ volatile("" : "+v"(ex));   // waited for here, not where every tile passes
    }
#pragma unroll
    for (int i = 0; i < H; ++i)
        e[i] = from_left(v[R - H + i], __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ex), i)));
    float f[W], ga = to_f32(c.eg);   // lane 32 + i: the window of the step i after the tile, and its gradient
    f[0] = ex;
#pragma unroll
    for (int k = 1; k < W; ++k) f[k] = from_right(f[k - 1], 0.0f);
#pragma unroll
    for (int j = 0; j < R; ++j) e[H + j] = v[j];
#pragma unroll
    for (int j = 0; j < R; ++j) gp[j] = gr[j];
    if (p.silu) {   // one branch for the run: its steps' exp2 and reciprocals overlap
#pragma unroll
        for (int j = 0; j < R; ++j) gp[j] = grad_pre<W>(e + j, w, bias, gr[j]);
        ga = grad_pre<W>(f, w, bias, ga);
    }
    if (!FULL) {
#pragma unroll
        for (int j = 0; j < R; ++j) gp[j] = j < n ? gp[j] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < H; ++i) {
        const float edge = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ga), 32 + i));
        gp[R + i] = from_right(gp[i], left > N + i ? edge : 0.0f);   // none after the row's last step
    }
    if (FULL && cut == first) add_steps<W>(acc, gp, e);
    else add_steps<W>(acc, gp, e, cut - first - lane * R, n);   // each step once, and none past the end
    const T* gl = p.glast ? (const T*)p.glast + ((int64_t)b * p.D + d) * H : nullptr;
    if (GX) {
        float o[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            float a = 0.0f;
#pragma unroll
            for (int q = 0; q < W; ++q) a = fmaf(w[q], gp[j + H - q], a);
            o[j] = a;
        }
        if (gl && left < N + H && n > 0 && n < R + H) {   // the last W-1 steps
#pragma unroll
            for (int j = 0; j < R; ++j)
                if (j < n && j + H >= n) o[j] += to_f32(gl[j + H - n]);
        }
        T* gx = (T*)p.gx + b * p.sgx[0] + d * p.sgx[1] + first;
        store_stream(gx + lane * R, o, FULL ? R : n);
    }
    if (p.ginit && first == 0 && lane == 0) {
        T* gi = (T*)p.ginit + ((int64_t)b * p.D + d) * H;
#pragma unroll
        for (int j = 0; j < H; ++j) {
            float a = 0.0f;
#pragma unroll
            for (int q = 0; q <= j; ++q) a = fmaf(w[q], gp[j - q], a);
            if (gl && j >= n) a += to_f32(gl[j - n]);
            gi[j] = from_f32<T>(a);
        }
    }
}
template <typename T, int W, bool X8, bool GX>
__global__ __launch_bounds__(256) void conv_bwd_rows_kernel(ConvParams p) {
    constexpr int N = 64 * kConvRun;
    const int d = blockIdx.x % p.D, part = blockIdx.x / p.D, wave = uniform((int)threadIdx.x >> 6);
    float w[W];
#pragma unroll
    for (int k = 0; k < W; ++k) w[k] = p.w[(int64_t)d * W + k];
    const float bias = p.bias ? p.bias[d] : 0.0f;
    float acc[W + 1] = {};
    // A row's end is a whole tile too, of its last N steps: those that the tile before has are formed again, to the same
    // values, and not added again.  (The runs of a checkpoint keep to its blocks.)
    const int rest = p.L - p.tiles * N;
    const bool whole = rest > 0 && (!X8 || p.L % kConvRun == 0);
    const int each = p.tiles + (whole ? 1 : 0);
    const int t0 = part * p.per_part + wave, t1 = min((part + 1) * p.per_part, p.B * each);   // tiles t0, t0 + 4, ..
    if (t0 < t1) {
        RowTile<T, W, X8> c, nx;
        int t = t0, b = t0 / each, seg = t0 - b * each, nb = b, ns = seg;
        auto next = [&] {   // the place of the wave's next tile; after the last one, that one's again
            if (t + 4 >= t1) return;
            ns += 4;
            while (ns >= each) {
                ns -= each;
                ++nb;
            }
        };
        auto first = [&](int s) { return s < p.tiles ? s * N : p.L - N; };
        c.load(p, b, d, first(seg));
        for (;;) {
            next();
            nx.load(p, nb, d, first(ns));
            bwd_tile<T, W, X8, GX, true>(p, c, b, d, first(seg), seg * N, w, bias, acc);
            b = nb; seg = ns; t += 4;
            if (t >= t1) break;
            next();
            c.load(p, nb, d, first(ns));
            bwd_tile<T, W, X8, GX, true>(p, nx, b, d, first(seg), seg * N, w, bias, acc);
            b = nb; seg = ns; t += 4;
            if (t >= t1) break;
        }
    }
    if (rest > 0 && !whole) {
        for (int b = part + p.parts * wave; b < p.B; b += p.parts * 4) {
            RowTile<T, W, X8> c;
            c.load(p, b, d, p.tiles * N, rest);
            bwd_tile<T, W, X8, GX, false>(p, c, b, d, p.tiles * N, p.tiles * N, w, bias, acc);
        }
    }
    bwd_sums<W>(p, d, part, acc);
}
// the parts of gw and gbias, added in order (10240 sums of 2 parts: 5 us, of which a launch is 3)
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

// the stream that a checkpoint stands for; workgroups as in the forward.  Bound by its writes.
template <typename T, int UNITS>
__global__ __launch_bounds__(256) void ckpt8_unpack_kernel(ConvParams p, int dblocks) {
    constexpr int R = kConvRun;
    const int run = blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.z, t0 = run * R;
    for (int db = blockIdx.y; db < dblocks; db += gridDim.y) {
        Run8 q[UNITS];
        int n[UNITS];
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int d = (db * UNITS + u) * blockDim.y + threadIdx.y;
            n[u] = d < p.D && run < p.nrun ? p.L - t0 : 0;
            const int64_t row = (int64_t)b * p.D + (n[u] > 0 ? d : 0);
            const int8_t* x8 = p.x8 + row * p.L + t0;
            const float* s = p.x8_scale + row * p.nblk + run / (kCkptBlock / R);
            if (n[u] >= R) q[u].load(x8, s);
            else q[u].load(x8, s, n[u]);
        }
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int d = (db * UNITS + u) * blockDim.y + threadIdx.y;
            float v[R];
            q[u].get(v);
            if (n[u] > 0) store_stream((T*)p.y + b * p.sy[0] + d * p.sy[1] + t0, v, n[u]);
        }
    }
}

// Lanes along a row's runs (at least 8: the lanes of a checkpoint block stay together), and whether there are
// workgroups enough to take two units each.
struct RowGrid {
    int tx, segs;
    bool two;
    explicit RowGrid(const ConvParams& p) {
        tx = 8;
        while (tx < 256 && tx < p.nrun) tx *= 2;
        const int ty = 256 / tx;
        segs = (p.nrun + tx - 1) / tx;
        two = (int64_t)segs * ((p.D + ty - 1) / ty) * p.B >= 4096;
    }
    dim3 block() const { return dim3(tx, 256 / tx); }
    int dblocks(const ConvParams& p, int units) const { return (p.D + units * (256 / tx) - 1) / (units * (256 / tx)); }
    dim3 grid(const ConvParams& p, int units) const { return dim3(segs, std::min(dblocks(p, units), 65535), p.B); }
};

template <typename T, int W, int UNITS>
void conv_fwd_u(const ConvParams& p, const RowGrid& r, hipStream_t st) {
    const dim3 g = r.grid(p, UNITS), t = r.block();
    const int db = r.dblocks(p, UNITS);
    if (p.o8) conv_fwd_kernel<T, W, false, true, UNITS><<<g, t, 0, st>>>(p, db);
    else if (p.x8) conv_fwd_kernel<T, W, true, false, UNITS><<<g, t, 0, st>>>(p, db);
    else conv_fwd_kernel<T, W, false, false, UNITS><<<g, t, 0, st>>>(p, db);
}
template <typename T, int W>
hipError_t conv_fwd_w(const ConvParams& p, hipStream_t st) {
    const RowGrid r(p);
    if (r.two) conv_fwd_u<T, W, 2>(p, r, st);
    else conv_fwd_u<T, W, 1>(p, r, st);
    return hipGetLastError();
}
template <typename T>
hipError_t unpack_t(const ConvParams& p, hipStream_t st) {
    const RowGrid r(p);
    if (r.two) ckpt8_unpack_kernel<T, 2><<<r.grid(p, 2), r.block(), 0, st>>>(p, r.dblocks(p, 2));
    else ckpt8_unpack_kernel<T, 1><<<r.grid(p, 1), r.block(), 0, st>>>(p, r.dblocks(p, 1));
    return hipGetLastError();
}
template <typename T, int W>
hipError_t conv_bwd_w(const ConvParams& p, hipStream_t st) {
    const int64_t blocks = (int64_t)p.D * p.parts;
    if (blocks >= (1LL << 31)) return hipErrorInvalidValue;
    if (p.tiles && p.x8) {
        if (p.gx) conv_bwd_rows_kernel<T, W, true, true><<<(unsigned)blocks, 256, 0, st>>>(p);
        else conv_bwd_rows_kernel<T, W, true, false><<<(unsigned)blocks, 256, 0, st>>>(p);
    } else if (p.tiles) {
        if (p.gx) conv_bwd_rows_kernel<T, W, false, true><<<(unsigned)blocks, 256, 0, st>>>(p);
        else conv_bwd_rows_kernel<T, W, false, false><<<(unsigned)blocks, 256, 0, st>>>(p);
    }
    else if (p.x8) conv_bwd_kernel<T, W, true><<<(unsigned)blocks, 256, 0, st>>>(p);
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
    return dtype == 1 ? unpack_t<bf16_t>(p, st) : unpack_t<float>(p, st);
}

}  // namespace ssm
