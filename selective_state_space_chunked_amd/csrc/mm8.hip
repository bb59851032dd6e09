// Rows in 8-bit integers and their product with 8-bit weights, with a scale for each row (token) and each channel:
//
//   x8 = rint(x 127 / amax),  scale = amax / 127 of a row,
//   y[t][n] = x8_scale[t] w8_scale[n] sum_k x8[t][k] w8[n][k] + bias[n].
//
// The sums are whole numbers in 32 bits, so they are exact and do not depend on the order they are formed in (at most
// 2^17 - 1 products of at most 2^14).  Both operands have k contiguous, as the matrix instructions take them: a lane
// holds 16 bytes of one row, at the same k for both operands.  The weights are the instruction's first operand, so a
// lane's results are consecutive channels of one row of y.
#include <algorithm>

#include "tokens.hpp"

namespace ssm {
namespace {

typedef int i4 __attribute__((ext_vector_type(4)));
typedef int i16v __attribute__((ext_vector_type(16)));
typedef int i4u __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

// 16 bytes of a row of K from byte k on; those from K on are 0.
__device__ __forceinline__ i4 row_chunk(const int8_t* row, int k, int K) {
    if (k + 16 <= K) return *reinterpret_cast<const i4u*>(row + k);
    if (k >= K) return i4(0);
    uint64_t lo = 0, hi = 0;
    if (K >= 16) {   // the row's last 16, moved down
        const i4 v = *reinterpret_cast<const i4u*>(row + K - 16);
        lo = (uint32_t)v[0] | (uint64_t)(uint32_t)v[1] << 32;
        hi = (uint32_t)v[2] | (uint64_t)(uint32_t)v[3] << 32;
        const int s = 8 * (k + 16 - K);   // 8 .. 120
        if (s < 64) {
            lo = lo >> s | hi << (64 - s);
            hi >>= s;
        } else {
            lo = hi >> (s - 64);
            hi = 0;
        }
    } else {
        for (int j = 0; j < 16; ++j)
            if (k + j < K) (j < 8 ? lo : hi) |= (uint64_t)(uint8_t)row[k + j] << (8 * (j & 7));
    }
    return i4{(int)(uint32_t)lo, (int)(lo >> 32), (int)(uint32_t)hi, (int)(hi >> 32)};
}

// four channels of a row of y, the first n of them
template <typename T>
__device__ __forceinline__ void put4(T* y, const float (&v)[4], int n) {
    Vec<T> o;
    o.set(v);
    if (n >= 4) o.store(y);
    else if (n > 0) o.store(y, n);
}
// four sums to four values of y: rounded to fp32 once (exact below 2^24), then scaled and rounded to y's type
template <typename T>
__device__ __forceinline__ void finish4(const Mm8Params& p, const i4 acc, int t, int n0, const float (&sw)[4],
                                        const float (&bias)[4]) {
    if (t >= p.T || n0 >= p.N) return;
    const float sx = p.xs[t];
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = fmaf((float)acc[e], sx * sw[e], bias[e]);
    put4<T>((T*)p.y + (int64_t)t * p.sy + n0, v, p.N - n0);
}
__device__ __forceinline__ void channels4(const Mm8Params& p, int n0, float (&sw)[4], float (&bias)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int n = min(n0 + e, p.N - 1);
        sw[e] = p.ws[n];
        bias[e] = p.bias ? p.bias[n] : 0.0f;
    }
}

// Few rows: bound by reading the weights once.  A workgroup takes 16 channels and up to 16 TT rows, its waves the
// k of a row in turns of 128 bytes -- whole lines of the weights -- and the waves' sums are added in LDS.
constexpr int kFewWaves = 8, kFewStep = 128;
template <typename T, int TT>
__global__ __launch_bounds__(64 * kFewWaves) void mm8_few_kernel(Mm8Params p) {
    __shared__ i4 part[kFewWaves][TT][64];
    const int l = lane_id(), w = uniform(threadIdx.x >> 6), K = p.K;
    const int n0 = blockIdx.x * 16;
    const int8_t* const wr = p.w + (int64_t)min(n0 + l % 16, p.N - 1) * p.sw;
    const int8_t* xr[TT];
    i4 acc[TT];
#pragma unroll
    for (int i = 0; i < TT; ++i) {
        xr[i] = p.x + (int64_t)min(16 * i + l % 16, p.T - 1) * p.sx;
        acc[i] = i4(0);
    }
    const int kl = (l / 16) * 16;
    int k = w * kFewStep;
#pragma unroll 2
    for (; k + kFewStep <= K; k += kFewStep * kFewWaves) {
        i4 a[2], b[2][TT];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            a[h] = *reinterpret_cast<const i4u*>(wr + k + 64 * h + kl);
#pragma unroll
            for (int i = 0; i < TT; ++i) b[h][i] = *reinterpret_cast<const i4u*>(xr[i] + k + 64 * h + kl);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < TT; ++i) acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[h], b[h][i], acc[i], 0, 0, 0);
    }
    if (k < K) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const i4 a = row_chunk(wr, k + 64 * h + kl, K);
#pragma unroll
            for (int i = 0; i < TT; ++i)
                acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, row_chunk(xr[i], k + 64 * h + kl, K), acc[i], 0, 0, 0);
        }
    }
#pragma unroll
    for (int i = 0; i < TT; ++i) part[w][i][l] = acc[i];
    __syncthreads();
    // wave i finishes the i-th 16 rows: lane l has row l % 16 and channels 4 (l / 16) ..
    if (w >= TT) return;
    const int n = n0 + 4 * (l / 16);
    float sw[4], bias[4];
    channels4(p, n, sw, bias);
    i4 s(0);
#pragma unroll
    for (int v = 0; v < kFewWaves; ++v) s += part[v][w][l];
    finish4<T>(p, s, 16 * w + l % 16, n, sw, bias);
}

// Many rows: a workgroup takes BN channels and BT rows, 128 bytes of k at a time through LDS, WN x WT waves of 32 x 32
// tiles each.  A row's eight 16-byte chunks lie in LDS at places exchanged by the row's number (chunk c of row r at
// c ^ r % 8), so the lanes of a matrix instruction, which read the same chunk of 32 rows, meet all banks.
constexpr int kStep = 128;
template <typename T, int BN, int BT, int WN, int WT>
__global__ __launch_bounds__(64 * WN * WT) void mm8_tile_kernel(Mm8Params p, int nblocks) {
    constexpr int TH = 64 * WN * WT, CH = (BN + BT) * 8 / TH, MN = BN / WN / 32, MT = BT / WT / 32;
    __shared__ i4 lds[(BN + BT) * 8];
    const int l = lane_id(), wave = uniform(threadIdx.x >> 6), K = p.K;
    const int n0 = (blockIdx.x % nblocks) * BN, t0 = (blockIdx.x / nblocks) * BT;
    const int wn = (wave % WN) * (BN / WN), wt = (wave / WN) * (BT / WT);
    // chunk i of the thread: row i * TH / 8 + threadIdx.x / 8 of the channels, then of the rows
    const int c = threadIdx.x % 8;
    const int8_t* src[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int r = i * (TH / 8) + threadIdx.x / 8;
        src[i] = r < BN ? p.w + (int64_t)min(n0 + r, p.N - 1) * p.sw : p.x + (int64_t)min(t0 + r - BN, p.T - 1) * p.sx;
    }
    const int put = (threadIdx.x / 8) * 8 + (c ^ (threadIdx.x / 8) % 8);   // TH / 8 is a multiple of 8
    i4 next[CH];
    auto load = [&](int k) {
        if (k + kStep <= K) {
#pragma unroll
            for (int i = 0; i < CH; ++i) next[i] = *reinterpret_cast<const i4u*>(src[i] + k + 16 * c);
        } else {
#pragma unroll
            for (int i = 0; i < CH; ++i) next[i] = row_chunk(src[i], k + 16 * c, K);
        }
    };
    i16v acc[MN][MT];
#pragma unroll
    for (int i = 0; i < MN; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] = i16v(0);
    load(0);
    for (int k = 0; k < K; k += kStep) {
        __syncthreads();   // the step before is done with LDS
#pragma unroll
        for (int i = 0; i < CH; ++i) lds[i * TH + put] = next[i];
        __syncthreads();
        if (k + kStep < K) load(k + kStep);
#pragma unroll
        for (int s = 0; s < kStep / 32; ++s) {
            const int ch = (2 * s + l / 32) ^ (l % 8);
            i4 a[MN], b[MT];
#pragma unroll
            for (int i = 0; i < MN; ++i) a[i] = lds[(wn + 32 * i + l % 32) * 8 + ch];
#pragma unroll
            for (int j = 0; j < MT; ++j) b[j] = lds[(BN + wt + 32 * j + l % 32) * 8 + ch];
#pragma unroll
            for (int i = 0; i < MN; ++i)
#pragma unroll
                for (int j = 0; j < MT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[i], b[j], acc[i][j], 0, 0, 0);
        }
    }
#pragma unroll
    for (int i = 0; i < MN; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int n = n0 + wn + 32 * i + 8 * g + 4 * (l / 32);
            float sw[4], bias[4];
            channels4(p, n, sw, bias);
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                const i4 s = {acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
                finish4<T>(p, s, t0 + wt + 32 * j + l % 32, n, sw, bias);
            }
        }
}

// ---------------------------------------------------------------------------
// rows to 8 bits
// ---------------------------------------------------------------------------
constexpr float kTiny8 = 0x1p-100f;         // rows below it are all zeros
constexpr float kTop8 = 0x1.020406p+121f;   // the largest scale whose product with 127 is finite

__device__ __forceinline__ int wave_max(int v) {
    v = max(v, dpp_i<SSM_DPP_QUAD(1, 0, 3, 2)>(0, v));
    v = max(v, dpp_i<SSM_DPP_QUAD(2, 3, 0, 1)>(0, v));
    v = max(v, dpp_i<SSM_DPP_ROW_HALF_MIRROR>(0, v));
    v = max(v, dpp_i<SSM_DPP_ROW_MIRROR>(0, v));
    return max(max(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16)),
               max(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48)));
}
// A team -- a wave or a workgroup -- takes a row: four elements a lane at a time, the first kHeld of these kept from
// the largest magnitude's pass for the second one; longer rows are read again (from the caches).
constexpr int kHeld = 8;
template <typename T, int TEAM>
__global__ __launch_bounds__(256) void pack8_kernel(Pack8Params p) {
    __shared__ int most[4];
    const int l = TEAM == 64 ? lane_id() : (int)threadIdx.x;
    const int t = TEAM == 64 ? blockIdx.x * 4 + uniform(threadIdx.x >> 6) : blockIdx.x;
    if (t >= p.T) return;
    const T* const x = (const T*)p.x + (int64_t)t * p.sx;
    int8_t* const o = p.o + (int64_t)t * p.so;
    Vec<T> held[kHeld];
    int m = 0;   // magnitudes compare as whole numbers, NaN above all
    auto largest = [&](const Vec<T>& v) {
        float f[4];
        v.get(f);
#pragma unroll
        for (int e = 0; e < 4; ++e) m = max(m, __float_as_int(f[e]) & 0x7fffffff);
    };
    auto load = [&](Vec<T>& v, int k) {
        if (k + 4 <= p.K) v.load(x + k);
        else v.load(x + k, p.K - k);   // (none, where k is past the row)
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i) load(held[i], (i * TEAM + l) * 4);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) largest(held[i]);
    for (int k = (kHeld * TEAM + l) * 4; k < p.K; k += TEAM * 4) {
        Vec<T> v;
        load(v, k);
        largest(v);
    }
    m = wave_max(m);
    if (TEAM > 64) {
        if (lane_id() == 0) most[threadIdx.x >> 6] = m;
        __syncthreads();
        m = max(max(most[0], most[1]), max(most[2], most[3]));
    }
    const float amax = __int_as_float(m);
    const bool bad = m >= 0x7f800000, zero = amax < kTiny8;
    const float scale = bad ? __int_as_float(0x7fc00000) : zero ? 0.0f : fminf(amax / 127.0f, kTop8);
    const float inv = bad || zero ? 0.0f : 127.0f / amax;
    if (l == 0) p.scale[t] = scale;
    auto put = [&](const Vec<T>& v, int k) {
        if (k >= p.K) return;
        float f[4];
        v.get(f);
        int q[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) q[e] = bad ? 0 : (int)rintf(f[e] * inv);
        const uint32_t w = (q[0] & 255) | (q[1] & 255) << 8 | (q[2] & 255) << 16 | (uint32_t)(q[3] & 255) << 24;
        if (k + 4 <= p.K) {
            typedef uint32_t u1 __attribute__((aligned(1)));
            *reinterpret_cast<u1*>(o + k) = w;
        } else {
            for (int e = 0; e < p.K - k; ++e) o[k + e] = (int8_t)(w >> (8 * e));
        }
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i) put(held[i], (i * TEAM + l) * 4);
    for (int k = (kHeld * TEAM + l) * 4; k < p.K; k += TEAM * 4) {
        Vec<T> v;
        load(v, k);
        put(v, k);
    }
}

template <typename T>
hipError_t launch(const Mm8Params& p, hipStream_t st) {
    const int few = (p.T + 15) / 16;
    if (p.tile == 0) {
        const unsigned blocks = (unsigned)((p.N + 15) / 16);
        if (few == 1) mm8_few_kernel<T, 1><<<blocks, 64 * kFewWaves, 0, st>>>(p);
        else if (few == 2) mm8_few_kernel<T, 2><<<blocks, 64 * kFewWaves, 0, st>>>(p);
        else mm8_few_kernel<T, 4><<<blocks, 64 * kFewWaves, 0, st>>>(p);
    } else {
        const int nb = (p.N + p.tile - 1) / p.tile;
        const unsigned blocks = (unsigned)nb * (unsigned)((p.T + p.tile - 1) / p.tile);
        if (p.tile == 64) mm8_tile_kernel<T, 64, 64, 2, 2><<<blocks, 256, 0, st>>>(p, nb);
        else mm8_tile_kernel<T, 128, 128, 2, 2><<<blocks, 256, 0, st>>>(p, nb);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mm8(const Mm8Params& p, int dtype, hipStream_t st) {
    return dtype ? launch<bf16_t>(p, st) : launch<float>(p, st);
}
hipError_t launch_pack8(const Pack8Params& p, int dtype, hipStream_t st) {
    const bool wave = p.K <= 64 * 4 * kHeld;
    const unsigned blocks = (unsigned)(wave ? (p.T + 3) / 4 : p.T);
    if (dtype) {
        if (wave) pack8_kernel<bf16_t, 64><<<blocks, 256, 0, st>>>(p);
        else pack8_kernel<bf16_t, 256><<<blocks, 256, 0, st>>>(p);
    } else {
        if (wave) pack8_kernel<float, 64><<<blocks, 256, 0, st>>>(p);
        else pack8_kernel<float, 256><<<blocks, 256, 0, st>>>(p);
    }
    return hipGetLastError();
}

}  // namespace ssm
