// Rows in 8-bit integers and their product with 8-bit weights, with a scale for each row (token) and each channel:
//
//   x8 = rint(x 127 / amax),  scale = amax / 127 of a row,
//   y[t][n] = x8_scale[t] w8_scale[n] sum_k x8[t][k] w8[n][k] + bias[n].
//
// The sums are whole numbers in 32 bits, so they are exact and do not depend on the order they are formed in (at most
// 2^17 - 1 products of at most 2^14).  Both operands have k contiguous, as the matrix instructions take them: a lane
// holds 16 bytes of one row, at the same k for both operands.  The weights are the instruction's first operand, so a
// lane's results are consecutive channels of one row of y.
//
// 8192 x 4096 x 8192 to bf16 takes 244 us while the card is cool (2.2 Pop/s; the library's product of the same operands,
// without scales, 252) and 275 to 285 with one product after the other, when its power limit lowers the clock.  The
// matrix instructions are busy for 54 to 62 % of the cycles; of 424 thousand, the results' scaling and stores are 34, the
// loads 64.  64 x 4096 x 2048 takes 5.3 us and 1 x 2048 x 4096 3.5, where the weights alone are 1.8 us of traffic: latency.
// Rows to 8 bits: 8192 x 4096 bf16 in 20 to 22 us (101 MB, 4.6 to 5.0 TB/s).
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

// 16 or 4 bytes of every lane's address, one lane's after the other's, to a place in LDS (no register takes the data).
// Of the builtins for it the compiler waits for all before the next read of LDS, the step's own among them, whatever part
// of LDS is read; these are waited for by wait_barrier alone.
__device__ __forceinline__ uint32_t lds_place(const void* p) {
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p);
}
__device__ __forceinline__ void to_lds16(const void* from, const void* to) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "s"(lds_place(to)) : "memory", "m0");
}
// The same at a row's end: zeros from the lanes that are past it.  (Each of a load's rows has 16 bytes at least, so the
// load goes out whatever the lanes: waits may count it.)
__device__ __forceinline__ void to_lds16_until(const void* from, i4* to, bool inside) {
    if (inside) to_lds16(from, to);
    else to[lane_id()] = i4(0);
}
__device__ __forceinline__ void to_lds4(const void* from, const void* to) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(from), "s"(lds_place(to)) : "memory", "m0");
}
// Few rows: bound by reading the weights once.  A workgroup takes 16 channels and 16 TT rows, its waves the k of a row in
// turns of 128 bytes -- whole lines of the weights -- and the waves' sums are added in LDS.  A wave's steps come by way of
// LDS of its own, a line by eight neighbouring lanes, so there is no barrier before the sums; loaded as the matrix
// instructions hold them, every lane's 16 bytes are a request of their own (64 x 4096 x 2048: 8.7 us, this way 5.3).
// DIRECT: rows aligned to 16 bytes and K a multiple of 16 go to LDS directly, two steps under way; others through
// registers, one step ahead.
constexpr int kFewWaves = 8, kFewStep = 128;
template <typename T, int TT, bool DIRECT>
__global__ __launch_bounds__(64 * kFewWaves) void mm8_few_kernel(Mm8Params p) {
    constexpr int ROWS = 16 + 16 * TT, LD = ROWS / 8;
    __shared__ __align__(16) i4 lds[kFewWaves][2][ROWS * 8];
    const int l = lane_id(), w = uniform(threadIdx.x >> 6), steps = (p.K + kFewStep - 1) / kFewStep;
    const int n0 = blockIdx.x * 16, t0 = blockIdx.y * 16 * TT;
    const int8_t* row[LD];
    int at[LD];   // the lane's byte of a step: chunk c of row r lies at c ^ r / 2 % 8
#pragma unroll
    for (int j = 0; j < LD; ++j) {
        const int r = 8 * j + l / 8;
        row[j] = j < 2 ? p.w + (int64_t)min(n0 + r, p.N - 1) * p.sw : p.x + (int64_t)min(t0 + r - 16, p.T - 1) * p.sx;
        at[j] = ((l % 8) ^ (r / 2 % 8)) * 16;
    }
    i4 held[LD];   // not DIRECT: the next step's
    auto load = [&](int k, int stage) {
        const int k0 = k * kFewStep;
#pragma unroll
        for (int j = 0; j < LD; ++j) {
            if (!DIRECT) held[j] = row_chunk(row[j], k0 + at[j], p.K);
            else if (k0 + kFewStep <= p.K) to_lds16(row[j] + k0 + at[j], &lds[w][stage][64 * j]);
            else to_lds16_until(row[j] + k0 + at[j], &lds[w][stage][64 * j], k0 + at[j] < p.K);
        }
    };
    i4 acc[TT];
#pragma unroll
    for (int i = 0; i < TT; ++i) acc[i] = i4(0);
    constexpr int AHEAD = DIRECT ? 2 * kFewWaves : kFewWaves;
    if (w < steps) load(w, 0);
    if (DIRECT && w + kFewWaves < steps) load(w + kFewWaves, 1);
    const int r = l % 16, sw = r / 2 % 8;
    int stage = 0;
    for (int k = w; k < steps; k += kFewWaves, stage ^= 1) {
        if (!DIRECT) {
#pragma unroll
            for (int j = 0; j < LD; ++j) lds[w][stage][64 * j + l] = held[j];
        } else if (k + kFewWaves < steps) {
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LD) : "memory");   // the next step may be under way
        } else {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
        if (!DIRECT && k + AHEAD < steps) load(k + AHEAD, stage);
        if (DIRECT) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // zeros past a row's end
        i4 a[2], b[2][TT];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const i4* const from = lds[w][stage] + r * 8 + ((4 * h + l / 16) ^ sw);
            a[h] = from[0];
#pragma unroll
            for (int i = 0; i < TT; ++i) b[h][i] = from[128 * (i + 1)];
        }
        if (DIRECT) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the stage is read
            if (k + AHEAD < steps) load(k + AHEAD, stage);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < TT; ++i) acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[h], b[h][i], acc[i], 0, 0, 0);
    }
    // wave i finishes the i-th 16 rows: lane l has row l % 16 and channels 4 (l / 16) ..
    i4* const part = lds[w][0];   // the wave's own: nothing is under way to it
#pragma unroll
    for (int i = 0; i < TT; ++i) part[64 * i + l] = acc[i];
    const int n = n0 + 4 * (l / 16);
    float scale[4], bias[4];
    if (w < TT) channels4(p, n, scale, bias);
    __syncthreads();
    if (w >= TT) return;
    i4 s(0);
#pragma unroll
    for (int v = 0; v < kFewWaves; ++v) s += lds[v][0][64 * w + l];
    finish4<T>(p, s, t0 + 16 * w + l % 16, n, scale, bias);
}

// What a tile's results are scaled with, in LDS (places past the last one: the last one's).
template <int BN, int BT> struct Scales {
    float w[BN], bias[BN], x[BT];
};

// A wave's MN x MT tiles of sums, from channel n0 + wn and row t0 + wt on: lane l has row l % 32 of a tile and four times
// four consecutive channels.  Where all of them are places of y they go by way of LDS, 32 rows at a time and up to 256
// bytes of each, and out in whole lines: stored from where they are, 8 bytes to each of 32 rows, they took 104 of
// 371 us (8192 x 4096 x 8192, bf16).  Returns whether they did.
template <typename T, bool WHOLE, int MN, int MT, int BN, int BT>
__device__ __forceinline__ void finish_wave(const Mm8Params& p, const i16v (&acc)[MN][MT], int n0, int t0, int wn, int wt,
                                            const Scales<BN, BT>& sc, i4* lds) {
    constexpr int E = 16 / (int)sizeof(T), IW = MN * 32 < 16 * E ? MN : 16 * E / 32, NC = IW * 32 / E;
    const int l = lane_id(), t = l % 32, q = l / 32;
#pragma unroll
    for (int j = 0; j < MT; ++j) {
        const int row = t0 + wt + 32 * j;
        const float sx = sc.x[wt + 32 * j + t];
#pragma unroll
        for (int i0 = 0; i0 < MN; i0 += IW) {
#pragma unroll
            for (int i = i0; i < i0 + IW; ++i)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int n = 32 * i + 8 * g + 4 * q;
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] = fmaf((float)acc[i][j][4 * g + e], sx * sc.w[wn + n + e], sc.bias[wn + n + e]);
                    if (WHOLE) {   // chunk c of a row of NC lies at c ^ row % NC
                        const int in = n - 32 * i0, c = in / E;
                        put4<T>((T*)(lds + t * NC + (c ^ (t % NC))) + in % E, v, 4);
                    } else if (row + t < p.T) {
                        put4<T>((T*)p.y + (int64_t)(row + t) * p.sy + n0 + wn + n, v, p.N - n0 - wn - n);
                    }
                }
            if (WHOLE) {
#pragma unroll
                for (int k = 0; k < NC / 2; ++k) {
                    const int u = (64 * k + l) / NC, c = l % NC;
                    const i4 o = lds[u * NC + (c ^ (u % NC))];
                    typedef int i4e __attribute__((ext_vector_type(4), aligned(2)));
                    *reinterpret_cast<i4e*>((T*)p.y + (int64_t)(row + u) * p.sy + n0 + wn + 32 * i0 + c * E) = o;
                }
            }
            __builtin_amdgcn_sched_barrier(0);   // not all of it at once: the sums fill the registers
        }
    }
}
template <typename T, int MN, int MT, int BN, int BT>
__device__ __forceinline__ bool finish_tiles(const Mm8Params& p, const i16v (&acc)[MN][MT], int n0, int t0, int wn, int wt,
                                             const Scales<BN, BT>& sc, i4* lds) {
    const bool whole = n0 + wn + 32 * MN <= p.N && t0 + wt + 32 * MT <= p.T;
    if (whole) finish_wave<T, true>(p, acc, n0, t0, wn, wt, sc, lds);
    else finish_wave<T, false>(p, acc, n0, t0, wn, wt, sc, lds);
    return whole;
}
// A workgroup's tile: the workgroups of an XCD (every eighth one) take neighbouring tiles, in patches of up to eight
// tiles of rows by as many of channels as come next, so that what they read at a time is in its L2.
__device__ __forceinline__ int2 tile_of(int id, int nblocks, int tblocks) {
    const int total = nblocks * tblocks, per = total / 8, rest = total % 8, xcd = id % 8;
    const int i = xcd * per + min(xcd, rest) + id / 8;   // the first `rest` XCDs have one tile more
    const int rows = 8, patch = rows * nblocks, t = i / patch * rows, in = i % patch, h = min(rows, tblocks - t);
    return {in / h, t + in % h};
}

// Many rows: a workgroup takes BN channels and BT rows, 128 bytes of k at a time through LDS, WN x WT waves of 32 x 32
// tiles each.  A row's eight 16-byte chunks lie in LDS at places exchanged by half the row's number (chunk c of row r
// at c ^ r / 2 % 8): the 16 lanes that are read together, a chunk of 16 rows, meet all 64 banks.
constexpr int kStep = 128;
template <typename T, int BN, int BT, int WN, int WT>
__global__ __launch_bounds__(64 * WN * WT) void mm8_tile_kernel(Mm8Params p, int nblocks) {
    constexpr int TH = 64 * WN * WT, CH = (BN + BT) * 8 / TH, MN = BN / WN / 32, MT = BT / WT / 32;
    __shared__ __align__(16) i4 lds[(BN + BT) * 8];
    __shared__ Scales<BN, BT> sc;
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
    const int put = (threadIdx.x / 8) * 8 + (c ^ (threadIdx.x / 16) % 8);   // TH / 8 is a multiple of 16
    for (int i = threadIdx.x; i < BN; i += TH) {
        sc.w[i] = p.ws[min(n0 + i, p.N - 1)];
        sc.bias[i] = p.bias ? p.bias[min(n0 + i, p.N - 1)] : 0.0f;
    }
    for (int i = threadIdx.x; i < BT; i += TH) sc.x[i] = p.xs[min(t0 + i, p.T - 1)];
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
            const int ch = (2 * s + l / 32) ^ (l / 2 % 8);
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
    __syncthreads();
    finish_tiles<T, MN, MT>(p, acc, n0, t0, wn, wt, sc, lds + wave * ((BN + BT) * 8 / (WN * WT)));
}

// Many rows whose starts are aligned to 16 bytes and K a multiple of 16: the same with loads that go from memory to
// LDS directly, a step ahead of the products, and one barrier a step.  A workgroup
// goes on from tile to tile: the next tile's first step comes while a tile's results go out.
constexpr int kDirectStep = 128;
// The wave's memory accesses but the last N, and its LDS accesses, are done, then the workgroup's.
template <int N = 0> __device__ __forceinline__ void wait_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}
template <typename T, int BN, int BT, int WN, int WT>
__global__ __launch_bounds__(64 * WN * WT) void mm8_direct_kernel(Mm8Params p, int nblocks, int tblocks) {
    constexpr int W = WN * WT, MN = BN / WN / 32, MT = BT / WT / 32;
    constexpr int ROWS = BN + BT, LD = ROWS / 8 / W;   // loads of a wave, 8 rows each
    static_assert(BN % (8 * LD) == 0, "a wave's loads are of one operand");
    static_assert(BN / 64 + BT / 64 <= W, "a wave loads 64 scales");
    __shared__ __align__(16) i4 lds[2][ROWS * 8];
    __shared__ __align__(16) Scales<BN, BT> scales[2];
    const int l = lane_id(), wave = uniform(threadIdx.x >> 6), total = nblocks * tblocks;
    const int wn = (wave % WN) * (BN / WN), wt = (wave / WN) * (BT / WT);
    const int r0 = wave * LD * 8;   // the wave's first row of a step
    const bool of_w = r0 < BN;
    const int last = (of_w ? p.N : p.T) - 1;
    const int64_t stride = of_w ? p.sw : p.sx;
    const int8_t* src;
    uint32_t off[LD];
    int n0, t0, first;
    const int steps = (p.K + kDirectStep - 1) / kDirectStep;
    const bool ragged = p.K % kDirectStep != 0;
    auto load = [&](int k, int j0, int j1) {
#pragma unroll
        for (int j = j0; j < j1; ++j) to_lds16(src + (int64_t)k * kDirectStep + off[j], &lds[k & 1][(r0 + 8 * j) * 8]);
    };
    auto load_last = [&]() {   // the last step, where the row ends inside of it
        const int k = steps - 1, left = p.K - k * kDirectStep;
#pragma unroll 1
        for (int j = 0; j < LD; ++j) {
            const int r = 8 * j + l / 8, c = (l % 8) ^ ((r0 + r) / 2 % 8);
            to_lds16_until(src + (int64_t)k * kDirectStep + 16 * c + (int64_t)(max(0, min(first + r, last) - min(first, last))) * stride,
                           &lds[k & 1][(r0 + 8 * j) * 8], 16 * c < left);
        }
    };
    // tile `id`, its scales and its first step
    auto begin = [&](int id, Scales<BN, BT>& sc) {
        const int2 tile = tile_of(id, nblocks, tblocks);
        n0 = tile.x * BN;
        t0 = tile.y * BT;
        first = of_w ? n0 + r0 : t0 + r0 - BN;
        src = (of_w ? p.w : p.x) + min(first, last) * stride;
#pragma unroll
        for (int j = 0; j < LD; ++j) {
            const int r = 8 * j + l / 8;   // of the wave's rows; those past the operand's last one repeat it
            off[j] = (uint32_t)(max(0, min(first + r, last) - min(first, last)) * stride) + (((l % 8) ^ ((r0 + r) / 2 % 8)) * 16);
        }
        if (wave < BN / 64) {
            const int n = min(n0 + 64 * wave + l, p.N - 1);
            to_lds4(p.ws + n, &sc.w[64 * wave]);
            if (p.bias) to_lds4(p.bias + n, &sc.bias[64 * wave]);
        } else if (wave < BN / 64 + BT / 64) {
            const int at = 64 * (wave - BN / 64);
            to_lds4(p.xs + min(t0 + at + l, p.T - 1), &sc.x[at]);
        }
        if (steps > 1 || !ragged) load(0, 0, LD);
        else load_last();
    };
    const int fa = (wn + l % 32) * 8, fb = (BN + wt + l % 32) * 8, sw = l / 2 % 8;
    i4 a[2][MN], b[2][MT];   // of two quarters of a step
    i16v acc[MN][MT];
    auto fragments = [&](int k, int s) {
        const i4* const at = lds[k & 1] + ((2 * s + l / 32) ^ sw);
#pragma unroll
        for (int i = 0; i < MN; ++i) a[s & 1][i] = at[fa + 256 * i];
#pragma unroll
        for (int j = 0; j < MT; ++j) b[s & 1][j] = at[fb + 256 * j];
        __builtin_amdgcn_sched_barrier(0);
    };
    auto products = [&](int s, int i0, int i1) {
#pragma unroll
        for (int i = i0; i < i1; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[s & 1][i], b[s & 1][j], acc[i][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    };
    // A quarter's products run while the next quarter's operands are read, the first few before the reads so that what
    // they wait for is behind them already; the next step's loads go out between those of the first quarter.
    // next: 0 none, 1 a whole step, 2 the last one
    auto step = [&](int k, int next) {
#pragma unroll
        for (int s = 0; s < 3; ++s) {
            products(s, 0, 1);
            fragments(k, s + 1);
            if (MN == 1 && s == 0 && next == 1) load(k + 1, 0, LD);
            if (s == 0 && next == 2) load_last();
#pragma unroll
            for (int i = 1; i < MN; ++i) {
                if (s == 0 && next == 1) load(k + 1, LD * (i - 1) / (MN - 1), LD * i / (MN - 1));
                products(s, i, i + 1);
            }
        }
        products(3, 0, 1);
        wait_barrier();   // step k + 1 has come, and every wave has read step k
        products(3, 1, MN / 2 + 1);
        if (next) fragments(k + 1, 0);
        products(3, MN / 2 + 1, MN);
    };
    int buf = 0;
    for (int i = threadIdx.x; !p.bias && i < BN; i += 64 * W) scales[0].bias[i] = scales[1].bias[i] = 0.0f;
    begin(blockIdx.x, scales[0]);
    wait_barrier();
    for (int id = blockIdx.x;; buf ^= 1) {
#pragma unroll
        for (int i = 0; i < MN; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j) acc[i][j] = i16v(0);
        fragments(0, 0);
        for (int k = 0; k + 1 + ragged < steps; ++k) step(k, 1);
        if (ragged && steps > 1) step(steps - 2, 2);
        step(steps - 1, 0);
        // The next tile's first step comes while this one's results go out, by way of the other stage.
        const int n = n0, t = t0;
        id += gridDim.x;
        if (id < total) begin(id, scales[buf ^ 1]);
        const bool whole = finish_tiles<T, MN, MT>(p, acc, n, t, wn, wt, scales[buf], lds[1] + wave * (ROWS * 8 / W));
        if (id >= total) break;
        if (whole) wait_barrier<MN * MT * (int)sizeof(T)>();   // its stores may be under way: 16 bytes of 64 lanes each
        else wait_barrier();
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
    if (p.tile == 0) {
        const int few = (p.T + 15) / 16;
        const dim3 grid((p.N + 15) / 16, few == 1 ? 1 : (few + 1) / 2);
        if (few == 1 && p.direct) mm8_few_kernel<T, 1, true><<<grid, 64 * kFewWaves, 0, st>>>(p);
        else if (few == 1) mm8_few_kernel<T, 1, false><<<grid, 64 * kFewWaves, 0, st>>>(p);
        else if (p.direct) mm8_few_kernel<T, 2, true><<<grid, 64 * kFewWaves, 0, st>>>(p);
        else mm8_few_kernel<T, 2, false><<<grid, 64 * kFewWaves, 0, st>>>(p);
    } else {
        const int nb = (p.N + p.tile - 1) / p.tile, tb = (p.T + p.tile - 1) / p.tile;
        const unsigned blocks = (unsigned)nb * (unsigned)tb;
        // as many workgroups as the 256 CUs hold at a time: one, two or four by their LDS (137, 69 and 34 KB of 160)
        if (p.direct && p.tile == 256)
            mm8_direct_kernel<T, 256, 256, 2, 4><<<std::min(blocks, 256u), 512, 0, st>>>(p, nb, tb);
        else if (p.direct && p.tile == 128)
            mm8_direct_kernel<T, 128, 128, 2, 2><<<std::min(blocks, 512u), 256, 0, st>>>(p, nb, tb);
        else if (p.direct)
            mm8_direct_kernel<T, 64, 64, 2, 2><<<std::min(blocks, 1024u), 256, 0, st>>>(p, nb, tb);
        else if (p.tile == 64) mm8_tile_kernel<T, 64, 64, 2, 2><<<blocks, 256, 0, st>>>(p, nb);
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
