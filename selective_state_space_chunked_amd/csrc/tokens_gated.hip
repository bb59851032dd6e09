// The gated linear recurrence (gated.hpp) over packed rows, with a pool of states.
//
// Prompts, in one pass.  A workgroup takes a tile of 128 rows and 64 lanes' channels, each of its eight waves 16 of the
// rows: the streams are read once, along the channels as the projections write them, and what the gates make of them,
// a and b of h <- a h + b, stays in registers.  Where a sequence begins, its first state goes into b and
// nothing comes in from the row before, nor does it where no sequence owns a row: so from there on the rows are one
// recurrence, whatever the sequences' lengths.
// Waves compose their rows' maps, the workgroup its waves' through LDS, and tiles theirs through memory: a tile leaves
// the map of its rows as soon as it has it (for each channel one word of 64 bits, so that no reader sees half of it), the
// state at its end as soon as it knows that, and goes back to the last tile whose state is there and from it
// through the maps, so that every state is the same function of the rows whatever is there when.  The tiles of the same
// channels are taken in the order of a counter, so a workgroup waits only for ones that run already, and for
// nothing that these wait for; all the same the wait is bounded, and gives NaN where the bound is reached.
//
// 8192 rows of 4096 channels in 13 sequences, bf16, 280 MB, take 80 us (3.5 TB/s), of which the gates' 39 instructions an
// element issue for 46 %: reading, the gates and the wait for the rows before it follow each other in a tile and are
// hidden by the other tiles of a CU only in part.  A plan before it takes 3 to 6 us, a launch and the words' clearing.
// Two passes over ranges of rows, as the selective scan makes, formed the gates twice: 116 us.  Eight waves of eight
// rows took 91 us, four of 16 rows 82, 16 of eight rows 97, when this form took 75 (before it went forward through the
// maps): a tile has less under way then, or more waves to compose.
//
// Single tokens: a row a sequence, four channels a lane; 64 places of 2048 channels 4.1 us, a launch and its loads' latency.
#include <algorithm>

#include "gated.hpp"

namespace ssm {
namespace {

constexpr int kTileWaves = 8, kWaveRows = kGatedTile / kTileWaves;
constexpr uint32_t kNone = 0xffffffffu;   // a word that is not there yet; of the NaNs that a state may be, not one
constexpr int kPolls = 1 << 16;           // a tenth of a second and more

__device__ __forceinline__ uint32_t word_of(float v) {
    const uint32_t u = __float_as_uint(v);
    return u == kNone ? 0x7fc00000u : u;
}
template <typename W> __device__ __forceinline__ void put_word(W* p, W v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename W> __device__ __forceinline__ W get_word(const W* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Before the tiles: no words, no tiles taken, and each sequence's slot, or -1 for an empty place.
__global__ __launch_bounds__(256) void tok_gated_plan_kernel(TokGatedParams p, int64_t words) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, all = (int64_t)gridDim.x * 256;
    for (int64_t i = id; i < words; i += all) p.maps[i] = ~0ull;
    for (int64_t i = id; i < p.columns; i += all) p.ticket[i] = 0;
    for (int64_t s = id / 64; s < p.q.S; s += all / 64) {
        const int v = slot_of(p.q, (int)s);
        if (lane_id() == 0) p.slots[s] = v;
    }
}

// Two channels of bf16 or one of fp32, so that a wave reads 256 bytes of a row.  EVEN: the lane's channels are all channels of
// the layer, or, past the last one, the last ones again, whose results go nowhere; otherwise one by one.
template <typename T> struct Few;
template <> struct Few<bf16_t> {
    static constexpr int V = kGatedFew<1>;
    typedef uint32_t raw __attribute__((aligned(2)));
    uint32_t r;
    template <bool EVEN> __device__ __forceinline__ void load(const bf16_t* row, int d, int D) {
        if (EVEN) r = *reinterpret_cast<const raw*>(row + d);
        else r = (uint32_t)row[min(d, D - 1)] | (uint32_t)row[min(d + 1, D - 1)] << 16;
    }
    __device__ __forceinline__ float get(int e) const { return __uint_as_float(e ? r & 0xffff0000u : r << 16); }
    template <bool EVEN> __device__ __forceinline__ static void store(bf16_t* row, int d, int n, const float (&v)[2]) {
        if (EVEN) {
            if (n > 0) *reinterpret_cast<raw*>(row + d) = (uint32_t)to_stream<bf16_t>(v[0]) | (uint32_t)to_stream<bf16_t>(v[1]) << 16;
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (e < n) row[d + e] = to_stream<bf16_t>(v[e]);
        }
    }
};
template <> struct Few<float> {
    static constexpr int V = kGatedFew<0>;
    float r;
    template <bool EVEN> __device__ __forceinline__ void load(const float* row, int d, int D) { r = row[min(d, D - 1)]; }
    __device__ __forceinline__ float get(int) const { return r; }
    template <bool EVEN> __device__ __forceinline__ static void store(float* row, int d, int n, const float (&v)[1]) {
        if (n > 0) row[d] = v[0];
    }
};

// What a wave's rows are, in lane j that of row j: the slot of the sequence that owns it (-1: none), whether the row is
// its first one, its last one, and whether it begins with zeros.
struct RowInfo {
    int slot = -1, first = 0, last = 0, fresh = 0;
    RowInfo() = default;
    __device__ __forceinline__ RowInfo(const TokGatedParams& p, const SeqTable& q, int r0) {
        const int t = r0 + lane_id(), end = min(r0 + kWaveRows, p.q.T);
        int s = max(q.find(r0), 0);
        for (; s < p.q.S; ++s) {
            const int st = q.first(s);
            if (st >= end) break;
            const int en = q.end(s);
            if (st < 0 || en <= max(st, r0)) continue;
            int v = uniform(p.slots[s]);
            if (v >= p.q.slots) v = -1;   // (only in a workspace that another call has written to meanwhile)
            const bool f = q.fresh(s);
            if (t >= st && t < min(en, end)) {
                slot = v;
                first = t == st;
                last = t == en - 1;
                fresh = f;
            }
        }
    }
};

// The waves' maps, whether a wave's map forgets what comes in, and the state that comes into the tile.
template <int V> struct TileMaps {
    float P[kTileWaves][64 * V], S[kTileWaves][64 * V], carry[64 * V];
    int cut[kTileWaves];
};

template <typename T, bool EVEN, bool SLOW>
__device__ __forceinline__ void gated_tile(const TokGatedParams& p, int tile, int d0, const GateChannel (&c)[Few<T>::V],
                                           const SeqTable& seqs, TileMaps<Few<T>::V>& maps) {
    constexpr int V = Few<T>::V, R = kWaveRows;
    const int l = lane_id(), w = uniform(threadIdx.x >> 6), r0 = tile * kGatedTile + w * R;
    const int d = d0 + V * l, at = EVEN ? min(d, p.D - V) : d, n = max(0, min(V, p.D - d));
    float a[R][V], b[R][V];
    RowInfo info;
    {
        Few<T> x[R], r[R], g[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const int t = min(r0 + j, p.q.T - 1);
            x[j].template load<EVEN>((const T*)p.x + t * p.sx, at, p.D);
            r[j].template load<EVEN>((const T*)p.r + t * p.sr, at, p.D);
            g[j].template load<EVEN>((const T*)p.i + t * p.si, at, p.D);
        }
        info = RowInfo(p, seqs, r0);   // while the rows come
#pragma unroll
        for (int j = 0; j < R; ++j) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float v = gate_rest<SLOW>(c[e].rate * gate_open(r[j].get(e), c[e].rb), a[j][e]);
                b[j][e] = __builtin_amdgcn_sqrtf(v) * (gate_open(g[j].get(e), c[e].ib) * x[j].get(e));
            }
        }
    }
    // cut: rows that nothing comes into from the row before.  They are chosen, not multiplied by 0: a sequence's NaN or
    // infinity stays its own.
    const uint32_t owned = (uint32_t)__ballot(info.slot >= 0), first = (uint32_t)__ballot(info.first != 0) & owned;
    const uint32_t cut = first | (~owned & ((1u << R) - 1));
    if (cut) {
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if (!(owned >> j & 1)) {
#pragma unroll
                for (int e = 0; e < V; ++e) b[j][e] = 0.0f;
            } else if (first >> j & 1) {
                const float* const h0 = p.pool + __builtin_amdgcn_readlane(info.slot, j) * p.spool;
                if (!__builtin_amdgcn_readlane(info.fresh, j)) {
#pragma unroll
                    for (int e = 0; e < V; ++e) b[j][e] = fmaf(a[j][e], h0[min(d + e, p.D - 1)], b[j][e]);
                }
            }
        }
    }
    float P[V], S[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        P[e] = a[0][e];
        S[e] = b[0][e];
#pragma unroll
        for (int j = 1; j < R; ++j) {
            S[e] = cut >> j & 1 ? b[j][e] : fmaf(a[j][e], S[e], b[j][e]);
            P[e] *= a[j][e];
        }
        maps.P[w][V * l + e] = P[e];
        maps.S[w][V * l + e] = S[e];
    }
    if (l == 0) maps.cut[w] = cut != 0;
    __syncthreads();
    // the map of the rows of the workgroup before the wave's own; the first wave: of all, for the tiles behind
    bool forgets = false;   // nothing comes through: S is a state
#pragma unroll
    for (int e = 0; e < V; ++e) {
        P[e] = 1.0f;
        S[e] = 0.0f;
    }
    for (int k = 0; k < (w ? w : kTileWaves); ++k) {
        const bool c = uniform(maps.cut[k]) != 0;
        forgets |= c;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float m = maps.P[k][V * l + e], v = maps.S[k][V * l + e];
            S[e] = c ? v : fmaf(m, S[e], v);
            P[e] *= m;
        }
    }
    if (w == 0) {
        uint64_t* const map = p.maps + (int64_t)tile * p.D;
        uint32_t* const state = (uint32_t*)(p.maps + (int64_t)p.tiles * p.D) + (int64_t)tile * p.D;
        float C[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            C[e] = 0.0f;
            if (e < n) {   // (into the first tile nothing comes)
                if (tile == 0 || forgets) put_word(state + d + e, word_of(S[e]));
                else put_word(map + d + e, (uint64_t)word_of(S[e]) << 32 | word_of(P[e]));
            }
        }
        if (tile > 0 && !(cut & 1)) {   // otherwise no row takes what comes in
            // Back to the last tile before this one whose state is known, with all maps between there, eight tiles' words
            // under way together.
            constexpr int AHEAD = 8;
            const auto place = [&](int k, int e) { return (int64_t)(max(k, 0) - tile) * p.D + min(d + e, p.D - 1); };
            int k = tile - 1, polls = 0;
            for (bool found = false; !found;) {
                uint32_t h[AHEAD][V], m[AHEAD][V];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        h[i][e] = get_word(state + place(k - i, e));
                        m[i][e] = get_word((const uint32_t*)(map + place(k - i, e)));   // half of a map: all of it is there
                    }
                bool wait = false;
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    bool nostate = false, nomap = false;
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        nostate |= h[i][e] == kNone;
                        nomap |= m[i][e] == kNone;
                    }
                    if (found || wait) continue;
                    if (!__ballot(nostate)) found = true;
                    else if (k <= 0 || __ballot(nomap)) wait = true;   // (before the first tile there is none)
                    else --k;
                }
                if (wait) {
                    if (++polls > kPolls) break;
                    __builtin_amdgcn_s_sleep(1);
                } else {
                    polls = 0;
                }
            }
            // From there on through the maps: the same products and sums whichever tile it is, so the same bits.
#pragma unroll
            for (int e = 0; e < V; ++e) C[e] = polls > kPolls ? __uint_as_float(0x7fc00000u) : __uint_as_float(get_word(state + place(k, e)));
            while (++k < tile) {
                uint64_t m[AHEAD][V];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i)
#pragma unroll
                    for (int e = 0; e < V; ++e) m[i][e] = get_word(map + place(min(k + i, tile - 1), e));
#pragma unroll
                for (int i = 0; i < AHEAD; ++i)
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (k + i < tile)
                            C[e] = fmaf(__uint_as_float((uint32_t)m[i][e]), C[e], __uint_as_float((uint32_t)(m[i][e] >> 32)));
                k += AHEAD - 1;
            }
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (e < n && !forgets) put_word(state + d + e, word_of(fmaf(P[e], C[e], S[e])));
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            maps.carry[V * l + e] = C[e];
            P[e] = 1.0f;
            S[e] = 0.0f;
        }
    }
    __syncthreads();
    // the state that the wave's rows begin with
    float h[V];
    const bool through = w == 0 || !forgets;
#pragma unroll
    for (int e = 0; e < V; ++e) h[e] = through ? fmaf(P[e], maps.carry[V * l + e], S[e]) : S[e];
    const uint32_t last = (uint32_t)__ballot(info.last != 0) & owned;
#pragma unroll
    for (int j = 0; j < R; ++j) {
#pragma unroll
        for (int e = 0; e < V; ++e) h[e] = cut >> j & 1 ? b[j][e] : fmaf(a[j][e], h[e], b[j][e]);
        if (owned >> j & 1) Few<T>::template store<EVEN>((T*)p.y + (r0 + j) * p.sy, at, n, h);
        if (last >> j & 1) {
            float* const pool = p.pool + __builtin_amdgcn_readlane(info.slot, j) * p.spool;
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (e < n) pool[d + e] = h[e];
        }
    }
}
template <typename T>
__global__ __launch_bounds__(64 * kTileWaves, 4) void tok_gated_kernel(TokGatedParams p) {
    constexpr int V = Few<T>::V;
    __shared__ TileMaps<V> maps;
    __shared__ int taken;
    const int column = blockIdx.x % p.columns, d0 = column * 64 * V;
    const SeqTable seqs(p.q);
    if (threadIdx.x == 0) taken = __hip_atomic_fetch_add(p.ticket + column, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    GateChannel c[V];
    bool fast = false;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        c[e] = gate_channel(p.lam, p.rb, p.ib, p.power, min(d0 + V * lane_id() + e, p.D - 1));
        fast |= !(c[e].rate < kGateSlow);
    }
    const bool slow = __ballot(fast) == 0, even = p.D % V == 0 || d0 + 64 * V <= p.D;
    __syncthreads();
    const int tile = uniform(taken);
    if (tile < 0 || tile >= p.tiles) return;   // (as above)
    if (even && slow) gated_tile<T, true, true>(p, tile, d0, c, seqs, maps);
    else if (even) gated_tile<T, true, false>(p, tile, d0, c, seqs, maps);
    else gated_tile<T, false, false>(p, tile, d0, c, seqs, maps);
}

constexpr int kCh = 4;    // channels of a lane of the step kernel

// One row a sequence.  EVEN: as above, of four channels a lane.
template <typename T, bool EVEN>
__device__ __forceinline__ void step_row(const TokGatedParams& p, int s, int slot, int d0) {
    const bool live = d0 < p.D;
    const int n = max(0, min(kCh, p.D - d0)), d = EVEN ? min(d0, p.D - kCh) : min(d0, p.D - 1);
    float* const pool = p.pool + slot * p.spool + d;
    const T* const rows[3] = {(const T*)p.x + s * p.sx + d, (const T*)p.r + s * p.sr + d, (const T*)p.i + s * p.si + d};
    Vec<T> v[3];
    Vec<float> st;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        if (EVEN) v[k].load(rows[k]);
        else v[k].load(rows[k], n);
    }
    if (EVEN) st.load(pool);
    else st.load(pool, n);
    const bool fresh = p.q.fresh && p.q.fresh[s];
    GateChannel c[kCh];
#pragma unroll
    for (int e = 0; e < kCh; ++e) c[e] = gate_channel(p.lam, p.rb, p.ib, p.power, min(d + e, p.D - 1));
    if (slot_taken(p.q, s, slot)) return;
    float x[kCh], r[kCh], g[kCh], h[kCh];
    v[0].get(x);
    v[1].get(r);
    v[2].get(g);
    st.get(h);
#pragma unroll
    for (int e = 0; e < kCh; ++e) {
        float a;
        const float rest = gate_rest<false>(c[e].rate * gate_open(r[e], c[e].rb), a);
        const float b = __builtin_amdgcn_sqrtf(rest) * (gate_open(g[e], c[e].ib) * x[e]);
        h[e] = fresh ? b : fmaf(a, h[e], b);
    }
    Vec<T> o;
    o.set(h);
    st.set(h);
    T* const y = (T*)p.y + s * p.sy + d;
    if (EVEN) {
        if (live) {
            o.store(y);
            st.store(pool);
        }
    } else {
        o.store(y, n);
        st.store(pool, n);
    }
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

hipError_t launch_tok_gated_plan(const TokGatedParams& p, hipStream_t st) {
    const int64_t words = (int64_t)p.tiles * p.D + ((int64_t)p.tiles * p.D + 1) / 2;
    const int64_t blocks = std::max<int64_t>((words + 511) / 512, (p.q.S + 3) / 4);
    tok_gated_plan_kernel<<<(unsigned)std::min<int64_t>(blocks, 4096), 256, 0, st>>>(p, words);
    return hipGetLastError();
}
hipError_t launch_tok_gated(const TokGatedParams& p, int dtype, hipStream_t st) {
    const unsigned blocks = (unsigned)p.columns * (unsigned)p.tiles;
    if (dtype) tok_gated_kernel<bf16_t><<<blocks, 64 * kTileWaves, 0, st>>>(p);
    else tok_gated_kernel<float><<<blocks, 64 * kTileWaves, 0, st>>>(p);
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
