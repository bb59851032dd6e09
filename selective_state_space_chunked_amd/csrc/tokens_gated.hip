// The gated linear recurrence (gated.hpp) over packed rows, with a pool of states.
//
// Prompts, in one pass.  A workgroup takes a tile of 128 rows and 64 channels, each of its eight waves 16 of the
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
// 8192 rows of 4096 channels in 13 sequences, bf16, 276 MB, take 74 us (3.7 TB/s), of which the gates' 41 instructions an
// element issue for 53 %: reading, the gates and the wait for the rows before it follow each other in a tile and are
// hidden by the other tiles of a CU only in part.  A lane has one channel, so three workgroups fit a CU (two channels of
// bf16: two workgroups, 80 us).  Tiles by four waves take 82, by 16 waves of 16 rows 95, of eight rows 124, by eight waves
// of eight rows 100: fewer rows are under way for each wait, or more maps to compose.  Two passes over ranges of rows,
// as the selective scan makes, formed the gates twice: 116 us.  The plan before it takes 3 to 5 us, a launch and
// the words' clearing.
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
struct TileMaps {
    float P[kTileWaves][64], S[kTileWaves][64], carry[64];
    int cut[kTileWaves];
};

// A lane has one channel d, or, past the last one, the last one again, whose results go nowhere.
template <typename T, bool SLOW>
__device__ __forceinline__ void gated_tile(const TokGatedParams& p, int tile, int d, bool live, const GateChannel& c,
                                           const SeqTable& seqs, TileMaps& maps) {
    constexpr int R = kWaveRows;
    const int l = lane_id(), w = uniform(threadIdx.x >> 6), r0 = tile * kGatedTile + w * R;
    float a[R], b[R];
    RowInfo info;
    {
        T x[R], r[R], g[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const int t = min(r0 + j, p.q.T - 1);
            x[j] = ((const T*)p.x + t * p.sx)[d];
            r[j] = ((const T*)p.r + t * p.sr)[d];
            g[j] = ((const T*)p.i + t * p.si)[d];
        }
        info = RowInfo(p, seqs, r0);   // while the rows come
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const float v = gate_rest<SLOW>(c.rate * gate_open(to_f32(r[j]), c.rb), a[j]);
            b[j] = __builtin_amdgcn_sqrtf(v) * (gate_open(to_f32(g[j]), c.ib) * to_f32(x[j]));
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
                b[j] = 0.0f;
            } else if (first >> j & 1) {
                const float* const h0 = p.pool + __builtin_amdgcn_readlane(info.slot, j) * p.spool;
                if (!__builtin_amdgcn_readlane(info.fresh, j)) b[j] = fmaf(a[j], h0[d], b[j]);
            }
        }
    }
    float P = a[0], S = b[0];
#pragma unroll
    for (int j = 1; j < R; ++j) {
        S = cut >> j & 1 ? b[j] : fmaf(a[j], S, b[j]);
        P *= a[j];
    }
    maps.P[w][l] = P;
    maps.S[w][l] = S;
    if (l == 0) maps.cut[w] = cut != 0;
    __syncthreads();
    // the map of the rows of the workgroup before the wave's own; the first wave: of all, for the tiles behind
    bool forgets = false;   // nothing comes through: S is a state
    P = 1.0f;
    S = 0.0f;
    for (int k = 0; k < (w ? w : kTileWaves); ++k) {
        const bool c = uniform(maps.cut[k]) != 0;
        forgets |= c;
        const float m = maps.P[k][l], v = maps.S[k][l];
        S = c ? v : fmaf(m, S, v);
        P *= m;
    }
    if (w == 0) {
        uint64_t* const map = p.maps + (int64_t)tile * p.D + d;
        uint32_t* const state = (uint32_t*)(p.maps + (int64_t)p.tiles * p.D) + (int64_t)tile * p.D + d;
        float C = 0.0f;
        if (live) {   // (into the first tile nothing comes)
            if (tile == 0 || forgets) put_word(state, word_of(S));
            else put_word(map, (uint64_t)word_of(S) << 32 | word_of(P));
        }
        if (tile > 0 && !(cut & 1)) {   // otherwise no row takes what comes in
            // Back to the last tile before this one whose state is known, with all maps between there, eight tiles' words
            // under way together.
            constexpr int AHEAD = 8;
            const auto place = [&](int k) { return (int64_t)(max(k, 0) - tile) * p.D; };
            int k = tile - 1, polls = 0;
            for (bool found = false; !found;) {
                uint32_t h[AHEAD], m[AHEAD];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    h[i] = get_word(state + place(k - i));
                    m[i] = get_word((const uint32_t*)(map + place(k - i)));   // half of a map: all of it is there
                }
                bool wait = false;
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    if (found || wait) continue;
                    if (!__ballot(h[i] == kNone)) found = true;
                    else if (k <= 0 || __ballot(m[i] == kNone)) wait = true;   // (before the first tile there is none)
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
            C = polls > kPolls ? __uint_as_float(0x7fc00000u) : __uint_as_float(get_word(state + place(k)));
            while (++k < tile) {
                uint64_t m[AHEAD];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) m[i] = get_word(map + place(min(k + i, tile - 1)));
#pragma unroll
                for (int i = 0; i < AHEAD; ++i)
                    if (k + i < tile)
                        C = fmaf(__uint_as_float((uint32_t)m[i]), C, __uint_as_float((uint32_t)(m[i] >> 32)));
                k += AHEAD - 1;
            }
            if (live && !forgets) put_word(state, word_of(fmaf(P, C, S)));
        }
        maps.carry[l] = C;
        P = 1.0f;
        S = 0.0f;
    }
    __syncthreads();
    // the state that the wave's rows begin with
    float h = w == 0 || !forgets ? fmaf(P, maps.carry[l], S) : S;
    const uint32_t last = (uint32_t)__ballot(info.last != 0) & owned;
#pragma unroll
    for (int j = 0; j < R; ++j) {
        h = cut >> j & 1 ? b[j] : fmaf(a[j], h, b[j]);
        if (live && (owned >> j & 1)) ((T*)p.y + (r0 + j) * p.sy)[d] = to_stream<T>(h);
        if (live && (last >> j & 1)) p.pool[__builtin_amdgcn_readlane(info.slot, j) * p.spool + d] = h;
    }
}
template <typename T>
__global__ __launch_bounds__(64 * kTileWaves, 6) void tok_gated_kernel(TokGatedParams p) {
    __shared__ TileMaps maps;
    __shared__ int taken;
    const int column = blockIdx.x % p.columns, d = column * 64 + lane_id();
    const SeqTable seqs(p.q);
    if (threadIdx.x == 0) taken = __hip_atomic_fetch_add(p.ticket + column, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const GateChannel c = gate_channel(p.lam, p.rb, p.ib, p.power, min(d, p.D - 1));
    const bool slow = __ballot(!(c.rate < kGateSlow)) == 0;
    __syncthreads();
    const int tile = uniform(taken);
    if (tile < 0 || tile >= p.tiles) return;   // (as above)
    if (slow) gated_tile<T, true>(p, tile, min(d, p.D - 1), d < p.D, c, seqs, maps);
    else gated_tile<T, false>(p, tile, min(d, p.D - 1), d < p.D, c, seqs, maps);
}

constexpr int kCh = 4;    // channels of a lane of the step kernel

// One row a sequence, four channels a lane.  EVEN: the lane's channels are all channels of the layer, or, past the last
// one, the last ones again, whose results go nowhere; otherwise one by one.
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
