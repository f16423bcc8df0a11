// gspn_seq.hip -- the gated linear recurrence over packed sequences.
//
//   a_t = sigmoid(gate_t),  h_t = a_t h_{t-1} + in_t,  in_t = lam_t x_t or (1 - a_t) x_t,
//   y_t = u_t h_t or h_t
//
// per channel of every sequence (include/gspn.h has the whole definition),
// its backward and its step for single tokens.
//
// A stretch of tokens maps the state in front of it to the state behind it by
// h -> A h + B, A the product of its gates, and two stretches join to
// (A2 A1, A2 B1 + B2).  So a sequence is cut into tiles of kSeqTile tokens
// that work side by side:
//  * a workgroup owns one tile of one block of channels (a lane owns V
//    neighbouring channels), a wave kTokens tokens of it, held in registers:
//    every input is read once;
//  * each wave forms its stretch's (A, B), the waves join theirs in LDS, and
//    the workgroup publishes the tile's;
//  * a tile that is not its sequence's first looks back over the tiles in front
//    of it to one that has published the state behind itself, goes from there
//    through the (A, B) of those between, and publishes its own state;
//  * with the state in front of its tokens, each wave finishes them.
// A tile never holds rows of two sequences, so nothing passes between them.
//
// Every wait ends: workgroups take their tile from a counter (one for each
// block of channels) and wait only for tiles of the same block with smaller
// numbers, and so only for workgroups that already run.  Each of those publishes
// its (A, B) before it waits, and its state when its own wait ends; the one with
// the smallest number, and whatever tile the offsets make the first of a
// sequence, waits for nobody.
#include "gspn_device.h"
#include "gspn_kernels.h"
#include "gspn_rows.h"

namespace gspn {
namespace {

constexpr int kTokens = 16;                   // tokens of a wave
constexpr int kWaves = kSeqTile / kTokens;    // waves of a workgroup

// ---------------------------------------------------------------- rows
// V neighbouring channels of a row as they are stored.
template <typename T, int V> struct Raw;
template <> struct Raw<uint16_t, 1> { using type = uint16_t; };
template <> struct Raw<uint16_t, 2> { using type = uint32_t; };
template <> struct Raw<float, 1> { using type = float; };

template <int V> __device__ __forceinline__ float channel(uint16_t r, int) { return to_f32(r); }
template <int V> __device__ __forceinline__ float channel(uint32_t r, int v) { return v ? bf16_hi(r) : bf16_lo(r); }
template <int V> __device__ __forceinline__ float channel(float r, int) { return r; }

__device__ __forceinline__ void put(uint16_t* p, const float (&v)[1]) { *p = from_f32(v[0], p); }
__device__ __forceinline__ void put(uint16_t* p, const float (&v)[2]) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(v[0], v[1]);
}
__device__ __forceinline__ void put(float* p, const float (&v)[1]) { *p = v[0]; }

// ---------------------------------------------------------------- gates
// A gate is held as one number that loses no precision for a near 0 or near 1:
// the smaller of a and 1 - a, negative (-0 included) where that is 1 - a.
__device__ __forceinline__ bool open(float s) { return (__float_as_uint(s) >> 31) != 0; }

__device__ __forceinline__ float gate_of(float g) {
    const float e = fast_exp2(fabsf(g) * -1.44269504088896340736f);
    const float small = e * fast_rcp(1.0f + e);
    return g >= 0.0f ? -small : small;   // (NaN stays NaN)
}
__device__ __forceinline__ float take(float s) { return open(s) ? -s : 1.0f - s; }   // 1 - a
constexpr float kKeepAll = -0.0f;                                                    // a = 1

// a h.  For a near 1 it is h - (1 - a) h: the rounding of such an a (2^-24 of h
// at every token) would add up over the gate's memory, 1 / (1 - a) tokens;
// that of 1 - a does not.
__device__ __forceinline__ float keep(float s, float h) { return fmaf(s, h, open(s) ? h : 0.0f); }

// ---------------------------------------------------------------- tiles' results
// What a tile tells the tiles behind it about one channel, in one 64-bit word
// that is written and read whole: nothing yet (all ones), its (A, B), or the
// state behind it (kState in the place of A, which is never negative).
constexpr uint64_t kNothing = ~0ull;
constexpr uint32_t kState = 0xbf800000u;

__device__ __forceinline__ void publish(uint64_t* p, uint32_t a, float b) {
    __hip_atomic_store(p, ((uint64_t)a << 32) | __float_as_uint(b), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint32_t product_bits(float a) {
    return a == a ? __float_as_uint(a) : 0x7fc00000u;   // a NaN must not look like kNothing
}
__device__ __forceinline__ uint64_t peek(const uint64_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The state that the `most` >= 1 tiles before this one (the words of tile i are
// `stride` further each, i = 1 the nearest; the furthest is the sequence's
// end) leave in front of it.  Every wave looks at one tile a round, kWaves tiles
// further each round, until for each channel one of them has said its state;
// from there the (A, B) of the nearer ones lead back, h -> A h + B one tile after
// the other.  That is the arithmetic by which those tiles get their own states, so
// the result does not depend on who was first.  Behind kWindow tiles without a
// state the furthest are asked again: the first tile of a sequence waits for
// nobody, so each one after it gets its state in turn.
constexpr int kWindow = 32;

template <int V>
__device__ __forceinline__ void look_back(const uint64_t* words, int64_t stride, int64_t most, int wave, int lane,
                                          float2 (&board)[kWindow][V][64], float (&carry)[V]) {
    int from[V];   // the nearest tile that said its state, 0: none yet
#pragma unroll
    for (int v = 0; v < V; ++v) from[v] = 0;
    for (int first = 0;; first = first + kWaves < kWindow ? first + kWaves : first) {
        const int64_t i = first + wave + 1;
        if (i <= most) {
            const uint64_t* p = words + i * stride;
            uint64_t word[V];
            for (;;) {
                bool all = true;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    word[v] = peek(p + v);
                    all = all && word[v] != kNothing;
                }
                if (__all(all)) break;
                __builtin_amdgcn_s_sleep(1);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                // a sequence's furthest tile says its state; anything else there is an end too
                const bool state = (uint32_t)(word[v] >> 32) == kState || i == most;
                board[first + wave][v][lane] = make_float2(state ? -1.0f : __uint_as_float((uint32_t)(word[v] >> 32)),
                                                           __uint_as_float((uint32_t)word[v]));
            }
        }
        __syncthreads();
        bool every = true;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            for (int k = first; k < first + kWaves && k < most; ++k)
                if (!from[v] && board[k][v][lane].x == -1.0f) from[v] = k + 1;
            every = every && from[v];
        }
        // the same in every wave: all of them read the same board
        if (__all(every)) break;
        __syncthreads();
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float h = board[from[v] - 1][v][lane].y;
        for (int k = from[v] - 2; k >= 0; --k) {
            const float2 f = board[k][v][lane];
            h = fmaf(f.x, h, f.y);
        }
        carry[v] = h;
    }
}

// The workgroup's tile: from the counter where tiles wait for each other.
__device__ __forceinline__ uint32_t tile_number(uint32_t* __restrict__ counters, uint32_t blocks, uint32_t block,
                                                uint32_t* shared) {
    if (!counters) return blockIdx.x / blocks;
    if (threadIdx.x == 0) *shared = atomicAdd(counters + block * 16, 1u);
    __syncthreads();
    return uniform(*shared);
}

// ---------------------------------------------------------------- forward
struct Launch {
    uint32_t blocks;        // blocks of channels
    uint32_t tiles;         // of a sequence (rows of equal length), else of all
    uint32_t total;         // of all
    uint32_t* counters;     // NULL where no sequence can have two tiles
    uint64_t* words;        // [total][D]
};

template <typename T, int V, bool SHARED, bool LAM, bool U>
__global__ __launch_bounds__(kWaves * 64) void seq_fwd_kernel(gspn_seq s, Launch la) {
    using R = typename Raw<T, V>::type;
    using RG = typename Raw<T, SHARED ? 1 : V>::type;
    __shared__ float2 parts[kWaves][V][64], board[kWindow][V][64];
    __shared__ uint32_t number;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const uint32_t block = blockIdx.x % la.blocks;
    const uint32_t w = tile_number(la.counters, la.blocks, block, &number);
    const Tile tile = find_tile<kSeqTile>(s.offsets, s.T, s.N, la.tiles, w, lane);
    const int64_t D = s.D;
    const int64_t d_own = (int64_t)block * (64 * V) + lane * V;
    const bool valid = d_own < D;
    const int64_t d = valid ? d_own : D - V;   // lanes behind the last channel read it and write nothing
    uint64_t* words = la.words + (size_t)w * D + d;
    const int64_t start = tile.j * kSeqTile;   // in the sequence
    T* __restrict__ y = static_cast<T*>(s.y);

    if (tile.n == s.N || (start >= tile.rows && start > 0)) {   // no tokens here
        if (la.counters && wave == 0 && valid)
#pragma unroll
            for (int v = 0; v < V; ++v) publish(words + v, kState, 0.0f);
        if (tile.n == s.N && (s.flags & GSPN_SEQ_ZERO_TAIL) && valid) {
            const float zero[V] = {};
            for (int64_t t = start + wave; t < tile.rows && t < start + kSeqTile; t += kWaves)
                put(y + (tile.row + t) * s.y_stride + d, zero);
        }
        return;
    }

    const int64_t left = tile.rows - start - wave * kTokens;
    const int count = uniform((int)(left < 0 ? 0 : left < kTokens ? left : kTokens));   // tokens of this wave
    float h[kTokens][V], P[kTokens][V];   // state and product of gates from the wave's first token on
    R uv[kTokens];
    float p[V], b[V];
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = 1.0f, b[v] = 0.0f;
    if (count > 0) {
        const int64_t row = tile.row + start + wave * kTokens;
        const int64_t k = SHARED ? d / s.ch_per_weight : d;
        const T* __restrict__ gp = static_cast<const T*>(s.gate) + row * s.gate_stride;
        const T* __restrict__ xp = static_cast<const T*>(s.x) + row * s.x_stride;
        const T* __restrict__ lp = static_cast<const T*>(s.lam) + row * s.lam_stride;
        const T* __restrict__ up = static_cast<const T*>(s.u) + row * s.u_stride;
        RG gv[kTokens];
        R xv[kTokens], lv[kTokens];
#pragma unroll
        for (int t = 0; t < kTokens; ++t) {
            const int64_t i = t < count ? t : count - 1;   // rows behind the last read it again
            gv[t] = *reinterpret_cast<const RG*>(gp + i * s.gate_stride + k);
            xv[t] = *reinterpret_cast<const R*>(xp + i * s.x_stride + d);
            if constexpr (LAM) lv[t] = *reinterpret_cast<const R*>(lp + i * s.lam_stride + d);
            if constexpr (U) uv[t] = *reinterpret_cast<const R*>(up + i * s.u_stride + d);
        }
#pragma unroll
        for (int t = 0; t < kTokens; ++t) {
            float sg[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (v == 0 || !SHARED) sg[v] = t < count ? gate_of(channel<SHARED ? 1 : V>(gv[t], v)) : kKeepAll;
                else sg[v] = sg[0];
                float in = (LAM ? channel<V>(lv[t], v) : take(sg[v])) * channel<V>(xv[t], v);
                if (t >= count) in = 0.0f;
                b[v] = keep(sg[v], b[v]) + in;
                p[v] = keep(sg[v], p[v]);
                h[t][v] = b[v];
                P[t][v] = p[v];
            }
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) parts[wave][v][lane] = make_float2(p[v], b[v]);
    __syncthreads();
    // the stretch in front of this wave, and the whole tile
    float pa[V], pb[V], ta[V], tb[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        ta[v] = 1.0f, tb[v] = 0.0f;
#pragma unroll
        for (int k = 0; k < kWaves; ++k) {
            if (k == wave) pa[v] = ta[v], pb[v] = tb[v];
            const float2 f = parts[k][v][lane];
            tb[v] = fmaf(f.x, tb[v], f.y);
            ta[v] *= f.x;
        }
    }
    float carry[V];   // the state in front of the tile
    if (tile.j == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) carry[v] = s.h0 ? s.h0[tile.n * D + d + v] : 0.0f;
    } else {
        if (wave == 0 && valid)
#pragma unroll
            for (int v = 0; v < V; ++v) publish(words + v, product_bits(ta[v]), tb[v]);
        look_back<V>(words, -D, tile.j, wave, lane, board, carry);
    }
    if (wave == 0 && valid) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (la.counters) publish(words + v, kState, fmaf(ta[v], carry[v], tb[v]));
            if (s.states) s.states[(size_t)w * D + d + v] = carry[v];
        }
    }
    if (s.h_last && wave == 0 && valid && start + kSeqTile >= tile.rows)
#pragma unroll
        for (int v = 0; v < V; ++v) s.h_last[tile.n * D + d + v] = fmaf(ta[v], carry[v], tb[v]);
    if (!valid) return;
#pragma unroll
    for (int v = 0; v < V; ++v) carry[v] = fmaf(pa[v], carry[v], pb[v]);
    T* __restrict__ yp = y + (tile.row + start + wave * kTokens) * s.y_stride + d;
#pragma unroll
    for (int t = 0; t < kTokens; ++t) {
        if (t >= count) break;
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            o[v] = fmaf(P[t][v], carry[v], h[t][v]);
            if constexpr (U) o[v] *= channel<V>(uv[t], v);
        }
        put(yp + t * s.y_stride, o);
    }
}

// ---------------------------------------------------------------- backward
// The adjoint runs from a sequence's last tile to its first: with
// R_t = a_t G_t the number that token t hands to token t - 1,
// R_t = a_t (S_t + R_{t+1}), again R -> A R + B over a stretch.  The states
// come back from the one saved in front of the tile.
//
// A gate's gradient is a sum over the channels that share it: a wave adds
// groups of `group` of them (the largest power of two that divides
// ch_per_weight, at most a wave's channels) and writes the gradient, or, where
// a set has more, the group's part for reduce_gate_kernel.
template <typename T, int V, bool SHARED, bool LAM, bool U>
__global__ __launch_bounds__(kWaves * 64) void seq_bwd_kernel(gspn_seq s, gspn_seq_grad g, Launch la, int group,
                                                              float* __restrict__ partial) {
    using R = typename Raw<T, V>::type;
    using RG = typename Raw<T, SHARED ? 1 : V>::type;
    __shared__ float2 parts[kWaves][V][64], board[kWindow][V][64];
    __shared__ float back[kWaves][V][64];
    __shared__ uint32_t number;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const uint32_t block = blockIdx.x % la.blocks;
    const uint32_t w = la.total - 1 - tile_number(la.counters, la.blocks, block, &number);
    const Tile tile = find_tile<kSeqTile>(s.offsets, s.T, s.N, la.tiles, w, lane);
    const int64_t D = s.D;
    const int64_t d_own = (int64_t)block * (64 * V) + lane * V;
    const bool valid = d_own < D;
    const int64_t d = valid ? d_own : D - V;
    uint64_t* words = la.words + (size_t)w * D + d;
    const int64_t start = tile.j * kSeqTile;
    const int64_t k = SHARED ? d / s.ch_per_weight : d;
    T* __restrict__ gx = static_cast<T*>(g.gx);
    T* __restrict__ ggate = static_cast<T*>(g.ggate);
    T* __restrict__ glam = static_cast<T*>(g.glam);
    T* __restrict__ gu = static_cast<T*>(g.gu);

    if (tile.n == s.N || (start >= tile.rows && start > 0)) {
        if (la.counters && wave == 0 && valid)
#pragma unroll
            for (int v = 0; v < V; ++v) publish(words + v, kState, 0.0f);
        if (tile.n == s.N && (s.flags & GSPN_SEQ_ZERO_TAIL) && valid) {
            const float zero[V] = {}, zero1[1] = {};
            for (int64_t t = start + wave; t < tile.rows && t < start + kSeqTile; t += kWaves) {
                const int64_t row = tile.row + t;
                if (gx) put(gx + row * g.gx_stride + d, zero);
                if (LAM && glam) put(glam + row * g.glam_stride + d, zero);
                if (U && gu) put(gu + row * g.gu_stride + d, zero);
                if (ggate) {
                    if constexpr (!SHARED) put(ggate + row * g.ggate_stride + k, zero);
                    else if (d % s.ch_per_weight == 0) put(ggate + row * g.ggate_stride + k, zero1);
                }
            }
        }
        return;
    }

    const int64_t left = tile.rows - start - wave * kTokens;
    const int count = uniform((int)(left < 0 ? 0 : left < kTokens ? left : kTokens));
    const int64_t row = tile.row + start + wave * kTokens;
    float sg[kTokens][SHARED ? 1 : V];
    R xv[kTokens], lv[kTokens], uv[kTokens], gv[kTokens];
    float p[V], b[V], r[V];
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = 1.0f, b[v] = 0.0f, r[v] = 0.0f;
    // what the gradient of h_t is from y alone: u_t gy_t
    auto source = [&](int t, int v) {
        const float q = g.gy ? channel<V>(gv[t], v) : 0.0f;
        return U ? q * channel<V>(uv[t], v) : q;
    };
    if (count > 0) {
        const T* __restrict__ gp = static_cast<const T*>(s.gate) + row * s.gate_stride;
        const T* __restrict__ xp = static_cast<const T*>(s.x) + row * s.x_stride;
        const T* __restrict__ lp = static_cast<const T*>(s.lam) + row * s.lam_stride;
        const T* __restrict__ up = static_cast<const T*>(s.u) + row * s.u_stride;
        const T* __restrict__ yp = static_cast<const T*>(g.gy) + row * g.gy_stride;
        RG raw[kTokens];
#pragma unroll
        for (int t = 0; t < kTokens; ++t) {
            const int64_t i = t < count ? t : count - 1;
            raw[t] = *reinterpret_cast<const RG*>(gp + i * s.gate_stride + k);
            xv[t] = *reinterpret_cast<const R*>(xp + i * s.x_stride + d);
            if constexpr (LAM) lv[t] = *reinterpret_cast<const R*>(lp + i * s.lam_stride + d);
            if constexpr (U) uv[t] = *reinterpret_cast<const R*>(up + i * s.u_stride + d);
            if (g.gy) gv[t] = *reinterpret_cast<const R*>(yp + i * g.gy_stride + d);
        }
#pragma unroll
        for (int t = 0; t < kTokens; ++t) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (v == 0 || !SHARED) sg[t][v] = t < count ? gate_of(channel<SHARED ? 1 : V>(raw[t], v)) : kKeepAll;
                const float a = sg[t][SHARED ? 0 : v];
                float in = (LAM ? channel<V>(lv[t], v) : take(a)) * channel<V>(xv[t], v);
                if (t >= count) in = 0.0f;
                b[v] = keep(a, b[v]) + in;
                p[v] = keep(a, p[v]);
            }
        }
#pragma unroll
        for (int t = kTokens - 1; t >= 0; --t)
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (t < count) r[v] = keep(sg[t][SHARED ? 0 : v], source(t, v) + r[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        parts[wave][v][lane] = make_float2(p[v], b[v]);
        back[wave][v][lane] = r[v];
    }
    __syncthreads();
    float h0[V];                        // the state in front of this wave's tokens
    float pa[V], pb[V], ta[V], tb[V];   // the adjoint's stretches: behind this wave, the whole tile
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float f = s.states[(size_t)w * D + d + v];
#pragma unroll
        for (int q = 0; q < kWaves; ++q) {
            if (q == wave) h0[v] = f;
            f = fmaf(parts[q][v][lane].x, f, parts[q][v][lane].y);
        }
        ta[v] = 1.0f, tb[v] = 0.0f;
#pragma unroll
        for (int q = kWaves - 1; q >= 0; --q) {
            if (q == wave) pa[v] = ta[v], pb[v] = tb[v];
            const float a = parts[q][v][lane].x;
            tb[v] = fmaf(a, tb[v], back[q][v][lane]);
            ta[v] *= a;
        }
    }
    float carry[V];   // what the token behind the tile hands to its last
    const int64_t behind = (tile.rows + kSeqTile - 1) / kSeqTile - 1 - tile.j;
    if (behind <= 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) carry[v] = g.gh_last ? g.gh_last[tile.n * D + d + v] : 0.0f;
    } else {
        if (wave == 0 && valid)
#pragma unroll
            for (int v = 0; v < V; ++v) publish(words + v, product_bits(ta[v]), tb[v]);
        look_back<V>(words, D, behind, wave, lane, board, carry);
    }
    if (wave == 0 && valid) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float out = fmaf(ta[v], carry[v], tb[v]);
            if (la.counters) publish(words + v, kState, out);
            if (g.gh0 && tile.j == 0) g.gh0[tile.n * D + d + v] = out;
        }
    }
    if (count <= 0) return;
    float h[kTokens + 1][V], G[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        G[v] = fmaf(pa[v], carry[v], pb[v]);   // R of the token behind
        h[0][v] = h0[v];
#pragma unroll
        for (int t = 0; t < kTokens; ++t) {
            const float a = sg[t][SHARED ? 0 : v];
            h[t + 1][v] = keep(a, h[t][v]) + (LAM ? channel<V>(lv[t], v) : take(a)) * channel<V>(xv[t], v);
        }
    }
    const int lanes = group / V;   // lanes of a group
#pragma unroll
    for (int t = kTokens - 1; t >= 0; --t) {
        if (t >= count) continue;
        float ox[V], ol[V], ou[V], og[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float a = sg[t][SHARED ? 0 : v];
            const float x = channel<V>(xv[t], v), small = fabsf(a);
            G[v] += source(t, v);
            ox[v] = G[v] * (LAM ? channel<V>(lv[t], v) : take(a));
            ol[v] = G[v] * x;
            ou[v] = (g.gy ? channel<V>(gv[t], v) : 0.0f) * h[t + 1][v];
            og[v] = small * (1.0f - small) * G[v] * (LAM ? h[t][v] : h[t][v] - x);
            G[v] = keep(a, G[v]);
        }
        const int64_t i = row + t;
        if (valid) {
            if (gx) put(gx + i * g.gx_stride + d, ox);
            if (LAM && glam) put(glam + i * g.glam_stride + d, ol);
            if (U && gu) put(gu + i * g.gu_stride + d, ou);
        }
        if constexpr (!SHARED) {
            if (ggate && valid) put(ggate + i * g.ggate_stride + d, og);
        } else if (ggate) {
            float sum[1] = {og[0]};
            if constexpr (V == 2) sum[0] += og[1];
            for (int m = 1; m < lanes; m <<= 1) sum[0] += __shfl_xor(sum[0], m);
            if (valid && lane % lanes == 0) {
                if (partial) partial[i * (D / group) + d / group] = sum[0];
                else put(ggate + i * g.ggate_stride + k, sum);
            }
        }
    }
}

// ggate[t][k] = sum of the set's parts, for the rows of sequences.
template <typename T>
__global__ __launch_bounds__(256) void reduce_gate_kernel(gspn_seq s, gspn_seq_grad g, int group,
                                                          const float* __restrict__ partial) {
    const int64_t sets = s.D / s.ch_per_weight;
    const int parts = s.ch_per_weight / group;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t t = i / sets, k = i - t * sets;
    if (t >= (s.offsets ? (int64_t)s.offsets[s.N] : s.T) || t >= s.T) return;
    const float* __restrict__ p = partial + t * (s.D / group) + k * parts;
    float sum = 0.0f;
    for (int c = 0; c < parts; ++c) sum += p[c];
    static_cast<T*>(g.ggate)[t * g.ggate_stride + k] = from_f32(sum, (T*)nullptr);
}

// Clears what the tiles tell each other and their counters (a kernel, not a
// memset, so that the call can be captured into a graph).
__global__ __launch_bounds__(256) void seq_clear_kernel(uint4* __restrict__ counters, int64_t nc,
                                                        uint4* __restrict__ words, int64_t nw) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < nc + nw; i += (int64_t)gridDim.x * 256) {
        if (i < nc) counters[i] = make_uint4(0, 0, 0, 0);
        else words[i - nc] = make_uint4(~0u, ~0u, ~0u, ~0u);
    }
}

// ---------------------------------------------------------------- step
// One lane per channel of a row.  Rows of one slot are taken in their order
// by the lanes of the first of them; the others leave it to those.
template <typename T>
__global__ __launch_bounds__(256) void seq_step_kernel(gspn_seq_token s) {
    const int64_t blocks = (s.D + 255) / 256;
    const int64_t row = blockIdx.x / blocks;
    const int64_t d = (blockIdx.x - row * blocks) * 256 + threadIdx.x;
    const int64_t slot = s.slots ? s.slots[row] : row;
    if (slot < 0 || slot >= s.S) return;
    bool more = false;
    if (s.slots) {
        bool earlier = false, later = false;
        for (int64_t r = threadIdx.x; r < s.N; r += 256)
            if (r != row && s.slots[r] == slot) (r < row ? earlier : later) = true;
        if (__syncthreads_or(earlier)) return;
        more = __syncthreads_or(later);
    }
    if (d >= s.D) return;
    const int64_t k = d / s.ch_per_weight;
    float h = s.state[slot * s.D + d];
    for (int64_t r = row; r < s.N; ++r) {
        if (r != row && s.slots[r] != slot) continue;
        const float a = gate_of(to_f32(static_cast<const T*>(s.gate)[r * s.gate_stride + k]));
        const float xv = to_f32(static_cast<const T*>(s.x)[r * s.x_stride + d]);
        const float lv = s.lam ? to_f32(static_cast<const T*>(s.lam)[r * s.lam_stride + d]) : take(a);
        h = keep(a, h) + lv * xv;
        const float uv = s.u ? to_f32(static_cast<const T*>(s.u)[r * s.u_stride + d]) : 1.0f;
        static_cast<T*>(s.y)[r * s.y_stride + d] = from_f32(uv * h, (T*)nullptr);
        if (!more) break;
    }
    s.state[slot * s.D + d] = h;
}

// ---------------------------------------------------------------- host
// Whether a sequence may have two tiles.
bool tiles_wait(const gspn_seq& s) { return (s.offsets ? s.T : s.T / s.N) > kSeqTile; }

int64_t counter_bytes(const gspn_seq& s) { return (s.D + 63) / 64 * 64; }   // 64 for the narrowest block

int64_t words_bytes(const gspn_seq& s) { return ((int64_t)total_tiles<kSeqTile>(s.offsets, s.T, s.N) * s.D * 8 + 15) / 16 * 16; }

int power_of_two_in(int64_t v, int most) {
    int p = 1;
    while (p < most && v % (2 * p) == 0) p *= 2;
    return p;
}

bool even(const void* p, int64_t stride) { return ((uintptr_t)p & 3) == 0 && stride % 2 == 0; }

// Two channels a lane: bf16 rows whose pairs are whole 4-byte words, and no
// pair with two gates of a shared kind.
bool pairs(const gspn_seq& s) {
    return s.dtype == GSPN_BF16 && s.D % 2 == 0 && (s.ch_per_weight == 1 || s.ch_per_weight % 2 == 0) &&
           even(s.x, s.x_stride) && even(s.lam, s.lam ? s.lam_stride : 0) && even(s.u, s.u ? s.u_stride : 0) &&
           (s.ch_per_weight > 1 || even(s.gate, s.gate_stride));
}

Launch plan(const gspn_seq& s, int V) {
    Launch la;
    la.blocks = (uint32_t)((s.D + 64 * V - 1) / (64 * V));
    la.tiles = s.offsets ? 0 : tiles_of_sequence<kSeqTile>(s.T, s.N);
    la.total = total_tiles<kSeqTile>(s.offsets, s.T, s.N);
    la.counters = nullptr;
    la.words = nullptr;
    if (tiles_wait(s)) {
        la.counters = static_cast<uint32_t*>(s.work);
        la.words = reinterpret_cast<uint64_t*>(static_cast<char*>(s.work) + counter_bytes(s));
    }
    return la;
}

void clear(const gspn_seq& s, const Launch& la, hipStream_t stream) {
    if (!la.counters) return;
    const int64_t nc = counter_bytes(s) / 16, nw = words_bytes(s) / 16;
    const unsigned grid = (unsigned)std::min<int64_t>((nc + nw + 255) / 256, 2048);
    hipLaunchKernelGGL(seq_clear_kernel, dim3(grid), dim3(256), 0, stream, reinterpret_cast<uint4*>(la.counters), nc,
                       reinterpret_cast<uint4*>(la.words), nw);
}

// f(kernel) for the variant that the flags name.
template <typename T, int V, typename F>
void fwd_variant(bool shared, bool lam, bool u, F f) {
    if (shared) {
        if (lam) u ? f(seq_fwd_kernel<T, V, true, true, true>) : f(seq_fwd_kernel<T, V, true, true, false>);
        else u ? f(seq_fwd_kernel<T, V, true, false, true>) : f(seq_fwd_kernel<T, V, true, false, false>);
    } else {
        if (lam) u ? f(seq_fwd_kernel<T, V, false, true, true>) : f(seq_fwd_kernel<T, V, false, true, false>);
        else u ? f(seq_fwd_kernel<T, V, false, false, true>) : f(seq_fwd_kernel<T, V, false, false, false>);
    }
}

template <typename T, int V, typename F>
void bwd_variant(bool shared, bool lam, bool u, F f) {
    if (shared) {
        if (lam) u ? f(seq_bwd_kernel<T, V, true, true, true>) : f(seq_bwd_kernel<T, V, true, true, false>);
        else u ? f(seq_bwd_kernel<T, V, true, false, true>) : f(seq_bwd_kernel<T, V, true, false, false>);
    } else {
        if (lam) u ? f(seq_bwd_kernel<T, V, false, true, true>) : f(seq_bwd_kernel<T, V, false, true, false>);
        else u ? f(seq_bwd_kernel<T, V, false, false, true>) : f(seq_bwd_kernel<T, V, false, false, false>);
    }
}

}  // namespace

int64_t seq_workspace(const gspn_seq& s, bool backward) {
    int64_t bytes = tiles_wait(s) ? counter_bytes(s) + words_bytes(s) : 0;
    const int group = power_of_two_in(s.ch_per_weight, 64);   // the smallest that a launch may take
    if (backward && group < s.ch_per_weight) bytes += s.T * (s.D / group) * 4;
    return bytes;
}

hipError_t launch_seq_fwd(const gspn_seq& s, hipStream_t stream) {
    const int V = pairs(s) && even(s.y, s.y_stride) ? 2 : 1;
    const Launch la = plan(s, V);
    clear(s, la, stream);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(la.total * la.blocks), dim3(kWaves * 64), 0, stream, s, la);
    };
    const bool shared = s.ch_per_weight > 1;
    if (s.dtype == GSPN_F32) fwd_variant<float, 1>(shared, s.lam, s.u, go);
    else if (V == 2) fwd_variant<uint16_t, 2>(shared, s.lam, s.u, go);
    else fwd_variant<uint16_t, 1>(shared, s.lam, s.u, go);
    return hipGetLastError();
}

hipError_t launch_seq_bwd(const gspn_seq& s, const gspn_seq_grad& g, hipStream_t stream) {
    const int V = pairs(s) && even(g.gy, g.gy ? g.gy_stride : 0) && even(g.gx, g.gx ? g.gx_stride : 0) &&
                          even(g.glam, g.glam ? g.glam_stride : 0) && even(g.gu, g.gu ? g.gu_stride : 0) &&
                          (s.ch_per_weight > 1 || even(g.ggate, g.ggate ? g.ggate_stride : 0))
                      ? 2 : 1;
    const Launch la = plan(s, V);
    const int group = power_of_two_in(s.ch_per_weight, 64 * V);
    float* partial = nullptr;
    if (group < s.ch_per_weight && g.ggate)
        partial = reinterpret_cast<float*>(static_cast<char*>(s.work) +
                                           (la.counters ? counter_bytes(s) + words_bytes(s) : 0));
    clear(s, la, stream);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(la.total * la.blocks), dim3(kWaves * 64), 0, stream, s, g, la, group, partial);
    };
    const bool shared = s.ch_per_weight > 1;
    if (s.dtype == GSPN_F32) bwd_variant<float, 1>(shared, s.lam, s.u, go);
    else if (V == 2) bwd_variant<uint16_t, 2>(shared, s.lam, s.u, go);
    else bwd_variant<uint16_t, 1>(shared, s.lam, s.u, go);
    if (partial && s.T) {
        const dim3 grid((unsigned)((s.T * (s.D / s.ch_per_weight) + 255) / 256));
        if (s.dtype == GSPN_BF16)
            hipLaunchKernelGGL(reduce_gate_kernel<uint16_t>, grid, dim3(256), 0, stream, s, g, group, partial);
        else
            hipLaunchKernelGGL(reduce_gate_kernel<float>, grid, dim3(256), 0, stream, s, g, group, partial);
    }
    return hipGetLastError();
}

hipError_t launch_seq_step(const gspn_seq_token& t, hipStream_t stream) {
    const dim3 grid((unsigned)(t.N * ((t.D + 255) / 256)));
    if (t.dtype == GSPN_BF16) hipLaunchKernelGGL(seq_step_kernel<uint16_t>, grid, dim3(256), 0, stream, t);
    else hipLaunchKernelGGL(seq_step_kernel<float>, grid, dim3(256), 0, stream, t);
    return hipGetLastError();
}

}  // namespace gspn
