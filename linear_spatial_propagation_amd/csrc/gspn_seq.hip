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
// (A2 A1, A2 B1 + B2).  So a sequence is cut into tiles that work side by
// side:
//  * a workgroup owns one tile of one block of channels (a lane owns V
//    neighbouring channels), a wave TOKENS tokens of it, held in registers:
//    every input is read once;
//  * each wave forms its stretch's (A, B), the waves join theirs in LDS, and
//    the workgroup publishes the tile's;
//  * a tile that is not its sequence's first looks back over the tiles in front
//    of it to one that has published the state behind itself, goes from there
//    through the (A, B) of those between, and publishes its own state;
//  * with the state in front of its tokens, each wave finishes them.
// A tile never holds rows of two sequences, so nothing passes between them.
//
// Every number is read and written once (what the tiles tell each other is 4 to
// 8 % on top), so memory bounds the kernels: a copy reaches 5.1 TB/s here, and
//   16 rows of 2048 tokens, 1152 channels in bf16, a gate for 8, lam and u:
//     forward 76 us, 4.1 TB/s; backward 122 us, 4.5 TB/s;
//   one sequence of 131072 tokens, 1024 channels in bf16: forward 200 us, 4.0 TB/s;
//   24 sequences of 8192 tokens in all, 2048 channels in bf16, lam and u:
//     forward 50 us, 3.3 TB/s.  Its 1424 workgroups are three rounds of what fits
//     the chip, and neighbouring tiles of a sequence run at the same time, so that
//     the later waits for the slowest loads of the earlier ones.  Twice the waves
//     with half the tokens, or tiles of half the size, left that as it was or made
//     it slower (50 to 65 us); an order across the sequences, which rows of equal
//     length have, would need a table of tiles sorted before the launch.
// Reading the next tile's inputs while the present one is finished (workgroups that
// stay) came out no faster: the registers for it halve what is on its way.
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

#include <type_traits>

namespace gspn {
namespace {

using Yes = std::integral_constant<bool, true>;
using No = std::integral_constant<bool, false>;

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

// A walk down the rows of a tensor: the row is the same for a wave's lanes (a
// scalar register), a lane's place in it a 32-bit offset.
template <typename T> struct Walk {
    const char* p;
    int64_t step;
    __device__ Walk(const void* base, int64_t row, int64_t stride)
        : p(static_cast<const char*>(base) + row * stride * (int64_t)sizeof(T)), step(stride * (int64_t)sizeof(T)) {}
    template <typename R> __device__ R at(uint32_t offset) const { return *reinterpret_cast<const R*>(p + offset); }
    __device__ T* out(uint32_t offset) const { return reinterpret_cast<T*>(const_cast<char*>(p) + offset); }
    __device__ void down(bool go = true) { p += go ? step : 0; }
    __device__ void up() { p -= step; }
};

// ---------------------------------------------------------------- gates
// A gate as one number that loses no precision for a near 0 or near 1: the
// smaller of a and 1 - a, with the sign of the raw gate (positive, 0 included:
// it is 1 - a).  `most`, the larger of the two, is what the gate still has at
// hand where it is made.
__device__ __forceinline__ bool open(float s) { return (int32_t)__float_as_uint(s) >= 0; }

__device__ __forceinline__ float gate_of(float g, float& most) {
    const float e = fast_exp2(fabsf(g) * -1.44269504088896340736f);
    most = fast_rcp(1.0f + e);
    return __builtin_copysignf(e * most, g);
}
__device__ __forceinline__ float take(float s, float most) { return open(s) ? s : most; }   // 1 - a

// a h + in, in = l x.  For a near 1 it is h - (1 - a) h: the rounding of such an a
// (2^-24 of h at every token) would add up over the gate's memory, 1 / (1 - a)
// tokens; that of 1 - a does not.
__device__ __forceinline__ float keep(float s, float h) { return fmaf(-s, h, open(s) ? h : 0.0f); }
__device__ __forceinline__ float keep(float s, float h, float l, float x) {
    return fmaf(-s, h, fmaf(l, x, open(s) ? h : 0.0f));
}

// Rows behind a wave's last token are made to change nothing: their gate is
// +inf (a = 1) and their x (and lam) 0.
__device__ __forceinline__ void no_row(uint16_t& gate, uint16_t& x) { gate = 0x7f80u, x = 0; }
__device__ __forceinline__ void no_row(uint16_t& gate, uint32_t& x) { gate = 0x7f80u, x = 0; }
__device__ __forceinline__ void no_row(uint32_t& gate, uint32_t& x) { gate = 0x7f807f80u, x = 0; }
__device__ __forceinline__ void no_row(float& gate, float& x) { gate = __builtin_inff(), x = 0.0f; }

// The scheduler moves nothing across: loads above stay above, and what is below
// does not take registers up there.
__device__ __forceinline__ void hold() { __builtin_amdgcn_sched_barrier(0); }

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

// A tile's flag says how far it is: a hint, so that those who wait read four
// bytes a tile and not its words, which say the same by themselves.
constexpr uint32_t kHasProduct = 1, kHasState = 2;

__device__ __forceinline__ void raise(uint32_t* flag, uint32_t to) {
    __hip_atomic_store(flag, to, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The state that the `most` >= 1 tiles before this one leave in front of it (tile
// i's words are i strides further, i = 1 the nearest; the furthest is the
// sequence's end).  One wave looks at the flags of the nearest WINDOW tiles until
// one has its state and all nearer ones their (A, B); the waves then fetch those
// tiles' words, and from the state the (A, B) lead back, h -> A h + B one tile
// after the other.  That is the arithmetic by which those tiles get their own
// states, so the result does not depend on who was first.  Where the nearest
// WINDOW tiles have no state yet, one of them gets it in its turn: the first tile
// of a sequence waits for nobody.
template <int V, int WAVES, int WINDOW>
__device__ __forceinline__ void look_back(const uint64_t* words, int64_t stride, const uint32_t* flag,
                                          int flag_stride, int64_t most, int wave, int lane,
                                          float2 (&board)[WINDOW][V][64], int* shared, float (&carry)[V]) {
    constexpr int kFetch = WINDOW / WAVES;   // tiles that a wave fetches at most
    if (wave == 0) {
        const int in_reach = most < WINDOW ? (int)most : WINDOW;
        for (;;) {
            uint32_t f = 0;
            if (lane < in_reach)
                f = __hip_atomic_load(flag + (int64_t)(lane + 1) * flag_stride, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            const uint64_t state = __ballot(f == kHasState), some = __ballot(f != 0);
            if (state) {
                const int nearest = __ffsll((unsigned long long)state) - 1;
                const uint64_t nearer = ((uint64_t)1 << nearest) - 1;
                if ((some & nearer) == nearer) {
                    if (lane == 0) *shared = nearest + 1;
                    break;
                }
            }
            __builtin_amdgcn_s_sleep(1);
        }
    }
    __syncthreads();
    const int far = uniform(*shared);
    uint64_t word[kFetch][V];
#pragma unroll
    for (int a = 0; a < kFetch; ++a) {
        const int i = a * WAVES + wave + 1;
        if (i <= far)
#pragma unroll
            for (int v = 0; v < V; ++v) word[a][v] = peek(words + i * stride + v * 64);
    }
#pragma unroll
    for (int a = 0; a < kFetch; ++a) {
        const int i = a * WAVES + wave + 1;
        if (i <= far) {
            for (;;) {   // a flag may be seen before its tile's words
                bool all = true;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    all = all && (i < far ? word[a][v] != kNothing : (uint32_t)(word[a][v] >> 32) == kState);
                if (__all(all)) break;
                __builtin_amdgcn_s_sleep(1);
#pragma unroll
                for (int v = 0; v < V; ++v) word[a][v] = peek(words + i * stride + v * 64);
            }
#pragma unroll
            for (int v = 0; v < V; ++v)
                board[i - 1][v][lane] = make_float2(__uint_as_float((uint32_t)(word[a][v] >> 32)),
                                                    __uint_as_float((uint32_t)word[a][v]));
        }
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float h = board[far - 1][v][lane].y;   // a state
        for (int k = far - 2; k >= 0; --k) {
            const float2 f = board[k][v][lane];
            h = __float_as_uint(f.x) == kState ? f.y : fmaf(f.x, h, f.y);   // one may have got its state since
        }
        carry[v] = h;
    }
}

struct Launch {
    uint32_t blocks;        // blocks of channels
    uint32_t tiles;         // of a sequence (rows of equal length), else 0
    uint32_t total;         // of all
    uint32_t* counters;     // NULL where no sequence can have two tiles
    uint32_t* flags;        // [blocks][total]
    uint64_t* words;        // [total][blocks][V][64]: a lane's channels 64 words apart, so that each is one whole line's
    int spacing;            // tokens between two saved states
};

// How a call's tiles are laid out.  It goes by T, N and the layout alone, as
// `states` is sized before anything else is known.
//   kShort:  sequences of up to 32 tokens on average, which would leave most waves of
//            larger tiles without one: tiles of 32;
//   kMiddle: packed sequences of up to 96 on average: tiles of 64, backward 32 or 64
//            (8192 tokens of 2048 channels in bf16, a gate for each, sequences of 43
//            on average: 53 and 99 us, with 128 tokens a tile 76 and 153; of 96: 53
//            and 102, 56 and 112; of 128: 53 and 104 either way);
//   kRows:   many rows of equal length: a tile seldom waits (tile_number), and small
//            ones let more workgroups into a CU;
//   kLong:   the rest: the fewer tiles there are in a row, the fewer wait.
enum Kind { kShort, kMiddle, kRows, kLong };
inline Kind kind_of(int64_t T, int64_t N, bool packed) {
    return T <= 32 * N ? kShort : packed && T <= 96 * N ? kMiddle : !packed && N >= 8 ? kRows : kLong;
}

// Tokens between two saved states, of which the backward's tile is a multiple (64
// instead of 128 writes 1.5 % more in the forward).
inline int spacing_of(int64_t T, int64_t N, bool packed) {
    const Kind kind = kind_of(T, N, packed);
    return kind <= kMiddle ? 32 : N >= 8 ? 64 : 128;
}

// The row of `states` in front of token `first` of a sequence: sequences take rows
// as they take tiles of that size (find_tile).
__device__ __forceinline__ int64_t states_row(const Tile& tile, bool packed, int64_t first, int spacing) {
    const int64_t per = (tile.rows + spacing - 1) / spacing;
    return (packed ? tile.row / spacing + tile.n : tile.n * (per > 0 ? per : 1)) + first / spacing;
}

// The workgroup's tile: from the counter where tiles wait for each other.  Rows of
// equal length are taken tile by tile across the sequences (the backward: from
// the last), so that the tile in front of one's own was taken long ago.
__device__ __forceinline__ uint32_t tile_number(const Launch& la, uint32_t block, bool from_last, uint32_t* shared) {
    uint32_t k;
    if (!la.counters) {
        k = blockIdx.x / la.blocks;
    } else {
        if (threadIdx.x == 0) *shared = atomicAdd(la.counters + block * 16, 1u);
        __syncthreads();
        k = uniform(*shared);
    }
    if (from_last) k = la.total - 1 - k;
    if (la.tiles == 0) return k;
    const uint32_t sequences = la.total / la.tiles;
    return (k % sequences) * la.tiles + k / sequences;
}

// ---------------------------------------------------------------- forward
// Holds the state and the product of gates of all its tokens in registers, so
// that with the carry each output is one fma: y = u (P carry + h).  Loads all of
// a wave's tokens before the first is used (32 tokens by 128 channels in bf16: 16
// to 32 KB a wave on their way).
template <typename T, int V, bool SHARED, bool LAM, bool U, int TOKENS, int WAVES>
__global__ __launch_bounds__(WAVES * 64, 2) void seq_fwd_kernel(gspn_seq s, Launch la) {
    constexpr int TILE = TOKENS * WAVES, WINDOW = 4 * WAVES;
    using R = typename Raw<T, V>::type;
    using RG = typename Raw<T, SHARED ? 1 : V>::type;
    __shared__ float2 parts[WAVES][V][64], board[WINDOW][V][64];
    __shared__ uint32_t number;
    __shared__ int far;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const uint32_t block = blockIdx.x % la.blocks;
    const int32_t first_seen = first_offsets(s.offsets, s.N, lane);
    const uint32_t w = tile_number(la, block, false, &number);
    const Tile tile = find_tile<TILE>(s.offsets, s.T, s.N, la.tiles, w, lane, first_seen);
    const int64_t D = s.D;
    const int64_t d_own = (int64_t)block * (64 * V) + lane * V;
    const bool valid = d_own < D;
    const int64_t d = valid ? d_own : D - V;   // lanes behind the last channel read it and write nothing
    const uint32_t dd = (uint32_t)d * sizeof(T);
    uint64_t* words = la.words + ((size_t)w * la.blocks + block) * (64 * V) + lane;
    uint32_t* flag = la.flags + (size_t)block * la.total + w;
    const int64_t start = tile.j * TILE;   // in the sequence
    T* __restrict__ y = static_cast<T*>(s.y);

    if (tile.n == s.N || (start >= tile.rows && start > 0)) {   // no tokens here
        if (la.counters && wave == 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) publish(words + v * 64, kState, 0.0f);
            if (lane == 0) raise(flag, kHasState);
        }
        if (tile.n == s.N && (s.flags & GSPN_SEQ_ZERO_TAIL) && valid) {
            const float zero[V] = {};
            for (int64_t t = start + wave; t < tile.rows && t < start + TILE; t += WAVES)
                put(y + (tile.row + t) * s.y_stride + d, zero);
        }
        return;
    }

    const int64_t left = tile.rows - start - wave * TOKENS;
    const int count = uniform((int)(left < 0 ? 0 : left < TOKENS ? left : TOKENS));   // tokens of this wave
    float h[TOKENS][V], P[TOKENS][V];   // state and product of gates from the wave's first token on
    R uv[TOKENS];
    float p[V], b[V];
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = 1.0f, b[v] = 0.0f;
    if (count > 0) {
        const int64_t row = tile.row + start + wave * TOKENS;
        const uint32_t dk = (SHARED ? (uint32_t)d / (uint32_t)s.ch_per_weight : (uint32_t)d) * sizeof(T);
        Walk<T> gp(s.gate, row, s.gate_stride), xp(s.x, row, s.x_stride);
        Walk<T> lp(s.lam, row, s.lam_stride), up(s.u, row, s.u_stride);
        RG gv[TOKENS];
        R xv[TOKENS], lv[TOKENS];
#pragma unroll
        for (int t = 0; t < TOKENS; ++t) {
            gv[t] = gp.template at<RG>(dk);
            xv[t] = xp.template at<R>(dd);
            if constexpr (LAM) lv[t] = lp.template at<R>(dd);
            if constexpr (U) uv[t] = up.template at<R>(dd);
            const bool more = t + 1 < count;   // rows behind the last read it again
            gp.down(more), xp.down(more);
            if constexpr (LAM) lp.down(more);
            if constexpr (U) up.down(more);
        }
        hold();
        if (count < TOKENS)
#pragma unroll
            for (int t = 0; t < TOKENS; ++t)
                if (t >= count) {
                    no_row(gv[t], xv[t]);
                    if constexpr (LAM) lv[t] = R(0);
                }
#pragma unroll
        for (int t = 0; t < TOKENS; ++t) {
            float sg = 0.0f, most = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (v == 0 || !SHARED) sg = gate_of(channel<SHARED ? 1 : V>(gv[t], v), most);
                b[v] = keep(sg, b[v], LAM ? channel<V>(lv[t], v) : take(sg, most), channel<V>(xv[t], v));
                p[v] = keep(sg, p[v]);
                h[t][v] = b[v];
                P[t][v] = p[v];
            }
            if (t % 2) hold();
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) parts[wave][v][lane] = make_float2(p[v], b[v]);
    __syncthreads();
    // the stretch in front of this wave, and (wave 0, which tells) the whole tile
    float pa[V], pb[V], ta[V], tb[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float2 f[WAVES];
#pragma unroll
        for (int k = 0; k < WAVES; ++k) f[k] = parts[k][v][lane];
        pa[v] = 1.0f, pb[v] = 0.0f, ta[v] = 1.0f, tb[v] = 0.0f;
#pragma unroll
        for (int k = 0; k < WAVES; ++k) {
            if (k < wave) pb[v] = fmaf(f[k].x, pb[v], f[k].y), pa[v] *= f[k].x;
            if (wave == 0) tb[v] = fmaf(f[k].x, tb[v], f[k].y), ta[v] *= f[k].x;
        }
        hold();
    }
    float carry[V];   // the state in front of the tile
    if (tile.j == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) carry[v] = s.h0 ? s.h0[tile.n * D + d + v] : 0.0f;
    } else {
        if (wave == 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) publish(words + v * 64, product_bits(ta[v]), tb[v]);
            if (lane == 0) raise(flag, kHasProduct);
        }
        look_back<V, WAVES, WINDOW>(words, -(int64_t)la.blocks * (64 * V), flag, -1, tile.j, wave, lane, board, &far, carry);
    }
    if (wave == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (la.counters) publish(words + v * 64, kState, fmaf(ta[v], carry[v], tb[v]));
        }
        if (la.counters && lane == 0) raise(flag, kHasState);
    }
    if (s.h_last && wave == 0 && valid && start + TILE >= tile.rows)
#pragma unroll
        for (int v = 0; v < V; ++v) s.h_last[tile.n * D + d + v] = fmaf(ta[v], carry[v], tb[v]);
    if (!valid) return;
#pragma unroll
    for (int v = 0; v < V; ++v) carry[v] = fmaf(pa[v], carry[v], pb[v]);
    const int64_t first = start + wave * TOKENS;
    if (s.states && first % la.spacing == 0 && (first == 0 || first < tile.rows)) {
        const int64_t at = states_row(tile, s.offsets != nullptr, first, la.spacing);
#pragma unroll
        for (int v = 0; v < V; ++v) s.states[at * D + d + v] = carry[v];
    }
    Walk<T> yp(s.y, tile.row + start + wave * TOKENS, s.y_stride);
#pragma unroll
    for (int t = 0; t < TOKENS; ++t) {
        if (t < count) {
            float o[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                o[v] = fmaf(P[t][v], carry[v], h[t][v]);
                if constexpr (U) o[v] *= channel<V>(uv[t], v);
            }
            put(yp.out(dd), o);
        }
        yp.down();
    }
}

// ---------------------------------------------------------------- backward
// v[t] of `lanes` (a power of two) neighbouring lanes added up; the last of them
// has the sum.
template <int CTRL> __device__ __forceinline__ float other(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int COUNT> __device__ __forceinline__ void add_lanes(float (&v)[COUNT], int lanes) {
    if (lanes >= 2)
#pragma unroll
        for (int t = 0; t < COUNT; ++t) v[t] += other<0xb1>(v[t]);    // quad_perm [1, 0, 3, 2]
    if (lanes >= 4)
#pragma unroll
        for (int t = 0; t < COUNT; ++t) v[t] += other<0x4e>(v[t]);    // quad_perm [2, 3, 0, 1]
    if (lanes >= 8)
#pragma unroll
        for (int t = 0; t < COUNT; ++t) v[t] += other<0x141>(v[t]);   // row_half_mirror
    if (lanes >= 16)
#pragma unroll
        for (int t = 0; t < COUNT; ++t) v[t] += other<0x140>(v[t]);   // row_mirror
    if (lanes >= 32)
#pragma unroll
        for (int t = 0; t < COUNT; ++t) v[t] += other<0x142>(v[t]);   // row_bcast:15, into the next row
    if (lanes >= 64)
#pragma unroll
        for (int t = 0; t < COUNT; ++t) v[t] += other<0x143>(v[t]);   // row_bcast:31, into the upper half
}

// The adjoint runs from a sequence's last tile to its first: with
// R_t = a_t G_t the number that token t hands to token t - 1,
// R_t = a_t (S_t + R_{t+1}), again R -> A R + B over a stretch.  The states
// come back from the one saved in front of the tile.
//
// A gate's gradient is a sum over the channels that share it: a wave adds
// groups of `group` of them (the largest power of two that divides
// ch_per_weight, at most a wave's channels) and writes the gradient, or, where
// a set has more, the group's part for reduce_gate_kernel.  No atomics: sums
// have one order.
//
// Nothing that the forward computed but states some tokens apart comes from
// memory: gates and states are made again from inputs that the gradients need
// anyway.  A wave of whole tokens with every gradient asked for takes a copy of
// the last loop without checks (8 rows of 2048 tokens, 4096 channels: 304 -> 287 us).
template <typename T, int V, bool SHARED, bool LAM, bool U, int TOKENS, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void seq_bwd_kernel(gspn_seq s, gspn_seq_grad g, Launch la, int group,
                                                             float* __restrict__ partial) {
    constexpr int TILE = TOKENS * WAVES, WINDOW = 4 * WAVES;   // TILE is a multiple of the states' spacing
    using R = typename Raw<T, V>::type;
    using RG = typename Raw<T, SHARED ? 1 : V>::type;
    __shared__ float2 parts[WAVES][V][64], board[WINDOW][V][64];
    __shared__ float back[WAVES][V][64];
    __shared__ uint32_t number;
    __shared__ int far;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const uint32_t block = blockIdx.x % la.blocks;
    const int32_t first_seen = first_offsets(s.offsets, s.N, lane);
    const uint32_t w = tile_number(la, block, true, &number);
    const Tile tile = find_tile<TILE>(s.offsets, s.T, s.N, la.tiles, w, lane, first_seen);
    const int64_t D = s.D;
    const int64_t d_own = (int64_t)block * (64 * V) + lane * V;
    const bool valid = d_own < D;
    const int64_t d = valid ? d_own : D - V;
    const uint32_t dd = (uint32_t)d * sizeof(T);
    uint64_t* words = la.words + ((size_t)w * la.blocks + block) * (64 * V) + lane;
    uint32_t* flag = la.flags + (size_t)block * la.total + w;
    const int64_t start = tile.j * TILE;
    const uint32_t k = SHARED ? (uint32_t)d / (uint32_t)s.ch_per_weight : (uint32_t)d;
    const uint32_t dk = k * sizeof(T);
    T* __restrict__ gx = static_cast<T*>(g.gx);
    T* __restrict__ ggate = static_cast<T*>(g.ggate);
    T* __restrict__ glam = static_cast<T*>(g.glam);
    T* __restrict__ gu = static_cast<T*>(g.gu);

    if (tile.n == s.N || (start >= tile.rows && start > 0)) {
        if (la.counters && wave == 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) publish(words + v * 64, kState, 0.0f);
            if (lane == 0) raise(flag, kHasState);
        }
        if (tile.n == s.N && (s.flags & GSPN_SEQ_ZERO_TAIL) && valid) {
            const float zero[V] = {}, zero1[1] = {};
            for (int64_t t = start + wave; t < tile.rows && t < start + TILE; t += WAVES) {
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

    const int64_t left = tile.rows - start - wave * TOKENS;
    const int count = uniform((int)(left < 0 ? 0 : left < TOKENS ? left : TOKENS));
    const int64_t row = tile.row + start + wave * TOKENS;
    float sg[TOKENS][SHARED ? 1 : V];
    R xv[TOKENS], lv[TOKENS], uv[TOKENS], gv[TOKENS];
    float p[V], b[V], r[V];
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = 1.0f, b[v] = 0.0f, r[v] = 0.0f;
    // what the gradient of h_t is from y alone: u_t gy_t
    auto source = [&](int t, int v) {
        const float q = channel<V>(gv[t], v);
        return U ? q * channel<V>(uv[t], v) : q;
    };
    if (count > 0) {
        Walk<T> gp(s.gate, row, s.gate_stride), xp(s.x, row, s.x_stride), yp(g.gy, row, g.gy_stride);
        Walk<T> lp(s.lam, row, s.lam_stride), up(s.u, row, s.u_stride);
        RG raw[TOKENS];
#pragma unroll
        for (int t = 0; t < TOKENS; ++t) {
            raw[t] = gp.template at<RG>(dk);
            xv[t] = xp.template at<R>(dd);
            if constexpr (LAM) lv[t] = lp.template at<R>(dd);
            if constexpr (U) uv[t] = up.template at<R>(dd);
            gv[t] = R(0);
            if (g.gy) gv[t] = yp.template at<R>(dd);
            const bool more = t + 1 < count;   // rows behind the last read it again
            gp.down(more), xp.down(more), yp.down(more);
            if constexpr (LAM) lp.down(more);
            if constexpr (U) up.down(more);
        }
        hold();
        if (count < TOKENS)
#pragma unroll
            for (int t = 0; t < TOKENS; ++t)
                if (t >= count) {
                    no_row(raw[t], xv[t]);
                    gv[t] = R(0);
                    if constexpr (LAM) lv[t] = R(0);
                }
#pragma unroll
        for (int t = 0; t < TOKENS; ++t) {
            float most = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (v == 0 || !SHARED) sg[t][v] = gate_of(channel<SHARED ? 1 : V>(raw[t], v), most);
                const float a = sg[t][SHARED ? 0 : v];
                b[v] = keep(a, b[v], LAM ? channel<V>(lv[t], v) : take(a, most), channel<V>(xv[t], v));
                p[v] = keep(a, p[v]);
            }
        }
#pragma unroll
        for (int t = TOKENS - 1; t >= 0; --t)
#pragma unroll
            for (int v = 0; v < V; ++v) r[v] = keep(sg[t][SHARED ? 0 : v], source(t, v) + r[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        parts[wave][v][lane] = make_float2(p[v], b[v]);
        back[wave][v][lane] = r[v];
    }
    __syncthreads();
    float h0[V];                        // the state in front of this wave's tokens
    float pa[V], pb[V], ta[V], tb[V];   // the adjoint's stretches: behind this wave, (wave 0) the whole tile
    {
        float2 f[WAVES][V];
        float e[WAVES][V];
        const int64_t at = states_row(tile, s.offsets != nullptr, start, la.spacing);
#pragma unroll
        for (int q = 0; q < WAVES; ++q)
#pragma unroll
            for (int v = 0; v < V; ++v) f[q][v] = parts[q][v][lane], e[q][v] = back[q][v][lane];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            h0[v] = s.states[at * D + d + v];
            pa[v] = 1.0f, pb[v] = 0.0f, ta[v] = 1.0f, tb[v] = 0.0f;
        }
#pragma unroll
        for (int q = 0; q < WAVES; ++q)
            if (q < wave)
#pragma unroll
                for (int v = 0; v < V; ++v) h0[v] = fmaf(f[q][v].x, h0[v], f[q][v].y);
#pragma unroll
        for (int q = WAVES - 1; q >= 0; --q) {
            if (q > wave)
#pragma unroll
                for (int v = 0; v < V; ++v) pb[v] = fmaf(f[q][v].x, pb[v], e[q][v]), pa[v] *= f[q][v].x;
            if (wave == 0)
#pragma unroll
                for (int v = 0; v < V; ++v) tb[v] = fmaf(f[q][v].x, tb[v], e[q][v]), ta[v] *= f[q][v].x;
        }
    }
    float carry[V];   // what the token behind the tile hands to its last
    const int64_t behind = (tile.rows + TILE - 1) / TILE - 1 - tile.j;
    if (behind <= 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) carry[v] = g.gh_last ? g.gh_last[tile.n * D + d + v] : 0.0f;
    } else {
        if (wave == 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) publish(words + v * 64, product_bits(ta[v]), tb[v]);
            if (lane == 0) raise(flag, kHasProduct);
        }
        look_back<V, WAVES, WINDOW>(words, (int64_t)la.blocks * (64 * V), flag, 1, behind, wave, lane, board, &far, carry);
    }
    if (wave == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float out = fmaf(ta[v], carry[v], tb[v]);
            if (la.counters) publish(words + v * 64, kState, out);
            if (g.gh0 && valid && tile.j == 0) g.gh0[tile.n * D + d + v] = out;
        }
        if (la.counters && lane == 0) raise(flag, kHasState);
    }
    if (count <= 0 || !valid) return;   // groups of lanes that add up are valid or not as one
    float h[TOKENS + 1][V], G[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        G[v] = fmaf(pa[v], carry[v], pb[v]);   // R of the token behind
        h[0][v] = h0[v];
#pragma unroll
        for (int t = 0; t < TOKENS; ++t) {
            const float a = sg[t][SHARED ? 0 : v];
            h[t + 1][v] = keep(a, h[t][v], LAM ? channel<V>(lv[t], v) : take(a, 1.0f + a), channel<V>(xv[t], v));
        }
    }
    float sum[SHARED ? TOKENS : 1];   // a gate's gradient, of the lane's channels
    auto finish = [&](auto whole) {   // WHOLE: all of the wave's tokens, and all gradients
        constexpr bool WHOLE = decltype(whole)::value;
        const int64_t end = row + count - 1;   // the rows go up from the wave's last
        Walk<T> ox(g.gx, end, g.gx_stride), ol(g.glam, end, g.glam_stride), ou(g.gu, end, g.gu_stride);
        Walk<T> og(g.ggate, end, g.ggate_stride);
#pragma unroll
        for (int t = TOKENS - 1; t >= 0; --t) {
            if (WHOLE || t < count) {
                float vx[V], vl[V], vu[V], vg[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float a = sg[t][SHARED ? 0 : v];
                    const float x = channel<V>(xv[t], v), small = fabsf(a);
                    G[v] += source(t, v);
                    vx[v] = G[v] * (LAM ? channel<V>(lv[t], v) : take(a, 1.0f + a));
                    vl[v] = G[v] * x;
                    vu[v] = channel<V>(gv[t], v) * h[t + 1][v];
                    vg[v] = fmaf(-small, small, small) * G[v] * (LAM ? h[t][v] : h[t][v] - x);
                    G[v] = keep(a, G[v]);
                }
                if (WHOLE || g.gx) put(ox.out(dd), vx);
                if (LAM && (WHOLE || g.glam)) put(ol.out(dd), vl);
                if (U && (WHOLE || g.gu)) put(ou.out(dd), vu);
                if (!SHARED && (WHOLE || g.ggate)) put(og.out(dd), vg);
                ox.up();
                if constexpr (LAM) ol.up();
                if constexpr (U) ou.up();
                if constexpr (!SHARED) og.up();
                if constexpr (SHARED) {
                    sum[t] = vg[0];
                    if constexpr (V == 2) sum[t] += vg[1];
                }
            }
        }
        if constexpr (SHARED) {
            if (!WHOLE && !g.ggate) return;
            const int lanes = group / V;   // of a group; its last one ends up with the sum
            add_lanes(sum, lanes);
            if (lane % lanes != lanes - 1) return;
            if (partial) {
                const int64_t width = D / group;
                float* __restrict__ pp = partial + row * width + (uint32_t)d / (uint32_t)group;
#pragma unroll
                for (int t = 0; t < TOKENS; ++t) {
                    if (WHOLE || t < count) *pp = sum[t];
                    pp += width;
                }
            } else {
                Walk<T> og(g.ggate, row, g.ggate_stride);
#pragma unroll
                for (int t = 0; t < TOKENS; ++t) {
                    const float one[1] = {sum[t]};
                    if (WHOLE || t < count) put(og.out(dk), one);
                    og.down();
                }
            }
        }
    };
    if (count == TOKENS && g.gx && g.ggate && (!LAM || g.glam) && (!U || g.gu)) finish(Yes());
    else finish(No());
}

// ggate[t][k] = sum of the set's parts, for the rows of sequences.
template <typename T>
__global__ __launch_bounds__(256) void reduce_gate_kernel(gspn_seq s, gspn_seq_grad g, int group,
                                                          const float* __restrict__ partial) {
    const int64_t sets = s.D / s.ch_per_weight;
    const int parts = s.ch_per_weight / group;
    const int64_t given = s.offsets ? (int64_t)s.offsets[s.N] : s.T, rows = given < s.T ? given : s.T;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * sets; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / sets, k = i - t * sets;
        const float* __restrict__ p = partial + t * (s.D / group) + k * parts;
        float sum = 0.0f;
        for (int c = 0; c < parts; ++c) sum += p[c];
        static_cast<T*>(g.ggate)[t * g.ggate_stride + k] = from_f32(sum, (T*)nullptr);
    }
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
// V channels of a row: 16 bytes of state and 8 or 16 of the others where V is 4.
template <typename T> struct Four;
template <> struct Four<uint16_t> { typedef uint32_t type __attribute__((ext_vector_type(2))); };
template <> struct Four<float> { typedef float type __attribute__((ext_vector_type(4))); };

template <typename T, int V> __device__ __forceinline__ void get(const T* p, float (&v)[V]) {
    if constexpr (V == 1) {
        v[0] = to_f32(*p);
    } else {
        const typename Four<T>::type r = *reinterpret_cast<const typename Four<T>::type*>(p);
        if constexpr (sizeof(T) == 2) v[0] = bf16_lo(r.x), v[1] = bf16_hi(r.x), v[2] = bf16_lo(r.y), v[3] = bf16_hi(r.y);
        else v[0] = r.x, v[1] = r.y, v[2] = r.z, v[3] = r.w;
    }
}
template <typename T, int V> __device__ __forceinline__ void set(T* p, const float (&v)[V]) {
    if constexpr (V == 1) {
        *p = from_f32(v[0], p);
    } else {
        typename Four<T>::type r;
        if constexpr (sizeof(T) == 2) r.x = pack_bf16x2(v[0], v[1]), r.y = pack_bf16x2(v[2], v[3]);
        else r.x = v[0], r.y = v[1], r.z = v[2], r.w = v[3];
        *reinterpret_cast<typename Four<T>::type*>(p) = r;
    }
}

// One lane for V channels of a row, read and written once.  What bounds a step
// is the time of its few accesses behind one another, so a lane asks for all it
// needs before its workgroup knows whether the row is its own to take: rows of
// one slot are taken in their order by the lanes of the first of them.  256
// requests of 2560 channels in bf16: 7.7 us -> 4.6 (the bytes alone: 2.1); one
// request of 1152 channels: 3.6 -> 2.2, about what an empty launch takes.
constexpr int kStepLanes = 256;

template <typename T, int V, bool SHARED>
__global__ __launch_bounds__(kStepLanes) void seq_step_kernel(gspn_seq_token s, uint32_t blocks) {
    __shared__ int found[kStepLanes / 64];
    const uint32_t row = blockIdx.x / blocks;
    const int64_t d = (int64_t)(blockIdx.x - row * blocks) * (kStepLanes * V) + threadIdx.x * V;
    const int64_t slot = s.slots ? s.slots[row] : row;
    const bool mine = d < s.D;
    if (slot < 0 || slot >= s.S) {
        const float zero[V] = {};
        if ((s.flags & GSPN_SEQ_ZERO_TAIL) && mine) set<T, V>(static_cast<T*>(s.y) + row * s.y_stride + d, zero);
        return;
    }
    const uint32_t k = SHARED ? (uint32_t)d / (uint32_t)s.ch_per_weight : (uint32_t)d;
    float h[V], g[V], x[V], l[V], u[V];
    auto fetch = [&](int64_t r) {
        const T* gp = static_cast<const T*>(s.gate) + r * s.gate_stride;
        if constexpr (!SHARED) {
            get<T, V>(gp + d, g);
        } else if (V == 1 || s.ch_per_weight % 4 == 0) {
            g[0] = to_f32(gp[k]);
#pragma unroll
            for (int v = 1; v < V; ++v) g[v] = g[0];
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) g[v] = to_f32(gp[(uint32_t)(d + v) / (uint32_t)s.ch_per_weight]);
        }
        get<T, V>(static_cast<const T*>(s.x) + r * s.x_stride + d, x);
        if (s.lam) get<T, V>(static_cast<const T*>(s.lam) + r * s.lam_stride + d, l);
        if (s.u) get<T, V>(static_cast<const T*>(s.u) + r * s.u_stride + d, u);
    };
    if (mine) {
        get<float, V>(s.state + slot * s.D + d, h);
        fetch(row);
    }
    int others = 0;   // 1: an earlier row has the slot, 2: a later one
    if (s.slots && s.N > 1) {
        for (int64_t r = threadIdx.x; r < s.N; r += kStepLanes)
            if (r != row && s.slots[r] == slot) others |= r < row ? 1 : 2;
        const int any = (__ballot(others & 1) ? 1 : 0) | (__ballot(others & 2) ? 2 : 0);
        if ((threadIdx.x & 63) == 0) found[threadIdx.x >> 6] = any;
        __syncthreads();
        others = 0;
#pragma unroll
        for (int i = 0; i < kStepLanes / 64; ++i) others |= found[i];
    }
    if ((others & 1) || !mine) return;
    for (int64_t r = row;;) {
        float y[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float most;
            const float a = gate_of(g[v], most);
            h[v] = keep(a, h[v], s.lam ? l[v] : take(a, most), x[v]);
            y[v] = s.u ? u[v] * h[v] : h[v];
        }
        set<T, V>(static_cast<T*>(s.y) + r * s.y_stride + d, y);
        if (!(others & 2)) break;
        do ++r;
        while (r < s.N && s.slots[r] != slot);
        if (r >= s.N) break;
        fetch(r);
    }
    set<float, V>(s.state + slot * s.D + d, h);
}

// ---------------------------------------------------------------- host
Kind kind_of(const gspn_seq& s) { return kind_of(s.T, s.N, s.offsets != nullptr); }

// Tokens of a forward tile (bf16, lam and u):
//   512 sequences of 16 tokens, 2048 channels: 34 us with tiles of 32, 56 with 64;
//   16 rows of 2048, 1152 channels, a gate for 8: 75 us with 64, 83 with 128, 92 with 256;
//   40 sequences of 12001 tokens, 2048 channels: 49 us with 128 (two workgroups of
//   it fit a CU), 56 with 256;
//   one of 131072, 1024 channels, no lam or u: 220 us with 256, 271 with 128.
int forward_tile(const gspn_seq& s) {
    const Kind kind = kind_of(s);
    if (kind != kLong) return kind == kShort ? 32 : 64;
    return s.N * ((s.D + 127) / 128) >= 64 ? 128 : 256;
}

// The backward holds more for a token: at most 128, and a multiple of the spacing.
// With a gate for each channel 128 (12 equal rows of 704 tokens, 2048 channels in
// bf16: 85 us, 97 with 64; 16 of 4096, 512 channels: 157 and 176), or 32 where
// packed sequences are shorter.  Shared gates take less of a tile's registers and 64
// for all but the shortest and the longest (16 equal rows of 2048, 1152 channels, a
// gate for 8: 122 us, 136 with 128; 8192 packed tokens, 2048 channels, a gate for
// 128, sequences of 96 on average: 71 us, 84 with 32; of 200: 68, 78 with 128).
int backward_tile(const gspn_seq& s) {
    const Kind kind = kind_of(s);
    const int spacing = spacing_of(s.T, s.N, s.offsets != nullptr);
    if (kind == kShort) return 32;
    if (s.ch_per_weight > 1 && spacing <= 64 && (kind == kRows || s.T <= 512 * s.N)) return 64;
    return kind == kMiddle ? 32 : 128;
}

int tile_of(const gspn_seq& s, bool backward) { return backward ? backward_tile(s) : forward_tile(s); }

uint32_t tiles_of_sequence(const gspn_seq& s, int tile) {
    const int64_t rows = s.T / s.N;
    return (uint32_t)(rows > 0 ? (rows + tile - 1) / tile : 1);
}
uint32_t total_tiles(const gspn_seq& s, int tile) {
    return s.offsets ? (uint32_t)(s.T / tile + s.N + 1) : (uint32_t)s.N * tiles_of_sequence(s, tile);
}

// Whether a sequence may have two tiles.
bool tiles_wait(const gspn_seq& s, int tile) { return (s.offsets ? s.T : s.T / s.N) > tile; }

// What the workgroups tell each other: counters | flags | words.
int64_t counter_bytes(const gspn_seq& s) { return (s.D + 63) / 64 * 64; }   // 64 for the narrowest block

int64_t flags_bytes(const gspn_seq& s, int tile) {
    return ((s.D + 63) / 64 * total_tiles(s, tile) * 4 + 15) / 16 * 16;
}

int64_t words_bytes(const gspn_seq& s, int tile) {
    return (int64_t)total_tiles(s, tile) * ((s.D + 127) / 128 * 128) * 8;
}

int64_t exchange_bytes(const gspn_seq& s, int tile) {
    return tiles_wait(s, tile) ? counter_bytes(s) + flags_bytes(s, tile) + words_bytes(s, tile) : 0;
}

int power_of_two_in(int64_t v, int most) {
    int p = 1;
    while (p < most && v % (2 * p) == 0) p *= 2;
    return p;
}

bool even(const void* p, int64_t stride) { return ((uintptr_t)p & 3) == 0 && (!p || stride % 2 == 0); }

// Two channels a lane: bf16 rows whose pairs are whole 4-byte words, and no
// pair with two gates of a shared kind.
bool pairs(const gspn_seq& s) {
    return s.dtype == GSPN_BF16 && s.D % 2 == 0 && (s.ch_per_weight == 1 || s.ch_per_weight % 2 == 0) &&
           even(s.x, s.x_stride) && even(s.lam, s.lam_stride) && even(s.u, s.u_stride) &&
           (s.ch_per_weight > 1 || even(s.gate, s.gate_stride));
}

// The launch, with what the workgroups tell each other cleared.
Launch plan(const gspn_seq& s, int V, int tile, hipStream_t stream) {
    Launch la;
    la.blocks = (uint32_t)((s.D + 64 * V - 1) / (64 * V));
    la.tiles = s.offsets ? 0 : tiles_of_sequence(s, tile);
    la.total = total_tiles(s, tile);
    la.counters = nullptr;
    la.flags = nullptr;
    la.words = nullptr;
    la.spacing = spacing_of(s.T, s.N, s.offsets != nullptr);
    if (tiles_wait(s, tile)) {
        la.counters = static_cast<uint32_t*>(s.work);
        la.flags = la.counters + counter_bytes(s) / 4;
        la.words = reinterpret_cast<uint64_t*>(la.flags + flags_bytes(s, tile) / 4);
        const int64_t nc = (counter_bytes(s) + flags_bytes(s, tile)) / 16, nw = words_bytes(s, tile) / 16;
        const unsigned grid = (unsigned)std::min<int64_t>((nc + nw + 255) / 256, 2048);
        hipLaunchKernelGGL(seq_clear_kernel, dim3(grid), dim3(256), 0, stream, reinterpret_cast<uint4*>(la.counters),
                           nc, reinterpret_cast<uint4*>(la.words), nw);
    }
    return la;
}

// f(kernel) for the variant that the flags name.
template <typename T, int V, int TOKENS, int WAVES, typename F>
void fwd_variant(const gspn_seq& s, F f) {
    const bool lam = s.lam != nullptr, u = s.u != nullptr;
    if (s.ch_per_weight > 1) {
        if (lam) u ? f(seq_fwd_kernel<T, V, true, true, true, TOKENS, WAVES>) : f(seq_fwd_kernel<T, V, true, true, false, TOKENS, WAVES>);
        else u ? f(seq_fwd_kernel<T, V, true, false, true, TOKENS, WAVES>) : f(seq_fwd_kernel<T, V, true, false, false, TOKENS, WAVES>);
    } else {
        if (lam) u ? f(seq_fwd_kernel<T, V, false, true, true, TOKENS, WAVES>) : f(seq_fwd_kernel<T, V, false, true, false, TOKENS, WAVES>);
        else u ? f(seq_fwd_kernel<T, V, false, false, true, TOKENS, WAVES>) : f(seq_fwd_kernel<T, V, false, false, false, TOKENS, WAVES>);
    }
}

template <typename T, int V, int TOKENS, int WAVES, typename F>
void bwd_variant(const gspn_seq& s, F f) {
    const bool lam = s.lam != nullptr, u = s.u != nullptr;
    if (s.ch_per_weight > 1) {
        if (lam) u ? f(seq_bwd_kernel<T, V, true, true, true, TOKENS, WAVES>) : f(seq_bwd_kernel<T, V, true, true, false, TOKENS, WAVES>);
        else u ? f(seq_bwd_kernel<T, V, true, false, true, TOKENS, WAVES>) : f(seq_bwd_kernel<T, V, true, false, false, TOKENS, WAVES>);
    } else {
        if (lam) u ? f(seq_bwd_kernel<T, V, false, true, true, TOKENS, WAVES>) : f(seq_bwd_kernel<T, V, false, true, false, TOKENS, WAVES>);
        else u ? f(seq_bwd_kernel<T, V, false, false, true, TOKENS, WAVES>) : f(seq_bwd_kernel<T, V, false, false, false, TOKENS, WAVES>);
    }
}

template <int TOKENS, int WAVES>
void fwd_launch(const gspn_seq& s, hipStream_t stream) {
    const int V = pairs(s) && even(s.y, s.y_stride) ? 2 : 1;
    const Launch la = plan(s, V, TOKENS * WAVES, stream);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(la.total * la.blocks), dim3(WAVES * 64), 0, stream, s, la);
    };
    if (s.dtype == GSPN_F32) fwd_variant<float, 1, TOKENS, WAVES>(s, go);
    else if (V == 2) fwd_variant<uint16_t, 2, TOKENS, WAVES>(s, go);
    else fwd_variant<uint16_t, 1, TOKENS, WAVES>(s, go);
}

template <int TOKENS, int WAVES>
void bwd_launch(const gspn_seq& s, const gspn_seq_grad& g, hipStream_t stream) {
    const int V = pairs(s) && even(g.gy, g.gy_stride) && even(g.gx, g.gx_stride) && even(g.glam, g.glam_stride) &&
                          even(g.gu, g.gu_stride) && (s.ch_per_weight > 1 || even(g.ggate, g.ggate_stride))
                      ? 2 : 1;
    const Launch la = plan(s, V, TOKENS * WAVES, stream);
    const int group = power_of_two_in(s.ch_per_weight, 64 * V);
    float* partial = nullptr;
    if (group < s.ch_per_weight && g.ggate)
        partial = reinterpret_cast<float*>(static_cast<char*>(s.work) + exchange_bytes(s, TOKENS * WAVES));
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(la.total * la.blocks), dim3(WAVES * 64), 0, stream, s, g, la, group, partial);
    };
    if (s.dtype == GSPN_F32) bwd_variant<float, 1, TOKENS, WAVES>(s, go);
    else if (V == 2) bwd_variant<uint16_t, 2, TOKENS, WAVES>(s, go);
    else bwd_variant<uint16_t, 1, TOKENS, WAVES>(s, go);
    if (partial && s.T) {
        const dim3 grid((unsigned)std::min<int64_t>((s.T * (s.D / s.ch_per_weight) + 255) / 256, 4096));
        if (s.dtype == GSPN_BF16)
            hipLaunchKernelGGL(reduce_gate_kernel<uint16_t>, grid, dim3(256), 0, stream, s, g, group, partial);
        else
            hipLaunchKernelGGL(reduce_gate_kernel<float>, grid, dim3(256), 0, stream, s, g, group, partial);
    }
}

}  // namespace

int64_t seq_states_rows(int64_t T, int64_t N, bool packed) { return T / spacing_of(T, N, packed) + N; }

int64_t seq_workspace(const gspn_seq& s, bool backward) {
    int64_t bytes = exchange_bytes(s, tile_of(s, backward));
    const int group = power_of_two_in(s.ch_per_weight, 64);   // the smallest that a launch may take
    if (backward && group < s.ch_per_weight) bytes += s.T * (s.D / group) * 4;
    return bytes;
}

hipError_t launch_seq_fwd(const gspn_seq& s, hipStream_t stream) {
    switch (forward_tile(s)) {
        case 32: fwd_launch<8, 4>(s, stream); break;
        case 64: fwd_launch<16, 4>(s, stream); break;
        case 128: fwd_launch<32, 4>(s, stream); break;
        default: fwd_launch<32, 8>(s, stream); break;
    }
    return hipGetLastError();
}

hipError_t launch_seq_bwd(const gspn_seq& s, const gspn_seq_grad& g, hipStream_t stream) {
    switch (backward_tile(s)) {
        case 32: bwd_launch<8, 4>(s, g, stream); break;
        case 64: bwd_launch<8, 8>(s, g, stream); break;
        default: bwd_launch<16, 8>(s, g, stream); break;
    }
    return hipGetLastError();
}

hipError_t launch_seq_step(const gspn_seq_token& t, hipStream_t stream) {
    // four channels a lane where every row of four is a whole 16- or 8-byte piece
    auto fours = [&](const void* p, int64_t stride, size_t es) {
        return ((uintptr_t)p & (4 * es - 1)) == 0 && (!p || stride % 4 == 0);
    };
    const size_t es = t.dtype == GSPN_BF16 ? 2 : 4;
    const bool shared = t.ch_per_weight > 1;
    const int V = t.D % 4 == 0 && fours(t.state, 4, 4) && fours(t.x, t.x_stride, es) && fours(t.lam, t.lam_stride, es) &&
                          fours(t.u, t.u_stride, es) && fours(t.y, t.y_stride, es) &&
                          (shared || fours(t.gate, t.gate_stride, es))
                      ? 4 : 1;
    const uint32_t blocks = (uint32_t)((t.D + kStepLanes * V - 1) / (kStepLanes * V));
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)t.N * blocks), dim3(kStepLanes), 0, stream, t, blocks);
    };
    if (t.dtype == GSPN_BF16) {
        if (V == 4) shared ? go(seq_step_kernel<uint16_t, 4, true>) : go(seq_step_kernel<uint16_t, 4, false>);
        else shared ? go(seq_step_kernel<uint16_t, 1, true>) : go(seq_step_kernel<uint16_t, 1, false>);
    } else {
        if (V == 4) shared ? go(seq_step_kernel<float, 4, true>) : go(seq_step_kernel<float, 4, false>);
        else shared ? go(seq_step_kernel<float, 1, true>) : go(seq_step_kernel<float, 1, false>);
    }
    return hipGetLastError();
}

}  // namespace gspn
