// gspn_adapter.hip -- low-rank adapters of many requests beside a shared
// projection:  out[t] = base[t] + scale[i] b[i] (a[i] x[t]),  i = ids[request of t].
//
// Two launches over tiles of up to 64 rows of one request (gspn_rows.h):
//  * shrink_kernel: v[t] = a[i] x[t], r numbers a row in fp32.  The long axis K
//    is split over waves, which add up in LDS, and over `splits` workgroups,
//    whose sums stay apart in the workspace.
//  * expand_kernel: out[t] = base[t] + b[i] (scale[i] sum of the splits' v[t]),
//    64 columns of 16 rows at a time.
// Both are matrix products on the matrix cores, with 2 r operations for every
// element of x and base: memory bounds them at any rank allowed.  An operand's
// lanes hold different rows, so loading operands straight from memory asks for 64
// addresses far apart with every instruction (16384 tokens, 4096 columns, r 64 in
// bf16: 198 us for both launches); so every tile comes in whole row pieces, eight
// lanes to 128 bytes of a row, and is turned in LDS, and the results go out the
// same way.  What the next tile needs is loaded while the present one is multiplied.
//
// Measured in bf16 (shrink + expand):
//   8 requests of 16384 tokens in all, 4096 -> 4096, r 64: 38 + 66 us, where x,
//   base and out alone are 80 us at a copy's 5.1 TB/s;
//   64 requests of 2560 tokens (prompts and single tokens), 4096 -> 4096, r 16:
//   8.5 + 15 to 21 us (the bytes: 14.6); a wave has four turns of 64 columns there,
//   and the chain of note, v and b in front of the first costs as much as they do;
//   one token of one request, 1152 -> 1152, r 8: 3.3 + 4.4 us, two empty launches.
//
// Rows need not be aligned to 16 bytes: the pieces are read and written at
// their elements' alignment, which the memory pipeline takes.
#include "gspn_device.h"
#include "gspn_kernels.h"
#include "gspn_rows.h"

#include <type_traits>

namespace gspn {
namespace {

constexpr int kRows = 64;     // rows of a tile
constexpr int kRB = kRows / 16;
constexpr int kRanks = 64;    // ranks of a shrink workgroup
constexpr int kWaves = 4;     // of a workgroup
constexpr int kSplits = 16;   // workgroups that share K, at most

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------- operands
// Eight neighbouring elements along the summed axis: lane l holds row (or
// column) l % 16 and the elements 8 (l / 16) .. + 7 of a step of 32.
template <typename T> struct Frag;
template <> struct Frag<uint16_t> { bf16x8 v; };
template <> struct Frag<float> { float v[8]; };

__device__ __forceinline__ void zero(Frag<uint16_t>& f) { f.v = __builtin_bit_cast(bf16x8, u32x4{0, 0, 0, 0}); }
__device__ __forceinline__ void zero(Frag<float>& f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f.v[e] = 0.0f;
}

// 16 and 8 bytes at the alignment of their elements.
template <typename T> struct Piece;
template <> struct Piece<uint16_t> {
    typedef uint32_t x4 __attribute__((ext_vector_type(4), aligned(2)));
    typedef uint32_t x2 __attribute__((ext_vector_type(2), aligned(2)));
};
template <> struct Piece<float> { typedef float x4 __attribute__((ext_vector_type(4), aligned(4))); };

__device__ __forceinline__ Frag<uint16_t> load8(const uint16_t* __restrict__ p) {
    Frag<uint16_t> f;
    f.v = __builtin_bit_cast(bf16x8, (u32x4)*reinterpret_cast<const Piece<uint16_t>::x4*>(p));
    return f;
}
__device__ __forceinline__ Frag<float> load8(const float* __restrict__ p) {
    Frag<float> f;
    const f32x4 lo = *reinterpret_cast<const Piece<float>::x4*>(p), hi = *reinterpret_cast<const Piece<float>::x4*>(p + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) f.v[e] = lo[e], f.v[4 + e] = hi[e];
    return f;
}
// Those of p[0 .. 7] in front of `left`, and zeros.
__device__ __forceinline__ Frag<uint16_t> load8(const uint16_t* __restrict__ p, int64_t left) {
    if (left >= 8) return load8(p);
    Frag<uint16_t> f;
    zero(f);
    if (left <= 0) return f;
    if (left == 4) {
        const auto v = *reinterpret_cast<const Piece<uint16_t>::x2*>(p);
        f.v = __builtin_bit_cast(bf16x8, u32x4{v.x, v.y, 0, 0});
        return f;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < left) f.v[e] = __builtin_bit_cast(__bf16, p[e]);
    return f;
}
__device__ __forceinline__ Frag<float> load8(const float* __restrict__ p, int64_t left) {
    if (left >= 8) return load8(p);
    Frag<float> f;
    zero(f);
    if (left >= 4) {
        const f32x4 v = *reinterpret_cast<const Piece<float>::x4*>(p);
#pragma unroll
        for (int e = 0; e < 4; ++e) f.v[e] = v[e];
#pragma unroll
        for (int e = 4; e < 7; ++e)
            if (e < left) f.v[e] = p[e];
        return f;
    }
#pragma unroll
    for (int e = 0; e < 3; ++e)
        if (e < left) f.v[e] = p[e];
    return f;
}

// p[0 .. 3] in the low half of a piece.
__device__ __forceinline__ void load4(Frag<uint16_t>& f, int half, const uint16_t* __restrict__ p) {
    const auto v = *reinterpret_cast<const Piece<uint16_t>::x2*>(p);
    u32x4 w = __builtin_bit_cast(u32x4, f.v);
    w[2 * half] = v.x, w[2 * half + 1] = v.y;
    f.v = __builtin_bit_cast(bf16x8, w);
}
__device__ __forceinline__ void load4(Frag<float>& f, int half, const float* __restrict__ p) {
    const f32x4 v = *reinterpret_cast<const Piece<float>::x4*>(p);
#pragma unroll
    for (int e = 0; e < 4; ++e) f.v[4 * half + e] = v[e];
}
__device__ __forceinline__ void keep4(uint16_t* p, const Frag<uint16_t>& f, int half) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const u32x4 w = __builtin_bit_cast(u32x4, f.v);
    *reinterpret_cast<u32x2*>(p) = u32x2{w[2 * half], w[2 * half + 1]};
}
__device__ __forceinline__ void keep4(float* p, const Frag<float>& f, int half) {
    *reinterpret_cast<f32x4*>(p) = f32x4{f.v[4 * half], f.v[4 * half + 1], f.v[4 * half + 2], f.v[4 * half + 3]};
}

// Lanes of a wave hand each other data through LDS.  A wave's accesses to LDS
// complete in their order; this keeps the compiler to that order.
__device__ __forceinline__ void handover() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Eight elements to and from LDS (16-byte aligned there).
__device__ __forceinline__ void keep8(uint16_t* p, const Frag<uint16_t>& f) { *reinterpret_cast<bf16x8*>(p) = f.v; }
__device__ __forceinline__ void keep8(float* p, const Frag<float>& f) {
    *reinterpret_cast<f32x4*>(p) = f32x4{f.v[0], f.v[1], f.v[2], f.v[3]};
    *reinterpret_cast<f32x4*>(p + 4) = f32x4{f.v[4], f.v[5], f.v[6], f.v[7]};
}
__device__ __forceinline__ Frag<uint16_t> kept8(const uint16_t* p) {
    Frag<uint16_t> f;
    f.v = *reinterpret_cast<const bf16x8*>(p);
    return f;
}
__device__ __forceinline__ Frag<float> kept8(const float* p) {
    Frag<float> f;
    const f32x4 lo = *reinterpret_cast<const f32x4*>(p), hi = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) f.v[e] = lo[e], f.v[4 + e] = hi[e];
    return f;
}

// c[m][n] += sum over a step of 32 of a[m][k] b[n][k].  Lane l holds
// c[4 (l / 16) + 0 .. 3][l % 16].  fp32 takes eight products of four elements;
// which element of the step is the e-th lane group's does not matter as long
// as both operands agree.
__device__ __forceinline__ void multiply(f32x4& c, const Frag<uint16_t>& a, const Frag<uint16_t>& b) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ void multiply(f32x4& c, const Frag<float>& a, const Frag<float>& b) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], c, 0, 0, 0);
}

// fp32 numbers as an operand.  bf16: as two parts, the number rounded and what
// the rounding left, rounded (2^-18 of the number is lost instead of 2^-9; the
// second product costs nothing next to the rows' bytes).
template <typename T> struct Parts;
template <> struct Parts<uint16_t> {
    Frag<uint16_t> hi, lo;
    __device__ void set(int e, float v) {
        hi.v[e] = (__bf16)v;
        const float rest = v - (float)hi.v[e];
        lo.v[e] = (__bf16)(fabsf(rest) < __builtin_inff() ? rest : 0.0f);   // an infinity has no rest
    }
};
template <> struct Parts<float> {
    Frag<float> hi;
    __device__ void set(int e, float v) { hi.v[e] = v; }
};
__device__ __forceinline__ void multiply(f32x4& c, const Frag<uint16_t>& a, const Parts<uint16_t>& b) {
    multiply(c, a, b.lo);
    multiply(c, a, b.hi);
}
__device__ __forceinline__ void multiply(f32x4& c, const Frag<float>& a, const Parts<float>& b) { multiply(c, a, b.hi); }

// What shrink_kernel finds out about a tile and expand_kernel reads back in one
// load (finding the tile, its adapter and its scale takes four that wait for
// each other).
struct __attribute__((aligned(16))) TileNote {
    int32_t row, count;   // first row, rows (0: nothing to do)
    int32_t id;           // the adapter, kNone or kTail
    float scale;
};
constexpr int32_t kNone = -1, kTail = -2;   // a request without an adapter; rows of no request

struct Launch {
    TileNote* notes;    // [total]
    float* v;           // [splits][T][pitch]
    uint32_t tiles;     // of a request (rows of equal length), else 0
    uint32_t total;     // of all
    uint32_t groups;    // shrink: groups of kRanks ranks
    uint32_t splits;    // shrink: workgroups that share K
    int64_t slice;      // shrink: K of a workgroup, a multiple of 64
    int64_t pitch;      // ranks of a row of v: r rounded up to 16
    uint32_t parts;     // expand: workgroups that share M
    int64_t columns;    // expand: columns of a workgroup, a multiple of 256
};

// ---------------------------------------------------------------- shrink
// RB: blocks of 16 ranks of the workgroup.  A wave turns its own tiles in LDS of
// its own: no barriers before the waves' sums are added, in a fixed order.
template <typename T, int RB, int WAVES>
__global__ __launch_bounds__(WAVES * 64, 2) void shrink_kernel(gspn_adapter s, Launch la) {
    constexpr int kWide = 128 / sizeof(T);          // elements of K of a wave's tile: 128 bytes of a row
    constexpr int kPitch = kWide + 16 / sizeof(T);  // in LDS; 16 bytes more spread the rows over the banks
    constexpr int kPieces = kWide / 8;              // pieces of eight elements of a row
    constexpr int kAtOnce = 64 / kPieces;           // rows of a wave's load
    constexpr int kStage = (kRB + RB) * 16 * kPitch * sizeof(T);   // bytes of LDS of a wave
    __shared__ __attribute__((aligned(16))) char lds[WAVES * kStage];
    static_assert(kStage >= kRB * RB * 64 * 16, "the sums take the tiles' place");
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int q = lane >> 4, c = lane & 15;
    const uint32_t split = blockIdx.x % la.splits, rest = blockIdx.x / la.splits;
    const uint32_t group = rest % la.groups, w = rest / la.groups;
    const Tile tile = find_tile<kRows>(s.offsets, s.T, s.N, la.tiles, w, lane, first_offsets(s.offsets, s.N, lane));
    const int64_t start = tile.j * kRows;
    const int64_t left = tile.rows - start;
    const int count = uniform((int)(left < 0 ? 0 : left < kRows ? left : kRows));
    const int64_t row = tile.row + start;
    int64_t id = tile.n == s.N ? kTail : s.ids[tile.n];
    if (tile.n != s.N && (id < 0 || id >= s.R)) id = kNone;
    if (split == 0 && group == 0 && threadIdx.x == 0)
        la.notes[w] = TileNote{(int32_t)row, count, (int32_t)id, id >= 0 && s.scale ? s.scale[id] : 1.0f};
    if (count == 0 || id < 0) return;
    const int64_t end = ((int64_t)split + 1) * la.slice < s.K ? ((int64_t)split + 1) * la.slice : s.K;
    f32x4* sums = reinterpret_cast<f32x4*>(lds);    // [WAVES][kRB * RB][64]

    auto products = [&](auto blocks) {
        constexpr int NB = decltype(blocks)::value;                       // blocks of 16 rows
        constexpr int NX = NB * 16 / kAtOnce, NA = RB * 16 / kAtOnce;     // loads of a tile
        T* xs = reinterpret_cast<T*>(lds + wave * kStage);
        T* as = xs + NB * 16 * kPitch;
        const int piece = lane % kPieces, line = lane / kPieces;
        const T* __restrict__ xp[NX];
        const T* __restrict__ ap[NA];
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int t = i * kAtOnce + line;   // rows behind the last read it again
            xp[i] = static_cast<const T*>(s.x) + (row + (t < count ? t : count - 1)) * s.x_stride + 8 * piece;
        }
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            // ranks behind the last likewise; their sums are not kept
            const int64_t j = (int64_t)group * kRanks + i * kAtOnce + line;
            ap[i] = static_cast<const T*>(s.a) + (id * s.r + (j < s.r ? j : s.r - 1)) * s.K + 8 * piece;
        }
        Frag<T> x[NX], a[NA];
        auto load = [&](int64_t k) {
            if (k + kWide <= end) {
#pragma unroll
                for (int i = 0; i < NX; ++i) x[i] = load8(xp[i] + k);
#pragma unroll
                for (int i = 0; i < NA; ++i) a[i] = load8(ap[i] + k);
            } else {
                const int64_t left = end - k - 8 * piece;
#pragma unroll
                for (int i = 0; i < NX; ++i) x[i] = load8(xp[i] + k, left);
#pragma unroll
                for (int i = 0; i < NA; ++i) a[i] = load8(ap[i] + k, left);
            }
        };
        f32x4 acc[NB][RB] = {};
        int64_t k = (int64_t)split * la.slice + wave * kWide;
        if (k < end) load(k);
        for (; k < end; k += WAVES * kWide) {
#pragma unroll
            for (int i = 0; i < NX; ++i) keep8(xs + (i * kAtOnce + line) * kPitch + 8 * piece, x[i]);
#pragma unroll
            for (int i = 0; i < NA; ++i) keep8(as + (i * kAtOnce + line) * kPitch + 8 * piece, a[i]);
            handover();
            if (k + WAVES * kWide < end) load(k + WAVES * kWide);
#pragma unroll
            for (int h = 0; h < kWide / 32; ++h) {
                Frag<T> fa[RB];
#pragma unroll
                for (int i = 0; i < RB; ++i) fa[i] = kept8(as + (i * 16 + c) * kPitch + 32 * h + 8 * q);
#pragma unroll
                for (int t = 0; t < NB; ++t) {
                    const Frag<T> fx = kept8(xs + (t * 16 + c) * kPitch + 32 * h + 8 * q);
#pragma unroll
                    for (int i = 0; i < RB; ++i) multiply(acc[t][i], fa[i], fx);
                }
            }
            handover();
        }
        __syncthreads();   // every wave is done with its tiles
#pragma unroll
        for (int t = 0; t < NB; ++t)
#pragma unroll
            for (int i = 0; i < RB; ++i) sums[(wave * kRB * RB + t * RB + i) * 64 + lane] = acc[t][i];
    };
    // one block of rows, or all four (rows behind the last are copies of it)
    if (count <= 16) products(std::integral_constant<int, 1>());
    else products(std::integral_constant<int, kRB>());
    __syncthreads();
    float* __restrict__ v = la.v + (size_t)split * s.T * la.pitch;
    for (int b = wave; b < kRB * RB; b += WAVES) {
        const int t = (b / RB) * 16 + c, i = b % RB;
        if (t >= count) continue;
        f32x4 sum = sums[b * 64 + lane];
#pragma unroll
        for (int o = 1; o < WAVES; ++o) sum += sums[(o * kRB * RB + b) * 64 + lane];
        const int64_t j = (int64_t)group * kRanks + i * 16 + 4 * q;
        if (j >= la.pitch) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (j + e >= s.r) sum[e] = 0.0f;
        *reinterpret_cast<f32x4*>(v + (size_t)(row + t) * la.pitch + j) = sum;
    }
}

// ---------------------------------------------------------------- expand
// STEPS: steps of 32 ranks whose v a wave keeps for all its columns; 0: any
// number, one or two steps at a time, v is read again for every 64 columns.
// PIECE: 8 or 4 where r is a multiple of it (b comes in pieces of that many
// elements, 64 columns as one stretch of memory), else 1 (a column a lane).
//
// The waves of a tile of more than 16 rows have 16 rows each and walk the same
// columns: each brings a quarter of b's and they share it (two buffers, a
// barrier a turn; 86 -> 76 us with it at r 64).  The waves of up to 16 rows have
// columns of their own.  base is asked for one turn ahead: 70 us; with
// none ahead 73, with two 72, and more came out slower still.
//
// Two steps in 16 bits fit four workgroups on a CU with five registers put
// aside (16384 tokens, 4096 columns, r 64: 71 -> 66 us); the others' loops
// would spill, or fit already.
template <typename T, int STEPS, int PIECE>
__global__ __launch_bounds__(kWaves * 64, STEPS == 2 && PIECE == 8 && sizeof(T) == 2 ? 4 : 2) void expand_kernel(gspn_adapter s, Launch la) {
    constexpr int kSteps = STEPS ? STEPS : sizeof(T) == 2 ? 2 : 1;
    constexpr int kPitch = 32 * kSteps + 16 / sizeof(T);   // of b's rows in LDS
    constexpr int kOPitch = 64 + 4;                        // of a row of sums, fp32
    constexpr int kStage = 64 * kPitch * sizeof(T);        // bytes of LDS of 64 columns of b
    constexpr int kSums = 16 * kOPitch * 4;                // of a wave's sums
    static_assert(kStage >= kSums, "the sums take the place of a wave's own b");
    constexpr int kLds = kWaves * kStage > 2 * kStage + kWaves * kSums ? kWaves * kStage : 2 * kStage + kWaves * kSums;
    constexpr int kPart = PIECE > 1 ? PIECE : 8;
    constexpr int kOut = 16 * 64 * sizeof(T) / 1024;       // 16-byte pieces of base for a lane
    constexpr int kPer = 16 / sizeof(T);                   // elements of such a piece
    __shared__ __attribute__((aligned(16))) char lds[kLds];
    typedef typename Piece<T>::x4 Out;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int q = lane >> 4, c = lane & 15;
    const uint32_t part = blockIdx.x % la.parts, w = blockIdx.x / la.parts;
    const TileNote note = la.notes[w];
    const int count = uniform(note.count);
    const int64_t id = uniform(note.id);
    if (count == 0) return;
    const T* base = static_cast<const T*>(s.base);   // may be out itself: a lane reads what it then writes
    T* out = static_cast<T*>(s.out);
    int64_t first = part * la.columns;
    const int64_t last = first + la.columns < s.M ? first + la.columns : s.M;
    const int block = count <= 16 ? 0 : wave, stride = count <= 16 ? 64 * kWaves : 64;
    if (count <= 16) first += 64 * wave;
    const int mine = count - block * 16 < 16 ? count - block * 16 : 16;   // rows of this wave, if any
    const int64_t row = uniform(note.row) + block * 16;
    if (id < 0) {
        // rows of no request (zero, or as they were), or of one without an adapter (base's)
        if (id == kTail ? !(s.flags & GSPN_SEQ_ZERO_TAIL) : base == out) return;
        for (int t = 0; t < mine; ++t)
            for (int64_t m = first + lane; m < last; m += stride)
                out[(row + t) * s.out_stride + m] =
                    id == kTail ? from_f32(0.0f, (T*)nullptr) : base[(row + t) * s.base_stride + m];
        return;
    }
    const T* __restrict__ bp = static_cast<const T*>(s.b) + id * s.M * s.r;
    const float scale = note.scale;
    // v of the lane's row, ranks 32 k + 8 q .. + 7: the splits' sums, scaled
    // (rows behind the last read it again)
    const float* __restrict__ vp =
        la.v + (size_t)(row + (c < mine ? c : mine - 1)) * la.pitch + 8 * q;
    auto load_v = [&](int k) {
        f32x4 lo = {}, hi = {};
        if (32 * k + 8 * q < la.pitch) {
            const float* __restrict__ p = vp + 32 * k;
            for (uint32_t i = 0; i < la.splits; ++i, p += s.T * la.pitch) {
                lo += *reinterpret_cast<const f32x4*>(p);
                hi += *reinterpret_cast<const f32x4*>(p + 4);
            }
        }
        Parts<T> f;
#pragma unroll
        for (int e = 0; e < 4; ++e) f.set(e, scale * lo[e]), f.set(4 + e, scale * hi[e]);
        return f;
    };
    // base of 16 rows of 64 columns, in pieces of whole rows
    constexpr int kLine = 64 / kPer;   // lanes of a row
    const int oc = (lane % kLine) * kPer, orow = lane / kLine;

    auto walk = [&](auto shared) {
        constexpr bool SHARED = decltype(shared)::value;
        constexpr int kBring = 4 * kSteps * 8 / kPart / (SHARED ? kWaves : 1);   // pieces of b for a lane, at most
        const int from = SHARED ? wave : 0, by = SHARED ? kWaves : 1;
        float* os = reinterpret_cast<float*>(SHARED ? lds + 2 * kStage + wave * kSums : lds + wave * kStage);
        Frag<T> b[kBring * kPart / 8 > 0 ? kBring * kPart / 8 : 1];
        int place[STEPS && PIECE > 1 ? kBring : 1];   // where in LDS a lane's pieces go
        if constexpr (STEPS != 0 && PIECE > 1) {
            const int pieces = (int)s.r / PIECE;   // of a column
#pragma unroll
            for (int i = 0; i < kBring; ++i) {
                const int e = (i * by + from) * 64 + lane;
                place[i] = (e / pieces) * kPitch + PIECE * (e % pieces);
            }
        }
        // 64 columns of b and up to 32 kSteps ranks from rank j0 on
        auto load_b = [&](int64_t m, int64_t j0) {
            const int ranks = (int)(s.r - j0 < 32 * kSteps ? s.r - j0 : 32 * kSteps);
            const int pieces = ranks / kPart;
#pragma unroll
            for (int i = 0; i < kBring; ++i) {
                if (i * by + from < pieces) {
                    const int e = (i * by + from) * 64 + lane;
                    int64_t at;   // columns behind the last read what is in front of them
                    if constexpr (STEPS != 0) {
                        at = m * s.r + (int64_t)e * PIECE;
                        if (at > s.M * s.r - PIECE) at = s.M * s.r - PIECE;
                    } else {
                        const int64_t o = m + e / pieces;
                        at = (o < s.M ? o : s.M - 1) * s.r + j0 + PIECE * (e % pieces);
                    }
                    if constexpr (PIECE == 8) b[i] = load8(bp + at);
                    else load4(b[i / 2], i % 2, bp + at);
                }
            }
        };
        // into rows of LDS, zeros behind the last rank
        auto keep_b = [&](T* bs, int64_t m, int64_t j0) {
            const int ranks = (int)(s.r - j0 < 32 * kSteps ? s.r - j0 : 32 * kSteps);
            if constexpr (PIECE > 1) {
                const int pieces = ranks / PIECE;
#pragma unroll
                for (int i = 0; i < kBring; ++i) {
                    if (i * by + from < pieces) {
                        const int e = (i * by + from) * 64 + lane;
                        T* p = bs + (STEPS ? place[STEPS ? i : 0] : (e / pieces) * kPitch + PIECE * (e % pieces));
                        if constexpr (PIECE == 8) keep8(p, b[i]);
                        else keep4(p, b[i / 2], i % 2);
                    }
                }
                Frag<T> none;
                zero(none);
                for (int j = ranks + PIECE * q; j < (ranks + 31) / 32 * 32; j += 4 * PIECE)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (SHARED && i != wave) continue;
                        T* p = bs + (16 * i + c) * kPitch + j;
                        if constexpr (PIECE == 8) keep8(p, none);
                        else keep4(p, none, 0);
                    }
            } else {
                const int64_t o = m + lane < s.M ? m + lane : s.M - 1;   // columns behind the last read it again
                const T* __restrict__ p = bp + o * s.r + j0;
                for (int j = 8 * from; j < (ranks + 31) / 32 * 32; j += 8 * by)
                    keep8(bs + lane * kPitch + j, load8(p + j, ranks - j));
            }
        };
        Out old[kOut];
        auto load_base = [&](int64_t m) {
#pragma unroll
            for (int i = 0; i < kOut; ++i) {
                const int t = i * (64 / kLine) + orow;
                if (t < mine && m + oc + kPer <= s.M)
                    old[i] = *reinterpret_cast<const Out*>(base + (row + t) * s.base_stride + m + oc);
            }
        };
        if constexpr (PIECE > 1) load_b(first, 0);
        if (first < last) load_base(first);
        Parts<T> v[kSteps];
#pragma unroll
        for (int k = 0; k < STEPS; ++k) v[k] = load_v(k);
        int buffer = 0;
        for (int64_t m = first; m < last; m += stride) {
            f32x4 acc[4] = {};
            Out now[kOut];
#pragma unroll
            for (int i = 0; i < kOut; ++i) now[i] = old[i];
            const bool more = m + stride < last;
            for (int64_t j0 = 0; j0 < (STEPS ? 1 : s.r); j0 += 32 * kSteps, buffer ^= 1) {
                T* bs = reinterpret_cast<T*>(lds + (SHARED ? buffer : wave) * kStage);
                keep_b(bs, m, j0);
                if constexpr (SHARED) __syncthreads();
                else handover();
                const int64_t next = j0 + 32 * kSteps;
                if constexpr (PIECE > 1) {
                    if (STEPS == 0 && next < s.r) load_b(m, next);
                    else if (more) load_b(m + stride, 0);
                }
                if (j0 == 0 && more) load_base(m + stride);
                if constexpr (STEPS == 0) {
#pragma unroll
                    for (int k = 0; k < kSteps; ++k) v[k] = load_v((int)(j0 / 32) + k);
                }
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
                    if (j0 + 32 * k < s.r)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            multiply(acc[i], kept8(bs + (16 * i + c) * kPitch + 32 * k + 8 * q), v[k]);
                handover();
            }
            // lane l holds row c of the columns 16 i + 4 q .. + 3
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<f32x4*>(os + c * kOPitch + 16 * i + 4 * q) = acc[i];
            handover();
#pragma unroll
            for (int i = 0; i < kOut; ++i) {
                const int t = i * (64 / kLine) + orow;
                float sum[kPer];
#pragma unroll
                for (int e = 0; e < kPer; e += 4) {
                    const f32x4 f = *reinterpret_cast<const f32x4*>(os + t * kOPitch + oc + e);
#pragma unroll
                    for (int k = 0; k < 4; ++k) sum[e + k] = f[k];
                }
                if (t >= mine) continue;
                const int64_t left = s.M - m - oc;
                T* po = out + (row + t) * s.out_stride + m + oc;
                if (left >= kPer) {
                    Out o;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (sizeof(T) == 2)
                            o[e] = pack_bf16x2(bf16_lo(now[i][e]) + sum[2 * e], bf16_hi(now[i][e]) + sum[2 * e + 1]);
                        else
                            o[e] = now[i][e] + sum[e];
                    }
                    *reinterpret_cast<Out*>(po) = o;
                } else {
                    const T* pb = base + (row + t) * s.base_stride + m + oc;
#pragma unroll
                    for (int e = 0; e < kPer - 1; ++e)
                        if (e < left) po[e] = from_f32(to_f32(pb[e]) + sum[e], (T*)nullptr);
                }
            }
            handover();
        }
    };
    if (count <= 16) walk(std::integral_constant<bool, false>());
    else walk(std::integral_constant<bool, true>());
}

// ---------------------------------------------------------------- host
// Waves of a shrink workgroup: eight where a wave's tiles are so large that a CU
// holds eight at all; then rows with a workgroup for each CU need no splits,
// which the second launch would read one by one (16384 tokens, r 64: expand 77 -> 72
// us; 2395 tokens of 27 requests, r 128: 26 -> 21).
int shrink_waves(const gspn_adapter& s) { return s.r > 32 ? 8 : 4; }

// Sizes of the launches; the workspace holds the tiles' notes and v.
Launch plan(const gspn_adapter& s) {
    Launch la;
    la.tiles = s.offsets ? 0 : tiles_of_sequence<kRows>(s.T, s.N);
    la.total = total_tiles<kRows>(s.offsets, s.T, s.N);
    la.groups = (uint32_t)((s.r + kRanks - 1) / kRanks);
    la.pitch = (s.r + 15) / 16 * 16;
    // K is shared by more workgroups while there are fewer than eight waves for a
    // CU, as long as each has 64 of it
    const int64_t blocks = (s.K + 63) / 64, waves = shrink_waves(s);
    const int64_t most = std::min<int64_t>(kSplits, (blocks + waves - 1) / waves);
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(most, 2048 / waves / ((int64_t)la.total * la.groups)));
    la.slice = (blocks + want - 1) / want * 64;
    la.splits = (uint32_t)((s.K + la.slice - 1) / la.slice);
    // a workgroup takes up to 1024 columns while workgroups are many
    int64_t columns = 256;
    while (columns < 1024 && la.total * ((s.M + columns - 1) / columns) > 2048) columns *= 2;
    la.columns = columns;
    la.parts = (uint32_t)((s.M + columns - 1) / columns);
    la.notes = static_cast<TileNote*>(s.work);
    la.v = reinterpret_cast<float*>(la.notes + la.total);
    return la;
}

template <typename T, int PIECE, typename F>
void expand_pieces(const gspn_adapter& s, F f) {
    if (s.r <= 32) f(expand_kernel<T, 1, PIECE>);
    else if (s.r <= 64) f(expand_kernel<T, 2, PIECE>);
    else if (sizeof(T) == 2 && s.r <= 128) f(expand_kernel<T, sizeof(T) == 2 ? 4 : 0, PIECE>);
    else f(expand_kernel<T, 0, PIECE>);
}

template <typename T>
void launch_typed(const gspn_adapter& s, const Launch& la, hipStream_t stream) {
    const dim3 gs(la.total * la.groups * la.splits), ge(la.total * la.parts);
    auto shrink = [&](auto kernel) { hipLaunchKernelGGL(kernel, gs, dim3(shrink_waves(s) * 64), 0, stream, s, la); };
    auto expand = [&](auto kernel) { hipLaunchKernelGGL(kernel, ge, dim3(kWaves * 64), 0, stream, s, la); };
    if (s.r <= 16) shrink(shrink_kernel<T, 1, 4>);
    else if (s.r <= 32) shrink(shrink_kernel<T, 2, 4>);
    else shrink(shrink_kernel<T, 4, 8>);
    if (s.r % 8 == 0) expand_pieces<T, 8>(s, expand);
    else if (s.r % 4 == 0) expand_pieces<T, 4>(s, expand);
    else expand_pieces<T, 1>(s, expand);
}

}  // namespace

int64_t adapter_workspace(const gspn_adapter& s) {
    const Launch la = plan(s);
    return (int64_t)la.total * (int64_t)sizeof(TileNote) + (int64_t)la.splits * s.T * la.pitch * 4;
}

hipError_t launch_adapter(const gspn_adapter& s, hipStream_t stream) {
    const Launch la = plan(s);
    if (s.dtype == GSPN_BF16) launch_typed<uint16_t>(s, la, stream);
    else launch_typed<float>(s, la, stream);
    return hipGetLastError();
}

}  // namespace gspn
