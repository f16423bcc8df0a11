// gspn_adapter.hip -- low-rank adapters of many requests beside a shared
// projection:  out[t] = base[t] + scale[i] b[i] (a[i] x[t]),  i = ids[request of t].
//
// Two launches over tiles of up to 64 rows of one request (gspn_rows.h):
//  * shrink_kernel: v[t] = a[i] x[t], r numbers a row in fp32.  The long axis K
//    is split over the four waves of a workgroup, which add up in LDS, and over
//    `splits` workgroups, whose sums stay apart in the workspace.
//  * expand_kernel: out[t] = base[t] + b[i] (scale[i] sum of the splits' v[t]);
//    a wave owns the tile's rows of 64 columns at a time.
// Both are matrix products on the matrix cores, with the adapter as the left
// operand: lane l of a wave ends up with row l % 16 of the tile's, and
// neighbouring ranks (columns) of it, so that v and out are written in whole
// 16-byte pieces.  Tiles of up to 16 rows do a quarter of a full tile's
// products: what a single token waits for is its adapter.
#include "gspn_device.h"
#include "gspn_kernels.h"
#include "gspn_rows.h"

#include <type_traits>

namespace gspn {
namespace {

constexpr int kRows = 64;     // rows of a tile
constexpr int kRB = kRows / 16;
constexpr int kRanks = 64;    // ranks of a shrink workgroup
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

// p[0 .. 7], or those of them in front of `left` and zeros.  VEC: p is 16-byte
// aligned and `left` a multiple of 8.
template <bool VEC>
__device__ __forceinline__ Frag<uint16_t> load8(const uint16_t* __restrict__ p, int64_t left) {
    Frag<uint16_t> f;
    if constexpr (VEC) {
        if (left > 0) f.v = *reinterpret_cast<const bf16x8*>(p);
        else zero(f);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f.v[e] = __builtin_bit_cast(__bf16, e < left ? p[e] : (uint16_t)0);
    }
    return f;
}
template <bool VEC>
__device__ __forceinline__ Frag<float> load8(const float* __restrict__ p, int64_t left) {
    Frag<float> f;
    if constexpr (VEC) {
        if (left > 0) {
            const f32x4 lo = *reinterpret_cast<const f32x4*>(p), hi = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) f.v[e] = lo[e], f.v[4 + e] = hi[e];
        } else {
            zero(f);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f.v[e] = e < left ? p[e] : 0.0f;
    }
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
        lo.v[e] = (__bf16)(fabsf(v) < __builtin_inff() ? rest : 0.0f);   // an infinite v has no rest
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

struct Launch {
    uint32_t tiles;     // of a request (rows of equal length), else 0
    uint32_t total;     // of all
    uint32_t groups;    // shrink: groups of kRanks ranks
    uint32_t splits;    // shrink: workgroups that share K
    int64_t slice;      // shrink: K of a workgroup, a multiple of 64
    int64_t pitch;      // ranks of a row of v: r rounded up to 16
    uint32_t parts;     // expand: workgroups that share M
    int64_t columns;    // expand: columns of a wave, a multiple of 64
};

// ---------------------------------------------------------------- shrink
// RB: blocks of 16 ranks of the workgroup.
template <typename T, int RB, bool VEC>
__global__ __launch_bounds__(256) void shrink_kernel(gspn_adapter s, Launch la) {
    __shared__ f32x4 sums[4][kRB * RB][64];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int q = lane >> 4, c = lane & 15;
    const uint32_t split = blockIdx.x % la.splits, rest = blockIdx.x / la.splits;
    const uint32_t group = rest % la.groups, w = rest / la.groups;
    const Tile tile = find_tile<kRows>(s.offsets, s.T, s.N, la.tiles, w, lane);
    const int64_t start = tile.j * kRows;
    if (tile.n == s.N || start >= tile.rows) return;
    const int64_t id = s.ids[tile.n];
    if (id < 0 || id >= s.R) return;
    const int count = uniform((int)(tile.rows - start < kRows ? tile.rows - start : kRows));
    const int64_t row = tile.row + start;

    const T* __restrict__ ap[RB];
    const T* __restrict__ xp[kRB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        // ranks behind the last read it again; their sums are not kept
        const int64_t j = (int64_t)group * kRanks + i * 16 + c;
        ap[i] = static_cast<const T*>(s.a) + (id * s.r + (j < s.r ? j : s.r - 1)) * s.K + 8 * q;
    }
#pragma unroll
    for (int i = 0; i < kRB; ++i) {
        const int t = i * 16 + c;   // rows behind the last likewise
        xp[i] = static_cast<const T*>(s.x) + (row + (t < count ? t : count - 1)) * s.x_stride + 8 * q;
    }
    const int64_t end = ((int64_t)split + 1) * la.slice < s.K ? ((int64_t)split + 1) * la.slice : s.K;
    auto products = [&](auto blocks) {
        constexpr int NB = decltype(blocks)::value;   // blocks of 16 rows
        f32x4 acc[NB][RB] = {};
        for (int64_t k = (int64_t)split * la.slice + wave * 64; k < end; k += 256) {
            Frag<T> a[2][RB], x[2][NB];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t at = k + 32 * h, left = s.K - at - 8 * q;
#pragma unroll
                for (int i = 0; i < RB; ++i) a[h][i] = load8<VEC>(ap[i] + at, left);
#pragma unroll
                for (int t = 0; t < NB; ++t) x[h][t] = load8<VEC>(xp[t] + at, left);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int t = 0; t < NB; ++t)
#pragma unroll
                    for (int i = 0; i < RB; ++i) multiply(acc[t][i], a[h][i], x[h][t]);
        }
#pragma unroll
        for (int t = 0; t < NB; ++t)
#pragma unroll
            for (int i = 0; i < RB; ++i) sums[wave][t * RB + i][lane] = acc[t][i];
    };
    // one block of rows, or all four (rows behind the last are copies of it)
    if (count <= 16) products(std::integral_constant<int, 1>());
    else products(std::integral_constant<int, kRB>());
    __syncthreads();
    float* __restrict__ v = static_cast<float*>(s.work) + (size_t)split * s.T * la.pitch;
    for (int b = wave; b < kRB * RB; b += 4) {
        const int t = (b / RB) * 16 + c, i = b % RB;
        if (t >= count) continue;
        f32x4 sum = sums[0][b][lane];
#pragma unroll
        for (int o = 1; o < 4; ++o) sum += sums[o][b][lane];
        const int64_t j = (int64_t)group * kRanks + i * 16 + 4 * q;
        if (j >= la.pitch) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (j + e >= s.r) sum[e] = 0.0f;
        *reinterpret_cast<f32x4*>(v + (size_t)(row + t) * la.pitch + j) = sum;
    }
}

// ---------------------------------------------------------------- expand
// Sixteen neighbouring columns of a row: out = base + sum, or base, or 0.
template <typename T, bool VEC>
__device__ __forceinline__ void finish(const T* base, T* out, int64_t left, const f32x4 (&sum)[4]) {
    if constexpr (VEC && sizeof(T) == 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (8 * h >= left) break;
            const u32x4 b = *reinterpret_cast<const u32x4*>(base + 8 * h);
            u32x4 o;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f32x4& f = sum[2 * h + e / 2];
                o[e] = pack_bf16x2(bf16_lo(b[e]) + f[2 * (e & 1)], bf16_hi(b[e]) + f[2 * (e & 1) + 1]);
            }
            *reinterpret_cast<u32x4*>(out + 8 * h) = o;
        }
    } else if constexpr (VEC) {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            if (4 * h >= left) break;
            *reinterpret_cast<f32x4*>(out + 4 * h) = *reinterpret_cast<const f32x4*>(base + 4 * h) + sum[h];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (e < left) out[e] = from_f32(to_f32(base[e]) + sum[e / 4][e % 4], (T*)nullptr);
    }
}

// STEPS: steps of 32 ranks whose v a wave keeps for all its columns; 0: any
// number, v is read again for every 64 columns.
template <typename T, int STEPS, bool VEC>
__global__ __launch_bounds__(256) void expand_kernel(gspn_adapter s, Launch la) {
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int q = lane >> 4, c = lane & 15;
    const uint32_t part = blockIdx.x % la.parts, w = blockIdx.x / la.parts;
    const Tile tile = find_tile<kRows>(s.offsets, s.T, s.N, la.tiles, w, lane);
    const int64_t start = tile.j * kRows;
    if (start >= tile.rows) return;
    const int count = uniform((int)(tile.rows - start < kRows ? tile.rows - start : kRows));
    const int64_t row = tile.row + start;
    const int64_t first = ((int64_t)part * 4 + wave) * la.columns;
    const int64_t last = first + la.columns < s.M ? first + la.columns : s.M;
    const T* base = static_cast<const T*>(s.base);   // may be out itself: a lane reads what it then writes
    T* out = static_cast<T*>(s.out);
    const int64_t id = tile.n == s.N ? -1 : s.ids[tile.n];
    if (tile.n == s.N || id < 0 || id >= s.R) {
        // rows of no request (zero, or as they were), or of one without an adapter (base's)
        if (tile.n == s.N ? !(s.flags & GSPN_SEQ_ZERO_TAIL) : base == out) return;
        for (int t = 0; t < count; ++t)
            for (int64_t m = first + lane; m < last; m += 64)
                out[(row + t) * s.out_stride + m] =
                    tile.n == s.N ? from_f32(0.0f, (T*)nullptr) : base[(row + t) * s.base_stride + m];
        return;
    }
    const float scale = s.scale ? s.scale[id] : 1.0f;
    // v of row 16 t + c, ranks 32 k + 8 q .. + 7: the splits' sums, scaled
    auto load_v = [&](int t, int k) {
        const int at = t * 16 + c;
        const int64_t j = 32 * k + 8 * q;
        const float* __restrict__ p =
            static_cast<const float*>(s.work) + (size_t)(row + (at < count ? at : count - 1)) * la.pitch + j;
        f32x4 lo = {}, hi = {};
        if (j < la.pitch)
            for (uint32_t i = 0; i < la.splits; ++i, p += s.T * la.pitch) {
                lo += *reinterpret_cast<const f32x4*>(p);
                hi += *reinterpret_cast<const f32x4*>(p + 4);
            }
        Parts<T> f;
#pragma unroll
        for (int e = 0; e < 4; ++e) f.set(e, scale * lo[e]), f.set(4 + e, scale * hi[e]);
        return f;
    };
    constexpr int kKeep = STEPS ? STEPS : 1;
    const T* __restrict__ bp = static_cast<const T*>(s.b) + id * s.M * s.r;
    auto columns = [&](auto blocks) {
        constexpr int NB = decltype(blocks)::value;   // blocks of 16 rows
        Parts<T> v[NB][kKeep];
        if constexpr (STEPS != 0) {
#pragma unroll
            for (int t = 0; t < NB; ++t)
#pragma unroll
                for (int k = 0; k < STEPS; ++k) v[t][k] = load_v(t, k);
        }
        for (int64_t m = first; m < last; m += 64) {
            f32x4 acc[NB][4] = {};
            // block i of 16 columns holds m + 16 (row / 4) + 4 i + row % 4: lane l's
            // sums of the four blocks are sixteen neighbouring columns, m + 16 q on
            int64_t column[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t o = m + 16 * (c >> 2) + 4 * i + (c & 3);
                column[i] = o < s.M ? o : s.M - 1;   // columns behind the last read it again
            }
            auto step = [&](int k, int slot) {
                const int64_t j = 32 * k + 8 * q;
                Frag<T> b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) b[i] = load8<VEC>(bp + column[i] * s.r + j, s.r - j);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int t = 0; t < NB; ++t) multiply(acc[t][i], b[i], v[t][slot]);
            };
            if constexpr (STEPS != 0) {
#pragma unroll
                for (int k = 0; k < STEPS; ++k) step(k, k);
            } else {
                for (int k = 0; 32 * k < s.r; ++k) {
#pragma unroll
                    for (int t = 0; t < NB; ++t) v[t][0] = load_v(t, k);
                    step(k, 0);
                }
            }
            const int64_t at = m + 16 * q, left = s.M - at;
#pragma unroll
            for (int t = 0; t < NB; ++t)
                if (t * 16 + c < count && left > 0)
                    finish<T, VEC>(base + (row + t * 16 + c) * s.base_stride + at,
                                   out + (row + t * 16 + c) * s.out_stride + at, left, acc[t]);
        }
    };
    if (count <= 16) columns(std::integral_constant<int, 1>());
    else columns(std::integral_constant<int, kRB>());
}

// ---------------------------------------------------------------- host
// Sizes of the launches; the workspace holds [splits][T][pitch] fp32.
Launch plan(const gspn_adapter& s) {
    Launch la;
    la.tiles = s.offsets ? 0 : tiles_of_sequence<kRows>(s.T, s.N);
    la.total = total_tiles<kRows>(s.offsets, s.T, s.N);
    la.groups = (uint32_t)((s.r + kRanks - 1) / kRanks);
    la.pitch = (s.r + 15) / 16 * 16;
    // K is shared by more workgroups while there are fewer than some four for
    // a CU, as long as each of their waves has 64 of it
    const int64_t blocks = (s.K + 63) / 64, most = std::min<int64_t>(kSplits, (blocks + 3) / 4);
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(most, 1024 / ((int64_t)la.total * la.groups)));
    la.slice = (blocks + want - 1) / want * 64;
    la.splits = (uint32_t)((s.K + la.slice - 1) / la.slice);
    // a wave takes up to four times 64 columns while workgroups are many
    int64_t columns = 64;
    while (columns < 256 && la.total * ((s.M + 4 * columns - 1) / (4 * columns)) > 2048) columns *= 2;
    la.columns = columns;
    la.parts = (uint32_t)((s.M + 4 * columns - 1) / (4 * columns));
    return la;
}

bool aligned(const void* p, int64_t stride, int64_t to) { return ((uintptr_t)p & 15) == 0 && stride % to == 0; }

template <typename T>
void launch_typed(const gspn_adapter& s, const Launch& la, hipStream_t stream) {
    constexpr int64_t to = 16 / sizeof(T);   // elements of a 16-byte piece
    const dim3 gs(la.total * la.groups * la.splits), ge(la.total * la.parts), threads(256);
    const bool vs = s.K % 8 == 0 && aligned(s.a, 0, to) && aligned(s.x, s.x_stride, to);
    const bool ve = s.r % 8 == 0 && s.M % 8 == 0 && aligned(s.b, 0, to) && aligned(s.base, s.base_stride, to) &&
                    aligned(s.out, s.out_stride, to);
    auto shrink = [&](auto kernel) { hipLaunchKernelGGL(kernel, gs, threads, 0, stream, s, la); };
    auto expand = [&](auto kernel) { hipLaunchKernelGGL(kernel, ge, threads, 0, stream, s, la); };
    if (s.r <= 16) vs ? shrink(shrink_kernel<T, 1, true>) : shrink(shrink_kernel<T, 1, false>);
    else if (s.r <= 32) vs ? shrink(shrink_kernel<T, 2, true>) : shrink(shrink_kernel<T, 2, false>);
    else vs ? shrink(shrink_kernel<T, 4, true>) : shrink(shrink_kernel<T, 4, false>);
    if (s.r <= 32) ve ? expand(expand_kernel<T, 1, true>) : expand(expand_kernel<T, 1, false>);
    else if (s.r <= 64) ve ? expand(expand_kernel<T, 2, true>) : expand(expand_kernel<T, 2, false>);
    else ve ? expand(expand_kernel<T, 0, true>) : expand(expand_kernel<T, 0, false>);
}

}  // namespace

int64_t adapter_workspace(const gspn_adapter& s) {
    const Launch la = plan(s);
    return (int64_t)la.splits * s.T * la.pitch * 4;
}

hipError_t launch_adapter(const gspn_adapter& s, hipStream_t stream) {
    const Launch la = plan(s);
    if (s.dtype == GSPN_BF16) launch_typed<uint16_t>(s, la, stream);
    else launch_typed<float>(s, la, stream);
    return hipGetLastError();
}

}  // namespace gspn
