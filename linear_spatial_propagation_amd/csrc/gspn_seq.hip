// gspn_seq.hip -- the gated linear recurrence over packed sequences.
//
//   a_t = sigmoid(gate_t),  h_t = a_t h_{t-1} + in_t,  in_t = lam_t x_t or (1 - a_t) x_t,
//   y_t = u_t h_t or h_t
//
// per channel of every sequence (include/gspn.h has the whole definition),
// its backward and its step for single tokens.
//
// One lane owns one channel of one sequence and walks its tokens; the state
// stays in a register.  The backward walks from the last token to the first,
// tile by tile: it recomputes a tile's states from the one the forward saved
// in front of the tile.
#include "gspn_device.h"
#include "gspn_kernels.h"

namespace gspn {
namespace {

constexpr int kLanes = 64;

// a = sigmoid(g) held so that neither a near 1 nor a near 0 loses precision:
// `small` is the smaller of a and 1 - a, and `open` says which (true: a is
// the larger one, small = 1 - a).
struct Gate {
    float small, large;
    bool open;
    __device__ float keep() const { return open ? large : small; }     // a
    __device__ float take() const { return open ? small : large; }     // 1 - a
    // a h + in.  For a near 1 it is h - (1 - a) h + in: a's own rounding (2^-24
    // of h at every token) would add up over the gate's memory, 1 / (1 - a)
    // tokens, where the rounding of 1 - a does not.
    __device__ float step(float h, float in) const {
        return fmaf(open ? -small : small, h, open ? h : 0.0f) + in;
    }
};

__device__ __forceinline__ Gate make_gate(float g) {
    const float e = fast_exp2(-fabsf(g) * 1.44269504088896340736f);
    Gate r;
    r.large = fast_rcp(1.0f + e);
    r.small = e * r.large;
    r.open = g >= 0.0f;
    return r;
}

// The rows of sequence n (n = N: the rows behind the last one).
__device__ __forceinline__ void rows_of(const int32_t* __restrict__ offsets, int64_t n, int64_t N, int64_t T,
                                        int64_t& begin, int64_t& end) {
    if (!offsets) {
        begin = n * (T / N);
        end = n == N ? begin : begin + T / N;
        return;
    }
    begin = offsets[n];
    end = n == N ? T : offsets[n + 1];
    // whatever the offsets hold, rows stay inside the tensors
    begin = begin < 0 ? 0 : begin > T ? T : begin;
    end = end < begin ? begin : end > T ? T : end;
}

// First row of `states` of a sequence: sequences take begin / kSeqTile + n,
// which leaves each of them at least ceil(length / kSeqTile) rows, and one.
__device__ __forceinline__ int64_t first_tile(int64_t begin, int64_t n) { return begin / kSeqTile + n; }

template <typename T>
__global__ __launch_bounds__(kLanes) void seq_fwd_kernel(gspn_seq s) {
    const T* __restrict__ x = static_cast<const T*>(s.x);
    const T* __restrict__ gate = static_cast<const T*>(s.gate);
    const T* __restrict__ lam = static_cast<const T*>(s.lam);
    const T* __restrict__ u = static_cast<const T*>(s.u);
    T* __restrict__ y = static_cast<T*>(s.y);
    const int64_t blocks = (s.D + kLanes - 1) / kLanes;
    const int64_t n = blockIdx.x / blocks;
    const int64_t d = (blockIdx.x - n * blocks) * kLanes + threadIdx.x;
    if (d >= s.D) return;
    int64_t begin, end;
    rows_of(s.offsets, n, s.N, s.T, begin, end);
    if (n == s.N) {
        if (s.flags & GSPN_SEQ_ZERO_TAIL)
            for (int64_t t = begin; t < end; ++t) y[t * s.y_stride + d] = from_f32(0.0f, (T*)nullptr);
        return;
    }
    const int64_t k = d / s.ch_per_weight;
    float h = s.h0 ? s.h0[n * s.D + d] : 0.0f;
    for (int64_t t = begin; t < end; ++t) {
        if (s.states && (t - begin) % kSeqTile == 0)
            s.states[(first_tile(begin, n) + (t - begin) / kSeqTile) * s.D + d] = h;
        const Gate a = make_gate(to_f32(gate[t * s.gate_stride + k]));
        const float xv = to_f32(x[t * s.x_stride + d]);
        h = a.step(h, (lam ? to_f32(lam[t * s.lam_stride + d]) : a.take()) * xv);
        y[t * s.y_stride + d] = from_f32(u ? to_f32(u[t * s.u_stride + d]) * h : h, (T*)nullptr);
    }
    if (s.h_last) s.h_last[n * s.D + d] = h;
}

// dgate: [T][D] fp32, each channel's own gate gradient, where a gate is
// shared (reduce_gate_kernel sums a set's); NULL where it is not.
template <typename T>
__global__ __launch_bounds__(kLanes) void seq_bwd_kernel(gspn_seq s, gspn_seq_grad g, float* __restrict__ dgate) {
    const T* __restrict__ x = static_cast<const T*>(s.x);
    const T* __restrict__ gate = static_cast<const T*>(s.gate);
    const T* __restrict__ lam = static_cast<const T*>(s.lam);
    const T* __restrict__ u = static_cast<const T*>(s.u);
    const T* __restrict__ gy = static_cast<const T*>(g.gy);
    T* __restrict__ gx = static_cast<T*>(g.gx);
    T* __restrict__ ggate = static_cast<T*>(g.ggate);
    T* __restrict__ glam = static_cast<T*>(g.glam);
    T* __restrict__ gu = static_cast<T*>(g.gu);
    __shared__ float before[kSeqTile + 1][kLanes];   // a tile's states, each in front of its token
    const int64_t blocks = (s.D + kLanes - 1) / kLanes;
    const int64_t n = blockIdx.x / blocks;
    const int64_t d = (blockIdx.x - n * blocks) * kLanes + threadIdx.x;
    if (d >= s.D) return;
    int64_t begin, end;
    rows_of(s.offsets, n, s.N, s.T, begin, end);
    const int64_t k = d / s.ch_per_weight;
    if (n == s.N) {
        if (!(s.flags & GSPN_SEQ_ZERO_TAIL)) return;
        const T zero = from_f32(0.0f, (T*)nullptr);
        for (int64_t t = begin; t < end; ++t) {
            if (gx) gx[t * g.gx_stride + d] = zero;
            if (glam) glam[t * g.glam_stride + d] = zero;
            if (gu) gu[t * g.gu_stride + d] = zero;
            if (ggate && d % s.ch_per_weight == 0) ggate[t * g.ggate_stride + k] = zero;
        }
        return;
    }
    const int lane = threadIdx.x;
    float carry = g.gh_last ? g.gh_last[n * s.D + d] : 0.0f;   // a_{t+1} G_{t+1}
    for (int64_t j = (end - begin + kSeqTile - 1) / kSeqTile - 1; j >= 0; --j) {
        const int64_t t0 = begin + j * kSeqTile;
        const int count = (int)(end - t0 < kSeqTile ? end - t0 : kSeqTile);
        before[0][lane] = s.states[(first_tile(begin, n) + j) * s.D + d];
        for (int i = 0; i < count; ++i) {
            const int64_t t = t0 + i;
            const Gate a = make_gate(to_f32(gate[t * s.gate_stride + k]));
            const float xv = to_f32(x[t * s.x_stride + d]);
            before[i + 1][lane] = a.step(before[i][lane], (lam ? to_f32(lam[t * s.lam_stride + d]) : a.take()) * xv);
        }
        for (int i = count - 1; i >= 0; --i) {
            const int64_t t = t0 + i;
            const Gate a = make_gate(to_f32(gate[t * s.gate_stride + k]));
            const float xv = to_f32(x[t * s.x_stride + d]);
            const float gyv = gy ? to_f32(gy[t * g.gy_stride + d]) : 0.0f;
            const float G = (u ? to_f32(u[t * s.u_stride + d]) : 1.0f) * gyv + carry;
            const float lv = lam ? to_f32(lam[t * s.lam_stride + d]) : a.take();
            if (gx) gx[t * g.gx_stride + d] = from_f32(G * lv, (T*)nullptr);
            if (glam) glam[t * g.glam_stride + d] = from_f32(G * xv, (T*)nullptr);
            if (gu) gu[t * g.gu_stride + d] = from_f32(gyv * before[i + 1][lane], (T*)nullptr);
            const float dg = a.small * a.large * G * (lam ? before[i][lane] : before[i][lane] - xv);
            if (dgate) dgate[t * s.D + d] = dg;
            else if (ggate) ggate[t * g.ggate_stride + k] = from_f32(dg, (T*)nullptr);
            carry = a.step(G, 0.0f);
        }
    }
    if (g.gh0) g.gh0[n * s.D + d] = carry;
}

// ggate[t][k] = sum of the set's gate gradients, for the rows of sequences.
template <typename T>
__global__ __launch_bounds__(256) void reduce_gate_kernel(gspn_seq s, gspn_seq_grad g,
                                                          const float* __restrict__ dgate) {
    const int64_t sets = s.D / s.ch_per_weight;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t t = i / sets, k = i - t * sets;
    if (t >= (s.offsets ? (int64_t)s.offsets[s.N] : s.T) || t >= s.T) return;
    const float* __restrict__ p = dgate + t * s.D + k * s.ch_per_weight;
    float sum = 0.0f;
    for (int c = 0; c < s.ch_per_weight; ++c) sum += p[c];
    static_cast<T*>(g.ggate)[t * g.ggate_stride + k] = from_f32(sum, (T*)nullptr);
}

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
        const Gate a = make_gate(to_f32(static_cast<const T*>(s.gate)[r * s.gate_stride + k]));
        const float xv = to_f32(static_cast<const T*>(s.x)[r * s.x_stride + d]);
        const float lv = s.lam ? to_f32(static_cast<const T*>(s.lam)[r * s.lam_stride + d]) : a.take();
        h = a.step(h, lv * xv);
        const float uv = s.u ? to_f32(static_cast<const T*>(s.u)[r * s.u_stride + d]) : 1.0f;
        static_cast<T*>(s.y)[r * s.y_stride + d] = from_f32(uv * h, (T*)nullptr);
        if (!more) break;
    }
    s.state[slot * s.D + d] = h;
}

}  // namespace

int64_t seq_workspace(const gspn_seq& s, bool backward) {
    return backward && s.ch_per_weight > 1 ? s.T * s.D * 4 : 0;
}

hipError_t launch_seq_fwd(const gspn_seq& s, hipStream_t stream) {
    const dim3 grid((unsigned)((s.N + (s.offsets ? 1 : 0)) * ((s.D + kLanes - 1) / kLanes)));
    if (s.dtype == GSPN_BF16) hipLaunchKernelGGL(seq_fwd_kernel<uint16_t>, grid, dim3(kLanes), 0, stream, s);
    else hipLaunchKernelGGL(seq_fwd_kernel<float>, grid, dim3(kLanes), 0, stream, s);
    return hipGetLastError();
}

hipError_t launch_seq_bwd(const gspn_seq& s, const gspn_seq_grad& g, hipStream_t stream) {
    const dim3 grid((unsigned)((s.N + (s.offsets ? 1 : 0)) * ((s.D + kLanes - 1) / kLanes)));
    float* dgate = s.ch_per_weight > 1 && g.ggate ? static_cast<float*>(s.work) : nullptr;
    const dim3 grid_r((unsigned)((s.T * (s.D / s.ch_per_weight) + 255) / 256));
    if (s.dtype == GSPN_BF16) {
        hipLaunchKernelGGL(seq_bwd_kernel<uint16_t>, grid, dim3(kLanes), 0, stream, s, g, dgate);
        if (dgate && s.T) hipLaunchKernelGGL(reduce_gate_kernel<uint16_t>, grid_r, dim3(256), 0, stream, s, g, dgate);
    } else {
        hipLaunchKernelGGL(seq_bwd_kernel<float>, grid, dim3(kLanes), 0, stream, s, g, dgate);
        if (dgate && s.T) hipLaunchKernelGGL(reduce_gate_kernel<float>, grid_r, dim3(256), 0, stream, s, g, dgate);
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
