// gspn_adapter.hip -- low-rank adapters of many requests beside a shared
// projection:  out[t] = base[t] + scale[i] b[i] (a[i] x[t]),  i = ids[request of t].
//
// Two launches: v[t] = a[i] x[t] (r numbers a row, fp32, in the workspace),
// then out[t] = base[t] + scale[i] b[i] v[t].
#include "gspn_device.h"
#include "gspn_kernels.h"

namespace gspn {
namespace {

// The request of row t, or -1 behind the last one: the largest n with
// offsets[n] <= t among those that hold a row.
__device__ __forceinline__ int64_t request_of(const gspn_adapter& a, int64_t t) {
    if (!a.offsets) return t / (a.T / a.N);
    int64_t lo = 0, hi = a.N;   // offsets[lo] <= t, and offsets[hi] > t if any is
    if (t >= a.offsets[a.N]) return -1;
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) / 2;
        if (a.offsets[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// One wave per row and rank.
template <typename T>
__global__ __launch_bounds__(64) void shrink_kernel(gspn_adapter a) {
    const int64_t t = blockIdx.x / a.r, j = blockIdx.x - t * a.r;
    const int64_t n = request_of(a, t);
    if (n < 0) return;
    const int64_t i = a.ids[n];
    if (i < 0 || i >= a.R) return;
    const T* __restrict__ w = static_cast<const T*>(a.a) + (i * a.r + j) * a.K;
    const T* __restrict__ x = static_cast<const T*>(a.x) + t * a.x_stride;
    float sum = 0.0f;
    for (int64_t k = threadIdx.x; k < a.K; k += 64) sum = fmaf(to_f32(w[k]), to_f32(x[k]), sum);
    for (int m = 32; m; m >>= 1) sum += __shfl_xor(sum, m);
    if (threadIdx.x == 0) static_cast<float*>(a.work)[t * a.r + j] = sum;
}

// One lane per output.
template <typename T>
__global__ __launch_bounds__(256) void expand_kernel(gspn_adapter a) {
    const int64_t blocks = (a.M + 255) / 256;
    const int64_t t = blockIdx.x / blocks, m = (blockIdx.x - t * blocks) * 256 + threadIdx.x;
    if (m >= a.M) return;
    T* __restrict__ out = static_cast<T*>(a.out) + t * a.out_stride + m;
    const int64_t n = request_of(a, t);
    if (n < 0) {
        if (a.flags & GSPN_SEQ_ZERO_TAIL) *out = from_f32(0.0f, (T*)nullptr);
        return;
    }
    const T base = static_cast<const T*>(a.base)[t * a.base_stride + m];
    const int64_t i = a.ids[n];
    if (i < 0 || i >= a.R) {
        *out = base;
        return;
    }
    const T* __restrict__ w = static_cast<const T*>(a.b) + (i * a.M + m) * a.r;
    const float* __restrict__ v = static_cast<const float*>(a.work) + t * a.r;
    float sum = 0.0f;
    for (int64_t j = 0; j < a.r; ++j) sum = fmaf(to_f32(w[j]), v[j], sum);
    *out = from_f32(fmaf(a.scale ? a.scale[i] : 1.0f, sum, to_f32(base)), (T*)nullptr);
}

}  // namespace

int64_t adapter_workspace(const gspn_adapter& a) { return a.T * a.r * 4; }

hipError_t launch_adapter(const gspn_adapter& a, hipStream_t stream) {
    const dim3 shrink((unsigned)(a.T * a.r)), expand((unsigned)(a.T * ((a.M + 255) / 256)));
    if (a.dtype == GSPN_BF16) {
        hipLaunchKernelGGL(shrink_kernel<uint16_t>, shrink, dim3(64), 0, stream, a);
        hipLaunchKernelGGL(expand_kernel<uint16_t>, expand, dim3(256), 0, stream, a);
    } else {
        hipLaunchKernelGGL(shrink_kernel<float>, shrink, dim3(64), 0, stream, a);
        hipLaunchKernelGGL(expand_kernel<float>, expand, dim3(256), 0, stream, a);
    }
    return hipGetLastError();
}

}  // namespace gspn
