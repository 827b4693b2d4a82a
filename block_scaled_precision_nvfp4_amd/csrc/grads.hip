// grads.hip -- the global 2-norm of many gradient tensors, and the gradients scaled to a largest norm.
//
//   N = sqrt(sum over tensors and elements of g^2),  c = min(1, max_norm / (N + 1e-6)),  out = c g.
//
// Both passes are bound by memory: 4 (or 2) bytes read per element for the norm, the same read and
// written for the scaling.  Squares are summed in binary64 throughout: the square of any finite
// binary32 is finite and nonzero there, so neither overflow nor underflow changes the norm, and the
// conversion and the fused multiply-add per element hide behind the loads.  Each workgroup's sum
// goes to its own slot and the slots are added in a fixed order, so the result does not depend on
// the order in which workgroups finish.
//
// The tensors are described by a table in the kernel's arguments (no device table to upload, so a
// call is safe under graph capture and the host arrays may be reused as soon as it returns); a
// launch takes up to GRAD_TABLE tensors.  Elements are dealt in chunks of GRAD_CHUNK, a workgroup
// taking a contiguous range of them: it finds its first tensor with one search and walks on.
#include "device_common.hpp"
#include "launch.hpp"

namespace bsq {

constexpr int GRAD_TABLE = 112;
constexpr int GRAD_THREADS = 256;
constexpr int GRAD_BLOCKS = 2048;    // workgroups of a launch at most: 8 of 256 threads per CU
constexpr int GRAD_CHUNK = 8192;     // elements

struct GradTable {
    const void* src[GRAD_TABLE];
    void* dst[GRAD_TABLE];
    int64_t numel[GRAD_TABLE];
    uint32_t first[GRAD_TABLE + 1];   // chunks before tensor i
    uint8_t bf16[GRAD_TABLE];
    int count;
};
static_assert(sizeof(GradTable) <= 3584, "the table travels in the 4 KiB of kernel arguments");

// Calls body(tensor, first element, elements) for every chunk of this workgroup's range.
template <class F>
__device__ __forceinline__ void for_chunks(const GradTable& t, F&& body) {
    const uint32_t total = t.first[t.count];
    const uint32_t c0 = (uint32_t)((uint64_t)total * blockIdx.x / gridDim.x);
    const uint32_t c1 = (uint32_t)((uint64_t)total * (blockIdx.x + 1) / gridDim.x);
    if (c0 >= c1) return;
    int lo = 0, hi = t.count - 1;   // the last tensor whose first chunk is at or before c0
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= c0) lo = mid;
        else hi = mid - 1;
    }
    for (uint32_t c = c0; c < c1; ++c) {
        while (t.first[lo + 1] <= c) ++lo;   // skips empty tensors; first[count] > c ends it
        const int64_t e0 = (int64_t)(c - t.first[lo]) * GRAD_CHUNK;
        const int64_t left = t.numel[lo] - e0;
        body(lo, e0, (int)(left < GRAD_CHUNK ? left : GRAD_CHUNK));
    }
}

__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.0;
    for (int i = 0; i < (int)blockDim.x / 64; ++i) s += red[i];
    __syncthreads();
    return s;
}

__device__ __forceinline__ double sq(float v) { return (double)v * (double)v; }

// Sum of squares of this workgroup's chunks -> part[blockIdx.x].
__global__ __launch_bounds__(GRAD_THREADS) void grad_sumsq_kernel(GradTable t, double* part) {
    __shared__ double red[GRAD_THREADS / 64];
    double acc = 0.0;
    for_chunks(t, [&](int i, int64_t e0, int n) {
        if (t.bf16[i]) {
            const uint16_t* p = (const uint16_t*)t.src[i] + e0;
            for (int e = threadIdx.x; e < n; e += GRAD_THREADS) acc += sq(__uint_as_float((uint32_t)p[e] << 16));
        } else {
            const float* p = (const float*)t.src[i] + e0;
            for (int e = threadIdx.x; e < n; e += GRAD_THREADS) acc += sq(p[e]);
        }
    });
    const double s = block_sum(acc, red);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The slots added in a fixed order.
__global__ __launch_bounds__(GRAD_THREADS) void grad_finish_kernel(const double* part, int n, double* sumsq) {
    __shared__ double red[GRAD_THREADS / 64];
    double acc = 0.0;
    for (int i = threadIdx.x; i < n; i += GRAD_THREADS) acc += part[i];
    const double s = block_sum(acc, red);
    if (threadIdx.x == 0) *sumsq = s;
}

// c = min(1, max_norm / (N + 1e-6)); NaN stays NaN (a NaN among the gradients, or infinite ones times 0).
__device__ __forceinline__ float clip_factor(double sumsq, double max_norm) {
    const double c = max_norm / (sqrt(sumsq) + 1e-6);
    return c > 1.0 ? 1.0f : (float)c;
}

__global__ __launch_bounds__(GRAD_THREADS) void grad_clip_kernel(GradTable t, const double* sumsq, double max_norm,
                                                                 float* norm, int in_place) {
    const double s = *sumsq;
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)sqrt(s);
    const float c = clip_factor(s, max_norm);
    if (in_place && c == 1.0f) return;   // nothing to scale: every gradient keeps its bits
    for_chunks(t, [&](int i, int64_t e0, int n) {
        if (t.bf16[i]) {
            const uint16_t* p = (const uint16_t*)t.src[i] + e0;
            uint16_t* q = (uint16_t*)t.dst[i] + e0;
            for (int e = threadIdx.x; e < n; e += GRAD_THREADS)
                q[e] = (uint16_t)bf16x2_rne(__uint_as_float((uint32_t)p[e] << 16) * c, 0.0f);
        } else {
            const float* p = (const float*)t.src[i] + e0;
            float* q = (float*)t.dst[i] + e0;
            for (int e = threadIdx.x; e < n; e += GRAD_THREADS) q[e] = p[e] * c;
        }
    });
}

// Fills the table with tensors from `at` on; returns the first one that it leaves out.
static int64_t fill_table(GradTable& t, const void* const* grads, void* const* outs, const int64_t* numels,
                          const int* dtypes, int64_t count, int64_t at) {
    t.count = 0;
    t.first[0] = 0;
    while (at < count && t.count < GRAD_TABLE) {
        const int64_t chunks = (numels[at] + GRAD_CHUNK - 1) / GRAD_CHUNK;
        if ((int64_t)t.first[t.count] + chunks > 0x7FFFFFFF) break;
        if (numels[at] > 0) {
            const int k = t.count++;
            t.src[k] = grads[at];
            t.dst[k] = outs ? outs[at] : const_cast<void*>(grads[at]);
            t.numel[k] = numels[at];
            t.bf16[k] = dtypes[at] == 0;
            t.first[k + 1] = t.first[k] + (uint32_t)chunks;
        }
        ++at;
    }
    return at;
}

static unsigned blocks_of(const GradTable& t) {
    const uint32_t c = t.first[t.count];
    return c < (uint32_t)GRAD_BLOCKS ? c : (uint32_t)GRAD_BLOCKS;
}

int64_t grad_workspace_slots(int64_t count) { return ((count + GRAD_TABLE - 1) / GRAD_TABLE + 1) * GRAD_BLOCKS; }

int launch_grad_sumsq(const void* const* grads, const int64_t* numels, const int* dtypes, int64_t count,
                      double* sumsq, double* workspace, void* hip_stream) {
    hipStream_t s = (hipStream_t)hip_stream;
    GradTable t;
    int64_t at = 0;
    int parts = 0;
    while (at < count) {
        at = fill_table(t, grads, nullptr, numels, dtypes, count, at);
        if (t.count == 0) continue;
        const unsigned b = blocks_of(t);
        hipLaunchKernelGGL(grad_sumsq_kernel, dim3(b), dim3(GRAD_THREADS), 0, s, t, workspace + parts);
        const int e = (int)hipGetLastError();
        if (e) return e;
        parts += (int)b;
    }
    hipLaunchKernelGGL(grad_finish_kernel, dim3(1), dim3(GRAD_THREADS), 0, s, (const double*)workspace, parts, sumsq);
    return (int)hipGetLastError();
}

int launch_grad_clip(const void* const* grads, void* const* outs, const int64_t* numels, const int* dtypes,
                     int64_t count, const double* sumsq, double max_norm, float* norm, void* hip_stream) {
    hipStream_t s = (hipStream_t)hip_stream;
    GradTable t;
    int64_t at = 0;
    bool first = true;
    do {
        at = fill_table(t, grads, outs, numels, dtypes, count, at);
        if (t.count == 0 && !(first && at >= count)) continue;   // an empty list still writes the norm
        const unsigned b = t.count ? blocks_of(t) : 1u;
        if (t.count == 0) t.first[0] = 0;
        hipLaunchKernelGGL(grad_clip_kernel, dim3(b), dim3(GRAD_THREADS), 0, s, t, sumsq, max_norm,
                           first ? norm : nullptr, outs ? 0 : 1);
        const int e = (int)hipGetLastError();
        if (e) return e;
        first = false;
    } while (at < count);
    return 0;
}

}  // namespace bsq
