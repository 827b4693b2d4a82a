// grads.hip -- the global 2-norm of many gradient tensors, and the gradients scaled to a largest norm.
//
//   N = sqrt(sum over tensors and elements of g^2),  c = min(1, max_norm / (N + 1e-6)),  out = c g.
//
// Both passes are bound by memory: 4 (or 2) bytes read per element for the norm, the same read and
// written for the scaling.  Squares are summed in binary64 throughout: the square of any finite
// binary32 is finite and nonzero there, so neither overflow nor underflow changes the norm, and the
// conversion and the fused multiply-add per element hide behind the loads.  Each workgroup's sum
// goes to its own slot and the slots are added in a fixed order, so the result does not depend on
// the order in which workgroups finish; the scaling kernel's workgroups each add the slots up for
// themselves, 16 KiB from L2 for each launch of the norm.  That costs less than a finishing launch in
// between while the launches are few, more when they are many.  us of kernels in one call and in two, for
// mixed tensors of 20 thousand elements scaled into outputs: 100 tensors 10.0 and 11.1, 280 18.9 and 19.2, 500
// 35.8 and 34.8, 1000 82 and 74, 5000 624 and 447; the host's side hides it (calls of 56, 133, 229, 438 and
// 2149 us, and of 79, 188, 328, 635 and 3123).
//
// The tensors are described by a table in the kernel's arguments (no device table to upload, so a
// call is safe under graph capture and the host arrays may be reused as soon as it returns); a
// launch takes up to 280 tensors, or 176 with separate outputs.  Elements are dealt in chunks of
// GRAD_CHUNK, a workgroup taking a contiguous range of them: it finds its first tensor with one
// search and walks on.  The scaling walks each range backwards: what the norm read last is what the
// caches still hold.  A chunk is read in 16-byte vectors from its first element, wherever that lies:
// tensors in a flat bucket start at any multiple of their element.
//
// 352 M fp32 elements: 800 us, in place 812; the norm 231 us (6.1 TB/s), the scaling 530 us (5.3 TB/s read and
// written; a large copy reaches 4.7).  The same in bf16: 412, in place 435.  30 thousand elements in 37
// tensors: 5 + 6 us of kernels.
#include "device_common.hpp"
#include "launch.hpp"

namespace bsq {

constexpr int GRAD_THREADS = 256;
constexpr int GRAD_BLOCKS = 2048;    // workgroups of a launch at most: 8 of 256 threads per CU
constexpr int GRAD_CHUNK = 8192;     // elements
constexpr int GRAD_BF16 = 0x8000;

template <int CAP>
struct GradTable {
    const void* src[CAP];
    uint32_t first[CAP + 1];   // chunks before tensor i
    uint16_t last[CAP];        // elements of its last chunk, | GRAD_BF16
    int count;
};
struct GradList : GradTable<280> {   // the norm; scaling in place
    static constexpr int CAP = 280;
    __device__ __forceinline__ void* out(int i) const { return const_cast<void*>(src[i]); }
    void set_out(int, void*) {}
};
struct GradPairs : GradTable<176> {
    static constexpr int CAP = 176;
    void* dst[CAP];
    __device__ __forceinline__ void* out(int i) const { return dst[i]; }
    void set_out(int i, void* p) { dst[i] = p; }
};
static_assert(sizeof(GradList) <= 4000 && sizeof(GradPairs) <= 4000, "the table travels in the 4 KiB of kernel arguments");

// Calls body(tensor, first element, elements) for every chunk of this workgroup's range, last one first if
// BACK.
template <bool BACK, class T, class F>
__device__ __forceinline__ void for_chunks(const T& t, F&& body) {
    const uint32_t total = t.first[t.count];
    const uint32_t c0 = (uint32_t)((uint64_t)total * blockIdx.x / gridDim.x);
    const uint32_t c1 = (uint32_t)((uint64_t)total * (blockIdx.x + 1) / gridDim.x);
    if (c0 >= c1) return;
    const uint32_t start = BACK ? c1 - 1 : c0;
    int i = 0, hi = t.count - 1;   // the tensor of chunk `start`: the last whose first chunk is at or before it
    while (i < hi) {
        const int mid = (i + hi + 1) >> 1;
        if (t.first[mid] <= start) i = mid;
        else hi = mid - 1;
    }
    for (uint32_t n = 0; n < c1 - c0; ++n) {   // every tensor of the table has a chunk
        const uint32_t c = BACK ? start - n : start + n;
        if (BACK && c < t.first[i]) --i;
        if (!BACK && c >= t.first[i + 1]) ++i;
        const int64_t e0 = (int64_t)(c - t.first[i]) * GRAD_CHUNK;
        body(i, e0, c + 1 == t.first[i + 1] ? (int)(t.last[i] & ~GRAD_BF16) : GRAD_CHUNK);
    }
}

// 16 bytes at any multiple of an element.
struct __attribute__((packed, aligned(4))) GradF4 { float v[4]; };
struct __attribute__((packed, aligned(2))) GradB8 { uint32_t w[4]; };

// body(vector index) for n / PER vectors of a chunk, all loads of a whole chunk in flight at once, and
// tail(element) for the rest.
template <int PER, class L, class V, class S>
__device__ __forceinline__ void for_vectors(int n, L&& load, V&& use, S&& tail) {
    constexpr int N = GRAD_CHUNK / PER / GRAD_THREADS;
    using T = decltype(load(0));
    if (n == GRAD_CHUNK) {
        T v[N];
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = load(k * GRAD_THREADS + (int)threadIdx.x);
#pragma unroll
        for (int k = 0; k < N; ++k) use(k * GRAD_THREADS + (int)threadIdx.x, v[k]);
        return;
    }
    const int whole = n / PER;
    T v[N];
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (k * GRAD_THREADS + (int)threadIdx.x < whole) v[k] = load(k * GRAD_THREADS + (int)threadIdx.x);
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (k * GRAD_THREADS + (int)threadIdx.x < whole) use(k * GRAD_THREADS + (int)threadIdx.x, v[k]);
    const int e = whole * PER + (int)threadIdx.x;
    if (e < n) tail(e);
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

__device__ __forceinline__ float bf16_value(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// Sum of squares of this workgroup's chunks -> part[blockIdx.x].
__global__ __launch_bounds__(GRAD_THREADS) void grad_sumsq_kernel(GradList t, double* part) {
    __shared__ double red[GRAD_THREADS / 64];
    double acc = 0.0;
    for_chunks<false>(t, [&](int i, int64_t e0, int n) {
        if (t.last[i] & GRAD_BF16) {
            const uint16_t* p = (const uint16_t*)t.src[i] + e0;
            for_vectors<8>(
                n, [&](int v) { return *(const GradB8*)(p + 8 * v); },
                [&](int, const GradB8& q) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc += sq(bf16_lo(q.w[k])) + sq(bf16_hi(q.w[k]));
                },
                [&](int e) { acc += sq(bf16_value(p[e])); });
        } else {
            const float* p = (const float*)t.src[i] + e0;
            for_vectors<4>(
                n, [&](int v) { return *(const GradF4*)(p + 4 * v); },
                [&](int, const GradF4& q) { acc += (sq(q.v[0]) + sq(q.v[1])) + (sq(q.v[2]) + sq(q.v[3])); },
                [&](int e) { acc += sq(p[e]); });
        }
    });
    const double s = block_sum(acc, red);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The n slots added in a fixed order (the same wherever they are added).
__device__ __forceinline__ double sum_parts(const double* part, int n, double* red) {
    double acc = 0.0;
    for (int i = threadIdx.x; i < n; i += GRAD_THREADS) acc += part[i];
    return block_sum(acc, red);
}

__global__ __launch_bounds__(GRAD_THREADS) void grad_finish_kernel(const double* part, int n, double* sumsq) {
    __shared__ double red[GRAD_THREADS / 64];
    const double s = sum_parts(part, n, red);
    if (threadIdx.x == 0) *sumsq = s;
}

// c = min(1, max_norm / (N + 1e-6)); NaN stays NaN (a NaN among the gradients, or infinite ones times 0).
__device__ __forceinline__ double clip_factor(double sumsq, double max_norm) {
    const double c = max_norm / (sqrt(sumsq) + 1e-6);
    return c > 1.0 ? 1.0 : c;
}

// Every gradient of this workgroup's chunks replaced by, or written out as, scale(gradient).
template <class T, class F>
__device__ __forceinline__ void scale_chunks(const T& t, F&& scale) {
    for_chunks<true>(t, [&](int i, int64_t e0, int n) {
        if (t.last[i] & GRAD_BF16) {
            const uint16_t* p = (const uint16_t*)t.src[i] + e0;
            uint16_t* q = (uint16_t*)t.out(i) + e0;
            for_vectors<8>(
                n, [&](int v) { return *(const GradB8*)(p + 8 * v); },
                [&](int v, GradB8 x) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) x.w[k] = bf16x2_rne(scale(bf16_lo(x.w[k])), scale(bf16_hi(x.w[k])));
                    *(GradB8*)(q + 8 * v) = x;
                },
                [&](int e) { q[e] = (uint16_t)bf16x2_rne(scale(bf16_value(p[e])), 0.0f); });
        } else {
            const float* p = (const float*)t.src[i] + e0;
            float* q = (float*)t.out(i) + e0;
            for_vectors<4>(
                n, [&](int v) { return *(const GradF4*)(p + 4 * v); },
                [&](int v, GradF4 x) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) x.v[k] = scale(x.v[k]);
                    *(GradF4*)(q + 4 * v) = x;
                },
                [&](int e) { q[e] = scale(p[e]); });
        }
    });
}

// sums: `n` slots to add (1: the sum itself).  c is rounded to binary32, except below its normal range (norms
// above 2^126 max_norm), where it would lose bits, or be 0, while its products are still normal values.
template <class T>
__global__ __launch_bounds__(GRAD_THREADS) void grad_clip_kernel(T t, const double* sums, int n, double max_norm,
                                                                 float* norm) {
    __shared__ double red[GRAD_THREADS / 64];
    const double s = n == 1 ? *sums : sum_parts(sums, n, red);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)sqrt(s);
    const double cd = clip_factor(s, max_norm);
    if (cd > 0.0 && cd < 0x1p-126) {
        scale_chunks(t, [&](float v) { return (float)((double)v * cd); });
        return;
    }
    const float c = (float)cd;
    if (std::is_same<T, GradList>::value && c == 1.0f) return;   // in place: every gradient keeps its bits
    scale_chunks(t, [&](float v) { return v * c; });
}

// Fills the table with tensors from `at` on; returns the first one that it leaves out.
template <class T>
static int64_t fill_table(T& t, const void* const* grads, void* const* outs, const int64_t* numels, const int* dtypes,
                          int64_t count, int64_t at) {
    t.count = 0;
    t.first[0] = 0;
    while (at < count && t.count < T::CAP) {
        const int64_t chunks = (numels[at] + GRAD_CHUNK - 1) / GRAD_CHUNK;
        if ((int64_t)t.first[t.count] + chunks > 0x7FFFFFFF) break;   // a tensor has at most 2^27
        if (numels[at] > 0) {
            const int k = t.count++;
            t.src[k] = grads[at];
            if (outs) t.set_out(k, outs[at]);
            t.last[k] = (uint16_t)((numels[at] - (chunks - 1) * GRAD_CHUNK) | (dtypes[at] == 0 ? GRAD_BF16 : 0));
            t.first[k + 1] = t.first[k] + (uint32_t)chunks;
        }
        ++at;
    }
    return at;
}

template <class T>
static unsigned blocks_of(const T& t) {
    const uint32_t c = t.first[t.count];
    return c < (uint32_t)GRAD_BLOCKS ? c : (uint32_t)GRAD_BLOCKS;
}

int64_t grad_workspace_slots(int64_t count) { return ((count + GradList::CAP - 1) / GradList::CAP + 1) * GRAD_BLOCKS; }

// The workgroups' sums -> workspace; parts: how many.
static int launch_parts(const void* const* grads, const int64_t* numels, const int* dtypes, int64_t count,
                        double* workspace, int& parts, hipStream_t s) {
    GradList t;
    int64_t at = 0;
    parts = 0;
    while (at < count) {
        at = fill_table(t, grads, nullptr, numels, dtypes, count, at);
        if (t.count == 0) continue;
        const unsigned b = blocks_of(t);
        hipLaunchKernelGGL(grad_sumsq_kernel, dim3(b), dim3(GRAD_THREADS), 0, s, t, workspace + parts);
        const int e = (int)hipGetLastError();
        if (e) return e;
        parts += (int)b;
    }
    return 0;
}

int launch_grad_sumsq(const void* const* grads, const int64_t* numels, const int* dtypes, int64_t count,
                      double* sumsq, double* workspace, void* hip_stream) {
    hipStream_t s = (hipStream_t)hip_stream;
    int parts;
    const int e = launch_parts(grads, numels, dtypes, count, workspace, parts, s);
    if (e) return e;
    hipLaunchKernelGGL(grad_finish_kernel, dim3(1), dim3(GRAD_THREADS), 0, s, (const double*)workspace, parts, sumsq);
    return (int)hipGetLastError();
}

template <class T>
static int launch_scale(const void* const* grads, void* const* outs, const int64_t* numels, const int* dtypes,
                        int64_t count, const double* sums, int n, double max_norm, float* norm, hipStream_t s) {
    T t;
    int64_t at = 0;
    do {
        at = fill_table(t, grads, outs, numels, dtypes, count, at);
        // the first launch writes the norm, even of an empty list
        if (t.count > 0 || (norm && at >= count)) {
            const unsigned b = t.count ? blocks_of(t) : 1u;
            hipLaunchKernelGGL((grad_clip_kernel<T>), dim3(b), dim3(GRAD_THREADS), 0, s, t, sums, n, max_norm, norm);
            const int e = (int)hipGetLastError();
            if (e) return e;
            norm = nullptr;
        }
    } while (at < count);
    return 0;
}

static int launch_scale_any(const void* const* grads, void* const* outs, const int64_t* numels, const int* dtypes,
                            int64_t count, const double* sums, int n, double max_norm, float* norm, hipStream_t s) {
    return outs ? launch_scale<GradPairs>(grads, outs, numels, dtypes, count, sums, n, max_norm, norm, s)
                : launch_scale<GradList>(grads, nullptr, numels, dtypes, count, sums, n, max_norm, norm, s);
}

int launch_grad_clip(const void* const* grads, void* const* outs, const int64_t* numels, const int* dtypes,
                     int64_t count, const double* sumsq, double max_norm, float* norm, void* hip_stream) {
    return launch_scale_any(grads, outs, numels, dtypes, count, sumsq, 1, max_norm, norm, (hipStream_t)hip_stream);
}

int launch_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* numels, const int* dtypes,
                          int64_t count, double max_norm, float* norm, double* workspace, void* hip_stream) {
    hipStream_t s = (hipStream_t)hip_stream;
    int parts;
    const int e = launch_parts(grads, numels, dtypes, count, workspace, parts, s);
    if (e) return e;
    return launch_scale_any(grads, outs, numels, dtypes, count, workspace, parts, max_norm, norm, s);
}

}  // namespace bsq
