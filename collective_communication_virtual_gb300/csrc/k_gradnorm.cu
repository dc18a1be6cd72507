// k_gradnorm.cu -- the global 2-norm of many tensors' gradients, and clipping by it.
//
//   norm = sqrt(sum over all tensors of g^2),  g' = g min(1, maxNorm / (norm + 1e-6))
//
// The tensors are one flat space of 32 KiB chunks, so a launch covers large and small ones
// alike.  A thread sums the squares of its part of a chunk in fp32 (at most 64 terms) and adds
// chunks and threads in fp64; every sum's order follows from the sizes alone.
#include "norm.cuh"

namespace vc {

namespace {

// The item that holds a chunk: the last whose first chunk is not beyond it.
template <int CAP>
__device__ __forceinline__ int find_item(const unsigned int* start, int n, unsigned int chunk) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= chunk) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <int E>
__device__ __forceinline__ Span span_long(long long e0, long long count) {
    Span s;
    s.lo = e0 < 0 ? (int)-e0 : 0;
    s.hi = count - e0 < E ? (int)max(count - e0, 0ll) : E;
    return s;
}

// Sum of squares of a thread's part of chunk `chunk` of a tensor.
template <int DT>
__device__ __forceinline__ float chunk_squares(const GradItem& it, unsigned int chunk) {
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    const int shift = (int)((uintptr_t)it.in & 15u) / ESZ;
    const long long k0 = (long long)chunk * kGradChunkVecs + threadIdx.x;
    const char* p = (const char*)it.in - shift * ESZ + k0 * 16;
    const long long count = (long long)it.count;
    uint4 raw[kGradVecs];
#pragma unroll
    for (int i = 0; i < kGradVecs; i++) {
        const long long e0 = (k0 + i * kGradThreads) * E - shift;
        raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (e0 < count) raw[i] = ld_once(p + (size_t)i * kGradThreads * 16);
    }
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kGradVecs; i++) {
        const long long e0 = (k0 + i * kGradThreads) * E - shift;
        float f[E];
        widen_vec<DT>(raw[i], f);
        if (e0 < 0 || e0 + E > count) {                // elements of other tensors
            const Span sp = span_long<E>(e0, count);
#pragma unroll
            for (int j = 0; j < E; j++) f[j] = sp.has(j) ? f[j] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < E; j++) s[j & 3] = fmaf(f[j], f[j], s[j & 3]);
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

template <int DT>
__device__ __forceinline__ void chunk_scale(const GradItem& it, unsigned int chunk, float factor) {
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    const int shift = (int)((uintptr_t)it.out & 15u) / ESZ;
    const long long k0 = (long long)chunk * kGradChunkVecs + threadIdx.x;
    const ptrdiff_t off = (ptrdiff_t)k0 * 16 - shift * ESZ;
    const long long count = (long long)it.count;
    uint4 raw[kGradVecs];
#pragma unroll
    for (int i = 0; i < kGradVecs; i++) {
        const long long e0 = (k0 + i * kGradThreads) * E - shift;
        if (e0 < count)
            raw[i] = load_vec<ESZ, true>((const char*)it.in + off + (ptrdiff_t)i * kGradThreads * 16,
                                         span_long<E>(e0, count));
    }
#pragma unroll
    for (int i = 0; i < kGradVecs; i++) {
        const long long e0 = (k0 + i * kGradThreads) * E - shift;
        if (e0 >= count) continue;
        float f[E];
        widen_vec<DT>(raw[i], f);
#pragma unroll
        for (int j = 0; j < E; j++) f[j] *= factor;
        store_vec<DT, true>((char*)it.out + off + (ptrdiff_t)i * kGradThreads * 16, span_long<E>(e0, count), f);
    }
}

// Sum over the CTA in fp64, in an order that the CTA's size fixes; every thread gets it.
__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < warps ? red[lane] : 0.0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

}  // namespace

template <int CAP>
__global__ void __launch_bounds__(kGradThreads) k_grad_squares(const __grid_constant__ GradArgs<CAP> a) {
    pdl_begin();
    __shared__ unsigned int start[CAP];
    __shared__ double red[32];
    for (int i = threadIdx.x; i < a.nItems; i += kGradThreads) start[i] = a.items[i].chunk0;
    __syncthreads();
    double sum = 0.0;
    for (unsigned int c = blockIdx.x; c < a.nChunks; c += gridDim.x) {
        const GradItem& it = a.items[find_item<CAP>(start, a.nItems, c)];
        const unsigned int chunk = c - it.chunk0;
        if (it.dt == kF32) sum += (double)chunk_squares<kF32>(it, chunk);
        else if (it.dt == kF16) sum += (double)chunk_squares<kF16>(it, chunk);
        else sum += (double)chunk_squares<kBF16>(it, chunk);
    }
    sum = block_sum(sum, red);
    if (threadIdx.x == 0) a.partials[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(1024) k_grad_norm(const double* partials, int n, float* norm) {
    pdl_begin();
    __shared__ double red[32];
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += blockDim.x) s += partials[i];
    s = block_sum(s, red);
    if (threadIdx.x == 0) *norm = (float)sqrt(s);
}

template <int CAP>
__global__ void __launch_bounds__(kGradThreads) k_grad_clip(const __grid_constant__ GradArgs<CAP> a) {
    pdl_begin();
    __shared__ unsigned int start[CAP];
    for (int i = threadIdx.x; i < a.nItems; i += kGradThreads) start[i] = a.items[i].chunk0;
    __syncthreads();
    float factor = a.maxNorm / (*a.norm + 1e-6f);
    factor = factor > 1.0f ? 1.0f : factor;            // a NaN stays
    for (unsigned int c = blockIdx.x; c < a.nChunks; c += gridDim.x) {
        const GradItem& it = a.items[find_item<CAP>(start, a.nItems, c)];
        if (factor == 1.0f && it.in == it.out) continue;
        const unsigned int chunk = c - it.chunk0;
        if (it.dt == kF32) chunk_scale<kF32>(it, chunk, factor);
        else if (it.dt == kF16) chunk_scale<kF16>(it, chunk, factor);
        else chunk_scale<kBF16>(it, chunk, factor);
    }
}

template <int CAP>
cudaError_t launch_grad_squares(const GradArgs<CAP>& a, int grid, cudaStream_t s) {
    return pdl_launch(k_grad_squares<CAP>, (unsigned)grid, kGradThreads, 0, s, a);
}
cudaError_t launch_grad_norm(const double* partials, int n, float* norm, cudaStream_t s) {
    return pdl_launch(k_grad_norm, 1u, 1024u, 0, s, partials, n, norm);
}
template <int CAP>
cudaError_t launch_grad_clip(const GradArgs<CAP>& a, cudaStream_t s) {
    return pdl_launch(k_grad_clip<CAP>, a.nChunks, kGradThreads, 0, s, a);
}
template cudaError_t launch_grad_squares<kGradItemsSmall>(const GradArgs<kGradItemsSmall>&, int, cudaStream_t);
template cudaError_t launch_grad_squares<kGradItemsLarge>(const GradArgs<kGradItemsLarge>&, int, cudaStream_t);
template cudaError_t launch_grad_clip<kGradItemsSmall>(const GradArgs<kGradItemsSmall>&, cudaStream_t);
template cudaError_t launch_grad_clip<kGradItemsLarge>(const GradArgs<kGradItemsLarge>&, cudaStream_t);

}  // namespace vc
