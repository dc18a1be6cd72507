// k_gradnorm.cu -- the global 2-norm of many tensors' gradients, and clipping by it.
//
//   norm = sqrt(sum over all tensors of g^2),  g' = g min(1, maxNorm / (norm + 1e-6))
//
// The tensors are cut into chunks of 32 KiB, listed once in device memory, so one launch
// covers any number of large and small ones and a CTA finds its work with one load.  A thread
// adds the squares of its part of a chunk in fp32 (at most 64 terms) and chunks and threads in
// fp64; the order of every sum follows from the sizes and the tensors' offsets from 16 bytes,
// whichever CTA ends last.
//
// Bound by memory: the norm reads every gradient once (8 x 33.5 M bf16 elements, 537 MB: 78 us,
// 1.01 of the measured copy rate), the clipping reads it again, as the factor depends on all of
// it, and writes it (537 M fp32 elements, 2.1 GB: 917 us, 1.03 of the copy rate on those three
// passes).  Small lists are bound by the chain launch, chunk, data, counter, sums: 5.2 us for
// 0.2 MB.  Eight vectors a thread and four CTAs an SM keep 128 KiB under way per SM; four
// vectors and six CTAs measured 81 us, two CTAs 82 us.
#include "norm.cuh"

namespace vc {

namespace {

__device__ __forceinline__ GradChunk load_chunk(const GradChunk* p) {
    GradChunk c;
    const uint4 lo = *reinterpret_cast<const uint4*>(p);
    const uint2 hi = *reinterpret_cast<const uint2*>(reinterpret_cast<const char*>(p) + 16);
    c.in = (const char*)(((uint64_t)lo.y << 32) | lo.x);
    c.out = (char*)(((uint64_t)lo.w << 32) | lo.z);
    c.count = (int)hi.x;
    c.dt = (int)hi.y;
    return c;
}

// Sum of squares of a thread's part of a chunk.
template <int DT>
__device__ __forceinline__ float chunk_squares(const GradChunk& c) {
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    const int shift = (int)((uintptr_t)c.in & 15u) / ESZ;
    const char* p = c.in - shift * ESZ + (size_t)threadIdx.x * 16;
    const int e0 = (int)threadIdx.x * E - shift;
    uint4 raw[kGradVecs];
#pragma unroll
    for (int i = 0; i < kGradVecs; i++) {
        raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (e0 + i * kGradThreads * E < c.count) raw[i] = ld_once(p + i * kGradThreads * 16);
    }
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kGradVecs; i++) {
        const int e = e0 + i * kGradThreads * E;
        float f[E];
        widen_vec<DT>(raw[i], f);
        if (e < 0 || e + E > c.count) {                // elements of other chunks
#pragma unroll
            for (int j = 0; j < E; j++) f[j] = e + j >= 0 && e + j < c.count ? f[j] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < E; j++) s[j & 3] = fmaf(f[j], f[j], s[j & 3]);
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// Scale a thread's part of a chunk.  A thread's loads are all under way before its first store.
// Gradients and outputs at different offsets from 16 bytes go element by element (134 MB: 134 us,
// 59 at one offset).
template <int DT>
__device__ __forceinline__ void chunk_scale(const GradChunk& c, float factor) {
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    if ((((uintptr_t)c.in ^ (uintptr_t)c.out) & 15u) != 0) {
#pragma unroll 8
        for (int e = threadIdx.x; e < c.count; e += kGradThreads)
            st_elem<ESZ>(c.out, e, f32_to_elem<DT>(elem_to_f32<DT>(ld_elem<ESZ>(c.in, e)) * factor));
        return;
    }
    const int shift = (int)((uintptr_t)c.out & 15u) / ESZ;
    const ptrdiff_t off = (ptrdiff_t)threadIdx.x * 16 - shift * ESZ;
    const int e0 = (int)threadIdx.x * E - shift;
    uint4 raw[kGradVecs];
#pragma unroll
    for (int i = 0; i < kGradVecs; i++)
        if (e0 + i * kGradThreads * E < c.count) raw[i] = ld_once(c.in + off + i * kGradThreads * 16);
#pragma unroll
    for (int i = 0; i < kGradVecs; i++) {
        const int e = e0 + i * kGradThreads * E;
        if (e >= c.count) continue;
        float f[E];
        widen_vec<DT>(raw[i], f);
        scale_by(f, factor);
        if (e >= 0 && e + E <= c.count) {
            st_stream(c.out + off + i * kGradThreads * 16, narrow_vec<DT>(f));
        } else {                                       // the vector that begins or ends the chunk
#pragma unroll
            for (int j = 0; j < E; j++)
                if (e + j >= 0 && e + j < c.count) st_elem<ESZ>(c.out, e + j, f32_to_elem<DT>(f[j]));
        }
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
    for (int o = warps >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return __shfl_sync(~0u, v, 0);
}

}  // namespace

// The CTA that ends last adds all CTAs' sums, so that the norm takes one launch.
__global__ void __launch_bounds__(kGradThreads) k_grad_norm(const __grid_constant__ GradNormArgs a) {
    pdl_begin();
    __shared__ double red[2][32];
    __shared__ bool last;
    double sum = 0.0;
    GradChunk c;
    if (blockIdx.x < a.nChunks) c = load_chunk(a.chunks + blockIdx.x);
    for (unsigned int i = blockIdx.x; i < a.nChunks; i += gridDim.x) {
        GradChunk next = c;
        if (a.nChunks - i > gridDim.x) next = load_chunk(a.chunks + i + gridDim.x);
        if (c.dt == kF32) sum += (double)chunk_squares<kF32>(c);
        else if (c.dt == kF16) sum += (double)chunk_squares<kF16>(c);
        else sum += (double)chunk_squares<kBF16>(c);
        c = next;
    }
    sum = block_sum(sum, red[0]);
    if (threadIdx.x == 0) {
        __stcg(a.partials + blockIdx.x, sum);
        __threadfence();
        last = atomicAdd(a.done, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    double all = 0.0;
    for (unsigned int i = threadIdx.x; i < gridDim.x; i += kGradThreads) all += __ldcg(a.partials + i);
    all = block_sum(all, red[1]);
    if (threadIdx.x == 0) {
        *a.norm = (float)sqrt(all);
        *a.done = 0u;
    }
}

// One chunk a CTA, in order from the last one: the norm has just read those, so up to the size
// of L2 they need not be read from memory again.  No hint keeps them there or lets the outputs go
// first: in place, 34 MB, such hints saved the call 3 us and cost the next kernels 7, whose data
// the kept lines displaced.
__global__ void __launch_bounds__(kGradThreads) k_grad_clip(const __grid_constant__ GradClipArgs a) {
    pdl_begin();
    const GradChunk c = load_chunk(a.chunks + (gridDim.x - 1 - blockIdx.x));
    float factor = a.maxNorm / (*a.norm + 1e-6f);
    factor = factor > 1.0f ? 1.0f : factor;            // a NaN stays
    if (factor == 1.0f && c.in == c.out) return;
    if (c.dt == kF32) chunk_scale<kF32>(c, factor);
    else if (c.dt == kF16) chunk_scale<kF16>(c, factor);
    else chunk_scale<kBF16>(c, factor);
}

cudaError_t launch_grad_norm(const GradNormArgs& a, int grid, cudaStream_t s) {
    return pdl_launch(k_grad_norm, (unsigned)grid, kGradThreads, 0, s, a);
}
cudaError_t launch_grad_clip(const GradClipArgs& a, cudaStream_t s) {
    return pdl_launch(k_grad_clip, a.nChunks, kGradThreads, 0, s, a);
}

}  // namespace vc
