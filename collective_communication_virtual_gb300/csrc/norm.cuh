// norm.cuh -- what the RMS norm kernels share: 16-byte vectors of a row wherever the row
// starts, their fp32 values, and the reductions over the threads that share a row.
//
// A row is cut into vectors of E = 16 / elemSize elements from its first element on, so a
// thread holds the same columns of every row.  GENERAL kernels serve rows that start off a
// 16-byte boundary or end inside a vector: inputs are cut from the two aligned blocks that
// hold a vector's bytes, outputs leave through a row buffer in shared memory as whole aligned
// blocks.  No load leaves the aligned 16-byte blocks that hold elements of the row.
#pragma once

#include <cuda_fp8.h>

#include "device.cuh"
#include "operators.h"

namespace vc {

template <int DT> constexpr int kVecElems = 16 / DTypeOf<DT>::size;

template <int DT>
__device__ __forceinline__ void widen_vec(const uint4& v, float (&f)[kVecElems<DT>]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if (DT == kF32) {
            f[i] = __uint_as_float(w[i]);
        } else if (DT == kBF16) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = p.x;
            f[2 * i + 1] = p.y;
        }
    }
}

// Rounded to the storage type (to nearest even), the only rounding of a 16-bit output.
template <int DT>
__device__ __forceinline__ uint4 narrow_vec(const float (&f)[kVecElems<DT>]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if (DT == kF32) {
            w[i] = __float_as_uint(f[i]);
        } else if (DT == kBF16) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&p);
        } else {
            const __half2 p = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A thread's vectors of a row: columns [e0 + v step, e0 + v step + E).
template <int DT, int V>
struct RowVecs {
    static constexpr int E = kVecElems<DT>;
    int e0, step;
    int left[V];                     // elements of vector v inside the row: E for a whole one
    bool last[V];                    // the row has no vector behind it
    __device__ __forceinline__ RowVecs(int first, int stride, int width) : e0(first), step(stride) {
#pragma unroll
        for (int v = 0; v < V; v++) {
            left[v] = max(0, min(E, width - (e0 + v * step)));
            last[v] = e0 + v * step + E >= width;
        }
    }
    // Zero what lies behind the row's end.
    __device__ __forceinline__ void mask(float (&f)[V][E]) const {
#pragma unroll
        for (int v = 0; v < V; v++) {
            if (left[v] == E) continue;
#pragma unroll
            for (int j = 0; j < E; j++) f[v][j] = j < left[v] ? f[v][j] : 0.0f;
        }
    }
};

// Two fp32 additions, products or fused steps in one instruction (each rounded as the single
// ones are).
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
// max(a, |b|, |c|), where a NaN wins.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
    return r;
}
template <int E>
__device__ __forceinline__ void add_to(float (&acc)[E], const float (&f)[E]) {
#pragma unroll
    for (int j = 0; j < E; j += 2) {
        const float2 s = add2(make_float2(acc[j], acc[j + 1]), make_float2(f[j], f[j + 1]));
        acc[j] = s.x;
        acc[j + 1] = s.y;
    }
}
template <int E>
__device__ __forceinline__ void scale_by(float (&acc)[E], float k) {
#pragma unroll
    for (int j = 0; j < E; j += 2) {
        const float2 s = mul2(make_float2(acc[j], acc[j + 1]), make_float2(k, k));
        acc[j] = s.x;
        acc[j + 1] = s.y;
    }
}
template <int E>
__device__ __forceinline__ void mul_by(float (&acc)[E], const float (&f)[E]) {
#pragma unroll
    for (int j = 0; j < E; j += 2) {
        const float2 s = mul2(make_float2(acc[j], acc[j + 1]), make_float2(f[j], f[j + 1]));
        acc[j] = s.x;
        acc[j + 1] = s.y;
    }
}

// Bytes [4 W + r / 8, + 16) of the 32 bytes a, b, for r in 0..24 bits.
template <int W>
__device__ __forceinline__ uint4 shift_words(const uint4& a, const uint4& b, unsigned r) {
    const uint32_t w[9] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, 0u};
    return make_uint4(__funnelshift_r(w[W], w[W + 1], r), __funnelshift_r(w[W + 1], w[W + 2], r),
                      __funnelshift_r(w[W + 2], w[W + 3], r), __funnelshift_r(w[W + 3], w[W + 4], r));
}
// f(shift) with shift(a, b) = bytes [sh, sh + 16) of a, b: one branch for any number of vectors.
template <typename F>
__device__ __forceinline__ void with_shift(unsigned sh, F f) {
    const unsigned r = (sh & 3u) * 8u;
    switch (sh >> 2) {
    case 0: f([r](const uint4& a, const uint4& b) { return shift_words<0>(a, b, r); }); break;
    case 1: f([r](const uint4& a, const uint4& b) { return shift_words<1>(a, b, r); }); break;
    case 2: f([r](const uint4& a, const uint4& b) { return shift_words<2>(a, b, r); }); break;
    default: f([r](const uint4& a, const uint4& b) { return shift_words<3>(a, b, r); }); break;
    }
}

// Streamed once, so kept out of L1.  volatile: never moved above the wait for the previous
// kernel, nor merged with another load of the address.
__device__ __forceinline__ uint4 ld_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// Read by every row, so through L1.  Not by the read-only path: the kernel may become resident
// while the previous one still writes what it reads.
__device__ __forceinline__ uint4 ld_shared_by_rows(const void* p) { return *reinterpret_cast<const uint4*>(p); }

// The 16 bytes at p, of which the first `left` elements are wanted (at least one).  GENERAL
// false: p is 16-byte aligned.  The other elements come back undefined.
template <int ESZ, bool GENERAL, bool ONCE = true>
__device__ __forceinline__ uint4 load_vec(const char* p, int left) {
    const auto ld = [](const char* q) { return ONCE ? ld_once(q) : ld_shared_by_rows(q); };
    if (!GENERAL) return ld(p);
    const unsigned sh = (unsigned)((uintptr_t)p & 15u);
    if (sh == 0) return ld(p);
    const uint4 a = ld(p - sh);
    uint4 b = make_uint4(0u, 0u, 0u, 0u);
    if (left > (int)(16u - sh) / ESZ) b = ld(p - sh + 16);
    return shift_bytes(a, b, sh);
}

// The weight's E values from element e on (`left` of them inside the row).
template <int DT, bool GENERAL>
__device__ __forceinline__ void load_weight(const void* w, bool f32, int e, int left, float (&f)[kVecElems<DT>]) {
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    if constexpr (DT != kF32) {
        if (f32) {
#pragma unroll
            for (int i = 0; i < E; i += 4) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (left > i) v = load_vec<4, GENERAL, false>((const char*)w + (size_t)(e + i) * 4, left - i);
                f[i] = __uint_as_float(v.x);
                f[i + 1] = __uint_as_float(v.y);
                f[i + 2] = __uint_as_float(v.z);
                f[i + 3] = __uint_as_float(v.w);
            }
            return;
        }
    }
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (left > 0) v = load_vec<ESZ, GENERAL, false>((const char*)w + (size_t)e * ESZ, left);
    widen_vec<DT>(v, f);
}

// Sum over the ranks, in rank order and in fp32, of one row's vectors of a thread.  UN ranks'
// loads are in flight before the first is added.
template <int DT, int V, bool GENERAL>
__device__ __forceinline__ void sum_ranks(const void* const* send, int N, size_t off, bool live, const RowVecs<DT, V>& rv,
                                          float (&acc)[V][kVecElems<DT>]) {
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    constexpr int UN = GENERAL ? (V == 1 ? 4 : V == 2 ? 2 : 1) : 8 / V;
#pragma unroll
    for (int v = 0; v < V; v++)
#pragma unroll
        for (int j = 0; j < E; j++) acc[v][j] = 0.0f;
    for (int r = 0; r < N; r += UN) {
        uint4 raw[UN][V];
#pragma unroll
        for (int i = 0; i < UN; i++) {
            if (r + i < N) {
                const char* p = (const char*)send[r + i] + off;
#pragma unroll
                for (int v = 0; v < V; v++) {
                    raw[i][v] = make_uint4(0u, 0u, 0u, 0u);
                    if (live && rv.left[v] > 0)
                        raw[i][v] = load_vec<ESZ, GENERAL>(p + (size_t)v * rv.step * ESZ, rv.left[v]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < UN; i++) {
            if (r + i < N) {
#pragma unroll
                for (int v = 0; v < V; v++) {
                    float f[E];
                    widen_vec<DT>(raw[i][v], f);
                    add_to(acc[v], f);
                }
            }
        }
    }
}

// ---- outputs ---------------------------------------------------------------------------------

__device__ __forceinline__ uint4 ld_smem(uint32_t p) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_smem(uint32_t p, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" :: "r"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// `bytes` bytes at the 16-byte aligned shared address `src` to dst (any alignment), by a team of
// `threads`: whole aligned blocks of dst, each cut from the two of src that hold it, and the
// ends in OSZ-byte elements.
template <int OSZ>
__device__ __forceinline__ void copy_out(char* dst, uint32_t src, int bytes, int t, int threads) {
    const unsigned sh = (16u - (unsigned)((uintptr_t)dst & 15u)) & 15u;    // bytes before the first block
    const int blocks = (bytes - (int)sh) >> 4;
    if (sh == 0) {
        for (int i = t; i < blocks; i += threads) st_stream(dst + (size_t)i * 16, ld_smem(src + 16 * i));
    } else {
        with_shift(sh, [&](auto shift) {
#pragma unroll 2
            for (int i = t; i < blocks; i += threads)
                st_stream(dst + sh + (size_t)i * 16, shift(ld_smem(src + 16 * i), ld_smem(src + 16 * i + 16)));
        });
    }
    const int head = min((int)sh, bytes), tail = head + max(blocks, 0) * 16;
    for (int k = t * OSZ; k < head + bytes - tail; k += threads * OSZ) {
        const int at = k < head ? k : tail + k - head;
        uint32_t v;
        if (OSZ == 1) {
            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(src + at) : "memory");
            *(uint8_t*)(dst + at) = (uint8_t)v;
        } else if (OSZ == 2) {
            asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(src + at) : "memory");
            *(uint16_t*)(dst + at) = (uint16_t)v;
        } else {
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(src + at) : "memory");
            *(uint32_t*)(dst + at) = v;
        }
    }
}

// The same to n >= 2 outputs that all lie at one offset from 16 bytes: each block is cut once
// (8 x 2000 x 4097: 60 us, 66 one output at a time).
template <int OSZ>
__device__ __forceinline__ void copy_out_same(void* const* dst, int n, size_t off, uint32_t src, int bytes, int t, int threads) {
    const unsigned sh = (16u - (unsigned)(((uintptr_t)dst[0] + off) & 15u)) & 15u;
    const int blocks = (bytes - (int)sh) >> 4;
    for (int i = t; i < blocks; i += threads) {
        uint4 v = ld_smem(src + 16 * i);
        if (sh != 0) v = shift_bytes(v, ld_smem(src + 16 * i + 16), sh);
        for (int o = 0; o < n; o++) st_stream((char*)dst[o] + off + sh + (size_t)i * 16, v);
    }
    const int head = min((int)sh, bytes), tail = head + max(blocks, 0) * 16;
    for (int k = t * OSZ; k < head + bytes - tail; k += threads * OSZ) {
        const int at = k < head ? k : tail + k - head;
        uint32_t v;
        if (OSZ == 1) asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(src + at) : "memory");
        else if (OSZ == 2) asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(src + at) : "memory");
        else asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(src + at) : "memory");
        for (int o = 0; o < n; o++) {
            char* p = (char*)dst[o] + off + at;
            if (OSZ == 1) *(uint8_t*)p = (uint8_t)v;
            else if (OSZ == 2) *(uint16_t*)p = (uint16_t)v;
            else *(uint32_t*)p = v;
        }
    }
}
template <int OSZ>
__device__ __forceinline__ void copy_out_all(void* const* dst, int n, bool same, size_t off, uint32_t src, int bytes, int t,
                                             int threads) {
    if (same && n > 1) {
        copy_out_same<OSZ>(dst, n, off, src, bytes, t, threads);
        return;
    }
    for (int o = 0; o < n; o++) copy_out<OSZ>((char*)dst[o] + off, src, bytes, t, threads);
}

// ---- reductions over a team ---------------------------------------------------------------

__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Store a word at the address that `local` has here in the shared memory of CTA `rank`.
__device__ __forceinline__ void st_cluster(const void* local, unsigned rank, uint32_t v) {
    uint32_t a = (uint32_t)__cvta_generic_to_shared(local), r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    asm volatile("st.shared::cluster.u32 [%0], %1;" :: "r"(r), "r"(v) : "memory");
}

// Sum of `s` and, with MAX, the maximum of `m` (not negative; a NaN wins) over the threads of a team.  The
// order of the additions depends on the shape alone.  All threads of the CTA call it; on a
// cluster, cluster_arrive() has been called once before.  The words of `red` are not reused
// by the same CTA before another barrier of it has passed.
struct TeamScratch {
    float sum[32];
    float max[32];
    float clusterSum[kNormMaxCluster];
    float clusterMax[kNormMaxCluster];
};
template <bool MAX>
__device__ __forceinline__ void team_reduce(TeamScratch& red, const NormShape& sh, float& s, float& m) {
    const int lanes = sh.teamThreads < 32 ? sh.teamThreads : 32;
    for (int o = lanes >> 1; o > 0; o >>= 1) {
        s += __shfl_xor_sync(~0u, s, o);
        if (MAX) m = max_abs(m, __shfl_xor_sync(~0u, m, o), 0.0f);
    }
    if (sh.teamThreads <= 32) return;
    const int warps = (int)blockDim.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
        red.sum[threadIdx.x >> 5] = s;
        if (MAX) red.max[threadIdx.x >> 5] = m;
    }
    __syncthreads();
    s = lane < warps ? red.sum[lane] : 0.0f;
    if (MAX) m = lane < warps ? red.max[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(~0u, s, o);
        if (MAX) m = max_abs(m, __shfl_xor_sync(~0u, m, o), 0.0f);
    }
    if (sh.cluster == 1) return;
    cluster_wait();                  // every CTA of the cluster has started
    if (threadIdx.x < (unsigned)sh.cluster) {
        const unsigned me = cluster_rank();
        st_cluster(&red.clusterSum[me], threadIdx.x, __float_as_uint(s));
        if (MAX) st_cluster(&red.clusterMax[me], threadIdx.x, __float_as_uint(m));
    }
    cluster_arrive();
    cluster_wait();
    s = 0.0f;
    for (int c = 0; c < sh.cluster; c++) {
        s += red.clusterSum[c];
        if (MAX) m = max_abs(m, red.clusterMax[c], 0.0f);
    }
}

// Let a kernel use `bytes` of dynamic shared memory.  The limit belongs to the kernel, not to the
// launch, and host threads share it: it is set to one value, the most that any shape takes, so that
// no thread lowers it between another's setting and launch.
static_assert(2 * sizeof(TeamScratch) <= kNormStaticSmem, "the kernels' static arrays");
template <typename K>
inline cudaError_t allow_smem(K kernel, size_t bytes) {
    if (bytes <= 32 * 1024) return cudaSuccess;        // with the static arrays, below the default 48 KiB
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormMaxSmem);
}

template <typename K, typename... Args>
inline cudaError_t norm_launch(K kernel, unsigned grid, const NormShape& sh, size_t smem, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((unsigned)sh.threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (pdl_enabled()) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (sh.cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)sh.cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = (unsigned)n;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace vc
