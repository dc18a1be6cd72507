// norm.cuh -- what the RMS norm kernels share: 16-byte vectors of a row wherever the row
// starts, their fp32 values, and the reductions over the threads that share a row.
//
// A row is cut into vectors of E = 16 / elemSize elements.  Vector k covers the elements
// [k E - shift, k E - shift + E), where shift is the row's offset (in elements) from a
// 16-byte boundary in the first output, so that the stores of that output are whole
// aligned vectors but for the first and the last.  Inputs with another offset are cut from
// the two aligned vectors that hold the bytes.  No load leaves the aligned 16-byte blocks
// that hold elements of the row.
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

// Elements of a vector that lie inside its row: [lo, hi).
struct Span {
    int lo, hi;
    __device__ __forceinline__ bool full(int e) const { return lo == 0 && hi == e; }
    __device__ __forceinline__ bool any() const { return lo < hi; }
    __device__ __forceinline__ bool has(int j) const { return j >= lo && j < hi; }
};
template <int E>
__device__ __forceinline__ Span span_of(int e0, int width) {
    Span s;
    s.lo = e0 < 0 ? -e0 : 0;
    s.hi = width - e0 < E ? width - e0 : E;
    return s;
}

// A thread's vectors of one row.
template <int DT, int V>
struct RowVecs {
    static constexpr int E = kVecElems<DT>;
    static constexpr int ESZ = DTypeOf<DT>::size;
    int e0, step;                    // first element of vector 0, elements between vectors
    Span sp[V];
    bool on[V];                      // the vector holds elements of a row that exists
    __device__ __forceinline__ void set(int e0_, int step_, int width, bool live) {
        e0 = e0_;
        step = step_;
#pragma unroll
        for (int v = 0; v < V; v++) {
            sp[v] = span_of<E>(e0 + v * step, width);
            on[v] = live && sp[v].any();
        }
    }
    // Zero what lies outside the row (all of a vector that is not on).
    __device__ __forceinline__ void mask(float (&f)[V][E]) const {
#pragma unroll
        for (int v = 0; v < V; v++) {
            if (sp[v].full(E)) continue;
#pragma unroll
            for (int j = 0; j < E; j++) f[v][j] = sp[v].has(j) ? f[v][j] : 0.0f;
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

// The 16 bytes at p (any element-aligned address).  GENERAL false: p is 16-byte aligned and
// the whole vector lies in the row.  Elements outside the span come back undefined.
template <int ESZ, bool GENERAL>
__device__ __forceinline__ uint4 load_vec(const char* p, Span sp) {
    if (!GENERAL) return ld_once(p);
    const unsigned sh = (unsigned)((uintptr_t)p & 15u);
    const char* q = p - sh;
    if (sh == 0) return ld_once(q);
    const int inFirst = (int)(16u - sh) / ESZ;         // elements that the first block holds
    uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
    if (sp.lo < inFirst) a = *reinterpret_cast<const uint4*>(q);
    if (sp.hi > inFirst) b = *reinterpret_cast<const uint4*>(q + 16);
    return shift_bytes(a, b, sh);
}

// Store the span of a vector at p: whole and aligned in one access, else by element.
template <int DT, bool GENERAL>
__device__ __forceinline__ void store_vec(char* p, Span sp, const float (&f)[kVecElems<DT>]) {
    constexpr int E = kVecElems<DT>;
    const uint4 v = narrow_vec<DT>(f);
    if (!GENERAL || (sp.full(E) && ((uintptr_t)p & 15u) == 0)) {
        st_stream(p, v);
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < E; j++) {
        if (!sp.has(j)) continue;
        if (DT == kF32) *(uint32_t*)(p + 4 * j) = w[j & 3];
        else *(uint16_t*)(p + 2 * j) = (uint16_t)(w[(j >> 1) & 3] >> (16 * (j & 1)));
    }
}

// The weight's E values for the elements [e0, e0 + E) of a row, in its own type.
template <int DT>
struct WeightVec {
    static constexpr int E = kVecElems<DT>;
    uint4 raw[E / 4];                // E fp32 values, or one vector of the data's type
    template <bool GENERAL>
    __device__ __forceinline__ void load(const void* w, bool f32, int e0, Span sp) {
        if (DT == kF32 || !f32) {
            raw[0] = load_weight<DTypeOf<DT>::size, GENERAL>((const char*)w + (ptrdiff_t)e0 * DTypeOf<DT>::size, sp);
        } else {
#pragma unroll
            for (int i = 0; i < E / 4; i++) {
                Span part;
                part.lo = sp.lo - 4 * i < 0 ? 0 : sp.lo - 4 * i;
                part.hi = sp.hi - 4 * i > 4 ? 4 : sp.hi - 4 * i;
                raw[i] = make_uint4(0u, 0u, 0u, 0u);
                if (!GENERAL || part.any())
                    raw[i] = load_weight<4, GENERAL>((const char*)w + ((ptrdiff_t)e0 + 4 * i) * 4, part);
            }
        }
    }
    __device__ __forceinline__ void get(bool f32, float (&f)[E]) const {
        if (DT == kF32 || !f32) {
            widen_vec<DT>(raw[0], f);
        } else {
#pragma unroll
            for (int i = 0; i < E / 4; i++) {
                f[4 * i] = __uint_as_float(raw[i].x);
                f[4 * i + 1] = __uint_as_float(raw[i].y);
                f[4 * i + 2] = __uint_as_float(raw[i].z);
                f[4 * i + 3] = __uint_as_float(raw[i].w);
            }
        }
    }

private:
    // Every row reads the weight, so it goes through L1, unlike the streamed buffers.
    template <int ESZ, bool GENERAL>
    static __device__ __forceinline__ uint4 load_weight(const char* p, Span sp) {
        if (!GENERAL) return ld_shared_by_rows(p);
        const unsigned sh = (unsigned)((uintptr_t)p & 15u);
        const char* q = p - sh;
        if (sh == 0) return ld_shared_by_rows(q);
        const int inFirst = (int)(16u - sh) / ESZ;
        uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
        if (sp.lo < inFirst) a = ld_shared_by_rows(q);
        if (sp.hi > inFirst) b = ld_shared_by_rows(q + 16);
        return shift_bytes(a, b, sh);
    }
};

// Sum over the ranks, in rank order and in fp32, of one row's vectors of a thread.  UN ranks'
// loads are in flight before the first is added.
template <int DT, int V, bool GENERAL>
__device__ __forceinline__ void sum_ranks(const void* const* send, int N, ptrdiff_t off, const RowVecs<DT, V>& rv,
                                          float (&acc)[V][kVecElems<DT>]) {
    constexpr int E = kVecElems<DT>;
    constexpr int ESZ = DTypeOf<DT>::size;
    constexpr int UN = GENERAL ? (V == 1 ? 4 : 2) : 8 / V;
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
                for (int v = 0; v < V; v++)
                    if (rv.on[v]) raw[i][v] = load_vec<ESZ, GENERAL>(p + (ptrdiff_t)v * rv.step * ESZ, rv.sp[v]);
            }
        }
#pragma unroll
        for (int i = 0; i < UN; i++) {
            if (r + i < N) {
#pragma unroll
                for (int v = 0; v < V; v++) {
                    if (rv.on[v]) {
                        float f[E];
                        widen_vec<DT>(raw[i][v], f);
                        add_to(acc[v], f);
                    }
                }
            }
        }
    }
}

// ---- outputs that start at another offset from 16 bytes than the row's vectors -------------

__device__ __forceinline__ uint4 ld_smem(uint32_t p) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_smem(uint32_t p, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" :: "r"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// `bytes` bytes at shared address `src` (any alignment) to dst, by a team of `threads`: whole
// aligned 16-byte blocks, each cut from the two that hold it, and the ends in OSZ-byte elements.
// Element stores alone would take 8 (16 for bytes) per vector; measured on 3 x 1537 x 2731 fp16
// with every rank at its own offset, they made 41 us of a pass that takes FINAL_RAGGED.
template <int OSZ>
__device__ __forceinline__ void copy_out(char* dst, uint32_t src, int bytes, int t, int threads) {
    const int head = min((int)((16u - (unsigned)((uintptr_t)dst & 15u)) & 15u), bytes);
    const int blocks = (bytes - head) >> 4;
    const unsigned sh = (src + head) & 15u;
    const uint32_t from = src + head - sh;
    for (int i = t; i < blocks; i += threads) {
        const uint4 a = ld_smem(from + 16 * i);
        st_stream(dst + head + (size_t)i * 16, sh == 0 ? a : shift_bytes(a, ld_smem(from + 16 * i + 16), sh));
    }
    const int tail = head + blocks * 16;
    for (int k = t * OSZ; k < head + bytes - tail; k += threads * OSZ) {
        const int at = k < head ? k : tail + k - head;
        if (OSZ == 1) {
            uint32_t v;
            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(src + at) : "memory");
            *(uint8_t*)(dst + at) = (uint8_t)v;
        } else if (OSZ == 2) {
            uint16_t v;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(src + at) : "memory");
            *(uint16_t*)(dst + at) = v;
        } else {
            uint32_t v;
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(src + at) : "memory");
            *(uint32_t*)(dst + at) = v;
        }
    }
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

// Let a kernel use `bytes` of dynamic shared memory.
template <typename K>
inline cudaError_t allow_smem(K kernel, size_t bytes) {
    if (bytes <= 32 * 1024) return cudaSuccess;        // with the static arrays, below the default 48 KiB
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
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
