// norm_stage.cuh -- rows staged through shared memory by asynchronous copies, for CTAs that
// stride over many rows.
//
// A thread copies the 16-byte blocks that it will need of the next row (of every input) into
// blocks of shared memory of its own, and reads them back when their turn comes: no thread
// reads another's blocks, so no barrier and no wait but the copies' own is needed.  While one
// row is reduced, scaled and stored, the next one's loads are under way, and they cost no
// registers.  Measured against direct loads (8 x 4096 x 4096 bf16 forward, one CTA per row):
// see the kernels.
#pragma once

#include "norm.cuh"

namespace vc {

__device__ __forceinline__ void copy_block_async(uint32_t smem, const char* p) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(smem), "l"(p) : "memory");
}
// Neighbouring threads copy a block twice where rows are realigned: the second comes from L1.
__device__ __forceinline__ void copy_block_async_l1(uint32_t smem, const char* p) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" :: "r"(smem), "l"(p) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// The shared memory of a thread for one row: block (segment, v) at base + (segment * V + v) *
// pitch, and, where rows are realigned, the block behind it at `second` bytes further.
struct StageAddr {
    uint32_t base, pitch, second;
};

// Start the copies of one input's part of a row.  p: address of the row's element e0 (which
// may lie before the row).
template <int DT, int V, bool GENERAL>
__device__ __forceinline__ void stage_segment(const StageAddr& s, int seg, const char* p, const RowVecs<DT, V>& rv) {
    constexpr int ESZ = DTypeOf<DT>::size;
    const uint32_t at = s.base + (uint32_t)(seg * V) * s.pitch;
    const unsigned sh = GENERAL ? (unsigned)((uintptr_t)p & 15u) : 0u;
#pragma unroll
    for (int v = 0; v < V; v++) {
        if (!rv.on[v]) continue;
        const char* q = p + (ptrdiff_t)v * rv.step * ESZ;
        if (!GENERAL || sh == 0) {
            copy_block_async(at + v * s.pitch, q);
            continue;
        }
        const int inFirst = (int)(16u - sh) / ESZ;
        if (rv.sp[v].lo < inFirst) copy_block_async_l1(at + v * s.pitch, q - sh);
        if (rv.sp[v].hi > inFirst) copy_block_async_l1(at + v * s.pitch + s.second, q - sh + 16);
    }
}
// The vector back from shared memory (elements outside its span are undefined; on aligned rows
// a vector outside the row is zero).
template <int DT, int V, bool GENERAL>
__device__ __forceinline__ uint4 staged(const StageAddr& s, int seg, int v, unsigned sh) {
    const uint32_t at = s.base + (uint32_t)(seg * V + v) * s.pitch;
    if (!GENERAL || sh == 0) return ld_smem(at);
    return shift_bytes(ld_smem(at), ld_smem(at + s.second), sh);
}
// Aligned rows: the vectors of a thread that lie outside every row are never copied, and are
// zero from here on, so that nothing but the stores need ask for them.
template <int DT, int V>
__device__ __forceinline__ void stage_zeros(const StageAddr& s, int segments, const RowVecs<DT, V>& rv) {
#pragma unroll
    for (int v = 0; v < V; v++) {
        if (rv.sp[v].any()) continue;
        for (int seg = 0; seg < segments; seg++)
            st_smem(s.base + (uint32_t)(seg * V + v) * s.pitch, make_uint4(0u, 0u, 0u, 0u));
    }
}

// The weight in shared memory, in its own type: element j at base + j * size.
struct WeightSmem {
    uint32_t base;
    int f32;
};
// Starts the copies (all threads; the caller waits and synchronises).  There is room to read a
// vector that hangs over either end; behind the weight are zeros, up to the last vector of a
// team.
constexpr int kWeightGuard = 32;
__device__ __forceinline__ WeightSmem stage_weight(const void* w, bool f32, int size, int width, uint32_t smem, int bytes) {
    const unsigned sh = (unsigned)((uintptr_t)w & 15u);
    const char* q = (const char*)w - sh;
    const int blocks = (width * size + (int)sh + 15) / 16;
    for (int i = threadIdx.x; i < blocks; i += blockDim.x) copy_block_async(smem + kWeightGuard + i * 16, q + (size_t)i * 16);
    for (int i = blocks + threadIdx.x; i < (bytes - kWeightGuard) / 16; i += blockDim.x)
        st_smem(smem + kWeightGuard + i * 16, make_uint4(0u, 0u, 0u, 0u));
    WeightSmem s;
    s.base = smem + kWeightGuard + sh;
    s.f32 = f32;
    return s;
}
// The weight's values for the vector that starts at element e (undefined outside the row).
template <int DT, bool GENERAL>
__device__ __forceinline__ void weight_vec(const WeightSmem& w, int e, float (&f)[kVecElems<DT>]) {
    constexpr int E = kVecElems<DT>;
    if (DT == kF32 || !w.f32) {
        const uint32_t at = w.base + (uint32_t)(e * DTypeOf<DT>::size);
        const unsigned sh = GENERAL ? at & 15u : 0u;
        widen_vec<DT>(sh == 0 ? ld_smem(at) : shift_bytes(ld_smem(at - sh), ld_smem(at - sh + 16), sh), f);
        return;
    }
    const uint32_t at = w.base + (uint32_t)(e * 4);
    const unsigned sh = GENERAL ? at & 15u : 0u;
    uint4 v[E / 4 + 1];
#pragma unroll
    for (int i = 0; i < E / 4; i++) v[i] = ld_smem(at - sh + 16 * i);
    if (sh != 0) {
        v[E / 4] = ld_smem(at - sh + 16 * (E / 4));
#pragma unroll
        for (int i = 0; i < E / 4; i++) v[i] = shift_bytes(v[i], v[i + 1], sh);
    }
#pragma unroll
    for (int i = 0; i < E / 4; i++) {
        f[4 * i] = __uint_as_float(v[i].x);
        f[4 * i + 1] = __uint_as_float(v[i].y);
        f[4 * i + 2] = __uint_as_float(v[i].z);
        f[4 * i + 3] = __uint_as_float(v[i].w);
    }
}

// One input's part of a row, back from shared memory and added.
template <int DT, int V, bool GENERAL>
__device__ __forceinline__ void add_segment(const StageAddr& s, int seg, unsigned sh, const RowVecs<DT, V>& rv,
                                            float (&acc)[V][kVecElems<DT>]) {
    uint4 raw[V];
#pragma unroll
    for (int v = 0; v < V; v++)
        if (!GENERAL || rv.on[v]) raw[v] = staged<DT, V, GENERAL>(s, seg, v, sh);
#pragma unroll
    for (int v = 0; v < V; v++) {
        float f[kVecElems<DT>];
        widen_vec<DT>(raw[v], f);
        add_to(acc[v], f);
    }
}

}  // namespace vc
